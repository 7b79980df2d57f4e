"""The attention side of a serving step at the edges of its range: magnitudes of
queries and scales, calls whose arguments or device data do not fit together.
References and tolerances are those of test_attention.py.
"""
import numpy as np
import pytest

from test_attention import (PATHS, Case, L, _run_step, _step_case, _torch, ref_attend,  # noqa: F401  (L: a fixture)
                            ref_step)

gpu = pytest.mark.gpu
SLOPES = [2.0 ** -(h + 1) for h in range(4)]


# ---------------------------------------------------------------------------
# Scores far from 1
# ---------------------------------------------------------------------------
@gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("kw", [dict(slopes=SLOPES), dict(softcap=30.0), dict(softcap=30.0, slopes=SLOPES),
                                dict(softcap=1e-5), dict(softcap=1e6), dict(softcap=3e38)], ids=str)
@pytest.mark.parametrize("power", [90, 70, 40, 20, 0, -20, -40, -90])
def test_scores_at_query_magnitudes(L, power, kw, path, fp8):  # noqa: F811
    """Queries times a power of two and the scale divided by it: scores, biases and
    caps stay what they were, in tiles that a mask cuts and in tiles that none does."""
    c = Case(L, [700, 150], [2, 60], 4, 2, 64, seed=14, fp8=fp8)
    c.q_big.mul_(2.0 ** power)
    scale = 64 ** -0.5 * 2.0 ** -power
    c.run(path, scale=scale, **kw).check(path, scale=scale, **kw)


@gpu
@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("kw", [dict(scale=-0.125), dict(scale=-0.125, slopes=SLOPES), dict(scale=-0.125, softcap=4.0),
                                dict(scale=0.0, softcap=4.0, slopes=SLOPES)], ids=str)
def test_scale_not_positive(L, kw, path):  # noqa: F811
    c = Case(L, [700, 150], [2, 60], 4, 2, 128, seed=15)
    c.run(path, **kw).check(path, **kw)


@gpu
@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("kw", [dict(), dict(slopes=SLOPES), dict(softcap=20.0), dict(softcap=20.0, slopes=SLOPES)],
                         ids=str)
def test_score_of_minus_infinity(L, kw, path):  # noqa: F811
    """A key with an infinity whose score is -inf has weight 0 (under a cap: the cap's
    weight), in a tile that no mask cuts; everything else is as without it."""
    torch = _torch()
    c = Case(L, [700], [60 if path == "prompt" else 2], 4, 2, 64, seed=16)
    heads = c.q_big[:, 8:8 + 4 * 64].view(c.T, 4, 64)
    heads[:, :, 0] = heads[:, :, 0].abs() + 0.5
    c.kv.k[c.table[0, 0].item(), 5, :, 0] = float("-inf")
    c.run(path, **kw)
    assert c.att.err.item() == 0
    q = c.q.double().cpu().numpy().reshape(c.T, 4, 64)
    got = c.out.double().cpu().numpy().reshape(c.T, 4, 64)
    slopes, cap = kw.get("slopes"), kw.get("softcap", 0.0)
    big = ref_attend(q, c.k[0], c.v[0], 64 ** -0.5, cap, 0, slopes, 700)[3]  # the other keys' largest score
    c.k[0][5, :, 0] = -np.inf
    ref, lse, size, _ = ref_attend(q, c.k[0], c.v[0], 64 ** -0.5, cap, 0, slopes, 700)
    weights = 2.0 ** -8 if path == "prompt" else 2.0 ** -11
    tol = 2.0 ** -8 * np.abs(ref) + (weights * 1.01 + 2.0 ** -18 * (1 + max(big.max(), cap))) * size
    assert (np.abs(got - ref) <= tol).all()
    assert (np.abs(c.lse.double().cpu().numpy() - lse) <= 2.0 ** -18 * (1 + big)).all()
    assert torch.isfinite(c.out).all()


# ---------------------------------------------------------------------------
# Steps with more tokens than rows
# ---------------------------------------------------------------------------
@gpu
@pytest.mark.parametrize("n,ps,ctx_hi,new_hi,part", [
    (1, 16, 40, 4000, 0.0), (1, 16, 40, 4000, 0.3), (1, 1, 9, 3000, 0.5), (37, 16, 200, 60, 0.5), (37, 128, 500, 300, 0.9),
    (1500, 16, 50, 40, 0.02), (1500, 16, 50, 40, 0.6), (2100, 64, 10, 200, 0.999), (5, 1024, 5000, 3000, 0.2)])
@pytest.mark.parametrize("short", [False, True])
def test_step_tables_of_tokens_past_the_rows(L, n, ps, ctx_hi, new_hi, part, short):  # noqa: F811
    """The tokens past T are dropped; the table holds all pages of the requests that were
    served, as `taken` and kv_lens count them."""
    torch = _torch()
    ctx, new, table, free = _step_case(3 * n + ps, n, ps, ctx_hi, new_hi, zero=0.1 if n > 1 else 0.0)
    T = int(part * sum(new))
    if short:
        free = free[:2 * len(free) // 3]
    st = _run_step(L, ctx, new, ps, free, table, T, ld_pad=2)
    q_off, kv, pos, seq, slots, taken, want, errors = ref_step(ctx, new, ps, free, table, T)
    assert sum(new) > T and st.err.item() in errors
    assert torch.equal(st.block_table.cpu(), torch.tensor(want, dtype=torch.int32))
    assert st.taken.item() == taken and st.kv_lens.tolist() == kv and st.q_offsets.tolist() == q_off
    assert (st.positions.tolist(), st.seq_ids.tolist(), st.slot_map.tolist()) == (pos, seq, slots)


# ---------------------------------------------------------------------------
# What the binding hands over (host tensors that say they are on the device, and a
# library that only records)
# ---------------------------------------------------------------------------
class OnDevice:
    """Wraps a host tensor for the binding's checks; no kernel sees it."""

    def __new__(cls, t):
        torch = _torch()
        kind = type("OnDeviceTensor", (torch.Tensor,), {"is_cuda": True})
        return t.as_subclass(kind)


@pytest.fixture
def recorded(L, monkeypatch):  # noqa: F811
    calls = []

    class Library:
        def __getattr__(self, name):
            return lambda *args: calls.append((name, args)) or 0
    from rank_adapter_gemm_gb300 import attention
    attention._types()
    monkeypatch.setattr(attention, "load", Library)
    monkeypatch.setattr(attention, "_on", lambda stream: 0)
    return calls


def _attend_args(table, n, T=4, width=2 * 16):
    from rank_adapter_gemm_gb300._lib import lora_attention_t, lora_kv_t
    torch = _torch()
    q, out = (OnDevice(torch.zeros(T, width, dtype=torch.bfloat16)) for _ in range(2))
    off, lens = (OnDevice(torch.zeros(m, dtype=torch.int32)) for m in (n + 1, n))
    kv = lora_kv_t(1 << 20, 1 << 21, 8, 16, 1, 16, 256, 16, 16, 0, 1.0, 1.0)
    ws = OnDevice(torch.zeros(64, dtype=torch.uint8))
    return dict(q=q, out=out, q_offsets=off, kv_lens=lens, block_table=table, kv=kv,
                att=lora_attention_t(2, 0.1, 0.0, 0, None), ws=ws, err=None)


def _tables():
    torch = _torch()
    row = torch.arange(6, dtype=torch.int32)
    return {"shared": row.expand(4, 6), "overlapping": torch.arange(20, dtype=torch.int32).as_strided((4, 6), (3, 1)),
            "one a request": torch.zeros(4, 6, dtype=torch.int32), "part of wider rows": torch.zeros(
                4, 9, dtype=torch.int32)[:, :6], "a single expanded row": row.expand(1, 6)}


@pytest.mark.parametrize("name,ld", [("shared", None), ("overlapping", None), ("one a request", 6),
                                     ("part of wider rows", 9), ("a single expanded row", 6)])
def test_tables_whose_rows_overlap_are_refused(L, recorded, name, ld):  # noqa: F811
    """A row stride below the width is not replaced by the width: the kernels would read,
    and the step tables write, past such a table's memory."""
    torch = _torch()
    t = OnDevice(_tables()[name])
    n = t.shape[0]
    step = L.KVStep(n, 8, 6, 16, device="cpu")
    step.block_table = t
    i = OnDevice(torch.zeros(n, dtype=torch.int32))
    if ld is None:
        with pytest.raises(ValueError):
            L.lora_attend(**_attend_args(t, n))
        with pytest.raises(ValueError):
            step.build(i, i, i)
        assert not recorded
    else:
        L.lora_attend(**_attend_args(t, n))
        step.build(i, i, i)
        (_, a), (_, b) = recorded
        assert (a[10], a[11]) == (ld, 6) and (b[7], b[8]) == (ld, 6)


def test_workspaces_off_the_device_are_refused(L, recorded):  # noqa: F811
    torch = _torch()
    table = OnDevice(torch.zeros(4, 6, dtype=torch.int32))
    kw = _attend_args(table, 4)
    with pytest.raises(TypeError):
        L.lora_attend(**dict(kw, ws=torch.zeros(1 << 20, dtype=torch.uint8)))
    with pytest.raises(ValueError):
        L.lora_attend(**dict(kw, ws=OnDevice(torch.zeros(1 << 10, dtype=torch.uint8))[::2]))
    assert not recorded
    L.lora_attend(**kw)
    assert len(recorded) == 1


# ---------------------------------------------------------------------------
# Offsets out of order
# ---------------------------------------------------------------------------
@gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("n", [3, 31, 39])
def test_offsets_that_go_back(L, n, path, fp8):  # noqa: F811
    """[0, T, 0, T, ...]: every other request ends before it begins and is skipped, the rest
    all own the same rows: more work than T rows stand for.  They are alike here, so their
    rows come out whole whoever writes them, and the workspace stays usable."""
    torch = _torch()
    T = 1000 if path == "prompt" else 10
    c = Case(L, [1000], [T], 4, 1, 64, seed=17, fp8=fp8)
    c.run(path)
    att = L.Attention(n, T, 4, c.kv)
    off = torch.tensor([0, T] * ((n + 1) // 2), dtype=torch.int32, device="cuda")
    lens, table = c.lens_dev.repeat(n), c.table.repeat(n, 1)
    c.out.fill_(float("nan"))
    att.run(c.q, c.out, off, lens, table, T, path=path, lse=c.lse)
    torch.cuda.synchronize()
    assert att.err.item() == 1
    # the rows that this call wrote
    q, got = (t.double().cpu().numpy().reshape(T, 4, 64) for t in (c.q, c.out))
    ref, lse, size, big = ref_attend(q, c.k[0], c.v[0], 64 ** -0.5, 0.0, 0, None, 1000)
    weights = 2.0 ** -8 if path == "prompt" else 2.0 ** -11
    tol = 2.0 ** -8 * np.abs(ref) + (weights * 1.01 + 2.0 ** -18 * (1 + big[..., None])) * size
    assert (np.abs(got - ref) <= tol).all()
    assert (np.abs(c.lse.double().cpu().numpy() - lse) <= 2.0 ** -18 * (1 + big)).all()
    c.out.fill_(float("nan"))
    c.att.ws = att.ws  # a call in the other's workspace gives what the first one did
    c.att.run(c.q, c.out, c.off, c.lens_dev, c.table, T, path=path, lse=c.lse)
    c.check(path)


# ---------------------------------------------------------------------------
# Waits that give up (by reading: a stalled block is not run)
# ---------------------------------------------------------------------------
def _prompt_source():
    import os
    import re
    here = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(here, "rank_adapter_gemm_gb300", "csrc", "attend_prompt.cu")).read()
    return re.sub(r"//[^\n]*", "", text)


def test_waits_that_give_up_take_the_whole_warp():
    """A wait's outcome is a lane's own: the phase, the stop flag and the clock are read lane
    by lane.  It may steer a warp only through a vote of all its lanes, as what follows
    (votes, shuffles, elections, tensor-memory loads) wants the whole warp."""
    import re
    text = _prompt_source()
    kernel = text[text.index("attend_prompt_kernel(const AttendArgs a"):]
    # one form votes at once, the other is a helper that returns nothing and stops the block's
    # other waits ...
    voted = "__all_sync(0xffffffffu, tc::mbar_wait("
    assert text.count("tc::mbar_wait(") == 2 and text.count(voted) == 1
    at = text.replace(voted, "".ljust(len(voted))).index("tc::mbar_wait(")
    helper = text[text.rindex("const auto", 0, at):]
    helper = helper[:helper.index("};")]
    name = re.match(r"const auto (\w+)", helper)[1]
    assert "return" not in helper and "break" not in helper and "s_abort = 1;" in helper
    # ... which is called as a statement, in a condition's body at most, also through a shorthand
    shorthands = re.findall(r"const auto (\w+) = \[&\]\([^)]*\) \{ %s\([^;{}]*\); \};" % name, text)
    for h in [name] + shorthands:
        for m in re.finditer(r"[^\n]*\b%s\(&?[^\n]*" % h, text):
            line = m[0].strip()
            assert re.match(r"(const auto \w+ = .*|%s\(.*\);|if \((?:(?!%s).)*\) %s\(.*\);)$" % (h, h, h), line), line
    # what the lanes remember is asked for by votes alone
    for m in re.finditer(r"[^\n]*\bfine\b[^\n]*", kernel):
        line = m[0].strip()
        assert re.search(r"bool fine = true;|fine = false;|fine = fine && there;|__all_sync\(0xffffffffu, fine\)", line), line


# ---------------------------------------------------------------------------
# Sums over very long caches
# ---------------------------------------------------------------------------
@gpu
@pytest.mark.parametrize("fp8,hd,T,kw", [
    (False, 128, 1301, dict()), (True, 64, 1301, dict(softcap=5.0, window=3000001)), (True, 128, 21, dict()),
    (False, 64, 21, dict(slopes=[-1e-9] * 16)), (False, 64, 200, dict(window=70001))], ids=str)
@pytest.mark.parametrize("power", [16, 17, 20, 22])
def test_sums_over_very_long_caches(L, power, fp8, hd, T, kw):  # noqa: F811
    """Prompt rows over up to 2^22 keys: eight pages again and again, so that every sum has
    few terms in the reference and all of them on the device.  Values of one sign and
    saturated caps leave no error to cancel."""
    torch = _torch()
    n, H, ps, P = 2 ** power, 16, 1024, 8
    rng = np.random.default_rng(power + hd)
    dtype = torch.float8_e4m3fn if fp8 else torch.bfloat16
    kv = L.PagedKV.empty(P, ps, 1, hd, dtype)
    for t, shift in ((kv.k, 0.0), (kv.v, 1.0)):
        t.copy_(torch.from_numpy((rng.standard_normal((P, ps, 1, hd)) + shift).astype(np.float32)).cuda().to(dtype))
    k, v = (t.double().cpu().numpy().reshape(P * ps, hd) for t in (kv.k, kv.v))
    table = (torch.arange(n // ps, dtype=torch.int32, device="cuda") % P)[None].contiguous()
    scale = 20 * hd ** -0.5 if kw.get("softcap") else hd ** -0.5
    q = torch.from_numpy(rng.standard_normal((T, H * hd)).astype(np.float32)).cuda().bfloat16()
    out, lse = torch.empty_like(q), torch.empty(T, H, device="cuda")
    slopes = None if "slopes" not in kw else torch.tensor(kw["slopes"], device="cuda")
    att = L.Attention(1, T, H, kv, scale, kw.get("softcap", 0.0), kw.get("window", 0), slopes)
    att.run(q, out, torch.tensor([0, T], dtype=torch.int32, device="cuda"),
            torch.tensor([n], dtype=torch.int32, device="cuda"), table, T, lse=lse, path="prompt")
    torch.cuda.synchronize()
    assert att.err.item() == 0
    for t in {0, T // 2, T - 1}:
        p = n - T + t
        lo = max(0, p - kw["window"] + 1) if "window" in kw else 0
        # how often the row sees each of the P * ps keys
        times = np.bincount(np.arange(lo, p + 1) % (P * ps), minlength=P * ps)
        s = q[t].double().cpu().numpy().reshape(H, hd) @ k.T * scale
        if kw.get("softcap"):
            s = kw["softcap"] * np.tanh(s / kw["softcap"])
        w = np.where(times > 0, times * np.exp(s - s.max()), 0.0)
        ref, size = w @ v / w.sum(1, keepdims=True), w @ np.abs(v) / w.sum(1, keepdims=True)
        big = np.abs(s).max() + (0 if slopes is None else 1e-9 * n)
        tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 * 1.01 + 2.0 ** -18 * (1 + big)) * size
        if slopes is not None:  # the bias moves a weight by 1e-9 a key at most; it is not in ref
            tol = tol + 2 * (np.exp(1e-9 * n) - 1) * size
        assert (np.abs(out[t].double().cpu().numpy().reshape(H, hd) - ref) <= tol).all()
        if slopes is None:
            assert (np.abs(lse[t].double().cpu().numpy() - (np.log(w.sum(1)) + s.max()))
                    <= 2.0 ** -18 * (1 + big)).all()


# ---------------------------------------------------------------------------
# Calls without a hint
# ---------------------------------------------------------------------------
@gpu
@pytest.mark.parametrize("rows,n,want", [(1, 64, "decode"), (1, 300, "decode"), (4, 40, "decode"), (600, 2, "prompt"),
                                         (40, 1, "prompt")])
def test_without_a_hint_rows_count_as_shared_evenly(L, rows, n, want):  # noqa: F811
    """The path is the one that a hint of T / n_seq takes: same bits (the paths round weights
    differently, so that the other path's differ)."""
    torch = _torch()
    c = Case(L, [max(rows, 300)] * n, [rows] * n, 8, 2, 64, seed=18)
    assert L.lora_attend_resolve_path("auto", c.run(want).att.c, c.kv.c, n, rows) == want
    outs = {p: c.run(p).out.clone() for p in PATHS}
    assert not torch.equal(*outs.values())
    assert torch.equal(c.run("auto", hint=0).out, outs[want])
    assert torch.equal(c.run("auto", hint=rows).out, outs[want])


@gpu
def test_more_decode_steps_than_32_bits_count(L):  # noqa: F811
    """2^12 requests of 2^25 tokens, all of them the same page: 2^32 steps.  The call reports
    it and writes nothing."""
    torch = _torch()
    n = L.LORA_MAX_SEQS
    kv = L.PagedKV.empty(1, 1024, 1, 128)
    for t in (kv.k, kv.v):
        t.zero_()
    table = torch.zeros(n, 2 ** 15, dtype=torch.int32, device="cuda")
    q = torch.zeros(n, 128, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 7.0)
    att = L.Attention(n, n, 1, kv)
    lens = torch.full((n,), 2 ** 25, dtype=torch.int32, device="cuda")
    off = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    att.run(q, out, off, lens, table, 1, path="decode")
    assert att.err.item() == 9 and bool((out == 7.0).all())
    assert not bool(att.ws.any())
    # the same call with shorter requests is served in the same workspace
    att.err.zero_()
    att.run(q, out, off, lens // 2 ** 18, table, 1, path="decode")
    assert att.err.item() == 0 and bool((out == 0.0).all())
