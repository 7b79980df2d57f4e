"""The attention side of a serving step (include/lora_attention.h): step tables,
rotary append and paged attention against plain 64-bit implementations, and
their refusals.

Tolerances (u = 2^-8, the unit roundoff of bf16):
- rotary: inputs are exact, the angle is exact to 2^-32 turns, sine and cosine
  to 2^-20, so a result is within u |ref| + 2^-18 (|a| + |b|) mscale of the
  definition; e4m3 (3 mantissa bits, smallest step 2^-9) within 2^-4 |ref| +
  2^-10 of the clamped quotient, plus the same small term.
- attention: one rounding of the output, u |ref|, and the rounding of the
  weights before the product with v: with A = sum_j p_j |v_j| at most u A where
  weights are bf16 (prompt path), 2^-11 A where they carry 11 bits or more
  (decode path: f16, or two bf16 parts); scores carry fp32 rounding, which
  moves a weight by 2^-18 (1 + max |s|) at most.
- lse: fp32 sums of positive terms, 2^-18 (1 + max |s|).
"""
import ctypes
import math
import os
import re
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "lora_attention.h")
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    from rank_adapter_gemm_gb300 import build
    build.build()
    import rank_adapter_gemm_gb300 as lib
    return lib


def _torch():
    import torch
    return torch


# ---------------------------------------------------------------------------
# Host side
# ---------------------------------------------------------------------------
def test_attention_header_is_exported(L):
    from rank_adapter_gemm_gb300 import _lib
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = sorted(set(re.findall(r"\b(lora_[a-z0-9_]+)\s*\(", text)))
    assert set(declared) == set(_lib.EXPORTED_ATTENTION)
    out = subprocess.run(["nm", "-D", "--defined-only", _lib.library_path()], capture_output=True, text=True).stdout
    exported = set(re.findall(r" T (lora_[a-z0-9_]+)$", out, flags=re.M))
    assert set(declared) <= exported
    assert L.lora_status_string(10).startswith("LORA_ERR_NO_PAGES")


LLAMA3 = {"kind": "llama3", "factor": 8.0, "low_freq_factor": 1.0, "high_freq_factor": 4.0, "original": 8192}
YARN = {"kind": "yarn", "factor": 16.0, "beta_fast": 32.0, "beta_slow": 1.0, "original": 4096}


def ref_frequencies(rot, theta, scaling):
    """Radians a position of each pair, and the factor on cos and sin, in 64 bits."""
    j = np.arange(rot // 2)
    kind = scaling["kind"] if scaling else "plain"
    if kind == "ntk":
        theta = theta * scaling["factor"] ** (rot / (rot - 2))
    f = theta ** (-2.0 * j / rot)
    if kind == "linear":
        return f / scaling["factor"], 1.0
    if kind == "llama3":
        turns = scaling["original"] * f / (2 * np.pi)
        t = np.clip((turns - scaling["low_freq_factor"]) / (scaling["high_freq_factor"] - scaling["low_freq_factor"]),
                    0, 1)
        return f * t + f / scaling["factor"] * (1 - t), 1.0
    if kind == "yarn":
        at = [rot * math.log(scaling["original"] / (b * 2 * math.pi)) / (2 * math.log(theta))
              for b in (scaling["beta_fast"], scaling["beta_slow"])]
        lo, hi = max(0, math.floor(at[0])), min(rot - 1, math.ceil(at[1]))
        r = np.clip((j - lo) / max(hi - lo, 1e-3), 0, 1)
        return f * (1 - r) + f / scaling["factor"] * r, 0.1 * math.log(scaling["factor"]) + 1
    return f, 1.0


@pytest.mark.parametrize("rot,theta,scaling", [
    (128, 10000.0, None), (64, 500000.0, LLAMA3), (128, 500000.0, YARN), (16, 10000.0, {"kind": "linear", "factor": 4}),
    (128, 10000.0, {"kind": "ntk", "factor": 2.5}), (256, 1e6, {"kind": "yarn", "factor": 1.0, "beta_fast": 2,
                                                               "beta_slow": 1, "original": 8})])
def test_rope_phases_match_the_formula(L, rot, theta, scaling):
    phases, m = L.lora_rope_phases(rot, theta, scaling)
    f, want_m = ref_frequencies(rot, theta, scaling)
    assert phases.shape == (rot // 2,)
    # the fixed point holds half a unit of 2^-64 turns; 64-bit floating point the rest
    got = phases.astype(np.float64) / 2.0 ** 64 * 2 * np.pi
    assert (np.abs(got - f) <= 2 * np.pi * 2.0 ** -65 + 2.0 ** -48 * f).all()
    assert m == np.float32(want_m)


def test_rope_phases_refusals(L):
    for rot, theta, scaling, status in [
            (8, 1e4, None, 2), (24, 1e4, None, 2), (272, 1e4, None, 2), (64, 1.0, None, 1), (64, math.nan, None, 1),
            (64, 1e4, {"kind": "linear", "factor": 0.5}, 1), (64, 1e4, {"kind": "linear", "factor": math.inf}, 1),
            (64, 1e4, dict(LLAMA3, high_freq_factor=1.0), 1), (64, 1e4, dict(YARN, beta_slow=0.0), 1),
            (64, 1e4, dict(YARN, original=0.0), 1)]:
        with pytest.raises(L.LoraError) as e:
            L.lora_rope_phases(rot, theta, scaling)
        assert e.value.status == status, (rot, theta, scaling)
    with pytest.raises(ValueError):
        L.lora_rope_phases(64, 1e4, {"kind": "other", "factor": 2.0})
    with pytest.raises(ValueError):
        L.lora_rope_phases(64, 1e4, {"kind": "linear", "times": 2.0})


def _kv(**kw):
    from rank_adapter_gemm_gb300._lib import lora_kv_t
    c = dict(k=1 << 20, v=1 << 21, n_pages=8, page_size=16, n_kv=2, head_dim=128, page_stride=4096, token_stride=256,
             head_stride=128, type=0, k_scale=1.0, v_scale=1.0)
    c.update(kw)
    return lora_kv_t(**c)


BAD_KV = [(dict(k=None), 1), (dict(v=0), 1), (dict(n_pages=0), 1), (dict(page_size=24), 1), (dict(page_size=2048), 1),
          (dict(page_size=0), 1), (dict(n_kv=0), 1), (dict(head_dim=0), 1), (dict(head_dim=272), 1), (dict(type=2), 1),
          (dict(page_stride=-8), 1), (dict(head_dim=72), 2), (dict(k=(1 << 20) + 8), 2), (dict(token_stride=260), 2),
          (dict(type=1, token_stride=264), 2), (dict(type=1, k_scale=0.0), 1), (dict(type=1, v_scale=math.inf), 1)]


@pytest.mark.parametrize("bad,status", BAD_KV)
def test_cache_descriptions_refused(L, bad, status):
    """Every call that takes a cache refuses the same descriptions, before any device work."""
    from rank_adapter_gemm_gb300._lib import lora_attention_t, lora_rope_t
    lib, P = L._lib.load(), 1 << 20
    kv, att = _kv(**bad), lora_attention_t(8, 0.1, 0.0, 0, None)
    size = ctypes.c_size_t(0)
    assert lib.lora_attend_workspace_bytes(att, kv, ctypes.byref(size)) == status
    assert lib.lora_rope_append(P, 1536, 4, 8, lora_rope_t(16, 0, 1.0, P), P, P, P, 1024, kv, None, None) == status
    assert lib.lora_attend(P, 1024, P, 1024, None, 4, 1, P, P, P, 4, 4, kv, att, 1, 0, P, 1 << 30, None,
                           None) == status


def test_host_refusals(L):
    """Argument errors return before anything is enqueued (no pointer is followed)."""
    from rank_adapter_gemm_gb300._lib import lora_attention_t, lora_rope_t
    lib, P, kv = L._lib.load(), 1 << 20, _kv()

    def step(**kw):
        a = dict(ctx=P, new=P, n=4, ps=16, free=P, nf=8, table=P, ld=8, w=8, T=16, qo=P, kl=P, pos=P, seq=P, sm=P,
                 tk=P)
        a.update(kw)
        return lib.lora_kv_step(a["ctx"], a["new"], a["n"], a["ps"], a["free"], a["nf"], a["table"], a["ld"], a["w"],
                                a["T"], a["qo"], a["kl"], a["pos"], a["seq"], a["sm"], a["tk"], None, None)
    for kw in (dict(n=-1), dict(nf=-1), dict(T=-1), dict(w=-1), dict(ld=4), dict(ps=12), dict(ps=0), dict(ps=2048),
               dict(qo=None), dict(tk=None), dict(ctx=None), dict(new=None), dict(kl=None), dict(table=None),
               dict(free=None), dict(pos=None), dict(seq=None), dict(sm=None)):
        assert step(**kw) == 1, kw

    def rope(qkv=P, ld=1536, T=4, H=8, r=lora_rope_t(128, 0, 1.0, P), pos=P, sm=P, q=P, ldq=1024):
        return lib.lora_rope_append(qkv, ld, T, H, r, pos, sm, q, ldq, kv, None, None)
    for kw, status in ((dict(T=-1), 1), (dict(H=0), 1), (dict(r=None), 1), (dict(r=lora_rope_t(128, 0, 1.0, None)), 1),
                       (dict(ld=1528), 1), (dict(ld=1540), 2), (dict(ldq=1016), 1), (dict(qkv=None), 1),
                       (dict(q=P + 8), 2), (dict(pos=None), 1), (dict(sm=None), 1), (dict(H=1 << 30), 1),
                       (dict(r=lora_rope_t(0, 0, 1.0, P)), 2), (dict(r=lora_rope_t(144, 0, 1.0, P)), 2),
                       (dict(r=lora_rope_t(24, 0, 1.0, P)), 2), (dict(r=lora_rope_t(64, 0, 1.0, P + 8)), 2)):
        assert rope(**kw) == status, kw
    assert rope(T=0, qkv=None, q=None, pos=None, sm=None) == 0

    def attend(q=P, ldq=1024, out=P, ldo=1024, T=4, n=1, qo=P, kl=P, tab=P, ldt=8, w=8, kv=kv, att=(8, 0.1, 0.0, 0),
               path=0, ws=P, wb=1 << 30):
        return lib.lora_attend(q, ldq, out, ldo, None, T, n, qo, kl, tab, ldt, w, kv,
                               None if att is None else lora_attention_t(*att, None), 1, path, ws, wb, None, None)
    for kw, status in ((dict(T=-1), 1), (dict(n=-1), 1), (dict(n=L.LORA_MAX_SEQS + 1), 1), (dict(qo=None), 1),
                       (dict(kl=None), 1), (dict(tab=None), 1), (dict(ldt=4), 1), (dict(w=-1), 1), (dict(path=3), 1),
                       (dict(path=-1), 1), (dict(att=None), 1), (dict(att=(7, 0.1, 0.0, 0)), 1),
                       (dict(att=(0, 0.1, 0.0, 0)), 1), (dict(att=(8, math.nan, 0.0, 0)), 1),
                       (dict(att=(8, 0.1, -1.0, 0)), 1), (dict(att=(8, 0.1, math.nan, 0)), 1),
                       (dict(att=(8, 0.1, 0.0, -1)), 1), (dict(q=None), 1), (dict(out=P + 2), 2), (dict(ldq=1028), 2),
                       (dict(ldo=1016), 1), (dict(ws=None), 6), (dict(wb=16), 6), (dict(ws=P + 8), 2),
                       (dict(kv=_kv(head_dim=96)), 9), (dict(kv=_kv(head_dim=256, head_stride=256)), 9)):
        assert attend(**kw) == status, kw
    assert attend(T=0, q=None, out=None) == 0 and attend(n=0) == 0


def test_attend_path_choice(L):
    from rank_adapter_gemm_gb300._lib import lora_attention_t
    att, kv = lora_attention_t(8, 0.1, 0.0, 0, None), _kv()  # 4 query heads a key head

    def path(n_seq, max_q, asked="auto"):
        return L.lora_attend_resolve_path(asked, att, kv, n_seq, max_q)
    assert path(1, 1) == path(4096, 1) == path(4096, 4) == "decode"
    assert path(1, 1000) == path(300, 8) == path(2, 1 << 30) == "prompt"
    # few requests: both paths split the cache, the prompt path into fewer and larger pieces
    assert path(1, 4) == "decode" and path(1, 64) == path(64, 64) == "prompt"
    assert path(1, 1000, "decode") == "decode" and path(1, 1, "prompt") == "prompt"


def test_binding_refuses_host_tensors_and_wrong_types(L):
    torch = _torch()
    with pytest.raises(TypeError):
        L.PagedKV(torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16), torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16))
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(TypeError):
        L.lora_kv_step(i, i, 16, i, torch.zeros(4, 4, dtype=torch.int32), i, i, i, i, i, i, i)


# ---------------------------------------------------------------------------
# Step tables
# ---------------------------------------------------------------------------
def ref_step(ctx, new, ps, free, table, T):
    """The definition, request by request and token by token."""
    table, at = [list(r) for r in table], 0
    width = len(table[0]) if table else 0
    q_off, kv, pos, seq, slots, taken, errors = [0], [], [], [], [], 0, set()
    for i, (c, m) in enumerate(zip(ctx, new)):
        ok = c >= 0 and m >= 0 and -(-(c + m) // ps) <= width
        errors |= set() if ok else {1}
        c0, m0 = max(c, 0), max(m, 0)
        need = -(-(c + m) // ps) - -(-c // ps) if ok else 0
        served = ok and (need == 0 or at + need <= len(free))
        if ok and not served:
            errors.add(10)
        for u in range(need if served else 0):
            table[i][-(-c // ps) + u] = free[at + u]
            taken = at + need
        for p in range(c0, c0 + min(m0, max(0, T + 1 - len(pos)))):  # (one past T tells of the rest)
            page = table[i][p // ps] if served else -1
            if served and page < 0:
                errors.add(4)
            pos.append(p)
            seq.append(i)
            slots.append(page * ps + p % ps if page >= 0 else -1)
        at += need
        q_off.append(min(q_off[-1] + m0, 2 ** 31 - 1))
        kv.append(c0 + m0 if served else c0)
    if len(pos) > T:
        errors.add(1)
    pad = max(0, T - len(pos))
    return (q_off, kv, (pos + [0] * pad)[:T], (seq + [-1] * pad)[:T], (slots + [-1] * pad)[:T], taken, table, errors)


def _run_step(L, ctx, new, ps, free, table, T, ld_pad=0):
    torch = _torch()
    n, width = len(ctx), len(table[0]) if table else 0
    big = torch.full((n, width + ld_pad), -99, dtype=torch.int32, device="cuda")
    big[:, :width] = torch.tensor(table, dtype=torch.int32).reshape(n, width).cuda()
    st = L.KVStep(n, T, width, ps)
    st.block_table = big[:, :width]
    for t in (st.q_offsets, st.kv_lens, st.positions, st.seq_ids, st.slot_map, st.taken):
        t.fill_(-77)
    i = [torch.tensor(v, dtype=torch.int32).cuda() for v in (ctx, new, free)]
    st.build(*i)
    torch.cuda.synchronize()
    assert bool((big[:, width:] == -99).all())
    return st


def _check_step(L, ctx, new, ps, free, table, T, ld_pad=0):
    st = _run_step(L, ctx, new, ps, free, table, T, ld_pad)
    q_off, kv, pos, seq, slots, taken, want_table, errors = ref_step(ctx, new, ps, free, table, T)
    assert st.q_offsets.tolist() == q_off
    assert st.kv_lens.tolist() == kv
    assert st.positions.tolist() == pos
    assert st.seq_ids.tolist() == seq
    assert st.slot_map.tolist() == slots
    assert st.taken.item() == taken
    if sum(new) <= T:
        assert st.block_table.tolist() == want_table
    err = st.err.item()
    assert (err in errors) if errors else err == 0
    return errors


def _step_case(seed, n, ps, ctx_hi, new_hi, spare=0, zero=0.2):
    rng = np.random.default_rng(seed)
    ctx, new = rng.integers(0, ctx_hi + 1, n), rng.integers(0, new_hi + 1, n)
    ctx[rng.random(n) < zero] = 0
    new[rng.random(n) < zero] = 0
    have = -(-ctx // ps)
    width = int((-(-(ctx + new) // ps)).max(initial=0)) + 2
    need = int((-(-(ctx + new) // ps) - have).sum())
    pages = rng.permutation(int(have.sum()) + need + spare + 5)
    table, at = np.full((n, width), -1), 0
    for i in range(n):
        table[i, :have[i]] = pages[at:at + have[i]]
        at += have[i]
    return ctx.tolist(), new.tolist(), table.tolist(), pages[at:at + need + spare].tolist()


@gpu
@pytest.mark.parametrize("n,ps,ctx_hi,new_hi,pad", [
    (1, 16, 0, 1, 0), (1, 16, 100, 1, 5), (3, 1, 7, 3, 0), (37, 16, 200, 1, 11), (64, 128, 3000, 40, 0),
    (1023, 16, 50, 3, 1), (1025, 32, 50, 3, 2000), (3000, 16, 40, 6, 0), (5, 1024, 5000, 3000, 0),
    (256, 64, 1000, 0, 7)])
def test_step_tables(L, n, ps, ctx_hi, new_hi, pad):
    ctx, new, table, free = _step_case(n + ps, n, ps, ctx_hi, new_hi, spare=3)
    assert not _check_step(L, ctx, new, ps, free, table, sum(new) + pad, ld_pad=n % 3)


@gpu
def test_step_edges(L):
    # no requests, no tokens, no room
    _check_step(L, [], [], 16, [], [], 0)
    _check_step(L, [], [], 16, [4], [], 9)
    _check_step(L, [5, 0], [0, 0], 16, [], [[7, -1], [-1, -1]], 0)
    # pages end exactly at the new tokens' ends
    _check_step(L, [15, 16, 17, 0], [1, 16, 15, 32], 16, [9, 8, 7, 6], [[1, -1], [2, -1], [3, 4], [-1, -1]], 64)
    # ids whose slots pass 32 bits
    _check_step(L, [0], [3], 1024, [2 ** 31 - 1], [[-1]], 3)


@gpu
def test_step_device_errors(L):
    t = [[10, -1, -1, -1] for _ in range(4)]
    # the second request needs two pages and one is left: it and all that need pages after it wait
    assert _check_step(L, [16, 16, 5, 16], [16, 17, 3, 1], 16, [1, 2], t, 37) == {10}
    assert _check_step(L, [-1, 3], [2, 2], 16, [5], t[:2], 4) == {1}
    assert _check_step(L, [3, 3], [-2, 2], 16, [5], t[:2], 2) == {1}
    assert _check_step(L, [60, 3], [5, 2], 16, [5, 6], t[:2], 7) == {1}
    assert _check_step(L, [3, 3], [5, 2], 16, [5, 6], t[:2], 4) == {1}
    assert _check_step(L, [3], [2], 16, [], [[-5, 0]], 2) == {4}
    assert _check_step(L, [2 ** 31 - 1, 1], [2 ** 31 - 1, 1], 1024, [3], [[1, 2], [1, 2]], 1) == {1}


# ---------------------------------------------------------------------------
# Rotary append
# ---------------------------------------------------------------------------
def _bf16(a):
    return _torch().from_numpy(np.asarray(a, np.float32)).bfloat16().cuda()


def ref_rope(x, positions, rot, interleaved, f, m):
    """x [T, heads, hd] in 64 bits, and the size of the terms of each result."""
    ang = positions.astype(np.float64)[:, None] * f[None]
    z = (m * np.exp(1j * ang))[:, None]
    out, size = x.copy(), np.zeros_like(x)
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    w = (a + 1j * b) * z
    s = (np.abs(a) + np.abs(b)) * m
    if interleaved:
        out[..., 0:rot:2], out[..., 1:rot:2], size[..., 0:rot:2], size[..., 1:rot:2] = w.real, w.imag, s, s
    else:
        out[..., :rot], size[..., :rot] = np.concatenate([w.real, w.imag], -1), np.concatenate([s, s], -1)
    return out, size


@gpu
@pytest.mark.parametrize("T,H,KV,hd,rot,inter,scaling,fp8,ps,base", [
    (1, 32, 8, 128, 128, False, LLAMA3, False, 16, 8000), (1, 1, 1, 64, 64, True, None, False, 16, 10),
    (7, 6, 2, 128, 64, True, None, True, 1, 4000), (33, 8, 8, 64, 32, False, YARN, True, 32, 100000),
    (130, 4, 1, 80, 80, False, {"kind": "linear", "factor": 3.0}, False, 64, 131072),
    (65, 3, 3, 256, 16, True, {"kind": "ntk", "factor": 4.0}, False, 16, 2 ** 31 - 66),
    (9, 5, 5, 96, 48, False, None, True, 1024, 0), (300, 40, 8, 16, 16, False, None, False, 16, 5)])
def test_rope_append(L, T, H, KV, hd, rot, inter, scaling, fp8, ps, base):
    torch = _torch()
    rng = np.random.default_rng(T * 7 + H)
    width = (H + 2 * KV) * hd
    big = _bf16(rng.standard_normal((T, width + 24)) * 2)
    qkv = big[:, 8:8 + width]
    q_big = torch.full((T + 2, H * hd + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    q_out = q_big[1:T + 1, :H * hd]
    pos = base + np.arange(T) if base > 2 ** 20 else rng.integers(0, base + 1, T)
    pos[T // 2] = base if T > 2 else -3 if T == 1 and base < 100 else pos[T // 2]
    n_pages = -(-T // ps) + 2
    slots = rng.permutation(n_pages * ps)[:T].astype(np.int64)
    if T > 3:
        slots[2] = -1
    dtype = torch.float8_e4m3fn if fp8 else torch.bfloat16
    ks, vs = (0.05, 0.4) if fp8 else (1.0, 1.0)
    kv = L.PagedKV.empty(n_pages, ps, KV, hd, dtype, ks, vs)
    for t in (kv.k, kv.v):
        t.view(torch.uint8).fill_(0x2A)
    before = kv.k.view(torch.uint8).clone()
    theta = 500000.0
    rope = L.Rope(hd, rot, theta, inter, scaling)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    src = qkv.clone()
    rope.append(qkv, q_out, H, kv, torch.from_numpy(pos.astype(np.int32)).cuda(), torch.from_numpy(slots).cuda(), err)
    torch.cuda.synchronize()
    assert err.item() == 0 and torch.equal(qkv, src)
    f, m = ref_frequencies(rot, theta, scaling)
    # the phases round the frequency to 64 bits of a turn; the reference's product has 53
    x = qkv.double().cpu().numpy().reshape(T, H + 2 * KV, hd)
    ref, size = ref_rope(x[:, :H + KV], pos, rot, inter, f, m)
    slack = 2.0 ** -18 * size + 2 * np.pi * np.abs(pos)[:, None, None] * 2.0 ** -52 * size
    got = q_out.double().cpu().numpy().reshape(T, H, hd)
    assert (np.abs(got - ref[:, :H]) <= 2.0 ** -8 * np.abs(ref[:, :H]) + slack[:, :H]).all()
    assert bool(q_big[0].isnan().all()) and bool(q_big[:, H * hd:].isnan().all())
    put = slots >= 0
    page, off = slots[put] // ps, slots[put] % ps
    for cache, want, scale, term in ((kv.k, ref[:, H:], ks, slack[:, H:]), (kv.v, x[:, H + KV:], vs, 0 * slack[:, H:])):
        got = cache[torch.from_numpy(page).cuda(), torch.from_numpy(off).cuda()].double().cpu().numpy()
        if fp8:
            want = np.clip(want / scale, -448, 448)
            tol = 2.0 ** -4 * np.abs(want) + 2.0 ** -10 + term / scale
        else:
            tol = 2.0 ** -8 * np.abs(want) + term
        assert (np.abs(got - want[put]) <= tol[put]).all()
    # every other slot keeps its bytes
    untouched = torch.ones(n_pages, ps, dtype=torch.bool, device="cuda")
    untouched[torch.from_numpy(page).cuda(), torch.from_numpy(off).cuda()] = False
    for cache in (kv.k, kv.v):
        assert torch.equal(cache.view(torch.uint8)[untouched], before[untouched])


@gpu
def test_rope_in_place_and_token_major_cache(L):
    """q turned inside the packed rows equals q_out, bit for bit; a token-major
    cache with k and v interleaved a page holds what a head-major one does."""
    torch = _torch()
    T, H, KV, hd, ps = 50, 8, 2, 128, 16
    rng = np.random.default_rng(5)
    qkv = _bf16(rng.standard_normal((T, (H + 2 * KV) * hd)))
    pos = torch.arange(T, dtype=torch.int32, device="cuda") + 900
    slots = torch.randperm(6 * ps, device="cuda")[:T]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    rope = L.Rope(hd)
    a = L.PagedKV.empty(6, ps, KV, hd)
    both = torch.zeros(6, 2, ps, KV, hd, dtype=torch.bfloat16, device="cuda")
    b = L.PagedKV(both[:, 0], both[:, 1])
    for t in (a.k, a.v):
        t.zero_()
    q = torch.empty(T, H * hd, dtype=torch.bfloat16, device="cuda")
    rope.append(qkv, q, H, a, pos, slots, err)
    inplace = qkv.clone()
    rope.append(inplace, inplace, H, b, pos, slots, err)
    torch.cuda.synchronize()
    assert torch.equal(inplace[:, :H * hd], q) and torch.equal(inplace[:, H * hd:], qkv[:, H * hd:])
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v) and err.item() == 0


@gpu
def test_rope_bad_slots_special_values_and_saturation(L):
    torch = _torch()
    T, H, KV, hd, ps = 4, 1, 1, 32, 16
    x = torch.zeros(T, 3 * hd, dtype=torch.bfloat16, device="cuda")
    x[0, 2 * hd:2 * hd + 5] = torch.tensor([float("inf"), -float("inf"), float("nan"), 1e30, -1e30])
    x[1, 2 * hd] = 7.0
    kv = L.PagedKV.empty(2, ps, KV, hd, torch.float8_e4m3fn, 0.5, 0.5)
    for t in (kv.k, kv.v):
        t.view(torch.uint8).fill_(0x11)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = torch.empty(T, hd, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([0, 2 * ps, -2, 2 ** 40], device="cuda")
    L.Rope(hd).append(x, q, H, kv, torch.zeros(T, dtype=torch.int32, device="cuda"), slots, err)
    torch.cuda.synchronize()
    assert err.item() == 4
    assert kv.v.view(torch.uint8)[0, 0, 0, :5].tolist() == [0x7E, 0xFE, 0x7F, 0x7E, 0xFE]
    assert bool((kv.v.view(torch.uint8)[0, 1:] == 0x11).all()) and bool((kv.v.view(torch.uint8)[1] == 0x11).all())


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------
def ref_attend(q, k, v, scale, softcap, window, slopes, length):
    """One request in 64 bits: q [m, H, hd], k and v [length, KV, hd].  Returns
    out, lse, sum_j p_j |v_j| and max |s|."""
    m, H, hd = q.shape
    G = H // k.shape[1]
    out, lse, size = np.zeros((m, H, hd)), np.full((m, H), -np.inf), np.zeros((m, H, hd))
    big = np.zeros((m, H))
    for i in range(m):
        p = length - m + i
        lo = max(0, p - window + 1) if window else 0
        if p < 0:
            continue
        for h in range(H):
            s = k[lo:p + 1, h // G] @ q[i, h] * scale
            if softcap:
                s = softcap * np.tanh(s / softcap)
            if slopes is not None:
                s = s + slopes[h] * (np.arange(lo, p + 1) - p)
            top = s.max()
            w = np.exp(s - top)
            out[i, h], size[i, h] = w @ v[lo:p + 1, h // G] / w.sum(), w @ np.abs(v[lo:p + 1, h // G]) / w.sum()
            lse[i, h], big[i, h] = top + np.log(w.sum()), np.abs(s).max()
    return out, lse, size, big


class Case:
    """Requests over a paged cache whose unused parts hold NaN."""

    def __init__(self, L, lens, q_lens, H, KV, hd, ps=16, fp8=False, layout="head", seed=0, pad=0, q_scale=1.5,
                 table_pad=1, v_shift=0.0, n_spare=2):
        torch = _torch()
        rng = np.random.default_rng(seed)
        self.lens, self.q_lens, self.H, self.KV, self.hd, self.L = lens, q_lens, H, KV, hd, L
        n = len(lens)
        used = [-(-max(x, 0) // ps) for x in lens]
        n_pages, width = sum(used) + n_spare, max(used + [0]) + table_pad
        dtype = torch.float8_e4m3fn if fp8 else torch.bfloat16
        self.ks, self.vs = (0.5, 0.125) if fp8 else (1.0, 1.0)
        shape = {"head": (n_pages, KV, ps, hd), "token": (n_pages, ps, KV, hd), "both": (n_pages, 2, ps, KV, hd),
                 "slot": (ps, n_pages, KV, hd)}[layout]
        raw = [torch.full(shape, 0x7F if fp8 else 0x7FC1, dtype=torch.uint8 if fp8 else torch.int16, device="cuda")
               for _ in range(1 if layout == "both" else 2)]
        view = {"head": lambda t: t.transpose(1, 2), "token": lambda t: t, "slot": lambda t: t.transpose(0, 1)}
        if layout == "both":
            k, v = raw[0][:, 0], raw[0][:, 1]
        else:
            k, v = (view[layout](t) for t in raw)
        k, v = k.view(dtype), v.view(dtype)
        order = rng.permutation(n_pages)
        table = np.full((n, width), -1)
        self.k, self.v, at = [], [], 0
        for i, x in enumerate(lens):
            x = max(x, 0)
            table[i, :used[i]] = order[at:at + used[i]]
            at += used[i]
            for cache, keep, shift, s in ((k, self.k, 0.0, self.ks), (v, self.v, v_shift, self.vs)):
                val = torch.from_numpy((rng.standard_normal((x, KV, hd)) + shift).astype(np.float32)).cuda()
                val = (val / s).to(dtype)
                slot = torch.arange(x, device="cuda")
                pages = torch.from_numpy(table[i]).cuda()[slot // ps] if x else slot
                if x:
                    cache.view(torch.uint8 if fp8 else torch.int16)[pages, slot % ps] = val.view(
                        torch.uint8 if fp8 else torch.int16)
                keep.append(val.double().cpu().numpy() * s)
        self.kv = L.PagedKV(k, v, self.ks, self.vs)
        self.T = sum(q_lens) + pad
        self.q_big = _bf16(rng.standard_normal((self.T, H * hd + 16)) * q_scale)
        self.q = self.q_big[:, 8:8 + H * hd]
        self.off = torch.tensor(np.concatenate([[0], np.cumsum(q_lens)]), dtype=torch.int32).cuda()
        self.lens_dev = torch.tensor(lens, dtype=torch.int32).cuda()
        self.table = torch.from_numpy(table.astype(np.int32)).cuda()

    def run(self, path, softcap=0.0, window=0, slopes=None, scale=None, hint=None, lse=True):
        torch = _torch()
        self.out_big = torch.full((self.T + 2, self.H * self.hd + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.out = self.out_big[1:self.T + 1, :self.H * self.hd]
        self.lse = torch.full((self.T, self.H), 77.0, device="cuda") if lse else None
        self.slopes = None if slopes is None else torch.tensor(slopes, dtype=torch.float32, device="cuda")
        self.att = self.L.Attention(len(self.lens), self.T, self.H, self.kv, scale, softcap, window, self.slopes)
        self.att.run(self.q, self.out, self.off, self.lens_dev, self.table,
                     max(self.q_lens + [0]) if hint is None else hint, lse=self.lse, path=path)
        torch.cuda.synchronize()
        return self

    def check(self, path, softcap=0.0, window=0, slopes=None, scale=None, err=0):
        scale = self.hd ** -0.5 if scale is None else scale
        slopes = None if self.slopes is None else self.slopes.double().cpu().numpy()
        assert self.att.err.item() == err
        q = self.q.double().cpu().numpy().reshape(self.T, self.H, self.hd)
        out = self.out.double().cpu().numpy().reshape(self.T, self.H, self.hd)
        weights = 2.0 ** -8 if path == "prompt" else 2.0 ** -11
        at = 0
        for i, (x, m) in enumerate(zip(self.lens, self.q_lens)):
            ref, lse, size, big = ref_attend(q[at:at + m], self.k[i], self.v[i], scale, softcap, window, slopes, x)
            tol = 2.0 ** -8 * np.abs(ref) + (weights * 1.01 + 2.0 ** -18 * (1 + big[..., None])) * size
            bad = ~(np.abs(out[at:at + m] - ref) <= tol)
            assert not bad.any(), (i, x, m, int(bad.sum()), np.argwhere(bad)[:5].tolist())
            if self.lse is not None:
                got = self.lse[at:at + m].double().cpu().numpy()
                fine = np.isfinite(lse)
                assert np.array_equal(fine, np.isfinite(got)) and (got[~fine] == -np.inf).all()
                assert (np.abs(got[fine] - lse[fine]) <= (2.0 ** -18 * (1 + big))[fine]).all()
            at += m
        # rows outside every request, and everything around the output
        o = self.out_big
        assert bool(o[0].isnan().all()) and bool(o[at + 1:].isnan().all()) and bool(o[:, self.H * self.hd:].isnan().all())
        if self.lse is not None:
            assert bool((self.lse[at:] == 77.0).all())
        # the workspace is left as it was found: a second call gives the same bits
        first = self.out.clone()
        self.out.fill_(float("nan"))
        self.att.run(self.q, self.out, self.off, self.lens_dev, self.table, max(self.q_lens + [0]), lse=self.lse,
                     path=path)
        assert bool((first.view(_torch().int16) == self.out.view(_torch().int16)).all())


PATHS = ("decode", "prompt")
SHAPES = [  # lens, q_lens, H, KV, hd, more
    ([1], [1], 1, 1, 128, {}),
    ([100], [1], 32, 8, 128, {}),
    ([0, 5, 16, 17, 31, 32, 33, 200], [1] * 8, 8, 2, 128, dict(pad=3)),
    ([300, 0, 64, 4], [4, 2, 4, 4], 8, 2, 64, dict(ps=32)),
    ([1000, 1, 129], [7, 3, 0], 6, 2, 128, dict(layout="token")),
    ([2, 0, 40], [5, 3, 9], 12, 4, 64, dict(layout="both", ps=8)),
    ([513, 77], [1, 2], 16, 1, 128, dict(ps=1)),
    ([700, 130], [130, 129], 4, 2, 128, dict(ps=128)),
    ([260, 128, 127, 1], [260, 128, 127, 1], 3, 1, 64, dict(layout="slot")),
    ([400], [37], 10, 2, 128, dict(pad=2)),
    ([3000], [1], 8, 8, 128, dict(ps=64)),
    ([150, 20], [40, 20], 24, 1, 64, dict(ps=16)),
]


@gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_attend_shapes(L, i, path, fp8):
    lens, q_lens, H, KV, hd, more = SHAPES[i]
    c = Case(L, lens, q_lens, H, KV, hd, fp8=fp8, seed=i, **more)
    c.run(path).check(path)


SCORES = [dict(softcap=20.0), dict(window=1), dict(window=40), dict(slopes=True), dict(softcap=5.0, window=100, slopes=True),
          dict(scale=0.5), dict(scale=0.0), dict(window=10 ** 9)]


@gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("i", range(len(SCORES)))
def test_attend_scores(L, i, path, fp8):
    kw = dict(SCORES[i])
    if kw.get("slopes"):
        kw["slopes"] = [2.0 ** -(h + 1) for h in range(8)]
    c = Case(L, [333, 41, 1, 150], [3, 1, 1, 150], 8, 2, 128 if i % 2 else 64, ps=32, fp8=fp8, seed=50 + i)
    c.run(path, **kw).check(path, **kw)


@gpu
@pytest.mark.parametrize("path", PATHS)
def test_attend_long_ragged_batches(L, path):
    """Many requests, split and joined over the whole GPU, and one long one."""
    rng = np.random.default_rng(3)
    lens = [int(x) for x in np.exp(rng.uniform(0, math.log(1500), 70))]
    Case(L, lens, [min(2, x) for x in lens], 8, 2, 64, seed=8).run(path).check(path)
    if path == "decode":
        Case(L, [20001], [1], 2, 1, 128, seed=9).run(path).check(path)
        Case(L, [9000], [4], 8, 2, 128, seed=10, fp8=True).run(path, window=5000, softcap=30.0).check(
            path, window=5000, softcap=30.0)
    else:
        Case(L, [1100], [1100], 2, 1, 128, seed=9).run(path).check(path)
        Case(L, [900], [600], 4, 2, 64, seed=10, fp8=True).run(path, window=333).check(path, window=333)


@gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hd,rows", [(128, 9), (64, 40), (128, 64)])
def test_attend_keys_in_parts(L, hd, rows, fp8):
    """Few rows over caches of 1 to 71 key steps: every number of parts from 1 to 16, with
    a request of each in one call too."""
    lens = [500, 900, 1100, 1700, 2200, 2700, 3300, 4000, 4500, 5200, 9000]
    for i, n in enumerate(lens[::3] if rows > 9 else lens):
        Case(L, [n], [min(n, rows)], 4, 1, hd, ps=64, fp8=fp8, seed=20 + i).run("prompt").check("prompt")
    c = Case(L, [2200, 90, 0, 1300, 4000], [rows, 3, 2, 1, rows], 8, 2, hd, ps=32, fp8=fp8, seed=40)
    c.run("prompt").check("prompt")
    kw = dict(softcap=20.0, window=1500, slopes=[2.0 ** -(h + 4) for h in range(8)])
    c.run("prompt", **kw).check("prompt", **kw)


@gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hd", [64, 128])
def test_attend_many_prompts(L, hd, fp8):
    """More items than half of the SMs: whole ones, of up to and of more than 32 requests."""
    rng = np.random.default_rng(hd)
    for n in (13, 40):
        q = [int(x) for x in rng.integers(0, 150, n)]
        lens = [x + int(y) for x, y in zip(q, rng.integers(0, 300, n))]
        c = Case(L, lens, q, 16, 8, hd, fp8=fp8, seed=60 + n)
        c.run("prompt").check("prompt")
        kw = dict(softcap=20.0, window=100, slopes=[2.0 ** -(h / 2 + 1) for h in range(16)])
        c.run("prompt", **kw).check("prompt", **kw)


@gpu
@pytest.mark.parametrize("path", PATHS)
def test_attend_large_scores(L, path):
    """Scores far apart and far from zero: one key takes all, sums do not overflow."""
    c = Case(L, [200, 70], [2, 70], 4, 2, 128, seed=4, q_scale=40.0)
    c.run(path, scale=1.0).check(path, scale=1.0)
    c = Case(L, [200, 70], [2, 70], 4, 2, 64, seed=5, fp8=True, q_scale=3000.0)
    c.run(path).check(path)


@gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("power", [90, -90])
def test_attend_query_magnitudes(L, power, path, fp8):
    """Queries far from 1 with a scale that brings the scores back: powers of two
    change nothing but exponents."""
    c = Case(L, [77, 150], [1, 60], 4, 2, 64, seed=13, fp8=fp8)
    scale = 64 ** -0.5
    want = c.run(path, scale=scale).out.clone()
    c.q_big.mul_(2.0 ** power)
    c.run(path, scale=scale * 2.0 ** -power).check(path, scale=scale * 2.0 ** -power)
    assert _torch().equal(c.out, want)


@gpu
def test_attend_many_weights_of_little_mass(L):
    """A few strong keys and a long tail whose weights are far below the largest
    one but whose mass is not."""
    torch = _torch()
    for fp8 in (False, True):
        c = Case(L, [30000], [1], 4, 1, 64, seed=6, fp8=fp8, v_shift=1.0)
        c.q_big.mul_(0.05)
        hot = c.table[0, 100].item()
        c.k[0][1600] = 0.0
        c.kv.k[hot, 0] = torch.zeros(1, 64, device="cuda").to(c.kv.k.dtype)
        c.run("decode", slopes=[0.0] * 4).check("decode")


@gpu
def test_attend_offsets_past_32_bits(L):
    """A cache of more than 2^32 elements, pages of one request on both ends of it."""
    torch = _torch()
    for fp8 in (False, True):
        dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
        ps, KV, hd, n_pages = 16, 8, 128, (1 << 32) // (16 * 8 * 128) + 40
        kv = L.PagedKV.empty(n_pages, ps, KV, hd, dt)
        g = torch.Generator(device="cuda").manual_seed(1)
        pages = [n_pages - 1, 0, n_pages - 2, 7]
        small = L.PagedKV.empty(4, ps, KV, hd, dt)
        for j, p in enumerate(pages):
            for a, b in ((kv.k, small.k), (kv.v, small.v)):
                val = torch.randn(ps, KV, hd, generator=g, device="cuda").to(dt)
                a[p], b[j] = val, val
        q = torch.randn(1 + 40, 8 * hd, generator=g, device="cuda").bfloat16()
        off = torch.tensor([0, 1, 41], dtype=torch.int32, device="cuda")
        lens = torch.tensor([60, 64], dtype=torch.int32, device="cuda")
        outs = []
        for cache, row in ((kv, pages), (small, [0, 1, 2, 3])):
            table = torch.tensor([row, row], dtype=torch.int32, device="cuda")
            for path in PATHS:
                att = L.Attention(2, 41, 8, cache)
                out = torch.zeros(41, 8 * hd, dtype=torch.bfloat16, device="cuda")
                att.run(q, out, off, lens, table, 40, path=path)
                outs.append(out)
        assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])
        assert bool(outs[0].isfinite().all()) and outs[0].abs().max() > 0
        # the append writes there too
        qkv = torch.randn(2, 24 * hd, generator=g, device="cuda").bfloat16()
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        L.Rope(hd).append(qkv, torch.empty(2, 8 * hd, dtype=torch.bfloat16, device="cuda"), 8, kv,
                          torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                          torch.tensor([n_pages * ps - 1, 3], device="cuda"), err)
        assert torch.equal(kv.v[n_pages - 1, 15].float(), qkv[0, 16 * hd:].view(8, hd).to(dt).float())
        assert err.item() == 0
        del kv
        torch.cuda.empty_cache()


@gpu
@pytest.mark.parametrize("path", PATHS)
def test_attend_device_errors(L, path):
    """Bad lengths, offsets and page ids are reported and stay inside the buffers."""
    torch = _torch()
    c = Case(L, [40, 50, 30], [2, 2, 2], 4, 2, 64, seed=1)
    good = c.run(path).out.clone()
    # a length beyond the table row, a negative one: those requests are skipped
    for bad in (10 ** 9, -4, 2 ** 31 - 1):
        c.lens_dev = torch.tensor([40, bad, 30], dtype=torch.int32).cuda()
        c.run(path)
        assert c.att.err.item() == 1
        assert torch.equal(c.out[:2], good[:2]) and torch.equal(c.out[4:], good[4:])
    c.lens_dev = torch.tensor([40, 50, 30], dtype=torch.int32).cuda()
    for off in ([0, 4, 2, 6], [0, 2, 4, 70000], [-5, 2, 4, 6]):
        c.off = torch.tensor(off, dtype=torch.int32).cuda()
        c.run(path)
        assert c.att.err.item() == 1
    c.off = torch.tensor([0, 2, 4, 6], dtype=torch.int32).cuda()
    # page ids outside the cache read as zeros
    for bad in (-1, 10 ** 9):
        c.table[1, 1] = bad
        c.run(path)
        assert c.att.err.item() == 4
        assert torch.equal(c.out[:2], good[:2]) and torch.equal(c.out[4:], good[4:])
        c.k[1][16:32], c.v[1][16:32] = 0.0, 0.0
        c.check(path, err=4)


@gpu
@pytest.mark.parametrize("path", PATHS)
def test_attend_other_stream_and_graph(L, path):
    torch = _torch()
    c = Case(L, [500, 90, 33], [2, 2, 2], 8, 2, 128, seed=2)
    want = c.run(path).out.clone()
    s = torch.cuda.Stream()
    c.out.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        c.att.run(c.q, c.out, c.off, c.lens_dev, c.table, 2, path=path)
    s.synchronize()
    assert torch.equal(c.out, want)
    c.out.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.att.run(c.q, c.out, c.off, c.lens_dev, c.table, 2, path=path)
    for _ in range(3):
        c.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.out, want)


@gpu
def test_paths_agree_and_auto_is_one_of_them(L):
    torch = _torch()
    c = Case(L, [700, 64], [8, 8], 8, 2, 128, seed=11)
    outs = {p: c.run(p).out.float().clone() for p in ("decode", "prompt", "auto")}
    assert torch.equal(outs["auto"], outs["decode"]) or torch.equal(outs["auto"], outs["prompt"])
    assert (outs["decode"] - outs["prompt"]).abs().max() < 0.05
    # the hint may be loose
    assert torch.equal(c.run("decode", hint=0).out.float(), outs["decode"])
    assert torch.equal(c.run("prompt", hint=1).out.float(), outs["prompt"])


# ---------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------
@gpu
def test_two_steps_through_one_cache(L):
    """A prompt step, then decode steps, through lora_kv_step, lora_rope_append
    and lora_attend on one cache: each equals attention over the whole history."""
    torch = _torch()
    n, H, KV, hd, ps = 3, 8, 2, 64, 16
    rng = np.random.default_rng(12)
    kv = L.PagedKV.empty(40, ps, KV, hd)
    for t in (kv.k, kv.v):
        t.view(torch.int16).fill_(0x7FC1)
    rope = L.Rope(hd, theta=500000.0)
    f, m = ref_frequencies(hd, 500000.0, None)
    step = L.KVStep(n, 100, 8, ps)
    free, used = torch.randperm(40, device="cuda").to(torch.int32), 0
    ctx, hist_k, hist_v = [0] * n, [np.zeros((0, KV, hd))] * n, [np.zeros((0, KV, hd))] * n
    for new in ([50, 0, 17], [1, 20, 1], [1, 1, 1]):
        T = 100
        qkv = _bf16(rng.standard_normal((T, (H + 2 * KV) * hd)))
        i32 = dict(dtype=torch.int32, device="cuda")
        step.build(torch.tensor(ctx, **i32), torch.tensor(new, **i32), free[used:].contiguous())
        used += step.taken.item()
        q, out = torch.empty(T, H * hd, dtype=torch.bfloat16, device="cuda"), torch.zeros(
            T, H * hd, dtype=torch.bfloat16, device="cuda")
        rope.append(qkv, q, H, kv, step.positions, step.slot_map, step.err)
        att = L.Attention(n, T, H, kv)
        att.run(q, out, step.q_offsets, step.kv_lens, step.block_table, max(new))
        torch.cuda.synchronize()
        assert step.err.item() == 0 and att.err.item() == 0
        x = qkv.double().cpu().numpy().reshape(T, H + 2 * KV, hd)
        at = 0
        for i in range(n):
            rows = slice(at, at + new[i])
            pos = np.arange(ctx[i], ctx[i] + new[i])
            k_new = torch.from_numpy(ref_rope(x[rows, H:H + KV], pos, hd, False, f, m)[0]).bfloat16().double().numpy()
            hist_k[i] = np.concatenate([hist_k[i], k_new])
            hist_v[i] = np.concatenate([hist_v[i], x[rows, H + KV:]])
            ctx[i] += new[i]
            qr = q[rows].double().cpu().numpy().reshape(new[i], H, hd)
            ref, _, size, big = ref_attend(qr, hist_k[i], hist_v[i], hd ** -0.5, 0.0, 0, None, ctx[i])
            got = out[rows].double().cpu().numpy().reshape(new[i], H, hd)
            # a k may round the other way where the turned value is near a tie: 2^-8 of a score's terms
            tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 * 1.01 + 2.0 ** -8 * (1 + big[..., None])) * size
            assert (np.abs(got - ref) <= tol).all()
            at += new[i]


@gpu
@pytest.mark.parametrize("kw", [dict(), dict(cache_type="e4m3", softcap=30.0, window=40)])
def test_layer_example(L, kw):
    """The example's layer: LoRA projections, rotary append and attention on one
    cache over a prompt step and decode steps, each call against a plain fp32 form.
    Every output is rounded to bf16 once by each side (relative rms about 2^-9.3
    each), the attention's weights once more: below 2^-7 together."""
    torch = _torch()
    import importlib.util
    spec = importlib.util.spec_from_file_location("attention_layer", os.path.join(ROOT, "examples",
                                                                                  "attention_layer.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    kw = dict(kw)
    if kw.get("cache_type") == "e4m3":
        kw["cache_type"] = torch.float8_e4m3fn
    layer = ex.Layer(512, 8, 2, 64, 3, 16, 6, 16, 16, **kw)
    worst, _ = ex.serve(layer, [33, 1, 70, 128, 5, 16], 3, 512, check=True)
    assert worst < 2.0 ** -7


# ---------------------------------------------------------------------------
# Over the range
# ---------------------------------------------------------------------------
@gpu
@pytest.mark.parametrize("seed", range(24))
def test_attend_drawn(L, seed):
    """Drawn head layouts, lengths, page sizes, strides, types and score forms on
    both paths: requests without rows or cached tokens, rows before the first key,
    one request or many, few keys or enough to be split."""
    rng = np.random.default_rng(1000 + seed)
    path = PATHS[seed % 2]
    KV, G, hd = int(rng.choice([1, 2, 3, 8])), int(rng.choice([1, 2, 3, 5, 8, 16])), int(rng.choice([64, 128]))
    n = int(rng.choice([1, 2, 5, 40]))
    q_hi = int(rng.choice([1, 2, 6])) if path == "decode" else int(rng.choice([1, 30, 150]))
    top = 4000 // (n * max(1, q_hi // 8)) + 1
    lens = [int(x) for x in np.exp(rng.uniform(0, math.log(top), n))]
    q_lens = [int(rng.integers(0, q_hi + 1)) for _ in range(n)]
    for i in range(n):
        if rng.random() < 0.1:
            lens[i] = 0
    c = Case(L, lens, q_lens, KV * G, KV, hd, ps=int(2 ** rng.integers(0, 8)), fp8=bool(rng.random() < 0.5),
             layout=str(rng.choice(["head", "token", "both", "slot"])), seed=seed, pad=int(rng.integers(0, 3)),
             v_shift=float(rng.choice([0.0, 0.5])))
    kw = dict(softcap=float(rng.choice([0.0, 0.0, 8.0, 50.0])), window=int(rng.choice([0, 0, 3, 100, 1000])))
    if rng.random() < 0.4:
        kw["slopes"] = [float(2.0 ** -rng.uniform(0, 8)) for _ in range(KV * G)]
    c.run(path, **kw).check(path, **kw)
