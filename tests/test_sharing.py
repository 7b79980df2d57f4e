"""Requests that share what they have cached (include/lora_sharing.h): beam
selection, table fork and compaction, page copies and shared-prefix attention
against plain 64-bit implementations, and their refusals.

Tolerances (u = 2^-8, bf16's rounding by half a step):
- selection: a score is rounded once to fp32, 2^-24 |c|.  In ln sum exp a term e^d
  carries the rounding of d log2(e), 2^-23 |d|, and 2^-22 of the exponential; the
  terms' mean of |d| is at most ln(vocab) + 1 < 18; 32 terms and a tree of 8
  levels are added in fp32, 40 2^-24.  Together 18 2^-23 + 2^-22 + 40 2^-24 < 2^-18.
  Tokens and parents are compared where neighbouring candidates lie further apart.
- tables, lists, copies: equal.
- attention: one rounding of the output, u |ref|, and of the weights before the
  product with v, at most u A with A = sum_j p_j |v_j| (prefix, bf16 weights);
  scores carry fp32 rounding, which moves a weight by 2^-18 (1 + max |s|).
- lse: 2^-18 (1 + max |s|).
"""
import ctypes
import math
import os
import re
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "lora_sharing.h")
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


def dev(x, dtype=None):
    torch = _torch()
    return torch.tensor(x, dtype=dtype or torch.int32).cuda()


# ---------------------------------------------------------------------------
# Host side
# ---------------------------------------------------------------------------
def test_sharing_header_is_exported(L):
    from rank_adapter_gemm_gb300 import _lib
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = sorted(set(re.findall(r"\b(lora_[a-z0-9_]+)\s*\(", text)))
    assert set(declared) == set(_lib.EXPORTED_SHARING)
    out = subprocess.run(["nm", "-D", "--defined-only", _lib.library_path()], capture_output=True, text=True).stdout
    assert set(declared) <= set(re.findall(r" T (lora_[a-z0-9_]+)$", out, flags=re.M))
    for name in ("LORA_MAX_BEAMS", "LORA_MAX_KV_LAYERS"):
        assert int(re.search(rf"#define {name} (\d+)", text).group(1)) == getattr(_lib, name)
    for name in ("LORA_MAX_VOCAB", "LORA_MAX_PAGES"):
        assert 1 << int(re.search(rf"#define {name} \(1 << (\d+)\)", text).group(1)) == getattr(_lib, name)


P = 1 << 20  # an address that host checks only look at


def test_select_refusals(L):
    lib = L._lib.load()
    need = L.lora_beam_select_workspace_bytes(2, 4, 4, 1000)
    good = dict(logits=P, ld=1000, type=0, n=2, beams=4, vocab=1000, keep=4, scores=P, ended=None, eos=-1, parents=P,
                tokens=P, out_scores=P, out_ended=P, ws=P, bytes=need)

    def call(**kw):
        return lib.lora_beam_select(*{**good, **kw}.values(), None)

    for bad, status in [(dict(n=-1), 1), (dict(n=4097), 1), (dict(beams=0), 1), (dict(beams=65), 1), (dict(keep=0), 1),
                        (dict(keep=65), 1), (dict(vocab=0), 1), (dict(vocab=(1 << 24) + 1), 1), (dict(ld=999), 1),
                        (dict(type=2), 1), (dict(eos=1000), 1), (dict(eos=-2), 1), (dict(ended=P), 1),
                        (dict(logits=None), 1), (dict(scores=None), 1), (dict(parents=None), 1), (dict(tokens=None), 1),
                        (dict(out_scores=None), 1), (dict(out_ended=None), 1), (dict(logits=P + 1), 2),
                        (dict(logits=P + 2, type=1), 2), (dict(ws=None), 6), (dict(bytes=need - 1), 6),
                        (dict(ws=P + 8), 2)]:
        assert call(**bad) == status, bad
    assert call(n=0, logits=None, scores=None, parents=None, tokens=None, out_scores=None, out_ended=None) == 0
    with pytest.raises(L.LoraError):
        L.lora_beam_select_workspace_bytes(1, 65, 1, 10)


def _pages_call(L, name, **kw):
    lib = L._lib.load()
    if name == "fork":
        good = dict(src=P, ld_src=8, src_width=8, lens=P, n_src=4, parents=P, n_dst=4, ps=16, pages=100, held=None,
                    n_held=0, dst=2 * P, ld_dst=8, dst_width=8, dst_lens=2 * P, copies=P, free=P, n_free=P)
        return lib.lora_kv_fork(*{**good, **kw}.values(), None, None)
    good = dict(src=P, ld_src=8, width=8, lens=P, n=4, ps=16, pages=100, held=None, n_held=0, dst=2 * P, ld_dst=8,
                dst_held=None, moves=P, n_moves=P, free=P, n_free=P)
    return lib.lora_kv_compact(*{**good, **kw}.values(), None, None)


BAD_PAGES = [(dict(ps=0), 1), (dict(ps=24), 1), (dict(ps=2048), 1), (dict(pages=0), 1), (dict(pages=(1 << 20) + 1), 9),
             (dict(n_held=-1), 1), (dict(n_held=3), 1), (dict(free=None), 1), (dict(n_free=None), 1),
             (dict(lens=None), 1), (dict(src=None), 1), (dict(dst=None), 1), (dict(ld_src=7), 1), (dict(ld_dst=7), 1),
             (dict(dst=P + 4 * 31), 1), (dict(dst=P - 4 * 31), 1)]


@pytest.mark.parametrize("bad,status", BAD_PAGES + [
    (dict(n_src=-1), 1), (dict(n_src=4097), 1), (dict(n_dst=-1), 1), (dict(n_dst=4097), 1), (dict(src_width=-1), 1),
    (dict(dst_width=-1), 1), (dict(parents=None), 1), (dict(dst_lens=None), 1), (dict(copies=None), 1),
    (dict(dst_lens=P + 4), 1)])
def test_fork_refusals(L, bad, status):
    assert _pages_call(L, "fork", **bad) == status


@pytest.mark.parametrize("bad,status", BAD_PAGES + [
    (dict(n=-1), 1), (dict(n=4097), 1), (dict(width=-1), 1), (dict(moves=None), 1), (dict(n_moves=None), 1),
    (dict(held=P, n_held=3), 1)])
def test_compact_refusals(L, bad, status):
    assert _pages_call(L, "compact", **bad) == status


def _kv(**kw):
    from rank_adapter_gemm_gb300._lib import lora_kv_t
    c = dict(k=1 << 20, v=1 << 21, n_pages=8, page_size=16, n_kv=2, head_dim=128, page_stride=4096, token_stride=256,
             head_stride=128, type=0, k_scale=1.0, v_scale=1.0)
    c.update(kw)
    return lora_kv_t(**c)


def test_copy_refusals(L):
    from rank_adapter_gemm_gb300._lib import lora_kv_t
    lib = L._lib.load()

    def call(kvs, n=None, copies=P, n_copies=4):
        arr = (lora_kv_t * max(1, len(kvs)))(*kvs)
        return lib.lora_kv_copy(arr, len(kvs) if n is None else n, copies, n_copies, None, None, None)

    assert call([_kv()], n=0) == 1 and call([_kv()] * 129) == 1 and call([_kv()], n_copies=-1) == 1
    assert call([_kv()], copies=None) == 1 and lib.lora_kv_copy(None, 1, P, 1, None, None, None) == 1
    assert call([_kv()], n_copies=0, copies=None) == 0
    for other in (dict(n_pages=9), dict(page_size=8), dict(n_kv=1), dict(head_dim=64), dict(page_stride=8192),
                  dict(token_stride=128), dict(head_stride=256), dict(type=1)):
        assert call([_kv(), _kv(**other)]) == 1, other
    assert call([_kv(), _kv(k=None)]) == 1 and call([_kv(k=(1 << 20) + 8)]) == 2 and call([_kv(head_dim=72)]) == 2


def test_shared_refusals(L):
    from rank_adapter_gemm_gb300._lib import lora_attention_t, lora_prefix_t
    lib, kv = L._lib.load(), _kv()
    att = lora_attention_t(8, 0.1, 0.0, 0, None)
    need = L.lora_attend_shared_workspace_bytes(att, kv, 4, 2)
    good = dict(q=P, ldq=1024, out=P, ldo=1024, lse=None, T=4, n=2, off=P, lens=P, table=P, ld=4, width=4,
                prefix=lora_prefix_t(P, P, 1, 0), kv=kv, att=att, hint=1, ws=P, bytes=need)

    def call(**kw):
        return lib.lora_attend_shared(*{**good, **kw}.values(), None, None)

    for bad, status in [(dict(T=-1), 1), (dict(n=-1), 1), (dict(n=4097), 1), (dict(width=5), 1), (dict(q=None), 1),
                        (dict(out=None), 1), (dict(off=None), 1), (dict(lens=None), 1), (dict(table=None), 1),
                        (dict(ldq=1016), 1), (dict(q=P + 8), 2), (dict(ldo=1028), 2), (dict(prefix=None), 1),
                        (dict(prefix=lora_prefix_t(None, P, 1, 0)), 1), (dict(prefix=lora_prefix_t(P, None, 1, 0)), 1),
                        (dict(prefix=lora_prefix_t(P, P, -1, 0)), 1), (dict(prefix=lora_prefix_t(P, P, 4097, 0)), 1), (dict(prefix=lora_prefix_t(P, P, 1, 2)), 1),
                        (dict(kv=_kv(n_pages=0)), 1), (dict(kv=_kv(head_dim=96)), 9),
                        (dict(att=lora_attention_t(7, 0.1, 0.0, 0, None)), 1),
                        (dict(att=lora_attention_t(8, math.nan, 0.0, 0, None)), 1),
                        (dict(att=lora_attention_t(8, 0.1, -1.0, 0, None)), 1),
                        (dict(att=lora_attention_t(8, 0.1, 0.0, -1, None)), 1), (dict(ws=None), 6),
                        (dict(bytes=need - 1), 6), (dict(ws=P + 4), 2)]:
        assert call(**bad) == status, bad
    assert call(T=0, q=None, out=None) == 0 and call(n=0, lens=None, table=None) == 0
    with pytest.raises(L.LoraError):
        L.lora_attend_shared_workspace_bytes(att, kv, -1, 2)


# ---------------------------------------------------------------------------
# Selection
# ---------------------------------------------------------------------------
def ref_select(x, scores, ended, eos, keep):
    """(parent, token, score) of every request's candidates in order: x [n, beams, V] in 64 bits."""
    n, beams, V = x.shape
    got = []
    for r in range(n):
        cand = []
        for b in range(beams):
            s = float(scores[r, b])
            if not -math.inf < s < math.inf:
                continue
            if ended is not None and ended[r, b]:
                cand.append((-s, b, eos))
                continue
            row = x[r, b]
            if np.isnan(row).any() or row.max() in (math.inf, -math.inf):
                continue
            c = s + row - (row.max() + math.log(np.exp(row - row.max()).sum()))
            order = np.lexsort((np.arange(V), -c))[:keep]
            cand += [(-c[v], b, int(v)) for v in order if c[v] > -math.inf]
        got.append([(r * beams + b, v, -s) for s, b, v in sorted(cand)[:keep + 1]])
    return got


def check_select(sel, x, scores, ended, eos, keep):
    parents, tokens, out, over = (t.cpu().numpy().reshape(len(x), keep) for t in
                                  (sel.parents, sel.tokens, sel.scores, sel.ended))
    tol = 2.0 ** -18
    sure = 0
    for r, cand in enumerate(ref_select(x, scores, ended, eos, keep)):
        beams = x.shape[1]
        for k in range(keep):
            if k >= len(cand):
                assert (parents[r, k], tokens[r, k], out[r, k], over[r, k]) == (-1, -1, -math.inf, 0)
                continue
            p, v, c = cand[k]
            assert abs(out[r, k] - c) <= tol + 2.0 ** -24 * abs(c)
            apart = [abs(c - cand[j][2]) for j in (k - 1, k + 1) if 0 <= j < len(cand)]
            same_beam = [cand[j][0] == p for j in (k - 1, k + 1) if 0 <= j < len(cand)]
            # equal candidates of one beam have an order; those of two beams within the tolerance may swap
            if all(s or a > 2 * tol for a, s in zip(apart, same_beam)):
                sure += 1
                assert (parents[r, k], tokens[r, k]) == (p, v), (r, k)
                done = ended is not None and bool(ended[r, p - r * beams])
                assert over[r, k] == int(done or v == eos)
    assert sure > 0 or all(not c for c in ref_select(x, scores, ended, eos, keep))


def run_select(L, x, scores, keep, dtype, ended=None, eos=-1, ld=None, skip=0):
    torch = _torch()
    n, beams, V = x.shape
    full = torch.full((n * beams, (ld or V) + skip), 7.0, dtype=dtype, device="cuda")
    view = full[:, skip:skip + V]
    view.copy_(torch.from_numpy(x.reshape(n * beams, V)))
    sel = L.BeamSelect(n, beams, keep, V, eos=eos, dtype=dtype)
    s = torch.from_numpy(np.asarray(scores, np.float32).reshape(-1)).cuda()
    e = None if ended is None else dev(np.asarray(ended).reshape(-1))
    for _ in range(2):  # the workspace is left as it was
        sel.run(view, s, e)
    torch.cuda.synchronize()
    assert int(sel.ws[:16384].count_nonzero()) == 0
    return sel, view.double().cpu().numpy().reshape(n, beams, V), s.double().cpu().numpy().reshape(n, beams)


@gpu
@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("n,beams,keep,V", [
    (1, 1, 1, 1), (1, 1, 5, 3), (2, 4, 4, 100), (3, 3, 6, 8192), (1, 4, 4, 8193), (2, 5, 10, 20011), (1, 64, 64, 300),
    (4, 1, 64, 40000), (7, 2, 33, 999)])
def test_select(L, n, beams, keep, V, fp32):
    torch = _torch()
    rng = np.random.default_rng(n * 1000 + V)
    x = rng.standard_normal((n, beams, V)) * 3
    scores = -5 * rng.random((n, beams))
    sel, x, s = run_select(L, x, scores, keep, torch.float32 if fp32 else torch.bfloat16)
    check_select(sel, x, s, None, -1, keep)


@gpu
@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("ld,skip", [(1003, 0), (1001, 1), (1008, 5), (1024, 7)])
def test_select_rows_of_any_alignment(L, ld, skip, fp32):
    torch = _torch()
    rng = np.random.default_rng(ld)
    sel, x, s = run_select(L, rng.standard_normal((2, 3, 1001)), rng.random((2, 3)), 6,
                           torch.float32 if fp32 else torch.bfloat16, ld=ld, skip=skip)
    check_select(sel, x, s, None, -1, 6)


@gpu
@pytest.mark.parametrize("fp32", [False, True])
def test_select_ended_beams_and_eos(L, fp32):
    torch = _torch()
    rng = np.random.default_rng(5)
    n, beams, V, eos = 6, 4, 500, 17
    x = rng.standard_normal((n, beams, V))
    x[:, :, eos] += 6.0  # often among the best
    ended = (rng.random((n, beams)) < 0.4).astype(np.int32)
    ended[1] = 1
    x[0, ended[0] == 1] = math.nan  # an ended beam's logits are not read
    sel, x, s = run_select(L, x, -rng.random((n, beams)), 5, torch.float32 if fp32 else torch.bfloat16, ended, eos)
    check_select(sel, x, s, ended, eos, 5)


@gpu
@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("keep", [3, 64])
def test_select_equal_logits_lowest_token_first(L, keep, fp32):
    """Constant rows, rising rows, rows of few values, signed zeros: whole chunks reach the bound."""
    torch = _torch()
    V = 9000
    x = np.zeros((1, 5, V))
    x[0, 1] = np.arange(V) // 100
    x[0, 2] = np.arange(V)[::-1] // 100
    x[0, 3] = np.where(np.arange(V) % 2 == 0, -0.0, 0.0)
    x[0, 4] = np.where(np.arange(V) // 64 % 64 == 5, 3.0, -2.0)
    for b in range(5):
        sel, y, s = run_select(L, x[:, b:b + 1], np.zeros((1, 1)), keep, torch.float32 if fp32 else torch.bfloat16)
        want = np.lexsort((np.arange(V), -y[0, 0]))[:keep]
        assert (sel.tokens.cpu().numpy() == want).all(), b


@gpu
@pytest.mark.parametrize("keep", [5, 64])
def test_select_equal_beams(L, keep):
    """64 beams of the same logits and scores: more candidates reach the bound than are gathered."""
    torch = _torch()
    sel, y, s = run_select(L, np.zeros((2, 64, 70)), np.zeros((2, 64)), keep, torch.bfloat16)
    assert sel.parents.tolist() == [0] * keep + [64] * keep
    assert sel.tokens.tolist() == 2 * list(range(keep))


@gpu
@pytest.mark.parametrize("fp32", [False, True])
def test_select_masks_and_numbers_out_of_range(L, fp32):
    torch = _torch()
    rng = np.random.default_rng(9)
    x = rng.standard_normal((5, 3, 700))
    scores = -rng.random((5, 3))
    x[0, :, 3:] = -math.inf            # two or three tokens left a beam
    x[0, 1] = -math.inf                # none at all
    x[1, 0, 5], x[1, 1, 6] = math.nan, math.inf
    scores[2] = [0.0, -math.inf, math.nan]
    scores[3] = -math.inf              # nothing to continue
    x[4] = np.where(rng.random((3, 700)) < 0.5, torch.finfo(torch.bfloat16).min, x[4])  # the type's lowest value
    sel, y, s = run_select(L, x, scores, 12, torch.float32 if fp32 else torch.bfloat16)
    check_select(sel, y, s, None, -1, 12)


@gpu
def test_select_in_place_and_captured(L):
    torch = _torch()
    rng = np.random.default_rng(11)
    n, beams, V = 3, 4, 2000
    x = [torch.from_numpy(rng.standard_normal((n * beams, V))).cuda().bfloat16() for _ in range(3)]
    a, b = (L.BeamSelect(n, beams, beams, V, eos=7) for _ in range(2))
    scores, ended = torch.zeros(n * beams, device="cuda"), torch.zeros(n * beams, dtype=torch.int32, device="cuda")
    for step in x:  # through fresh inputs
        a.run(step, scores, ended)
        scores, ended = a.scores.clone(), a.ended.clone()
    for step in x:  # in place
        b.run(step, b.scores, b.ended)
    for name in ("parents", "tokens", "scores", "ended"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name
    c, held = L.BeamSelect(n, beams, beams, V, eos=7), x[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(held, c.scores, c.ended)
    for step in x:
        held.copy_(step)
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.tokens, c.tokens) and torch.equal(a.scores, c.scores)
    with pytest.raises(ValueError):
        d = L.BeamSelect(n, beams, 2 * beams, V)
        d.run(x[0], d.scores, None)


# ---------------------------------------------------------------------------
# Tables
# ---------------------------------------------------------------------------
def ref_free(n_pages, used):
    free = [p for p in range(n_pages) if p not in used]
    return free


def ref_fork(src, lens, parents, ps, n_pages, dst, held):
    """(dst, lens, copies, free, n_free, error seen) by the definition, row by row."""
    dst, new_lens, copies, used, seen, bad = dst.copy(), [], [], set(), set(), False
    jobs = []
    for h in held:
        if h != -1:
            if 0 <= h < n_pages:
                used.add(h)
            else:
                bad = True
    for i, p in enumerate(parents):
        n = 0
        if p < -1 or p >= len(lens):
            bad, p = True, -1
        if p >= 0:
            n = int(lens[p])
            if n < 0 or -(-n // ps) > min(src.shape[1], dst.shape[1]):
                bad, n = True, 0
        pages = -(-n // ps)
        copy = n % ps != 0 and p in seen
        if p >= 0:
            seen.add(p)
        new_lens.append(n)
        copies.append([-1, -1, 0])
        for e in range(pages - int(copy)):
            dst[i, e] = src[p, e]
            if 0 <= src[p, e] < n_pages:
                used.add(int(src[p, e]))
            else:
                bad = True
        if copy:
            jobs.append((i, pages - 1, int(src[p, pages - 1]), n % ps))
    free = ref_free(n_pages, used)
    for u, (i, e, page, m) in enumerate(jobs):
        if u >= len(free):
            bad = True
            new_lens[i] -= m
            continue
        dst[i, e] = free[u]
        if 0 <= page < n_pages:
            copies[i] = [page, free[u], m]
        else:
            bad = True
    free = free[len(jobs):]
    return dst, new_lens, copies, free + [-1] * (n_pages - len(free)), len(free), bad


def random_tables(rng, n, ps, hi, width, n_pages, share):
    """Rows of which `share` neighbours begin with common full pages; the last page that is not full is a row's own."""
    lens = rng.integers(0, hi + 1, n)
    ids = rng.permutation(n_pages)
    table, at = rng.integers(-5, n_pages + 5, (n, width)).astype(np.int32), 0
    for i in range(n):
        pages = -(-int(lens[i]) // ps)
        first = i // share * share
        common = int(min(lens[i] // ps, lens[first] // ps) * rng.random()) if i != first else 0
        table[i, :common] = table[first, :common]
        table[i, common:pages] = ids[at:at + pages - common]
        at += pages - common
    return table, lens.astype(np.int32), at


def run_fork(L, src, lens, parents, ps, n_pages, dst, held=()):
    torch = _torch()
    n = len(parents)
    out = dict(dst=dev(dst), lens=torch.full((n,), -7, dtype=torch.int32, device="cuda"),
               copies=torch.full((n, 3), -7, dtype=torch.int32, device="cuda"),
               free=torch.full((n_pages,), -7, dtype=torch.int32, device="cuda"),
               n_free=torch.full((1,), -7, dtype=torch.int32, device="cuda"),
               err=torch.zeros(1, dtype=torch.int32, device="cuda"))
    L.lora_kv_fork(dev(src), dev(lens), dev(parents), ps, out["dst"], out["lens"], out["copies"], out["free"],
                   out["n_free"], out["err"], held=dev(held) if len(held) else None)
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in out.items()}


def check_fork(got, want):
    dst, lens, copies, free, n_free, bad = want
    assert (got["dst"] == dst).all()
    assert got["lens"].tolist() == lens and got["copies"].tolist() == copies
    assert got["n_free"].tolist() == [n_free] and got["free"].tolist() == free
    assert (got["err"][0] != 0) == bad


@gpu
@pytest.mark.parametrize("n,out,ps,hi,share", [
    (1, 1, 16, 5, 1), (1, 9, 16, 100, 1), (8, 8, 16, 300, 2), (40, 64, 1, 50, 4), (33, 20, 64, 5000, 3),
    (300, 300, 16, 2000, 8), (7, 7, 1024, 9000, 2), (4096, 4096, 16, 60, 4), (2, 2, 16, 20000, 1)])
def test_fork(L, n, out, ps, hi, share):
    rng = np.random.default_rng(n + out + ps)
    width = -(-hi // ps) + 2
    src, lens, used = random_tables(rng, n, ps, hi, width, n * width + 40, share)
    n_pages = n * width + 40
    held = np.concatenate([rng.integers(0, n_pages, 5), [-1]]).astype(np.int32)
    parents = rng.integers(0, n, out)
    parents[rng.random(out) < 0.1] = -1
    dst = rng.integers(-9, 9, (out, width + 1)).astype(np.int32)
    check_fork(run_fork(L, src, lens, parents, ps, n_pages, dst, held),
               ref_fork(src, lens, parents, ps, n_pages, dst, held))


@gpu
def test_fork_without_rows_pages_or_room(L):
    rng = np.random.default_rng(2)
    # no rows at all: every page is free but the held ones
    got = run_fork(L, np.zeros((0, 4), np.int32), np.zeros(0, np.int32), np.zeros(0, np.int32), 16, 37,
                   np.zeros((0, 4), np.int32), [3, 36])
    assert got["n_free"][0] == 35 and got["free"][:35].tolist() == [p for p in range(37) if p not in (3, 36)]
    # rows that all branch from one, with pages for some of the copies only
    src, lens = rng.permutation(12)[:8].reshape(1, 8).astype(np.int32), np.array([117], np.int32)
    dst = np.full((9, 8), -3, np.int32)
    for n_pages in (8, 12):
        s = src % 8 if n_pages == 8 else src
        s = np.arange(8, dtype=np.int32)[None] if n_pages == 8 else s
        want = ref_fork(s, lens, [0] * 9, 16, n_pages, dst, [])
        got = run_fork(L, s, lens, [0] * 9, 16, n_pages, dst)
        check_fork(got, want)
        assert got["err"][0] == 10 and want[5]
        assert got["lens"].tolist()[:1 + n_pages - 8] == [117] * (n_pages - 7)
    # one page, one row, nothing to branch
    got = run_fork(L, [[0]], [1], [0], 16, 1, np.full((1, 1), -1, np.int32))
    assert got["dst"].tolist() == [[0]] and got["n_free"][0] == 0 and got["free"].tolist() == [-1] and got["err"][0] == 0


@gpu
@pytest.mark.parametrize("what,status", [("parent", 1), ("below", 1), ("length", 1), ("negative", 1), ("page", 4),
                                         ("last", 4), ("held", 4)])
def test_fork_bad_data(L, what, status):
    rng = np.random.default_rng(4)
    src, lens, _ = random_tables(rng, 6, 16, 100, 8, 60, 1)
    lens[1], lens[2] = 70, 77
    src[1, :5], src[2, :5] = np.arange(50, 55), np.arange(55, 60)
    parents, held = np.array([0, 1, 1, 2, 3, 4, 5, 2]), [7]
    if what == "parent":
        parents[3] = 6
    elif what == "below":
        parents[3] = -2
    elif what == "length":
        lens[1] = 8 * 16 + 1
    elif what == "negative":
        lens[1] = -4
    elif what == "page":
        src[1, 2] = 60
    elif what == "last":
        src[2, 4] = -1
    else:
        held = [7, 60]
    dst = np.full((8, 8), -3, np.int32)
    want = ref_fork(src, lens, parents, 16, 60, dst, held)
    got = run_fork(L, src, lens, parents, 16, 60, dst, held)
    check_fork(got, want)
    assert got["err"][0] == status and want[5]


def ref_compact(src, lens, ps, n_pages, dst, held):
    dst, used, bad, rows = dst.copy(), set(), False, []
    for i, n in enumerate(lens):
        n = int(n)
        if n < 0 or -(-n // ps) > src.shape[1]:
            bad, n = True, 0
        rows.append(-(-n // ps))
        for p in src[i, :rows[-1]]:
            if 0 <= p < n_pages:
                used.add(int(p))
            else:
                bad = True
    for h in held:
        if 0 <= h < n_pages:
            used.add(int(h))
        elif h != -1:
            bad = True
    count = len(used)
    holes = [p for p in range(count) if p not in used]
    moves = list(zip(sorted(p for p in used if p >= count), holes))
    to = dict(moves)
    for i, n in enumerate(rows):
        dst[i, :n] = [to.get(int(p), p) for p in src[i, :n]]
    new_held = [int(to.get(int(h), h)) for h in held]
    free = list(range(count, n_pages)) + [-1] * count
    moves = [[a, b, ps] for a, b in moves]
    return dst, new_held, moves + [[-1, -1, 0]] * (n_pages // 2 - len(moves)), len(moves), free, n_pages - count, bad


def run_compact(L, src, lens, ps, n_pages, dst, held):
    torch = _torch()
    i32 = dict(dtype=torch.int32, device="cuda")
    out = dict(dst=dev(dst), moves=torch.full((n_pages // 2, 3), -7, **i32), n_moves=torch.full((1,), -7, **i32),
               free=torch.full((n_pages,), -7, **i32), n_free=torch.full((1,), -7, **i32), err=torch.zeros(1, **i32),
               held=torch.full((len(held),), -7, **i32))
    L.lora_kv_compact(dev(src), dev(lens), ps, out["dst"], out["moves"], out["n_moves"], out["free"], out["n_free"],
                      out["err"], held=dev(held) if len(held) else None, new_held=out["held"] if len(held) else None)
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in out.items()}


def check_compact(got, want):
    dst, held, moves, n_moves, free, n_free, bad = want
    assert (got["dst"] == dst).all() and got["held"].tolist() == held
    assert got["n_moves"].tolist() == [n_moves] and got["moves"].tolist() == moves
    assert got["n_free"].tolist() == [n_free] and got["free"].tolist() == free
    assert (got["err"][0] != 0) == bad


@gpu
@pytest.mark.parametrize("n,ps,hi,share,spread", [
    (1, 16, 5, 1, 3.0), (8, 16, 300, 2, 1.0), (40, 1, 50, 4, 1.2), (33, 64, 5000, 3, 5.0), (300, 16, 2000, 8, 2.0),
    (4096, 16, 60, 4, 2.0), (2, 16, 20000, 1, 1.5), (0, 16, 0, 1, 1.0)])
def test_compact(L, n, ps, hi, share, spread):
    rng = np.random.default_rng(n + ps)
    width = -(-hi // ps) + 1
    n_pages = int((n * width + 9) * spread)
    src, lens, used = random_tables(rng, n, ps, hi, width, n_pages, share)
    for held in ([], rng.integers(-1, n_pages, 9).tolist()):
        dst = rng.integers(-9, 9, (n, width)).astype(np.int32)
        check_compact(run_compact(L, src, lens, ps, n_pages, dst, held),
                      ref_compact(src, lens, ps, n_pages, dst, held))


@gpu
@pytest.mark.parametrize("n_pages", [1, 2, 31, 32, 33, 1023, 1024, 1025, 1 << 20])
def test_compact_full_and_empty_caches(L, n_pages):
    """All pages in use, none, the last one alone."""
    for ids in (range(min(n_pages, 5000)), (), (n_pages - 1,)):
        src = np.array([list(ids)[::-1] + [0]], np.int32)
        lens, dst = [len(ids)], np.full_like(src, -1)
        check_compact(run_compact(L, src, lens, 1, n_pages, dst, []), ref_compact(src, lens, 1, n_pages, dst, []))


@gpu
@pytest.mark.parametrize("what,status", [("length", 1), ("negative", 1), ("page", 4), ("held", 4)])
def test_compact_bad_data(L, what, status):
    rng = np.random.default_rng(6)
    src, lens, _ = random_tables(rng, 6, 16, 100, 8, 60, 1)
    lens[1], held = 70, [5]
    src[1, :5] = np.arange(50, 55)
    if what == "length":
        lens[1] = 8 * 16 + 1
    elif what == "negative":
        lens[1] = -1
    elif what == "page":
        src[1, 2] = -9
    else:
        held = [5, -3]
    dst = np.full((6, 8), -3, np.int32)
    got = run_compact(L, src, lens, 16, 60, dst, held)
    check_compact(got, ref_compact(src, lens, 16, 60, dst, held))
    assert got["err"][0] == status


# ---------------------------------------------------------------------------
# Copies
# ---------------------------------------------------------------------------
def make_layers(L, rng, layers, pages, ps, KV, hd, fp8, order):
    torch = _torch()
    axes = {"head": (0, 2, 1, 3), "token": (0, 1, 2, 3), "page_last": (2, 1, 0, 3)}[order]  # memory order of the dims
    dims = (pages, ps, KV, hd)
    kvs = []
    for _ in range(layers):
        both = []
        for _ in range(2):
            t = torch.from_numpy(rng.integers(0, 100, [dims[a] for a in axes], dtype=np.uint8)).cuda()
            t = t if fp8 else t.to(torch.bfloat16)
            both.append(t.permute(*np.argsort(axes).tolist()))
        kvs.append(L.PagedKV(*both))
    return kvs


@gpu
@pytest.mark.parametrize("order", ["head", "token", "page_last"])
@pytest.mark.parametrize("layers,pages,ps,KV,hd,fp8", [
    (1, 3, 1, 1, 16, True), (2, 9, 16, 2, 128, False), (3, 40, 32, 3, 48, True), (128, 6, 16, 1, 64, False),
    (1, 300, 16, 8, 128, True), (1, 5, 1024, 2, 256, False)])
def test_copy(L, order, layers, pages, ps, KV, hd, fp8):
    torch = _torch()
    rng = np.random.default_rng(layers + pages)
    kvs = make_layers(L, rng, layers, pages, ps, KV, hd, fp8, order)
    ids = rng.permutation(pages)
    n = pages // 2
    jobs = [[int(ids[2 * i]), int(ids[2 * i + 1]), int(rng.integers(0, ps + 1))] for i in range(n)] + [[-1, 0, 5], [0, -1, 1]]
    want = []
    for kv in kvs:
        for t in (kv.k, kv.v):
            w = t.clone()
            for a, b, m in jobs[:n]:
                w[b, :m] = t[a, :m]
            want.append(w)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.KVLayers(kvs).copy(dev(jobs), err)
    torch.cuda.synchronize()
    assert int(err) == 0
    got = [t for kv in kvs for t in (kv.k, kv.v)]
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@gpu
def test_copy_counts_and_bad_rows(L):
    torch = _torch()
    rng = np.random.default_rng(1)
    for jobs, count, first, status in [
            ([[0, 4, 16], [1, 5, 16], [2, 6, 16]], 2, [0, 1], 0), ([[0, 4, 16], [1, 5, 16]], 0, [], 0),
            ([[0, 4, 16], [1, 5, 16]], 3, [0, 1], 1), ([[0, 4, 16], [1, 5, 16]], -1, [], 1),
            ([[0, 4, 16], [8, 5, 16], [2, 6, 16]], None, [0, 2], 4), ([[0, 4, 16], [1, -2, 16]], None, [0], 4),
            ([[0, 4, 17], [1, 5, 16]], None, [1], 1), ([[0, 4, -1], [1, 5, 16]], None, [1], 1)]:
        (kv,) = make_layers(L, rng, 1, 8, 16, 2, 64, False, "head")
        want = kv.k.clone(), kv.v.clone()
        for i in first:
            a, b, m = jobs[i]
            for w, t in zip(want, (kv.k, kv.v)):
                w[b, :m] = t[a, :m]
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        L.KVLayers([kv]).copy(dev(jobs), err, count=None if count is None else dev([count]))
        torch.cuda.synchronize()
        assert int(err) == status, (jobs, count)
        assert torch.equal(kv.k, want[0]) and torch.equal(kv.v, want[1]), (jobs, count)


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------
class Batch:
    """A batch whose groups share prefixes: groups is a list of (prefix, [(own tokens, rows), ...])."""

    def __init__(self, groups, H, KV, hd, ps, fp8=False, order="head", seed=0, alone=(), twins=False, rows_after=0):
        torch = _torch()
        rng = np.random.default_rng(seed)
        reqs, starts = [], [0]
        for prefix, own in groups:
            reqs += [(prefix, c, m) for c, m in own]
            starts.append(len(reqs))
        reqs += [(0, c, m) for c, m in alone]  # requests outside every group
        n = len(reqs)
        self.n, self.H, self.KV, self.hd, self.ps, self.fp8 = n, H, KV, hd, ps, fp8
        self.starts, self.prefix = starts, [p for p, _ in groups]
        self.new = [m for _, _, m in reqs]
        self.lens = [p + c + m for p, c, m in reqs]
        self.T = sum(self.new)
        self.rows = self.T + rows_after
        width = max([-(-x // ps) for x in self.lens] + [1]) + 1
        total = sum(-(-x // ps) for x in self.lens) + 3
        ids = rng.permutation(total)
        self.table = np.full((n, width), -1, np.int32)
        self.k, self.v = np.zeros((total, ps, KV, hd)), np.zeros((total, ps, KV, hd))
        at = 0
        keys = [(rng.standard_normal((p, KV, hd)), rng.standard_normal((p, KV, hd)) + 0.1) for p, _ in groups]
        for g, (p, _) in enumerate(groups):
            for i in range(starts[g], starts[g + 1]):
                shared = 0 if twins or i == starts[g] else p // ps  # twins: the same tokens in other pages
                self.table[i, :shared] = self.table[starts[g], :shared]
                for e in range(shared, -(-self.lens[i] // ps)):
                    self.table[i, e] = ids[at]
                    at += 1
                own = self.lens[i] - p
                kk = np.concatenate([keys[g][0], rng.standard_normal((own, KV, hd))])
                vv = np.concatenate([keys[g][1], rng.standard_normal((own, KV, hd)) + 0.1])
                self._put(i, kk, vv)
        for i in range(starts[-1], n):
            for e in range(-(-self.lens[i] // ps)):
                self.table[i, e] = ids[at]
                at += 1
            self._put(i, rng.standard_normal((self.lens[i], KV, hd)), rng.standard_normal((self.lens[i], KV, hd)))
        axes = (0, 2, 1, 3) if order == "head" else (0, 1, 2, 3)
        dtype = torch.float8_e4m3fn if fp8 else torch.bfloat16
        self.dk, self.dv = (torch.from_numpy(np.ascontiguousarray(x.transpose(axes))).float().to(dtype).cuda()
                            .permute(*np.argsort(axes).tolist()) for x in (self.k, self.v))
        self.scales = (0.5, 0.25) if fp8 else (1.0, 1.0)
        self.dq = torch.from_numpy(rng.standard_normal((self.rows, H * hd))).cuda().bfloat16()

    def _put(self, i, kk, vv):
        for j in range(self.lens[i]):
            self.k[self.table[i, j // self.ps], j % self.ps] = kk[j]
            self.v[self.table[i, j // self.ps], j % self.ps] = vv[j]

    def run(self, L, softcap=0.0, window=0, slopes=None, scale=None, hint=0, prefix=None, starts=None, att=None, lens=None,
            repeat=1, share="always"):
        torch = _torch()
        kv = L.PagedKV(self.dk, self.dv, *self.scales)
        s = None if slopes is None else dev(slopes, torch.float32)
        att = att or L.SharedAttention(self.n, self.rows, self.H, kv, scale=scale, softcap=softcap, window=window, slopes=s)
        out = torch.full((self.rows, self.H * self.hd), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((self.rows, self.H), 7.0, device="cuda")
        off = np.concatenate([[0], np.cumsum(self.new)])
        for _ in range(repeat):
            att.run(self.dq, out, dev(off), dev(self.lens if lens is None else lens), dev(self.table),
                    dev(self.starts if starts is None else starts), dev(self.prefix if prefix is None else prefix),
                    hint, kv=kv, lse=lse, share=share)
        torch.cuda.synchronize()
        self.err = int(att.err)
        return out, lse

    def check(self, out, lse, softcap=0.0, window=0, slopes=None, scale=None, skip=()):
        """Every request by the definition, through its own row, in 64 bits."""
        torch = _torch()
        G = self.H // self.KV
        k, v = (x.double().cpu().numpy() * s for x, s in zip((self.dk, self.dv), self.scales))
        q = self.dq.double().cpu().numpy().reshape(self.rows, self.H, self.hd)
        out, lse = out.double().cpu().numpy().reshape(self.rows, self.H, self.hd), lse.double().cpu().numpy()
        scale = self.hd ** -0.5 if scale is None else scale
        at, u = 0, 2.0 ** -8
        for i, (m, n) in enumerate(zip(self.new, self.lens)):
            j = np.arange(n)
            page, offs = self.table[i, j // self.ps], j % self.ps
            kk, vv = k[page, offs], v[page, offs]
            pos = np.arange(n - m, n)
            seen = j[None] <= pos[:, None]
            if window:
                seen &= j[None] > pos[:, None] - window
            kk, vv = (np.where(seen.any(0)[:, None, None], x, 0.0) for x in (kk, vv))  # (what no row sees may be NaN)
            for h in range(self.H):
                if i in skip:
                    assert (out[at:at + m, h] == 7.0).all()
                    continue
                s = scale * q[at:at + m, h] @ kk[:, h // G].T
                if softcap:
                    s = softcap * np.tanh(s / softcap)
                if slopes is not None:
                    s = s + slopes[h] * (j[None] - pos[:, None])
                s = np.where(seen, s, -np.inf)
                top = s.max(1, keepdims=True, initial=-np.inf)
                e = np.exp(s - np.where(np.isfinite(top), top, 0.0))
                total = e.sum(1, keepdims=True)
                p = e / np.where(total > 0, total, 1.0)
                big = np.abs(np.where(seen, s, 0.0)).max(1, initial=0.0)
                eps = 2.0 ** -18 * (1 + big)
                ref, A = p @ vv[:, h // G], p @ np.abs(vv[:, h // G])
                tol = u * np.abs(ref) + (u + 2 * eps[:, None]) * A + 2.0 ** -20
                assert (np.abs(out[at:at + m, h] - ref) <= tol).all(), (i, h, np.abs(out[at:at + m, h] - ref).max())
                with np.errstate(divide="ignore"):
                    want = top[:, 0] + np.log(total[:, 0])
                got = lse[at:at + m, h]
                assert (np.where(total[:, 0] > 0, np.abs(got - np.where(total[:, 0] > 0, want, 0.0)) <= eps,
                                 got == -np.inf)).all()
            at += m
        assert (out[at:] == 7.0).all()  # rows behind the last request stay


GROUPS = {
    "pair": [(40, [(3, 1), (0, 1)])],
    "samples": [(500, [(i * 7, 1) for i in range(9)])],
    "many": [(p, [(c, 1) for c in range(s)]) for p, s in [(0, 3), (1, 2), (127, 4), (128, 1), (129, 5), (300, 7), (64, 0)]],
    "spec": [(200, [(5, 4), (60, 2), (0, 4)]), (77, [(1, 3), (0, 1)])],
    "large": [(700, [(i % 11, 1) for i in range(130)])],
    "rows": [(260, [(10, 70), (0, 33), (300, 1), (5, 0)])],
    "idle": [(150, [(3, 0), (0, 1), (5, 2), (0, 0), (40, 1)]), (90, [(7, 0), (8, 0)]), (200, [(0, 1), (0, 0)])],
}


@gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H,KV,hd,ps", [(8, 2, 128, 16), (4, 4, 64, 32), (6, 2, 64, 16), (16, 1, 128, 1)])
@pytest.mark.parametrize("groups", sorted(GROUPS))
def test_shared_prefix(L, groups, H, KV, hd, ps, fp8):
    b = Batch(GROUPS[groups], H, KV, hd, ps, fp8, order="head" if H == 8 else "token", alone=[(20, 1), (0, 2)],
              rows_after=3, seed=len(groups) + H)
    for share in ("always", "auto"):
        out, lse = b.run(L, repeat=2, share=share)
        b.check(out, lse)
        assert b.err == 0


@gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw", [dict(softcap=20.0), dict(window=1), dict(window=100), dict(window=450, softcap=5.0),
                                dict(slopes=True), dict(slopes=True, window=333, softcap=30.0), dict(scale=0.0),
                                dict(scale=-0.05), dict(softcap=0.01)])
def test_shared_prefix_masks_caps_and_bias(L, kw, fp8):
    H = 8
    kw = {k: [2.0 ** (-8 * (h + 1) / H) for h in range(H)] if k == "slopes" else v for k, v in kw.items()}
    b = Batch([(600, [(c, 1) for c in (0, 1, 90, 300)]), (130, [(200, 3), (0, 2)])], H, 2, 64 if fp8 else 128, 16, fp8,
              alone=[(40, 2)])
    out, lse = b.run(L, **kw)
    b.check(out, lse, **kw)
    assert b.err == 0


@gpu
def test_shared_prefix_in_other_pages_cut_and_absent(L):
    """The same tokens in other pages; prefixes longer than what a request has cached before its rows; no groups."""
    b = Batch([(300, [(10, 1), (0, 1), (2, 2)])], 8, 2, 128, 16, twins=True)
    b.check(*b.run(L))
    # every request holds its whole cache in common but its own rows: a prefix beyond that is cut
    c = Batch([(200, [(0, 1), (0, 1), (0, 2)])], 8, 2, 128, 16)
    c.check(*c.run(L, prefix=[100000]))
    assert c.err == 0
    c.check(*c.run(L, prefix=[0]))
    c.check(*c.run(L, prefix=[], starts=[0]))
    c.check(*c.run(L, prefix=[200, 200], starts=[0, 0, 3]))  # an empty group in front
    assert c.err == 0


@gpu
def test_shared_prefix_bad_data(L):
    b = Batch([(200, [(5, 1), (0, 1), (7, 1)]), (90, [(5, 1), (3, 1)])], 8, 2, 128, 16)
    for kw, status in [(dict(prefix=[-1, 90]), 1), (dict(starts=[0, 9, 5]), 1), (dict(starts=[-1, 3, 5]), 1),
                       (dict(starts=[0, 3, 2]), 1), (dict(starts=[3, 2, 5]), 1)]:
        out, lse = b.run(L, **kw)
        assert b.err == status, kw
        b.check(out, lse)  # such a group shares nothing
    lens = list(b.lens)
    lens[1] = 1 << 26
    out, lse = b.run(L, lens=lens)
    assert b.err == 1
    b.check(out, lse, skip=[1])
    lens[1] = -3
    out, lse = b.run(L, lens=lens)
    assert b.err == 1
    b.check(out, lse, skip=[1])
    # a page of the prefix that does not exist: its keys and values read as zeros
    c = Batch([(200, [(5, 1), (0, 1), (7, 1)])], 8, 2, 128, 16)
    page = c.table[0, 3]
    c.table[:, 3] = 1 << 30
    out, lse = c.run(L)
    assert c.err == 4
    c.table[:, 3] = page
    c.dk[int(page)], c.dv[int(page)] = 0, 0
    c.check(out, lse)


@gpu
def test_shared_prefix_unseen_cache_is_not_used(L):
    """What the cache holds behind a request's last token, in free pages and out of every row's window."""
    torch = _torch()
    b = Batch([(200, [(5, 1), (0, 1), (30, 1)]), (64, [(0, 1), (1, 1)])], 8, 2, 128, 16)
    used = np.zeros(b.k.shape[:2], bool)
    for i, n in enumerate(b.lens):
        j = np.arange(n)
        used[b.table[i, j // 16], j % 16] = True
    mask = torch.from_numpy(~used).cuda()
    b.dk[mask], b.dv[mask] = math.nan, math.nan
    b.check(*b.run(L))
    w = Batch([(400, [(5, 1), (0, 1), (30, 1)])], 8, 2, 128, 16)
    page = torch.from_numpy(w.table[0, :8].astype(np.int64)).cuda()
    w.dk[page], w.dv[page] = math.nan, math.inf  # keys 0..127: beyond a window of 250 of every row
    w.check(*w.run(L, window=250), window=250)


@gpu
def test_shared_prefix_long_cache_and_repeats(L):
    """A prefix over many parts; results are the same bits over runs; a captured call."""
    torch = _torch()
    b = Batch([(20000, [(c, 1) for c in (0, 9, 400, 31)])], 8, 2, 64, 64)
    out, lse = b.run(L)
    b.check(out, lse)
    for _ in range(3):
        again = b.run(L, repeat=2)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    kv = L.PagedKV(b.dk, b.dv, *b.scales)
    att = L.SharedAttention(b.n, b.rows, b.H, kv)
    args = [b.dq, torch.zeros_like(out), dev(np.concatenate([[0], np.cumsum(b.new)])), dev(b.lens), dev(b.table),
            dev(b.starts), dev(b.prefix), 0, None, None, "always"]
    att.run(*args)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        att.run(*args)
        att.run(*args)
    for _ in range(3):
        args[1].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(args[1], out)


@gpu
def test_shared_workspace_over_calls_of_other_sizes(L):
    """One workspace, made for the largest, over batches of other shapes and rows."""
    torch = _torch()
    shapes = [GROUPS["large"], GROUPS["pair"], GROUPS["spec"], GROUPS["samples"]]
    batches = [Batch(g, 8, 2, 128, 16, seed=i) for i, g in enumerate(shapes)]
    top = max(b.rows for b in batches)
    kv = L.PagedKV(batches[0].dk, batches[0].dv)
    att = L.SharedAttention(max(b.n for b in batches), top, 8, kv)
    for b in batches * 2:
        b.check(*b.run(L, att=att))
        assert b.err == 0


def check_against_each(L, b, out, lse):
    """What lora_attend gives, every request on its own: roundings of both outputs, 2^-8 each, and of the prefix's weights,
    2^-8 of max |v| < 6."""
    torch = _torch()
    kv = L.PagedKV(b.dk, b.dv, *b.scales)
    att = L.Attention(b.n, b.rows, b.H, kv)
    ref, ref_lse = torch.full_like(out, 7.0), torch.full_like(lse, 7.0)
    att.run(b.dq, ref, dev(np.concatenate([[0], np.cumsum(b.new)])), dev(b.lens), dev(b.table), max(b.new), lse=ref_lse)
    torch.cuda.synchronize()
    assert (out.float() - ref.float()).abs().max() <= 3 * 6 * 2.0 ** -8
    # sums of a few thousand terms in another order
    assert (lse - ref_lse).abs().max() <= 2.0 ** -16 * ref_lse.abs().max()


@gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_shared_prefix_of_many_groups(L, fp8):
    """1,200 requests in 300 groups, many pieces a block; groups of one and of no rows between them."""
    rng = np.random.default_rng(7)
    groups = [(int(rng.integers(0, 300)), [(int(rng.integers(0, 9)), int(rng.integers(0, 3))) for _ in range(g % 8)])
              for g in range(300)]
    b = Batch(groups, 4, 2, 64, 16, fp8, seed=1)
    out, lse = b.run(L)
    assert b.err == 0
    check_against_each(L, b, out, lse)


@gpu
@pytest.mark.parametrize("groups", [[(9000, [(c, 1) for c in range(0, 320, 5)])], [(9000, [(3, 1)] * 3), (40, [(5, 1)] * 60)],
                                    [(2500, [(c, 1) for c in range(4)])] * 16])
def test_shared_prefix_decided_on_the_device(L, groups):
    """Tables long enough for prefixes worth sharing: shared beside the own keys, some of it, in turn."""
    b = Batch(groups, 16, 4, 64, 64, seed=3)
    out, lse = b.run(L, share="auto", repeat=2)
    assert b.err == 0
    check_against_each(L, b, out, lse)
    again = b.run(L, share="auto")
    assert _torch().equal(out, again[0]) and _torch().equal(lse, again[1])
    b.starts[-1] = b.n + 1  # groups out of range are reported on this way too
    b.run(L, share="auto")
    assert b.err == 1


@gpu
@pytest.mark.parametrize("share", ["always", "auto"])
def test_shared_prefix_reads_what_the_kernels_before_wrote(L, share):
    """Queries, lengths, tables and caches written on the stream right before each call, without a wait; two streams
    with a workspace each at once.  Every call must give what it gives alone."""
    torch = _torch()
    steps = [Batch([(300 + 40 * i, [(c, 1) for c in (i, 9, 40, 3 * i)]), (64, [(i, 1), (0, 1)])], 8, 2, 128, 16, seed=i)
             for i in range(6)]
    pages, width = max(b.dk.shape[0] for b in steps), max(b.table.shape[1] for b in steps)
    alone = [b.run(L, share=share) for b in steps]

    def room():
        k, v = (torch.zeros(pages, 16, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        n, T = steps[0].n, steps[0].rows
        i32 = dict(dtype=torch.int32, device="cuda")
        kv = L.PagedKV(k, v)
        return dict(kv=kv, k=k, v=v, q=torch.zeros(T, 1024, dtype=torch.bfloat16, device="cuda"), lens=torch.zeros(n, **i32),
                    table=torch.zeros(n, width, **i32), prefix=torch.zeros(2, **i32), starts=dev(steps[0].starts),
                    off=dev(np.arange(n + 1)), att=L.SharedAttention(n, T, 8, kv), stream=torch.cuda.Stream())

    rooms = [room(), room()]
    inputs = [(b.dk, b.dv, b.dq, dev(b.lens), dev(np.pad(b.table, ((0, 0), (0, width - b.table.shape[1])))), dev(b.prefix))
              for b in steps]
    torch.cuda.synchronize()
    got = [[], []]
    for turn in range(5):
        for s, r in enumerate(rooms):
            with torch.cuda.stream(r["stream"]):
                for i, (k, v, q, lens, table, prefix) in enumerate(inputs):
                    r["k"].zero_()
                    r["k"][:k.shape[0]].copy_(k)
                    r["v"][:v.shape[0]].copy_(v)
                    r["table"].copy_(table)
                    r["prefix"].copy_(prefix)
                    r["lens"].copy_(lens)
                    r["q"].copy_(q)
                    out = torch.zeros_like(q)
                    r["att"].run(r["q"], out, r["off"], r["lens"], r["table"], r["starts"], r["prefix"], share=share)
                    got[s].append((i, out))
    torch.cuda.synchronize()
    for s, r in enumerate(rooms):
        assert int(r["att"].err) == 0
        for i, out in got[s]:
            assert torch.equal(out, alone[i][0]), (s, i)


@gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_shared_prefix_of_many_million_keys(L, fp8):
    """A prefix of 2^24 keys whose table names one page over and over: pieces of more than 512 steps, added up in fp32.
    Products on tensor cores lose 2^-24 of what they add to with every 16 keys, below 2^-11 of 65,536 keys."""
    torch = _torch()
    rng = np.random.default_rng(8)
    H, hd, ps, repeats = 4, 64, 1024, 1 << 14
    dtype, scales = (torch.float8_e4m3fn, (0.5, 0.25)) if fp8 else (torch.bfloat16, (1.0, 1.0))
    k, v = (torch.from_numpy(rng.standard_normal((3, ps, 1, hd))).float().to(dtype).cuda() for _ in range(2))
    kv = L.PagedKV(k, v, *scales)
    q = torch.from_numpy(rng.standard_normal((3, H * hd))).cuda().bfloat16()
    table = np.zeros((2, repeats + 1), np.int32)
    table[:, -1] = [1, 2]
    prefix, own = repeats * ps, [7, 1000]
    att = L.SharedAttention(2, 3, H, kv)
    out, lse = torch.empty_like(q), torch.empty(3, H, device="cuda")
    att.run(q, out, dev([0, 1, 3]), dev([prefix + n for n in own]), dev(table), dev([0, 2]), dev([prefix]), 2, lse=lse,
            share="always")
    torch.cuda.synchronize()
    assert int(att.err) == 0
    kk, vv, x = k.double().cpu().numpy() * scales[0], v.double().cpu().numpy() * scales[1], q.double().cpu().numpy()
    for t, (i, seen) in enumerate([(0, 7), (1, 999), (1, 1000)]):
        for h in range(H):
            one = x[t, h * hd:(h + 1) * hd]
            s0, s1 = kk[0, :, 0] @ one * hd ** -0.5, kk[1 + i, :seen, 0] @ one * hd ** -0.5
            top = max(s0.max(), s1.max())
            e0, e1 = repeats * np.exp(s0 - top), np.exp(s1 - top)
            total = e0.sum() + e1.sum()
            ref = (e0 @ vv[0, :, 0] + e1 @ vv[1 + i, :seen, 0]) / total
            A = (e0 @ np.abs(vv[0, :, 0]) + e1 @ np.abs(vv[1 + i, :seen, 0])) / total
            eps = 2.0 ** -18 * (1 + np.abs(s0).max())
            got = out[t, h * hd:(h + 1) * hd].double().cpu().numpy()
            assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -11 + 2 * eps) * A).all(), (t, h)
            want = top + math.log(total)
            assert abs(float(lse[t, h]) - want) <= 2.0 ** -18 * (1 + abs(want)) + 2.0 ** -16


# ---------------------------------------------------------------------------
# A run of them together
# ---------------------------------------------------------------------------
@gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_beams_over_a_paged_cache(L, fp8):
    """Steps of beam search, two layers: select, fork, copy, step, rotary append, shared attention, a compaction on
    the way.  Every beam's attention must be what the dense history of its own tokens gives."""
    torch = _torch()
    H, KV, hd, ps, V, n_req, beams, n_pages = 4, 2, 64, 16, 200, 3, 4, 120
    rng = np.random.default_rng(3)
    n, dtype = n_req * beams, torch.float8_e4m3fn if fp8 else torch.bfloat16
    embed = torch.from_numpy(rng.standard_normal((V, 2, (H + 2 * KV) * hd))).cuda().bfloat16()
    head = torch.from_numpy(rng.standard_normal((H * hd, V))).cuda().float() * 0.3
    kvs = [L.PagedKV.empty(n_pages, ps, KV, hd, dtype=dtype, k_scale=0.05, v_scale=0.05) for _ in range(2)]
    for kv in kvs:
        kv.k.view(torch.uint8).zero_()
        kv.v.view(torch.uint8).zero_()
    layers, rope = L.KVLayers(kvs), L.Rope(hd)
    tables = L.PageTables(n, 8, ps, n_pages)
    select = L.BeamSelect(n_req, beams, beams, V, eos=5)
    prompts = [rng.integers(0, V, int(m)).tolist() for m in (37, 16, 50)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    histories = None

    def step(tokens, groups, prefix):
        """One step of all rows with `tokens` (a list a row); the second layer's attention of each row's last token."""
        m = [len(t) for t in tokens]
        T = sum(m)
        st = L.KVStep(len(m), T, 8, ps)
        st.block_table = tables.block_table
        st.build(tables.lens.contiguous(), dev(m), tables.free_pages)
        x = embed[dev(sum(tokens, []), torch.int64)]
        out = torch.empty(T, H * hd, dtype=torch.bfloat16, device="cuda")
        for i, kv in enumerate(kvs):
            q = torch.empty(T, H * hd, dtype=torch.bfloat16, device="cuda")
            rope.append(x[:, i].contiguous(), q, H, kv, st.positions, st.slot_map, st.err)
            att = L.SharedAttention(len(m), T, H, kv)
            att.run(q, out, st.q_offsets, st.kv_lens, st.block_table, dev(groups), dev(prefix), max(m),
                    share="always" if i else "auto")
            torch.cuda.synchronize()
            assert int(att.err) == 0 and int(st.err) == 0
        tables.lens.copy_(st.kv_lens)
        ends = np.cumsum(m) - 1
        ends = dev(ends, torch.int64)
        return out[ends], q[ends].double().cpu().numpy().reshape(len(m), H, hd)

    def check(i, history, got, q):
        """Row i: its pages hold its own tokens' keys and values, up to their rounding; its attention over them."""
        x = embed[dev(history, torch.int64)].double().cpu().numpy()[:, 1].reshape(len(history), H + 2 * KV, hd)
        pos = np.arange(len(history))
        z = np.exp(1j * pos[:, None] * 10000.0 ** (-np.arange(0, hd, 2) / hd))[:, None]
        w = (x[:, H:H + KV, :hd // 2] + 1j * x[:, H:H + KV, hd // 2:]) * z
        kv, row = kvs[1], tables.block_table[i].cpu().numpy()
        at = (torch.from_numpy(row[pos // ps].astype(np.int64)).cuda(), torch.from_numpy(pos % ps).cuda())
        scale = 0.05 if fp8 else 1.0
        k, v = ((t[at].double().cpu().numpy() * scale) for t in (kv.k, kv.v))
        # half a step of the type, and 2^-18 of fp32 angles and products, which may move a value over a border
        step_ = 2.0 ** -3 if fp8 else 2.0 ** -7
        for t, ref in ((k, np.concatenate([w.real, w.imag], -1)), (v, x[:, H + KV:])):
            assert (np.abs(t - ref) <= step_ * np.abs(ref) + scale * 2.0 ** -9).all(), i
        for h in range(H):
            s = k[:, h // (H // KV)] @ q[h] * hd ** -0.5
            p = np.exp(s - s.max()) / np.exp(s - s.max()).sum()
            ref, A = p @ v[:, h // (H // KV)], p @ np.abs(v[:, h // (H // KV)])
            eps = 2.0 ** -18 * (1 + np.abs(s).max())
            assert (np.abs(got[h] - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2 * eps) * A + 2.0 ** -20).all(), (i, h)

    tables.fork(dev([-1] * n_req))          # three empty requests
    prompt_out, _ = step(prompts, list(range(n_req + 1)), [0] * n_req)
    first = L.BeamSelect(n_req, 1, beams, V)
    first.run((prompt_out.float() @ head).contiguous().bfloat16(), torch.zeros(n_req, device="cuda"))
    parents, tokens, scores = first.parents, first.tokens, first.scores.clone()
    ended = torch.zeros(n, dtype=torch.int32, device="cuda")
    histories = [list(p) for p in prompts]
    for it in range(6):
        tables.fork(parents)
        layers.copy(tables.copies, err)
        if it == 3:
            tables.compact()
            layers.copy(tables.copies, err, tables.n_copies)
        new = tokens.cpu().tolist()
        histories = [histories[p] + [t] for p, t in zip(parents.cpu().tolist(), new)]
        out, q = step([[t] for t in new], [beams * i for i in range(n_req + 1)], [len(p) for p in prompts])
        got = out.double().cpu().numpy().reshape(n, H, hd)
        for i, hist in enumerate(histories):
            check(i, hist, got[i], q[i])
        select.run((out.float() @ head).contiguous().bfloat16(), scores, ended)
        parents, tokens = select.parents.clone(), select.tokens.clone()
        scores, ended = select.scores.clone(), select.ended.clone()
    torch.cuda.synchronize()
    assert int(err) == 0 and int(tables.err) == 0
    # what is free and what the rows hold are all pages
    held = {int(p) for row, m in zip(tables.block_table.cpu().numpy(), tables.lens.tolist()) for p in row[:-(-m // ps)]}
    tables.fork(dev(list(range(n))))
    free = tables.free_pages.cpu().numpy()[:int(tables.n_free)]
    assert not held & set(free.tolist()) and len(held) + len(free) == n_pages
