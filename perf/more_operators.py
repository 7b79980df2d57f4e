"""Cases and plain forms of the operators for requests that share what they have cached.

Five operators of parallel samples, beams and shared system prompts, used in a row with the step tables, the rotary
append and the attention of one serving step:

  select   the best continuations of each request over its beams and the vocabulary
  fork     the next batch's block tables from the parents of its rows, pages that come free, copies on write
  compact  block tables after the pages in use have moved to the front of the cache
  copy     the pages' data, all layers
  attend   attention in which a prefix that a group of requests shares is read once for all of them

Where `own` is false, run() computes them with elementary torch operations in 32 bits, rounded once at the end
(64 bits for the log-probabilities that select compares); where it is true, with the package's entry points.
exact() computes them in 64 bits, request by request.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


# ---------------------------------------------------------------------------------------------------------------
# The cases
# ---------------------------------------------------------------------------------------------------------------
def _select(name, n, beams, keep, V, fp32, ended, mix):
    return {"name": name, "op": "select", "n": n, "beams": beams, "keep": keep, "V": V, "fp32": fp32, "ended": ended,
            "mix": mix}


def _fork(name, n, out, ctx, ps, share, held, mix):
    return {"name": name, "op": "fork", "n": n, "out": out, "ctx_lo": ctx[0], "ctx_hi": ctx[1], "ps": ps,
            "share": share, "held": held, "mix": mix}


def _compact(name, n, ctx, ps, share, held, spread, mix):
    return {"name": name, "op": "compact", "n": n, "ctx_lo": ctx[0], "ctx_hi": ctx[1], "ps": ps, "share": share,
            "held": held, "spread": spread, "mix": mix}


def _copy(name, jobs, layers, KV, hd, ps, fp8, head_major, whole, mix):
    return {"name": name, "op": "copy", "jobs": jobs, "layers": layers, "KV": KV, "hd": hd, "ps": ps, "fp8": fp8,
            "head_major": head_major, "whole": whole, "mix": mix}


def _attend(name, groups, size, prefix, ctx, q, H, KV, hd, ps, mix, fp8=False, softcap=0.0, window=0, alibi=False,
            head_major=True, packed=False):
    return {"name": name, "op": "attend", "groups": groups, "size_lo": size[0], "size_hi": size[1],
            "pre_lo": prefix[0], "pre_hi": prefix[1], "ctx_lo": ctx[0], "ctx_hi": ctx[1], "q_lo": q[0], "q_hi": q[1],
            "H": H, "KV": KV, "hd": hd, "ps": ps, "mix": mix, "fp8": fp8, "softcap": softcap, "window": window,
            "alibi": alibi, "head_major": head_major, "packed": packed}


def listed():
    return [
        # one request's 4 beams, fp32 logits of a small vocabulary: the latency of a beam step
        _select("select_1x4", 1, 4, 4, 32000, True, 0.0, 1),
        # 32 requests of 4 beams, twice as many continuations as beams, some beams ended
        _select("select_32x4", 32, 4, 8, 128256, False, 0.1, 2),
        # the tables of 32 requests of 4 beams after a selection
        _fork("fork_beams_128", 128, 128, (100, 4000), 16, 4, 0, 3),
        # a full batch of 1,024 rows in which some requests end and others branch
        _fork("fork_batch_1024", 1024, 1000, (1, 16000), 16, 8, 100, 4),
        # a small batch after its neighbours have left
        _compact("compact_16", 16, (1, 2000), 32, 2, 0, 3.0, 5),
        # a full batch's pages moved to the front of a cache of twice their number
        _compact("compact_1024", 1024, (1, 16000), 16, 4, 50, 2.0, 6),
        # one branch of one request: part of a page in each of 4 layers
        _copy("copy_1", 1, 4, 8, 128, 16, False, True, False, 7),
        # the copies of 96 branching beams in all 32 layers
        _copy("copy_beams_96x32", 96, 32, 8, 128, 16, False, True, False, 8),
        # 4 samples of one short prompt: latency
        _attend("samples_1x4", 1, (4, 4), (500, 500), (0, 200), (1, 1), 32, 8, 128, 16, 9),
        # 64 requests behind one system prompt, Llama-3-8B heads
        _attend("system_prompt_64", 1, (64, 64), (8000, 8000), (100, 1000), (1, 1), 32, 8, 128, 16, 10),
        # 32 requests of 1 to 4 beams with 4 speculative rows each, FP8 cache, capped scores, a sliding window, 64-wide heads
        _attend("beams_32x4_fp8", 32, (1, 4), (200, 6000), (0, 100), (4, 4), 16, 4, 64, 32, 11, fp8=True, softcap=30.0,
                window=4096),
        # 16 prompts of up to 30,000 tokens with 16 samples each: the largest
        _attend("samples_16x16_long", 16, (16, 16), (20000, 30000), (10, 2000), (1, 1), 32, 8, 128, 64, 12),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(("select", "fork", "compact", "copy", "attend", "attend", "attend"))
    mix, ps = rng.randrange(1 << 30), rng.choice((16, 32, 64, 128))
    if kind == "select":
        beams = _log(rng, 1, 16)
        keep = min(32, rng.choice((beams, 2 * beams, _log(rng, 1, 32))))
        V = _log(rng, 100, 131072)
        c = _select("", _log(rng, 1, max(1, min(128, 30000000 // (beams * V)))), beams, keep, V, rng.random() < 0.3,
                    rng.choice((0.0, 0.2)), mix)
    elif kind == "fork":
        n = _log(rng, 1, 1024)
        hi = _log(rng, 1, 16000)
        c = _fork("", n, max(1, int(n * rng.choice((1.0, 1.0, 0.5, 1.9)))), (hi // rng.choice((1, 5, 50)), hi), ps,
                  rng.choice((1, 4, 16)), rng.choice((0, _log(rng, 1, 300))), mix)
    elif kind == "compact":
        hi = _log(rng, 1, 16000)
        c = _compact("", _log(rng, 1, 1024), (hi // rng.choice((1, 5, 50)), hi), ps, rng.choice((1, 4, 16)),
                     rng.choice((0, _log(rng, 1, 300))), rng.choice((1.0, 1.1, 2.0, 6.0)), mix)
    elif kind == "copy":
        KV, hd, layers = rng.choice((1, 2, 8)), rng.choice((64, 128)), _log(rng, 1, 48)
        fp8 = rng.random() < 0.4
        most = max(1, 150000000 // (layers * KV * hd * ps * (2 if fp8 else 4)))
        c = _copy("", _log(rng, 1, min(500, most)), layers, KV, hd, ps, fp8, rng.random() < 0.6, rng.random() < 0.3,
                  mix)
    else:
        hd, KV, G = rng.choice((64, 128)), rng.choice((1, 2, 4, 8)), rng.choice((1, 3, 4, 8))
        groups = _log(rng, 1, 64)
        size = _log(rng, 1, max(1, 256 // groups))
        prefix = _log(rng, 1, min(60000, 300000 // groups))
        q = rng.choice((1, 1, 1, 2, 4, 7))
        c = _attend("", groups, (max(1, size // rng.choice((1, 1, 4))), size),
                    (prefix // rng.choice((1, 2, 30)), prefix), (0, _log(rng, 1, min(4000, 400000 // (groups * size)))),
                    (1 if rng.random() < 0.5 else q, q), KV * G, KV, hd, ps, mix, fp8=rng.random() < 0.4,
                    softcap=rng.choice((0.0, 0.0, 30.0)), window=rng.choice((0, 0, 0, _log(rng, 16, 8192))),
                    alibi=rng.random() < 0.25, head_major=rng.random() < 0.6, packed=rng.random() < 0.5)
        while work(c)["flops"] > 1e11:
            c["pre_lo"], c["pre_hi"] = c["pre_lo"] // 2, c["pre_hi"] // 2
    del c["name"]
    return c


# ---------------------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------------------
def _lengths(case, n, lo, hi, salt):
    """n lengths spread over the logarithm; from the case alone."""
    rng = random.Random(case["mix"] * 31 + salt)
    return [lo if lo == hi else int(math.exp(rng.uniform(math.log(lo + 1), math.log(hi + 1.999)))) - 1
            for _ in range(n)]


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 29)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _int(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype).to(DEV)


def _up(a, b):
    return -(-a // b)


def _tables(case, g):
    """Rows of a batch in which `share` neighbours at a time begin with the same full pages, and ids for them out of
    a cache with `spread` times as many pages: (rows, lengths, number of pages, held ids)."""
    n, ps, rng = case["n"], case["ps"], random.Random(case["mix"])
    lens = _lengths(case, n, case["ctx_lo"], case["ctx_hi"], 1)
    have = np.array([_up(x, ps) for x in lens])
    width = max(1, int(have.max())) + 1
    first = np.arange(n) // case["share"] * case["share"]
    full = np.array(lens) // ps
    common = np.array([min(full[i], full[f]) * rng.random() if i != f else 0 for i, f in enumerate(first)]).astype(int)
    new = have - common
    at = np.concatenate([[0], np.cumsum(new)])
    entry = np.arange(width)[None]
    rows = at[:-1, None] + entry - common[:, None]
    rows = np.where(entry < common[:, None], at[first][:, None] + entry - common[first][:, None], rows)
    used, held = int(at[-1]), case["held"]
    n_pages = max(1, int((used + held) * case.get("spread", 1.3))) + 8 + case.get("out", 0)
    ids = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    rows = torch.from_numpy(np.where(entry < have[:, None], rows, 0)).to(DEV)
    table = torch.where(torch.from_numpy(entry < have[:, None]).to(DEV), ids[rows], -1).to(torch.int32)
    return table, lens, n_pages, ids[used:used + held].contiguous()


def _parents(case):
    """Who each row of the next batch continues: neighbours of `share` rows compete, some rows start anew."""
    n, out, share = case["n"], case["out"], case["share"]
    rng = random.Random(case["mix"] + 1)
    got = []
    for i in range(out):
        lo = min(n - 1, i * n // out // share * share)
        got.append(-1 if rng.random() < 0.02 else rng.randrange(lo, min(n, lo + share)))
    return got


def _jobs(case):
    """(source, destination, tokens) of each copy, out of a cache of `pages` pages; some rows have none."""
    rng, n = random.Random(case["mix"]), case["jobs"]
    pages = 2 * n + 8
    ids = rng.sample(range(pages - 1), 2 * n)  # the last page stays free
    jobs = [(ids[2 * i], ids[2 * i + 1], case["ps"] if case["whole"] else rng.randrange(1, case["ps"]))
            for i in range(n)]
    return [(-1, -1, 0) if n > 4 and rng.random() < 0.05 else j for j in jobs], pages


def _sizes(case):
    rng = random.Random(case["mix"] + 2)
    return [rng.randint(case["size_lo"], case["size_hi"]) for _ in range(case["groups"])]


def _prompt(case):
    """Requests of each group, prefix of each group, own tokens and rows of each request."""
    sizes = _sizes(case)
    return (sizes, _lengths(case, case["groups"], case["pre_lo"], case["pre_hi"], 3),
            _lengths(case, sum(sizes), case["ctx_lo"], case["ctx_hi"], 1),
            _lengths(case, sum(sizes), case["q_lo"], case["q_hi"], 2))


def _slopes(H):
    return [2.0 ** (-8.0 * (h + 1) / H) for h in range(H)]


def _fill(g, shape, dtype, shift):
    t = torch.empty(shape, dtype=dtype, device=DEV)
    part = max(1, (1 << 28) // math.prod(shape[1:]))
    for a in range(0, shape[0], part):
        t[a:a + part] = (_randn(g, min(part, shape[0] - a), *shape[1:]) + shift).to(dtype)
    return t


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if own:
        import rank_adapter_gemm_gb300 as L
    if case["op"] == "select":
        n, beams, V = case["n"], case["beams"], case["V"]
        dtype = torch.float32 if case["fp32"] else BF16
        # a language model's logits: a long flat part and a few tokens that stand out
        x = _randn(g, n * beams, V).mul_(1.5)
        top = torch.randint(0, V, (n * beams, 12), generator=g, device=DEV)
        x.scatter_add_(1, top, 6.0 + 2.0 * _randn(g, n * beams, 12))
        s["logits"] = x.to(dtype)
        s["scores"] = -5.0 * torch.rand(n * beams, generator=g, device=DEV)
        s["ended"] = (torch.rand(n * beams, generator=g, device=DEV) < case["ended"]).to(torch.int32)
        s["eos"] = V // 3
        if own:
            s["select"] = L.BeamSelect(n, beams, case["keep"], V, eos=s["eos"], dtype=dtype, device=DEV)
        return s
    if case["op"] in ("fork", "compact"):
        s["rows"], lens, s["n_pages"], s["held"] = _tables(case, g)
        s["lens"] = _int(lens)
        n = case["out"] if case["op"] == "fork" else case["n"]
        s["new_rows"] = torch.full((n, s["rows"].shape[1]), -1, dtype=torch.int32, device=DEV)
        if case["op"] == "fork":
            s["parents"] = _int(_parents(case))
        if own:
            i32 = dict(dtype=torch.int32, device=DEV)
            s |= {"new_lens": torch.empty(n, **i32), "free": torch.empty(s["n_pages"], **i32),
                  "n_free": torch.empty(1, **i32), "err": torch.zeros(1, **i32),
                  "copies": torch.empty(n if case["op"] == "fork" else s["n_pages"] // 2, 3, **i32),
                  "n_copies": torch.empty(1, **i32), "new_held": torch.empty_like(s["held"])}
        return s
    if case["op"] == "copy":
        jobs, pages = _jobs(case)
        KV, ps, hd = case["KV"], case["ps"], case["hd"]
        shape = (case["layers"] * pages, KV, ps, hd) if case["head_major"] else (case["layers"] * pages, ps, KV, hd)
        for name in ("k", "v"):
            t = _fill(g, shape, E4M3 if case["fp8"] else BF16, 0.0)
            t = t.view(case["layers"], pages, *shape[1:])
            s[name] = t.transpose(2, 3) if case["head_major"] else t
        s["copies"] = _int(jobs)
        if own:
            s["err"] = torch.zeros(1, dtype=torch.int32, device=DEV)
            s["cache"] = L.KVLayers([L.PagedKV(s["k"][i], s["v"][i]) for i in range(case["layers"])])
        return s
    H, KV, hd, ps = (case[k] for k in ("H", "KV", "hd", "ps"))
    sizes, prefix, ctx, new = _prompt(case)
    n, T, G = sum(sizes), sum(new), len(sizes)
    group = np.repeat(np.arange(G), sizes)
    starts = np.concatenate([[0], np.cumsum(sizes)])
    lens = np.array(prefix)[group] + ctx + new
    pages = -(-lens // ps)
    common = np.array(prefix)[group] // ps
    common[starts[:-1]] = 0  # a group's first request brings the shared pages
    at = np.concatenate([[0], np.cumsum(pages - common)])
    n_pages, width = int(at[-1]) + 1, int(pages.max())
    entry = np.arange(width)[None]
    first = starts[group]
    rows = np.where(entry < common[:, None], at[first][:, None] + entry, at[:-1, None] + entry - common[:, None])
    ids = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    rows = np.where(entry < pages[:, None], rows, 0)
    s["rows"] = ids[torch.from_numpy(rows).to(DEV)].contiguous()
    dtype = E4M3 if case["fp8"] else BF16
    shape = (n_pages, KV, ps, hd) if case["head_major"] else (n_pages, ps, KV, hd)
    # a page that the prefix ends in is each request's own, with the same tokens in front
    ends = np.array(prefix)[group]
    part = [(int(rows[i, ends[i] // ps]), int(rows[first[i], ends[i] // ps]), int(ends[i] % ps)) for i in range(n)
            if i != first[i] and ends[i] % ps]
    for name, shift in (("k", 0.0), ("v", 0.1)):
        t = _fill(g, shape, dtype, shift)
        t = t.transpose(1, 2) if case["head_major"] else t
        flat = t.view(torch.uint8) if case["fp8"] else t
        for off in range(ps if part else 0):
            pair = [(a, b) for a, b, m in part if off < m]
            if pair:
                a, b = (ids[_int(x, torch.int64)].long() for x in zip(*pair))
                flat[a, off] = flat[b, off]
        s[name] = t
    s["k_scale"], s["v_scale"] = (0.5, 0.25) if case["fp8"] else (1.0, 1.0)
    ld = (H + 2 * KV) * hd if case["packed"] else H * hd
    # rows of a packed projection, or rows of q alone; the heads differ in how sharply they look
    sharp = torch.linspace(0.5, 2.0, H, device=DEV).repeat_interleave(hd)
    s["q"] = (_randn(g, T, ld).to(BF16))[:, :H * hd]
    s["q"].mul_(sharp.to(BF16))
    s |= {"lens": _int(lens.tolist()), "q_offsets": _int(np.concatenate([[0], np.cumsum(new)]).tolist()),
          "groups": _int(starts.tolist()), "prefix": _int(prefix), "T": T, "scale": hd ** -0.5,
          "slopes": _int(_slopes(H), torch.float32) if case["alibi"] else None}
    if own:
        kv = L.PagedKV(s["k"], s["v"], s["k_scale"], s["v_scale"])
        s["attention"] = L.SharedAttention(n, T, H, kv, scale=s["scale"], softcap=case["softcap"],
                                           window=case["window"], slopes=s["slopes"], device=DEV)
        s["out"] = torch.empty(T, H * hd, dtype=BF16, device=DEV)
        s["lse"] = torch.empty(T, H, dtype=torch.float32, device=DEV)
    return s


# ---------------------------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------------------------
def _plain_select(s):
    c = s["case"]
    n, beams, keep, V = (c[k] for k in ("n", "beams", "keep", "V"))
    x = s["logits"].double()
    top = x.amax(1, keepdim=True)
    x = x - (top + torch.exp(x - top).sum(1, keepdim=True).log())
    ended = s["ended"].bool()[:, None]
    is_eos = (torch.arange(V, device=x.device) == s["eos"])[None]
    x = torch.where(ended, torch.where(is_eos, 0.0, -math.inf), x) + s["scores"].double()[:, None]
    value, at = torch.sort(x.view(n, beams * V), dim=1, descending=True, stable=True)
    value, at = value[:, :keep], at[:, :keep]
    if value.shape[1] < keep:
        more = (0, keep - value.shape[1])
        value = torch.nn.functional.pad(value, more, value=-math.inf)
        at = torch.nn.functional.pad(at, more)
    there = value > -math.inf
    parent = torch.arange(n, device=x.device)[:, None] * beams + at // V
    token = at % V
    over = there & (s["ended"].bool()[parent] | (token == s["eos"]))
    i32 = torch.int32
    return {"parents": torch.where(there, parent, -1).flatten().to(i32), "ended": over.flatten().to(i32),
            "tokens": torch.where(there, token, -1).flatten().to(i32), "scores": value.flatten().float()}


def _plain_used(s, rows, keep):
    """Truth values: which pages the kept entries and the held ids name."""
    used = torch.zeros(s["n_pages"] + 1, dtype=torch.bool, device=rows.device)
    used[torch.where(keep, rows.long(), s["n_pages"])] = True  # (one place more takes the others)
    used[s["held"].long()] = True
    return used[:-1]


def _plain_fork(s):
    c, n_pages = s["case"], s["n_pages"]
    ps, out = c["ps"], c["out"]
    parents, i = s["parents"].long(), torch.arange(c["out"], device=DEV)
    ok, from_row = parents >= 0, parents.clamp(min=0)
    lens = torch.where(ok, s["lens"].long()[from_row], 0)
    have = (lens + ps - 1) // ps
    first = torch.full((c["n"],), out, device=DEV).scatter_reduce_(
        0, from_row, torch.where(ok, i, out), "amin")
    job = ok & (first[from_row] != i) & (lens % ps != 0)
    rows = s["rows"][from_row]
    entry = torch.arange(rows.shape[1], device=DEV)[None]
    used = _plain_used(s, rows, entry < (have - job.long())[:, None])
    free = torch.argsort(used.to(torch.uint8), stable=True)
    n_free = n_pages - used.sum() - job.sum()
    page = free[(torch.cumsum(job, 0) - 1).clamp(min=0)]
    last = (entry == have[:, None] - 1) & job[:, None]
    src = rows.long().gather(1, (have - 1).clamp(min=0)[:, None])[:, 0]
    table = torch.where(entry < have[:, None], torch.where(last, page[:, None], rows.long()), s["new_rows"].long())
    copies = torch.stack([torch.where(job, src, -1), torch.where(job, page, -1), torch.where(job, lens % ps, 0)], 1)
    f = torch.arange(n_pages, device=DEV)
    free = torch.where(f < n_free, free[(f + job.sum()).clamp(max=n_pages - 1)], -1)
    i32 = torch.int32
    return {"rows": table.to(i32), "lens": lens.to(i32), "copies": copies.to(i32), "free": free.to(i32),
            "n_free": n_free.reshape(1).to(i32)}


def _plain_compact(s):
    ps, n_pages = s["case"]["ps"], s["n_pages"]
    rows = s["rows"].long()
    there = torch.arange(rows.shape[1], device=DEV)[None] < ((s["lens"].long() + ps - 1) // ps)[:, None]
    used = _plain_used(s, rows, there)
    p, count = torch.arange(n_pages, device=DEV), used.sum()
    free = torch.argsort(used.to(torch.uint8), stable=True)
    moves = used & (p >= count)
    r = torch.cumsum(moves, 0) - 1
    new = torch.where(moves, free[r.clamp(min=0)], p)
    i = torch.arange(n_pages // 2, device=DEV)
    here = i < moves.sum()
    src = torch.argsort((~moves).to(torch.uint8), stable=True)[:n_pages // 2]
    copies = torch.stack([torch.where(here, src, -1), torch.where(here, free[:n_pages // 2], -1),
                          torch.where(here, ps, 0)], 1)
    i32 = torch.int32
    return {"rows": torch.where(there, new[rows.clamp(min=0)], s["new_rows"].long()).to(i32),
            "held": new[s["held"].long()].to(i32), "copies": copies.to(i32),
            "n_copies": moves.sum().reshape(1).to(i32), "n_free": (n_pages - count).reshape(1).to(i32),
            "free": torch.where(p < n_pages - count, p + count, -1).to(i32)}


def _plain_copy(s):
    ps = s["case"]["ps"]
    src, dst, tokens = s["copies"].long().unbind(1)
    # rows without a job write the last page, which no job names, back to itself
    spare = s["k"].shape[1] - 1
    off = torch.arange(ps, device=src.device)
    take = (src >= 0)[:, None] & (off[None] < tokens[:, None])
    src, dst = torch.where(src >= 0, src, spare), torch.where(dst >= 0, dst, spare)
    for x in (s["k"], s["v"]):
        for layer in (x.view(torch.uint8) if s["case"]["fp8"] else x):
            layer[dst] = torch.where(take[..., None, None], layer[src], layer[dst])
    return {"k": s["k"], "v": s["v"]}


def _plain_attend(s):
    c = s["case"]
    H, KV, hd, ps = (c[k] for k in ("H", "KV", "hd", "ps"))
    sizes, prefix, ctx, new = _prompt(c)
    G, w = H // KV, c["window"]
    out = torch.empty(s["T"], H, hd, device=DEV)
    lse = torch.empty(s["T"], H, device=DEV)
    first = row = 0
    for size, pre in zip(sizes, prefix):
        ids = range(first, first + size)
        m, own_len = [new[i] for i in ids], [ctx[i] + new[i] for i in ids]
        Q, S = max(m), max(own_len)
        i = torch.arange(Q, device=DEV)
        m_d, len_d = s["q_offsets"][first + 1:first + size + 1] - s["q_offsets"][first:first + size], s["lens"][first:first + size]
        at = s["q_offsets"][first:first + size, None] + i[None]
        q = s["q"][at.clamp(max=s["T"] - 1)].float().view(size, Q, KV, G, hd).permute(2, 0, 3, 1, 4)
        pos = (len_d - m_d)[:, None] + i[None]  # [size, Q]

        def part(keys, k, there):
            """scores [KV, size, G, Q, keys] of keys at the positions `keys` ([size or 1, keys])"""
            sc = (q.reshape(KV, size * G * Q, hd) @ k.transpose(-1, -2) if k.dim() == 3 else
                  q.reshape(KV, size, G * Q, hd) @ k.transpose(-1, -2)).view(KV, size, G, Q, -1) * s["scale"]
            if c["softcap"]:
                sc = torch.tanh(sc / c["softcap"]) * c["softcap"]
            away = keys[:, None] - pos[..., None]  # [size, Q, keys]
            if c["alibi"]:
                sc = sc + s["slopes"].view(KV, 1, G, 1, 1) * away[None, :, None].float()
            seen = (away <= 0) & there[:, None]
            if w:
                seen &= away > -w
            return sc.masked_fill(~seen[None, :, None], -math.inf)

        # the prefix, through the first request's row; then the requests' own tokens
        key = torch.arange(pre, device=DEV)
        pages = s["rows"][first][key // ps].long()
        k1, v1 = (s[x][pages, key % ps].float().transpose(0, 1) * s[x + "_scale"] for x in ("k", "v"))
        key2 = pre + torch.arange(S, device=DEV)
        there = key2[None] < len_d[:, None]
        pages = s["rows"][first:first + size].gather(1, (key2 // ps).clamp(max=s["rows"].shape[1] - 1)[None]
                                                     .expand(size, S)).long()
        k2, v2 = (torch.where(there[..., None, None], s[x][pages, key2 % ps].float(), 0.0).permute(2, 0, 1, 3) *
                  s[x + "_scale"] for x in ("k", "v"))
        s1 = part(key[None], k1, torch.ones(1, pre, dtype=torch.bool, device=DEV))
        s2 = part(key2[None], k2, there)
        top = s2.amax(-1)
        if pre:
            top = torch.maximum(top, s1.amax(-1))
        ref = torch.where(torch.isfinite(top), top, 0.0)[..., None]
        s1, s2 = torch.exp(s1 - ref), torch.exp(s2 - ref)
        total = s1.sum(-1) + s2.sum(-1)
        o = (s1.reshape(KV, size * G * Q, pre) @ v1).view(KV, size, G, Q, hd) + (
            s2.reshape(KV, size, G * Q, S) @ v2).view(KV, size, G, Q, hd)
        o = torch.where(total[..., None] > 0, o / total[..., None], 0.0)
        logs = torch.where(total > 0, ref[..., 0] + total.log(), -math.inf)
        o, logs = o.permute(1, 3, 0, 2, 4).reshape(size, Q, H, hd), logs.permute(1, 3, 0, 2).reshape(size, Q, H)
        if Q == 1:
            out[row:row + size], lse[row:row + size] = o[:, 0], logs[:, 0]
        else:
            for j, x in enumerate(m):
                a = row + sum(m[:j])
                out[a:a + x], lse[a:a + x] = o[j, :x], logs[j, :x]
        first, row = first + size, row + sum(m)
    return {"out": out.view(s["T"], H * hd).to(BF16), "lse": lse}


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"select": _plain_select, "fork": _plain_fork, "compact": _plain_compact, "copy": _plain_copy,
                "attend": _plain_attend}[c["op"]](s)
    if c["op"] == "select":
        sel = s["select"]
        sel.run(s["logits"], s["scores"], s["ended"])
        return {"parents": sel.parents, "ended": sel.ended, "tokens": sel.tokens, "scores": sel.scores}
    if c["op"] == "copy":
        s["cache"].copy(s["copies"], s["err"])
        return {"k": s["k"], "v": s["v"]}
    if c["op"] == "attend":
        s["attention"].run(s["q"], s["out"], s["q_offsets"], s["lens"], s["rows"], s["groups"], s["prefix"],
                           c["q_hi"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    import rank_adapter_gemm_gb300 as L
    if c["op"] == "fork":
        L.lora_kv_fork(s["rows"], s["lens"], s["parents"], c["ps"], s["new_rows"], s["new_lens"], s["copies"],
                       s["free"], s["n_free"], s["err"], held=s["held"])
        return {"rows": s["new_rows"], "lens": s["new_lens"], "copies": s["copies"], "free": s["free"],
                "n_free": s["n_free"]}
    L.lora_kv_compact(s["rows"], s["lens"], c["ps"], s["new_rows"], s["copies"], s["n_copies"], s["free"],
                      s["n_free"], s["err"], held=s["held"], new_held=s["new_held"])
    return {"rows": s["new_rows"], "held": s["new_held"], "copies": s["copies"], "n_copies": s["n_copies"],
            "n_free": s["n_free"], "free": s["free"]}


# ---------------------------------------------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------
def work(case):
    if case["op"] == "select":
        rows, V = case["n"] * case["beams"], case["V"]
        return {"bytes": rows * (V * (4 if case["fp32"] else 2) + 8) + 16 * case["n"] * case["keep"],
                "flops": 3 * rows * V}
    if case["op"] in ("fork", "compact"):
        n, ps = case["n"], case["ps"]
        have = [_up(x, ps) for x in _lengths(case, n, case["ctx_lo"], case["ctx_hi"], 1)]
        lists = 4 * sum(have)  # about the pages of the cache, a free list's length at most
        if case["op"] == "fork":
            parents = [p for p in _parents(case) if p >= 0]
            return {"bytes": 4 * (sum(have[p] for p in set(parents)) + sum(have[p] for p in parents)) + lists +
                    4 * (n + 5 * case["out"] + case["held"]), "flops": 0}
        return {"bytes": 8 * sum(have) + lists + 4 * (n + 2 * case["held"]), "flops": 0}
    if case["op"] == "copy":
        tokens = sum(t for _, _, t in _jobs(case)[0])
        return {"bytes": 4 * tokens * case["layers"] * case["KV"] * case["hd"] * (1 if case["fp8"] else 2) +
                12 * case["jobs"], "flops": 0}
    H, KV, hd, w = (case[k] for k in ("H", "KV", "hd", "window"))
    sizes, prefix, ctx, new = _prompt(case)
    pairs = keys = first = 0
    for size, pre in zip(sizes, prefix):
        seen = 0  # keys of the prefix that some row sees
        for i in range(first, first + size):
            see = np.arange(pre + ctx[i] + 1, pre + ctx[i] + new[i] + 1)
            pairs += int((np.minimum(see, w) if w else see).sum())
            lo = max(0, int(see[0]) - w) if w else 0
            seen = max(seen, pre - lo)
            keys += pre + ctx[i] + new[i] - max(lo, pre)
        keys += seen
        first += size
    T = sum(new)
    return {"bytes": keys * KV * hd * 2 * (1 if case["fp8"] else 2) + T * H * (4 * hd + 4) + 4 * keys // case["ps"],
            "flops": 4 * pairs * H * hd}


# ---------------------------------------------------------------------------------------------------------------
# In 64 bits
# ---------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "select":
        n, beams, keep, V = (case[k] for k in ("n", "beams", "keep", "V"))
        scores = torch.full((n, keep), -math.inf, dtype=torch.float64, device=DEV)
        for r in range(n):
            every = []
            for b in range(r * beams, (r + 1) * beams):
                if s["ended"][b]:
                    every.append(s["scores"][b:b + 1].double())
                else:
                    every.append(torch.log_softmax(s["logits"][b].double(), 0) + s["scores"][b].double())
            best = torch.cat(every).topk(min(keep, sum(len(e) for e in every))).values
            scores[r, :len(best)] = best
        return {"parents": None, "ended": None, "tokens": None, "scores": scores.flatten()}
    if case["op"] == "copy":
        out = {}
        for name in ("k", "v"):
            x = s[name].double().clone()
            for a, b, m in s["copies"].tolist():
                if a >= 0:
                    x[:, b, :m] = x[:, a, :m]
            out[name] = x
        return out
    if work(case)["flops"] > 3e12:
        return None
    H, KV, hd, ps = (case[k] for k in ("H", "KV", "hd", "ps"))
    sizes, _, _, new = _prompt(case)
    out = torch.zeros(s["T"], H, hd, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["T"], H, dtype=torch.float64, device=DEV)
    at = 0
    for r, (m, length) in enumerate(zip(new, s["lens"].tolist())):
        pages = s["rows"][r, :_up(length, ps)].long()  # every request through its own row
        lo = max(0, length - m + 1 - case["window"]) if case["window"] else 0
        where = torch.arange(lo, length, device=DEV)
        k, v = (s[x][pages[where // ps], where % ps].double().transpose(0, 1) * s[x + "_scale"] for x in ("k", "v"))
        pos = torch.arange(length - m, length, device=DEV)
        back = (pos[:, None] - where[None]).double()
        ok = back >= 0
        if case["window"]:
            ok &= back < case["window"]
        q = s["q"][at:at + m].double().view(m, KV, H // KV, hd).permute(1, 2, 0, 3)  # [KV, G, m, hd]
        y = (q.reshape(KV, H // KV * m, hd) @ k.transpose(1, 2)).view(KV, H // KV, m, -1) / math.sqrt(hd)
        if case["softcap"]:
            y = case["softcap"] * torch.tanh(y / case["softcap"])
        if case["alibi"]:
            y = y - torch.tensor(_slopes(H), dtype=torch.float64, device=DEV).view(KV, -1, 1, 1) * back
        y = torch.where(ok, y, torch.full_like(y, -math.inf))
        lse[at:at + m] = torch.logsumexp(y, -1).permute(2, 0, 1).reshape(m, H)
        o = torch.softmax(y, -1).reshape(KV, H // KV * m, len(where)) @ v
        out[at:at + m] = o.view(KV, H // KV, m, hd).permute(2, 0, 1, 3).reshape(m, H, hd)
        at += m
    return {"out": out.view(s["T"], H * hd), "lse": lse}
