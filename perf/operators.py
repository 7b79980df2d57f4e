"""Cases and plain forms of the attention-side operators of one serving step.

Four operators that run between the packed QKV projection (with its LoRA branch) and the output projection:

  step    block tables, slot map, positions and request ids of a step, from request lengths
  rope    rotary positions of q and k, q to its own rows, k and v into the paged cache
  attend  attention of few new tokens per request over the paged cache (decode, speculative decode)
  attend  the same over prompt chunks (causal over the chunk and everything cached before it)

Where `own` is false, run() computes them with elementary torch operations in 32 bits, rounded once at the end;
where it is true, with the package's entry points.  exact() computes them in 64 bits, request by request.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn
LLAMA3 = {"kind": "llama3", "factor": 8.0, "low_freq_factor": 1.0, "high_freq_factor": 4.0, "original": 8192}
YARN = {"kind": "yarn", "factor": 16.0, "beta_fast": 32.0, "beta_slow": 1.0, "original": 8192}
LINEAR = {"kind": "linear", "factor": 4.0}
SCALINGS = {"none": None, "linear": LINEAR, "llama3": LLAMA3, "yarn": YARN}


# ---------------------------------------------------------------------------------------------------------------
# The cases
# ---------------------------------------------------------------------------------------------------------------
def _step(name, n, ps, ctx, new, mix, pad=0):
    return {"name": name, "op": "step", "n": n, "ps": ps, "ctx_lo": ctx[0], "ctx_hi": ctx[1], "new_lo": new[0],
            "new_hi": new[1], "mix": mix, "pad": pad}


def _rope(name, T, H, KV, hd, rot, interleaved, scaling, fp8, ps, base):
    return {"name": name, "op": "rope", "T": T, "H": H, "KV": KV, "hd": hd, "rot": rot, "interleaved": interleaved,
            "scaling": scaling, "theta": 500000.0, "fp8": fp8, "ps": ps, "base": base, "mix": T}


def _attend(name, n, q, ctx, H, KV, hd, ps, mix, fp8=False, softcap=0.0, window=0, alibi=False, head_major=True,
            packed=False):
    return {"name": name, "op": "attend", "n": n, "q_lo": q[0], "q_hi": q[1], "ctx_lo": ctx[0], "ctx_hi": ctx[1],
            "H": H, "KV": KV, "hd": hd, "ps": ps, "mix": mix, "fp8": fp8, "softcap": softcap, "window": window,
            "alibi": alibi, "head_major": head_major, "packed": packed}


def listed():
    return [
        # the bookkeeping of a small decode step: one new token for each of 32 requests
        _step("step_decode_32", 32, 16, (1, 4000), (1, 1), 3),
        # a step that mixes decode with chunks of many prompts: about 84,000 tokens of 1024 requests
        _step("step_mixed_1024", 1024, 16, (0, 16000), (1, 512), 5, pad=100),
        # one token of one request (Llama-3-8B heads): the smallest call of a decode loop
        _rope("rope_one_token", 1, 32, 8, 128, 128, False, "llama3", False, 16, 5000),
        # a decode step of 256 tokens into an FP8 cache, half of each head rotated, interleaved pairs
        _rope("rope_decode_256_fp8", 256, 32, 8, 128, 64, True, "none", True, 16, 2000),
        # a prefill step of 16,384 tokens, long-context frequencies
        _rope("rope_chunk_16384", 16384, 32, 8, 128, 128, False, "yarn", False, 64, 100000),
        # one user, a short conversation: latency
        _attend("decode_1x100", 1, (1, 1), (99, 99), 32, 8, 128, 16, 7),
        # an ordinary decode step: 64 requests of ragged lengths, Llama-3-8B heads
        _attend("decode_64_ragged", 64, (1, 1), (100, 8000), 32, 8, 128, 16, 8),
        # speculative decode, 64 sequences of 4 tokens, FP8 cache, capped scores, a sliding window
        _attend("spec_64x4_fp8_window", 64, (4, 4), (500, 8000), 32, 8, 128, 16, 9, fp8=True, softcap=30.0,
                window=4096),
        # one user, a very long context: the cache's length is all there is to split
        _attend("decode_1x131071", 1, (1, 1), (131070, 131070), 32, 8, 128, 64, 10),
        # a full decode batch: the largest cache traffic
        _attend("decode_256x8k", 256, (1, 1), (2000, 8191), 32, 8, 128, 16, 11),
        # ragged prompt chunks over an FP8 cache, some of the prompt cached before, 64-wide heads, ALiBi, capped scores
        _attend("prompts_8_ragged_fp8", 8, (200, 2000), (0, 2000), 16, 4, 64, 16, 12, fp8=True, softcap=50.0,
                alibi=True),
        # one long prompt, Llama-3-8B heads, causal
        _attend("prompt_8192", 1, (8192, 8192), (0, 0), 32, 8, 128, 64, 13),
    ]


def _log(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))
    v = min(hi, max(lo, v))
    return v + 1 if v == 3072 else v


def draw(rng):
    kind = rng.choice(("step", "rope", "decode", "decode", "prompt", "prompt"))
    ps = rng.choice((16, 32, 64, 128))
    mix = rng.randrange(1 << 30)
    if kind == "step":
        n = _log(rng, 1, 1024)
        new = _log(rng, 1, max(1, min(4096, 200000 // n)))
        c = _step("", n, ps, (0, _log(rng, 1, 16000)), (1, new), mix, pad=rng.choice((0, _log(rng, 1, 500))))
    elif kind == "rope":
        hd, KV = rng.choice((64, 128)), rng.choice((1, 2, 8))
        c = _rope("", _log(rng, 1, 16384), KV * rng.choice((1, 3, 4)), KV, hd, rng.choice((hd, hd // 2)),
                  rng.random() < 0.5, rng.choice(sorted(SCALINGS)), rng.random() < 0.4, ps, _log(rng, 1, 100000))
        c["mix"] = mix
    else:
        hd, KV, G = rng.choice((64, 128)), rng.choice((1, 2, 4, 8)), rng.choice((1, 3, 4, 8))
        more = {"fp8": rng.random() < 0.4, "softcap": rng.choice((0.0, 0.0, 30.0)), "alibi": rng.random() < 0.3,
                "window": rng.choice((0, 0, _log(rng, 16, 4096))), "head_major": rng.random() < 0.6,
                "packed": rng.random() < 0.5}
        if kind == "decode":
            n = _log(rng, 1, 256)
            ctx = _log(rng, 1, min(131070, 2000000 // n))
            q = rng.choice((1, 1, 2, 4, 7))
            c = _attend("", n, (1 if rng.random() < 0.5 else q, q), (max(0, ctx // rng.choice((1, 4, 40))), ctx),
                        KV * G, KV, hd, ps, mix, **more)
        else:
            n = _log(rng, 1, 12)
            q = _log(rng, 17, max(18, int(6000 / math.sqrt(n))))
            ctx = rng.choice((0, _log(rng, 1, 3000)))
            c = _attend("", n, (max(1, q // rng.choice((1, 3, 20))), q), (0, ctx), KV * G, KV, hd, ps, mix, **more)
    del c["name"]
    return c


# ---------------------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------------------
def _lengths(case, lo, hi, salt):
    """One length for each request, spread over the logarithm; from the case alone."""
    rng = random.Random(case["mix"] * 31 + salt)
    return [lo if lo == hi else int(math.exp(rng.uniform(math.log(lo + 1), math.log(hi + 1.999)))) - 1
            for _ in range(case["n"])]


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 17)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _int(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype).to(DEV)


def _slopes(H):
    return [2.0 ** (-8.0 * (h + 1) / H) for h in range(H)]


def _frequencies(case):
    """Radians a position step of each rotated pair, and the factor on cos and sin."""
    rot, s = case["rot"], SCALINGS[case["scaling"]]
    f = [case["theta"] ** (-2.0 * i / rot) for i in range(rot // 2)]
    if s is None:
        return f, 1.0
    if s["kind"] == "linear":
        return [x / s["factor"] for x in f], 1.0
    if s["kind"] == "llama3":
        out = []
        for x in f:
            turns = s["original"] * x / (2 * math.pi)  # turns over the original context
            t = min(1.0, max(0.0, (turns - s["low_freq_factor"]) / (s["high_freq_factor"] - s["low_freq_factor"])))
            out.append(x * t + x / s["factor"] * (1 - t))
        return out, 1.0

    def pair(turns):
        return rot * math.log(s["original"] / (turns * 2 * math.pi)) / (2 * math.log(case["theta"]))

    lo, hi = max(0, math.floor(pair(s["beta_fast"]))), min(rot - 1, math.ceil(pair(s["beta_slow"])))
    ramp = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3))) for i in range(rot // 2)]
    return [x * (1 - r) + x / s["factor"] * r for x, r in zip(f, ramp)], 0.1 * math.log(s["factor"]) + 1.0


def _cache(g, case, n_pages, zero=False):
    """k and v as [page, token, head, dim], each head's tokens of a page side by side where head_major."""
    KV, ps, hd = case["KV"], case["ps"], case["hd"]
    dtype = E4M3 if case["fp8"] else BF16
    shape = (n_pages, KV, ps, hd) if case.get("head_major", True) else (n_pages, ps, KV, hd)
    both = []
    for shift in (0.0, 0.1):
        if zero:
            t = torch.zeros(shape, dtype=torch.uint8 if case["fp8"] else BF16, device=DEV)
            t = t.view(E4M3) if case["fp8"] else t
        else:
            t = torch.empty(shape, dtype=dtype, device=DEV)
            part = max(1, (1 << 28) // (KV * ps * hd))
            for a in range(0, n_pages, part):
                t[a:a + part] = (_randn(g, min(part, n_pages - a), *shape[1:]) + shift).to(dtype)
        both.append(t.transpose(1, 2) if case.get("head_major", True) else t)
    return both


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "step":
        ctx, new = _lengths(case, case["ctx_lo"], case["ctx_hi"], 1), _lengths(case, case["new_lo"], case["new_hi"], 2)
        ps, n = case["ps"], case["n"]
        have = [-(-c // ps) for c in ctx]
        width = max(-(-(c + m) // ps) for c, m in zip(ctx, new)) + 1
        need = sum(-(-(c + m) // ps) - h for c, m, h in zip(ctx, new, have))
        pages = torch.randperm(sum(have) + need + 64, generator=g, device=DEV).to(torch.int32)
        rows = torch.full((n, width), -1, dtype=torch.int32, device=DEV)
        own_pages = torch.arange(width, device=DEV)[None] < _int(have)[:, None]
        rows[own_pages] = pages[:sum(have)]
        s |= {"ctx": _int(ctx), "new": _int(new), "rows": rows, "T": sum(new) + case["pad"],
              "free": pages[sum(have):].contiguous()}
        if own:
            import rank_adapter_gemm_gb300 as L
            s["step"] = L.KVStep(n, s["T"], width, ps, device=DEV)
            s["step"].block_table.copy_(rows)
        return s
    if case["op"] == "rope":
        T, H, KV, hd, ps = (case[k] for k in ("T", "H", "KV", "hd", "ps"))
        s["qkv"] = _randn(g, T, (H + 2 * KV) * hd).to(BF16)
        n_pages = -(-T // ps) + 3
        rng = random.Random(case["mix"])
        first = rng.randrange(case["base"]) if T > 300 else None  # a chunk of one prompt, or tokens of many requests
        s["positions"] = (torch.arange(T, device=DEV, dtype=torch.int32) + first if first is not None else
                          torch.randint(0, case["base"], (T,), generator=g, device=DEV, dtype=torch.int32))
        order = torch.randperm(n_pages - 1, generator=g, device=DEV)  # the last page stays free
        at = torch.arange(T, device=DEV)
        s["slots"] = order[at // ps] * ps + at % ps
        if T > 8:
            s["slots"][T // 2] = -1  # a padding token: its k and v go nowhere
        s["k"], s["v"] = _cache(g, case, n_pages, zero=True)
        s["k_scale"], s["v_scale"] = (0.0625, 0.03125) if case["fp8"] else (1.0, 1.0)
        f, s["mscale"] = _frequencies(case)
        s["freq"] = _int(f, torch.float32)
        if own:
            import rank_adapter_gemm_gb300 as L
            s["kv"] = L.PagedKV(s["k"], s["v"], s["k_scale"], s["v_scale"])
            s["rope"] = L.Rope(hd, case["rot"], theta=case["theta"], interleaved=case["interleaved"],
                               scaling=SCALINGS[case["scaling"]], device=DEV)
            s["q_out"] = torch.empty(T, H * hd, dtype=BF16, device=DEV)
            s["err"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        return s
    H, KV, hd, ps, n = (case[k] for k in ("H", "KV", "hd", "ps", "n"))
    new, ctx = _lengths(case, case["q_lo"], case["q_hi"], 2), _lengths(case, case["ctx_lo"], case["ctx_hi"], 1)
    lens = [a + b for a, b in zip(new, ctx)]
    used = [-(-x // ps) for x in lens]
    n_pages, width, T = sum(used) + 1, max(used), sum(new)
    s["k"], s["v"] = _cache(g, case, n_pages)
    s["k_scale"], s["v_scale"] = (0.5, 0.25) if case["fp8"] else (1.0, 1.0)
    rows = torch.zeros(n, width, dtype=torch.int32, device=DEV)
    rows[torch.arange(width, device=DEV)[None] < _int(used)[:, None]] = torch.randperm(
        n_pages, generator=g, device=DEV)[:sum(used)].to(torch.int32)
    ld = (H + 2 * KV) * hd if case["packed"] else H * hd
    # rows of a packed projection, or rows of q alone; the heads differ in how sharply they look
    sharp = torch.linspace(0.5, 2.0, H, device=DEV).repeat_interleave(hd)
    s["q"] = (_randn(g, T, ld).to(BF16))[:, :H * hd]
    s["q"].mul_(sharp.to(BF16))
    s |= {"rows": rows, "lens": _int(lens), "T": T, "new": new, "len_list": lens,
          "q_offsets": _int(np.concatenate([[0], np.cumsum(new)]).tolist()), "scale": hd ** -0.5,
          "slopes": _int(_slopes(H), torch.float32) if case["alibi"] else None}
    if own:
        import rank_adapter_gemm_gb300 as L
        kv = L.PagedKV(s["k"], s["v"], s["k_scale"], s["v_scale"])
        s["attention"] = L.Attention(n, T, H, kv, scale=s["scale"], softcap=case["softcap"], window=case["window"],
                                     slopes=s["slopes"], device=DEV)
        s["out"] = torch.empty(T, H * hd, dtype=BF16, device=DEV)
    return s


# ---------------------------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------------------------
def _plain_step(s):
    ps, T = s["case"]["ps"], s["T"]
    ctx, new, rows, free = s["ctx"].long(), s["new"].long(), s["rows"].long(), s["free"].long()
    have, then = (ctx + ps - 1) // ps, (ctx + new + ps - 1) // ps
    ends = torch.cumsum(then - have, 0)
    at = ends - (then - have)
    served = (ends <= free.numel()) | (then == have)
    kv_lens = torch.where(served, ctx + new, ctx)
    q_off = torch.cat([new.new_zeros(1), torch.cumsum(new, 0)])
    t = torch.arange(T, device=ctx.device)
    real = t < q_off[-1]
    seq = torch.searchsorted(q_off[1:].contiguous(), t, right=True).clamp(max=ctx.numel() - 1)
    pos = ctx[seq] + t - q_off[seq]
    page_of = pos // ps
    fresh = free[(at[seq] + page_of - have[seq]).clamp(0, free.numel() - 1)]
    page = torch.where(page_of < have[seq], rows[seq, page_of.clamp(max=rows.shape[1] - 1)], fresh)
    slots = torch.where(real & served[seq], page * ps + pos % ps, -1)
    e = torch.arange(rows.shape[1], device=ctx.device)[None]
    taken = (e >= have[:, None]) & (e < then[:, None]) & served[:, None]
    table = torch.where(taken, free[(at[:, None] + e - have[:, None]).clamp(0, free.numel() - 1)], rows)
    count = torch.where(served, then - have, 0).sum().reshape(1)
    i32 = torch.int32
    return {"block_table": table.to(i32), "q_offsets": q_off.to(i32), "kv_lens": kv_lens.to(i32),
            "positions": torch.where(real, pos, 0).to(i32), "seq_ids": torch.where(real, seq, -1).to(i32),
            "slot_map": slots, "taken": count.to(i32)}


def _plain_rope(s):
    c = s["case"]
    T, H, KV, hd, rot, ps = (c[k] for k in ("T", "H", "KV", "hd", "rot", "ps"))
    x = s["qkv"].float().view(T, H + 2 * KV, hd)
    angle = s["positions"].float()[:, None] * s["freq"][None]
    cos, sin = (angle.cos() * s["mscale"])[:, None], (angle.sin() * s["mscale"])[:, None]
    qk = x[:, :H + KV]
    if c["interleaved"]:
        a, b = qk[..., 0:rot:2], qk[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = qk[..., :rot // 2], qk[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    qk = torch.cat([turned, qk[..., rot:]], -1)
    slots = s["slots"]
    put = slots >= 0
    page, off = torch.where(put, slots // ps, s["k"].shape[0] - 1), slots.clamp(min=0) % ps
    for cache, new, scale in ((s["k"], qk[:, H:], s["k_scale"]), (s["v"], x[:, H + KV:], s["v_scale"])):
        flat = cache.view(torch.uint8) if c["fp8"] else cache
        new = ((new / scale).clamp(-448, 448).to(E4M3).view(torch.uint8) if c["fp8"] else new.to(BF16))
        # a padding token writes back what the free page holds
        flat[page, off] = torch.where(put[:, None, None], new, flat[page, off])
    return {"q": qk[:, :H].reshape(T, H * hd).to(BF16), "k": s["k"], "v": s["v"]}


def _plain_attend(s):
    c = s["case"]
    H, KV, hd, ps, n = (c[k] for k in ("H", "KV", "hd", "ps", "n"))
    G, Q, T = H // KV, c["q_hi"], s["T"]
    lens, off = s["lens"].long(), s["q_offsets"].long()
    rows = s["rows"].long()
    span = rows.shape[1] * ps
    key = torch.arange(span, device=rows.device)
    there = key[None] < lens[:, None]
    k = s["k"][rows].float().reshape(n, span, KV, hd) * s["k_scale"]
    v = s["v"][rows].float().reshape(n, span, KV, hd) * s["v_scale"]
    v = torch.where(there[..., None, None], v, 0.0)
    i = torch.arange(Q, device=rows.device)
    q_len = off[1:] - off[:-1]
    q = s["q"][(off[:-1, None] + i[None]).clamp(max=T - 1)].float().view(n, Q, KV, G, hd)
    score = torch.matmul(q.permute(0, 2, 3, 1, 4).reshape(n, KV, G * Q, hd), k.permute(0, 2, 3, 1))
    score = score.view(n, KV, G, Q, span) * s["scale"]
    del k
    if c["softcap"]:
        score = torch.tanh(score / c["softcap"]) * c["softcap"]
    pos = (lens - q_len)[:, None] + i[None]
    away = key[None, None] - pos[..., None]
    if c["alibi"]:
        score = score + s["slopes"].view(1, KV, G, 1, 1) * away[:, None, None].float()
    seen = (away <= 0) & there[:, None]
    if c["window"]:
        seen &= away > -c["window"]
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isfinite(top), top, 0.0))
    del score
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(n, KV, G * Q, span), v.permute(0, 2, 1, 3)).view(n, KV, G, Q, hd)
    out = torch.where(total > 0, out / total, 0.0)
    t = torch.arange(T, device=rows.device)
    seq = torch.searchsorted(off[1:].contiguous(), t, right=True)
    return out.permute(0, 3, 1, 2, 4)[seq, t - off[seq]].reshape(T, H * hd).to(BF16)


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"step": _plain_step, "rope": _plain_rope, "attend": _plain_attend}[c["op"]](s)
    if c["op"] == "step":
        st = s["step"]
        st.build(s["ctx"], s["new"], s["free"])
        return {"block_table": st.block_table, "q_offsets": st.q_offsets, "kv_lens": st.kv_lens,
                "positions": st.positions, "seq_ids": st.seq_ids, "slot_map": st.slot_map, "taken": st.taken}
    if c["op"] == "rope":
        s["rope"].append(s["qkv"], s["q_out"], c["H"], s["kv"], s["positions"], s["slots"], s["err"])
        return {"q": s["q_out"], "k": s["k"], "v": s["v"]}
    s["attention"].run(s["q"], s["out"], s["q_offsets"], s["lens"], s["rows"], c["q_hi"])
    return s["out"]


# ---------------------------------------------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------
def work(case):
    if case["op"] == "step":
        ctx, new = _lengths(case, case["ctx_lo"], case["ctx_hi"], 1), _lengths(case, case["new_lo"], case["new_hi"], 2)
        ps = case["ps"]
        taken = sum(-(-(c + m) // ps) + -c // ps for c, m in zip(ctx, new))
        last = sum(c % ps != 0 for c in ctx)  # pages that the first tokens go on filling
        T = sum(new) + case["pad"]
        return {"bytes": 16 * case["n"] + 4 * last + 8 * taken + 16 * T + 8, "flops": 0}
    if case["op"] == "rope":
        T, H, KV, hd = (case[k] for k in ("T", "H", "KV", "hd"))
        size = 1 if case["fp8"] else 2
        return {"bytes": T * (2 * (H + 2 * KV) * hd + 2 * H * hd + 2 * KV * hd * size + 12) + 8 * case["rot"] // 2,
                "flops": 3 * T * (H + KV) * case["rot"]}
    new, ctx = _lengths(case, case["q_lo"], case["q_hi"], 2), _lengths(case, case["ctx_lo"], case["ctx_hi"], 1)
    H, KV, hd, w = (case[k] for k in ("H", "KV", "hd", "window"))
    pairs = keys = 0
    for q, c in zip(new, ctx):
        see = np.arange(c + 1, c + q + 1)
        pairs += int((np.minimum(see, w) if w else see).sum())
        keys += min(c + q, w + q - 1) if w else c + q
    T = sum(new)
    return {"bytes": keys * KV * hd * 2 * (1 if case["fp8"] else 2) + 4 * T * H * hd + 4 * keys // case["ps"],
            "flops": 4 * pairs * H * hd}


# ---------------------------------------------------------------------------------------------------------------
# In 64 bits
# ---------------------------------------------------------------------------------------------------------------
def _exact_rope(s):
    c = s["case"]
    T, H, KV, hd, rot, ps = (c[k] for k in ("T", "H", "KV", "hd", "rot", "ps"))
    f = np.float64(c["theta"]) ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    scaling, m = c["scaling"], 1.0
    if scaling == "linear":
        f = f / LINEAR["factor"]
    elif scaling == "llama3":
        wave, o = 2 * np.pi / f, LLAMA3["original"]
        lo, hi, by = LLAMA3["low_freq_factor"], LLAMA3["high_freq_factor"], LLAMA3["factor"]
        smooth = (o / wave - lo) / (hi - lo)
        f = np.where(wave < o / hi, f, np.where(wave > o / lo, f / by, (1 - smooth) * f / by + smooth * f))
    elif scaling == "yarn":
        bound = [rot * np.log(YARN["original"] / (b * 2 * np.pi)) / (2 * np.log(c["theta"]))
                 for b in (YARN["beta_fast"], YARN["beta_slow"])]
        lo, hi = max(np.floor(bound[0]), 0), min(np.ceil(bound[1]), rot - 1)
        mask = 1 - np.clip((np.arange(rot // 2) - lo) / (hi - lo), 0, 1)
        f, m = f / YARN["factor"] * (1 - mask) + f * mask, 1 + 0.1 * np.log(YARN["factor"])
    a = s["positions"].double()[:, None] * torch.from_numpy(f).to(DEV)
    z = torch.polar(torch.full_like(a, float(m)), a)[:, None]
    x = s["qkv"].double().view(T, H + 2 * KV, hd).clone()
    part = x[:, :H + KV, :rot]
    if c["interleaved"]:
        x[:, :H + KV, :rot] = torch.view_as_real(torch.view_as_complex(
            part.reshape(T, H + KV, rot // 2, 2).contiguous()) * z).flatten(-2)
    else:
        w = torch.complex(part[..., :rot // 2].contiguous(), part[..., rot // 2:].contiguous()) * z
        x[:, :H + KV, :rot] = torch.cat([w.real, w.imag], -1)
    out = {"q": x[:, :H].reshape(T, H * hd)}
    put = (s["slots"] >= 0).nonzero()[:, 0]
    slot = s["slots"][put]
    for name, new in (("k", x[:, H:H + KV]), ("v", x[:, H + KV:])):
        cache = s[name].double().clone()
        new = new[put] / s[name + "_scale"]
        cache[slot // ps, slot % ps] = new.clamp(-448, 448) if c["fp8"] else new
        out[name] = cache
    return out


def exact(case, seed):
    if case["op"] == "step":
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s)
    if work(case)["flops"] > 3e12:
        return None
    H, KV, hd, ps = (case[k] for k in ("H", "KV", "hd", "ps"))
    G = H // KV
    out = torch.zeros(s["T"], H, hd, dtype=torch.float64, device=DEV)
    at = 0
    for r, (m, length) in enumerate(zip(s["new"], s["len_list"])):
        pages = s["rows"][r, :-(-length // ps)].long()
        k, v = (s[x][pages].double().reshape(-1, KV, hd)[:length] * s[x + "_scale"] for x in ("k", "v"))
        where = torch.arange(length, device=DEV, dtype=torch.float64)
        pos = torch.arange(length - m, length, device=DEV, dtype=torch.float64)
        back = pos[:, None] - where[None]
        ok = back >= 0
        if case["window"]:
            ok &= back < case["window"]
        q = s["q"][at:at + m].double().view(m, H, hd)
        for h in range(H):
            w = (q[:, h] @ k[:, h // G].T) / math.sqrt(hd)
            if case["softcap"]:
                w = case["softcap"] * torch.tanh(w / case["softcap"])
            if case["alibi"]:
                w = w - _slopes(H)[h] * back
            w = torch.softmax(torch.where(ok, w, torch.full_like(w, -math.inf)), -1)
            out[at:at + m, h] = w @ v[:, h // G]
        at += m
    return out.view(s["T"], H * hd)
