"""One attention layer of a multi-adapter serving engine, prompt and decode steps.

    python examples/attention_layer.py            # Llama-3-8B layer shapes, 64 requests, times each step
    python examples/attention_layer.py --small    # small shapes, every step against a plain fp32 form

Per step: cache pages, slots and positions from the requests' lengths (KVStep), the
token index of the adapters from the step's request ids, then per layer
    qkv = x W_qkv^T + branch          base projection, then lora_apply
    q, cache = rope.append(qkv)       positions on q and k, k and v into the cache
    a = attention(q, cache)
    out = a W_o^T + branch
"""
import argparse
import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import rank_adapter_gemm_gb300 as L  # noqa: E402

BF16 = torch.bfloat16


class Projection:
    """A base weight [sum of widths, k] and S adapters of rank r on its output slices."""

    def __init__(self, k, widths, S, r, g, scale=0.5):
        def randn(*shape, std):
            return (torch.randn(*shape, generator=g, device="cuda") * std).to(BF16)
        self.w = randn(sum(widths), k, std=k ** -0.5)
        self.A = [[randn(r, k, std=k ** -0.5) for _ in widths] for _ in range(S)]
        self.B = [[randn(d, r, std=0.3) for d in widths] for _ in range(S)]
        self.scale, self.S = scale, S
        self.shape = L.make_shape(S, r, k, widths)
        self.table = L.SlotTable(S, len(widths), r)
        self.table.set([r] * S, [scale] * S, [a.data_ptr() for row in self.A for a in row],
                       [b.data_ptr() for row in self.B for b in row])
        self._ws = {}

    def __call__(self, x, y, index):
        torch.matmul(x, self.w.t(), out=y)
        T = x.shape[0]
        if T not in self._ws:
            self._ws[T] = L.Workspace(T, self.shape)
        L.apply(x, y, self.table, index, self._ws[T], self.shape)

    def plain(self, x, slots):
        """The same in fp32 from the definition; rounded as the two calls round."""
        y = (x.float() @ self.w.float().t()).to(BF16).float()
        for s in range(self.S):
            rows = slots == s
            for i, (a, b) in enumerate(zip(self.A[s], self.B[s])):
                at = sum(m.shape[0] for m in self.B[s][:i])
                y[rows, at:at + b.shape[0]] += self.scale * (x[rows].float() @ a.float().t()) @ b.float().t()
        return y.to(BF16)


class Layer:
    def __init__(self, hidden, H, KV, hd, S, r, n_seq, max_pages, page_size, cache_type=BF16, softcap=0.0, window=0,
                 theta=500000.0, scaling=None, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.H, self.KV, self.hd, self.page_size, self.n_seq = H, KV, hd, page_size, n_seq
        self.qkv = Projection(hidden, [H * hd, KV * hd, KV * hd], S, r, g)
        self.o = Projection(H * hd, [hidden], S, r, g)
        scales = (1.0, 1.0) if cache_type == BF16 else (0.0625, 0.0625)
        self.kv = L.PagedKV.empty(n_seq * max_pages, page_size, KV, hd, cache_type, *scales)
        self.rope = L.Rope(hd, theta=theta, scaling=scaling)
        self.attention = L.Attention(n_seq, 0, H, self.kv, softcap=softcap, window=window)
        self.seq_slot = torch.arange(n_seq, device="cuda", dtype=torch.int32) % (S + 1) - 1  # some without an adapter
        self.start = torch.zeros(n_seq, dtype=torch.int32, device="cuda")

    def forward(self, x, step, max_q):
        """x [T, hidden] of the step's T tokens -> (output, what lies between)."""
        T = x.shape[0]
        index = L.TokenIndex(T, self.qkv.S)
        index.build_activated(step.seq_ids, step.positions, self.seq_slot, self.start, self.qkv.table)
        y = torch.empty(T, (self.H + 2 * self.KV) * self.hd, dtype=BF16, device="cuda")
        q, a = (torch.empty(T, self.H * self.hd, dtype=BF16, device="cuda") for _ in range(2))
        out = torch.empty(T, x.shape[1], dtype=BF16, device="cuda")
        self.qkv(x, y, index)
        self.rope.append(y, q, self.H, self.kv, step.positions, step.slot_map, step.err)
        self.attention.run(q, a, step.q_offsets, step.kv_lens, step.block_table, max_q)
        self.o(a, out, index)
        return out, (index, y, q, a)


def plain_attention(layer, q, step, lens, new):
    """Attention of the step's rows in fp32 over the cache's own values."""
    out, at, G = [], 0, layer.H // layer.KV
    c = layer.kv.c
    for i, (n, m) in enumerate(zip(lens, new)):
        pages = step.block_table[i, :-(-n // layer.page_size)].long()
        k, v = (t[pages].float().reshape(-1, layer.KV, layer.hd)[:n] * s
                for t, s in ((layer.kv.k, c.k_scale), (layer.kv.v, c.v_scale)))
        k, v = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
        rows = q[at:at + m].float().view(m, layer.H, layer.hd)
        s = torch.einsum("qhd,khd->hqk", rows, k) * layer.hd ** -0.5
        cap, window = layer.attention.c.softcap, layer.attention.c.window
        if cap:
            s = cap * torch.tanh(s / cap)
        back = torch.arange(n - m, n, device="cuda")[:, None] - torch.arange(n, device="cuda")[None]
        hidden = (back < 0) | ((back >= window) if window else torch.zeros_like(back, dtype=torch.bool))
        out.append(torch.einsum("hqk,khd->qhd", s.masked_fill(hidden, -math.inf).softmax(-1), v).reshape(m, -1))
        at += m
    return torch.cat(out)


def serve(layer, prompts, decode_steps, hidden, check=False, seed=1):
    """A prompt step of the given lengths, then decode steps of one token each;
    returns the largest relative error of attention and projections (check) and
    the device times of the steps in us."""
    n, ps = layer.n_seq, layer.page_size
    max_pages = -(-(max(prompts) + decode_steps) // ps)
    free = torch.randperm(layer.kv.k.shape[0], device="cuda").to(torch.int32)
    ctx, worst, times, table = [0] * n, 0.0, [], None
    g = torch.Generator(device="cuda").manual_seed(seed)
    for new in [list(prompts)] + [[1] * n] * decode_steps:
        T = sum(new)
        step = L.KVStep(n, T, max_pages, ps)
        if table is not None:
            step.block_table = table
        i32 = dict(dtype=torch.int32, device="cuda")
        x = torch.randn(T, hidden, generator=g, device="cuda").to(BF16)
        old, fresh = torch.tensor(ctx, **i32), torch.tensor(new, **i32)
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        step.build(old, fresh, free)
        out, (index, y, q, att) = layer.forward(x, step, max(new))
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b) * 1e3)
        free, table = free[step.taken.item():].contiguous(), step.block_table
        assert step.err.item() == 0 and index.err.item() == 0 and layer.attention.err.item() == 0
        ctx = [c + m for c, m in zip(ctx, new)]
        if check:
            slots = layer.seq_slot[step.seq_ids.long()]
            for got, want in ((y, layer.qkv.plain(x, slots)), (att, plain_attention(layer, q, step, ctx, new)),
                              (out, layer.o.plain(att, slots))):
                worst = max(worst, ((got.float() - want.float()).norm() / want.float().norm()).item())
    return worst, times


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--small", action="store_true")
    a = ap.parse_args()
    if a.small:
        for kw in (dict(), dict(cache_type=torch.float8_e4m3fn, softcap=30.0, window=40)):
            layer = Layer(512, 8, 2, 64, 3, 16, 6, 16, 16, **kw)
            worst, _ = serve(layer, [33, 1, 70, 128, 5, 16], 3, 512, check=True)
            print(f"{kw}: largest relative error {worst:.2e}")
            assert worst < 8e-3, worst
        return
    layer = Layer(4096, 32, 8, 128, 16, 16, 64, 132, 16)
    _, times = serve(layer, [100 + 29 * i for i in range(64)], 8, 4096)
    print(f"prompt step {times[0]:.0f} us (first call), decode steps {', '.join('%.0f' % t for t in times[2:])} us")


if __name__ == "__main__":
    main()
