"""Requests that share what they have cached, at the edges of the calls' range: device data that does not fit
together, sums over many tokens.  Batches and tolerances are those of test_sharing.py.
"""
import numpy as np
import pytest

from test_sharing import (Batch, L, _torch, check_against_each, check_compact, check_fork, dev, random_tables,  # noqa: F401
                          ref_compact, ref_fork, run_compact, run_fork)  # (L: a fixture)

gpu = pytest.mark.gpu


# ---------------------------------------------------------------------------
# Attention: row offsets out of order or range
# ---------------------------------------------------------------------------
def definition(b, i, q0, q1):
    """(out, tolerance, lse, tolerance) of request i's rows [q0, q1), its last positions, as Batch.check has them."""
    k, v = (x.double().cpu().numpy() * s for x, s in zip((b.dk, b.dv), b.scales))
    q = b.dq.double().cpu().numpy().reshape(b.rows, b.H, b.hd)
    n, m, G = b.lens[i], q1 - q0, b.H // b.KV
    j = np.arange(n)
    kk, vv = (x[b.table[i, j // b.ps], j % b.ps] for x in (k, v))
    seen = j[None] <= np.arange(n - m, n)[:, None]
    out, tol = np.zeros((m, b.H, b.hd)), np.zeros((m, b.H, b.hd))
    lse, lse_tol = np.zeros((m, b.H)), np.zeros((m, b.H))
    for h in range(b.H):
        s = b.hd ** -0.5 * q[q0:q1, h] @ kk[:, h // G].T
        eps = 2.0 ** -18 * (1 + np.abs(np.where(seen, s, 0.0)).max(1, initial=0.0))
        s = np.where(seen, s, -np.inf)
        top = s.max(1, keepdims=True)
        e = np.exp(s - top)
        total = e.sum(1, keepdims=True)
        out[:, h], A = e / total @ vv[:, h // G], e / total @ np.abs(vv[:, h // G])
        tol[:, h] = 2.0 ** -8 * np.abs(out[:, h]) + (2.0 ** -8 + 2 * eps[:, None]) * A + 2.0 ** -20
        lse[:, h], lse_tol[:, h] = (top + np.log(total))[:, 0], eps
    return out, tol, lse, lse_tol


def check_offsets(L, b, off, att, share):  # noqa: F811
    """Requests whose offsets fit have their rows by definition where no other has them too; rows of none stay."""
    torch = _torch()
    out = torch.full((b.rows, b.H * b.hd), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((b.rows, b.H), 7.0, device="cuda")
    att.err.zero_()
    att.run(b.dq, out, dev(off), dev(b.lens), dev(b.table), dev(b.starts), dev(b.prefix), kv=L.PagedKV(b.dk, b.dv, *b.scales),
            lse=lse, share=share)
    torch.cuda.synchronize()
    assert int(att.err) == 1
    out, lse = out.double().cpu().numpy().reshape(b.rows, b.H, b.hd), lse.double().cpu().numpy()
    good = [(i, off[i], off[i + 1]) for i in range(b.n) if 0 <= off[i] <= off[i + 1] <= b.rows]
    owners = np.zeros(b.rows, int)
    for _, q0, q1 in good:
        owners[q0:q1] += 1
    for i, q0, q1 in good:
        ref, tol, ref_lse, lse_tol = definition(b, i, q0, q1)
        one = owners[q0:q1] == 1
        assert (np.abs(out[q0:q1] - ref) <= tol)[one].all(), (off, i)
        assert (np.abs(lse[q0:q1] - ref_lse) <= lse_tol)[one].all(), (off, i)
    assert (out[owners == 0] == 7.0).all() and (lse[owners == 0] == 7.0).all()


OFFSETS = [[0, 4, 2, 7, 10, 12], [4, 2, 6, 7, 10, 12], [-3, 4, 6, 7, 10, 12], [0, 4, 6, 7, 10, 9], [0, 4, 6, 7, 10, 99],
           [0, 4, 6, 99, 10, 12], [8, 12, 0, 1, 4, 6], [0, 4, 6, -1, 10, 12], [0, 0, 0, 0, 2 ** 31 - 1, 12]]


@gpu
@pytest.mark.parametrize("used", [False, True], ids=["zeroed", "used"])
@pytest.mark.parametrize("share", ["always", "auto"])
@pytest.mark.parametrize("hd,fp8", [(128, False), (64, True)])
def test_shared_prefix_row_offsets_out_of_order(L, hd, fp8, share, used):  # noqa: F811
    """Offsets that fall inside a group, at its ends and between groups, that are negative or beyond T; with a workspace
    fresh or last used for more rows, so that its parts lay elsewhere."""
    b = Batch([(300, [(10, 4), (5, 2), (0, 1)]), (130, [(20, 3), (4, 2)])], 8, 2, hd, 16, fp8, rows_after=5)
    c = Batch([(90, [(i, 3) for i in range(20)])], 8, 2, hd, 16, fp8)
    kv = L.PagedKV(b.dk, b.dv, *b.scales)
    for off in OFFSETS:
        att = L.SharedAttention(c.n, c.rows, 8, kv)
        if used:
            c.run(L, att=att)
        check_offsets(L, b, off, att, share)
        # the workspace serves calls whose offsets fit
        att.err.zero_()
        b.check(*b.run(L, att=att, share=share))
        assert b.err == 0


@gpu
@pytest.mark.parametrize("used", [False, True], ids=["zeroed", "used"])
def test_shared_prefix_rows_of_a_request_past_its_group(L, used):  # noqa: F811
    """Two requests, offsets 0, 100, 2: the first one's rows lie beyond the group's last."""
    b = Batch([(200, [(120, 100), (5, 2)])], 8, 2, 128, 16)
    c = Batch([(90, [(i, 3) for i in range(60)])], 8, 2, 128, 16)
    att = L.SharedAttention(c.n, c.rows, 8, L.PagedKV(b.dk, b.dv))
    if used:
        c.run(L, att=att)
    check_offsets(L, b, [0, 100, 2], att, "always")


# ---------------------------------------------------------------------------
# Attention: calls that are refused on the device
# ---------------------------------------------------------------------------
@gpu
@pytest.mark.parametrize("share", ["always", "auto"])
def test_shared_prefix_more_own_steps_than_32_bits_count(L, share):  # noqa: F811
    """4,096 requests of 2^25 tokens in two groups, a short prefix in common, one page over and over: 2^32 steps of own
    keys.  The call reports it and writes nothing, with a workspace last used for more rows; the same call with shorter
    requests is served in it."""
    torch = _torch()
    n = L.LORA_MAX_SEQS
    kv = L.PagedKV.empty(1, 1024, 1, 128)
    kv.k.zero_(), kv.v.fill_(0.5)
    table = torch.zeros(n, 2 ** 15, dtype=torch.int32, device="cuda")
    att = L.SharedAttention(n, 2 * n, 1, kv)
    q = torch.zeros(2 * n, 128, dtype=torch.bfloat16, device="cuda")
    groups, prefix = dev([0, n // 2, n]), dev([2048, 3000])

    def run(rows, length):
        out, lse = torch.full((rows * n, 128), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((rows * n, 1), 7.0, device="cuda")
        lens = torch.full((n,), length, dtype=torch.int32, device="cuda")
        off = rows * torch.arange(n + 1, dtype=torch.int32, device="cuda")
        att.run(q[:rows * n], out, off, lens, table, groups, prefix, rows, lse=lse, share=share)
        torch.cuda.synchronize()
        return out, lse

    out, _ = run(2, 5000)
    assert att.err.item() == 0 and bool((out == 0.5).all())
    out, lse = run(1, 2 ** 25)
    assert att.err.item() == 9 and bool((out == 7.0).all()) and bool((lse == 7.0).all())
    att.err.zero_()
    out, lse = run(1, 4096)
    # equal scores of 0: weights 1 of 4,096 keys, sums of powers of two
    assert att.err.item() == 0 and bool((out == 0.5).all())
    assert bool(((lse - 12 * np.log(2.0)).abs() <= 2.0 ** -18 * 13).all())


@gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_shared_prefix_pieces_of_a_call_that_gave_up(L, fp8):  # noqa: F811
    """A wait that gave up leaves a word in the workspace (a word of the counters' KB) because pieces are missing: nothing
    is joined, the call reports it, requests that share nothing have their rows, and the rest stays as it was.  The
    zeroed workspace serves again."""
    torch = _torch()
    b = Batch([(300, [(10, 1), (5, 2), (0, 1)])], 8, 2, 128, 16, fp8, alone=[(40, 2), (7, 1)], rows_after=2)
    att = L.SharedAttention(b.n, b.rows, 8, L.PagedKV(b.dk, b.dv, *b.scales))
    b.check(*b.run(L, att=att))
    words = att.ws[:1024].view(torch.int32)
    assert not bool(words.any())
    words[1016 // 4] = 1
    for _ in range(2):
        att.err.zero_()
        out, lse = b.run(L, att=att)
        assert b.err == 7
        b.check(out, lse, skip=[0, 1, 2])
    att.ws.zero_()
    att.err.zero_()
    b.check(*b.run(L, att=att))
    assert b.err == 0 and not bool(words.any())


# ---------------------------------------------------------------------------
# Attention: groups of one
# ---------------------------------------------------------------------------
@gpu
@pytest.mark.parametrize("share", ["always", "auto"])
@pytest.mark.parametrize("hd,fp8", [(128, False), (64, True)])
def test_a_group_of_one_request_shares_nothing(L, hd, fp8, share):  # noqa: F811
    """A request that is alone in its group, or alone there with rows, gives the bits of the call without groups (a
    prefix read apart would round weights on the way)."""
    torch = _torch()
    b = Batch([(4000, [(10, 3)]), (9000, [(0, 0), (700, 5), (3, 0)]), (300, [(0, 0)])], 8, 2, hd, 64, fp8, alone=[(40, 2)])
    want = b.run(L, starts=[0], prefix=[], hint=5)
    assert b.err == 0
    b.check(*want)
    got = b.run(L, hint=5, share=share)
    assert b.err == 0
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    # with company the prefix is shared: other bits
    c = Batch([(4000, [(10, 3), (0, 1)])], 8, 2, hd, 64, fp8)
    alone, shared = c.run(L, starts=[0], prefix=[], hint=3), c.run(L, hint=3)
    assert not all(torch.equal(x, y) for x, y in zip(alone, shared))
    c.check(*shared)


# ---------------------------------------------------------------------------
# Selection: sums over many tokens
# ---------------------------------------------------------------------------
# A term's exponent carries two roundings and that of log2 e, 2.25 2^-24 of its distance from the largest logit (of which the
# weighted mean is below 13 up to 2^24 tokens; references lie up to 4 below, twice); an exponential 2^-22, and each of four moves
# of a reference another; additions 25 2^-24.  (2.25 (13 + 8) + 5 * 4 + 25) 2^-24 < 2^-17: what the header states.  In the rows
# below the mean distance is below 8, one of the references lies below, and a term's weight counts for two moves:
# (2.25 (8 + 4) + 3 * 4 + 25) 2^-24 = 2^-18.  Scores that meet the sum half way leave candidates near 0, whose own
# rounding to fp32 is nothing beside that.
def select_values(L, x, top, total, keep):  # noqa: F811
    """The selection of rows x, a beam each, with `total` the logarithm of their sums and `top` their largest logits (64
    bits): the best candidates' logits as the scores give them back."""
    torch = _torch()
    rows, V = x.shape
    scores = torch.full((rows,), total - top, dtype=torch.float32, device="cuda")
    sel = L.BeamSelect(rows, 1, keep, V, dtype=x.dtype)
    sel.run(x, scores)
    return sel, sel.scores.double().reshape(rows, keep) - (scores.double() - (total - top))[:, None] + top


@gpu
@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("rows,V", [(305, 131072), (305, 1 << 20), (305, 1 << 22), (1, 1 << 20), (1, 1 << 24), (40, 1 << 21)])
def test_select_sums_of_equal_logits_below_some(L, rows, V, fp32):  # noqa: F811
    """Rows of equal logits behind 512 larger ones, a few for every thread that adds: additions that all round the same
    way, where one part takes the row and where hundreds do."""
    torch = _torch()
    for tail in (-0.6953125, -2.296875, -5.125, -9.6875, -12.1875, -14.125):
        x = torch.full((rows, V), tail, dtype=torch.float32 if fp32 else torch.bfloat16, device="cuda")
        x[:, :2048:4] = 0.0
        sel, got = select_values(L, x, 0.0, np.log(512 + (V - 512) * np.exp(tail)), 2)
        assert float(got.abs().max()) <= 2.0 ** -18, tail
        assert sel.tokens.reshape(rows, 2).tolist() == [[0, 4]] * rows


@gpu
@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("rows,V", [(305, 131072), (305, 1 << 20), (305, 1 << 22), (2, 1 << 22)])
@pytest.mark.parametrize("kind", ["rising", "slowly", "falling", "waves", "normal"])
def test_select_sums_of_rows_that_move_their_reference(L, kind, rows, V, fp32):  # noqa: F811
    torch = _torch()
    at = torch.arange(V, dtype=torch.float64, device="cuda") / V
    gen = torch.Generator(device="cuda").manual_seed(V)
    row = {"rising": 20.0 * at, "slowly": at, "falling": -20.0 * at, "waves": 15.0 * at + torch.sin(300.0 * at),
           "normal": 2.0 * torch.randn(V, generator=gen, device="cuda", dtype=torch.float64)}[kind]
    row = row.to(torch.float32 if fp32 else torch.bfloat16)
    order = torch.sort(row.double(), descending=True, stable=True)
    total = float(torch.logsumexp(row.double(), 0))
    sel, got = select_values(L, row.expand(rows, V).contiguous(), float(order.values[0]), total, 4)
    want = order.values[:4]
    # (scores: distances from the largest logit, rounded to fp32)
    assert bool(((got - want).abs() <= 2.0 ** -18 + 2.0 ** -24 * (want - want[0]).abs()).all()), float((got - want).abs().max())
    assert sel.tokens.reshape(rows, 4).tolist() == [order.indices[:4].tolist()] * rows


# ---------------------------------------------------------------------------
# The largest calls
# ---------------------------------------------------------------------------
@gpu
def test_tables_of_the_most_rows_and_pages(L):  # noqa: F811
    """4,096 rows and 2^20 pages at once: the table kernels' shared memory is full."""
    rng = np.random.default_rng(1)
    n, ps, n_pages = L.LORA_MAX_SEQS, 16, 1 << 20
    src, lens, _ = random_tables(rng, n, ps, 300, 20, n_pages, 3)
    held = rng.integers(0, n_pages, 5000).astype(np.int32)
    parents = rng.integers(-1, n, n)
    dst = rng.integers(-9, 9, (n, 20)).astype(np.int32)
    check_fork(run_fork(L, src, lens, parents, ps, n_pages, dst, held), ref_fork(src, lens, parents, ps, n_pages, dst, held))
    check_compact(run_compact(L, src, lens, ps, n_pages, dst, held), ref_compact(src, lens, ps, n_pages, dst, held))


@gpu
@pytest.mark.parametrize("n,beams,keep,V", [(4096, 64, 64, 5), (4096, 3, 64, 40), (9, 64, 64, 3000)])
def test_select_of_the_most_rows(L, n, beams, keep, V):  # noqa: F811
    torch = _torch()
    rng = np.random.default_rng(V)
    x = torch.from_numpy(rng.standard_normal((n * beams, V))).cuda().bfloat16()
    scores = torch.from_numpy(-rng.random(n * beams)).float().cuda()
    sel = L.BeamSelect(n, beams, keep, V)
    sel.run(x, scores)
    c = (torch.log_softmax(x.double(), 1) + scores.double()[:, None]).view(n, beams * V)
    k = min(keep, beams * V)
    best = c.topk(k, 1).values
    got = sel.scores.double().view(n, keep)
    assert bool(((got[:, :k] - best).abs() <= 2.0 ** -18 + 2.0 ** -24 * best.abs()).all())
    assert bool((got[:, k:] == -np.inf).all()) and bool((sel.parents.view(n, keep)[:, k:] == -1).all())
    # the candidates named have these scores, none of them twice, in falling order
    at = ((sel.parents.view(n, keep)[:, :k].long() - beams * torch.arange(n, device="cuda")[:, None]) * V +
          sel.tokens.view(n, keep)[:, :k])
    assert bool((c.gather(1, at) - got[:, :k]).abs().max() <= 2.0 ** -18 + 2.0 ** -24 * 20)
    assert bool((at.sort(1).values.diff(dim=1) > 0).all()) and bool((got.diff(dim=1)[:, :k - 1] <= 0).all())


@gpu
@pytest.mark.parametrize("share", ["always", "auto"])
def test_shared_prefix_of_the_most_requests_and_groups(L, share):  # noqa: F811
    """4,096 requests in 4,096 groups, a third of them without requests, with one, with two."""
    rng = np.random.default_rng(2)
    groups = [(int(rng.integers(0, 200)), [(int(rng.integers(0, 5)), int(rng.random() < 0.9))] * (0, 1, 2)[g % 3])
              for g in range(L.LORA_MAX_SEQS)]
    b = Batch(groups, 2, 1, 64, 16, seed=1)
    assert b.n == 1365 + 2 * 1365 and len(b.prefix) == 4096
    out, lse = b.run(L, share=share)
    assert b.err == 0
    check_against_each(L, b, out, lse)


# ---------------------------------------------------------------------------
# Attention: scores far from 1
# ---------------------------------------------------------------------------
SLOPES = [2.0 ** -(h + 1) for h in range(8)]


@gpu
@pytest.mark.parametrize("hd,fp8", [(128, False), (64, True)])
@pytest.mark.parametrize("kw", [dict(slopes=SLOPES), dict(softcap=30.0, slopes=SLOPES), dict(softcap=1e-5), dict(softcap=3e38),
                                dict(softcap=30.0, window=130)], ids=str)
@pytest.mark.parametrize("power", [90, 40, -40, -90])
def test_shared_prefix_at_query_magnitudes(L, power, kw, hd, fp8):  # noqa: F811
    """Queries times a power of two and the scale divided by it; groups of few and of many rows."""
    b = Batch([(600, [(c, 1) for c in (0, 1, 90, 300)]), (130, [(200, 3), (0, 2)]), (400, [(i, 1) for i in range(40)])], 8, 2,
              hd, 16, fp8, alone=[(40, 2)])
    b.dq.mul_(2.0 ** power)
    for scale in (hd ** -0.5 * 2.0 ** -power, -hd ** -0.5 * 2.0 ** -power):
        out, lse = b.run(L, scale=scale, **kw)
        b.check(out, lse, scale=scale, **kw)
        assert b.err == 0
