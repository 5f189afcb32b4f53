"""hs2_add_rmsnorm, hs2_paged_append and hs2_paged_evict against their definitions in 64 bits.

Tolerances.  RMS norm: y is off by its fp32 steps (the sum of squares over the row, the
root, two products): 16 * 2^-24 relative; a bf16 output adds 2^-8, the sum output is one
bf16 rounding (2^-8: half a step, torch.finfo(bfloat16).eps / 2).  A code is right when it is the nearest E4M3 value of some y within
that (plus one rounding of the scale's reciprocal); scales agree to 16 * 2^-24.  Append:
scales are one fp32 division of an exact maximum (2^-24), codes those of x / s within
2 * 2^-24.  Eviction moves bits: everything is equal.
"""

import pytest
import torch

import long_context_hs2_b200 as hs2
import paged_testlib as P

pytestmark = pytest.mark.gpu


def status_ok():
    st = hs2.hs2_last_device_status()
    assert st == 0, hs2.hs2_status_string(st)


# ----------------------------------------------------------------------- norm --
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,hidden", [(1, 16), (150, 16), (9, 48), (41, 80), (5, 128), (33, 144), (7, 512), (6, 528), (3, 4096),
                                      (2, 8208), (3, 16384), (2, 32768), (1000, 1040)])
def test_norm(T, hidden, residual):
    g = torch.Generator().manual_seed(T + hidden)
    x = torch.randn(T, hidden, generator=g).bfloat16()
    r = (3 * torch.randn(T, hidden, generator=g)).bfloat16() if residual else None
    gamma = (1 + 0.3 * torch.randn(hidden, generator=g)).bfloat16()
    if T > 2:
        x[1] = 0
        if residual:
            r[1] = 0                     # a row of zeros: scale 1, codes 0
    d = lambda t: None if t is None else t.cuda()       # noqa: E731
    s, y = (torch.empty(T, hidden, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    yq = torch.empty(T, hidden, dtype=P.E4M3, device="cuda")
    ys = torch.empty(T, -(-hidden // 128), device="cuda")
    hs2.hs2_add_rmsnorm(d(x), d(r), d(gamma), T, hidden, 1e-6, s, y, yq, ys)
    status_ok()
    h = x.double() + (r.double() if residual else 0)
    want = h / torch.sqrt(h.square().mean(1, keepdim=True) + 1e-6) * gamma.double()
    eps = 16 * 2.0 ** -24 * want.abs()
    assert ((s.cpu().double() - h).abs() <= 2.0 ** -8 * h.abs()).all()
    assert ((y.cpu().double() - want).abs() <= 2.0 ** -8 * want.abs() + 2 * eps).all()
    _, scale = P.quantise(want, 128)
    ys = ys.cpu()
    assert ((ys.double() - scale).abs() <= 20 * 2.0 ** -24 * scale).all()
    wide = ys.repeat_interleave(128, 1)[:, :hidden]
    P.assert_codes(yq.cpu(), want, wide, eps + 4 * 2.0 ** -24 * want.abs())


def test_norm_in_place_and_single_outputs():
    g = torch.Generator().manual_seed(5)
    x, r = (torch.randn(9, 256, generator=g).bfloat16().cuda() for _ in range(2))
    gamma = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    h = x.double().cpu() + r.double().cpu()
    y = torch.empty_like(x)
    hs2.hs2_add_rmsnorm(x, r, gamma, 9, 256, 0.0, r, y)          # the residual's own buffer
    status_ok()
    assert ((r.cpu().double() - h).abs() <= 2.0 ** -8 * h.abs()).all()
    want = h / torch.sqrt(h.square().mean(1, keepdim=True))
    assert ((y.cpu().double() - want).abs() <= (2.0 ** -8 + 2.0 ** -19) * want.abs()).all()
    # the output in X's own buffer, the sum in X's
    a, b = (torch.randn(5, 1040, generator=g).bfloat16().cuda() for _ in range(2))
    w = torch.ones(1040, dtype=torch.bfloat16, device="cuda")
    want_sum, want_y = torch.empty_like(a), torch.empty_like(a)
    hs2.hs2_add_rmsnorm(a, b, w, 5, 1040, 1e-6, want_sum, want_y)
    y2, s2 = a.clone(), a.clone()
    hs2.hs2_add_rmsnorm(y2, b, w, 5, 1040, 1e-6, None, y2)
    hs2.hs2_add_rmsnorm(s2, b, w, 5, 1040, 1e-6, s2)
    status_ok()
    assert torch.equal(y2, want_y) and torch.equal(s2, want_sum)
    # tiny values: the scale's reciprocal would overflow, the codes still stand for x
    gamma.fill_(2.0 ** -126)
    codes = torch.empty(9, 256, dtype=P.E4M3, device="cuda")
    scale = torch.empty(9, 2, device="cuda")
    hs2.hs2_add_rmsnorm(x, None, gamma, 9, 256, 1e-6, None, None, codes, scale)
    status_ok()
    assert (codes.float().abs().amax(1) == 448).all() and (scale > 0).all()


# --------------------------------------------------------------------- append --
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,rows,heads,D,page", [
    ([1, 7, 64, 130], None, 1, 128, 16),
    ([5, 200, 0, 33], [5, 130, 0, 1], 2, 64, 32),
    ([40, 41], [0, 41], 8, 128, 1),
    ([1000], [999], 1, 128, 64),
])
def test_append(lens, rows, heads, D, page, fp8):
    c = P.Cache(lens, page, heads, D, fp8, seed=20, weight=True)
    n_of = [1] * len(lens) if rows is None else rows
    lead, tail = (0, 0) if rows is None else (3, 2)      # rows that are no token's
    n = lead + sum(n_of) + tail
    g = torch.Generator().manual_seed(21)
    kv = torch.randn(n, 2 * heads * D + 8, generator=g).bfloat16()
    kv[lead + sum(n_of) - 1, :D] = 0
    start = None
    if rows is not None:
        start = [lead]
        for k in n_of:
            start.append(start[-1] + k)
        start = torch.tensor(start, dtype=torch.int32, device="cuda")
    before = c.pools()
    dev = kv.cuda()
    hs2.hs2_paged_append(dev[:, :heads * D], dev[:, heads * D:], kv.shape[1], n, start, c.struct,
                         c.B, heads, D, c.dt)
    status_ok()
    after = c.pools()
    touched = torch.zeros(c.n_pages * page, dtype=torch.bool)
    at = lead
    for b, k in enumerate(n_of):
        if not k:
            continue
        rows_b = c.slots(b, range(lens[b] - k, lens[b]))
        touched[rows_b] = True
        for i, name in enumerate(("k", "v")):
            x = kv[at:at + k, i * heads * D:(i + 1) * heads * D].reshape(k, heads, D)
            if fp8:
                _, s = P.quantise(x)
                got = after[name + "_scale"][rows_b]
                assert ((got.double() - s.squeeze(-1)).abs() <= 2.0 ** -23 * s.squeeze(-1)).all()
                P.assert_codes(after[name][rows_b], x, got[..., None],
                               2.0 ** -22 * x.double().abs())
            else:
                assert torch.equal(after[name][rows_b], x)
        assert (after["weight"][rows_b] == 0).all()
        at += k
    for name, t in after.items():      # nothing else moved, bit for bit
        bits = lambda a: a[~touched].contiguous().view(torch.uint8)     # noqa: E731
        assert torch.equal(bits(t), bits(before[name])), name


def test_append_reports_rows_without_a_place():
    c = P.Cache([2, 3], 16, 1, 64, False, seed=22)
    kv = torch.randn(8, 64).bfloat16().cuda()
    before = c.pools()
    start = torch.tensor([0, 5, 8], dtype=torch.int32, device="cuda")   # 5 rows, 2 positions
    hs2.hs2_paged_append(kv, kv, 64, 8, start, c.struct, 2, 1, 64, c.dt)
    assert hs2.hs2_last_device_status() == 6
    after = c.pools()
    assert torch.equal(after["k"][c.slots(0, range(2))], kv[3:5].cpu()[:, None])
    assert torch.equal(after["k"][c.slots(1, range(3))], kv[5:].cpu()[:, None])
    dead = ~c.live
    assert torch.equal(after["k"][dead].view(torch.int16), before["k"][dead].view(torch.int16))


# ------------------------------------------------------------------- eviction --
def evict_case(lens, topk, window, heads, D, page, fp8, in_place, weights, seed=30, **kw):
    c = P.Cache(lens, page, heads, D, fp8, seed=seed, weight=True, stale=1.0, **kw)
    c.w = weights(c.w)
    c.upload()
    slots = topk + window
    before = c.pools()
    kept = torch.full((c.B, slots), -7, dtype=torch.int32, device="cuda")
    new_len = c.len_dev if in_place else torch.full((c.B,), -7, dtype=torch.int32, device="cuda")
    dst = None
    if not in_place:
        per = -(-min(slots, c.max_pages * page) // page)
        assert len(c.free) >= c.B * per
        dst = c.free[:c.B * per].reshape(c.B, per)
    hs2.hs2_paged_evict(c.struct, c.B, heads, D, c.dt, topk, window,
                        None if in_place else dst.cuda(), kept, new_len)
    status_ok()
    kept, new_len, after = kept.cpu(), new_len.cpu(), c.pools()
    touched = torch.zeros(c.n_pages * page, dtype=torch.bool)
    for b, n in enumerate(lens):
        w = before["weight"][c.slots(b, range(n))].tolist()
        want = P.survivors(w, n, topk, window)
        m = len(want)
        assert int(new_len[b]) == m
        assert kept[b, :m].tolist() == want and (kept[b, m:] == -1).all()
        src = c.slots(b, want)
        to = c.slots(b, range(m), None if in_place else dst)
        touched[to] = True
        for name, t in after.items():
            bits = lambda a: a.contiguous().view(torch.uint8)       # noqa: E731
            assert torch.equal(bits(t[to]), bits(before[name][src])), (name, b)
    for name, t in after.items():
        bits = lambda a: a[~touched].contiguous().view(torch.uint8)     # noqa: E731
        assert torch.equal(bits(t), bits(before[name])), name


HEAVY = lambda w: torch.exp(8 * w - 4)                              # noqa: E731
TIES = lambda w: torch.floor(w * 3)                                 # noqa: E731


def ODD(w):
    w = w.clone()
    w[::7] = float("nan")
    w[1::11] = float("inf")
    w[2::13] = -0.0
    w[3::17] = 0.0
    w[4::19] = -1.0
    return w


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("lens,topk,window,heads,D,page,fp8", [
    ([1, 5, 0], 4, 2, 1, 64, 8, False),
    ([100, 33, 6], 20, 8, 1, 128, 16, True),
    ([1217, 1152, 1153], 1024, 128, 1, 128, 16, True),
    ([500, 40], 0, 32, 2, 64, 32, False),
    ([700, 300], 511, 1, 4, 128, 1, False),
    ([9000, 2000], 1024, 128, 1, 128, 64, False),
    ([4100], 4000, 1, 8, 64, 256, True),
])
def test_evict(lens, topk, window, heads, D, page, fp8, in_place):
    spare = len(lens) * (-(-(topk + window) // page)) + 1
    for weights in (HEAVY, TIES, ODD):
        evict_case(lens, topk, window, heads, D, page, fp8, in_place, weights, spare=spare)


def test_evict_from_a_cache_beyond_shared_memory():
    # more candidates per CTA than it keeps in shared memory
    evict_case([250000, 10], 300, 16, 1, 64, 128, True, True, HEAVY)
    evict_case([250000], 5000, 16, 1, 64, 128, True, True, TIES)


def test_evict_refuses_a_short_destination_table():
    c = P.Cache([40, 40], 16, 1, 64, False, seed=31, weight=True)
    kept = torch.empty(2, 24, dtype=torch.int32, device="cuda")
    short = torch.zeros(1, 2, dtype=torch.int32, device="cuda")      # one row for two sequences
    with pytest.raises(hs2.Hs2Error):
        hs2.hs2_paged_evict(c.struct, 2, 1, 64, c.dt, 20, 4, short, kept, kept[:, 0].contiguous())


def test_evict_twice_and_replayed():
    # into the same pages twice, and from a graph: the source stays as it was
    c = P.Cache([900, 300], 16, 2, 64, True, seed=32, weight=True, spare=2 * 8 + 1)
    dst = c.free[:16].reshape(2, 8).cuda()
    kept = torch.empty(2, 128, dtype=torch.int32, device="cuda")
    new_len = torch.empty(2, dtype=torch.int32, device="cuda")
    call = lambda: hs2.hs2_paged_evict(c.struct, 2, 2, 64, c.dt, 100, 28, dst, kept, new_len)  # noqa: E731
    call()
    status_ok()
    first = [t.clone() for t in (c.k.view(torch.uint8), c.v_scale, c.weight, kept, new_len)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(2):
        kept.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(first, (c.k.view(torch.uint8), c.v_scale, c.weight, kept, new_len)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_evict_large_batch():
    evict_case([50 + 3 * i for i in range(300)], 64, 16, 1, 64, 16, False, True, HEAVY)


# ------------------------------------------------------------- the path as a whole --
@pytest.mark.parametrize("fp8", [False, True])
def test_decode_steps_with_eviction(fp8):
    """Append, attend with weights, evict, again: the cache stays what the definitions make it."""
    B, heads, H, D, page, topk, window = 3, 2, 16, 64, 16, 24, 8
    c = P.Cache([30, 1, 31], page, heads, D, fp8, seed=40, weight=True, max_pages=4, spare=8)
    # every sequence owns its four pages for good
    c.table = torch.randperm(c.n_pages, generator=torch.Generator().manual_seed(1))[:12].to(
        torch.int32).reshape(3, 4)
    c.table_dev.copy_(c.table.cuda())
    c.len_dev.zero_()
    c.lens = [0, 0, 0]
    g = torch.Generator().manual_seed(41)
    model = [[] for _ in range(B)]        # per sequence: (k, v, weight) rows in order
    kept = torch.empty(B, topk + window, dtype=torch.int32, device="cuda")
    scale = D ** -0.5
    for step in range(45):
        kv = torch.randn(B, 2, heads * D, generator=g).bfloat16()
        c.len_dev += 1
        c.lens = [n + 1 for n in c.lens]
        dev = kv.cuda()
        hs2.hs2_paged_append(dev[:, 0], dev[:, 1], dev.stride(0), B, None, c.struct, B, heads, D,
                             c.dt)
        pools = c.pools()
        for b in range(B):
            slot = c.slots(b, [c.lens[b] - 1])
            rows = []
            for i, name in enumerate(("k", "v")):
                r = pools[name][slot][0].double()
                if fp8:
                    r = r * pools[name + "_scale"][slot][0].double()[:, None]
                x = kv[b, i].view(heads, D).double()
                assert ((r - x).abs() <= (2.0 ** -4 if fp8 else 0) * x.abs()
                        + (2.0 ** -10 * x.abs().amax() if fp8 else 0)).all()
                rows.append(r)
            model[b].append(rows + [0.0])
        for b in range(B):                 # what the model says the cache holds
            slots = c.slots(b, range(c.lens[b]))
            c.k64[slots] = torch.stack([r[0] for r in model[b]])
            c.v64[slots] = torch.stack([r[1] for r in model[b]])
        if fp8:
            c.vc, c.vs = pools["v"], pools["v_scale"]
        q = (2 * torch.randn(B, H, D, generator=g)).bfloat16()
        o, lse = P.run_attention(c, q, scale, accumulate=True)
        eo, el, gain, mass, floor = P.attention(c, q, scale)
        assert (lse.double() - el).abs().max() <= 1e-4
        assert ((o.double() - eo).abs() <= 2.0 ** -8 * eo.abs() + (2.0 ** -8 + 1e-4) * mass
                + floor).all()
        weight = c.weight.cpu().flatten()
        for b in range(B):
            slots = c.slots(b, range(c.lens[b]))
            for j, s in enumerate(slots.tolist()):
                model[b][j][2] += float(gain[s])
                assert abs(float(weight[s]) - model[b][j][2]) <= 1e-3 * model[b][j][2] + 1e-6
        hs2.hs2_paged_evict(c.struct, B, heads, D, c.dt, topk, window, None, kept, c.len_dev)
        status_ok()
        for b in range(B):
            w = [float(weight[s]) for s in c.slots(b, range(c.lens[b])).tolist()]
            want = P.survivors(w, c.lens[b], topk, window)
            assert kept[b, :len(want)].tolist() == want
            model[b] = [model[b][j] for j in want]
            c.lens[b] = len(want)
        assert c.len_dev.tolist() == c.lens
    assert c.lens == [topk + window] * B


def test_pools_beyond_32_bits():
    """Pages whose rows lie more than 2^32 bytes into their pools give what the same pages
    in a small pool give, bit for bit."""
    page, D, lens = 64, 128, [200, 70]
    small = P.Cache(lens, page, 1, D, False, seed=50, weight=True, stale=1.0, spare=4)
    n = 300_000                                      # 4.9 GB for K and as much for V
    high = n - small.n_pages                         # the small pool's pages, at the end
    k, v = (torch.empty(n, page, 1, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    weight = torch.empty(n, page, device="cuda")
    for big, t in ((k, small.k), (v, small.v), (weight, small.weight)):
        big[high:] = t
    table = (small.table_dev.long().clamp(max=small.n_pages) + high).clamp(max=n - 1).int()
    lens_dev = small.len_dev.clone()
    big = hs2.paged_cache(k, v, table, lens_dev, weight=weight)
    q = torch.randn(2, 32, D, generator=torch.Generator().manual_seed(51)).bfloat16().cuda()
    rows = torch.randn(2, 2, D, generator=torch.Generator().manual_seed(52)).bfloat16().cuda()
    ws = torch.empty(hs2.hs2_paged_attn_workspace(2, 32, 1, D), dtype=torch.uint8, device="cuda")
    results = []
    for cache, length in ((small.struct, small.len_dev), (big, lens_dev)):
        o, lse = torch.empty_like(q), torch.empty(2, 32, device="cuda")
        kept = torch.empty(2, 60, dtype=torch.int32, device="cuda")
        hs2.hs2_paged_append(rows[:, 0], rows[:, 1], rows.stride(0), 2, None, cache, 2, 1, D, 0)
        hs2.hs2_paged_attn(q, cache, 2, 32, 1, D, D ** -0.5, 0, o, lse, True, ws, ws.numel())
        hs2.hs2_paged_evict(cache, 2, 1, D, 0, 40, 20, None, kept, length)
        status_ok()
        results.append((o, lse, kept, length))
    for a, b in zip(*results):
        assert torch.equal(a, b)
    for t, s in ((k, small.k), (v, small.v), (weight, small.weight)):
        assert torch.equal(t[high:], s)
