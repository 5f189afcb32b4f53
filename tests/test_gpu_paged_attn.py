"""Paged decode attention (hs2_paged_attn) against its definition in 64 bits.

Tolerances.  Logits: bf16 products are exact in fp32 and E4M3 codes exact in f16, so a
logit is off by the fp32 accumulation of D products (D * 2^-24 of the sum of their
magnitudes) and two or three fp32 multiplications; with |s| < 40 here that is below
2^-24 * 16 * 40 < 4e-5, relative in p.  lse: 1e-4 absolute covers that and log2's error.
O: P is rounded to bf16 (2^-8 of each term; f16 2^-11 for E4M3, below 2^-14 with the
absolute floor that paged_testlib.attention states), the output to bf16 (2^-8):
|err| <= 2^-8 |o| + (2^-8 + 1e-4) * sum_j p_j |v_j| + floor.  Weights: every head's p is
off by 1e-4 relative at most, plus fp32's 2^-23 of the old weight.
"""

import math

import pytest
import torch

import long_context_hs2_b200 as hs2
import paged_testlib as P

pytestmark = pytest.mark.gpu


def queries(B, H, D, seed=1, size=1.0):
    return (size * torch.randn(B, H, D, generator=torch.Generator().manual_seed(seed))).bfloat16()


def check(cache, q, o, lse, scale):
    eo, el, gain, mass, floor = P.attention(cache, q, scale)
    empty = torch.isinf(el)
    assert torch.equal(torch.isinf(lse), empty) and (lse[empty] < 0).all()
    assert (lse.double() - el)[~empty].abs().max() <= 1e-4 if (~empty).any() else True
    err = (o.double() - eo).abs()
    tol = 2.0 ** -8 * eo.abs() + (2.0 ** -8 + 1e-4) * mass + floor
    assert (err <= tol).all(), (err - tol).max()
    return gain


CASES = [
    # lens, H, heads, D, page
    ([1], 8, 1, 64, 16),
    ([777], 8, 1, 64, 16),
    ([127, 128, 129], 32, 1, 128, 64),
    ([0, 1, 2, 15, 16, 17, 500], 32, 1, 128, 16),
    ([1000, 0, 3000, 5, 0], 16, 4, 128, 32),
    ([300, 299], 6, 2, 64, 8),
    ([1500, 33], 24, 8, 128, 256),
    ([257, 1], 32, 32, 64, 128),
    ([400, 90], 32, 1, 128, 1),
    ([211, 64], 20, 1, 64, 4),
    ([513], 17, 1, 128, 2),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,H,heads,D,page", CASES)
def test_matches_definition(lens, H, heads, D, page, fp8):
    c = P.Cache(lens, page, heads, D, fp8, seed=3)
    q = queries(c.B, H, D)
    o, lse = P.run_attention(c, q, 1 / math.sqrt(D))
    check(c, q, o, lse, 1 / math.sqrt(D))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,H,heads,D,page", CASES[3:9])
def test_weights_accumulate(lens, H, heads, D, page, fp8):
    c = P.Cache(lens, page, heads, D, fp8, seed=4, weight=True)
    q = queries(c.B, H, D, seed=5, size=2.0)
    before = c.w.clone()
    for n in (1, 2):
        o, lse = P.run_attention(c, q, 1 / math.sqrt(D), accumulate=True)
        gain = check(c, q, o, lse, 1 / math.sqrt(D))
        got = c.weight.cpu().flatten().double()
        want = before.double() + n * gain
        assert ((got - want).abs() <= 1e-4 * n * gain + 2.0 ** -22 * want).all()
    assert torch.equal(c.weight.cpu().flatten()[~c.live], before[~c.live])   # others untouched


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,H,heads,page", [([150, 20, 300], 32, 32, 16), ([700, 129], 40, 20, 8),
                                               ([260, 5], 160, 5, 64)])
def test_weights_of_many_heads(lens, H, heads, page, fp8):
    # more rows than the weights' tcgen05 pass keeps queries of (256), and an odd number of tiles
    c = P.Cache(lens, page, heads, 128, fp8, seed=15, weight=True)
    q = queries(c.B, H, 128, seed=16, size=2.0)
    before = c.w.double()
    o, lse = P.run_attention(c, q, 1 / math.sqrt(128), accumulate=True)
    gain = check(c, q, o, lse, 1 / math.sqrt(128))
    want = before + gain
    assert ((c.weight.cpu().flatten().double() - want).abs() <= 1e-4 * gain + 2.0 ** -22 * want).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,page", [(128, 16), (64, 16), (128, 4)])
def test_a_live_nan_stays_in_its_sequence(D, page, fp8):
    lens = [300, 260, 140, 1, 90]
    c = P.Cache(lens, page, 1, D, fp8, seed=17, weight=True)
    for b, pool, j in ((0, c.kc, 37), (2, c.vc, 139)):
        row = c.slots(b, [j])
        (pool.view(torch.uint8) if fp8 else pool)[row] = 0x7f if fp8 else float("nan")
    c.upload()
    q = queries(c.B, 32, D, seed=18)
    o, lse = P.run_attention(c, q, 1 / math.sqrt(D), accumulate=True)
    assert torch.isnan(o[0]).all() and torch.isnan(lse[0]).all()
    assert torch.isnan(o[2]).all() and torch.isfinite(lse[2]).all()
    eo, el, _, mass, floor = P.attention(c, q, 1 / math.sqrt(D))
    for b in (1, 3, 4):
        assert (lse[b].double() - el[b]).abs().max() <= 1e-4
        tol = 2.0 ** -8 * eo[b].abs() + (2.0 ** -8 + 1e-4) * mass[b] + floor[b]
        assert ((o[b].double() - eo[b]).abs() <= tol).all()
    w = c.weight.cpu().flatten()
    for b in (1, 3, 4):
        assert torch.isfinite(w[c.slots(b, range(lens[b]))]).all()


def test_call_after_call_and_side_by_side():
    # two caches, two workspaces, two streams at once; then the same call twice in a row
    cs = [P.Cache([3000, 17], 64, 1, 128, fp8, seed=19) for fp8 in (False, True)]
    q = queries(2, 32, 128, seed=20)
    want = [P.run_attention(c, q, 0.1) for c in cs]
    n = hs2.hs2_paged_attn_workspace(2, 32, 1, 128)
    qd = q.cuda()
    bufs = [(torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty_like(qd),
             torch.empty(2, 32, device="cuda"), torch.cuda.Stream()) for _ in cs]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, (ws, o, lse, stream) in zip(cs, bufs):
            hs2.hs2_paged_attn(qd, c.struct, 2, 32, 1, 128, 0.1, c.dt, o, lse, False, ws, n,
                               stream=stream)
    torch.cuda.synchronize()
    for (ws, o, lse, _), (wo, wl) in zip(bufs, want):
        assert torch.equal(o.cpu(), wo) and torch.equal(lse.cpu(), wl)


@pytest.mark.parametrize("fp8", [False, True])
def test_long_ragged_batch(fp8):
    # more items than CTAs, and one sequence over many CTAs
    lens = [20000, 3, 0, 7000] + [(37 * i) % 300 for i in range(200)]
    c = P.Cache(lens, 64, 1, 128, fp8, seed=6)
    q = queries(c.B, 32, 128, seed=7)
    o, lse = P.run_attention(c, q, 1 / math.sqrt(128))
    check(c, q, o, lse, 1 / math.sqrt(128))


@pytest.mark.parametrize("D,page,spare", [(64, 1, 0), (128, 1, 0), (128, 8, 0), (128, 512, 1)])
def test_smallest_pools_and_empty_batches(D, page, spare):
    for lens in ([1], [0, 0], [0, 1, 0]):
        if sum(lens) + spare == 0:
            spare = 1
        c = P.Cache(lens, page, 1, D, False, seed=21, spare=spare, weight=True)
        q = queries(c.B, 8, D, seed=22)
        o, lse = P.run_attention(c, q, 0.1, accumulate=True)
        gain = check(c, q, o, lse, 0.1)
        assert ((c.weight.cpu().flatten().double() - c.w.double() - gain).abs() <= 2.0 ** -20).all()


def test_sharp_softmax_raises_references_late():
    # logits that grow along the cache, the heaviest position last
    c = P.Cache([2000], 32, 1, 128, False, seed=8)
    q = queries(1, 32, 128, seed=9)
    ramp = torch.linspace(0, 1.5, 2000)[:, None] * q[0].float().mean(0)[None]
    rows = c.slots(0, range(2000))
    c.kc[rows, 0] = (c.kc[rows, 0].float() * 0.1 + 4 * ramp).bfloat16()
    c.k64 = c.kc.double()
    c.upload()
    o, lse = P.run_attention(c, q, 0.5)
    check(c, q, o, lse, 0.5)


def test_e4m3_scales_of_any_size():
    # v_scale from 1e-6 to 1e6 in one cache, and queries beyond f16's range
    c = P.Cache([600, 140], 16, 1, 128, True, seed=10, scale_range=(1e-6, 1e6))
    c.ks = torch.rand(c.ks.shape, generator=torch.Generator().manual_seed(2)) * 1e-7
    c.k64 = c.kc.double() * c.ks.double()[..., None]
    c.k64[~c.live] = 0
    c.upload()
    q = queries(2, 32, 128, seed=11, size=1e6)
    o, lse = P.run_attention(c, q, 1 / math.sqrt(128))
    check(c, q, o, lse, 1 / math.sqrt(128))


def test_bad_pages_and_lengths_are_reported_and_left_out():
    c = P.Cache([300, 200], 16, 1, 64, False, seed=12)
    bad = c.table.clone()
    bad[0, 3] = -1                      # positions 48..63
    bad[0, 7] = c.n_pages               # positions 112..127
    c.table_dev.copy_(bad.cuda())
    q = queries(2, 8, 64)
    ws = torch.empty(hs2.hs2_paged_attn_workspace(2, 8, 1, 64), dtype=torch.uint8, device="cuda")
    o = torch.empty(2, 8, 64, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(2, 8, device="cuda")
    hs2.hs2_paged_attn(q.cuda(), c.struct, 2, 8, 1, 64, 0.125, c.dt, o, lse, False, ws, ws.numel())
    assert hs2.hs2_last_device_status() == 6
    keep = [j for j in range(300) if not (48 <= j < 64 or 112 <= j < 128)]
    rows = c.slots(0, keep)
    for h in range(8):
        s = c.k64[rows, 0] @ q[0, h].double() * 0.125
        assert abs(float(lse[0, h]) - float(torch.logsumexp(s, 0))) <= 1e-4
    assert torch.isfinite(o).all()
    # a length beyond the table is cut to what the table names
    c.table_dev.copy_(c.table.cuda())
    c.len_dev[1] = c.max_pages * 16 + 1
    c.table_dev[1] = c.table_dev[0]
    hs2.hs2_paged_attn(q.cuda(), c.struct, 2, 8, 1, 64, 0.125, c.dt, o, lse, False, ws, ws.numel())
    assert hs2.hs2_last_device_status() == 6
    assert hs2.hs2_last_device_status() == 0


def test_shared_pages_streams_and_replay():
    # two sequences over the same pages; on another stream; captured and replayed
    c = P.Cache([500, 500], 32, 2, 128, False, seed=13)
    c.table[1] = c.table[0]
    c.live[:] = False
    c.live[c.slots(0, range(500))] = True
    c.table_dev.copy_(c.table.cuda())
    q = queries(2, 16, 128, seed=14)
    scale = 1 / math.sqrt(128)
    want = P.run_attention(c, q, scale)
    check(c, q, *want, scale)
    n = hs2.hs2_paged_attn_workspace(2, 16, 2, 128)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    qd, o, lse = q.cuda(), torch.empty(2, 16, 128, dtype=torch.bfloat16, device="cuda"), \
        torch.empty(2, 16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        hs2.hs2_paged_attn(qd, c.struct, 2, 16, 2, 128, scale, c.dt, o, lse, False, ws, n)
    side.synchronize()
    assert torch.equal(o.cpu(), want[0]) and torch.equal(lse.cpu(), want[1])
    graphs = []
    for _ in range(2):                 # two graphs over one workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            hs2.hs2_paged_attn(qd, c.struct, 2, 16, 2, 128, scale, c.dt, o, lse, False, ws, n)
        graphs.append(g)
    for g in graphs + graphs:
        o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o.cpu(), want[0]) and torch.equal(lse.cpu(), want[1])
    # lengths are read when the work runs: the replay follows the cache's growth
    c.len_dev.copy_(torch.tensor([499, 37], dtype=torch.int32))
    c.lens = [499, 37]
    graphs[0].replay()
    torch.cuda.synchronize()
    check(c, q, o.cpu(), lse.cpu(), scale)
