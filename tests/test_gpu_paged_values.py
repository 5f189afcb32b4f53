"""Values that the paged decode path meets at its edges, against the definitions in 64 bits:
rows of zeros, scales of any size, infinities and NaN among live values, rows that are no
token's.

Tolerances.  As in test_gpu_paged_attn.py, without its floor: over E4M3 pages a probability
times its v_scale goes to the tensor cores as two bf16 terms, which are off by 2^-8 * 2^-8 of
it at any size, so |err| <= 2^-8 |o| + (2^-8 + 1e-4) * sum_j p_j |v_j|, and rows that add
nothing to the output widen nothing.
"""

import math

import pytest
import torch

import long_context_hs2_b200 as hs2
import paged_testlib as P

pytestmark = pytest.mark.gpu

PATHS = [(128, 16), (64, 16), (128, 4)]      # head size, page: tcgen05, warp MMAs, small pages


def pull(c, q, positions, gap):
    """These positions of sequence 0 get a key whose logit (scale 1 / sqrt(D)) is `gap` nats for
    every query row of q, which must share a direction: q[0, :, 0] == 8."""
    rows = c.slots(0, positions)
    c.kc.view(torch.uint8)[rows] = 0
    c.kc.view(torch.uint8)[rows, :, 0] = 0x78                     # 256
    c.ks[rows] = gap * math.sqrt(c.D) / (8 * 256.0)
    c.k64[rows] = c.kc.view(torch.uint8)[rows].view(P.E4M3).double() * c.ks[rows].double()[..., None]


def queries(B, H, D, seed=1):
    q = 0.3 * torch.randn(B, H, D, generator=torch.Generator().manual_seed(seed))
    q[:, :, 0] = 8
    return q.bfloat16()


def check(c, q, o, lse, size=40):
    # a logit of magnitude `size` is off by 16 * 2^-24 of it (4e-5 of 40); log2 and the sums by
    # 6e-5 more
    eps = 16 * 2.0 ** -24 * size + 6e-5
    eo, el, gain, mass, _ = P.attention(c, q, c.D ** -0.5)
    assert (lse.double() - el).abs().max() <= eps
    tol = 2.0 ** -8 * eo.abs() + (2.0 ** -8 + eps) * mass
    assert ((o.double() - eo).abs() <= tol).all(), ((o.double() - eo).abs() / tol).max()
    return gain


@pytest.mark.parametrize("D,page", PATHS)
@pytest.mark.parametrize("gap,scale", [(10, 1e-3), (10, 1e-4), (10, 1e-7), (0, 1e-7), (20, 1e-5)])
@pytest.mark.parametrize("codes", ["zeros", "one column"])
def test_a_heavy_v_row_that_adds_little(D, page, gap, scale, codes):
    # hs2_paged_append gives a row of zeros the scale 1, whatever its neighbours' scales are
    c = P.Cache([700, 90], page, 1, D, True, seed=60, scale_range=(scale / 3, scale * 3), weight=True)
    c.ks = c.ks * (1e-1 / scale)                          # logits of ordinary size
    c.k64 = c.kc.double() * c.ks.double()[..., None]
    c.k64[~c.live] = 0
    q = queries(2, 32, D)
    for j in (5, 300):
        pull(c, q, [j], gap)
        row = c.slots(0, [j])
        c.vc.view(torch.uint8)[row] = 0
        if codes == "one column":
            c.vc.view(torch.uint8)[row, :, 3] = 0x7e         # 448
        c.vs[row] = 1.0
        c.v64[row] = c.vc.view(torch.uint8)[row].view(P.E4M3).double()
    c.upload()
    before = c.w.double()
    o, lse = P.run_attention(c, q, D ** -0.5, accumulate=True)
    gain = check(c, q, o, lse)
    want = before + gain
    assert ((c.weight.cpu().flatten().double() - want).abs() <= 1e-4 * gain + 2.0 ** -22 * want).all()


@pytest.mark.parametrize("D,page", PATHS)
@pytest.mark.parametrize("lo,hi", [(1e-35, 1e-33), (1e-30, 1e-3), (1e-12, 1e12), (1e20, 1e22)])
def test_v_scales_of_any_size(D, page, lo, hi):
    c = P.Cache([400, 33], page, 1, D, True, seed=61, scale_range=(lo, hi))
    c.ks = torch.rand(c.ks.shape, generator=torch.Generator().manual_seed(2)) * 1e-2
    c.k64 = c.kc.double() * c.ks.double()[..., None]
    c.k64[~c.live] = 0
    c.upload()
    q = queries(2, 20, D, seed=62)
    check(c, q, *P.run_attention(c, q, D ** -0.5))


@pytest.mark.parametrize("D,page", PATHS)
def test_a_flat_tail_under_peaks_without_values(D, page):
    # every 50th position takes nearly all probability and has no value; the others' are 2^-27 of it
    c = P.Cache([5000], page, 1, D, True, seed=63)
    c.kc.view(torch.uint8)[c.live] = 0
    c.k64 = torch.zeros_like(c.k64)
    q = queries(1, 8, D, seed=64)
    peaks = range(7, 5000, 50)
    pull(c, q, peaks, 27 * math.log(2))
    rows = c.slots(0, peaks)
    c.vc.view(torch.uint8)[rows] = 0
    c.v64[rows] = 0
    c.upload()
    check(c, q, *P.run_attention(c, q, D ** -0.5))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,page", PATHS)
def test_rows_of_nan(D, page, fp8):
    # a NaN query; a sequence whose only key is NaN; sixteen NaN keys side by side
    lens = [300, 1, 260, 700]
    c = P.Cache(lens, page, 1, D, fp8, seed=67, weight=True)
    for b, js in ((1, [0]), (2, range(128, 144)), (3, range(700))):
        (c.kc.view(torch.uint8) if fp8 else c.kc)[c.slots(b, js)] = 0x7f if fp8 else float("nan")
    c.upload()
    q = torch.randn(4, 32, D, generator=torch.Generator().manual_seed(68)).bfloat16()
    q[0, 9] = float("nan")
    o, lse = P.run_attention(c, q, D ** -0.5, accumulate=True)
    undefined = torch.zeros(4, 32, dtype=torch.bool)
    undefined[1:] = True
    undefined[0, 9] = True
    assert torch.equal(torch.isnan(o).all(2), undefined)
    assert torch.equal(torch.isnan(lse), undefined)
    assert torch.isfinite(o[~undefined]).all() and torch.isfinite(lse[~undefined]).all()
    w = c.weight.cpu().flatten()
    for b, n in enumerate(lens):         # every head's probability is in the sum
        assert torch.isnan(w[c.slots(b, range(n))]).all()


@pytest.mark.parametrize("D,page", PATHS)
@pytest.mark.parametrize("sign", [0, 1, -1])
@pytest.mark.parametrize("value", [math.inf, -math.inf])
def test_an_infinite_query_is_undefined(D, page, sign, value):
    # its logits are infinities of one sign (all codes of that column of one sign) or of both,
    # and exp(s - lse) is NaN in each case; no other row notices
    c = P.Cache([300, 40], page, 1, D, True, seed=65)
    if sign:
        c.kc[:, :, 7] = (c.kc[:, :, 7].float().abs().clamp(min=1) * sign).to(P.E4M3)
        c.k64 = c.kc.double() * c.ks.double()[..., None]
        c.k64[~c.live] = 0
        c.upload()
    q = torch.randn(2, 32, D, generator=torch.Generator().manual_seed(66)).bfloat16()
    q[0, 5, 7] = value
    o, lse = P.run_attention(c, q, D ** -0.5)
    assert torch.isnan(o[0, 5]).all() and not torch.isfinite(lse[0, 5])
    q[0, 5] = 0
    o[0, 5], lse[0, 5] = (t[0, 5] for t in P.run_attention(c, q, D ** -0.5))
    check(c, q, o, lse)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lead,n_rows", [(0, 50_000), (37, 5_000), (64, 107)])
def test_append_with_an_upper_bound_of_rows(lead, n_rows, fp8):
    # K and V hold the 43 tokens' rows only; row `lead` of the call is their first
    lens, rows = [40, 3, 9], [31, 3, 9]
    c = P.Cache(lens, 16, 2, 64, fp8, seed=70, weight=True)
    kv = torch.randn(2, sum(rows), 128, generator=torch.Generator().manual_seed(71)).bfloat16()
    dev = kv.cuda()
    start = torch.tensor([lead, lead + 31, lead + 34, lead + 43], dtype=torch.int32, device="cuda")
    k, v = (t.data_ptr() - lead * 128 * 2 for t in dev)
    before = c.pools()
    hs2.hs2_paged_append(k, v, 128, n_rows, start, c.struct, 3, 2, 64, c.dt)
    assert hs2.hs2_last_device_status() == 0
    after = c.pools()
    touched = torch.zeros(c.n_pages * 16, dtype=torch.bool)
    for b, n in enumerate(rows):
        slots = c.slots(b, range(lens[b] - n, lens[b]))
        touched[slots] = True
        for name, x in zip(("k", "v"), kv[:, sum(rows[:b]):sum(rows[:b + 1])].unflatten(-1, (2, 64))):
            if fp8:
                got = after[name + "_scale"][slots]
                assert ((got.double() - x.double().abs().amax(-1) / 448).abs()
                        <= 2.0 ** -23 * got).all()
                P.assert_codes(after[name][slots], x, got[..., None], 2.0 ** -22 * x.double().abs())
            else:
                assert torch.equal(after[name][slots], x)
    for name, t in after.items():
        bits = lambda a: a[~touched].contiguous().view(torch.uint8)     # noqa: E731
        assert torch.equal(bits(t), bits(before[name])), name


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("size", [1.0, 1e-30, 1e30, 3e-37])
def test_append_writes_the_definitions_codes(D, size):
    # bf16 values lie half-way between two codes often: one in 4,000 of these, at size 1
    n = 3000
    c = P.Cache([n], 64, 1, D, True, seed=72)
    kv = (size * torch.randn(n, 2 * D, generator=torch.Generator().manual_seed(73))).bfloat16()
    kv[5, ::3] = -0.0
    kv[9, 7] = math.inf
    kv[11, :] = 0
    dev = kv.cuda()
    start = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    hs2.hs2_paged_append(dev[:, :D], dev[:, D:], 2 * D, n, start, c.struct, 1, 1, D, c.dt)
    assert hs2.hs2_last_device_status() == 0
    after = c.pools()
    rows = c.slots(0, range(n))
    for name, x in (("k", kv[:, :D].float()), ("v", kv[:, D:].float())):
        s = x.abs().amax(1) / 448
        s = torch.where(s > 0, s, torch.ones_like(s))
        codes = (x / s[:, None]).to(P.E4M3).view(torch.uint8)
        assert torch.equal(after[name + "_scale"][rows, 0], s)
        got = after[name].view(torch.uint8)[rows, 0]
        bad = torch.isnan(x / s[:, None])
        assert torch.equal(got[~bad], codes[~bad])
        assert (got[bad] & 0x7f == 0x7f).all()


@pytest.mark.parametrize("hidden", [48, 4096])
def test_norm_writes_the_definitions_codes_of_powers_of_two(hidden):
    # rows of +-1 and of halves and quarters of it have a norm and quotients that are exact but
    # for the scale: many quotients are ties
    g = torch.Generator().manual_seed(74)
    x = torch.ones(200, hidden) * (torch.randint(0, 2, (200, hidden), generator=g) * 2 - 1)
    gamma = (torch.randint(1, 256, (hidden,), generator=g) / 256).bfloat16()
    codes = torch.empty(200, hidden, dtype=P.E4M3, device="cuda")
    scale = torch.empty(200, -(-hidden // 128), device="cuda")
    hs2.hs2_add_rmsnorm(x.bfloat16().cuda(), None, gamma.cuda(), 200, hidden, 0.0, None, None, codes,
                        scale)
    assert hs2.hs2_last_device_status() == 0
    y = x * gamma.float()                            # mean(x^2) = 1, exactly
    for i, part in enumerate(y.split(128, 1)):
        s = part.abs().amax(1, keepdim=True) / 448
        assert torch.equal(scale[:, i].cpu(), s[:, 0])
        want = (part / s).to(P.E4M3).view(torch.uint8)
        got = codes.cpu().view(torch.uint8)[:, i * 128:i * 128 + part.shape[1]]
        assert torch.equal(got, want)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,page", PATHS)
def test_logits_that_overflow_for_one_row(D, page, fp8):
    # the first keys are out of row 0's reach (its logit with them is below fp32's range, the
    # other rows' is small), and its logits with the others are all near -400
    c = P.Cache([900], page, 1, D, fp8, seed=75)
    k = 0.5 * torch.randn(900, D, generator=torch.Generator().manual_seed(76))
    k[:, 0] = 0
    k[:, 1] = -400 * math.sqrt(D) / 8
    far = torch.zeros(900, dtype=torch.bool)
    far[:500] = True
    far[700] = True
    rows = c.slots(0, range(900))
    if fp8:
        codes, scale = P.quantise(k)
        codes.view(torch.uint8)[far] = 0
        codes.view(torch.uint8)[far, 0] = 0xfe               # -448
        scale[far] = 1e36
        c.kc.view(torch.uint8)[rows, 0] = codes.view(torch.uint8)
        c.ks[rows] = scale.float()
        c.k64[rows, 0] = codes.double() * scale.float().double()
    else:
        k[far] = 0
        k[far, 0] = -3e38
        c.kc[rows, 0] = k.bfloat16()
        c.k64[rows, 0] = k.bfloat16().double()
    c.upload()
    q = torch.randn(1, 32, D, generator=torch.Generator().manual_seed(77))
    q[0, :, :2] = 0
    q[0, 0, 0] = 256
    q[0, :5, 1] = 8
    check(c, q.bfloat16(), *P.run_attention(c, q.bfloat16(), D ** -0.5), size=420)
