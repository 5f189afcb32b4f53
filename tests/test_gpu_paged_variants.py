"""Variants of the paged decode path's kernels that sizes or alignment choose: E4M3 scales off
16 bytes, evictions from many caches of more candidates than a CTA keeps.
Tolerances as in test_gpu_paged_attn.py; evictions move bits."""

import pytest
import torch

import long_context_hs2_b200 as hs2
import paged_testlib as P
import test_gpu_paged_cache as cache_tests

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("off", [1, 2, 3])
def test_e4m3_scales_off_16_bytes(page, off):
    # whole tiles of one head, whose scales are copied four at a time where they are aligned
    c = P.Cache([1000, 300, 128], page, 1, 128, True, seed=80, weight=True)
    shifted = []
    for s in (c.k_scale, c.v_scale):
        flat = torch.empty(s.numel() + 4, device="cuda")
        flat[off:off + s.numel()] = s.flatten()
        shifted.append(flat[off:off + s.numel()].view_as(s))
        assert shifted[-1].data_ptr() % 16 == 4 * off
    q = torch.randn(3, 32, 128, generator=torch.Generator().manual_seed(81)).bfloat16()
    want = P.run_attention(c, q, 128 ** -0.5, accumulate=True)
    weight = c.weight.clone()
    c.upload()
    c.struct = hs2.paged_cache(c.k, c.v, c.table_dev, c.len_dev, *shifted, c.weight)
    o, lse = P.run_attention(c, q, 128 ** -0.5, accumulate=True)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert torch.equal(c.weight.cpu(), weight.cpu())
    eo, el, _, mass, floor = P.attention(c, q, 128 ** -0.5)
    assert (lse.double() - el).abs().max() <= 1e-4
    assert ((o.double() - eo).abs() <= 2.0 ** -8 * eo.abs() + (2.0 ** -8 + 1e-4) * mass).all()


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("B", [14, 17, 33, 70])
def test_evictions_from_many_long_caches(B, in_place):
    # clusters of 8, 4, 2 and 1 CTAs, all with more candidates than a CTA keeps keys of
    lens = [9000 + 17 * b for b in range(B)]
    for weights in (cache_tests.HEAVY, cache_tests.ODD):
        cache_tests.evict_case(lens, 150, 10, 1, 64, 64, False, in_place, weights, seed=82 + B,
                               spare=3 * B)


def test_the_cache_s_own_table_as_destination_is_in_place():
    outputs = []
    for own in (False, True):
        c = P.Cache([500, 60, 0], 16, 2, 64, True, seed=83, weight=True, stale=1.0)
        kept = torch.empty(3, 80, dtype=torch.int32, device="cuda")
        hs2.hs2_paged_evict(c.struct, 3, 2, 64, c.dt, 70, 10, c.table_dev if own else None, kept,
                            c.len_dev)
        assert hs2.hs2_last_device_status() == 0
        outputs.append([kept.cpu(), c.len_dev.cpu()] + [t.contiguous().view(torch.uint8)
                                                       for t in c.pools().values()])
    for a, b in zip(*outputs):
        assert torch.equal(a, b)
    assert outputs[0][1].tolist() == [80, 60, 0]
