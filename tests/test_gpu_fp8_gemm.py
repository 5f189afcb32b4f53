"""hs2_fp8_gemm against its definition in 64 bits.

Tolerance.  Products of E4M3 codes are exact in fp32; a block's 128 of them are summed on
the tensor cores in fp32 (each of the few sequential additions off by at most 2^-23 of the
partial sum's magnitude, which sum |a b| bounds: under 128 * 2^-23), then scaled and added
over the blocks in fp32 (kb + 2 roundings of 2^-24 each, and up to 8 more to join a split).
With S = sum_kb s_kb sum |a b|:  |err| <= 2^-8 |c| + (128 * 2^-23 + (kb + 10) * 2^-24) S.
"""

import pytest
import torch

import long_context_hs2_b200 as hs2
import paged_testlib as P

pytestmark = pytest.mark.gpu


def operands(M, N, K, seed=0, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    kb, nb = -(-K // 128), -(-N // 128)
    a = torch.randn(M, K, generator=g).mul(100).clamp(-448, 448).to(P.E4M3)
    b = torch.randn(N, K, generator=g).mul(100).clamp(-448, 448).to(P.E4M3)
    sa = torch.exp(spread * torch.randn(M, kb, generator=g)) / 100
    sb = torch.exp(spread * torch.randn(nb, kb, generator=g)) / 100
    return a, sa, b, sb


def definition(a, sa, b, sb):
    """(C, S) in 64 bits, on the GPU for speed."""
    a, sa, b, sb = (t.cuda().double() for t in (a, sa, b, sb))
    M, K = a.shape
    N = b.shape[0]
    rows = torch.arange(N, device="cuda") // 128
    c = torch.zeros(M, N, dtype=torch.float64, device="cuda")
    s = torch.zeros_like(c)
    for kb, k0 in enumerate(range(0, K, 128)):
        x, y = a[:, k0:k0 + 128], b[:, k0:k0 + 128]
        f = sa[:, kb, None] * sb[rows, kb]
        c += f * (x @ y.t())
        s += f.abs() * (x.abs() @ y.abs().t())
    return c, s


def run(a, sa, b, sb):
    M, K = a.shape
    N = b.shape[0]
    c = torch.full((M + 1, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    hs2.hs2_fp8_gemm(a.cuda(), sa.cuda(), M, b.cuda(), sb.cuda(), N, K, c)
    st = hs2.hs2_last_device_status()
    assert st == 0, hs2.hs2_status_string(st)
    assert torch.isnan(c[M]).all()                  # nothing behind the last row
    return c[:M]


def check(a, sa, b, sb):
    got = run(a, sa, b, sb)
    c, s = definition(a, sa, b, sb)
    kb = -(-a.shape[1] // 128)
    tol = 2.0 ** -8 * c.abs() + (128 * 2.0 ** -23 + (kb + 10) * 2.0 ** -24) * s
    assert ((got.double() - c).abs() <= tol).all()
    return got


@pytest.mark.parametrize("M", [1, 8, 16, 17, 33, 64, 65, 128, 129, 200, 400, 1003])
@pytest.mark.parametrize("N,K", [(1536, 4096), (1, 16), (130, 144), (257, 1040)])
def test_sizes(M, N, K):
    check(*operands(M, N, K, seed=M + N))


@pytest.mark.parametrize("M,N,K", [(5000, 1536, 256), (2500, 2049, 400), (20000, 40, 128),
                                   (300, 8192, 128), (3, 5000, 2048), (128, 127, 16),
                                   (20000, 333, 144), (9000, 1030, 64), (700, 36, 272)])
def test_shapes_of_every_variant(M, N, K):
    check(*operands(M, N, K, seed=3))


def test_scales_of_any_size_and_zero_rows():
    a, sa, b, sb = operands(150, 300, 512, seed=4, spread=8.0)
    a[7] = torch.zeros(512).to(P.E4M3)
    got = check(a, sa, b, sb)
    assert (got[7] == 0).all()
    a, sa, b, sb = operands(9, 300, 512, seed=5, spread=8.0)
    check(a, sa, b, sb)


def test_largest_codes():
    for M in (20, 300):
        a, sa, b, sb = operands(M, 256, 1024, seed=6)
        a = torch.full((M, 1024), 448.0).to(P.E4M3)
        b = torch.full((256, 1024), -448.0).to(P.E4M3)
        check(a, sa, b, sb)


def test_runs_agree_bit_for_bit_and_replay():
    for M in (24, 700):
        a, sa, b, sb = (t.cuda() for t in operands(M, 1536, 1024, seed=7))
        want = run(a, sa, b, sb)
        c = torch.empty(M, 1536, dtype=torch.bfloat16, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            hs2.hs2_fp8_gemm(a, sa, M, b, sb, 1536, 1024, c)
        for _ in range(3):
            c.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(c, want)


def test_norm_feeds_the_product():
    """The projection of a normalised hidden state, as the decode path runs it."""
    T, hidden, N = 70, 1040, 384
    g = torch.Generator().manual_seed(8)
    x = torch.randn(T, hidden, generator=g).bfloat16()
    gamma = (1 + 0.2 * torch.randn(hidden, generator=g)).bfloat16()
    _, _, b, sb = operands(T, N, hidden, seed=9)
    yq = torch.empty(T, hidden, dtype=P.E4M3, device="cuda")
    ys = torch.empty(T, -(-hidden // 128), device="cuda")
    hs2.hs2_add_rmsnorm(x.cuda(), None, gamma.cuda(), T, hidden, 1e-6, None, None, yq, ys)
    check(yq.cpu(), ys.cpu(), b, sb)
