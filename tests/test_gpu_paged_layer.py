"""A layer's decode step over a paged cache (long_context_hs2_b200/paged.py), all five
operators in order, against the same step in 64 bits on the values that the GPU cached.

Tolerances.  The step's parts are held to their own bounds by their own tests; here the
parts are checked where they meet.  The residual: one bf16 rounding (2^-8).  Queries and
K/V rows: the projection of the E4M3 codes, in 64 bits from the codes and scales the GPU
wrote: 2^-8 |c| + 2^-15 S (test_gpu_fp8_gemm.py's bound, kb <= 8).  The attention: as in
test_gpu_paged_attn.py, from the rows in the GPU's pages.  Kept positions: equal.
"""

import pytest
import torch

import long_context_hs2_b200 as hs2
import paged_testlib as P
from long_context_hs2_b200.paged import PagedConfig, PagedLayer

pytestmark = pytest.mark.gpu


def make(fp8, D=128, H=32, kv_heads=1, seed=0, **kw):
    cfg = PagedConfig(B=3, hidden=528, H=H, kv_heads=kv_heads, D=D, fp8=fp8, page_size=16, topk=20,
                      window=12, interval=16, **kw)
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)          # noqa: E731
    gamma = (1 + 0.2 * rnd(cfg.hidden)).bfloat16().cuda()
    w_q = (rnd(H * D, cfg.hidden) / cfg.hidden ** 0.5 * 1.5).bfloat16().cuda()
    w_kv = (rnd(2 * kv_heads * D, cfg.hidden) / cfg.hidden ** 0.5).bfloat16().cuda()
    return cfg, PagedLayer(cfg, gamma, w_q, w_kv), rnd


def product(codes, scale, w, w_scale):
    a, b = codes.cpu().double(), w.cpu().double()
    c, s = 0, 0
    rows = torch.arange(b.shape[0]) // 128
    for kb, k0 in enumerate(range(0, a.shape[1], 128)):
        f = scale.cpu().double()[:, kb, None] * w_scale.cpu().double()[rows, kb]
        x, y = a[:, k0:k0 + 128], b[:, k0:k0 + 128]
        c, s = c + f * (x @ y.t()), s + f * (x.abs() @ y.abs().t())
    return c, s


class View:
    """What paged_testlib.attention wants, from a layer's pages."""

    def __init__(self, layer):
        c = layer.cfg
        self.lens, self.page, self.heads, self.fp8 = layer.seq_len.tolist(), c.page_size, c.kv_heads, c.fp8
        self.n_pages, self.table = layer.k.shape[0], layer.table.cpu()
        k, v = (t.cpu().flatten(0, 1) for t in (layer.k, layer.v))
        if c.fp8:
            k, v = k.view(P.E4M3), v.view(P.E4M3)
            ks, self.vs = (t.cpu().flatten(0, 1) for t in (layer.k_scale, layer.v_scale))
            self.vc = v
            self.k64 = k.double() * ks.double()[..., None]
            self.v64 = v.double() * self.vs.double()[..., None]
        else:
            self.k64, self.v64 = k.double(), v.double()

    slots = P.Cache.slots


@pytest.mark.parametrize("fp8,D,H,kv_heads", [(True, 128, 32, 1), (False, 128, 16, 2),
                                              (True, 64, 8, 4), (False, 64, 32, 1)])
def test_steps(fp8, D, H, kv_heads):
    cfg, layer, rnd = make(fp8, D, H, kv_heads)
    residual = rnd(cfg.B, cfg.hidden).bfloat16().cuda()
    n = 0
    for step in range(70):
        x = rnd(cfg.B, cfg.hidden).bfloat16().cuda()
        h = x.cpu().double() + residual.cpu().double()
        evicts = layer.steps == cfg.interval
        before = [layer.weight.cpu().flatten()[View(layer).slots(b, range(n))].tolist()
                  for b in range(cfg.B)] if evicts else None
        out = layer.step(x, residual)
        assert hs2.hs2_last_device_status() == 0
        if evicts:
            m = min(n, cfg.topk + cfg.window)
            for b in range(cfg.B):
                assert layer.kept[b, :m].tolist() == P.survivors(before[b], n, cfg.topk, cfg.window)
            n = m
        n += 1
        assert layer.seq_len.tolist() == [n] * cfg.B
        assert ((residual.cpu().double() - h).abs() <= 2.0 ** -8 * h.abs()).all()
        for got, w, s in ((layer.q, layer.w_q, layer.w_q_scale),
                          (layer.kv, layer.w_kv, layer.w_kv_scale)):
            c, mass = product(layer.codes, layer.codes_scale, w, s)
            got = got.cpu().double().reshape(cfg.B, -1)
            assert ((got - c).abs() <= 2.0 ** -8 * c.abs() + 2.0 ** -15 * mass).all()
        if step % 5 == 0 or evicts:
            eo, el, _, mass, floor = P.attention(View(layer), layer.q.cpu(), D ** -0.5)
            assert (layer.lse.cpu().double() - el).abs().max() <= 1e-4
            assert ((out.cpu().double() - eo).abs() <= 2.0 ** -8 * eo.abs()
                    + (2.0 ** -8 + 1e-4) * mass + floor).all()
    assert n <= cfg.topk + cfg.window + cfg.interval


def test_replayed_steps_match():
    """A captured step (and one with the eviction) replays as the eager ones run."""
    runs = []
    for graph in (False, True):
        cfg, layer, rnd = make(True, seed=3)
        x, residual = (rnd(cfg.B, cfg.hidden).bfloat16().cuda() for _ in range(2))
        layer.step(x, residual)                       # (loads the kernels)
        graphs = {}
        for step in range(1, 40):
            x.copy_(rnd(cfg.B, cfg.hidden).bfloat16())
            if not graph:
                layer.step(x, residual)
                continue
            evicts = layer.steps == cfg.interval
            if evicts not in graphs:
                torch.cuda.synchronize()
                graphs[evicts] = torch.cuda.CUDAGraph()
                steps = layer.steps
                with torch.cuda.graph(graphs[evicts]):
                    layer.step(x, residual)
                layer.steps = steps
            graphs[evicts].replay()
            layer.steps = 1 if evicts else layer.steps + 1
        torch.cuda.synchronize()
        assert hs2.hs2_last_device_status() == 0
        runs.append([t.cpu() for t in (layer.out, layer.lse, layer.weight, layer.seq_len,
                                       layer.kept, residual, layer.k, layer.k_scale)])
    for a, b in zip(*runs):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
