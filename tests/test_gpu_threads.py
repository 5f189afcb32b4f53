"""Calls from several host threads, each on its own stream and buffers.  A kernel's settings
belong to the function: one thread's must not fail another's launch.  A thread that has made
no CUDA call yet has no context of its own: the first one may be this library's."""

import threading

import pytest
import torch

import long_context_hs2_b200 as hs2
import paged_testlib as P

pytestmark = pytest.mark.gpu


def side_by_side(calls, n=16000):
    """Runs every call (a function of a stream) n times in a thread of its own."""
    errors, start = [], threading.Barrier(len(calls))

    def loop(call):
        stream = torch.cuda.Stream()
        start.wait()
        try:
            for _ in range(n):
                call(stream)
        except Exception as e:      # noqa: BLE001 (told to the main thread)
            errors.append(e)

    threads = [threading.Thread(target=loop, args=(c,)) for c in calls]
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    assert hs2.hs2_last_device_status() == 0


def test_evictions_of_caches_of_different_reach():
    calls, results = [], []
    for n, page, topk in ((9000, 64, 1000), (90, 16, 40), (60, 8, 20), (70, 16, 30)):
        c = P.Cache([n], page, 1, 64, False, seed=1, weight=True, stale=1.0,
                    spare=-(-(topk + 8) // page) + 1)
        dst = c.free[:-(-(topk + 8) // page)].reshape(1, -1).cuda()
        kept = torch.empty(1, topk + 8, dtype=torch.int32, device="cuda")
        new_len = torch.empty(1, dtype=torch.int32, device="cuda")
        want = P.survivors(c.w[c.slots(0, range(n))].tolist(), n, topk, 8)
        calls.append(lambda s, a=(c.struct, 1, 1, 64, 0, topk, 8, dst, kept, new_len):
                     hs2.hs2_paged_evict(*a, stream=s))
        results.append((kept, want, c))
    side_by_side(calls)
    for kept, want, _ in results:
        assert kept[0].tolist() == want


def test_the_first_cuda_call_of_a_thread():
    g = torch.Generator().manual_seed(3)
    a, b = (torch.randn(n, 256, generator=g).to(P.E4M3).cuda() for n in (64, 128))
    sa, sb = torch.ones(64, 2, device="cuda"), torch.ones(1, 2, device="cuda")
    c, few = (torch.zeros(m, 128, dtype=torch.bfloat16, device="cuda") for m in (64, 8))
    w = P.Cache([300], 16, 1, 128, False, seed=4)
    q = torch.randn(1, 8, 128, generator=g).bfloat16().cuda()
    o, lse = torch.zeros_like(q), torch.zeros(1, 8, device="cuda")
    n = hs2.hs2_paged_attn_workspace(1, 8, 1, 128)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    x, wt = (torch.randn(m, 256, generator=g).bfloat16().cuda() for m in (40, 256))
    k, v = (torch.zeros(1, 40, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    stream = torch.cuda.current_stream().cuda_stream
    calls = [lambda: hs2.hs2_fp8_gemm(a, sa, 64, b, sb, 128, 256, c, stream=stream),
             lambda: hs2.hs2_fp8_gemm(a, sa, 8, b, sb, 128, 256, few, stream=stream),
             lambda: hs2.hs2_paged_attn(q, w.struct, 1, 8, 1, 128, 0.1, 0, o, lse, False, ws, n,
                                        stream=stream),
             lambda: hs2.hs2_bridge_kv(x, 40, 256, wt, 1, 128, 0, [hs2.kv_cache(k, v)], 0,
                                       stream=stream)]
    outputs = [c, few, o, k]
    for call, out in zip(calls, outputs):
        call()
        torch.cuda.synchronize()
        want = out.clone()
        out.zero_()
        torch.cuda.synchronize()
        errors = []

        def run():
            try:
                call()
            except Exception as e:      # noqa: BLE001 (told to the main thread)
                errors.append(e)

        t = threading.Thread(target=run)
        t.start()
        t.join()
        torch.cuda.synchronize()
        assert not errors, errors
        assert torch.equal(out, want)


def test_merged_selections_of_different_sizes():
    g = torch.Generator().manual_seed(2)
    calls, results = [], []
    for G, topk in ((12, 2000), (2, 16), (3, 40), (1, 8)):
        score = torch.rand(G, 1, 1, topk, generator=g).cuda()
        idx = torch.stack([torch.arange(r * topk, (r + 1) * topk) for r in range(G)]).int()
        idx = idx.reshape(G, 1, 1, topk).cuda()
        sel = torch.empty(1, 1, topk + 4, dtype=torch.int32, device="cuda")
        n_sel = torch.empty(1, 1, dtype=torch.int32, device="cuda")
        last = G * topk + 3                    # every candidate lies before the window
        calls.append(lambda s, a=(score, idx, G, 1, 1, last, topk, 4, sel, n_sel):
                     hs2.hs2_cp_merge_select(*a, stream=s))
        best = torch.topk(score.flatten(), topk).indices.sort().values
        results.append((sel, idx.flatten()[best].tolist() + list(range(last - 3, last + 1))))
    side_by_side(calls)
    for sel, want in results:
        assert sel.flatten().tolist() == want


def test_selections_of_different_lengths():
    # token selection (after the separate passes of a chunk) and selection in blocks of one
    H, D, topk, window = 32, 128, 8, 4
    calls, results = [], []
    for blocks in (False, True):
        for L in (40000, 300, 400):
            T = 1 if blocks else 4
            k, v = (torch.randn(1, L, D, device="cuda").bfloat16() for _ in range(2))
            q = torch.randn(1, T, H, D, device="cuda").bfloat16()
            kv = hs2.kv_cache(k, v)
            n = hs2.hs2_full_attn_select_workspace(1, T, L, H, D, topk, window, 0)
            ws = torch.empty(n, dtype=torch.uint8, device="cuda")
            o, lse = torch.empty(1, T, H, D, device="cuda"), torch.empty(1, T, H, device="cuda")
            idx = torch.empty(1, T, topk + window, dtype=torch.int32, device="cuda")
            ns = torch.empty(1, T, dtype=torch.int32, device="cuda")
            head = (q, kv, 1, T, L, H, D, D ** -0.5, topk, window)
            tail = (0, o, lse, idx, ns, ws, n)
            call = ((lambda s, a=head + (1,) + tail: hs2.hs2_full_attn_select_blocks(*a, stream=s))
                    if blocks else
                    (lambda s, a=head + tail: hs2.hs2_full_attn_select(*a, stream=s)))
            call(None)
            torch.cuda.synchronize()
            calls.append(call)
            results.append((idx, idx.clone(), ws, k, v))
    side_by_side(calls[:3], 4000)
    side_by_side(calls[3:], 4000)
    for idx, want, *_ in results:
        assert torch.equal(idx, want)
