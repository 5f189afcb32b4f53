"""Host threads that make the same call with different sizes, each on its own stream and
buffers: a kernel's settings belong to the function, and one thread's must not fail the
other's launch."""

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
