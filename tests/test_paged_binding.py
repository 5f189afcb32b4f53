"""What the paged decode path's binding hands to the library, and what it refuses, on the CPU:
tensors that claim to be on the current device, and a library that records its calls."""

import pytest
import torch

import long_context_hs2_b200 as hs2

BF16, F32, I32, E4M3 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn


class OnDevice(torch.Tensor):
    def get_device(self):
        return 0


def t(shape, dtype):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnDevice)


@pytest.fixture
def calls(monkeypatch):
    made = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: made.append((name, a)) or 0

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(hs2, "load_library", lambda *a: Library())
    return made


def cache(fp8=False, **kw):
    pool = (4, 16, 2)
    a = dict(k=t(pool + (64,), E4M3 if fp8 else BF16), v=t(pool + (64,), E4M3 if fp8 else BF16),
             page_table=t((3, 4), I32), seq_len=t((3,), I32), weight=t(pool[:2], F32))
    if fp8:
        a.update(k_scale=t(pool, F32), v_scale=t(pool, F32))
    a.update(kw)
    return hs2.paged_cache(**a)


def norm(**kw):
    a = dict(X=t((5, 256), BF16), R=t((5, 256), BF16), gamma=t((256,), BF16), sum=t((5, 256), BF16),
             Y=t((5, 256), BF16), Yq=t((5, 256), E4M3), Yq_scale=t((5, 2), F32))
    a.update(kw)
    hs2.hs2_add_rmsnorm(T=5, hidden=256, eps=1e-6, stream=0, **a)


def gemm(**kw):
    a = dict(A=t((5, 256), E4M3), A_scale=t((5, 2), F32), B=t((130, 256), E4M3),
             B_scale=t((2, 2), F32), C=t((5, 130), BF16))
    a.update(kw)
    hs2.hs2_fp8_gemm(M=5, N=130, K=256, stream=0, **a)


def append(**kw):
    a = dict(K=t((7, 128), BF16), V=t((7, 128), BF16), ld=128, n_rows=7, row_start=t((4,), I32),
             cache=cache())
    a.update(kw)
    hs2.hs2_paged_append(B=3, kv_heads=2, D=64, dt=0, stream=0, **a)


def attn(**kw):
    a = dict(Q=t((3, 8, 64), BF16), O=t((3, 8, 64), BF16), lse=t((3, 8), F32),
             workspace=t((1000,), torch.uint8), cache=cache())
    a.update(kw)
    hs2.hs2_paged_attn(B=3, H=8, kv_heads=2, D=64, scale=0.1, dt=0, accumulate=False,
                       workspace_bytes=1000, stream=0, **a)


def evict(**kw):
    a = dict(dst_table=t((3, 2), I32), kept=t((3, 20), I32), new_len=t((3,), I32), cache=cache())
    a.update(kw)
    hs2.hs2_paged_evict(B=3, kv_heads=2, D=64, dt=0, topk=16, window=4, stream=0, **a)


def test_calls_as_documented_pass(calls):
    for f in (norm, gemm, append, attn, evict):
        f()
    norm(Yq=t((5, 256), torch.uint8))
    cache(fp8=True)
    cache(fp8=True, k=t((4, 16, 2, 64), torch.uint8), v=t((4, 16, 2, 64), torch.uint8))
    attn(lse=None, workspace=t((1000,), torch.int8))
    assert [n for n, _ in calls] == ["hs2_add_rmsnorm", "hs2_fp8_gemm", "hs2_paged_append",
                                     "hs2_paged_attn", "hs2_paged_evict", "hs2_add_rmsnorm",
                                     "hs2_paged_attn"]


WRONG = {BF16: (torch.float16, torch.int16), F32: (I32, torch.uint32), I32: (F32, torch.uint32),
         E4M3: (torch.int8, torch.float8_e5m2)}
ARGS = [(norm, "X", (5, 256), BF16), (norm, "R", (5, 256), BF16), (norm, "gamma", (256,), BF16),
        (norm, "sum", (5, 256), BF16), (norm, "Y", (5, 256), BF16), (norm, "Yq", (5, 256), E4M3),
        (norm, "Yq_scale", (5, 2), F32), (gemm, "A", (5, 256), E4M3),
        (gemm, "A_scale", (5, 2), F32), (gemm, "B", (130, 256), E4M3),
        (gemm, "B_scale", (2, 2), F32), (gemm, "C", (5, 130), BF16), (append, "K", (7, 128), BF16),
        (append, "V", (7, 128), BF16), (append, "row_start", (4,), I32),
        (attn, "Q", (3, 8, 64), BF16), (attn, "O", (3, 8, 64), BF16), (attn, "lse", (3, 8), F32),
        (evict, "dst_table", (3, 2), I32), (evict, "kept", (3, 20), I32),
        (evict, "new_len", (3,), I32)]


@pytest.mark.parametrize("call,name,shape,right", ARGS)
def test_another_type_of_the_same_size_is_refused(calls, call, name, shape, right):
    for wrong in WRONG[right]:
        with pytest.raises(hs2.Hs2Error):
            call(**{name: t(shape, wrong)})
    assert not calls


@pytest.mark.parametrize("fp8", [False, True])
def test_caches_of_another_type_are_refused(calls, fp8):
    pool = (4, 16, 2)
    wrong = [dict(page_table=t((3, 4), F32)), dict(seq_len=t((3,), F32)),
             dict(weight=t(pool[:2], I32))]
    if fp8:
        wrong += [dict(k_scale=t(pool, I32)), dict(v_scale=t(pool, I32))]
    for w in WRONG[E4M3 if fp8 else BF16]:
        both = t(pool + (64,), w)
        wrong += [dict(k=both, v=both)]
    for kw in wrong:
        with pytest.raises(hs2.Hs2Error):
            cache(fp8=fp8, **kw)


def test_workspaces_are_bytes(calls):
    for dtype in (F32, torch.float16):
        with pytest.raises(hs2.Hs2Error):
            attn(workspace=t((1000,), dtype))


def test_append_takes_rows_without_gaps(calls):
    kv = t((7, 2, 2, 64), BF16)                    # K and V side by side, heads apart
    append(K=kv[:, 0], V=kv[:, 1], ld=256)
    append(K=kv.flatten(1)[:, :128], V=kv.flatten(1)[:, 128:], ld=256)
    append(K=t((7, 1, 2, 64), BF16), V=t((9, 2, 64), BF16))
    append(K=t((7, 2, 64), BF16)[:1], V=t((1, 128), BF16), n_rows=1, ld=4096)   # one row: no distance
    assert len(calls) == 4
    for bad, ld in ((t((7, 2, 2, 64), BF16)[:, :, 0], 256),       # heads 2 D apart
                    (t((7, 64, 2), BF16).transpose(1, 2), 128),   # [heads][D] not in order
                    (t((7, 2, 128), BF16)[:, :, :64], 256),       # a gap behind every head
                    (t((7, 128, 2), BF16)[:, :, 0], 256),         # every other element
                    (t((14, 64), BF16), 64),                      # half rows
                    (t((14, 192), BF16)[:, :64], 192),            # half rows of a wider tensor
                    (t((896,), BF16), 1)):
        for kw in (dict(K=bad), dict(V=bad)):
            with pytest.raises(hs2.Hs2Error):
                append(ld=ld, **dict(dict(K=t((7, ld), BF16), V=t((7, ld), BF16)), **kw))
    assert len(calls) == 4


def test_evict_takes_a_raw_destination_table(calls):
    evict()
    evict(dst_table=4096, dst_max_pages=2)
    evict(dst_table=None)
    assert [a[7:9] for _, a in calls][1:] == [(4096, 2), (None, 0)] and calls[0][1][8] == 2
    for kw in (dict(dst_table=4096), dict(dst_table=t((6,), I32)),
               dict(dst_table=t((3, 2), I32), dst_max_pages=3), dict(dst_table=t((2, 2), I32))):
        with pytest.raises(hs2.Hs2Error):
            evict(**kw)
    assert len(calls) == 3


def test_the_version_counts_the_paged_entry_points():
    from long_context_hs2_b200 import build
    build.build()
    assert hs2.load_library().hs2_version() >= 102      # 101 had none of them
