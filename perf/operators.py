"""The operators of the paged decode path and what a pass through each costs.

Five operators carry one decode step of a layer whose cache is paged: the RMS
norm that adds the residual and packs its output in E4M3, the E4M3 projection
with a scale per block of 128, the append of the new K/V rows to their pages,
the attention of one new token per sequence over those pages (which can add
every position's head-summed probability to a running weight), and the eviction
of the positions that gathered the least weight.

With ``own`` false, ``run`` computes an operator from elementary torch
operations in 32 bits; with ``own`` true it makes the library's calls.
"""

import math
import random

import torch

own = False

E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
BLOCK = 128


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # the norm before a projection at decode: 8 sequences, one token each
        dict(name="norm_decode", op="norm", T=8, hidden=4096, residual=True, out="e4m3"),
        # the same over the prompt that the bridge projects
        dict(name="norm_prompt", op="norm", T=131072, hidden=4096, residual=True, out="e4m3"),
        # K and V of six layers for the new tokens of 8 sequences
        dict(name="gemm_decode", op="gemm", M=8, N=1536, K=4096),
        # the same for a short chunk of an odd length
        dict(name="gemm_chunk", op="gemm", M=1003, N=1536, K=4096),
        # the same for a whole prompt
        dict(name="gemm_prompt", op="gemm", M=131072, N=1536, K=4096),
        # one new bf16 row for each of 64 sequences
        dict(name="append_decode", op="append", B=64, rows=64, max_len=4096, kv_heads=1, D=128,
             page=64, fp8=False),
        # the rows of four prompts of unequal length, packed in E4M3
        dict(name="append_prompt", op="append", B=4, rows=65536, max_len=32768, kv_heads=1, D=128,
             page=64, fp8=True),
        # a single user's short context: latency only
        dict(name="attn_short", op="attn", B=1, max_len=777, ragged=False, H=8, kv_heads=1, D=64,
             page=16, fp8=False, weight=False),
        # 8 users with contexts of unequal length up to 32K, weights kept for the eviction
        dict(name="attn_32k", op="attn", B=8, max_len=32768, ragged=True, H=32, kv_heads=1, D=128,
             page=64, fp8=False, weight=True),
        # 4 users at 256K in E4M3
        dict(name="attn_256k_e4m3", op="attn", B=4, max_len=262144, ragged=False, H=32, kv_heads=1,
             D=128, page=64, fp8=True, weight=False),
        # a budget just passed: a few rows of each cache leave it
        dict(name="evict_few", op="evict", B=8, max_len=1216, ragged=False, kv_heads=1, D=128,
             page=16, fp8=True, topk=1024, window=128),
        # a first eviction from long caches down to the budget
        dict(name="evict_32k", op="evict", B=8, max_len=32768, ragged=True, kv_heads=1, D=128,
             page=64, fp8=False, topk=1024, window=128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "gemm", "append", "attn", "evict"])
    if op == "norm":
        hidden = 16 * _log(rng, 4, 1024)
        return dict(op=op, T=_log(rng, 1, min(131072, 131072 * 4096 // hidden)), hidden=hidden,
                    residual=rng.random() < 0.7, out=rng.choice(["e4m3", "e4m3", "bf16"]))
    if op == "gemm":
        K, N = 16 * _log(rng, 1, 1024), _log(rng, 1, 8192)
        most = 131072 * 1536 * 4096 // (K * N)
        return dict(op=op, M=_log(rng, 1, max(1, min(131072, most, (1 << 29) // K, (1 << 28) // N))),
                    N=N, K=K)
    heads = rng.choice([1, 1, 2, 4, 8])
    D = rng.choice([64, 128])
    page = rng.choice([1, 8, 16, 32, 64, 128, 256])
    fp8 = rng.random() < 0.5
    if op == "append":
        B = _log(rng, 1, 128)
        rows = max(B, _log(rng, 1, 65536 * 128 // (heads * D)))
        return dict(op=op, B=B, rows=rows, max_len=-(-rows // B) * 2 + rng.randrange(64),
                    kv_heads=heads, D=D, page=page, fp8=fp8)
    B = _log(rng, 1, 64)
    max_len = _log(rng, 1, 4 * 262144 * 128 // (2 * B * heads * D))
    if op == "attn":
        max_len = min(max_len, 262144)
        return dict(op=op, B=B, max_len=max_len, ragged=rng.random() < 0.7,
                    H=heads * rng.choice([1, 2, 3, 4, 8, 16, 32]), kv_heads=heads, D=D, page=page,
                    fp8=fp8, weight=rng.random() < 0.5)
    max_len = min(max_len, 32768)
    return dict(op=op, B=B, max_len=max_len, ragged=rng.random() < 0.7, kv_heads=heads, D=D,
                page=page, fp8=fp8, topk=_log(rng, 1, 2048), window=_log(rng, 1, 256))


def _lens(case):
    """Length of every sequence's cache: the first is the longest."""
    n = case["max_len"]
    if case["op"] == "append":
        rows = _rows(case)
        return [max(r, n - (7 * b) % (n // 4 + 1)) for b, r in enumerate(rows)]
    if not case["ragged"]:
        return [n] * case["B"]
    return [n - int(n * ((b * 0.6180339887) % 1.0) * 0.95) for b in range(case["B"])]


def _rows(case):
    """New rows of every sequence: one each, or unequal shares of a prompt."""
    B, rows = case["B"], case["rows"]
    cuts = [rows * b // B for b in range(B + 1)]
    if rows >= 4 * B:
        shift = rows // (4 * B)
        cuts = [c if b in (0, B) else c + (shift if b % 2 else -shift // 2)
                for b, c in enumerate(cuts)]
    return [cuts[b + 1] - cuts[b] for b in range(B)]


def work(case):
    op = case["op"]
    if op == "norm":
        n = case["T"] * case["hidden"]
        blocks = case["T"] * -(-case["hidden"] // BLOCK)
        out = n + 4 * blocks if case["out"] == "e4m3" else 2 * n
        return dict(bytes=2 * n * (3 if case["residual"] else 1) + out + 2 * case["hidden"],
                    flops=8 * n)
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        kb = -(-K // BLOCK)
        return dict(bytes=M * K + N * K + 2 * M * N + 4 * kb * (M + -(-N // BLOCK)),
                    flops=2 * M * N * K)
    heads, D = case["kv_heads"], case["D"]
    row = 2 * heads * (D + 4 if case["fp8"] else 2 * D)      # K and V of one position
    if op == "append":
        n = case["rows"]
        return dict(bytes=n * (4 * heads * D + row + 4), flops=6 * n * heads * D)
    total = sum(_lens(case))
    if op == "attn":
        return dict(bytes=total * (row + (8 if case["weight"] else 0)) + 4 * case["B"] * case["H"] * D,
                    flops=4 * total * case["H"] * D)
    kept = sum(min(n, case["topk"] + min(case["window"], n)) for n in _lens(case))
    return dict(bytes=4 * total + kept * (2 * row + 12), flops=total)


# ------------------------------------------------------------------ inputs --
def _pack(x, dim_block):
    """E4M3 codes and scales of x over blocks of its last dimension."""
    blocks = x.unflatten(-1, (-1, dim_block))
    s = blocks.abs().amax(-1, keepdim=True) / E4M3_MAX
    s = torch.where(s > 0, s, torch.ones_like(s))
    return (blocks / s).to(E4M3).flatten(-2), s.squeeze(-1)


def _paged(case, g):
    """A pool of pages in random order, its page table and the lengths."""
    B, ps, heads, D = case["B"], case["page"], case["kv_heads"], case["D"]
    lens = _lens(case)
    per = [-(-n // ps) for n in lens]
    width = max(1, max(per))
    n_pages = sum(per) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    k = torch.randn(n_pages, ps, heads, D, generator=g, device="cuda")
    v = torch.randn(n_pages, ps, heads, D, generator=g, device="cuda")
    s = dict(table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    if case["fp8"]:
        (s["k"], ks), (s["v"], vs) = _pack(k, D), _pack(v, D)
        s["k_scale"], s["v_scale"] = ks.squeeze(-1).contiguous(), vs.squeeze(-1).contiguous()
    else:
        s["k"], s["v"] = k.bfloat16(), v.bfloat16()
        s["k_scale"] = s["v_scale"] = None
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *shape: torch.randn(*shape, generator=g, device="cuda")   # noqa: E731
    op = case["op"]
    s = dict(case=case)
    if op == "norm":
        T, hidden = case["T"], case["hidden"]
        s["x"] = randn(T, hidden).bfloat16()
        s["r"] = (4 * randn(T, hidden)).bfloat16() if case["residual"] else None
        s["gamma"] = (1 + 0.2 * randn(hidden)).bfloat16()
        s["sum"] = torch.empty_like(s["x"]) if case["residual"] else None
        e = case["out"] == "e4m3"
        s["y"] = None if e else torch.empty_like(s["x"])
        s["codes"] = torch.empty(T, hidden, dtype=E4M3, device="cuda") if e else None
        s["scale"] = torch.empty(T, -(-hidden // BLOCK), device="cuda") if e else None
        return s
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        kb, nb = -(-K // BLOCK), -(-N // BLOCK)
        a = randn(M, kb * BLOCK)
        a[:, K:] = 0
        a *= torch.exp(0.5 * randn(M, 1))              # tokens of unequal size
        a, s["a_scale"] = _pack(a, BLOCK)
        s["a"] = a[:, :K].contiguous()
        b = randn(nb * BLOCK, kb * BLOCK) / math.sqrt(K)
        b[N:] = 0
        b[:, K:] = 0
        b = b.view(nb, BLOCK, kb, BLOCK)
        sb = b.abs().amax((1, 3)) / E4M3_MAX
        s["b_scale"] = sb
        s["b"] = ((b / sb[:, None, :, None]).to(E4M3).view(nb * BLOCK, kb * BLOCK)[:N, :K]
                  .contiguous())
        s["c"] = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        return s
    s.update(_paged(case, g))
    B, heads, D = case["B"], case["kv_heads"], case["D"]
    pool = s["k"].shape[:2]
    if op == "append":
        cuts = [0]
        for n in _rows(case):
            cuts.append(cuts[-1] + n)
        s["row_start"] = (None if case["rows"] == B
                          else torch.tensor(cuts, dtype=torch.int32, device="cuda"))
        # K and V as the projection leaves them: side by side in one row
        s["kv"] = randn(case["rows"], 2, heads * D).bfloat16()
        s["weight"] = torch.rand(*pool, generator=g, device="cuda")
        return s
    if op == "attn":
        s["q"] = (2 * randn(B, case["H"], D)).bfloat16()    # a softmax with heavy positions
        s["weight"] = torch.rand(*pool, generator=g, device="cuda") if case["weight"] else None
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(B, case["H"], device="cuda")
        return s
    # accumulated weights: a few heavy positions, a long tail, and new positions at zero
    w = torch.exp(2.5 * randn(*pool)) * 1e-3
    s["weight"] = torch.where(torch.rand(*pool, generator=g, device="cuda") < 0.05,
                              torch.zeros_like(w), w)
    # the survivors move to pages of their own, behind the source pages
    slots, ps = case["topk"] + case["window"], case["page"]
    most = -(-min(slots, case["max_len"]) // ps)
    n_src = s["k"].shape[0]
    grow = lambda t: None if t is None else torch.cat(                      # noqa: E731
        [t.view(torch.uint8) if t.dtype == E4M3 else t,
         torch.zeros(B * most, *t.shape[1:], dtype=torch.uint8 if t.dtype == E4M3 else t.dtype,
                     device="cuda")]).view(t.dtype)
    for name in ("k", "v", "k_scale", "v_scale", "weight"):
        s[name] = grow(s[name])
    s["dst"] = (n_src + torch.arange(B * most, dtype=torch.int32, device="cuda")).view(B, most)
    s["kept"] = torch.empty(B, slots, dtype=torch.int32, device="cuda")
    s["new_len"] = torch.empty(B, dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------- plain forms --
def _quantise(y, n):
    """E4M3 codes and scales of fp32 values over blocks of n columns (the last may be short)."""
    cols = y.shape[-1]
    pad = -cols % n
    z = torch.nn.functional.pad(y, (0, pad)) if pad else y
    z = z.unflatten(-1, (-1, n))
    amax = z.abs().amax(-1, keepdim=True)
    scale = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
    return (z / scale).to(E4M3).flatten(-2)[..., :cols].contiguous(), scale.squeeze(-1)


def _plain_norm(s):
    h = s["x"].float()
    if s["r"] is not None:
        h = h + s["r"].float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + 1e-6) * s["gamma"].float()
    out = {}
    if s["r"] is not None:
        out["sum"] = h.bfloat16()
    if s["codes"] is None:
        out["y"] = y.bfloat16()
    else:
        out["codes"], out["scale"] = _quantise(y, BLOCK)
    return out


def _plain_gemm(s):
    K, N = s["a"].shape[1], s["b"].shape[0]
    sa = s["a_scale"].repeat_interleave(BLOCK, 1)[:, :K]
    sb = s["b_scale"].repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]
    return {"c": ((s["a"].float() * sa) @ (s["b"].float() * sb).t()).bfloat16()}


def _slots(s, table, pos):
    """Pool rows of positions pos [B, n] (entries of unmapped pages give a negative row)."""
    ps = s["case"]["page"]
    return table.long().gather(1, (pos // ps).clamp_(max=table.shape[1] - 1)) * ps + pos % ps


def _pool(t):
    """Rows of a pool; E4M3 codes as bytes, which can be indexed."""
    return (t.view(torch.uint8) if t.dtype == E4M3 else t).flatten(0, 1)


def _plain_append(s):
    case, lens = s["case"], s["lens"].long()
    n = s["kv"].shape[0]
    r = torch.arange(n, device="cuda")
    if s["row_start"] is None:
        seq, pos = r, lens - 1
    else:
        start = s["row_start"].long()
        seq = torch.searchsorted(start, r, right=True) - 1
        pos = lens[seq] - start[seq + 1] + r
    ps = case["page"]
    slot = s["table"].long()[seq, pos // ps] * ps + pos % ps
    rows = s["kv"].view(n, 2, case["kv_heads"], case["D"])
    out = {"weight": s["weight"]}
    s["weight"].view(-1)[slot] = 0
    for i, name in enumerate(("k", "v")):
        pool = _pool(s[name])
        if case["fp8"]:
            codes, scale = _quantise(rows[:, i].float(), case["D"])
            pool[slot] = codes.view(torch.uint8)
            s[name + "_scale"].flatten(0, 1)[slot] = scale.squeeze(-1)
            out[name + "_scale"] = s[name + "_scale"]
        else:
            pool[slot] = rows[:, i]
        out[name] = s[name]
    return out


def _plain_attn(s):
    case = s["case"]
    B, H, heads, D = case["B"], case["H"], case["kv_heads"], case["D"]
    pos = torch.arange(case["max_len"], device="cuda").expand(B, -1)
    live = pos < s["lens"][:, None]
    slot = _slots(s, s["table"], pos).clamp_(min=0)

    def rows(name):
        x = _pool(s[name])[slot].view(s[name].dtype).float()
        if case["fp8"]:
            x = x * s[name + "_scale"].flatten(0, 1)[slot][..., None]
        return x.permute(0, 2, 1, 3)                                  # [B, heads, len, D]

    q = s["q"].float().view(B, heads, H // heads, D)
    x = (q @ rows("k").transpose(-1, -2)) / math.sqrt(D)
    x = x.masked_fill(~live[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    v = rows("v").masked_fill(~live[:, None, :, None], 0)
    out = {"o": (p @ v).view(B, H, D).bfloat16(), "lse": (m + torch.log(total)).view(B, H)}
    if case["weight"]:
        gain = p.sum((1, 2)).masked_fill(~live, 0)
        s["weight"].view(-1).index_add_(0, slot.reshape(-1), gain.reshape(-1))
        out["weight"] = s["weight"]
    return out


def _plain_evict(s):
    case = s["case"]
    topk, window, slots = case["topk"], case["window"], case["topk"] + case["window"]
    pos = torch.arange(case["max_len"], device="cuda").expand(case["B"], -1)
    lens = s["lens"].long()[:, None]
    slot = _slots(s, s["table"], pos).clamp_(min=0)
    w = s["weight"].view(-1)[slot]
    w = torch.where(pos < lens - window, w, torch.full_like(w, -1.0))   # weights are not negative
    best = torch.sort(w, dim=1, descending=True, stable=True).indices   # ties: the lower first
    rank = torch.empty_like(best).scatter_(1, best, pos)
    keep = ((pos < lens - window) & (rank < topk)) | ((pos >= lens - window) & (pos < lens))
    far = torch.where(keep, pos, torch.full_like(pos, case["max_len"]))
    kept = torch.sort(far, dim=1).values[:, :slots]
    if kept.shape[1] < slots:
        kept = torch.nn.functional.pad(kept, (0, slots - kept.shape[1]), value=case["max_len"])
    valid = kept < case["max_len"]
    # padding repeats the first survivor's move
    r = torch.arange(slots, device="cuda").expand(case["B"], -1)
    src = _slots(s, s["table"], torch.where(valid, kept, kept[:, :1]))
    dst = _slots(s, s["dst"], torch.where(valid, r, torch.zeros_like(r)))
    out = {"kept": torch.where(valid, kept, torch.full_like(kept, -1)).int(),
           "new_len": keep.sum(1).int()}
    for name in ("k", "v", "k_scale", "v_scale", "weight"):
        if s[name] is not None:
            pool = _pool(s[name])
            pool[dst] = pool[src]
            out[name] = s[name]
    return out


# --------------------------------------------------------- the library's calls --
def _own_norm(s):
    import long_context_hs2_b200 as hs2
    hs2.hs2_add_rmsnorm(s["x"], s["r"], s["gamma"], s["x"].shape[0], s["x"].shape[1], 1e-6,
                        s["sum"], s["y"], s["codes"], s["scale"])
    return {k: s[k] for k in ("sum", "y", "codes", "scale") if s[k] is not None}


def _own_gemm(s):
    import long_context_hs2_b200 as hs2
    c = s["case"]
    hs2.hs2_fp8_gemm(s["a"], s["a_scale"], c["M"], s["b"], s["b_scale"], c["N"], c["K"], s["c"])
    return {"c": s["c"]}


def _cache(s):
    """The cache's handle, which a program keeps as long as the cache."""
    import long_context_hs2_b200 as hs2
    if "cache" not in s:
        s["cache"] = hs2.paged_cache(s["k"], s["v"], s["table"], s["lens"], s["k_scale"],
                                     s["v_scale"], s["weight"])
    return hs2, s["cache"], hs2.HS2_KV_FP8_E4M3 if s["case"]["fp8"] else hs2.HS2_KV_BF16


def _own_append(s):
    hs2, cache, dt = _cache(s)
    c = s["case"]
    k, v = s["kv"][:, 0], s["kv"][:, 1]
    hs2.hs2_paged_append(k, v, s["kv"].stride(0), c["rows"], s["row_start"], cache, c["B"],
                         c["kv_heads"], c["D"], dt)
    return {k: s[k] for k in ("k", "v", "k_scale", "v_scale", "weight") if s[k] is not None}


def _own_attn(s):
    hs2, cache, dt = _cache(s)
    c = s["case"]
    if "ws" not in s:
        n = hs2.hs2_paged_attn_workspace(c["B"], c["H"], c["kv_heads"], c["D"])
        s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    hs2.hs2_paged_attn(s["q"], cache, c["B"], c["H"], c["kv_heads"], c["D"],
                       1.0 / math.sqrt(c["D"]), dt, s["o"], s["lse"], c["weight"], s["ws"],
                       s["ws"].numel())
    out = {"o": s["o"], "lse": s["lse"]}
    if c["weight"]:
        out["weight"] = s["weight"]
    return out


def _own_evict(s):
    hs2, cache, dt = _cache(s)
    c = s["case"]
    hs2.hs2_paged_evict(cache, c["B"], c["kv_heads"], c["D"], dt, c["topk"], c["window"],
                        s["dst"], s["kept"], s["new_len"])
    return {k: s[k] for k in ("kept", "new_len", "k", "v", "k_scale", "v_scale", "weight")
            if s[k] is not None}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "gemm": _own_gemm, "append": _own_append, "attn": _own_attn,
                "evict": _own_evict}[op](state)
    return {"norm": _plain_norm, "gemm": _plain_gemm, "append": _plain_append,
            "attn": _plain_attn, "evict": _plain_evict}[op](state)


# ------------------------------------------------------------- in 64 bits --
def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    op = case["op"]
    if op == "norm":
        out = {}
        sums, ys, scales = [], [], []
        for rows in torch.arange(case["T"], device="cuda").split(8192):
            h = s["x"][rows].to(f64)
            if s["r"] is not None:
                h = h + s["r"][rows].to(f64)
            y = h / torch.sqrt(h.square().sum(1, keepdim=True) / case["hidden"] + 1e-6)
            y = y * s["gamma"].to(f64)
            sums.append(h)
            if s["codes"] is not None:
                parts, tops = [], []
                for part in y.split(BLOCK, 1):
                    top = part.abs().max(1, keepdim=True).values / E4M3_MAX
                    top = torch.where(top == 0, torch.ones_like(top), top)
                    parts.append(part / top)
                    tops.append(top)
                y = torch.cat(parts, 1)
                scales.append(torch.cat(tops, 1))
            ys.append(y.float() if s["codes"] is not None else y)
        if s["r"] is not None:
            out["sum"] = torch.cat(sums)
        if s["codes"] is not None:
            out["codes"], out["scale"] = torch.cat(ys).to(f64), torch.cat(scales)
        else:
            out["y"] = torch.cat(ys)
        return out
    if op == "gemm":
        N, K = case["N"], case["K"]
        c = torch.zeros(case["M"], N, dtype=f64, device="cuda")
        n_block = torch.arange(N, device="cuda") // BLOCK
        for kb, k0 in enumerate(range(0, K, BLOCK)):
            a = s["a"][:, k0:k0 + BLOCK].to(f64)
            b = s["b"][:, k0:k0 + BLOCK].to(f64)
            c += (a @ b.t()) * s["a_scale"][:, kb, None].to(f64) * s["b_scale"][n_block, kb].to(f64)
        return {"c": c}
    ps, heads, D = case["page"], case["kv_heads"], case["D"]
    lens = _lens(case)

    def where(b, positions, table="table"):
        at = torch.as_tensor(positions, device="cuda")
        return s[table][b].long()[at // ps] * ps + at % ps

    if op == "append":
        pools = {n: s[n].flatten(0, 1).to(f64) for n in ("k", "v")}
        scales = {n: None if s[n + "_scale"] is None else s[n + "_scale"].flatten(0, 1).to(f64)
                  for n in ("k", "v")}
        weight = s["weight"].flatten().to(f64)
        at = 0
        for b, n in enumerate(_rows(case)):
            if not n:
                continue
            slot = where(b, list(range(lens[b] - n, lens[b])))
            weight[slot] = 0
            for i, name in enumerate(("k", "v")):
                x = s["kv"][at:at + n, i].to(f64).view(n, heads, D)
                if case["fp8"]:
                    top = x.abs().max(2).values / E4M3_MAX
                    top = torch.where(top == 0, torch.ones_like(top), top)
                    scales[name][slot] = top
                    x = x / top[..., None]
                pools[name][slot] = x
            at += n
        out = {"weight": weight, "k": pools["k"], "v": pools["v"]}
        if case["fp8"]:
            out["k_scale"], out["v_scale"] = scales["k"], scales["v"]
        return out
    if op == "attn":
        group = case["H"] // heads
        o = torch.zeros(case["B"], case["H"], D, dtype=f64, device="cuda")
        lse = torch.full((case["B"], case["H"]), -math.inf, dtype=f64, device="cuda")
        weight = None if s["weight"] is None else s["weight"].flatten().to(f64)
        for b, n in enumerate(lens):
            if not n:
                continue
            slot = where(b, torch.arange(n))
            for h in range(heads):
                kv = []
                for name in ("k", "v"):
                    x = s[name].flatten(0, 1)[:, h].to(torch.float32)[slot].to(f64)
                    if case["fp8"]:
                        x = x * s[name + "_scale"].flatten(0, 1)[slot, h, None].to(f64)
                    kv.append(x)
                mine = slice(h * group, (h + 1) * group)
                logits = s["q"][b, mine].to(f64) @ kv[0].t() / D ** 0.5
                lse[b, mine] = torch.logsumexp(logits, 1)
                p = torch.exp(logits - lse[b, mine, None])
                o[b, mine] = p @ kv[1]
                if weight is not None:
                    weight[slot] += p.sum(0)
        out = {"o": o, "lse": lse}
        if weight is not None:
            out["weight"] = weight
        return out
    topk, window = case["topk"], case["window"]
    names = [n for n in ("k", "v", "k_scale", "v_scale", "weight") if s[n] is not None]
    out = {n: s[n].flatten(0, 1).to(f64) for n in names}
    weight = s["weight"].flatten().cpu()
    kept = torch.full((case["B"], topk + window), -1, dtype=torch.int32, device="cuda")
    new_len = []
    for b, n in enumerate(lens):
        first = max(0, n - window)
        w = weight[where(b, torch.arange(n)).cpu()].tolist()
        order = sorted(range(first), key=lambda j: (-w[j], j))[:topk]
        stay = sorted(order) + list(range(first, n))
        kept[b, :len(stay)] = torch.tensor(stay, dtype=torch.int32, device="cuda")
        new_len.append(len(stay))
        src, dst = where(b, stay), where(b, list(range(len(stay))), "dst")
        for name in names:
            out[name][dst] = out[name][src]
    out["kept"] = kept
    out["new_len"] = torch.tensor(new_len, dtype=torch.int32, device="cuda")
    return out
