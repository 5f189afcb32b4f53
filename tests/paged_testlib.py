"""Helpers of the paged decode path's tests: caches with shuffled pages whose stale rows
hold NaN and infinities, and the operators' definitions in 64 bits (plain torch, CPU)."""

import math

import torch

import long_context_hs2_b200 as hs2

E4M3 = torch.float8_e4m3fn
F64 = torch.float64


def quantise(x, n=None):
    """E4M3 codes (float32 cast, round to nearest even) and float64 scales over blocks of n
    columns of the last dimension (all of it by default; the last block may be short)."""
    x = x.to(F64)
    n = n or x.shape[-1]
    parts, scales = [], []
    for part in x.split(n, -1):
        s = part.abs().amax(-1, keepdim=True) / 448.0
        s = torch.where(s > 0, s, torch.ones_like(s)).float().to(F64)
        parts.append((part / s).float().to(E4M3))
        scales.append(s)
    codes = torch.cat([p.view(torch.uint8) for p in parts], -1).view(E4M3)
    return codes, torch.cat(scales, -1)


def assert_codes(codes, x, s, eps):
    """codes are a rounding of x / s, where x is known to +-eps: the code of some value within."""
    x, s = x.to(F64), s.to(F64)
    lo = ((x - eps) / s).clamp(-448, 448).float().to(E4M3).to(F64)
    hi = ((x + eps) / s).clamp(-448, 448).float().to(E4M3).to(F64)
    c = codes.to(F64)
    assert ((c >= lo) & (c <= hi)).all()


class Cache:
    """A paged cache on the GPU and what its live rows hold (float64, CPU)."""

    def __init__(self, lens, page, heads, D, fp8, seed=0, spare=2, weight=False, stale=float("nan"),
                 max_pages=None, scale_range=(1e-3, 3.0)):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.page, self.heads, self.D, self.fp8 = list(lens), page, heads, D, fp8
        self.B = len(lens)
        self.dt = hs2.HS2_KV_FP8_E4M3 if fp8 else hs2.HS2_KV_BF16
        per = [-(-n // page) for n in lens]
        self.max_pages = max_pages or max(1, max(per))
        self.n_pages = sum(per) + spare
        order = torch.randperm(self.n_pages, generator=g).to(torch.int32)
        table = torch.full((self.B, self.max_pages), 2 ** 30, dtype=torch.int32)   # never read
        at = 0
        for b, n in enumerate(per):
            table[b, :n] = order[at:at + n]
            at += n
        self.free = order[at:]
        self.table = table
        slots = self.n_pages * page
        shape = (slots, heads, D)
        self.live = torch.zeros(slots, dtype=torch.bool)
        for b, n in enumerate(lens):
            self.live[self.slots(b, range(n))] = True
        dead = ~self.live
        if fp8:
            self.kc, self.vc = (torch.randn(shape, generator=g).mul(100).clamp(-448, 448).to(E4M3)
                                for _ in range(2))
            lo, hi = (math.log(v) for v in scale_range)
            self.ks, self.vs = (torch.exp(torch.rand(slots, heads, generator=g) * (hi - lo) + lo)
                                for _ in range(2))
            self.ks = self.ks / 100          # logits of ordinary size
            self.k64 = self.kc.to(F64) * self.ks.to(F64)[..., None]
            self.v64 = self.vc.to(F64) * self.vs.to(F64)[..., None]
            if not math.isfinite(stale):
                for c, s in ((self.kc, self.ks), (self.vc, self.vs)):
                    c.view(torch.uint8)[dead] = 0x7f
                    s[dead] = stale
        else:
            self.kc, self.vc = (torch.randn(shape, generator=g).bfloat16() for _ in range(2))
            self.ks = self.vs = None
            self.k64, self.v64 = self.kc.to(F64), self.vc.to(F64)
            self.kc[dead] = stale
            self.vc[dead] = stale
        self.w = torch.rand(slots, generator=g) if weight else None
        self.upload()

    def slots(self, b, positions, table=None):
        t = self.table if table is None else table
        p = torch.as_tensor(list(positions), dtype=torch.long)
        return t[b].long()[p // self.page] * self.page + p % self.page

    def upload(self):
        pool = (self.n_pages, self.page, self.heads)
        up = lambda t, *s: None if t is None else t.reshape(s).contiguous().cuda()   # noqa: E731
        self.k, self.v = (up(c, *pool, self.D) for c in (self.kc, self.vc))
        self.k_scale, self.v_scale = (up(s, *pool) for s in (self.ks, self.vs))
        self.weight = up(self.w, *pool[:2])
        self.table_dev = self.table.cuda()
        self.len_dev = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.struct = hs2.paged_cache(self.k, self.v, self.table_dev, self.len_dev, self.k_scale,
                                      self.v_scale, self.weight)

    def pools(self):
        """The GPU's pools now, rows flattened, on the CPU."""
        out = {"k": self.k, "v": self.v, "k_scale": self.k_scale, "v_scale": self.v_scale,
               "weight": self.weight}
        return {n: t.cpu().flatten(0, 1) for n, t in out.items() if t is not None}


def attention(cache, q, scale):
    """(o, lse, weight gain per slot, sum of |terms| of o, floor) in 64 bits; q [B, H, D] on the
    CPU.  floor (E4M3): an f16 probability below 2^-14 is off by up to 2^-25 of the reference
    (the largest logit's probability times the largest v_scale), so o by up to 2^-25 sum |code|
    max(v_scale) / sum exp(s - max s)."""
    B, H, D = q.shape
    G = H // cache.heads
    o, lse = torch.zeros(B, H, D, dtype=F64), torch.full((B, H), -math.inf, dtype=F64)
    mass = torch.zeros(B, H, D, dtype=F64)
    floor = torch.zeros(B, H, D, dtype=F64)
    gain = torch.zeros(cache.n_pages * cache.page, dtype=F64)
    for b, n in enumerate(cache.lens):
        if n == 0:
            continue
        rows = cache.slots(b, range(n))
        for h in range(H):
            s = cache.k64[rows, h // G] @ q[b, h].to(F64) * scale
            lse[b, h] = torch.logsumexp(s, 0)
            p = torch.exp(s - lse[b, h])
            o[b, h] = p @ cache.v64[rows, h // G]
            mass[b, h] = p @ cache.v64[rows, h // G].abs()
            gain.index_add_(0, rows, p)
            if cache.fp8:
                floor[b, h] = (2.0 ** -25 * cache.vc[rows, h // G].to(F64).abs().sum(0)
                               * float(cache.vs[rows, h // G].max()) / torch.exp(lse[b, h] - s.max()))
    return o, lse, gain, mass, floor


def run_attention(cache, q, scale, accumulate=False, workspace=None):
    B, H, D = q.shape
    n = hs2.hs2_paged_attn_workspace(B, H, cache.heads, D)
    assert n > 0
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if workspace is None else workspace
    ws.fill_(0xff)                                 # NaN: nothing may be read before it is written
    o = torch.full((B, H, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, H), float("nan"), device="cuda")
    hs2.hs2_paged_attn(q.cuda(), cache.struct, B, H, cache.heads, D, scale, cache.dt, o, lse,
                       accumulate, ws, n)
    st = hs2.hs2_last_device_status()
    assert st == 0, hs2.hs2_status_string(st)
    return o.cpu(), lse.cpu()


def survivors(weight, n, topk, window):
    """Positions that stay, of n with these weights (a list of floats), by the definition."""
    first = max(0, n - window)
    key = lambda j: (-weight[j] if weight[j] == weight[j] else math.inf, j)   # noqa: E731
    return sorted(sorted(range(first), key=key)[:topk]) + list(range(first, n))
