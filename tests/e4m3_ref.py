"""The 8-bit cache and its attention written out in 64 bits (torch on the CPU), and the bound of
what the bf16 and fp32 computations may be off from it.

Unit roundoffs: bf16 2^-8, fp32 2^-24 (half a step of the type, relative to the value).
"""
from __future__ import annotations

import math

import torch

BF16, F32 = 2.0 ** -8, 2.0 ** -24
D = 64


def quantise(x):
    """Values q (64 bits, what the e4m3 bytes say) and scale bytes of rows x [..., 64]."""
    x = x.double()
    bad = ~torch.isfinite(x).all(-1)
    amax = torch.where(bad[..., None], 0.0, x).abs().amax(-1)
    frac, power = torch.frexp(amax)                  # amax = frac * 2^power, 0.5 <= frac < 1
    e = torch.where(frac <= 448 / 512, power - 9, power - 8)   # 448 = 448/512 * 2^9
    e = torch.where(amax > 0, e, -100).clamp(min=-100)
    y = torch.ldexp(torch.where(bad[..., None], 0.0, x), -e[..., None])
    step = torch.ldexp(torch.ones_like(y), (torch.frexp(y)[1] - 1).clamp(min=-6) - 3)
    q = torch.round(y / step) * step                 # half to even
    q = torch.where(bad[..., None], math.nan, q)
    return q, torch.where(bad, 255, e + 127).to(torch.uint8)


def values(q, byte):
    """q * 2^(byte - 127), NaN for the byte 255."""
    e = byte.to(torch.int32)
    v = torch.ldexp(q.double(), e[..., None] - 127)
    return torch.where((e == 255)[..., None], math.nan, v)


class Cache:
    """An 8-bit cache on the CPU: pools of 64-bit values, scale bytes, and the untouched rows'
    canary.  `cuda()` gives the tensors the library takes."""

    def __init__(self, B, H, bs, mbps, seed, spare=3):
        g = torch.Generator().manual_seed(seed)
        self.B, self.H, self.bs, self.mbps = B, H, bs, mbps
        self.nb = B * mbps + spare
        self.table = torch.randperm(self.nb, generator=g)[:B * mbps].reshape(B, mbps).to(torch.int32)
        # NaN bytes and the NaN scale wherever nothing was written: a stray read poisons a result
        self.k = torch.full((self.nb, H, bs, D), 0x7f, dtype=torch.uint8)
        self.v = torch.full((self.nb, H, bs, D), 0xff, dtype=torch.uint8)
        self.scale = torch.full((self.nb, H, 2, bs), 255, dtype=torch.uint8)

    def append(self, k_new, v_new, lens):
        """Rows past the table or in an invalid block are dropped."""
        for i, (new, pool) in enumerate(((k_new, self.k), (v_new, self.v))):
            q, byte = quantise(new)
            bits = q.float().to(torch.float8_e4m3fn).view(torch.uint8)
            bits = torch.where((byte == 255)[..., None], 0x7f, bits)
            for b in range(new.shape[0]):
                for t in range(new.shape[1]):
                    p = int(lens[b]) + t
                    if p < 0 or p // self.bs >= self.mbps:
                        continue
                    blk = int(self.table[b, p // self.bs])
                    if 0 <= blk < self.nb:
                        pool[blk, :, p % self.bs] = bits[b, t]
                        self.scale[blk, :, i, p % self.bs] = byte[b, t]

    def history(self, b, n):
        """The values [n, H, 64] of K and V at positions 0 .. n-1; zeros where the block is invalid."""
        ks, vs = torch.zeros(n, self.H, D, dtype=torch.float64), torch.zeros(n, self.H, D, dtype=torch.float64)
        for p in range(n):
            blk = int(self.table[b, p // self.bs])
            if 0 <= blk < self.nb:
                s = p % self.bs
                ks[p] = values(self.k[blk, :, s].view(torch.float8_e4m3fn).double(), self.scale[blk, :, 0, s])
                vs[p] = values(self.v[blk, :, s].view(torch.float8_e4m3fn).double(), self.scale[blk, :, 1, s])
        return ks, vs

    def cuda(self):
        return (self.k.view(torch.float8_e4m3fn).cuda(), self.v.view(torch.float8_e4m3fn).cuda(),
                self.scale.cuda(), self.table.cuda())

    def same(self, k_pool, v_pool, scale):
        return (torch.equal(k_pool.view(torch.uint8).cpu(), self.k) and
                torch.equal(v_pool.view(torch.uint8).cpu(), self.v) and torch.equal(scale.cpu(), self.scale))


def attention(q, u, vb, rel, history, C, scale, dtype, K=None):
    """One stream: out [T, H, 64] in 64 bits and the elementwise bound of a bf16 or fp32 result.

    history: K and V values [>= K, H, 64]; K keys (default C + T).

    The bound, for keys j of query i, unit roundoff r of the type (bf16 inputs are exact):
      score   q + u and q + v are rounded once each and the position term once more (bf16), each to
              half a step: |ds_ij| <= scale * r * (sum|q+u||k_j| + 2 sum|q+v||rel| ) and, for the fp32
              sums of 2 * 64 products in any order, 2^-24 * 130 times the same sums.
              fp32 keeps q + u in fp32: only the second part, with the additions' roundings in it.
              Second-order terms and the change of units by log2(e) are covered by a factor 1.05.
      weights p_ij = exp(s_ij) / sum: a change of every score by at most ds changes p by at most a
              factor exp(2 ds); exp2 and the row sum add less than 2^-20 * (1 + K * 2^-4).
              bf16 rounds each weight once more: r.  Where rows of V differ by octaves the weights are
              held in fp16 relative to the largest contribution p_j 2^e_j: one below 2^-14 of it is off by
              up to 2^-25 of it, 2^-25 * 448 2^e_j <= 2^-24 of max|v_j| (a row's largest value is above
              224 2^e), for at most K keys.
      result  rounded once: r |out|.
    """
    T, H, _ = q.shape
    R = rel.shape[0]
    K = C + T if K is None else K
    k, v = history[0][:K], history[1][:K]
    a, b = q.double() + u.double(), q.double() + vb.double()
    i, j = torch.arange(T)[:, None], torch.arange(K)
    rho = R - T - C + j - i
    rows = torch.where(((rho >= 0) & (rho < R))[..., None, None], rel.double()[rho.clamp(0, R - 1)], 0.0)  # [T, K, H, 64]
    s = scale * (torch.einsum("ihd,jhd->hij", a, k) + torch.einsum("ihd,ijhd->hij", b, rows))
    p = torch.softmax(s, -1)
    out = torch.einsum("hij,jhd->ihd", p, v)
    sk = torch.einsum("ihd,jhd->hij", a.abs(), k.abs())
    sr = torch.einsum("ihd,ijhd->hij", b.abs(), rows.abs())
    r = BF16 if dtype == torch.bfloat16 else F32
    ds = abs(scale) * 1.05 * (130 * F32 * (sk + sr) + (r * (sk + 2 * sr) if dtype == torch.bfloat16 else 0))
    ds = ds.amax(-1)                                           # [H, T]
    weight = torch.expm1(2 * ds) + 2.0 ** -20 * (1 + K / 16) + (r if dtype == torch.bfloat16 else 0)
    mag = torch.einsum("hij,jhd->ihd", p, v.abs())
    top = (p * v.abs().amax(-1).t()[:, None]).amax(-1) * K * 2.0 ** -24 if dtype == torch.bfloat16 else torch.zeros_like(ds)
    return out, (weight.t()[..., None] * mag + top.t()[..., None]) * 1.05 + r * out.abs() + 1e-30
