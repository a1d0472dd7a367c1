"""Plain 64-bit definitions of the attention operators, and the error bounds of their
BF16 kernels. Works on the device of its inputs; shares no code with the library."""
import torch

U = 2.0 ** -8  # unit roundoff of BF16 (8 significant bits)


class Batch:
    """A token batch: new[s] tokens and kv[s] cached keys (those included) per sequence,
    on a cache of shuffled pages, with `pad` more rows than tokens."""

    def __init__(self, new, kv, page=16, kv_heads=2, dim=128, pad=0, free=2, seed=0, fill=None, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.new, self.kv, self.page, self.T = list(new), list(kv), page, max(1, sum(new) + pad)
        self.device = torch.device(device)
        starts = [0]
        for n in new:
            starts.append(starts[-1] + n)
        self.starts_list = starts
        self.starts = torch.tensor(starts, dtype=torch.int32, device=device)
        self.lens = torch.tensor(self.kv, dtype=torch.int32, device=device)
        need = [-(-n // page) for n in self.kv]
        width = max(1, max(need))
        self.pages = sum(need) + free
        order = torch.randperm(self.pages, generator=g, device=device).to(torch.int32)
        self.table = torch.full((len(need), width), -1, dtype=torch.int32, device=device)
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = order[at:at + n]
            at += n
        shape = (self.pages, kv_heads, page, dim)
        self.k_cache = torch.randn(shape, generator=g, device=device).bfloat16()
        self.v_cache = torch.randn(shape, generator=g, device=device).bfloat16()
        self.gen = g
        if fill is not None:  # what lies past each length, and the free pages
            keep = torch.zeros(self.pages, page, dtype=torch.bool, device=device)
            for s, n in enumerate(self.kv):
                pos = torch.arange(n, device=device)
                keep[self.table[s].long()[pos // page], pos % page] = True
            drop = ~keep[:, None, :, None].expand(shape)
            self.k_cache[drop] = fill
            self.v_cache[drop] = fill

    def randn(self, *shape, std=1.0):
        return (std * torch.randn(shape, generator=self.gen, device=self.device)).bfloat16()

    def rows(self, cache, s):
        """Cached rows [kv heads, kv_len, dim] of sequence s."""
        n = self.kv[s]
        pos = torch.arange(n, device=cache.device)
        return cache[self.table[s].long()[pos // self.page], :, pos % self.page].transpose(0, 1)


def attend(q, k, v, last, scale):
    """q [n, heads, dim] over k, v [kv heads, keys, dim]: query i sees keys 0..last[i].
    Returns (out, bound of |error|, lse, bound of its |error|).

    Bounds: the weights and the output are rounded to BF16 once each, U relative, so
    2 U sum(p |v|) / sum(p) to first order; the scores' fp32 sums (8 steps of 16 products,
    2^-23 each, of sum |q k|) shift a weight by 2^-20 B relative, B = scale max_j sum |q k|,
    and the maximum and exp2 by a few 2^-22 of B and of 1."""
    n, heads, dim = q.shape
    group = heads // k.shape[0]
    q, k, v = q.double(), k.double().repeat_interleave(group, 0), v.double().repeat_interleave(group, 0)
    s = torch.einsum("nhd,hjd->hnj", q, k) * scale
    seen = torch.arange(k.shape[1], device=q.device)[None, :] <= last[:, None]
    s = s.masked_fill(~seen, -torch.inf)
    if k.shape[1] == 0:
        z = torch.zeros(n, heads, dim, dtype=torch.float64, device=q.device)
        return z, z, torch.full((n, heads), -torch.inf, device=q.device, dtype=torch.float64), z[..., 0]
    top = s.amax(-1, keepdim=True).clamp_min(-1e300)
    p = torch.exp(s - top)
    total = p.sum(-1)
    w = p / total.clamp_min(1e-300)[..., None]
    out = torch.einsum("hnj,hjd->nhd", w, v)
    mag = torch.einsum("hnj,hjd->nhd", w, v.abs())
    b = scale * torch.where(seen, torch.einsum("nhd,hjd->hnj", q.abs(), k.abs()), 0.0).amax(-1)
    shift = 2.0 ** -19 * (1 + b)
    lse = torch.where(total > 0, top[..., 0] + torch.log(total.clamp_min(1e-300)), -torch.inf)
    return out, mag * (2.1 * U + 2 * shift.T[..., None]) + 1e-30, lse.T, shift.T


def rotate(x, cos, sin, interleaved):
    """x [T, heads, dim], cos and sin [T, rot / 2]: (rotated, bound of |error|): one BF16
    rounding, and two products and a sum in fp32."""
    rot = 2 * cos.shape[-1]
    x, y = x.double(), x.double().clone()
    e = torch.zeros_like(x)
    c, s = cos.double()[:, None], sin.double()[:, None]
    ia = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    ib = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    e[..., ia] = e[..., ib] = 2.0 ** -22 * (a.abs() + b.abs())
    return y, e * 1.01 + 1.01 * U * y.abs()


def within(got, ref, bound, what):
    got = got.double()
    bad = ~((got - ref).abs() <= bound) & ~(torch.isinf(ref) & (got == ref))
    assert not bad.any(), "%s: %d of %d out of bound; first at %s: %r, expected %r +- %r" % (
        what, int(bad.sum()), bad.numel(), bad.nonzero()[0].tolist(), got[bad][0].item(), ref[bad][0].item(),
        bound.expand_as(ref)[bad][0].item())
