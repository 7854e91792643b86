"""Plain 64-bit restatements of the rotation and of the 4-bit pages, and a filled 4-bit cache,
for the tests of the rotary append and of the 4-bit operators."""
import math
import random

import torch


def turned(x, row, rot, interleaved):
    """x [T, H, D] (float64) with its first `rot` elements turned; row [T, rot]: cosines, sines."""
    c, s = row.double()[:, None].chunk(2, -1)
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, b * c + a * s
    return y


def quantised(x, group, dtype):
    """x [..., D] (float64) -> (codes int64 [..., D], affine [..., D / group, 2] of dtype)."""
    g = x.unflatten(-1, (-1, group))
    low, high = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    scale, bias = ((high - low) / 15).float().to(dtype), low.float().to(dtype)
    bad = ~torch.isfinite(g.float()).all(-1, keepdim=True) | ~torch.isfinite(bias) | ~torch.isfinite(scale)
    s, b = scale.double(), bias.double()
    s = torch.where(s == 0, 1.0, s)
    d = g - b
    q = d / s
    codes = q.round()
    # where the quotient comes out as k + 1/2, what 64 bits dropped from g - b decides (an element of 2^-60
    # beside a bias of -1, say)
    k, w = q.floor(), d - g
    left = (d - (k + 0.5) * s) + ((g - (d - w)) - (b + w))
    codes = torch.where((q - k == 0.5) & (left != 0), torch.where(left > 0, k + 1, k), codes).clamp(0, 15)
    s = scale.double()
    codes = torch.where(bad | (s == 0), 0.0, codes).long()
    nan = torch.full_like(scale, float("nan"))
    return codes.flatten(-2), torch.cat([torch.where(bad, nan, scale), torch.where(bad, nan, bias)], -1)


def pack(codes):
    """Codes [..., D] -> int32 words [..., D / 8]: quad q of the row (4 codes, lowest nibble first) is
    elements 32 j + 4 g .. + 3 with g = q // (D / 32), j = q % (D / 32)."""
    d = codes.shape[-1]
    words = torch.zeros(*codes.shape[:-1], d // 8, dtype=torch.int64, device=codes.device)
    for e in range(d):
        q = (e % 32) // 4 * (d // 32) + e // 32
        words[..., q // 2] |= codes[..., e].long() << (16 * (q % 2) + 4 * (e % 4))
    return torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)


def unpack(words):
    d = 8 * words.shape[-1]
    w = words.long() & 0xffffffff
    out = torch.empty(*words.shape[:-1], d, dtype=torch.int64, device=words.device)
    for e in range(d):
        q = (e % 32) // 4 * (d // 32) + e // 32
        out[..., e] = (w[..., q // 2] >> (16 * (q % 2) + 4 * (e % 4))) & 15
    return out


def values(words, affine):
    """float64 values, and |scale * code| + |bias|."""
    c = unpack(words).double()
    group = c.shape[-1] // affine.shape[-2]
    a = affine.double()
    sc, b = c.unflatten(-1, (-1, group)) * a[..., 0:1], a[..., 1:2]
    return (sc + b).flatten(-2), (sc.abs() + b.abs()).flatten(-2)


def visible(n, length, window=0, parents=None):
    """[n, length] bool: which keys each of the last n tokens sees."""
    see = torch.zeros(n, length, dtype=torch.bool)
    prefix = length - n
    for i in range(n):
        if parents is None:
            lo = max(0, prefix + i - window + 1) if window else 0
            see[i, lo:max(lo, prefix + i + 1)] = True
        else:
            see[i, :max(prefix, 0)] = True
            a = i
            while True:
                if prefix + a >= 0:
                    see[i, prefix + a] = True
                p = parents[a]
                if not 0 <= p < a:
                    break
                a = p
    return see


def reference(q, k, v, mags, see, scale, half):
    """(out, tolerance) in float64 of one request: q [n, H, D]; k, v, mags [length, Hk, D].

    half = eps / 2 of the 16-bit type.  What the kernels round:
      half |ref|           the output
      2 half W             a weight times a scale, or a weight and a value, each to 16 bits (W: what
                           the weights make of |scale code| + |bias|)
      d (W + |ref|)        the keys' rounding to 16 bits: a logit is off by scale sum q_i k_i e_i with
                           |e_i| <= half, as good as independent: standard deviation
                           half / sqrt(3) scale sqrt(sum (q_i k_i)^2), taken six times
      2^-12 W              f32 work: a logit is off by at most D 2^-24 sum |q k| scale, its weight as much
      2^-25 max |v| length (f16) weights below the normal range, relative to a sum >= 1
    """
    n, h, d = q.shape
    g = h // k.shape[1]
    out = torch.zeros(n, h, d, dtype=torch.float64, device=q.device)
    tol = torch.full_like(out, 1e-30)
    see = see.to(q.device)
    live, used = see.any(1), see.any(0)
    if not bool(live.any()):
        return out, tol
    for i in range(h):
        kk = torch.where(used[:, None], k[:, i // g], 0.0)
        vv, mm = (torch.where(used[:, None], x[:, i // g], 0.0) for x in (v, mags))
        qi = q[:, i].double()
        s = torch.where(see, qi @ kk.T * scale, -math.inf)
        w = torch.softmax(s[live], -1)
        off = half * 3 ** -0.5 * abs(scale) * torch.where(see, (qi ** 2) @ (kk ** 2).T, 0.0).amax(1, keepdim=True).sqrt()
        big = w @ mm
        out[live, i] = w @ vv
        o = out[live, i].abs()
        tol[live, i] += half * o + (2 * half + 2.0 ** -12) * big + 6 * off[live] * (big + o)
        if half < 2.0 ** -10:
            tol[live, i] += 2.0 ** -25 * vv.abs().max() * see.shape[1]
    return out, tol


def check(got, ref, tol):
    assert bool(torch.isfinite(got.double()).all()), "non-finite output"
    worst = ((got.double() - ref).abs() - tol).max().item()
    assert worst <= 0, "off by %.3g over the tolerance (max err %.3g)" % (worst, (got.double() - ref).abs().max().item())


def offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class QuantPaged:
    """A 4-bit paged cache filled for requests of `lens` keys, `new` of them new.  What no request
    holds is NaN scales and biases over random codes."""

    def __init__(self, ta, lens, new, h, hk, d, ps, group, dtype, seed=0, pad=0, spare=3, nhd=False, tree=False):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rnd = random.Random(seed)
        self.lens, self.new, self.h, self.hk, self.d, self.ps, self.dtype = lens, new, h, hk, d, ps, dtype
        self.scale, self.half = d ** -0.5, torch.finfo(dtype).eps / 2
        need = [-(-n // ps) for n in lens]
        n_pages = sum(need) + spare
        lead = (n_pages, ps, hk) if nhd else (n_pages, hk, ps)
        parts = []
        for _ in "kv":
            c = torch.randint(-2 ** 31, 2 ** 31, (*lead, d // 8), generator=g, device="cuda").to(torch.int32)
            a = torch.full((*lead, d // group, 2), float("nan"), dtype=dtype, device="cuda")
            parts += [c.transpose(1, 2), a.transpose(1, 2)] if nhd else [c, a]
        self.cache = ta.PagedQuantCache(*parts)
        order = list(range(n_pages))
        rnd.shuffle(order)
        self.table = torch.full((len(lens), max(1, max(need)) + 1), -7, dtype=torch.int32)
        self.keys, self.vals, self.mags = [], [], []
        at = 0
        for b, n in enumerate(lens):
            rows = []
            for _ in "kv":
                x = torch.randn(n, hk, d, generator=g, device="cuda") + 0.3 * torch.randn(d, generator=g, device="cuda")
                codes, affine = quantised(x.to(dtype).double(), group, dtype)
                rows += [pack(codes), affine]
            self.keys.append(values(*rows[:2])[0])
            v, m = values(*rows[2:])
            self.vals.append(v)
            self.mags.append(m)
            for j in range(need[b]):
                page = order[at]
                at += 1
                self.table[b, j] = page
                m = min(ps, n - j * ps)
                for part, row in zip(self.cache, rows):
                    part[page, :, :m] = row[j * ps:j * ps + m].transpose(0, 1)
        self.table = self.table.cuda()
        self.cu = offsets(new)
        self.q = (torch.randn(self.cu[-1] + pad, h, d, generator=g, device="cuda") * 2).to(dtype)
        self.parents = [[rnd.randrange(-1 if rnd.random() < 0.1 else 0, i) if i else -1 for i in range(n)]
                        for n in new] if tree else None

    def flat_parents(self):
        if self.parents is None:
            return None
        p = [x for r in self.parents for x in r]
        return i32(p + [-1] * (self.q.shape[0] - len(p)))

    def run(self, ta, **kw):
        a = dict(scale=self.scale, max_q_len=max(1, max(self.new)), parents=self.flat_parents())
        a.update(kw)
        if a.get("out") is None:                # a row that is not written shows
            a["out"] = torch.full_like(self.q, 77.0)
        return ta.paged_quant_attention(self.q, self.cache, self.table, i32(self.cu), i32(self.lens), **a)

    def check(self, got, window=0, only=None):
        """All requests' rows, or those of the requests `only`."""
        for b, (n, m) in enumerate(zip(self.lens, self.new)):
            if only is None or b in only:
                see = visible(m, n, window, self.parents[b] if self.parents else None)
                s = slice(self.cu[b], self.cu[b + 1])
                ref, tol = reference(self.q[s], self.keys[b], self.vals[b], self.mags[b], see, self.scale, self.half)
                if m:
                    check(got[s], ref, tol)
