"""Attention over 4-bit pages at the ends of its range (scales, queries and weights that differ by many orders of
magnitude, keys and pages that are not there): every kernel family against 64 bits."""
import math

import pytest
import torch

from quant_pages import QuantPaged, check, i32, pack, quantised, turned, values, visible

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
FAMILIES = [1, 0, 2, 3]


@pytest.fixture(scope="module")
def ta():
    import tree_masked_speculative_gb300 as m
    return m


def shared_pages(ta, logits, v_scale, v_codes, v_bias, ps, group, dtype, batch, new, h):
    """A cache that `batch` requests share, one KV head, with logits given exactly (a key's K scale is 0 and its bias one
    number for all elements; queries are one number a head, so no key is rounded): keys with the given logits [n] (for a head whose
    queries are 1; every other head has queries of 1/2) and V scales and biases [n], codes [n, D].
    Returns attend(kernel), the output [new, h, D] in 64 bits and its tolerance."""
    n, d = v_codes.shape
    pages = -(-n // ps)
    cache = ta.paged_quant_cache(pages, 1, ps, d, group_size=group, dtype=dtype)
    slot = torch.arange(n, device="cuda")
    ka = torch.zeros(n, 1, d // group, 2, device="cuda")
    ka[..., 1] = logits[:, None, None]
    va = torch.stack([v_scale, v_bias], -1)[:, None, None].expand(n, 1, d // group, 2)
    cache.k_affine[slot // ps, :, slot % ps] = ka.to(dtype)
    cache.v_affine[slot // ps, :, slot % ps] = va.to(dtype)
    cache.v_codes[slot // ps, :, slot % ps] = pack(v_codes)[:, None]
    cache.k_codes.random_(-2 ** 31, 2 ** 31 - 1)
    assert torch.equal(ka.to(dtype).float(), ka)
    table = torch.arange(pages, device="cuda", dtype=torch.int32).repeat(batch, 1)
    q = torch.ones(batch * new, h, d, dtype=dtype, device="cuda")
    q[:, 1::2] = 0.5
    cu, lens = torch.arange(batch + 1, device="cuda", dtype=torch.int32) * new, i32([n] * batch)

    def attend(kernel, **kw):
        return ta.paged_quant_attention(q, cache, table, cu, lens, scale=1.0 / d, max_q_len=new, kernel=kernel, **kw)

    half = torch.finfo(dtype).eps / 2
    s, b = (va[:, 0, 0].to(dtype).double()[:, i] for i in (0, 1))
    val = s[:, None] * v_codes + b[:, None]
    mag = (s[:, None] * v_codes).abs() + b[:, None].abs()
    ref = torch.zeros(new, h, d, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(ref)
    see = visible(new, n).cuda()
    for i in range(h):
        t = logits.double() * (0.5 if i % 2 else 1.0)
        w = torch.softmax(torch.where(see, t, -math.inf), -1)
        ref[:, i] = w @ val
        # half |ref|           the output
        # 2 half W, 2^-12 W    weights and values to 16 bits; f32 work (see quant_pages.reference; the keys are exact)
        # 15 sum_k min(2^-30 max_j w_j s_j, 2^-20 s_k)
        #                      P s as f16, off by 2^-25 at most: of the largest of a row and group, 2^5 at least,
        #                      that is 2^-30; of a weight (the largest 2^7 at least) 2^-20, as scales below 2^-12
        #                      there are not taken in f16; a code is 15 at most
        # 2^-32 sum_k |v_k|    (f16) weights below the normal range
        top = (w * s.abs()).amax(-1, keepdim=True)
        lost = 15 * torch.minimum(2.0 ** -30 * top, 2.0 ** -20 * s.abs()).sum(-1, keepdim=True)
        tol[:, i] = half * ref[:, i].abs() + (2 * half + 2.0 ** -12) * (w @ mag) + lost + 1e-30
        if dtype == torch.float16:
            tol[:, i] += 2.0 ** -32 * mag.sum(0) + 2.0 ** -25       # (and half a subnormal step of the output)
    return attend, ref, tol


# base scale, scale of the odd keys, their logit, which keys those are (the warp-MMA kernel's warps take every fourth
# 16 keys each: all of these are in the same warp as the key of the largest weight, 2000)
ODD_KEYS = [
    ("f16", 0.3, 4000.0, -41.5, [17]),                   # next to no weight, before the key of the largest weight
    ("f16", 2.0 ** -12, 2.0 ** 12, -20.0, [17, 5010]),
    ("bf16", 1.0, 2.0 ** 28, -41.5, [17]),
    ("bf16", 1.0, 2.0 ** 40, -55.0, [17]),
    ("bf16", 1.0, 2.0 ** 40, -55.0, [4051, 8976]),       # behind it
    ("bf16", 1.0, 2.0 ** 40, -55.0, list(range(300))),   # the running max rises far above them
    ("bf16", 1.0, 2.0 ** 30, -2.75, [17]),               # weight 1/16: elements of code 0 still see the others
    ("f16", 2.0 ** -10, 2.0 ** 11, -2.75, [17, 4051]),
    ("bf16", 2.0 ** -100, 2.0 ** 20, -2.75, [300]),
]


@pytest.mark.parametrize("d,group", [(64, 32), (128, 32), (128, 64), (256, 64)])
@pytest.mark.parametrize("odd", range(len(ODD_KEYS)))
@pytest.mark.parametrize("new", [1, 4])
def test_keys_of_odd_scales(ta, new, odd, d, group):
    """A few keys whose V scale is many orders above the others', of little weight or of some: what the others
    add up to stays."""
    name, base, far, t, keys = ODD_KEYS[odd]
    g = torch.Generator(device="cuda")
    g.manual_seed(odd)
    n = 9000
    logits = torch.full((n,), -11.0, device="cuda")
    logits[:300] -= 30
    logits[2000] = 0.0
    scale = torch.full((n,), base, device="cuda")
    logits[keys], scale[keys] = t, far
    codes = torch.randint(0, 16, (n, d), generator=g, device="cuda")
    bias = torch.randn(n, generator=g, device="cuda") * base * 4
    bias[keys] = 0.0
    attend, ref, tol = shared_pages(ta, logits, scale, codes, bias, 64, group, DT[name], 456, new, 4)
    for kernel in FAMILIES:
        got = attend(kernel).view(456, new, 4, d)
        check(got, ref, tol)


@pytest.mark.parametrize("d,group", [(64, 64), (128, 32), (256, 32)])
def test_scales_of_zero_beside_others(ta, d, group):
    """Groups of one value (scale 0) among groups of all sizes."""
    g = torch.Generator(device="cuda")
    g.manual_seed(d)
    n = 3000
    logits = torch.randint(-40, 1, (n,), generator=g, device="cuda") * 0.25
    scale = 2.0 ** torch.randint(-30, 3, (n,), generator=g, device="cuda").float()
    scale[torch.rand(n, generator=g, device="cuda") < 0.3] = 0.0
    codes = torch.randint(0, 16, (n, d), generator=g, device="cuda")
    bias = torch.randn(n, generator=g, device="cuda") * 0.1
    attend, ref, tol = shared_pages(ta, logits, scale, codes, bias, 32, group, torch.bfloat16, 30, 2, 4)
    for kernel in FAMILIES:
        check(attend(kernel).view(30, 2, 4, d), ref, tol)


@pytest.mark.parametrize("new,d,group", [(1, 128, 64), (4, 64, 32), (2, 256, 32)])
@pytest.mark.parametrize("power", [18, 60, 110, 117, 118])
def test_queries_near_the_largest(ta, power, new, d, group):
    """bf16 queries whose products with the keys f32 still holds: the row is the value of its best key, whose
    logit is 2^9 above the others' at least.  (The tensor-core kernel takes logits up to 2^24.)"""
    families = FAMILIES if power < 20 else [1, 0, 3]
    g = torch.Generator(device="cuda")
    g.manual_seed(power)
    n = 70
    codes = torch.randint(0, 16, (n, d), generator=g, device="cuda")
    c = QuantPaged(ta, [n], [new], 4, 1, d, 16, group, torch.bfloat16, seed=power)
    order = torch.randperm(n, generator=g, device="cuda")
    pages = c.table[0, :-(-n // 16)].long()
    at = torch.arange(n, device="cuda")
    page, inside = pages[at // 16], at % 16
    t = (order.float() / 128).to(torch.bfloat16)                 # distinct, below 1
    c.cache.k_affine[page, 0, inside] = torch.stack([torch.zeros_like(t), t], -1)[:, None]
    for many in (True, False):
        c.q.zero_()
        if many:                                                 # d of them: sums up to 2^(power + 8)
            c.q.fill_(2.0 ** power)
        else:                                                    # one, up to the type's largest power
            for r in range(new):
                for h in range(4):
                    c.q[r, h, (37 * r + 19 * h) % d] = 2.0 ** (power + 8)
        for kernel in families:
            got = c.run(ta, kernel=kernel, scale=1.0 / 8)
            for r in range(new):
                best = int(order[:n - new + 1 + r].argmax())
                ref = c.vals[0][best, 0].double().expand(4, d)
                mag = c.mags[0][best, 0]
                # the value to 16 bits, the output, the weight (1 exactly, times a scale)
                check(got[r], ref, (2.0 ** -8 * 3 + 2.0 ** -12) * mag.expand(4, d))
    # the same with codes: one element of the query, and a key whose code there is the largest
    e = (5 * power) % d
    kc = torch.randint(0, 15, (n, d), generator=g, device="cuda")
    top = int(torch.randint(0, n - new + 1, (1,), generator=g, device="cuda"))
    kc[top, e] = 15
    c.cache.k_codes[page, 0, inside] = pack(kc)
    c.cache.k_affine[page, 0, inside] = torch.tensor([0.125, 0.0], dtype=torch.bfloat16, device="cuda").expand(n, d // group, 2)
    c.q.zero_()
    c.q[:, :, e] = 2.0 ** (power + 6)
    ref, mag = c.vals[0][top, 0].double().expand(new, 4, d), c.mags[0][top, 0]
    for kernel in families:
        check(c.run(ta, kernel=kernel, scale=1.0 / 8), ref, (2.0 ** -8 * 3 + 2.0 ** -12) * mag)


# powers of two on queries and K scales: of most groups, and of the last one
@pytest.mark.parametrize("name,q_most,k_most,q_last,k_last", [
    ("bf16", 0, 0, -34, 34), ("bf16", 0, 0, -60, 59), ("f16", 12, -12, -14, 13)])
@pytest.mark.parametrize("new,h,hk,d,group", [(1, 8, 2, 128, 64), (1, 4, 4, 64, 32), (4, 4, 1, 128, 32), (1, 6, 1, 256, 32),
                                              (20, 4, 2, 128, 64)])
def test_groups_of_small_queries_on_large_keys(ta, new, h, hk, d, group, name, q_most, k_most, q_last, k_last):
    """A group's queries are many orders below the others', its keys as many above: both parts of a logit count."""
    dt = DT[name]
    c = QuantPaged(ta, [300, 45], [new, new], h, hk, d, 16, group, dt, seed=-q_last)
    q, k = (torch.full((d,), 2.0 ** x, dtype=torch.float64, device="cuda") for x in (q_most, k_most))
    q[-group:], k[-group:] = 2.0 ** q_last, 2.0 ** k_last
    c.q = (c.q.double() * q).to(dt)
    c.cache.k_affine.copy_((c.cache.k_affine.double() * k[::group, None]).to(dt))
    for b, n in enumerate(c.lens):
        pages = c.table[b, :-(-n // 16)].long()
        w, a = (c.cache[i][pages].transpose(1, 2).flatten(0, 1)[:n] for i in (0, 1))
        c.keys[b] = values(w, a)[0]
    for kernel in FAMILIES:
        c.check(c.run(ta, kernel=kernel))


@pytest.mark.parametrize("power", [90, 101, 108])
@pytest.mark.parametrize("new,d,group", [(1, 128, 64), (3, 64, 32), (1, 256, 32), (30, 128, 32)])
def test_values_of_large_scales(ta, new, d, group, power):
    """V scales and biases of 2^power and more: a row's weighted sums are within f32."""
    c = QuantPaged(ta, [200, 33], [new, new], 4, 2, d, 16, group, torch.bfloat16, seed=power)
    c.cache.v_affine.copy_((c.cache.v_affine.double() * 2.0 ** power).to(c.dtype))
    for x in (c.vals, c.mags):
        for b in range(2):
            x[b] = x[b] * 2.0 ** power
    for kernel in FAMILIES:
        c.check(c.run(ta, kernel=kernel))


@pytest.mark.parametrize("kernel", FAMILIES)
@pytest.mark.parametrize("new,d,group", [(1, 128, 64), (3, 64, 64), (1, 256, 32), (4, 128, 32), (40, 128, 32)])
def test_bad_pages_do_not_read_others(ta, new, d, group, kernel):
    """A table cell outside the cache: the row is not valid, but it holds nothing of any page either."""
    c = QuantPaged(ta, [200, 60], [new, new], 4, 2, d, 16, group, torch.bfloat16, seed=6)
    tmp = ta.paged_quant_attention_workspace(c.q, c.cache, c.table, max_q_len=new, kernel=kernel)
    mine = set(c.table[0, :13].tolist())
    c.table[0, 2] = -1
    c.table[0, 7] = c.cache[0].shape[0]
    got = []
    for fill in (1.0, 2.0, math.nan):
        for page in range(c.cache[0].shape[0]):                  # every page that is not the request's
            if page not in mine:
                c.cache.k_affine[page] = fill
                c.cache.v_affine[page] = fill
        got.append(c.run(ta, kernel=kernel, tmp=tmp)[c.cu[0]:c.cu[1]])
        assert int(tmp[:1].view(torch.int32)) == 2
        tmp[:1].zero_()
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


@pytest.mark.parametrize("kernel", FAMILIES)
@pytest.mark.parametrize("fill", [math.nan, math.inf, 1000.0])
@pytest.mark.parametrize("new,d", [(1, 128), (3, 64), (6, 256), (40, 128)])
def test_keys_outside_every_row_do_not_matter(ta, new, d, fill, kernel):
    """Scales, biases and codes behind the last key and before the window, changed between two calls."""
    c = QuantPaged(ta, [200 + new, 64, new + 3], [new, 0, new], 4, 2, d, 16, 32, torch.bfloat16, seed=3)
    for window in (0, 50):
        want = c.run(ta, kernel=kernel, window=window)
        c.check(want, window)
        keep = [x.clone() for x in c.cache]
        for b, n in enumerate(c.lens):
            first = max(0, n - c.new[b] - window + 1) if window else 0
            for j in [*range(first), *range(n, -(-n // 16) * 16)]:
                page = int(c.table[b, j // 16])
                for x in (c.cache.k_affine, c.cache.v_affine):
                    x[page, :, j % 16] = fill
                for x in (c.cache.k_codes, c.cache.v_codes):
                    x[page, :, j % 16] = -1
        assert torch.equal(c.run(ta, kernel=kernel, window=window), want)
        for x, y in zip(c.cache, keep):
            x.copy_(y)


@pytest.mark.parametrize("new,h,hk,d,group", [(1, 8, 2, 128, 64), (4, 4, 4, 64, 32), (3, 8, 2, 128, 32), (2, 4, 1, 256, 32), (30, 4, 2, 128, 64)])
@pytest.mark.parametrize("far_q", [False, True])
def test_wide_scales_under_every_mask(ta, far_q, new, h, hk, d, group):
    """V scales over 2^16 from key to key, a few of them 0, some rows with a group of queries far below the others: causal,
    windowed and tree rows, pages behind the window gone, NaN in a query, the same call twice and on ordinary data after it."""
    g = torch.Generator(device="cuda")
    g.manual_seed(d + new)
    for tree in (False, True):
        c = QuantPaged(ta, [500, new, 77, 260], [new, new, 0, new], h, hk, d, 16, group, torch.bfloat16, seed=d, tree=tree)
        ordinary = [c.run(ta, kernel=k) for k in FAMILIES]
        keep = [x.clone() for x in c.cache]
        size = torch.randint(-16, 1, c.cache.v_affine.shape[:-1], generator=g, device="cuda")
        scale = c.cache.v_affine[..., 0].double() * 2.0 ** size
        scale[torch.rand(scale.shape, generator=g, device="cuda") < 0.05] = 0.0
        c.cache.v_affine[..., 0] = scale.to(c.dtype)
        q = c.q.clone()
        if far_q:
            c.q[::2, :, :32] *= 2.0 ** -20
        for b, n in enumerate(c.lens):
            pages = c.table[b, :-(-n // 16)].long()
            w, a = (c.cache[i][pages].transpose(1, 2).flatten(0, 1)[:n] for i in (2, 3))
            c.vals[b], c.mags[b] = values(w, a)
        for kernel in FAMILIES:
            for window in (0,) if tree else (0, 1, 50):
                got = c.run(ta, kernel=kernel, window=window)
                c.check(got, window)
                assert torch.equal(c.run(ta, kernel=kernel, window=window), got)
                if window:
                    table = c.table.clone()
                    for b, n in enumerate(c.lens):
                        c.table[b, :max(0, n - new - window + 1) // 16] = -1
                    assert torch.equal(c.run(ta, kernel=kernel, window=window), got)
                    c.table = table
            got, was = c.run(ta, kernel=kernel), float(c.q[0, 1, 5])
            c.q[0, 1, 5] = math.nan
            bad = c.run(ta, kernel=kernel)
            assert bool(torch.isnan(bad[0, 1]).all())
            bad[0, 1] = got[0, 1]
            assert torch.equal(bad, got)
            c.q[0, 1, 5] = was
        c.q = q
        for x, y in zip(c.cache, keep):
            x.copy_(y)
        assert all(torch.equal(c.run(ta, kernel=k), want) for k, want in zip(FAMILIES, ordinary))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("group", [32, 64])
def test_turns_that_cancel(ta, group, inter, dtype):
    """Pairs whose two products nearly or wholly take each other away, tables of sizes other than 1: codes, scales and
    biases are still those of exact arithmetic."""
    g, dt = torch.Generator(device="cuda"), DT[dtype]
    g.manual_seed(group)
    t, hk, d, ps, n_pos = 6000, 2, 128, 64, 512
    angle = math.pi / 4 + torch.randint(-3, 4, (n_pos, d // 2), generator=g, device="cuda") * 2.0 ** -torch.randint(
        10, 25, (n_pos, d // 2), generator=g, device="cuda").double()
    size = torch.tensor([1.0, 1.37, 2.0 ** -9, 700.0], dtype=torch.float64, device="cuda")[torch.arange(n_pos, device="cuda") % 4, None]
    table = torch.cat([angle.cos() * size, angle.sin() * size], -1).float()
    x = torch.randn(t, hk, d // 2, generator=g, device="cuda").to(dt)
    ulp = torch.randint(-1, 2, x.shape, generator=g, device="cuda").to(torch.int16)
    y = (x.view(torch.int16) + ulp).view(dt)                     # x, or a step off
    y = torch.where(torch.rand(x.shape, generator=g, device="cuda") < 0.1, torch.randn(x.shape, generator=g, device="cuda").to(dt) * 0.01, y)
    k = torch.stack([x, y], -1).flatten(-2) if inter else torch.cat([x, y], -1)
    k = k.contiguous()
    pos = torch.randint(0, n_pos, (t,), generator=g, device="cuda").to(torch.int32)
    slot = torch.arange(t, device="cuda")
    cache = ta.paged_quant_cache(-(-t // ps), hk, ps, d, group_size=group, dtype=dt)
    ta.paged_quant_append(k, k, cache, slot, positions=pos, rotary=table, interleaved=inter)
    codes, affine = quantised(turned(k.double(), table[pos.long()], d, inter), group, dt)
    assert torch.equal(cache.k_affine[slot // ps, :, slot % ps], affine)
    assert torch.equal(cache.k_codes[slot // ps, :, slot % ps], pack(codes))
