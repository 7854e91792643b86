"""Rotary append, 4-bit append and read, and attention over 4-bit pages on the GPU, against the
64-bit restatements of quant_pages.py."""
import math
import random

import pytest
import torch

from quant_pages import (QuantPaged, check, i32, offsets, pack, quantised, reference, turned, unpack, values, visible)

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
FAMILIES = [1, 0, 2, 3]


@pytest.fixture(scope="module")
def ta():
    import tree_masked_speculative_gb300 as m
    return m


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def slots_of(g, t, n_slots, skip=0.1):
    """t distinct slots in any order, some of them -1."""
    s = torch.randperm(n_slots, generator=g, device="cuda")[:t]
    s[torch.rand(t, generator=g, device="cuda") < skip] = -1
    return s


# -------------------------------------------------------------- rotary append
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("t,h,hk,d,rot,ps,nhd", [
    (1, 4, 4, 64, 64, 16, False), (7, 8, 2, 128, 128, 32, True), (33, 6, 1, 128, 48, 64, False),
    (130, 5, 3, 256, 256, 128, False), (3000, 9, 6, 128, 128, 16, True), (17, 2, 2, 64, 16, 256, False)])
def test_append_rotary(ta, t, h, hk, d, rot, ps, nhd, inter, dtype):
    g, dt = gen(t + d), DT[dtype]
    n_pages = -(-t // ps) + 2
    q, k, v = randn(g, t, h, d, dtype=dt, std=2.0), randn(g, t, hk, d, dtype=dt), randn(g, t, hk, d, dtype=dt)
    shape = (n_pages, ps, hk, d) if nhd else (n_pages, hk, ps, d)
    kc, vc = randn(g, *shape, dtype=dt), randn(g, *shape, dtype=dt)
    if nhd:
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    table = ta.rotary_table(700, rot)
    pos = torch.randint(0, 700, (t,), generator=g, device="cuda").to(torch.int32)
    pos[torch.rand(t, generator=g, device="cuda") < 0.1] = -1
    if t > 5:
        pos[2], pos[3], pos[4] = 0, 700, 2 ** 31 - 1
    slot = slots_of(g, t, n_pages * ps)
    if t > 5:
        slot[5] = n_pages * ps
    live = (pos >= 0) & (pos < 700)
    row = table[pos.clamp(0, 699).long()]
    # the turned values: products of 16-bit and 32-bit numbers in f32 (three roundings of terms up to
    # |x1| + |x2|), then one 16-bit rounding
    half = torch.finfo(dt).eps / 2

    def near(got, ref, x):
        tol = half * (1 + 2.0 ** -10) * ref.abs() + 2.0 ** -22 * x.abs().amax(-1, keepdim=True) + (2.0 ** -25 if dtype == "f16" else 0)
        assert bool(((got.double() - ref).abs() <= tol).all())

    kw, vw = kc.clone(), vc.clone()
    ok = live & (slot >= 0) & (slot < n_pages * ps)
    at = slot[ok]
    qw, kr = turned(q.double(), row, rot, inter), turned(k.double(), row, rot, inter)
    out = torch.full_like(q, 5.0)
    got = ta.paged_append_rotary(q, k, v, kc, vc, slot, pos, table, interleaved=inter, q_out=out)
    assert got is out and bool((out[~live] == 5.0).all())
    near(out[live], qw[live], q[live].double())
    assert torch.equal(out[live][..., rot:], q[live][..., rot:])
    near(kc[at // ps, :, at % ps], kr[ok], k[ok].double())
    vw[at // ps, :, at % ps] = v[ok]
    assert torch.equal(vc, vw)
    kw[at // ps, :, at % ps] = kc[at // ps, :, at % ps]
    assert torch.equal(kc, kw)                               # nothing else was written
    # in place, and without q
    again = q.clone()
    assert ta.paged_append_rotary(again, k, v, kc, vc, slot, pos, table, interleaved=inter, q_out=again) is again
    assert torch.equal(again[live], out[live]) and torch.equal(again[~live], q[~live])
    k2, v2 = torch.zeros_like(kc), torch.zeros_like(vc)
    assert ta.paged_append_rotary(None, k, v, k2, v2, slot, pos, table, interleaved=inter) is None
    assert torch.equal(k2[at // ps, :, at % ps], kc[at // ps, :, at % ps])


def test_append_rotary_of_a_fused_projection(ta):
    g = gen(5)
    t, h, hk, d, ps = 70, 8, 2, 128, 16
    qkv = randn(g, t, h + 2 * hk, d, dtype=torch.bfloat16)
    q, k, v = qkv[:, :h], qkv[:, h:h + hk], qkv[:, h + hk:]
    table, pos = ta.rotary_table(100, d), torch.arange(t, device="cuda", dtype=torch.int32)
    slot = torch.arange(t, device="cuda")
    caches = [torch.zeros(6, hk, ps, d, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    want = ta.paged_append_rotary(q.contiguous(), k.contiguous(), v.contiguous(), *caches[:2], slot, pos, table)
    rest = qkv[:, h:].clone()
    got = ta.paged_append_rotary(q, k, v, *caches[2:], slot, pos, table, q_out=q)
    assert got is q and torch.equal(qkv[:, :h], want) and torch.equal(qkv[:, h:], rest)
    assert torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])
    x = torch.zeros(h, t, d, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    ta.paged_append_rotary(q.contiguous().copy_(qkv[:, :h]), k, v, *caches[:2], slot, pos * 0, table, q_out=x)
    assert torch.equal(x, want) and torch.equal(caches[0], k.new_zeros(6 * ps, hk, d).index_copy(0, slot, k).view(6, ps, hk, d).transpose(1, 2))


# ------------------------------------------------------------------ 4-bit rows
def special_rows(g, t, hk, d, dt):
    """Rows where a code or a scale is hard to get right: ties, constant groups, a far offset, tiny and huge
    ranges, zeros, the largest values, infinities and NaN."""
    x = torch.randn(t, hk, d, generator=g, device="cuda")
    kind = torch.randint(0, 12, (t, hk, d // 32), generator=g, device="cuda").repeat_interleave(32, -1)
    small = torch.randint(0, 31, (t, hk, d), generator=g, device="cuda").float()
    big = torch.finfo(dt).max
    tiny = torch.finfo(dt).smallest_normal
    x = torch.where(kind == 1, small * 0.5, x)                   # scale 1 where 0 and 15 occur: ties
    x = torch.where(kind == 2, torch.full_like(x, 0.7), x)
    x = torch.where(kind == 3, 100 + x, x)
    x = torch.where(kind == 4, x * tiny * 3, x)
    x = torch.where(kind == 5, x.sign() * big * 0.6, x)
    x = torch.where(kind == 6, torch.zeros_like(x), x)
    x = torch.where(kind == 7, small * 2.0 ** -9, x)
    x = torch.where((kind == 8) & (small == 3), torch.full_like(x, math.inf), x)
    x = torch.where((kind == 9) & (small == 4), torch.full_like(x, math.nan), x)
    x = torch.where(kind == 10, x * 1000, x)
    x = torch.where(kind == 11, torch.where(small == 5, torch.full_like(x, big), x * 0.01), x)
    return x.to(dt)


def same(a, b):
    """Equal values, NaN equal to NaN."""
    return bool(((a == b) | (torch.isnan(a) & torch.isnan(b))).all())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("group", [32, 64])
@pytest.mark.parametrize("t,h,hk,d,rot,inter,ps,nhd", [
    (1, 0, 4, 64, 0, False, 16, False), (9, 0, 3, 128, 0, False, 32, True), (2500, 0, 2, 256, 0, False, 64, False),
    (1, 4, 1, 128, 128, False, 16, False), (65, 8, 2, 128, 128, True, 32, True), (130, 3, 3, 256, 128, False, 128, False),
    (3001, 6, 5, 64, 48, False, 16, False), (40, 0, 2, 256, 208, True, 256, False)])
def test_quant_append_and_read(ta, t, h, hk, d, rot, inter, ps, nhd, group, dtype):
    """Codes, scales and biases are those of exact arithmetic, bit for bit."""
    g, dt = gen(t + d + group), DT[dtype]
    n_pages = -(-t // ps) + 2
    lead = (n_pages, ps, hk) if nhd else (n_pages, hk, ps)
    parts = []
    for _ in "kv":
        c = torch.randint(-2 ** 31, 2 ** 31, (*lead, d // 8), generator=g, device="cuda").to(torch.int32)
        a = randn(g, *lead, d // group, 2, dtype=dt)
        parts += [c.transpose(1, 2), a.transpose(1, 2)] if nhd else [c, a]
    cache = ta.PagedQuantCache(*parts)
    k = special_rows(g, t, hk, d, dt) if not rot or t > 64 else randn(g, t, hk, d, dtype=dt)
    v = special_rows(g, t, hk, d, dt)
    slot = slots_of(g, t, n_pages * ps)
    ok = slot >= 0
    kw = {}
    k64 = k.double()
    if rot:
        table = ta.rotary_table(5000, rot)
        pos = torch.randint(0, 5000, (t,), generator=g, device="cuda").to(torch.int32)
        pos[torch.rand(t, generator=g, device="cuda") < 0.1] = -1
        if t > 9:
            pos[4], pos[5], pos[6], pos[7] = 0, 1, 5000, 0
        live = (pos >= 0) & (pos < 5000)
        ok &= live
        k64 = turned(k64, table[pos.clamp(0, 4999).long()], rot, inter)
        kw = dict(positions=pos, rotary=table, interleaved=inter)
        if h:
            kw["q"] = randn(g, t, h, d, dtype=dt, std=2.0)
            kw["q_out"] = torch.full_like(kw["q"], 5.0)
    want = [p.clone() for p in cache]
    at = slot[ok]
    for i, x in enumerate((k64, v.double())):
        codes, affine = quantised(x[ok], group, dt)
        want[2 * i][at // ps, :, at % ps] = pack(codes)
        want[2 * i + 1][at // ps, :, at % ps] = affine
    got = ta.paged_quant_append(k, v, cache, slot, **kw)
    for i in (1, 3):
        assert same(cache[i], want[i])
    for i in (0, 2):
        assert torch.equal(cache[i], want[i])
    if h:
        assert got is kw["q_out"] and bool((got[~live] == 5.0).all())
        kc, vc = (torch.zeros(n_pages, hk, ps, d, dtype=dt, device="cuda") for _ in range(2))
        q16 = ta.paged_append_rotary(kw["q"], k, v, kc, vc, slot, pos, table, interleaved=inter)
        assert torch.equal(got[live], q16[live])
    else:
        assert got is None
    # rows read back, slots twice and outside the cache among them
    ask = torch.cat([slot, slot.flip(0), torch.tensor([-1, n_pages * ps, 0], device="cuda")])
    out = tuple(torch.full((ask.numel(), hk, d), 5.0, dtype=dt, device="cuda") for _ in range(2))
    k2, v2 = ta.paged_quant_read(cache, ask, out=out)
    inside = (ask >= 0) & (ask < n_pages * ps)
    for x, c, a in ((k2, cache[0], cache[1]), (v2, cache[2], cache[3])):
        a_ = ask[inside]
        w = values(c[a_ // ps, :, a_ % ps], a[a_ // ps, :, a_ % ps])[0]
        assert same(x[inside], w.float().to(dt)) and not bool(x[~inside].any())
    k3, v3 = ta.paged_quant_read(cache, ask[:1].clone().fill_(-1))
    assert k3.shape == (1, hk, d) and not bool(k3.any()) and not bool(v3.any())


def test_pack_is_its_own_inverse():
    c = torch.randint(0, 16, (5, 128), device="cuda")
    assert torch.equal(unpack(pack(c)), c)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
def test_many_turned_rows_are_exact(ta, inter, dtype):
    """Tens of millions of elements, none next to a border is taken wrong."""
    g, dt = gen(11), DT[dtype]
    t, hk, d, group, ps = 20000, 8, 128, 64 if inter else 32, 64
    k = randn(g, t, hk, d, dtype=dt)
    cache = ta.paged_quant_cache(-(-t // ps), hk, ps, d, group_size=group, dtype=dt)
    table = ta.rotary_table(100000, d)
    pos = torch.randint(0, 100000, (t,), generator=g, device="cuda").to(torch.int32)
    slot = torch.randperm(cache[0].shape[0] * ps, generator=g, device="cuda")[:t]
    ta.paged_quant_append(k, k, cache, slot, positions=pos, rotary=table, interleaved=inter)
    for i, x in enumerate((turned(k.double(), table[pos.long()], d, inter), k.double())):
        codes, affine = quantised(x, group, dt)
        assert torch.equal(cache[2 * i + 1][slot // ps, :, slot % ps], affine)
        assert torch.equal(cache[2 * i][slot // ps, :, slot % ps], pack(codes))


# ------------------------------------------------------------------- attention
@pytest.mark.parametrize("ps", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("h,hk,d,group", [(4, 4, 64, 32), (2, 1, 64, 64), (8, 2, 128, 64), (6, 2, 256, 32), (16, 1, 128, 32), (8, 1, 256, 64)])
def test_decode(ta, h, hk, d, group, dtype, ps):
    lens = [1, 700, 16, 33, 129, 0, 255, 1300]
    new = [1, 1, 1, 1, 1, 0, 1, 1]
    c = QuantPaged(ta, lens, new, h, hk, d, ps, group, DT[dtype], seed=ps + d)
    for kernel in FAMILIES:
        for window in (0, 1, 100):
            c.check(c.run(ta, kernel=kernel, window=window), window)


@pytest.mark.parametrize("h,hk,d,ps,group,dtype,new", [
    (8, 2, 128, 16, 64, "bf16", [4, 1, 3, 0, 2]), (8, 2, 128, 16, 32, "f16", [2, 3, 4, 1, 4]),
    (8, 2, 128, 32, 64, "bf16", [40, 1, 129, 0, 64]), (6, 1, 256, 64, 32, "f16", [90, 2, 31, 0, 50]),
    (4, 4, 64, 16, 32, "bf16", [300, 7, 1, 5, 128]), (32, 1, 128, 64, 32, "bf16", [9, 1, 30, 2, 3]),
    (10, 2, 128, 128, 64, "f16", [77, 1, 0, 0, 260]), (12, 4, 256, 16, 64, "bf16", [5, 1, 4, 2, 3]),
    (4, 2, 64, 256, 64, "f16", [3, 1, 2, 8, 4]), (4, 2, 128, 16, 32, "bf16", [7, 1, 8, 0, 3])])
def test_chunks(ta, h, hk, d, ps, group, dtype, new):
    lens = [x + n for x, n in zip([0, 900, 250, 0, 77], new)]
    c = QuantPaged(ta, lens, new, h, hk, d, ps, group, DT[dtype], seed=d + ps, pad=3)
    for kernel in FAMILIES:
        for window in (0, 5, 130):
            out = torch.full_like(c.q, 5.0)
            c.check(c.run(ta, kernel=kernel, window=window, out=out), window)
            assert bool((out[c.cu[-1]:] == 5.0).all())


@pytest.mark.parametrize("h,hk,d,ps,group,dtype,new", [
    (8, 2, 128, 16, 64, "bf16", [4, 1, 3, 0, 2]), (8, 2, 128, 16, 32, "bf16", [40, 1, 200, 0, 64]),
    (24, 4, 256, 64, 64, "f16", [32, 32, 31, 0, 5]), (4, 4, 64, 32, 32, "f16", [256, 7, 1, 5, 128]),
    (16, 2, 128, 128, 64, "f16", [8, 16, 2, 1, 0]), (8, 2, 128, 16, 32, "f16", [7, 8, 2, 1, 6])])
def test_trees(ta, h, hk, d, ps, group, dtype, new):
    lens = [x + n for x, n in zip([0, 900, 250, 0, 77], new)]
    c = QuantPaged(ta, lens, new, h, hk, d, ps, group, DT[dtype], seed=d + ps, pad=1, tree=True)
    for kernel in FAMILIES:
        c.check(c.run(ta, kernel=kernel))


@pytest.mark.parametrize("kernel", FAMILIES)
@pytest.mark.parametrize("new", [1, 3, 7, 40])
def test_fewer_keys_than_tokens(ta, new, kernel):
    """Tokens before position 0 see nothing and give zeros."""
    lens = [new - 1, max(0, new - 2), new + 20, 0]
    c = QuantPaged(ta, lens, [new] * 4, 8, 2, 128, 16, 64, torch.bfloat16, seed=new)
    got = c.run(ta, kernel=kernel)
    c.check(got)
    for b, n in enumerate(lens):
        assert not bool(got[b * new:b * new + max(0, new - n)].any())


@pytest.mark.parametrize("kernel", FAMILIES)
@pytest.mark.parametrize("new,d", [(1, 128), (5, 64), (60, 256)])
def test_nhd_cache_and_strided_rows(ta, new, d, kernel):
    lens = [300, 77, new]
    c = QuantPaged(ta, lens, [new] * 3, 8, 2, d, 32, 32, torch.float16, seed=new, nhd=True)
    wide = torch.zeros(c.q.shape[0], 12, d, dtype=c.dtype, device="cuda")
    wide[:, 2:10] = c.q
    c.q = wide[:, 2:10]
    out = torch.zeros(8, c.q.shape[0], d, dtype=c.dtype, device="cuda").transpose(0, 1)
    got = c.run(ta, kernel=kernel, out=out)
    assert got is out
    c.check(got)


@pytest.mark.parametrize("kernel", FAMILIES)
@pytest.mark.parametrize("fill", [math.nan, math.inf, -math.inf, 60000.0])
@pytest.mark.parametrize("new,d", [(1, 128), (3, 64), (6, 256), (40, 128)])
def test_masked_keys_do_not_matter(ta, new, d, fill, kernel):
    """Scales and biases of keys that a row does not see, whatever they hold: the last token's row
    for the rows before it, keys before the window, and everything behind the last key."""
    lens = [200 + new, 64, new + 3]
    new = [new, 0, new]
    c = QuantPaged(ta, lens, new, 4, 2, d, 16, 32, torch.bfloat16, seed=3)
    for window in (0, 50):
        clean = c.run(ta, kernel=kernel, window=window)
        spoilt = c.run(ta, kernel=kernel, window=window, out=torch.zeros_like(c.q))
        assert torch.equal(clean, spoilt)
    keep = [x.clone() for x in c.cache]
    clean = c.run(ta, kernel=kernel)
    for b in (0, 2):                                        # the last key of each request
        j = lens[b] - 1
        page = int(c.table[b, j // 16])
        c.cache[1][page, :, j % 16] = fill
        c.cache[3][page, :, j % 16] = fill
    got = c.run(ta, kernel=kernel)
    for b in (0, 2):
        s = slice(c.cu[b], c.cu[b + 1] - 1)
        assert torch.equal(got[s], clean[s])
        if not math.isfinite(fill) and fill != -math.inf:
            assert bool(torch.isnan(got[c.cu[b + 1] - 1]).all())
    for x, y in zip(c.cache, keep):
        x.copy_(y)
    first = c.run(ta, kernel=kernel, window=30)             # keys before every row's window
    page = int(c.table[0, 0])
    c.cache[1][page] = fill
    c.cache[3][page] = fill
    assert torch.equal(c.run(ta, kernel=kernel, window=30), first)


@pytest.mark.parametrize("kernel", FAMILIES)
@pytest.mark.parametrize("new", [1, 4, 50])
def test_nan_logits_reach_the_rows_that_see_them(ta, new, kernel):
    """A NaN in a query makes its row NaN, one in a seen key's scale the rows that see it."""
    c = QuantPaged(ta, [300, 120], [new, new], 8, 2, 128, 16, 64, torch.float16, seed=9)
    clean = c.run(ta, kernel=kernel)
    c.q[0, 3, 17] = math.nan
    got = c.run(ta, kernel=kernel)
    assert bool(torch.isnan(got[0, 3]).all())
    mine = torch.ones_like(got, dtype=torch.bool)
    mine[0, 3] = False
    assert torch.equal(got[mine], clean[mine])
    c.q[0, 3, 17] = 1.0
    clean = c.run(ta, kernel=kernel)
    page = int(c.table[1, 2])
    c.cache[1][page, 1, 5, 0, 1] = math.nan                 # key 37 of request 1, KV head 1
    got = c.run(ta, kernel=kernel)
    assert bool(torch.isnan(got[new:, 4:]).all())
    assert torch.equal(got[:new], clean[:new]) and torch.equal(got[new:, :4], clean[new:, :4])


@pytest.mark.parametrize("kernel", FAMILIES)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("new", [1, 4, 40])
def test_scales_of_all_sizes(ta, new, dtype, kernel):
    """Values whose groups' scales and biases differ by many orders, from key to key and from group to
    group, and rows of large and of tiny queries."""
    c = QuantPaged(ta, [500, 90], [new, new], 8, 2, 128, 16, 32, DT[dtype], seed=new)
    g = gen(4)
    exps = torch.tensor([-6, -3, 0, 3] if dtype == "f16" else [-30, -10, 0, 30], device="cuda")
    grp = exps.view(4, 1)
    key = torch.randint(-6, 5, (c.cache[3].shape[0], 2, 16, 1, 1), generator=g, device="cuda")
    c.cache[3].copy_((c.cache[3].double() * 2.0 ** (grp + key)).to(c.dtype))
    c.q[::3] *= 2.0 ** -12
    big = c.q[1::3].clone()
    c.q[1::3] = big * 2
    for b, n in enumerate(c.lens):
        pages = c.table[b, :-(-n // 16)].long()
        w, a = (c.cache[i][pages].transpose(1, 2).flatten(0, 1)[:n] for i in (2, 3))
        c.vals[b], c.mags[b] = values(w, a)
    got = c.run(ta, kernel=kernel)
    for b, n in enumerate(c.lens):
        s = slice(c.cu[b], c.cu[b + 1])
        for j in range(4):                                  # a group's tolerance does not see the others
            e = slice(32 * j, 32 * j + 32)
            see = visible(c.new[b], n)
            ref, tol = reference(c.q[s], c.keys[b], torch.where(torch.arange(128, device="cuda") // 32 == j, c.vals[b], 0.0),
                                 torch.where(torch.arange(128, device="cuda") // 32 == j, c.mags[b], 0.0), see, c.scale, c.half)
            # f16 results below the normal range are half a subnormal step off
            check(got[s][..., e], ref[..., e], tol[..., e] + (2.0 ** -25 if dtype == "f16" else 0))


@pytest.mark.parametrize("kernel", FAMILIES)
def test_scales_of_the_logits(ta, kernel):
    """A scale of zero weighs every visible key alike; a negative one turns the order."""
    c = QuantPaged(ta, [300, 40], [1, 1], 8, 2, 128, 16, 64, torch.bfloat16, seed=3)
    for c.scale in (0.0, -0.1, 1e-30, 0.2):
        c.check(c.run(ta, kernel=kernel))
    c = QuantPaged(ta, [300, 90], [50, 50], 8, 2, 128, 16, 64, torch.bfloat16, seed=4)
    for c.scale in (0.0, -0.1, 1e-30, 0.2):
        c.check(c.run(ta, kernel=kernel))


@pytest.mark.parametrize("h,hk,d,group,new,batch", [(4, 2, 64, 32, 1, 700), (8, 2, 128, 64, 2, 300), (2, 2, 128, 32, 1, 2),
                                                    (4, 1, 256, 64, 20, 400), (8, 1, 256, 32, 1, 2)])
def test_many_or_long_requests(ta, h, hk, d, group, new, batch):
    """More requests than a block has threads; contexts cut into many pieces."""
    rnd = random.Random(batch)
    lens = [rnd.randint(new, 90) for _ in range(batch)] if batch > 2 else [30000, 9001]
    new = [new if batch == 2 or rnd.random() < 0.9 else 0 for _ in lens]
    c = QuantPaged(ta, lens, new, h, hk, d, 16, group, torch.bfloat16, seed=batch)
    got, want = c.run(ta), c.run(ta, kernel=1)
    # both within the weights', the keys' and the output's rounding of one value (values up to 6)
    assert bool(((got - want).abs() <= 2.0 ** -7 * want.abs() + 6 * 2.0 ** -8).all())
    if batch == 2:
        c.check(got)


@pytest.mark.parametrize("kernel", FAMILIES)
@pytest.mark.parametrize("new", [1, 4, 60])
def test_bad_pages_set_the_status(ta, new, kernel):
    c = QuantPaged(ta, [300, 90, 200], [new] * 3, 4, 2, 128, 16, 32, torch.bfloat16, seed=6)
    tmp = ta.paged_quant_attention_workspace(c.q, c.cache, c.table, max_q_len=new, kernel=kernel)
    c.check(c.run(ta, kernel=kernel, tmp=tmp))
    assert int(tmp[:1].view(torch.int32)) == 0
    for bad in (-1, c.cache[0].shape[0], 2 ** 31 - 1):
        t = c.table.clone()
        t[1, 2] = bad
        keep, c.table = c.table, t
        got = c.run(ta, kernel=kernel, tmp=tmp)
        c.table = keep
        assert int(tmp[:1].view(torch.int32)) == 2
        tmp[:1].zero_()
        c.check(got, only=(0, 2))


@pytest.mark.parametrize("kernel", FAMILIES)
@pytest.mark.parametrize("new", [1, 4, 60])
def test_pages_behind_the_window_may_be_gone(ta, new, kernel):
    c = QuantPaged(ta, [300, 90, 200], [new] * 3, 4, 2, 128, 16, 64, torch.bfloat16, seed=6)
    tmp = ta.paged_quant_attention_workspace(c.q, c.cache, c.table, max_q_len=new, kernel=kernel, window=20)
    for b, n in enumerate(c.lens):
        c.table[b, :max(0, n - new - 20 + 1) // 16] = -1
    c.check(c.run(ta, kernel=kernel, tmp=tmp, window=20), 20)
    assert int(tmp[:1].view(torch.int32)) == 0


@pytest.mark.parametrize("kernel", FAMILIES)
@pytest.mark.parametrize("max_q", [2, 60])
def test_contradicting_lengths_set_the_status(ta, max_q, kernel):
    c = QuantPaged(ta, [90, 40, 60], [2, 1, 2], 4, 2, 128, 16, 64, torch.bfloat16, seed=8)
    tmp = ta.paged_quant_attention_workspace(c.q, c.cache, c.table, max_q_len=max_q, kernel=kernel)

    def status(cu, lens):
        ta.paged_quant_attention(c.q, c.cache, c.table, i32(cu), i32(lens), scale=0.1, max_q_len=max_q, kernel=kernel, tmp=tmp)
        s = int(tmp[:1].view(torch.int32))
        tmp[:1].zero_()
        return s

    assert status(c.cu, c.lens) == 0
    cap = c.table.shape[1] * 16
    for cu, lens in (([0, 2, 1, 5], c.lens), ([0, 2, 3, 99], c.lens), ([-1, 2, 3, 5], c.lens), (c.cu, [90, -4, 60]),
                     (c.cu, [90, 40, cap + 1]), (c.cu, [2 ** 31 - 1, 40, 60])):
        # (a length that the table row holds may name cells of -7: a bad page as well)
        assert status(cu, lens) & 4


def test_cache_beyond_32_bit_offsets(ta):
    """Pages more than 2^31 words from the cache's start."""
    n_pages, hk, ps, d, group = 9, 1, 16, 128, 64
    stride = 2 ** 28 + 64
    c = QuantPaged(ta, [100], [1], 4, hk, d, ps, group, torch.bfloat16, spare=2, seed=2)
    # K's and V's pages in turn in one allocation, far apart
    room = torch.empty(stride * n_pages, dtype=torch.int32, device="cuda")
    far = [room[o:].as_strided((n_pages, hk, ps, d // 8), (stride, ps * d // 8, d // 8, 1)) for o in (0, ps * d // 8)]
    assert c.cache[0].shape[0] == n_pages and stride * (n_pages - 1) > 2 ** 31
    far[0].copy_(c.cache[0])
    far[1].copy_(c.cache[2])
    c.cache = ta.PagedQuantCache(far[0], c.cache[1], far[1], c.cache[3])
    for k in FAMILIES:
        c.check(c.run(ta, kernel=k))
    new = torch.randn(2, hk, d, device="cuda").to(torch.bfloat16)
    slot = torch.tensor([8 * ps + 3, -1], device="cuda")
    ta.paged_quant_append(new, new, c.cache, slot)
    codes, affine = quantised(new.double(), group, torch.bfloat16)
    for x in ta.paged_quant_read(c.cache, slot):
        assert torch.equal(x[0], values(pack(codes), affine)[0].float().to(torch.bfloat16)[0])


@pytest.mark.parametrize("new", [1, 4, 60])
def test_repeats_streams_and_graphs(ta, new):
    """The same call gives the same bits; on another stream; captured and replayed with other lengths."""
    c = QuantPaged(ta, [400, 90, 33, 1000], [new, 0, min(new, 33), new], 8, 2, 128, 16, 64, torch.bfloat16, seed=new)
    want = c.run(ta, out=torch.zeros_like(c.q))
    for _ in range(3):
        assert torch.equal(c.run(ta, out=torch.zeros_like(c.q)), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = c.run(ta, out=torch.zeros_like(c.q), stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
    lens, cu, out = i32(c.lens), i32(c.cu), torch.zeros_like(c.q)
    tmp = ta.paged_quant_attention_workspace(c.q, c.cache, c.table, max_q_len=new)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ta.paged_quant_attention(c.q, c.cache, c.table, cu, lens, scale=c.scale, max_q_len=new, tmp=tmp, out=out)
    out.zero_()
    graph.replay()
    assert torch.equal(out, want)
    lens.copy_(i32([399, 90, 33, 500]))
    want2 = ta.paged_quant_attention(c.q, c.cache, c.table, cu, lens, scale=c.scale, max_q_len=new, out=torch.zeros_like(c.q))
    graph.replay()
    assert torch.equal(out, want2) and not torch.equal(out, want)
    assert int(tmp[:1].view(torch.int32)) == 0


@pytest.mark.parametrize("d,h,hk,ps,group,dtype,inter", [
    (128, 8, 2, 16, 64, "bf16", False), (64, 4, 4, 32, 32, "f16", True), (256, 6, 1, 64, 32, "bf16", False)])
def test_a_serving_run(ta, d, h, hk, ps, group, dtype, inter):
    """Steps of plan, quantized append with rotation and attention, as a server makes them (prompt chunks, tokens,
    drafts of which a part is kept), against 64-bit attention over the values that the cache stands for."""
    g, dt, rnd = gen(d), DT[dtype], random.Random(d)
    batch, width, most = 5, 12, 40
    cache = ta.paged_quant_cache(batch * width, hk, ps, d, group_size=group, dtype=dt)
    table = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
    pages = torch.randperm(batch * width, generator=g, device="cuda").to(torch.int32)
    held, n_free = i32([0] * batch), i32([batch * width])
    rotary = ta.rotary_table(width * ps, d)
    have = [0] * batch
    rows = [torch.zeros(0, hk, d, dtype=torch.float64, device="cuda") for _ in range(batch)]
    vals = [x.clone() for x in rows]
    mags = [x.clone() for x in rows]
    for step in range(6):
        keep = [rnd.randint(max(0, n - 2), n) for n in have]
        new = [rnd.randint(0, 40) if step == 0 else rnd.randint(0, 4) for _ in range(batch)]
        t = sum(new) + 2
        plan = ta.paged_plan(i32(keep), i32(new), held, table, pages, n_free, page_size=ps, max_tokens=t)
        assert int(plan.status) == 0
        held, n_free = plan.held, plan.n_free
        q, k, v = randn(g, t, h, d, dtype=dt, std=2.0), randn(g, t, hk, d, dtype=dt), randn(g, t, hk, d, dtype=dt)
        qr = ta.paged_quant_append(k, v, cache, plan.slot_map, q=q, positions=plan.positions, rotary=rotary,
                                   interleaved=inter, q_out=torch.zeros_like(q))
        out = ta.paged_quant_attention(qr, cache, table, plan.cu_q, plan.kv_lens, scale=d ** -0.5, max_q_len=most,
                                       out=torch.zeros_like(q))
        cu = offsets(new)
        for b in range(batch):
            s = slice(cu[b], cu[b + 1])
            pos = torch.arange(keep[b], keep[b] + new[b], device="cuda")
            kk = values(*[f(x) for f, x in zip((pack, lambda y: y), quantised(turned(k[s].double(), rotary[pos], d, inter), group, dt))])
            vv = values(*[f(x) for f, x in zip((pack, lambda y: y), quantised(v[s].double(), group, dt))])
            rows[b] = torch.cat([rows[b][:keep[b]], kk[0]])
            vals[b], mags[b] = torch.cat([vals[b][:keep[b]], vv[0]]), torch.cat([mags[b][:keep[b]], vv[1]])
            have[b] = keep[b] + new[b]
            if new[b]:
                ref, tol = reference(qr[s], rows[b], vals[b], mags[b], visible(new[b], have[b]), d ** -0.5, torch.finfo(dt).eps / 2)
                check(out[s], ref, tol)


# ------------------------------------------------------------------ calls as others make them
@pytest.mark.parametrize("kernel", FAMILIES)
@pytest.mark.parametrize("h,d", [(24, 64), (56, 128), (128, 128), (5, 256), (128, 256)])
def test_many_heads_of_one_kv_head(ta, h, d, kernel):
    """Units of one or a few tokens, rows that do not divide by the heads."""
    c = QuantPaged(ta, [150, 64, 9], [1, 5, 9], h, 1, d, 32, 32, torch.float16, seed=h, tree=True)
    c.check(c.run(ta, kernel=kernel))


@pytest.mark.parametrize("new", [1, 40])
def test_requests_that_share_pages(ta, new):
    """A common prefix: both requests' tables name the same pages."""
    c = QuantPaged(ta, [320, 330], [new, new], 8, 2, 128, 32, 64, torch.bfloat16, seed=18)
    c.table[1, :8] = c.table[0, :8]
    for rows in (c.keys, c.vals, c.mags):
        rows[1][:256] = rows[0][:256]
    c.check(c.run(ta))


@pytest.mark.parametrize("new", [1, 5, 90])
def test_two_streams_at_once(ta, new):
    cs = [QuantPaged(ta, [2000, 77 + new, 300], [new] * 3, 8, 2, 128, 16, 64, torch.bfloat16, seed=19 + i) for i in range(2)]
    want = [c.run(ta, out=torch.zeros_like(c.q)) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    tmps = [ta.paged_quant_attention_workspace(c.q, c.cache, c.table, max_q_len=new) for c in cs]
    rows, lens = [i32(c.cu) for c in cs], [i32(c.lens) for c in cs]
    got = [[torch.zeros_like(c.q) for c in cs] for _ in range(20)]
    torch.cuda.synchronize()
    for pair in got:
        for i, c in enumerate(cs):
            ta.paged_quant_attention(c.q, c.cache, c.table, rows[i], lens[i], scale=c.scale, max_q_len=new, tmp=tmps[i],
                                     out=pair[i], stream=streams[i])
    torch.cuda.synchronize()
    for pair in got:
        assert all(torch.equal(x, y) for x, y in zip(pair, want))
    assert not any(int(tmp.view(torch.int32)[0]) for tmp in tmps)


@pytest.mark.parametrize("kernel", FAMILIES)
@pytest.mark.parametrize("new", [4, 70])
def test_parents_outside_their_node_end_the_chain(ta, new, kernel):
    """Itself, a later node, a value past every node or far below: each is the end of the chain."""
    c = QuantPaged(ta, [300, 90], [new, new], 8, 2, 64, 32, 32, torch.bfloat16, seed=29, tree=True)
    for odd in (lambda i: i, lambda i: i + 1, lambda i: 2 ** 31 - 1, lambda i: -2 ** 31, lambda i: new):
        c.parents = [[odd(i) if i % 3 == 0 else i - 1 for i in range(new)] for _ in c.new]
        c.check(c.run(ta, kernel=kernel))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 3, 40])
def test_a_workspace_serves_other_batches(ta, d, new):
    """The tmp of one request takes the calls of twenty, and the other way round."""
    one, many = (QuantPaged(ta, [90 + 7 * i for i in range(b)], [new] * b, 4, 2, d, 16, 64, torch.bfloat16, seed=30 + b)
                 for b in (1, 20))
    tmps = [ta.paged_quant_attention_workspace(c.q, c.cache, c.table, max_q_len=new) for c in (one, many)]
    for c in (one, many):
        for tmp in tmps:
            c.check(c.run(ta, tmp=tmp))
            assert int(tmp.view(torch.int32)[0]) == 0


@pytest.mark.parametrize("new", [1, 40])
def test_two_graphs_on_one_workspace(ta, new):
    """Replayed one after the other, in either order, with the workspace filled in between but for its status."""
    cs = [QuantPaged(ta, [2000, 77 + new], [new] * 2, 8, 2, 128, 16, 32, torch.float16, seed=50 + i) for i in range(2)]
    want = [c.run(ta, out=torch.zeros_like(c.q)) for c in cs]
    tmp = ta.paged_quant_attention_workspace(cs[0].q, cs[0].cache, cs[0].table, max_q_len=new)
    rows, lens, outs, graphs = [i32(c.cu) for c in cs], [i32(c.lens) for c in cs], [torch.zeros_like(c.q) for c in cs], []
    for i, c in enumerate(cs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            ta.paged_quant_attention(c.q, c.cache, c.table, rows[i], lens[i], scale=c.scale, max_q_len=new, tmp=tmp, out=outs[i])
    for order in ((0, 1), (1, 0), (0, 0), (1, 1)):
        for o in outs:
            o.zero_()
        tmp[64:].fill_(float("nan"))
        for i in order:
            graphs[i].replay()
        for i in set(order):
            assert torch.equal(outs[i], want[i])
    assert int(tmp.view(torch.int32)[0]) == 0


def test_appends_and_reads_in_graphs_and_on_streams(ta):
    """Captured and replayed with other rows, slots and positions; on another stream than the current one."""
    g, t, h, hk, d, ps = gen(77), 37, 8, 2, 128, 16
    rotary = ta.rotary_table(500, d)
    q, k, v = (randn(g, t, n, d, dtype=torch.bfloat16) for n in (h, hk, hk))
    slot, pos = slots_of(g, t, 6 * ps), torch.randint(-1, 510, (t,), generator=g, device="cuda", dtype=torch.int32)

    def fresh():
        return ([torch.zeros(6, hk, ps, d, dtype=torch.bfloat16, device="cuda") for _ in "kv"],
                ta.paged_quant_cache(6, hk, ps, d, group_size=32), [torch.zeros_like(q) for _ in range(2)],
                [torch.zeros_like(k) for _ in range(2)])

    def run(state, **kw):
        pages, cache, qs, kv = state
        ta.paged_append_rotary(q, k, v, *pages, slot, pos, rotary, q_out=qs[0], **kw)
        ta.paged_quant_append(k, v, cache, slot, q=q, positions=pos, rotary=rotary, q_out=qs[1], **kw)
        ta.paged_quant_read(cache, slot, out=tuple(kv), **kw)
        return [*pages, *cache, *qs, *kv]

    want, state = run(fresh()), fresh()
    side, stream = fresh(), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = run(side, stream=stream)
    torch.cuda.current_stream().wait_stream(stream)
    assert all(same(x, y) for x, y in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(state)
    graph.replay()
    assert all(same(x, y) for x, y in zip(got, want))
    for x, y in ((q, randn(g, *q.shape, dtype=q.dtype)), (k, randn(g, *k.shape, dtype=k.dtype)), (slot, slots_of(g, t, 6 * ps)),
                 (pos, pos.flip(0))):
        x.copy_(y)
    for x in got:
        x.zero_()
    want = run(fresh())
    graph.replay()
    assert all(same(x, y) for x, y in zip(got, want))


def test_slots_read_again(ta):
    """A slot named by several rows of one read, in any order."""
    g, hk, d, ps = gen(5), 3, 64, 16
    cache = ta.paged_quant_cache(4, hk, ps, d, group_size=64, dtype=torch.float16)
    k, v = (randn(g, 4 * ps, hk, d, dtype=torch.float16) for _ in "kv")
    ta.paged_quant_append(k, v, cache, torch.arange(4 * ps, device="cuda"))
    whole = ta.paged_quant_read(cache, torch.arange(4 * ps, device="cuda"))
    pick = torch.randint(0, 4 * ps, (1000,), generator=g, device="cuda")
    for x, y in zip(ta.paged_quant_read(cache, pick), whole):
        assert torch.equal(x, y[pick])


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("d,group", [(64, 32), (128, 64), (256, 32)])
def test_waits_that_give_up_set_the_status(ta, d, group, tree):
    """Every wait bounded by a few polls: CTAs give up at different places, let their copies and
    products end, say so in the status word and return; the next call on the same workspace is right."""
    c = QuantPaged(ta, [900, 60, 3000, 61], [60, 60, 33, 7], 8, 2, d, 16, group, torch.bfloat16, seed=27, tree=tree)
    want = c.run(ta, kernel=2)
    tmp = ta.paged_quant_attention_workspace(c.q, c.cache, c.table, max_q_len=60, kernel=2)
    word = tmp.view(torch.int32)
    cu, lens, parents = i32(c.cu), i32(c.lens), c.flat_parents()
    p = ta.PagedQuantParams(4, 8, 2, d, c.q.shape[0], 60, 0, 16, c.cache[0].shape[0], c.table.shape[1], group, 2, c.scale)
    for polls in (0, 0, 1, 2, 4, 8):
        out = torch.full_like(c.q, 77.0)
        ta.ta_test_paged_quant_attn_fwd_wait_limit(polls, p, c.q, c.cache, c.table, cu, lens, parents, tmp, out)
        torch.cuda.synchronize()
        status = int(word[0])
        assert status == 1 if polls == 0 else status in (0, 1)
        assert status or torch.equal(out, want)
        word[0] = 0
        assert torch.equal(c.run(ta, kernel=2, tmp=tmp), want)
        assert int(word[0]) == 0
    with pytest.raises(ta.TreeAttentionError, match="tensor-core kernel only"):
        p.kernel = 1
        ta.ta_test_paged_quant_attn_fwd_wait_limit(0, p, c.q, c.cache, c.table, cu, lens, parents, tmp, out)
