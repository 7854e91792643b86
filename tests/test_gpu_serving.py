"""Batched serving operators (paged_plan, paged_append, paged_attention,
prompt_attention) on the GPU, against plain float64 restatements of their
definitions."""
import math
import random

import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
FAMILIES = [0, 1, 2, 3]


@pytest.fixture(scope="module")
def ta():
    import tree_masked_speculative_gb300 as m
    return m


# ---------------------------------------------------------------- references
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


def reference(q, keys, values, see, scale):
    """(out, attention of |v|) in float64 for one request: q [n, H, D],
    keys / values [length, Hk, D]; rows that see nothing give zeros."""
    n, h, d = q.shape
    g = h // keys.shape[1]
    out = torch.zeros(n, h, d, dtype=torch.float64, device=q.device)
    spread = torch.zeros_like(out)
    see = see.to(q.device)
    live = see.any(1)
    if not bool(live.any()):
        return out, spread
    for i in range(h):
        s = q[:, i].double() @ keys[:, i // g].double().T * scale
        s = torch.where(see, s, torch.full_like(s, -math.inf))
        w = torch.softmax(s[live], -1)
        v = values[:, i // g].double()
        # keys nobody sees do not count, whatever they hold
        v = torch.where(see.any(0)[:, None], v, torch.zeros_like(v))
        out[live, i] = w @ v
        spread[live, i] = w @ v.abs()
    return out, spread


def check(got, ref, spread, dtype, keys):
    """|got - ref| against the roundings of the kernels.

    eps / 2 |ref|      the output's own rounding
    eps / 2 spread     the weights P rounded once to 16 bits (|v| weighted by P)
    2^-12 spread       f32 work: a logit is off by at most D 2^-24 sum|q k| scale
                       (<= 256 x 6e-8 x 16 = 2.4e-4 here), its weight by as much
    f16: keys 2^-25 x max|v| (<= 8 here): weights below the f16 normal range
                       are off by half a subnormal step each, relative to a sum >= 1
    """
    half = torch.finfo(dtype).eps / 2
    tol = half * ref.abs() + (half + 2.0 ** -12) * spread + 1e-30
    if dtype == torch.float16:
        tol = tol + keys * 2.0 ** -25 * 8
    err = (got.double() - ref).abs()
    assert bool(torch.isfinite(got.double()).all()), "non-finite output"
    worst = (err - tol).max().item()
    assert worst <= 0, "off by %.3g over the tolerance (max err %.3g)" % (worst, err.max().item())


def randn(gen, *shape, dtype, std=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)


def offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Paged:
    """A paged cache filled for requests of `lens` keys, `new` of them new."""

    def __init__(self, lens, new, h, hk, d, ps, dtype, seed=0, pad=0, spare=3, nhd=False, tree=False, fill=None):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rnd = random.Random(seed)
        self.lens, self.new, self.h, self.hk, self.d, self.ps, self.dtype = lens, new, h, hk, d, ps, dtype
        self.scale = d ** -0.5
        need = [-(-n // ps) for n in lens]
        n_pages = sum(need) + spare
        shape = (n_pages, ps, hk, d) if nhd else (n_pages, hk, ps, d)
        full = float("nan") if fill is None else fill
        self.k = torch.full(shape, full, dtype=dtype, device="cuda")
        self.v = torch.full(shape, full, dtype=dtype, device="cuda")
        if nhd:
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        order = list(range(n_pages))
        rnd.shuffle(order)
        width = max(1, max(need)) + 1
        self.table = torch.full((len(lens), width), -7, dtype=torch.int32)
        self.keys, self.values = [], []
        at = 0
        for b, n in enumerate(lens):
            kk, vv = randn(g, n, hk, d, dtype=dtype), randn(g, n, hk, d, dtype=dtype)
            self.keys.append(kk)
            self.values.append(vv)
            for j in range(need[b]):
                page = order[at]
                at += 1
                self.table[b, j] = page
                m = min(ps, n - j * ps)
                self.k[page, :, :m] = kk[j * ps:j * ps + m].transpose(0, 1)
                self.v[page, :, :m] = vv[j * ps:j * ps + m].transpose(0, 1)
        self.table = self.table.cuda()
        self.cu = offsets(new)
        self.q = randn(g, self.cu[-1] + pad, h, d, dtype=dtype, std=2.0)
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
        return ta.paged_attention(self.q, self.k, self.v, self.table, i32(self.cu), i32(self.lens), **a)

    def expect(self, window=0):
        outs = []
        for b, (n, m) in enumerate(zip(self.lens, self.new)):
            see = visible(m, n, window, self.parents[b] if self.parents else None)
            outs.append(reference(self.q[self.cu[b]:self.cu[b + 1]], self.keys[b], self.values[b], see, self.scale))
        return torch.cat([o for o, _ in outs]), torch.cat([s for _, s in outs])

    def check(self, got, window=0, only=None):
        """All requests' rows, or those of the requests `only`."""
        ref, spread = self.expect(window)
        for b in range(len(self.lens)) if only is not None else ():
            s = slice(self.cu[b], self.cu[b + 1])
            if b in only:
                check(got[s], ref[s], spread[s], self.dtype, max(self.lens))
        if only is None:
            check(got[:self.cu[-1]], ref, spread, self.dtype, max(self.lens))


# -------------------------------------------------------------------- prompts
PROMPTS = [[1], [2, 0, 5], [200, 1, 33], [129, 127, 128, 64, 0, 0], [513], [70] * 9, [1000, 3]]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens", PROMPTS, ids=lambda x: "-".join(map(str, x))[:20])
@pytest.mark.parametrize("h,hk,d", [(4, 4, 64), (8, 2, 128), (6, 1, 128), (6, 2, 256), (12, 2, 64)])
def test_prompt(ta, lens, h, hk, d, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(len(lens) + d)
    t, cu, dt = sum(lens), offsets(lens), DT[dtype]
    q, k, v = (randn(g, t + 2, n, d, dtype=dt, std=s) for n, s in ((h, 2.0), (hk, 1.0), (hk, 1.0)))
    for kernel in (0, 1):
        for window in (0, 1, 37, 150):
            out = torch.full((t + 2, h, d), 5.0, dtype=dt, device="cuda")
            ta.prompt_attention(q, k, v, i32(cu), scale=d ** -0.5, window=window, out=out, kernel=kernel)
            assert bool((out[t:] == 5.0).all())
            for b, n in enumerate(lens):
                if n:
                    s = slice(cu[b], cu[b + 1])
                    ref, spread = reference(q[s], k[s], v[s], visible(n, n, window), d ** -0.5)
                    check(out[s], ref, spread, dt, n)


@pytest.mark.parametrize("h,hk,d,window", [(8, 2, 128, 0), (8, 2, 128, 1500), (3, 1, 256, 0), (2, 2, 64, 700)])
def test_long_prompt(ta, h, hk, d, window):
    """More row tiles than a warp has lanes, units cut between CTAs."""
    g = torch.Generator(device="cuda")
    g.manual_seed(d)
    lens = [4700, 0, 333]
    q, k, v = (randn(g, sum(lens), n, d, dtype=torch.bfloat16, std=s) for n, s in ((h, 2.0), (hk, 1.0), (hk, 1.0)))
    cu = offsets(lens)
    out = ta.prompt_attention(q, k, v, i32(cu), scale=d ** -0.5, window=window)
    for b, n in enumerate(lens):
        if n:
            s = slice(cu[b], cu[b + 1])
            i = torch.arange(n)
            see = (i[None] <= i[:, None]) & ((i[None] > i[:, None] - window) if window else True)
            ref, spread = reference(q[s], k[s], v[s], see, d ** -0.5)
            check(out[s], ref, spread, torch.bfloat16, n)


def test_many_short_prompts(ta):
    """More requests than a block has threads."""
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    rnd = random.Random(2)
    lens = [rnd.choice([0, 1, 2, 3, 9]) for _ in range(1300)]
    q, k, v = (randn(g, sum(lens), n, 64, dtype=torch.float16) for n in (4, 2, 2))
    out = ta.prompt_attention(q, k, v, i32(offsets(lens)), scale=0.125)
    want = ta.prompt_attention(q, k, v, i32(offsets(lens)), scale=0.125, kernel=1)
    # each side within half a step of its own value, plus P's rounding on values up to 5
    assert bool(((out - want).abs() <= 2.0 ** -10 * want.abs() + 5 * 2.0 ** -10).all())


@pytest.mark.parametrize("kernel", [0, 1, 2, 3])
def test_scales(ta, kernel):
    """A scale of zero weighs every visible key alike; a negative one turns the order."""
    g = torch.Generator(device="cuda")
    g.manual_seed(12)
    lens, h, hk, d = [90, 200], 4, 2, 128
    q, k, v = (randn(g, sum(lens), n, d, dtype=torch.bfloat16) for n in (h, hk, hk))
    cu = offsets(lens)
    for scale in (0.0, -0.2, 1e-30, 0.7):
        out = ta.prompt_attention(q, k, v, i32(cu), scale=scale, window=2 ** 31 - 1, kernel=kernel)
        for b, n in enumerate(lens):
            s = slice(cu[b], cu[b + 1])
            ref, spread = reference(q[s], k[s], v[s], visible(n, n), scale)
            # |scale| 0.7: sum |q k| scale is up to 8 times what check() allows for
            check(out[s], ref, spread * (1 + 2.0 ** -8), torch.bfloat16, n)
    c = Paged([300, 40], [1, 1], 8, 2, 128, 16, torch.bfloat16, seed=3)
    c.scale = -0.1
    c.check(c.run(ta, kernel=kernel))
    c.scale = 0.0
    c.check(c.run(ta, kernel=kernel))


def test_prompt_strides_of_a_fused_projection(ta):
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    lens, h, hk, d = [150, 40], 8, 2, 128
    qkv = randn(g, sum(lens), (h + 2 * hk) * d, dtype=torch.bfloat16).view(sum(lens), h + 2 * hk, d)
    q, k, v = qkv[:, :h], qkv[:, h:h + hk], qkv[:, h + hk:]
    out = torch.zeros(h, sum(lens), d, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    got = ta.prompt_attention(q, k, v, i32(offsets(lens)), scale=0.09, out=out)
    assert got is out
    want = ta.prompt_attention(q.contiguous(), k.contiguous(), v.contiguous(), i32(offsets(lens)), scale=0.09)
    assert torch.equal(out, want)


def test_prompt_neighbours_do_not_leak(ta):
    """NaN in another prompt's K and V, and in later rows of the same prompt's."""
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    lens, h, hk, d = [100, 60, 90], 4, 2, 128
    q, k, v = (randn(g, sum(lens), n, d, dtype=torch.float16) for n in (h, hk, hk))
    clean = ta.prompt_attention(q, k, v, i32(offsets(lens)), scale=0.1)
    for x in (k, v):
        x[:100], x[160:] = float("nan"), float("inf")
    x = ta.prompt_attention(q, k, v, i32(offsets(lens)), scale=0.1)
    assert torch.equal(x[100:160], clean[100:160])
    v2 = v.clone()
    v2[130, 1, 7] = float("nan")                    # row 30 of the middle prompt: seen from there on
    v2[141, 0, 3] = float("inf")
    x = ta.prompt_attention(q, k, v2, i32(offsets(lens)), scale=0.1)
    same = torch.ones(60, h, d, dtype=torch.bool, device="cuda")
    same[30:, 2:, 7] = False
    same[41:, :2, 3] = False
    assert torch.equal(x[100:160][same], clean[100:160][same])
    assert not bool(torch.isfinite(x[100:160][~same]).any())


# ---------------------------------------------------------------------- paged
@pytest.mark.parametrize("ps", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("h,hk,d", [(4, 4, 64), (8, 2, 128), (6, 2, 256), (16, 1, 128)])
def test_decode(ta, h, hk, d, dtype, ps):
    lens = [1, 700, 16, 33, 129, 0, 255, 1300]
    new = [1, 1, 1, 1, 1, 0, 1, 1]
    c = Paged(lens, new, h, hk, d, ps, DT[dtype], seed=ps + d)
    for kernel in FAMILIES:
        for window in (0, 1, 100):
            c.check(c.run(ta, kernel=kernel, window=window), window)


@pytest.mark.parametrize("h,hk,d,new,batch", [(4, 2, 64, 1, 700), (8, 2, 128, 2, 300), (2, 2, 128, 1, 2), (4, 1, 256, 20, 600)])
def test_many_or_long_requests(ta, h, hk, d, new, batch):
    """More requests than a block has threads; contexts cut into many pieces."""
    rnd = random.Random(batch)
    lens = [rnd.randint(new, 90) for _ in range(batch)] if batch > 2 else [30000, 9001]
    c = Paged(lens, [new if batch == 2 or rnd.random() < 0.9 else 0 for _ in lens], h, hk, d, 16, torch.bfloat16, seed=batch)
    got, want = c.run(ta), c.run(ta, kernel=1)
    # both within P's and the output's rounding of one value (values up to 6)
    assert bool(((got - want).abs() <= 2.0 ** -7 * want.abs() + 6 * 2.0 ** -8).all())
    if batch == 2:
        c.check(got)


@pytest.mark.parametrize("h,hk,d,ps,dtype,new", [
    (8, 2, 128, 16, "bf16", [4, 1, 3, 0, 2]), (8, 2, 128, 16, "f16", [2, 3, 4, 1, 4]),
    (8, 2, 128, 32, "bf16", [40, 1, 129, 0, 64]), (6, 1, 256, 64, "f16", [90, 2, 31, 0, 50]),
    (4, 4, 64, 16, "bf16", [300, 7, 1, 5, 128]), (32, 1, 128, 64, "bf16", [9, 1, 30, 2, 3]),
    (10, 2, 128, 128, "f16", [77, 1, 0, 0, 260]), (12, 4, 256, 16, "bf16", [5, 1, 4, 2, 3])])
def test_chunks(ta, h, hk, d, ps, dtype, new):
    lens = [x + n for x, n in zip([0, 900, 250, 0, 77], new)]
    c = Paged(lens, new, h, hk, d, ps, DT[dtype], seed=d + ps, pad=3)
    for kernel in FAMILIES:
        for window in (0, 5, 130):
            out = torch.full_like(c.q, 5.0)
            c.check(c.run(ta, kernel=kernel, window=window, out=out), window)
            assert bool((out[c.cu[-1]:] == 5.0).all())


@pytest.mark.parametrize("h,hk,d,ps,dtype,new", [
    (8, 2, 128, 16, "bf16", [4, 1, 3, 0, 2]), (8, 2, 128, 16, "bf16", [40, 1, 200, 0, 64]),
    (24, 4, 256, 64, "f16", [32, 32, 31, 0, 5]), (4, 4, 64, 32, "f16", [256, 7, 1, 5, 128]),
    (16, 2, 128, 128, "f16", [8, 16, 2, 1, 0])])
def test_trees(ta, h, hk, d, ps, dtype, new):
    lens = [x + n for x, n in zip([0, 900, 250, 0, 77], new)]
    c = Paged(lens, new, h, hk, d, ps, DT[dtype], seed=d + ps, pad=1, tree=True)
    for kernel in FAMILIES:
        c.check(c.run(ta, kernel=kernel))


@pytest.mark.parametrize("new", [1, 3, 60])
def test_tree_chain_is_causal(ta, new):
    c = Paged([500, 90], [new, new], 8, 2, 128, 32, torch.bfloat16, seed=5)
    chain = i32(([-1] + list(range(new - 1))) * 2)
    assert torch.equal(c.run(ta), c.run(ta, parents=chain))


@pytest.mark.parametrize("new", [1, 4, 70])
@pytest.mark.parametrize("kernel", FAMILIES)
def test_fewer_keys_than_tokens(ta, new, kernel):
    """kv_len < q_len: the first rows stand before position 0 and see nothing."""
    c = Paged([200, 200], [new, new], 8, 2, 128, 16, torch.float16, seed=6)
    short = max(0, new - 2)
    out = ta.paged_attention(c.q, c.k, c.v, c.table, i32(c.cu), i32([200, short]), scale=c.scale, max_q_len=new,
                             kernel=kernel)
    ref, spread = reference(c.q[new:], c.keys[1][:short], c.values[1][:short], visible(new, short), c.scale)
    check(out[new:], ref, spread, torch.float16, short + 1)
    assert bool((out[new:new + new - short] == 0).all())


@pytest.mark.parametrize("new", [1, 4, 70])
@pytest.mark.parametrize("kernel", FAMILIES)
def test_nhd_cache_and_strided_rows(ta, new, kernel):
    a = Paged([333, 64, new], [new] * 3, 8, 2, 128, 32, torch.bfloat16, seed=7)
    b = Paged([333, 64, new], [new] * 3, 8, 2, 128, 32, torch.bfloat16, seed=7, nhd=True)
    want = a.run(ta, kernel=kernel)
    wide = torch.zeros(a.q.shape[0], 11, 128, dtype=torch.bfloat16, device="cuda")
    wide[:, 1:9] = a.q
    b.q = wide[:, 1:9]
    out = torch.zeros(a.q.shape[0], 8, 256, dtype=torch.bfloat16, device="cuda")[:, :, 128:]
    assert torch.equal(b.run(ta, kernel=kernel, out=out), want)


@pytest.mark.parametrize("kernel", FAMILIES)
@pytest.mark.parametrize("new", [2, 5, 64])
def test_masked_keys_do_not_matter(ta, new, kernel):
    """Infinities and NaN in keys and values that a row does not see: behind the
    last key (every cache of this file), left of a window, later tokens, other
    branches of a draft tree."""
    for tree, window in ((False, 0), (False, 40), (True, 0)):
        c = Paged([300, 130], [new, new], 4, 1, 128, 16, torch.bfloat16, seed=8, tree=tree)
        clean = c.run(ta, window=window, kernel=kernel)
        assert bool(torch.isfinite(clean).all())
        j = 300 - 1                                              # the last new token of request 0
        page, off = int(c.table[0, j // 16]), j % 16
        c.v[page, 0, off, 5] = float("nan")
        c.v[page, 0, off, 77] = float("-inf")
        seen = visible(new, 300, window, c.parents[0] if tree else None)[:, j].cuda()
        if window:
            c.k[int(c.table[0, 0])] = float("nan")
            c.v[int(c.table[0, 0])] = float("inf")
            page = int(c.table[0, (300 - new - window) // 16])    # the page of the window's left edge
            for o in range(16):
                if (300 - new - window) // 16 * 16 + o <= 300 - new - window:
                    c.v[page, 0, o], c.k[page, 0, o] = float("nan"), float("nan")
        got = c.run(ta, window=window, kernel=kernel)
        keep = torch.ones_like(got, dtype=torch.bool)
        keep[:new][seen] = torch.tensor([d not in (5, 77) for d in range(128)], device="cuda")
        assert torch.equal(got[keep], clean[keep])
        assert not bool(torch.isfinite(got[~keep]).any())


@pytest.mark.parametrize("kernel", FAMILIES)
@pytest.mark.parametrize("new", [1, 60])
def test_masked_key_values_of_the_lowest_kind(ta, new, kernel):
    """K of unseen keys at the type's extremes: logits that overflow there stay there."""
    c = Paged([257, 30 + new], [new, new], 4, 2, 64, 16, torch.float16, seed=9)
    clean = c.run(ta, kernel=kernel)
    for b, n in enumerate(c.lens):
        page, off = int(c.table[b, n // 16]) if n % 16 else -1, n % 16
        if page >= 0:
            c.k[page, :, off:] = 65504.0
            c.v[page, :, off:] = -65504.0
    assert torch.equal(c.run(ta, kernel=kernel), clean)


@pytest.mark.parametrize("kernel", FAMILIES)
@pytest.mark.parametrize("new", [1, 40])
def test_bad_pages_set_the_status(ta, new, kernel):
    """Pages outside the cache are never read as addresses; other requests stand."""
    c = Paged([200, 100, 150], [new] * 3, 8, 2, 128, 16, torch.bfloat16, seed=10, fill=0.0)
    clean = c.run(ta, kernel=kernel)
    tmp = ta.paged_attention_workspace(c.q, c.k, c.table, max_q_len=new, kernel=kernel)
    got = c.run(ta, kernel=kernel, tmp=tmp)
    assert torch.equal(got, clean) and int(tmp.view(torch.int32)[0]) == 0
    for bad in (-1, c.k.shape[0], 2 ** 31 - 1, -2 ** 31):
        tmp.view(torch.int32)[0] = 0
        table = c.table.clone()
        table[1, 2] = bad
        c2 = c.table
        c.table = table
        got = c.run(ta, kernel=kernel, tmp=tmp)
        c.table = c2
        assert int(tmp.view(torch.int32)[0]) == 2
        assert torch.equal(got[:new], clean[:new]) and torch.equal(got[2 * new:], clean[2 * new:])


@pytest.mark.parametrize("kernel", FAMILIES)
@pytest.mark.parametrize("ps", [16, 32, 128])
@pytest.mark.parametrize("new", [1, 3, 200])
def test_pages_behind_the_window_may_be_gone(ta, new, ps, kernel):
    """Cells of pages that lie before every row's window hold no page of the cache."""
    c = Paged([900, 431, 5 + new], [new, max(new - 2, 1), new], 8, 2, 64, ps, torch.bfloat16, seed=17)
    window = 70
    for b, n in enumerate(c.lens):
        c.table[b, :max(0, n - c.new[b] - window + 1) // ps] = -1
    tmp = ta.paged_attention_workspace(c.q, c.k, c.table, max_q_len=new, kernel=kernel)
    c.check(c.run(ta, window=window, tmp=tmp, kernel=kernel), window)
    assert int(tmp.view(torch.int32)[0]) == 0



@pytest.mark.parametrize("kernel", FAMILIES)
@pytest.mark.parametrize("max_q", [4, 64])
def test_contradicting_lengths_set_the_status(ta, max_q, kernel):
    # (not the same bits as a call with sound lengths: where units are cut between CTAs, and so
    # the rounding, follows from all lengths of a batch)
    c = Paged([200, 100, 150], [4, 4, 4], 8, 2, 128, 16, torch.bfloat16, seed=11)

    def go(cu, lens):
        tmp = ta.paged_attention_workspace(c.q, c.k, c.table, max_q_len=max_q, kernel=kernel)
        out = torch.full_like(c.q, 5.0)
        ta.paged_attention(c.q, c.k, c.v, c.table, i32(cu), i32(lens), scale=c.scale, max_q_len=max_q, tmp=tmp,
                           out=out, kernel=kernel)
        return out, int(tmp.view(torch.int32)[0])

    out, st = go([0, 4, 8, 12], [200, -5, 150])
    assert st == 4 and bool((out[4:8] == 0).all())
    c.check(out, only=(0, 2))
    out, st = go([0, 4, 2 ** 30, 12], [200, 100, 150])        # runs past the rows, then backwards
    assert st & 4
    c.check(out, only=(0,))
    out, st = go([-3, 4, 8, 12], [200, 100, 150])
    assert st & 4
    c.check(out, only=(1, 2))
    # more keys than a table row holds
    out, st = go([0, 4, 8, 12], [200, 2 ** 31 - 1, 150])
    assert st & 4
    c.check(out, only=(0, 2))


def test_rows_past_max_q_len_are_left(ta):
    for max_q in (2, 40):
        c = Paged([200, 190], [50, 1], 8, 2, 128, 16, torch.bfloat16, seed=12)
        tmp = ta.paged_attention_workspace(c.q, c.k, c.table, max_q_len=max_q)
        out = torch.full_like(c.q, 5.0)
        c.run(ta, max_q_len=max_q, tmp=tmp, out=out)
        assert int(tmp.view(torch.int32)[0]) == 4
        assert bool((out[max_q:50] == 5.0).all())
        c.check(torch.cat([c.run(ta)[:50], out[50:]]))


@pytest.mark.parametrize("new", [1, 40])
def test_cache_beyond_32_bit_offsets(ta, new):
    """Pages whose element offsets pass 2^32."""
    ps, hk, d = 64, 8, 128
    n_pages = (1 << 32) // (ps * hk * d) + 40
    k = torch.empty(n_pages, hk, ps, d, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    c = Paged([300, 100], [new, new], 8, 8, d, ps, torch.bfloat16, seed=13)
    used = sorted({int(x) for x in c.table.flatten() if x >= 0})
    to = {p: n_pages - 1 - i for i, p in enumerate(used)}
    for p, n in to.items():
        k[n], v[n] = c.k[p], c.v[p]
    table = c.table.clone()
    for p, n in to.items():
        table[c.table == p] = n
    want = c.run(ta)
    c.k, c.v, c.table = k, v, table
    assert torch.equal(c.run(ta), want)
    rows = torch.ones(2, hk, d, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([n_pages * ps - 1, (n_pages - 30) * ps + 5], dtype=torch.int64, device="cuda")
    ta.paged_append(rows, rows * 2, k, v, slots)
    assert bool((k[-1, :, -1] == 1).all()) and bool((v[-30, :, 5] == 2).all())
    del k, v
    c.k = c.v = None
    torch.cuda.empty_cache()


@pytest.mark.parametrize("new", [1, 40])
def test_repeats_streams_and_graphs(ta, new):
    a = Paged([900, 77, 300], [new] * 3, 8, 2, 128, 16, torch.bfloat16, seed=14)
    b = Paged([40 + new, 500, 1000], [new] * 3, 8, 2, 128, 16, torch.bfloat16, seed=15)
    want_a, want_b = a.run(ta), b.run(ta)
    assert torch.equal(a.run(ta), want_a)                       # the same bits again
    s = torch.cuda.Stream()
    got = a.run(ta, stream=s)
    s.synchronize()
    assert torch.equal(got, want_a)
    # two graphs that share one workspace, replayed in turn on one stream; then
    # other lengths in the same buffers
    tmp = ta.paged_attention_workspace(a.q, a.k, a.table, max_q_len=new)
    graphs = []
    for c in (a, b):
        cu, lens, out = i32(c.cu), i32(c.lens), torch.empty_like(c.q)
        def call(c=c, cu=cu, lens=lens, out=out):
            ta.paged_attention(c.q, c.k, c.v, c.table, cu, lens, scale=c.scale, max_q_len=new, tmp=tmp, out=out)
        call()
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            call()
        graphs.append((gr, lens, out, cu))
    for _ in range(3):
        for gr, _, out, _ in graphs:
            out.zero_()
            gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][2], want_a) and torch.equal(graphs[1][2], want_b)
    fewer = [500, 50 + new // 2, 200]
    graphs[0][1].copy_(i32(fewer))
    graphs[0][0].replay()
    want = ta.paged_attention(a.q, a.k, a.v, a.table, i32(a.cu), i32(fewer), scale=a.scale, max_q_len=new)
    assert torch.equal(graphs[0][2], want)


@pytest.mark.parametrize("h,d", [(128, 64), (128, 256), (100, 128), (33, 256), (17, 64)])
@pytest.mark.parametrize("kernel", [0, 2])
def test_many_heads_of_one_kv_head(ta, h, d, kernel):
    """Units of one or a few tokens, rows that do not divide by the heads."""
    g = torch.Generator(device="cuda")
    g.manual_seed(h)
    lens = [1, 70, 0, 3, 131]
    cu = offsets(lens)
    q, k, v = (randn(g, cu[-1], n, d, dtype=torch.bfloat16, std=s) for n, s in ((h, 2.0), (1, 1.0), (1, 1.0)))
    out = ta.prompt_attention(q, k, v, i32(cu), scale=d ** -0.5, kernel=kernel)
    for b, n in enumerate(lens):
        r = slice(cu[b], cu[b + 1])
        if n:
            check(out[r], *reference(q[r], k[r], v[r], visible(n, n), d ** -0.5), torch.bfloat16, n)
    c = Paged([150, 64, 9], [1, 5, 9], h, 1, d, 32, torch.float16, seed=h, tree=True)
    c.check(c.run(ta, kernel=kernel))


@pytest.mark.parametrize("new", [1, 40])
def test_requests_that_share_pages(ta, new):
    """A common prefix: both requests' tables name the same pages."""
    c = Paged([320, 330], [new, new], 8, 2, 128, 32, torch.bfloat16, seed=18)
    shared = 256 // 32
    c.table[1, :shared] = c.table[0, :shared]
    c.keys[1][:256], c.values[1][:256] = c.keys[0][:256], c.values[0][:256]
    c.check(c.run(ta))


@pytest.mark.parametrize("new", [1, 5, 90])
def test_two_streams_at_once(ta, new):
    cs = [Paged([2000, 77 + new, 300], [new] * 3, 8, 2, 128, 16, torch.bfloat16, seed=19 + i) for i in range(2)]
    want = [c.run(ta) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    tmps = [ta.paged_attention_workspace(c.q, c.k, c.table, max_q_len=new) for c in cs]
    rows, lens = [i32(c.cu) for c in cs], [i32(c.lens) for c in cs]
    torch.cuda.synchronize()
    got = [[ta.paged_attention(c.q, c.k, c.v, c.table, rows[i], lens[i], scale=c.scale, max_q_len=new, tmp=tmps[i],
                               stream=streams[i]) for i, c in enumerate(cs)] for _ in range(20)]
    torch.cuda.synchronize()
    for pair in got:
        assert all(torch.equal(x, y) for x, y in zip(pair, want))
    assert not any(int(tmp.view(torch.int32)[0]) for tmp in tmps)


# ----------------------------------------------------------------- append
@pytest.mark.parametrize("hk,d,ps,t,nhd", [(8, 128, 16, 1, False), (1, 64, 16, 77, True), (4, 256, 64, 500, False),
                                           (3, 128, 256, 1000, True)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_append(ta, hk, d, ps, t, nhd, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(t)
    n_pages = -(-t // ps) + 4
    shape = (n_pages, ps, hk, d) if nhd else (n_pages, hk, ps, d)
    k, v = (randn(g, *shape, dtype=DT[dtype]) for _ in range(2))
    if nhd:
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    both = randn(g, t, 2 * hk + 1, d, dtype=DT[dtype])
    kn, vn = both[:, :hk], both[:, hk:2 * hk]
    slots = torch.randperm(n_pages * ps, generator=g, device="cuda")[:t]
    slots[::7] = -1
    slots[3::11] = n_pages * ps
    if t > 20:
        slots[20] = 2 ** 62
    want_k, want_v = k.clone(), v.clone()
    for i, s in enumerate(slots.tolist()):
        if 0 <= s < n_pages * ps:
            want_k[s // ps, :, s % ps], want_v[s // ps, :, s % ps] = kn[i], vn[i]
    ta.paged_append(kn, vn, k, v, slots)
    assert torch.equal(k, want_k) and torch.equal(v, want_v)
    ta.paged_append(kn[:0], vn[:0], k, v, slots[:0])
    assert torch.equal(k, want_k)


# ------------------------------------------------------------------- planning
def plan_reference(keep, new, held, table, stack, n_free, ps, max_tokens):
    """The definition, cell by cell; None when the step does not fit."""
    table, stack = [list(r) for r in table], list(stack)
    need = [-(-(a + b) // ps) for a, b in zip(keep, new)]
    top = n_free
    for b, h in enumerate(held):
        for j in range(need[b], h):
            if top >= len(stack):
                return None
            stack[top] = table[b][j]
            top += 1
    for b, h in enumerate(held):
        for j in range(h, need[b]):
            if top == 0 or j >= len(table[b]):
                return None
            top -= 1
            table[b][j] = stack[top]
    if sum(new) > max_tokens:
        return None
    slot, pos = [], []
    for b in range(len(keep)):
        for p in range(keep[b], keep[b] + new[b]):
            slot.append(table[b][p // ps] * ps + p % ps)
            pos.append(p)
    rest = [-1] * (max_tokens - len(slot))
    return table, stack, need, top, offsets(new), [a + b for a, b in zip(keep, new)], slot + rest, pos + rest


def make_plan(rnd, batch, ps, width, most_new, pad=5):
    pages = list(range(batch * width + 20))
    rnd.shuffle(pages)
    table, held, keep, new, at = [], [], [], [], 0
    for b in range(batch):
        h = rnd.randint(0, width)
        table.append(pages[at:at + h] + [-9] * (width - h))
        at += h
        held.append(h)
        keep.append(rnd.randint(max(0, h * ps - 2 * ps), h * ps) if rnd.random() < 0.8 else 0)
        new.append(rnd.randint(0, min(most_new, width * ps - keep[-1])))
    free = pages[at:]
    return keep, new, held, table, free + [-9] * (len(pages) - len(free)), len(free), sum(new) + pad


@pytest.mark.parametrize("batch,ps,width,most", [(1, 16, 3, 1), (7, 16, 9, 40), (513, 16, 8, 2), (300, 64, 12, 300),
                                                (1500, 32, 5, 1), (16384, 16, 2, 1), (40, 256, 30, 2000)])
def test_plan(ta, batch, ps, width, most):
    rnd = random.Random(batch)
    for alias in (False, True):
        keep, new, held, table, stack, n_free, rows = make_plan(rnd, batch, ps, width, most)
        want = plan_reference(keep, new, held, table, stack, n_free, ps, rows)
        t, s, h, n = i32(table), i32(stack), i32(held), i32([n_free])
        e = lambda k, dt=torch.int32: torch.full((k,), 77, dtype=dt, device="cuda")
        out = (h if alias else e(batch), n if alias else e(1), e(batch + 1), e(batch), e(rows, torch.int64), e(rows),
               torch.zeros(1, dtype=torch.int32, device="cuda"))
        got = ta.paged_plan(i32(keep), i32(new), h, t, s, n, page_size=ps, max_tokens=rows, out=out)
        assert int(got.status) == 0 and want is not None
        for x, y in zip((t, s, got.held, got.n_free, got.cu_q, got.kv_lens, got.slot_map, got.positions), want):
            assert torch.equal(x.cpu().long(), torch.tensor(y).reshape(x.shape))


@pytest.mark.parametrize("what,bit", [("pages", 1), ("negative", 2), ("width", 2), ("held", 2), ("tokens", 4),
                                      ("stack", 8), ("n_free", 8), ("overflow", 2)])
@pytest.mark.parametrize("batch", [6, 600])
def test_plan_refuses_as_a_whole(ta, what, bit, batch):
    rnd = random.Random(5)
    keep, new, held, table, stack, n_free, rows = make_plan(rnd, batch, 16, 6, 30)
    if what == "pages":
        keep, new, held, n_free = [0] * batch, [30] * batch, [0] * batch, 2 * batch - 1
        stack, rows = [1] * (2 * batch), 30 * batch
    elif what == "negative":
        new[3] = -1
    elif what == "width":
        keep[2], new[2] = 6 * 16 - 1, 2
    elif what == "held":
        held[1] = 7
    elif what == "tokens":
        rows = sum(new) - 1
    elif what == "stack":
        keep, new, held, n_free = [0] * batch, [0] * batch, [1] * batch, len(stack) - batch + 1
    elif what == "n_free":
        n_free = len(stack) + 1
    else:
        keep[0], new[0] = 2 ** 31 - 1, 2 ** 31 - 1
    t, s = i32(table), i32(stack)
    got = ta.paged_plan(i32(keep), i32(new), i32(held), t, s, i32([n_free]), page_size=16, max_tokens=rows)
    assert int(got.status) & bit
    assert torch.equal(t.cpu(), torch.tensor(table, dtype=torch.int32)) and torch.equal(s.cpu(), torch.tensor(stack, dtype=torch.int32))
    assert got.held.tolist() == held and int(got.n_free) == n_free
    assert not bool(got.cu_q.any()) and not bool(got.kv_lens.any())
    assert bool((got.slot_map == -1).all()) and bool((got.positions == -1).all())


# ------------------------------------------------------------- all of them together
@pytest.mark.parametrize("d,h,hk,ps,dtype", [(128, 8, 2, 16, "bf16"), (64, 4, 4, 32, "f16"), (256, 6, 1, 64, "f16")])
def test_a_serving_run(ta, d, h, hk, ps, dtype):
    """Requests come, grow by prompts, chunks, single tokens and draft trees,
    lose rejected drafts and end; after every step the paged attention equals
    the definition on each request's whole history."""
    g = torch.Generator(device="cuda")
    g.manual_seed(d)
    rnd = random.Random(d)
    dt, batch, width = DT[dtype], 5, 24
    n_pages = batch * width * 2 // 3
    kc, vc = (torch.full((n_pages, hk, ps, d), float("nan"), dtype=dt, device="cuda") for _ in range(2))
    table = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
    stack, n_free = torch.randperm(n_pages, device="cuda").to(torch.int32), i32([n_pages])
    held = i32([0] * batch)
    hist = [[torch.zeros(0, hk, d, dtype=dt, device="cuda")] * 2 for _ in range(batch)]
    for step, kind in enumerate(["prompt", "decode", "chunk", "tree", "decode", "end", "prompt", "tree", "decode"]):
        keep = [x[0].shape[0] for x in hist]
        if kind == "tree" or step and rnd.random() < 0.5:
            keep = [max(0, n - rnd.randint(0, 3)) for n in keep]          # rejected drafts
        if kind in ("prompt", "end"):
            keep = [n if rnd.random() < 0.5 else 0 for n in keep]
        most = {"prompt": 100, "decode": 1, "chunk": 60, "tree": 30, "end": 0}[kind]
        new = [rnd.randint(min(1, most), most) for _ in keep]
        rows = sum(new)
        q, kn, vn = (randn(g, rows, n, d, dtype=dt) for n in (h, hk, hk))
        plan = ta.paged_plan(i32(keep), i32(new), held, table, stack, n_free, page_size=ps, max_tokens=rows,
                             out=(held, n_free, i32([0] * (batch + 1)), i32([0] * batch),
                                  torch.empty(rows, dtype=torch.int64, device="cuda"), i32([0] * rows), i32([0])))
        assert int(plan.status) == 0
        assert int(plan.n_free) + int(plan.held.sum()) == n_pages
        ta.paged_append(kn, vn, kc, vc, plan.slot_map)
        parents = [[rnd.randrange(0, i) if i else -1 for i in range(n)] for n in new] if kind == "tree" else None
        flat = i32([p for r in parents for p in r]) if parents else None
        out = ta.paged_attention(q, kc, vc, table, plan.cu_q, plan.kv_lens, scale=d ** -0.5,
                                 max_q_len=max(1, most), parents=flat)
        cu = offsets(new)
        fresh = kind == "prompt" and not any(keep)
        if fresh:
            other = ta.prompt_attention(q, kn, vn, plan.cu_q, scale=d ** -0.5)
        for b in range(batch):
            s = slice(cu[b], cu[b + 1])
            hist[b] = [torch.cat([x[:keep[b]], y[s]]) for x, y in zip(hist[b], (kn, vn))]
            if not new[b]:
                continue
            see = visible(new[b], keep[b] + new[b], 0, parents[b] if parents else None)
            ref, spread = reference(q[s], hist[b][0], hist[b][1], see, d ** -0.5)
            check(out[s], ref, spread, dt, keep[b] + new[b])
            if fresh:
                check(other[s], ref, spread, dt, new[b])


# ----------------------------------------------------- values that are not finite
NAN_KEYS = [1, 17, 300]                      # one key; one alone in its block of 16; many blocks


def nan_rows(clean, got, hit):
    """Exactly the rows `hit` ([T, H] bool) are NaN, the others have the clean bits."""
    hit = hit.cuda()
    assert bool(torch.isfinite(clean).all())
    assert bool(torch.isnan(got[hit]).all()), "a NaN logit was lost"
    assert torch.equal(got[~hit], clean[~hit])


@pytest.mark.parametrize("keys", NAN_KEYS)
@pytest.mark.parametrize("new", [1, 3, 40])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kernel", [0, 2, 3])
def test_nan_logits_reach_the_rows_that_see_them(ta, kernel, d, new, keys):
    """A NaN in a row's query, or in K of a key that it sees (the first, one in the middle, the last of
    the prefix, the last of all), makes the whole row NaN."""
    nan_case(ta, kernel, d, new, keys)


def nan_case(ta, kernel, d, new, keys):
    h, hk = 8, 2
    c = Paged([keys + new - 1, 90 + new], [new, new], h, hk, d, 16, torch.bfloat16, seed=21)
    for window in (0, 20):
        clean = c.run(ta, kernel=kernel, window=window)
        q = c.q.clone()
        c.q[new - 1, 5, 3] = float("nan")
        hit = torch.zeros(2 * new, h, dtype=torch.bool)
        hit[new - 1, 5] = True
        nan_rows(clean, c.run(ta, kernel=kernel, window=window), hit)
        c.q = q
        see = visible(new, c.lens[0], window)
        for j in sorted({0, c.lens[0] // 2, keys - 1, c.lens[0] - 1}):
            page, off = int(c.table[0, j // 16]), j % 16
            was = c.k[page, 1, off, 2].clone()
            c.k[page, 1, off, 2] = float("nan")
            hit = torch.zeros(2 * new, h, dtype=torch.bool)
            hit[:new, 4:] = see[:, j, None]
            nan_rows(clean, c.run(ta, kernel=kernel, window=window), hit)
            c.k[page, 1, off, 2] = was


@pytest.mark.parametrize("lens", [[1, 5], [17, 3], [300, 40]])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_nan_logits_of_prompts(ta, d, lens):
    nan_prompt(ta, 0, d, lens)


def nan_prompt(ta, kernel, d, lens):
    g = torch.Generator(device="cuda")
    g.manual_seed(22)
    t, h, hk, cu = sum(lens), 4, 2, i32(offsets(lens))
    q, k, v = (randn(g, t, n, d, dtype=torch.float16) for n in (h, hk, hk))
    clean = ta.prompt_attention(q, k, v, cu, scale=0.1, kernel=kernel)
    n = lens[0]
    for j in sorted({0, n // 2, n - 1}):
        for what in "qk":
            q2, k2 = q.clone(), k.clone()
            hit = torch.zeros(t, h, dtype=torch.bool)
            if what == "q":
                q2[j, 1, 0] = float("nan")
                hit[j, 1] = True
            else:
                k2[j, 1, 7] = float("nan")
                hit[j:n, 2:] = True
            nan_rows(clean, ta.prompt_attention(q2, k2, v, cu, scale=0.1, kernel=kernel), hit)


@pytest.mark.parametrize("keys", NAN_KEYS)
@pytest.mark.parametrize("new", [1, 3, 40])
@pytest.mark.parametrize("d", [64, 256])
def test_nan_logits_on_the_cuda_cores(ta, d, new, keys):
    """The same wherever the NaN stands among a row's keys, the first included."""
    nan_case(ta, 1, d, new, keys)


@pytest.mark.parametrize("lens", [[1, 5], [17, 3], [300, 40]])
def test_nan_logits_of_prompts_on_the_cuda_cores(ta, lens):
    nan_prompt(ta, 1, 128, lens)


# a contradiction that no row of q belongs to
@pytest.mark.parametrize("kernel", FAMILIES)
@pytest.mark.parametrize("max_q", [4, 64])
@pytest.mark.parametrize("cu,lens", [([0, 4, 4, 12], [200, -5, 150]), ([0, 4, 4, 12], [200, 2 ** 30, 150]),
                                     ([0, 8, 4, 12], [200, 100, 150])])
def test_contradictions_without_rows_set_the_status(ta, cu, lens, max_q, kernel):
    c = Paged([200, 100, 150], [4, 4, 4], 8, 2, 128, 16, torch.bfloat16, seed=11)
    tmp = ta.paged_attention_workspace(c.q, c.k, c.table, max_q_len=max_q, kernel=kernel)
    ta.paged_attention(c.q, c.k, c.v, c.table, i32(cu), i32(lens), scale=c.scale, max_q_len=max_q, tmp=tmp, kernel=kernel)
    assert int(tmp.view(torch.int32)[0]) == 4


def test_contradictions_of_more_requests_than_rows_set_the_status(ta):
    """The last of 5000 requests, on a call of one row."""
    c = Paged([20], [1], 1, 1, 64, 16, torch.bfloat16, seed=23)
    table = c.table[:1].expand(5000, -1).contiguous()
    for kernel in FAMILIES:
        tmp = ta.paged_attention_workspace(c.q, c.k, table, max_q_len=1, kernel=kernel)
        ta.paged_attention(c.q, c.k, c.v, table, i32([0] + [1] * 5000), i32([20] + [0] * 4998 + [-1]), scale=1.0, max_q_len=1,
                           tmp=tmp, kernel=kernel)
        assert int(tmp.view(torch.int32)[0]) == 4


# --------------------------------------------------------------- small weights
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("new,kernel", [(1, 0), (2, 1), (1, 2), (40, 0)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_many_small_weights_beside_a_large_one(ta, d, new, kernel, dtype):
    """One key takes almost all the weight, thousands have about 2^-25 of it each and the values
    that count.  The tolerance of check() but for its last term: with P held 2^7 higher an f16
    weight below the normal range is off by 2^-25 (half a subnormal step) 2^-7 = 2^-32."""
    dt, n, batch, hk = DT[dtype], 6000, 32, 2
    g = torch.Generator(device="cuda")
    g.manual_seed(24)
    ps = 64
    pages = -(-n // ps)
    k = torch.zeros(pages, hk, ps, d, dtype=dt, device="cuda")
    v = torch.zeros(pages, hk, ps, d, dtype=dt, device="cuda")
    # logits 8 k: 8 for key 0, 17.4 to 17.8 lower (2^-25.1 to 2^-25.7) for the others
    k[..., 0] = (-1.175 - 0.05 * torch.rand(pages, hk, ps, generator=g, device="cuda")).to(dt)
    v.copy_(torch.rand(v.shape, generator=g, device="cuda") * 32 + 32)
    k[0, :, 0, 0], v[0, :, 0] = 1.0, 0.0
    q = torch.zeros(batch * new, hk, d, dtype=dt, device="cuda")
    q[..., 0] = 8.0
    table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(batch, -1).contiguous()
    out = ta.paged_attention(q, k, v, table, i32([new * b for b in range(batch + 1)]), i32([n] * batch), scale=1.0,
                             max_q_len=new, kernel=kernel)
    keys, values = (x.transpose(1, 2).reshape(-1, hk, d)[:n] for x in (k, v))
    ref, spread = reference(q[:new], keys, values, visible(new, n), 1.0)
    half = torch.finfo(dt).eps / 2
    tol = half * ref.abs() + (half + 2.0 ** -12) * spread + (n * 2.0 ** -32 * 64 if dtype == "f16" else 0)
    # the output's own subnormal steps (f16, below 2^-14)
    tol = tol + 2.0 ** -25
    err = (out.view(batch, new, hk, d).double() - ref).abs()
    assert bool((err <= tol).all()), "off by %.3g, values around %.3g" % (err.max().item(), ref.mean().item())


# ------------------------------------------------------------------ streams, arguments
def test_stream_handle_zero_is_the_default_stream(ta):
    """0 is the handle of the default stream, not a request for a stream of its own."""
    c = Paged([300, 40], [3, 3], 8, 2, 128, 16, torch.bfloat16, seed=25)
    want = c.run(ta)
    q, tmp, out = c.q, ta.paged_attention_workspace(c.q, c.k, c.table, max_q_len=3), torch.zeros_like(c.q)
    cu, lens = i32(c.cu), i32(c.lens)
    late, side = torch.zeros_like(q), torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)                 # the default stream is about 10 ms behind
    late.copy_(q)
    with torch.cuda.stream(side):
        ta.paged_attention(late, c.k, c.v, c.table, cu, lens, scale=c.scale, max_q_len=3, tmp=tmp, out=out, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert torch.cuda.default_stream().cuda_stream == 0


def test_parents_of_no_token_are_refused(ta):
    """An empty or too short `parents` is an error, not the causal rule."""
    c = Paged([300, 40], [3, 3], 8, 2, 128, 16, torch.bfloat16, seed=26, tree=True)
    for bad in (torch.empty(0, dtype=torch.int32, device="cuda"), c.flat_parents()[:5]):
        with pytest.raises((ValueError, ta.TreeAttentionError), match="parents"):
            c.run(ta, parents=bad)


def test_workspaces_of_windowed_calls(ta):
    """A call whose work is in range only with its window has a workspace of that window."""
    t = 2 ** 23
    q = torch.empty(t, 2, 64, dtype=torch.float16, device="cuda")
    with pytest.raises(ta.TreeAttentionError, match="tokens x keys"):
        ta.prompt_attention_workspace(q, q, i32([0, t]))
    assert ta.prompt_attention_workspace(q, q, i32([0, t]), window=4096).numel() > 64
    k = torch.empty(4, 2, 256, 64, dtype=torch.float16, device="cuda")
    table = torch.zeros(1, 2 ** 20, dtype=torch.int32, device="cuda")
    with pytest.raises(ta.TreeAttentionError, match="tokens x keys"):
        ta.paged_attention_workspace(q, k, table, max_q_len=t)
    assert ta.paged_attention_workspace(q, k, table, max_q_len=t, window=4096).numel() > 64


# ------------------------------------------------------------- waits that give up
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_waits_that_give_up_set_the_status(ta, d, tree):
    """Every wait bounded by a few polls: CTAs give up at different places, let their copies and
    products end, say so in the status word and return; the next call on the same workspace is right."""
    c = Paged([900, 60, 3000, 61], [60, 60, 33, 7], 8, 2, d, 16, torch.bfloat16, seed=27, tree=tree)
    want = c.run(ta, kernel=2)
    tmp = ta.paged_attention_workspace(c.q, c.k, c.table, max_q_len=60, kernel=2)
    word = tmp.view(torch.int32)
    cu, lens, parents = i32(c.cu), i32(c.lens), c.flat_parents()
    p = ta.PagedParams(4, 8, 2, d, c.q.shape[0], 60, 0, 16, c.k.shape[0], c.table.shape[1], 2, c.scale)
    for polls in (0, 0, 1, 2, 4, 8):
        out = torch.zeros_like(c.q)
        ta.ta_test_paged_attn_fwd_wait_limit(polls, p, c.q, c.k, c.v, c.table, cu, lens, parents, tmp, out)
        torch.cuda.synchronize()
        status = int(word[0])
        assert status == 1 if polls == 0 else status in (0, 1)
        assert status or torch.equal(out, want)
        word[0] = 0
        assert torch.equal(c.run(ta, kernel=2, tmp=tmp), want)
        assert int(word[0]) == 0
    with pytest.raises(ta.TreeAttentionError, match="tensor-core kernel only"):
        p.kernel = 1
        ta.ta_test_paged_attn_fwd_wait_limit(0, p, c.q, c.k, c.v, c.table, cu, lens, parents, tmp, out)


# ------------------------------------------------------------------ odd trees
@pytest.mark.parametrize("kernel", FAMILIES)
@pytest.mark.parametrize("new", [2, 4, 70])
def test_trees_of_fewer_keys_than_tokens(ta, new, kernel):
    """kv_len < q_len with parents: nodes before position 0 are no keys, and give zeros."""
    c = Paged([200, 200], [new, new], 8, 2, 128, 16, torch.float16, seed=28, tree=True)
    for short in sorted({0, 1, new - 1, new // 2}):
        out = ta.paged_attention(c.q, c.k, c.v, c.table, i32(c.cu), i32([200, short]), scale=c.scale, max_q_len=new,
                                 parents=c.flat_parents(), kernel=kernel)
        see = visible(new, 200, 0, c.parents[1])[:, 200 - short:]
        ref, spread = reference(c.q[new:], c.keys[1][:short], c.values[1][:short], see, c.scale)
        check(out[new:], ref, spread, torch.float16, short + 1)
        assert bool((out[new:][~see.any(1)] == 0).all())


@pytest.mark.parametrize("kernel", FAMILIES)
@pytest.mark.parametrize("new", [4, 70])
def test_parents_outside_their_node_end_the_chain(ta, new, kernel):
    """Itself, a later node, a value past every node or far below: each is the end of the chain."""
    c = Paged([300, 90], [new, new], 8, 2, 64, 32, torch.bfloat16, seed=29, tree=True)
    for odd in (lambda i: i, lambda i: i + 1, lambda i: 2 ** 31 - 1, lambda i: -2 ** 31, lambda i: new):
        c.parents = [[odd(i) if i % 3 == 0 else i - 1 for i in range(new)] for _ in c.new]
        c.check(c.run(ta, kernel=kernel))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 3, 40])
def test_a_workspace_serves_other_batches(ta, d, new):
    """The tmp of one request takes the calls of twenty, and the other way round."""
    one, many = (Paged([90 + 7 * i for i in range(b)], [new] * b, 4, 2, d, 16, torch.bfloat16, seed=30 + b) for b in (1, 20))
    tmps = [ta.paged_attention_workspace(c.q, c.k, c.table, max_q_len=new) for c in (one, many)]
    for c in (one, many):
        for tmp in tmps:
            c.check(c.run(ta, tmp=tmp))
            assert int(tmp.view(torch.int32)[0]) == 0
