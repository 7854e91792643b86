"""Operators of a serving step on rotated keys and a 4-bit paged K/V cache: what is
computed, on which sizes, and what each pass cannot do without.

rotary   the step's queries and keys turned by their positions, K/V rows written to 16-bit pages
append   the same into 4-bit pages: groups of elements as codes with a scale and a bias; a pass
         reads the cache back, since codes are compared as the values they stand for
attend   attention of every request's new tokens (one token, a chunk or a draft tree) over its
         4-bit pages

4-bit pages: value = scale * code + bias of its group of 32 or 64 elements.  A token's row of
a KV head is D / 8 words of 32 bits: 16-bit quads (4 elements, lowest nibble first), quad g of
32-element block j at place g * (D / 32) + j.  Scale and bias stand side by side in the cache's
16-bit type, [pages, Hk, page, D / group, 2].

Plain forms are elementary torch operations in 32 bits, in 64 where a code is rounded;
``exact`` restates the definitions in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # one layer of a decode step of 64 requests: latency
        dict(name="rotary step 64", op="rotary", tokens=64, hq=32, hk=8, dim=128, rot=128, inter=0, page=16,
             dtype="bf16", far=32768),
        # a large prompt batch, odd count, half of each head turned, neighbours paired: bandwidth
        dict(name="rotary prompts 16k", op="rotary", tokens=16381, hq=24, hk=4, dim=256, rot=128, inter=1, page=64,
             dtype="f16", far=131072),
        # one layer of a decode step of 48 requests into 4 bits: latency
        dict(name="append step 48", op="append", tokens=48, hq=32, hk=8, dim=128, rot=128, inter=0, page=16, group=64,
             dtype="bf16", far=32768),
        # a prompt batch into 4 bits, odd count
        dict(name="append prompts 16k", op="append", tokens=16381, hq=32, hk=8, dim=128, rot=128, inter=0, page=32,
             group=32, dtype="f16", far=32768),
        # three requests decoding one token each on short contexts: latency
        dict(name="decode 3", op="attend", batch=3, hq=32, hk=8, dim=128, page=16, group=64, dtype="bf16", ctx_lo=200,
             ctx_hi=2100, new_lo=1, new_hi=1, window=0, tree=0, pad=0, lens=21),
        # a full decode batch on ragged contexts: bandwidth
        dict(name="decode 64", op="attend", batch=64, hq=32, hk=8, dim=128, page=16, group=64, dtype="bf16",
             ctx_lo=900, ctx_hi=16384, new_lo=1, new_hi=1, window=0, tree=0, pad=0, lens=22),
        # one very long context: its keys have to be shared out over the whole GPU
        dict(name="decode long", op="attend", batch=1, hq=24, hk=4, dim=256, page=64, group=32, dtype="f16",
             ctx_lo=131001, ctx_hi=131001, new_lo=1, new_hi=1, window=0, tree=0, pad=0, lens=23),
        # one KV head per query head, one to three tokens of many requests, sliding window, small groups
        dict(name="decode heads 64", op="attend", batch=96, hq=16, hk=16, dim=64, page=32, group=32, dtype="f16",
             ctx_lo=100, ctx_hi=6000, new_lo=1, new_hi=3, window=2000, tree=0, pad=3, lens=24),
        # small draft trees, a handful of rows per KV head
        dict(name="drafts 16", op="attend", batch=16, hq=32, hk=8, dim=128, page=16, group=32, dtype="bf16",
             ctx_lo=300, ctx_hi=9000, new_lo=5, new_hi=7, window=0, tree=1, pad=0, lens=25),
        # draft trees of 32 nodes of eight requests (the fixed-tree configuration's heads), contexts around 4096
        dict(name="verify trees 8", op="attend", batch=8, hq=24, hk=4, dim=256, page=64, group=64, dtype="f16",
             ctx_lo=2500, ctx_hi=4096, new_lo=32, new_hi=32, window=0, tree=1, pad=0, lens=26),
        # prompt chunks of up to 512 tokens of twelve requests over what they have cached
        dict(name="chunks 12", op="attend", batch=12, hq=32, hk=8, dim=128, page=32, group=64, dtype="bf16",
             ctx_lo=0, ctx_hi=8192, new_lo=1, new_hi=512, window=0, tree=0, pad=5, lens=27),
        # two long chunks with a sliding window, six query heads per KV head, head dimension 256
        dict(name="chunks window 256", op="attend", batch=2, hq=24, hk=4, dim=256, page=128, group=32, dtype="f16",
             ctx_lo=3000, ctx_hi=7000, new_lo=1000, new_hi=2047, window=1500, tree=0, pad=0, lens=28),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.99)))))))


def draw(rng):
    case = _draw(rng)
    # no drawn case costs more than the largest listed ones
    while case["op"] == "attend" and case["batch"] > 1 and (
            work(case)["flops"] > 2e11 or work(case)["bytes"] > 5e8):
        case["batch"] = (case["batch"] + 1) // 2
    return case


def _draw(rng):
    op = rng.choice(["rotary", "append", "append", "attend", "attend", "attend", "attend"])
    dtype, page = rng.choice(["f16", "bf16"]), rng.choice([16, 32, 64, 128])
    hk, dim = rng.choice([(8, 128), (4, 128), (8, 64), (4, 256)])
    hq = hk * rng.choice([1, 2, 3, 4, 6, 8] if hk == 4 else [1, 2, 4])
    if op != "attend":
        case = dict(op=op, tokens=_log(rng, 1, 16000), hq=rng.choice([hq, hq, 0]) if op == "append" else hq, hk=hk,
                    dim=dim, rot=rng.choice([dim, dim // 2, 16 * rng.randint(1, dim // 16)]), inter=rng.randrange(2),
                    page=page, dtype=dtype, far=_log(rng, 1000, 131072))
        if op == "append":
            case["group"] = rng.choice([32, 64])
            if rng.random() < 0.3:
                case.update(rot=0, hq=0)             # plain keys
        while case["tokens"] * case["dim"] * (2 * case["hq"] + 5 * case["hk"]) > 16381 * 256 * 68:
            case["tokens"] = (case["tokens"] + 1) // 2
        return case
    lens, group = rng.randrange(100, 1 << 30), rng.choice([32, 64])
    base = dict(op=op, hq=hq, hk=hk, dim=dim, page=page, group=group, dtype=dtype, ctx_lo=0, lens=lens)
    kind = rng.choice(["decode", "decode", "chunk", "tree"])
    if kind == "decode":
        ctx_hi = _log(rng, 32, 60000)
        return dict(base, batch=_log(rng, 1, 96), ctx_hi=ctx_hi, new_lo=1, new_hi=rng.choice([1, 1, 2, 3]),
                    window=rng.choice([0, 0, 1 + ctx_hi // 3]), tree=0, pad=rng.randrange(0, 4))
    if kind == "chunk":
        ctx_hi = _log(rng, 64, 8000)
        return dict(base, batch=_log(rng, 1, 8), ctx_hi=ctx_hi, new_lo=0, new_hi=_log(rng, 16, 500),
                    window=rng.choice([0, 0, 1 + ctx_hi // 3]), tree=0, pad=rng.randrange(0, 9))
    return dict(base, batch=_log(rng, 1, 10), ctx_hi=_log(rng, 64, 8000), new_lo=1, new_hi=_log(rng, 4, 100),
                window=0, tree=1, pad=rng.randrange(0, 4))


def _lengths(case):
    """Host lists of the case's lengths: (context tokens, new tokens).  They belong
    to the case, not to the seed, so that its work is known."""
    r = random.Random(case["lens"])
    n = case["batch"]
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(n)]
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(n)]
    ctx[-1], new[-1] = case["ctx_hi"], max(1, case["new_hi"])
    return ctx, new


def _pairs(ctx, new, window):
    """Visible (token, key) pairs of a causal chunk behind ctx tokens."""
    if not window:
        return new * ctx + new * (new + 1) // 2
    return sum(min(ctx + i + 1, window) for i in range(new))


def _pages_of(case):
    return -(-(case["tokens"] + case["page"] - 1) // case["page"]) + 3


def work(case):
    if case["op"] != "attend":
        t, hq, hk, d, r = (case[n] for n in ("tokens", "hq", "hk", "dim", "rot"))
        # q in and out, K/V in, slots, positions and the table's rows
        moved = t * (4 * hq * d + 4 * hk * d + 8) + (4 * t + 4 * min(t, case["far"]) * r if r else 0)
        turn = 3 * t * (hq + hk) * r
        if case["op"] == "rotary":
            return {"bytes": moved + 4 * t * hk * d, "flops": turn}
        row = hk * (d // 2 + 4 * d // case["group"])
        slots = _pages_of(case) * case["page"]
        # K/V rows out in 4 bits; the whole cache in, its values and the slot numbers out and in
        return {"bytes": moved + 2 * t * row + slots * (2 * row + 4 * hk * d + 8), "flops": turn + 8 * t * hk * d}
    ctx, new = _lengths(case)
    pairs, keys = 0, 0
    for c, n in zip(ctx, new):
        if case["tree"]:
            # a tree node sees at least the prefix and itself; the few ancestors are not counted
            pairs += n * (c + 1)
            keys += c + n
        elif n:
            pairs += _pairs(c, n, case["window"])
            keys += min(c + n, case["window"] + n - 1) if case["window"] else c + n
    rows, d = sum(new), case["dim"]
    return {"bytes": 2 * keys * case["hk"] * (d // 2 + 4 * d // case["group"]) + 4 * rows * case["hq"] * d,
            "flops": 4 * d * case["hq"] * pairs}


# ------------------------------------------------------------------ the inputs
def _tree_parents(r, n):
    """Parents of a random draft tree: node 0 is the root."""
    return [-1] + [r.randrange(0, i) for i in range(1, n)]


def _packed(codes):
    """Codes [..., D] as the cache's words [..., D / 8]."""
    c = codes.to(torch.int32).unflatten(-1, (-1, 8, 4))
    quads = (c[..., 0] | c[..., 1] << 4 | c[..., 2] << 8 | c[..., 3] << 12).to(torch.int16)
    return quads.transpose(-1, -2).flatten(-2).contiguous().view(torch.int32)


def _cache(g, shape, group, dtype):
    """Codes and affine of normally distributed rows with an offset of their own in each channel."""
    x = torch.randn(*shape, generator=g, device="cuda")
    x += 0.5 * torch.randn(shape[-1], generator=g, device="cuda")
    x = x.unflatten(-1, (-1, group))
    low = x.amin(-1, keepdim=True).to(dtype)
    scale = ((x.amax(-1, keepdim=True) - low.float()) / 15).to(dtype)
    codes = ((x - low.float()) / scale.float()).round().clamp(0, 15).to(torch.int8)
    return _packed(codes.flatten(-2)), torch.cat([scale, low], -1)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    r = random.Random(seed)
    i32 = dict(dtype=torch.int32, device=dev)
    dtype = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(dtype)

    st = {"case": case}
    hq, hk, d, ps = case["hq"], case["hk"], case["dim"], case["page"]
    if case["op"] != "attend":
        t, rot, far = case["tokens"], case["rot"], case["far"]
        n_pages = _pages_of(case)
        st.update(q=normal(t, hq, d, std=2.0) if hq else None, k_new=normal(t, hk, d), v_new=normal(t, hk, d))
        # whole pages in any order, entered at an odd place, and a few rows that are not to be written
        order = torch.randperm(n_pages, generator=g, device=dev)
        at = torch.arange(t, device=dev) + r.randrange(1, ps)
        slot = order[at // ps] * ps + at % ps
        slot[torch.rand(t, generator=g, device=dev) < 0.01] = -1
        st["slot"] = slot
        if rot:
            # runs of neighbouring positions, as prompts have them
            first = torch.randint(0, far, (1 + t // 500,), generator=g, device=dev)
            run = torch.arange(t, device=dev)
            st["pos"] = ((first[run // 500] + run % 500) % far).to(torch.int32)
            turn = 10000.0 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot)
            angle = torch.arange(far, device=dev, dtype=torch.float64)[:, None] * turn
            st["rotary"] = torch.cat([angle.cos(), angle.sin()], -1).float()
        if case["op"] == "rotary":
            st.update(k=normal(n_pages, hk, ps, d), v=normal(n_pages, hk, ps, d))
        else:
            st["cache"] = (*_cache(g, (n_pages, hk, ps, d), case["group"], dtype),
                           *_cache(g, (n_pages, hk, ps, d), case["group"], dtype))
            st["slots"] = torch.arange(n_pages * ps, device=dev)
        return st
    ctx, new = _lengths(case)
    b = case["batch"]
    rows = sum(new) + case["pad"]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    lens = [c + n for c, n in zip(ctx, new)]
    width = max(1, max(-(-n // ps) for n in lens))
    n_pages = sum(-(-n // ps) for n in lens) + 5
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    need = torch.tensor([-(-n // ps) for n in lens], device=dev)
    first = torch.cumsum(need, 0) - need
    col = torch.arange(width, device=dev)[None, :]
    table = torch.where(col < need[:, None], order[(first[:, None] + col).clamp(max=n_pages - 1)], -1)
    st.update(q=normal(rows, hq, d, std=2.0), cu=torch.tensor(cu, **i32), scale=d ** -0.5, max_new=max(new),
              out=torch.zeros(rows, hq, d, dtype=dtype, device=dev),
              cache=(*_cache(g, (n_pages, hk, ps, d), case["group"], dtype),
                     *_cache(g, (n_pages, hk, ps, d), case["group"], dtype)),
              table=table.to(torch.int32).contiguous(), lens=torch.tensor(lens, **i32), longest=max(lens), parents=None)
    if case["tree"]:
        par = [p for n in new for p in _tree_parents(r, n)] + [-1] * case["pad"]
        st["parents"] = torch.tensor(par, **i32)
    return st


# -------------------------------------------------------------- the plain forms
def _turned(x, st):
    """x [T, H, D] with its first `rot` elements turned by the rows' positions, unrounded in x's type."""
    case = st["case"]
    rot = case["rot"]
    if not rot:
        return x
    cos, sin = st["rotary"][st["pos"].long()].to(x.dtype)[:, None].chunk(2, -1)
    y = x[..., :rot]
    if case["inter"]:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y.chunk(2, -1)
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_rotary(st):
    ps, dtype = st["case"]["page"], st["q"].dtype
    q = _turned(st["q"].float(), st).to(dtype)
    k = _turned(st["k_new"].float(), st).to(dtype)
    live = st["slot"] >= 0
    slot = st["slot"][live]
    st["k"][slot // ps, :, slot % ps] = k[live]
    st["v"][slot // ps, :, slot % ps] = st["v_new"][live]
    return {"q": q, "k": st["k"], "v": st["v"]}


def _quantised(x, group, dtype):
    """(codes, scale and bias) of x [..., D] in 64 bits, scale and bias as the 16-bit type holds them."""
    x = x.unflatten(-1, (-1, group))
    low, high = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    scale, bias = ((high - low) / 15).float().to(dtype), low.float().to(dtype)
    s = scale.double()
    codes = ((x - bias.double()) / torch.where(s == 0, 1.0, s)).round().clamp(0, 15)
    return torch.where(s == 0, 0.0, codes).flatten(-2), torch.cat([scale, bias], -1)


def _values(codes, affine, group):
    """Words and affine as 32-bit values [..., D]."""
    quads = codes.view(torch.int16).unflatten(-1, (8, -1)).transpose(-1, -2).flatten(-2).to(torch.int32)
    c = torch.stack([(quads >> s) & 15 for s in (0, 4, 8, 12)], -1).flatten(-2).unflatten(-1, (-1, group))
    a = affine.float()
    return (c.float() * a[..., 0:1] + a[..., 1:2]).flatten(-2)


def _plain_append(st):
    case = st["case"]
    ps, group, dtype = case["page"], case["group"], st["k_new"].dtype
    live = st["slot"] >= 0
    slot = st["slot"][live]
    got = {} if st["q"] is None else {"q": _turned(st["q"].float(), st).to(dtype)}
    rows = {"k": _turned(st["k_new"].double(), st), "v": st["v_new"].double()}
    for i, x in enumerate("kv"):
        words, affine = st["cache"][2 * i:2 * i + 2]
        codes, new = _quantised(rows[x][live], group, dtype)
        words[slot // ps, :, slot % ps] = _packed(codes)
        affine[slot // ps, :, slot % ps] = new
        got[x] = _values(words, affine, group).to(dtype).transpose(1, 2).flatten(0, 1)
    return got


def _softmax_rows(q, k, v, see, scale):
    """softmax(q k^T scale) v over the visible keys; rows that see none give zeros."""
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(scale).masked_fill_(~see, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(total == 0, 1.0, total)


def _plain_attend(st):
    case = st["case"]
    cu, q, out = st["cu"].long(), st["q"], st["out"]
    b, hq, hk, d = case["batch"], case["hq"], case["hk"], case["dim"]
    n, grp, most, longest = cu[-1:], case["hq"] // case["hk"], st["max_new"], st["longest"]
    new, lens = cu[1:] - cu[:-1], st["lens"].long()
    i = torch.arange(most, device=q.device)
    j = torch.arange(longest, device=q.device)
    rows = (cu[:-1, None] + i).clamp(max=q.shape[0] - 1)                 # [B, most]
    qq = q[rows].float().view(b, most, hk, grp, d).permute(0, 2, 3, 1, 4).reshape(b, hk, grp * most, d)
    table = st["table"].clamp(min=0).long()
    kk, vv = (_values(w[table], a[table], case["group"]).transpose(1, 2).reshape(b, hk, -1, d)[:, :, :longest]
              for w, a in (st["cache"][:2], st["cache"][2:]))
    base = (lens - new)[:, None, None]                                   # [B, 1, 1]
    pos = base + i[None, :, None]
    if case["tree"]:
        par = st["parents"][rows].long()                                 # [B, most]
        step = ((par[:, :, None] == i) & (par[:, :, None] >= 0)).double()
        # powers of (I + step) have a positive cell exactly where a chain of parents leads
        sees = torch.linalg.matrix_power(step + torch.eye(most, device=q.device, dtype=torch.float64), most) > 0
        node = (j[None, :] - base[:, 0]).clamp(0, most - 1)               # [B, keys]
        inside = torch.gather(sees, 2, node[:, None, :].expand(-1, most, -1))
        see = torch.where(j < base, torch.ones_like(inside), inside) & (j < lens[:, None, None])
    else:
        see = (j <= pos) & (j < lens[:, None, None])
        if case["window"]:
            see = see & (j > pos - case["window"])
    vv = vv * (j < lens[:, None, None])[:, None, 0, :, None]
    see = see[:, None, None].expand(b, 1, grp, most, longest).reshape(b, 1, grp * most, longest)
    o = _softmax_rows(qq, kk, vv, see, st["scale"])
    o = o.view(b, hk, grp, most, d).permute(0, 3, 1, 2, 4).reshape(b, most, hq, d)
    t = torch.arange(q.shape[0], device=q.device)
    rb = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=b - 1)
    got = o[rb, (t - cu[rb]).clamp(max=most - 1)].to(q.dtype)
    return torch.where((t < n)[:, None, None], got, out)


# ---------------------------------------------------------------------- a pass
def run(st):
    case = st["case"]
    if not own:
        return {"rotary": _plain_rotary, "append": _plain_append, "attend": _plain_attend}[case["op"]](st)
    import tree_masked_speculative_gb300 as ta
    if case["op"] == "rotary":
        q = ta.paged_append_rotary(st["q"], st["k_new"], st["v_new"], st["k"], st["v"], st["slot"], st["pos"],
                                   st["rotary"], interleaved=bool(case["inter"]))
        return {"q": q, "k": st["k"], "v": st["v"]}
    cache = ta.PagedQuantCache(*st["cache"])
    if case["op"] == "append":
        q = ta.paged_quant_append(st["k_new"], st["v_new"], cache, st["slot"], q=st["q"], positions=st.get("pos"),
                                  rotary=st.get("rotary"), interleaved=bool(case["inter"]))
        k, v = ta.paged_quant_read(cache, st["slots"])
        return {"k": k, "v": v} if q is None else {"q": q, "k": k, "v": v}
    if "tmp" not in st:
        st["tmp"] = ta.paged_quant_attention_workspace(st["q"], cache, st["table"], max_q_len=st["max_new"])
    return ta.paged_quant_attention(st["q"], cache, st["table"], st["cu"], st["lens"], scale=st["scale"],
                                    max_q_len=st["max_new"], window=case["window"], parents=st["parents"],
                                    tmp=st["tmp"], out=st["out"])


# ------------------------------------------------------------------ in 64 bits
def _exact_values(words, affine, d, group):
    """[N, ..., D] in 64 bits, one element of the head at a time."""
    a = affine.double()
    out = torch.empty(*words.shape[:-1], d, dtype=torch.float64, device=words.device)
    for e in range(d):
        quad = (e % 32) // 4 * (d // 32) + e // 32
        code = (words[..., quad // 2] >> (16 * (quad % 2) + 4 * (e % 4))) & 15
        out[..., e] = code * a[..., e // group, 0] + a[..., e // group, 1]
    return out


def _exact_turned(x, st):
    """A turn as a product with each position's matrix, by complex numbers."""
    rot = st["case"]["rot"]
    x = x.double()
    if not rot:
        return x
    h = rot // 2
    first = torch.arange(h, device=x.device) * (2 if st["case"]["inter"] else 1)
    second = first + (1 if st["case"]["inter"] else h)
    row = st["rotary"].double()[st["pos"].long()]
    z = torch.complex(x[..., first], x[..., second]) * torch.complex(row[:, :h], row[:, h:])[:, None]
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    """Rows of an append one by one in a flat view of the cache; attention by its
    definition, one request and one head at a time."""
    st = prepare(case, seed)
    d, hk = case["dim"], case["hk"]
    if case["op"] != "attend":
        got = {} if st["q"] is None else {"q": _exact_turned(st["q"], st)}
        live = st["slot"] >= 0
        rows = {"k": _exact_turned(st["k_new"], st)[live], "v": st["v_new"].double()[live]}
        slot = st["slot"][live]
        if case["op"] == "rotary":
            for x in "kv":
                n, _, ps, _ = st[x].shape
                flat = st[x].double().transpose(1, 2).reshape(n * ps, hk, d)
                flat[slot] = rows[x]
                got[x] = flat.view(n, ps, hk, d).transpose(1, 2)
            return got
        dtype, group = st["k_new"].dtype, case["group"]
        for i, x in enumerate("kv"):
            words, affine = st["cache"][2 * i:2 * i + 2]
            flat = _exact_values(words, affine, d, group).transpose(1, 2).reshape(-1, hk, d)
            for first in range(0, d, group):
                part = rows[x][..., first:first + group]
                least = part.min(-1, keepdim=True).values
                step = ((part.max(-1, keepdim=True).values - least) / 15).float().to(dtype).double()
                least = least.float().to(dtype).double()
                code = torch.clamp(torch.round((part - least) / step), 0, 15)
                flat[slot, :, first:first + group] = torch.where(step == 0, 0.0, code) * step + least
            got[x] = flat
        return got
    ctx, new = _lengths(case)
    grp, ps = case["hq"] // hk, case["page"]
    if 4e-12 * work(case)["flops"] > 20:
        return None
    out = st["out"].double()
    start = 0
    for b in range(case["batch"]):
        n, length = new[b], ctx[b] + new[b]
        if not n:
            continue
        cells = st["table"][b, :-(-length // ps)].long()
        keys, values = (_exact_values(w[cells], a[cells], d, case["group"]).permute(0, 2, 1, 3).reshape(-1, hk, d)[:length]
                        for w, a in (st["cache"][:2], st["cache"][2:]))
        hidden = torch.ones(n, length, dtype=torch.bool, device=out.device)
        if case["tree"]:
            hidden[:, :ctx[b]] = False
            par = st["parents"][start:start + n].tolist()
            for i in range(n):
                a = i
                while a >= 0:
                    hidden[i, ctx[b] + a] = False
                    a = par[a]
        else:
            hidden = torch.triu(hidden, ctx[b] + 1)
            if case["window"]:
                hidden |= torch.tril(torch.ones_like(hidden), ctx[b] - case["window"])
        for h in range(case["hq"]):
            logits = st["q"][start:start + n, h].double() @ keys[:, h // grp].T / math.sqrt(d)
            weights = torch.softmax(logits.masked_fill(hidden, -math.inf), -1)
            out[start:start + n, h] = weights @ values[:, h // grp]
        start += n
    return out
