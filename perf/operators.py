"""Serving operators of the library on a paged K/V cache: what is computed, on
which sizes, and what each pass cannot do without.

Four operators, in the order a serving step uses them:

plan     block tables, slot map and row offsets of a step from request lengths
append   the step's new K/V rows written to their pages
paged    attention of every request's new tokens (one token, a chunk or a draft
         tree) over its pages
prompt   causal attention over whole prompts packed one behind the other

Plain forms are elementary torch operations in 32 bits; ``exact`` restates the
definitions in 64 bits, request by request.
"""
import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step of a small server: every request grows by one token, latency counts
        dict(name="plan decode 48", op="plan", batch=48, page=16, ctx_lo=1, ctx_hi=4096, new_lo=1, new_hi=1, pad=0,
             lens=1),
        # admission of a large batch: prompts of up to 512 tokens, many new pages, rejected drafts give pages back
        dict(name="plan prompts 512", op="plan", batch=512, page=16, ctx_lo=0, ctx_hi=8192, new_lo=0, new_hi=512,
             pad=7, lens=2),
        # the K/V rows of one decode step of 64 requests
        dict(name="append step 64", op="append", tokens=64, hk=8, dim=128, page=16, dtype="bf16", lens=3),
        # the K/V rows of a large prompt batch, odd count, head dimension 256
        dict(name="append prompts 32k", op="append", tokens=32749, hk=4, dim=256, page=64, dtype="f16", lens=4),
        # three requests decoding one token each on short contexts: latency
        dict(name="decode 3", op="paged", batch=3, hq=32, hk=8, dim=128, page=16, dtype="bf16", ctx_lo=200,
             ctx_hi=2100, new_lo=1, new_hi=1, window=0, tree=0, pad=0, lens=5),
        # a full decode batch on ragged contexts: bandwidth
        dict(name="decode 64", op="paged", batch=64, hq=32, hk=8, dim=128, page=16, dtype="bf16", ctx_lo=900,
             ctx_hi=16384, new_lo=1, new_hi=1, window=0, tree=0, pad=0, lens=6),
        # draft trees of 32 nodes of eight requests (the fixed-tree configuration's heads), contexts around 4096
        dict(name="verify trees 8", op="paged", batch=8, hq=24, hk=4, dim=256, page=64, dtype="f16", ctx_lo=2500,
             ctx_hi=4096, new_lo=32, new_hi=32, window=0, tree=1, pad=0, lens=7),
        # prompt chunks of up to 512 tokens of twelve requests over what they have cached
        dict(name="chunks 12", op="paged", batch=12, hq=32, hk=8, dim=128, page=32, dtype="bf16", ctx_lo=0,
             ctx_hi=8192, new_lo=1, new_hi=512, window=0, tree=0, pad=5, lens=8),
        # short prompts of 1 to 200 tokens, one KV head per query head, head dimension 64
        dict(name="prompts short", op="prompt", batch=24, hq=16, hk=16, dim=64, dtype="f16", len_lo=1, len_hi=200,
             window=0, pad=3, lens=9),
        # a packed batch of ragged prompts
        dict(name="prompts packed", op="prompt", batch=10, hq=32, hk=8, dim=128, dtype="bf16", len_lo=60,
             len_hi=4096, window=0, pad=0, lens=10),
        # one long prompt
        dict(name="prompt 8192", op="prompt", batch=1, hq=32, hk=8, dim=128, dtype="bf16", len_lo=8192, len_hi=8192,
             window=0, pad=0, lens=11),
        # two prompts with a sliding window, six query heads per KV head, head dimension 256
        dict(name="prompts window 256", op="prompt", batch=2, hq=24, hk=4, dim=256, dtype="f16", len_lo=2000,
             len_hi=6000, window=1000, pad=0, lens=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.99)))))))


def draw(rng):
    case = _draw(rng)
    # no drawn case costs more than the largest listed ones
    while case["op"] not in ("plan", "append") and case["batch"] > 1 and (
            work(case)["flops"] > 4e11 or work(case)["bytes"] > 1.5e9):
        case["batch"] = (case["batch"] + 1) // 2
    return case


def _draw(rng):
    op = rng.choice(["plan", "append", "paged", "paged", "prompt", "prompt"])
    lens = rng.randrange(100, 1 << 30)
    dtype = rng.choice(["f16", "bf16"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        return dict(op=op, batch=_log(rng, 1, 512), page=page, ctx_lo=0, ctx_hi=_log(rng, 64, 8192), new_lo=0,
                    new_hi=_log(rng, 1, 512), pad=rng.randrange(0, 9), lens=lens)
    if op == "append":
        hk, dim = rng.choice([(8, 128), (4, 256), (8, 64), (1, 128), (2, 256)])
        return dict(op=op, tokens=_log(rng, 1, 32000), hk=hk, dim=dim, page=page, dtype=dtype, lens=lens)
    hk, dim = rng.choice([(8, 128), (4, 128), (8, 64), (4, 256)])
    hq = hk * rng.choice([1, 2, 3, 4, 6, 8] if hk == 4 else [1, 2, 4])
    if op == "paged":
        kind = rng.choice(["decode", "chunk", "tree"])
        if kind == "decode":
            ctx_hi = _log(rng, 32, 16000)
            return dict(op=op, batch=_log(rng, 1, 60), hq=hq, hk=hk, dim=min(dim, 128), page=page, dtype=dtype,
                        ctx_lo=0, ctx_hi=ctx_hi, new_lo=1, new_hi=rng.choice([1, 1, 2, 3]),
                        window=rng.choice([0, 0, 1 + ctx_hi // 3]), tree=0, pad=rng.randrange(0, 4), lens=lens)
        if kind == "chunk":
            ctx_hi = _log(rng, 64, 8000)
            return dict(op=op, batch=_log(rng, 1, 8), hq=hq, hk=hk, dim=dim, page=page, dtype=dtype, ctx_lo=0,
                        ctx_hi=ctx_hi, new_lo=0, new_hi=_log(rng, 16, 500),
                        window=rng.choice([0, 0, 1 + ctx_hi // 3]), tree=0, pad=rng.randrange(0, 9), lens=lens)
        return dict(op=op, batch=_log(rng, 1, 10), hq=hq, hk=hk, dim=dim, page=page, dtype=dtype, ctx_lo=0,
                    ctx_hi=_log(rng, 64, 8000), new_lo=1, new_hi=_log(rng, 4, 100), window=0, tree=1,
                    pad=rng.randrange(0, 4), lens=lens)
    len_hi = _log(rng, 24, 4096)
    return dict(op=op, batch=_log(rng, 1, 10), hq=hq, hk=hk, dim=dim, dtype=dtype, len_lo=rng.choice([0, 1, len_hi // 2]),
                len_hi=len_hi, window=rng.choice([0, 0, 1 + len_hi // 3]), pad=rng.randrange(0, 9), lens=lens)


def _lengths(case):
    """Host lists of the case's lengths: (kept or context tokens, new tokens).
    They belong to the case, not to the seed, so that its work is known."""
    r = random.Random(case["lens"])
    n = case["batch"]
    if case["op"] == "prompt":
        new = [r.randint(case["len_lo"], case["len_hi"]) for _ in range(n)]
        new[0] = max(1, case["len_hi"])
        return [0] * n, new
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(n)]
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(n)]
    ctx[-1], new[-1] = case["ctx_hi"], max(1, case["new_hi"])
    return ctx, new


def _pairs(ctx, new, window):
    """Visible (token, key) pairs of a causal chunk behind ctx tokens."""
    if not window:
        return new * ctx + new * (new + 1) // 2
    return sum(min(ctx + i + 1, window) for i in range(new))


def work(case):
    if case["op"] == "plan":
        ctx, new = _lengths(case)
        b, t, ps = case["batch"], sum(new) + case["pad"], case["page"]
        cells = sum(-(-(c + n) // ps) - c // ps for c, n in zip(ctx, new) if n)
        return {"bytes": 4 * (3 * b + 1) + 4 * (3 * b + 2) + 12 * t + 8 * cells, "flops": 0}
    if case["op"] == "append":
        return {"bytes": 4 * case["tokens"] * case["hk"] * case["dim"] * 2 + 8 * case["tokens"], "flops": 0}
    ctx, new = _lengths(case)
    pairs, keys = 0, 0
    for c, n in zip(ctx, new):
        if case.get("tree"):
            # a tree node sees at least the prefix and itself; the few ancestors are not counted
            pairs += n * (c + 1)
            keys += c + n
        elif n:
            pairs += _pairs(c, n, case["window"])
            keys += min(c + n, case["window"] + n - 1) if case["window"] else c + n
    rows = sum(new)
    return {"bytes": 2 * (2 * keys * case["hk"] * case["dim"] + 2 * rows * case["hq"] * case["dim"]),
            "flops": 4 * case["dim"] * case["hq"] * pairs}


# ------------------------------------------------------------------ the inputs
def _tree_parents(r, n):
    """Parents of a random draft tree: node 0 is the root."""
    return [-1] + [r.randrange(0, i) for i in range(1, n)]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    r = random.Random(seed)
    i32 = dict(dtype=torch.int32, device=dev)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(DTYPES[case["dtype"]])

    def pages(table_cells):
        return torch.randperm(table_cells, generator=g, device=dev).to(torch.int32)

    st = {"case": case}
    if case["op"] == "plan":
        ctx, new = _lengths(case)
        b, ps = case["batch"], case["page"]
        width = max(-(-(c + n) // ps) for c, n in zip(ctx, new)) + 2
        # pages held from the step before: most rows hold exactly their kept tokens' pages, some hold more
        # (rejected draft tokens, finished requests)
        held = [min(width, -(-c // ps) + (r.randint(1, 3) if r.random() < 0.25 else 0)) for c in ctx]
        total = b * width + 64
        perm = pages(total)
        table = perm[:b * width].reshape(b, width).contiguous()
        stack = torch.full((total,), -1, **i32)
        need = sum(max(0, -(-(c + n) // ps) - h) for c, n, h in zip(ctx, new, held))
        used = torch.arange(width, device=dev)[None, :] < torch.tensor(held, device=dev)[:, None]
        free = torch.cat([perm[b * width:], table.reshape(-1)[~used.reshape(-1)]])
        n_free = max(need, free.numel() - r.randint(0, 40))
        stack[:n_free] = free[:n_free]
        tokens = sum(new) + case["pad"]
        st.update(keep=torch.tensor(ctx, **i32), new=torch.tensor(new, **i32), held=torch.tensor(held, **i32),
                  table=torch.where(used, table, -1).to(torch.int32), stack=stack,
                  n_free=torch.tensor([n_free], **i32), tokens=tokens,
                  out=(torch.empty(b, **i32), torch.empty(1, **i32), torch.empty(b + 1, **i32),
                       torch.empty(b, **i32), torch.empty(tokens, dtype=torch.int64, device=dev),
                       torch.empty(tokens, **i32), torch.zeros(1, **i32)))
        return st
    if case["op"] == "append":
        t, hk, d, ps = case["tokens"], case["hk"], case["dim"], case["page"]
        n_pages = -(-t // ps) * 2 + 3
        st.update(k_new=normal(t, hk, d), v_new=normal(t, hk, d), k=normal(n_pages, hk, ps, d),
                  v=normal(n_pages, hk, ps, d))
        # whole pages in any order, entered at an odd place, and a few rows that are not to be written
        order = pages(n_pages).to(torch.int64)
        at = torch.arange(t, device=dev) + r.randrange(1, ps)
        slot = order[at // ps] * ps + at % ps
        slot[torch.rand(t, generator=g, device=dev) < 0.01] = -1
        st["slot"] = slot
        return st
    ctx, new = _lengths(case)
    b, hq, hk, d = case["batch"], case["hq"], case["hk"], case["dim"]
    rows = sum(new) + case["pad"]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    st.update(q=normal(rows, hq, d, std=2.0), cu=torch.tensor(cu, **i32), scale=d ** -0.5, max_new=max(new),
              out=torch.zeros(rows, hq, d, dtype=DTYPES[case["dtype"]], device=dev))
    if case["op"] == "prompt":
        st.update(k=normal(rows, hk, d), v=normal(rows, hk, d))
        return st
    ps = case["page"]
    lens = [c + n for c, n in zip(ctx, new)]
    width = max(1, max(-(-n // ps) for n in lens))
    n_pages = sum(-(-n // ps) for n in lens) + 5
    order = pages(n_pages)
    need = torch.tensor([-(-n // ps) for n in lens], device=dev)
    first = torch.cumsum(need, 0) - need
    col = torch.arange(width, device=dev)[None, :]
    table = torch.where(col < need[:, None], order[(first[:, None] + col).clamp(max=n_pages - 1)], -1)
    st.update(k=normal(n_pages, hk, ps, d), v=normal(n_pages, hk, ps, d), table=table.to(torch.int32).contiguous(),
              lens=torch.tensor(lens, **i32), longest=max(lens), parents=None)
    if case["tree"]:
        par = [p for n in new for p in _tree_parents(r, n)] + [-1] * case["pad"]
        st["parents"] = torch.tensor(par, **i32)
    return st


# -------------------------------------------------------------- the plain forms
def _plain_plan(st):
    keep, new, held, table, stack = (st[n] for n in ("keep", "new", "held", "table", "stack"))
    ps, tokens = st["case"]["page"], st["tokens"]
    lens = keep + new
    need = (lens + ps - 1) // ps
    back = (held - need).clamp(min=0)
    grow = (need - held).clamp(min=0)
    at = st["n_free"] + torch.cumsum(back, 0) - back            # where a row's pages go on the stack
    col = torch.arange(table.shape[1], device=table.device, dtype=torch.int32)[None, :]
    # pages given back, in row order, then in column order (cells that give none write the spare last entry)
    give = (col >= need[:, None]) & (col < held[:, None])
    spare = torch.cat([stack, stack[:1]])
    spare[torch.where(give, at[:, None] + col - need[:, None], stack.numel()).long()] = table
    stack.copy_(spare[:-1])
    top = st["n_free"] + back.sum()
    took = torch.cumsum(grow, 0) - grow
    take = (col >= held[:, None]) & (col < need[:, None])
    src = torch.where(take, top - 1 - took[:, None] - col + held[:, None], 0)
    table.copy_(torch.where(take, stack[src.long()], table))
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device=table.device), torch.cumsum(new, 0)])
    t = torch.arange(tokens, device=table.device)
    b = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=keep.numel() - 1)
    pos = keep[b] + t - cu[b]
    live = t < cu[-1]
    page = table[b, (pos // ps).clamp(max=table.shape[1] - 1)]
    return {"table": table, "stack": stack, "held": need.to(torch.int32), "n_free": (top - grow.sum()).to(torch.int32),
            "cu": cu.to(torch.int32), "lens": lens.to(torch.int32),
            "slot": torch.where(live, page.long() * ps + pos % ps, -1), "pos": torch.where(live, pos, -1).to(torch.int32)}


def _plain_append(st):
    ps = st["case"]["page"]
    live = st["slot"] >= 0
    slot = st["slot"][live]
    st["k"][slot // ps, :, slot % ps] = st["k_new"][live]
    st["v"][slot // ps, :, slot % ps] = st["v_new"][live]
    return {"k": st["k"], "v": st["v"]}


def _softmax_rows(q, k, v, see, scale):
    """softmax(q k^T scale) v over the visible keys; rows that see none give zeros."""
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(scale).masked_fill_(~see, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(total == 0, 1.0, total)


def _plain_attention(st):
    case = st["case"]
    cu, q, out = st["cu"].long(), st["q"], st["out"]
    b, hq, hk, d = case["batch"], case["hq"], case["hk"], case["dim"]
    n, grp, most = cu[-1:], case["hq"] // case["hk"], st["max_new"]
    new = cu[1:] - cu[:-1]
    i = torch.arange(most, device=q.device)
    rows = (cu[:-1, None] + i).clamp(max=q.shape[0] - 1)                 # [B, most]
    qq = q[rows].float().view(b, most, hk, grp, d).permute(0, 2, 3, 1, 4).reshape(b, hk, grp * most, d)
    if case["op"] == "prompt":
        kk, vv, lens = (st["k"][rows].float().transpose(1, 2), st["v"][rows].float().transpose(1, 2), new)
        longest = most
    else:
        ps, table = case["page"], st["table"].clamp(min=0).long()
        kk, vv = (st[x][table].transpose(1, 2).reshape(b, hk, -1, d)[:, :, :st["longest"]].float() for x in "kv")
        lens, longest = st["lens"].long(), st["longest"]
    j = torch.arange(longest, device=q.device)
    base = (lens - new)[:, None, None]                                   # [B, 1, 1]
    pos = base + i[None, :, None]
    if case.get("tree"):
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
        return {"plan": _plain_plan, "append": _plain_append}.get(case["op"], _plain_attention)(st)
    import tree_masked_speculative_gb300 as ta
    if case["op"] == "plan":
        s = ta.paged_plan(st["keep"], st["new"], st["held"], st["table"], st["stack"], st["n_free"],
                          page_size=case["page"], max_tokens=st["tokens"], out=st["out"])
        return {"table": st["table"], "stack": st["stack"], "held": s.held, "n_free": s.n_free, "cu": s.cu_q,
                "lens": s.kv_lens, "slot": s.slot_map, "pos": s.positions}
    if case["op"] == "append":
        ta.paged_append(st["k_new"], st["v_new"], st["k"], st["v"], st["slot"])
        return {"k": st["k"], "v": st["v"]}
    if case["op"] == "paged":
        if "tmp" not in st:
            st["tmp"] = ta.paged_attention_workspace(st["q"], st["k"], st["table"], max_q_len=st["max_new"])
        return ta.paged_attention(st["q"], st["k"], st["v"], st["table"], st["cu"], st["lens"], scale=st["scale"],
                                  max_q_len=st["max_new"], window=case["window"], parents=st["parents"],
                                  tmp=st["tmp"], out=st["out"])
    if "tmp" not in st:
        st["tmp"] = ta.prompt_attention_workspace(st["q"], st["k"], st["cu"])
    return ta.prompt_attention(st["q"], st["k"], st["v"], st["cu"], scale=st["scale"], window=case["window"],
                               tmp=st["tmp"], out=st["out"])


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """Attention by its definition, one request and one head at a time; the rows
    of an append in a flat [slots, Hk, D] view of the cache."""
    if case["op"] == "plan":
        return None
    st = prepare(case, seed)
    if case["op"] == "append":
        got = {}
        for x in "kv":
            n, hk, ps, d = st[x].shape
            flat = torch.cat([st[x].double().transpose(1, 2).reshape(n * ps, hk, d),
                              torch.zeros(1, hk, d, dtype=torch.float64, device=st[x].device)])
            flat[st["slot"]] = st[x + "_new"].double()      # slot -1: the extra last row
            got[x] = flat[:-1].view(n, ps, hk, d).transpose(1, 2)
        return got
    ctx, new = _lengths(case)
    grp, d = case["hq"] // case["hk"], case["dim"]
    if 4e-12 * work(case)["flops"] > 20:
        return None
    out = st["out"].double()
    start = 0
    for b in range(case["batch"]):
        n, length = new[b], ctx[b] + new[b]
        if not n:
            continue
        if case["op"] == "prompt":
            keys, values = st["k"][start:start + n], st["v"][start:start + n]
        else:
            ps = case["page"]
            cells = st["table"][b, :-(-length // ps)].long()
            keys, values = (st[x][cells].permute(0, 2, 1, 3).reshape(-1, case["hk"], d)[:length] for x in "kv")
        hidden = torch.ones(n, length, dtype=torch.bool, device=out.device)
        if case.get("tree"):
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
            logits = st["q"][start:start + n, h].double() @ keys[:, h // grp].double().T / math.sqrt(d)
            weights = torch.softmax(logits.masked_fill(hidden, -math.inf), -1)
            out[start:start + n, h] = weights @ values[:, h // grp].double()
        start += n
    return out
