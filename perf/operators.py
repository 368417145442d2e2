"""Cases of the paged-cache operators: building block tables and slot maps, writing keys and
values into the pages, the masks of drafted token trees, and the attention of those trees over
the cache.

Together they are one round of speculative decoding (and, with one token a request, of ordinary
decoding): drafted tokens attend to the cache and to their ancestors, the accepted ones get
slots, their keys and values go into the pages.
"""
import math
import random

import torch

own = False

DTYPES = {"float16": torch.float16, "bfloat16": torch.bfloat16}


def listed():
    return [
        # one request, one new token, a moderate context: the latency of a single decode step
        dict(name="attn_decode_1", op="attention", dtype="float16", batch=1, tree=1, ctx=2048,
             ragged=False, kv_heads=8, group=4, dim=128, page=16, masked=False),
        # a small server without shared heads, head width 64, chains of drafted tokens
        dict(name="attn_chain_16_heads", op="attention", dtype="float16", batch=16, tree=6,
             ctx=1777, ragged=True, kv_heads=16, group=1, dim=64, page=32, masked=False),
        # few requests with very long contexts and a tree each
        dict(name="attn_long_tree", op="attention", dtype="bfloat16", batch=2, tree=27,
             ctx=131072, ragged=True, kv_heads=8, group=4, dim=128, page=64, masked=True),
        # wide trees: 64 drafted tokens of 8 query heads a key head, bound by the products
        dict(name="attn_wide_tree", op="attention", dtype="bfloat16", batch=16, tree=64, ctx=4096,
             ragged=False, kv_heads=8, group=8, dim=128, page=16, masked=True),
        # a full server: many requests, trees of up to 16, the cache of one layer is 2 GB
        dict(name="attn_server_64", op="attention", dtype="bfloat16", batch=64, tree=16, ctx=8192,
             ragged=True, kv_heads=8, group=4, dim=128, page=16, masked=True),
        # one decode step of 64 requests: a token each
        dict(name="plan_decode_64", op="plan", batch=64, lens=4096, add=1, page=16, kind="append"),
        # accepted tokens of 256 trees get their slots
        dict(name="plan_accept_256", op="plan", batch=256, lens=8192, add=5, page=16,
             kind="accept"),
        # a large server's step: prompts, decodes, roll-backs and finished requests together
        dict(name="plan_mixed_4096", op="plan", batch=4096, lens=4096, add=128, page=32,
             kind="mixed"),
        # the accepted tokens of 64 trees of 16: a third of the rows are kept
        dict(name="write_accepted", op="write", dtype="bfloat16", tokens=1024, keep=33, kv_heads=8,
             dim=128, page=16, pages=4096, fused=True),
        # a long prompt
        dict(name="write_prompt", op="write", dtype="float16", tokens=40000, keep=100, kv_heads=8,
             dim=128, page=16, pages=4096, fused=False),
        # trees of 64 requests
        dict(name="mask_64", op="mask", batch=64, tree=64, ragged=True),
        # a few very large trees
        dict(name="mask_1000", op="mask", batch=16, tree=1000, ragged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "plan", "write", "mask"])
    if op == "attention":
        batch, tree = _log(rng, 1, 96), _log(rng, 1, 200)
        group, kv_heads = rng.choice([1, 2, 3, 4, 5, 7, 8, 16]), rng.choice([1, 2, 4, 8, 16])
        dim = rng.choice([64, 128])
        # at most the largest listed cases' cache, products and plain-form scores
        row = batch * kv_heads
        ctx = _log(rng, 8, 131072)
        ctx = min(ctx, 64 * 8 * 8192 * 128 // (row * dim), 2 ** 29 // (row * tree * group))
        return dict(op=op, dtype=rng.choice(list(DTYPES)), batch=batch, tree=tree, ctx=ctx,
                    ragged=rng.random() < 0.7, kv_heads=kv_heads, group=group, dim=dim,
                    page=rng.choice([8, 16, 32, 64, 128, 256]), masked=rng.random() < 0.7)
    if op == "plan":
        kind = rng.choice(["append", "accept", "mixed"])
        batch = _log(rng, 1, 4096)
        return dict(op=op, batch=batch, lens=_log(rng, 1, min(100000, 2 ** 24 // batch)),
                    add=_log(rng, 1, min(4096, 2 ** 18 // batch)), page=rng.choice([8, 16, 32, 64, 128, 256]),
                    kind=kind)
    if op == "write":
        tokens, page = _log(rng, 1, 40000), rng.choice([8, 16, 32, 64, 128, 256])
        return dict(op=op, dtype=rng.choice(list(DTYPES)), tokens=tokens, keep=rng.randint(10, 100),
                    kv_heads=rng.choice([1, 2, 4, 8]), dim=rng.choice([64, 128]), page=page,
                    pages=65536 // page, fused=rng.random() < 0.5)
    return dict(op=op, batch=_log(rng, 1, 128), tree=_log(rng, 1, 1000), ragged=rng.random() < 0.7)


# ---------------------------------------------------------------- sizes of a case

def _sizes(case):
    """Per-request sizes: a function of the case alone, so that its work is known without a seed."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    B = case["batch"]
    if case["op"] == "plan":
        lens = [rng.randint(0, case["lens"]) for _ in range(B)]
        tree = [rng.randint(1, 2 * case["add"]) for _ in range(B)]
        add = [rng.randint(0, case["add"]) if case["add"] > 1 else 1 for _ in range(B)]
        if case["kind"] == "accept":
            add = [min(a, t) for a, t in zip(add, tree)]
        if case["kind"] == "mixed":
            for b in range(B):
                u = rng.random()
                if u < 0.1:
                    add[b] = -lens[b]                       # a finished request
                elif u < 0.2:
                    add[b] = -rng.randint(0, min(64, lens[b]))   # a roll-back
                elif u < 0.9:
                    add[b] = 1
        return lens, add, tree
    if not case["ragged"]:
        return [case["tree"]] * B, [case.get("ctx", 0)] * B
    tree = [case["tree"]] + [rng.randint(1, case["tree"]) for _ in range(B - 1)]
    ctx = [case.get("ctx", 0)] + [rng.randint(case.get("ctx", 0) // 8, case.get("ctx", 0))
                                  for _ in range(B - 1)]
    return tree, ctx


def work(case):
    op = case["op"]
    if op == "attention":
        tree, ctx = _sizes(case)
        size, row = 2, case["kv_heads"] * case["dim"]
        n = sum(tree)
        # cache, drafted keys and values, queries, outputs, block tables, mask
        by = 2 * size * row * (sum(ctx) + n) + 2 * size * row * case["group"] * n
        by += 4 * sum(-(-c // case["page"]) for c in ctx)
        if case["masked"]:
            by += 4 * n * _words(case)
        # two products over the context and the drafted tokens of the request
        fl = sum(4 * row * case["group"] * t * (c + (t if case["masked"] else (t + 1) / 2))
                 for t, c in zip(tree, ctx))
        return {"bytes": by, "flops": fl}
    if op == "plan":
        lens, add, tree = _sizes(case)
        n = sum(tree) if case["kind"] == "accept" else sum(max(a, 0) for a in add)
        P = case["page"]
        moved = sum(abs(-(-(l + a) // P) - -(-l // P)) for l, a in zip(lens, add))
        # lengths and additions in, lengths and starts out, pages in and out, slots and positions
        by = 16 * case["batch"] + 8 * moved + 12 * n + (4 * n if case["kind"] == "accept" else 0)
        return {"bytes": by, "flops": 0}
    if op == "write":
        row = 2 * 2 * case["kv_heads"] * case["dim"]     # keys and values, two bytes each
        kept = _kept(case)
        return {"bytes": 2 * row * kept + 8 * case["tokens"], "flops": 0}
    tree, _ = _sizes(case)
    return {"bytes": sum(tree) * (4 + 4 + 4 * _words(case)), "flops": 0}


def _words(case):
    return (case["tree"] + 31) // 32


def _kept(case):
    return max(1, case["tokens"] * case["keep"] // 100)


# ---------------------------------------------------------------- inputs

def _starts(counts, dev):
    t = torch.tensor([0] + counts, dtype=torch.int64)
    return torch.cumsum(t, 0).to(torch.int32).to(dev)


def _parents(tree, starts, g, dev):
    """A random tree per request: the parent of a token is one of the few before it, or the context."""
    n = sum(tree)
    first = torch.repeat_interleave(starts[:-1].long(), torch.tensor(tree, device=dev))
    i = torch.arange(n, device=dev) - first
    back = (torch.rand(n, generator=g, device=dev) ** 2 * 7).long() + 1
    return torch.clamp(i - back, min=-1).to(torch.int32)


def _pages(used, P, spare, g, dev):
    """Block tables of the requests' `used` page counts, and the ring of free pages: pages are dealt
    in random order, as after hours of serving."""
    total = int(used.sum()) + spare
    order = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    width = int(used.max()) if used.numel() else 0
    return total, order, width


def _prepare_attention(case, g, dev):
    tree, ctx = _sizes(case)
    dt, P = DTYPES[case["dtype"]], case["page"]
    H, D = case["kv_heads"], case["dim"]
    starts, n = _starts(tree, dev), sum(tree)
    lens = torch.tensor(ctx, dtype=torch.int32, device=dev)
    used = (lens.long() + P - 1) // P
    total, order, width = _pages(used, P, 3, g, dev)
    width += 2                               # a table has room for more than is used
    col = torch.arange(width, device=dev)
    tables = torch.zeros(case["batch"], width, dtype=torch.int32, device=dev)
    tables[col[None] < used[:, None]] = order[:int(used.sum())]
    cache = torch.randn(2, total, P, H, D, generator=g, device=dev, dtype=dt)
    # keys, values and queries as one projection makes them: slices of one tensor
    qkv = torch.randn(n, H * (case["group"] + 2), D, generator=g, device=dev, dtype=dt)
    q, k, v = qkv.split([H * case["group"], H, H], dim=1)
    mask = None
    if case["masked"]:
        words = _words(case)
        mask = _mask_plain(_parents(tree, starts, g, dev), starts, words)[0]
    return dict(case=case, q=q, k=k, v=v, k_cache=cache[0], v_cache=cache[1], tables=tables,
                lens=lens, starts=starts, mask=mask, tree=max(tree), ctx=max(ctx),
                out=torch.zeros(n, H * case["group"], D, dtype=dt, device=dev))


def _prepare_plan(case, g, dev):
    lens, add, tree = _sizes(case)
    P, B = case["page"], case["batch"]
    order_rows = torch.randperm(B, generator=g, device=dev)      # which request has which length
    lens_t = torch.tensor(lens, dtype=torch.int32, device=dev)[order_rows].contiguous()
    add_t = torch.tensor(add, dtype=torch.int32, device=dev)[order_rows].contiguous()
    tree_t = torch.tensor(tree, device=dev)[order_rows]
    used = (lens_t.long() + P - 1) // P
    after = (lens_t.long() + add_t.long() + P - 1) // P
    need = int(torch.clamp(after - used, min=0).sum())
    total, order, _ = _pages(used, P, need + 17, g, dev)
    width = int(torch.maximum(used, after).max()) + 2
    col = torch.arange(width, device=dev)
    tables = torch.zeros(B, width, dtype=torch.int32, device=dev)
    tables[col[None] < used[:, None]] = order[:int(used.sum())]
    head = int(torch.randint(0, total, (1,), generator=g, device=dev))
    free = total - int(used.sum())
    free_pages = torch.zeros(total, dtype=torch.int32, device=dev)
    free_pages[(head + torch.arange(free, device=dev)) % total] = order[int(used.sum()):]
    ring = torch.tensor([head, free], dtype=torch.int32, device=dev)
    starts = offsets = None
    tokens = int(torch.clamp(add_t, min=0).sum())
    if case["kind"] == "accept":
        starts = torch.zeros(B + 1, dtype=torch.int32, device=dev)
        starts[1:] = torch.cumsum(tree_t, 0)
        tokens = int(tree_t.sum())
        # a random increasing path of add tokens through each tree: the rest is not kept
        row = torch.repeat_interleave(torch.arange(B, device=dev), tree_t)
        key = torch.rand(tokens, generator=g, device=dev)
        rank = torch.argsort(torch.argsort(key + row)) - starts[row].long()
        keep = rank < add_t[row]
        before = torch.cumsum(keep, 0) - keep.long()
        offsets = torch.where(keep, before - before[starts[row].long()], -1).to(torch.int32)
    i32 = dict(dtype=torch.int32, device=dev)
    out = (torch.zeros(B, **i32), torch.zeros(2, **i32), torch.zeros(B + 1, **i32),
           torch.zeros(tokens, dtype=torch.int64, device=dev), torch.zeros(tokens, **i32),
           torch.zeros(1, **i32))
    return dict(case=case, lens=lens_t, add=add_t, ring=ring, free_pages=free_pages, tables=tables,
                tokens=tokens, starts=starts, offsets=offsets, out=out)


def _prepare_write(case, g, dev):
    dt, H, D, n = DTYPES[case["dtype"]], case["kv_heads"], case["dim"], case["tokens"]
    cache = torch.randn(2, case["pages"], case["page"], H, D, generator=g, device=dev, dtype=dt)
    if case["fused"]:
        k, v = torch.randn(n, 2 * H, D, generator=g, device=dev, dtype=dt).split([H, H], dim=1)
    else:
        k, v = torch.randn(2, n, H, D, generator=g, device=dev, dtype=dt)
    P = case["page"]
    # tokens in order fill pages that lie anywhere
    page = torch.randperm(case["pages"], generator=g, device=dev)
    kept = torch.randperm(n, generator=g, device=dev)[:_kept(case)].sort().values
    at = torch.arange(kept.numel(), device=dev)
    slots = torch.full((n,), -1, dtype=torch.int64, device=dev)
    slots[kept] = page[at // P] * P + at % P
    return dict(case=case, k=k, v=v, slots=slots, k_cache=cache[0], v_cache=cache[1])


def _prepare_mask(case, g, dev):
    tree, _ = _sizes(case)
    starts, n = _starts(tree, dev), sum(tree)
    words = _words(case)
    out = (torch.zeros(n, words, dtype=torch.int32, device=dev),
           torch.zeros(n, dtype=torch.int32, device=dev))
    return dict(case=case, parents=_parents(tree, starts, g, dev), starts=starts, words=words,
                out=out)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(dev).manual_seed(seed)
    make = dict(attention=_prepare_attention, plan=_prepare_plan, write=_prepare_write,
                mask=_prepare_mask)
    return make[case["op"]](case, g, dev)


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return _run_own(op, state)
    if op == "attention":
        return _attention_plain(state)
    if op == "plan":
        return _plan_plain(state)
    if op == "write":
        return _write_plain(state)
    return _mask_plain(state["parents"], state["starts"], state["words"])


def _run_own(op, s):
    from tensor_core_gemm_fp16_b200 import binding
    if op == "attention":
        return binding.tree_attention(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"],
                                      s["tables"], s["lens"], s["starts"], s["mask"], out=s["out"])
    if op == "plan":
        p = binding.cache_plan(s["lens"], s["add"], s["ring"], s["free_pages"], s["tables"],
                               s["case"]["page"], s["tokens"], starts=s["starts"],
                               offsets=s["offsets"], out=s["out"])
        return (p.lens, p.ring, p.starts, p.slots, p.positions, p.status, s["tables"],
                s["free_pages"])
    if op == "write":
        binding.cache_write(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"])
        return s["k_cache"], s["v_cache"]
    return binding.tree_mask(s["parents"], s["starts"], s["words"], out=s["out"])


def _attention_plain(s):
    case = s["case"]
    B, H, G, D, P = (case[k] for k in ("batch", "kv_heads", "group", "dim", "page"))
    T, dev = s["tree"], s["q"].device
    L = -(-s["ctx"] // P) * P
    starts, n = s["starts"].long(), s["q"].shape[0]
    count = starts[1:] - starts[:-1]
    i = torch.arange(T, device=dev)
    real = i[None] < count[:, None]                                     # [B, T]
    at = torch.clamp(starts[:-1, None] + i[None], max=n - 1)
    ids = s["tables"][:, :L // P].long()

    def cached(c):   # [B, H, L, D] in 32 bits
        return c[ids].reshape(B, L, H, D).float().transpose(1, 2)

    def drafted(x, heads):   # [B, heads, T, D]
        return x[at].float().transpose(1, 2)

    q = drafted(s["q"], H * G).reshape(B, H, G * T, D) * (1.0 / math.sqrt(D))
    sc = q @ cached(s["k_cache"]).transpose(2, 3)
    seen = torch.arange(L, device=dev)[None] < s["lens"][:, None]
    sc.masked_fill_(~seen[:, None, None], -math.inf)
    st = q @ drafted(s["k"], H).transpose(2, 3)                         # [B, H, G T, T]
    if s["mask"] is None:
        sees = (i[None, :] <= i[:, None])[None].expand(B, T, T)
    else:
        sees = (s["mask"][at][:, :, i // 32] >> (i % 32)) & 1           # [B, T, T]
        sees = sees.bool()
    sees = sees & real[:, None, :]
    st = st.view(B, H, G, T, T).masked_fill(~sees[:, None, None], -math.inf).view(B, H, G * T, T)
    m = torch.maximum(sc.amax(3) if L else torch.full_like(st[..., 0], -math.inf), st.amax(3))
    m = torch.where(m == -math.inf, 0.0, m)[..., None]
    sc, st = sc.sub_(m).exp_(), st.sub_(m).exp_()
    o = sc @ cached(s["v_cache"]) + st @ drafted(s["v"], H)
    total = (sc.sum(3) + st.sum(3))[..., None]
    o = torch.where(total > 0, o / total, 0.0)
    o = o.view(B, H * G, T, D).transpose(1, 2)                          # [B, T, heads, D]
    s["out"][at[real]] = o[real].to(s["out"].dtype)
    return s["out"]


def _plan_plain(s):
    lens, add = s["lens"].long(), s["add"].long()
    tables, pages, P = s["tables"], s["free_pages"], s["case"]["page"]
    dev, B, width = lens.device, lens.numel(), s["tables"].shape[1]
    cap, head, free = pages.numel(), s["ring"][0].long(), s["ring"][1].long()
    after = lens + add
    have, want = (lens + P - 1) // P, (after + P - 1) // P
    grow, drop = torch.clamp(want - have, min=0), torch.clamp(have - want, min=0)
    if s["starts"] is None:
        starts = torch.zeros(B + 1, dtype=torch.int64, device=dev)
        starts[1:] = torch.cumsum(torch.clamp(add, min=0), 0)
    else:
        starts = s["starts"].long()
    status = ((grow.sum() > free) * 1 + (want > width).any() * 2 + (after < 0).any() * 4 +
              (starts[B] > s["tokens"]) * 8)
    fine = status == 0
    # pages taken from the head of the ring, in the requests' order
    col = torch.arange(width, device=dev)[None]
    src = head + (torch.cumsum(grow, 0) - grow)[:, None] + col - have[:, None]
    new = (col >= have[:, None]) & (col < want[:, None]) & fine
    # pages given back behind its tail
    old = (col >= want[:, None]) & (col < have[:, None]) & fine
    dst = head + free + (torch.cumsum(drop, 0) - drop)[:, None] + col - want[:, None]
    back = torch.where(old, tables, 0)
    tables.copy_(torch.where(new, pages[src % cap], tables))
    ext = torch.cat([pages, pages[:1]])
    ext.scatter_(0, torch.where(old, dst % cap, cap).view(-1), back.view(-1))
    pages.copy_(ext[:cap])
    # slots and positions of the tokens
    i = torch.arange(s["tokens"], device=dev)
    b = torch.clamp(torch.searchsorted(starts[1:].contiguous(), i, right=True), max=B - 1)
    off = i - starts[b] if s["offsets"] is None else s["offsets"].long()
    kept = fine & (i < starts[B]) & (off >= 0) & (off < add[b])
    pos = torch.where(kept, lens[b] + off, 0)
    slot = tables[b, pos // P].long() * P + pos % P
    lens_out, ring_out, starts_out, slots, positions, stat = s["out"]
    lens_out.copy_(torch.where(fine, after, lens))
    ring_out[0] = torch.where(fine, (head + grow.sum()) % cap, head)
    ring_out[1] = torch.where(fine, free - grow.sum() + drop.sum(), free)
    starts_out.copy_(starts)
    slots.copy_(torch.where(kept, slot, -1))
    positions.copy_(torch.where(kept, pos, -1))
    stat.copy_(status[None])
    return lens_out, ring_out, starts_out, slots, positions, stat, tables, pages


def _write_plain(s):
    kept = s["slots"] >= 0
    at = s["slots"][kept]
    for cache, x in ((s["k_cache"], s["k"]), (s["v_cache"], s["v"])):
        cache.view(-1, *cache.shape[2:])[at] = x[kept]
    return s["k_cache"], s["v_cache"]


def _mask_plain(parents, starts, words):
    """Ancestors by doubling: after step s a token has those less than 2^s generations above it."""
    n, dev = parents.numel(), parents.device
    b = torch.searchsorted(starts[1:].contiguous(), torch.arange(n, device=dev, dtype=torch.int32),
                           right=True)
    first = starts.long()[b]
    i = torch.arange(n, device=dev) - first
    bit = torch.zeros(n + 1, words * 32, dtype=torch.bool, device=dev)      # row n: no token
    bit[torch.arange(n, device=dev), i] = True
    up = torch.full((n + 1,), n, dtype=torch.int64, device=dev)
    up[:n] = torch.where(parents >= 0, first + parents.long(), n)
    for _ in range(max(1, (words * 32 - 1).bit_length())):
        bit = bit | bit[up]
        up = up[up]
    depth = bit[:n].sum(1).to(torch.int32) - 1
    shift = torch.arange(32, device=dev, dtype=torch.int64)
    mask = (bit[:n].view(n, words, 32).long() << shift).sum(2)
    return torch.where(mask >= 2 ** 31, mask - 2 ** 32, mask).to(torch.int32), depth


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    """The attention by its definition, request by request in 64 bits; the written caches. Tables,
    slots and masks are whole numbers."""
    if case["op"] == "write":
        s = prepare(case, seed)
        both = []
        for c, x in ((s["k_cache"], s["k"]), (s["v_cache"], s["v"])):
            c = c.double().flatten(0, 1)
            t = torch.nonzero(s["slots"] >= 0)[:, 0]
            c.index_copy_(0, s["slots"][t], x[t].double())
            both.append(c.view(s["k_cache"].shape))
        return tuple(both)
    if case["op"] != "attention":
        return None
    s = prepare(case, seed)
    G, D = case["group"], case["dim"]
    out = s["out"].double()
    starts, lens = s["starts"].tolist(), s["lens"].tolist()
    for b in range(case["batch"]):
        t0, t1 = starts[b], starts[b + 1]
        pos = torch.arange(lens[b], device=out.device)
        page, slot = s["tables"][b].long()[pos // case["page"]], pos % case["page"]
        if s["mask"] is None:
            sees = torch.ones(t1 - t0, t1 - t0, device=out.device).tril() > 0
        else:
            bits = s["mask"][t0:t1].long() & 0xFFFFFFFF
            j = torch.arange(t1 - t0, device=out.device)
            sees = torch.bitwise_and(torch.bitwise_right_shift(bits[:, j // 32], j % 32), 1) > 0
        sees = torch.cat([torch.ones(t1 - t0, lens[b], device=out.device) > 0, sees], 1)
        for h in range(case["kv_heads"]):
            keys = torch.cat([s["k_cache"][page, slot, h], s["k"][t0:t1, h]]).double()
            values = torch.cat([s["v_cache"][page, slot, h], s["v"][t0:t1, h]]).double()
            q = s["q"][t0:t1, h * G:(h + 1) * G].double()
            z = torch.einsum("tgd,kd->gtk", q, keys) / D ** 0.5
            z = torch.where(sees, z, -torch.inf)
            w = torch.exp(z - torch.logsumexp(z, 2, keepdim=True))
            out[t0:t1, h * G:(h + 1) * G] = torch.einsum("gtk,kd->tgd", torch.nan_to_num(w), values)
    return out
