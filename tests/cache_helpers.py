"""Plain references of the paged-cache operators, by their definitions: request by request, the
attention in 64 bits, and the bound of its error."""
import math

import torch

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}     # half a step, relative


def plan_reference(lens, add, ring, free_pages, tables, page, tokens, starts=None, offsets=None):
    """tg_cache_plan on Python lists; returns (lens, ring, starts, slots, positions, status,
    free_pages, tables), the inputs unchanged."""
    B, cap, width = len(lens), len(free_pages), len(tables[0]) if tables else 0
    pages_of = lambda n: -(-n // page)   # noqa: E731
    packing = starts
    if packing is None:
        packing = [0]
        for a in add:
            packing.append(packing[-1] + max(a, 0))
    have = [pages_of(max(n, 0)) for n in lens]
    want = [pages_of(max(n + a, 0)) for n, a in zip(lens, add)]
    grow = sum(max(w - h, 0) for h, w in zip(have, want))
    drop = sum(max(h - w, 0) for h, w in zip(have, want))
    head, count = ring
    status = 0
    if grow > count:
        status |= 1
    if any(max(h, w) > width for h, w in zip(have, want)):
        status |= 2
    if any(n < 0 or not 0 <= n + a < 2 ** 31 for n, a in zip(lens, add)):
        status |= 4
    if starts is None:
        if packing[-1] > tokens:
            status |= 8
    elif any(s < 0 or e < s or e > tokens for s, e in zip(starts, starts[1:])):
        status |= 8
    if not (0 <= head < cap and 0 <= count <= cap) or count + drop > cap:
        status |= 16
    slots, positions = [-1] * tokens, [-1] * tokens
    free, tab = list(free_pages), [list(r) for r in tables]
    if status:
        return list(lens), list(ring), packing, slots, positions, status, free, tab
    taken = 0
    for b in range(B):
        for i in range(have[b], want[b]):
            tab[b][i] = free_pages[(head + taken) % cap]
            taken += 1
    given = 0
    for b in range(B):
        for i in range(want[b], have[b]):
            free[(head + count + given) % cap] = tables[b][i]
            given += 1
    for b in range(B):
        for t in range(packing[b], packing[b + 1]):
            off = t - packing[b] if offsets is None else offsets[t]
            if 0 <= off < add[b]:
                p = lens[b] + off
                slots[t] = tab[b][p // page] * page + p % page
                positions[t] = p
    after = [n + a for n, a in zip(lens, add)]
    return (after, [(head + taken) % cap, count - taken + given], packing, slots, positions, 0,
            free, tab)


def tree_reference(parents, starts, words):
    """tg_tree_mask on Python lists: rows of bits (a set of ancestors each) and depths."""
    n = len(parents)
    sees, depth = [set() for _ in range(n)], [-1] * n
    for s, e in zip(starts, starts[1:]):
        for i in range(min(e - s, 32 * words)):
            up = parents[s + i]
            if up == -1:
                sees[s + i], depth[s + i] = {i}, 0
            elif 0 <= up < i and depth[s + up] >= 0:
                sees[s + i], depth[s + i] = sees[s + up] | {i}, depth[s + up] + 1
    return sees, depth


def pack_bits(sees, words):
    """Sets of key indexes -> (tokens, words) int32."""
    rows = []
    for s in sees:
        w = [0] * words
        for j in s:
            w[j // 32] |= 1 << (j % 32)
        rows.append([x - 2 ** 32 if x >= 2 ** 31 else x for x in w])
    return torch.tensor(rows, dtype=torch.int64).to(torch.int32).view(len(sees), words)


def attention_reference(q, k, v, k_cache, v_cache, tables, lens, starts, sees, scale=None):
    """The attention by its definition in 64 bits (on the tensors' device), with what it does not
    see left out; sees: per row a list of drafted indexes, or None: up to its own.  Returns
    (out, bound): rows outside every request are NaN in out.

    The bound: probabilities are rounded to the tensors' type (half a step u of each, or half of
    fp16's smallest step, 2^-25, where they are subnormal), so the output is off by
    u sum w|v| + 2^-25 sum |v| / L at most, L = sum exp(s - max); rounding it costs u |out|.
    A score is a sum of D products in 32 bits, off by D 2^-23 scale sum |q k| at most (2^-23:
    the sum need not round to nearest), plus the multiply-add and the exponential's error, 2^-20
    of the exponent's size together; an error d of the scores changes the weights by 2d of
    themselves.  Sums and merges in 32 bits are covered by 2^-16 of sum w|v|.
    """
    n, heads, D = q.shape
    kv_heads, page = k_cache.shape[2], k_cache.shape[1]
    G = heads // kv_heads
    sc = scale if scale else 1.0 / math.sqrt(D)
    u = U[q.dtype]
    out = torch.full((n, heads, D), math.nan, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    for b in range(len(lens)):
        t0, t1 = starts[b], starts[b + 1]
        pos = torch.arange(lens[b], device=q.device)
        at = tables[b].long()[pos // page]
        kc = k_cache[at, pos % page].double()
        vc = v_cache[at, pos % page].double()
        for t in range(t0, t1):
            js = list(range(t - t0 + 1)) if sees is None else sorted(sees[t])
            js = torch.tensor([t0 + j for j in js if t0 + j < t1], dtype=torch.long,
                              device=q.device)
            keys = torch.cat([kc, k[js].double()])             # (N, kv_heads, D)
            vals = torch.cat([vc, v[js].double()])
            if keys.shape[0] == 0:
                out[t] = 0
                continue
            qq = q[t].double().view(kv_heads, G, D)
            s = torch.einsum("hgd,khd->hgk", qq, keys) * sc
            e = torch.exp(s - s.amax(2, keepdim=True))
            L = e.sum(2, keepdim=True)
            w = e / L
            o = torch.einsum("hgk,khd->hgd", w, vals)
            a = torch.einsum("hgk,khd->hgd", w, vals.abs())
            mag = torch.einsum("hgd,khd->hgk", qq.abs(), keys.abs()).amax(2, keepdim=True) * sc
            d = D * 2.0 ** -23 * mag + 2.0 ** -20 * (s.abs().amax(2, keepdim=True) + 1)
            tiny = 2.0 ** -25 * vals.abs().sum(0)[:, None] / L if q.dtype == torch.float16 else 0
            err = (u + 2 * d + 2.0 ** -16) * a + tiny + u * o.abs()
            out[t] = o.reshape(heads, D)
            bound[t] = (err * 1.01 + 2.0 ** -24).reshape(heads, D)
    return out, bound


def assert_attention(got, ref, bound, what=""):
    got = got.double().to(ref.device)
    rows = ~torch.isnan(ref).all(-1)
    nan = torch.isnan(ref) & rows[..., None]
    assert torch.equal(torch.isnan(got) & rows[..., None], nan), f"{what}: NaN places differ"
    fine = torch.isfinite(ref)
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), f"{what}: infinities differ"
    err = (got[fine] - ref[fine]).abs()
    assert bool(torch.isfinite(got[fine]).all()), f"{what}: not finite"
    over = err > bound[fine]
    if bool(over.any()):
        i = int(torch.argmax(err / bound[fine]))
        raise AssertionError(f"{what}: {int(over.sum())} of {err.numel()} over the bound; worst "
                             f"got {got[fine][i]} want {ref[fine][i]} bound {bound[fine][i]}")
