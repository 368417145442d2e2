"""The attention of drafted tokens over a paged cache by its definition in 64 bits, a request and a
key head at a time (long contexts and long prompts), with the bound of the error in 32- and 16-bit
arithmetic, and the division of the kernel's work restated."""
import math

import torch

from cache_helpers import U


def definition(q, k, v, k_cache, v_cache, tables, lens, starts, sees=None, scale=None):
    """o_t = sum_j w_tj v_j over the cached tokens of the request and the drafted tokens in
    sees[t] (a set of indexes; sees None: up to its own), w = softmax(scale q.k).

    Returns (out, bound, rows): rows (tokens,) says which rows belong to a request.  Infinities and
    NaN that a row sees enter as w_tj v_j does in IEEE arithmetic with the exact weight (0 where
    the score is -inf); what it does not see does not enter.

    The bound of a finite element, with u half a step of the type, L = sum exp(s - max), and N the
    keys of the row:
      probabilities   rounded to the type: u sum w|v|; in fp16 at least half a smallest step each.
                      They are held times 2^7 of the weight against the running maximum (which is
                      at most the row's), so that is 2^-25 2^-7 sum |v| / L.
      result          rounded once: u |out|.
      scores          sums of D products in 32 bits, D 2^-23 scale sum |q k|; the multiply-add and
                      the exponential, 2^-20 of (|s| + 1) together.  An error d of the scores
                      changes the weights by 2 d of themselves.
      sums            N / 16 products of 16 keys add up one after the other, each off by 2^-22 of
                      the running sum at most, and N / 64 rescales by 2^-22 each; joins of parts
                      and the division 2^-16: 2^-16 + N 2^-25.
    Keys with a score of -inf have weight 0 and are left out of |s| and sum |q k|.
    """
    n, heads, D = q.shape
    page, kv_heads = k_cache.shape[1], k_cache.shape[2]
    G = heads // kv_heads
    sc = scale if scale else 1.0 / math.sqrt(D)
    u = U[q.dtype]
    dev = q.device
    out = torch.zeros(n, heads, D, dtype=torch.float64, device=dev)
    bound = torch.zeros_like(out)
    rows = torch.zeros(n, dtype=torch.bool, device=dev)
    for b, L in enumerate(lens):
        t0, t1 = starts[b], starts[b + 1]
        T = t1 - t0
        if T <= 0:
            continue
        rows[t0:t1] = True
        pos = torch.arange(L, device=dev)
        at = tables[b].long()[pos // page]
        if sees is None:
            drafted = torch.ones(T, T, dtype=torch.bool, device=dev).tril()
        else:
            drafted = torch.zeros(T, T, dtype=torch.bool)
            for t in range(T):
                drafted[t, [j for j in sees[t0 + t] if j < T]] = True
            drafted = drafted.to(dev)
        vis = torch.cat([torch.ones(T, L, dtype=torch.bool, device=dev), drafted], 1)
        vis = vis[:, None].expand(T, G, L + T).reshape(T * G, L + T)
        N = vis.sum(1, keepdim=True)
        for h in range(kv_heads):
            keys = torch.cat([k_cache[at, pos % page, h], k[t0:t1, h]]).double()
            vals = torch.cat([v_cache[at, pos % page, h], v[t0:t1, h]]).double()
            qq = q[t0:t1, h * G:(h + 1) * G].reshape(T * G, D).double()
            s = (qq @ keys.T) * sc
            s = torch.where(vis, s, -math.inf)
            top = s.amax(1, keepdim=True) if L + T else torch.full_like(N, -math.inf).double()
            e = torch.exp(s - torch.where(N == 0, 0.0, top))
            tot = e.sum(1, keepdim=True)
            w = torch.where(N == 0, 0.0, e / tot)
            fin = torch.isfinite(vals)
            clean = torch.where(fin, vals, 0.0)
            o, a = w @ clean, w @ clean.abs()
            for j in torch.nonzero((~fin).any(1))[:, 0].tolist():
                odd = torch.where(fin[j], 0.0, w[:, j:j + 1] * vals[j])
                o = torch.where(vis[:, j:j + 1], o + odd, o)
            there = torch.isfinite(s)
            mag = torch.where(there, qq.abs() @ keys.abs().T, 0.0).amax(1, keepdim=True) * sc
            far = torch.where(there, s.abs(), 0.0).amax(1, keepdim=True)
            d = D * 2.0 ** -23 * mag + 2.0 ** -20 * (far + 1)
            tiny = 0.0
            if q.dtype == torch.float16:
                tiny = torch.where(N == 0, 0.0,
                                   2.0 ** -32 * (vis.double() @ clean.abs()) / tot)
            err = (u + 2 * d + 2.0 ** -16 + N * 2.0 ** -25) * a + tiny + u * o.abs()
            # 2^-24: a result in fp16's (or bf16's) subnormal range
            out[t0:t1, h * G:(h + 1) * G] = o.view(T, G, D)
            bound[t0:t1, h * G:(h + 1) * G] = (err * 1.01 + 2.0 ** -24).view(T, G, D)
    return out, bound, rows


def assert_rows(got, ref, bound, rows, what=""):
    """Every row of every request: the same NaN, the same infinities, and the rest within the
    bound, which has to be finite there."""
    assert int(rows.sum()) > 0
    got, ref, bound = got[rows].double(), ref[rows], bound[rows]
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN places differ"
    inf = torch.isinf(ref)
    assert torch.equal(torch.isinf(got), inf), f"{what}: places of infinities differ"
    assert torch.equal(got[inf], ref[inf]), f"{what}: infinities differ"
    fine = torch.isfinite(ref)
    assert bool(torch.isfinite(bound[fine]).all()), f"{what}: the bound says nothing"
    err, most = (got[fine] - ref[fine]).abs(), bound[fine]
    if bool((err > most).any()):
        i = int(torch.argmax(err / most))
        raise AssertionError(f"{what}: {int((err > most).sum())} of {err.numel()} over the bound; "
                             f"worst got {got[fine][i]} want {ref[fine][i]} bound {most[i]}")


def parts(trees, lens, kv_heads, group, ctas=148):
    """How the kernel divides its work: per CTA a list of (key tiles, key tiles of the unit, query
    tiles) for each part of its share."""
    tile = 128 // group
    units = []
    for n, c in zip(trees, lens):
        length = -(-c // 128) + -(-n // 128)
        q_tiles = -(-n // tile)
        for _ in range(kv_heads):
            units += [(length, min(2, q_tiles - 2 * p)) for p in range((q_tiles + 1) // 2)]
    share = -(-sum(n for n, _ in units) // ctas)
    out, cur, left = [], [], share
    for length, q_tiles in units:
        todo = length
        while todo:
            take = min(todo, left)
            cur.append((take, length, q_tiles))
            todo -= take
            left -= take
            if left == 0:
                out.append(cur)
                cur, left = [], share
    return out + [cur] if cur else out
