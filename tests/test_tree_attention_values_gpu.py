"""The attention of drafted trees where weights are very small or values are not finite."""
import math

import pytest
import torch

from attention_helpers import assert_rows, definition, parts
from cache_helpers import pack_bits
from test_tree_attention_gpu import DEV, INF, NAN, Problem

pytestmark = pytest.mark.gpu


def check(p, what="", **kw):
    ref, bound, rows = definition(p.q, p.k, p.v, p.kc, p.vc, p.tables, p.lens, p.starts, p.sees,
                                  kw.get("scale"))
    out = p.run(**kw)
    assert_rows(out, ref, bound, rows, what)
    return out


def set_cached(p, b, pos, cache, head, dim, value):
    page = int(p.tables[b, pos // p.page])
    cache[page, pos % p.page, head, dim] = value


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("tree", [1, 40])
def test_many_small_weights_beside_dominant_ones(tree, dim, dtype):
    """32768 keys of weight 2^-25.2 beside two dominant ones, whose values are 0: the small
    weights make up the whole output.  148 requests that share one context give each CTA a whole
    unit, so that small and dominant ones meet under one running maximum."""
    n, B = 32768, 148
    p = Problem([tree], [n], heads=1, group=4, dim=dim, page=64, dtype=dtype, masked=False)
    p.q.zero_()
    p.q[..., 0] = 1.0
    for c in (p.k, p.kc):
        c.nan_to_num_().zero_()
    for c in (p.v, p.vc):
        c.nan_to_num_().fill_(1.0)
    for pos in (5, 200):                        # key tiles 0 and 1: one of either softmax group
        set_cached(p, 0, pos, p.kc, 0, 0, 17.5)
        set_cached(p, 0, pos, p.vc, 0, slice(None), 0.0)
    p.q, p.k, p.v = (x.repeat(B, 1, 1) for x in (p.q, p.k, p.v))
    p.tables = p.tables.repeat(B, 1)
    p.lens, p.trees = [n] * B, [tree] * B
    p.starts = [tree * b for b in range(B + 1)]
    assert all(len(c) == 1 and c[0][0] == c[0][1] for c in parts(p.trees, p.lens, 1, 4))
    check(p, scale=1.0)


def replicate(p, B):
    """The same request B times (sharing its pages)."""
    n = p.trees[0]
    p.q, p.k, p.v = (x[:n].repeat(B, 1, 1) for x in (p.q, p.k, p.v))
    p.mask = p.mask[:n].repeat(B, 1)
    p.sees = p.sees[:n] * B
    p.tables = p.tables[:1].repeat(B, 1)
    p.lens, p.trees, p.starts = p.lens * B, p.trees * B, [n * b for b in range(B + 1)]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("tree", [6, 70, 150])
def test_infinite_values_of_small_weight(tree, dtype):
    """A drafted token with an infinite value makes the rows that see it infinite, however small
    its weight is beside the context's, whether its unit is divided or not."""
    p = Problem([tree], [1000], heads=2, group=2, dim=64, dtype=dtype, seed=31)
    p.q[..., 0] = 8.0
    p.k[..., 0] = 0.0
    set_cached(p, 0, 100, p.kc, slice(None), 0, 512.0)      # some 512 above all others
    p.v[2, 0, 5] = INF
    p.v[tree - 1, 1, 7] = -INF
    p.sees[tree - 1] = p.sees[tree - 1] | {2}
    p.mask = pack_bits(p.sees, p.words).to(DEV)
    assert all(c[0][0] < c[0][1] for c in parts(p.trees, p.lens, 2, 2))
    out = check(p, "divided")
    assert bool(torch.isinf(out).any())
    replicate(p, 296)
    whole = [n == u for c in parts(p.trees, p.lens, 2, 2) for n, u, _ in c]
    assert sum(whole) > len(whole) // 2
    check(p, "many requests")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("tree", [6, 70, 150])
def test_values_of_keys_with_weight_zero(tree, dtype):
    """A drafted token whose score is -inf has weight 0: a finite value does not enter, and an
    infinite one makes the element NaN (0 times infinity)."""
    p = Problem([tree], [1000], heads=2, group=2, dim=64, dtype=dtype, seed=32)
    p.q[..., 3] = 1.0
    p.k[2, 0, 3] = -INF
    check(p, "finite value")
    p.v[2, 0, 5] = INF
    p.v[2, 0, 6] = -INF
    p.v[1, 0, 9] = INF                                      # of positive weight
    p.sees[tree - 1] = p.sees[tree - 1] | {1, 2}
    p.mask = pack_bits(p.sees, p.words).to(DEV)
    out = check(p, "divided")
    assert bool(torch.isnan(out).any()) and bool(torch.isinf(out).any())
    replicate(p, 296)
    check(p, "many requests")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("trees,lens", [([6, 3], [40, 300]), ([40], [700]), ([5, 130], [3000, 60])])
def test_queries_and_keys_that_are_not_finite(trees, lens, dtype):
    """A NaN query makes its own (token, head) row NaN and no other.  An infinite cached key makes
    rows with a score of +inf NaN and has weight 0 in those with -inf; so does a drafted one in
    the rows that see it."""
    p = Problem(trees, lens, heads=2, group=4, dim=64, dtype=dtype, seed=23)
    p.q[2, 3, 7] = NAN
    out = check(p, "query")
    assert bool(torch.isnan(out[2, 3]).all()) and int(torch.isnan(out).sum()) == 64
    p.q[2, 3, 7] = 0.5
    set_cached(p, 0, 33, p.kc, 1, 5, INF)
    out = check(p, "cached key")
    nan = torch.isnan(out[:trees[0], 4:]).all(-1)
    assert torch.equal(nan, p.q[:trees[0], 4:, 5] > 0) and bool(nan.any()) and not bool(nan.all())
    p.k[1, 0, 9] = -INF
    check(p, "drafted key")


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("dtype,log_a,log_b", [
    (torch.float16, 4, 2), (torch.float16, 9, 9), (torch.float16, 12, 10), (torch.float16, 15, 14),
    (torch.bfloat16, 9, 9), (torch.bfloat16, 15, 15), (torch.bfloat16, 30, 30)])
@pytest.mark.parametrize("tree,n", [(1, 1500), (40, 700), (6, 0)])
def test_scores_far_from_zero(tree, n, dtype, log_a, log_b, sign):
    """Scores of 2^13 to 2^67, exact in 32 bits and distinct by far: the output is the mean of the
    values of the two keys that share the largest, whatever the scores' rounding against the
    running maximum.  With u half a step of the type: the two weights are rounded to the type
    and their sum is not, so w = (1 + d) / 2 with |d| <= u each, u (|v0| + |v1|) / 2 together;
    32-bit sums and the division add 2^-20 of that size at most, the result's rounding u of it."""
    p = Problem([tree], [n], heads=2, group=2, dim=64, dtype=dtype, seed=51, masked=False)
    g = torch.Generator(DEV).manual_seed(tree + n)
    p.q.fill_(2.0 ** log_a)
    level = torch.randint(0, 62, (n + tree,), generator=g, device=DEV)
    top = [100, n - 7] if n else [0, 1]
    level[top] = 63
    key = ((64 + level) / 64 if sign > 0 else (level - 128) / 64) * 2.0 ** log_b
    pos = torch.arange(n, device=DEV)
    page = p.tables[0].long()
    p.kc[page[pos // 16], pos % 16] = key[:n, None, None].to(dtype)
    p.k.copy_(key[n:, None, None].expand_as(p.k))
    v = [(p.vc[page[j // 16], j % 16] if n else p.v[j]).double() for j in top]
    want = ((v[0] + v[1]) / 2).repeat_interleave(2, 0)
    size = (v[0].abs() + v[1].abs()).repeat_interleave(2, 0)
    u = torch.finfo(dtype).eps / 2
    most = u * want.abs() + (u / 2 + 2.0 ** -20) * size * (1 + u) + 2.0 ** -24
    rows = range(0 if n else 1, tree)           # without a context the first row sees one key
    out = p.run(scale=1.0)
    for t in rows:
        assert bool(((out[t].double() - want).abs() <= most).all()), t
    B = 100                                     # whole units as well
    p.q, p.k, p.v = (x.repeat(B, 1, 1) for x in (p.q, p.k, p.v))
    p.tables, p.lens = p.tables.repeat(B, 1), p.lens * B
    p.starts = [tree * b for b in range(B + 1)]
    out = p.run(scale=1.0).view(B, tree, 4, 64)
    for t in rows:
        assert bool(((out[:, t].double() - want).abs() <= most).all()), t


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("tree", [1, 40])
def test_far_scores_one_step_of_32_bits_apart(tree, dtype):
    """Scores of 2^26 and, late in the context, 2^26 + 8: the next number in 32 bits, 11.5 more in
    log2 units.  The running maximum has to move, or the weight overflows fp16.  The weights are
    exact but for u each; sums and exponentials 2^-16."""
    n, B = 3000, 148
    p = Problem([tree], [n], heads=1, group=4, dim=64, page=16, dtype=dtype, masked=False)
    p.q.zero_()
    p.q[..., 0], p.q[..., 1] = 2.0 ** 13, 1.0
    for c in (p.k, p.v, p.kc, p.vc):
        c.nan_to_num_().zero_()
    p.k[..., 0] = p.kc[..., 0] = 2.0 ** 13
    p.vc[..., 0] = 1.0
    late = (1300, 2500)
    for pos in late:
        set_cached(p, 0, pos, p.kc, 0, 1, 8.0)
        set_cached(p, 0, pos, p.vc, 0, 0, 0.0)
        set_cached(p, 0, pos, p.vc, 0, 1, 1.0)
    p.q, p.k, p.v = (x.repeat(B, 1, 1) for x in (p.q, p.k, p.v))
    p.tables, p.lens, p.trees = p.tables.repeat(B, 1), [n] * B, [tree] * B
    p.starts = [tree * b for b in range(B + 1)]
    assert all(len(c) == 1 and c[0][0] == c[0][1] for c in parts(p.trees, p.lens, 1, 4))
    out = p.run(scale=1.0).view(B, tree, 4, 64).double()
    u = torch.finfo(dtype).eps / 2
    small = 2.718281828459045 ** -8
    for t in range(tree):
        total = 2 + (n - 2 + t + 1) * small
        for e, want in ((0, (n - 2) * small / total), (1, 2 / total), (2, 0.0)):
            assert bool(((out[:, t, :, e] - want).abs() <= (2 * u + 2.0 ** -16) * want).all())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("scale,log_a,step", [(1.0, 13, 8.0), (2.0 ** -20, 13, 8.0),
                                              (2.0 ** 99, 15, 128.0)])
def test_far_scores_in_a_divided_unit(scale, log_a, step, dtype):
    """One request whose key tiles lie in as many CTAs: parts with neighbouring maxima of 2^26 and
    2^26 + 8 (or 2^30 and 2^30 + 128, beyond 32 bits after a scale of 2^99) are joined by their
    distance."""
    n = 3000
    p = Problem([1], [n], heads=1, group=4, dim=64, page=16, dtype=dtype, masked=False)
    p.q.zero_()
    p.q[..., 0], p.q[..., 1] = 2.0 ** log_a, 1.0
    for c in (p.k, p.v, p.kc, p.vc):
        c.nan_to_num_().zero_()
    p.k[..., 0] = p.kc[..., 0] = 2.0 ** log_a
    p.vc[..., 0] = 1.0
    for pos in (1300, 2500):
        set_cached(p, 0, pos, p.kc, 0, 1, step)
        set_cached(p, 0, pos, p.vc, 0, 0, 0.0)
        set_cached(p, 0, pos, p.vc, 0, 1, 1.0)
    assert all(len(c) == 1 and c[0][0] == 1 for c in parts(p.trees, p.lens, 1, 4))
    out = p.run(scale=scale)[0].double()
    u = torch.finfo(dtype).eps / 2
    small = math.exp(-step * scale)
    total = 2 + (n - 2 + 1) * small
    for e, want in ((0, (n - 2) * small / total), (1, 2 / total), (2, 0.0)):
        assert bool(((out[:, e] - want).abs() <= (2 * u + 2.0 ** -16) * want).all()), (e, want)
