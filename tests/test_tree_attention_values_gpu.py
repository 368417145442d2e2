"""The attention of drafted trees where weights are very small or values are not finite."""
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
