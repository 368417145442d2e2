"""The attention's main loop: parts of many key tiles, many parts a CTA, prompts and batches of
single tokens. What a call does is the division of its work, so each test states the parts that it
is about."""

import pytest
import torch

from attention_helpers import assert_rows, definition, parts
from cache_helpers import pack_bits, tree_reference
from tensor_core_gemm_fp16_b200 import binding
from test_tree_attention_gpu import DEV, INF, NAN, Problem

pytestmark = pytest.mark.gpu
LONG = 16       # key tiles from which on unused query rows are zeroed


def check(p, what="", **kw):
    ref, bound, rows = definition(p.q, p.k, p.v, p.kc, p.vc, p.tables, p.lens, p.starts, p.sees,
                                  kw.get("scale"))
    out = p.run(**kw)
    assert_rows(out, ref, bound, rows, what)
    assert bool((out[p.starts[-1]:] == 7.0).all()), "rows behind the last request"
    return out


def runs_of_pages(page):
    """Key tiles that one run of 32 page entries fills."""
    return max(1, 32 * page // 128) if page < 128 else 32


def long_parts(p, heads, group, page, runs):
    """Parts that zero query rows and go through `runs` runs of page entries."""
    got = [x for c in parts(p.trees, p.lens, heads, group) for x in c]
    need = max(LONG, runs_of_pages(page) * runs + 1)
    return [x for x in got if x[0] >= need]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256])
def test_long_parts(page, dim, dtype):
    """Ragged contexts of up to 11,000 tokens, with one and two query tiles a unit: each CTA has
    some 70 key tiles, every ring stage and page buffer is used many times."""
    heads, group = 8, 4
    trees = [1, 27, 40, 5, 64, 33, 2, 16, 3, 50, 1, 32, 7, 90, 20, 11]
    lens = [11000 - 511 * (b % 5) - 37 * b for b in range(16)]
    p = Problem(trees, lens, heads=heads, group=group, dim=dim, page=page, dtype=dtype, seed=page,
                pad=2, layout="interleaved" if page in (16, 128) else "plain")
    # reuse of both buffers of page entries: three runs (pages of 128 and more: two)
    found = long_parts(p, heads, group, page, 3 if page < 128 else 2)
    assert {t for _, _, t in found} == {1, 2}
    check(p)
    if page == 16:
        p.mask = p.sees = None
        check(p, "without a mask")


@pytest.mark.parametrize("tree", [3, 40])
@pytest.mark.parametrize("dim", [64, 128])
def test_three_runs_of_large_pages(dim, tree):
    """Parts of more than 64 key tiles with pages of 128: the third run of page entries."""
    p = Problem([tree] * 19, [13000 + 100 * b for b in range(19)], heads=8, group=4, dim=dim,
                page=128, seed=tree, dtype=torch.bfloat16)
    assert len(long_parts(p, 8, 4, 128, 2)) > 30
    check(p)


@pytest.mark.parametrize("step", [0.02, -0.02, 0.3])
@pytest.mark.parametrize("tree,group", [(1, 1), (6, 4), (40, 4)])
def test_scores_that_grow_or_fall_along_a_long_context(tree, group, step):
    """Scores move by 64 step a half tile: growing ones raise the running maximum on every half
    tile (0.3: by more than fp16's range), falling ones never."""
    heads, n = 8, 9000
    p = Problem([tree] * 19, [n - 100 * b for b in range(19)], heads=heads, group=group, dim=64,
                page=32, seed=6)
    p.q[..., 0] = 4.0
    ramp = step * torch.arange(n, device=DEV) / 4
    for b, c in enumerate(p.lens):
        pos = torch.arange(c, device=DEV)
        p.kc[p.tables[b].long()[pos // 32], pos % 32, :, 0] = ramp[:c].half()[:, None]
    assert len(long_parts(p, heads, group, 32, 2)) > 30
    check(p, scale=1.0)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
def test_many_short_units(dim, dtype):
    """Hundreds of requests with contexts of none to a few tiles: a CTA has more than ten parts,
    of one and two query tiles in turn."""
    B, heads, group = 700, 4, 4
    trees = [(1, 40, 0, 3, 33, 64, 2)[b % 7] for b in range(B)]
    lens = [(0, 130, 50, 500, 64, 129, 0, 300, 1)[b % 9] for b in range(B)]
    p = Problem(trees, lens, heads=heads, group=group, dim=dim, seed=40, dtype=dtype, pad=3)
    assert min(len(c) for c in parts(trees, lens, heads, group)[:-1]) > 10
    check(p)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("dim", [64, 128])
def test_a_decoding_step_of_many_requests(dim, page, dtype):
    """One token each, no mask, ragged contexts of up to 8192 tokens."""
    B, heads, group = 64, 8, 4
    lens = [(8192 * (b + 1) // B - b * b % 97) for b in range(B)]
    lens[5] = 0
    p = Problem([1] * B, lens, heads=heads, group=group, dim=dim, page=page, dtype=dtype, seed=41,
                masked=False)
    assert long_parts(p, heads, group, page, 1)
    check(p)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("trees,lens,heads,group", [
    ([2048], [0], 4, 4), ([1500, 1, 0, 700], [0, 40, 9, 8000], 2, 4), ([4097], [0], 2, 1),
    ([513, 1025], [1000, 127], 8, 3), ([1200], [65], 1, 8)])
def test_prompts(trees, lens, heads, group, dtype):
    """Many new tokens without a mask: a token sees those up to itself.  Values and keys that are
    not finite reach the rows from theirs on and no others."""
    p = Problem(trees, lens, heads=heads, group=group, dim=128, page=16, dtype=dtype, seed=42,
                masked=False, pad=1)
    check(p)
    n = trees[0]
    p.v[n - 3, 0, 5] = INF
    p.v[n // 2, heads - 1, 100] = NAN
    p.v[n // 2 + 200, 0, 17] = -INF
    out = check(p, "values")
    assert bool(torch.isfinite(out[:n // 2]).all())
    p.k[n - 100, 0, 9] = NAN
    out = check(p, "key")
    assert bool(torch.isfinite(out[:n // 2]).all())
    assert bool(torch.isnan(out[n - 100:n, :group]).all())


def test_a_prompt_as_a_masked_chain():
    """The chain's mask says the same as no mask."""
    p = Problem([1000, 300], [200, 3000], heads=2, group=4, dim=128, seed=43, masked=False)
    want = p.run()
    parents = [i - 1 for n in p.trees for i in range(n)]
    p.mask = binding.tree_mask(torch.tensor(parents, dtype=torch.int32, device=DEV),
                               torch.tensor(p.starts, dtype=torch.int32, device=DEV), 32)[0]
    assert torch.equal(p.run(), want)


def test_a_long_batch_does_not_vary_and_replays():
    """Repeated calls, and a captured one, give the same bits."""
    p = Problem([9, 40, 1, 64] * 5, [6000, 9000, 3000, 7000] * 5, heads=4, group=4, dim=128,
                page=16, seed=44, dtype=torch.bfloat16)
    first = check(p)
    lens = torch.tensor(p.lens, dtype=torch.int32, device=DEV)
    starts = torch.tensor(p.starts, dtype=torch.int32, device=DEV)
    out = torch.zeros_like(first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.tree_attention(p.q, p.k, p.v, p.kc, p.vc, p.tables, lens, starts, p.mask, out=out)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first) and torch.equal(p.run(), first)


def test_masks_with_starts_out_of_range():
    """Clamped starts: the masks of the requests that are left, and empty rows outside them."""
    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)

    for starts, clamped in (([-5, 2, 2 ** 31 - 1], [0, 2, 3]), ([2, 1, 0], [2, 2, 2]),
                            ([-9, -1, 2], [0, 0, 2]), ([1, 3, 3], [1, 3, 3])):
        parents = [-1, 0, 1]
        out = (torch.full((3, 2), 77, dtype=torch.int32, device=DEV),
               torch.full((3,), 77, dtype=torch.int32, device=DEV))
        m, d = binding.tree_mask(i32(parents), i32(starts), 2, out=out)
        sees, depth = tree_reference(parents, clamped, 2)
        assert d.tolist() == depth and torch.equal(m.cpu(), pack_bits(sees, 2))
