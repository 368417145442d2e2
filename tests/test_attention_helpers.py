"""The references of the GPU tests against one another and against mistakes, on the CPU."""
import math
import random

import pytest
import torch

from attention_helpers import assert_rows, definition, parts
from cache_helpers import attention_reference, tree_reference

NAN, INF = float("nan"), float("inf")


def problem(trees, lens, masked, dtype=torch.float16, heads=2, group=2, dim=64, page=16):
    torch.manual_seed(1)
    rng = random.Random(1)
    starts = [0]
    for n in trees:
        starts.append(starts[-1] + n)
    n, width = starts[-1] + 2, max(-(-c // page) for c in lens) + 1        # two rows of padding
    kc, vc = torch.randn(2, width * len(lens), page, heads, dim).to(dtype)
    tables = torch.arange(width * len(lens), dtype=torch.int32).view(len(lens), width)
    q = torch.randn(n, heads * group, dim).to(dtype)
    k, v = torch.randn(2, n, heads, dim).to(dtype)
    sees = None
    if masked:
        parents = [rng.randint(max(-1, i - 3), i - 1) for t in trees for i in range(t)]
        sees = tree_reference(parents, starts, 4)[0] + [set(), set()]
    return [q, k, v, kc, vc, tables, lens, starts, sees]


@pytest.mark.parametrize("masked", [True, False])
@pytest.mark.parametrize("trees,lens", [([3, 0, 5], [40, 9, 0]), ([40], [100])])
def test_the_two_references_agree(trees, lens, masked):
    args = problem(trees, lens, masked)
    args[2][1, 0, 3] = NAN
    args[2][2, 1, 4] = -INF
    a, _ = attention_reference(*args)
    b, bound, rows = definition(*args)
    assert rows.tolist() == [i < args[7][-1] for i in range(len(rows))]
    assert torch.allclose(a[rows], b[rows], rtol=1e-9, atol=1e-12, equal_nan=True)
    assert_rows(b.half(), b, bound, rows)


def test_mistakes_are_found():
    """What a wrong kernel might give: in a NaN row, beside an infinite key, in an idle row, and a
    weight that is lost."""
    args = problem([4], [60], True)
    args[0][2, 3, 7] = NAN                                  # a query
    args[3][1, 5, 1, 5] = INF                               # a cached key
    ref, bound, rows = definition(*args)
    assert bool(torch.isnan(ref[2, 3]).all())
    infinite = args[0][:4, 2:, 5] > 0                       # scores of +inf
    assert torch.equal(torch.isnan(ref[:4, 2:]).all(-1), infinite | torch.isnan(args[0][:4, 2:, 7]))
    assert_rows(ref, ref, bound, rows)
    fine = torch.nonzero(torch.isfinite(ref[:4]))
    for at, wrong in ((torch.tensor([2, 3, 0]), 123.0), (fine[0], -999.0), (fine[-1], NAN),
                      (fine[5], INF), (fine[7], float(ref[tuple(fine[7])]) + 0.01)):
        got = ref.clone()
        got[tuple(at)] = wrong
        with pytest.raises(AssertionError):
            assert_rows(got, ref, bound, rows)


def test_a_row_without_keys_is_zero_and_scores_of_minus_infinity_weigh_nothing():
    args = problem([3], [0], True, heads=1, group=1)
    args[8][1] = set()
    args[1][0, 0, 0], args[0][:, :, 0] = -INF, 1.0
    args[8][2] = {0, 2}
    ref, bound, rows = definition(*args)
    assert int(torch.count_nonzero(ref[1])) == 0
    assert torch.allclose(ref[2, 0], args[2][2, 0].double())       # only the second key counts
    assert math.isnan(ref[0, 0, 0])                                 # 0 / 0


def test_parts_cover_the_work():
    got = parts([6, 70, 0, 1], [1000, 300, 5, 0], 2, 4, ctas=7)
    tiles = 2 * (9 + 2 * 4 + 1)             # 70 tokens of 4 heads: three query tiles, two pairs
    assert sum(n for c in got for n, _, _ in c) == tiles
    assert all(sum(n for n, _, _ in c) == -(-tiles // 7) for c in got[:-1])
