"""cache_plan with a packing: a request cannot append more tokens than it has in it."""
import pytest

from tensor_core_gemm_fp16_b200 import binding
from test_cache_gpu import run_plan

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("offsets", [None, [0, 1, 2, 0, 1, 0, 0]])
@pytest.mark.parametrize("add,fits", [([3, 2], True), ([0, 0], True), ([-16, 2], True),
                                      ([4, 2], False), ([3, 3], False), ([-16, 3], False),
                                      ([0, 2 ** 31 - 40], False)])
def test_appended_tokens_are_in_the_packing(add, fits, offsets):
    lens, ring, free = [16, 33], [3, 3], [0, 1, 2, 3, 4, 5]
    tables, starts = [[2, 9, 9, 9], [1, 0, 5, 9]], [0, 3, 5]
    got = run_plan(lens, add, ring, free, tables, 16, 7, starts=starts, offsets=offsets)
    assert bool(got[5] & binding.TG_PLAN_BAD_TOKENS) == (not fits)
    if fits:
        assert got[5] == 0 and got[0] == [n + a for n, a in zip(lens, add)]
        # every appended place has its token
        for b in range(2):
            kept = [p for p in got[4][starts[b]:starts[b + 1]] if p >= 0]
            assert kept == list(range(lens[b], lens[b] + max(add[b], 0)))
    else:
        assert got[0] == lens and got[1] == ring and got[6] == free and got[7] == tables
        assert got[3] == [-1] * 7 and got[4] == [-1] * 7
