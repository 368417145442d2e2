"""The attention of drafted trees over the paged cache against its definition in 64 bits, within
the bound that cache_helpers.attention_reference derives."""
import random

import pytest
import torch

from cache_helpers import assert_attention, attention_reference, pack_bits, plan_reference, \
    tree_reference
from tensor_core_gemm_fp16_b200 import binding

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
NAN, INF = float("nan"), float("inf")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Problem:
    """A packed batch over a paged cache whose unused rows and pages hold NaN."""

    def __init__(self, trees, lens, *, heads=2, group=4, dim=128, page=16, dtype=torch.float16,
                 masked=True, layout="plain", seed=0, pad=0, spare=3, scale=1.0):
        g = torch.Generator(DEV).manual_seed(seed)
        rng = random.Random(seed)
        self.trees, self.lens, self.dtype, self.page = trees, lens, dtype, page
        self.starts = [0]
        for n in trees:
            self.starts.append(self.starts[-1] + n)
        n = self.starts[-1] + pad
        used = [-(-c // page) for c in lens]
        pages = sum(used) + spare
        order = list(range(pages))
        rng.shuffle(order)
        width = max(used, default=0) + 1
        tab, at = [], 0
        for u in used:
            # entries that are not in use are junk
            tab.append(order[at:at + u] + [rng.choice([-1, pages, 2 ** 31 - 1, 0])] * (width - u))
            at += u
        self.tables = i32(tab).view(len(lens), width)
        if layout == "plain":
            c = torch.full((2, pages, page, heads, dim), NAN, dtype=dtype, device=DEV)
            self.kc, self.vc = c[0], c[1]
        elif layout == "interleaved":
            c = torch.full((pages, 2, page, heads, dim), NAN, dtype=dtype, device=DEV)
            self.kc, self.vc = c[:, 0], c[:, 1]
        elif layout == "padded":        # heads 8 elements further apart than they are wide
            c = torch.full((2, pages, page, heads, dim + 8), NAN, dtype=dtype, device=DEV)
            self.kc, self.vc = c[0, ..., :dim], c[1, ..., :dim]
        else:
            c = torch.full((2, pages, heads, page, dim), NAN, dtype=dtype, device=DEV)
            self.kc, self.vc = c[0].transpose(1, 2), c[1].transpose(1, 2)
        for b, c in enumerate(lens):
            pos = torch.arange(c, device=DEV)
            p = self.tables[b].long()[pos // page]
            for cache in (self.kc, self.vc):
                cache[p, pos % page] = torch.randn(c, heads, dim, generator=g, device=DEV).to(dtype)
        qkv = torch.randn(n, heads * (group + 2), dim, generator=g, device=DEV).to(dtype)
        self.q, self.k, self.v = qkv.split([heads * group, heads, heads], dim=1)
        self.q *= scale
        if layout == "plain":
            self.q, self.k, self.v = (x.contiguous() for x in (self.q, self.k, self.v))
        self.words = max(1, (max(trees, default=1) + 31) // 32)
        self.sees = self.mask = None
        if masked:
            parents = []
            for t in trees:
                parents += [rng.randint(max(-1, i - 4), i - 1) for i in range(t)]
            self.sees = tree_reference(parents, self.starts, self.words)[0] + [set()] * pad
            self.mask = pack_bits(self.sees, self.words).to(DEV)

    def run(self, **kw):
        kw.setdefault("out", torch.full_like(self.q, 7.0).contiguous())
        out = binding.tree_attention(self.q, self.k, self.v, self.kc, self.vc, self.tables,
                                     i32(self.lens), i32(self.starts), self.mask, **kw)
        torch.cuda.synchronize()
        assert binding.tg_gemm_check_error(torch.cuda.current_stream().cuda_stream) == binding.TG_OK
        return out

    def check(self, what="", **kw):
        ref, bound = attention_reference(self.q, self.k, self.v, self.kc, self.vc, self.tables,
                                         self.lens, self.starts, self.sees, kw.get("scale"))
        out = self.run(**kw)
        assert_attention(out, ref, bound, what)
        assert bool((out[self.starts[-1]:] == 7.0).all()), "rows behind the last request"
        return out


SHAPES = [  # trees, lens, heads, group, page
    ([1], [0], 1, 1, 16),                               # one token that sees itself alone
    ([1], [1], 1, 1, 8),
    ([1, 1, 1], [15, 16, 17], 2, 4, 16),
    ([3, 1, 7], [127, 128, 129], 2, 4, 32),
    ([5, 0, 2, 0, 0, 9], [300, 50, 0, 0, 7, 511], 1, 8, 64),    # idle requests in between
    ([64], [700], 2, 4, 16),                            # two query tiles
    ([33, 40], [260, 90], 2, 4, 128),                   # two tiles, the second nearly empty
    ([100], [333], 1, 3, 256),                          # group 3: 126 rows of a tile
    ([130, 20], [40, 1000], 3, 1, 8),                   # more drafted tokens than a key tile
    ([17], [200], 1, 7, 16),
    ([9, 4], [65, 900], 1, 16, 16),
    ([3], [140], 1, 128, 32),                           # a token a tile: three tiles
    ([2, 1], [30, 3000], 1, 65, 16),
]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_shapes(shape, dim, dtype):
    trees, lens, heads, group, page = SHAPES[shape]
    for masked in (True, False):
        Problem(trees, lens, heads=heads, group=group, page=page, dim=dim, dtype=dtype,
                masked=masked, seed=shape, pad=3 if shape % 2 else 0).check(f"masked={masked}")


@pytest.mark.parametrize("page", [8, 16, 128, 256])
@pytest.mark.parametrize("layout", ["interleaved", "heads_first", "padded"])
@pytest.mark.parametrize("dim", [64, 128])
def test_strided_caches_and_projections(dim, layout, page):
    p = Problem([6, 20, 1], [90, 400, 33], heads=3, group=2, dim=dim, layout=layout, seed=3, pad=2,
                page=page)
    wide = torch.full((p.q.shape[0], p.q.shape[1] + 1, dim + 8), 7.0, dtype=p.dtype, device=DEV)
    p.check(layout, out=wide[:, 1:, :dim])
    assert bool((wide[:, 0] == 7.0).all()) and bool((wide[:, :, dim:] == 7.0).all())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("seed", range(6))
def test_random_batches(seed, dtype):
    rng = random.Random(seed)
    B = rng.choice([1, 5, 40])
    trees = [rng.choice([0, 1, 2, rng.randint(0, 70)]) for _ in range(B)]
    lens = [rng.choice([0, rng.randint(0, 300), rng.randint(0, 1500)]) for _ in range(B)]
    Problem(trees, lens, heads=rng.choice([1, 2, 5]), group=rng.choice([1, 2, 4, 6, 8]),
            dim=rng.choice([64, 128]), page=rng.choice([8, 16, 32, 64, 128, 256]), dtype=dtype,
            masked=rng.random() < 0.7, layout=rng.choice(["plain", "interleaved"]), seed=seed,
            pad=rng.choice([0, 5])).check()


@pytest.mark.parametrize("tree", [1, 70])
def test_more_requests_than_threads(tree):
    """The CTAs' sums over the requests take several rounds; most requests are idle."""
    B = 1000
    trees, lens = [0] * B, [13] * B
    for b in (0, 319, 320, 321, 500, 639, 640, 999):
        trees[b], lens[b] = 1 + b % 3, 100 + b
    trees[700] = tree
    Problem(trees, lens, heads=1, group=2, dim=64, seed=tree).check()


def test_a_long_context_is_divided_over_all_sms():
    p = Problem([3, 65], [20000, 9000], heads=1, group=4, dim=128, page=64, seed=4,
                dtype=torch.bfloat16)
    p.check()


def test_explicit_scale_and_large_scores():
    """Nearly one-hot rows: the running maximum moves by far more than 2^8 between tiles."""
    p = Problem([6, 30], [700, 300], heads=2, group=2, dim=64, seed=5)
    for scale in (1.0, 0.01, 3.0):
        p.check(f"scale {scale}", scale=scale)


def test_growing_scores_rescale_on_every_tile():
    p = Problem([2], [1000], heads=1, group=1, dim=64, seed=6)
    p.q.zero_()
    p.q[..., 0] = 1.0
    pos = torch.arange(1000, device=DEV)
    page = p.tables[0].long()[pos // 16]
    p.kc[page, pos % 16, :, 0] = torch.linspace(0, 200, 1000, device=DEV).half()[:, None]
    p.check(scale=1.0)


def test_one_visible_key_is_copied_exactly():
    p = Problem([5, 3], [0, 0], heads=2, group=4, seed=7)
    p.sees = [{i % 5} if i < 5 else {i - 5} for i in range(8)]
    p.mask = pack_bits(p.sees, 1).to(DEV)
    out = p.run()
    assert torch.equal(out.view(8, 2, 4, 128), p.v[:, :, None].expand(8, 2, 4, 128))


def test_rows_that_see_nothing_are_zero():
    p = Problem([5, 40, 3], [0, 0, 50], heads=2, group=4, seed=8)
    p.sees = [set() if i % 2 else s for i, s in enumerate(p.sees)]
    p.mask = pack_bits(p.sees, p.words).to(DEV)
    out = p.check()
    assert int(torch.count_nonzero(out[1:45:2])) == 0
    assert int(torch.count_nonzero(out[45:])) > 0            # the context is always seen


def test_mask_bits_past_the_request_are_ignored():
    """A mask of ones everywhere: only the request's own drafted tokens count."""
    p = Problem([5, 40, 3], [20, 0, 50], heads=1, group=4, seed=9)
    p.mask = torch.full_like(p.mask, -1)
    p.sees = [set(range(n)) for n in p.trees for _ in range(n)]
    p.check()


def test_tokens_past_the_masks_width_are_not_seen():
    p = Problem([50], [20], heads=1, group=2, seed=10)
    p.mask = p.mask[:, :1].contiguous()
    p.sees = [{j for j in s if j < 32} for s in p.sees]
    p.check()
    p.mask = torch.cat([p.mask, p.mask], 1)[:, :1]           # rows further apart
    p.check()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("trees,lens", [([6], [40]), ([70], [200]), ([150], [3]),
                                        ([6, 6], [5000, 0])])
def test_values_that_are_not_finite(trees, lens, dtype):
    """Infinities and NaN in drafted tokens: rows that see them get what the sum gives, and
    those that do not are not touched (the other unused rows are NaN throughout)."""
    p = Problem(trees, lens, heads=2, group=4, dim=128, dtype=dtype, seed=11)
    n = p.q.shape[0]
    p.v[2, 0, 5] = INF
    p.v[3, 0, 5] = -INF
    p.v[4, 1, 127] = NAN
    p.v[1, 1, 64] = -INF
    p.v[n - 1, 0, 0] = INF
    p.check("values")
    p.k[n - 2, 1, 3] = NAN                                   # a key: rows that see it are NaN
    ref, bound = attention_reference(p.q, p.k, p.v, p.kc, p.vc, p.tables, p.lens, p.starts, p.sees)
    out = p.run()
    sees = torch.tensor([n - 2 - p.starts[len(trees) - 1] in s and i >= p.starts[len(trees) - 1]
                         for i, s in enumerate(p.sees)], device=DEV)
    heads = slice(4, 8)
    assert bool(torch.isnan(out[sees][:, heads]).all())
    rest = ~sees
    ref[sees] = NAN
    bound[sees] = 0
    assert_attention(out[rest], ref[rest], bound[rest], "rows that do not see the NaN key")


def test_nan_in_the_context_reaches_every_row_of_the_request():
    p = Problem([4, 4], [300, 300], heads=1, group=2, dim=64, seed=12)
    page = p.tables[0].long()[200 // 16]
    p.vc[page, 200 % 16, 0, 9] = NAN
    p.check()
    p.vc[page, 200 % 16, 0, 9] = 1.0
    p.kc[page, 200 % 16, 0, 9] = NAN
    out = p.run()
    assert bool(torch.isnan(out[:4]).all()) and bool(torch.isfinite(out[4:]).all())


@pytest.mark.parametrize("trees,lens", [([6, 3], [40, 300]), ([40], [700])])
def test_rows_that_are_not_finite_stay_alone(trees, lens):
    """A NaN query makes its own (token, head) row NaN and no other; an infinite key makes the
    rows that see it with a score of +inf NaN, and has weight 0 where the score is -inf."""
    p = Problem(trees, lens, heads=2, group=4, dim=64, seed=23)
    p.q[2, 3, 7] = NAN
    p.check()
    p.q[2, 3, 7] = 0.5
    page = p.tables[0].long()[33 // 16]
    p.kc[page, 33 % 16, 1, 5] = INF
    p.check()


def test_a_batch_of_padding_only():
    p = Problem([0, 0, 0], [40, 0, 300], heads=1, group=2, dim=64, seed=24, pad=5)
    assert bool((p.run() == 7.0).all())


def test_many_idle_requests_and_one_token_at_the_end():
    B = 5000
    p = Problem([0] * (B - 1) + [1], [0] * (B - 1) + [77], heads=2, group=2, dim=64, seed=25)
    p.check()


def test_page_entries_out_of_range_read_as_zeros():
    p = Problem([3], [100], heads=1, group=2, dim=64, seed=13, masked=False)
    out = p.run()
    assert bool(torch.isfinite(out).all())
    pos = torch.arange(16, 48, device=DEV)
    p.tables[0, 1], p.tables[0, 2] = -3, 2 ** 31 - 1
    got = p.run()
    zero = p.kc.shape[0]
    p.kc = torch.cat([p.kc, torch.zeros_like(p.kc[:1])])
    p.vc = torch.cat([p.vc, torch.zeros_like(p.vc[:1])])
    p.tables[0, 1] = p.tables[0, 2] = zero
    ref, bound = attention_reference(p.q, p.k, p.v, p.kc, p.vc, p.tables, p.lens, p.starts, None)
    assert_attention(got, ref, bound)
    assert pos.numel() == 32


def test_lengths_and_starts_are_clamped():
    """Lengths past the block table, negative ones, starts out of range: nothing outside the
    arrays is read or written, and sound requests are right."""
    p = Problem([3, 4, 2], [90, 50, 20], heads=1, group=2, dim=64, seed=14)
    ref, bound = attention_reference(p.q, p.k, p.v, p.kc, p.vc, p.tables, p.lens, p.starts, p.sees)
    p.lens = [90, 2 ** 31 - 1, -5]
    out = p.run()
    assert_attention(out[:3], ref[:3], bound[:3])
    p.lens, p.starts = [90, 50, 20], [0, 3, 3, 2 ** 31 - 1]
    out = p.run()
    assert_attention(out[:3], ref[:3], bound[:3])
    p.starts = [-7, 3, 1, 0]
    assert_attention(p.run()[:1], ref[:1], bound[:1])


def test_no_cache_no_tokens_no_requests():
    p = Problem([5, 3], [0, 0], heads=2, group=2, dim=64, seed=15)
    want = p.check()
    p.tables = torch.empty(2, 0, dtype=torch.int32, device=DEV)
    assert torch.equal(p.run(), want)
    p.kc, p.vc = p.kc[:0], p.vc[:0]
    assert torch.equal(p.run(), want)
    e = p.q[:0]
    out = binding.tree_attention(e, p.k[:0], p.v[:0], p.kc, p.vc, p.tables, i32(p.lens),
                                 i32([0, 0, 0]))
    assert out.shape == e.shape
    out = torch.full_like(p.q, 7.0)
    binding.tree_attention(p.q, p.k, p.v, p.kc, p.vc, p.tables[:0], i32([]), i32([0]), out=out)
    assert bool((out == 7.0).all())


def test_past_32_bit_offsets():
    """The used pages lie past 2^31 elements of the cache."""
    heads, dim, page = 8, 128, 64
    pages = 2 ** 31 // (heads * dim * page) + 40
    p = Problem([4, 2], [700, 130], heads=heads, group=2, dim=dim, page=page, seed=16)
    c = torch.empty(2, pages, page, heads, dim, dtype=torch.float16, device=DEV)
    old = p.kc.shape[0]
    c[0, pages - old:], c[1, pages - old:] = p.kc, p.vc
    p.kc, p.vc = c[0], c[1]
    p.tables += pages - old
    p.check()


def test_results_do_not_vary():
    p = Problem([9, 33, 1, 70], [3000, 800, 77, 0], heads=3, group=4, dim=128, seed=17)
    first = p.run()
    for _ in range(5):
        assert torch.equal(p.run(), first)


def test_graph_replay_with_other_lengths_and_other_streams():
    p = Problem([4, 9, 1], [500, 90, 1000], heads=2, group=4, dim=128, seed=18)
    lens, starts = i32(p.lens), i32(p.starts)
    out = torch.zeros_like(p.q)
    args = (p.q, p.k, p.v, p.kc, p.vc, p.tables, lens, starts, p.mask)
    binding.tree_attention(*args, out=out)
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    out2 = torch.zeros_like(out)
    with torch.cuda.graph(g1):
        binding.tree_attention(*args, out=out)
    with torch.cuda.graph(g2):
        binding.tree_attention(*args, out=out2)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for new in ([500, 90, 1000], [17, 0, 999], [128, 64, 0]):
        p.lens = new
        lens.copy_(i32(new))
        out.zero_()
        out2.zero_()
        torch.cuda.synchronize()
        for s, g in ((s1, g1), (s2, g2)):         # two graphs at once
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        ref, bound = attention_reference(p.q, p.k, p.v, p.kc, p.vc, p.tables, p.lens, p.starts,
                                         p.sees)
        assert_attention(out, ref, bound)
        assert torch.equal(out, out2)
    # eager calls at once on two streams
    outs = []
    for s in (s1, s2, s1, s2):
        with torch.cuda.stream(s):
            outs.append(binding.tree_attention(*args))
    torch.cuda.synchronize()
    assert all(torch.equal(o, out) for o in outs)


def test_given_workspace_and_refusals():
    p = Problem([4, 9], [500, 90], heads=2, group=4, dim=128, seed=19)
    need = binding.tg_tree_attention_workspace_size(128)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)      # NaN throughout
    p.check(workspace=ws)
    for call in (lambda: p.run(workspace=ws[:-256]), lambda: p.run(scale=-1.0),
                 lambda: p.run(out=p.q), lambda: p.run(inject=9)):
        with pytest.raises(binding.TgError):
            call()
    for kw in (dict(out=torch.empty(3, 8, 128, dtype=p.dtype, device=DEV)),
               dict(workspace=ws.cpu())):
        with pytest.raises(ValueError):
            p.run(**kw)
    with pytest.raises(TypeError):
        p.run(out=torch.empty(p.q.shape, device=DEV))
    t = p.tables
    for bad in (t.long(), t.float()):
        p.tables = bad
        with pytest.raises(TypeError):
            p.run()
    p.tables = t[:1]
    with pytest.raises(ValueError):
        p.run()


def test_a_wait_that_runs_out_is_reported():
    """The first CTA skips its first key load, so a bounded wait expires; the call after it is
    right again."""
    p = Problem([4, 9], [500, 90], heads=2, group=4, dim=128, seed=20)
    binding.tree_attention(p.q, p.k, p.v, p.kc, p.vc, p.tables, i32(p.lens), i32(p.starts), p.mask,
                           wait_limit_ns=20_000_000, inject=binding.TG_INJECT_SKIP_FIRST_LOAD)
    torch.cuda.synchronize()
    stream = torch.cuda.current_stream().cuda_stream
    assert binding.tg_gemm_check_error(stream) == binding.TG_ERR_TIMEOUT
    assert binding.tg_gemm_check_error(stream) == binding.TG_OK
    p.check()


def test_decoding_steps_end_to_end():
    """Drafted trees are masked, attended and accepted for several steps through all four
    operators; each step equals dense attention over the accepted tokens so far."""
    rng = random.Random(21)
    heads, group, dim, page, B = 2, 4, 128, 16, 5
    cap, width = 120, 24
    kc, vc = torch.full((2, cap, page, heads, dim), NAN, dtype=torch.float16, device=DEV)
    tables = i32([[0] * width] * B)
    free, ring, lens = i32(rng.sample(range(cap), cap)), i32([7, cap]), i32([0] * B)
    dense = [(torch.empty(0, heads, dim, device=DEV).half(),) * 2 for _ in range(B)]

    def commit(k, v, add, starts, offsets):
        nonlocal ring, lens
        before = (lens.tolist(), add, ring.tolist(), free.tolist(), tables.tolist())
        p = binding.cache_plan(lens, i32(add), ring, free, tables, page, k.shape[0],
                               starts=i32(starts), offsets=i32(offsets))
        binding.cache_write(k, v, p.slots, kc, vc)
        want = plan_reference(*before, page, k.shape[0], starts, offsets)
        assert p.slots.tolist() == want[3] and p.status.tolist() == [0]
        assert tables.tolist() == want[7] and free.tolist() == want[6]
        ring, lens = p.ring, p.lens
        return p

    # prompts first
    n0 = [5, 16, 0, 40, 130]
    starts = [0]
    for n in n0:
        starts.append(starts[-1] + n)
    k, v = torch.randn(2, starts[-1], heads, dim, device=DEV).half()
    commit(k, v, n0, starts, [t for n in n0 for t in range(n)])
    dense = [(k[s:e], v[s:e]) for s, e in zip(starts, starts[1:])]
    for step in range(6):
        trees = [rng.choice([1, 3, 8, 20]) for _ in range(B)]
        parents, starts = [], [0]
        for n in trees:
            parents += [rng.randint(max(-1, i - 3), i - 1) for i in range(n)]
            starts.append(len(parents))
        n = starts[-1]
        q = torch.randn(n, heads * group, dim, device=DEV).half()
        k, v = torch.randn(2, n, heads, dim, device=DEV).half()
        mask, depth = binding.tree_mask(i32(parents), i32(starts), 1)
        out = binding.tree_attention(q, k, v, kc, vc, tables, lens, i32(starts), mask)
        sees = tree_reference(parents, starts, 1)[0]
        # the same over dense tensors: a cache of one page per request
        add, offsets = [], [-1] * n
        for b in range(B):
            kd, vd = dense[b]
            L = kd.shape[0]
            one = torch.arange(max(L, 1), device=DEV, dtype=torch.int32)[None]
            qs = slice(starts[b], starts[b + 1])
            ref, bound = attention_reference(
                q[qs], k[qs], v[qs], kd[:, None], vd[:, None], one, [L], [0, trees[b]],
                sees[qs])
            assert_attention(out[qs], ref, bound, f"step {step} request {b}")
            leaf = rng.randrange(trees[b])                      # accept the path to a random leaf
            path = sorted(sees[starts[b] + leaf])
            assert len(path) == int(depth[starts[b] + leaf]) + 1
            for i, j in enumerate(path):
                offsets[starts[b] + j] = i
            add.append(len(path))
            rows = torch.tensor(path, device=DEV) + starts[b]
            dense[b] = (torch.cat([kd, k[rows]]), torch.cat([vd, v[rows]]))
        commit(k, v, add, starts, offsets)
        assert lens.tolist() == [d[0].shape[0] for d in dense]
    # every request ends: all pages are free again
    p = binding.cache_plan(lens, -lens, ring, free, tables, page, 0)
    assert p.ring.tolist()[1] == cap and p.lens.tolist() == [0] * B
    assert sorted(free.tolist()) == list(range(cap))
