"""Block tables and slot maps, cache writes and tree masks on the GPU against plain references.
Every result is a whole number or a copied bit pattern, so every comparison is exact."""
import random

import pytest
import torch

from cache_helpers import pack_bits, plan_reference, tree_reference
from tensor_core_gemm_fp16_b200 import binding

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------- cache_plan

def make_state(rng, B, page, max_len, width, spare):
    """Lengths, tables, free ring of a server in the middle of its work."""
    lens = [rng.choice([0, 1, page - 1, page, page + 1, rng.randint(0, max_len)])
            for _ in range(B)]
    lens = [min(n, width * page) for n in lens]
    used = sum(-(-n // page) for n in lens)
    cap = used + spare
    order = list(range(cap))
    rng.shuffle(order)
    tables, at = [], 0
    for n in lens:
        k = -(-n // page)
        tables.append(order[at:at + k] + [rng.randint(-5, cap + 5) for _ in range(width - k)])
        at += k
    head = rng.randrange(cap)
    free = [rng.randint(-9, -1) for _ in range(cap)]          # entries that are not free: junk
    for i in range(spare):
        free[(head + i) % cap] = order[used + i]
    return lens, tables, free, [head, spare]


def run_plan(lens, add, ring, free, tables, page, tokens, starts=None, offsets=None, pad=0):
    B, width = len(lens), len(tables[0]) if tables else 0
    wide = torch.full((B, width + pad), -77, dtype=torch.int32, device=DEV)
    if B and width:
        wide[:, :width] = i32(tables)
    tab = wide[:, :width]
    fr = i32(free)
    p = binding.cache_plan(i32(lens), i32(add), i32(ring), fr, tab, page, tokens,
                           starts=None if starts is None else i32(starts),
                           offsets=None if offsets is None else i32(offsets))
    torch.cuda.synchronize()
    assert bool((wide[:, width:] == -77).all())
    return (p.lens.tolist(), p.ring.tolist(), p.starts.tolist(), p.slots.tolist(),
            p.positions.tolist(), int(p.status), fr.tolist(), tab.tolist())


def check_plan(*args, **kw):
    pad = kw.pop("pad", 0)
    want = plan_reference(*args, **kw)
    got = run_plan(*args, pad=pad, **kw)
    for name, g, w in zip(("lens", "ring", "starts", "slots", "positions", "status", "free pages",
                           "tables"), got, want):
        assert g == w, name
    return got


@pytest.mark.parametrize("page", [8, 16, 64, 256])
@pytest.mark.parametrize("B", [1, 2, 33, 511, 512, 513, 1100])
def test_plan_appends(B, page):
    rng = random.Random(B * 1000 + page)
    width = 9
    lens, tables, free, ring = make_state(rng, B, page, 5 * page, width, 4 * B + 3)
    add = [rng.choice([0, 1, 1, 2, page, rng.randint(0, 3 * page)]) for _ in range(B)]
    n = sum(add)
    check_plan(lens, add, ring, free, tables, page, n, pad=3)
    # a padded batch: rows behind the last request get -1
    got = check_plan(lens, add, ring, free, tables, page, n + 37)
    assert got[3][n:] == [-1] * 37 and got[4][n:] == [-1] * 37


@pytest.mark.parametrize("B", [1, 7, 300, 2049])
def test_plan_mixes_growth_rollback_and_release(B):
    rng = random.Random(B)
    page, width = 16, 12
    lens, tables, free, ring = make_state(rng, B, page, 8 * page, width, 4 * B + 1)
    add = []
    for n in lens:
        u = rng.random()
        add.append(-n if u < 0.3 else -rng.randint(0, n) if u < 0.6 else rng.randint(0, 3 * page))
    check_plan(lens, add, ring, free, tables, page, sum(max(a, 0) for a in add))


def test_plan_of_accepted_tree_tokens():
    rng = random.Random(5)
    B, page, width = 40, 16, 8
    lens, tables, free, ring = make_state(rng, B, page, 5 * page, width, 100)
    starts, offsets, add = [3], [-1, 0, 7], []        # rows before the first request are not kept
    for b in range(B):
        tree = rng.randint(0, 9)
        kept = sorted(rng.sample(range(tree), rng.randint(0, tree)))
        off = [-1] * tree
        for k, t in enumerate(kept):
            off[t] = k
        if tree and rng.random() < 0.3:
            off[rng.randrange(tree)] = len(kept) + rng.randint(0, 5)      # past the kept ones
        add.append(len(kept))
        starts.append(starts[-1] + tree)
        offsets += off
    tokens = starts[-1] + 5
    offsets += [0] * 5                                # rows behind the last request: not kept
    check_plan(lens, add, ring, free, tables, page, tokens, starts=starts, offsets=offsets)
    check_plan(lens, add, ring, free, tables, page, tokens, starts=starts)


def test_plan_of_one_long_prompt_and_the_largest_batch():
    rng = random.Random(6)
    lens, tables, free, ring = make_state(rng, 2, 16, 100, 6300, 6400)
    check_plan(lens, [100003, 1], ring, free, tables, 16, 100004)
    B = binding.TG_CACHE_MAX_BATCH
    lens, tables, free, ring = make_state(rng, B, 8, 30, 6, 3 * B)
    add = [rng.choice([-1, 0, 1, 5]) if n else 1 for n in lens]
    check_plan(lens, add, ring, free, tables, 8, sum(max(a, 0) for a in add))


def test_plan_without_requests_or_tokens():
    got = check_plan([], [], [2, 1], [5, 6, 7], [], 16, 4)
    assert got[3] == [-1] * 4
    check_plan([20, 0], [0, 0], [0, 2], [9, 8, 7, 6], [[1, 2], [3, 3]], 16, 0)


def test_plan_takes_exactly_the_last_page():
    check_plan([16, 16], [1, 16], [3, 2], [0, 1, 2, 3], [[2, 9], [1, 9]], 16, 17)


@pytest.mark.parametrize("what", ["pages", "width", "length", "shrink", "tokens", "descending",
                                  "starts", "head", "count", "overfull", "huge", "several"])
def test_plan_refuses_on_the_device_and_changes_nothing(what):
    lens, add, ring, free = [16, 33], [1, 16], [3, 3], [0, 1, 2, 3, 4, 5]
    tables, tokens, starts, bit = [[2, 9, 9, 9], [1, 0, 5, 9]], 17, None, 0
    if what == "pages":
        ring, bit = [3, 1], 1
    elif what == "width":
        add, tokens, ring, bit = [49, 0], 49, [0, 6], 2
    elif what == "length":
        lens, add, bit = [-1, 33], [1, 16], 4
    elif what == "shrink":
        add, bit = [-17, 16], 4
    elif what == "tokens":
        tokens, bit = 16, 8
    elif what == "descending":
        starts, bit = [0, 5, 4], 8
    elif what == "starts":
        starts, bit = [-1, 5, 17], 8
    elif what == "head":
        ring, bit = [6, 3], 16
    elif what == "count":
        ring, bit = [0, 7], 16
    elif what == "overfull":
        add, tokens, ring, bit = [-16, -33], 0, [0, 5], 16
    elif what == "huge":
        lens, add, bit = [2 ** 31 - 1, 2 ** 31 - 1], [2 ** 31 - 1, 2 ** 31 - 1], 1 | 2 | 4 | 8
    elif what == "several":
        add, ring, bit = [200, -40], [0, 7], 1 | 2 | 4 | 8 | 16
    if what == "huge":
        got = run_plan(lens, add, ring, free, tables, 16, tokens)
        assert got[2] == [0, 2 ** 31 - 1, 2 ** 31 - 1]         # saturated
    else:
        got = check_plan(lens, add, ring, free, tables, 16, tokens, starts=starts)
    assert got[5] == bit and got[0] == lens and got[1] == ring
    assert got[6] == free and got[7] == tables
    assert got[3] == [-1] * tokens and got[4] == [-1] * tokens


# ---------------------------------------------------------------- cache_write

def make_caches(pages, page, heads, dim, layout, dtype=torch.float16):
    def fill(*shape):
        return torch.randint(-2 ** 15, 2 ** 15, shape, dtype=torch.int16, device=DEV).view(dtype)
    if layout == "plain":
        return fill(pages, page, heads, dim), fill(pages, page, heads, dim)
    if layout == "interleaved":         # one tensor per layer holds keys and values
        c = fill(pages, 2, page, heads, dim)
        return c[:, 0], c[:, 1]
    if layout == "heads_first":
        return (fill(pages, heads, page, dim).transpose(1, 2),
                fill(pages, heads, page, dim).transpose(1, 2))
    c = fill(pages, page, heads, 2, dim)                 # keys and values side by side
    return c[:, :, :, 0], c[:, :, :, 1]


@pytest.mark.parametrize("layout", ["plain", "interleaved", "heads_first", "side_by_side"])
@pytest.mark.parametrize("heads,dim,page,n", [(1, 64, 8, 1), (2, 128, 16, 37), (3, 64, 32, 300),
                                              (8, 128, 16, 2000), (17, 128, 256, 90),
                                              (40, 64, 64, 65)])
def test_write_copies_kept_rows_and_nothing_else(layout, heads, dim, page, n):
    g = torch.Generator().manual_seed(n)
    pages = -(-n // page) + 2
    kc, vc = make_caches(pages, page, heads, dim, layout)
    qkv = torch.randint(-2 ** 15, 2 ** 15, (n, 2 * heads + 3, dim), dtype=torch.int16,
                        device=DEV).view(torch.float16)
    k, v = qkv[:, 3:3 + heads], qkv[:, 3 + heads:]
    slots = torch.randperm(pages * page, generator=g)[:n]
    slots[torch.rand(n, generator=g) < 0.3] = -1
    slots[::7] = pages * page + torch.arange(len(slots[::7])) * 10 ** 12      # out of range
    slots[::11] = -10 ** 15
    slots = slots.to(DEV)
    want_k, want_v = kc.clone().view(torch.int16), vc.clone().view(torch.int16)
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < pages * page:
            want_k[s // page, s % page] = k[t].view(torch.int16)
            want_v[s // page, s % page] = v[t].view(torch.int16)
    out = binding.cache_write(k, v, slots, kc, vc)
    torch.cuda.synchronize()
    assert out[0] is kc and out[1] is vc
    assert torch.equal(kc.view(torch.int16), want_k) and torch.equal(vc.view(torch.int16), want_v)


def test_write_of_no_tokens_and_bf16():
    kc, vc = make_caches(2, 16, 2, 64, "plain", torch.bfloat16)
    before = kc.clone().view(torch.int16)
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    binding.cache_write(e, e, torch.empty(0, dtype=torch.int64, device=DEV), kc, vc)
    assert torch.equal(kc.view(torch.int16), before)
    k = torch.randn(1, 2, 64, device=DEV).bfloat16()
    binding.cache_write(k, k, torch.tensor([17], device=DEV), kc, vc)
    assert torch.equal(kc[1, 1], k[0]) and torch.equal(vc[1, 1], k[0])


def test_write_past_32_bit_offsets():
    """A cache of more than 2^31 elements: the last page lies past 32-bit element offsets."""
    heads, dim, page = 8, 128, 256
    pages = 2 ** 31 // (heads * dim * page) + 2
    c = torch.empty(2, pages, page, heads, dim, dtype=torch.float16, device=DEV)
    c[:, -1] = 0
    c[:, 0] = 0
    k = torch.randn(3, heads, dim, device=DEV).half()
    slots = torch.tensor([pages * page - 1, 5, (pages - 1) * page], device=DEV)
    binding.cache_write(k, -k, slots, c[0], c[1])
    assert torch.equal(c[0, -1, -1], k[0]) and torch.equal(c[1, -1, -1], -k[0])
    assert torch.equal(c[0, 0, 5], k[1]) and torch.equal(c[1, -1, 0], -k[2])
    assert int(torch.count_nonzero(c[0, -1])) == int(torch.count_nonzero(k[[0, 2]]))


# ---------------------------------------------------------------- tree_mask

def check_mask(parents, starts, words, out=None):
    sees, depth = tree_reference(parents, starts, words)
    m, d = binding.tree_mask(i32(parents), i32(starts), words, out=out)
    torch.cuda.synchronize()
    assert d.tolist() == depth
    assert torch.equal(m.cpu(), pack_bits(sees, words))


def random_tree(rng, n, back):
    return [rng.randint(max(-1, i - back), i - 1) for i in range(n)]


@pytest.mark.parametrize("sizes,words", [([1], 1), ([32], 1), ([33], 2), ([0, 5, 0, 31, 64], 2),
                                         ([200, 1, 128], 7), ([1000, 999], 32),
                                         ([2048, 3], 64)])
@pytest.mark.parametrize("back", [1, 7, 3000])
def test_mask_of_random_trees(sizes, words, back):
    rng = random.Random(sum(sizes) + back)
    starts, parents = [0], []
    for n in sizes:
        parents += random_tree(rng, n, back)
        starts.append(len(parents))
    check_mask(parents, starts, words)


def test_mask_of_chains_and_roots():
    check_mask(list(range(-1, 2047)), [0, 2048], 64)        # the deepest chain
    check_mask([-1] * 100, [0, 40, 100], 2)                 # every token a root


def test_mask_of_invalid_parents_and_rows_outside():
    """A parent not below its child, or under -1, empties the token's row and its descendants';
    so do tokens past the mask's width; rows outside every request are empty."""
    parents = [7, 7, -1, 1, -2, 0, 2, 3, 4, -1, 9] + [-1, 0, 1] * 14 + [5, 5]
    check_mask(parents, [2, 11, 53], 1)        # the second request has 42 tokens, 32 fit
    check_mask([-1, 0, 2 ** 31 - 1, 2, -2 ** 31], [0, 5], 1)


def test_mask_writes_into_given_outputs():
    out = (torch.full((6, 3), 77, dtype=torch.int32, device=DEV),
           torch.full((6,), 77, dtype=torch.int32, device=DEV))
    check_mask([-1, 0, 0, -1, 0, 1], [0, 3, 6], 3, out=out)


def test_mask_without_requests():
    check_mask([-1, 0], [0], 1)


def test_mask_clamps_starts():
    """Starts out of range are clamped: nothing outside the arrays is touched."""
    m, d = binding.tree_mask(i32([-1, 0, 1]), i32([-5, 2, 2 ** 31 - 1]), 1)
    assert d.tolist() == [0, 1, -1]         # the third token is its request's first: parent 1 is not below it
    m, d = binding.tree_mask(i32([-1, 0, 1]), i32([2, 1, 0]), 1)      # descending: no requests
    assert m.shape == (3, 1)


# ---------------------------------------------------------------- streams, graphs, devices

def test_operators_run_on_the_current_stream_and_in_graphs():
    """Captured once, replayed with other contents of the same tensors."""
    rng = random.Random(9)
    B, page, width = 20, 16, 8
    states = [make_state(rng, B, page, 4 * page, width, 70) for _ in range(3)]
    adds = [[rng.randint(0, 20) for _ in range(B)] for _ in range(3)]
    cap, tokens, heads, dim = 256, 400, 2, 64
    buf = dict(lens=i32([0] * B), add=i32([0] * B), ring=i32([0, 0]), free=i32([0] * cap),
               tables=i32([[0] * width] * B))
    k, v = torch.randn(2, tokens, heads, dim, device=DEV).half()
    kc, vc = make_caches(cap, page, heads, dim, "plain")
    p = binding.cache_plan(buf["lens"], buf["add"], buf["ring"], buf["free"], buf["tables"], page,
                           tokens)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        binding.cache_plan(buf["lens"], buf["add"], buf["ring"], buf["free"], buf["tables"], page,
                           tokens, out=p)
        binding.cache_write(k, v, p.slots, kc, vc)
    for (lens, tables, free, ring), add in zip(states, adds):
        # the ring's capacity is the tensor's: pad it behind the free entries
        head, count = ring
        order = [free[(head + i) % len(free)] for i in range(count)]
        free, ring = order + [-1] * (cap - count), [0, count]
        for name, x in (("lens", lens), ("add", add), ("ring", ring), ("free", free),
                        ("tables", tables)):
            buf[name].copy_(i32(x))
        k.normal_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = plan_reference(lens, add, ring, free, tables, page, tokens)
        assert p.slots.tolist() == want[3] and p.lens.tolist() == want[0]
        kept = p.slots >= 0
        assert torch.equal(kc.view(-1, heads, dim)[p.slots[kept]], k[kept])


def test_binding_refusals_on_the_gpu():
    B = 3
    lens, ring, free, tab = i32([1, 2, 3]), i32([0, 4]), i32([0, 1, 2, 3]), i32([[0] * 4] * B)
    ok = binding.cache_plan(lens, lens.clone(), ring, free, tab, 16, 6)
    with pytest.raises(TypeError):
        binding.cache_plan(lens.long(), lens, ring, free, tab, 16, 6)
    with pytest.raises(ValueError):
        binding.cache_plan(lens, lens[:2], ring, free, tab, 16, 6)
    with pytest.raises(ValueError):
        binding.cache_plan(lens, lens, ring, free, tab.t(), 16, 6)
    with pytest.raises(binding.TgError):
        binding.cache_plan(lens, lens, ring, free, tab, 20, 6)                # page size
    with pytest.raises(binding.TgError):                                      # in place
        binding.cache_plan(lens, lens.clone(), ring, free, tab, 16, 6, out=ok._replace(lens=lens))
    with pytest.raises(binding.TgError):                                      # offsets alone
        binding.cache_plan(lens, lens, ring, free, tab, 16, 6, offsets=i32([0] * 6))
    k = torch.zeros(2, 2, 64, dtype=torch.float16, device=DEV)
    c = torch.zeros(2, 16, 2, 64, dtype=torch.float16, device=DEV)
    s = torch.zeros(2, dtype=torch.int64, device=DEV)
    with pytest.raises(TypeError):
        binding.cache_write(k.float(), k.float(), s, c.float(), c.float())
    with pytest.raises(TypeError):
        binding.cache_write(k, k, s.int(), c, c.clone())
    with pytest.raises(ValueError):
        binding.cache_write(k, k[:1], s, c, c.clone())
    with pytest.raises(ValueError):
        binding.cache_write(k, k, s, c, c.clone()[:1])
    with pytest.raises(binding.TgError):
        binding.cache_write(k, k, s, c, c)                                    # one cache twice
    with pytest.raises(binding.TgError):
        binding.tree_mask(i32([-1]), i32([0, 1]), 65)
    with pytest.raises(ValueError):
        binding.tree_mask(i32([-1]), i32([0, 1]), 1, out=(lens, lens))
