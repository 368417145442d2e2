"""Keys and values that lie differently in memory: fresh tensors beside slices of a projection."""
import pytest
import torch

from attention_helpers import assert_rows, definition
from tensor_core_gemm_fp16_b200 import binding

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def decode(n, heads, dim, pages, page=16, dtype=torch.float16, caches="plain"):
    """Keys of their own (as a rotation of them leaves them), values a slice of the projection;
    n new tokens of one request over a cache of `pages` pages."""
    torch.manual_seed(n + heads + pages)
    q = torch.randn(n, 4 * heads, dim, device=DEV).to(dtype)
    k = torch.randn(n, heads, dim, device=DEV).to(dtype)
    v = torch.randn(n, 3 * heads, dim, device=DEV).to(dtype)[:, 2 * heads:]
    kc = torch.randn(pages, page, heads, dim, device=DEV).to(dtype)
    if caches == "plain":
        vc = torch.randn(pages, page, heads, dim, device=DEV).to(dtype)
    else:                                   # a page of a larger tensor, heads of another
        vc = torch.randn(pages, page, 2 * heads, dim, device=DEV).to(dtype)[:, :, :heads]
    return q, k, v, kc, vc


def check(q, k, v, kc, vc):
    n, heads, dim = k.shape
    pages, page = kc.shape[:2]
    lens, starts = [pages * page - n - 1], [0, n]
    tables = torch.arange(pages, device=DEV, dtype=torch.int32)[None]
    for mask, sees in ((None, None),
                       (i32([[(1 << (t % 31)) - 1 | 1 << (t % 31)] for t in range(n)]),
                        [set(range(t % 31 + 1)) for t in range(n)])):
        out = binding.tree_attention(q, k, v, kc, vc, tables, i32(lens), i32(starts), mask)
        ref, bound, rows = definition(q, k, v, kc, vc, tables, lens, starts, sees)
        assert_rows(out, ref, bound, rows)
    slots = torch.arange(lens[0], lens[0] + n, device=DEV)
    want_k, want_v = kc.clone(), vc.clone()
    want_k.flatten(0, 1)[slots], want_v.flatten(0, 1)[slots] = k, v
    binding.cache_write(k, v, slots, kc, vc)
    for got, want in ((kc, want_k), (vc, want_v)):
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("dim", [64, 128])
def test_strides_of_single_elements_do_not_count(dim):
    """One token, one head, one page: torch's strides of such dimensions differ between tensors
    that lie the same way."""
    q, k, v, kc, vc = decode(1, 2, dim, 7)
    assert k.stride() != v.stride() and v.is_contiguous()
    check(q, k, v, kc, vc)
    # one head: only the token strides count, and they are the same
    q, k, v, kc, vc = decode(5, 1, dim, 7)
    k = torch.randn(5, 3, dim, device=DEV).half()[:, 1:2]
    v = torch.randn(5, 3 * dim, device=DEV).half().as_strided((5, 1, dim), (3 * dim, 7, 1))
    assert k.stride(0) == v.stride(0) and k.stride() != v.stride()
    check(q, k, v, kc, vc)
    # one page of one head
    q, k, v, kc, vc = decode(1, 1, dim, 1)
    vc = torch.randn(2, 16, 1, dim, device=DEV).half()[::2]
    assert kc.stride() != vc.stride()
    check(q, k, v, kc, vc)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("n,heads,dim", [(2, 2, 64), (9, 1, 128), (40, 3, 64), (150, 2, 128)])
def test_keys_of_their_own_beside_values_of_the_projection(n, heads, dim, dtype):
    q, k, v, kc, vc = decode(n, heads, dim, 20, dtype=dtype)
    assert k.stride(0) != v.stride(0)
    check(q, k, v, kc, vc)
    check(q, v, k, kc, vc)
    # heads first
    check(q, k.transpose(0, 1).contiguous().transpose(0, 1), v, kc, vc)


def test_values_that_are_not_finite_with_strides_of_their_own():
    q, k, v, kc, vc = decode(40, 2, 64, 20)
    v[3, 1, 5], v[7, 0, 63] = float("inf"), float("nan")
    k[5, 0, 2] = float("-inf")
    v[5, 0, 9] = float("inf")
    check(q, k, v, kc, vc)


def test_values_without_strides_are_refused():
    """Broadcast values: the attention needs rows of their own, the write copies them."""
    q, k, v, kc, vc = decode(4, 2, 64, 3)
    args = (kc, vc, i32([[0, 1, 2]]), i32([9]), i32([0, 4]))
    for x in (v[:1, :1].expand(4, 2, 64), v[:1].expand(4, 2, 64), v[:, :1].expand(4, 2, 64)):
        with pytest.raises(binding.TgError):
            binding.tree_attention(q, k, x, *args)
        with pytest.raises(binding.TgError):
            binding.tree_attention(q, x, v, *args)
        slots = torch.tensor([3, 40, -1, 17], device=DEV)
        binding.cache_write(k, x, slots, kc, vc)
        for t, s in ((0, 3), (1, 40), (3, 17)):
            assert torch.equal(vc[s // 16, s % 16], x[t]) and torch.equal(kc[s // 16, s % 16], k[t])
    with pytest.raises(ValueError):
        binding.cache_write(k, v.transpose(1, 2).contiguous().transpose(1, 2), slots, kc, vc)
