"""Host checks of keys and values with strides of their own (no GPU)."""
import pytest

from tensor_core_gemm_fp16_b200 import binding
from test_cache_abi import BAD, M, MIS, NO_DEVICE, OK, attend, no_device_only


def write(**kw):
    a = dict(k=1 * M, k_token_stride=128, k_head_stride=64, v=2 * M, v_token_stride=384,
             v_head_stride=64, tokens=8, heads=2, head_dim=64, slots=3 * M, k_cache=4 * M,
             v_cache=5 * M, num_pages=4, page_size=16, page_stride=2048, slot_stride=128,
             cache_head_stride=64)
    a.update(kw)
    return binding.tg_cache_write_ex(**a)


@no_device_only
def test_cache_write_ex_refusals():
    assert write() == NO_DEVICE
    assert write(v_token_stride=0, v_head_stride=0) == NO_DEVICE           # a broadcast source
    assert write(tokens=1, v_token_stride=3, k_token_stride=-5) == NO_DEVICE     # unused
    assert write(tokens=0) == OK
    for kw in (dict(v_token_stride=-8), dict(k_token_stride=-8), dict(v_head_stride=-8),
               dict(v_token_stride=1 << 40), dict(v=5 * M - 5632 + 16), dict(v=None)):
        assert write(**kw) == BAD, kw
    for kw in (dict(v_token_stride=132), dict(k_head_stride=68), dict(v_head_stride=65)):
        assert write(**kw) == MIS, kw


@no_device_only
@pytest.mark.parametrize("own", [1, -1])
def test_tree_attention_with_strides_of_the_values(own):
    def call(**kw):
        return attend(own_v_strides=own, **{**dict(v_token_stride=384, v_head_stride=64), **kw})
    assert call() == NO_DEVICE
    assert call(tokens=1, v_token_stride=0) == NO_DEVICE                   # unused
    for kw in (dict(v_token_stride=0), dict(v_head_stride=0), dict(v_token_stride=0,
               v_head_stride=0), dict(v_token_stride=-384), dict(v_head_stride=1 << 38),
               dict(v=10 * M - 5632 + 16)):
        assert call(**kw) == BAD, kw
    for kw in (dict(v_token_stride=132), dict(v_head_stride=68)):
        assert call(**kw) == MIS, kw
    assert attend(v_token_stride=0, v_head_stride=3) == NO_DEVICE          # k's strides count


def test_packed_struct_matches_the_declared_one():
    """The bytes that the binding packs are the struct's, field by field."""
    import ctypes
    fields = binding.tg_tree_attention_t._fields_
    assert binding._TREE_ARGS.size == ctypes.sizeof(binding.tg_tree_attention_t)
    values = list(range(1, len(fields) + 1))
    s = binding.tg_tree_attention_t.from_buffer_copy(binding._TREE_ARGS.pack(*values))
    assert [getattr(s, name) for name, _ in fields] == values
