"""Refusals of the paged-cache operators that need no GPU: everything here is rejected (or found
empty) on the host before any device call."""
import pytest
import torch

from tensor_core_gemm_fp16_b200 import binding

BAD, MIS, OK = binding.TG_ERR_INVALID_ARG, binding.TG_ERR_MISALIGNED, binding.TG_OK

# Made-up addresses: only where no device exists, so that a regression never reaches a GPU.
no_device_only = pytest.mark.skipif(torch.cuda.is_available(),
                                    reason="made-up addresses: host-only check")
NO_DEVICE = binding.TG_ERR_UNSUPPORTED_DEVICE
M = 1 << 20


def test_symbols_are_declared_and_exported():
    names = binding.header_symbols()
    for name in ("tg_cache_plan", "tg_cache_write", "tg_tree_mask", "tg_tree_attention",
                 "tg_tree_attention_workspace_size"):
        assert name in names and hasattr(binding.load(), name)


def test_constants_match_the_header():
    import os
    import re
    with open([h for h in binding.HEADERS if h.endswith("tg_cache.h")][0]) as f:
        text = f.read()
    for name in ("TG_TYPE_FP16", "TG_TYPE_BF16", "TG_PLAN_NO_PAGES", "TG_PLAN_TABLE_FULL",
                 "TG_PLAN_BAD_LENGTH", "TG_PLAN_BAD_TOKENS", "TG_PLAN_BAD_RING"):
        assert int(re.search(rf"\b{name} = (\d+)", text).group(1)) == getattr(binding, name)
    for name in ("TG_CACHE_MAX_BATCH", "TG_TREE_MAX_WORDS"):
        assert int(re.search(rf"#define {name} (\d+)", text).group(1)) == getattr(binding, name)
    assert os.path.basename(binding.HEADERS[-1]) == "tg_cache.h"


def plan(**kw):
    a = dict(lens=1 * M, add=2 * M, batch=4, starts=None, offsets=None, tokens=16,
             block_tables=3 * M, table_stride=8, max_pages=8, page_size=16, free_pages=4 * M,
             num_pages=64, ring=5 * M, lens_out=6 * M, ring_out=7 * M, starts_out=8 * M,
             slots=9 * M, positions=10 * M, status=11 * M)
    a.update(kw)
    return binding.tg_cache_plan(**a)


@no_device_only
def test_cache_plan_refusals():
    assert plan() == NO_DEVICE                                  # passes every check
    assert plan(starts_out=None) == NO_DEVICE
    assert plan(starts=12 * M, offsets=13 * M) == NO_DEVICE
    assert plan(batch=0, lens=None, add=None, lens_out=None, block_tables=None) == NO_DEVICE
    for kw in (dict(batch=-1), dict(batch=8193), dict(tokens=-1), dict(tokens=1 << 31),
               dict(page_size=0), dict(page_size=4), dict(page_size=24), dict(page_size=512),
               dict(max_pages=-1), dict(table_stride=7), dict(num_pages=0), dict(offsets=13 * M),
               dict(ring=None), dict(ring_out=None), dict(status=None), dict(free_pages=None),
               dict(lens=None), dict(add=None), dict(lens_out=None), dict(block_tables=None),
               dict(slots=None), dict(positions=None),
               dict(lens_out=1 * M), dict(ring_out=5 * M), dict(lens_out=2 * M + 12),
               dict(free_pages=3 * M + 64), dict(slots=10 * M - 64), dict(status=7 * M + 4),
               dict(starts=8 * M)):
        assert plan(**kw) == BAD, kw
    for kw in (dict(lens=M + 2), dict(slots=9 * M + 4), dict(ring=5 * M + 1),
               dict(positions=10 * M + 2)):
        assert plan(**kw) == MIS, kw


def write(**kw):
    a = dict(k=1 * M, v=2 * M, tokens=8, heads=2, head_dim=64, token_stride=128, head_stride=64,
             slots=3 * M, k_cache=4 * M, v_cache=5 * M, num_pages=4, page_size=16,
             page_stride=2048, slot_stride=128, cache_head_stride=64)
    a.update(kw)
    return binding.tg_cache_write(**a)


@no_device_only
def test_cache_write_refusals():
    assert write() == NO_DEVICE
    assert write(token_stride=0, head_stride=0) == NO_DEVICE     # a broadcast source
    assert write(heads=1, head_stride=3, cache_head_stride=5) == NO_DEVICE   # unused strides
    assert write(v_cache=4 * M + 128, slot_stride=256, page_stride=4096) == NO_DEVICE
    for kw in (dict(tokens=0), dict(heads=0), dict(num_pages=0)):
        assert write(**kw) == OK, kw
    for kw in (dict(tokens=-1), dict(tokens=1 << 31), dict(heads=-1), dict(head_dim=96),
               dict(page_size=20), dict(num_pages=-1), dict(k=None), dict(v=None),
               dict(slots=None), dict(k_cache=None), dict(v_cache=None), dict(token_stride=-8),
               dict(slot_stride=0), dict(page_stride=8), dict(cache_head_stride=32),
               dict(v_cache=4 * M), dict(k_cache=1 * M + 1024), dict(slots=5 * M + 64)):
        assert write(**kw) == BAD, kw
    for kw in (dict(k=M + 8), dict(v=M * 2 + 2), dict(k_cache=4 * M + 8), dict(slots=3 * M + 4),
               dict(token_stride=132), dict(slot_stride=132), dict(page_stride=2052)):
        assert write(**kw) == MIS, kw


def mask(**kw):
    a = dict(parents=1 * M, tokens=8, starts=2 * M, batch=2, words=1, mask=3 * M, depth=4 * M)
    a.update(kw)
    return binding.tg_tree_mask(**a)


@no_device_only
def test_tree_mask_refusals():
    assert mask() == NO_DEVICE and mask(batch=0) == NO_DEVICE and mask(words=64) == NO_DEVICE
    assert mask(tokens=0, parents=None, mask=None, depth=None) == OK
    for kw in (dict(tokens=-1), dict(batch=-1), dict(words=0), dict(words=65), dict(parents=None),
               dict(starts=None), dict(mask=None), dict(depth=None), dict(mask=1 * M + 16),
               dict(depth=3 * M + 28), dict(depth=2 * M + 8)):
        assert mask(**kw) == BAD, kw
    for kw in (dict(parents=M + 1), dict(starts=2 * M + 2), dict(mask=3 * M + 2),
               dict(depth=4 * M + 1)):
        assert mask(**kw) == MIS, kw


def attend(**kw):
    ws = binding.tg_tree_attention_workspace_size(64)
    a = dict(type=0, tokens=8, batch=2, kv_heads=2, group=4, head_dim=64, scale=0.0, q=1 * M,
             q_token_stride=512, q_head_stride=64, k=2 * M, v=3 * M, kv_token_stride=128,
             kv_head_stride=64, k_cache=4 * M, v_cache=5 * M, num_pages=4, page_size=16,
             page_stride=2048, slot_stride=128, cache_head_stride=64, block_tables=6 * M,
             table_stride=2, max_pages=2, lens=7 * M, starts=8 * M, mask=9 * M, words=1,
             mask_stride=1, out=10 * M, out_token_stride=512, out_head_stride=64,
             workspace=256 * M, workspace_bytes=ws, wait_limit_ns=0, inject=0)
    a.update(kw)
    return binding.tg_tree_attention(binding.tg_tree_attention_t(**a))


@no_device_only
def test_tree_attention_refusals():
    assert attend() == NO_DEVICE
    assert attend(mask=None, words=0, mask_stride=0) == NO_DEVICE
    assert attend(max_pages=0, block_tables=None, k_cache=None, v_cache=None) == NO_DEVICE
    assert attend(type=1, group=128, q_token_stride=1 << 14, out_token_stride=1 << 14,
                  out=100 * M) == NO_DEVICE
    for kw in (dict(tokens=0, q=None), dict(batch=0), dict(kv_heads=0)):
        assert attend(**kw) == OK, kw
    assert binding.load().tg_tree_attention(None, None) == BAD
    for kw in (dict(type=2), dict(type=-1), dict(tokens=-1), dict(tokens=(1 << 31) - 100),
               dict(batch=-1), dict(kv_heads=-1), dict(group=0), dict(group=129),
               dict(head_dim=96), dict(scale=-1.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(scale=1e-31), dict(scale=2e30), dict(page_size=4), dict(page_size=48),
               dict(page_size=512), dict(num_pages=-1), dict(max_pages=-1), dict(table_stride=1),
               dict(max_pages=1 << 28, table_stride=1 << 28), dict(words=0), dict(mask_stride=0),
               dict(inject=2), dict(q=None), dict(k=None), dict(v=None), dict(out=None),
               dict(lens=None), dict(starts=None), dict(k_cache=None), dict(v_cache=None),
               dict(block_tables=None), dict(workspace=None), dict(workspace_bytes=1000),
               dict(q_token_stride=0), dict(kv_token_stride=32), dict(slot_stride=0),
               dict(page_stride=0), dict(out_token_stride=8), dict(out_head_stride=0),
               dict(out=1 * M + 512), dict(out=4 * M), dict(out=256 * M), dict(workspace=5 * M)):
        assert attend(**kw) == BAD, kw
    for kw in (dict(q=M + 8), dict(k=2 * M + 2), dict(v=3 * M + 8), dict(out=10 * M + 8),
               dict(k_cache=4 * M + 8), dict(workspace=256 * M + 16), dict(lens=7 * M + 2),
               dict(starts=8 * M + 1), dict(mask=9 * M + 2), dict(block_tables=6 * M + 2),
               dict(q_token_stride=516), dict(kv_token_stride=132), dict(slot_stride=132),
               dict(out_token_stride=516)):
        assert attend(**kw) == MIS, kw


def test_workspace_size():
    f = binding.tg_tree_attention_workspace_size
    assert f(64) < f(128) < 64 << 20
    assert f(96) == 0 and f(0) == 0


def test_binding_refuses_host_tensors_and_wrong_types():
    i32, h = torch.zeros(4, dtype=torch.int32), torch.zeros(4, 2, 64, dtype=torch.float16)
    c = torch.zeros(2, 16, 2, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        binding.cache_plan(i32, i32, i32[:2], i32, i32.view(4, 1), 16, 4)
    with pytest.raises(ValueError):
        binding.cache_write(h, h, i32.long(), c, c.clone())
    with pytest.raises(ValueError):
        binding.tree_mask(i32, i32[:2], 1)
    with pytest.raises(ValueError):
        binding.tree_attention(h, h, h, c, c.clone(), i32.view(4, 1), i32, i32)


def test_header_compiles_as_strict_c99(tmp_path):
    """A C program that uses the header compiles, links and runs its host-only parts."""
    import os
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "client.c"
    src.write_text('''#include <stdio.h>
#include "tg_cache.h"
int main(void)
{
    tg_tree_attention_t a = {0};
    a.tokens = -1;
    printf("%d %d %zu %zu\\n", (int)tg_tree_attention(&a, NULL),
           (int)tg_tree_mask(NULL, 0, NULL, 0, 1, NULL, NULL, NULL), sizeof a,
           tg_tree_attention_workspace_size(128));
    return 0;
}
''')
    libdir = os.path.dirname(binding.LIB_PATH)
    subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I",
                    os.path.dirname(binding.HEADER), str(src), "-L", libdir, "-ltg_gemm",
                    f"-Wl,-rpath,{libdir}", "-o", str(tmp_path / "client")], check=True)
    out = subprocess.run([str(tmp_path / "client")], capture_output=True, text=True, timeout=120)
    import ctypes
    want = f"{BAD} {OK} {ctypes.sizeof(binding.tg_tree_attention_t)} " \
           f"{binding.tg_tree_attention_workspace_size(128)}"
    assert out.stdout.strip() == want
