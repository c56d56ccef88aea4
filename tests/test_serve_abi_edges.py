"""Host-side checks of the serving operators at the ends of their ranges (no GPU
needed)."""
import ctypes
import types

import pytest
import torch

from sparse_moe_decode_router_amd import attention, serving
from sparse_moe_decode_router_amd.binding import MoEError
from test_serve_abi import cache, status


def workspace(c, cfg, tokens):
    w, n = ctypes.c_size_t(), ctypes.c_size_t()
    assert status("moe_attn_workspace", ctypes.addressof(c), ctypes.addressof(cfg), tokens,
                  ctypes.byref(w), ctypes.byref(n)) == 0
    return w.value, n.value


@pytest.mark.parametrize("batch", [1, 16, 64, 256, 4096])
@pytest.mark.parametrize("heads,kv_heads,dim,longest,window", [
    (56, 8, 128, 131072, 0), (7, 1, 128, 131072, 0), (14, 2, 64, 8192, 4096),
    (64, 64, 256, 32768, 0), (1024, 1, 192, 131072, 0)])
def test_the_workspace_of_prompts_has_a_bound(heads, kv_heads, dim, longest, window, batch):
    """Whatever the batch and the length planned for: four partial results (128 rows
    of outputs, a maximum and a sum) for each workgroup that fits on the chip, or
    two for each equal share; and for few tokens no more than their rows take."""
    c = cache(kv_heads=kv_heads, head_dim=dim, seqs=4096, cols=8192, pages=1 << 20)
    cfg = serving.AttnConfig(heads, batch, longest, window, 0, 0.1)
    slots, group = 512 if dim <= 128 else 256, heads // kv_heads
    row_tile = 4 * 128 * (dim + 2)
    for tokens in (1, 2, 16, 100, 1000, 8192, 1 << 20):
        w, n = workspace(c, cfg, tokens)
        assert w <= row_tile * 4 * slots
        tiles = tokens * group // 128 + min(batch, tokens)
        assert w <= row_tile * 64 * tiles * kv_heads and n == 4 * tiles * kv_heads


def test_decode_refuses_more_workgroups_than_a_grid_has():
    """(Their number used to wrap round; here it would be 4096 times 2^24.)"""
    c = cache(kv_heads=64, head_dim=64, seqs=1 << 24, cols=1)
    for batch, want in ((1 << 24, -2), (1 << 13, -2)):
        cfg = serving.AttnConfig(64 * 1024, batch, 16, 0, 0, 0.1)
        assert status("moe_attn_decode", ctypes.addressof(c), ctypes.addressof(cfg), 0, 4096, 0,
                      64 * 1024 * 64, 64, batch, 4096, 4096, 4096, 4096, None) == want


@pytest.mark.parametrize("kw", [dict(window=(1 << 32) + 5), dict(longest=(1 << 32) + 500),
                                dict(sinks=-(1 << 32)), dict(batch=(1 << 32) + 1), dict(window=1.5),
                                dict(window=-1), dict(q_heads=(1 << 32) + 4)])
def test_plans_refuse_numbers_beyond_32_bits(kw):
    """They used to be cut to their low 32 bits."""
    c = cache(head_dim=64)
    kv = types.SimpleNamespace(_ref=ctypes.addressof(c), head_dim=64, kv_heads=2,
                               device=torch.device("cuda", 0))
    plan = dict(q_heads=4, batch=2, longest=100)
    attention.PagedAttention(kv, **plan)
    with pytest.raises(MoEError):
        attention.PagedAttention(kv, **{**plan, **kw})
