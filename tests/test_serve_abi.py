"""Host-side checks of the serving operators' C ABI (no GPU needed): exports,
refusals of arguments, workspace sizes; and the 64-bit references the GPU tests
rest on, against plain torch."""
import ctypes
import math
import os
import re

import pytest
import torch

import serve_util as su
from sparse_moe_decode_router_amd import attention, serving, w4
from sparse_moe_decode_router_amd.binding import MoEError

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_header_and_module_agree():
    text = open(os.path.join(ROOT, "include", "moe_serve.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(moe_\w+)\s*\(", text)))
    assert names == sorted(serving.EXPORTED)
    for n in names:
        assert hasattr(serving.lib(), n)


def test_refuses_to_run_without_the_library(tmp_path, monkeypatch):
    monkeypatch.setattr(serving, "_lib", None)
    monkeypatch.setattr(serving, "LIB_PATH", str(tmp_path / "missing.so"))
    with pytest.raises(MoEError):
        serving.lib()


# Addresses that only have to look right: no call here gets as far as the GPU.
OK = dict(data=4096, tables=4096, lengths=4096, refs=4096, k_scale=None, v_scale=None, flags=4096,
          dtype=0, layers=2, pages=100, kv_heads=2, page=16, head_dim=128, seqs=4, cols=32)


def cache(**kw):
    return serving.Cache(*[{**OK, **kw}[n] for n, _ in serving.Cache._fields_])


def status(f, *args):
    return getattr(serving.lib(), f)(*args)


@pytest.mark.parametrize("kw,want", [
    ({}, 0), (dict(dtype=2, k_scale=4096), 0), (dict(page=1024), 0), (dict(head_dim=96), 0),
    (dict(data=None), -1), (dict(data=4104), -1), (dict(tables=None), -1), (dict(flags=None), -1),
    (dict(pages=0), -1), (dict(cols=0), -1), (dict(dtype=3), -1), (dict(v_scale=4096), -1),
    (dict(page=8), -2), (dict(page=24), -2), (dict(page=2048), -2), (dict(head_dim=80), -2),
    (dict(head_dim=0), -2), (dict(seqs=1 << 16, cols=1 << 15), -2), (dict(cols=1 << 27), -2),
])
def test_cache_checks(kw, want):
    c = cache(**kw)
    assert status("moe_kv_validate", ctypes.addressof(c)) == want


@pytest.mark.parametrize("kw,want", [
    ({}, 0), (dict(window=5, sinks=3), 0), (dict(q_heads=34), 0), (dict(q_heads=7), -1),
    (dict(q_heads=0), -1), (dict(batch=5), -1), (dict(batch=0), -1), (dict(longest=0), -1),
    (dict(window=-1), -1), (dict(sinks=-1), -1), (dict(scale=0.0), -1),
    (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
])
def test_attention_checks(kw, want):
    base = dict(q_heads=14, batch=4, longest=500, window=0, sinks=0, scale=0.1)
    cfg = serving.AttnConfig(*[{**base, **kw}[n] for n, _ in serving.AttnConfig._fields_])
    assert status("moe_attn_validate", ctypes.addressof(cache()), ctypes.addressof(cfg)) == want


def test_calls_refuse_before_any_launch():
    c, cfg = cache(), serving.AttnConfig(14, 4, 500, 0, 0, 0.1)
    kv, at = ctypes.addressof(c), ctypes.addressof(cfg)
    append = lambda **k: status("moe_kv_append", *{**dict(  # noqa: E731
        kv=kv, layer=0, k=4096, v=4096, dtype=0, ts=256, hs=128, tokens=2, cu=None, batch=2,
        stream=None), **k}.values())
    for k in (dict(layer=2), dict(layer=-1), dict(dtype=1), dict(dtype=2), dict(ts=255), dict(hs=64),
              dict(hs=-128), dict(k=4100), dict(v=None), dict(tokens=-1), dict(batch=5, tokens=5),
              dict(tokens=3)):
        assert append(**k) == -1, k
    assert append(tokens=0, batch=0) == 0
    decode = lambda **k: status("moe_attn_decode", *{**dict(  # noqa: E731
        kv=kv, cfg=at, layer=0, q=4096, dtype=0, ts=1792, hs=128, batch=4, out=4096, lse=4096,
        ws=4096, ctr=4096, stream=None), **k}.values())
    for k in (dict(cfg=None), dict(kv=None), dict(layer=2), dict(q=None), dict(q=8), dict(dtype=1),
              dict(ts=4), dict(hs=8), dict(batch=0), dict(batch=5), dict(out=None), dict(lse=None)):
        assert decode(**k) == -1, k
    assert decode(ws=None) == -4 and decode(ctr=None) == -4 and decode(ws=4104) == -4
    prompt = lambda **k: status("moe_attn_prompt", *{**dict(  # noqa: E731
        kv=kv, cfg=at, layer=0, q=4096, dtype=0, ts=1792, hs=128, tokens=9, cu=4096, batch=4,
        out=4096, lse=4096, ws=4096, ctr=4096, stream=None), **k}.values())
    for k in (dict(cu=None), dict(tokens=-1), dict(batch=0), dict(out=8)):
        assert prompt(**k) == -1, k
    assert prompt(tokens=0) == 0
    for f, args in (("moe_kv_free", (4096, 5, None)), ("moe_kv_free", (None, 1, None)),
                    ("moe_kv_fork", (4096, None, 1, 4096, None)),
                    ("moe_kv_fork", (4096, 4096, -1, 4096, None)),
                    ("moe_kv_extend", (None, None, 1, 4096, None)),
                    ("moe_kv_compact", (None, 4096, 4096, None))):
        assert status(f, kv, *args) == -1, f
    for f, args in (("moe_kv_fork", (4096, 4096, 1, None, None)),
                    ("moe_kv_extend", (None, 4096, 1, None, None)),
                    ("moe_kv_compact", (4096, 4096, None, None))):
        assert status(f, kv, *args) == -4, f
    assert status("moe_kv_free", kv, None, 0, None) == 0
    w = lambda **k: status("moe_w4_linear", *{**dict(  # noqa: E731
        x=4096, xs=128, dtype=0, codes=4096, scales=4096, zeros=None, t=1, k=128, n=8, group=64,
        y=4096, stream=None), **k}.values())
    for k in (dict(x=None), dict(x=8), dict(xs=12), dict(dtype=2), dict(codes=None), dict(y=None),
              dict(codes=8), dict(t=-1), dict(n=0)):
        assert w(**k) == -1, k
    assert w(group=16) == -2 and w(group=256) == -2 and w(k=96) == -2
    assert w(t=0) == 0


def test_w4_refuses_strides_beyond_its_offsets():
    args = lambda xs: (4096, xs, 0, 4096, 4096, None, 1, 128, 8, 64, 4096,  # noqa: E731
                       None)
    assert status("moe_w4_linear", *args((1 << 25) + 8)) == -2


def test_workspace_sizes():
    c, cfg = cache(), serving.AttnConfig(14, 4, 500, 0, 0, 0.1)
    w, n = ctypes.c_size_t(), ctypes.c_size_t()
    size = lambda t: (status("moe_attn_workspace", ctypes.addressof(c), ctypes.addressof(cfg),  # noqa: E731
                             t, ctypes.byref(w), ctypes.byref(n)), w.value, n.value)
    rc, ws, ctr = size(0)
    # at most a unit per 128 positions, and one more per sequence, each of 16
    # rows of outputs, maxima and sums; a counter per (sequence, kv head)
    assert (rc, ctr) == (0, 4 * 2 * 4) and 0 < ws <= 4 * 16 * 130 * 2 * (4 * 4 + 4)
    assert size(-1)[0] == -1
    rc, ws, ctr = size(20000)             # equal shares: two parts for each, whatever the tokens
    assert rc == 0 and ws >= 4 * 128 * 130 * 2 * 512 and ctr >= 4 * 2 * (20000 * 7 // 128)
    assert size(1 << 20)[:2] == (0, ws)
    assert serving.lib().moe_kv_scratch_size(ctypes.addressof(c), 4) >= 4 * 3 * 100


@pytest.mark.parametrize("heads,kv_heads,dim,longest,window", [
    (4, 1, 128, 8192, 0), (14, 2, 128, 8192, 4096), (7, 1, 256, 3000, 0), (64, 64, 64, 500, 0),
    (1, 1, 128, 131072, 0)])
def test_a_space_for_more_tokens_serves_fewer(heads, kv_heads, dim, longest, window):
    """Fewer tokens are split into more parts, and still have room."""
    c = cache(kv_heads=kv_heads, head_dim=dim, cols=8192)
    cfg = serving.AttnConfig(heads, 3, longest, window, 0, 0.1)
    w, n = ctypes.c_size_t(), ctypes.c_size_t()
    slots, group = 512 if dim <= 128 else 256, heads // kv_heads
    keys = min(longest, window + 128) if window else longest
    last = (0, 0)
    for t in sorted({*range(1, 300), *(2 ** i + d for i in range(4, 21) for d in (-1, 0, 1))}):
        assert status("moe_attn_workspace", ctypes.addressof(c), ctypes.addressof(cfg), t,
                      ctypes.byref(w), ctypes.byref(n)) == 0
        assert (w.value, n.value) >= last and n.value >= last[1]
        last = (w.value, n.value)
        # What a call of that many tokens can take: a part for every row tile and
        # split, as many as the chip holds at once, or two for each equal share.
        full, tiles = t * group // 128, t * group // 128 + min(3, t)
        sure = max(1, full) * kv_heads
        key_tiles = -(-keys // 64)
        split = max(1, min(slots // sure, key_tiles // 4, math.isqrt(key_tiles - 1) + 1, 64))
        need = 2 * (slots // kv_heads) if sure > slots else tiles * split if split > 1 else 0
        assert w.value >= 4 * 128 * (dim + 2) * need * kv_heads
        assert n.value >= 4 * tiles * kv_heads


def test_modules_refuse_cpu_tensors():
    z = torch.zeros
    with pytest.raises(MoEError):
        attention.PagedKV(z((1, 2, 4, 1, 16, 64), dtype=torch.bfloat16), z((1, 4), dtype=torch.int32),
                          z(1, dtype=torch.int32), z(4, dtype=torch.int32))
    with pytest.raises(MoEError):
        w4.W4Linear(z((4, 64), dtype=torch.uint8), z((4, 1), dtype=torch.bfloat16))


def test_reference_attention_is_softmax_attention():
    """Without a window the reference is torch's own attention in 64 bits."""
    c = su.HostCache([40], 2, 16, 64, seed=1)
    q = torch.randn(40, 6, 64).to(torch.bfloat16)
    out, lse, _, _ = su.attention(c, 0, q, [0, 40])
    k, v = (c.row(0, w, 0, 40)[0].transpose(0, 1).repeat_interleave(3, 0) for w in (0, 1))
    want = torch.nn.functional.scaled_dot_product_attention(q.double().transpose(0, 1), k, v,
                                                            is_causal=True)
    assert torch.allclose(out.transpose(0, 1), want, rtol=1e-12, atol=1e-12)
    win, _, _, _ = su.attention(c, 0, q, [0, 40], window=7, sinks=2)
    t = torch.arange(40)
    sees = (t[None] <= t[:, None]) & ((t[None] > t[:, None] - 7) | (t[None] < 2))
    want = torch.nn.functional.scaled_dot_product_attention(q.double().transpose(0, 1), k, v,
                                                            attn_mask=sees)
    assert torch.allclose(win.transpose(0, 1), want, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("window,sinks", [(0, 0), (9, 3)])
def test_reference_attention_of_many_heads(window, sinks):
    c = su.HostCache([50, 20, 0], 2, 16, 64, seed=2)
    cu = [0, 30, 50, 52]
    q = torch.randn(52, 6, 64).to(torch.bfloat16)
    for a, b in zip(su.attention(c, 0, q, cu, window, sinks),
                    su.attention_dense(c, 0, q, cu, window, sinks)):
        assert torch.allclose(a, b, rtol=1e-9, atol=1e-12)


def test_reference_w4():
    codes = torch.tensor([[0x21, 0x43] * 16], dtype=torch.uint8)
    w = su.w4_weights(codes, None, 32)
    assert w[0, :4].tolist() == [-7.0, -6.0, -5.0, -4.0]
    x = torch.ones((1, 64), dtype=torch.bfloat16)
    y, _ = su.w4(x, codes, torch.full((1, 2), 0.5, dtype=torch.bfloat16), None, 32)
    assert y.item() == -22.0 * 16 * 0.5
