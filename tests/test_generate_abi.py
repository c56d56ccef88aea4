"""Host-side checks of the rotated append, decode over shared prefixes and sampling (no
GPU needed): refusals of arguments, plans and workspace sizes; and the 64-bit
references the GPU tests rest on."""
import ctypes
import math

import numpy as np
import pytest
import torch

import generate_util as gu
from sparse_moe_decode_router_amd import attention, rotary, sampling, serving
from sparse_moe_decode_router_amd.binding import MoEError
from test_serve_abi import cache, status


def config(**kw):
    base = dict(q_heads=14, batch=4, longest=500, window=0, sinks=0, scale=0.1)
    return serving.AttnConfig(*[{**base, **kw}[n] for n, _ in serving.AttnConfig._fields_])


@pytest.mark.parametrize("kw", [
    dict(turns=None), dict(turns=4100), dict(first=8), dict(first=-16), dict(rot=0), dict(rot=24),
    dict(rot=144), dict(first=64, rot=80), dict(first=144, rot=16), dict(interleaved=2)])
def test_rotated_append_refuses_rotations(kw):
    turn = serving.RotaryStruct(*[{**dict(turns=4096, first=0, rot=128, interleaved=0, amplitude=1.0),
                                   **kw}[n] for n, _ in serving.RotaryStruct._fields_])
    c = cache()
    assert status("moe_kv_append_rotated", ctypes.addressof(c), 0, ctypes.addressof(turn), 4096, 2304,
                  128, 14, 4096, 4096, 0, 2304, 128, 2, None, 2, None, 4096, None) == -1


@pytest.mark.parametrize("kw,want", [
    (dict(rotary=None), -1), (dict(layer=2), -1), (dict(q=None), -1), (dict(q=4104), -1),
    (dict(out=None), -1), (dict(out=4104), -1), (dict(qts=2300), -1), (dict(qhs=64), -1),
    (dict(q_heads=0), -1), (dict(q_heads=1 << 21), -2), (dict(k=4104), -1), (dict(v=None), -1),
    (dict(dtype=1), -1), (dict(dtype=3), -1), (dict(hs=120), -1), (dict(tokens=3), -1),
    (dict(tokens=-1), -1), (dict(batch=5, tokens=5), -1), (dict(tokens=0, batch=0), 0)])
def test_rotated_append_refuses_arguments(kw, want):
    turn, c = serving.RotaryStruct(4096, 0, 128, 0, 1.0), cache()
    args = dict(kv=ctypes.addressof(c), layer=0, rotary=ctypes.addressof(turn), q=4096, qts=2304,
                qhs=128, q_heads=14, k=4096, v=4096, dtype=0, ts=2304, hs=128, tokens=2, cu=None,
                batch=2, granted=None, out=4096, stream=None)
    assert status("moe_kv_append_rotated", *{**args, **kw}.values()) == want


def plan(c, cfg, groups, prefix, batch, least=0):
    """(status, plan, its data as an array)"""
    cu = [0]
    for g in groups:
        cu.append(cu[-1] + len(g))
    arr = lambda v: (ctypes.c_int32 * max(1, len(v)))(*v)  # noqa: E731
    p = serving.SharedPlan()
    args = (ctypes.addressof(c), ctypes.addressof(cfg), batch, len(groups), arr(cu),
            arr([m for g in groups for m in g]), arr(prefix), least, ctypes.addressof(p))
    s = status("moe_attn_share", *args, None)
    if s:
        return s, p, None
    data = np.full(p.ints + 8, -77, dtype=np.int32)
    s = status("moe_attn_share", *args, data.ctypes.data)
    assert np.all(data[p.ints:] == -77)
    return s, p, data[:p.ints]


@pytest.mark.parametrize("groups,prefix,batch", [
    ([[0, 4]], [16], 4), ([[0, -1]], [16], 4), ([[0, 1], [1]], [16, 16], 4), ([[0, 1]], [-1], 4),
    ([[0, 1]], [16], 5), ([[0]], [16], 0), ([[0, 1, 2, 3, 0]], [16], 4)])
def test_share_refuses(groups, prefix, batch):
    assert plan(cache(), config(), groups, prefix, batch)[0] == -1


@pytest.mark.parametrize("heads,kv_heads,dim,groups,members,prefix,window,sinks", [
    (14, 2, 128, 1, 2, 16, 0, 0), (56, 8, 128, 1, 64, 8192, 0, 0), (56, 8, 128, 4, 16, 32768, 0, 0),
    (14, 2, 256, 3, 5, 1000, 0, 0), (1024, 1, 64, 2, 200, 5000, 0, 0), (8, 8, 64, 100, 2, 64, 0, 0),
    (14, 2, 128, 2, 4, 500, 100, 16), (14, 2, 128, 2, 4, 500, 100, 501), (14, 2, 128, 5, 1, 500, 0, 0),
    (7, 1, 128, 1, 8, 0, 0, 0), (7, 1, 128, 1, 8, 10 ** 9, 0, 0)])
def test_a_plan_takes_every_row_and_key_once(heads, kv_heads, dim, groups, members, prefix, window,
                                             sinks):
    """Units cover each row tile with all of its parts, in slots of their own that the rows
    find again; sequences know their prefix, or have none."""
    n, page = groups * members, 64
    c = cache(kv_heads=kv_heads, head_dim=dim, seqs=n, cols=4096, page=page, pages=1 << 20)
    cfg = config(q_heads=heads, batch=n, longest=40000, window=window, sinks=sinks)
    order = np.random.RandomState(1).permutation(n).tolist()
    lists = [order[g * members:(g + 1) * members] for g in range(groups)]
    prefixes = [prefix - g for g in range(groups)] if prefix > groups else [prefix] * groups
    s, p, data = plan(c, cfg, lists, prefixes, n)
    assert s == 0 and p.ints == len(data) and p.slots * kv_heads == p.units
    units, tiles = (data[8 * i:8 * j].reshape(-1, 8) for i, j in
                    ((0, p.units), (p.units, p.units + p.tiles)))
    own, flat = data[8 * (p.units + p.tiles):][:n], data[8 * (p.units + p.tiles) + n:]
    assert flat.tolist() == order
    assert sorted(units[:, [6, 7]].tolist()) == [[i, h] for i in range(p.slots) for h in range(kv_heads)]
    group = heads // kv_heads
    slots = {}
    for first, count, pre, row0, part, parts, slot, head in units.tolist():
        assert 0 <= part < parts <= 128 and row0 % 128 == 0 and row0 < count * group
        assert slots.setdefault((first, row0, part), slot) == slot
    used, tile = 0, 0
    for g, members_of in enumerate(lists):
        apart = len(members_of) > 1 and prefixes[g] > 0 and (window == 0 or sinks <= prefixes[g])
        assert all(own[m] == (prefixes[g] if apart else 0) for m in members_of)
        for row0 in range(0, len(members_of) * group, 128) if apart else ():
            first, count, pre, at, part, parts, slot, _ = tiles[tile].tolist()
            assert (first, count, pre, at, part) == (g * members, members, prefixes[g], row0, 0)
            assert [slots[(first, row0, i)] for i in range(parts)] == list(range(slot, slot + parts))
            tile, used = tile + 1, used + parts
    assert tile == p.tiles
    assert used == p.slots
    assert 1 <= p.tail <= 40000
    # one round of workgroups where that is possible, never more than four
    at_once = 512 if dim <= 128 else 256
    least = sum(-(-len(g) * group // 128) for g in lists)
    assert p.units <= max(4 * at_once, least * kv_heads)


def test_shared_calls_refuse():
    c, cfg = cache(), config()
    _, p, _ = plan(c, cfg, [[0, 1]], [16], 4)
    p.data = 4096
    kv, at = ctypes.addressof(c), ctypes.addressof(cfg)
    w, n = ctypes.c_size_t(), ctypes.c_size_t()
    d, m = ctypes.c_size_t(), ctypes.c_size_t()
    assert status("moe_attn_shared_workspace", kv, at, ctypes.addressof(p), ctypes.byref(w),
                  ctypes.byref(n)) == 0
    assert status("moe_attn_workspace", kv, at, 0, ctypes.byref(d), ctypes.byref(m)) == 0
    assert w.value >= d.value + 4 * 128 * 130 * p.slots * 2 and n.value == m.value
    call = lambda **k: status("moe_attn_decode_shared", *{**dict(  # noqa: E731
        kv=kv, cfg=at, plan=ctypes.addressof(p), layer=0, q=4096, dtype=0, ts=1792, hs=128, out=4096,
        lse=4096, ws=4096, counters=4096, stream=None), **k}.values())
    for k in (dict(plan=None), dict(layer=2), dict(q=None), dict(dtype=1), dict(ts=1790), dict(hs=64),
              dict(out=4104), dict(lse=None)):
        assert call(**k) == -1
    assert call(ws=None) == call(counters=None) == call(ws=4100) == -4
    for name, value in (("data", None), ("data", 4100), ("q_heads", 28), ("kv_heads", 1),
                        ("head_dim", 64), ("window", 5), ("batch", 5), ("units", -1)):
        other = serving.SharedPlan.from_buffer_copy(p)
        setattr(other, name, value)
        assert call(plan=ctypes.addressof(other)) == -1
        if name in ("q_heads", "kv_heads", "head_dim"):
            assert status("moe_attn_shared_workspace", kv, at, ctypes.addressof(other),
                          ctypes.byref(w), ctypes.byref(n)) == -1


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), -1), (dict(dtype=4), -1), (dict(rows=-1), -1), (dict(vocab=0), -1),
    (dict(stride=99), -1), (dict(filters=None), -1), (dict(x=None), -1), (dict(x=4098), -1),
    (dict(u=None), -1), (dict(token=None), -1), (dict(lp=4098), -1), (dict(ws=None), -4),
    (dict(counters=4100), -4), (dict(vocab=(1 << 19) + 1, stride=1 << 20), -2),
    (dict(stride=1 << 41), -2), (dict(rows=1 << 21), -2), (dict(rows=0), 0),
    (dict(filters="top_k"), -1)])
def test_sampling_refuses(kw, want):
    good, odd = serving.SamplingStruct(), serving.SamplingStruct(top_k=4098)
    args = dict(x=4096, dtype=3, stride=100, rows=2, vocab=100, u=4096,
                filters=ctypes.addressof(good), token=4096, lp=4096, ws=4096, counters=4096,
                stream=None)
    kw = {k: ctypes.addressof(odd) if v == "top_k" else v for k, v in kw.items()}
    assert status("moe_sample", *{**args, **kw}.values()) == want


def test_sampling_workspace_grows_with_its_rows():
    w, n, last = ctypes.c_size_t(), ctypes.c_size_t(), 0
    for vocab in (1, 1000, 163840, 1 << 19):
        last = 0
        for rows in (1, 2, 3, 7, 64, 65, 300, 1024, 5000):
            assert status("moe_sample_workspace", rows, vocab, ctypes.byref(w), ctypes.byref(n)) == 0
            assert w.value >= last and n.value == 4 * rows
            last = w.value
    for bad in ((0, 10), (10, 0)):
        assert status("moe_sample_workspace", *bad, ctypes.byref(w), ctypes.byref(n)) == -1
    assert status("moe_sample_workspace", 1 << 21, 10, ctypes.byref(w), ctypes.byref(n)) == -2


def test_modules_refuse():
    for f in (lambda: rotary.frequencies(15), lambda: rotary.frequencies(64, base=0),
              lambda: rotary.frequencies(64, factor=-1), lambda: rotary.frequencies(64, slow=9, fast=9)):
        with pytest.raises(MoEError):
            f()
    f = rotary.frequencies(64)
    for kw in (dict(frequencies=f[:4]), dict(frequencies=f[None]), dict(first=8), dict(first=-16),
               dict(first=208), dict(amplitude=math.inf), dict(frequencies=f * math.nan)):
        with pytest.raises(MoEError):
            rotary.Rotary(**{**dict(frequencies=f, device="cpu"), **kw})
    for a in ((0, 10), (10, 0), (1.5, 10), (10, 1 << 20)):
        with pytest.raises(MoEError):
            sampling.Sampler(*a)


def test_frequencies():
    f = rotary.frequencies(8, 10000.0)
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64))
    assert torch.equal(rotary.frequencies(8, factor=4.0), f / 4)
    g = rotary.frequencies(128, 10000.0, factor=8.0, original=4096)
    plain = rotary.frequencies(128)
    turns = 4096 * plain / (2 * math.pi)
    assert torch.equal(g[turns >= 32], plain[turns >= 32])
    assert torch.equal(g[turns <= 1], plain[turns <= 1] / 8)
    assert torch.all(g[1:] < g[:-1])


def test_reference_rotation_is_a_complex_product():
    x = torch.randn((3, 2, 32), dtype=torch.float64)
    f = rotary.frequencies(16, 100.0)
    for pairs in (False, True):
        y, _ = gu.rotate(x, [0, 5, -1], f, 16, pairs, 2.0)
        assert torch.equal(y[2], x[2]) and torch.equal(y[..., :16], x[..., :16])
        z = x[..., 16:].unflatten(-1, (8, 2) if pairs else (2, 8))
        z = torch.complex(z[..., 0], z[..., 1]) if pairs else torch.complex(z[..., 0, :], z[..., 1, :])
        z = 2 * z * torch.exp(1j * torch.tensor([0.0, 5.0, 0.0])[:, None, None] * f)
        got = y[..., 16:].unflatten(-1, (8, 2) if pairs else (2, 8))
        got = torch.complex(got[..., 0], got[..., 1]) if pairs else \
            torch.complex(got[..., 0, :], got[..., 1, :])
        assert torch.allclose(got[:2], z[:2])


def test_reference_sampling():
    """Over a grid of u each token comes up as often as the filtered weights say."""
    x = [1.0, 3.0, -math.inf, 3.0, 2.0, math.nan, 0.0]
    n = 4000
    for kw, keep in ((dict(), [0, 1, 3, 4, 6]), (dict(top_k=1), [1]), (dict(top_k=3), [1, 3, 4]),
                     (dict(top_p=0.3), [1]), (dict(top_p=0.6), [1, 3]), (dict(min_p=0.3), [1, 3, 4]),
                     (dict(top_k=4, top_p=0.9), [1, 3, 4])):
        kw = {**dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0), **kw}
        got = [gu.sample(x, (i + 0.5) / n, **kw) for i in range(n)]
        count = np.bincount([t for t, _ in got], minlength=7) / n
        w = np.array([math.exp(x[i]) if i in keep else 0.0 for i in range(7)])
        assert np.abs(count - w / w.sum()).max() <= 1.0001 / n
        assert all(abs(lp - math.log(w[t] / w.sum())) < 1e-12 for t, lp in got)
    assert gu.sample(x, 0.9, 0.0, 0, 1.0, 0.0) == (1, 0.0)
    assert gu.sample([-math.inf, math.nan], 0.5, 1.0, 0, 1.0, 0.0)[0] == -1
