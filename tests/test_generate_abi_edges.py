"""Host-side checks of edges of the rotated append, decode over shared prefixes and
sampling that the tests of their refusals and plans leave out (no GPU needed)."""
import ctypes
import os
import shutil
import subprocess
import types

import pytest
import torch

from sparse_moe_decode_router_amd import rotary, serve_layer, serving
from sparse_moe_decode_router_amd.binding import MoEError
from test_generate_abi import config, plan
from test_serve_abi import cache, status

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_moe_decode_router_amd", "csrc_serve")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


@pytest.mark.skipif(shutil.which(HIPCC) is None, reason="hipcc not available")
def test_arrays_of_a_draw_that_waves_use_at_once_are_apart(tmp_path):
    """The last scan of a row's sums reads wave_d behind its last barrier, while waves that
    are ahead write the ends of their share of the list: nothing that is written there
    may have wave_d's place."""
    src = tmp_path / "apart.hip"
    src.write_text("""
#include <cstddef>
#include "sample.h"
using namespace moe::serve;
template <int T>
constexpr bool apart(size_t at, size_t size) {
    return at + size <= offsetof(SampleLds<T>, wave_d) ||
           offsetof(SampleLds<T>, wave_d) + sizeof(SampleLds<T>::wave_d) <= at;
}
#define CHECK(T, member) \\
    static_assert(apart<T>(offsetof(SampleLds<T>, member), sizeof(SampleLds<T>::member)), #member)
#define CHECKS(T) CHECK(T, wave_u); CHECK(T, wave_i); CHECK(T, quanta); CHECK(T, list_first); \\
    CHECK(T, list_end); CHECK(T, place); CHECK(T, list)
CHECKS(0); CHECKS(1); CHECKS(kSampleF32);
""")
    run = subprocess.run(
        [HIPCC, "--offload-arch=gfx950", "--offload-host-only", "-fsyntax-only", "-std=c++17",
         "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "sparse_moe_decode_router_amd",
                                                                "csrc"), "-I", CSRC, str(src)],
        capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-3000:]


def shared_plan(window, sinks, prefix, members=16, groups=1, least=-1, longest=40000, heads=56,
                kv_heads=8):
    n = members * groups
    c = cache(kv_heads=kv_heads, head_dim=128, seqs=n, cols=4096, page=64, pages=1 << 16)
    cfg = config(q_heads=heads, batch=n, longest=longest, window=window, sinks=sinks)
    lists = [list(range(g * members, (g + 1) * members)) for g in range(groups)]
    s, p, data = plan(c, cfg, lists, [prefix] * groups, n, least)
    assert s == 0
    return p, data


@pytest.mark.parametrize("members,prefix,window,sinks", [
    (2, 131072, 64, 4), (16, 32768, 512, 4), (16, 32768, 128, 0), (64, 32768, 128, 1)])
def test_little_to_spare_within_a_window(members, prefix, window, sinks):
    """What reading a prefix apart spares is no more than members see of it: a window's
    positions and the sinks (4 KB each here)."""
    most = (members - 1) * (window + sinks) * 4096
    assert most < 40000000
    assert shared_plan(window, sinks, prefix, members)[0].units == 0
    assert shared_plan(0, 0, prefix, members)[0].units > 0
    assert shared_plan(window, sinks, prefix, members, least=most + 1)[0].units == 0
    assert shared_plan(window, sinks, prefix, members, least=most)[0].units > 0


@pytest.mark.parametrize("members,prefix,window,sinks", [
    (2, 131072, 64, 4), (16, 32768, 512, 4), (64, 65536, 4096, 0), (8, 131072, 70, 64)])
def test_parts_of_what_is_seen_of_a_prefix(members, prefix, window, sinks):
    """No more parts than there are fours of the tiles of 64 keys that a window and its sinks
    lie in, and as many workgroups as for a prefix of that length without a window."""
    p, data = shared_plan(window, sinks, prefix, members, least=0)
    tiles = -(-window // 64) + 1 + -(-sinks // 64)
    assert 1 <= p.parts <= -(-tiles // 4)
    assert p.units <= 512 or p.parts == 1
    # (a prefix that a window sees all of is cut as it is without one)
    a, b = shared_plan(prefix, 0, prefix, members, least=0), shared_plan(0, 0, prefix, members, least=0)
    assert abs(a[0].parts - b[0].parts) <= 1


def test_a_window_longer_than_the_prefix_changes_nothing():
    a, x = shared_plan(50000, 16, 8192, 64, longest=8704)
    b, y = shared_plan(0, 0, 8192, 64, longest=8704)
    assert a.units == b.units > 0 and x.tolist() == y.tolist() and a.tail == b.tail


def test_a_plan_for_longer_sequences_is_refused():
    """The workspace is that of the configuration: a plan of more positions would cut its
    sequences into more parts than there is room for."""
    c, long, short = cache(), config(longest=40000), config(longest=500)
    _, p, _ = plan(c, long, [[0, 1]], [16], 4)
    assert p.units > 0 and p.tail > 500
    p.data = 4096
    kv, at = ctypes.addressof(c), ctypes.addressof(p)
    sizes = [ctypes.byref(ctypes.c_size_t()) for _ in range(2)]
    for cfg, want in ((long, 0), (short, -1), (config(longest=40000, batch=3), -1)):
        assert status("moe_attn_shared_workspace", kv, ctypes.addressof(cfg), at, *sizes) == want
    for cfg in (short, config(longest=40000, batch=3)):
        assert status("moe_attn_decode_shared", kv, ctypes.addressof(cfg), at, 0, 4096, 0, 1792, 128,
                      4096, 4096, 4096, 4096, None) == -1
    p.slots = -1
    assert status("moe_attn_decode_shared", kv, ctypes.addressof(long), at, 0, 4096, 0, 1792, 128,
                  4096, 4096, 4096, 4096, None) == -1


def test_rotated_append_refuses_more_workgroups_than_a_grid_has():
    """Tokens of many heads take a workgroup of 256 threads each."""
    turn, c = serving.RotaryStruct(4096, 0, 128, 0, 1.0), cache()
    for tokens, want in ((1 << 24, -2), ((1 << 24) + 1, -1)):
        assert status("moe_kv_append_rotated", ctypes.addressof(c), 0, ctypes.addressof(turn), 4096,
                      1 << 17, 128, 1024, 4096, 4096, 0, 2304, 128, tokens, 4096, 4, None, 4096,
                      None) == want


@pytest.mark.parametrize("vocab", [1000, 32000, 65000])
def test_sampling_workspace_of_many_rows(vocab):
    """A row that one workgroup takes keeps its histogram and its list in LDS: beyond the 511
    rows that may have several, a row adds its sums alone, below 1 KB."""
    def size(rows):
        w, n = ctypes.c_size_t(), ctypes.c_size_t()
        assert status("moe_sample_workspace", rows, vocab, ctypes.byref(w), ctypes.byref(n)) == 0
        return w.value
    assert size(4096) - size(511) <= 1024 * (4096 - 511)
    assert size(511) <= 2 * 32768 * 1023 + 1024 * 1023


def test_amplitudes_are_held_in_32_bits():
    """(A larger one used to become infinite.)"""
    f = rotary.frequencies(64)
    rotary.Rotary(f, amplitude=-3.4e38, device="cpu")
    for bad in (3.5e38, -1e300):
        with pytest.raises(MoEError):
            rotary.Rotary(f, amplitude=bad, device="cpu")


@pytest.mark.parametrize("kw", [
    dict(steps=0), dict(continuations=0), dict(prompts=()), dict(prompts=(5, 0)), dict(vocab=0),
    dict(layer=dict(vocab=501)), dict(layer=dict(vocab=0)), dict(layer=dict(rotary=None)),
    dict(layer=dict(seqs=5)), dict(layer=dict(lengths=[0, 0, 7, 0, 0, 0]))], ids=str)
def test_generate_refuses(kw):
    """(Tokens beyond a layer's embedding used to be looked up in it, and sequences that a cache
    held already were taken for parts of the prompts.)"""
    own = {**dict(vocab=500, rotary=1, seqs=6, lengths=[0] * 6), **kw.pop("layer", {})}
    layer = types.SimpleNamespace(rotary=own["rotary"], vocab=own["vocab"], kv=types.SimpleNamespace(
        seqs=own["seqs"], lengths=torch.tensor(own["lengths"])))
    with pytest.raises(MoEError):
        serve_layer.generate(**{**dict(steps=4, prompts=(70, 33), continuations=3, vocab=500,
                                       layer=layer), **kw})


@pytest.mark.parametrize("kw,in_place", [
    (dict(), False), (dict(qts=14 * 128), True), (dict(qts=14 * 128, qhs=256), False),
    (dict(tokens=1, batch=1), True), (dict(tokens=1, batch=1, qts=0), True),
    (dict(q_heads=1, qhs=0, qts=128), True), (dict(q_heads=1, qhs=0, qts=256), False)], ids=str)
def test_rotated_append_in_place_needs_queries_without_gaps(kw, in_place):
    """(Here there is no device: what is not refused for its arguments gets as far as that.)"""
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    turn, c = serving.RotaryStruct(4096, 0, 128, 0, 1.0), cache()
    args = dict(kv=ctypes.addressof(c), layer=0, rotary=ctypes.addressof(turn), q=4096, qts=2304,
                qhs=128, q_heads=14, k=8192, v=8192, dtype=0, ts=2304, hs=128, tokens=2, cu=None,
                batch=2, granted=None, out=4096, stream=None)
    assert status("moe_kv_append_rotated", *{**args, **kw}.values()) == (-3 if in_place else -1)
