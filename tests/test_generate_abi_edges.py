"""Host-side checks of edges of the rotated append, decode over shared prefixes and
sampling that the tests of their refusals and plans leave out (no GPU needed)."""
import os
import shutil
import subprocess

import pytest

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
