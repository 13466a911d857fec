"""How attention over the 4-bit cache is divided: the rule, and that the GPU tests' sizes reach the kernels they are for."""

import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_block_scaled_nvfp4_amd", "csrc")

CALL = '''
#include "attention_internal.h"
extern "C" void test_plan(int64_t t, int64_t h, int64_t kv, int64_t d, int64_t r, int64_t mq, int64_t ms, int64_t* out) {
  const nvfp4::AttnPlan p = nvfp4::plan_attention_fp4(t, h, kv, d, r, mq < t ? mq : t, ms);
  const int64_t v[] = {(int64_t)p.kernel, p.rows, p.join_rows, p.workers, p.row_tiles, p.workspace, p.wide};
  for (int i = 0; i < 7; ++i) out[i] = v[i];
}
'''


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    tmp = tmp_path_factory.mktemp("plan4")
    call = tmp / "call.cpp"
    call.write_text(CALL)
    lib = tmp / "libplan4.so"
    subprocess.run(["g++", "-x", "c++", "-std=c++17", "-O1", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", os.path.join(CSRC, "attention_plan.hip"), str(call), "-o", str(lib)],
                   check=True, capture_output=True, text=True)
    fn = ctypes.CDLL(str(lib)).test_plan
    fn.argtypes = [ctypes.c_int64] * 7 + [ctypes.POINTER(ctypes.c_int64)]
    fn.restype = None

    def get(tokens, heads, kv_heads, head_dim, requests, new, longest):
        out = (ctypes.c_int64 * 7)()
        fn(tokens, heads, kv_heads, head_dim, requests, new, longest, out)
        return dict(zip(("kernel", "rows", "join_rows", "workers", "row_tiles", "workspace", "wide"), out))

    return get


@pytest.mark.parametrize("head_dim", [64, 128, 256])
@pytest.mark.parametrize("rows,short,long", [(1, 16, 16), (16, 16, 16), (17, 32, 32), (32, 32, 32), (33, 32, 48), (48, 32, 48), (49, 32, 32),
                                             (64, 32, 32), (65, 32, 48), (96, 32, 48), (97, 256, 256), (600, 256, 256)])
def test_rows_of_a_tile(plan, head_dim, rows, short, long):
    for longest, want in ((4095, short), (4096, long), (100000, long)):
        if head_dim == 256 and want == 48:
            want = 32  # no registers for 48 rows of 256 dims
        p = plan(16 * rows, 4, 4, head_dim, 16, rows, longest)
        assert p["rows"] == want and p["kernel"] == {16: 0, 32: 1, 256: 2, 48: 3}[want], (longest, p)
        assert p["join_rows"] == min(rows, want) and p["row_tiles"] * want >= rows
        assert (p["workers"] > 0) == (p["workspace"] > 0) and p["workers"] % 256 == 0


def test_sizes_of_the_gpu_tests_reach_48_rows(plan):
    for new, heads, kv_heads in ((11, 3, 1), (12, 8, 2), (48, 2, 2), (13, 10, 2), (24, 4, 1), (33, 4, 2)):
        assert plan(2 * new + new // 2, heads, kv_heads, 128, 4, new, 5000)["rows"] == 48
    p = plan(130 * 8, 32, 8, 64, 130, 9, 5000)
    assert p["rows"] == 48 and p["workers"] == 0


@pytest.mark.parametrize("head_dim", [64, 128, 256])
def test_eight_wavefronts(plan, head_dim):
    """Where a workgroup has the keys to itself, more than one step of them and a compute unit of its own."""
    wide = lambda requests, rows, longest: plan(requests * rows, 4, 4, head_dim, requests, rows, longest)["wide"]  # noqa: E731
    assert bool(wide(1, 1, 500)) == bool(wide(64, 16, 1024)) == bool(wide(64, 1, 257)) == (head_dim <= 128)
    assert bool(wide(8, 32, 1024)) == bool(wide(8, 40, 1024)) == bool(wide(1, 300, 1024)) == (head_dim == 64)
    assert not wide(65, 1, 1024) and not wide(1, 1, 256) and not wide(1, 1, 1025) and not wide(64, 300, 1024)
    for requests, rows, longest in ((3, 7, 500), (300, 1, 500), (3, 7, 5000), (64, 48, 1024)):
        p = plan(requests * rows, 4, 4, head_dim, requests, rows, longest)
        assert not (p["wide"] and p["workers"])
