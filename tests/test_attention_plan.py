"""The division of an attention call's work (csrc/attention_plan.hip) on the CPU: built with the host layer under the
address and undefined-behaviour sanitizers and called over its whole range, and the kernels and
divisions that the GPU tests' sizes and bounds lead to."""

import ctypes
import os
import random
import subprocess
import sys

import pytest

from .test_asan_host import _asan_runtime
from .test_abi import _gpu_visible

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_block_scaled_nvfp4_amd", "csrc")

pytestmark = pytest.mark.skipif(_gpu_visible(), reason="host-only build with stubbed launchers")

STUBS = '''
#include "attention_internal.h"
namespace nvfp4 {
hipError_t launch_block_tables(const TablesArgs&, hipStream_t) { return hipSuccess; }
// what the kernels take for granted about a plan
hipError_t launch_attention(const AttnArgs& a, const AttnPlan& p, int head_dim, bool, hipStream_t) {
  const bool ok = a.workers == p.workers && a.row_tiles == p.row_tiles && a.all_tiles == p.all_tiles && p.rows % 16 == 0 &&
                  p.row_tiles >= 1 && p.row_tiles <= 65535 && p.all_tiles >= 0 && p.all_tiles <= 65535 && a.requests <= 65535 &&
                  p.workers % kComputeUnits == 0 && (p.workers == 0) == (p.workspace == 0) && p.join_rows >= 1 && p.join_rows <= p.rows &&
                  (!p.workers || (char*)a.headers - (char*)a.part + p.workers * 8 * 4 == p.workspace) && head_dim > 0;
  return ok ? hipSuccess : hipErrorInvalidValue;
}
}
extern "C" int test_plan(int64_t t, int64_t h, int64_t kv, int64_t d, int64_t r, int64_t mq, int64_t ms, int64_t* out) {
  const nvfp4::AttnPlan p = nvfp4::plan_attention(t, h, kv, d, r, mq < t ? mq : t, ms);
  const int64_t v[] = {(int64_t)p.kernel, p.rows, p.join_rows, p.workers, p.row_tiles, p.all_tiles, p.workspace};
  for (int i = 0; i < 7; ++i) out[i] = v[i];
  return 0;
}
'''


def _build(tmp_path, flags, name):
    base = ["-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fPIC", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
            f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", *flags]
    stubs = tmp_path / "stubs.cpp"
    stubs.write_text(STUBS)
    objs = []
    for src in (os.path.join(CSRC, "attention_api.hip"), os.path.join(CSRC, "attention_plan.hip"), str(stubs)):
        obj = tmp_path / (os.path.basename(src) + ".o")
        subprocess.run(["g++", "-x", "c++", *base, "-c", src, "-o", str(obj)], check=True, capture_output=True, text=True)
        objs.append(str(obj))
    lib = tmp_path / name
    subprocess.run(["g++", "-shared", *flags, "-o", str(lib), *objs], check=True, capture_output=True, text=True)
    return lib


def test_division_and_host_layer_under_sanitizers(tmp_path):
    rt = _asan_runtime()
    if rt is None:
        pytest.skip("g++ with libasan is not available")
    lib = _build(tmp_path, ["-fsanitize=address,undefined", "-fno-sanitize-recover=undefined"], "libplan_asan.so")
    prog = tmp_path / "run.py"
    prog.write_text(f'''
import ctypes, itertools, random, sys
sys.path.insert(0, {ROOT!r})
from bit_block_scaled_nvfp4_amd import attention as at
lib = ctypes.CDLL({str(lib)!r})
at.declare(lib)
P = 0x10000
rng = random.Random(1)
ends = lambda hi: [1, 2, 3, 16, 17, 96, 97, 256, 257, 1024, 1025, hi - 1, hi, rng.randrange(1, hi + 1)]
n = 0
for d in (64, 128, 256):
    for h, kv in ((1, 1), (7, 1), (24, 4), (32, 8), (1024, 1), (1024, 1024), (1000, 8)):
        most = (2 ** 31 - 1) // h
        for t, r, mq, ms in itertools.product(ends(most), (1, 2, 255, 256, 257, 8192), (1, 2, 5, 24, 25, 4096, 2 ** 31 - 1),
                                              (1, 256, 257, 1024, 1025, 2 ** 31 - 1)):
            if t > most:
                continue
            need = lib.nvfp4_kv_fp8_attention_workspace(t, h, kv, d, r, mq, ms)
            assert 0 <= need < 2 ** 29 and need % 16 == 0
            a = dict(q=P, dt=1, T=t, H=h, Hk=kv, D=d, qts=0, qhs=0, kc=P, vc=P, ks=P, vs=P, slots=64, cld=kv * d, table=P, R=r, W=4, tld=4, bs=16,
                     qs=P, lens=P, scale=0.1, cap=0.0, slopes=None, m0=None, m1=None, mq=mq, ms=ms, out=P, ots=h * d, ohs=d, ws=P, wsb=need, stream=None)
            got = lib.nvfp4_kv_fp8_attention(*a.values())
            assert got == (2 if (t - 1) * h * d + (h - 1) * d + d > 2 ** 40 else 0), (got, t, h, d)
            if need:
                assert lib.nvfp4_kv_fp8_attention(*{{**a, "wsb": need - 1}}.values()) in (2,)
            n += 1
print("passed", n)
''')
    env = dict(os.environ, LD_PRELOAD=rt, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    res = subprocess.run([sys.executable, str(prog)], capture_output=True, text=True, env=env, timeout=300)
    out = res.stdout + res.stderr
    assert res.returncode == 0 and "passed" in out, out[-4000:]
    assert "ERROR: AddressSanitizer" not in out and "runtime error" not in out


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    lib = ctypes.CDLL(str(_build(tmp_path_factory.mktemp("plan"), [], "libplan.so")))
    lib.test_plan.argtypes = [ctypes.c_int64] * 7 + [ctypes.POINTER(ctypes.c_int64)]

    def call(tokens, heads, kv_heads, head_dim, requests, max_query_len, max_seq_len):
        out = (ctypes.c_int64 * 7)()
        lib.test_plan(tokens, heads, kv_heads, head_dim, requests, max_query_len, max_seq_len, out)
        kernel, rows, join_rows, workers, row_tiles, all_tiles, workspace = out
        return dict(kernel=("stream16", "stream32", "tiled")[kernel], rows=rows, join_rows=join_rows, workers=workers,
                    row_tiles=row_tiles, all_tiles=all_tiles, workspace=workspace)

    return call


@pytest.mark.parametrize("new,split,kernel", [(1, False, "stream16"), (1, True, "stream16"), (9, False, "stream32"), (9, True, "stream32"),
                                              (40, False, "stream32"), (40, True, "tiled"), (130, False, "tiled"), (130, True, "tiled")])
@pytest.mark.parametrize("head_dim", [64, 128, 256])
def test_sizes_of_the_gpu_tests_reach_the_kernels_they_name(plan, new, split, kernel, head_dim):
    from .test_gpu_attention_scores import hints, problem

    p = problem(new, head_dim)
    h = hints(new, split)
    got = plan(p.tokens, p.heads, p.kv_heads, head_dim, p.requests, h["max_query_len"], h["max_seq_len"])
    assert got["kernel"] == kernel and (got["workers"] > 0) == split and got["all_tiles"] == 0, got


def test_other_divisions_of_the_gpu_tests(plan):
    """One prompt among single tokens: row tiles are searched; the masks' sizes: 16, 32 and 256 rows."""
    lens = [((i * 7) % 40, i % 3 % 2) for i in range(60)]
    lens[20] = (11, 300)
    got = plan(sum(n for _, n in lens) + 3, 4, 2, 64, 60, 300, 256)
    assert got["kernel"] == "tiled" and got["all_tiles"] > 0 and got["workers"] == 0
    assert [plan(60, 4, 2, 64, 1, n, 2000 if n == 60 else 60)["kernel"] for n in (1, 12, 60)] == ["stream16", "stream32", "tiled"]


def test_grids_hold_every_row_tile(plan):
    """The grid by requests has the row tiles that the longest may have, the searched one those of all tokens, up to the
    bound of a grid dimension (beyond it the kernels' strides go on)."""
    rng = random.Random(5)
    for _ in range(3000):
        heads, kv = rng.choice([(1, 1), (24, 4), (32, 8), (16, 1), (8, 8)])
        r = rng.randrange(1, 400)
        lens = [rng.choice([0, 1, 1, 2, rng.randrange(1, 3000)]) for _ in range(r)]
        longest, tokens = max(1, max(lens)), max(1, sum(lens))
        p = plan(tokens, heads, kv, rng.choice([64, 128, 256]), r, longest, rng.choice([longest, 300, 5000, 100000]))
        tiles = [-(-n * (heads // kv) // p["rows"]) for n in lens]
        if p["all_tiles"]:
            assert p["kernel"] == "tiled" and p["all_tiles"] >= min(4096, sum(tiles))
        assert p["row_tiles"] == min(4096, max(1, max(tiles)))
        assert (p["workspace"] > 0) == (p["workers"] > 0) and not (p["workers"] and p["all_tiles"])
