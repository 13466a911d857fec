"""The attention part of the C ABI (include/nvfp4_attention.h) and its binding on the CPU: exports,
refusals before any HIP call, workspace sizes, the binding's checks, and the host layer under the address
and undefined-behaviour sanitizers.

The calls pass fake device addresses and fail validation (or are empty problems): no GPU is needed."""

import ctypes
import os
import re
import subprocess
import sys

import pytest

import bit_block_scaled_nvfp4_amd as nv
from bit_block_scaled_nvfp4_amd import attention as at

from .test_asan_host import _asan_runtime
from .test_abi import _gpu_visible

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_block_scaled_nvfp4_amd", "csrc")
HEADER = os.path.join(ROOT, "include", "nvfp4_attention.h")

pytestmark = [
    pytest.mark.skipif(not os.path.exists(nv.LIB_PATH), reason="libnvfp4.so not built"),
    pytest.mark.skipif(_gpu_visible(), reason="host-only checks with fake device addresses"),
]

P = 0x10000
OK, EINVAL, ESHAPE, EALIGN = nv.NVFP4_OK, nv.NVFP4_EINVAL, nv.NVFP4_ESHAPE, nv.NVFP4_EALIGN


def _lib():
    lib = nv.load_library()
    at.declare(lib)
    return lib


def test_header_and_library_agree():
    src = open(HEADER).read()
    names = sorted(set(re.findall(r"^\S[^\n(]*?\b(nvfp4_\w+)\s*\(", src, re.M)))
    assert sorted(at.ATTENTION_SYMBOLS) == names
    out = subprocess.run(["nm", "-D", "--defined-only", nv.LIB_PATH], capture_output=True, text=True, check=True).stdout
    exported = {ln.split()[-1] for ln in out.splitlines() if " T " in ln}
    assert set(names) <= exported
    assert int(re.search(r"NVFP4_MAX_REQUESTS (\d+)", src).group(1)) == at.MAX_REQUESTS
    assert int(re.search(r"NVFP4_MAX_TREE_WORDS (\d+)", src).group(1)) == at.MAX_TREE_WORDS


def _tables(**kw):
    a = dict(ctx=P, new=P, R=4, bs=16, free=P, F=10, start=None, table=P, W=8, ld=8, slots=P, pos=P, T=100,
             qs=P, lens=P, need=P, stream=None)
    a.update(kw)
    return _lib().nvfp4_kv_block_tables(*a.values())


def test_block_tables_validation():
    for name in ("ctx", "new", "free", "table", "slots", "pos", "qs", "lens", "need"):
        assert _tables(**{name: None}) == EINVAL, name
    for kw in (dict(R=-1), dict(R=8193), dict(bs=0), dict(bs=(1 << 24) + 1), dict(F=-1), dict(F=1 << 31),
               dict(T=-1), dict(T=(1 << 31) - 256), dict(ld=7), dict(W=-1), dict(ld=1 << 40), dict(W=1 << 31, ld=1 << 31)):
        assert _tables(**kw) == ESHAPE, kw
    for name in ("ctx", "new", "free", "start", "table", "pos", "qs", "lens", "need"):
        assert _tables(**{name: P + 2}) == EALIGN, name
    assert _tables(slots=P + 4) == EALIGN


def _args(**kw):
    a = dict(q=P, dt=nv.NVFP4_BF16, T=8, H=8, Hk=2, D=128, qts=1024, qhs=128, kc=P, vc=P, ks=P, vs=P, slots=64,
             cld=256, table=P, R=2, W=4, tld=4, bs=16, qs=P, lens=P, scale=0.1, cap=0.0, slopes=None)
    tail = dict(mq=8, ms=64, out=P, ots=1024, ohs=128, ws=None, wsb=0, stream=None)
    for k, v in kw.items():
        if k in a:
            a[k] = v
        elif k in tail:
            tail[k] = v
    return a, tail


def _attn(**kw):
    a, tail = _args(**kw)
    mid = dict(doc=kw.get("doc"), prefix=kw.get("prefix"))
    return _lib().nvfp4_kv_fp8_attention(*a.values(), *mid.values(), *tail.values())


def _tree(**kw):
    a, tail = _args(**kw)
    mid = dict(mask=kw.get("mask", P), words=kw.get("words", 1), mld=kw.get("mld", 1), positions=kw.get("positions"))
    return _lib().nvfp4_kv_fp8_tree_attention(*a.values(), *mid.values(), *tail.values())


@pytest.mark.parametrize("call", [_attn, _tree])
def test_attention_validation(call):
    for name in ("q", "kc", "vc", "ks", "vs", "table", "qs", "lens", "out"):
        assert call(**{name: None}) == EINVAL, name
    nan, inf = float("nan"), float("inf")
    for kw in (dict(dt=nv.NVFP4_F32), dict(dt=7), dict(scale=nan), dict(scale=inf), dict(cap=-1.0), dict(cap=nan),
               dict(cap=inf)):
        assert call(**kw) == EINVAL, kw
    for kw in (dict(T=-1), dict(H=0), dict(H=1025, Hk=1025), dict(Hk=0), dict(Hk=3), dict(D=96), dict(D=0),
               dict(T=1 << 30), dict(R=-1), dict(R=8193), dict(mq=0), dict(ms=0), dict(ms=1 << 31), dict(tld=3),
               dict(bs=0), dict(slots=0), dict(slots=1 << 31), dict(cld=255), dict(cld=1 << 31),
               dict(qts=-8), dict(qhs=-8), dict(qts=1 << 41), dict(ots=8), dict(ohs=64), dict(ots=0), dict(ohs=0),
               dict(ots=1 << 40)):
        assert call(**kw) == ESHAPE, kw
    for kw in (dict(q=P + 8), dict(out=P + 8), dict(qts=1028), dict(qhs=132), dict(ots=1028), dict(ohs=132, ots=2048),
               dict(kc=P + 8), dict(vc=P + 8), dict(cld=264), dict(ks=P + 2), dict(vs=P + 2), dict(table=P + 2),
               dict(qs=P + 2), dict(lens=P + 2), dict(slopes=P + 2)):
        assert call(**kw) == EALIGN, kw
    # nothing to compute
    assert call(T=0, q=None, out=None) == OK
    assert call(R=0, lens=None, table=None) == OK
    # overlapping outputs are refused, head-major ones are not (they pass the check that follows: the
    # missing workspace of a long call)
    assert call(ots=128, ohs=1024, ms=10 ** 6) == EINVAL


def test_attention_own_arguments():
    assert _attn(doc=P + 2) == EALIGN
    assert _attn(prefix=P + 2) == EALIGN
    assert _tree(mask=None) == EINVAL
    assert _tree(mask=P + 4) == EALIGN
    assert _tree(positions=P + 2) == EALIGN
    for kw in (dict(words=0, mld=1), dict(words=65, mld=65), dict(words=2, mld=1), dict(mld=1 << 40)):
        assert _tree(**kw) == ESHAPE, kw


def test_workspace():
    ws = _lib().nvfp4_kv_fp8_attention_workspace
    need = ws(8, 8, 2, 128, 2, 8, 10 ** 6)
    assert need > 0 and need % 16 == 0
    assert _attn(ms=10 ** 6) == EINVAL  # none given
    assert _attn(ms=10 ** 6, ws=P, wsb=need - 1) == ESHAPE
    assert _attn(ms=10 ** 6, ws=P + 8, wsb=need) == EALIGN
    assert ws(8, 8, 2, 128, 2, 8, 64) == 0
    assert ws(8, 8, 3, 128, 2, 8, 10 ** 6) == 0  # invalid
    assert ws(0, 8, 2, 128, 2, 8, 10 ** 6) == 0
    # a bound above the tokens says nothing more
    assert ws(8, 8, 2, 128, 2, 10 ** 6, 10 ** 6) == need
    # every size that is allowed fits 64 bits, and what is needed stays bounded
    for D in (64, 128, 256):
        for H, Hk in ((1, 1), (1024, 1), (1024, 1024)):
            for mq in (1, 3, 40, 10 ** 6):
                got = ws(10 ** 6, H, Hk, D, 8192, mq, 2 ** 31 - 1)
                assert 0 <= got < 2 ** 29


def _t(shape, dtype, device="meta"):
    import torch

    return torch.empty(shape, dtype=dtype, device=device)


def test_binding_refuses_cpu_tensors_and_bad_shapes():
    import torch

    i32, u8, f32, bf = torch.int32, torch.uint8, torch.float32, torch.bfloat16
    with pytest.raises(ValueError, match="GPU"):
        nv.nvfp4_kv_block_tables(torch.zeros(2, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(4, dtype=i32),
                                 torch.zeros((2, 4), dtype=i32), 16, 8)
    with pytest.raises(ValueError, match="GPU"):
        nv.nvfp4_kv_fp8_attention(torch.zeros((2, 4, 64), dtype=bf), torch.zeros((16, 64), dtype=u8),
                                  torch.zeros((16, 64), dtype=u8), torch.ones(1), torch.ones(1),
                                  torch.zeros((1, 1), dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(1, dtype=i32),
                                  block_size=16, num_kv_heads=1)


class _Dev:
    """A tensor that claims to live on the GPU: shape, dtype and stride checks run, no memory is touched."""

    def __init__(self, t):
        self._t = t

    is_cuda = True

    def __getattr__(self, name):
        return getattr(self._t, name)


def _call(which, **kw):
    import torch

    i32, u8, f32, bf = torch.int32, torch.uint8, torch.float32, torch.bfloat16
    a = dict(q=_t((6, 4, 64), bf), key_cache=_t((32, 128), u8), value_cache=_t((32, 128), u8), key_scale=_t((1,), f32),
             value_scale=_t((1,), f32), block_table=_t((2, 3), i32), query_start=_t((3,), i32), seq_lens=_t((2,), i32),
             block_size=16, num_kv_heads=2)
    if which == "tree":
        a["tree_mask"] = _t((6, 1), torch.int64)
    a.update(kw)
    a["q"] = _Dev(a["q"])
    fn = nv.nvfp4_kv_fp8_tree_attention if which == "tree" else nv.nvfp4_kv_fp8_attention
    return fn(**a)


@pytest.mark.parametrize("which", ["prompt", "tree"])
def test_binding_checks_of_the_attentions(which):
    import torch

    i32, u8, f32, bf, f16 = torch.int32, torch.uint8, torch.float32, torch.bfloat16, torch.float16
    bad = [dict(q=_t((6, 4, 64), f32)), dict(q=_t((6, 256), bf)), dict(q=_t((6, 4, 96), bf)), dict(num_kv_heads=3),
           dict(num_kv_heads=0), dict(block_size=0), dict(key_cache=_t((32, 64), u8)), dict(key_cache=_t((32, 128), f16)),
           dict(value_cache=_t((31, 128), u8)), dict(value_cache=_t((32, 160), u8)[:, :128]),
           dict(key_scale=_t((2,), f32)), dict(value_scale=_t((1,), bf)), dict(block_table=_t((3, 3), i32)),
           dict(block_table=_t((2, 3), torch.int64)), dict(block_table=_t((3, 2), i32).t()),
           dict(query_start=_t((2,), i32)), dict(seq_lens=_t((2,), torch.int64)), dict(slopes=_t((3,), f32)),
           dict(out=_t((6, 4, 64), f16)), dict(out=_t((6, 4, 32), bf)), dict(q=_t((6, 64, 4), bf).transpose(1, 2)),
           dict(seq_lens=torch.empty(2, dtype=i32)), dict(query_start=_t((6,), i32)[::2])]
    if which == "tree":
        bad += [dict(tree_mask=_t((6, 1), i32)), dict(tree_mask=_t((5, 1), torch.int64)),
                dict(tree_mask=_t((6, 65), torch.int64)), dict(tree_mask=_t((6, 0), torch.int64)),
                dict(tree_mask=_t((2, 6), torch.int64).t()), dict(positions=_t((5,), i32))]
    else:
        bad += [dict(doc_start=_t((5,), i32)), dict(doc_start=_t((6,), torch.int64)), dict(prefix_lens=_t((3,), i32))]
    for kw in bad:
        with pytest.raises(ValueError):
            _call(which, **kw)


def test_host_layer_under_address_and_ub_sanitizers(tmp_path):
    rt = _asan_runtime()
    if rt is None:
        pytest.skip("g++ with libasan is not available")
    lib = tmp_path / "libnvfp4_attention_asan.so"
    flags = ["-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fPIC", "-fsanitize=address,undefined",
             "-fno-sanitize-recover=undefined", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
             f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}"]
    stubs = tmp_path / "stubs.cpp"
    stubs.write_text('''
#include "attention_internal.h"
namespace nvfp4 {
AttnPlan plan_attention(int64_t, int64_t, int64_t, int64_t head_dim, int64_t, int64_t, int64_t max_seq_len) {
  AttnPlan p{};
  p.rows = 16;
  p.workers = max_seq_len > 1024 ? 256 : 0;
  p.workspace = p.workers ? (int64_t)p.workers * (2 * 16 * (head_dim + 2) + 8) * 4 : 0;
  return p;
}
hipError_t launch_block_tables(const TablesArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_attention(const AttnArgs&, const AttnPlan&, int, bool, hipStream_t) { return hipSuccess; }
}
''')
    objs = []
    for src in (os.path.join(CSRC, "attention_api.hip"), str(stubs)):
        obj = tmp_path / (os.path.basename(src) + ".o")
        subprocess.run(["g++", "-x", "c++", *flags, "-c", src, "-o", str(obj)], check=True, capture_output=True, text=True)
        objs.append(str(obj))
    subprocess.run(["g++", "-shared", "-fsanitize=address,undefined", "-o", str(lib), *objs], check=True,
                   capture_output=True, text=True)
    prog = tmp_path / "run.py"
    prog.write_text(f'''
import ctypes, sys
sys.path.insert(0, {ROOT!r})
from bit_block_scaled_nvfp4_amd import attention as at
lib = ctypes.CDLL({str(lib)!r})
at.declare(lib)
P, big = 0x10000, [0, 1, -1, 7, 2**31 - 1, 2**31, 2**40, 2**62, -2**62, 2**63 - 1, -2**63]
def attn(**kw):
    a = dict(q=P, dt=1, T=8, H=8, Hk=2, D=128, qts=1024, qhs=128, kc=P, vc=P, ks=P, vs=P, slots=64, cld=256, table=P,
             R=2, W=4, tld=4, bs=16, qs=P, lens=P, scale=0.1, cap=0.0, slopes=None, m0=None, m1=None, mq=8, ms=64,
             out=P, ots=1024, ohs=128, ws=P, wsb=1 << 30, stream=None)
    a.update(kw)
    return lib.nvfp4_kv_fp8_attention(*a.values())
def tree(**kw):
    a = dict(q=P, dt=1, T=8, H=8, Hk=2, D=128, qts=1024, qhs=128, kc=P, vc=P, ks=P, vs=P, slots=64, cld=256, table=P,
             R=2, W=4, tld=4, bs=16, qs=P, lens=P, scale=0.1, cap=0.0, slopes=None, mask=P, words=1, mld=1, pos=None,
             mq=8, ms=64, out=P, ots=1024, ohs=128, ws=P, wsb=1 << 30, stream=None)
    a.update(kw)
    return lib.nvfp4_kv_fp8_tree_attention(*a.values())
def tables(**kw):
    a = dict(ctx=P, new=P, R=4, bs=16, free=P, F=10, start=None, table=P, W=8, ld=8, slots=P, pos=P, T=100, qs=P,
             lens=P, need=P, stream=None)
    a.update(kw)
    return lib.nvfp4_kv_block_tables(*a.values())
assert attn() == 0 and tree() == 0 and tables() == 0 and attn(ms=5000) == 0
n = 0
for v in big:
    for name in ("T", "H", "Hk", "D", "qts", "qhs", "slots", "cld", "R", "W", "tld", "bs", "mq", "ms", "ots", "ohs", "wsb"):
        assert 0 <= attn(**{{name: v}}) <= 3 and 0 <= tree(**{{name: v}}) <= 3
        for w in big:
            for other in ("T", "R", "qts", "ots", "tld"):
                if other != name:
                    n += attn(**{{name: v, other: w}})
    for name in ("words", "mld"):
        assert 0 <= tree(**{{name: v}}) <= 3
    for name in ("R", "bs", "F", "W", "ld", "T"):
        assert 0 <= tables(**{{name: v}}) <= 3
    lib.nvfp4_kv_fp8_attention_workspace(v, 8, 2, 128, 2, 8, 64)
    lib.nvfp4_kv_fp8_attention_workspace(8, v, v, 128, v, v, v)
print("passed", n)
''')
    env = dict(os.environ, LD_PRELOAD=rt, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    res = subprocess.run([sys.executable, str(prog)], capture_output=True, text=True, env=env, timeout=300)
    out = res.stdout + res.stderr
    assert res.returncode == 0 and "passed" in out, out[-4000:]
    assert "ERROR: AddressSanitizer" not in out and "runtime error" not in out
