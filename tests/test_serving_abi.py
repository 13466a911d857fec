"""The serving part of the C ABI (include/nvfp4_serving.h) and its binding on the CPU: exports, refusals before any HIP
call, workspace sizes, the binding's checks, and the host layer under the address and undefined-behaviour sanitizers.

The calls pass fake device addresses and fail validation (or are empty problems): no GPU is needed."""

import ctypes
import os
import re
import subprocess
import sys

import pytest

import bit_block_scaled_nvfp4_amd as nv
from bit_block_scaled_nvfp4_amd import serving as sv

from .test_abi import _gpu_visible
from .test_asan_host import _asan_runtime
from .test_attention_abi import _Dev, _t

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_block_scaled_nvfp4_amd", "csrc")
HEADER = os.path.join(ROOT, "include", "nvfp4_serving.h")

pytestmark = [
    pytest.mark.skipif(not os.path.exists(nv.LIB_PATH), reason="libnvfp4.so not built"),
    pytest.mark.skipif(_gpu_visible(), reason="host-only checks with fake device addresses"),
]

P = 0x10000
OK, EINVAL, ESHAPE, EALIGN = nv.NVFP4_OK, nv.NVFP4_EINVAL, nv.NVFP4_ESHAPE, nv.NVFP4_EALIGN
NAN, INF = float("nan"), float("inf")


def _lib():
    lib = nv.load_library()
    sv.declare(lib)
    return lib


def test_header_and_library_agree():
    src = open(HEADER).read()
    names = sorted(set(re.findall(r"^\S[^\n(]*?\b(nvfp4_\w+)\s*\(", src, re.M)))
    assert sorted(sv.SERVING_SYMBOLS) == names
    out = subprocess.run(["nm", "-D", "--defined-only", nv.LIB_PATH], capture_output=True, text=True, check=True).stdout
    exported = {ln.split()[-1] for ln in out.splitlines() if " T " in ln}
    assert set(names) <= exported
    assert int(re.search(r"NVFP4_MAX_HEAD_DIM (\d+)", src).group(1)) == sv.MAX_HEAD_DIM
    for n in names:
        if not n.endswith("_workspace"):
            assert callable(getattr(nv, n)), n


def _rope(**kw):
    a = dict(q=P, H=4, qts=512, qhs=128, k=P, Hk=2, kts=256, khs=128, dt=nv.NVFP4_BF16, T=8, D=128, pos=P, freq=P, n=32,
             pairs=0, qw=P, kw=P, wt=nv.NVFP4_F32, eps=1e-6, off=0.0, qo=P, qots=512, qohs=128, ko=P, kots=256, kohs=128,
             stream=None)
    a.update(kw)
    return _lib().nvfp4_qk_norm_rope(*a.values())


def test_rope_validation():
    for name in ("q", "k", "pos", "freq", "qo", "ko"):
        assert _rope(**{name: None}) == EINVAL, name
    for kw in (dict(dt=3), dict(pairs=2), dict(pairs=-1), dict(wt=9), dict(eps=-1.0), dict(eps=NAN), dict(eps=INF),
               dict(off=NAN), dict(off=INF)):
        assert _rope(**kw) == EINVAL, kw
    for kw in (dict(T=-1), dict(T=1 << 31), dict(H=0), dict(H=1025), dict(Hk=-1), dict(Hk=1025), dict(D=0), dict(D=24),
               dict(D=528), dict(n=-8), dict(n=12), dict(n=72), dict(qts=-512), dict(khs=-128), dict(qts=1 << 41), dict(qts=1 << 31), dict(kohs=1 << 31),
               dict(qots=256), dict(qohs=64), dict(kots=0), dict(kohs=0)):
        assert _rope(**kw) == ESHAPE, kw
    for kw in (dict(q=P + 8), dict(k=P + 8), dict(qo=P + 8), dict(ko=P + 8), dict(qts=516), dict(khs=132, kts=512),
               dict(qots=516), dict(pos=P + 2), dict(freq=P + 2), dict(qw=P + 2), dict(kw=P + 2)):
        assert _rope(**kw) == EALIGN, kw
    # an F32 vector may begin every four elements; a weight is aligned to its own type
    assert _rope(dt=nv.NVFP4_F32, qts=516, q=P + 8) == EALIGN
    assert _rope(wt=nv.NVFP4_BF16, qw=P + 2, kw=P + 2, q=None) == EINVAL
    assert _rope(T=0, q=None, k=None, qo=None, ko=None, pos=None, freq=None) == OK


def _append(which, **kw):
    a = dict(k=P, v=P, dt=nv.NVFP4_BF16, T=8, Hk=2, D=128, kts=256, khs=128, vts=256, vhs=128, pos=P, freq=P, n=32,
             pairs=0, kw=P, wt=nv.NVFP4_F32, eps=1e-6, off=0.0, ks=P, vs=P, slots=P)
    tail = dict(kc=P, vc=P, S=64, ld=256, stream=None) if which == "fp8" else dict(kc=P, kcs=P, vc=P, vcs=P, B=4, bs=16, stream=None)
    for key, x in kw.items():
        (a if key in a else tail)[key] = x
    return getattr(_lib(), f"nvfp4_kv_{which}_append")(*a.values(), *tail.values())


@pytest.mark.parametrize("which", ["fp8", "fp4"])
def test_append_validation(which):
    for name in ("k", "v", "pos", "freq", "ks", "vs", "kc", "vc") + (("kcs", "vcs") if which == "fp4" else ()):
        assert _append(which, **{name: None}) == EINVAL, name
    for kw in (dict(dt=3), dict(pairs=2), dict(wt=9), dict(eps=-1.0), dict(eps=NAN), dict(off=INF)):
        assert _append(which, **kw) == EINVAL, kw
    for kw in (dict(T=-1), dict(T=1 << 31), dict(Hk=0), dict(Hk=1025), dict(D=96), dict(D=512), dict(n=12), dict(n=72),
               dict(kts=-256), dict(vhs=-128), dict(vts=1 << 41)):
        assert _append(which, **kw) == ESHAPE, kw
    for kw in (dict(k=P + 8), dict(v=P + 8), dict(kts=260), dict(vhs=132), dict(pos=P + 2), dict(freq=P + 2), dict(kw=P + 2),
               dict(ks=P + 2), dict(vs=P + 2), dict(slots=P + 4), dict(kc=P + 8), dict(vc=P + 8)):
        assert _append(which, **kw) == EALIGN, kw
    if which == "fp8":
        for kw in (dict(S=-1), dict(S=1 << 41), dict(ld=240), dict(ld=1 << 41), dict(S=1 << 30, ld=1 << 20)):
            assert _append(which, **kw) == ESHAPE, kw
        assert _append(which, ld=264) == EALIGN
        assert _append(which, S=0, kc=None, vc=None) == OK
    else:
        for kw in (dict(B=-1), dict(B=1 << 31), dict(bs=0), dict(bs=(1 << 24) + 1), dict(B=1 << 26), dict(B=1 << 10, bs=1 << 20),
                   dict(n=40), dict(n=8)):
            assert _append(which, **kw) == ESHAPE, kw
        assert _append(which, n=40, pairs=1, k=None) == EINVAL  # neighbouring pairs: a multiple of 8 will do
        assert _append(which, kcs=P + 8) == EALIGN and _append(which, vcs=P + 8) == EALIGN
        assert _append(which, B=0, kc=None, vc=None, kcs=None, vcs=None) == OK
    assert _append(which, T=0, k=None, v=None, pos=None, freq=None, slots=None) == OK


def _load(**kw):
    a = dict(c=P, s=P, B=4, Hk=2, bs=16, D=128, g=P, slots=P, T=8, out=P, dt=nv.NVFP4_F32, stream=None)
    a.update(kw)
    return _lib().nvfp4_kv_fp4_load(*a.values())


def test_load_validation():
    for name in ("c", "s", "g", "out"):
        assert _load(**{name: None}) == EINVAL, name
    assert _load(dt=nv.NVFP4_F16) == EINVAL
    for kw in (dict(B=-1), dict(B=1 << 27), dict(Hk=0), dict(Hk=1025), dict(bs=0), dict(D=96), dict(T=-1), dict(T=1 << 31),
               dict(Hk=1024, D=256, T=(1 << 31) - 1, B=1)):
        assert _load(**kw) == ESHAPE, kw
    for kw in (dict(c=P + 8), dict(s=P + 8), dict(out=P + 8), dict(g=P + 2), dict(slots=P + 4)):
        assert _load(**kw) == EALIGN, kw
    assert _load(T=0, out=None, c=None) == OK


def _args(**kw):
    a = dict(q=P, dt=nv.NVFP4_BF16, T=8, H=8, Hk=2, D=128, qts=1024, qhs=128, kc=P, kcs=P, vc=P, vcs=P, ks=P, vs=P, B=4,
             bs=16, table=P, R=2, W=4, tld=4, qs=P, lens=P, scale=0.1, cap=0.0, slopes=None)
    tail = dict(mq=8, ms=64, out=P, ots=1024, ohs=128, ws=None, wsb=0, stream=None)
    for k, v in kw.items():
        if k in a:
            a[k] = v
        elif k in tail:
            tail[k] = v
    return a, tail


def _attn(**kw):
    a, tail = _args(**kw)
    return _lib().nvfp4_kv_fp4_attention(*a.values(), kw.get("doc"), kw.get("prefix"), *tail.values())


def _tree(**kw):
    a, tail = _args(**kw)
    mid = dict(mask=kw.get("mask", P), words=kw.get("words", 1), mld=kw.get("mld", 1), positions=kw.get("positions"))
    return _lib().nvfp4_kv_fp4_tree_attention(*a.values(), *mid.values(), *tail.values())


@pytest.mark.parametrize("call", [_attn, _tree])
def test_attention_validation(call):
    for name in ("q", "kc", "kcs", "vc", "vcs", "ks", "vs", "table", "qs", "lens", "out"):
        assert call(**{name: None}) == EINVAL, name
    for kw in (dict(dt=nv.NVFP4_F32), dict(dt=7), dict(scale=NAN), dict(scale=INF), dict(cap=-1.0), dict(cap=NAN), dict(cap=INF)):
        assert call(**kw) == EINVAL, kw
    for kw in (dict(T=-1), dict(H=0), dict(H=1025, Hk=1025), dict(Hk=0), dict(Hk=3), dict(D=96), dict(T=1 << 30), dict(R=-1),
               dict(R=8193), dict(mq=0), dict(ms=0), dict(ms=1 << 31), dict(tld=3), dict(bs=0), dict(bs=1 << 25), dict(B=0),
               dict(B=-1), dict(B=1 << 31), dict(B=1 << 26), dict(qts=-8), dict(qts=1 << 41), dict(ots=8), dict(ohs=64),
               dict(ots=0), dict(ots=1 << 40)):
        assert call(**kw) == ESHAPE, kw
    for kw in (dict(q=P + 8), dict(out=P + 8), dict(qts=1028), dict(ots=1028), dict(kc=P + 8), dict(kcs=P + 8), dict(vc=P + 8),
               dict(vcs=P + 8), dict(ks=P + 2), dict(vs=P + 2), dict(table=P + 2), dict(qs=P + 2), dict(lens=P + 2),
               dict(slopes=P + 2)):
        assert call(**kw) == EALIGN, kw
    assert call(T=0, q=None, out=None) == OK
    assert call(R=0, lens=None, table=None) == OK
    assert call(ots=128, ohs=1024, ms=10 ** 6) == EINVAL  # the missing workspace of a long call


def test_attention_own_arguments_and_workspace():
    assert _attn(doc=P + 2) == EALIGN and _attn(prefix=P + 2) == EALIGN
    assert _tree(mask=None) == EINVAL and _tree(mask=P + 4) == EALIGN and _tree(positions=P + 2) == EALIGN
    for kw in (dict(words=0, mld=1), dict(words=65, mld=65), dict(words=2, mld=1), dict(mld=1 << 40)):
        assert _tree(**kw) == ESHAPE, kw
    ws = _lib().nvfp4_kv_fp4_attention_workspace
    need = ws(8, 8, 2, 128, 2, 8, 10 ** 6)
    assert need > 0 and need % 16 == 0
    assert _attn(ms=10 ** 6, ws=P, wsb=need - 1) == ESHAPE
    assert _attn(ms=10 ** 6, ws=P + 8, wsb=need) == EALIGN
    assert ws(8, 8, 2, 128, 2, 8, 64) == 0 and ws(8, 8, 3, 128, 2, 8, 10 ** 6) == 0 and ws(0, 8, 2, 128, 2, 8, 10 ** 6) == 0
    for D in (64, 128, 256):
        for H, Hk in ((1, 1), (1024, 1), (1024, 1024)):
            for mq in (1, 3, 40, 10 ** 6):
                assert 0 <= ws(10 ** 6, H, Hk, D, 8192, mq, 2 ** 31 - 1) < 2 ** 29


def _verify(**kw):
    a = dict(p=P, pld=100, q=P, qld=100, rows=8, V=100, tok=P, qs=P, R=2, au=P, su=P, acc=P, out=P, ws=P, wsb=1 << 20,
             stream=None)
    a.update(kw)
    return _lib().nvfp4_verify_drafted(*a.values())


def test_verify_validation():
    for name in ("p", "tok", "qs", "au", "su", "acc", "out", "ws"):
        assert _verify(**{name: None}) == EINVAL, name
    for kw in (dict(rows=-1), dict(rows=1 << 31), dict(V=0), dict(V=1 << 31, pld=1 << 31, qld=1 << 31), dict(R=-1), dict(R=8193),
               dict(pld=99), dict(qld=99), dict(pld=1 << 40), dict(qld=1 << 40), dict(wsb=31)):
        assert _verify(**kw) == ESHAPE, kw
    for name in ("p", "q", "tok", "qs", "au", "su", "acc", "out"):
        assert _verify(**{name: P + 2}) == EALIGN, name
    assert _verify(ws=P + 8) == EALIGN
    assert _verify(R=0, p=None, qs=None, ws=None) == OK
    ws = _lib().nvfp4_verify_drafted_workspace
    assert ws(2, 100) == 32 and ws(3, 4097) == 96 and ws(0, 100) == 0 and ws(8193, 100) == 0 and ws(1, 0) == 0
    assert 0 < ws(8192, 2 ** 31 - 5000) < 2 ** 37


def test_rows_whose_numbers_leave_32_bits_are_refused():
    """A workgroup steps over a request's rows by 64 and 256: past a last row close to 2^31 the step would overflow."""
    for rows in (2 ** 31 - 1, 2 ** 31 - 256, 2 ** 31 - 4096):
        assert _verify(rows=rows, V=1, pld=1, qld=1) == ESHAPE, rows
    assert _verify(rows=2 ** 31 - 4097, V=1, pld=1, qld=1, ws=None) == EINVAL


# ---- the binding ------------------------------------------------------------------------------


def test_binding_refuses_cpu_tensors():
    import torch

    x = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    one, i32 = torch.ones(1), torch.zeros(2, dtype=torch.int32)
    cache = (u8(1, 4, 16, 32), u8(1, 4, 16, 4))
    for call in (lambda: nv.nvfp4_qk_norm_rope(x), lambda: nv.nvfp4_kv_fp8_append(x, x, None, None, one, one, u8(16, 256), u8(16, 256)),
                 lambda: nv.nvfp4_kv_fp4_append(x, x, None, None, one, one, *cache, *cache), lambda: nv.nvfp4_kv_fp4_load(*cache, one),
                 lambda: nv.nvfp4_kv_fp4_attention(x, *cache, *cache, one, one, i32[None], i32, i32[:1]),
                 lambda: nv.nvfp4_verify_drafted(torch.zeros(2, 9), None, i32, i32, one, one[:1])):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_binding_checks_of_the_head_vectors():
    import torch

    bf, f16, f32, i32 = torch.bfloat16, torch.float16, torch.float32, torch.int32
    good = dict(q=_t((6, 4, 128), bf), k=_t((6, 2, 128), bf), positions=_t((6,), i32), inv_freq=_t((32,), f32))
    bad = [dict(q=_t((6, 4, 128), torch.float64)), dict(q=_t((6, 512), bf)), dict(q=_t((6, 4, 24), bf), k=None, inv_freq=None, positions=None),
           dict(q=_t((6, 4, 528), bf), k=None), dict(q=_t((6, 1025, 16), bf), k=None, positions=None, inv_freq=None),
           dict(q=_t((6, 128, 4), bf).transpose(1, 2)), dict(k=_t((5, 2, 128), bf)), dict(k=_t((6, 2, 64), bf)), dict(k=_t((6, 2, 128), f16)),
           dict(positions=None), dict(inv_freq=None), dict(positions=_t((5,), i32)), dict(positions=_t((6,), torch.int64)),
           dict(inv_freq=_t((32,), bf)), dict(inv_freq=_t((12,), f32)), dict(inv_freq=_t((72,), f32)), dict(inv_freq=_t((4, 8), f32)),
           dict(inv_freq=_t((64,), f32)[::2]), dict(q_weight=_t((64,), f32)), dict(q_weight=_t((128,), torch.float64)),
           dict(q_weight=_t((128,), f32), k_weight=_t((128,), bf)), dict(interleaved=2), dict(k=None, k_weight=_t((128,), bf)),
           dict(k=None, k_out=_t((6, 2, 128), bf)), dict(q_out=_t((6, 4, 64), bf)), dict(q_out=_t((6, 4, 128), f16)),
           dict(k_out=_t((6, 4, 128), bf)), dict(q_out=_t((6, 128, 4), bf).transpose(1, 2))]
    for kw in bad:
        a = {**good, **kw}
        a["q"] = _Dev(a["q"])
        with pytest.raises(ValueError):
            nv.nvfp4_qk_norm_rope(**a)


def test_outputs_that_meet_other_memory_are_refused():
    import torch

    def base(T=6, H=4, Hk=2, D=64):
        store = torch.zeros(T, H + 2 * Hk, D, dtype=torch.bfloat16)
        return store, store[:, :H], store[:, H:H + Hk]

    def call(q, k, **kw):
        T, D = q.shape[0], q.shape[2]
        qs, ks = tuple(q.stride()[:2]), tuple(k.stride()[:2])
        qo, ko = kw.get("q_out"), kw.get("k_out")
        sv._refuse_meeting(q, qs, k, ks, qo, qo.stride()[:2] if qo is not None else None, ko, ko.stride()[:2] if ko is not None else None)

    store, q, k = base()
    fresh = torch.zeros(6, 4, 64, dtype=torch.bfloat16)
    call(q, k, q_out=q, k_out=k)  # in place
    call(q, k, q_out=fresh)
    call(q, k, k_out=store[:, 6:8])  # the values' columns of the fused row
    for kw in (dict(k_out=store[:, 3:5]), dict(q_out=store[:, 1:5]), dict(q_out=store[:, 2:6]), dict(q_out=fresh, k_out=fresh[:, 2:]),
               dict(k_out=q[:, :2]), dict(q_out=store.flatten()[64:64 + 5 * 512 + 256].as_strided((6, 4, 64), (512, 64, 1), 64))):
        with pytest.raises(ValueError, match="share no memory"):
            call(q, k, **kw)
    # head-major storage, side by side in one buffer
    major = torch.zeros(10, 6, 64, dtype=torch.bfloat16)
    qm, km = major[:4].transpose(0, 1), major[4:6].transpose(0, 1)
    call(qm, km, q_out=major[6:].transpose(0, 1), k_out=km)
    with pytest.raises(ValueError, match="share no memory"):
        call(qm, km, q_out=major[5:9].transpose(0, 1))
    # rows interleaved token by token
    two = torch.zeros(12, 4, 64, dtype=torch.bfloat16)
    call(two[::2], torch.zeros(6, 2, 64, dtype=torch.bfloat16), q_out=two[1::2])


def _cache(B=2, Hk=2, bs=16, D=128):
    import torch

    return _t((B, Hk, bs, D // 2), torch.uint8), _t((B, Hk, bs, D // 16), torch.uint8)


def test_binding_checks_of_the_appends():
    import torch

    bf, f32, i32, i64, u8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8
    kc, kcs = _cache()
    common = dict(key=_t((6, 2, 128), bf), value=_t((6, 2, 128), bf), positions=_t((6,), i32), inv_freq=_t((32,), f32),
                  slot_mapping=_t((6,), i64))
    fp8 = dict(common, key_scale=_t((1,), f32), value_scale=_t((1,), f32), key_cache=_t((32, 256), u8), value_cache=_t((32, 256), u8))
    fp4 = dict(common, key_gscale=_t((1,), f32), value_gscale=_t((1,), f32), key_codes=kc, key_scales=kcs, value_codes=kc, value_scales=kcs)
    both = [dict(key=_t((6, 2, 96), bf)), dict(key=_t((6, 256), bf)), dict(value=_t((6, 1, 128), bf)), dict(value=_t((6, 2, 128), f32)),
            dict(value=_t((6, 256), bf)), dict(positions=None), dict(inv_freq=_t((12,), f32)), dict(slot_mapping=_t((6,), i32)),
            dict(slot_mapping=_t((5,), i64)), dict(k_weight=_t((64,), f32)), dict(interleaved="yes"), dict(key=_t((6, 1025, 64), bf))]
    own8 = [dict(key_cache=_t((32, 128), u8)), dict(key_cache=_t((32, 256), bf)), dict(value_cache=_t((31, 256), u8)),
            dict(value_cache=_t((32, 272), u8)[:, :256]), dict(key_scale=_t((2,), f32)), dict(value_scale=_t((1,), bf))]
    own4 = [dict(key_codes=_t((2, 2, 16, 32), u8)), dict(key_scales=_t((2, 2, 16, 4), u8)), dict(key_codes=_t((2, 2, 16, 64), bf)),
            dict(key_codes=_t((2, 16, 2, 64), u8).transpose(1, 2)), dict(value_codes=_t((3, 2, 16, 64), u8), value_scales=_t((3, 2, 16, 8), u8)),
            dict(key_codes=_t((2, 4, 16, 64), u8), key_scales=_t((2, 4, 16, 8), u8), value_codes=_t((2, 4, 16, 64), u8),
                 value_scales=_t((2, 4, 16, 8), u8)), dict(inv_freq=_t((40,), f32)), dict(key_gscale=_t((2,), f32)),
            dict(key_codes=_t((32, 128), u8))]
    for fn, good, bad in ((nv.nvfp4_kv_fp8_append, fp8, both + own8), (nv.nvfp4_kv_fp4_append, fp4, both + own4)):
        for kw in bad:
            a = {**good, **kw}
            a["key"] = _Dev(a["key"])
            with pytest.raises(ValueError):
                fn(**a)


def test_caches_whose_rows_share_memory_are_refused():
    import torch

    bf, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
    row = _t((1, 256), u8)
    for kc, vc in ((row.expand(32, 256), row.expand(32, 256)), (_t((1, 256), u8).expand(32, 256), row.expand(32, 256)),
                   (_t((8192,), u8).as_strided((32, 256), (128, 1)), _t((8192,), u8).as_strided((32, 256), (128, 1)))):
        with pytest.raises(ValueError, match="rows of their own"):
            nv.nvfp4_kv_fp8_append(_Dev(_t((6, 2, 128), bf)), _t((6, 2, 128), bf), None, None, _t((1,), f32), _t((1,), f32), kc, vc)


def test_ranges_that_meet_are_refused():
    sv._refuse_ranges([("a", 0, 16), ("b", 16, 32)], [("x", 32, 64), ("y", 40, 50), ("z", 7, 7)])
    for outs, ins in (([("a", 0, 16), ("b", 15, 32)], []), ([("a", 10, 20)], [("x", 0, 11)]), ([("a", 10, 20)], [("x", 0, 100)])):
        with pytest.raises(ValueError, match="must not share memory"):
            sv._refuse_ranges(outs, ins)


@pytest.mark.parametrize("which", ["prompt", "tree"])
def test_binding_checks_of_the_attentions(which):
    import torch

    i32, u8, f32, bf, f16 = torch.int32, torch.uint8, torch.float32, torch.bfloat16, torch.float16
    kc, kcs = _cache(D=64)
    good = dict(q=_t((6, 4, 64), bf), key_codes=kc, key_scales=kcs, value_codes=kc, value_scales=kcs, key_gscale=_t((1,), f32),
                value_gscale=_t((1,), f32), block_table=_t((2, 3), i32), query_start=_t((3,), i32), seq_lens=_t((2,), i32))
    wide = _cache(D=128)
    bad = [dict(q=_t((6, 4, 64), f32)), dict(q=_t((6, 256), bf)), dict(q=_t((6, 4, 128), bf)), dict(q=_t((6, 3, 64), bf)),
           dict(key_codes=_t((2, 2, 16, 32), f16)), dict(key_scales=_t((2, 2, 16, 2), u8)), dict(value_codes=wide[0], value_scales=wide[1]),
           dict(key_codes=_t((2, 2, 16, 48), u8), key_scales=_t((2, 2, 16, 6), u8)), dict(key_gscale=_t((2,), f32)), dict(value_gscale=_t((1,), bf)),
           dict(block_table=_t((3, 3), i32)), dict(block_table=_t((2, 3), torch.int64)), dict(query_start=_t((2,), i32)),
           dict(seq_lens=_t((2,), torch.int64)), dict(slopes=_t((3,), f32)), dict(out=_t((6, 4, 64), f16)), dict(out=_t((6, 4, 32), bf)),
           dict(key_codes=_t((2, 16, 2, 32), u8).transpose(1, 2))]
    fn = nv.nvfp4_kv_fp4_attention
    if which == "tree":
        fn, good["tree_mask"] = nv.nvfp4_kv_fp4_tree_attention, _t((6, 1), torch.int64)
        bad += [dict(tree_mask=_t((6, 1), i32)), dict(tree_mask=_t((5, 1), torch.int64)), dict(tree_mask=_t((6, 65), torch.int64)),
                dict(positions=_t((5,), i32))]
    else:
        bad += [dict(doc_start=_t((5,), i32)), dict(prefix_lens=_t((3,), i32))]
    for kw in bad:
        a = {**good, **kw}
        a["q"] = _Dev(a["q"])
        with pytest.raises(ValueError):
            fn(**a)


def test_binding_checks_of_the_verification():
    import torch

    i32, f32 = torch.int32, torch.float32
    good = dict(target_probs=_t((6, 50), f32), draft_probs=_t((6, 50), f32), tokens=_t((6,), i32), query_start=_t((3,), i32),
                accept_u=_t((6,), f32), sample_u=_t((2,), f32))
    bad = [dict(target_probs=_t((6, 50), torch.bfloat16)), dict(target_probs=_t((300,), f32)), dict(target_probs=_t((50, 6), f32).t()),
           dict(target_probs=_t((1, 50), f32).expand(6, 50)), dict(target_probs=_t((6, 0), f32)), dict(draft_probs=_t((5, 50), f32)),
           dict(draft_probs=_t((6, 49), f32)), dict(tokens=_t((6,), torch.int64)), dict(tokens=_t((5,), i32)), dict(query_start=_t((2,), i32)),
           dict(accept_u=_t((2,), f32)), dict(accept_u=_t((6,), torch.float64)), dict(sample_u=_t((6,), f32)), dict(sample_u=_t((2, 1), f32)),
           dict(accepted=_t((3,), i32)), dict(out=_t((6,), torch.int64)), dict(out=_t((5,), i32))]
    for kw in bad:
        a = {**good, **kw}
        a["target_probs"] = _Dev(a["target_probs"])
        with pytest.raises(ValueError):
            nv.nvfp4_verify_drafted(**a)


# ---- the host layer under sanitizers ----------------------------------------------------------

STUBS = '''
#include "serving_internal.h"
namespace nvfp4 {
// what the kernels take for granted
hipError_t launch_heads(HeadArgs a, nvfp4_dtype, HeadSink sink, hipStream_t) {
  const bool ok = a.tokens >= 1 && a.head_dim % 16 == 0 && a.num_freq % 8 == 0 && 2 * a.num_freq <= a.head_dim && a.group[0].heads.d >= 1 &&
                  a.group[0].heads.d + a.group[1].heads.d <= 2048 && (a.num_freq == 0 || (a.positions && a.inv_freq)) &&
                  (sink == HeadSink::Same ? a.group[0].out != nullptr : a.group[0].cache && a.group[1].cache && a.num_slots > 0) &&
                  (sink != HeadSink::Fp4 || (a.num_slots * a.group[0].heads.d < (1ll << 31) && (a.interleaved || a.num_freq % 16 == 0)));
  return ok ? hipSuccess : hipErrorInvalidValue;
}
hipError_t launch_fp4_load(Fp4LoadArgs a, bool, hipStream_t) {
  return a.tokens > 0 && a.head_bits >= 6 && a.head_bits <= 8 && a.num_slots * a.kv_heads < (1ll << 31) ? hipSuccess : hipErrorInvalidValue;
}
hipError_t launch_verify(const VerifyArgs& a, hipStream_t) {
  return a.requests > 0 && a.requests <= 8192 && (int64_t)a.chunks * kVerifyChunk < (1ll << 31) && a.sums ? hipSuccess : hipErrorInvalidValue;
}
hipError_t launch_attention_fp4(const AttnArgs& a, const AttnPlan& p, int, bool, hipStream_t) {
  const bool ok = a.kbs && a.vbs && (int64_t)a.num_slots * a.kv_heads < (1ll << 31) && a.num_slots > 0 && a.workers == p.workers &&
                  (!p.workers || (char*)a.headers - (char*)a.part + p.workers * 8 * 4 == p.workspace);
  return ok ? hipSuccess : hipErrorInvalidValue;
}
}
'''


def test_host_layer_under_address_and_ub_sanitizers(tmp_path):
    rt = _asan_runtime()
    if rt is None:
        pytest.skip("g++ with libasan is not available")
    lib = tmp_path / "libnvfp4_serving_asan.so"
    flags = ["-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fPIC", "-fsanitize=address,undefined",
             "-fno-sanitize-recover=undefined", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
             f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}"]
    stubs = tmp_path / "stubs.cpp"
    stubs.write_text(STUBS)
    objs = []
    for src in (os.path.join(CSRC, "serving_api.hip"), os.path.join(CSRC, "attention_plan.hip"), str(stubs)):
        obj = tmp_path / (os.path.basename(src) + ".o")
        subprocess.run(["g++", "-x", "c++", *flags, "-c", src, "-o", str(obj)], check=True, capture_output=True, text=True)
        objs.append(str(obj))
    subprocess.run(["g++", "-shared", "-fsanitize=address,undefined", "-o", str(lib), *objs], check=True, capture_output=True, text=True)
    prog = tmp_path / "run.py"
    prog.write_text(f'''
import ctypes, sys
sys.path.insert(0, {ROOT!r})
from bit_block_scaled_nvfp4_amd import serving as sv
lib = ctypes.CDLL({str(lib)!r})
sv.declare(lib)
P, big = 0x10000, [0, 1, -1, 7, 16, 2**31 - 1, 2**31, 2**40, 2**62, -2**62, 2**63 - 1, -2**63]
calls = dict(
    rope=(lib.nvfp4_qk_norm_rope, dict(q=P, H=4, qts=512, qhs=128, k=P, Hk=2, kts=256, khs=128, dt=1, T=8, D=128, pos=P, freq=P,
          n=32, pairs=0, qw=P, kw=P, wt=0, eps=1e-6, off=0.0, qo=P, qots=512, qohs=128, ko=P, kots=256, kohs=128, s=None)),
    fp8=(lib.nvfp4_kv_fp8_append, dict(k=P, v=P, dt=1, T=8, Hk=2, D=128, kts=256, khs=128, vts=256, vhs=128, pos=P, freq=P, n=32,
         pairs=0, kw=P, wt=0, eps=1e-6, off=0.0, ks=P, vs=P, slots=P, kc=P, vc=P, S=64, ld=256, s=None)),
    fp4=(lib.nvfp4_kv_fp4_append, dict(k=P, v=P, dt=1, T=8, Hk=2, D=128, kts=256, khs=128, vts=256, vhs=128, pos=P, freq=P, n=32,
         pairs=0, kw=P, wt=0, eps=1e-6, off=0.0, ks=P, vs=P, slots=P, kc=P, kcs=P, vc=P, vcs=P, B=4, bs=16, s=None)),
    load=(lib.nvfp4_kv_fp4_load, dict(c=P, cs=P, B=4, Hk=2, bs=16, D=128, g=P, slots=P, T=8, out=P, dt=0, s=None)),
    attn=(lib.nvfp4_kv_fp4_attention, dict(q=P, dt=1, T=8, H=8, Hk=2, D=128, qts=1024, qhs=128, kc=P, kcs=P, vc=P, vcs=P, ks=P, vs=P,
          B=4, bs=16, table=P, R=2, W=4, tld=4, qs=P, lens=P, scale=0.1, cap=0.0, slopes=None, doc=None, prefix=None, mq=8, ms=64, out=P,
          ots=1024, ohs=128, ws=P, wsb=1 << 30, s=None)),
    tree=(lib.nvfp4_kv_fp4_tree_attention, dict(q=P, dt=1, T=8, H=8, Hk=2, D=128, qts=1024, qhs=128, kc=P, kcs=P, vc=P, vcs=P, ks=P,
          vs=P, B=4, bs=16, table=P, R=2, W=4, tld=4, qs=P, lens=P, scale=0.1, cap=0.0, slopes=None, mask=P, words=1, mld=1, tp=None, mq=8,
          ms=64, out=P, ots=1024, ohs=128, ws=P, wsb=1 << 30, s=None)),
    verify=(lib.nvfp4_verify_drafted, dict(p=P, pld=100, q=P, qld=100, rows=8, V=100, tok=P, qs=P, R=2, au=P, su=P, acc=P, out=P, ws=P,
            wsb=1 << 20, s=None)),
)
n = 0
for name, (fn, good) in calls.items():
    assert fn(*good.values()) == 0, name
    sizes = [k for k, v in good.items() if isinstance(v, int) and v != P]
    for k in sizes:
        if k in ("dt", "wt", "pairs"):
            for v in (-1, 0, 1, 2, 3, 99):
                assert 0 <= fn(*{{**good, k: v}}.values()) <= 3, (name, k, v)
            continue
        for v in big:
            got = fn(*{{**good, k: v}}.values())
            assert 0 <= got <= 3, (name, k, v, got)  # never the device's error: what passes is what the kernels expect
            for j in sizes:
                if j != k and j not in ("dt", "wt", "pairs"):
                    for w in big:
                        got = fn(*{{**good, k: v, j: w}}.values())
                        assert 0 <= got <= 3, (name, k, v, j, w, got)
                        n += 1
for v in big:
    lib.nvfp4_verify_drafted_workspace(v, 100), lib.nvfp4_verify_drafted_workspace(2, v)
    lib.nvfp4_kv_fp4_attention_workspace(v, 8, 2, 128, 2, 8, 64), lib.nvfp4_kv_fp4_attention_workspace(8, v, v, 128, v, v, v)
print("passed", n)
''')
    env = dict(os.environ, LD_PRELOAD=rt, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    res = subprocess.run([sys.executable, str(prog)], capture_output=True, text=True, env=env, timeout=300)
    out = res.stdout + res.stderr
    assert res.returncode == 0 and "passed" in out, out[-4000:]
    assert "ERROR: AddressSanitizer" not in out and "runtime error" not in out
