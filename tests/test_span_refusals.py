"""Host-side argument checks of the span attention, read-back and verification
calls: they answer before anything is launched, so no GPU is needed."""
import ctypes

import pytest

from paged_kv_decode_ns_gb300 import _build, binding

OK, INVALID, UNSUPPORTED = 0, -1, -2
A = 1 << 20  # a 16-byte aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return binding.lib()


def prompt(lib, q=A, k=A, v=A, qsl=A, ksl=A, S=2, T=8, Tk=8, hq=14, hkv=2, d=64, qs=None, ks=None, vs=None, scale=0.125,
           out=A, dtype=0, ws=A, wsb=1 << 40):
    return lib.ns_prompt_attn(q, k, v, qsl, ksl, S, T, Tk, hq, hkv, d, hq * d if qs is None else qs,
                              hkv * d if ks is None else ks, hkv * d if vs is None else vs, scale, out, None, dtype, ws,
                              wsb)


@pytest.mark.parametrize("change,want", [
    (dict(hq=0), INVALID), (dict(hkv=0), INVALID), (dict(hq=15), UNSUPPORTED), (dict(hq=130, hkv=2), UNSUPPORTED),
    (dict(d=96), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(S=-1), INVALID), (dict(T=-1), INVALID),
    (dict(Tk=-1), INVALID), (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(ksl=None, Tk=9), INVALID), (dict(qs=14 * 64 - 8), INVALID), (dict(qs=14 * 64 + 4), INVALID),
    (dict(ks=64), INVALID), (dict(vs=1 << 40), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(qsl=None), INVALID), (dict(out=None), INVALID), (dict(ws=None), INVALID),
    (dict(q=A + 8), INVALID), (dict(k=A + 2), INVALID), (dict(out=A + 4), INVALID), (dict(ws=A + 8), INVALID),
    (dict(wsb=16), INVALID), (dict(T=0, q=None, ksl=A), OK), (dict(S=0), OK)])
def test_prompt_attn_checks(lib, change, want):
    assert prompt(lib, **change) == want


def prefill(lib, q=A, qsl=A, kc=A, ks=A, vc=A, vs=A, bt=A, cl=A, S=2, T=8, hq=14, hkv=2, d=64, bs=16, scale=0.125, out=A,
            width=8, nb=10, dtype=0, ws=A, wsb=1 << 40):
    return lib.ns_paged_attn_prefill_q8_0(q, qsl, kc, ks, vc, vs, bt, cl, S, T, hq, hkv, d, bs, scale, out, None, width,
                                          nb, dtype, ws, wsb)


@pytest.mark.parametrize("change,want", [
    (dict(d=128), UNSUPPORTED), (dict(bs=32), UNSUPPORTED), (dict(bs=8), UNSUPPORTED), (dict(hq=15), UNSUPPORTED),
    (dict(hq=65, hkv=1), UNSUPPORTED), (dict(dtype=9), UNSUPPORTED), (dict(width=1 << 30), UNSUPPORTED),
    (dict(width=0), INVALID), (dict(nb=0), INVALID), (dict(S=-1), INVALID), (dict(T=-3), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(q=None), INVALID), (dict(kc=None), INVALID), (dict(ks=None), INVALID),
    (dict(vc=None), INVALID), (dict(vs=None), INVALID), (dict(bt=None), INVALID), (dict(cl=None), INVALID),
    (dict(ks=A + 2), INVALID), (dict(wsb=0), INVALID), (dict(T=0), OK), (dict(S=0), OK)])
def test_prefill_q8_0_checks(lib, change, want):
    assert prefill(lib, **change) == want


def gather(lib, q8=False, k=A, ks=A, v=A, vs=A, bt=A, sl=A, S=2, T=8, hkv=2, d=64, bs=16, ko=A, vo=A, width=4, nb=9,
           dtype=0):
    pools = (k, ks, v, vs) if q8 else (k, v)
    f = lib.ns_kv_gather_q8_0 if q8 else lib.ns_kv_gather
    return f(*pools, bt, sl, S, T, hkv, d, bs, ko, vo, None, width, nb, dtype)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("change,want", [
    (dict(d=32), UNSUPPORTED), (dict(bs=12), UNSUPPORTED), (dict(d=128, bs=8), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED),
    (dict(hkv=0), INVALID), (dict(S=-1), INVALID), (dict(T=-1), INVALID), (dict(width=0), INVALID),
    (dict(nb=0), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(bt=None), INVALID),
    (dict(sl=None), INVALID), (dict(ko=None), INVALID), (dict(vo=A + 8), INVALID), (dict(S=0), OK), (dict(T=0), OK)])
def test_gather_checks(lib, q8, change, want):
    assert gather(lib, q8, **change) == want


def test_gather_q8_0_has_its_own_checks(lib):
    assert gather(lib, True, d=128) == UNSUPPORTED
    assert gather(lib, True, ks=None) == INVALID
    assert gather(lib, True, vs=A + 2) == INVALID


def verify(lib, p=A, q=A, x=A, sl=A, a=A, s=A, S=2, T=5, V=100, ps=100, qs=100, out=A, num=A):
    return lib.ns_verify_drafts(p, q, x, sl, a, s, S, T, V, ps, qs, out, num, None)


@pytest.mark.parametrize("change,want", [
    (dict(S=-1), INVALID), (dict(T=-1), INVALID), (dict(V=0), INVALID), (dict(ps=99), INVALID), (dict(qs=99), INVALID),
    (dict(p=None), INVALID), (dict(p=A + 4), INVALID), (dict(x=None), INVALID), (dict(sl=None), INVALID),
    (dict(a=None), INVALID), (dict(s=None), INVALID), (dict(out=None), INVALID), (dict(num=None), INVALID),
    (dict(S=0x7fffffff, T=0x7fffffff), INVALID), (dict(S=0), OK)])
def test_verify_checks(lib, change, want):
    assert verify(lib, **change) == want


def test_workspace_sizes(lib):
    assert lib.ns_span_attn_workspace_bytes(64) > 0 and lib.ns_span_attn_workspace_bytes(128) > 0
    assert lib.ns_span_attn_workspace_bytes(96) == 0
    assert ctypes.sizeof(ctypes.c_size_t) == 8


def test_verify_refuses_a_vocabulary_beyond_its_positions(lib):
    assert verify(lib, V=(1 << 30) + 1, ps=1 << 31, qs=1 << 31) == UNSUPPORTED
    assert verify(lib, V=1 << 30, ps=1 << 31, qs=1 << 31, out=None) == INVALID
