"""Host-side argument checks of the rotary append and the q4_0 calls: they answer before anything is
launched, so no GPU is needed."""
import os
import re

import pytest
import torch

from paged_kv_decode_ns_gb300 import _build, binding

OK, INVALID, UNSUPPORTED = 0, -1, -2
A = 1 << 20  # a 16-byte aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return binding.lib()


def rope(lib, pool="16", q=A, k=A, v=A, pos=A, cs=A, slots=A, qo=A, ko=A, kp=A, ks=A, vp=A, vs=A, T=4, hq=14, hkv=2, d=64,
         r=64, il=0, maxp=100, qs=None, kst=None, vst=None, qos=None, kos=None, bs=16, nb=10, dtype=0):
    pools = (kp, vp) if pool == "16" else (kp, ks, vp, vs)
    f = {"16": lib.ns_rope_kv_append, "q8_0": lib.ns_rope_kv_append_q8_0, "q4_0": lib.ns_rope_kv_append_q4_0}[pool]
    w, kw = hq * d, hkv * d
    return f(q, k, v, pos, cs, slots, qo, ko, *pools, T, hq, hkv, d, r, il, maxp, w if qs is None else qs,
             kw if kst is None else kst, kw if vst is None else vst, w if qos is None else qos, kw if kos is None else kos,
             bs, nb, dtype, None)


@pytest.mark.parametrize("pool", ["16", "q8_0", "q4_0"])
@pytest.mark.parametrize("change,want", [
    (dict(hq=0), INVALID), (dict(hkv=0), INVALID), (dict(T=-1), INVALID), (dict(nb=0), INVALID), (dict(maxp=0), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(d=32, r=32), UNSUPPORTED), (dict(bs=64), UNSUPPORTED), (dict(bs=0), UNSUPPORTED),
    (dict(dtype=2), UNSUPPORTED), (dict(r=0), UNSUPPORTED), (dict(r=8), UNSUPPORTED), (dict(r=24), UNSUPPORTED),
    (dict(r=80), UNSUPPORTED), (dict(r=-16), UNSUPPORTED), (dict(qs=14 * 64 - 8), INVALID), (dict(qs=14 * 64 + 4), INVALID),
    (dict(kst=120), INVALID), (dict(vst=1 << 40), INVALID), (dict(qos=0), INVALID), (dict(kos=64), INVALID),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(pos=None), INVALID),
    (dict(cs=None), INVALID), (dict(slots=None), INVALID), (dict(qo=None), INVALID), (dict(kp=None), INVALID),
    (dict(vp=None), INVALID), (dict(q=A + 8), INVALID), (dict(k=A + 2), INVALID), (dict(v=A + 4), INVALID),
    (dict(cs=A + 4), INVALID), (dict(qo=A + 8), INVALID), (dict(ko=A + 8), INVALID), (dict(kp=A + 8), INVALID),
    (dict(d=128, r=128, bs=32), UNSUPPORTED), (dict(T=0, q=None, pos=None, kp=None), OK)])
def test_rope_append_checks(lib, pool, change, want):
    assert rope(lib, pool, **change) == want


def test_rows_whose_offsets_pass_32_bits_are_refused(lib):
    assert rope(lib, hq=(1 << 24) + 1) == UNSUPPORTED and rope(lib, hkv=(1 << 24) + 1) == UNSUPPORTED
    assert rope(lib, "q4_0", hq=(1 << 31) - 1) == UNSUPPORTED and append(lib, hkv=(1 << 31) - 1) == UNSUPPORTED
    assert rope(lib, hq=1 << 24, T=0) == OK and append(lib, hkv=1 << 24, T=0) == OK


def test_rope_append_pools_of_their_own(lib):
    assert rope(lib, "q8_0", d=128, r=64) == UNSUPPORTED
    for pool in ("q8_0", "q4_0"):
        assert rope(lib, pool, ks=None) == INVALID and rope(lib, pool, vs=A + 2) == INVALID


def append(lib, k=A, v=A, slots=A, kc=A, ks=A, vc=A, vs=A, T=4, hkv=2, d=64, bs=16, nb=10, dtype=0):
    return lib.ns_kv_append_q4_0(k, v, slots, kc, ks, vc, vs, T, hkv, d, bs, nb, dtype, None)


@pytest.mark.parametrize("change,want", [
    (dict(T=-1), INVALID), (dict(hkv=0), INVALID), (dict(nb=0), INVALID), (dict(d=96), UNSUPPORTED),
    (dict(bs=12), UNSUPPORTED), (dict(d=128, bs=8), UNSUPPORTED), (dict(dtype=7), UNSUPPORTED), (dict(k=None), INVALID),
    (dict(slots=None), INVALID), (dict(ks=None), INVALID), (dict(vc=A + 8), INVALID), (dict(T=0, k=None), OK)])
def test_append_checks(lib, change, want):
    assert append(lib, **change) == want


def gather(lib, k=A, ks=A, v=A, vs=A, bt=A, sl=A, S=2, T=8, hkv=2, d=64, bs=16, ko=A, vo=A, width=4, nb=9, dtype=0):
    return lib.ns_kv_gather_q4_0(k, ks, v, vs, bt, sl, S, T, hkv, d, bs, ko, vo, None, width, nb, dtype)


@pytest.mark.parametrize("change,want", [
    (dict(S=-1), INVALID), (dict(T=-1), INVALID), (dict(hkv=0), INVALID), (dict(width=0), INVALID), (dict(d=32), UNSUPPORTED),
    (dict(d=128, bs=4), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED), (dict(ks=None), INVALID), (dict(vo=None), INVALID),
    (dict(ko=A + 2), INVALID), (dict(S=0), OK), (dict(T=0), OK)])
def test_gather_checks(lib, change, want):
    assert gather(lib, **change) == want


def decode(lib, q=A, kc=A, ks=A, vc=A, vs=A, bt=A, cl=A, S=2, hq=14, hkv=2, d=64, bs=16, scale=0.125, out=A, width=8, nb=10,
           dtype=0, ws=A, wsb=1 << 40):
    return lib.ns_paged_attn_decode_q4_0(q, kc, ks, vc, vs, bt, cl, S, hq, hkv, d, bs, scale, out, None, width, nb, dtype,
                                         ws, wsb)


@pytest.mark.parametrize("change,want", [
    (dict(S=-1), INVALID), (dict(hq=0), INVALID), (dict(hkv=0), INVALID), (dict(hq=15), UNSUPPORTED),
    (dict(hq=65, hkv=1), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(d=128, bs=32), UNSUPPORTED),
    (dict(bs=64), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(width=0), INVALID), (dict(nb=0), INVALID),
    (dict(width=1 << 30), UNSUPPORTED), (dict(S=1 << 20, width=1 << 20, bs=32), UNSUPPORTED),
    (dict(hq=1 << 27, hkv=1 << 27), UNSUPPORTED),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(q=None), INVALID),
    (dict(ks=None), INVALID), (dict(bt=None), INVALID), (dict(cl=None), INVALID), (dict(out=None), INVALID),
    (dict(ws=None), INVALID), (dict(vc=A + 8), INVALID), (dict(out=A + 2), INVALID), (dict(wsb=100), INVALID),
    (dict(S=0), OK)])
def test_decode_checks(lib, change, want):
    assert decode(lib, **change) == want


def test_workspace_counts_groups_that_are_not_cut_evenly(lib):
    size = lib.ns_paged_attn_workspace_bytes
    base = size(10000, 8, 1, 64)
    assert size(10000, 9, 1, 64) - base >= 10000 * 4 - 256 and size(10000, 17, 1, 64) - base >= 20000 * 4 - 256
    assert decode(lib, S=10000, hq=9, hkv=1, wsb=base) == INVALID


def prefill(lib, q=A, qsl=A, kc=A, ks=A, vc=A, vs=A, bt=A, cl=A, S=2, T=8, hq=14, hkv=2, d=64, bs=16, scale=0.125, out=A,
            width=8, nb=10, dtype=0, ws=A, wsb=1 << 40):
    return lib.ns_paged_attn_prefill_q4_0(q, qsl, kc, ks, vc, vs, bt, cl, S, T, hq, hkv, d, bs, scale, out, None, width,
                                          nb, dtype, ws, wsb)


@pytest.mark.parametrize("change,want", [
    (dict(d=96), UNSUPPORTED), (dict(bs=32), UNSUPPORTED), (dict(d=128, bs=8), UNSUPPORTED), (dict(hq=15), UNSUPPORTED), (dict(hq=65, hkv=1), UNSUPPORTED),
    (dict(dtype=9), UNSUPPORTED), (dict(width=1 << 30), UNSUPPORTED), (dict(width=0), INVALID), (dict(S=-1), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(q=None), INVALID), (dict(vs=None), INVALID), (dict(ks=A + 2), INVALID),
    (dict(wsb=0), INVALID), (dict(d=128, wsb=0), INVALID), (dict(d=128, T=0), OK), (dict(T=0), OK), (dict(S=0), OK)])
def test_prefill_checks(lib, change, want):
    assert prefill(lib, **change) == want


# ---------------------------------------------------------------- the binding's own checks
def cpu(*shape, dtype=torch.float16):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_refuses_shapes_that_do_not_match():
    q, k, cs = cpu(3, 14, 64), cpu(3, 2, 64), cpu(10, 64, dtype=torch.float32)
    pos, slots = cpu(3, dtype=torch.int32), cpu(3, dtype=torch.int64)
    pool = cpu(4, 2, 16, 64)
    for bad in (dict(k=cpu(2, 2, 64)), dict(v=cpu(3, 1, 64)), dict(q=cpu(3, 14, 32)), dict(positions=cpu(4, dtype=torch.int32)),
                dict(cos_sin=cpu(10, dtype=torch.float32)), dict(q_out=cpu(3, 13, 64)), dict(k_out=cpu(3, 14, 64)),
                dict(k_pool=cpu(4, 3, 16, 64)), dict(v_pool=cpu(5, 2, 16, 64)), dict(q=q)):
        args = dict(q=q, k=k, v=k, positions=pos, cos_sin=cs, slot_mapping=slots, q_out=q, k_pool=pool, v_pool=pool)
        args.update(bad)
        with pytest.raises(ValueError):  # the last one: host tensors
            binding.ns_rope_kv_append(**args)
    codes, steps = cpu(4, 2, 16, 32, dtype=torch.uint8), cpu(4, 2, 16, 2)
    bt, cl, ws = cpu(3, 4, dtype=torch.int32), cpu(3, dtype=torch.int32), cpu(8, dtype=torch.uint8)
    with pytest.raises(ValueError):
        binding.ns_paged_attn_decode_q4_0(q, codes, cpu(4, 2, 16, 4), codes, steps, bt, cl, 0.1, q, ws)
    with pytest.raises(ValueError):
        binding.ns_kv_append_q4_0(k, k, slots, codes, steps, cpu(4, 2, 16, 64, dtype=torch.uint8), steps)


class Elsewhere(torch.Tensor):
    """A tensor that says it is on GPU 7."""
    is_cuda = True

    def get_device(self):
        return 7


def test_binding_refuses_tensors_of_another_device(monkeypatch):
    monkeypatch.setattr(binding, "_raw_device", lambda: 0)
    monkeypatch.setattr(binding, "_invoke", lambda *a: pytest.fail("called"))
    def there(*shape, dtype=torch.float16):
        return torch.zeros(*shape, dtype=dtype).as_subclass(Elsewhere)
    codes, steps = there(4, 2, 16, 32, dtype=torch.uint8), there(4, 2, 16, 2)
    q, k, slots = there(3, 14, 64), there(3, 2, 64), there(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="current CUDA device"):
        binding.ns_kv_append_q4_0(k, k, slots, codes, steps, codes, steps)
    with pytest.raises(ValueError, match="current CUDA device"):
        binding.ns_rope_kv_append(q, k, k, there(3, dtype=torch.int32), there(9, 64, dtype=torch.float32), slots, q,
                                  there(4, 2, 16, 64), there(4, 2, 16, 64))
    codes8 = there(4, 2, 16, 64, dtype=torch.int8)
    with pytest.raises(ValueError, match="current CUDA device"):
        binding.ns_rope_kv_append_q8_0(q, k, k, there(3, dtype=torch.int32), there(9, 64, dtype=torch.float32), slots, q,
                                       codes8, steps, codes8, steps)


# ---------------------------------------------------------------- order on the stream
@pytest.mark.parametrize("name,kernel", [("rope_append.cu", "rope_append_kernel"), ("decode_q4.cu", "decode_q4_kernel"),
                                         ("kv_gather.cu", "kv_gather_kernel")])
def test_kernels_launched_early_wait_for_the_grid_in_front(name, kernel):
    """They start while the grid in front ends (launch_early): nothing is read before the wait, and nothing
    through the read-only path."""
    with open(os.path.join(_build.CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    assert "launch_early(" in text
    body = re.search(r"__global__[^;{]*?\b" + kernel + r"\s*\(.*?\n}\n", text, re.S).group(0)
    before = body[:body.index("grid_dependency_wait()")]
    assert "a.slot_mapping" not in before and "context_lens" not in before and "start_loc" not in before
    assert "__ldg" not in text and "__restrict__" not in text and "ld.global.nc" not in text
