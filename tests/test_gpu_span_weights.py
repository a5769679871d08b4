"""GPU: softmax weights far below a row's largest, in the span attention.

Weights are fp16 for the value product, between 2^7 and 2^15 for the largest one of
a row, so that each of the others is off by half of fp16's step: 2^-11 of itself, or
2^-25 / 2^7 = 2^-32 of the largest weight where that is more (fp16's least step is
2^-24)."""
import math

import numpy as np
import pytest
import torch

import _gpu
import _span
from paged_kv_decode_ns_gb300 import binding as nb
from paged_kv_decode_ns_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

Q, K, SCALE = 4.0, 35.0, 0.125
LEAST = math.exp(-SCALE * Q * K)  # weight of an ordinary key beside the first one's, 2^-25.2


def check(out, keys, value, dtype):
    """Every element of out against `keys` ordinary keys of that value beside one of 0."""
    want = value * keys * LEAST / (1.0 + keys * LEAST)
    got = _gpu.to_f64(out)
    # 2^-32 a key, or 2^-11 of its weight; the exponential's 2^-22 and the score's rounding,
    # 2^-24 of 25.2 units, are 2^-18 together; half a step of the output
    allowed = value * keys * 2.0 ** -32 + want * (2.0 ** -11 + 2.0 ** -18) + 0.5 * _gpu.ulp(np.array(want), dtype)
    assert allowed < want / 8  # the bound tells a vanished weight from one that counts
    assert np.abs(got - want).max() <= allowed
    _gpu.assert_no_device_status()


def prompt(tokens, keys, hq, hkv, d, dtype, value):
    td = _span.TORCH[dtype]
    q = torch.zeros(tokens, hq, d, dtype=td, device="cuda")
    k = torch.zeros(1 + keys, hkv, d, dtype=td, device="cuda")
    v = torch.full_like(k, value)
    q[..., 0], k[0, :, 0], v[0] = Q, K, 0
    out = torch.empty_like(q)
    # every token sees all of the keys: `tokens` sequences would each need keys of their own,
    # so a span whose own keys are at the end, with values of 0 and scores that vanish
    if tokens > 1:
        pad = torch.zeros(tokens - 1, hkv, d, dtype=td, device="cuda")
        low = pad.clone()
        low[..., 0] = -4 * K
        k, v = torch.cat([k, low]), torch.cat([v, pad])
    starts = _gpu.dev_ints([0, tokens], np.int32)
    kstarts = _gpu.dev_ints([0, k.shape[0]], np.int32)
    nb.ns_prompt_attn(q, k, v, starts, SCALE, out, nb.alloc_span_workspace(d), key_start_loc=kstarts)
    return out


@pytest.mark.parametrize("dtype", [wl.F16, wl.BF16])
@pytest.mark.parametrize("hq,hkv,d", [(14, 2, 64), (4, 2, 128)])
def test_keys_far_below_one(dtype, hq, hkv, d):
    for keys in (200, 63):  # a unit that is not cut, several tiles and one
        check(prompt(1, keys, hq, hkv, d, dtype, 1024.0), keys, 1024.0, dtype)


@pytest.mark.parametrize("dtype", [wl.F16, wl.BF16])
def test_one_key_over_128_k_others(dtype):
    """Units enough that one CTA sees half of a row's keys."""
    check(prompt(304, 131072, 64, 1, 64, dtype, 1.0), 131072, 1.0, dtype)


@pytest.mark.parametrize("dtype", [wl.F16, wl.BF16])
def test_keys_far_below_one_over_a_q8_0_cache(dtype):
    keys, value = 200, 1016.0
    nblk = -(-(keys + 1) // 16)
    kc = torch.zeros(nblk, 2, 16, 64, dtype=torch.int8, device="cuda")
    ks = torch.ones(nblk, 2, 16, 2, dtype=torch.float16, device="cuda")
    vc, vs = torch.full_like(kc, 127), torch.full_like(ks, value / 127)
    kc[0, :, 0, 0], vc[0, :, 0] = int(K), 0
    q = torch.zeros(1, 14, 64, dtype=_span.TORCH[dtype], device="cuda")
    q[..., 0] = Q
    out = torch.empty_like(q)
    table = torch.arange(nblk, dtype=torch.int32, device="cuda")[None]
    nb.ns_paged_attn_prefill_q8_0(q, _gpu.dev_ints([0, 1], np.int32), kc, ks, vc, vs, table,
                                  _gpu.dev_ints([keys + 1], np.int32), SCALE, out, nb.alloc_span_workspace(64))
    check(out, keys, value, dtype)
