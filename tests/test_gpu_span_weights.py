"""GPU: softmax weights far below a row's largest, in the span attention.

Weights are fp16 for the value product, between 2^7 and 2^15 for the largest one of
a row, so that each of the others is off by half of fp16's step: 2^-11 of itself, or
2^-25 / 2^7 = 2^-32 of the largest weight where that is more (fp16's least step is
2^-24).  The largest bf16 value that a unit has met is laid out at 2^11 or more, the
largest q8_0 scale at 2^4, so that no value is off by more than 2^-25 / 2^11 of the one
or 127 times 2^-25 / 2^4 of the other."""
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


def near(got, want, size, least, dtype):
    """Element by element: the weights and the values each rounded to fp16 (2^-11 of
    `size`, the weighted mean of |v|), the exponential and the score (2^-18), `least` by
    which any value is off, half a step of the output."""
    allowed = size.numpy() * (2.0 ** -10 + 2.0 ** -18) + least + 0.5 * _gpu.ulp(want.numpy(), dtype)
    assert np.all(np.abs(_gpu.to_f64(got) - want.numpy()) <= allowed)
    _gpu.assert_no_device_status()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tokens,keys,key,outlier", [(1, 250, 20.0, 2.0 ** 20),
                                                     (304, 8192, 18.0, 2.0 ** 12)])
def test_one_large_value_leaves_the_weights_of_other_keys(tokens, keys, key, outlier, d):
    """One key holds as much weight as many others, or thirty times that, and a value far above theirs in
    one channel: in the other channels it is one value among many, before and behind it."""
    hq, hkv = (64, 1) if tokens > 1 else (4, 2)
    g = torch.Generator().manual_seed(keys)
    v = 1.0 + 0.5 * torch.randn(keys + 1, hkv, d, generator=g)
    for at in (0, keys // 2, keys):
        vals = v.clone()
        vals[at, :, 0] = outlier
        vals = torch.cat([vals, torch.zeros(tokens - 1, hkv, d)]).bfloat16()
        k = torch.zeros(keys + tokens, hkv, d)
        k[at, :, 0], k[keys + 1:, :, 0] = key, -4 * K  # the span's own tokens have no weight
        q = torch.zeros(tokens, hq, d, dtype=torch.bfloat16, device="cuda")
        q[..., 0] = Q
        out = torch.empty_like(q)
        nb.ns_prompt_attn(q, k.bfloat16().cuda(), vals.cuda(), _gpu.dev_ints([0, tokens], np.int32), SCALE, out,
                          nb.alloc_span_workspace(d), key_start_loc=_gpu.dev_ints([0, keys + tokens], np.int32))
        w = torch.exp(SCALE * Q * k[:keys + 1, 0, 0].double() - SCALE * Q * key)
        w = w / w.sum()
        vals = vals[:keys + 1].double()
        mean = lambda x: torch.einsum("k,khd->hd", w, x).repeat_interleave(hq // hkv, 0)  # noqa: E731
        want, size = (mean(x).expand(tokens, hq, d).clone() for x in (vals, vals.abs()))
        near(out, want, size, outlier * 2.0 ** -36, wl.BF16)


@pytest.mark.parametrize("dtype,plain,large", [(wl.F16, 2.0 ** -14, 8.0), (wl.BF16, 2.0 ** -6, 2.0 ** 15)])
def test_one_large_scale_leaves_the_weights_of_other_keys(dtype, plain, large):
    """The same over a q8_0 cache: the block of 32 channels with the large scale, and the other."""
    keys, key = 250, 20
    rng = np.random.default_rng(3)
    nblk = -(-(keys + 1) // 16)
    for at in (0, keys // 2, keys):
        codes = rng.integers(30, 128, (nblk * 16, 2, 64)).astype(np.int8)
        scales = np.full((nblk * 16, 2, 2), plain, np.float16)
        scales[at, :, 0] = large
        scales[keys + 1:] = np.nan  # behind the last key
        kcodes = np.zeros_like(codes)
        kcodes[at, :, 0] = key
        rows = lambda a: torch.from_numpy(  # noqa: E731
            np.ascontiguousarray(a.reshape(nblk, 16, 2, -1).swapaxes(1, 2))).cuda()
        q = torch.zeros(1, 14, 64, dtype=_span.TORCH[dtype], device="cuda")
        q[..., 0] = Q
        out = torch.empty_like(q)
        table = torch.arange(nblk, dtype=torch.int32, device="cuda")[None]
        nb.ns_paged_attn_prefill_q8_0(q, _gpu.dev_ints([0, 1], np.int32), rows(kcodes), rows(np.ones_like(scales)),
                                      rows(codes), rows(scales), table, _gpu.dev_ints([keys + 1], np.int32), SCALE, out,
                                      nb.alloc_span_workspace(64))
        w = torch.exp(torch.tensor([0.0 if i == at else -SCALE * Q * key for i in range(keys + 1)]).double())
        vals = torch.from_numpy(codes[:keys + 1].astype(np.float64) * np.repeat(scales[:keys + 1].astype(np.float64), 32, -1))
        want = torch.einsum("k,khd->hd", w / w.sum(), vals).repeat_interleave(7, 0)[None]
        near(out, want, want, 127 * large * 2.0 ** -29, dtype)  # all values are positive


def test_a_large_value_that_is_not_seen():
    """Rows in front of a value 2^20 times theirs share its tile and keep their accuracy."""
    g = torch.Generator().manual_seed(5)
    n = 300
    q, k = torch.randn(n, 4, 64, generator=g).bfloat16(), torch.randn(n, 2, 64, generator=g).bfloat16()
    v = (1.0 + torch.rand(n, 2, 64, generator=g)).bfloat16()
    v[200] = 2.0 ** 20
    out = torch.empty(n, 4, 64, dtype=torch.bfloat16, device="cuda")
    nb.ns_prompt_attn(q.cuda(), k.cuda(), v.cuda(), _gpu.dev_ints([0, n], np.int32), SCALE, out, nb.alloc_span_workspace(64))
    want = _span.attend(q, k, v, SCALE)
    # scores of N(0, 1) rows, 64 products in fp32: 2^-18 again
    near(out[:200], want[:200], want[:200], 2.0 ** 20 * 2.0 ** -36, wl.BF16)
