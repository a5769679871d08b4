"""GPU: the span attention calls with scores up to the size that they are documented for (2^22, times log2 e).
Keys are exact in fp16 (4- and 8-bit ones by steps that are powers of two), so that a score is off by a few 2^-24
of itself and the rounding of its reference, 2^-2, at most.  The largest two of 600 normal ones of 2^19 lie
20 or more apart but for 2^-12 of the rows: one key has all the weight, and the output is its row of V (rounded to
fp16 where the calls say so, and to the output's type)."""
import numpy as np
import pytest
import torch

import _gpu
import _q4
import _span
from _q4 import wl
from paged_kv_decode_ns_gb300 import binding as nb

pytestmark = pytest.mark.gpu

HQ, HKV = 2, 1
SPANS = [(1, 1), (3, 33), (40, 130), (1, 640)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,scale,q_amp", [(wl.F16, 0.125, 1e4), (wl.F16, -1e4, 0.125), (wl.BF16, 0.125, 1e4), (wl.BF16, 1e-26, 1.25e29)])
def test_prompts(dtype, scale, q_amp, d):
    """Over rows of 40 prompts' keys: standard deviations of 5e5 (D 64) and 7e5."""
    rng = np.random.default_rng(5)
    T, L = sum(n for n, _ in SPANS), sum(L for _, L in SPANS)
    q, k, v = (_q4.to16(rng.standard_normal((n, h, d)).astype(np.float32) * np.float32(amp), dtype)
               for n, h, amp in ((T, HQ, q_amp), (L, HKV, 35.0), (L, HKV, 1.0)))
    at, ks = _span.starts([n for n, _ in SPANS]), _span.starts([L for _, L in SPANS])
    out = torch.full((T, HQ, d), float("nan"), dtype=q.dtype, device="cuda")
    nb.ns_prompt_attn(q.cuda(), k.cuda(), v.cuda(), torch.from_numpy(at).cuda(), scale, out, nb.alloc_span_workspace(d),
                      key_start_loc=torch.from_numpy(ks).cuda())
    ref = torch.cat([_span.attend(q[a:b], k[c:e], v[c:e], scale) for a, b, c, e in zip(at, at[1:], ks, ks[1:])])
    _span.compare(out, ref, dtype)
    _gpu.assert_no_device_status()


@pytest.mark.parametrize("pool,d", [("q8_0", 64), ("q4_0", 64), ("q4_0", 128)])
@pytest.mark.parametrize("dtype,scale,q_amp", [(wl.F16, 0.125, 1e4), (wl.F16, -1e4, 0.125), (wl.BF16, 0.125, 1e4), (wl.BF16, 1e-26, 1.25e29)])
def test_spans(pool, d, dtype, scale, q_amp):
    rng = np.random.default_rng(6)
    cache = (_span.Q8Cache if pool == "q8_0" else _q4.Cache)(rng, [L for _, L in SPANS], HKV, 16, d)
    cache.ks[...] = np.where(np.isnan(cache.ks), cache.ks, np.float16(8.0 if pool == "q4_0" else 0.5))
    values = _q4.values if pool == "q4_0" else _span.q8.dequantize_q8_0
    for s, (_, L) in enumerate(SPANS):
        p = np.arange(L)
        at = (cache.tables[s, p // 16], slice(None), p % 16)
        cache.k[s] = torch.from_numpy(values(cache.kc[at], cache.ks[at]))
    T = sum(n for n, _ in SPANS)
    q = _q4.to16(rng.standard_normal((T, HQ, d)).astype(np.float32) * np.float32(q_amp), dtype)
    kc, ks, vc, vs, bt = cache.dev()
    out = torch.full((T, HQ, d), float("nan"), dtype=q.dtype, device="cuda")
    call = nb.ns_paged_attn_prefill_q8_0 if pool == "q8_0" else nb.ns_paged_attn_prefill_q4_0
    call(q.cuda(), torch.from_numpy(_span.starts([n for n, _ in SPANS])).cuda(), kc, ks, vc, vs, bt,
         _gpu.dev_ints([L for _, L in SPANS], np.int32), scale, out, nb.alloc_span_workspace(d))
    _span.compare(out, _q4.attend_all(q, SPANS, cache, scale), dtype, q8=True)
    _gpu.assert_no_device_status()
