"""GPU: the q4_0 calls where the others' tests do not look: repeated small calls, scores of any size."""
import numpy as np
import pytest
import torch

import _gpu
import _q4
from _q4 import wl
from _span import attend as exact_attend, compare as span_compare
from paged_kv_decode_ns_gb300 import binding as nb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[200, 64, 17, 1], [333] * 32, [4096, 5]])
def test_few_sequences_many_times(lens, d):
    """Up to 32 sequences: the warps of a CTA meet at no barrier before they leave records of cut pairs to each
    other.  300 calls, each into an output of its own, behind kernels that leave the SMs at different times."""
    rng = np.random.default_rng(1)
    cache = _q4.Cache(rng, lens, 2, 16, d)
    q = _q4.to16(rng.standard_normal((len(lens), 14, d)).astype(np.float32), wl.F16)
    ref = _q4.attend_all(q, [(1, n) for n in lens], cache, d ** -0.5).numpy()
    pools, cl, ws, qd = cache.dev(), _gpu.dev_ints(lens, np.int32), nb.alloc_workspace(len(lens), 14, 2, d), q.cuda()
    outs = torch.full((300, *q.shape), float("nan"), dtype=q.dtype, device="cuda")
    load = torch.zeros(1 << 22, device="cuda")
    for i in range(300):
        if i % 3 == 0:
            load[: 1 + (i * 7919) % load.numel()].add_(1.0)
        nb.ns_paged_attn_decode_q4_0(qd, *pools, cl, d ** -0.5, outs[i], ws)
    torch.cuda.synchronize()
    _q4.compare(outs[0], ref, wl.F16)
    assert (outs.view(torch.int16) == outs[0].view(torch.int16)).all() and _q4.status() == 0


def attend(cache, q, lens, scale, dtype):
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    nb.ns_paged_attn_decode_q4_0(q.cuda(), *cache.dev(), _gpu.dev_ints(lens, np.int32), scale, out,
                                 nb.alloc_workspace(len(lens), q.shape[1], cache.kc.shape[1], q.shape[2]))
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale,amp", [(0.0, 1e-30), (1e-30, 1e-30), (0.125, 1e-37), (1e-38, 1.0), (-1e-30, 1e-20), (0.0, 1e30)])
def test_scores_that_vanish(scale, amp, d):
    """The mean of the values, also beside tokens that are not there: the last tile's, and a bad block's."""
    rng = np.random.default_rng(2)
    lens = [1, 33, 100, 700]
    cache = _q4.Cache(rng, lens, 2, 16, d)
    q = _q4.to16(rng.standard_normal((4, 14, d)).astype(np.float32) * np.float32(amp), wl.BF16)
    ref = _q4.attend_all(q, [(1, n) for n in lens], cache, scale).numpy()
    _q4.compare(attend(cache, q, lens, scale, wl.BF16), ref, wl.BF16)
    assert _q4.status() == 0
    cache.tables[2, 1] = -1
    keep = np.r_[0:16, 32:100]
    ref[2] = exact_attend(q[2:3], cache.k[2][keep], cache.v[2][keep], scale).numpy()[0]
    _q4.compare(attend(cache, q, lens, scale, wl.BF16), ref, wl.BF16)
    assert _q4.status() == 1


def rows_of(cache, s, L):
    """fp64 K and V [L, Hkv, D] of a sequence through its table, whose entries may repeat."""
    p = np.arange(L)
    at = (cache.tables[s, p // 16], slice(None), p % 16)
    return (torch.from_numpy(_q4.values(c[at], st[at])) for c, st in ((cache.kc, cache.ks), (cache.vc, cache.vs)))


# Scores from 2^24 on.  They are far apart (the chance that the largest two of up to 800 differ by less
# than 2^-20 of themselves, where fp32 scores could change places, is about 800 2^-20 a row), so that one key, or
# equal ones, has all the weight, and the output is its row of V to the last rounding.
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,scale,q_amp,amp", [
    (wl.F16, 0.125, 1e4, 3000.0), (wl.BF16, 0.125, 1e9, 1.0), (wl.BF16, 0.125, 1e20, 1.0), (wl.BF16, 0.125, 1e37, 1.0),
    (wl.BF16, -1.0, 1e37, 30.0), (wl.F16, 1e9, 1.0, 1.0), (wl.F16, 3e38, 100.0, 1.0), (wl.BF16, 1e30, 1e30, 1.0),
    (wl.BF16, 1e-30, 1e37, 30.0)])
def test_scores_of_any_size(dtype, scale, q_amp, amp, d):
    rng = np.random.default_rng(3)
    lens = [1, 33, 100, 777]
    cache = _q4.Cache(rng, lens, 2, 16, d, amp)
    q = _q4.to16(rng.standard_normal((4, 14, d)).astype(np.float32) * np.float32(q_amp), dtype)
    ref = _q4.attend_all(q, [(1, n) for n in lens], cache, scale).numpy()
    _q4.compare(attend(cache, q, lens, scale, dtype), ref, dtype)
    assert _q4.status() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_amp", [1.0, 1e9, 1e37])
def test_large_scores_that_recur_across_pieces(q_amp, d):
    """The same keys again and again along a sequence that every CTA has a piece of, its second half
    among keys whose values are 2^12 larger: the pieces agree on the weights of equal scores."""
    rng = np.random.default_rng(4)
    cache = _q4.Cache(rng, [80, 80], 1, 16, d, 1.0)
    near, far = cache.tables[0].copy(), cache.tables[1].copy()
    cache.vs[far] = (cache.vs[far].astype(np.float32) * 4096).astype(np.float16)
    if q_amp > 1:  # no weight there
        cache.ks[far] = (cache.ks[far].astype(np.float32) / 64).astype(np.float16)
    cache.tables = np.concatenate((np.resize(near, 200), np.resize(np.concatenate((near, far)), 200)))[None].astype(np.int32)
    L = 400 * 16
    q = _q4.to16(rng.standard_normal((1, 8, d)).astype(np.float32) * np.float32(q_amp), wl.BF16)
    ref = exact_attend(q, *rows_of(cache, 0, L), d ** -0.5).numpy()
    got = attend(cache, q, [L], d ** -0.5, wl.BF16)
    if q_amp > 1:
        _q4.compare(got, ref, wl.BF16)
    else:  # a rounding of each weight times its step by 2^-11, against values of 2^12 times 5; and the output's
        assert (np.abs(_gpu.to_f64(got) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -11 * 4096 * 5).all()
    assert _q4.status() == 0


@pytest.mark.parametrize("dtype", [wl.F16, wl.BF16])
@pytest.mark.parametrize("d,amp", [(64, 1.0), (64, 1e-4), (64, 30.0), (64, 3000.0), (128, 1.0), (128, 1e-2)])
def test_every_element_is_off_by_its_roundings(dtype, d, amp):
    """Element by element.  With weights p_j: the product of a weight and its step is off by 2^-11 of itself, so a sum
    by 2^-11 sum p |v|; a score by what an fp32 sum of terms up to 15 |q_i| d and their 8 |q_i| d loses (2^-21 of
    sum |q_i| 16 d), which moves the weights by as much, in numerator and denominator; sums of 700 terms
    by 700 2^-24.  Then the output's own half step, or fp16's least one."""
    rng = np.random.default_rng(8)
    lens = [700, 40, 3]
    cache = _q4.Cache(rng, lens, 2, 16, d, amp)
    q = _q4.to16(rng.standard_normal((3, 14, d)).astype(np.float32), dtype)
    scale = d ** -0.5 / amp
    got = _gpu.to_f64(attend(cache, q, lens, scale, dtype))
    half = torch.finfo(q.dtype).eps / 2
    for s, n in enumerate(lens):
        for j in range(14):
            k, v = cache.k[s][:, j // 7], cache.v[s][:, j // 7]
            x = q[s, j].double()
            p = torch.softmax(scale * (k @ x), 0)
            ref, size = p @ v, p @ v.abs()
            off = scale * 2.0 ** -21 * 16 * float(x.abs().sum()) * amp  # (a step is 5/8 of that at most)
            bound = half * ref.abs() + 2.0 ** -25 + (2.0 ** -11 + 2 * off + 700 * 2.0 ** -24) * size
            err = (torch.from_numpy(got[s, j]) - ref).abs()
            assert (err <= bound).all(), (s, j, float((err / bound).max()))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("call", ["decode", "spans", "prompts"])
def test_scales_below_the_normal_numbers(call, d):
    """Scores of ordinary size from a subnormal scale and large queries (a prompt's products stay below fp32's end)."""
    rng = np.random.default_rng(9)
    lens, scale = [1, 33, 400], float(np.float32(5e-40))
    cache = _q4.Cache(rng, lens, 2, 16, d)
    q = _q4.to16(rng.standard_normal((3, 14, d)).astype(np.float32) * np.float32(3e38 / (64 if call == "prompts" else 8)), wl.BF16)
    one, out = _gpu.dev_ints([0, 1, 2, 3], np.int32), torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    k, v = cache.k, cache.v
    if call == "decode":
        out = attend(cache, q, lens, scale, wl.BF16)
    elif call == "spans":
        nb.ns_paged_attn_prefill_q4_0(q.cuda(), one, *cache.dev(), _gpu.dev_ints(lens, np.int32), scale, out,
                                      nb.alloc_span_workspace(d))
    else:
        k, v = ([x.to(torch.bfloat16) for x in y] for y in (k, v))
        nb.ns_prompt_attn(q.cuda(), torch.cat(k).cuda(), torch.cat(v).cuda(), one, scale, out, nb.alloc_span_workspace(d),
                          key_start_loc=_gpu.dev_ints(np.cumsum([0] + lens), np.int32))
    ref = torch.cat([exact_attend(q[s:s + 1], k[s], v[s], scale) for s in range(3)])
    span_compare(out, ref, wl.BF16, q8=True)
    assert _q4.status() == 0
