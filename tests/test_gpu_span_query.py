"""GPU: how the span attention takes its queries: scales of either sign in every
form, query rows of other sequences and of none beside a tile's, strided rows, and
units whose query tiles have no tokens or no keys.  Tolerances are those of the single
calls' tests."""
import numpy as np
import pytest
import torch

import _gpu
import _span
from paged_kv_decode_ns_gb300 import binding as nb
from paged_kv_decode_ns_gb300 import workloads as wl
from test_gpu_span_attn import Chunks, Prompts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [wl.F16, wl.BF16])
@pytest.mark.parametrize("hq,hkv,d", [(14, 2, 64), (5, 1, 128)])
@pytest.mark.parametrize("scale", [-0.09, 0.0, 0.3])
def test_scales_of_every_prompt_form(dtype, hq, hkv, d, scale):
    p = Prompts([130, 9, 700], dtype, hq, hkv, d, seed=21)
    p.scale = scale
    p.call()
    p.check(f"scale {scale}")


def error_bound(q, k, v, scale):
    """What the roundings of a q8_0 call may move an output by, element by element, w the softmax.
    A key's elements are off by 2^-11 of themselves, so its score by e_p <= |scale| 2^-11 sum |q k|
    and the output by sum w_p e_p |v_p - o|; values and weights are off by 2^-11 each (weights below
    2^-14 of the reference by 2^-25 of it): 2 * 2^-11 sum w |v| + L 2^-25 max |v|.  A tenth covers
    the products of these, 2e-5 the fp32 sums."""
    n, hq, d = q.shape
    L, hkv, _ = k.shape
    out = torch.zeros(n, hq, d, dtype=torch.float64)
    for j in range(hq):
        qj, kj, vj = q[:, j].double(), k[:, j // (hq // hkv)].double(), v[:, j // (hq // hkv)].double()
        see = torch.arange(L) <= (L - n + torch.arange(n))[:, None]
        w = torch.softmax(torch.where(see, scale * (qj @ kj.T), -torch.inf), -1)
        e = abs(scale) * (qj.abs() @ kj.abs().T)
        spread = ((w * e)[..., None] * (vj[None] - (w @ vj)[:, None]).abs()).sum(1)
        out[:, j] = 2.0 ** -11 * (spread + 2 * (w @ vj.abs())) + L * 2.0 ** -25 * vj.abs().max()
    return 1.1 * out + 2e-5


@pytest.mark.parametrize("dtype", [wl.F16, wl.BF16])
@pytest.mark.parametrize("scale", [-0.125, 0.0, 0.4])
def test_scales_over_a_q8_0_cache(dtype, scale):
    c = Chunks([(40, 300), (1, 700), (3, 3)], dtype, seed=22)
    c.scale = scale
    got, want, q = c.call().double().cpu(), c.ref(), c.q.cpu()
    bound = torch.cat([error_bound(q[a:b], c.cache.k[s], c.cache.v[s], scale)
                       for s, (a, b) in enumerate(zip(c.qsl, c.qsl[1:]))])
    half = torch.from_numpy(0.5 * _gpu.ulp(want.numpy(), dtype))
    assert bool(((got - want).abs() <= bound + half).all())
    _gpu.assert_no_device_status()


@pytest.mark.parametrize("dtype", [wl.F16, wl.BF16])
@pytest.mark.parametrize("hq,hkv,d", [(7, 1, 64), (7, 1, 128), (32, 8, 128), (10, 2, 64), (64, 1, 64)])
def test_query_rows_of_others_do_not_reach_a_row(dtype, hq, hkv, d):
    """A query tile's rows behind its sequence hold NaN and infinity of the next one, or of no sequence."""
    lens = [50, 3, 1, 37, 300]
    p = Prompts(lens, dtype, hq, hkv, d, seed=23, first=5, behind=70)
    clean = p.call().clone()
    bad = torch.tensor([float("nan"), float("inf"), -float("inf")], dtype=p.rows.dtype, device="cuda").repeat(200)
    for s in (1, 3):
        a, b = int(p.qsl[s]), int(p.qsl[s + 1])
        p.rows[a:b] = bad[:b - a, None, None]
    p.rows[:5] = bad[:5, None, None]
    p.rows[int(p.qsl[-1]):] = bad[:70, None, None]
    got = p.call()
    torch.cuda.synchronize()
    for s in (0, 2, 4):
        a, b = int(p.qsl[s]), int(p.qsl[s + 1])
        assert torch.equal(got[a:b], clean[a:b]), f"sequence {s}"
    _gpu.assert_no_device_status()


@pytest.mark.parametrize("dtype", [wl.F16, wl.BF16])
def test_query_rows_of_others_over_a_q8_0_cache(dtype):
    c = Chunks([(20, 90), (4, 4), (5, 200), (1, 50)], dtype, seed=24, behind=40)
    clean = c.call().clone()
    c.q[20:24] = float("nan")
    c.q[30:] = float("inf")
    got = c.call()
    assert torch.equal(got[:20], clean[:20]) and torch.equal(got[24:30], clean[24:30])
    assert bool(torch.isnan(got[20:24]).all())


@pytest.mark.parametrize("d", [64, 128])
def test_rows_far_apart(d):
    """q, k and v with row strides of their own, wider than their heads."""
    p = Prompts([140, 33], wl.F16, 6, 2, d, seed=25)
    wide = torch.full((173, 6 * d + 24), float("nan"), dtype=torch.float16, device="cuda")
    wide[:, :6 * d] = p.q.reshape(173, -1)
    want = p.call().clone()
    p.out.fill_(7.0)
    p.q = wide[:, :6 * d].unflatten(1, (6, d))
    p.call()
    torch.cuda.synchronize()
    assert torch.equal(p.out, want)


@pytest.mark.parametrize("dtype,d", [(wl.F16, 64), (wl.BF16, 128)])
def test_units_without_tokens_or_keys(dtype, d):
    """Tiles that see nothing, beside and between ones that do; more units than are announced at once."""
    lens = [300, 1, 0, 280, 90, 5] * 3
    keys = [0, 1, 4, 300, 2, 700] * 3
    p = Prompts(lens, dtype, 7, 1, d, seed=26, keys=keys)
    p.call()
    p.check("tiles without keys")


def test_one_token():
    for dtype, d in ((wl.F16, 64), (wl.BF16, 64), (wl.F16, 128)):
        p = Prompts([1], dtype, 3, 1, d, seed=27)
        p.call()
        p.check("one token")
