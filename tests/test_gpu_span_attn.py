"""GPU parity of the span attention: whole packed prompts (ns_prompt_attn) and
new tokens over a q8_0 cache (ns_paged_attn_prefill_q8_0), against fp64.

Tolerance: that of the other attention tests (2e-3 beyond half a step of the
output type, relative L2 1e-3 against the rounded exact value).  The 16-bit steps
of the computation are worth at most this much of it at N(0, 1) inputs: a weight
p <= 1 rounded to fp16 is off by p 2^-11, so a row by sum p |v| 2^-11 / sum p <=
4.5 * 2^-11 = 2.2e-3 if every error had one sign, and by 2^-11 / sqrt(3) of its own
size (2.8e-4) as independent ones; a q8_0 value rounded to fp16 moves a score by
scale sqrt(64) 2^-11 / sqrt(3) = 2.8e-4 and an output by as much again (_span.py has
what that makes of bf16 outputs).
"""
import numpy as np
import pytest
import torch

import _gpu
import _span
from paged_kv_decode_ns_gb300 import binding as nb
from paged_kv_decode_ns_gb300 import workloads as wl

pytestmark = pytest.mark.gpu


class Prompts:
    """Packed sequences whose q, k and v are slices of one projection."""

    def __init__(self, lens, dtype, hq=14, hkv=2, d=64, seed=0, first=0, behind=0, keys=None):
        g = torch.Generator().manual_seed(seed)
        self.dtype, self.scale, self.lens, self.keys = dtype, d ** -0.5, list(lens), list(keys or lens)
        self.qsl = _span.starts(lens, first)
        self.ksl = self.qsl if keys is None else _span.starts(keys, 3)
        t = int(self.qsl[-1]) + behind
        tk = t if keys is None else int(self.ksl[-1]) + behind
        rows = torch.randn(max(t, tk), hq + 2 * hkv, d, generator=g).to(_span.TORCH[dtype])
        self.rows = rows.cuda()
        self.q, self.k, self.v = self.rows[:t, :hq], self.rows[:tk, hq:hq + hkv], self.rows[:tk, hq + hkv:]
        self.out = torch.full((t, hq, d), 7.0, dtype=rows.dtype, device="cuda")
        self.start = _gpu.dev_ints(self.qsl, np.int32)
        self.kstart = None if keys is None else _gpu.dev_ints(self.ksl, np.int32)
        self.ws = nb.alloc_span_workspace(d)

    def call(self, **kw):
        nb.ns_prompt_attn(self.q, self.k, self.v, self.start, self.scale, self.out, self.ws,
                          key_start_loc=self.kstart, **kw)
        return self.out

    def check(self, what=""):
        q, k, v = self.q.cpu(), self.k.cpu(), self.v.cpu()
        want = torch.full(tuple(self.out.shape), 7.0, dtype=torch.float64)
        for s, n in enumerate(self.lens):
            a, b, c, e = self.qsl[s], self.qsl[s + 1], self.ksl[s], self.ksl[s + 1]
            want[a:b] = _span.attend(q[a:b], k[c:e], v[c:e], self.scale)
        torch.cuda.synchronize()
        _gpu.assert_no_device_status()
        outside = torch.ones(self.out.shape[0], dtype=torch.bool)
        outside[self.qsl[0]:self.qsl[-1]] = False
        assert bool((self.out.cpu()[outside] == 7.0).all()), "rows of no sequence were written"
        inside = ~outside
        if inside.any():
            _span.compare(self.out[inside.cuda()], want[inside], self.dtype, what)


RAGGED = [1, 0, 17, 127, 128, 129, 2, 300, 0, 64, 255, 257]


@pytest.mark.parametrize("dtype", [wl.F16, wl.BF16])
@pytest.mark.parametrize("hq,hkv,d", [(14, 2, 64), (8, 8, 64), (6, 2, 64), (5, 1, 64), (32, 2, 64), (9, 1, 64),
                                      (64, 1, 64), (32, 8, 128), (7, 1, 128), (2, 2, 128)])
def test_packed_prompts(dtype, hq, hkv, d):
    p = Prompts(RAGGED, dtype, hq, hkv, d, seed=hq * d, first=2, behind=5)
    p.call()
    p.check(f"{dtype} {hq}/{hkv}/{d}")


@pytest.mark.parametrize("dtype,d", [(wl.F16, 64), (wl.BF16, 64), (wl.BF16, 128)])
def test_long_and_short_prompts_together(dtype, d):
    """One prompt is cut across many CTAs, the others are whole."""
    p = Prompts([2500, 3, 700, 1, 33], dtype, 4, 2, d, seed=3)
    p.call()
    p.check("long")


@pytest.mark.parametrize("dtype", [wl.F16, wl.BF16])
@pytest.mark.parametrize("lens,keys", [([5, 1, 40, 130], [300, 1000, 2100, 131]),
                                       ([20, 4, 150, 3, 0], [7, 0, 140, 3, 9]),   # rows that see nothing
                                       ([1] * 9, [0, 1, 2, 127, 128, 129, 500, 4, 1])])
def test_keys_of_their_own(dtype, lens, keys):
    p = Prompts(lens, dtype, 14, 2, 64, seed=11, keys=keys, behind=4)
    p.call()
    p.check("own keys")


@pytest.mark.parametrize("scale", [-0.125, 0.0, 1.0])
def test_scales(scale):
    p = Prompts([130, 9], wl.F16, 4, 2, 64, seed=5)
    p.scale = scale
    p.call()
    p.check(f"scale {scale}")


@pytest.mark.parametrize("dtype", [wl.F16, wl.BF16])
def test_other_sequences_do_not_reach_a_row(dtype):
    """NaN and infinity in one sequence, and in the rows of none, stay there."""
    p = Prompts([100, 60, 90], dtype, 14, 2, 64, seed=6, first=7, behind=200)
    bad = torch.tensor([float("nan"), float("inf"), -float("inf")], dtype=p.rows.dtype, device="cuda").repeat(200)
    clean = p.call().clone()
    a, b = int(p.qsl[1]), int(p.qsl[2])
    for rows in (p.rows[a:b], p.rows[:7], p.rows[int(p.qsl[3]):]):
        rows.copy_(bad[:rows.shape[0], None, None].expand_as(rows))
    p.call()
    torch.cuda.synchronize()
    keep = torch.ones(p.out.shape[0], dtype=torch.bool, device="cuda")
    keep[a:b] = False
    assert torch.equal(p.out[keep], clean[keep])
    _gpu.assert_no_device_status()


@pytest.mark.parametrize("amp", [2.0 ** -60, 2.0 ** -20, 2.0 ** 14, 2.0 ** 60])
def test_bf16_values_of_any_size(amp):
    """bf16 reaches far beyond fp16: tiny and huge values keep their relative precision."""
    p = Prompts([300, 20], wl.BF16, 4, 2, 64, seed=8)
    p.v.mul_(amp)
    got = p.call().double().cpu() / amp
    for s, (a, b) in enumerate(zip(p.qsl, p.qsl[1:])):
        want = _span.attend(p.q[a:b].cpu(), p.k[a:b].cpu(), p.v[a:b].cpu().double() / amp, p.scale)
        assert float((got[a:b] - want).norm() / want.norm()) < 2.0 ** -8 / 3 ** 0.5 + 1e-3
    _gpu.assert_no_device_status()


def test_bf16_values_of_mixed_size():
    """Stretches of a prompt whose values differ by 2^40, a stretch of zeros among them."""
    p = Prompts([900], wl.BF16, 2, 1, 64, seed=9)
    factor = torch.ones(900, device="cuda")
    factor[:256], factor[256:420], factor[420:700] = 2.0 ** -20, 0.0, 2.0 ** 20
    p.v.mul_(factor[:, None, None])
    got = p.call().double().cpu()
    want = _span.attend(p.q.cpu(), p.k.cpu(), p.v.cpu(), p.scale)
    err = (got - want).norm(dim=-1) / want.norm(dim=-1)
    assert float(err.max()) < 2.0 ** -8 + 4e-3  # a half step of each element, and sum p |v| 2^-11 / |o| over few keys
    _gpu.assert_no_device_status()


def test_values_that_vanish_beside_others_still_count_in_the_sum():
    """Stretches of 2^-60, of zeros and of 2^60 in one prompt: the small ones add nothing
    to a row that sees the large ones, but their weights divide it."""
    p = Prompts([900], wl.BF16, 2, 1, 64, seed=19)
    factor = torch.ones(900, device="cuda")
    factor[:256], factor[256:420], factor[420:700] = 2.0 ** -60, 0.0, 2.0 ** 60
    p.v.mul_(factor[:, None, None])
    got = p.call().double().cpu()
    want = _span.attend(p.q.cpu(), p.k.cpu(), p.v.cpu(), p.scale)
    err = (got - want).norm(dim=-1) / want.norm(dim=-1)
    assert float(err.max()) < 2.0 ** -8 + 4e-3  # as above
    _gpu.assert_no_device_status()


def test_large_scores():
    """Scores far apart: the running maximum moves by hundreds within a row."""
    p = Prompts([700, 128], wl.F16, 4, 2, 64, seed=10)
    p.q.mul_(16.0)
    p.call()
    p.check("large scores")


class Chunks:
    """Spans of n new tokens over caches of L tokens (with them) in a q8_0 pool."""

    def __init__(self, spans, dtype, hq=14, hkv=2, seed=0, behind=0, amp=1.0):
        rng = np.random.default_rng(seed)
        self.spans, self.dtype, self.scale = spans, dtype, 0.125
        self.cache = _span.Q8Cache(rng, [L for _, L in spans], hkv, amp=amp)
        self.qsl = _span.starts([n for n, _ in spans])
        t = int(self.qsl[-1]) + behind
        self.q = torch.from_numpy(rng.standard_normal((t, hq, 64)).astype(np.float32)).to(_span.TORCH[dtype]).cuda()
        self.out = torch.full_like(self.q, 7.0)
        self.pools = self.cache.dev()
        self.start = _gpu.dev_ints(self.qsl, np.int32)
        self.lens = _gpu.dev_ints([L for _, L in spans], np.int32)
        self.ws = nb.alloc_span_workspace(64)

    def call(self, **kw):
        nb.ns_paged_attn_prefill_q8_0(self.q, self.start, *self.pools[:4], self.pools[4], self.lens, self.scale,
                                      self.out, self.ws, **kw)
        return self.out

    def ref(self):
        want = torch.full(tuple(self.out.shape), 7.0, dtype=torch.float64)
        q = self.q.cpu()
        for s, (a, b) in enumerate(zip(self.qsl, self.qsl[1:])):
            want[a:b] = _span.attend(q[a:b], self.cache.k[s], self.cache.v[s], self.scale)
        return want

    def check(self, what=""):
        torch.cuda.synchronize()
        _gpu.assert_no_device_status()
        end = int(self.qsl[-1])
        assert bool((self.out[end:] == 7.0).all())
        _span.compare(self.out[:end], self.ref()[:end], self.dtype, what, q8=True)


SPANS = [(1, 1), (1, 500), (5, 5), (0, 40), (8, 300), (33, 129), (200, 456), (1, 16), (3, 17), (2, 128), (130, 130)]


@pytest.mark.parametrize("dtype", [wl.F16, wl.BF16])
@pytest.mark.parametrize("hq,hkv", [(14, 2), (8, 8), (5, 1), (32, 2), (18, 2)])
def test_spans_over_a_q8_0_cache(dtype, hq, hkv):
    c = Chunks(SPANS, dtype, hq, hkv, seed=hq, behind=3)
    c.call()
    c.check(f"{dtype} {hq}/{hkv}")


@pytest.mark.parametrize("dtype", [wl.F16, wl.BF16])
def test_q8_0_chunk_far_into_a_context(dtype):
    c = Chunks([(90, 4000), (1, 4096), (4, 2500)], dtype, seed=2)
    c.call()
    c.check("far")


@pytest.mark.parametrize("amp", [1e-4, 30.0, 400.0])
def test_q8_0_values_of_any_size(amp):
    """Scales near both ends of fp16; large keys make the softmax pick one key, so
    the queries shrink with them."""
    c = Chunks([(40, 200), (1, 33)], wl.BF16, seed=4, amp=amp)
    c.q.mul_(min(1.0, 1.0 / amp))
    got, want = c.call().double().cpu(), c.ref()
    assert float((got - want).norm() / want.norm()) < 2.0 ** -8 / 3 ** 0.5 + 1e-3
    _gpu.assert_no_device_status()


def test_q8_0_single_tokens_equal_the_decode():
    """Spans of one token are a decode step."""
    c = Chunks([(1, L) for L in (1, 17, 64, 200, 333)], wl.F16, seed=5)
    c.call()
    c.check("single")
    out = torch.empty_like(c.q)
    nb.ns_paged_attn_decode_q8_0(c.q, *c.pools[:4], c.pools[4], c.lens, c.scale, out,
                                 nb.alloc_workspace(5, 14, 2))
    # both are within the tolerance of the exact value
    assert float((out.float() - c.out.float()).abs().max()) <= 2 * _gpu.MAX_ABS + 2.0 ** -10


def test_same_bits_every_time_captured_and_on_two_streams():
    """No result depends on the order in which CTAs finish; a captured call replays it."""
    p, c = Prompts([900, 77, 1], wl.BF16, seed=12), Chunks([(300, 900), (1, 700)], wl.F16, seed=13)
    a, b = p.call().clone(), c.call().clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    p.out.fill_(0)
    c.out.fill_(0)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        p.call()
    c.call(stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert torch.equal(p.out, a) and torch.equal(c.out, b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.call()
        c.call()
    for _ in range(3):
        p.out.fill_(0)
        c.out.fill_(0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(p.out, a) and torch.equal(c.out, b)
    _gpu.assert_no_device_status()


def test_prepared_calls():
    p = Prompts([100, 5], wl.F16, seed=14)
    want = p.call().clone()
    run = nb.prepare(nb.ns_prompt_attn, p.q, p.k, p.v, p.start, p.scale, p.out, p.ws)
    p.out.fill_(0)
    run()
    torch.cuda.synchronize()
    assert torch.equal(p.out, want)


def test_bad_device_data_is_skipped_and_reported():
    """Spans and lengths that do not fit are left out, every other sequence is right."""
    c = Chunks([(4, 40), (9, 60), (3, 30)], wl.F16, seed=15)
    c.lens[1] = 8  # shorter than its span
    c.call()
    torch.cuda.synchronize()
    assert nb.ns_get_device_status() == 0x20
    c.lens[1] = c.pools[4].shape[1] * 16 + 1
    c.call()
    torch.cuda.synchronize()
    assert nb.ns_get_device_status() == 0x2
    ref, a, b = c.ref(), int(c.qsl[1]), int(c.qsl[2])
    assert bool((c.out[a:b] == 7.0).all())
    for lo, hi in ((0, a), (b, int(c.qsl[3]))):
        _span.compare(c.out[lo:hi], ref[lo:hi], wl.F16, "neighbours")
    c.lens[1] = 60
    for bad in (-5, c.pools[0].shape[0], 1 << 30):
        c.pools[4][1, 2] = bad
        c.call()
        torch.cuda.synchronize()
        assert nb.ns_get_device_status() == 0x1
        assert bool(torch.isfinite(c.out.float()).all())

    p = Prompts([10, 20, 30], wl.F16, seed=16)
    for i, value in ((3, 61), (1, -1), (1, 40)):
        p.start.copy_(_gpu.dev_ints(p.qsl, np.int32))
        p.start[i] = value
        p.out.fill_(7.0)
        p.call()
        torch.cuda.synchronize()
        assert nb.ns_get_device_status() == 0x20


def test_refusals():
    p = Prompts([10, 20], wl.F16, seed=17)
    with pytest.raises(nb.NsError) as e:
        nb.ns_prompt_attn(p.q, p.k, p.v, p.start, p.scale, p.out, p.ws[:100])
    assert e.value.status == -1
    with pytest.raises(nb.NsError) as e:
        nb.ns_prompt_attn(p.q, p.k, p.v, p.start, float("nan"), p.out, p.ws)
    assert e.value.status == -1
    with pytest.raises(ValueError):  # keys without their own starts must be the queries' rows
        nb.ns_prompt_attn(p.q, p.k[:20], p.v[:20], p.start, p.scale, p.out, p.ws)
    with pytest.raises(TypeError):
        nb.ns_prompt_attn(p.q, p.k.bfloat16(), p.v, p.start, p.scale, p.out, p.ws)
    with pytest.raises(ValueError):  # heads that are not dense within a row
        wide = torch.empty(30, 14, 128, dtype=torch.float16, device="cuda")[:, :, :64]
        nb.ns_prompt_attn(wide, p.k, p.v, p.start, p.scale, p.out, p.ws)
    torch.cuda.synchronize()
    assert bool((p.out == 7.0).all())
