"""The q4_0 cache on the GPU: append bit for bit, read-back, decode and span attention against fp64."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import _gpu
import _q4
import _span
from _q4 import wl
from paged_kv_decode_ns_gb300 import binding as nb

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- append, read-back
@pytest.mark.parametrize("dtype", [wl.F16, wl.BF16])
@pytest.mark.parametrize("d,bs", [(64, 4), (64, 8), (64, 16), (64, 32), (128, 16)])
@pytest.mark.parametrize("T,hkv,amp", [(1, 1, 1.0), (37, 3, 1.0), (500, 2, 100.0), (64, 2, 1e-6)])
def test_append_and_read_back(dtype, d, bs, T, hkv, amp):
    rng = np.random.default_rng(T + d)
    k, v = (_q4.to16(rng.standard_normal((T, hkv, d)).astype(np.float32) * np.float32(amp), dtype) for _ in range(2))
    k[0, 0, :32] = 0.0
    if T > 5:
        v[3, 0, 1], v[3, 0, 2] = 4000.0, -4000.0
    nbk = -(-T // bs) + 2
    slots = rng.permutation(nbk * bs)[:T].astype(np.int64)
    if T > 5:
        slots[2] = -1
    pools = [torch.full((nbk, hkv, bs, d // 2), 17, dtype=torch.uint8), torch.full((nbk, hkv, bs, d // 32), 2.0, dtype=torch.float16)] * 2
    want, dev = [p.clone() for p in pools], [p.clone().cuda() for p in pools]
    at = np.nonzero(slots >= 0)[0]
    for i, x in enumerate((k, v)):
        codes, steps = _q4.quantise(_q4.f32(x))
        want[2 * i][slots[at] // bs, :, slots[at] % bs] = torch.from_numpy(codes[at])
        want[2 * i + 1][slots[at] // bs, :, slots[at] % bs] = torch.from_numpy(steps[at])
    nb.ns_kv_append_q4_0(k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), *dev)
    for got, ref in zip(dev, want):
        assert _q4.same_bits(got, ref)
    assert _q4.status() == 0
    # every block of the pool, read back as one sequence
    tables = torch.arange(nbk, dtype=torch.int32).flip(0)[None].contiguous().cuda()
    start = torch.tensor([0, nbk * bs], dtype=torch.int32, device="cuda")
    out = [torch.empty(nbk * bs, hkv, d, dtype=k.dtype, device="cuda") for _ in range(2)]
    nb.ns_kv_gather_q4_0(*dev, tables, start, *out)
    for i in range(2):
        val = _q4.values(want[2 * i].flip(0).numpy(), want[2 * i + 1].flip(0).numpy())
        ref = _gpu.round_to_dtype(val.transpose(0, 2, 1, 3).reshape(-1, hkv, d), dtype)
        assert np.array_equal(_gpu.to_f64(out[i]), ref)
    assert _q4.status() == 0


def test_append_of_what_is_not_finite_and_of_slots_outside():
    x = torch.ones(4, 1, 64, dtype=torch.bfloat16)
    x[0, 0, 3], x[1, 0, 40], x[2, 0, 63] = float("nan"), float("inf"), -float("inf")
    pools = [torch.zeros(1, 1, 16, 32, dtype=torch.uint8), torch.zeros(1, 1, 16, 2, dtype=torch.float16)] * 2
    dev = [p.clone().cuda() for p in pools]
    nb.ns_kv_append_q4_0(x.cuda(), x.cuda(), torch.tensor([0, 1, 2, 16]).cuda(), *dev)
    assert _q4.status() == 0x4
    codes, steps = _q4.quantise(_q4.f32(x))
    for i in (0, 2):
        assert torch.equal(dev[i].cpu()[0, 0, :3], torch.from_numpy(codes[:3, 0])) and not dev[i].cpu()[0, 0, 3:].any()
        s = dev[i + 1].cpu()[0, 0, :3]
        assert torch.equal(torch.isnan(s), torch.tensor([[True, False], [False, True], [False, True]]))
        assert torch.equal(s.nan_to_num(), torch.from_numpy(steps[:3, 0]).nan_to_num())


def test_read_back_leaves_rows_behind_the_last_sequence_and_bad_blocks():
    rng = np.random.default_rng(1)
    cache = _q4.Cache(rng, [20, 0, 5])
    kc, ks, vc, vs, tables = cache.dev()
    tables[0, 1] = 1 << 20
    out = [torch.full((30, 2, 64), 9.0, dtype=torch.float16, device="cuda") for _ in range(2)]
    start = torch.tensor([2, 22, 22, 27], dtype=torch.int32, device="cuda")
    nb.ns_kv_gather_q4_0(kc, ks, vc, vs, tables, start, *out)
    assert _q4.status() == 0x1
    for got, ref in zip(out, (cache.k, cache.v)):
        got = _gpu.to_f64(got)
        assert (got[:2] == 9).all() and (got[27:] == 9).all() and (got[18:22] == 9).all()
        assert np.array_equal(got[2:18], ref[0][:16].numpy().astype(np.float16).astype(np.float64))
        assert np.array_equal(got[22:27], ref[2].numpy().astype(np.float16).astype(np.float64))


# ---------------------------------------------------------------- decode
def decode(cache, q, lens, scale, dtype, ws=None, tables=None, out=None, hkv=None):
    kc, ks, vc, vs, bt = cache.dev()
    bt = bt if tables is None else tables
    S, hq, d = q.shape
    out = torch.full((S, hq, d), 5.0, dtype=_span.TORCH[dtype], device="cuda") if out is None else out
    ws = nb.alloc_workspace(S, hq, kc.shape[1], d) if ws is None else ws
    nb.ns_paged_attn_decode_q4_0(q.cuda(), kc, ks, vc, vs, bt, torch.tensor(lens, dtype=torch.int32, device="cuda"), scale,
                                 out, ws)
    torch.cuda.synchronize()
    return out


def rows(rng, S, hq, d, dtype, amp=1.0):
    return _q4.to16(rng.standard_normal((S, hq, d)).astype(np.float32) * np.float32(amp), dtype)


def check_decode(seed, lens, hq, hkv, d, dtype, bs=16, amp=1.0, scale=None):
    rng = np.random.default_rng(seed)
    cache = _q4.Cache(rng, lens, hkv, bs, d, amp)
    q = rows(rng, len(lens), hq, d, dtype)
    scale = d ** -0.5 if scale is None else scale
    got = decode(cache, q, lens, scale, dtype)
    ref = _q4.attend_all(q, [(1, n) for n in lens], cache, scale)
    _q4.compare(got, ref.numpy(), dtype, f"{lens[:6]} {hq}/{hkv} d{d}")
    assert _q4.status() == 0
    return got


LENS = [[1], [0, 1, 2], [15, 16, 17], [31, 32, 33, 64, 65], [1, 17, 64, 200], [700], [0, 0, 0], [5000, 1, 0, 333]]


@pytest.mark.parametrize("dtype", [wl.F16, wl.BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", LENS)
def test_decode_lengths(dtype, d, lens):
    check_decode(len(lens), lens, 14, 2, d, dtype)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (3, 3), (8, 1), (9, 1), (16, 2), (20, 2), (17, 1), (64, 1), (96, 3), (5, 5)])
def test_decode_groups(d, hq, hkv):
    check_decode(hq, [77, 1, 300], hq, hkv, d, wl.F16)


@pytest.mark.parametrize("bs", [4, 8, 16, 32])
@pytest.mark.parametrize("dtype", [wl.F16, wl.BF16])
def test_decode_block_sizes(bs, dtype):
    check_decode(bs, [bs - 1, bs, bs + 1, 3 * bs + 1, 257], 14, 2, 64, dtype, bs)


@pytest.mark.parametrize("lens", [[9000] * 2, [4096] * 8, [100] * 300, [1] * 700, [0] * 513 + [40], list(range(0, 640))])
def test_decode_splits_and_batches(lens):
    """Pairs cut by many CTAs, whole ones, and more sequences than a CTA has threads."""
    check_decode(3, lens, 4, 2, 64, wl.F16)


@pytest.mark.parametrize("lens", [[12000], [3000, 2500, 10, 4000], [130] * 400])
def test_decode_splits_head_dim_128(lens):
    check_decode(4, lens, 8, 2, 128, wl.BF16)


@pytest.mark.parametrize("d,hq,hkv,length", [(64, 2, 1, 300001), (128, 9, 1, 100003)])
def test_decode_one_pair_across_every_cta(d, hq, hkv, length):
    check_decode(6, [length], hq, hkv, d, wl.F16)


@pytest.mark.parametrize("amp", [1e-4, 30.0, 3000.0])
@pytest.mark.parametrize("dtype", [wl.F16, wl.BF16])
def test_decode_size_of_the_values(amp, dtype):
    """K and V of any size (the scale keeps the scores in hand): errors relative to the values."""
    rng = np.random.default_rng(9)
    lens = [40, 700, 3]
    cache = _q4.Cache(rng, lens, 2, 16, 64, amp)
    q = rows(rng, 3, 14, 64, dtype)
    got = _gpu.to_f64(decode(cache, q, lens, 0.125 / amp, dtype))
    ref = _q4.attend_all(q, [(1, n) for n in lens], cache, 0.125 / amp).numpy()
    eps = torch.finfo(_span.TORCH[dtype]).eps / 2
    # the output's rounding (fp16: or half its least step), and a rounding of each weight by 2^-11
    assert (np.abs(got - ref) <= eps * np.abs(ref) + 2.0 ** -25 + 2.0 ** -10 * amp * 4).all()
    assert _q4.status() == 0


def test_decode_one_large_step_beside_small_ones():
    """Values 2^12 larger at one key: the others keep their weights."""
    rng = np.random.default_rng(10)
    cache = _q4.Cache(rng, [400], 1, 16, 64)
    q = rows(rng, 1, 8, 64, wl.BF16)
    blk = cache.tables[0, 399 // 16]
    cache.vs[blk, :, 399 % 16] = (cache.vs[blk, :, 399 % 16].astype(np.float32) * 4096).astype(np.float16)
    cache.v[0][399] *= 4096
    got = _gpu.to_f64(decode(cache, q, [400], 0.125, wl.BF16))
    ref = _q4.attend_all(q, [(1, 400)], cache, 0.125).numpy()
    assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -11 * float(cache.v[0][399].abs().max()) * 0.04 + 2e-3).all()


def test_decode_rising_scores_and_zero_or_negative_scale():
    rng = np.random.default_rng(11)
    lens = [600]
    cache = _q4.Cache(rng, lens, 1, 16, 64, 1.0)
    for p in range(600):  # keys that grow along the sequence move the reference again and again
        b = cache.tables[0, p // 16]
        cache.ks[b, :, p % 16] *= np.float16(1 + p / 40)
        cache.k[0][p] = torch.from_numpy(_q4.values(cache.kc[b, :, p % 16], cache.ks[b, :, p % 16]))
    q = rows(rng, 1, 7, 64, wl.F16, 2.0)
    for scale in (0.125, -0.125, 0.0, 1e-30):
        got = decode(cache, q, lens, scale, wl.F16)
        _q4.compare(got, _q4.attend_all(q, [(1, 600)], cache, scale).numpy(), wl.F16, str(scale))


def test_decode_what_no_token_fills_is_not_seen():
    """Unused slots hold NaN steps (the cache's own fill); unused table entries point anywhere."""
    rng = np.random.default_rng(12)
    lens = [33, 0, 5]
    cache = _q4.Cache(rng, lens, 2, 16, 64)
    q = rows(rng, 3, 14, 64, wl.F16)
    a = decode(cache, q, lens, 0.125, wl.F16)
    cache.tables[1] = 1 << 29
    cache.tables[2, 1:] = -7
    cache.kc[cache.tables[2, 0], :, 5:] = 0xff
    cache.vs[cache.tables[2, 0], :, 5:] = np.inf
    b = decode(cache, q, lens, 0.125, wl.F16)
    assert _q4.same_bits(a, b) and (a[1] == 0).all() and _q4.status() == 0


def test_decode_bad_blocks_and_lengths():
    rng = np.random.default_rng(13)
    lens = [100, 48, 20]
    cache = _q4.Cache(rng, lens, 2, 16, 64)
    q = rows(rng, 3, 14, 64, wl.F16)
    good = decode(cache, q, lens, 0.125, wl.F16)
    tables = torch.from_numpy(cache.tables).cuda()
    tables[0, 2], tables[1, :3] = cache.kc.shape[0], -1
    got = decode(cache, q, lens, 0.125, wl.F16, tables=tables)
    assert _q4.status() == 0x1
    keep = np.r_[0:32, 48:100]
    ref = _span.attend(q[:1], cache.k[0][keep], cache.v[0][keep], 0.125)
    _q4.compare(got[:1], ref.numpy(), wl.F16)
    assert (got[1] == 0).all() and _q4.same_bits(got[2], good[2])
    got = decode(cache, q, [-4, 48, 1 << 30], 0.125, wl.F16)
    assert _q4.status() & 0x2
    assert (got[0] == 0).all() and _q4.same_bits(got[1], good[1])


def test_decode_nan_stays_in_its_rows():
    rng = np.random.default_rng(14)
    lens = [50, 400]
    cache = _q4.Cache(rng, lens, 2, 16, 64)
    q = rows(rng, 2, 14, 64, wl.F16)
    good = decode(cache, q, lens, 0.125, wl.F16)
    q[0, 3, 5], q[1, 9, 60] = float("nan"), float("inf")
    got = decode(cache, q, lens, 0.125, wl.F16)
    assert torch.isnan(got[0, 3].float()).all() and torch.isnan(got[1, 9].float()).all()
    mask = torch.ones(2, 14, dtype=torch.bool)
    mask[0, 3] = mask[1, 9] = False
    assert _q4.same_bits(got.cpu()[mask], good.cpu()[mask])
    # a NaN step of V reaches its group of elements, one of K the whole row, of that kv head alone
    q = rows(rng, 2, 14, 64, wl.F16)
    good = decode(cache, q, lens, 0.125, wl.F16)
    cache.vs[cache.tables[0, 1], 1, 3, 0] = np.nan
    cache.ks[cache.tables[1, 2], 0, 4, 1] = np.nan
    got = decode(cache, q, lens, 0.125, wl.F16).cpu()
    assert torch.isnan(got[0, 7:, :32].float()).all() and torch.isnan(got[1, :7].float()).all()
    assert _q4.same_bits(got[0, :7], good.cpu()[0, :7])
    # the other elements' weights may be laid out for another largest step: 2^-11 of each, |v| <= 8
    assert (got[0, 7:, 32:].float() - good.cpu()[0, 7:, 32:].float()).abs().max() <= 2 * 8 * 2.0 ** -11 + 2.0 ** -9
    assert _q4.same_bits(got[1, 7:], good.cpu()[1, 7:])


def test_decode_repeats_to_the_bit_and_shares_the_16_bit_decodes_workspace():
    rng = np.random.default_rng(15)
    lens = [4000, 3, 2500, 0, 900]
    cache = _q4.Cache(rng, lens, 2, 16, 64)
    q = rows(rng, 5, 14, 64, wl.BF16)
    ws = nb.alloc_workspace(5, 14, 2, 64)
    first = decode(cache, q, lens, 0.125, wl.BF16, ws)
    st = _gpu.DevStep(wl.tiny_decode())
    want = st.decode().clone()
    ws4 = nb.alloc_workspace(8, 14, 2, 64)
    for _ in range(3):
        assert _q4.same_bits(first, decode(cache, q, lens, 0.125, wl.BF16, ws4))
        st.ws = ws4
        assert _q4.same_bits(st.decode(), want)


def test_decode_captured_replayed_and_on_another_stream():
    rng = np.random.default_rng(16)
    lens = [3000, 17, 640]
    cache = _q4.Cache(rng, lens, 2, 16, 128)
    q = rows(rng, 3, 14, 128, wl.F16)
    want = decode(cache, q, lens, 0.09, wl.F16)
    kc, ks, vc, vs, bt = cache.dev()
    qd, cl = q.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, ws = torch.zeros_like(qd), nb.alloc_workspace(3, 14, 2, 128)
    call = nb.prepare(nb.ns_paged_attn_decode_q4_0, qd, kc, ks, vc, vs, bt, cl, 0.09, out, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for _ in range(4):
            call()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert _q4.same_bits(out, want)
    out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    call(stream=side)
    side.synchronize()
    assert _q4.same_bits(out, want) and _q4.status() == 0


FIRST_CALL = """
import sys
sys.path[:0] = [%r, %r]
import numpy as np, torch
import _gpu, _q4
from paged_kv_decode_ns_gb300 import binding as nb
rng = np.random.default_rng(1)
cache = _q4.Cache(rng, [300, 5], 2, 16, 128)
q = _q4.to16(rng.standard_normal((2, 14, 128)).astype(np.float32), _q4.wl.F16)
kc, ks, vc, vs, bt = cache.dev()
qd, cl, ws = q.cuda(), _gpu.dev_ints([300, 5], np.int32), nb.alloc_workspace(2, 14, 2, 128)
out, rows = torch.zeros_like(qd), [torch.zeros(305, 2, 128, dtype=qd.dtype, device="cuda") for _ in range(2)]
start = _gpu.dev_ints([0, 300, 305], np.int32)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    nb.ns_paged_attn_decode_q4_0(qd, kc, ks, vc, vs, bt, cl, 0.1, out, ws)
    nb.ns_kv_gather_q4_0(kc, ks, vc, vs, bt, start, *rows)
graph.replay()
torch.cuda.synchronize()
_q4.compare(out, _q4.attend_all(q, [(1, 300), (1, 5)], cache, 0.1).numpy(), _q4.wl.F16)
assert np.array_equal(_gpu.to_f64(rows[0]), torch.cat(cache.k).numpy().astype(np.float16).astype(np.float64))
print("captured")
"""


def test_the_first_calls_of_a_process_are_captured():
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL % (here, os.path.dirname(here))], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


# ---------------------------------------------------------------- spans
def check_spans(seed, spans, hq, hkv, dtype, amp=1.0, d=64):
    scale = d ** -0.5  # scores of the same spread at either width, and so the same errors of the weights
    rng = np.random.default_rng(seed)
    cache = _q4.Cache(rng, [L for _, L in spans], hkv, 16, d, amp)
    T = sum(n for n, _ in spans)
    q = rows(rng, T, hq, d, dtype)
    kc, ks, vc, vs, bt = cache.dev()
    out = torch.full((T + 3, hq, d), 5.0, dtype=q.dtype, device="cuda")
    start = torch.from_numpy(_span.starts([n for n, _ in spans])).cuda()
    cl = torch.tensor([L for _, L in spans], dtype=torch.int32, device="cuda")
    padded = torch.cat((q, torch.full((3, hq, d), float("nan"), dtype=q.dtype))).cuda()
    nb.ns_paged_attn_prefill_q4_0(padded, start, kc, ks, vc, vs, bt, cl, scale, out, nb.alloc_span_workspace(d))
    assert (out[T:] == 5.0).all()  # rows behind the last sequence
    _span.compare(out[:T], _q4.attend_all(q, spans, cache, scale), dtype, str(spans[:4]), q8=True)
    assert _q4.status() == 0


SPANS = [[(1, 1)], [(1, 40), (3, 17), (16, 16)], [(5, 300), (0, 20), (130, 130)], [(64, 1000), (1, 2000)],
         [(257, 700)], [(4, 4)] * 40, [(3, 130 + i) for i in range(33)], [(300, 5000)]]


@pytest.mark.parametrize("dtype", [wl.F16, wl.BF16])
@pytest.mark.parametrize("spans", SPANS)
def test_spans(dtype, spans):
    check_spans(len(spans), spans, 14, 2, dtype)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 8), (9, 1), (32, 2), (64, 1)])
def test_span_groups(hq, hkv):
    check_spans(hq, [(9, 100), (40, 333)], hq, hkv, wl.F16)


def test_span_values_of_other_sizes():
    check_spans(5, [(20, 200), (3, 600)], 14, 2, wl.BF16, amp=0.01)


@pytest.mark.parametrize("dtype", [wl.F16, wl.BF16])
@pytest.mark.parametrize("spans", SPANS + [[(1, n) for n in (15, 16, 17, 63, 64, 65, 127, 128, 129)]])
def test_spans_head_dim_128(dtype, spans):
    check_spans(len(spans) + 50, spans, 32, 8, dtype, d=128)


@pytest.mark.parametrize("dtype", [wl.F16, wl.BF16])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 8), (9, 1), (64, 1)])
def test_span_groups_head_dim_128(hq, hkv, dtype):
    check_spans(hq + 50, [(9, 100), (40, 333)], hq, hkv, dtype, d=128)


def test_span_values_of_other_sizes_head_dim_128():
    check_spans(6, [(20, 200), (3, 600)], 14, 2, wl.BF16, amp=0.01, d=128)
    check_spans(7, [(20, 200), (3, 600)], 14, 2, wl.F16, amp=0.01, d=128)


def test_spans_bad_blocks_head_dim_128():
    # pages left out in the first key tile, in the middle and at the end of one behind it, and all of one sequence's
    rng = np.random.default_rng(71)
    cache = _q4.Cache(rng, [230, 60, 20], 2, 16, 128)
    q = rows(rng, 15, 14, 128, wl.F16)
    kc, ks, vc, vs, bt = cache.dev()
    bad = {0: [1, 5, 7], 1: [], 2: [0, 1]}
    for s, blocks in bad.items():
        for i, b in enumerate(blocks):
            bt[s, b] = (-1, kc.shape[0], 2 ** 31 - 1)[i]
    out = torch.zeros(15, 14, 128, dtype=q.dtype, device="cuda")
    nb.ns_paged_attn_prefill_q4_0(q.cuda(), torch.tensor([0, 7, 12, 15], dtype=torch.int32, device="cuda"), kc, ks, vc, vs, bt,
                                  torch.tensor([230, 60, 20], dtype=torch.int32, device="cuda"), 128 ** -0.5, out,
                                  nb.alloc_span_workspace(128))
    assert _q4.status() == 0x1
    keep = np.setdiff1d(np.arange(230), np.r_[16:32, 80:96, 112:128])
    _span.compare(out[:7], _span.attend(q[:7], cache.k[0][keep], cache.v[0][keep], 128 ** -0.5), wl.F16, q8=True)
    _span.compare(out[7:12], _span.attend(q[7:12], cache.k[1], cache.v[1], 128 ** -0.5), wl.F16, q8=True)
    assert (out[12:] == 0).all()


def test_spans_what_no_token_fills_and_bad_blocks():
    rng = np.random.default_rng(21)
    cache = _q4.Cache(rng, [100, 60], 2, 16, 64)
    q = rows(rng, 12, 14, 64, wl.F16)
    kc, ks, vc, vs, bt = cache.dev()
    start = torch.tensor([0, 7, 12], dtype=torch.int32, device="cuda")
    cl = torch.tensor([100, 60], dtype=torch.int32, device="cuda")
    out = torch.zeros(12, 14, 64, dtype=q.dtype, device="cuda")
    bt[0, 1] = -1
    nb.ns_paged_attn_prefill_q4_0(q.cuda(), start, kc, ks, vc, vs, bt, cl, 0.125, out, nb.alloc_span_workspace(64))
    assert _q4.status() == 0x1
    keep = np.r_[0:16, 32:100]
    ref = _span.attend(q[:7], cache.k[0][keep], cache.v[0][keep], 0.125)
    _span.compare(out[:7], ref, wl.F16, q8=True)
    _span.compare(out[7:], _span.attend(q[7:], cache.k[1], cache.v[1], 0.125), wl.F16, q8=True)


def test_a_span_of_one_token_and_the_decode_agree():
    rng = np.random.default_rng(22)
    lens = [40, 1, 999]
    cache = _q4.Cache(rng, lens, 2, 16, 64)
    q = rows(rng, 3, 14, 64, wl.F16)
    a = decode(cache, q, lens, 0.125, wl.F16)
    kc, ks, vc, vs, bt = cache.dev()
    out = torch.zeros_like(a)
    nb.ns_paged_attn_prefill_q4_0(q.cuda(), torch.arange(4, dtype=torch.int32, device="cuda"), kc, ks, vc, vs, bt,
                                  torch.tensor(lens, dtype=torch.int32, device="cuda"), 0.125, out, nb.alloc_span_workspace(64))
    ref = _q4.attend_all(q, [(1, n) for n in lens], cache, 0.125)
    _span.compare(out, ref, wl.F16, q8=True)
    assert (out.float() - a.float()).abs().max() < 4e-3
