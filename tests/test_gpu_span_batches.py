"""GPU: the span attention in batches of many sequences (more than one warp plans),
NaN in single rows, and captured calls side by side; the verification around the
batch sizes at which it takes fewer CTAs a sequence.  Tolerances are those of the
single calls' tests."""
import numpy as np
import pytest
import torch

import _gpu
import _span
from paged_kv_decode_ns_gb300 import binding as nb
from paged_kv_decode_ns_gb300 import workloads as wl
from test_gpu_span_attn import Chunks, Prompts
from test_gpu_verify_drafts import Drafts

pytestmark = pytest.mark.gpu


def ragged(n, seed, most=70, long=()):
    lens = np.random.default_rng(seed).integers(0, most, n).tolist()
    for i, x in long:
        lens[i] = x
    return lens


@pytest.mark.parametrize("dtype,hq,hkv,d", [(wl.F16, 4, 2, 64), (wl.BF16, 14, 2, 64), (wl.BF16, 4, 1, 128)])
@pytest.mark.parametrize("n,long", [(32, ((0, 1100),)), (33, ((32, 1500),)), (40, ()), (512, ((511, 700), (3, 900))),
                                    (513, ((500, 2100),)), (700, ((699, 300),))])
def test_prompts_of_many_sequences(dtype, hq, hkv, d, n, long):
    p = Prompts(ragged(n, n, long=long), dtype, hq, hkv, d, seed=n, first=1, behind=3)
    p.call()
    p.check(f"{n} sequences")


@pytest.mark.parametrize("n", [45, 600])
def test_keys_of_their_own_in_many_sequences(n):
    lens, keys = ragged(n, 1, 20), ragged(n, 2, 200, ((n - 2, 2000),))
    p = Prompts(lens, wl.BF16, 14, 2, 64, seed=n, keys=keys)
    p.call()
    p.check("own keys")


@pytest.mark.parametrize("dtype", [wl.F16, wl.BF16])
@pytest.mark.parametrize("n", [33, 200, 600])
def test_q8_0_spans_of_many_sequences(dtype, n):
    new, old = ragged(n, n, 12), ragged(n, n + 1, 150, ((n // 2, 1800),))
    c = Chunks([(a, max(1, a + b)) for a, b in zip(new, old)], dtype, seed=n, behind=2)
    c.call()
    c.check(f"{n} sequences")


def test_bad_entries_among_many_sequences():
    p = Prompts([5] * 600, wl.F16, 4, 2, 64, seed=3)
    clean = p.call().clone()
    p.start[300] = 2000  # sequence 299 ends behind 300's end: 300 is out of order, 299 sees others' rows
    p.out.fill_(7.0)
    p.call()
    torch.cuda.synchronize()
    assert nb.ns_get_device_status() == 0x20
    keep = torch.ones(3000, dtype=torch.bool, device="cuda")
    keep[299 * 5:2000] = False
    assert torch.equal(p.out[keep], clean[keep])

    c = Chunks([(2, 30)] * 100, wl.F16, seed=4)
    clean = c.call().clone()
    c.lens[70] = 1  # shorter than its span
    c.out.fill_(7.0)
    c.call()
    torch.cuda.synchronize()
    assert nb.ns_get_device_status() == 0x20
    assert bool((c.out[140:142] == 7.0).all())
    keep = torch.ones(200, dtype=torch.bool, device="cuda")
    keep[140:142] = False
    assert torch.equal(c.out[keep], clean[keep])


@pytest.mark.parametrize("dtype", [wl.F16, wl.BF16])
@pytest.mark.parametrize("lens", [[300, 20], [2500, 40]])  # whole units; units cut and joined
def test_nan_in_one_query_or_key_shows_where_it_is_seen(dtype, lens):
    p = Prompts(lens, dtype, 4, 2, 64, seed=5)
    clean = p.call().clone()
    row = lens[0] - 33
    p.q[row, 1, 7] = float("nan")
    got = p.call()
    assert bool(torch.isnan(got[row, 1]).all())
    keep = torch.ones(got.shape[:2], dtype=torch.bool, device="cuda")
    keep[row, 1] = False
    assert torch.equal(got[keep], clean[keep])
    p.q[row, 1, 7] = 0.5
    p.k[row, 0, 3] = float("nan")  # kv head 0: query heads 0 and 1, of this row and the later ones
    got = p.call()
    assert bool(torch.isnan(got[row:lens[0], :2]).all())
    assert torch.equal(got[:row], clean[:row]) and torch.equal(got[lens[0]:], clean[lens[0]:])
    assert torch.equal(got[row + 1:, 2:], clean[row + 1:, 2:])
    _gpu.assert_no_device_status()


def test_nan_in_one_query_over_a_q8_0_cache():
    for dtype in (wl.F16, wl.BF16):
        c = Chunks([(40, 900), (3, 50)], dtype, seed=6)
        clean = c.call().clone()
        c.q[17, 3, 5] = float("nan")
        got = c.call()
        assert bool(torch.isnan(got[17, 3]).all())
        keep = torch.ones(got.shape[:2], dtype=torch.bool, device="cuda")
        keep[17, 3] = False
        assert torch.equal(got[keep], clean[keep])


def test_two_captured_graphs_at_once():
    """Graphs with a workspace each replay side by side on two streams."""
    p, c = Prompts([1700, 300], wl.BF16, 4, 2, 64, seed=7), Chunks([(200, 3000), (1, 90)], wl.F16, seed=8)
    want = [p.call().clone(), c.call().clone()]
    graphs = []
    for call in (p.call, c.call):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    p.out.fill_(0)
    c.out.fill_(0)
    torch.cuda.synchronize()
    for _ in range(4):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(p.out, want[0]) and torch.equal(c.out, want[1])
    _gpu.assert_no_device_status()


def test_prepared_calls_of_the_other_entry_points():
    c = Chunks([(3, 70), (1, 9)], wl.F16, seed=9)
    want = c.call().clone()
    run = nb.prepare(nb.ns_paged_attn_prefill_q8_0, c.q, c.start, *c.pools[:4], c.pools[4], c.lens, c.scale, c.out, c.ws)
    c.out.fill_(0)
    run()
    torch.cuda.synchronize()
    assert torch.equal(c.out, want)

    start = _gpu.dev_ints(_span.starts([70, 9]), np.int32)
    rows = [torch.zeros(79, 2, 64, dtype=torch.float16, device="cuda") for _ in range(4)]
    nb.ns_kv_gather_q8_0(*c.pools[:4], c.pools[4], start, *rows[:2])
    nb.prepare(nb.ns_kv_gather_q8_0, *c.pools[:4], c.pools[4], start, *rows[2:])()
    torch.cuda.synchronize()
    assert torch.equal(rows[0], rows[2]) and torch.equal(rows[1], rows[3]) and bool((rows[0] != 0).any())

    d = Drafts([2, 3, 0], 100, seed=10)
    dev = d.dev()
    out = [torch.full((8,), -9, dtype=torch.int32, device="cuda") for _ in range(2)]
    num = [torch.full((3,), -9, dtype=torch.int32, device="cuda") for _ in range(2)]
    nb.ns_verify_drafts(*dev, out[0], num[0])
    nb.prepare(nb.ns_verify_drafts, *dev, out[1], num[1])()
    torch.cuda.synchronize()
    assert torch.equal(out[0], out[1]) and torch.equal(num[0], num[1])


@pytest.mark.parametrize("n", [1, 37, 38, 39, 75, 76, 77, 151, 152, 153, 305])
@pytest.mark.parametrize("certain", [False, True])
def test_verify_at_any_batch_size(n, certain):
    counts = np.random.default_rng(n).integers(0, 5, n).tolist()
    Drafts(counts, 700, certain, seed=n).check()


def test_verify_stretches_without_weight():
    """Most of the vocabulary has probability 0, whole stretches of it: the drawn token has not."""
    for n in (3, 100, 400):
        d = Drafts([1] * n, 9001, seed=n)
        keep = np.zeros(9001, bool)
        keep[[0, 17, 4096, 8999, 9000]] = True
        for a in (d.p, d.q):
            a[:, ~keep] = 0
        d.drafts[:] = np.array([0, 17, 4096, 8999, 9000])[np.arange(n) % 5]
        d.check()
