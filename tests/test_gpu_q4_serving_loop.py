"""GPU: the calls of a serving loop over a q4_0 cache as they are used.  Prompts are rotated,
appended and attended from the rotated rows; decode steps rotate, append and attend over the
cache, with a padded batch; drafted tokens go through the span call; the cache is read back and
serves as the prefix of a new prompt.  Every step against fp64.  Then the same calls captured
behind one another, and behind a call that outlasts its set-up."""
import numpy as np
import pytest
import torch

import _gpu
import _q4
import _span
from _q4 import wl
from paged_kv_decode_ns_gb300 import binding as nb

pytestmark = pytest.mark.gpu

BS = 16


class Server:
    def __init__(self, dtype, hq, hkv, d, rotary, interleaved, lens, room=24, seed=3):
        self.rng, self.g = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
        self.dtype, self.td, self.hq, self.hkv, self.d, self.il = dtype, _span.TORCH[dtype], hq, hkv, d, interleaved
        self.scale = d ** -0.5
        S = len(lens)
        self.ctx = np.zeros(S, int)
        self.tables = self.rng.permutation(S * room).reshape(S, room).astype(np.int32)
        self.bt = _gpu.dev_ints(self.tables, np.int32)
        self.angles = _q4.table(room * BS, rotary)
        self.cos_sin = torch.from_numpy(self.angles).cuda()
        shape = (S * room, hkv, BS)
        self.pools = [t for _ in range(2) for t in (torch.full((*shape, d // 2), 0x3c, dtype=torch.uint8, device="cuda"),
                                                    torch.full((*shape, d // 32), float("nan"), dtype=torch.float16, device="cuda"))]
        self.held = [[torch.zeros(0, hkv, d, dtype=torch.float64) for _ in range(S)] for _ in range(2)]
        self.ws, self.sws = nb.alloc_workspace(64, hq, hkv, d), nb.alloc_span_workspace(d)

    def step(self, counts, pad=0, k_out=False):
        """New tokens of each sequence: rotated, appended; (q_out, k_out, v, exact q, exact k) without the padding."""
        counts = np.asarray(counts)
        T = int(counts.sum())
        pos = np.concatenate([np.arange(c, c + n) for c, n in zip(self.ctx, counts)]).astype(np.int32)
        seq = np.repeat(np.arange(len(counts)), counts)
        slots = self.tables[seq, pos // BS].astype(np.int64) * BS + pos % BS
        rows = torch.randn(T + pad, self.hq + 2 * self.hkv, self.d, generator=self.g).to(self.td).cuda()
        q, k, v = rows[:, :self.hq], rows[:, self.hq:self.hq + self.hkv], rows[:, self.hq + self.hkv:]
        qo = torch.full((T + pad, self.hq, self.d), 9.0, dtype=self.td, device="cuda")
        ko = torch.full((T + pad, self.hkv, self.d), 9.0, dtype=self.td, device="cuda") if k_out else None
        nb.ns_rope_kv_append_q4_0(q, k, v, _gpu.dev_ints(np.r_[pos, np.zeros(pad)], np.int32), self.cos_sin,
                                  _gpu.dev_ints(np.r_[slots, np.full(pad, -1)], np.int64), qo, *self.pools, k_out=ko,
                                  interleaved=self.il)
        assert (qo[T:] == 9.0).all()
        turned = [_q4.rotate(_q4.f32(x[:T]), self.angles, pos, self.il) for x in (q, k)]
        for x, side in ((turned[1], self.held[0]), (_q4.f32(v[:T]), self.held[1])):
            vals = torch.from_numpy(_q4.values(*_q4.quantise(x)))
            for s in range(len(counts)):
                side[s] = torch.cat([side[s], vals[seq == s]])
        self.ctx = self.ctx + counts
        return qo[:T], (None if ko is None else ko[:T]), v[:T]

    def lens(self):
        return _gpu.dev_ints(self.ctx, np.int32)

    def exact(self, q, counts):
        qsl = _span.starts(counts)
        return torch.cat([_span.attend(q[a:b].cpu(), self.held[0][s][:self.ctx[s]], self.held[1][s][:self.ctx[s]], self.scale)
                          for s, (a, b) in enumerate(zip(qsl, qsl[1:]))])

    def decode(self, q):
        out = torch.empty_like(q)
        nb.ns_paged_attn_decode_q4_0(q, *self.pools, self.bt, self.lens(), self.scale, out, self.ws)
        return out


@pytest.mark.parametrize("dtype", [wl.F16, wl.BF16])
@pytest.mark.parametrize("hq,hkv,d,rotary,interleaved", [(14, 2, 64, 64, False), (9, 1, 64, 32, True), (32, 8, 128, 128, False),
                                                         (20, 2, 128, 64, True)])
def test_prompts_steps_drafts_and_read_back(dtype, hq, hkv, d, rotary, interleaved):
    lens = np.array([37, 200, 1, 130])
    sv = Server(dtype, hq, hkv, d, rotary, interleaved, lens)
    # prompts attend from the rotated rows
    q, k, v = sv.step(lens, k_out=True)
    qsl = _span.starts(lens)
    out = torch.empty_like(q)
    nb.ns_prompt_attn(q, k, v, _gpu.dev_ints(qsl, np.int32), sv.scale, out, sv.sws)
    ref = torch.cat([_span.attend(q[a:b].cpu(), k[a:b].cpu(), v[a:b].cpu(), sv.scale) for a, b in zip(qsl, qsl[1:])])
    _span.compare(out, ref, dtype, "prompts")
    # decode steps, a padded batch
    for i in range(3):
        q, _, _ = sv.step([1, 1, 1, 1], pad=i)
        _q4.compare(sv.decode(q), sv.exact(q, [1] * 4).numpy(), dtype, f"step {i}")
    # drafted tokens; some are dropped, and their places taken again
    for i in range(2):
        counts = [4, 1, 6, 3]
        q, _, _ = sv.step(counts)
        out = torch.empty_like(q)
        nb.ns_paged_attn_prefill_q4_0(q, _gpu.dev_ints(_span.starts(counts), np.int32), *sv.pools, sv.bt, sv.lens(),
                                      sv.scale, out, sv.sws)
        _span.compare(out, sv.exact(q, counts), dtype, f"drafts {i}", q8=True)
        sv.ctx = sv.ctx - np.array([2, 0, 5, 1])
        for side in sv.held:
            for s in range(4):
                side[s] = side[s][:sv.ctx[s]]
    # read back, as the prefix of a new prompt
    ksl = _span.starts(sv.ctx)
    kr = torch.empty(int(ksl[-1]), hkv, d, dtype=sv.td, device="cuda")
    vr = torch.empty_like(kr)
    nb.ns_kv_gather_q4_0(*sv.pools, sv.bt, _gpu.dev_ints(ksl, np.int32), kr, vr)
    for got, side in ((kr, sv.held[0]), (vr, sv.held[1])):
        assert np.array_equal(_gpu.to_f64(got), _gpu.round_to_dtype(torch.cat(side).numpy(), dtype))
    new = np.array([9, 1, 30, 4])
    before = sv.ctx.copy()
    q, k, v = sv.step(new, k_out=True)
    qsl, full = _span.starts(new), _span.starts(before + new)
    ks, vs = (torch.cat([t for s in range(4) for t in (r[ksl[s]:ksl[s + 1]], x[qsl[s]:qsl[s + 1]])]) for r, x in ((kr, k), (vr, v)))
    out = torch.empty_like(q)
    nb.ns_prompt_attn(q, ks, vs, _gpu.dev_ints(qsl, np.int32), sv.scale, out, sv.sws, key_start_loc=_gpu.dev_ints(full, np.int32))
    ref = torch.cat([_span.attend(q[qsl[s]:qsl[s + 1]].cpu(), ks[full[s]:full[s + 1]].cpu(), vs[full[s]:full[s + 1]].cpu(), sv.scale)
                     for s in range(4)])
    _span.compare(out, ref, dtype, "prefix")
    _gpu.assert_no_device_status()


class Chain:
    """A decode step (rotation and append, then attention) and a read-back, on the buffers of one captured graph."""

    def __init__(self, d, dtype=wl.F16):
        hq, hkv = 14, 2
        self.sv = sv = Server(dtype, hq, hkv, d, d, False, [0] * 6, seed=d)
        sv.step([300, 17, 1, 64, 250, 33])
        self.counts = sv.ctx.copy()
        S = 6
        pos = self.counts.astype(np.int32)
        slots = sv.tables[np.arange(S), pos // BS].astype(np.int64) * BS + pos % BS
        self.new = torch.randn(S, hq + 2 * hkv, d, generator=sv.g).to(sv.td).cuda()
        self.rows = torch.zeros_like(self.new)
        self.pos, self.slots = torch.zeros(S, dtype=torch.int32, device="cuda"), torch.zeros(S, dtype=torch.int64, device="cuda")
        self.lens = torch.zeros(S, dtype=torch.int32, device="cuda")
        self.src = [self.new, _gpu.dev_ints(pos, np.int32), _gpu.dev_ints(slots, np.int64), _gpu.dev_ints(self.counts + 1, np.int32)]
        self.q = torch.zeros(S, hq, d, dtype=sv.td, device="cuda")
        self.out = torch.zeros_like(self.q)
        self.start = _gpu.dev_ints(_span.starts(self.counts + 1), np.int32)
        self.back = [torch.zeros(int(self.counts.sum()) + S, hkv, d, dtype=sv.td, device="cuda") for _ in range(2)]
        self.clean = [p.clone() for p in sv.pools]

    def copies(self):  # what a serving loop uploads
        for dst, src in zip((self.rows, self.pos, self.slots, self.lens), self.src):
            dst.copy_(src)

    def append(self):
        r, sv = self.rows, self.sv
        nb.ns_rope_kv_append_q4_0(r[:, :14], r[:, 14:16], r[:, 16:], self.pos, sv.cos_sin, self.slots, self.q, *sv.pools)

    def attend(self):
        nb.ns_paged_attn_decode_q4_0(self.q, *self.sv.pools, self.sv.bt, self.lens, self.sv.scale, self.out, self.sv.ws)

    def gather(self):
        nb.ns_kv_gather_q4_0(*self.sv.pools, self.sv.bt, self.start, *self.back)

    def reset(self):
        for t in (self.rows, self.pos, self.slots, self.lens, self.q, self.out, *self.back):
            t.zero_()
        for p, c in zip(self.sv.pools, self.clean):
            p.copy_(c)
        torch.cuda.synchronize()

    def results(self):
        torch.cuda.synchronize()
        return [t.clone() for t in (self.q, self.out, *self.back, *self.sv.pools)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("captured", [False, True])
def test_order_of_copies_append_attention_and_read_back(d, captured):
    c = Chain(d)
    steps = [c.copies, c.append, c.attend, c.gather]
    c.reset()
    for f in steps:
        f()
        torch.cuda.synchronize()
    want = c.results()

    def run():
        for f in steps:
            f()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        run = graph.replay
    for _ in range(5):
        c.reset()
        run()
        for a, b in zip(c.results(), want):
            assert _q4.same_bits(a, b)
    assert _q4.status() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_span_calls_captured_replayed_and_on_another_stream(d):
    """The rotation of drafted tokens and their attention, twice on one workspace, in a graph and on a stream."""
    c = Chain(d)
    c.copies()
    c.append()
    start = torch.arange(7, dtype=torch.int32, device="cuda")
    outs = [torch.zeros_like(c.q) for _ in range(2)]

    def run():
        c.append()
        for out in outs:
            nb.ns_paged_attn_prefill_q4_0(c.q, start, *c.sv.pools, c.sv.bt, c.lens, c.sv.scale, out, c.sv.sws)
    run()
    torch.cuda.synchronize()
    want = outs[0].clone()
    assert (want != 0).any() and _q4.same_bits(outs[1], want)
    c.attend()
    # the decode's output: four roundings to fp16 (V, the weights, and scores of keys there; w dv here), 2^-11 of a
    # value below 4.5 each, and the two outputs', 2^-10 each below 4
    assert (want.float() - c.out.float()).abs().max() < 4 * 4.5 * 2 ** -11 + 2 * 2 ** -10
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    side = torch.cuda.Stream()
    for again in (graph.replay, graph.replay, run):
        for out in outs:
            out.zero_()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            again()
        torch.cuda.synchronize()
        assert _q4.same_bits(outs[0], want) and _q4.same_bits(outs[1], want)
    assert _q4.status() == 0


def test_calls_behind_a_long_walk_wait_for_what_they_share():
    """A prefill whose single-token row outlasts its chunk, then a rotation in place of its output and a
    q4_0 decode that reads that: the results are those with a synchronisation between the calls."""
    from test_gpu_stream_order import Prefill
    pre = Prefill()
    c = Chain(64)
    c.copies()
    c.append()
    angles = torch.from_numpy(_q4.table(10, 64)).cuda()
    pos, slots = torch.arange(3, dtype=torch.int32, device="cuda"), torch.arange(3, device="cuda")
    pool = [torch.zeros(1, 2, 16, 64, dtype=torch.float16, device="cuda") for _ in range(2)]
    bt, lens = c.sv.bt[:3].contiguous(), _gpu.dev_ints([200, 17, 1], np.int32)
    out = torch.zeros_like(pre.out)
    k, v = (torch.randn(3, 2, 64, generator=torch.Generator().manual_seed(8 + i)).half().cuda() for i in range(2))

    def run(sync):
        pre.call()
        sync()
        nb.ns_rope_kv_append(pre.out, k, v, pos, angles, slots, pre.out, *pool)
        sync()
        nb.ns_paged_attn_decode_q4_0(pre.out, *c.sv.pools, bt, lens, 0.125, out, c.sv.ws)
        sync()
    results = []
    for sync in (torch.cuda.synchronize, lambda: None, lambda: None):
        pre.reset()
        out.zero_()
        run(sync)
        torch.cuda.synchronize()
        results.append([t.clone() for t in (pre.out, out, *pool)])
    for got in results[1:]:
        for a, b in zip(got, results[0]):
            assert _q4.same_bits(a, b)
    assert _q4.status() == 0


def test_two_streams_with_workspaces_of_their_own():
    cs = [Chain(64), Chain(128)]
    want = []
    for c in cs:
        c.reset()
        c.copies()
        c.append()
        c.attend()
        want.append(c.results())
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(4):
        for c in cs:
            c.reset()
        for c, st in zip(cs, streams):
            with torch.cuda.stream(st):
                c.copies()
                for _ in range(8):
                    c.append()
                    c.attend()
        for c, w in zip(cs, want):
            for a, b in zip(c.results(), w):
                assert _q4.same_bits(a, b)
    assert _q4.status() == 0


def test_long_offsets_in_a_large_pool():
    """Blocks whose bytes lie past 2^32 of a pool's start, for every call."""
    hkv, d, nbk = 4, 128, (1 << 32) // (4 * 16 * 64) + 100  # codes of 4.3 GB, twice
    pools = [t for _ in range(2) for t in (torch.zeros(nbk, hkv, 16, d // 2, dtype=torch.uint8, device="cuda"),
                                           torch.zeros(nbk, hkv, 16, d // 32, dtype=torch.float16, device="cuda"))]
    rng = np.random.default_rng(5)
    lens = [70, 33]
    tables = np.array([[nbk - 1, nbk - 30, 3, nbk - 77, nbk - 2], [nbk - 50, 0, nbk - 51, -1, -1]], np.int32)
    T = sum(lens)
    seq = np.repeat([0, 1], lens)
    pos = np.concatenate([np.arange(n) for n in lens])
    slots = tables[seq, pos // 16].astype(np.int64) * 16 + pos % 16
    x = [_q4.to16(rng.standard_normal((T, h, d)).astype(np.float32), wl.BF16).cuda() for h in (8, hkv, hkv)]
    angles = _q4.table(100, d)
    q_out = torch.empty_like(x[0])
    nb.ns_rope_kv_append_q4_0(*x, _gpu.dev_ints(pos, np.int32), torch.from_numpy(angles).cuda(), _gpu.dev_ints(slots, np.int64),
                              q_out, *pools)
    held = [torch.from_numpy(_q4.values(*_q4.quantise(y))) for y in (_q4.rotate(_q4.f32(x[1]), angles, pos, False), _q4.f32(x[2]))]
    bt, last = _gpu.dev_ints(tables, np.int32), np.cumsum(lens) - 1
    q = q_out[torch.from_numpy(last).cuda()].contiguous()
    out = torch.empty_like(q)
    nb.ns_paged_attn_decode_q4_0(q, *pools, bt, _gpu.dev_ints(lens, np.int32), d ** -0.5, out, nb.alloc_workspace(2, 8, hkv, d))
    ref = torch.cat([_span.attend(q[s:s + 1].cpu(), held[0][seq == s], held[1][seq == s], d ** -0.5) for s in range(2)])
    _q4.compare(out, ref.numpy(), wl.BF16, "far blocks")
    counts = [5, 1]
    qs = torch.cat([q_out[65:70], q_out[T - 1:]])
    out = torch.empty_like(qs)
    nb.ns_paged_attn_prefill_q4_0(qs, _gpu.dev_ints(_span.starts(counts), np.int32), *pools, bt, _gpu.dev_ints(lens, np.int32),
                                  d ** -0.5, out, nb.alloc_span_workspace(d))
    ref = torch.cat([_span.attend(x.cpu(), held[0][seq == s], held[1][seq == s], d ** -0.5) for s, x in enumerate((qs[:5], qs[5:]))])
    _span.compare(out, ref, wl.BF16, "far blocks, spans", q8=True)
    rows = [torch.empty(T, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    nb.ns_kv_gather_q4_0(*pools, bt, _gpu.dev_ints(_span.starts(lens), np.int32), *rows)
    for got, want in zip(rows, held):
        assert np.array_equal(_gpu.to_f64(got), _gpu.round_to_dtype(want.numpy(), wl.BF16))
    assert _q4.status() == 0
