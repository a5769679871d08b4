"""GPU: calls on one stream take effect in their order.  A prefill whose long
single-token row outlasts its short chunk is followed at once by calls that read its
output, or write where it reads and writes; the results are those of the same calls
with a synchronisation between them."""
import numpy as np
import pytest
import torch

import _gpu
import _span
from paged_kv_decode_ns_gb300 import binding as nb
from paged_kv_decode_ns_gb300 import workloads as wl
from test_gpu_kv_gather import Pool16
from test_gpu_span_attn import Chunks
from test_gpu_verify_drafts import Drafts

pytestmark = pytest.mark.gpu

HQ, HKV, D, LONG = 14, 2, 64, 300000  # the long row's cache (154 MB) takes its few CTAs hundreds of microseconds


class Prefill:
    """One row over LONG tokens beside a chunk of two tokens."""

    def __init__(self):
        g = torch.Generator(device="cuda").manual_seed(1)
        nblk = LONG // 16 + 1
        self.k, self.v = (torch.randn(nblk, HKV, 16, D, generator=g, device="cuda").half() for _ in range(2))
        self.tables = torch.zeros(2, nblk, dtype=torch.int32, device="cuda")
        self.tables[0] = torch.arange(nblk, device="cuda")
        self.tables[1] = nblk - 1
        self.lens = _gpu.dev_ints([LONG, 2], np.int32)
        self.starts = _gpu.dev_ints([0, 1, 3], np.int32)
        self.q0 = torch.randn(3, HQ, D, generator=g, device="cuda").half()
        self.q, self.out = torch.empty_like(self.q0), torch.empty_like(self.q0)
        self.ws = nb.alloc_workspace(3, HQ, HKV, D)

    def reset(self):
        self.q.copy_(self.q0)
        self.out.fill_(7.0)
        torch.cuda.synchronize()

    def call(self):
        nb.ns_paged_attn_prefill(self.q, self.starts, self.k, self.v, self.tables, self.lens, 0.125, self.out, self.ws)


def prompt_reads_out(pre):
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn(3, HKV, D, generator=g).half().cuda() for _ in range(2))
    out, ws, starts = torch.zeros_like(pre.out), nb.alloc_span_workspace(64), _gpu.dev_ints([0, 3], np.int32)
    return lambda: nb.ns_prompt_attn(pre.out, k, v, starts, 0.125, out, ws), [out]


def prompt_writes(pre, where):
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(3, h, D, generator=g).half().cuda() for h in (HQ, HKV, HKV))
    ws, starts = nb.alloc_span_workspace(64), _gpu.dev_ints([0, 3], np.int32)
    return lambda: nb.ns_prompt_attn(q, k, v, starts, 0.125, where, ws), []


def chunk_reads_out(pre):
    c = Chunks([(2, 40), (1, 17)], wl.F16, HQ, HKV, seed=4)
    c.q = pre.out
    c.out.fill_(0)
    return c.call, [c.out]


def chunk_writes(pre, where):
    c = Chunks([(2, 40), (1, 17)], wl.F16, HQ, HKV, seed=4)
    c.out = where
    return c.call, []


def gather_writes(pre, where):
    c = Pool16([10, 11], HKV, 16, D, seed=5)
    k, v, t = _gpu.to_dev(c.k, wl.F16), _gpu.to_dev(c.v, wl.F16), _gpu.dev_ints(c.tables, np.int32)
    rows = where.view(-1, HKV, D)  # 21 rows
    other, starts = torch.zeros_like(rows), _gpu.dev_ints([0, 10, 21], np.int32)
    return lambda: nb.ns_kv_gather(k, v, t, starts, rows, other), []


def verify_writes(pre, where):
    d = Drafts([3] * 4, 500, seed=6)
    args = d.dev()
    flat = where.view(torch.int32).flatten()
    # over the long row
    return lambda: nb.ns_verify_drafts(*args, flat[:16], flat[32:36]), []


AFTER = {
    "prompt reads out": lambda p: prompt_reads_out(p),
    "prompt writes out": lambda p: prompt_writes(p, p.out),
    "prompt writes q": lambda p: prompt_writes(p, p.q),
    "chunk reads out": lambda p: chunk_reads_out(p),
    "chunk writes out": lambda p: chunk_writes(p, p.out),
    "chunk writes q": lambda p: chunk_writes(p, p.q),
    "gather writes out": lambda p: gather_writes(p, p.out),
    "gather writes q": lambda p: gather_writes(p, p.q),
    "verify writes out": lambda p: verify_writes(p, p.out),
    "verify writes q": lambda p: verify_writes(p, p.q),
}


@pytest.fixture(scope="module")
def prefill():
    return Prefill()


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("what", sorted(AFTER))
def test_call_behind_a_prefill_whose_walk_is_the_longer_part(prefill, what, captured):
    call, outs = AFTER[what](prefill)
    outs = [prefill.out, prefill.q, *outs]
    prefill.reset()
    prefill.call()
    torch.cuda.synchronize()
    assert bool(torch.isfinite(prefill.out.float()).all())
    call()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    run = lambda: (prefill.call(), call())  # noqa: E731
    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        run = g.replay
    for _ in range(3):
        prefill.reset()
        run()
        torch.cuda.synchronize()
        for got, w in zip(outs, want):
            assert torch.equal(got.view(torch.int16), w.view(torch.int16))
    _gpu.assert_no_device_status()


def test_the_prefill_alone_is_right(prefill):
    """The long row against fp64 (the chunk's tokens share the last block)."""
    prefill.reset()
    prefill.call()
    torch.cuda.synchronize()
    k = prefill.k.transpose(1, 2).reshape(-1, HKV, D)[:LONG].double()
    v = prefill.v.transpose(1, 2).reshape(-1, HKV, D)[:LONG].double()
    for j in (0, 13):
        w = torch.softmax(0.125 * (k[:, j // 7] @ prefill.q[0, j].double()), 0)
        want = w @ v[:, j // 7]
        _gpu.compare(prefill.out[0, j], want.cpu().numpy(), wl.F16, "long row")
    _gpu.assert_no_device_status()


def calls():
    """Each entry point on inputs of its own: (call, the buffers it reads that a copy can fill, outputs)."""
    g = torch.Generator().manual_seed(9)
    q, k, v = (torch.randn(700, h, D, generator=g).half().cuda() for h in (HQ, HKV, HKV))
    out, ws, starts = torch.empty_like(q), nb.alloc_span_workspace(64), _gpu.dev_ints([0, 600, 700], np.int32)
    yield "prompt", lambda: nb.ns_prompt_attn(q, k, v, starts, 0.125, out, ws), q, [out]
    c = Chunks([(2, 40), (1, 900)], wl.BF16, HQ, HKV, seed=10)
    yield "chunk", c.call, c.q, [c.out]
    p = Pool16([10, 11], HKV, 16, D, seed=11)
    kp, vp, t = _gpu.to_dev(p.k, wl.F16), _gpu.to_dev(p.v, wl.F16), _gpu.dev_ints(p.tables, np.int32)
    ko, vo = (torch.zeros(21, HKV, D, dtype=torch.float16, device="cuda") for _ in range(2))
    gs = _gpu.dev_ints([0, 10, 21], np.int32)
    yield "gather", lambda: nb.ns_kv_gather(kp, vp, t, gs, ko, vo), kp, [ko, vo]
    d = Drafts([3] * 4, 500, seed=12).dev()
    tokens, num = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (16, 4))
    yield "verify", lambda: nb.ns_verify_drafts(*d, tokens, num), d[0], [tokens, num]


@pytest.mark.parametrize("front", ["copy", "memset", "join", "nothing"])
def test_captured_behind_other_nodes(front):
    """A captured call whose input comes from a copy, or that stands behind a memset, or where two streams
    join, or first in its graph."""
    for what, call, src, outs in calls():
        call()
        torch.cuda.synchronize()
        want, kept = [o.clone() for o in outs], src.clone()
        side = torch.cuda.Stream()
        big = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            main = torch.cuda.current_stream()
            if front == "copy":
                big[:1 << 27].copy_(big[1 << 27:])
                src.copy_(kept)
            elif front == "memset":
                outs[0].view(torch.uint8).zero_()
            elif front == "join":
                side.wait_stream(main)
                with torch.cuda.stream(side):
                    big.fill_(1)
                    src.copy_(kept)
                outs[0].fill_(0)
                main.wait_stream(side)
            call()
        for _ in range(2):
            if front in ("copy", "join"):
                src.zero_()
            for o in outs:
                o.fill_(5)
            graph.replay()
            torch.cuda.synchronize()
            for o, w in zip(outs, want):
                assert torch.equal(o.view(torch.int16), w.view(torch.int16)), (what, front)
            src.copy_(kept)
    _gpu.assert_no_device_status()
