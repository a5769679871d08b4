"""GPU: one workspace, zero-filled once, serves calls of every size up to the one that it was sized for: few long
sequences, whose pairs are cut across CTAs, between many short ones, over 16-, 8- and 4-bit pools and
beside a mixed prefill."""
import numpy as np
import pytest
import torch

import _gpu
import _q4
from _q4 import wl
from paged_kv_decode_ns_gb300 import binding as nb
from test_gpu_q8 import Q8Step

pytestmark = pytest.mark.gpu

HQ, HKV, MANY = 16, 8, 300


def lengths(rng, many):
    return wl.lognormal_lengths(rng, MANY, 150, 1.0, 1200) if many else np.full(4, 4096, np.int32)


class Over16:
    def __init__(self, rng, many, d, dtype, orc):
        lens = lengths(rng, many)
        st = wl.make_step(rng, lens, np.ones_like(lens), dtype=dtype, num_q_heads=HQ, num_kv_heads=HKV, head_dim=d)
        self.d = _gpu.DevStep(st)
        self.d.append()
        self.out, self.dtype = self.d.out, dtype
        self.exact = lambda: orc.step(st, num_threads=orc.max_threads())[0]

    def call(self, ws):
        self.d.ws = ws
        self.d.decode()


class Prefill(Over16):
    def __init__(self, rng, many, d, dtype, orc):
        lens = np.array([70] * 40 + [900, 130, 130], np.int32)
        st = wl.make_step(rng, lens, np.array([1] * 40 + [1, 100, 130], np.int32), dtype=dtype, num_q_heads=HQ,
                          num_kv_heads=HKV, head_dim=d)
        self.d = _gpu.DevStep(st)
        self.d.append()
        self.out, self.dtype = self.d.out, dtype
        self.exact = lambda: orc.step(st, num_threads=orc.max_threads())[0]

    def call(self, ws):
        self.d.ws = ws
        self.d.prefill()


class Over8:
    def __init__(self, rng, many, d, dtype, orc):
        lens = lengths(rng, many)
        self.s = Q8Step(wl.make_step(rng, lens, np.ones_like(lens), dtype=dtype, num_q_heads=HQ, num_kv_heads=HKV))
        s, t = self.s, self.s.d
        nb.ns_kv_append_q8_0(t.k_new, t.v_new, t.slot_mapping, s.kc, s.ks, s.vc, s.vs)
        self.out, self.dtype, self.exact = torch.empty_like(t.q), dtype, s.ref

    def call(self, ws):
        s, t = self.s, self.s.d
        nb.ns_paged_attn_decode_q8_0(t.q, s.kc, s.ks, s.vc, s.vs, t.block_tables, t.context_lens, s.st.scale, self.out, ws)


class Over4:
    def __init__(self, rng, many, d, dtype, orc):
        lens = lengths(rng, many)
        cache = _q4.Cache(rng, lens, HKV, 16, d)
        q = _q4.to16(rng.standard_normal((len(lens), HQ, d)).astype(np.float32), dtype)
        self.q, self.pools, self.lens = q.cuda(), cache.dev(), _gpu.dev_ints(lens, np.int32)
        self.out, self.dtype, self.scale = torch.empty_like(self.q), dtype, d ** -0.5
        self.exact = lambda: _q4.attend_all(q, [(1, n) for n in lens], cache, self.scale).numpy()

    def call(self, ws):
        nb.ns_paged_attn_decode_q4_0(self.q, *self.pools, self.lens, self.scale, self.out, ws)


@pytest.mark.parametrize("d,dtype", [(64, wl.F16), (64, wl.BF16), (128, wl.BF16)])
def test_calls_of_other_sizes_leave_a_workspace_ready(d, dtype, orc):
    rng = np.random.default_rng(d)
    kinds = [Over4, Over16] + ([Over8] if d == 64 else [])
    few, many = ([kind(rng, big, d, dtype, orc) for kind in kinds] for big in (False, True))
    pre = Prefill(rng, True, d, dtype, orc)
    # each on a workspace of its own, against fp64
    want = {}
    for c in (*few, *many, pre):
        c.out.fill_(float("nan"))
        c.call(nb.alloc_workspace(MANY, HQ, HKV, d))
        torch.cuda.synchronize()
        compare = _q4.compare if isinstance(c, Over4) else _gpu.compare
        compare(c.out, c.exact(), dtype, type(c).__name__)
        want[c] = c.out.clone()
    # and all of them on one
    ws = nb.alloc_workspace(MANY, HQ, HKV, d)
    for c in (*few, *many, pre, *reversed(many), *reversed(few), pre, *many, *few, *many):
        c.out.fill_(float("nan"))
        c.call(ws)
        torch.cuda.synchronize()
        assert _q4.same_bits(c.out, want[c]), f"{type(c).__name__}, {len(c.out)} rows"
    _gpu.assert_no_device_status()


def test_a_workspace_of_both_widths_sizes_together(orc):
    """head_dim 64 and 128 on one workspace, as large as the sizes for either together."""
    rng = np.random.default_rng(9)
    calls = [kind(rng, many, d, wl.F16, orc) for d in (64, 128) for kind in (Over4, Over16) for many in (True, False)]
    want, sizes = [], [nb.ns_paged_attn_workspace_bytes(MANY, HQ, HKV, d) for d in (64, 128)]
    for c, d in zip(calls, [64] * 4 + [128] * 4):
        c.call(nb.alloc_workspace(MANY, HQ, HKV, d))
        torch.cuda.synchronize()
        want.append(c.out.clone())
    ws = torch.zeros(sum(sizes), dtype=torch.uint8, device="cuda")
    for i in (0, 5, 4, 1, 7, 2, 6, 3, 0, 1, 4, 5, 2, 3, 6, 7):
        calls[i].out.fill_(float("nan"))
        calls[i].call(ws)
        torch.cuda.synchronize()
        assert _q4.same_bits(calls[i].out, want[i]), f"{type(calls[i]).__name__}, call {i}"
    _gpu.assert_no_device_status()
