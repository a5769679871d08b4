"""Rotary append on the GPU: the rotated rows within half a step of the type, caches bit for bit."""
import numpy as np
import pytest
import torch

import _q4
from _q4 import wl
from oracle import q8
from paged_kv_decode_ns_gb300 import binding as nb

pytestmark = pytest.mark.gpu


class Step:
    """T tokens' fused projection rows, positions, slots, a table and pools of the kind `pool`."""

    def __init__(self, seed, T, hq, hkv, d, dtype, pool, rotary, bs=16, positions=300, amp=1.0, slots=None, gap=0, x=None):
        rng = np.random.default_rng(seed)
        self.hq, self.hkv, self.d, self.dtype, self.pool, self.bs = hq, hkv, d, dtype, pool, bs
        nbk = -(-max(T, 1) // bs) + 3
        x = rng.standard_normal((T, hq + 2 * hkv, d)).astype(np.float32) * np.float32(amp) if x is None else x
        wide = np.full((T, (hq + 2 * hkv) * d + gap), np.nan, np.float32)
        wide[:, :(hq + 2 * hkv) * d] = x.reshape(T, (hq + 2 * hkv) * d)
        self.rows = _q4.to16(wide, dtype).cuda()
        qkv = self.rows[:, :(hq + 2 * hkv) * d].unflatten(-1, (hq + 2 * hkv, d))
        self.q, self.k, self.v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        self.pos = rng.integers(0, positions, T).astype(np.int32)
        self.slots = rng.permutation(nbk * bs)[:T].astype(np.int64) if slots is None else np.asarray(slots, np.int64)
        self.table = _q4.table(positions, rotary)
        self.q_out = torch.full((T, hq, d), 7.0, dtype=self.q.dtype, device="cuda")
        self.k_out = torch.full((T, hkv, d), 7.0, dtype=self.q.dtype, device="cuda")
        shape = (nbk, hkv, bs)
        if pool == "16":
            self.pools = [torch.full(shape + (d,), 3.0, dtype=self.q.dtype) for _ in range(2)]
        else:
            width, t = (d, torch.int8) if pool == "q8_0" else (d // 2, torch.uint8)
            self.pools = [p for _ in range(2) for p in (torch.full(shape + (width,), 90, dtype=t),
                                                        torch.full(shape + (d // 32,), 5.0, dtype=torch.float16))]
        self.pools = [p.cuda() for p in self.pools]

    def call(self, interleaved=False, q_out=None, k_out=None, no_k=False, **kw):
        fn = {"16": nb.ns_rope_kv_append, "q8_0": nb.ns_rope_kv_append_q8_0, "q4_0": nb.ns_rope_kv_append_q4_0}[self.pool]
        fn(self.q, self.k, self.v, torch.from_numpy(self.pos).cuda(), torch.from_numpy(self.table).cuda(),
           torch.from_numpy(self.slots).cuda(), self.q_out if q_out is None else q_out, *self.pools,
           k_out=None if no_k else self.k_out if k_out is None else k_out, interleaved=interleaved, **kw)

    def want(self, interleaved=False, skip=()):
        """(q_out, k_out, pools) as the definition has them, from the state before the call."""
        on = (self.slots >= 0) & ~np.isin(np.arange(len(self.slots)), skip)
        pos = np.where(on, self.pos, 0)
        q, k = (_q4.rotate(_q4.f32(t), self.table, pos, interleaved) for t in (self.q, self.k))
        v = _q4.f32(self.v)
        q_out, k_out, pools = self.q_out.cpu().clone(), self.k_out.cpu().clone(), [p.cpu().clone() for p in self.pools]
        at = np.nonzero(on)[0]
        q_out[at], k_out[at] = _q4.to16(q, self.dtype)[at], _q4.to16(k, self.dtype)[at]
        blk, off = self.slots[at] // self.bs, self.slots[at] % self.bs
        for i, x in enumerate((k, v)):
            if self.pool == "16":
                pools[i][blk, :, off] = _q4.to16(x, self.dtype)[at]
                continue
            codes, steps = q8.quantize_q8_0(x) if self.pool == "q8_0" else _q4.quantise(x)
            pools[2 * i][blk, :, off] = torch.from_numpy(codes[at])
            pools[2 * i + 1][blk, :, off] = torch.from_numpy(steps[at])
        return q_out, k_out, pools

    def check(self, interleaved=False, skip=(), **kw):
        q_out, k_out, pools = self.want(interleaved, skip)
        self.call(interleaved, **kw)
        torch.cuda.synchronize()
        assert _q4.same_bits(self.q_out, q_out)
        if not kw.get("no_k"):
            assert _q4.same_bits(self.k_out, k_out)
        for got, ref in zip(self.pools, pools):
            assert _q4.same_bits(got, ref)


POOLS = ["16", "q8_0", "q4_0"]


@pytest.mark.parametrize("dtype", [wl.F16, wl.BF16])
@pytest.mark.parametrize("pool", POOLS)
@pytest.mark.parametrize("T,hq,hkv", [(1, 14, 2), (4, 14, 2), (77, 5, 1), (33, 3, 4), (260, 1, 1)])
def test_rows_and_pools(dtype, pool, T, hq, hkv):
    Step(T, T, hq, hkv, 64, dtype, pool, 64).check()
    assert _q4.status() == 0


@pytest.mark.parametrize("dtype", [wl.F16, wl.BF16])
@pytest.mark.parametrize("pool", ["16", "q4_0"])
@pytest.mark.parametrize("T,hq,hkv", [(1, 32, 8), (50, 28, 4), (9, 7, 3)])
def test_head_dim_128(dtype, pool, T, hq, hkv):
    Step(T, T, hq, hkv, 128, dtype, pool, 128).check()
    assert _q4.status() == 0


@pytest.mark.parametrize("d,rotary", [(64, r) for r in (16, 32, 48, 64)] + [(128, r) for r in (16, 80, 96, 112, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("pool", ["16", "q4_0"])
def test_part_of_the_width(d, rotary, interleaved, pool):
    Step(rotary, 21, 6, 3, d, wl.BF16, pool, rotary).check(interleaved)


@pytest.mark.parametrize("bs", [4, 8, 16, 32])
@pytest.mark.parametrize("pool", POOLS)
def test_block_sizes_and_strided_rows(bs, pool):
    Step(bs, 45, 14, 2, 64, wl.F16, pool, 32, bs=bs, gap=24).check()


@pytest.mark.parametrize("pool", POOLS)
def test_many_tokens_share_a_warp_each(pool):
    Step(3, 3001, 14, 2, 64, wl.BF16, pool, 64).check()
    assert _q4.status() == 0


@pytest.mark.parametrize("pool", POOLS)
def test_padding_rows_stay_as_they_were(pool):
    st = Step(5, 40, 14, 2, 64, wl.F16, pool, 64)
    st.slots[[0, 7, 38, 39]] = [-1, -5, -1, -(1 << 40)]
    st.pos[[0, 39]] = [-3, 1 << 30]  # not looked at
    st.check()
    assert _q4.status() == 0


@pytest.mark.parametrize("pool", POOLS)
def test_bad_slots_and_positions_are_skipped_and_reported(pool):
    st = Step(6, 12, 4, 2, 64, wl.F16, pool, 64)
    st.slots[3] = st.pools[0].shape[0] * 16
    st.check(skip=(3,))
    assert _q4.status() == 0x4
    st = Step(6, 12, 4, 2, 64, wl.F16, pool, 64)
    st.pos[[2, 9]] = [300, -1]
    st.check(skip=(2, 9))
    assert _q4.status() == 0x100
    st = Step(6, 3, 4, 2, 64, wl.F16, pool, 64)
    st.slots[1] = 1 << 45
    st.check(skip=(1,))
    assert _q4.status() == 0x4


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("pool", POOLS)
def test_in_place(interleaved, pool):
    st = Step(8, 19, 14, 2, 64, wl.BF16, pool, 48, gap=8)
    q_out, k_out, pools = st.want(interleaved)
    st.call(interleaved, q_out=st.q, k_out=st.k)
    assert _q4.same_bits(st.q.contiguous(), q_out) and _q4.same_bits(st.k.contiguous(), k_out)
    for got, ref in zip(st.pools, pools):
        assert _q4.same_bits(got, ref)
    assert torch.isnan(st.rows[:, -8:].float()).all()  # nothing between the rows is written


@pytest.mark.parametrize("pool", POOLS)
def test_without_the_rotated_keys(pool):
    st = Step(9, 30, 9, 3, 64, wl.F16, pool, 64)
    st.check(no_k=True)
    assert (st.k_out == 7.0).all()


@pytest.mark.parametrize("pool", ["q8_0", "q4_0"])
def test_codes_equal_rotation_and_append_of_the_pools_own_calls(pool):
    """With angles that fp16 rows keep exactly, the call equals the separate append of the rotated rows."""
    st = Step(10, 64, 4, 2, 64, wl.F16, pool, 64)
    st.table[:, :32], st.table[:, 32:] = 0.0, 1.0
    st.call()
    again = [torch.zeros_like(p) for p in st.pools]
    append = nb.ns_kv_append_q8_0 if pool == "q8_0" else nb.ns_kv_append_q4_0
    append(st.k_out, st.v.contiguous(), torch.from_numpy(st.slots).cuda(), *again)
    blk, off = torch.from_numpy(st.slots // 16).cuda(), torch.from_numpy(st.slots % 16).cuda()
    for a, b in zip(st.pools, again):
        assert _q4.same_bits(a[blk, :, off], b[blk, :, off])


def test_values_that_are_not_finite_stay_in_their_pairs_and_groups():
    st = Step(11, 6, 2, 1, 64, wl.BF16, "q4_0", 32)
    with torch.no_grad():
        st.q[1, 0, 3] = float("nan")
        st.k[2, 0, 40] = float("inf")
        st.v[3, 0, 5] = float("nan")
    _, _, pools = st.want()
    st.call()
    bad = torch.isnan(st.q_out[1, 0].float()).nonzero().flatten().tolist()
    assert bad == [3, 19]
    for i in (0, 2):
        assert _q4.same_bits(st.pools[i], pools[i])
    for i in (1, 3):
        a, b = st.pools[i].cpu(), pools[i]
        assert torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(), b.nan_to_num())


@pytest.mark.parametrize("pool", POOLS)
def test_no_tokens(pool):
    st = Step(12, 0, 14, 2, 64, wl.F16, pool, 64)
    before = [p.clone() for p in st.pools]
    st.call()
    assert all(_q4.same_bits(a, b) for a, b in zip(st.pools, before))


def test_captured_and_replayed_on_another_stream():
    st = Step(13, 40, 14, 2, 64, wl.BF16, "q4_0", 64)
    q_out, k_out, pools = st.want()
    call = nb.prepare(nb.ns_rope_kv_append_q4_0, st.q, st.k, st.v, torch.from_numpy(st.pos).cuda(),
                      torch.from_numpy(st.table).cuda(), torch.from_numpy(st.slots).cuda(), st.q_out, *st.pools, k_out=st.k_out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    assert (st.q_out == 7.0).all()
    for _ in range(2):
        st.q_out.fill_(1.0)
        graph.replay()
    torch.cuda.synchronize()
    assert _q4.same_bits(st.q_out, q_out) and _q4.same_bits(st.k_out, k_out)
    for got, ref in zip(st.pools, pools):
        assert _q4.same_bits(got, ref)
