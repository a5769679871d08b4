"""GPU: reading sequences back from the paged cache, against a numpy gather.  The
16-bit form copies bits; the q8_0 form rounds fp16(d) * code once."""
import numpy as np
import pytest
import torch

import _gpu
import _span
from paged_kv_decode_ns_gb300 import binding as nb
from paged_kv_decode_ns_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

LENS = [1, 0, 17, 64, 200, 15, 16, 33]


class Pool16:
    def __init__(self, lens, hkv, bs, d, seed=0):
        rng = np.random.default_rng(seed)
        need = [max(1, -(-n // bs)) for n in lens]
        nblk = sum(need) + 3
        order = rng.permutation(nblk)
        self.tables = np.full((len(lens), max(need)), -1, np.int32)
        at = 0
        for s, n in enumerate(need):
            self.tables[s, :n] = order[at:at + n]
            at += n
        self.k = rng.integers(0, 1 << 16, (nblk, hkv, bs, d)).astype(np.uint16)  # every bit pattern
        self.v = rng.integers(0, 1 << 16, (nblk, hkv, bs, d)).astype(np.uint16)
        self.bs = bs

    def rows(self, pool, s, n):
        p = np.arange(n)
        return pool[self.tables[s, p // self.bs], :, p % self.bs]


@pytest.mark.parametrize("dtype", [wl.F16, wl.BF16])
@pytest.mark.parametrize("hkv,bs,d", [(2, 16, 64), (1, 4, 64), (3, 8, 64), (2, 32, 64), (8, 16, 128), (1, 16, 128)])
def test_gather_copies_bits(dtype, hkv, bs, d):
    c = Pool16(LENS, hkv, bs, d)
    sl = _span.starts(LENS, 3)
    t = int(sl[-1]) + 4  # rows before and behind the sequences
    k, v = (_gpu.to_dev(np.full((t, hkv, d), 0x1234, np.uint16), dtype) for _ in range(2))
    nb.ns_kv_gather(_gpu.to_dev(c.k, dtype), _gpu.to_dev(c.v, dtype), _gpu.dev_ints(c.tables, np.int32),
                    _gpu.dev_ints(sl, np.int32), k, v)
    torch.cuda.synchronize()
    _gpu.assert_no_device_status()
    for got, pool in ((k, c.k), (v, c.v)):
        want = np.full((t, hkv, d), 0x1234, np.uint16)
        for s, n in enumerate(LENS):
            want[sl[s]:sl[s + 1]] = c.rows(pool, s, n)
        assert np.array_equal(_gpu.to_bits(got), want)


@pytest.mark.parametrize("dtype", [wl.F16, wl.BF16])
@pytest.mark.parametrize("bs,hkv", [(16, 2), (4, 1), (32, 3)])
def test_gather_q8_0_rounds_once(dtype, bs, hkv):
    c = _span.Q8Cache(np.random.default_rng(bs), LENS, hkv, bs=bs)
    sl = _span.starts(LENS)
    k, v = (torch.full((int(sl[-1]) + 2, hkv, 64), 7.0, dtype=_span.TORCH[dtype], device="cuda") for _ in range(2))
    kc, ks, vc, vs, tables = c.dev()
    nb.ns_kv_gather_q8_0(kc, ks, vc, vs, tables, _gpu.dev_ints(sl, np.int32), k, v)
    torch.cuda.synchronize()
    _gpu.assert_no_device_status()
    for got, vals in ((k, c.k), (v, c.v)):
        want = _gpu.round_to_dtype(np.concatenate([x.numpy() for x in vals]), dtype)
        assert np.array_equal(_gpu.to_f64(got)[:sl[-1]], want)
        assert bool((got[sl[-1]:] == 7.0).all())


def test_gather_undoes_append():
    st = wl.decode_batch32()
    d = _gpu.DevStep(st)
    d.append()
    sl = _span.starts(st.context_lens)
    k = torch.empty(int(sl[-1]), st.num_kv_heads, 64, dtype=d.q.dtype, device="cuda")
    v = torch.empty_like(k)
    nb.ns_kv_gather(d.k_pool, d.v_pool, d.block_tables, _gpu.dev_ints(sl, np.int32), k, v)
    last = torch.from_numpy(sl[1:].astype(np.int64) - 1).cuda()
    assert torch.equal(k[last], d.k_new) and torch.equal(v[last], d.v_new)


def test_many_sequences_and_a_long_one():
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(0, 40, 1500)] + [5000]
    c = Pool16(lens, 2, 16, 64, seed=4)
    sl = _span.starts(lens)
    k = torch.empty(int(sl[-1]), 2, 64, dtype=torch.float16, device="cuda")
    v = torch.empty_like(k)
    nb.ns_kv_gather(_gpu.to_dev(c.k, wl.F16), _gpu.to_dev(c.v, wl.F16), _gpu.dev_ints(c.tables, np.int32),
                    _gpu.dev_ints(sl, np.int32), k, v)
    torch.cuda.synchronize()
    _gpu.assert_no_device_status()
    want = np.concatenate([c.rows(c.v, s, n) for s, n in enumerate(lens)])
    assert np.array_equal(_gpu.to_bits(v), want)


def test_bad_device_data():
    c = Pool16([20, 30, 10], 2, 16, 64)
    kp, vp = _gpu.to_dev(c.k, wl.F16), _gpu.to_dev(c.v, wl.F16)
    for change, bits in (((1, 0, 9999), 0x1), ((1, 0, -7), 0x1), (None, 0x2)):
        tables, sl = c.tables.copy(), _span.starts([20, 30, 10])
        if change:
            tables[change[0], change[1]] = change[2]
            lost = range(20, 36)  # its block's rows
        else:
            sl = _span.starts([20, 33, 10])  # one token more than the two blocks of a table row
            lost = range(20, 53)
        k, v = (_gpu.to_dev(np.full((int(sl[-1]), 2, 64), 0x1234, np.uint16), wl.F16) for _ in range(2))
        nb.ns_kv_gather(kp, vp, _gpu.dev_ints(tables, np.int32), _gpu.dev_ints(sl, np.int32), k, v)
        torch.cuda.synchronize()
        assert nb.ns_get_device_status() == bits
        got = _gpu.to_bits(k)
        assert (got[list(lost)] == 0x1234).all()
        assert np.array_equal(got[:20], c.rows(c.k, 0, 20)) and np.array_equal(got[-10:], c.rows(c.k, 2, 10))
    k = _gpu.to_dev(np.full((25, 2, 64), 0x1234, np.uint16), wl.F16)
    v = k.clone()
    nb.ns_kv_gather(kp, vp, _gpu.dev_ints(c.tables, np.int32), _gpu.dev_ints([0, 20, 50, 60], np.int32), k, v)
    torch.cuda.synchronize()
    assert nb.ns_get_device_status() == 0x20
    assert np.array_equal(_gpu.to_bits(k)[:20], c.rows(c.k, 0, 20))


@pytest.mark.parametrize("sl", [[0, 20, 10, 30], [0, 20, 60, 70], [-1, 5, 10, 20], [0, 60, 60, 61]])
def test_entries_out_of_order_are_reported(sl):
    c = Pool16([64, 64, 64], 2, 16, 64)
    k = _gpu.to_dev(np.full((60, 2, 64), 0x1234, np.uint16), wl.F16)
    nb.ns_kv_gather(_gpu.to_dev(c.k, wl.F16), _gpu.to_dev(c.v, wl.F16), _gpu.dev_ints(c.tables, np.int32),
                    _gpu.dev_ints(sl, np.int32), k, k.clone())
    torch.cuda.synchronize()
    assert nb.ns_get_device_status() == 0x20


def test_refusals():
    c = _span.Q8Cache(np.random.default_rng(0), [20])
    kc, ks, vc, vs, tables = c.dev()
    sl = _gpu.dev_ints([0, 20], np.int32)
    out = torch.empty(20, 2, 64, dtype=torch.float16, device="cuda")
    with pytest.raises(TypeError):
        nb.ns_kv_gather_q8_0(kc, ks, vc, vs, tables, sl, out.float(), out.float())
    with pytest.raises(ValueError):
        nb.ns_kv_gather_q8_0(kc, ks, vc, vs, tables, sl, out, out[:10])
    with pytest.raises(ValueError):
        nb.ns_kv_gather_q8_0(kc, ks, vc, vs, tables, sl[:1], out, out.clone())
