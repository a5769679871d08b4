"""GPU: the calls of a serving loop over a q8_0 cache, one after another as they
are used: prompts attend straight from their projection while their K/V are
quantised into the cache; drafted tokens are appended and attend over the cache;
the drafts are verified and the rejected ones dropped; the cache is read back and
serves as the prefix of a new prompt.  Every step against fp64."""
import numpy as np
import pytest
import torch

import _gpu
import _span
from oracle import q8
from paged_kv_decode_ns_gb300 import binding as nb
from paged_kv_decode_ns_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

HQ, HKV, D, BS, SCALE = 14, 2, 64, 16, 0.125


@pytest.mark.parametrize("dtype", [wl.F16, wl.BF16])
def test_prompt_then_drafts_then_read_back(dtype):
    rng = np.random.default_rng(17)
    g = torch.Generator().manual_seed(17)
    td = _span.TORCH[dtype]
    lens = np.array([37, 200, 1, 130])
    S, room = len(lens), 20  # blocks a sequence may fill
    tables = rng.permutation(S * room).reshape(S, room).astype(np.int32)
    shape = (S * room, HKV, BS, D)
    pools = [torch.zeros(shape, dtype=torch.int8, device="cuda"),
             torch.full((*shape[:3], 2), float("nan"), dtype=torch.float16, device="cuda")]
    pools = [pools[0], pools[1], pools[0].clone(), pools[1].clone()]
    bt = _gpu.dev_ints(tables, np.int32)
    ws = nb.alloc_span_workspace(64)
    held = [[], []]  # the cache's exact values: K and V per sequence
    for x in held:
        x.extend(torch.zeros(0, HKV, D, dtype=torch.float64) for _ in range(S))

    def slots(ctx, counts):
        return np.concatenate([tables[s, p // BS].astype(np.int64) * BS + p % BS
                               for s in range(S) for p in [np.arange(ctx[s] - counts[s], ctx[s])]])

    def append(k, v, ctx, counts):
        nb.ns_kv_append_q8_0(k, v, _gpu.dev_ints(slots(ctx, counts), np.int64), *pools)
        for x, side in ((k, held[0]), (v, held[1])):
            vals = torch.from_numpy(q8.dequantize_q8_0(*q8.quantize_q8_0(x.float().cpu().numpy())))
            at = 0
            for s, n in enumerate(counts):
                side[s] = torch.cat([side[s], vals[at:at + n]])
                at += n

    def projection(t):
        rows = torch.randn(t, HQ + 2 * HKV, D, generator=g).to(td).cuda()
        return rows[:, :HQ], rows[:, HQ:HQ + HKV], rows[:, HQ + HKV:]

    # prompts
    qsl = _span.starts(lens)
    q, k, v = projection(int(qsl[-1]))
    out = torch.empty(q.shape, dtype=td, device="cuda")
    nb.ns_prompt_attn(q, k, v, _gpu.dev_ints(qsl, np.int32), SCALE, out, ws)
    append(k.contiguous(), v.contiguous(), lens, lens)
    ref = torch.cat([_span.attend(q[a:b].cpu(), k[a:b].cpu(), v[a:b].cpu(), SCALE) for a, b in zip(qsl, qsl[1:])])
    _span.compare(out, ref, dtype, "prompts")

    # two rounds of drafts
    ctx = lens.copy()
    for step in range(2):
        drafts = np.array([3, 5, 0, 2])
        spans = drafts + 1  # the last accepted token and the drafts behind it
        ctx = ctx + spans
        qsl = _span.starts(spans)
        q, k, v = projection(int(qsl[-1]))
        q = q.contiguous()
        append(k.contiguous(), v.contiguous(), ctx, spans)
        out = torch.empty_like(q)
        nb.ns_paged_attn_prefill_q8_0(q, _gpu.dev_ints(qsl, np.int32), *pools, bt, _gpu.dev_ints(ctx, np.int32),
                                      SCALE, out, ws)
        ref = torch.cat([_span.attend(q[a:b].cpu(), held[0][s], held[1][s], SCALE)
                         for s, (a, b) in enumerate(zip(qsl, qsl[1:]))])
        _span.compare(out, ref, dtype, f"drafts {step}", q8=True)
        # the model's head: one row of logits per query row
        head = torch.randn(HQ * D, 1000, generator=g).cuda() * 0.3
        p = torch.softmax(out.float().flatten(1) @ head, -1)
        mine = np.concatenate([np.arange(a, b - 1) for a, b in zip(qsl, qsl[1:])])
        dq = torch.softmax(torch.log(p[mine]) + 0.5 * torch.randn(len(mine), 1000, generator=g).cuda(), -1)
        x = dq.argmax(-1).to(torch.int32)
        dsl = _span.starts(drafts)
        u, r = torch.rand(len(mine), generator=g).cuda(), torch.rand(S, generator=g).cuda()
        toks = torch.empty(len(p), dtype=torch.int32, device="cuda")
        num = torch.empty(S, dtype=torch.int32, device="cuda")
        nb.ns_verify_drafts(p, dq, x, _gpu.dev_ints(dsl, np.int32), u, r, toks, num)
        want = _span.verify(p.cpu().numpy(), dq.cpu().numpy(), x.cpu().numpy(), dsl, u.cpu().numpy(), r.cpu().numpy())
        assert np.array_equal(toks.cpu().numpy(), want[0]) and np.array_equal(num.cpu().numpy(), want[1])
        # the rejected drafts' tokens leave the cache: the length goes back
        ctx = ctx - (drafts - want[1])
        for side in held:
            for s in range(S):
                side[s] = side[s][:ctx[s]]

    # read back, and serve as the prefix of a new prompt
    ksl = _span.starts(ctx)
    kr = torch.empty(int(ksl[-1]), HKV, D, dtype=td, device="cuda")
    vr = torch.empty_like(kr)
    nb.ns_kv_gather_q8_0(*pools, bt, _gpu.dev_ints(ksl, np.int32), kr, vr)
    want = _gpu.round_to_dtype(torch.cat(held[0]).numpy(), dtype)
    assert np.array_equal(_gpu.to_f64(kr), want)
    new = np.array([9, 1, 30, 4])
    qsl = _span.starts(new)
    q, k, v = projection(int(qsl[-1]))
    ks = torch.cat([t for s in range(S) for t in (kr[ksl[s]:ksl[s + 1]], k[qsl[s]:qsl[s + 1]])])
    vs = torch.cat([t for s in range(S) for t in (vr[ksl[s]:ksl[s + 1]], v[qsl[s]:qsl[s + 1]])])
    full = _span.starts(ctx + new)
    out = torch.empty(q.shape, dtype=td, device="cuda")
    nb.ns_prompt_attn(q, ks, vs, _gpu.dev_ints(qsl, np.int32), SCALE, out, ws, key_start_loc=_gpu.dev_ints(full, np.int32))
    ref = torch.cat([_span.attend(q[qsl[s]:qsl[s + 1]].cpu(), ks[full[s]:full[s + 1]].cpu(),
                                  vs[full[s]:full[s + 1]].cpu(), SCALE) for s in range(S)])
    _span.compare(out, ref, dtype, "prefix")
    _gpu.assert_no_device_status()
