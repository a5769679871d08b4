"""GPU: q4_0 contexts of more than 2^30 tokens, whose tables name two blocks again and again.  The first block's keys lie
along the query, the other one's against it, so that the first 16 tokens have all the weight."""
import numpy as np
import pytest
import torch

import _gpu
import _q4
import _span
from _q4 import wl
from paged_kv_decode_ns_gb300 import binding as nb

pytestmark = pytest.mark.gpu

L = (1 << 30) + 200


@pytest.mark.parametrize("dtype", [wl.F16, wl.BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("spans", [True, False])
def test_far_positions(d, dtype, spans):
    rng = np.random.default_rng(7)
    q = _q4.to16(rng.standard_normal((1, 2, d)).astype(np.float32), dtype)
    # keys of 4 to 7 steps of 1/2, exact in fp16, with the signs of both heads' sum, in which either has a share
    codes = 8 + (np.sign(_q4.f32(q)[0].sum(0)) * np.array([1, -1])[:, None, None, None] * rng.integers(4, 8, (2, 1, 16, 1))).astype(np.uint8)
    kc, ks = codes[..., 0::2] | (codes[..., 1::2] << 4), np.full((2, 1, 16, d // 32), 0.5, np.float16)
    vc, vs = _q4.quantise(rng.standard_normal((2, 1, 16, d)).astype(np.float32))
    exact_k, exact_v = (torch.from_numpy(_q4.values(c, s))[0].transpose(0, 1) for c, s in ((kc, ks), (vc, vs)))
    scores = torch.from_numpy(_q4.values(kc, ks))[:, 0] @ q[0].double().T  # [2, 16, 2]
    assert float(scores[0].min() - scores[1].max()) > 100  # a weight of e^-100 at most
    tables = torch.ones(1, -(-L // 16), dtype=torch.int32, device="cuda")
    tables[0, 0] = 0
    pools = [torch.from_numpy(x).cuda() for x in (kc, ks, vc, vs)]
    lens = _gpu.dev_ints([L], np.int32)
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    if spans:
        nb.ns_paged_attn_prefill_q4_0(q.cuda(), _gpu.dev_ints([0, 1], np.int32), *pools, tables, lens, 1.0, out,
                                      nb.alloc_span_workspace(d))
    else:
        nb.ns_paged_attn_decode_q4_0(q.cuda(), *pools, tables, lens, 1.0, out, nb.alloc_workspace(1, 2, 1, d))
    torch.cuda.synchronize()
    _span.compare(out, _span.attend(q, exact_k, exact_v, 1.0), dtype, q8=True)
    assert _q4.status() == 0
