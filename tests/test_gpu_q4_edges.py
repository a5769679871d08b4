"""GPU: the q4_0 calls where the others' tests do not look: repeated small calls, scores of any size."""
import numpy as np
import pytest
import torch

import _gpu
import _q4
from _q4 import wl
from paged_kv_decode_ns_gb300 import binding as nb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[200, 64, 17, 1], [333] * 32, [4096, 5]])
def test_few_sequences_many_times(lens, d):
    """Up to 32 sequences: the warps of a CTA meet at no barrier before they leave records of cut pairs to each
    other.  300 calls, each into an output of its own, behind kernels that leave the SMs at different times."""
    rng = np.random.default_rng(1)
    cache = _q4.Cache(rng, lens, 2, 16, d)
    q = _q4.to16(rng.standard_normal((len(lens), 14, d)).astype(np.float32), wl.F16)
    ref = _q4.attend_all(q, [(1, n) for n in lens], cache, d ** -0.5).numpy()
    pools, cl, ws, qd = cache.dev(), _gpu.dev_ints(lens, np.int32), nb.alloc_workspace(len(lens), 14, 2, d), q.cuda()
    outs = torch.full((300, *q.shape), float("nan"), dtype=q.dtype, device="cuda")
    load = torch.zeros(1 << 22, device="cuda")
    for i in range(300):
        if i % 3 == 0:
            load[: 1 + (i * 7919) % load.numel()].add_(1.0)
        nb.ns_paged_attn_decode_q4_0(qd, *pools, cl, d ** -0.5, outs[i], ws)
    torch.cuda.synchronize()
    _q4.compare(outs[0], ref, wl.F16)
    assert (outs.view(torch.int16) == outs[0].view(torch.int16)).all() and _q4.status() == 0


def attend(cache, q, lens, scale, dtype):
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    nb.ns_paged_attn_decode_q4_0(q.cuda(), *cache.dev(), _gpu.dev_ints(lens, np.int32), scale, out,
                                 nb.alloc_workspace(len(lens), q.shape[1], cache.kc.shape[1], q.shape[2]))
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale,amp", [(0.0, 1e-30), (1e-30, 1e-30), (0.125, 1e-37), (1e-38, 1.0), (-1e-30, 1e-20), (0.0, 1e30)])
def test_scores_that_vanish(scale, amp, d):
    """The mean of the values, also beside tokens that are not there: the last tile's, and a bad block's."""
    rng = np.random.default_rng(2)
    lens = [1, 33, 100, 700]
    cache = _q4.Cache(rng, lens, 2, 16, d)
    q = _q4.to16(rng.standard_normal((4, 14, d)).astype(np.float32) * np.float32(amp), wl.BF16)
    ref = _q4.attend_all(q, [(1, n) for n in lens], cache, scale).numpy()
    _q4.compare(attend(cache, q, lens, scale, wl.BF16), ref, wl.BF16)
    assert _q4.status() == 0
    cache.tables[2, 1] = -1
    keep = np.r_[0:16, 32:100]
    ref[2] = _q4.attend(q[2:3], cache.k[2][keep], cache.v[2][keep], scale).numpy()[0]
    _q4.compare(attend(cache, q, lens, scale, wl.BF16), ref, wl.BF16)
    assert _q4.status() == 1
