"""Plain fp64 forms of the span attention, the cache read-back and the draft
verification, and the inputs their tests share.  Torch in double precision; it
shares no code with the CUDA library."""
from __future__ import annotations

import numpy as np
import torch

import _gpu
from oracle import q8
from paged_kv_decode_ns_gb300 import workloads as wl

TORCH = {wl.F16: torch.float16, wl.BF16: torch.bfloat16}


def attend(q, k, v, scale):
    """q [n, Hq, D] over k, v [L, Hkv, D]: the rows are the last n of L tokens; a
    row that sees no key gives 0."""
    n, hq, d = q.shape
    L, hkv, _ = k.shape
    out = torch.zeros(n, hq, d, dtype=torch.float64)
    for j in range(hq):
        h = j // (hq // hkv)
        z = scale * (q[:, j].double() @ k[:, h].double().T)
        see = torch.arange(L) <= (L - n + torch.arange(n))[:, None]
        top = torch.where(see, z, -torch.inf).amax(-1, keepdim=True) if L else torch.zeros(n, 1)
        w = torch.where(see, torch.exp(z - torch.where(torch.isfinite(top), top, 0.0)), 0.0)
        total = w.sum(-1, keepdim=True)
        # a key that is not seen counts for nothing, whatever it holds
        vals = torch.where(see[..., None], v[:, h].double()[None], 0.0) if not torch.isfinite(v).all() else None
        o = w @ v[:, h].double() if vals is None else (w[..., None] * vals).sum(1)
        out[:, j] = torch.where(total > 0, o / torch.where(total > 0, total, 1.0), 0.0)
    return out


def starts(lens, first=0):
    return np.concatenate([[first], first + np.cumsum(lens)]).astype(np.int32)


# Relative L2 against the rounded exact value, bf16 outputs over a q8_0 cache.  An
# error d of an element moves it across a rounding border with probability |d| / ulp,
# by one ulp, so E (difference)^2 = E|d| ulp.  Three roundings to fp16 (K, V, the
# weights; each half a step 2^-11, uniform) make d of standard deviation sqrt(3)
# 2^-11 / sqrt(3) = 4.9e-4 of the element; E|d| <= that; the mean ulp of a bf16 value is
# 2^-7 / (2 ln 2) = 5.6e-3 of it: sqrt(4.9e-4 * 5.6e-3) = 1.66e-3.  (fp16's ulp is an
# eighth: 5.9e-4, below the 1e-3 of the other attention tests.)
REL_Q8_BF16 = 1.66e-3


def compare(got, ref, dtype, what="", q8=False):
    """The tolerance of the other attention tests; `q8`: over a q8_0 cache."""
    if not (q8 and dtype == wl.BF16):
        return _gpu.compare(got, ref.numpy(), dtype, what)
    g, r64 = _gpu.to_f64(got), ref.numpy()
    r = _gpu.round_to_dtype(r64, dtype)
    assert np.all(np.isfinite(g)), f"{what}: non-finite output"
    excess = float(np.max(np.abs(g - r64) - 0.5 * _gpu.ulp(r64, dtype), initial=0.0))
    rel = float(np.linalg.norm(g - r) / max(np.linalg.norm(r), 1e-30))
    assert excess <= _gpu.MAX_ABS, f"{what}: max-abs {excess:.3g} beyond the output rounding"
    assert rel <= REL_Q8_BF16, f"{what}: rel-L2 {rel:.3g}"


class Q8Cache:
    """Sequences of `lens` tokens in a q8_0 pool of shuffled blocks; slots that no
    token fills hold code 77 and a NaN scale."""

    def __init__(self, rng, lens, hkv=2, bs=16, d=64, amp=1.0, spare=2):
        self.lens = list(lens)
        need = [max(1, -(-n // bs)) for n in lens]
        nb = sum(need) + spare
        order = rng.permutation(nb)
        self.tables = np.full((len(lens), max(need)), -1, np.int32)
        self.kc = np.full((nb, hkv, bs, d), 77, np.int8)
        self.vc = self.kc.copy()
        self.ks = np.full((nb, hkv, bs, d // 32), np.nan, np.float16)
        self.vs = self.ks.copy()
        self.k, self.v = [], []
        at = 0
        for s, n in enumerate(lens):
            blocks = order[at:at + -(-n // bs)]
            at += len(blocks)
            self.tables[s, :len(blocks)] = blocks
            p = np.arange(n)
            for codes, scales, keep in ((self.kc, self.ks, self.k), (self.vc, self.vs, self.v)):
                x = rng.standard_normal((n, hkv, d)).astype(np.float32) * np.float32(amp)
                c, sc = q8.quantize_q8_0(x)
                codes[blocks[p // bs], :, p % bs] = c
                scales[blocks[p // bs], :, p % bs] = sc
                keep.append(torch.from_numpy(q8.dequantize_q8_0(c, sc)))

    def dev(self):
        return [torch.from_numpy(a).cuda() for a in (self.kc, self.ks, self.vc, self.vs, self.tables)]


def verify(p, q, drafts, start, accept, sample):
    """The definition, sequence by sequence, in fp64."""
    tokens, accepted = np.full(p.shape[0], -1, np.int32), []
    for s, (a, b) in enumerate(zip(start[:-1], start[1:])):
        took, w = b - a, p[b + s].astype(np.float64)
        for i in range(a, b):
            x = drafts[i]
            qi = q[i].astype(np.float64) if q is not None else (np.arange(p.shape[1]) == x).astype(np.float64)
            pi = p[i + s].astype(np.float64)
            if not float(accept[i]) * qi[x] < pi[x]:
                took, w = i - a, np.maximum(pi - qi, 0.0)
                if not w.sum() > 0:
                    w = np.maximum(pi, 0.0)
                break
        cum = np.cumsum(w)
        over = np.nonzero(cum > float(sample[s]) * cum[-1])[0]
        tokens[a + s:a + s + took] = drafts[a:a + took]
        tokens[a + s + took] = over[0] if len(over) else -1
        accepted.append(took)
    return tokens, np.array(accepted, np.int32)
