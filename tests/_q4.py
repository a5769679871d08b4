"""Plain forms of the q4_0 cache and of the rotary append, and the inputs their tests
share.  numpy and torch in double precision (fp32 step by step where the format decides
in fp32); they share no code with the CUDA library."""
from __future__ import annotations

import numpy as np
import torch

import _gpu
from _span import TORCH, attend
from paged_kv_decode_ns_gb300 import workloads as wl

F32 = np.float32


def quantise(x):
    """Rows x [..., D] (float32 values) -> (codes uint8 [..., D/2], steps float16 [..., D/32])."""
    b = np.asarray(x, F32).reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    at = np.abs(b).argmax(-1)
    m = np.take_along_axis(b, at[..., None], -1)[..., 0]
    m = np.where((b == np.abs(m)[..., None]).any(-1), np.abs(m), m).astype(F32)  # of +a and -a the positive one
    with np.errstate(all="ignore"):
        d = (m / F32(-8)).astype(F32)
        s = np.clip(d, -65504, 65504).astype(np.float16)
        inv = np.where(s != 0, F32(1) / d, F32(0)).astype(F32)
        y = ((b * inv[..., None]).astype(F32) + F32(8.5)).astype(F32)
        c = np.minimum(np.floor(y), 15)
    c = np.where((s == 0)[..., None], 8, c)
    bad = ~np.isfinite(b).all(-1)
    s = np.where(bad, np.float16(np.nan), s)
    c = np.where(bad[..., None], 8, c).astype(np.uint8).reshape(x.shape)
    return c[..., 0::2] | (c[..., 1::2] << 4), s


def values(codes, steps):
    """float64 [..., D]."""
    c = np.stack((codes & 15, codes >> 4), -1).reshape(*steps.shape, 32).astype(np.float64) - 8
    return (c * steps.astype(np.float64)[..., None]).reshape(*steps.shape[:-1], 32 * steps.shape[-1])


def rotate(x, cos_sin, pos, interleaved):
    """Rows x [T, H, D] in float32, each product and sum rounded to it."""
    y = np.asarray(x, F32).copy()
    half = cos_sin.shape[1] // 2
    c, s = cos_sin[pos, None, :half].astype(F32), cos_sin[pos, None, half:].astype(F32)
    i = np.arange(half)
    lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    a, b = y[..., lo].copy(), y[..., hi].copy()
    with np.errstate(all="ignore"):
        y[..., lo] = (a * c).astype(F32) - (b * s).astype(F32)
        y[..., hi] = (b * c).astype(F32) + (a * s).astype(F32)
    return y


def table(positions, rotary, base=10000.0):
    angle = np.arange(positions)[:, None] * base ** (-np.arange(0, rotary, 2) / rotary)
    return np.concatenate((np.cos(angle), np.sin(angle)), -1).astype(F32)


def to16(x, dtype):
    """float values -> a torch tensor of the type (one rounding)."""
    return torch.from_numpy(np.ascontiguousarray(x)).to(TORCH[dtype])


def f32(t):
    return t.detach().cpu().float().numpy()


class Cache:
    """Sequences of `lens` tokens in a q4_0 pool of shuffled blocks; slots that no token fills hold
    codes 0xa5 and a NaN step."""

    def __init__(self, rng, lens, hkv=2, bs=16, d=64, amp=1.0, spare=2):
        self.lens = list(lens)
        need = [max(1, -(-n // bs)) for n in lens]
        nb = sum(need) + spare
        order = rng.permutation(nb)
        self.tables = np.full((len(lens), max(need)), -1, np.int32)
        self.kc = np.full((nb, hkv, bs, d // 2), 0xa5, np.uint8)
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
            for codes, steps, keep in ((self.kc, self.ks, self.k), (self.vc, self.vs, self.v)):
                x = rng.standard_normal((n, hkv, d)).astype(F32) * F32(amp)
                c, st = quantise(x)
                codes[blocks[p // bs], :, p % bs] = c
                steps[blocks[p // bs], :, p % bs] = st
                keep.append(torch.from_numpy(values(c, st)))

    def dev(self):
        return [torch.from_numpy(a).cuda() for a in (self.kc, self.ks, self.vc, self.vs, self.tables)]


def attend_all(q, spans, cache, scale):
    """fp64 [T, Hq, D]: the last n of each sequence's tokens over its first L; spans [(n, L)]."""
    out, at = [], 0
    for s, (n, L) in enumerate(spans):
        out.append(attend(q[at:at + n], cache.k[s][:L], cache.v[s][:L], scale))
        at += n
    return torch.cat(out)


# Relative L2 against the rounded exact value, bf16 outputs of the q4_0 decode.  An error d of an
# element moves it across a rounding border with probability |d| / ulp, by one ulp, so
# E (difference)^2 = E|d| ulp.  One rounding to fp16 (the weight times its step; half a step is 2^-11,
# uniform) of each key's share, with independent signs, makes d of standard deviation 2^-11 / sqrt(3) =
# 2.8e-4 of the element at most; the mean ulp of a bf16 value is 2^-7 / (2 ln 2) = 5.6e-3 of it:
# sqrt(2.8e-4 * 5.6e-3) = 1.25e-3.  (fp16's ulp is an eighth: 4.4e-4, below the 1e-3 of the others.)
REL_BF16 = 1.25e-3


def compare(got, ref64, dtype, what=""):
    """The tolerance of the other attention tests, with REL_BF16 for bf16."""
    if dtype != wl.BF16:
        return _gpu.compare(got, ref64, dtype, what)
    g, r = _gpu.to_f64(got).reshape(ref64.shape), _gpu.round_to_dtype(ref64, dtype)
    assert np.all(np.isfinite(g)), f"{what}: non-finite output"
    excess = float(np.max(np.abs(g - ref64) - 0.5 * _gpu.ulp(ref64, dtype), initial=0.0))
    rel = float(np.linalg.norm(g - r) / max(np.linalg.norm(r), 1e-30))
    assert excess <= _gpu.MAX_ABS, f"{what}: max-abs {excess:.3g} beyond the output rounding"
    assert rel <= REL_BF16, f"{what}: rel-L2 {rel:.3g}"


def same_bits(a, b):
    a, b = torch.as_tensor(a).cpu().contiguous(), torch.as_tensor(b).cpu().contiguous()
    return a.dtype == b.dtype and a.shape == b.shape and torch.equal(a.flatten().view(torch.uint8), b.flatten().view(torch.uint8))


def status():
    from paged_kv_decode_ns_gb300 import binding as nb
    return nb.ns_get_device_status(clear=True)
