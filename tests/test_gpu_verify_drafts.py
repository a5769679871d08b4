"""GPU: verification of drafted tokens against the definition in fp64.  Tokens and
counts are whole numbers and have to be equal."""
import numpy as np
import pytest
import torch

import _gpu
import _span
from paged_kv_decode_ns_gb300 import binding as nb

pytestmark = pytest.mark.gpu


def softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


class Drafts:
    def __init__(self, counts, vocab, certain=False, seed=0, noise=0.7):
        rng = np.random.default_rng(seed)
        n, s = sum(counts), len(counts)
        self.start = _span.starts(counts)
        logits = 2.0 * rng.standard_normal((n + s, vocab))
        owner = np.repeat(np.arange(s), counts)
        guess = logits[np.arange(n) + owner] + noise * rng.standard_normal((n, vocab))
        self.p = softmax(logits)
        self.q = None if certain else softmax(guess)
        pick = guess if certain else guess + rng.gumbel(size=guess.shape)
        self.drafts = pick.argmax(-1).astype(np.int32) if n else np.zeros(0, np.int32)
        self.accept = rng.random(n, dtype=np.float32)
        self.sample = rng.random(s, dtype=np.float32)

    def dev(self, pad=0, shift=0):
        """On the device; `pad`: rows that far apart beyond their width."""
        def rows(a):
            if a is None:
                return None
            wide = torch.full((a.shape[0], a.shape[1] + pad), float("nan"), device="cuda")
            wide[:, :a.shape[1]] = torch.from_numpy(a)
            return wide[:, :a.shape[1]]
        f = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        return [rows(self.p), rows(self.q), f(self.drafts), f(self.start), f(self.accept), f(self.sample)]

    def run(self, pad=0):
        s = len(self.sample)
        out = torch.full((len(self.drafts) + s,), -9, dtype=torch.int32, device="cuda")
        num = torch.full((s,), -9, dtype=torch.int32, device="cuda")
        nb.ns_verify_drafts(*self.dev(pad), out, num)
        torch.cuda.synchronize()
        return out.cpu().numpy(), num.cpu().numpy()

    def check(self, pad=0):
        tokens, accepted = self.run(pad)
        _gpu.assert_no_device_status()
        want = _span.verify(self.p, self.q, self.drafts, self.start, self.accept, self.sample)
        assert np.array_equal(accepted, want[1])
        assert np.array_equal(tokens, want[0])
        return want


@pytest.mark.parametrize("vocab", [1, 2, 31, 32, 33, 511, 4096, 4097, 50257, 151936])
@pytest.mark.parametrize("certain", [False, True])
def test_verify(vocab, certain):
    counts = [4, 0, 1, 7, 3, 2] if vocab > 20000 else [4, 0, 1, 7, 3, 2, 40, 5, 0, 65] + [3] * 20
    _, accepted = Drafts(counts, vocab, certain, seed=vocab).check()
    if vocab > 2 and not (certain and vocab > 20000):  # a certain draft among 50 000 tokens is seldom accepted
        assert 0 < accepted.sum() < sum(counts)  # both outcomes occur


@pytest.mark.parametrize("pad", [1, 4, 64])
def test_rows_apart(pad):
    Drafts([3, 1, 2] * 6, 1000, seed=pad).check(pad)
    Drafts([3, 1, 2] * 6, 1001, seed=pad).check(pad)


def test_many_sequences():
    Drafts([i % 4 for i in range(700)], 300, seed=9).check()


def test_no_drafts_at_all():
    """Plain sampling: every sequence draws one token."""
    Drafts([0, 0, 0], 5000, seed=1).check()
    Drafts([0], 130, certain=True, seed=2).check()


def test_drawn_tokens_follow_the_weights():
    """Weights that are powers of two: the border of every token is a float, and a
    uniform that lies on a border belongs to the token behind it."""
    vocab, p = 64, np.zeros((4, 64), np.float32)
    p[:, [3, 10, 40, 63]] = [0.5, 0.25, 0.125, 0.125]
    d = Drafts([0, 0, 0, 0], vocab, seed=3)
    d.p = p
    for u, want in ((0.0, 3), (0.49999997, 3), (0.5, 10), (0.75, 40), (0.875, 63), (0.99999994, 63)):
        d.sample = np.full(4, u, np.float32)
        assert (d.check()[0] == want).all()


def test_borders_of_acceptance():
    """u q < p decides: equality rejects, a draft of probability 0 is accepted when the target has any."""
    p = np.array([[0.25, 0.75], [0.5, 0.5]], np.float32)
    for q0, u, x, accepted in ((0.5, 0.5, 0, 0), (0.5, 0.49999997, 0, 1), (0.0, 0.999, 0, 1), (0.0, 0.999, 1, 0),
                              (1.0, 0.25, 0, 0)):
        d = Drafts([1], 2, seed=4)
        d.p, d.q = p, np.array([[q0, 1 - q0]], np.float32)
        d.drafts, d.accept = np.array([x], np.int32), np.array([u], np.float32)
        assert d.check()[1][0] == accepted


def test_degenerate_rows():
    """The draft's distribution leaves nothing of p: p itself is drawn from; a row of
    zeros draws nothing; NaN counts as 0."""
    d = Drafts([1, 1], 100, seed=5)
    d.p[0], d.q[0] = 0, 0
    d.p[0, 7], d.p[0, 9], d.drafts[0], d.q[0, [7, 9, 50]] = 0.25, 0.25, 50, 0.5
    d.accept[0] = 0.9
    d.check()
    d.p[0] = 0
    tokens, accepted = d.run()
    assert accepted[0] == 0 and tokens[0] == -1 and tokens[1] == -1
    d = Drafts([0, 0], 1000, seed=6)
    want, _ = d.check()
    keep = np.ones(1000, bool)
    keep[want[0]] = False
    d.p[0, np.nonzero(d.p[0] < 1e-3)[0][0]] = 0.0
    a, _ = d.check()
    d.p[0, d.p[0] == 0] = np.nan
    b, _ = d.run()
    assert np.array_equal(a, b)


def test_bad_device_data():
    d = Drafts([2, 3, 1], 50, seed=7)
    want, num = _span.verify(d.p, d.q, d.drafts, d.start, d.accept, d.sample)
    keep = d.drafts.copy()
    for bad in (-1, 50, 1 << 30):
        d.drafts = keep.copy()
        d.drafts[3] = bad
        tokens, accepted = d.run()
        assert nb.ns_get_device_status() == 0x80
        assert list(accepted) == [num[0], -1, num[2]] and (tokens[3:7] == -1).all()
        assert np.array_equal(tokens[:3], want[:3]) and np.array_equal(tokens[7:], want[7:])
    d.drafts = keep
    for start in ([0, 2, 5, 7], [-1, 2, 5, 6], [0, 5, 2, 6]):
        d.start = np.array(start, np.int32)
        d.run()
        assert nb.ns_get_device_status() == 0x20


def test_captured():
    d = Drafts([3, 0, 5], 5000, seed=8)
    args = d.dev()
    out = torch.empty(11, dtype=torch.int32, device="cuda")
    num = torch.empty(3, dtype=torch.int32, device="cuda")
    nb.ns_verify_drafts(*args, out, num)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nb.ns_verify_drafts(*args, out, num)
    d.sample, d.accept = d.sample[::-1].copy(), d.accept[::-1].copy()
    args[4].copy_(torch.from_numpy(d.accept))
    args[5].copy_(torch.from_numpy(d.sample))
    g.replay()
    torch.cuda.synchronize()
    want = _span.verify(d.p, d.q, d.drafts, d.start, d.accept, d.sample)
    assert np.array_equal(out.cpu().numpy(), want[0]) and np.array_equal(num.cpu().numpy(), want[1])


def test_refusals():
    d = Drafts([1, 2], 10, seed=9)
    p, q, x, start, a, s = d.dev()
    out, num = torch.empty(5, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        nb.ns_verify_drafts(p.half(), q, x, start, a, s, out, num)
    with pytest.raises(ValueError):
        nb.ns_verify_drafts(p[:4], q, x, start, a, s, out, num)
    with pytest.raises(ValueError):
        nb.ns_verify_drafts(p, q[:, :9], x, start, a, s, out, num)
    with pytest.raises(ValueError):
        nb.ns_verify_drafts(p.t().contiguous().t(), q, x, start, a, s, out, num)
    with pytest.raises(TypeError):
        nb.ns_verify_drafts(p, q, x.long(), start, a, s, out, num)
