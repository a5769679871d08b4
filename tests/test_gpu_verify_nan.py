"""GPU: a NaN probability counts as 0 in the verification, in the target's rows and in
the drafts', for the acceptance and for the weights."""
import numpy as np
import pytest

import _gpu
import _span
from test_gpu_verify_drafts import Drafts

pytestmark = pytest.mark.gpu


def check(d):
    """`d` with NaN as it is, against the definition with zeros in their place."""
    tokens, accepted = d.run()
    _gpu.assert_no_device_status()
    zero = lambda a: None if a is None else np.where(np.isnan(a), np.float32(0), a)  # noqa: E731
    want = _span.verify(zero(d.p), zero(d.q), d.drafts, d.start, d.accept, d.sample)
    assert np.array_equal(accepted, want[1]) and np.array_equal(tokens, want[0])
    return want


@pytest.mark.parametrize("vocab", [64, 1000, 1001, 9000])
@pytest.mark.parametrize("n", [5, 400])
def test_nan_anywhere(vocab, n):
    """Rows with NaN strewn over them: the tokens they stand at can be drawn where only q has one."""
    d = Drafts([1 + i % 3 for i in range(n)], vocab, seed=vocab + n)
    rng = np.random.default_rng(vocab)
    for a in (d.p, d.q):
        a[rng.random(a.shape) < 0.2] = np.nan
    want = check(d)
    drawn = 0
    for s, (a, b) in enumerate(zip(d.start[:-1], d.start[1:])):
        if want[1][s] < b - a:  # refused: drawn from max(p - q, 0)
            drawn += bool(np.isnan(d.q[a + want[1][s], want[0][a + s + want[1][s]]]))
    assert drawn > 0 or n < 100


def test_nan_at_the_drafted_token():
    """q(x) = NaN is 0: accepted wherever the target gives x any probability; p(x) = NaN is 0: refused."""
    d = Drafts([1] * 6, 128, seed=3)
    rows = np.arange(6)
    d.p[2 * rows, d.drafts] = [0.0, 1e-6, 0.5, np.nan, np.nan, 0.25]
    d.q[rows, d.drafts] = [np.nan, np.nan, np.nan, 0.5, np.nan, 0.1]
    d.accept[:] = 0.999
    assert list(check(d)[1]) == [0, 1, 1, 0, 0, 1]


def test_rows_of_nan():
    """A draft's row of NaN alone takes nothing away; a target's row of NaN alone draws nothing."""
    d = Drafts([1, 1, 1], 500, seed=4)
    d.q[0] = np.nan
    d.p[0, d.drafts[0]] = 0.0  # refused, drawn from p
    d.p[2], d.q[1, d.drafts[1]] = np.nan, 0.5
    tokens, accepted = check(d)
    assert list(accepted[:2]) == [0, 0] and tokens[0] >= 0 and tokens[2] == -1
