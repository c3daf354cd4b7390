"""Softmax reading of logits far from zero, where fp32 numbers are coarse, against the
fp64 oracle.

Around 65,536 fp32 numbers are 2^-8 or 2^-7 apart, yet z - m is exact there, so log p =
(z - m) - log S keeps the error that it has near zero: u |z - m| + u |log p| and what the
sums are off by, 2^-18 of themselves (u = 2^-24); the entropy likewise.  Only lse itself
rounds at its own size.
"""
import numpy as np
import pytest

from oracle import oracle as O
from structured_sparse_output_b200 import haste as H
from tests.helpers import to_np64
from tests.test_gpu_logprob import U, _lists, _logits, _near, _run

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

S = 2.0 ** -18


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    H.lib()
    yield
    torch.cuda.synchronize()
    assert H.haste_device_status() == H.HASTE_OK


def _check(out, z, rp, ids, k):
    logp, lse, ent, tl, ti = O.logprob(z, rp, ids, k)
    g = [None if t is None else to_np64(t) for t in out]
    m = z.max(axis=1)
    row = np.repeat(np.arange(len(z)), np.diff(rp))
    _near(g[0], logp, S + U * (np.abs(z[row, ids] - m[row]) + np.abs(logp)), "logp")
    _near(g[1], lse, S + 2 * U * np.abs(lse), "lse")
    _near(g[2], ent, 2 * S * (1 + ent), "entropy")
    if k:
        assert np.array_equal(g[4].astype(np.int64), ti), "alternatives"
        _near(g[3], tl, S + 2 * U * np.abs(tl), "top_logp")


BLOCK = 4096      # fp32 logits of one block of a row


def _rising(B, n_blocks, centre, rng):
    """Rows whose maximum passes `centre` between blocks, in steps of 0.1 to 3 a block; every
    fourth row falls, so that only the join of its parts passes it."""
    step, at = rng.uniform(0.1, 3, (B, 1)), rng.uniform(-0.5, 0.5, (B, 1))
    base = centre + (np.arange(n_blocks) - n_blocks / 2 + at) * step
    r = np.repeat(base, BLOCK, axis=1) - rng.exponential(1.0, (B, n_blocks * BLOCK))
    r[3::4] = r[3::4, ::-1]
    return r


@pytest.mark.parametrize("centre", [65_536.0, -65_536.0, 60_000.0, -60_000.0, 9_000.0, 300.0])
@pytest.mark.parametrize("B,n_blocks", [(32, 3), (64, 8), (128, 6), (4, 12), (1, 40), (3, 64)])
def test_maximum_that_rises_far_from_zero(B, n_blocks, centre):
    """Rows of several blocks by one CTA, and rows split into runs; 65,536 is where the sums'
    exponents change their form."""
    rng = np.random.default_rng(B + n_blocks)
    for k in (0, 5):
        zt, z = _logits(_rising(B, n_blocks, centre, rng), "f32", offset=k)
        rp, ids = _lists([4] * B, z.shape[1], rng)
        ids[::4] = z.argmax(axis=1)      # a likely label in every row
        for b in range(B):
            ids[4 * b:4 * b + 4].sort()
        _check(_run(zt, rp, ids, k), z, rp, ids, k)
