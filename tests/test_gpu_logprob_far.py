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
    row = np.repeat(np.arange(len(z)), np.diff(rp))
    m = z.max(axis=1)
    zm = z[row, ids] - np.where(np.isfinite(m), m, 0)[row]
    finite = np.isfinite(logp)
    _near(g[0], logp, S + U * (np.abs(np.where(finite, zm, 0)) + np.abs(np.where(finite, logp, 0))), "logp")
    _near(g[1], lse, S + 2 * U * np.abs(np.where(np.isfinite(lse), lse, 0)), "lse")
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


def _far_rows(N, dt, rng):
    """Rows whose lse is too coarse to hold log S: of the type's lowest value, of that and
    -inf, around +-70,000, 10^6, 10^30 and just beyond +-65,536."""
    low = float(torch.finfo({"f32": torch.float32, "bf16": torch.bfloat16}[dt]).min)
    half = rng.random(N) < 0.5
    near = lambda c: c + rng.standard_normal(N) * 2 if dt == "f32" else np.where(half, c, c + 512)  # noqa: E731
    rows = [np.full(N, low), np.where(half, low, -np.inf), near(70_000.0), near(-70_000.0), near(65_540.0), near(-65_600.0),
            near(1e6), np.full(N, -1e30), np.where(half, 1e30, -1e30), np.full(N, -low), rng.standard_normal(N),
            np.where(half, low, 1.0), np.where(half, -70_000.0, -np.inf)]
    rows[-1][N // 2] = -70_000.0
    return np.stack(rows)


def _check_grad(got, z, rp, ids, g, gh, dt):
    """p = e^((z - lse) - log S'), S' the row's sum of e^(z - lse): off by 2^-18 of itself for
    the sum, u |z - lse| and u |log p| for the two differences and a few u for the
    exponential; log p by the same amounts; the entropy by 2^-17 (1 + H); sums over a
    list of m terms by m u; then half a step of the output type."""
    ref = O.logprob_backward(z, rp, ids, g, gh)
    _, _, Hr, _, _ = O.logprob(z, np.zeros(len(z) + 1, np.int64), [], 0)
    m = z.max(axis=1)
    lp = z - np.where(np.isfinite(m), m, 0.0)[:, None]
    e = np.exp(lp)
    p = e / np.where(e.sum(axis=1) > 0, e.sum(axis=1), 1.0)[:, None]
    lp = np.where(p > 0, np.abs(np.log(np.where(p > 0, p, 1.0))), 0.0)
    row = np.repeat(np.arange(len(z)), np.diff(rp))
    G, Ga = np.zeros(len(z)), np.zeros(z.shape)
    np.add.at(G, row, np.abs(g))
    np.add.at(Ga, (row, ids), np.abs(g))
    gha, Hc = np.abs(gh)[:, None], Hr[:, None]
    m = 8 + int(np.diff(rp).max())
    rel = S + U * (m + 4 * lp)
    tol = (torch.finfo(torch.bfloat16 if dt == "bf16" else torch.float32).eps / 2 * np.abs(ref) + U * m * Ga
           + 2 * rel * p * (G[:, None] + gha * (lp + Hc)) + p * gha * (rel + 2 * S * (1 + Hc)) + 1e-37)
    _near(got, ref, tol, "d_logits")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("N", [1, 70, 1000, 2000, 9000, 70_001, 300_000])
def test_gradient_where_lse_cannot_hold_the_sum(N, dt):
    rng = np.random.default_rng(N)
    r = _far_rows(N, dt, rng)
    zt, z = _logits(r, dt, offset=N % 3)
    rp, ids = _lists([min(3, N)] * len(r), N, rng)
    g, gh = rng.standard_normal(len(ids)).astype(np.float32), rng.standard_normal(len(r)).astype(np.float32)
    out = _run(zt, rp, ids, 0)
    _check(out, z, rp, ids, 0)
    _, lse, ent, _, _ = out
    dev = lambda a: torch.as_tensor(a, device="cuda")  # noqa: E731
    outs = []
    for _ in range(2):
        dz = torch.full_like(zt, 9.0)
        H.haste_logprob_backward(zt, lse, ent, dev(rp), dev(ids), dev(g), dev(gh), dz)
        outs.append(dz)
    assert torch.equal(*outs)
    _check_grad(to_np64(outs[0]), z, rp, ids, g, gh, dt)


@pytest.mark.parametrize("N", [2 ** 31 - 1, 2 ** 31 - 9])
def test_longest_row(N):
    """One bf16 row of as many labels as there are ids: the sums, the alternatives and the
    gradient at both ends and past 2^30, by closed forms."""
    z = torch.full((1, N), float("-inf"), dtype=torch.bfloat16, device="cuda")
    at = [0, 5, 2 ** 30 - 1, 2 ** 30, N - 2, N - 1]
    v = torch.tensor([1.0, 0.0, 2.0, 0.5, 2.0, 1.0])
    z[0, torch.tensor(at, device="cuda")] = v.bfloat16().cuda()
    p = torch.softmax(v.double(), 0)
    lp = torch.log_softmax(v.double(), 0)
    ids = np.array([N - 1, 7, 2 ** 30, 0], np.int32)
    rp = np.array([0, 4], np.int32)
    logp, lse, ent, tl, ti = _run(z, rp, ids, 8)
    assert abs(lse.item() - torch.logsumexp(v.double(), 0).item()) < 2 * S
    assert abs(ent.item() + (p * lp).sum().item()) < 4 * S
    assert np.allclose(logp.cpu(), [lp[5], -np.inf, lp[3], lp[0]], atol=2 * S)
    assert ti[0].tolist() == [2 ** 30 - 1, N - 2, 0, N - 1, 2 ** 30, 5, 1, 2]
    assert np.allclose(tl[0, :6].cpu(), lp[[2, 4, 0, 5, 3, 1]], atol=2 * S) and (tl[0, 6:] == -np.inf).all()
    dz = torch.empty_like(z)
    dev = lambda a: torch.as_tensor(a, device="cuda")  # noqa: E731
    H.haste_logprob_backward(z, lse, None, dev(rp), dev(ids), dev(np.array([3, 5, 2, 1], np.float32)), None, dz)
    want = -11 * p
    want[5] += 3
    want[3] += 2
    want[0] += 1
    assert np.allclose(dz[0, torch.tensor(at, device="cuda")].double().cpu(), want, rtol=2.0 ** -8 + 2.0 ** -16)
    assert dz[0, 7].item() == 5.0 and sum((c != 0).sum().item() for c in dz[0].split(2 ** 28)) == 7
