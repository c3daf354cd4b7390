"""GPU parity of the softmax reading of the logits (haste_logprob and its gradient)
against the fp64 oracle.

Tolerances, from the formulas (u = 2^-24, the fp32 half step):
* log p = (z - m) - log S and lse = m + log S round twice, 2 u (|z| + |lse|) at most;
  S is a sum of positive terms, each e^x with an error of a few u (1 + |x|), summed
  over at most some tens of terms in a row: S is off by less than 2^-18 of itself,
  which log S shows as an absolute 2^-18.
* entropy = log S + T / S, T likewise: 2^-18 (1 + entropy), and its own rounding.
* d_logits = sum g - p c, c = G + gH (log p + H): p = e^(z - lse) is off by
  u (|z| + 2 |lse|) + a few u of itself, c by the rounding of its terms; then half a
  step of the output type.
The alternatives are copies of inputs: their ids must be exact.
"""
import numpy as np
import pytest

from oracle import oracle as O
from structured_sparse_output_b200 import haste as H
from structured_sparse_output_b200 import inputs as I
from tests.helpers import assert_close, to_np64, to_torch

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    H.lib()
    yield
    torch.cuda.synchronize()
    assert H.haste_device_status() == H.HASTE_OK


def _dev(a, dtype=None):
    return torch.as_tensor(np.asarray(a), dtype=dtype, device="cuda")


def _logits(z, dt, offset=0):
    """z on the GPU in type dt, `offset` elements into a larger buffer; and what it holds."""
    t = torch.as_tensor(np.asarray(z, dtype=np.float32)).to(DT[dt])
    buf = torch.full((t.numel() + offset + 64,), float("nan"), dtype=DT[dt], device="cuda")
    v = buf[offset:offset + t.numel()].view(t.shape)
    v.copy_(t)
    return v, t.double().numpy()


def _lists(counts, N, rng, messy=False):
    """CSR lists of the given lengths; messy: any order, with repeats."""
    counts = np.asarray(counts) if messy else np.minimum(counts, N)
    rp = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    ids = [rng.integers(0, N, c) if messy else np.sort(rng.choice(N, c, replace=False)) for c in counts]
    return rp, np.concatenate(ids + [np.zeros(0)]).astype(np.int32)


def _run(zt, rp, ids, k, stream=None):
    B, N = zt.shape
    rp, ids = _dev(rp), _dev(ids)
    f = lambda *s: torch.full(s, 777.0, device="cuda")  # noqa: E731
    out = [f(len(ids)), f(B), f(B), f(B, k) if k else None,
           torch.full((B, k), -7, dtype=torch.int32, device="cuda") if k else None]
    ws = torch.empty(H.haste_logprob_workspace_size(B, N, H.dtype_code(zt), k), dtype=torch.uint8, device="cuda")
    H.haste_logprob(zt, rp, ids, *out, ws, stream=stream)
    return out


def _same_special(got, ref, what):
    assert np.array_equal(np.isnan(got), np.isnan(ref)), what
    inf = np.isinf(ref)
    assert np.array_equal(np.isinf(got), inf) and np.array_equal(got[inf], ref[inf]), what


def _near(got, ref, tol, what):
    _same_special(got, ref, what)
    ok = np.isfinite(ref)
    err = np.abs(got[ok] - ref[ok]) - np.broadcast_to(tol, ref.shape)[ok]
    assert err.size == 0 or err.max() <= 0, (what, err.max())


def _check(out, z, rp, ids, k):
    logp, lse, ent, tl, ti = O.logprob(z, rp, ids, k)
    g = [None if t is None else to_np64(t) for t in out]
    fin = np.where(np.isfinite(lse), np.abs(lse), 0.0)
    row = np.repeat(np.arange(len(z)), np.diff(rp))
    S = 2.0 ** -18

    def tol(lp, b):    # |z| <= |lp| + |lse|
        return S + 2 * U * (np.where(np.isfinite(lp), np.abs(lp), 0) + 2 * fin[b])

    _near(g[0], logp, tol(logp, row), "logp")
    _near(g[1], lse, S + 2 * U * fin, "lse")
    _near(g[2], ent, S * (1 + np.where(np.isfinite(ent), ent, 0)) * 2, "entropy")
    if k:
        assert np.array_equal(g[4].astype(np.int64), ti), "alternatives"
        _near(g[3], tl, tol(tl, np.arange(len(z))[:, None]), "top_logp")


SHAPES = [(1, 1), (3, 2), (5, 33), (2, 100), (7, 255), (4, 1000), (2, 4096), (3, 4097), (300, 513), (2, 8192), (3, 8193),
          (2, 16_384), (2, 16_385), (5, 32_003), (1, 70_001), (2, 262_147), (1, 1_048_583)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("B,N", SHAPES)
def test_logprob_matches_oracle(B, N, dt):
    rng = np.random.default_rng(B * 1000 + N)
    for k in sorted({0, min(1, N), min(5, N), min(64, N)}):
        zt, z = _logits(rng.standard_normal((B, N)) * 3, dt, offset=(3 * k + N) % 9)
        rp, ids = _lists(rng.integers(0, 9, B), N, rng, messy=k % 2 == 1)
        out = _run(zt, rp, ids, k)
        _check(out, z, rp, ids, k)
        again = _run(zt, rp, ids, k)                                  # the same bits on every run
        assert all(a is None or torch.equal(a, b) for a, b in zip(out, again))


def _patterns(N, rng):
    asc = np.linspace(-20, 20, N)
    spike = np.full(N, -np.inf)
    spike[N // 3] = 2.5
    mask = np.where(rng.random(N) < 0.5, -np.inf, rng.standard_normal(N))
    zeros = np.where(rng.random(N) < 0.5, 0.0, -0.0)
    lowest = np.where(rng.random(N) < 0.9, -3.3895314e38, rng.standard_normal(N))
    nan, inf = rng.standard_normal(N), rng.standard_normal(N)
    nan[N // 2], inf[N - 1] = np.nan, np.inf
    blocks = np.repeat(rng.standard_normal((N + 15) // 16), 16)[:N]   # long runs of equal values
    return {"equal": np.full(N, 1.25), "ascending": asc, "descending": asc[::-1], "spike": spike, "masked": mask,
            "none": np.full(N, -np.inf), "signed zeros": zeros, "lowest": lowest, "nan": nan, "inf": inf,
            "huge": rng.standard_normal(N) * 1e37, "blocks": blocks, "one hot": np.where(np.arange(N) == 1, 90.0, 0.0),
            "coarse": np.round(rng.standard_normal(N) * 2) / 2, "nan in none": np.where(np.arange(N) == 0, np.nan, -np.inf)}


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("N", [65, 5000, 40_000, 150_001])
def test_logprob_patterns_ties_and_masks(N, dt):
    rng = np.random.default_rng(N)
    pats = _patterns(N, rng)
    zt, z = _logits(np.stack(list(pats.values())), dt, offset=1)
    rp, ids = _lists([3] * len(z), N, rng)
    for k in (1, 20, 64):
        _check(_run(zt, rp, ids, k), z, rp, ids, k)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_logprob_short_rows(dt):
    """Row lengths and numbers of alternatives around the changes of method: every logit
    ranked, groups of one thread, of several; random, tied, ascending and masked rows."""
    for N in (2, 7, 8, 9, 63, 64, 65, 127, 128, 129, 200, 255, 256, 257, 300, 511, 512, 513, 700, 1024, 1025, 2047, 2049):
        rng = np.random.default_rng(N)
        r = rng.standard_normal((6, N)) * 2
        r[1] = np.round(r[1])
        r[2] = np.sort(r[2])
        r[3, rng.random(N) < 0.9] = -np.inf
        r[4] = 0.5
        r[5, N // 2:] = np.nan
        zt, z = _logits(r, dt, offset=N % 5)
        rp, ids = _lists([2] * 6, N, rng)
        for k in sorted({min(k, N) for k in (1, 5, 16, 17, 40, 64)}):
            _check(_run(zt, rp, ids, k), z, rp, ids, k)


def _many_short_rows(B, N, rng):
    """Random, rounded, ascending, mostly masked, constant, NaN, fully masked, lowest-value
    and far rows in turn."""
    r = rng.standard_normal((B, N)) * 2
    r[1::9] = np.round(r[1::9])
    r[2::9] = np.sort(r[2::9])
    r[3::9][rng.random(r[3::9].shape) < 0.95] = -np.inf
    r[4::9] = 0.5
    r[5::9, N // 2:] = np.nan
    r[6::9] = -np.inf
    r[7::9][rng.random(r[7::9].shape) < 0.5] = -3.3895313892515355e38      # the lowest value of both types
    r[8::9] += 70_000
    return r


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n", [33, 128, 129, 500, 1000, 1024, 1025, 2040, 2048, 2049, 4000, 4089, 4096, 4097])
def test_logprob_many_short_rows(n, dt):
    """Batches of rows of up to 8 KB, one after another and on and off the 16-byte boundary."""
    N = n if dt == "bf16" or n < 130 else n // 2
    B = 1030 if n < 2049 else 1027
    rng = np.random.default_rng(n)
    zt, z = _logits(_many_short_rows(B, N, rng), dt, offset=n % 2 * 3)
    rp, ids = _lists(rng.integers(0, 5, B), N, rng, messy=True)
    for k in (0, 1, 9, 32, 64):
        if k <= N:
            _check(_run(zt, rp, ids, k), z, rp, ids, k)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("N", [70, 700, 1400, 2000])
def test_logprob_and_gradient_of_short_rows_with_infinities(N, dt):
    """+inf, NaN and one or two finite logits in the first, a middle and the last column."""
    rng = np.random.default_rng(N)
    B = 1200
    r = rng.standard_normal((B, N))
    col = np.array([0, N // 2, N - 1])[np.arange(B) % 3]
    one = np.arange(B)
    r[one[0::4], col[0::4]] = np.inf
    r[one[1::4], col[1::4]] = np.nan
    keep = r[one[2::4], col[2::4]]
    r[2::4] = -np.inf
    r[one[2::4], col[2::4]] = keep
    zt, z = _logits(r, dt, offset=N % 3)
    rp, ids = _lists([2] * B, N, rng)
    for k in (1, 6, 33):
        _check(_run(zt, rp, ids, k), z, rp, ids, k)
    _, lse, ent, _, _ = _run(zt, rp, ids, 0)
    g, gh = rng.standard_normal(len(ids)).astype(np.float32), rng.standard_normal(B).astype(np.float32)
    dz = torch.empty_like(zt)
    H.haste_logprob_backward(zt, lse, ent, _dev(rp), _dev(ids), _dev(g), _dev(gh), dz)
    got, ref = to_np64(dz), O.logprob_backward(z, rp, ids, g, gh)
    bad = np.isnan(ref).any(1)
    assert np.isnan(got[bad]).all() and np.isfinite(got[~bad]).all()
    _check_grad(got[~bad], z[~bad], np.arange(0, 2 * (~bad).sum() + 1, 2), ids.reshape(B, 2)[~bad].reshape(-1),
                g.reshape(B, 2)[~bad].reshape(-1), gh[~bad], dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("blocks", [5, 9, 37])
def test_logprob_few_long_rows_around_whole_blocks(blocks, dt):
    """Rows in runs of one 16 KB block, whose last one is short, whole or longer; rows that
    start anywhere; more alternatives than runs and fewer."""
    per = 8192 if dt == "bf16" else 4096
    rng = np.random.default_rng(blocks)
    for more in (0, 1, per // 2 - 1, per // 2, per // 2 + 1, per - 1):
        N, B = blocks * per + more, 3 if blocks < 30 else 2
        r = rng.standard_normal((B, N)) * 2
        r[0] = np.round(r[0])
        r[1, : N - 30] = -np.inf
        for off in (0, more % 7 + 1):
            zt, z = _logits(r, dt, offset=off)
            rp, ids = _lists([3] * B, N, rng)
            for k in (0, 1, 20, 64):
                _check(_run(zt, rp, ids, k), z, rp, ids, k)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_logprob_runs_with_few_or_no_finite_logits(dt):
    """Rows split into runs of which most are masked: the alternatives come from one run,
    from several, or are masked labels in the order of their ids."""
    N, k = 400_003, 64
    r = np.full((5, N), -np.inf)
    r[0, 399_000:399_100] = np.linspace(0, 1, 100)
    r[1, ::20_001] = np.arange(len(range(0, N, 20_001)))
    r[2, N - 1] = 3.0
    r[3, 200_000:200_040] = 1.0
    r[4, :30] = np.nan
    zt, z = _logits(r, dt, offset=3)
    rp, ids = _lists([2] * 5, N, np.random.default_rng(0))
    for kk in (1, 7, k):
        _check(_run(zt, rp, ids, kk), z, rp, ids, kk)


def test_logprob_lists_out_of_range_ids_and_odd_row_ptr():
    rng = np.random.default_rng(3)
    zt, z = _logits(rng.standard_normal((4, 50)), "f32")
    i32 = lambda v: np.array(v, np.int32)  # noqa: E731
    rp, ids = i32([0, 3, 3, 9, 10]), i32([4, -1, 4, 50, 2 ** 31 - 1, 0, 49, 0, -2 ** 31, 7])
    _check(_run(zt, rp, ids, 2), z, rp, ids, 2)
    # entries of row_ptr outside [0, nnz] are kept within it; what no row holds stays
    out = _run(zt, i32([-5, 2, 2, 4, 3]), i32([1, 2, 3, 4, 5]), 0)
    _near(to_np64(out[0])[:4], O.logprob(z, [0, 2, 2, 4, 4], [1, 2, 3, 4], 0)[0], 1e-5, "logp")
    assert out[0][4].item() == 777.0
    out = _run(zt, i32([0, 1, 400, 9, 400]), i32([1, 2, 3, 4, 5]), 0)
    _near(to_np64(out[0]), O.logprob(z, [0, 1, 5, 5, 5], [1, 2, 3, 4, 5], 0)[0], 1e-5, "logp")


def test_logprob_optional_outputs():
    rng = np.random.default_rng(4)
    zt, z = _logits(rng.standard_normal((3, 700)), "bf16")
    _, lse, ent, _, _ = O.logprob(z, [0] * 4, [], 0)
    a, b = torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
    H.haste_logprob(zt, lse=a)
    H.haste_logprob(zt, entropy=b)
    H.haste_logprob(zt)
    assert np.allclose(a.cpu(), lse, atol=1e-5) and np.allclose(b.cpu(), ent, atol=1e-4)
    none = torch.empty(0, device="cuda")
    H.haste_logprob(zt, torch.zeros(4, dtype=torch.int32, device="cuda"), none.int(), none, lse=a)
    assert np.allclose(a.cpu(), lse, atol=1e-5)


def test_logprob_offsets_beyond_32_bits():
    """The last rows start more than 2^32 bytes (and 2^31 elements) into the logits."""
    B, N = 2100, 1_048_583
    z = torch.full((B, N), float("-inf"), dtype=torch.bfloat16, device="cuda")
    z[B - 1, N - 1], z[B - 1, 5], z[B - 2, 77] = 1.0, 1.0, 3.0
    rp, ids = np.zeros(B + 1, np.int32), np.array([77, N - 1], np.int32)
    rp[B - 1:] = [1, 2]
    logp, lse, ent, tl, ti = _run(z, rp, ids, 2)
    assert abs(lse[B - 1].item() - (1 + np.log(2))) < 1e-6 and abs(ent[B - 1].item() - np.log(2)) < 1e-6
    assert lse[B - 2].item() == 3.0 and torch.isinf(lse[:B - 2]).all()
    assert ti[B - 1].tolist() == [5, N - 1] and ti[B - 2].tolist() == [77, 0] and ti[0].tolist() == [0, 1]
    assert np.allclose(logp.cpu(), [0, -np.log(2)], atol=1e-6)
    dz = torch.empty_like(z)
    g = torch.tensor([2.0, 4.0], device="cuda")
    H.haste_logprob_backward(z, lse, None, _dev(rp), _dev(ids), g, None, dz)
    assert dz[B - 1, N - 1].item() == 2.0 and dz[B - 1, 5].item() == -2.0 and dz[B - 2, 77].item() == 0.0
    assert (dz != 0).sum().item() == 2


# ------------------------------------------------------------------ the gradient
def _check_grad(got, z, rp, ids, g, gh, dt):
    ref = O.logprob_backward(z, rp, ids, g, gh)
    _, lse, H_, _, _ = O.logprob(z, np.zeros(len(z) + 1, np.int64), [], 0)
    fin = np.where(np.isfinite(lse), lse, 0.0)[:, None]
    zf = np.where(np.isfinite(z), np.abs(z), 0.0)
    lp = np.where(np.isfinite(z), z - fin, 0.0)
    p = np.where(np.isfinite(lse)[:, None], np.exp(np.where(np.isfinite(z), z - fin, -np.inf)), 0.0)
    row = np.repeat(np.arange(len(z)), np.diff(rp))
    G, Ga = np.zeros(len(z)), np.zeros(z.shape)
    ok = (ids >= 0) & (ids < z.shape[1])
    np.add.at(G, row[ok], np.abs(g[ok]))
    np.add.at(Ga, (row[ok], ids[ok]), np.abs(g[ok]))
    gha = np.zeros(len(z)) if gh is None else np.abs(gh)
    c = G[:, None] + gha[:, None] * (np.abs(lp) + np.abs(np.where(np.isfinite(H_), H_, 0))[:, None])
    m = 8 + int(np.diff(rp).max(initial=0))                       # terms of the sums over a row's list
    tol = (torch.finfo(DT[dt]).eps / 2 * np.where(np.isfinite(ref), np.abs(ref), 0) + U * m * Ga
           + U * (m + 8 + 2 * zf + 4 * np.abs(fin)) * 2 * p * c + 1e-37)
    # c can be 0 (one label left: log p = H = 0) while log p is rounded: lse = m + log S
    # twice, 2 u |lse|, and z - lse once, u (|z| + |lse|); its part of c is gH times that.
    tol = tol + p * gha[:, None] * U * (zf + 3 * np.abs(fin))
    _near(got, ref, tol, "d_logits")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("B,N", SHAPES)
def test_gradient_matches_oracle(B, N, dt):
    rng = np.random.default_rng(B * 7 + N)
    for case in range(3):
        zt, z = _logits(rng.standard_normal((B, N)) * 3, dt, offset=(case + N) % 9)
        rp, ids = _lists(rng.integers(0, 9, B), N, rng, messy=case == 1)
        g, gh = rng.standard_normal(len(ids)).astype(np.float32), rng.standard_normal(B).astype(np.float32)
        _, lse, ent, _, _ = _run(zt, rp, ids, 0)
        buf = torch.full((B * N + 32,), 55.0, dtype=DT[dt], device="cuda")
        dz = buf[case:case + B * N].view(B, N)
        H.haste_logprob_backward(zt, lse, ent if case else None, _dev(rp), _dev(ids), _dev(g),
                                 _dev(gh) if case else None, dz)
        _check_grad(to_np64(dz), z, rp, ids, g, gh if case else None, dt)
        assert (buf[:case] == 55).all() and (buf[case + B * N:] == 55).all()      # nothing beside the output


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("N", [65, 40_000])
def test_gradient_patterns(N, dt):
    rng = np.random.default_rng(N)
    pats = _patterns(N, rng)
    zt, z = _logits(np.stack(list(pats.values())), dt, offset=1)
    rp, ids = _lists([4] * len(z), N, rng, messy=True)
    ids[3::4] = ids[2::4]                                             # a repeat in every row
    ids[1] = -1
    g, gh = rng.standard_normal(len(ids)).astype(np.float32), rng.standard_normal(len(z)).astype(np.float32)
    _, lse, ent, _, _ = _run(zt, rp, ids, 0)
    outs = []
    for _ in range(2):
        dz = torch.full_like(zt, 9.0)
        H.haste_logprob_backward(zt, lse, ent, _dev(rp), _dev(ids), _dev(g), _dev(gh), dz)
        outs.append(dz)
    a, b = (o.view(torch.int16 if dt == "bf16" else torch.int32) for o in outs)
    assert torch.equal(a, b)
    _check_grad(to_np64(outs[0]), z, rp, ids, g, gh, dt)


def test_gradient_long_list_and_no_terms():
    rng = np.random.default_rng(8)
    zt, z = _logits(rng.standard_normal((3, 3000)), "f32")
    rp, ids = _lists([2500, 1], 3000, rng, messy=True)
    rp, ids = np.concatenate([rp, [rp[-1] + 3000]]).astype(np.int32), np.concatenate([ids, np.arange(3000, dtype=np.int32)])
    g = rng.standard_normal(len(ids)).astype(np.float32)
    _, lse, ent, _, _ = _run(zt, rp, ids, 0)
    dz = torch.empty_like(zt)
    H.haste_logprob_backward(zt, lse, None, _dev(rp), _dev(ids), _dev(g), None, dz)
    _check_grad(to_np64(dz), z, rp, ids, g, None, "f32")
    H.haste_logprob_backward(zt, lse, None, None, None, None, None, dz)
    assert not dz.any()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 33, 1000, 1025, 2048, 4089, 4096])
def test_gradient_many_short_rows(n, dt):
    N = n if dt == "bf16" or n < 130 else n // 2
    B = 1030
    rng = np.random.default_rng(n + 5)
    r = _many_short_rows(B, N, rng)
    zt, z = _logits(r, dt, offset=n % 2 * 3)
    counts = rng.integers(0, 5, B)
    counts[::50] = rng.integers(30, 600, len(counts[::50]))                # with repeats, in any order
    rp, ids = _lists(counts, N, rng, messy=True)
    for b in range(0, B, 3):
        ids[rp[b]:rp[b + 1]] = np.sort(ids[rp[b]:rp[b + 1]])
    ids[rng.random(len(ids)) < 0.02] = N + 7
    g, gh = rng.standard_normal(len(ids)).astype(np.float32), rng.standard_normal(B).astype(np.float32)
    _, lse, ent, _, _ = _run(zt, rp, np.minimum(ids, N - 1), 0)
    buf = torch.full((B * N + 32,), 55.0, dtype=DT[dt], device="cuda")
    for off in (0, n % 2 * 3):
        dz = buf[off:off + B * N].view(B, N)
        H.haste_logprob_backward(zt, lse, ent, _dev(rp), _dev(ids), _dev(g), _dev(gh), dz)
        _check_grad(to_np64(dz), z, rp, ids, g, gh, dt)
        assert (buf[off + B * N:] == 55).all()
        buf.fill_(55.0)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("N", [60, 33_000, 140_003])
def test_gradient_lists_in_any_order(N, dt):
    """Long and short lists that do not ascend: shuffled without a repeat, labels 32,768
    apart, one label throughout, two in turn, a repeat at both ends, ids outside the row."""
    rng = np.random.default_rng(N + 1)
    apart = np.arange(N % 32_768 % 50, N, 32_768)
    lists = [rng.permutation(N)[:n] for n in (31, 32, 33, 60, 127, 128, 129, 300, 2_000)]
    lists += [rng.permutation(np.concatenate([apart, apart, rng.integers(0, N, 200)])), np.full(700, N - 1),
              np.tile([N - 1, 0], 130), rng.integers(0, N, 515), np.array([3, 2]), np.array([2, 2]), np.arange(50)[::-1],
              np.arange(0), rng.integers(-N, 2 * N, 400)]
    end = rng.permutation(N)[:257]
    end[-1] = end[0]
    lists.append(end)
    rp = np.concatenate([[0], np.cumsum([len(x) for x in lists])]).astype(np.int32)
    ids = np.concatenate(lists).astype(np.int32)
    zt, z = _logits(rng.standard_normal((len(lists), N)) * 2, dt, offset=3)
    g, gh = rng.standard_normal(len(ids)).astype(np.float32), rng.standard_normal(len(z)).astype(np.float32)
    _, lse, ent, _, _ = _run(zt, rp, np.clip(ids, 0, N - 1), 0)
    outs = []
    for _ in range(2):
        dz = torch.full_like(zt, 9.0)
        H.haste_logprob_backward(zt, lse, ent, _dev(rp), _dev(ids), _dev(g), _dev(gh), dz)
        outs.append(dz)
    assert torch.equal(*outs)
    _check_grad(to_np64(outs[0]), z, rp, ids, g, gh, dt)


def test_gradient_against_differences():
    """Central differences of the GPU's own forward values on fp32 logits."""
    rng = np.random.default_rng(9)
    z = rng.standard_normal((2, 12)).astype(np.float32)
    rp, ids = np.array([0, 2, 3], np.int32), np.array([3, 7, 0], np.int32)
    g, gh = rng.standard_normal(3), rng.standard_normal(2)

    def f(z):
        out = _run(_logits(z, "f32")[0], rp, ids, 0)
        return float(g @ out[0].double().cpu().numpy() + gh @ out[2].double().cpu().numpy())

    zt = _logits(z, "f32")[0]
    _, lse, ent, _, _ = _run(zt, rp, ids, 0)
    dz = torch.empty_like(zt)
    H.haste_logprob_backward(zt, lse, ent, _dev(rp), _dev(ids), _dev(g, torch.float32), _dev(gh, torch.float32), dz)
    h = 2.0 ** -6    # truncation h^2 f''' / 6 < 4e-4, rounding 5 * 2^-18 / h < 2e-3
    for b in range(2):
        for j in range(12):
            a, c = z.copy(), z.copy()
            a[b, j] += h
            c[b, j] -= h
            assert abs((f(a) - f(c)) / (2 * h) - dz[b, j].item()) < 3e-3


# ------------------------------------------------- streams, graphs, a run of calls
def test_on_another_stream_and_captured():
    rng = np.random.default_rng(11)
    zt, z = _logits(rng.standard_normal((6, 50_000)), "bf16")
    rp, ids = _lists([2] * 6, 50_000, rng)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = _run(zt, rp, ids, 7)
    out2 = _run(zt, rp, ids, 7, stream=s)
    torch.cuda.synchronize()
    _check(out, z, rp, ids, 7)
    _check(out2, z, rp, ids, 7)
    # forward and gradient in a graph, replayed on new logits
    rpt, idt = _dev(rp), _dev(ids)
    o = [torch.empty(12, device="cuda"), torch.empty(6, device="cuda"), torch.empty(6, device="cuda"),
         torch.empty(6, 7, device="cuda"), torch.empty(6, 7, dtype=torch.int32, device="cuda")]
    ws = torch.empty(H.haste_logprob_workspace_size(6, 50_000, H.HASTE_BF16, 7), dtype=torch.uint8, device="cuda")
    g, dz = torch.ones(12, device="cuda"), torch.empty_like(zt)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        H.haste_logprob(zt, rpt, idt, *o, ws)
        H.haste_logprob_backward(zt, o[1], None, rpt, idt, g, None, dz)
    for seed in range(3):
        new = np.random.default_rng(seed).standard_normal((6, 50_000)) * (seed + 1)
        zt.copy_(torch.as_tensor(new))
        z = zt.double().cpu().numpy()
        graph.replay()
        torch.cuda.synchronize()
        _check(o, z, rp, ids, 7)
        _check_grad(to_np64(dz), z, rp, ids, np.ones(12, np.float32), None, "bf16")


def test_two_calls_at_once_on_two_streams_and_in_one_graph():
    """Calls on two streams with a workspace each, eagerly and captured as a fork that
    joins; then two graphs that share one workspace, replayed in turn."""
    rng = np.random.default_rng(12)
    B, N, k = 3, 300_000, 9
    zs = [_logits(rng.standard_normal((B, N)) * (i + 1), "bf16") for i in range(2)]
    outs = [[None, torch.empty(B, device="cuda"), torch.empty(B, device="cuda"), torch.empty(B, k, device="cuda"),
             torch.empty(B, k, dtype=torch.int32, device="cuda")] for _ in range(2)]
    size = H.haste_logprob_workspace_size(B, N, H.HASTE_BF16, k)
    assert size > 0
    ws = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    none = np.zeros(B + 1, np.int32)

    def call(i, w):
        H.haste_logprob(zs[i][0], lse=outs[i][1], entropy=outs[i][2], top_logp=outs[i][3], top_id=outs[i][4], ws=w)

    def check():
        torch.cuda.synchronize()
        for i in range(2):
            _check([torch.empty(0)] + outs[i][1:], zs[i][1], none, np.zeros(0, np.int32), k)
            for t in outs[i][1:]:
                t.fill_(-3)
        torch.cuda.synchronize()

    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()

    def fork():
        side.wait_stream(main)
        call(0, ws[0])
        with torch.cuda.stream(side):
            call(1, ws[1])
        main.wait_stream(side)

    with torch.cuda.stream(main):
        for _ in range(5):
            fork()
    check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=main):
        fork()
        fork()
    g.replay()
    check()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i in range(2):
        with torch.cuda.graph(graphs[i]):
            call(i, ws[0])
    for _ in range(3):
        graphs[0].replay()
        graphs[1].replay()
    check()


def test_non_contiguous_and_mixed_tensors_are_refused():
    z = torch.zeros(4, 64, device="cuda")
    f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    for call, what in [(lambda: H.haste_logprob(z[:, ::2], lse=f(4)), "contiguous"),
                       (lambda: H.haste_logprob(z.t(), lse=f(64)), "contiguous"),
                       (lambda: H.haste_logprob(z, lse=f(8)[::2]), "contiguous"),
                       (lambda: H.haste_logprob(z, lse=torch.zeros(4)), "lse"),
                       (lambda: H.haste_logprob(z, lse=f(5)), "shape"),
                       (lambda: H.haste_logprob_backward(z, f(4), None, None, None, None, None, f(64, 4).t()), "contiguous")]:
        with pytest.raises(ValueError, match=what):
            call()
    with pytest.raises(H.HasteError) as e:
        H.haste_logprob_backward(z, f(4), None, None, None, None, None, z)      # in place
    assert e.value.status == H.HASTE_ERR_INVALID_ARG
    k = torch.zeros(4, 65, dtype=torch.int32, device="cuda")
    with pytest.raises(H.HasteError) as e:
        H.haste_logprob(z, top_logp=f(4, 65), top_id=k)
    assert e.value.status == H.HASTE_ERR_INVALID_ARG
    long = torch.zeros(2, 400_000, device="cuda")
    with pytest.raises(H.HasteError) as e:
        H.haste_logprob(long, lse=f(2))                                          # split rows need a workspace
    assert e.value.status == H.HASTE_ERR_WORKSPACE


def test_softmax_training_step_of_the_head():
    """Head forward -> log probabilities -> gradient -> head backward, against fp64:
    the cross entropy of given labels, dWh and dXh."""
    B, Hh, d = 96, 1000, 136
    X, W = I.make_normal((B, d), 1.0, 1, 5, "bf16"), I.make_normal((Hh, d), 0.1, 1, 6, "bf16")
    rng = np.random.default_rng(5)
    rp, ids = _lists([1] * B, Hh, rng)
    Xt, Wt = to_torch(X), to_torch(W)
    ws = torch.empty(H.haste_head_workspace_size(B, Hh, d, H.HASTE_BF16), dtype=torch.uint8, device="cuda")
    z = torch.empty((B, Hh), dtype=torch.bfloat16, device="cuda")
    H.haste_head_forward(Xt, Wt, z, ws)
    logp, lse, ent, _, ti = _run(z, rp, ids, 3)
    dz = torch.empty_like(z)
    H.haste_logprob_backward(z, lse, None, _dev(rp), _dev(ids), torch.full((B,), -1.0 / B, device="cuda"), None, dz)
    dW, dX = torch.empty_like(Wt), torch.empty((B, d), device="cuda")
    H.haste_head_backward(Xt, Wt, dz, dW, dX, ws)
    # the logits are held to fp64 first; what follows is held to what it was given, the
    # logits in bf16, whose rounding moves a p by 2^-9 |z| of itself
    assert_close(to_np64(z), O.head_forward(X, W), "logits of the softmax step")
    ref_z = to_np64(z)
    lp, _, _, _, _ = O.logprob(ref_z, rp, ids, 0)
    rdz = O.logprob_backward(ref_z, rp, ids, np.full(B, -1.0 / B))
    rdW, rdX = O.head_backward(X, W, rdz)
    assert abs(logp.mean().item() - lp.mean()) <= 5e-3 * abs(lp.mean())
    # d_logits round to bf16, at most half a step (2^-8) of each: their products' sums are
    # off by 2^-8 sum |dz| |x|; dWh rounds once more.  One sample's given label has |dz|
    # of about 1 / B where the rest of its row has 1e-3 / B, so dWh's elements differ
    # widely and a bound relative to their rms would not follow from the roundings.
    h = 2.0 ** -8
    dw_tol, dx_tol = O.head_backward(np.abs(O.to_f64(X)), np.abs(O.to_f64(W)), np.abs(rdz))
    _near(to_np64(dW), rdW, h * 1.01 * (dw_tol + np.abs(rdW)), "dWh of the softmax step")
    _near(to_np64(dX), rdX, h * 1.01 * dx_tol, "dXh of the softmax step")
