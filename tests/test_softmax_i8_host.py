"""Softmax and 8-bit scoring calls without a GPU: the oracle's definitions (closed
forms, finite differences, rational arithmetic) and every refusal, which the
library and the binding make before they look for a device."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import oracle as O
from structured_sparse_output_b200 import haste as H
from structured_sparse_output_b200 import inputs as I


# ------------------------------------------------------------------ the oracle
def test_oracle_quantisation_is_the_exact_rounding():
    """Against rational arithmetic: the scale is the nearest fp32 number to max / 127
    and q the nearest whole number to x / scale, halves to even."""
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((40, 33)) * 10.0 ** rng.integers(-30, 30, (40, 1))).astype(np.float32)
    x[3] = 0
    x[5, 1:] = x[5, 0] / 127 * (np.arange(32) - 15.5).astype(np.float32)      # next to halves
    x[6] = np.float32(1e-44)                                                  # the scale underflows to 0
    q, s = O.quantize_rows(x)
    for r in range(len(x)):
        amax = max(abs(Fraction(float(v))) for v in x[r])
        near = [np.nextafter(s[r], np.float32(0)), s[r], np.nextafter(s[r], np.float32(np.inf))]
        assert min(near, key=lambda v: abs(Fraction(float(v)) - amax / 127)) == s[r]
        for v, got in zip(x[r], q[r]):
            want = 0 if s[r] == 0 else round(Fraction(float(v)) / Fraction(float(s[r])))
            assert got == max(-127, min(127, want))
    bad = np.ones((2, 4), np.float32)
    bad[0, 1], bad[1, 2] = np.nan, -np.inf
    q, s = O.quantize_rows(bad)
    assert np.isnan(s).all() and not q.any()


def test_oracle_logprob_closed_forms():
    z = np.zeros((1, 8), np.float32)
    lp, lse, h, tl, ti = O.logprob(z, [0, 2], [3, 9], 3)
    assert np.isclose(lp[0], -np.log(8)) and np.isnan(lp[1])
    assert np.isclose(lse[0], np.log(8)) and np.isclose(h[0], np.log(8))
    assert ti.tolist() == [[0, 1, 2]]                                         # ties: smaller id first
    z = np.array([[0.0, -np.inf, np.log(3.0), -np.inf]])
    lp, lse, h, tl, ti = O.logprob(z, [0, 1], [1], 4)
    assert lp[0] == -np.inf and np.isclose(lse[0], np.log(4))
    assert np.isclose(h[0], -(0.25 * np.log(0.25) + 0.75 * np.log(0.75)))
    assert ti.tolist() == [[2, 0, 1, 3]] and tl[0, 3] == -np.inf
    _, lse, h, tl, ti = O.logprob(np.full((1, 3), -np.inf), [0, 0], [], 2)
    assert lse[0] == -np.inf and h[0] == 0 and ti.tolist() == [[0, 1]]
    _, lse, h, _, _ = O.logprob(np.array([[0, np.nan], [np.inf, 1]]), [0, 0, 0], [], 0)
    assert np.isnan(lse).all() and np.isnan(h).all()


def test_oracle_logprob_gradient_against_differences():
    rng = np.random.default_rng(1)
    z = rng.standard_normal((3, 7))
    z[1, 2] = -np.inf
    rp, ids = np.array([0, 3, 4, 4]), np.array([2, 5, 2, 0])                  # a repeat, an empty list
    g, gh = rng.standard_normal(4), rng.standard_normal(3)

    def f(z):
        lp, _, h, _, _ = O.logprob(z, rp, ids, 0)
        return float(g @ lp + gh @ h)

    got = O.logprob_backward(z, rp, ids, g, gh)
    step = 1e-6
    for b in range(3):
        for j in range(7):
            if np.isinf(z[b, j]):
                assert got[b, j] == 0
                continue
            a, c = z.copy(), z.copy()
            a[b, j] += step
            c[b, j] -= step
            assert abs((f(a) - f(c)) / (2 * step) - got[b, j]) < 1e-8
    assert not O.logprob_backward(np.full((1, 4), -np.inf), [0, 1], [2], [1.0], [1.0]).any()


def test_oracle_head_i8_is_near_the_unquantised_head():
    """Each factor is within half a step of its value: |q s - x| <= s / 2 for both, so a
    logit is off by at most sum |x| sw / 2 + |w| sx / 2 + sx sw / 4 over the features."""
    x = I.make_normal((9, 50), 1.0, 3, 1, "f32")
    w = I.make_normal((21, 50), 0.2, 3, 2, "f32")
    wq, ws = O.quantize_rows(w)
    _, xs = O.quantize_rows(x)
    z = O.head_forward_i8(x, wq, ws)
    x64, w64 = x.astype(np.float64), w.astype(np.float64)
    bound = (np.abs(x64).sum(1)[:, None] * ws[None, :] / 2 + np.abs(w64).sum(1)[None, :] * xs[:, None] / 2
             + 50 * xs[:, None].astype(np.float64) * ws[None, :] / 4)
    assert np.all(np.abs(z - x64 @ w64.T) <= bound * (1 + 1e-6))


# ---------------------------------------------------------------- the refusals
P = 4096      # an aligned address that is never read: every call below is refused first


def _targets(rp=P, ids=P):
    return H.Targets(rp, ids)


def _quantize(rows=4, n=64, dt=H.HASTE_F32, x=P, q=P, s=P):
    return H.lib().haste_quantize_rows(rows, n, dt, x, q, s, None)


def _head(B=4, Hh=32, d=64, dt=H.HASTE_BF16, x=P, w=P, s=P, odt=H.HASTE_F32, out=P, ws=P, nws=1 << 20):
    return H.lib().haste_head_forward_i8(B, Hh, d, dt, x, w, s, odt, out, ws, nws, None)


def _logprob(B=4, N=100, dt=H.HASTE_F32, z=P, rp=P, ids=P, nnz=4, k=2, lp=P, tl=P, ti=P, ws=P, nws=1 << 30):
    return H.lib().haste_logprob(B, N, dt, z, _targets(rp, ids), nnz, k, lp, P, P, tl, ti, ws, nws, None)


def _grad(B=4, N=100, dt=H.HASTE_F32, z=P, lse=P, ent=P, rp=P, ids=P, nnz=4, g=P, gh=P, dz=1 << 20):
    return H.lib().haste_logprob_backward(B, N, dt, z, lse, ent, _targets(rp, ids), nnz, g, gh, dz, None)


ARG, SHAPE, WS = H.HASTE_ERR_INVALID_ARG, H.HASTE_ERR_UNSUPPORTED_SHAPE, H.HASTE_ERR_WORKSPACE


@pytest.mark.parametrize("call,kw,status", [
    (_quantize, dict(rows=0), ARG), (_quantize, dict(rows=1 << 31), ARG), (_quantize, dict(n=0), ARG),
    (_quantize, dict(n=131_073), SHAPE), (_quantize, dict(dt=2), ARG), (_quantize, dict(x=None), ARG),
    (_quantize, dict(q=None), ARG), (_quantize, dict(s=None), ARG), (_quantize, dict(q=P + 8), ARG),
    (_quantize, dict(x=P + 2), ARG), (_quantize, dict(s=P + 1), ARG),
    (_head, dict(B=0), ARG), (_head, dict(Hh=0), ARG), (_head, dict(d=-1), ARG), (_head, dict(d=131_073), SHAPE),
    (_head, dict(dt=7), ARG), (_head, dict(odt=-1), ARG), (_head, dict(x=None), ARG), (_head, dict(w=None), ARG),
    (_head, dict(s=None), ARG), (_head, dict(out=None), ARG), (_head, dict(w=P + 4), ARG),
    (_head, dict(x=P + 1), ARG), (_head, dict(out=P + 2), ARG), (_head, dict(ws=None), ARG),
    (_head, dict(ws=P + 8), ARG), (_head, dict(nws=511), WS), (_head, dict(B=(1 << 30) + 1), SHAPE),
    (_head, dict(B=1 << 26, Hh=1 << 30), SHAPE),
    (_logprob, dict(B=0), ARG), (_logprob, dict(N=0), ARG), (_logprob, dict(N=1 << 31), SHAPE),
    (_logprob, dict(dt=3), ARG), (_logprob, dict(z=None), ARG), (_logprob, dict(z=P + 2), ARG),
    (_logprob, dict(k=-1), ARG), (_logprob, dict(k=65), ARG), (_logprob, dict(N=1, k=2), ARG),
    (_logprob, dict(nnz=-1), ARG), (_logprob, dict(nnz=1 << 31), ARG), (_logprob, dict(rp=None), ARG),
    (_logprob, dict(ids=None), ARG), (_logprob, dict(lp=None), ARG), (_logprob, dict(tl=None), ARG),
    (_logprob, dict(ti=None), ARG),
    (_grad, dict(B=-3), ARG), (_grad, dict(N=0), ARG), (_grad, dict(dt=9), ARG), (_grad, dict(z=None), ARG),
    (_grad, dict(lse=None), ARG), (_grad, dict(ent=None), ARG), (_grad, dict(g=None), ARG),
    (_grad, dict(rp=None), ARG), (_grad, dict(dz=None), ARG), (_grad, dict(dz=P), ARG),
    (_grad, dict(dz=P + 1596), ARG), (_grad, dict(dz=P - 4), ARG), (_grad, dict(z=P + 3), ARG),
], ids=lambda v: getattr(v, "__name__", str(v)))
def test_library_refuses(call, kw, status):
    assert call(**kw) == status
    assert H.lib().haste_last_error()


def test_sizes_are_host_only():
    assert [H.haste_i8_pitch(n) for n in (-1, 0, 1, 16, 17)] == [0, 0, 16, 16, 32]
    assert H.haste_head_i8_workspace_size(0, 4, 4) == 0 == H.haste_head_i8_workspace_size(4, 4, 131_073)
    assert H.haste_head_i8_workspace_size(3, 4, 100) >= 3 * 112 + 3 * 4
    assert H.haste_logprob_workspace_size(0, 5, H.HASTE_F32, 1) == 0


def test_binding_refuses_before_any_pointer():
    torch = pytest.importorskip("torch")
    bf, f32, i32, i8 = torch.bfloat16, torch.float32, torch.int32, torch.int8
    z = lambda *s, dtype=f32: torch.zeros(*s, dtype=dtype)  # noqa: E731
    x, q, s = z(3, 20), z(3, 32, dtype=i8), z(3)
    cases = [
        (lambda: H.haste_quantize_rows(x, z(3, 20, dtype=i8), s), "shape"),
        (lambda: H.haste_quantize_rows(x, z(3, 32, dtype=i32), s), "dtype"),
        (lambda: H.haste_quantize_rows(x, q, z(3, dtype=bf)), "dtype"),
        (lambda: H.haste_quantize_rows(x, q, s), "CUDA"),
        (lambda: H.haste_head_forward_i8(x, z(5, 20, dtype=i8), z(5), z(3, 5), None), "shape"),
        (lambda: H.haste_head_forward_i8(x, z(5, 32, dtype=i8), z(4), z(3, 5), None), "shape"),
        (lambda: H.haste_head_forward_i8(x, z(5, 32, dtype=i8), z(5), z(3, 6), None), "shape"),
        (lambda: H.haste_head_forward_i8(x, z(5, 32, dtype=i8), z(5), z(3, 5), None), "CUDA"),
        (lambda: H.haste_logprob(x, z(3, dtype=i32), z(4, dtype=i32), z(4)), "row_ptr"),
        (lambda: H.haste_logprob(x, z(4, dtype=i32), z(4, dtype=torch.int64), z(4)), "ids"),
        (lambda: H.haste_logprob(x, z(4, dtype=i32), z(4, dtype=i32), z(5)), "logp"),
        (lambda: H.haste_logprob(x, z(4, dtype=i32), z(4, dtype=i32), None), "logp"),
        (lambda: H.haste_logprob(x, None, z(4, dtype=i32), None), "row_ptr"),
        (lambda: H.haste_logprob(x, lse=z(4)), "lse"),
        (lambda: H.haste_logprob(x, entropy=z(3, dtype=bf)), "entropy"),
        (lambda: H.haste_logprob(x, top_id=z(3, 2, dtype=i32)), "together"),
        (lambda: H.haste_logprob(x, top_id=z(3, 2, dtype=i32), top_logp=z(3, 3)), "top_logp"),
        (lambda: H.haste_logprob(x, top_id=z(3, 2, dtype=torch.int64), top_logp=z(3, 2)), "top_id"),
        (lambda: H.haste_logprob(x, lse=s), "CUDA"),
        (lambda: H.haste_logprob_backward(x, z(4), None, None, None, None, None, x), "lse"),
        (lambda: H.haste_logprob_backward(x, s, None, None, None, None, s, x), "entropy"),
        (lambda: H.haste_logprob_backward(x, s, s, None, None, None, z(2), x), "d_entropy"),
        (lambda: H.haste_logprob_backward(x, s, s, None, None, z(2), s, x), "row_ptr"),
        (lambda: H.haste_logprob_backward(x, s, None, None, None, None, None, z(3, 20, dtype=bf)), "dtype"),
        (lambda: H.haste_logprob_backward(x, s, None, None, None, None, None, z(3, 20)), "CUDA"),
    ]
    for call, what in cases:
        with pytest.raises(ValueError, match=what):
            call()
    with pytest.raises(TypeError):
        H.haste_logprob(z(3, 20, dtype=torch.float16), lse=s)
    with pytest.raises(TypeError):
        H.haste_head_forward_i8(x, z(5, 32, dtype=i8), z(5), z(3, 5, dtype=torch.float64), None)


def test_valid_calls_need_a_device():
    """With nothing to refuse, a machine without a GPU gets HASTE_ERR_CUDA and no launch."""
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for call in (_quantize, _head, _logprob, _grad):
        assert call() == H.HASTE_ERR_CUDA


def test_oracle_softmax_does_not_depend_on_where_the_logits_lie():
    """Rows of the types' lowest value and rows around 1e30, where a log sum of 8 is lost in
    fp64: log p, the entropy and the gradient are those of the same row around 0."""
    low = -3.3895313892515355e38
    for z in (np.full((1, 8), low), np.full((1, 8), 1e30), np.full((1, 8), float(np.finfo(np.float32).max))):
        lp, _, h, tl, _ = O.logprob(z, [0, 1], [3], 2)
        assert np.allclose(lp, -np.log(8)) and np.allclose(tl, -np.log(8)) and np.isclose(h[0], np.log(8))
        dz = O.logprob_backward(z, [0, 1], [3], [1.0], [2.0])
        assert np.allclose(dz, np.eye(8)[3] - 1 / 8)
    z = np.where(np.arange(8) % 2, low, -np.inf)[None]
    assert np.allclose(O.logprob_backward(z, [0, 1], [3], [1.0]), np.eye(8)[3] - (np.arange(8) % 2) / 4)
