"""Softmax training over the sparse tail: haste_forward -> haste_logprob ->
haste_logprob_backward -> haste_backward_dw and haste_backward_dx, against fp64."""
import math

import numpy as np
import pytest

from oracle import oracle as O
from structured_sparse_output_b200 import haste as H
from structured_sparse_output_b200 import inputs as I
from tests.helpers import assert_close, to_np64, to_torch
from tests.test_gpu_logprob import _check, _check_grad, _dev, _lists, _near, _run

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    H.lib()
    yield
    torch.cuda.synchronize()
    assert H.haste_device_status() == H.HASTE_OK


@pytest.mark.parametrize("B,d,n_groups,G,k,dt", [(130, 200, 100, 32, 64, "f32"), (200, 320, 333, 32, 64, "bf16"),
                                                 (256, 768, 500, 64, 128, "bf16"), (1, 256, 50, 32, 64, "bf16"),
                                                 (37, 96, 1100, 48, 64, "bf16")])
def test_softmax_training_step_of_the_tail(B, d, n_groups, G, k, dt):
    """Cross entropy of the given labels, averaged, with an entropy bonus.  The logits are
    held to fp64 first; what follows is held to what it was given.  d_logits round to their
    type, half a step h of each (bf16 2^-8); the products read fp32 operands as tf32, cut
    to 10 bits: 2^-10 of each of the two.  Their sums are off by that much of sum |dz| |x|
    and sum |dz| |w|, and dW rounds once more.  p is off by 2^-24 (|z| + 2 |lse|) beside
    that, and log p and the sums by 2^-18 and less (within the 1.02)."""
    L = n_groups * G
    idx = I.make_idx(n_groups, k, d, 3)
    X, W = I.make_normal((B, d), 1.0, 3, 1, dt), I.make_normal((L, k), 2.0 / math.sqrt(k), 3, 2, dt)
    rng = np.random.default_rng(B)
    rp, ids = _lists(rng.integers(0, 6, B) if B > 1 else [3], L, rng)
    plan = H.haste_plan(idx, G, d)
    Xt, Wt = to_torch(X), to_torch(W)
    code = H.dtype_code(Xt)
    ws = torch.empty(plan.workspace_size(B, code), dtype=torch.uint8, device="cuda")
    z = torch.empty((B, L), dtype=Xt.dtype, device="cuda")
    H.haste_forward(plan, Xt, Wt, z, ws)
    out = _run(z, rp, ids, 5)
    g, gh = np.full(len(ids), -1.0 / B, np.float32), np.full(B, -0.01 / B, np.float32)
    dz = torch.empty_like(z)
    H.haste_logprob_backward(z, out[1], out[2], _dev(rp), _dev(ids), _dev(g), _dev(gh), dz)
    dW, dX = torch.empty_like(Wt), torch.empty((B, d), device="cuda")
    H.haste_backward_dw(plan, Xt, dz, dW, ws)
    H.haste_backward_dx(plan, Wt, dz, dX, ws)
    torch.cuda.synchronize()

    assert_close(to_np64(z), O.forward(X, W, idx, G), "logits of the softmax step")
    rz = to_np64(z)
    _check(out, rz, rp, ids, 5)
    _check_grad(to_np64(dz), rz, rp, ids, g, gh, dt)
    rdz = O.logprob_backward(rz, rp, ids, g, gh)
    h = 1.02 * (2.0 ** -8 if dt == "bf16" else 2 * 2.0 ** -10)
    ref = O.backward_dw(X, rdz, idx, G)
    tol = O.backward_dw(np.abs(O.to_f64(X)), np.abs(rdz), idx, G)
    _near(to_np64(dW), ref, h * (tol + np.abs(ref)), "dW of the softmax step")
    ref = O.backward_dx(W, rdz, idx, G, d)
    tol = O.backward_dx(np.abs(O.to_f64(W)), np.abs(rdz), idx, G, d)
    _near(to_np64(dX), ref, h * tol, "dX of the softmax step")
