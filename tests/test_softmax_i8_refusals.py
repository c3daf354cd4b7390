"""Refusals of the softmax and 8-bit scoring calls at the edges of what their header allows,
on the host: the library makes them before it looks for a device."""
import pytest

from structured_sparse_output_b200 import haste as H

P = 4096      # an aligned address that is never read: every call below is refused first
ARG, SHAPE = H.HASTE_ERR_INVALID_ARG, H.HASTE_ERR_UNSUPPORTED_SHAPE


def _logprob(B=4, N=100, z=P, rp=P, ids=P, nnz=4, k=2, logp=P, lse=P, entropy=P, top_logp=P, top_id=P):
    return H.lib().haste_logprob(B, N, H.HASTE_F32, z, H.Targets(rp, ids), nnz, k, logp, lse, entropy, top_logp, top_id, P,
                                 1 << 30, None)


def _grad(B=4, N=100, z=P, lse=P, entropy=P, rp=P, ids=P, nnz=4, d_logp=P, d_entropy=P, dz=1 << 20):
    return H.lib().haste_logprob_backward(B, N, H.HASTE_F32, z, lse, entropy, H.Targets(rp, ids), nnz, d_logp, d_entropy,
                                          dz, None)


@pytest.mark.parametrize("off", [1, 2, 3])
@pytest.mark.parametrize("call,name", [(_logprob, n) for n in ("rp", "ids", "logp", "lse", "entropy", "top_logp", "top_id")]
                         + [(_grad, n) for n in ("lse", "entropy", "rp", "ids", "d_logp", "d_entropy")],
                         ids=lambda v: getattr(v, "__name__", v))
def test_addresses_off_their_element_size_are_refused(call, name, off):
    """A load or store of 4 bytes there would fault on the GPU."""
    assert call(**{name: P + off}) == ARG
    assert b"aligned" in H.lib().haste_last_error()


def test_addresses_that_a_call_does_not_touch_are_not_looked_at():
    """Lists without entries, no alternatives, entropies without their gradient: what is wrong
    with such a call is found elsewhere, here in the logits' address."""
    for call in (lambda: _logprob(nnz=0, rp=P + 1, ids=P + 1, logp=P + 1, z=P + 2),
                 lambda: _logprob(k=0, top_logp=P + 1, top_id=P + 1, rp=P + 2),
                 lambda: _grad(nnz=0, rp=P + 1, ids=P + 1, d_logp=P + 1, lse=P + 2),
                 lambda: _grad(d_entropy=None, entropy=P + 1, d_logp=P + 2)):
        assert call() == ARG
        assert [w for w in (b"logits", b"row_ptr", b"lse", b"d_logp") if w in H.lib().haste_last_error()]


def _head(B, Hh):
    """The 8-bit head's status with a workspace of no bytes, so that no call gets to a device."""
    return H.lib().haste_head_forward_i8(B, Hh, 64, H.HASTE_BF16, P, P, P, H.HASTE_F32, P, P, 0, None)


@pytest.mark.parametrize("B,Hh", [(16 << 15, 128 << 15), (1, 1 << 30), (1 << 30, 1), (1 << 30, 2048), (2048, 1 << 30)])
def test_head_i8_takes_up_to_2_30_tiles(B, Hh):
    """Tile numbers count on by the number of CTAs beyond the last one, in 32 bits."""
    assert _head(B, Hh) == H.HASTE_ERR_WORKSPACE


@pytest.mark.parametrize("B,Hh", [((16 << 15) + 1, 128 << 15), (16 << 15, (128 << 15) + 1), (4096, 1 << 30), (1 << 30, 2049),
                                  ((1 << 31) // 2 + 1, 1), (16 << 16, (128 << 15) - 128)])
def test_head_i8_refuses_more_than_2_30_tiles(B, Hh):
    assert _head(B, Hh) == SHAPE
