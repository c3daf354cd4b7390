"""GPU parity of the 8-bit head (haste_quantize_rows, haste_head_forward_i8) against
the fp64 oracle.

Quantised rows and scales must be equal: both are roundings of exact values.  A
logit is (float)acc * (sx * sw): the sum acc is exact, so three fp32 roundings, 3
half steps of 2^-24 of its value (no cancellation), then half a step of the output
type.
"""
import numpy as np
import pytest

from oracle import oracle as O
from structured_sparse_output_b200 import haste as H
from structured_sparse_output_b200 import inputs as I
from tests.helpers import to_np64

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    H.lib()
    yield
    torch.cuda.synchronize()
    assert H.haste_device_status() == H.HASTE_OK


def _at(a, dt, offset=0):
    """a in type dt on the GPU, `offset` elements into a larger buffer; and what it holds."""
    t = torch.as_tensor(np.asarray(a, dtype=np.float32)).to(DT[dt])
    buf = torch.full((t.numel() + offset + 64,), float("nan"), dtype=DT[dt], device="cuda")
    v = buf[offset:offset + t.numel()].view(t.shape)
    v.copy_(t)
    return v, t.double().numpy()


def _quantize(xt):
    rows, n = xt.shape
    q = torch.full((rows, H.haste_i8_pitch(n)), 99, dtype=torch.int8, device="cuda")
    s = torch.full((rows,), -5.0, device="cuda")
    H.haste_quantize_rows(xt, q, s)
    return q, s


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("rows,n", [(1, 1), (3, 15), (5, 16), (2, 17), (700, 100), (9, 768), (33, 1000), (4, 1023),
                                    (3, 4096), (2, 4101), (2, 20_000), (1, 131_072)])
def test_quantize_rows_is_exact(rows, n, dt):
    rng = np.random.default_rng(rows + n)
    x = rng.standard_normal((rows, n)) * 10.0 ** rng.integers(-35, 35, (rows, 1))
    x = np.clip(x, -3.3e38, 3.3e38).astype(np.float32)
    xt, x64 = _at(x, dt, offset=n % 5)
    q, s = _quantize(xt)
    rq, rs = O.quantize_rows(x64)
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(q.cpu().numpy()[:, :n], rq) and not q[:, n:].any()


def test_quantize_rows_halves_zeros_and_non_finite():
    """Quotients next to halves, an all-zero row, scales that are subnormal or 0, rows
    with a NaN or an infinity."""
    rows = []
    for seed in range(200):
        rng = np.random.default_rng(seed)
        amax = np.float32(rng.uniform(1, 2) * 2.0 ** rng.integers(-20, 20))
        s = np.float32(np.float64(amax) / 127)
        half = (rng.integers(-126, 126, 63) + 0.5) * np.float64(s)
        near = half.astype(np.float32)
        if seed % 2:
            near = np.nextafter(near, np.where(rng.random(63) < 0.5, np.inf, -np.inf).astype(np.float32))
        rows.append(np.concatenate([[amax], near]))
    rows += [np.zeros(64), np.full(64, 1e-44), np.linspace(-1, 1, 64) * 3e-43, np.linspace(-1, 1, 64) * 1e-39]
    for bad in (np.nan, np.inf, -np.inf):
        r = np.ones(64)
        r[17] = bad
        rows.append(r)
    x = np.stack(rows).astype(np.float32)
    xt, x64 = _at(x, "f32")
    q, s = _quantize(xt)
    rq, rs = O.quantize_rows(x64)
    assert np.array_equal(s.cpu().numpy(), rs, equal_nan=True)
    assert np.array_equal(q.cpu().numpy(), rq)


def _head(xt, q, s, out_dt, offset=0, ws=None, stream=None):
    B, d = xt.shape
    Hh = q.shape[0]
    buf = torch.full((B * Hh + 64,), 31.0, dtype=DT[out_dt], device="cuda")
    out = buf[offset:offset + B * Hh].view(B, Hh)
    if ws is None:
        ws = torch.empty(H.haste_head_i8_workspace_size(B, Hh, d), dtype=torch.uint8, device="cuda")
    H.haste_head_forward_i8(xt, q, s, out, ws, stream=stream)
    return out, buf


def _check(out, x64, q, s, out_dt):
    d = x64.shape[1]
    ref = O.head_forward_i8(x64, q[:, :d].cpu().numpy(), s.cpu().numpy())
    got = to_np64(out)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    tol = (3 * 2.0 ** -24 + (torch.finfo(DT[out_dt]).eps / 2 if out_dt == "bf16" else 0)) * 1.001
    ok = ~np.isnan(ref)
    assert np.all(np.abs(got - ref)[ok] <= tol * np.abs(ref[ok]) + 1e-37), np.max(np.abs(got - ref)[ok])


HEADS = [(1, 1, 1), (1, 4096, 768), (2, 100, 17), (3, 129, 128), (16, 128, 16), (17, 300, 130), (37, 10_007, 1000),
         (64, 1024, 256), (65, 257, 4096), (100, 500, 200), (128, 4096, 768), (129, 640, 384), (200, 333, 777),
         (256, 1000, 768), (257, 1000, 1024), (300, 77, 31), (512, 2049, 1024), (700, 260, 100), (1000, 40, 64),
         # few samples, one launch: each width, rows of one and several rounds, more labels than warps
         (1, 3, 4096), (2, 5000, 1040), (4, 30_001, 96), (5, 513, 2000), (7, 64, 4096), (8, 4099, 1500), (8, 70, 4097),
         (1, 50, 32_768), (1, 77, 32_769), (3, 40_007, 33), (3, 5001, 1000), (4, 16_384, 20), (2, 70_001, 800),
         # many samples and labels, one and several tiles a CTA, ragged in each direction
         (129, 8192, 16), (256, 8200, 768), (200, 16_513, 130), (384, 9001, 777), (512, 40_000, 256), (1025, 8321, 300)]


@pytest.mark.parametrize("B,Hh,d", HEADS)
@pytest.mark.parametrize("dt,out_dt", [("bf16", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
def test_head_forward_i8_matches_oracle(B, Hh, d, dt, out_dt):
    rng = np.random.default_rng(B + Hh + d)
    q, s = _quantize(_at(rng.standard_normal((Hh, d)) / np.sqrt(d), "f32")[0])
    xt, x64 = _at(rng.standard_normal((B, d)), dt, offset=d % 3)
    off = (B + Hh) % 4
    out, buf = _head(xt, q, s, out_dt, offset=off)
    _check(out, x64, q, s, out_dt)
    assert (buf[:off] == 31).all() and (buf[off + B * Hh:] == 31).all()
    again, _ = _head(xt, q, s, out_dt, offset=off)
    assert torch.equal(out, again)


def test_head_forward_i8_extremes():
    """The largest sums (every product 127 * 127, d = 131072), zero samples and labels, a
    sample with a NaN, garbage in the weights' padding columns."""
    d = 131_072
    x = np.ones((3, d), np.float32)
    x[1] = -2.0
    x[2] = 0
    q = torch.full((5, d), 127, dtype=torch.int8, device="cuda")
    q[1] = -127
    q[2] = 0
    s = torch.tensor([1.0, 0.5, 1.0, 0.0, float("nan")], device="cuda")
    xt, x64 = _at(x, "f32")
    out, _ = _head(xt, q, s, "f32")
    _check(out, x64, q, s, "f32")
    x = np.random.default_rng(0).standard_normal((4, 50)).astype(np.float32)
    x[2, 3] = np.nan
    xt, x64 = _at(x, "f32")
    q = torch.randint(-127, 128, (90, 64), dtype=torch.int8, device="cuda")   # columns 50 .. 63 are no weights
    s = torch.rand(90, device="cuda")
    out, _ = _head(xt, q, s, "f32")
    _check(out, x64, q, s, "f32")
    assert torch.isnan(out[2]).all()


def test_offsets_beyond_32_bits():
    """Logits past 2^31 elements: the last samples and labels."""
    B, Hh, d = 2200, 1_000_003, 16
    x = torch.zeros(B, d, device="cuda")
    x[B - 1] = 1.0
    q = torch.zeros(Hh, d, dtype=torch.int8, device="cuda")
    q[Hh - 1], q[5] = 127, -1
    s = torch.ones(Hh, device="cuda")
    out, _ = _head(x, q, s, "bf16")
    assert out[B - 1, Hh - 1].item() == 127 * 16 and out[B - 1, 5].item() == -16
    assert not out[:B - 1].any() and not out[B - 1, 6:Hh - 1].any() and not out[B - 1, :5].any()


def test_streams_graphs_and_shared_workspace():
    rng = np.random.default_rng(2)
    q, s = _quantize(_at(rng.standard_normal((3000, 500)), "f32")[0])
    xt, x64 = _at(rng.standard_normal((70, 500)), "bf16")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        out, _ = _head(xt, q, s, "f32")
    torch.cuda.synchronize()
    _check(out, x64, q, s, "f32")
    # calls in a row share one workspace on a stream; captured, then replayed on new features
    ws = torch.empty(H.haste_head_i8_workspace_size(70, 3000, 500), dtype=torch.uint8, device="cuda")
    x2, o1, o2 = torch.zeros_like(xt), torch.empty(70, 3000, device="cuda"), torch.empty(70, 3000, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        H.haste_head_forward_i8(xt, q, s, o1, ws)
        H.haste_head_forward_i8(x2, q, s, o2, ws)
    for seed in range(3):
        r = np.random.default_rng(seed)
        xt.copy_(torch.as_tensor(r.standard_normal((70, 500))))
        x2.copy_(torch.as_tensor(r.standard_normal((70, 500))))
        graph.replay()
        torch.cuda.synchronize()
        _check(o1, xt.double().cpu().numpy(), q, s, "f32")
        _check(o2, x2.double().cpu().numpy(), q, s, "f32")


def test_short_wait_limit_unwinds_and_the_context_survives():
    """A 1 ns limit on the product's inter-warp waits: the kernel unwinds and the error
    word says so; with the default restored the same call is right."""
    rng = np.random.default_rng(4)
    q, s = _quantize(_at(rng.standard_normal((3000, 800)), "f32")[0])
    xt, x64 = _at(rng.standard_normal((200, 800)), "bf16")
    torch.cuda.synchronize()
    assert H.haste_device_status() == H.HASTE_OK
    H.haste_set_wait_limit_ns(1)
    try:
        _head(xt, q, s, "f32")
        assert H.haste_device_status() == H.HASTE_ERR_TIMEOUT
    finally:
        H.haste_set_wait_limit_ns(0)
    assert H.haste_device_status() == H.HASTE_OK
    out, _ = _head(xt, q, s, "f32")
    _check(out, x64, q, s, "f32")


def test_binding_refuses_what_the_calls_cannot_read():
    x, q, s = torch.zeros(3, 40, device="cuda"), torch.zeros(5, 48, dtype=torch.int8, device="cuda"), torch.ones(5, device="cuda")
    out, ws = torch.zeros(3, 5, device="cuda"), torch.empty(4096, dtype=torch.uint8, device="cuda")
    H.haste_head_forward_i8(x, q, s, out, ws)
    for call, what in [(lambda: H.haste_head_forward_i8(x.t().contiguous().t(), q, s, out, ws), "contiguous"),
                       (lambda: H.haste_head_forward_i8(x, q[:, :40], s, out, ws), "shape"),
                       (lambda: H.haste_head_forward_i8(x, q, s, out[:, :4], ws), "shape"),
                       (lambda: H.haste_head_forward_i8(x, q, s.cpu(), out, ws), "w_scale"),
                       (lambda: H.haste_quantize_rows(x, q, s), "shape")]:
        with pytest.raises(ValueError, match=what):
            call()
    for w, status in [(None, H.HASTE_ERR_WORKSPACE), (ws[:64], H.HASTE_ERR_WORKSPACE), (ws[1:], H.HASTE_ERR_INVALID_ARG)]:
        with pytest.raises(H.HasteError) as e:
            H.haste_head_forward_i8(x, q, s, out, w)
        assert e.value.status == status
    off = torch.zeros(5 * 48 + 8, dtype=torch.int8, device="cuda")[8:].view(5, 48)
    with pytest.raises(H.HasteError) as e:
        H.haste_head_forward_i8(x, off, s, out, ws)                               # rows must start on 16 bytes
    assert e.value.status == H.HASTE_ERR_INVALID_ARG


def test_scoring_run_quantise_product_alternatives():
    """Weights quantised once, 8-bit logits, log probabilities with the best labels: the
    whole run against fp64.  The logits are the same fp32 numbers on both sides (an
    exact sum, three roundings), so the ids must be equal."""
    B, Hh, d, k = 130, 4096, 768, 8
    W, X = I.make_normal((Hh, d), 0.05, 1, 6, "bf16"), I.make_normal((B, d), 1.0, 1, 5, "bf16")
    wt = torch.from_numpy(W.view(np.int16).copy()).view(torch.bfloat16).cuda()
    xt = torch.from_numpy(X.view(np.int16).copy()).view(torch.bfloat16).cuda()
    q, s = _quantize(wt)
    z, _ = _head(xt, q, s, "f32")
    lse, ent = torch.empty(B, device="cuda"), torch.empty(B, device="cuda")
    tl, ti = torch.empty(B, k, device="cuda"), torch.empty(B, k, dtype=torch.int32, device="cuda")
    ws = torch.empty(H.haste_logprob_workspace_size(B, Hh, H.HASTE_F32, k), dtype=torch.uint8, device="cuda")
    H.haste_logprob(z, lse=lse, entropy=ent, top_logp=tl, top_id=ti, ws=ws)
    wq, wsc = O.quantize_rows(W)
    xq, xsc = O.quantize_rows(X)
    acc = (xq @ wq.T).astype(np.float32)
    z32 = acc * (xsc[:, None] * wsc[None, :])
    assert np.array_equal(z.cpu().numpy(), z32)
    _, rlse, rent, rtl, rti = O.logprob(z32, np.zeros(B + 1, int), [], k)
    assert np.array_equal(ti.cpu().numpy(), rti)
    assert np.allclose(lse.cpu(), rlse, atol=2e-5) and np.allclose(ent.cpu(), rent, atol=5e-5)
    assert np.allclose(tl.cpu(), rtl, atol=2e-5)
