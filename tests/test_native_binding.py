"""The binding's C++ argument checks: their binary belongs to one torch and one interpreter,
and without it the Python checks make the same calls."""
import os

import pytest

from structured_sparse_output_b200 import haste as H
from structured_sparse_output_b200.csrc import build

torch = pytest.importorskip("torch")


@pytest.fixture
def fresh(monkeypatch):
    """A binding that has not looked for the binary yet."""
    monkeypatch.setattr(H, "_native_module", None)


def _refused_by_python():
    """A call that gets as far as the Python checks."""
    with pytest.raises(ValueError, match="CUDA"):
        H.haste_logprob(torch.zeros(2, 3), lse=torch.zeros(2))
    with pytest.raises(ValueError, match="CUDA"):
        H.haste_logprob_backward(torch.zeros(2, 3), torch.zeros(2), None, None, None, None, None, torch.zeros(2, 3))
    with pytest.raises(ValueError, match="CUDA"):
        H.haste_head_forward_i8(torch.zeros(2, 3), torch.zeros(5, 16, dtype=torch.int8), torch.zeros(5), torch.zeros(2, 5),
                                None)


def test_binary_is_built_and_taken(fresh):
    assert os.path.exists(build.build_native())
    H._native()
    assert H._native_module.__file__ == build.native_path()


@pytest.mark.parametrize("what", ["torch", "abi", "python"])
def test_binary_of_another_torch_or_interpreter_is_not_taken(fresh, monkeypatch, what):
    """It reads tensors by the layout of the headers that it was built with."""
    mine = build.native_path()
    if what == "torch":
        monkeypatch.setattr(torch, "__version__", "2.99.0+cu999")
    elif what == "abi":
        monkeypatch.setattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", not torch._C._GLIBCXX_USE_CXX11_ABI)
    else:
        monkeypatch.setattr(build.sys.implementation, "cache_tag", "cpython-399")
    assert build.native_path() != mine
    with pytest.warns(RuntimeWarning, match="build.py"):
        _refused_by_python()


@pytest.mark.parametrize("content", [None, b"", b"no library"])
def test_calls_do_without_the_binary(fresh, monkeypatch, tmp_path, content):
    path = tmp_path / "_native.so"
    if content is not None:
        path.write_bytes(content)
    monkeypatch.setattr(build, "native_path", lambda: str(path))
    with pytest.warns(RuntimeWarning, match="build.py") as seen:
        _refused_by_python()
    assert len(seen) == 1      # said once, not at every call


@pytest.mark.gpu
def test_results_without_the_binary_are_the_same(fresh, monkeypatch, tmp_path):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(5, 40, generator=g, device="cuda")
    q = torch.randint(-127, 128, (300, 48), generator=g, device="cuda").to(torch.int8)
    s = torch.rand(300, generator=g, device="cuda")
    rp = torch.arange(0, 11, 2, dtype=torch.int32, device="cuda")
    ids = torch.randint(0, 300, (10,), generator=g, device="cuda").int()
    d = torch.randn(10, generator=g, device="cuda")

    def run():
        e = lambda *n, t=torch.float32: torch.full(n, 3, dtype=t, device="cuda")  # noqa: E731
        z, logp, lse, ent, tl, ti, dz = e(5, 300), e(10), e(5), e(5), e(5, 4), e(5, 4, t=torch.int32), e(5, 300)
        H.haste_head_forward_i8(x, q, s, z, e(H.haste_head_i8_workspace_size(5, 300, 40), t=torch.uint8))
        H.haste_logprob(z, rp, ids, logp, lse, ent, tl, ti)
        H.haste_logprob_backward(z, lse, ent, rp, ids, d, d[:5], dz)
        return z, logp, lse, ent, tl, ti, dz

    one = run()
    monkeypatch.setattr(H, "_native_module", None)
    monkeypatch.setattr(build, "native_path", lambda: str(tmp_path / "none.so"))
    with pytest.warns(RuntimeWarning):
        two = run()
    assert all(torch.equal(a, b) for a, b in zip(one, two))
