"""Corners of the training operators that need no GPU."""

import contextlib
import os
import shutil
import subprocess
import types

import pytest
import torch

import matrix_orthogonalising_optimizer_amd as dm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "matrix_orthogonalising_optimizer_amd", "csrc")


def test_chunks_of_rows_at_any_element_stay_inside_their_matrix(tmp_path):
    cxx = shutil.which("g++") or shutil.which("clang++")
    if not cxx:
        pytest.skip("no host compiler")
    exe = str(tmp_path / "raw_rows_check")
    subprocess.run([cxx, "-O2", "-std=c++17", "-I", CSRC, os.path.join(ROOT, "tests", "raw_rows_check.cpp"), "-o", exe],
                   check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
    assert int(r.stdout) > 10 ** 6


class GpuTensor(torch.Tensor):
    """A host tensor that the binding takes for one on the GPU and that counts its record_stream calls."""
    is_cuda = True

    def get_device(self):
        return 0

    def record_stream(self, stream):
        self.seen = getattr(self, "seen", []) + [stream]


S = types.SimpleNamespace(device=torch.device("cpu"))  # the host tensors' own device


def gpu(*shape):
    return torch.zeros(shape).as_subclass(GpuTensor)


@pytest.fixture
def fake(monkeypatch):
    """The binding's view of torch, with no device behind it."""
    cuda = types.SimpleNamespace(current_device=lambda: 0, device=lambda d: contextlib.nullcontext(),
                                 stream=lambda s: contextlib.nullcontext())
    monkeypatch.setattr(dm, "_torch", lambda: types.SimpleNamespace(Tensor=torch.Tensor, cuda=cuda))


def test_tensors_by_keyword_are_recorded_on_the_given_stream(fake):
    @dm._on_stream
    def op(x, weight, bias=None, *, scale=1.0):
        return x, weight, bias, scale
    x, w, b = gpu(2), gpu(3), gpu(4)
    assert op(x, weight=w, bias=b, scale=2.0, stream=S) == (x, w, b, 2.0)
    assert [t.seen for t in (x, w, b)] == [[S]] * 3


def test_every_argument_may_be_given_by_keyword(fake):
    @dm._on_stream
    def op(dy, x, weight, *, act="silu"):
        return dy, x, weight, act
    dy, x, w = gpu(2), gpu(3), gpu(4)
    want = (dy, x, w, "gelu")
    assert op(dy, x=x, weight=w, act="gelu") == want
    assert op(dy=dy, x=x, weight=w, act="gelu", stream=S) == want
    assert op(weight=w, x=x, dy=dy, act="gelu") == want
    assert [t.seen for t in (dy, x, w)] == [[S]] * 3
    with pytest.raises(TypeError):
        op()
    with pytest.raises(TypeError):
        op(dy, dy=dy, x=x, weight=w)
    with pytest.raises(ValueError, match="GPU"):
        op(dy=torch.zeros(2), x=x, weight=w)


def test_streams_of_another_device_are_refused(fake):
    @dm._on_stream
    def op(x):
        return x
    with pytest.raises(ValueError, match="stream"):
        op(gpu(2), stream=types.SimpleNamespace(device=torch.device("cuda:1")))
