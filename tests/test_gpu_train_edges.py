"""Corners of the training operators on the GPU: widths of a few elements,
values at the ends of fp32's range, calls by keyword, very long batches."""

import pytest
import torch

import matrix_orthogonalising_optimizer_amd as dm
from test_gpu_train import BF16, F32, ce_inputs, ffn_inputs, kernels, run_ce, run_ffn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dm.load_library()


# rows at any element, so narrow that a 16-byte chunk spans several: the rows behind the
# last whole step of K hold less than a chunk
@pytest.mark.parametrize("dtype,k", [(BF16, 65), (BF16, 66), (BF16, 70), (F32, 33), (F32, 34)])
@pytest.mark.parametrize("n", [1, 2, 3])
def test_narrow_rows_end_inside_a_chunk(n, k, dtype):
    args = ce_inputs(3, n, k, dtype, masked=0.0)
    _, names = kernels(lambda: run_ce(*args))
    assert any(", kr, out, raw>" in s for s in names), names
    run_ffn(*ffn_inputs(3, n, k, dtype), "silu")
    run_ffn(*ffn_inputs(3, k, n, dtype), "silu")
