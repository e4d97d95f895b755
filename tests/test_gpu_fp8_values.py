"""What the 8-bit steps make of the smallest blocks, and of infinities and NaN over whole blocks and
rows."""
import numpy as np
import pytest
import torch

import linear_attention_state_zero_b200 as tr
from gpu_util import f64
from oracle import layer_ops as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def back(q, s, block_rows):
    with np.errstate(invalid="ignore"):
        return f64(q) * ref.expand_scales(f64(s), block_rows, *q.shape)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("xd", [BF, F32])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_a_block_that_is_not_finite_reads_back_as_nan(cuda_device, block_rows, xd, bad):
    """All of it, and nothing beside it; an infinity next to a NaN too."""
    x = torch.ones(300, 400, dtype=xd)
    x[130, 131] = bad
    x[130, 399] = float("inf")
    x[130, 390] = bad
    v = back(*tr.quantize_fp8(x.to(cuda_device), block_rows=block_rows), block_rows)
    rows = slice(130, 131) if block_rows == 1 else slice(128, 256)
    touched = np.zeros(x.shape, dtype=bool)
    touched[rows, 128:256] = touched[rows, 384:] = True
    assert np.isnan(v[touched]).all() and np.isfinite(v[~touched]).all()


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("D", [400, 4096])
def test_norm_of_a_row_that_is_not_finite(cuda_device, D, bad):
    """A NaN makes its row NaN.  Against an infinity finite values are 0, and its own block is NaN
    (infinity over infinity), as the definition has it.  Other rows are what they were."""
    x = torch.ones(5, D, dtype=BF)
    x[3, 131] = bad
    q, s, out = tr.rmsnorm_fp8(x.to(cuda_device), residual=torch.zeros(5, D, device=cuda_device))
    v = back(q, s, 1)
    assert np.isfinite(v[[0, 1, 2, 4]]).all() and np.isnan(v[3, 128:256]).all()
    rest = np.r_[v[3, :128], v[3, 256:]]
    assert np.isnan(rest).all() if np.isnan(bad) else (rest == 0).all()
    assert np.array_equal(f64(out), f64(x), equal_nan=True)


def test_smallest_blocks(cuda_device):
    """Largest magnitudes around 448 x 2^-126, where the scale stays at 2^-126, and below."""
    x = torch.randn(40, 256, generator=torch.Generator().manual_seed(2)).clamp(-3, 3)
    x = (x / 3 * 448 * 2.0 ** -126 * torch.logspace(-3, 1, 40, base=2)[:, None]).to(BF)
    q, s = tr.quantize_fp8(x.to(cuda_device))
    v = f64(x)
    full = ref.expand_scales(ref.block_scales(v, 1), 1, *v.shape)
    assert (np.abs(f64(s) - ref.block_scales(v, 1)) <= 2.0 ** -24 * f64(s)).all() and f64(s).min() == 2.0 ** -126
    # half a step of q, next to which the scale, its reciprocal and the product are off by 2^-24 each
    assert (np.abs(f64(q) * full - v) <= np.maximum(np.abs(v) * 2.0 ** -4, full * 2.0 ** -10) * (1 + 2.0 ** -22)).all()
