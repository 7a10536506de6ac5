"""Few-token operators where their definitions are easily missed."""
import pytest
import torch

from . import few_reference as R
from .test_gpu_few import experts, normal, on_gpu, routing

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from nvfp4_block_scaled_07_gb300 import build
    build.build()
    from nvfp4_block_scaled_07_gb300 import binding
    binding.device_check()
    binding.sync_status()
    return binding


# ---- the gated products between the two products ------------------------------------------------------------------
def ones(E, N, K, fmt):
    """Matrices of zeros whose scales are all 1."""
    m = R.Matrices(E, N, K, fmt, seed=0)
    m.packed.zero_()
    m.scales.fill_(0x38 if fmt == "nvfp4" else 127)
    if m.gscale is not None:
        m.gscale.fill_(1.0)
    return m


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T", [1, 3, 8])
def test_experts_differences_of_near_products(B, T, fmt):
    """Two columns of h that are 2^-14 apart, relative to them, and a down row of +1 and -1 over them.

    x = (1, 2^-14, 0, ..): gate is 1 in every row, up 1 + 2^-14 in the even rows and 1 in the odd ones, both exactly.  The
    product of both columns with s = silu(1) takes one rounding each (2^-24 s), the operand of the tensor core two halves of
    11 bits (2^-22 s each), and the sum of their four parts at most four truncated additions (2^-23 s each); what silu is off
    by (2^-21 relative) is common to both.  The result 2^-14 s is 22 times all of that; h in 11 bits would be off by 2^-11 s."""
    E, H, I = 2, 256, 128
    gu, d = ones(E, 2 * I, H, fmt), ones(E, H, I, fmt)
    gu.packed[:, :I, 0] = 0x02                    # code 2 is 1.0; the low half of a byte is the even column
    gu.packed[:, I::2, 0] = 0x22
    gu.packed[:, I + 1::2, 0] = 0x02
    rows = torch.arange(H)
    d.packed[:, rows, rows % (I // 2)] = 0xA2     # +1 at the even column, -1 at the odd one
    x = torch.zeros(T, H, dtype=torch.bfloat16)
    x[:, 0], x[:, 1] = 1.0, 2.0 ** -14
    idx, w = torch.arange(T, dtype=torch.int32)[:, None] % E, torch.ones(T, 1)
    out = experts(B, fmt, x.cuda(), idx.cuda(), w.cuda(), on_gpu(B, gu, False), on_gpu(B, d, False))
    s = torch.sigmoid(torch.ones((), dtype=torch.float64)).expand(T, H)
    ref = s * 2.0 ** -14
    tol = s * (2 * 2.0 ** -24 + 2 * 2.0 ** -22 + 4 * 2.0 ** -23) + (2.0 ** -20 + R.half_step(x.dtype)) * ref
    R.check(out, ref, tol)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,k", [(7, 18), (8, 15), (4, 31), (8, 16)])
def test_experts_of_many_rows_of_few_tokens(B, T, k, fmt):
    """Around the most rows of h that a block of the small kernel holds."""
    gu, d = R.Matrices(40, 256, 128, fmt, seed=T), R.Matrices(40, 128, 128, fmt, seed=T + 1)
    x, (idx, w) = normal(T, 128, seed=k), routing(T, 40, k, seed=k)
    out = experts(B, fmt, x.cuda(), idx.cuda(), w.cuda(), on_gpu(B, gu, True), on_gpu(B, d, True))
    ref, tol = R.experts(x, idx, w, gu, d)
    R.check(out, ref, tol)
