"""Few-token operators where their definitions are easily missed."""
import itertools

import pytest
import torch

from . import few_reference as R
from .test_gpu_few import check_route, experts, matvec, normal, on_gpu, routing

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


# ---- MXFP4 scales far apart -----------------------------------------------------------------------------------------
@pytest.mark.parametrize("T,N,K", [(1, 128, 512), (5, 256, 1280), (8, 128, 384), (9, 128, 512), (20, 256, 640)])
@pytest.mark.parametrize("far", [28, 60, 120])
def test_mxfp4_scales_far_apart_in_a_row(B, T, N, K, far):
    """Blocks with large scales meet activations of 0: what is left comes from blocks 2^-28 and less of them, and counts."""
    m = R.Matrices(1, N, K, "mxfp4", seed=far)
    x = normal(T, K, seed=2).view(T, -1, 32).clone()
    large = torch.arange(K // 32) % 3 == 1
    m.scales[:, :, large] = 127 + far // 2
    m.scales[:, :, ~large] = 127 + far // 2 - far
    m.scales[:, ::5, ~large] -= 3
    x[:, large] = 0
    x = x.view(T, K)
    y = matvec(B, "mxfp4", x.cuda(), on_gpu(B, m, True))
    keep = m.values(0) * (~large).repeat_interleave(32)
    ref, tol = R.product(x.double(), keep)
    R.check(y, ref, tol + R.half_step(x.dtype) * (ref.abs() + tol) + 2.0 ** -133)


@pytest.mark.parametrize("T", [1, 4, 8])
def test_mxfp4_scales_of_every_size_in_a_row(B, T):
    """Scales from 2^-100 to 2^100 side by side, the activations of each block small where its scale is large."""
    K = 768
    m = R.Matrices(1, 128, K, "mxfp4", seed=3)
    e = torch.tensor([(i * 37) % 201 - 100 for i in range(K // 32)])
    m.scales[:] = (127 + e).to(torch.uint8)
    for i in range(K // 32):                      # one block at a time: the others meet zeros
        x = torch.zeros(T, K // 32, 32)
        x[:, i] = normal(T, 32, seed=i).float() * 2.0 ** (-float(e[i]))
        x = x.view(T, K).to(torch.bfloat16)
        y = matvec(B, "mxfp4", x.cuda(), on_gpu(B, m, False))
        keep = torch.zeros_like(m.values(0))
        keep[:, 32 * i:32 * i + 32] = m.values(0)[:, 32 * i:32 * i + 32]
        ref, tol = R.product(x.double(), keep)
        R.check(y, ref, tol + R.half_step(x.dtype) * (ref.abs() + tol), f"block {i}")


@pytest.mark.parametrize("T", [1, 4, 8])
def test_mxfp4_experts_with_scales_far_apart(B, T):
    """In both products: x is 0 where the gate's and up's scales are large, h where the down matrix's are."""
    E, k, H, I, far = 3, 2, 512, 384, 60
    gu, d = R.Matrices(E, 2 * I, H, "mxfp4", seed=1), R.Matrices(E, H, I, "mxfp4", seed=2)
    x, (idx, w) = normal(T, H, seed=4), routing(T, E, k, seed=T)
    large = torch.arange(H // 32) % 3 == 1
    gu.scales[:, :, large] += far
    x.view(T, -1, 32)[:, large] = 0
    large = torch.arange(I // 32) % 4 == 2
    d.scales[:, :, large] += far
    gu.packed[:, I:][:, large.repeat_interleave(32)] = 0
    out = experts(B, "mxfp4", x.cuda(), idx.cuda(), w.cuda(), on_gpu(B, gu, True), on_gpu(B, d, True))
    # the reference on matrices without the blocks that meet zeros: its bounds are those of the others
    gu.scales[:, :, torch.arange(H // 32) % 3 == 1] -= far
    d.scales[:, :, large] -= far
    ref, tol = R.experts(x, idx, w, gu, d)
    R.check(out, ref, tol)


# ---- routing ----------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("score_fn,renormalize", list(itertools.product(["sigmoid", "softmax"], [True, False])))
@pytest.mark.parametrize("E,k,n_group,topk_group", [(4, 1, 1, 1), (8, 3, 1, 1), (32, 8, 4, 2), (40, 6, 8, 3), (64, 8, 1, 1),
                                                    (256, 8, 8, 4), (1024, 20, 16, 5)])
def test_route_of_zeros_of_both_signs(B, E, k, n_group, topk_group, score_fn, renormalize):
    """-0 and +0 are equal: the lower index first, with few zeros and with many."""
    g = torch.Generator().manual_seed(E)
    zeros = torch.where(torch.rand(24, E, generator=g) < 0.5, -0.0, 0.0)
    negative = -1.0 - torch.rand(24, E, generator=g)
    logits = torch.where(torch.rand(24, E, generator=g) < torch.linspace(0.02, 1.0, 24)[:, None], zeros, negative)
    logits[0] = negative[0]
    logits[0, 0], logits[0, 1] = -0.0, 0.0
    logits[1] = logits[0].flip(0)
    logits[2, ::3] = 1.0
    for bias in (None, torch.zeros(E), torch.full((E,), -0.0)):
        check_route(B, logits, bias, k, score_fn=score_fn, renormalize=renormalize, n_group=n_group, topk_group=topk_group,
                    group_best=1)


def test_route_of_zeros_agrees_with_the_plain_router(B):
    logits = torch.where(torch.rand(40, 96, generator=torch.Generator().manual_seed(1)) < 0.5, -0.0, 0.0).cuda()
    logits[:20] -= (torch.arange(96, device="cuda") % 7 > 1).float()
    for score_fn, renorm in itertools.product(["sigmoid", "softmax"], [True, False]):
        assert torch.equal(B.moe_route_topk(logits, 8, score_fn, renorm)[0], B.moe_route_grouped(logits, 8, score_fn, renorm)[0])


@pytest.mark.parametrize("score_fn,renormalize", list(itertools.product(["sigmoid", "softmax"], [True, False])))
@pytest.mark.parametrize("scale", [2.5, -1.0, 9.9e29, 1e-20])
def test_route_weights_of_logits_far_to_the_left(B, score_fn, renormalize, scale):
    """Scores below float32's numbers: their ratios are the weights, and a large factor brings them back."""
    g = torch.Generator().manual_seed(4)
    logits = -90.0 - 60.0 * torch.rand(12, 64, generator=g)
    logits[0] = -100.0 - torch.arange(64)
    logits[1, :2] = torch.tensor([-90.0, -90.1])
    logits[2] *= 4.0                               # down to -600
    logits[3, 5] = -5.0
    logits[4, 9] = 3.0
    logits[5, ::2] = -float("inf")
    logits[6] = -800.0 - torch.arange(64)          # below e^-709 a sigmoid counts as 0
    logits[7] = torch.finfo(torch.float32).min
    logits[7, 3] = -700.0
    logits[8] = -16.0 - torch.rand(64, generator=g)
    logits[9] = -80.0 - 16.0 * torch.rand(64, generator=g)
    logits[10] = torch.finfo(torch.float32).min
    logits[11] = 40.0 - 4.0 * torch.arange(64)
    for bias in (None, 0.1 * torch.randn(64, generator=g)):
        check_route(B, logits, bias, 4, score_fn=score_fn, renormalize=renormalize, scale=scale)
        check_route(B, logits, bias, 30, score_fn=score_fn, renormalize=renormalize, scale=scale, n_group=8, topk_group=5)


INF, MIN, MAX = float("inf"), torch.finfo(torch.float32).min, torch.finfo(torch.float32).max


def bias_of(kind, E, n_group, g):
    """Biases of which some are the type's ends; the others random."""
    b = (0.1 * torch.randn(E, generator=g)).view(n_group, -1)
    per = b.shape[1]
    if kind == "one infinite, the rest masked":          # the sum of two is -inf: the last group
        b[0, 0], b[0, 1:] = INF, -INF
    elif kind == "one infinite":
        b[n_group - 1, 0] = INF
    elif kind == "infinite in several":
        b[0, 0] = INF
        b[1, :2] = INF
        b[n_group - 1, per - 1] = MAX
    elif kind == "all infinite":
        b[:] = INF
    elif kind == "all the largest":
        b[:] = MAX
    elif kind == "a group of the lowest":
        b[1] = MIN
    elif kind == "a group masked":
        b[0] = -INF
    elif kind == "lowest and masked":
        b[0], b[1] = -INF, MIN
        b[2:, 1:] = MIN
    elif kind == "all but one masked":
        b[:, 1:] = -INF
    elif kind == "one expert left":
        b[:] = -INF
        b[n_group - 1, 1] = 0.0
    elif kind == "-1e9":
        b[1] = -1e9
        b[2, 1:] = -1e9
    elif kind == "nan":
        b[0] = float("nan")
        b[2, 0] = INF
    return b.reshape(E)


@pytest.mark.parametrize("kind", [
    "one infinite, the rest masked", "one infinite", "infinite in several", "all infinite", "all the largest",
    "a group of the lowest", "a group masked", "lowest and masked", "all but one masked", "one expert left", "-1e9", "nan"])
@pytest.mark.parametrize("E,k,n_group,topk_group", [(8, 2, 4, 1), (32, 4, 4, 2), (64, 8, 8, 3), (64, 8, 32, 20), (40, 6, 4, 3),
                                                    (256, 8, 8, 4), (512, 8, 4, 1)])
def test_route_of_biases_at_the_ends_of_the_type(B, E, k, n_group, topk_group, kind):
    """+inf is the largest float32, NaN is -inf, and sums are those of float64: (largest + largest) is above (largest + 1),
    (lowest + lowest) above -inf."""
    g = torch.Generator().manual_seed(E)
    logits = torch.randn(20, E, generator=g)
    bias = bias_of(kind, E, n_group, g)
    for score_fn, best, groups in itertools.product(["sigmoid", "softmax"], [2, 1], [n_group, 1]):
        keep = topk_group if groups > 1 else 1
        idx, w = B.moe_route_grouped(logits.cuda(), k, score_fn, select_bias=bias.cuda(), n_group=groups, topk_group=keep,
                                     group_best=best)
        for t in range(20):
            ri, rw = R.route(logits[t], bias, k, score_fn, True, groups, keep, best, 1.0)
            assert idx[t].tolist() == ri, (score_fn, best, groups, t)
            ref = torch.tensor(rw, dtype=torch.float64)
            assert ((w[t].double().cpu() - ref).abs() <= 1e-6 * ref).all()
    B.sync_status()


@pytest.mark.parametrize("mask", [-INF, MIN, -1e9, -1000.0])
@pytest.mark.parametrize("spread", [1.0, 2.0 ** -13, 2.0 ** -20])
def test_route_of_close_scores_beside_masked_groups(B, spread, mask):
    """Groups that are close to one another and groups, or most of a group's experts, that are far below all."""
    g = torch.Generator().manual_seed(7)
    logits = 0.5 + spread * torch.randn(200, 64, generator=g)
    logits[::4] = 0.5 + spread * torch.randint(0, 4, (50, 64), generator=g).float()
    bias = spread * torch.randint(-3, 4, (64,), generator=g).float()
    bias[8:16] = mask
    bias[17:24] = mask
    for score_fn, keep, best in itertools.product(["sigmoid", "softmax"], [2, 6], [1, 2]):
        check_route(B, logits, bias, 8, score_fn=score_fn, n_group=8, topk_group=keep, group_best=best)
