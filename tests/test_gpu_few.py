"""Few-token operators on the GPU against their 64-bit definitions: matrix-vector products with 4-bit weights, the
experts' products, grouped routing."""
import itertools

import pytest
import torch

from . import few_reference as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def B():
    from nvfp4_block_scaled_07_gb300 import build
    build.build()
    from nvfp4_block_scaled_07_gb300 import binding
    binding.device_check()
    binding.sync_status()
    return binding


def on_gpu(B, m, tiled):
    packed = m.packed.cuda()
    return (B.tile_expert_weights(packed) if tiled else packed, m.blocked().cuda(),
            None if m.gscale is None else m.gscale.cuda())


def matvec(B, fmt, x, w, **kw):
    return B.moe_matvec_nvfp4(x, *w, **kw) if fmt == "nvfp4" else B.moe_matvec_mxfp4(x, *w[:2], **kw)


def normal(*shape, seed=0, dtype=torch.bfloat16):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


# ---- matrix-vector products ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("fmt,tiled,dtype", list(itertools.product(["nvfp4", "mxfp4"], [False, True], ["bf16", "fp16"])))
@pytest.mark.parametrize("T,N,K", [(1, 128, 128), (2, 256, 384), (3, 128, 640), (5, 384, 1024), (8, 128, 2048), (9, 256, 256),
                                   (16, 128, 1152), (17, 128, 384), (25, 256, 896), (32, 384, 512), (1, 640, 14336),
                                   (7, 128, 9088), (32, 128, 4224), (32, 1024, 4224), (17, 512, 2304), (31, 8192, 640), (9, 4096, 1152), (20, 256, 128), (4, 1152, 4096), (8, 640, 2048), (1, 4096, 9088)])
def test_matvec(B, T, N, K, fmt, tiled, dtype):
    m = R.Matrices(1, N, K, fmt, seed=T + N)
    x = normal(T, K, seed=K, dtype=DT[dtype])
    y = matvec(B, fmt, x.cuda(), on_gpu(B, m, tiled))
    B.sync_status()
    ref, tol = R.product(x.double(), m.values(0))
    R.check(y, ref, tol + R.half_step(x.dtype) * (ref.abs() + tol) + 2.0 ** -25)


@pytest.mark.parametrize("T,K", [(1, 64), (3, 192), (12, 320), (4, 4160)])
def test_matvec_of_a_partial_step(B, T, K):
    """NVFP4 columns that are no multiple of 128; a tiled matrix pads them."""
    m = R.Matrices(1, 128, K, "nvfp4", seed=K)
    x = normal(T, K, seed=1)
    for tiled in (False, True):
        y = matvec(B, "nvfp4", x.cuda(), on_gpu(B, m, tiled))
        ref, tol = R.product(x.double(), m.values(0))
        R.check(y, ref, tol + R.half_step(x.dtype) * (ref.abs() + tol) + 1e-30)


@pytest.mark.parametrize("T", [1, 2, 6, 20])
def test_matvec_views(B, T):
    """Rows of a wider tensor, one row again and again, weights that start between 32-byte boundaries, a caller's output
    and workspace: the same bits."""
    K, N = 1024, 256
    m = R.Matrices(1, N, K, "nvfp4", seed=3)
    w = on_gpu(B, m, False)
    wide = normal(T, K + 72, seed=2).cuda()
    x = wide[:, 8:8 + K]
    want = matvec(B, "nvfp4", x.contiguous(), w)
    assert torch.equal(matvec(B, "nvfp4", x, w), want)
    out = torch.full_like(want, float("nan"))
    ws = torch.empty(max(256, B.moe_matvec_workspace_size(T, N, K)), dtype=torch.uint8, device="cuda")
    assert matvec(B, "nvfp4", x, w, out=out, workspace=ws) is out and torch.equal(out, want)
    same = x[:1].expand(T, K)
    assert torch.equal(matvec(B, "nvfp4", same, w), matvec(B, "nvfp4", same.contiguous(), w))
    room = torch.zeros(m.packed.numel() + 16, dtype=torch.uint8, device="cuda")
    shifted = room[16:].view(1, N, K // 2)
    shifted.copy_(w[0])
    assert shifted.data_ptr() % 32 == 16
    assert torch.equal(matvec(B, "nvfp4", x, (shifted, *w[1:])), want)
    assert torch.equal(matvec(B, "nvfp4", x, (w[0][0], *w[1:])), want)          # [N, K/2]


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("exponent", [-100, -20, 20, 90])
def test_matvec_scales_with_its_input(B, fmt, exponent):
    """Powers of two pass through every step exactly: a row's results have the same bits but for the exponent."""
    m = R.Matrices(1, 128, 768, fmt, seed=5)
    w = on_gpu(B, m, True)
    x = normal(3, 768, seed=4).cuda()
    y = matvec(B, fmt, x, w).double()
    x[1] *= 2.0 ** exponent
    z = matvec(B, fmt, x, w).double()
    assert torch.equal(z[0], y[0]) and torch.equal(z[2], y[2]) and torch.equal(z[1], y[1] * 2.0 ** exponent)


def test_matvec_keeps_infinities_and_nan_in_their_rows(B):
    m = R.Matrices(1, 128, 512, "nvfp4", seed=6)
    w = on_gpu(B, m, False)
    x = normal(5, 512, seed=5).cuda()
    y = matvec(B, "nvfp4", x, w)
    x[1, 300], x[3, 7] = float("inf"), float("nan")
    z = matvec(B, "nvfp4", x, w)
    assert torch.equal(z[[0, 2, 4]], y[[0, 2, 4]]) and z[3].isnan().all()
    column = m.values(0)[:, 300]
    assert torch.equal(z[1].cpu() == float("inf"), column > 0) and torch.equal(z[1].cpu() == -float("inf"), column < 0)


@pytest.mark.parametrize("T", [9, 20])
def test_matvec_stream_of_special_rows(B, T):
    """An infinity, a NaN, zeros, tiny and huge rows among others: each row's results are its own."""
    m = R.Matrices(1, 256, 1536, "nvfp4", seed=6)
    w = on_gpu(B, m, False)
    x = normal(T, 1536, seed=5).cuda()
    y = matvec(B, "nvfp4", x, w)
    x[1, 300], x[3, 7] = float("inf"), float("nan")
    x[4] = 0.0
    x[5] *= 2.0 ** -60
    x[6] *= 2.0 ** 90
    z = matvec(B, "nvfp4", x, w)
    same = [t for t in range(T) if t not in (1, 3, 4, 5, 6)]
    assert torch.equal(z[same], y[same]) and not z[[1, 3]].isfinite().any() and (z[4] == 0).all()
    assert torch.equal(z[5].double(), y[5].double() * 2.0 ** -60) and torch.equal(z[6].double(), y[6].double() * 2.0 ** 90)


def test_matvec_of_zeros(B):
    m = R.Matrices(1, 128, 512, "nvfp4", seed=6)
    assert (matvec(B, "nvfp4", torch.zeros(4, 512, dtype=torch.bfloat16, device="cuda"), on_gpu(B, m, False)) == 0).all()
    m.scales.zero_()
    assert (matvec(B, "nvfp4", normal(4, 512).cuda(), on_gpu(B, m, False)) == 0).all()
    assert matvec(B, "nvfp4", normal(0, 512).cuda(), on_gpu(B, m, False)).shape == (0, 128)


@pytest.mark.parametrize("fmt,lo,hi", [("nvfp4", 0, 0x10), ("nvfp4", 0, 0x7F), ("nvfp4", 0x78, 0x7F), ("mxfp4", 1, 20),
                                       ("mxfp4", 220, 240), ("mxfp4", 100, 127), ("mxfp4", 127, 150)])
@pytest.mark.parametrize("T", [6, 11, 20])
def test_matvec_takes_the_scales_range(B, fmt, lo, hi, T):
    """Subnormal and the largest ue4m3 scales, small and large E8M0 ones, up to 2^26 apart in a row."""
    m = R.Matrices(1, 128, 1280, fmt, seed=lo, lo=lo, hi=hi)
    if fmt == "mxfp4" and hi > 200:
        x = normal(T, 1280, seed=9).float() * 2.0 ** -110
    elif fmt == "mxfp4" and hi < 50:
        x = normal(T, 1280, seed=9).float() * 2.0 ** 110
    else:
        x = normal(T, 1280, seed=9).float()
    x = x.to(torch.bfloat16)
    y = matvec(B, fmt, x.cuda(), on_gpu(B, m, True))
    ref, tol = R.product(x.double(), m.values(0))
    R.check(y, ref, tol + R.half_step(x.dtype) * (ref.abs() + tol) + 2.0 ** -133)


def test_matvec_of_a_wide_range_of_activations(B):
    """Values down to 2^-28 of the largest of their 256 are exact: here the large ones meet zero weights."""
    m = R.Matrices(1, 128, 512, "nvfp4", seed=8)
    m.packed[:, :, ::8] = 0
    x = normal(4, 512, seed=3).double() * 2.0 ** -20
    x = x.to(torch.bfloat16)
    x[:, 0::16] = 100.0
    x[:, 1::16] = -77.0
    y = matvec(B, "nvfp4", x.cuda(), on_gpu(B, m, False))
    small = x.clone()
    small[:, 0::16] = 0
    small[:, 1::16] = 0
    ref, tol = R.product(small.double(), m.values(0))
    wsum = m.values(0).abs().sum(1)
    R.check(y, ref, tol + 2.0 ** -38 * 100.0 * wsum + R.half_step(x.dtype) * (ref.abs() + tol))


def test_matvec_rows_do_not_see_each_other(B):
    """A token alone and among others, of each size class, gives the same up to the order of sums."""
    K = 1280
    m = R.Matrices(1, 256, K, "mxfp4", seed=2)
    w = on_gpu(B, m, True)
    x = normal(32, K, seed=1).cuda()
    ref, tol = R.product(x.double().cpu(), m.values(0))
    tol = tol + R.half_step(x.dtype) * (ref.abs() + tol)
    for T in (1, 2, 4, 8, 9, 16, 17, 32):
        y = matvec(B, "mxfp4", x[:T], w)
        R.check(y, ref[:T], tol[:T], f"T = {T}")
        assert torch.equal(y, matvec(B, "mxfp4", x[:T], w))


# ---- the experts' products ----------------------------------------------------------------------------------------
def layer(E, H, I, fmt, seed):
    return R.Matrices(E, 2 * I, H, fmt, seed), R.Matrices(E, H, I, fmt, seed + 1)


def experts(B, fmt, x, idx, w, gu, d, **kw):
    if fmt == "nvfp4":
        return B.moe_experts_nvfp4(x, idx, w, *gu, *d, **kw)
    return B.moe_experts_mxfp4(x, idx, w, *gu[:2], *d[:2], **kw)


def routing(T, E, k, seed):
    g = torch.Generator().manual_seed(seed)
    idx = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int() if T else torch.zeros(0, k).int()
    return idx, torch.rand(T, k, generator=g)


@pytest.mark.parametrize("fmt,tiled", list(itertools.product(["nvfp4", "mxfp4"], [False, True])))
@pytest.mark.parametrize("T,E,k,H,I", [(1, 4, 2, 256, 128), (1, 1, 1, 128, 128), (3, 8, 2, 256, 128), (8, 8, 8, 384, 256),
                                       (9, 16, 4, 256, 384), (16, 5, 3, 128, 256), (23, 40, 8, 256, 128),
                                       (32, 3, 1, 256, 256), (32, 64, 6, 128, 128), (32, 128, 32, 128, 128), (8, 1024, 32, 128, 128), (2, 6, 3, 4096, 640), (1, 12, 8, 640, 2304)])
def test_experts(B, T, E, k, H, I, fmt, tiled):
    gu, d = layer(E, H, I, fmt, seed=T + E)
    x = normal(T, H, seed=I)
    idx, w = routing(T, E, k, seed=k)
    out = experts(B, fmt, x.cuda(), idx.cuda(), w.cuda(), on_gpu(B, gu, tiled), on_gpu(B, d, tiled))
    B.sync_status()
    ref, tol = R.experts(x, idx, w, gu, d)
    R.check(out, ref, tol)


@pytest.mark.parametrize("T", [1, 6, 20])
def test_experts_named_twice(B, T):
    """An expert that a token names twice or three times gets the sum of the weights."""
    gu, d = layer(4, 256, 128, "nvfp4", seed=1)
    x = normal(T, 256, seed=2)
    idx, w = routing(T, 4, 3, seed=5)
    idx[::2, 1] = idx[::2, 0]
    idx[::3] = 2
    out = experts(B, "nvfp4", x.cuda(), idx.cuda(), w.cuda(), on_gpu(B, gu, False), on_gpu(B, d, False))
    ref, tol = R.experts(x, idx, w, gu, d)
    R.check(out, ref, tol)


@pytest.mark.parametrize("T", [1, 5, 17])
def test_experts_ids_out_of_range(B, T):
    """Contribute nothing and are reported; a token with none of its experts gets zeros."""
    gu, d = layer(4, 256, 128, "mxfp4", seed=1)
    gu_g, d_g = on_gpu(B, gu, True), on_gpu(B, d, True)
    x = normal(T, 256, seed=2)
    idx, w = routing(T, 4, 3, seed=5)
    idx[0] = torch.tensor([-1, 4, 2 ** 31 - 1])
    if T > 1:
        idx[T - 1, 1] = -7
    out = torch.full((T, 256), float("nan"), dtype=torch.bfloat16, device="cuda")
    experts(B, "mxfp4", x.cuda(), idx.cuda(), w.cuda(), gu_g, d_g, out=out)
    with pytest.raises(B.Nvfp4MoeError) as e:
        B.sync_status()
    assert e.value.status == B.ERR_DEVICE_DATA
    ref, tol = R.experts(x, idx, w, gu, d)
    R.check(out, ref, tol)
    assert (out[0] == 0).all()
    B.sync_status()


def test_experts_do_not_reach_tokens_that_are_not_theirs(B):
    """A NaN scale of an expert, an infinite token: only what is routed to them sees them."""
    gu, d = layer(6, 256, 128, "nvfp4", seed=3)
    x = normal(12, 256, seed=3)
    idx, w = routing(12, 6, 2, seed=9)           # more than eight tokens: the stream kernel
    want = experts(B, "nvfp4", x.cuda(), idx.cuda(), w.cuda(), on_gpu(B, gu, False), on_gpu(B, d, False))
    gu.scales[2, 5, 3] = 0x7F
    d.scales[4, 7, 2] = 0x7F
    x[3, 10] = float("inf")
    got = experts(B, "nvfp4", x.cuda(), idx.cuda(), w.cuda(), on_gpu(B, gu, False), on_gpu(B, d, False))
    for t in range(12):
        if t == 3:
            assert not got[t].isfinite().any()
        elif 2 in idx[t]:
            assert got[t].isnan().all()
        elif 4 in idx[t]:
            assert got[t, 7].isnan() and torch.equal(got[t, :7], want[t, :7]) and torch.equal(got[t, 8:], want[t, 8:])
        else:
            assert torch.equal(got[t], want[t])


def test_experts_views_workspace_and_repeats(B):
    gu, d = layer(8, 512, 256, "nvfp4", seed=3)
    gu, d = on_gpu(B, gu, True), on_gpu(B, d, True)
    idx, w = routing(32, 8, 4, seed=1)
    idx, w = idx.cuda(), w.cuda()
    wide = normal(32, 600, seed=1).cuda()
    ws = torch.empty(B.moe_experts_workspace_size(32, 4, 512, 256), dtype=torch.uint8, device="cuda")
    for T in (32, 1, 9, 32):                   # one workspace, whatever it holds
        x = wide[:T, 16:528]
        want = experts(B, "nvfp4", x.contiguous(), idx[:T], w[:T], gu, d)
        ws.fill_(0xFF)
        assert torch.equal(experts(B, "nvfp4", x, idx[:T], w[:T], gu, d, workspace=ws), want)
        assert torch.equal(experts(B, "nvfp4", x, idx[:T], w[:T], gu, d, workspace=ws), want)
    assert experts(B, "nvfp4", wide[:0, :512], idx[:0], w[:0], gu, d).shape == (0, 512)


def test_few_calls_in_a_graph_and_on_a_stream(B):
    """Captured once, replayed on new inputs; the same bits as eager calls on another stream."""
    gu, d = layer(8, 512, 256, "mxfp4", seed=3)
    gu, d = on_gpu(B, gu, True), on_gpu(B, d, True)
    x, logits = normal(6, 512, seed=1).cuda(), normal(6, 8, seed=2).float().cuda()
    bias = torch.linspace(-0.1, 0.1, 8, device="cuda")
    ws = torch.empty(B.moe_experts_workspace_size(6, 2, 512, 256), dtype=torch.uint8, device="cuda")
    idx, w, out = torch.empty(6, 2, dtype=torch.int32, device="cuda"), torch.empty(6, 2, device="cuda"), torch.empty_like(x)

    def step():
        B.moe_route_grouped(logits, 2, select_bias=bias, n_group=4, topk_group=2, topk_idx=idx, topk_w=w)
        experts(B, "mxfp4", x, idx, w, gu, d, out=out, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    for seed in (5, 6, 7):
        x.copy_(normal(6, 512, seed=seed))
        logits.copy_(normal(6, 8, seed=seed + 50).float())
        graph.replay()
        got = out.clone()
        out.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            step()
        side.synchronize()
        assert torch.equal(got, out)
    B.sync_status()


# ---- grouped routing ----------------------------------------------------------------------------------------------
def check_route(B, logits, bias, k, **kw):
    idx, w = B.moe_route_grouped(logits.cuda(), k, select_bias=None if bias is None else bias.cuda(), **kw)
    B.sync_status()
    args = dict(score_fn="sigmoid", renormalize=True, n_group=1, topk_group=1, group_best=2, scale=1.0) | kw
    args["renorm"] = args.pop("renormalize")
    for t in range(logits.shape[0]):
        ri, rw = R.route(logits[t], bias, k, **args)
        if idx[t].tolist() != ri and args["n_group"] > 1:       # another of the choices that float64 leaves open?
            for kept in R.groups_that_tie(logits[t], bias, k, **args):
                oi, ow = R.route(logits[t], bias, k, **args, kept=kept)
                if oi == idx[t].tolist():
                    ri, rw = oi, ow
        assert idx[t].tolist() == ri, (t, idx[t].tolist(), ri)
        ref = torch.tensor(rw, dtype=torch.float64)
        assert ((w[t].double().cpu() - ref).abs() <= 1e-6 * ref.abs() + 1e-37).all(), (t, w[t].tolist(), rw)


@pytest.mark.parametrize("score_fn,renormalize,with_bias", list(itertools.product(["sigmoid", "softmax"], [True, False], [True, False])))
@pytest.mark.parametrize("T,E,k,n_group,topk_group,group_best", [
    (1, 256, 8, 8, 4, 2), (37, 256, 8, 8, 4, 2), (64, 256, 8, 1, 1, 2), (9, 8, 2, 2, 1, 2), (33, 40, 6, 8, 3, 2),
    (16, 160, 6, 8, 3, 1), (20, 64, 6, 1, 1, 1), (5, 1, 1, 1, 1, 1), (11, 512, 10, 8, 2, 2), (7, 1024, 32, 32, 9, 2),
    (13, 1000, 7, 10, 10, 1), (6, 384, 1, 32, 1, 2), (17, 33, 33 - 1, 1, 1, 2), (10, 72, 9, 24, 5, 1)])
def test_route(B, T, E, k, n_group, topk_group, group_best, score_fn, renormalize, with_bias):
    g = torch.Generator().manual_seed(T * E)
    logits = torch.randn(T, E, generator=g) * 1.5
    bias = 0.1 * torch.randn(E, generator=g) if with_bias else None
    check_route(B, logits, bias, k, score_fn=score_fn, renormalize=renormalize, n_group=n_group, topk_group=topk_group,
                group_best=group_best, scale=2.5)


@pytest.mark.parametrize("score_fn", ["sigmoid", "softmax"])
def test_route_of_near_and_exact_ties(B, score_fn):
    """Scores that float32 cannot tell apart, far out on the sigmoid and one step of a logit apart; equal ones go to the
    lower index."""
    g = torch.Generator().manual_seed(1)
    rows = [torch.zeros(64), torch.full((64,), 3.0), torch.randint(-2, 3, (64,), generator=g).float()]
    base = torch.full((64,), 12.0)
    for i in range(64):
        base[i] = torch.tensor(12.0 + ((i * 37) % 64) * 2.0 ** -20)
    rows += [base, -base, base.flip(0), 9.0 + torch.rand(64, generator=g) * 2.0 ** -18]
    logits = torch.stack(rows)
    for bias in (None, torch.zeros(64), torch.full((64,), 0.125), (torch.arange(64) % 4) * 0.25):
        for groups, keep, best in ((1, 1, 1), (8, 3, 2), (8, 3, 1)):
            check_route(B, logits, bias, 8, score_fn=score_fn, n_group=groups, topk_group=keep, group_best=best)


@pytest.mark.parametrize("E,k,n_group,topk_group,group_best", [(256, 8, 8, 4, 2), (256, 6, 8, 3, 1), (60, 4, 6, 3, 2), (96, 9, 32, 20, 2),
                                                              (128, 8, 32, 3, 2), (1024, 20, 16, 5, 2), (40, 8, 20, 7, 2)])
@pytest.mark.parametrize("spread", [1.0, 2.0 ** -13, 2.0 ** -20])
def test_route_of_many_close_scores(B, E, k, n_group, topk_group, group_best, spread):
    """Scores a few float32 steps apart: of the groups, of the experts of a group's value, of the chosen; among them rows
    with many that are equal."""
    g = torch.Generator().manual_seed(E + k)
    logits = 0.5 + spread * torch.randn(1500, E, generator=g)
    logits[::5] = 0.5 + spread * torch.randint(0, 4, (300, E), generator=g).float()
    bias = spread * torch.randint(-3, 4, (E,), generator=g).float()
    for b, score_fn in ((bias, "sigmoid"), (bias, "softmax"), (None, "sigmoid")):
        check_route(B, logits, b, k, score_fn=score_fn, n_group=n_group, topk_group=topk_group, group_best=group_best)


def test_route_of_group_values_that_almost_tie(B):
    """Two groups whose sums of two differ in the last bits of float64 only."""
    logits = torch.zeros(4, 32)
    logits[:, 0], logits[:, 1] = 2.0, 1.0
    for t in range(4):
        logits[t, 8], logits[t, 9] = 2.0, 1.0 + (t - 1) * 2.0 ** -23
        logits[t, 16], logits[t, 17] = 1.0 + (t - 2) * 2.0 ** -23, 2.0
    check_route(B, logits, torch.zeros(32), 4, n_group=4, topk_group=2, group_best=2)
    check_route(B, logits, None, 4, n_group=4, topk_group=1, group_best=2)


@pytest.mark.parametrize("score_fn,renormalize", list(itertools.product(["sigmoid", "softmax"], [True, False])))
def test_route_of_masked_experts(B, score_fn, renormalize):
    """-inf and NaN logits, rows of nothing else, infinities, biases of -inf: choices in range and finite weights."""
    inf, nan = float("inf"), float("nan")
    g = torch.Generator().manual_seed(3)
    logits = torch.randn(8, 32, generator=g)
    logits[0, ::2] = -inf
    logits[1, 5:] = -inf
    logits[2] = -inf
    logits[3, 1::3] = nan
    logits[4] = nan
    logits[5, 7] = inf
    logits[6] = 200.0 * logits[6]
    logits[7] = torch.finfo(torch.float32).min
    bias = 0.1 * torch.randn(32, generator=g)
    masked = bias.clone()
    masked[::3] = -inf
    masked[1] = nan
    for b in (None, bias, masked):
        for groups, keep, best in ((1, 1, 1), (4, 2, 2), (4, 2, 1)):
            check_route(B, logits, b, 6, score_fn=score_fn, renormalize=renormalize, n_group=groups, topk_group=keep,
                        group_best=best)


def test_route_agrees_with_the_plain_router(B):
    """Without groups, bias and factor it is moe_route_topk."""
    logits = normal(50, 256, seed=1).float().cuda()
    for score_fn, renorm in itertools.product(["sigmoid", "softmax"], [True, False]):
        a, b = B.moe_route_topk(logits, 8, score_fn, renorm), B.moe_route_grouped(logits, 8, score_fn, renorm)
        assert torch.equal(a[0], b[0]) and ((a[1] - b[1]).abs() <= 2e-6 * a[1]).all()
    assert B.moe_route_grouped(logits[:0], 8)[0].shape == (0, 8)
