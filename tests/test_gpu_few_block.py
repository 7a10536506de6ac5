"""The few-token operators as they are used together: a layer with grouped routing and few tokens, and decode steps of the
example's block (page plan, attention, router, experts) as graphs."""
import pytest
import torch

from . import few_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from nvfp4_block_scaled_07_gb300 import build
    build.build()
    from nvfp4_block_scaled_07_gb300 import binding
    binding.device_check()
    binding.sync_status()
    return binding


def weights(E, H, I, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [(torch.randn(s, generator=g, device="cuda") * 0.05).to(torch.bfloat16) for s in ((E, 2 * I, H), (E, H, I))]


def batch(T, H, E, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16), torch.randn((T, E), generator=g, device="cuda")


GROUPS = dict(n_group=4, topk_group=2, group_best=2, routed_scale=2.5)


@pytest.mark.parametrize("fmt,tiled", [("nvfp4", True), ("nvfp4", False), ("mxfp4", True)])
@pytest.mark.parametrize("T", [1, 4, 9, 32])
def test_layer_of_few_tokens_is_its_two_calls(B, fmt, tiled, T):
    gu, d = weights(16, 256, 384)
    bias = torch.linspace(-0.2, 0.2, 16, device="cuda")
    layer = B.MoELayer(gu, d, 4, fmt=fmt, tiled_weights=tiled, select_bias=bias, few_tokens=32, **GROUPS)
    x, logits = batch(T, 256, 16, seed=T)
    y = layer(x, logits).clone()
    idx, w = B.moe_route_grouped(logits, 4, select_bias=bias, n_group=4, topk_group=2, scale=2.5)
    assert torch.equal(layer.topk_idx, idx) and torch.equal(layer.topk_w, w)
    args = [layer.w_gu_packed, layer.w_gu_scales, layer.w_d_packed, layer.w_d_scales]
    if fmt == "nvfp4":
        want = B.moe_experts_nvfp4(x, idx, w, args[0], args[1], layer.w_gu_gscale, args[2], args[3], layer.w_d_gscale)
        assert layer.launches_per_forward == 1 + B._lib.moe_experts_launches(T, 4, 256, 384)
    else:
        want = B.moe_experts_mxfp4(x, idx, w, *args)
    assert torch.equal(y, want)
    for step in (lambda: layer.prepare(x, logits), layer.gemm_gate_up, layer.gemm_down, layer.finalize,
                 lambda: layer.autotune(x, logits)):
        with pytest.raises(ValueError, match="steps"):
            step()
    out = torch.empty_like(y)
    assert layer(x, logits, out=out) is out and torch.equal(out, y)
    B.sync_status()


@pytest.mark.parametrize("k_primary", [None, 2])
def test_layer_of_few_tokens_with_the_other_routers(B, k_primary):
    gu, d = weights(16, 256, 128)
    bias = torch.linspace(-0.3, 0.3, 16, device="cuda")
    few = B.MoELayer(gu, d, 4, bias=bias, k_primary=k_primary, few_tokens=16, score_fn="softmax")
    many = B.MoELayer(gu, d, 4, bias=bias, k_primary=k_primary, score_fn="softmax", autotune=False, fused_prepare=False)
    x, logits = batch(11, 256, 16, seed=9)
    y = few(x, logits)
    many(x, logits)
    assert torch.equal(few.topk_idx, many.topk_idx) and torch.equal(few.topk_w, many.topk_w)
    assert torch.equal(y, B.moe_experts_nvfp4(x, many.topk_idx, many.topk_w, few.w_gu_packed, few.w_gu_scales, few.w_gu_gscale,
                                              few.w_d_packed, few.w_d_scales, few.w_d_gscale))
    assert few.launches_per_forward == (1 if k_primary is None else 2) + B._lib.moe_experts_launches(11, 4, 256, 128)
    B.sync_status()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_layer_of_few_tokens_is_near_the_quantised_one(B, fmt):
    """The large-batch form quantises x and h to four bits: each by up to half a step of 1 / 6 of a block's largest value,
    about a tenth of a normal value's size each, so a quarter of the result's size is never reached."""
    gu, d = weights(16, 512, 256)
    few = B.MoELayer(gu, d, 4, fmt=fmt, few_tokens=32, autotune=False, **GROUPS)
    many = B.MoELayer(gu, d, 4, fmt=fmt, autotune=False, **GROUPS)
    assert not many.fused_prepare
    x, logits = batch(20, 512, 16, seed=3)
    a, b = few(x, logits).float(), many(x, logits).float()
    B.sync_status()
    assert torch.equal(few.topk_idx, many.topk_idx) and torch.equal(few.topk_w, many.topk_w)
    assert float((a - b).norm() / b.norm()) < 0.25
    # and the same layer takes both kinds of batches in turn
    x2, logits2 = batch(40, 512, 16, seed=4)
    assert torch.equal(few(x2, logits2), many(x2, logits2))
    assert torch.equal(few(x, logits).float(), a)
    B.sync_status()


@pytest.mark.parametrize("T", [3, 40])
def test_layer_capture(B, T):
    gu, d = weights(16, 256, 256)
    layer = B.MoELayer(gu, d, 2, few_tokens=8, autotune=False, **GROUPS)
    x, logits = batch(T, 256, 16, seed=1)
    graph = layer.capture(x, logits)
    for seed in (2, 3):
        nx, nl = batch(T, 256, 16, seed=seed)
        x.copy_(nx), logits.copy_(nl)
        graph.replay()
        got = layer.out.clone()
        assert torch.equal(layer(x, logits), got)
    B.sync_status()


def test_layer_refusals(B):
    gu, d = weights(8, 256, 128)
    with pytest.raises(ValueError, match="few_tokens"):
        B.MoELayer(gu, d, 2, few_tokens=33)
    with pytest.raises(ValueError, match="exclude"):
        B.MoELayer(gu, d, 2, bias=torch.zeros(8, device="cuda"), n_group=2)
    with pytest.raises(ValueError, match="exclude"):
        B.MoELayer(gu, d, 2, k_primary=1, routed_scale=2.0)


def test_empty_batch(B):
    gu, d = weights(8, 256, 128)
    layer = B.MoELayer(gu, d, 2, few_tokens=4, **GROUPS)
    x, logits = batch(0, 256, 8, seed=1)
    assert layer(x, logits).shape == (0, 256)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("lengths", [(37, 130, 5), (63,), (64, 1)])
def test_decode_steps_as_graphs(B, fmt, lengths):
    """Page plan, latent attention, grouped router and experts in one graph give the eager steps' bits."""
    from examples import decoder_block as E
    block = E.Block(fmt=fmt, few_tokens=8, select_bias=torch.linspace(-0.1, 0.1, 8, device="cuda"), **GROUPS)
    eager, whole = E.serve(lengths=lengths, steps=3, block=block)
    graph, _ = E.serve(lengths=lengths, steps=3, block=block, graph=True)
    assert torch.equal(eager, graph) and bool(eager.isfinite().all())
    # prefill quantises the experts' input to four bits and decoding does not: a tenth of the experts' part each, which with
    # a factor of 2.5 is about as large as the residual
    assert float((eager.double() - whole.double()).norm() / whole.double().norm()) < 0.25


def test_prefill_between_steps_of_a_graph(B):
    """A batch of another size in between replaces the layer's buffers, not those of the captured step."""
    from examples import decoder_block as E
    block = E.Block(few_tokens=8, **GROUPS)
    x = torch.randn((2, 3, block.D), generator=torch.Generator(device="cuda").manual_seed(5), device="cuda").bfloat16()

    def steps(between):
        cache = torch.zeros((3, E.PAGE, E.mla.ROW), dtype=torch.bfloat16, device="cuda")
        lens, free, count = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 0, 0], [2, 0, 1], [3]))
        step = E.Stepper(block, cache, lens, torch.full((3, 1), -1, dtype=torch.int32, device="cuda"), free, count)
        first = step(x[0]).clone()
        if between:
            for T in (20, 5, 40):
                kept = [block.experts(*batch(T, block.D, 8, seed=T)) for _ in range(2)]
            del kept
        return first, step(x[1]).clone()

    plain, mixed = steps(False), steps(True)
    assert all(torch.equal(a, b) and bool(a.isfinite().all()) for a, b in zip(plain, mixed))
    B.sync_status()


def test_calls_at_once_on_two_streams(B):
    """Calls with workspaces of their own, on two streams at the same time, each give what they give alone."""
    gu, d = R.Matrices(8, 1024, 512, "nvfp4", 1), R.Matrices(8, 512, 512, "nvfp4", 2)
    args = [t for m in (gu, d) for t in (m.packed.cuda(), m.blocked().cuda(), m.gscale.cuda())]
    m = R.Matrices(1, 2048, 2048, "mxfp4", 3)
    dense = (m.packed.cuda()[0], m.blocked().cuda())
    calls = []
    for T in (2, 20):
        x, logits = batch(T, 512, 8, seed=T)
        idx, w = B.moe_route_grouped(logits, 2)
        z = batch(T, 2048, 1, seed=T + 1)[0]
        calls.append(lambda x=x, idx=idx, w=w: B.moe_experts_nvfp4(x, idx, w, *args))
        calls.append(lambda z=z: B.moe_matvec_mxfp4(z, *dense))
    want = [call() for call in calls]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in calls]
    got = [[] for _ in calls]
    for _ in range(20):
        for side, call, outs in zip(sides, calls, got):
            with torch.cuda.stream(side):
                outs.append(call())
    torch.cuda.synchronize()
    assert all(torch.equal(o, y) for y, outs in zip(want, got) for o in outs)
    B.sync_status()


def test_two_graphs_with_one_workspace_in_turn(B):
    gu, d = R.Matrices(8, 512, 512, "nvfp4", 1), R.Matrices(8, 512, 256, "nvfp4", 2)
    args = [t for m in (gu, d) for t in (m.packed.cuda(), m.blocked().cuda(), m.gscale.cuda())]
    ws = torch.empty(B.moe_experts_workspace_size(20, 2, 512, 256), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    made = []
    for T in (20, 3, 12):
        x, logits = batch(T, 512, 8, seed=T)
        idx, w = B.moe_route_grouped(logits, 2)
        out = torch.empty_like(x)

        def call():
            B.moe_experts_nvfp4(x, idx, w, *args, out=out, workspace=ws)

        want = B.moe_experts_nvfp4(x, idx, w, *args)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                call()
        made.append((graph, out, want, (x, idx, w)))
    for _ in range(3):
        for graph, out, want, _ in made:
            out.fill_(float("nan"))
            graph.replay()
            assert torch.equal(out, want)
    B.sync_status()
