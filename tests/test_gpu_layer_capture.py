"""MoELayer.capture with batches of other sizes between its replays."""
import gc

import pytest
import torch

from .test_gpu_few_block import GROUPS, batch, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from nvfp4_block_scaled_07_gb300 import build
    build.build()
    from nvfp4_block_scaled_07_gb300 import binding
    binding.device_check()
    binding.sync_status()
    return binding


@pytest.mark.parametrize("T,fmt,kw", [(3, "nvfp4", GROUPS), (8, "mxfp4", {}), (40, "nvfp4", GROUPS), (40, "mxfp4", {}),
                                      (70, "nvfp4", dict(fused_finalize=True))])
def test_other_batches_between_replays(B, T, fmt, kw):
    """The graph's buffers are its own: no other tensor gets their memory, and the results stay those of an eager layer."""
    gu, d = weights(16, 256, 256)
    layer = B.MoELayer(gu, d, 2, few_tokens=8, autotune=False, fmt=fmt, **kw)
    eager = B.MoELayer(gu, d, 2, few_tokens=8, autotune=False, fmt=fmt, **kw)
    x, logits = batch(T, 256, 16, seed=1)
    graph = layer.capture(x, logits)
    assert graph.out is layer.out
    taken = []
    for i, other in enumerate((5, 64, 1, 20, T)):
        layer(*batch(other, 256, 16, seed=other))
        gc.collect()
        # what was freed goes to these
        taken += [torch.full((n,), 37, dtype=torch.uint8, device="cuda") for n in (512, 2048, 8192, 65536, 1 << 20) for _ in range(8)]
        nx, nl = batch(T, 256, 16, seed=10 + i)
        x.copy_(nx), logits.copy_(nl)
        want = eager(nx, nl).clone()
        graph.replay()
        got = graph.out.clone()
        if kw.get("fused_finalize"):           # the order of its atomics is free: one step of bf16
            assert ((got.float() - want.float()).abs() <= 2.0 ** -7 * want.float().abs() + 1e-6).all()
        else:
            assert torch.equal(got, want)
        assert all(bool((t == 37).all()) for t in taken)
    B.sync_status()


def test_the_graph_keeps_its_layer_and_inputs(B):
    gu, d = weights(16, 256, 256)
    layer = B.MoELayer(gu, d, 2, few_tokens=8, autotune=False)
    x, logits = batch(4, 256, 16, seed=1)
    want = layer(x, logits).clone()
    graph = layer.capture(x, logits)
    del layer, x, logits, gu, d
    gc.collect()
    taken = [torch.full((n,), 37, dtype=torch.uint8, device="cuda") for n in (512, 2048, 8192, 1 << 20) for _ in range(8)]
    graph.out.zero_()
    graph.replay()
    assert torch.equal(graph.out, want) and all(bool((t == 37).all()) for t in taken)
    B.sync_status()
