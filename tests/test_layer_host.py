"""MoELayer on the host: what it keeps and what it refuses, without a GPU (the kernels are left out)."""
import gc
import weakref

import pytest
import torch


@pytest.fixture(scope="module")
def B():
    from nvfp4_block_scaled_07_gb300 import build
    build.build()
    from nvfp4_block_scaled_07_gb300 import binding
    return binding


@pytest.fixture
def layer(B, monkeypatch):
    """A layer whose weights are placeholders and whose kernels do nothing; .capturing says what the stream does."""
    state = {"capturing": False}
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state["capturing"])
    nothing = torch.zeros(1, dtype=torch.uint8)
    monkeypatch.setattr(B, "quantize_expert_weights", lambda w: (nothing, nothing, nothing))
    for name in ("moe_prepare", "moe_grouped_gemm_nvfp4", "moe_route_grouped", "moe_finalize", "moe_route_topk"):
        monkeypatch.setattr(B, name, lambda *a, **kw: kw.get("out"))
    monkeypatch.setattr(B, "moe_experts_nvfp4", lambda *a, **kw: kw["out"])

    def make(**kw):
        args = dict(few_tokens=8, autotune=False, tiled_weights=False, dynamic_schedule=False) | kw
        made = B.MoELayer(torch.zeros(8, 256, 256, dtype=torch.bfloat16), torch.zeros(8, 256, 128, dtype=torch.bfloat16), 2,
                          **args)
        made.state = state
        return made

    return make


def step(layer, T):
    return layer(torch.zeros(T, 256, dtype=torch.bfloat16), torch.zeros(T, 8))


def refs(layer):
    return {n: weakref.ref(t) for n, t in layer._buffers().items() if isinstance(t, torch.Tensor)}


@pytest.mark.parametrize("T", [4, 40])
def test_captured_buffers_outlive_other_batches(layer, T):
    """What a forward() inside a capture of the caller's used stays allocated; what none used does not pile up."""
    moe = layer()
    step(moe, T)
    moe.state["capturing"] = True
    step(moe, T)
    moe.state["capturing"] = False
    held = refs(moe)
    for other in (T + 1, 20, T, 20):
        step(moe, other)
    gc.collect()
    assert held and all(r() is not None for r in held.values())
    assert len(moe._kept) == 1
    last = refs(moe)
    step(moe, 21)
    gc.collect()
    assert last["out"]() is None
    del moe
    gc.collect()
    assert all(r() is None for r in held.values())


def test_captured_steps_outlive_other_batches(layer):
    """The steps of forward() captured one by one."""
    moe = layer()
    step(moe, 40)
    moe.state["capturing"] = True
    moe.gemm_gate_up()
    moe.state["capturing"] = False
    held = refs(moe)
    step(moe, 3)
    gc.collect()
    assert all(r() is not None for r in held.values())


@pytest.mark.parametrize("kw", [
    dict(topk_group=2), dict(topk_group=0), dict(group_best=3), dict(group_best=0), dict(n_group=4, topk_group=5),
    dict(n_group=3), dict(n_group=8), dict(n_group=16, group_best=1), dict(n_group=8, topk_group=1, group_best=1),
    dict(n_group=4, topk_group=0)])
def test_groups_that_do_not_fit_are_refused(layer, kw):
    """At construction: without groups too, where they would be passed over in silence."""
    with pytest.raises(ValueError, match="group"):
        layer(**kw)


@pytest.mark.parametrize("kw", [dict(), dict(group_best=1), dict(n_group=4), dict(n_group=8, topk_group=2, group_best=1),
                                dict(n_group=2, topk_group=2), dict(n_group=1, topk_group=1, routed_scale=2.0)])
def test_groups_that_fit(layer, kw):
    assert layer(**kw).few_tokens == 8
