"""Host side of the few-token calls and the page plan: the ABI of include/nvfp4few.h and every refusal, without a GPU."""
import ctypes
import os
import re

import pytest
import torch

from . import few_reference as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "nvfp4few.h")


@pytest.fixture(scope="session")
def B():
    from nvfp4_block_scaled_07_gb300 import build
    build.build()
    from nvfp4_block_scaled_07_gb300 import binding
    return binding


@pytest.fixture(scope="session")
def M(B):
    from nvfp4_block_scaled_07_gb300 import mla
    return mla


def declarations():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    text = re.sub(r"^\s*#.*$", "", text, flags=re.M)
    kinds = {"int": ctypes.c_int, "int64_t": ctypes.c_int64, "size_t": ctypes.c_size_t, "float": ctypes.c_float}

    def kind(decl):
        return ctypes.c_void_p if "*" in decl or "cudaStream_t" in decl else kinds[decl.split()[0]]

    return {m.group(2): (kinds[m.group(1)], [kind(a.strip()) for a in m.group(3).split(",")])
            for m in re.finditer(r"\b(int|size_t)\s+(moe_\w+)\s*\(([^;]*?)\)\s*;", text, flags=re.S)}


def test_binding_signatures_match_the_header(B):
    assert declarations() == {k: (r, list(a)) for k, (r, a) in B._FEW_SIGS.items()}


def _no_device():
    if torch.cuda.is_available():
        pytest.skip("host-validation cases with dummy pointers run only without a GPU")


P = ctypes.c_void_p
D = P(4096)            # never followed: each call is refused before any device work


def status(fn, args, **change):
    a = dict(args)
    for k, v in change.items():
        assert k in a, k
        a[k] = v
    return fn(*a.values())


ROUTE = dict(logits=D, bias=D, T=4, E=64, k=8, n_group=8, topk_group=4, best=2, score=1, renorm=1, scale=1.0, idx=D, w=D,
             stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), 1), (dict(E=0), 2), (dict(E=1025), 2), (dict(k=0), 2), (dict(k=65), 2), (dict(k=33), 2), (dict(n_group=0), 2),
    (dict(n_group=7), 2), (dict(n_group=64), 2), (dict(topk_group=0), 1), (dict(topk_group=9), 1),
    (dict(topk_group=1, k=9), 1), (dict(best=0), 1), (dict(best=3), 1), (dict(E=8, k=2, n_group=8, best=2), 1),
    (dict(score=2), 1), (dict(scale=float("inf")), 1), (dict(scale=float("nan")), 1), (dict(logits=None), 1),
    (dict(idx=None), 1), (dict(w=None), 1), (dict(logits=P(4098)), 1), (dict(bias=P(4097)), 1), (dict(T=0, logits=None), 0)])
def test_route_refusals(B, change, code):
    _no_device()
    assert status(B._lib.moe_route_grouped, ROUTE, **change) == code


MATVEC = dict(x=D, stride=512, T=4, dtype=0, packed=D, scales=D, gscale=D, N=256, K=512, layout=0, out=D, ws=D,
              ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), 1), (dict(T=33), 2), (dict(dtype=2), 1), (dict(layout=2), 1), (dict(K=0), 2), (dict(K=96), 2),
    (dict(N=0), 2), (dict(N=192), 2), (dict(packed=None), 1), (dict(scales=None), 1), (dict(gscale=None), 1),
    (dict(packed=P(4104)), 1), (dict(scales=P(4104)), 1), (dict(gscale=P(4098)), 1), (dict(x=None), 1), (dict(out=None), 1),
    (dict(x=P(4104)), 1), (dict(out=P(4104)), 1), (dict(stride=-8), 1), (dict(stride=516), 1), (dict(T=0, x=None), 0),
    (dict(T=32, K=1 << 14, ws=None), 4), (dict(T=32, K=1 << 14, ws_bytes=64), 4), (dict(T=32, K=1 << 14, ws=P(4112)), 4)])
def test_matvec_refusals(B, change, code):
    _no_device()
    assert status(B._lib.moe_matvec_nvfp4, MATVEC, **change) == code
    if "gscale" not in change:
        mx = {k: v for k, v in MATVEC.items() if k != "gscale"}
        assert status(B._lib.moe_matvec_mxfp4, mx, **change) == code
    if change == dict(K=96):
        assert status(B._lib.moe_matvec_mxfp4, mx, K=192) == 2


EXPERTS = dict(x=D, stride=512, idx=D, w=D, T=4, k=2, E=8, H=512, I=256, gu=D, gu_s=D, gu_g=D, d=D, d_s=D, d_g=D, layout=1,
               out=D, ws=D, ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), 1), (dict(T=33), 2), (dict(E=0), 2), (dict(E=1025), 2), (dict(k=0), 2), (dict(k=33), 2), (dict(H=0), 2),
    (dict(H=192), 2), (dict(H=100), 2), (dict(I=0), 2), (dict(I=192), 2), (dict(I=1 << 30), 2), (dict(layout=-1), 1),
    (dict(gu=None), 1), (dict(gu_s=None), 1), (dict(gu_g=None), 1), (dict(d=None), 1), (dict(d_s=None), 1),
    (dict(d_g=None), 1), (dict(gu=P(4104)), 1), (dict(d_s=P(4104)), 1), (dict(x=None), 1), (dict(idx=None), 1),
    (dict(w=None), 1), (dict(out=None), 1), (dict(x=P(4104)), 1), (dict(idx=P(4098)), 1), (dict(stride=12), 1),
    (dict(ws=None), 4), (dict(ws_bytes=1024), 4), (dict(ws=P(4112)), 4), (dict(T=0, x=None, ws=None), 0)])
def test_experts_refusals(B, change, code):
    _no_device()
    assert status(B._lib.moe_experts_nvfp4, EXPERTS, **change) == code
    if not {"gu_g", "d_g"} & set(change):
        mx = {k: v for k, v in EXPERTS.items() if k not in ("gu_g", "d_g")}
        assert status(B._lib.moe_experts_mxfp4, mx, **change) == code


PLAN = dict(past=D, new=D, B=4, page=64, tables=D, stride=8, max_pages=8, free=D, num_free=8, count=D, T=16, positions=D,
            slots=D, cu=D, lens=D, granted=D, count_out=D, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(B=-1), 1), (dict(T=-1), 1), (dict(max_pages=-1), 1), (dict(num_free=-1), 1), (dict(page=8), 2), (dict(page=48), 2),
    (dict(page=0), 2), (dict(stride=7), 1), (dict(past=None), 1), (dict(new=None), 1), (dict(tables=None), 1),
    (dict(free=None), 1), (dict(count=None), 1), (dict(positions=None), 1), (dict(slots=None), 1), (dict(cu=None), 1),
    (dict(lens=None), 1), (dict(granted=None), 1), (dict(count_out=None), 1), (dict(slots=P(4100)), 1),
    (dict(past=P(4098)), 1), (dict(tables=P(4097)), 1)])
def test_plan_refusals(M, change, code):
    _no_device()
    assert status(M._lib.mla_plan, PLAN, **change) == code


def test_python_checks_come_before_the_call(B, M):
    bf, i32, z = torch.bfloat16, torch.int32, torch.zeros
    with pytest.raises(TypeError, match="logits"):
        B.moe_route_grouped(z(4, 8, dtype=bf), 2)
    with pytest.raises(ValueError, match="CUDA"):
        B.moe_route_grouped(z(4, 8), 2)
    with pytest.raises(TypeError, match="x"):
        B.moe_matvec_nvfp4(z(4, 128), z(128, 64, dtype=torch.uint8), z(1024, dtype=torch.uint8), z(1))
    with pytest.raises(ValueError, match="CUDA"):
        B.moe_matvec_mxfp4(z(4, 128, dtype=bf), z(128, 64, dtype=torch.uint8), z(512, dtype=torch.uint8))
    with pytest.raises(TypeError, match="x"):
        B.moe_experts_mxfp4(z(4, 128, dtype=torch.float16), z(4, 2, dtype=i32), z(4, 2), *[z(1, dtype=torch.uint8)] * 4)
    with pytest.raises(ValueError, match="CUDA"):
        M.mla_plan(z(1, dtype=i32), z(1, dtype=i32), z(1, 1, dtype=i32), z(1, dtype=i32), z(1, dtype=i32), 16, 4)


def test_workspace_sizes(B):
    assert B.moe_matvec_workspace_size(1, 128, 1024) == 0 and B.moe_matvec_workspace_size(33, 128, 1024) == 0
    assert B.moe_matvec_workspace_size(32, 128, 8192) >= 32 * 8192 * 2
    assert B.moe_experts_workspace_size(1, 8, 6144, 2048) >= 8 * 2048 * 4
    assert B.moe_experts_workspace_size(32, 33, 6144, 2048) == 0


def test_reference_plan_by_hand():
    tables = [[5, -1, -1], [-1, -1, -1], [7, 8, -1]]
    got = R.plan([10, 0, 32], [8, 17, 1], tables, [1, 2, 3, 4], 3, 16, 28)
    assert tables == [[5, 3, -1], [2, 1, -1], [7, 8, -1]]      # one, two and then none left
    assert got["granted"] == [8, 17, 0] and got["seq_lens"] == [18, 17, 32] and got["cu_seqlens"] == [0, 8, 25, 26]
    assert got["slots"][:8] == [5 * 16 + 10 + i for i in range(6)] + [3 * 16, 3 * 16 + 1]
    assert got["slots"][24:] == [16, -1, -1, -1] and got["positions"][24:] == [16, 32, 0, 0] and got["free_count"] == [0]


def test_reference_route_by_hand():
    v = torch.tensor([0.0, 1.0, 2.0, 3.0, -1.0, 2.5, 2.5, 0.5])
    assert R.route(v, None, 3, "sigmoid", True, 1, 1, 2, 1.0)[0] == [3, 5, 6]
    # groups of two: sums of sigmoids 1.23, 1.83, 1.19, 1.55 -> groups 1 and 3
    assert R.route(v, None, 3, "sigmoid", True, 4, 2, 2, 1.0)[0] == [3, 6, 2]
    idx, w = R.route(v, torch.tensor([9.0] + [0.0] * 7), 2, "softmax", False, 1, 1, 1, 2.0)
    assert idx == [0, 3] and abs(w[1] / w[0] - float(torch.exp(torch.tensor(3.0)))) < 1e-5
