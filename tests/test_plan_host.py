"""mla_plan's refusals of arrays that share memory, without a GPU."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def M():
    from nvfp4_block_scaled_07_gb300 import build
    build.build()
    from nvfp4_block_scaled_07_gb300 import mla
    return mla


def call(M, **change):
    """The status of a call whose arrays, of 4 requests, 16 rows and tables of [4, 8], lie 4096 bytes apart (never followed)."""
    at = {n: 4096 * (i + 1) for i, n in enumerate(("past", "new", "tables", "free", "count", "positions", "slots", "cu", "lens",
                                                   "granted", "count_out"))}
    stride = change.pop("stride", 8)
    for name, where in change.items():
        at[name] = at[where] if isinstance(where, str) else at[where[0]] + where[1]
    p = {n: ctypes.c_void_p(a) for n, a in at.items()}
    return M._lib.mla_plan(p["past"], p["new"], 4, 64, p["tables"], stride, 8, p["free"], 8, p["count"], 16, p["positions"],
                           p["slots"], p["cu"], p["lens"], p["granted"], p["count_out"], None)


@pytest.mark.parametrize("change,allowed", [
    (dict(), True), (dict(lens="past"), True), (dict(granted="new"), True), (dict(count_out="count"), True),
    (dict(lens="past", granted="new", count_out="count"), True),
    (dict(lens=("past", 4)), False), (dict(lens=("past", 12)), False), (dict(lens=("past", 16)), True), (dict(lens=("past", -16)), True),
    (dict(lens="new"), False), (dict(granted="past"), False), (dict(granted="lens"), False), (dict(cu="lens"), False),
    (dict(cu="past"), False), (dict(cu=("past", 16)), True), (dict(lens=("cu", 16)), False), (dict(lens=("cu", 20)), True),
    (dict(positions="slots"), False), (dict(positions=("slots", 128)), True), (dict(positions=("slots", 124)), False),
    (dict(positions="free"), False), (dict(count_out=("free", 28)), False), (dict(count_out=("free", 32)), True),
    (dict(count_out="lens"), False), (dict(slots="tables"), False), (dict(slots=("tables", 128)), True),
    (dict(lens=("tables", 124)), False), (dict(free="tables"), False), (dict(past=("tables", 64)), False),
    (dict(lens=("tables", -12)), False), (dict(lens=("tables", -16)), True),
    # rows of 32 bytes, 48 apart: 16 bytes between them are not the table's
    (dict(stride=12, lens=("tables", 32)), True), (dict(stride=12, lens=("tables", 28)), False),
    (dict(stride=12, lens=("tables", 36)), False), (dict(stride=12, lens=("tables", 80)), True),
    (dict(stride=12, lens=("tables", 144)), False), (dict(stride=12, lens=("tables", 176)), True),
    (dict(stride=12, slots=("tables", 32)), False)])
def test_arrays_that_share_memory(M, change, allowed):
    if torch.cuda.is_available():
        pytest.skip("dummy pointers: only without a GPU")
    status = call(M, **change)
    assert (status != 1) == allowed, M._lib.nvfp4moe_last_error_detail()
