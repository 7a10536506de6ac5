"""Host side of the latent-attention calls: the ABI of include/nvfp4mla.h and every refusal, without a GPU."""
import ctypes
import os
import random
import re
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "nvfp4mla.h")


@pytest.fixture(scope="session")
def M():
    from nvfp4_block_scaled_07_gb300 import build
    build.build()
    from nvfp4_block_scaled_07_gb300 import mla
    return mla


def declarations():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    text = re.sub(r"^\s*#.*$", "", text, flags=re.M)
    kinds = {"int": ctypes.c_int, "int64_t": ctypes.c_int64, "size_t": ctypes.c_size_t, "float": ctypes.c_float}

    def kind(decl):
        if "*" in decl or "cudaStream_t" in decl:
            return ctypes.c_void_p
        return kinds[decl.split()[0]]

    return {m.group(2): (kinds[m.group(1)], [kind(a.strip()) for a in m.group(3).split(",") if a.strip() != "void"])
            for m in re.finditer(r"\b(int|size_t)\s+(mla_\w+)\s*\(([^;]*?)\)\s*;", text, flags=re.S)}


def test_binding_signatures_match_the_header(M):
    assert declarations() == {k: (r, list(a)) for k, (r, a) in M._SIGS.items()}


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


APPEND = dict(latent=D, latent_stride=576, k_rope=D, k_rope_stride=576, norm_weight=D, eps=1e-6, positions=D, slots=D,
              T=4, table=D, max_positions=8, interleaved=1, dtype=0, cache=D, num_slots=64, rows_out=None, q=D,
              q_tok=192, q_head=192, H=2, q_out=D, qo_tok=128, qo_head=64, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), 1), (dict(H=-1), 2), (dict(H=1025), 2), (dict(dtype=2), 1), (dict(interleaved=2), 1),
    (dict(num_slots=-1), 1), (dict(max_positions=0), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(latent=None), 1), (dict(k_rope=None), 1), (dict(positions=None), 1), (dict(slots=None), 1),
    (dict(table=None), 1), (dict(cache=None), 1), (dict(q=None), 1), (dict(q_out=None), 1),
    (dict(latent=P(4104)), 1), (dict(latent_stride=577), 1), (dict(k_rope=P(4100)), 1), (dict(k_rope_stride=-8), 1),
    (dict(q_tok=4), 1), (dict(q_head=65), 1), (dict(qo_tok=1), 1), (dict(qo_head=2), 1), (dict(norm_weight=P(2)), 1),
    (dict(rows_out=P(8)), 1), (dict(slots=P(4100)), 1), (dict(positions=P(2)), 1), (dict(table=P(4100)), 1),
    (dict(T=1 << 30, H=1024), 2), (dict(T=0, latent=None, cache=None), 0)])
def test_append_refusals(M, change, code):
    _no_device()
    assert status(M._lib.mla_append, APPEND, **change) == code


@pytest.mark.parametrize("T,H,fits", [(1 << 27, 1024, True), (1 << 30, 16, True), (1 << 30, 224, True),
                                      (264305000, 1024, True), (264306000, 1024, False), (1 << 30, 240, False)])
def test_append_takes_what_its_grid_takes(M, T, H, fits):
    """8 units a block, a unit is a token's row or 16 of its heads, 2^31 - 1 blocks: what fits is not refused for its size
    (and then ends here for want of a device)."""
    _no_device()
    assert fits == (T * (1 + -(-H // 16)) <= 8 * (2 ** 31 - 1))
    assert (status(M._lib.mla_append, APPEND, T=T, H=H) != 2) == fits


@pytest.mark.parametrize("change,code", [
    (dict(qo_head=0), 1), (dict(qo_tok=0), 1), (dict(qo_head=56), 1), (dict(qo_tok=120), 1), (dict(qo_tok=64), 1),
    (dict(qo_tok=64, qo_head=248), 1), (dict(qo_tok=0, qo_head=0, T=1), 1), (dict(qo_tok=0, qo_head=64, T=1), 0),
    (dict(qo_tok=64, qo_head=0, H=1), 0), (dict(qo_tok=64, qo_head=256), 0), (dict(q_tok=0), 0), (dict(q_head=0), 0)])
def test_append_refuses_query_rows_that_overlap(M, change, code):
    """Outputs that overlap would be written by several threads at once; inputs may be broadcast (and then the call ends
    here for want of a device)."""
    _no_device()
    got = status(M._lib.mla_append, APPEND, **change)
    assert got == 1 if code else got not in (0, 1, 2)


DECODE = dict(q=D, cache=D, num_pages=8, page=64, tables=D, stride=4, max_pages=4, lens=D, B=2, Sq=1, H=16, scale=0.1,
              dtype=0, out=D, lse=D, ws=D, ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(B=-1), 1), (dict(Sq=0), 1), (dict(H=0), 1), (dict(max_pages=-1), 1), (dict(B=1 << 16, H=1 << 15), 2),
    (dict(dtype=-1), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(page=8), 2), (dict(page=48), 2), (dict(num_pages=0), 2),
    (dict(num_pages=1 << 27), 2), (dict(stride=3), 1), (dict(q=None), 1), (dict(cache=None), 1),
    (dict(tables=None), 1), (dict(lens=None), 1), (dict(out=None), 1), (dict(lse=None), 1), (dict(q=P(4104)), 1),
    (dict(cache=P(4104)), 1), (dict(out=P(4104)), 1), (dict(lse=P(4098)), 1), (dict(ws=None), 4),
    (dict(ws_bytes=64), 4), (dict(ws=P(4112)), 4), (dict(B=0, q=None, out=None), 0)])
def test_decode_refusals(M, change, code):
    _no_device()
    assert status(M._lib.mla_decode, DECODE, **change) == code


PREFILL = dict(q=D, q_tok=384, q_head=192, kn=D, kn_tok=512, kn_head=256, kr=D, kr_tok=64, v=D, v_tok=512, v_head=256,
               cu_q=D, cu_k=D, B=2, Tq=100, Tk=100, H=2, scale=0.1, causal=1, dtype=0, out=D, lse=D, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(B=-1), 1), (dict(Tq=-1), 1), (dict(Tk=-1), 1), (dict(H=-2), 1), (dict(Tq=1 << 30, H=2), 2),
    (dict(Tk=1 << 30, H=2), 2), (dict(B=1 << 30, H=2), 2), (dict(dtype=2), 1), (dict(causal=2), 1), (dict(scale=0.0), 1),
    (dict(scale=float("nan")), 1), (dict(q=None), 1), (dict(kn=None), 1), (dict(kr=None), 1), (dict(v=None), 1),
    (dict(cu_q=None), 1), (dict(cu_k=None), 1), (dict(out=None), 1), (dict(lse=None), 1), (dict(q_tok=0), 1),
    (dict(q_head=196), 1), (dict(kn_tok=-8), 1), (dict(kn_head=4), 1), (dict(kr_tok=0), 1), (dict(v_tok=1 << 38), 1),
    (dict(v_head=1), 1), (dict(q=P(4104)), 1), (dict(kn=P(4104)), 1), (dict(kr=P(4104)), 1), (dict(v=P(4104)), 1),
    (dict(out=P(4104)), 1), (dict(lse=P(4098)), 1), (dict(cu_q=P(4098)), 1), (dict(B=0, q=None), 0),
    (dict(Tq=0, out=None), 0), (dict(H=0, lse=None), 0)])
def test_prefill_refusals(M, change, code):
    _no_device()
    assert status(M._lib.mla_prefill, PREFILL, **change) == code


def test_python_checks_come_before_the_call(M):
    """Types and shapes are refused with the argument's name, and CPU tensors are not taken."""
    bf, f32, i32, i64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
    z = torch.zeros
    with pytest.raises(TypeError, match="latent"):
        M.mla_append(z(4, 512), z(4, 64), z(4, dtype=i32), z(4, dtype=i64), z(8, 64), z(1, 16, 576))
    with pytest.raises(ValueError, match="latent"):
        M.mla_append(z(4, 500, dtype=bf), z(4, 64, dtype=bf), z(4, dtype=i32), z(4, dtype=i64), z(8, 64),
                     z(1, 16, 576, dtype=bf))
    with pytest.raises(ValueError, match="CUDA"):
        M.mla_append(z(4, 512, dtype=bf), z(4, 64, dtype=bf), z(4, dtype=i32), z(4, dtype=i64), z(8, 64),
                     z(1, 16, 576, dtype=bf))
    with pytest.raises(TypeError, match="q"):
        M.mla_decode(z(1, 1, 16, 576), z(1, 16, 576, dtype=bf), z(1, 1, dtype=i32), z(1, dtype=i32), 0.1)
    with pytest.raises(ValueError, match="q"):
        M.mla_decode(z(1, 1, 16, 512, dtype=bf), z(1, 16, 576, dtype=bf), z(1, 1, dtype=i32), z(1, dtype=i32), 0.1)
    assert f32 == M.rope_table(3, device="cpu").dtype


def test_rope_table_is_the_rounded_64_bit_angle(M):
    import math
    t = M.rope_table(100001, base=10000.0, device="cpu")
    for p in (0, 1, 77777, 100000):
        for i in (0, 1, 17, 31):
            a = p * 10000.0 ** (-i / 32)
            assert abs(float(t[p, i]) - math.cos(a)) < 2e-7 and abs(float(t[p, 32 + i]) - math.sin(a)) < 2e-7


JOIN = r"""
#include <cstdio>
#include <vector>
#include "mla_join.h"
// stdin: cases of "ranges min_share items tiles...": prints how often each item is joined
int main() {
  int ranges, least, n;
  while (std::scanf("%d %d %d", &ranges, &least, &n) == 3) {
    std::vector<int> tiles(n), start(n), joined(n, 0);
    int total = 0;
    for (int i = 0; i < n; ++i) {
      if (std::scanf("%d", &tiles[i]) != 1) return 1;
      start[i] = total;
      total += tiles[i];
    }
    int share = (total + ranges - 1) / ranges;
    if (share < least) share = least;
    for (int c = 0; c + 1 < ranges; ++c) {      // block c looks at the item that range c + 1 begins with
      const long long pos = (long long)share * (c + 1);
      int at = 0, k = 0, i = 0;
      if (pos < total) {
        while (start[i] + tiles[i] <= pos) ++i;
        at = start[i], k = tiles[i];
      }
      if (nvfp4moe::border_joins(c, at, k, share)) ++joined[i];
    }
    for (int i = 0; i < n; ++i) std::printf("%d ", joined[i]);
    std::printf("\n");
  }
}
"""


def test_every_cut_item_is_joined_once(tmp_path):
    """Items of random sizes, and of sizes that begin and end at the borders of ranges."""
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    (tmp_path / "join.cpp").write_text(JOIN)
    csrc = os.path.join(ROOT, "nvfp4_block_scaled_07_gb300", "csrc")
    subprocess.run([cxx, "-O1", "-I", csrc, str(tmp_path / "join.cpp"), "-o", str(tmp_path / "join")], check=True)
    rng = random.Random(1)
    cases = [(152, 2, [4] * 76), (76, 2, [4] * 38), (10, 2, [6] * 4), (10, 2, [20]), (3, 2, [1]), (152, 2, [1] * 1000)]
    for _ in range(400):
        top = rng.choice([1, 2, 5, 40, 300])
        cases.append((rng.randint(1, 160), 2, [rng.randint(1, top) for _ in range(rng.randint(1, 60))]))
    text = "".join(f"{r} {m} {len(t)} {' '.join(map(str, t))}\n" for r, m, t in cases)
    got = subprocess.run([str(tmp_path / "join")], input=text, capture_output=True, text=True, check=True).stdout.splitlines()
    assert len(got) == len(cases)
    for (ranges, least, tiles), line in zip(cases, got):
        share, at, want = max(-(-sum(tiles) // ranges), least), 0, []
        for t in tiles:
            want.append(int(at // share != (at + t - 1) // share))
            at += t
        assert [int(v) for v in line.split()] == want, (ranges, tiles)
