"""Latent attention against 64-bit references: cache append, absorbed decode, expanded prefill.

The shapes are those where such kernels go wrong: lengths of 0, 1 and around a
tile, pages that end inside a tile, row blocks that are not full, rows that
see nothing, non-finite values wherever nothing may be read, ranges that cut
a sequence, maxima that grow from tile to tile."""
import math
import random

import pytest
import torch

from tests import mla_reference as R

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5
BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def M():
    from nvfp4_block_scaled_07_gb300 import build
    build.build()
    from nvfp4_block_scaled_07_gb300 import binding, mla
    binding.device_check()
    binding.sync_status()
    return mla


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, dtype=BF16, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


# ---- append --------------------------------------------------------------------------------------------------
def append_case(M, T, H, dtype, interleaved, norm, page, seed, span=5000):
    g = gen(seed)
    n_pages = -(-T // page) + 2
    kv, qp = normal(g, T, 576, dtype=dtype, std=3.0), normal(g, T, H, 192, dtype=dtype)
    w = normal(g, 512, dtype=dtype) if norm else None
    pos = torch.randint(0, span, (T,), generator=g, device="cuda", dtype=torch.int32)
    slots = torch.randperm(n_pages * page, generator=g, device="cuda")[:T]
    slots[1::5] = -1
    table = M.rope_table(span)
    cache = normal(g, n_pages, page, 576, dtype=dtype)
    return dict(kv=kv, qp=qp, w=w, pos=pos, slots=slots, table=table, cache=cache, interleaved=interleaved)


def append_reference(c, eps=1e-6):
    x = c["kv"].double()
    lat = x[:, :512]
    if c["w"] is not None:
        lat = lat / torch.sqrt(lat.square().mean(1, keepdim=True) + eps) * c["w"].double()
    cs = c["table"].double()[c["pos"].long()]
    rows = torch.cat([lat, R.rotate(x[:, 512:], cs[:, :32], cs[:, 32:], c["interleaved"])], 1)
    q = R.rotate(c["qp"].double()[..., 128:], cs[:, None, :32], cs[:, None, 32:], c["interleaved"])
    return rows, q


def append_close(got, ref, size, dtype, what):
    # one rounding; float32 steps before it (square sum of 512, root, two products): 2^-18 of the terms
    tol = R.half_step(dtype) * ref.abs() + 2.0 ** -18 * size + (2.0 ** -25 if dtype == FP16 else 1e-38)
    assert bool(((got.double() - ref).abs() <= tol).all()), what


@pytest.mark.parametrize("T,H,dtype,interleaved,norm,page", [
    (1, 1, BF16, True, True, 16), (1, 0, BF16, False, False, 16), (2, 3, FP16, True, False, 32),
    (33, 8, BF16, False, True, 64), (128, 64, FP16, False, True, 128), (257, 9, BF16, True, True, 16),
    (1000, 17, BF16, False, False, 64), (4099, 16, FP16, True, True, 64)])
def test_append_matches_reference(M, T, H, dtype, interleaved, norm, page):
    c = append_case(M, T, H, dtype, interleaved, norm, page, seed=T + H)
    rows, q = append_reference(c)
    before = c["cache"].clone()
    buf = torch.full((T, H, 576), 7.0, dtype=dtype, device="cuda")
    out_rows = torch.empty((T, 576), dtype=dtype, device="cuda")
    r = M.mla_append(c["kv"][:, :512], c["kv"][:, 512:], c["pos"], c["slots"], c["table"], c["cache"],
                     norm_weight=c["w"], interleaved=interleaved, q_rope=c["qp"][..., 128:] if H else None,
                     q_out=buf[..., 512:] if H else None, rows_out=out_rows)
    M.sync_status()
    size = torch.cat([rows[:, :512].abs(), c["kv"].double()[:, 512:].abs().amax(1, keepdim=True).expand(-1, 64) * 2], 1)
    append_close(out_rows, rows, size, dtype, "rows")
    if H:
        append_close(buf[..., 512:], q, c["qp"].double().abs().amax() * 2, dtype, "queries")
        assert r.data_ptr() == buf[..., 512:].data_ptr() and bool((buf[..., :512] == 7.0).all())
    # the cache: the written rows bit for bit, every other slot as it was
    flat, old = c["cache"].view(-1, 576), before.view(-1, 576)
    kept = c["slots"] >= 0
    assert torch.equal(flat[c["slots"][kept]], out_rows[kept])
    other = torch.ones(flat.shape[0], dtype=torch.bool, device="cuda")
    other[c["slots"][kept]] = False
    assert torch.equal(flat[other], old[other])


def test_append_in_place_queries_and_no_copy(M):
    c = append_case(M, 65, 5, BF16, True, True, 64, seed=5)
    _, q = append_reference(c)
    first = M.mla_append(c["kv"][:, :512], c["kv"][:, 512:], c["pos"], c["slots"], c["table"], c["cache"],
                         norm_weight=c["w"], q_rope=c["qp"][..., 128:])
    nope = c["qp"][..., :128].clone()
    M.mla_append(c["kv"][:, :512], c["kv"][:, 512:], c["pos"], c["slots"], c["table"], c["cache"],
                 norm_weight=c["w"], q_rope=c["qp"][..., 128:], q_out=c["qp"][..., 128:])
    M.sync_status()
    assert torch.equal(first, c["qp"][..., 128:]) and torch.equal(nope, c["qp"][..., :128])
    append_close(first, q, q.abs().amax() * 2, BF16, "queries")


def test_append_far_position_and_far_slot(M):
    """The last row of a cache whose byte offsets pass 32 bits, at the last position of a long table."""
    page, n_pages = 64, 65536                              # 4.8 GB
    cache = torch.zeros(n_pages, page, 576, dtype=BF16, device="cuda")
    span = 1 << 20
    c = append_case(M, 3, 2, BF16, True, True, 16, seed=6)
    c["pos"] = torch.tensor([0, span - 1, span // 2 + 1], device="cuda", dtype=torch.int32)
    c["slots"] = torch.tensor([n_pages * page - 1, 0, n_pages * page // 2 + 3], device="cuda")
    c["table"] = M.rope_table(span)
    rows, _ = append_reference(c)
    M.mla_append(c["kv"][:, :512], c["kv"][:, 512:], c["pos"], c["slots"], c["table"], cache, norm_weight=c["w"])
    M.sync_status()
    got = cache.view(-1, 576)[c["slots"]]
    append_close(got, rows, rows.abs().amax() * 2, BF16, "rows")
    assert int((cache.view(-1, 576)[:, 0] != 0).sum()) == 3


def test_append_skips_and_reports_bad_positions_and_slots(M):
    c = append_case(M, 8, 2, BF16, True, True, 16, seed=7)
    c["slots"] = torch.arange(8, device="cuda")
    n_slots = c["cache"].shape[0] * 16
    c["pos"][2] = 5000                                     # one past the table
    c["pos"][3] = -1
    c["slots"][5] = n_slots
    before = c["cache"].clone().view(-1, 576)
    rows_out = torch.full((8, 576), 3.0, dtype=BF16, device="cuda")
    q_out = torch.full((8, 2, 64), 3.0, dtype=BF16, device="cuda")
    M.mla_append(c["kv"][:, :512], c["kv"][:, 512:], c["pos"], c["slots"], c["table"], c["cache"],
                 norm_weight=c["w"], q_rope=c["qp"][..., 128:], q_out=q_out, rows_out=rows_out)
    with pytest.raises(M.Nvfp4MoeError) as e:
        M.sync_status()
    assert e.value.status == 7
    M.sync_status()
    after = c["cache"].view(-1, 576)
    assert torch.equal(after[[2, 3, 5]], before[[2, 3, 5]]) and not torch.equal(after[4], before[4])
    assert bool((rows_out[[2, 3]] == 3.0).all()) and bool((q_out[[2, 3]] == 3.0).all())
    assert torch.equal(rows_out[4], after[4]) and not bool((rows_out[5] == 3.0).all())


def test_append_empty_batch(M):
    cache = torch.zeros(1, 16, 576, dtype=BF16, device="cuda")
    e = torch.empty(0, 576, dtype=BF16, device="cuda")
    M.mla_append(e[:, :512], e[:, 512:], torch.empty(0, dtype=torch.int32, device="cuda"),
                 torch.empty(0, dtype=torch.int64, device="cuda"), M.rope_table(4), cache)
    M.sync_status()


# ---- decode --------------------------------------------------------------------------------------------------
def decode_case(B, Sq, H, lens, page, dtype, seed, q_std=1.0, spare=3):
    """Pages in random order; NaN in every cache row that no sequence owns, page ids of -1 and 2^30 past the ends."""
    g = gen(seed)
    need = [-(-n // page) for n in lens]
    total = sum(need) + spare
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    cache = normal(g, total, page, 576, dtype=dtype)
    width = max(max(need), 1) + 1
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    table[:, 1::2] = 1 << 30
    used = torch.zeros(total, page, dtype=torch.bool, device="cuda")
    at = 0
    for b, n in enumerate(lens):
        ids = order[at:at + need[b]]
        table[b, :need[b]] = ids
        at += need[b]
        for i, j in enumerate(ids.tolist()):
            used[j, :min(page, n - i * page)] = True
    cache[~used] = math.nan
    return dict(q=normal(g, B, Sq, H, 576, dtype=dtype, std=q_std), cache=cache, table=table,
                lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), lens_host=lens, page=page)


def decode_check(c, out, lse, scale=SCALE, what="", only=None):
    B, Sq, H, _ = c["q"].shape
    for b in (range(B) if only is None else only):
        n = c["lens_host"][b]
        ids = c["table"][b, :-(-n // c["page"])].long()
        kv = c["cache"][ids].reshape(-1, 576)[:n].double()
        sees = (n - Sq + 1 + torch.arange(Sq, device="cuda").repeat_interleave(H)).clamp(0)
        ref = R.attend(c["q"][b].double().reshape(Sq * H, 576), kv, kv[:, :512], scale, sees)
        R.check(out[b].reshape(Sq * H, 512), lse[b].reshape(-1), ref[0], ref[1], ref[2], ref[3], c["q"].dtype, n,
                f"{what} sequence {b} of {n}")


@pytest.mark.parametrize("B,Sq,H,lens,page,dtype", [
    (1, 1, 16, [1], 16, BF16), (1, 1, 16, [64], 64, BF16), (1, 1, 16, [37], 16, FP16), (1, 1, 64, [65], 16, BF16),
    (3, 1, 1, [0, 1, 63], 32, BF16), (2, 1, 7, [128, 129], 64, FP16), (4, 2, 16, [0, 1, 2, 200], 16, BF16),
    (3, 4, 16, [3, 64, 257], 32, BF16), (2, 3, 40, [500, 61], 128, FP16), (2, 1, 128, [300, 77], 64, BF16),
    (2, 1, 65, [190, 1000], 256, BF16), (1, 2, 96, [1500], 64, FP16), (1, 5, 200, [333], 16, BF16),
    (40, 1, 16, [17 * i for i in range(40)], 16, BF16), (70, 1, 8, [(37 * i) % 400 for i in range(70)], 64, FP16)])
def test_decode_matches_reference(M, B, Sq, H, lens, page, dtype):
    c = decode_case(B, Sq, H, lens, page, dtype, seed=B * 1000 + H)
    out, lse = M.mla_decode(c["q"], c["cache"], c["table"], c["lens"], SCALE)
    M.sync_status()
    decode_check(c, out, lse)


@pytest.mark.parametrize("B,Sq,H,lens,page", [
    (1, 1, 64, [20000], 64), (2, 2, 64, [9001, 30011], 32), (5, 1, 16, [12000, 1, 0, 7777, 65], 16),
    (150, 1, 64, [64 * (1 + i % 7) for i in range(150)], 64), (33, 1, 128, [701 + 13 * i for i in range(33)], 64)])
def test_decode_ranges_that_cut_sequences(M, B, Sq, H, lens, page):
    c = decode_case(B, Sq, H, lens, page, BF16, seed=B + H)
    ws = torch.full((M.mla_decode_workspace_size(),), 255, dtype=torch.uint8, device="cuda")   # NaN everywhere
    out, lse = M.mla_decode(c["q"], c["cache"], c["table"], c["lens"], SCALE, workspace=ws)
    again = M.mla_decode(c["q"], c["cache"], c["table"], c["lens"], SCALE, workspace=ws)
    M.sync_status()
    decode_check(c, out, lse)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])       # the same sums in the same order


@pytest.mark.parametrize("B,Sq,H,lens,page", [
    (8, 1, 64, [3000 - 211 * i for i in range(8)], 64), (20, 1, 16, [(397 * i) % 2100 for i in range(20)], 32),
    (1, 1, 5, [9001], 16), (9, 1, 33, [4000 if i % 4 == 0 else 64 * i for i in range(9)], 64),
    (1, 2, 60, [7003], 64), (3, 3, 50, [0, 6000, 129], 128)])
def test_decode_joins_of_few_sequences(M, B, Sq, H, lens, page):
    """Every way in which partial results are joined: by item with several warps a row, eight warps a quarter row."""
    c = decode_case(B, Sq, H, lens, page, FP16, seed=B + 7 * H)
    ws = torch.full((M.mla_decode_workspace_size(),), 255, dtype=torch.uint8, device="cuda")   # NaN everywhere
    out, lse = M.mla_decode(c["q"], c["cache"], c["table"], c["lens"], SCALE, workspace=ws)
    M.sync_status()
    decode_check(c, out, lse)


@pytest.mark.parametrize("Sq,H,dtype,top", [(1, 128, BF16, 128), (1, 96, FP16, 128), (2, 64, BF16, 128), (1, 128, BF16, 300)])
def test_decode_many_short_sequences_on_pairs(M, Sq, H, dtype, top):
    """Ranges of many items back to back, most of one tile: an item's sums are read before the next item's maxima
    take their place.  The same bits each time."""
    B = 1000
    c = decode_case(B, Sq, H, [(37 * i) % top + 1 for i in range(B)], 16, dtype, seed=H + top)
    # scores of very different sizes from one item to the next, so that a maximum taken for a sum would show
    c["q"] *= torch.linspace(0.1, 6.0, 7, device="cuda")[torch.arange(B, device="cuda") % 7].to(dtype)[:, None, None, None]
    out, lse = M.mla_decode(c["q"], c["cache"], c["table"], c["lens"], SCALE)
    decode_check(c, out, lse, only=range(0, B, 13))
    for _ in range(20):
        again = M.mla_decode(c["q"], c["cache"], c["table"], c["lens"], SCALE)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    M.sync_status()


@pytest.mark.parametrize("top", [30, 64, 100, 300])
def test_decode_pairs_whose_odd_cta_has_no_keys_to_copy(M, top):
    """Tiles of at most 64 (or 96) keys of 128: the odd CTA's warps copy nothing and still keep step with the even one's.
    Every call writes outputs that hold NaN, and is looked at on its own."""
    B, H = 3000, 80
    c = decode_case(B, 1, H, [(53 * i) % top + 1 for i in range(B)], 64, BF16, seed=top)
    out, lse = M.mla_decode(c["q"], c["cache"], c["table"], c["lens"], SCALE)
    M.sync_status()
    decode_check(c, out, lse, only=range(0, B, 101))
    got, got_lse = torch.empty_like(out), torch.empty_like(lse)
    for i in range(30):
        got.fill_(math.nan)
        got_lse.fill_(math.nan)
        M.mla_decode(c["q"], c["cache"], c["table"], c["lens"], SCALE, out=got, lse=got_lse)
        M.sync_status()
        assert torch.equal(got, out) and torch.equal(got_lse, lse), f"call {i}"


@pytest.mark.parametrize("B,H,n", [(76, 64, 256), (38, 128, 512), (76, 16, 250), (50, 48, 1200)])
def test_decode_items_that_begin_at_a_border(M, B, H, n):
    """Sequences of equal length whose tiles are a multiple of a range's (152 SMs), and others near it."""
    c = decode_case(B, 1, H, [n] * B, 64, BF16, seed=n + H)
    ws = torch.full((M.mla_decode_workspace_size(),), 255, dtype=torch.uint8, device="cuda")   # NaN everywhere
    out, lse = M.mla_decode(c["q"], c["cache"], c["table"], c["lens"], SCALE, workspace=ws)
    M.sync_status()
    decode_check(c, out, lse)


@pytest.mark.parametrize("B,Sq,H,top", [(6, 1, 128, 5000), (7, 1, 128, 5000), (12, 1, 80, 3000), (19, 2, 40, 2100), (3, 2, 128, 4000)])
def test_decode_joins_of_pairs(M, B, Sq, H, top):
    """Both ways in which the pairs' partial results are joined, on both sides of the rule between them."""
    c = decode_case(B, Sq, H, [max(0, top - 317 * i) for i in range(B)], 64, BF16, seed=B + H)
    ws = torch.full((M.mla_decode_workspace_size(),), 255, dtype=torch.uint8, device="cuda")   # NaN everywhere
    out, lse = M.mla_decode(c["q"], c["cache"], c["table"], c["lens"], SCALE, workspace=ws)
    M.sync_status()
    decode_check(c, out, lse)


def test_decode_random_shapes(M):
    rng = random.Random(3)
    for i in range(24):
        B, Sq, H = rng.choice([1, 2, 3, 9, 31, 33]), rng.choice([1, 1, 2, 3, 4]), rng.choice([1, 5, 16, 31, 64, 80, 128])
        top = rng.choice([3, 70, 500, 3001])
        lens = [rng.randint(0, top) for _ in range(B)]
        c = decode_case(B, Sq, H, lens, rng.choice([16, 32, 64, 128]), rng.choice([BF16, FP16]), seed=i)
        out, lse = M.mla_decode(c["q"], c["cache"], c["table"], c["lens"], SCALE)
        M.sync_status()
        decode_check(c, out, lse, what=f"draw {i}")


@pytest.mark.parametrize("order", ["rising", "falling", "spiky"])
def test_decode_scores_that_grow(M, order):
    """Scores of up to several hundred whose maximum moves from tile to tile (or sits in the first)."""
    n, H = 900, 48
    c = decode_case(1, 1, H, [n], 64, BF16, seed=11)
    ramp = torch.linspace(0.0, 12.0, n, device="cuda")
    if order == "falling":
        ramp = ramp.flip(0)
    if order == "spiky":
        ramp = torch.where(torch.arange(n, device="cuda") % 97 == 13, ramp, ramp * 0.1)
    ids = c["table"][0, :-(-n // 64)].long()
    rows = c["cache"][ids].reshape(-1, 576)
    rows[:n] = (torch.ones(n, 576, device="cuda") * ramp[:, None] / 4 + 0.1 * rows[:n].float()).to(BF16)
    c["cache"][ids] = rows.view(-1, 64, 576)
    c["q"] = (c["q"].float() * 0.2 + 1.0).to(BF16)
    out, lse = M.mla_decode(c["q"], c["cache"], c["table"], c["lens"], SCALE)
    M.sync_status()
    decode_check(c, out, lse, what=order)


# Softmax weights far below a row's largest.  float16 ends at 2^-24 (steps of 2^-24, so off by 2^-25 at most); a row's
# weights are held against a reference that leaves the largest between 2^7 and 2^15, so that a weight is off by its half
# step or by 2^-25 / 2^7 of the largest one, whichever is more: keys * 2^-32 * max |v| of a result.  In units of
# R.check's spread, which it multiplies with half a step:
def small_weights(spread, keys, v, dtype):
    return spread + (keys * 2.0 ** -32 * v.abs().amax() / R.half_step(dtype) if dtype == FP16 else 0.0)


def sink_rows(n, gap, g, dtype):
    """Cached rows: key 0 is `gap` above the others, which are alike, and its values are zero; queries of (0, 1)."""
    rows = torch.zeros(n, 576, device="cuda")
    rows[1:, :512] = 40.0 + normal(g, n - 1, 512, dtype=torch.float32)
    rows[0, 512:] = gap / (64 * SCALE)
    return rows.to(dtype)


@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("gap", [12.0, 15.0, 17.5, 19.0])
@pytest.mark.parametrize("H", [16, 128])
def test_decode_weights_far_below_the_largest(M, H, gap, dtype):
    n = 120
    c = decode_case(1, 1, H, [n], 64, dtype, seed=15)
    rows = sink_rows(n, gap, gen(16), dtype)
    ids = c["table"][0, :2].long()
    c["cache"][ids] = torch.cat([rows, rows[:8]]).view(2, 64, 576)
    c["q"] = torch.cat([torch.zeros(512), torch.ones(64)]).to("cuda", dtype).expand(1, 1, H, 576).contiguous()
    out, lse = M.mla_decode(c["q"], c["cache"], c["table"], c["lens"], SCALE)
    M.sync_status()
    kv = rows.double()
    ref = R.attend(c["q"].double().reshape(H, 576), kv, kv[:, :512], SCALE, torch.full((H,), n, device="cuda"))
    R.check(out.view(H, 512), lse.view(H), ref[0], ref[1], small_weights(ref[2], n, kv[:, :512], dtype), ref[3], dtype, n)


@pytest.mark.parametrize("H,tile", [(16, 64), (128, 128)])
def test_decode_maxima_that_grow_by_just_less_than_a_rescaling(M, H, tile):
    """The largest weights that float16 has to hold: every tile's maximum is 2^7.9 times the one before."""
    n = 4 * tile
    c = decode_case(1, 1, H, [n], 64, FP16, seed=17)
    g = gen(18)
    rows = normal(g, n, 576, dtype=torch.float32)
    rows[:, 512:] = (5.47 * (torch.arange(n, device="cuda") // tile) / (64 * SCALE))[:, None]
    rows = rows.to(FP16)
    c["cache"][c["table"][0, :n // 64].long()] = rows.view(-1, 64, 576)
    c["q"] = torch.cat([torch.zeros(512), torch.ones(64)]).to("cuda", FP16).expand(1, 1, H, 576).contiguous()
    out, lse = M.mla_decode(c["q"], c["cache"], c["table"], c["lens"], SCALE)
    M.sync_status()
    kv = rows.double()
    ref = R.attend(c["q"].double().reshape(H, 576), kv, kv[:, :512], SCALE, torch.full((H,), n, device="cuda"))
    R.check(out.view(H, 512), lse.view(H), ref[0], ref[1], small_weights(ref[2], n, kv[:, :512], FP16), ref[3], FP16, n)


def test_decode_non_finite_scores_stay_in_their_rows(M):
    """A NaN query spoils its own row and no other."""
    c = decode_case(2, 1, 16, [200, 90], 16, BF16, seed=12)
    clean, clean_lse = M.mla_decode(c["q"], c["cache"], c["table"], c["lens"], SCALE)
    c["q"][0, 0, 5, 3] = math.nan
    out, lse = M.mla_decode(c["q"], c["cache"], c["table"], c["lens"], SCALE)
    M.sync_status()
    assert bool(out[0, 0, 5].isnan().all()) and bool(lse[0, 0, 5].isnan())
    out[0, 0, 5], lse[0, 0, 5] = clean[0, 0, 5], clean_lse[0, 0, 5]
    assert torch.equal(out, clean) and torch.equal(lse, clean_lse)


def test_decode_bad_pages_and_lengths_are_reported(M):
    """Host-visible status, zero rows in the place of a page that does not exist, lengths clamped."""
    c = decode_case(3, 1, 16, [100, 64, 130], 64, BF16, seed=13)
    want, want_lse = M.mla_decode(c["q"], c["cache"], c["table"], c["lens"], SCALE)
    M.sync_status()
    table = c["table"].clone()
    table[0, 1] = c["cache"].shape[0]                      # one past the last page
    out, lse = M.mla_decode(c["q"], c["cache"], table, c["lens"], SCALE)
    with pytest.raises(M.Nvfp4MoeError) as e:
        M.sync_status()
    assert e.value.status == 7
    assert torch.equal(out[1:], want[1:]) and torch.equal(lse[1:], want_lse[1:])
    assert bool(out.isfinite().all())
    c["lens"][1] = -5
    out, lse = M.mla_decode(c["q"], c["cache"], c["table"], c["lens"], SCALE)
    with pytest.raises(M.Nvfp4MoeError):
        M.sync_status()
    assert bool((out[1] == 0).all()) and bool((lse[1] == -math.inf).all()) and torch.equal(out[2], want[2])
    c["lens"][1] = 1 << 30                                 # clamped to the table's width, whose last ids are bad
    M.mla_decode(c["q"], c["cache"], c["table"], c["lens"], SCALE)
    with pytest.raises(M.Nvfp4MoeError):
        M.sync_status()
    M.sync_status()


def test_decode_wide_table_view_graph_and_streams(M):
    """A block table that is a slice of a wider one; a captured call replayed on new lengths; a side stream."""
    c = decode_case(6, 2, 16, [900, 33, 64, 5, 2000, 650], 64, BF16, seed=14)
    wide = torch.full((6, c["table"].shape[1] + 40), -7, dtype=torch.int32, device="cuda")
    wide[:, :c["table"].shape[1]] = c["table"]
    view = wide[:, :c["table"].shape[1]]
    ws = torch.empty(M.mla_decode_workspace_size(), dtype=torch.uint8, device="cuda")
    out, lse = M.mla_decode(c["q"], c["cache"], view, c["lens"], SCALE, workspace=ws)
    M.sync_status()
    decode_check(c, out, lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        M.mla_decode(c["q"], c["cache"], view, c["lens"], SCALE, out=out, lse=lse, workspace=ws)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            M.mla_decode(c["q"], c["cache"], view, c["lens"], SCALE, out=out, lse=lse, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    c["lens_host"] = [20, 3, 64, 2, 1999, 0]
    c["lens"].copy_(torch.tensor(c["lens_host"], dtype=torch.int32))
    graph.replay()
    M.sync_status()
    decode_check(c, out, lse, what="replay")


def test_decode_empty_batch(M):
    out, lse = M.mla_decode(torch.empty(0, 1, 16, 576, dtype=BF16, device="cuda"),
                            torch.zeros(1, 16, 576, dtype=BF16, device="cuda"),
                            torch.empty(0, 4, dtype=torch.int32, device="cuda"),
                            torch.empty(0, dtype=torch.int32, device="cuda"), SCALE)
    assert out.shape == (0, 1, 16, 512) and lse.shape == (0, 1, 16)


# ---- prefill -------------------------------------------------------------------------------------------------
def prefill_case(lens, H, dtype, seed, pad=5, q_std=1.0):
    """lens: (queries, keys) of each sequence.  `pad` tokens of NaN follow the last sequence."""
    g = gen(seed)
    cu_q = [0]
    cu_k = [0]
    for n, m in lens:
        cu_q.append(cu_q[-1] + n)
        cu_k.append(cu_k[-1] + m)
    Tq, Tk = cu_q[-1] + pad, cu_k[-1] + pad
    q = normal(g, Tq, H, 192, dtype=dtype, std=q_std)
    up, kr = normal(g, Tk, H, 256, dtype=dtype), normal(g, Tk, 576, dtype=dtype)
    for x, n in ((q, cu_q[-1]), (up, cu_k[-1]), (kr, cu_k[-1])):
        x[n:] = math.nan
    return dict(q=q, up=up, kr=kr[:, 512:], lens=lens, host_q=cu_q, host_k=cu_k,
                cu_q=torch.tensor(cu_q, dtype=torch.int32, device="cuda"),
                cu_k=torch.tensor(cu_k, dtype=torch.int32, device="cuda"))


def prefill_run(M, c, causal=True, **kw):
    return M.mla_prefill(c["q"], c["up"][..., :128], c["kr"], c["up"][..., 128:], c["cu_q"], c["cu_k"], SCALE,
                         causal=causal, **kw)


def prefill_check(c, out, lse, causal=True, what="", only=None, heads=None):
    H = c["q"].shape[1]
    for b in (range(len(c["lens"])) if only is None else only):
        n, m = c["lens"][b]
        if n == 0:
            continue
        q0, k0 = c["host_q"][b], c["host_k"][b]
        sees = (m - n + 1 + torch.arange(n, device="cuda")).clamp(0, m) if causal else torch.full((n,), m, device="cuda")
        for h in (range(H) if heads is None else heads):
            k = torch.cat([c["up"][k0:k0 + m, h, :128], c["kr"][k0:k0 + m]], 1).double()
            v = c["up"][k0:k0 + m, h, 128:].double()
            ref = R.attend(c["q"][q0:q0 + n, h].double(), k, v, SCALE, sees)
            R.check(out[q0:q0 + n, h], lse[q0:q0 + n, h], ref[0], ref[1], ref[2], ref[3], c["q"].dtype, m,
                    f"{what} sequence {b} ({n} of {m}) head {h}")


@pytest.mark.parametrize("lens,H,dtype", [
    ([(1, 1)], 1, BF16), ([(19, 19)], 2, BF16), ([(128, 128)], 1, FP16), ([(129, 129)], 1, BF16),
    ([(256, 256)], 2, BF16), ([(257, 257)], 1, BF16), ([(1, 300)], 3, FP16), ([(130, 517)], 2, BF16),
    ([(64, 64), (0, 0), (1, 1), (200, 333), (0, 40), (300, 300)], 3, BF16), ([(5, 0), (7, 3), (300, 129)], 2, BF16),
    ([(1000, 1000)], 5, FP16), ([(300, 2000), (77, 1024), (513, 513)], 2, BF16),
    ([(1 + 3 * i, 1 + 5 * i) for i in range(70)], 1, BF16)])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_matches_reference(M, lens, H, dtype, causal):
    c = prefill_case(lens, H, dtype, seed=len(lens) + H)
    out = torch.full((c["q"].shape[0], H, 128), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((c["q"].shape[0], H), 7.0, device="cuda")
    prefill_run(M, c, causal, out=out, lse=lse)
    M.sync_status()
    prefill_check(c, out, lse, causal)
    assert bool((out[c["host_q"][-1]:] == 7.0).all()) and bool((lse[c["host_q"][-1]:] == 7.0).all())


def test_prefill_long_and_repeatable(M):
    c = prefill_case([(5000, 5000)], 4, BF16, seed=21)
    out, lse = prefill_run(M, c)
    again = prefill_run(M, c)
    M.sync_status()
    prefill_check(c, out, lse, heads=[0, 3])
    n = c["host_q"][-1]
    assert torch.equal(out[:n], again[0][:n]) and torch.equal(lse[:n], again[1][:n])


@pytest.mark.parametrize("order", ["rising", "falling"])
def test_prefill_scores_that_grow(M, order):
    n = 700
    c = prefill_case([(n, n)], 2, BF16, seed=22)
    ramp = torch.linspace(0.0, 20.0, n, device="cuda")
    if order == "falling":
        ramp = ramp.flip(0)
    c["up"][:n, :, :128] = (ramp[:, None, None] / 4 + 0.1 * c["up"][:n, :, :128].float()).to(BF16)
    c["q"][:n] = (c["q"][:n].float() * 0.2 + 1.0).to(BF16)
    out, lse = prefill_run(M, c)
    M.sync_status()
    prefill_check(c, out, lse, what=order)


@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("gap", [12.0, 15.0, 17.5, 19.0])
def test_prefill_weights_far_below_the_largest(M, gap, dtype):
    n = 300
    c = prefill_case([(n, n)], 2, dtype, seed=26, pad=0)
    rows = sink_rows(n, gap, gen(27), dtype)
    c["up"][..., :128] = 0.0
    c["up"][..., 128:] = rows[:, None, :128]
    c["kr"] = rows[:, 512:]
    c["q"][...] = 0.0
    c["q"][..., 128:] = 1.0
    out, lse = prefill_run(M, c)
    M.sync_status()
    v, k = rows[:, :128].double(), torch.cat([torch.zeros(n, 128, device="cuda"), rows[:, 512:]], 1).double()
    ref = R.attend(c["q"][:, 0].double(), k, v, SCALE, torch.arange(1, n + 1, device="cuda"))
    for h in range(2):
        R.check(out[:, h], lse[:, h], ref[0], ref[1], small_weights(ref[2], n, v, dtype), ref[3], dtype, n)


def test_prefill_maxima_that_grow_by_just_less_than_a_rescaling(M):
    n = 512
    c = prefill_case([(n, n)], 1, FP16, seed=28, pad=0)
    c["up"][..., :128] = 0.0
    c["kr"] = (5.47 * (torch.arange(n, device="cuda") // 128) / (64 * SCALE))[:, None].expand(n, 64).to(FP16).contiguous()
    c["q"][..., :128] = 0.0
    c["q"][..., 128:] = 1.0
    out, lse = prefill_run(M, c)
    M.sync_status()
    v, k = c["up"][:, 0, 128:].double(), torch.cat([c["up"][:, 0, :128], c["kr"]], 1).double()
    ref = R.attend(c["q"][:, 0].double(), k, v, SCALE, torch.arange(1, n + 1, device="cuda"))
    R.check(out[:, 0], lse[:, 0], ref[0], ref[1], small_weights(ref[2], n, v, FP16), ref[3], FP16, n)


def test_prefill_random_shapes(M):
    rng = random.Random(4)
    for i in range(16):
        B, H, top = rng.choice([1, 2, 5, 33]), rng.choice([1, 3, 8]), rng.choice([2, 130, 700])
        lens = [(rng.randint(0, top), rng.randint(0, top)) for _ in range(B)]
        causal = rng.random() < 0.7
        c = prefill_case(lens, H, rng.choice([BF16, FP16]), seed=50 + i)
        out, lse = prefill_run(M, c, causal)
        M.sync_status()
        prefill_check(c, out, lse, causal, what=f"draw {i}", heads=[0, H - 1])


def test_prefill_non_finite_stays_in_its_sequence_and_row(M):
    c = prefill_case([(100, 100), (150, 150)], 2, BF16, seed=23)
    clean, clean_lse = prefill_run(M, c)
    c["up"][:100] = math.nan                               # all of sequence 0's keys and values
    c["q"][100 + 7, 1, 3] = math.nan                       # one query of sequence 1
    out, lse = prefill_run(M, c)
    M.sync_status()
    assert bool(out[:100].isnan().all()) and bool(out[107, 1].isnan().all()) and bool(lse[107, 1].isnan())
    out[107, 1], lse[107, 1] = clean[107, 1], clean_lse[107, 1]
    assert torch.equal(out[100:250], clean[100:250]) and torch.equal(lse[100:250], clean_lse[100:250])


def test_prefill_bad_offsets_are_clamped_and_reported(M):
    c = prefill_case([(100, 100), (60, 60)], 2, BF16, seed=24, pad=0)
    want, want_lse = prefill_run(M, c)
    M.sync_status()
    for name, i, value in (("cu_q", 2, 1000), ("cu_k", 2, 1 << 30), ("cu_q", 0, -5), ("cu_k", 0, -1)):
        bad = dict(c)
        bad[name] = c[name].clone()
        bad[name][i] = value
        out, lse = prefill_run(M, bad)
        with pytest.raises(M.Nvfp4MoeError) as e:
            M.sync_status()
        assert e.value.status == 7
        assert torch.equal(out, want) and torch.equal(lse, want_lse)       # clamping restores these offsets
    bad = dict(c)
    bad["cu_q"] = torch.tensor([100, 0, 160], dtype=torch.int32, device="cuda")   # descending: an empty sequence
    prefill_run(M, bad)
    with pytest.raises(M.Nvfp4MoeError):
        M.sync_status()
    M.sync_status()


def test_prefill_graph_replays_on_new_offsets(M):
    c = prefill_case([(150, 150), (300, 400)], 2, BF16, seed=25)
    out, lse = prefill_run(M, c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        prefill_run(M, c, out=out, lse=lse)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            prefill_run(M, c, out=out, lse=lse)
    torch.cuda.current_stream().wait_stream(side)
    c["lens"], c["host_q"], c["host_k"] = [(430, 430), (20, 120)], [0, 430, 450], [0, 430, 550]
    c["cu_q"].copy_(torch.tensor(c["host_q"], dtype=torch.int32))
    c["cu_k"].copy_(torch.tensor(c["host_k"], dtype=torch.int32))
    graph.replay()
    M.sync_status()
    prefill_check(c, out, lse, what="replay")


def test_prefill_without_tokens_or_sequences(M):
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    e = torch.empty(0, 2, 192, dtype=BF16, device="cuda")
    out, lse = M.mla_prefill(e, e[..., :128], torch.empty(0, 64, dtype=BF16, device="cuda"), e[..., :128], z, z, SCALE)
    assert out.shape == (0, 2, 128) and lse.shape == (0, 2)
    q = torch.ones(3, 2, 192, dtype=BF16, device="cuda")                   # queries, but no keys at all
    cu = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    out, lse = M.mla_prefill(q, e[..., :128], torch.empty(0, 64, dtype=BF16, device="cuda"), e[..., :128], cu,
                             torch.zeros(2, dtype=torch.int32, device="cuda"), SCALE)
    M.sync_status()
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())
