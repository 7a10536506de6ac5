"""Latent attention and the expert layer run together: the example's block, and the attention of a layer
against its definition in 64 bits."""
import math

import pytest
import torch

from tests import mla_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    from nvfp4_block_scaled_07_gb300 import build
    build.build()
    from nvfp4_block_scaled_07_gb300 import binding, mla
    binding.device_check()
    return mla


def layer(M, D=256, H=3, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def w(*shape, std):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)

    return M.LatentAttention(w(H * 192, D, std=D ** -0.5), w(576, D, std=D ** -0.5), w(512, std=0.1) + 1.0,
                             w(H * 256, 512, std=512 ** -0.5), w(D, H * 128, std=(H * 128) ** -0.5), M.rope_table(1000))


def definition(a, x):
    """The attention of one whole sequence in 64 bits, from the layer's weights."""
    T, H = x.shape[0], a.H
    x = x.double()
    q = (x @ a.w_q.double().T).view(T, H, 192)
    kv = x @ a.w_kv.double().T
    lat = kv[:, :512] / torch.sqrt(kv[:, :512].square().mean(1, keepdim=True) + a.eps) * a.kv_norm.double()
    cs = a.rope_table.double()[:T]
    kr = R.rotate(kv[:, 512:], cs[:, :32], cs[:, 32:], a.interleaved)
    qr = R.rotate(q[..., 128:], cs[:, None, :32], cs[:, None, 32:], a.interleaved)
    up = (lat @ a.w_up.double().T).view(T, H, 256)
    s = (torch.einsum("thd,shd->hts", q[..., :128], up[..., :128]) + torch.einsum("thd,sd->hts", qr, kr)) * a.scale
    s = s.masked_fill(torch.ones(T, T, device="cuda").triu(1).bool(), -math.inf)
    out = torch.einsum("hts,shd->thd", s.softmax(-1), up[..., 128:])
    return out.reshape(T, H * 128) @ a.w_o.double().T


# The layer rounds to bfloat16 (at most 2^-8 a time, 2^-8 / sqrt(3) rms) at x, q, kv, rows, up (or the
# absorbed queries and outputs), weights, heads and the result: at most nine roundings on a path, each of
# a factor of the result or (q, kr, up in the scores, of standard deviation about 1.3) of the exponent,
# which scales them by up to 2: rms of sqrt(9) * 2 * 2^-8 / sqrt(3) = 1.35e-2.
TOL = 1.4e-2


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("lens", [(1,), (70, 3, 200)])
def test_prefill_and_decode_follow_the_definition(M, lens):
    a = layer(M)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    xs = [torch.randn((m, 256), generator=g, device="cuda").to(torch.bfloat16) for m in lens]
    want = [definition(a, x) for x in xs]
    page = 16
    need = [-(-m // page) for m in lens]
    tables = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        tables[b, :n] = torch.arange(at, at + n, device="cuda", dtype=torch.int32)
        at += n
    cache = torch.full((at, page, 576), math.nan, dtype=torch.bfloat16, device="cuda")
    pos = torch.cat([torch.arange(m, device="cuda") for m in lens])
    seq = torch.cat([torch.full((m,), b, device="cuda") for b, m in enumerate(lens)])
    slots = tables.long()[seq, pos // page] * page + pos % page
    cu = torch.tensor([0, *lens], device="cuda").cumsum(0).to(torch.int32)
    y = a.prefill(torch.cat(xs), pos.to(torch.int32), slots, cache, cu)
    M.sync_status()
    assert rel(y, torch.cat(want)) < TOL
    # the last token again, by decoding: its row is written a second time
    last = torch.tensor([m - 1 for m in lens], device="cuda")
    lens_d = (last + 1).to(torch.int32)
    rows = torch.stack([tables.long()[b, m // page] * page + m % page for b, m in enumerate(last)])
    z = a.decode(torch.stack([x[-1] for x in xs]), last.to(torch.int32), rows, cache, tables, lens_d)
    M.sync_status()
    assert rel(z, torch.stack([w[-1] for w in want])) < TOL


def no_tokens(x):
    return torch.empty(x, dtype=torch.int32, device="cuda"), torch.empty(x, dtype=torch.int64, device="cuda")


def test_empty_batches_give_empty_results(M):
    """A batch that has drained: no prompts, or no sequences to decode."""
    a = layer(M)
    cache = torch.zeros((2, 16, 576), dtype=torch.bfloat16, device="cuda")
    x = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    pos, slots = no_tokens(0)
    y = a.prefill(x, pos, slots, cache, torch.zeros(1, dtype=torch.int32, device="cuda"))
    z = a.decode(x, pos, slots, cache, torch.empty((0, 2), dtype=torch.int32, device="cuda"), no_tokens(0)[0])
    M.sync_status()
    assert y.shape == z.shape == (0, 256) and y.dtype == z.dtype == torch.bfloat16


@pytest.mark.parametrize("tokens,sequences", [(3, 2), (0, 2), (1, 0)])
def test_decode_refuses_unequal_tokens_before_the_cache_is_written(M, tokens, sequences):
    a = layer(M)
    cache = torch.zeros((2, 16, 576), dtype=torch.bfloat16, device="cuda")
    x = torch.ones((tokens, 256), dtype=torch.bfloat16, device="cuda")
    at = torch.arange(tokens, device="cuda")
    with pytest.raises(ValueError, match="tokens"):
        a.decode(x, at.to(torch.int32), at, cache, torch.zeros((sequences, 2), dtype=torch.int32, device="cuda"),
                 torch.full((sequences,), 3, dtype=torch.int32, device="cuda"))
    M.sync_status()
    assert bool((cache == 0).all())


def test_example_block_decodes_what_it_prefills(M):
    from examples import decoder_block as E
    decoded, whole = E.serve(lengths=(37, 130, 5), steps=3)
    # The attention agrees within 2 TOL; the experts quantise their input to four bits, which turns a small
    # difference at a rounding border into a step, of at most 1/4 of a value, and the residual x (of size 1,
    # attention and experts add about as much or less) keeps the sum below 0.1.
    assert rel(decoded, whole.double()) < 0.1
    assert bool(decoded.isfinite().all())
