"""Latent attention: ctypes binding of include/nvfp4mla.h.

Like `binding`, argument marshalling only: every function checks types,
shapes, strides and devices, allocates what the caller does not pass and
calls the C entry point of the same name on the current CUDA stream.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding as _b
from .binding import Nvfp4MoeError, sync_status  # noqa: F401  (part of this module's surface)

LATENT, ROPE, ROW = 512, 64, 576          # latent and rotary values of a cached row
NOPE, VALUE = 128, 128                    # expanded form: unrotated values of a key, values of a head
DTYPE = {torch.bfloat16: 0, torch.float16: 1}

_i, _i64, _sz, _p, _f = ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_float
_SIGS = {
    "mla_append": (_i, [_p, _i64, _p, _i64, _p, _f, _p, _p, _i, _p, _i64, _i, _i, _p, _i64, _p, _p, _i64, _i64, _i, _p,
                        _i64, _i64, _p]),
    "mla_decode_workspace_size": (_sz, []),
    "mla_prefill": (_i, [_p, _i64, _i64, _p, _i64, _i64, _p, _i64, _p, _i64, _i64, _p, _p, _i, _i, _i, _i, _f, _i, _i, _p,
                         _p, _p]),
    "mla_decode": (_i, [_p, _p, _i, _i, _p, _i64, _i, _p, _i, _i, _i, _f, _i, _p, _p, _p, _sz, _p]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(_b._lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args
_lib = _b._lib


def _typed(t, dtype, shape, name):
    """Checks everything but the layout; a None in `shape` is any size."""
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.dim() != len(shape) or any(s is not None and s != n for s, n in zip(shape, t.shape)):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple('*' if s is None else s for s in shape)}")
    return t


def _dense(t, dtype, shape, name):
    _typed(t, dtype, shape, name)
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _strided(t, dtype, shape, name):
    """A view whose innermost dimension is contiguous and whose rows start on 16-byte boundaries."""
    _typed(t, dtype, shape, name)
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.numel() and (t.stride(-1) != 1 or t.data_ptr() % 16 or
                      any(s % 8 for n, s in zip(t.shape[:-1], t.stride()[:-1]) if n > 1)):
        raise ValueError(f"{name}: strides {t.stride()} (innermost 1, others multiples of 8, 16-byte aligned)")
    return t


def _step(t, dim):
    """Stride of a dimension; 0 where it has one entry, whose stride says nothing."""
    return t.stride(dim) if t.shape[dim] > 1 else 0


def _one_device(**tensors):
    devices = {t.device for t in tensors.values() if t is not None}
    if len(devices) > 1:
        raise ValueError(f"tensors on different devices: {sorted(str(d) for d in devices)}")


def _dtype(t, name):
    if t.dtype not in DTYPE:
        raise TypeError(f"{name}: dtype {t.dtype}, expected torch.bfloat16 or torch.float16")
    return DTYPE[t.dtype]


def rope_table(max_positions, base=10000.0, device="cuda"):
    """float32 [max_positions, 64]: cosines then sines of the 32 angles p * base^(-i / 32),
    from angles in 64 bits (float32 angles lose the fraction of far positions)."""
    inv = float(base) ** (-torch.arange(0, ROPE, 2, dtype=torch.float64, device=device) / ROPE)
    ang = torch.arange(max_positions, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], dim=1).to(torch.float32)


def mla_append(latent, k_rope, positions, slots, rope_table, cache, norm_weight=None, eps=1e-6, interleaved=True,
               q_rope=None, q_out=None, rows_out=None):
    """Normalises and rotates T new tokens and writes their rows to the cache
    slots; rotates their queries.

    latent [T, 512], k_rope [T, 64], q_rope [T, H, 64] may be slices of a
    projection's output; cache [num_pages, page_size, 576].  rows_out [T, 576]
    takes a copy of the rows (what the expanded form projects).  q_out [T, H,
    64] may be a slice of the queries' buffer or q_rope itself; it is made when
    q_rope comes without it.  Returns q_out (None without queries)."""
    dt = _dtype(latent, "latent")
    T, t = latent.shape[0], latent.dtype
    _strided(latent, t, (None, LATENT), "latent")
    _strided(k_rope, t, (T, ROPE), "k_rope")
    _dense(positions, torch.int32, (T,), "positions")
    _dense(slots, torch.int64, (T,), "slots")
    _dense(rope_table, torch.float32, (None, ROPE), "rope_table")
    _dense(cache, t, (None, None, ROW), "cache")
    if norm_weight is not None:
        _dense(norm_weight, t, (LATENT,), "norm_weight")
    if rows_out is not None:
        _dense(rows_out, t, (T, ROW), "rows_out")
    H = 0
    if q_rope is not None:
        H = q_rope.shape[1]
        _strided(q_rope, t, (T, None, ROPE), "q_rope")
        if q_out is None:
            q_out = torch.empty((T, H, ROPE), dtype=t, device=latent.device)
        _strided(q_out, t, (T, H, ROPE), "q_out")
    elif q_out is not None:
        raise ValueError("q_out without q_rope")
    _one_device(latent=latent, k_rope=k_rope, positions=positions, slots=slots, rope_table=rope_table, cache=cache,
                norm_weight=norm_weight, rows_out=rows_out, q_rope=q_rope, q_out=q_out)
    q = (_b._ptr(q_rope), _step(q_rope, 0), _step(q_rope, 1), H, _b._ptr(q_out), _step(q_out, 0), _step(q_out, 1)) \
        if H else (None, 0, 0, 0, None, 0, 0)
    _b._check(_lib.mla_append(_b._ptr(latent), _step(latent, 0), _b._ptr(k_rope), _step(k_rope, 0),
                              _b._ptr(norm_weight), float(eps), _b._ptr(positions), _b._ptr(slots), T,
                              _b._ptr(rope_table), rope_table.shape[0], int(bool(interleaved)), dt, _b._ptr(cache),
                              cache.shape[0] * cache.shape[1], _b._ptr(rows_out), *q, _b._stream()), "mla_append")
    return q_out


def mla_decode_workspace_size():
    return int(_lib.mla_decode_workspace_size())


def mla_decode(q, cache, block_tables, seq_lens, scale, out=None, lse=None, workspace=None):
    """Absorbed attention of the Sq newest tokens of each sequence over the paged cache.

    q [B, Sq, H, 576], cache [num_pages, page_size, 576], block_tables int32
    [B, max_pages], seq_lens int32 [B] (the new tokens counted).  Returns (out
    [B, Sq, H, 512], lse float32 [B, Sq, H])."""
    dt = _dtype(q, "q")
    t = q.dtype
    _dense(q, t, (None, None, None, ROW), "q")
    B, Sq, H, _ = q.shape
    _dense(cache, t, (None, None, ROW), "cache")
    _typed(block_tables, torch.int32, (B, None), "block_tables")
    if not block_tables.is_cuda or (block_tables.numel() and block_tables.stride(1) != 1):
        raise ValueError("block_tables must be a CUDA tensor with contiguous rows")
    _dense(seq_lens, torch.int32, (B,), "seq_lens")
    out = torch.empty((B, Sq, H, LATENT), dtype=t, device=q.device) if out is None else out
    lse = torch.empty((B, Sq, H), dtype=torch.float32, device=q.device) if lse is None else lse
    _dense(out, t, (B, Sq, H, LATENT), "out")
    _dense(lse, torch.float32, (B, Sq, H), "lse")
    if workspace is None:
        workspace = torch.empty((mla_decode_workspace_size(),), dtype=torch.uint8, device=q.device)
    _dense(workspace, torch.uint8, (None,), "workspace")
    _one_device(q=q, cache=cache, block_tables=block_tables, seq_lens=seq_lens, out=out, lse=lse, workspace=workspace)
    max_pages = block_tables.shape[1]
    _b._check(_lib.mla_decode(_b._ptr(q), _b._ptr(cache), cache.shape[0], cache.shape[1], _b._ptr(block_tables),
                              max(max_pages, block_tables.stride(0) if B > 1 else 0), max_pages, _b._ptr(seq_lens), B,
                              Sq, H, float(scale), dt, _b._ptr(out), _b._ptr(lse), _b._ptr(workspace),
                              workspace.numel(), _b._stream()), "mla_decode")
    return out, lse


def _span(t, dim, dense):
    """Stride of a dimension; `dense` where it has at most one entry, whose stride says nothing."""
    return t.stride(dim) if t.shape[dim] > 1 else dense


def mla_prefill(q, k_nope, k_rope, v, cu_q, cu_k, scale, causal=True, out=None, lse=None):
    """Expanded attention over a ragged batch; queries are the last of their sequence's keys.

    q [Tq, H, 192], k_nope [Tk, H, 128], k_rope [Tk, 64] and v [Tk, H, 128] may
    be slices of projections' outputs; cu_q, cu_k int32 [B + 1] are the
    sequences' offsets.  Returns (out [Tq, H, 128], lse float32 [Tq, H])."""
    dt = _dtype(q, "q")
    t = q.dtype
    _strided(q, t, (None, None, NOPE + ROPE), "q")
    Tq, H, _ = q.shape
    _strided(k_nope, t, (None, H, NOPE), "k_nope")
    Tk = k_nope.shape[0]
    _strided(k_rope, t, (Tk, ROPE), "k_rope")
    _strided(v, t, (Tk, H, VALUE), "v")
    _dense(cu_q, torch.int32, (None,), "cu_q")
    B = cu_q.shape[0] - 1
    if B < 0:
        raise ValueError("cu_q must have an entry more than there are sequences")
    _dense(cu_k, torch.int32, (B + 1,), "cu_k")
    out = torch.empty((Tq, H, VALUE), dtype=t, device=q.device) if out is None else out
    lse = torch.empty((Tq, H), dtype=torch.float32, device=q.device) if lse is None else lse
    _dense(out, t, (Tq, H, VALUE), "out")
    _dense(lse, torch.float32, (Tq, H), "lse")
    _one_device(q=q, k_nope=k_nope, k_rope=k_rope, v=v, cu_q=cu_q, cu_k=cu_k, out=out, lse=lse)
    _b._check(_lib.mla_prefill(
        _b._ptr(q), _span(q, 0, 192 * max(H, 1)), _span(q, 1, 192),
        _b._ptr(k_nope), _span(k_nope, 0, NOPE * max(H, 1)), _span(k_nope, 1, NOPE),
        _b._ptr(k_rope), _span(k_rope, 0, ROPE), _b._ptr(v), _span(v, 0, VALUE * max(H, 1)), _span(v, 1, VALUE),
        _b._ptr(cu_q), _b._ptr(cu_k), B, Tq, Tk, H, float(scale), int(bool(causal)), dt, _b._ptr(out), _b._ptr(lse),
        _b._stream()), "mla_prefill")
    return out, lse
