"""Latent attention: ctypes binding of include/nvfp4mla.h.

Like `binding`, argument marshalling only: every function checks types,
shapes, strides and devices, allocates what the caller does not pass and
calls the C entry point of the same name on the current CUDA stream.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import binding as _b
from .binding import Nvfp4MoeError, sync_status  # noqa: F401  (part of this module's surface)

LATENT, ROPE, ROW = 512, 64, 576          # latent and rotary values of a cached row
NOPE, VALUE = 128, 128                    # expanded form: unrotated values of a key, values of a head
DTYPE = {torch.bfloat16: 0, torch.float16: 1}

_i, _i64, _sz, _p, _f = ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_float
_SIGS = {
    "mla_plan": (_i, [_p, _p, _i, _i, _p, _i64, _i, _p, _i, _p, _i, _p, _p, _p, _p, _p, _p, _p]),
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
_DECODE_WORKSPACE = int(_lib.mla_decode_workspace_size())


# The checks below run on every call of a decode step, whose kernels take
# microseconds: they read each property once and build no message before it is
# needed.
def _refuse(t, dtype, shape, name, device):
    """The error of a tensor that is not what a call needs."""
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {shape}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, the first tensor on cuda:{device}")
    raise ValueError(f"{name} must be contiguous")


def _dense(t, dtype, shape, name, device):
    """A contiguous tensor's data pointer."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
        return t.data_ptr()
    _refuse(t, dtype, shape, name, device)


def _strided(t, dtype, shape, name, device):
    """A view whose innermost dimension is contiguous and whose rows start on
    16-byte boundaries.  Returns the pointer and the other dimensions' strides,
    which say nothing (a dense tensor's are given) where a dimension has one
    entry."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device:
        _refuse(t, dtype, shape, name, device)
    p, stride = t.data_ptr(), t.stride()
    if len(shape) == 2:
        steps = (stride[0] if shape[0] > 1 else shape[1],)
        bad = steps[0] % 8
    else:
        steps = (stride[0] if shape[0] > 1 else shape[1] * shape[2] or 8, stride[1] if shape[1] > 1 else shape[2])
        bad = steps[0] % 8 or steps[1] % 8
    if bad or p % 16 or stride[-1] != 1 and t.numel():
        raise ValueError(f"{name}: strides {stride}, address {p:#x} (innermost 1, others multiples of 8, 16-byte aligned)")
    return (p, *steps)


def _first(t, name, dims):
    """The first tensor of a call sets its dtype and device: (dtype, its code, device index)."""
    if t.dtype not in DTYPE:
        raise TypeError(f"{name}: dtype {t.dtype}, expected torch.bfloat16 or torch.float16")
    if t.dim() != dims:
        raise ValueError(f"{name}: {t.dim()} dimensions, expected {dims}")
    return t.dtype, DTYPE[t.dtype], t.get_device()


def _on_cuda(device, name):
    if device < 0:
        raise ValueError(f"{name} must be a CUDA tensor")


def _stream(device):
    """The device's current stream; calls are made with that device current."""
    if device != torch._C._cuda_getDevice():
        raise ValueError(f"tensors on cuda:{device}, but the current device is cuda:{torch.cuda.current_device()}")
    return torch._C._cuda_getCurrentRawStream(device)


def rope_table(max_positions, base=10000.0, device="cuda"):
    """float32 [max_positions, 64]: cosines then sines of the 32 angles p * base^(-i / 32),
    from angles in 64 bits (float32 angles lose the fraction of far positions)."""
    inv = float(base) ** (-torch.arange(0, ROPE, 2, dtype=torch.float64, device=device) / ROPE)
    ang = torch.arange(max_positions, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], dim=1).to(torch.float32)


@dataclass
class TokenPlan:
    """Where a step's new tokens go: what the other calls take (see mla_plan)."""
    positions: torch.Tensor     # int32 [T]
    slots: torch.Tensor         # int64 [T]
    cu_seqlens: torch.Tensor    # int32 [B + 1]
    seq_lens: torch.Tensor      # int32 [B]
    granted: torch.Tensor       # int32 [B]
    free_count: torch.Tensor    # int32 [1]


def alloc_token_plan(B, T, device, free_count=None):
    """Buffers for mla_plan(out=...); free_count: the caller's, updated in place."""
    empty, i32 = torch.empty, torch.int32
    return TokenPlan(empty(T, dtype=i32, device=device), empty(T, dtype=torch.int64, device=device),
                     empty(B + 1, dtype=i32, device=device), empty(B, dtype=i32, device=device),
                     empty(B, dtype=i32, device=device), empty(1, dtype=i32, device=device) if free_count is None else free_count)


def mla_plan(past_lens, new_lens, block_tables, free_pages, free_count, page_size, tokens, out=None):
    """Pages and slots of a step's new tokens, on the GPU.

    past_lens, new_lens int32 [B]: tokens that each request has in the cache and
    brings; block_tables int32 [B, max_pages], whose new entries are written;
    free_pages int32 [n] with free_count int32 [1] of them free, popped from the
    end; tokens: rows of the step's buffers (those past the last token get slot
    -1).  A request whose pages are not there is refused: granted 0, slots -1.
    Returns a TokenPlan (`out`, if given).  out.seq_lens may be past_lens,
    out.granted new_lens and out.free_count free_count; outputs that share
    memory otherwise, with one another, the inputs or the tables, are refused."""
    dev = past_lens.get_device()
    _on_cuda(dev, "past_lens")
    B = past_lens.shape[0]
    i32 = torch.int32
    past_at = _dense(past_lens, i32, (B,), "past_lens", dev)
    if block_tables.dim() != 2:
        raise ValueError("block_tables has two dimensions")
    max_pages = block_tables.shape[1]
    if block_tables.dtype is not i32 or block_tables.shape[0] != B or block_tables.get_device() != dev:
        _refuse(block_tables, i32, (B, max_pages), "block_tables", dev)
    step = block_tables.stride()
    if (max_pages > 1 and step[1] != 1) or (B > 1 and step[0] < max_pages):
        raise ValueError(f"block_tables: strides {step}, rows must be contiguous and apart")
    free = free_pages.numel()
    if out is None:                           # what is made here needs no check
        out = alloc_token_plan(B, tokens, past_lens.device)
        at = [t.data_ptr() for t in (out.positions, out.slots, out.cu_seqlens, out.seq_lens, out.granted, out.free_count)]
    else:
        at = [_dense(out.positions, i32, (tokens,), "positions", dev), _dense(out.slots, torch.int64, (tokens,), "slots", dev),
              _dense(out.cu_seqlens, i32, (B + 1,), "cu_seqlens", dev), _dense(out.seq_lens, i32, (B,), "seq_lens", dev),
              _dense(out.granted, i32, (B,), "granted", dev), _dense(out.free_count, i32, (1,), "free_count_out", dev)]
    _b._check(_lib.mla_plan(
        past_at, _dense(new_lens, i32, (B,), "new_lens", dev), B, page_size, block_tables.data_ptr(),
        step[0] if B > 1 else max_pages, max_pages, _dense(free_pages, i32, (free,), "free_pages", dev), free,
        _dense(free_count, i32, (1,), "free_count", dev), tokens, *at, _stream(dev)), "mla_plan")
    return out


def mla_append(latent, k_rope, positions, slots, rope_table, cache, norm_weight=None, eps=1e-6, interleaved=True,
               q_rope=None, q_out=None, rows_out=None):
    """Normalises and rotates T new tokens and writes their rows to the cache
    slots; rotates their queries.

    latent [T, 512], k_rope [T, 64], q_rope [T, H, 64] may be slices of a
    projection's output; cache [num_pages, page_size, 576].  rows_out [T, 576]
    takes a copy of the rows (what the expanded form projects).  q_out [T, H,
    64] may be a slice of the queries' buffer or q_rope itself; it is made when
    q_rope comes without it.  A token whose position is outside the table is
    not written anywhere (sync_status reports it).  Returns q_out (None without queries)."""
    t, code, dev = _first(latent, "latent", 2)
    T = len(latent)
    latent_at = _strided(latent, t, (T, LATENT), "latent", dev)
    _on_cuda(dev, "latent")
    rope_at = _strided(k_rope, t, (T, ROPE), "k_rope", dev)
    if cache.dim() != 3 or rope_table.dim() != 2 or (q_rope is not None and q_rope.dim() != 3):
        raise ValueError("cache and q_rope have three dimensions, rope_table has two")
    pages, page, _ = cache.shape
    cache_at = _dense(cache, t, (pages, page, ROW), "cache", dev)
    span = len(rope_table)
    q_at, q_out_at, H = (None, 0, 0), (None, 0, 0), 0
    if q_rope is not None:
        H = q_rope.shape[1]
        if q_out is None:
            q_out = torch.empty((T, H, ROPE), dtype=t, device=latent.device)
        if H:
            q_at = _strided(q_rope, t, (T, H, ROPE), "q_rope", dev)
            q_out_at = _strided(q_out, t, (T, H, ROPE), "q_out", dev)
    elif q_out is not None:
        raise ValueError("q_out without q_rope")
    _b._check(_lib.mla_append(
        *latent_at, *rope_at, None if norm_weight is None else _dense(norm_weight, t, (LATENT,), "norm_weight", dev),
        eps, _dense(positions, torch.int32, (T,), "positions", dev), _dense(slots, torch.int64, (T,), "slots", dev), T,
        _dense(rope_table, torch.float32, (span, ROPE), "rope_table", dev), span, 1 if interleaved else 0, code,
        cache_at, pages * page, None if rows_out is None else _dense(rows_out, t, (T, ROW), "rows_out", dev),
        *q_at, H, *q_out_at, _stream(dev)), "mla_append")
    return q_out


def mla_decode_workspace_size():
    return _DECODE_WORKSPACE


def mla_decode(q, cache, block_tables, seq_lens, scale, out=None, lse=None, workspace=None):
    """Absorbed attention of the Sq newest tokens of each sequence over the paged cache.

    q [B, Sq, H, 576], cache [num_pages, page_size, 576], block_tables int32
    [B, max_pages], seq_lens int32 [B] (the new tokens counted).  Returns (out
    [B, Sq, H, 512], lse float32 [B, Sq, H])."""
    t, code, dev = _first(q, "q", 4)
    B, Sq, H, _ = q.shape
    q_at = _dense(q, t, (B, Sq, H, ROW), "q", dev)
    _on_cuda(dev, "q")
    if cache.dim() != 3 or block_tables.dim() != 2:
        raise ValueError("cache has three dimensions, block_tables two")
    pages, page, _ = cache.shape
    rows, max_pages = block_tables.shape
    if block_tables.dtype is not torch.int32 or rows != B or block_tables.get_device() != dev:
        _refuse(block_tables, torch.int32, (B, max_pages), "block_tables", dev)
    step = block_tables.stride()
    if max_pages > 1 and step[1] != 1:
        raise ValueError(f"block_tables: strides {step}, rows must be contiguous")
    if out is None:                           # what is made here needs no check
        out = torch.empty((B, Sq, H, LATENT), dtype=t, device=q.device)
        out_at = out.data_ptr()
    else:
        out_at = _dense(out, t, (B, Sq, H, LATENT), "out", dev)
    if lse is None:
        lse = torch.empty((B, Sq, H), dtype=torch.float32, device=q.device)
        lse_at = lse.data_ptr()
    else:
        lse_at = _dense(lse, torch.float32, (B, Sq, H), "lse", dev)
    if workspace is None:
        workspace = torch.empty((_DECODE_WORKSPACE,), dtype=torch.uint8, device=q.device)
        ws_at, ws_bytes = workspace.data_ptr(), _DECODE_WORKSPACE
    else:
        ws_bytes = workspace.numel()
        ws_at = _dense(workspace, torch.uint8, (ws_bytes,), "workspace", dev)
    _b._check(_lib.mla_decode(
        q_at, _dense(cache, t, (pages, page, ROW), "cache", dev), pages, page, block_tables.data_ptr(),
        step[0] if B > 1 else max_pages, max_pages, _dense(seq_lens, torch.int32, (B,), "seq_lens", dev), B, Sq, H,
        scale, code, out_at, lse_at, ws_at, ws_bytes, _stream(dev)), "mla_decode")
    return out, lse


def mla_prefill(q, k_nope, k_rope, v, cu_q, cu_k, scale, causal=True, out=None, lse=None):
    """Expanded attention over a ragged batch; queries are the last of their sequence's keys.

    q [Tq, H, 192], k_nope [Tk, H, 128], k_rope [Tk, 64] and v [Tk, H, 128] may
    be slices of projections' outputs; cu_q, cu_k int32 [B + 1] are the
    sequences' offsets.  Returns (out [Tq, H, 128], lse float32 [Tq, H]), whose
    rows of tokens in no sequence are not written."""
    t, code, dev = _first(q, "q", 3)
    Tq, H, _ = q.shape
    q_at = _strided(q, t, (Tq, H, NOPE + ROPE), "q", dev)
    _on_cuda(dev, "q")
    Tk, B = len(k_nope), cu_q.numel() - 1
    if B < 0:
        raise ValueError("cu_q: one entry more than there are sequences")
    if out is None:
        out = torch.empty((Tq, H, VALUE), dtype=t, device=q.device)
        out_at = out.data_ptr()
    else:
        out_at = _dense(out, t, (Tq, H, VALUE), "out", dev)
    if lse is None:
        lse = torch.empty((Tq, H), dtype=torch.float32, device=q.device)
        lse_at = lse.data_ptr()
    else:
        lse_at = _dense(lse, torch.float32, (Tq, H), "lse", dev)
    _b._check(_lib.mla_prefill(
        *q_at, *_strided(k_nope, t, (Tk, H, NOPE), "k_nope", dev), *_strided(k_rope, t, (Tk, ROPE), "k_rope", dev),
        *_strided(v, t, (Tk, H, VALUE), "v", dev), _dense(cu_q, torch.int32, (B + 1,), "cu_q", dev),
        _dense(cu_k, torch.int32, (B + 1,), "cu_k", dev), B, Tq, Tk, H, scale, 1 if causal else 0, code,
        out_at, lse_at, _stream(dev)), "mla_prefill")
    return out, lse


# ---- the whole attention of a layer --------------------------------------------------
class LatentAttention:
    """Weights of one layer's latent attention and its two forms.

    prefill() takes whole prompts: it appends their rows to the cache and
    attends in the expanded form.  decode() takes the newest tokens of
    sequences whose rows are in the cache: it appends theirs and attends in the
    absorbed form, with the keys' and values' projections folded into the
    queries and the outputs.  The projections are plain matrix products.

    w_q [H * 192, D], w_kv [576, D], kv_norm [512], w_up [H * 256, 512] (of each
    head first the 128 rows of its keys, then of its values), w_o [D, H * 128],
    all of one 16-bit type; rope_table as mla_append takes it."""

    def __init__(self, w_q, w_kv, kv_norm, w_up, w_o, rope_table, eps=1e-6, interleaved=True, scale=None):
        self.H = w_up.shape[0] // (NOPE + VALUE)
        for name, w, shape in (("w_q", w_q, (self.H * (NOPE + ROPE), w_q.shape[1])), ("w_kv", w_kv, (ROW, w_q.shape[1])),
                               ("kv_norm", kv_norm, (LATENT,)), ("w_up", w_up, (self.H * (NOPE + VALUE), LATENT)),
                               ("w_o", w_o, (w_q.shape[1], self.H * VALUE))):
            _dense(w, w_q.dtype, shape, name, w_q.get_device())
        self.w_q, self.w_kv, self.kv_norm, self.w_up, self.w_o = w_q, w_kv, kv_norm, w_up, w_o
        up = w_up.view(self.H, NOPE + VALUE, LATENT)
        self.w_uk, self.w_uv = up[:, :NOPE], up[:, NOPE:].transpose(1, 2)   # [H, 128, 512], [H, 512, 128]
        self.rope_table, self.eps, self.interleaved = rope_table, eps, interleaved
        self.scale = (NOPE + ROPE) ** -0.5 if scale is None else scale

    def _project(self, x):
        return (x @ self.w_q.T).view(x.shape[0], self.H, NOPE + ROPE), x @ self.w_kv.T

    def _append(self, kv, positions, slots, cache, q_rope, q_out, rows_out=None):
        mla_append(kv[:, :LATENT], kv[:, LATENT:], positions, slots, self.rope_table, cache, norm_weight=self.kv_norm,
                   eps=self.eps, interleaved=self.interleaved, q_rope=q_rope, q_out=q_out, rows_out=rows_out)

    def prefill(self, x, positions, slots, cache, cu_seqlens):
        """x [T, D]: the tokens of whole prompts, sequence b from cu_seqlens[b] on.  Returns [T, D]."""
        q, kv = self._project(x)
        rows = torch.empty_like(kv)
        self._append(kv, positions, slots, cache, q[..., NOPE:], q[..., NOPE:], rows)
        up = (rows[:, :LATENT] @ self.w_up.T).view(-1, self.H, NOPE + VALUE)
        out, _ = mla_prefill(q, up[..., :NOPE], rows[:, LATENT:], up[..., NOPE:], cu_seqlens, cu_seqlens, self.scale)
        return out.flatten(1) @ self.w_o.T

    def decode(self, x, positions, slots, cache, block_tables, seq_lens, workspace=None):
        """x [B * Sq, D]: the Sq newest tokens of each sequence, seq_lens counting them.  Returns [B * Sq, D]."""
        B, tokens = seq_lens.shape[0], x.shape[0]
        Sq = tokens // B if B else 1
        if Sq == 0 or tokens != B * Sq:       # before the cache is written
            raise ValueError(f"x: {tokens} tokens are not as many for each of {B} sequences")
        q, kv = self._project(x)
        absorbed = torch.empty((x.shape[0], self.H, ROW), dtype=x.dtype, device=x.device)
        absorbed[..., :LATENT] = torch.bmm(q[..., :NOPE].transpose(0, 1), self.w_uk).transpose(0, 1)
        self._append(kv, positions, slots, cache, q[..., NOPE:], absorbed[..., LATENT:])
        out, _ = mla_decode(absorbed.view(B, Sq, self.H, ROW), cache, block_tables, seq_lens, self.scale,
                            workspace=workspace)
        heads = torch.bmm(out.view(-1, self.H, LATENT).transpose(0, 1), self.w_uv)
        return heads.transpose(0, 1).flatten(1) @ self.w_o.T
