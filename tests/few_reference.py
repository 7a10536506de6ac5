"""The few-token operators in 64 bits, written out from their definitions, and the error bounds of the kernels.

Bounds, element by element, with u = eps / 2 of the 16-bit result type:
  sums     float32 sums of n products: n 2^-23 sum |x w| (2^-23 and not 2^-24: the tensor core may truncate);
  x        the stream kernel's eight 4-bit terms: each leaves at most 0.1875 (0.2 with E8M0 scales) of the largest value
           of its 16 (32), 0.2^8 < 2^-18 of it; and 2^-34 of the row's largest where a block's scale leaves ue4m3's
           normal numbers.  The other kernel's float16 with an exponent for 256 values: 2^-40 of their largest;
  result   one rounding, u |y|.
The experts' h carries the errors of gate and up (a silu's slope is below 1.1), the exponential's 2^-21 and its own
rounding to 11 bits, 2^-11 |h|; each goes through |W_d| and the token's weight.
"""
import itertools

import torch

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
BLOCK = {"nvfp4": 16, "mxfp4": 32}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


class Matrices:
    """E random 4-bit matrices [N, K]: codes, scale bytes (row-major), per-matrix scales, and their float64 values."""

    def __init__(self, E, N, K, fmt, seed, lo=None, hi=None, device="cpu"):
        g = torch.Generator().manual_seed(seed)
        self.E, self.N, self.K, self.fmt = E, N, K, fmt
        lo, hi = (0x28, 0x50) if lo is None and fmt == "nvfp4" else (118, 124) if lo is None else (lo, hi)
        self.packed = torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.uint8)
        self.scales = torch.randint(lo, hi, (E, N, K // BLOCK[fmt]), generator=g, dtype=torch.uint8)
        self.gscale = (0.01 + 0.05 * torch.rand(E, generator=g)).float() if fmt == "nvfp4" else None

    def values(self, e):
        codes = torch.stack([self.packed[e] & 15, self.packed[e] >> 4], dim=-1).flatten(1).long()
        v = E2M1[codes & 7] * torch.where(codes >= 8, -1.0, 1.0)
        s = self.scales[e]
        if self.fmt == "nvfp4":
            exp, man = (s >> 3).double(), (s & 7).double()
            s = torch.where(s < 8, man * 2.0 ** -9, (1 + man / 8) * torch.exp2(exp - 7))
        else:
            s = torch.exp2(s.double() - 127)
        v = v * s.repeat_interleave(BLOCK[self.fmt], dim=1)
        return v if self.gscale is None else v * self.gscale[e].double()

    def blocked(self):
        E, N, S = self.scales.shape
        return self.scales.view(E, N // 128, 4, 32, S // 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(E, -1).contiguous()


def product(x, w, block=32):
    """x [T, K] and w [N, K] float64: (y, the kernel's error before its rounding)."""
    K = x.shape[1]
    size = x.abs() @ w.abs().T
    pad = torch.nn.functional.pad(x.abs(), (0, -K % block)).view(x.shape[0], -1, block).amax(2)
    wsum = torch.nn.functional.pad(w.abs(), (0, -K % block)).view(w.shape[0], -1, block).sum(2)
    rows = x.abs().amax(1, keepdim=True) * 2.0 ** -34
    return x @ w.T, K * 2.0 ** -23 * size + (2.0 ** -18 * pad + rows) @ wsum.T


def experts(x, idx, topk_w, gu, d, dtype=torch.bfloat16):
    """(out, tolerance) [T, H] of the expert layer after the router; ids out of range contribute nothing."""
    T, H = x.shape
    out, tol = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    size = torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for j, e in enumerate(idx[t].tolist()):
            if not 0 <= e < gu.E:
                continue
            w = float(topk_w[t, j])
            z, ez = product(x[t:t + 1].double(), gu.values(e))
            (gate, up), (eg, eu) = z.chunk(2, dim=1), ez.chunk(2, dim=1)
            s = gate * torch.sigmoid(gate)
            h = s * up
            eh = 1.1 * eg * up.abs() + s.abs() * eu + 1.1 * eg * eu + (2.0 ** -11 + 2.0 ** -20) * h.abs()
            wd = d.values(e)
            y, ey = product(h, wd)
            out[t] += w * y[0]
            tol[t] += abs(w) * (ey + (1 + 2.0 ** -10) * eh @ wd.abs().T)[0]
            size[t] += abs(w) * (h.abs() @ wd.abs().T)[0]
    n = idx.shape[1] + 8
    return out, tol + n * 2.0 ** -23 * size + half_step(dtype) * (out.abs() + tol) + 1e-38


def check(got, ref, tol, what=""):
    err = (got.double().cpu() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / tol).nan_to_num(1e9).max()):.2f} x its bound"


def route(logits, bias, k, score_fn, renorm, n_group, topk_group, group_best, scale, kept=None):
    """One token: (indices, weights) in float64 by repeated search.  `kept` takes other groups than the best: of those that
    float64 cannot tell apart (groups_that_tie)."""
    v = [(-float("inf") if x != x else min(x, 3.4028234663852886e38)) for x in logits.double().tolist()]
    t = torch.tensor(v, dtype=torch.float64)
    if score_fn == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-t))
    else:
        top = t.max()
        s = torch.exp(t - top) if top > -float("inf") else torch.zeros_like(t)
        s = s / s.sum() if float(s.sum()) > 0 else s
    order = t if bias is None and (n_group == 1 or group_best == 1) else s.clone()
    if bias is not None:
        b = bias.double()
        b = torch.where(torch.isnan(b), torch.tensor(-float("inf"), dtype=torch.float64), b).clamp(max=3.4028234663852886e38)
        order = s + b
    c = order.tolist()
    E, per = len(c), len(c) // n_group
    value = []
    for g in range(n_group):
        part = sorted(c[g * per:(g + 1) * per], reverse=True)
        value.append(part[0] + (part[1] if group_best == 2 and n_group > 1 else 0.0))
    if kept is None:
        kept = sorted(range(n_group), key=lambda g: (-value[g], g))[:topk_group]
    elif kept == "values":
        return value, s.tolist(), c
    cand = sorted((e for e in range(E) if e // per in kept), key=lambda e: (-c[e], e))[:k]
    w = s[cand]
    if renorm:
        w = w / w.sum() if float(w.sum()) > 0 else torch.zeros_like(w)
    return cand, (w * scale).tolist()


def groups_that_tie(logits, bias, k, score_fn, renorm, n_group, topk_group, group_best, scale):
    """Every choice of groups that float64 allows.  A group's value is the sum of two c = s + b: three roundings of 2^-53 of
    the parts, and s is itself off, a sigmoid by 4 such steps (exp, sum, quotient), a softmax by that and the E - 1 additions
    of its sum in whatever order.  Values that differ by less than both sides' errors (1 and 2: sums such as (s + 3) + (z - 2)
    and (s + 1) + z are equal but round apart) may go either way."""
    value, s, c = route(logits, bias, k, score_fn, renorm, n_group, topk_group, group_best, scale, kept="values")
    E, size = len(c), 2.0 * max(abs(x) for x in c if abs(x) < float("inf")) if any(abs(x) < float("inf") for x in c) else 0.0
    off = 2.0 ** -53 * (2.0 * (4 + (E if score_fn == "softmax" else 0)) * max(s) + 3.0 * size)
    edge = sorted(value, reverse=True)[topk_group - 1]
    inside = [g for g in range(n_group) if value[g] > edge + 2 * off]
    near = [g for g in range(n_group) if abs(value[g] - edge) <= 2 * off]
    return [inside + list(some) for some in itertools.combinations(near, topk_group - len(inside))] if len(near) <= 12 else []


def plan(past, new, tables, free_pages, count, page, T):
    """The page plan of one step in plain Python: a dict of lists; tables is changed."""
    max_pages = len(tables[0]) if tables else 0
    count = min(max(count, 0), len(free_pages))
    asked, left, at = 0, count, 0
    out = dict(positions=[0] * T, slots=[-1] * T, cu_seqlens=[0], seq_lens=[], granted=[])
    for b, (p, n) in enumerate(zip(past, new)):
        p, n = max(p, 0), max(n, 0)
        held, after = -(-p // page), -(-(p + n) // page)
        ok = after <= max_pages and at + n <= T
        if ok and after > held:
            asked += after - held
            ok = asked <= count
            for c in range(held, after if ok else held):
                left -= 1
                tables[b][c] = free_pages[left]
        for i in range(n):
            if at + i < T:
                out["positions"][at + i] = min(p + i, 2 ** 31 - 1)
                if ok and tables[b][(p + i) // page] >= 0:
                    out["slots"][at + i] = tables[b][(p + i) // page] * page + (p + i) % page
        at += n
        out["cu_seqlens"].append(min(at, T))
        out["seq_lens"].append(p + n if ok else p)
        out["granted"].append(n if ok else 0)
    out["free_count"] = [left]
    return out
