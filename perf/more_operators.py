"""A decode step of few tokens: the operators around the expert layer and the latent cache, their plain forms and the
cases that are timed.

  route    scores of the experts, a bias that only selects, groups of experts, the best k, renormalised and scaled weights
  matvec   y = x W^T for a few rows x of 16 bits and a matrix of 4-bit codes with a scale for each 16 or 32 of them
  experts  the chosen experts' gated products of a few tokens with such matrices, and their weighted sum
  plan     block tables, slots, positions and offsets of a step's new tokens, from the requests' lengths and the free pages

`own` chooses between the plain form (False) and the framework's calls (True).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
BLOCK = {"nvfp4": 16, "mxfp4": 32}                        # elements that share a scale
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one user's next token: the latency of a call
        dict(name="route_token", op="route", T=1, E=256, k=8, groups=8, keep=4, best=2, score="sigmoid", bias=True,
             renorm=True, scale=2.5),
        # a batch of a layer with few experts, without groups and without a bias
        dict(name="route_t1000", op="route", T=1000, E=64, k=6, groups=1, keep=1, best=1, score="softmax", bias=False,
             renorm=False, scale=1.0),
        # the tokens of a prefill step
        dict(name="route_t16384", op="route", T=16384, E=256, k=8, groups=8, keep=4, best=2, score="sigmoid", bias=True,
             renorm=True, scale=2.5),
        # one token through a small projection: the latency of a call
        dict(name="matvec_small", op="matvec", T=1, N=512, K=2048, fmt="nvfp4", dtype="bf16", tiled=False),
        # five tokens to verify, through a wide projection
        dict(name="matvec_t5", op="matvec", T=5, N=6144, K=8192, fmt="mxfp4", dtype="fp16", tiled=True),
        # a full batch of small requests through the largest matrix
        dict(name="matvec_t32", op="matvec", T=32, N=32768, K=7168, fmt="nvfp4", dtype="bf16", tiled=True),
        # three tokens of a tiny layer: the latency of a call
        dict(name="experts_tiny", op="experts", T=3, E=8, k=2, H=256, I=128, fmt="nvfp4", tiled=False),
        # one user's next token through the decode layer
        dict(name="experts_token", op="experts", T=1, E=256, k=8, H=6144, I=2048, fmt="nvfp4", tiled=True),
        # an odd small batch through wide experts, most of them hit
        dict(name="experts_t23", op="experts", T=23, E=64, k=8, H=7168, I=4096, fmt="mxfp4", tiled=True),
        # one user's next token
        dict(name="plan_one", op="plan", B=1, past=1023, new=1, page=64, room=1.5),
        # the decode step of a large batch, up to three tokens each, not enough free pages for all
        dict(name="plan_b700", op="plan", B=700, past=5000, new=3, page=16, room=0.9),
        # prompts of several users
        dict(name="plan_prefill", op="plan", B=37, past=3000, new=7000, page=64, room=1.2),
    ]


def draw(rng):
    def spread(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["route", "matvec", "experts", "plan"])
    if op == "route":
        E = rng.choice([8, 40, 64, 128, 160, 256, 384, 512])
        groups = rng.choice([g for g in (1, 1, 2, 4, 8) if E // g >= 2])
        keep = rng.randint(1, groups)
        return dict(op=op, T=min(spread(1, 16384), 16384 * 256 // E), E=E, k=rng.randint(1, min(8, keep * (E // groups))),
                    groups=groups, keep=keep, best=rng.choice([1, 2]), score=rng.choice(["sigmoid", "sigmoid", "softmax"]),
                    bias=rng.random() < 0.7, renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]))
    fmt = rng.choice(["nvfp4", "nvfp4", "mxfp4"])
    step = 64 if fmt == "nvfp4" else 128
    if op == "matvec":
        N = spread(1, 256) * 128
        K = min(spread(128, 16384), 32768 * 7168 // N) // step * step
        return dict(op=op, T=spread(1, 32), N=N, K=K, fmt=fmt, dtype=rng.choice(["bf16", "fp16"]), tiled=rng.random() < 0.5)
    if op == "experts":
        E = rng.choice([4, 8, 16, 32, 64, 128, 256])
        H, I = spread(2, 56) * 128, spread(1, 32) * 128
        while E * H * I > 64 * 7168 * 4096:
            E //= 2
        return dict(op=op, T=spread(1, 23), E=E, k=rng.randint(1, min(8, E)), H=H, I=I, fmt=fmt, tiled=rng.random() < 0.7)
    B = spread(1, 2048)
    new = rng.choice([1, 1, 4, spread(1, 130000 // B)])
    return dict(op=op, B=B, past=rng.choice([0, spread(1, 100000 // B + 100)]), new=new, page=rng.choice([16, 32, 64, 128]),
                room=rng.choice([0.5, 1.0, 1.5]))


# ---- inputs ----------------------------------------------------------------------------------------------------
def _quantise(w, fmt):
    """float32 [rows, K] -> (packed codes [rows, K/2], scale bytes [rows, K/block], per-tensor scale)."""
    rows, K = w.shape
    b = w.view(rows, -1, BLOCK[fmt])
    top = b.abs().amax(-1)
    if fmt == "nvfp4":
        tensor = w.abs().amax() / 2688.0
        sb = (top / 6.0 / tensor).to(torch.float8_e4m3fn)
        step = sb.float() * tensor
    else:
        tensor = torch.ones((), device=w.device)
        exponent = (torch.floor(torch.log2(top.clamp(min=1e-30))) - 2).clamp(-127, 127)
        sb = (exponent + 127).to(torch.uint8)
        step = torch.exp2(exponent)
    q = b / step.clamp(min=1e-30)[..., None]
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
    code = torch.bucketize(q.abs(), borders).to(torch.uint8) | ((q < 0).to(torch.uint8) << 3)
    code = code.view(rows, K)
    return code[:, 0::2] | (code[:, 1::2] << 4), sb.view(torch.uint8), tensor


def _blocked(scales, fmt):
    """Row-major scale bytes [E, N, K/block] -> the blocked layout: 128 rows x 4 scales in 512 bytes, row r's four
    at (r % 32) * 16 + (r / 32) * 4."""
    E, N, S = scales.shape
    return scales.view(E, N // 128, 4, 32, S // 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(E, -1)


def _tiled(packed):
    """Packed codes [rows, K/2] -> boxes of 128 rows x 128 bytes, bytes past K/2 zero."""
    rows, half = packed.shape
    wide = -(-half // 128) * 128
    if wide != half:
        packed = torch.nn.functional.pad(packed, (0, wide - half))
    return packed.view(rows // 128, 128, wide // 128, 128).transpose(1, 2).reshape(-1)


def _matrices(case, E, N, K, g):
    """E matrices of quantised normal values, whose rows are drawn from 1024 quantised ones, as a program keeps them:
    the codes row by row or tiled, the scales row by row (plain form) and blocked (the framework's), scales of the tensors."""
    fmt = case["fmt"]
    codes, scales, tensor = _quantise(torch.randn((1024, K), generator=g, device="cuda") * 0.02, fmt)
    packed = torch.empty((E, N, K // 2), dtype=torch.uint8, device="cuda")
    rows = torch.empty((E, N, K // BLOCK[fmt]), dtype=torch.uint8, device="cuda")
    for e in range(E):
        pick = torch.randint(0, 1024, (N,), generator=g, device="cuda")
        packed[e], rows[e] = codes[pick], scales[pick]
    each = tensor * (0.75 + 0.5 * torch.rand(E, generator=g, device="cuda")) if fmt == "nvfp4" else None
    return dict(packed=packed, scales=rows, gscale=each, blocked=_blocked(rows, fmt), N=N, K=K, E=E, fmt=fmt,
                tiled=_tiled(packed.view(E * N, -1)) if case["tiled"] else None)


def _capacity(case):
    return -(-(case["B"] * case["new"] + 1) // 8) * 8


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    if case["op"] == "route":
        T, E = case["T"], case["E"]
        s.update(logits=torch.randn((T, E), generator=g, device="cuda") * 1.5,
                 select_bias=0.1 * torch.randn(E, generator=g, device="cuda") if case["bias"] else None)
    elif case["op"] == "matvec":
        s.update(x=torch.randn((case["T"], case["K"]), generator=g, device="cuda").to(DTYPES[case["dtype"]]),
                 w=_matrices(case, 1, case["N"], case["K"], g))
    elif case["op"] == "experts":
        T, E, k = case["T"], case["E"], case["k"]
        scores = torch.sigmoid(torch.randn((T, E), generator=g, device="cuda"))
        top = scores.topk(k, dim=1)
        s.update(x=torch.randn((T, case["H"]), generator=g, device="cuda").to(torch.bfloat16),
                 topk_idx=top.indices.to(torch.int32), topk_w=(top.values / top.values.sum(1, keepdim=True)).contiguous(),
                 w_gu=_matrices(case, E, 2 * case["I"], case["H"], g), w_d=_matrices(case, E, case["H"], case["I"], g))
    else:
        B, page = case["B"], case["page"]
        past = torch.randint(case["past"] // 2, case["past"] + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        new = torch.randint((case["new"] + 1) // 2, case["new"] + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        held, after = -(-past // page), -(-(past + new) // page)
        used = int(held.sum())
        free = max(1, int(case["room"] * int((after - held).sum())))
        order = torch.randperm(used + free, generator=g, device="cuda").to(torch.int32)
        tables = torch.full((B, -(-(case["past"] + case["new"]) // page) + 2), -1, dtype=torch.int32, device="cuda")
        tables[torch.arange(tables.shape[1], device="cuda") < held[:, None]] = order[:used]
        # the batch's buffers have room for the most tokens that a step can have
        s.update(past_lens=past, new_lens=new, tables=tables, free_pages=order[used:].contiguous(),
                 free_count=torch.full((1,), free, dtype=torch.int32, device="cuda"), tokens=_capacity(case))
    return s


# ---- plain forms -----------------------------------------------------------------------------------------------
def _route(s):
    T, E = s["logits"].shape
    v = s["logits"].double()                              # scores next to a border decide which expert is taken
    if s["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-v))
    else:
        score = torch.exp(v - v.amax(1, keepdim=True))
        score = score / score.sum(1, keepdim=True)
    c = score if s["select_bias"] is None else score + s["select_bias"].double()
    if s["groups"] > 1:
        parts = c.view(T, s["groups"], -1)
        value = parts.sort(dim=2, descending=True).values[..., :s["best"]].sum(2)
        kept = value.sort(dim=1, descending=True, stable=True).indices[:, :s["keep"]]
        mask = torch.zeros_like(value, dtype=torch.bool).scatter_(1, kept, True)
        c = parts.masked_fill(~mask[..., None], -math.inf).view(T, E)
    idx = c.sort(dim=1, descending=True, stable=True).indices[:, :s["k"]]
    w = score.gather(1, idx)
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return dict(topk_idx=idx.to(torch.int32), topk_w=(w * s["scale"]).float())


def _values(w, at):
    """The matrix `at` (a device index) of w as float32 values, without the tensor's scale."""
    packed, sb = w["packed"].index_select(0, at)[0], w["scales"].index_select(0, at)[0].to(torch.int32)
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=packed.device)
    pair = torch.stack([table[(packed & 15).int()], table[(packed >> 4).int()]], dim=-1)
    if w["fmt"] == "nvfp4":
        e, m = sb >> 3, (sb & 7).float()
        step = torch.where(e == 0, m * 2.0 ** -9, (8.0 + m) * torch.exp2((e - 10).float()))
    else:
        step = torch.exp2((sb - 127).float())
    return (pair.view(w["N"], -1, BLOCK[w["fmt"]]) * step[..., None]).view(w["N"], w["K"])


def _scale(w, at):
    return 1.0 if w["gscale"] is None else w["gscale"].index_select(0, at)


def _matvec(s):
    first = torch.zeros(1, dtype=torch.int64, device=s["x"].device)
    return (s["x"].float() @ _values(s["w"], first).T * _scale(s["w"], first)).to(s["x"].dtype)


def _experts(s):
    x, gu, d = s["x"].float(), s["w_gu"], s["w_d"]
    T, k, I = s["T"], s["k"], s["I"]

    def expert(at, rows):
        z = rows @ _values(gu, at).T * _scale(gu, at)
        gate, up = z[:, :I], z[:, I:]
        return gate / (1.0 + torch.exp(-gate)) * up @ _values(d, at).T * _scale(d, at)

    out = torch.zeros((T, s["H"]), device=x.device)
    if T * k <= s["E"]:                                   # routed row by routed row
        for t in range(T):
            for j in range(k):
                out[t] += s["topk_w"][t, j] * expert(s["topk_idx"][t, j:j + 1].long(), x[t:t + 1])[0]
    else:                                                 # expert by expert
        for e in range(s["E"]):
            coef = (s["topk_w"] * (s["topk_idx"] == e)).sum(1, keepdim=True)
            out += torch.where(coef != 0, coef * expert(torch.full((1,), e, device=x.device), x), 0.0)
    return out.to(s["x"].dtype)


def _plan(s):
    past, new, page, tables = s["past_lens"].long(), s["new_lens"].long(), s["page"], s["tables"]
    held, after = (past + page - 1) // page, (past + new + page - 1) // page
    fits = after <= tables.shape[1]
    need = torch.where(fits, after - held, 0)
    upto = need.cumsum(0)
    ok = fits & ((need == 0) | (upto <= s["free_count"]))
    given = torch.where(ok, need, 0)
    # the i-th new page of request b is the (upto[b] - need[b] + i)-th popped from the end of the free pages
    col = torch.arange(tables.shape[1], device=past.device)
    fresh = ok[:, None] & (col >= held[:, None]) & (col < after[:, None])
    popped = (upto - need)[:, None] + col - held[:, None]
    at = (s["free_count"].long() - 1 - popped).clamp(0, s["free_pages"].numel() - 1)
    tables.copy_(torch.where(fresh, s["free_pages"][at], tables))
    cu = torch.cat([torch.zeros_like(new[:1]), new.cumsum(0)])
    t = torch.arange(s["tokens"], device=past.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    real = b < new.numel()
    b = b.clamp(max=new.numel() - 1)
    position = torch.where(real, past[b] + t - cu[b], 0)
    where = tables[b, (position // page).clamp(max=tables.shape[1] - 1)].long()
    slots = torch.where(real & ok[b] & (where >= 0), where * page + position % page, -1)
    return dict(positions=position.int(), slots=slots, cu_seqlens=cu.int(),
                seq_lens=torch.where(ok, past + new, past).int(), granted=torch.where(ok, new, 0).int(),
                free_count=(s["free_count"] - given.sum()).int(), tables=tables)


def _codes(B, w):
    return w["packed"] if w["tiled"] is None else B.TiledWeights(w["tiled"], w["E"], w["N"], w["K"])


def run(state):
    s = state
    if not own:
        return {"route": _route, "matvec": _matvec, "experts": _experts, "plan": _plan}[s["op"]](s)
    from nvfp4_block_scaled_07_gb300 import binding as B
    if s["op"] == "route":
        idx, w = B.moe_route_grouped(s["logits"], s["k"], s["score"], s["renorm"], select_bias=s["select_bias"],
                                     n_group=s["groups"], topk_group=s["keep"], group_best=s["best"], scale=s["scale"])
        return dict(topk_idx=idx, topk_w=w)
    if s["op"] == "matvec":
        w = s["w"]
        if w["fmt"] == "nvfp4":
            return B.moe_matvec_nvfp4(s["x"], _codes(B, w), w["blocked"], w["gscale"])
        return B.moe_matvec_mxfp4(s["x"], _codes(B, w), w["blocked"])
    if s["op"] == "experts":
        gu, d = s["w_gu"], s["w_d"]
        if gu["fmt"] == "nvfp4":
            return B.moe_experts_nvfp4(s["x"], s["topk_idx"], s["topk_w"], _codes(B, gu), gu["blocked"], gu["gscale"],
                                       _codes(B, d), d["blocked"], d["gscale"])
        return B.moe_experts_mxfp4(s["x"], s["topk_idx"], s["topk_w"], _codes(B, gu), gu["blocked"], _codes(B, d),
                                   d["blocked"])
    from nvfp4_block_scaled_07_gb300 import mla
    p = mla.mla_plan(s["past_lens"], s["new_lens"], s["tables"], s["free_pages"], s["free_count"], s["page"], s["tokens"])
    return dict(positions=p.positions, slots=p.slots, cu_seqlens=p.cu_seqlens, seq_lens=p.seq_lens, granted=p.granted,
                free_count=p.free_count, tables=s["tables"])


def work(case):
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * (4 * E + 8 * k) + 4 * E * case["bias"], "flops": 4 * T * E}
    if case["op"] == "plan":
        B, page = case["B"], case["page"]
        new = B * (case["new"] + (case["new"] + 1) // 2) // 2             # on average
        pages = max(1, new // page)
        return {"bytes": 12 * _capacity(case) + 20 * B + 4 + 8 * pages + 8, "flops": 4 * new}
    each = 0.5 + 1.0 / BLOCK[case["fmt"]]                                 # bytes of a weight with its share of a scale
    T = case["T"]
    if case["op"] == "matvec":
        N, K = case["N"], case["K"]
        return {"bytes": int(N * K * each) + 2 * T * (N + K), "flops": 2 * T * N * K}
    E, k, H, I = case["E"], case["k"], case["H"], case["I"]
    hit = E * (1.0 - (1.0 - k / E) ** T)                                  # distinct experts, on average
    return {"bytes": int(hit * 3 * H * I * each) + 4 * T * H + 8 * T * k, "flops": 6 * T * k * H * I}


# ---- the definitions in 64 bits --------------------------------------------------------------------------------
def _decoded(w, e):
    """Matrix e of w in float64, by the formats' own types."""
    low, high = w["packed"][e] & 0xF, w["packed"][e] >> 4
    code = torch.stack([low, high], dim=2).flatten(1).long()
    mag = code & 7
    value = torch.where(mag < 2, mag * 0.5, (2 + (mag & 1)).double() * 2.0 ** ((mag >> 1) - 2).double())
    value = torch.where(code >= 8, -value, value)
    sb = w["scales"][e]
    step = sb.view(torch.float8_e4m3fn).double() if w["fmt"] == "nvfp4" else torch.ldexp(
        torch.ones_like(sb, dtype=torch.float64), sb.double() - 127)
    value = value * step.repeat_interleave(BLOCK[w["fmt"]], dim=1)
    return value if w["gscale"] is None else value * w["gscale"][e].double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "matvec":
        return s["x"].double() @ _decoded(s["w"], 0).T
    if case["op"] == "experts":
        out = torch.zeros((case["T"], case["H"]), dtype=torch.float64, device="cuda")
        chosen = s["topk_idx"].tolist()
        for e in sorted({e for row in chosen for e in row}):
            rows = [t for t, row in enumerate(chosen) if e in row]
            gate, up = (s["x"][rows].double() @ _decoded(s["w_gu"], e).T).split(case["I"], dim=1)
            y = torch.nn.functional.silu(gate) * up @ _decoded(s["w_d"], e).T
            for i, t in enumerate(rows):
                out[t] += s["topk_w"][t, chosen[t].index(e)].double() * y[i]
        return out
    if case["op"] == "route":
        v = s["logits"].double()
        score = torch.sigmoid(v) if case["score"] == "sigmoid" else torch.softmax(v, dim=1)
        c = score.clone() if s["select_bias"] is None else score + s["select_bias"].double()
        if case["groups"] > 1:
            per = case["E"] // case["groups"]
            left = torch.stack([part.topk(case["best"], dim=1).values.sum(1) for part in c.split(per, dim=1)], dim=1)
            keep = torch.zeros_like(left, dtype=torch.bool)
            for _ in range(case["keep"]):
                top = (left == left.amax(1, keepdim=True)).int().argmax(1, keepdim=True)      # the lowest of equals
                keep.scatter_(1, top, True)
                left.scatter_(1, top, -math.inf)
            c[~keep.repeat_interleave(per, dim=1)] = -math.inf
        picks = []
        for _ in range(case["k"]):
            top = (c == c.amax(1, keepdim=True)).int().argmax(1, keepdim=True)
            picks.append(top)
            c.scatter_(1, top, -math.inf)
        idx = torch.cat(picks, dim=1)
        w = score.gather(1, idx)
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True)
        return dict(topk_idx=idx.to(torch.int32), topk_w=w * case["scale"])
    past, new, free = s["past_lens"].tolist(), s["new_lens"].tolist(), s["free_pages"].tolist()
    page, tables = case["page"], s["tables"].tolist()
    left, asked = len(free), 0
    positions, slots, cu, lens, granted = [], [], [0], [], []
    for b, (p, n) in enumerate(zip(past, new)):
        held, after = -(-p // page), -(-(p + n) // page)
        ok = after <= len(tables[b])
        if ok:
            asked += after - held
            ok = after == held or asked <= len(free)
        if ok:
            for c in range(held, after):
                left -= 1
                tables[b][c] = free[left]
        positions += range(p, p + n)
        slots += [tables[b][q // page] * page + q % page if ok else -1 for q in range(p, p + n)]
        cu.append(cu[-1] + n)
        lens.append(p + n if ok else p)
        granted.append(n if ok else 0)
    pad = s["tokens"] - len(positions)

    def ints(values, dtype=torch.int32):
        return torch.tensor(values, dtype=dtype, device="cuda")

    return dict(positions=ints(positions + [0] * pad), slots=ints(slots + [-1] * pad, torch.int64), cu_seqlens=ints(cu),
                seq_lens=ints(lens), granted=ints(granted), free_count=ints([left]), tables=ints(tables))
