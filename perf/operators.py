"""Latent attention next to the expert layer: the three operators of its path, their plain forms and the cases
that are timed.

A layer with latent attention keeps one shared vector a token, 512 latent values and 64 rotated ones, in a paged
cache that every query head reads:

  append   normalises the latent part, rotates the rotary part of the key and of the queries, writes the cache
  decode   the absorbed form: queries of 576 values against the cached vectors themselves, values are the
           first 512 of each, a few new tokens a sequence, the cache read through block tables
  prefill  the expanded form: keys of 128 + 64 values and values of 128 for each head, ragged batches, causal

`own` chooses between the plain form (False) and the framework's calls (True).
"""
import math
import random

import torch

own = False

LATENT, ROPE, NOPE, VDIM = 512, 64, 128, 128
ROW = LATENT + ROPE          # one cached token
QK = NOPE + ROPE             # one expanded key or query
SCALE = QK ** -0.5
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # one user's next token: the latency of a call
        dict(name="append_token", op="append", T=1, H=16, page=64, span=4096, interleaved=True, dtype="bf16"),
        # the decode batch of 128 sequences, one token each
        dict(name="append_t128", op="append", T=128, H=64, page=64, span=8192, interleaved=False, dtype="fp16"),
        # the prompt tokens of a prefill step
        dict(name="append_t16384", op="append", T=16384, H=16, page=64, span=16384, interleaved=True, dtype="bf16"),
        # one user, the beginning of an answer, small pages: the latency of a call
        dict(name="decode_one", op="decode", B=1, Sq=1, H=16, lo=37, hi=37, page=16, dtype="bf16"),
        # a serving batch whose heads are spread over several GPUs
        dict(name="decode_b128_h16", op="decode", B=128, Sq=1, H=16, lo=300, hi=4100, page=32, dtype="bf16"),
        # a middling batch with all of 64 heads
        dict(name="decode_b32_h64", op="decode", B=32, Sq=1, H=64, lo=1000, hi=8191, page=64, dtype="fp16"),
        # the large serving batch, 128 heads
        dict(name="decode_b128_h128", op="decode", B=128, Sq=1, H=128, lo=2048, hi=8192, page=64, dtype="bf16"),
        # two users with very long contexts, and two tokens a step to verify
        dict(name="decode_long", op="decode", B=2, Sq=2, H=64, lo=100001, hi=131072, page=64, dtype="bf16"),
        # a question of a few words
        dict(name="prefill_short", op="prefill", B=1, H=16, qlo=19, qhi=19, past=0, dtype="bf16"),
        # prompts of several users in one batch, all lengths odd
        dict(name="prefill_ragged", op="prefill", B=7, H=16, qlo=101, qhi=2500, past=0, dtype="bf16"),
        # the next chunk of two long prompts
        dict(name="prefill_chunk", op="prefill", B=2, H=32, qlo=1000, qhi=1024, past=7001, dtype="fp16"),
        # one long document
        dict(name="prefill_t16384", op="prefill", B=1, H=16, qlo=16384, qhi=16384, past=0, dtype="bf16"),
    ]


def draw(rng):
    def spread(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    dtype = rng.choice(["bf16", "bf16", "fp16"])
    op = rng.choice(["append", "decode", "decode", "prefill"])
    if op == "append":
        return dict(op=op, T=spread(1, 16384), H=rng.choice([1, 5, 8, 16]), page=rng.choice([16, 32, 64, 128]),
                    span=spread(1024, 16384), interleaved=rng.random() < 0.5, dtype=dtype)
    if op == "decode":
        B, H, Sq = spread(1, 128), rng.choice([1, 7, 8, 16, 32, 40, 64, 96, 128]), rng.choice([1, 1, 2, 3, 4])
        most = max(64, min(131072, 128 * 4096 // B, 128 * 128 * 4096 // (B * H * Sq)))
        hi = spread(1, most)
        return dict(op=op, B=B, Sq=Sq, H=H, lo=max(1, hi // rng.choice([1, 2, 10])), hi=hi,
                    page=rng.choice([16, 32, 64, 128]), dtype=dtype)
    B, H = spread(1, 16), rng.choice([1, 3, 8, 16, 24])
    hi = spread(1, 8192 // B)
    return dict(op=op, B=B, H=H, qlo=max(1, hi // rng.choice([1, 3, 20])), qhi=hi,
                past=rng.choice([0, 0, spread(1, 4096)]), dtype=dtype)


def _lengths(case):
    """The case's sequence lengths: (queries, keys) of each sequence.  They go by the case alone."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    if case["op"] == "decode":
        keys = [rng.randint(case["lo"], case["hi"]) for _ in range(case["B"])]
        keys[-1] = case["hi"]
        return [case["Sq"]] * case["B"], [max(k, case["Sq"]) for k in keys]
    queries = [rng.randint(case["qlo"], case["qhi"]) for _ in range(case["B"])]
    queries[-1] = case["qhi"]
    return queries, [q + (rng.randint(case["past"] // 2, case["past"]) if case["past"] else 0) for q in queries]


def _pages(total, page, g):
    """A random order of `total` cache pages: the allocator's, after a while."""
    return torch.randperm(total, generator=g, device="cuda").to(torch.int32)


def _table(span):
    """cos | sin of the 32 angles of each position, in float32, from 64-bit angles."""
    inv = 10000.0 ** (-torch.arange(0, ROPE, 2, dtype=torch.float64, device="cuda") / ROPE)
    ang = torch.arange(span, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], dim=1).to(torch.float32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dt)

    s = dict(op=case["op"])
    if case["op"] == "append":
        T, H, page, span = case["T"], case["H"], case["page"], case["span"]
        n_pages = -(-T // page) + 3
        kv = normal(T, ROW, std=2.0)
        q = normal(T, H, QK)
        # tokens take scattered slots; in a batch of more than 8 the last one is padding, without a slot
        slots = torch.randperm(n_pages * page, generator=g, device="cuda")[:T]
        if T > 8:
            slots[-1] = -1
        s.update(latent=kv[:, :LATENT], k_rope=kv[:, LATENT:], q_rope=q[..., NOPE:],
                 norm_weight=(1 + 0.1 * torch.randn(LATENT, generator=g, device="cuda")).to(dt),
                 positions=torch.randint(0, span, (T,), generator=g, device="cuda", dtype=torch.int32), slots=slots,
                 table=_table(span), cache=normal(n_pages, page, ROW), q=normal(T, H, ROW),
                 rows=torch.empty(T, ROW, device="cuda", dtype=dt), interleaved=case["interleaved"])
    elif case["op"] == "decode":
        _, keys = _lengths(case)
        B, page = case["B"], case["page"]
        need = [-(-n // page) for n in keys]
        order = _pages(sum(need) + 5, page, g)
        table = torch.full((B, max(need)), -1, device="cuda", dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        cache = torch.empty(sum(need) + 5, page, ROW, device="cuda", dtype=dt)
        for i in range(0, cache.shape[0], 4096):
            cache[i:i + 4096] = normal(*cache[i:i + 4096].shape)
        s.update(q=normal(B, case["Sq"], case["H"], ROW), cache=cache, block_tables=table, longest=max(keys),
                 seq_lens=torch.tensor(keys, device="cuda", dtype=torch.int32))
    else:
        queries, keys = _lengths(case)
        H, Tk = case["H"], sum(keys)
        up = normal(Tk, H, NOPE + VDIM)
        s.update(q=normal(sum(queries), H, QK), k_nope=up[..., :NOPE], v=up[..., NOPE:],
                 k_rope=normal(Tk, ROW)[:, LATENT:], max_q=max(queries), max_k=max(keys),
                 cu_q=torch.tensor([0] + queries, device="cuda").cumsum(0).to(torch.int32),
                 cu_k=torch.tensor([0] + keys, device="cuda").cumsum(0).to(torch.int32))
    return s


# ---- plain forms ---------------------------------------------------------------------------------------------
def _rotate(x, cos, sin, interleaved):
    """Rotates the 32 pairs of the last dimension: neighbours, or values 32 apart."""
    pairs = x.unflatten(-1, (ROPE // 2, 2)) if interleaved else x.unflatten(-1, (2, ROPE // 2)).transpose(-1, -2)
    a, b = pairs[..., 0], pairs[..., 1]
    r = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return (r if interleaved else r.transpose(-1, -2)).flatten(-2)


def _append(s):
    lat = s["latent"].float()
    lat = lat * torch.rsqrt((lat * lat).mean(dim=-1, keepdim=True) + EPS) * s["norm_weight"].float()
    cs = s["table"][s["positions"].long()]
    cos, sin = cs[:, :ROPE // 2], cs[:, ROPE // 2:]
    rows = torch.cat([lat, _rotate(s["k_rope"].float(), cos, sin, s["interleaved"])], dim=-1).to(s["cache"].dtype)
    s["rows"].copy_(rows)
    kept = s["slots"] >= 0
    s["cache"].view(-1, ROW)[s["slots"][kept]] = rows[kept]
    s["q"][..., LATENT:] = _rotate(s["q_rope"].float(), cos[:, None], sin[:, None], s["interleaved"]).to(s["q"].dtype)
    return dict(cache=s["cache"], rows=s["rows"], q=s["q"])


def _softmax(scores, seen):
    """(weights, log of the sum) over the last dimension; a row that sees nothing has weights of zero."""
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(dim=-1, keepdim=True)
    p = torch.exp(scores - top.masked_fill(top == -math.inf, 0.0))
    total = p.sum(dim=-1, keepdim=True)
    return p / total.masked_fill(total == 0, 1.0), (top + torch.log(total)).squeeze(-1)


def _decode(s):
    q, lens, page = s["q"], s["seq_lens"].long(), s["cache"].shape[1]
    B, Sq, H, _ = q.shape
    at = torch.arange(s["longest"], device=q.device)
    inside = at < lens[:, None]
    pages = s["block_tables"].long()[:, at // page].clamp(min=0)
    kv = s["cache"].view(-1, ROW)[pages * page + at % page].float()
    scores = (q.float().flatten(1, 2) @ kv.transpose(1, 2) * SCALE).unflatten(1, (Sq, H))
    last = lens[:, None] - Sq + torch.arange(Sq, device=q.device)
    p, lse = _softmax(scores, (inside[:, None] & (at <= last[..., None]))[:, :, None])
    out = (p.flatten(1, 2) @ kv[..., :LATENT]).unflatten(1, (Sq, H))
    return dict(out=out.to(q.dtype), lse=lse)


def _prefill(s):
    q, cu_q, cu_k = s["q"], s["cu_q"].long(), s["cu_k"].long()
    nq, nk = cu_q.diff(), cu_k.diff()
    iq, ik = torch.arange(s["max_q"], device=q.device), torch.arange(s["max_k"], device=q.device)
    at_q = (cu_q[:-1, None] + iq).clamp(max=q.shape[0] - 1)
    at_k = (cu_k[:-1, None] + ik).clamp(max=s["v"].shape[0] - 1)
    k = torch.cat([s["k_nope"], s["k_rope"][:, None].expand(-1, q.shape[1], -1)], dim=-1)
    scores = q[at_q].float().transpose(1, 2) @ k[at_k].float().permute(0, 2, 3, 1) * SCALE
    seen = (ik < nk[:, None])[:, None] & (ik <= (nk - nq)[:, None, None] + iq[:, None])
    p, lse = _softmax(scores, seen[:, None])
    out = (p @ s["v"][at_k].float().transpose(1, 2)).transpose(1, 2)
    t = torch.arange(q.shape[0], device=q.device)
    b = torch.searchsorted(cu_q, t, right=True) - 1
    return dict(out=out[b, t - cu_q[b]].to(q.dtype), lse=lse.transpose(1, 2)[b, t - cu_q[b]].contiguous())


def run(state):
    s = state
    if own:
        from nvfp4_block_scaled_07_gb300 import mla as B
        if s["op"] == "append":
            B.mla_append(s["latent"], s["k_rope"], s["positions"], s["slots"], s["table"], s["cache"],
                         norm_weight=s["norm_weight"], eps=EPS, interleaved=s["interleaved"], q_rope=s["q_rope"],
                         q_out=s["q"][..., LATENT:], rows_out=s["rows"])
            return dict(cache=s["cache"], rows=s["rows"], q=s["q"])
        if s["op"] == "decode":
            out, lse = B.mla_decode(s["q"], s["cache"], s["block_tables"], s["seq_lens"], SCALE)
        else:
            out, lse = B.mla_prefill(s["q"], s["k_nope"], s["k_rope"], s["v"], s["cu_q"], s["cu_k"], SCALE)
        return dict(out=out, lse=lse)
    return {"append": _append, "decode": _decode, "prefill": _prefill}[s["op"]](s)


def work(case):
    H = case["H"]
    if case["op"] == "append":
        T, span = case["T"], case["span"]
        # kv in, the cached row and its copy out, the rotary part of each head in and out, the angles (a position's
        # only once), slots and positions
        return {"bytes": T * (3 * ROW * 2 + H * ROPE * 4 + 12) + min(T, span) * ROPE * 4 + LATENT * 2,
                "flops": T * (4 * LATENT + 3 * ROPE * (H + 1))}
    queries, keys = _lengths(case)
    # query i of a sequence sees keys - queries + i + 1 keys
    pairs = sum(q * (k - q) + q * (q + 1) // 2 for q, k in zip(queries, keys))
    if case["op"] == "decode":
        rows = case["B"] * case["Sq"] * H
        return {"bytes": sum(keys) * ROW * 2 + rows * ((ROW + LATENT) * 2 + 4)
                + 4 * (case["B"] + sum(-(-k // case["page"]) for k in keys)), "flops": 2 * H * pairs * (ROW + LATENT)}
    return {"bytes": 2 * H * (sum(queries) * (QK + VDIM + 2) + sum(keys) * (NOPE + VDIM)) + sum(keys) * ROPE * 2
            + 8 * (case["B"] + 1), "flops": 2 * H * pairs * (QK + VDIM)}


# ---- the definitions in 64 bits ------------------------------------------------------------------------------
def _attend64(q, k, v, offset):
    """Row i of q sees keys 0 .. offset + i: (out, lse), in pieces of rows."""
    n, m = q.shape[0], k.shape[0]
    out = torch.zeros(n, v.shape[1], dtype=torch.float64, device=q.device)
    lse = torch.full((n,), -math.inf, dtype=torch.float64, device=q.device)
    for i in range(0, n, 2048):
        j = min(n, i + 2048)
        sees = min(m, offset + j)
        if sees <= 0:
            continue
        x = q[i:j] @ k[:sees].T * SCALE
        hidden = torch.arange(sees, device=q.device) > offset + torch.arange(i, j, device=q.device)[:, None]
        x[hidden] = -math.inf
        lse[i:j] = torch.logsumexp(x, dim=1)
        x = torch.exp(x - lse[i:j, None])
        out[i:j] = torch.nan_to_num(x) @ v[:sees]
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        x = s["latent"].double()
        norm = (x.square().sum(1) / LATENT + EPS).sqrt()
        x = x / norm[:, None] * s["norm_weight"].double()
        turn = torch.complex(*s["table"].double()[s["positions"].long()].split(ROPE // 2, dim=1))

        def rotated(r):
            r = r.double()
            z = torch.complex(r[..., 0::2], r[..., 1::2]) if case["interleaved"] else torch.complex(*r.split(ROPE // 2, dim=-1))
            z = z * (turn if r.dim() == 2 else turn[:, None])
            return torch.view_as_real(z).flatten(-2) if case["interleaved"] else torch.cat([z.real, z.imag], dim=-1)

        rows = torch.cat([x, rotated(s["k_rope"])], dim=1)
        cache = s["cache"].double().reshape(-1, ROW)
        for t, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                cache[slot] = rows[t]
        q = s["q"].double()
        q[..., LATENT:] = rotated(s["q_rope"])
        return dict(cache=cache.view(s["cache"].shape), rows=rows, q=q)
    queries, keys = _lengths(case)
    H = case["H"]
    outs, lses = [], []
    at_q = at_k = 0
    for b, (n, m) in enumerate(zip(queries, keys)):
        if case["op"] == "decode":
            page = case["page"]
            ids = s["block_tables"][b, :-(-m // page)].long()
            kv = s["cache"][ids].reshape(-1, ROW)[:m].double()
            x = s["q"][b].double().flatten(0, 1) @ kv.T * SCALE
            hidden = torch.arange(m, device=x.device) > m - n + torch.arange(n, device=x.device)[:, None]
            x[hidden.repeat_interleave(H, dim=0)] = -math.inf
            lse = torch.logsumexp(x, dim=1)
            outs.append((torch.exp(x - lse[:, None]) @ kv[:, :LATENT]).view(n, H, LATENT))
            lses.append(lse.view(n, H))
            continue
        kr = s["k_rope"][at_k:at_k + m].double()
        heads = [_attend64(s["q"][at_q:at_q + n, h].double(),
                           torch.cat([s["k_nope"][at_k:at_k + m, h].double(), kr], dim=1),
                           s["v"][at_k:at_k + m, h].double(), m - n) for h in range(H)]
        outs.append(torch.stack([o for o, _ in heads], dim=1))
        lses.append(torch.stack([e for _, e in heads], dim=1))
        at_q, at_k = at_q + n, at_k + m
    if case["op"] == "decode":
        return dict(out=torch.stack(outs), lse=torch.stack(lses))
    return dict(out=torch.cat(outs), lse=torch.cat(lses))
