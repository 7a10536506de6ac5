"""mla_plan in place (lengths, grants and the count of free pages updated where they are), and at the ends of its ranges."""
import pytest
import torch

from . import few_reference as R
from .test_gpu_plan import I32, M, case, check  # noqa: F401  (M is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,most,page", [(1, 1, 16), (5, 40, 16), (700, 3, 16), (40, 900, 64), (300, 30, 64), (2000, 70, 128)])
@pytest.mark.parametrize("share", [0.6, 1.5])
def test_plan_in_place(M, B, most, page, share):  # noqa: F811
    """seq_lens into past_lens, granted into new_lens, the count into itself: with one kernel and with two."""
    g = torch.Generator().manual_seed(B)
    past = torch.randint(0, 500, (B,), generator=g).tolist()
    new = torch.randint(1, most + 1, (B,), generator=g).tolist()
    if B > 3:
        past[2] = -5
        new[3] = 0
    need = sum(-(-(max(p, 0) + n) // page) - -(-max(p, 0) // page) for p, n in zip(past, new))
    c = case([max(p, 0) for p in past], new, page, free=int(share * need) + 1, seed=B, T=sum(new) + 3) | dict(past=past)
    lens, fresh = torch.tensor(past, **I32), torch.tensor(new, **I32)
    tables, free, count = torch.tensor(c["tables"], **I32), torch.tensor(c["free"], **I32), torch.tensor([len(c["free"])], **I32)
    out = M.alloc_token_plan(B, c["T"], "cuda", count)
    out.seq_lens, out.granted = lens, fresh
    M.mla_plan(lens, fresh, tables, free, count, page, c["T"], out=out)
    if B > 3:
        with pytest.raises(M.Nvfp4MoeError) as e:
            M.sync_status()
        assert e.value.status == 7
    M.sync_status()
    want_tables = [list(r) for r in c["tables"]]
    want = R.plan(past, new, want_tables, c["free"], len(c["free"]), page, c["T"])
    for name, value in want.items():
        assert getattr(out, name).tolist() == value, name
    assert tables.tolist() == want_tables


def test_plan_refuses_outputs_that_overlap(M):  # noqa: F811
    B, T = 4, 16
    buf = torch.zeros(64, **I32)
    tables, free, count = torch.full((B, 4), -1, **I32), torch.arange(8, **I32), torch.tensor([8], **I32)
    lens, new = buf[:4], torch.ones(4, **I32)
    for name, part in (("seq_lens", buf[1:5]), ("granted", buf[3:7]), ("cu_seqlens", buf[2:7]), ("positions", buf[:16]),
                       ("free_count", buf[:1]), ("free_count", free[:1]), ("granted", tables[1])):
        out = M.alloc_token_plan(B, T, "cuda")
        setattr(out, name, part)
        with pytest.raises(M.Nvfp4MoeError) as e:
            M.mla_plan(lens, new, tables, free, count, 16, T, out=out)
        assert e.value.status == 1 and "overlaps" in str(e.value)
    assert (buf == 0).all() and (tables == -1).all() and count.item() == 8
    M.sync_status()


def test_steps_of_several_tokens_in_a_graph_in_place(M):  # noqa: F811
    """A replayed step whose lengths are its own input: 200 requests of seven tokens, two kernels."""
    page, B, n = 16, 200, 7
    g = torch.Generator().manual_seed(2)
    lens0 = torch.randint(0, 40, (B,), generator=g).tolist()
    c = case(lens0, [60] * B, page, free=600, seed=1)
    lens, new = torch.tensor(lens0, **I32), torch.full((B,), n, **I32)
    tables, free, count = torch.tensor(c["tables"], **I32), torch.tensor(c["free"], **I32), torch.tensor([600], **I32)
    T = B * n + 300
    out = M.alloc_token_plan(B, T, "cuda", count)
    out.seq_lens = lens
    start = [t.clone() for t in (lens, tables, count)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        M.mla_plan(lens, new, tables, free, count, page, T, out=out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            M.mla_plan(lens, new, tables, free, count, page, T, out=out)
    torch.cuda.current_stream().wait_stream(side)
    for t, s in zip((lens, tables, count), start):
        t.copy_(s)
    now, want, left = lens0, [list(r) for r in c["tables"]], 600
    for _ in range(6):
        graph.replay()
        ref = R.plan(now, [n] * B, want, c["free"], left, page, T)
        assert out.slots.tolist() == ref["slots"] and out.positions.tolist() == ref["positions"]
        assert tables.tolist() == want and count.tolist() == ref["free_count"]
        now, left = ref["seq_lens"], ref["free_count"][0]
        assert lens.tolist() == now
    M.sync_status()


@pytest.mark.parametrize("new", [1, 2, 3, 12, 3000])
def test_plan_of_the_longest_requests(M, new):  # noqa: F811
    """Lengths up to 2^31 - 1, in large pages; a request that would pass that is refused, the others go on."""
    page, top = 1 << 20, 2 ** 31 - 1
    past = [top - 2, 5, top - new, top, top - 1]
    tables = torch.full((5, 2049), -1, **I32)
    tables[:, :2048] = torch.arange(2048, **I32)
    tables[1] = -1
    tables[1, 0] = 7
    want_tables = tables.tolist()
    free, T = list(range(3000, 3010)), 5 * new + 2
    p = M.mla_plan(torch.tensor(past, **I32), torch.full((5,), new, **I32), tables, torch.tensor(free, **I32),
                   torch.tensor([10], **I32), page, T)
    M.sync_status()
    granted = [new if q + new <= top else 0 for q in past]
    assert p.granted.tolist() == granted and p.granted.tolist()[1:4] == [new, new, 0]
    assert p.seq_lens.tolist() == [q + n for q, n in zip(past, granted)]
    assert p.cu_seqlens.tolist() == [i * new for i in range(6)] and p.free_count.item() == 10
    slots, positions = p.slots.tolist(), p.positions.tolist()
    for b, q in enumerate(past):
        for i in range(0, new, max(1, new // 5)):
            t, at = b * new + i, q + i
            assert positions[t] == min(at, top)
            assert slots[t] == ((7 if b == 1 else at // page) * page + at % page if granted[b] else -1)
    assert slots[-2:] == [-1, -1] and tables.tolist() == want_tables


BORDER = 1 << 20          # rows and free pages up to which tokens and pages share one scan


def many(c, num_free, count):
    """The case with a free list of num_free pages, of which the first `count` are free."""
    own = c["free"][:count]
    return c | dict(free=own + list(range(10 ** 7, 10 ** 7 + num_free - len(own)))), len(own)


@pytest.mark.parametrize("num_free,T", [(BORDER - 1, 40), (BORDER, 40), (BORDER + 1, 40), (9, BORDER), (9, BORDER + 1), (9, BORDER + 3000),
                                        (BORDER + 1, BORDER + 1)])
@pytest.mark.parametrize("kind", ["few", "many tokens", "many requests", "refused"])
def test_plan_around_the_border_of_one_scan(M, num_free, T, kind):  # noqa: F811
    """Few valid requests among many free pages or padded rows, on both sides of the border."""
    if kind == "few":
        c, bad = case([14, 0, 31, 16], [3, 1, 0, 8], 16, free=9), False
    elif kind == "many tokens":               # a request of more tokens than its thread writes by itself
        c, bad = case([14, 0, 31], [20, 2, 17], 16, free=9), False
    elif kind == "many requests":             # several pieces
        new = [1] * 30 + [0] * 2000 + [1] * 9
        c, bad = case([15 + i % 3 for i in range(len(new))], new, 16, free=9), False
    else:                                     # tokens past the rows
        c, bad = case([14, 0, 31, 5], [3, T, 2, 1], 16, free=9), True
        for row in c["tables"]:
            del row[4:]
    c, count = many(c | dict(T=T), num_free, 9)
    check(M, c, count=count, bad=bad)


@pytest.mark.parametrize("free", [0, 3, 19, 20, 21])
def test_plan_of_a_request_that_misses_more_than_all_pages(M, free):  # noqa: F811
    """Those after it that miss none go on; the others miss what it asked for too."""
    for tail in ([1, 2], [1] * 40):
        past = [0, 20, 16] + [17] * len(tail)
        p = check(M, case(past, [320, 5, 1] + tail, 16, free=free))
        assert p.granted.tolist()[0] == (320 if free >= 20 else 0) and p.granted.tolist()[1] == 5
        assert p.granted.tolist()[2] == (1 if free >= 21 else 0) and p.granted.tolist()[3:] == tail
