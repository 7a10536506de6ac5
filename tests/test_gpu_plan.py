"""mla_plan on the GPU against its definition: pages, slots, offsets, refusals."""
import pytest
import torch

from . import few_reference as R

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module")
def M():
    from nvfp4_block_scaled_07_gb300 import build
    build.build()
    from nvfp4_block_scaled_07_gb300 import mla
    mla.sync_status()
    return mla


def case(past, new, page, free, extra_cols=1, seed=0, T=None):
    """Tables with the held pages filled in, in a random order, and `free` free ones."""
    g = torch.Generator().manual_seed(seed)
    held = [-(-p // page) for p in past]
    cols = max([-(-(p + n) // page) for p, n in zip(past, new)] + [0]) + extra_cols
    ids = torch.randperm(sum(held) + free, generator=g).tolist()
    tables = []
    for h in held:
        tables.append(ids[:h] + [-1] * (cols - h))
        ids = ids[h:]
    return dict(past=past, new=new, tables=tables, free=ids, page=page, T=sum(new) + 5 if T is None else T)


def check(M, c, count=None, bad=False, in_place=False, strided=False, num_free=None):
    B, cols = len(c["past"]), len(c["tables"][0]) if c["tables"] else 0
    room = torch.full((B, cols + 3), -9, **I32)
    tables = room[:, :cols] if strided else torch.empty(B, cols, **I32)
    if B:
        tables.copy_(torch.tensor(c["tables"], dtype=torch.int32).view(B, cols))
    n = len(c["free"]) if count is None else count
    free_count = torch.tensor([n], **I32)
    out = M.alloc_token_plan(B, c["T"], "cuda", free_count if in_place else None)
    for t in (out.positions, out.slots, out.seq_lens, out.granted, out.cu_seqlens):
        t.fill_(77)
    free = torch.tensor(c["free"], **I32)
    p = M.mla_plan(torch.tensor(c["past"], **I32), torch.tensor(c["new"], **I32), tables, free, free_count, c["page"], c["T"],
                   out=out)
    if bad:
        with pytest.raises(M.Nvfp4MoeError) as e:
            M.sync_status()
        assert e.value.status == 7
    M.sync_status()
    want_tables = [list(r) for r in c["tables"]]
    want = R.plan(c["past"], c["new"], want_tables, c["free"], n, c["page"], c["T"])
    for name, value in want.items():
        assert getattr(p, name).tolist() == value, name
    assert tables.tolist() == want_tables
    assert (room[:, cols:] == -9).all() and free.tolist() == c["free"]
    assert in_place or free_count.item() == n
    return p


@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("past,new", [
    ([0], [1]), ([63], [1]), ([64], [1]), ([65], [0]), ([0], [300]), ([0, 0, 0], [0, 0, 0]), ([127, 128, 129, 0], [1, 1, 1, 1]),
    ([5, 600, 0, 33, 64], [3, 0, 200, 31, 64]), ([10000], [1000])])
def test_plan(M, page, past, new):
    check(M, case(past, new, page, free=100))
    check(M, case(past, new, page, free=100, extra_cols=0, T=sum(new)), in_place=True, strided=True)


@pytest.mark.parametrize("B,most,page", [(700, 3, 16), (1024, 2, 16), (1025, 2, 64), (3000, 1, 32), (40, 900, 64), (2500, 9, 16)])
@pytest.mark.parametrize("share", [0.0, 0.5, 1.0, 2.0])
def test_plan_of_many_requests(M, B, most, page, share):
    """One block's pieces and two kernels; all, half and none of the pages that are missing."""
    g = torch.Generator().manual_seed(B)
    past = torch.randint(0, 500, (B,), generator=g).tolist()
    new = torch.randint(0, most + 1, (B,), generator=g).tolist()
    need = sum(-(-(p + n) // page) - -(-p // page) for p, n in zip(past, new))
    check(M, case(past, new, page, free=int(share * need) + 1, seed=B))


def test_plan_refuses_whole_requests(M):
    """Pages that end within a request, tables that are too short, rows that end within a request."""
    c = case([0, 0, 16, 0, 10], [33, 40, 1, 16, 2], 16, free=4)
    p = check(M, c)
    assert p.granted.tolist() == [33, 0, 0, 0, 2] and p.free_count.item() == 1
    c = case([0, 100, 8], [20, 60, 8], 16, free=40)
    for row in c["tables"]:
        del row[7:]
    assert check(M, c).granted.tolist() == [20, 0, 8]
    c = case([0, 100, 8], [20, 60, 8], 16, free=40, T=50)
    assert check(M, c, bad=True).granted.tolist() == [20, 0, 0]
    c = case([3, 9], [1, 2], 16, free=3, T=0)
    assert check(M, c, bad=True).granted.tolist() == [0, 0]


def test_plan_of_bad_data(M):
    """Negative lengths count as 0, a count outside the list as its end, table entries below 0 give no slot."""
    check(M, case([0, 20], [1, 1], 16, free=5) | dict(past=[-4, 20]), bad=True)
    check(M, case([0, 20], [1, 1], 16, free=5) | dict(new=[1, -3]), bad=True)
    check(M, case([0, 20], [1, 1], 16, free=5), count=9, bad=True)
    check(M, case([0, 20], [1, 1], 16, free=5), count=-1, bad=True)
    c = case([20, 20], [1, 1], 16, free=5)
    c["tables"][0][1] = -1
    assert check(M, c).slots.tolist()[0] == -1
    c = case([0], [4], 16, free=5)
    c |= dict(past=[2 ** 31 - 2])
    assert check(M, c).granted.tolist() == [0]


def test_plan_of_nothing(M):
    check(M, case([], [], 16, free=3, T=4))
    check(M, case([], [], 16, free=0, T=0))
    check(M, case([5], [1], 16, free=0))
    c = case([0], [1], 16, free=2)
    c["tables"] = [[]]
    assert check(M, c).granted.tolist() == [0]


@pytest.mark.parametrize("T", [8191, 8192, 8193, 70000])
def test_plan_rows_past_the_last_token(M, T):
    check(M, case([7, 0, 100], [1000, 3000, 4000], 64, free=200, T=T), bad=T < 8000)


def test_steps_in_a_graph(M):
    """Captured with the count in place: each replay takes further pages, the lengths come from the last one."""
    page, B = 16, 3
    past, new = torch.tensor([14, 0, 31], **I32), torch.ones(B, **I32)
    tables = torch.tensor([[9, -1, -1, -1], [-1, -1, -1, -1], [4, 7, -1, -1]], **I32)
    free, count = torch.tensor([0, 1, 2, 3, 5, 6, 8], **I32), torch.tensor([7], **I32)
    out = M.alloc_token_plan(B, 4, "cuda", count)

    def step():
        M.mla_plan(past, new, tables, free, count, page, 4, out=out)
        past.copy_(out.seq_lens)

    start = (past.clone(), tables.clone(), count.clone())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    for t, s in zip((past, tables, count), start):
        t.copy_(s)
    lens, want, left = [14, 0, 31], start[1].tolist(), 7
    for _ in range(20):
        graph.replay()
        ref = R.plan(lens, [1] * B, want, free.tolist(), left, page, 4)
        assert out.slots.tolist() == ref["slots"] and tables.tolist() == want and count.tolist() == ref["free_count"]
        lens, left = ref["seq_lens"], ref["free_count"][0]
        assert past.tolist() == lens
    M.sync_status()
