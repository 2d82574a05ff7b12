"""GPU check of the step plan against the oracle: whole numbers, equal in every entry."""
import numpy as np
import pytest
import torch

from oracle.attention import plan_step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ssd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from selective_state_space_04_gb300 import build
    build.build()
    from selective_state_space_04_gb300 import ssd as mod
    return mod


def make(seed, n, ps, cols, longest, newest, free, done=0.1, extra=0):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, longest + 1, n)
    new = rng.integers(0, newest + 1, n)
    new[rng.random(n) < done] = -1
    held = -(-lens // ps)
    cap = int(held.sum()) + free + extra
    ids = rng.permutation(cap)
    table = np.full((n, cols), -1)
    at = 0
    for r in range(n):
        table[r, :held[r]] = ids[at:at + held[r]]
        at += held[r]
    head = int(rng.integers(0, 4 * max(cap, 1)))
    ring = np.full(max(cap, 1), -5)
    ring[(head + np.arange(free)) % max(cap, 1)] = ids[at:at + free]
    return dict(lens=lens, new=new, table=table, ring=ring, pos=np.array([head, head + free]))


def run(ssd, c, ps, room, in_place=False, out=None):
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).cuda()  # noqa: E731
    lens, new, table, ring, pos = i32(c["lens"]), i32(c["new"]), i32(c["table"]), i32(c["ring"]), torch.from_numpy(c["pos"]).cuda()
    if in_place:
        n = len(c["lens"])
        out = dict(lens=lens, granted=i32(np.zeros(n)), start=i32(np.zeros(n + 1)), positions=i32(np.zeros(room)),
                   token_req=i32(np.zeros(room)), slots=torch.zeros(room, dtype=torch.int64, device="cuda"), ring_pos=pos,
                   counts=i32(np.zeros(4)))
    got = ssd.paged_plan(lens, new, table, ring, pos, page_size=ps, max_tokens=room, out=out)
    torch.cuda.synchronize()
    return dict(got, table=table, ring=ring)


def check(got, c, ps, room):
    ref = plan_step(c["lens"], c["new"], c["table"], c["ring"], c["pos"], ps, room)
    for k in ref:
        assert np.array_equal(got[k].cpu().numpy(), ref[k]), k
    return ref


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n,ps,cols,longest,newest,free,room", [
    (1, 16, 4, 20, 5, 3, 8),
    (1, 1, 30, 20, 5, 8, 5),
    (7, 16, 8, 100, 20, 12, 140),
    (128, 16, 40, 500, 1, 40, 128),
    (128, 16, 40, 500, 1, 3, 128),          # the pages run out
    (128, 16, 40, 500, 30, 400, 500),       # the rows run out
    (1000, 7, 30, 150, 40, 6000, 30000),
    (1025, 24, 5, 119, 40, 2500, 30001),    # some do not fit their tables
    (3000, 1, 60, 50, 12, 30000, 20000),
    (8192, 128, 2, 200, 3, 900, 9000),
])
def test_against_oracle(ssd, n, ps, cols, longest, newest, free, room, in_place):
    c = make(n + ps, n, ps, cols, longest, newest, free)
    check(run(ssd, c, ps, room, in_place), c, ps, room)


def test_long_prompts(ssd):
    c = make(3, 40, 32, 2000, 9000, 1, 8000)
    c["new"][::9] = 30000
    ref = check(run(ssd, c, 32, 150016), c, 32, 150016)
    assert ref["counts"][0] > 100000


@pytest.mark.parametrize("what", ["all finished", "nothing new", "no room", "no pages"])
def test_edges(ssd, what):
    c = make(4, 300, 16, 40, 500, 9, 900)
    room = 4000
    if what == "all finished":
        c["new"][:] = -1
    elif what == "nothing new":
        c["new"][:] = 0
    elif what == "no room":
        room = 0
    else:
        c["pos"][1] = c["pos"][0]
    check(run(ssd, c, 16, room), c, 16, room)


def test_no_requests(ssd):
    c = dict(lens=np.zeros(0), new=np.zeros(0), table=np.zeros((0, 4)), ring=np.arange(6), pos=np.array([2, 5]))
    got = run(ssd, c, 16, 10)
    assert got["start"].tolist() == [0] and (got["positions"] == -1).all() and (got["slots"] == -1).all()
    assert got["ring_pos"].tolist() == [2, 5] and got["counts"].tolist() == [0, 0, 0, 0]


def test_lengths_near_the_limit(ssd):
    # page_size * max_pages just under 2^31: sums and roundings must not overflow
    ps, cols = 2 ** 20, 2047
    c = dict(lens=np.array([ps * cols - 3, ps * cols - 2, ps * cols]), new=np.array([3, 3, 0]), table=np.arange(3 * cols).reshape(3, -1),
             ring=np.arange(8), pos=np.array([5, 9]))
    got = run(ssd, c, ps, 16)
    assert got["granted"].tolist() == [3, 0, 0] and got["counts"].tolist() == [3, 0, 0, 1]
    check(got, c, ps, 16)


def test_many_steps(ssd):
    # a server's life: every step's result feeds the next, in place
    rng = np.random.default_rng(9)
    n, ps, cap, room = 37, 8, 200, 90
    c = dict(lens=np.zeros(n, dtype=int), new=None, table=np.full((n, 12), -1), ring=rng.permutation(cap), pos=np.array([0, cap]))
    for _ in range(40):
        c["new"] = rng.integers(-1, 25, n)
        got = run(ssd, c, ps, room, in_place=True)
        ref = check(got, c, ps, room)
        c = dict(lens=ref["lens"], table=ref["table"], ring=ref["ring"], pos=ref["ring_pos"])


def test_refusals(ssd):
    c = make(5, 8, 16, 8, 100, 4, 20)
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).cuda()  # noqa: E731
    ok = dict(lens=i32(c["lens"]), new_lens=i32(c["new"]), block_table=i32(c["table"]), free_ring=i32(c["ring"]),
              ring_pos=torch.from_numpy(c["pos"]).cuda(), page_size=16, max_tokens=64)
    for bad in (dict(lens=ok["lens"].long()), dict(new_lens=ok["new_lens"][:3]), dict(block_table=ok["block_table"].t()),
                dict(ring_pos=ok["ring_pos"].int()), dict(page_size=0), dict(page_size=2 ** 30), dict(new_lens=ok["lens"].cpu()),
                dict(lens=i32(np.zeros(9000)), new_lens=i32(np.zeros(9000)), block_table=i32(np.zeros((9000, 1)))),
                dict(free_ring=ok["block_table"].view(-1))):
        with pytest.raises((ValueError, ssd.SsdError)):
            ssd.paged_plan(**dict(ok, **bad))
