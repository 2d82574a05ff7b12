"""GPU parity of attention over the paged cache against the fp64 oracle.

Tolerance, per element, from the arithmetic (A = sum_t p_t |v_t|):
* out: its one rounding (2^-8 |ref| for bf16, 2^-22 |ref| for fp32, twice the
  half-ulp) + c A, with c the relative error of the weights p.  A score's error
  is at most the accumulation's: D products of magnitude below 4, in fp32, so
  below 2^-13 for D <= 256; the same bound holds for p (e^x - 1 ~ x), and it
  covers two-term bf16 weights (2^-17) and two-term tf32 products (2^-21 of
  sum |q k| scale, below 2^-15).
* lse: 2^-13 + 2^-22 |ref|.
Whatever a row does not see holds NaN here.
"""
import numpy as np
import pytest
import torch

from oracle.attention import paged_attention

pytestmark = pytest.mark.gpu

C = 2.0 ** -13
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -22}
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ssd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from selective_state_space_04_gb300 import build
    build.build()
    from selective_state_space_04_gb300 import ssd as mod
    return mod


def make(seed, lens, new, H, hk, D, ps, dtype, layout="nhd", table_cols=None, spare=3):
    """Requests of ``lens`` cached tokens, the last ``new[r]`` of them query rows (None: one row each, no start).  All
    other cache contents are NaN, table entries past a request's pages are out of range."""
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens)
    held = -(-lens // ps)
    npages = int(held.sum()) + spare
    cols = max(1, int(held.max(initial=0))) + 1 if table_cols is None else table_cols
    table = np.full((len(lens), cols), npages + 5, dtype=np.int32)
    table[:, 1::2] = -7
    ids = rng.permutation(npages)[:held.sum()]
    at = 0
    shape = {"nhd": (npages, ps, hk, D), "hnd": (npages, hk, ps, D), "kv": (npages, 2, ps, hk, D)}[layout]
    both = [torch.full(shape, float("nan"), dtype=dtype)] * 1
    kc = both[0]
    vc = torch.full(shape, float("nan"), dtype=dtype)
    if layout == "kv":
        kc, vc = kc[:, 0], kc[:, 1]
    elif layout == "hnd":
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    for r, n in enumerate(lens):
        table[r, :held[r]] = ids[at:at + held[r]]
        at += held[r]
        t = np.arange(n)
        page = torch.from_numpy(table[r, t // ps].astype(np.int64))
        for c in (kc, vc):
            c[page, torch.from_numpy(t % ps)] = torch.from_numpy(rng.standard_normal((n, hk, D)).astype(np.float32)).to(dtype)
    if new is None:
        start, pos = None, lens - 1
    else:
        start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        pos = np.concatenate([np.arange(n - m, n) for n, m in zip(lens, new)] + [np.zeros(0)])
    rows = len(pos)
    q = torch.from_numpy((1.5 * rng.standard_normal((rows, H, D))).astype(np.float32)).to(dtype)
    return dict(q=q, kc=kc, vc=vc, table=torch.from_numpy(table), pos=torch.from_numpy(np.asarray(pos, dtype=np.int32)),
                start=None if start is None else torch.from_numpy(start))


def to_gpu(x):
    """Keeps strides (views of one buffer need not stay in one)."""
    if x is None:
        return None
    y = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda")
    y.copy_(x)
    return y


def run(ssd, c, **kw):
    out, lse = ssd.paged_attn_fwd(*(to_gpu(c[k]) for k in ("q", "kc", "vc", "table", "pos", "start")), **kw)
    torch.cuda.synchronize()
    return out, lse


def check(out, lse, c, scale=None, window=0, rows=slice(None)):
    D = c["q"].shape[2]
    ref, rlse, size = paged_attention(c["q"], c["kc"], c["vc"], c["table"], c["pos"], c["start"],
                                      D ** -0.5 if scale is None else scale, window)
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    bad = np.abs(got - ref) - (ROUND[out.dtype] * np.abs(ref) + C * size)
    assert bad.max(initial=-1) <= 0, f"out off by {bad.max()} over its bound"
    got = lse.double().cpu().numpy()
    empty = np.isneginf(rlse)
    assert np.array_equal(np.isneginf(got), empty)
    assert (np.abs(got[~empty] - rlse[~empty]) <= C + 2.0 ** -22 * np.abs(rlse[~empty])).all()
    assert (out.double().cpu().numpy()[empty] == 0).all()


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("lens,H,hk,D,ps,layout", [
    ([1], 1, 1, 64, 16, "nhd"),
    ([1, 2, 15, 16, 17, 31, 33, 64, 65], 4, 1, 64, 16, "nhd"),
    ([100, 1, 700], 8, 2, 128, 16, "hnd"),
    ([63, 640, 5], 6, 2, 80, 24, "kv"),          # a head size and a page that fit no tile
    ([129, 300], 20, 4, 96, 1, "nhd"),           # pages of one token
    ([77, 1030], 16, 1, 128, 128, "hnd"),        # one key head for all
    ([50, 333], 40, 1, 64, 64, "nhd"),           # more query heads per key head than a tile has rows
    ([90, 500], 2, 2, 256, 32, "kv"),
    ([41, 222], 3, 1, 8, 7, "nhd"),
    ([41, 222], 10, 2, 200, 20, "hnd"),
    ([4000], 2, 1, 192, 48, "nhd"),
])
def test_one_token_each(ssd, dtype, lens, H, hk, D, ps, layout):
    c = make(11, lens, None, H, hk, D, ps, dtype, layout)
    check(*run(ssd, c), c)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("lens,H,hk,D,ps", [
    ([30000] + [3] * 160, 4, 2, 64, 16),      # one long request among many short ones: cut into many parts
    ([20] * 150 + [9000, 1] + [33] * 9, 8, 4, 128, 24),
    ([300, 41], 1300, 1300, 8, 16),           # more heads than the GPU has warps
    ([90, 17, 5], 700, 350, 64, 16),
    ([2, 40, 18] * 70, 32, 1, 128, 16),
])
def test_uneven_work(ssd, dtype, lens, H, hk, D, ps):
    c = make(27, lens, None, H, hk, D, ps, dtype)
    check(*run(ssd, c), c)


@pytest.mark.parametrize("scale", [-0.7, 0.0, 1e-3])
@pytest.mark.parametrize("dtype", [BF, F])
def test_any_scale(ssd, dtype, scale):
    c = make(28, [50, 200], None, 4, 2, 64, 16, dtype)
    check(*run(ssd, c, scale=scale), c, scale=scale)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("lens,new,H,hk,D,ps", [
    ([40, 9, 300], [4, 9, 1], 8, 2, 128, 16),
    ([40, 9, 300, 17], [0, 5, 0, 17], 6, 2, 64, 8),     # requests that bring nothing; whole prompts
    ([260], [200], 4, 1, 64, 16),
    ([70, 71], [3, 40], 24, 1, 128, 24),
    ([70, 33], [6, 2], 5, 5, 256, 24),
])
@pytest.mark.parametrize("window", [0, 1, 7, 50])
def test_several_tokens_each(ssd, dtype, lens, new, H, hk, D, ps, window):
    c = make(12, lens, new, H, hk, D, ps, dtype)
    check(*run(ssd, c, window=window), c, window=window)


@pytest.mark.parametrize("window", [1, 15, 16, 17, 100, 5000])
def test_window_over_one_token(ssd, window):
    c = make(13, [1, 16, 40, 1000], None, 8, 2, 128, 24, BF)
    check(*run(ssd, c, window=window), c, window=window)


@pytest.mark.parametrize("dtype", [BF, F])
def test_rows_that_see_nothing(ssd, dtype):
    c = make(14, [20, 0, 33, 0], None, 4, 2, 64, 16, dtype)
    assert c["pos"].tolist() == [19, -1, 32, -1]
    out, lse = run(ssd, c)
    check(out, lse, c)
    # padding rows past start[nreq], and a request whose table names no page
    c = make(15, [20, 30], [3, 2], 4, 2, 64, 16, dtype)
    q = torch.cat([c["q"], torch.full((4, 4, 64), float("nan"), dtype=dtype)])
    c = dict(c, q=q, pos=torch.cat([c["pos"], torch.full((4,), 7, dtype=torch.int32)]))
    c["table"][1] = -1
    out, lse = run(ssd, c)
    assert (out[3:] == 0).all() and torch.isneginf(lse[3:]).all()
    c["q"] = torch.nan_to_num(c["q"])
    check(out, lse, c)


def test_padding_only_with_more_heads_than_warps(ssd):
    # a step without tokens leaves every share empty, those after a warp's first one too: nothing of a used workspace
    # may be taken for parts (here: one part, of row 1, in each entry)
    c = make(29, [20, 30], [0, 0], 1300, 1300, 8, 16, BF)
    c = dict(c, q=torch.ones(3, 1300, 8, dtype=BF), pos=torch.full((3,), 7, dtype=torch.int32))
    g = {k: to_gpu(c[k]) for k in ("q", "kc", "vc", "table")}
    ws = torch.ones(ssd.paged_attn_workspace_size(*g.values()) // 4, dtype=torch.int32, device="cuda")
    out, lse = run(ssd, c, workspace=ws)
    assert (out == 0).all() and torch.isneginf(lse).all()


def test_no_rows_and_no_requests(ssd):
    c = make(16, [8], None, 4, 2, 64, 16, BF)
    out, lse = ssd.paged_attn_fwd(torch.empty(0, 4, 64, dtype=BF, device="cuda"), to_gpu(c["kc"]), to_gpu(c["vc"]),
                                  torch.empty(0, 3, dtype=torch.int32, device="cuda"),
                                  torch.empty(0, dtype=torch.int32, device="cuda"))
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    # rows, but no request: all padding
    out, lse = ssd.paged_attn_fwd(to_gpu(c["q"]), to_gpu(c["kc"]), to_gpu(c["vc"]),
                                  torch.empty(0, 3, dtype=torch.int32, device="cuda"), to_gpu(c["pos"]),
                                  torch.zeros(1, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert (out == 0).all() and torch.isneginf(lse).all()


def test_missing_page_inside_a_request(ssd):
    # a table entry out of range hides its tokens, and only those
    c = make(17, [200], None, 4, 2, 64, 16, BF)
    c["table"][0, 3], c["table"][0, 9] = -1, c["kc"].shape[0]
    check(*run(ssd, c), c)


def test_position_past_the_table(ssd):
    c = make(18, [64], None, 4, 2, 64, 16, BF, table_cols=4)
    c["pos"] = torch.tensor([2 ** 31 - 1], dtype=torch.int32)
    check(*run(ssd, c), c)


@pytest.mark.parametrize("dtype", [BF, F])
def test_large_scores(ssd, dtype):
    # scores of hundreds, rising along the row: the running maximum moves all the time
    c = make(19, [300, 45], None, 4, 2, 64, 16, dtype)
    c["kc"] *= torch.linspace(0.1, 3.0, 16)[None, :, None, None].to(dtype)
    D = 64
    out, lse = run(ssd, c, scale=4.0)
    ref, rlse, size = paged_attention(c["q"], c["kc"], c["vc"], c["table"], c["pos"], None, 4.0, 0)
    # products reach 64 * 4 * |q k| ~ 3000: the scores' fp32 error, and so the weights', grows in proportion
    rel = 2.0 ** -22 * 4.0 * np.sqrt(D) * 8 * float(c["q"].abs().max()) * 12
    got = out.double().cpu().numpy()
    assert (np.abs(got - ref) <= ROUND[dtype] * np.abs(ref) + rel * size + C * size).all()
    assert (np.abs(lse.double().cpu().numpy() - rlse) <= rel + 2.0 ** -20 * np.abs(rlse)).all()


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("up", [True, False])
@pytest.mark.parametrize("D,new", [(64, 1), (128, 5), (80, 5)])
def test_scores_that_climb_or_fall(ssd, dtype, up, D, new):
    # from 0 to 20 (or back) along 700 tokens: within a unit by less than the maximum may lag behind, over all by more
    c = make(31, [700, 260], [new, new], 4, 1, D, 24, dtype)
    c["q"] *= 0.05
    c["q"][:, :, 0] = 4.0
    for r, n in enumerate((700, 260)):
        t = np.arange(n)
        page = torch.from_numpy(c["table"][r].numpy()[t // 24].astype(np.int64))
        climb = torch.from_numpy(5.0 * (t if up else 700 - t) / 700).to(dtype)
        c["kc"][page, torch.from_numpy(t % 24), :, 0] = climb[:, None]
    check(*run(ssd, c, scale=1.0), c, scale=1.0)


def test_infinite_and_nan_values_reach_only_rows_that_see_them(ssd):
    # the last token's value is infinite: only the last of three rows sees it
    c = make(20, [50], [3], 4, 2, 64, 16, BF)
    c["vc"][c["table"][0, 49 // 16], 49 % 16] = float("inf")
    out, lse = run(ssd, c)
    assert torch.isfinite(out[:2]).all() and torch.isinf(out[2]).all()
    one = dict(c, q=c["q"][:2], pos=c["pos"][:2], start=torch.tensor([0, 2], dtype=torch.int32))
    check(out[:2], lse[:2], one)
    # so with a key, and with a window's oldest token
    c = make(21, [50], [3], 4, 2, 64, 16, BF)
    c["kc"][c["table"][0, 49 // 16], 49 % 16] = float("nan")
    c["vc"][c["table"][0, 38 // 16], 38 % 16] = float("nan")
    out, lse = run(ssd, c, window=10)   # row 0 sees 38 .. 47, row 1 39 .. 48, row 2 40 .. 49
    assert torch.isnan(out[0]).all() and torch.isfinite(out[1]).all() and torch.isnan(out[2]).all()
    one = dict(c, q=c["q"][1:2], pos=c["pos"][1:2], start=None)
    check(out[1:2], lse[1:2], one, window=10)


def test_strided_operands_and_in_place(ssd):
    c = make(22, [70, 200, 31], None, 8, 2, 64, 16, BF)
    qkv = torch.zeros(3, 12, 64, dtype=BF, device="cuda")
    qkv[:, :8] = c["q"].cuda()
    wide = torch.full((3, c["table"].shape[1] + 5), -1, dtype=torch.int32, device="cuda")
    wide[:, 2:2 + c["table"].shape[1]] = c["table"].cuda()
    q, table = qkv[:, :8], wide[:, 2:2 + c["table"].shape[1]]
    args = (to_gpu(c["kc"]), to_gpu(c["vc"]), table, c["pos"].cuda())
    ref, rl = run(ssd, c)
    out, lse = ssd.paged_attn_fwd(q, *args)
    assert torch.equal(out, ref) and torch.equal(lse, rl)
    hm = torch.empty(8, 3, 64, dtype=BF, device="cuda").transpose(0, 1)   # heads outermost
    ssd.paged_attn_fwd(q, *args, out=hm, return_lse=False)
    assert torch.equal(hm, ref)
    ssd.paged_attn_fwd(q, *args, out=q)
    assert torch.equal(q, ref) and (qkv[:, 8:] == 0).all()


def test_workspace_and_repeat_bits(ssd):
    c = make(23, [3000, 10, 999], None, 8, 2, 128, 16, BF)
    args = tuple(to_gpu(c[k]) for k in ("q", "kc", "vc", "table", "pos", "start"))
    a, al = ssd.paged_attn_fwd(*args)
    need = ssd.paged_attn_workspace_size(*args[:4])
    ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        b, bl = ssd.paged_attn_fwd(*args, workspace=ws)
        assert torch.equal(a, b) and torch.equal(al, bl)
    if need:
        with pytest.raises(ssd.SsdError):
            ssd.paged_attn_fwd(*args, workspace=ws[:need - 16])


def test_other_stream(ssd):
    c = make(24, [500, 64], None, 8, 2, 128, 16, BF)
    st = torch.cuda.Stream()
    args = tuple(to_gpu(c[k]) for k in ("q", "kc", "vc", "table", "pos", "start"))
    torch.cuda.synchronize()
    q = torch.zeros_like(args[0])
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(20_000_000)
        q.copy_(args[0])
        out, lse = ssd.paged_attn_fwd(q, *args[1:])
    out2, lse2 = ssd.paged_attn_fwd(*args)
    torch.cuda.synchronize()
    check(out, lse, c)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_offsets_past_32_bits(ssd):
    # a cache of more than 2^32 elements, the request's pages at its far end
    D, hk, ps, n = 128, 8, 64, 300
    npages = (1 << 32) // (D * hk * ps) + 9
    small = make(25, [n], None, 16, hk, D, ps, BF)
    kc = torch.empty(npages, ps, hk, D, dtype=BF, device="cuda")
    vc = torch.empty(npages, ps, hk, D, dtype=BF, device="cuda")
    far = npages - small["kc"].shape[0]
    kc[far:], vc[far:] = small["kc"].cuda(), small["vc"].cuda()
    table = small["table"].clone()
    table[0, :-(-n // ps)] += far
    out, lse = ssd.paged_attn_fwd(small["q"].cuda(), kc, vc, table.cuda(), small["pos"].cuda())
    torch.cuda.synchronize()
    check(out, lse, small)


def test_refusals(ssd):
    c = make(26, [40, 20], None, 8, 2, 64, 16, BF)
    q, kc, vc, table, pos = (to_gpu(c[k]) for k in ("q", "kc", "vc", "table", "pos"))
    for bad in (dict(q=q.half()), dict(q=q.float()), dict(q=q[:, :7]), dict(kc=kc[..., :32]), dict(pos=pos.long()),
                dict(pos=pos[:1]), dict(table=table.long()), dict(table=table[:1]), dict(q=q.cpu()),
                dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)), dict(vc=vc[:1])):
        a = dict(dict(q=q, kc=kc, vc=vc, table=table, pos=pos), **bad)
        with pytest.raises((ValueError, ssd.SsdError)):
            ssd.paged_attn_fwd(a["q"], a["kc"], a["vc"], a["table"], a["pos"])
    with pytest.raises(ssd.SsdError):
        ssd.paged_attn_fwd(q, kc, vc, table, pos, window=-1)
    with pytest.raises(ssd.SsdError):
        ssd.paged_attn_fwd(q, kc, vc, table, pos, scale=float("nan"))
    with pytest.raises(ssd.SsdError):   # an output over an input
        ssd.paged_attn_fwd(q, kc, vc, table, pos, out=kc.view(-1)[:q.numel()].view(q.shape))
    with pytest.raises(ValueError):
        ssd.paged_attn_fwd(q, kc, vc, table, pos, torch.zeros(2, dtype=torch.int32, device="cuda"))
