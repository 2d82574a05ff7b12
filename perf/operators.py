"""Timed and compared cases of the operators around the attention layers of a hybrid state-space model.

Four operators, one pass of one of them per case ("op"):

* ``plan``: block tables, positions and slot maps of one serving step, built on the GPU from request lengths;
* ``qk_fwd``: RMSNorm of every query and key head with the rotary position in the same pass; when serving, keys and
  values go straight into the paged cache;
* ``qk_bwd``: its gradients;
* ``attn``: attention of new tokens over a paged key-value cache.

With ``own`` false :func:`run` computes them in elementary torch operations in fp32; with ``own`` true it calls the
package.  :func:`exact` computes them from their definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------------

def _plan(name, nreq, page, width, longest, prompts, prompt_len, done):
    """``prompts`` of the requests bring up to ``prompt_len`` tokens, ``done`` are finished, the others bring one token."""
    return dict(name=name, op="plan", nreq=nreq, page=page, width=width, longest=longest, prompts=prompts, prompt_len=prompt_len,
                done=done)


def _qk(name, op, tokens, hq, hk, dim, rot, dtype, interleaved, cache, page=16):
    return dict(name=name, op=op, tokens=tokens, hq=hq, hk=hk, dim=dim, rot=rot, dtype=dtype, interleaved=interleaved, cache=cache,
                page=page)


def _attn(name, nreq, new, shortest, longest, hq, hk, dim, page, window, dtype, layout):
    """``nreq`` requests of ``shortest`` .. ``longest`` tokens, the last ``new`` of them the query rows."""
    return dict(name=name, op="attn", nreq=nreq, new=new, shortest=shortest, longest=longest, hq=hq, hk=hk, dim=dim, page=page,
                window=window, dtype=dtype, layout=layout)


def listed():
    return [
        # a decode step of 128 sequences: every request brings one token, a few are finished
        _plan("plan_decode_128", 128, 16, 256, 4000, 0, 1, 5),
        # a large step of mixed work: 2048 requests, 48 of them prompts of up to 4096 tokens
        _plan("plan_mixed_2048", 2048, 32, 512, 12000, 48, 4096, 60),
        # one attention layer's queries and keys of the 128-sequence decode step, into the cache
        _qk("qk_decode_128", "qk_fwd", 128, 32, 8, 128, 128, "bf16", False, True),
        # the same layer over prompts of 8 x 4096 tokens, into the cache
        _qk("qk_prompt_32768", "qk_fwd", 32768, 32, 8, 128, 128, "bf16", False, True, 32),
        # fp32, heads of 80 with part of each rotated, adjacent pairs, a token count that fits no tile
        _qk("qk_f32_partial_1037", "qk_fwd", 1037, 20, 4, 80, 32, "f32", True, False),
        # training on 8 x 4096 tokens: gradients of the layer's queries, keys and norm weights
        _qk("qk_bwd_32768", "qk_bwd", 32768, 32, 8, 128, 128, "bf16", False, False),
        # the same in fp32 with as many key heads as query heads, a short odd batch
        _qk("qk_bwd_f32_1999", "qk_bwd", 1999, 24, 24, 64, 64, "f32", False, False),
        # one user, one token, a short context: latency counts
        _attn("attn_one_1000", 1, 1, 1000, 1000, 32, 8, 128, 16, 0, "bf16", "nhd"),
        # the decode step of 128 sequences with ragged contexts
        _attn("attn_decode_128", 128, 1, 1, 4096, 32, 8, 128, 16, 0, "bf16", "nhd"),
        # one sequence of 64k tokens, 32 heads in 8 groups, heads of 64
        _attn("attn_long_65536", 1, 1, 65536, 65536, 32, 8, 64, 64, 0, "bf16", "hnd"),
        # the largest: 128 long ragged sequences, 4 new tokens each (drafted tokens to be verified)
        _attn("attn_draft_128x4", 128, 4, 500, 12000, 32, 8, 128, 32, 0, "bf16", "kv"),
        # fp32 with one key head per query head, a sliding window that starts inside a page
        _attn("attn_f32_window", 24, 1, 1, 3500, 24, 24, 64, 24, 1000, "f32", "nhd"),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo .. hi, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "qk_fwd", "qk_bwd", "attn", "attn", "attn"])
    if op == "plan":
        nreq = _spread(rng, 1, 3000)
        prompt_len = _spread(rng, 1, 5000)
        prompts = min(nreq, _spread(rng, 1, max(1, min(200, 120000 // prompt_len))))
        longest = _spread(rng, 16, 12000)
        page = rng.choice([p for p in (1, 8, 16, 24, 32, 64, 128) if nreq * ((longest + prompt_len) // p + 1) <= 1 << 20])
        done = rng.randrange(0, (nreq - prompts) // 4 + 1)
        return _plan(None, nreq, page, -(-(longest + prompt_len) // page), longest, prompts, prompt_len, done)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op in ("qk_fwd", "qk_bwd"):
        dim = rng.choice([64, 80, 96, 128, 192, 256])
        rot = rng.choice([dim, dim, 32, dim // 32 * 16])
        hk = rng.choice([1, 2, 4, 8, 16])
        hq = hk * rng.choice([1, 2, 4, 5, 8])
        most = min(32768, 32768 * 5000 // ((hq + hk) * dim) // (2 if dtype == "f32" else 1))
        tokens = _spread(rng, 1, most)
        return _qk(None, op, tokens, hq, hk, dim, rot, dtype, rng.random() < 0.4, op == "qk_fwd" and rng.random() < 0.6,
                   rng.choice([16, 24, 64]))
    dim = rng.choice([64, 64, 80, 128, 128, 256])
    hk = rng.choice([1, 2, 4, 8, 8])
    hq = hk * rng.choice([1, 3, 4, 4, 8, 16])
    new = rng.choice([1, 1, 1, 2, 5])
    nreq = _spread(rng, 1, 300)
    longest = _spread(rng, 64, 66000)
    room = (3 << 28) // (hk * dim) // new // (2 if dtype == "f32" else 1)  # tokens in all: at most 3.2 GB read
    longest = max(8, min(longest, room // nreq))
    shortest = rng.choice([1, longest // 2 + 1, longest])
    window = rng.choice([0, 0, 0, _spread(rng, 16, 5000)])
    return _attn(None, nreq, new, shortest, longest, hq, hk, dim, rng.choice([16, 16, 24, 32, 64, 128]), window, dtype,
                 rng.choice(["nhd", "hnd", "kv"]))


# ---------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------

def _evenly(n, lo, hi):
    """n whole numbers from hi down to lo in even steps (the same multiset for every seed)."""
    return np.round(np.linspace(hi, lo, n)).astype(np.int64)


def _plan_lengths(c):
    """Per request, before shuffling: tokens cached, and tokens it brings (-1: finished)."""
    n = c["nreq"]
    lens = _evenly(n, 1, c["longest"])
    new = np.ones(n, dtype=np.int64)
    if c["prompts"]:
        new[-c["prompts"]:] = _evenly(c["prompts"], max(1, c["prompt_len"] // 4), c["prompt_len"])
        lens[-c["prompts"]:] = 0
    new[:c["done"]] = -1
    return lens, new


def _plan_room(c):
    """Rows of the step's token arrays: what the step brings, rounded up as a program with fixed buffers does."""
    _, new = _plan_lengths(c)
    return -(-int(new[new > 0].sum()) // 128) * 128


def _prepare_plan(c, seed):
    rng = np.random.default_rng(seed)
    lens, new = _plan_lengths(c)
    order = rng.permutation(c["nreq"])
    lens, new = lens[order], new[order]
    held = -(-lens // c["page"])
    need = -(-np.maximum(lens + new, lens) // c["page"])
    spare = int((need - held).sum()) + 64
    cap = int(held.sum()) + spare
    pages = rng.permutation(cap).astype(np.int32)
    table = np.full((c["nreq"], c["width"]), -1, dtype=np.int32)
    inside = np.arange(c["width"])[None, :] < held[:, None]
    table[inside] = pages[:held.sum()]
    # a program that has served for a while: the ring of free pages starts anywhere in its array and wraps around
    head = int(rng.integers(0, 5 * cap))
    ring = np.full(cap, -1, dtype=np.int32)
    ring[(head + np.arange(spare)) % cap] = pages[held.sum():]
    dev = lambda a, t: torch.from_numpy(np.ascontiguousarray(a)).to(device="cuda", dtype=t)  # noqa: E731
    n, room = c["nreq"], _plan_room(c)
    empty = lambda k, t=torch.int32: torch.empty(k, dtype=t, device="cuda")  # noqa: E731
    # the buffers that a program keeps for the step's plan
    kept = dict(lens=empty(n), granted=empty(n), start=empty(n + 1), positions=empty(room), token_req=empty(room),
                slots=empty(room, torch.int64), ring_pos=empty(2, torch.int64), counts=empty(4))
    return dict(op="plan", case=c, lens=dev(lens, torch.int32), new=dev(new, torch.int32), table=dev(table, torch.int32),
                ring=dev(ring, torch.int32), ring_pos=dev(np.array([head, head + spare]), torch.int64), page=c["page"], room=room,
                kept=kept)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 11)


def _rope_angles(positions, rot):
    """cos and sin [positions, rot/2] of the usual geometric frequencies, in fp64."""
    freq = 10000.0 ** (-np.arange(rot // 2, dtype=np.float64) * 2.0 / rot)
    ang = np.asarray(positions, dtype=np.float64)[:, None] * freq[None, :]
    return np.cos(ang), np.sin(ang)


def _qk_positions(c):
    """Positions of the tokens: sequences of up to 4096 tokens one after another when there are many, else one token of each."""
    t = np.arange(c["tokens"])
    return t % 4096 if c["tokens"] > 512 else (t * 31 + 7) % 4096


def _prepare_qk(c, seed):
    g, dt = _gen(seed), _TYPES[c["dtype"]]
    T, hq, hk, D = c["tokens"], c["hq"], c["hk"], c["dim"]
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    # the fused projection's output; heads differ in scale
    qkv = (normal(T, hq + 2 * hk, D) * (0.5 + 2.0 * torch.rand(hq + 2 * hk, 1, generator=g, device="cuda"))).to(dt)
    cos, sin = _rope_angles(np.arange(4096), c["rot"])
    f32 = lambda a: torch.from_numpy(a.astype(np.float32)).cuda()  # noqa: E731
    s = dict(op=c["op"], case=c, q=qkv[:, :hq], k=qkv[:, hq:hq + hk], v=qkv[:, hq + hk:], qw=1.0 + 0.2 * normal(D), kw=1.0 + 0.2 * normal(D),
             cos=f32(cos), sin=f32(sin), pos=torch.from_numpy(_qk_positions(c)).to("cuda", torch.int32), eps=1e-6,
             interleaved=c["interleaved"])
    if c["op"] == "qk_bwd":
        s["dq"], s["dk"] = normal(T, hq, D).to(dt), normal(T, hk, D).to(dt)
    if c["cache"]:
        pages = -(-T // c["page"]) + 3
        slots = np.random.default_rng(seed).permutation(pages)[np.arange(T) // c["page"]] * c["page"] + np.arange(T) % c["page"]
        s["slots"] = torch.from_numpy(slots.astype(np.int64)).cuda()
        s["kc"] = torch.zeros(pages, c["page"], hk, D, dtype=dt, device="cuda")
        s["vc"] = torch.zeros(pages, c["page"], hk, D, dtype=dt, device="cuda")
    return s


def _attn_lengths(c):
    return np.maximum(_evenly(c["nreq"], c["shortest"], c["longest"]), c["new"])


def _prepare_attn(c, seed):
    rng, g, dt = np.random.default_rng(seed), _gen(seed), _TYPES[c["dtype"]]
    hq, hk, D, ps = c["hq"], c["hk"], c["dim"], c["page"]
    lens = rng.permutation(_attn_lengths(c))
    held = -(-lens // ps)
    npages = int(held.sum()) + 7
    table = np.full((c["nreq"], int(held.max())), -1, dtype=np.int32)
    table[np.arange(table.shape[1])[None, :] < held[:, None]] = rng.permutation(npages)[:held.sum()]
    shape = {"nhd": (npages, ps, hk, D), "hnd": (npages, hk, ps, D), "kv": (npages, 2, ps, hk, D)}[c["layout"]]

    def cache():
        return torch.empty(shape, dtype=dt, device="cuda").normal_(generator=g)

    if c["layout"] == "kv":
        both = cache()
        kc, vc = both[:, 0], both[:, 1]
    else:
        kc, vc = cache(), cache()
        if c["layout"] == "hnd":
            kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    rows = c["nreq"] * c["new"]
    pos = (lens[:, None] - c["new"] + np.arange(c["new"])[None, :]).reshape(-1)
    qkv = torch.empty(rows, hq + 2 * hk, D, dtype=dt, device="cuda").normal_(std=1.5, generator=g)
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to("cuda", torch.int32)  # noqa: E731
    return dict(op="attn", case=c, q=qkv[:, :hq], kc=kc, vc=vc, table=i32(table), pos=i32(pos),
                start=i32(np.arange(c["nreq"] + 1) * c["new"]) if c["new"] > 1 else None,
                scale=1.0 / math.sqrt(D), window=c["window"], out=torch.empty(rows, hq, D, dtype=dt, device="cuda"),
                lse=torch.empty(rows, hq, dtype=torch.float32, device="cuda"))


def prepare(case, seed):
    return {"plan": _prepare_plan, "qk_fwd": _prepare_qk, "qk_bwd": _prepare_qk, "attn": _prepare_attn}[case["op"]](case, seed)


# ---------------------------------------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------------------------------------

def _run_plan(s):
    lens, new, table, ring = s["lens"].long(), s["new"].long(), s["table"], s["ring"]
    ps, room, width, cap = s["page"], s["room"], table.shape[1], ring.numel()
    head, tail = s["ring_pos"][0], s["ring_pos"][1]
    held = (lens + ps - 1) // ps
    fits = (new > 0) & (lens + new <= width * ps)
    tokens = torch.where(fits, new, 0)
    pages = torch.where(fits, (lens + new + ps - 1) // ps - held, 0)
    admit = fits & (tokens.cumsum(0) <= room) & (pages.cumsum(0) <= tail - head)
    granted = torch.where(admit, new, 0)
    done = new < 0
    taken, back = torch.where(admit, pages, 0), torch.where(done, held, 0)
    start = torch.nn.functional.pad(granted.cumsum(0), (1, 0))
    col = torch.arange(width, device="cuda")[None, :]
    # pages drawn from the ring's head, in request order
    drawn = head + (taken.cumsum(0) - taken)[:, None] + col - held[:, None]
    table.copy_(torch.where((col >= held[:, None]) & (col < (held + taken)[:, None]), ring[drawn % cap], table))
    # pages given back at its tail
    to = (tail + (back.cumsum(0) - back)[:, None] + col) % cap
    to = torch.where(col < back[:, None], to, cap)
    ring.copy_(torch.nn.functional.pad(ring, (0, 1)).scatter(0, to.reshape(-1), table.reshape(-1))[:cap])
    t = torch.arange(room, device="cuda")
    live = t < start[-1]
    req = torch.searchsorted(start[1:], t, right=True).clamp(max=lens.numel() - 1)
    pos = lens[req] + t - start[req]
    page = table[req, (pos // ps).clamp(max=width - 1)].long()
    ints = lambda a: a.to(torch.int32)  # noqa: E731
    return dict(lens=ints(torch.where(done, 0, lens + granted)), granted=ints(granted), start=ints(start),
                positions=ints(torch.where(live, pos, -1)), token_req=ints(torch.where(live, req, -1)),
                slots=torch.where(live, page * ps + pos % ps, -1), ring_pos=torch.stack([head + taken.sum(), tail + back.sum()]),
                counts=ints(torch.stack([start[-1], taken.sum(), back.sum(), ((new > 0) & ~admit).sum()])), table=table, ring=ring)


def _pairs(x, rot, interleaved):
    """The two members of each rotated pair of the last axis, and the axis's unrotated rest."""
    if interleaved:
        return x[..., 0:rot:2], x[..., 1:rot:2], x[..., rot:]
    return x[..., :rot // 2], x[..., rot // 2:rot], x[..., rot:]


def _unpairs(a, b, rest, interleaved):
    if interleaved:
        return torch.cat([torch.stack([a, b], -1).flatten(-2), rest], -1)
    return torch.cat([a, b, rest], -1)


def _norm_rope(x, w, cos, sin, eps, interleaved):
    x = x.float()
    n = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w
    a, b, rest = _pairs(n, 2 * cos.shape[-1], interleaved)
    return _unpairs(a * cos - b * sin, b * cos + a * sin, rest, interleaved)


def _run_qk_fwd(s):
    cos, sin = s["cos"][s["pos"].long()][:, None], s["sin"][s["pos"].long()][:, None]
    q = _norm_rope(s["q"], s["qw"], cos, sin, s["eps"], s["interleaved"]).to(s["q"].dtype)
    k = _norm_rope(s["k"], s["kw"], cos, sin, s["eps"], s["interleaved"]).to(s["k"].dtype)
    if "kc" not in s:
        return dict(q=q, k=k)
    s["kc"].flatten(0, 1)[s["slots"]] = k
    s["vc"].flatten(0, 1)[s["slots"]] = s["v"]
    return dict(q=q, k_cache=s["kc"], v_cache=s["vc"])


def _norm_rope_grad(x, w, d, cos, sin, eps, interleaved):
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)
    a, b, rest = _pairs(d.float(), 2 * cos.shape[-1], interleaved)
    g = _unpairs(a * cos + b * sin, b * cos - a * sin, rest, interleaved)
    n = x * r
    dw = (g * n).sum((0, 1))
    g = g * w
    return r * (g - n * (g * n).mean(-1, keepdim=True)), dw


def _run_qk_bwd(s):
    cos, sin = s["cos"][s["pos"].long()][:, None], s["sin"][s["pos"].long()][:, None]
    dq, dqw = _norm_rope_grad(s["q"], s["qw"], s["dq"], cos, sin, s["eps"], s["interleaved"])
    dk, dkw = _norm_rope_grad(s["k"], s["kw"], s["dk"], cos, sin, s["eps"], s["interleaved"])
    return dict(dq=dq.to(s["q"].dtype), dk=dk.to(s["k"].dtype), dq_weight=dqw, dk_weight=dkw)


def _run_attn(s):
    q, pos, ps = s["q"].float(), s["pos"].long(), s["kc"].shape[1]
    rows, hq, D = q.shape
    hk = s["kc"].shape[2]
    pages = s["table"].clamp(min=0).long()
    new = rows // pages.shape[0]
    at = torch.arange(pages.shape[1] * ps, device="cuda")
    seen = at[None, :] <= pos[:, None]
    if s["window"]:
        seen = seen & (at[None, :] > pos[:, None] - s["window"])
    seen = seen.view(-1, new, 1, 1, at.numel())
    k = s["kc"][pages].float().flatten(1, 2)
    score = torch.einsum("nihgd,nlhd->nihgl", q.view(-1, new, hk, hq // hk, D), k) * s["scale"]
    del k
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top > -math.inf, top, 0.0))
    total = p.sum(-1, keepdim=True)
    v = s["vc"][pages].float().flatten(1, 2)
    v = torch.where(seen.any(1)[:, 0, 0, :, None, None], v, 0.0)
    out = torch.einsum("nihgl,nlhd->nihgd", p, v) / torch.where(total > 0, total, 1.0)
    return dict(out=out.reshape(rows, hq, D).to(s["q"].dtype), lse=(top + torch.log(total)).reshape(rows, hq))


# ---------------------------------------------------------------------------------------------------------------------
# the package's operators
# ---------------------------------------------------------------------------------------------------------------------

def _own_plan(s):
    from selective_state_space_04_gb300 import ssd
    r = ssd.paged_plan(s["lens"], s["new"], s["table"], s["ring"], s["ring_pos"], page_size=s["page"], max_tokens=s["room"],
                       out=s["kept"])
    return dict(r, table=s["table"], ring=s["ring"])


def _own_qk_fwd(s):
    from selective_state_space_04_gb300 import ssd
    if "kc" not in s:
        q, k = ssd.qk_norm_rope_fwd(s["q"], s["k"], s["qw"], s["kw"], s["cos"], s["sin"], s["pos"], eps=s["eps"],
                                    interleaved=s["interleaved"])
        return dict(q=q, k=k)
    q, _ = ssd.qk_norm_rope_fwd(s["q"], s["k"], s["qw"], s["kw"], s["cos"], s["sin"], s["pos"], eps=s["eps"],
                                interleaved=s["interleaved"], v=s["v"], k_cache=s["kc"], v_cache=s["vc"], slots=s["slots"],
                                return_k=False)
    return dict(q=q, k_cache=s["kc"], v_cache=s["vc"])


def _own_qk_bwd(s):
    from selective_state_space_04_gb300 import ssd
    return ssd.qk_norm_rope_bwd(s["q"], s["k"], s["qw"], s["kw"], s["cos"], s["sin"], s["pos"], s["dq"], s["dk"], eps=s["eps"],
                                interleaved=s["interleaved"])


def _own_attn(s):
    from selective_state_space_04_gb300 import ssd
    out, lse = ssd.paged_attn_fwd(s["q"], s["kc"], s["vc"], s["table"], s["pos"], s["start"], scale=s["scale"], window=s["window"],
                                  out=s["out"], lse=s["lse"])
    return dict(out=out, lse=lse)


def run(state):
    if own:
        return {"plan": _own_plan, "qk_fwd": _own_qk_fwd, "qk_bwd": _own_qk_bwd, "attn": _own_attn}[state["op"]](state)
    return {"plan": _run_plan, "qk_fwd": _run_qk_fwd, "qk_bwd": _run_qk_bwd, "attn": _run_attn}[state["op"]](state)


# ---------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "plan":
        lens, new = _plan_lengths(c)
        held = -(-lens // c["page"])
        taken = int((-(-np.maximum(lens + new, lens) // c["page"]) - held)[new > 0].sum())
        back = int(held[new < 0].sum())
        # lengths in and out, what was granted, where each request starts; a page moved is read and written; per token its
        # position, request and slot
        nbytes = c["nreq"] * 20 + (taken + back) * 8 + _plan_room(c) * 16 + 52
        return {"bytes": nbytes, "flops": 0}
    size = 4 if c["dtype"] == "f32" else 2
    if c["op"] in ("qk_fwd", "qk_bwd"):
        T, D, heads = c["tokens"], c["dim"], c["hq"] + c["hk"]
        angles = len(np.unique(_qk_positions(c))) * c["rot"] * 4
        if c["op"] == "qk_fwd":
            moved = 2 * heads + (2 * c["hk"] if c["cache"] else 0)
            return {"bytes": T * moved * D * size + angles + T * (12 if c["cache"] else 4) + 8 * D, "flops": T * heads * (4 * D + 3 * c["rot"])}
        return {"bytes": T * 3 * heads * D * size + angles + T * 4 + 16 * D, "flops": T * heads * (12 * D + 3 * c["rot"])}
    lens, new = _attn_lengths(c), c["new"]
    end = (lens - new + 1)[:, None] + np.arange(new)[None, :]
    first = np.maximum(0, end - c["window"]) if c["window"] else np.zeros_like(end)
    seen, read = int((end - first).sum()), int((lens - first[:, 0]).sum())
    rows = c["nreq"] * new
    nbytes = read * c["hk"] * c["dim"] * 2 * size + rows * c["hq"] * (2 * c["dim"] * size + 4) + rows * 4 + int((-(-lens // c["page"])).sum()) * 4
    return {"bytes": nbytes, "flops": 4 * seen * c["hq"] * c["dim"]}


# ---------------------------------------------------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------------------------------------------------

def _exact_plan(c, seed):
    s = _prepare_plan(c, seed)
    lens, new = s["lens"].tolist(), s["new"].tolist()
    table, ring = s["table"].cpu().numpy().copy(), s["ring"].cpu().numpy().copy()
    head, tail = s["ring_pos"].tolist()
    ps, room, cap, limit = c["page"], s["room"], len(ring), table.shape[1] * c["page"]
    free, first, at_tail = tail - head, head, tail
    asked_tokens = asked_pages = refused = given = 0
    lens_out, granted, start, positions, token_req, slots = [], [], [0], [], [], []
    old = ring.copy()
    for r, (n, m) in enumerate(zip(lens, new)):
        got, held = 0, -(-n // ps)
        if m < 0:
            for j in range(held):
                ring[at_tail % cap] = table[r, j]
                at_tail += 1
            given += held
        elif m > 0:
            want = -(-(n + m) // ps) - held
            if n + m <= limit:
                asked_tokens += m
                asked_pages += want
            if n + m <= limit and asked_tokens <= room and asked_pages <= free:
                got = m
                for j in range(want):
                    table[r, held + j] = old[first % cap]
                    first += 1
                at = np.arange(n, n + m)
                positions.append(at)
                token_req.append(np.full(m, r))
                slots.append(table[r, at // ps].astype(np.int64) * ps + at % ps)
            else:
                refused += 1
        granted.append(got)
        lens_out.append(0 if m < 0 else n + got)
        start.append(start[-1] + got)
    full = lambda parts: torch.from_numpy(np.concatenate([*parts, np.full(room - start[-1], -1)]).astype(np.int64))  # noqa: E731
    ints = lambda a: torch.as_tensor(a, dtype=torch.int32)  # noqa: E731
    return dict(lens=ints(lens_out), granted=ints(granted), start=ints(start), positions=full(positions).to(torch.int32),
                token_req=full(token_req).to(torch.int32), slots=full(slots), ring_pos=torch.tensor([first, at_tail]),
                counts=ints([start[-1], first - head, given, refused]), table=torch.from_numpy(table), ring=torch.from_numpy(ring))


def _rotation(c, s):
    """Per token, the pair partner's place and the two coefficients of each element: y_i = c_i n_i + s_i n_partner(i)."""
    D, rot = c["dim"], c["rot"]
    cos, sin = s["cos"][s["pos"].long()].double(), s["sin"][s["pos"].long()].double()
    i = torch.arange(D, device="cuda")
    if c["interleaved"]:
        partner, pair, second = i ^ 1, i // 2, (i % 2) == 1
    else:
        partner, pair, second = (i + rot // 2) % rot, i % (rot // 2), i >= rot // 2
    partner, pair = torch.where(i < rot, partner, i), torch.where(i < rot, pair, 0)
    cc = torch.where(i < rot, cos[:, pair], 1.0)
    ss = torch.where(i < rot, torch.where(second, sin[:, pair], -sin[:, pair]), 0.0)
    return partner, cc[:, None], ss[:, None]


def _exact_qk_fwd(c, seed):
    s = _prepare_qk(c, seed)
    partner, cc, ss = _rotation(c, s)
    got = []
    for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
        x = x.double()
        n = x / (x.pow(2).sum(-1, keepdim=True) / c["dim"] + s["eps"]).sqrt() * w.double()
        got.append(cc * n + ss * n[..., partner])
    if not c["cache"]:
        return dict(q=got[0], k=got[1])
    kc, vc = s["kc"].double(), s["vc"].double()
    kc.view(-1, c["hk"], c["dim"]).index_copy_(0, s["slots"], got[1])
    vc.view(-1, c["hk"], c["dim"]).index_copy_(0, s["slots"], s["v"].double())
    return dict(q=got[0], k_cache=kc, v_cache=vc)


def _exact_qk_bwd(c, seed):
    s = _prepare_qk(c, seed)
    partner, cc, ss = _rotation(c, s)
    back = torch.argsort(partner)
    got = {}
    for name, x, w, d in (("q", s["q"], s["qw"], s["dq"]), ("k", s["k"], s["kw"], s["dk"])):
        x, d, w = x.double(), d.double(), w.double()
        g = cc * d + (ss * d)[..., back]
        r2 = 1.0 / (x.pow(2).sum(-1, keepdim=True) / c["dim"] + s["eps"])
        r = r2.sqrt()
        got["d%s_weight" % name] = torch.einsum("thd,thd->d", g, x * r)
        gw = g * w
        got["d%s" % name] = r * gw - x * (r * r2 / c["dim"]) * (gw * x).sum(-1, keepdim=True)
    return dict(dq=got["dq"], dk=got["dk"], dq_weight=got["dq_weight"], dk_weight=got["dk_weight"])


def _exact_attn(c, seed):
    s = _prepare_attn(c, seed)
    group = c["hq"] // c["hk"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    for n, pages in enumerate(s["table"]):
        last = int(s["pos"][(n + 1) * c["new"] - 1])
        pages = pages[:last // c["page"] + 1].long()
        k, v = (x[pages].flatten(0, 1)[:last + 1].double().transpose(0, 1) for x in (s["kc"], s["vc"]))
        for row in range(n * c["new"], (n + 1) * c["new"]):
            end = int(s["pos"][row]) + 1
            begin = max(0, end - c["window"]) if c["window"] else 0
            q = s["q"][row].double().view(c["hk"], group, c["dim"])
            z = s["scale"] * torch.matmul(q, k[:, begin:end].transpose(1, 2))
            lse[row] = torch.logsumexp(z, -1).view(-1)
            out[row] = torch.matmul(torch.softmax(z, -1), v[:, begin:end]).view(c["hq"], c["dim"])
    return dict(out=out, lse=lse)


def exact(case, seed):
    return {"plan": _exact_plan, "qk_fwd": _exact_qk_fwd, "qk_bwd": _exact_qk_bwd, "attn": _exact_attn}[case["op"]](case, seed)
