"""Timed and compared cases of the operators around the scan in one state-space layer's step with 8-bit projections.

Four operators, one pass per case ("op"):

* ``norm``: the residual's addition with RMSNorm, out in the input's type or in 8 bits with a scale per row;
  ``norm_grad``: its gradients;
* ``matmul``: products of 8-bit integers with scales per token and per output channel; ``gate_matmul``: the gated norm
  of a scan's output into 8 bits, and the output projection that takes it;
* ``step``: the short causal convolution and the scan for single tokens, on a pool of carried states.

With ``own`` false :func:`run` computes them in elementary torch operations in fp32; with ``own`` true it calls the
package.  :func:`exact` computes them from their definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_EPS = 1e-5


# ---------------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------------

def _norm(name, rows, dim, dtype, residual, q8):
    """``residual``: the type of the residual stream, or "none"."""
    return dict(name=name, op="norm", rows=rows, dim=dim, dtype=dtype, residual=residual, q8=q8)


def _norm_grad(name, rows, dim, dtype, residual):
    return dict(name=name, op="norm_grad", rows=rows, dim=dim, dtype=dtype, residual=residual)


def _matmul(name, tokens, features, inner, dtype):
    return dict(name=name, op="matmul", tokens=tokens, features=features, inner=inner, dtype=dtype)


def _gate_matmul(name, tokens, features, inner, dtype):
    return dict(name=name, op="gate_matmul", tokens=tokens, features=features, inner=inner, dtype=dtype)


def _step(name, nseq, padding, heads, headdim, dstate, groups, taps, dtype, fresh):
    """``nseq`` sequences of one token each and ``padding`` empty rows; ``fresh`` of the sequences begin with this token."""
    return dict(name=name, op="step", nseq=nseq, padding=padding, heads=heads, headdim=headdim, dstate=dstate, groups=groups, taps=taps,
                dtype=dtype, fresh=fresh)


def listed():
    return [
        # the norm in front of the input projection of a 2560-wide layer, decode step of 128 sequences, for an 8-bit product
        _norm("norm_q8_decode_128", 128, 2560, "bf16", "f32", True),
        # the same norm in training: 8 x 4096 tokens, residual stream in bf16
        _norm("norm_32768", 32768, 2560, "bf16", "bf16", False),
        # its gradients, with that of the residual stream
        _norm_grad("norm_grad_32768", 32768, 2560, "bf16", "bf16"),
        # fp32, a width that fits no power of two, a short odd batch
        _norm_grad("norm_grad_f32_1999", 1999, 1000, "f32", "none"),
        # the input projection (z, x, B, C and dt of 80 heads of 64, state 128) for one token of one user
        _matmul("matmul_one", 1, 10576, 2560, "bf16"),
        # the same for the decode step of 128 sequences
        _matmul("matmul_decode_128", 128, 10576, 2560, "bf16"),
        # and for a prompt of 8192 tokens: the largest
        _matmul("matmul_prompt_8192", 8192, 10576, 2560, "bf16"),
        # fp32 out, sizes that fit no tile
        _matmul("matmul_f32_odd", 77, 333, 1001, "f32"),
        # scan output to residual width for a prompt of 4096 tokens: gated norm, 8 bits, output projection
        _gate_matmul("gate_matmul_4096", 4096, 2560, 5120, "bf16"),
        # one user's next token in a layer of 80 heads
        _step("step_one", 1, 0, 80, 64, 128, 1, 4, "bf16", 0),
        # the decode step of 128 sequences, three of them new, in a batch padded to a fixed size
        _step("step_decode_128", 125, 3, 80, 64, 128, 1, 4, "bf16", 3),
        # fp32, small states in groups, a short filter
        _step("step_f32_groups", 37, 3, 24, 48, 20, 3, 3, "f32", 1),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo .. hi, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "matmul", "matmul", "matmul", "gate_matmul", "step", "step"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op in ("norm", "norm_grad"):
        dim = 8 * _spread(rng, 8, 1024)
        rows = _spread(rng, 1, min(65536, (84 << 20) // dim // (2 if dtype == "f32" else 1)))
        residual = rng.choice(["none", dtype, "f32"])
        return _norm(None, rows, dim, dtype, residual, rng.random() < 0.6) if op == "norm" else _norm_grad(None, rows, dim, dtype, residual)
    if op in ("matmul", "gate_matmul"):
        inner = _spread(rng, 64, 8192) if op == "matmul" else 8 * _spread(rng, 16, 1024)
        features = _spread(rng, 16, 16384)
        most = min(8192 if op == "matmul" else 4096, 400_000_000_000 // (2 * inner * features))
        tokens = _spread(rng, 1, max(1, most))
        return (_matmul if op == "matmul" else _gate_matmul)(None, tokens, features, inner, dtype)
    groups = rng.choice([1, 1, 2, 4])
    heads = groups * _spread(rng, 2, 40)
    headdim, dstate = rng.choice([32, 64, 64, 80, 128]), rng.choice([16, 64, 128, 128, 256])
    most = (80 << 20) // (heads * headdim * dstate)
    nseq = _spread(rng, 1, max(1, min(512, most)))
    return _step(None, nseq, rng.choice([0, 0, 5]), heads, headdim, dstate, groups, rng.choice([2, 3, 4, 4]), dtype, min(nseq, rng.choice([0, 2])))


# ---------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 23)


def _prepare_norm(c, seed):
    g, dt = _gen(seed), _TYPES[c["dtype"]]
    n, D = c["rows"], c["dim"]
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    # tokens differ in scale; a few channels of the residual stream are much larger than the others, as in trained layers
    channel = torch.exp(0.5 * normal(D))
    channel[torch.randperm(D, generator=g, device="cuda")[:max(1, D // 256)]] *= 8.0
    s = dict(op=c["op"], case=c, w=1.0 + 0.2 * normal(D), eps=_EPS)
    s["x"] = (normal(n, D) * (0.5 + torch.rand(n, 1, generator=g, device="cuda"))).to(dt)
    s["residual"] = None if c["residual"] == "none" else (normal(n, D) * channel).to(_TYPES[c["residual"]])
    if c["op"] == "norm" and c["q8"]:
        s["values"] = torch.empty(n, D, dtype=torch.bfloat16, device="cuda")
    if c["op"] == "norm_grad":
        # what the forward pass kept (the sum, in the residual stream's type), and the gradients of its two outputs
        s["h"] = s.pop("x") if s["residual"] is None else (s.pop("x").float() + s["residual"].float()).to(s["residual"].dtype)
        s["dout"] = normal(n, D).to(dt)
        s["dres"] = None if s["residual"] is None else normal(n, D).to(s["residual"].dtype)
        del s["residual"]
    return s


def _prepare_weight(c, g):
    """8-bit weights [features, inner] with a scale per feature, as a matrix and in the order in which the package keeps
    them: tiles of 128 features; in each, blocks of 16 inner elements with the features side by side; zeros where a tile
    or the last 64 inner elements are not full."""
    N, K = c["features"], c["inner"]
    wq = torch.clamp(torch.round(torch.empty(N, K, device="cuda").normal_(std=36.0, generator=g)), -127, 127).to(torch.int8)
    scale = (0.5 + torch.rand(N, generator=g, device="cuda")) / (36.0 * math.sqrt(K))
    n, k = -(-N // 128) * 128, -(-K // 64) * 64
    full = torch.zeros(n, k, dtype=torch.int8, device="cuda")
    full[:N, :K] = wq
    packed = full.view(n // 128, 128, k // 16, 16).transpose(1, 2).contiguous().view(-1)
    return wq, scale, packed


def _prepare_matmul(c, seed):
    g = _gen(seed)
    M, K = c["tokens"], c["inner"]
    wq, wscale, packed = _prepare_weight(c, g)
    a = torch.empty(M, K, device="cuda").normal_(generator=g) * torch.exp(0.4 * torch.randn(K, generator=g, device="cuda"))
    scale = a.abs().amax(1) / 127.0
    aq = torch.clamp(torch.round(a / scale[:, None]), -127, 127).to(torch.int8)
    return dict(op="matmul", case=c, a=aq, a_scale=scale, w=wq, w_scale=wscale, packed=packed, dtype=_TYPES[c["dtype"]])


def _prepare_gate_matmul(c, seed):
    g, dt = _gen(seed), _TYPES[c["dtype"]]
    M, K = c["tokens"], c["inner"]
    wq, wscale, packed = _prepare_weight(c, g)
    y = torch.empty(M, K, device="cuda").normal_(generator=g) * torch.exp(0.5 * torch.randn(K, generator=g, device="cuda"))
    z = torch.empty(M, K, device="cuda").normal_(generator=g)
    return dict(op="gate_matmul", case=c, y=y.to(dt), z=z.to(dt), nw=1.0 + 0.2 * torch.randn(K, generator=g, device="cuda"), eps=_EPS, w=wq,
                w_scale=wscale, packed=packed, dtype=dt)


def _channels(c):
    return c["heads"] * c["headdim"] + 2 * c["groups"] * c["dstate"]


def _prepare_step(c, seed):
    rng, g, dt = np.random.default_rng(seed), _gen(seed), _TYPES[c["dtype"]]
    n, rows, H, P, N = c["nseq"], c["nseq"] + c["padding"], c["heads"], c["headdim"], c["dstate"]
    C, K = _channels(c), c["taps"]
    pool = n + 4
    slots = np.full(rows, -1)
    positions = np.zeros(rows, dtype=np.int64)
    live = np.sort(rng.permutation(rows)[:n])
    slots[live] = rng.permutation(pool - 1)[:n]   # the last slot stays free
    positions[live] = rng.integers(1, 5000, n)
    positions[live[rng.permutation(n)[:c["fresh"]]]] = 0
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    # the fused projection's output: z, then x, B and C, then dt
    proj = torch.empty(rows, H * P + C + H, dtype=dt, device="cuda").normal_(generator=g)
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to("cuda", torch.int32)  # noqa: E731
    return dict(op="step", case=c, xbc=proj[:, H * P:H * P + C], dt=proj[:, H * P + C:], ring=normal(pool, K, C).to(dt),
                states=torch.empty(pool, H, P, N, device="cuda").normal_(generator=g), cw=normal(C, K) / math.sqrt(K), cb=0.1 * normal(C),
                dt_bias=normal(H) - 2.0, A_log=torch.log(1.0 + 15.0 * torch.rand(H, generator=g, device="cuda")), D=1.0 + 0.1 * normal(H),
                slots=i32(slots), positions=i32(positions), y=torch.empty(rows, H, P, dtype=dt, device="cuda"))


def prepare(case, seed):
    return {"norm": _prepare_norm, "norm_grad": _prepare_norm, "matmul": _prepare_matmul, "gate_matmul": _prepare_gate_matmul,
            "step": _prepare_step}[case["op"]](case, seed)


# ---------------------------------------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------------------------------------

def _quantize(v):
    """Whole numbers -127 .. 127 (as floats) and a scale per row."""
    scale = v.abs().amax(-1) / 127.0
    q = torch.round(v / torch.where(scale > 0, scale, 1.0)[:, None])
    return torch.clamp(q, -127, 127), scale


def _run_norm(s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    n = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + s["eps"]) * s["w"]
    kept = {} if s["residual"] is None else {"residual": h.to(s["residual"].dtype)}
    if "values" not in s:
        return dict(kept, out=n.to(s["x"].dtype))
    q, scale = _quantize(n)
    return dict(kept, values=(q * scale[:, None]).to(torch.bfloat16), scale=scale)


def _run_norm_grad(s):
    h, d = s["h"].float(), s["dout"].float()
    r = torch.rsqrt((h * h).mean(-1, keepdim=True) + s["eps"])
    n = h * r
    dw = (d * n).sum(0)
    d = d * s["w"]
    dh = r * (d - n * (d * n).mean(-1, keepdim=True))
    if s["dres"] is not None:
        dh = dh + s["dres"].float()
    return dict(dx=dh.to(s["dout"].dtype), dweight=dw) if s["dres"] is None else dict(dx=dh.to(s["dres"].dtype), dweight=dw)


def _run_matmul(s):
    y = torch.matmul(s["a"].float(), s["w"].float().t())
    return dict(y=(y * s["a_scale"][:, None] * s["w_scale"]).to(s["dtype"]))


def _run_gate_matmul(s):
    y, z = s["y"].float(), s["z"].float()
    n = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + s["eps"]) * s["nw"] * z / (1.0 + torch.exp(-z))
    q, scale = _quantize(n)
    return dict(y=(torch.matmul(q, s["w"].float().t()) * scale[:, None] * s["w_scale"]).to(s["dtype"]))


def _run_step(s):
    c = s["case"]
    H, P, N, G, K = c["heads"], c["headdim"], c["dstate"], c["groups"], c["taps"]
    slots, pos, spare = s["slots"].long(), s["positions"].long(), s["states"].shape[0] - 1
    live = slots >= 0
    at = torch.where(live, slots, spare)
    # the window of inputs pos-K+1 .. pos, zero before the sequence's beginning
    t = pos[:, None] - (K - 1) + torch.arange(K, device="cuda")
    window = s["ring"][at[:, None], t % K].float()
    window = torch.where((t >= 0)[:, :, None], window, 0.0)
    window[:, K - 1] = s["xbc"].float()
    conv = (window * s["cw"].flip(1).t()).sum(1) + s["cb"]   # (tap j multiplies the input j steps back)
    conv = conv / (1.0 + torch.exp(-conv))
    x = conv[:, :H * P].view(-1, H, P)
    B = conv[:, H * P:H * P + G * N].view(-1, G, 1, N).expand(-1, G, H // G, N).reshape(-1, H, 1, N)
    C = conv[:, H * P + G * N:].view(-1, G, 1, N).expand(-1, G, H // G, N).reshape(-1, H, 1, N)
    z = s["dt"].float() + s["dt_bias"]
    dt = torch.clamp(z, min=0.0) + torch.log1p(torch.exp(-z.abs()))
    decay = torch.exp(-dt * torch.exp(s["A_log"]))
    old = s["states"][at]
    h = torch.where((pos > 0)[:, None, None, None], old, 0.0) * decay[:, :, None, None] + (dt[:, :, None] * x)[..., None] * B
    y = (h * C).sum(-1) + s["D"][:, None] * x
    # padding rows write the spare slot's own contents back
    s["states"][at] = torch.where(live[:, None, None, None], h, old)
    s["ring"][at, pos % K] = torch.where(live[:, None], s["xbc"], s["ring"][at, pos % K])
    return dict(y=torch.where(live[:, None, None], y, 0.0).to(s["y"].dtype), states=s["states"], ring=s["ring"])


# ---------------------------------------------------------------------------------------------------------------------
# the package's operators
# ---------------------------------------------------------------------------------------------------------------------

def _own_norm(s):
    from selective_state_space_04_gb300 import ssd
    if "values" not in s:
        out, residual = ssd.add_rmsnorm_fwd(s["x"], s["w"], s["residual"], eps=s["eps"])
        return dict(out=out) if residual is None else dict(out=out, residual=residual)
    q, scale, residual = ssd.add_rmsnorm_q8_fwd(s["x"], s["w"], s["residual"], eps=s["eps"])
    values = torch.mul(q, scale[:, None], out=s["values"])   # what the 8 bits stand for
    return dict(values=values, scale=scale) if residual is None else dict(values=values, scale=scale, residual=residual)


def _own_norm_grad(s):
    from selective_state_space_04_gb300 import ssd
    dx, dweight = ssd.add_rmsnorm_bwd(s["h"], s["w"], s["dout"], s["dres"], eps=s["eps"])
    return dict(dx=dx, dweight=dweight)


def _own_matmul(s):
    from selective_state_space_04_gb300 import ssd
    return dict(y=ssd.q8_matmul(s["a"], s["a_scale"], s["packed"], s["w_scale"], dtype=s["dtype"]))


def _own_gate_matmul(s):
    from selective_state_space_04_gb300 import ssd
    q, scale = ssd.gated_rmsnorm_q8_fwd(s["y"], s["z"], s["nw"], s["eps"])
    return dict(y=ssd.q8_matmul(q, scale, s["packed"], s["w_scale"], dtype=s["dtype"]))


def _own_step(s):
    from selective_state_space_04_gb300 import ssd
    y = ssd.conv_scan_step(s["xbc"], s["ring"], s["cw"], s["cb"], s["dt"], s["dt_bias"], s["A_log"], s["D"], s["states"], s["slots"],
                           s["positions"], ngroups=s["case"]["groups"], y=s["y"])
    return dict(y=y, states=s["states"], ring=s["ring"])


def run(state):
    if own:
        return {"norm": _own_norm, "norm_grad": _own_norm_grad, "matmul": _own_matmul, "gate_matmul": _own_gate_matmul,
                "step": _own_step}[state["op"]](state)
    return {"norm": _run_norm, "norm_grad": _run_norm_grad, "matmul": _run_matmul, "gate_matmul": _run_gate_matmul,
            "step": _run_step}[state["op"]](state)


# ---------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------------

def work(case):
    c = case
    size = {"bf16": 2, "f32": 4, "none": 0}
    if c["op"] in ("norm", "norm_grad"):
        n, D, es, rs = c["rows"], c["dim"], size[c["dtype"]], size[c["residual"]]
        if c["op"] == "norm":
            # x, the residual in and out, the result (8 bits with a scale) and what its values are returned in
            moved = es + 2 * rs + (3 if c["q8"] else es)
            return {"bytes": n * D * moved + 4 * D + (4 * n if c["q8"] else 0), "flops": n * D * (8 if c["q8"] else 5)}
        # the sum, the gradients of the outputs, the gradient
        return {"bytes": n * D * ((rs or es) + es + rs + (rs or es)) + 8 * D, "flops": n * D * 11}
    if c["op"] in ("matmul", "gate_matmul"):
        M, N, K, es = c["tokens"], c["features"], c["inner"], size[c["dtype"]]
        taken = M * K if c["op"] == "matmul" else M * K * 2 * es + 4 * K
        return {"bytes": taken + N * K + M * N * es + 4 * (M + N), "flops": 2 * M * N * K}
    n, rows, H, P, N, C, K, es = c["nseq"], c["nseq"] + c["padding"], c["heads"], c["headdim"], c["dstate"], _channels(c), c["taps"], size[c["dtype"]]
    state = H * P * N * 4
    nbytes = n * state + (n - c["fresh"]) * state + n * C * es * 2 + (n - c["fresh"]) * (K - 1) * C * es + n * H * es + rows * (H * P * es + 8)
    return {"bytes": nbytes + C * (K + 1) * 4 + 12 * H, "flops": n * (5 * H * P * N + 2 * K * C)}


# ---------------------------------------------------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------------------------------------------------

def _normalized(h, w, eps):
    return h / (h.square().sum(1, keepdim=True) / h.shape[1] + eps).sqrt() * w.double()


def _whole(v):
    """The 8-bit values that rows of v are rounded to, and their scales."""
    scale = v.abs().max(1).values / 127
    return (v / torch.where(scale == 0, 1, scale)[:, None]).round(), scale


def _exact_norm(c, seed):
    s = _prepare_norm(c, seed)
    h = s["x"].double() + (0 if s["residual"] is None else s["residual"].double())
    got = {} if s["residual"] is None else dict(residual=h)
    v = _normalized(h, s["w"], s["eps"])
    if not c["q8"]:
        return dict(got, out=v)
    q, scale = _whole(v)
    return dict(got, values=q * scale[:, None], scale=scale)


def _exact_norm_grad(c, seed):
    s = _prepare_norm(c, seed)
    h, d, w = s["h"].double(), s["dout"].double(), s["w"].double()
    m = h.square().sum(1, keepdim=True) / c["dim"] + s["eps"]
    dh = d * w / m.sqrt() - h * (d * w * h).sum(1, keepdim=True) / (c["dim"] * m * m.sqrt())
    return dict(dx=dh if s["dres"] is None else dh + s["dres"].double(), dweight=torch.einsum("td,td->d", d, h / m.sqrt()))


def _product(q, w):
    """q w^T in 64 bits, a few thousand rows of w at a time."""
    return torch.cat([q @ part.double().t() for part in w.split(4096)], 1)


def _exact_matmul(c, seed):
    s = _prepare_matmul(c, seed)
    if c["tokens"] * c["features"] * c["inner"] > 4e12:
        return None
    return dict(y=_product(s["a"].double(), s["w"]) * s["a_scale"].double()[:, None] * s["w_scale"].double())


def _exact_gate_matmul(c, seed):
    s = _prepare_gate_matmul(c, seed)
    z = s["z"].double()
    q, scale = _whole(_normalized(s["y"].double(), s["nw"], s["eps"]) * z * torch.sigmoid(z))
    return dict(y=_product(q, s["w"]) * scale[:, None] * s["w_scale"].double())


def _exact_step(c, seed):
    s = _prepare_step(c, seed)
    H, P, N, G, K = c["heads"], c["headdim"], c["dstate"], c["groups"], c["taps"]
    xbc, ring, states = s["xbc"].double(), s["ring"].double(), s["states"].double()
    cw, cb, dt_bias, D = s["cw"].double(), s["cb"].double(), s["dt_bias"].double(), s["D"].double()
    rate = s["A_log"].double().exp()
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
    head_group = torch.arange(H, device="cuda") // (H // G)
    for i, (slot, t) in enumerate(zip(s["slots"].tolist(), s["positions"].tolist())):
        if slot < 0:
            continue
        u = cb + cw[:, 0] * xbc[i]
        for back in range(1, min(K - 1, t) + 1):
            u = u + cw[:, back] * ring[slot, (t - back) % K]
        u = u * torch.sigmoid(u)
        x, B, C = u[:H * P].view(H, P), u[H * P:H * P + G * N].view(G, N)[head_group], u[H * P + G * N:].view(G, N)[head_group]
        dt = torch.logaddexp(s["dt"][i].double() + dt_bias, torch.zeros((), dtype=torch.float64, device="cuda"))
        h = torch.einsum("h,hp,hn->hpn", dt, x, B)
        if t > 0:
            h = h + torch.exp(-dt * rate)[:, None, None] * states[slot]
        y[i] = torch.einsum("hpn,hn->hp", h, C) + D[:, None] * x
        states[slot] = h
        ring[slot, t % K] = xbc[i]
    return dict(y=y, states=states, ring=ring)


def exact(case, seed):
    return {"norm": _exact_norm, "norm_grad": _exact_norm_grad, "matmul": _exact_matmul, "gate_matmul": _exact_gate_matmul,
            "step": _exact_step}[case["op"]](case, seed)
