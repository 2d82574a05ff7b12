"""Serving a small hybrid stack (state-space and attention layers, random weights) with continuous batching.

Every step takes whatever tokens its requests bring -- whole prompts, or the one token each generated last -- through the
library's operators: one :func:`ssd.paged_plan` for the step, then per attention layer the queries' and keys' norm and
rotary position into the paged cache (:func:`ssd.qk_norm_rope_fwd`) and the attention over it
(:func:`ssd.paged_attn_fwd`), and per state-space layer the scan or, for single tokens, its decode step
(:func:`ssd.ssd_scan_fwd`).  Requests join and leave between steps; their pages go back to the pool.

``--layers`` takes one letter per layer: s and a as above, m a whole state-space layer with its norm, short convolution,
gate and projections in 8-bit integers (:func:`ssd.add_rmsnorm_q8_fwd`, :func:`ssd.q8_matmul`,
:func:`ssd.conv_scan_step` for single tokens, :func:`ssd.gated_rmsnorm_q8_fwd`).

    python examples/hybrid_decode.py --requests 8 --new-tokens 24
    python examples/hybrid_decode.py --layers mama
"""
from __future__ import annotations

import argparse
import os
import sys
import time
from dataclasses import dataclass

import torch

if __package__ in (None, ""):
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from selective_state_space_04_gb300 import ssd


@dataclass(frozen=True)
class Config:
    vocab: int = 512
    d_model: int = 256
    layers: str = "sasa"       # s: state space, a: attention, m: state space with conv, gate and 8-bit projections
    nheads: int = 8            # state-space heads of 64, state size 128, one group
    headdim: int = 64
    dstate: int = 128
    taps: int = 4              # of the short convolution (m)
    q_heads: int = 8           # attention
    kv_heads: int = 2
    attn_dim: int = 64
    window: int = 0
    page_size: int = 16
    max_len: int = 512
    dtype: torch.dtype = torch.bfloat16


def make_weights(c: Config, seed: int = 0) -> dict:
    g = torch.Generator(device="cpu").manual_seed(seed)

    def mat(rows, cols, dtype=c.dtype):
        return (torch.randn(rows, cols, generator=g) / cols ** 0.5).to("cuda", dtype)

    w = dict(embed=mat(c.vocab, c.d_model), head=mat(c.vocab, c.d_model), layers=[])
    for kind in c.layers:
        if kind == "s":
            inner = c.nheads * c.headdim
            w["layers"].append(dict(
                w_in=mat(inner + 2 * c.dstate, c.d_model), w_dt=mat(c.nheads, c.d_model), out=mat(c.d_model, inner),
                dt_bias=torch.full((c.nheads,), -3.0, device="cuda"),
                A_log=torch.linspace(0.0, 2.0, c.nheads).cuda(), D=torch.ones(c.nheads, device="cuda")))
        elif kind == "m":
            inner = c.nheads * c.headdim
            C = inner + 2 * c.dstate
            w["layers"].append(dict(
                norm=torch.ones(c.d_model, device="cuda"), w_in=quantized(mat(inner + C + c.nheads, c.d_model, torch.float32)),
                conv=mat(C, c.taps, torch.float32), conv_bias=torch.zeros(C, device="cuda"),
                dt_bias=torch.full((c.nheads,), -3.0, device="cuda"), A_log=torch.linspace(0.0, 2.0, c.nheads).cuda(),
                D=torch.ones(c.nheads, device="cuda"), gate_norm=torch.ones(inner, device="cuda"),
                out=quantized(mat(c.d_model, inner, torch.float32))))
        else:
            w["layers"].append(dict(
                w_qkv=mat((c.q_heads + 2 * c.kv_heads) * c.attn_dim, c.d_model), out=mat(c.d_model, c.q_heads * c.attn_dim),
                q_weight=torch.ones(c.attn_dim, device="cuda"), k_weight=torch.ones(c.attn_dim, device="cuda")))
    return w


def quantized(w):
    """A weight as 8-bit integers with a scale per output channel, in the order that ssd.q8_matmul reads."""
    scale = w.abs().amax(1) / 127.0
    rows = torch.where(scale > 0, scale, 1.0)[:, None]   # (a channel of zeros stays zeros, with scale 0)
    return ssd.q8_pack_weight(torch.clamp(torch.round(w / rows), -127, 127).to(torch.int8)), scale


def rms(x):
    return (x.float() * torch.rsqrt(x.float().pow(2).mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


class Server:
    """Holds up to ``slots`` requests.  ``step`` runs their tokens and returns each request's next-token logits."""

    def __init__(self, c: Config, w: dict, slots: int, pages: int):
        self.c, self.w, self.slots = c, w, slots
        dev = dict(device="cuda")
        self.max_pages = -(-c.max_len // c.page_size)
        self.lens = torch.zeros(slots, dtype=torch.int32, **dev)
        self.block_table = torch.full((slots, self.max_pages), -1, dtype=torch.int32, **dev)
        self.free_ring = torch.arange(pages, dtype=torch.int32, **dev)
        self.ring_pos = torch.tensor([0, pages], dtype=torch.int64, **dev)
        self.cos, self.sin = ssd.rope_table(c.max_len, c.attn_dim)
        self.held = [0] * slots   # tokens of each slot's request so far
        self.state = []
        for kind in c.layers:
            if kind == "s":
                self.state.append(torch.zeros(slots, c.nheads, c.headdim, c.dstate, **dev))
            elif kind == "m":   # the convolution's inputs and the states; what is left of another request is not read
                C = c.nheads * c.headdim + 2 * c.dstate
                self.state.append((torch.zeros(slots, c.taps, C, dtype=c.dtype, **dev),
                                   torch.zeros(slots, c.nheads, c.headdim, c.dstate, **dev)))
            else:
                shape = (pages, c.page_size, c.kv_heads, c.attn_dim)
                self.state.append((torch.zeros(shape, dtype=c.dtype, **dev), torch.zeros(shape, dtype=c.dtype, **dev)))

    def step(self, work: dict, finished=()) -> torch.Tensor:
        """``work``: slot -> its new tokens (a list); ``finished``: slots whose requests are done.  Returns logits
        [slots, vocab] (rows of slots without work are not meaningful)."""
        c = self.c
        new = [0] * self.slots
        for s in finished:
            new[s] = -1
        for s, toks in work.items():
            new[s] = len(toks)
        order = sorted(work)
        tokens = [t for s in order for t in work[s]]
        n = len(tokens)
        plan = ssd.paged_plan(self.lens, torch.tensor(new, dtype=torch.int32, device="cuda"), self.block_table, self.free_ring,
                              self.ring_pos, page_size=c.page_size, max_tokens=n)
        if int(plan["counts"][3]):   # (a scheduler would keep such requests waiting)
            raise RuntimeError("no room in the cache for the step's tokens")
        self.lens, self.ring_pos = plan["lens"], plan["ring_pos"]
        for s in finished:
            self.held[s] = 0
            for st in self.state:
                if isinstance(st, torch.Tensor):
                    st[s].zero_()
        if n == 0:
            return None
        ends, at = {}, 0
        for s in order:
            ends[s] = (at, at + len(work[s]))
            at += len(work[s])
        x = self.w["embed"][torch.tensor(tokens, device="cuda")]
        for kind, lw, st in zip(c.layers, self.w["layers"], self.state):
            if kind == "m":
                x = self._layer8(lw, st, x, ends, plan)
                continue
            h = rms(x)
            x = x + (self._scan(lw, st, h, ends) if kind == "s" else self._attention(lw, st, h, plan))
        for s in work:
            self.held[s] += len(work[s])
        last = torch.tensor([ends[s][1] - 1 if s in ends else 0 for s in range(self.slots)], device="cuda")
        return rms(x)[last].float() @ self.w["head"].float().t()

    def _attention(self, lw, cache, h, plan):
        c, n = self.c, h.shape[0]
        qkv = (h @ lw["w_qkv"].t()).view(n, c.q_heads + 2 * c.kv_heads, c.attn_dim)
        q, k, v = qkv.split((c.q_heads, c.kv_heads, c.kv_heads), dim=1)
        q, _ = ssd.qk_norm_rope_fwd(q, k, lw["q_weight"], lw["k_weight"], self.cos, self.sin, plan["positions"], v=v,
                                    k_cache=cache[0], v_cache=cache[1], slots=plan["slots"], return_k=False)
        out, _ = ssd.paged_attn_fwd(q, *cache, self.block_table, plan["positions"], plan["start"], window=c.window,
                                    return_lse=False)
        return out.flatten(1) @ lw["out"].t()

    def _scan(self, lw, state, h, ends):
        c = self.c
        inner = c.nheads * c.headdim
        xbc, dt = h @ lw["w_in"].t(), (h @ lw["w_dt"].t()).float()
        y = torch.empty(h.shape[0], inner, dtype=c.dtype, device="cuda")
        single = [s for s, (a, b) in ends.items() if b == a + 1]
        groups = [(torch.tensor(single, device="cuda"), torch.tensor([ends[s][0] for s in single], device="cuda")[:, None])] if single else []
        groups += [(torch.tensor([s], device="cuda"), torch.arange(a, b, device="cuda")[None]) for s, (a, b) in ends.items() if b > a + 1]
        for slots, rows in groups:   # rows [requests, tokens]
            u, B, L = xbc[rows], *rows.shape
            xs = u[..., :inner].reshape(B, L, c.nheads, c.headdim).contiguous()
            Bm, Cm = (u[..., inner + i * c.dstate:inner + (i + 1) * c.dstate].reshape(B, L, 1, c.dstate).contiguous() for i in (0, 1))
            yy, final = ssd.ssd_scan_fwd(xs, dt[rows].contiguous(), lw["dt_bias"], lw["A_log"], Bm, Cm, lw["D"],
                                         state[slots].contiguous(), chunk=64)
            state[slots] = final
            y[rows.reshape(-1)] = yy.reshape(B * L, inner)
        return y @ lw["out"].t()


    def _layer8(self, lw, state, x, ends, plan):
        """norm -> 8-bit input projection -> conv and scan -> gated norm -> 8-bit output projection, and the residual."""
        c, (ring, states) = self.c, state
        H, P, N = c.nheads, c.headdim, c.dstate
        inner, C = H * P, H * P + 2 * N
        q, scale, _ = ssd.add_rmsnorm_q8_fwd(x, lw["norm"])
        proj = ssd.q8_matmul(q, scale, *lw["w_in"], dtype=c.dtype)
        z, xbc, dt = proj[:, :inner], proj[:, inner:inner + C], proj[:, inner + C:]
        # single tokens together; a row of a prompt is padding there
        lone = torch.full((x.shape[0],), -1, dtype=torch.int32)
        for s, (a, b) in ends.items():
            if b == a + 1:
                lone[a] = s
        y = ssd.conv_scan_step(xbc, ring, lw["conv"], lw["conv_bias"], dt, lw["dt_bias"], lw["A_log"], lw["D"], states,
                               lone.cuda(), plan["positions"], ngroups=1)
        for s, (a, b) in ends.items():
            if b > a + 1:   # several tokens of one request: the conv and scan over them, from what is carried
                held, before = self.held[s], None
                if held:
                    at = torch.arange(held - c.taps + 1, held, device="cuda")
                    before = torch.where((at >= 0)[:, None], ring[s, at % c.taps], 0)[None].contiguous()
                xs, Bm, Cm, carried = ssd.conv1d_silu_fwd(xbc[None, a:b].contiguous(), lw["conv"], lw["conv_bias"], before,
                                                          nheads=H, headdim=P, ngroups=1, dstate=N)
                yy, final = ssd.ssd_scan_fwd(xs, dt[None, a:b].float().contiguous(), lw["dt_bias"], lw["A_log"], Bm, Cm,
                                             lw["D"], states[s:s + 1].contiguous() if held else None, chunk=64)
                y[a:b] = yy[0]
                states[s] = final[0]
                ssd.conv_ring_store(ring, carried, torch.tensor([s], device="cuda"), torch.tensor([held + b - a], device="cuda"))
        q, scale = ssd.gated_rmsnorm_q8_fwd(y.view(-1, inner), z, lw["gate_norm"])
        return x + ssd.q8_matmul(q, scale, *lw["out"], dtype=c.dtype)


def generate(c: Config, w: dict, prompts: list, new_tokens: int, slots: int, pages: int):
    """Greedy continuations of ``prompts``, ``slots`` of them at a time.  Returns the token lists."""
    server = Server(c, w, slots, pages)
    waiting, running, done = list(enumerate(prompts)), {}, {}
    finished, steps = [], 0
    while waiting or running:
        work = {s: [r[1][-1]] for s, r in running.items()}
        for s in range(slots):   # requests join where a slot is free (and has been given back)
            if waiting and s not in running and s not in finished:
                i, p = waiting.pop(0)
                running[s] = (i, list(p), len(p) + new_tokens)
                work[s] = list(p)
        logits = server.step(work, finished)
        finished, steps = [], steps + 1
        nxt = logits.argmax(-1).tolist() if work else []
        for s in list(work):
            i, toks, stop = running[s]
            toks.append(nxt[s])
            if len(toks) >= stop:
                done[i] = toks
                del running[s]
                finished.append(s)
    return [done[i] for i in range(len(prompts))], steps


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--new-tokens", type=int, default=24)
    ap.add_argument("--slots", type=int, default=4)
    ap.add_argument("--seed", type=int, default=0)
    ap.add_argument("--layers", default=Config.layers)
    a = ap.parse_args()
    c = Config(layers=a.layers)
    w = make_weights(c, a.seed)
    g = torch.Generator().manual_seed(a.seed + 1)
    prompts = [torch.randint(c.vocab, (int(n),), generator=g).tolist() for n in torch.randint(3, 120, (a.requests,), generator=g)]
    torch.cuda.synchronize()
    t = time.perf_counter()
    out, steps = generate(c, w, prompts, a.new_tokens, a.slots, pages=a.slots * (-(-c.max_len // c.page_size)))
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    for p, o in zip(prompts, out):
        print(f"prompt of {len(p):3d} tokens -> {o[len(p):]}")
    print(f"{steps} steps, {sum(len(o) for o in out)} tokens, {t * 1e3:.1f} ms")


if __name__ == "__main__":
    main()
