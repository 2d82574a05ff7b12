"""fp64 oracle for the attention layers of hybrid stacks -- TEST INFRASTRUCTURE.

Only ``tests/`` use it; the product library never imports it.

* :func:`plan_step` -- block tables, positions and slots of one serving step,
  request after request.
* :func:`qk_norm_rope`, :func:`qk_norm_rope_grad` -- per-head RMSNorm of
  queries and keys with the rotary position, and its gradients.
* :func:`paged_attention` -- attention of new tokens over a paged cache, row by
  row, with the size of the sums behind each output (for derived tolerances).
"""
from __future__ import annotations

import numpy as np

from .neighbors import _f64


def plan_step(lens, new_lens, table, ring, ring_pos, page_size, max_tokens):
    """One step's plan.  ``table`` and ``ring`` are not changed; returns a dict with
    their new contents beside the plan's arrays."""
    table, ring = np.array(table), np.array(ring)
    given = ring.copy()
    head, tail = int(ring_pos[0]), int(ring_pos[1])
    cap, free = len(ring), min(max(tail - head, 0), len(ring))
    first, at_tail, asked_tok, asked_pg = head, tail, 0, 0
    out = dict(lens=[], granted=[], start=[0], positions=[], token_req=[], slots=[])
    back = refused = 0
    for r, (n, m) in enumerate(zip((max(int(v), 0) for v in lens), (int(v) for v in new_lens))):
        held, got = -(-n // page_size), 0
        if m < 0:
            for j in range(min(held, table.shape[1])):
                ring[at_tail % cap] = table[r, j]
                at_tail += 1
                back += 1
        elif m > 0:
            fits = n + m <= table.shape[1] * page_size
            want = -(-(n + m) // page_size) - held
            if fits:
                asked_tok, asked_pg = asked_tok + m, asked_pg + want
            if fits and asked_tok <= max_tokens and asked_pg <= free:
                got = m
                for j in range(want):
                    table[r, held + j] = given[first % cap]
                    first += 1
                for p in range(n, n + m):
                    out["positions"].append(p)
                    out["token_req"].append(r)
                    out["slots"].append(int(table[r, p // page_size]) * page_size + p % page_size)
            else:
                refused += 1
        out["lens"].append(0 if m < 0 else n + got)
        out["granted"].append(got)
        out["start"].append(out["start"][-1] + got)
    for k in ("positions", "token_req", "slots"):
        out[k] += [-1] * (max_tokens - len(out[k]))
    out = {k: np.array(v, dtype=np.int64) for k, v in out.items()}
    out["ring_pos"] = np.array([first, at_tail])
    out["counts"] = np.array([out["start"][-1], first - head, back, refused])
    out["table"], out["ring"] = table, ring
    return out


def _pair_index(D, R, interleaved):
    """Element numbers of the first and second members of the rotated pairs."""
    i = np.arange(R // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)


def _angles(cos, sin, positions):
    cos, sin, positions = _f64(cos), _f64(sin), np.asarray(positions, dtype=np.int64)
    live = (positions >= 0) & (positions < len(cos))
    at = np.where(live, positions, 0)
    if len(cos) == 0:
        z = np.zeros((len(positions), 1, cos.shape[1]))
        return z, z, live
    return cos[at][:, None, :], sin[at][:, None, :], live


def qk_norm_rope(x, weight, cos, sin, positions, eps, interleaved):
    """Returns ``(y, size)``: the outputs [T,H,D], zero for padding tokens, and the
    magnitude of the terms behind each row ([T,H,1])."""
    x = _f64(x)
    D = x.shape[-1]
    w = np.ones(D) if weight is None else _f64(weight)
    c, s, live = _angles(cos, sin, positions)
    n = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    y = n.copy()
    ia, ib = _pair_index(D, 2 * c.shape[-1], interleaved)
    y[..., ia] = n[..., ia] * c - n[..., ib] * s
    y[..., ib] = n[..., ib] * c + n[..., ia] * s
    keep = live[:, None, None]
    return np.where(keep, y, 0.0), np.where(keep, 2 * np.abs(n).max(-1, keepdims=True), 0.0)


def qk_norm_rope_grad(x, weight, cos, sin, positions, dy, eps, interleaved):
    """Returns ``(dx, dweight, size of dx's terms [T,H,1], size of dweight's [D])``."""
    x, dy = _f64(x), _f64(dy)
    D = x.shape[-1]
    w = np.ones(D) if weight is None else _f64(weight)
    c, s, live = _angles(cos, sin, positions)
    g = dy.copy()
    ia, ib = _pair_index(D, 2 * c.shape[-1], interleaved)
    g[..., ia] = dy[..., ia] * c + dy[..., ib] * s
    g[..., ib] = dy[..., ib] * c - dy[..., ia] * s
    keep = live[:, None, None]
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    gw = g * w
    dx = np.where(keep, r * (gw - x * r * r * (gw * x).mean(-1, keepdims=True)), 0.0)
    terms = np.where(keep, g * x * r, 0.0)
    g_abs = np.abs(gw).max(-1, keepdims=True)
    size = np.where(keep, r * (2 * g_abs + np.abs(x).max(-1, keepdims=True) * r * r * np.abs(gw * x).mean(-1, keepdims=True)), 0.0)
    return dx, terms.sum((0, 1)), size, np.abs(terms).sum((0, 1))


def paged_attention(q, k_cache, v_cache, table, positions, start, scale, window):
    """Returns ``(out, lse, size)``; ``size[i,h]`` [D] is sum_t p_t |v_t|."""
    q, kc, vc = _f64(q), _f64(k_cache), _f64(v_cache)
    npages, ps, hk, D = kc.shape
    rows, H, _ = q.shape
    table, positions = np.asarray(table), np.asarray(positions).astype(np.int64)
    req = np.full(rows, -1)
    if start is None:
        req = np.arange(rows)
    else:
        for r in range(len(start) - 1):
            req[start[r]:start[r + 1]] = r
    out, lse, size = np.zeros((rows, H, D)), np.full((rows, H), -np.inf), np.zeros((rows, H, D))
    for i in range(rows):
        if req[i] < 0 or positions[i] < 0:
            continue
        first = max(0, positions[i] - window + 1) if window else 0
        t = np.arange(first, min(positions[i] + 1, table.shape[1] * ps))
        page = table[req[i], t // ps]
        ok = (page >= 0) & (page < npages)
        t, page = t[ok], page[ok]
        if len(t) == 0:
            continue
        for h in range(H):
            g = h // (H // hk)
            s = scale * (kc[page, t % ps, g] @ q[i, h])
            e = np.exp(s - s.max())
            p = e / e.sum()
            out[i, h] = p @ vc[page, t % ps, g]
            size[i, h] = p @ np.abs(vc[page, t % ps, g])
            lse[i, h] = s.max() + np.log(e.sum())
    return out, lse, size
