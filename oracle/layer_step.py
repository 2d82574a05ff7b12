"""fp64 oracles of one layer's step around the scan: the residual's addition with RMSNorm, its gradients, rows of 8-bit
whole numbers, their products, and the conv and scan for single tokens on a pool of states.  numpy, from the formulas."""
import numpy as np


def _f64(a):
    """A torch tensor or array as fp64."""
    return a.detach().cpu().double().numpy() if hasattr(a, "detach") else np.asarray(a, dtype=np.float64)


def silu(v):
    return v * 0.5 * (1.0 + np.tanh(0.5 * v))


def inv_rms(h, eps):
    m = (h * h).mean(-1, keepdims=True) + eps
    return np.where(m > 0, 1.0 / np.sqrt(np.where(m > 0, m, 1.0)), 0.0)


def add_rmsnorm(x, weight, residual, eps, gate=None):
    """(out, h): h = x + residual, out = h / rms(h) * weight (* SiLU(gate))."""
    h = _f64(x) + (0.0 if residual is None else _f64(residual))
    out = h * inv_rms(h, eps) * _f64(weight)
    return (out if gate is None else out * silu(_f64(gate))), h


def add_rmsnorm_grad(h, weight, dout, dresidual, eps):
    """(dx, dweight, magnitude of dx's terms, magnitude of dweight's terms)."""
    h, w, d = _f64(h), _f64(weight), _f64(dout)
    r = inv_rms(h, eps)
    g = d * w
    pull = h * r * r * (g * h).mean(-1, keepdims=True)
    res = np.zeros_like(h) if dresidual is None else _f64(dresidual)
    dw = d * h * r
    size = r * (np.abs(g) + np.abs(h) * r * r * np.abs(g * h).mean(-1, keepdims=True)) + np.abs(res)
    return r * (g - pull) + res, dw.sum(0), size, np.abs(dw).sum(0)


def q8_scale(v):
    """Scale of each row of v as 8-bit whole numbers."""
    return np.abs(v).max(-1) / 127.0


def q8_matmul(a, w):
    """The sums of the products, as int64 [tokens, channels]."""
    return a.cpu().numpy().astype(np.int64) @ w.cpu().numpy().astype(np.int64).T


def conv_scan_step(xbc, ring, weight, bias, dt_raw, dt_bias, A_log, D, states, slots, positions, G):
    """(y, ring, states, magnitude of y's terms) after one token of each row."""
    xbc, ring, weight, states = _f64(xbc), _f64(ring).copy(), _f64(weight), _f64(states).copy()
    dt_raw, dt_bias, A, D = _f64(dt_raw), _f64(dt_bias), -np.exp(_f64(A_log)), _f64(D)
    S, H, P, N = states.shape
    C, K = weight.shape
    b = np.zeros(C) if bias is None else _f64(bias)
    y = np.zeros((xbc.shape[0], H, P))
    size = np.zeros_like(y)
    for i, (s, t) in enumerate(zip(np.asarray(slots.cpu()), np.asarray(positions.cpu()))):
        if s < 0 or s >= S or t < 0:
            continue
        taps = np.zeros((K, C))   # the inputs 0 .. K-1 steps back
        for j in range(K):
            if j == 0:
                taps[0] = xbc[i]
            elif t >= j:
                taps[j] = ring[s, (t - j) % K]
        u = silu(b + (taps.T * weight).sum(1))
        x, B, Cm = u[:H * P].reshape(H, P), u[H * P:H * P + G * N].reshape(G, N), u[H * P + G * N:].reshape(G, N)
        B, Cm = np.repeat(B, H // G, 0), np.repeat(Cm, H // G, 0)
        z = dt_raw[i] + dt_bias
        dt = np.maximum(z, 0) + np.log1p(np.exp(-np.abs(z)))
        old = states[s] if t > 0 else np.zeros((H, P, N))
        h = np.exp(dt * A)[:, None, None] * old + (dt[:, None] * x)[:, :, None] * B[:, None, :]
        y[i] = np.einsum("hpn,hn->hp", h, Cm) + D[:, None] * x
        size[i] = np.einsum("hpn,hn->hp", np.abs(h), np.abs(Cm)) + np.abs(D[:, None] * x)
        states[s] = h
        ring[s, t % K] = xbc[i]
    return y, ring, states, size
