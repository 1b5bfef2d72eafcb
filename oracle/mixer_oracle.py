"""fp64 oracle of the mixer operators beside the Swimba layer: linear attention with a decay for each
head (forward, step, gradients) and the norms around a block (forward, gradients). Plain numpy, token by
token and row by row; test infrastructure only.

Beside every value the functions return what its tolerance is made of: ``once``, the sum of the absolute
values that the bf16 kernels round to bf16 before adding them up (the masked scores of a chunk times the
values, the query times the carried state), and ``mag``, the sum of the absolute products themselves,
which fp32 rounding is relative to.
"""
from __future__ import annotations

import numpy as np

CHUNK = 128


def _walk(x, y, w, M0, gamma, rev, s_inter, s_u):
    """One head's recurrence in role form: x, y [n, dx], w [n, dw], M0 [dx, dw]; out [n, dw], M after."""
    n = x.shape[0]
    M = M0.copy()
    out = np.zeros((n, w.shape[1]))
    for t in range(n - 1, -1, -1) if rev else range(n):
        u = s_u * np.outer(y[t], w[t])
        if rev:
            G = M + u
            out[t] = s_inter * (x[t] @ G)
            M = gamma * G
        else:
            M = gamma * M + u
            out[t] = s_inter * (x[t] @ M)
    return out, M


def _once(x, y, w, M0, gamma, rev, s_inter, s_u):
    """Per output: Σ over its chunk of |score| |value|, plus |decay| Σ |x| |M at the chunk's start|."""
    n = x.shape[0]
    got = np.zeros((n, w.shape[1]))
    M = M0.copy()
    starts = list(range(0, n, CHUNK))
    for t0 in reversed(starts) if rev else starts:
        t1 = min(t0 + CHUNK, n)
        i = np.arange(t1 - t0)
        e = (i[None, :] - i[:, None]) if rev else (i[:, None] - i[None, :])
        D = np.where(e >= 0, gamma ** np.maximum(e, 0), 0.0)
        P = (x[t0:t1] @ y[t0:t1].T) * D * s_u * s_inter
        into = gamma ** ((t1 - t0 - 1 - i) if rev else (i + 1)) * s_inter
        got[t0:t1] = np.abs(P) @ np.abs(w[t0:t1]) + into[:, None] * (np.abs(x[t0:t1]) @ np.abs(M))
        _, M = _walk(x[t0:t1], y[t0:t1], w[t0:t1], M, gamma, rev, s_inter, s_u)
    return got


class _Role:
    """All heads of one role: streams [B, L, heads, d] (shared heads repeated), states [B, H, dx, dw]."""

    def __init__(self, x, y, w, M0, gamma, lens, rev, s_inter, s_u):
        B, L, H, _ = x.shape
        self.out, self.once, self.mag = (np.zeros((B, L, H, w.shape[3])) for _ in range(3))
        self.M, self.M_mag = np.zeros((B, H, x.shape[3], w.shape[3])), np.zeros((B, H, x.shape[3], w.shape[3]))
        for b in range(B):
            n = int(np.clip(lens[b], 0, L))
            for h in range(H):
                a = (x[b, :n, h], y[b, :n, h], w[b, :n, h], M0[b, h], gamma[h], rev, s_inter, s_u)
                self.out[b, :n, h], self.M[b, h] = _walk(*a)
                self.once[b, :n, h] = _once(*a)
                m = tuple(np.abs(v) for v in a[:4]) + (gamma[h], rev, abs(s_inter), abs(s_u))
                self.mag[b, :n, h], self.M_mag[b, h] = _walk(*m)


def _inputs(q, k, v, log_decay, lens, S0):
    B, L, H, dk = q.shape
    group = H // k.shape[2]
    k, v = np.repeat(k, group, axis=2), np.repeat(v, group, axis=2)
    lens = np.full(B, L) if lens is None else lens
    S0 = np.zeros((B, H, dk, v.shape[3])) if S0 is None else S0
    # rows behind a sequence's end are never used, whatever they hold
    return q, k, v, np.exp(log_decay), lens, S0


def linattn_forward(q, k, v, log_decay, scale, lens=None, S0=None):
    """q [B, L, H, dk], k [B, L, Hkv, dk], v [B, L, Hkv, dv]: a _Role with out = o and M = the final state."""
    q, k, v, gamma, lens, S0 = _inputs(q, k, v, log_decay, lens, S0)
    return _Role(q, k, v, S0, gamma, lens, False, scale, 1.0)


def linattn_backward(q, k, v, log_decay, scale, g_o, lens=None, S0=None, g_S=None):
    """Roles of dq, dk, dv (dk and dv per query head: sum_shared adds them up); dv's M is dS0."""
    q, k, v, gamma, lens, S0 = _inputs(q, k, v, log_decay, lens, S0)
    T = lambda m: np.swapaxes(m, 2, 3)
    g_S = np.zeros_like(S0) if g_S is None else g_S
    dq = _Role(g_o, v, k, T(S0), gamma, lens, False, scale, 1.0)
    dk = _Role(v, g_o, q, T(g_S), gamma, lens, True, 1.0, scale)
    dv = _Role(k, q, g_o, g_S, gamma, lens, True, 1.0, scale)
    return dq, dk, dv


def sum_shared(a, n_kv_heads):
    """[B, L, H, d] summed over the query heads that share a key/value head: [B, L, Hkv, d]."""
    B, L, H, d = a.shape
    return a.reshape(B, L, n_kv_heads, H // n_kv_heads, d).sum(3)


# ---- norms around a block -----------------------------------------------------------------------------

def _sigmoid(z):
    return 1 / (1 + np.exp(-z))


def _over_groups(a, groups):
    """Mean over each group, back at full width."""
    g = a.reshape(a.shape[0], groups, -1)
    return np.repeat(g.mean(-1), g.shape[2], axis=1)


def block_norm_forward(y, z, w_post, res, w_pre, groups=1, eps=1e-5, gate_last=False, res_scale=1.0, out_scale=1.0):
    """Rows [R, W]; any of z, w_post, res, w_pre (and y, with res) may be None. Returns a dict with h, n (None
    without w_pre), the intermediate values the gradients use, and h_mag."""
    f = dict(gate=None if z is None else z * _sigmoid(z))
    p = np.zeros_like(res) if y is None else y.copy()
    if z is not None and not gate_last:
        p = p * f["gate"]
    f["r"] = None
    if w_post is not None:
        f["r"] = 1 / np.sqrt(_over_groups(p * p, groups) + eps)
        f["hat"] = p * f["r"]
        p = f["hat"] * w_post
    else:
        f["hat"] = p
    f["p"] = p
    if z is not None and gate_last:
        p = p * f["gate"]
    f["h"] = out_scale * p
    f["h_mag"] = np.abs(f["h"])
    if res is not None:
        f["h"] = f["h"] + res_scale * res
        f["h_mag"] = f["h_mag"] + np.abs(res_scale * res)
    f["n"], f["n_mag"] = None, None
    if w_pre is not None:
        f["rh"] = 1 / np.sqrt((f["h"] ** 2).mean(-1, keepdims=True) + eps)
        f["hh"] = f["h"] * f["rh"]
        f["n"] = f["hh"] * w_pre
        # h's rounding passes through the row's scale too
        hm = f["h_mag"] * f["rh"]
        f["hh_mag"] = hm + np.abs(f["hh"]) * (np.abs(f["hh"]) * hm).mean(-1, keepdims=True)
        f["n_mag"] = f["hh_mag"] * np.abs(w_pre)
    return f


def block_norm_backward(y, z, w_post, res, w_pre, g_h, g_n, groups=1, eps=1e-5, gate_last=False, res_scale=1.0,
                        out_scale=1.0):
    """Reverse mode of block_norm_forward: {name: (gradient, sum of the absolute terms it is made of)}."""
    f = block_norm_forward(y, z, w_post, res, w_pre, groups, eps, gate_last, res_scale, out_scale)
    out = {}
    dh = np.zeros_like(f["h"]) if g_h is None else g_h.copy()
    dm = np.abs(dh)
    if w_pre is not None:
        gw = g_n * w_pre
        gm = np.abs(gw)
        dh = dh + f["rh"] * (gw - f["hh"] * (gw * f["hh"]).mean(-1, keepdims=True))
        dm = dm + f["rh"] * (gm + f["hh_mag"] * (gm * f["hh_mag"]).mean(-1, keepdims=True)) * 2
        out["dw_pre"] = (g_n * f["hh"]).sum(0), (np.abs(g_n) * f["hh_mag"]).sum(0)
    if res is not None:
        out["dres"] = res_scale * dh, np.abs(res_scale) * dm
    d, dm = out_scale * dh, np.abs(out_scale) * dm
    if y is None:
        return out
    if z is not None:
        sg = _sigmoid(z)
        slope = sg * (1 + z * (1 - sg))
        slope_mag = sg * (1 + np.abs(z))
    if z is not None and gate_last:
        out["dz"] = d * f["p"] * slope, dm * np.abs(f["p"]) * slope_mag
        d, dm = d * f["gate"], dm * np.abs(f["gate"])
    if w_post is not None:
        ah = np.abs(f["hat"])
        out["dw_post"] = (d * f["hat"]).sum(0), (dm * ah).sum(0)
        gw, gm = d * w_post, dm * np.abs(w_post)
        d = f["r"] * (gw - f["hat"] * _over_groups(gw * f["hat"], groups))
        dm = f["r"] * (gm + ah * _over_groups(gm * ah, groups)) * 2
    if z is not None and not gate_last:
        out["dz"] = d * y * slope, dm * np.abs(y) * slope_mag
        d, dm = d * f["gate"], dm * np.abs(f["gate"])
    out["dy"] = d, dm
    return out
