"""The mixer operators run together as a block uses them: norm before the block -> one in-projection to
[q | k | v] and the gate -> linear attention on the projection's columns -> gated group norm -> out-projection
-> residual and the next block's norm; the same for single tokens from the prompt's state; and the
backward of the gated norm feeding that of the attention. Every stage is checked against the fp64 oracle
on the inputs it really got, with that operator's own tolerance (see their tests)."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import mixer_oracle as M

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

B, L, H, KV, D = 2, 200, 4, 2, 64
DM = 192  # width of the residual stream
QKV = (H + 2 * KV) * D


@pytest.fixture(scope="module")
def S():
    from parameter_space_moe_swimba_b200 import swimba

    return swimba


def f64(x):
    return x.double().cpu().numpy()


def within(got, want, tol, what):
    off = np.abs(f64(got).reshape(want.shape) - want) - tol
    assert (off <= 1e-30).all(), (what, float(off.max()))


class Block:
    def __init__(self, S, dtype):
        g = torch.Generator(device="cuda")
        g.manual_seed(11)
        self.S, self.dtype = S, dtype
        self.t = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.half = 2.0 ** -8 if dtype == "bf16" else 0.0
        n = lambda *s: torch.randn(s, generator=g, device="cuda")
        self.W_in = (n(DM, QKV + H * D) * DM ** -0.5).to(self.t)
        self.W_out = (n(H * D, DM) * (H * D) ** -0.5).to(self.t)
        self.w_pre, self.w_post, self.w_next = (1 + 0.2 * n(w) for w in (DM, H * D, DM))
        self.g = -torch.exp2(torch.linspace(-1, -7, H, device="cuda"))
        self.x = n(B, L + 3, DM)  # the residual stream, fp32
        self.ws = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")

    def gemm(self, A, W, outs):
        S, (K, N) = self.S, W.shape
        rows = A.numel() // K
        split = outs[0].shape[-1]
        c1 = outs[1] if len(outs) > 1 else None
        S.check(S.swimba_block_gemm(S.dtype_code(self.dtype), rows, N, K, A, K, W, N, outs[0], split, c1, N - split, split,
                                    None, 0, self.ws, self.ws.numel()))
        want = f64(A).reshape(rows, K) @ f64(W)
        mag = np.abs(f64(A)).reshape(rows, K) @ np.abs(f64(W))
        tol = self.half * np.abs(want) + (K + 16) * 2.0 ** -24 * mag
        within(outs[0], want[:, :split], tol[:, :split], "gemm")
        if c1 is not None:
            within(c1, want[:, split:], tol[:, split:], "gemm, second part")

    def norm(self, y, z, w_post, res, w_pre, h, n, **kw):
        S = self.S
        like = h if h is not None else res if res is not None else y
        d = S.make_norm_dims(y if y is not None else n, like, eps=1e-5, **kw)
        S.check(S.swimba_block_norm_fwd(d, y, z, w_post, res, w_pre, h, n))
        rows = lambda x: None if x is None else f64(x).reshape(-1, x.shape[-1])
        vec = lambda x: None if x is None else f64(x)
        f = M.block_norm_forward(rows(y), rows(z), vec(w_post), rows(res), vec(w_pre), eps=float(np.float32(1e-5)), **kw)
        for got, k in ((h, "h"), (n, "n")):
            if got is not None:
                half = 2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0
                within(got, f[k], half * np.abs(f[k]) + (got.shape[-1] + 96) * 2.0 ** -24 * f[k + "_mag"], k)
        return f

    def mix(self, x, state):
        """x [B, T, DM] -> (residual stream behind the block, input of the next one); the state is replaced."""
        S, t = self.S, self.t
        T = x.shape[1]
        new = lambda *s: torch.empty(s, device="cuda", dtype=t)
        n = new(B, T, DM)
        self.norm(None, None, None, x, self.w_pre, None, n)
        qkv, z = new(B, T, QKV), new(B, T, H * D)
        self.gemm(n, self.W_in, (qkv, z))
        q, k, v = (p.unflatten(2, (-1, D)) for p in qkv.split([H * D, KV * D, KV * D], dim=2))
        o = new(B, T, H, D)
        d = S.make_linattn_dims(q, k, v, D ** -0.5)
        start = f64(state)
        if T == 1:
            S.check(S.swimba_linattn_step(d, q, k, v, self.g, state, o, state))
        else:
            ws = S.new_linattn_workspace(d, S.SWIMBA_OP_LINATTN_FWD)
            S.check(S.swimba_linattn_fwd(d, q, k, v, self.g, None, state, o, state, ws, ws.numel()))
            assert S.swimba_get_device_status(ws) == 0
        scale = float(np.float32(D ** -0.5))
        r = M.linattn_forward(f64(q), f64(k), f64(v), f64(self.g), scale, None, start)
        tol = (2 * T + D + 16) * 2.0 ** -24 + 2.0 ** -20
        within(o, r.out, self.half * (np.abs(r.out) + (r.once if T > 1 else 0)) + tol * r.mag, "o")
        within(state, r.M, tol * r.M_mag, "state")
        p = new(B, T, H * D)
        self.norm(o.flatten(2), z, self.w_post, None, None, p, None, groups=H)
        y = new(B, T, DM)
        self.gemm(p, self.W_out, (y,))
        h, nxt = torch.empty(B, T, DM, device="cuda"), new(B, T, DM)
        self.norm(y, None, None, x, self.w_next, h, nxt, out_scale=0.5)
        self.kept = q, k, v, o, z, start
        return h, nxt


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompt_then_tokens(S, dtype):
    blk = Block(S, dtype)
    state = torch.zeros(B, H, D, D, device="cuda")
    h, nxt = blk.mix(blk.x[:, :L].contiguous(), state)
    assert torch.isfinite(h).all() and torch.isfinite(nxt.float()).all()
    for t in range(L, L + 3):
        h, nxt = blk.mix(blk.x[:, t:t + 1].contiguous(), state)
    assert torch.isfinite(h).all() and torch.isfinite(state).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradient_through_the_gated_norm_into_the_attention(S, dtype):
    blk = Block(S, dtype)
    state = torch.zeros(B, H, D, D, device="cuda")
    blk.mix(blk.x[:, :L].contiguous(), state)
    q, k, v, o, z, _ = blk.kept
    y = o.flatten(2)
    g_h = torch.randn_like(y, dtype=torch.float32).to(blk.t)
    d = S.make_norm_dims(y, g_h, groups=H, eps=1e-5)
    ws = S.new_norm_workspace(d)
    dy, dz, dw = torch.empty_like(y), torch.empty_like(z), torch.empty_like(blk.w_post)
    S.check(S.swimba_block_norm_bwd(d, y, z, blk.w_post, None, None, g_h, None, dy, dz, None, dw, None, ws, ws.numel()))
    rows = lambda x: f64(x).reshape(-1, H * D)
    want = M.block_norm_backward(rows(y), rows(z), f64(blk.w_post), None, None, rows(g_h), None, groups=H,
                                 eps=float(np.float32(1e-5)))
    for got, name, terms in ((dy, "dy", 0), (dz, "dz", 0), (dw, "dw_post", B * L)):
        w, mag = want[name]
        half = 0.0 if got.dtype == torch.float32 else 2.0 ** -8
        within(got, w, half * np.abs(w) + (terms + H * D + 96) * 2.0 ** -24 * mag, name)
    ld = S.make_linattn_dims(q, k, v, D ** -0.5)
    lws = S.new_linattn_workspace(ld, S.SWIMBA_OP_LINATTN_BWD)
    dqkv = torch.full((B, L, QKV), float("nan"), device="cuda", dtype=blk.t)  # the in-projection's output gradient
    dq, dk, dv = (p.unflatten(2, (-1, D)) for p in dqkv.split([H * D, KV * D, KV * D], dim=2))
    S.check(S.swimba_linattn_bwd(ld, q, k, v, blk.g, None, None, dy, None, dq, dk, dv, None, lws, lws.numel()))
    assert S.swimba_get_device_status(lws) == 0
    g_o = f64(dy).reshape(B, L, H, D)
    rq, rk, rv = M.linattn_backward(f64(q), f64(k), f64(v), f64(blk.g), float(np.float32(D ** -0.5)), g_o)
    tol = (2 * L + D + 16) * 2.0 ** -24 + 2.0 ** -20
    for got, r, what in ((dq, rq, "dq"), (dk, rk, "dk"), (dv, rv, "dv")):
        add = (lambda x: x) if what == "dq" else (lambda x: M.sum_shared(x, KV))
        out, once, mag = add(r.out), add(r.once), add(r.mag)
        within(got, out, blk.half * (np.abs(out) + once) + tol * mag, what)
