"""The mixer operators that stand beside the Swimba layer, as one list of measurable cases: linear
attention with a decay for each head (whole prompts, single tokens, backward) and the norms around
a block fused with its gate and residual scales (forward, backward).

    S_t = exp(g_h) S_{t-1} + k_t v_t^T          o_t = scale S_t^T q_t          (one state per head)

    a = y SiLU(z);  p = RMSNorm_groups(a) w_post  (or  p = RMSNorm_groups(y) w_post SiLU(z))
    h = res_scale res + out_scale p;  n = RMSNorm(h) w_pre

``run`` computes a case in elementary torch operations in 32 bits (``own = False``) or through the
library's entry points (``own = True``); ``exact`` is the definition in 64 bits, token by token.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
CHUNK = 128  # tokens per chunk of the plain form


# ---- cases -----------------------------------------------------------------------------------------

def _la(op, name=None, **kw):
    c = dict(op=op, B=1, L=1, H=1, KV=0, dk=64, dv=64, dtype=BF16, lens=False, start=False, fused=False)
    c.update(kw)
    c["KV"] = c["KV"] or c["H"]
    return dict(c, name=name) if name else c


def _norm(op, name=None, **kw):
    c = dict(op=op, rows=1, width=64, groups=1, dtype=BF16, res_dtype=BF16, gate=True, gate_last=False, post=True,
             res=True, pre=True, res_scale=1.0, out_scale=1.0)
    c.update(kw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # a handful of short prompts of a 1536-channel mixer: the launch and one pass of latency
        _la("la_fwd", "la_fwd_short", B=4, L=96, H=24, dk=64, dv=64),
        # prefill of 8 prompts of 4096 tokens, 4096 channels
        _la("la_fwd", "la_fwd_prompt", B=8, L=4096, H=32, dk=128, dv=128),
        # one long document, few heads, continued from a cached state
        _la("la_fwd", "la_fwd_long", B=1, L=65536, H=16, dk=128, dv=128, start=True),
        # a padded batch of prompts of unequal lengths (empty ones among them), shared key/value heads,
        # q, k and v as columns of one projection's output
        _la("la_fwd", "la_fwd_ragged", B=6, L=1531, H=20, KV=5, dk=64, dv=128, lens=True, start=True, fused=True),
        # decoding: three sequences in fp32; 256 sequences of a 4096-channel mixer (1 GiB of state)
        _la("la_step", "la_step_few", B=3, H=32, dk=128, dv=128, dtype=F32),
        _la("la_step", "la_step_many", B=256, H=32, dk=128, dv=128),
        # a training step's backward; a small fp32 one with shared heads, odd sizes and padding
        _la("la_bwd", "la_bwd_train", B=8, L=2048, H=32, dk=128, dv=128),
        _la("la_bwd", "la_bwd_f32", B=2, L=333, H=8, KV=4, dk=64, dv=96, dtype=F32, lens=True, start=True),
        # the norm, gate, residual and next norm of one decode step, and of a prefill
        _norm("norm_fwd", "norm_fwd_decode", rows=256, width=4096, groups=32, res_dtype=F32),
        _norm("norm_fwd", "norm_fwd_prefill", rows=32768, width=4096, groups=1, out_scale=0.5),
        # training: a small fp32 mixer with the gate after the norm, and 16384 tokens of a 4096-channel one
        _norm("norm_bwd", "norm_bwd_small", rows=777, width=1536, groups=12, dtype=F32, res_dtype=F32, gate_last=True),
        _norm("norm_bwd", "norm_bwd_train", rows=16384, width=4096, groups=1, res_dtype=F32, out_scale=0.5),
    ]


def _log(rng, lo, hi):
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["la_fwd", "la_fwd", "la_step", "la_bwd", "la_bwd", "norm_fwd", "norm_bwd"])
    dtype = F32 if rng.random() < 0.25 else BF16
    if op.startswith("la"):
        head = lambda: rng.choice([64, 64, 128, 128, 8 * rng.randint(2, 16)])
        dk, dv = head(), head()
        group = rng.choice([1, 1, 2, 3])
        KV = _log(rng, 1, 16)
        H = KV * group
        most = {"la_fwd": 2 ** 27, "la_step": 2 ** 30, "la_bwd": 2 ** 26}[op] // (8 if dtype == F32 else 1)
        per = H * max(dk, dv) * (dk if op == "la_step" else 1)
        if op == "la_step":
            B, L = _log(rng, 1, max(1, min(512, most // (4 * per)))), 1
        else:
            B = _log(rng, 1, 16)
            L = _log(rng, 1, max(1, min(65536 if dtype == BF16 else 4096, most // (B * per))))
        return _la(op, B=B, L=L, H=H, KV=KV, dk=dk, dv=dv, dtype=dtype, lens=op != "la_step" and rng.random() < 0.4,
                   start=rng.random() < 0.5, fused=rng.random() < 0.3)
    groups = rng.choice([1, 1, 2, 8, 12, 32])
    width = groups * 8 * _log(rng, 1 if groups > 1 else 8, 8192 // (8 * groups))
    most = (2 ** 27 if op == "norm_fwd" else 2 ** 26) // (2 if dtype == F32 else 1)
    rows = _log(rng, 1, min(65536, most // width))
    return _norm(op, rows=rows, width=width, groups=groups, dtype=dtype, res_dtype=rng.choice([dtype, F32]),
                 gate=rng.random() < 0.7, gate_last=rng.random() < 0.5, post=rng.random() < 0.7, res=rng.random() < 0.8,
                 pre=rng.random() < 0.8, res_scale=rng.choice([1.0, 0.75]), out_scale=rng.choice([1.0, 0.5]))


# ---- inputs ----------------------------------------------------------------------------------------

def _t(dtype):
    return torch.bfloat16 if dtype == BF16 else torch.float32


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")
    s = dict(case=dict(case))
    if case["op"].startswith("la"):
        B, L, H, KV, dk, dv = (case[n] for n in ("B", "L", "H", "KV", "dk", "dv"))
        t = _t(case["dtype"])
        widths = (H * dk, KV * dk, KV * dv)
        if case["fused"]:  # the columns of one projection's output
            q, k, v = randn(B, L, sum(widths)).to(t).split(widths, dim=2)
        else:
            q, k, v = (randn(B, L, w).to(t) for w in widths)
        s.update(q=q.unflatten(2, (H, dk)), k=k.unflatten(2, (KV, dk)), v=v.unflatten(2, (KV, dv)))
        # decays from about 0.54 to 0.996 a token, one per head
        s["log_decay"] = -torch.exp2(torch.linspace(-0.7, -8.0, H, device="cuda", dtype=torch.float64)).float()
        s["scale"] = dk ** -0.5
        s["S0"] = 0.3 * randn(B, H, dk, dv) if case["start"] or case["op"] == "la_step" else None
        if case["lens"]:
            n = torch.randint(0, L + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
            n[0] = L
            if B > 2:
                n[1] = 0
            s["lens"] = n
        else:
            s["lens"] = None
        if case["op"] == "la_bwd":
            s["g_o"] = randn(B, L, H, dv).to(t)
            s["g_S"] = 0.3 * randn(B, H, dk, dv) if case["start"] else None
            # the gradients lie as q, k and v do
            if case["fused"]:
                grads = torch.zeros(B, L, sum(widths), device="cuda", dtype=t).split(widths, dim=2)
            else:
                grads = [torch.zeros(B, L, w, device="cuda", dtype=t) for w in widths]
            s["dq"], s["dk"], s["dv"] = (x.unflatten(2, (n, -1)) for x, n in zip(grads, (H, KV, KV)))
            s["dS0"] = torch.zeros(B, H, dk, dv, device="cuda") if case["start"] else None
        else:
            s["o"] = torch.zeros(B, L, H, dv, device="cuda", dtype=t)
            s["S"] = torch.zeros(B, H, dk, dv, device="cuda")
        return s
    R, W, t, rt = case["rows"], case["width"], _t(case["dtype"]), _t(case["res_dtype"])
    s["y"] = randn(R, W).to(t)
    s["z"] = randn(R, W).to(t) if case["gate"] else None
    s["w_post"] = 1 + 0.2 * randn(W) if case["post"] else None
    s["res"] = (2 * randn(R, W)).to(rt) if case["res"] else None
    s["w_pre"] = 1 + 0.2 * randn(W) if case["pre"] else None
    if case["op"] == "norm_fwd":
        s["h"] = torch.zeros(R, W, device="cuda", dtype=rt)
        s["n"] = torch.zeros(R, W, device="cuda", dtype=t) if case["pre"] else None
    else:
        s["g_h"] = randn(R, W).to(rt)
        s["g_n"] = randn(R, W).to(t) if case["pre"] else None
        s["dy"] = torch.zeros(R, W, device="cuda", dtype=t)
        s["dz"] = torch.zeros(R, W, device="cuda", dtype=t) if case["gate"] else None
        s["dres"] = torch.zeros(R, W, device="cuda", dtype=rt) if case["res"] else None
        s["dw_post"] = torch.zeros(W, device="cuda") if case["post"] else None
        s["dw_pre"] = torch.zeros(W, device="cuda") if case["pre"] else None
    return s


EPS = 1e-5


def work(case):
    """Every input read once and every output written once; the recurrent form's multiply-adds."""
    e = 2 if case["dtype"] == BF16 else 4
    if case["op"].startswith("la"):
        B, L, H, KV, dk, dv = (case[n] for n in ("B", "L", "H", "KV", "dk", "dv"))
        T, state = B * L, B * H * dk * dv * 4
        q, k, v, o = T * H * dk * e, T * KV * dk * e, T * KV * dv * e, T * H * dv * e
        pair = 2 * T * H * dk * dv  # one product of a token with its head's state
        if case["op"] == "la_bwd":  # dq, dk, dv and the two states' updates
            return {"bytes": 2 * (q + k + v) + o + (3 * state if case["start"] else 0), "flops": 5 * pair}
        starts = case["start"] or case["op"] == "la_step"
        return {"bytes": q + k + v + o + state * (2 if starts else 1), "flops": 2 * pair}
    n, r = case["rows"] * case["width"] * e, case["rows"] * case["width"] * (2 if case["res_dtype"] == BF16 else 4)
    gate, res, pre = int(case["gate"]), int(case["res"]), int(case["pre"])
    ws = 4 * case["width"] * (int(case["post"]) + pre)
    if case["op"] == "norm_fwd":
        return {"bytes": n * (1 + gate + pre) + r * (res + 1) + ws, "flops": 12 * case["rows"] * case["width"]}
    return {"bytes": n * (2 + 2 * gate + pre) + r * (1 + 2 * res) + 2 * ws, "flops": 30 * case["rows"] * case["width"]}


# ---- the plain forms -------------------------------------------------------------------------------

def _heads(x, H):
    """[B, L, h, d] with every shared head repeated for the query heads that read it."""
    return x.repeat_interleave(H // x.shape[2], dim=2)


def _chunks(x, L):
    """[B, L, H, d] -> fp32 [B, H, chunks, CHUNK, d], zeros after the last token."""
    x = x.float().permute(0, 2, 1, 3)
    n = -(-L // CHUNK)
    return torch.nn.functional.pad(x, (0, 0, 0, n * CHUNK - L)).unflatten(2, (n, CHUNK))


def _powers(g, e):
    """exp(g e) for head decays g [H] and exponents e >= 0 (0 where e < 0), in 64 bits, rounded to 32."""
    e = e.double()
    g = g.double().reshape((-1,) + (1,) * e.dim())
    return torch.where(e >= 0, torch.exp(g * e.clamp(min=0)), 0.0).float()


def _valid(s, B, L):
    t = torch.arange(L, device="cuda")
    lens = s["lens"] if s["lens"] is not None else torch.full((B,), L, device="cuda", dtype=torch.int32)
    return (t[None, :] < lens[:, None])[:, :, None, None], lens


def _decay_to_end(g, lens, L):
    """exp(g (len - 1 - t)) for t < len, else 0: [B, H, L]."""
    e = lens[:, None].double() - 1 - torch.arange(L, device="cuda")[None, :]
    return _powers(g, e).transpose(0, 1)


def _plain_states(kc, vc, g, S0):
    """The state before every chunk, [B, H, chunks, dk, dv]."""
    n = kc.shape[2]
    i, c = torch.arange(CHUNK, device="cuda"), torch.arange(n, device="cuda")
    U = (kc * _powers(g, CHUNK - 1 - i)[:, None, :, None]).transpose(-1, -2) @ vc
    T = _powers(g, CHUNK * (c[:, None] - 1 - c[None, :]))
    S = (T @ U.flatten(3)).unflatten(3, U.shape[3:])
    if S0 is not None:
        S = S + _powers(g, CHUNK * c)[:, :, None, None] * S0[:, :, None]
    return S


def _plain_la_fwd(s):
    c, g = s["case"], s["log_decay"]
    B, L, H = c["B"], c["L"], c["H"]
    valid, lens = _valid(s, B, L)
    k, v = (torch.where(valid, _heads(s[n], H), 0) for n in ("k", "v"))
    qc, kc, vc = _chunks(s["q"], L), _chunks(k, L), _chunks(v, L)
    i = torch.arange(CHUNK, device="cuda")
    D = _powers(g, i[:, None] - i[None, :])[:, None]
    S = _plain_states(kc, vc, g, s["S0"])
    o = ((qc @ kc.transpose(-1, -2)) * D) @ vc + _powers(g, i + 1)[:, None, :, None] * (qc @ S)
    o = (s["scale"] * o).flatten(2, 3)[:, :, :L].permute(0, 2, 1, 3)
    o = torch.where(valid, o, 0).to(s["o"].dtype)
    w = _decay_to_end(g, lens, L)[..., None]
    S_end = (k.float().permute(0, 2, 1, 3) * w).transpose(-1, -2) @ v.float().permute(0, 2, 1, 3)
    if s["S0"] is not None:
        S_end = S_end + _powers(g, lens).transpose(0, 1)[..., None, None] * s["S0"]
    return o, S_end


def _plain_la_step(s):
    H = s["case"]["H"]
    q, k, v = (_heads(s[n], H)[:, 0].float() for n in ("q", "k", "v"))
    S = torch.exp(s["log_decay"])[:, None, None] * s["S0"] + k[..., :, None] * v[..., None, :]
    o = s["scale"] * (q[..., :, None] * S).sum(-2)
    return o[:, None].to(s["o"].dtype), S


def _plain_la_bwd(s):
    c, g = s["case"], s["log_decay"]
    B, L, H, KV = c["B"], c["L"], c["H"], c["KV"]
    valid, lens = _valid(s, B, L)
    q, do = (torch.where(valid, s[n], 0) for n in ("q", "g_o"))
    k, v = (torch.where(valid, _heads(s[n], H), 0) for n in ("k", "v"))
    qc, kc, vc, dc = _chunks(q, L), _chunks(k, L), _chunks(v, L), s["scale"] * _chunks(do, L)
    n = qc.shape[2]
    i, m = torch.arange(CHUNK, device="cuda"), torch.arange(n, device="cuda")
    D = _powers(g, i[:, None] - i[None, :])[:, None]
    S = _plain_states(kc, vc, g, s["S0"])
    # the states' adjoint after every chunk, brought to its last token
    W = (qc * _powers(g, i + 1)[:, None, :, None]).transpose(-1, -2) @ dc
    M = (_powers(g, CHUNK * (m[None, :] - 1 - m[:, None])) @ W.flatten(3)).unflatten(3, W.shape[3:])
    A, P = (qc @ kc.transpose(-1, -2)) * D, (dc @ vc.transpose(-1, -2)) * D
    tail = _powers(g, CHUNK - 1 - i)[:, None, :, None]
    dq = P @ kc + _powers(g, i + 1)[:, None, :, None] * (dc @ S.transpose(-1, -2))
    dk = P.transpose(-1, -2) @ qc + tail * (vc @ M.transpose(-1, -2))
    dv = A.transpose(-1, -2) @ dc + tail * (kc @ M)
    back = lambda x: x.flatten(2, 3)[:, :, :L]
    dq, dk, dv = back(dq), back(dk), back(dv)
    if s["g_S"] is not None:
        w = _decay_to_end(g, lens, L)[..., None]
        dk = dk + w * (back(vc) @ s["g_S"].transpose(-1, -2))
        dv = dv + w * (back(kc) @ s["g_S"])
    dq, dk, dv = (torch.where(valid, x.permute(0, 2, 1, 3), 0) for x in (dq, dk, dv))
    dk, dv = (x.unflatten(2, (KV, H // KV)).sum(3) for x in (dk, dv))
    out = [x.to(s["dq"].dtype) for x in (dq, dk, dv)]
    if s["dS0"] is not None:
        e = torch.arange(L, device="cuda") + 1
        dS0 = (back(qc) * _powers(g, e)[None, :, :, None]).transpose(-1, -2) @ back(dc)
        if s["g_S"] is not None:
            dS0 = dS0 + _powers(g, lens).transpose(0, 1)[..., None, None] * s["g_S"]
        out.append(dS0)
    return tuple(out)


def _grouped(x, groups):
    return x.unflatten(1, (groups, -1))


def _plain_norm_parts(s):
    c = s["case"]
    y = s["y"].float()
    z = s["z"].float() if s["z"] is not None else None
    gate = z * torch.sigmoid(z) if z is not None else None
    a = y * gate if gate is not None and not c["gate_last"] else y
    r = torch.rsqrt(_grouped(a, c["groups"]).square().mean(-1, keepdim=True) + EPS) if s["w_post"] is not None else None
    hat = (_grouped(a, c["groups"]) * r).flatten(1) if r is not None else a
    p = hat * s["w_post"] if s["w_post"] is not None else hat
    out = p * gate if gate is not None and c["gate_last"] else p
    h = c["out_scale"] * out
    if s["res"] is not None:
        h = h + c["res_scale"] * s["res"].float()
    return y, z, gate, r, hat, p, h


def _plain_norm_fwd(s):
    h = _plain_norm_parts(s)[-1]
    out = [h.to(s["h"].dtype)]
    if s["w_pre"] is not None:
        n = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["w_pre"]
        out.append(n.to(s["n"].dtype))
    return tuple(out)


def _plain_norm_bwd(s):
    c, G = s["case"], s["case"]["groups"]
    y, z, gate, r, hat, p, h = _plain_norm_parts(s)
    out = {}
    dh = s["g_h"].float()
    if s["w_pre"] is not None:
        rh = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
        hh, gn = h * rh, s["g_n"].float()
        out["dw_pre"] = (gn * hh).sum(0)
        gw = gn * s["w_pre"]
        dh = dh + rh * (gw - hh * (gw * hh).mean(-1, keepdim=True))
    if s["res"] is not None:
        out["dres"] = (c["res_scale"] * dh).to(s["dres"].dtype)
    do = c["out_scale"] * dh
    dgate = None
    if gate is not None and c["gate_last"]:
        dgate, do = do * p, do * gate
    if s["w_post"] is not None:
        out["dw_post"] = (do * hat).sum(0)
        gw = _grouped(do * s["w_post"], G)
        do = (r * (gw - _grouped(hat, G) * (gw * _grouped(hat, G)).mean(-1, keepdim=True))).flatten(1)
    if gate is not None:
        if not c["gate_last"]:
            dgate, do = do * y, do * gate
        sg = torch.sigmoid(z)
        out["dz"] = (dgate * sg * (1 + z * (1 - sg))).to(s["dz"].dtype)
    out["dy"] = do.to(s["dy"].dtype)
    return out


# ---- the library's entry points --------------------------------------------------------------------

def _own_la(s):
    from parameter_space_moe_swimba_b200 import swimba as S

    c = s["case"]
    if "dims" not in s:  # kept by a program that calls this shape again
        s["dims"] = S.make_linattn_dims(s["q"], s["k"], s["v"], s["scale"])
        if c["op"] == "la_fwd":
            s["ws"] = S.new_linattn_workspace(s["dims"], S.SWIMBA_OP_LINATTN_FWD)
        elif c["op"] == "la_bwd":
            s["ws"] = S.new_linattn_workspace(s["dims"], S.SWIMBA_OP_LINATTN_BWD)
    d = s["dims"]
    if c["op"] == "la_step":
        S.check(S.swimba_linattn_step(d, s["q"], s["k"], s["v"], s["log_decay"], s["S0"], s["o"], s["S"]),
                "swimba_linattn_step")
        return s["o"], s["S"]
    if c["op"] == "la_fwd":
        S.check(S.swimba_linattn_fwd(d, s["q"], s["k"], s["v"], s["log_decay"], s["lens"], s["S0"], s["o"], s["S"],
                                     s["ws"], s["ws"].numel()), "swimba_linattn_fwd")
        return s["o"], s["S"]
    S.check(S.swimba_linattn_bwd(d, s["q"], s["k"], s["v"], s["log_decay"], s["lens"], s["S0"], s["g_o"], s["g_S"],
                                 s["dq"], s["dk"], s["dv"], s["dS0"], s["ws"], s["ws"].numel()), "swimba_linattn_bwd")
    out = [s["dq"], s["dk"], s["dv"]]
    return tuple(out if s["dS0"] is None else out + [s["dS0"]])


def _own_norm(s):
    from parameter_space_moe_swimba_b200 import swimba as S

    c = s["case"]
    if "dims" not in s:
        s["dims"] = S.make_norm_dims(s["y"], s["h"] if c["op"] == "norm_fwd" else s["g_h"], groups=c["groups"], eps=EPS,
                                     gate_last=c["gate_last"], res_scale=c["res_scale"], out_scale=c["out_scale"])
        if c["op"] == "norm_bwd":
            s["ws"] = S.new_norm_workspace(s["dims"])
    d = s["dims"]
    if c["op"] == "norm_fwd":
        S.check(S.swimba_block_norm_fwd(d, s["y"], s["z"], s["w_post"], s["res"], s["w_pre"], s["h"], s["n"]),
                "swimba_block_norm_fwd")
        return (s["h"],) if s["n"] is None else (s["h"], s["n"])
    S.check(S.swimba_block_norm_bwd(d, s["y"], s["z"], s["w_post"], s["res"], s["w_pre"], s["g_h"], s["g_n"], s["dy"],
                                    s["dz"], s["dres"], s["dw_post"], s["dw_pre"], s["ws"], s["ws"].numel()),
            "swimba_block_norm_bwd")
    return {n: s[n] for n in ("dy", "dz", "dres", "dw_post", "dw_pre") if s[n] is not None}


def run(state):
    op = state["case"]["op"]
    if own:
        return _own_la(state) if op.startswith("la") else _own_norm(state)
    return {"la_fwd": _plain_la_fwd, "la_step": _plain_la_step, "la_bwd": _plain_la_bwd, "norm_fwd": _plain_norm_fwd,
            "norm_bwd": _plain_norm_bwd}[op](state)


# ---- the definitions in 64 bits --------------------------------------------------------------------

def _exact_la(s):
    """Token by token: the state, its readout, and for gradients the adjoint walked back."""
    c = s["case"]
    B, L, H, KV, dk, dv = (c[n] for n in ("B", "L", "H", "KV", "dk", "dv"))
    z = lambda *shape: torch.zeros(shape, device="cuda", dtype=torch.float64)
    decay = torch.exp(s["log_decay"].double())[:, None, None]
    of = torch.arange(H, device="cuda") // (H // KV)
    at = lambda n, t: s[n][:, t].double()
    live = torch.ones(B, L, device="cuda", dtype=torch.bool)
    if s["lens"] is not None:
        live = torch.arange(L, device="cuda")[None] < s["lens"][:, None]
    S = s["S0"].double().clone() if s["S0"] is not None else z(B, H, dk, dv)
    bwd = c["op"] == "la_bwd"
    out = z(B, L, H, dk if bwd else dv)
    for t in range(L):
        on = live[:, t, None, None, None]
        k, v = at("k", t)[:, of], at("v", t)[:, of]
        S = torch.where(on, decay * S + k[..., :, None] * v[..., None, :], S)
        x = at("g_o", t)[..., None, :] if bwd else at("q", t)[..., :, None]
        out[:, t] = torch.where(on[..., 0], s["scale"] * (S * x).sum(-1 if bwd else -2), 0)
    if not bwd:
        return out, S
    N = s["g_S"].double().clone() if s["g_S"] is not None else z(B, H, dk, dv)  # adjoint flowing in from later tokens
    dK, dV = z(B, L, H, dk), z(B, L, H, dv)
    for t in reversed(range(L)):
        on = live[:, t, None, None, None]
        k, v = at("k", t)[:, of], at("v", t)[:, of]
        lam = N + s["scale"] * at("q", t)[..., :, None] * at("g_o", t)[..., None, :]
        dK[:, t] = torch.where(on[..., 0], (lam * v[..., None, :]).sum(-1), 0)
        dV[:, t] = torch.where(on[..., 0], (lam * k[..., :, None]).sum(-2), 0)
        N = torch.where(on, decay * lam, N)
    got = [out, z(B, L, KV, dk).index_add_(2, of, dK), z(B, L, KV, dv).index_add_(2, of, dV)]
    return tuple(got if s["dS0"] is None else got + [N])


def _exact_norm(s):
    c = s["case"]
    leaf = {n: s[n].double().requires_grad_(c["op"] == "norm_bwd") for n in ("y", "z", "w_post", "res", "w_pre")
            if s[n] is not None}

    def rms(x, groups):
        xg = x.reshape(x.shape[0], groups, -1)
        return (xg / torch.sqrt((xg * xg).sum(-1, keepdim=True) / xg.shape[-1] + EPS)).reshape(x.shape)

    silu = lambda x: x / (1 + torch.exp(-x))
    p = leaf["y"]
    if "z" in leaf and not c["gate_last"]:
        p = p * silu(leaf["z"])
    if "w_post" in leaf:
        p = rms(p, c["groups"]) * leaf["w_post"]
    if "z" in leaf and c["gate_last"]:
        p = p * silu(leaf["z"])
    h = p * c["out_scale"]
    if "res" in leaf:
        h = h + leaf["res"] * c["res_scale"]
    n = rms(h, 1) * leaf["w_pre"] if "w_pre" in leaf else None
    if c["op"] == "norm_fwd":
        return (h,) if n is None else (h, n)
    loss = (h * s["g_h"].double()).sum()
    if n is not None:
        loss = loss + (n * s["g_n"].double()).sum()
    grads = torch.autograd.grad(loss, list(leaf.values()))
    names = {"y": "dy", "z": "dz", "w_post": "dw_post", "res": "dres", "w_pre": "dw_pre"}
    return {names[k]: g for k, g in zip(leaf, grads)}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_la(s) if case["op"].startswith("la") else _exact_norm(s)
