"""Argument checks and workspace sizes of the mixer operators (linear attention, block norms), on the
host: every refusal comes back before anything is launched, so no device is needed."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

FAKE = 1 << 40  # never dereferenced: every case fails validation first
INVALID, UNSUPPORTED, ALIGN, WORKSPACE = 1, 2, 3, 4


@pytest.fixture(scope="module")
def S():
    from parameter_space_moe_swimba_b200 import build

    build.build()
    from parameter_space_moe_swimba_b200 import swimba

    return swimba


def la_dims(S, **kw):
    d = dict(batch=2, seqlen=300, n_heads=6, n_kv_heads=2, d_k=64, d_v=128, io_dtype=S.SWIMBA_BF16, scale=1.0)
    d.update(kw)
    d.setdefault("q_stride", d["n_heads"] * d["d_k"])
    d.setdefault("k_stride", d["n_kv_heads"] * d["d_k"])
    d.setdefault("v_stride", d["n_kv_heads"] * d["d_v"])
    return S.swimba_linattn_dims(**d)


BAD = [(dict(batch=0), INVALID), (dict(seqlen=0), INVALID), (dict(n_heads=0), INVALID), (dict(d_k=0), INVALID),
       (dict(d_v=-8), INVALID), (dict(n_kv_heads=4), INVALID), (dict(n_kv_heads=0), INVALID), (dict(io_dtype=2), INVALID),
       (dict(d_k=68), UNSUPPORTED), (dict(d_v=136), UNSUPPORTED), (dict(d_k=4), UNSUPPORTED),
       (dict(q_stride=376), INVALID), (dict(k_stride=120), INVALID), (dict(v_stride=248), INVALID),
       (dict(q_stride=388), UNSUPPORTED), (dict(seqlen=1 << 31), UNSUPPORTED), (dict(batch=1 << 21), UNSUPPORTED),
       (dict(q_stride=1 << 32), UNSUPPORTED), (dict(seqlen=1 << 30, batch=4), UNSUPPORTED)]


def fwd(S, d, **kw):
    a = dict(q=FAKE, k=FAKE + 1024, v=FAKE + 2048, g=FAKE, lens=None, S0=None, o=FAKE + 4096, S_final=None, ws=FAKE,
             n=1 << 40)
    a.update(kw)
    return S.swimba_linattn_fwd(d, a["q"], a["k"], a["v"], a["g"], a["lens"], a["S0"], a["o"], a["S_final"], a["ws"],
                                a["n"], 0)


def bwd(S, d, **kw):
    a = dict(q=FAKE, k=FAKE + 1024, v=FAKE + 2048, g=FAKE, lens=None, S0=None, g_o=FAKE + 4096, g_S=None, dq=FAKE + 8192,
             dk=FAKE + 9216, dv=FAKE + 10240, dS0=None, ws=FAKE, n=1 << 40)
    a.update(kw)
    return S.swimba_linattn_bwd(d, *(a[x] for x in ("q", "k", "v", "g", "lens", "S0", "g_o", "g_S", "dq", "dk", "dv",
                                                    "dS0", "ws", "n")), 0)


def step(S, d, **kw):
    a = dict(q=FAKE, k=FAKE + 1024, v=FAKE + 2048, g=FAKE, S_in=FAKE, o=FAKE + 4096, S_out=FAKE)
    a.update(kw)
    return S.swimba_linattn_step(d, *(a[x] for x in ("q", "k", "v", "g", "S_in", "o", "S_out")), 0)


@pytest.mark.parametrize("kw,status", BAD)
def test_linattn_dims(S, kw, status):
    d = la_dims(S, **kw)
    for op in (S.SWIMBA_OP_LINATTN_FWD, S.SWIMBA_OP_LINATTN_BWD):
        assert S.swimba_linattn_workspace_size(d, op) == 0
    assert fwd(S, d) == status and bwd(S, d) == status and step(S, d) == status


def test_linattn_arguments(S):
    d = la_dims(S)
    need = S.swimba_linattn_workspace_size(d, S.SWIMBA_OP_LINATTN_FWD)
    assert need >= 256 and S.swimba_linattn_workspace_size(d, S.SWIMBA_OP_LINATTN_FWD + 5) == 0
    # few heads need no room for states handed from CTA to CTA, many do
    many = la_dims(S, batch=64)
    assert need < 4096 and S.swimba_linattn_workspace_size(many, S.SWIMBA_OP_LINATTN_FWD) >= 148 * 65536
    for x in ("q", "k", "v", "g", "o"):
        assert fwd(S, d, **{x: None}) == INVALID
    for x in ("q", "k", "v", "o", "S0", "S_final", "ws"):
        assert fwd(S, d, **{x: FAKE + 4}) == ALIGN
    assert fwd(S, d, o=FAKE) == INVALID  # the output over an input
    assert fwd(S, d, ws=None) == WORKSPACE and fwd(S, d, n=need - 1) == WORKSPACE
    need = S.swimba_linattn_workspace_size(d, S.SWIMBA_OP_LINATTN_BWD)
    # the per-head partials of the shared heads' gradients are in there
    assert need >= 256 + 4 * 2 * 300 * 6 * (64 + 128)
    for x in ("q", "k", "v", "g", "g_o", "dq", "dk", "dv"):
        assert bwd(S, d, **{x: None}) == INVALID
    for x in ("q", "k", "v", "g_o", "dq", "dk", "dv", "S0", "g_S", "dS0", "ws"):
        assert bwd(S, d, **{x: FAKE + 8}) == ALIGN
    for x in ("dq", "dk", "dv"):
        assert bwd(S, d, **{x: FAKE + 2048}) == INVALID
    assert bwd(S, d, dq=FAKE + 9216) == INVALID and bwd(S, d, dv=FAKE + 8192) == INVALID
    assert bwd(S, d, g_S=FAKE + 64, dS0=FAKE + 64) == INVALID and bwd(S, d, S0=FAKE + 64, dS0=FAKE + 64) == INVALID
    assert bwd(S, d, ws=None) == WORKSPACE and bwd(S, d, n=need - 1) == WORKSPACE
    assert step(S, d) == INVALID  # more than one token
    one = la_dims(S, seqlen=1)
    for x in ("q", "k", "v", "g", "S_in", "o", "S_out"):
        assert step(S, one, **{x: None}) == INVALID
    for x in ("q", "k", "v", "S_in", "o", "S_out"):
        assert step(S, one, **{x: FAKE + 2}) == ALIGN


def test_linattn_layouts(S):
    """make_linattn_dims takes dense tensors and columns of one buffer, and refuses what the layout does
    not cover rather than reading other elements."""
    buf = torch.zeros(2, 5, 4 * 16 + 2 * 16 + 2 * 8)
    q, k, v = buf.split([64, 32, 16], dim=2)
    q, k, v = q.unflatten(2, (4, 16)), k.unflatten(2, (2, 16)), v.unflatten(2, (2, 8))
    d = S.make_linattn_dims(q, k, v, 0.5)
    assert (d.q_stride, d.k_stride, d.v_stride, d.n_heads, d.n_kv_heads, d.d_k, d.d_v) == (112, 112, 112, 4, 2, 16, 8)
    d = S.make_linattn_dims(q.contiguous(), k, v, 0.5)
    assert (d.q_stride, d.k_stride) == (64, 112)
    one = torch.zeros(3, 1, 2, 8)
    assert S.make_linattn_dims(one, one, one, 1.0).q_stride == 16
    heads_first = torch.zeros(2, 4, 5, 16).transpose(1, 2)
    for bad in ((heads_first, k, v), (q, k, v.bfloat16()), (q, k[:, :4], v), (q, k, v[:, :, :1]), (q[..., :8], k, v),
                (q[:, ::2], k[:, ::2], v[:, ::2])):
        with pytest.raises(S.SwimbaError):
            S.make_linattn_dims(*bad, 1.0)
    # CPU tensors are on another device than a call's
    state, o = torch.zeros(2, 4, 16, 16), torch.zeros(2, 5, 4, 16)
    d = S.make_linattn_dims(o, o, o, 0.5)
    assert S.swimba_linattn_fwd(d, o, o, o, FAKE, None, state, FAKE + 4096, state, FAKE, 1 << 40, 0) == INVALID


def test_tensors_lie_as_the_dims_say(S, monkeypatch):
    """Inputs and gradients have the dims' token strides and the rest is dense; anything else is refused,
    for it would be read as other elements. CPU tensors stand in for the device's: the device is named -1."""
    monkeypatch.setattr(S.torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(S.torch.cuda, "current_device", lambda: -1)
    buf = torch.zeros(2, 5, 4 * 16 + 2 * 16 + 2 * 16)
    q, k, v = buf.split([64, 32, 32], dim=2)
    q, k, v = q.unflatten(2, (4, 16)), k.unflatten(2, (2, 16)), v.unflatten(2, (2, 16))
    d = S.make_linattn_dims(q, k, v, 0.5)
    lies = lambda dims, x, dense=(): S._pointers(dense, dims, ((x, dims.q_stride, dims.d_k),)) is not None
    assert lies(d, q) and not lies(d, q.contiguous()) and not lies(d, torch.zeros(2, 4, 5, 16).transpose(1, 2))
    state = torch.zeros(2, 4, 16, 16)
    assert lies(d, q, (state, None, FAKE)) and not lies(d, q, (state.transpose(2, 3),))
    # part of a longer buffer, heads apart, elements apart: the token stride alone would fit
    assert not lies(d, torch.zeros(2, 6, 128)[:, :5, :64].unflatten(2, (4, 16)))
    assert not lies(d, buf.unflatten(2, (4, 32))[..., :16])
    assert not lies(d, buf.unflatten(2, (16, 8))[..., :4].transpose(2, 3))
    # one token: the distance between sequences counts
    d = S.make_linattn_dims(q[:, :1], k[:, :1], v[:, :1], 0.5)
    assert d.q_stride == 5 * 128 and lies(d, q[:, :1]) and not lies(d, q[:, :1].contiguous())
    assert lies(d, q[:1, :1].contiguous())


def norm_dims(S, **kw):
    d = dict(rows=10, width=512, groups=4, io_dtype=S.SWIMBA_BF16, res_dtype=S.SWIMBA_F32, gate_last=0, eps=1e-5,
             res_scale=1.0, out_scale=1.0)
    d.update(kw)
    return S.swimba_norm_dims(**d)


NORM_FWD = ("y", "z", "w_post", "res", "w_pre", "h", "n")
NORM_BWD = ("y", "z", "w_post", "res", "w_pre", "g_h", "g_n", "dy", "dz", "dres", "dw_post", "dw_pre")


def norm_fwd(S, d, **kw):
    a = {x: FAKE + 1024 * i for i, x in enumerate(NORM_FWD)}
    a.update(kw)
    return S.swimba_block_norm_fwd(d, *(a[x] for x in NORM_FWD), 0)


def norm_bwd(S, d, ws=FAKE, n=1 << 40, **kw):
    a = {x: FAKE + 1024 * i for i, x in enumerate(NORM_BWD)}
    a.update(kw)
    return S.swimba_block_norm_bwd(d, *(a[x] for x in NORM_BWD), ws, n, 0)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=0), INVALID), (dict(width=0), INVALID), (dict(groups=0), INVALID), (dict(eps=0.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(io_dtype=5), INVALID), (dict(res_dtype=-1), INVALID),
    (dict(gate_last=2), INVALID), (dict(width=516), UNSUPPORTED), (dict(width=16392, groups=1), UNSUPPORTED),
    (dict(groups=5), UNSUPPORTED), (dict(groups=128), UNSUPPORTED), (dict(rows=1 << 32), UNSUPPORTED)])
def test_norm_dims(S, kw, status):
    d = norm_dims(S, **kw)
    assert norm_fwd(S, d) == status and norm_bwd(S, d) == status and S.swimba_block_norm_workspace_size(d) == 0


def test_norm_arguments(S):
    d = norm_dims(S)
    assert norm_fwd(S, d, y=None) == INVALID and norm_fwd(S, d, y=None, z=None, w_post=None, res=None) == INVALID
    assert norm_fwd(S, d, h=None, n=None) == INVALID and norm_fwd(S, d, h=None, n=None, w_pre=None) == INVALID
    assert norm_fwd(S, d, n=None) == INVALID and norm_fwd(S, d, w_pre=None) == INVALID  # w_pre without n, n without it
    same = FAKE + 99 * 1024
    assert norm_fwd(S, d, h=same, n=same) == INVALID and norm_fwd(S, d, y=same, h=same) == INVALID
    assert norm_fwd(S, d, res=same, n=same) == INVALID
    for x in NORM_FWD:
        assert norm_fwd(S, d, **{x: same + 8}) == ALIGN
    need = S.swimba_block_norm_workspace_size(d)
    assert need >= 256
    for x in NORM_BWD:
        if x != "g_h":  # every part has its gradient and the other way round
            assert norm_bwd(S, d, **{x: None}) == INVALID
        assert norm_bwd(S, d, **{x: same + 4}) == ALIGN
    assert norm_bwd(S, d, g_h=None, g_n=None, w_pre=None, dw_pre=None) == INVALID
    assert norm_bwd(S, d, ws=None) == WORKSPACE and norm_bwd(S, d, n=need - 1) == WORKSPACE
    assert norm_bwd(S, d, ws=FAKE + 8) == ALIGN
    with pytest.raises(S.SwimbaError):
        S.make_norm_dims(torch.zeros(3, 8), torch.zeros(4, 8))


class Called:
    """Stands in for the library: a call that got past the binding's checks."""

    def __init__(self):
        self.args = None

    def __getattr__(self, name):
        def call(*args):
            self.args = args
            return 0

        return call


@pytest.fixture
def taken(S, monkeypatch):
    """Runs a binding call on CPU tensors that stand in for the device's (named -1), without the library."""
    monkeypatch.setattr(S.torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(S.torch.cuda, "current_device", lambda: -1)
    lib = Called()
    monkeypatch.setattr(S, "_lib", lib)
    return lib


# Of each tensor: another type, a smaller batch or fewer tokens, more of them.
def _others(x):
    other = {torch.float32: torch.bfloat16, torch.bfloat16: torch.float16, torch.int32: torch.int64}[x.dtype]
    return x.to(other), x[1:], x[:, :-1] if x.dim() > 1 else x[:-1], torch.cat((x, x))


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B", [1, 2])
def test_linattn_tensors_have_the_dims_types_and_sizes(S, taken, t, B):
    """lens as int64, a state in the io type, an output of a smaller batch, gradients of fewer tokens: refused."""
    L, H, KV, dk, dv = 5, 4, 2, 16, 24
    new = lambda *s, t=t: torch.zeros(s, dtype=t)
    state = lambda: new(B, H, dk, dv, t=torch.float32)
    rows = dict(q=new(B, L, H, dk), k=new(B, L, KV, dk), v=new(B, L, KV, dv))
    d = S.make_linattn_dims(*rows.values(), 0.5)
    g, lens, o = new(H, t=torch.float32), new(B, t=torch.int32), new(B, L, H, dv)
    ws = torch.zeros(64, dtype=torch.uint8)
    calls = {
        "swimba_linattn_fwd": dict(**rows, log_decay=g, lens=lens, S0=state(), o=o, S_final=state()),
        "swimba_linattn_bwd": dict(**rows, log_decay=g, lens=lens, S0=state(), g_o=o, g_S=state(),
                                   **{"d" + n: x.clone() for n, x in rows.items()}, dS0=state()),
    }
    one = {n: x[:, :1].contiguous() for n, x in rows.items()}
    calls["swimba_linattn_step"] = dict(**one, log_decay=g, S_in=state(), o=o[:, :1].contiguous(), S_out=state())
    for name, a in calls.items():
        step = name.endswith("step")
        dims = S.make_linattn_dims(*one.values(), 0.5) if step else d
        tail = () if step else (ws, 64)
        call = lambda **kw: getattr(S, name)(dims, *{**a, **kw}.values(), *tail, 0)
        assert call() == 0
        for n, x in a.items():
            for bad in _others(x):
                assert call(**{n: bad}) == INVALID, (name, n, bad.shape, bad.dtype)
    # a workspace is no longer than it is
    taken.args = None
    assert S.swimba_linattn_fwd(d, *calls["swimba_linattn_fwd"].values(), ws, 1 << 30, 0) == 0 and taken.args[-2] == 64


@pytest.mark.parametrize("io,res_t", [(torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)])
def test_norm_tensors_have_the_dims_types_and_sizes(S, taken, io, res_t):
    rows, width = 6, 32
    row = lambda t: torch.zeros(rows, width, dtype=t)
    d = S.make_norm_dims(row(io), row(res_t))
    types = dict(y=io, z=io, w_post=None, res=res_t, w_pre=None, h=res_t, n=io, g_h=res_t, g_n=io, dy=io, dz=io,
                 dres=res_t, dw_post=None, dw_pre=None)
    x = {n: torch.zeros(width) if t is None else row(t) for n, t in types.items()}
    ws = torch.zeros(64, dtype=torch.uint8)
    fwd = lambda **kw: S.swimba_block_norm_fwd(d, *({**x, **kw}[n] for n in NORM_FWD), 0)
    bwd = lambda **kw: S.swimba_block_norm_bwd(d, *({**x, **kw}[n] for n in NORM_BWD), ws, 1 << 30, 0)
    for names, call in ((NORM_FWD, fwd), (NORM_BWD, bwd)):
        assert call() == 0
        for n in names:
            for bad in _others(x[n]):
                assert call(**{n: bad}) == INVALID, (n, bad.shape, bad.dtype)
    assert bwd() == 0 and taken.args[-2] == 64


def test_makers_of_dims_refuse_other_types_and_ranks(S):
    half = torch.zeros(2, 5, 4, 16, dtype=torch.float16)
    for bad in (half, half.float()[0]):
        with pytest.raises(S.SwimbaError):
            S.make_linattn_dims(bad, bad, bad, 1.0)
    for y, h in ((half, half.float()), (half.float(), half)):
        with pytest.raises(S.SwimbaError):
            S.make_norm_dims(y, h)
