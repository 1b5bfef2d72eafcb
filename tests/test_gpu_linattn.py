"""Decay linear attention through the C ABI against the fp64 oracle: prompts, single tokens, gradients.

Tolerances. fp32: each of a token's products and sums is off by at most 2^-24 of the terms it adds, and an
error made at one token is carried on like the state itself, so a result after n tokens with d-long
readouts is within (2 n + d + 16) 2^-24 of the sum of absolute terms (``mag``). bf16: besides that, the
kernel rounds a chunk's masked scores, and the state's copy it reads out, to bf16 once (2^-8 of the terms
they make: ``once``), and the output once (2^-8 of it). The decays are powers that fp32's exp2 gives to
within 2^-21, on exponents rounded to 2^-24 relative: |log decay| times the distance, itself a factor of
the term's own decay, e^-x x <= 1, so another 2^-20 of ``mag`` covers them."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import mixer_oracle as M

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

HALF_BF16 = 2.0 ** -8


@pytest.fixture(scope="module")
def S():
    from parameter_space_moe_swimba_b200 import swimba

    return swimba


class Case:
    """Inputs on the GPU (q, k, v possibly columns of one buffer) and the same values in fp64."""

    def __init__(self, seed, B, L, H, KV, dk, dv, dtype, lens=None, start=True, fused=False, decay=None, scale=0.3):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        t = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.dtype, self.t, self.scale, self.shape = dtype, t, scale, (B, L, H, KV, dk, dv)
        randn = lambda *s: torch.randn(s, generator=g, device="cuda")
        self.fused, self.widths = fused, [H * dk, KV * dk, KV * dv]
        flat = self.rows(lambda w: randn(B, L, w).to(t))
        self.q, self.k, self.v = flat
        self.g_o = randn(B, L, H, dv).to(t)
        self.S0 = randn(B, H, dk, dv) if start else None
        self.g_S = randn(B, H, dk, dv) if start else None
        if decay is None:
            decay = -torch.exp2(torch.linspace(0, -9, H))
        elif not isinstance(decay, torch.Tensor):
            decay = torch.full((H,), float(decay))
        self.g = decay.float().cuda()
        self.lens = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.np = {n: self.f64(getattr(self, n)) for n in ("q", "k", "v", "g_o", "S0", "g_S", "g")}
        self.np_lens = None if lens is None else np.array(lens)
        if lens is not None:  # what lies behind a sequence's end is anybody's
            for b, n in enumerate(lens):
                for x in (self.q, self.k, self.v, self.g_o):
                    x[b, max(0, n):] = float("nan")

    def rows(self, make):
        B, L, H, KV, dk, dv = self.shape
        flat = make(sum(self.widths)).split(self.widths, dim=2) if self.fused else [make(w) for w in self.widths]
        return [x.unflatten(2, s) for x, s in zip(flat, ((H, dk), (KV, dk), (KV, dv)))]

    @staticmethod
    def f64(x):
        return None if x is None else x.double().cpu().numpy()

    def dims(self, S):
        return S.make_linattn_dims(self.q, self.k, self.v, self.scale)

    def forward(self, S, o=None, S_final=None, stream=None):
        B, L, H, KV, dk, dv = self.shape
        d = self.dims(S)
        ws = S.new_linattn_workspace(d, S.SWIMBA_OP_LINATTN_FWD)
        o = torch.empty(B, L, H, dv, device="cuda", dtype=self.t) if o is None else o
        S_final = torch.empty(B, H, dk, dv, device="cuda") if S_final is None else S_final
        S.check(S.swimba_linattn_fwd(d, self.q, self.k, self.v, self.g, self.lens, self.S0, o, S_final, ws, ws.numel(),
                                     stream))
        assert S.swimba_get_device_status(ws, stream) == 0
        return o, S_final

    def backward(self, S):
        B, L, H, KV, dk, dv = self.shape
        d = self.dims(S)
        ws = S.new_linattn_workspace(d, S.SWIMBA_OP_LINATTN_BWD)
        nan = float("nan")
        grads = self.rows(lambda w: torch.full((B, L, w), nan, device="cuda", dtype=self.t))
        dS0 = torch.full((B, H, dk, dv), nan, device="cuda")
        S.check(S.swimba_linattn_bwd(d, self.q, self.k, self.v, self.g, self.lens, self.S0, self.g_o, self.g_S, *grads,
                                     dS0, ws, ws.numel()))
        assert S.swimba_get_device_status(ws) == 0
        return (*grads, dS0)

    def n(self):
        return min(self.shape[1], 10 ** 9)

    def close(self, got, want, once, mag, what, out=True):
        d = max(self.shape[4], self.shape[5])
        tol = ((2 * self.n() + d + 16) * 2.0 ** -24 + 2.0 ** -20) * mag
        if out and self.dtype == "bf16":
            tol = tol + HALF_BF16 * (once + np.abs(want))
        off = np.abs(got - want) - tol
        assert (off <= 1e-30).all(), (what, float(off.max()), float(np.abs(got - want).max()))


CASES = {
    # lengths around the chunk of 128, from one token on
    **{f"L{n}": dict(B=2, L=n, H=2, KV=2, dk=64, dv=64) for n in (1, 2, 31, 127, 128, 129, 256, 300)},
    # head sizes, equal and unequal, padded inside the tiles
    **{f"d{a}x{b}": dict(B=1, L=200, H=2, KV=2, dk=a, dv=b)
       for a, b in ((8, 8), (16, 128), (64, 128), (128, 64), (128, 128), (72, 40), (96, 96), (24, 112))},
    # shared heads, columns of one buffer
    "shared": dict(B=2, L=150, H=6, KV=2, dk=64, dv=128, fused=True),
    "one_kv": dict(B=1, L=140, H=5, KV=1, dk=32, dv=64, fused=True),
    # padded batches: empty sequences, ends at, before and after a chunk's, lengths out of range
    "lens": dict(B=7, L=300, H=2, KV=1, dk=64, dv=64, lens=[300, 0, 1, 128, 129, 257, 255]),
    "lens_out_of_range": dict(B=3, L=130, H=1, KV=1, dk=64, dv=128, lens=[-5, 1000, 130], fused=True),
    # decays: none, total, strong (the state underflows inside a chunk), tiny
    **{f"decay{g}": dict(B=1, L=270, H=2, KV=2, dk=64, dv=64, decay=g) for g in (0.0, -float("inf"), -20.0, -1e-6)},
    # few heads and many chunks: the sequence is split into segments
    "split": dict(B=1, L=1500, H=1, KV=1, dk=64, dv=64),
    "split_lens": dict(B=2, L=1700, H=2, KV=1, dk=32, dv=64, lens=[1430, 400]),
    # more heads than SMs, not a multiple: sequences are cut between two CTAs
    "cut": dict(B=1, L=900, H=149, KV=149, dk=16, dv=24),
    # the longest sequences that bf16 takes token by token, and the shortest that it does not
    "short": dict(B=3, L=8, H=6, KV=2, dk=64, dv=128, fused=True),
    "short_lens": dict(B=4, L=7, H=4, KV=1, dk=128, dv=72, lens=[7, 0, 3, 9]),
    "chunk_of_9": dict(B=3, L=9, H=6, KV=2, dk=64, dv=128, fused=True),
    "no_start": dict(B=2, L=200, H=2, KV=2, dk=128, dv=128, start=False),
    "split_no_start": dict(B=1, L=1500, H=1, KV=1, dk=128, dv=128, start=False),
}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", CASES)
def test_forward(S, name, dtype):
    c = Case(1, dtype=dtype, **CASES[name])
    B, L, H, KV, dk, dv = c.shape
    o = torch.full((B, L, H, dv), 7.0, device="cuda", dtype=c.t)
    o, S_final = c.forward(S, o)
    a = c.np
    r = M.linattn_forward(a["q"], a["k"], a["v"], a["g"], c.scale, c.np_lens, a["S0"])
    lens = np.full(B, L) if c.np_lens is None else np.clip(c.np_lens, 0, L)
    got = Case.f64(o)
    for b in range(B):
        assert (got[b, lens[b]:] == 7.0).all()
        got[b, lens[b]:] = 0
    c.close(got, r.out, r.once, r.mag, "o")
    c.close(Case.f64(S_final), r.M, None, r.M_mag, "S_final", out=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", CASES)
def test_backward(S, name, dtype):
    c = Case(2, dtype=dtype, **CASES[name])
    dq, dk, dv, dS0 = (Case.f64(x) for x in c.backward(S))
    a, KV = c.np, c.shape[3]
    rq, rk, rv = M.linattn_backward(a["q"], a["k"], a["v"], a["g"], c.scale, a["g_o"], c.np_lens, a["S0"], a["g_S"])
    c.close(dq, rq.out, rq.once, rq.mag, "dq")
    for got, r, what in ((dk, rk, "dk"), (dv, rv, "dv")):
        c.close(got, *(M.sum_shared(x, KV) for x in (r.out, r.once, r.mag)), what)
    c.close(dS0, rv.M, None, rv.M_mag, "dS0", out=False)


@pytest.mark.parametrize("L", [1, 3, 8])
def test_a_few_bf16_tokens_are_rounded_at_the_end_only(S, L):
    c = Case(11, 2, L, 4, 4, 128, 64, "bf16")
    a = c.np
    o, S_final = c.forward(S)
    r = M.linattn_forward(a["q"], a["k"], a["v"], a["g"], c.scale, None, a["S0"])
    c.close(Case.f64(o), r.out, 0, r.mag, "o")
    c.close(Case.f64(S_final), r.M, None, r.M_mag, "S_final", out=False)
    got = [Case.f64(x) for x in c.backward(S)]
    roles = M.linattn_backward(a["q"], a["k"], a["v"], a["g"], c.scale, a["g_o"], None, a["S0"], a["g_S"])
    for x, r, what in zip(got, roles, ("dq", "dk", "dv")):
        c.close(x, r.out, 0, r.mag, what)
    c.close(got[3], roles[2].M, None, roles[2].M_mag, "dS0", out=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 64, 64), (5, 6, 2, 128, 128), (3, 4, 4, 8, 128), (2, 3, 3, 128, 8),
                                   (2, 2, 1, 96, 24), (300, 2, 2, 64, 128)])
def test_step(S, shape, dtype):
    B, H, KV, dk, dv = shape
    c = Case(3, B, 1, H, KV, dk, dv, dtype, fused=True)
    o = torch.empty(B, 1, H, dv, device="cuda", dtype=c.t)
    out = torch.empty_like(c.S0)
    S.check(S.swimba_linattn_step(c.dims(S), c.q, c.k, c.v, c.g, c.S0, o, out))
    a = c.np
    r = M.linattn_forward(a["q"], a["k"], a["v"], a["g"], c.scale, None, a["S0"])
    c.close(Case.f64(o), r.out, 0, r.mag, "o")
    c.close(Case.f64(out), r.M, None, r.M_mag, "S", out=False)
    o2, state = torch.empty_like(o), c.S0.clone()
    S.check(S.swimba_linattn_step(c.dims(S), c.q, c.k, c.v, c.g, state, o2, state))
    assert torch.equal(o, o2) and torch.equal(out, state)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_prompt_then_tokens_is_the_longer_prompt(S, dtype):
    """Prefill of 200 tokens and 60 single tokens from its state, against one prompt of 260."""
    c = Case(4, 2, 260, 3, 3, 64, 128, dtype)
    whole, end = c.forward(S)
    head = Case(4, 2, 260, 3, 3, 64, 128, dtype)
    head.q, head.k, head.v = (x[:, :200].contiguous() for x in (c.q, c.k, c.v))
    head.shape = (2, 200, 3, 3, 64, 128)
    _, state = head.forward(S)
    a = c.np
    r = M.linattn_forward(a["q"], a["k"], a["v"], a["g"], c.scale, None, a["S0"])
    for t in range(200, 260):
        q, k, v = (x[:, t:t + 1].contiguous() for x in (c.q, c.k, c.v))
        o = torch.empty(2, 1, 3, 128, device="cuda", dtype=c.t)
        S.check(S.swimba_linattn_step(S.make_linattn_dims(q, k, v, c.scale), q, k, v, c.g, state, o, state))
        c.close(Case.f64(o)[:, 0], r.out[:, t], 0, r.mag[:, t], f"token {t}")
    c.close(Case.f64(state), r.M, None, r.M_mag, "state", out=False)
    c.close(Case.f64(end), r.M, None, r.M_mag, "S_final", out=False)
    c.close(Case.f64(whole), r.out, r.once, r.mag, "o")


@pytest.mark.parametrize("name", ["lens", "split", "split_lens", "shared", "cut"])
def test_in_place_state_repeats_graphs_and_streams(S, name):
    """S_final over S0, two runs, a captured and replayed call, and a call on another stream give the same
    bits (every sum has a fixed order)."""
    c = Case(5, dtype="bf16", **CASES[name])
    B, L, H, KV, dk, dv = c.shape
    o = torch.zeros(B, L, H, dv, device="cuda", dtype=c.t)
    o, S_final = c.forward(S, o)
    start = c.S0.clone()
    o2 = torch.zeros_like(o)
    c.forward(S, o2, c.S0)
    assert torch.equal(c.S0, S_final)
    c.S0 = start
    live = lambda x: torch.nan_to_num(x.float(), nan=0.0)
    assert torch.equal(live(o), live(o2))
    d = c.dims(S)
    ws = S.new_linattn_workspace(d, S.SWIMBA_OP_LINATTN_FWD)
    o3, S3 = torch.zeros_like(o), torch.empty_like(S_final)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call = lambda s: S.check(S.swimba_linattn_fwd(d, c.q, c.k, c.v, c.g, c.lens, c.S0, o3, S3, ws, ws.numel(), s))
    call(side)
    side.synchronize()
    assert torch.equal(live(o3), live(o)) and torch.equal(S3, S_final)
    o3.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side, capture_error_mode="relaxed"):
        call(torch.cuda.current_stream())
    for _ in range(2):
        S3.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(live(o3), live(o)) and torch.equal(S3, S_final)
    del graph
    first = c.backward(S)
    again = c.backward(S)
    assert all(torch.equal(x, y) for x, y in zip(first, again))


@pytest.mark.parametrize("d", [64, 128])
def test_sequences_cut_between_ctas_are_whole(S, d):
    """160 heads share the SMs chunk by chunk, 80 do not: the same bits, for outputs and gradients."""
    c = Case(8, 1, 1900, 160, 160, d, d, "bf16", scale=0.1)
    o, S_final = c.forward(S)
    grads = c.backward(S)
    for h in (0, 80):
        part = Case(8, 1, 1900, 80, 80, d, d, "bf16", scale=0.1)
        cut = lambda x: x[:, :, h:h + 80].contiguous()
        part.q, part.k, part.v, part.g_o = (cut(x) for x in (c.q, c.k, c.v, c.g_o))
        part.S0, part.g_S, part.g = c.S0[:, h:h + 80].contiguous(), c.g_S[:, h:h + 80].contiguous(), c.g[h:h + 80].contiguous()
        po, pS = part.forward(S)
        assert torch.equal(cut(o), po) and torch.equal(S_final[:, h:h + 80], pS)
        for got, want in zip(grads[:3], part.backward(S)[:3]):
            assert torch.equal(cut(got), want)


def test_a_value_that_is_not_finite_stays_in_its_sequence(S):
    c = Case(6, 3, 300, 2, 2, 64, 64, "bf16")
    clean, end = c.forward(S)
    c.v[1, 200] = float("nan")
    c.k[1, 290] = float("inf")
    o, S_final = c.forward(S)
    for b in (0, 2):
        assert torch.equal(o[b], clean[b]) and torch.equal(S_final[b], end[b])
    assert torch.equal(o[1, :128], clean[1, :128])  # earlier chunks too
    assert not torch.isfinite(o[1, 200]).any()


def test_offsets_past_32_bits(S):
    """q, k, v as columns of a buffer whose last tokens lie more than 2^31 elements in."""
    L, width = 300, 2 ** 23
    free = torch.cuda.mem_get_info()[0]
    if free < 12 << 30:
        pytest.skip("needs 6 GB of device memory")
    buf = torch.zeros(1, L, width, device="cuda", dtype=torch.bfloat16)
    c = Case(7, 1, L, 1, 1, 64, 64, "bf16")
    want = c.forward(S)
    views = [buf[:, :, i * 64:(i + 1) * 64].unflatten(2, (1, 64)) for i in range(3)]
    for view, x in zip(views, (c.q, c.k, c.v)):
        view.copy_(x)
    c.q, c.k, c.v = views
    got = c.forward(S)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# Log decays whose γ and γ^128 lie far from the fp32 number next to them (0.05 to 0.5 of its last place), and slow enough
# that a state outlives thousands of tokens. Larger than a state's own last place: what a slower decay takes from
# an fp32 state at a token is lost in its rounding.
SLOW = [-1.0e-5, -2.3e-5, -2.0 ** -12 * 1.01, -3.3e-4]


def mean_drift(got, start, g, n):
    """Per head, the mean over its elements of the error of a state that only decayed, relative to the state. An
    update rounds each element by at most 2^-24 of it, to either side: over the 4096 elements or more of a head the
    mean of 4096 updates' roundings has a standard deviation below 2^-24 64 / 64 = 2^-24. The decays' own error is
    2^-23 of the whole exponent (at most 2 here). 2^-20 is beyond both; γ rounded to fp32 leaves n 2^-27 or more."""
    want = start.double() * torch.exp(g.double() * n)[None, :, None, None]
    return ((got.double() - want) / want).mean(dim=(0, 2, 3)).abs().max().item()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_single_tokens_keep_the_decay(S, dtype):
    """4096 tokens of zero keys: the state is its start times exp(4096 log_decay)."""
    c = Case(12, 2, 1, len(SLOW), len(SLOW), 64, 64, dtype, decay=torch.tensor(SLOW))
    c.k.zero_()
    start = 1 + torch.rand_like(c.S0)
    state, o, d = start.clone(), torch.empty(2, 1, len(SLOW), 64, device="cuda", dtype=c.t), c.dims(S)
    for _ in range(4096):
        S.check(S.swimba_linattn_step(d, c.q, c.k, c.v, c.g, state, o, state))
    assert mean_drift(state, start, c.g, 4096) < 2.0 ** -20


@pytest.mark.parametrize("dtype,H,L", [("bf16", 3, 32768), ("bf16", 150, 32768), ("bf16", 150, 32700), ("f32", 3, 32768)])
def test_long_sequences_keep_the_decay(S, dtype, H, L):
    """Zero keys leave S_final = exp(L log_decay) S0, zero g_o leaves dS0 = exp(L log_decay) g_S: over segments (3
    heads), and over 256 chunks in a row in whole and cut sequences (150 heads)."""
    t, d = (torch.bfloat16 if dtype == "bf16" else torch.float32), 64
    g = torch.tensor([-1.0e-5, -1.728e-5, -1.97e-5, -2.4557e-5, -4.6393e-5, -5.3672e-5], device="cuda")
    g = g.repeat(H // 6 + 1)[:H].contiguous()
    q, k = torch.ones(1, L, H, d, device="cuda", dtype=t), torch.zeros(1, L, H, d, device="cuda", dtype=t)
    dims = S.make_linattn_dims(q, k, k, 1.0)
    start, end, o = 1 + torch.rand(1, H, d, d, device="cuda"), torch.empty(1, H, d, d, device="cuda"), torch.empty_like(q)
    ws = S.new_linattn_workspace(dims, S.SWIMBA_OP_LINATTN_FWD)
    S.check(S.swimba_linattn_fwd(dims, q, k, k, g, None, start, o, end, ws, ws.numel()))
    assert S.swimba_get_device_status(ws) == 0
    assert mean_drift(end, start, g, L) < 2.0 ** -20
    ws = S.new_linattn_workspace(dims, S.SWIMBA_OP_LINATTN_BWD)
    grads = [torch.empty_like(q) for _ in range(3)]
    S.check(S.swimba_linattn_bwd(dims, q, k, k, g, None, None, k, start, *grads, end, ws, ws.numel()))
    assert S.swimba_get_device_status(ws) == 0
    assert mean_drift(end, start, g, L) < 2.0 ** -20


@pytest.mark.parametrize("H,L", [(149, 16384), (160, 16384), (175, 20000)])
def test_more_heads_than_sms_stay_whole(S, H, L):
    """Long sequences of a few more heads than SMs go in equal shares and not through segments, which read keys and
    values twice: one launch, and the results that the same heads give in calls of fewer, which go another way."""
    c = Case(13, 1, 1, H, H, 16, 8, "bf16", decay=-torch.exp2(torch.linspace(-1, -14, H)))
    g = torch.Generator(device="cuda")
    g.manual_seed(14)
    q, k, v = (torch.randn(1, L, H, d, generator=g, device="cuda").bfloat16() for d in (16, 16, 8))

    def forward(first, last):
        x = [t[:, :, first:last].contiguous() for t in (q, k, v)]
        S0, decay = c.S0[:, first:last].contiguous(), c.g[first:last].contiguous()
        d = S.make_linattn_dims(*x, 0.25)
        ws = S.new_linattn_workspace(d, S.SWIMBA_OP_LINATTN_FWD)
        o, end = torch.empty_like(x[2]), torch.empty_like(S0)
        before = S.swimba_kernel_launches()
        S.check(S.swimba_linattn_fwd(d, *x, decay, None, S0, o, end, ws, ws.numel()))
        assert S.swimba_get_device_status(ws) == 0
        return o, end, S.swimba_kernel_launches() - before

    o, end, launches = forward(0, H)
    assert launches == 1
    for first in range(0, H, 100):
        part, part_end, _ = forward(first, min(first + 100, H))
        # the two ways differ in where fp32 sums are cut: the states by roundings of their own size, the outputs
        # where such a difference crosses a bf16 rounding of the scores, of the state's copy or of the output
        got, want = o[:, :, first:first + 100].float(), part.float()
        size = want.square().mean().sqrt()
        assert (got - want).abs().max() <= 2.0 ** -8 * (want.abs() + 4 * size).max()
        assert (got - want).square().mean().sqrt() <= 2.0 ** -10 * size
        state = part_end.square().mean().sqrt()
        assert (end[:, first:first + 100] - part_end).abs().max() <= 2.0 ** -17 * (part_end.abs().max() + state)


# Sizes that pad differently (other instances of the kernel; gradients in two launches), in segments and in shares.
UNEVEN = {
    "split_64x128": dict(B=1, L=1500, H=1, KV=1, dk=64, dv=128),
    "split_128x64": dict(B=1, L=1500, H=1, KV=1, dk=128, dv=64, start=False),
    "split_lens_72x40": dict(B=2, L=1700, H=2, KV=1, dk=72, dv=40, lens=[1430, 400]),
    "split_lens_24x104": dict(B=3, L=1700, H=2, KV=2, dk=24, dv=104, lens=[1537, 0, 129], fused=True),
    "cut_16x72": dict(B=1, L=900, H=149, KV=149, dk=16, dv=72),
    "cut_72x16_shared": dict(B=1, L=700, H=150, KV=50, dk=72, dv=16),
}


@pytest.mark.parametrize("name", UNEVEN)
def test_uneven_head_sizes_in_segments_and_shares(S, name):
    c = Case(15, dtype="bf16", **UNEVEN[name])
    B, L, H, KV, dk, dv = c.shape
    o, S_final = c.forward(S, torch.zeros(B, L, H, dv, device="cuda", dtype=c.t))
    a = c.np
    r = M.linattn_forward(a["q"], a["k"], a["v"], a["g"], c.scale, c.np_lens, a["S0"])
    c.close(Case.f64(o), r.out, r.once, r.mag, "o")
    c.close(Case.f64(S_final), r.M, None, r.M_mag, "S_final", out=False)
    dq, dk, dv, dS0 = (Case.f64(x) for x in c.backward(S))
    rq, rk, rv = M.linattn_backward(a["q"], a["k"], a["v"], a["g"], c.scale, a["g_o"], c.np_lens, a["S0"], a["g_S"])
    c.close(dq, rq.out, rq.once, rq.mag, "dq")
    for got, r, what in ((dk, rk, "dk"), (dv, rv, "dv")):
        c.close(got, *(M.sum_shared(x, KV) for x in (r.out, r.once, r.mag)), what)
    c.close(dS0, rv.M, None, rv.M_mag, "dS0", out=False)


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (64, 128)])
def test_gradients_of_cut_sequences_are_those_of_whole_ones(S, dk, dv):
    """160 heads make 480 pieces of work, in equal shares over the SMs; 40 heads 120, fewer than there are SMs, which
    are never cut: the same bits, the states' gradients included."""
    c = Case(16, 1, 1900, 160, 160, dk, dv, "bf16", scale=0.1)
    whole = c.backward(S)
    for h in range(0, 160, 40):
        part = Case(16, 1, 1900, 40, 40, dk, dv, "bf16", scale=0.1)
        cut = lambda x: x[:, :, h:h + 40].contiguous()
        part.q, part.k, part.v, part.g_o = (cut(x) for x in (c.q, c.k, c.v, c.g_o))
        part.S0, part.g_S = c.S0[:, h:h + 40].contiguous(), c.g_S[:, h:h + 40].contiguous()
        part.g = c.g[h:h + 40].contiguous()
        *grads, dS0 = part.backward(S)
        for got, want in zip(whole, grads):
            assert torch.equal(cut(got), want)
        assert torch.equal(whole[3][:, h:h + 40], dS0)


def two_part_loss(w, v):
    """What of the fp32 product w v its first two truncated bf16 parts leave out, relative to the product."""
    top = lambda x: (x.view(np.uint32) & np.uint32(0xffff0000)).view(np.float32)
    x = (np.float32(w) * v).astype(np.float32)
    rest = x - top(x)
    return (rest - top(rest)) / x


@pytest.mark.parametrize("L,at", [(32, 0), (672, 0), (672, 640), (1536, 0), (1536, 1504)])
def test_states_hold_24_bits(S, L, at):
    """S_final and dS0 from values whose decayed products need all 24 bits: of every bf16 in [1, 2) the one whose product
    loses most in two parts. 32 tokens of them stand at the sequence's beginning or end, zeros elsewhere; all
    terms have one sign, so that what is lost adds up. (The longest go in segments.)
    Tolerance: a power is off by 2 fp32 steps, 2^-22, its factor and the product by 2^-24 each; the 32 tokens are
    2 steps of 16 of 3 parts each, 6 products whose running sum is kept to 2^-22; 11 chunks or segments more round the state by 2^-24
    each: 41 2^-24, below 3 2^-20. Two parts would be off by more than twice that."""
    tol, g, d = 3 * 2.0 ** -20, -1e-3, 64
    values = (1 + np.arange(128) / 128).astype(np.float32)
    gd = float(np.float32(g))
    tokens = np.arange(at, at + 32)
    in_chunk = tokens % 128
    size = min(128, L - at // 128 * 128)
    decay = torch.tensor([g], device="cuda")
    ones, zeros = torch.ones(1, 1, 1, d, device="cuda").bfloat16(), torch.zeros(1, L, 1, d, device="cuda").bfloat16()

    def stream(weights):
        """[1, L, 1, d] of the chosen values, and those in fp64; the loss of two parts is past the tolerance."""
        chosen = np.array([values[np.argmax(two_part_loss(w, values))] for w in weights])
        lost = np.array([float(two_part_loss(w, v[None])[0]) for w, v in zip(weights, chosen)])
        assert (lost * weights * chosen).sum() > 2 * tol * (weights * chosen).sum()
        x = zeros.clone()
        x[0, tokens, 0] = torch.from_numpy(chosen).cuda().bfloat16()[:, None]
        return x, chosen.astype(np.float64)

    def near(got, want):
        assert (got.double() / want - 1).abs().max().item() < tol

    one = zeros.clone()
    one[0, tokens, 0] = 1
    v, chosen = stream(np.exp(gd * (size - 1 - in_chunk)).astype(np.float32))
    dims = S.make_linattn_dims(one, one, v, 1.0)
    ws = S.new_linattn_workspace(dims, S.SWIMBA_OP_LINATTN_FWD)
    o, state = torch.empty_like(v), torch.empty(1, 1, d, d, device="cuda")
    S.check(S.swimba_linattn_fwd(dims, one, one, v, decay, None, None, o, state, ws, ws.numel()))
    assert S.swimba_get_device_status(ws) == 0
    near(state, (np.exp(gd * (L - 1 - tokens)) * chosen).sum())
    g_o, chosen = stream(np.exp(gd * (in_chunk + 1)).astype(np.float32))
    ws = S.new_linattn_workspace(dims, S.SWIMBA_OP_LINATTN_BWD)
    grads = [torch.empty_like(v) for _ in range(3)]
    S.check(S.swimba_linattn_bwd(dims, one, one, v, decay, None, None, g_o, None, *grads, state, ws, ws.numel()))
    assert S.swimba_get_device_status(ws) == 0
    near(state, (np.exp(gd * (tokens + 1)) * chosen).sum())


@pytest.mark.parametrize("B", [2, 148])
def test_fp32_keeps_decays_next_to_one(S, B):
    """Decays of which a token takes about one last place of an fp32 state, or fewer: zero keys leave the start times
    exp(L log_decay), zero g_o the end's gradient times it, over segments (8 heads) and token by token (592 heads).
    Rounded at every token they would be off by a part of that place each time, all in one direction: 4e-5 of the state.
    Decayed every 16 tokens, an element's 256 roundings of at most 2^-24 of it may all be alike, but not those
    of a head's 512 elements or more: their mean has a standard deviation below 256 2^-24 / 22 / 3^0.5 = 4e-7 for 2
    sequences and 5e-8 for 148, 7 of which are below 3e-6 and 2^-20 with the decays' own 2^-23."""
    L, d = 4096, 16
    g = -torch.tensor([1.5 * 2.0 ** -24, 1.3 * 2.0 ** -23, 1.5 * 2.0 ** -22, 2.0 ** -20], device="cuda")
    H = len(g)
    q, k = torch.ones(B, L, H, d, device="cuda"), torch.zeros(B, L, H, d, device="cuda")
    dims = S.make_linattn_dims(q, k, k, 1.0)
    start, end, o = 1 + torch.rand(B, H, d, d, device="cuda"), torch.empty(B, H, d, d, device="cuda"), torch.empty_like(q)
    ws = S.new_linattn_workspace(dims, S.SWIMBA_OP_LINATTN_FWD)
    S.check(S.swimba_linattn_fwd(dims, q, k, k, g, None, start, o, end, ws, ws.numel()))
    tol = 3e-6 if B == 2 else 2.0 ** -20
    assert mean_drift(end, start, g, L) < tol
    ws = S.new_linattn_workspace(dims, S.SWIMBA_OP_LINATTN_BWD)
    grads = [torch.empty_like(q) for _ in range(3)]
    S.check(S.swimba_linattn_bwd(dims, q, k, k, g, None, None, k, start, *grads, end, ws, ws.numel()))
    assert mean_drift(end, start, g, L) < tol


@pytest.mark.parametrize("decay", [0.0, -1e-5, -0.3, -0.7])
def test_an_infinite_state_stays_infinite(S, decay):
    """A single token, and segments that hand the state on: infinite elements stay what they are, the others too."""
    for L in (1, 1500):
        c = Case(17, 1, L, 1, 1, 64, 64, "bf16", decay=decay if L == 1 else decay / 500)
        states = []
        for _ in range(2):
            o, end = torch.empty_like(c.q), torch.empty_like(c.S0)
            if L == 1:
                S.check(S.swimba_linattn_step(c.dims(S), c.q, c.k, c.v, c.g, c.S0, o, end))
            else:
                c.forward(S, o, end)
            states.append(end)
            c.S0[0, 0, 3, 5], c.S0[0, 0, 60, 1] = float("inf"), -float("inf")
        want = states[0].clone()
        want[0, 0, 3, 5], want[0, 0, 60, 1] = float("inf"), -float("inf")
        assert torch.equal(states[1], want)
