"""The norms around a block through the C ABI against the fp64 oracle, forward and backward.

Tolerances: the kernel works in fp32 on values each of which is off by at most 2^-24 of the terms it adds,
over sums of at most `width` terms; the exponential and reciprocal of the gate are within 2^-20 (their
fp32 argument up to |z| = 8 included). So a result is within (width + 96) 2^-24 of the sum of its absolute
terms (the oracle's ``mag``), a weight gradient within (rows + width + 96) 2^-24, and a bf16 result
within half a bf16 step, 2^-8 of it, of that."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import mixer_oracle as M

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def S():
    from parameter_space_moe_swimba_b200 import swimba

    return swimba


T = {"f32": torch.float32, "bf16": torch.bfloat16}


class Case:
    def __init__(self, seed, rows, width, groups=1, io="bf16", res_t="bf16", z=True, post=True, res=True, pre=True,
                 gate_last=False, y=True, g_h=True, res_scale=0.75, out_scale=0.5, eps=1e-5):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        n = lambda *s: torch.randn(s, generator=g, device="cuda")
        self.io, self.res_t, self.rows, self.width = io, res_t, rows, width
        row = lambda on, t: n(rows, width).to(T[t]) if on else None
        self.y, self.z, self.res = row(y, io), row(z, io), row(res, res_t)
        if self.z is not None:
            self.z.clamp_(-8, 8)
        self.w_post, self.w_pre = (1 + 0.3 * n(width) if on else None for on in (post, pre))
        self.g_h, self.g_n = row(g_h, res_t), row(pre, io)
        self.kw = dict(groups=groups, eps=eps, gate_last=gate_last, res_scale=res_scale, out_scale=out_scale)

    def inputs(self):
        return self.y, self.z, self.w_post, self.res, self.w_pre

    def np(self):
        return [None if x is None else x.double().cpu().numpy() for x in self.inputs()]

    def dims(self, S):
        like = lambda t: torch.empty(self.rows, self.width, dtype=T[t], device="meta")
        return S.make_norm_dims(like(self.io), like(self.res_t), **self.kw)

    def forward(self, S, want_h=True, stream=None):
        h = torch.full((self.rows, self.width), 7.0, device="cuda", dtype=T[self.res_t]) if want_h else None
        n = torch.full((self.rows, self.width), 7.0, device="cuda", dtype=T[self.io]) if self.w_pre is not None else None
        S.check(S.swimba_block_norm_fwd(self.dims(S), *self.inputs(), h, n, stream))
        return h, n

    def backward(self, S, stream=None):
        like = lambda x: None if x is None else torch.full_like(x, 7.0)
        out = dict(dy=like(self.y), dz=like(self.z), dres=like(self.res), dw_post=like(self.w_post), dw_pre=like(self.w_pre))
        d = self.dims(S)
        ws = S.new_norm_workspace(d)
        S.check(S.swimba_block_norm_bwd(d, *self.inputs(), self.g_h, self.g_n, out["dy"], out["dz"], out["dres"],
                                        out["dw_post"], out["dw_pre"], ws, ws.numel(), stream))
        return out

    def close(self, got, want, mag, what, t, terms=0):
        got = got.double().cpu().numpy()
        tol = (terms + self.width + 96) * 2.0 ** -24 * mag
        if t == "bf16":
            tol = tol + 2.0 ** -8 * np.abs(want)
        off = np.abs(got - want) - tol
        assert (off <= 1e-30).all(), (what, float(off.max()), float(np.abs(got - want).max()))

    def check(self, S):
        f = M.block_norm_forward(*self.np(), **self.kw)
        h, n = self.forward(S)
        self.close(h, f["h"], f["h_mag"], "h", self.res_t)
        if n is not None:
            self.close(n, f["n"], f["n_mag"], "n", self.io)
        g = [None if x is None else x.double().cpu().numpy() for x in (self.g_h, self.g_n)]
        want = M.block_norm_backward(*self.np(), *g, **self.kw)
        got = {k: v for k, v in self.backward(S).items() if v is not None}
        assert set(got) == set(want)
        for k, (w, mag) in want.items():
            t = "f32" if k.startswith("dw") else self.res_t if k == "dres" else self.io
            self.close(got[k], w, mag, k, t, terms=self.rows if k.startswith("dw") else 0)


TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")]


@pytest.mark.parametrize("io,res_t", TYPES)
@pytest.mark.parametrize("rows,width,groups", [
    (1, 8, 1), (5, 24, 3), (3, 64, 8), (7, 256, 1), (9, 264, 3), (4, 512, 4), (130, 520, 5), (6, 1024, 32), (5, 1032, 1),
    (3, 1536, 12), (2, 2048, 16), (3, 2056, 257), (2, 4096, 1), (300, 4096, 32), (2, 4104, 3), (2, 8192, 8), (1, 8200, 5),
    (2, 16384, 1), (1, 16384, 2048)])
def test_sizes(S, rows, width, groups, io, res_t):
    Case(1, rows, width, groups, io, res_t).check(S)


@pytest.mark.parametrize("gate_last", [False, True])
@pytest.mark.parametrize("rows,width,groups,io,res_t", [
    (900, 4096, 1, "bf16", "f32"), (900, 4096, 16, "f32", "f32"), (900, 4080, 5, "f32", "f32"), (460, 8192, 2, "bf16", "f32"),
    (460, 16384, 1, "bf16", "bf16"), (460, 12288, 3, "f32", "bf16")])
def test_wide_rows_one_after_the_other(S, rows, width, groups, io, res_t, gate_last):
    """Several rows per CTA where shared memory holds one, one and a half, or two."""
    Case(10, rows, width, groups, io, res_t, gate_last=gate_last).check(S)


@pytest.mark.parametrize("gate_last", [False, True])
@pytest.mark.parametrize("parts", ["z", "post", "res", "pre", "z post", "z res", "post pre", "z pre", "post res", "res pre",
                                   "z post res", "z post pre", "z res pre", "post res pre", "z post res pre", ""])
def test_parts(S, parts, gate_last):
    on = {n: n in parts.split() for n in ("z", "post", "res", "pre")}
    Case(2, 11, 768, 6, "bf16", "f32", gate_last=gate_last, **on).check(S)


@pytest.mark.parametrize("res_t", ["bf16", "f32"])
def test_without_a_mixer_output(S, res_t):
    """y NULL: the residual stream's own norm."""
    Case(3, 9, 512, 1, "bf16", res_t, z=False, post=False, y=False).check(S)


def test_without_g_h(S):
    Case(4, 9, 512, 4, "bf16", "f32", g_h=False).check(S)


@pytest.mark.parametrize("rows", [1, 3, 4, 295, 296, 297, 1185, 2000])
def test_weight_gradients_over_rows(S, rows):
    """Row counts around the backward's grid, at a warp and at a CTA per row."""
    Case(5, rows, 64, 2, "f32", "f32").check(S)
    Case(6, rows, 1536, 1, "bf16", "bf16").check(S)


@pytest.mark.parametrize("size,eps", [(1e-12, 1e-28), (1e12, 1e-5), (0.0, 1e-30)])
def test_sizes_of_values_far_from_one(S, size, eps):
    """Rows of tiny, huge and no values: no intermediate leaves fp32's range where the results do not."""
    c = Case(12, 20, 1024, io="f32", res_t="f32", z=False, post=False, eps=eps)
    c.y *= size
    c.res *= size
    c.g_h *= min(1.0, 1 / max(size, 1e-12))
    c.check(S)


def test_rows_of_zeros_and_rows_that_are_not_finite(S):
    c = Case(7, 6, 256, 2, "bf16", "bf16", gate_last=True)
    clean = c.forward(S)
    grads = c.backward(S)
    c.y[1] = 0
    c.res[1] = 0
    h, n = c.forward(S)
    assert not h[1].any() and not n[1].any()
    assert all(torch.isfinite(v).all() for v in c.backward(S).values())
    c.y[2, 5] = float("inf")
    c.z[3, 7] = float("nan")
    h, n = c.forward(S)
    g = c.backward(S)
    for b in (0, 4, 5):
        assert torch.equal(h[b], clean[0][b]) and torch.equal(n[b], clean[1][b])
        assert all(torch.equal(g[k][b], grads[k][b]) for k in ("dy", "dz", "dres"))


def test_in_place_outputs_repeats_and_graphs(S):
    """h over res, n over y; dres over g_h, dy over g_n, dz over z; a captured call: the same bits."""
    c = Case(8, 70, 1536, 12, "bf16", "bf16")
    h, n = c.forward(S)
    grads = c.backward(S)
    y, z, res = c.y.clone(), c.z.clone(), c.res.clone()
    S.check(S.swimba_block_norm_fwd(c.dims(S), y, z, c.w_post, res, c.w_pre, res, y))
    assert torch.equal(res, h) and torch.equal(y, n)
    z, g_h, g_n = c.z.clone(), c.g_h.clone(), c.g_n.clone()
    d = c.dims(S)
    ws = S.new_norm_workspace(d)
    dp, dn = torch.empty_like(c.w_post), torch.empty_like(c.w_pre)
    S.check(S.swimba_block_norm_bwd(d, c.y, z, c.w_post, c.res, c.w_pre, g_h, g_n, g_n, z, g_h, dp, dn, ws, ws.numel()))
    for got, k in ((g_n, "dy"), (z, "dz"), (g_h, "dres"), (dp, "dw_post"), (dn, "dw_pre")):
        assert torch.equal(got, grads[k]), k
    out = {k: torch.zeros_like(v) for k, v in grads.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side, capture_error_mode="relaxed"):
        S.check(S.swimba_block_norm_bwd(d, *c.inputs(), c.g_h, c.g_n, out["dy"], out["dz"], out["dres"], out["dw_post"],
                                        out["dw_pre"], ws, ws.numel(), torch.cuda.current_stream()))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out[k], grads[k]) for k in out)
    del graph


def test_offsets_past_32_bits(S):
    """Rows more than 2^31 elements in give the bits that they give as the first rows."""
    rows, width = 2 ** 18 + 40, 8192
    if torch.cuda.mem_get_info()[0] < 28 << 30:
        pytest.skip("needs 18 GB of device memory")
    c = Case(9, 50, width, groups=2, z=False, res=False)
    h, n = c.forward(S)
    back = c.backward(S)
    big = Case(9, 50, width, groups=2, z=False, res=False)
    big.rows = rows
    big.y, big.g_h, big.g_n = (torch.zeros(rows, width, device="cuda", dtype=x.dtype) for x in (c.y, c.g_h, c.g_n))
    for x, part in ((big.y, c.y), (big.g_h, c.g_h), (big.g_n, c.g_n)):
        x[-50:] = part
    got_h, got_n = big.forward(S)
    assert torch.equal(got_h[-50:], h) and torch.equal(got_n[-50:], n) and not got_n[:-50].any()
    del got_h, got_n
    dy = big.backward(S)["dy"]
    assert torch.equal(dy[-50:], back["dy"]) and not dy[:-50].any()
