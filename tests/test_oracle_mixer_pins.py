"""Pins of the mixer oracle: linear attention against the brute-force double sum, its pieces and its
gradients against central differences; the block norms' gradients against central differences and their
parts against closed forms. CPU, fp64."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import mixer_oracle as M


def draw(rng, B=2, L=7, H=4, KV=2, dk=3, dv=5):
    n = rng.standard_normal
    return dict(q=n((B, L, H, dk)), k=n((B, L, KV, dk)), v=n((B, L, KV, dv)), g=-rng.random(H), S0=n((B, H, dk, dv)),
                g_o=n((B, L, H, dv)), g_S=n((B, H, dk, dv)), lens=np.array([L, 4])[:B], scale=0.7)


def test_forward_is_the_double_sum():
    a = draw(np.random.default_rng(0))
    r = M.linattn_forward(a["q"], a["k"], a["v"], a["g"], a["scale"], a["lens"], a["S0"])
    for b in range(2):
        for h in range(4):
            kv = h // 2
            for t in range(a["lens"][b]):
                o = np.exp(a["g"][h] * (t + 1)) * a["q"][b, t, h] @ a["S0"][b, h]
                for s in range(t + 1):
                    o = o + np.exp(a["g"][h] * (t - s)) * (a["q"][b, t, h] @ a["k"][b, s, kv]) * a["v"][b, s, kv]
                np.testing.assert_allclose(r.out[b, t, h], a["scale"] * o, rtol=1e-12, atol=1e-12)
    assert not r.out[1, 4:].any()


def test_a_state_carries_a_sequence_on():
    a = draw(np.random.default_rng(1))
    whole = M.linattn_forward(a["q"], a["k"], a["v"], a["g"], a["scale"], None, a["S0"])
    cut = lambda lo, hi: (a["q"][:, lo:hi], a["k"][:, lo:hi], a["v"][:, lo:hi], a["g"], a["scale"], None)
    first = M.linattn_forward(*cut(0, 3), a["S0"])
    second = M.linattn_forward(*cut(3, 7), first.M)
    np.testing.assert_allclose(np.concatenate([first.out, second.out], 1), whole.out, rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(second.M, whole.M, rtol=1e-12, atol=1e-12)


def test_no_decay_and_full_decay():
    a = draw(np.random.default_rng(2), B=1, KV=4)
    zero = np.zeros(4)
    r = M.linattn_forward(a["q"], a["k"], a["v"], zero, 1.0)
    want = np.einsum("bthd,bshd,ts,bshc->bthc", a["q"], a["k"], np.tril(np.ones((7, 7))), a["v"])
    np.testing.assert_allclose(r.out, want, rtol=1e-12, atol=1e-12)
    r = M.linattn_forward(a["q"], a["k"], a["v"], np.full(4, -np.inf), 1.0, None, a["S0"])
    np.testing.assert_allclose(r.out, (a["q"] * a["k"]).sum(-1, keepdims=True) * a["v"], rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("name", ["q", "k", "v", "S0"])
def test_gradients_are_the_differences(name):
    rng = np.random.default_rng(3)
    a = draw(rng)

    def loss(x):
        c = dict(a, **{name: x})
        r = M.linattn_forward(c["q"], c["k"], c["v"], c["g"], c["scale"], c["lens"], c["S0"])
        return (r.out * a["g_o"]).sum() + (r.M * a["g_S"]).sum()

    dq, dk, dv = M.linattn_backward(a["q"], a["k"], a["v"], a["g"], a["scale"], a["g_o"], a["lens"], a["S0"], a["g_S"])
    grad = {"q": dq.out, "k": M.sum_shared(dk.out, 2), "v": M.sum_shared(dv.out, 2), "S0": dv.M}[name]
    for _ in range(4):
        d = rng.standard_normal(a[name].shape)
        e = 1e-5
        got = (loss(a[name] + e * d) - loss(a[name] - e * d)) / (2 * e)
        assert abs(got - (grad * d).sum()) <= 1e-7 * (1 + abs(got))


def test_an_empty_sequence_keeps_its_state():
    a = draw(np.random.default_rng(4))
    lens = np.array([0, 7])
    r = M.linattn_forward(a["q"], a["k"], a["v"], a["g"], 1.0, lens, a["S0"])
    assert np.array_equal(r.M[0], a["S0"][0]) and not r.out[0].any()
    _, _, dv = M.linattn_backward(a["q"], a["k"], a["v"], a["g"], 1.0, a["g_o"], lens, a["S0"], a["g_S"])
    assert np.array_equal(dv.M[0], a["g_S"][0])


def test_tolerance_parts_bound_the_values():
    a = draw(np.random.default_rng(5), B=1, L=300, H=2, KV=2)
    r = M.linattn_forward(a["q"], a["k"], a["v"], a["g"], 0.5, None, a["S0"])
    for role in (r, *M.linattn_backward(a["q"], a["k"], a["v"], a["g"], 0.5, a["g_o"], None, a["S0"], a["g_S"])):
        assert (np.abs(role.out) <= role.once * (1 + 1e-9)).all() and (role.once <= role.mag * (1 + 1e-9)).all()


NORMS = [dict(z=1, post=1, res=1, pre=1, groups=1), dict(z=1, post=1, res=1, pre=1, groups=3, gate_last=True),
         dict(z=1, post=1, res=0, pre=0, groups=2), dict(z=0, post=0, res=1, pre=1, groups=1),
         dict(z=1, post=0, res=1, pre=1, groups=1), dict(z=1, post=0, res=0, pre=0, groups=1, gate_last=True)]


def norm_case(rng, c, R=3, W=12):
    n = rng.standard_normal
    t = dict(y=n((R, W)), z=n((R, W)) if c["z"] else None, w_post=n(W) if c["post"] else None,
             res=n((R, W)) if c["res"] else None, w_pre=n(W) if c["pre"] else None)
    return t, dict(groups=c["groups"], gate_last=c.get("gate_last", False), eps=1e-3, res_scale=0.9, out_scale=0.6)


@pytest.mark.parametrize("c", NORMS)
def test_norm_gradients_are_the_differences(c):
    rng = np.random.default_rng(6)
    t, kw = norm_case(rng, c)
    g_h, g_n = rng.standard_normal(t["y"].shape), rng.standard_normal(t["y"].shape) if c["pre"] else None

    def loss(**over):
        f = M.block_norm_forward(*(dict(t, **over)[n] for n in ("y", "z", "w_post", "res", "w_pre")), **kw)
        return (f["h"] * g_h).sum() + ((f["n"] * g_n).sum() if g_n is not None else 0)

    got = M.block_norm_backward(t["y"], t["z"], t["w_post"], t["res"], t["w_pre"], g_h, g_n, **kw)
    assert set(got) == {"d" + n for n, v in t.items() if v is not None}
    for n, v in t.items():
        if v is None:
            continue
        grad, mag = got["d" + n]
        assert (np.abs(grad) <= mag * (1 + 1e-9)).all(), n
        for _ in range(3):
            d, e = rng.standard_normal(v.shape), 1e-6
            diff = (loss(**{n: v + e * d}) - loss(**{n: v - e * d})) / (2 * e)
            assert abs(diff - (grad * d).sum()) <= 1e-6 * (1 + abs(diff)), n


def test_norm_parts():
    rng = np.random.default_rng(7)
    y, res, w = rng.standard_normal((2, 8)), rng.standard_normal((2, 8)), rng.standard_normal(8)
    f = M.block_norm_forward(y, None, None, res, None, res_scale=0.5, out_scale=2.0)
    np.testing.assert_allclose(f["h"], 0.5 * res + 2 * y)
    assert f["n"] is None
    f = M.block_norm_forward(None, None, None, res, w, eps=1e-9)
    np.testing.assert_allclose(f["n"], res / np.sqrt((res ** 2).mean(1, keepdims=True)) * w, rtol=1e-8)
    f = M.block_norm_forward(y, None, np.ones(8), None, None, groups=2, eps=1e-12)
    np.testing.assert_allclose((f["h"].reshape(2, 2, 4) ** 2).mean(-1), np.ones((2, 2)), rtol=1e-9)
