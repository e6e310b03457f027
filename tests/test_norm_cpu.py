"""moe_block_norm without a GPU: refusals of the C call and of the binding, and the reference against
hand-made rows.  Pointers are fake and never dereferenced."""
import ctypes

import numpy as np
import pytest

import norm_ref
import quantized_sparse_moe_amd as q

A = 0x7F0000000000
STEP = 1 << 32                     # tensors far apart


def N(**kw):
    n = q.moe_norm(q.MOE_NORM_RMS, q.MOE_F32, 1e-6, 0.0, A + 10 * STEP, None)
    for k, v in kw.items():
        setattr(n, k, v)
    return n


def call(T=4, H=64, **kw):
    a = dict(y=A, dy=q.MOE_BF16, ldy=H, r=A + STEP, dr=q.MOE_BF16, ldr=H, post=None, gate=None, dg=0, ldg=H, gc=H, act=0,
             scale=1.0, pre=N(), ro=A + 2 * STEP, dro=q.MOE_BF16, ldro=H, x=A + 3 * STEP, dx=q.MOE_BF16, ldx=H)
    a.update(kw)
    p = lambda n: None if n is None else ctypes.byref(n)
    return q.lib().moe_block_norm(a["y"], a["dy"], a["ldy"], a["r"], a["dr"], a["ldr"], p(a["post"]), a["gate"], a["dg"],
                                  a["ldg"], a["gc"], a["act"], a["scale"], p(a["pre"]), a["ro"], a["dro"], a["ldro"], a["x"],
                                  a["dx"], a["ldx"], T, H, None)


INVALID = [
    dict(T=-1), dict(H=-1), dict(dy=3), dict(dr=-1), dict(dro=3), dict(dx=7), dict(act=3), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(ldy=63), dict(ldr=63), dict(ldro=63), dict(ldx=63), dict(y=A + 1), dict(r=A + STEP + 1),
    dict(ro=A + 2 * STEP + 2, dro=q.MOE_F32), dict(x=A + 3 * STEP + 1), dict(y=None), dict(y=None, r=None, ro=None),
    dict(y=None, ro=None, post=N()), dict(y=None, ro=None, gate=A + 4 * STEP), dict(pre=None), dict(x=None),
    dict(pre=None, x=None, ro=None), dict(gate=A + 4 * STEP, gc=2, ldg=64), dict(gate=A + 4 * STEP, gc=0),
    dict(gate=A + 4 * STEP, ldg=63), dict(gate=A + 4 * STEP, dg=3), dict(pre=N(kind=2)), dict(pre=N(dtype=3)),
    dict(post=N(kind=-1)), dict(pre=N(eps=-1.0)), dict(pre=N(eps=float("nan"))), dict(pre=N(offset=float("inf"))),
    dict(pre=N(weight=A + 2)), dict(pre=N(bias=A + 10 * STEP + 1)),
    # memory shared otherwise than value for value
    dict(ro=A + 2), dict(ro=A, ldro=72), dict(ro=A, dro=q.MOE_F16), dict(x=A + STEP + 128), dict(x=A + 2 * STEP),
    dict(ro=A + 64, ldro=128, ldy=128), dict(x=A + 10 * STEP), dict(ro=A + 10 * STEP + 252),
    dict(gate=A + 4 * STEP, gc=1, ldg=1, x=A + 4 * STEP),
]


@pytest.mark.parametrize("i", range(len(INVALID)))
def test_invalid(i):
    assert call(**INVALID[i]) == q.MOE_ERR_INVALID, INVALID[i]


def test_limits_and_nothing_to_do():
    assert call(H=0) == q.MOE_ERR_UNSUPPORTED
    assert call(H=16385) == q.MOE_ERR_UNSUPPORTED
    assert call(T=(1 << 26) + 1) == q.MOE_ERR_UNSUPPORTED
    assert call(T=0, y=None, r=None, x=None) == q.MOE_OK


def test_binding_checks_its_arguments():
    import torch
    y, w = torch.zeros(3, 8), torch.ones(8)
    bad = [dict(), dict(y=y, residual=torch.zeros(3, 9)), dict(y=y, gate=torch.zeros(3, 2)), dict(y=y, gate=torch.zeros(2)),
           dict(y=y, gate_act="relu"), dict(residual=y, r_out=y), dict(y=y, x_out=y), dict(y=y, r_out=torch.zeros(2, 8)),
           dict(y=y, pre=q.Norm(weight=torch.ones(9))), dict(y=y, post=q.Norm(weight=torch.ones(7))),
           dict(y=y, pre=q.Norm(), x_out=torch.zeros(3, 7)), dict(y=y.double()), dict(y=torch.zeros(8)),
           dict(y=torch.zeros(3, 16)[:, ::2]), dict(y=y, pre=q.Norm(weight=w))]       # (the last: on the host)
    for kw in bad:
        with pytest.raises(q.QsmoeError):
            q.moe_block_norm(**kw)
    for kw in (dict(kind="batch"), dict(weight=w, bias=torch.zeros(9)), dict(weight=w, bias=torch.zeros(8).half()),
               dict(weight=torch.ones(2, 4)), dict(weight=torch.ones(16)[::2]), dict(weight=w.double())):
        with pytest.raises(q.QsmoeError):
            q.Norm(**kw)


def test_reference_by_hand():
    v = np.array([[3.0, -4.0], [0.0, 0.0]])
    o, b = norm_ref.norm(v, 0 * v, "rms", 0.5, 1.0, np.array([1.0, 2.0]), np.array([0.0, 1.0]))
    assert np.allclose(o, [[6 / np.sqrt(13), 1 - 12 / np.sqrt(13)], [0, 1]]) and (b < 1e-5).all()
    o, _ = norm_ref.norm(v[:1], 0 * v[:1], "layer", 0.0, 0.0, None, None)
    assert np.allclose(o, [[1, -1]])
    g = np.array([[0.0], [2.0]])
    (t, _), (x, _) = norm_ref.block(v, np.ones_like(v), None, g, "sigmoid", 2.0, None)
    assert np.allclose(t, [[4.0, -3.0], [1.0, 1.0]]) and x is None
    (t, _), _ = norm_ref.block(v, None, None, g, "silu", 1.0, None)
    assert np.allclose(t, 0.0)
