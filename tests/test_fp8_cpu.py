"""The grouped router's and the 8-bit layer's oracle against its pins, and the refusals of their entry points (checked
on the host before any HIP call, so these run without a GPU)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import sparse_mixture_experts_48_amd as moe
from oracle import fp8_oracle as F
from sparse_mixture_experts_48_amd.binding import GemmFp8Desc, MoeDesc, RouterDesc

OK, NULL, SHAPE, UNSUP, WS = 0, 1, 2, 3, 4
FAKE = 0x10000  # a 256-byte aligned, never dereferenced address


# ---------------------------------------------------------------------------- the oracle

def test_e4m3_table_is_torchs():
    b = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(b, F.TABLE.astype(np.float32), equal_nan=True)


def test_nearest_is_torchs_rounding():
    r = np.random.default_rng(1)
    x = (r.standard_normal(20000) * 2.0 ** r.integers(-12, 8, 20000)).astype(np.float32).clip(-448, 448)
    mid = (F._POS[1:] + F._POS[:-1]).astype(np.float32) / 2  # every tie
    x = np.concatenate([x, mid, -mid, F._POS.astype(np.float32)])
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(F.nearest(x), want)


@pytest.mark.parametrize("top,e", [(448.0, 0), (448.5, 1), (896.0, 1), (1.0, -8), (1.75, -8), (1.7500001, -7), (0.0, -127),
                                   (2.0 ** -140, -127), (3.0e38, 120)])
def test_exponent(top, e):
    assert F.exponent(top) == e


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_grad_is_the_difference_quotient(score, renorm):
    r = np.random.default_rng(2)
    l, dg = r.standard_normal((3, 7)), r.standard_normal((3, 3))
    idx, _ = F.route(l, "float32", None, 3, score, renorm, 1.7, 1, 1, 1)
    got, _ = F.route_grad(l, "float32", idx, dg, score, renorm, 1.7)

    def loss(m):
        return sum(float(u) * g for t in range(3)
                   for u, g in zip(dg[t], F.gates(F.scores(m[t], score, -1e300)[0], idx[t], renorm, 1.7,
                                                m[t] if score == "softmax" else None)))
    for t in range(3):
        for e in range(7):
            m = l.copy()
            m[t, e] += 1e-5
            up = loss(m)
            m[t, e] -= 2e-5
            # second-order differences: error about 1e-10 relative to terms of order 1
            assert abs((up - loss(m)) / 2e-5 - got[t, e]) < 1e-8


def test_route_closed_forms():
    # one group and softmax: the K largest logits; gates of equal logits are equal
    l = np.array([[0.0, 3.0, 3.0, -1.0]])
    idx, gate = F.route(l, "float32", None, 2, "softmax", True, 1.0, 1, 1, 1)
    assert idx.tolist() == [[1, 2]] and np.allclose(gate, 0.5)
    # the bias steers the choice, not the gates
    idx, gate = F.route(l, "float32", [9, 0, 0, 0], 2, "sigmoid", False, 2.0, 1, 1, 1)
    assert idx.tolist() == [[0, 1]] and np.allclose(gate, [[1.0, 2 / (1 + math.exp(-3))]])
    # two groups: by the best expert the first wins, by the sum of two the second
    l = np.array([[5.0, -9.0, 3.0, 3.0]])
    one = F.route(l, "float32", None, 1, "sigmoid", False, 1.0, 2, 1, 1)[0]
    two = F.route(l, "float32", None, 1, "sigmoid", False, 1.0, 2, 1, 2)[0]
    assert one.tolist() == [[0]] and two.tolist() == [[2]]
    # a row that its mask leaves nothing of
    idx, gate = F.route(np.full((1, 4), -np.inf), "float32", None, 2, "softmax", True, 1.0, 1, 1, 1)
    assert idx.tolist() == [[F.NONE_ID] * 2] and gate.tolist() == [[0.0, 0.0]]


def test_group_is_stable():
    c, o, st, ts = F.group(np.array([[1, 0], [1, 9], [0, 1]]), 3)
    assert c.tolist() == [2, 3, 0] and o.tolist() == [0, 2, 5, 5]
    assert st.tolist() == [0, 2, 0, 1, 2, -1] and ts.tolist() == [[2, 0], [3, -1], [1, 4]]


# ---------------------------------------------------------------------------- refusals

def _r(T=64, E=64, K=2, groups=8, top_groups=4, group_top=2, score=1, renorm=1, scale=1.0):
    return RouterDesc(T, E, K, groups, top_groups, group_top, score, renorm, scale)


def _route(d, logits=FAKE, dtype=0, bias=None, idx=FAKE, gate=FAKE):
    return moe.lib().moe_route_grouped(ctypes.byref(d), logits, dtype, bias, idx, gate, None)


def _route_bwd(d, logits=FAKE, dtype=0, idx=FAKE, dgate=FAKE, dlogits=FAKE):
    return moe.lib().moe_route_grouped_backward(ctypes.byref(d), logits, dtype, idx, dgate, dlogits, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), SHAPE), (dict(E=0), SHAPE), (dict(K=0), SHAPE), (dict(groups=0), SHAPE), (dict(groups=7), SHAPE),
    (dict(top_groups=0), SHAPE), (dict(top_groups=9), SHAPE), (dict(K=8, E=16, top_groups=3), SHAPE),
    (dict(scale=float("nan")), SHAPE), (dict(scale=float("inf")), SHAPE), (dict(group_top=0), UNSUP),
    (dict(group_top=3), UNSUP), (dict(score=2), UNSUP), (dict(renorm=2), UNSUP), (dict(E=520), UNSUP),
    (dict(K=9), UNSUP), (dict(groups=64, top_groups=64), UNSUP), (dict(T=2 ** 31 // 2), UNSUP),
    (dict(T=2 ** 25, E=512, K=1), UNSUP),
])
def test_router_refusals(kw, status):
    assert _route(_r(**kw)) == status
    assert _route_bwd(_r(**kw)) == status


def test_router_argument_refusals():
    d = _r()
    assert moe.lib().moe_route_grouped(None, FAKE, 0, None, FAKE, FAKE, None) == NULL
    assert _route(d, logits=None) == NULL
    assert _route(d, idx=None) == NULL
    assert _route(d, gate=None) == NULL
    assert _route(d, dtype=2) == UNSUP
    assert _route(d, logits=FAKE + 4) == UNSUP
    assert _route(d, bias=FAKE + 4) == UNSUP
    assert moe.lib().moe_route_grouped_backward(None, FAKE, 0, FAKE, FAKE, FAKE, None) == NULL
    for k in ("logits", "idx", "dgate", "dlogits"):
        assert _route_bwd(d, **{k: None}) == NULL
        assert _route_bwd(d, **{k: FAKE + 8}) == UNSUP
    assert _route_bwd(d, dtype=-1) == UNSUP
    # no tokens: nothing to do, no tensor needed
    e = _r(T=0)
    assert _route(e, logits=None, idx=None, gate=None) == OK
    assert _route_bwd(e, logits=None, idx=None, dgate=None, dlogits=None) == OK


def test_group_refusals():
    L = moe.lib()
    n = ctypes.c_size_t(0)
    by = ctypes.byref
    for args, status in [((-1, 8, 2), SHAPE), ((4, 0, 2), SHAPE), ((4, 8, 0), SHAPE), ((4, 513, 2), UNSUP),
                         ((4, 512, 9), UNSUP), ((2 ** 30, 8, 2), UNSUP), ((0, 8, 2), OK), ((16384, 256, 8), OK)]:
        assert L.moe_group_workspace_size(*args, by(n)) == status, args
    assert L.moe_group_workspace_size(4, 8, 2, None) == NULL

    def group(idx=FAKE, counts=FAKE, offs=FAKE, st=FAKE, ts=FAKE, ws=FAKE, size=n.value):
        return L.moe_group(16384, 256, 8, idx, counts, offs, st, ts, ws, size, None)
    assert n.value > 0
    for k in ("idx", "counts", "offs", "st", "ts"):
        assert group(**{k: None}) == NULL
        assert group(**{k: FAKE + 4}) == UNSUP
    assert group(ws=None) == WS
    assert group(ws=FAKE + 16) == WS
    assert group(size=n.value - 1) == WS


def _quant(x=FAKE, dtype=1, mats=1, rows=4, cols=128, br=1, q=FAKE, s=FAKE):
    return moe.lib().moe_quantize_fp8(x, dtype, mats, rows, cols, br, q, s, None)


def test_quantize_refusals():
    for kw, status in [(dict(x=None), NULL), (dict(q=None), NULL), (dict(s=None), NULL), (dict(x=FAKE + 8), UNSUP),
                       (dict(dtype=2), UNSUP), (dict(mats=-1), SHAPE), (dict(rows=-1), SHAPE), (dict(cols=0), SHAPE),
                       (dict(cols=24), UNSUP), (dict(br=2), UNSUP), (dict(br=0), UNSUP), (dict(cols=2 ** 20 + 16), UNSUP),
                       (dict(rows=2 ** 31 - 1, cols=2 ** 20), UNSUP), (dict(rows=2 ** 32), UNSUP),
                       (dict(rows=0, x=None, q=None, s=None), OK), (dict(mats=0, x=None, q=None, s=None), OK)]:
        assert _quant(**kw) == status, kw


def test_one_launch_covers_the_call():
    """A launch holds fewer than 2^32 threads; what would need more is refused."""
    for kw in (dict(rows=2 ** 28), dict(rows=2 ** 21, cols=2 ** 14), dict(mats=2 ** 14, rows=2 ** 14),
               dict(mats=2 ** 24, rows=1, br=128), dict(mats=2 ** 14, rows=2 ** 14, cols=2 ** 10, br=128)):
        assert _quant(**kw) == UNSUP, kw
    assert _route(_r(T=2 ** 28, E=4, K=1, groups=1, top_groups=1)) == UNSUP
    assert _route_bwd(_r(T=2 ** 28, E=4, K=1, groups=1, top_groups=1)) == UNSUP


def _gemm(S=64, x_rows=64, E=8, N=256, Kd=128, max_rows=0, out_dtype=1, bias_dtype=1, x=FAKE, xs=FAKE, rows=None,
          offs=FAKE, W=FAKE, ws=FAKE, bias=None, out=FAKE):
    d = GemmFp8Desc(S, x_rows, E, N, Kd, max_rows, out_dtype, bias_dtype)
    return moe.lib().moe_grouped_gemm_fp8(ctypes.byref(d), x, xs, rows, offs, W, ws, bias, out, None)


def test_gemm_refusals():
    assert moe.lib().moe_grouped_gemm_fp8(None, FAKE, FAKE, None, FAKE, FAKE, FAKE, None, FAKE, None) == NULL
    for kw, status in [
            (dict(S=-1), SHAPE), (dict(x_rows=-1), SHAPE), (dict(E=0), SHAPE), (dict(N=0), SHAPE), (dict(Kd=0), SHAPE),
            (dict(max_rows=-1), SHAPE), (dict(E=513), UNSUP), (dict(N=24), UNSUP), (dict(Kd=40), UNSUP),
            (dict(N=2 ** 20 + 16), UNSUP), (dict(out_dtype=2), UNSUP), (dict(bias_dtype=7), UNSUP),
            (dict(x_rows=65), SHAPE), (dict(x_rows=0, rows=FAKE), SHAPE), (dict(offs=None), NULL), (dict(x=None), NULL),
            (dict(xs=None), NULL), (dict(W=None), NULL), (dict(ws=None), NULL), (dict(out=None), NULL),
            (dict(x=FAKE + 8), UNSUP), (dict(xs=FAKE + 1), UNSUP), (dict(W=FAKE + 8), UNSUP), (dict(ws=FAKE + 8), UNSUP),
            (dict(bias=FAKE + 2), UNSUP), (dict(rows=FAKE + 4), UNSUP), (dict(offs=FAKE + 4), UNSUP),
            (dict(S=2 ** 20, x_rows=2 ** 20, N=4096), UNSUP), (dict(S=2 ** 20, x_rows=2 ** 20, N=16, Kd=4096), UNSUP),
            (dict(N=2 ** 16, Kd=2 ** 15), UNSUP), (dict(S=0, x_rows=0, x=None, xs=None, out=None), OK)]:
        assert _gemm(**kw) == status, kw


def _d(T=64, d=256, E=8, K=2, w=512, act=1, gate=0, dtype=1, capacity=0, bias_mode=0):
    return MoeDesc(T, d, E, K, w, act, gate, dtype, capacity, bias_mode)


def _size(d):
    n = ctypes.c_size_t(0)
    assert moe.lib().moe_fp8_workspace_size(ctypes.byref(d), ctypes.byref(n)) == OK
    return n.value


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), SHAPE), (dict(d=0), SHAPE), (dict(w=0), SHAPE), (dict(E=0), SHAPE), (dict(K=0), SHAPE),
    (dict(K=9), SHAPE), (dict(K=9, E=64), UNSUP), (dict(E=513), UNSUP), (dict(E=512), OK), (dict(d=248), UNSUP),
    (dict(w=1368), UNSUP), (dict(act=2), UNSUP), (dict(dtype=7), UNSUP), (dict(capacity=4), UNSUP),
    (dict(capacity=-1), SHAPE), (dict(bias_mode=1), UNSUP), (dict(T=2 ** 30), UNSUP),
])
def test_layer_descriptor_refusals(kw, status):
    n = ctypes.c_size_t(0)
    assert moe.lib().moe_fp8_workspace_size(ctypes.byref(_d(**kw)), ctypes.byref(n)) == status


def _forward(d, r, h=FAKE, logits=FAKE, dtype=0, bias=None, W1=FAKE, s1=FAKE, b1=None, W3=FAKE, s3=FAKE, W2=FAKE, s2=FAKE,
             b2=None, y=FAKE, idx=None, gate=None, counts=None, ws=FAKE, size=None):
    size = _size(d) if size is None else size
    return moe.lib().moe_forward_fp8(ctypes.byref(d), None if r is None else ctypes.byref(r), h, logits, dtype, bias, W1,
                                     s1, b1, W3, s3, W2, s2, b2, y, idx, gate, counts, ws, size, None)


def _ffn(d, x=FAKE, xs=FAKE, rows=None, offs=FAKE, W1=FAKE, s1=FAKE, b1=None, W3=FAKE, s3=FAKE, W2=FAKE, s2=FAKE,
         b2=None, o=FAKE, ws=FAKE, size=None):
    size = _size(d) if size is None else size
    return moe.lib().moe_expert_ffn_fp8(ctypes.byref(d), x, xs, rows, offs, W1, s1, b1, W3, s3, W2, s2, b2, o, ws, size,
                                        None)


def test_layer_refusals():
    d, r = _d(), _r(E=8, groups=1, top_groups=1)
    assert moe.lib().moe_fp8_workspace_size(None, ctypes.byref(ctypes.c_size_t(0))) == NULL
    assert moe.lib().moe_fp8_workspace_size(ctypes.byref(d), None) == NULL
    assert _forward(d, None) == NULL
    for k in ("h", "logits", "W1", "s1", "W3", "s3", "W2", "s2", "y"):
        assert _forward(d, r, **{k: None}) == NULL, k
        assert _forward(d, r, **{k: FAKE + 8}) == UNSUP, k
    for k in ("bias", "idx", "gate", "counts"):
        assert _forward(d, r, **{k: FAKE + 4}) == UNSUP, k
    assert _forward(d, r, b1=FAKE) == UNSUP  # SwiGLU experts have no biases
    assert _forward(d, r, dtype=3) == UNSUP
    assert _forward(d, _r(T=63, E=8, groups=1, top_groups=1)) == SHAPE
    assert _forward(d, _r()) == SHAPE
    assert _forward(d, _r(E=8, groups=3)) == SHAPE
    assert _forward(d, r, ws=None) == WS
    assert _forward(d, r, ws=FAKE + 16) == WS
    assert _forward(d, r, size=_size(d) - 1) == WS
    for k in ("x", "xs", "offs", "W1", "s1", "W3", "s3", "W2", "s2", "o"):
        assert _ffn(d, **{k: None}) == NULL, k
        assert _ffn(d, **{k: FAKE + 8}) == UNSUP, k
    assert _ffn(d, rows=FAKE + 8) == UNSUP
    assert _ffn(d, size=0) == WS
    assert _ffn(_d(T=0), x=None, xs=None, offs=None, o=None) == OK


def test_combine_takes_the_grouped_routers_experts():
    assert moe.lib().moe_combine(ctypes.byref(_d(E=512)), FAKE, FAKE, None, FAKE, None) == NULL
    assert moe.lib().moe_combine(ctypes.byref(_d(E=513)), FAKE, FAKE, None, FAKE, None) == UNSUP


def test_binding_refuses():
    with pytest.raises(ValueError):
        moe.router_desc(4, 8, 2, score="tanh")
    x = torch.zeros(4, 128)
    for call in (lambda: moe.fp8._arg("x", x, (4, 128), torch.float32, 0),
                 lambda: moe.fp8._dtype("x", x.half()), lambda: moe.fp8._space(torch.zeros(4), 0)):
        with pytest.raises(ValueError):
            call()
