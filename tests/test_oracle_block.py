"""Pins of the oracle for scored routing, the norms around a block and 8-bit
products, and the library's refusals of bad arguments (no GPU)."""
import ctypes

import numpy as np
import pytest

import expert_offload_b200 as eo
from oracle import norm, q8, route, scored


# ------------------------------------------------------------------ routing

def test_plain_softmax_rule_is_moe_route():
    l = np.random.default_rng(0).standard_normal((40, 32)).astype(np.float32)
    i0, w0 = route.route(l, 5)
    i1, w1 = scored.route(l, 5)
    np.testing.assert_array_equal(i0, i1)
    np.testing.assert_allclose(w0, w1, rtol=1e-12)


def test_hand_worked_groups_and_bias():
    # four groups of two; sigmoid(0) = 1/2, sigmoid(ln 3) = 3/4, sigmoid(-ln 3) = 1/4
    h = float(np.log(3.0))
    l = np.array([0, 0, h, -h, -h, -h, h, h], dtype=np.float64)
    # sums of two: 1, 1, 1/2, 3/2: groups 3 and (a tie, the lower) 0
    idx, w = scored.route_row(l, 3, sigmoid=True, n_groups=4, topk_groups=2, group_top=2)
    assert idx.tolist() == [6, 7, 0]
    np.testing.assert_allclose(w, np.array([0.75, 0.75, 0.5]) / 2.0, rtol=1e-12)
    # best member: 1/2, 3/4, 1/4, 3/4: groups 1 and 3
    idx, _ = scored.route_row(l, 3, sigmoid=True, n_groups=4, topk_groups=2, group_top=1)
    assert idx.tolist() == [2, 6, 7]
    # a bias moves the selection, not the weights
    b = np.zeros(8)
    b[4] = 1.0
    idx, w = scored.route_row(l, 2, sigmoid=True, bias=b, renormalise=False, scale=2.0)
    assert idx.tolist() == [4, 2]
    np.testing.assert_allclose(w, [0.5, 1.5], rtol=1e-12)


def test_masked_experts_come_last_and_weigh_nothing():
    ninf, nan = -np.inf, np.nan
    idx, w = scored.route_row([ninf, 1.0, nan, 2.0], 3)
    assert idx.tolist() == [3, 1, 0] and w[2] == 0
    idx, w = scored.route_row([ninf] * 4, 2)
    assert idx.tolist() == [0, 1] and (w == 0).all()
    idx, w = scored.route_row([3.0, 1.0, 0.0, 2.0], 2, bias=[ninf, 0, 0, 0])
    assert idx.tolist() == [3, 1]
    # a group with one live member counts that one alone
    idx, _ = scored.route_row([5.0, ninf, 1.0, 1.0], 1, sigmoid=True, n_groups=2, topk_groups=1, group_top=2)
    assert idx.tolist() == [2]


# --------------------------------------------------------------------- norm

def test_norm_of_a_hand_worked_row():
    np.testing.assert_allclose(norm.rms_norm([[3.0, 4.0]], eps=0.0), [[3 / 12.5 ** 0.5, 4 / 12.5 ** 0.5]])
    np.testing.assert_allclose(norm.rms_norm([[3.0, 4.0]], [1.0, 2.0], eps=0.0, offset=1.0),
                               [[6 / 12.5 ** 0.5, 12 / 12.5 ** 0.5]])
    x = norm.join([[1.0, 2.0]], [[3.0, 4.0]], alpha=0.5, beta=2.0, gate=np.array([[0.5], ]))
    np.testing.assert_allclose(x, [[3.5, 5.0]])
    x = norm.join([[0.0, 0.0]], [[1.0, 1.0]], y2=[[2.0, 4.0]], y2_gate=[0.0])
    np.testing.assert_allclose(x, [[2.0, 3.0]])


# -------------------------------------------------------------------- 8 bits

def test_quantiser_fp64_is_the_exact_quotient():
    rng = np.random.default_rng(1)
    v = rng.standard_normal((6, 50)).astype(np.float32)
    v[1] = np.float32(0.5) * np.arange(50, dtype=np.float32)     # many halves: 127 / 49 * c / 2
    v[2] = (np.arange(50) - 24.5).astype(np.float32) * 2.0 ** -140
    v[3, :2] = [127.0, 63.5]
    v[3, 2:] = 0.5 * np.arange(48)                               # amax 127: ties at every odd c
    a, sa = q8.quantise(v)
    b, sb = q8.quantise(v, exact=True)
    np.testing.assert_array_equal(a, b)
    np.testing.assert_array_equal(sa, sb)
    assert a[3, 1] == 64 and a[3, 3] == 0 and a[3, 5] == 2       # half to even
    assert np.abs(a.astype(int)).max() == 127


# ----------------------------------------------------------------- refusals

@pytest.fixture(scope="module")
def lib():
    from expert_offload_b200 import build
    build.build()
    return eo.lib()


A = 4096                     # an aligned address that no refused call may touch


def _route(lib, dtype=0, ld=0, T=4, E=64, k=8, n=8, tg=4, gt=2, score=1, scale=1.0, logits=A, bias=A, rule=True,
           lists=(None, None, None), ws=None, wsb=0, idx=A, wts=A):
    r = eo.RouteRule(score, n, tg, gt, True, scale)
    return lib.moe_route_scored(logits, dtype, ld, T, E, bias, ctypes.byref(r.struct) if rule else None, k, idx, wts,
                                *lists, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), -1), (dict(rule=False), -1), (dict(idx=None), -1), (dict(dtype=2), -1), (dict(ld=63), -1),
    (dict(T=0), -3), (dict(T=65537), -3), (dict(E=513, n=1, tg=1), -3), (dict(k=17), -3), (dict(k=0), -3),
    (dict(n=7), -3), (dict(n=64), -3), (dict(n=0), -3), (dict(tg=0), -1), (dict(tg=9), -1), (dict(gt=3), -1),
    (dict(gt=0), -1), (dict(E=32, n=32, tg=32, gt=2), -1), (dict(k=9, tg=1), -1), (dict(score=2), -1),
    (dict(scale=float("inf")), -1), (dict(scale=float("nan")), -1), (dict(logits=A + 2), -2), (dict(bias=A + 1), -2),
    (dict(dtype=1, logits=A + 1), -2), (dict(lists=(A, A, None)), -1), (dict(lists=(A, A, A), T=40), -8),
    (dict(lists=(A, A, A), T=40, ws=A, wsb=16), -8), (dict(lists=(A, A, A), T=40, ws=A + 4, wsb=1 << 20), -2),
    (dict(wts=A + 2), -2)])
def test_route_refusals(lib, kw, status):
    assert _route(lib, **kw) == status
    assert eo.last_error()


def _norm(lib, rule=None, T=4, H=64, x=A, xd=1, ldx=0, y=A, y2=None, yd=0, ldy=0, g2=None, gate=None, x_out=A, xn=A,
          xnd=1, xq=None, xs=None):
    r = eo.NormRule(**(rule or {}))
    return lib.moe_norm_residual(ctypes.byref(r.struct), T, H, x, xd, ldx, y, y2, yd, ldy, g2, gate, x_out, xn, xnd,
                                 xq, xs, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), -1), (dict(x_out=None, xn=None), -1), (dict(xd=2), -1), (dict(yd=-1), -1), (dict(xnd=7), -1),
    (dict(rule=dict(w_dtype=3)), -1), (dict(T=0), -3), (dict(T=65537), -3), (dict(H=0), -3), (dict(H=8193), -3),
    (dict(ldx=63), -1), (dict(ldy=1), -1), (dict(rule=dict(eps=-1.0)), -1), (dict(rule=dict(eps=float("nan"))), -1),
    (dict(rule=dict(residual_scale=float("inf"))), -1), (dict(rule=dict(gate_kind=4)), -1),
    (dict(rule=dict(gate_kind=1)), -1), (dict(gate=A), -1), (dict(rule=dict(gate_kind=1, gate_act=2), gate=A), -1),
    (dict(y=None, y2=A), -1), (dict(y=None, gate=A, rule=dict(gate_kind=1)), -1), (dict(g2=A), -1),
    (dict(xq=A), -1), (dict(xs=A), -1), (dict(x=A + 1), -2), (dict(y=A + 2), -2), (dict(xq=A + 8, xs=A), -2),
    (dict(rule=dict(w_pre=A + 1)), -2)])
def test_norm_refusals(lib, kw, status):
    assert _norm(lib, **kw) == status
    assert eo.last_error()


def _linear(lib, x=A, xd=1, ldx=0, T=4, K=64, wq=A, ldw=0, ws=A, N=32, y=A, yd=1, ldy=0, work=256, wb=1 << 30):
    return lib.q8_linear(x, xd, ldx, T, K, wq, ldw, ws, N, y, yd, ldy, work, wb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), -1), (dict(wq=None), -1), (dict(ws=None), -1), (dict(y=None), -1), (dict(xd=5), -1),
    (dict(yd=5), -1), (dict(T=0), -3), (dict(T=65537), -3), (dict(K=0), -3), (dict(K=16385), -3), (dict(N=0), -3),
    (dict(N=65537), -3), (dict(ldx=63), -1), (dict(ldw=63), -1), (dict(ldw=72), -1), (dict(ldy=31), -1),
    (dict(wq=A + 8), -2), (dict(x=A + 1), -2), (dict(y=A + 1), -2), (dict(ws=A + 2), -2)])
def test_q8_linear_refusals(lib, kw, status):
    assert _linear(lib, **kw) == status
    assert eo.last_error()


def test_q8_workspace_refusals(lib):
    T, K, N = 4096, 512, 1024
    need = lib.q8_linear_workspace_bytes(T, K, N)
    assert need >= T * K + 4 * T
    assert _linear(lib, T=T, K=K, N=N, work=None, wb=0) == -8
    assert _linear(lib, T=T, K=K, N=N, wb=need - 1) == -8
    assert _linear(lib, T=T, K=K, N=N, work=256 + 16) == -2
    assert lib.q8_linear_workspace_bytes(0, K, N) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), -1), (dict(q=None), -1), (dict(scale=None), -1), (dict(act=2), -1), (dict(xd=3), -1),
    (dict(rows=0), -3), (dict(rows=65537), -3), (dict(cols=16385), -3), (dict(cols=2 ** 31 - 1, act=1), -3),
    (dict(ldx=99), -1), (dict(act=1, ldx=199), -1), (dict(ldq=96), -1), (dict(ldq=104), -1), (dict(q=A + 4), -2),
    (dict(scale=A + 1), -2), (dict(x=A + 1), -2)])
def test_quantise_refusals(lib, kw, status):
    d = dict(x=A, xd=0, ldx=0, rows=4, cols=100, act=0, q=A, ldq=0, scale=A)
    d.update(kw)
    assert lib.q8_quantize_rows(d["x"], d["xd"], d["ldx"], d["rows"], d["cols"], d["act"], d["q"], d["ldq"],
                                d["scale"], None) == status
    assert eo.last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(xq=None), -1), (dict(xs=None), -1), (dict(ldxq=48), -1), (dict(ldxq=72), -1), (dict(xq=A + 1), -2),
    (dict(xs=A + 1), -2), (dict(N=0), -3), (dict(ldw=65), -1)])
def test_matmul_refusals(lib, kw, status):
    d = dict(xq=A, ldxq=0, xs=A, T=2, K=64, wq=A, ldw=0, ws=A, N=8, y=A, yd=0, ldy=0)
    d.update(kw)
    assert lib.q8_matmul(*d.values(), None) == status
    assert eo.last_error()


def test_route_workspace_bytes(lib):
    f = lib.moe_route_scored_workspace_bytes
    assert f(16, 256, 8) == 0 and f(0, 256, 8) == 0       # up to 16 tokens: one block, no workspace
    assert f(17, 256, 8) >= 3 * 256
    for T in (1184, 1185, 2368, 2369, 8192, 8193, 65536):
        assert f(T, 512, 8) % 4 == 0 and f(T, 512, 8) >= 512 * (T // 32)


def test_binding_checks_sizes_and_raw_addresses(lib):
    with pytest.raises(eo.HfqError) as e:
        eo.q8_quantize_rows(A, eo.HFQ_F32, 2 ** 32 + 4, 64, A, A)
    assert e.value.status == -1 and "range" in e.value.message
    with pytest.raises(eo.HfqError) as e:
        eo.q8_quantize_rows(A, eo.HFQ_F32, 4, 64, A + 4, A)
    assert e.value.status == -2 and "q must be 16-byte aligned" in e.value.message
    with pytest.raises(TypeError):
        eo.q8_quantize_rows(A, eo.HFQ_F32, 4.5, 64, A, A)
    with pytest.raises(eo.HfqError) as e:
        eo.moe_norm_residual(eo.NormRule(), 4, 64, A, 9, xn=A)
    assert e.value.status == -1


def test_binding_refuses_tensors_it_cannot_use():
    torch = pytest.importorskip("torch")
    t = torch.zeros(4, 64)
    for bad in (t, np.zeros((4, 64), np.float32)):
        with pytest.raises(eo.HfqError) as e:
            eo.q8_quantize_rows(bad, eo.HFQ_F32, 4, 64, 4096, 4096)
        assert e.value.status == -1 and "x " in e.value.message
