"""What the binding of routing, norms and 8-bit products makes of its operands'
shapes and strides, without a GPU: CPU tensors that say they lie on the
current device go through the native marshalling, which either refuses them by
name or hands them on.  So that nothing is ever launched, each call that ought
to pass names one misaligned address, which the library finds before a launch.
"""
import warnings

import numpy as np
import pytest

import expert_offload_b200 as eo

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="CPU tensors pose as the current device's")
A = 1 << 20                                              # an aligned address that is never read
ARG, ALIGN = -1, -2


class OnDevice(torch.Tensor):
    def get_device(self):
        return 0


def _t(*shape, dt=torch.float32):
    return torch.zeros(*shape, dtype=dt).as_subclass(OnDevice)


@pytest.fixture(autouse=True)
def _binding(monkeypatch):
    from expert_offload_b200 import build
    build.build()
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(eo, "_stream", lambda s: None)
    eo._call = None                                      # bound afresh here, and again by whoever comes next
    yield
    eo._call = None


def _status(call):
    with pytest.raises(eo.HfqError) as e:
        call()
    return e.value.status, e.value.message


def _refused(call, name):
    st, why = _status(call)
    assert st == ARG and why.startswith(name + " "), (st, why)


def _passes(call):
    assert _status(call)[0] == ALIGN


def _quantise(x=A, rows=4, cols=64, q=A, ldx=0, ldq=0, scale=A + 2, act=0):
    return lambda: eo.q8_quantize_rows(x, eo.HFQ_F32, rows, cols, q, scale, ldx=ldx, ldq=ldq, act=act)


def _matmul(xq=A, xs=A, T=4, K=60, wq=A, ws=A, N=8, y=A + 2, ldxq=0, ldw=0, ldy=0):
    return lambda: eo.q8_matmul(xq, xs, T, K, wq, ws, N, y, eo.HFQ_F32, ldxq=ldxq, ldw=ldw, ldy=ldy)


def _norm(T=4, H=64, x=A, rule=None, **kw):
    kw.setdefault("xn", A + 1)
    return lambda: eo.moe_norm_residual(rule or eo.NormRule(), T, H, x, eo.HFQ_F32, **kw)


def _route(logits=A, T=4, E=64, k=8, idx=A, wts=A + 2, **kw):
    return lambda: eo.moe_route_scored(logits, eo.HFQ_F32, T, E, k, eo.RouteRule(), idx, wts, **kw)


def test_gates_and_scales_are_dense():
    column = _t(4, 512)[:, 3:4]                          # T values, 512 apart
    _refused(_norm(y=A, y2=A, y2_gate=column), "y2_gate")
    _refused(_norm(y=A, gate=column, rule=eo.NormRule(gate_kind=eo.GATE_TOKEN)), "gate")
    _refused(_norm(y=A, gate=_t(4, 128)[:, :64], rule=eo.NormRule(gate_kind=eo.GATE_FULL)), "gate")
    _refused(_norm(xq=A, xq_scale=_t(4, 2)[:, :1]), "xq_scale")
    _refused(_quantise(scale=_t(4, 2)[:, 0]), "scale")
    _refused(_matmul(xs=_t(8)[::2]), "xs")
    _refused(_matmul(ws=_t(8, 3)[:, 1:2]), "ws")
    _refused(_route(bias=_t(64, 2)[:, :1]), "bias")
    _passes(_norm(y=A, y2=A, y2_gate=column.contiguous()))
    _passes(_norm(T=1, y=A, y2=A, y2_gate=column[:1]))   # one token: one value
    _passes(_matmul(xs=_t(4, 1), ws=_t(1, 8)))


def test_outputs_without_a_row_step_are_dense():
    i32 = torch.int32
    _refused(_route(idx=_t(4, 16, dt=i32)[:, :8]), "idx")
    _refused(_route(wts=_t(4, 16)[:, :8]), "wts")
    _refused(_norm(xn=_t(4, 128, dt=torch.bfloat16)[:, :64]), "xn")
    _refused(_norm(xq=_t(4, 128, dt=torch.int8)[:, :64], xq_scale=A), "xq")
    for name, n in (("cnt", 64), ("off", 65), ("perm", 32)):
        lists = dict(cnt=A, off=A, perm=A)
        _refused(_route(**dict(lists, **{name: _t(n, 2, dt=i32)[:, 0]})), name)
    _refused(_route(cnt=A, off=A, perm=A, workspace=_t(64, 64, dt=torch.uint8)[:, :32]), "workspace")
    _passes(_route(idx=_t(4, 8, dt=i32)))
    _passes(_route(idx=_t(40, dt=i32)))


def test_rows_lie_as_far_apart_as_the_call_says():
    wide = _t(4, 200)
    _refused(_quantise(x=wide[:, :64]), "x")             # 200 apart, taken for 64
    _refused(_quantise(x=wide), "x")                     # dense, but not in rows of 64
    _refused(_quantise(x=wide[:, :64], ldx=100), "x")
    _refused(_quantise(x=wide[:, :60], ldx=200), "x")    # 60 of 64 columns
    _refused(_quantise(x=wide[:3, :64], ldx=200), "x")   # 3 of 4 rows
    _refused(_quantise(x=_t(64).expand(4, 64)), "x")
    _refused(_quantise(x=_t(64, 4).t()), "x")
    _refused(_norm(x=wide[:, :64]), "x")
    _refused(_norm(y=wide[:, 8:72]), "y")
    _refused(_norm(y=A, y2=wide[:, 8:72], ldy=72), "y2")
    _refused(_norm(x_out=wide[:, :64]), "x_out")
    _refused(_route(logits=wide[:, :64]), "logits")
    _refused(_matmul(y=_t(4, 16)[:, :8]), "y")
    b = _t(8, 128, dt=torch.int8)
    _refused(_matmul(wq=b[:, :64]), "wq")
    _refused(_matmul(xq=b[:4, :64], ldxq=64), "xq")
    _refused(_quantise(q=b[:4, :60], ldq=128, cols=60), "q")      # its tail is written, too
    _passes(_quantise(x=wide[:, :64], ldx=200))
    _passes(_quantise(x=wide[:, 136:], ldx=200))
    _passes(_quantise(x=wide, ldx=200))
    _passes(_quantise(x=wide[:1, :64], rows=1))
    _passes(_quantise(x=_t(40, 64)))                     # buffers for more rows than the call has
    _passes(_quantise(x=_t(40, 64), rows=1))
    _passes(_quantise(x=_t(40, 4, 16)))
    _passes(_quantise(x=_t(6, 5, 64)))
    _refused(_quantise(x=_t(64, 40)), "x")               # as many elements in other rows
    _refused(_quantise(x=_t(8, 128)), "x")
    _passes(_quantise(x=_t(4, 4, 16)))                   # heads side by side: one row
    _passes(_quantise(x=_t(2, 2, 64)))                   # two dimensions of rows
    _passes(_quantise(x=_t(2, 2, 100)[:, :, :64], ldx=100))
    _refused(_quantise(x=_t(2, 3, 100)[:, :2, :64], ldx=100), "x")
    _passes(_quantise(x=_t(3 * 100 + 64), ldx=100))      # flat: up to the last row's end
    _passes(_quantise(x=_t(4, 1, 64)[:, :, :], rows=4))
    _passes(_matmul(wq=b[:, :60], ldw=128))              # bytes behind K are read and do not count
    _passes(_matmul(xq=_t(4, 64, dt=torch.int8), wq=_t(8, 64, dt=torch.int8)))
    _passes(_quantise(x=_t(4, 128), act=eo.ACT_SWIGLU))
    _refused(_quantise(x=_t(4, 200)[:, :128], act=eo.ACT_SWIGLU), "x")


def test_a_view_is_no_larger_than_itself():
    pool = _t(4096)
    _refused(_quantise(x=pool[:255]), "x")
    _refused(_norm(y=pool[:255]), "y")
    _refused(_route(wts=pool[:31]), "wts")
    _refused(_norm(y=A, y2=A, y2_gate=pool[:3]), "y2_gate")
    _passes(_quantise(x=pool[:256]))
    q = _t(600, dt=torch.int8)
    _passes(_matmul(wq=q[:7 * 64 + 60]))                 # all of the last row; its unread tail lies in the storage
    _refused(_matmul(wq=q[-(7 * 64 + 60):]), "wq")       # ... and here behind it
    _refused(_matmul(wq=q[:7 * 64 + 59]), "wq")


def test_a_rules_weights_are_dense():
    class W(OnDevice):
        is_cuda = True

    def weights(t):
        return eo.NormRule(w_pre=t.as_subclass(W), w_dtype=eo.HFQ_F32)

    _refused(_norm(rule=weights(_t(64, 2)[:, :1])), "w_pre")
    _refused(_norm(rule=weights(_t(4096)[:63])), "w_pre")
    _passes(_norm(rule=weights(_t(64))))


def test_sizes_of_numpy_do_not_wrap_around():
    n = np.int32(65536)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        _refused(_quantise(x=_t(256), rows=n, ldx=n), "x")
        _refused(_matmul(y=_t(256), T=n, N=n), "y")
        _refused(_norm(x=_t(256), T=n, ldx=n), "x")
        _refused(_norm(T=n, H=n, xn=_t(256, dt=torch.bfloat16)), "xn")
        _passes(_quantise(x=_t(4, 64), rows=np.int64(4), cols=np.int32(64)))


def test_an_address_is_no_workspace():
    """A workspace's size comes with its tensor."""
    for call in (_route(cnt=A, off=A, perm=A, workspace=A),
                 lambda: eo.q8_linear(A, eo.HFQ_F32, 64, 512, A, A, 512, A, eo.HFQ_F32, A)):
        _refused(call, "workspace")
