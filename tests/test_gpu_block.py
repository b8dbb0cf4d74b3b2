"""A layer as a decoder runs it: norm before the block (with its 8-bit form),
router, scored routing, routed HFQ4 experts beside an 8-bit shared expert, and
the join (shared gate, post norm, residual) fused with the next norm.

Every step is compared with the oracle on the inputs that the step itself had,
so that no error is excused by an earlier one; then the whole run is captured
into a graph and replayed over a new stream, with the bits of an eager run.

Bounds: the steps' own tests give them (u = 2^-24): logits (H + 1) u sum |x w|,
weights 2 (d + 24) u, 8-bit products 3 u, norms 24 u, each with half a step of
the output's type; the experts the library's 1e-3 of the row's largest.
"""
import numpy as np
import pytest

from oracle import moe, norm, q8, route, scored
from synth import workloads as W
from tests.gpu_util import TOL, OraclePackedLayer, device_fill, max_rel_err
from tests.test_gpu_parity import eo  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
U = 2.0 ** -24


class Model:
    """The tiny layer (H 256, I 128, E 16, top-4) with a router and a shared expert."""

    def __init__(self, eo):
        from expert_offload_b200.model import ExpertStore
        w = W.WORKLOADS[1]
        self.eo = eo
        H, I, E = w.hidden, w.inter, w.experts
        self.H, self.I, self.E, self.k = H, I, E, w.top_k
        self.store = ExpertStore(torch, 1, E, H, I, device_fill(torch, w))
        self.cache = moe.ExpertCache(OraclePackedLayer(w, 0), H, I)
        g = torch.Generator(device="cuda").manual_seed(5)

        def randn(*s, std=1.0, dt=torch.float32):
            return (torch.randn(*s, generator=g, device="cuda") * std).to(dt)

        self.router = randn(E, H, std=0.05, dt=torch.bfloat16)
        self.bias = randn(E, std=0.05)
        self.gu_q, self.gu_s = self.pack(randn(2 * I, H, std=0.05))
        self.dn_q, self.dn_s = self.pack(randn(H, I, std=0.05))
        self.shared_gate = randn(H, std=0.05)
        self.w_pre, self.w_post = randn(H, std=0.1) + 1, randn(H, std=0.1) + 1
        self.first = eo.NormRule(w_pre=self.w_pre, w_dtype=eo.HFQ_F32)
        self.join = eo.NormRule(w_post=self.w_post, w_pre=self.w_pre, w_dtype=eo.HFQ_F32, residual_scale=1.0,
                                branch_scale=0.5)
        self.rule = eo.RouteRule(score=eo.SCORE_SIGMOID, n_groups=4, topk_groups=2, group_top=2, scale=1.5)

    def pack(self, w):
        """Weights through the library's own quantiser: a row is a channel."""
        q = torch.empty(w.shape, dtype=torch.int8, device="cuda")
        s = torch.empty(w.shape[0], device="cuda")
        self.eo.q8_quantize_rows(w, self.eo.HFQ_F32, w.shape[0], w.shape[1], q, s)
        return q, s


@pytest.fixture(scope="module")
def model(eo):
    m = Model(eo)
    yield m
    m.store.close()


class Run:
    """Buffers of one batch size and the calls over them."""

    def __init__(self, m, T):
        self.m, self.T = m, T
        H, I, E, k, eo = m.H, m.I, m.E, m.k, m.eo

        def new(*s, dt=torch.float32):
            return torch.zeros(*s, dtype=dt, device="cuda")

        self.x = new(T, H, dt=torch.bfloat16)
        self.xn = [new(T, H, dt=torch.bfloat16) for _ in range(2)]
        self.xq, self.xs = [new(T, H, dt=torch.int8) for _ in range(2)], [new(T) for _ in range(2)]
        self.x_out = new(T, H, dt=torch.bfloat16)
        self.logits, self.idx, self.wts = new(T, E), new(T, k, dt=torch.int32), new(T, k)
        self.lists = [new(n, dt=torch.int32) for n in (E, E + 1, T * k)] if T > 8 else [None] * 3
        self.rws = new(max(1, eo.moe_route_scored_workspace_bytes(T, E, k)), dt=torch.uint8)
        self.ws = new(eo.hfq4_moe_workspace_bytes(T, k, H, I, E), dt=torch.uint8)
        self.y, self.gu, self.y2 = new(T, H), new(T, 2 * I), new(T, H)
        self.hq, self.hs, self.sg = new(T, I, dt=torch.int8), new(T), new(T)

    def go(self):
        m, eo, T = self.m, self.m.eo, self.T
        H, I, E, k = m.H, m.I, m.E, m.k
        bf, f32 = eo.HFQ_BF16, eo.HFQ_F32
        eo.moe_norm_residual(m.first, T, H, self.x, bf, xn=self.xn[0], xq=self.xq[0], xq_scale=self.xs[0])
        eo.moe_router_logits(self.xn[0], bf, T, H, m.router, bf, E, self.logits)
        eo.moe_route_scored(self.logits, f32, T, E, k, m.rule, self.idx, self.wts, bias=m.bias, cnt=self.lists[0],
                            off=self.lists[1], perm=self.lists[2], workspace=self.rws)
        eo.hfq4_moe_forward(m.store.layers[0], self.xn[0], bf, T, self.idx, self.wts, k, self.y, self.ws,
                            cnt=self.lists[0], off=self.lists[1], perm=self.lists[2])
        eo.q8_matmul(self.xq[0], self.xs[0], T, H, m.gu_q, m.gu_s, 2 * I, self.gu, f32)
        eo.q8_quantize_rows(self.gu, f32, T, I, self.hq, self.hs, act=eo.ACT_SWIGLU)
        eo.q8_matmul(self.hq, self.hs, T, I, m.dn_q, m.dn_s, H, self.y2, f32)
        torch.mv(self.xn[0].float(), m.shared_gate, out=self.sg)
        eo.moe_norm_residual(m.join, T, H, self.x, bf, y=self.y, y2=self.y2, y2_gate=self.sg, x_out=self.x_out,
                             xn=self.xn[1], xq=self.xq[1], xq_scale=self.xs[1])

    def outputs(self):
        return [self.xn[0], self.xq[0], self.logits, self.idx, self.wts, self.y, self.gu, self.hq, self.y2, self.x_out,
                self.xn[1], self.xq[1], self.xs[1]]


def _x(T, H, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(T, H, generator=g, device="cuda").bfloat16()


def _n(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("T", [1, 3, 8, 40, 300])
def test_a_layer_step_by_step(eo, model, T):
    m, r = model, Run(model, T)
    r.x.copy_(_x(T, m.H, T))
    r.go()
    torch.cuda.synchronize()
    x, xn = _n(r.x), _n(r.xn[0])
    ref = norm.rms_norm(x, _n(m.w_pre))
    assert np.all(np.abs(xn - ref) <= (24 * U + 2.0 ** -8) * np.abs(ref))
    q, s = q8.quantise(xn.astype(np.float32))
    np.testing.assert_array_equal(r.xq[0].cpu().numpy(), q)
    np.testing.assert_array_equal(r.xs[0].cpu().numpy(), s)
    lg = _n(r.logits)
    ref = route.router_logits(xn, _n(m.router))
    assert np.all(np.abs(lg - ref) <= (m.H + 1) * U * (np.abs(xn) @ np.abs(_n(m.router)).T))
    idx, wts = scored.route(lg, m.k, sigmoid=True, bias=_n(m.bias), n_groups=4, topk_groups=2, group_top=2, scale=1.5)
    np.testing.assert_array_equal(r.idx.cpu().numpy(), idx)
    tol = 2 * (2 * np.abs(lg).max(1, keepdims=True) + 24) * U
    assert np.all(np.abs(_n(r.wts) - wts) <= tol * wts)
    w = _n(r.wts)
    y = np.stack([sum(w[t, j] * moe.expert_ffn(*m.cache(int(idx[t, j])), xn[t]) for j in range(m.k)) for t in range(T)])
    assert max_rel_err(_n(r.y), y) <= TOL
    gu, _ = q8.matmul(q, s, m.gu_q.cpu().numpy(), _n(m.gu_s))
    assert np.all(np.abs(_n(r.gu) - gu) <= 3.01 * U * np.abs(gu))
    v = q8.swiglu(_n(r.gu))
    sc = _n(r.hs)[:, None]
    assert np.all(np.abs(_n(r.hq) * sc - v) <= 0.5 * sc * (1 + 1e-4) + 12 * U * np.abs(v))
    y2, _ = q8.matmul(r.hq.cpu().numpy(), _n(r.hs), m.dn_q.cpu().numpy(), _n(m.dn_s))
    assert np.all(np.abs(_n(r.y2) - y2) <= 3.01 * U * np.abs(y2))
    out = norm.join(x, _n(r.y), _n(r.y2), _n(r.sg), _n(m.w_post), beta=0.5)
    got = _n(r.x_out)
    b = _n(r.y) + norm.sigmoid(_n(r.sg))[:, None] * _n(r.y2)
    mag = np.abs(_n(r.y)) + norm.sigmoid(_n(r.sg))[:, None] * np.abs(_n(r.y2))
    rms = np.sqrt(np.mean(b * b, 1, keepdims=True) + 1e-6)
    cancel = np.sqrt(np.mean(mag * mag, 1, keepdims=True)) / rms
    tol = 40 * U * (np.abs(x) + 0.5 * mag / rms * np.abs(_n(m.w_post)) * (1 + 0.3 * cancel)) + 2.0 ** -8 * np.abs(out)
    assert np.all(np.abs(got - out) <= tol)
    ref = norm.rms_norm(got, _n(m.w_pre))
    assert np.all(np.abs(_n(r.xn[1]) - ref) <= (24 * U + 2.0 ** -8) * np.abs(ref))
    q, s = q8.quantise(_n(r.xn[1]).astype(np.float32))
    np.testing.assert_array_equal(r.xq[1].cpu().numpy(), q)
    np.testing.assert_array_equal(r.xs[1].cpu().numpy(), s)
    eo.hfq_workspace_status(r.ws)
    eo.hfq_workspace_status(None)


@pytest.mark.parametrize("T", [1, 5, 40])
def test_a_layer_captured_and_replayed(eo, model, T):
    eager, r = Run(model, T), Run(model, T)
    r.x.copy_(_x(T, model.H, 1))
    r.go()                                               # kernels loaded before the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r.go()
    for seed in (2, 3):
        for b in (eager, r):
            b.x.copy_(_x(T, model.H, seed))
        eager.go()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager.outputs(), r.outputs()):
            assert torch.equal(a, b)
