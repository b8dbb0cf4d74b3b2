"""moe_norm_residual on the GPU against the fp64 oracle.

Bounds, with u = 2^-24 and h = half a step of the output's type: a sum of
squares of at most 8192 terms, 16 in a thread's chain, then two butterflies of
5, is within 30 u of its value, its root within 16 u, the quotient adds 2 u; a
sigmoid (expf 2 ulp, sum, quotient) is within 8 u; each further product or sum
adds 1 u.  An element of x' is alpha x + beta g r w (y + g2 y2): every term
carries fewer than 40 u of its own magnitude, so
    |err| <= 40 u (alpha |x| + beta |g r w| (|y| + g2 |y2|)) + h |x'|.
The mean that r comes from is taken of values b = y + g2 y2 whose own error is
relative to |y| + g2 |y2|; its part in r is that error's root mean square over
b's, at most 12 u cancel with cancel = rms(|y| + g2 |y2|) / rms(b).
xn is checked against the norm of the x' that the call itself wrote, which
is what it is defined as: |err| <= (24 u + h) |xn|.
"""
import numpy as np
import pytest

from oracle import norm, q8
from tests.test_gpu_parity import eo  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
GUARD = 12345.0


def _t(g, *shape, dt="f32", std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(DT[dt])


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


class Case:
    """One call's inputs and guarded outputs."""

    def __init__(self, eo, T, H, x="bf16", y="f32", w=None, xn=None, post=True, pre=True, shared=None, gate="none",
                 act=1, alpha=1.0, beta=1.0, offset=0.0, eps=1e-6, ldx=0, ldy=0, shift=0, seed=0, out=True,
                 inplace=False, quant=False, branch=True):
        g = torch.Generator(device="cuda").manual_seed(seed + T * 31 + H)
        w, xn = w or x, xn or x
        self.eo, self.T, self.H, self.kinds = eo, T, H, (x, y, w, xn)
        self.ldx, self.ldy = ldx or H, ldy or H

        def rows(ld, dt, std=1.0, n=T):                  # a buffer `shift` elements off a 16-byte address
            return _t(g, n * ld + shift, dt=dt, std=std)[shift:]

        self.x = rows(self.ldx, x)
        self.y = rows(self.ldy, y, 0.5) if branch else None
        self.y2 = rows(self.ldy, y, 0.5) if shared else None
        self.y2_gate = _t(g, T) if shared == "gate" else None
        self.w_post = _t(g, H, dt=w) if post and branch else None
        self.w_pre = _t(g, H, dt=w) if pre else None
        shape = {"none": None, "token": (T,), "channel": (H,), "full": (T, H)}[gate]
        self.gate = _t(g, *shape) if shape else None
        self.kind = ("none", "token", "channel", "full").index(gate)
        self.act, self.alpha, self.beta, self.offset, self.eps = act, alpha, beta, offset, eps
        self.x0 = self.x.clone()
        self.x_out = self.x if inplace else (torch.full_like(self.x, GUARD) if out else None)
        self.xn = torch.full((T * H + 8,), GUARD, dtype=DT[xn], device="cuda")
        self.h16 = -(-H // 16) * 16
        self.xq = torch.full((T * self.h16 + 16,), 77, dtype=torch.int8, device="cuda") if quant else None
        self.xs = torch.full((T + 4,), GUARD, dtype=torch.float32, device="cuda") if quant else None

    def call(self, stream=None, with_xn=True):
        eo, (x, y, w, xn) = self.eo, self.kinds
        dt = {"f32": eo.HFQ_F32, "bf16": eo.HFQ_BF16}
        rule = eo.NormRule(self.w_post, self.w_pre, dt[w], self.eps, self.offset, self.alpha, self.beta, self.kind,
                           self.act)
        eo.moe_norm_residual(rule, self.T, self.H, self.x, dt[x], y=self.y, y_dtype=dt[y], y2=self.y2,
                             y2_gate=self.y2_gate, gate=self.gate, x_out=self.x_out, xn=self.xn if with_xn else None,
                             xn_dtype=dt[xn], xq=self.xq, xq_scale=self.xs, ldx=self.ldx, ldy=self.ldy, stream=stream)
        torch.cuda.synchronize()
        return self

    def rows(self, t, ld):
        return None if t is None else _np(t)[:self.T * ld].reshape(self.T, ld)[:, :self.H]

    def check(self):
        T, H, (xk, _, _, xnk) = self.T, self.H, self.kinds
        x0, y, y2 = self.rows(self.x0, self.ldx), self.rows(self.y, self.ldy), self.rows(self.y2, self.ldy)
        g = 1.0
        if self.gate is not None:
            g = norm.sigmoid(_np(self.gate)) if self.act else _np(self.gate)
            g = g[:, None] if self.kind == 1 else g
        ref = x0
        if y is not None:
            ref = norm.join(x0, y, y2, _np(self.y2_gate), _np(self.w_post), g, self.eps, self.offset, self.alpha,
                            self.beta)
            g2 = 0.0 if y2 is None else (norm.sigmoid(_np(self.y2_gate))[:, None] if self.y2_gate is not None else 1.0)
            mag = np.abs(y) + (0.0 if y2 is None else g2 * np.abs(y2))
            b = y + (0.0 if y2 is None else g2 * y2)
            cancel = 0.0
            if self.w_post is not None:
                rms = np.sqrt(np.mean(b * b, 1, keepdims=True) + self.eps)
                cancel = np.sqrt(np.mean(mag * mag, 1, keepdims=True)) / rms
                mag = mag / rms * np.abs(_np(self.w_post) + self.offset)
            mag = abs(self.alpha) * np.abs(x0) + abs(self.beta) * np.abs(g) * mag * (1 + 0.3 * cancel)
            tol = 40 * U * mag + HALF[xk] * np.abs(ref)
        else:
            tol = 0.0
        got = ref
        if self.x_out is not None:
            got = self.rows(self.x_out, self.ldx)
            assert np.all(np.abs(got - ref) <= tol), float(np.max(np.abs(got - ref) / np.maximum(tol, 1e-300)))
            if self.ldx > H:                             # between the rows: untouched
                flat = _np(self.x_out)[:T * self.ldx].reshape(T, self.ldx)[:, H:]
                want = _np(self.x0)[:T * self.ldx].reshape(T, self.ldx)[:, H:] if self.x_out is self.x else GUARD_OF[xk]
                assert np.all(flat == want)
        elif y is not None:
            return self
        want = norm.rms_norm(got, _np(self.w_pre), self.eps, self.offset if self.w_pre is not None else 0.0)
        xn = _np(self.xn)
        assert np.all(xn[T * H:] == GUARD_OF[xnk])
        xn = xn[:T * H].reshape(T, H)
        assert np.all(np.abs(xn - want) <= (24 * U + HALF[xnk]) * np.abs(want) + 1e-38)
        if self.xq is not None:
            q, s = q8.quantise(xn.astype(np.float32))
            buf = self.xq.cpu().numpy()
            assert np.all(buf[T * self.h16:] == 77) and np.all(_np(self.xs)[T:] == GUARD)
            buf = buf[:T * self.h16].reshape(T, self.h16)
            np.testing.assert_array_equal(buf[:, :H], q)
            assert np.all(buf[:, H:] == 0)
            np.testing.assert_array_equal(self.xs.cpu().numpy()[:T], s)
        return self


GUARD_OF = {"f32": GUARD, "bf16": float(torch.tensor(GUARD).bfloat16())}


@pytest.mark.parametrize("T", [1, 3, 300])
@pytest.mark.parametrize("H", [1, 7, 8, 128, 255, 256, 1001, 2048, 2049, 4096, 8191, 8192])
@pytest.mark.parametrize("x,y", [("bf16", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("f32", "f32")])
def test_join_and_norm(eo, T, H, x, y):
    if T * H > 1 << 21:
        T = 17
    Case(eo, T, H, x, y, shared="gate", gate="token").call().check()
    Case(eo, T, H, x, y, gate="channel", act=0, alpha=0.5, beta=0.25, offset=1.0, quant=True).call().check()


@pytest.mark.parametrize("H", [24, 1000, 2048, 2050, 8192])
@pytest.mark.parametrize("gate", ["none", "token", "channel", "full"])
@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("shared", [None, "plain", "gate"])
def test_every_part(eo, H, gate, act, post, shared):
    Case(eo, 5, H, "bf16", "f32", post=post, gate=gate, act=act, shared=shared, alpha=0.7, beta=1.3).call().check()


@pytest.mark.parametrize("x,w,xn", [("bf16", "f32", "bf16"), ("bf16", "bf16", "f32"), ("f32", "bf16", "bf16")])
@pytest.mark.parametrize("H", [96, 2047, 4104])
def test_mixed_types(eo, x, w, xn, H):
    Case(eo, 9, H, x, "f32", w=w, xn=xn, quant=True).call().check()


@pytest.mark.parametrize("H", [8, 1001, 2048, 8192])
def test_plain_norm_and_its_8_bits(eo, H):
    Case(eo, 11, H, branch=False, quant=True).call().check()
    Case(eo, 11, H, branch=False, pre=False, out=False).call().check()
    c = Case(eo, 11, H, quant=True, seed=3)
    a = c.call().check().xq.clone()
    c.xq.fill_(77)
    c.call(with_xn=False)                                # the same bytes without the row itself
    assert torch.equal(a, c.xq)


@pytest.mark.parametrize("H,ldx,ldy,shift", [(256, 264, 300, 0), (256, 256, 256, 1), (100, 111, 103, 3),
                                             (2048, 4096, 2056, 8), (8192, 8200, 8192, 5)])
@pytest.mark.parametrize("inplace", [False, True])
def test_strides_alignment_and_in_place(eo, H, ldx, ldy, shift, inplace):
    for x, y in (("bf16", "f32"), ("f32", "bf16")):
        Case(eo, 13, H, x, y, ldx=ldx, ldy=ldy, shift=shift, inplace=inplace, shared="gate").call().check()


def test_rows_of_zeros_and_without_eps(eo):
    c = Case(eo, 4, 512, "f32", "f32", eps=0.0, quant=True)
    c.x[:512] = 0
    c.y[:512] = 0
    c.x0 = c.x.clone()
    c.call()
    assert torch.isnan(c.x_out[:512]).all()              # 0 / 0, as the formula has it
    c = Case(eo, 4, 512, "f32", "f32", quant=True)
    c.x[:512] = 0
    c.y[:512] = 0
    c.x0 = c.x.clone()
    c.call().check()
    assert float(c.xs[0]) == 0.0


def test_rows_whose_squares_leave_the_f32_range(eo):
    c = Case(eo, 3, 1000, "f32", "f32", post=False)
    c.x.mul_(1e25)
    c.y.mul_(1e25)
    c.x0 = c.x.clone()
    c.call().check()
    c = Case(eo, 3, 1000, "f32", "f32", post=True)
    c.y.mul_(1e30)
    c.call().check()


@pytest.mark.parametrize("H", [64, 1000, 1001, 8192])
def test_rows_at_the_ends_of_the_f32_range(eo, H):
    """Rows up to the largest f32, and rows whose squares underflow where no eps covers them."""
    for scale, eps in ((1.0, 1e-6), (2.0 ** -100, 0.0), (2.0 ** -70, 0.0), (2.0 ** -30, 2.0 ** -62)):
        c = Case(eo, 3, H, "f32", "f32", branch=False, eps=eps)
        c.x.copy_(c.x / c.x.abs().max() * (3.4e38 if scale == 1.0 else 1.0) * scale)
        c.x0 = c.x.clone()
        c.call().check()


@pytest.mark.parametrize("H", [1, 64, 1001, 8192])
def test_rows_of_the_least_f32_values(eo, H):
    """Below 2^-126, where a value has few bits left but its norm has them all."""
    for scale in (2.0 ** -126, 2.0 ** -140, 2.0 ** -149):
        c = Case(eo, 3, H, "f32", "f32", branch=False, eps=0.0)
        c.x.copy_(torch.round(c.x / c.x.abs().max() * 2.0 ** 9).double() * scale)
        c.x[::H] = 2.0 ** -149                           # no row of zeros
        assert (c.x.view(3, H) != 0).any(1).all() and float(c.x.abs().max()) <= 2.0 ** 9 * scale
        c.x0 = c.x.clone()
        c.call().check()
        c = Case(eo, 3, H, "f32", "f32", eps=0.0)        # the branch's own norm
        c.y.copy_(torch.round(c.y / c.y.abs().max() * 2.0 ** 9).double() * scale)
        c.y[::H] = 2.0 ** -149
        c.call().check()


def test_a_rule_with_a_gate_serves_a_row_without_a_block(eo):
    """A gate's kind says nothing where there is no block: the plain norm."""
    for gate in ("token", "channel", "full"):
        c = Case(eo, 7, 256, branch=False)
        c.kind = ("none", "token", "channel", "full").index(gate)
        c.call().check()


def test_nan_and_infinity_stay_in_their_row(eo):
    for H in (256, 1001):
        a = Case(eo, 6, H, "bf16", "f32", shared="gate", quant=True, seed=1)
        good = a.call().check().xn.clone()
        b = Case(eo, 6, H, "bf16", "f32", shared="gate", quant=True, seed=1)
        b.y[1 * H + 5] = float("nan")
        b.y[4 * H + H - 1] = float("inf")
        b.call()
        for t in (0, 2, 3, 5):
            assert torch.equal(b.xn[t * H:(t + 1) * H], good[t * H:(t + 1) * H])
        for t in (1, 4):
            assert torch.isnan(b.xn[t * H:(t + 1) * H]).any() and torch.isnan(b.xs[t])
            assert (b.xq[t * b.h16:(t + 1) * b.h16] == 0).all()


def test_many_rows(eo):
    Case(eo, 8192, 256, "bf16", "bf16", shared="plain", quant=True).call().check()
    c = Case(eo, 65536, 40, "bf16", "bf16", post=False).call().check()
    with pytest.raises(eo.HfqError):
        c.T = 65537
        c.call()


def test_captured_call_and_another_stream(eo):
    c = Case(eo, 130, 2048, shared="gate", gate="full", quant=True)
    a = c.call().check().xn.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.xn.fill_(GUARD)
    torch.cuda.synchronize()
    assert torch.equal(c.call(stream=s).xn, a)
    rule = eo.NormRule(c.w_post, c.w_pre, eo.HFQ_BF16, c.eps, 0.0, 1.0, 1.0, c.kind, c.act)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        eo.moe_norm_residual(rule, c.T, c.H, c.x, eo.HFQ_BF16, y=c.y, y2=c.y2, y2_gate=c.y2_gate, gate=c.gate,
                             x_out=c.x_out, xn=c.xn)
    c.xn.fill_(GUARD)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.xn, torch.cat([a[:-8], c.xn[-8:]]))
    c.y.neg_()
    g.replay()
    torch.cuda.synchronize()
    c.quantless = c.xq, c.xq
    c.xq = None
    c.check()


def test_a_rules_weights_belong_to_the_current_device(eo, monkeypatch):
    c = Case(eo, 4, 256).call().check()
    rule = eo.NormRule(None, c.w_pre, eo.HFQ_BF16)
    eo.moe_norm_residual(rule, 4, 256, c.x, eo.HFQ_BF16, xn=c.xn)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)      # as if another were current
    with pytest.raises(eo.HfqError, match="w_pre"):
        rule_call = dict(x_dtype=eo.HFQ_BF16, xn=c.xn, stream=torch.cuda.default_stream(0))
        eo.moe_norm_residual(rule, 4, 256, c.x, **rule_call)
    monkeypatch.undo()
    with pytest.raises(eo.HfqError, match="w_pre"):
        eo.moe_norm_residual(eo.NormRule(None, c.w_pre.cpu(), eo.HFQ_BF16), 4, 256, c.x, eo.HFQ_BF16, xn=c.xn)
