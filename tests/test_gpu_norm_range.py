"""The join where its factors leave the f32 range together though the formula
does not: a row's norm, its gate and the branch scale are one number for the
row, and their product can be 0 or infinite where the branch, normed first and
scaled after that, is an ordinary number.  The residual is scaled by 0, so that
the branch is all there is to see.

Bounds are those of the join's own tests (40 u of the terms' magnitude): the
factors multiplied one after the other are one rounding more, of the 12 or so
that the bound leaves room for.
"""
import pytest

from tests.test_gpu_norm import Case, DT  # noqa: F401
from tests.test_gpu_parity import eo  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

# y's factor, branch scale, gate's factor (linear), eps; outputs stay above 2^-126, below which a
# rounding is no longer relative
ENDS = [(1e16, 1.0, 1e-30, 1e-6), (1e16, 1e-30, 1.0, 1e-6), (1e18, 1e-20, 1e-10, 1e-6), (1.0, 1e-30, 1e30, 1e-6),
        (1.0, 1e30, 1e-30, 1e-6), (1e-25, 1.0, 1e20, 0.0), (1e-25, 1e25, 1.0, 0.0), (2.0 ** -140, 1.0, 1e20, 0.0),
        (2.0 ** -140, 1e20, 1.0, 0.0), (2.0 ** -140, 1e-20, 1e30, 0.0), (3e30, 1e-10, 1e-20, 1e-6),
        (3e30, 1e10, 1e20, 1e-6), (1e-3, 1e-35, 1e35, 1e-6), (1.0, 0.0, 1.0, 1e-6), (1e16, 1e-28, 1.0, 1e-6)]


def _case(eo, T, H, gate, y_factor, beta, g_factor, eps, **kw):
    c = Case(eo, T, H, "f32", "f32", gate=gate, act=0, alpha=0.0, beta=beta, eps=eps, **kw)
    y = c.y.double() / c.y.abs().max().double()
    if y_factor < 2.0 ** -126:                           # whole numbers of the least f32, none of the rows 0
        y = torch.round(y * 512)
        y[::H] = 1.0
    c.y.copy_(y * y_factor)
    if c.gate is not None:
        c.gate.copy_((c.gate.sign() + 0.1 * c.gate).double() * g_factor)
    return c


def _ahead(b, beta, g):
    """An element's gate comes after the branch scale: that times the branch has
    to be in the range, so what is beyond goes to the gate."""
    least, most = 1e-25 / b, 1e25 / b
    clipped = beta if beta == 0.0 else min(max(beta, least), most)
    return clipped, g * (beta / clipped if clipped else 1.0)


@pytest.mark.parametrize("H", [64, 1001, 2048, 4096, 8191])
@pytest.mark.parametrize("gate", ["none", "token", "channel", "full"])
@pytest.mark.parametrize("ends", ENDS)
def test_norm_gate_and_scale_at_both_ends(eo, H, gate, ends):
    if gate == "none" and ends[2] != 1.0:
        ends = (ends[0], ends[1] * ends[2], 1.0, ends[3])
    if gate in ("channel", "full"):
        ends = (ends[0],) + _ahead(1.0, ends[1], ends[2]) + ends[3:]
    _case(eo, 3, H, gate, *ends).call().check()


@pytest.mark.parametrize("H", [64, 1001, 8192])
@pytest.mark.parametrize("gate", ["token", "channel", "full"])
@pytest.mark.parametrize("ends", [e for e in ENDS if 1e-12 < e[0] * e[1] * e[2] < 1e12])
def test_without_a_post_norm(eo, H, gate, ends):
    """b = y: a token's gate and the branch scale meet first."""
    if gate != "token":
        ends = (ends[0],) + _ahead(ends[0], ends[1], ends[2]) + ends[3:]
    _case(eo, 3, H, gate, *ends, post=False).call().check()


@pytest.mark.parametrize("H", [64, 1001, 8192])
def test_weights_at_both_ends(eo, H):
    """1 / rms times a weight can leave the range, too, where the normed row
    times the weight does not: of the post norm and of the next one."""
    for factor, w in ((1e-25, 1e25), (1e16, 1e-30), (2.0 ** -140, 1e30), (1e30, 1e-25)):
        c = _case(eo, 3, H, "none", factor, 1.0, 1.0, 0.0)
        c.w_post.mul_(w)
        c.call().check()
        c = Case(eo, 3, H, "f32", "f32", branch=False, eps=0.0)
        x = c.x.double() / c.x.abs().max().double()
        c.x.copy_(torch.round(x * 512).double() * factor if factor < 1e-30 else x * factor)
        c.x[::H] = max(factor, 2.0 ** -149)
        c.x0 = c.x.clone()
        c.w_pre.mul_(w)
        c.call().check()


@pytest.mark.parametrize("H", [64, 2048, 8191])
def test_sigmoid_gates_that_are_nearly_closed(eo, H):
    for y_factor in (1.0, 1e16):
        c = Case(eo, 5, H, "f32", "f32", gate="token", act=1, alpha=0.0)
        c.y.mul_(y_factor)
        c.gate.copy_(torch.tensor([-20.0, -25.0, -40.0, -60.0, -80.0]))
        c.call().check()
