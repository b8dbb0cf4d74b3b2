"""Operands that the kernel directly before writes anew each time.

The calls beside the experts are set up while their predecessor on the stream
still runs; whatever it writes (weights and their scales, token scales, a
selection bias) they have to find as it left it.  A captured run of the two is
replayed over changing inputs and compared with the same calls made one by one
with the device idle between them, bit for bit.
"""
import pytest

from tests.test_gpu_parity import eo  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def _randn(seed, *shape, dt=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dt)


def _replay(steps, outs, change, rounds=6):
    """`steps`: the calls in order; `change(i)` makes the inputs of round i."""
    def eager():
        for f in steps:
            f()
            torch.cuda.synchronize()
        return [o.clone() for o in outs]

    change(0)
    eager()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):                               # the run's own end comes before its start, too
            for f in steps:
                f()
    seen = []
    for i in range(1, rounds + 1):
        change(i)
        want = eager()
        change(i - 1)
        for f in steps:                                  # what they held before: another round's
            f()
        torch.cuda.synchronize()
        change(i)
        graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
        seen.append(want)
    assert any(not torch.equal(a, b) for a, b in zip(seen[0], seen[1]))


@pytest.mark.parametrize("T,K,N", [(1, 2048, 512), (2, 512, 300), (5, 1024, 700), (8, 8192, 256), (40, 1024, 300),
                                   (300, 200, 1500), (1024, 512, 4096)])
def test_weights_and_their_scales(eo, T, K, N):
    """The dot kernel, the fused one, tiles with K split and whole, CTA pairs."""
    k16 = -(-K // 16) * 16
    w, x = torch.empty(N, K, device="cuda"), torch.empty(T, K, device="cuda")
    wq, ws = torch.empty(N, k16, dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda")
    xq, xs = torch.empty(T, k16, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    y, z = torch.empty(T, N, device="cuda"), torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    work = torch.zeros(eo.q8_linear_workspace_bytes(T, K, N) or 1, dtype=torch.uint8, device="cuda")

    def change(i):
        w.copy_(_randn(10 + i, N, K) * (1 + i))
        x.copy_(_randn(50 + i, T, K) * (9 - i))

    _replay([lambda: eo.q8_quantize_rows(x, eo.HFQ_F32, T, K, xq, xs),
             lambda: eo.q8_quantize_rows(w, eo.HFQ_F32, N, K, wq, ws),
             lambda: eo.q8_matmul(xq, xs, T, K, wq, ws, N, y, eo.HFQ_F32),
             lambda: eo.q8_quantize_rows(w, eo.HFQ_F32, N, K, wq, ws),
             lambda: eo.q8_linear(x, eo.HFQ_F32, T, K, wq, ws, N, z, eo.HFQ_BF16, work)], [y, z], change)


@pytest.mark.parametrize("T,K,N", [(1, 2048, 512), (5, 8192, 640), (40, 1024, 300), (1024, 512, 4096)])
def test_token_scales(eo, T, K, N):
    k16 = -(-K // 16) * 16
    x = torch.empty(T, K, device="cuda")
    wq = torch.empty(N, k16, dtype=torch.int8, device="cuda")
    ws = torch.empty(N, device="cuda")
    eo.q8_quantize_rows(_randn(3, N, K), eo.HFQ_F32, N, K, wq, ws)
    xq, xs = torch.empty(T, k16, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    y = torch.empty(T, N, device="cuda")
    _replay([lambda: eo.q8_quantize_rows(x, eo.HFQ_F32, T, K, xq, xs),
             lambda: eo.q8_matmul(xq, xs, T, K, wq, ws, N, y, eo.HFQ_F32)], [y],
            lambda i: x.copy_(_randn(50 + i, T, K) * (9 - i)))


@pytest.mark.parametrize("T,E", [(1, 256), (8, 512), (16, 64), (300, 160), (2000, 512)])
def test_selection_bias(eo, T, E):
    """The bias is what a norm has just written."""
    raw = torch.empty(1, E, device="cuda")
    bias = torch.empty(1, E, device="cuda")
    logits, k = _randn(4, T, E), 6
    rule, r = eo.NormRule(residual_scale=1.0), eo.RouteRule(score=eo.SCORE_SIGMOID)
    idx, wts = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    idx2, wts2 = torch.empty_like(idx), torch.empty_like(wts)
    lists = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (E, E + 1, T * k)]
    work = torch.zeros(eo.moe_route_scored_workspace_bytes(T, E, k) or 16, dtype=torch.uint8, device="cuda")

    def norm():
        eo.moe_norm_residual(rule, 1, E, raw, eo.HFQ_F32, xn=bias, xn_dtype=eo.HFQ_F32)

    _replay([norm, lambda: eo.moe_route_scored(logits, eo.HFQ_F32, T, E, k, r, idx, wts, bias=bias), norm,
             lambda: eo.moe_route_scored(logits, eo.HFQ_F32, T, E, k, r, idx2, wts2, bias=bias, cnt=lists[0],
                                         off=lists[1], perm=lists[2], workspace=work)],
            [idx, wts, idx2, wts2] + lists, lambda i: raw.copy_(_randn(20 + i, 1, E)))
