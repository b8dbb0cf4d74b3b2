"""Forms of the calls beside the experts that their documents allow: a join
without its residual output, list borders, rules that send ordinary scores to
64 bits, branches of a captured graph, and calls from two threads."""
import threading

import numpy as np
import pytest

from oracle import route
from tests.test_gpu_norm import Case
from tests.test_gpu_parity import eo  # noqa: F401
from tests.test_gpu_scored_route import _bias, _check, _rand, _run

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("H", [64, 1001, 2048, 4096, 8191])
@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_a_join_that_keeps_no_residual(eo, H, x):
    """x_out NULL: x' is rounded to x's type all the same, so xn, xq and their
    scales are the bits of the call that writes x'."""
    for kw in (dict(shared="gate", gate="token"), dict(gate="full", post=False, ldx=H + 3, shift=1)):
        with_x = Case(eo, 7, H, x, "f32", quant=True, **kw).call().check()
        without = Case(eo, 7, H, x, "f32", quant=True, out=False, **kw).call()
        assert without.x_out is None and torch.equal(without.x, without.x0)
        for a, b in ((with_x.xn, without.xn), (with_x.xq, without.xq), (with_x.xs, without.xs)):
            assert torch.equal(a, b)
        without.xq.fill_(77)
        without.call(with_xn=False)                      # the 8-bit row alone
        assert torch.equal(with_x.xq, without.xq)


@pytest.mark.parametrize("T", [16, 17, 1184, 1185, 2368, 2369, 8191, 8192, 8193])
@pytest.mark.parametrize("E,k", [(512, 8), (33, 3), (16, 16)])
def test_lists_where_their_ways_change(eo, T, E, k):
    """One block alone up to 16 tokens; chunks of 8 tokens up to 1184, of 16 up to
    2368, of 32 behind; a kernel of its own for the counts of more than 256 chunks."""
    l = _rand(T, E, T + E, std=2.0)
    got = _run(eo, l, k, dict(score=0), lists=True)
    idx = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :k].int().cpu().numpy()
    np.testing.assert_array_equal(got[0], idx)
    for a, b in zip(got[2:], route.group_by_expert(idx, E)):
        np.testing.assert_array_equal(a, b)


@pytest.mark.parametrize("T,lists", [(1, False), (9, True), (150, True), (150, False)])
@pytest.mark.parametrize("E,k,n,tg", [(512, 16, 8, 4), (512, 14, 8, 4), (256, 16, 8, 4), (512, 8, 8, 1), (512, 8, 16, 2),
                                      (512, 8, 32, 4), (512, 16, 1, 1)])
@pytest.mark.parametrize("score", [0, 1], ids=["softmax", "sigmoid"])
def test_ordinary_scores_that_64_bits_decide(eo, T, lists, E, k, n, tg, score):
    """Distinct scores under rules that leave few live lanes for k experts: the
    bound from the lanes' best then lets more than 32 candidates through."""
    l = _rand(T, E, T + E + k)
    assert all(len(set(r)) == E for r in l.cpu().tolist())
    for gt in (1, 2):
        for bias in (None, _bias(E, 5, 0.1 if score else 0.5 / E)):
            _check(eo, l, k, dict(score=score, n_groups=n, topk_groups=tg, group_top=gt, scale=2.5), bias, lists=lists)


@pytest.mark.parametrize("T", [1, 5, 40, 300])
def test_branches_of_a_captured_graph(eo, T):
    """The shared expert on a stream of its own beside the routing, both behind
    one norm and before one join, captured and replayed over new rows."""
    H, I, E, k = 1024, 640, 64, 6
    g = torch.Generator(device="cuda").manual_seed(T)
    bf, f32 = eo.HFQ_BF16, eo.HFQ_F32

    def randn(*s, dt=torch.float32, std=1.0):
        return (torch.randn(*s, generator=g, device="cuda") * std).to(dt)

    x, router, gate = randn(T, H, dt=torch.bfloat16), randn(E, H, dt=torch.bfloat16, std=0.05), randn(T)
    wq, ws = torch.empty(H, H, dtype=torch.int8, device="cuda"), torch.empty(H, device="cuda")
    eo.q8_quantize_rows(randn(H, H, std=0.05), f32, H, H, wq, ws)
    xn, xq, xs = (torch.empty(*s, dtype=d, device="cuda") for s, d in
                  (((T, H), torch.bfloat16), ((T, H), torch.int8), ((T,), torch.float32)))
    logits, y, y2 = (torch.empty(T, n, device="cuda") for n in (E, H, H))
    idx, wts = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    lists = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (E, E + 1, T * k)]
    rws = torch.zeros(eo.moe_route_scored_workspace_bytes(T, E, k) or 16, dtype=torch.uint8, device="cuda")
    qws = [torch.zeros(eo.q8_linear_workspace_bytes(T, H, H) or 16, dtype=torch.uint8, device="cuda") for _ in range(2)]
    x_out, xn2 = torch.empty_like(x), torch.empty_like(x)
    rule = eo.RouteRule(score=eo.SCORE_SIGMOID, n_groups=4, topk_groups=2, group_top=2)
    first = eo.NormRule(None, randn(H, dt=torch.bfloat16), bf)
    join = eo.NormRule(randn(H, dt=torch.bfloat16), randn(H, dt=torch.bfloat16), bf)
    side = torch.cuda.Stream()

    def run():
        main = torch.cuda.current_stream()
        eo.moe_norm_residual(first, T, H, x, bf, xn=xn, xq=xq, xq_scale=xs)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            eo.q8_matmul(xq, xs, T, H, wq, ws, H, y2, f32)
        eo.moe_router_logits(xn, bf, T, H, router, bf, E, logits)
        eo.moe_route_scored(logits, f32, T, E, k, rule, idx, wts, cnt=lists[0], off=lists[1], perm=lists[2],
                            workspace=rws)
        eo.q8_linear(xn, bf, T, H, wq, ws, H, y, f32, qws[0])
        main.wait_stream(side)
        eo.moe_norm_residual(join, T, H, x, bf, y=y, y2=y2, y2_gate=gate, x_out=x_out, xn=xn2)

    outs = [idx, wts, *lists, y, y2, x_out, xn2]
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            run()
    for _ in range(4):
        x.copy_(randn(T, H, dt=torch.bfloat16))
        torch.cuda.synchronize()
        run()
        torch.cuda.synchronize()
        want = [o.clone() for o in outs]
        for o in outs:
            o.zero_()
        for _ in range(5):
            graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
    assert torch.equal(y, y2)                            # the same product by two ways
    eo.hfq_workspace_status(None)


def test_calls_from_two_threads(eo):
    """Each thread its stream, buffers and workspace."""
    shapes = [(5, 1024, 512), (300, 512, 1000), (2, 512, 300), (1024, 256, 4096)]
    bad = []

    def work(seed):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for i in range(40):
                    T, K, N = shapes[(i + seed) % len(shapes)]
                    x = _rand(T, K, 100 * seed + i)
                    w = torch.randint(-127, 128, (N, K), device="cuda").to(torch.int8)
                    ws, y, z = torch.rand(N, device="cuda"), torch.empty(T, N, device="cuda"), torch.empty(T, N, device="cuda")
                    q, s = torch.empty(T, K, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
                    buf = torch.empty(eo.q8_linear_workspace_bytes(T, K, N) or 16, dtype=torch.uint8, device="cuda")
                    eo.q8_linear(x, eo.HFQ_F32, T, K, w, ws, N, y, eo.HFQ_F32, buf)
                    eo.q8_quantize_rows(x, eo.HFQ_F32, T, K, q, s)
                    eo.q8_matmul(q, s, T, K, w, ws, N, z, eo.HFQ_F32)
                    ref = (q.double() @ w.double().t()) * s.double()[:, None] * ws.double()
                    if not torch.equal(y, z) or not ((z - ref).abs() <= 4 * 2.0 ** -24 * ref.abs() + 1e-44).all():
                        bad.append((seed, i))
                    torch.cuda.current_stream().synchronize()
        except Exception as e:                           # noqa: BLE001  (reported by the main thread)
            bad.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(n,)) for n in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
    eo.hfq_workspace_status(None)
