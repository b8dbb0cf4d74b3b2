"""A launch that fails is the failing call's alone: the next call, which checks
its own launch, finds no error of an earlier one.  The failures are the host's:
calls on a stream whose capture is no longer valid."""
import ctypes

import pytest

from tests.test_gpu_parity import eo  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
THREAD_LOCAL = 1


def _good_calls(eo):
    """Calls of this library that read the last error after their launch."""
    logits = torch.randn(4, 64, device="cuda")
    idx, wts = torch.empty(4, 4, dtype=torch.int32, device="cuda"), torch.empty(4, 4, device="cuda")
    x, wr = torch.randn(4, 256, device="cuda"), torch.randn(64, 256, device="cuda")
    w, ws = torch.ones(64, 256, dtype=torch.int8, device="cuda"), torch.ones(64, device="cuda")
    y = torch.empty(4, 64, device="cuda")
    return [lambda: eo.moe_route(logits, 4, 64, 4, idx, wts),
            lambda: eo.moe_router_logits(x, eo.HFQ_F32, 4, 256, wr, eo.HFQ_F32, 64, logits),
            lambda: eo.q8_linear(x, eo.HFQ_F32, 4, 256, w, ws, 64, y, eo.HFQ_F32),
            lambda: eo.moe_norm_residual(eo.NormRule(), 4, 256, x, eo.HFQ_F32, xn=x.clone(), xn_dtype=eo.HFQ_F32)]


def _bad_calls(eo, s):
    logits = torch.randn(300, 64, device="cuda")
    idx, wts = torch.empty(300, 4, dtype=torch.int32, device="cuda"), torch.empty(300, 4, device="cuda")
    lists = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (64, 65, 1200)]
    work = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    x = torch.randn(300, 256, device="cuda")
    w, ws = torch.ones(4096, 256, dtype=torch.int8, device="cuda"), torch.ones(4096, device="cuda")
    q, qs = torch.empty(300, 256, dtype=torch.int8, device="cuda"), torch.ones(300, device="cuda")
    y = torch.empty(2048 * 4096, device="cuda")          # flat: rows as each call says
    big, bs = torch.ones(2048, 256, dtype=torch.int8, device="cuda"), torch.ones(2048, device="cuda")
    f32 = eo.HFQ_F32
    return {"status": lambda: eo.hfq_workspace_status(None, stream=s),
            "norm": lambda: eo.moe_norm_residual(eo.NormRule(), 300, 256, x, f32, xn=x.clone(), xn_dtype=f32, stream=s),
            "route": lambda: eo.moe_route_scored(logits, f32, 300, 64, 4, eo.RouteRule(), idx, wts, stream=s),
            "lists": lambda: eo.moe_route_scored(logits, f32, 300, 64, 4, eo.RouteRule(), idx, wts, cnt=lists[0],
                                                 off=lists[1], perm=lists[2], workspace=work, stream=s),
            "quantise": lambda: eo.q8_quantize_rows(x, f32, 300, 256, q, qs, stream=s),
            "dot": lambda: eo.q8_matmul(q, qs, 1, 256, w, ws, 64, y, f32, stream=s),
            "tiles": lambda: eo.q8_matmul(q, qs, 300, 256, w, ws, 64, y, f32, stream=s),
            "pairs": lambda: eo.q8_matmul(big, bs, 2048, 256, w, ws, 4096, y, f32, stream=s),
            "fused": lambda: eo.q8_linear(x, f32, 5, 256, w, ws, 4096, y, f32, stream=s),
            "linear": lambda: eo.q8_linear(x, f32, 300, 256, w, ws, 4096, y, f32, work, stream=s)}


@pytest.mark.parametrize("which", ["status", "norm", "route", "lists", "quantise", "dot", "tiles", "pairs", "fused",
                                   "linear"])
def test_a_failed_call_leaves_no_error(eo, which):
    cuda = ctypes.CDLL("libcuda.so.1")
    good = _good_calls(eo)
    for f in good:
        f()
    s = torch.cuda.Stream()
    bad = _bad_calls(eo, s)
    torch.cuda.synchronize()
    for f in good:
        handle, graph = ctypes.c_void_p(s.cuda_stream), ctypes.c_void_p()
        assert cuda.cuStreamBeginCapture_v2(handle, THREAD_LOCAL) == 0
        try:
            assert cuda.cuStreamSynchronize(handle) != 0     # not while capturing: the capture ends here
            with pytest.raises(eo.HfqError) as e:
                bad[which]()
            assert e.value.status == -5                      # HFQ_ERR_CUDA
        finally:
            assert cuda.cuStreamEndCapture(handle, ctypes.byref(graph)) != 0
        f()
    torch.cuda.synchronize()
    bad[which]()                                             # the stream is as it was
    torch.cuda.synchronize()
