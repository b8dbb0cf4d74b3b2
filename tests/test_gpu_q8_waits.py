"""Waits of the 8-bit products that run out while copies are on their way.

With the shortest deadline (1 us) and an arrival that never comes, a kernel
gives up while its first tiles are still being copied into shared memory, and
in a CTA pair or a cluster each CTA at another time.  It has to wait for what
is in flight before it leaves: the status says that a wait ran out, and what
runs next (other kernels on the same shared memory, the same product with the
ordinary deadline) is right.
"""
import pytest

from tests.test_gpu_parity import eo  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("T,K,N", [(40, 8192, 300), (300, 200, 3000), (5, 4096, 1024), (8, 2048, 8192),
                                   (2048, 512, 3000), (1024, 8192, 4096), (4096, 4096, 4096)],
                         ids=["cluster", "tiles", "fused-cluster", "fused", "pairs", "pairs-long", "pairs-many"])
def test_a_deadline_that_passes_while_copies_are_in_flight(eo, T, K, N):
    g = torch.Generator(device="cuda").manual_seed(T + N)
    k16 = -(-K // 16) * 16
    x = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    w = torch.randint(-127, 128, (N, k16), generator=g, device="cuda").to(torch.int8)
    ws = torch.rand(N, generator=g, device="cuda")
    y = torch.empty(T, N, device="cuda")
    work = torch.zeros(eo.q8_linear_workspace_bytes(T, K, N) or 1, dtype=torch.uint8, device="cuda")

    def call():
        eo.q8_linear(x, eo.HFQ_BF16, T, K, w, ws, N, y, eo.HFQ_F32, work)

    call()
    torch.cuda.synchronize()
    eo.hfq_workspace_status(None)
    want = y.clone()
    try:
        for _ in range(5):
            eo.hfq_set_option(eo.OPT_WAIT_TIMEOUT_NS, 1000)
            eo.hfq_set_option(eo.OPT_TEST_MISSING_ARRIVALS, 1)
            call()
            with pytest.raises(eo.HfqError) as e:
                eo.hfq_workspace_status(None)
            assert e.value.status == -6
            eo.hfq_set_option(eo.OPT_WAIT_TIMEOUT_NS, 1_000_000_000)
            y.fill_(7.0)
            call()
            eo.hfq_workspace_status(None)
            assert torch.equal(y, want)
    finally:
        eo.hfq_set_option(eo.OPT_WAIT_TIMEOUT_NS, 1_000_000_000)
        eo.hfq_set_option(eo.OPT_TEST_MISSING_ARRIVALS, 0)
