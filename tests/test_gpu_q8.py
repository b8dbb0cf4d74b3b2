"""8-bit products on the GPU against the oracle.

The quantised values and scales have to be the oracle's bit for bit, the
integer sums are exact, so an output is acc * xs * ws with the conversion of
acc and two products in f32 (3 u, u = 2^-24) and the rounding to its type
(half a step): |err| <= (3 u + half) |y|.
"""
import numpy as np
import pytest

from oracle import q8
from tests.test_gpu_parity import eo  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
U = 2.0 ** -24
HALF = {"f32": 0.0, "bf16": 2.0 ** -8}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _hfq(eo, k):
    return eo.HFQ_F32 if k == "f32" else eo.HFQ_BF16


def _r16(n):
    return -(-n // 16) * 16


def _randn(seed, *shape, dt="f32"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(DT[dt])


def _quantise(eo, x, rows, cols, kind, act=0, ldx=0, ldq=0):
    ld = ldq or _r16(cols)
    q = torch.full((rows * ld + 32,), 99, dtype=torch.int8, device="cuda")
    s = torch.full((rows + 4,), -3.0, dtype=torch.float32, device="cuda")
    eo.q8_quantize_rows(x, _hfq(eo, kind), rows, cols, q, s, act=act, ldx=ldx, ldq=ldq)
    torch.cuda.synchronize()
    assert (q[(rows - 1) * ld + _r16(cols):] == 99).all() and (s[rows:] == -3.0).all()
    buf = q[:rows * ld].view(rows, ld)
    assert (buf[:, cols:_r16(cols)] == 0).all() and (buf[:, _r16(cols):] == 99).all()
    return buf, s[:rows]


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 15), (2, 16), (5, 17), (1, 256), (7, 1000), (4, 2048), (3, 2001),
                                       (2, 8192), (2, 16384), (2, 16383), (700, 96), (65536, 3)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_quantiser_bits(eo, rows, cols, kind):
    x = _randn(rows + cols, rows, cols, dt=kind)
    q, s = _quantise(eo, x, rows, cols, kind)
    rq, rs = q8.quantise(x.float().cpu().numpy())
    np.testing.assert_array_equal(q[:, :cols].cpu().numpy(), rq)
    np.testing.assert_array_equal(s.cpu().numpy(), rs)


def test_quantiser_borders_and_ranges(eo):
    """Quotients on and next to a half, tiny and huge rows, zeros, infinities."""
    C = 512
    v = np.zeros((12, C), np.float32)
    v[0] = 0.5 * np.arange(C)                            # with amax 255.5: many ties and near ties
    v[1] = 0.5 * (np.arange(C) % 255)                    # amax 127: every odd one a tie
    for r, e in ((2, -149), (3, -140), (4, -126), (5, -118), (6, -117), (7, 100)):
        v[r] = np.ldexp(np.arange(C) - 200.0, e).astype(np.float32)
    v[8] = np.float32(3.4e38) * np.linspace(-1, 1, C).astype(np.float32)
    half = (np.arange(127) + np.float32(0.5)).astype(np.float32)
    v[9, :127], v[9, 127:254], v[9, 254:381] = half, np.nextafter(half, np.float32(0)), np.nextafter(half, np.float32(999))
    v[9, 400] = 127.0
    v[10, :127] = half * np.float32(1.7)
    v[10, 400] = np.float32(127.0) * np.float32(1.7)
    q, s = _quantise(eo, torch.from_numpy(v).cuda(), 12, C, "f32")
    rq, rs = q8.quantise(v, exact=True)
    np.testing.assert_array_equal(q[:, :C].cpu().numpy(), rq)
    np.testing.assert_array_equal(s.cpu().numpy(), rs)
    w = _randn(1, 6, 100)
    w[0], w[1, 3], w[2, 99], w[3, 0] = 0, float("nan"), float("inf"), float("-inf")
    q, s = _quantise(eo, w, 6, 100, "f32")
    assert (q[:4, :100] == 0).all() and s[0] == 0 and torch.isnan(s[1:4]).all() and (s[4:] > 0).all()


def test_every_bf16_quotient(eo):
    """Each significand of a row's largest value against each significand of a
    value, over the binary places in which a quotient of 1/2 or more can lie:
    all the quotients that bf16 rows have, exact halves among them."""
    sig = np.arange(128, 256, dtype=np.float64)
    v = np.concatenate([sig * 2.0 ** -d for d in range(11)])
    for e in (-7, 60):
        rows = np.zeros((128, len(v) + 1))
        for r, top in enumerate(sig):
            rows[r, 1:] = np.where(v <= top, v, 0) * np.where(np.arange(len(v)) % 2, 1, -1)
            rows[r, 0] = top
        x = torch.from_numpy(rows * 2.0 ** e).bfloat16().cuda()
        assert torch.equal(x.double().cpu(), torch.from_numpy(rows * 2.0 ** e))      # all of them bf16 values
        q, s = _quantise(eo, x, 128, rows.shape[1], "bf16")
        rq, rs = q8.quantise((rows * 2.0 ** e).astype(np.float32))
        np.testing.assert_array_equal(q[:, :rows.shape[1]].cpu().numpy(), rq)
        np.testing.assert_array_equal(s.cpu().numpy(), rs)
        y = torch.empty(128, 16, device="cuda")          # the fused quantisers' bits, a row at a time
        eye, one = torch.eye(16, 1424, dtype=torch.int8, device="cuda"), torch.ones(16, device="cuda")
        for cols in range(0, 1408, 352):
            part = torch.cat([x[:, :1], x[:, 1 + cols:1 + cols + 15]], 1).contiguous()
            for r in range(0, 128, 5):
                n = min(5, 128 - r)
                eo.q8_linear(part[r:r + n], eo.HFQ_BF16, n, 16, eye, one, 16, y[r:r + n], eo.HFQ_F32,
                             torch.zeros(1 << 16, dtype=torch.uint8, device="cuda"), ldw=1424)
            pq, ps = q8.quantise(part.float().cpu().numpy())
            torch.cuda.synchronize()
            np.testing.assert_array_equal(y.cpu().numpy(), pq.astype(np.float32) * ps[:, None])


@pytest.mark.parametrize("rows,cols,ldx,ldq,shift", [(4, 100, 103, 128, 1), (4, 64, 72, 64, 0), (3, 4096, 4100, 4112, 3),
                                                     (2, 2048, 2049, 2048, 0)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_quantiser_strides(eo, rows, cols, ldx, ldq, shift, kind):
    x = _randn(9, rows * ldx + shift, dt=kind)[shift:]
    q, s = _quantise(eo, x, rows, cols, kind, ldx=ldx, ldq=ldq)
    rq, rs = q8.quantise(x[:rows * ldx].view(rows, ldx)[:, :cols].float().cpu().numpy())
    np.testing.assert_array_equal(q[:, :cols].cpu().numpy(), rq)
    np.testing.assert_array_equal(s.cpu().numpy(), rs)


@pytest.mark.parametrize("rows,cols,ldx,shift", [(9, 512, 1030, 0), (7, 520, 1048, 8), (70, 4096, 8192, 1),
                                                 (3, 4097, 8200, 0), (2, 16383, 32766, 3), (600, 1, 2, 0)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_swiglu_quantiser_strides(eo, rows, cols, ldx, shift, kind):
    """The bytes do not hang on how a row lies: those of the same rows, dense and
    aligned where their length allows it."""
    base = _randn(rows + cols, rows * ldx + shift, dt=kind)[shift:]
    q, s = _quantise(eo, base, rows, cols, kind, act=eo.ACT_SWIGLU, ldx=ldx)
    dense = base[:rows * ldx].view(rows, ldx)[:, :2 * cols].contiguous()
    q2, s2 = _quantise(eo, dense, rows, cols, kind, act=eo.ACT_SWIGLU)
    assert torch.equal(q, q2) and torch.equal(s, s2)
    v = q8.swiglu(dense.float().cpu().numpy())
    assert np.all(np.abs(s.double().cpu().numpy() - np.abs(v).max(1) / 127) <= 11 * U * np.abs(v).max(1) / 127)


@pytest.mark.parametrize("rows,cols", [(1, 512), (5, 96), (3, 1001), (2, 16384)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_swiglu_quantiser(eo, rows, cols, kind):
    """v = silu(g) u in f32: expf 2 ulp, sum, quotient and product, 9 u of |v|."""
    x = _randn(rows, rows, 2 * cols, dt=kind) * 2
    q, s = _quantise(eo, x, rows, cols, kind, act=eo.ACT_SWIGLU)
    v = q8.swiglu(x.float().cpu().numpy())
    amax = np.abs(v).max(1, keepdims=True)
    sc = s.double().cpu().numpy()[:, None]
    assert np.all(np.abs(sc - amax / 127) <= 11 * U * amax / 127)
    got = q[:, :cols].double().cpu().numpy() * sc
    assert np.all(np.abs(got - v) <= 0.5 * sc * (1 + 1e-4) + 12 * U * np.abs(v))
    x[0, 0], x[0, cols] = -1e30 if kind == "f32" else -3e38, 1.0   # silu of a far negative value is 0, not NaN
    q, s = _quantise(eo, x, rows, cols, kind, act=eo.ACT_SWIGLU)
    assert torch.isfinite(s).all() and q[0, 0] == 0


def _weights(seed, N, K, ld, full=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.randint(-128 if full else -127, 128, (N, ld), generator=g, device="cuda").to(torch.int8)
    s = torch.rand(N, generator=g, device="cuda") * 0.01 + 1e-4
    return w, s                                          # bytes behind K hold anything


def _exact(q, s, w, ws, K):
    acc = q[:, :K].double() @ w[:, :K].double().t()      # whole numbers below 2^53: exact
    return (acc * s.double()[:, None] * ws.double()).cpu().numpy()


def _close(y, ref, kind):
    y = y.double().cpu().numpy()
    err = np.abs(y - ref)
    assert np.all(err <= (3.01 * U + HALF[kind]) * np.abs(ref) + 1e-44), float(np.max(err / (np.abs(ref) + 1e-44)))


def _both(eo, T, K, N, x="bf16", y="f32", ldw=0, ldy=0, ldx=0, shift=0, seed=0):
    """q8_linear against the oracle's values, and against the two calls bit for bit."""
    xv = _randn(seed + T, T * (ldx or K) + shift, dt=x)[shift:]
    w, ws = _weights(seed + N, N, K, ldw or _r16(K))
    out = torch.full((T * (ldy or N) + 16 + shift,), 555.0, dtype=DT[y], device="cuda")[shift:]
    work = torch.full((eo.q8_linear_workspace_bytes(T, K, N) or 1,), 0xA5, dtype=torch.uint8, device="cuda")
    eo.q8_linear(xv, _hfq(eo, x), T, K, w, ws, N, out, _hfq(eo, y), work, ldx=ldx, ldw=ldw, ldy=ldy)
    torch.cuda.synchronize()
    rows = out[:T * (ldy or N)].view(T, -1)
    filler = torch.tensor(555.0).to(DT[y]).item()
    assert (out[T * (ldy or N):] == filler).all() and (rows[:, N:] == filler).all()
    v = xv[:T * (ldx or K)].view(T, -1)[:, :K].float()
    amax = v.abs().amax(1, keepdim=True).double()
    q = torch.where(amax > 0, torch.round(v.double() * 127 / amax), 0.0)
    ref = _exact(q, (amax[:, 0] / 127).float(), w, ws, K)
    _close(rows[:, :N], ref, y)
    bq = torch.zeros(T, _r16(K), dtype=torch.int8, device="cuda")
    bs = torch.zeros(T, dtype=torch.float32, device="cuda")
    eo.q8_quantize_rows(xv, _hfq(eo, x), T, K, bq, bs, ldx=ldx)
    out2 = torch.full((T, N), 555.0, dtype=DT[y], device="cuda")
    eo.q8_matmul(bq, bs, T, K, w, ws, N, out2, _hfq(eo, y), ldw=ldw)
    torch.cuda.synchronize()
    assert torch.equal(out2, rows[:, :N])


@pytest.mark.parametrize("T", [1, 2, 5, 8, 9, 16, 17, 31, 33, 64, 65, 127, 129, 200, 257, 300])
@pytest.mark.parametrize("K,N", [(2048, 1024), (512, 2048), (256, 256), (2001, 1503), (1, 1), (17, 129), (130, 64)])
def test_linear(eo, T, K, N):
    _both(eo, T, K, N)


@pytest.mark.parametrize("T,K,N", [(1, 16384, 300), (3, 8192, 1000), (70, 16383, 130), (513, 2048, 2048),
                                   (1000, 640, 4096), (2048, 512, 3000), (1100, 1111, 1111), (600, 16384, 256),
                                   (65536, 64, 40), (4, 128, 65536), (1, 128, 65536), (300, 100, 20000)])
@pytest.mark.parametrize("x,y", [("bf16", "bf16"), ("f32", "f32")])
def test_linear_large(eo, T, K, N, x, y):
    _both(eo, T, K, N, x, y)


@pytest.mark.parametrize("T,K,N", [(1, 8192, 100), (1, 8193, 100), (2, 2048, 900), (2, 2049, 900), (8, 4096, 500),
                                   (8, 4097, 500), (5, 8192, 2048), (8, 16384, 130), (33, 2048, 1024),
                                   (33, 2049, 1024), (290, 1030, 1000), (600, 2048, 333), (1100, 300, 260)])
@pytest.mark.parametrize("x,y", [("bf16", "f32"), ("f32", "bf16")])
def test_linear_where_the_kernels_meet(eo, T, K, N, x, y):
    _both(eo, T, K, N, x, y)


@pytest.mark.parametrize("T", [1, 7, 40, 150, 700])
@pytest.mark.parametrize("K,N,ldx,ldw,ldy,shift", [(300, 200, 301, 320, 203, 1), (512, 384, 520, 1024, 400, 0),
                                                   (1000, 1001, 1000, 1008, 1001, 3), (64, 8, 64, 64, 8, 4)])
@pytest.mark.parametrize("x,y", [("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
def test_strides_and_alignment(eo, T, K, N, ldx, ldw, ldy, shift, x, y):
    _both(eo, T, K, N, x, y, ldw=ldw, ldy=ldy, ldx=ldx, shift=shift)


@pytest.mark.parametrize("T", [1, 6, 50, 600])
def test_extreme_integers_and_garbage_tails(eo, T):
    """All of -128 .. 127 on both sides, sums up to 2^28, anything behind K."""
    K, N = 16380, 260
    xq = torch.full((T, 16384), -128, dtype=torch.int8, device="cuda")
    w = torch.full((N, 16400), -128, dtype=torch.int8, device="cuda")
    w[1::2] = 127
    xq[T // 2:, ::3] = 127
    xs, ws = torch.rand(T, device="cuda") + 0.5, torch.rand(N, device="cuda") + 0.5
    y = torch.empty(T, N, device="cuda")
    eo.q8_matmul(xq, xs, T, K, w, ws, N, y, eo.HFQ_F32, ldw=16400)
    torch.cuda.synchronize()
    _close(y, _exact(xq, xs, w, ws, K), "f32")
    xq2, ws2 = _weights(3, T, K, 16384, full=True)
    eo.q8_matmul(xq2, xs, T, K, w, ws, N, y, eo.HFQ_F32, ldw=16400)
    torch.cuda.synchronize()
    _close(y, _exact(xq2, xs, w, ws, K), "f32")


@pytest.mark.parametrize("T", [3, 100, 500])
def test_zero_and_unfinite_tokens(eo, T):
    K, N = 300, 200
    x = _randn(1, T, K)
    x[0] = 0
    x[1, 7] = float("inf")
    x[2, 8] = float("nan")
    w, ws = _weights(2, N, K, _r16(K))
    y = torch.empty(T, N, device="cuda")
    work = torch.zeros(eo.q8_linear_workspace_bytes(T, K, N) or 1, dtype=torch.uint8, device="cuda")
    eo.q8_linear(x, eo.HFQ_F32, T, K, w, ws, N, y, eo.HFQ_F32, work)
    torch.cuda.synchronize()
    assert (y[0] == 0).all() and torch.isnan(y[1:3]).all() and torch.isfinite(y[3:]).all()


@pytest.mark.parametrize("T", [2, 48, 400])
def test_captured_another_stream_and_twice_the_same_bits(eo, T):
    K, N = 1024, 768
    x = _randn(5, T, K, dt="bf16")
    w, ws = _weights(6, N, K, K)
    work = torch.full((eo.q8_linear_workspace_bytes(T, K, N) or 1,), 0x77, dtype=torch.uint8, device="cuda")
    ys = [torch.zeros(T, N, dtype=torch.bfloat16, device="cuda") for _ in range(3)]

    def call(y, stream=None):
        eo.q8_linear(x, eo.HFQ_BF16, T, K, w, ws, N, y, eo.HFQ_BF16, work, stream=stream)

    call(ys[0])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call(ys[1], s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(ys[2])
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])
    x.copy_(_randn(77, T, K, dt="bf16"))
    g.replay()
    call(ys[0])
    torch.cuda.synchronize()
    assert torch.equal(ys[0], ys[2]) and not torch.equal(ys[0], ys[1])


def test_products_on_two_streams_at_once(eo):
    """CTA pairs, which take all of an SM's tensor memory, beside clusters that
    split K, and the other kernels beside both: each stream's results are those
    that it has alone."""
    shapes = [[(1024, 512, 4096), (1024, 2048, 4096)], [(16, 2048, 1024), (40, 1024, 2048), (5, 2048, 1024)],
              [(300, 128, 3000), (2, 1024, 1024)]]
    streams = [torch.cuda.Stream() for _ in shapes]
    calls, alone = [], []
    for i, group in enumerate(shapes):
        mine = []
        for T, K, N in group:
            x = _randn(T + i, T, K, dt="bf16")
            w, ws = _weights(N + i, N, K, K)
            work = torch.zeros(eo.q8_linear_workspace_bytes(T, K, N) or 1, dtype=torch.uint8, device="cuda")
            mine.append((x, T, K, w, ws, N, torch.zeros(T, N, device="cuda"), work))
        calls.append(mine)

    def run(c, stream):
        x, T, K, w, ws, N, y, work = c
        eo.q8_linear(x, eo.HFQ_BF16, T, K, w, ws, N, y, eo.HFQ_F32, work, stream=stream)

    for mine in calls:
        for c in mine:
            run(c, None)
    torch.cuda.synchronize()
    alone = [[c[6].clone() for c in mine] for mine in calls]
    for mine in calls:
        for c in mine:
            c[6].zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for mine, s in zip(calls, streams):
            for c in mine:
                run(c, s)
    torch.cuda.synchronize()
    eo.hfq_workspace_status(None)
    for mine, want in zip(calls, alone):
        for c, y in zip(mine, want):
            assert torch.equal(c[6], y)


def test_offsets_past_32_bits(eo):
    """An output of more than 2^32 bytes: its last rows and channels."""
    T, K, N = 40000, 32, 65536
    x = _randn(5, T, K, dt="bf16")
    w, ws = _weights(6, N, K, K)
    y = torch.zeros(T, N, dtype=torch.bfloat16, device="cuda")
    work = torch.zeros(eo.q8_linear_workspace_bytes(T, K, N), dtype=torch.uint8, device="cuda")
    eo.q8_linear(x, eo.HFQ_BF16, T, K, w, ws, N, y, eo.HFQ_BF16, work)
    torch.cuda.synchronize()
    q, s = q8.quantise(x.float().cpu().numpy())
    q, s = torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda()
    for a, b in ((0, 300), (T - 300, T)):
        _close(y[a:b], _exact(q[a:b], s[a:b], w, ws, K), "bf16")


def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(eo):
    """The test hook makes the tensor-core kernel wait for an arrival that never
    comes; the wait is bounded, the status says so once."""
    eo.hfq_set_option(eo.OPT_WAIT_TIMEOUT_NS, 2_000_000)
    try:
        for T, K, N in ((40, 1024, 300), (40, 128, 300), (5, 1024, 300), (1024, 256, 4096)):
            # a cluster, one CTA alone, the fused kernel, CTA pairs
            x = torch.randint(-9, 10, (T, K), device="cuda").float()
            x[:, 0] = 127.0                              # scale 1: the values are the integers
            q, one = x.to(torch.int8), torch.ones(T, device="cuda")
            w, ws = _weights(1, N, K, K)
            y = torch.empty(T, N, device="cuda")
            work = torch.zeros(eo.q8_linear_workspace_bytes(T, K, N) or 1, dtype=torch.uint8, device="cuda")

            def call():
                eo.q8_linear(x, eo.HFQ_F32, T, K, w, ws, N, y, eo.HFQ_F32, work)

            eo.hfq_set_option(eo.OPT_TEST_MISSING_ARRIVALS, 1)
            call()
            with pytest.raises(eo.HfqError) as e:
                eo.hfq_workspace_status(None)
            assert e.value.status == -6
            eo.hfq_workspace_status(None)
            call()
            eo.hfq_workspace_status(None)
            _close(y, _exact(q, one, w, ws, K), "f32")
    finally:
        eo.hfq_set_option(eo.OPT_WAIT_TIMEOUT_NS, 1_000_000_000)
        eo.hfq_set_option(eo.OPT_TEST_MISSING_ARRIVALS, 0)
