"""moe_route_scored on the GPU against the fp64 oracle: the selection exactly,
the weights within the error of their f32 arithmetic, the lists exactly.

Weight bound: a renormalised weight is v_j / sum v with v = exp(d) (times a
sigmoid factor), d = l_j - max.  Rounding d costs |d| 2^-24 relative, expf 2 ulp
(4 * 2^-24), the sigmoid factor 4 + 1 + 2, the quotient and the scale 2 each,
the sum of k <= 16 positive terms 4 additions plus the terms' own errors; with
u = 2^-24 that is under 2 (|d|max + 24) u.
"""
import numpy as np
import pytest

from oracle import route, scored
from tests.test_gpu_parity import eo  # noqa: F401  (fixture: the built library)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
GUARD = -7


def _run(eo, logits, k, rule, bias=None, lists=False, ld=0, stream=None):
    T, E = logits.shape[0], rule.pop("E", logits.shape[1])
    r = eo.RouteRule(**rule)
    idx = torch.full((T * k + 8,), GUARD, dtype=torch.int32, device="cuda")
    wts = torch.full((T * k + 8,), float(GUARD), dtype=torch.float32, device="cuda")
    kw = {}
    if lists:
        kw = {n: torch.full((m + 8,), GUARD, dtype=torch.int32, device="cuda")
              for n, m in (("cnt", E), ("off", E + 1), ("perm", T * k))}
        kw["workspace"] = torch.full((max(16, eo.moe_route_scored_workspace_bytes(T, E, k)),), 0xA5,
                                     dtype=torch.uint8, device="cuda")
    dt = eo.HFQ_BF16 if logits.dtype == torch.bfloat16 else eo.HFQ_F32
    eo.moe_route_scored(logits, dt, T, E, k, r, idx, wts, bias=bias, ld=ld, stream=stream, **kw)
    torch.cuda.synchronize()
    for t in [idx, wts] + [kw[n] for n in ("cnt", "off", "perm") if lists]:
        assert (t[-8:] == GUARD).all()
    out = [idx[:-8].view(T, k).cpu().numpy(), wts[:-8].view(T, k).cpu().numpy()]
    return out + [kw[n][:-8].cpu().numpy() for n in ("cnt", "off", "perm") if lists]


def _check(eo, logits, k, rule, bias=None, lists=False, ld=0):
    E = rule.get("E", logits.shape[1])
    got = _run(eo, logits, k, dict(rule), bias, lists, ld)
    l = logits[:, :E].float().cpu().numpy()
    b = None if bias is None else bias.cpu().numpy()
    kw = {("sigmoid" if n == "score" else n): (v == eo.SCORE_SIGMOID if n == "score" else v)
          for n, v in rule.items() if n != "E"}
    idx, w = scored.route(l, k, bias=b, **kw)
    np.testing.assert_array_equal(got[0], idx)
    d = np.where(np.isfinite(l), np.abs(l.astype(np.float64)), 0).max(1, keepdims=True) * 2
    tol = 2 * (d + 24) * 2.0 ** -24
    if not rule.get("renormalise", True):
        tol = tol + E * 2.0 ** -24                       # the sum over all experts
    assert np.all(np.abs(got[1] - w) <= tol * np.abs(w) + 1e-37)
    if lists:
        cnt, off, perm = route.group_by_expert(idx, E)
        np.testing.assert_array_equal(got[2], cnt)
        np.testing.assert_array_equal(got[3], off)
        np.testing.assert_array_equal(got[4], perm)
    return got


def _rand(T, E, seed, dtype=torch.float32, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(T, E, generator=g, device="cuda") * std).to(dtype)


def _bias(E, seed, std):
    return _rand(1, E, seed, std=std)[0]


@pytest.mark.parametrize("T", [1, 2, 5, 31, 33, 200])
@pytest.mark.parametrize("E,k,n,tg,gt", [(256, 8, 8, 4, 2), (512, 8, 1, 1, 1), (160, 6, 8, 3, 1), (16, 4, 4, 2, 2),
                                         (1, 1, 1, 1, 1), (33, 16, 1, 1, 1), (510, 5, 17, 9, 2), (510, 7, 3, 2, 2),
                                         (64, 3, 32, 5, 2), (512, 16, 32, 1, 1), (9, 9, 1, 1, 1)])
@pytest.mark.parametrize("score", [0, 1], ids=["softmax", "sigmoid"])
def test_routing_against_the_oracle(eo, T, E, k, n, tg, gt, score):
    rule = dict(score=score, n_groups=n, topk_groups=tg, group_top=gt)
    seed = T * 1000 + E
    for bias in (None, _bias(E, seed + 1, 0.1 if score else 0.5 / E)):
        _check(eo, _rand(T, E, seed), k, dict(rule, renormalise=True, scale=2.5), bias, lists=T > 2)
        _check(eo, _rand(T, E, seed + 2, torch.bfloat16, 2.0), k, dict(rule, renormalise=False, scale=1.0), bias,
               lists=T % 2 == 1)


@pytest.mark.parametrize("T,E,k", [(1500, 512, 8), (4097, 256, 16), (3000, 64, 3), (2, 512, 1)])
def test_lists_of_large_batches(eo, T, E, k):
    l = _rand(T, E, T, std=3.0)
    l[:, 3] += 6.0                                       # one expert that most tokens choose
    _check(eo, l, k, dict(score=0, renormalise=True), lists=True)


def test_rows_further_apart_and_unaligned(eo):
    base = _rand(40, 300, 5)
    view = base[:, 3:3 + 200]                            # row stride 300, 12 bytes off a 16-byte address
    _check(eo, view, 7, dict(score=1, n_groups=4, topk_groups=2, group_top=2, E=200), ld=300)
    half = base.to(torch.bfloat16)[:, 1:]
    _check(eo, half, 7, dict(score=0, E=200), ld=300, bias=_bias(200, 6, 0.01))


def test_equal_scores_go_to_the_lower_expert(eo):
    for score in (0, 1):
        _check(eo, torch.zeros(6, 256, device="cuda"), 8, dict(score=score, n_groups=8, topk_groups=4, group_top=2),
               lists=True)
        _check(eo, torch.zeros(6, 256, device="cuda"), 8, dict(score=score), bias=torch.zeros(256, device="cuda"))
        # few distinct values, so that ties are everywhere
        l = torch.round(_rand(50, 96, 8, std=1.0))
        _check(eo, l, 16, dict(score=score, n_groups=6, topk_groups=3, group_top=2), lists=True)
        _check(eo, l, 16, dict(score=score, n_groups=6, topk_groups=3, group_top=1),
               bias=torch.round(_bias(96, 9, 2.0)) / 4)
    z = torch.zeros(3, 64, device="cuda")
    z[:, ::2] = -0.0                                     # the two zeros are equal
    _check(eo, z, 5, dict(score=0))


@pytest.mark.parametrize("score", [0, 1], ids=["softmax", "sigmoid"])
def test_scores_closer_than_32_bits_tell_apart(eo, score):
    """Pairs of experts whose score plus bias differ by 1e-9 and less: f32
    cannot order them, the definition does."""
    rng = np.random.default_rng(3)
    T, E = 64, 128
    l = rng.standard_normal((T, E)).astype(np.float32)
    l[1:] = l[0]                                         # one row of scores, ...
    p = 1 / (1 + np.exp(-l[0].astype(np.float64))) if score else np.exp(l[0].astype(np.float64)) / np.exp(l[0].astype(np.float64)).sum()
    bias = (0.75 - p).astype(np.float32)                 # ... all brought to 0.75 within f32 rounding
    c = p + bias.astype(np.float64)
    assert np.unique(c.astype(np.float32)).size < 16 and np.unique(c).size == E
    l[1:, :] += (rng.random((T - 1, E)) < 0.02).astype(np.float32) * 1e-6
    d = torch.from_numpy(l).cuda()
    b = torch.from_numpy(bias).cuda()
    _check(eo, d, 8, dict(score=score), bias=b)
    _check(eo, d, 8, dict(score=score, n_groups=8, topk_groups=3, group_top=2), bias=b)
    _check(eo, d, 5, dict(score=score, n_groups=8, topk_groups=3, group_top=1), bias=b)


@pytest.mark.parametrize("score", [0, 1], ids=["softmax", "sigmoid"])
def test_masked_experts(eo, score):
    E = 64
    l = _rand(12, E, 11)
    ninf, nan = float("-inf"), float("nan")
    l[0] = ninf                                          # nothing left
    l[1, 1:] = ninf                                      # one left
    l[2, ::3] = ninf
    l[3, 5:9] = nan
    l[4, 7] = float("inf")
    l[5, 3:5] = float("inf")
    l[6] = float(np.finfo(np.float32).min)               # the lowest finite value is no mask
    l[7, :60] = float(np.finfo(np.float32).min)
    l[8] = -200.0                                        # scores that underflow together
    l[9, :] = 60.0                                       # sigmoids that are all 1 in 64 bits
    l[9, 40] = 61.0
    l[10, 8:] = ninf                                     # only the first group is left
    for bias in (None, _bias(E, 12, 0.01)):
        for n, tg, gt in ((1, 1, 1), (8, 3, 2), (8, 3, 1)):
            rule = dict(score=score, n_groups=n, topk_groups=tg, group_top=gt)
            got = _check(eo, l, 8, rule, bias, lists=True)
            assert (got[1][0] == 0).all() and np.isfinite(got[1]).all()
            assert all(len(set(r)) == 8 for r in got[0].tolist())
            _check(eo, l, 8, dict(rule, renormalise=False), bias)
    b = _bias(E, 13, 0.01)
    b[2], b[9], b[30] = ninf, nan, float("inf")
    _check(eo, l, 8, dict(score=score, n_groups=8, topk_groups=3, group_top=2), b)


def test_bf16_masks_and_every_finite_bf16(eo):
    """All finite bf16 values appear as logits somewhere."""
    bits = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).cuda()
    l = bits.view(128, 512)
    for score in (0, 1):
        _check(eo, l, 8, dict(score=score))


def test_same_bits_every_time_and_on_another_stream(eo):
    l = _rand(700, 256, 21)
    b = _bias(256, 22, 0.1)
    rule = dict(score=1, n_groups=8, topk_groups=4, group_top=2)
    a = _run(eo, l, 8, dict(rule), b, lists=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c = _run(eo, l, 8, dict(rule), b, lists=True, stream=s)
    with torch.cuda.stream(s):
        d = _run(eo, l, 8, dict(rule), b, lists=True)
    for x, y, z in zip(a, c, d):
        assert x.tobytes() == y.tobytes() == z.tobytes()


def test_captured_and_replayed_with_a_shared_workspace(eo):
    """Two captured calls of different sizes on one workspace, replayed in turn
    over new logits."""
    E, k = 256, 8
    ls = [_rand(T, E, T) for T in (900, 70)]
    r = eo.RouteRule(score=1, n_groups=8, topk_groups=4, group_top=2)
    b = _bias(E, 2, 0.1)
    ws = torch.full((eo.moe_route_scored_workspace_bytes(900, E, k),), 0x5A, dtype=torch.uint8, device="cuda")
    outs, graphs = [], []
    for l in ls:
        T = l.shape[0]
        o = [torch.zeros(m, dtype=dt, device="cuda") for m, dt in
             ((T * k, torch.int32), (T * k, torch.float32), (E, torch.int32), (E + 1, torch.int32), (T * k, torch.int32))]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            eo.moe_route_scored(l, eo.HFQ_F32, T, E, k, r, o[0], o[1], bias=b, cnt=o[2], off=o[3], perm=o[4],
                                workspace=ws)
        outs.append(o)
        graphs.append(g)
    for seed in range(3):
        for l in ls:
            l.copy_(_rand(l.shape[0], E, 100 + seed))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for l, o in zip(ls, outs):
            idx, _ = scored.route(l.cpu().numpy(), k, sigmoid=True, bias=b.cpu().numpy(), n_groups=8, topk_groups=4,
                                  group_top=2)
            np.testing.assert_array_equal(o[0].view(-1, k).cpu().numpy(), idx)
            for t, v in zip(o[2:], route.group_by_expert(idx, E)):
                np.testing.assert_array_equal(t.cpu().numpy(), v)


@pytest.mark.parametrize("T", [1, 16, 17, 70])
@pytest.mark.parametrize("score", [0, 1], ids=["softmax", "sigmoid"])
def test_groups_closer_than_32_bits_tell_apart(eo, T, score):
    """Sums of a group's two best that differ by less than an f32 step, through
    the bias; ordinary members below them."""
    rng = np.random.default_rng(T + score)
    E, n = 256, 8
    l = rng.standard_normal((1, E)).astype(np.float32).repeat(T, 0)
    x = l[0].astype(np.float64)
    p = 1 / (1 + np.exp(-x)) if score else np.exp(x - x.max()) / np.exp(x - x.max()).sum()
    bias = np.zeros(E, np.float32)
    for g in range(n):                                   # two members each near 2, the sum within f32 rounding of 4
        for j, target in ((3, 2.0), (9, 2.0)):
            bias[g * 32 + j] = np.float32(target - p[g * 32 + j])
    _check(eo, torch.from_numpy(l).cuda(), 8, dict(score=score, n_groups=n, topk_groups=4, group_top=2),
           bias=torch.from_numpy(bias).cuda(), lists=True)
    _check(eo, torch.from_numpy(l).cuda(), 3, dict(score=score, n_groups=n, topk_groups=2, group_top=1),
           bias=torch.from_numpy(bias).cuda(), lists=True)


@pytest.mark.parametrize("T,E,k", [(5000, 300, 5), (9000, 512, 8), (16384, 64, 2), (16385, 33, 4), (65536, 16, 1)])
def test_lists_of_every_chunk_size(eo, T, E, k):
    """Chunks of 16, 32 and 64 tokens, counts added up by the placing blocks and by a kernel between."""
    l = _rand(T, E, T + 1, std=2.0)
    got = _run(eo, l, k, dict(score=0), lists=True)
    idx = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :k].int().cpu().numpy()
    np.testing.assert_array_equal(got[0], idx)
    flat = idx.reshape(-1).astype(np.int64)
    cnt = np.bincount(flat, minlength=E)
    np.testing.assert_array_equal(got[2], cnt)
    np.testing.assert_array_equal(got[3], np.concatenate([[0], np.cumsum(cnt)]))
    np.testing.assert_array_equal(got[4], np.argsort(flat, kind="stable"))


@pytest.mark.parametrize("score", [0, 1], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("E,n", [(8, 2), (16, 4), (24, 3), (64, 8), (256, 8), (510, 17)])
def test_biases_of_the_ends_of_the_range(eo, score, E, n):
    """Biases of f32's lowest and largest values and of +inf: two of them add up
    to an infinity in 32 bits, and infinities have no distance."""
    size, big, inf = E // n, float(np.finfo(np.float32).max), float("inf")
    l = _rand(9, E, E + n)
    l[5, : E // 2] = -inf
    rng = np.random.default_rng(E)
    for gt in (1, 2):
        for tg in {1, n // 2, n - 1}:
            rule = dict(score=score, n_groups=n, topk_groups=tg, group_top=gt)
            for values in ([-big], [-big, -inf], [big], [inf], [big, inf], [-big, 0.0], [inf, 0.0], [-big, big, -inf],
                           [-big, inf, 0.25, -inf]):
                each = torch.from_numpy(rng.choice(np.float32(values), E)).cuda()
                lead = torch.full((E,), values[0], device="cuda")
                lead[:size] = values[-1]                 # the first group unlike the others
                last = lead.flip(0)
                for bias in (each, lead, last):
                    _check(eo, l, min(3, tg * size), rule, bias=bias)
                    # every bias of a group one value, of the groups in turn
                by_group = torch.tensor(values, device="cuda")[torch.arange(E, device="cuda") // size % len(values)]
                _check(eo, l, min(3, tg * size), rule, bias=by_group)
