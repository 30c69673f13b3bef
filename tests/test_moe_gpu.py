"""The operators around the experts' products on the GPU, against the float64
oracle: routing and its gradient, the experts' rows, dispatch, the quantiser
with fp32 scales, combine and its gradients.

Tolerances count the kernels' roundings. u = 2^-24 is half a step of fp32
relative to the value, 2^-8 of bf16. expf is within 2 ulp = 4 u of the true
value (CUDA's documentation), each other fp32 operation within u."""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_tcgen05_b200 as dg
from oracle import moe as om

from helpers import fill_sentinel, is_sentinel
from test_capture_gpu import eager_equals_replay

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16 = 2.0 ** -8


@pytest.fixture(autouse=True)
def _init():
    dg.init()
    yield
    assert dg.device_error(clear=True) == 0


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def weight_bound(logits, k, score):
    """Relative error of a weight: the score's exponential (4 u, and for softmax
    the rounding of x - max, |x - max| u in the exponent), the sums over at most
    E or k scores (their terms' errors, and one u per level of the tree: 5 for a
    warp, E/32 for a lane's part), three quotients or products; doubled for the
    quotient of two such values."""
    x = np.asarray(logits, np.float64)
    finite = x[np.isfinite(x)]
    spread = 0.0 if score == "sigmoid" or finite.size == 0 else finite.max() - finite.min()
    return 2 * (4 + spread + 5 + x.shape[1] / 32 + 4) * U


ROUTE = [  # T, E, k, score, bias, groups, top_groups, group_top, renorm, bf16
    (1, 1, 1, "softmax", False, 1, 1, 1, True, False),
    (5, 8, 2, "softmax", False, 1, 1, 1, True, True),
    (33, 20, 3, "sigmoid", True, 4, 2, 2, True, False),
    (64, 256, 8, "sigmoid", True, 8, 4, 2, True, False),
    (64, 256, 8, "sigmoid", False, 8, 4, 2, True, True),
    (40, 160, 6, "softmax", False, 8, 3, 1, False, False),
    (40, 160, 6, "softmax", True, 8, 3, 1, False, True),
    (17, 60, 4, "softmax", True, 4, 4, 1, True, False),
    (17, 60, 4, "softmax", True, 4, 1, 2, True, False),
    (9, 257, 8, "softmax", False, 1, 1, 2, True, False),
    (9, 384, 32, "sigmoid", True, 8, 5, 2, True, False),
    (6, 512, 16, "sigmoid", True, 32, 3, 2, False, True),
    (7, 1024, 32, "softmax", True, 32, 32, 1, True, False),
    (7, 1000, 8, "sigmoid", True, 4, 2, 2, True, False),
    (12, 32, 32, "sigmoid", True, 1, 1, 1, True, False),
    (12, 96, 5, "sigmoid", True, 32, 7, 2, True, False),
    (300, 192, 8, "sigmoid", True, 3, 2, 2, True, False),
]


def route_inputs(T, E, bias, bf16, seed):
    g = torch.Generator().manual_seed(seed)
    x = 2 * torch.randn((T, E), generator=g)
    x = x.to(torch.bfloat16) if bf16 else x
    return x, 0.1 * torch.randn((E,), generator=g) if bias else None


@pytest.mark.parametrize("case", ROUTE)
def test_route(case):
    T, E, k, score, bias, n, top, gt, renorm, bf16 = case
    x, b = route_inputs(T, E, bias, bf16, seed=E + T)
    ids, w = dg.moe_route(x.cuda(), k, bias=None if b is None else b.cuda(), score=score, n_groups=n, top_groups=top,
                          group_top=gt, renormalize=renorm, scale=2.5)
    ref_ids, ref_w = om.route(f64(x), k, None if b is None else f64(b), score, n, top, gt, renorm, 2.5)
    assert np.array_equal(ids.cpu().numpy(), ref_ids)
    assert np.all(np.abs(f64(w) - ref_w) <= weight_bound(f64(x), k, score) * np.abs(ref_w))


def test_route_ties_go_to_the_lowest_index():
    for E, k, n, top in ((64, 8, 1, 1), (64, 8, 8, 3), (60, 6, 4, 2)):
        x = torch.zeros((3, E))
        x[1, ::2] = 1.0
        x[2, 0], x[2, 1] = -0.0, 0.0
        for bias in (None, torch.zeros(E)):
            ids, w = dg.moe_route(x.cuda(), k, bias=None if bias is None else bias.cuda(), score="sigmoid", n_groups=n,
                                  top_groups=top)
            ref = om.route(f64(x), k, None if bias is None else f64(bias), "sigmoid", n, top)[0]
            assert np.array_equal(ids.cpu().numpy(), ref)


@pytest.mark.parametrize("n,top,gt", [(1, 1, 1), (8, 4, 2), (8, 4, 1)])
@pytest.mark.parametrize("E,tied", [(64, 64), (64, 2), (64, 5), (256, 3), (512, 4), (60, 2)])
def test_route_choices_closer_than_fp32(n, top, gt, E, tied):
    """Keys that differ by 2^-26 in runs of `tied` experts: the bias makes up all
    but that of the score's difference, so fp32 keys tie or swap, and the 64-bit
    order must come out."""
    if E % n:
        n, top = 4, 2
    T, k = 64, 8
    g = torch.Generator().manual_seed(5)
    x = torch.randn((T, E), generator=g).double()
    base = torch.sigmoid(x[0].float().double())
    step = torch.randperm(E, generator=g)
    want = 0.7 + 2.0 ** -26 * step.double() + 1e-3 * (step // tied).double()
    bias = (want - base).float()
    x = x[:1].float().expand(T, E).contiguous()
    x[1:] += 1e-7 * torch.randn((T - 1, E), generator=g)
    ids, _ = dg.moe_route(x.cuda(), k, bias=bias.cuda(), score="sigmoid", n_groups=n, top_groups=top, group_top=gt)
    assert np.array_equal(ids.cpu().numpy(), om.route(f64(x), k, f64(bias), "sigmoid", n, top, gt)[0])


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("size,gap", [(0.5, 1e-2), (64.0, 3e-5), (1000.0, 5e-4)])
@pytest.mark.parametrize("E,n,top", [(64, 8, 4), (256, 8, 3), (60, 4, 2), (512, 32, 7)])
def test_route_groups_whose_two_best_keys_cancel(E, n, top, size, gap, score):
    """Group scores are small sums of large keys of both signs: fp32 keys are off by
    more than the sums are apart, and the 64-bit order must come out."""
    T, k = 40, top   # the best key of every group that stays
    r = np.random.default_rng(E + n)
    per = E // n
    x = r.standard_normal(E).astype(np.float32)
    s64 = 1 / (1 + np.exp(-x.astype(np.float64)))
    if score == "softmax":
        s64 = np.exp(x.astype(np.float64)) / np.exp(x.astype(np.float64)).sum()
    bias = np.full(E, -3 * size, np.float32)
    want = 0.1 + gap * r.permutation(n)
    for g in range(n):
        i, j = g * per + r.permutation(per)[:2]
        bias[i] = size * (1 + r.random())
        bias[j] = want[g] - (s64[i] + np.float64(bias[i])) - s64[j]
    xs = np.repeat(x[None], T, 0)
    xs[1:] += (1e-7 * r.standard_normal((T - 1, E))).astype(np.float32)
    ids, _ = dg.moe_route(torch.from_numpy(xs).cuda(), k, bias=torch.from_numpy(bias).cuda(), score=score, n_groups=n,
                          top_groups=top, group_top=2)
    ref = om.route(xs.astype(np.float64), k, bias.astype(np.float64), score, n, top, 2)[0]
    assert np.array_equal(ids.cpu().numpy(), ref)


@pytest.mark.parametrize("E,n", [(32, 8), (60, 4)])
def test_route_groups_whose_sum_passes_the_largest_number(E, n):
    """Keys next to the type's lowest value: two of them have no fp32 sum, and their groups are still ranked."""
    r = np.random.default_rng(7)
    per = E // n
    x = r.standard_normal((6, E)).astype(np.float32)
    bias = (-3.0e38 - 5e35 * r.permutation(E)).astype(np.float32)
    bias[:per] = 0.1 * r.standard_normal(per)
    ids, _ = dg.moe_route(torch.from_numpy(x).cuda(), per + 3, bias=torch.from_numpy(bias).cuda(), score="sigmoid", n_groups=n,
                          top_groups=2, group_top=2)
    assert np.array_equal(ids.cpu().numpy(), om.route(x.astype(np.float64), per + 3, bias.astype(np.float64), "sigmoid", n, 2, 2)[0])


def test_route_rows_with_nothing_or_with_what_is_not_finite():
    inf, nan = float("inf"), float("nan")
    x = torch.full((6, 40), -inf)
    x[1, 7] = 1.0                      # one expert left
    x[2, 3], x[2, 5] = -1e30, 2.0
    x[3] = torch.arange(40).float()
    x[3, 39] = nan
    x[4] = torch.arange(40).float()
    x[4, 3] = inf
    x[5] = -200.0
    ids, w = dg.moe_route(x.cuda(), 4, score="softmax")
    ids, w = ids.cpu(), w.cpu()
    assert ids[0].tolist() == [0, 1, 2, 3] and w[0].tolist() == [0, 0, 0, 0]
    assert ids[1].tolist() == [7, 0, 1, 2] and w[1].tolist() == [1, 0, 0, 0]
    assert ids[2].tolist() == [5, 3, 0, 1] and w[2].tolist() == [1, 0, 0, 0]
    assert ids[3].tolist() == [38, 37, 36, 35] and torch.isnan(w[3]).all()
    assert ids[4].tolist() == [3, 39, 38, 37] and torch.isnan(w[4]).all()
    assert ids[5].tolist() == [0, 1, 2, 3] and torch.equal(w[5], torch.full((4,), 0.25))
    for bias in (None, torch.zeros(40)):
        b = None if bias is None else bias.cuda()
        i2, w2 = dg.moe_route(x.cuda(), 4, bias=b, score="sigmoid", n_groups=4, top_groups=2)
        i2, w2 = i2.cpu(), w2.cpu()
        assert all(len(set(r)) == 4 and 0 <= min(r) and max(r) < 40 for r in i2.tolist())
        assert w2[0].tolist() == [0, 0, 0, 0]
        assert torch.isfinite(w2[5]).all()
        assert not torch.isnan(w2[3]).any()   # the NaN expert ranks last and is not chosen


def lane_experts(E):
    """Experts of a lane: the smallest built number that holds E experts in 32 lanes."""
    return next(v for v in (1, 2, 3, 4, 5, 6, 8, 12, 16, 32) if 32 * v >= E)


def check_route_exactly(x, bias, k, score, n, top, gt):
    T, E = x.shape
    ids, w = dg.moe_route(x.cuda(), k, bias=None if bias is None else bias.cuda(), score=score, n_groups=n, top_groups=top,
                          group_top=gt)
    ref_ids, ref_w = om.route(f64(x), k, None if bias is None else f64(bias), score, n, top, gt)
    assert np.array_equal(ids.cpu().numpy(), ref_ids)
    there = ~np.isnan(ref_w)
    err = np.abs(f64(w) - ref_w)
    assert np.all(err[there] <= (weight_bound(f64(x), k, score) * np.abs(ref_w))[there])
    assert np.isnan(f64(w)[~there]).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("n,top,gt", [(8, 4, 2), (8, 4, 1)])
@pytest.mark.parametrize("E", [64, 96, 128, 160, 256, 512])
@pytest.mark.parametrize("kind", ["lane", "lane and a half", "every other lane", "all but one of a group", "group", "half"])
def test_route_groups_of_experts_taken_out_by_a_bias_of_minus_infinity(kind, E, n, top, gt, score):
    """Groups that are runs of lanes, with lanes that hold nothing but -inf beside others."""
    T, k, V, size = 200, 8, lane_experts(E), E // n
    g = torch.Generator().manual_seed(E + gt)
    x = 1.5 * torch.randn((T, E), generator=g)
    bias = 0.05 * torch.randn((E,), generator=g)
    out = torch.zeros(E, dtype=torch.bool)
    if kind == "lane":
        out[:V] = out[E // 2:E // 2 + V] = True
    elif kind == "lane and a half":
        out[:V + (V + 1) // 2] = out[5 * size:5 * size + V + (V + 1) // 2] = True
    elif kind == "every other lane":
        out[torch.arange(E) // V % 2 == 1] = True
    elif kind == "all but one of a group":
        out[size:2 * size] = out[3 * size:4 * size] = True
        out[size + 1] = out[4 * size - 1] = False
    elif kind == "group":
        out[2 * size:3 * size] = out[7 * size:] = True
    else:
        out[torch.randperm(E, generator=g)[:E // 2]] = True
    bias[out] = -np.inf
    check_route_exactly(x, bias, k, score, n, top, gt)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("n,top,gt", [(1, 1, 1), (8, 4, 2), (8, 4, 1)])
@pytest.mark.parametrize("E", [64, 128, 160, 256, 512])
def test_route_fewer_experts_than_choices_left_by_the_bias(E, n, top, gt, score):
    """Choices among equal infinite keys go to the lowest index, of both signs."""
    g = torch.Generator().manual_seed(E)
    x = torch.randn((40, E), generator=g)
    for alive in ([5], [3, 10], [0, E // 2, E - 1], list(range(7))):
        bias = torch.full((E,), -np.inf)
        bias[alive] = 0.0
        for k in (4, 8):
            check_route_exactly(x, bias, k, score, n, top, gt)
    for chosen in ([5, 9, 20], [E - 1, E // 2, 1], list(range(0, E, 5))):
        bias = 0.1 * torch.randn((E,), generator=g)
        bias[chosen] = np.inf
        for k in (2, 8):
            check_route_exactly(x, bias, k, score, n, top, gt)


def test_route_worked_examples_of_infinite_biases():
    bias = torch.full((256,), -np.inf)
    bias[5] = 0.0
    assert dg.moe_route(torch.zeros((1, 256)).cuda(), 4, bias=bias.cuda(), score="sigmoid")[0].tolist() == [[5, 0, 1, 2]]
    bias = torch.zeros(256)
    bias[[5, 9, 70]] = np.inf
    assert dg.moe_route(torch.zeros((1, 256)).cuda(), 2, bias=bias.cuda(), score="sigmoid")[0].tolist() == [[5, 9]]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("n,top,gt", [(1, 1, 1), (8, 4, 2), (8, 4, 1)])
@pytest.mark.parametrize("E", [40, 64, 160, 256])
def test_route_logits_that_are_not_finite_under_a_bias(E, n, top, gt, score):
    """A NaN logit takes its expert (softmax: its row) out, and so does -inf; a lane of them, a group, all."""
    V, size = lane_experts(E), E // 8
    g = torch.Generator().manual_seed(E)
    x = torch.randn((24, E), generator=g)
    bias = 0.1 * torch.randn((E,), generator=g)
    for t, value in enumerate([np.nan, -np.inf] * 6):
        x[2 * t, [slice(0, 1), slice(V, 2 * V), slice(0, V + 1), slice(size, 2 * size), slice(2, E), slice(0, E)][t // 2]] = value
    if score == "softmax":
        x[1, 7] = np.inf
    check_route_exactly(x, bias, 4, score, n, top, gt)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("n,top,gt", [(1, 1, 1), (8, 4, 2), (8, 4, 1)])
@pytest.mark.parametrize("E", [40, 64, 160, 256])
def test_route_logits_that_are_not_finite_without_a_bias(E, n, top, gt, score, bf16):
    """Lanes, a group and all but a few of the experts at NaN, -inf or +inf: exact ids."""
    V, size = lane_experts(E), E // 8
    g = torch.Generator().manual_seed(E + 1)
    x = torch.randn((18, E), generator=g)
    for t, value in enumerate([np.nan, -np.inf, np.inf] * 6):
        x[t, [slice(0, 1), slice(V, 2 * V), slice(0, V + 1), slice(size, 2 * size), slice(2, E), slice(0, E)][t // 3]] = value
    check_route_exactly(x.to(torch.bfloat16) if bf16 else x, None, 4, score, n, top, gt)


def test_route_many_tokens():
    """More tokens than warps at once, among them the choices that 16384 random
    tokens leave undecided in fp32."""
    T, E, k = 16384, 256, 8
    g = torch.Generator().manual_seed(77)
    x = 1.5 * torch.randn((T, E), generator=g)
    b = 0.05 * torch.randn((E,), generator=g)
    ids, w = dg.moe_route(x.cuda(), k, bias=b.cuda(), score="sigmoid", n_groups=8, top_groups=4)
    s = torch.sigmoid(x.double())
    key = s + b.double()
    best = key.view(T, 8, 32).sort(dim=2, descending=True).values[:, :, :2].sum(2)
    kept = best.sort(dim=1, descending=True, stable=True).indices[:, :4]
    mask = torch.zeros((T, 8), dtype=torch.bool).scatter_(1, kept, True).repeat_interleave(32, dim=1)
    want = key.masked_fill(~mask, -np.inf).sort(dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(ids.cpu().long(), want)
    ref = s.gather(1, want)
    ref = (ref / ref.sum(1, keepdim=True)).numpy()
    assert np.all(np.abs(f64(w) - ref) <= weight_bound(f64(x[:1]), k, "sigmoid") * ref)


@pytest.mark.parametrize("case", ROUTE)
def test_route_backward(case):
    T, E, k, score, bias, n, top, gt, renorm, bf16 = case
    x, b = route_inputs(T, E, bias, bf16, seed=E + 7 * T)
    ids = om.route(f64(x), k, None if b is None else f64(b), score, n, top, gt, renorm, 2.5)[0]
    g = torch.randn((T, k), generator=torch.Generator().manual_seed(3))
    d = dg.moe_route_backward(x.cuda(), torch.from_numpy(ids).cuda(), g.cuda(), score=score, renormalize=renorm,
                              scale=2.5)
    ref, mag = om.route_backward(f64(x), ids, f64(g), score, renorm, 2.5)
    assert d.dtype == x.dtype and d.shape == x.shape
    # every factor of a term carries a weight's error; the sum over k terms adds at most k u of their magnitudes
    bound = (3 * weight_bound(f64(x), k, score) + (k + 8) * U) * mag
    if bf16:
        bound = bound * (1 + BF16) + BF16 * np.abs(ref)
    err = np.abs(f64(d) - ref)
    assert np.all(err <= bound + 1e-38), (err - bound).max()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("gap", [4.0, 12.0, 16.0, 24.0])
@pytest.mark.parametrize("E,k,chosen", [(8, 2, None), (256, 8, None), (20, 3, [4, 4, -1]), (33, 4, [7, 32, 7, 0]), (7, 7, None)])
def test_softmax_gradient_of_a_peaked_row(E, k, chosen, gap, bf16):
    """Not renormalised, and one expert far above the rest: its gradient s (ds - sum ds s)
    is a small difference, which must keep its digits. The expert's slots have the
    largest gradients of their row and the others' are not negative, so that
        d = s (sum over the other chosen of s_l (D - D_l) + D (sum of s over those not chosen)),
    D the sum of an expert's slots, has no term below zero: the bound is relative to
    the gradient itself. Scores are within a weight's error, three of them meet in a
    term; D_l carry k u of their sum, at most D; the sums add E/32 + 5 + 2 k levels."""
    T = 16
    g = torch.Generator().manual_seed(E + int(gap))
    x = torch.rand((T, E), generator=g)
    ids = np.argsort(-f64(x), axis=1)[:, :k].astype(np.int32)
    if chosen is not None:
        ids[:] = chosen
    d = torch.rand((T, k), generator=g)
    for t in range(T):
        x[t, ids[t, 0]] += gap
        d[t] = torch.where(torch.from_numpy(ids[t] == ids[t, 0]), 3.0 + d[t], d[t] / k)
    x = x.to(torch.bfloat16) if bf16 else x
    got = f64(dg.moe_route_backward(x.cuda(), torch.from_numpy(ids).cuda(), d.cuda(), renormalize=False, scale=1.5))
    s, gr = om.scores(f64(x), "softmax"), f64(d)
    for t in range(T):
        D = np.zeros(E)
        for j in range(k):
            if ids[t, j] >= 0:
                D[ids[t, j]] += 1.5 * gr[t, j]
        rest = np.setdiff1d(np.arange(E), ids[t])
        e = ids[t, 0]
        want = s[t, e] * ((s[t] * (D[e] - D))[np.setdiff1d(np.arange(E), np.r_[rest, e])].sum() + D[e] * s[t, rest].sum())
        # (D - D_l >= D / 2: its error of (k + 2) u D is within 2 (k + 2) u of it)
        rel = 3 * weight_bound(f64(x[t:t + 1]), k, "softmax") + (2 * (k + 2) + E / 32 + 5 + 2 * k + 4) * U + (BF16 if bf16 else 0)
        assert abs(got[t, e] - want) <= rel * want * (1 + BF16), (t, got[t, e], want)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward_against_differences(score, renorm):
    """The kernel's gradient against central differences of the float64 forward:
    a step of 1e-4 leaves a truncation error of order 1e-8 (third derivatives of
    order one) and rounding of order 1e-11, far below fp32's own."""
    r = np.random.default_rng(4)
    x = r.standard_normal((6, 24)).astype(np.float32)
    g = r.standard_normal((6, 4)).astype(np.float32)
    ids = om.route(x, 4, score=score)[0]
    d = f64(dg.moe_route_backward(*(torch.from_numpy(v).cuda() for v in (x, ids, g)), score=score, renormalize=renorm))
    for e in range(24):
        step = np.zeros((1, 24))
        step[0, e] = 1e-4
        hi, lo = ((g * om.route_weights(x + s * step, ids, score, renorm)).sum(1) for s in (1, -1))
        assert np.all(np.abs((hi - lo) / 2e-4 - d[:, e]) <= 1e-7 + 200 * U * np.abs(g).sum(1))


def test_route_backward_with_other_ids():
    """Ids outside the experts count as not chosen; an expert named twice gets both gradients."""
    x = torch.randn((4, 10), generator=torch.Generator().manual_seed(8))
    ids = np.array([[3, 3, -1], [-1, -1, 10], [0, 9, 5], [2, 2, 2]], np.int32)
    g = torch.randn((4, 3), generator=torch.Generator().manual_seed(9))
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            d = f64(dg.moe_route_backward(x.cuda(), torch.from_numpy(ids).cuda(), g.cuda(), score=score,
                                          renormalize=renorm))
            ref, mag = om.route_backward(f64(x), ids, f64(g), score, renorm)
            assert np.all(np.abs(d - ref) <= (3 * weight_bound(f64(x), 3, score) + 11 * U) * mag + 1e-38)
            assert np.all(d[1] == 0)


# -------------------------------------------------------------------- rows ----

ROWS = [(1, 1, 1), (1, 8, 256), (3, 2, 2), (64, 8, 32), (511, 8, 256), (513, 8, 60), (1025, 5, 1024), (4096, 8, 8),
        (1000, 32, 1000)]


def choices(T, k, G, seed, stray=0.0, skew=False):
    r = np.random.default_rng(seed)
    ids = r.integers(0, G, (T, k)) if not skew else np.minimum(r.integers(0, G, (T, k)), r.integers(0, 2, (T, k)))
    ids[r.random((T, k)) < stray] = -1
    if stray:
        ids[r.random((T, k)) < stray / 2] = G
    return ids.astype(np.int32)


@pytest.mark.parametrize("T,k,G", ROWS)
@pytest.mark.parametrize("kind", ["even", "stray", "skewed", "none"])
def test_rows(T, k, G, kind):
    ids = choices(T, k, G, seed=T + k, stray={"stray": 0.3, "none": 1.1}.get(kind, 0.0), skew=kind == "skewed")
    dev = torch.from_numpy(ids).cuda()
    extra = 300
    m = torch.full((om.rows_bound(T, k, G) + extra,), 77, dtype=torch.int32, device="cuda")
    row_of, m_idx, counts = dg.moe_rows_contiguous(dev, G, m_indices=m)
    ref_row, ref_counts, first = om.expert_rows(ids, G)
    assert np.array_equal(row_of.cpu().numpy(), ref_row)
    assert np.array_equal(counts.cpu().numpy(), ref_counts)
    assert np.array_equal(m_idx.cpu().numpy(), om.m_indices(ref_counts, first, m.numel()))
    for max_m in (1, 7, T):
        row_of, masked_m, counts = dg.moe_rows_masked(dev, G, max_m)
        ref_row, ref_counts, _ = om.expert_rows(ids, G, max_m)
        assert np.array_equal(row_of.cpu().numpy(), ref_row)
        assert np.array_equal(counts.cpu().numpy(), ref_counts)
        assert np.array_equal(masked_m.cpu().numpy(), np.minimum(ref_counts, max_m))


@pytest.mark.parametrize("T,k,G", [(9001, 8, 256), (16411, 5, 3), (2100, 32, 1024), (4100, 1, 1)])
def test_rows_of_many_choices(T, k, G):
    """Several whole batches of a warp's steps and a rest; ids outside the experts share low bits with those inside."""
    r = np.random.default_rng(T)
    ids = r.integers(0, G, (T, k)).astype(np.int64)
    out = r.random((T, k)) < 0.1
    ids[out] += r.choice([G, 1024, 2048, 2 ** 30, -G, -(2 ** 31)], size=int(out.sum()))
    ids = ids.clip(-(2 ** 31), 2 ** 31 - 1).astype(np.int32)
    row_of, m_idx, counts = dg.moe_rows_contiguous(torch.from_numpy(ids).cuda(), G)
    ref_row, ref_counts, first = om.expert_rows(ids, G)
    assert np.array_equal(row_of.cpu().numpy(), ref_row)
    assert np.array_equal(counts.cpu().numpy(), ref_counts)
    assert np.array_equal(m_idx.cpu().numpy(), om.m_indices(ref_counts, first, m_idx.numel()))


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 31, 32, 33, 127, 128, 129, 1023])
def test_rows_around_powers_of_two_of_experts(G):
    ids = choices(700, 6, G, seed=G, stray=0.2)
    row_of, masked_m, counts = dg.moe_rows_masked(torch.from_numpy(ids).cuda(), G, 50)
    ref_row, ref_counts, _ = om.expert_rows(ids, G, 50)
    assert np.array_equal(row_of.cpu().numpy(), ref_row)
    assert np.array_equal(counts.cpu().numpy(), ref_counts)
    assert np.array_equal(masked_m.cpu().numpy(), np.minimum(ref_counts, 50))


@pytest.mark.parametrize("T,k,G", [(9001, 8, 256), (2100, 32, 1024), (700, 6, 33)])
def test_rows_on_a_device_without_a_place_for_16_ctas(T, k, G):
    """The hook stands in for the device: the largest cluster that fits takes the choices."""
    ids = choices(T, k, G, seed=G, stray=0.1)
    dev = torch.from_numpy(ids).cuda()
    want = dg.moe_rows_contiguous(dev, G)
    try:
        dg.set_test_hooks(2, 0)
        got = dg.moe_rows_contiguous(dev, G)
    finally:
        dg.set_test_hooks(0, 0)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    ref_row, ref_counts, first = om.expert_rows(ids, G)
    assert np.array_equal(got[0].cpu().numpy(), ref_row) and np.array_equal(got[2].cpu().numpy(), ref_counts)


# ---------------------------------------------------- dispatch and quantiser ----

def activations(T, H, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, H), generator=g) * torch.exp(3 * torch.randn((T, 1), generator=g))
    if T > 2:
        x[1] = 0
        x[2, :128] = 448.0 * 2.0 ** torch.randint(-3, 4, (1,), generator=g)
        x[2, 5] = 1e-7
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,k,G,H", [(1, 1, 1, 128), (3, 2, 4, 384), (130, 8, 16, 640), (65, 4, 8, 1024), (9, 32, 64, 7168)])
@pytest.mark.parametrize("packed", [True, False])
def test_dispatch(T, k, G, H, dtype, packed):
    x = activations(T, H, dtype, seed=T)
    ids = choices(T, k, G, seed=T + H, stray=0.2)
    row_of, m_idx, _ = dg.moe_rows_contiguous(torch.from_numpy(ids).cuda(), G)
    rows = m_idx.numel()
    q = torch.full((rows, H), 0xAB, dtype=torch.uint8, device="cuda")
    if packed:
        sf = torch.full((rows, (H // 128 + 3) // 4), -7, dtype=torch.int32, device="cuda")
    else:
        sf = torch.full((rows, H // 128), -7.0, device="cuda")
    dg.moe_dispatch_fp8(x.cuda(), row_of, q, sf)
    want = om.dispatch(x.float().numpy(), row_of.cpu().numpy(), rows, packed)
    q, sf = q.cpu().numpy(), sf.cpu().numpy()
    for r in range(rows):
        if r in want:
            assert np.array_equal(q[r], want[r][0]) and np.array_equal(sf[r], want[r][1])
        else:
            assert np.all(q[r] == 0xAB) and np.all(sf[r] == -7)


def test_dispatch_skips_rows_outside_the_buffer():
    x = activations(4, 256, torch.bfloat16, seed=1)
    buf = torch.full((12, 256), 0xAB, dtype=torch.uint8, device="cuda")
    sf = torch.full((12, 2), -7.0, device="cuda")
    row_of = torch.tensor([[0, -5], [4, 2], [3, 100000], [-2 ** 31, 2 ** 31 - 1]], dtype=torch.int32).cuda()
    dg.moe_dispatch_fp8(x.cuda(), row_of, buf[4:8], sf[4:8])
    got = (buf != 0xAB).any(1).cpu()
    assert got.tolist() == [i in (4, 6, 7) for i in range(12)]
    assert ((sf != -7).any(1).cpu() == got).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,K", [(1, 128), (7, 512), (300, 7168), (5, 640)])
def test_quantiser_with_fp32_scales(rows, K, dtype):
    x = activations(rows, K, dtype, seed=rows)
    q, sf = dg.quantize_fp8_1x128_sf_f32(x.cuda())
    want_q, want_sf = om.quantize_fp8_1x128_sf_f32(x.float().numpy())
    assert np.array_equal(q.cpu().numpy(), want_q) and np.array_equal(sf.cpu().numpy(), want_sf)


def test_quantiser_passes_on_what_is_not_finite():
    x = torch.ones((3, 256))
    x[0, 3], x[1, 130] = float("inf"), float("nan")
    q, sf = dg.quantize_fp8_1x128_sf_f32(x.cuda())
    assert torch.isfinite(sf).cpu().tolist() == [[False, True], [True, False], [True, True]]


# ----------------------------------------------------------------- combine ----

def combine_case(T, k, G, H, seed, drop):
    g = torch.Generator().manual_seed(seed)
    ids = choices(T, k, G, seed=seed, stray=drop)
    row_of, _, first = om.expert_rows(ids, G)
    rows = om.rows_bound(T, k, G)
    y = torch.randn((rows, H), generator=g).to(torch.bfloat16)
    named = set(row_of.ravel().tolist())
    y[[r for r in range(rows) if r not in named]] = float("nan")   # padding is never read
    return y, torch.from_numpy(row_of), torch.randn((T, k), generator=g), torch.randn((T, H), generator=g).to(torch.bfloat16)


COMBINE = [(1, 1, 1, 8, 0.0), (5, 2, 4, 24, 0.3), (64, 8, 16, 256, 0.2), (33, 9, 12, 2056, 0.1), (7, 32, 40, 7168, 0.4),
           (4, 4, 4, 512, 1.1)]


@pytest.mark.parametrize("T,k,G,H,drop", COMBINE)
@pytest.mark.parametrize("weighted", [True, False])
def test_combine(T, k, G, H, drop, weighted):
    y, row_of, w, _ = combine_case(T, k, G, H, T + k, drop)
    out = dg.moe_combine(y.cuda(), row_of.cuda(), w.cuda() if weighted else None)
    ref, mag = om.combine(f64(y), row_of.numpy(), f64(w) if weighted else None)
    bound = (k + 1) * U * mag
    assert np.all(np.abs(f64(out) - ref) <= bound * (1 + BF16) + BF16 * np.abs(ref))


@pytest.mark.parametrize("T,k,G,H,drop", COMBINE)
@pytest.mark.parametrize("weighted", [True, False])
def test_combine_backward(T, k, G, H, drop, weighted):
    y, row_of, w, d_out = combine_case(T, k, G, H, T + k, drop)
    d_y = fill_sentinel(torch.empty(y.shape, dtype=torch.bfloat16, device="cuda"))
    _, d_w = dg.moe_combine_backward(y.cuda(), row_of.cuda(), w.cuda() if weighted else None, d_out.cuda(), d_y)
    want, ref_w, mag = om.combine_backward(f64(y), row_of.numpy(), f64(w) if weighted else None, f64(d_out))
    left = is_sentinel(d_y).all(axis=1)
    got = f64(d_y)
    for r in range(y.shape[0]):
        if r in want:
            assert np.all(np.abs(got[r] - want[r]) <= (BF16 + 2 * U) * np.abs(want[r]))
        else:
            assert left[r]
    # a thread adds 8 products per pass over the columns, then 5 levels of a warp and at most 8 warps
    terms = 8 * -(-H // 8 // min(256, -(-H // 8 // 32) * 32)) + 5 + 8 + 1
    assert np.all(np.abs(f64(d_w) - ref_w) <= (terms + 8) * U * mag)


def test_combine_gradient_against_differences():
    """<d_out, out(y, w)> is linear in each of y and w, so one difference of the
    float64 forward is exact: d_w must match it to fp32 sums and d_y to bf16."""
    y, row_of, w, d_out = combine_case(4, 3, 4, 64, 11, 0.2)
    d_y = torch.zeros(y.shape, dtype=torch.bfloat16, device="cuda")
    _, d_w = dg.moe_combine_backward(y.cuda(), row_of.cuda(), w.cuda(), d_out.cuda(), d_y)
    y0 = np.nan_to_num(f64(y))
    f = lambda yy, ww: (f64(d_out) * om.combine(yy, row_of.numpy(), ww)[0]).sum()
    base = f(y0, f64(w))
    for t in range(4):
        for j in range(3):
            ww = f64(w)
            ww[t, j] += 1
            assert f(y0, ww) - base == pytest.approx(f64(d_w)[t, j], abs=200 * U * np.abs(y0).sum())
    for r in set(row_of.numpy().ravel()) - {-1}:
        yy = y0.copy()
        yy[r, 5] += 1
        assert f(yy, f64(w)) - base == pytest.approx(f64(d_y)[r, 5], rel=BF16 + 2 * U, abs=1e-9)


# ------------------------------------------------------- sizes past a C int ----

def test_sizes_past_a_c_int_are_refused():
    big = 2 ** 32
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    x = torch.zeros((4, 16), device="cuda")
    for call in (lambda: dg.moe_rows_masked(ids, 8, big + 4), lambda: dg.moe_rows_masked(ids, big + 8, 4),
                 lambda: dg.moe_rows_contiguous(ids, big + 8), lambda: dg.moe_route(x, big + 2),
                 lambda: dg.moe_route(x, 2, n_groups=big + 4), lambda: dg.moe_route(x, 2, n_groups=4, top_groups=big + 2),
                 lambda: dg.moe_route(x, 2, group_top=big + 1)):
        with pytest.raises(dg.DgError) as e:
            call()
        assert e.value.status == 3
    wide = torch.empty((1, big + 128), dtype=torch.bfloat16, device="cuda")
    row = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    for call in (lambda: dg.quantize_fp8_1x128_sf_f32(wide), lambda: dg.moe_combine(wide, row),
                 lambda: dg.moe_combine_backward(wide, row, None, wide, wide)):
        with pytest.raises(dg.DgError) as e:
            call()
        assert e.value.status == 3
    del wide
    torch.cuda.empty_cache()


# ------------------------------------------------- captured, streams, repeats ----

def test_captured_and_replayed():
    T, E, k, H = 96, 64, 4, 256
    x, b = route_inputs(T, E, True, False, 1)
    x, b = x.cuda(), b.cuda()
    act = activations(T, H, torch.bfloat16, 2).cuda()
    g = torch.randn((T, k), device="cuda")
    d_out = torch.randn((T, H), device="cuda").to(torch.bfloat16)
    rows = dg.moe_rows_bound(T, k, E)
    i32 = dict(dtype=torch.int32, device="cuda")
    ids, row_of, counts, m = (torch.empty(s, **i32) for s in ((T, k), (T, k), (E,), (rows,)))
    w, dw, dl = (torch.empty(s, device="cuda") for s in ((T, k), (T, k), (T, E)))
    q, sf = torch.empty((rows, H), dtype=torch.uint8, device="cuda"), torch.empty((rows, H // 128), device="cuda")
    y = torch.randn((rows, H), device="cuda").to(torch.bfloat16)
    out, d_y = torch.empty((T, H), dtype=torch.bfloat16, device="cuda"), torch.empty_like(y)

    def call():
        dg.moe_route(x, k, bias=b, score="sigmoid", n_groups=8, top_groups=4, ids=ids, weights=w)
        dg.moe_rows_contiguous(ids, E, row_of=row_of, m_indices=m, counts=counts)
        dg.moe_dispatch_fp8(act, row_of, q, sf)
        dg.moe_combine(y, row_of, w, out)
        dg.moe_combine_backward(y, row_of, w, d_out, d_y, dw)
        dg.moe_route_backward(x, ids, dw, score="sigmoid", d_logits=dl)

    outs = [ids, row_of, counts, m, w, q.view(torch.int16), sf, out, d_y, dw, dl]

    def reset():
        for o in outs:
            o.zero_()

    eager_equals_replay(call, outs, reset)


def test_rows_replayed_with_other_choices():
    T, k, G = 1300, 7, 200
    batches = [choices(T, k, G, seed=s, stray=0.1) for s in range(3)]
    ids = torch.from_numpy(batches[0]).cuda()
    out = dg.moe_rows_contiguous(ids, G)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dg.moe_rows_contiguous(ids, G, row_of=out[0], m_indices=out[1], counts=out[2])
    for b in batches[1:]:
        ids.copy_(torch.from_numpy(b))
        g.replay()
        ref_row, ref_counts, first = om.expert_rows(b, G)
        assert np.array_equal(out[0].cpu().numpy(), ref_row) and np.array_equal(out[2].cpu().numpy(), ref_counts)
        assert np.array_equal(out[1].cpu().numpy(), om.m_indices(ref_counts, first, out[1].numel()))
    del g


def test_other_streams_and_two_calls_at_once():
    T, E, k = 700, 128, 8
    x = [torch.randn((T, E), device="cuda") for _ in range(2)]
    want = [dg.moe_route(v, k) for v in x]
    rows = [dg.moe_rows_contiguous(i, E) for i, _ in want]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for s, (st, v) in enumerate(zip(streams, x)):
            with torch.cuda.stream(st):
                i, w = dg.moe_route(v, k)
                got[s].append((i, w, *dg.moe_rows_contiguous(i, E)))
    torch.cuda.synchronize()
    for s in range(2):
        for r in got[s]:
            assert all(torch.equal(a, b) for a, b in zip(r, (*want[s], *rows[s])))
