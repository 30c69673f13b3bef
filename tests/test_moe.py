"""Pins of the oracle for the operators around the experts' products, and the
host-side refusals of their C entry points and binding (CPU only)."""

import ctypes

import numpy as np
import pytest
import torch

import moe_grouped_gemm_tcgen05_b200 as dg
from moe_grouped_gemm_tcgen05_b200 import build as dgbuild
from oracle import moe as om

VP, I, I64, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
GOOD = VP(0x10000)


@pytest.fixture(scope="module")
def lib():
    dgbuild.build()
    return dg.load()


# ----------------------------------------------------------------- oracle ----

def test_route_worked_example():
    x = np.array([[0.0, 2.0, 1.0, 2.0]])
    ids, w = om.route(x, 2)
    assert ids.tolist() == [[1, 3]] and np.allclose(w, 0.5)              # equal logits: the lower index first
    ids, w = om.route(x, 3, renormalize=False, scale=2.0)
    e = np.exp([0.0, 2.0, 1.0, 2.0])
    assert ids.tolist() == [[1, 3, 2]] and np.allclose(w[0], 2 * e[[1, 3, 2]] / e.sum())
    # groups {0, 1} and {2, 3}: the best expert is in the first, the better pair in the second
    x = np.array([[3.0, -9.0, 2.0, 2.0]])
    assert om.route(x, 1, score="sigmoid", n_groups=2, top_groups=1, group_top=1)[0].tolist() == [[0]]
    assert om.route(x, 1, score="sigmoid", n_groups=2, top_groups=1, group_top=2)[0].tolist() == [[2]]
    # the bias moves the choice and not the weight
    ids, w = om.route(np.zeros((1, 4)), 1, bias=[0, 0, 1, 0], score="sigmoid", renormalize=False)
    assert ids.tolist() == [[2]] and w[0, 0] == 0.5


def test_route_keys_that_are_not_finite():
    inf, nan = np.inf, np.nan
    bias = np.full(8, -inf)
    bias[5] = 0.0
    assert om.route(np.zeros((1, 8)), 4, bias, "sigmoid")[0].tolist() == [[5, 0, 1, 2]]
    assert om.route(np.zeros((1, 8)), 3, [0, 0, inf, 0, 0, inf, 0, inf], "sigmoid")[0].tolist() == [[2, 5, 7]]
    # a NaN ranks below every number, as an expert and in its group's score
    x = np.array([[3.0, nan, 0.0, 0.0]])
    assert om.route(x, 4, np.zeros(4), "sigmoid")[0].tolist() == [[0, 2, 3, 1]]
    assert om.route(x, 2, np.zeros(4), "sigmoid", 2, 1, 2)[0].tolist() == [[2, 3]]
    assert om.route(x, 2, np.zeros(4), "softmax")[0].tolist() == [[0, 1]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("k", [1, 3])
def test_route_gradient_against_differences(score, renorm, k):
    r = np.random.default_rng(1)
    x, g = r.standard_normal((4, 7)), r.standard_normal((4, k))
    ids = om.route(x, k, score=score)[0]
    d = om.route_backward(x, ids, g, score, renorm, 1.5)[0]
    h = 1e-5
    for e in range(7):
        step = np.zeros((1, 7))
        step[0, e] = h
        f = [(g * om.route_weights(x + s * step, ids, score, renorm, 1.5)).sum(1) for s in (1, -1)]
        assert np.allclose((f[0] - f[1]) / (2 * h), d[:, e], atol=1e-8)


def test_expert_rows_worked_example():
    ids = np.array([[1, 0], [1, 3], [-1, 1]])
    row_of, counts, first = om.expert_rows(ids, 3)
    assert counts.tolist() == [1, 3, 0] and first.tolist() == [0, 128, 256]
    assert row_of.tolist() == [[128, 0], [129, -1], [-1, 130]]
    assert om.expert_rows(ids, 3, max_m=2)[0].tolist() == [[2, 0], [3, -1], [-1, -1]]  # the third of expert 1 is past max_m


def test_rows_bound_is_reached():
    """One choice per expert fills min(G, n) blocks, the bound's worst case."""
    for T, k, G in ((1, 8, 256), (3, 2, 4), (1, 1, 1), (40, 8, 16)):
        ids = np.arange(T * k).reshape(T, k) % G
        counts, first = om.expert_rows(ids, G)[1:]
        used = first[-1] + -(-counts[-1] // 128) * 128
        assert used <= om.rows_bound(T, k, G) < used + 128 * min(G, T * k) + 128


def test_quantiser_with_fp32_scales():
    x = np.zeros((1, 256), np.float32)
    x[0, 0], x[0, 1], x[0, 200] = 7.0, -3.5, 1e-6
    q, sf = om.quantize_fp8_1x128_sf_f32(x)
    assert sf[0, 0] == np.float32(7.0) / np.float32(448) and sf[0, 1] == np.float32(1e-4) / np.float32(448)
    assert om.dequant_sf_f32(q, sf)[0, 0] == pytest.approx(7.0, rel=1e-6)
    assert om.dequant_sf_f32(q, sf)[0, 1] == pytest.approx(-3.5, rel=1e-6)


def test_combine_is_the_transpose_of_its_gradient():
    r = np.random.default_rng(2)
    y, d = r.standard_normal((9, 8)), r.standard_normal((3, 8))
    row_of, w = np.array([[0, 8], [3, -1], [5, 2]]), r.standard_normal((3, 2))
    out = om.combine(y, row_of, w)[0]
    d_y, d_w, _ = om.combine_backward(y, row_of, w, d)
    assert (out * d).sum() == pytest.approx(sum((y[i] * v).sum() for i, v in d_y.items()))
    assert (out * d).sum() == pytest.approx((w * d_w).sum())


# --------------------------------------------------------------- refusals ----

def route_call(lib, **kw):
    a = dict(logits=GOOD, f32=1, bias=None, ids=GOOD, w=GOOD, T=4, E=16, k=2, score=0, n=1, top=1, gt=2, renorm=1,
             scale=1.0)
    a.update(kw)
    return lib.moe_route(a["logits"], a["f32"], a["bias"], a["ids"], a["w"], a["T"], a["E"], a["k"], a["score"],
                         a["n"], a["top"], a["gt"], a["renorm"], a["scale"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), 1), (dict(ids=None), 1), (dict(w=None), 1), (dict(f32=2), 1), (dict(renorm=-1), 1),
    (dict(T=0), 1), (dict(T=-3), 1), (dict(E=0), 1), (dict(k=0), 1), (dict(k=17), 1), (dict(E=1025), 3),
    (dict(E=64, k=33), 3), (dict(T=(1 << 30) + 1), 3), (dict(score=2), 1), (dict(n=3), 1), (dict(n=0), 1), (dict(n=4, top=5), 1),
    (dict(n=4, top=0), 1), (dict(gt=3), 1), (dict(gt=0), 1), (dict(E=64, n=64), 3), (dict(n=8, top=1, k=3), 1),
    (dict(logits=VP(0x10002)), 2), (dict(f32=0, logits=VP(0x10001)), 2), (dict(bias=VP(0x10002)), 2),
    (dict(ids=VP(0x10002)), 2), (dict(w=VP(0x10001)), 2)])
def test_route_refusals(lib, kw, status):
    assert route_call(lib, **kw) == status


def test_route_backward_refusals(lib):
    def call(logits=GOOD, f32=1, ids=GOOD, dw=GOOD, dl=VP(0x20000), T=4, E=16, k=2, score=0, renorm=1):
        return lib.moe_route_backward(logits, f32, ids, dw, dl, T, E, k, score, renorm, 1.0, None)
    for kw in (dict(logits=None), dict(ids=None), dict(dw=None), dict(dl=None), dict(T=0), dict(k=0), dict(k=17),
               dict(score=-1), dict(f32=3), dict(renorm=2), dict(dl=GOOD)):
        assert call(**kw) == 1, kw
    assert call(E=2000) == 3
    assert call(dl=VP(0x20002)) == 2 and call(ids=VP(0x10001)) == 2 and call(dw=VP(0x10003)) == 2


def test_rows_refusals(lib):
    def cont(ids=GOOD, row=GOOD, m=GOOD, c=GOOD, T=4, k=2, G=8, rows=1024):
        return lib.moe_rows_contiguous(ids, row, m, c, T, k, G, rows, None)
    for kw in (dict(ids=None), dict(row=None), dict(m=None), dict(c=None), dict(T=0), dict(k=0), dict(G=0),
               dict(rows=896), dict(T=1 << 30, k=32, G=1, rows=1 << 30)):
        assert cont(**kw) == 1, kw
    assert om.rows_bound(4, 2, 8) == lib.moe_rows_bound(4, 2, 8) == 1024
    assert cont(G=2000, rows=1 << 20) == 3 and cont(k=33, rows=1 << 20) == 3 and cont(rows=1 << 31) == 3
    assert cont(ids=VP(0x10002)) == 2 and cont(m=VP(0x10001)) == 2

    def masked(ids=GOOD, row=GOOD, m=GOOD, c=GOOD, T=4, k=2, G=8, mm=4):
        return lib.moe_rows_masked(ids, row, m, c, T, k, G, mm, None)
    for kw in (dict(ids=None), dict(row=None), dict(m=None), dict(c=None), dict(T=0), dict(k=0), dict(G=0), dict(mm=0)):
        assert masked(**kw) == 1, kw
    assert masked(G=1024, mm=1 << 21) == 3 and masked(G=1025) == 3 and masked(T=1 << 30, k=32) == 3
    assert masked(T=(1 << 30) + 1, k=1) == 3 and cont(T=(1 << 30) + 1, k=1, G=1, rows=(1 << 30) + 4096) == 3
    for T, k, G in ((1, 1, 1), (7, 3, 5), (4096, 8, 256), (0, 4, 4)):
        assert lib.moe_rows_bound(T, k, G) == (om.rows_bound(T, k, G) if T else 0)


def test_dispatch_and_quantiser_refusals(lib):
    def disp(x=GOOD, xf=0, row=GOOD, q=GOOD, sf=GOOD, sff=1, rows=128, T=4, k=2, H=256):
        return lib.moe_dispatch_fp8(x, xf, row, q, sf, sff, rows, T, k, H, None)
    for kw in (dict(x=None), dict(row=None), dict(q=None), dict(sf=None), dict(xf=2), dict(sff=-1), dict(rows=0),
               dict(T=0), dict(k=0), dict(H=0), dict(H=200)):
        assert disp(**kw) == 1, kw
    assert disp(k=33) == 3 and disp(rows=1 << 31) == 3 and disp(rows=1 << 30, H=1024) == 3
    assert disp(x=VP(0x10008)) == 2 and disp(q=VP(0x10008)) == 2 and disp(sf=VP(0x10002)) == 2

    def quant(x=GOOD, xf=0, q=GOOD, sf=GOOD, rows=4, K=256):
        return lib.quantize_fp8_1x128_sf_f32(x, xf, q, sf, rows, K, None)
    for kw in (dict(x=None), dict(q=None), dict(sf=None), dict(xf=5), dict(rows=0), dict(K=0), dict(K=100)):
        assert quant(**kw) == 1, kw
    assert quant(rows=1 << 31) == 3 and quant(x=VP(0x10004)) == 2 and quant(q=VP(0x10004)) == 2


def test_token_matrices_past_the_limit_are_refused(lib):
    T, H = 1 << 30, 1024   # 2^40 values
    assert lib.moe_dispatch_fp8(GOOD, 0, GOOD, GOOD, GOOD, 1, 128, T, 2, H, None) == 3
    assert lib.moe_combine(GOOD, GOOD, None, VP(0x20000), 128, T, 2, H, None) == 3
    assert lib.moe_combine_backward(GOOD, GOOD, GOOD, GOOD, VP(0x20000), GOOD, 128, T, 2, H, None) == 3


def test_combine_refusals(lib):
    def comb(y=GOOD, row=GOOD, w=None, out=VP(0x20000), rows=128, T=4, k=2, H=64):
        return lib.moe_combine(y, row, w, out, rows, T, k, H, None)
    for kw in (dict(y=None), dict(row=None), dict(out=None), dict(rows=0), dict(T=0), dict(k=0), dict(H=0), dict(H=12)):
        assert comb(**kw) == 1, kw
    assert comb(k=33) == 3 and comb(rows=1 << 31) == 3
    assert comb(y=VP(0x10008)) == 2 and comb(out=VP(0x10008)) == 2 and comb(w=VP(0x10002)) == 2

    def back(y=GOOD, row=GOOD, w=GOOD, do=GOOD, dy=VP(0x20000), dw=GOOD, rows=128, T=4, k=2, H=64):
        return lib.moe_combine_backward(y, row, w, do, dy, dw, rows, T, k, H, None)
    for kw in (dict(y=None), dict(do=None), dict(dy=None), dict(dw=None), dict(dy=GOOD), dict(T=0), dict(H=4)):
        assert back(**kw) == 1, kw
    assert back(dy=VP(0x20008)) == 2 and back(dw=VP(0x20002)) == 2


def test_sf_f32_gemm_refusals(lib):
    def dense(a=GOOD, sfa=GOOD, b=GOOD, sfb=GOOD, gran=128, c=None, d=GOOD, M=64, N=128, K=256, f32=0):
        return lib.fp8_gemm_nt_sf_f32(a, sfa, b, sfb, gran, c, d, M, N, K, f32, None)

    def cont(a=GOOD, sfa=GOOD, b=GOOD, sfb=GOOD, d=GOOD, m=GOOD, M=64, N=128, K=256, G=2):
        return lib.m_grouped_fp8_gemm_nt_contiguous_sf_f32(a, sfa, b, sfb, d, m, M, N, K, G, None)

    def masked(a=GOOD, sfa=GOOD, b=GOOD, sfb=GOOD, d=GOOD, m=GOOD, M=64, N=128, K=256, G=2):
        return lib.m_grouped_fp8_gemm_nt_masked_sf_f32(a, sfa, b, sfb, d, m, G, M, N, K, None)

    for call in (dense, cont, masked):
        for kw in (dict(a=None), dict(sfa=None), dict(b=None), dict(sfb=None), dict(d=None), dict(M=0), dict(N=0),
                   dict(K=0), dict(K=100), dict(N=12)):
            assert call(**kw) == 1, kw
        assert call(K=(1 << 20) + 128) == 3 and call(M=(1 << 30) + 1) == 3 and call(N=(1 << 30) + 8) == 3
        for name in ("a", "b", "d"):
            assert call(**{name: VP(0x10008)}) == 2
        assert call(sfa=VP(0x10002)) == 2 and call(sfb=VP(0x10001)) == 2
    for kw in (dict(gran=64), dict(gran=0), dict(f32=2)):
        assert dense(**kw) == 1
    assert dense(c=VP(0x10008)) == 2
    for call in (cont, masked):
        assert call(m=None) == 1 and call(G=0) == 1 and call(m=VP(0x10002)) == 2
    assert masked(G=1025) == 3


def test_binding_refusals():
    """The binding takes CUDA tensors of the right types only, and names the argument."""
    x, ids = torch.zeros((4, 256)), torch.zeros((4, 2), dtype=torch.int32)
    for call in (lambda: dg.moe_route(x, 2), lambda: dg.moe_route_backward(x, ids, x[:, :2]),
                 lambda: dg.moe_rows_contiguous(ids, 4), lambda: dg.moe_rows_masked(ids, 4, 4),
                 lambda: dg.moe_dispatch_fp8(x, ids, x, x), lambda: dg.quantize_fp8_1x128_sf_f32(x),
                 lambda: dg.moe_combine(x.to(torch.bfloat16), ids),
                 lambda: dg.moe_combine_backward(x.to(torch.bfloat16), ids, None, x, x)):
        with pytest.raises((ValueError, TypeError)):
            call()
    with pytest.raises(ValueError, match="score"):
        dg._score("tanh")


def test_sizes_past_a_c_int_are_refused(lib):
    """Not cut down to their lowest 32 bits, which may be a size that the call takes."""
    for sizes in ((2 ** 31,), (4, 2 ** 32 + 8), (-2 ** 32 + 2, 1)):
        with pytest.raises(dg.DgError) as e:
            dg._fits("moe_route", *sizes)
        assert e.value.status == 3
    dg._fits("moe_route", 2 ** 31 - 1, 0, -2 ** 31)
    for sizes in ((2 ** 32 + 1, 1, 1), (1, 2 ** 32 + 1, 1), (1, 1, -2 ** 32 + 1)):
        with pytest.raises(dg.DgError):
            dg.moe_rows_bound(*sizes)


def test_binding_refuses_another_device(monkeypatch):
    class On:
        def __init__(self, index):
            self.index, self.device = index, f"cuda:{index}"

        def get_device(self):
            return self.index
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(dg, "_stream", lambda device: 7)
    assert dg._here(On(0), None, On(0)) == 7
    with pytest.raises(ValueError, match="cuda:1"):
        dg._here(On(0), On(1))
