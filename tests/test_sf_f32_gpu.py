"""GEMMs with fp32 block scales on the GPU, against the float64 oracle.

Tolerance. With u = 2^-24 (half a step of fp32) and mag = the sum of the
absolute values of a result's terms: the tensor core adds the 128 products of a
block (exact in fp32: 4-bit significands) in any order, each addition within a
whole step 2u since it may cut instead of round; the block's product of scales
and its FMA into the accumulator take one u each, the K/128 blocks are added
with one u each, and C with one more. A bf16 D is rounded once (2^-8)."""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_tcgen05_b200 as dg
from oracle import moe as om

from helpers import fill_sentinel, is_sentinel
from test_capture_gpu import eager_equals_replay

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(autouse=True)
def _reset():
    dg.init()
    dg.device_error(clear=True)
    yield
    dg.set_block_n(0)
    dg.set_cta_group(0)
    dg.set_splits(0)
    assert dg.device_error(clear=True) == 0


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def codes(shape, seed):
    """Finite E4M3 codes."""
    r = np.random.default_rng(seed)
    c = r.integers(0, 256, shape).astype(np.uint8)
    c[(c & 0x7F) == 0x7F] = 0x30
    return c


def scales(shape, seed):
    """fp32 scales of any mantissa, over a few binades."""
    r = np.random.default_rng(seed)
    return (2.0 ** r.uniform(-6, 2, shape)).astype(np.float32)


def operands(M, N, K, gran=128, seed=0, lead=()):
    a, b = codes((*lead, M, K), seed), codes((*lead, N, K), seed + 1)
    return a, scales((*lead, M, K // 128), seed + 2), b, scales((*lead, N if gran == 1 else -(-N // 128), K // 128), seed + 3)


def dev(*xs):
    return [torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in xs]


def bound(ref, mag, K, bf16):
    b = (2 * 128 + 2 + K // 128 + 1) * U * mag
    return b * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref) if bf16 else b


def check(d, ref, mag, K):
    got = f64(d)
    err = np.abs(got - ref) - bound(ref, mag, K, d.dtype == torch.bfloat16)
    assert np.all(err <= 0), f"{int((err > 0).sum())} of {err.size} off, worst by {err.max():.3g}"


TILES = [(128, 1), (128, 2)]
SHAPES = [(1, 8, 128), (7, 136, 384), (128, 128, 512), (130, 264, 640), (257, 520, 1152), (300, 1000, 2048)]


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_dense_every_tile(M, N, K, tile):
    ops = operands(M, N, K, seed=M + N)
    dg.set_block_n(tile[0])
    dg.set_cta_group(tile[1])
    d = fill_sentinel(torch.empty((M, N), dtype=torch.bfloat16, device="cuda"))
    dg.fp8_gemm_nt_sf_f32(*dev(*ops), d)
    check(d, *om.fp8_gemm_nt_sf_f32(*ops), K)


@pytest.mark.parametrize("tile", [(128, 1), (128, 2)])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_dense_scales_per_row_of_b(M, N, K, tile):
    ops = operands(M, N, K, gran=1, seed=M + N + 1)
    dg.set_block_n(tile[0])
    dg.set_cta_group(tile[1])
    d = torch.empty((M, N), dtype=torch.float32, device="cuda")
    dg.fp8_gemm_nt_sf_f32(*dev(*ops), d, sfb_gran_n=1)
    check(d, *om.fp8_gemm_nt_sf_f32(*ops, gran=1), K)


@pytest.mark.parametrize("M,N,K", [(1, 64, 128), (1, 4096, 7168), (33, 520, 1152), (2048, 768, 256), (129, 7168, 384)])
def test_dense_own_choice(M, N, K):
    ops = operands(M, N, K, seed=K)
    d = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    dg.fp8_gemm_nt_sf_f32(*dev(*ops), d)
    check(d, *om.fp8_gemm_nt_sf_f32(*ops), K)


@pytest.mark.parametrize("gran", [1, 128])
@pytest.mark.parametrize("splits,K", [(2, 1024), (3, 1664), (8, 4096)])
@pytest.mark.parametrize("M,N", [(1, 64), (37, 264), (128, 136), (200, 128)])
def test_split_k(M, N, K, splits, gran):
    ops = operands(M, N, K, gran=gran, seed=M + K)
    dg.set_splits(splits)
    d = torch.empty((M, N), dtype=torch.float32, device="cuda")
    args = dev(*ops)
    dg.fp8_gemm_nt_sf_f32(*args, d, sfb_gran_n=gran)
    check(d, *om.fp8_gemm_nt_sf_f32(*ops, gran=gran), K)
    again = torch.empty_like(d)
    for _ in range(3):
        dg.fp8_gemm_nt_sf_f32(*args, again, sfb_gran_n=gran)
        assert torch.equal(d, again)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tile", TILES + [(128, 1, 4)])
@pytest.mark.parametrize("in_place", [False, True])
def test_accumulate(tile, dtype, in_place):
    M, N, K = 260, 472, 2048
    ops = operands(M, N, K, seed=9)
    dg.set_block_n(tile[0])
    dg.set_cta_group(tile[1])
    dg.set_splits(tile[2] if len(tile) > 2 else 0)
    c = (1e3 * torch.randn((M, N), generator=torch.Generator().manual_seed(1))).to(dtype)
    d = c.cuda() if in_place else torch.empty((M, N), dtype=dtype, device="cuda")
    dg.fp8_gemm_nt_sf_f32(*dev(*ops), d, c=d if in_place else c.cuda())
    check(d, *om.fp8_gemm_nt_sf_f32(*ops, c=f64(c)), K)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gran", [1, 128])
@pytest.mark.parametrize("M,N,K,cg", [(1290, 2504, 256, 1), (2590, 2504, 128, 2), (1, 8, 128, 1), (130, 136, 384, 2),
                                      (95, 200, 640, 1)])
def test_accumulate_over_many_tiles(M, N, K, cg, gran, dtype):
    """Several tiles per CTA, whose parts of C follow one another; ragged rows and columns; rows around D stay."""
    ops = operands(M, N, K, gran=gran, seed=M + gran)
    dg.set_cta_group(cg)
    dg.set_splits(1)
    c = (100 * torch.randn((M, N), generator=torch.Generator().manual_seed(2))).to(dtype)
    buf = torch.full((M + 64, N), 3.0, dtype=dtype, device="cuda")
    d = buf[32:32 + M]
    args = dev(*ops)
    dg.fp8_gemm_nt_sf_f32(*args, d, c=c.cuda(), sfb_gran_n=gran)
    check(d, *om.fp8_gemm_nt_sf_f32(*ops, gran=gran, c=f64(c)), K)
    want = d.clone()
    d.copy_(c)
    dg.fp8_gemm_nt_sf_f32(*args, d, c=d, sfb_gran_n=gran)
    assert torch.equal(d, want)
    assert (buf[:32] == 3).all() and (buf[32 + M:] == 3).all()


@pytest.mark.parametrize("cg", [1, 2])
def test_a_wait_that_runs_out_with_c_under_way(cg):
    M, N, K = 300, 512, 2048
    ops = operands(M, N, K, gran=1, seed=6)
    args = dev(*ops)
    c = torch.randn((M, N), generator=torch.Generator().manual_seed(3))
    d = torch.empty((M, N), device="cuda")
    dg.set_cta_group(cg)
    dg.set_splits(1)
    try:
        dg.set_test_hooks(1, 200)
        dg.fp8_gemm_nt_sf_f32(*args, d, c=c.cuda(), sfb_gran_n=1)
        torch.cuda.synchronize()
        assert dg.device_error(clear=True) == dg.DEVERR_TIMEOUT
    finally:
        dg.set_test_hooks(0, 0)
    dg.fp8_gemm_nt_sf_f32(*args, d, c=c.cuda(), sfb_gran_n=1)
    check(d, *om.fp8_gemm_nt_sf_f32(*ops, gran=1, c=f64(c)), K)


def test_scales_off_a_16_byte_boundary_and_of_every_size():
    """One element into a buffer: the 16-byte reads of scale rows must not be taken."""
    M, N, K = 140, 264, 1024
    ops = operands(M, N, K, seed=21)
    a, sfa, b, sfb = dev(*ops)
    off = []
    for s in (sfa, sfb):
        t = torch.empty(s.numel() + 1, device="cuda")[1:].view(s.shape)
        off.append(t.copy_(s))
    d = torch.empty((M, N), dtype=torch.float32, device="cuda")
    dg.fp8_gemm_nt_sf_f32(a, off[0], b, off[1], d)
    check(d, *om.fp8_gemm_nt_sf_f32(*ops), K)
    want = d.clone()
    dg.fp8_gemm_nt_sf_f32(a, sfa, b, sfb, d)
    assert torch.equal(d, want)


def test_power_of_two_scales_agree_with_the_block_scaled_call():
    """Scales that UE8M0 can hold: the two calls compute the same sums in another order."""
    M, N, K = 300, 520, 1024
    a, sfa, b, sfb = operands(M, N, K, seed=31)
    sfa, sfb = (np.exp2(np.round(np.log2(s))).astype(np.float32) for s in (sfa, sfb))
    args = dev(a, sfa, b, sfb)
    d, e = (torch.empty((M, N), dtype=torch.float32, device="cuda") for _ in range(2))
    dg.fp8_gemm_nt_sf_f32(*args, d)
    dg.fp8_gemm_nt_acc(args[0], dg.pack_ue8m0(args[1]), args[2], dg.pack_ue8m0(args[3]), e)
    ref, mag = om.fp8_gemm_nt_sf_f32(a, sfa, b, sfb)
    check(d, ref, mag, K)
    assert np.all(np.abs(f64(d) - f64(e)) <= 2 * bound(ref, mag, K, False) + K * 2 * U * mag)


def test_what_is_not_finite_stays_in_its_row():
    M, N, K = 131, 264, 512
    a, sfa, b, sfb = operands(M, N, K, seed=41)
    a[3, 100] = 0x7F                       # NaN code
    sfa[70, 2] = np.inf
    sfa[130, 0] = np.nan
    d = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    dg.fp8_gemm_nt_sf_f32(*dev(a, sfa, b, sfb), d)
    bad = ~torch.isfinite(d).cpu()
    rows = bad.any(1).nonzero()[:, 0].tolist()
    assert rows == [3, 70, 130] and bad[[3, 70, 130]].all()


def test_guard_bands():
    """D between sentinel rows in one buffer: nothing outside it is written."""
    for M, N, K, tile in ((130, 264, 256, (128, 1)), (130, 264, 256, (128, 2)), (300, 136, 256, (128, 2)),
                          (1, 8, 512, (128, 1))):
        for dtype in (torch.bfloat16, torch.float32):
            dg.set_block_n(tile[0])
            dg.set_cta_group(tile[1])
            band = 64
            buf = torch.full(((M + 2 * band), N), 3.0, dtype=dtype, device="cuda")
            ops = operands(M, N, K, seed=M)
            dg.fp8_gemm_nt_sf_f32(*dev(*ops), buf[band:band + M])
            check(buf[band:band + M], *om.fp8_gemm_nt_sf_f32(*ops), K)
            assert (buf[:band] == 3).all() and (buf[band + M:] == 3).all()


# ------------------------------------------------------------ grouped forms ----

@pytest.mark.parametrize("tile", [(0, 0), (128, 1)])
@pytest.mark.parametrize("rows,N,K", [([130, 0, 1, 300], 264, 640), ([5], 136, 128), ([128, 128, 256], 512, 1024)])
def test_contiguous(rows, N, K, tile):
    G = len(rows)
    idx = np.concatenate([np.r_[np.full(r, e), np.full(-r % 128, -1)] for e, r in enumerate(rows)] + [np.full(128, -1)])
    idx = idx.astype(np.int32)
    M = len(idx)
    a, sfa, _, _ = operands(M, 8, K, seed=N)
    _, _, b, sfb = operands(1, N, K, seed=N + 5, lead=(G,))
    a[idx < 0], sfa[idx < 0] = 0x7F, np.nan          # padding holds anything
    dg.set_block_n(tile[0])
    dg.set_cta_group(tile[1])
    d = fill_sentinel(torch.empty((M, N), dtype=torch.bfloat16, device="cuda"))
    dg.m_grouped_fp8_gemm_nt_contiguous_sf_f32(*dev(a, sfa, b, sfb), d, *dev(idx))
    assert is_sentinel(d)[idx < 0].all()
    for e in range(G):
        mine = idx == e
        if mine.any():
            check(d[torch.from_numpy(mine).cuda()], *om.fp8_gemm_nt_sf_f32(a[mine], sfa[mine], b[e], sfb[e]), K)


def test_contiguous_mixed_block_is_flagged():
    idx = np.array([0] * 64 + [1] * 64, np.int32)
    a, sfa, _, _ = operands(128, 8, 128, seed=2)
    _, _, b, sfb = operands(1, 128, 128, seed=3, lead=(2,))
    d = fill_sentinel(torch.empty((128, 128), dtype=torch.bfloat16, device="cuda"))
    dg.m_grouped_fp8_gemm_nt_contiguous_sf_f32(*dev(a, sfa, b, sfb), d, *dev(idx))
    assert dg.device_error(clear=True) == dg.DEVERR_MIXED_EXPERT_BLOCK
    assert is_sentinel(d)[:64].all()
    check(d[64:], *om.fp8_gemm_nt_sf_f32(a[64:], sfa[64:], b[1], sfb[1]), 128)


@pytest.mark.parametrize("counts,max_m,N,K", [([5, 0, 130, 256], 256, 264, 640), ([1], 1, 8, 128), ([-3, 999, 64], 100, 136, 1024),
                                              ([0, 0], 64, 128, 256), ([7] * 40, 9, 128, 384)])
def test_masked(counts, max_m, N, K):
    G = len(counts)
    a, sfa, _, _ = operands(max_m, 8, K, seed=N, lead=(G,))
    _, _, b, sfb = operands(1, N, K, seed=N + 5, lead=(G,))
    d = fill_sentinel(torch.empty((G, max_m, N), dtype=torch.bfloat16, device="cuda"))
    live = np.clip(counts, 0, max_m)
    for g, m in enumerate(live):
        a[g, m:], sfa[g, m:] = 0x7F, np.nan
    dg.m_grouped_fp8_gemm_nt_masked_sf_f32(*dev(a, sfa, b, sfb), d, *dev(np.array(counts, np.int32)))
    left = is_sentinel(d)
    for g, m in enumerate(live):
        assert left[g, m:].all()
        if m:
            check(d[g, :m], *om.fp8_gemm_nt_sf_f32(a[g, :m], sfa[g, :m], b[g], sfb[g]), K)


def test_masked_replay_with_other_counts():
    G, max_m, N, K = 6, 140, 264, 512
    a, sfa, _, _ = operands(max_m, 8, K, seed=1, lead=(G,))
    _, _, b, sfb = operands(1, N, K, seed=2, lead=(G,))
    args, mm = dev(a, sfa, b, sfb), torch.zeros(G, dtype=torch.int32, device="cuda")
    d = torch.empty((G, max_m, N), dtype=torch.bfloat16, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dg.m_grouped_fp8_gemm_nt_masked_sf_f32(*args, d, mm)
    for counts in ([1, 140, 0, 129, 7, 64], [0] * 6, [140] * 6):
        mm.copy_(torch.tensor(counts, dtype=torch.int32))
        fill_sentinel(d)
        g.replay()
        torch.cuda.synchronize()
        left = is_sentinel(d)
        for i, m in enumerate(counts):
            assert left[i, m:].all()
            if m:
                check(d[i, :m], *om.fp8_gemm_nt_sf_f32(a[i, :m], sfa[i, :m], b[i], sfb[i]), K)


# --------------------------------------------- captured, streams, failure path ----

@pytest.mark.parametrize("M,tile,gran", [(300, (128, 2), 128), (300, (128, 2), 1), (64, (128, 1), 128), (1, (0, 0), 128)])
def test_captured_and_replayed(M, tile, gran):
    ops = dev(*operands(M, 400, 2048, gran=gran, seed=M))
    dg.set_block_n(tile[0])
    dg.set_cta_group(tile[1])
    d = torch.empty((M, 400), dtype=torch.float32, device="cuda")
    eager_equals_replay(lambda: dg.fp8_gemm_nt_sf_f32(*ops, d, sfb_gran_n=gran), [d], lambda: d.zero_())


@pytest.mark.parametrize("gran,cg", [(1, 2), (128, 1)])
def test_accumulation_in_place_replayed(gran, cg):
    """Every replay adds once more, as every eager call does."""
    M, N, K = 700, 1160, 384
    ops = dev(*operands(M, N, K, gran=gran, seed=8))
    dg.set_cta_group(cg)
    dg.set_splits(1)
    want = torch.ones((M, N), device="cuda")
    for _ in range(3):
        dg.fp8_gemm_nt_sf_f32(*ops, want, c=want, sfb_gran_n=gran)
    d = torch.ones((M, N), device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dg.fp8_gemm_nt_sf_f32(*ops, d, c=d, sfb_gran_n=gran)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(d, want)
    del g


def test_two_calls_at_once():
    cases = [dev(*operands(M, 520, 2048, seed=M)) for M in (16, 300)]
    outs = [[torch.empty((c[0].shape[0], 520), dtype=torch.bfloat16, device="cuda") for _ in range(8)] for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for i in range(8):
        for c, o, s in zip(cases, outs, streams):
            with torch.cuda.stream(s):
                dg.fp8_gemm_nt_sf_f32(*c, o[i])
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        ref = om.fp8_gemm_nt_sf_f32(*(t.cpu().numpy() for t in c))
        check(o[0], *ref, 2048)
        assert all(torch.equal(o[0], x) for x in o)


@pytest.mark.parametrize("form", ["single", "pairs", "split", "masked"])
def test_a_wait_that_runs_out_is_reported(form):
    M, N, K = 200, 512, 2048
    ops = dev(*operands(M, N, K, seed=5))
    d = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    dg.set_cta_group({"pairs": 2, "single": 1}.get(form, 0))
    dg.set_splits(4 if form == "split" else 0)
    if form == "masked":
        ops = dev(*operands(M, N, K, seed=5, lead=(1,)))
        d = d.view(1, M, N)
        mm = torch.tensor([M], dtype=torch.int32, device="cuda")

    def call():
        if form == "masked":
            dg.m_grouped_fp8_gemm_nt_masked_sf_f32(*ops, d, mm)
        else:
            dg.fp8_gemm_nt_sf_f32(*ops, d)
        torch.cuda.synchronize()

    try:
        dg.set_test_hooks(1, 200)
        call()
        assert dg.device_error(clear=True) == dg.DEVERR_TIMEOUT
    finally:
        dg.set_test_hooks(0, 0)
    call()
    check(d.view(M, N), *om.fp8_gemm_nt_sf_f32(*(t.cpu().numpy().reshape(-1, t.shape[-1]) for t in ops)), K)


def test_a_forced_tile_that_is_not_built_is_refused():
    ops = dev(*operands(256, 256, 256, seed=5))
    d = torch.empty((256, 256), dtype=torch.bfloat16, device="cuda")
    dg.set_block_n(96)
    with pytest.raises(dg.DgError) as e:
        dg.fp8_gemm_nt_sf_f32(*ops, d)
    assert e.value.status == 3


# ------------------------------------------------------------- used together ----

def quantised_rows(x):
    q, sf = dg.quantize_fp8_1x128_sf_f32(x)
    return q, sf


def test_backward_of_a_linear_layer():
    """Y = X W^T and its gradients, all as this call: dX = dY W with W's codes and
    scales transposed, dW += dY^T X with both operands quantised along the
    tokens. Each product must match the float64 product of the same codes."""
    M, N, K = 256, 384, 640
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    dy = torch.randn((M, N), generator=g, device="cuda").to(torch.bfloat16)
    wq, ws = codes((N, K), 7), scales((N // 128, K // 128), 8)
    w, sw = dev(wq, ws)
    dyq, dys = quantised_rows(dy)
    dx = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    dg.fp8_gemm_nt_sf_f32(dyq, dys, w.t().contiguous(), sw.t().contiguous(), dx)
    ref = om.dequant_sf_f32(dyq.cpu().numpy(), f64(dys)) @ om.dequant_sf_f32(wq, ws, 128)
    mag = abs(om.dequant_sf_f32(dyq.cpu().numpy(), f64(dys))) @ abs(om.dequant_sf_f32(wq, ws, 128))
    check(dx, ref, mag, N)
    aq, sa = quantised_rows(dy.t().contiguous())
    bq, sb = quantised_rows(x.t().contiguous())
    dw = torch.ones((N, K), device="cuda")
    dg.fp8_gemm_nt_sf_f32(aq, sa, bq, sb, dw, c=dw, sfb_gran_n=1)
    check(dw, *om.fp8_gemm_nt_sf_f32(aq.cpu().numpy(), f64(sa), bq.cpu().numpy(), f64(sb), gran=1, c=np.ones((N, K))), M)


@pytest.mark.parametrize("masked", [False, True])
def test_a_layer_of_experts(masked):
    """Routing, the experts' rows, dispatch, two products and combine, as a layer
    runs them, against the same steps in float64 from the same codes."""
    T, E, k, H, F = 70, 16, 4, 256, 384
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    logits = torch.randn((T, E), generator=g, device="cuda")
    up, down = codes((E, F, H), 1), codes((E, H, F), 2)
    s_up, s_down = scales((E, F // 128, H // 128), 3) / 64, scales((E, H // 128, F // 128), 4) / 64
    ids, w = dg.moe_route(logits, k, score="sigmoid", n_groups=4, top_groups=2, scale=2.5)
    if masked:
        row_of, meta, _ = dg.moe_rows_masked(ids, E, T)
        lead, gemm = (E, T), dg.m_grouped_fp8_gemm_nt_masked_sf_f32
    else:
        row_of, meta, _ = dg.moe_rows_contiguous(ids, E)
        lead, gemm = (meta.numel(),), dg.m_grouped_fp8_gemm_nt_contiguous_sf_f32
    zeros = lambda *s, dt: torch.zeros((*lead, *s), dtype=dt, device="cuda")
    q, sf = zeros(H, dt=torch.uint8), zeros(H // 128, dt=torch.float32)
    dg.moe_dispatch_fp8(x, row_of, q, sf)
    h = zeros(F, dt=torch.bfloat16)
    gemm(q, sf, *dev(up, s_up), h, meta)
    q2, sf2 = dg.quantize_fp8_1x128_sf_f32(h.view(-1, F))
    y = zeros(H, dt=torch.bfloat16)
    gemm(q2.view(*lead, F), sf2.view(*lead, F // 128), *dev(down, s_down), y, meta)
    out = dg.moe_combine(y, row_of, w)

    r_ids, r_w = om.route(f64(logits), k, None, "sigmoid", 4, 2, 2, True, 2.5)
    assert np.array_equal(ids.cpu().numpy(), r_ids)
    xq, xs = om.quantize_fp8_1x128_sf_f32(x.float().cpu().numpy())
    rows, hq, hs = row_of.cpu().numpy(), q2.cpu().numpy(), f64(sf2)
    hh, yy = f64(h.view(-1, F)), f64(y.view(-1, H))
    for t in range(T):
        for j in range(k):
            r, e = rows[t, j], r_ids[t, j]
            ref, mag = om.fp8_gemm_nt_sf_f32(xq[t:t + 1], xs[t:t + 1], up[e], s_up[e])
            assert np.all(np.abs(hh[r] - ref[0]) <= bound(ref[0], mag[0], H, True))
            ref, mag = om.fp8_gemm_nt_sf_f32(hq[r:r + 1], hs[r:r + 1], down[e], s_down[e])
            assert np.all(np.abs(yy[r] - ref[0]) <= bound(ref[0], mag[0], F, True))
    ref, mag = om.combine(yy, rows, f64(w))
    assert np.all(np.abs(f64(out) - ref) <= (k + 1) * U * mag * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref))
