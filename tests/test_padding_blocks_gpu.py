"""Contiguous grouped GEMMs on layouts with 128-row blocks of padding only (moe_rows_contiguous leaves them behind the
last expert, and an index past the experts of this GPU makes them anywhere): such blocks are not computed, and those
around them are right."""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_tcgen05_b200 as dg
from oracle import moe as om

from helpers import bf16_to_f64, check_fp, fill_sentinel, is_sentinel
from test_sf_f32_gpu import check, codes, dev, scales

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _reset():
    dg.init()
    dg.device_error(clear=True)
    yield
    dg.set_cta_group(0)
    dg.set_test_hooks(0, 0)
    assert dg.device_error(clear=True) == 0


def problem(blocks, G, N, K, seed):
    """`blocks`: the expert of every 128-row block, -1 for padding only, 99 for experts that are not here. The last
    rows of a block are padding. Scales are powers of two, which both forms take."""
    r = np.random.default_rng(seed)
    idx = np.repeat(np.array(blocks, np.int32), 128)
    idx[idx >= 0] = np.where((np.arange(len(idx)) % 128 < r.integers(1, 129, len(blocks)).repeat(128))[idx >= 0], idx[idx >= 0], -1)
    two = lambda *s: np.exp2(r.integers(-4, 3, s)).astype(np.float32)
    a, sfa = codes((len(idx), K), seed), two(len(idx), K // 128)
    dead = (idx < 0) | (idx >= G)
    a[dead], sfa[dead] = 0x7F, 1.0
    return idx, a, sfa, codes((G, N, K), seed + 1), two(G, -(-N // 128), K // 128)


def run(form, idx, a, sfa, b, sfb, d):
    if form == "fp32 scales":
        dg.m_grouped_fp8_gemm_nt_contiguous_sf_f32(*dev(a, sfa, b, sfb), d, *dev(idx))
    else:
        a, sfa, b, sfb, idx = dev(a, sfa, b, sfb, idx)
        dg.m_grouped_fp8_gemm_nt_contiguous(a, dg.pack_ue8m0(sfa), b, dg.pack_ue8m0(sfb), d, idx)


FORMS = ["fp32 scales", "block-scaled", "block-scaled pairs"]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("blocks", [[-1], [-1] * 40, [99, -1, 99], [-1] * 1100])
def test_a_layout_of_padding_alone_is_not_computed(form, blocks):
    """The hook makes CTA 0 wait in vain on its first tile: with no tile there is no wait."""
    idx, a, sfa, b, sfb = problem(blocks, 2, 520, 256, seed=1)
    d = fill_sentinel(torch.empty((len(idx), 520), dtype=torch.bfloat16, device="cuda"))
    dg.set_cta_group(2 if form == "block-scaled pairs" else 0)
    dg.set_test_hooks(1, 200)
    run(form, idx, a, sfa, b, sfb, d)
    torch.cuda.synchronize()
    assert dg.device_error(clear=True) == 0
    assert is_sentinel(d).all()


BLOCKS = {"first": [-1, -1, -1, 0, 1, 2], "last": [0, 0, 1, 2] + [-1] * 20, "between": [0, -1, 0, 99, -1, 1, -1, 2, -1],
          "one tile": [-1] * 33 + [1], "more than a band": [0] * 5 + [-1] * 30 + [1] * 17 + [-1] * 16 + [2],
          "more than the table": [-1] * 1030 + [2, -1, 0] + [-1] * 40}


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("where", list(BLOCKS))
@pytest.mark.parametrize("N,K", [(136, 384), (2056, 640)])
def test_blocks_around_padding(where, form, N, K):
    idx, a, sfa, b, sfb = problem(BLOCKS[where], 3, N, K, seed=N)
    d = fill_sentinel(torch.empty((len(idx), N), dtype=torch.bfloat16, device="cuda"))
    dg.set_cta_group({"block-scaled": 1, "block-scaled pairs": 2}.get(form, 0))
    run(form, idx, a, sfa, b, sfb, d)
    live = (idx >= 0) & (idx < 3)
    assert is_sentinel(d)[~live].all()
    for e in range(3):
        mine = idx == e
        if mine.any():
            ref, mag = om.fp8_gemm_nt_sf_f32(a[mine], sfa[mine], b[e], sfb[e])
            got = d[torch.from_numpy(mine).cuda()]
            if form == "fp32 scales":
                check(got, ref, mag, K)
            else:
                check_fp(bf16_to_f64(got), ref, where)


@pytest.mark.parametrize("T,k,E,here", [(64, 8, 256, 256), (300, 8, 64, 8), (1, 8, 256, 256)])
def test_the_layout_of_moe_rows_contiguous(T, k, E, here):
    """Choices of E experts of which the first `here` live on this GPU, from ids to products."""
    N, K = 264, 256
    r = np.random.default_rng(T)
    ids = np.argsort(r.random((T, E)), axis=1)[:, :k].astype(np.int32)
    row_of, m_indices, _ = dg.moe_rows_contiguous(torch.from_numpy(ids).cuda(), here)
    rows, idx = row_of.cpu().numpy(), m_indices.cpu().numpy()
    M = len(idx)
    a, sfa, b, sfb = codes((M, K), 3), scales((M, K // 128), 4), codes((here, N, K), 5), scales((here, 3, K // 128), 6)
    d = fill_sentinel(torch.empty((M, N), dtype=torch.bfloat16, device="cuda"))
    run("fp32 scales", idx, a, sfa, b, sfb, d)
    assert is_sentinel(d)[idx < 0].all() and (idx >= 0).sum() == (rows >= 0).sum()
    for e in np.unique(idx[idx >= 0]):
        mine = idx == e
        check(d[torch.from_numpy(mine).cuda()], *om.fp8_gemm_nt_sf_f32(a[mine], sfa[mine], b[e], sfb[e]), K)


def test_more_experts_than_a_list_entry_holds():
    """2^21 + 1 experts of 8x128: the blocks are found without the list, padding-only ones skipped as well."""
    G, N, K = (1 << 21) + 1, 8, 128
    of = [0, -1, 1 << 21, 77, -1, (1 << 21) - 1]
    idx = np.repeat(np.array(of, np.int32), 128)
    a, sfa = codes((len(idx), K), 9), scales((len(idx), 1), 10)
    b = torch.zeros((G, N, K), dtype=torch.uint8, device="cuda")
    sfb = torch.ones((G, 1, 1), device="cuda")
    rows = {e: codes((N, K), 20 + i) for i, e in enumerate(of) if e >= 0}
    for e, w in rows.items():
        b[e] = torch.from_numpy(w).cuda()
    for form in FORMS[:2]:
        d = fill_sentinel(torch.empty((len(idx), N), dtype=torch.bfloat16, device="cuda"))
        if form == "fp32 scales":
            dg.m_grouped_fp8_gemm_nt_contiguous_sf_f32(*dev(a, sfa), b, sfb, d, *dev(idx))
        else:
            two = np.ones_like(sfa)
            dg.m_grouped_fp8_gemm_nt_contiguous(dev(a)[0], dg.pack_ue8m0(dev(two)[0]), b, dg.pack_ue8m0(sfb), d, *dev(idx))
        assert is_sentinel(d)[idx < 0].all()
        for e, w in rows.items():
            mine = idx == e
            ref, mag = om.fp8_gemm_nt_sf_f32(a[mine], sfa[mine] if form == "fp32 scales" else two[mine], w, np.ones((1, 1), np.float32))
            check(d[torch.from_numpy(mine).cuda()], ref, mag, K)


@pytest.mark.parametrize("form", FORMS)
def test_replayed_with_padding_elsewhere(form):
    """The blocks that a captured call skips are those of the m_indices at the replay."""
    N, K = 264, 384
    layouts = [[0, 1, 2, -1, -1, -1, -1], [-1] * 7, [-1, 2, -1, 0, 0, -1, 1], [1] * 7]
    idx, a, sfa, b, sfb = problem(layouts[3], 3, N, K, seed=7)
    a[a == 0x7F] = 0x30
    da, dsa, db, dsb = dev(a, sfa, b, sfb)
    pa, pb = dg.pack_ue8m0(dsa), dg.pack_ue8m0(dsb)
    m = torch.empty(len(idx), dtype=torch.int32, device="cuda")
    d = torch.empty((len(idx), N), dtype=torch.bfloat16, device="cuda")
    dg.set_cta_group({"block-scaled": 1, "block-scaled pairs": 2}.get(form, 0))
    m.fill_(-1)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        if form == "fp32 scales":
            dg.m_grouped_fp8_gemm_nt_contiguous_sf_f32(da, dsa, db, dsb, d, m)
        else:
            dg.m_grouped_fp8_gemm_nt_contiguous(da, pa, db, pb, d, m)
    for blocks in layouts:
        now = np.repeat(np.array(blocks, np.int32), 128)
        m.copy_(torch.from_numpy(now))
        fill_sentinel(d)
        g.replay()
        torch.cuda.synchronize()
        assert is_sentinel(d)[now < 0].all()
        for e in range(3):
            mine = now == e
            if mine.any():
                ref, mag = om.fp8_gemm_nt_sf_f32(a[mine], sfa[mine], b[e], sfb[e])
                got = d[torch.from_numpy(mine).cuda()]
                check(got, ref, mag, K) if form == "fp32 scales" else check_fp(bf16_to_f64(got), ref, str(blocks))
    del g
