"""The operators around the experts' products that this library is measured on,
each in a plain form (elementary torch operations) and as the library's calls.

Operators: routing of tokens to experts (forward, and with its gradient); the
8-bit matrix product with an fp32 scale per block of 128 (dense, contiguous and
masked); moving tokens to their experts' rows (with the 8-bit cast) and adding
the experts' rows back up (forward, and with its gradients).

``run`` computes the plain form, or makes the library's calls when ``own`` is
set. ``exact`` states the same results in 64 bits, written apart from both.
"""

import math
import random

import torch

own = False

_library = None  # imported and set up at the first call that needs it


def _dg():
    global _library
    if _library is None:
        import moe_grouped_gemm_tcgen05_b200 as dg
        dg.init()
        _library = dg
    return _library


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # one decode step of a served batch: 64 tokens choose 8 of 256 experts, 4 of 8 expert groups
        dict(name="route decode", op="route", T=64, E=256, k=8, score="sigmoid", bias=True, groups=8, top_groups=4,
             group_top=2, renorm=True, scale=2.5, bf16=False, train=False),
        # a long prefill batch through the same router
        dict(name="route prefill", op="route", T=16384, E=256, k=8, score="sigmoid", bias=True, groups=8,
             top_groups=4, group_top=2, renorm=True, scale=2.5, bf16=False, train=False),
        # a training step's router: softmax over 32 experts in bf16, and the gradient of its weights; an odd token count
        dict(name="route training", op="route", T=8191, E=32, k=4, score="softmax", bias=False, groups=1,
             top_groups=1, group_top=1, renorm=True, scale=1.0, bf16=True, train=True),
        # one token through a projection: the weights are all there is to read
        dict(name="product one token", op="dense", M=1, N=4096, K=7168, gran=128, f32=False, acc=False),
        # the widest prefill projection of the benchmark's shapes
        dict(name="product prefill", op="dense", M=4096, N=7168, K=16384, gran=128, f32=False, acc=False),
        # a weight gradient added to an fp32 buffer: both operands scaled per row and 128 tokens; ragged output
        dict(name="product weight gradient", op="dense", M=2112, N=7168, K=4096, gran=1, f32=True, acc=True),
        # experts' rows of a prefill batch, laid out by expert in whole 128-row blocks
        dict(name="product experts prefill", op="contiguous", G=8, lo=3500, hi=4700, N=4096, K=7168, rows_seed=1),
        # a decode step of 32 experts with about 96 tokens each
        dict(name="product experts decode", op="masked", G=32, lo=67, hi=124, max_m=256, N=4096, K=7168, rows_seed=2),
        # a prefill batch goes to its experts' rows: 8 copies of every token, cast to 8 bits
        dict(name="dispatch prefill", op="dispatch", T=8192, H=7168, G=256, k=8, max_m=0, x_f32=False),
        # a decode batch goes to the masked layout
        dict(name="dispatch decode", op="dispatch", T=64, H=7168, G=32, k=8, max_m=64, x_f32=False),
        # the experts' outputs of a training batch are added up, and the gradients go back
        dict(name="combine training", op="combine", T=4096, H=7168, G=32, k=8, max_m=0, drop=0.0, train=True),
        # a decode batch's outputs are added up, some experts living on another GPU
        dict(name="combine decode", op="combine", T=64, H=7168, G=32, k=8, max_m=64, drop=0.25, train=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "dense", "dense", "contiguous", "masked", "dispatch", "dispatch", "combine",
                     "combine"])
    if op == "route":
        E = rng.choice([8, 20, 32, 60, 64, 96, 128, 160, 256, 257, 384, 512])
        groups = rng.choice([g for g in (1, 2, 4, 8) if E % g == 0])
        top_groups = rng.randint(1, groups)
        k = rng.randint(1, min(16, E // groups * top_groups))
        return dict(op="route", T=_log_int(rng, 1, 16384), E=E, k=k, score=rng.choice(["sigmoid", "softmax"]),
                    bias=rng.random() < 0.6, groups=groups, top_groups=top_groups, group_top=rng.choice([1, 2]),
                    renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]), bf16=rng.random() < 0.4,
                    train=rng.random() < 0.4)
    if op == "dense":
        gran = rng.choice([128, 128, 1])
        f32 = gran == 1 or rng.random() < 0.3
        return dict(op="dense", M=_log_int(rng, 1, 4096), N=8 * _log_int(rng, 8, 896), K=128 * _log_int(rng, 1, 128),
                    gran=gran, f32=f32, acc=f32 and rng.random() < 0.5)
    if op == "contiguous":
        hi = _log_int(rng, 4, 4700)
        return dict(op="contiguous", G=rng.randint(1, 8), lo=rng.randint(0, hi), hi=hi, N=8 * _log_int(rng, 16, 512),
                    K=128 * _log_int(rng, 1, 56), rows_seed=rng.randint(0, 1 << 20))
    if op == "masked":
        max_m = _log_int(rng, 1, 256)
        hi = rng.randint(1, max_m)
        return dict(op="masked", G=_log_int(rng, 1, 32), lo=rng.randint(0, hi), hi=hi, max_m=max_m,
                    N=8 * _log_int(rng, 16, 512), K=128 * _log_int(rng, 1, 56), rows_seed=rng.randint(0, 1 << 20))
    G = rng.choice([8, 32, 60, 128, 256])
    k = rng.randint(1, 8)
    if rng.random() < 0.5:
        T = _log_int(rng, 1, 256)
        max_m = T
        G = min(G, 32)
    else:
        T = _log_int(rng, 1, 4096)
        max_m = 0
    H = 128 * _log_int(rng, 2, 56)
    if op == "dispatch":
        return dict(op="dispatch", T=T, H=H, G=G, k=k, max_m=max_m, x_f32=rng.random() < 0.3)
    return dict(op="combine", T=T, H=H, G=G, k=k, max_m=max_m, drop=rng.choice([0.0, 0.25]), train=rng.random() < 0.5)


def _group_rows(case):
    """Valid rows of each expert: fixed by the case, so that its work is."""
    r = random.Random(case["rows_seed"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["G"])]


def _padded(rows):
    return (rows + 127) // 128 * 128


def _row_bound(T, k, G):
    """Rows that hold T*k expert rows in whole 128-row blocks, however they fall."""
    n = T * k
    return _padded(n + min(G, n) * 127)


# ----------------------------------------------------------------- inputs ----

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _quantised(g, shape, rows_per_scale):
    """E4M3 codes and fp32 scales amax / 448 of normal values, one scale per 128
    values of `rows_per_scale` rows."""
    *lead, R, K = shape
    q = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    nr = -(-R // rows_per_scale)
    sf = torch.empty((*lead, nr, K // 128), dtype=torch.float32, device="cuda")
    qs, ss = q.view(-1, R, K), sf.view(-1, nr, K // 128)
    for i in range(qs.shape[0]):
        x = torch.randn((R, K), generator=g, device="cuda")
        # channels of unlike size, as weights and activations have
        x *= torch.exp(0.5 * torch.randn((1, K), generator=g, device="cuda"))
        pad = nr * rows_per_scale - R
        xp = torch.nn.functional.pad(x, (0, 0, 0, pad)) if pad else x
        xb = xp.view(nr, rows_per_scale, K // 128, 128)
        s = xb.abs().amax(dim=(1, 3)).clamp_min(1e-4) / 448
        ss[i] = s
        qs[i] = (xb / s[:, None, :, None]).view(-1, K)[:R].to(torch.float8_e4m3fn)
    return q, sf


def _choices(g, T, G, k):
    """k different experts for each token, some experts more popular than others."""
    p = torch.rand((T, G), generator=g, device="cuda") + 0.5 * torch.rand((1, G), generator=g, device="cuda")
    return p.topk(k, dim=1).indices.to(torch.int32).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    op = case["op"]
    if op == "route":
        T, E = case["T"], case["E"]
        x = 1.5 * torch.randn((T, E), generator=g, device="cuda")
        s["logits"] = x.to(torch.bfloat16) if case["bf16"] else x
        s["bias"] = 0.05 * torch.randn((E,), generator=g, device="cuda") if case["bias"] else None
        s["grad"] = torch.randn((T, case["k"]), generator=g, device="cuda") if case["train"] else None
    elif op == "dense":
        M, N, K = case["M"], case["N"], case["K"]
        s["a"], s["sfa"] = _quantised(g, (M, K), 1)
        s["b"], s["sfb"] = _quantised(g, (N, K), case["gran"])
        dt = torch.float32 if case["f32"] else torch.bfloat16
        s["c"] = torch.randn((M, N), generator=g, device="cuda").to(dt) if case["acc"] else None
        s["d"] = torch.zeros((M, N), dtype=dt, device="cuda")
    elif op == "contiguous":
        rows = _group_rows(case)
        total = max(128, sum(_padded(r) for r in rows))
        s["a"], s["sfa"] = _quantised(g, (total, case["K"]), 1)
        s["b"], s["sfb"] = _quantised(g, (case["G"], case["N"], case["K"]), 128)
        idx, at = torch.full((total,), -1, dtype=torch.int32), 0
        for e, r in enumerate(rows):
            idx[at:at + r] = e
            at += _padded(r)
        s["m_indices"] = idx.cuda()
        s["d"] = torch.zeros((total, case["N"]), dtype=torch.bfloat16, device="cuda")
    elif op == "masked":
        G, mm = case["G"], case["max_m"]
        s["a"], s["sfa"] = _quantised(g, (G, mm, case["K"]), 1)
        s["b"], s["sfb"] = _quantised(g, (G, case["N"], case["K"]), 128)
        s["masked_m"] = torch.tensor(_group_rows(case), dtype=torch.int32).cuda()
        s["d"] = torch.zeros((G, mm, case["N"]), dtype=torch.bfloat16, device="cuda")
    else:
        T, H, G, k, mm = case["T"], case["H"], case["G"], case["k"], case["max_m"]
        s["ids"] = _choices(g, T, G, k)
        R = G * mm if mm else _row_bound(T, k, G)
        if op == "dispatch":
            x = torch.randn((T, H), generator=g, device="cuda")
            x *= torch.exp(0.5 * torch.randn((1, H), generator=g, device="cuda"))
            s["x"] = x if case["x_f32"] else x.to(torch.bfloat16)
            s["q"] = torch.zeros((R, H), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
            s["sf"] = torch.zeros((R, H // 128), dtype=torch.float32, device="cuda")
        else:
            s["y"] = torch.randn((R, H), generator=g, device="cuda").to(torch.bfloat16)
            w = torch.rand((T, k), generator=g, device="cuda") + 0.1
            s["w"] = w / w.sum(1, keepdim=True)
            row_of = _row_of(s["ids"], G, mm)[0]
            if case["drop"]:
                row_of[torch.rand((T, k), generator=g, device="cuda") < case["drop"]] = -1
            s["row_of"] = row_of
            if case["train"]:
                s["d_out"] = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
                s["d_y"] = torch.zeros((R, H), dtype=torch.bfloat16, device="cuda")
    return s


# ------------------------------------------------------------ plain forms ----

def _scores(x, score):
    """Scores in 64 bits: the choice between two experts can hang on the last bits."""
    x = x.double()
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    e = torch.exp(x - x.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _plain_route(s):
    c = s["case"]
    x = s["logits"]
    T, E, k, n = c["T"], c["E"], c["k"], c["groups"]
    p = _scores(x, c["score"])
    key = p if s["bias"] is None else p + s["bias"].double()
    if c["top_groups"] < n:
        best = key.view(T, n, E // n).sort(dim=2, descending=True).values[:, :, :c["group_top"]].sum(2)
        chosen = best.sort(dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        keep = torch.zeros((T, n), dtype=torch.bool, device=x.device).scatter_(1, chosen, True)
        key = key.masked_fill(~keep.repeat_interleave(E // n, dim=1), -math.inf)
    ids = key.sort(dim=1, descending=True, stable=True).indices[:, :k]
    picked = p.gather(1, ids)
    total = picked.sum(1, keepdim=True) + 1e-20 if c["renorm"] else 1.0
    out = [ids.to(torch.int32), (c["scale"] * picked / total).float()]
    if c["train"]:
        grad = s["grad"].double()
        if c["renorm"]:
            # grad_j - mean as a sum of differences, which keeps its digits where the weights leave none free (k = 1)
            differ = ((grad[:, :, None] - grad[:, None, :]) * picked[:, None, :]).sum(2)
            ds = c["scale"] / total ** 2 * (differ + 1e-20 * grad)
        else:
            ds = c["scale"] * grad
        d = torch.zeros((T, E), dtype=torch.float64, device=x.device).scatter_(1, ids, ds)
        if c["score"] == "sigmoid":
            d = d * p * (1 - p)
        else:
            d = p * (d - (d * p).sum(1, keepdim=True))
        out.append(d.to(x.dtype))
    return out


def _values(q, sf, rows_per_scale):
    """The fp32 values that codes and scales stand for."""
    R, K = q.shape[-2:]
    s = sf.repeat_interleave(rows_per_scale, dim=-2)[..., :R, :]
    return (q.float().unflatten(-1, (K // 128, 128)) * s[..., None]).flatten(-2)


def _plain_dense(s):
    c = s["case"]
    r = _values(s["a"], s["sfa"], 1) @ _values(s["b"], s["sfb"], c["gran"]).t()
    if s["c"] is not None:
        r = s["c"].float() + r
    s["d"].copy_(r)
    return s["d"]


def _plain_contiguous(s):
    c, idx = s["case"], s["m_indices"].long()
    total = idx.shape[0]
    counts = torch.zeros(c["G"] + 1, dtype=torch.int64, device="cuda").scatter_add_(0, idx + 1, torch.ones_like(idx))[1:]
    first = torch.cumsum((counts + 127) // 128 * 128, 0) - (counts + 127) // 128 * 128
    slot = torch.arange(c["hi"], device="cuda")
    rows = (first[:, None] + slot).clamp_max(total - 1)                       # [G, hi]
    r = torch.bmm(_values(s["a"], s["sfa"], 1)[rows], _values(s["b"], s["sfb"], 128).transpose(1, 2))
    there = slot < counts[:, None]
    s["d"][rows[there]] = r[there].to(torch.bfloat16)
    return s["d"]


def _plain_masked(s):
    r = torch.bmm(_values(s["a"], s["sfa"], 1), _values(s["b"], s["sfb"], 128).transpose(1, 2))
    there = torch.arange(s["a"].shape[1], device="cuda") < s["masked_m"][:, None]
    s["d"].copy_(torch.where(there[:, :, None], r, s["d"].float()))
    return s["d"]


def _row_of(ids, G, max_m):
    """The row of every (token, slot) in its expert's rows, in token order; and
    the rows' experts (contiguous) or the experts' row counts (masked); and how
    many tokens chose each expert."""
    flat = ids.reshape(-1).long()
    counts = torch.bincount(flat, minlength=G)
    order = flat.sort(stable=True).indices
    begin = torch.cumsum(counts, 0) - counts
    rank = torch.empty_like(flat)
    rank[order] = torch.arange(flat.numel(), device=ids.device) - begin[flat[order]]
    if max_m:
        row = torch.where(rank < max_m, flat * max_m + rank, -1)
        meta = counts.clamp_max(max_m)
    else:
        blocks = (counts + 127) // 128 * 128
        row = (torch.cumsum(blocks, 0) - blocks)[flat] + rank
        meta = torch.full((_row_bound(*ids.shape, G),), -1, dtype=torch.int64, device=ids.device)
        meta[row] = flat
    return row.view(ids.shape).to(torch.int32), meta.to(torch.int32), counts.to(torch.int32)


def _plain_dispatch(s):
    c, x = s["case"], s["x"].float()
    row_of, meta, counts = _row_of(s["ids"], c["G"], c["max_m"])
    xb = x.view(c["T"], -1, 128)
    amax = xb.abs().amax(2).clamp_min(1e-4)
    sf = amax / 448
    q = (xb * (448 / amax)[:, :, None]).view(c["T"], -1).to(torch.float8_e4m3fn)
    kept = row_of.view(-1) >= 0
    row = row_of.view(-1)[kept].long()
    token = torch.arange(c["T"], device="cuda").repeat_interleave(c["k"])[kept]
    s["q"].view(torch.uint8)[row] = q.view(torch.uint8)[token]
    s["sf"][row] = sf[token]
    return [row_of, meta, counts, s["q"], s["sf"]]


def _plain_combine(s):
    row = s["row_of"].long()
    kept = row >= 0
    y = s["y"].float()[row.clamp_min(0)] * kept[:, :, None]                   # [T, k, H]
    out = [(y * s["w"][:, :, None]).sum(1).to(torch.bfloat16)]
    if s["case"]["train"]:
        d = s["d_out"].float()
        s["d_y"][row[kept]] = (s["w"][:, :, None] * d[:, None, :])[kept].to(torch.bfloat16)
        out += [s["d_y"], (y * d[:, None, :]).sum(2)]
    return out


# -------------------------------------------------------------------- run ----

def _own_run(s):
    dg, c, op = _dg(), s["case"], s["case"]["op"]
    if op == "route":
        ids, w = dg.moe_route(s["logits"], c["k"], bias=s["bias"], score=c["score"], n_groups=c["groups"],
                              top_groups=c["top_groups"], group_top=c["group_top"], renormalize=c["renorm"],
                              scale=c["scale"])
        if not c["train"]:
            return [ids, w]
        return [ids, w, dg.moe_route_backward(s["logits"], ids, s["grad"], score=c["score"], renormalize=c["renorm"],
                                              scale=c["scale"])]
    if op == "dense":
        return dg.fp8_gemm_nt_sf_f32(s["a"], s["sfa"], s["b"], s["sfb"], s["d"], c=s["c"], sfb_gran_n=c["gran"])
    if op == "contiguous":
        return dg.m_grouped_fp8_gemm_nt_contiguous_sf_f32(s["a"], s["sfa"], s["b"], s["sfb"], s["d"], s["m_indices"])
    if op == "masked":
        return dg.m_grouped_fp8_gemm_nt_masked_sf_f32(s["a"], s["sfa"], s["b"], s["sfb"], s["d"], s["masked_m"])
    if op == "dispatch":
        if c["max_m"]:
            row_of, meta, counts = dg.moe_rows_masked(s["ids"], c["G"], c["max_m"])
        else:
            row_of, meta, counts = dg.moe_rows_contiguous(s["ids"], c["G"])
        dg.moe_dispatch_fp8(s["x"], row_of, s["q"], s["sf"])
        return [row_of, meta, counts, s["q"], s["sf"]]
    out = [dg.moe_combine(s["y"], s["row_of"], s["w"])]
    if c["train"]:
        out += dg.moe_combine_backward(s["y"], s["row_of"], s["w"], s["d_out"], s["d_y"])
    return out


def run(state):
    if own:
        return _own_run(state)
    op = state["case"]["op"]
    if op == "route":
        return _plain_route(state)
    if op == "dense":
        return _plain_dense(state)
    if op == "contiguous":
        return _plain_contiguous(state)
    if op == "masked":
        return _plain_masked(state)
    if op == "dispatch":
        return _plain_dispatch(state)
    return _plain_combine(state)


# ------------------------------------------------------------------- work ----

def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        size = 2 if case["bf16"] else 4
        b = T * E * size + T * k * 8 + (4 * E if case["bias"] else 0)
        if case["train"]:
            b += T * E * size + T * k * 4                  # the gradient of the logits, and of the weights
        return {"bytes": b, "flops": T * E * (12 if case["train"] else 6)}
    if op == "dense":
        M, N, K = case["M"], case["N"], case["K"]
        size = 4 if case["f32"] else 2
        sfb = N if case["gran"] == 1 else -(-N // 128)
        return {"bytes": (M + N) * K + (M + sfb) * (K // 128) * 4 + M * N * size * (2 if case["acc"] else 1),
                "flops": 2 * M * N * K}
    if op in ("contiguous", "masked"):
        rows, N, K = _group_rows(case), case["N"], case["K"]
        R, live = sum(rows), sum(r > 0 for r in rows)
        return {"bytes": R * K + live * N * K + (R + live * -(-N // 128)) * (K // 128) * 4 + R * N * 2
                + 4 * (sum(map(_padded, rows)) if op == "contiguous" else case["G"]),
                "flops": max(1, 2 * R * N * K)}
    T, H, G, k = case["T"], case["H"], case["G"], case["k"]
    if op == "dispatch":
        meta = G if case["max_m"] else _row_bound(T, k, G)
        b = 4 * T * k * 2 + 4 * meta + 4 * G + T * H * (4 if case["x_f32"] else 2) + T * k * (H + H // 128 * 4)
        return {"bytes": b, "flops": 4 * T * H}
    kept = round(T * k * (1 - case["drop"]))
    b = kept * H * 2 + T * k * 8 + T * H * 2
    if case["train"]:
        b += T * H * 2 + kept * H * 2 + T * k * 4          # d_out in, d_y and d_weights out
    return {"bytes": b, "flops": kept * H * (5 if case["train"] else 2)}


# ------------------------------------------------------------------ exact ----

def _exact_product(a, sfa, b, sfb, gran):
    """sum_k a b with both scales of each 128-block, in 64 bits, block by block."""
    r = torch.zeros((a.shape[0], b.shape[0]), dtype=torch.float64, device="cuda")
    step = 2048
    for k0 in range(0, a.shape[1], step):
        cols = torch.arange(k0, min(k0 + step, a.shape[1]), device="cuda")
        x = a[:, k0:k0 + step].double() * sfa.double()[:, cols // 128]
        rows = torch.arange(b.shape[0], device="cuda") // gran
        w = b[:, k0:k0 + step].double() * sfb.double()[rows][:, cols // 128]
        r.addmm_(x, w.t())
    return r


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "route":
        x = s["logits"].double()
        T, E, k = case["T"], case["E"], case["k"]
        if case["score"] == "sigmoid":
            p = torch.sigmoid(x)
        else:
            p = torch.softmax(x, 1)
        key = p + (0 if s["bias"] is None else s["bias"].double())
        size = E // case["groups"]
        group = torch.arange(E, device="cuda") // size
        if case["top_groups"] < case["groups"]:
            per = torch.stack([key[:, group == j].topk(min(case["group_top"], size), dim=1).values.sum(1)
                               for j in range(case["groups"])], 1)
            for _ in range(case["groups"] - case["top_groups"]):   # drop the worst group, the last among equals
                worst = per.flip(1).argmin(1)
                worst = case["groups"] - 1 - worst
                per[torch.arange(T, device="cuda"), worst] = math.inf
                key = torch.where(group[None] == worst[:, None], -math.inf, key)
        ids = torch.argsort(-key, dim=1, stable=True)[:, :k]
        chosen = torch.gather(p, 1, ids)
        w = case["scale"] * chosen
        if case["renorm"]:
            w = w / (chosen.sum(1, keepdim=True) + 1e-20)
        out = [None, w]
        if case["train"]:
            # the Jacobians, applied to the gradient one after the other
            gr = s["grad"].double()
            if case["renorm"]:
                # d w_j / d s_l = (delta_jl S - s_j) / S^2, summed over j pair by pair
                S = chosen.sum(1, keepdim=True) + 1e-20
                gp = 1e-20 * gr
                for j in range(k):
                    gp = gp + chosen[:, j:j + 1] * (gr - gr[:, j:j + 1])
                gp = case["scale"] * gp / S ** 2
            else:
                gp = case["scale"] * gr
            full = torch.zeros_like(p).scatter_(1, ids, gp)
            if case["score"] == "sigmoid":
                out.append(full * (p - p * p))
            else:
                out.append(full * p - p * torch.einsum("te,te->t", full, p)[:, None])
        return out
    if op == "dense":
        r = _exact_product(s["a"], s["sfa"], s["b"], s["sfb"], case["gran"])
        return r if s["c"] is None else r + s["c"].double()
    if op == "contiguous":
        r = torch.zeros(s["d"].shape, dtype=torch.float64, device="cuda")
        for e in range(case["G"]):
            mine = (s["m_indices"] == e).nonzero()[:, 0]
            r[mine] = _exact_product(s["a"].view(torch.uint8)[mine].view(torch.float8_e4m3fn), s["sfa"][mine],
                                     s["b"][e], s["sfb"][e], 128)
        return r
    if op == "masked":
        r = torch.zeros(s["d"].shape, dtype=torch.float64, device="cuda")
        for e, m in enumerate(_group_rows(case)):
            if m:
                r[e, :m] = _exact_product(s["a"][e, :m], s["sfa"][e, :m], s["b"][e], s["sfb"][e], 128)
        return r
    T, H, G, k, mm = case["T"], case["H"], case["G"], case["k"], case["max_m"]
    if op == "dispatch":
        x = s["x"].double()
        sf = torch.stack([b.abs().amax(1) for b in x.split(128, dim=1)], 1)
        sf = torch.maximum(sf, torch.full_like(sf, 1e-4)) / 448
        q = torch.cat([b / sf[:, j:j + 1] for j, b in enumerate(x.split(128, dim=1))], 1)
        rq = torch.zeros((s["q"].shape[0], H), dtype=torch.float64, device="cuda")
        rs = torch.zeros(s["sf"].shape, dtype=torch.float64, device="cuda")
        at = 0
        for e in range(G):
            token = (s["ids"] == e).nonzero()[:, 0]
            n = min(token.numel(), mm) if mm else token.numel()
            at = e * mm if mm else at
            rq[at:at + n], rs[at:at + n] = q[token[:n]], sf[token[:n]]
            at += -(-n // 128) * 128
        return [None, None, None, rq.float().to(torch.float8_e4m3fn), rs]
    out = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for j in range(k):
        row = s["row_of"][:, j].long()
        live = (row >= 0).nonzero()[:, 0]
        out[live] += s["w"][live, j, None].double() * s["y"][row[live]].double()
    if not case["train"]:
        return [out]
    d_y = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
    d_w = torch.zeros((T, k), dtype=torch.float64, device="cuda")
    for j in range(k):
        row = s["row_of"][:, j].long()
        live = (row >= 0).nonzero()[:, 0]
        g = s["d_out"][live].double()
        d_y[row[live]] = s["w"][live, j, None].double() * g
        d_w[live, j] = (g * s["y"][row[live]].double()).sum(1)
    return [out, d_y, d_w]
