"""Timing cases of the MoE layer's two ends and of its experts in 4 bits: the
top-k router with its gradient, the weighted return of the experts' rows to
their tokens with its gradient, and the experts' product over 4-bit weights with
group scales.

With ``own`` false ``run`` computes the plain form in elementary torch
operations in 32 bits; with ``own`` true it makes the library's calls.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # router of the smallest layer: the latency of a call
        dict(name="route tiny", op="route", T=64, E=8, K=2, dtype="f32", score="softmax",
             renormalize=False, bias=False),
        # router of a large prefill over many experts: biased choice, sigmoid scores
        dict(name="route prefill", op="route", T=32768, E=160, K=8, dtype="f32", score="sigmoid",
             renormalize=True, bias=True),
        # gradients of both: softmax over all experts, 16-bit logits (many ties); the large one
        dict(name="route grad bf16", op="route_grad", T=4096, E=64, K=8, dtype="bf16", score="softmax",
             renormalize=False, bias=False),
        dict(name="route grad prefill", op="route_grad", T=32768, E=160, K=8, dtype="f32",
             score="softmax", renormalize=False, bias=True),
        # rows back to the tokens of a decode batch
        dict(name="combine decode", op="combine", T=256, K=8, E=64, H=7168, align=16,
             routing="uniform", inactive=0.0, dtype="bf16", residual=False),
        # of the large skewed prefill, added to the residual stream
        dict(name="combine zipf", op="combine", T=16384, K=8, E=32, H=7168, align=1,
             routing="zipf", inactive=0.05, dtype="bf16", residual=True),
        # gradient of rows and weights: uniform routing in fp16 with aligned segments; the large one
        dict(name="combine grad fp16", op="combine_grad", T=4096, K=8, E=32, H=4096, align=128,
             routing="uniform", inactive=0.0, dtype="fp16"),
        dict(name="combine grad zipf", op="combine_grad", T=16384, K=8, E=32, H=7168, align=1,
             routing="zipf", inactive=0.05, dtype="bf16"),
        # 4-bit product of the smallest layer: latency
        dict(name="w4 tiny", op="w4", T=64, K=2, E=8, N=512, Kd=512, group=32, zeros=True, align=1,
             routing="uniform", inactive=0.1, dtype="bf16"),
        # one token's eight experts: every weight is read for a single row
        dict(name="w4 one token", op="w4", T=1, K=8, E=64, N=4096, Kd=7168, group=128, zeros=False,
             align=1, routing="uniform", inactive=0.0, dtype="bf16"),
        # down_proj of a small decode batch, fp16 with zero points, skewed
        dict(name="w4 down zipf", op="w4", T=48, K=8, E=64, N=7168, Kd=2048, group=64, zeros=True,
             align=1, routing="zipf", inactive=0.0, dtype="fp16"),
        # gate_up of a decode batch: 32 rows for every expert
        dict(name="w4 decode", op="w4", T=256, K=8, E=64, N=4096, Kd=7168, group=128, zeros=True,
             align=1, routing="uniform", inactive=0.0, dtype="bf16"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_grad", "combine", "combine_grad", "w4", "w4", "w4"])
    if op in ("route", "route_grad"):
        E = _log_uniform(rng, 2, 1024)
        most = min(131072, 32768 * 160 // E)
        return dict(op=op, T=_log_uniform(rng, 1, most), E=E, K=min(E, rng.choice([1, 2, 4, 6, 8, 16])),
                    dtype=rng.choice(["f32", "bf16", "fp16"]), score=rng.choice(["softmax", "sigmoid"]),
                    renormalize=rng.random() < 0.5, bias=rng.random() < 0.5)
    E = rng.choice([2, 6, 8, 16, 32, 64, 160])
    case = dict(op=op, E=E, K=min(E, rng.choice([1, 2, 3, 6, 8])), align=rng.choice([1, 1, 8, 16, 128]),
                routing=rng.choice(["uniform", "uniform", "zipf"]),
                inactive=rng.choice([0.0, 0.05, 0.3]), dtype=rng.choice(["bf16", "bf16", "fp16"]))
    if op in ("combine", "combine_grad"):
        case |= dict(T=_log_uniform(rng, 1, 16384), H=8 * _log_uniform(rng, 8, 896))
        case["inactive"] *= case["T"] >= 16   # a batch with tokens
        return case | (dict(residual=rng.random() < 0.5) if op == "combine" else {})
    while True:
        T, N, Kd = _log_uniform(rng, 1, 512), 8 * _log_uniform(rng, 8, 896), 32 * _log_uniform(rng, 2, 224)
        if E * N * Kd <= 64 * 4096 * 7168 and T * case["K"] * N * Kd <= 2048 * 4096 * 7168:
            break
    case["inactive"] *= T >= 16
    group = rng.choice([g for g in (32, 64, 128) if Kd % g == 0])
    return case | dict(T=T, N=N, Kd=Kd, group=group, zeros=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _capacity(T, K, E, align):
    A = T * K
    ne = min(A, E)
    return align * (ne + (A - ne) // align)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, *shape, dtype=torch.float32, std=1.0):
    """Normal values of ``dtype``, made in pieces so that no 32-bit copy of a
    large tensor is held."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for a in range(0, flat.numel(), 1 << 27):
        piece = flat[a:a + (1 << 27)]
        piece.copy_(torch.randn(piece.numel(), generator=g, device="cuda").mul_(std))
    return out


def _layout(case, g):
    """Routing of T tokens to K experts each and the rows it gives: expert e's
    rows are [start[e], psum[e]), segments begin on multiples of align, pairs
    in ascending (token, k) order."""
    T, K, E, align = case["T"], case["K"], case["E"], case["align"]
    logits = torch.zeros(E, device="cuda")
    if case["routing"] == "zipf":
        rank = torch.randperm(E, generator=g, device="cuda").float() + 1
        logits = -1.2 * rank.log()
        zero = max(0, min(E // 8, E - K))
        if zero:  # the least popular experts get no rows at all
            logits[rank > E - zero] = -1e9
    u = torch.rand(T, E, generator=g, device="cuda").clamp_(1e-9, 1 - 1e-7)
    ids = (logits - (-u.log()).log()).topk(K, dim=1).indices.to(torch.int32)
    ids[torch.rand(T, generator=g, device="cuda") < case["inactive"]] = -1
    flat = ids.view(-1).long()
    counts = torch.bincount(flat[flat >= 0], minlength=E)
    up = (counts + align - 1) // align * align
    start = up.cumsum(0) - up
    order = torch.argsort(torch.where(flat < 0, E, flat), stable=True)
    sorted_ids = torch.where(flat < 0, E, flat)[order]
    first = torch.cat([counts.cumsum(0) - counts, counts.sum()[None]])
    dest = torch.cat([start, torch.full((1,), -1, device="cuda")])[sorted_ids]
    rows = torch.where(sorted_ids < E, dest + torch.arange(T * K, device="cuda") - first[sorted_ids], -1)
    src2dst = torch.empty(T * K, dtype=torch.int64, device="cuda")
    src2dst[order] = rows
    i32 = lambda t: t.to(torch.int32).contiguous()  # noqa: E731
    return dict(start=i32(start), psum=i32(start + counts), total=i32(up.sum()[None]),
                src2dst=i32(src2dst).view(T, K), E=E, align=align,
                M_cap=max(1, _capacity(T, K, E, align))), counts


def _handle(lay):
    """The library's name for the same arrays."""
    import expanded_layout_expert_gb300 as mx
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    return mx.Layout(psum=lay["psum"], start=lay["start"], total=lay["total"], m_indices=none,
                     src2dst=lay["src2dst"], tile_prefix=none, E=lay["E"], align=lay["align"],
                     M_cap=lay["M_cap"])


def prepare(case, seed):
    g = _gen(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    st = dict(op=op, case=case, dt=dt)
    if op in ("route", "route_grad"):
        T, E, K = case["T"], case["E"], case["K"]
        st["logits"] = _normal(g, T, E, dtype=dt, std=1.5)
        st["bias"] = _normal(g, E, std=0.3) if case["bias"] else None
        if op == "route_grad":
            st["ids"] = _chosen(st["logits"], st["bias"], K).to(torch.int32)
            st["dw"] = _normal(g, T, K, std=0.1)
        return st
    lay, counts = _layout(case, g)
    M, E, T, K = lay["M_cap"], lay["E"], case["T"], case["K"]
    st |= dict(lay=lay, total=int(lay["total"]))
    if own:
        st["own_lay"] = _handle(lay)
    if op == "w4":
        N, Kd, G = case["N"], case["Kd"], case["Kd"] // case["group"]
        st["x"] = _normal(g, M, Kd, dtype=dt)
        st["codes"] = torch.randint(0, 256, (E, N, Kd // 2), generator=g, device="cuda", dtype=torch.uint8)
        st["scales"] = (torch.rand(E, N, G, generator=g, device="cuda") * 0.004 + 0.002).to(dt)
        st["zeros"] = (torch.randint(5, 11, (E, N, G), generator=g, device="cuda", dtype=torch.uint8)
                       if case["zeros"] else None)
        st["out"] = torch.zeros(M, N, dtype=dt, device="cuda")
        # the experts with rows, and the most rows that one has
        st["live"] = torch.nonzero(counts)[:, 0]
        st["most"] = int(counts.max())
        return st
    H = case["H"]
    st["rows"] = _normal(g, M, H, dtype=dt)
    st["w"] = torch.rand(T, K, generator=g, device="cuda")
    if op == "combine":
        st["residual"] = _normal(g, T, H, dtype=dt) if case["residual"] else None
        st["out"] = torch.zeros(T, H, dtype=dt, device="cuda")
    else:
        st["dy"] = _normal(g, T, H, dtype=dt, std=0.05)
        st["drows"] = torch.zeros(M, H, dtype=dt, device="cuda")
        st["dtopk_w"] = torch.zeros(T, K, device="cuda")
    return st


# ------------------------------------------------------------------ the pass
def _chosen(logits, bias, K):
    """The K largest of logit + bias in float32, ties to the lowest index."""
    key = logits.float() if bias is None else logits.float() + bias
    return key.sort(dim=1, descending=True, stable=True).indices[:, :K]


def run(st):
    return _run_own(st) if own else _PLAIN[st["op"]](st)


def _plain_route(st):
    case = st["case"]
    ids = _chosen(st["logits"], st["bias"], case["K"])
    l = st["logits"].float()
    if case["score"] == "sigmoid":
        w = 1.0 / (1.0 + (-l.gather(1, ids)).exp())
    else:
        p = (l - l.amax(1, keepdim=True)).exp()
        w = p.gather(1, ids) / p.sum(1, keepdim=True)
    if case["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    return {"ids": ids.to(torch.int32), "w": w}


def _plain_route_grad(st):
    case, ids, dw = st["case"], st["ids"].long(), st["dw"]
    l = st["logits"].float()
    zero = torch.zeros_like(l)
    if case["score"] == "sigmoid":
        s = 1.0 / (1.0 + (-l.gather(1, ids)).exp())
        if case["renormalize"]:
            r = s / s.sum(1, keepdim=True)
            dl = r * (1.0 - s) * (dw - (dw * r).sum(1, keepdim=True))
        else:
            dl = dw * s * (1.0 - s)
        return zero.scatter(1, ids, dl).to(st["dt"])
    p = (l - l.amax(1, keepdim=True)).exp()
    if case["renormalize"]:
        r = p.gather(1, ids)
        r = r / r.sum(1, keepdim=True)
        return zero.scatter(1, ids, r * (dw - (dw * r).sum(1, keepdim=True))).to(st["dt"])
    p = p / p.sum(1, keepdim=True)
    mean = (dw * p.gather(1, ids)).sum(1, keepdim=True)
    return (p * (zero.scatter(1, ids, dw) - mean)).to(st["dt"])


def _plain_combine(st):
    src = st["lay"]["src2dst"].long()
    rows = st["rows"][src.clamp(min=0)].float() * torch.where(src >= 0, st["w"], 0.0)[..., None]
    y = rows.sum(1)
    st["out"].copy_(y if st["residual"] is None else y + st["residual"].float())
    return st["out"]


def _plain_combine_grad(st):
    src = st["lay"]["src2dst"].long()
    T, K = src.shape
    valid = src >= 0
    dy = st["dy"].float()
    dots = (st["rows"][src.clamp(min=0)].float() * dy[:, None]).sum(2)
    st["dtopk_w"].copy_(torch.where(valid, dots, 0.0))
    pair = torch.full((st["lay"]["M_cap"] + 1,), -1, device="cuda")   # the pair of each row; the last: no row
    pair[torch.where(valid, src, -1).view(-1)] = torch.arange(T * K, device="cuda")
    pair = pair[:st["total"]]
    w = torch.where(pair >= 0, st["w"].view(-1)[pair.clamp(min=0)], 0.0)
    st["drows"][:st["total"]] = dy[pair.clamp(min=0) // K] * w[:, None]
    return {"drows": st["drows"], "dtopk_w": st["dtopk_w"]}


def _plain_w4(st):
    if not len(st["live"]):
        return st["out"]
    case, lay, live = st["case"], st["lay"], st["live"]
    codes = st["codes"][live]
    q = torch.stack([codes & 15, codes >> 4], dim=3).view(len(live), case["N"], -1, case["group"]).float()
    z = 8.0 if st["zeros"] is None else st["zeros"][live].float()[..., None]
    w = ((q - z) * st["scales"][live].float()[..., None]).view(len(live), case["N"], case["Kd"])
    # every expert's rows, filled up to the most that one has
    at = lay["start"][live].long()[:, None] + torch.arange(st["most"], device="cuda")
    has = at < lay["psum"][live][:, None]
    y = st["x"][torch.where(has, at, 0)].float() @ w.transpose(1, 2)
    st["out"][at[has]] = y[has].to(st["dt"])
    return st["out"]


_PLAIN = {"route": _plain_route, "route_grad": _plain_route_grad, "combine": _plain_combine,
          "combine_grad": _plain_combine_grad, "w4": _plain_w4}


def _run_own(st):
    import expanded_layout_expert_gb300 as mx
    op, case = st["op"], st["case"]
    if op == "route":
        ids, w = mx.route_topk(st["logits"], case["K"], score=case["score"],
                               renormalize=case["renormalize"], bias=st["bias"])
        return {"ids": ids, "w": w}
    if op == "route_grad":
        return mx.route_topk_backward(st["dw"], st["logits"], st["ids"], score=case["score"],
                                      renormalize=case["renormalize"])
    lay = st["own_lay"]
    if op == "combine":
        return mx.combine_rows(st["rows"], lay, st["w"], residual=st["residual"], out=st["out"])
    if op == "combine_grad":
        drows, dtopk_w = mx.combine_rows_backward(st["dy"], st["rows"], lay, st["w"], drows=st["drows"],
                                                  dtopk_w=st["dtopk_w"])
        return {"drows": drows, "dtopk_w": dtopk_w}
    return mx.grouped_matmul_w4(st["x"], st["codes"], st["scales"], lay, zeros=st["zeros"], out=st["out"])


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, T, K, E = case["op"], case["T"], case["K"], case["E"]
    size = 4 if case["dtype"] == "f32" else 2
    if op == "route":
        return {"bytes": T * (size * E + 8 * K) + (4 * E if case["bias"] else 0), "flops": 4 * T * E}
    if op == "route_grad":
        return {"bytes": T * (2 * size * E + 8 * K), "flops": 6 * T * E}
    pairs = T * K * (1 - case["inactive"])
    if op == "combine":
        return {"bytes": 2 * case["H"] * (pairs + T * (2 if case["residual"] else 1)) + 8 * T * K,
                "flops": 2 * pairs * case["H"]}
    if op == "combine_grad":
        return {"bytes": 2 * case["H"] * (2 * pairs + T) + 12 * T * K, "flops": 3 * pairs * case["H"]}
    N, Kd = case["N"], case["Kd"]
    live = E - (max(0, min(E // 8, E - K)) if case["routing"] == "zipf" else 0)
    hit = live * (1 - (1 - min(1.0, K / live)) ** (T * (1 - case["inactive"])))   # experts with rows
    weights = N * Kd * (0.5 + (3 if case["zeros"] else 2) / case["group"])
    return {"bytes": hit * weights + 2 * pairs * (N + Kd), "flops": 2 * pairs * N * Kd}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    f64, op = torch.float64, case["op"]
    if op in ("route", "route_grad"):
        return _exact_route(case, st)
    if op == "w4":
        y = torch.zeros(st["out"].shape, dtype=f64, device="cuda")
        bounds = zip(st["lay"]["start"].tolist(), st["lay"]["psum"].tolist())
        for e, (lo, hi) in enumerate(bounds):
            if hi == lo:
                continue
            w = torch.empty(case["N"], case["Kd"], dtype=f64, device="cuda")
            w[:, 0::2] = (st["codes"][e] % 16).to(f64)
            w[:, 1::2] = (st["codes"][e] // 16).to(f64)
            groups = lambda t: t[e].to(f64).repeat_interleave(case["group"], dim=1)  # noqa: E731
            w -= 8 if st["zeros"] is None else groups(st["zeros"])
            w *= groups(st["scales"])
            y[lo:hi] = torch.einsum("rk,nk->rn", st["x"][lo:hi].to(f64), w)
        return y
    src = st["lay"]["src2dst"].long()
    if op == "combine":
        y = torch.zeros(st["out"].shape, dtype=f64, device="cuda")
        if st["residual"] is not None:
            y += st["residual"].to(f64)
        for k in range(case["K"]):
            t = torch.nonzero(src[:, k] >= 0)[:, 0]
            y.index_add_(0, t, st["rows"][src[t, k]].to(f64) * st["w"][t, k, None].to(f64))
        return y
    drows = torch.zeros(st["drows"].shape, dtype=f64, device="cuda")
    dw = torch.zeros(src.shape, dtype=f64, device="cuda")
    for k in range(case["K"]):
        t = torch.nonzero(src[:, k] >= 0)[:, 0]
        r, d = src[t, k], st["dy"][t].to(f64)
        drows[r] = d * st["w"][t, k, None].to(f64)
        dw[t, k] = torch.einsum("th,th->t", d, st["rows"][r].to(f64))
    return {"drows": drows, "dtopk_w": dw}


def _exact_route(case, st):
    f64 = torch.float64
    l = st["logits"].to(f64)
    if case["op"] == "route":
        key = st["logits"].to(torch.float32)   # the choice goes by the sum in 32 bits
        if st["bias"] is not None:
            key = key + st["bias"]
        ids = torch.argsort(key, dim=1, descending=True, stable=True)[:, :case["K"]]
    else:
        ids = st["ids"].long()
    picked = torch.zeros_like(l, dtype=torch.bool).scatter(1, ids, True)
    if case["score"] == "sigmoid":
        score = torch.sigmoid(l)
        w = score / (score * picked).sum(1, keepdim=True) if case["renormalize"] else score
    else:
        w = torch.softmax(l.masked_fill(~picked, -math.inf) if case["renormalize"] else l, dim=1)
    if case["op"] == "route":
        return {"ids": ids.to(torch.int32), "w": w.gather(1, ids)}
    g = torch.zeros_like(l).scatter(1, ids, st["dw"].to(f64))
    if case["score"] == "softmax":
        return w * (g - (g * w).sum(1, keepdim=True))
    if case["renormalize"]:
        return picked * w * (1 - score) * (g - (g * w * picked).sum(1, keepdim=True))
    return picked * g * score * (1 - score)
