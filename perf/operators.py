"""Timing cases of the expert-training operators: the grouped products of an
MoE layer's experts in 16 bits with both gradients, the row expansion that
feeds them, SwiGLU with the routing weight and its gradient, and AdamW over
many tensors with 32-bit or 8-bit states.

With ``own`` false ``run`` computes the plain form in elementary torch
operations in 32 bits; with ``own`` true it makes the library's calls.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}
GRID = 128          # values that share a scale in an 8-bit AdamW state
E4M3_MAX = 448.0
E4M3_TINY = 2.0 ** -9   # smallest positive e4m3 value
TINY_AMAX = 1e-30   # a block whose largest magnitude is below this is stored as zeros


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the smallest layer of the repository's workloads: latency of one product
        dict(name="forward tiny", op="forward", T=64, K=2, E=8, N=512, Kd=512, align=32,
             routing="uniform", inactive=0.1, dtype="bf16"),
        # a decode batch: every expert's weights are read for a few rows each
        dict(name="forward decode", op="forward", T=256, K=8, E=64, N=4096, Kd=7168, align=1,
             routing="uniform", inactive=0.0, dtype="bf16"),
        # gate_up of the large skewed prefill: experts without rows, one with most tokens
        dict(name="forward zipf", op="forward", T=16384, K=8, E=32, N=4096, Kd=7168, align=1,
             routing="zipf", inactive=0.05, dtype="bf16"),
        # gradient of a product's input, uniform routing, fp16, 128-row segments
        dict(name="input grad fp16", op="input_grad", T=4096, K=8, E=32, N=4096, Kd=4096, align=128,
             routing="uniform", inactive=0.0, dtype="fp16"),
        # gradient of the weights, added to a 32-bit sum over micro-batches
        dict(name="weight grad f32 sum", op="weight_grad", T=4096, K=8, E=32, N=4096, Kd=4096, align=1,
             routing="uniform", inactive=0.0, dtype="bf16", out="f32", accumulate=True),
        # gradient of down_proj's weights of the large skewed batch
        dict(name="weight grad zipf", op="weight_grad", T=16384, K=8, E=32, N=7168, Kd=2048, align=1,
             routing="zipf", inactive=0.05, dtype="bf16", out="bf16", accumulate=False),
        # tokens to expert rows: a decode batch, then the large one
        dict(name="expand decode", op="expand", T=256, K=8, E=64, H=7168, align=16,
             routing="uniform", inactive=0.0, dtype="bf16"),
        dict(name="expand zipf", op="expand", T=16384, K=8, E=32, H=7168, align=1,
             routing="zipf", inactive=0.05, dtype="bf16"),
        # activation between the products, and its gradient with that of the routing weight
        dict(name="swiglu uniform", op="swiglu", T=4096, K=8, E=32, I=2048, align=128,
             routing="uniform", inactive=0.0, dtype="bf16"),
        dict(name="swiglu grad zipf", op="swiglu_grad", T=16384, K=8, E=32, I=2048, align=1,
             routing="zipf", inactive=0.05, dtype="bf16"),
        # optimizer step: many tensors of very different sizes, 32-bit states, bf16 gradients
        dict(name="adamw 32-bit many", op="adamw", tensors=200, smallest=1, largest=4_000_000,
             bits=32, grad="bf16", copy=True, scaled=True, spread=7),
        # optimizer step over the experts' weights themselves, 8-bit states
        dict(name="adamw 8-bit experts", op="adamw", tensors=16, smallest=8_000_000, largest=60_000_000,
             bits=8, grad="f32", copy=True, scaled=False, spread=3),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _routing(rng):
    E = rng.choice([2, 6, 8, 16, 32, 64, 160])
    return dict(E=E, K=min(E, rng.choice([1, 2, 3, 6, 8])), align=rng.choice([1, 1, 8, 16, 128]),
                routing=rng.choice(["uniform", "uniform", "zipf"]),
                inactive=rng.choice([0.0, 0.05, 0.3]), dtype=rng.choice(["bf16", "bf16", "fp16"]))


def draw(rng):
    op = rng.choice(["forward", "forward", "input_grad", "input_grad", "weight_grad", "weight_grad",
                     "expand", "swiglu", "swiglu_grad", "adamw", "adamw"])
    if op == "adamw":
        n = _log_uniform(rng, 1, 300)
        hi = _log_uniform(rng, 64, min(60_000_000, 500_000_000 // n))
        return dict(op=op, tensors=n, smallest=max(1, hi // rng.choice([1, 30, 100000])), largest=hi,
                    bits=rng.choice([32, 8]), grad=rng.choice(["bf16", "f32"]),
                    copy=rng.random() < 0.5, scaled=rng.random() < 0.5, spread=rng.randrange(1 << 20))
    r = _routing(rng)
    T = _log_uniform(rng, 1, 16384)
    T += T == 3072
    if op in ("forward", "input_grad", "weight_grad"):
        while True:
            N, Kd = 8 * _log_uniform(rng, 8, 896), 8 * _log_uniform(rng, 8, 896)
            if 3072 not in (N, Kd) and r["E"] * N * Kd <= 64 * 4096 * 7168 \
                    and T * r["K"] * N * Kd <= 16384 * 8 * 4096 * 7168:
                break
        more = {}
        if op == "weight_grad":
            more = dict(out=rng.choice([r["dtype"], "f32"]), accumulate=rng.random() < 0.4)
        return dict(op=op, T=T, N=N, Kd=Kd, **r, **more)
    width = 8 * _log_uniform(rng, 8, 896)
    width += 8 if width in (1536, 3072) else 0
    return dict(op=op, T=T, **({"H": width} if op == "expand" else {"I": min(width, 2048)}), **r)


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
    total = int(up.sum())
    source = torch.full((max(total, 1),), -1, dtype=torch.int64, device="cuda")   # row -> token
    keep = src2dst >= 0
    source[src2dst[keep]] = torch.arange(T * K, device="cuda")[keep] // K
    i32 = lambda t: t.to(torch.int32).contiguous()  # noqa: E731
    lay = dict(start=i32(start), psum=i32(start + counts), total=i32(up.sum()[None]),
               src2dst=i32(src2dst).view(T, K), E=E, align=align,
               M_cap=max(1, _capacity(T, K, E, align)))
    bounds = list(zip(start.tolist(), (start + counts).tolist()))
    return lay, bounds, total, source[:total]


def _own_layout(lay):
    import expanded_layout_expert_gb300 as mx
    dev = lay["start"].device
    return mx.Layout(psum=lay["psum"], start=lay["start"], total=lay["total"],
                     m_indices=torch.empty(0, dtype=torch.int32, device=dev),
                     src2dst=lay["src2dst"],
                     tile_prefix=torch.empty(0, dtype=torch.int32, device=dev),
                     E=lay["E"], align=lay["align"], M_cap=lay["M_cap"])


def _sizes(case):
    """Tensor sizes spread over the logarithm of [smallest, largest], odd ones
    among them, made from the case alone."""
    n, lo, hi = case["tensors"], case["smallest"], case["largest"]
    got = []
    x = case["spread"]
    for _ in range(n):
        x = (x * 1103515245 + 12345) % (1 << 31)
        got.append(max(lo, min(hi, int(round(lo * (hi / lo) ** (x / (1 << 31)))))))
    return got


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "adamw":
        return _prepare_adamw(case, g)
    dt = DTYPES[case["dtype"]]
    lay, bounds, total, source = _layout(case, g)
    M, E = lay["M_cap"], lay["E"]
    st = dict(op=op, case=case, lay=lay, bounds=bounds, total=total, source=source, dt=dt)
    if op in ("forward", "input_grad", "weight_grad"):
        N, Kd = case["N"], case["Kd"]
        if op != "weight_grad":
            st["w"] = _normal(g, E, N, Kd, dtype=dt, std=0.02)
        if op != "input_grad":
            st["x"] = _normal(g, M, Kd, dtype=dt)
        if op != "forward":
            st["dy"] = _normal(g, M, N, dtype=dt, std=0.05)
        if op == "weight_grad":
            st["acc"] = bool(case["accumulate"])
            st["out"] = (_normal(g, E, N, Kd, dtype=DTYPES[case["out"]], std=0.5) if st["acc"] else
                         torch.zeros(E, N, Kd, dtype=DTYPES[case["out"]], device="cuda"))
        else:
            st["out"] = torch.zeros(M, N if op == "forward" else Kd, dtype=dt, device="cuda")
    elif op == "expand":
        st["x"] = _normal(g, case["T"], case["H"], dtype=dt)
        st["out"] = torch.zeros(M, case["H"], dtype=dt, device="cuda")
    else:
        I = case["I"]
        st["gu"] = _normal(g, M, 2 * I, dtype=dt)
        st["row_w"] = torch.rand(M, generator=g, device="cuda")
        if op == "swiglu":
            st["out"] = torch.zeros(M, I, dtype=dt, device="cuda")
        else:
            st["dh"] = _normal(g, M, I, dtype=dt, std=0.05)
            st["dgu"] = torch.zeros(M, 2 * I, dtype=dt, device="cuda")
            st["drow_w"] = torch.zeros(M, device="cuda")
    if own:
        st["own_lay"] = _own_layout(lay)
    return st


HYPER = dict(lr=3e-4, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
STEP = 100


def _to_8_bits(v, floor):
    """Codes' values and block scales of a flat tensor of whole blocks."""
    b = v.view(-1, GRID)
    amax = b.abs().amax(1, keepdim=True)
    live = amax >= TINY_AMAX
    inv = torch.where(live, E4M3_MAX / amax, 0.0)
    q = (b * inv).to(torch.float8_e4m3fn)
    if floor:
        q = torch.where((q.float() == 0) & (b > 0) & live, E4M3_TINY, q.float()).to(torch.float8_e4m3fn)
    return q.view(-1), torch.where(live, amax * (1.0 / E4M3_MAX), 0.0).view(-1)


def _prepare_adamw(case, g):
    sizes = _sizes(case)
    at, total = [], 0
    for n in sizes:  # every tensor begins on a block of its own in the flat buffers
        at.append(total)
        total += (n + GRID - 1) // GRID * GRID
    used = torch.zeros(total + 1, dtype=torch.int8, device="cuda")
    ends = torch.tensor(at, device="cuda"), torch.tensor(sizes, device="cuda")
    used.index_add_(0, ends[0], torch.ones(len(at), dtype=torch.int8, device="cuda"))
    used.index_add_(0, ends[0] + ends[1], -torch.ones(len(at), dtype=torch.int8, device="cuda"))
    used = used[:total].cumsum(0, dtype=torch.int8)
    p = _normal(g, total, std=0.02) * used
    grad = (_normal(g, total, std=1e-3) * used).to(DTYPES[case["grad"]])
    m = _normal(g, total, std=3e-4) * used
    v = _normal(g, total, std=1e-3).square_() * used
    st = dict(op="adamw", case=case, p=p, grad=grad, step=STEP, sizes=sizes, at=at,
              copy=torch.zeros(total, dtype=torch.bfloat16, device="cuda") if case["copy"] else None,
              scale=torch.rand(1, generator=g, device="cuda") if case["scaled"] else None)
    if case["bits"] == 8:
        st["m"], st["ms"] = _to_8_bits(m, False)
        st["v"], st["vs"] = _to_8_bits(v.sqrt(), True)
        st["m"], st["v"] = st["m"].view(torch.uint8), st["v"].view(torch.uint8)
    else:
        st["m"], st["v"] = m, v
    if own:
        import expanded_layout_expert_gb300 as mx
        cut = lambda t, d=1: None if t is None else [  # noqa: E731
            t[a // d:a // d + (n + d - 1) // d] for a, n in zip(at, sizes)]
        st["opt"] = mx.AdamW(cut(p), copies=cut(st["copy"]), state_bits=case["bits"], **HYPER,
                             exp_avg=cut(st["m"]), exp_avg_sq=cut(st["v"]),
                             exp_avg_scale=cut(st.get("ms"), GRID),
                             exp_avg_sq_scale=cut(st.get("vs"), GRID), step=STEP)
        st["grads"] = cut(grad)
    return st


# ------------------------------------------------------------------ the pass
def run(st):
    if own:
        return _run_own(st)
    op = st["op"]
    if op == "adamw":
        return _plain_adamw(st)
    dt = st["dt"]
    if op in ("forward", "input_grad"):
        a = st["x"] if op == "forward" else st["dy"]
        for e, (lo, hi) in enumerate(st["bounds"]):  # the experts' row counts differ: one product each
            if hi > lo:
                w = st["w"][e].float()
                st["out"][lo:hi] = a[lo:hi].float() @ (w.t() if op == "forward" else w)
        return st["out"]
    if op == "weight_grad":
        for e, (lo, hi) in enumerate(st["bounds"]):
            dw = st["dy"][lo:hi].float().t() @ st["x"][lo:hi].float()
            st["out"][e] = st["out"][e].float() + dw if st["acc"] else dw
        return st["out"]
    n, out = st["total"], st.get("out")
    if op == "expand":
        src = st["source"]
        out[:n] = torch.where((src >= 0)[:, None], st["x"][src.clamp(min=0)], 0)
        return out
    I = st["case"]["I"]
    gate, up = st["gu"][:n, :I].float(), st["gu"][:n, I:].float()
    w = st["row_w"][:n, None]
    s = 1.0 / (1.0 + (-gate).exp())
    if op == "swiglu":
        out[:n] = gate * s * up * w
        return out
    dh = st["dh"][:n].float()
    dw = dh * w
    st["dgu"][:n, :I] = dw * up * (s * (1.0 + gate * (1.0 - s)))
    st["dgu"][:n, I:] = dw * (gate * s)
    st["drow_w"][:n] = (dh * (gate * s * up)).sum(1)
    return {"dgu": st["dgu"], "drow_w": st["drow_w"]}


def _plain_adamw(st):
    (b1, b2), lr, eps = HYPER["betas"], HYPER["lr"], HYPER["eps"]
    st["step"] += 1
    step_size = lr / (1 - b1 ** st["step"])
    root = 1.0 / math.sqrt(1 - b2 ** st["step"])
    g = st["grad"].float()
    if st["scale"] is not None:
        g = g * st["scale"]
    eight = st["case"]["bits"] == 8
    if eight:
        m = (st["m"].view(torch.float8_e4m3fn).float().view(-1, GRID) * st["ms"][:, None]).view(-1)
        v = (st["v"].view(torch.float8_e4m3fn).float().view(-1, GRID) * st["vs"][:, None]).view(-1)
        v = v * v
    else:
        m, v = st["m"], st["v"]
    m = m * b1 + g * (1 - b1)
    v = v * b2 + (g * g) * (1 - b2)
    r = v.sqrt()
    st["p"].copy_(st["p"] * (1 - lr * HYPER["weight_decay"]) - (m * step_size) / (r * root + eps))
    if st["copy"] is not None:
        st["copy"].copy_(st["p"])
    if eight:
        for name, value in (("m", m), ("v", r)):
            q, s = _to_8_bits(value, name == "v")
            st[name].copy_(q.view(torch.uint8))
            st[name + "s"].copy_(s)
    else:
        st["m"].copy_(m)
        st["v"].copy_(v)
    return _adamw_outputs(st)


def _adamw_outputs(st):
    out = {"p": st["p"]}
    if st["copy"] is not None:
        out["copy"] = st["copy"]
    if st["case"]["bits"] == 8:  # the codes as the values they stand for, and their blocks' scales
        out |= {"m": st["m"].view(torch.float8_e4m3fn), "m_scale": st["ms"],
                "v": st["v"].view(torch.float8_e4m3fn), "v_scale": st["vs"]}
    else:
        out |= {"m": st["m"], "v": st["v"]}
    return out


def _run_own(st):
    import expanded_layout_expert_gb300 as mx
    op = st["op"]
    if op == "adamw":
        st["opt"].step(st["grads"], grad_scale=st["scale"])
        return _adamw_outputs(st)
    lay = st["own_lay"]
    if op == "forward":
        return mx.grouped_matmul(st["x"], st["w"], lay, out=st["out"])
    if op == "input_grad":
        return mx.grouped_matmul_dgrad(st["dy"], st["w"], lay, out=st["out"])
    if op == "weight_grad":
        return mx.grouped_matmul_wgrad(st["dy"], st["x"], lay, out=st["out"], accumulate=st["acc"])
    if op == "expand":
        return mx.expand_rows(st["x"], lay, out=st["out"])
    if op == "swiglu":
        return mx.swiglu(st["gu"], lay, st["row_w"], out=st["out"])
    dgu, drow_w = mx.swiglu_backward(st["dh"], st["gu"], lay, st["row_w"], dgu=st["dgu"],
                                     drow_w=st["drow_w"])
    return {"dgu": dgu, "drow_w": drow_w}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "adamw":
        n = sum(_sizes(case))
        grad = 2 if case["grad"] == "bf16" else 4
        states = 16 if case["bits"] == 32 else 4 + 16 / GRID
        return {"bytes": n * (8 + grad + states + (2 if case["copy"] else 0)), "flops": 14 * n}
    T, K, E = case["T"], case["K"], case["E"]
    rows = T * K * (1 - case["inactive"])
    live = E - (max(0, min(E // 8, E - K)) if case["routing"] == "zipf" else 0)
    hit = live * (1 - (1 - min(1.0, K / live)) ** (T * (1 - case["inactive"])))   # experts with rows
    if op in ("forward", "input_grad"):
        N, Kd = case["N"], case["Kd"]
        return {"bytes": 2 * (rows * (N + Kd) + hit * N * Kd), "flops": 2 * rows * N * Kd}
    if op == "weight_grad":
        N, Kd = case["N"], case["Kd"]
        size = (4 if case["out"] == "f32" else 2) * (2 if case["accumulate"] else 1)
        return {"bytes": 2 * rows * (N + Kd) + size * (hit if case["accumulate"] else E) * N * Kd,
                "flops": 2 * rows * N * Kd}
    if op == "expand":
        return {"bytes": 2 * case["H"] * (T * (1 - case["inactive"]) + rows) + 4 * T * K, "flops": 0}
    I = case["I"]
    if op == "swiglu":
        return {"bytes": rows * (6 * I + 4), "flops": 8 * rows * I}
    return {"bytes": rows * (10 * I + 8), "flops": 20 * rows * I}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "adamw":
        return _exact_adamw(case, st)
    f64 = torch.float64
    if op in ("forward", "input_grad"):
        y = torch.zeros(st["out"].shape, dtype=f64, device="cuda")
        for e, (lo, hi) in enumerate(st["bounds"]):
            if op == "forward":
                torch.matmul(st["x"][lo:hi].to(f64), st["w"][e].to(f64).transpose(0, 1), out=y[lo:hi])
            else:
                torch.matmul(st["dy"][lo:hi].to(f64), st["w"][e].to(f64), out=y[lo:hi])
        return y
    if op == "weight_grad":
        dw = torch.zeros(st["out"].shape, dtype=f64, device="cuda")
        for e, (lo, hi) in enumerate(st["bounds"]):
            dw[e] = torch.matmul(st["dy"][lo:hi].to(f64).transpose(0, 1), st["x"][lo:hi].to(f64))
        return dw + st["out"].to(f64) if case["accumulate"] else dw
    n = st["total"]
    valid = torch.zeros(n, dtype=torch.bool, device="cuda")
    for lo, hi in st["bounds"]:
        valid[lo:hi] = True
    if op == "expand":
        y = torch.zeros(st["out"].shape, dtype=f64, device="cuda")
        pairs = st["lay"]["src2dst"].long()
        token, k = torch.nonzero(pairs >= 0, as_tuple=True)
        y[pairs[token, k]] = st["x"].to(f64)[token]
        return y
    I = case["I"]
    g, u = st["gu"][:n].to(f64).split(I, dim=1)
    w = st["row_w"][:n].to(f64).unsqueeze(1)
    sig = torch.sigmoid(g)
    if op == "swiglu":
        y = torch.zeros(st["out"].shape, dtype=f64, device="cuda")
        y[:n] = w * u * g * sig
        return y
    d = st["dh"][:n].to(f64)
    dgu = torch.zeros(st["dgu"].shape, dtype=f64, device="cuda")
    dgu[:n] = torch.cat([d * w * u * sig * (1 + g - g * sig), d * w * g * sig], dim=1)
    dr = torch.zeros(st["drow_w"].shape, dtype=f64, device="cuda")
    dr[:n] = torch.einsum("ri,ri->r", d, u * g * sig)
    return {"dgu": dgu, "drow_w": dr}


def _exact_adamw(case, st):
    f64 = torch.float64
    t = STEP + 1
    (b1, b2), lr, eps, wd = HYPER["betas"], HYPER["lr"], HYPER["eps"], HYPER["weight_decay"]
    grad = st["grad"].to(f64) * (1.0 if st["scale"] is None else st["scale"].to(f64))

    def state(name):
        if case["bits"] == 32:
            return st[name].to(f64)
        values = st[name].view(torch.float8_e4m3fn).to(f64)
        return values * st[name + "s"].to(f64).repeat_interleave(GRID)

    m = b1 * state("m") + (1 - b1) * grad
    v = b2 * (state("v") if case["bits"] == 32 else state("v").square()) + (1 - b2) * grad.square()
    p = st["p"].to(f64) * (1 - lr * wd)
    p = p - lr * (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + eps)
    out = {"p": p}
    if st["copy"] is not None:
        out["copy"] = p
    if case["bits"] == 32:
        return out | {"m": m, "v": v}
    # the codes are decisions of the rounding, so they have no value in 64 bits; the scales do
    for name, value in (("m", m), ("v", v.sqrt())):
        out[name] = None
        out[name + "_scale"] = value.view(-1, GRID).abs().amax(1) / E4M3_MAX
    return out
