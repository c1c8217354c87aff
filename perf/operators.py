"""What is timed of the expert-layer operators: routing, block quantisation to FP8, the block-scaled FP8 product
(one matrix and one per expert) and the weighted combination of the experts' rows.

Each case is one call (or, for training, a forward and its backward) as a program makes it.  `run` computes it in
elementary torch operations in 32 bits, or, with `own` set, through the package's operators.
"""
import math
import random

import torch

own = False
_tg = None

BLOCK = 128
FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
OUT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


def _lib():
    global _tg
    if _tg is None:
        import tiled_tensor_core_gemm_gb300
        _tg = tiled_tensor_core_gemm_gb300
    return _tg


def _cdiv(a, b):
    return -(-a // b)


# ------------------------------------------------------------------- cases ---
def listed():
    return [
        # A decode step of a serving batch: sigmoid scores, a balance bias, experts in groups; all latency.
        dict(name="route-step", op="route", tokens=48, experts=256, top_k=8, score="sigmoid", bias=True, groups=8,
             top_groups=4, group_score="top2", renormalize=True, dtype="f32", backward=False),
        # One training batch's router, with the gradient of its logits.
        dict(name="route-train", op="route", tokens=16384, experts=128, top_k=8, score="softmax", bias=False, groups=1,
             top_groups=1, group_score="max", renormalize=True, dtype="bf16", backward=True),
        # Activations of a prefill quantised by row blocks and laid out in expert order, eight copies of each token.
        dict(name="quantize-dispatch", op="quantize", batch=1, rows=8192, cols=4096, block="row", copies=8,
             dtype="bf16", to="e4m3"),
        # Activations of a training step quantised along the tokens, for the weight gradient; an odd token count.
        dict(name="quantize-columns", op="quantize", batch=1, rows=8191, cols=5120, block="col", copies=0,
             dtype="bf16", to="e4m3"),
        # A linear layer of a decode step: the weight stream is all of it.
        dict(name="scaled-step", op="scaled", m=8, n=8192, k=8192, a_block="row", b_block="tile", a_major="k",
             b_major="k", dtype="e4m3", out="bf16", bias=False, act="none"),
        # Nothing a multiple of a tile, with bias and GELU; C's pitch is odd too.
        dict(name="scaled-ragged", op="scaled", m=1000, n=4095, k=4099, a_block="row", b_block="tile", a_major="k",
             b_major="k", dtype="e4m3", out="bf16", bias=True, act="gelu"),
        # The forward product of a large training batch.
        dict(name="scaled-forward", op="scaled", m=8192, n=8192, k=8192, a_block="row", b_block="tile", a_major="k",
             b_major="k", dtype="e4m3", out="bf16", bias=False, act="none"),
        # The weight gradient dW = dY^T X of a training step: both operands with scales along the tokens, read as
        # they were stored (token-major), the result in 32 bits.
        dict(name="scaled-weight-gradient", op="scaled", m=4096, n=4096, k=8192, a_block="col", b_block="col",
             a_major="m", b_major="n", dtype="e4m3", out="f32", bias=False, act="none"),
        # A decode step through the experts: four rows an expert, every expert's weights read.
        dict(name="experts-step", op="experts", tokens=64, top_k=8, experts=128, n=2048, k=4096, w_major="k",
             dtype="e4m3", out="bf16", act="none"),
        # A prefill through the experts, GELU in the epilogue.
        dict(name="experts-prefill", op="experts", tokens=4096, top_k=8, experts=32, n=4096, k=2048, w_major="k",
             dtype="e4m3", out="bf16", act="gelu"),
        # A decode step's combination.
        dict(name="combine-step", op="combine", tokens=48, top_k=8, hidden=4096, dtype="bf16", backward=False),
        # A training step's combination with its gradients.
        dict(name="combine-train", op="combine", tokens=8192, top_k=8, hidden=4096, dtype="bf16", backward=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(("route", "quantize", "scaled", "scaled", "experts", "combine"))
    if op == "route":
        groups = rng.choice((1, 1, 2, 4, 8))
        experts = groups * rng.choice((8, 16, 24, 32, 60)) if groups > 1 else rng.choice((8, 16, 60, 64, 128, 160, 256, 384))
        top_groups = rng.randint(max(1, groups // 2), groups)
        top_k = rng.randint(1, min(10, top_groups * (experts // groups)))
        score = rng.choice(("softmax", "sigmoid"))
        bias = rng.random() < 0.5
        return dict(op=op, tokens=_log_int(rng, 1, 16384), experts=experts, top_k=top_k, score=score, bias=bias,
                    groups=groups, top_groups=top_groups, group_score=rng.choice(("max", "top2")),
                    renormalize=rng.random() < 0.7, dtype=rng.choice(("f32", "bf16", "f16")),
                    backward=rng.random() < 0.5)
    if op == "quantize":
        block = rng.choice(("row", "row", "col", "tile"))
        copies = rng.choice((0, 2, 6, 8)) if block == "row" else 0
        cols = rng.randint(16, 8192)
        batch = rng.choice((1, 3, 8)) if block == "tile" else 1
        return dict(op=op, batch=batch, rows=_log_int(rng, 1, 8192) if batch == 1 else _log_int(rng, 1, 2048), cols=cols,
                    block=block, copies=copies, dtype=rng.choice(("f32", "bf16", "f16")),
                    to=rng.choice(("e4m3", "e4m3", "e5m2")))
    if op == "scaled":
        kind = rng.choice(("forward", "forward", "input", "weight"))
        m, n, k = _log_int(rng, 1, 8192), _log_int(rng, 16, 8192), _log_int(rng, 16, 8192)
        if rng.random() < 0.5:
            n, k = n // 16 * 16, k // 16 * 16
        if kind == "weight":
            return dict(op=op, m=n, n=k, k=m, a_block="col", b_block="col", a_major="m", b_major="n",
                        dtype=rng.choice(("e4m3", "e5m2")), out="f32", bias=False, act="none")
        return dict(op=op, m=m, n=n, k=k, a_block="row", b_block="tile", a_major="k",
                    b_major="k" if kind == "forward" else "n", dtype=rng.choice(("e4m3", "e4m3", "e5m2")),
                    out=rng.choice(("bf16", "f16", "f32")), bias=rng.random() < 0.4,
                    act=rng.choice(("none", "relu", "gelu")))
    if op == "experts":
        experts = rng.choice((8, 16, 32, 60, 64, 128))
        top_k = rng.randint(1, 8)
        n, k = rng.randint(64, 2048), rng.randint(64, 4096)
        return dict(op=op, tokens=_log_int(rng, 1, 4096), top_k=top_k, experts=experts, n=n, k=k,
                    w_major=rng.choice(("k", "k", "n")), dtype="e4m3", out=rng.choice(("bf16", "f16", "f32")),
                    act=rng.choice(("none", "gelu")))
    return dict(op=op, tokens=_log_int(rng, 1, 8192), top_k=rng.randint(1, 8), hidden=rng.randint(16, 4096),
                dtype=rng.choice(("bf16", "bf16", "f16", "f32")), backward=rng.random() < 0.5)


# ----------------------------------------------------------------- prepare ---
def _randn(shape, gen, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


def _padded(shape, dtype):
    """A tensor whose rows start on 16 bytes."""
    pitch = _cdiv(shape[-1], 16) * 16
    return torch.empty((*shape[:-1], pitch), dtype=dtype, device="cuda")[..., :shape[-1]]


def _made_fp8(rows, cols, block, to, gen, batch=None):
    """An FP8 matrix and its block scales, as an earlier quantisation left them: activations and weights are near
    normal with rows (and columns) of unequal size, so the scales differ."""
    dt, top = FP8[to]
    shape = (rows, cols) if batch is None else (batch, rows, cols)
    x = torch.randn(shape, generator=gen, device="cuda")
    x *= torch.exp(0.5 * torch.randn(shape[:-1] + (1,), generator=gen, device="cuda"))
    x *= torch.exp(0.3 * torch.randn(shape[:-2] + (1, cols), generator=gen, device="cuda"))
    q, s = _plain_quantize(x, block, dt, top)
    del x
    held = _padded(shape, dt)
    held.copy_(q)
    if block == "row":       # scales of one block side by side, as they are read
        s = s.transpose(-1, -2).contiguous().transpose(-1, -2)
    return held, s


def _made_routing(tokens, top_k, experts, gen):
    """The rows of each expert for a batch: experts of unequal popularity, distinct within a token."""
    score = torch.rand((tokens, experts), generator=gen, device="cuda")
    score += 0.25 * torch.rand((experts,), generator=gen, device="cuda")
    idx = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :top_k]
    return _plain_order(idx, experts)


def _plain_order(idx, experts):
    tokens, top_k = idx.shape
    flat = idx.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    slots = torch.empty_like(order)
    slots[order] = torch.arange(order.numel(), device=order.device)
    counts = (flat[None, :] == torch.arange(experts, device=flat.device)[:, None]).sum(1)
    offsets = torch.zeros(experts + 1, dtype=torch.int64, device=flat.device)
    offsets[1:] = torch.cumsum(counts, 0)
    return order.to(torch.int32), slots.view(tokens, top_k).to(torch.int32), offsets.to(torch.int32)


def _apart(logits, bias, c, gen):
    """Draws again the logits of tokens whose choice hangs on a difference of a few units in the last place: which
    expert such a token takes says nothing about an implementation."""
    T, E, G = c["tokens"], c["experts"], c["groups"]
    near = 4e-6
    for _ in range(6):
        x = logits.double()
        s = torch.softmax(x, 1) if c["score"] == "softmax" else torch.sigmoid(x)
        key = s + bias.double() if bias is not None else s
        bad = torch.zeros(T, dtype=torch.bool, device=x.device)
        if G > 1 and c["top_groups"] < G:
            g = key.view(T, G, E // G)
            top = torch.sort(g, dim=2, descending=True).values
            gs = top[:, :, :2].sum(2) if c["group_score"] == "top2" else top[:, :, 0]
            gsort = torch.sort(gs, dim=1, descending=True)
            bad |= gsort.values[:, c["top_groups"] - 1] - gsort.values[:, c["top_groups"]] < near
            keep = torch.zeros(T, G, dtype=torch.bool, device=x.device)
            keep.scatter_(1, gsort.indices[:, :c["top_groups"]], True)
            key = torch.where(keep.repeat_interleave(E // G, 1), key, -1.0e3)
        v = torch.sort(key, dim=1, descending=True).values[:, :c["top_k"] + 1]
        bad |= ((v[:, :-1] - v[:, 1:]) < near).any(1)
        fresh = (1.5 * torch.randn((T, E), generator=gen, device="cuda")).to(logits.dtype)
        logits = torch.where(bad[:, None], fresh, logits)
    return logits


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    st = {"case": c}
    if c["op"] == "route":
        T, E = c["tokens"], c["experts"]
        logits = _randn((T, E), gen) * 1.5
        st["bias"] = None
        if c["bias"]:
            st["bias"] = _randn((E,), gen) * (0.05 if c["score"] == "sigmoid" else 0.2 / E)
        logits = logits.to(TYPES[c["dtype"]])
        if c["bias"] or (c["groups"] > 1 and c["group_score"] == "top2"):
            # (by the logits themselves, ties are equal logits and go to the lowest index everywhere)
            logits = _apart(logits, st["bias"], c, gen)
        st["logits"] = logits
        if c["backward"]:
            st["grad"] = _randn((T, c["top_k"]), gen)
    elif c["op"] == "quantize":
        shape = (c["rows"], c["cols"]) if c["batch"] == 1 else (c["batch"], c["rows"], c["cols"])
        x = _randn(shape, gen)
        x *= torch.exp(0.7 * _randn(shape[:-1] + (1,), gen))
        st["x"] = x.to(TYPES[c["dtype"]])
        st["slots"] = None
        if c["copies"]:
            perm = torch.randperm(c["rows"] * c["copies"], generator=gen, device="cuda")
            st["slots"] = perm.view(c["rows"], c["copies"]).to(torch.int32)
    elif c["op"] == "scaled":
        # column blocks lie along the tokens: K here, rows of both stored operands
        if c["a_major"] == "k":
            a, sa = _made_fp8(c["m"], c["k"], c["a_block"], c["dtype"], gen)
        else:
            a, sa = _made_fp8(c["k"], c["m"], c["a_block"], c["dtype"], gen)
            a, sa = a.t(), sa.t()
        if c["b_major"] == "k":
            b, sb = _made_fp8(c["n"], c["k"], c["b_block"], c["dtype"], gen)
            b, sb = b.t(), sb.t()
        else:
            b, sb = _made_fp8(c["k"], c["n"], c["b_block"], c["dtype"], gen)
        st.update(a=a, sa=sa, b=b, sb=sb)
        st["bias"] = _randn((c["n"],), gen) if c["bias"] else None
    elif c["op"] == "experts":
        R = c["tokens"] * c["top_k"]
        _, _, st["offsets"] = _made_routing(c["tokens"], c["top_k"], c["experts"], gen)
        st["a"], st["sa"] = _made_fp8(R, c["k"], "row", c["dtype"], gen)
        if c["w_major"] == "k":
            w, sw = _made_fp8(c["n"], c["k"], "tile", c["dtype"], gen, c["experts"])
            w, sw = w.transpose(1, 2), sw.transpose(1, 2)
        else:
            w, sw = _made_fp8(c["k"], c["n"], "tile", c["dtype"], gen, c["experts"])
        st["w"], st["sw"] = w, sw
        counts = (st["offsets"][1:] - st["offsets"][:-1]).tolist()
        st["most"] = max(counts)        # for the plain form: rows of the busiest expert
    else:
        dt = TYPES[c["dtype"]]
        R = c["tokens"] * c["top_k"]
        st["order"], st["slots"], _ = _made_routing(c["tokens"], c["top_k"], max(16, c["top_k"]), gen)
        st["y"] = _randn((R, c["hidden"]), gen, dt)
        w = torch.rand((c["tokens"], c["top_k"]), generator=gen, device="cuda") + 0.05
        st["weights"] = w / w.sum(1, keepdim=True)
        if c["backward"]:
            st["grad"] = _randn((c["tokens"], c["hidden"]), gen, dt)
    return st


# --------------------------------------------------------------------- run ---
def run(st):
    return (_RUN_OWN if own else _RUN_PLAIN)[st["case"]["op"]](st)


def _own_route(st):
    tg, c = _lib(), st["case"]
    r = tg.route(st["logits"], c["top_k"], score=c["score"], bias=st["bias"], groups=c["groups"],
                 top_groups=c["top_groups"], group_score=c["group_score"], renormalize=c["renormalize"], scale=1.5)
    out = [r.indices, r.weights, r.offsets, r.order, r.slots]
    if c["backward"]:
        out.append(tg.route_backward(st["grad"], st["logits"], r.indices, score=c["score"],
                                     renormalize=c["renormalize"], scale=1.5))
    return out


def _own_quantize(st):
    c = st["case"]
    return _lib().quantize_block(st["x"], block=c["block"], dtype=c["to"], scatter=st["slots"])


def _own_scaled(st):
    c = st["case"]
    return _lib().gemm_scaled(st["a"], st["sa"], st["b"], st["sb"], bias=st["bias"], act=c["act"], out=c["out"])


def _own_experts(st):
    c = st["case"]
    return _lib().gemm_experts(st["a"], st["sa"], st["w"], st["sw"], st["offsets"], act=c["act"], out=c["out"])


def _own_combine(st):
    tg = _lib()
    out = tg.combine(st["y"], st["slots"], st["weights"])
    if not st["case"]["backward"]:
        return out
    dy, dw = tg.combine_backward(st["grad"], st["y"], st["slots"], st["weights"], st["order"])
    return out, dy, dw


def _plain_scores(x, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    e = torch.exp(x - x.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _plain_route(st):
    c = st["case"]
    T, E, G, k = c["tokens"], c["experts"], c["groups"], c["top_k"]
    x = st["logits"].float()
    s = _plain_scores(x, c["score"])
    key = s + st["bias"] if st["bias"] is not None else x
    if G > 1 and c["top_groups"] < G:
        if c["group_score"] == "top2":
            by = key if st["bias"] is not None else s
            gs = torch.sort(by.view(T, G, E // G), dim=2, descending=True).values[:, :, :2].sum(2)
        else:
            gs = key.view(T, G, E // G).amax(2)
        chosen = torch.sort(gs, dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        keep = torch.zeros((T, G), dtype=torch.bool, device=x.device)
        keep.scatter_(1, chosen, True)
        key = torch.where(keep.repeat_interleave(E // G, 1), key, -math.inf)
    idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    picked = torch.gather(s, 1, idx)
    total = picked.sum(1, keepdim=True)
    w = 1.5 * (picked / total if c["renormalize"] else picked)
    order, slots, offsets = _plain_order(idx, E)
    out = [idx.to(torch.int32), w, offsets, order, slots]
    if c["backward"]:
        g = 1.5 * st["grad"]
        if c["renormalize"]:
            g = (g - (g * picked).sum(1, keepdim=True) / total) / total
        ds = torch.zeros_like(s).scatter_(1, idx, g)
        dx = ds * s * (1.0 - s) if c["score"] == "sigmoid" else s * (ds - (ds * s).sum(1, keepdim=True))
        out.append(dx.to(st["logits"].dtype))
    return out


def _plain_quantize(x, block, dt, top):
    """x in blocks of 128 along the columns ("row"), along the rows ("col") or both ("tile"), each divided by its
    largest magnitude over the type's."""
    *lead, m, n = x.shape
    bm, bn = (1 if block == "row" else BLOCK), (1 if block == "col" else BLOCK)
    mb, nb = _cdiv(m, bm), _cdiv(n, bn)
    held = x.float()
    if mb * bm != m or nb * bn != n:
        held = torch.nn.functional.pad(held, (0, nb * bn - n, 0, mb * bm - m))
    held = held.reshape(*lead, mb, bm, nb, bn)
    s = (held.abs().amax(dim=(-3, -1)) / top).clamp_min(2.0 ** -126)
    q = (held * (1.0 / s)[..., :, None, :, None]).to(dt)
    q = q.reshape(*lead, mb * bm, nb * bn)[..., :m, :n]
    return q, s


def _plain_quantize_run(st):
    c = st["case"]
    dt, top = FP8[c["to"]]
    q, s = _plain_quantize(st["x"], c["block"], dt, top)
    if st["slots"] is None:
        return q, s
    rows = st["slots"].reshape(-1).long()
    src = torch.arange(c["rows"], device=rows.device).repeat_interleave(c["copies"])
    qo = torch.empty((rows.numel(), q.shape[1]), dtype=torch.uint8, device=rows.device)
    qo[rows] = q.view(torch.uint8)[src]
    so = torch.empty((rows.numel(), s.shape[1]), device=rows.device)
    so[rows] = s[src]
    return qo.view(dt), so


def _plain_values(q, s):
    """The FP32 values of an FP8 matrix (or a batch of them) under its block scales."""
    v = q.float()
    if s.shape[-2] != v.shape[-2]:
        s = s.repeat_interleave(BLOCK, -2)[..., :v.shape[-2], :]
    if s.shape[-1] != v.shape[-1]:
        s = s.repeat_interleave(BLOCK, -1)[..., :v.shape[-1]]
    return v * s


def _plain_act(y, act):
    if act == "relu":
        return y.clamp_min(0.0)
    if act == "gelu":
        return 0.5 * y * (1.0 + torch.erf(y * 0.7071067811865476))
    return y


def _plain_scaled(st):
    c = st["case"]
    y = _plain_values(st["a"], st["sa"]) @ _plain_values(st["b"], st["sb"])
    if st["bias"] is not None:
        y = y + st["bias"]
    return _plain_act(y, c["act"]).to(OUT[c["out"]])


def _plain_experts(st):
    c = st["case"]
    a, w = _plain_values(st["a"], st["sa"]), _plain_values(st["w"], st["sw"])
    start, end = st["offsets"][:-1].long(), st["offsets"][1:].long()
    at = start[:, None] + torch.arange(st["most"], device=a.device)            # each expert's rows, as many as the busiest has
    real = at < end[:, None]
    y = torch.bmm(a[at.clamp_max(a.shape[0] - 1)], w)
    out = torch.empty((a.shape[0], c["n"]), dtype=OUT[c["out"]], device=a.device)
    out[at[real]] = _plain_act(y[real], c["act"]).to(out.dtype)
    return out


def _plain_combine(st):
    c = st["case"]
    rows = st["y"].float()[st["slots"].long()]                                 # tokens x top_k x hidden
    w = st["weights"]
    out = (w[:, :, None] * rows).sum(1).to(st["y"].dtype)
    if not c["backward"]:
        return out
    g = st["grad"].float()
    dw = (rows * g[:, None, :]).sum(2)
    dy = torch.empty_like(st["y"])
    dy[st["slots"].long().reshape(-1)] = (w[:, :, None] * g[:, None, :]).to(dy.dtype).reshape(-1, c["hidden"])
    return out, dy, dw


_RUN_OWN = {"route": _own_route, "quantize": _own_quantize, "scaled": _own_scaled, "experts": _own_experts,
            "combine": _own_combine}
_RUN_PLAIN = {"route": _plain_route, "quantize": _plain_quantize_run, "scaled": _plain_scaled,
              "experts": _plain_experts, "combine": _plain_combine}


# -------------------------------------------------------------------- work ---
def work(case):
    c = case
    if c["op"] == "route":
        T, E, k = c["tokens"], c["experts"], c["top_k"]
        size = T * E * BYTES[c["dtype"]]
        byte = size + (4 * E if c["bias"] else 0) + T * k * 16 + 4 * (E + 1)
        if c["backward"]:
            byte += size + T * k * 4
        return {"bytes": byte, "flops": 6 * T * E * (2 if c["backward"] else 1)}
    if c["op"] == "quantize":
        m, n = c["rows"], c["cols"]
        mb = m if c["block"] == "row" else _cdiv(m, BLOCK)
        nb = n if c["block"] == "col" else _cdiv(n, BLOCK)
        copies = c["copies"] or 1
        byte = m * n * BYTES[c["dtype"]] + copies * (m * n + 4 * mb * nb) + (4 * m * copies if c["copies"] else 0)
        return {"bytes": c["batch"] * byte, "flops": c["batch"] * 4 * m * n}
    if c["op"] == "scaled":
        m, n, k = c["m"], c["n"], c["k"]
        kb = _cdiv(k, BLOCK)
        sa = kb * m                                      # one scale a row (or column) and block
        sb = kb * (_cdiv(n, BLOCK) if c["b_block"] == "tile" else n)
        return {"bytes": m * k + k * n + 4 * (sa + sb) + m * n * BYTES[c["out"]] + (4 * n if c["bias"] else 0),
                "flops": 2 * m * n * k}
    if c["op"] == "experts":
        R, n, k = c["tokens"] * c["top_k"], c["n"], c["k"]
        kb = _cdiv(k, BLOCK)
        used = min(c["experts"], R)                      # experts that can have rows at all
        byte = R * k + 4 * kb * R + used * (n * k + 4 * kb * _cdiv(n, BLOCK)) + R * n * BYTES[c["out"]]
        return {"bytes": byte, "flops": 2 * R * n * k}
    T, k, h, b = c["tokens"], c["top_k"], c["hidden"], BYTES[c["dtype"]]
    byte = T * k * h * b + T * h * b + T * k * 8
    flops = 2 * T * k * h
    if c["backward"]:                                    # grad in, the rows' gradient out (the rows are counted above)
        byte += T * h * b + T * k * h * b + T * k * 8
        flops += 3 * T * k * h
    return {"bytes": byte, "flops": flops}


# ------------------------------------------------------------------- exact ---
def exact(case, seed):
    """The operators from their definitions in 64 bits, on the same inputs."""
    st = prepare(case, seed)
    return {"route": _exact_route, "quantize": _exact_quantize, "scaled": _exact_scaled, "experts": _exact_experts,
            "combine": _exact_combine}[case["op"]](st, case)


def _exact_route(st, c):
    x = st["logits"].to(torch.float64)
    T, E = x.shape
    p = torch.softmax(x, dim=1) if c["score"] == "softmax" else torch.special.expit(x)
    rank = p + st["bias"].to(torch.float64) if st["bias"] is not None else x.clone()
    G = c["groups"]
    if G > 1 and c["top_groups"] < G:
        per = E // G
        cols = (rank if (st["bias"] is not None or c["group_score"] == "max") else p).split(per, dim=1)
        value = torch.stack([torch.topk(col, 2 if c["group_score"] == "top2" else 1, dim=1).values.sum(1) for col in cols], 1)
        for g in range(G):          # a group stays if fewer than top_groups come before it
            ahead = (value > value[:, g:g + 1]).sum(1) + (value[:, :g] == value[:, g:g + 1]).sum(1)
            rank[:, g * per:(g + 1) * per].masked_fill_((ahead >= c["top_groups"])[:, None], -math.inf)
    ids = torch.empty((T, c["top_k"]), dtype=torch.int64, device=x.device)
    left = rank.clone()
    at = torch.arange(E, device=x.device)
    for j in range(c["top_k"]):     # the first of the largest, then without it
        ids[:, j] = torch.where(left == left.amax(1, keepdim=True), at, E).amin(1)
        left.scatter_(1, ids[:, j:j + 1], -math.inf)
    sel = p.gather(1, ids)
    z = sel.sum(1, keepdim=True) if c["renormalize"] else torch.ones_like(sel[:, :1])
    weights = 1.5 * sel / z
    out = [None, weights, None, None, None]
    if c["backward"]:
        up = st["grad"].to(torch.float64)
        # d weights_j / d sel_i = 1.5 (delta_ij - sel_j / z [renormalised]) / z
        dsel = 1.5 * up / z
        if c["renormalize"]:
            dsel = dsel - (up * weights).sum(1, keepdim=True) / z
        if c["score"] == "sigmoid":
            dx = torch.zeros_like(x).scatter_(1, ids, dsel * sel * (1 - sel))
        else:
            dx = -p * (dsel * sel).sum(1, keepdim=True)
            dx.scatter_add_(1, ids, dsel * sel)
        out.append(dx)
    return out


def _exact_quantize(st, c):
    x = st["x"].to(torch.float64)
    if x.dim() == 2:
        x = x[None]
    _, m, n = x.shape
    dt, top = FP8[c["to"]]
    size = x.abs()
    if c["block"] != "col":
        size = torch.stack([s.amax(2) for s in size.split(BLOCK, dim=2)], 2)
    if c["block"] != "row":
        size = torch.stack([s.amax(1) for s in size.split(BLOCK, dim=1)], 1)
    scale = torch.clamp(size / top, min=2.0 ** -126)
    full = scale
    if c["block"] != "col":
        full = full.repeat_interleave(BLOCK, 2)[:, :, :n]
    if c["block"] != "row":
        full = full.repeat_interleave(BLOCK, 1)[:, :m]
    q = (x / full).to(torch.float32).to(dt).to(torch.float64)
    if st["slots"] is not None:
        q2, s2 = q.new_empty((1, m * c["copies"], n)), scale.new_empty((1, m * c["copies"], scale.shape[2]))
        for j in range(c["copies"]):
            at = st["slots"][:, j].long()
            q2[0, at], s2[0, at] = q[0], scale[0]
        q, scale = q2, s2
    return (q[0], scale[0]) if c["batch"] == 1 else (q, scale)


def _exact_matrix(q, s, rows, cols):
    v = q.to(torch.float64)
    i = torch.arange(rows, device=v.device)
    j = torch.arange(cols, device=v.device)
    i = i if s.shape[0] == rows else i // BLOCK
    j = j if s.shape[1] == cols else j // BLOCK
    return v * s.to(torch.float64)[i][:, j]


def _exact_act(y, act):
    return torch.relu(y) if act == "relu" else y * torch.special.ndtr(y) if act == "gelu" else y


def _exact_scaled(st, c):
    y = torch.mm(_exact_matrix(st["a"], st["sa"], c["m"], c["k"]), _exact_matrix(st["b"], st["sb"], c["k"], c["n"]))
    if st["bias"] is not None:
        y += st["bias"].to(torch.float64)
    return _exact_act(y, c["act"])


def _exact_experts(st, c):
    off = st["offsets"].tolist()
    out = torch.empty((off[-1], c["n"]), dtype=torch.float64, device=st["a"].device)
    a = _exact_matrix(st["a"], st["sa"], c["tokens"] * c["top_k"], c["k"])
    for e in range(c["experts"]):
        if off[e + 1] > off[e]:
            out[off[e]:off[e + 1]] = a[off[e]:off[e + 1]] @ _exact_matrix(st["w"][e], st["sw"][e], c["k"], c["n"])
    return _exact_act(out, c["act"])


def _exact_combine(st, c):
    T, k, h = c["tokens"], c["top_k"], c["hidden"]
    y = st["y"].to(torch.float64)
    w = st["weights"].to(torch.float64)
    out = torch.zeros((T, h), dtype=torch.float64, device=y.device)
    for j in range(k):
        out += w[:, j:j + 1] * y[st["slots"][:, j].long()]
    if not c["backward"]:
        return out
    g = st["grad"].to(torch.float64)
    dy, dw = torch.zeros_like(y), torch.zeros_like(w)
    for j in range(k):
        at = st["slots"][:, j].long()
        dy[at] = w[:, j:j + 1] * g
        dw[:, j] = (g * y[at]).sum(1)
    return out, dy, dw
