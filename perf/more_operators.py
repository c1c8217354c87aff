"""What is timed of the products around a language model's weights: the loss of the output projection over a large
vocabulary with its gradients, and low-rank adapters of many requests beside a shared projection with theirs.

Each case is one call (or, for training, a forward and its backward) as a program makes it.  `run` computes it in
elementary torch operations in 32 bits, or, with `own` set, through the package's operators.
"""
import math
import random

import torch

own = False
_tg = None

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
PIECE = 8192          # vocabulary entries the plain form takes at a time


def _lib():
    global _tg
    if _tg is None:
        import tiled_tensor_core_gemm_gb300
        _tg = tiled_tensor_core_gemm_gb300
    return _tg


# ------------------------------------------------------------------- cases ---
def listed():
    return [
        # Scoring a handful of positions (the candidates of a re-ranking): the weight stream is all of it; an odd vocabulary.
        dict(name="loss-few", op="loss", tokens=5, dim=2048, vocab=50021, dtype="bf16", layout="vd", backward=False,
             softcap=0.0, smoothing=0.0, z_loss=0.0),
        # An evaluation batch: losses only.
        dict(name="loss-evaluation", op="loss", tokens=2048, dim=4096, vocab=65536, dtype="bf16", layout="vd",
             backward=False, softcap=0.0, smoothing=0.0, z_loss=0.0),
        # A small model's training step.
        dict(name="loss-train-small", op="loss", tokens=512, dim=512, vocab=8000, dtype="f16", layout="vd", backward=True,
             softcap=0.0, smoothing=0.0, z_loss=1e-4),
        # Nothing a multiple of a tile, capped logits, label smoothing, the weights held as dim x vocab.
        dict(name="loss-train-ragged", op="loss", tokens=1999, dim=1032, vocab=50021, dtype="bf16", layout="dv",
             backward=True, softcap=30.0, smoothing=0.1, z_loss=0.0),
        # The loss and its gradients of a training batch with a large vocabulary.
        dict(name="loss-train", op="loss", tokens=8192, dim=4096, vocab=131072, dtype="bf16", layout="vd", backward=True,
             softcap=0.0, smoothing=0.0, z_loss=0.0),
        # One request decoding: a single token with its adapter.
        dict(name="adapters-single", op="adapters", tokens=1, k=4096, n=4096, rank=16, adapters=8, dtype="bf16",
             order="mixed", plan="kept", bias=False, act="none", backward=False),
        # A decode step of a batch in which nearly every request has an adapter of its own.
        dict(name="adapters-step", op="adapters", tokens=48, k=4096, n=4096, rank=16, adapters=64, dtype="bf16",
             order="mixed", plan="made", bias=False, act="none", backward=False),
        # The same for a wide projection with a larger rank; the plan serves all of a step's layers.
        dict(name="adapters-step-wide", op="adapters", tokens=64, k=4096, n=12288, rank=64, adapters=32, dtype="bf16",
             order="mixed", plan="kept", bias=False, act="none", backward=False),
        # Prompts of several requests, one after another.
        dict(name="adapters-prefill", op="adapters", tokens=8192, k=4096, n=4096, rank=16, adapters=32, dtype="bf16",
             order="requests", plan="made", bias=False, act="none", backward=False),
        # Odd sizes, a rank that is no power of two, bias and GELU, 16-bit floats.
        dict(name="adapters-ragged", op="adapters", tokens=777, k=1001, n=2504, rank=24, adapters=7, dtype="f16",
             order="mixed", plan="made", bias=True, act="gelu", backward=False),
        # A training step of several adapters at once on a shared frozen projection.
        dict(name="adapters-train", op="adapters", tokens=8192, k=4096, n=4096, rank=32, adapters=4, dtype="bf16",
             order="requests", plan="made", bias=False, act="none", backward=True),
        # A small, ragged one, tokens of the adapters in any order.
        dict(name="adapters-train-ragged", op="adapters", tokens=1000, k=2056, n=1016, rank=8, adapters=5, dtype="bf16",
             order="mixed", plan="made", bias=False, act="none", backward=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    if rng.random() < 0.5:
        backward = rng.random() < 0.5
        tokens = _log_int(rng, 64 if backward else 1, 8192)
        dim = _log_int(rng, 64, 4096)
        vocab = _log_int(rng, 1000, 131072)
        if rng.random() < 0.7:
            dim = max(8, dim // 8 * 8)
        return dict(op="loss", tokens=tokens, dim=dim, vocab=vocab, dtype=rng.choice(("bf16", "bf16", "f16")),
                    layout=rng.choice(("vd", "vd", "dv")), backward=backward,
                    softcap=rng.choice((0.0, 0.0, 20.0, 50.0)), smoothing=rng.choice((0.0, 0.0, 0.1)),
                    z_loss=rng.choice((0.0, 0.0, 1e-3)))
    backward = rng.random() < 0.4
    k, n = (_log_int(rng, 64, 4096) // 8 * 8 for _ in range(2))
    if not backward:                # the activations' rows may start anywhere, and outputs end anywhere
        if rng.random() < 0.3:
            k += rng.randint(1, 7)
        if rng.random() < 0.3:
            n += rng.randint(1, 7)
    return dict(op="adapters", tokens=_log_int(rng, 64 if backward else 1, 8192), k=k, n=n,
                rank=rng.choice((1, 4, 8, 16, 16, 24, 32, 64, 128)), adapters=_log_int(rng, 1, 64),
                dtype=rng.choice(("bf16", "bf16", "f16")), order=rng.choice(("mixed", "requests")),
                plan=rng.choice(("made", "kept")), bias=not backward and rng.random() < 0.3,
                act="none" if backward else rng.choice(("none", "none", "relu", "gelu")), backward=backward)


# ----------------------------------------------------------------- prepare ---
def _padded(shape, dtype):
    """A tensor whose rows start on 16 bytes (weights are laid out so once)."""
    pitch = -(-shape[-1] // 8) * 8
    return torch.empty((*shape[:-1], pitch), dtype=dtype, device="cuda")[..., :shape[-1]]


def _weights(shape, scale, dtype, gen):
    held = _padded(shape, dtype)
    flat = held if held.dim() == 3 else held[None]
    for part in flat:
        rows = max(1, (1 << 27) // part.shape[1])
        for at in range(0, part.shape[0], rows):
            part[at:at + rows] = torch.randn(part[at:at + rows].shape, generator=gen, device="cuda") * scale
    return held


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c, dt = case, TYPES[case["dtype"]]
    if c["op"] == "loss":
        T, D, V = c["tokens"], c["dim"], c["vocab"]
        # logits of spread 1.5; the weights in the layout the model holds them in
        if c["layout"] == "vd":
            W = _weights((V, D), 1.5 * D ** -0.5, dt, gen)
        else:
            W = _weights((D, V), 1.5 * D ** -0.5, dt, gen).t()
        # frequent and rare labels; a part of the positions is padding or prompt and has none
        labels = (V * torch.rand(T, generator=gen, device="cuda", dtype=torch.float64) ** 3).long().clamp_max(V - 1)
        # hidden states point more or less at their label, as a trained model's do
        sure = 4.0 * torch.rand((T, 1), generator=gen, device="cuda")
        H = torch.randn((T, D), generator=gen, device="cuda") + sure * W[labels].float()
        H = H.to(dt)
        labels[torch.rand(T, generator=gen, device="cuda") < 0.1] = -100
        grad = None
        if c["backward"]:                 # of a mean over the positions that have a label
            grad = (1.0 / (labels >= 0).sum().clamp_min(1).float()).expand(T)
        return dict(case=c, H=H, W=W, labels=labels, grad=grad)
    T, K, N, r, L = c["tokens"], c["k"], c["n"], c["rank"], c["adapters"]
    X = torch.randn((T, K), generator=gen, device="cuda").to(dt)
    W = _weights((K, N), K ** -0.5, dt, gen)
    A = _weights((L, r, K), K ** -0.5, dt, gen)
    B = _weights((L, r, N), 0.5 * r ** -0.5, dt, gen)
    scales = 0.5 + 1.5 * torch.rand(L, generator=gen, device="cuda")
    # one request in ten or so runs without an adapter (-1)
    if c["order"] == "mixed":
        ids = torch.randint(0, L, (T,), generator=gen, device="cuda", dtype=torch.int32)
        ids[torch.rand(T, generator=gen, device="cuda") < 0.1] = -1
        if T == 1:
            ids.clamp_min_(0)
    else:
        requests = max(1, T // 512)
        ends = torch.rand(requests, generator=gen, device="cuda").sort().values * T
        whose = torch.randint(-1 if L > 9 else 0, L, (requests + 1,), generator=gen, device="cuda", dtype=torch.int32)
        ids = whose[torch.searchsorted(ends, torch.arange(T, device="cuda", dtype=torch.float32))]
    bias = torch.randn(N, generator=gen, device="cuda") if c["bias"] else None
    grad = torch.randn((T, N), generator=gen, device="cuda").to(dt) if c["backward"] else None
    state = dict(case=c, X=X, W=W, A=A, B=B, scales=scales, ids=ids, bias=bias, grad=grad, plan=None)
    if own and c["plan"] == "kept":
        state["plan"] = _lib().adapter_plan(ids, L, backward=c["backward"])
    return state


# --------------------------------------------------------------------- run ---
def run(state):
    c = state["case"]
    if c["op"] == "loss":
        return (_own_loss if own else _plain_loss)(state)
    return (_own_adapters if own else _plain_adapters)(state)


def _own_loss(st):
    tg, c = _lib(), st["case"]
    how = dict(softcap=c["softcap"], smoothing=c["smoothing"], z_loss=c["z_loss"])
    loss, lse = tg.project_loss(st["H"], st["W"], st["labels"], **how)
    if not c["backward"]:
        return loss, lse
    dH, dW = tg.project_loss_backward(st["grad"], st["H"], st["W"], st["labels"], lse, **how)
    return loss, lse, dH, dW


def _own_adapters(st):
    tg, c = _lib(), st["case"]
    plan = st["plan"]
    if plan is None:
        plan = tg.adapter_plan(st["ids"], c["adapters"], backward=c["backward"])
    y = tg.gemm_adapters(st["X"], st["W"], st["A"], st["B"], plan, scales=st["scales"], bias=st["bias"], act=c["act"])
    if not c["backward"]:
        return y
    dX, dA, dB = tg.gemm_adapters_backward(st["grad"], st["X"], st["W"], st["A"], st["B"], plan, scales=st["scales"])
    return y, dX, dA, dB


def _cap(z, softcap):
    return softcap * torch.tanh(z / softcap) if softcap else z


def _plain_loss(st):
    """The vocabulary in pieces: a running maximum and sum, the label's logit, and for the gradients the pieces again."""
    c, labels = st["case"], st["labels"]
    V = c["vocab"]
    H = st["H"].float()
    T = H.shape[0]
    at = torch.arange(T, device=H.device)
    counted = (labels >= 0) & (labels < V)
    top = torch.full((T,), -math.inf, device=H.device)
    total, mean, hit = (torch.zeros(T, device=H.device) for _ in range(3))
    for v in range(0, V, PIECE):
        z = _cap(H @ st["W"][v:v + PIECE].float().t(), c["softcap"])
        new = torch.maximum(top, z.amax(1))
        total = total * torch.exp(top - new) + torch.exp(z - new[:, None]).sum(1)
        top = new
        if c["smoothing"]:
            mean += z.sum(1)
        here = counted & (labels >= v) & (labels < v + z.shape[1])
        hit = torch.where(here, z[at, (labels - v).clamp(0, z.shape[1] - 1)], hit)
    lse = top + torch.log(total)
    s = c["smoothing"]
    loss = lse - (1.0 - s) * hit - (s / V) * mean + c["z_loss"] * lse * lse
    loss = torch.where(counted, loss, 0.0)
    if not c["backward"]:
        return loss, lse
    g = torch.where(counted, st["grad"], 0.0)
    W, dW = st["W"], torch.empty_like(st["W"])
    dH = torch.zeros_like(H)
    for v in range(0, V, PIECE):
        w = W[v:v + PIECE].float()
        z = _cap(H @ w.t(), c["softcap"])
        d = torch.exp(z - lse[:, None]) * (1.0 + 2.0 * c["z_loss"] * lse)[:, None] - s / V
        here = counted & (labels >= v) & (labels < v + z.shape[1])
        d[at, (labels - v).clamp(0, z.shape[1] - 1)] -= (1.0 - s) * here
        if c["softcap"]:
            d = d * (1.0 - (z / c["softcap"]) ** 2)
        d = d * g[:, None]
        dH += d @ w
        dW[v:v + PIECE] = (d.t() @ H).to(dW.dtype)
    return loss, lse, dH.to(st["H"].dtype), dW


def _plain_act(y, act):
    if act == "relu":
        return y.clamp_min(0.0)
    if act == "gelu":
        return 0.5 * y * (1.0 + torch.erf(y * 0.7071067811865476))
    return y


def _plain_adapters(st):
    """All adapters of all tokens, those that are not a token's masked."""
    c = st["case"]
    L, r, K = st["A"].shape
    T, N = c["tokens"], c["n"]
    X, W = st["X"].float(), st["W"].float()
    A, B = st["A"].float().reshape(L * r, K), st["B"].float().reshape(L * r, N)
    mine = (st["ids"][:, None] == torch.arange(L, device=X.device)) * st["scales"]        # T x L
    S = ((X @ A.t()).view(T, L, r) * mine[:, :, None]).view(T, L * r)
    y = X @ W + S @ B
    if st["bias"] is not None:
        y = y + st["bias"]
    y = _plain_act(y, c["act"]).to(st["X"].dtype)
    if not c["backward"]:
        return y
    G = st["grad"].float()
    U = ((G @ B.t()).view(T, L, r) * mine[:, :, None]).view(T, L * r)
    dX = G @ W.t() + U @ A
    dA, dB = U.t() @ X, S.t() @ G
    dt = st["X"].dtype
    return y, dX.to(dt), dA.view(L, r, K).to(dt), dB.view(L, r, N).to(dt)


# -------------------------------------------------------------------- work ---
def work(case):
    c = case
    if c["op"] == "loss":
        T, D, V = c["tokens"], c["dim"], c["vocab"]
        byte, flops = 2 * (T * D + V * D) + 8 * T + 8 * T, 2 * T * V * D
        if c["backward"]:               # the logits' gradient goes into two more products
            byte, flops = byte + 2 * (T * D + V * D), 3 * flops
        return {"bytes": byte, "flops": flops}
    T, K, N, r = c["tokens"], c["k"], c["n"], c["rank"]
    used = min(c["adapters"], T)
    byte = 2 * (T * K + K * N + used * r * (K + N) + T * N) + 4 * T + (4 * N if c["bias"] else 0)
    flops = 2 * T * K * N + 2 * T * r * (K + N)
    if c["backward"]:
        byte += 2 * (T * N + T * K + c["adapters"] * r * (K + N))
        flops += flops + 2 * T * r * (K + N)
    return {"bytes": byte, "flops": flops}


# ------------------------------------------------------------------- exact ---
def exact(case, seed):
    """The operators from their definitions in 64 bits, on the same inputs."""
    flops = work(case)["flops"] * (4 / 3 if case["op"] == "loss" and case["backward"] else 1)
    if flops > 8e12:                    # (over about 20 seconds in 64 bits)
        return None
    st = prepare(case, seed)
    return (_exact_loss if case["op"] == "loss" else _exact_adapters)(st, case)


def _exact_loss(st, c):
    f64 = torch.float64
    H, W, labels = st["H"].to(f64), st["W"], st["labels"]
    T, V = H.shape[0], c["vocab"]
    loss, lse = torch.zeros(T, dtype=f64, device=H.device), torch.empty(T, dtype=f64, device=H.device)
    dH = torch.zeros_like(H) if c["backward"] else None
    dW = torch.zeros(W.shape, dtype=f64, device=H.device) if c["backward"] else None
    w = W.to(f64)
    rows = max(1, (1 << 28) // V)
    for a in range(0, T, rows):           # some tokens' whole distributions at a time
        h, y = H[a:a + rows], labels[a:a + rows]
        raw = torch.mm(h, w.t())
        z = c["softcap"] * torch.tanh(raw / c["softcap"]) if c["softcap"] else raw
        logp = torch.log_softmax(z, dim=1)
        total = torch.logsumexp(z, dim=1)
        lse[a:a + rows] = total
        has = ((y >= 0) & (y < V)).to(f64)
        target = torch.zeros_like(z).scatter_(1, y.clamp(0, V - 1)[:, None], 1.0)
        target = (1.0 - c["smoothing"]) * target + c["smoothing"] / V
        loss[a:a + rows] = has * (-(target * logp).sum(1) + c["z_loss"] * total ** 2)
        if c["backward"]:
            p = torch.exp(logp)
            d = (p - target + 2.0 * c["z_loss"] * total[:, None] * p) * (has * st["grad"][a:a + rows].to(f64))[:, None]
            if c["softcap"]:
                d = d / torch.cosh(raw / c["softcap"]) ** 2
            dH[a:a + rows] = torch.mm(d, w)
            dW += torch.mm(d.t(), h)
    return (loss, lse, dH, dW) if c["backward"] else (loss, lse)


def _exact_adapters(st, c):
    f64 = torch.float64
    X, W, A, B = (st[n].to(f64) for n in ("X", "W", "A", "B"))
    y = torch.mm(X, W)
    if c["backward"]:
        G = st["grad"].to(f64)
        dX, dA, dB = torch.mm(G, W.t()), torch.zeros_like(A), torch.zeros_like(B)
    for i in range(c["adapters"]):
        t = (st["ids"] == i).nonzero()[:, 0]
        s = float(st["scales"][i])
        if not len(t):
            continue
        low = s * torch.mm(X[t], A[i].t())
        y[t] += torch.mm(low, B[i])
        if c["backward"]:
            up = s * torch.mm(G[t], B[i].t())
            dX[t] += torch.mm(up, A[i])
            dA[i] = torch.mm(up.t(), X[t])
            dB[i] = torch.mm(low.t(), G[t])
    if c["bias"]:
        y = y + st["bias"].to(f64)
    if c["act"] == "relu":
        y = torch.relu(y)
    elif c["act"] == "gelu":
        y = y * torch.special.ndtr(y)
    return (y, dX, dA, dB) if c["backward"] else y
