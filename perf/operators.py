"""Cases and plain forms of the operators around many adapters on one frozen base.

Three operators, each in its public form (``own``) and in a plain form of elementary torch
operations in 32 bits:

* ``fwd`` / ``group``: h = x What^T + s[a] (x A[a]^T) B[a]^T, where every token (row of x)
  names its adapter a in ``ids``; a token whose id is outside 0 .. n - 1 gets the base alone.
  The base is double-quantized NF4 or bf16. ``group`` is the same for the layers of one
  decoding step.
* ``bwd``: its gradients dX, dA[a], dB[a] (those of an adapter sum over its own tokens).
* ``clip``: the 2-norm of each adapter's gradient over a list of tensors, and the list
  scaled by min(1, max_norm / (norm + 1e-6)).
"""
from __future__ import annotations

import math

import torch

own = False

# The layer shapes of the bench's Llama-2-7B set, as (out features, in features).
SET = ((4096, 4096), (4096, 4096), (4096, 4096), (4096, 4096), (11008, 4096), (11008, 4096), (4096, 11008))


def listed():
    def linear(name, op, base, M, N, K, n, r, mix):
        return dict(name=name, op=op, base=base, M=M, N=N, K=K, n=n, r=r, mix=mix)

    return [
        # one user, one token: the latency of a single layer
        linear("decode_1", "fwd", "nf4", 1, 4096, 4096, 8, 16, "tokens"),
        # a full decoding batch of the streaming kernel, most tokens with an adapter of their own
        linear("decode_16", "fwd", "nf4", 16, 11008, 4096, 32, 16, "tokens"),
        # the seven projections of a layer in one decoding step of four users
        dict(name="decode_set_4", op="group", base="nf4", M=4, n=8, r=64, mix="tokens"),
        # a larger decoding batch over many adapters
        linear("batch_64", "fwd", "nf4", 64, 4096, 11008, 64, 16, "tokens"),
        # prompts of a few requests packed together, odd length, the largest rank
        linear("prefill_1531", "fwd", "nf4", 1531, 5120, 5120, 8, 64, "runs"),
        # the same through a layer that stays in 16 bits
        linear("prefill_dense_2048", "fwd", "dense", 2048, 4096, 4096, 4, 16, "runs"),
        # long prompts
        linear("prefill_8192", "fwd", "nf4", 8192, 11008, 4096, 16, 16, "runs"),
        # a tiny ragged training batch: no size a multiple of a tile
        linear("train_333", "bwd", "nf4", 333, 1000, 448, 3, 5, "runs"),
        # four adapters trained on one batch of 4 x 1024 tokens
        linear("train_4096", "bwd", "nf4", 4096, 4096, 4096, 4, 16, "runs"),
        # the widest projection of the 13B-shaped stack
        linear("train_8192", "bwd", "nf4", 8192, 5120, 13824, 8, 64, "runs"),
        # a layer's gradients in 16 bits, four adapters
        dict(name="clip_layer", op="clip", layers=1, n=4, r=8, bf16=True),
        # every adapter gradient of a 32-layer model
        dict(name="clip_model", op="clip", layers=32, n=1, r=16, bf16=False),
    ]


def draw(rng):
    def around(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["fwd", "fwd", "fwd", "bwd", "bwd", "group", "clip"])
    if op == "clip":
        layers, r, n = around(1, 32), around(1, 64), around(1, 8)
        while layers * r * n > 512:
            layers, r, n = max(1, layers // 2), max(1, r // 2), max(1, n - 1)
        return dict(op=op, layers=layers, n=n, r=r, bf16=rng.random() < 0.5)
    if op == "group":
        return dict(op=op, base="nf4", M=rng.randint(1, 16), n=around(1, 16), r=around(1, 64), mix="tokens")
    K = 64 * around(4, 172)
    if op == "fwd":
        M, N = around(1, 8192), around(256, 11008)
    else:
        M, N = around(17, 8192), 8 * around(32, 1376)
    while M * N * K > 8192 * 11008 * 4096:
        M, N = M // 2, (N // 2 + 7) // 8 * 8
    mix = "tokens" if M <= 256 and rng.random() < 0.5 else "runs"
    return dict(op=op, base=rng.choice(["nf4", "nf4", "dense"]), M=M, N=N, K=K, n=around(1, 64 if M <= 256 else 16),
                r=rng.choice([8, 16, 32, 64, rng.randint(1, 64)]), mix=mix)


# ----------------------------------------------------------------------------- inputs
def _levels():
    """The 16 NF4 levels: normal quantiles, 8 above zero and 7 below, scaled to [-1, 1]."""
    top = 1.0 - (1.0 / 32.0 + 1.0 / 30.0) / 2.0
    up = torch.special.ndtri(torch.linspace(0.5, top, 9, dtype=torch.float64))
    down = -torch.special.ndtri(torch.linspace(0.5, top, 8, dtype=torch.float64)).flip(0)
    return (torch.cat([down, up[1:]]) / up[-1]).float().cuda()


def _quantized(W, lv):
    """A bf16 weight as packed NF4 codes with double-quantized block constants."""
    b = W.float().view(-1, 64)
    c = b.abs().amax(1)
    codes = torch.bucketize(b / c[:, None].clamp_min(1e-30), (lv[1:] + lv[:-1]) / 2).to(torch.uint8)
    packed = (codes[:, 0::2] << 4) | codes[:, 1::2]
    mean = c.double().mean().float()
    d = torch.nn.functional.pad(c - mean, (0, -c.numel() % 256)).view(-1, 256)
    scale2 = d.abs().amax(1) / 448.0
    code2 = (d / scale2[:, None].clamp_min(1e-30)).to(torch.float8_e4m3fn).view(torch.uint8).reshape(-1)[: c.numel()]
    return dict(packed=packed.reshape(-1).contiguous(), code2=code2.contiguous(), scale2=scale2.contiguous(),
                mean=mean.reshape(1).contiguous())


def _ids(g, M, n, mix):
    """Adapter of every token: drawn for each token, or runs of tokens (the requests or
    samples of a packed batch); about one in n + 3 names none."""
    if mix == "tokens":
        ids = torch.randint(-1, n + 2, (M,), generator=g, device="cuda")
    else:
        runs = max(1, min(M, 2 * n))
        cuts = torch.sort(torch.randint(0, M, (runs - 1,), generator=g, device="cuda")).values
        of = torch.randint(-1, n + 2, (runs,), generator=g, device="cuda")
        ids = of[torch.searchsorted(cuts, torch.arange(M, device="cuda"), right=True)]
    return torch.where(ids < n, ids, ids - n).to(torch.int32)


def _normal(g, std, *shape):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def _layer(g, c, N, K, lv):
    W = _normal(g, 0.02, N, K)
    return dict(N=N, K=K, **(_quantized(W, lv) if c["base"] == "nf4" else dict(W=W)), x=_normal(g, 1.0, c["M"], K),
                A=_normal(g, 0.02, c["n"], c["r"], K), B=_normal(g, 0.05, c["n"], N, c["r"]))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = dict(case)
    if c["op"] == "clip":
        dt = torch.bfloat16 if c["bf16"] else torch.float32
        shapes = [s for _ in range(c["layers"]) for N, K in SET for s in ((c["n"], c["r"], K), (c["n"], N, c["r"]))]
        size = torch.rand(len(shapes), generator=g, device="cuda").tolist()
        grads = [(torch.randn(s, generator=g, device="cuda") * (0.02 * v)).to(dt) for s, v in zip(shapes, size)]
        # the trainer keeps the scaled gradients in one flat buffer
        flat = torch.empty(sum(t.numel() for t in grads), dtype=dt, device="cuda")
        views = [v.view(s) for v, s in zip(flat.split([t.numel() for t in grads]), shapes)]
        return dict(c=c, grads=grads, flat=flat, views=views, max_norm=0.3)
    lv = _levels()
    s = dict(c=c, lv=lv, ids=_ids(g, c["M"], c["n"], c["mix"]),
             scales=32.0 / c["r"] * (0.5 + torch.rand(c["n"], generator=g, device="cuda")))
    s["layers"] = [_layer(g, c, N, K, lv) for N, K in (SET if c["op"] == "group" else ((c["N"], c["K"]),))]
    if c["op"] == "bwd":
        s["dY"] = _normal(g, 1.0, c["M"], c["N"])
    return s


# ----------------------------------------------------------------------------- one pass
def run(state):
    c = state["c"]
    if c["op"] == "clip":
        return _own_clip(state) if own else _plain_clip(state)
    if c["op"] == "group":
        return _own_group(state) if own else [_plain_fwd(state, s) for s in state["layers"]]
    if c["op"] == "fwd":
        return _own_fwd(state, state["layers"][0]) if own else _plain_fwd(state, state["layers"][0])
    return _own_bwd(state, state["layers"][0]) if own else _plain_bwd(state, state["layers"][0])


def _base(q, s):
    return s["W"] if "W" in s else q.Nf4Weight(s["N"], s["K"], s["packed"], s["code2"], s["scale2"], s["mean"])


def _own_fwd(state, s):
    import bit_nf4_quantized_04_b200 as q
    f = q.dense_linear_multi_fwd if "W" in s else q.qlora_linear_multi_fwd
    return f(_base(q, s), s["x"], state["ids"], s["A"], s["B"], state["scales"])


def _own_group(state):
    import bit_nf4_quantized_04_b200 as q
    L = state["layers"]
    return q.qlora_linear_multi_fwd_group([_base(q, s) for s in L], [s["x"] for s in L], state["ids"],
                                          [s["A"] for s in L], [s["B"] for s in L], state["scales"])


def _own_bwd(state, s):
    import bit_nf4_quantized_04_b200 as q
    f = q.dense_linear_multi_bwd if "W" in s else q.qlora_linear_multi_bwd
    return f(_base(q, s), s["x"], state["dY"], state["ids"], s["A"], s["B"], state["scales"])


def _own_clip(state):
    import bit_nf4_quantized_04_b200 as q
    _, norm = q.clip_grad_norm(state["grads"], state["max_norm"], n=state["c"]["n"], out=state["views"])
    return state["flat"], norm


def _weight(state, s):
    """The fp32 weight a layer's stored form stands for."""
    if "W" in s:
        return s["W"].float()
    p = s["packed"]
    codes = torch.stack([p >> 4, p & 15], 1).view(-1, 64)
    const = s["code2"].view(torch.float8_e4m3fn).float() * s["scale2"].repeat_interleave(256)[: s["code2"].numel()] + s["mean"]
    return (state["lv"][codes.int()] * const[:, None]).view(s["N"], s["K"])


def _own_scale(state):
    """[M, n]: the adapter's scale where a token names it, else zero."""
    n = state["c"]["n"]
    return (state["ids"][:, None] == torch.arange(n, device="cuda")).float() * state["scales"]


def _plain_fwd(state, s):
    n, r = state["c"]["n"], state["c"]["r"]
    x = s["x"].float()
    u = (x @ s["A"].float().view(n * r, -1).T).view(-1, n, r) * _own_scale(state)[:, :, None]
    h = x @ _weight(state, s).T + u.reshape(-1, n * r) @ s["B"].float().transpose(1, 2).reshape(n * r, -1)
    return h.to(torch.bfloat16)


def _plain_bwd(state, s):
    n, r = state["c"]["n"], state["c"]["r"]
    x, dY, of = s["x"].float(), state["dY"].float(), _own_scale(state)[:, :, None]
    A = s["A"].float().view(n * r, -1)
    Bt = s["B"].float().transpose(1, 2).reshape(n * r, -1)
    u = ((x @ A.T).view(-1, n, r) * of).view(-1, n * r)
    v = ((dY @ Bt.T).view(-1, n, r) * of).view(-1, n * r)
    dX = (dY @ _weight(state, s) + v @ A).to(torch.bfloat16)
    dA = (v.T @ x).view(n, r, -1)
    dB = (dY.T @ u).view(-1, n, r).transpose(0, 1).contiguous()
    return dX, dA, dB


def _plain_clip(state):
    n = state["c"]["n"]
    norm = torch.stack([t.float().view(n, -1).square().sum(1) for t in state["grads"]]).sum(0).sqrt()
    coef = (state["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    torch.cat([(t.float() * coef.view(n, 1, 1)).to(t.dtype).view(-1) for t in state["grads"]], out=state["flat"])
    return state["flat"], norm


# ----------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "clip":
        m = c["layers"] * c["n"] * c["r"] * sum(N + K for N, K in SET)
        return dict(bytes=m * (4 if c["bf16"] else 8), flops=3 * m)
    M, n, r = c["M"], c["n"], c["r"]
    used = min(n, M)  # adapters that some token can name
    total = dict(bytes=4 * M + 4 * n, flops=0)
    for N, K in SET if c["op"] == "group" else ((c["N"], c["K"]),):
        base = N * K * 2 if c["base"] == "dense" else N * K // 2 + N * K // 64 + N * K // 4096 + 4
        total["bytes"] += base + 2 * M * (N + K) + 2 * used * r * (N + K)
        total["flops"] += 2 * M * N * K + 2 * M * r * (N + K)
        if c["op"] == "bwd":  # dX, and dA and dB of every adapter in fp32
            total["bytes"] += 2 * M * K + 4 * n * r * (N + K)
            total["flops"] += 2 * M * r * (N + K) + 2 * M * r * K
    return total


# ----------------------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    state = prepare(case, seed)
    c = state["c"]
    if c["op"] == "clip":
        sq = torch.zeros(c["n"], dtype=torch.float64, device="cuda")
        for t in state["grads"]:
            for a in range(c["n"]):
                sq[a] += t[a].double().norm() ** 2
        factor = torch.minimum(torch.ones_like(sq), state["max_norm"] / (sq.sqrt() + 1e-6))
        return torch.cat([(t[a].double() * factor[a]).flatten() for t in state["grads"] for a in range(c["n"])]), sq.sqrt()
    outs = []
    for s in state["layers"]:
        W = torch.empty(s["N"] * s["K"], dtype=torch.float64, device="cuda")
        if "W" in s:
            W.copy_(s["W"].view(-1))
        else:
            W[0::2] = state["lv"].double().index_select(0, (s["packed"] // 16).int())
            W[1::2] = state["lv"].double().index_select(0, (s["packed"] % 16).int())
            block = torch.arange(s["code2"].numel(), device="cuda")
            W.view(-1, 64).mul_((s["code2"].view(torch.float8_e4m3fn).double() * s["scale2"].double()[block // 256]
                                 + s["mean"].double())[:, None])
        W = W.view(s["N"], s["K"])
        x = s["x"].double()
        if c["op"] == "bwd":
            dY = state["dY"].double()
            dX = dY @ W
            dA = torch.zeros(s["A"].shape, dtype=torch.float64, device="cuda")
            dB = torch.zeros(s["B"].shape, dtype=torch.float64, device="cuda")
        else:
            h = x @ W.T
        for a in range(c["n"]):
            at = torch.nonzero(state["ids"] == a).flatten()
            if not at.numel():
                continue
            Aa, Ba, f = s["A"][a].double(), s["B"][a].double(), state["scales"][a].double()
            if c["op"] == "bwd":
                dX[at] += f * (dY[at] @ Ba) @ Aa
                dA[a] = f * (dY[at] @ Ba).T @ x[at]
                dB[a] = f * dY[at].T @ (x[at] @ Aa.T)
            else:
                h[at] += f * (x[at] @ Aa.T) @ Ba.T
        outs.append((dX, dA, dB) if c["op"] == "bwd" else h)
    return outs if c["op"] == "group" else outs[0]
