"""The many-adapter linear layer and its gradients against float64.

Bounds, elementwise, with u = 2^-24 and b = 2^-8 (half a step of bf16):
* the adapter product alone (a base whose weight is zero): s u enters as bf16, so at most
  b |su| |B|^T, the output is rounded once, b |h|, and the sums are fp32: a tensor-core sum
  of C products makes C / 16 additions, each off by at most one step, 2 u, of the running
  sum, which the sum of magnitudes bounds;
* dX likewise; dA and dB are fp32 sums over tokens of projections held as three bf16 parts,
  whose remainder is at most b^3 of the value: (b^3 + 2 u (M / 16 + 64)) sum |P| |X|
  + 2 u (C / 16 + 64) sum |X| (magnitude of P's own contraction).
With a nonzero base the weight's own rounding to bf16 joins: b per weight (three roundings of
b where few tokens take the table lookup), independent from weight to weight, so the whole
output is held to (3 + 2) b in the 2-norm, beside the bounds of the two parts above.
"""
import pytest
import torch

import multi_ref
import synth

pytestmark = pytest.mark.gpu

U2 = 2.0 ** -23
BF = 2.0 ** -8

CASES = [  # N, K, M, n, r, ids
    (256, 512, 1, 1, 8, "one"), (256, 512, 1, 4, 16, "none"), (40, 448, 5, 3, 4, "tokens"),
    (1000, 4096, 16, 32, 16, "tokens"), (200, 192, 17, 2, 17, "tokens"), (512, 640, 33, 40, 16, "tokens"),
    (384, 640, 64, 64, 64, "tokens"), (264, 960, 130, 5, 33, "runs"), (136, 1024, 300, 8, 8, "wild"),
    (320, 512, 700, 7, 48, "runs"), (1024, 2048, 513, 300, 1, "tokens"), (2048, 1024, 2048, 6, 16, "runs"),
    (128, 64, 256, 2, 64, "none"), (4096, 4096, 1025, 3, 32, "runs"),
    # the product over a 16-bit base: ranks of each padded width, many adapters per tile, none, one
    (264, 448, 800, 9, 33, "tokens"), (512, 192, 900, 40, 8, "tokens"), (1000, 320, 769, 2, 64, "one"),
    (256, 64, 1024, 4, 17, "none"), (136, 576, 1500, 12, 3, "wild"),
]


def _inputs(N, K, M, n, r, mix, seed):
    x = synth.normal_bf16((M, K), 1.0, seed, "cuda")
    A = synth.normal_bf16((n, r, K), 0.05, seed + 1, "cuda")
    B = synth.normal_bf16((n, N, r), 0.05, seed + 2, "cuda")
    dY = synth.normal_bf16((M, N), 1.0, seed + 3, "cuda")
    ids = multi_ref.make_ids(mix, M, n, seed + 4, "cuda")
    scales = (0.5 + torch.rand(n, generator=torch.Generator().manual_seed(seed))).cuda()
    return x, A, B, dY, ids, scales


def _base(q, kind, W):
    if kind == "nf4":
        w = q.quantize_weight(W)
        return w, q.dequant(w), q.qlora_linear_multi_fwd, q.qlora_linear_multi_bwd
    return W, W, q.dense_linear_multi_fwd, q.dense_linear_multi_bwd


def _within(got, want, bound, what):
    assert bool(torch.isfinite(got).all()), what
    over = (got.double() - want).abs() - bound
    assert over.max().item() <= 0, f"{what}: {over.max().item():.3e} beyond its bound"


def _norm_off(got, want):
    return ((got.double() - want).norm() / want.norm().clamp_min(1e-300)).item()


def _check_fwd(q, kind, N, K, M, n, r, mix, seed):
    x, A, B, _, ids, s = _inputs(N, K, M, n, r, mix, seed)
    for W in (torch.zeros(N, K, dtype=torch.bfloat16, device="cuda"), synth.llama_weight((N, K), seed, device="cuda")):
        base, What, fwd, _ = _base(q, kind, W)
        h = fwd(base, x, ids, A, B, s)
        q.check()
        want, mag, magw = multi_ref.forward(What, x, ids, A, B, s)
        if not bool(What.any()):
            _within(h, want, BF * want.abs() * 1.01 + BF * 1.01 * mag + U2 * ((K + 64 * n) / 16 + 64) * mag * 2, "h")
        else:
            assert _norm_off(h, want) <= 5 * BF
            if mix == "none":
                assert torch.equal(h, fwd(base, x, ids, A * 0, B, s))


def _check_bwd(q, kind, N, K, M, n, r, mix, seed):
    x, A, B, dY, ids, s = _inputs(N, K, M, n, r, mix, seed)
    for W in (torch.zeros(N, K, dtype=torch.bfloat16, device="cuda"), synth.llama_weight((N, K), seed, device="cuda")):
        base, What, _, bwd = _base(q, kind, W)
        dX, dA, dB = bwd(base, x, dY, ids, A, B, s)
        q.check()
        (wX, mX, mW), (wA, pA, cA), (wB, pB, cB) = multi_ref.backward(What, x, dY, ids, A, B, s)
        if not bool(What.any()):
            _within(dX, wX, BF * wX.abs() * 1.01 + BF * 1.01 * mX + U2 * ((N + 64 * n) / 16 + 64) * mX * 2, "dX")
        else:
            assert _norm_off(dX, wX) <= 5 * BF
        tok = BF ** 3 + U2 * (M / 16 + 64)
        _within(dA, wA, tok * pA + U2 * (N / 16 + 64) * cA, "dA")
        _within(dB, wB, tok * pB + U2 * (K / 16 + 64) * cB, "dB")
        for a in range(n):
            if not bool((ids == a).any()):
                assert not bool(dA[a].any()) and not bool(dB[a].any())


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("kind", ["nf4", "dense"])
def test_forward(case, kind):
    import bit_nf4_quantized_04_b200 as q
    _check_fwd(q, kind, *case, 300)


@pytest.mark.parametrize("case", [(333, 320, 257, 3, 5, "runs"), (17, 64, 9, 2, 3, "tokens"),
                                  (131, 128, 40, 9, 64, "tokens")], ids=str)
@pytest.mark.parametrize("kind", ["nf4", "dense"])
def test_forward_of_odd_output_widths(case, kind):
    import bit_nf4_quantized_04_b200 as q
    _check_fwd(q, kind, *case, 310)


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("kind", ["nf4", "dense"])
def test_backward(case, kind):
    import bit_nf4_quantized_04_b200 as q
    _check_bwd(q, kind, *case, 320)


@pytest.mark.parametrize("M", [3, 16, 40, 300, 900])
def test_tokens_of_one_adapter_get_what_the_single_adapter_call_gives(M):
    import bit_nf4_quantized_04_b200 as q
    N, K, n, r = 512, 1024, 4, 16
    x, A, B, dY, ids, s = _inputs(N, K, M, n, r, "tokens", 330)
    w = q.quantize_weight(synth.llama_weight((N, K), 330, device="cuda"))
    h = q.qlora_linear_multi_fwd(w, x, ids, A, B, s)
    dX, _, _ = q.qlora_linear_multi_bwd(w, x, dY, ids, A, B, s)
    for a in range(n):
        at = multi_ref.tokens_of(ids, a)
        if at.numel():
            one = q.qlora_linear_fwd(w, x, A[a].contiguous(), B[a].contiguous(), s[a].item())
            # s u may fall on the other side of a bf16 step: two steps of the result
            assert _norm_off(h[at], one[at].double()) <= 2 * BF
            d1 = q.qlora_linear_bwd(w, x, dY, A[a].contiguous(), B[a].contiguous(), s[a].item())[0]
            assert _norm_off(dX[at], d1[at].double()) <= 2 * BF


@pytest.mark.parametrize("M", [1, 16, 40, 300, 600, 900])
@pytest.mark.parametrize("kind", ["nf4", "dense"])
def test_a_broken_adapter_reaches_its_own_tokens_only(M, kind):
    # adapter 1 holds NaN, +inf and -inf in single rows: its tokens get them there, by IEEE
    # arithmetic, and every other token what it gets without them
    import bit_nf4_quantized_04_b200 as q
    N, K, n, r = 264, 320, 5, 8
    x, A, B, dY, ids, s = _inputs(N, K, M, n, r, "tokens", 340)
    if M == 1:
        ids.fill_(1)
    base, _, fwd, bwd = _base(q, kind, synth.llama_weight((N, K), 340, device="cuda"))
    good = fwd(base, x, ids, A, B, s)
    goodX, goodA, goodB = bwd(base, x, dY, ids, A, B, s)
    B2, A2 = B.clone(), A.clone()
    B2[1, 3, 2], B2[1, 100, 0], B2[1, 263, 7] = float("nan"), float("inf"), float("-inf")
    h = fwd(base, x, ids, A, B2, s)
    mine = ids == 1
    assert torch.equal(h[~mine], good[~mine])
    keep = torch.ones(N, dtype=torch.bool, device="cuda")
    keep[[3, 100, 263]] = False
    assert torch.equal(h[mine][:, keep], good[mine][:, keep])
    if bool(mine.any()):
        u = x[mine].double() @ A[1].double().T
        assert bool(h[mine][:, 3].isnan().all())
        assert torch.equal(h[mine][:, 100], torch.where(u[:, 0] > 0, float("inf"), float("-inf")).bfloat16())
        assert torch.equal(h[mine][:, 263], torch.where(u[:, 7] > 0, float("-inf"), float("inf")).bfloat16())
    A2[1, 4, 5], A2[1, 0, 319] = float("nan"), float("inf")
    dX, dA, dB = bwd(base, x, dY, ids, A2, B, s)
    assert torch.equal(dX[~mine], goodX[~mine])
    keep = torch.ones(K, dtype=torch.bool, device="cuda")
    keep[[5, 319]] = False
    assert torch.equal(dX[mine][:, keep], goodX[mine][:, keep])
    if bool(mine.any()):
        assert bool(dX[mine][:, 5].isnan().all()) and bool(dX[mine][:, 319].isinf().all())
    others = [a for a in range(n) if a != 1]
    assert torch.equal(dA[others], goodA[others]) and torch.equal(dB[others], goodB[others])
    q.check()


@pytest.mark.parametrize("M", [16, 300, 900])
def test_a_broken_token_stays_alone(M):
    # infinities and NaNs in one token's x and dY: other tokens, and adapters without that
    # token, keep their values
    import bit_nf4_quantized_04_b200 as q
    N, K, n, r = 264, 320, 5, 8
    x, A, B, dY, ids, s = _inputs(N, K, M, n, r, "tokens", 350)
    ids[7] = 2
    w = q.quantize_weight(synth.llama_weight((N, K), 350, device="cuda"))
    good, grads = q.qlora_linear_multi_fwd(w, x, ids, A, B, s), q.qlora_linear_multi_bwd(w, x, dY, ids, A, B, s)
    x[7, 11], dY[7, 13] = float("inf"), float("nan")
    h, bad = q.qlora_linear_multi_fwd(w, x, ids, A, B, s), q.qlora_linear_multi_bwd(w, x, dY, ids, A, B, s)
    q.check()
    rows = [m for m in range(M) if m != 7]
    ads = [a for a in range(n) if a != 2]
    assert torch.equal(h[rows], good[rows]) and torch.equal(bad[0][rows], grads[0][rows])
    assert torch.equal(bad[1][ads], grads[1][ads]) and torch.equal(bad[2][ads], grads[2][ads])
    assert not bool(torch.isfinite(bad[1][2]).all()) and not bool(torch.isfinite(h[7]).all())


def test_gradient_of_b_against_differences():
    # with a zero base h is linear in B: <dB, d> = sum dY (h(B + d) - h(B)), up to the
    # roundings of the two outputs and of s u (which is the same in both)
    import bit_nf4_quantized_04_b200 as q
    N, K, M, n, r = 128, 256, 200, 3, 8
    x, A, B, dY, ids, s = _inputs(N, K, M, n, r, "runs", 360)
    d = synth.normal_bf16((n, N, r), 0.5, 361, "cuda")
    B = (B * 0).bfloat16()
    w = q.quantize_weight(torch.zeros(N, K, dtype=torch.bfloat16, device="cuda"))
    h1 = q.qlora_linear_multi_fwd(w, x, ids, A, B + d, s).double()
    h0 = q.qlora_linear_multi_fwd(w, x, ids, A, B, s).double()
    dB = q.qlora_linear_multi_bwd(w, x, dY, ids, A, B, s)[2].double()
    q.check()
    _, mag, _ = multi_ref.forward(torch.zeros(N, K, device="cuda"), x, ids, A, d, s)
    bound = (dY.double().abs() * (2 * BF * h1.abs() + 2 * BF * mag)).sum().item()
    diff = (dY.double() * (h1 - h0)).sum().item()
    assert h0.abs().max().item() == 0 and abs((dB * d.double()).sum().item() - diff) <= bound
    assert abs(diff) > 3 * bound or (dB * d.double()).abs().sum().item() > 3 * bound


@pytest.mark.parametrize("M", [4, 300, 900])
def test_same_bits_every_time_and_in_graphs(M):
    # two captured graphs that share one workspace, replayed in turn on one stream, on the
    # inputs' new values: each equals the eager call
    import bit_nf4_quantized_04_b200 as q
    N, K, n, r = 512, 448, 3, 16
    x, A, B, dY, ids, s = _inputs(N, K, M, n, r, "runs", 370)
    w = q.quantize_weight(synth.llama_weight((N, K), 370, device="cuda"))
    ws = torch.empty(max(q.multi_workspace_size(op, N, K, M, n, r) for op in (q._lib.OP_FWD, q._lib.OP_BWD)),
                     dtype=torch.uint8, device="cuda")
    h = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    outs = q.qlora_linear_multi_bwd(w, x, dY, ids, A, B, s, ws=ws)
    q.qlora_linear_multi_fwd(w, x, ids, A, B, s, h=h, ws=ws)
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        q.qlora_linear_multi_fwd(w, x, ids, A, B, s, h=h, ws=ws)
    with torch.cuda.graph(g2):
        q.qlora_linear_multi_bwd(w, x, dY, ids, A, B, s, *outs, ws=ws)
    for k in range(3):
        ids.copy_(multi_ref.make_ids("tokens" if k else "runs", M, n, 380 + k))
        x.copy_(synth.normal_bf16((M, K), 1.0, 390 + k))
        want = [q.qlora_linear_multi_fwd(w, x, ids, A, B, s), *q.qlora_linear_multi_bwd(w, x, dY, ids, A, B, s)]
        h.fill_(float("nan"))
        for t in outs:
            t.fill_(float("nan"))
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip([h, *outs], want))


def test_no_tokens():
    import bit_nf4_quantized_04_b200 as q
    N, K, n, r = 128, 64, 3, 4
    x, A, B, dY, ids, s = _inputs(N, K, 0, n, r, "none", 400)
    w = q.quantize_weight(synth.llama_weight((N, K), 400, device="cuda"))
    assert q.qlora_linear_multi_fwd(w, x, ids, A, B, s).shape == (0, N)
    dA, dB = torch.full((n, r, K), 7.0, device="cuda"), torch.full((n, N, r), 7.0, device="cuda")
    dX, dA, dB = q.qlora_linear_multi_bwd(w, x, dY, ids, A, B, s, dA=dA, dB=dB)
    assert dX.shape == (0, K) and not bool(dA.any()) and not bool(dB.any())


@pytest.mark.parametrize("M,r", [(1, 16), (4, 64), (16, 5)])
def test_group_equals_single_calls(M, r):
    import bit_nf4_quantized_04_b200 as q
    n = 5
    shapes = [(512, 512), (200, 448), (1000, 512), (512, 1024), (64, 64)]
    ids = multi_ref.make_ids("tokens", M, n, 410, "cuda")
    s = (0.5 + torch.rand(n)).cuda()
    ws_, xs, As, Bs = [], [], [], []
    for i, (N, K) in enumerate(shapes):
        ws_.append(q.quantize_weight(synth.llama_weight((N, K), 420 + i, device="cuda")))
        xs.append(synth.normal_bf16((M, K), 1.0, 430 + i, "cuda"))
        As.append(synth.normal_bf16((n, r, K), 0.05, 440 + i, "cuda"))
        Bs.append(synth.normal_bf16((n, N, r), 0.05, 450 + i, "cuda"))
    hs = q.qlora_linear_multi_fwd_group(ws_, xs, ids, As, Bs, s)
    q.check()
    for i in range(len(shapes)):
        assert torch.equal(hs[i], q.qlora_linear_multi_fwd(ws_[i], xs[i], ids, As[i], Bs[i], s))


def test_a_step_of_several_adapters_forward_backward_clip():
    # the operators together, as a trainer of several adapters uses them: two layers, the
    # loss's gradient at the output, each adapter's gradients clipped by its own norm
    import bit_nf4_quantized_04_b200 as q
    M, n, r, D = 190, 3, 8, 256
    ids = multi_ref.make_ids("runs", M, n, 500, "cuda")
    s = torch.tensor([2.0, 1.0, 0.5], device="cuda")
    W = [synth.llama_weight((D, D), 501 + i, std=0.06, device="cuda") for i in range(2)]
    bases = [q.quantize_weight(W[0]), W[1]]  # the second layer is protected: 16 bits
    A = [synth.normal_bf16((n, r, D), 0.05, 510 + i, "cuda") for i in range(2)]
    B = [synth.normal_bf16((n, D, r), 0.05, 520 + i, "cuda") for i in range(2)]
    x = synth.normal_bf16((M, D), 1.0, 530, "cuda")
    h1 = q.qlora_linear_multi_fwd(bases[0], x, ids, A[0], B[0], s)
    y = q.dense_linear_multi_fwd(bases[1], h1, ids, A[1], B[1], s)
    dY = y.clone()  # loss = sum y^2 / 2
    d1, dA1, dB1 = q.dense_linear_multi_bwd(bases[1], h1, dY, ids, A[1], B[1], s)
    _, dA0, dB0 = q.qlora_linear_multi_bwd(bases[0], x, d1, ids, A[0], B[0], s)
    grads = [dA0, dB0, dA1, dB1]
    keep = [t.clone() for t in grads]
    out, norm = q.clip_grad_norm(grads, 1.0, n=n, out=grads)
    q.check()
    # every gradient from its call's own inputs, in float64
    _, (a1, pa1, ca1), (b1, pb1, cb1) = multi_ref.backward(W[1], h1, dY, ids, A[1], B[1], s)
    _, (a0, pa0, ca0), (b0, pb0, cb0) = multi_ref.backward(q.dequant(bases[0]), x, d1, ids, A[0], B[0], s)
    want, mags = [a0, b0, a1, b1], [(pa0, ca0), (pb0, cb0), (pa1, ca1), (pb1, cb1)]
    for g, w, (p, c) in zip(keep, want, mags):
        _within(g, w, (BF ** 3 + U2 * (M / 16 + 64)) * p + U2 * (D / 16 + 64) * c, "gradient")
    exact = torch.stack([t.double().reshape(n, -1).square().sum(1) for t in keep]).sum(0).sqrt()
    assert bool(((norm.double() - exact).abs() <= 1.01 * 2.0 ** -24 * exact).all())
    for g, k in zip(out, keep):
        ref = k.double() * (1.0 / (exact + 1e-6)).clamp(max=1.0)[:, None, None]
        assert bool(((g.double() - ref).abs() <= 4.01 * 2.0 ** -24 * ref.abs()).all())


def test_refusals_of_the_binding():
    import bit_nf4_quantized_04_b200 as q
    N, K, M, n, r = 128, 64, 5, 3, 4
    x, A, B, dY, ids, s = _inputs(N, K, M, n, r, "tokens", 540)
    w = q.quantize_weight(synth.llama_weight((N, K), 540, device="cuda"))
    f = q.qlora_linear_multi_fwd
    for args in [(x[:, :32].contiguous(), ids, A, B, s), (x, ids[:4].contiguous(), A, B, s),
                 (x, ids, A[:2].contiguous(), B, s), (x, ids, A, B[:, :64].contiguous(), s),
                 (x, ids, A, B, s[:2].contiguous()), (x, ids.cpu(), A, B, s), (x.t(), ids, A, B, s),
                 (x, ids, A[0], B[0], s)]:
        with pytest.raises(ValueError):
            f(w, *args)
    for args in [(x, ids.long(), A, B, s), (x.float(), ids, A, B, s), (x, ids, A, B, s.double())]:
        with pytest.raises(TypeError):
            f(w, *args)
    with pytest.raises(ValueError):
        f(w, x, ids, A, B, s, h=torch.empty(M, N + 1, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        f(w, x, ids, A, B, s, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        q.qlora_linear_multi_bwd(w, x, dY[:, :64].contiguous(), ids, A, B, s)
    big = torch.zeros(n, 65, K, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(q.Qnf4Error, match="ERR_ARG"):
        f(w, x, ids, big, torch.zeros(n, N, 65, dtype=torch.bfloat16, device="cuda"), s)
    with pytest.raises(ValueError):
        q.qlora_linear_multi_fwd_group([w], [torch.zeros(17, K, dtype=torch.bfloat16, device="cuda")],
                                       torch.zeros(17, dtype=torch.int32, device="cuda"), [A], [B], s)


@pytest.mark.parametrize("case", [(1000, 704, 1100, 4, 16, "runs"), (2560, 1280, 2500, 3, 24, "runs"),
                                  (256, 6400, 256, 2, 8, "runs"), (4864, 256, 1030, 5, 64, "runs"),
                                  (4096, 1024, 4096, 3, 16, "runs")], ids=str)
@pytest.mark.parametrize("kind", ["nf4", "dense"])
def test_long_contractions_and_partial_tiles(case, kind):
    # few tiles with long contractions, and sizes just past a tile; twice for equal bits
    import bit_nf4_quantized_04_b200 as q
    _check_fwd(q, kind, *case, 600)
    _check_bwd(q, kind, *case, 610)
    N, K, M, n, r, mix = case
    x, A, B, dY, ids, s = _inputs(N, K, M, n, r, mix, 620)
    base, _, fwd, bwd = _base(q, kind, synth.llama_weight((N, K), 620, device="cuda"))
    one, two = [[fwd(base, x, ids, A, B, s), *bwd(base, x, dY, ids, A, B, s)] for _ in range(2)]
    assert all(torch.equal(a, b) for a, b in zip(one, two))


@pytest.mark.parametrize("M", [7, 130, 900])
def test_the_most_adapters(M):
    """The limit on adapters (4096), the last of them named, with few tokens for each."""
    import bit_nf4_quantized_04_b200 as q
    N, K, n, r = 64, 128, 4096, 2
    x, A, B, dY, ids, s = _inputs(N, K, M, n, r, "tokens", 551)
    ids[M // 2] = n - 1
    w = q.quantize_weight(torch.zeros(N, K, dtype=torch.bfloat16, device="cuda"))
    for base, fwd, bwd in ((w, q.qlora_linear_multi_fwd, q.qlora_linear_multi_bwd),
                           (q.dequant(w).bfloat16(), q.dense_linear_multi_fwd, q.dense_linear_multi_bwd)):
        h = fwd(base, x, ids, A, B, s)
        dX, dA, dB = bwd(base, x, dY, ids, A, B, s)
        q.check()
        want, mag, _ = multi_ref.forward(q.dequant(w), x, ids, A, B, s)
        _within(h, want, BF * want.abs() * 1.01 + BF * 1.01 * mag + U2 * (K / 16 + 64) * mag * 2, "h")
        (wX, mX, _), (wA, pA, cA), (wB, pB, cB) = multi_ref.backward(q.dequant(w), x, dY, ids, A, B, s)
        _within(dX, wX, BF * wX.abs() * 1.01 + BF * 1.01 * mX + U2 * (N / 16 + 64) * mX * 2, "dX")
        tok = BF ** 3 + U2 * (M / 16 + 64)
        _within(dA, wA, tok * pA + U2 * (N / 16 + 64) * cA, "dA")
        _within(dB, wB, tok * pB + U2 * (K / 16 + 64) * cB, "dB")
    with pytest.raises(q.Qnf4Error, match="ERR_ARG"):
        q.qlora_linear_multi_fwd(w, x, ids, torch.cat([A, A[:1]]), torch.cat([B, B[:1]]), torch.cat([s, s[:1]]))


def test_a_base_on_another_device_is_refused():
    import bit_nf4_quantized_04_b200 as q
    N, K, M, n, r = 128, 64, 5, 3, 4
    x, A, B, dY, ids, s = _inputs(N, K, M, n, r, "tokens", 552)
    W = synth.llama_weight((N, K), 552, device="cuda")
    w = q.quantize_weight(W)
    far = q.Nf4Weight(N, K, w.packed, w.code2.cpu(), w.scale2, w.mean)
    with pytest.raises(ValueError, match="base weight"):
        q.qlora_linear_multi_fwd(far, x, ids, A, B, s)
    with pytest.raises(ValueError, match="base weight"):
        q.qlora_linear_multi_fwd_group([w, far], [x, x], ids, [A, A], [B, B], s)
    with pytest.raises(ValueError, match="base weight"):
        q.qlora_linear_multi_bwd(far, x, dY, ids, A, B, s)
    for f, args in ((q.dense_linear_multi_fwd, (x,)), (q.dense_linear_multi_bwd, (x, dY))):
        with pytest.raises(ValueError):
            f(W.cpu(), *args, ids, A, B, s)


def test_outputs_that_overlap_an_argument_are_refused():
    import bit_nf4_quantized_04_b200 as q
    N = K = 128
    M, n, r = 64, 3, 4
    x, A, B, dY, ids, s = _inputs(N, K, M, n, r, "tokens", 553)
    w = q.quantize_weight(synth.llama_weight((N, K), 553, device="cuda"))
    dA = torch.empty(n, r, K, device="cuda")
    room = torch.empty(M + 1, N, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="overlaps"):
        q.qlora_linear_multi_fwd(w, x, ids, A, B, s, h=x)
    for kw in (dict(dX=x), dict(dX=dY), dict(dA=dA, dB=dA.view(n, N, r))):
        with pytest.raises(ValueError, match="overlaps"):
            q.qlora_linear_multi_bwd(w, x, dY, ids, A, B, s, **kw)
    with pytest.raises(ValueError, match="overlaps"):
        q.qlora_linear_multi_fwd_group([w, w], [x[:8], x[:8]], ids[:8], [A, A], [B, B], s, hs=[room[:8], room[4:12]])
    # neighbours are no overlap
    h = q.qlora_linear_multi_fwd(w, x, ids, A, B, s, h=room[1:])
    assert torch.equal(h, q.qlora_linear_multi_fwd(w, x, ids, A, B, s))
