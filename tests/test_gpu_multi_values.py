"""Infinities and NaNs in x and dY, through the many-adapter layer and its gradients: every output
element is what IEEE arithmetic gives for its formula (a sum of products is NaN where a term is, or
where infinities of both signs meet, else infinite with the sign of its infinite terms), and the
elements that meet no such value keep their bits. No tolerances."""
import pytest
import torch

import multi_ref
import synth
from test_gpu_multi import _base, _inputs

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def _mm(a, b):
    """a @ b in float64, term by term."""
    return torch.cat([(r.double()[:, :, None] * b.double()[None]).sum(1) for r in a.split(64)])


def _ieee(W, x, dY, ids, A, B, s):
    """h, dX, dA, dB by their formulas."""
    h, dX = _mm(x, W.T), _mm(dY, W)
    dA, dB = torch.zeros(A.shape, dtype=torch.float64, device="cuda"), torch.zeros(B.shape, dtype=torch.float64, device="cuda")
    for a in range(A.shape[0]):
        at = multi_ref.tokens_of(ids, a)
        if at.numel():
            u, v = s[a].double() * _mm(x[at], A[a].T), s[a].double() * _mm(dY[at], B[a])
            h[at] += _mm(u, B[a].T)
            dX[at] += _mm(v, A[a])
            dA[a], dB[a] = _mm(v.T, x[at]), _mm(dY[at].T, u)
    return h, dX, dA, dB


def _check(kind, ids, bad_x, bad_dY):
    import bit_nf4_quantized_04_b200 as q
    M, n = ids.numel(), int(ids.max()) + 1
    N, K, r = 264, 320, 8
    x, A, B, dY, _, s = _inputs(N, K, M, n, r, "one", 700)
    base, What, fwd, bwd = _base(q, kind, synth.llama_weight((N, K), 700, device="cuda"))
    W = What.bfloat16()
    good = [fwd(base, x, ids, A, B, s), *bwd(base, x, dY, ids, A, B, s)]
    for m, f, v in bad_x:
        x[m, f] = v
    for m, f, v in bad_dY:
        dY[m, f] = v
    got = [fwd(base, x, ids, A, B, s), *bwd(base, x, dY, ids, A, B, s)]
    q.check()
    for t, w, g, name in zip(got, _ieee(W, x, dY, ids, A, B, s), good, ("h", "dX", "dA", "dB")):
        assert torch.equal(t.isnan(), w.isnan()), name
        at = w.isinf()
        assert torch.equal(t.isinf(), at) and torch.equal(t[at].double(), w[at]), name
        at = w.isfinite()
        assert torch.equal(t[at], g[at]), name


BAD = {
    "x": ([(5, 11, INF), (70, 12, -INF)], []),
    "dY": ([], [(9, 13, -INF), (100, 3, INF)]),
    "both": ([(20, 4, INF), (90, 7, INF)], [(20, 6, -INF), (90, 6, -INF)]),
    "nan": ([(5, 11, NAN)], [(70, 3, NAN)]),
    "against": ([(5, 11, INF), (6, 11, -INF)], [(70, 3, INF), (71, 3, -INF)]),
}


@pytest.mark.parametrize("kind", ["nf4", "dense"])
@pytest.mark.parametrize("bad", BAD)
def test_infinities_with_every_step_full(kind, bad):
    # two adapters of 64 tokens each
    ids = (torch.arange(128, device="cuda") // 64).to(torch.int32)
    _check(kind, ids, *BAD[bad])


@pytest.mark.parametrize("kind", ["nf4", "dense"])
@pytest.mark.parametrize("M", [1, 5, 16, 33, 70, 131, 300, 900])
def test_infinities_in_the_last_token_of_an_adapter(kind, M):
    ids = (torch.arange(M, device="cuda") % 3).to(torch.int32)
    if M > 4:
        ids[M // 2] = -1
    _check(kind, ids, [(M - 1, 11, -INF)], [])
    _check(kind, ids, [], [(M - 1, 13, INF)])
    _check(kind, ids, [(M - 1, 11, INF)], [(max(M - 2, 0), 13, INF)])
