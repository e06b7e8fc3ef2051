"""The base product of the many-adapter layer held element by element, on each of its paths.

Bounds, with u = 2^-24 and b = 2^-8 (half a step of bf16), against float64 with the weight
bf16(W_hat) that the layer is defined with:
* an output is rounded once, b |h|; s u (s v for dX) enters as bf16, b |su| |B|^T; the sums are
  fp32: a tensor-core sum of C products makes C / 16 additions, each off by at most one step, 2 u,
  of the running sum, which the sum of magnitudes bounds (twice, for the alignment within one step).
* up to 32 tokens the weight comes from a table of level pairs and is rounded up to three times,
  3 b beside the b of bf16(W_hat): 4 b |x| |W|^T at most. Those roundings are independent from
  weight to weight, at most b / sqrt(3) each in the root mean square, so a block of 32 tokens x 8
  features is off by about sqrt(5 / 3) b = 1.3 b of its norm, and 5 b is never met.
* the framework's own rule for the whole output: 5e-3 of the norm, 2e-2 of the largest element.
A 64-wide step of the contraction lost or taken twice changes a block by sqrt(64 / C) of its norm,
0.09 for the longest contraction here, and a wrong element fails its own bound.
"""
import threading

import pytest
import torch

import multi_ref
import synth
from test_gpu_multi import BF, U2, _base, _inputs, _within

pytestmark = pytest.mark.gpu


def _blocks(t):
    """Sums of squares over blocks of 32 rows x 8 columns."""
    M, F = t.shape
    t = torch.nn.functional.pad(t.square(), (0, -F % 8, 0, -M % 32))
    return t.view(t.shape[0] // 32, 32, t.shape[1] // 8, 8).sum((1, 3))


def _hold(got, want, mag, magw, C, n, table, what):
    bound = BF * 1.01 * (want.abs() + mag) + U2 * ((C + 64 * n) / 16 + 64) * (magw + mag) * 2
    _within(got, want, bound + (4.05 * BF * magw if table else 0.0), what)
    err = got.double() - want
    assert bool((_blocks(err) <= (5 * BF) ** 2 * _blocks(want)).all()), what
    assert err.norm().item() <= 5e-3 * want.norm().item(), what
    assert err.abs().max().item() <= 2e-2 * want.abs().max().item(), what


def _check(q, kind, N, K, M, n, r, mix, seed, ops=("fwd", "bwd")):
    x, A, B, dY, ids, s = _inputs(N, K, M, n, r, mix, seed)
    base, What, fwd, bwd = _base(q, kind, synth.llama_weight((N, K), seed, device="cuda"))
    W = What.bfloat16()
    table = kind == "nf4" and M <= 32
    if "fwd" in ops:
        h = fwd(base, x, ids, A, B, s)
        q.check()
        _hold(h, *multi_ref.forward(W, x, ids, A, B, s), K, n, table, "h")
    if "bwd" in ops:
        dX = bwd(base, x, dY, ids, A, B, s)[0]
        q.check()
        _hold(dX, *multi_ref.backward(W, x, dY, ids, A, B, s)[0], N, n, table, "dX")


@pytest.mark.parametrize("case", [
    (1000, 4096, 1, 3, 16, "one"), (520, 2048, 16, 32, 16, "tokens"), (264, 960, 17, 20, 17, "tokens"),
    (1000, 1024, 32, 5, 64, "tokens"), (512, 4096, 64, 40, 16, "tokens"), (2048, 2048, 130, 5, 33, "runs"),
    (1032, 448, 300, 8, 8, "wild"), (1024, 4096, 767, 7, 16, "runs"), (264, 448, 800, 9, 33, "tokens"),
    (1000, 320, 769, 2, 64, "one"), (4096, 4096, 1025, 3, 32, "runs"), (4096, 1024, 4096, 3, 16, "runs"),
    (1008, 8192, 1300, 6, 16, "none"), (2000, 5056, 2100, 40, 5, "tokens"),
], ids=str)
@pytest.mark.parametrize("kind", ["nf4", "dense"])
def test_every_element(case, kind):
    import bit_nf4_quantized_04_b200 as q
    _check(q, kind, *case, 800)


# more tiles of 128 features x 256 tokens than a B200 has SMs, so that whole tiles run first and the
# rest is cut along the contraction into slices that meet in partial tiles (172 tiles: 148 and 24 x 6
# slices; 216: 148 and 68 x 2), with the adapter chunks dealt to the slices
CUT = [(11008, 4096, 512, 8, 16, "runs"), (11008, 4096, 500, 64, 16, "tokens"), (13824, 5120, 300, 64, 64, "tokens"),
       (13824, 5120, 300, 3, 33, "runs")]


@pytest.mark.parametrize("case", CUT, ids=str)
@pytest.mark.parametrize("kind", ["nf4", "dense"])
def test_whole_tiles_beside_a_cut_last_wave(case, kind):
    import bit_nf4_quantized_04_b200 as q
    N, K, *rest = case
    _check(q, kind, N, K, *rest, 810, ops=("fwd",))
    _check(q, kind, K, N, *rest, 820, ops=("bwd",))


@pytest.mark.parametrize("N,K,M,n,r", [(5120, 13824, 300, 64, 64), (4096, 11008, 500, 64, 16), (4160, 11008, 500, 50, 64),
                                       (4224, 11008, 500, 40, 33), (11008, 4096, 500, 64, 16), (13824, 5120, 300, 64, 64)])
@pytest.mark.parametrize("kind", ["nf4", "dense"])
def test_many_chunks_between_the_tiles_of_a_cta(kind, N, K, M, n, r):
    # adapter chunks are short steps beside the base's: a CTA's converters run far ahead of the loads
    # where one tile's chunks end and the next tile's base begins, for several remainders of the tiles'
    # steps by the number of converter sets; twenty calls, equal bits, the first within its bounds
    import bit_nf4_quantized_04_b200 as q
    x, A, B, dY, ids, s = _inputs(N, K, M, n, r, "tokens", 850)
    base, What, fwd, bwd = _base(q, kind, synth.llama_weight((N, K), 850, device="cuda"))
    W = What.bfloat16()
    first = [fwd(base, x, ids, A, B, s), *bwd(base, x, dY, ids, A, B, s)]
    for _ in range(20):
        again = [fwd(base, x, ids, A, B, s), *bwd(base, x, dY, ids, A, B, s)]
        assert [torch.equal(a, b) for a, b in zip(again, first)] == [True] * 4
    q.check()
    _hold(first[0], *multi_ref.forward(W, x, ids, A, B, s), K, n, False, "h")
    _hold(first[1], *multi_ref.backward(W, x, dY, ids, A, B, s)[0], N, n, False, "dX")


@pytest.mark.parametrize("kind", ["nf4", "dense"])
def test_broken_adapters_in_a_cut_last_wave(kind):
    # two of 40 adapters hold infinities, which land in chunks of different slices: their own tokens
    # get them, every other token and feature its bits
    import bit_nf4_quantized_04_b200 as q
    N, K, M, n, r = 11008, 4096, 500, 40, 16
    x, A, B, dY, ids, s = _inputs(N, K, M, n, r, "tokens", 830)
    ids[:4] = torch.tensor([3, 35, 3, 35], dtype=torch.int32)
    base, _, fwd, _ = _base(q, kind, synth.llama_weight((N, K), 830, device="cuda"))
    good = fwd(base, x, ids, A, B, s)
    B2 = B.clone()
    B2[3, 100, 2], B2[35, N - 1, 15] = float("inf"), float("-inf")
    h = fwd(base, x, ids, A, B2, s)
    q.check()
    want = good.clone()
    for a, f, j, v in ((3, 100, 2, 1.0), (35, N - 1, 15, -1.0)):
        at = multi_ref.tokens_of(ids, a)
        u = x[at].double() @ A[a, j].double()
        want[at, f] = (u * v * float("inf")).bfloat16()
    assert torch.equal(h, want)


def test_side_streams_of_two_threads():
    # two threads, a stream each, their calls interleaved as they come: the results of the same calls
    # made one after another on the default stream
    import bit_nf4_quantized_04_b200 as q
    jobs = []
    for i, (N, K, M, n, r) in enumerate([(1024, 2048, 1100, 6, 16), (512, 1024, 300, 40, 8), (2048, 1024, 12, 5, 16)]):
        x, A, B, dY, ids, s = _inputs(N, K, M, n, r, "tokens", 840 + i)
        for kind in ("nf4", "dense"):
            base, _, fwd, bwd = _base(q, kind, synth.llama_weight((N, K), 840 + i, device="cuda"))

            def job(base=base, fwd=fwd, bwd=bwd, x=x, A=A, B=B, dY=dY, ids=ids, s=s, n=n):
                h = fwd(base, x, ids, A, B, s)
                dX, dA, dB = bwd(base, x, dY, ids, A, B, s)
                out, norm = q.clip_grad_norm([dA, dB], 0.5, n=n)
                return [h, dX, dA, dB, *out, norm]
            jobs.append(job)
    want = [j() for j in jobs]
    torch.cuda.synchronize()
    failed = []

    def work(order):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(6):
                    got = [(k, jobs[k]()) for k in order]
            stream.synchronize()
            for k, g in got:
                if not all(torch.equal(a, b) for a, b in zip(g, want[k])):
                    failed.append(k)
        except Exception as e:  # noqa: BLE001  (reported by the test's own thread)
            failed.append(e)

    threads = [threading.Thread(target=work, args=(o,)) for o in (range(6), range(5, -1, -1))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    q.check()
    assert not failed, failed
