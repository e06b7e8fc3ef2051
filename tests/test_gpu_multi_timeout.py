"""Failure detection in the many-adapter kernels without a fault: bounded waits that run out.

As for the single-adapter kernels, the wait limit is set far below the time the work needs, so
that waits give up on purpose; the kernels (clusters and CTA pairs among them) end by themselves,
qnf4_check reports the timeout, and after the limit is restored the next calls give exactly the
results of calls that never timed out.
"""
import pytest
import torch

import multi_ref
import synth

pytestmark = pytest.mark.gpu

DEFAULT_NS = 1_000_000_000


@pytest.fixture()
def q():
    import bit_nf4_quantized_04_b200 as q
    yield q
    q.set_wait_timeout_ns(DEFAULT_NS)


@pytest.mark.parametrize("M", [300, 1500])
@pytest.mark.parametrize("kind", ["nf4", "dense"])
def test_wait_timeout_reports_and_recovers(q, kind, M):
    N, K, n, r = 2048, 4096, 3, 16
    W = synth.llama_weight((N, K), 921, device="cuda")
    base = q.quantize_weight(W) if kind == "nf4" else W
    fwd = q.qlora_linear_multi_fwd if kind == "nf4" else q.dense_linear_multi_fwd
    bwd = q.qlora_linear_multi_bwd if kind == "nf4" else q.dense_linear_multi_bwd
    x = synth.normal_bf16((M, K), 1.0, 922, "cuda")
    dY = synth.normal_bf16((M, N), 1.0, 923, "cuda")
    A = synth.normal_bf16((n, r, K), 0.02, 924, "cuda")
    B = synth.normal_bf16((n, N, r), 0.02, 925, "cuda")
    ids = multi_ref.make_ids("runs", M, n, 926, "cuda")
    s = torch.ones(n, device="cuda")
    ref = [fwd(base, x, ids, A, B, s), *bwd(base, x, dY, ids, A, B, s)]
    q.check()
    for call in (lambda: fwd(base, x, ids, A, B, s), lambda: bwd(base, x, dY, ids, A, B, s)):
        q.set_wait_timeout_ns(100)
        call()
        with pytest.raises(q.Qnf4Error) as ei:
            q.check()
        assert ei.value.status == 5 and "site" in str(ei.value)
        q.check()
        q.set_wait_timeout_ns(DEFAULT_NS)
        got = [fwd(base, x, ids, A, B, s), *bwd(base, x, dY, ids, A, B, s)]
        q.check()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
