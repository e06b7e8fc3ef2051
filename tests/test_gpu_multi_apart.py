"""Outputs of the many-adapter calls over and beside other buffers."""
import pytest
import torch

import multi_ref
import synth

pytestmark = pytest.mark.gpu


def test_grouped_outputs_over_and_beside_other_buffers():
    import bit_nf4_quantized_04_b200 as q
    M, n, r = 8, 3, 4
    shapes = [(128, 128), (64, 192)]
    ids = multi_ref.make_ids("tokens", M, n, 900, "cuda")
    s = torch.ones(n, device="cuda")
    ws_ = [q.quantize_weight(synth.llama_weight(sh, 901 + i, device="cuda")) for i, sh in enumerate(shapes)]
    xs = [synth.normal_bf16((M, K), 1.0, 903 + i, "cuda") for i, (_, K) in enumerate(shapes)]
    # both layers' adapters and outputs side by side in one buffer
    sizes = [n * r * K for _, K in shapes] + [n * N * r for N, _ in shapes] + [M * N for N, _ in shapes]
    flat = synth.normal_bf16((sum(sizes),), 0.05, 905, "cuda")
    parts = flat.split(sizes)
    As = [parts[i].view(n, r, shapes[i][1]) for i in range(2)]
    Bs = [parts[2 + i].view(n, shapes[i][0], r) for i in range(2)]
    hs = [parts[4 + i].view(M, shapes[i][0]) for i in range(2)]
    want = q.qlora_linear_multi_fwd_group(ws_, xs, ids, As, Bs, s)
    got = q.qlora_linear_multi_fwd_group(ws_, xs, ids, As, Bs, s, hs=hs)
    assert all(a is b for a, b in zip(got, hs)) and all(torch.equal(a, b) for a, b in zip(got, want))
    for t in (As[1].reshape(-1)[: M * 128], Bs[1].reshape(-1)[-M * 64:]):
        bad = [t.view(M, 128), hs[1]] if t.numel() == M * 128 else [hs[0], t.view(M, 64)]
        with pytest.raises((ValueError, q.Qnf4Error), match="overlaps"):
            q.qlora_linear_multi_fwd_group(ws_, xs, ids, As, Bs, s, hs=bad)
    over = ws_[1].packed.view(torch.bfloat16)
    with pytest.raises((ValueError, q.Qnf4Error), match="overlaps"):
        q.qlora_linear_multi_fwd_group(ws_[::-1], xs[::-1], ids, As[::-1], Bs[::-1], s, hs=[over[: M * 64].view(M, 64), hs[0]])
    q.check()
