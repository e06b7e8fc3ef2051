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


@pytest.mark.parametrize("M", [4, 40, 900])
def test_workspaces_over_and_beside_other_buffers(M):
    import bit_nf4_quantized_04_b200 as q
    N, K, n, r = 128, 192, 3, 4
    ids = multi_ref.make_ids("tokens", M, n, 910, "cuda")
    s = torch.ones(n, device="cuda")
    w = q.quantize_weight(synth.llama_weight((N, K), 911, device="cuda"))
    A, B = synth.normal_bf16((n, r, K), 0.05, 912, "cuda"), synth.normal_bf16((n, N, r), 0.05, 913, "cuda")
    need = q.multi_workspace_size(q._lib.OP_FWD, N, K, M, n, r)
    room = torch.zeros(need + 2 * M * K, dtype=torch.uint8, device="cuda")
    x = room[need:].view(torch.bfloat16).view(M, K)  # right behind the workspace
    x.copy_(synth.normal_bf16((M, K), 1.0, 914, "cuda"))
    want = q.qlora_linear_multi_fwd(w, x.clone(), ids, A, B, s)
    assert torch.equal(q.qlora_linear_multi_fwd(w, x, ids, A, B, s, ws=room[:need]), want)
    over = torch.zeros(max(need, 2 * M * K), dtype=torch.uint8, device="cuda")
    xo = over[: 2 * M * K].view(torch.bfloat16).view(M, K)
    with pytest.raises((ValueError, q.Qnf4Error), match="overlaps"):
        q.qlora_linear_multi_fwd(w, xo, ids, A, B, s, ws=over)
    q.check()
