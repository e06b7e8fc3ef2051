"""Out-of-bounds writes of the many-adapter calls and of clipping, caught two ways, as for the
single-adapter calls: guard bytes around every output and around a workspace of exactly the size
asked for, and the checked build, which must report nothing and give the same bits.
"""
import os
import subprocess
import sys

import pytest
import torch

import multi_ref
import synth
from test_gpu_guard import Guarded, ROOT, _check_all

pytestmark = pytest.mark.gpu

CASES = [  # N, K, M, n, r, ids
    (40, 448, 5, 3, 3, "tokens"), (200, 192, 17, 20, 17, "tokens"), (264, 960, 130, 5, 33, "runs"),
    (1000, 4096, 64, 70, 16, "tokens"), (136, 1024, 300, 300, 8, "tokens"), (264, 704, 897, 6, 24, "runs"),
    (1032, 448, 1300, 3, 64, "wild"), (64, 64, 4097, 2, 1, "runs"),
]


def _case(q, N, K, M, n, r, mix, seed):
    W = synth.llama_weight((N, K), seed, device="cuda")
    w = q.quantize_weight(W)
    x = synth.normal_bf16((M, K), 1.0, seed + 1, "cuda")
    A = synth.normal_bf16((n, r, K), 0.05, seed + 2, "cuda")
    B = synth.normal_bf16((n, N, r), 0.05, seed + 3, "cuda")
    dY = synth.normal_bf16((M, N), 1.0, seed + 4, "cuda")
    ids = multi_ref.make_ids(mix, M, n, seed + 5, "cuda")
    s = torch.ones(n, device="cuda")
    out = {}
    for kind, base, fwd, bwd in (("nf4", w, q.qlora_linear_multi_fwd, q.qlora_linear_multi_bwd),
                                 ("dense", W, q.dense_linear_multi_fwd, q.dense_linear_multi_bwd)):
        g = {k: Guarded(sh, d) for k, (sh, d) in {
            "h": ((M, N), torch.bfloat16), "dX": ((M, K), torch.bfloat16), "dA": ((n, r, K), torch.float32),
            "dB": ((n, N, r), torch.float32), "cA": ((n, r, K), torch.float32), "cB": ((n, N, r), torch.float32),
            "norm": ((n,), torch.float32),
            "wsf": ((q.multi_workspace_size(q._lib.OP_FWD, N, K, M, n, r),), torch.uint8),
            "wsb": ((q.multi_workspace_size(q._lib.OP_BWD, N, K, M, n, r),), torch.uint8)}.items()}
        fwd(base, x, ids, A, B, s, h=g["h"].t, ws=g["wsf"].t)
        bwd(base, x, dY, ids, A, B, s, dX=g["dX"].t, dA=g["dA"].t, dB=g["dB"].t, ws=g["wsb"].t)
        q.clip_grad_norm([g["dA"].t, g["dB"].t], 0.5, n=n, out=[g["cA"].t, g["cB"].t], norm=g["norm"].t)
        _check_all(q, g)
        out.update({f"{kind}.{k}": v.t.clone() for k, v in g.items() if not k.startswith("ws")})
    return out


def _all_cases(q):
    out = {}
    for i, c in enumerate(CASES):
        out.update({f"{i}.{k}": v for k, v in _case(q, *c, 7000 + 17 * i).items()})
    return out


def test_guard_bytes_survive():
    import bit_nf4_quantized_04_b200 as q
    out = _all_cases(q)
    dump = os.environ.get("QNF4_GUARD_DUMP")
    if dump:  # the child run below: hand the outputs to the parent
        torch.save({k: v.cpu() for k, v in out.items()}, dump)


@pytest.mark.skipif(os.environ.get("QNF4_LIB") == "checked", reason="runs in the child only")
def test_checked_build_reports_nothing_and_matches(tmp_path):
    import bit_nf4_quantized_04_b200 as q
    dump = str(tmp_path / "checked.pt")
    env = dict(os.environ, QNF4_LIB="checked", QNF4_GUARD_DUMP=dump)
    res = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-p", "no:cacheprovider",
                          os.path.abspath(__file__), "-k", "guard_bytes_survive"],
                         cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    assert res.returncode == 0, res.stdout[-3000:] + res.stderr[-3000:]
    theirs, ours = torch.load(dump), _all_cases(q)
    assert set(theirs) == set(ours)
    diff = [k for k in ours if not torch.equal(ours[k].cpu(), theirs[k])]
    assert not diff, f"checked build differs from the default build in: {diff[:10]}"
