"""The float64 reference of the many-adapter layer against autograd and differences (CPU)."""
import torch

import multi_ref


def _plain(x, ids, A, B, s, W):
    rows = []
    for m in range(x.shape[0]):
        h, a = W @ x[m], int(ids[m])
        if 0 <= a < A.shape[0]:
            h = h + s[a] * (B[a] @ (A[a] @ x[m]))
        rows.append(h)
    return torch.stack(rows)


def test_reference_matches_autograd_and_differences():
    torch.manual_seed(0)
    M, N, K, n, r = 7, 6, 5, 3, 2
    ids = torch.tensor([0, 2, -1, 2, 0, 5, 2], dtype=torch.int32)
    W, s, dY = torch.randn(N, K).double(), torch.rand(n).double() + 0.5, torch.randn(M, N).double()
    x, A, B = (torch.randn(*sh, dtype=torch.float64, requires_grad=True) for sh in ((M, K), (n, r, K), (n, N, r)))
    h = _plain(x, ids, A, B, s, W)
    want = torch.autograd.grad((h * dY).sum(), (x, A, B))
    with torch.no_grad():
        assert torch.allclose(multi_ref.forward(W, x, ids, A, B, s)[0], h, rtol=0, atol=1e-12)
        got = multi_ref.backward(W, x, dY, ids, A, B, s)
    for g, w in zip(got, want):
        assert torch.allclose(g[0], w, rtol=0, atol=1e-12)
    assert bool((got[1][0][1] == 0).all())  # adapter 1 has no token
    assert torch.autograd.gradcheck(lambda x, A, B: _plain(x, ids, A, B, s, W), (x, A, B))
