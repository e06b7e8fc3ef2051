"""Plain float64 form of the many-adapter linear layer and its gradients, token groups in a
loop over the adapters, with the magnitudes the tests' error bounds are built from. Works on
any device; shares no code with the library."""
import torch


def make_ids(mix, M, n, seed, device="cpu"):
    g = torch.Generator().manual_seed(seed)
    if mix == "none":
        ids = torch.full((M,), -1)
    elif mix == "one":
        ids = torch.full((M,), n - 1)
    elif mix == "tokens":
        ids = torch.randint(-1, n, (M,), generator=g)
    elif mix == "wild":  # most ids name nothing, some of them far out of range
        far = torch.tensor([-2 ** 31, 2 ** 31 - 1, n, -7, n + 1000, 0])
        ids = far[torch.randint(0, len(far), (M,), generator=g)]
    else:  # runs of tokens
        runs = max(1, min(M, 2 * n + 1))
        cuts = torch.sort(torch.randint(0, M, (runs - 1,), generator=g)).values
        of = torch.randint(-1, n, (runs,), generator=g)
        ids = of[torch.searchsorted(cuts, torch.arange(M), right=True)]
    return ids.to(torch.int32).to(device)


def tokens_of(ids, a):
    return torch.nonzero(ids == a).flatten()


def forward(W, x, ids, A, B, scales):
    """(h, |su| |B|^T per token, |x| |W|^T) in float64; W is the weight the base stands for."""
    W, x, A, B, s = W.double(), x.double(), A.double(), B.double(), scales.double()
    h = x @ W.T
    mag = torch.zeros_like(h)
    for a in range(A.shape[0]):
        at = tokens_of(ids, a)
        if at.numel():
            su = s[a] * (x[at] @ A[a].T)
            h[at] += su @ B[a].T
            mag[at] = su.abs() @ B[a].abs().T
    return h, mag, x.abs() @ W.abs().T


def backward(W, x, dY, ids, A, B, scales):
    """dX, dA, dB in float64 and, per output, the bound's magnitudes: for dX those of
    |sv| |A| and |dY| |W|; for dA and dB (sum of |P| |X|, sum of |X| times the magnitude of
    P's own contraction), P being the projection the sum runs over."""
    W, x, dY, A, B, s = W.double(), x.double(), dY.double(), A.double(), B.double(), scales.double()
    dX = dY @ W
    magX = torch.zeros_like(dX)
    dA, dB = torch.zeros_like(A), torch.zeros_like(B)
    magA, magB = [torch.zeros_like(A), torch.zeros_like(A)], [torch.zeros_like(B), torch.zeros_like(B)]
    for a in range(A.shape[0]):
        at = tokens_of(ids, a)
        if not at.numel():
            continue
        sv, su = s[a] * (dY[at] @ B[a]), s[a] * (x[at] @ A[a].T)
        svm = s[a].abs() * (dY[at].abs() @ B[a].abs())
        sum_ = s[a].abs() * (x[at].abs() @ A[a].abs().T)
        dX[at] += sv @ A[a]
        magX[at] = sv.abs() @ A[a].abs()
        dA[a] = sv.T @ x[at]
        dB[a] = dY[at].T @ su
        magA[0][a], magA[1][a] = sv.abs().T @ x[at].abs(), svm.T @ x[at].abs()
        magB[0][a], magB[1][a] = dY[at].abs().T @ su.abs(), dY[at].abs().T @ sum_
    return (dX, magX, dY.abs() @ W.abs()), (dA, *magA), (dB, *magB)
