"""The argument checks of the many-adapter calls and of gradient clipping, without a GPU: every
call here is refused on the host, before a launch and before any pointer is read."""
import ctypes as C

import pytest
import torch

FAKE = 1 << 20  # never dereferenced


@pytest.fixture(scope="module")
def q():
    import __graft_entry__
    __graft_entry__.build()
    import bit_nf4_quantized_04_b200 as q
    return q


def _grad_args(ptrs=(FAKE, FAKE), dtypes=(0, 1), elems=(12, 24)):
    k = len(ptrs)
    keep = ((C.c_void_p * k)(*ptrs), (C.c_int32 * k)(*dtypes), (C.c_int64 * k)(*elems))
    return keep, [C.addressof(a) for a in keep]


def test_grad_norm_refusals(q):
    f = q.lib.qnf4_grad_norm
    keep, a = _grad_args()
    assert f(-1, *a, 1, FAKE, FAKE, 1 << 20, None) == 1
    assert f(2, *a, 0, FAKE, FAKE, 1 << 20, None) == 1
    assert f(2, None, a[1], a[2], 1, FAKE, FAKE, 1 << 20, None) == 1
    assert f(2, *a, 1, None, FAKE, 1 << 20, None) == 1
    assert f(2, *a, 1, FAKE + 4, FAKE, 1 << 20, None) == 3
    assert f(2, *a, 5, FAKE, FAKE, 1 << 20, None) == 2       # 12 elements are not 5 parts
    assert f(2, *a, 4, FAKE, FAKE, 16, None) == 6
    assert f(2, *a, 4, FAKE, None, 1 << 20, None) == 6
    keep, a = _grad_args(dtypes=(0, 2))
    assert f(2, *a, 1, FAKE, FAKE, 1 << 20, None) == 1
    keep, a = _grad_args(ptrs=(FAKE, None))
    assert f(2, *a, 1, FAKE, FAKE, 1 << 20, None) == 1
    keep, a = _grad_args(ptrs=(FAKE + 2, FAKE))              # an fp32 tensor on a 2-byte boundary
    assert f(2, *a, 1, FAKE, FAKE, 1 << 20, None) == 3
    keep, a = _grad_args(elems=(-4, 4))
    assert f(2, *a, 1, FAKE, FAKE, 1 << 20, None) == 2


def test_clip_refusals(q):
    f = q.lib.qnf4_clip_grad_norm
    keep, a = _grad_args()
    out = (C.c_void_p * 2)(FAKE, FAKE)
    for bad in (-0.5, float("inf"), float("nan")):
        assert f(2, *a, 1, bad, C.addressof(out), FAKE, FAKE, 1 << 20, None) == 1
    assert f(2, *a, 1, 1.0, None, FAKE, FAKE, 1 << 20, None) == 1
    none = (C.c_void_p * 2)(FAKE, None)
    assert f(2, *a, 1, 1.0, C.addressof(none), FAKE, FAKE, 1 << 20, None) == 1
    odd = (C.c_void_p * 2)(FAKE, FAKE + 1)                    # a bf16 output on an odd address
    assert f(2, *a, 1, 1.0, C.addressof(odd), FAKE, FAKE, 1 << 20, None) == 3


def test_grad_workspace_size(q):
    keep, a = _grad_args(elems=(4096 * 3, 8))
    # room for a sum per piece, then the factors, both on 256-byte boundaries
    size = q.lib.qnf4_grad_workspace_size(2, a[2], 1)
    assert size % 256 == 0 and size >= 512
    assert q.lib.qnf4_grad_workspace_size(2, a[2], 4) >= size
    assert q.lib.qnf4_grad_workspace_size(2, a[2], 0) == 0
    assert q.lib.qnf4_grad_workspace_size(0, None, 1) == 256


def test_binding_refuses_cpu_tensors(q):
    with pytest.raises(ValueError):
        q.grad_norm([torch.ones(4)])
    with pytest.raises(TypeError):
        q.grad_norm([torch.ones(4, dtype=torch.float64)])
    with pytest.raises(ValueError):
        q.clip_grad_norm([torch.ones(4)], 1.0)


def test_multi_refusals(q):
    w = q.Qnf4Weight(8, 64, 64, 256, FAKE, FAKE, FAKE, FAKE)
    big = 1 << 40

    def fwd(w=w, x=FAKE, M=4, ids=FAKE, n=3, A=FAKE, B=FAKE, r=8, s=FAKE, h=FAKE, ws=FAKE, size=big):
        return q.lib.qnf4_qlora_linear_multi_fwd(C.byref(w), x, M, ids, n, A, B, r, s, h, ws, size, None)

    def bwd(w=w, x=FAKE, dY=FAKE, M=4, ids=FAKE, n=3, A=FAKE, B=FAKE, r=8, s=FAKE, dX=FAKE, dA=FAKE, dB=FAKE,
            ws=FAKE, size=big):
        return q.lib.qnf4_qlora_linear_multi_bwd(C.byref(w), x, dY, M, ids, n, A, B, r, s, dX, dA, dB, ws, size, None)

    for f in (fwd, bwd):
        assert f(n=0) == 1 and f(n=4097) == 1
        assert f(r=0) == 1 and f(r=65) == 1
        assert f(M=-1) == 2
        for arg in ("x", "ids", "A", "B", "s"):
            assert f(**{arg: None}) == 1 and f(**{arg: FAKE + 8}) == 3
        assert f(size=16) == 6 and f(ws=None) == 6
    assert fwd(M=100, ws=FAKE + 8) == 3 and bwd(ws=FAKE + 8) == 3
    assert fwd(M=0, ws=None, size=0) == 0
    assert fwd(h=None) == 1
    assert bwd(w=q.Qnf4Weight(12, 64, 64, 256, FAKE, FAKE, FAKE, FAKE)) == 2   # N not a multiple of 8
    assert fwd(w=q.Qnf4Weight(8, 96, 64, 256, FAKE, FAKE, FAKE, FAKE)) == 2
    d = q.lib.qnf4_dense_linear_multi_fwd
    assert d(FAKE, 8, 96, FAKE, 4, FAKE, 3, FAKE, FAKE, 8, FAKE, FAKE, FAKE, big, None) == 2
    assert d(None, 8, 64, FAKE, 4, FAKE, 3, FAKE, FAKE, 8, FAKE, FAKE, FAKE, big, None) == 1
    d = q.lib.qnf4_dense_linear_multi_bwd
    assert d(FAKE, 8, 64, FAKE, FAKE, 4, FAKE, 0, FAKE, FAKE, 8, FAKE, FAKE, FAKE, FAKE, FAKE, big, None) == 1


def test_multi_workspace_sizes(q):
    size = q.multi_workspace_size
    for op in (q._lib.OP_FWD, q._lib.OP_BWD):
        assert 0 < size(op, 4096, 4096, 1, 1, 1) <= size(op, 4096, 4096, 4096, 1, 16) <= size(op, 4096, 4096, 4096, 64, 16)
    assert size(q._lib.OP_QUANTIZE, 4096, 4096, 16, 4, 16) == 0
    assert size(q._lib.OP_FWD, 4096, 4096, 16, 0, 16) == 0


def test_multi_group_refusals(q):
    w = q.Qnf4Weight(8, 64, 64, 256, FAKE, FAKE, FAKE, FAKE)
    arr = (q.Qnf4Weight * 2)(w, w)
    p = (C.c_void_p * 2)(FAKE, FAKE)

    def f(k=2, x=p, M=4, ids=FAKE, n=3, A=p, B=p, r=8, s=FAKE, h=p, ws=FAKE, size=1 << 30):
        return q.lib.qnf4_qlora_linear_multi_fwd_group(k, arr, x, M, ids, n, A, B, r, s, h, ws, size, None)

    assert f(k=0) == 1 and f(k=9) == 1
    assert f(M=0) == 2 and f(M=17) == 2
    assert f(x=None) == 1 and f(ids=None) == 1 and f(s=FAKE + 4) == 3 and f(ids=FAKE + 4) == 3
    assert f(n=0) == 1 and f(r=65) == 1 and f(r=0) == 1
    assert f(A=(C.c_void_p * 2)(FAKE, None)) == 1


def test_clip_outputs_that_overlap(q):
    f = q.lib.qnf4_clip_grad_norm
    keep, a = _grad_args(ptrs=(FAKE, FAKE + 4096), elems=(12, 24))   # 48 bytes, 48 bytes

    def st(o0, o1):
        out = (C.c_void_p * 2)(o0, o1)
        return f(2, *a, 1, 1.0, C.addressof(out), FAKE, FAKE, 16, None)  # (the workspace is too small)

    assert st(FAKE, FAKE + 4096) == 6 and st(FAKE + 48, FAKE + 96) == 6 and st(FAKE + 8192, FAKE + 4096) == 6
    assert st(FAKE + 8192, FAKE + 8192) == 1 and st(FAKE + 8192, FAKE + 8192 + 46) == 1   # one another
    assert st(FAKE + 4096, FAKE + 8192) == 1 and st(FAKE + 4100, FAKE + 8192) == 1        # another gradient
    assert st(FAKE + 4, FAKE + 8192) == 1 and st(FAKE + 8192, FAKE + 46) == 1             # part of a gradient
