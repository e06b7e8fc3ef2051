"""More refusals on the host of the linear calls and of clipping, without a GPU: no pointer is read and
nothing is launched."""
import ctypes as C

import pytest
import torch

FAKE = 1 << 20  # never dereferenced
BIG = 1 << 40
ERR_ARG, ERR_ALIGN = 1, 3


@pytest.fixture(scope="module")
def q():
    import __graft_entry__
    __graft_entry__.build()
    import bit_nf4_quantized_04_b200 as q
    return q


@pytest.mark.parametrize("M", [1, 16, 17, 100, 1000])
@pytest.mark.parametrize("off", [1, 4, 8])
def test_a_workspace_off_its_alignment_is_refused(q, M, off):
    # at every number of tokens alike
    w = q.Qnf4Weight(8, 64, 64, 256, FAKE, FAKE, FAKE, FAKE)
    ws, lib = FAKE + off, q.lib
    st = [lib.qnf4_qlora_linear_multi_fwd(C.byref(w), FAKE, M, FAKE, 3, FAKE, FAKE, 8, FAKE, FAKE, ws, BIG, None),
          lib.qnf4_dense_linear_multi_fwd(FAKE, 8, 64, FAKE, M, FAKE, 3, FAKE, FAKE, 8, FAKE, FAKE, ws, BIG, None),
          lib.qnf4_qlora_linear_multi_bwd(C.byref(w), FAKE, FAKE, M, FAKE, 3, FAKE, FAKE, 8, FAKE, FAKE, FAKE, FAKE, ws,
                                          BIG, None)]
    if M <= 16:
        ws_, p = (q.Qnf4Weight * 2)(w, w), (C.c_void_p * 2)(FAKE, FAKE)
        st.append(lib.qnf4_qlora_linear_multi_fwd_group(2, ws_, p, M, FAKE, 3, p, p, 8, FAKE, p, ws, BIG, None))
        if off < 4:  # the sums of the one-adapter calls are fp32 words
            st += [lib.qnf4_qlora_linear_fwd(C.byref(w), FAKE, M, FAKE, FAKE, 8, 1.0, FAKE, ws, BIG, None),
                   lib.qnf4_qlora_linear_fwd_group(2, ws_, p, M, p, p, 8, 1.0, p, ws, BIG, None)]
    assert st == [ERR_ALIGN] * len(st)


class Buffers:
    """Addresses of one many-adapter call's buffers, each of its own megabyte."""
    N, K, n, r = 64, 128, 3, 8

    def __init__(self, q, M, first=0):
        self.q, self.M = q, M
        names = ("packed code2 scale2 mean W x dY ids A B s h dX dA dB ws").split()
        for i, k in enumerate(names):
            setattr(self, k, FAKE * (1 + first + i))

    def weight(self):
        return self.q.Qnf4Weight(self.N, self.K, 64, 256, self.packed, self.code2, self.scale2, self.mean)

    def call(self, fn):
        b, w = self, self.weight()
        base = (C.byref(w),) if "qlora" in fn else (b.W, b.N, b.K)
        d = (b.dY,) if fn.endswith("bwd") else ()
        out = (b.dX, b.dA, b.dB) if fn.endswith("bwd") else (b.h,)
        return getattr(self.q.lib, "qnf4_" + fn)(*base, b.x, *d, b.M, b.ids, b.n, b.A, b.B, b.r, b.s, *out, b.ws, BIG, None)


READ = {"qlora": "packed code2 scale2 mean x ids A B s", "dense": "W x ids A B s"}


@pytest.mark.parametrize("M", [1, 16, 100, 1000])
@pytest.mark.parametrize("fn", ["qlora_linear_multi_fwd", "dense_linear_multi_fwd", "qlora_linear_multi_bwd",
                                "dense_linear_multi_bwd"])
def test_an_output_over_another_buffer_is_refused(q, fn, M):
    bwd = fn.endswith("bwd")
    for out in ("dX", "dA", "dB") if bwd else ("h",):
        for other in READ[fn[:5]].split() + (["dY", "dX", "dA", "dB"] if bwd else []):
            if other != out:
                b = Buffers(q, M)
                setattr(b, out, getattr(b, other))
                assert b.call(fn) == ERR_ARG, (out, other)
                b = Buffers(q, M)
                setattr(b, other, getattr(b, out) + 16 if other != "mean" else getattr(b, out))  # inside the output
                assert b.call(fn) == ERR_ARG, (out, other)


def _group(q, ls, n, r):
    ws_ = (q.Qnf4Weight * len(ls))(*[b.weight() for b in ls])
    p = lambda k: (C.c_void_p * len(ls))(*[getattr(b, k) for b in ls])  # noqa: E731
    return q.lib.qnf4_qlora_linear_multi_fwd_group(len(ls), ws_, p("x"), ls[0].M, ls[0].ids, n, p("A"), p("B"), r,
                                                   ls[0].s, p("h"), ls[0].ws, BIG, None)


@pytest.mark.parametrize("layers", [2, 8])
def test_a_grouped_output_over_any_layers_buffer_is_refused(q, layers):
    for other in READ["qlora"].split() + ["h"]:
        for at in range(1, layers) if other not in ("ids", "s") else (0,):
            ls = [Buffers(q, 4, 16 * i) for i in range(layers)]
            ls[0].h = getattr(ls[at], other)
            assert _group(q, ls, 3, 8) == ERR_ARG, (other, at)


@pytest.mark.parametrize("M", [1, 16, 100, 1000])
@pytest.mark.parametrize("fn", ["qlora_linear_multi_fwd", "dense_linear_multi_fwd", "qlora_linear_multi_bwd",
                                "dense_linear_multi_bwd"])
def test_a_workspace_over_another_buffer_is_refused(q, fn, M):
    for other in READ[fn[:5]].split() + (["dY", "dX", "dA", "dB"] if fn.endswith("bwd") else ["h"]):
        b = Buffers(q, M)
        b.ws = getattr(b, other)
        assert b.call(fn) == ERR_ARG, other


def test_a_groups_workspace_over_any_layers_buffer_is_refused(q):
    for other in READ["qlora"].split() + ["h"]:
        for at in range(3) if other not in ("ids", "s") else (0,):
            ls = [Buffers(q, 4, 16 * i) for i in range(3)]
            ls[0].ws = getattr(ls[at], other)
            assert _group(q, ls, 3, 8) == ERR_ARG, (other, at)


@pytest.mark.parametrize("clip", [False, True])
def test_norms_and_workspaces_over_gradients_are_refused(q, clip):
    # two gradients of 4096 fp32 and 4096 bf16, 4 adapters, scaled into buffers of their own
    g, out, norm, ws = (FAKE, 2 * FAKE), (3 * FAKE, 4 * FAKE), 5 * FAKE, 6 * FAKE
    elems = (C.c_int64 * 2)(4096, 4096)
    need = q.lib.qnf4_grad_workspace_size(2, C.addressof(elems), 4)

    def f(norm=norm, ws=ws):
        p, o, dt = (C.c_void_p * 2)(*g), (C.c_void_p * 2)(*out), (C.c_int32 * 2)(0, 1)
        a = (2, C.addressof(p), C.addressof(dt), C.addressof(elems), 4)
        if clip:
            return q.lib.qnf4_clip_grad_norm(*a, 1.0, C.addressof(o), norm, ws, need, None)
        return q.lib.qnf4_grad_norm(*a, norm, ws, need, None)

    tensors = [(g[0], 4 * 4096), (g[1], 2 * 4096)] + ([(out[0], 4 * 4096), (out[1], 2 * 4096)] if clip else [])
    for at, size in tensors:
        for p in (at, at + size - 16):
            assert f(norm=p) == ERR_ARG and f(ws=p) == ERR_ARG
        assert f(ws=at - need + 16) == ERR_ARG
    assert f(norm=ws) == ERR_ARG and f(norm=ws + need - 16) == ERR_ARG


def test_workspace_sizes_are_each_devices_own(q, monkeypatch):
    # the library's answer depends on the current device's SMs: one that was asked on another device
    # is asked again
    sms, now = {0: 148, 1: 132}, [0]
    monkeypatch.setattr(q.torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(q.torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(q.lib, "qnf4_multi_workspace_size", lambda op, N, K, M, n, r: N * sms[now[0]])
    for d in (0, 1, 0, 1):
        now[0] = d
        assert q.multi_workspace_size(q._lib.OP_FWD, 123456, 64, 77, 3, 8) == 123456 * sms[d]


def test_workspaces_that_are_not_contiguous_are_refused(q):
    # 64 elements in one byte, or in every second one
    like, room = torch.zeros(4), torch.zeros(128, dtype=torch.uint8)
    for ws in (room[:1].expand(64), room[::2]):
        with pytest.raises(ValueError, match="contiguous"):
            q._multi_ws(32, like, ws)
    assert q._multi_ws(32, like, room[64:])[1] == 64
