"""More refusals on the host of the linear calls and of clipping, without a GPU: no pointer is read and
nothing is launched."""
import ctypes as C

import pytest

FAKE = 1 << 20  # never dereferenced
BIG = 1 << 40
ERR_ALIGN = 3


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
