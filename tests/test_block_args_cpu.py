"""Arguments that the expert-block entry points take and refuse, on the CPU: a
call that passes the checks of its matrices ends at its missing workspace, which
is asked for after them and before any device call."""
import ctypes

import pytest

import exact_lloyd_means_flashassign_amd as fk
from test_block_cpu import BF16, F32, INVALID, NO_DEVICE, WORKSPACE, P, lib, said, shape  # noqa: F401


def linear(lib, h, X=0x10000, W=0x2000000, Y=0x3000000, R=0, pre=0):  # noqa: F811
    return lib.fk_linear(ctypes.byref(h), P(X), P(W), None, P(R), None, None, P(Y), P(pre), None, 0, None)


def backward(lib, h, dY=0x10000, X=0x1000000, W=0x2000000, pre=0, dX=0x4000000, dW=0x5000000):  # noqa: F811
    return lib.fk_linear_backward(ctypes.byref(h), P(dY), P(X), P(W), P(pre), None, None, P(dX), P(dW), None, None, 0,
                                  None)


def norm_backward(lib, dY, X, dX, rows=4, d=64, ld=192):  # noqa: F811
    return lib.fk_layer_norm_backward(BF16, F32, P(dY), ld, P(X), ld, rows, d, P(0x300000), P(0x400000), None, P(dX), ld,
                                      None, None, None, 0, None)


@pytest.mark.parametrize("order", [(0, 1, 2), (2, 1, 0), (1, 2, 0)])
def test_column_slices_of_one_buffer_are_apart(lib, order):  # noqa: F811
    """Three slices of 64 columns of a buffer with rows of 192 (bf16)."""
    dY, X, dX = (0x10000 + 128 * i for i in order)
    assert norm_backward(lib, dY, X, dX) == WORKSPACE
    # a row further up or down they are as far apart
    assert norm_backward(lib, dY, X, dX + 384) == WORKSPACE
    assert norm_backward(lib, dY + 384, X + 384, dX) == WORKSPACE
    h = shape(M=50, N=32, K=64, ldx=128, ldw=64, ldy=128, ldpre=128, ldr=128)
    a, b, c = (0x10000 + 64 * i for i in (0, 2, 3))
    assert linear(lib, h, X=a, Y=b, pre=c) == WORKSPACE
    assert linear(lib, h, X=a, Y=c, R=b) == WORKSPACE


def test_slices_that_meet_are_refused(lib):  # noqa: F811
    base = 0x10000
    for off in (2, 126, 384 - 126, 384 - 2):  # into the next slice, or round into the next row
        assert norm_backward(lib, 0x200000, base, base + off) == INVALID and said(lib, "dX overlaps X"), off
        assert norm_backward(lib, 0x200000, base + off, base) == INVALID and said(lib, "dX overlaps X"), off
    assert norm_backward(lib, 0x200000, base, base + 128) == WORKSPACE
    assert norm_backward(lib, 0x200000, base, base + 256) == WORKSPACE
    # other row strides may meet anywhere
    h = shape(M=50, N=32, K=64, ldx=128, ldw=64, ldy=136)
    assert linear(lib, h, X=0x10000, Y=0x10080) == INVALID and said(lib, "Y overlaps X")
    # a vector among the rows
    st = lib.fk_layer_norm_backward(BF16, F32, P(0x200000), 192, P(0x10000), 192, 4, 64, P(0x300000), P(0x400000), None,
                                    P(0x500000), 192, P(0x10080), None, None, 0, None)
    assert st == INVALID and said(lib, "dweight overlaps X")


def test_where_rows_may_start(lib):  # noqa: F811
    """Rows of whole 16-byte chunks on 16 bytes; others on their elements."""
    whole, odd = shape(M=50), shape(M=50, K=127, ldx=127, ldw=127, N=31, ldy=31, ldr=31, ldpre=31)
    assert linear(lib, whole, X=0x10002) == INVALID and said(lib, "16-byte")
    assert linear(lib, whole, W=0x2000008) == INVALID and said(lib, "16-byte")
    assert backward(lib, whole, dY=0x10002) == INVALID and said(lib, "16-byte")
    for off in (0, 2, 14):
        assert linear(lib, odd, X=0x10000 + off) == WORKSPACE
        assert linear(lib, odd, W=0x2000000 + off) == WORKSPACE
        assert linear(lib, odd, Y=0x3000000 + off, R=0x8000002, pre=0x9000002) == WORKSPACE
        assert backward(lib, odd, dY=0x10000 + off, X=0x1000000 + off, W=0x2000000 + off) == WORKSPACE
    assert linear(lib, odd, X=0x10001) == INVALID and said(lib, "elements")
    # a stride of whole chunks does not make the columns whole
    assert linear(lib, shape(M=50, K=127), X=0x10002) == WORKSPACE
    assert linear(lib, shape(M=50, ldx=129), X=0x10002) == WORKSPACE
    assert backward(lib, shape(act=4), pre=0x9000002) == WORKSPACE  # pre may start anywhere


def test_workspace_of_rows_in_order(lib):  # noqa: F811
    """Groups of rows that lie in order need no copy of X or dY, however large;
    rows by slots do past the reach of 32-bit offsets."""
    size = lambda h, b: lib.fk_linear_workspace_size(ctypes.byref(h), b)  # noqa: E731
    M, N, K = 1 << 20, 2048, 2048
    h = shape(groups=4, M=M, N=N, K=K, ldx=K, ldw=K, ldy=N, ldr=N, ldpre=N)
    assert size(h, 0) >= M * K * 2 and size(h, 1) >= M * (K + N) * 2
    assert size(h, 2) < 1 << 20
    assert size(h, 3) < M // 32 * N * 4 + (64 << 20)  # dbias's column sums, one row for 64
    for b in (0, 1):
        few = shape(groups=4, M=4096, N=N, K=K, ldx=K, ldw=K, ldy=N, ldr=N, ldpre=N)
        assert size(few, b) == size(few, b + 2)
        plain = shape(M=4096, N=N, K=K, ldx=K, ldw=K, ldy=N, ldr=N, ldpre=N)
        assert size(plain, b) == size(plain, b + 2)
    # the calls ask for what they need themselves
    call = lambda slots: lib.fk_linear(ctypes.byref(h), P(1 << 40), P(2 << 40), None, None, P(slots), P(4 << 40),  # noqa: E731
                                       P(3 << 40), None, P(5 << 40), 1 << 20, None)
    assert call(6 << 40) == WORKSPACE
    if not __import__("torch").cuda.device_count():
        assert call(0) == NO_DEVICE
