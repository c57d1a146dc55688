"""Argument checks of the operators of include/lpc_ops.h on the host, no GPU needed: every call here is one that
validation must refuse or that has nothing to do, so the fake addresses are never used.  Also the host-side sizes and
the AdamW plan."""
import ctypes

import pytest
import torch

from fp8_precision_allreduce_amd import lpc

OK, NULL, SHAPE, RANKS, DTYPE, ALIGN, HIP = range(7)
A, B = 0x10000, 0x10008
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def L():
    if torch.cuda.device_count() > 0:
        pytest.skip("fake-pointer ABI checks run only where no GPU is visible")
    return lpc.lib()


def replaced(args, **kw):
    a = list(args)
    for k, v in kw.items():
        a[int(k[1:])] = v
    return a


def test_gemm_errors(L):
    f = L.lpc_gemm_fp8
    ok = [A, A, 4, 256, A, A, 100, 2, A, A, BF16, None]
    assert f(*ok) == HIP                                     # passes the checks; no device
    assert f(*replaced(ok, _10=2)) == DTYPE
    assert f(*replaced(ok, _2=0, _0=None)) == OK and f(*replaced(ok, _6=0, _9=None)) == OK
    for i in (0, 1, 4, 5, 8, 9):
        assert f(*replaced(ok, **{"_%d" % i: None})) == NULL, i
    assert f(*replaced(ok, _8=None, _7=1)) == HIP            # one group needs no counts
    for i in (0, 1, 4, 5, 9):
        assert f(*replaced(ok, **{"_%d" % i: B})) == ALIGN, i
    assert f(*replaced(ok, _8=A + 2)) == ALIGN and f(*replaced(ok, _8=A + 4)) == HIP
    for bad in (dict(_3=0), dict(_3=100), dict(_7=0), dict(_7=1025), dict(_7=-1), dict(_2=1 << 31), dict(_6=1 << 31),
                dict(_2=1 << 30, _3=1 << 20), dict(_6=1 << 25, _3=1 << 14, _7=1024)):
        assert f(*replaced(ok, **bad)) == SHAPE, bad


def test_padded_rows(L):
    for rows, groups, want in ((0, 3, 0), (1, 1, 128), (128, 1, 128), (129, 1, 256), (1, 8, 1024), (16384, 8, 17280),
                               (5, 0, 0), (5, -1, 0)):
        assert lpc.lpc_padded_rows(rows, groups) == want
    for rows, groups in ((1, 8), (300, 3), (1000, 7)):       # enough for any counts
        worst = sum(-(-c // 128) for c in [1] * min(groups - 1, rows) + [max(0, rows - groups + 1)])
        assert lpc.lpc_padded_rows(rows, groups) >= 128 * worst


def test_cols_errors(L):
    f = L.lpc_quantize_fp8_cols
    ok = [A, BF16, 5, 256, 2, A, A, A, A, A, None]
    assert f(*ok) == HIP and f(*replaced(ok, _8=None, _9=None)) == HIP
    assert f(*replaced(ok, _1=5)) == DTYPE
    assert f(*replaced(ok, _2=0)) == OK and f(*replaced(ok, _3=0, _0=None)) == OK
    for i in (0, 5, 6, 7, 8, 9):
        assert f(*replaced(ok, **{"_%d" % i: None})) == NULL, i
    for i in (0, 6, 7, 8, 9):
        assert f(*replaced(ok, **{"_%d" % i: B})) == ALIGN, i
    for bad in (dict(_3=100), dict(_4=0), dict(_4=1025), dict(_2=1 << 31)):
        assert f(*replaced(ok, **bad)) == SHAPE, bad
    g = L.lpc_requantize_fp8_cols
    ok = [A, A, 5, 256, 2, A, A, A, None]
    assert g(*ok) == HIP and g(*replaced(ok, _2=0)) == OK
    for i in (0, 1, 5, 6, 7):
        assert g(*replaced(ok, **{"_%d" % i: None})) == NULL, i
    for i in (0, 1, 6, 7):
        assert g(*replaced(ok, **{"_%d" % i: B})) == ALIGN, i
    assert g(*replaced(ok, _3=129)) == SHAPE and g(*replaced(ok, _4=0)) == SHAPE


def test_wgrad_errors(L):
    f = L.lpc_gemm_fp8_wgrad
    ok = [A, A, 7, A, A, 9, 5, 2, A, A, None]
    assert f(*ok) == HIP
    assert f(*replaced(ok, _2=0)) == OK and f(*replaced(ok, _5=0)) == OK
    for i in (0, 1, 3, 4, 8, 9):
        assert f(*replaced(ok, **{"_%d" % i: None})) == NULL, i
    assert f(None, None, 7, None, None, 9, 0, 2, A, A, None) == HIP    # no rows: zeros are still written
    for i in (0, 1, 3, 4, 9):
        assert f(*replaced(ok, **{"_%d" % i: B})) == ALIGN, i
    for bad in (dict(_7=0), dict(_7=1025), dict(_6=1 << 31), dict(_2=1 << 31), dict(_2=1 << 21, _5=1 << 20)):
        assert f(*replaced(ok, **bad)) == SHAPE, bad


def test_row_counts_that_wrap_are_refused(L):
    """Rounding such a count up to whole blocks passes SIZE_MAX; a negative Python int becomes one."""
    for rows in ((1 << 64) - 1, (1 << 64) - 99, (1 << 64) - 127, (1 << 64) - 128, 1 << 63, 1 << 32, 1 << 31):
        for groups in (1, 2, 1024):
            assert L.lpc_padded_rows(rows, groups) == 0, (rows, groups)
            assert L.lpc_quantize_fp8_cols(A, BF16, rows, 256, groups, A, A, A, A, A, None) == SHAPE, (rows, groups)
            assert L.lpc_requantize_fp8_cols(A, A, rows, 256, groups, A, A, A, None) == SHAPE, (rows, groups)
            assert L.lpc_gemm_fp8_wgrad(A, A, 7, A, A, 9, rows, groups, A, A, None) == SHAPE, (rows, groups)
            assert L.lpc_gemm_fp8(A, A, rows, 256, A, A, 100, groups, A, A, BF16, None) == SHAPE, (rows, groups)
        assert L.lpc_router_workspace_bytes(rows, 60) == 0
        assert L.lpc_router_forward(A, BF16, rows, 60, 4, 1, 0.01, None, A, A, A, A, A, A, A, 1 << 30, None) == SHAPE
        assert L.lpc_router_backward(A, F32, rows, 60, 4, 1, None, A, A, A, A, A, None) == SHAPE
    assert lpc.lpc_padded_rows(-1, 2) == 0


def test_router_errors(L):
    f, g = L.lpc_router_forward, L.lpc_router_backward
    need = lpc.lpc_router_workspace_bytes(1000, 60)
    ok = [A, BF16, 1000, 60, 4, 1, 0.01, A, A, A, A, A, A, A, A, need, None]
    assert f(*ok) == HIP and f(*replaced(ok, _7=None)) == HIP and f(*replaced(ok, _7=A + 1, _13=A + 4)) == HIP
    assert f(*replaced(ok, _1=9)) == DTYPE
    for i in (0, 8, 9, 10, 11, 12, 13, 14):
        assert f(*replaced(ok, **{"_%d" % i: None})) == NULL, i
    for i in (0, 8, 9, 10, 11, 12, 14):
        assert f(*replaced(ok, **{"_%d" % i: B})) == ALIGN, i
    assert f(*replaced(ok, _13=A + 2)) == ALIGN
    assert f(*replaced(ok, _2=0, _0=None, _8=None, _9=None)) == HIP    # no rows: zero totals are still written
    for bad in (dict(_3=0), dict(_3=1025), dict(_4=0), dict(_4=61), dict(_4=17), dict(_15=need - 1), dict(_2=1 << 31)):
        assert f(*replaced(ok, **bad)) == SHAPE, bad
    assert lpc.lpc_router_workspace_bytes(5, 0) == 0 and lpc.lpc_router_workspace_bytes(5, 1025) == 0
    ok = [A, F32, 1000, 60, 4, 1, A, A, A, A, A, A, None]
    assert g(*ok) == HIP and g(*replaced(ok, _6=None)) == HIP and g(*replaced(ok, _10=A + 4)) == HIP
    assert g(*replaced(ok, _1=3)) == DTYPE and g(*replaced(ok, _2=0)) == OK
    for i in (0, 7, 8, 9, 10, 11):
        assert g(*replaced(ok, **{"_%d" % i: None})) == NULL, i
    for i in (0, 7, 8, 9, 11):
        assert g(*replaced(ok, **{"_%d" % i: B})) == ALIGN, i
    for bad in (dict(_3=0), dict(_3=1025), dict(_4=0), dict(_4=61), dict(_4=17)):
        assert g(*replaced(ok, **bad)) == SHAPE, bad


def test_router_without_workspace(L):
    """Few rows need none; more than one workgroup's do."""
    for rows, experts, none in ((0, 60, True), (1, 64, True), (64, 256, True), (65, 256, False), (16, 1024, True), (17, 1024, False)):
        need = lpc.lpc_router_workspace_bytes(rows, experts)
        assert (need == 0) == none, (rows, experts, need)
        args = [A, F32, rows, experts, 2, 1, 0.01, None, A, A, A, A, A, A, None, 0, None]
        assert L.lpc_router_forward(*args) == (HIP if none else NULL), (rows, experts)


def plan(L, rows, grad=F32, bits=32):
    t = (lpc._AdamwTensor * max(len(rows), 1))(*[lpc._AdamwTensor(*r) for r in rows])
    size = L.lpc_adamw_plan_bytes(t, len(rows))
    host = (ctypes.c_uint8 * max(size, 1))()
    chunks = ctypes.c_size_t(99)
    st = L.lpc_adamw_plan(t, len(rows), grad, bits, host, size, ctypes.byref(chunks))
    return st, chunks.value, bytes(host[:size])


def test_adamw_plan(L):
    row = (A, A, A, A, None, None, None, 5000)
    eight = (A, A, A, A, A, A, A, 4096)
    assert plan(L, [])[:2] == (OK, 0) and plan(L, [(None,) * 7 + (0,)])[:2] == (OK, 0)
    st, chunks, data = plan(L, [row, (None,) * 7 + (0,), (A + 64, A, A, A, None, None, None, 1)])
    assert (st, chunks) == (OK, 3)
    table = [int.from_bytes(data[4 * i:4 * i + 4], "little") for i in range(6)]
    assert table == [0, 0, 0, 1, 1, 0]                       # (tensor, number of the chunk within it)
    first = lpc._AdamwTensor.from_buffer_copy(data[32:96])
    second = lpc._AdamwTensor.from_buffer_copy(data[96:160])
    assert len(data) == 160 and (first.param, first.n, second.param, second.n) == (A, 5000, A + 64, 1)
    assert plan(L, [eight], BF16, 8)[:2] == (OK, 1)
    assert plan(L, [row], 5)[0] == DTYPE and plan(L, [row], F32, 16)[0] == DTYPE
    assert plan(L, [row], F32, 8)[0] == NULL                 # 8-bit moments need scales
    for i in range(4):
        assert plan(L, [row[:i] + (None,) + row[i + 1:]])[0] == NULL
        assert plan(L, [row[:i] + (B,) + row[i + 1:]])[0] == ALIGN
    for i in (4, 5):
        assert plan(L, [eight[:i] + (B,) + eight[i + 1:]], BF16, 8)[0] == ALIGN
    assert plan(L, [row[:6] + (B, 5000)])[0] == ALIGN
    assert plan(L, [row, row[:6] + (A, 5000)])[0] == NULL    # copies for some tensors only
    assert plan(L, [row[:7] + ((1 << 40) + 1,)])[0] == SHAPE
    t = (lpc._AdamwTensor * 1)(lpc._AdamwTensor(*row))
    c = ctypes.c_size_t(0)
    host = (ctypes.c_uint8 * 4096)()
    assert L.lpc_adamw_plan(t, 1, F32, 32, host, L.lpc_adamw_plan_bytes(t, 1) - 1, ctypes.byref(c)) == SHAPE
    assert L.lpc_adamw_plan(t, 1, F32, 32, None, 4096, ctypes.byref(c)) == NULL
    assert L.lpc_adamw_plan(t, 1, F32, 32, host, 4096, None) == NULL
    assert L.lpc_adamw_plan(t, -1, F32, 32, host, 4096, ctypes.byref(c)) == SHAPE


def test_adamw_step_errors(L):
    f = L.lpc_adamw_step
    ok = [A, 3, F32, 8, 1, 1e-3, 0.9, 0.99, 1e-8, 0.1, None, None]
    assert f(*ok) == HIP and f(*replaced(ok, _10=A + 4)) == HIP
    assert f(*replaced(ok, _2=4)) == DTYPE and f(*replaced(ok, _3=4)) == DTYPE
    assert f(*replaced(ok, _1=0, _0=None)) == OK
    assert f(*replaced(ok, _0=None)) == NULL
    assert f(*replaced(ok, _0=B)) == ALIGN and f(*replaced(ok, _10=A + 2)) == ALIGN
    assert f(*replaced(ok, _4=0)) == SHAPE and f(*replaced(ok, _1=1 << 31)) == SHAPE


def test_adamw_step_refuses_betas_that_are_no_means(L):
    ok = [A, 3, F32, 32, 1, 1e-3, 0.9, 0.99, 1e-8, 0.1, None, None]
    for i in (6, 7):
        for beta in (1.0, 1.5, -0.1, float("nan"), float("inf"), -float("inf")):
            assert L.lpc_adamw_step(*replaced(ok, **{"_%d" % i: beta})) == SHAPE, (i, beta)
        for beta in (0.0, 0.5, 1.0 - 2.0 ** -53):
            assert L.lpc_adamw_step(*replaced(ok, **{"_%d" % i: beta})) == HIP, (i, beta)


def test_binding_refuses_host_tensors(L):
    u8, f32 = torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(4, 1)
    with pytest.raises(ValueError, match="GPU tensor"):
        lpc.lpc_gemm_fp8(u8, f32, u8, f32, torch.zeros(4, 4))
    with pytest.raises(ValueError, match="w has shape"):
        lpc.lpc_gemm_fp8(u8, f32, torch.zeros(4, 256, dtype=torch.uint8), f32, torch.zeros(4, 4))
    with pytest.raises(ValueError, match="GPU tensor"):
        lpc.AdamW([f32], [f32], [f32], [f32])
    with pytest.raises(ValueError, match="come together"):
        lpc.AdamW([f32], [f32], [u8], [u8], m_scales=[f32])
