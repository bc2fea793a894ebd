"""The 8-bit operators' layout, definitions and refusals; nothing here is launched."""
import ctypes

import pytest
import torch

import sharded_mixed_precision_amd as D
from tests import fp8_harness as F

INVALID = -1
AT = 1 << 40  # device addresses of calls that are refused before any launch


def dense(rows, cols, dtype=D.DOPT_BF16, at=AT, ld=None):
    return D.dopt_dense(at, rows, cols, cols if ld is None else ld, dtype, 0)


def fp8(rows, cols, kind="row", at=AT + (1 << 36), **other):
    o = D.dopt_fp8_layout(rows, cols, kind)
    d = dict(codes=at, scales=at + (1 << 34), rows=rows, cols=cols, ld=o["ld"], scale_ld=o["scale_ld"], kind=D.FP8_KINDS[kind])
    d.update(other)
    return D.dopt_fp8_matrix(d["codes"], d["scales"], d["rows"], d["cols"], d["ld"], d["scale_ld"], d["kind"], 0)


def refused(rc, text):
    assert rc == INVALID
    assert text in D.dopt_last_error()


@pytest.mark.parametrize("rows,cols,kind,want", [
    (1, 1, "row", (128, 16, 128, 16)), (17, 129, "row", (256, 32, 17 * 256, 64)), (129, 128, "tile", (128, 2, 129 * 128, 2)),
    (0, 5, "row", (128, 0, 0, 0)), (5, 0, "tile", (0, 1, 0, 0)), (128256, 8192, "tile", (8192, 1002, 128256 * 8192, 64 * 1002))])
def test_layout(rows, cols, kind, want):
    o = D.dopt_fp8_layout(rows, cols, kind)
    assert (o["ld"], o["scale_ld"], o["codes_bytes"], o["scales_bytes"]) == want


def test_layout_refusals():
    for args in ((-1, 1, 0), (1, -1, 0), (1, (1 << 22) + 1, 0), ((1 << 30) + 1, 1, 0), (1, 1, 2)):
        refused(D.lib().dopt_fp8_layout(*args, ctypes.byref(D.dopt_fp8_sizes())), "bad")
    refused(D.lib().dopt_fp8_layout(1, 1, 0, None), "null output")
    with pytest.raises(D.DoptError):
        D.dopt_fp8_layout(1, 1, "column")


def test_definition_of_the_format():
    """The harness's rounding on numbers known by hand: e least with A <= 448 * 2^e, ties to even, non-finite to NaN."""
    x = torch.zeros(1, 128)
    x[0, :8] = torch.tensor([448.0, 1.0, 17.0, 19.0, -27.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10])
    c, e = F.encode(x, "row")
    assert e.item() == 0
    assert c[0, :8].tolist() == [448.0, 1.0, 16.0, 20.0, -28.0, 2.0 ** -9, 0.0, 2.0 ** -8]
    x[0, 0] = 449.0
    c, e = F.encode(x, "row")
    assert e.item() == 1 and c[0, 0].item() == 224.0
    x[0, 0] = float("inf")
    x[0, 1] = float("nan")
    c, e = F.encode(x, "row")
    assert e.item() == -4 and torch.isnan(c[0, :2]).all() and c[0, 4].item() == -448.0  # 27 <= 448 / 16 = 28
    c, e = F.encode(torch.zeros(3, 5), "row")
    assert (e == -126).all() and (c == 0).all()
    c, e = F.encode(torch.full((130, 130), 2.0 ** -149), "tile")
    assert (e == -126).all() and e.shape == (2, 2)


def test_cast_refusals():
    L, call = D.lib(), D.lib().dopt_fp8_cast
    x = dense(10, 300)
    q, t = fp8(10, 300), fp8(300, 10, at=AT + (1 << 37))
    refused(call(None, None, None, 0, q, None, None), "x: null")
    refused(call(x, None, None, 0, None, None, None), "neither")
    refused(call(dense(10, 300, 7), None, None, 0, q, None, None), "bad dtype")
    refused(call(dense(10, 300, ld=299), None, None, 0, q, None, None), "distance")
    refused(call(dense(10, 300, ld=1 << 23), None, None, 0, q, None, None), "distance")
    refused(call(dense(10, 300, at=None), None, None, 0, q, None, None), "null device pointer")
    refused(call(dense(10, 300, at=AT + 1), None, None, 0, q, None, None), "aligned")
    refused(call(dense(-1, 300), None, None, 0, q, None, None), "bad size")
    refused(call(dense((1 << 30) + 1, 1), None, None, 0, q, None, None), "bad size")
    refused(call(dense((1 << 22) + 1, 1), None, None, 0, None, D.dopt_fp8_matrix(AT + (1 << 36), AT + (1 << 38), 1, (1 << 22) + 1, 1 << 23, 16, 0, 0),
                 None), "bad size")
    refused(call(x, None, None, 0, fp8(11, 300), None, None), "not of x's size")
    refused(call(x, None, None, 0, None, q, None), "transpose")
    refused(call(x, None, None, 0, q, fp8(300, 10, "tile"), None), "kind")
    refused(call(x, None, None, 0, fp8(10, 300, ld=368), None, None), "rows of codes")
    refused(call(x, None, None, 0, fp8(10, 300, ld=385), None, None), "rows of codes")
    refused(call(x, None, None, 0, fp8(10, 300, scale_ld=8), None, None), "rows of scales")
    refused(call(x, None, None, 0, fp8(10, 300, scale_ld=13), None, None), "rows of scales")
    refused(call(x, None, None, 0, fp8(10, 300, codes=None), None, None), "null device pointer")
    refused(call(x, None, None, 0, fp8(10, 300, codes=AT + 8), None, None), "16-byte")
    refused(call(x, None, None, 0, fp8(10, 300, scales=AT + 2), None, None), "4-byte")
    refused(call(x, None, None, 0, fp8(10, 300, kind="row", codes=AT), None, None), "overlaps x")
    refused(call(x, None, None, 0, q, fp8(300, 10), None), "overlaps")
    refused(call(x, AT + (1 << 38), None, 0, q, t, None), "together")
    refused(call(x, AT + (1 << 38), AT + (1 << 39), 9, q, t, None), "bad dtype")
    refused(call(x, AT + (1 << 38) + 2, AT + (1 << 39), 0, q, t, None), "aligned")
    refused(call(x, q.codes, AT + (1 << 39), 0, q, t, None), "overlaps row_factor")
    for rows, cols in ((0, 300), (10, 0), (0, 0)):  # nothing to do: no pointer is looked at
        assert call(dense(rows, cols, at=None), None, None, 0, fp8(rows, cols, codes=None, scales=None), None, None) == 0


def test_gemm_refusals():
    call = D.lib().dopt_fp8_gemm
    a, b, o = fp8(100, 300), fp8(50, 300, "tile", at=AT + (1 << 37)), dense(100, 50)
    need = D.dopt_fp8_gemm_workspace_bytes(100, 50, 300)
    ws = AT + (1 << 38)
    refused(call(None, b, o, 0, ws, need, None), "a: null")
    refused(call(a, b, None, 0, ws, need, None), "out: null")
    refused(call(fp8(100, 300, "tile"), b, o, 0, ws, need, None), "kind ROW")
    refused(call(a, fp8(50, 301), o, 0, ws, need, None), "differ in columns")
    refused(call(a, b, dense(100, 51), 0, ws, need, None), "a's rows x b's rows")
    refused(call(a, b, dense(100, 50, 3), 0, ws, need, None), "bad dtype")
    refused(call(a, b, dense(100, 50, at=a.codes), 0, ws, need, None), "overlaps a")
    refused(call(a, b, dense(100, 50, at=b.scales), 0, ws, need, None), "overlaps b's scales")
    big = fp8(100, 1 << 20), fp8(50, 1 << 20, at=AT + (1 << 37))
    need = D.dopt_fp8_gemm_workspace_bytes(100, 50, 1 << 20)
    assert need > 0
    refused(call(*big, o, 0, None, need, None), "workspace")
    refused(call(*big, o, 0, ws, need - 1, None), "workspace")
    refused(call(*big, o, 0, ws + 8, need, None), "workspace")
    refused(call(*big, o, 0, AT, need, None), "overlaps")
    for m, n, k in ((0, 50, 300), (100, 0, 300), (0, 0, 0)):
        none = lambda rows, i: fp8(rows, k, at=AT + (i << 36)) if rows else fp8(0, k, codes=None, scales=None)  # noqa: E731
        assert call(none(m, 1), none(n, 2), dense(m, n, at=None), 0, None, 0, None) == 0
    assert call(fp8(100, 0), fp8(50, 0), o, 1, None, 0, None) == 0  # adds nothing
    for m, n, k in ((-1, 1, 1), (1, 1 << 23, 1), (1, 1, (1 << 22) + 1)):
        with pytest.raises(D.DoptError):
            D.dopt_fp8_gemm_workspace_bytes(m, n, k)


def test_norm_refusals():
    call = D.lib().dopt_rmsnorm
    x, w, at = dense(10, 300), AT + (1 << 35), lambda i: AT + (i << 28)
    q = fp8(10, 300)
    refused(call(None, None, w, 0, 1e-5, None, None, q, None, None), "x: null")
    refused(call(x, None, w, 0, 1e-5, None, None, None, None, None), "neither")
    refused(call(x, dense(10, 301, at=at(1)), w, 0, 1e-5, None, None, q, None, None), "another size")
    refused(call(x, dense(10, 300, D.DOPT_F32, at=at(1)), w, 0, 1e-5, None, None, q, None, None), "another type")
    refused(call(x, None, w, 0, 1e-5, dense(9, 300, at=at(1)), None, q, None, None), "another size")
    refused(call(x, None, w, 0, 1e-5, None, dense(10, 300, D.DOPT_F16, at=at(1)), q, None, None), "another type")
    refused(call(x, None, w, 0, 1e-5, None, None, fp8(10, 299), None, None), "another size")
    refused(call(x, None, w, 0, 1e-5, None, None, fp8(10, 300, "tile"), None, None), "kind ROW")
    refused(call(x, None, w, 0, -1.0, None, None, q, None, None), "eps")
    refused(call(x, None, w, 0, float("nan"), None, None, q, None, None), "eps")
    refused(call(x, None, None, 0, 1e-5, None, None, q, None, None), "weight")
    refused(call(x, None, w, 5, 1e-5, None, None, q, None, None), "weight: bad dtype")
    refused(call(x, None, w, 0, 1e-5, None, None, q, w + 2, None), "rstd")
    refused(call(x, None, w, 0, 1e-5, None, x, q, None, None), "y overlaps x")
    refused(call(x, dense(10, 300, at=at(1)), w, 0, 1e-5, dense(10, 300, at=at(1) + 2), None, q, None, None), "h overlaps residual")
    refused(call(x, dense(10, 300, at=at(1)), w, 0, 1e-5, dense(10, 300, ld=301), None, q, None, None), "h overlaps x")
    refused(call(x, None, w, 0, 1e-5, dense(10, 300, at=at(1)), dense(10, 300, at=at(1)), q, None, None), "y overlaps h")
    refused(call(x, None, w, 0, 1e-5, None, None, q, w, None), "rstd overlaps weight")
    assert call(dense(0, 300, at=None), None, w, 0, 1e-5, None, None, fp8(0, 300), None, None) == 0
    assert call(dense(3, 0, at=None), None, None, 0, 1e-5, None, None, fp8(3, 0), None, None) == 0


def test_columns_side_by_side_do_not_overlap():
    """Column slices of one matrix are apart if their columns are; a call gets past the check to the next refusal."""
    call, w = D.lib().dopt_rmsnorm, AT + (1 << 35)
    at = lambda c: AT + (1 << 30) + 2 * c  # noqa: E731
    x = dense(10, 300)
    for a, b, meet in ((0, 300, False), (700, 1000, False), (0, 299, True), (1100, 0, True), (800, 0, False), (700, 999, True), (650, 300, False),
                       (300, 0, False), (299, 0, True), (950, 200, False), (1250, 2 * 1300 + 900, False), (1250, 2 * 1300 + 1249, True)):
        rc = call(x, None, w, 0, 1e-5, dense(10, 300, at=at(a), ld=1300), dense(10, 300, at=at(b), ld=1300), None, w, None)
        refused(rc, "y overlaps h" if meet else "rstd overlaps weight")


def test_norm_grad_refusals():
    call = D.lib().dopt_rmsnorm_grad
    at = lambda i: AT + (i << 28)  # noqa: E731
    dy, h, dx = dense(10, 300, at=at(1)), dense(10, 300, at=at(2)), dense(10, 300, at=at(3))
    w, r, dw, ws = at(4), at(5), at(6), at(7)
    need = D.dopt_rmsnorm_grad_workspace_bytes(10, 300)

    def go(dy=dy, h=h, dh=None, w=w, wt=0, r=r, dx=dx, dw=dw, dwt=0, ws=ws, n=need):
        return call(dy, h, dh, w, wt, r, dx, dw, dwt, 0, ws, n, None)

    refused(go(h=None), "h: null")
    refused(go(dy=dense(10, 299, at=at(1))), "another size")
    refused(go(dy=dense(10, 300, D.DOPT_F16, at=at(1))), "neither of h's type nor fp32")
    refused(go(dh=dense(10, 300, D.DOPT_F32, at=at(8))), "another type")
    refused(go(dx=dense(10, 300, D.DOPT_F32, at=at(8))), "another type")
    refused(go(dx=None), "dx: null")
    refused(go(w=None), "weight")
    refused(go(r=None), "rstd")
    refused(go(dw=None), "dweight")
    refused(go(dwt=4), "dweight: bad dtype")
    refused(go(ws=None), "workspace")
    refused(go(n=need - 1), "workspace")
    refused(go(ws=at(7) + 4), "workspace")
    refused(go(dx=h), "dx overlaps h")
    refused(go(dw=w), "dweight overlaps weight")
    refused(go(dw=at(2)), "dweight overlaps h")
    refused(go(ws=at(1)), "workspace overlaps dy")
    refused(go(dx=dense(10, 300, at=at(1) + 2)), "dx overlaps dy")
    refused(go(dy=dense(10, 300, D.DOPT_F32, at=at(3))), "dx overlaps dy")
    assert call(dense(3, 0), dense(3, 0), None, None, 0, r, dense(3, 0), None, 0, 0, None, 0, None) == 0
    for rows, cols in ((-1, 1), (1, (1 << 22) + 1)):
        with pytest.raises(D.DoptError):
            D.dopt_rmsnorm_grad_workspace_bytes(rows, cols)


def test_binding_refuses_host_tensors_and_bad_matrices():
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    with pytest.raises(D.DoptError, match="kind"):
        D.fp8_matrix(u8(2, 128), u8(1, 16), 2, 100, "column")
    with pytest.raises(D.DoptError, match="codes"):
        D.fp8_matrix(u8(2, 100), u8(1, 16), 2, 100)
    with pytest.raises(D.DoptError, match="not a matrix of bytes"):
        D.fp8_matrix(torch.zeros(2, 128), u8(1, 16), 2, 100)
    with pytest.raises(D.DoptError, match="not a device tensor"):
        D.fp8_matrix(u8(2, 128), u8(1, 16), 2, 100)


def test_gemm_coarse_refusals():
    """As dopt_fp8_gemm's, and fp32 outputs."""
    call = D.lib().dopt_fp8_gemm_coarse
    a, b, o = fp8(100, 300), fp8(50, 300, "tile", at=AT + (1 << 37)), dense(100, 50)
    refused(call(a, b, dense(100, 50, D.DOPT_F32), 0, None, 0, None), "coarse")
    refused(call(None, b, o, 0, None, 0, None), "a: null")
    refused(call(a, fp8(50, 301), o, 0, None, 0, None), "differ in columns")
    refused(call(a, b, dense(100, 50, at=a.codes), 0, None, 0, None), "overlaps a")
    big = fp8(100, 1 << 20), fp8(50, 1 << 20, at=AT + (1 << 37))
    refused(call(*big, o, 0, None, 0, None), "workspace")
    assert call(fp8(0, 300, codes=None, scales=None), b, dense(0, 50, at=None), 0, None, 0, None) == 0


def test_grids_past_the_limit_of_a_launch():
    """Sizes whose tiles take 2^32 threads or more along one dimension are refused before any launch."""
    L, m = D.lib(), 1 << 30
    refused(L.dopt_fp8_cast(dense(m, 256), None, None, 0, fp8(m, 256, at=AT + (1 << 41), scales=AT + (1 << 43)), None, None), "too large")  # 2^24 tiles
    a, b = fp8(m, 128, at=AT + (1 << 42), scales=AT + (1 << 43)), fp8(257, 128, at=AT + (1 << 44))
    assert D.dopt_fp8_gemm_workspace_bytes(m, 257, 128) == 0
    refused(L.dopt_fp8_gemm(a, b, dense(m, 257), 0, None, 0, None), "too large")  # 2^22 x 2 tiles of 512 threads, or 2^23 x 3 of 256
    refused(L.dopt_fp8_gemm_coarse(a, fp8(1025, 128, at=AT + (1 << 44)), dense(m, 1025), 0, None, 0, None), "too large")


def test_nothing_overlaps_nothing():
    """A workspace of which no byte is needed may lie anywhere: the call gets past the check to the next refusal."""
    m = 1 << 30
    a, b = fp8(m, 128, at=AT + (1 << 42), scales=AT + (1 << 43)), fp8(257, 128, at=AT + (1 << 44))
    assert D.dopt_fp8_gemm_workspace_bytes(m, 257, 128) == 0
    for ws in (AT + (1 << 30), AT + (1 << 42) + (1 << 30)):
        refused(D.lib().dopt_fp8_gemm(a, b, dense(m, 257), 0, ws, 1 << 20, None), "out: too large")
