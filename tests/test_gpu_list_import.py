"""GPU tests of what an import makes of values that 8 bits cannot hold, each in a block of its own."""
import math

import numpy as np
import pytest
import torch

from tests import list_harness as H

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("state", ["e4m3", "e4m3_sr"])
def test_import_of_infinities_and_nans_block_by_block(state):
    """An infinite m or v is cut to a finite number of its sign and drops its
    block's others to zero or the least code; a NaN and a negative v make their own block NaN."""
    c = H.ListCase([128 * 8], [("f32", "f32")], state)
    c.init()
    x = torch.ones(3, 1024, device="cuda")
    x[1, 130], x[1, 260], x[1, 390] = math.inf, -math.inf, math.nan
    x[2, 130], x[2, 260], x[2, 390], x[2, 520] = math.inf, -1.0, math.nan, 3e38
    c.D.dopt_list_import(c.L, c.t, *x, c.A.workspace, c.stream)
    out = [torch.empty(1024, device="cuda") for _ in range(3)]
    c.D.dopt_list_export(c.L, c.t, *out, c.A.workspace, c.stream)
    m, v = (o.cpu().numpy().reshape(8, 128) for o in out[1:])
    scale = [c.A.state[k].cpu().numpy() for k in ("exp_avg_scale", "exp_avg_sq_scale")]
    one = (0, 5, 6, 7)
    # a block of ones: 448 codes * fp32(1/448), two roundings; v squares it
    assert np.allclose(m[(0, 4, 5, 6, 7), :], 1.0, rtol=2 ** -23, atol=0) and np.allclose(v[one, :], 1.0, rtol=2 ** -22, atol=0)
    cap = float(H.CAP["m"])
    assert math.isclose(m[1, 2], cap, rel_tol=2 ** -23) and math.isclose(m[2, 4], -cap, rel_tol=2 ** -23)
    assert (np.delete(m[1], 2) == 0).all() and (np.delete(m[2], 4) == 0).all()
    assert np.isnan(m[3]).all() and np.isnan(scale[0][3]) and np.isfinite(np.delete(scale[0], 3)).all()
    # the largest number whose square is finite, and finite squares
    assert np.isfinite(v[1]).all() and v[1, 2] == np.float32(H.CAP["r"]) ** 2 > 3.4e38
    least = np.float32(H.LEAST) * scale[1][1]
    assert (np.delete(v[1], 2) == least * least).all() and least > 0
    assert np.isnan(v[2]).all() and np.isnan(v[3]).all()
    # sqrt(3e38), within half a step of its code (it is its block's largest) and 4 roundings of v
    assert math.isclose(v[4, 8], 3e38, rel_tol=2 ** -22)
    assert np.isfinite(np.delete(scale[1], [2, 3])).all() and np.isnan(scale[1][[2, 3]]).all()


@pytest.mark.parametrize("state", ["f32", "e4m3"])
def test_a_flat_fp32_buffer_is_its_own_master_array(state):
    """fp32 params back to back in list order may be the checkpoint's master
    array: export and import leave them as they are and move the moments."""
    import sharded_mixed_precision_amd as D
    from sharded_mixed_precision_amd.arena import ListArrays
    sizes = [5000, 3, 0, 4096, 777]
    flat = torch.randn(sum(sizes), device="cuda")
    begin = flat.clone()
    L = D.dopt_list_build([D.TensorSpec(n, "f32", "f32") for n in sizes], state)
    A, stream = ListArrays(L), torch.cuda.current_stream()
    t = D.list_tensors(L, list(flat.split(sizes)), None, A.state)
    D.dopt_list_init(L, t, D.scaler_cfg(), A.workspace, stream)
    m, v = torch.randn(L.numel, device="cuda"), torch.randn(L.numel, device="cuda").square()
    D.dopt_list_import(L, t, flat, m, v, A.workspace, stream)
    x, y = torch.empty_like(m), torch.empty_like(v)
    D.dopt_list_export(L, t, flat, x, y, A.workspace, stream)
    assert torch.equal(flat, begin)
    if state == "f32":
        assert torch.equal(x, m) and torch.equal(y, v)
    with pytest.raises(D.DoptError, match="overlaps param 0"):
        D.dopt_list_export(L, t, x, flat, y, A.workspace, stream)
    with pytest.raises(D.DoptError, match="overlaps the master array"):
        D.dopt_list_export(L, t, x, x, y, A.workspace, stream)
    with pytest.raises(D.DoptError, match="overlaps"):
        D.dopt_list_export(L, t, x, A.state["exp_avg"].data_ptr(), y, A.workspace, stream)
