"""What the export and import of a list refuse: arrays on another device, and
arrays that overlap one another, the params or the state.  All of it is decided
before anything touches a device."""
import pytest
import torch

import sharded_mixed_precision_amd as D
from tests.test_list_cpu import _dev, _err, spec

MB = 1 << 20


def _case(state="e4m3"):
    """A list whose arrays lie a MB apart: tensors of 1000 bf16, 300 fp32 and no elements."""
    L = D.dopt_list_build([spec(1000), spec(300, "f32", "f32"), spec(0)], state)
    names = ["master", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"]
    at = {k: (i + 1) * MB for i, k in enumerate(names) if k in L.state_arrays()}
    params = [10 * MB, 11 * MB, None]
    return L, D.list_tensors(L, params, None, at), at, params


@pytest.mark.parametrize("state", list(D.STATE_KINDS))
def test_arrays_within_the_state_are_refused(state):
    L, t, at, _ = _case(state)
    size = {k: n * (1 if dt == "e4m3" else 4) for k, (dt, n) in L.state_arrays().items()}
    x = 4 * L.numel
    for call in (D.dopt_list_export, D.dopt_list_import):
        for i, name in enumerate(("master", "exp_avg", "exp_avg_sq")):
            for key, a in at.items():
                for where in (a, a + size[key] - 4, a - x + 4):
                    arrays = [20 * MB, 21 * MB, 22 * MB]
                    arrays[i] = where
                    _err(lambda: call(L, t, *arrays, 30 * MB), f"{name} array", f"state {key}")


def test_arrays_within_the_params_are_refused():
    L, t, _, (a, b, _) = _case()
    x = 4 * L.numel
    for call in (D.dopt_list_export, D.dopt_list_import):
        for i in range(3):
            for p, n, word in ((a, 2000, "param 0"), (b, 1200, "param 1")):
                for where in (p, p + n - 4, p - x + 4):
                    arrays = [20 * MB, 21 * MB, 22 * MB]
                    arrays[i] = where
                    _err(lambda: call(L, t, *arrays, 30 * MB), "array", word)
    # fp32 params are their own masters, and may be: of the moments they are not
    for call in (D.dopt_list_export, D.dopt_list_import):
        _err(lambda: call(L, t, 20 * MB, b - 4 * 1000, 22 * MB, 30 * MB), "exp_avg array", "param 1")


def test_exported_arrays_overlap_none_of_the_others():
    L, t, _, _ = _case()
    a, x = 20 * MB, 4 * L.numel
    for arrays in ((a, a, a + MB), (a, a + x - 4, a + MB), (a + MB, a, a - x + 4), (a, a + MB, a)):
        _err(lambda: D.dopt_list_export(L, t, *arrays, 30 * MB), "overlap")


def test_arrays_on_another_device_are_refused(monkeypatch):
    L, t, _, _ = _case()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    for call, word in ((D.dopt_list_export, "export"), (D.dopt_list_import, "import")):
        for i, name in enumerate(("master", "exp_avg", "exp_avg_sq")):
            arrays = [20 * MB, 21 * MB, 22 * MB]
            arrays[i] = _dev(L.numel, torch.float32)
            _err(lambda: call(L, t, *arrays, 30 * MB), f"{word} {name} on device", "current device is 3")
