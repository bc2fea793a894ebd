"""Tensor lists on the CPU: offsets, the shard lists of a layout, the plain
8-bit encoding itself, and every refusal of the binding and the library that
fires before anything touches a device."""
import ctypes

import numpy as np
import pytest
import torch

import sharded_mixed_precision_amd as D
from synth import PARAM_LISTS, WORKLOADS
from synth.models import ParamSpec
from tests import list_harness as H

HP = [(1e-3, 0.9, 0.999, 1e-8, 0.01)]


def _err(fn, *words, code=-1):
    with pytest.raises(D.DoptError) as e:
        fn()
    for w in words:
        assert w in str(e.value), str(e.value)
    assert e.value.code == code


def spec(n, pd="bf16", gd="bf16", h=0):
    return D.TensorSpec(n, pd, gd, h)


@pytest.mark.parametrize("sizes", [[], [0], [1], [0, 1, 0, 128, 129, 0], [2047, 2048, 2049], [5] * 600])
@pytest.mark.parametrize("state", ["f32", "e4m3"])
def test_offsets(sizes, state):
    L = D.dopt_list_build([spec(n) for n in sizes], state)
    at = blocks = 0
    for n, t in zip(sizes, L.tensors()):
        assert (t["numel"], t["arena_offset"], t["export_offset"], t["param"]) == (n, 128 * blocks, at, -1)
        at += n
        blocks += -(-n // 128)
    assert (L.n_tensors, L.numel, L.arena_numel, L.n_blocks) == (len(sizes), at, 128 * blocks, blocks)
    assert L.has_master == bool(sizes) and L.state_kind == state
    assert L.workspace_bytes % 256 == 0 and L.workspace_bytes > L.stats_record_offset
    assert set(L.state_arrays()) == ({"master"} if sizes else set()) | {"exp_avg", "exp_avg_sq"} | (
        {"exp_avg_scale", "exp_avg_sq_scale"} if state == "e4m3" else set())
    _err(lambda: L.tensor(len(sizes)), "tensor index", code=-5)


@pytest.mark.parametrize("name", ["tiny", "gpt2-small", "llama3-8b", "llama3-70b"])
def test_shard_list_is_the_layouts_model_space(name):
    w = WORKLOADS[name]
    params = PARAM_LISTS[w.model]()
    lay = D.dopt_build_ranges(params, w.dp_size, w.dp_rank, w.bucket_size, w.pad_for_high_busbw)
    L = D.dopt_list_from_layout(lay, "e4m3")
    assert L.numel == lay.state_numel
    for t in L.tensors():
        q = lay.param(t["param"])
        assert q["has_shard"] and t["numel"] == q["param"][1] - q["param"][0]
        assert t["export_offset"] == q["export_offset"] and t["hgroup"] == q["hgroup"]
        assert (t["param_dtype"], t["grad_dtype"]) == params[t["param"]][2:4]
    assert [t["param"] for t in L.tensors()] == [p for p in range(len(params)) if lay.param(p)["has_shard"]]


def test_shard_views():
    params = [ParamSpec("a", 1000, "bf16", "f32"), ParamSpec("b", 300, "f32", "f32"), ParamSpec("c", 77, "bf16", "f32")]
    lay = D.dopt_build_ranges(params, 2, 1, 0)
    L = D.dopt_list_from_layout(lay)
    bufs = [{"param": torch.arange(i["arena_numel"]), "grad": -torch.arange(i["arena_numel"])} for i in lay.infos()]
    ps, gs = D.shard_views(lay, L, bufs)
    for t, p, g in zip(L.tensors(), ps, gs):
        a = lay.param(t["param"])["arena_offset"]
        assert p.tolist() == list(range(a, a + t["numel"])) and g.tolist() == [-x for x in p.tolist()]
    own = D.dopt_list_build([spec(3)])
    _err(lambda: D.shard_views(lay, own, bufs), "not built from a layout")


def test_build_refusals():
    _err(lambda: D.dopt_list_build([spec(3), spec(-1)]), "tensor 1", "numel")
    _err(lambda: D.dopt_list_build([spec(3, pd=7)]), "tensor 0", "dtype")
    _err(lambda: D.dopt_list_build([spec(3, gd=-1)]), "tensor 0", "dtype")
    _err(lambda: D.dopt_list_build([spec(3, h=16)]), "hgroup")
    _err(lambda: D.dopt_list_build([spec(3, h=-1)]), "hgroup")
    _err(lambda: D.dopt_list_build([spec(1 << 37), spec(1 << 37), spec(1)]), "2^38")
    _err(lambda: D.dopt_list_build([spec(3)], "int8"), "int8")
    h = ctypes.c_void_p()
    assert D.lib().dopt_list_build(None, 1, 0, ctypes.byref(h)) == -1
    assert D.lib().dopt_list_build(None, -1, 0, ctypes.byref(h)) == -1
    assert D.lib().dopt_list_build(None, 0, 2, ctypes.byref(h)) == -1
    assert D.lib().dopt_list_from_layout(None, 0, ctypes.byref(h)) == -1
    assert D.lib().dopt_list_query(None, None) == -1


def _raw_state(L):
    return {k: 4096 for k in L.state_arrays()}


def test_marshalling_refusals():
    L = D.dopt_list_build([spec(100), spec(7, "f32", "f32"), spec(0)], "e4m3")
    st = _raw_state(L)
    D.list_tensors(L, [4096, 8192, None], [4098, 8196, None], st)
    _err(lambda: D.list_tensors(L, [4096, 8192], None, st), "2 params")
    _err(lambda: D.list_tensors(L, [4096, 8192, None], [4096], st), "1 grads")
    _err(lambda: D.list_tensors(L, [4096, None, None], None, st), "tensor 1 param", "missing")
    _err(lambda: D.list_tensors(L, [torch.zeros(100), 8192, None], None, st), "tensor 0 param", "dtype")
    host = torch.zeros(100, dtype=torch.bfloat16)
    _err(lambda: D.list_tensors(L, [host, 8192, None], None, st), "tensor 0 param", "not a device tensor")
    _err(lambda: D.list_tensors(L, [torch.zeros(100, 2, dtype=torch.bfloat16)[:, 0], 8192, None], None, st), "contiguous")
    _err(lambda: D.list_tensors(L, [4096, 8192, None], None, {**st, "exp_avg": torch.zeros(256)}), "exp_avg", "dtype")
    _err(lambda: D.list_tensors(L, [4096, 8192, None], None, {**st, "master": torch.zeros(255)}), "master", "at least 256")
    _err(lambda: D.list_tensors(L, [4096, 8192, None], None, {k: v for k, v in st.items() if k != "exp_avg_sq_scale"}),
         "exp_avg_sq_scale", "missing")


class _Dev(torch.Tensor):
    """A host tensor that says it is a device tensor, for the checks that come after that one."""
    is_cuda = True


def _dev(n, dt=torch.bfloat16):
    return torch.zeros(n, dtype=dt).as_subclass(_Dev)


def test_overlaps_are_refused():
    L = D.dopt_list_build([spec(100), spec(50)], "f32")
    st = _raw_state(L)
    a = _dev(150)
    D.list_tensors(L, [a[:100], a[100:]], None, st)
    _err(lambda: D.list_tensors(L, [a[:100], a[99:149]], None, st), "tensor 1 param overlaps tensor 0 param")
    b = _dev(100)
    _err(lambda: D.list_tensors(L, [b, a[:50]], [a[100:150].repeat(2)[:100].as_subclass(_Dev), a[49:99]], st),
         "tensor 1 grad overlaps tensor 1 param")
    g = _dev(100)
    D.list_tensors(L, [b, a[:50]], [g, g[:50]], st)  # shared grads are only read
    _err(lambda: D.list_tensors(L, [b, b[:50]], None, st), "tensor 0 param overlaps tensor 1 param")
    both = D.dopt_list_build([D.TensorSpec(256, "f32", "f32")], "f32")
    w = _dev(256, torch.float32)
    _err(lambda: D.list_tensors(both, [w], None, {**_raw_state(both), "exp_avg": w}), "param overlaps state exp_avg")
    m = _dev(256, torch.float32)
    _err(lambda: D.list_tensors(L, [b, a[:50]], None, {**st, "exp_avg": m, "exp_avg_sq": m}), "overlaps state")
    _err(lambda: D.list_tensors(L, [b, a[:50]], [_dev(99), g[:50]], st), "tensor 0 grad", "99 elements")


def test_call_refusals():
    """Raw addresses pass the binding; the library refuses before any launch."""
    L = D.dopt_list_build([spec(100, h=1), spec(7, "f32", "f32")], "e4m3")
    st = _raw_state(L)
    t = D.list_tensors(L, [4096, 8192], [4096, 8192], st)
    nograd = D.list_tensors(L, [4096, 8192], None, st)
    other = D.dopt_list_build([spec(100)], "e4m3")
    hp2 = HP * 2
    _err(lambda: D.dopt_list_step(other, t, HP, 1.0, 4096), "another list")
    _err(lambda: D.dopt_list_step(L, nograd, hp2, 1.0, 4096), "without grads")
    _err(lambda: D.dopt_list_step(L, t, HP, 1.0, 4096), "n_hgroups")
    _err(lambda: D.dopt_list_step(L, t, [(-1, 0.9, 0.999, 1e-8, 0.0)] * 2, 1.0, 4096), "hparams 0")
    _err(lambda: D.dopt_list_step(L, t, hp2, 1.0, 4096 + 128), "workspace", "aligned")
    _err(lambda: D.dopt_list_finalize(L, HP, 1.0, 4096), "n_hgroups")
    _err(lambda: D.dopt_list_stats(L, t, torch.zeros(L.workspace_bytes - 1, dtype=torch.uint8)), "workspace", "bytes")
    odd = D.list_tensors(L, [4097, 8192], [4096, 8192], st)
    for call in (lambda: D.dopt_list_step(L, odd, hp2, 1.0, 4096), lambda: D.dopt_list_apply(L, odd, 4096),
                 lambda: D.dopt_list_init(L, odd, D.scaler_cfg(), 4096),
                 lambda: D.dopt_list_export(L, odd, 4096, 4096, 4096, 4096)):
        _err(call, "tensor 0", "not aligned to its element")
    odd = D.list_tensors(L, [4096, 8192], [4096, 8194], st)
    _err(lambda: D.dopt_list_stats(L, odd, 4096), "tensor 1", "not aligned")
    odd = D.list_tensors(L, [4096, 8192], [4096, 8192], {**st, "exp_avg_sq": 4096 + 128})
    _err(lambda: D.dopt_list_apply(L, odd, 4096), "state", "256-byte")
    _err(lambda: D.dopt_list_init(L, t, D.scaler_cfg(initial_scale=float("inf")), 4096), "scale")
    _err(lambda: D.dopt_list_import(L, t, 4096, 4098, 4096, 4096), "4-byte")
    _err(lambda: D.dopt_list_export(L, t, torch.zeros(106), 4096, 4096, 4096), "export master", "at least 107")
    _err(lambda: D.dopt_list_scalars_set(L, 4096, {"step_count": -1, "loss_scale": 1.0, "growth_tracker": 0,
                                                   "hysteresis_tracker": 1}), "step_count")
    lib, z = D.lib(), D.dopt_list_state()
    hp = D.hparams_array(hp2)
    assert lib.dopt_list_step(L.handle, t.ptrs, ctypes.byref(z), hp, 2, 1.0, 4096, None, None) == -1
    assert "null device pointer" in D.dopt_last_error()
    assert lib.dopt_list_step(L.handle, None, ctypes.byref(t.state), hp, 2, 1.0, 4096, None, None) == -1
    assert lib.dopt_list_step(L.handle, t.ptrs, None, hp, 2, 1.0, 4096, None, None) == -1
    assert lib.dopt_list_step(L.handle, t.ptrs, ctypes.byref(t.state), None, 2, 1.0, 4096, None, None) == -1
    assert lib.dopt_list_step(None, t.ptrs, ctypes.byref(t.state), hp, 2, 1.0, 4096, None, None) == -1
    assert lib.dopt_list_read_stats(L.handle, None, None, None) == -1


def test_tensors_of_a_freed_list_are_refused():
    """Lists built and dropped in turn, whose handles may reuse an address:
    tensors marshalled for one never pass for the next."""
    old = []
    for n in range(1, 40):
        L = D.dopt_list_build([spec(n)], "f32")
        for t in old:
            _err(lambda: D.dopt_list_stats(L, t, 4096 + 128), "another list")
        old.append(D.list_tensors(L, [4096], [4096], _raw_state(L)))
        del L


class _Elsewhere:
    """Stands for a stream of another device than the current one."""
    cuda_stream = 0

    class device:
        index = 5


def test_other_devices_are_refused(monkeypatch):
    L = D.dopt_list_build([spec(100)], "f32")
    t = D.list_tensors(L, [4096], [4096], _raw_state(L))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    _err(lambda: D.dopt_list_step(L, t, HP, 1.0, 4096, _Elsewhere()), "stream on device 5", "current device is 3")
    _err(lambda: D.dopt_list_finalize(L, HP, 1.0, 4096, _Elsewhere()), "stream on device 5")
    t.device = 4
    _err(lambda: D.dopt_list_apply(L, t, 4096), "tensors on device 4")


# ---- the plain encoding that the GPU tests compare with ---------------------------------------

def test_e4m3_rounding_is_nearest_even():
    grid = np.sort(np.unique(H._CODES[np.isfinite(H._CODES)])).astype(np.float64)
    mid = (grid[1:] + grid[:-1]) / 2
    q = np.concatenate([grid, mid, np.nextafter(mid, 1e9), np.nextafter(mid, -1e9)])
    got = H.e4m3_round(q)
    d = np.abs(q[:, None] - grid[None])
    assert np.array_equal(np.abs(q - got), d.min(1))
    ties = (d == d.min(1)[:, None]).sum(1) == 2
    assert ties.sum() >= 250
    code = H.e4m3_code(got[ties])
    assert (code[got[ties] != 0] & 1 == 0).all()


@pytest.mark.parametrize("kind", ["m", "r"])
@pytest.mark.parametrize("spread", [1.0, 4.0, 20.0])
def test_plain_encoding_holds_its_bounds(kind, spread):
    rng = np.random.default_rng(int(spread))
    x = (np.exp(rng.standard_normal(5000) * spread) * np.where(rng.random(5000) < 0.5, -1, 1)).astype(np.float32)
    x[rng.random(5000) < 0.1] = 0
    if kind == "r":
        x = np.minimum(np.abs(x), H.CAP["r"])  # the root of an fp32 number is below 2^64
    c, s = H.encode(x, kind)
    H.near_e4m3(kind, c, s, x.astype(np.float64), np.zeros(5000), kind == "r")
    if kind == "r":
        assert ((H.e4m3_value(c) > 0) == (x > 0)).all()


def test_plain_encoding_at_its_ends():
    x = np.zeros(128 * 7, np.float32)
    x[0], x[1] = 2.0 ** -101, -2.0 ** -110          # below the smallest block: zeros
    x[128], x[129] = 3e38, -1e38                    # cut at 2^127, finite
    x[256], x[257] = np.inf, 1.0
    x[384], x[385] = np.nan, 1.0
    x[512] = 2.0 ** -100
    x[640:768] = 1.0
    c, s = H.encode(x, "m")
    with np.errstate(all="ignore"):
        y = H.decode(c, s)
    assert s[0] == 0 and not c[:128].any()
    assert np.isfinite(y[128:384]).all() and y[128] > 1.6e38 and y[256] > 1.6e38
    assert np.isnan(y[384:512]).all() and not np.isnan(y[512:]).any()
    assert y[512] > 0 and np.allclose(y[640:768], 1.0, rtol=2e-7)
    assert s[6] == 0
