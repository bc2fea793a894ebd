"""Python binding of libdopt.so, the shard-local mixed-precision AdamW step
of a ZeRO-1 distributed optimizer for AMD Instinct MI355X (gfx950), and the
same step over a list of separate tensors with fp32 or 8-bit moments.

Argument marshalling only: every computation happens in the library (host
range mapper in C++, the step in HIP kernels).  Function names match the C
ABI in include/dopt.h and include/dopt_list.h.  Device buffers may be given as PyTorch CUDA tensors
or raw integer addresses; PyTorch is used only to own device memory and
streams.  There is no fallback: if the library is not built, import fails.
"""
from __future__ import annotations

import ctypes
import os
from typing import Dict, List, NamedTuple, Optional, Sequence, Tuple

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdopt.so")

DOPT_F32, DOPT_BF16, DOPT_F16 = 0, 1, 2
DTYPES = {"f32": DOPT_F32, "bf16": DOPT_BF16, "f16": DOPT_F16}
DTYPE_NAMES = {v: k for k, v in DTYPES.items()}
DOPT_SCALER_CONSTANT, DOPT_SCALER_DYNAMIC = 0, 1
GROUP_KINDS = {"model_float16": 0, "model_fp32": 1, "shard_float16": 2, "shard_fp32_from_float16": 3,
               "shard_fp32": 4}
DOPT_MAX_HGROUPS = 16
DOPT_ARENA_ALIGN = 2048
DOPT_PTR_ALIGN = 256


DOPT_STATE_F32, DOPT_STATE_E4M3, DOPT_STATE_E4M3_SR = 0, 1, 3
STATE_KINDS = {"f32": DOPT_STATE_F32, "e4m3": DOPT_STATE_E4M3, "e4m3_sr": DOPT_STATE_E4M3_SR}
STATE_NAMES = {v: k for k, v in STATE_KINDS.items()}
DOPT_LIST_BLOCK = 128


class DoptError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"dopt error {code}: {msg}")
        self.code = code


class dopt_param_desc(ctypes.Structure):
    _fields_ = [("numel", ctypes.c_int64), ("param_dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32),
                ("requires_new_bucket", ctypes.c_int32), ("hgroup", ctypes.c_int32)]


class dopt_shard_cfg(ctypes.Structure):
    _fields_ = [("dp_size", ctypes.c_int32), ("dp_rank", ctypes.c_int32), ("bucket_size", ctypes.c_int64),
                ("pad_for_high_busbw", ctypes.c_int32), ("num_instances", ctypes.c_int32)]


class dopt_sharding_info(ctypes.Structure):
    _fields_ = [("dp_size", ctypes.c_int32), ("dp_rank", ctypes.c_int32), ("num_instances", ctypes.c_int32),
                ("instance_size", ctypes.c_int32), ("instance_index", ctypes.c_int32),
                ("instance_rank", ctypes.c_int32)]


class dopt_range(ctypes.Structure):
    _fields_ = [("start", ctypes.c_int64), ("end", ctypes.c_int64)]

    def tuple(self):
        return (self.start, self.end)


class dopt_buffer_info(ctypes.Structure):
    _fields_ = [("param_dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32), ("n_buckets", ctypes.c_int32),
                ("n_params", ctypes.c_int32), ("numel", ctypes.c_int64), ("numel_unpadded", ctypes.c_int64),
                ("window_numel", ctypes.c_int64), ("arena_numel", ctypes.c_int64), ("shard_numel", ctypes.c_int64),
                ("apply_bnd", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class dopt_bucket_info(ctypes.Structure):
    _fields_ = [("offset", ctypes.c_int64), ("numel", ctypes.c_int64), ("numel_unpadded", ctypes.c_int64),
                ("shard_size", ctypes.c_int64), ("window_start", ctypes.c_int64), ("arena_offset", ctypes.c_int64),
                ("n_params", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class dopt_param_info(ctypes.Structure):
    _fields_ = [("buffer", ctypes.c_int32), ("bucket", ctypes.c_int32), ("has_shard", ctypes.c_int32),
                ("hgroup", ctypes.c_int32), ("start", ctypes.c_int64), ("end", ctypes.c_int64),
                ("gbuf_world", dopt_range), ("gbuf_world_in_bucket", dopt_range), ("gbuf_local", dopt_range),
                ("param", dopt_range), ("arena_offset", ctypes.c_int64), ("export_offset", ctypes.c_int64)]


class dopt_buffer_tensors(ctypes.Structure):
    _fields_ = [("grad", ctypes.c_void_p), ("param", ctypes.c_void_p), ("master", ctypes.c_void_p),
                ("exp_avg", ctypes.c_void_p), ("exp_avg_sq", ctypes.c_void_p)]


class dopt_scaler_cfg(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("hysteresis", ctypes.c_int32), ("growth_interval", ctypes.c_int64),
                ("initial_scale", ctypes.c_double), ("growth_factor", ctypes.c_double),
                ("backoff_factor", ctypes.c_double), ("min_scale", ctypes.c_double)]


class dopt_hparams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double)]


class dopt_state_scalars(ctypes.Structure):
    _fields_ = [("step_count", ctypes.c_int64), ("loss_scale", ctypes.c_double),
                ("growth_tracker", ctypes.c_int64), ("hysteresis_tracker", ctypes.c_int64)]


class dopt_stats(ctypes.Structure):
    _fields_ = [("found_inf", ctypes.c_int32), ("skipped", ctypes.c_int32), ("clip_applied", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("sumsq", ctypes.c_double), ("grad_norm", ctypes.c_double),
                ("clip_coef", ctypes.c_double), ("num_zeros", ctypes.c_uint64), ("loss_scale_used", ctypes.c_double),
                ("loss_scale_next", ctypes.c_double), ("step_count", ctypes.c_int64)]

    def as_dict(self) -> Dict:
        return {name: getattr(self, name) for name, _ in self._fields_ if name != "reserved"}


class dopt_tensor_desc(ctypes.Structure):
    _fields_ = [("numel", ctypes.c_int64), ("param_dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32),
                ("hgroup", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class dopt_list_info(ctypes.Structure):
    _fields_ = [("n_tensors", ctypes.c_int64), ("numel", ctypes.c_int64), ("arena_numel", ctypes.c_int64),
                ("n_blocks", ctypes.c_int64), ("workspace_bytes", ctypes.c_int64),
                ("stats_record_offset", ctypes.c_int64), ("state_kind", ctypes.c_int32),
                ("has_master", ctypes.c_int32)]


class dopt_list_tensor_info(ctypes.Structure):
    _fields_ = [("numel", ctypes.c_int64), ("arena_offset", ctypes.c_int64), ("export_offset", ctypes.c_int64),
                ("param", ctypes.c_int64), ("param_dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32),
                ("hgroup", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class dopt_list_ptrs(ctypes.Structure):
    _fields_ = [("grad", ctypes.c_void_p), ("param", ctypes.c_void_p)]


class dopt_list_state(ctypes.Structure):
    _fields_ = [("master", ctypes.c_void_p), ("exp_avg", ctypes.c_void_p), ("exp_avg_sq", ctypes.c_void_p),
                ("exp_avg_scale", ctypes.c_void_p), ("exp_avg_sq_scale", ctypes.c_void_p)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() or "
                          "python sharded_mixed_precision_amd/build.py")
    L = ctypes.CDLL(LIB_PATH)
    P, I32, I64, VP, D = ctypes.POINTER, ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_double
    sig = {
        "dopt_build_ranges": ([P(dopt_param_desc), I64, P(dopt_shard_cfg), P(VP)], ctypes.c_int),
        "dopt_layout_free": ([VP], None),
        "dopt_layout_num_buffers": ([VP], I32),
        "dopt_layout_sharding": ([VP, P(dopt_sharding_info)], ctypes.c_int),
        "dopt_layout_buffer": ([VP, I32, P(dopt_buffer_info)], ctypes.c_int),
        "dopt_layout_bucket": ([VP, I32, I32, P(dopt_bucket_info)], ctypes.c_int),
        "dopt_layout_rank_window": ([VP, I32, I32, I32, P(dopt_range)], ctypes.c_int),
        "dopt_layout_param": ([VP, I64, P(dopt_param_info)], ctypes.c_int),
        "dopt_layout_group": ([VP, I32, I32, VP, I64], I64),
        "dopt_layout_state_numel": ([VP], I64),
        "dopt_workspace_bytes": ([VP], I64),
        "dopt_init_state": ([VP, P(dopt_buffer_tensors), P(dopt_scaler_cfg), VP, VP], ctypes.c_int),
        "dopt_step": ([VP, P(dopt_buffer_tensors), P(dopt_hparams), I32, D, VP, VP, P(dopt_stats)], ctypes.c_int),
        "dopt_step_prepare": ([VP, P(dopt_buffer_tensors), P(dopt_hparams), I32, D, VP, VP], ctypes.c_int),
        "dopt_step_stats": ([VP, P(dopt_buffer_tensors), VP, VP], ctypes.c_int),
        "dopt_reduce_prepare": ([VP, P(dopt_buffer_tensors), P(VP), P(I64), I32, I32, ctypes.c_float, P(dopt_hparams),
                                 I32, D, VP, VP], ctypes.c_int),
        "dopt_check_grads": ([VP, I32, VP, D, VP, VP, VP], ctypes.c_int),
        "dopt_check_grads_noalloc": ([VP, I32, VP, D, VP, VP], ctypes.c_int),
        "dopt_step_finalize": ([VP, P(dopt_hparams), I32, D, VP, VP], ctypes.c_int),
        "dopt_step_apply": ([VP, P(dopt_buffer_tensors), VP, VP], ctypes.c_int),
        "dopt_state_export": ([VP, P(dopt_buffer_tensors), VP, VP, VP, VP, VP], ctypes.c_int),
        "dopt_state_import": ([VP, P(dopt_buffer_tensors), VP, VP, VP, VP, VP], ctypes.c_int),
        "dopt_state_scalars_get": ([VP, VP, VP, P(dopt_state_scalars)], ctypes.c_int),
        "dopt_state_scalars_set": ([VP, VP, VP, P(dopt_state_scalars)], ctypes.c_int),
        "dopt_stats_record_offset": ([VP], I64),
        "dopt_read_stats": ([VP, VP, VP, P(dopt_stats)], ctypes.c_int),
        "dopt_last_error": ([], ctypes.c_char_p),
        "dopt_list_build": ([P(dopt_tensor_desc), I64, I32, P(VP)], ctypes.c_int),
        "dopt_list_from_layout": ([VP, I32, P(VP)], ctypes.c_int),
        "dopt_list_free": ([VP], None),
        "dopt_list_query": ([VP, P(dopt_list_info)], ctypes.c_int),
        "dopt_list_tensor": ([VP, I64, P(dopt_list_tensor_info)], ctypes.c_int),
        "dopt_list_init": ([VP, P(dopt_list_ptrs), P(dopt_list_state), P(dopt_scaler_cfg), VP, VP], ctypes.c_int),
        "dopt_list_step": ([VP, P(dopt_list_ptrs), P(dopt_list_state), P(dopt_hparams), I32, D, VP, VP,
                            P(dopt_stats)], ctypes.c_int),
        "dopt_list_prepare": ([VP, P(dopt_list_ptrs), P(dopt_hparams), I32, D, VP, VP], ctypes.c_int),
        "dopt_list_stats": ([VP, P(dopt_list_ptrs), VP, VP], ctypes.c_int),
        "dopt_list_finalize": ([VP, P(dopt_hparams), I32, D, VP, VP], ctypes.c_int),
        "dopt_list_apply": ([VP, P(dopt_list_ptrs), P(dopt_list_state), VP, VP], ctypes.c_int),
        "dopt_list_export": ([VP, P(dopt_list_ptrs), P(dopt_list_state), VP, VP, VP, VP, VP], ctypes.c_int),
        "dopt_list_import": ([VP, P(dopt_list_ptrs), P(dopt_list_state), VP, VP, VP, VP, VP], ctypes.c_int),
        "dopt_list_set_seed": ([VP, ctypes.c_uint64, VP, VP], ctypes.c_int),
        "dopt_list_scalars_get": ([VP, VP, VP, P(dopt_state_scalars)], ctypes.c_int),
        "dopt_list_scalars_set": ([VP, VP, VP, P(dopt_state_scalars)], ctypes.c_int),
        "dopt_list_read_stats": ([VP, VP, VP, P(dopt_stats)], ctypes.c_int),
        "dopt_vmm_granularity": ([I32, P(ctypes.c_size_t)], ctypes.c_int),
        "dopt_vmm_reserve": ([ctypes.c_size_t, ctypes.c_size_t, P(ctypes.c_uint64)], ctypes.c_int),
        "dopt_vmm_free": ([ctypes.c_uint64, ctypes.c_size_t], ctypes.c_int),
        "dopt_vmm_create": ([I32, ctypes.c_size_t, P(ctypes.c_uint64)], ctypes.c_int),
        "dopt_vmm_map": ([ctypes.c_uint64, ctypes.c_size_t, ctypes.c_uint64], ctypes.c_int),
        "dopt_vmm_set_access": ([ctypes.c_uint64, ctypes.c_size_t, I32], ctypes.c_int),
        "dopt_vmm_unmap": ([ctypes.c_uint64, ctypes.c_size_t], ctypes.c_int),
        "dopt_vmm_release": ([ctypes.c_uint64], ctypes.c_int),
    }
    for name, (args, res) in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = res
    return L


_lib = _load()
EXPORTED = ("dopt_build_ranges", "dopt_layout_free", "dopt_layout_num_buffers", "dopt_layout_sharding",
            "dopt_layout_buffer",
            "dopt_layout_bucket", "dopt_layout_rank_window", "dopt_layout_param", "dopt_layout_group",
            "dopt_layout_state_numel", "dopt_workspace_bytes", "dopt_init_state", "dopt_step", "dopt_step_prepare", "dopt_step_stats",
            "dopt_step_finalize", "dopt_step_apply", "dopt_reduce_prepare", "dopt_check_grads",
            "dopt_check_grads_noalloc",
            "dopt_state_export", "dopt_state_import", "dopt_state_scalars_get", "dopt_state_scalars_set",
            "dopt_stats_record_offset",
            "dopt_read_stats",
            "dopt_last_error",
            "dopt_list_build", "dopt_list_from_layout", "dopt_list_free", "dopt_list_query", "dopt_list_tensor",
            "dopt_list_init", "dopt_list_step", "dopt_list_prepare", "dopt_list_stats", "dopt_list_finalize",
            "dopt_list_apply", "dopt_list_export", "dopt_list_import", "dopt_list_set_seed", "dopt_list_scalars_get",
            "dopt_list_scalars_set", "dopt_list_read_stats",
            "dopt_vmm_granularity", "dopt_vmm_reserve", "dopt_vmm_free", "dopt_vmm_create", "dopt_vmm_map",
            "dopt_vmm_set_access", "dopt_vmm_unmap", "dopt_vmm_release")


def lib():
    return _lib


def _check(rc: int):
    if rc != 0:
        raise DoptError(rc, _lib.dopt_last_error().decode())


def _addr(x) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


DOPT_ERR_INVALID = -1
_TORCH_DTYPE_NAMES = {"f32": "torch.float32", "bf16": "torch.bfloat16", "f16": "torch.float16",
                      "e4m3": "torch.float8_e4m3fn"}


_dtype_names: Dict = {}  # of the element types seen


def _dtype_name(dt) -> str:
    name = _dtype_names.get(dt)
    if name is None:
        name = _dtype_names[dt] = str(dt)
    return name


def _what(name) -> str:
    """An argument's name: a text, or (word, index, word), joined only when it is needed."""
    return name if isinstance(name, str) else "%s %d %s" % name


def _dev(x, what, dtype: Optional[str] = None, min_numel: int = 0, min_bytes: int = 0) -> int:
    """Device address of ``x`` after checking it against what the library
    will touch: a contiguous device tensor of the given element type holding
    at least ``min_numel`` elements / ``min_bytes`` bytes.  The library cannot
    check sizes itself (it receives bare pointers), and a short buffer would
    make its kernels read or write past the end.  A raw integer address is
    passed through: its size and type are then the caller's to guarantee."""
    if x is None:
        raise DoptError(DOPT_ERR_INVALID, f"{_what(what)}: missing")
    if isinstance(x, int):
        return x
    if dtype is not None and _dtype_name(x.dtype) != _TORCH_DTYPE_NAMES[dtype]:
        raise DoptError(DOPT_ERR_INVALID, f"{_what(what)}: dtype {x.dtype}, the layout needs {_TORCH_DTYPE_NAMES[dtype]}")
    if x.numel() < min_numel:
        raise DoptError(DOPT_ERR_INVALID, f"{_what(what)}: {x.numel()} elements, the layout needs at least {min_numel}")
    if x.numel() * x.element_size() < min_bytes:
        raise DoptError(DOPT_ERR_INVALID,
                        f"{_what(what)}: {x.numel() * x.element_size()} bytes, the layout needs at least {min_bytes}")
    if not x.is_contiguous():
        raise DoptError(DOPT_ERR_INVALID, f"{_what(what)}: not contiguous")
    if not getattr(x, "is_cuda", False):
        raise DoptError(DOPT_ERR_INVALID, f"{_what(what)}: not a device tensor")
    return x.data_ptr()


def _stream(s) -> Optional[int]:
    if s is None:
        return None
    if isinstance(s, int):
        return s
    return s.cuda_stream


class Layout:
    """Owns a dopt_layout handle (freed with the object)."""

    def __init__(self, handle: ctypes.c_void_p, dp_size: int, dp_rank: int, n_params: int):
        self._h = handle
        self._free = _lib.dopt_layout_free  # kept so that freeing works during interpreter shutdown
        self.dp_size, self.dp_rank, self.n_params = dp_size, dp_rank, n_params

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None:
            self._free(h)
            self._h = None

    @property
    def handle(self):
        return self._h

    @property
    def num_buffers(self) -> int:
        return int(_lib.dopt_layout_num_buffers(self._h))

    def infos(self) -> List[Dict]:
        """dopt_layout_buffer of every buffer, with the dtype names (cached;
        the layout is immutable)."""
        if getattr(self, "_infos", None) is None:
            out = []
            for k in range(self.num_buffers):
                b = self.buffer(k)
                out.append({**b, "pd": DTYPE_NAMES[b["param_dtype"]], "gd": DTYPE_NAMES[b["grad_dtype"]]})
            self._infos = out
        return self._infos

    def sharding(self) -> Dict:
        o = dopt_sharding_info()
        _check(_lib.dopt_layout_sharding(self._h, ctypes.byref(o)))
        return {name: getattr(o, name) for name, _ in o._fields_}

    def buffer(self, k: int) -> Dict:
        o = dopt_buffer_info()
        _check(_lib.dopt_layout_buffer(self._h, k, ctypes.byref(o)))
        return {name: getattr(o, name) for name, _ in o._fields_ if name != "reserved"}

    def bucket(self, k: int, b: int) -> Dict:
        o = dopt_bucket_info()
        _check(_lib.dopt_layout_bucket(self._h, k, b, ctypes.byref(o)))
        return {name: getattr(o, name) for name, _ in o._fields_ if name != "reserved"}

    def rank_window(self, k: int, b: int, rank: int):
        o = dopt_range()
        _check(_lib.dopt_layout_rank_window(self._h, k, b, rank, ctypes.byref(o)))
        return o.tuple()

    def param(self, p: int) -> Dict:
        o = dopt_param_info()
        _check(_lib.dopt_layout_param(self._h, p, ctypes.byref(o)))
        d = {name: getattr(o, name) for name, _ in o._fields_}
        for key in ("gbuf_world", "gbuf_world_in_bucket", "gbuf_local", "param"):
            d[key] = d[key].tuple()
        return d

    def group(self, kind: str, hgroup: int = 0) -> List[int]:
        k = GROUP_KINDS[kind]
        n = _lib.dopt_layout_group(self._h, k, hgroup, None, 0)
        if n < 0:
            _check(int(n))
        arr = (ctypes.c_int64 * max(n, 1))()
        _lib.dopt_layout_group(self._h, k, hgroup, arr, n)
        return list(arr[:n])

    @property
    def state_numel(self) -> int:
        return int(_lib.dopt_layout_state_numel(self._h))

    @property
    def workspace_bytes(self) -> int:
        return int(_lib.dopt_workspace_bytes(self._h))

    @property
    def stats_record_offset(self) -> int:
        return int(_lib.dopt_stats_record_offset(self._h))


def dopt_build_ranges(params: Sequence, dp_size: int, dp_rank: int, bucket_size: int = 0,
                      pad_for_high_busbw: int = 0, num_instances: int = 1) -> Layout:
    """params: objects with numel, param_dtype, grad_dtype ('f32'|'bf16'|'f16'),
    optional requires_new_bucket and hgroup, in model order."""
    n = len(params)
    arr = (dopt_param_desc * n)()
    for i, p in enumerate(params):
        arr[i].numel = p.numel
        arr[i].param_dtype = DTYPES[p.param_dtype] if isinstance(p.param_dtype, str) else p.param_dtype
        arr[i].grad_dtype = DTYPES[p.grad_dtype] if isinstance(p.grad_dtype, str) else p.grad_dtype
        arr[i].requires_new_bucket = int(getattr(p, "requires_new_bucket", 0))
        arr[i].hgroup = int(getattr(p, "hgroup", 0))
    cfg = dopt_shard_cfg(dp_size, dp_rank, bucket_size, pad_for_high_busbw, num_instances)
    h = ctypes.c_void_p()
    _check(_lib.dopt_build_ranges(arr, n, ctypes.byref(cfg), ctypes.byref(h)))
    return Layout(h, dp_size, dp_rank, n)


class Tensors:
    """The device arrays of every flat buffer, checked against one layout and
    marshalled into the C array of dopt_buffer_tensors (make it once with
    tensors() and pass it to every step)."""

    def __init__(self, layout: "Layout", arr: ctypes.Array, need_grad: bool):
        self.handle, self.arr, self.need_grad = layout.handle.value, arr, need_grad


def tensors(layout: "Layout", bufs: Sequence[Dict], need_grad: bool = True) -> Tensors:
    """bufs: per flat buffer a dict with grad, param, master (None for fp32
    params), exp_avg and exp_avg_sq, each of the buffer's arena_numel
    elements: device tensors (checked here) or raw device addresses."""
    infos = layout.infos()
    if len(bufs) != len(infos):
        raise DoptError(DOPT_ERR_INVALID, f"{len(bufs)} buffer entries, the layout has {len(infos)}")
    arr = (dopt_buffer_tensors * len(bufs))()
    for k, (b, inf) in enumerate(zip(bufs, infos)):
        n, pre = inf["arena_numel"], f"buffer {k} "
        if need_grad or b.get("grad") is not None:
            arr[k].grad = _dev(b.get("grad"), pre + "grad", inf["gd"], n)
        arr[k].param = _dev(b.get("param"), pre + "param", inf["pd"], n)
        if inf["pd"] != "f32":
            arr[k].master = _dev(b.get("master"), pre + "master", "f32", n)
        arr[k].exp_avg = _dev(b.get("exp_avg"), pre + "exp_avg", "f32", n)
        arr[k].exp_avg_sq = _dev(b.get("exp_avg_sq"), pre + "exp_avg_sq", "f32", n)
    return Tensors(layout, arr, need_grad)


def _marshal(layout: "Layout", bufs, need_grad: bool = True) -> ctypes.Array:
    if isinstance(bufs, Tensors):
        if bufs.handle != layout.handle.value:
            raise DoptError(DOPT_ERR_INVALID, "tensors were marshalled for another layout")
        if need_grad and not bufs.need_grad:
            raise DoptError(DOPT_ERR_INVALID, "tensors were marshalled without grads")
        return bufs.arr
    return tensors(layout, bufs, need_grad).arr


def _ws(layout: "Layout", workspace) -> int:
    return _dev(workspace, "workspace", None, 0, layout.workspace_bytes)


def scaler_cfg(dynamic: bool = False, initial_scale: float = 1.0, growth_factor: float = 2.0,
               backoff_factor: float = 0.5, growth_interval: int = 1000, hysteresis: int = 1,
               min_scale: float = 1.0) -> dopt_scaler_cfg:
    return dopt_scaler_cfg(DOPT_SCALER_DYNAMIC if dynamic else DOPT_SCALER_CONSTANT, hysteresis, growth_interval,
                           initial_scale, growth_factor, backoff_factor, min_scale)


def _hparams(hps: Sequence) -> ctypes.Array:
    arr = (dopt_hparams * len(hps))()
    for i, h in enumerate(hps):
        arr[i] = dopt_hparams(*h) if not isinstance(h, dopt_hparams) else h
    return arr


def dopt_init_state(layout: Layout, bufs: Sequence[Dict], scaler: dopt_scaler_cfg, workspace, stream=None):
    _check(_lib.dopt_init_state(layout.handle, _marshal(layout, bufs, False), ctypes.byref(scaler),
                                _ws(layout, workspace), _stream(stream)))


def dopt_step(layout: Layout, bufs, hparams: Sequence, max_grad_norm: float, workspace, stream=None,
              want_stats: bool = True):
    st = dopt_stats() if want_stats else None
    t = _marshal(layout, bufs)
    hp = hparams if isinstance(hparams, ctypes.Array) else _hparams(hparams)
    _check(_lib.dopt_step(layout.handle, t, hp, len(hparams), max_grad_norm, _ws(layout, workspace),
                          _stream(stream), ctypes.byref(st) if st is not None else None))
    return st.as_dict() if st is not None else None


def dopt_step_prepare(layout: Layout, bufs, hparams, max_grad_norm: float, workspace, stream=None):
    t = _marshal(layout, bufs)
    hp = hparams if isinstance(hparams, ctypes.Array) else _hparams(hparams)
    _check(_lib.dopt_step_prepare(layout.handle, t, hp, len(hp), max_grad_norm, _ws(layout, workspace),
                                  _stream(stream)))


def dopt_reduce_prepare(layout: Layout, bufs, chunks: Sequence, wire_dtype: str, n_chunks: int, scale: float,
                        hparams, max_grad_norm: float, workspace, stream=None, chunk_strides: Optional[Sequence] = None):
    """chunks: one device buffer per flat buffer holding n_chunks arenas,
    chunk j at element j * stride (stride = chunk_strides[k], default
    arena_numel: back to back).  hparams None: stats only (finalize later with
    dopt_step_finalize)."""
    t = _marshal(layout, bufs)
    infos = layout.infos()
    if len(chunks) != len(infos):
        raise DoptError(DOPT_ERR_INVALID, f"{len(chunks)} chunk buffers, the layout has {len(infos)}")
    if chunk_strides is not None and len(chunk_strides) != len(infos):
        raise DoptError(DOPT_ERR_INVALID, f"{len(chunk_strides)} chunk strides, the layout has {len(infos)} buffers")
    strides = [int(chunk_strides[k]) if chunk_strides is not None else inf["arena_numel"]
               for k, inf in enumerate(infos)]
    for k, (st, inf) in enumerate(zip(strides, infos)):
        if st < inf["arena_numel"]:
            raise DoptError(DOPT_ERR_INVALID, f"buffer {k}: chunk stride {st} below the arena ({inf['arena_numel']})")
    ch = (ctypes.c_void_p * len(chunks))(*[_dev(c, f"buffer {k} chunks", wire_dtype,
                                                max(n_chunks - 1, 0) * st + inf["arena_numel"])
                                            for k, (c, st, inf) in enumerate(zip(chunks, strides, infos))])
    cs = None if chunk_strides is None else (ctypes.c_int64 * len(strides))(*strides)
    if hparams is None:
        hp, nh = None, 0
    else:
        hp = hparams if isinstance(hparams, ctypes.Array) else _hparams(hparams)
        nh = len(hp)
    _check(_lib.dopt_reduce_prepare(layout.handle, t, ch, cs, DTYPES[wire_dtype], n_chunks, scale, hp, nh,
                                    max_grad_norm, _ws(layout, workspace), _stream(stream)))


class dopt_bucket_check(ctypes.Structure):
    _fields_ = [("sumsq", ctypes.c_double), ("max_abs", ctypes.c_float), ("has_nan", ctypes.c_int32),
                ("has_inf", ctypes.c_int32), ("large", ctypes.c_int32)]


BUCKET_CHECK_BYTES = ctypes.sizeof(dopt_bucket_check)


def dopt_check_grads(layout: Layout, k: int, grad_buffer, large_threshold: float, out, workspace, stream=None):
    """out: device buffer of n_buckets * BUCKET_CHECK_BYTES bytes (e.g. a uint8 CUDA tensor)."""
    infos = layout.infos()
    if not 0 <= k < len(infos):
        raise DoptError(-5, f"buffer index {k} out of range")
    g = _dev(grad_buffer, f"buffer {k} grad buffer", infos[k]["gd"], infos[k]["numel"])
    o = _dev(out, "bucket check output", None, 0, infos[k]["n_buckets"] * BUCKET_CHECK_BYTES)
    _check(_lib.dopt_check_grads(layout.handle, k, g, large_threshold, o, _ws(layout, workspace), _stream(stream)))


NOALLOC_SCRATCH_BYTES = 16 << 20


def dopt_check_grads_noalloc(layout: Layout, k: int, grad_buffer, large_threshold: float, out, stream=None):
    """dopt_check_grads without a workspace: the library's static device
    scratch holds the tables and partials (no allocation in the call)."""
    infos = layout.infos()
    if not 0 <= k < len(infos):
        raise DoptError(-5, f"buffer index {k} out of range")
    g = _dev(grad_buffer, f"buffer {k} grad buffer", infos[k]["gd"], infos[k]["numel"])
    o = _dev(out, "bucket check output", None, 0, infos[k]["n_buckets"] * BUCKET_CHECK_BYTES)
    _check(_lib.dopt_check_grads_noalloc(layout.handle, k, g, large_threshold, o, _stream(stream)))


def bucket_checks(raw: bytes, n: int) -> List[Dict]:
    """Decode n dopt_bucket_check records copied to the host."""
    arr = (dopt_bucket_check * n).from_buffer_copy(raw)
    return [{name: getattr(r, name) for name, _ in r._fields_} for r in arr]


def dopt_step_stats(layout: Layout, bufs, workspace, stream=None):
    t = _marshal(layout, bufs)
    _check(_lib.dopt_step_stats(layout.handle, t, _ws(layout, workspace), _stream(stream)))


def dopt_step_finalize(layout: Layout, hparams, max_grad_norm: float, workspace, stream=None):
    hp = hparams if isinstance(hparams, ctypes.Array) else _hparams(hparams)
    _check(_lib.dopt_step_finalize(layout.handle, hp, len(hp), max_grad_norm, _ws(layout, workspace),
                                   _stream(stream)))


def dopt_step_apply(layout: Layout, bufs, workspace, stream=None):
    t = _marshal(layout, bufs)
    _check(_lib.dopt_step_apply(layout.handle, t, _ws(layout, workspace), _stream(stream)))


def dopt_read_stats(layout: Layout, workspace, stream=None) -> Dict:
    st = dopt_stats()
    _check(_lib.dopt_read_stats(layout.handle, _ws(layout, workspace), _stream(stream), ctypes.byref(st)))
    return st.as_dict()


def dopt_state_export(layout: Layout, bufs, master, exp_avg, exp_avg_sq, workspace, stream=None):
    """Write the rank's (master, m, v) shards in model order into three fp32
    device arrays of layout.state_numel() elements."""
    t = _marshal(layout, bufs, False)
    x = [_dev(a, f"export {name}", "f32", layout.state_numel)
         for a, name in ((master, "master"), (exp_avg, "exp_avg"), (exp_avg_sq, "exp_avg_sq"))]
    _check(_lib.dopt_state_export(layout.handle, t, *x, _ws(layout, workspace), _stream(stream)))


def dopt_state_import(layout: Layout, bufs, master, exp_avg, exp_avg_sq, workspace, stream=None):
    """Inverse of dopt_state_export; also rewrites the param window from the master."""
    t = _marshal(layout, bufs, False)
    x = [_dev(a, f"import {name}", "f32", layout.state_numel)
         for a, name in ((master, "master"), (exp_avg, "exp_avg"), (exp_avg_sq, "exp_avg_sq"))]
    _check(_lib.dopt_state_import(layout.handle, t, *x, _ws(layout, workspace), _stream(stream)))


def dopt_state_scalars_get(layout: Layout, workspace, stream=None) -> Dict:
    st = dopt_state_scalars()
    _check(_lib.dopt_state_scalars_get(layout.handle, _ws(layout, workspace), _stream(stream), ctypes.byref(st)))
    return {name: getattr(st, name) for name, _ in st._fields_}


def dopt_state_scalars_set(layout: Layout, workspace, scalars: Dict, stream=None):
    st = dopt_state_scalars(**scalars)
    _check(_lib.dopt_state_scalars_set(layout.handle, _ws(layout, workspace), _stream(stream), ctypes.byref(st)))


def dopt_last_error() -> str:
    return _lib.dopt_last_error().decode()


# ---- the step over a list of tensors (include/dopt_list.h) ----

class TensorSpec(NamedTuple):
    """One tensor of a list ('f32' | 'bf16' | 'f16' types)."""
    numel: int
    param_dtype: str
    grad_dtype: str
    hgroup: int = 0


class TensorList:
    """Owns a dopt_list handle (freed with the object)."""

    def __init__(self, handle: ctypes.c_void_p):
        self._h = handle
        self._free = _lib.dopt_list_free  # kept so that freeing works during interpreter shutdown
        o = dopt_list_info()
        _check(_lib.dopt_list_query(handle, ctypes.byref(o)))
        self.n_tensors, self.numel, self.arena_numel, self.n_blocks = o.n_tensors, o.numel, o.arena_numel, o.n_blocks
        self.workspace_bytes, self.stats_record_offset = o.workspace_bytes, o.stats_record_offset
        self.state_kind = STATE_NAMES[o.state_kind]
        self.has_master = bool(o.has_master)

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None:
            self._free(h)
            self._h = None

    @property
    def handle(self):
        return self._h

    def tensor(self, i: int) -> Dict:
        o = dopt_list_tensor_info()
        _check(_lib.dopt_list_tensor(self._h, i, ctypes.byref(o)))
        d = {name: getattr(o, name) for name, _ in o._fields_ if name != "reserved"}
        d["param_dtype"], d["grad_dtype"] = DTYPE_NAMES[d["param_dtype"]], DTYPE_NAMES[d["grad_dtype"]]
        return d

    def tensors(self) -> List[Dict]:
        """dopt_list_tensor of every tensor (cached; the list is immutable)."""
        if getattr(self, "_tensors", None) is None:
            self._tensors = [self.tensor(i) for i in range(self.n_tensors)]
        return self._tensors

    def state_arrays(self) -> Dict[str, Tuple[str, int]]:
        """The state arrays a list needs: name -> (element type, elements)."""
        e = self.state_kind != "f32"
        out = {"master": ("f32", self.arena_numel)} if self.has_master else {}
        out.update(exp_avg=("e4m3" if e else "f32", self.arena_numel),
                   exp_avg_sq=("e4m3" if e else "f32", self.arena_numel))
        if e:
            out.update(exp_avg_scale=("f32", self.n_blocks), exp_avg_sq_scale=("f32", self.n_blocks))
        return out


def _state_kind(state: str) -> int:
    if state not in STATE_KINDS:
        raise DoptError(DOPT_ERR_INVALID, f"state {state!r}: one of {sorted(STATE_KINDS)}")
    return STATE_KINDS[state]


def dopt_list_build(specs: Sequence, state: str = "f32") -> TensorList:
    """specs: objects with numel, param_dtype, grad_dtype ('f32'|'bf16'|'f16')
    and optional hgroup, in the order of the list; state: 'f32', or 8-bit
    moments, 'e4m3_sr' for whole runs (rounded by chance with the mean kept)
    and 'e4m3' (rounded to nearest: over a run sqrt(v) does not follow the
    grads)."""
    n = len(specs)
    arr = (dopt_tensor_desc * n)()
    for i, p in enumerate(specs):
        arr[i].numel = p.numel
        arr[i].param_dtype = DTYPES[p.param_dtype] if isinstance(p.param_dtype, str) else p.param_dtype
        arr[i].grad_dtype = DTYPES[p.grad_dtype] if isinstance(p.grad_dtype, str) else p.grad_dtype
        arr[i].hgroup = int(getattr(p, "hgroup", 0))
    h = ctypes.c_void_p()
    _check(_lib.dopt_list_build(arr, n, _state_kind(state), ctypes.byref(h)))
    return TensorList(h)


def dopt_list_from_layout(layout: Layout, state: str = "f32") -> TensorList:
    """The list of a layout's param shards, in model order (see shard_views)."""
    h = ctypes.c_void_p()
    _check(_lib.dopt_list_from_layout(layout.handle, _state_kind(state), ctypes.byref(h)))
    return TensorList(h)


def shard_views(layout: Layout, lst: TensorList, bufs: Sequence[Dict]):
    """(params, grads) of a dopt_list_from_layout list: views of the shards in
    the flat buffers' param and grad arenas."""
    params, grads = [], []
    for t in lst.tensors():
        if t["param"] < 0:
            raise DoptError(DOPT_ERR_INVALID, "the list was not built from a layout")
        info = layout.param(t["param"])
        a, b = info["arena_offset"], bufs[info["buffer"]]
        params.append(b["param"][a:a + t["numel"]])
        grads.append(b["grad"][a:a + t["numel"]])
    return params, grads


class ListTensors:
    """A list's params, grads and state, checked and marshalled (make it once
    with list_tensors() and pass it to every call; make it anew when a tensor
    is replaced).  Holds the list and the tensors, so that they live as long."""

    def __init__(self, lst: TensorList, ptrs, state, has_grads: bool, device: Optional[int], held):
        self.lst, self.ptrs, self.state, self.has_grads, self.device = lst, ptrs, state, has_grads, device
        self._held = held


def _spans(named):
    """(first byte, past the last, name) of each of the (name, tensor) that holds any, ascending."""
    return sorted(((x.data_ptr(), x.data_ptr() + x.numel() * x.element_size(), name) for name, x in named
                   if x is not None and not isinstance(x, int) and x.numel() > 0), key=lambda span: span[:2])


def list_tensors(lst: TensorList, params: Sequence, grads: Optional[Sequence], state: Dict) -> ListTensors:
    """params, grads: per tensor of the list a contiguous device tensor of its
    type and size, at any element-aligned address, or a raw device address;
    grads None for the calls that read none (init, export, import).  state: the
    arrays of lst.state_arrays().  Refused: wrong types or sizes, host
    tensors, tensors of several devices, and params that overlap each other, a
    grad or a state array."""
    infos = lst.tensors()
    if len(params) != len(infos):
        raise DoptError(DOPT_ERR_INVALID, f"{len(params)} params, the list has {len(infos)} tensors")
    if grads is not None and len(grads) != len(infos):
        raise DoptError(DOPT_ERR_INVALID, f"{len(grads)} grads, the list has {len(infos)} tensors")
    ptrs = (dopt_list_ptrs * len(infos))()
    for key, seq in (("param", params), ("grad", grads)):
        if seq is None:
            continue
        for i, (x, t) in enumerate(zip(seq, infos)):
            n = t["numel"]
            if n == 0 and x is None:
                continue
            if x is not None and not isinstance(x, int) and x.numel() != n:
                raise DoptError(DOPT_ERR_INVALID, f"tensor {i} {key}: {x.numel()} elements, the list has {n}")
            setattr(ptrs[i], key, _dev(x, ("tensor", i, key), t[key + "_dtype"]))
    st = dopt_list_state()
    need = lst.state_arrays()
    for name in need:
        setattr(st, name, _dev(state.get(name), f"state {name}", need[name][0], need[name][1]))
    written = _spans([(f"state {n}", state[n]) for n in need] + [(("tensor", i, "param"), x) for i, x in enumerate(params)])
    end, last = 0, ""
    for lo, hi, name in written:
        if lo < end:
            raise DoptError(DOPT_ERR_INVALID, f"{_what(name)} overlaps {_what(last)}")
        end, last = hi, name
    at = 0
    for lo, hi, name in _spans((("tensor", i, "grad"), x) for i, x in enumerate(grads or [])):
        # grads may overlap one another: they are only read
        while at < len(written) and written[at][1] <= lo:
            at += 1
        if at < len(written) and written[at][0] < hi:
            raise DoptError(DOPT_ERR_INVALID, f"{_what(name)} overlaps {_what(written[at][2])}")
    held = list(params) + list(grads or []) + [state[n] for n in need]
    devices = {x.device.index for x in held if x is not None and not isinstance(x, int) and x.numel() > 0}
    if len(devices) > 1:
        raise DoptError(DOPT_ERR_INVALID, f"tensors on several devices: {sorted(devices)}")
    return ListTensors(lst, ptrs, st, grads is not None, devices.pop() if devices else None, held)


_torch = None  # the module whose tensors and streams the calls are given


def _list_ws(lst: TensorList, workspace, stream, device: Optional[int] = None):
    """(workspace address, stream) of a call, which the library launches on the
    current device: the workspace, the stream and the tensors' `device` have
    to be there."""
    global _torch
    ws = _dev(workspace, "workspace", None, 0, lst.workspace_bytes)
    if _torch is None:
        if device is None and isinstance(workspace, int) and (stream is None or isinstance(stream, int)):
            return ws, stream
        import torch
        _torch = torch
    current = _torch.cuda.current_device() if device is not None or workspace is not ws else None
    if device is not None and device != current:
        _elsewhere("tensors", device)
    if workspace is not ws and workspace.get_device() != current:
        _elsewhere("workspace", workspace.get_device())
    if stream is None or isinstance(stream, int):
        return ws, stream
    index = stream.device.index
    if index != (_torch.cuda.current_device() if current is None else current):
        _elsewhere("stream", index)
    return ws, stream.cuda_stream


def _current_device() -> int:
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch.cuda.current_device()


def _elsewhere(what: str, index: int):
    raise DoptError(DOPT_ERR_INVALID, f"{what} on device {index}, the current device is {_current_device()}")


def _list_args(lst: TensorList, t: ListTensors, workspace, stream, need_grads: bool = True):
    """(tensors, workspace address, stream) of a call, after checking that they belong together."""
    if t.lst is not lst:
        raise DoptError(DOPT_ERR_INVALID, "tensors were marshalled for another list")
    if need_grads and not t.has_grads:
        raise DoptError(DOPT_ERR_INVALID, "tensors were marshalled without grads")
    return (t.ptrs, *_list_ws(lst, workspace, stream, t.device))


def dopt_list_init(lst: TensorList, t: ListTensors, scaler: dopt_scaler_cfg, workspace, stream=None):
    """Masters from the params, zero moments, step 0; synchronizes the stream."""
    p, ws, s = _list_args(lst, t, workspace, stream, False)
    _check(_lib.dopt_list_init(lst.handle, p, ctypes.byref(t.state), ctypes.byref(scaler), ws, s))


def dopt_list_step(lst: TensorList, t: ListTensors, hparams, max_grad_norm: float, workspace, stream=None,
                   want_stats: bool = True):
    p, ws, s = _list_args(lst, t, workspace, stream)
    hp = hparams if isinstance(hparams, ctypes.Array) else _hparams(hparams)
    st = dopt_stats() if want_stats else None
    _check(_lib.dopt_list_step(lst.handle, p, ctypes.byref(t.state), hp, len(hp), max_grad_norm, ws, s,
                               ctypes.byref(st) if st is not None else None))
    return st.as_dict() if st is not None else None


def dopt_list_prepare(lst: TensorList, t: ListTensors, hparams, max_grad_norm: float, workspace, stream=None):
    p, ws, s = _list_args(lst, t, workspace, stream)
    hp = hparams if isinstance(hparams, ctypes.Array) else _hparams(hparams)
    _check(_lib.dopt_list_prepare(lst.handle, p, hp, len(hp), max_grad_norm, ws, s))


def dopt_list_stats(lst: TensorList, t: ListTensors, workspace, stream=None):
    p, ws, s = _list_args(lst, t, workspace, stream)
    _check(_lib.dopt_list_stats(lst.handle, p, ws, s))


def dopt_list_finalize(lst: TensorList, hparams, max_grad_norm: float, workspace, stream=None):
    hp = hparams if isinstance(hparams, ctypes.Array) else _hparams(hparams)
    _check(_lib.dopt_list_finalize(lst.handle, hp, len(hp), max_grad_norm, *_list_ws(lst, workspace, stream)))


def dopt_list_apply(lst: TensorList, t: ListTensors, workspace, stream=None):
    p, ws, s = _list_args(lst, t, workspace, stream)
    _check(_lib.dopt_list_apply(lst.handle, p, ctypes.byref(t.state), ws, s))


def _list_copy(fn, word: str, lst: TensorList, t: ListTensors, master, exp_avg, exp_avg_sq, workspace, stream):
    p, ws, s = _list_args(lst, t, workspace, stream, False)
    x = []
    for a, name in ((master, "master"), (exp_avg, "exp_avg"), (exp_avg_sq, "exp_avg_sq")):
        x.append(_dev(a, f"{word} {name}", "f32", lst.numel))
        if not isinstance(a, int) and a.numel() > 0 and a.get_device() != _current_device():
            _elsewhere(f"{word} {name}", a.get_device())
    _check(fn(lst.handle, p, ctypes.byref(t.state), *x, ws, s))


def dopt_list_export(lst: TensorList, t: ListTensors, master, exp_avg, exp_avg_sq, workspace, stream=None):
    """Write master, m and v of the list's tensors, back to back in list order,
    into three fp32 device arrays of lst.numel elements."""
    _list_copy(_lib.dopt_list_export, "export", lst, t, master, exp_avg, exp_avg_sq, workspace, stream)


def dopt_list_import(lst: TensorList, t: ListTensors, master, exp_avg, exp_avg_sq, workspace, stream=None):
    """Inverse of dopt_list_export; also rewrites the params from the master."""
    _list_copy(_lib.dopt_list_import, "import", lst, t, master, exp_avg, exp_avg_sq, workspace, stream)


def dopt_list_set_seed(lst: TensorList, seed: int, workspace, stream=None):
    """The seed of an 'e4m3_sr' list's rounding, 0 after init; takes 64 bits."""
    if not 0 <= seed < 1 << 64:
        raise DoptError(DOPT_ERR_INVALID, f"seed {seed}: not in [0, 2^64)")
    _check(_lib.dopt_list_set_seed(lst.handle, seed, *_list_ws(lst, workspace, stream)))


def dopt_list_scalars_get(lst: TensorList, workspace, stream=None) -> Dict:
    st = dopt_state_scalars()
    _check(_lib.dopt_list_scalars_get(lst.handle, *_list_ws(lst, workspace, stream), ctypes.byref(st)))
    return {name: getattr(st, name) for name, _ in st._fields_}


def dopt_list_scalars_set(lst: TensorList, workspace, scalars: Dict, stream=None):
    st = dopt_state_scalars(**scalars)
    _check(_lib.dopt_list_scalars_set(lst.handle, *_list_ws(lst, workspace, stream), ctypes.byref(st)))


def dopt_list_read_stats(lst: TensorList, workspace, stream=None) -> Dict:
    st = dopt_stats()
    _check(_lib.dopt_list_read_stats(lst.handle, *_list_ws(lst, workspace, stream), ctypes.byref(st)))
    return st.as_dict()


# ---- device-memory placement helpers (include/dopt_vmm.h) ----

def dopt_vmm_granularity(device: int = 0) -> int:
    out = ctypes.c_size_t()
    _check(_lib.dopt_vmm_granularity(device, ctypes.byref(out)))
    return out.value


def dopt_vmm_reserve(nbytes: int, align: int = 0) -> int:
    out = ctypes.c_uint64()
    _check(_lib.dopt_vmm_reserve(nbytes, align, ctypes.byref(out)))
    return out.value


def dopt_vmm_free(va: int, nbytes: int):
    _check(_lib.dopt_vmm_free(va, nbytes))


def dopt_vmm_create(nbytes: int, device: int = 0) -> int:
    out = ctypes.c_uint64()
    _check(_lib.dopt_vmm_create(device, nbytes, ctypes.byref(out)))
    return out.value


def dopt_vmm_map(va: int, nbytes: int, handle: int):
    _check(_lib.dopt_vmm_map(va, nbytes, handle))


def dopt_vmm_set_access(va: int, nbytes: int, device: int = 0):
    _check(_lib.dopt_vmm_set_access(va, nbytes, device))


def dopt_vmm_unmap(va: int, nbytes: int):
    _check(_lib.dopt_vmm_unmap(va, nbytes))


def dopt_vmm_release(handle: int):
    _check(_lib.dopt_vmm_release(handle))


hparams_array = _hparams
