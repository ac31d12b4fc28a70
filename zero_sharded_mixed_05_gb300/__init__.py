"""GB300 per-shard mixed-precision ZeRO optimizer step.

A thin ctypes binding of the C ABI in ``include/zero_opt.h``: the functions
here carry the same names as the C entry points and only marshal arguments
(torch tensors become device pointers, the current torch stream becomes the
``cudaStream_t``).  Every step of the computation runs in the library's CUDA
kernels (``csrc/``); there is no Python or CPU fallback, and importing this
package fails loudly when the compiled library is missing.

Build the library with ``zero_sharded_mixed_05_gb300._build.build()`` (or
``__graft_entry__.build()``).
"""
from __future__ import annotations

import ctypes
import os
import struct

from . import _build

FP16 = 0
BF16 = 1
FP32 = 2      # where a call says it takes it

ZERO_OK, ZERO_EINVAL, ZERO_ERANGE, ZERO_ENOMEM, ZERO_ECUDA, ZERO_ENOTSUP = range(6)

_i32, _i64, _f32, _f64, _vp = (ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                              ctypes.c_double, ctypes.c_void_p)


class zero_opt_config(ctypes.Structure):
    _fields_ = [("numel", _i64), ("world", _i32), ("grad_dtype", _i32),
                ("param_dtype", _i32), ("bias_correction", _i32),
                ("lr", _f64), ("beta1", _f64), ("beta2", _f64), ("eps", _f64),
                ("weight_decay", _f64), ("max_grad_norm", _f64),
                ("dynamic_scale", _i32), ("hysteresis", _i32),
                ("init_scale", _f64), ("min_scale", _f64), ("scale_factor", _f64),
                ("scale_window", _i64), ("warmup_min_lr", _f64), ("warmup_max_lr", _f64),
                ("warmup_num_steps", _i64), ("master16", _i32), ("table_kib", _i32)]


class zero_opt_buffers(ctypes.Structure):
    _fields_ = [("master", _vp), ("m", _vp), ("v", _vp), ("param16", _vp),
                ("grads", ctypes.POINTER(_vp)), ("n_ranks", _i32), ("n_micro", _i32),
                ("grads_shard_local", _i32), ("param16_shard_local", _i32),
                ("divisor", _f64), ("stash", _vp)]


class zero_opt_tensor(ctypes.Structure):
    _fields_ = [("numel", _i64), ("master", _vp), ("m", _vp), ("v", _vp),
                ("param16", _vp), ("grads", ctypes.POINTER(_vp))]


class zero_opt_tensor_list(ctypes.Structure):
    _fields_ = [("tensors", ctypes.POINTER(zero_opt_tensor)), ("n_tensors", _i32),
                ("n_ranks", _i32), ("n_micro", _i32), ("divisor", _f64),
                ("stash", _vp)]


class zero_opt_stats(ctypes.Structure):
    _fields_ = [("sumsq", _f64), ("nonfinite", _i32), ("reserved", _i32)]


class zero_opt_step_info(ctypes.Structure):
    _fields_ = [("sumsq", _f64), ("norm", _f64), ("coef", _f32), ("scale_used", _f32),
                ("skipped", _i32), ("nonfinite", _i32), ("t", _i64), ("fault", _i32),
                ("reserved", _i32)]


class zero_opt_scaler_state(ctypes.Structure):
    _fields_ = [("scale", _f32), ("last_skipped", _i32), ("clean_steps", _i64),
                ("t", _i64), ("skipped_total", _i64), ("overflows", _i32),
                ("reserved", _i32)]

    def as_tuple(self):
        """(scale, clean_steps, t, skipped_total, last_skipped)."""
        return (float(self.scale), int(self.clean_steps), int(self.t),
                int(self.skipped_total), int(self.last_skipped))


class zero_opt_counters(ctypes.Structure):
    _fields_ = [("launches", _i64), ("table_uploads", _i64), ("table_waits", _i64),
                ("device_allocs", _i64), ("device_frees", _i64), ("tables_cached", _i64),
                ("tables_pinned", _i64), ("table_bytes", _i64)]

    def as_dict(self):
        return {name: int(getattr(self, name)) for name, _ in self._fields_}


class zero_opt_ckpt_info(ctypes.Structure):
    _fields_ = [("numel", _i64), ("world", _i32), ("rank", _i32), ("begin", _i64),
                ("real_len", _i64), ("scaler", zero_opt_scaler_state)]


MUON_SCALE_ONE, MUON_SCALE_RMS, MUON_SCALE_ASPECT = range(3)
MUON_MAX_STEPS = 16


class zero_muon_config(ctypes.Structure):
    _fields_ = [("grad_dtype", _i32), ("param_dtype", _i32), ("nesterov", _i32), ("steps", _i32),
                ("scale_rule", _i32), ("reserved", _i32), ("lr", _f64), ("momentum", _f64),
                ("weight_decay", _f64), ("eps", _f64), ("coef", _f64 * 3 * MUON_MAX_STEPS)]


class zero_muon_shape(ctypes.Structure):
    _fields_ = [("rows", _i64), ("cols", _i64), ("batch", _i64)]


class zero_muon_operand(ctypes.Structure):
    _fields_ = [("src", _vp), ("dst", _vp), ("in_row", _i64), ("in_batch", _i64),
                ("out_row", _i64), ("out_batch", _i64)]


class zero_muon_matrix(ctypes.Structure):
    _fields_ = [("grad", _vp), ("momentum", _vp), ("master", _vp), ("param16", _vp)]


class zero_muon_info(ctypes.Structure):
    _fields_ = [("skipped", _i32), ("fault", _i32)]


class zero_qk_config(ctypes.Structure):
    _fields_ = [("q_heads", _i32), ("k_heads", _i32), ("head_dim", _i32), ("rotary_dim", _i32),
                ("dtype", _i32), ("interleaved", _i32), ("gain_per_head", _i32),
                ("reserved", _i32), ("eps", _f64)]


class zero_qk_tensor(ctypes.Structure):
    _fields_ = [("data", _vp), ("token_stride", _i64), ("head_stride", _i64)]


class zero_qk_buffers(ctypes.Structure):
    _fields_ = [("tokens", _i64), ("n_pos", _i64), ("q", zero_qk_tensor), ("k", zero_qk_tensor),
                ("q_out", zero_qk_tensor), ("k_out", zero_qk_tensor), ("dq", zero_qk_tensor),
                ("dk", zero_qk_tensor), ("q_gain", _vp), ("k_gain", _vp), ("dq_gain", _vp),
                ("dk_gain", _vp), ("cos", _vp), ("sin", _vp), ("positions", _vp),
                ("positions64", _i32), ("reserved", _i32)]


class ZeroOptError(RuntimeError):
    def __init__(self, status: int, where: str, message: str):
        super().__init__(f"{where}: status {status}: {message}")
        self.status = status


# ---------------------------------------------------------------- loading

LIB_PATH = _build.LIB

# (name, restype, argtypes) of every entry point in include/zero_opt.h
_P = ctypes.POINTER
SIGNATURES = [
    ("zero_opt_config_default", _i32, [_P(zero_opt_config)]),
    ("zero_opt_create", _i32, [_P(zero_opt_config), _P(_vp)]),
    ("zero_opt_destroy", _i32, [_vp]),
    ("zero_opt_shard_bounds", _i32, [_vp, _i32, _P(_i64), _P(_i64), _P(_i64), _P(_i64)]),
    ("zero_opt_memory_bytes", _i32, [_i64, _i32, _i32, _P(_i64)]),
    ("zero_opt_grad_stats", _i32, [_vp, _i32, _P(zero_opt_buffers), _vp, _P(zero_opt_stats)]),
    ("zero_opt_fold_stats", _i32, [_P(zero_opt_stats), _i32, _P(zero_opt_stats)]),
    ("zero_opt_step", _i32, [_vp, _i32, _P(zero_opt_buffers), _vp, _P(zero_opt_stats)]),
    ("zero_opt_grad_stats_async", _i32, [_vp, _i32, _P(zero_opt_buffers), _vp, _vp]),
    ("zero_opt_step_folded", _i32, [_vp, _i32, _P(zero_opt_buffers), _vp, _vp, _i32]),
    ("zero_opt_grad_stats_tensors", _i32,
     [_vp, _i32, _P(zero_opt_tensor_list), _vp, _P(zero_opt_stats)]),
    ("zero_opt_step_tensors", _i32,
     [_vp, _i32, _P(zero_opt_tensor_list), _vp, _P(zero_opt_stats)]),
    ("zero_opt_loss_scale", _i32, [_vp, _i32, _vp, _P(zero_opt_scaler_state)]),
    ("zero_opt_set_loss_scale", _i32, [_vp, _i32, _vp, _P(zero_opt_scaler_state)]),
    ("zero_opt_set_lr", _i32, [_vp, _f64]),
    ("zero_opt_last_step", _i32, [_vp, _vp, _P(zero_opt_step_info)]),
    ("zero_opt_set_events", _i32, [_vp, _vp, _vp, _vp]),
    ("zero_opt_inject_wait_fault", _i32, [_vp]),
    ("zero_opt_launch_count", _i32, [_vp, _P(_i64)]),
    ("zero_opt_get_counters", _i32, [_vp, _P(zero_opt_counters)]),
    ("zero_opt_ckpt_write", _i32, [ctypes.c_char_p, _P(zero_opt_ckpt_info), _vp, _vp, _vp]),
    ("zero_opt_ckpt_read", _i32, [ctypes.c_char_p, _P(zero_opt_ckpt_info), _vp, _vp, _vp]),
    ("zero_opt_save_shard", _i32, [_vp, _i32, _vp, _vp, _vp, _vp, ctypes.c_char_p]),
    ("zero_opt_save_shard16", _i32, [_vp, _i32, _vp, _i32, _vp, _vp, _vp, ctypes.c_char_p]),
    ("zero_opt_load_shard", _i32, [_vp, _i32, _vp, _vp, _vp, _vp, _i32, _vp, ctypes.c_char_p]),
    ("zero_opt_consolidate_fp32", _i32, [_P(ctypes.c_char_p), _i32, _i64, _vp]),
    ("zero_opt_grad_stats_noalloc", _i32, [_P(_vp), _i32, _i32, _i64, _vp, _vp]),
    ("zero_host_create", _i32, [_P(zero_opt_config), _i32, _P(_vp)]),
    ("zero_host_destroy", _i32, [_vp]),
    ("zero_host_threads", _i32, [_vp, _P(_i32)]),
    ("zero_host_grad_stats", _i32, [_vp, _i32, _P(zero_opt_buffers), _P(zero_opt_stats)]),
    ("zero_host_step", _i32, [_vp, _i32, _P(zero_opt_buffers), _P(zero_opt_stats)]),
    ("zero_host_grad_stats_tensors", _i32,
     [_vp, _i32, _P(zero_opt_tensor_list), _P(zero_opt_stats)]),
    ("zero_host_step_tensors", _i32, [_vp, _i32, _P(zero_opt_tensor_list), _P(zero_opt_stats)]),
    ("zero_host_loss_scale", _i32, [_vp, _i32, _P(zero_opt_scaler_state)]),
    ("zero_host_set_loss_scale", _i32, [_vp, _i32, _P(zero_opt_scaler_state)]),
    ("zero_host_last_step", _i32, [_vp, _P(zero_opt_step_info)]),
    ("zero_opt_decision", _i32, [_vp, _P(_vp)]),
    ("zero_muon_config_default", _i32, [_P(zero_muon_config)]),
    ("zero_muon_create", _i32, [_P(zero_muon_config), _P(zero_muon_shape), _i32, _P(_vp)]),
    ("zero_muon_destroy", _i32, [_vp]),
    ("zero_muon_workspace_bytes", _i32, [_vp, _P(_i64)]),
    ("zero_muon_set_lr", _i32, [_vp, _f64]),
    ("zero_muon_orthogonalize", _i32, [_vp, _P(zero_muon_operand), _i32, _i32, _vp]),
    ("zero_muon_step", _i32, [_vp, _P(zero_muon_matrix), _f64, _vp, _vp]),
    ("zero_muon_last_step", _i32, [_vp, _vp, _P(zero_muon_info)]),
    ("zero_muon_fault_count", _i32, [_vp, _vp, _P(_i64)]),
    ("zero_muon_inject_wait_fault", _i32, [_vp]),
    ("zero_muon_launch_count", _i32, [_vp, _P(_i64)]),
    ("zero_qk_create", _i32, [_P(zero_qk_config), _P(_vp)]),
    ("zero_qk_destroy", _i32, [_vp]),
    ("zero_qk_norm_rope", _i32, [_vp, _vp, _vp]),
    ("zero_qk_norm_rope_backward", _i32, [_vp, _vp, _vp]),
    ("zero_qk_launch_count", _i32, [_vp, _P(_i64)]),
    ("zero_opt_status_string", ctypes.c_char_p, [_i32]),
    ("zero_opt_last_error", ctypes.c_char_p, []),
]

_lib = None


def lib():
    """The loaded CUDA library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is missing: the CUDA library must be built first "
                "(zero_sharded_mixed_05_gb300._build.build()); there is no fallback")
        L = ctypes.CDLL(LIB_PATH)
        for name, res, args in SIGNATURES:
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(status: int, where: str) -> None:
    if status != ZERO_OK:
        msg = lib().zero_opt_last_error().decode(errors="replace")
        raise ZeroOptError(status, where, msg)


def _ptr(x):
    """Address of a torch tensor or numpy array (or an int address)."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    return x.ctypes.data


def current_stream(device=None) -> int:
    import torch
    return torch.cuda.current_stream(device).cuda_stream


def _stream(s):
    if type(s) is int:
        return s
    if s is None:
        import torch
        if torch.cuda.is_available():
            return current_stream()
        return None
    if isinstance(s, int):
        return s
    return s.cuda_stream


def dtype_code(torch_dtype) -> int:
    import torch
    if torch_dtype == torch.float16:
        return FP16
    if torch_dtype == torch.bfloat16:
        return BF16
    raise ValueError(f"unsupported 16-bit dtype {torch_dtype}")


# ---------------------------------------------------------------- descriptors

def make_config(numel=0, world=1, grad_dtype=FP16, param_dtype=None, lr=2e-5,
                betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, max_grad_norm=0.0,
                bias_correction=True, dynamic_scale=True, init_scale=65536.0,
                min_scale=1.0, scale_factor=2.0, scale_window=1000,
                hysteresis=1, warmup=(0.0, 0.0, 0), master16=False,
                table_kib=0) -> zero_opt_config:
    """`warmup` = (warmup_min_lr, warmup_max_lr, warmup_num_steps); 0 steps
    keeps lr constant.  `master16`: the 16-bit parameters are the master
    weights (no fp32 master array).  `table_kib`: KiB of the handle's
    run-table arena (0: 1024)."""
    cfg = zero_opt_config()
    _check(lib().zero_opt_config_default(ctypes.byref(cfg)), "zero_opt_config_default")
    cfg.numel = numel
    cfg.world = world
    cfg.grad_dtype = grad_dtype
    cfg.param_dtype = grad_dtype if param_dtype is None else param_dtype
    cfg.lr = lr
    cfg.beta1, cfg.beta2 = betas
    cfg.eps = eps
    cfg.weight_decay = weight_decay
    cfg.max_grad_norm = max_grad_norm
    cfg.bias_correction = int(bias_correction)
    cfg.dynamic_scale = int(dynamic_scale)
    cfg.init_scale = init_scale
    cfg.min_scale = min_scale
    cfg.scale_factor = scale_factor
    cfg.scale_window = scale_window
    cfg.hysteresis = hysteresis
    cfg.warmup_min_lr, cfg.warmup_max_lr, cfg.warmup_num_steps = warmup
    cfg.master16 = int(master16)
    cfg.table_kib = int(table_kib)
    return cfg


def _ptr_array(items):
    arr = (_vp * max(len(items), 1))()
    for i, g in enumerate(items):
        arr[i] = _ptr(g)
    return arr


def make_buffers(master, m, v, param16, grads, n_ranks=None, n_micro=1,
                 grads_shard_local=False, param16_shard_local=False, divisor=0.0,
                 stash=None) -> zero_opt_buffers:
    """Flat-shard buffers; `grads` lists the R*K gradient buffers rank-major."""
    grads = list(grads)
    if n_ranks is None:
        n_ranks = len(grads) // n_micro
    arr = _ptr_array(grads)
    b = zero_opt_buffers(_ptr(master), _ptr(m), _ptr(v), _ptr(param16),
                         ctypes.cast(arr, _P(_vp)), n_ranks, n_micro,
                         int(grads_shard_local), int(param16_shard_local),
                         float(divisor), _ptr(stash))
    b._keep = (arr, grads, master, m, v, param16, stash)
    return b


def make_tensor_list(tensors, n_ranks=1, n_micro=1, divisor=0.0,
                     stash=None) -> zero_opt_tensor_list:
    """Per-tensor list; each item is a dict with numel (optional), master, m, v,
    param16 and grads (R*K tensors, rank-major)."""
    items = (zero_opt_tensor * max(len(tensors), 1))()
    keep = []
    for i, t in enumerate(tensors):
        garr = _ptr_array(t["grads"])
        keep.append((garr, t))
        numel = t["numel"] if "numel" in t else t["master"].numel()
        items[i] = zero_opt_tensor(numel, _ptr(t["master"]), _ptr(t["m"]), _ptr(t["v"]),
                                   _ptr(t["param16"]), ctypes.cast(garr, _P(_vp)))
    lst = zero_opt_tensor_list(ctypes.cast(items, _P(zero_opt_tensor)), len(tensors),
                               n_ranks, n_micro, float(divisor), _ptr(stash))
    lst._keep = (items, keep, stash)
    return lst


# ---------------------------------------------------------------- entry points

def zero_opt_config_default() -> zero_opt_config:
    cfg = zero_opt_config()
    _check(lib().zero_opt_config_default(ctypes.byref(cfg)), "zero_opt_config_default")
    return cfg


def zero_opt_create(cfg: zero_opt_config) -> int:
    h = _vp()
    _check(lib().zero_opt_create(ctypes.byref(cfg), ctypes.byref(h)), "zero_opt_create")
    return h.value


def zero_opt_destroy(h) -> None:
    _check(lib().zero_opt_destroy(h), "zero_opt_destroy")


def zero_opt_shard_bounds(h, rank: int):
    """(begin, real_end, shard_len, padded_numel)."""
    out = [_i64() for _ in range(4)]
    _check(lib().zero_opt_shard_bounds(h, rank, *[ctypes.byref(o) for o in out]),
           "zero_opt_shard_bounds")
    return tuple(o.value for o in out)


def zero_opt_memory_bytes(numel: int, world: int, stage: int) -> int:
    out = _i64()
    _check(lib().zero_opt_memory_bytes(numel, world, stage, ctypes.byref(out)),
           "zero_opt_memory_bytes")
    return out.value


def zero_opt_grad_stats(h, rank: int, bufs: zero_opt_buffers, stream=None) -> zero_opt_stats:
    out = zero_opt_stats()
    _check(lib().zero_opt_grad_stats(h, rank, ctypes.byref(bufs), _stream(stream),
                                     ctypes.byref(out)), "zero_opt_grad_stats")
    return out


def zero_opt_step(h, rank: int, bufs: zero_opt_buffers, stream=None,
                  global_stats: zero_opt_stats | None = None) -> None:
    gs = ctypes.byref(global_stats) if global_stats is not None else None
    _check(lib().zero_opt_step(h, rank, ctypes.byref(bufs), _stream(stream), gs),
           "zero_opt_step")


def zero_opt_grad_stats_async(h, rank: int, bufs: zero_opt_buffers, out_dev,
                              stream=None) -> None:
    """Shard statistics into `out_dev`, a device buffer of 16 bytes (one
    zero_opt_stats), without synchronizing."""
    _check(lib().zero_opt_grad_stats_async(h, rank, ctypes.byref(bufs), _stream(stream),
                                           _ptr(out_dev)), "zero_opt_grad_stats_async")


def zero_opt_step_folded(h, rank: int, bufs: zero_opt_buffers, per_rank_dev, n: int,
                         stream=None) -> None:
    """Step with the global statistics folded on the device from `n` per-rank
    zero_opt_stats records at `per_rank_dev` (device, rank order)."""
    _check(lib().zero_opt_step_folded(h, rank, ctypes.byref(bufs), _stream(stream),
                                      _ptr(per_rank_dev), n), "zero_opt_step_folded")


def zero_opt_grad_stats_tensors(h, rank: int, lst: zero_opt_tensor_list,
                                stream=None) -> zero_opt_stats:
    out = zero_opt_stats()
    _check(lib().zero_opt_grad_stats_tensors(h, rank, ctypes.byref(lst), _stream(stream),
                                             ctypes.byref(out)),
           "zero_opt_grad_stats_tensors")
    return out


def zero_opt_step_tensors(h, rank: int, lst: zero_opt_tensor_list, stream=None,
                          global_stats: zero_opt_stats | None = None) -> None:
    gs = ctypes.byref(global_stats) if global_stats is not None else None
    _check(lib().zero_opt_step_tensors(h, rank, ctypes.byref(lst), _stream(stream), gs),
           "zero_opt_step_tensors")


def zero_opt_loss_scale(h, rank: int, stream=None) -> zero_opt_scaler_state:
    out = zero_opt_scaler_state()
    _check(lib().zero_opt_loss_scale(h, rank, _stream(stream), ctypes.byref(out)),
           "zero_opt_loss_scale")
    return out


def zero_opt_set_loss_scale(h, rank: int, state: zero_opt_scaler_state, stream=None) -> None:
    _check(lib().zero_opt_set_loss_scale(h, rank, _stream(stream), ctypes.byref(state)),
           "zero_opt_set_loss_scale")


def zero_opt_set_lr(h, lr: float) -> None:
    _check(lib().zero_opt_set_lr(h, lr), "zero_opt_set_lr")


def zero_opt_last_step(h, stream=None) -> zero_opt_step_info:
    out = zero_opt_step_info()
    _check(lib().zero_opt_last_step(h, _stream(stream), ctypes.byref(out)),
           "zero_opt_last_step")
    return out


def zero_opt_set_events(h, ev_start=None, ev_mid=None, ev_end=None) -> None:
    """Record torch.cuda.Event objects (or raw cudaEvent_t ints) around the
    passes of subsequent steps; no arguments turns the hook off."""
    def raw(e):
        if e is None or isinstance(e, int):
            return e
        return e.cuda_event
    _check(lib().zero_opt_set_events(h, raw(ev_start), raw(ev_mid), raw(ev_end)),
           "zero_opt_set_events")


def zero_opt_inject_wait_fault(h) -> None:
    """Arm the failure-detection test hook for the next statistics pass."""
    _check(lib().zero_opt_inject_wait_fault(h), "zero_opt_inject_wait_fault")


def zero_opt_launch_count(h) -> int:
    out = _i64()
    _check(lib().zero_opt_launch_count(h, ctypes.byref(out)), "zero_opt_launch_count")
    return out.value


def zero_opt_get_counters(h) -> zero_opt_counters:
    """Launches, run-table uploads and waits, and allocations after creation."""
    out = zero_opt_counters()
    _check(lib().zero_opt_get_counters(h, ctypes.byref(out)), "zero_opt_get_counters")
    return out


def zero_opt_status_string(status: int) -> str:
    return lib().zero_opt_status_string(status).decode()


def zero_opt_fold_stats(per_rank) -> zero_opt_stats:
    """The scalar all-reduce of per-rank statistics, folded in rank order."""
    per_rank = list(per_rank)
    arr = (zero_opt_stats * max(len(per_rank), 1))(*per_rank)
    out = zero_opt_stats()
    _check(lib().zero_opt_fold_stats(arr, len(per_rank), ctypes.byref(out)),
           "zero_opt_fold_stats")
    return out


def allgather_fold(own: zero_opt_stats, group=None) -> zero_opt_stats:
    """The scalar all-reduce of a multi-process run: every rank contributes its
    shard's statistics, all ranks receive all of them (torch.distributed
    all_gather on a tiny tensor) and fold them in rank order with
    zero_opt_fold_stats, so every rank gets bit-identical totals."""
    import torch
    import torch.distributed as dist
    ws = dist.get_world_size(group)
    mine = torch.tensor([own.sumsq, float(own.nonfinite)], dtype=torch.float64)
    if dist.get_backend(group) == "nccl":
        mine = mine.cuda()
    parts = [torch.empty_like(mine) for _ in range(ws)]
    dist.all_gather(parts, mine, group=group)
    per = [zero_opt_stats(float(p[0]), int(p[1]), 0) for p in (q.cpu() for q in parts)]
    return zero_opt_fold_stats(per)


# ---------------------------------------------------------------- checkpoints

def _np_ptr(a):
    if a is None:
        return None
    assert a.flags["C_CONTIGUOUS"] and a.dtype.itemsize == 4
    return a.ctypes.data


def zero_opt_ckpt_write(path: str, info: zero_opt_ckpt_info, master, m, v) -> None:
    """Write one shard file from host float32 numpy arrays."""
    _check(lib().zero_opt_ckpt_write(os.fsencode(path), ctypes.byref(info), _np_ptr(master),
                                     _np_ptr(m), _np_ptr(v)), "zero_opt_ckpt_write")


def zero_opt_ckpt_read(path: str, with_payload: bool = True):
    """(info, master, m, v) of a shard file, arrays as host numpy float32."""
    import numpy as np
    info = zero_opt_ckpt_info()
    _check(lib().zero_opt_ckpt_read(os.fsencode(path), ctypes.byref(info), None, None, None),
           "zero_opt_ckpt_read")
    if not with_payload:
        return info, None, None, None
    arrs = [np.empty(info.real_len, np.float32) for _ in range(3)]
    _check(lib().zero_opt_ckpt_read(os.fsencode(path), ctypes.byref(info),
                                    *[_np_ptr(a) for a in arrs]), "zero_opt_ckpt_read")
    return (info, *arrs)


def zero_opt_save_shard(h, rank: int, master, m, v, path: str, stream=None) -> None:
    _check(lib().zero_opt_save_shard(h, rank, _ptr(master), _ptr(m), _ptr(v), _stream(stream),
                                     os.fsencode(path)), "zero_opt_save_shard")


def zero_opt_save_shard16(h, rank: int, param16, m, v, path: str,
                          param16_shard_local: bool = False, stream=None) -> None:
    """Shard file of a master16 handle: its 16-bit masters (widened exactly), m, v
    and loss-scaler replica."""
    _check(lib().zero_opt_save_shard16(h, rank, _ptr(param16), int(param16_shard_local),
                                       _ptr(m), _ptr(v), _stream(stream), os.fsencode(path)),
           "zero_opt_save_shard16")


def zero_opt_load_shard(h, rank: int, master, m, v, path: str, param16=None,
                        param16_shard_local: bool = False, stream=None) -> None:
    _check(lib().zero_opt_load_shard(h, rank, _ptr(master), _ptr(m), _ptr(v), _ptr(param16),
                                     int(param16_shard_local), _stream(stream),
                                     os.fsencode(path)), "zero_opt_load_shard")


def zero_opt_consolidate_fp32(paths, numel: int):
    """Full fp32 master weights (numpy) merged from one checkpoint's shard files."""
    import numpy as np
    arr = (ctypes.c_char_p * len(paths))(*[os.fsencode(p) for p in paths])
    out = np.empty(numel, np.float32)
    _check(lib().zero_opt_consolidate_fp32(arr, len(paths), numel, _np_ptr(out)),
           "zero_opt_consolidate_fp32")
    return out


def zero_opt_grad_stats_noalloc(grads, grad_dtype: int, n: int, out, stream=None) -> None:
    """Statistics of the sum of `grads` (device tensors) written into `out`, a
    device buffer of at least 16 bytes holding one zero_opt_stats; allocates
    nothing on the device.

    The C entry point receives bare pointers and cannot check them, so this
    binding does: every gradient must be a contiguous CUDA tensor of the
    current device with the dtype `grad_dtype` names and at least `n`
    elements, and `out` a contiguous CUDA tensor of the current device of at
    least 16 bytes.  Anything else raises ValueError before a launch."""
    import torch
    want = {FP16: torch.float16, BF16: torch.bfloat16}.get(grad_dtype)
    if want is None:
        raise ValueError(f"grad_dtype must be FP16 or BF16, not {grad_dtype}")
    grads = list(grads)
    dev = torch.cuda.current_device()

    def on_device(t):
        return isinstance(t, torch.Tensor) and t.is_cuda and t.device.index == dev \
            and t.is_contiguous()
    for i, g in enumerate(grads):
        if not on_device(g):
            raise ValueError(f"grads[{i}] must be a contiguous CUDA tensor on device {dev}")
        if g.dtype != want:
            raise ValueError(f"grads[{i}] is {g.dtype}, grad_dtype names {want}")
        if g.numel() < n:
            raise ValueError(f"grads[{i}] holds {g.numel()} elements, fewer than n = {n}")
    if not on_device(out) or out.numel() * out.element_size() < 16:
        raise ValueError(f"out must be a contiguous CUDA tensor on device {dev} of at least "
                         "16 bytes (one zero_opt_stats)")
    arr = _ptr_array(grads)
    _check(lib().zero_opt_grad_stats_noalloc(ctypes.cast(arr, _P(_vp)), len(grads), grad_dtype,
                                             n, _stream(stream), _ptr(out)),
           "zero_opt_grad_stats_noalloc")


# ---------------------------------------------------------------- offloaded (host) step
# Same calls on host-resident buffers (numpy arrays or CPU tensors); no GPU.

def zero_host_create(cfg: zero_opt_config, n_threads: int = 0) -> int:
    h = _vp()
    _check(lib().zero_host_create(ctypes.byref(cfg), n_threads, ctypes.byref(h)),
           "zero_host_create")
    return h.value


def zero_host_destroy(h) -> None:
    _check(lib().zero_host_destroy(h), "zero_host_destroy")


def zero_host_threads(h) -> int:
    n = _i32()
    _check(lib().zero_host_threads(h, ctypes.byref(n)), "zero_host_threads")
    return n.value


def zero_host_grad_stats(h, rank: int, bufs: zero_opt_buffers) -> zero_opt_stats:
    out = zero_opt_stats()
    _check(lib().zero_host_grad_stats(h, rank, ctypes.byref(bufs), ctypes.byref(out)),
           "zero_host_grad_stats")
    return out


def zero_host_step(h, rank: int, bufs: zero_opt_buffers, global_stats=None) -> None:
    gs = ctypes.byref(global_stats) if global_stats is not None else None
    _check(lib().zero_host_step(h, rank, ctypes.byref(bufs), gs), "zero_host_step")


def zero_host_grad_stats_tensors(h, rank: int, lst: zero_opt_tensor_list) -> zero_opt_stats:
    out = zero_opt_stats()
    _check(lib().zero_host_grad_stats_tensors(h, rank, ctypes.byref(lst), ctypes.byref(out)),
           "zero_host_grad_stats_tensors")
    return out


def zero_host_step_tensors(h, rank: int, lst: zero_opt_tensor_list, global_stats=None) -> None:
    gs = ctypes.byref(global_stats) if global_stats is not None else None
    _check(lib().zero_host_step_tensors(h, rank, ctypes.byref(lst), gs), "zero_host_step_tensors")


def zero_host_loss_scale(h, rank: int) -> zero_opt_scaler_state:
    out = zero_opt_scaler_state()
    _check(lib().zero_host_loss_scale(h, rank, ctypes.byref(out)), "zero_host_loss_scale")
    return out


def zero_host_set_loss_scale(h, rank: int, state: zero_opt_scaler_state) -> None:
    _check(lib().zero_host_set_loss_scale(h, rank, ctypes.byref(state)),
           "zero_host_set_loss_scale")


def zero_host_last_step(h) -> zero_opt_step_info:
    out = zero_opt_step_info()
    _check(lib().zero_host_last_step(h, ctypes.byref(out)), "zero_host_last_step")
    return out


def zero_opt_decision(h) -> int:
    """Device address of the handle's last decision (for `zero_muon_step`)."""
    out = _vp()
    _check(lib().zero_opt_decision(h, ctypes.byref(out)), "zero_opt_decision")
    return out.value


# ---------------------------------------------------------------- orthogonalised updates

# What a handle was made for, so that the binding can check tensors against it:
# (shapes, grad_dtype, param_dtype, device), an object of the handle's own.
_muon_handles = {}


def make_muon_config(grad_dtype=FP16, param_dtype=None, lr=2e-2, momentum=0.95, nesterov=True,
                     weight_decay=0.0, steps=5, coefs=None, eps=1e-7,
                     scale_rule=MUON_SCALE_ONE) -> zero_muon_config:
    """`coefs`: (a, b, c) for every step, or a list of one triple a step."""
    cfg = zero_muon_config()
    _check(lib().zero_muon_config_default(ctypes.byref(cfg)), "zero_muon_config_default")
    cfg.grad_dtype = grad_dtype
    cfg.param_dtype = grad_dtype if param_dtype is None else param_dtype
    cfg.lr, cfg.momentum, cfg.weight_decay, cfg.eps = lr, momentum, weight_decay, eps
    cfg.nesterov, cfg.steps, cfg.scale_rule = int(nesterov), steps, scale_rule
    if coefs is not None:
        each = list(coefs) if hasattr(coefs[0], "__len__") else [coefs] * min(steps, MUON_MAX_STEPS)
        if len(each) != steps:
            raise ValueError(f"{len(each)} coefficient triples for {steps} steps")
        for i, abc in enumerate(each[:MUON_MAX_STEPS]):
            cfg.coef[i][:] = [float(c) for c in abc]
    return cfg


def zero_muon_create(cfg: zero_muon_config, shapes) -> int:
    """Handle for matrices of `shapes`: (rows, cols) or (rows, cols, batch) each."""
    full = [tuple(s) + (1,) * (3 - len(s)) for s in shapes]
    arr = (zero_muon_shape * max(len(full), 1))(*full)
    h = _vp()
    _check(lib().zero_muon_create(ctypes.byref(cfg), arr, len(full), ctypes.byref(h)),
           "zero_muon_create")
    import torch
    dev = torch.cuda.current_device() if torch.cuda.is_available() else -1
    _muon_handles[h.value] = (full, cfg.grad_dtype, cfg.param_dtype, dev)
    return h.value


def _muon_handle(h):
    made = _muon_handles.get(h)
    if made is None:
        raise ValueError("not a handle of zero_muon_create")
    return made


def zero_muon_destroy(h) -> None:
    _muon_handles.pop(h, None)
    _check(lib().zero_muon_destroy(h), "zero_muon_destroy")


def zero_muon_workspace_bytes(h) -> int:
    out = _i64()
    _check(lib().zero_muon_workspace_bytes(h, ctypes.byref(out)), "zero_muon_workspace_bytes")
    return out.value


def zero_muon_set_lr(h, lr: float) -> None:
    _check(lib().zero_muon_set_lr(h, lr), "zero_muon_set_lr")


def zero_muon_orthogonalize(h, ins, outs, stream=None) -> None:
    """The orthogonalised form of every matrix of `ins` into `outs`: one tensor
    per shape of the handle, [rows, cols] or [batch, rows, cols], with
    contiguous rows; all inputs of one dtype (float16, bfloat16 or float32),
    all outputs of one."""
    import torch
    shapes = _muon_handle(h)[0]
    if len(ins) != len(shapes) or len(outs) != len(shapes):
        raise ValueError(f"{len(shapes)} inputs and outputs are wanted")
    codes = {torch.float16: FP16, torch.bfloat16: BF16, torch.float32: FP32}
    dev = torch.cuda.current_device()
    arr = (zero_muon_operand * max(len(shapes), 1))()
    dtypes = []
    for i, (rows, cols, batch) in enumerate(shapes):
        at = []
        for name, t, first in (("ins", ins[i], ins[0]), ("outs", outs[i], outs[0])):
            if not t.is_cuda or t.device.index != dev or t.dtype != first.dtype \
                    or t.dtype not in codes or t.shape[-2:] != (rows, cols) \
                    or (t.stride(-1) != 1 and cols > 1) \
                    or not (t.dim() == 3 and t.shape[0] == batch or t.dim() == 2 and batch == 1):
                raise ValueError(f"{name}[{i}] must be a CUDA tensor of the current device with "
                                 f"shape ({batch}, {rows}, {cols}), contiguous rows and the dtype "
                                 "of the others")
            at.append((t.stride(-2), t.stride(0) if t.dim() == 3 else 0))
            dtypes.append(codes[t.dtype])
        arr[i] = zero_muon_operand(ins[i].data_ptr(), outs[i].data_ptr(), *at[0], *at[1])
    _check(lib().zero_muon_orthogonalize(h, arr, dtypes[0] if dtypes else FP16,
                                         dtypes[1] if dtypes else FP16, _stream(stream)),
           "zero_muon_orthogonalize")


_MUON_ARRAYS = ("grad", "momentum", "master", "param16")


class _MuonList(tuple):
    """(array of zero_muon_matrix, items, their dicts), and the handle's entry
    in `_muon_handles` that the tensors have been checked against."""
    fits = None


def make_muon_list(mats):
    """Per-matrix list for `zero_muon_step`; each item is a dict with grad,
    momentum, master (or None: param16 is the master) and param16, contiguous:
    [batch, rows, cols], [batch * rows, cols], or the same numbers in one
    dimension (a slice of a flat buffer).  An address (int) is taken as it is."""
    arr = (zero_muon_matrix * max(len(mats), 1))()
    for i, m in enumerate(mats):
        for name in _MUON_ARRAYS:
            t = m[name]
            if hasattr(t, "is_contiguous") and not t.is_contiguous():
                raise ValueError(f"item {i}: {name} must be contiguous")
        arr[i] = zero_muon_matrix(*(_ptr(m[name]) for name in _MUON_ARRAYS))
    return _MuonList((arr, len(mats), [dict(m) for m in mats]))


def _muon_check(made, mats):
    """Compare every tensor of a list with what the handle was made for."""
    import torch
    shapes, grad, param, dev = made
    if mats[1] != len(shapes):
        raise ValueError(f"the list has {mats[1]} matrices, the handle {len(shapes)}")
    half = (torch.float16, torch.bfloat16)
    dtypes = dict(grad=half[grad], momentum=torch.float32, master=torch.float32, param16=half[param])
    for i, ((rows, cols, batch), m) in enumerate(zip(shapes, mats[2])):
        for name in _MUON_ARRAYS:
            t = m[name]
            if t is None or isinstance(t, int):
                continue
            if not isinstance(t, torch.Tensor) or t.get_device() != dev or not t.is_cuda \
                    or t.dtype is not dtypes[name] or t.numel() != batch * rows * cols \
                    or not (t.dim() == 1 or t.shape[-2:] == (rows, cols)
                            or t.shape == (batch * rows, cols)):
                raise ValueError(f"item {i}: {name} must be a {dtypes[name]} tensor of "
                                 f"{(batch, rows, cols)} on cuda:{dev}")
    mats.fits = made


def zero_muon_step(h, mats, grad_scale=1.0, decision=None, stream=None) -> None:
    """Step of every matrix (`mats` from `make_muon_list`, one item per shape of
    the handle).  `decision`: None, or the address from `zero_opt_decision`."""
    made = _muon_handle(h)
    if mats.fits is not made:
        _muon_check(made, mats)
    _check(lib().zero_muon_step(h, mats[0], grad_scale, _ptr(decision), _stream(stream)),
           "zero_muon_step")


def zero_muon_last_step(h, stream=None) -> zero_muon_info:
    out = zero_muon_info()
    _check(lib().zero_muon_last_step(h, _stream(stream), ctypes.byref(out)),
           "zero_muon_last_step")
    return out


def zero_muon_fault_count(h, stream=None) -> int:
    """Calls of the handle that have ended in a fault since its creation."""
    out = _i64()
    _check(lib().zero_muon_fault_count(h, _stream(stream), ctypes.byref(out)),
           "zero_muon_fault_count")
    return out.value


def zero_muon_inject_wait_fault(h) -> None:
    """Arm the failure-detection test hook for the next call."""
    _check(lib().zero_muon_inject_wait_fault(h), "zero_muon_inject_wait_fault")


def zero_muon_launch_count(h) -> int:
    out = _i64()
    _check(lib().zero_muon_launch_count(h, ctypes.byref(out)), "zero_muon_launch_count")
    return out.value


# ---------------------------------------------------------------- query/key norm and rotation

# What a handle was made for, so that the binding can check tensors against it
# (head counts, head_dim, rotary_dim / 2, dtype, gain_per_head, device), and
# memory for one call's zero_qk_buffers (calls on one handle are ordered).
_qk_handles = {}
_qk_pack = struct.Struct("=27qii").pack_into


def make_qk_config(q_heads, k_heads, head_dim, rotary_dim=None, dtype=BF16, interleaved=False,
                   eps=1e-6, gain_per_head=False) -> zero_qk_config:
    """`rotary_dim` None: the whole head rotates.  `dtype` FP16, BF16 or FP32."""
    return zero_qk_config(q_heads, k_heads, head_dim,
                          head_dim if rotary_dim is None else rotary_dim, dtype,
                          int(interleaved), int(gain_per_head), 0, eps)


def zero_qk_create(cfg: zero_qk_config) -> int:
    h = _vp()
    _check(lib().zero_qk_create(ctypes.byref(cfg), ctypes.byref(h)), "zero_qk_create")
    import torch
    dtype = (torch.float16, torch.bfloat16, torch.float32)[cfg.dtype]
    dev = torch.cuda.current_device() if torch.cuda.is_available() else -1
    b = zero_qk_buffers()
    _qk_handles[h.value] = (cfg.q_heads, cfg.k_heads, cfg.head_dim, cfg.rotary_dim // 2, dtype,
                            bool(cfg.gain_per_head), dev, b, ctypes.addressof(b))
    return h.value


def zero_qk_destroy(h) -> None:
    _qk_handles.pop(h, None)
    _check(lib().zero_qk_destroy(h), "zero_qk_destroy")


def _qk_refuse(name, what):
    raise ValueError(f"{name} must be {what}")


def _qk_heads(t, name, n, heads, dim, dtype, dev):
    """(address, token stride, head stride) of a [tokens, heads, D] tensor."""
    st, sh, sd = t.stride() if t.dim() == 3 else (0, 0, 0)
    if t.dtype is not dtype or t.shape != (n, heads, dim) or t.get_device() != dev or sd != 1:
        _qk_refuse(name, f"a {dtype} tensor of {(n, heads, dim)} with contiguous heads on "
                   f"cuda:{dev}")
    return t.data_ptr(), st, sh


def _qk_flat(t, name, shape, dtype, dev):
    """Address of a contiguous tensor."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        _qk_refuse(name, f"a contiguous {dtype} tensor of {tuple(shape)} on cuda:{dev}")
    return t.data_ptr()


_NO_HEADS = (0, 0, 0)


def _qk_call(fn, h, names, q, k, qo, ko, dq, dk, q_gain, k_gain, dq_gain, dk_gain, cos, sin,
             positions, stream):
    """Check the tensors against the handle and make the call."""
    import torch
    if h not in _qk_handles:
        raise ValueError("not a handle of zero_qk_create")
    hq, hk, dim, half, dtype, per_head, dev, b, at = _qk_handles[h]
    n = q.shape[0]
    f32 = torch.float32
    tq = _qk_heads(q, "q", n, hq, dim, dtype, dev)
    tqo = _qk_heads(qo, names[0], n, hq, dim, dtype, dev)
    tdq = _NO_HEADS if dq is None else _qk_heads(dq, "dq", n, hq, dim, dtype, dev)
    shape = (hq, dim) if per_head else (dim,)
    gq = 0 if q_gain is None else _qk_flat(q_gain, "q_gain", shape, f32, dev)
    dgq = 0 if dq_gain is None else _qk_flat(dq_gain, "dq_gain", shape, f32, dev)
    tk = tko = tdk = _NO_HEADS
    gk = dgk = 0
    if hk:
        tk = _qk_heads(k, "k", n, hk, dim, dtype, dev)
        tko = _qk_heads(ko, names[1], n, hk, dim, dtype, dev)
        if dk is not None:
            tdk = _qk_heads(dk, "dk", n, hk, dim, dtype, dev)
        if per_head:
            shape = (hk, dim)
        if k_gain is not None:
            gk = _qk_flat(k_gain, "k_gain", shape, f32, dev)
        if dk_gain is not None:
            dgk = _qk_flat(dk_gain, "dk_gain", shape, f32, dev)
    n_pos = pc = ps = 0
    if half:
        n_pos = cos.shape[0]
        table = (n_pos, half)
        pc = _qk_flat(cos, "cos", table, f32, dev)
        ps = _qk_flat(sin, "sin", table, f32, dev)
    wide = positions.dtype is torch.int64
    pp = _qk_flat(positions, "positions", (n,), torch.int64 if wide else torch.int32, dev)
    _qk_pack(b, 0, n, n_pos, *tq, *tk, *tqo, *tko, *tdq, *tdk, gq, gk, dgq, dgk, pc, ps, pp, wide, 0)
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev) if dev >= 0 else None
    status = fn(h, at, _stream(stream))
    if status:
        _check(status, fn.__name__)


def zero_qk_norm_rope(h, q, k, q_out, k_out, q_gain, k_gain, cos, sin, positions,
                      stream=None) -> None:
    """Normalise and rotate every head of `q` [tokens, q_heads, D] and `k` into
    `q_out` and `k_out` (which may be `q` and `k`).  `k`, `k_out` are not looked
    at by a handle with k_heads 0; a gain may be None (ones).  A token of
    position -1 is padding and gets zeros."""
    _qk_call(lib().zero_qk_norm_rope, h, ("q_out", "k_out"), q, k, q_out, k_out, None, None, q_gain,
             k_gain, None, None, cos, sin, positions, stream)


def zero_qk_norm_rope_backward(h, dq_out, dk_out, q, k, dq, dk, dq_gain, dk_gain, q_gain, k_gain,
                               cos, sin, positions, stream=None) -> None:
    """Gradients of `zero_qk_norm_rope`: from `dq_out`, `dk_out` and the
    forward call's inputs into `dq`, `dk` (which may be `dq_out`, `dk_out`) and
    the gains' float32 gradients (None: not wanted)."""
    _qk_call(lib().zero_qk_norm_rope_backward, h, ("dq_out", "dk_out"), q, k, dq_out, dk_out, dq, dk,
             q_gain, k_gain, dq_gain, dk_gain, cos, sin, positions, stream)


def zero_qk_launch_count(h) -> int:
    out = _i64()
    _check(lib().zero_qk_launch_count(h, ctypes.byref(out)), "zero_qk_launch_count")
    return out.value
