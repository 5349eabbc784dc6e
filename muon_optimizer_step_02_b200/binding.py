"""ctypes binding of libmuonb200.so (include/muon_b200.h).

Argument marshalling only: every step of the optimizer runs in the library's
CUDA kernels.  PyTorch provides device memory and streams.  There is no CPU
fallback: if the library is missing or a call fails, an exception is raised.
"""

from __future__ import annotations

import ctypes
import os
import warnings
from ctypes import (POINTER, Structure, c_char_p, c_double, c_float, c_int32,
                    c_int64, c_size_t, c_uint64, c_void_p)
from typing import List, Optional, Sequence, Tuple

_PKG = os.path.dirname(os.path.abspath(__file__))
# MUONB200_LIB selects another build of the library, e.g. the device-checked
# one (CHECKED_LIB_PATH), for a whole process.
LIB_PATH = os.environ.get("MUONB200_LIB") or os.path.join(_PKG, "libmuonb200.so")
CHECKED_LIB_PATH = os.path.join(_PKG, "libmuonb200_checked.so")

MUON_OK = 0
MUON_ERR_INVALID_ARG = -1
MUON_ERR_UNSUPPORTED = -2
MUON_ERR_ALIGNMENT = -3
MUON_ERR_CUDA = -4
MUON_ERR_TIMEOUT = -5
MUON_ERR_WORKSPACE = -6
MUON_ERR_DEVICE_CHECK = -7

KIND_NAMES = ("prologue", "gram", "poly", "apply", "final", "ns", "scale")


class muon_matrix_t(Structure):
    _fields_ = [("w", c_void_p), ("momentum", c_void_p),
                ("grad_bf16", c_void_p), ("update_out", c_void_p),
                ("rows", c_int32), ("cols", c_int32),
                ("update_scale", c_float)]


class muon_hyper_t(Structure):
    _fields_ = [("momentum", c_float), ("lr", c_float),
                ("weight_decay", c_float), ("eps_row", c_float),
                ("eps_frob", c_float), ("nesterov", c_int32),
                ("eq_r", c_int32)]


class muon_ramp_t(Structure):
    _fields_ = [("v0", c_float), ("v1", c_float), ("t0", c_int32),
                ("t1", c_int32)]


class muon_schedule_t(Structure):
    _fields_ = [("momentum", muon_ramp_t), ("lr", muon_ramp_t)]


def make_schedule(momentum_ramp, lr_ramp) -> muon_schedule_t:
    """(v0, v1, t0, t1) ramps for the momentum and the learning rate."""
    m, l = momentum_ramp, lr_ramp
    return muon_schedule_t(muon_ramp_t(float(m[0]), float(m[1]), int(m[2]), int(m[3])),
                           muon_ramp_t(float(l[0]), float(l[1]), int(l[2]), int(l[3])))


class adamw_hyper_t(Structure):
    _fields_ = [("lr", c_float), ("beta1", c_float), ("beta2", c_float),
                ("eps", c_float), ("weight_decay", c_float)]


class adamw_tensor_t(Structure):
    _fields_ = [("param", c_void_p), ("grad", c_void_p), ("exp_avg", c_void_p),
                ("exp_avg_sq", c_void_p), ("ema", c_void_p), ("numel", c_int64)]


MUON_F32, MUON_BF16 = 0, 1
_ROUNDINGS = {"nearest": 0, "stochastic": 1}
ADAM8_BLOCK = 256          # elements that share one pair of scale bytes


class adamw_mixed_hyper_t(Structure):
    _fields_ = [("lr", c_double), ("beta1", c_double), ("beta2", c_double),
                ("eps", c_double), ("weight_decay", c_double),
                ("ema_decay", c_double), ("seed", c_uint64), ("rounding", c_int32)]


class adamw_mixed_tensor_t(Structure):
    _fields_ = [("param", c_void_p), ("grad", c_void_p), ("exp_avg", c_void_p),
                ("exp_avg_sq", c_void_p), ("scale", c_void_p), ("ema", c_void_p),
                ("copy_bf16", c_void_p), ("numel", c_int64), ("lr_scale", c_float),
                ("wd_scale", c_float), ("grad_dtype", c_int32)]


class grad_tensor_t(Structure):
    _fields_ = [("grad", c_void_p), ("numel", c_int64), ("dtype", c_int32)]


class adam8_tensor_t(Structure):
    _fields_ = [("exp_avg8", c_void_p), ("root8", c_void_p), ("scale", c_void_p),
                ("exp_avg", c_void_p), ("second", c_void_p), ("numel", c_int64)]


class MuonError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} ({status})")
        self.status = status


_lib = None


def lib():
    """Loads the library once.  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: build it with "
            "`python -m muon_optimizer_step_02_b200._build` (no CPU fallback)")
    L = ctypes.CDLL(LIB_PATH)
    L.muon_plan_create.argtypes = [POINTER(c_int32), POINTER(c_int32), c_int32,
                                   c_int32, POINTER(c_void_p)]
    L.muon_plan_create.restype = c_int32
    L.muon_plan_workspace_bytes.argtypes = [c_void_p]
    L.muon_plan_workspace_bytes.restype = c_size_t
    L.muon_step_batched.argtypes = [c_void_p, POINTER(muon_matrix_t),
                                    POINTER(muon_hyper_t), POINTER(c_float),
                                    c_int32, c_void_p, c_size_t, c_void_p]
    L.muon_step_batched.restype = c_int32
    L.ema_update_batched.argtypes = [POINTER(c_void_p), POINTER(c_void_p),
                                     POINTER(c_int64), c_int32, c_float,
                                     c_void_p]
    L.ema_update_batched.restype = c_int32
    L.muon_get_last_error.argtypes = [c_void_p, c_void_p]
    L.muon_get_last_error.restype = c_int32
    L.muon_status_string.argtypes = [c_int32]
    L.muon_status_string.restype = c_char_p
    L.muon_plan_destroy.argtypes = [c_void_p]
    L.muon_plan_destroy.restype = None
    L.muon_plan_set_timing.argtypes = [c_void_p, c_int32]
    L.muon_plan_set_timing.restype = c_int32
    L.muon_plan_timing_read.argtypes = [c_void_p, POINTER(c_int32),
                                        POINTER(c_double), c_int32]
    L.muon_plan_timing_read.restype = c_int32
    L.muon_step_batched_sched.argtypes = [c_void_p, POINTER(muon_matrix_t),
                                          POINTER(muon_hyper_t),
                                          POINTER(muon_schedule_t), c_void_p,
                                          POINTER(c_float), c_int32, c_void_p,
                                          c_size_t, c_void_p]
    L.muon_step_batched_sched.restype = c_int32
    L.adamw_ema_batched.argtypes = [POINTER(adamw_tensor_t), c_int32,
                                    POINTER(adamw_hyper_t), c_int32, c_void_p,
                                    c_float, c_void_p]
    L.adamw_ema_batched.restype = c_int32
    L.adamw_ema_launches.argtypes = [c_int32, c_int32]
    L.adamw_ema_launches.restype = c_int32
    L.muon_plan_error_async.argtypes = [c_void_p, c_void_p, c_void_p]
    L.muon_plan_error_async.restype = c_int32
    L.muon_step_launches.argtypes = [c_int32]
    L.muon_step_launches.restype = c_int32
    L.muon_plan_step_launches.argtypes = [c_void_p, c_int32]
    L.muon_plan_step_launches.restype = c_int32
    L.ema_update_launches.argtypes = [c_int32]
    L.ema_update_launches.restype = c_int32
    L.muon_plan_set_fault.argtypes = [c_void_p, c_int32]
    L.muon_plan_set_fault.restype = c_int32
    L.muon_abi_version.argtypes = []
    L.muon_abi_version.restype = c_int32
    L.muon_step_batched_noalloc.argtypes = [POINTER(muon_matrix_t), c_int32,
                                            POINTER(muon_hyper_t),
                                            POINTER(c_float), c_int32,
                                            c_void_p]
    L.muon_step_batched_noalloc.restype = c_int32
    L.muon_noalloc_error_async.argtypes = [c_void_p, c_void_p]
    L.muon_noalloc_error_async.restype = c_int32
    L.muon_noalloc_set_fault.argtypes = [c_int32]
    L.muon_noalloc_set_fault.restype = c_int32
    L.muon_f32_to_bf16.argtypes = [c_void_p, c_void_p, c_int64, c_void_p]
    L.muon_f32_to_bf16.restype = c_int32
    L.adamw_mixed_batched.argtypes = [POINTER(adamw_mixed_tensor_t), c_int32,
                                      POINTER(adamw_mixed_hyper_t), c_int32,
                                      c_void_p, c_void_p, c_void_p, c_void_p]
    L.adamw_mixed_batched.restype = c_int32
    L.grad_norm_workspace_bytes.argtypes = []
    L.grad_norm_workspace_bytes.restype = c_size_t
    L.grad_norm_batched.argtypes = [POINTER(grad_tensor_t), c_int32, c_double,
                                    c_void_p, c_size_t, c_void_p, c_void_p]
    L.grad_norm_batched.restype = c_int32
    for f in (L.adam8_write_batched, L.adam8_read_batched):
        f.argtypes = [POINTER(adam8_tensor_t), c_int32, c_int32, c_void_p]
        f.restype = c_int32
    for f in (L.adamw_mixed_launches, L.grad_norm_launches, L.adam8_launches):
        f.argtypes = [c_int32]
        f.restype = c_int32
    L.muon_device_checks.argtypes = []
    L.muon_device_checks.restype = c_int32
    L.muon_device_allocation_count.argtypes = []
    L.muon_device_allocation_count.restype = c_int64
    _lib = L
    return L


def status_string(status: int) -> str:
    return lib().muon_status_string(status).decode()


def _check(status: int, what: str):
    if status != MUON_OK:
        raise MuonError(status, what)


def _stream_handle(stream) -> Optional[int]:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") \
        else int(stream)


def _check_tensor(t, dtype, shape, what):
    import torch
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} must have shape {tuple(shape)}, got "
                         f"{tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")


class MuonPlan:
    """A plan for a fixed list of matrix shapes (rows, cols)."""

    def __init__(self, shapes: Sequence[Tuple[int, int]], max_ns_steps: int = 5):
        L = lib()
        self.shapes = [(int(r), int(c)) for r, c in shapes]
        n = len(self.shapes)
        rows = (c_int32 * n)(*[r for r, _ in self.shapes])
        cols = (c_int32 * n)(*[c for _, c in self.shapes])
        h = c_void_p()
        _check(L.muon_plan_create(rows, cols, n, int(max_ns_steps),
                                  ctypes.byref(h)), "muon_plan_create")
        self._h = h
        self.max_ns_steps = int(max_ns_steps)
        self.workspace_bytes = int(L.muon_plan_workspace_bytes(h))

    @property
    def handle(self):
        return self._h

    def alloc_workspace(self, device=None):
        import torch
        return torch.empty(max(self.workspace_bytes, 1), dtype=torch.uint8,
                           device=device or "cuda")

    def step(self, weights, momenta, grads, hyper, coeffs, workspace,
             update_scales: Optional[Sequence[float]] = None,
             update_out=None, stream=None, schedule=None, step_dev=None):
        """One batched Muon step (muon_step_batched, or with `schedule` and
        `step_dev` muon_step_batched_sched).  weights/momenta: fp32 CUDA
        tensors (updated in place); grads: bf16 CUDA tensors; hyper: an
        object with momentum, lr, weight_decay, eps_row, eps_frob, nesterov,
        eq_r; coeffs: ns_steps rows of (a, b, c)."""
        self.bind(weights, momenta, grads, hyper, coeffs, workspace,
                  update_scales, update_out, schedule, step_dev)(stream)

    def bind(self, weights, momenta, grads, hyper, coeffs, workspace,
             update_scales: Optional[Sequence[float]] = None,
             update_out=None, schedule=None, step_dev=None):
        """Checks and marshals the arguments once; returns a callable
        `run(stream=None)` that enqueues muon_step_batched with them (or
        muon_step_batched_sched when `schedule`, a pair of (v0, v1, t0, t1)
        ramps for momentum and lr, and `step_dev`, a one-element int32 CUDA
        tensor holding the step number, are given).  The tensors must stay
        alive and in place while the callable is used."""
        import torch
        n = len(self.shapes)
        if not (len(weights) == len(momenta) == len(grads) == n):
            raise ValueError("one weight, momentum and gradient per matrix")
        if update_out is not None and len(update_out) != n:
            raise ValueError("update_out must list one tensor (or None) per "
                             "matrix")
        mats = (muon_matrix_t * n)()
        for i, (r, c) in enumerate(self.shapes):
            _check_tensor(weights[i], torch.float32, (r, c), f"weights[{i}]")
            _check_tensor(momenta[i], torch.float32, (r, c), f"momenta[{i}]")
            _check_tensor(grads[i], torch.bfloat16, (r, c), f"grads[{i}]")
            o = update_out[i] if update_out is not None else None
            if o is not None:
                _check_tensor(o, torch.float32, (r, c), f"update_out[{i}]")
            s = (update_scales[i] if update_scales is not None
                 else max(1.0, r / c) ** 0.5)
            mats[i] = muon_matrix_t(weights[i].data_ptr(),
                                    momenta[i].data_ptr(),
                                    grads[i].data_ptr(),
                                    o.data_ptr() if o is not None else None,
                                    r, c, float(s))
        hp = muon_hyper_t(float(hyper.momentum), float(hyper.lr),
                          float(hyper.weight_decay), float(hyper.eps_row),
                          float(hyper.eps_frob), int(bool(hyper.nesterov)),
                          int(bool(hyper.eq_r)))
        if any(len(row) != 3 for row in coeffs):
            raise ValueError("coeffs: one (a, b, c) row per Newton-Schulz step")
        flat = [float(v) for row in coeffs for v in row]
        k = len(flat) // 3
        carr = (c_float * max(len(flat), 1))(*flat)
        _check_tensor(workspace, torch.uint8, (workspace.numel(),),
                      "workspace")
        hp_ref = ctypes.byref(hp)
        ws_ptr, ws_n = workspace.data_ptr(), workspace.numel()
        # The callable holds the plan (so that it outlives every bound call)
        # and reads its handle at call time (so that a closed plan raises
        # instead of handing a freed handle to the library).
        plan = self
        keep = (mats, hp, carr, weights, momenta, grads, update_out, workspace)
        if schedule is not None:
            if step_dev is None:
                raise ValueError("a schedule needs step_dev")
            _check_tensor(step_dev, torch.int32, (1,), "step_dev")
            sch = make_schedule(*schedule)
            fn_s = lib().muon_step_batched_sched
            sch_ref, sp = ctypes.byref(sch), step_dev.data_ptr()
            keep = keep + (sch, step_dev)

            def run_sched(stream=None):
                _ = keep
                _check(fn_s(plan._live_handle(), mats, hp_ref, sch_ref, sp, carr,
                            k, ws_ptr, ws_n, _stream_handle(stream)),
                       "muon_step_batched_sched")
            return run_sched
        fn = lib().muon_step_batched

        def run(stream=None):
            _ = keep
            _check(fn(plan._live_handle(), mats, hp_ref, carr, k, ws_ptr, ws_n,
                      _stream_handle(stream)), "muon_step_batched")
        return run

    def _live_handle(self):
        if self._h is None:
            raise MuonError(MUON_ERR_INVALID_ARG, "the plan has been closed")
        return self._h

    def last_error(self, stream=None) -> int:
        return int(lib().muon_get_last_error(self._h, _stream_handle(stream)))

    def error_async(self, host_word, stream=None):
        """Enqueues a copy of the device error word into `host_word` (a
        one-element int32 CPU tensor, pinned for the copy to be asynchronous);
        read it after the stream has passed this point."""
        import torch
        if host_word.dtype != torch.int32 or host_word.device.type != "cpu" or \
                host_word.numel() < 1:
            raise ValueError("host_word must be an int32 CPU tensor")
        _check(lib().muon_plan_error_async(self._h, host_word.data_ptr(),
                                           _stream_handle(stream)),
               "muon_plan_error_async")

    def step_launches(self, ns_steps: int) -> int:
        return int(lib().muon_plan_step_launches(self._h, int(ns_steps)))

    def set_timing(self, enable: bool):
        _check(lib().muon_plan_set_timing(self._h, int(enable)),
               "muon_plan_set_timing")

    def timing_read(self):
        n = len(KIND_NAMES)
        launches = (c_int32 * n)()
        ms = (c_double * n)()
        _check(lib().muon_plan_timing_read(self._h, launches, ms, n),
               "muon_plan_timing_read")
        return {KIND_NAMES[k]: (int(launches[k]), float(ms[k]))
                for k in range(n)}

    def set_fault(self, fault: int):
        _check(lib().muon_plan_set_fault(self._h, int(fault)),
               "muon_plan_set_fault")

    def close(self):
        if getattr(self, "_h", None):
            lib().muon_plan_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def muon_step_batched(plan: MuonPlan, *args, **kw):
    plan.step(*args, **kw)


def ema_update_batched(emas: Sequence, params: Sequence, decay: float,
                       stream=None):
    """E <- decay E + (1 - decay) P for every (E, P) pair (fp32 CUDA
    tensors, contiguous, same numel)."""
    ema_bind(emas, params, decay)(stream)


def ema_bind(emas: Sequence, params: Sequence, decay: float):
    """Checks and marshals the arguments of ema_update_batched once; returns
    a callable `run(stream=None)`."""
    import torch
    n = len(emas)
    if len(params) != n:
        raise ValueError("one parameter tensor per EMA tensor")
    e_arr = (c_void_p * max(n, 1))()
    p_arr = (c_void_p * max(n, 1))()
    num = (c_int64 * max(n, 1))()
    for i in range(n):
        e, p = emas[i], params[i]
        for t, what in ((e, f"emas[{i}]"), (p, f"params[{i}]")):
            if not t.is_cuda or t.dtype != torch.float32 or \
                    not t.is_contiguous():
                raise ValueError(f"{what} must be a contiguous fp32 CUDA "
                                 "tensor")
        if e.numel() != p.numel():
            raise ValueError(f"emas[{i}] and params[{i}] differ in size")
        e_arr[i] = e.data_ptr()
        p_arr[i] = p.data_ptr()
        num[i] = e.numel()
    fn = lib().ema_update_batched
    keep = (e_arr, p_arr, num, list(emas), list(params))
    d = float(decay)

    def run(stream=None):
        _ = keep
        _check(fn(e_arr, p_arr, num, n, d, _stream_handle(stream)),
               "ema_update_batched")
    return run


def step_launches(ns_steps: int) -> int:
    return int(lib().muon_step_launches(int(ns_steps)))


def adamw_ema_bind(params: Sequence, grads: Sequence, exp_avgs: Sequence,
                   exp_avg_sqs: Sequence, emas: Sequence, hyper, ema_decay: float,
                   step: int = 1, step_dev=None):
    """Marshals adamw_ema_batched once and returns `run(step_now=None,
    stream=None)`.  All tensors fp32 CUDA, contiguous, same numel per index;
    emas[i] may be None.  hyper: an object with lr, beta1, beta2, eps,
    weight_decay.  With step_dev (one-element int32 CUDA tensor) the device
    counter gives the step; otherwise `step`, or run's `step_now`."""
    import torch
    n = len(params)
    if not (len(grads) == len(exp_avgs) == len(exp_avg_sqs) == len(emas) == n):
        raise ValueError("one grad, exp_avg, exp_avg_sq and ema entry per param")
    arr = (adamw_tensor_t * max(n, 1))()
    for i in range(n):
        k = params[i].numel()
        for t, what in ((params[i], "params"), (grads[i], "grads"),
                        (exp_avgs[i], "exp_avgs"), (exp_avg_sqs[i], "exp_avg_sqs")):
            _check_tensor(t, torch.float32, (t.numel(),) if t.dim() == 1 else tuple(t.shape),
                          f"{what}[{i}]")
            if t.numel() != k:
                raise ValueError(f"{what}[{i}] has {t.numel()} elements, expected {k}")
        e = emas[i]
        if e is not None:
            _check_tensor(e, torch.float32, tuple(e.shape), f"emas[{i}]")
            if e.numel() != k:
                raise ValueError(f"emas[{i}] has {e.numel()} elements, expected {k}")
        arr[i] = adamw_tensor_t(params[i].data_ptr(), grads[i].data_ptr(),
                                exp_avgs[i].data_ptr(), exp_avg_sqs[i].data_ptr(),
                                e.data_ptr() if e is not None else None, k)
    hp = adamw_hyper_t(float(hyper.lr), float(hyper.beta1), float(hyper.beta2),
                       float(hyper.eps), float(hyper.weight_decay))
    sp = None
    if step_dev is not None:
        _check_tensor(step_dev, torch.int32, (1,), "step_dev")
        sp = step_dev.data_ptr()
    fn = lib().adamw_ema_batched
    keep = (arr, hp, list(params), list(grads), list(exp_avgs), list(exp_avg_sqs),
            list(emas), step_dev)
    hp_ref = ctypes.byref(hp)

    def run(step_now: Optional[int] = None, stream=None):
        _ = keep
        _check(fn(arr, n, hp_ref, int(step if step_now is None else step_now), sp,
                  float(ema_decay), _stream_handle(stream)), "adamw_ema_batched")
    return run


def adamw_ema_batched(params, grads, exp_avgs, exp_avg_sqs, emas, hyper,
                      ema_decay: float, step: int = 1, step_dev=None, stream=None):
    adamw_ema_bind(params, grads, exp_avgs, exp_avg_sqs, emas, hyper, ema_decay,
                   step, step_dev)(stream=stream)


def adamw_ema_launches(n_tensors: int, with_step_dev: bool = False) -> int:
    return int(lib().adamw_ema_launches(int(n_tensors), int(bool(with_step_dev))))


# ---- AdamW with 32-bit or 8-bit moments --------------------------------------

def _dense(t, dtypes, numel, what, device=None, i=None):
    """Checks a contiguous CUDA tensor of one of `dtypes` with `numel` elements
    (None: any number) on `device` (None: any); returns it.  what, i: its name
    and place in a list."""
    import torch
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in dtypes and \
            t.is_contiguous() and (numel is None or t.numel() == numel) and \
            (device is None or t.get_device() == device.index):
        return t
    what = _name(what, i)
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{what} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{what} has {t.numel()} elements, expected {numel}")
    raise ValueError(f"{what} is on {t.device}, expected {device}")


def _int32(x, what):
    x = int(x)
    if not -0x80000000 <= x <= 0x7FFFFFFF:
        raise ValueError(f"{what} {x} does not fit 32 bits")
    return x


def _name(what, i):
    return what if i is None else what.format(i)


def _check_overlap(written, read):
    """Raises if a written array shares memory with any other array of the
    call (the same tensor passed twice among them).  Entries: (tensor, name,
    place in a list or None)."""
    spans = []
    for w, group in ((True, written), (False, read)):
        for x in group:
            t = x[0]
            if t is not None and (k := t.numel()):
                p = t.data_ptr()
                spans.append((p, p + k * t.element_size(), w, x))
    spans.sort(key=lambda x: x[:2])
    end = end_w = 0        # furthest ends so far, of any array and of a written one,
    far = far_w = None     # and whose they are
    for b, e, w, x in spans:
        if b < end_w or (w and b < end):
            raise ValueError(f"{_name(*x[1:])} overlaps "
                             f"{_name(*(far_w if b < end_w else far)[1:])}")
        if e > end:
            end, far = e, x
        if w and e > end_w:
            end_w, far_w = e, x


def _bound(fn, what, device, keep):
    """run(args, stream=None): fn(*args, stream handle) with `device` current, on
    `stream` or the device's current stream; raises on an error status.  keep:
    what has to live as long as the callable."""
    import torch
    index = None if device is None else device.index
    current_device = torch.cuda.current_device
    # the current stream's handle without an object around it (3 us a call)
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
        (lambda i: torch.cuda.current_stream(i).cuda_stream)

    def elsewhere(args, stream):
        if device is None:
            return fn(*args, _stream_handle(stream))
        if stream is not None and getattr(stream, "device", device) != device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
        with torch.cuda.device(index):
            return fn(*args, raw(index) if stream is None else _stream_handle(stream))

    def run(args, stream=None):
        _ = keep
        status = fn(*args, raw(index)) if stream is None and index == current_device() \
            else elsewhere(args, stream)
        if status != MUON_OK:
            raise MuonError(status, what)
    return run


class Adam8State:
    """AdamW's moments of one tensor in 8 bits: codes of the first moment and
    of the second moment's root (uint8, one per element) and two scale bytes
    for every ADAM8_BLOCK elements begun.  The three tensors are what a
    checkpoint keeps; all zero is the state before the first step."""

    def __init__(self, exp_avg, root, scale):
        import torch
        n = _dense(exp_avg, (torch.uint8,), None, "exp_avg").numel()
        _dense(root, (torch.uint8,), n, "root", exp_avg.device)
        _dense(scale, (torch.uint8,), 2 * self.blocks(n), "scale", exp_avg.device)
        self.exp_avg, self.root, self.scale, self.numel = exp_avg, root, scale, n

    @staticmethod
    def blocks(numel: int) -> int:
        return -(-numel // ADAM8_BLOCK)

    def _checked(self, numel, device, i):
        """(exp_avg, root, scale) of the state at place i of a call, checked again:
        a checkpoint's loader may have put others in their places."""
        import torch
        u8 = (torch.uint8,)
        return (_dense(self.exp_avg, u8, numel, "states[{}].exp_avg", device, i),
                _dense(self.root, u8, numel, "states[{}].root", device, i),
                _dense(self.scale, u8, 2 * self.blocks(numel), "states[{}].scale", device, i))

    @classmethod
    def zeros(cls, numel: int, device=None) -> "Adam8State":
        import torch
        z = lambda k: torch.zeros(k, dtype=torch.uint8, device=device or "cuda")  # noqa: E731
        return cls(z(numel), z(numel), z(2 * cls.blocks(numel)))


def grad_norm_workspace(device=None):
    """A workspace of grad_norm_bind: zeroed, 16-byte aligned.  One for every
    group of calls (captured graphs among them) that are ordered."""
    import torch
    return torch.zeros(int(lib().grad_norm_workspace_bytes()), dtype=torch.uint8,
                       device=device or "cuda")


def grad_norm_bind(grads: Sequence, max_norm: float, out, workspace):
    """Marshals grad_norm_batched once and returns `run(stream=None)`: the norm
    of all gradients (contiguous fp32 or bf16 CUDA tensors) to out[0] and the
    coefficient that clips it at max_norm to out[1] (out: two fp32; NaN if a
    gradient is not finite).  adamw_mixed_bind reads the coefficient as its
    grad_scale; the Muon step does not.  Nothing is reduced across ranks."""
    import torch
    n = len(grads)
    dev = _dense(out, (torch.float32,), 2, "out").device
    _dense(workspace, (torch.uint8,), None, "workspace", dev)
    arr, kinds = (grad_tensor_t * max(n, 1))(), (torch.float32, torch.bfloat16)
    for i, g in enumerate(grads):
        _dense(g, kinds, None, "grads[{}]", dev, i)
        arr[i] = grad_tensor_t(g.data_ptr(), g.numel(),
                               MUON_BF16 if g.dtype == torch.bfloat16 else MUON_F32)
    _check_overlap([(out, "out", None), (workspace, "workspace", None)],
                   [(g, "grads[{}]", i) for i, g in enumerate(grads)])
    args = (arr, n, float(max_norm), workspace.data_ptr(), workspace.numel(), out.data_ptr())
    call = _bound(lib().grad_norm_batched, "grad_norm_batched", dev,
                  (arr, list(grads), out, workspace))

    def run(stream=None):
        call(args, stream)
    return run


def grad_norm_batched(grads, max_norm: float, out, workspace, stream=None):
    grad_norm_bind(grads, max_norm, out, workspace)(stream)


def adamw_mixed_bind(params: Sequence, grads: Sequence, states: Sequence, hyper,
                     emas: Optional[Sequence] = None, copies: Optional[Sequence] = None,
                     ema_decay: float = 0.0, step: int = 1, step_dev=None, lr_dev=None,
                     grad_scale=None, lr_scales: Optional[Sequence[float]] = None,
                     wd_scales: Optional[Sequence[float]] = None,
                     rounding: Optional[str] = None, seed: int = 0):
    """Marshals adamw_mixed_batched once and returns `run(step_now=None,
    stream=None)`.  All tensors contiguous, on one CUDA device, none sharing
    memory with another.

    params: fp32; grads: fp32 or bf16; states[i]: an Adam8State, or a pair
    (exp_avg, exp_avg_sq) of fp32 tensors; emas[i] (fp32) and copies[i] (bf16,
    receives the new parameters) may be None, as may the lists.  hyper: an
    object with lr, beta1, beta2, eps, weight_decay; lr_scales and wd_scales
    multiply lr and weight_decay per tensor.  With step_dev (two int32, zero
    before the first step) the device counts the steps; otherwise `step`, or
    run's `step_now`.  lr_dev: one fp32 read in place of hyper.lr.
    grad_scale: one fp32 that multiplies the gradients, such as out[1:] of
    grad_norm_bind; a value that is not finite skips the step.  rounding
    ("nearest" or "stochastic") and seed: how new moments go to 8 bits; calls
    on different tensors want different seeds, and counters of their own.
    Training wants "stochastic": over many steps nearest rounding leaves
    first moments whose gradients stopped above zero, so that their parameters
    go on moving, and roots far from AdamW's (muon_round_t in the header says
    how far).  None is "nearest", with a warning if there is an Adam8State.
    The callable keeps the tensors alive; they must stay in place."""
    import torch
    f32 = (torch.float32,)
    n = len(params)
    emas = [None] * n if emas is None else list(emas)
    copies = [None] * n if copies is None else list(copies)
    lr_scales = [1.0] * n if lr_scales is None else [float(x) for x in lr_scales]
    wd_scales = [1.0] * n if wd_scales is None else [float(x) for x in wd_scales]
    if not (len(grads) == len(states) == len(emas) == len(copies) == len(lr_scales)
            == len(wd_scales) == n):
        raise ValueError("one grad, state, ema, copy and scale entry per param")
    step = _int32(step, "step")
    if rounding is None:
        rounding = "nearest"
        if any(isinstance(s, Adam8State) for s in states):
            warnings.warn("8-bit moments rounded to the nearest lose track of AdamW over many "
                          "steps: pass rounding='stochastic' to train, or rounding='nearest' if "
                          "it is meant", stacklevel=2)
    if rounding not in _ROUNDINGS:
        raise ValueError(f"rounding must be one of {sorted(_ROUNDINGS)}, got {rounding!r}")
    dev = next((t.device for t in (*params, step_dev) if isinstance(t, torch.Tensor)), None)
    written, read = [], []
    arr = (adamw_mixed_tensor_t * max(n, 1))()
    b16, either = (torch.bfloat16,), (torch.float32, torch.bfloat16)
    for i in range(n):
        p = _dense(params[i], f32, None, "params[{}]", dev, i)
        k = p.numel()
        g = _dense(grads[i], either, k, "grads[{}]", dev, i)
        if isinstance(states[i], Adam8State):
            m, v, s = states[i]._checked(k, dev, i)
        else:
            (m, v), s = states[i], None
            _dense(m, f32, k, "states[{}][0]", dev, i)
            _dense(v, f32, k, "states[{}][1]", dev, i)
        e, c = emas[i], copies[i]
        if e is not None:
            _dense(e, f32, k, "emas[{}]", dev, i)
        if c is not None:
            _dense(c, b16, k, "copies[{}]", dev, i)
        arr[i] = adamw_mixed_tensor_t(
            p.data_ptr(), g.data_ptr(), m.data_ptr(), v.data_ptr(),
            None if s is None else s.data_ptr(), None if e is None else e.data_ptr(),
            None if c is None else c.data_ptr(), k, lr_scales[i], wd_scales[i],
            MUON_BF16 if g.dtype == torch.bfloat16 else MUON_F32)
        written += ((p, "params[{}]", i), (m, "states[{}]'s first moment", i),
                    (v, "states[{}]'s second moment", i), (s, "states[{}]'s scale", i),
                    (e, "emas[{}]", i), (c, "copies[{}]", i))
        read.append((g, "grads[{}]", i))
    for t, dt, k, what in ((step_dev, torch.int32, 2, "step_dev"),
                           (lr_dev, torch.float32, 1, "lr_dev"),
                           (grad_scale, torch.float32, 1, "grad_scale")):
        if t is not None:
            _dense(t, (dt,), k, what, dev)
            (written if what == "step_dev" else read).append((t, what, None))
    _check_overlap(written, read)
    hp = adamw_mixed_hyper_t(float(hyper.lr), float(hyper.beta1), float(hyper.beta2),
                             float(hyper.eps), float(hyper.weight_decay), float(ema_decay),
                             int(seed) & 0xFFFFFFFFFFFFFFFF, _ROUNDINGS[rounding])
    hp_ref = ctypes.byref(hp)
    dptr = lambda t: t.data_ptr() if t is not None else None  # noqa: E731
    pointers = (dptr(step_dev), dptr(lr_dev), dptr(grad_scale))
    args = (arr, n, hp_ref, step, *pointers)
    call = _bound(lib().adamw_mixed_batched, "adamw_mixed_batched", dev,
                  (arr, hp, written, read))

    def run(step_now: Optional[int] = None, stream=None):
        if step_now is None:
            call(args, stream)
        else:
            call((arr, n, hp_ref, _int32(step_now, "step_now"), *pointers), stream)
    return run


def adamw_mixed_batched(params, grads, states, hyper, stream=None, **kw):
    """One step of adamw_mixed_bind(params, grads, states, hyper, **kw)."""
    adamw_mixed_bind(params, grads, states, hyper, **kw)(stream=stream)


def _adam8_bind(states, exp_avgs, seconds, write: bool):
    import torch
    n = len(states)
    if not (len(exp_avgs) == len(seconds) == n):
        raise ValueError("one exp_avg and one second entry per state")
    arr = (adam8_tensor_t * max(n, 1))()
    dtype = exp_avgs[0].dtype if n else torch.float32
    if dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"plain moments must be torch.float32 or torch.bfloat16, got {dtype}")
    dev = states[0].exp_avg.device if n else None
    coded, plain, kind = [], [], (dtype,)
    for i, (s, m, v) in enumerate(zip(states, exp_avgs, seconds)):
        m8, r8, sc = s._checked(s.numel, dev, i)
        _dense(m, kind, s.numel, "exp_avgs[{}]", dev, i)
        _dense(v, kind, s.numel, "seconds[{}]", dev, i)
        arr[i] = adam8_tensor_t(m8.data_ptr(), r8.data_ptr(), sc.data_ptr(),
                                m.data_ptr(), v.data_ptr(), s.numel)
        coded += ((m8, "states[{}].exp_avg", i), (r8, "states[{}].root", i),
                  (sc, "states[{}].scale", i))
        plain += ((m, "exp_avgs[{}]", i), (v, "seconds[{}]", i))
    _check_overlap(coded if write else plain, plain if write else coded)
    what = "adam8_write_batched" if write else "adam8_read_batched"
    args = (arr, n, MUON_BF16 if dtype == torch.bfloat16 else MUON_F32)
    call = _bound(getattr(lib(), what), what, dev, (arr, coded, plain))

    def run(stream=None):
        call(args, stream)
    return run


def adam8_write_bind(states: Sequence, exp_avgs: Sequence, seconds: Sequence):
    """Marshals adam8_write_batched once and returns `run(stream=None)`:
    states[i] (Adam8State) <- plain moments, rounded to the nearest code.
    fp32 tensors hold the first and the second moment, bf16 tensors the first
    moment and the second moment's root."""
    return _adam8_bind(states, exp_avgs, seconds, True)


def adam8_read_bind(states: Sequence, exp_avgs: Sequence, seconds: Sequence):
    """Marshals adam8_read_batched once and returns `run(stream=None)`: plain
    moments <- what states[i] (Adam8State) stand for, exact in fp32 (first and
    second moment) and in bf16 (first moment and the second moment's root)."""
    return _adam8_bind(states, exp_avgs, seconds, False)


def adam8_write_batched(states, exp_avgs, seconds, stream=None):
    adam8_write_bind(states, exp_avgs, seconds)(stream)


def adam8_read_batched(states, exp_avgs, seconds, stream=None):
    adam8_read_bind(states, exp_avgs, seconds)(stream)


def adamw_mixed_launches(n_tensors: int) -> int:
    return int(lib().adamw_mixed_launches(int(n_tensors)))


def grad_norm_launches(n_tensors: int) -> int:
    return int(lib().grad_norm_launches(int(n_tensors)))


def adam8_launches(n_tensors: int) -> int:
    return int(lib().adam8_launches(int(n_tensors)))


def ema_launches(n_tensors: int) -> int:
    return int(lib().ema_update_launches(int(n_tensors)))


NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024
NOALLOC_MAX_MATS = 64


def muon_step_batched_noalloc(weights, momenta, grads, hyper, coeffs,
                              update_scales: Optional[Sequence[float]] = None,
                              update_out=None, stream=None):
    """One batched Muon step through muon_step_batched_noalloc: no plan and
    no workspace; the library's fixed device scratch array is used instead
    (for callers that cannot allocate device memory).  Same tensor rules as
    MuonPlan.step."""
    import torch
    n = len(weights)
    if not (len(momenta) == len(grads) == n):
        raise ValueError("one weight, momentum and gradient per matrix")
    mats = (muon_matrix_t * max(n, 1))()
    for i in range(n):
        if weights[i].dim() != 2:
            raise ValueError(f"weights[{i}] must be a matrix")
        r, c = (int(v) for v in weights[i].shape)
        _check_tensor(weights[i], torch.float32, (r, c), f"weights[{i}]")
        _check_tensor(momenta[i], torch.float32, (r, c), f"momenta[{i}]")
        _check_tensor(grads[i], torch.bfloat16, (r, c), f"grads[{i}]")
        o = update_out[i] if update_out is not None else None
        if o is not None:
            _check_tensor(o, torch.float32, (r, c), f"update_out[{i}]")
        s = (update_scales[i] if update_scales is not None
             else max(1.0, r / c) ** 0.5)
        mats[i] = muon_matrix_t(weights[i].data_ptr(), momenta[i].data_ptr(),
                                grads[i].data_ptr(),
                                o.data_ptr() if o is not None else None,
                                r, c, float(s))
    hp = muon_hyper_t(float(hyper.momentum), float(hyper.lr),
                      float(hyper.weight_decay), float(hyper.eps_row),
                      float(hyper.eps_frob), int(bool(hyper.nesterov)),
                      int(bool(hyper.eq_r)))
    if any(len(row) != 3 for row in coeffs):
        raise ValueError("coeffs: one (a, b, c) row per Newton-Schulz step")
    flat = [float(v) for row in coeffs for v in row]
    carr = (c_float * max(len(flat), 1))(*flat)
    _check(lib().muon_step_batched_noalloc(mats, n, ctypes.byref(hp), carr,
                                           len(flat) // 3,
                                           _stream_handle(stream)),
           "muon_step_batched_noalloc")


def noalloc_error_async(host_word, stream=None):
    """Enqueues a copy of the allocation-free path's error word into
    `host_word` (a one-element int32 CPU tensor, pinned for the copy to be
    asynchronous); non-zero once the stream has passed this point means the
    last muon_step_batched_noalloc call gave up on a bounded wait."""
    import torch
    if host_word.dtype != torch.int32 or host_word.device.type != "cpu" or \
            host_word.numel() < 1:
        raise ValueError("host_word must be an int32 CPU tensor")
    _check(lib().muon_noalloc_error_async(host_word.data_ptr(),
                                          _stream_handle(stream)),
           "muon_noalloc_error_async")


def noalloc_set_fault(fault: int):
    """Test hook of the allocation-free path (see muon_plan_set_fault)."""
    _check(lib().muon_noalloc_set_fault(int(fault)), "muon_noalloc_set_fault")


def device_allocation_count() -> int:
    """Device allocations the library has made in this process so far."""
    return int(lib().muon_device_allocation_count())


def f32_to_bf16(dst, src, stream=None):
    """dst (bf16 CUDA tensor) <- src (fp32 CUDA tensor, same numel) rounded to
    nearest even, by the library's conversion kernel."""
    import torch
    if not (src.is_cuda and dst.is_cuda) or src.dtype != torch.float32 or \
            dst.dtype != torch.bfloat16 or src.numel() != dst.numel() or \
            not (src.is_contiguous() and dst.is_contiguous()):
        raise ValueError("f32_to_bf16: contiguous fp32 src and bf16 dst CUDA "
                         "tensors of one size")
    _check(lib().muon_f32_to_bf16(dst.data_ptr(), src.data_ptr(), src.numel(),
                                  _stream_handle(stream)), "muon_f32_to_bf16")
