"""Python binding of libccl.so, the C ABI in include/ccl.h.

AllReduce, ReduceScatter and AllGather over p rank buffers resident in one
GPU's memory, computed by hand-written sm_103a kernels.  Every function here
has the name of the C entry point it calls and only marshals arguments:
device pointers and streams are plain integers (``tensor.data_ptr()``,
``torch.cuda.current_stream().cuda_stream``); enum arguments accept the C
value or its name ("sum", "bf16", "ring", ...).  A non-OK status raises
:class:`CclError` carrying the status and ``ccl_last_error()``.

The library is built in-tree by :func:`reducescatter_reduction_gb300.build.build`;
calling any function before it exists raises ``RuntimeError`` (there is no
fallback implementation).
"""
from __future__ import annotations

import ctypes
import os
import struct

_HERE = os.path.dirname(os.path.abspath(__file__))
# CCL_LIBRARY names another build of this library to load instead (the
# checked build, libccl_checked.so, for tests)
LIB_PATH = os.environ.get("CCL_LIBRARY") or os.path.join(_HERE, "libccl.so")

CCL_OK, CCL_ERR_INVALID_ARG, CCL_ERR_UNSUPPORTED, CCL_ERR_CUDA, CCL_ERR_TIMEOUT, CCL_ERR_NOMEM, CCL_ERR_BOUNDS = range(7)
CCL_SUM, CCL_PROD, CCL_MIN, CCL_MAX, CCL_AVG = range(5)
CCL_F32, CCL_F16, CCL_BF16, CCL_I32 = range(4)
CCL_SCHED_AUTO, CCL_SCHED_RING, CCL_SCHED_ALLPAIRS, CCL_SCHED_CUSTOM = range(4)
(CCL_VARIANT_AUTO, CCL_VARIANT_LDST, CCL_VARIANT_TMA, CCL_VARIANT_TMA_BULKRED, CCL_VARIANT_RING_STEPWISE,
 CCL_VARIANT_ONE_PHASE) = range(6)
CCL_PASS_FORWARD, CCL_PASS_BACKWARD, CCL_PASS_BOTH = 1, 2, 3
CCL_MAX_RANKS = 64

OPS = {"sum": CCL_SUM, "prod": CCL_PROD, "min": CCL_MIN, "max": CCL_MAX, "avg": CCL_AVG}
DTYPES = {"f32": CCL_F32, "f16": CCL_F16, "bf16": CCL_BF16, "i32": CCL_I32}
SCHEDULES = {"auto": CCL_SCHED_AUTO, "ring": CCL_SCHED_RING, "allpairs": CCL_SCHED_ALLPAIRS,
             "custom": CCL_SCHED_CUSTOM}
VARIANTS = {"auto": CCL_VARIANT_AUTO, "ldst": CCL_VARIANT_LDST, "tma": CCL_VARIANT_TMA,
            "tma_bulkred": CCL_VARIANT_TMA_BULKRED, "ring_stepwise": CCL_VARIANT_RING_STEPWISE,
            "one_phase": CCL_VARIANT_ONE_PHASE}
PASSES = {"forward": CCL_PASS_FORWARD, "backward": CCL_PASS_BACKWARD, "both": CCL_PASS_BOTH}
STATUS_NAMES = {CCL_OK: "CCL_OK", CCL_ERR_INVALID_ARG: "CCL_ERR_INVALID_ARG",
                CCL_ERR_UNSUPPORTED: "CCL_ERR_UNSUPPORTED", CCL_ERR_CUDA: "CCL_ERR_CUDA",
                CCL_ERR_TIMEOUT: "CCL_ERR_TIMEOUT", CCL_ERR_NOMEM: "CCL_ERR_NOMEM", CCL_ERR_BOUNDS: "CCL_ERR_BOUNDS"}

# Every symbol include/ccl.h declares.
EXPORTS = (
    "ccl_comm_create", "ccl_comm_set_outputs", "ccl_comm_set_schedule", "ccl_set_launch", "ccl_comm_set_debug",
    "ccl_comm_destroy", "ccl_comm_check", "ccl_allreduce", "ccl_reduce_scatter", "ccl_all_gather",
    "ccl_allreduce_static", "ccl_allreduce_static_set_debug", "ccl_allreduce_residual_rmsnorm",
    "ccl_logit_rules", "ccl_distill_topk", "ccl_balance_loss",
    "ccl_allreduce_residual_rmsnorm_e4m3", "ccl_expert_sort", "ccl_expert_dispatch", "ccl_expert_combine",
    "ccl_expert_combine_grad", "ccl_grad_norm", "ccl_grad_clip",
    "ccl_schedule_build", "ccl_schedule_check", "ccl_cost_estimate", "ccl_select_schedule", "ccl_launch_estimate",
    "ccl_last_error", "ccl_comm_last_launch", "ccl_comm_launch_count", "ccl_comm_ranks", "ccl_version", "ccl_bounds_checked",
)


class CclError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


class CostParams(ctypes.Structure):
    """ccl_cost_params_t."""
    _fields_ = [("alpha_s", ctypes.c_double), ("bw_bytes_per_s", ctypes.c_double),
                ("eff_ring", ctypes.c_double), ("eff_allpairs", ctypes.c_double)]


class LogitRules(ctypes.Structure):
    """ccl_logit_rules_t: device pointers as integers, by keyword; what is left out is no rule."""
    _fields_ = [("repetition", ctypes.c_void_p), ("frequency", ctypes.c_void_p), ("presence", ctypes.c_void_p),
                ("history", ctypes.c_void_p), ("history_ld", ctypes.c_size_t), ("history_len", ctypes.c_void_p),
                ("prompt_len", ctypes.c_void_p), ("bias_offsets", ctypes.c_void_p), ("bias_tokens", ctypes.c_void_p),
                ("bias_values", ctypes.c_void_p), ("bias_count", ctypes.c_size_t), ("mask", ctypes.c_void_p),
                ("mask_rows", ctypes.c_size_t), ("mask_ld", ctypes.c_size_t), ("mask_index", ctypes.c_void_p)]


class Tensor(ctypes.Structure):
    """ccl_tensor_t: device pointers as integers; dtype a CCL_ value; an array of them is (Tensor * n)(...)."""
    _fields_ = [("in_", ctypes.c_void_p), ("out", ctypes.c_void_p), ("n", ctypes.c_size_t), ("dtype", ctypes.c_int),
                ("copy", ctypes.c_int32)]


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libccl.so and declare the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with reducescatter_reduction_gb300.build.build()")
    L = ctypes.CDLL(path)
    vp, i, sz, u64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_uint64
    pvp = ctypes.POINTER(ctypes.c_void_p)
    sigs = {
        "ccl_comm_create": (i, [ctypes.POINTER(vp), i, pvp]),
        "ccl_comm_set_outputs": (i, [vp, pvp]),
        "ccl_comm_set_schedule": (i, [vp, ctypes.POINTER(ctypes.c_uint8)]),
        "ccl_set_launch": (i, [vp, i, i, sz]),
        "ccl_comm_set_debug": (i, [vp, ctypes.c_longlong, i]),
        "ccl_comm_destroy": (i, [vp]),
        "ccl_comm_check": (i, [vp]),
        "ccl_allreduce": (i, [vp, i, i, sz, i, vp]),
        "ccl_reduce_scatter": (i, [vp, i, i, sz, i, vp]),
        "ccl_all_gather": (i, [vp, i, sz, vp]),
        "ccl_allreduce_static": (i, [i, pvp, pvp, i, i, sz, i, vp]),
        "ccl_allreduce_static_set_debug": (i, [ctypes.c_longlong, i]),
        "ccl_allreduce_residual_rmsnorm": (i, [vp, i, sz, sz, vp, vp, vp, ctypes.c_float, i, vp]),
        "ccl_logit_rules": (i, [vp, i, sz, sz, sz, ctypes.POINTER(LogitRules), vp]),
        "ccl_distill_topk": (i, [vp, i, i, sz, sz, sz, sz, vp, vp, i, ctypes.c_float, vp, vp, vp, vp]),
        "ccl_balance_loss": (i, [vp, i, i, sz, sz, sz, pvp, pvp, ctypes.c_float, vp, vp, vp, vp, vp]),
        "ccl_allreduce_residual_rmsnorm_e4m3": (i, [vp, i, sz, sz, vp, vp, vp, vp, sz, ctypes.c_float, i, vp]),
        "ccl_expert_sort": (i, [vp, sz, sz, sz, vp, vp, sz, vp, vp, vp]),
        "ccl_expert_dispatch": (i, [vp, i, sz, sz, sz, vp, vp, sz, vp]),
        "ccl_expert_combine": (i, [vp, i, sz, sz, sz, vp, vp, sz, vp]),
        "ccl_expert_combine_grad": (i, [vp, i, sz, sz, sz, vp, vp, vp, sz, vp, vp]),
        "ccl_grad_norm": (i, [vp, sz, ctypes.POINTER(Tensor), vp, vp]),
        "ccl_grad_clip": (i, [vp, sz, ctypes.POINTER(Tensor), ctypes.c_float, vp, vp]),
        "ccl_schedule_build": (i, [i, u64, i, ctypes.POINTER(u64), ctypes.POINTER(ctypes.c_uint8)]),
        "ccl_schedule_check": (i, [i, u64, ctypes.POINTER(u64), ctypes.POINTER(ctypes.c_uint8)]),
        "ccl_cost_estimate": (ctypes.c_double, [i, ctypes.c_double, i, ctypes.POINTER(CostParams)]),
        "ccl_select_schedule": (i, [i, ctypes.c_double, ctypes.POINTER(CostParams)]),
        "ccl_launch_estimate": (i, [i, i, i, sz, i, ctypes.POINTER(ctypes.c_double)]),
        "ccl_last_error": (ctypes.c_char_p, []),
        "ccl_comm_last_launch": (i, [vp, ctypes.c_char_p, sz]),
        "ccl_comm_launch_count": (u64, [vp]),
        "ccl_comm_ranks": (i, [vp]),
        "ccl_version": (i, []),
        "ccl_bounds_checked": (i, []),
    }
    for name, (res, args) in sigs.items():
        f = getattr(L, name)
        f.restype, f.argtypes = res, args
    _lib = L
    return L


def _code(table, v):
    return table[v] if isinstance(v, str) else int(v)


def _check(status: int):
    if status != CCL_OK:
        raise CclError(status, ccl_last_error())


def _ptr_array(ptrs):
    return (ctypes.c_void_p * len(ptrs))(*[int(x) for x in ptrs])


def _params(params):
    if params is None:
        return None
    if isinstance(params, CostParams):
        return ctypes.byref(params)
    return ctypes.byref(CostParams(*params))


# --------------------------------------------------------------------------
# entry points
# --------------------------------------------------------------------------

def _want_len(ptrs, p: int, what: str):
    # the C side reads exactly p pointers: a shorter list would be read past its end
    if ptrs is not None and len(ptrs) != int(p):
        raise CclError(CCL_ERR_INVALID_ARG, f"{what} has {len(ptrs)} pointers, p = {int(p)}")


def ccl_comm_create(p: int, rank_ptrs) -> int:
    _want_len(rank_ptrs, p, "rank_ptrs")
    h = ctypes.c_void_p()
    _check(load_library().ccl_comm_create(ctypes.byref(h), int(p), _ptr_array(rank_ptrs)))
    return h.value


def ccl_comm_set_outputs(comm: int, out_ptrs=None) -> None:
    arr = None if out_ptrs is None else _ptr_array(out_ptrs)
    _check(load_library().ccl_comm_set_outputs(comm, arr))


def ccl_comm_set_schedule(comm: int, order) -> None:
    flat = [int(v) for row in order for v in (row if hasattr(row, "__len__") else [row])]
    arr = (ctypes.c_uint8 * len(flat))(*flat)
    _check(load_library().ccl_comm_set_schedule(comm, arr))


def ccl_set_launch(comm: int, sm_budget: int = 0, variant=CCL_VARIANT_AUTO,
                   pipeline_chunk_bytes: int = 0) -> None:
    _check(load_library().ccl_set_launch(comm, int(sm_budget), _code(VARIANTS, variant),
                                         int(pipeline_chunk_bytes)))


def ccl_comm_set_debug(comm: int, wait_limit_ns: int = 0, stall_test: int = 0) -> None:
    _check(load_library().ccl_comm_set_debug(comm, int(wait_limit_ns), int(stall_test)))


def ccl_comm_destroy(comm: int) -> None:
    _check(load_library().ccl_comm_destroy(comm))


def ccl_comm_check(comm: int) -> None:
    _check(load_library().ccl_comm_check(comm))


def ccl_allreduce(comm: int, op, dtype, n: int, schedule=CCL_SCHED_AUTO, stream: int = 0) -> None:
    _check(load_library().ccl_allreduce(comm, _code(OPS, op), _code(DTYPES, dtype), int(n),
                                        _code(SCHEDULES, schedule), stream or None))


def ccl_reduce_scatter(comm: int, op, dtype, n: int, schedule=CCL_SCHED_AUTO, stream: int = 0) -> None:
    _check(load_library().ccl_reduce_scatter(comm, _code(OPS, op), _code(DTYPES, dtype), int(n),
                                             _code(SCHEDULES, schedule), stream or None))


def ccl_all_gather(comm: int, dtype, n: int, stream: int = 0) -> None:
    _check(load_library().ccl_all_gather(comm, _code(DTYPES, dtype), int(n), stream or None))


def ccl_allreduce_static(p: int, in_ptrs, out_ptrs, op, dtype, n: int, schedule=CCL_SCHED_AUTO,
                         stream: int = 0) -> None:
    """The allocation-free AllReduce (see include/ccl.h): for callers that may
    not allocate device memory; needs no communicator."""
    _want_len(in_ptrs, p, "in_ptrs")
    _want_len(out_ptrs, p, "out_ptrs")
    _check(load_library().ccl_allreduce_static(int(p), _ptr_array(in_ptrs), _ptr_array(out_ptrs),
                                               _code(OPS, op), _code(DTYPES, dtype), int(n),
                                               _code(SCHEDULES, schedule), stream or None))


def ccl_allreduce_static_set_debug(wait_limit_ns: int = 0, stall_test: int = 0) -> None:
    _check(load_library().ccl_allreduce_static_set_debug(int(wait_limit_ns), int(stall_test)))


def ccl_allreduce_residual_rmsnorm(comm: int, dtype, rows: int, hidden: int, residual_in: int,
                                   residual_out: int, gamma: int, eps: float = 1e-6,
                                   schedule=CCL_SCHED_AUTO, stream: int = 0) -> None:
    _check(load_library().ccl_allreduce_residual_rmsnorm(comm, _code(DTYPES, dtype), int(rows), int(hidden),
                                                         residual_in, residual_out, gamma, float(eps),
                                                         _code(SCHEDULES, schedule), stream or None))


def ccl_logit_rules(comm: int, dtype, rows: int, vocab: int, rules: LogitRules, ld: int = 0, stream: int = 0) -> None:
    """Penalties, biases and grammar masks on one decode step's logits (see include/ccl.h)."""
    _check(load_library().ccl_logit_rules(comm, _code(DTYPES, dtype), int(rows), int(vocab), int(ld),
                                          None if rules is None else ctypes.byref(rules), stream or None))


def ccl_distill_topk(comm: int, dtype, steps, rows: int, vocab: int, k: int, teacher_ids: int, teacher_logits: int,
                     teacher_dtype="f32", temperature: float = 1.0, row_weight: int = 0, loss: int = 0, stats: int = 0,
                     ld: int = 0, stream: int = 0) -> None:
    """The loss against a teacher's top k logits and its gradient; steps: "forward", "backward" or "both"."""
    _check(load_library().ccl_distill_topk(comm, _code(DTYPES, dtype), _code(PASSES, steps), int(rows), int(vocab),
                                           int(ld), int(k), teacher_ids, teacher_logits, _code(DTYPES, teacher_dtype),
                                           float(temperature), row_weight or None, loss or None, stats or None,
                                           stream or None))


def ccl_balance_loss(comm: int, dtype, steps, rows: int, experts: int, k: int, expert_ids, valid, coef: float,
                     dloss: int, counts: int, tokens: int, loss: int = 0, stream: int = 0) -> None:
    """A router's load-balance loss, per-expert counts and gradient.  expert_ids and valid are lists with one device
    pointer for each of the communicator's ranks (or None; see include/ccl.h)."""
    lib = load_library()
    p = lib.ccl_comm_ranks(comm)
    for ptrs, what in ((expert_ids, "expert_ids"), (valid, "valid")):
        _want_len(ptrs, p, what)
    _check(lib.ccl_balance_loss(comm, _code(DTYPES, dtype), _code(PASSES, steps), int(rows), int(experts), int(k),
                                None if expert_ids is None else _ptr_array(expert_ids),
                                None if valid is None else _ptr_array(valid), float(coef), dloss or None,
                                counts or None, tokens or None, loss or None, stream or None))


_PACK = [struct.Struct(f"{p}Q").pack for p in range(CCL_MAX_RANKS + 1)]


def _rank_array(p: int, ptrs, what: str):
    """One device pointer for each of p ranks, as the bytes of the C array (None: NULL)."""
    if ptrs is None:
        return None
    if len(ptrs) != p:
        _want_len(ptrs, p, what)
    return _PACK[p](*ptrs)


def _tensors(tensors):
    return tensors if isinstance(tensors, ctypes.Array) else (Tensor * len(tensors))(*tensors)


def ccl_allreduce_residual_rmsnorm_e4m3(comm: int, dtype, rows: int, hidden: int, residual_in: int, residual_out: int,
                                        gamma: int, scales, group: int = 0, eps: float = 1e-6, schedule=CCL_SCHED_AUTO,
                                        stream: int = 0) -> None:
    """AllReduce, residual and RMSNorm with e4m3 codes in the outputs; scales: a device pointer for each rank."""
    lib = load_library()
    p = lib.ccl_comm_ranks(comm)
    _check(lib.ccl_allreduce_residual_rmsnorm_e4m3(comm, _code(DTYPES, dtype), int(rows), int(hidden), residual_in or None,
                                                   residual_out or None, gamma or None, _rank_array(p, scales, "scales"),
                                                   int(group), float(eps), _code(SCHEDULES, schedule), stream or None))


def ccl_expert_sort(comm: int, rows: int, experts: int, k: int, expert_ids, valid, capacity: int, slots, offsets: int,
                    stream: int = 0) -> None:
    """The rows of all ranks' choices in their experts' buffers (see include/ccl.h); expert_ids, valid (or None) and
    slots: lists with a device pointer for each rank."""
    lib = load_library()
    p = lib.ccl_comm_ranks(comm)
    _check(lib.ccl_expert_sort(comm, int(rows), int(experts), int(k), _rank_array(p, expert_ids, "expert_ids"),
                               _rank_array(p, valid, "valid"), int(capacity), _rank_array(p, slots, "slots"),
                               offsets or None, stream or None))


def ccl_expert_dispatch(comm: int, dtype, rows: int, hidden: int, k: int, slots, weights, capacity: int,
                        stream: int = 0) -> None:
    """Tokens to the rows of their experts; slots and weights (or None): lists with a device pointer for each rank."""
    lib = load_library()
    p = lib.ccl_comm_ranks(comm)
    _check(lib.ccl_expert_dispatch(comm, _code(DTYPES, dtype), int(rows), int(hidden), int(k), _rank_array(p, slots, "slots"),
                                   _rank_array(p, weights, "weights"), int(capacity), stream or None))


def ccl_expert_combine(comm: int, dtype, rows: int, hidden: int, k: int, slots, weights, capacity: int,
                       stream: int = 0) -> None:
    """The experts' rows back to their tokens, weighted and summed; lists as ccl_expert_dispatch."""
    lib = load_library()
    p = lib.ccl_comm_ranks(comm)
    _check(lib.ccl_expert_combine(comm, _code(DTYPES, dtype), int(rows), int(hidden), int(k), _rank_array(p, slots, "slots"),
                                  _rank_array(p, weights, "weights"), int(capacity), stream or None))


def ccl_expert_combine_grad(comm: int, dtype, rows: int, hidden: int, k: int, slots, weights, expert_rows, capacity: int,
                            dweights, stream: int = 0) -> None:
    """The gradient of ccl_expert_combine by the experts' rows (the outputs) and by the weights."""
    lib = load_library()
    p = lib.ccl_comm_ranks(comm)
    _check(lib.ccl_expert_combine_grad(comm, _code(DTYPES, dtype), int(rows), int(hidden), int(k),
                                       _rank_array(p, slots, "slots"), _rank_array(p, weights, "weights"),
                                       _rank_array(p, expert_rows, "expert_rows"), int(capacity),
                                       _rank_array(p, dweights, "dweights"), stream or None))


def ccl_grad_norm(comm: int, tensors, norm: int, stream: int = 0) -> None:
    """The global norm of gradient tensors; tensors: a list of Tensor, or an array of them kept from call to call."""
    arr = _tensors(tensors)
    _check(load_library().ccl_grad_norm(comm, len(arr), arr, norm or None, stream or None))


def ccl_grad_clip(comm: int, tensors, max_norm: float, norm: int, stream: int = 0) -> None:
    """Clips gradient tensors by the global norm that norm[0] holds; norm[1] receives the factor."""
    arr = _tensors(tensors)
    _check(load_library().ccl_grad_clip(comm, len(arr), arr, float(max_norm), norm or None, stream or None))


def ccl_schedule_build(p: int, n: int, schedule):
    """Returns (bounds: list of p+1 ints, order: list of p rows of p ranks)."""
    bounds = (ctypes.c_uint64 * (p + 1))()
    order = (ctypes.c_uint8 * (p * p))()
    _check(load_library().ccl_schedule_build(int(p), int(n), _code(SCHEDULES, schedule), bounds, order))
    return list(bounds), [list(order[c * p:(c + 1) * p]) for c in range(p)]


def ccl_schedule_check(p: int, n: int, bounds, order) -> int:
    """Returns the status (CCL_OK or CCL_ERR_INVALID_ARG); does not raise."""
    b = (ctypes.c_uint64 * len(bounds))(*[int(v) for v in bounds])
    flat = [int(v) for row in order for v in row]
    o = (ctypes.c_uint8 * len(flat))(*flat)
    return load_library().ccl_schedule_check(int(p), int(n), b, o)


def ccl_cost_estimate(p: int, nbytes: float, schedule, params=None) -> float:
    return load_library().ccl_cost_estimate(int(p), float(nbytes), _code(SCHEDULES, schedule),
                                            _params(params))


def ccl_select_schedule(p: int, nbytes: float, params=None) -> int:
    return load_library().ccl_select_schedule(int(p), float(nbytes), _params(params))


def ccl_launch_estimate(p: int, dtype, sm_budget: int, bytes_per_rank: int, variant) -> float:
    """The launch table's per-call time estimate (us) for the ld/st or TMA kernel."""
    us = ctypes.c_double()
    _check(load_library().ccl_launch_estimate(int(p), _code(DTYPES, dtype), int(sm_budget), int(bytes_per_rank),
                                              _code(VARIANTS, variant), ctypes.byref(us)))
    return us.value


def ccl_last_error() -> str:
    msg = load_library().ccl_last_error()
    return msg.decode() if msg else ""


def ccl_comm_last_launch(comm: int) -> str:
    buf = ctypes.create_string_buffer(512)
    _check(load_library().ccl_comm_last_launch(comm, buf, len(buf)))
    return buf.value.decode()


def ccl_comm_launch_count(comm: int) -> int:
    return load_library().ccl_comm_launch_count(comm)


def ccl_comm_ranks(comm: int) -> int:
    return load_library().ccl_comm_ranks(comm)


def ccl_version() -> int:
    return load_library().ccl_version()


def ccl_bounds_checked() -> bool:
    """True when the loaded library is the checked build (CCL_BOUNDS_CHECK)."""
    return bool(load_library().ccl_bounds_checked())
