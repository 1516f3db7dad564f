"""ctypes binding of libddl (include/ddl.h): the same entry points, same names.

Argument marshalling only: every step of the all-reduce runs in the library's
CUDA kernels.  There is no fallback -- if libddl.so is missing, importing this
module raises.  PyTorch is optional plumbing: ``Plan.allreduce`` accepts torch
CUDA tensors (their ``data_ptr`` and the current stream) as well as raw device
pointers.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
# DDL_LIBRARY may name another build of the same library (e.g. one compiled
# with different kernel tuning macros); the default is the in-tree build.
LIB_PATH = os.environ.get("DDL_LIBRARY") or os.path.join(_HERE, "libddl.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run gradient_all_reduce_ddl_gb300.build.build() "
                      "(or __graft_entry__.build()) first")

_lib = ctypes.CDLL(LIB_PATH)

# ddl_status_t
DDL_OK, DDL_ERR_INVALID_ARG, DDL_ERR_UNSUPPORTED, DDL_ERR_OOM, DDL_ERR_CUDA, DDL_ERR_DEVICE_CHECK = range(6)
# ddl_dtype_t
DDL_FP32, DDL_FP16, DDL_BF16 = 0, 1, 2
# ddl_topo_kind_t
DDL_RING, DDL_MULTIRING, DDL_TORUS = 0, 1, 2
# ddl_mode_t
DDL_MODE_FUSED, DDL_MODE_STEPWISE, DDL_MODE_RANKORDER = 0, 1, 2
# ddl_kernel_t
DDL_KERNEL_AUTO, DDL_KERNEL_LDG, DDL_KERNEL_BULK_LOAD, DDL_KERNEL_CHUNKED = 0, 1, 3, 5
# ddl_act_t
DDL_ACT_NONE, DDL_ACT_RELU, DDL_ACT_GELU, DDL_ACT_SILU = range(4)

EXPORTS = [
    "ddl_plan_create", "ddl_plan_set_layers", "ddl_plan_set_mode", "ddl_plan_set_kernel", "ddl_allreduce",
    "ddl_allreduce_bucket", "ddl_allreduce_host", "ddl_overlap_begin", "ddl_bucket_ready", "ddl_overlap_end",
    "ddl_plan_num_buckets", "ddl_plan_bucket_range", "ddl_plan_traffic", "ddl_plan_fold_order",
    "ddl_plan_launches", "ddl_plan_kernel_name", "ddl_plan_check", "ddl_status_string", "ddl_plan_destroy",
    "ddl_allreduce_noalloc", "ddl_plan_cost", "ddl_plan_set_torus_dims", "ddl_allreduce_sgd", "ddl_selftest_wait_timeout",
    "ddl_allreduce_slab", "ddl_noalloc_check",
    "ddl_linear_create", "ddl_linear_forward", "ddl_linear_backward", "ddl_linear_check", "ddl_linear_destroy",
    "ddl_ortho_create", "ddl_ortho_set_polynomial", "ddl_ortho_run", "ddl_ortho_muon", "ddl_ortho_check",
    "ddl_ortho_destroy", "ddl_linear_selftest_wait_timeout", "ddl_ortho_selftest_wait_timeout",
    "ddl_xent_create", "ddl_xent_forward", "ddl_xent_backward", "ddl_xent_check", "ddl_xent_selftest_wait_timeout",
    "ddl_xent_destroy",
    "ddl_adam_create", "ddl_adam_set_betas", "ddl_adam_blocks", "ddl_adam_step", "ddl_adam_destroy",
]


class ddl_topology_t(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("k", ctypes.c_int32), ("X", ctypes.c_int32), ("Y", ctypes.c_int32)]


class ddl_matrix_t(ctypes.Structure):
    _fields_ = [("offset", ctypes.c_size_t), ("rows", ctypes.c_size_t), ("cols", ctypes.c_size_t),
                ("ld", ctypes.c_size_t)]


class ddl_tensor_t(ctypes.Structure):
    _fields_ = [("offset", ctypes.c_size_t), ("count", ctypes.c_size_t), ("lr_scale", ctypes.c_float),
                ("decay_scale", ctypes.c_float)]


_vp, _i, _sz, _u64, _f = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_uint64, ctypes.c_float
_P = ctypes.POINTER


def _sig(name, res, *args):
    fn = getattr(_lib, name)
    fn.restype = res
    fn.argtypes = list(args)
    return fn


_sig("ddl_plan_create", _i, _i, _sz, _i, ddl_topology_t, _sz, _P(_vp))
_sig("ddl_plan_set_layers", _i, _vp, _i, _P(_sz))
_sig("ddl_plan_set_mode", _i, _vp, _i)
_sig("ddl_plan_set_torus_dims", _i, _vp, _i, _P(_i))
_sig("ddl_plan_set_kernel", _i, _vp, _i)
_sig("ddl_allreduce", _i, _vp, _P(_vp), _f, _vp)
_sig("ddl_allreduce_bucket", _i, _vp, _i, _P(_vp), _f, _vp)
_sig("ddl_allreduce_slab", _i, _vp, _vp, _sz, _f, _vp)
_sig("ddl_allreduce_sgd", _i, _vp, _P(_vp), _P(_vp), _P(_vp), _f, _f, _f, _f, _i, _vp)
_sig("ddl_allreduce_host", _i, _vp, _P(_vp), _P(_vp), _f, _vp)
_sig("ddl_overlap_begin", _i, _vp, _P(_vp), _f, _vp)
_sig("ddl_bucket_ready", _i, _vp, _i, _vp)
_sig("ddl_overlap_end", _i, _vp, _vp)
_sig("ddl_plan_num_buckets", _i, _vp, _P(_i))
_sig("ddl_plan_bucket_range", _i, _vp, _i, _P(_sz), _P(_sz))
_sig("ddl_plan_traffic", _i, _vp, _P(_u64), _P(_u64))
_sig("ddl_plan_cost", _i, _vp, ctypes.c_double, ctypes.c_double, _i, _P(ctypes.c_double))
_sig("ddl_plan_fold_order", _i, _vp, _sz, _P(ctypes.c_int32), _P(ctypes.c_int32), _P(ctypes.c_int32))
_sig("ddl_plan_launches", _i, _vp, _P(_u64))
_sig("ddl_plan_kernel_name", _i, _vp, _P(ctypes.c_char_p))
_sig("ddl_plan_check", _i, _vp)
_sig("ddl_selftest_wait_timeout", _i, _vp, ctypes.c_uint32, _vp)
_sig("ddl_status_string", ctypes.c_char_p, _i)
_sig("ddl_plan_destroy", _i, _vp)
_sig("ddl_allreduce_noalloc", _i, _i, _sz, _i, ddl_topology_t, _sz, _i, _P(_sz), _P(_vp), _f, _vp)
_sig("ddl_noalloc_check", _i, _vp)
_sig("ddl_linear_create", _i, _sz, _sz, _sz, _i, _i, _P(_vp))
_sig("ddl_linear_forward", _i, _vp, _sz, _vp, _sz, _vp, _sz, _vp, _vp, _sz, _vp, _sz, _vp, _sz, _vp)
_sig("ddl_linear_backward", _i, _vp, _sz, _vp, _sz, _vp, _sz, _vp, _sz, _vp, _sz, _vp, _sz, _vp, _sz, _vp, _i, _i, _vp)
_sig("ddl_linear_check", _i, _vp, _vp)
_sig("ddl_linear_destroy", _i, _vp)
_sig("ddl_linear_selftest_wait_timeout", _i, _vp, *[ctypes.c_uint32] * 4)
_sig("ddl_ortho_create", _i, _i, _P(ddl_matrix_t), _i, _P(_vp))
_sig("ddl_ortho_set_polynomial", _i, _vp, _i, _f, _f, _f, _f)
_sig("ddl_ortho_run", _i, _vp, _vp, _vp, _vp)
_sig("ddl_ortho_muon", _i, _vp, _vp, _i, _P(_vp), _vp, _f, _f, _f, _i, _vp)
_sig("ddl_ortho_check", _i, _vp, _vp)
_sig("ddl_ortho_destroy", _i, _vp)
_sig("ddl_ortho_selftest_wait_timeout", _i, _vp, *[ctypes.c_uint32] * 4)

_sig("ddl_xent_create", _i, _sz, _sz, _sz, _i, _f, _P(_vp))
_sig("ddl_xent_forward", _i, _vp, _sz, _vp, _sz, _vp, _sz, _vp, _vp, _vp, _vp, _vp)
_sig("ddl_xent_backward", _i, _vp, _sz, _vp, _sz, _vp, _sz, _vp, _vp, _vp, _vp, _vp, _sz, _vp, _sz, _vp, _i, _i, _vp)
_sig("ddl_xent_check", _i, _vp, _vp)
_sig("ddl_xent_destroy", _i, _vp)
_sig("ddl_xent_selftest_wait_timeout", _i, _vp, *[ctypes.c_uint32] * 4)
_sig("ddl_adam_create", _i, _i, _P(ddl_tensor_t), _i, _i, _P(_vp))
_sig("ddl_adam_set_betas", _i, _vp, *[ctypes.c_double] * 3)
_sig("ddl_adam_blocks", _i, _vp, _P(_sz))
_sig("ddl_adam_step", _i, _vp, _vp, _i, _P(_vp), _P(_vp), _i, _vp, _vp, _vp, _vp, _f, _f, _f, _f, _vp, _vp)
_sig("ddl_adam_destroy", _i, _vp)


class DDLError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {ddl_status_string(status)}")


def _ok(status: int, where: str) -> None:
    if status != DDL_OK:
        raise DDLError(status, where)


def ddl_status_string(status: int) -> str:
    return _lib.ddl_status_string(status).decode()


def _ptr_array(ptrs):
    return (_vp * len(ptrs))(*ptrs)


def _dev_ptrs(bufs):
    return [b.data_ptr() if hasattr(b, "data_ptr") else int(b) for b in bufs]


_raw_stream = None  # torch's lookup of the current stream's handle, once found


def _stream_handle(stream):
    global _raw_stream
    if stream is None:
        try:
            if _raw_stream is not None:
                return _raw_stream(_current_device())
            return _find_raw_stream()
        except Exception:  # noqa: BLE001 - no torch / no GPU: the legacy default stream
            return 0
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _find_raw_stream():
    """The current stream's handle by torch's public call; keeps the direct lookups it is made of for later calls."""
    global _raw_stream, _current_device
    import torch
    handle = torch.cuda.current_stream().cuda_stream
    try:
        raw, device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
        if raw(device()) == handle:
            _raw_stream, _current_device = raw, device
    except AttributeError:
        pass
    return handle


# -- thin wrappers with the C names ------------------------------------------

def ddl_plan_create(P, N, dtype, topology, bucket_bytes=0):
    """topology: ddl_topology_t, or a dict(kind=..., k=..., X=..., Y=...)."""
    if isinstance(topology, dict):
        topology = ddl_topology_t(topology.get("kind", DDL_RING), topology.get("k", 1), topology.get("X", 0),
                                  topology.get("Y", 0))
    h = ctypes.c_void_p()
    _ok(_lib.ddl_plan_create(P, N, dtype, topology, bucket_bytes, ctypes.byref(h)), "ddl_plan_create")
    return h


def ddl_plan_set_layers(plan, numel_fwd_order):
    arr = (ctypes.c_size_t * len(numel_fwd_order))(*[int(v) for v in numel_fwd_order])
    _ok(_lib.ddl_plan_set_layers(plan, len(numel_fwd_order), arr), "ddl_plan_set_layers")


def ddl_plan_set_torus_dims(plan, dims):
    arr = (ctypes.c_int * len(dims))(*[int(d) for d in dims])
    _ok(_lib.ddl_plan_set_torus_dims(plan, len(dims), arr), "ddl_plan_set_torus_dims")


def ddl_plan_set_mode(plan, mode):
    _ok(_lib.ddl_plan_set_mode(plan, mode), "ddl_plan_set_mode")


def ddl_plan_set_kernel(plan, kernel):
    _ok(_lib.ddl_plan_set_kernel(plan, kernel), "ddl_plan_set_kernel")


def ddl_allreduce(plan, rank_bufs, scale, stream=None):
    _ok(_lib.ddl_allreduce(plan, _ptr_array(_dev_ptrs(rank_bufs)), scale, _stream_handle(stream)),
        "ddl_allreduce")


def ddl_allreduce_sgd(plan, grad_bufs, param_bufs, mom_bufs, scale, lr, momentum=0.0, weight_decay=0.0,
                      keep_grads=True, stream=None):
    moms = None if mom_bufs is None else _ptr_array(_dev_ptrs(mom_bufs))
    _ok(_lib.ddl_allreduce_sgd(plan, _ptr_array(_dev_ptrs(grad_bufs)), _ptr_array(_dev_ptrs(param_bufs)), moms,
                               scale, lr, momentum, weight_decay, 1 if keep_grads else 0, _stream_handle(stream)),
        "ddl_allreduce_sgd")


def ddl_allreduce_slab(plan, base, rank_stride_bytes, scale, stream=None):
    """base: device pointer (or tensor) of the slab; rank r at base + r * stride."""
    ptr = base.data_ptr() if hasattr(base, "data_ptr") else int(base)
    _ok(_lib.ddl_allreduce_slab(plan, ptr, rank_stride_bytes, scale, _stream_handle(stream)), "ddl_allreduce_slab")


def ddl_allreduce_bucket(plan, bucket, rank_bufs, scale, stream=None):
    _ok(_lib.ddl_allreduce_bucket(plan, bucket, _ptr_array(_dev_ptrs(rank_bufs)), scale,
                                  _stream_handle(stream)), "ddl_allreduce_bucket")


def ddl_allreduce_host(plan, host_bufs, dev_bufs, scale, stream=None):
    """dev_bufs None: the fused pass works on the host buffers in place."""
    dev = None if dev_bufs is None else _ptr_array(_dev_ptrs(dev_bufs))
    _ok(_lib.ddl_allreduce_host(plan, _ptr_array(_dev_ptrs(host_bufs)), dev, scale, _stream_handle(stream)),
        "ddl_allreduce_host")


def ddl_overlap_begin(plan, rank_bufs, scale, stream=None):
    _ok(_lib.ddl_overlap_begin(plan, _ptr_array(_dev_ptrs(rank_bufs)), scale, _stream_handle(stream)),
        "ddl_overlap_begin")


def ddl_bucket_ready(plan, bucket, stream=None):
    _ok(_lib.ddl_bucket_ready(plan, bucket, _stream_handle(stream)), "ddl_bucket_ready")


def ddl_overlap_end(plan, stream=None):
    _ok(_lib.ddl_overlap_end(plan, _stream_handle(stream)), "ddl_overlap_end")


def ddl_plan_num_buckets(plan):
    n = ctypes.c_int()
    _ok(_lib.ddl_plan_num_buckets(plan, ctypes.byref(n)), "ddl_plan_num_buckets")
    return n.value


def ddl_plan_bucket_range(plan, bucket):
    b, e = ctypes.c_size_t(), ctypes.c_size_t()
    _ok(_lib.ddl_plan_bucket_range(plan, bucket, ctypes.byref(b), ctypes.byref(e)), "ddl_plan_bucket_range")
    return b.value, e.value


def ddl_plan_traffic(plan):
    m, s = ctypes.c_uint64(), ctypes.c_uint64()
    _ok(_lib.ddl_plan_traffic(plan, ctypes.byref(m), ctypes.byref(s)), "ddl_plan_traffic")
    return m.value, s.value


def ddl_plan_cost(plan, alpha_s, beta_s_per_byte, links_per_worker=1):
    t = ctypes.c_double()
    _ok(_lib.ddl_plan_cost(plan, alpha_s, beta_s_per_byte, links_per_worker, ctypes.byref(t)), "ddl_plan_cost")
    return t.value


def ddl_plan_fold_order(plan, i, P):
    order = (ctypes.c_int32 * P)()
    inner, groups = ctypes.c_int32(), ctypes.c_int32()
    _ok(_lib.ddl_plan_fold_order(plan, i, order, ctypes.byref(inner), ctypes.byref(groups)), "ddl_plan_fold_order")
    return list(order), inner.value, groups.value


def ddl_plan_kernel_name(plan):
    """The kernel ddl_allreduce launches for the plan with 16-byte-aligned buffers."""
    name = ctypes.c_char_p()
    _ok(_lib.ddl_plan_kernel_name(plan, ctypes.byref(name)), "ddl_plan_kernel_name")
    return name.value.decode()


def ddl_plan_launches(plan):
    n = ctypes.c_uint64()
    _ok(_lib.ddl_plan_launches(plan, ctypes.byref(n)), "ddl_plan_launches")
    return n.value


def ddl_plan_check(plan):
    return _lib.ddl_plan_check(plan)


def ddl_selftest_wait_timeout(plan, limit_us, stream=None):
    _ok(_lib.ddl_selftest_wait_timeout(plan, limit_us, _stream_handle(stream)), "ddl_selftest_wait_timeout")


def ddl_plan_destroy(plan):
    _ok(_lib.ddl_plan_destroy(plan), "ddl_plan_destroy")


def ddl_allreduce_noalloc(P, N, dtype, topology, bucket_bytes, layers, rank_bufs, scale, stream=None):
    """Allocation-free all-reduce (no plan): tables in the library's static
    device array.  dtype: DDL_FP32/DDL_FP16; topology: ddl_topology_t or dict;
    layers: None or the tensor sizes in forward order."""
    if isinstance(topology, dict):
        topology = ddl_topology_t(topology.get("kind", DDL_RING), topology.get("k", 1), topology.get("X", 0),
                                  topology.get("Y", 0))
    layers = list(layers or [])
    arr = (ctypes.c_size_t * max(1, len(layers)))(*[int(v) for v in layers])
    _ok(_lib.ddl_allreduce_noalloc(P, N, dtype, topology, bucket_bytes, len(layers), arr,
                                   _ptr_array(_dev_ptrs(rank_bufs)), scale, _stream_handle(stream)),
        "ddl_allreduce_noalloc")


def ddl_noalloc_check(stream=None):
    """Status of the last allocation-free call's kernel on the current device
    (waits for `stream`); DDL_ERR_DEVICE_CHECK raises."""
    _ok(_lib.ddl_noalloc_check(_stream_handle(stream)), "ddl_noalloc_check")


def ddl_linear_create(max_tokens, in_features, out_features, dtype, act=DDL_ACT_NONE):
    h = ctypes.c_void_p()
    _ok(_lib.ddl_linear_create(max_tokens, in_features, out_features, dtype, act, ctypes.byref(h)), "ddl_linear_create")
    return h


def ddl_linear_forward(layer, tokens, x, ldx, w, ldw, bias, residual, ldr, z, ldz, y, ldy, stream=None):
    """Device pointers (or None) and row strides in elements."""
    _ok(_lib.ddl_linear_forward(layer, tokens, x, ldx, w, ldw, bias, residual, ldr, z, ldz, y, ldy,
                                _stream_handle(stream)), "ddl_linear_forward")


def ddl_linear_backward(layer, tokens, dy, ldy, x, ldx, w, ldw, z, ldz, dx, lddx, dw, lddw, db, grad_dtype,
                        accumulate=False, stream=None):
    """Device pointers (or None) and row strides in elements."""
    _ok(_lib.ddl_linear_backward(layer, tokens, dy, ldy, x, ldx, w, ldw, z, ldz, dx, lddx, dw, lddw, db, grad_dtype,
                                 1 if accumulate else 0, _stream_handle(stream)), "ddl_linear_backward")


def ddl_linear_check(layer, stream=None):
    _ok(_lib.ddl_linear_check(layer, _stream_handle(stream)), "ddl_linear_check")


_NEVER = 0xFFFFFFFF


def ddl_linear_selftest_wait_timeout(layer, limit_us, products=_NEVER, loads_even=_NEVER, loads_odd=_NEVER):
    _ok(_lib.ddl_linear_selftest_wait_timeout(layer, limit_us, products, loads_even, loads_odd),
        "ddl_linear_selftest_wait_timeout")


def ddl_linear_destroy(layer):
    _ok(_lib.ddl_linear_destroy(layer), "ddl_linear_destroy")


def ddl_ortho_create(matrices, dtype):
    """matrices: (offset, rows, cols) or (offset, rows, cols, ld) each."""
    arr = (ddl_matrix_t * max(1, len(matrices)))()
    for a, m in zip(arr, matrices):
        a.offset, a.rows, a.cols = (int(v) for v in m[:3])
        a.ld = int(m[3]) if len(m) > 3 else a.cols
    h = ctypes.c_void_p()
    _ok(_lib.ddl_ortho_create(len(matrices), arr, dtype, ctypes.byref(h)), "ddl_ortho_create")
    return h


def ddl_ortho_set_polynomial(ortho, steps, a, b, c, eps):
    _ok(_lib.ddl_ortho_set_polynomial(ortho, steps, a, b, c, eps), "ddl_ortho_set_polynomial")


def ddl_ortho_run(ortho, inp, out, stream=None):
    _ok(_lib.ddl_ortho_run(ortho, *_dev_ptrs([inp, out]), _stream_handle(stream)), "ddl_ortho_run")


def ddl_ortho_muon(ortho, grad, param_bufs, mom, lr, momentum=0.95, weight_decay=0.0, nesterov=True, stream=None):
    g, m = _dev_ptrs([grad, mom])
    _ok(_lib.ddl_ortho_muon(ortho, g, len(param_bufs), _ptr_array(_dev_ptrs(param_bufs)), m, lr, momentum,
                            weight_decay, 1 if nesterov else 0, _stream_handle(stream)), "ddl_ortho_muon")


def ddl_ortho_check(ortho, stream=None):
    _ok(_lib.ddl_ortho_check(ortho, _stream_handle(stream)), "ddl_ortho_check")


def ddl_ortho_selftest_wait_timeout(ortho, limit_us, products=_NEVER, loads_even=_NEVER, loads_odd=_NEVER):
    _ok(_lib.ddl_ortho_selftest_wait_timeout(ortho, limit_us, products, loads_even, loads_odd),
        "ddl_ortho_selftest_wait_timeout")


def ddl_ortho_destroy(ortho):
    _ok(_lib.ddl_ortho_destroy(ortho), "ddl_ortho_destroy")


def ddl_xent_create(max_tokens, in_features, vocab, dtype, smoothing=0.0):
    h = ctypes.c_void_p()
    _ok(_lib.ddl_xent_create(max_tokens, in_features, vocab, dtype, smoothing, ctypes.byref(h)), "ddl_xent_create")
    return h


def ddl_xent_forward(xent, tokens, x, ldx, w, ldw, bias, labels, loss, lse, stream=None):
    """Device pointers (or None) and row strides in elements."""
    _ok(_lib.ddl_xent_forward(xent, tokens, x, ldx, w, ldw, bias, labels, loss, lse, _stream_handle(stream)),
        "ddl_xent_forward")


def ddl_xent_backward(xent, tokens, x, ldx, w, ldw, bias, labels, lse, dloss, dx, lddx, dw, lddw, db, grad_dtype,
                      accumulate=False, stream=None):
    """Device pointers (or None) and row strides in elements."""
    _ok(_lib.ddl_xent_backward(xent, tokens, x, ldx, w, ldw, bias, labels, lse, dloss, dx, lddx, dw, lddw, db, grad_dtype,
                               1 if accumulate else 0, _stream_handle(stream)), "ddl_xent_backward")


def ddl_xent_check(xent, stream=None):
    _ok(_lib.ddl_xent_check(xent, _stream_handle(stream)), "ddl_xent_check")


def ddl_xent_selftest_wait_timeout(xent, limit_us, products=_NEVER, loads_even=_NEVER, loads_odd=_NEVER):
    _ok(_lib.ddl_xent_selftest_wait_timeout(xent, limit_us, products, loads_even, loads_odd), "ddl_xent_selftest_wait_timeout")


def ddl_xent_destroy(xent):
    _ok(_lib.ddl_xent_destroy(xent), "ddl_xent_destroy")


def ddl_adam_create(tensors, grad_dtype, state_bits):
    """tensors: (offset, count), (offset, count, lr_scale) or (offset, count, lr_scale, decay_scale) each."""
    arr = (ddl_tensor_t * max(1, len(tensors)))()
    for a, t in zip(arr, tensors):
        a.offset, a.count = int(t[0]), int(t[1])
        a.lr_scale = float(t[2]) if len(t) > 2 else 1.0
        a.decay_scale = float(t[3]) if len(t) > 3 else 1.0
    h = ctypes.c_void_p()
    _ok(_lib.ddl_adam_create(len(tensors), arr, grad_dtype, state_bits, ctypes.byref(h)), "ddl_adam_create")
    return h


def ddl_adam_set_betas(adam, beta1, beta2, eps):
    _ok(_lib.ddl_adam_set_betas(adam, beta1, beta2, eps), "ddl_adam_set_betas")


def ddl_adam_blocks(adam):
    n = ctypes.c_size_t()
    _ok(_lib.ddl_adam_blocks(adam, ctypes.byref(n)), "ddl_adam_blocks")
    return n.value


def ddl_adam_step(adam, grad, param_bufs, operand_bufs, operand_dtype, m, v, scales, step, lr, weight_decay=0.0,
                  grad_scale=1.0, max_norm=0.0, norm=None, stream=None):
    """operand_bufs, scales, norm: None where there are none."""
    g, pm, pv, ps = _dev_ptrs([grad, m, v, step])
    sc, nm = (None if t is None else _dev_ptrs([t])[0] for t in (scales, norm))
    out = None if operand_bufs is None else _ptr_array(_dev_ptrs(operand_bufs))
    _ok(_lib.ddl_adam_step(adam, g, len(param_bufs), _ptr_array(_dev_ptrs(param_bufs)), out, operand_dtype, pm, pv, sc, ps,
                           lr, weight_decay, grad_scale, max_norm, nm, _stream_handle(stream)), "ddl_adam_step")


def ddl_adam_destroy(adam):
    _ok(_lib.ddl_adam_destroy(adam), "ddl_adam_destroy")


# -- convenience object --------------------------------------------------------

# the per-call path of Plan.allreduce: the same entry point without argtypes,
# given ready-made ctypes arguments (no conversion on each call)
_ddl_allreduce = ctypes.CDLL(LIB_PATH).ddl_allreduce
_ddl_allreduce.restype = ctypes.c_int
_ddl_allreduce_sgd = ctypes.CDLL(LIB_PATH).ddl_allreduce_sgd
_ddl_allreduce_sgd.restype = ctypes.c_int
_NO_STREAM = object()  # no stream object seen yet (None means the current stream, looked up each call)

TOPOLOGIES = {"ring": DDL_RING, "multiring": DDL_MULTIRING, "torus": DDL_TORUS, "torus_nd": DDL_RING}
DTYPES = {"f32": DDL_FP32, "f16": DDL_FP16}
OPERAND_DTYPES = {"f32": DDL_FP32, "f16": DDL_FP16, "bf16": DDL_BF16}
ACTIVATIONS = {"none": DDL_ACT_NONE, "relu": DDL_ACT_RELU, "gelu": DDL_ACT_GELU, "silu": DDL_ACT_SILU}
MODES = {"fused": DDL_MODE_FUSED, "stepwise": DDL_MODE_STEPWISE, "rankorder": DDL_MODE_RANKORDER}
KERNELS = {"auto": DDL_KERNEL_AUTO, "ldg": DDL_KERNEL_LDG, "bulkload": DDL_KERNEL_BULK_LOAD,
           "chunked": DDL_KERNEL_CHUNKED}


class Plan:
    """An all-reduce plan for P rank buffers of N elements (owns a ddl_plan_t)."""

    def __init__(self, P, N, dtype="f32", topo="ring", k=1, X=0, Y=0, bucket_bytes=0, layers=None,
                 mode="fused", kernel="auto", dims=None):
        self.P, self.N, self.dtype = int(P), int(N), dtype
        self._last_ptrs, self._last_arr = None, None
        self._last_stream, self._last_handle = _NO_STREAM, None
        self._sgd_key, self._sgd_arrs = None, None
        self._sgd_hyper, self._sgd_c = None, None
        self._scale, self._c_scale = None, None
        topo_t = ddl_topology_t(TOPOLOGIES[topo], int(k), int(X), int(Y))
        self.handle = ddl_plan_create(self.P, self.N, DTYPES[dtype], topo_t, int(bucket_bytes))
        self._c_handle = self.handle  # a ctypes.c_void_p
        try:
            if layers is not None:
                ddl_plan_set_layers(self.handle, list(layers))
            if topo == "torus_nd":
                ddl_plan_set_torus_dims(self.handle, list(dims))
            if mode != "fused":
                ddl_plan_set_mode(self.handle, MODES[mode])
            if kernel != "auto":
                ddl_plan_set_kernel(self.handle, KERNELS[kernel])
        except Exception:
            ddl_plan_destroy(self.handle)
            self.handle = None
            self._c_handle = ctypes.c_void_p(None)
            raise

    @classmethod
    def for_workload(cls, w, **kw):
        return cls(w.P, w.N, w.dtype, w.topo, k=w.k, X=w.X, Y=w.Y, bucket_bytes=w.bucket_bytes,
                   layers=w.layers, dims=getattr(w, "dims", None), **kw)

    def _stream_c(self, stream):
        # the stream handle, kept for the stream object last seen (None: the
        # current stream, looked up on every call)
        if stream is None or stream is not self._last_stream:
            self._last_stream, self._last_handle = stream, ctypes.c_void_p(_stream_handle(stream))
            if stream is None:
                self._last_stream = _NO_STREAM
        return self._last_handle

    def _rank_array(self, rank_bufs, stream):
        # the per-call path of small all-reduces: the ctypes pointer array is
        # rebuilt only when the buffers change
        try:
            ptrs = [b.data_ptr() for b in rank_bufs]
        except AttributeError:
            ptrs = _dev_ptrs(rank_bufs)
        if ptrs != self._last_ptrs:
            self._last_ptrs, self._last_arr = ptrs, _ptr_array(ptrs)
        return self._last_arr, self._stream_c(stream)

    def allreduce(self, rank_bufs, scale, stream=None):
        arr, handle = self._rank_array(rank_bufs, stream)
        if scale != self._scale:
            self._scale, self._c_scale = scale, ctypes.c_float(scale)
        status = _ddl_allreduce(self._c_handle, arr, self._c_scale, handle)
        if status:
            raise DDLError(status, "ddl_allreduce")

    def allreduce_sgd(self, grad_bufs, param_bufs, mom_bufs, scale, lr, momentum=0.0, weight_decay=0.0,
                      keep_grads=True, stream=None):
        # as in allreduce: the three pointer arrays are rebuilt only when a
        # buffer changes (the pointers are compared on every call)
        try:
            key = ([b.data_ptr() for b in grad_bufs], [b.data_ptr() for b in param_bufs],
                   None if mom_bufs is None else [b.data_ptr() for b in mom_bufs])
        except AttributeError:
            key = (_dev_ptrs(grad_bufs), _dev_ptrs(param_bufs), None if mom_bufs is None else _dev_ptrs(mom_bufs))
        if key != self._sgd_key:
            self._sgd_key = key
            self._sgd_arrs = (_ptr_array(key[0]), _ptr_array(key[1]), None if key[2] is None else _ptr_array(key[2]))
        g, pa, m = self._sgd_arrs
        hyper = (scale, lr, momentum, weight_decay, bool(keep_grads))
        if hyper != self._sgd_hyper:  # the scalars as ctypes values, rebuilt when one changes
            self._sgd_hyper = hyper
            self._sgd_c = tuple(ctypes.c_float(v) for v in hyper[:4]) + (ctypes.c_int(1 if keep_grads else 0),)
        status = _ddl_allreduce_sgd(self._c_handle, g, pa, m, *self._sgd_c, self._stream_c(stream))
        if status:
            raise DDLError(status, "ddl_allreduce_sgd")

    def allreduce_slab(self, base, rank_stride_bytes, scale, stream=None):
        ddl_allreduce_slab(self.handle, base, rank_stride_bytes, scale, stream)

    def allreduce_bucket(self, bucket, rank_bufs, scale, stream=None):
        arr, handle = self._rank_array(rank_bufs, stream)
        _ok(_lib.ddl_allreduce_bucket(self.handle, bucket, arr, scale, handle.value), "ddl_allreduce_bucket")

    def allreduce_host(self, host_bufs, dev_bufs, scale, stream=None):
        ddl_allreduce_host(self.handle, host_bufs, dev_bufs, scale, stream)

    def overlap_begin(self, rank_bufs, scale, stream=None):
        ddl_overlap_begin(self.handle, rank_bufs, scale, stream)

    def bucket_ready(self, bucket, stream=None):
        ddl_bucket_ready(self.handle, bucket, stream)

    def overlap_end(self, stream=None):
        ddl_overlap_end(self.handle, stream)

    def set_mode(self, mode):
        ddl_plan_set_mode(self.handle, MODES[mode])

    def set_kernel(self, kernel):
        ddl_plan_set_kernel(self.handle, KERNELS[kernel])

    @property
    def num_buckets(self):
        return ddl_plan_num_buckets(self.handle)

    def bucket_range(self, b):
        return ddl_plan_bucket_range(self.handle, b)

    def buckets(self):
        return [self.bucket_range(b) for b in range(self.num_buckets)]

    def traffic(self):
        return ddl_plan_traffic(self.handle)

    def fold_order(self, i):
        return ddl_plan_fold_order(self.handle, i, self.P)

    @property
    def kernel_name(self):
        """The kernel ddl_allreduce launches (16-byte-aligned buffers)."""
        return ddl_plan_kernel_name(self.handle)

    def cost(self, alpha_s, beta_s_per_byte, links=1):
        """alpha-beta model of this schedule on P real workers with `links`
        network links each (seconds)."""
        return ddl_plan_cost(self.handle, alpha_s, beta_s_per_byte, links)

    @property
    def launches(self):
        return ddl_plan_launches(self.handle)

    def check(self):
        _ok(ddl_plan_check(self.handle), "ddl_plan_check")

    def close(self):
        if self.handle is not None:
            ddl_plan_destroy(self.handle)
            self.handle = None
            self._c_handle = ctypes.c_void_p(None)  # a later call gets DDL_ERR_INVALID_ARG

    def __del__(self):
        try:
            self.close()
        except Exception:  # noqa: BLE001 - interpreter shutdown
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()


def _matrix(t, rows, cols, dtype, name):
    """(pointer, row stride) of a rows x cols tensor with contiguous rows; (None, 0) for None."""
    if t is None:
        return None, 0
    if t.shape != (rows, cols):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {(rows, cols)}")
    if t.dtype is not dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    ld, unit = t.stride()
    if not t.is_cuda or (unit != 1 and cols > 1) or (ld < cols and rows > 1):
        raise ValueError(f"{name}: expected a CUDA tensor with contiguous, non-overlapping rows, strides {t.stride()}")
    return t.data_ptr(), ld if rows > 1 else cols


def _vector(t, n, dtype, name):
    if t is None:
        return None
    if t.dtype is dtype and t.is_cuda and t.dim() == 1 and t.numel() == n and t.is_contiguous():
        return t.data_ptr()
    if t.shape != (n,):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {(n,)}")
    if t.dtype is not dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    raise ValueError(f"{name}: expected a contiguous CUDA vector")


def _torch_dtype(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def _grad_dtype(t):
    name = str(t.dtype)
    if name not in ("torch.float32", "torch.float16"):
        raise ValueError(f"gradients: dtype {name}, expected torch.float32 or torch.float16")
    return DDL_FP32 if name == "torch.float32" else DDL_FP16


class Linear:
    """A linear layer y = act(x w^T + bias) + residual and its backward pass
    (owns a ddl_linear_t).  Tensors are the caller's: 16-bit of ``dtype``, rows
    contiguous at any stride; gradients binary32 or binary16, e.g. views into a
    rank's flat gradient buffer.  Nothing is recorded for autograd, whatever
    requires_grad says: backward() is the caller's to call."""

    def __init__(self, in_features, out_features, max_tokens, dtype="f16", act="none"):
        self.n_in, self.n_out, self.max_tokens, self.dtype, self.act = in_features, out_features, max_tokens, dtype, act
        self._dtype = _torch_dtype(dtype)
        self.handle = None
        self.handle = ddl_linear_create(max_tokens, in_features, out_features, OPERAND_DTYPES[dtype], ACTIVATIONS[act])

    def forward(self, x, w, y, bias=None, residual=None, z=None, stream=None):
        """Writes y (and the pre-activations z, where given); returns y."""
        t, d = x.shape[0], self._dtype
        px, ldx = _matrix(x, t, self.n_in, d, "x")
        pw, ldw = _matrix(w, self.n_out, self.n_in, d, "w")
        pr, ldr = _matrix(residual, t, self.n_out, d, "residual")
        pz, ldz = _matrix(z, t, self.n_out, d, "z")
        py, ldy = _matrix(y, t, self.n_out, d, "y")
        ddl_linear_forward(self.handle, t, px, ldx, pw, ldw, _vector(bias, self.n_out, d, "bias"), pr, ldr, pz, ldz, py,
                           ldy, stream)
        return y

    def backward(self, dy, x=None, w=None, z=None, dx=None, dw=None, db=None, accumulate=False, stream=None):
        """Writes dx; writes dw and db, or adds to them."""
        t, d = dy.shape[0], self._dtype
        some = dw if dw is not None else db
        g, grad_dtype = (None, DDL_FP32) if some is None else (some.dtype, _grad_dtype(some))
        pdy, ldy = _matrix(dy, t, self.n_out, d, "dy")
        px, ldx = _matrix(x, t, self.n_in, d, "x")
        pw, ldw = _matrix(w, self.n_out, self.n_in, d, "w")
        pz, ldz = _matrix(z, t, self.n_out, d, "z")
        pdx, lddx = _matrix(dx, t, self.n_in, d, "dx")
        pdw, lddw = _matrix(dw, self.n_out, self.n_in, g, "dw")
        ddl_linear_backward(self.handle, t, pdy, ldy, px, ldx, pw, ldw, pz, ldz, pdx, lddx, pdw, lddw,
                            _vector(db, self.n_out, g, "db"), grad_dtype, accumulate, stream)

    def check(self, stream=None):
        ddl_linear_check(self.handle, stream)

    def close(self):
        handle, self.handle = self.handle, None  # destroyed once, also where that reports an error
        if handle is not None:
            ddl_linear_destroy(handle)

    def __del__(self):
        try:
            self.close()
        except Exception:  # noqa: BLE001 - interpreter shutdown
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()


class Ortho:
    """Newton-Schulz orthogonalisation of the matrices of a flat buffer, alone
    or inside the Muon step (owns a ddl_ortho_t).  matrices: (offset, rows,
    cols) or (offset, rows, cols, ld) each, in elements."""

    def __init__(self, matrices, dtype="f32", steps=5, coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7):
        self.matrices = [tuple(int(v) for v in m) for m in matrices]
        self.dtype = dtype
        self.extent = max((m[0] + (m[1] - 1) * (m[3] if len(m) > 3 else m[2]) + m[2] for m in self.matrices), default=0)
        self._dtype, self._f32 = _torch_dtype(dtype), _torch_dtype("f32")
        self.handle = None
        self.handle = ddl_ortho_create(self.matrices, OPERAND_DTYPES[dtype])
        ddl_ortho_set_polynomial(self.handle, steps, *coefficients, eps)

    def _flat(self, t, dtype, name):
        if t.dim() != 1 or t.numel() < self.extent or t.dtype is not dtype or not t.is_cuda or (
                t.numel() > 1 and t.stride(0) != 1):
            raise ValueError(f"{name}: expected a contiguous CUDA vector of {dtype} with at least {self.extent} elements")
        return t

    def run(self, inp, out, stream=None):
        """Orthogonalises every matrix of inp into out; returns out."""
        ddl_ortho_run(self.handle, self._flat(inp, self._dtype, "inp"), self._flat(out, self._dtype, "out"), stream)
        return out

    def muon(self, grad, params, mom, lr, momentum=0.95, weight_decay=0.0, nesterov=True, stream=None):
        """Updates mom and every copy in params (a list, one per rank) in place."""
        ddl_ortho_muon(self.handle, self._flat(grad, self._dtype, "grad"),
                       [self._flat(p, self._f32, "params") for p in params],
                       self._flat(mom, self._f32, "mom"), lr, momentum, weight_decay, nesterov, stream)

    def check(self, stream=None):
        ddl_ortho_check(self.handle, stream)

    def close(self):
        handle, self.handle = self.handle, None  # destroyed once, also where that reports an error
        if handle is not None:
            ddl_ortho_destroy(handle)

    def __del__(self):
        try:
            self.close()
        except Exception:  # noqa: BLE001 - interpreter shutdown
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()


class CrossEntropy:
    """Softmax cross entropy of a linear head z = x w^T + bias over a vocabulary,
    and its backward pass; the logits are never kept (owns a ddl_xent_t).  Tensors
    are the caller's, as for Linear; labels are int64, negative ones ignored; loss,
    lse and dloss are binary32.  Nothing is recorded for autograd."""

    def __init__(self, in_features, vocab, max_tokens, dtype="f16", smoothing=0.0):
        self.n_in, self.vocab, self.max_tokens, self.dtype, self.smoothing = in_features, vocab, max_tokens, dtype, smoothing
        self._dtype, self._f32 = _torch_dtype(dtype), _torch_dtype("f32")
        import torch
        self._i64 = torch.int64
        self.handle = None
        self.handle = ddl_xent_create(max_tokens, in_features, vocab, OPERAND_DTYPES[dtype], smoothing)

    def forward(self, x, w, labels, loss, lse=None, bias=None, stream=None):
        """Writes every token's loss (and the logarithm of its softmax sum, where given); returns loss.  Either may be None."""
        t, d = x.shape[0], self._dtype
        px, ldx = _matrix(x, t, self.n_in, d, "x")
        pw, ldw = _matrix(w, self.vocab, self.n_in, d, "w")
        ddl_xent_forward(self.handle, t, px, ldx, pw, ldw, _vector(bias, self.vocab, d, "bias"),
                         _vector(labels, t, self._i64, "labels"), _vector(loss, t, self._f32, "loss"),
                         _vector(lse, t, self._f32, "lse"), stream)
        return loss

    def backward(self, x, w, labels, lse, dloss=None, bias=None, dx=None, dw=None, db=None, accumulate=False, stream=None):
        """From forward's lse and the gradient of every token's loss (None: ones) writes dx; writes dw and db, or adds to them."""
        t, d = x.shape[0], self._dtype
        some = dw if dw is not None else db
        g, grad_dtype = (None, DDL_FP32) if some is None else (some.dtype, _grad_dtype(some))
        px, ldx = _matrix(x, t, self.n_in, d, "x")
        pw, ldw = _matrix(w, self.vocab, self.n_in, d, "w")
        pdx, lddx = _matrix(dx, t, self.n_in, d, "dx")
        pdw, lddw = _matrix(dw, self.vocab, self.n_in, g, "dw")
        ddl_xent_backward(self.handle, t, px, ldx, pw, ldw, _vector(bias, self.vocab, d, "bias"),
                          _vector(labels, t, self._i64, "labels"), _vector(lse, t, self._f32, "lse"),
                          _vector(dloss, t, self._f32, "dloss"), pdx, lddx, pdw, lddw, _vector(db, self.vocab, g, "db"),
                          grad_dtype, accumulate, stream)

    def check(self, stream=None):
        ddl_xent_check(self.handle, stream)

    def close(self):
        handle, self.handle = self.handle, None  # destroyed once, also where that reports an error
        if handle is not None:
            ddl_xent_destroy(handle)

    def __del__(self):
        try:
            self.close()
        except Exception:  # noqa: BLE001 - interpreter shutdown
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()


class Adam:
    """AdamW steps over the tensors of flat buffers, on every rank's copy of the
    parameters (owns a ddl_adam_t).  tensors: (offset, count), optionally with the
    tensor's factors of lr and weight_decay, in elements; dtype: the gradient's;
    state: "f32" or "8bit"."""

    def __init__(self, tensors, dtype="f32", state="f32", betas=(0.9, 0.999), eps=1e-8):
        self.tensors = [tuple(t) for t in tensors]
        self.dtype, self.state = dtype, state
        self.extent = max((int(t[0]) + int(t[1]) for t in self.tensors), default=0)
        import torch
        self._grad, self._f32, self._i64 = _torch_dtype(dtype), torch.float32, torch.int64
        self._operands = {torch.float16: DDL_FP16, torch.bfloat16: DDL_BF16}
        self._state = {"f32": (torch.float32,), "8bit": (torch.uint8, torch.float8_e4m3fn)}[state]
        self.handle = None
        self.handle = ddl_adam_create(self.tensors, OPERAND_DTYPES[dtype], 8 if state == "8bit" else 32)
        ddl_adam_set_betas(self.handle, *betas, eps)
        self.n_blocks = ddl_adam_blocks(self.handle)

    def _flat(self, t, dtypes, name, n):
        """The address of a buffer of at least n elements."""
        if t.dtype in dtypes and t.is_cuda and t.numel() >= n and t.is_contiguous():
            return t.data_ptr()
        raise ValueError(f"{name}: expected a contiguous CUDA tensor of {dtypes[0]} with at least {n} elements")

    def new_state(self, device="cuda"):
        """The states before the first step, as step() takes them: m, v, step and (8 bits) scales."""
        import torch
        state = {k: torch.zeros(self.extent, dtype=self._state[0], device=device) for k in ("m", "v")}
        state["step"] = torch.zeros(1, dtype=torch.int64, device=device)
        if self.state == "8bit":
            state["scales"] = torch.zeros(2, self.n_blocks, device=device)
        return state

    def step(self, grad, params, m, v, step, lr, weight_decay=0.0, scales=None, operands=None, grad_scale=1.0, max_norm=0.0,
             norm=None, stream=None):
        """Updates every copy in params (a list, one per rank), the states and
        the step count (one int64 on the device) in place; writes the copies'
        16-bit operands and the gradient's norm where they are given."""
        flat, f32, n = self._flat, (self._f32,), self.extent
        out, out_dtype = None, DDL_FP16
        if operands is not None:
            if len(operands) != len(params):
                raise ValueError(f"operands: {len(operands)} buffers for {len(params)} copies")
            kind = operands[0].dtype if len(operands) else None
            if kind not in self._operands:
                raise ValueError(f"operands: dtype {kind}, expected torch.float16 or torch.bfloat16")
            out_dtype = self._operands[kind]
            out = _ptr_array([flat(o, (kind,), "operands", n) for o in operands])
        if scales is not None:
            if self.state != "8bit" or scales.numel() != 2 * self.n_blocks:
                raise ValueError(f"scales: a tensor of {2 * self.n_blocks} elements, with 8-bit states only")
            scales = flat(scales, f32, "scales", 0)
        _ok(_lib.ddl_adam_step(self.handle, flat(grad, (self._grad,), "grad", n), len(params),
                               _ptr_array([flat(p, f32, "params", n) for p in params]), out, out_dtype,
                               flat(m, self._state, "m", n), flat(v, self._state, "v", n), scales,
                               flat(step, (self._i64,), "step", 1), lr, weight_decay, grad_scale, max_norm,
                               None if norm is None else flat(norm, f32, "norm", 1), _stream_handle(stream)), "ddl_adam_step")

    def close(self):
        handle, self.handle = self.handle, None  # destroyed once, also where that reports an error
        if handle is not None:
            ddl_adam_destroy(handle)

    def __del__(self):
        try:
            self.close()
        except Exception:  # noqa: BLE001 - interpreter shutdown
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()
