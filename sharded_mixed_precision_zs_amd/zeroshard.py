"""Python binding of libzeroshard (ctypes): argument marshalling only.

Each function has the name of the C entry point it calls (include/zeroshard.h
documents the semantics and cites the pages). Device buffers are torch CUDA
tensors (or raw integer device addresses); torch supplies memory and the
stream, every step of the computation runs in the library's HIP kernels.
The binding checks that each tensor is a contiguous CUDA tensor of the right
element size holding at least the elements the kernel will touch, then passes
plain pointers. There is no fallback: if the library is missing, importing
this module raises.
"""
import ctypes as C
import os
from typing import Optional, Sequence

from . import build as _build

ZS_ABI_VERSION = 7
ZS_MAX_WORLD = 64
ZS_BF16, ZS_FP16, ZS_FP32 = 0, 1, 2
ZS_WIRE_FP32, ZS_WIRE_BF16, ZS_WIRE_FP16 = 0, 1, 2
ZS_STATE_SPLIT, ZS_STATE_GROUPED = 0, 1
ZS_STATE_GROUP = 1024
ZS_MX_E2M1, ZS_MX_E4M3 = 0, 1
ZS_MX_BLOCK, ZS_MX_GROUP = 32, 128
ZS_DISTILL_MAX_SLOTS = 1024
ZS_ACT_NONE, ZS_ACT_RELU, ZS_ACT_GELU, ZS_ACT_SILU = 0, 1, 2, 3
ZS_PREFERENCE_SIGMOID, ZS_PREFERENCE_HINGE, ZS_PREFERENCE_SQUARE = 0, 1, 2
ZS_OK, ZS_ERR_INVALID_ARG, ZS_ERR_UNSUPPORTED, ZS_ERR_ALIAS, ZS_ERR_HIP = range(5)

LIB_PATH = _build.LIB


class ZsError(RuntimeError):
    def __init__(self, fn, status, detail):
        super().__init__(f"{fn}: {zs_status_string(status)}: {detail}")
        self.status = status


class zs_adamw_hparams(C.Structure):
    _fields_ = [("lr", C.c_float), ("beta1", C.c_float), ("beta2", C.c_float),
                ("eps", C.c_float), ("weight_decay", C.c_float),
                ("loss_scale", C.c_float), ("step_t", C.c_uint32)]


class zs_step_args(C.Structure):
    _fields_ = [("world", C.c_uint32), ("rank", C.c_uint32), ("n", C.c_uint64),
                ("grad_dtype", C.c_int32), ("param_dtype", C.c_int32),
                ("worker_grads", C.POINTER(C.c_void_p)),
                ("acc_in", C.c_void_p),
                ("master_in", C.c_void_p), ("m_in", C.c_void_p), ("v_in", C.c_void_p),
                ("master_out", C.c_void_p), ("m_out", C.c_void_p), ("v_out", C.c_void_p),
                ("gather_buf", C.c_void_p), ("gather_offset", C.c_uint64),
                ("overflow_flag", C.c_void_p),
                ("hp", zs_adamw_hparams), ("wire_dtype", C.c_int32),
                ("state_layout", C.c_int32)]


def grouped_len(n):
    """Floats in a grouped state buffer for n elements (whole groups)."""
    return -(-n // ZS_STATE_GROUP) * 3 * ZS_STATE_GROUP


class zs_loss_scaler(C.Structure):
    _fields_ = [("scale", C.c_float), ("clean_steps", C.c_uint32),
                ("growth_interval", C.c_uint32), ("dynamic", C.c_uint32),
                ("step_t", C.c_uint64), ("skipped", C.c_uint64)]


class zs_device_scaler(C.Structure):
    _fields_ = [("scale", C.c_float), ("clean_steps", C.c_uint32),
                ("growth_interval", C.c_uint32), ("dynamic", C.c_uint32),
                ("step_t", C.c_uint64), ("skipped", C.c_uint64),
                ("beta1_t", C.c_double), ("beta2_t", C.c_double),
                ("epoch", C.c_uint64), ("flag_epoch", C.c_uint64), ("checked_epoch", C.c_uint64),
                ("last_flag", C.c_uint32), ("bad_scale", C.c_uint32),
                ("last_alpha", C.c_float), ("last_bc2", C.c_float)]


class zs_dropout_rule(C.Structure):
    _fields_ = [("p", C.c_float), ("seed", C.c_uint64), ("offset", C.c_uint64),
                ("dev_offset", C.c_void_p)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libzeroshard is not built ({LIB_PATH}); "
                          "run __graft_entry__.build() -- there is no fallback path")
    # the library maps torch's HIP runtime whatever the import order (see
    # build.py), so it shares torch's streams and allocations
    lib = C.CDLL(LIB_PATH)
    vp, u32, u64, f32, i32 = C.c_void_p, C.c_uint32, C.c_uint64, C.c_float, C.c_int
    rule = C.POINTER(zs_dropout_rule)
    sig = {
        "zs_abi_version": ([], i32),
        "zs_status_string": ([i32], C.c_char_p),
        "zs_last_error": ([], C.c_char_p),
        "zs_partition": ([u64, u32, u32, C.POINTER(u64), C.POINTER(u64), C.POINTER(u64)], i32),
        "zs_reduce_scatter_avg": ([C.POINTER(vp), i32, i32, u32, u32, u64, vp, i32, vp, f32, vp],
                                  i32),
        "zs_check_overflow": ([vp, u64, f32, vp, vp], i32),
        "zs_adamw_step": ([vp, vp, vp, vp, u64, C.POINTER(zs_adamw_hparams), vp, vp], i32),
        "zs_cast_gather": ([vp, vp, i32, u64, u64, vp, vp], i32),
        "zs_step_fused": ([C.POINTER(zs_step_args), vp], i32),
        "zs_scaler_update": ([C.POINTER(zs_loss_scaler), u32], i32),
        "zs_step_commit": ([C.POINTER(zs_step_args), C.POINTER(zs_loss_scaler), vp, vp, vp, vp,
                            C.POINTER(C.c_int)], i32),
        "zs_step_commit_noalloc": ([C.POINTER(zs_step_args), C.POINTER(zs_loss_scaler), vp, vp,
                                    vp, vp, C.POINTER(C.c_int)], i32),
        "zs_all_gather_step": ([C.POINTER(vp), u32, u64, u32, u32, vp], i32),
        "zs_cpu_step": ([vp, vp, vp, vp, u64, C.POINTER(zs_adamw_hparams), vp, i32, i32,
                         C.POINTER(u32)], i32),
        "zs_cpu_update": ([vp, vp, vp, vp, u64, C.POINTER(zs_adamw_hparams), vp, i32, i32], i32),
        "zs_device_scaler_make": ([C.POINTER(zs_loss_scaler), f32, f32,
                                   C.POINTER(zs_device_scaler)], i32),
        "zs_step_device": ([C.POINTER(zs_step_args), vp, vp, vp, vp], i32),
        "zs_mx_quantize": ([vp, i32, u64, u64, u64, i32, i32, vp, vp, vp, i32, vp], i32),
        "zs_mx_matmul_workspace": ([u64, u64, u64], u64),
        "zs_mx_matmul": ([vp, vp, i32, vp, vp, u64, u64, u64, vp, i32, u64, vp, u64, vp], i32),
        "zs_rmsnorm_forward": ([vp, vp, vp, i32, u64, u64, f32, vp, vp, vp, vp, vp, vp], i32),
        "zs_rmsnorm_backward_workspace": ([u64, u64], u64),
        "zs_rmsnorm_backward": ([vp, vp, vp, vp, vp, i32, u64, u64, vp, vp, vp, u64, vp], i32),
        "zs_distill_workspace": ([u64, u64, u32, i32], u64),
        "zs_distill": ([vp, i32, u64, u64, u64, vp, vp, u32, f32, vp, vp, f32, vp, vp, vp, u64,
                        vp, u64, vp], i32),
        "zs_dropout": ([vp, vp, i32, u64, u64, rule, vp, vp], i32),
        "zs_block_norm_forward": ([vp, vp, vp, vp, vp, i32, u64, u64, f32, f32, f32, rule, vp, vp,
                                   vp, vp, vp, vp, vp], i32),
        "zs_block_norm_backward_workspace": ([u64, u64], u64),
        "zs_block_norm_backward": ([vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, u64, u64, f32, f32,
                                    rule, vp, vp, vp, vp, vp, vp, u64, vp], i32),
        "zs_mx_linear": ([vp, vp, i32, vp, vp, u64, u64, u64, vp, i32, vp, u64, vp, vp, i32, u64, vp,
                          u64, vp], i32),
        "zs_activation_backward_workspace": ([u64, u64], u64),
        "zs_activation_backward": ([vp, vp, i32, i32, u64, u64, vp, vp, vp, u64, vp], i32),
        "zs_logprob_workspace": ([u64, u64, i32], u64),
        "zs_logprob": ([vp, i32, u64, u64, u64, vp, f32, vp, vp, u64, vp], i32),
        "zs_policy_workspace": ([u64, u64, i32], u64),
        "zs_policy": ([vp, i32, u64, u64, u64, vp, f32, vp, vp, vp, f32, f32, f32, vp, f32, vp, vp,
                       vp, vp, u64, vp, u64, vp], i32),
        "zs_preference_workspace": ([u64, u64, i32], u64),
        "zs_preference": ([vp, i32, u64, u64, u64, vp, vp, u64, f32, vp, i32, f32, f32, i32, vp,
                           f32, vp, vp, vp, vp, u64, i32, vp, u64, vp], i32),
        "zs_offload_step": ([vp, vp, vp, vp, vp, vp, vp, u64, C.POINTER(zs_adamw_hparams), i32,
                             vp, vp, i32, i32, vp, C.POINTER(C.c_int)], i32),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes, f.restype = args, res
    if lib.zs_abi_version() != ZS_ABI_VERSION:
        raise ImportError("libzeroshard ABI version mismatch")
    return lib


_lib = _load()


# ---- marshalling helpers ----------------------------------------------------

def _torch():
    import torch
    return torch


def _dtype_code(t, explicit):
    if explicit is not None:
        return int(explicit)
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return ZS_BF16
    if t.dtype == torch.float16:
        return ZS_FP16
    raise TypeError(f"16-bit float tensor expected, got {t.dtype}; pass the dtype explicitly")


def _ptr(x, n, elem, what, offset=0):
    """Device address of x after checking it holds offset+n elements of `elem` bytes."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if not x.is_cuda:
        raise ValueError(f"{what}: CUDA tensor expected")
    if not x.is_contiguous():
        raise ValueError(f"{what}: contiguous tensor expected")
    if x.element_size() != elem:
        raise ValueError(f"{what}: {elem}-byte elements expected, got {x.element_size()}")
    if x.numel() < offset + n:
        raise ValueError(f"{what}: needs {offset + n} elements, has {x.numel()}")
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        return C.c_void_p(_torch().cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return C.c_void_p(stream)
    return C.c_void_p(stream.cuda_stream)


def _check(fn, status, detail=None):
    if status != ZS_OK:
        raise ZsError(fn, status, detail if detail is not None else zs_last_error())


# The host update (offload_cpu.cpp) reports status codes only.
_CPU_DETAIL = {
    ZS_ERR_INVALID_ARG: "a null pointer, a bad param dtype, a loss scale that is not finite "
                        "and > 0, step_t == 0, or a hyper-parameter out of range",
    ZS_ERR_UNSUPPORTED: "n exceeds 2^48 elements",
}


def hparams(lr, beta1, beta2, eps, weight_decay, loss_scale, step_t):
    return zs_adamw_hparams(lr, beta1, beta2, eps, weight_decay, loss_scale, step_t)


# ---- entry points -----------------------------------------------------------

def zs_abi_version():
    return _lib.zs_abi_version()


def zs_status_string(status):
    return _lib.zs_status_string(status).decode()


def zs_last_error():
    return _lib.zs_last_error().decode()


def zs_partition(phi, world, rank):
    """Returns (chunk, offset, count)."""
    p, o, c = C.c_uint64(), C.c_uint64(), C.c_uint64()
    _check("zs_partition", _lib.zs_partition(phi, world, rank, C.byref(p), C.byref(o), C.byref(c)))
    return p.value, o.value, c.value


def _grad_array(worker_grads, n):
    ptrs = [_ptr(g, n, 2, f"worker_grads[{k}]") for k, g in enumerate(worker_grads)]
    return (C.c_void_p * len(ptrs))(*ptrs)


def zs_reduce_scatter_avg(worker_grads: Sequence, grad_dtype: Optional[int], world: int,
                          rank: int, n: int, grad_part, accumulate=False,
                          overflow_flag=None, loss_scale=1.0, stream=None,
                          wire_dtype=ZS_WIRE_FP32):
    if len(worker_grads) != world:
        raise ValueError("len(worker_grads) must equal world")
    arr = _grad_array(worker_grads, n)
    dt = _dtype_code(worker_grads[0], grad_dtype) if world else 0
    _check("zs_reduce_scatter_avg", _lib.zs_reduce_scatter_avg(
        arr, dt, wire_dtype, world, rank, n, _ptr(grad_part, n, 4, "grad_part"),
        1 if accumulate else 0, _ptr(overflow_flag, 1, 4, "overflow_flag"), loss_scale,
        _stream(stream)))


def zs_check_overflow(grad_part, n, loss_scale, overflow_flag, stream=None):
    _check("zs_check_overflow", _lib.zs_check_overflow(
        _ptr(grad_part, n, 4, "grad_part"), n, loss_scale,
        _ptr(overflow_flag, 1, 4, "overflow_flag"), _stream(stream)))


def zs_adamw_step(master, m, v, grad_part, n, hp: zs_adamw_hparams, overflow_flag=None,
                  stream=None):
    _check("zs_adamw_step", _lib.zs_adamw_step(
        _ptr(master, n, 4, "master"), _ptr(m, n, 4, "m"), _ptr(v, n, 4, "v"),
        _ptr(grad_part, n, 4, "grad_part"), n, C.byref(hp),
        _ptr(overflow_flag, 1, 4, "overflow_flag"), _stream(stream)))


def zs_cast_gather(master, gather_buf, param_dtype: Optional[int], offset, n,
                   overflow_flag=None, stream=None):
    dt = _dtype_code(gather_buf, param_dtype)
    _check("zs_cast_gather", _lib.zs_cast_gather(
        _ptr(master, n, 4, "master"), _ptr(gather_buf, n, 2, "gather_buf", offset), dt,
        offset, n, _ptr(overflow_flag, 1, 4, "overflow_flag"), _stream(stream)))


class StepArgs:
    """A prepared zs_step_args: built once, re-pointed cheaply between steps
    (swap() exchanges the input and output sets after a committed step)."""

    def __init__(self, worker_grads, rank, n, master_in, m_in, v_in, master_out, m_out, v_out,
                 gather_buf, gather_offset, overflow_flag, hp: zs_adamw_hparams,
                 acc_in=None, grad_dtype=None, param_dtype=None, gather_in=None,
                 wire_dtype=ZS_WIRE_FP32, state_layout=ZS_STATE_SPLIT):
        """state_layout ZS_STATE_GROUPED: master_in / master_out are grouped
        state buffers (grouped_len(n) floats); m_in, v_in, m_out, v_out None."""
        world = len(worker_grads)
        self._grads = _grad_array(worker_grads, n)
        a = zs_step_args()
        a.world, a.rank, a.n = world, rank, n
        a.grad_dtype = _dtype_code(worker_grads[0], grad_dtype)
        a.param_dtype = _dtype_code(gather_buf, param_dtype)
        a.worker_grads = C.cast(self._grads, C.POINTER(C.c_void_p))
        a.acc_in = _ptr(acc_in, n, 4, "acc_in")
        ns = grouped_len(n) if state_layout == ZS_STATE_GROUPED else n
        a.master_in, a.m_in, a.v_in = (_ptr(master_in, ns, 4, "master_in"), _ptr(m_in, n, 4, "m_in"),
                                       _ptr(v_in, n, 4, "v_in"))
        a.master_out, a.m_out, a.v_out = (_ptr(master_out, ns, 4, "master_out"),
                                          _ptr(m_out, n, 4, "m_out"), _ptr(v_out, n, 4, "v_out"))
        a.state_layout = state_layout
        a.gather_buf = _ptr(gather_buf, n, 2, "gather_buf", gather_offset)
        # Optional second gather buffer: with one per set, a skipped step also
        # leaves the current set's 16-bit parameters untouched.
        self._gather_in = _ptr(gather_in, n, 2, "gather_in", gather_offset)
        a.gather_offset = gather_offset
        a.overflow_flag = _ptr(overflow_flag, 1, 4, "overflow_flag")
        a.hp = hp
        a.wire_dtype = wire_dtype
        self.args = a

    def set_grads(self, worker_grads):
        n = self.args.n
        for k, g in enumerate(worker_grads):
            self._grads[k] = _ptr(g, n, 2, f"worker_grads[{k}]")

    def swap(self):
        a = self.args
        a.master_in, a.master_out = a.master_out, a.master_in
        a.m_in, a.m_out = a.m_out, a.m_in
        a.v_in, a.v_out = a.v_out, a.v_in
        if self._gather_in is not None:
            a.gather_buf, self._gather_in = self._gather_in, a.gather_buf


def zs_step_fused(args, stream=None):
    """args: a StepArgs (or a raw zs_step_args)."""
    raw = args.args if isinstance(args, StepArgs) else args
    _check("zs_step_fused", _lib.zs_step_fused(C.byref(raw), _stream(stream)))


def zs_scaler_update(state: zs_loss_scaler, overflow):
    _check("zs_scaler_update", _lib.zs_scaler_update(C.byref(state), 1 if overflow else 0))


def zs_step_commit(args, scaler: zs_loss_scaler, host_flag, stream=None, ev_start=None,
                   ev_stop=None):
    """Fused step + flag readback + scaler update (blocks). host_flag: a
    (pinned) host tensor or address of at least 4 bytes. Returns committed."""
    raw = args.args if isinstance(args, StepArgs) else args
    hf = host_flag if isinstance(host_flag, int) else host_flag.data_ptr()
    committed = C.c_int(0)
    _check("zs_step_commit", _lib.zs_step_commit(C.byref(raw), C.byref(scaler), hf,
                                                 _stream(stream), ev_start, ev_stop,
                                                 C.byref(committed)))
    return bool(committed.value)


def zs_step_commit_noalloc(args, scaler: zs_loss_scaler, host_flag, stream=None, ev_start=None,
                           ev_stop=None):
    """zs_step_commit with the overflow word in the library's own device
    memory (args' overflow_flag is not used). Returns committed."""
    raw = args.args if isinstance(args, StepArgs) else args
    hf = host_flag if isinstance(host_flag, int) else host_flag.data_ptr()
    committed = C.c_int(0)
    _check("zs_step_commit_noalloc",
           _lib.zs_step_commit_noalloc(C.byref(raw), C.byref(scaler), hf, _stream(stream),
                                       ev_start, ev_stop, C.byref(committed)))
    return bool(committed.value)


DEVICE_SCALER_BYTES = C.sizeof(zs_device_scaler)


def zs_device_scaler_make(scaler: zs_loss_scaler, beta1: float, beta2: float) -> zs_device_scaler:
    """Host image of a device-resident scaler continuing from `scaler`."""
    out = zs_device_scaler()
    _check("zs_device_scaler_make", _lib.zs_device_scaler_make(C.byref(scaler), beta1, beta2,
                                                               C.byref(out)))
    return out


def device_scaler_upload(image: zs_device_scaler, device="cuda"):
    """A device buffer (uint8 CUDA tensor) holding `image`."""
    torch = _torch()
    raw = bytes(memoryview(image).cast("B"))
    host = torch.frombuffer(bytearray(raw), dtype=torch.uint8)
    return host.to(device)


def device_scaler_read(dev_buf) -> zs_device_scaler:
    """Host copy of a device scaler buffer. Waits for all work on the
    buffer's device first: steps may be queued on any stream."""
    torch = _torch()
    torch.cuda.synchronize(dev_buf.device)
    raw = dev_buf[:DEVICE_SCALER_BYTES].cpu().numpy().tobytes()
    return zs_device_scaler.from_buffer_copy(raw)


def device_scaler_write(dev_buf, image: zs_device_scaler):
    """Overwrite a device scaler buffer with `image`. Waits for all work on
    the device before and after the copy, so no queued step on any stream
    sees a partly written scaler."""
    torch = _torch()
    raw = bytes(memoryview(image).cast("B"))
    torch.cuda.synchronize(dev_buf.device)
    dev_buf[:DEVICE_SCALER_BYTES].copy_(torch.frombuffer(bytearray(raw), dtype=torch.uint8))
    torch.cuda.synchronize(dev_buf.device)


def _dev_scaler_ptr(dev):
    return _ptr(dev, DEVICE_SCALER_BYTES, 1, "device scaler")


def zs_step_device(args, dev, stream=None, ev_start=None, ev_stop=None):
    """Fused step + on-device commit or skip (never waits). dev: the device
    scaler buffer (device_scaler_upload) or its address."""
    raw = args.args if isinstance(args, StepArgs) else args
    _check("zs_step_device", _lib.zs_step_device(C.byref(raw), _dev_scaler_ptr(dev),
                                                 _stream(stream), ev_start, ev_stop))


def zs_all_gather_step(replicas: Sequence, phi: int, step: int, sigma: int = 0, stream=None):
    """One ring all-gather step over len(replicas) flat 16-bit buffers."""
    ptrs = [_ptr(r, phi, 2, f"replicas[{k}]") for k, r in enumerate(replicas)]
    arr = (C.c_void_p * len(ptrs))(*ptrs)
    _check("zs_all_gather_step", _lib.zs_all_gather_step(arr, len(ptrs), phi, sigma, step,
                                                         _stream(stream)))


def _host_args(fn, master, m, v, grad_part, params16, param_dtype):
    """Pointers and size of host tensors/arrays (torch CPU tensors or numpy
    arrays, contiguous) for the host update entry points."""
    def hptr(x, elem, what):
        if hasattr(x, "data_ptr"):
            if x.is_cuda or not x.is_contiguous() or x.element_size() != elem:
                raise ValueError(f"{what}: contiguous host tensor of {elem}-byte elements expected")
            return x.data_ptr(), x.numel()
        if not x.flags.c_contiguous or x.itemsize != elem:
            raise ValueError(f"{what}: contiguous array of {elem}-byte elements expected")
        return x.ctypes.data, x.size
    (pm, n), (p1, n1), (p2, n2), (pg, n3) = (hptr(master, 4, "master"), hptr(m, 4, "m"),
                                              hptr(v, 4, "v"), hptr(grad_part, 4, "grad_part"))
    pp, n4 = hptr(params16, 2, "params16")
    if not (n == n1 == n2 == n3 <= n4):
        raise ValueError(f"{fn}: size mismatch")
    if param_dtype is None:
        param_dtype = _dtype_code(params16, None) if hasattr(params16, "dtype") and \
            str(params16.dtype).startswith("torch") else ZS_BF16
    return pm, p1, p2, pg, n, pp, param_dtype


def zs_cpu_step(master, m, v, grad_part, hp: zs_adamw_hparams, params16, param_dtype=None,
                threads=0):
    """ZeRO-Offload update on host memory. Returns the overflow flag (1: skipped)."""
    pm, p1, p2, pg, n, pp, dt = _host_args("zs_cpu_step", master, m, v, grad_part, params16,
                                           param_dtype)
    flag = C.c_uint32(0)
    rc = _lib.zs_cpu_step(pm, p1, p2, pg, n, C.byref(hp), pp, dt, threads, C.byref(flag))
    _check("zs_cpu_step", rc, _CPU_DETAIL.get(rc, ""))
    return int(flag.value)


def zs_cpu_update(master, m, v, grad_part, hp: zs_adamw_hparams, params16, param_dtype=None,
                  threads=0):
    """zs_cpu_step without its check (the caller has checked the gradient)."""
    pm, p1, p2, pg, n, pp, dt = _host_args("zs_cpu_update", master, m, v, grad_part, params16,
                                           param_dtype)
    rc = _lib.zs_cpu_update(pm, p1, p2, pg, n, C.byref(hp), pp, dt, threads)
    _check("zs_cpu_update", rc, _CPU_DETAIL.get(rc, ""))


def _host_ptr(x, n, elem, what):
    """Address of a contiguous host (CPU) tensor or array of >= n elements of
    `elem` bytes."""
    if hasattr(x, "data_ptr"):
        if x.is_cuda or not x.is_contiguous() or x.element_size() != elem or x.numel() < n:
            raise ValueError(f"{what}: contiguous host tensor of >= {n} {elem}-byte elements "
                             "expected")
        return x.data_ptr()
    if not x.flags.c_contiguous or x.itemsize != elem or x.size < n:
        raise ValueError(f"{what}: contiguous array of >= {n} {elem}-byte elements expected")
    return x.ctypes.data


def zs_offload_step(grad_dev, grad_host, master, m, v, params_host, params_dev,
                    hp: zs_adamw_hparams, flag_dev, flag_host, param_dtype=None, threads=0,
                    pieces=16, stream=None):
    """Pipelined ZeRO-Offload step (blocks until the host update is done).
    grad_dev, params_dev, flag_dev: CUDA tensors; grad_host, master, m, v,
    params_host, flag_host: host tensors (the staging ones pinned). n is
    master's length. Returns True when committed, False when skipped."""
    n = master.numel() if hasattr(master, "numel") else master.size
    if param_dtype is None:
        param_dtype = _dtype_code(params_dev, None)
    committed = C.c_int(0)
    rc = _lib.zs_offload_step(
        _ptr(grad_dev, n, 4, "grad_dev"), _host_ptr(grad_host, n, 4, "grad_host"),
        _host_ptr(master, n, 4, "master"), _host_ptr(m, n, 4, "m"), _host_ptr(v, n, 4, "v"),
        _host_ptr(params_host, n, 2, "params_host"), _ptr(params_dev, n, 2, "params_dev"), n,
        C.byref(hp), param_dtype, _ptr(flag_dev, 1, 4, "flag_dev"),
        _host_ptr(flag_host, 1, 4, "flag_host"), threads, pieces, _stream(stream),
        C.byref(committed))
    _check("zs_offload_step", rc)
    return bool(committed.value)


# ---- operators of a low-precision model's output end --------------------------

class _Torch:
    """torch's names that every call looks up, found once."""

    def __init__(self):
        import torch
        self.u8, self.i32, self.f32 = torch.uint8, torch.int32, torch.float32
        self.codes = {torch.bfloat16: ZS_BF16, torch.float16: ZS_FP16}
        self.codes32 = {**self.codes, torch.float32: ZS_FP32}
        try:    # the current stream's handle without an object around it
            raw, device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
            self.stream, self.device = lambda: raw(device()), device
        except AttributeError:
            self.device = torch.cuda.current_device
            self.stream = lambda: torch.cuda.current_stream().cuda_stream
        if not torch.cuda.is_available():   # then no tensor is on it
            self.device = lambda: 0


_names = None


def _t():
    global _names
    if _names is None:
        _names = _Torch()
    return _names


def _raw_stream(stream):
    if stream is None:
        return _t().stream()
    return stream if isinstance(stream, int) else stream.cuda_stream


def _here(stream, *tensors):
    """The stream's handle, where all tensors are on the current device: the kernels run there."""
    device = _t().device()
    for x in tensors:
        if x is not None and x.get_device() != device:
            raise ValueError(f"tensor on {x.device}, but the current device is {device}")
    if stream is None:
        return _t().stream()
    if getattr(stream, "device_index", device) != device:
        raise ValueError(f"stream of device {stream.device_index}, but the current is {device}")
    return _raw_stream(stream)


def _float_code(t, what, fp32=False):
    """zs_dtype of a tensor's element type."""
    code = (_t().codes32 if fp32 else _t().codes).get(t.dtype)
    if code is None:
        raise TypeError(f"{what}: {'float32, ' if fp32 else ''}bfloat16 or float16 tensor "
                        f"expected, got {t.dtype}")
    return code


def _where(x, device):
    return x.device if device is None else f"{x.device}, the current device is {device}"


def _rows(x, what, shape=None, device=None):
    """(address, rows, cols, row stride) of a 2-D CUDA tensor with contiguous rows; with
    `device`, on that one."""
    if not x.is_cuda if device is None else x.get_device() != device:
        raise ValueError(f"{what}: CUDA tensor expected, got one on {_where(x, device)}")
    if x.dim() != 2 or (shape is not None and x.shape != shape):
        raise ValueError(f"{what}: {'2-D' if shape is None else shape} tensor expected, "
                         f"got {tuple(x.shape)}")
    r, c = x.shape
    if x.is_contiguous():
        return x.data_ptr(), r, c, c
    ld = x.stride(0) if r > 1 else c
    if (c > 1 and x.stride(1) != 1) or ld < c:
        raise ValueError(f"{what}: rows must be contiguous and must not overlap")
    return x.data_ptr(), r, c, ld


def _dense(x, shape, dtype, what, device=None):
    """Address of a contiguous CUDA tensor of that shape and type (None stays None); with
    `device`, on that one."""
    if x is None:
        return None
    if (x.shape != shape or x.dtype is not dtype or not x.is_contiguous()
            or (not x.is_cuda if device is None else x.get_device() != device)):
        raise ValueError(f"{what}: contiguous {dtype} CUDA tensor of shape {tuple(shape)} "
                         f"expected, got {x.dtype} {tuple(x.shape)} on {_where(x, device)}")
    return x.data_ptr()


def _workspace(x, device=None):
    if x is None:
        return None, 0
    if (not x.is_contiguous()
            or (not x.is_cuda if device is None else x.get_device() != device)):
        raise ValueError(f"workspace: contiguous CUDA tensor expected, got one on "
                         f"{_where(x, device)}")
    return x.data_ptr(), x.nbytes


def mx_padded(k):
    """Elements of a microscaled row of k elements: whole groups."""
    return -(-k // ZS_MX_GROUP) * ZS_MX_GROUP


def mx_shapes(rows, k, fmt):
    """Shapes of the codes and scales (both uint8) of `rows` microscaled rows of k elements."""
    p = mx_padded(k)
    return (rows, p // 2 if fmt == ZS_MX_E2M1 else p), (rows, p // ZS_MX_BLOCK)


def mx_empty(rows, k, fmt, device="cuda"):
    """Uninitialised codes and scales for `rows` microscaled rows of k elements."""
    torch = _torch()
    return tuple(torch.empty(s, dtype=torch.uint8, device=device)
                 for s in mx_shapes(rows, k, fmt))


def _mx_ptrs(codes, scales, rows, k, fmt, what, device=None):
    cs, ss = mx_shapes(rows, k, fmt)
    u8 = _t().u8
    return (_dense(codes, cs, u8, f"{what} codes", device),
            _dense(scales, ss, u8, f"{what} scales", device))


def zs_mx_quantize(src, fmt, codes, scales, columns=False, values=None, stream=None):
    """Microscaled copy of the 2-D tensor src, along its rows or its columns
    (codes and scales: mx_empty of src's rows, or columns, by the other)."""
    p, r, c, ld = _rows(src, "src")
    cp, sp = _mx_ptrs(codes, scales, c if columns else r, r if columns else c, fmt, "mx")
    vp, vdt = None, ZS_BF16
    if values is not None:
        vdt = _float_code(values, "values")
        vp = _dense(values, (r, c), values.dtype, "values")
    _check("zs_mx_quantize", _lib.zs_mx_quantize(
        p, _float_code(src, "src", fp32=True), r, c, ld, fmt, 1 if columns else 0, cp, sp, vp,
        vdt, _raw_stream(stream)))


def zs_mx_matmul_workspace(m, n, k):
    """Bytes of workspace with which zs_mx_matmul splits k as far as it would."""
    return _lib.zs_mx_matmul_workspace(m, n, k)


def zs_mx_matmul(a_codes, a_scales, a_format, b_codes, b_scales, out, k, workspace=None,
                 stream=None):
    """out[m][n] = A B^T: A m microscaled rows of k elements in a_format, B n in ZS_MX_E2M1."""
    p, m, n, ld = _rows(out, "out")
    ac, asc = _mx_ptrs(a_codes, a_scales, m, k, a_format, "A")
    bc, bsc = _mx_ptrs(b_codes, b_scales, n, k, ZS_MX_E2M1, "B")
    wp, wb = _workspace(workspace)
    _check("zs_mx_matmul", _lib.zs_mx_matmul(
        ac, asc, a_format, bc, bsc, m, n, k, p, _float_code(out, "out", fp32=True), ld, wp, wb,
        _raw_stream(stream)))


def zs_rmsnorm_forward(x, gain, eps, h=None, rstd=None, residual=None, codes=None, scales=None,
                       y=None, stream=None):
    """Norm of x (+ residual, the sum going to h) into 8-bit microscaled rows
    (codes, scales) and / or a 16-bit y."""
    if x.dim() != 2:
        raise ValueError("x: 2-D tensor expected")
    shape, dt = x.shape, x.dtype
    cp = sp = None
    if codes is not None or scales is not None:
        if codes is None or scales is None:
            raise ValueError("codes and scales go together")
        cp, sp = _mx_ptrs(codes, scales, *shape, ZS_MX_E4M3, "y")
    _check("zs_rmsnorm_forward", _lib.zs_rmsnorm_forward(
        _dense(x, shape, dt, "x"), _dense(residual, shape, dt, "residual"),
        _dense(gain, shape[1:], dt, "gain"), _float_code(x, "x"), *shape, eps,
        _dense(h, shape, dt, "h"), _dense(rstd, shape[:1], _t().f32, "rstd"), cp, sp,
        _dense(y, shape, dt, "y"), _raw_stream(stream)))


def zs_rmsnorm_backward_workspace(rows, cols):
    """Bytes of workspace that zs_rmsnorm_backward needs."""
    return _lib.zs_rmsnorm_backward_workspace(rows, cols)


def zs_rmsnorm_backward(dy, h, rstd, gain, dx, dgain, workspace, dres=None, stream=None):
    """Gradients of zs_rmsnorm_forward: dx (of x and of the residual alike) and the fp32 dgain."""
    if dy.dim() != 2:
        raise ValueError("dy: 2-D tensor expected")
    shape, dt, f32 = dy.shape, dy.dtype, _t().f32
    wp, wb = _workspace(workspace)
    _check("zs_rmsnorm_backward", _lib.zs_rmsnorm_backward(
        _dense(dy, shape, dt, "dy"), _dense(h, shape, dt, "h"),
        _dense(rstd, shape[:1], f32, "rstd"), _dense(gain, shape[1:], dt, "gain"),
        _dense(dres, shape, dt, "dres"), _float_code(dy, "dy"), *shape,
        _dense(dx, shape, dt, "dx"), _dense(dgain, shape[1:], f32, "dgain"), wp, wb,
        _raw_stream(stream)))


def zs_distill_workspace(rows, vocab, slots, dtype):
    """Bytes of workspace that zs_distill needs; dtype: the logits' zs_dtype."""
    return _lib.zs_distill_workspace(rows, vocab, slots, dtype)


def zs_distill(logits, ids, teacher, temperature, loss, grad=None, teacher_lse=None,
               row_weight=None, loss_scale=1.0, dev_scaler=None, workspace=None, stream=None):
    """Loss per row against a teacher's top logits and, with grad, the logits'
    gradient times the loss scale (loss_scale, or dev_scaler's: the buffer of
    device_scaler_upload). grad may be logits itself."""
    p, rows, vocab, ld = _rows(logits, "logits")
    names = _t()
    f32 = names.f32
    slots = ids.shape[1] if ids.dim() == 2 else -1
    gp, gld = None, 0
    if grad is not None:
        if grad.dtype != logits.dtype:
            raise ValueError("grad: the logits' dtype expected")
        gp, _, _, gld = _rows(grad, "grad", (rows, vocab))
    wp, wb = _workspace(workspace)
    _check("zs_distill", _lib.zs_distill(
        p, _float_code(logits, "logits", fp32=True), rows, vocab, ld,
        _dense(ids, (rows, slots), names.i32, "ids"),
        _dense(teacher, (rows, slots), logits.dtype, "teacher"), slots, temperature,
        _dense(teacher_lse, (rows,), f32, "teacher_lse"),
        _dense(row_weight, (rows,), f32, "row_weight"), loss_scale,
        None if dev_scaler is None else _dev_scaler_ptr(dev_scaler),
        _dense(loss, (rows,), f32, "loss"), gp, gld, wp, wb, _raw_stream(stream)))


# ---- operators of the student's last block ------------------------------------

def _rule(dropout):
    """A zs_dropout_rule from (p, seed, offset) or (p, seed, offset, dev_offset), the last a
    CUDA int64 tensor of one element; None stays None."""
    if dropout is None or isinstance(dropout, zs_dropout_rule):
        return dropout
    p, seed, offset, *more = dropout
    dev = more[0] if more else None
    if dev is not None and (not dev.is_cuda or dev.element_size() != 8 or dev.numel() != 1):
        raise ValueError("dev_offset: CUDA tensor of one 64-bit element expected")
    if dev is not None:
        _here(0, dev)
    mask = (1 << 64) - 1
    return zs_dropout_rule(p, seed & mask, offset & mask, None if dev is None else dev.data_ptr())


def zs_dropout(x, out, rule, residual=None, stream=None):
    """out = residual + dropout(x) of a 2-D tensor; rule: (p, seed, offset[, dev_offset]).
    out may be x or residual."""
    if x.dim() != 2:
        raise ValueError("x: 2-D tensor expected")
    shape, dt, here = x.shape, x.dtype, _t().device()
    _check("zs_dropout", _lib.zs_dropout(
        _dense(x, shape, dt, "x", here), _dense(residual, shape, dt, "residual", here),
        _float_code(x, "x", fp32=True), *shape, _rule(rule), _dense(out, shape, dt, "out", here),
        _here(stream)))


def zs_block_norm_forward(x, residual, gain, eps, h, rstd=None, post_gain=None, post_rstd=None,
                          gate=None, residual_scale=1.0, branch_scale=1.0, dropout=None,
                          codes=None, scales=None, y=None, stream=None):
    """h = residual_scale * residual + branch_scale * dropout(gate * norm(x)), then h's norm
    into 8-bit microscaled rows (codes, scales) and / or a 16-bit y. Without post_gain x is
    taken as it is, without gate the gate is 1; dropout: (p, seed, offset[, dev_offset])."""
    if x.dim() != 2:
        raise ValueError("x: 2-D tensor expected")
    names = _t()
    shape, dt, f32, here = x.shape, x.dtype, names.f32, names.device()
    row, col = shape[:1], shape[1:]
    cp = sp = None
    if codes is not None or scales is not None:
        if codes is None or scales is None:
            raise ValueError("codes and scales go together")
        cp, sp = _mx_ptrs(codes, scales, *shape, ZS_MX_E4M3, "y", here)
    _check("zs_block_norm_forward", _lib.zs_block_norm_forward(
        _dense(x, shape, dt, "x", here), _dense(residual, shape, dt, "residual", here),
        _dense(post_gain, col, dt, "post_gain", here), _dense(gate, col, dt, "gate", here),
        _dense(gain, col, dt, "gain", here), _float_code(x, "x"), *shape, eps, residual_scale,
        branch_scale, _rule(dropout), _dense(h, shape, dt, "h", here),
        _dense(post_rstd, row, f32, "post_rstd", here), _dense(rstd, row, f32, "rstd", here), cp,
        sp, _dense(y, shape, dt, "y", here), _here(stream)))


def zs_block_norm_backward_workspace(rows, cols):
    """Bytes of workspace that zs_block_norm_backward needs."""
    return _lib.zs_block_norm_backward_workspace(rows, cols)


def zs_block_norm_backward(dy, h, rstd, gain, dx, dresidual, dgain, workspace, x=None,
                           post_gain=None, post_rstd=None, gate=None, dpost_gain=None, dgate=None,
                           dres=None, residual_scale=1.0, branch_scale=1.0, dropout=None,
                           stream=None):
    """Gradients of zs_block_norm_forward: dx and dresidual (16 bits) and the fp32 dgain,
    dpost_gain and dgate. dres: what h receives from elsewhere."""
    if dy.dim() != 2:
        raise ValueError("dy: 2-D tensor expected")
    names = _t()
    shape, dt, f32, here = dy.shape, dy.dtype, names.f32, names.device()
    row, col = shape[:1], shape[1:]
    wp, wb = _workspace(workspace, here)
    _check("zs_block_norm_backward", _lib.zs_block_norm_backward(
        _dense(dy, shape, dt, "dy", here), _dense(h, shape, dt, "h", here),
        _dense(rstd, row, f32, "rstd", here), _dense(gain, col, dt, "gain", here),
        _dense(dres, shape, dt, "dres", here), _dense(x, shape, dt, "x", here),
        _dense(post_rstd, row, f32, "post_rstd", here),
        _dense(post_gain, col, dt, "post_gain", here), _dense(gate, col, dt, "gate", here),
        _float_code(dy, "dy"), *shape, residual_scale, branch_scale, _rule(dropout),
        _dense(dx, shape, dt, "dx", here), _dense(dresidual, shape, dt, "dresidual", here),
        _dense(dgain, col, f32, "dgain", here), _dense(dpost_gain, col, f32, "dpost_gain", here),
        _dense(dgate, col, f32, "dgate", here), wp, wb, _here(stream)))


def zs_mx_linear(a_codes, a_scales, a_format, b_codes, b_scales, out, k, bias=None,
                 activation=ZS_ACT_NONE, residual=None, pre=None, workspace=None, stream=None):
    """out[m][n] = residual + act(A B^T + bias): A m microscaled rows of k elements in a_format,
    B n in ZS_MX_E2M1. pre: what the activation is applied to, 16 bits. out may be residual."""
    here = _t().device()
    p, m, n, ld = _rows(out, "out", device=here)
    dt = out.dtype
    ac, asc = _mx_ptrs(a_codes, a_scales, m, k, a_format, "A", here)
    bc, bsc = _mx_ptrs(b_codes, b_scales, n, k, ZS_MX_E2M1, "B", here)
    rp, rld = None, 0
    if residual is not None:
        if residual.dtype != dt:
            raise ValueError("residual: out's dtype expected")
        rp, _, _, rld = _rows(residual, "residual", (m, n), here)
    wp, wb = _workspace(workspace, here)
    _check("zs_mx_linear", _lib.zs_mx_linear(
        ac, asc, a_format, bc, bsc, m, n, k, _dense(bias, (n,), dt, "bias", here), activation, rp,
        rld, _dense(pre, (m, n), dt, "pre", here), p, _float_code(out, "out"), ld, wp, wb,
        _here(stream)))


def zs_activation_backward_workspace(rows, cols):
    """Bytes of workspace that zs_activation_backward needs for dbias."""
    return _lib.zs_activation_backward_workspace(rows, cols)


def zs_activation_backward(dout, pre, activation, dpre=None, dbias=None, workspace=None,
                           stream=None):
    """dpre = dout * act'(pre) and its sum over the rows, the fp32 dbias; pre: zs_mx_linear's
    (None without an activation). dpre may be dout or pre."""
    if dout.dim() != 2:
        raise ValueError("dout: 2-D tensor expected")
    shape, dt, here = dout.shape, dout.dtype, _t().device()
    wp, wb = _workspace(workspace, here)
    _check("zs_activation_backward", _lib.zs_activation_backward(
        _dense(dout, shape, dt, "dout", here), _dense(pre, shape, dt, "pre", here), activation,
        _float_code(dout, "dout"), *shape, _dense(dpre, shape, dt, "dpre", here),
        _dense(dbias, shape[1:], _t().f32, "dbias", here), wp, wb, _here(stream)))


# ---- losses on the log-probabilities of given tokens ---------------------------

def _scaler(dev):
    """Address of a device scaler on the current device (None stays None)."""
    if dev is not None and not isinstance(dev, int):
        _here(0, dev)
    return None if dev is None else _dev_scaler_ptr(dev)


def _grad_rows(grad, logits, rows, vocab, here=None):
    """(address, row stride) of a gradient of the logits' shape and type; (None, 0) without."""
    if grad is None:
        return None, 0
    if grad.dtype != logits.dtype:
        raise ValueError("grad: the logits' dtype expected")
    gp, _, _, gld = _rows(grad, "grad", (rows, vocab), here)
    return gp, gld


def zs_logprob_workspace(rows, vocab, dtype):
    """Bytes of workspace that zs_logprob needs; dtype: the logits' zs_dtype."""
    return _lib.zs_logprob_workspace(rows, vocab, dtype)


def zs_logprob(logits, ids, logp, temperature=1.0, workspace=None, stream=None):
    """Log-probability of each row's token ids[row] (0 where that is no token)."""
    names = _t()
    here = names.device()
    p, rows, vocab, ld = _rows(logits, "logits", device=here)
    wp, wb = _workspace(workspace, here)
    _check("zs_logprob", _lib.zs_logprob(
        p, _float_code(logits, "logits", fp32=True), rows, vocab, ld,
        _dense(ids, (rows,), names.i32, "ids", here), temperature,
        _dense(logp, (rows,), names.f32, "logp", here), wp, wb, _here(stream)))


def zs_policy_workspace(rows, vocab, dtype):
    """Bytes of workspace that zs_policy needs; dtype: the logits' zs_dtype."""
    return _lib.zs_policy_workspace(rows, vocab, dtype)


def zs_policy(logits, ids, advantage, loss, temperature=1.0, old_logp=None, ref_logp=None,
              clip_low=0.2, clip_high=0.2, kl_weight=0.0, row_weight=None, loss_scale=1.0,
              dev_scaler=None, logp=None, grad=None, workspace=None, stream=None):
    """Clipped policy loss per row and, with grad, the logits' gradient times the loss scale
    (loss_scale, or dev_scaler's). grad may be logits itself."""
    names = _t()
    f32, here = names.f32, names.device()
    p, rows, vocab, ld = _rows(logits, "logits", device=here)
    gp, gld = _grad_rows(grad, logits, rows, vocab, here)
    wp, wb = _workspace(workspace, here)
    each = (rows,)
    _check("zs_policy", _lib.zs_policy(
        p, _float_code(logits, "logits", fp32=True), rows, vocab, ld,
        _dense(ids, each, names.i32, "ids", here), temperature,
        _dense(advantage, each, f32, "advantage", here),
        _dense(old_logp, each, f32, "old_logp", here),
        _dense(ref_logp, each, f32, "ref_logp", here), clip_low, clip_high, kl_weight,
        _dense(row_weight, each, f32, "row_weight", here), loss_scale, _scaler(dev_scaler),
        _dense(logp, each, f32, "logp", here), _dense(loss, each, f32, "loss", here), gp, gld, wp,
        wb, _here(stream)))


def zs_preference_workspace(rows, vocab, dtype):
    """Bytes of workspace that zs_preference needs; dtype: the logits' zs_dtype."""
    return _lib.zs_preference_workspace(rows, vocab, dtype)


def zs_preference(logits, ids, starts, beta, loss, kind=ZS_PREFERENCE_SIGMOID, smoothing=0.0,
                  mean=False, temperature=1.0, ref_logp=None, pair_weight=None, loss_scale=1.0,
                  dev_scaler=None, seq_logp=None, grad=None, clear=False, workspace=None,
                  stream=None):
    """Preference loss per pair of sequences (rows starts[s] to starts[s + 1] of logits and ids;
    pair p prefers sequence 2p) and, with grad, the logits' gradient times the loss scale. grad
    may be logits itself; its rows outside all sequences are left as they were, or with clear
    filled with zeros."""
    names = _t()
    f32, i32, here = names.f32, names.i32, names.device()
    p, rows, vocab, ld = _rows(logits, "logits", device=here)
    pairs = loss.shape[0] if loss.dim() == 1 else -1
    gp, gld = _grad_rows(grad, logits, rows, vocab, here)
    wp, wb = _workspace(workspace, here)
    each, sequences = (pairs,), (2 * pairs,)
    _check("zs_preference", _lib.zs_preference(
        p, _float_code(logits, "logits", fp32=True), rows, vocab, ld,
        _dense(ids, (rows,), i32, "ids", here),
        _dense(starts, (2 * pairs + 1,), i32, "starts", here), pairs, temperature,
        _dense(ref_logp, sequences, f32, "ref_logp", here), kind, beta, smoothing,
        1 if mean else 0, _dense(pair_weight, each, f32, "pair_weight", here), loss_scale,
        _scaler(dev_scaler), _dense(seq_logp, sequences, f32, "seq_logp", here),
        _dense(loss, each, f32, "loss", here), gp, gld, 1 if clear else 0, wp, wb,
        _here(stream)))
