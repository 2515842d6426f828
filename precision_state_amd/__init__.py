"""Python binding of libps.so, the MI355X fused low-precision optimizer step.

Argument marshalling only: every function takes torch tensors that live in
device memory, passes their pointers and the current HIP stream to the C ABI
declared in include/ps.h, and raises PSError on a non-zero status. No step
of the computation runs in Python or PyTorch; if libps.so is missing the
import fails.

16-bit arrays (bf16 weights and gradients, residuals, moment codes) may be any
2-byte dtype (torch.int16, torch.uint16, torch.bfloat16): only their bits
matter. Scale and EMA arrays are torch.float32.
"""
import ctypes
import os
from dataclasses import dataclass
from typing import Optional, Sequence

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libps.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() (hipcc, gfx950)")

# libps.so needs libamdhip64.so.7. PyTorch ships a HIP runtime of its own:
# with torch loaded first the library binds to that one, and the process has a
# single HIP runtime whose device pointers and streams both sides share.
# Loaded first, the library would map the system runtime and torch its own
# afterwards: two runtimes on one GPU, each unable to use the other's memory
# and streams. So torch is imported before the library whenever it exists.
try:
    import torch  # noqa: F401
except ImportError:
    torch = None

_lib = ctypes.CDLL(LIB_PATH)

ALGO_ADAM, ALGO_NADAM = 0, 1
SPLIT_TRUNC, SPLIT_NEAREST_AWAY, SPLIT_STOCHASTIC = 0, 1, 2
MOMENT_SIGNED, MOMENT_UNSIGNED = 0, 1
TENSOR_FP32_MOMENTS, TENSOR_FP32_PARAM, TENSOR_F24_MOMENTS = 1, 2, 4
BLOCK = 256
TYPE_F32, TYPE_BF16, TYPE_F16 = 0, 1, 2
STATE_F32, STATE_E4M3 = 0, 1
ROUND_NEAREST, ROUND_STOCHASTIC = 0, 1
ADAMW_MAX_GROUPS = 16

STATUS = {0: "PS_OK", 1: "PS_ERR_INVALID_ARG", 2: "PS_ERR_ALIGNMENT", 3: "PS_ERR_SHAPE",
          4: "PS_ERR_UNSUPPORTED", 5: "PS_ERR_HIP", 6: "PS_ERR_NO_MEMORY", 7: "PS_ERR_WORKSPACE"}

EXPORTED = ["ps_opt_step_multi", "ps_step_scalars", "ps_split", "ps_join", "ps_encode_moments",
            "ps_decode_moments", "ps_factored_workspace_size", "ps_factored_step", "ps_factored_step_noalloc",
            "ps_adamw_workspace_size", "ps_adamw_plan_create", "ps_adamw_set_grads", "ps_adamw_grad_norm",
            "ps_adamw_step", "ps_adamw_plan_destroy", "ps_encode_fp8", "ps_decode_fp8",
            "ps_offload_plan_create", "ps_offload_plan_create_ex",
            "ps_offload_run", "ps_offload_bytes", "ps_offload_plan_destroy", "ps_status_string",
            "ps_last_error", "ps_version"]


class PSError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


class CTensor(ctypes.Structure):
    _fields_ = [("w_hi", ctypes.c_void_p), ("w_lo", ctypes.c_void_p), ("grad", ctypes.c_void_p),
                ("m_code", ctypes.c_void_p), ("m_scale", ctypes.c_void_p), ("v_code", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("row_ema", ctypes.c_void_p), ("col_ema", ctypes.c_void_p),
                ("numel", ctypes.c_int64), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("flags", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


class CHParams(ctypes.Structure):
    _fields_ = [("algo", ctypes.c_int32), ("split_mode", ctypes.c_int32), ("lr", ctypes.c_double),
                ("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("eps", ctypes.c_double),
                ("weight_decay", ctypes.c_double), ("momentum_decay", ctypes.c_double), ("seed", ctypes.c_uint64)]


class CFHParams(ctypes.Structure):
    _fields_ = [("split_mode", ctypes.c_int32), ("reserved", ctypes.c_int32), ("lr", ctypes.c_double),
                ("beta2", ctypes.c_double), ("eps1", ctypes.c_double), ("clip_threshold", ctypes.c_double),
                ("weight_decay", ctypes.c_double), ("decay_rate", ctypes.c_double), ("beta1", ctypes.c_double),
                ("seed", ctypes.c_uint64)]


class CAdamWTensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("copy", ctypes.c_void_p),
                ("grad", ctypes.c_void_p), ("m", ctypes.c_void_p), ("m_scale", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("numel", ctypes.c_int64),
                ("param_type", ctypes.c_int32), ("grad_type", ctypes.c_int32), ("copy_type", ctypes.c_int32),
                ("state_type", ctypes.c_int32), ("group", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class CAdamWControl(ctypes.Structure):
    _fields_ = [("norm", ctypes.c_float), ("grad_mul", ctypes.c_float), ("skip", ctypes.c_uint32),
                ("skipped", ctypes.c_uint32), ("step", ctypes.c_int64), ("lr_mul", ctypes.c_float),
                ("reserved", ctypes.c_uint32 * 9)]


class COffloadGroup(ctypes.Structure):
    _fields_ = [("tensors", ctypes.POINTER(CTensor)), ("n_tensors", ctypes.c_int32)]


class COffloadOptions(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int32), ("n_cus", ctypes.c_int32), ("reserved0", ctypes.c_int32),
                ("reserved1", ctypes.c_int32)]


OFFLOAD_DIRECT, OFFLOAD_STAGED = 0, 1
OFFLOAD_DEFAULT_CUS = 8


_vp, _i64, _i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
_f64 = ctypes.c_double
_sig = {
    "ps_opt_step_multi": [ctypes.POINTER(CTensor), _i32, ctypes.POINTER(CHParams), _i64, _vp],
    "ps_step_scalars": [ctypes.POINTER(CHParams), _i64, ctypes.POINTER(ctypes.c_float)],
    "ps_split": [_vp, _vp, _vp, _i64, _i32, _vp],
    "ps_join": [_vp, _vp, _vp, _i64, _i32, _vp],
    "ps_encode_moments": [_vp, _vp, _vp, _i64, _i32, _vp],
    "ps_decode_moments": [_vp, _vp, _vp, _i64, _i32, _vp],
    "ps_factored_workspace_size": [ctypes.POINTER(CTensor), _i32, ctypes.POINTER(ctypes.c_size_t)],
    "ps_factored_step": [ctypes.POINTER(CTensor), _i32, ctypes.POINTER(CFHParams), _i64, _vp, ctypes.c_size_t, _vp],
    "ps_factored_step_noalloc": [ctypes.POINTER(CTensor), _i32, ctypes.POINTER(CFHParams), _i64, _vp],
    "ps_adamw_workspace_size": [ctypes.POINTER(CAdamWTensor), _i32, ctypes.POINTER(ctypes.c_size_t)],
    "ps_adamw_plan_create": [ctypes.POINTER(CAdamWTensor), _i32, _vp, ctypes.c_size_t, _vp, ctypes.POINTER(_vp)],
    "ps_adamw_set_grads": [_vp, ctypes.POINTER(_vp), _i32, _vp],
    "ps_adamw_grad_norm": [_vp, _f64, _f64, _vp],
    "ps_adamw_step": [_vp, ctypes.POINTER(CHParams), _i32, _i64, _i32, _i32, _vp],
    "ps_adamw_plan_destroy": [_vp],
    "ps_encode_fp8": [_vp, _vp, _vp, _i64, _i32, _vp],
    "ps_decode_fp8": [_vp, _vp, _vp, _i64, _i32, _vp],
    "ps_offload_plan_create": [ctypes.POINTER(COffloadGroup), _i32, ctypes.POINTER(ctypes.c_void_p)],
    "ps_offload_plan_create_ex": [ctypes.POINTER(COffloadGroup), _i32, ctypes.POINTER(COffloadOptions),
                                  ctypes.POINTER(ctypes.c_void_p)],
    "ps_offload_run": [_vp, ctypes.POINTER(CHParams), _i64, _vp],
    "ps_offload_bytes": [_vp, ctypes.POINTER(ctypes.c_uint64), ctypes.POINTER(ctypes.c_uint64)],
    "ps_offload_plan_destroy": [_vp],
}
for _name, _args in _sig.items():
    _f = getattr(_lib, _name)
    _f.argtypes = _args
    _f.restype = ctypes.c_int32
_lib.ps_status_string.argtypes = [ctypes.c_int32]
_lib.ps_status_string.restype = ctypes.c_char_p
_lib.ps_last_error.argtypes = []
_lib.ps_last_error.restype = ctypes.c_char_p
_lib.ps_version.argtypes = []
_lib.ps_version.restype = ctypes.c_char_p


def lib():
    return _lib


def version():
    return _lib.ps_version().decode()


def last_error():
    return _lib.ps_last_error().decode()


def _check(status):
    if status != 0:
        raise PSError(status, last_error())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is not None:
        return ctypes.c_void_p(stream if isinstance(stream, int) else stream.cuda_stream)
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


# The device's current stream as an integer (without the Stream object, whose making takes 2 us).
_current_raw_stream = getattr(getattr(torch, "_C", None), "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


@dataclass
class HParams:
    algo: int = ALGO_NADAM
    split_mode: int = SPLIT_TRUNC
    lr: float = 3.5e-6
    beta1: float = 0.9
    beta2: float = 0.999
    eps: float = 1e-8
    weight_decay: float = 0.0
    momentum_decay: float = 4e-3
    seed: int = 0          # SPLIT_STOCHASTIC: the random stream's seed (see ps_hparams in include/ps.h)

    def c(self):
        return CHParams(self.algo, self.split_mode, self.lr, self.beta1, self.beta2, self.eps,
                        self.weight_decay, self.momentum_decay, self.seed)


@dataclass
class FactoredHParams:
    split_mode: int = SPLIT_TRUNC
    lr: float = 3.5e-6
    beta2: float = 0.999
    eps1: float = 1e-30
    clip_threshold: float = 1.0
    weight_decay: float = 0.0
    decay_rate: float = 0.0   # < 0: beta2 of update t is 1 - t^decay_rate (Adafactor's schedule)
    beta1: float = 0.0        # > 0: first moment of the clipped update in m_code / m_scale
    seed: int = 0             # SPLIT_STOCHASTIC: the random stream's seed

    def c(self):
        return CFHParams(self.split_mode, 0, self.lr, self.beta2, self.eps1, self.clip_threshold,
                         self.weight_decay, self.decay_rate, self.beta1, self.seed)


@dataclass
class TensorState:
    """Device state of one parameter tensor (see ps_tensor in include/ps.h)."""
    w_hi: object
    w_lo: object
    m_code: object = None
    m_scale: object = None
    v_code: object = None
    v_scale: object = None
    row_ema: object = None
    col_ema: object = None
    rows: int = 0
    cols: int = 0
    flags: int = 0

    @property
    def numel(self):
        return self.w_hi.numel()


class StateSlab:
    """Optimizer state of a whole tensor list in one contiguous device
    allocation per stream (bf16 weights, residuals, gradients, m codes, v codes,
    m scales, v scales); each tensor gets 256-byte-aligned views. Streaming
    the step over a few large allocations needs far fewer address translations
    than one allocation per tensor and stream.

    numels: element count of each tensor. Moments start as the zero codes with
    zero scales; weights, residuals and gradients are left uninitialised for
    the caller to fill (or copy into)."""

    ALIGN = 128    # elements of a 16-bit stream = 256 bytes

    def __init__(self, numels, device="cuda", with_grads=True, shapes2d=None, host_state=False, moments="codec"):
        """host_state=True puts residuals, codes and scales in pinned host
        memory (the layout ps_offload_* expects); weights and gradients stay
        on `device`. moments="f24" stores both moments as f24 arrays (3 bytes
        per value, zero-initialised, no scales; TENSOR_F24_MOMENTS)."""
        import torch
        self.numels = list(numels)
        offs, boffs, n_tot, nb_tot = [], [], 0, 0
        for n in self.numels:
            offs.append(n_tot)
            boffs.append(nb_tot)
            n_tot += (n + self.ALIGN - 1) // self.ALIGN * self.ALIGN
            nb_tot += ((n + BLOCK - 1) // BLOCK + 63) // 64 * 64
        if moments not in ("codec", "f24"):
            raise ValueError("moments must be 'codec' or 'f24'")
        f24 = moments == "f24"
        names = ["hi", "lo"] + ([] if f24 else ["mc", "vc"]) + (["g"] if with_grads else [])

        def where(k):
            return dict(device="cpu", pin_memory=True) if host_state and k in ("lo", "mc", "vc", "ms", "vs") \
                else dict(device=device)
        self.slab = {k: torch.empty(max(1, n_tot), dtype=torch.int16, **where(k)) for k in names}
        if f24:
            for k in ("mc", "vc"):
                self.slab[k] = torch.zeros(max(1, 3 * n_tot), dtype=torch.uint8, **where(k))
            self.scales = {}
        else:
            self.slab["mc"].fill_(-32768)          # 0x8000: the zero code of the signed kind
            self.slab["vc"].zero_()
            self.scales = {k: torch.zeros(max(1, nb_tot), dtype=torch.float32, **where(k)) for k in ("ms", "vs")}
        self.states, self.grads = [], []
        for i, n in enumerate(self.numels):
            o, bo, nb = offs[i], boffs[i], (n + BLOCK - 1) // BLOCK
            rows, cols = shapes2d[i] if shapes2d else (0, 0)
            if f24:
                self.states.append(TensorState(self.slab["hi"][o:o + n], self.slab["lo"][o:o + n],
                                               self.slab["mc"][3 * o:3 * (o + n)], None,
                                               self.slab["vc"][3 * o:3 * (o + n)], None,
                                               rows=rows, cols=cols, flags=TENSOR_F24_MOMENTS))
            else:
                self.states.append(TensorState(self.slab["hi"][o:o + n], self.slab["lo"][o:o + n],
                                               self.slab["mc"][o:o + n], self.scales["ms"][bo:bo + nb],
                                               self.slab["vc"][o:o + n], self.scales["vs"][bo:bo + nb],
                                               rows=rows, cols=cols))
            self.grads.append(self.slab["g"][o:o + n] if with_grads else None)

    def records(self, grads=None):
        return make_records(self.states, self.grads if grads is None else grads)


def make_records(states: Sequence[TensorState], grads: Sequence[Optional[object]]):
    """ctypes array of ps_tensor records (reusable while the tensors live)."""
    if len(states) != len(grads):
        raise ValueError("states and grads differ in length")
    arr = (CTensor * max(1, len(states)))()
    for i, (s, g) in enumerate(zip(states, grads)):
        arr[i] = CTensor(_ptr(s.w_hi), _ptr(s.w_lo), _ptr(g), _ptr(s.m_code), _ptr(s.m_scale), _ptr(s.v_code),
                         _ptr(s.v_scale), _ptr(s.row_ema), _ptr(s.col_ema), s.numel, s.rows, s.cols,
                         s.flags, 0)
    return arr, len(states)


def step_scalars(hp: HParams, step: int):
    out = (ctypes.c_float * 10)()
    h = hp.c()
    _check(_lib.ps_step_scalars(ctypes.byref(h), step, out))
    names = ("B1", "C1", "B2", "C2", "EPS", "A", "RS2", "AG", "AM", "CWD")
    return dict(zip(names, list(out)))


def opt_step_multi(states, grads=None, hp: HParams = None, step: int = 1, stream=None, records=None):
    """One fused (N)AdamW step over all tensors in one launch. Pass either
    (states, grads) or `records` from make_records()."""
    arr, n = records if records is not None else make_records(states, grads)
    h = (hp or HParams()).c()
    _check(_lib.ps_opt_step_multi(arr, n, ctypes.byref(h), step, _stream(stream)))


def split(w32, hi, lo, mode=SPLIT_TRUNC, stream=None):
    _check(_lib.ps_split(_ptr(w32), _ptr(hi), _ptr(lo), w32.numel(), mode, _stream(stream)))


def join(hi, lo, w32, mode=SPLIT_TRUNC, stream=None):
    _check(_lib.ps_join(_ptr(hi), _ptr(lo), _ptr(w32), hi.numel(), mode, _stream(stream)))


def encode_moments(x, code, scale, kind, stream=None):
    _check(_lib.ps_encode_moments(_ptr(x), _ptr(code), _ptr(scale), x.numel(), kind, _stream(stream)))


def decode_moments(code, scale, x, kind, stream=None):
    _check(_lib.ps_decode_moments(_ptr(code), _ptr(scale), _ptr(x), code.numel(), kind, _stream(stream)))


def factored_workspace_size(states, grads=None, records=None):
    arr, n = records if records is not None else make_records(states, grads)
    out = ctypes.c_size_t(0)
    _check(_lib.ps_factored_workspace_size(arr, n, ctypes.byref(out)))
    return out.value


def factored_step(states, grads=None, hp: FactoredHParams = None, step: int = 1, workspace=None, stream=None,
                  records=None):
    arr, n = records if records is not None else make_records(states, grads)
    h = (hp or FactoredHParams()).c()
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.ps_factored_step(arr, n, ctypes.byref(h), step, _ptr(workspace), ws_bytes, _stream(stream)))


NOALLOC_SCRATCH_BYTES = 32 << 20   # PS_NOALLOC_SCRATCH_BYTES


def factored_step_noalloc(states, grads=None, hp: FactoredHParams = None, step: int = 1, stream=None, records=None):
    """ps_factored_step_noalloc: the factored step with the library's built-in
    scratch as its workspace (no device allocation)."""
    arr, n = records if records is not None else make_records(states, grads)
    h = (hp or FactoredHParams()).c()
    _check(_lib.ps_factored_step_noalloc(arr, n, ctypes.byref(h), step, _stream(stream)))


class OffloadPlan:
    """Host-offload plan (ps_offload_*): groups of tensors whose residual and
    moment state live in pinned host memory. mode OFFLOAD_DIRECT (the step
    kernel works on the host arrays in place, on n_cus compute units) or
    OFFLOAD_STAGED (copies through two device staging slots)."""

    def __init__(self, groups, mode=OFFLOAD_DIRECT, n_cus=OFFLOAD_DEFAULT_CUS):
        # groups: list of (states, grads) with host-pinned lo/codes/scales
        self._recs = [make_records(s, g) for s, g in groups]
        garr = (COffloadGroup * max(1, len(groups)))()
        for i, (arr, n) in enumerate(self._recs):
            garr[i] = COffloadGroup(ctypes.cast(arr, ctypes.POINTER(CTensor)), n)
        self._garr = garr
        h = ctypes.c_void_p()
        opt = COffloadOptions(mode, n_cus, 0, 0)
        _check(_lib.ps_offload_plan_create_ex(garr, len(groups), ctypes.byref(opt), ctypes.byref(h)))
        self._h = h

    def run(self, hp: HParams, step: int, stream=None):
        h = hp.c()
        _check(_lib.ps_offload_run(self._h, ctypes.byref(h), step, _stream(stream)))

    def bytes(self):
        a, b = ctypes.c_uint64(0), ctypes.c_uint64(0)
        _check(_lib.ps_offload_bytes(self._h, ctypes.byref(a), ctypes.byref(b)))
        return a.value, b.value

    def close(self):
        if self._h:
            _check(_lib.ps_offload_plan_destroy(self._h))
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _raw_stream(device, stream):
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    return _current_raw_stream(device.index)


# What holds e4m3 codes: the type itself, or plain bytes. Other 8-bit floats are other values.
_E4M3_DTYPES = () if torch is None else (torch.float8_e4m3fn, torch.uint8, torch.int8)


def _fp8_check(x, code, scale):
    n = x.numel()
    if x.dtype != torch.float32 or scale.dtype != torch.float32:
        raise ValueError("x and scale are float32")
    if code.dtype not in _E4M3_DTYPES:
        raise ValueError(f"code has dtype {code.dtype}, not float8_e4m3fn, uint8 or int8")
    if code.numel() != n or scale.numel() != (n + BLOCK - 1) // BLOCK:
        raise ValueError("code needs x's size and scale one value for each 256 of them")
    if not (x.is_contiguous() and code.is_contiguous() and scale.is_contiguous()):
        raise ValueError("x, code and scale must be contiguous")
    device = x.device
    if code.device != device or scale.device != device:
        raise ValueError("x, code and scale must be on one device")
    if device.type != "cuda":
        raise ValueError("x, code and scale are not on a GPU")
    return n, device


def encode_fp8(x, code, scale, kind, stream=None):
    """float32 moments -> e4m3 codes and a power-of-two scale for each 256 (ps_encode_fp8); kind MOMENT_UNSIGNED
    codes the square root. code: torch.float8_e4m3fn, or its bytes as uint8 or int8."""
    n, device = _fp8_check(x, code, scale)
    with _on(device):
        _check(_lib.ps_encode_fp8(x.data_ptr(), code.data_ptr(), scale.data_ptr(), n, kind, _raw_stream(device, stream)))


def decode_fp8(code, scale, x, kind, stream=None):
    """The float32 moments that e4m3 codes and scales stand for (ps_decode_fp8)."""
    n, device = _fp8_check(x, code, scale)
    with _on(device):
        _check(_lib.ps_decode_fp8(code.data_ptr(), scale.data_ptr(), x.data_ptr(), n, kind, _raw_stream(device, stream)))


class _NoSwitch:
    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return False


_NO_SWITCH = _NoSwitch()


def _on(device):
    """Makes `device` the current one; nothing to do where it is."""
    if device.type != "cuda" or device.index is None or device.index == torch.cuda.current_device():
        return _NO_SWITCH
    return torch.cuda.device(device)


@dataclass
class AdamWTensor:
    """One parameter of an AdamWPlan (see ps_adamw_tensor in include/ps.h).

    param: float32, or bfloat16 (any other 2-byte dtype is read as bf16 bits);
    None if only the gradient's norm is wanted. grad: float32, bfloat16 or
    float16, or None; grad_dtype says what a later one will be (param's dtype if
    not given). m, v: float32, or e4m3 codes (float8_e4m3fn, or their bytes as
    uint8 or int8) with m_scale and v_scale (float32, read whole, written as
    powers of two). residual: a bf16 parameter's low halves. copy: bfloat16 or
    float16, written with a float32 parameter's new values. All contiguous and
    16-byte aligned, scales 4-byte."""
    param: object
    grad: object
    m: object = None
    v: object = None
    m_scale: object = None
    v_scale: object = None
    residual: object = None
    copy: object = None
    group: int = 0
    grad_dtype: object = None


def _adamw_record(i, t):
    def wrong(what):
        return ValueError(f"tensor {i}: {what}")
    ref = t.param if t.param is not None else t.grad
    if ref is None:
        raise wrong("param and grad are both None")
    n = ref.numel()
    types = {torch.float32: TYPE_F32, torch.bfloat16: TYPE_BF16, torch.float16: TYPE_F16}
    nb, device = (n + BLOCK - 1) // BLOCK, ref.get_device()

    def ptr(name, x, size):
        if x is None:
            return None
        if x.numel() != size:
            raise wrong(f"{name} has {x.numel()} elements, not {size}")
        if not x.is_contiguous():
            raise wrong(f"{name} is not contiguous")
        if x.get_device() != device:
            raise wrong(f"{name} is on {x.device}, not on {ref.device}")
        return x.data_ptr() if size else None
    rec = CAdamWTensor(ptr("param", t.param, n), ptr("residual", t.residual, n), ptr("copy", t.copy, n),
                       ptr("grad", t.grad, n), ptr("m", t.m, n), ptr("m_scale", t.m_scale, nb), ptr("v", t.v, n),
                       ptr("v_scale", t.v_scale, nb), n)
    rec.group = t.group
    if t.grad is not None:
        if t.grad.dtype not in types:
            raise wrong(f"grad has dtype {t.grad.dtype}")
        rec.grad_type = types[t.grad.dtype]
        if t.grad_dtype not in (None, t.grad.dtype):
            raise wrong(f"grad has dtype {t.grad.dtype}, not {t.grad_dtype}")
    elif t.grad_dtype is not None:
        if t.grad_dtype not in types:
            raise wrong(f"grad_dtype is {t.grad_dtype}")
        rec.grad_type = types[t.grad_dtype]
    elif t.param is not None:
        rec.grad_type = types.get(t.param.dtype, TYPE_BF16)
    if t.param is None:
        return rec
    if t.m is None or t.v is None:
        raise wrong("m and v are needed")
    if t.param.dtype == torch.float32:
        rec.param_type = TYPE_F32
    elif t.param.dtype == torch.float16 or t.param.element_size() != 2:
        raise wrong(f"param has dtype {t.param.dtype}")
    else:
        rec.param_type = TYPE_BF16
    if t.residual is not None and t.residual.element_size() != 2:
        raise wrong("residual has no 2-byte dtype")
    if t.copy is not None:
        if t.copy.dtype not in (torch.bfloat16, torch.float16):
            raise wrong(f"copy has dtype {t.copy.dtype}")
        rec.copy_type = types[t.copy.dtype]
    if t.m.dtype == torch.float32 and t.v.dtype == torch.float32:
        rec.state_type = STATE_F32
        if t.m_scale is not None or t.v_scale is not None:
            raise wrong("float32 moments have no scales")
    elif t.m.dtype in _E4M3_DTYPES and t.v.dtype in _E4M3_DTYPES:
        rec.state_type = STATE_E4M3
        if t.m_scale is None or t.v_scale is None:
            raise wrong("e4m3 moments need m_scale and v_scale")
        if t.m_scale.dtype != torch.float32 or t.v_scale.dtype != torch.float32:
            raise wrong("scales are float32")
    else:
        raise wrong(f"m and v have dtypes {t.m.dtype} and {t.v.dtype}")
    return rec


class AdamWPlan:
    """AdamW over a fixed list of tensors, and the norm of their gradients
    (ps_adamw_*). Made once; every call then runs on the plan's device, on
    `stream` or the device's current stream, with no allocation. Until it is
    closed the plan keeps the memory of its tensors alive, by references of its
    own: it neither changes the records nor reads them again (set_grads gives it
    other gradients). A graph that captured its calls needs the plan. What is
    released after calls on another stream than the one that was current when it
    was given is recorded on it, so a stream given as an integer has to exist as
    long as the plan.

    The control block's fields are 0-dim tensors in device memory, read and
    written in stream order: norm, grad_mul, skip, skipped, step_count, lr_mul."""

    _h = None

    def __init__(self, tensors: Sequence[AdamWTensor], device=None):
        tensors = list(tensors)
        recs = [_adamw_record(i, t) for i, t in enumerate(tensors)]
        devices = {(t.param if t.param is not None else t.grad).device for t in tensors}
        if len(devices) > 1:
            raise ValueError("the tensors are on several devices")
        self.device = devices.pop() if devices else torch.device(device or "cuda")
        if self.device.type != "cuda":
            raise ValueError("the tensors are not on a GPU")
        self._sizes = [(r.numel, r.grad_type) for r in recs]
        arr = (CAdamWTensor * max(1, len(recs)))(*recs)
        size = ctypes.c_size_t(0)
        _check(_lib.ps_adamw_workspace_size(arr, len(recs), ctypes.byref(size)))
        with _on(self.device):
            self.device = torch.device("cuda", torch.cuda.current_device())
            self._index = self.device.index
            self._stream0 = _current_raw_stream(self._index)
            self.workspace = torch.empty(size.value, dtype=torch.uint8, device=self.device)
            h = ctypes.c_void_p()
            _check(_lib.ps_adamw_plan_create(arr, len(recs), self.workspace.data_ptr(), size.value, self._stream0,
                                             ctypes.byref(h)))
        self._h = h
        # The plan's own references to the memory that its device tables address, the storages: what becomes of the
        # caller's records and tensors (another gradient, another storage) does not free it.
        self._arrays = [x.untyped_storage() for t in tensors
                        for x in (t.param, t.residual, t.copy, t.m, t.m_scale, t.v, t.v_scale) if x is not None]
        self._grads = [None if t.grad is None else t.grad.untyped_storage() for t in tensors]
        self._captured = []              # gradients of captured set_grads calls
        self._streams, self._last = {}, None   # those that the plan ran on, by their integers, and the last one
        self._seen = {self._stream0}     # and those that were current when it was given arrays
        ctl = self.workspace[:ctypes.sizeof(CAdamWControl)]

        def field(name, dtype):
            o = getattr(CAdamWControl, name).offset
            return ctl[o:o + dtype.itemsize].view(dtype).view(())
        self.norm, self.grad_mul = field("norm", torch.float32), field("grad_mul", torch.float32)
        self.skip, self.skipped = field("skip", torch.int32), field("skipped", torch.int32)
        self.step_count, self.lr_mul = field("step", torch.int64), field("lr_mul", torch.float32)
        self._groups = None

    def _on_stream(self, stream):
        if not self._h:
            raise ValueError("the plan is closed")
        raw = _current_raw_stream(self._index) if stream is None else _raw_stream(self.device, stream)
        if raw != self._last:
            self._last = raw
            if raw not in self._streams:
                self._streams[raw] = self._stream_object(stream, raw)
                self._seen.add(raw)
        return raw

    def _stream_object(self, stream, raw):
        if isinstance(stream, torch.cuda.Stream):
            return stream
        if raw == 0:    # ExternalStream(0) would be a new stream
            return torch.cuda.default_stream(self.device)
        return torch.cuda.ExternalStream(raw, device=self.device)

    def _release(self, storages):
        """Before the plan lets memory go: the allocator must not hand it out before the streams that the plan ran on
        are done with it. It does not where all was given and run on one stream."""
        if len(self._seen) == 1:
            return
        for s in storages:
            x = torch.empty(0, dtype=torch.uint8, device=self.device).set_(s)
            for stream in self._streams.values():
                x.record_stream(stream)

    def _run(self, f, *args):
        status = f(self._h, *args)
        if status and torch.cuda.current_device() != self._index:   # refused, for that or for another reason
            with torch.cuda.device(self.device):
                status = f(self._h, *args)
        _check(status)

    def _is_capturing(self, stream, raw):
        with _on(self.device):
            if stream is None or raw == _current_raw_stream(self._index):
                return torch.cuda.is_current_stream_capturing()
            with torch.cuda.stream(self._stream_object(stream, raw)):
                return torch.cuda.is_current_stream_capturing()

    def set_grads(self, grads, stream=None):
        """New gradients for all tensors, in list order; None: the tensor is passed by. The plan keeps them alive
        in place of the ones before; gradients of a captured call, which replays set again, as long as it lives."""
        if len(grads) != len(self._sizes):
            raise ValueError(f"{len(grads)} gradients for {len(self._sizes)} tensors")
        types, device = (torch.float32, torch.bfloat16, torch.float16), self.device
        arr = (ctypes.c_void_p * max(1, len(grads)))()
        for i, (g, (n, ty)) in enumerate(zip(grads, self._sizes)):
            if g is None:
                continue
            if g.dtype != types[ty] or g.numel() != n or not g.is_contiguous() or g.device != device:
                raise ValueError(f"tensor {i}: the gradient must be contiguous {types[ty]} on {device} with {n} elements")
            arr[i] = g.data_ptr()
        raw = self._on_stream(stream)
        self._run(_lib.ps_adamw_set_grads, arr, len(grads), raw)
        if self._is_capturing(stream, raw):          # the tables change when the graph runs
            self._captured += [g.untyped_storage() for g in grads if g is not None]
            return
        self._seen.add(_current_raw_stream(self._index))
        old, self._grads = self._grads, [None if g is None else g.untyped_storage() for g in grads]
        if len(self._seen) > 1:
            self._release([x for x, y in zip(old, self._grads)
                           if x is not None and (y is None or x.data_ptr() != y.data_ptr())])

    def grad_norm(self, max_norm=float("inf"), grad_scale=1.0, stream=None):
        """The gradients' global 2-norm and clip factor into the control block (ps_adamw_grad_norm)."""
        self._run(_lib.ps_adamw_grad_norm, max_norm, grad_scale, self._on_stream(stream))

    def step(self, groups, step=0, clipped=False, rounding=ROUND_NEAREST, stream=None):
        """One step (ps_adamw_step). groups: the HParams of each group. step: the update's number, from 1, or 0
        to count on the device."""
        key = [(g.algo, g.split_mode, g.lr, g.beta1, g.beta2, g.eps, g.weight_decay, g.momentum_decay, g.seed)
               for g in groups]
        if self._groups is None or self._groups[0] != key:
            self._groups = key, (CHParams * max(1, len(key)))(*[CHParams(*k) for k in key])
        self._run(_lib.ps_adamw_step, self._groups[1], len(key), step, int(clipped), rounding, self._on_stream(stream))

    def close(self):
        if self._h:
            h, self._h = self._h, None
            status = _lib.ps_adamw_plan_destroy(h)
            arrays = self._arrays + [g for g in self._grads if g is not None] + self._captured
            self._arrays, self._grads, self._captured = [], [], []
            self._release(arrays + [self.workspace.untyped_storage()])
            _check(status)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
