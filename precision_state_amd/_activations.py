"""Binding of the activation checkpoints (include/ps.h): the codec of saved
activations, feed-forward activations, block norms and weight gradients.
Imported into the package's own namespace.

Matrices are 2-dim tensors whose rows are contiguous and may lie apart (views of
some columns of a wider one); codes are whole, [rows, cols], float8_e4m3fn or
their bytes as uint8 or int8, with float32 scales [rows, ceil(cols / 128)].
Every function runs on the tensors' device, on `stream` or the device's current
stream."""
import ctypes
from dataclasses import dataclass

import torch

from . import (_E4M3_DTYPES, _check, _lib, _on, _raw_stream, ACT_BLOCK, NORM_GATE_BY_SEG, NORM_MOD_BY_SEG,
               NORM_MUL_PLUS_ONE, NORM_NONE, NORM_RMS, TYPE_BF16, TYPE_F16, TYPE_F32, CBlockNorm, CBlockNormBwd,
               CBlockNormFwd, CLinearWgrad)

_TYPES = {torch.float32: TYPE_F32, torch.bfloat16: TYPE_BF16, torch.float16: TYPE_F16}


def _like(x, name):
    """x as the first matrix of a call: shape, type and device that the others have to have, and pointer and distance
    between rows."""
    shape, dtype, device = x.shape, x.dtype, x.device
    if len(shape) != 2:
        raise ValueError(f"{name} has {len(shape)} dimensions, not 2")
    if dtype not in _TYPES:
        raise ValueError(f"{name} has dtype {dtype}, not float32, bfloat16 or float16")
    if not x.is_cuda:
        raise ValueError(f"{name} is not on a GPU")
    return shape, dtype, device, _rows(x, name, shape)


def _matrix(x, name, shape, dtype, device):
    """Pointer and distance between rows."""
    if x is None:
        return None, 0
    if x.shape != shape or x.dtype is not dtype or x.device != device:
        raise ValueError(f"{name} is {x.dtype} {tuple(x.shape)} on {x.device}, not {dtype} {tuple(shape)} on {device}")
    return _rows(x, name, shape)


def _rows(x, name, shape):
    row, col = x.stride()
    if col != 1 and shape[1] > 1:
        raise ValueError(f"the rows of {name} are not contiguous")
    at = x.data_ptr()
    if at < _LOW:
        _released(x, name)
    return at, row if shape[0] > 1 else shape[1]    # a single row has no distance to another


# A tensor whose storage was released has its offset for an address: NULL would mean that there is no such array, and
# nothing lies at the others. No allocation lies so low; the storage itself is looked at there only.
_LOW = 1 << 36


def _released(x, name):
    if x.numel() and not x.untyped_storage().nbytes():
        raise ValueError(f"the storage of {name} was released")


def _whole(x, name, shape, dtypes, device):
    """Pointer of a contiguous array."""
    if x is None:
        return None
    if x.shape != shape or x.dtype not in dtypes or x.device != device:
        raise ValueError(f"{name} is {x.dtype} {tuple(x.shape)} on {x.device}, not {dtypes[0]} {tuple(shape)} on {device}")
    if not x.is_contiguous():
        raise ValueError(f"{name} is not contiguous")
    at = x.data_ptr()
    if at < _LOW:
        _released(x, name)
    return at


_F32 = (torch.float32,)


def _code(code, scale, name, shape, device):
    if code is None and scale is None:
        return None, None
    return (_whole(code, f"{name}code", shape, _E4M3_DTYPES, device),
            _whole(scale, f"{name}scale", (shape[0], (shape[1] + ACT_BLOCK - 1) // ACT_BLOCK), _F32, device))


def _needed(**arrays):
    for name, x in arrays.items():
        if x is None:
            raise ValueError(f"{name} is needed")


def _room(workspace, size, device, stream):
    """The caller's workspace, or one for this call alone, and its bytes."""
    if workspace is None:
        if stream is None:
            workspace = torch.empty(size, dtype=torch.uint8, device=device)
        else:    # the allocator hands it out again in that stream's order
            if not isinstance(stream, int):
                obj = stream
            elif stream == 0:    # ExternalStream(0) would be a new stream
                obj = torch.cuda.default_stream(device)
            else:
                obj = torch.cuda.ExternalStream(stream, device=device)
            with torch.cuda.stream(obj):
                workspace = torch.empty(size, dtype=torch.uint8, device=device)
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace has to be contiguous on {device}")
    elif workspace.data_ptr() < _LOW:
        _released(workspace, "workspace")
    return workspace, workspace.numel() * workspace.element_size()


def encode_act(x, code, scale, stream=None):
    """A matrix -> e4m3 codes and a power-of-two scale for each 128 columns of a row (ps_encode_act)."""
    _needed(code=code, scale=scale)
    shape, dtype, device, (p, ld) = _like(x, "x")
    c, s = _code(code, scale, "", shape, device)
    with _on(device):
        _check(_lib.ps_encode_act(p, _TYPES[dtype], shape[0], shape[1], ld, c, s, _raw_stream(device, stream)))


def decode_act(code, scale, x, stream=None):
    """The matrix that codes and scales stand for (ps_decode_act)."""
    _needed(code=code, scale=scale)
    shape, dtype, device, (p, ld) = _like(x, "x")
    c, s = _code(code, scale, "", shape, device)
    with _on(device):
        _check(_lib.ps_decode_act(c, s, p, _TYPES[dtype], shape[0], shape[1], ld, _raw_stream(device, stream)))


def glu_forward(a, out, act, a_code=None, a_scale=None, b=None, b_code=None, b_scale=None, stream=None):
    """out = f(a) * b, or f(a) without b, f one of ACT_*; a and b saved in codes and scales if these are given
    (ps_glu_forward)."""
    shape, dtype, device, (pa, lda) = _like(a, "a")
    pb, ldb = _matrix(b, "b", shape, dtype, device)
    _needed(out=out)
    po, ldo = _matrix(out, "out", shape, dtype, device)
    ca, sa = _code(a_code, a_scale, "a_", shape, device)
    cb, sb = _code(b_code, b_scale, "b_", shape, device)
    with _on(device):
        _check(_lib.ps_glu_forward(shape[0], shape[1], _TYPES[dtype], act, pa, lda, pb, ldb, po, ldo, ca, sa, cb, sb,
                                   _raw_stream(device, stream)))


def glu_backward(dout, act, a_code, a_scale, da, b_code=None, b_scale=None, db=None, out=None, stream=None):
    """The gradients of a, and of b if it is gated, from the saved codes; and the output once more, if `out` is given
    (ps_glu_backward)."""
    _needed(a_code=a_code, a_scale=a_scale, da=da)
    shape, dtype, device, (pd, ldd) = _like(dout, "dout")
    ca, sa = _code(a_code, a_scale, "a_", shape, device)
    cb, sb = _code(b_code, b_scale, "b_", shape, device)
    pa, lda = _matrix(da, "da", shape, dtype, device)
    pb, ldb = _matrix(db, "db", shape, dtype, device)
    po, ldo = _matrix(out, "out", shape, dtype, device)
    with _on(device):
        _check(_lib.ps_glu_backward(shape[0], shape[1], _TYPES[dtype], act, pd, ldd, ca, sa, cb, sb, pa, lda, pb, ldb,
                                    po, ldo, _raw_stream(device, stream)))


@dataclass(frozen=True, eq=False)
class BlockNorm:
    """What a block norm is made of (see ps_block_norm in include/ps.h). The vectors have one dtype; gate, and mul and
    add together, are [cols], or [segments, cols] with a vector for each. segments: int32 tensor on the device, where
    each of the batch's packed sequences starts, and where the last one ends.

    Each call reads the vectors as they are then: a vector may be given other memory (`.data = ...`, a module that moves,
    a storage that is released and comes back) between calls. Checks are repeated where a vector's address, type or
    shape is not what it was."""
    pre_norm: int = NORM_RMS
    pre_eps: float = 1e-6
    post_norm: int = NORM_NONE
    post_eps: float = 1e-6
    residual_scale: float = 1.0
    branch_scale: float = 1.0
    post_weight: object = None
    gate: object = None
    mul: object = None
    add: object = None
    mul_plus_one: bool = False
    segments: object = None

    def _record(self, rows, cols, dtype, device):
        """A record of the call's own: two threads may use one norm."""
        made = self.__dict__.get("_made")
        vectors = made[0] if made else [v for v in (self.post_weight, self.gate, self.mul, self.add, self.segments) if v is not None]
        now = [cols, dtype, device]
        for v in vectors:    # an address is one device's
            now += v.data_ptr(), v.dtype, v.shape, v.is_contiguous()
        if made is None or made[1] != now:
            made = vectors, now, bytes(self._make(cols, dtype, device))
            object.__setattr__(self, "_made", made)
        rec = CBlockNorm.from_buffer_copy(made[2])
        rec.rows = rows
        return rec

    def __getstate__(self):
        """Without the record, which is this norm's alone."""
        return {k: v for k, v in self.__dict__.items() if k != "_made"}

    def _make(self, cols, dtype, device):
        segs = 0 if self.segments is None else self.segments.numel() - 1
        flags, vec, ptr = NORM_MUL_PLUS_ONE if self.mul_plus_one else 0, None, []
        for name, v, by_seg in (("post_weight", self.post_weight, 0), ("gate", self.gate, NORM_GATE_BY_SEG),
                                ("mul", self.mul, NORM_MOD_BY_SEG), ("add", self.add, NORM_MOD_BY_SEG)):
            if v is None:
                ptr.append(None)
                continue
            if vec is None:
                vec = v.dtype
                if vec not in _TYPES:
                    raise ValueError(f"{name} has dtype {vec}, not float32, bfloat16 or float16")
            wide = by_seg and v.dim() == 2
            ptr.append(_whole(v, name, (segs, cols) if wide else (cols,), (vec,), device))
            if wide:
                flags |= by_seg
        if self.mul is not None and self.add is not None and self.mul.dim() != self.add.dim():
            raise ValueError("mul and add have different shapes")
        starts = _whole(self.segments, "segments", (segs + 1,), (torch.int32,), device)
        return CBlockNorm(0, cols, starts, *ptr, self.post_eps, self.pre_eps, self.residual_scale, self.branch_scale,
                          _TYPES[dtype], _TYPES[vec or torch.float32], self.post_norm, self.pre_norm, segs, flags)


def block_norm_forward(norm: BlockNorm, x, n, y=None, h=None, h_code=None, h_rstd=None, y_code=None, y_scale=None,
                       y_rstd=None, stream=None):
    """h = residual_scale x + branch_scale gate N1(y) post_weight and n = N2(h) mul + add, with what the backward pass
    needs saved in h_code, h_rstd and, with a post norm or a gate, y_code and y_rstd or y_scale
    (ps_block_norm_forward)."""
    shape, dtype, device, first = _like(x, "x")
    _needed(n=n)
    rec = norm._record(shape[0], shape[1], dtype, device)
    hc, _ = _code(h_code, None, "h_", shape, device)
    yc, ys = _code(y_code, y_scale, "y_", shape, device)
    io = CBlockNormFwd(*first, *_matrix(y, "y", shape, dtype, device),
                       *_matrix(h, "h", shape, dtype, device), *_matrix(n, "n", shape, dtype, device),
                       hc, _whole(h_rstd, "h_rstd", shape[:1], _F32, device), yc, ys,
                       _whole(y_rstd, "y_rstd", shape[:1], _F32, device))
    with _on(device):
        _check(_lib.ps_block_norm_forward(rec, io, _raw_stream(device, stream)))


def block_norm_workspace_size(norm: BlockNorm, rows, cols):
    """Bytes of workspace of a backward call (ps_block_norm_workspace_size)."""
    segs = 0 if norm.segments is None else norm.segments.numel() - 1
    rec = CBlockNorm(rows, cols, norm.segments.data_ptr() if segs else None, pre_norm=NORM_RMS, n_segs=segs)
    out = ctypes.c_size_t(0)
    _check(_lib.ps_block_norm_workspace_size(rec, out))
    return out.value


def block_norm_backward(norm: BlockNorm, dn, h_code, h_rstd, dx, dh=None, dy=None, y_code=None, y_scale=None,
                        y_rstd=None, d_post_weight=None, d_gate=None, d_mul=None, d_add=None, accumulate=False,
                        workspace=None, stream=None):
    """The gradients dx and, with a branch, dy from those of n and h and what the forward pass saved, and the float32
    gradients of the vectors that are given (ps_block_norm_backward). workspace: block_norm_workspace_size bytes, or
    None for one of the call's own."""
    _needed(h_code=h_code, h_rstd=h_rstd, dx=dx)
    shape, dtype, device, first = _like(dn, "dn")
    rec = norm._record(shape[0], shape[1], dtype, device)
    hc, _ = _code(h_code, None, "h_", shape, device)
    yc, ys = _code(y_code, y_scale, "y_", shape, device)
    grads = []
    for name, d, v in (("post_weight", d_post_weight, norm.post_weight), ("gate", d_gate, norm.gate),
                       ("mul", d_mul, norm.mul), ("add", d_add, norm.add)):
        if d is not None and v is None:
            raise ValueError(f"d_{name} needs {name}")
        grads.append(None if d is None else _whole(d, f"d_{name}", v.shape, _F32, device))
    with _on(device):
        if workspace is None:
            size = ctypes.c_size_t(0)
            _check(_lib.ps_block_norm_workspace_size(rec, size))
            workspace, room = _room(None, size.value, device, stream)
        else:
            workspace, room = _room(workspace, 0, device, stream)
        io = CBlockNormBwd(*first, *_matrix(dh, "dh", shape, dtype, device), hc,
                           _whole(h_rstd, "h_rstd", shape[:1], _F32, device), yc, ys,
                           _whole(y_rstd, "y_rstd", shape[:1], _F32, device), *_matrix(dx, "dx", shape, dtype, device),
                           *_matrix(dy, "dy", shape, dtype, device), *grads, workspace.data_ptr(), room, int(accumulate))
        _check(_lib.ps_block_norm_backward(rec, io, _raw_stream(device, stream)))


def linear_wgrad_workspace_size(tokens, out_features, in_features):
    """Bytes of workspace of linear_wgrad (ps_linear_wgrad_workspace_size)."""
    out = ctypes.c_size_t(0)
    _check(_lib.ps_linear_wgrad_workspace_size(tokens, out_features, in_features, out))
    return out.value


def linear_wgrad(dy, code, dw, scale=None, db=None, mul=None, add=None, accumulate=False, workspace=None, stream=None):
    """The gradient dw [out, in] of a linear layer's weight from dy [tokens, out] and the codes of its input
    [tokens, in], with their scales or, for the h_code of a block norm, with the norm's vectors as mul and add; and that
    of its bias, db (ps_linear_wgrad). mul, add, db: float32. workspace: linear_wgrad_workspace_size bytes, or None for
    one of the call's own."""
    _needed(code=code, dw=dw)
    shape, dtype, device, (pd, ldd) = _like(dy, "dy")
    if code.dim() != 2:
        raise ValueError(f"code has {code.dim()} dimensions, not 2")
    tokens, n = shape
    k = code.shape[1]
    c, s = _code(code, scale, "", (tokens, k), device)
    if dw.dtype not in _TYPES:
        raise ValueError(f"dw has dtype {dw.dtype}, not float32, bfloat16 or float16")
    pw, ldw = _matrix(dw, "dw", (n, k), dw.dtype, device)
    vectors = [_whole(v, name, (size,), _F32, device) for name, v, size in (("mul", mul, k), ("add", add, k), ("db", db, n))]
    with _on(device):
        size = linear_wgrad_workspace_size(tokens, n, k) if workspace is None else 0
        workspace, room = _room(workspace, size, device, stream)
        args = CLinearWgrad(tokens, n, k, pd, ldd, c, s, vectors[0], vectors[1], pw, ldw, vectors[2],
                            workspace.data_ptr(), room, _TYPES[dtype], _TYPES[dw.dtype], int(accumulate))
        _check(_lib.ps_linear_wgrad(args, _raw_stream(device, stream)))
