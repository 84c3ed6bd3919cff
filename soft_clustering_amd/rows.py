"""Row operators of libflashgmm.so (C ABI in include/flashgmm_rows.h): rows
held in 4 or 8 bits, their products, draws from rows of logits, and losses over
them with their gradients.

Argument marshalling only, as in the binding of the mixture calls: tensors are
checked for dtype, device, layout and shape, then the HIP kernels run on the
current stream of the tensors' device.  Outputs come from torch's allocator;
the calls synchronise nothing and can be captured into a graph.  distill and
balance are differentiable in the logits.  Nothing else has a backward: rows,
products, results and teachers that require gradients are refused while
gradients are on (a draw's ids are whole numbers and never have one), and so are
tensors with a forward-mode tangent, logits included.  A result
that is given (out) must not share memory with an input.
"""
from __future__ import annotations

import ctypes

import torch
from torch.autograd import forward_ad

from ._lib import GMM_OK, GMMError, raw_library

TYPE_FLOAT, TYPE_BFLOAT, TYPE_HALF, TYPE_MX, TYPE_BYTE = 0, 1, 2, 3, 4
_TYPES = {torch.float32: TYPE_FLOAT, torch.bfloat16: TYPE_BFLOAT, torch.float16: TYPE_HALF}
ROW_EXPORTS = ["gmm_mx_quantize", "gmm_mx_dequantize", "gmm_mx_product_workspace", "gmm_mx_product",
               "gmm_byte_quantize", "gmm_byte_dequantize", "gmm_byte_product_workspace", "gmm_byte_product",
               "gmm_draw_workspace", "gmm_draw",
               "gmm_distill_workspace", "gmm_distill", "gmm_distill_backward",
               "gmm_balance_stats", "gmm_balance_workspace", "gmm_balance", "gmm_balance_backward"]

_lib = raw_library()


def _declare():
    vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    sig = {
        "gmm_mx_quantize": (i32, [vp, i32, i64, i32, i64, vp, i64, vp, i64, vp]),
        "gmm_mx_dequantize": (i32, [vp, i64, vp, i64, i64, i32, vp, i32, i64, vp]),
        "gmm_mx_product_workspace": (sz, [i32, i64, i64, i32]),
        "gmm_mx_product": (i32, [vp, i32, i64, vp, i64, i64, vp, i64, vp, i64, i64, i32, vp, vp, i32, i64, vp, sz, vp]),
        "gmm_draw_workspace": (sz, [i64, i32]),
        "gmm_draw": (i32, [vp, i32, i64, i32, i64, vp, vp, f32, vp, i32, vp, f32, vp, f32, vp, vp, sz, vp]),
    }
    distill = [vp, i32, i64, i32, i64, vp, i32, i64, vp, i32, i64, i32, f32]
    balance = [vp, i32, i64, i32, i64]
    sig.update({
        "gmm_distill_workspace": (sz, [i64, i32, i32]),
        "gmm_distill": (i32, [*distill, vp, vp, vp, f32, vp, i64, vp, sz, vp]),
        "gmm_distill_backward": (i32, [*distill, vp, vp, i64, vp, i64, vp]),
        "gmm_balance_stats": (sz, [i64, i32]),
        "gmm_balance_workspace": (sz, [i64, i32, i32]),
        "gmm_balance": (i32, [*balance, vp, i32, i64, i32, vp, vp, vp, f32, vp, i64, vp, sz, vp]),
        "gmm_balance_backward": (i32, [*balance, vp, vp, vp, i64, vp]),
    })
    for name in ("quantize", "dequantize", "product_workspace", "product"):
        sig["gmm_byte_" + name] = sig["gmm_mx_" + name]
    for name, (res, args) in sig.items():
        fn = getattr(_lib, name)
        fn.restype = res
        fn.argtypes = args


_declare()


# The tensors of a call are on a GPU, so it is initialised; a torch without GPU
# support has neither function and never makes a call.
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # the hipStream_t of a device's current stream


def _call(device, fn, *args):
    """fn(*args, stream) on the device's current stream; raises on a status."""
    index = device.index
    if _current_device() == index:
        st = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            st = fn(*args, _raw_stream(index))
    if st != GMM_OK:
        raise GMMError(st, _lib.gmm_last_error(None).decode())


def _rows(t, name):
    """(type, N, width, row stride) of a 2-D tensor of a supported type."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    code = _TYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got {t.dim()}-D")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU, got {t.device}")
    N, D = t.shape
    if D >= 1 << 31:  # widths are int32 in the C ABI, which refuses the others
        raise ValueError(f"{name} has rows of {D} values")
    ld, one = t.stride()
    if one != 1 and D > 1:
        raise ValueError(f"{name}'s rows must be contiguous (stride(1) == 1)")
    if ld < D:
        if N > 1:
            raise ValueError(f"{name}'s rows must not overlap (stride(0) >= {D})")
        ld = D
    return code, N, D, ld


def _no_tangent(t, name):
    """No call has a forward-mode derivative: a result without its tangent would
    read as a derivative of zero."""
    if forward_ad._current_level < 0:  # outside of any dual_level there are none (1 us less for a call)
        return
    if isinstance(t, torch.Tensor) and forward_ad.unpack_dual(t).tangent is not None:
        raise ValueError(f"{name} has a forward-mode tangent, for which there is no derivative here")


def _no_gradient(t, name):
    """There is no backward: what would need one is refused."""
    _no_tangent(t, name)
    if isinstance(t, torch.Tensor) and t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} requires gradients, which this call does not compute (detach it, or use no_grad)")


def _overlap(a, b):
    """Whether two tensors of contiguous rows (or one) share memory; where both
    have several rows at different strides, whether their ranges do."""
    if a.numel() == 0 or b.numel() == 0:
        return False

    def span(t):  # first byte, bytes of a row, of the step between rows, of all
        row = (t.shape[-1] if t.dim() > 1 else t.numel()) * t.element_size()
        step = t.stride(0) * t.element_size() if t.dim() > 1 and t.shape[0] > 1 else 0
        return t.data_ptr(), row, step, (t.shape[0] - 1) * step + row

    (pa, ra, sa, na), (pb, rb, sb, nb) = span(a), span(b)
    if pa + na <= pb or pb + nb <= pa:
        return False
    step = sa or sb
    if not step or (sa and sb and sa != sb):
        return True
    at = (pb - pa) % step  # b's rows seen from a's: in the gaps between them or not
    return at < ra or at + rb > step


def _apart(out, *inputs):
    """A result that is given must not lie over what the call reads."""
    for t in inputs:
        if isinstance(t, _HeldRows):
            _apart(out, t.codes, t.scales)
        elif isinstance(t, torch.Tensor) and _overlap(out, t):
            raise ValueError("out shares memory with an input")


def _out(out, shape, dtype, device, name="out"):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(out, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if out.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {out.dtype}")
    if out.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(out.shape)}")
    if out.device != device:
        raise ValueError(f"{name} must be on {device}, got {out.device}")
    return out


def _matrix(out, N, D, dtype, device):
    """(result, row stride): out, checked, or a new matrix."""
    if out is None:
        return torch.empty((N, D), dtype=dtype, device=device), D
    out = _out(out, (N, D), dtype, device)
    _no_gradient(out, "out")
    return out, _rows(out, "out")[3]


class _HeldRows:
    """Rows in codes and block scales (MXRows, ByteRows)."""

    __slots__ = ("codes", "scales", "dim")

    @staticmethod
    def _widths(groups):  # code and scale bytes of a row of so many groups of 128 values
        raise NotImplementedError

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, dim: int):
        groups = -(-int(dim) // 128)
        if dim < 1:
            raise ValueError("dim must be >= 1")
        code_width, scale_width = self._widths(groups)
        for t, width, unit, name in ((codes, code_width, 16, "codes"), (scales, scale_width, 4, "scales")):
            if not isinstance(t, torch.Tensor) or t.dtype != torch.uint8:
                raise TypeError(f"{name} must be a uint8 tensor")
            if t.dim() != 2 or t.shape[1] != width:
                raise ValueError(f"{name} of rows of {dim} values must be N x {width}, got {tuple(t.shape)}")
            if t.stride(1) != 1 or (t.shape[0] > 1 and (t.stride(0) < width or t.stride(0) % unit)):
                raise ValueError(f"{name}: rows must be contiguous, their stride a multiple of {unit}")
        if codes.shape[0] != scales.shape[0] or codes.device != scales.device:
            raise ValueError("codes and scales must have the same rows on the same device")
        self.codes, self.scales, self.dim = codes, scales, int(dim)

    def __len__(self):
        return self.codes.shape[0]

    def __getitem__(self, rows: slice):
        if not isinstance(rows, slice) or rows.step not in (None, 1):
            raise TypeError("rows are taken with a slice of step 1")
        return type(self)(self.codes[rows], self.scales[rows], self.dim)

    @property
    def device(self):
        return self.codes.device

    @property
    def nbytes(self):
        return self.codes.numel() + self.scales.numel()

    @classmethod
    def _empty(cls, N, D, device):
        """Rows to be written (nothing to check)."""
        code_width, scale_width = cls._widths(-(-D // 128))
        rows = object.__new__(cls)
        rows.codes = torch.empty((N, code_width), dtype=torch.uint8, device=device)
        rows.scales = torch.empty((N, scale_width), dtype=torch.uint8, device=device)
        rows.dim = D
        return rows

    def _args(self):
        c, s = self.codes, self.scales
        if c.shape[0] > 1:
            return c.data_ptr(), c.stride(0), s.data_ptr(), s.stride(0)
        return c.data_ptr(), c.shape[1], s.data_ptr(), s.shape[1]


class MXRows(_HeldRows):
    """Rows in 4 bits: codes uint8 (N, 64 G) and scales uint8 (N, 4 G) of rows
    of ``dim`` values, G = ceil(dim / 128).  Slicing with a step of one gives
    the rows in the slice, sharing memory."""

    __slots__ = ()

    @staticmethod
    def _widths(groups):
        return 64 * groups, 4 * groups


class ByteRows(_HeldRows):
    """Rows in 8 bits (E4M3, a power of two for each block of 128 values): codes
    uint8 (N, 128 G) and scales uint8 (N, 4 ceil(G / 4)) of rows of ``dim``
    values, G = ceil(dim / 128).  Slicing with a step of one gives the rows in
    the slice, sharing memory."""

    __slots__ = ()

    @staticmethod
    def _widths(groups):
        return 128 * groups, -(-groups // 4) * 4


def _held(t, kind, name):
    if not isinstance(t, kind):
        raise TypeError(f"{name} must be {kind.__name__}")
    if not t.codes.is_cuda:
        raise ValueError(f"{name} must be on a GPU, got {t.device}")
    return t


def _quantize(kind, fn, X, out):
    code, N, D, ld = _rows(X, "X")
    _no_gradient(X, "X")
    device = X.device
    if out is None:
        out = kind._empty(N, D, device)
    elif len(_held(out, kind, "out")) != N or out.dim != D or out.device != device:
        raise ValueError(f"out must hold {N} rows of {D} values on {device}")
    else:
        _apart(out.codes, X)
        _apart(out.scales, X)
    _call(device, fn, X.data_ptr(), code, N, D, ld, *out._args())
    return out


def _dequantize(kind, fn, rows, dtype, out):
    _held(rows, kind, "rows")
    if dtype not in _TYPES:
        raise TypeError(f"dtype must be float32, bfloat16 or float16, got {dtype}")
    device = rows.codes.device
    N, D = rows.codes.shape[0], rows.dim
    X, ld = _matrix(out, N, D, dtype, device)
    if out is not None:
        _apart(out, rows)
    _call(device, fn, *rows._args(), N, D, X.data_ptr(), _TYPES[dtype], ld)
    return X


def _product(kind, held_type, workspace, fn, A, B, bias, dtype, out):
    _held(B, kind, "B")
    if dtype not in _TYPES:
        raise TypeError(f"dtype must be float32, bfloat16 or float16, got {dtype}")
    device = B.device
    if isinstance(A, kind):
        M, D = len(A), A.dim
        a_type, (a, lda, a_scales, ldas) = held_type, A._args()
    else:
        a_type, M, D, lda = _rows(A, "A")
        _no_gradient(A, "A")
        a, a_scales, ldas = A.data_ptr(), None, 0
    if D != B.dim:
        raise ValueError(f"A has rows of {D} values, B of {B.dim}")
    if A.device != device:
        raise ValueError(f"A is on {A.device}, B on {device}")
    N = len(B)
    if bias is not None:
        if not isinstance(bias, torch.Tensor) or bias.dtype != torch.float32:
            raise TypeError("bias must be a float32 tensor")
        if bias.shape != (N,) or bias.device != device or not bias.is_contiguous():
            raise ValueError(f"bias must be {N} contiguous values on {device}")
        _no_gradient(bias, "bias")
    C, ldc = _matrix(out, M, N, dtype, device)
    if out is not None:
        _apart(out, A, B, bias)
    need = workspace(a_type, M, N, D)
    # the workspace belongs to this call: torch's allocator hands it on in stream order
    ws = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    _call(device, fn, a, a_type, lda, a_scales, ldas, M, *B._args(), N, D,
          None if bias is None else bias.data_ptr(), C.data_ptr(), _TYPES[dtype], ldc,
          None if ws is None else ws.data_ptr(), need)
    return C


def mx_quantize(X: torch.Tensor, out: MXRows | None = None) -> MXRows:
    """The rows of X (float32, bfloat16 or float16) in 4 bits."""
    return _quantize(MXRows, _lib.gmm_mx_quantize, X, out)


def mx_dequantize(rows: MXRows, dtype: torch.dtype = torch.float32, out: torch.Tensor | None = None) -> torch.Tensor:
    """The values that 4-bit rows stand for, rounded once to dtype (exact in
    float32 and bfloat16)."""
    return _dequantize(MXRows, _lib.gmm_mx_dequantize, rows, dtype, out)


def mx_product(A, B: MXRows, bias: torch.Tensor | None = None, dtype: torch.dtype = torch.float32,
               out: torch.Tensor | None = None) -> torch.Tensor:
    """A B^T + bias as a (rows of A) x (rows of B) matrix of dtype.  A: MXRows,
    or a tensor of rows that is quantised on the way (the same results)."""
    return _product(MXRows, TYPE_MX, _lib.gmm_mx_product_workspace, _lib.gmm_mx_product, A, B, bias, dtype, out)


def byte_quantize(X: torch.Tensor, out: ByteRows | None = None) -> ByteRows:
    """The rows of X (float32, bfloat16 or float16) in 8 bits."""
    return _quantize(ByteRows, _lib.gmm_byte_quantize, X, out)


def byte_dequantize(rows: ByteRows, dtype: torch.dtype = torch.float32,
                    out: torch.Tensor | None = None) -> torch.Tensor:
    """The values that 8-bit rows stand for, rounded once to dtype (exact in
    float32, and in bfloat16 from 2^-130 on)."""
    return _dequantize(ByteRows, _lib.gmm_byte_dequantize, rows, dtype, out)


def byte_product(A, B: ByteRows, bias: torch.Tensor | None = None, dtype: torch.dtype = torch.float32,
                 out: torch.Tensor | None = None) -> torch.Tensor:
    """A B^T + bias as a (rows of A) x (rows of B) matrix of dtype.  A: ByteRows,
    or a tensor of rows that is quantised on the way (the same results)."""
    return _product(ByteRows, TYPE_BYTE, _lib.gmm_byte_product_workspace, _lib.gmm_byte_product, A, B, bias, dtype,
                    out)


def _setting(value, dtype, N, device, name):
    """(array pointer or None, scalar) of a setting given for all rows or each."""
    if not isinstance(value, torch.Tensor):
        return None, value
    if value.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {value.dtype}")
    if value.shape != (N,) or value.device != device or not value.is_contiguous():
        raise ValueError(f"{name} must be one value or {N} contiguous values on {device}")
    return value.data_ptr(), 0


def draw(logits: torch.Tensor, u: torch.Tensor, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0,
         out: torch.Tensor | None = None) -> torch.Tensor:
    """One component of each row of logits (N x V), int32, drawn with the random
    numbers u (float32, N values in [0, 1)) after temperature, top-k, top-p and
    min-p; each setting is one number or a tensor with one for each row
    (float32, top_k int32).  Temperature 0 takes the largest logit; top_k < 1,
    top_p >= 1 and min_p <= 0 are off; -1 marks a row without a distribution
    (a NaN, a +inf, or nothing above -inf)."""
    code, N, V, ld = _rows(logits, "logits")
    dev = logits.device
    if not isinstance(u, torch.Tensor) or u.dtype != torch.float32:
        raise TypeError("u must be a float32 tensor")
    if u.shape != (N,) or u.device != dev or not u.is_contiguous():
        raise ValueError(f"u must be {N} contiguous values on {dev}")
    ids = _out(out, (N,), torch.int32, dev)
    if out is not None and not ids.is_contiguous():
        raise ValueError("out must be contiguous")
    t_ptr, t = _setting(temperature, torch.float32, N, dev, "temperature")
    k_ptr, k = _setting(top_k, torch.int32, N, dev, "top_k")
    p_ptr, p = _setting(top_p, torch.float32, N, dev, "top_p")
    m_ptr, m = _setting(min_p, torch.float32, N, dev, "min_p")
    if out is not None:
        _apart(out, logits, u, temperature, top_k, top_p, min_p)
    need = _lib.gmm_draw_workspace(N, V)
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    _call(dev, _lib.gmm_draw, logits.data_ptr(), code, N, V, ld, u.data_ptr(), t_ptr, float(t), k_ptr,
          min(max(int(k), 0), 2**31 - 1), p_ptr, float(p), m_ptr, float(m), ids.data_ptr(),
          None if ws is None else ws.data_ptr(), need)
    return ids


def _id_lists(ids, N, device, flat=False):
    """(pointer, bits, row stride, k) of lists of component ids, N x k (flat: or N)."""
    if not isinstance(ids, torch.Tensor) or ids.dtype not in (torch.int32, torch.int64):
        raise TypeError("ids must be an int32 or int64 tensor")
    if flat and ids.dim() == 1:
        ids = ids[:, None]
    if ids.dim() != 2 or ids.shape[0] != N or ids.device != device:
        raise ValueError(f"ids must have {N} rows on {device}, got {tuple(ids.shape)} on {ids.device}")
    k = ids.shape[1]
    if not 1 <= k <= 1024:
        raise ValueError(f"ids must list between 1 and 1024 components a row, got {k}")
    ld, one = ids.stride()
    if one != 1 and k > 1:
        raise ValueError("ids: rows must be contiguous (stride(1) == 1)")
    if ld < k:
        if N > 1:
            raise ValueError(f"ids: rows must not overlap (stride(0) >= {k})")
        ld = k
    return ids.data_ptr(), 32 if ids.dtype == torch.int32 else 64, ld, k


def _distill_args(logits, ids, teacher, temperature):
    code, N, V, ld = _rows(logits, "logits")
    device = logits.device
    ids_ptr, bits, ld_ids, k = _id_lists(ids, N, device)
    t_code, t_rows, t_k, ld_teacher = _rows(teacher, "teacher")
    if (t_rows, t_k) != (N, k) or teacher.device != device:
        raise ValueError(f"teacher must be {N} x {k} on {device}, got {t_rows} x {t_k} on {teacher.device}")
    _no_tangent(logits, "logits")
    _no_gradient(teacher, "teacher")
    _no_gradient(temperature, "temperature")
    return (logits.data_ptr(), code, N, V, ld, ids_ptr, bits, ld_ids, teacher.data_ptr(), t_code, ld_teacher, k,
            float(temperature))


def _distill(args, device, stats, weights=None, weight=0.0, grad=None, ld_grad=0):
    N, V, k = args[2], args[3], args[11]
    losses = torch.empty(N, dtype=torch.float32, device=device)
    need = _lib.gmm_distill_workspace(N, V, k)
    ws = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    _call(device, _lib.gmm_distill, *args, losses.data_ptr(), None if stats is None else stats.data_ptr(), weights,
          weight, None if grad is None else grad.data_ptr(), ld_grad, None if ws is None else ws.data_ptr(), need)
    return losses


class _Distill(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, ids, teacher, temperature):
        args = _distill_args(logits, ids, teacher, temperature)
        stats = torch.empty((args[2], 2), dtype=torch.float32, device=logits.device)
        losses = _distill(args, logits.device, stats)
        ctx.save_for_backward(logits, ids, teacher, stats)
        ctx.temperature = temperature
        return losses

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, weights):
        logits, ids, teacher, stats = ctx.saved_tensors
        _no_tangent(weights, "the losses' gradient")
        args = _distill_args(logits, ids, teacher, ctx.temperature)
        grad = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
        _call(logits.device, _lib.gmm_distill_backward, *args, stats.data_ptr(), weights.data_ptr(),
              weights.stride(0) if args[2] > 1 else 0, grad.data_ptr(), args[3])
        return grad, None, None, None


def distill(logits: torch.Tensor, ids: torch.Tensor, teacher: torch.Tensor, temperature: float = 1.0) -> torch.Tensor:
    """Distillation losses of rows of logits (N x V), float32, one for each row:
    T^2 KL(p || q), p the softmax of the teacher's logits / T over the components
    ids[n] that it lists (N x k, int32 or int64; negative: none), q the softmax
    of the row / T over all V.  Differentiable in the logits.  A row that lists
    nothing has loss and gradient 0; an id of V or more, or logits without a
    distribution, make a row's loss and gradient NaN."""
    if isinstance(logits, torch.Tensor) and logits.requires_grad and torch.is_grad_enabled():
        _no_tangent(logits, "logits")
        _no_gradient(teacher, "teacher")  # checked here: nothing requires gradients inside
        _no_gradient(temperature, "temperature")
        return _Distill.apply(logits, ids, teacher, float(temperature))
    return _distill(_distill_args(logits, ids, teacher, temperature), logits.device, None)


def distill_grad(logits: torch.Tensor, ids: torch.Tensor, teacher: torch.Tensor, weights=1.0, temperature: float = 1.0,
                 out: torch.Tensor | None = None):
    """(losses, gradient): the losses of distill and the gradient of
    sum(weights * losses) in the logits (in their type), in one pass over them.
    weights: one number or a float32 tensor with one for each row.  For programs
    that know a row's weight before its loss (a mean: 1 / N) and pass the
    gradient on themselves (``outputs.backward(gradient)``)."""
    args = _distill_args(logits, ids, teacher, temperature)
    _no_gradient(logits, "logits")
    device = logits.device
    _no_gradient(weights, "weights")
    w_ptr, w = _setting(weights, torch.float32, args[2], device, "weights")
    grad, ld_grad = _matrix(out, args[2], args[3], logits.dtype, device)
    if out is not None:
        _apart(out, logits, ids, teacher, weights)
    return _distill(args, device, None, w_ptr, float(w), grad, ld_grad), grad


def _balance(logits, ids, weight=0.0, grad=None, ld_grad=0):
    code, N, K, ld = _rows(logits, "logits")
    device = logits.device
    ids_ptr, bits, ld_ids, k = _id_lists(ids, N, device, flat=True)
    counts = torch.empty(K, dtype=torch.int64, device=device)
    loss = torch.empty((), dtype=torch.float32, device=device)
    stats = torch.empty(_lib.gmm_balance_stats(N, K), dtype=torch.float32, device=device)
    need = _lib.gmm_balance_workspace(N, K, k)
    ws = torch.empty(need, dtype=torch.uint8, device=device)
    _call(device, _lib.gmm_balance, logits.data_ptr(), code, N, K, ld, ids_ptr, bits, ld_ids, k, counts.data_ptr(),
          loss.data_ptr(), stats.data_ptr(), weight, None if grad is None else grad.data_ptr(), ld_grad,
          ws.data_ptr(), need)
    return loss, counts, stats


class _Balance(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, ids):
        loss, counts, stats = _balance(logits, ids)
        ctx.save_for_backward(logits, stats)
        ctx.mark_non_differentiable(counts)
        return loss, counts

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, weight, _):
        logits, stats = ctx.saved_tensors
        _no_tangent(weight, "the loss's gradient")
        code, N, K, ld = _rows(logits, "logits")
        grad = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
        _call(logits.device, _lib.gmm_balance_backward, logits.data_ptr(), code, N, K, ld, stats.data_ptr(),
              weight.data_ptr(), grad.data_ptr(), K)
        return grad, None


def balance(logits: torch.Tensor, ids: torch.Tensor):
    """(loss, counts): how evenly components are taken.  ids (N or N x k, int32 or
    int64) are the components that each row of logits (N x K) takes, as draw or a
    top-k gives them, negative ones none; counts (int64, K) how often each is.
    The loss is K sum_e (share of e in the counts) (mean softmax of e over the
    rows that take one), 1 where all is even.  Differentiable in the logits (the
    counts are constants).  An id of K or more makes loss and gradient NaN."""
    _no_tangent(logits, "logits")
    if isinstance(logits, torch.Tensor) and logits.requires_grad and torch.is_grad_enabled():
        return _Balance.apply(logits, ids)
    return _balance(logits, ids)[:2]


def balance_grad(logits: torch.Tensor, ids: torch.Tensor, weight: float = 1.0, out: torch.Tensor | None = None):
    """(loss, counts, gradient): loss and counts of balance and the gradient of
    weight * loss in the logits (in their type), in one pass over them."""
    _, N, K, _ = _rows(logits, "logits")
    _no_gradient(logits, "logits")
    _no_gradient(weight, "weight")
    grad, ld_grad = _matrix(out, N, K, logits.dtype, logits.device)
    if out is not None:
        _apart(out, logits)
        if isinstance(ids, torch.Tensor):
            _apart(out, ids if ids.dim() > 1 or ids.is_contiguous() else ids[:, None])
    loss, counts, _ = _balance(logits, ids, float(weight), grad, ld_grad)
    return loss, counts, grad


__all__ = ["MXRows", "mx_quantize", "mx_dequantize", "mx_product", "ByteRows", "byte_quantize", "byte_dequantize",
           "byte_product", "draw", "distill", "distill_grad", "balance", "balance_grad", "ROW_EXPORTS"]
