"""Row operators of libflashgmm.so (C ABI in include/flashgmm_rows.h): rows
held in 4 bits, their products, and draws from rows of logits.

Argument marshalling only, as in the binding of the mixture calls: tensors are
checked for dtype, device, layout and shape, then the HIP kernels run on the
current stream of the tensors' device.  Outputs come from torch's allocator;
the calls synchronise nothing and can be captured into a graph.  None has a
backward: rows, products and results that require gradients are refused while
gradients are on (a draw's ids are whole numbers and never have one).  A result
that is given (out) must not share memory with an input.
"""
from __future__ import annotations

import ctypes

import torch

from ._lib import GMM_OK, GMMError, raw_library

TYPE_FLOAT, TYPE_BFLOAT, TYPE_HALF, TYPE_MX = 0, 1, 2, 3
_TYPES = {torch.float32: TYPE_FLOAT, torch.bfloat16: TYPE_BFLOAT, torch.float16: TYPE_HALF}
ROW_EXPORTS = ["gmm_mx_quantize", "gmm_mx_dequantize", "gmm_mx_product_workspace", "gmm_mx_product",
               "gmm_draw_workspace", "gmm_draw"]

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


def _no_gradient(t, name):
    """There is no backward: what would need one is refused."""
    if t.requires_grad and torch.is_grad_enabled():
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
        if isinstance(t, MXRows):
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


class MXRows:
    """Rows in 4 bits: codes uint8 (N, 64 G) and scales uint8 (N, 4 G) of rows
    of ``dim`` values, G = ceil(dim / 128).  Slicing with a step of one gives
    the rows in the slice, sharing memory."""

    __slots__ = ("codes", "scales", "dim")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, dim: int):
        groups = -(-int(dim) // 128)
        if dim < 1:
            raise ValueError("dim must be >= 1")
        for t, width, unit, name in ((codes, 64 * groups, 16, "codes"), (scales, 4 * groups, 4, "scales")):
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
        return MXRows(self.codes[rows], self.scales[rows], self.dim)

    @property
    def device(self):
        return self.codes.device

    @property
    def nbytes(self):
        return self.codes.numel() + self.scales.numel()

    @staticmethod
    def _empty(N, D, device):
        """Rows to be written (nothing to check)."""
        G = -(-D // 128)
        rows = object.__new__(MXRows)
        rows.codes = torch.empty((N, 64 * G), dtype=torch.uint8, device=device)
        rows.scales = torch.empty((N, 4 * G), dtype=torch.uint8, device=device)
        rows.dim = D
        return rows

    def _args(self):
        c, s = self.codes, self.scales
        N, wc = c.shape
        if N > 1:
            return c.data_ptr(), c.stride(0), s.data_ptr(), s.stride(0)
        return c.data_ptr(), wc, s.data_ptr(), wc // 16


def _mx(t, name):
    if not isinstance(t, MXRows):
        raise TypeError(f"{name} must be MXRows")
    if not t.codes.is_cuda:
        raise ValueError(f"{name} must be on a GPU, got {t.device}")
    return t


def mx_quantize(X: torch.Tensor, out: MXRows | None = None) -> MXRows:
    """The rows of X (float32, bfloat16 or float16) in 4 bits."""
    code, N, D, ld = _rows(X, "X")
    _no_gradient(X, "X")
    device = X.device
    if out is None:
        out = MXRows._empty(N, D, device)
    elif len(_mx(out, "out")) != N or out.dim != D or out.device != device:
        raise ValueError(f"out must hold {N} rows of {D} values on {device}")
    else:
        _apart(out.codes, X)
        _apart(out.scales, X)
    _call(device, _lib.gmm_mx_quantize, X.data_ptr(), code, N, D, ld, *out._args())
    return out


def mx_dequantize(rows: MXRows, dtype: torch.dtype = torch.float32, out: torch.Tensor | None = None) -> torch.Tensor:
    """The values that 4-bit rows stand for, rounded once to dtype (exact in
    float32 and bfloat16)."""
    _mx(rows, "rows")
    if dtype not in _TYPES:
        raise TypeError(f"dtype must be float32, bfloat16 or float16, got {dtype}")
    device = rows.codes.device
    N, D = rows.codes.shape[0], rows.dim
    X, ld = _matrix(out, N, D, dtype, device)
    if out is not None:
        _apart(out, rows)
    _call(device, _lib.gmm_mx_dequantize, *rows._args(), N, D, X.data_ptr(), _TYPES[dtype], ld)
    return X


def mx_product(A, B: MXRows, bias: torch.Tensor | None = None, dtype: torch.dtype = torch.float32,
               out: torch.Tensor | None = None) -> torch.Tensor:
    """A B^T + bias as a (rows of A) x (rows of B) matrix of dtype.  A: MXRows,
    or a tensor of rows that is quantised on the way (the same results)."""
    _mx(B, "B")
    if dtype not in _TYPES:
        raise TypeError(f"dtype must be float32, bfloat16 or float16, got {dtype}")
    device = B.device
    if isinstance(A, MXRows):
        M, D = len(A), A.dim
        a_type, (a, lda, a_scales, ldas) = TYPE_MX, A._args()
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
    need = _lib.gmm_mx_product_workspace(a_type, M, N, D)
    # the workspace belongs to this call: torch's allocator hands it on in stream order
    ws = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    _call(device, _lib.gmm_mx_product, a, a_type, lda, a_scales, ldas, M, *B._args(), N, D,
          None if bias is None else bias.data_ptr(), C.data_ptr(), _TYPES[dtype], ldc,
          None if ws is None else ws.data_ptr(), need)
    return C


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


__all__ = ["MXRows", "mx_quantize", "mx_dequantize", "mx_product", "draw", "ROW_EXPORTS"]
