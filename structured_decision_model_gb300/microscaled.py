"""PyTorch-side helper around the microscaled 4-bit operators: device buffers and streams only.

    w = Fp4Linear(weight, bias)                  # weights laid out once, in 4 bits
    y = w(x)                                     # rows quantised and multiplied
    y, mean, rstd = w.normalized(x)              # the layer behind a LayerNorm whose weight it holds

and by single steps: ``quantize`` (an ``Fp4Matrix``), ``Fp4Matrix.dequantize`` and ``product``.
All arithmetic happens in libclef_head.so, on torch's current stream.  Nothing here waits
for the GPU but the first matrix on a device, whose words for reports are cleared from the host (and every 2048th
matrix of weights); ``device_status`` does, and reports what the kernels met.  A value is kept as
the nearest of 16 numbers times its block's scale: "mxfp4" (blocks of 32, a power of two)
or "nvfp4" (blocks of 16, three bits behind the point, and a power of two for each row).
Nothing here passes gradients on: inputs, outputs and a product's bias that require one are refused while grad mode
is on, and dual tensors of forward mode always.  A layer's weight and bias are frozen: taken as numbers, also where they
are parameters that require a gradient.
"""
import threading
from typing import Optional, Tuple

import torch
from torch.autograd import forward_ad as _forward

from . import binding as B
from .memory import _DTYPES, _current_device, _overlap, _raw_stream, _refuse

FORMATS = {"mxfp4": B.MXFP4, "nvfp4": B.NVFP4}
BLOCK = {"mxfp4": 32, "nvfp4": 16}
_FP32 = torch.float32
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", None) or torch.cuda.is_current_stream_capturing


# (input type, output type asked for): their codes, and the output's type
_TYPES = {(a, b): (_DTYPES[a], _DTYPES[b or a], b or a) for a in _DTYPES for b in (None, *_DTYPES)}


def _dual(t) -> bool:
    """Whether a tensor carries a tangent of forward-mode differentiation (asked on every call: no level, no look)."""
    return _forward._current_level >= 0 and _forward.unpack_dual(t).tangent is not None


def _up(n: int) -> int:
    return (n + 255) // 256 * 256


# Words that products report in, by device: [cleared ones, how many are taken].  Every matrix takes one at its first
# product, apart from every other matrix's, so that a word is clear for every stream from the start and no captured graph
# clears it again.
_WORDS = 4096
_words = {}
_words_lock = threading.Lock()


def _cleared_words(index, want):
    """The device's words with at least ``want`` to take, half of all where no capture keeps new ones from being cleared."""
    words = _words.get(index)
    if words is None or words[1] > _WORDS // 2:
        if not _capturing():
            # from the host, which waits for the copy: whatever stream uses a word first comes behind it
            words = _words[index] = [torch.zeros(_WORDS, dtype=torch.int32).to(torch.device("cuda", index)), 0]
        elif want and (words is None or words[1] == _WORDS):
            _refuse("a capture cannot clear flags: ask for the matrix's before it")
    return words


def _flag_word(index):
    with _words_lock:
        words = _cleared_words(index, 1)
        words[1] += 1
        return words[0][words[1] - 1:words[1]]


class Fp4Matrix:
    """Rows kept in 4 bits: codes, block scales and row scales, one after the other in ``data``.

    ``data`` (uint8, contiguous, of ``size_bytes``) may be a buffer of the caller, taken as it is: what an earlier
    matrix of the same shape and format held, for instance.  ``mean``, ``rstd`` and ``sums`` (fp32 [rows])
    are there where ``quantize`` was asked for them.
    """

    __slots__ = ("rows", "cols", "format", "data", "struct", "device", "mean", "rstd", "sums", "_flags", "_index")

    def __init__(self, rows: int, cols: int, format: str = "nvfp4", device="cuda", data: Optional[torch.Tensor] = None):
        code = FORMATS.get(format)
        if code is None:
            _refuse(f"format: one of {sorted(FORMATS)}")
        if not 1 <= rows < 2 ** 31 - 256 or not 1 <= cols <= B.FP4_MAX_COLS:
            _refuse(f"an Fp4Matrix has 1 to 2^31 - 257 rows of 1 to {B.FP4_MAX_COLS} values")
        # codes, scales and row scales, each from 256 bytes on (sizes as clef_fp4_size gives them)
        scales = _up(rows * ((cols + 31) // 32 * 16))
        row_scale = scales + (rows + 127) // 128 * ((cols + 255) // 256 * (2048 if code else 1024))
        size = row_scale + (4 * rows if code else 0)
        if data is None:
            data = torch.empty(size, dtype=torch.uint8, device=device)
        elif data.dtype != torch.uint8 or data.dim() != 1 or data.numel() != size or not data.is_contiguous() or \
                data.data_ptr() % 256:
            _refuse("Fp4Matrix: data is not a contiguous uint8 vector of size_bytes on 256 bytes")
        index = data.get_device()
        if index < 0:
            _refuse("Fp4Matrix: data is not on a GPU")
        base = data.data_ptr()
        self.rows, self.cols, self.format, self.data = rows, cols, format, data
        self.struct = B.ClefFp4(base, base + scales, base + row_scale if code else None, rows, cols, code)
        self.device, self._index = data.device, index
        if index not in _words:  # now, so that a later capture finds some
            with _words_lock:
                _cleared_words(index, 0)
        self.mean = self.rstd = self.sums = self._flags = None

    @property
    def size_bytes(self) -> int:
        return self.data.numel()

    @property
    def flags(self) -> torch.Tensor:
        """What the products with these weights report (int32 [1])."""
        if self._flags is None:
            self._flags = _flag_word(self._index)
        return self._flags

    def dequantize(self, dtype=torch.bfloat16, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """What the rows stand for, [rows, cols] in ``dtype`` (bf16, fp16 or fp32), rounded once.

        nvfp4 rows may stand for up to 18 / 17 of their largest value, which passes the type's range next to its end."""
        given = out is not None
        out = _out(out, self.rows, self.cols, dtype, self.device)
        if given and _overlap(out, self.data):
            _refuse("out lies apart from what is read")
        if _current_device() != self._index:
            with torch.cuda.device(self._index):
                return self.dequantize(dtype, out)
        B.clef_fp4_dequantize(self.struct, _DTYPES[dtype], out.data_ptr(), _row_stride(out), _raw_stream(self._index))
        return out

    def device_status(self) -> int:
        """Waits for the current stream, reads and clears what the products with these weights reported."""
        if _current_device() != self._index:
            with torch.cuda.device(self._index):
                return self.device_status()
        return B.clef_cache_status(self.flags.data_ptr(), _raw_stream(self._index))


def _out(out, rows, cols, dtype, device):
    if dtype not in _DTYPES:
        _refuse("outputs: bf16, fp16 or fp32")
    if out is None:
        return torch.empty((rows, cols), dtype=dtype, device=device)
    if out.dtype != dtype or out.shape != (rows, cols) or out.device != device or \
            (cols > 1 and out.stride(1) != 1) or (rows > 1 and out.stride(0) < cols):
        _refuse(f"out: {dtype} [{rows}, {cols}], values of a row contiguous, rows apart, on {device}")
    if (out.requires_grad and torch.is_grad_enabled()) or _dual(out):
        _refuse("out requires a gradient")
    return out


def _row_stride(t):
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


_lib = B.load


def quantize(x: torch.Tensor, format: str = "nvfp4", stats: bool = False, sums: bool = False,
             out: Optional[Fp4Matrix] = None) -> Fp4Matrix:
    """Rows x [rows, cols] (bf16, fp16 or fp32, any row stride, values contiguous) in 4 bits.

    ``stats``: also the rows' ``mean`` and ``rstd`` = 1 / sqrt(variance + 1e-5); ``sums``: also the
    sums of what the rows stand for once kept."""
    dtype, shape, strides = _DTYPES.get(x.dtype), x.shape, x.stride()
    if dtype is None or len(shape) != 2 or (strides[1] != 1 and shape[1] > 1) or not x.is_cuda:
        _refuse("x: bf16, fp16 or fp32 [rows, cols], values of a row contiguous, on a GPU")
    if (x.requires_grad and torch.is_grad_enabled()) or _dual(x):
        _refuse("x requires a gradient, which 4-bit rows do not pass on")
    rows, cols = shape
    if out is None:
        out = Fp4Matrix(rows, cols, format, x.device)
    elif (out.rows, out.cols, out.format, out.device) != (rows, cols, format, x.device):
        _refuse("out: an Fp4Matrix of x's shape and device and of the format")
    if _current_device() != out._index:
        with torch.cuda.device(out._index):
            return quantize(x, format, stats, sums, out)
    out.mean = out.rstd = out.sums = mean = rstd = total = None
    if stats:
        out.mean = torch.empty(rows, dtype=_FP32, device=x.device)
        out.rstd = torch.empty(rows, dtype=_FP32, device=x.device)
        mean, rstd = out.mean.data_ptr(), out.rstd.data_ptr()
    if sums:
        out.sums = torch.empty(rows, dtype=_FP32, device=x.device)
        total = out.sums.data_ptr()
    status = _lib().clef_fp4_quantize(out.struct, dtype, x.data_ptr(), strides[0] if rows > 1 else cols, mean, rstd, total,
                                      _raw_stream(out._index))
    if status:
        raise B.ClefError(status, "clef_fp4_quantize")
    return out


def product(x: Fp4Matrix, w: Fp4Matrix, bias: Optional[torch.Tensor] = None, dtype=torch.bfloat16,
            normalized: bool = False, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x w^T + bias: [x.rows, w.rows] in ``dtype`` (bf16, fp16 or fp32), sums in fp32, rounded once.

    ``normalized``: x's rows less their means and times their rstd (x quantised with ``stats``, w
    with ``sums``).  ``bias``: fp32 [w.rows]."""
    if x.format != w.format or x.cols != w.cols or x.device != w.device:
        _refuse("product: one format, number of columns and device")
    if bias is not None and (bias.dtype is not _FP32 or bias.shape != (w.rows,) or not bias.is_contiguous() or
                             bias.device != w.device or (bias.requires_grad and torch.is_grad_enabled()) or _dual(bias)):
        _refuse("bias: contiguous fp32 [w.rows], without a gradient, on the matrices' device")
    if normalized and (x.mean is None or w.sums is None):
        _refuse("normalized: x quantised with stats=True, w with sums=True")
    given = out is not None
    out = _out(out, x.rows, w.rows, dtype, w.device)
    if given and any(_overlap(out, t) for t in (x.data, w.data, bias, x.mean, x.rstd, w.sums) if t is not None):
        _refuse("out lies apart from what is read")
    if _current_device() != w._index:
        with torch.cuda.device(w._index):
            return product(x, w, bias, dtype, normalized, out)
    B.clef_fp4_product(x.struct, w.struct, None if bias is None else bias.data_ptr(),
                       x.mean.data_ptr() if normalized else None, x.rstd.data_ptr() if normalized else None,
                       w.sums.data_ptr() if normalized else None, _DTYPES[dtype], out.data_ptr(), max(_row_stride(out), w.rows),
                       w.flags.data_ptr(), _raw_stream(w._index))
    return out


class Fp4Linear:
    """A linear layer of 4-bit weights: its inputs are quantised row by row as they come.

    ``weight`` [outs, cols] (bf16, fp16 or fp32; or an ``Fp4Matrix``, quantised with ``sums`` where
    ``normalized`` is to be called) and ``bias`` [outs] (kept as it is where it is contiguous fp32) are laid out once; ``bias``
    may be set anew, the weight is one for the layer's life.  For ``normalized`` the weight
    holds the LayerNorm's weight (its columns times it) and the bias what the LayerNorm's bias brings.
    Both are frozen: parameters get no gradient through the layer."""

    def __init__(self, weight, bias: Optional[torch.Tensor] = None, format: str = "nvfp4"):
        if not isinstance(weight, Fp4Matrix):
            if _dual(weight):
                _refuse("weight: without a tangent")
            weight = quantize(weight.detach(), format, sums=True)
        elif weight.format != format:
            _refuse("weight: an Fp4Matrix of the format")
        self._weight, self.format = weight, format
        self.cols, self.outs = weight.cols, weight.rows
        self._device, self._index = weight.device, weight._index
        self.bias = bias
        self._flags = weight.flags.data_ptr()  # made here, outside of any later capture
        self._lib, self._struct = B.load(), weight.struct
        self._scratch = {}  # scratch bytes of the calls that the layer has met

    @property
    def weight(self) -> Fp4Matrix:
        return self._weight

    @property
    def bias(self) -> Optional[torch.Tensor]:
        """fp32 [outs], or None.  May be set, but not for graphs that have been captured: those keep the old one's address."""
        return self._bias_held

    @bias.setter
    def bias(self, bias: Optional[torch.Tensor]):
        if bias is not None:
            if bias.shape != (self.outs,) or bias.device != self._device or _dual(bias):
                _refuse("bias: [outs] on the weight's device, without a tangent")
            bias = bias.detach().to(_FP32).contiguous()
        self._bias_held, self._bias = bias, None if bias is None else bias.data_ptr()

    def _run(self, x, dtype, normalized):
        """Outputs, means and rstds of x's rows (the latter None where not ``normalized``)."""
        types, shape = _TYPES.get((x.dtype, dtype)), x.shape
        if types is None:
            _refuse("inputs and outputs: bf16, fp16 or fp32")
        if x.get_device() != self._index or not shape or shape[-1] != self.cols:
            _refuse(f"x: [..., {self.cols}] on the weight's device")
        if (x.requires_grad and torch.is_grad_enabled()) or _dual(x):
            _refuse("x requires a gradient, which a 4-bit layer does not pass on")
        rows = x if len(shape) == 2 else x.reshape(-1, self.cols)
        stride, step = rows.stride()
        if step != 1 and self.cols > 1:
            rows = rows.contiguous()
            stride = self.cols
        n = rows.shape[0]
        x_type, out_type, dtype = types
        if _current_device() != self._index:
            with torch.cuda.device(self._index):
                return self._run(x, dtype, normalized)
        y = torch.empty((n, self.outs), dtype=dtype, device=self._device)
        mean = rstd = mean_at = rstd_at = sums_at = None
        if normalized:
            if self._weight.sums is None:
                _refuse("normalized: the weight has no sums")
            mean = torch.empty(n, dtype=_FP32, device=self._device)
            rstd = torch.empty(n, dtype=_FP32, device=self._device)
            mean_at, rstd_at, sums_at = mean.data_ptr(), rstd.data_ptr(), self._weight.sums.data_ptr()
        if n:
            at, scratch = rows.data_ptr(), None
            stride = stride if n > 1 else self.cols
            few = n <= 16  # may go in one launch, which depends on whether a graph is being captured
            key = (n, x_type, normalized, (at | stride * x.element_size()) & 15 == 0, few and _capturing())
            size = self._scratch.get(key)
            if size is None:
                if len(self._scratch) >= 4096:
                    self._scratch.clear()
                size = self._scratch[key] = B.clef_fp4_linear_scratch(self._struct.format, x_type, n, self.cols, *key[2:4],
                                                                      self.outs, key[4])
            if size:  # a buffer of the call's own: overlapping calls and captured graphs never share one
                space = torch.empty(size, dtype=torch.uint8, device=self._device)
                scratch = space.data_ptr()
            status = self._lib.clef_fp4_linear(
                self._struct, x_type, at, stride, n, self._bias, sums_at, out_type, y.data_ptr(), self.outs, mean_at,
                rstd_at, scratch, size, self._flags, _raw_stream(self._index))
            if status:
                raise B.ClefError(status, "clef_fp4_linear")
        if len(shape) != 2:
            y = y.view(*shape[:-1], self.outs)
            if normalized:
                mean, rstd = mean.view(shape[:-1]), rstd.view(shape[:-1])
        return y, mean, rstd

    def __call__(self, x: torch.Tensor, dtype=None) -> torch.Tensor:
        """x [..., cols] (bf16, fp16 or fp32) through the layer: [..., outs] in ``dtype`` (x's own by default)."""
        return self._run(x, dtype, False)[0]

    def normalized(self, x: torch.Tensor, dtype=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
        """The layer behind a LayerNorm: outputs, and the rows' mean and 1 / sqrt(variance + 1e-5) (fp32 [...])."""
        return self._run(x, dtype, True)

    def device_status(self) -> int:
        """Waits for the current stream, reads and clears what the layer's products reported."""
        return self._weight.device_status()
