"""Torch-side convenience around the packed-row operators of the C ABI (include/zero_packed.h):
describes torch tensors to the library, allocates results and workspaces with torch and passes
torch's current HIP stream.  The work runs in libzero_shard.so; this module only marshals arguments."""

import torch

from . import _abi as abi

_DT = {torch.float16: abi.ZERO_F16, torch.bfloat16: abi.ZERO_BF16, torch.float32: abi.ZERO_F32}


def matrix(t, name, device=None):
    """zero_matrix_t of a 2-D tensor (or 1-D: one row) whose rows are consecutive elements."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} is {type(t).__name__}, not a tensor")
    if t.layout is not torch.strided or t.dtype not in _DT:
        raise ValueError(f"{name}: need a dense float16, bfloat16 or float32 tensor, got {t.dtype}, {t.layout}")
    if t.is_neg():
        raise ValueError(f"{name}: a lazily negated view; resolve_neg() it first")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the packed rows are on {device}")
    if t.dim() == 1:
        rows, cols, pitch, step = 1, t.shape[0], t.shape[0], t.stride(0)
    elif t.dim() == 2:
        rows, cols = t.shape
        pitch, step = t.stride()
    else:
        raise ValueError(f"{name}: need a matrix, got {t.dim()} dimensions")
    if rows > 1 and cols > 0 and (pitch < cols or (cols > 1 and step != 1)) or (rows == 1 and cols > 1 and step != 1):
        raise ValueError(f"{name}: shape {tuple(t.shape)} with strides {t.stride()} is not rows of consecutive elements; "
                         "make it contiguous first")
    return abi.zero_matrix_t(t.data_ptr(), rows, cols, max(pitch, cols), _DT[t.dtype])


class ZeroPacked:
    """A matrix [rows, cols] in packed rows: 8-bit integers `q` and one fp32 `scale` for each row, of which it stands for
    the products.  Rows are tokens (a layer's input, kept for its backward pass) or output channels (a layer's weights).

    `q` (int8, [rows, cols], its rows 16 bytes apart or a multiple) and `scale` ([rows]) are torch tensors that the object
    keeps; until a zero_packed_write or zero_packed_act they hold nothing.  rule: how the scales are chosen, ZERO_SCALE_POW2
    or ZERO_SCALE_MAX.

    Tensors given to the calls are matrices on the same GPU whose rows are consecutive elements, at any pitch; what a
    call writes must not overlap what it reads.  Calls use the current stream of that GPU, allocate results (unless out is
    given) and workspaces there, and write behind autograd's back, as into detached tensors.  As with any torch call,
    tensors used on another stream than the one they were allocated on must be kept until that stream is done with them,
    and tensors and packed rows used in a captured graph until its last replay is done.  Two calls that run at the same
    time must not write the same rows."""

    def __init__(self, rows, cols, rule=abi.ZERO_SCALE_POW2, device="cuda"):
        if rows < 0 or cols < 0:
            raise ValueError(f"rows and cols must not be negative, got {rows}, {cols}")
        device = torch.device(device)
        if device.type != "cuda":
            raise ValueError(f"packed rows are on a GPU, not on {device}")
        pitch = max(16, (cols + 15) // 16 * 16)
        self._set(torch.empty(rows, pitch, dtype=torch.int8, device=device),
                  torch.empty(rows, dtype=torch.float32, device=device), cols, rule)

    @classmethod
    def of(cls, q, scale, cols=None, rule=abi.ZERO_SCALE_POW2):
        """Packed rows that are there already: q int8 [rows, pitch], of which the first `cols` (all) count and the rest up to
        the next multiple of 16 are zeros; its rows begin on 16-byte boundaries.  scale fp32 [rows], contiguous."""
        if not (isinstance(q, torch.Tensor) and isinstance(scale, torch.Tensor)):
            raise ValueError("q and scale must be tensors")
        if q.dtype != torch.int8 or q.dim() != 2 or (q.shape[1] > 1 and q.stride(1) != 1):
            raise ValueError("q must be an int8 matrix whose rows are consecutive elements")
        if q.is_neg():
            raise ValueError("q: a lazily negated view; resolve_neg() it first")
        cols = q.shape[1] if cols is None else cols
        if scale.dtype != torch.float32 or scale.shape != q.shape[:1] or not scale.is_contiguous() or scale.is_neg():
            raise ValueError(f"scale must be {q.shape[0]} contiguous float32 values")
        if q.device != scale.device or q.device.type != "cuda":
            raise ValueError(f"q is on {q.device}, scale on {scale.device}; both must be on one GPU")
        if cols < 0 or (cols + 15) // 16 * 16 > q.shape[1]:
            raise ValueError(f"rows of {cols} columns need {(cols + 15) // 16 * 16} bytes, q's have {q.shape[1]}")
        p = cls.__new__(cls)
        p._set(q, scale, cols, rule)
        return p

    def _set(self, q, scale, cols, rule):
        if rule not in (abi.ZERO_SCALE_POW2, abi.ZERO_SCALE_MAX):
            raise ValueError("rule must be ZERO_SCALE_POW2 or ZERO_SCALE_MAX")
        pitch = q.stride(0) if q.shape[0] > 1 else max(16, (cols + 15) // 16 * 16)
        self._q, self.q, self.scale, self.rule = q, q[:, :cols], scale, rule
        self.rows, self.cols, self.device = q.shape[0], cols, q.device
        self._desc = abi.zero_packed_t(q.data_ptr(), scale.data_ptr(), self.rows, cols, pitch, rule)

    def __getitem__(self, rows):
        """The rows of a slice (step 1), as packed rows of their own on the same memory."""
        if not isinstance(rows, slice) or rows.step not in (None, 1):
            raise ValueError("rows are taken by a slice of step 1")
        return ZeroPacked.of(self._q[rows], self.scale[rows], self.cols, self.rule)

    @property
    def nbytes(self):
        """Bytes of device memory of the rows and their scales."""
        return self.rows * (self._desc.pitch + 4)

    def _run(self, call, *args):
        """Calls the library on this device, with torch's current stream there."""
        i = self.device.index
        if torch.cuda.current_device() == i:
            return call(*args, torch._C._cuda_getCurrentRawStream(i))
        with torch.cuda.device(i):
            return call(*args, torch._C._cuda_getCurrentRawStream(i))

    def _product(self, which, m, k, n, call, *args):
        need = abi.zero_packed_workspace(which, m, k, n)
        ws = torch.empty(need, dtype=torch.uint8, device=self.device) if need else None
        return self._run(call, *args, ws.data_ptr() if need else None, need)

    def _result(self, out, rows, cols, dtype):
        if out is None:
            if dtype not in _DT:
                raise ValueError(f"dtype must be float16, bfloat16 or float32, got {dtype}")
            return torch.empty(rows, cols, dtype=dtype, device=self.device)
        return out

    def _other(self, p, name):
        if not isinstance(p, ZeroPacked):
            raise ValueError(f"{name} is {type(p).__name__}, not ZeroPacked")
        if p.device != self.device:
            raise ValueError(f"{name} is on {p.device}, these packed rows are on {self.device}")
        return p._desc

    # calls of the C ABI, under its names
    def zero_packed_write(self, x):
        """Packs x [rows, cols] into these rows."""
        self._run(abi.zero_packed_write, matrix(x, "x", self.device), self._desc)
        return self

    def zero_packed_read(self, out=None, dtype=torch.bfloat16):
        """The values, into out or a new tensor of `dtype`."""
        out = self._result(out, self.rows, self.cols, dtype)
        self._run(abi.zero_packed_read, self._desc, matrix(out, "out", self.device))
        return out

    def zero_packed_linear(self, w, bias=None, out=None, dtype=torch.bfloat16):
        """y = x w^T + bias, in 8-bit integers: these rows are x [m, k], w is packed [n, k]; bias has n elements."""
        wd = self._other(w, "w")
        out = self._result(out, self.rows, w.rows, dtype)
        self._product(abi.ZERO_PACKED_LINEAR, self.rows, self.cols, w.rows, abi.zero_packed_linear, self._desc, wd,
                      None if bias is None else matrix(bias, "bias", self.device), matrix(out, "out", self.device))
        return out

    def zero_packed_weight_grad(self, dy, out=None, accumulate=False, dtype=torch.float32, bias_grad=None):
        """dw [n, k] = dy^T x, these rows being x [m, k], the layer's packed input, and dy [m, n] (16-bit); bias_grad (n
        elements) receives dy's column sums.  accumulate: added to what out and bias_grad hold."""
        if accumulate and out is None:
            raise ValueError("accumulate needs out")
        d = matrix(dy, "dy", self.device)
        out = self._result(out, d.cols, self.cols, dtype)
        self._product(abi.ZERO_PACKED_WEIGHT_GRAD, d.rows, self.cols, d.cols, abi.zero_packed_weight_grad, d, self._desc,
                      matrix(out, "out", self.device),
                      None if bias_grad is None else matrix(bias_grad, "bias_grad", self.device), accumulate)
        return out

    def zero_packed_input_grad(self, dy, out=None, accumulate=False, dtype=None):
        """dx [m, k] = dy w, these rows being w [n, k], the layer's packed weights, and dy [m, n] (16-bit).  accumulate: added
        to what out holds.  dtype: dy's unless given."""
        if accumulate and out is None:
            raise ValueError("accumulate needs out")
        d = matrix(dy, "dy", self.device)
        out = self._result(out, d.rows, self.cols, dtype or dy.dtype)
        self._product(abi.ZERO_PACKED_INPUT_GRAD, d.rows, self.cols, d.cols, abi.zero_packed_input_grad, d, self._desc,
                      matrix(out, "out", self.device), accumulate)
        return out

    def zero_packed_act(self, x, kind, gated=False, out=None, packed=None, dtype=None):
        """Activation function of x, kept here for its gradient: these rows receive x packed.  gated: x [m, 2n] holds the
        gate and the factor side by side.  The result goes into `packed` (packed rows [m, n]) and/or out; without packed,
        a new tensor of `dtype` (x's) is made for it.  Returns the tensor, or packed if there is none."""
        d = matrix(x, "x", self.device)
        n = d.cols // 2 if gated else d.cols
        if out is None and (packed is None or dtype is not None):
            out = self._result(None, d.rows, n, dtype or x.dtype)
        self._run(abi.zero_packed_act, kind, gated, d, self._desc, None if out is None else matrix(out, "out", self.device),
                  None if packed is None else self._other(packed, "packed"))
        return packed if out is None else out

    def zero_packed_act_grad(self, dy, kind, gated=False, out=None, dtype=None):
        """dx (of these rows' size) from dy and the packed input that zero_packed_act left here.  dtype: dy's unless given;
        out may be dy itself unless gated."""
        d = matrix(dy, "dy", self.device)
        out = self._result(out, self.rows, self.cols, dtype or dy.dtype)
        self._run(abi.zero_packed_act_grad, kind, gated, self._desc, d, matrix(out, "out", self.device))
        return out
