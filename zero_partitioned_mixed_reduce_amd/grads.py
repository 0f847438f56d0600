"""Torch-side convenience around the gradient-list operators of the C ABI
(include/zero_grads.h): describes torch tensors to the library, allocates the
workspace with torch and passes torch's current HIP stream.  The work runs in
libzero_shard.so; this module only marshals arguments."""
import operator

import torch

from . import _abi as abi

_dtype = operator.attrgetter("dtype")
_DT = {torch.float16: abi.ZERO_F16, torch.bfloat16: abi.ZERO_BF16, torch.float32: abi.ZERO_F32}


def _runs(shape, *strides):
    """A tensor's dimensions merged into (rows, cols, pitch, ...) with one pitch per stride list, in the order of
    the dimensions given, or None when they do not merge into rows of consecutive elements."""
    dims = []
    for n, *st in zip(shape, *strides):
        if n == 1:
            continue
        if dims and all(p == n * s for p, s in zip(dims[-1][1], st)):
            dims[-1] = (dims[-1][0] * n, st)
        else:
            dims.append((n, st))
    if not dims:
        return (1, 1) + (1,) * len(strides)
    if any(s != 1 for s in dims[-1][1]):
        dims.append((1, [1] * len(strides)))   # every element a row of its own
    if len(dims) == 1:
        return (1, dims[0][0]) + (dims[0][0],) * len(strides)
    if len(dims) > 2 or any(p < dims[1][0] for p in dims[0][1]):
        return None
    return (dims[0][0], dims[1][0]) + tuple(dims[0][1])


def describe(i, src, dst):
    """zero_grads_tensor_t of list entry i; dst None: in place."""
    if src.layout is not torch.strided or src.dtype not in _DT:
        raise ValueError(f"tensor {i}: need a dense float16, bfloat16 or float32 tensor, got {src.dtype}, {src.layout}")
    if dst is not None and (dst.layout is not torch.strided or dst.dtype not in _DT):
        raise ValueError(f"out {i}: need a dense float16, bfloat16 or float32 tensor, got {dst.dtype}, {dst.layout}")
    if src.is_neg() or (dst is not None and dst.is_neg()):
        raise ValueError(f"tensor {i}: a lazily negated view; resolve_neg() it first")
    if dst is not None and dst.numel() != src.numel():
        raise ValueError(f"out {i} has {dst.numel()} elements, tensor {i} has {src.numel()}")
    t = abi.zero_grads_tensor_t()
    t.src, t.src_dtype = src.data_ptr(), _DT[src.dtype]
    if dst is not None:
        t.dst, t.dst_dtype = dst.data_ptr(), _DT[dst.dtype]
    if src.numel() == 0:
        t.rows, t.cols = 1, 0
        return t
    if src.is_contiguous() and (dst is None or dst.is_contiguous()):
        t.rows, t.cols, t.src_pitch, t.dst_pitch = 1, src.numel(), src.numel(), src.numel()
        return t
    if dst is None or (src.shape == dst.shape and src.stride() == dst.stride()):
        # element for element: any order of the dimensions serves, so take the order of memory
        order = sorted(range(src.dim()), key=lambda k: -src.stride(k))
        r = _runs([src.shape[k] for k in order], [src.stride(k) for k in order])
        r = r and r + (r[2],)
    elif src.shape == dst.shape:
        r = _runs(src.shape, src.stride(), dst.stride())
    elif dst.is_contiguous():
        r = _runs(src.shape, src.stride())
        r = r and r + (r[1],)
    else:
        r = None
    if r is None:
        raise ValueError(f"tensor {i}: shape {tuple(src.shape)} with strides {src.stride()}"
                         + (f" into strides {dst.stride()}" if dst is not None else "")
                         + " is not rows of consecutive elements at one pitch; make it contiguous first")
    t.rows, t.cols, t.src_pitch, t.dst_pitch = r
    return t


class _Layout:
    """What the tensors of a list have to have in common with those bound in their places later: the device, dtypes and
    sizes, and for one that is not contiguous its shape and strides; none may be a lazily negated view.  Each property
    of all tensors is read by one map rather than in a loop over the tensors (5 to 8 us a property for 150 of them)."""

    def __init__(self, tensors):
        self.n, self.device = len(tensors), [tensors[0].get_device()] * len(tensors)
        self.dtype, self.numel = list(map(_dtype, tensors)), list(map(torch.Tensor.numel, tensors))
        self.dense = list(map(torch.Tensor.is_contiguous, tensors))
        self.strided = [(i, t.shape, t.stride()) for i, t in enumerate(tensors) if not self.dense[i]]

    def addresses(self, tensors, what):
        if len(tensors) != self.n:
            raise ValueError(f"the plan has {self.n} tensors, got {len(tensors)} {what}")
        try:
            same = (list(map(_dtype, tensors)) == self.dtype and list(map(torch.Tensor.numel, tensors)) == self.numel
                    and list(map(torch.Tensor.get_device, tensors)) == self.device
                    and list(map(torch.Tensor.is_contiguous, tensors)) == self.dense
                    and all(tensors[i].shape == shape and tensors[i].stride() == stride for i, shape, stride in self.strided))
            negated = True in map(torch.Tensor.is_neg, tensors)
            at = list(map(torch.Tensor.data_ptr, tensors))
        except (AttributeError, TypeError, RuntimeError) as e:   # no tensor, or one without strides or an address
            raise ValueError(f"{what}: one of them is not a dense tensor ({e})") from None
        if not same:
            raise ValueError(f"{what}: dtype, sizes, strides or device of one of them differ from the plan's")
        if negated:
            raise ValueError(f"{what}: one of them is a lazily negated view; resolve_neg() it first")
        return at


class ZeroGrads:
    """Norm, clipping and scaling of one list of gradients.

    tensors: CUDA tensors of one device, fp16, bf16 or fp32 in any mixture; contiguous, or slices whose elements
    form rows at one pitch.  A parameter without a gradient is left out, or stands there as a tensor of zeros where
    its place in a flat out has to be filled.  out: None (in place), one tensor per gradient with as many elements,
    or one flat contiguous tensor that takes them back to back in list order (e.g. a rank's buffer for
    zero_reduce_grads).
    The tensors' addresses are the plan's; zero_grads_bind gives new ones.

    After a norm, `norm` (0-dim) and, with per_tensor, `norms` [n] are fp32 device tensors in the workspace,
    `found_inf` (int32), `acc` and `tensor_acc` (fp64) likewise; they hold the handle's latest results.

    Results in place are written behind autograd's back, as into detached tensors.

    Calls use the current stream of the tensors' device, and the handle keeps the tensors alive until it is bound
    to others or closed, and those bound in a captured graph until it is closed; a captured graph needs the handle,
    whose workspace it uses, until its last replay is done, and binds its list whenever it is replayed.  The workspace
    may be used on any stream; as with any torch call, tensors used on another stream than the one they were allocated
    on must be kept until that stream is done with them."""

    def __init__(self, tensors, out=None):
        self._tensors = list(tensors)
        if not self._tensors:
            raise ValueError("an empty list")
        if out is not None and not isinstance(out, torch.Tensor):
            out = list(out)
        self._in_place = out is None
        dsts = self._check(self._tensors, out)
        self._out = out
        self._in_graphs = []                    # lists bound in captures: (tensors, out)
        self.device = self._tensors[0].device   # with its index
        desc = (abi.zero_grads_tensor_t * len(self._tensors))(
            *[describe(i, s, d) for i, (s, d) in enumerate(zip(self._tensors, dsts))])
        self._layout = _Layout(self._tensors)
        self._flat = isinstance(out, torch.Tensor)
        self._out_layout = None if out is None else _Layout([out] if self._flat else dsts)
        if self._flat:
            size, at = out.element_size(), 0
            self._offsets = []
            for t in self._tensors:
                self._offsets.append(at)
                at += t.numel() * size
        self.info = abi.zero_grads_plan(desc)
        self.h = None
        with torch.cuda.device(self.device):
            self.workspace = torch.empty(self.info.workspace_bytes, dtype=torch.uint8, device=self.device)
            self._streams = {torch._C._cuda_getCurrentRawStream(self.device.index)}   # that the workspace knows of
            self.h = abi.zero_grads_init(desc, self.workspace.data_ptr(), self.info.workspace_bytes, self._stream())
        n = len(self._tensors)
        base = self.workspace.data_ptr()
        views = []
        for ptr, size, dt in zip(abi.zero_grads_device(self.h), (8, 4, 4, 8 * n, 4 * n),
                                 (torch.float64, torch.int32, torch.float32, torch.float64, torch.float32)):
            views.append(self.workspace[ptr - base:ptr - base + size].view(dt))
        self.acc, self.found_inf, self.norm = (v[0] for v in views[:3])
        self.tensor_acc, self.norms = views[3:]

    def _check(self, tensors, out):
        """Checks a list and returns its destinations, one per tensor (None: in place)."""
        for i, t in enumerate([*tensors, *(out if isinstance(out, list) else [])]):
            if not isinstance(t, torch.Tensor):
                raise ValueError(f"tensor {i} of the list is {type(t).__name__}, not a tensor")
        dev = tensors[0].device
        for i, t in enumerate(tensors):
            if t.device.type != "cuda" or t.device != dev:
                raise ValueError(f"tensor {i} is on {t.device}; the list is on {dev}, and must be on one GPU")
        if out is None:
            return [None] * len(tensors)
        if isinstance(out, torch.Tensor):
            total = sum(t.numel() for t in tensors)
            if out.numel() != total or not out.is_contiguous():
                raise ValueError(f"a flat out must be contiguous with the list's {total} elements")
            out, at = out.view(-1), 0
            dsts = []
            for t in tensors:
                dsts.append(out[at:at + t.numel()])
                at += t.numel()
        else:
            dsts = out
            if len(dsts) != len(tensors):
                raise ValueError(f"{len(tensors)} tensors, {len(dsts)} out tensors")
        for i, t in enumerate(dsts):
            if t.device != dev:
                raise ValueError(f"out {i} is on {t.device}, the list on {dev}")
        return dsts

    def _stream(self):
        stream = torch._C._cuda_getCurrentRawStream(self.device.index)
        if stream not in self._streams:         # the workspace's memory is free when this one is done with it, too
            self.workspace.record_stream(torch.cuda.current_stream(self.device))
            self._streams.add(stream)
        return stream

    def _capturing(self):
        if torch.cuda.current_device() == self.device.index:
            return torch.cuda.is_current_stream_capturing()
        with torch.cuda.device(self.device):
            return torch.cuda.is_current_stream_capturing()

    # calls of the C ABI, under its names
    def zero_grads_bind(self, tensors, out=None):
        """The list's tensors at new addresses: the same dtypes, shapes and strides.  In a capture: whenever the graph is
        replayed, for the calls behind it."""
        tensors = list(tensors)
        if (out is None) != self._in_place:
            raise ValueError("the plan is in place: bind without out" if self._in_place
                             else "the plan is not in place: bind with out")
        if isinstance(out, torch.Tensor) != self._flat:
            raise ValueError("out is one flat tensor in the plan or a list in the plan, and not the other here")
        src, dst = self._layout.addresses(tensors, "tensors"), None
        if self._flat:
            base = self._out_layout.addresses([out], "out")[0]
            dst = [base + o for o in self._offsets]
        elif out is not None:
            out = list(out)
            dst = self._out_layout.addresses(out, "out tensors")
        abi.zero_grads_bind(self.h, src, dst, self._stream())
        if self._capturing():                   # bound when the graph is replayed, and not now
            self._in_graphs.append((tensors, out))
        else:
            self._tensors, self._out = tensors, out

    def zero_grads_norm(self, norm=abi.ZERO_NORM_L2, inv_loss_scale=1.0, per_tensor=False):
        abi.zero_grads_norm(self.h, norm, inv_loss_scale, per_tensor, self._stream())

    def zero_grads_clip(self, max_norm, scope=abi.ZERO_CLIP_GLOBAL, other_ranks_found_inf=False, other_ranks_acc=0.0):
        abi.zero_grads_clip(self.h, scope, other_ranks_found_inf, other_ranks_acc, max_norm, self._stream())

    def zero_grads_clip_norm(self, max_norm, norm=abi.ZERO_NORM_L2, inv_loss_scale=1.0, scope=abi.ZERO_CLIP_GLOBAL,
                             per_tensor=False):
        """Norm and clip in one call, for a list that no other rank shares."""
        abi.zero_grads_clip_norm(self.h, norm, inv_loss_scale, per_tensor, scope, max_norm, self._stream())

    def zero_grads_scale(self, factor):
        abi.zero_grads_scale(self.h, factor, self._stream())

    def query(self):
        """What the last clip used: dict(norm, found_inf, coef).  Synchronises the current stream.  ZERO_ESTATE if it
        found no norm of these values (replays of captured calls included) and so wrote nothing."""
        return abi.zero_grads_query(self.h, self._stream())

    def close(self):
        if self.h:
            abi.zero_grads_destroy(self.h)
            self.h = None
        self._tensors, self._out, self._in_graphs = [], None, []

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
