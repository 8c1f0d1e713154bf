"""The operators around the experts' products, on GPU tensors (include/moe.h defines them):

* ``rms_norm`` and ``rms_norm_backward``: the block's norm with the residual stream's addition, as activations, as MX-FP8
  rows for ``mx8_gemm``, or as both;
* ``select_experts`` and ``select_experts_backward``: the choice of experts from router logits under a ``RouterRule``;
* ``swiglu_checkpoint`` and ``swiglu_backward``: the experts' activation, with its inputs kept in 8 bits for the backward pass;
* ``mx8_quantize``, ``mx8_dequantize``: MX-FP8 rows and back; ``mx8_gemm``: their product with MX-FP4 weights
  (``runner.mx_quantize``), grouped by expert.

Every call works on its tensors' device and that device's current stream, allocates its outputs and scratch with torch's
allocator (so that it can be captured, and calls on several streams share nothing), and raises ValueError or TypeError for
tensors that do not fit, ``binding.MoeError`` for sizes that the library refuses.
"""

import functools
from dataclasses import dataclass, field

import torch

from . import binding as B
from .runner import _DTYPE, MxRows, ScaledRows, _on, _row_stride


def _mx8_strides(cols):
    """B.mx8_strides without the call (it also refuses what that refuses)."""
    if cols <= 0 or cols % 32 or cols > 1 << 24:
        return B.mx8_strides(cols)
    return cols, (cols // 32 + 15) // 16 * 16


class Mx8Rows(ScaledRows):
    """Rows of `cols` MX-FP8 values on the GPU (include/moe.h describes the format):
    codes [..., rows, cols] and scales [..., rows, cols / 32 rounded up to 16], uint8."""

    _strides = staticmethod(_mx8_strides)

    @property
    def shape(self):
        return tuple(self._codes.shape)   # a byte a value

    @classmethod
    def empty(cls, shape, device):
        """Rows of the given shape [..., rows, cols], not yet written."""
        cb, sb = _mx8_strides(shape[-1])
        codes = torch.empty(shape, dtype=torch.uint8, device=device)
        scales = torch.empty((*shape[:-1], sb), dtype=torch.uint8, device=device)
        return cls._made(codes, scales, shape[-1], cb, sb, (codes.data_ptr(), scales.data_ptr()))


def _code(t, what):
    c = _DTYPE.get(t.dtype)
    if c is None:
        raise TypeError(f"{what} is {t.dtype}, not bf16 or fp32")
    return c


def _like(t, shape, dtype, device, what):
    """A tensor of the caller's, checked."""
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{what} {tuple(t.shape)} {t.dtype}, expected {tuple(shape)} {dtype}")
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, not on {device}")


def _bytes(t, what):
    """Bytes from row to row of t [..., rows, cols]."""
    if t.is_contiguous() and t.dim() >= 2:
        return t.shape[-1] * t.itemsize
    return _row_stride(t, what) * t.itemsize


def _new(t):
    """A contiguous tensor like t."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _vector(t, n, device, what):
    if t.shape != (n,) or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{what} must be contiguous [{n}] on {device}")


def _counts(counts, groups, device):
    if counts is not None:
        if counts.dtype != torch.int32 or counts.shape != (groups,) or not counts.is_contiguous():
            raise ValueError("counts is a contiguous int32 tensor with one value a group")
        if counts.device != device:
            raise ValueError(f"counts is on {counts.device}, not on {device}")


def _eight(q, what):
    if not isinstance(q, Mx8Rows):
        raise TypeError(f"{what} is {type(q).__name__}, not Mx8Rows")
    return q


# ---------------------------------------------------------------- MX-FP8 rows

def mx8_quantize(x):
    """x [..., rows, cols] (bf16 or fp32, evenly spaced rows) as Mx8Rows."""
    code = _code(x, "x")
    st, dev = _on(x)
    ld = _bytes(x, "x")
    with dev:
        q = Mx8Rows.empty(x.shape, x.device)
        B.mx8_quantize(code, x.numel() // q.cols, q.cols, x, ld, q.arg, st)
    return q


def mx8_dequantize(q, dtype=torch.bfloat16):
    """The values of Mx8Rows q as a bf16 or fp32 tensor."""
    code = _DTYPE.get(dtype)
    if code is None:
        raise TypeError(f"mx8_dequantize gives bf16 or fp32, not {dtype}")
    st, dev = _on(_eight(q, "q").codes)
    with dev:
        out = torch.empty_like(q.codes, dtype=dtype, memory_format=torch.contiguous_format)
        B.mx8_dequantize(code, out.numel() // q.cols, q.cols, q.arg, out, q.cols * out.itemsize, st)
    return out


def mx8_gemm(a, b, counts=None, out=None, dtype=torch.bfloat16):
    """out[g] = a[g] . b[g]^T of Mx8Rows a [G, M, K] and runner.MxRows b [G, N, K] (or [M, K] and [N, K]) as bf16 or fp32.
    counts: int32 [G] rows of each group (the rows of `out` behind them are left as they were; a new `out` has zeros there)."""
    if not (isinstance(a, Mx8Rows) and isinstance(b, MxRows)):
        raise TypeError(f"mx8_gemm takes Mx8Rows and MxRows, not {type(a).__name__} and {type(b).__name__}")
    ca, cb = a.codes, b.codes
    sa, sb = ca.shape, cb.shape
    if len(sa) != len(sb) or len(sa) not in (2, 3) or a.cols != b.cols or sa[:-2] != sb[:-2]:
        raise ValueError(f"mx8_gemm of rows {a.shape} and {b.shape}")
    G, M = _groups(sa)
    N = sb[-2]
    st, dev = _on(ca)
    _counts(counts, G, ca.device)
    if cb.device != ca.device:
        raise ValueError(f"b is on {cb.device}, not on {ca.device}")
    shape = sa[:-1] + (N,)
    with dev:
        if out is None:
            out = (torch.empty if counts is None else torch.zeros)(shape, dtype=dtype, device=ca.device)
        _like(out, shape, out.dtype, ca.device, "out")
        B.mx8_gemm(_code(out, "out"), G, M, N, a.cols, a.arg, counts, b.arg, out, _bytes(out, "out"), st)
    return out


# ---------------------------------------------------------------- norm

def rms_norm(x, weight, residual=None, eps=1e-6, form="act"):
    """(y, s): s = x + residual, rounded as x is (x itself without a residual), and its root-mean-square norm times weight.

    x and residual [..., rows, cols], bf16 or fp32, evenly spaced rows; weight [cols], bf16 or fp32.  form: "act" (y like x),
    "mx8" (y as Mx8Rows) or "both" ((y, Mx8Rows))."""
    if form not in ("act", "mx8", "both"):
        raise ValueError(f"form={form!r}: 'act', 'mx8' or 'both'")
    code, wcode = _code(x, "x"), _code(weight, "weight")
    st, dev = _on(x)
    ldx, ldr, cols = _bytes(x, "x"), 0, x.shape[-1]
    _vector(weight, cols, x.device, "weight")
    if residual is not None:
        _like(residual, x.shape, x.dtype, x.device, "residual")
        ldr = _bytes(residual, "residual")
    ld = cols * x.itemsize
    with dev:
        s = _new(x) if residual is not None else None
        y = _new(x) if form != "mx8" else None
        q = Mx8Rows.empty(x.shape, x.device) if form != "act" else None
        B.rms_norm(code, x.numel() // cols if cols else 0, cols, x, ldx, residual, ldr, weight, wcode, eps, s, ld, y, ld,
                   None if q is None else q.arg, st)
    return (y if q is None else q if y is None else (y, q)), (x if s is None else s)


_workspace_bytes = functools.lru_cache(maxsize=256)(B.rms_norm_workspace_size)


def rms_norm_backward(dy, s, weight, dstream=None, eps=1e-6):
    """(dx, dweight): the gradient of x (and of the residual) like dy, and the weight's in fp32.  s as rms_norm gave it; dstream:
    the gradient that reached s beside the norm."""
    code, wcode = _code(dy, "dy"), _code(weight, "weight")
    st, dev = _on(dy)
    cols = dy.shape[-1]
    _like(s, dy.shape, dy.dtype, dy.device, "s")
    _vector(weight, cols, dy.device, "weight")
    if dstream is not None:
        _like(dstream, dy.shape, dy.dtype, dy.device, "dstream")
    ldy, lds, ldt = _bytes(dy, "dy"), _bytes(s, "s"), 0 if dstream is None else _bytes(dstream, "dstream")
    rows = dy.numel() // cols if cols else 0
    with dev:
        dx = _new(dy)
        dweight = torch.empty((cols,), dtype=torch.float32, device=dy.device)
        ws = torch.empty((_workspace_bytes(rows, cols),), dtype=torch.uint8, device=dy.device)
        B.rms_norm_backward(code, rows, cols, dy, ldy, s, lds, weight, wcode, eps, dstream, ldt, dx, cols * dy.itemsize,
                            dweight, ws, st)
    return dx, dweight


# ---------------------------------------------------------------- choice of experts

_SCORES = {"softmax": B.MOE_SCORE_SOFTMAX, "sigmoid": B.MOE_SCORE_SIGMOID}


@dataclass(frozen=True, eq=False)
class RouterRule:
    """How a router's logits choose and weight experts (moe_router_rule in include/moe.h).  The rule itself does not change;
    balance, fp32 [E], is read at each call, so that a program can adjust it in place (runner.RaggedOneRankLayer keeps the one
    that it was made with)."""

    top_k: int
    score: str = "softmax"        # or "sigmoid"
    balance: torch.Tensor = None  # added to the scores for the choice alone
    groups: int = 1
    top_groups: int = 1
    group_best: int = 2           # a group's score is the sum of that many of its best (1 or 2)
    renormalise: bool = True
    scale: float = 1.0
    arg: B.RouterRuleArg = field(init=False, repr=False)

    def __post_init__(self):
        if self.score not in _SCORES:
            raise ValueError(f"score={self.score!r}: 'softmax' or 'sigmoid'")
        object.__setattr__(self, "arg", B.RouterRuleArg(_SCORES[self.score], self.groups, self.top_groups, self.group_best,
                                                        1 if self.renormalise else 0, self.scale))

    def __getstate__(self):
        return {k: v for k, v in self.__dict__.items() if k != "arg"}   # ctypes structures do not go into copies

    def __setstate__(self, state):
        self.__dict__.update(state)
        self.__post_init__()

    def choose(self, logits, idx, w, stream=None):
        """Writes the choice for logits [T, E] into idx [T, k] int32 and w [T, k] fp32 (contiguous)."""
        T, E = _logits(logits)
        for t, dtype, what in ((idx, torch.int32, "idx"), (w, torch.float32, "w")):
            _like(t, (T, self.top_k), dtype, logits.device, what)
            if not t.is_contiguous():
                raise ValueError(f"{what} must be contiguous")
        st, dev = _on(logits)
        with dev:
            self._choose(logits, T, E, idx, w, st if stream is None else stream)

    def _choose(self, logits, T, E, idx, w, stream):
        if self.balance is not None:
            if self.balance.dtype != torch.float32:
                raise ValueError(f"balance is {self.balance.dtype}, not fp32")
            _vector(self.balance, E, logits.device, "balance")
        B.select(self.arg, T, E, self.top_k, logits, _row_stride(logits, "logits"), self.balance, idx, w, stream)


def _logits(logits):
    if logits.dtype != torch.float32 or logits.dim() != 2:
        raise ValueError(f"logits {tuple(logits.shape)} {logits.dtype}: fp32 [T, E] is needed")
    return logits.shape


def select_experts(logits, rule):
    """(idx, w): the rule's choice of experts for each row of logits [T, E], int32 and fp32 [T, k]."""
    T, E = _logits(logits)
    st, dev = _on(logits)
    with dev:
        idx = torch.empty((T, rule.top_k), dtype=torch.int32, device=logits.device)
        w = torch.empty((T, rule.top_k), dtype=torch.float32, device=logits.device)
        rule._choose(logits, T, E, idx, w, st)
    return idx, w


def select_experts_backward(dw, w, idx, logits, rule):
    """The gradient of the logits, fp32 [T, E], from that of the weights."""
    T, E = _logits(logits)
    st, dev = _on(logits)
    for t, dtype, what in ((dw, torch.float32, "dw"), (w, torch.float32, "w"), (idx, torch.int32, "idx")):
        _like(t, (T, rule.top_k), dtype, logits.device, what)
    with dev:
        dlogits = torch.empty((T, E), dtype=torch.float32, device=logits.device)
        B.select_backward(rule.arg, T, E, rule.top_k, dw.contiguous(), w.contiguous(), idx.contiguous(), logits,
                          _row_stride(logits, "logits"), dlogits, E, st)
    return dlogits


# ---------------------------------------------------------------- SwiGLU

def _groups(shape):
    if len(shape) not in (2, 3):
        raise ValueError(f"rows [G, M, n] or [M, n] are needed, not {tuple(shape)}")
    return (shape[0] if len(shape) == 3 else 1), shape[-2]


def swiglu_checkpoint(gate_up, counts=None, out=None, saved=None):
    """(h, saved): h = silu(gate) * up of gate_up [G, M, 2 H] (or [M, 2 H]; H gate values, then H up values), and gate_up as
    Mx8Rows for swiglu_backward.  counts: int32 [G] rows of each group (the rows of `out` and `saved` behind them are left as
    they were; a new `out` has zeros there)."""
    code = _code(gate_up, "gate_up")
    G, M = _groups(gate_up.shape)
    H = gate_up.shape[-1] // 2
    if gate_up.shape[-1] % 64:
        raise ValueError(f"gate_up has {gate_up.shape[-1]} columns, not a multiple of 64")
    st, dev = _on(gate_up)
    _counts(counts, G, gate_up.device)
    shape = gate_up.shape[:-1] + (H,)
    with dev:
        if out is None:
            out = (torch.empty if counts is None else torch.zeros)(shape, dtype=gate_up.dtype, device=gate_up.device)
        _like(out, shape, gate_up.dtype, gate_up.device, "out")
        if saved is None:
            saved = Mx8Rows.empty(gate_up.shape, gate_up.device)
        elif _eight(saved, "saved").shape != tuple(gate_up.shape) or saved.codes.device != gate_up.device:
            raise ValueError(f"saved has rows {saved.shape} on {saved.codes.device}")
        B.swiglu_checkpoint(code, G, M, H, gate_up, _bytes(gate_up, "gate_up"), counts, out, _bytes(out, "out"), saved.arg, st)
    return out, saved


def swiglu_backward(dh, saved, counts=None, out=None, hidden=True, hidden_out=None):
    """(dgate_up, h): the gradient of gate_up from that of h [G, M, H] (or [M, H]) at the saved values, like dh, and (hidden) h
    again from the saved values, else None.  counts as in swiglu_checkpoint."""
    code = _code(dh, "dh")
    G, M = _groups(dh.shape)
    H = dh.shape[-1]
    shape = dh.shape[:-1] + (2 * H,)
    if _eight(saved, "saved").shape != tuple(shape) or saved.codes.device != dh.device:
        raise ValueError(f"saved has rows {saved.shape} on {saved.codes.device}, expected {tuple(shape)} on {dh.device}")
    st, dev = _on(dh)
    _counts(counts, G, dh.device)
    new = torch.empty if counts is None else torch.zeros
    with dev:
        if out is None:
            out = new(shape, dtype=dh.dtype, device=dh.device)
        _like(out, shape, dh.dtype, dh.device, "out")
        if hidden_out is None and hidden:
            hidden_out = new(dh.shape, dtype=dh.dtype, device=dh.device)
        if hidden_out is not None:
            _like(hidden_out, dh.shape, dh.dtype, dh.device, "hidden_out")
        B.swiglu_backward(code, G, M, H, dh, _bytes(dh, "dh"), saved.arg, counts, out, _bytes(out, "out"), hidden_out,
                          0 if hidden_out is None else _bytes(hidden_out, "hidden_out"), st)
    return out, hidden_out
