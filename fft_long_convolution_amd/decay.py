"""ctypes binding of linear attention with a decay for each head
(:class:`DecayAttention`) and of layer norm (:class:`LayerNorm`), two further
operators beside the long convolution (include/fftconv.h).

Argument marshalling only: every step runs in the HIP library.  PyTorch
supplies device memory and the current stream; calls raise if the library is
not built.

A layer uses them together, with :class:`~.delta.QKNorm` between them:

>>> norm = LayerNorm(768)
>>> attend = DecayAttention(128, 128)
>>> y = norm.forward(x, weight, bias)                  # then q, k, v from y
>>> o, state = attend.forward(q, k, v, g)              # a prompt
>>> o = attend.step(q1, k1, v1, g1, state)             # then token by token
"""
from __future__ import annotations

import ctypes

import torch

from .delta import _LL3, _check, _dense, _given, _like, _Op, _ptr, _strided
from .delta import lib as _mixer_lib
from .fftconv import DTYPES


class LayerNormDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("rows", ctypes.c_size_t), ("D", ctypes.c_size_t),
                ("eps", ctypes.c_float), ("x_stride", ctypes.c_longlong)]


class DecayDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("B", ctypes.c_size_t), ("T", ctypes.c_size_t),
                ("Hk", ctypes.c_size_t), ("Hv", ctypes.c_size_t), ("Dk", ctypes.c_size_t),
                ("Dv", ctypes.c_size_t), ("sequences", ctypes.c_size_t),
                ("scale", ctypes.c_float), ("fixed_decay", ctypes.c_int), ("q_stride", _LL3),
                ("k_stride", _LL3), ("v_stride", _LL3), ("clear_unheld", ctypes.c_int)]


_ready = None


def lib() -> ctypes.CDLL:
    """libfftconv.so with the signatures of this module's calls."""
    global _ready
    L = _mixer_lib()
    if _ready is not L:
        vp, sz, i = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
        nd, dd = ctypes.POINTER(LayerNormDesc), ctypes.POINTER(DecayDesc)
        for name, res, args in (
                ("fftconv_layernorm_forward", i, [nd] + [vp] * 5),
                ("fftconv_layernorm_workspace_bytes", sz, [nd]),
                ("fftconv_layernorm_backward", i, [nd] + [vp] * 7 + [sz, vp]),
                ("fftconv_decay_forward", i, [dd] + [vp] * 9 + [sz, vp]),
                ("fftconv_decay_workspace_bytes", sz, [dd]),
                ("fftconv_decay_backward", i, [dd] + [vp] * 14 + [sz, vp]),
                ("fftconv_decay_backward_workspace_bytes", sz, [dd]),
                ("fftconv_decay_step", i, [dd] + [vp] * 5 + [sz, vp, vp, vp])):
            fn = getattr(L, name)
            fn.restype, fn.argtypes = res, args
        _ready = L
    return L


class LayerNorm(_Op):
    """Layer norm of rows of D elements: y = weight (x - mean) / sqrt(var + eps)
    + bias, the mean and the variance those of the row.  weight and bias are fp32
    [D], or None for 1 and 0."""

    def __init__(self, D: int, eps: float = 1e-5, dtype: str = "bf16"):
        super().__init__(dtype)
        self._lib = lib()
        self.D, self.eps = D, eps

    @property
    def _settings(self):
        return "layernorm", self.D, self.eps, self.dtype

    def _rows(self, x, name):
        """x [..., D] as [rows, D]."""
        if x.dim() < 1 or x.shape[-1] != self.D or self.D < 1:
            raise ValueError("%s must be [..., %d]" % (name, self.D))
        return x if x.dim() == 2 else x.reshape(x.numel() // self.D, self.D)

    def _describe(self, x, weight, bias):
        if not x.is_cuda:
            raise ValueError("x must be a CUDA tensor")
        dev, rows = x.device, x.shape[0]
        _check(x, "x", x.shape, self._dt, dev)
        for name, w in (("weight", weight), ("bias", bias)):
            if w is not None:
                _check(w, name, (self.D,), torch.float32, dev)
        # rows one after the other, or the same distance apart
        if x.stride(1) != 1 and self.D > 1 or rows > 1 and x.stride(0) < self.D:
            x = x.clone(memory_format=torch.contiguous_format)
        desc = LayerNormDesc(DTYPES[self.dtype], rows, self.D, self.eps,
                             x.stride(0) if rows > 1 else self.D)
        ref = ctypes.byref(desc)
        need = self._lib.fftconv_layernorm_workspace_bytes(ref)
        return ((dev, ref, need), (x, None if weight is None else weight.contiguous(),
                                   None if bias is None else bias.contiguous()))

    def forward(self, x, weight=None, bias=None, out=None, stream=None):
        """x [..., D] (strided views are fine) -> y, contiguous."""
        (dev, ref, _), ins, ptrs = self._checked("_describe", (self._rows(x, "x"), weight, bias))
        if out is None:
            out = torch.empty(x.shape, dtype=self._dt, device=dev)
        else:
            _given(out, "out", x.shape, self._dt, dev)
        self._call(self._lib.fftconv_layernorm_forward, dev, stream, (*ins, out), ref, *ptrs,
                   out.data_ptr())
        return out

    def backward(self, x, dy, weight=None, bias=None, workspace=None, stream=None):
        """Gradients for dy = dL/dy: returns (dx, dweight, dbias), the last two
        fp32 [D], or None where there is no weight or bias."""
        (dev, ref, need), ins, ptrs = self._checked("_describe", (self._rows(x, "x"), weight, bias))
        _check(dy, "dy", x.shape, self._dt, dev)
        dy = _dense(dy)
        dx = torch.empty(x.shape, dtype=self._dt, device=dev)
        dw, db = (None if w is None else _like(w) for w in ins[1:])
        ws = None
        if dw is not None or db is not None:
            ws = self._space(need, workspace, dev, "workspace")
        self._call(self._lib.fftconv_layernorm_backward, dev, stream, (*ins, dy, dx, dw, db, ws),
                   ref, ptrs[0], ptrs[1], dy.data_ptr(), dx.data_ptr(), _ptr(dw), _ptr(db),
                   _ptr(ws), self._bytes(ws))
        return dx, dw, db


class DecayAttention(_Op):
    """Linear attention with a decay for each head of D_k x D_v: from a state S,
    each token does S <- e^g S + k v^T, o = scale S^T q.

    q, k [B, T, Hk, D_k] and v [B, T, Hv, D_v] (strided views are fine; Hv a
    multiple of Hk); g fp32, [B, T, Hv] or, for one log decay a head, [Hv];
    states are fp32 [rows, Hv, D_k, D_v].  scale defaults to D_k ** -0.5.
    """

    def __init__(self, D_k: int, D_v: int, dtype: str = "bf16", scale: float | None = None):
        super().__init__(dtype)
        self._lib = lib()
        self.D_k, self.D_v = D_k, D_v
        self.scale = D_k ** -0.5 if scale is None else float(scale)

    @property
    def _settings(self):
        return "decay", self.D_k, self.D_v, self.dtype, self.scale

    def _describe(self, q, k, v, g, cu_seqlens, initial_state):
        dev = self._first(q, 4)
        B, T, Hk, _ = q.shape
        if v.dim() != 4:
            raise ValueError("v must be [B, T, Hv, %d]" % self.D_v)
        Hv = v.shape[2]
        _check(q, "q", (B, T, Hk, self.D_k), self._dt, dev)
        _check(k, "k", (B, T, Hk, self.D_k), self._dt, dev)
        _check(v, "v", (B, T, Hv, self.D_v), self._dt, dev)
        fixed = g.dim() == 1
        _check(g, "g", (Hv,) if fixed else (B, T, Hv), torch.float32, dev)
        rows, n = B, 0
        if cu_seqlens is not None:
            if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2 or B != 1:
                raise ValueError("cu_seqlens needs B = 1 and the bounds of at least one sequence")
            _check(cu_seqlens, "cu_seqlens", cu_seqlens.shape, torch.int64, dev)
            cu_seqlens = cu_seqlens.contiguous()
            rows = n = cu_seqlens.shape[0] - 1
        state = (rows, Hv, self.D_k, self.D_v)
        if initial_state is not None:
            _check(initial_state, "initial_state", state, torch.float32, dev)
            initial_state = initial_state.contiguous()
        q, k, v = (_strided(x if x.stride(1) < 1 << 24 else x.contiguous(), self._step)
                   for x in (q, k, v))
        # for a given o, and for a new one
        ref, new = (ctypes.byref(DecayDesc(
            DTYPES[self.dtype], B, T, Hk, Hv, self.D_k, self.D_v, n, self.scale, fixed,
            _LL3(*q.stride()[:3]), _LL3(*k.stride()[:3]), _LL3(*v.stride()[:3]), x))
            for x in (0, 1))
        L = self._lib
        sizes = L.fftconv_decay_workspace_bytes(ref), L.fftconv_decay_backward_workspace_bytes(ref)
        return ((dev, (ref, new), state, sizes),
                (q, k, v, g.contiguous(), cu_seqlens, initial_state))

    def forward(self, q, k, v, g, initial_state=None, cu_seqlens=None, out=None,
                final_state=None, workspace=None, stream=None):
        """Outputs [B, T, Hv, D_v] and final states [rows, Hv, D_k, D_v].
        cu_seqlens: int64 [n + 1] with the bounds of n sequences packed in the
        one batch row (they may be empty); rows = n then, B otherwise.  Tokens
        before the first bound and behind the last belong to no sequence: their
        outputs are 0, or what a given `out` holds."""
        (dev, refs, state, sizes), ins, ptrs = self._checked(
            "_describe", (q, k, v, g, cu_seqlens, initial_state))
        v, ref = ins[2], refs[out is None]
        out = _like(v) if out is None else _given(out, "out", v.shape, self._dt, dev)
        if final_state is None:
            final_state = torch.empty(state, dtype=torch.float32, device=dev)
        else:
            _given(final_state, "final_state", state, torch.float32, dev)
        ws = self._space(sizes[0], workspace, dev, "workspace") if sizes[0] else None
        self._call(self._lib.fftconv_decay_forward, dev, stream, (*ins, out, final_state, ws), ref,
                   *ptrs, out.data_ptr(), final_state.data_ptr(), _ptr(ws), self._bytes(ws))
        return out, final_state

    def backward(self, q, k, v, g, d_out, d_final_state=None, initial_state=None,
                 cu_seqlens=None, workspace=None, stream=None):
        """Gradients of forward, for the same inputs: d_out = dL/do,
        d_final_state = dL/d(final state) (None: 0).  Returns (dq, dk, dv, dg,
        d_initial_state), dg of g's shape; the last is None where there is no
        initial_state.  Tokens that no packed sequence holds have gradients of 0."""
        (dev, (ref, _), state, sizes), ins, ptrs = self._checked(
            "_describe", (q, k, v, g, cu_seqlens, initial_state))
        _check(d_out, "d_out", ins[2].shape, self._dt, dev)
        d_out = _dense(d_out)
        if d_final_state is not None:
            _check(d_final_state, "d_final_state", state, torch.float32, dev)
            d_final_state = _dense(d_final_state)
        ws = self._space(sizes[1], workspace, dev, "workspace")
        new = [_like(x) for x in ins[:4]]
        new.append(None if initial_state is None else _like(ins[5]))
        self._call(self._lib.fftconv_decay_backward, dev, stream,
                   (*ins, d_out, d_final_state, ws, *new), ref, *ptrs, _ptr(d_out),
                   _ptr(d_final_state), *map(_ptr, new), _ptr(ws), self._bytes(ws))
        return tuple(new)

    def _describe_step(self, q, k, v, g, slots, state):
        dev = self._first(q, 3)
        N, Hk, _ = q.shape
        if v.dim() != 3 or state.dim() != 4:
            raise ValueError("v must be [N, Hv, %d], state [pool, Hv, %d, %d]"
                             % (self.D_v, self.D_k, self.D_v))
        Hv, pool = v.shape[1], state.shape[0]
        _check(q, "q", (N, Hk, self.D_k), self._dt, dev)
        _check(k, "k", (N, Hk, self.D_k), self._dt, dev)
        _check(v, "v", (N, Hv, self.D_v), self._dt, dev)
        fixed = g.dim() == 1
        _check(g, "g", (Hv,) if fixed else (N, Hv), torch.float32, dev)
        _check(state, "state", (pool, Hv, self.D_k, self.D_v), torch.float32, dev)
        if not state.is_contiguous():
            raise ValueError("state must be contiguous")
        if slots is not None:
            _check(slots, "slots", (N,), torch.int64, dev)
            slots = slots.contiguous()
        q, k, v = (_strided(x, self._step) for x in (q, k, v))
        st = [_LL3(x.stride(0), 0, x.stride(1)) for x in (q, k, v)]
        desc = DecayDesc(DTYPES[self.dtype], N, 1, Hk, Hv, self.D_k, self.D_v, 0, self.scale,
                         fixed, *st)
        return (dev, ctypes.byref(desc), pool), (q, k, v, g.contiguous(), slots, state)

    def step(self, q, k, v, g, state, slots=None, out=None, stream=None):
        """One token for each of N requests: q, k [N, Hk, D_k], v [N, Hv, D_v],
        g [N, Hv] or [Hv]; state [pool, Hv, D_k, D_v] fp32, updated in place;
        slots int64 [N], the state of each request (default: request i has
        state i; outside the pool, such as -1: no state, output 0; two
        requests must not share one).  Returns o [N, Hv, D_v]."""
        if state.data_ptr() & 15:
            raise ValueError("state must be 16-byte aligned")
        (dev, ref, pool), ins, ptrs = self._checked("_describe_step", (q, k, v, g, slots, state))
        out = _like(v) if out is None else _given(out, "out", v.shape, self._dt, dev)
        self._call(self._lib.fftconv_decay_step, dev, stream, (*ins, out), ref, *ptrs[:4],
                   ptrs[5], pool, ptrs[4], out.data_ptr())
        return out
