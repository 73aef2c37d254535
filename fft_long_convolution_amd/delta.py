"""ctypes binding of the token mixers beside the long convolution
(include/fftconv.h): norms of queries and keys with the position rotation
(:class:`QKNorm`) and the gated delta rule (:class:`GatedDelta`).

Argument marshalling only: every step runs in the HIP library.  PyTorch
supplies device memory and the current stream; calls raise if the library is
not built.

A layer of the gated delta rule uses them together:

>>> norm = QKNorm(128, norm="l2", rotary_dim=128)
>>> rule = GatedDelta(128, 128)
>>> q, k = norm.forward(q, k, cos=cos, sin=sin, positions=pos)
>>> o, state = rule.forward(q, k, v, g, beta)             # a prompt
>>> o = rule.step(q1, k1, v1, g1, beta1, state)           # then token by token
"""
from __future__ import annotations

import ctypes

import torch

from .fftconv import DTYPES, FFTConvError
from .fftconv import lib as _base_lib

NORMS = {"rms": 0, "l2": 1}
TORCH_DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}

_LL3 = ctypes.c_longlong * 3


class QKNormDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("B", ctypes.c_size_t), ("T", ctypes.c_size_t),
                ("Hq", ctypes.c_size_t), ("Hk", ctypes.c_size_t), ("D", ctypes.c_size_t),
                ("rotary_dim", ctypes.c_size_t), ("interleaved", ctypes.c_int),
                ("norm", ctypes.c_int), ("eps", ctypes.c_float),
                ("table_rows", ctypes.c_size_t), ("q_stride", _LL3), ("k_stride", _LL3)]


class DeltaDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("B", ctypes.c_size_t), ("T", ctypes.c_size_t),
                ("Hk", ctypes.c_size_t), ("Hv", ctypes.c_size_t), ("Dk", ctypes.c_size_t),
                ("Dv", ctypes.c_size_t), ("sequences", ctypes.c_size_t),
                ("scale", ctypes.c_float), ("q_stride", _LL3), ("k_stride", _LL3),
                ("v_stride", _LL3), ("clear_unheld", ctypes.c_int)]


_ready = None


def lib() -> ctypes.CDLL:
    """libfftconv.so with the signatures of this module's calls."""
    global _ready
    L = _base_lib()
    if _ready is not L:
        vp, sz, i = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
        nd, dd = ctypes.POINTER(QKNormDesc), ctypes.POINTER(DeltaDesc)
        for name, res, args in (
                ("fftconv_qknorm_forward", i, [nd] + [vp] * 10),
                ("fftconv_qknorm_workspace_bytes", sz, [nd]),
                ("fftconv_qknorm_backward", i, [nd] + [vp] * 14 + [sz, vp]),
                ("fftconv_delta_forward", i, [dd] + [vp] * 10 + [sz, vp, sz, vp]),
                ("fftconv_delta_workspace_bytes", sz, [dd]),
                ("fftconv_delta_saved_bytes", sz, [dd]),
                ("fftconv_delta_backward", i, [dd] + [vp] * 7 + [sz] + [vp] * 9 + [sz, vp]),
                ("fftconv_delta_backward_workspace_bytes", sz, [dd]),
                ("fftconv_delta_step", i, [dd] + [vp] * 6 + [sz, vp, vp, vp])):
            fn = getattr(L, name)
            fn.restype, fn.argtypes = res, args
        _ready = L
    return L


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check(t, name, shape, dtype, device):
    """A tensor argument of exactly this shape, type and device."""
    if t.shape != shape:
        raise ValueError("%s must be %s, not %s" % (name, list(shape), list(t.shape)))
    if t.dtype != dtype:
        raise ValueError("%s dtype must be %s" % (name, dtype))
    if t.device != device:
        raise ValueError("%s must be on %s" % (name, device))


def _like(t):
    """A new contiguous tensor of t's shape, type and device."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _given(t, name, shape, dtype, device):
    """The caller's output tensor, checked."""
    _check(t, name, shape, dtype, device)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


def _strided(t, step):
    """t, or a copy of it where its strides do not suit the kernels' 16-byte
    accesses."""
    s = t.stride()
    if t.numel() and (s[-1] != 1 and t.shape[-1] > 1 or
                      any(x % step and n > 1 for x, n in zip(s[:-1], t.shape))):
        t = t.clone(memory_format=torch.contiguous_format)
    return t


def _dense(t):
    """t contiguous and 16-byte aligned."""
    t = t.contiguous()
    return t.clone() if t.data_ptr() & 15 else t


def _layout(ts):
    """What the checks of a call's tensors depend on."""
    return tuple([None if t is None else (t.shape, t.stride(), t.dtype, t.device) for t in ts])


class _Op:
    # descriptors of calls that passed the checks, by the operator's settings
    # and the sizes, strides, types and devices of the tensors
    _known = {}

    def __init__(self, dtype):
        if dtype not in DTYPES:
            raise ValueError("dtype must be one of %s" % list(DTYPES))
        self._dtype = dtype
        self._dt = TORCH_DTYPES[dtype]
        self._step = 4 if dtype == "f32" else 8
        self._lib = lib()

    @property
    def dtype(self):
        """Fixed: what else follows from it is made once."""
        return self._dtype

    def _checked(self, kind, ts):
        """The call's tensors in a layout the library takes, its descriptor
        and what else follows from the sizes: from `kind` (a method that
        checks and describes) where no such call was seen before.  Misaligned
        tensors are copied first: a copy has strides of its own, and the
        descriptor holds those of the tensor that goes in."""
        ptrs = [0 if t is None else t.data_ptr() for t in ts]
        for i, x in enumerate(ptrs):
            if x & 15 and (x & 7 or ts[i].dtype != torch.int64):
                ts = list(ts)
                ts[i] = ts[i].clone(memory_format=torch.contiguous_format)
                ptrs[i] = ts[i].data_ptr()
        key = (kind, self._settings, _layout(ts))
        found = self._known.get(key)
        if found is None:
            found, ts = getattr(self, kind)(*ts)
            if len(self._known) >= 4096:
                self._known.clear()
            # tensors that had to be copied have another layout now
            self._known[(kind, self._settings, _layout(ts))] = found
            ptrs = [0 if t is None else t.data_ptr() for t in ts]
        return found, ts, ptrs

    def _first(self, q, dims):
        if q.dim() != dims:
            raise ValueError("q must have %d dimensions" % dims)
        if not q.is_cuda:
            raise ValueError("q must be a CUDA tensor")
        return q.device

    def _call(self, fn, device, stream, kept, *args):
        """Run the entry point `fn` on `stream` (default: the device's
        current one).  kept: tensors made for this call, which the allocator
        must not hand out before `stream` has passed it."""
        if stream is None:
            # the handle alone: a Stream object takes 2 us to make
            handle = torch._C._cuda_getCurrentRawStream(device.index)
        else:
            handle, current = stream.cuda_stream, torch.cuda.current_stream(device)
            if stream != current:
                # what was made here has to be ready there, and to live until then
                stream.wait_stream(current)
                for t in kept:
                    if t is not None:
                        t.record_stream(stream)
        if torch.cuda.current_device() == device.index:
            st = fn(*args, handle)
        else:
            with torch.cuda.device(device):
                st = fn(*args, handle)
        if st != 0:
            raise FFTConvError(st, fn.__name__)

    @staticmethod
    def _space(nbytes, given, device, name):
        """A workspace of at least nbytes: the caller's or a new one."""
        if given is None:
            return torch.empty(nbytes, dtype=torch.uint8, device=device)
        if given.device != device or not given.is_contiguous():
            raise ValueError("%s must be contiguous on %s" % (name, device))
        return given

    @staticmethod
    def _bytes(t):
        return 0 if t is None else t.numel() * t.element_size()


class QKNorm(_Op):
    """Norms of queries and keys for each head of D elements, with the
    position rotation of the first ``rotary_dim`` of them in the same pass.

    norm: "rms" (root mean square) or "l2" (2-norm).  interleaved: rotate the
    pairs (2i, 2i+1) instead of (i, i + rotary_dim/2).
    """

    def __init__(self, D: int, rotary_dim: int = 0, norm: str = "rms", eps: float = 1e-6,
                 interleaved: bool = False, dtype: str = "bf16"):
        super().__init__(dtype)
        if norm not in NORMS:
            raise ValueError("norm must be one of %s" % list(NORMS))
        self.D, self.rotary_dim, self.norm = D, rotary_dim, norm
        self.eps, self.interleaved = eps, interleaved

    @property
    def _settings(self):
        return self.D, self.rotary_dim, self.norm, self.eps, self.interleaved, self.dtype

    def _describe(self, q, k, q_weight, k_weight, cos, sin, positions):
        dev = self._first(q, 4)
        B, T, Hq, D = q.shape
        if D != self.D:
            raise ValueError("q must be [B, T, Hq, %d]" % self.D)
        if k.dim() != 4:
            raise ValueError("k must be [B, T, Hk, %d]" % self.D)
        Hk = k.shape[2]
        _check(q, "q", q.shape, self._dt, dev)
        _check(k, "k", (B, T, Hk, D), self._dt, dev)
        for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
            if w is not None:
                _check(w, name, (D,), torch.float32, dev)
        rows = 0
        if self.rotary_dim:
            if cos is None or sin is None or positions is None:
                raise ValueError("rotation needs cos, sin and positions")
            rows = cos.shape[0]
            _check(cos, "cos", (rows, self.rotary_dim // 2), torch.float32, dev)
            _check(sin, "sin", (rows, self.rotary_dim // 2), torch.float32, dev)
            _check(positions, "positions", (B, T), torch.int64, dev)
            cos, sin, positions = cos.contiguous(), sin.contiguous(), positions.contiguous()
        else:
            cos = sin = positions = None
        q, k = _strided(q, self._step), _strided(k, self._step)
        q_weight = None if q_weight is None else q_weight.contiguous()
        k_weight = None if k_weight is None else k_weight.contiguous()
        desc = QKNormDesc(DTYPES[self.dtype], B, T, Hq, Hk, D, self.rotary_dim,
                          1 if self.interleaved else 0, NORMS[self.norm], self.eps, rows,
                          _LL3(*q.stride()[:3]), _LL3(*k.stride()[:3]))
        ref = ctypes.byref(desc)
        need = self._lib.fftconv_qknorm_workspace_bytes(ref)
        return (dev, ref, need), (q, k, q_weight, k_weight, cos, sin, positions)

    def forward(self, q, k, q_weight=None, k_weight=None, cos=None, sin=None, positions=None,
                out=None, stream=None):
        """q [B, T, Hq, D], k [B, T, Hk, D] (strided views are fine) ->
        normed and rotated (q, k).  weights: fp32 [D] or None; cos, sin: fp32
        [P, rotary_dim/2]; positions: int64 [B, T], rows of the tables (a
        position outside them gives NaN).  out: a pair of tensors."""
        (dev, ref, _), ins, ptrs = self._checked(
            "_describe", (q, k, q_weight, k_weight, cos, sin, positions))
        yq, yk = (None, None) if out is None else out
        yq = _like(q) if yq is None else _given(yq, "out[0]", q.shape, self._dt, dev)
        yk = _like(k) if yk is None else _given(yk, "out[1]", k.shape, self._dt, dev)
        self._call(self._lib.fftconv_qknorm_forward, dev, stream, (*ins, yq, yk), ref, *ptrs,
                   yq.data_ptr(), yk.data_ptr())
        return yq, yk

    def backward(self, q, k, dq_out, dk_out, q_weight=None, k_weight=None, cos=None, sin=None,
                 positions=None, workspace=None, stream=None):
        """Gradients for dq_out, dk_out = dL/d(outputs of forward): returns
        (dq, dk, dq_weight, dk_weight), the last two fp32 [D] or None where
        there is no weight."""
        (dev, ref, need), ins, ptrs = self._checked(
            "_describe", (q, k, q_weight, k_weight, cos, sin, positions))
        _check(dq_out, "dq_out", q.shape, self._dt, dev)
        _check(dk_out, "dk_out", k.shape, self._dt, dev)
        dq_out, dk_out = _dense(dq_out), _dense(dk_out)
        dq, dk = _like(q), _like(k)
        dwq = None if q_weight is None else _like(q_weight)
        dwk = None if k_weight is None else _like(k_weight)
        ws = None
        if dwq is not None or dwk is not None:
            ws = self._space(need, workspace, dev, "workspace")
        self._call(self._lib.fftconv_qknorm_backward, dev, stream,
                   (*ins, dq_out, dk_out, dq, dk, dwq, dwk, ws), ref, *ptrs, _ptr(dq_out),
                   _ptr(dk_out), _ptr(dq), _ptr(dk), _ptr(dwq), _ptr(dwk), _ptr(ws),
                   self._bytes(ws))
        return dq, dk, dwq, dwk


class GatedDelta(_Op):
    """The gated delta rule for heads of D_k x D_v: from a state S, each token
    does S <- e^g S, u = beta (v - S^T k), S <- S + k u^T, o = scale S^T q.

    q, k [B, T, Hk, D_k] and v [B, T, Hv, D_v] (strided views are fine; Hv a
    multiple of Hk), g and beta fp32 [B, T, Hv]; states are fp32
    [rows, Hv, D_k, D_v].  scale defaults to D_k ** -0.5.
    """

    def __init__(self, D_k: int, D_v: int, dtype: str = "bf16", scale: float | None = None):
        super().__init__(dtype)
        self.D_k, self.D_v = D_k, D_v
        self.scale = D_k ** -0.5 if scale is None else float(scale)

    @property
    def _settings(self):
        return self.D_k, self.D_v, self.dtype, self.scale

    def _describe(self, q, k, v, g, beta, cu_seqlens, initial_state):
        dev = self._first(q, 4)
        B, T, Hk, _ = q.shape
        if v.dim() != 4:
            raise ValueError("v must be [B, T, Hv, %d]" % self.D_v)
        Hv = v.shape[2]
        _check(q, "q", (B, T, Hk, self.D_k), self._dt, dev)
        _check(k, "k", (B, T, Hk, self.D_k), self._dt, dev)
        _check(v, "v", (B, T, Hv, self.D_v), self._dt, dev)
        _check(g, "g", (B, T, Hv), torch.float32, dev)
        _check(beta, "beta", (B, T, Hv), torch.float32, dev)
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
        ref, new = (ctypes.byref(DeltaDesc(
            DTYPES[self.dtype], B, T, Hk, Hv, self.D_k, self.D_v, n, self.scale,
            _LL3(*q.stride()[:3]), _LL3(*k.stride()[:3]), _LL3(*v.stride()[:3]), x))
            for x in (0, 1))
        L = self._lib
        sizes = (L.fftconv_delta_workspace_bytes(ref), L.fftconv_delta_saved_bytes(ref),
                 L.fftconv_delta_backward_workspace_bytes(ref))
        return ((dev, (ref, new), state, sizes),
                (q, k, v, g.contiguous(), beta.contiguous(), cu_seqlens, initial_state))

    def _forward(self, ins, out, final_state, saved, train, workspace, stream):
        (dev, refs, state, sizes), ins, ptrs = self._checked("_describe", ins)
        v, ref = ins[2], refs[out is None]
        out = _like(v) if out is None else _given(out, "out", v.shape, self._dt, dev)
        if final_state is None:
            final_state = torch.empty(state, dtype=torch.float32, device=dev)
        else:
            _given(final_state, "final_state", state, torch.float32, dev)
        ws = self._space(sizes[0], workspace, dev, "workspace")
        if train:
            saved = self._space(sizes[1], saved, dev, "saved")
        self._call(self._lib.fftconv_delta_forward, dev, stream,
                   (*ins, out, final_state, saved, ws), ref, *ptrs, out.data_ptr(),
                   final_state.data_ptr(), _ptr(saved), self._bytes(saved), ws.data_ptr(),
                   self._bytes(ws))
        return out, final_state, saved

    def forward(self, q, k, v, g, beta, initial_state=None, cu_seqlens=None, out=None,
                final_state=None, workspace=None, stream=None):
        """Outputs [B, T, Hv, D_v] and final states [rows, Hv, D_k, D_v].
        cu_seqlens: int64 [n + 1] with the bounds of n sequences packed in the
        one batch row (they may be empty); rows = n then, B otherwise.  Tokens
        before the first bound and behind the last belong to no sequence: their
        outputs are 0, or what a given `out` holds."""
        return self._forward((q, k, v, g, beta, cu_seqlens, initial_state), out, final_state,
                             None, False, workspace, stream)[:2]

    def forward_train(self, q, k, v, g, beta, initial_state=None, cu_seqlens=None, out=None,
                      final_state=None, saved=None, workspace=None, stream=None):
        """As forward, and what backward needs besides the inputs (an opaque
        tensor of bytes): returns (o, final_state, saved)."""
        return self._forward((q, k, v, g, beta, cu_seqlens, initial_state), out, final_state,
                             saved, True, workspace, stream)

    def backward(self, q, k, v, g, beta, d_out, saved, d_final_state=None, initial_state=None,
                 cu_seqlens=None, workspace=None, stream=None):
        """Gradients of forward_train, for the same inputs and what it saved:
        d_out = dL/do, d_final_state = dL/d(final state) (None: 0).  Returns
        (dq, dk, dv, dg, dbeta, d_initial_state); the last is None where there
        is no initial_state.  Tokens that no packed sequence holds have
        gradients of 0."""
        (dev, (ref, _), state, sizes), ins, ptrs = self._checked(
            "_describe", (q, k, v, g, beta, cu_seqlens, initial_state))
        _check(d_out, "d_out", ins[2].shape, self._dt, dev)
        d_out = _dense(d_out)
        if d_final_state is not None:
            _check(d_final_state, "d_final_state", state, torch.float32, dev)
            d_final_state = _dense(d_final_state)
        if saved.device != dev or not saved.is_contiguous():
            raise ValueError("saved must be what forward_train returned")
        ws = self._space(sizes[2], workspace, dev, "workspace")
        new = [_like(x) for x in ins[:5]]
        new.append(None if initial_state is None else _like(initial_state))
        self._call(self._lib.fftconv_delta_backward, dev, stream,
                   (*ins, saved, d_out, d_final_state, ws, *new), ref, *ptrs[:6], _ptr(saved),
                   self._bytes(saved), _ptr(d_out), _ptr(d_final_state), *map(_ptr, new),
                   _ptr(ws), self._bytes(ws))
        return tuple(new)

    def _describe_step(self, q, k, v, g, beta, slots, state):
        dev = self._first(q, 3)
        N, Hk, _ = q.shape
        if v.dim() != 3 or state.dim() != 4:
            raise ValueError("v must be [N, Hv, %d], state [pool, Hv, %d, %d]"
                             % (self.D_v, self.D_k, self.D_v))
        Hv, pool = v.shape[1], state.shape[0]
        _check(q, "q", (N, Hk, self.D_k), self._dt, dev)
        _check(k, "k", (N, Hk, self.D_k), self._dt, dev)
        _check(v, "v", (N, Hv, self.D_v), self._dt, dev)
        _check(g, "g", (N, Hv), torch.float32, dev)
        _check(beta, "beta", (N, Hv), torch.float32, dev)
        _check(state, "state", (pool, Hv, self.D_k, self.D_v), torch.float32, dev)
        if not state.is_contiguous():
            raise ValueError("state must be contiguous")
        if slots is not None:
            _check(slots, "slots", (N,), torch.int64, dev)
            slots = slots.contiguous()
        q, k, v = (_strided(x, self._step) for x in (q, k, v))
        st = [_LL3(x.stride(0), 0, x.stride(1)) for x in (q, k, v)]
        desc = DeltaDesc(DTYPES[self.dtype], N, 1, Hk, Hv, self.D_k, self.D_v, 0, self.scale,
                         *st)
        return ((dev, ctypes.byref(desc), pool),
                (q, k, v, g.contiguous(), beta.contiguous(), slots, state))

    def step(self, q, k, v, g, beta, state, slots=None, out=None, stream=None):
        """One token for each of N requests: q, k [N, Hk, D_k], v [N, Hv, D_v],
        g, beta [N, Hv]; state [pool, Hv, D_k, D_v] fp32, updated in place;
        slots int64 [N], the state of each request (default: request i has
        state i; outside the pool, such as -1: no state, output 0; two
        requests must not share one).  Returns o [N, Hv, D_v]."""
        if state.data_ptr() & 15:
            raise ValueError("state must be 16-byte aligned")
        (dev, ref, pool), ins, ptrs = self._checked("_describe_step",
                                                    (q, k, v, g, beta, slots, state))
        out = _like(v) if out is None else _given(out, "out", v.shape, self._dt, dev)
        self._call(self._lib.fftconv_delta_step, dev, stream, (*ins, out), ref, *ptrs[:5],
                   ptrs[6], pool, ptrs[5], out.data_ptr())
        return out
