"""Binding of linear attention with a decay for each head (``vimscan_linattn_*`` of include/vimscan.h):
whole sequences, their gradients, and single tokens.

As in ``binding``: a Prepared* object validates once and owns its output tensors, calling it queues
the kernels (one ctypes call) and does not synchronise. Work goes to torch's current stream for the
inputs' device at preparation time unless ``stream`` (a hipStream_t handle) is given.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding as _b
from .block import FLAG_REVERSE, _Call, _check_tensor, _output, _plan_dict, _ptr, _stream_of, _workspace

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64


class _LinAttn(ctypes.Structure):
    _fields_ = [("q", _vp), ("k", _vp), ("v", _vp), ("ld_q", _i64), ("ld_k", _i64), ("ld_v", _i64), ("hs_q", _i64),
                ("hs_k", _i64), ("hs_v", _i64), ("log_decay", _vp), ("ld_decay", _i64), ("h0", _vp), ("offsets", _vp),
                ("nseq", _i64), ("heads", _i64), ("groups", _i64), ("scale", ctypes.c_float)]


class _LinAttnGrad(ctypes.Structure):
    _fields_ = [("dy", _vp), ("ld_dy", _i64), ("hs_dy", _i64), ("dh_last", _vp), ("dq", _vp), ("dk", _vp), ("dv", _vp),
                ("dlog_decay", _vp), ("dh0", _vp)]


def declare(lib):
    """Argument types of this module's entry points on an opened library."""
    launch = ctypes.POINTER(_b._Launch)
    plan = ctypes.POINTER(_b._Plan)
    lib.vimscan_linattn_fwd.argtypes = [ctypes.POINTER(_LinAttn), _i64, _vp, _vp, launch]
    lib.vimscan_linattn_bwd.argtypes = [ctypes.POINTER(_LinAttn), _i64, ctypes.POINTER(_LinAttnGrad), launch]
    lib.vimscan_linattn_step.argtypes = [ctypes.POINTER(_LinAttn), _vp, _i64, _vp, _vp, _vp, launch]
    lib.vimscan_linattn_plan.argtypes = [launch, _i64, _i64, _i64, ctypes.c_int, _i64, ctypes.c_int, plan]
    for f in (lib.vimscan_linattn_fwd, lib.vimscan_linattn_bwd, lib.vimscan_linattn_step, lib.vimscan_linattn_plan):
        f.restype = ctypes.c_int


def head_strides(t, name):
    """Elements from token to token (evenly spaced over the leading dimensions) and from head to head of
    a (..., heads, d) tensor whose channels are contiguous."""
    heads, d = t.shape[-2:]
    if t.numel() == 0:
        return heads * d, d
    if d > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the channels of a head must be contiguous")
    ld = run = None
    for size, stride in zip(reversed(t.shape[:-2]), reversed(t.stride()[:-2])):
        if size == 1:
            continue
        if ld is None:
            ld = stride
        elif stride != run:
            raise ValueError(f"{name}: tokens must be evenly spaced over the leading dimensions")
        run = size * stride
    if ld is None:
        ld = heads * d
    if ld < d:
        raise ValueError(f"{name}: tokens overlap")
    return ld, (t.stride(-2) if heads > 1 else d)


def _decay_stride(log_decay, lead, heads, dev):
    """0 for a decay per head (heads,), the token stride for one per token and head (*lead, heads)."""
    if log_decay.dim() == 1:
        _check_tensor(log_decay, "log_decay", dev, torch.float32, (heads,))
        return 0
    _check_tensor(log_decay, "log_decay", dev, torch.float32, (*lead, heads), dense=False)
    ld, _ = head_strides(log_decay.unsqueeze(-2), "log_decay")
    return ld


class LinAttnInputs:
    """The validated inputs of a linear attention over whole sequences (see ``PreparedLinAttn``)."""

    def __init__(self, q, k, v, log_decay, scale=None, h0=None, seg_len=0, offsets=None, reverse=False):
        if q.dim() != 4 or v.dim() != 4:
            raise ValueError("q must be (batch, seqlen, groups, dk) and v (batch, seqlen, heads, dv)")
        dev = q.device
        if dev.type != "cuda":
            raise ValueError("inputs must be on a GPU device")
        self.io = _b._io_code(q.dtype)
        Bsz, L, G, dk = q.shape
        H, dv = v.shape[2:]
        _check_tensor(k, "k", dev, q.dtype, tuple(q.shape), dense=False)
        _check_tensor(v, "v", dev, q.dtype, (Bsz, L, H, dv), dense=False)
        if G == 0 or H % G != 0:
            raise ValueError("the groups of q and k must divide the heads of v")
        if offsets is not None:
            if seg_len != 0:
                raise ValueError("offsets and seg_len exclude each other")
            if offsets.dim() != 1 or offsets.numel() < 1:
                raise ValueError("offsets must be a (sequences + 1,) int32 tensor")
            _check_tensor(offsets, "offsets", dev, torch.int32, tuple(offsets.shape))
            self.nseq = offsets.numel() - 1
        else:
            T = seg_len if seg_len > 0 else L
            self.nseq = Bsz * (L // T) if T > 0 else Bsz
        self.state_shape = (self.nseq, H, dk, dv)
        if h0 is not None:
            _check_tensor(h0, "h0", dev, torch.float32, self.state_shape)
        self.decay_stride = _decay_stride(log_decay, (Bsz, L), H, dev)
        self.q, self.k, self.v, self.log_decay, self.h0, self.offsets = q, k, v, log_decay, h0, offsets
        self.scale = max(dk, 1) ** -0.5 if scale is None else float(scale)
        self.seg_len, self.reverse = int(seg_len), bool(reverse)
        self.dev, self.dtype = dev, q.dtype
        (ld_q, hs_q), (ld_k, hs_k), (ld_v, hs_v) = (head_strides(t, n) for t, n in ((q, "q"), (k, "k"), (v, "v")))
        self.struct = _LinAttn(_ptr(q), _ptr(k), _ptr(v), ld_q, ld_k, ld_v, hs_q, hs_k, hs_v, _ptr(log_decay),
                               self.decay_stride, _ptr(h0), None if offsets is None else offsets.data_ptr(),
                               self.nseq if offsets is not None else 0, H, G, self.scale)

    def launch(self, stream):
        Bsz, L, H, dv = self.v.shape
        launch = _b.make_launch(Bsz, L, H * dv, self.q.shape[3], self.io, 0, stream=stream)
        launch.flags = FLAG_REVERSE if self.reverse else 0
        return launch

    def plan(self, launch, backward):
        plan = _b._Plan()
        _b._check(_b.load_library().vimscan_linattn_plan(ctypes.byref(launch), self.seg_len, self.struct.heads,
                                                         self.struct.groups, int(self.offsets is not None), self.nseq,
                                                         int(backward), ctypes.byref(plan)))
        return plan


class PreparedLinAttn(_Call):
    """Linear attention with a decay for each head on fixed tensors (vimscan_linattn_fwd): per sequence and
    head, with a state of dk x dv,

        S_t = exp(g_t) S_{t-1} + k_t^T v_t, from h0 (or 0);  y_t = scale q_t S_t

    q, k: (B, L, G, dk), v: (B, L, H, dv) float32 or bfloat16, alike; G divides H, the H / G heads of a group
    share q and k. Tokens must be evenly spaced and channels contiguous (slices of one projection's output are fine). log_decay g:
    float32, (H,) or (B, L, H). scale: dk ** -0.5 when None. dk and dv up to 128. The B * L tokens in memory
    order are cut into sequences every seg_len tokens (L when 0) or at ``offsets``, int32 (sequences + 1,) from
    0 to B * L, which may hold empty sequences. h0: (sequences, H, dk, dv) float32 or None. reverse: walk every sequence from
    its end. Calling it fills ``y`` (B, L, H, dv) and ``h_last`` (sequences, H, dk, dv) float32 and returns y."""

    def __init__(self, q, k=None, v=None, log_decay=None, scale=None, h0=None, seg_len: int = 0, offsets=None,
                 reverse: bool = False, out=None, h_last=None, workspace=None, stream=None):
        inp = q if isinstance(q, LinAttnInputs) else LinAttnInputs(q, k, v, log_decay, scale, h0, seg_len, offsets, reverse)
        lib = _b.load_library()
        self.inputs, dev = inp, inp.dev
        self.y = _output(out, "out", dev, inp.dtype, tuple(inp.v.shape))
        self.h_last = _output(h_last, "h_last", dev, torch.float32, inp.state_shape)
        launch = inp.launch(_stream_of(dev, stream))
        plan = inp.plan(launch, False)
        self.plan = _plan_dict(plan)
        ws = _workspace(workspace, plan.workspace_bytes, dev, launch)
        args = (ctypes.byref(inp.struct), inp.seg_len, _ptr(self.y), _ptr(self.h_last), ctypes.byref(launch))
        own = [t for t, given in ((self.y, out), (self.h_last, h_last), (ws, workspace)) if t is not given]
        self._prepare(dev, stream, launch, lib.vimscan_linattn_fwd, args, own, (inp, ws))

    def __call__(self):
        self._queue()
        return self.y


class PreparedLinAttnGrad(_Call):
    """Gradients of a linear attention (vimscan_linattn_bwd). forward: a PreparedLinAttn or LinAttnInputs (nothing
    but the inputs is needed); dy like y (any strides that v may have) or None, dh_last like h_last or None. Calling it fills ``dq``, ``dk``, ``dv``
    (in the inputs' dtype, contiguous), ``dlog_decay`` (log_decay's shape, float32; None with ``decays`` false) and, with h0,
    ``dh0``; it returns dq."""

    def __init__(self, forward, dy=None, dh_last=None, decays: bool = True, workspace=None, stream=None):
        lib = _b.load_library()
        inp = forward.inputs if isinstance(forward, PreparedLinAttn) else forward
        dev = inp.dev
        shape = tuple(inp.v.shape)
        ld_dy = hs_dy = 0
        if dy is not None:
            _check_tensor(dy, "dy", dev, inp.dtype, shape, dense=False)
            ld_dy, hs_dy = head_strides(dy, "dy")
        if dh_last is not None:
            _check_tensor(dh_last, "dh_last", dev, torch.float32, inp.state_shape)
        self.dq, self.dk, self.dv = (torch.empty(tuple(t.shape), dtype=inp.dtype, device=dev) for t in (inp.q, inp.k, inp.v))
        self.dlog_decay = torch.empty(tuple(inp.log_decay.shape), dtype=torch.float32, device=dev) if decays else None
        self.dh0 = torch.empty(inp.state_shape, dtype=torch.float32, device=dev) if inp.h0 is not None else None
        launch = inp.launch(_stream_of(dev, stream))
        plan = inp.plan(launch, 1 if decays else 2)
        self.plan = _plan_dict(plan)
        ws = _workspace(workspace, plan.workspace_bytes, dev, launch)
        g = _LinAttnGrad(_ptr(dy), ld_dy, hs_dy, _ptr(dh_last), _ptr(self.dq), _ptr(self.dk), _ptr(self.dv),
                         _ptr(self.dlog_decay), _ptr(self.dh0))
        args = (ctypes.byref(inp.struct), inp.seg_len, ctypes.byref(g), ctypes.byref(launch))
        own = [self.dq, self.dk, self.dv, self.dlog_decay, self.dh0] + ([ws] if ws is not workspace else [])
        self._prepare(dev, stream, launch, lib.vimscan_linattn_bwd, args, own, (inp, g, dy, dh_last, ws))

    def __call__(self):
        self._queue()
        return self.dq


class PreparedLinAttnStep(_Call):
    """One token of a batch of streams (vimscan_linattn_step). q, k: (B, G, dk), v: (B, H, dv), as for
    ``PreparedLinAttn``; log_decay: float32, (H,) or (B, H); state: a pool (slots, H, dk, dv) float32 that the call
    updates. Row b reads state[slots_in[b]] and writes state[slots_out[b]] (int32 (B,); slots_in None: slot b;
    slots_out None: the slot it was read from); a row with a slot outside the pool is skipped and its y is zero. A slot that one row writes must not
    be read or written by another. Fills and returns ``y`` (B, H, dv)."""

    def __init__(self, q, k, v, log_decay, state, scale=None, slots_in=None, slots_out=None, out=None, stream=None):
        lib = _b.load_library()
        if q.dim() != 3 or v.dim() != 3:
            raise ValueError("q must be (batch, groups, dk) and v (batch, heads, dv)")
        dev = q.device
        if dev.type != "cuda":
            raise ValueError("inputs must be on a GPU device")
        io = _b._io_code(q.dtype)
        Bsz, G, dk = q.shape
        H, dv = v.shape[1:]
        _check_tensor(k, "k", dev, q.dtype, tuple(q.shape), dense=False)
        _check_tensor(v, "v", dev, q.dtype, (Bsz, H, dv), dense=False)
        if G == 0 or H % G != 0:
            raise ValueError("the groups of q and k must divide the heads of v")
        if state.dim() != 4:
            raise ValueError("state must be (slots, heads, dk, dv)")
        _check_tensor(state, "state", dev, torch.float32, (state.shape[0], H, dk, dv))
        for t, name in ((slots_in, "slots_in"), (slots_out, "slots_out")):
            if t is not None:
                _check_tensor(t, name, dev, torch.int32, (Bsz,))
        decay_stride = _decay_stride(log_decay, (Bsz,), H, dev)
        self.y = _output(out, "out", dev, q.dtype, (Bsz, H, dv))
        launch = _b.make_launch(Bsz, 1, H * dv, dk, io, 0, stream=_stream_of(dev, stream))
        (ld_q, hs_q), (ld_k, hs_k), (ld_v, hs_v) = (head_strides(t, n) for t, n in ((q, "q"), (k, "k"), (v, "v")))
        p = _LinAttn(_ptr(q), _ptr(k), _ptr(v), ld_q, ld_k, ld_v, hs_q, hs_k, hs_v, _ptr(log_decay), decay_stride, None,
                     None, 0, H, G, max(dk, 1) ** -0.5 if scale is None else float(scale))
        args = (ctypes.byref(p), _ptr(state), int(state.shape[0]), _ptr(slots_in), _ptr(slots_out), _ptr(self.y),
                ctypes.byref(launch))
        self._prepare(dev, stream, launch, lib.vimscan_linattn_step, args, [self.y] if out is None else [],
                      (p, q, k, v, log_decay, state, slots_in, slots_out))

    def __call__(self):
        self._queue()
        return self.y


def linattn_fwd(q, k, v, log_decay, scale=None, h0=None, seg_len: int = 0, offsets=None, reverse: bool = False, out=None):
    """Linear attention with a decay for each head on the GPU: (y, h_last); arguments as ``PreparedLinAttn``.
    Queued on torch's current stream; does not synchronise."""
    call = PreparedLinAttn(q, k, v, log_decay, scale, h0, seg_len, offsets, reverse, out)
    call()
    return call.y, call.h_last


def linattn_step(q, k, v, log_decay, state, scale=None, slots_in=None, slots_out=None, out=None):
    """One token of a batch of streams, ``state`` updated in place; arguments as ``PreparedLinAttnStep``."""
    return PreparedLinAttnStep(q, k, v, log_decay, state, scale, slots_in, slots_out, out)()


def linattn_info(batch, seqlen, heads, dk, dv, groups=None, seg_len=0, io_dtype="bf16", nseq=None, backward=False) -> dict:
    """The library's plan for a linear attention of this shape (host only; vimscan_linattn_plan); nseq: the
    number of sequences when they are given by offsets; backward: 2 is the backward pass without the decays' gradient."""
    code = _b.VIMSCAN_BF16 if io_dtype == "bf16" else _b.VIMSCAN_F32
    launch = _b.make_launch(batch, seqlen, heads * dv, dk, code)
    plan = _b._Plan()
    _b._check(_b.load_library().vimscan_linattn_plan(ctypes.byref(launch), int(seg_len), int(heads),
                                                     int(heads if groups is None else groups), int(nseq is not None),
                                                     int(nseq or 0), int(backward), ctypes.byref(plan)))
    return _plan_dict(plan)
