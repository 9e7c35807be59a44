"""Binding of the recurrent block's operators: the gated linear recurrence (``vimscan_gated_*``), the block
norm (``vimscan_norm_*``) and the layer norm (``vimscan_layernorm_*``) of include/vimscan.h, each with its backward pass.

As in ``binding``: a Prepared* object validates once and owns its output tensors, calling it queues
the kernels (one ctypes call) and does not synchronise. Work goes to torch's current stream for the
inputs' device at preparation time unless ``stream`` (a hipStream_t handle) is given.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding as _b

GATED_STRIDE = 64                      # VIMSCAN_GATED_STRIDE
FLAG_REVERSE = 8                       # VIMSCAN_FLAG_REVERSE
FLAG_GATE_AFTER = 16                   # VIMSCAN_FLAG_GATE_AFTER

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64


class _Gated(ctypes.Structure):
    _fields_ = [("x", _vp), ("r", _vp), ("i", _vp), ("ld_x", _i64), ("ld_r", _i64), ("ld_i", _i64), ("lam", _vp),
                ("h0", _vp), ("offsets", _vp), ("nseq", _i64), ("c", ctypes.c_float)]


class _GatedGrad(ctypes.Structure):
    _fields_ = [("dy", _vp), ("dh_last", _vp), ("states", _vp), ("dx", _vp), ("dr", _vp), ("di", _vp),
                ("ld_dy", _i64), ("ld_dx", _i64), ("ld_dr", _i64), ("ld_di", _i64), ("dlam", _vp), ("dh0", _vp)]


class _Norm(ctypes.Structure):
    _fields_ = [("x", _vp), ("z", _vp), ("ld_x", _i64), ("ld_z", _i64), ("w_post", _vp), ("residual", _vp),
                ("gamma", _vp), ("w_pre", _vp), ("eps", ctypes.c_float), ("res_dtype", ctypes.c_int32)]


class _NormGrad(ctypes.Structure):
    _fields_ = [("dsum", _vp), ("dn", _vp), ("dx", _vp), ("dz", _vp), ("ld_dx", _i64), ("ld_dz", _i64),
                ("dresidual", _vp), ("dw_post", _vp), ("dgamma", _vp), ("dw_pre", _vp)]


class _LayerNorm(ctypes.Structure):
    _fields_ = [("x", _vp), ("ld_x", _i64), ("residual", _vp), ("weight", _vp), ("bias", _vp), ("eps", ctypes.c_float),
                ("res_dtype", ctypes.c_int32)]


class _LayerNormGrad(ctypes.Structure):
    _fields_ = [("dsum", _vp), ("dn", _vp), ("dx", _vp), ("ld_dx", _i64), ("dresidual", _vp), ("dweight", _vp),
                ("dbias", _vp)]


def declare(lib):
    """Argument types of this module's entry points on an opened library."""
    launch = ctypes.POINTER(_b._Launch)
    plan = ctypes.POINTER(_b._Plan)
    lib.vimscan_gated_fwd.argtypes = [ctypes.POINTER(_Gated), _i64, _vp, _vp, _vp, launch]
    lib.vimscan_gated_bwd.argtypes = [ctypes.POINTER(_Gated), _i64, ctypes.POINTER(_GatedGrad), launch]
    lib.vimscan_gated_step.argtypes = [ctypes.POINTER(_Gated), _vp, _i64, _vp, _vp, _vp, launch]
    lib.vimscan_gated_plan.argtypes = [launch, _i64, ctypes.c_int, _i64, ctypes.c_int, plan]
    lib.vimscan_gated_wait_reads.argtypes = [ctypes.c_int32]
    lib.vimscan_gated_alone.argtypes = [ctypes.POINTER(ctypes.c_uint64)]
    lib.vimscan_norm_fwd.argtypes = [ctypes.POINTER(_Norm), _vp, _vp, launch]
    lib.vimscan_norm_bwd.argtypes = [ctypes.POINTER(_Norm), ctypes.POINTER(_NormGrad), launch]
    lib.vimscan_norm_plan.argtypes = [launch, ctypes.c_int, plan]
    lib.vimscan_layernorm_fwd.argtypes = [ctypes.POINTER(_LayerNorm), _vp, _vp, launch]
    lib.vimscan_layernorm_bwd.argtypes = [ctypes.POINTER(_LayerNorm), ctypes.POINTER(_LayerNormGrad), launch]
    lib.vimscan_layernorm_plan.argtypes = [launch, ctypes.c_int, plan]
    for f in (lib.vimscan_layernorm_fwd, lib.vimscan_layernorm_bwd, lib.vimscan_layernorm_plan, lib.vimscan_gated_fwd,
              lib.vimscan_gated_bwd, lib.vimscan_gated_step, lib.vimscan_gated_plan,
              lib.vimscan_gated_wait_reads, lib.vimscan_gated_alone, lib.vimscan_norm_fwd, lib.vimscan_norm_bwd,
              lib.vimscan_norm_plan):
        f.restype = ctypes.c_int


def _ptr(t):
    return None if t is None or t.numel() == 0 else t.data_ptr()


def row_stride(t, name):
    """Elements from one row of the last dimension to the next, over all leading dimensions: the
    rows must be evenly spaced and contiguous within."""
    d = t.shape[-1]
    if t.numel() == 0:
        return d
    if d > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the channels of a row must be contiguous")
    ld = run = None
    for size, stride in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if ld is None:
            ld = stride
        elif stride != run:
            raise ValueError(f"{name}: rows must be evenly spaced over the leading dimensions")
        run = size * stride
    if ld is None:
        return d
    if ld < d:
        raise ValueError(f"{name}: rows overlap")
    return ld


def _check_tensor(t, name, dev, dtype, shape, dense=True):
    if t.device != dev or t.dtype != dtype or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)} on {dev}, got {t.dtype} {tuple(t.shape)} "
                         f"on {t.device}")
    if dense and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _output(t, name, dev, dtype, shape, dense=True):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _check_tensor(t, name, dev, dtype, shape, dense)
    return t


def _plan_dict(plan):
    return {f: getattr(plan, f) for f, _ in _b._Plan._fields_}


class _Call:
    """A prepared ctypes call: the buffers it keeps alive, its launch description, its stream."""

    def _prepare(self, dev, stream, launch, fn, args, own, keep):
        # arguments as ctypes objects once, so that a call converts nothing
        args = tuple(t(a) if isinstance(a, int) else a for a, t in zip(args, fn.argtypes))
        self._launch, self._fn, self._args, self._keep = launch, fn, args, keep
        # with several GPUs the call must be made with the tensors' device current
        self._dev = dev if torch.cuda.device_count() > 1 else None
        if stream is not None:
            # buffers allocated here belong to torch's current stream: tell its allocator of the other one
            ext = torch.cuda.ExternalStream(stream, device=dev) if stream else torch.cuda.default_stream(dev)
            for t in own:
                if t is not None and t.numel():
                    t.record_stream(ext)

    def set_scan_events(self, ev0: int = 0, ev1: int = 0):
        """hipEvent_t handles recorded before the first and after the last kernel of each call."""
        self._launch.scan_events[0] = ev0 or None
        self._launch.scan_events[1] = ev1 or None

    def _queue(self):
        if self._dev is not None:
            with torch.cuda.device(self._dev):
                status = self._fn(*self._args)
        else:
            status = self._fn(*self._args)
        if status != 0:
            _b._check(status)


def _stream_of(dev, stream):
    return torch.cuda.current_stream(dev).cuda_stream if stream is None else stream


def _workspace(workspace, need, dev, launch):
    """A workspace of the plan's size (the caller's when it is large enough)."""
    if workspace is not None and (workspace.device != dev or not workspace.is_contiguous()):
        raise ValueError(f"workspace must be contiguous on {dev}")
    if need == 0:
        return None
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    launch.workspace = workspace.data_ptr()
    launch.workspace_bytes = workspace.numel() * workspace.element_size()
    return workspace


# ------------------------------------------------------------------------------------------
# Gated linear recurrence


class GatedInputs:
    """The validated inputs of a gated recurrence over whole sequences (see ``PreparedGated``)."""

    def __init__(self, x, r, i, lam, c=8.0, h0=None, seg_len=0, offsets=None, reverse=False):
        if x.dim() != 3:
            raise ValueError("x must be (batch, seqlen, d_inner)")
        dev = x.device
        if dev.type != "cuda":
            raise ValueError("inputs must be on a GPU device")
        self.io = _b._io_code(x.dtype)
        self.shape = tuple(x.shape)
        Bsz, L, D = x.shape
        for t, name in ((r, "r"), (i, "i")):
            _check_tensor(t, name, dev, x.dtype, self.shape, dense=False)
        _check_tensor(lam, "lam", dev, torch.float32, (D,))
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
        if h0 is not None:
            _check_tensor(h0, "h0", dev, torch.float32, (self.nseq, D))
        self.x, self.r, self.i, self.lam, self.h0, self.offsets = x, r, i, lam, h0, offsets
        self.c, self.seg_len, self.reverse = float(c), int(seg_len), bool(reverse)
        self.dev, self.dtype = dev, x.dtype
        self.struct = _Gated(_ptr(x), _ptr(r), _ptr(i), row_stride(x, "x"), row_stride(r, "r"), row_stride(i, "i"),
                             _ptr(lam), _ptr(h0), None if offsets is None else offsets.data_ptr(),
                             self.nseq if offsets is not None else 0, self.c)

    def launch(self, stream):
        Bsz, L, D = self.shape
        launch = _b.make_launch(Bsz, L, D, 1, self.io, 0, stream=stream)
        launch.flags = FLAG_REVERSE if self.reverse else 0
        return launch

    def plan(self, launch, backward):
        plan = _b._Plan()
        _b._check(_b.load_library().vimscan_gated_plan(ctypes.byref(launch), self.seg_len,
                                                       int(self.offsets is not None), self.nseq, int(backward),
                                                       ctypes.byref(plan)))
        return plan

    @property
    def states_shape(self):
        Bsz, L, D = self.shape
        return (-(-Bsz * L // GATED_STRIDE), D)


class PreparedGated(_Call):
    """The gated linear recurrence on fixed tensors (vimscan_gated_fwd): per sequence and channel

        u_t = -c softplus(lam) sigmoid(r_t), a_t = exp(u_t)
        h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t, from h0 (or 0);  y_t = h_t

    x, r, i: (B, L, D) float32 or bfloat16, alike, rows evenly spaced (slices of one projection's
    output are fine); lam (D,) float32. The B * L tokens in memory order are cut into sequences every
    seg_len tokens (L when 0) or at ``offsets``, int32 (sequences + 1,) from 0 to B * L, which may
    hold empty sequences. h0: (sequences, D) float32 or None. reverse: walk every sequence from its
    end. Calling it fills ``y`` (B, L, D), ``h_last`` (sequences, D) float32 and, with
    ``save_states``, the states that ``PreparedGatedGrad`` needs; it returns y."""

    def __init__(self, x, r, i, lam, c: float = 8.0, h0=None, seg_len: int = 0, offsets=None, reverse: bool = False,
                 out=None, h_last=None, save_states: bool = False, workspace=None, stream=None):
        inp = x if isinstance(x, GatedInputs) else GatedInputs(x, r, i, lam, c, h0, seg_len, offsets, reverse)
        lib = _b.load_library()
        self.inputs, dev, D = inp, inp.dev, inp.shape[2]
        self.y = _output(out, "out", dev, inp.dtype, inp.shape)
        self.h_last = _output(h_last, "h_last", dev, torch.float32, (inp.nseq, D))
        self.states = torch.empty(inp.states_shape, dtype=torch.float32, device=dev) if save_states else None
        launch = inp.launch(_stream_of(dev, stream))
        plan = inp.plan(launch, False)
        self.plan = _plan_dict(plan)
        ws = _workspace(workspace, plan.workspace_bytes, dev, launch)
        args = (ctypes.byref(inp.struct), inp.seg_len, _ptr(self.y), _ptr(self.h_last), _ptr(self.states),
                ctypes.byref(launch))
        own = [t for t, given in ((self.y, out), (self.h_last, h_last), (self.states, None), (ws, workspace))
               if t is not given]
        self._prepare(dev, stream, launch, lib.vimscan_gated_fwd, args, own, (inp, ws))

    def __call__(self):
        self._queue()
        return self.y


class PreparedGatedGrad(_Call):
    """Gradients of a gated recurrence (vimscan_gated_bwd). forward: the PreparedGated that was run
    with ``save_states`` (or a GatedInputs, with ``states``); dy like y (rows evenly spaced), dh_last
    like h_last or None. Calling it fills ``dx``, ``dr``, ``di`` (``grads`` gives tensors for them,
    slices of one array among them), ``dlam`` and, with h0, ``dh0``; it returns dx."""

    def __init__(self, forward, dy=None, dh_last=None, states=None, grads=None, workspace=None, stream=None):
        lib = _b.load_library()
        if isinstance(forward, PreparedGated):
            inp, states = forward.inputs, forward.states
        else:
            inp = forward
        if states is None:
            raise ValueError("the backward pass needs the forward pass's states (save_states=True)")
        dev, D = inp.dev, inp.shape[2]
        _check_tensor(states, "states", dev, torch.float32, inp.states_shape)
        if dy is not None:
            _check_tensor(dy, "dy", dev, inp.dtype, inp.shape, dense=False)
        if dh_last is not None:
            _check_tensor(dh_last, "dh_last", dev, torch.float32, (inp.nseq, D))
        given = grads if grads is not None else (None, None, None)
        outs = [_output(t, n, dev, inp.dtype, inp.shape, dense=False) for t, n in zip(given, ("dx", "dr", "di"))]
        self.dx, self.dr, self.di = outs
        self.dlam = torch.empty(D, dtype=torch.float32, device=dev)
        self.dh0 = torch.empty((inp.nseq, D), dtype=torch.float32, device=dev) if inp.h0 is not None else None
        launch = inp.launch(_stream_of(dev, stream))
        plan = inp.plan(launch, True)
        self.plan = _plan_dict(plan)
        ws = _workspace(workspace, plan.workspace_bytes, dev, launch)
        g = _GatedGrad(_ptr(dy), _ptr(dh_last), _ptr(states), _ptr(self.dx), _ptr(self.dr), _ptr(self.di),
                       row_stride(dy, "dy") if dy is not None else D, row_stride(self.dx, "dx"),
                       row_stride(self.dr, "dr"), row_stride(self.di, "di"), _ptr(self.dlam), _ptr(self.dh0))
        args = (ctypes.byref(inp.struct), inp.seg_len, ctypes.byref(g), ctypes.byref(launch))
        own = [t for t, gv in zip(outs, given) if t is not gv] + [self.dlam, self.dh0]
        own += [ws] if ws is not workspace else []
        self._prepare(dev, stream, launch, lib.vimscan_gated_bwd, args, own, (inp, g, dy, dh_last, states, ws))

    def __call__(self):
        self._queue()
        return self.dx


class PreparedGatedStep(_Call):
    """One token of a batch of streams (vimscan_gated_step). x, r, i: (B, D), rows evenly spaced; lam
    (D,) float32; state: a pool (slots, D) float32 that the call updates. Row b reads
    state[slots_in[b]] and writes state[slots_out[b]] (int32 (B,); slots_in None: slot b; slots_out
    None: the slot it was read from); a row with a slot outside the pool is skipped and its y is zero.
    A slot that one row writes must not be read or written by another. Fills and returns ``y`` (B, D)."""

    def __init__(self, x, r, i, lam, state, c: float = 8.0, slots_in=None, slots_out=None, out=None, stream=None):
        lib = _b.load_library()
        if x.dim() != 2:
            raise ValueError("x must be (batch, d_inner)")
        dev = x.device
        if dev.type != "cuda":
            raise ValueError("inputs must be on a GPU device")
        io = _b._io_code(x.dtype)
        Bsz, D = x.shape
        for t, name in ((r, "r"), (i, "i")):
            _check_tensor(t, name, dev, x.dtype, (Bsz, D), dense=False)
        _check_tensor(lam, "lam", dev, torch.float32, (D,))
        if state.dim() != 2:
            raise ValueError("state must be (slots, d_inner)")
        _check_tensor(state, "state", dev, torch.float32, (state.shape[0], D))
        for t, name in ((slots_in, "slots_in"), (slots_out, "slots_out")):
            if t is not None:
                _check_tensor(t, name, dev, torch.int32, (Bsz,))
        self.y = _output(out, "out", dev, x.dtype, (Bsz, D))
        launch = _b.make_launch(Bsz, 1, D, 1, io, 0, stream=_stream_of(dev, stream))
        g = _Gated(_ptr(x), _ptr(r), _ptr(i), row_stride(x, "x"), row_stride(r, "r"), row_stride(i, "i"), _ptr(lam),
                   None, None, 0, float(c))
        args = (ctypes.byref(g), _ptr(state), int(state.shape[0]), _ptr(slots_in), _ptr(slots_out), _ptr(self.y),
                ctypes.byref(launch))
        self._prepare(dev, stream, launch, lib.vimscan_gated_step, args, [self.y] if out is None else [],
                      (g, x, r, i, lam, state, slots_in, slots_out))

    def __call__(self):
        self._queue()
        return self.y


def gated_fwd(x, r, i, lam, c: float = 8.0, h0=None, seg_len: int = 0, offsets=None, reverse: bool = False, out=None):
    """The gated linear recurrence on the GPU: (y, h_last); arguments as ``PreparedGated``. Queued on
    torch's current stream; does not synchronise."""
    call = PreparedGated(x, r, i, lam, c, h0, seg_len, offsets, reverse, out)
    call()
    return call.y, call.h_last


def gated_step(x, r, i, lam, state, c: float = 8.0, slots_in=None, slots_out=None, out=None):
    """One token of a batch of streams, ``state`` updated in place; arguments as ``PreparedGatedStep``."""
    return PreparedGatedStep(x, r, i, lam, state, c, slots_in, slots_out, out)()


def gated_info(batch, seqlen, d_inner, seg_len=0, io_dtype="bf16", nseq=None, backward=False) -> dict:
    """The library's plan for a gated recurrence of this shape (host only; vimscan_gated_plan); nseq:
    the number of sequences when they are given by offsets."""
    code = _b.VIMSCAN_BF16 if io_dtype == "bf16" else _b.VIMSCAN_F32
    launch = _b.make_launch(batch, seqlen, d_inner, 1, code)
    plan = _b._Plan()
    _b._check(_b.load_library().vimscan_gated_plan(ctypes.byref(launch), int(seg_len), int(nseq is not None),
                                                   int(nseq or 0), int(backward), ctypes.byref(plan)))
    return _plan_dict(plan)


def gated_wait_reads(reads: int = 4096):
    """How often a workgroup of a gated recurrence reads a state that is not handed over yet before it goes on
    alone, from the inputs (vimscan_gated_wait_reads): for the calls queued from now on. The results do not
    depend on it."""
    _b._check(_b.load_library().vimscan_gated_wait_reads(int(reads)))


def gated_alone() -> int:
    """Workgroups of gated recurrences on the current device that went on alone since the library was loaded
    (vimscan_gated_alone). Synchronous."""
    n = ctypes.c_uint64(0)
    _b._check(_b.load_library().vimscan_gated_alone(ctypes.byref(n)))
    return int(n.value)


# ------------------------------------------------------------------------------------------
# Block norm


class _NormInputs:
    def __init__(self, x, z, w_post, residual, gamma, w_pre, eps, gate_after, res_dtype):
        if x.dim() < 1:
            raise ValueError("x must be (..., d)")
        dev = x.device
        if dev.type != "cuda":
            raise ValueError("inputs must be on a GPU device")
        self.io = _b._io_code(x.dtype)
        self.dev, self.dtype, self.shape = dev, x.dtype, tuple(x.shape)
        D = x.shape[-1]
        self.rows = 1
        for v in x.shape[:-1]:
            self.rows *= v
        if z is not None:
            _check_tensor(z, "z", dev, x.dtype, self.shape, dense=False)
        for t, name in ((w_post, "w_post"), (gamma, "gamma"), (w_pre, "w_pre")):
            if t is not None:
                _check_tensor(t, name, dev, torch.float32, (D,))
        if residual is not None:
            if res_dtype is not None and res_dtype != residual.dtype:
                raise ValueError("res_dtype is the residual's dtype")
            res_dtype = residual.dtype
            _check_tensor(residual, "residual", dev, res_dtype, self.shape)
        self.res_dtype = x.dtype if res_dtype is None else res_dtype
        if gate_after and (z is None or w_post is None):
            raise ValueError("gate_after needs z and w_post")
        self.flags = FLAG_GATE_AFTER if gate_after else 0
        self.tensors = (x, z, w_post, residual, gamma, w_pre)
        self.struct = _Norm(_ptr(x), _ptr(z), row_stride(x, "x"), row_stride(z, "z") if z is not None else D,
                            _ptr(w_post), _ptr(residual), _ptr(gamma), _ptr(w_pre), float(eps),
                            _b._io_code(self.res_dtype))

    def launch(self, stream):
        launch = _b.make_launch(self.rows, 1, self.shape[-1], 0, self.io, 0, stream=stream)
        launch.flags = self.flags
        return launch


class PreparedBlockNorm(_Call):
    """What stands between two blocks, fused (vimscan_norm_fwd). Per row of x (..., D):

        p = rmsnorm(x silu(z)) w_post          (gate_after: rmsnorm(x) w_post silu(z))
        sum = residual + gamma p,  n = rmsnorm(sum) w_pre

    Every argument but x may be None, which leaves its stage out. x, z: float32 or bfloat16, alike,
    rows evenly spaced; w_post, gamma, w_pre: (D,) float32; residual like x, contiguous, in x's dtype
    or float32. Calling it fills ``sum`` (the residual's dtype, without one res_dtype or x's; None
    with ``with_sum`` false) and ``n`` (x's dtype; None without w_pre) and returns both. ``out_sum``
    may be the residual itself."""

    def __init__(self, x, z=None, w_post=None, residual=None, gamma=None, w_pre=None, eps: float = 1e-5,
                 gate_after: bool = False, res_dtype=None, out_sum=None, out_n=None, with_sum: bool = True, stream=None):
        lib = _b.load_library()
        inp = _NormInputs(x, z, w_post, residual, gamma, w_pre, eps, gate_after, res_dtype)
        if not with_sum and (w_pre is None or out_sum is not None):
            raise ValueError("without the sum there must be w_pre and no out_sum")
        if w_pre is None and out_n is not None:
            raise ValueError("out_n needs w_pre")
        self.sum = _output(out_sum, "out_sum", inp.dev, inp.res_dtype, inp.shape) if with_sum else None
        self.n = _output(out_n, "out_n", inp.dev, inp.dtype, inp.shape) if w_pre is not None else None
        launch = inp.launch(_stream_of(inp.dev, stream))
        args = (ctypes.byref(inp.struct), _ptr(self.sum), _ptr(self.n), ctypes.byref(launch))
        own = [t for t, gv in ((self.sum, out_sum), (self.n, out_n)) if t is not gv]
        self._prepare(inp.dev, stream, launch, lib.vimscan_norm_fwd, args, own, (inp,))

    def __call__(self):
        self._queue()
        return self.sum, self.n


class PreparedBlockNormGrad(_Call):
    """Gradients of a block norm (vimscan_norm_bwd) from its inputs and the gradients dsum and dn of its
    outputs (None: zero). Calling it fills ``dx``, ``dz``, ``dresidual`` and the sums over the rows
    ``dw_post``, ``dgamma``, ``dw_pre`` (float32; ``weights`` false leaves them out); those of absent
    inputs are None."""

    def __init__(self, x, z=None, w_post=None, residual=None, gamma=None, w_pre=None, dsum=None, dn=None,
                 eps: float = 1e-5, gate_after: bool = False, res_dtype=None, weights: bool = True, workspace=None,
                 stream=None):
        lib = _b.load_library()
        if dsum is not None and residual is None and res_dtype is None:
            res_dtype = dsum.dtype
        inp = _NormInputs(x, z, w_post, residual, gamma, w_pre, eps, gate_after, res_dtype)
        dev, D = inp.dev, inp.shape[-1]
        if dn is not None and w_pre is None:
            raise ValueError("dn needs w_pre")
        if dsum is not None:
            _check_tensor(dsum, "dsum", dev, inp.res_dtype, inp.shape)
        if dn is not None:
            _check_tensor(dn, "dn", dev, inp.dtype, inp.shape)
        self.dx = torch.empty(inp.shape, dtype=inp.dtype, device=dev)
        self.dz = torch.empty(inp.shape, dtype=inp.dtype, device=dev) if z is not None else None
        self.dresidual = torch.empty(inp.shape, dtype=inp.res_dtype, device=dev) if residual is not None else None
        self.dw_post, self.dgamma, self.dw_pre = (
            torch.empty(D, dtype=torch.float32, device=dev) if weights and t is not None else None
            for t in (w_post, gamma, w_pre))
        launch = inp.launch(_stream_of(dev, stream))
        plan = _b._Plan()
        _b._check(lib.vimscan_norm_plan(ctypes.byref(launch), 1, ctypes.byref(plan)))
        self.plan = _plan_dict(plan)
        ws = _workspace(workspace, plan.workspace_bytes, dev, launch)
        g = _NormGrad(_ptr(dsum), _ptr(dn), _ptr(self.dx), _ptr(self.dz), D, D, _ptr(self.dresidual),
                      _ptr(self.dw_post), _ptr(self.dgamma), _ptr(self.dw_pre))
        args = (ctypes.byref(inp.struct), ctypes.byref(g), ctypes.byref(launch))
        own = [self.dx, self.dz, self.dresidual, self.dw_post, self.dgamma, self.dw_pre]
        own += [ws] if ws is not workspace else []
        self._prepare(dev, stream, launch, lib.vimscan_norm_bwd, args, own, (inp, g, dsum, dn, ws))

    def __call__(self):
        self._queue()
        return self.dx


def block_norm(x, z=None, w_post=None, residual=None, gamma=None, w_pre=None, eps: float = 1e-5,
               gate_after: bool = False, res_dtype=None, with_sum: bool = True):
    """The block norm on the GPU: (sum, n); arguments as ``PreparedBlockNorm``. Queued on torch's
    current stream; does not synchronise."""
    return PreparedBlockNorm(x, z, w_post, residual, gamma, w_pre, eps, gate_after, res_dtype, with_sum=with_sum)()


def norm_info(rows, d, io_dtype="bf16", backward=False) -> dict:
    """The library's plan for a block norm of this shape (host only; vimscan_norm_plan)."""
    code = _b.VIMSCAN_BF16 if io_dtype == "bf16" else _b.VIMSCAN_F32
    launch = _b.make_launch(rows, 1, d, 0, code)
    plan = _b._Plan()
    _b._check(_b.load_library().vimscan_norm_plan(ctypes.byref(launch), int(backward), ctypes.byref(plan)))
    return _plan_dict(plan)


# ------------------------------------------------------------------------------------------
# Layer norm


class _LayerNormInputs:
    def __init__(self, x, residual, weight, bias, eps, res_dtype):
        if x.dim() < 1:
            raise ValueError("x must be (..., d)")
        dev = x.device
        if dev.type != "cuda":
            raise ValueError("inputs must be on a GPU device")
        self.io = _b._io_code(x.dtype)
        self.dev, self.dtype, self.shape = dev, x.dtype, tuple(x.shape)
        self.rows = 1
        for v in x.shape[:-1]:
            self.rows *= v
        for t, name in ((weight, "weight"), (bias, "bias")):
            if t is not None:
                _check_tensor(t, name, dev, torch.float32, (x.shape[-1],))
        if residual is not None:
            if res_dtype is not None and res_dtype != residual.dtype:
                raise ValueError("res_dtype is the residual's dtype")
            res_dtype = residual.dtype
            _check_tensor(residual, "residual", dev, res_dtype, self.shape)
        self.res_dtype = x.dtype if res_dtype is None else res_dtype
        self.tensors = (x, residual, weight, bias)
        self.struct = _LayerNorm(_ptr(x), row_stride(x, "x"), _ptr(residual), _ptr(weight), _ptr(bias), float(eps),
                                 _b._io_code(self.res_dtype))

    def launch(self, stream):
        return _b.make_launch(self.rows, 1, self.shape[-1], 0, self.io, 0, stream=stream)


class PreparedLayerNorm(_Call):
    """Layer norm with the residual add in front of it (vimscan_layernorm_fwd). Per row of x (..., D):

        sum = x + residual,  n = (sum - mean) / sqrt(mean((sum - mean)^2) + eps) weight + bias

    residual, weight and bias may be None, which leaves them out. x: float32 or bfloat16, rows evenly spaced;
    weight, bias: (D,) float32; residual like x, contiguous, in x's dtype or float32. Calling it fills ``n`` (x's dtype) and
    ``sum`` (the residual's dtype, without one res_dtype or x's; None unless ``with_sum``, which is by default whether
    there is a residual) and returns both. ``out_sum`` may be the residual itself."""

    def __init__(self, x, residual=None, weight=None, bias=None, eps: float = 1e-5, res_dtype=None, out_sum=None,
                 out_n=None, with_sum=None, stream=None):
        lib = _b.load_library()
        inp = _LayerNormInputs(x, residual, weight, bias, eps, res_dtype)
        if with_sum is None:
            with_sum = residual is not None or out_sum is not None
        if not with_sum and out_sum is not None:
            raise ValueError("without the sum there must be no out_sum")
        self.sum = _output(out_sum, "out_sum", inp.dev, inp.res_dtype, inp.shape) if with_sum else None
        self.n = _output(out_n, "out_n", inp.dev, inp.dtype, inp.shape)
        launch = inp.launch(_stream_of(inp.dev, stream))
        args = (ctypes.byref(inp.struct), _ptr(self.sum), _ptr(self.n), ctypes.byref(launch))
        own = [t for t, gv in ((self.sum, out_sum), (self.n, out_n)) if t is not gv]
        self._prepare(inp.dev, stream, launch, lib.vimscan_layernorm_fwd, args, own, (inp,))

    def __call__(self):
        self._queue()
        return self.sum, self.n


class PreparedLayerNormGrad(_Call):
    """Gradients of a layer norm (vimscan_layernorm_bwd) from its inputs and the gradients dsum and dn of its
    outputs (None: zero). Calling it fills ``dx``, ``dresidual`` and the sums over the rows ``dweight`` and ``dbias``
    (float32; ``weights`` false leaves them out); those of absent inputs are None."""

    def __init__(self, x, residual=None, weight=None, bias=None, dsum=None, dn=None, eps: float = 1e-5, res_dtype=None,
                 weights: bool = True, workspace=None, stream=None):
        lib = _b.load_library()
        if dsum is not None and residual is None and res_dtype is None:
            res_dtype = dsum.dtype
        inp = _LayerNormInputs(x, residual, weight, bias, eps, res_dtype)
        dev, D = inp.dev, inp.shape[-1]
        if dsum is not None:
            _check_tensor(dsum, "dsum", dev, inp.res_dtype, inp.shape)
        if dn is not None:
            _check_tensor(dn, "dn", dev, inp.dtype, inp.shape)
        self.dx = torch.empty(inp.shape, dtype=inp.dtype, device=dev)
        self.dresidual = torch.empty(inp.shape, dtype=inp.res_dtype, device=dev) if residual is not None else None
        self.dweight, self.dbias = (torch.empty(D, dtype=torch.float32, device=dev) if weights and t is not None else None
                                    for t in (weight, bias))
        launch = inp.launch(_stream_of(dev, stream))
        plan = _b._Plan()
        _b._check(lib.vimscan_layernorm_plan(ctypes.byref(launch), 1, ctypes.byref(plan)))
        self.plan = _plan_dict(plan)
        ws = _workspace(workspace, plan.workspace_bytes, dev, launch)
        g = _LayerNormGrad(_ptr(dsum), _ptr(dn), _ptr(self.dx), D, _ptr(self.dresidual), _ptr(self.dweight), _ptr(self.dbias))
        args = (ctypes.byref(inp.struct), ctypes.byref(g), ctypes.byref(launch))
        own = [self.dx, self.dresidual, self.dweight, self.dbias] + ([ws] if ws is not workspace else [])
        self._prepare(dev, stream, launch, lib.vimscan_layernorm_bwd, args, own, (inp, g, dsum, dn, ws))

    def __call__(self):
        self._queue()
        return self.dx


def layer_norm(x, residual=None, weight=None, bias=None, eps: float = 1e-5, res_dtype=None, with_sum=None):
    """The layer norm on the GPU: (sum, n); arguments as ``PreparedLayerNorm``. Queued on torch's current
    stream; does not synchronise."""
    return PreparedLayerNorm(x, residual, weight, bias, eps, res_dtype, with_sum=with_sum)()


def layernorm_info(rows, d, io_dtype="bf16", backward=False) -> dict:
    """The library's plan for a layer norm of this shape (host only; vimscan_layernorm_plan)."""
    code = _b.VIMSCAN_BF16 if io_dtype == "bf16" else _b.VIMSCAN_F32
    launch = _b.make_launch(rows, 1, d, 0, code)
    plan = _b._Plan()
    _b._check(_b.load_library().vimscan_layernorm_plan(ctypes.byref(launch), int(backward), ctypes.byref(plan)))
    return _plan_dict(plan)
