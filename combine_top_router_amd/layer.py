"""Device buffers of one MoE layer pass, allocated with PyTorch, and the call order of
the C ABI.  Every step runs in libmoe; torch only provides memory and the stream."""
from __future__ import annotations

import weakref

import torch

from . import lib as L

_DT = {L.MOE_BF16: torch.bfloat16, L.MOE_F32: torch.float32}


def _p(t):
    return 0 if t is None else t.data_ptr()


def stream_handle(stream=None) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _device(device) -> torch.device:
    d = torch.device(device)
    if d.type == "cuda" and d.index is None:
        d = torch.device("cuda", torch.cuda.current_device())
    return d


# the raw handle of a device's current stream, without the Stream object that
# torch.cuda.current_stream builds around it (2 us of a call of 8), and the current device
# without the check that CUDA is initialised (an operator's buffers have done that); a torch
# that lacks them, as one built without a GPU does, has the public ones
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or (lambda: torch.cuda.current_device())


class _OnDevice:
    """Checks and streams of the operators around the layer.  A call runs on `stream`, or on
    the current stream of the operator's own device; its buffers are reused from call to
    call, so calls of one operator on several streams have to be ordered by the caller.  The
    buffers' memory is that of the stream that is current when they are made, whose earlier
    work may still use it: the first call on another stream waits for that work."""

    _birth, _ordered = None, ()

    def _place(self, device):
        self.device = _device(device)
        self._index = self.device.index

    def _allocated(self):
        """Called behind every allocation of buffers."""
        if self._index is None:
            return
        with torch.cuda.device(self._index):
            if torch.cuda.is_current_stream_capturing():
                return   # a graph's memory pool is its own, and an event inside a capture is no other stream's
            home = torch.cuda.current_stream()
            if self._birth is not None and home.cuda_stream not in self._ordered:
                home.wait_event(self._birth)   # the new event stands for the buffers before, too
            self._birth, self._ordered = home.record_event(), {home.cuda_stream}

    def _order(self, handle, stream):
        """`stream` (None: the current one), of that handle, has not been used with the buffers."""
        if self._birth is None:
            return
        s = torch.cuda.current_stream(self._index) if stream is None else stream
        with torch.cuda.stream(s):
            if torch.cuda.is_current_stream_capturing():
                return   # takes no wait for work outside: that is the launch's to order, or the capture's start
            s.wait_event(self._birth)
        self._ordered.add(handle)

    def _capturing(self, stream):
        """Whether a call on `stream` (None: the current one of the operator's device) is captured."""
        if stream is None and _current_device() == self._index:
            return torch.cuda.is_current_stream_capturing()
        with torch.cuda.stream(torch.cuda.current_stream(self._index) if stream is None else stream):
            return torch.cuda.is_current_stream_capturing()

    def _check(self, t, shape, dtype, name):
        if t.dtype != dtype or t.shape != shape or t.get_device() != self._index or not t.is_contiguous():
            raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)} on {self.device}, got "
                             f"{t.dtype} {tuple(t.shape)} on {t.device}")

    def _call(self, func, stream, *args):
        s = _raw_stream(self._index) if stream is None else stream.cuda_stream
        if s not in self._ordered:
            self._order(s, stream)
        if _current_device() == self._index:
            func(*args, s)
        else:
            with torch.cuda.device(self._index):
                func(*args, s)


class MoeNorm(_OnDevice):
    """The norm in front of the layer (layer norm, or rms norm), with the residual sum before
    it.  ``forward`` gives y, and leaves ``sum`` (with a residual), ``mean`` and ``rstd``;
    ``backward`` reads its x, residual and weight again, which have to be as they were (the
    stored sum has been rounded).  dx is the gradient of x and of the residual alike."""

    def __init__(self, T, H, kind=L.MOE_NORM_LAYER, dtype=L.MOE_BF16, eps=1e-5, device="cuda"):
        self.shape = L.MoeNormShape(T, H, dtype, kind, eps)
        scratch_b = L.moe_norm_scratch_bytes(self.shape)
        self._place(device)
        dev = self.device
        dt = self.dtype = _DT[dtype]
        self._row, self._vec = torch.Size((T, H)), torch.Size((H,))
        self.y = torch.empty(T, H, dtype=dt, device=dev)
        self._sum = torch.empty(T, H, dtype=dt, device=dev)
        self.mean = torch.empty(T, dtype=torch.float32, device=dev) if kind == L.MOE_NORM_LAYER else None
        self.rstd = torch.empty(T, dtype=torch.float32, device=dev)
        self.dx = torch.empty(T, H, dtype=dt, device=dev)
        self.dw = torch.empty(H, dtype=dt, device=dev)
        self.db = torch.empty(H, dtype=dt, device=dev)
        self.scratch = torch.empty(scratch_b, dtype=torch.uint8, device=dev)
        # the buffers stay where they are
        self._p_sum, self._p_y, self._p_mean, self._p_rstd = _p(self._sum), _p(self.y), _p(self.mean), _p(self.rstd)
        self._p_dx, self._p_dw, self._p_scratch = _p(self.dx), _p(self.dw), _p(self.scratch)
        self.sum = None
        self.inputs = None
        self._allocated()

    def forward(self, x, w, b=None, res=None, stream=None):
        self._check(x, self._row, self.dtype, "x")
        self._check(w, self._vec, self.dtype, "w")
        if b is not None:
            self._check(b, self._vec, self.dtype, "b")
        if res is not None:
            self._check(res, self._row, self.dtype, "res")
        self.sum = None if res is None else self._sum
        self.inputs = (x, res, w, b is not None)
        self._call(L.moe_norm_fwd, stream, self.shape, _p(x), _p(res), _p(w), _p(b), 0 if res is None else self._p_sum,
                   self._p_y, self._p_mean, self._p_rstd)
        return self.y

    def backward(self, dy, ds_in=None, stream=None):
        if self.inputs is None:
            raise RuntimeError("backward without a forward")
        self._check(dy, self._row, self.dtype, "dy")
        if ds_in is not None:
            self._check(ds_in, self._row, self.dtype, "ds_in")
        x, res, w, bias = self.inputs
        db = self.db if bias else None
        self._call(L.moe_norm_bwd, stream, self.shape, _p(dy), _p(x), _p(res), _p(w), self._p_mean, self._p_rstd,
                   _p(ds_in), self._p_dx, self._p_dw, _p(db), self._p_scratch)
        return {"dx": self.dx, "dw": self.dw, "db": db}


class BalanceLoss(_OnDevice):
    """The router's load-balance loss over all E experts.  ``forward`` gives the loss and
    leaves ``counts`` [E + 1] (per expert, then the counted tokens) and ``prob`` [E];
    ``backward`` gives d_logits, added to d_logits_in (in place if ``out`` is that)."""

    def __init__(self, T, E, k, device="cuda"):
        self.shape = L.MoeShape(T, 64, 64, E, k, 0, E, L.MOE_BF16, L.MOE_BWD_SAME, 1, L.MOE_FWD_SAME, 0, 0)
        scratch_b = L.moe_balance_scratch_bytes(self.shape)
        self._place(device)
        dev = self.device
        f32 = torch.float32
        self._logits, self._idx, self._mask = torch.Size((T, E)), torch.Size((T, k)), torch.Size((T,))
        self.loss = torch.empty(1, dtype=f32, device=dev)
        self.counts = torch.empty(E + 1, dtype=torch.int32, device=dev)
        self.prob = torch.empty(E, dtype=f32, device=dev)
        self.d_logits = torch.empty(T, E, dtype=f32, device=dev)
        self.scratch = torch.empty(scratch_b, dtype=torch.uint8, device=dev)
        self._p_fwd = (_p(self.loss), _p(self.counts), _p(self.prob), _p(self.scratch))
        self.inputs = None
        self._allocated()

    def forward(self, logits, topk_idx, coef, mask=None, stream=None):
        self._check(logits, self._logits, torch.float32, "logits")
        self._check(topk_idx, self._idx, torch.int32, "topk_idx")
        if mask is not None:
            self._check(mask, self._mask, torch.uint8, "mask")
        self.inputs = (logits, mask, float(coef))
        self._call(L.moe_balance_fwd, stream, self.shape, _p(logits), _p(topk_idx), _p(mask), coef, *self._p_fwd)
        return self.loss

    def backward(self, d_loss=None, d_logits_in=None, out=None, stream=None):
        if self.inputs is None:
            raise RuntimeError("backward without a forward")
        if d_loss is not None:
            self._check(d_loss, self.loss.shape, torch.float32, "d_loss")
        if d_logits_in is not None:
            self._check(d_logits_in, self._logits, torch.float32, "d_logits_in")
        if out is None:
            out = self.d_logits
        else:
            self._check(out, self._logits, torch.float32, "out")
        logits, mask, coef = self.inputs
        self._call(L.moe_balance_bwd, stream, self.shape, _p(logits), self._p_fwd[1], _p(mask), coef, _p(d_loss),
                   _p(d_logits_in), _p(out))
        return out


class Orthogonalizer(_OnDevice):
    """Orthogonalised updates of n weight matrices of one size (the experts' gradients, or
    their momentum), by Newton-Schulz steps as in the Muon optimiser.

    ``scratch``: uint8 memory of at least ``moe_orth_scratch_bytes``, such as that of another
    Orthogonalizer whose calls are ordered with this one's; by default it makes its own (about
    three times a bf16 g, and 4 m^2 bytes a matrix of shorter side m)."""

    def __init__(self, n, rows, cols, dtype=L.MOE_BF16, steps=5, device="cuda", scratch=None):
        self.shape = L.MoeOrthShape(n, rows, cols, dtype, steps)
        scratch_b = L.moe_orth_scratch_bytes(self.shape)
        self._place(device)
        dev = self.device
        self.dtype = _DT[dtype]
        self._size = torch.Size((n, rows, cols))
        self.o = None
        if scratch is None:
            scratch = torch.empty(scratch_b, dtype=torch.uint8, device=dev)
        else:
            self._check(scratch, scratch.shape, torch.uint8, "scratch")
            if scratch.numel() < scratch_b or scratch.data_ptr() % 256:
                raise ValueError(f"scratch: expected {scratch_b} bytes at a multiple of 256, got {scratch.numel()} "
                                 f"at {scratch.data_ptr():#x}")
        self.scratch = scratch
        self._allocated()

    def update(self, g, scale=1.0, out=None, stream=None):
        self._check(g, self._size, self.dtype, "g")
        if out is None:
            if self.o is None:
                self.o = torch.empty(self._size, dtype=torch.bfloat16, device=self.device)
                self._allocated()
            out = self.o
        else:
            self._check(out, self._size, torch.bfloat16, "out")
        self._call(L.moe_orthogonalize, stream, self.shape, _p(g), _p(out), scale, _p(self.scratch))
        return out


class Gate(_OnDevice):
    """Routing by scores: softmax or sigmoid, with a bias that evens the load, groups of experts
    and renormalised weights.  ``forward`` gives (topk_idx [T, k], topk_w [T, k]), and with
    ``count`` leaves the chosen slots per expert in ``counts`` [E]; ``backward`` reads its
    logits again and gives d_logits (to ``out``, if given); ``update_bias`` takes a step of the
    bias towards an even load, in place or to ``out``, by the last counts or the given ones
    (such as their sum over GPUs)."""

    def __init__(self, T, E, k, score=L.MOE_SCORE_SOFTMAX, groups=1, topk_groups=1, group_top=1, renorm=1, scale=1.0,
                 device="cuda"):
        self.shape = L.MoeGateShape(T, E, k, score, groups, topk_groups, group_top, renorm, scale)
        scratch_b = L.moe_gate_scratch_bytes(self.shape)
        self._place(device)
        dev, f32 = self.device, torch.float32
        self._logits, self._slots = torch.Size((T, E)), torch.Size((T, k))
        self._mask, self._bias = torch.Size((T,)), torch.Size((E,))
        self.topk_idx = torch.empty(T, k, dtype=torch.int32, device=dev)
        self.topk_w = torch.empty(T, k, dtype=f32, device=dev)
        self.d_logits = torch.empty(T, E, dtype=f32, device=dev)
        self.counts = torch.empty(E, dtype=torch.int32, device=dev)
        self.scratch = torch.empty(scratch_b, dtype=torch.uint8, device=dev)
        self._p_idx, self._p_w, self._p_counts = _p(self.topk_idx), _p(self.topk_w), _p(self.counts)
        self._p_scratch = _p(self.scratch)
        self.inputs, self._counted = None, False
        self.layer = None   # weak, the MoeLayer that routes by it
        self._allocated()

    def forward(self, logits, bias=None, mask=None, count=False, stream=None):
        self._check(logits, self._logits, torch.float32, "logits")
        if bias is not None:
            self._check(bias, self._bias, torch.float32, "bias")
        if mask is not None:
            self._check(mask, self._mask, torch.uint8, "mask")
        self.inputs, self._counted = logits, count
        self._call(L.moe_gate_fwd, stream, self.shape, _p(logits), _p(bias), _p(mask), self._p_idx, self._p_w,
                   self._p_counts if count else 0, self._p_scratch)
        return self.topk_idx, self.topk_w

    def backward(self, d_topk_w, out=None, stream=None):
        if self.inputs is None:
            raise RuntimeError("backward without a forward")
        self._check(d_topk_w, self._slots, torch.float32, "d_topk_w")
        if out is None:
            out = self.d_logits
        else:
            self._check(out, self._logits, torch.float32, "out")
        self._call(L.moe_gate_bwd, stream, self.shape, _p(self.inputs), self._p_idx, _p(d_topk_w), _p(out))
        return out

    def update_bias(self, bias, rate, counts=None, out=None, stream=None):
        if counts is None:
            if not self._counted:
                raise RuntimeError("update_bias without counts: the last forward has not counted")
            counts = self.counts
        else:
            self._check(counts, self._bias, torch.int32, "counts")
        self._check(bias, self._bias, torch.float32, "bias")
        if out is None:
            out = bias
        else:
            self._check(out, self._bias, torch.float32, "out")
        self._call(L.moe_gate_update_bias, stream, self.shape, _p(counts), _p(bias), rate, _p(out))
        return out


class Linear(_OnDevice):
    """y = act(x W + b) + res, W [K, N].  ``forward`` gives y; ``backward`` reads its x and W
    again, which have to be as they were, and gives dx (with ``dx_in`` added), dw and db; the
    gradient of res is dy.  ``train=False`` keeps nothing for a backward."""

    def __init__(self, T, K, N, act=L.MOE_ACT_NONE, dtype=L.MOE_BF16, train=True, device="cuda"):
        self.shape = L.MoeLinearShape(T, K, N, dtype, act)
        scratch_b = L.moe_linear_scratch_bytes(self.shape) if train else L.moe_linear_fwd_scratch_bytes(self.shape)
        self._place(device)
        dev = self.device
        dt = self.dtype = _DT[dtype]
        self._x, self._w, self._y, self._b = (torch.Size(d) for d in ((T, K), (K, N), (T, N), (N,)))
        self.train = train
        self.y = torch.empty(T, N, dtype=dt, device=dev)
        self.z = torch.empty(T, N, dtype=dt, device=dev) if train and act != L.MOE_ACT_NONE else None
        self.dx = torch.empty(T, K, dtype=dt, device=dev) if train else None
        self.dw = torch.empty(K, N, dtype=dt, device=dev) if train else None
        self.db = torch.empty(N, dtype=dt, device=dev) if train else None
        self.scratch = torch.empty(scratch_b, dtype=torch.uint8, device=dev)
        self._p_y, self._p_z, self._p_dx, self._p_dw = _p(self.y), _p(self.z), _p(self.dx), _p(self.dw)
        self._p_scratch = _p(self.scratch)
        self.inputs = None
        self._allocated()

    def forward(self, x, w, b=None, res=None, stream=None):
        self._check(x, self._x, self.dtype, "x")
        self._check(w, self._w, self.dtype, "w")
        if b is not None:
            self._check(b, self._b, self.dtype, "b")
        if res is not None:
            self._check(res, self._y, self.dtype, "res")
        self.inputs = (x, w, b is not None) if self.train else None
        self._call(L.moe_linear_fwd, stream, self.shape, _p(x), _p(w), _p(b), _p(res), self._p_z, self._p_y,
                   self._p_scratch)
        return self.y

    def backward(self, dy, dx_in=None, stream=None):
        if not self.train:
            raise RuntimeError("backward of a Linear made with train=False")
        if self.inputs is None:
            raise RuntimeError("backward without a forward")
        self._check(dy, self._y, self.dtype, "dy")
        if dx_in is not None:
            self._check(dx_in, self._x, self.dtype, "dx_in")
        x, w, bias = self.inputs
        db = self.db if bias else None
        self._call(L.moe_linear_bwd, stream, self.shape, _p(dy), _p(x), _p(w), self._p_z, _p(dx_in), self._p_dx,
                   self._p_dw, _p(db), self._p_scratch)
        return {"dx": self.dx, "dw": self.dw, "db": db}


class AdamW(_OnDevice):
    """AdamW over a list of parameter tensors (bf16 or fp32, in any mix), all in one call.

    The moments lie one tensor behind the other in ``m`` and ``v``, each from a multiple of 32
    elements on (``moments(i)`` gives a tensor's as fp32): fp32, or with MOE_STATE_8BIT E4M3
    codes with one e8m0 scale per 32 elements in ``m_scale`` and ``v_scale``.  ``master``: an
    fp32 copy of each bf16 parameter in the list ``master`` is what is updated.
    ``stochastic`` rounds 8-bit moments, and bf16 parameters without a copy, stochastically, by
    random bits from ``seed``, the step and the element's place.  ``t`` is the number of steps taken.  With
    ``capturable`` it is held on the device and counted there, so that a captured step goes on
    at every replay; reading and setting it then wait for the device."""

    def __init__(self, params, state=L.MOE_STATE_F32, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, master=False,
                 stochastic=False, seed=0, capturable=False):
        params = list(params)
        if not params:
            raise ValueError("params: no tensors")
        self._place(params[0].device)
        codes = {dt: c for c, dt in _DT.items()}
        for i, p in enumerate(params):
            if p.dtype not in codes:
                raise ValueError(f"params[{i}]: expected bfloat16 or float32, got {p.dtype}")
            if p.device != self.device or not p.is_contiguous():
                raise ValueError(f"params[{i}]: expected a contiguous tensor on {self.device}, got one on {p.device}")
        spans = sorted((p.data_ptr(), p.data_ptr() + p.numel() * p.element_size(), i) for i, p in enumerate(params)
                       if p.numel())
        for a, b in zip(spans, spans[1:]):
            if b[0] < a[1]:
                raise ValueError(f"params[{a[2]}] and params[{b[2]}] overlap")
        self.params = params
        self.hyper = L.MoeAdamwParams(0.0, betas[0], betas[1], eps, weight_decay, 1, seed & 0xFFFFFFFFFFFFFFFF, state,
                                      int(stochastic))
        L.moe_adamw(self.hyper, None, 0, 0, 0, 0)   # refuses what it would refuse at the first step
        dev, f32, u8 = self.device, torch.float32, torch.uint8
        self._at, total = [], 0
        for p in params:
            self._at.append(total)
            total += -(-p.numel() // 32) * 32
        eight = self._eight = state == L.MOE_STATE_8BIT
        self.m, self.v = (torch.zeros(total, dtype=u8 if eight else f32, device=dev) for _ in range(2))
        self.m_scale, self.v_scale = (torch.full((total // 32,), 127, dtype=u8, device=dev) if eight else None
                                      for _ in range(2))
        self.master = [p.detach().float() if p.dtype == torch.bfloat16 else None for p in params] if master else None
        self._clock = torch.zeros(L.MOE_ADAMW_CLOCK_BYTES // 8, dtype=torch.int64, device=dev) if capturable else None
        self._t = 0
        self._codes = codes
        self._ptrs = [p.data_ptr() for p in params]
        self._shapes = [p.shape for p in params]
        self._table = (L.MoeAdamwTensor * len(params))()
        self._entries = list(self._table)   # views of it
        width = 1 if eight else 4
        for i, (p, at, e) in enumerate(zip(params, self._at, self._entries)):
            e.p, e.m, e.v = self._ptrs[i], self.m.data_ptr() + at * width, self.v.data_ptr() + at * width
            if eight:
                e.m_scale, e.v_scale = self.m_scale.data_ptr() + at // 32, self.v_scale.data_ptr() + at // 32
            if master and self.master[i] is not None:
                e.master = self.master[i].data_ptr()
            e.n, e.at, e.p_dtype = p.numel(), at, codes[p.dtype]
        self._allocated()

    @property
    def t(self):
        if self._clock is None:
            return self._t
        self._finish()
        return int(self._clock[0])

    @t.setter
    def t(self, value):
        if self._clock is None:
            self._t = int(value)
        else:
            self._finish()
            self._clock[0] = int(value)
            self._finish()

    def _finish(self):
        """The clock is counted on the steps' streams, which may be others than the current one."""
        if self.device.type == "cuda":
            torch.cuda.synchronize(self.device)

    def moments(self, i):
        """(m, v) of tensor i as fp32 copies of its shape."""
        at, p = self._at[i], self.params[i]
        n, out = p.numel(), []
        for x, scale in ((self.m, self.m_scale), (self.v, self.v_scale)):
            if self._eight:
                end = at + -(-n // 32) * 32
                x = x[at:end].view(torch.float8_e4m3fn).float().view(-1, 32)
                # 2^(scale - 127) from its bits (a power function is not exact on the GPU), as the kernel has it
                e = scale[at // 32:end // 32].to(torch.int32).clamp(max=254)
                e = torch.where(e > 0, e << 23, 0x400000).to(torch.int32).view(torch.float32)
                x = (x * e[:, None]).view(-1)[:n]
                x = torch.square(x) if scale is self.v_scale else x
            else:
                x = x[at:at + n].clone()
            out.append(x.view(p.shape))
        return tuple(out)

    def step(self, grads, lr, grad_scale=None, stream=None):
        """One step with a gradient for each parameter (bf16 or fp32; None: that one is left
        alone).  lr: a number, or a device fp32 tensor [1], such as a captured step reads anew at
        every replay; grad_scale: a device fp32 tensor [1] that the gradients are multiplied by."""
        if self._clock is None and self.device.type == "cuda" and self._capturing(stream):
            raise RuntimeError("a captured step needs capturable=True: its number would be the same at every replay")
        if len(grads) != len(self.params):
            raise ValueError(f"grads: expected {len(self.params)}, got {len(grads)}")
        index, codes = self._index, self._codes
        for i, (g, e, p, ptr, shape) in enumerate(zip(grads, self._entries, self.params, self._ptrs, self._shapes)):
            if p.data_ptr() != ptr:
                raise ValueError(f"params[{i}] has been given other memory")
            if g is None:
                e.g = 0
                continue
            code = codes.get(g.dtype)
            if code is None or g.shape != shape or g.get_device() != index or not g.is_contiguous():
                raise ValueError(f"grads[{i}]: expected contiguous bfloat16 or float32 {tuple(shape)} on "
                                 f"{self.device}, got {g.dtype} {tuple(g.shape)} on {g.device}")
            e.g, e.g_dtype = g.data_ptr(), code
        if isinstance(lr, torch.Tensor):
            self._check(lr, torch.Size((1,)), torch.float32, "lr")
            p_lr = lr.data_ptr()
        else:
            self.hyper.lr, p_lr = lr, 0
        if grad_scale is not None:
            self._check(grad_scale, torch.Size((1,)), torch.float32, "grad_scale")
        self.hyper.step = self._t + 1
        self._call(L.moe_adamw, stream, self.hyper, self._table, len(self.params), p_lr, _p(grad_scale),
                   _p(self._clock))
        if self._clock is None:
            self._t += 1


class MoeLayer:
    """One GPU's share of a dropless MoE layer: experts [e_begin, e_begin + e_local) of E.

    ``forward`` runs route -> dispatch -> expert MLP -> combine and ``backward`` runs the
    expert backward and the router backward.  ``recompute=1`` keeps nothing between the two
    (activation checkpointing: the backward recomputes the gate/up GEMM).  With ``fuse_gather`` the token rows are
    read from x through row_src inside the GEMMs instead of a gathered copy xp.

    The shares of an expert-parallel layer see the same T tokens and all E logits; y, dx and
    d_logits of a share are its part of a sum over the shares.

    ``balance`` gives the load-balance loss of the last forward's routing, whole on every share
    (not to be summed over them); the backward then adds its gradient to d_logits, on the share
    that holds expert 0 alone, so that the sum counts it once.  ``orthogonalize`` turns the last backward's weight
    gradients into orthogonalised updates.  Both allocate their buffers on first use.

    ``gate``: a ``Gate`` of the same T, E and k routes in place of the softmax of the logits (and
    of ``renorm``); ``forward`` then takes its bias, its mask and ``count``, and tokens that the
    mask leaves out get y = 0.  ``balance`` has its own mask: without it such tokens' logits count
    in the loss.  A gate is one layer's: the backward reads what it holds.
    """

    def __init__(self, T, H, I, E, k, e_begin=0, e_local=None, dtype=L.MOE_BF16, bwd=L.MOE_BWD_SAME,
                 renorm=1, device="cuda", fuse_gather=True, fwd=L.MOE_FWD_SAME, recompute=0, row_tile=0, gate=None):
        e_local = E if e_local is None else e_local
        self.shape = L.MoeShape(T, H, I, E, k, e_begin, e_local, dtype, bwd, renorm, fwd, recompute, row_tile)
        self.device = torch.device(device)
        if self.device.type == "cuda" and self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.dtype = _DT[dtype]
        if gate is not None and ((gate.shape.T, gate.shape.E, gate.shape.k) != (T, E, k) or gate.device != self.device):
            raise ValueError(f"gate: expected T = {T}, E = {E}, k = {k} on {self.device}, got T = {gate.shape.T}, "
                             f"E = {gate.shape.E}, k = {gate.shape.k} on {gate.device}")
        if gate is not None:
            if gate.layer is not None and gate.layer() is not None:
                raise ValueError("gate: another layer has it, whose backward would find this one's routing")
            gate.layer = weakref.ref(self)
        self.gate = gate
        saved_b, scratch_b = L.moe_workspace_bytes(self.shape)
        self.R_cap = T * min(k, e_local)
        dev, i32, f32 = self.device, torch.int32, torch.float32
        self.topk_idx = torch.empty(T, k, dtype=i32, device=dev) if gate is None else gate.topk_idx
        self.topk_w = torch.empty(T, k, dtype=f32, device=dev) if gate is None else gate.topk_w
        self.counts = torch.empty(e_local, dtype=i32, device=dev)
        self.offsets = torch.empty(e_local + 1, dtype=i32, device=dev)
        self.row_src = torch.empty(max(self.R_cap, 1), dtype=i32, device=dev)
        self.row_of = torch.empty(max(T * k, 1), dtype=i32, device=dev)
        self.xp = None if fuse_gather else torch.empty(self.R_cap, H, dtype=self.dtype, device=dev)
        self.yp = torch.empty(max(self.R_cap, 1), H, dtype=self.dtype, device=dev)
        self.y = torch.empty(T, H, dtype=self.dtype, device=dev)
        # with recompute nothing is kept between forward and backward: no saved buffer at all
        self.saved = None if recompute else torch.empty(max(saved_b, 256), dtype=torch.uint8, device=dev)
        self.scratch = torch.empty(max(scratch_b, 256), dtype=torch.uint8, device=dev)
        self.dx = torch.empty(T, H, dtype=self.dtype, device=dev)
        self.dw_gate = torch.empty(e_local, H, I, dtype=self.dtype, device=dev)
        self.dw_up = torch.empty(e_local, H, I, dtype=self.dtype, device=dev)
        self.dw_down = torch.empty(e_local, I, H, dtype=self.dtype, device=dev)
        self.d_topk_w = torch.empty(T, k, dtype=f32, device=dev)
        self.d_logits = torch.empty(T, E, dtype=f32, device=dev)
        self.inputs = None
        self._balance, self._balanced = None, False
        self._orth, self._updates = {}, {}
        self._has_grads = False

    def _check(self, t, shape, dtype, name):
        if t.device != self.device or t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
            raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)} on {self.device}, got "
                             f"{t.dtype} {tuple(t.shape)} on {t.device}")

    def route(self, logits, stream=None, bias=None, mask=None, count=False):
        s = self.shape
        self._check(logits, (s.T, s.E), torch.float32, "logits")
        if self.gate is not None:
            self.gate.forward(logits, bias=bias, mask=mask, count=count, stream=stream)
            return
        if bias is not None or mask is not None or count:
            raise ValueError("bias, mask and count need a layer made with a gate")
        L.moe_route_topk(s, _p(logits), _p(self.topk_idx), _p(self.topk_w), stream_handle(stream))

    def dispatch(self, x, stream=None):
        self._balanced = False   # a new pass
        L.moe_dispatch(self.shape, _p(self.topk_idx), _p(x), _p(self.counts), _p(self.offsets), _p(self.row_src),
                       _p(self.row_of), _p(self.xp), _p(self.scratch), stream_handle(stream))

    def experts(self, x, w_gate, w_up, w_down, stream=None):
        L.moe_fwd(self.shape, _p(x), _p(self.xp), _p(self.offsets), _p(self.row_src), _p(self.topk_w), _p(w_gate),
                  _p(w_up), _p(w_down), _p(self.yp), _p(self.saved), _p(self.scratch), stream_handle(stream))

    def combine(self, stream=None):
        L.moe_combine(self.shape, _p(self.yp), _p(self.row_of), _p(self.y), stream_handle(stream))

    def forward(self, logits, x, w_gate, w_up, w_down, stream=None, bias=None, mask=None, count=False):
        s = self.shape
        self._check(x, (s.T, s.H), self.dtype, "x")
        self._check(w_gate, (s.e_local, s.H, s.I), self.dtype, "w_gate")
        self._check(w_up, (s.e_local, s.H, s.I), self.dtype, "w_up")
        self._check(w_down, (s.e_local, s.I, s.H), self.dtype, "w_down")
        self.inputs = (logits, x, w_gate, w_up, w_down)
        self.route(logits, stream, bias, mask, count)
        self.dispatch(x, stream)
        self.experts(x, w_gate, w_up, w_down, stream)
        self.combine(stream)
        return self.y

    def balance(self, coef, mask=None, stream=None):
        """The load-balance loss [1] of the last forward's routing, over all E experts and the
        tokens with mask != 0 (uint8 [T]); called between the forward and the backward.  The
        per-expert counts are then in ``balance_counts`` [E + 1]."""
        if self.inputs is None:
            raise RuntimeError("balance without a forward")
        if self._balance is None:
            self._balance = BalanceLoss(self.shape.T, self.shape.E, self.shape.k, device=self.device)
        loss = self._balance.forward(self.inputs[0], self.topk_idx, coef, mask=mask, stream=stream)
        self._balanced = True
        return loss

    @property
    def balance_counts(self):
        return None if self._balance is None else self._balance.counts

    def orthogonalize(self, steps=5, scale=1.0, stream=None):
        """Orthogonalised updates (bf16) of the last backward's dw_gate, dw_up and dw_down, in
        buffers that the next call overwrites."""
        if not self._has_grads:
            raise RuntimeError("orthogonalize without a backward")
        s, code = self.shape, self.shape.dtype

        # before the operators, whose calls on another stream wait for what was queued before them
        if not self._updates:
            self._updates = {n: torch.empty(g.shape, dtype=torch.bfloat16, device=self.device)
                             for n, g in (("gate", self.dw_gate), ("up", self.dw_up), ("down", self.dw_down))}

        def op(rows, cols):
            key = (rows, cols, steps)
            if key not in self._orth:   # they run in turn: one scratch, as far as it suffices
                need = L.moe_orth_scratch_bytes(L.MoeOrthShape(s.e_local, rows, cols, code, steps))
                have = [o.scratch for o in self._orth.values() if o.scratch.numel() >= need]
                self._orth[key] = Orthogonalizer(s.e_local, rows, cols, code, steps, self.device, *have[:1])
            return self._orth[key]

        for n, g in (("gate", self.dw_gate), ("up", self.dw_up), ("down", self.dw_down)):
            op(g.shape[1], g.shape[2]).update(g, scale, out=self._updates[n], stream=stream)
        return dict(self._updates)

    def backward(self, dy, stream=None, d_balance=None):
        """``d_balance`` [1]: the upstream gradient of ``balance``'s loss (None: 1), the same on
        every share."""
        s = self.shape
        self._check(dy, (s.T, s.H), self.dtype, "dy")
        if d_balance is not None:
            if not self._balanced:
                raise RuntimeError("d_balance without a balance loss in this pass")
            self._check(d_balance, (1,), torch.float32, "d_balance")
        logits, x, w_gate, w_up, w_down = self.inputs
        h = stream_handle(stream)
        L.moe_bwd(s, _p(dy), _p(x), _p(self.xp), _p(self.offsets), _p(self.row_src), _p(self.row_of),
                  _p(self.topk_w), _p(w_gate), _p(w_up), _p(w_down), _p(self.saved), _p(self.dx),
                  _p(self.dw_gate), _p(self.dw_up), _p(self.dw_down), _p(self.d_topk_w), _p(self.scratch), h)
        self._has_grads = True
        if self.gate is not None:
            self.gate.backward(self.d_topk_w, out=self.d_logits, stream=stream)
        else:
            L.moe_route_topk_bwd(s, _p(logits), _p(self.topk_idx), _p(self.topk_w), _p(self.d_topk_w),
                                 _p(self.d_logits), h)
        if self._balanced and s.e_begin == 0:
            self._balance.backward(d_balance, d_logits_in=self.d_logits, out=self.d_logits, stream=stream)
        return {"dx": self.dx, "dw_gate": self.dw_gate, "dw_up": self.dw_up, "dw_down": self.dw_down,
                "d_topk_w": self.d_topk_w, "d_logits": self.d_logits}
