"""Device buffers of one MoE layer pass, allocated with PyTorch, and the call order of
the C ABI.  Every step runs in libmoe; torch only provides memory and the stream."""
from __future__ import annotations

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
    """

    def __init__(self, T, H, I, E, k, e_begin=0, e_local=None, dtype=L.MOE_BF16, bwd=L.MOE_BWD_SAME,
                 renorm=1, device="cuda", fuse_gather=True, fwd=L.MOE_FWD_SAME, recompute=0, row_tile=0):
        e_local = E if e_local is None else e_local
        self.shape = L.MoeShape(T, H, I, E, k, e_begin, e_local, dtype, bwd, renorm, fwd, recompute, row_tile)
        self.device = torch.device(device)
        if self.device.type == "cuda" and self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.dtype = _DT[dtype]
        saved_b, scratch_b = L.moe_workspace_bytes(self.shape)
        self.R_cap = T * min(k, e_local)
        dev, i32, f32 = self.device, torch.int32, torch.float32
        self.topk_idx = torch.empty(T, k, dtype=i32, device=dev)
        self.topk_w = torch.empty(T, k, dtype=f32, device=dev)
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

    def route(self, logits, stream=None):
        s = self.shape
        self._check(logits, (s.T, s.E), torch.float32, "logits")
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

    def forward(self, logits, x, w_gate, w_up, w_down, stream=None):
        s = self.shape
        self._check(x, (s.T, s.H), self.dtype, "x")
        self._check(w_gate, (s.e_local, s.H, s.I), self.dtype, "w_gate")
        self._check(w_up, (s.e_local, s.H, s.I), self.dtype, "w_up")
        self._check(w_down, (s.e_local, s.I, s.H), self.dtype, "w_down")
        self.inputs = (logits, x, w_gate, w_up, w_down)
        self.route(logits, stream)
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
        L.moe_route_topk_bwd(s, _p(logits), _p(self.topk_idx), _p(self.topk_w), _p(self.d_topk_w),
                             _p(self.d_logits), h)
        if self._balanced and s.e_begin == 0:
            self._balance.backward(d_balance, d_logits_in=self.d_logits, out=self.d_logits, stream=stream)
        return {"dx": self.dx, "dw_gate": self.dw_gate, "dw_up": self.dw_up, "dw_down": self.dw_down,
                "d_topk_w": self.d_topk_w, "d_logits": self.d_logits}
