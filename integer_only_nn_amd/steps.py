"""Training steps as sequences of libionn calls on one stream.

Nothing here computes: each function allocates device buffers (PyTorch is
the allocator) and enqueues the library's kernels in the order the method
gives.  Shift values stay on the device; they are read back only when a
caller asks for them.

Order of a step ("Integer On-Device Training: Overview", sections 3, 4, 6.2):
forward (activations requantised with a dynamic NITI shift), the user loss
writes the output delta, then the backward pass per layer from the last:
delta propagation with the pre-update weights (ReLU mask, requantised to
target_bits = 7) and the weight gradient followed by the NITI update.
"""
from dataclasses import dataclass, field
from typing import List, Optional

import numpy as np
import torch

from . import ops

TB_WEIGHT = 8
MU_WEIGHT = 2
TB_DELTA = 7


def _i32(*shape, device):
    return torch.empty(shape, dtype=torch.int32, device=device)


def _i8(*shape, device):
    return torch.empty(shape, dtype=torch.int8, device=device)


# ---------------------------------------------------------------------------
# Single linear layer.
# ---------------------------------------------------------------------------

@dataclass
class LinearStepBuffers:
    """Device buffers of one linear-layer step (allocated once, reused).

    scal, int32[16]: [0:3] the max |Y|, |dX|, |G| of the last step, [3] the
    delta's shift, [4:6] the update's s, ws; [8:11] and [12:15] the two sets
    the maxima are max-combined into when steps alternate (alternate=True):
    each step's update clears the set the next step uses, so no fill kernel
    runs per step; the maxima of the step just taken are then in set
    `maxima()`."""
    Y: torch.Tensor
    dX: torch.Tensor
    G: torch.Tensor
    delta: torch.Tensor
    scal: torch.Tensor
    gq: Optional[torch.Tensor] = None
    alternate: bool = False
    phase: int = 0

    @staticmethod
    def make(B, IN, OUT, device, with_gq=False, alternate=False):
        return LinearStepBuffers(_i32(B, OUT, device=device), _i32(B, IN, device=device),
                                 _i32(OUT, IN, device=device), _i8(B, IN, device=device),
                                 torch.zeros(16, dtype=torch.int32, device=device),
                                 _i32(OUT, IN, device=device) if with_gq else None, alternate)

    def maxima(self):
        """The max |Y|, |dX|, |G| scalars of the last step (device view)."""
        if not self.alternate:
            return self.scal[0:3]
        o = 8 if self.phase == 1 else 12
        return self.scal[o:o + 3]


def linear_step(X, W, dY, buf: LinearStepBuffers, requant_delta=True, tb_w=TB_WEIGHT,
                mu=MU_WEIGHT, tb_d=TB_DELTA, stream=None):
    """fwd (int32 Y + max) -> dgrad (int32 dX + max) [-> delta, 7 bits] ->
    wgrad (int32 G + max) -> NITI update of W in place.  With
    buf.alternate the maxima go to one of two scalar sets and the update
    clears the other, instead of a fill before the step (a captured HIP
    graph must then hold an even number of steps)."""
    s = buf.scal
    if buf.alternate:
        m = s[8:11] if buf.phase == 0 else s[12:15]
        nxt = s[12:15] if buf.phase == 0 else s[8:11]
        buf.phase ^= 1
    else:
        m, nxt = s[0:3], None
        ops.ionn_fill_u32(m, 0, stream=stream)
    ops.int_linear_fwd(X, W, buf.Y, absmax_Y=m[0:1], stream=stream)
    ops.int_linear_dgrad(dY, W, buf.dX, absmax_dX=m[1:2], stream=stream)
    if requant_delta:
        ops.niti_quantize(buf.dX, m[1:2], tb_d, False, buf.delta, shift_out=s[3:4], stream=stream)
    ops.int_linear_wgrad(dY, X, buf.G, absmax_G=m[2:3], stream=stream)
    if nxt is None:
        ops.niti_quantize_update(buf.G, m[2:3], tb_w, mu, W, shifts_out=s[4:6], gq_out=buf.gq,
                                 stream=stream)
    else:
        ops.niti_quantize_update_clear(buf.G, m[2:3], tb_w, mu, W, nxt, shifts_out=s[4:6], gq_out=buf.gq,
                                       stream=stream)


def linear_step_small(X, W, dY, buf: LinearStepBuffers, tb_w=TB_WEIGHT, mu=MU_WEIGHT, tb_d=TB_DELTA,
                      stream=None):
    """The same step as linear_step (with the delta requantised) in one
    launch, for layers that int_linear_step_small_fits takes: the maxima go
    to buf.scal[0:3] (written, not combined) and the shifts s_d, s, ws to
    buf.scal[3:6]."""
    s = buf.scal
    ops.int_linear_step_small(X, W, dY, tb_w, mu, tb_d, buf.Y, buf.dX, buf.delta, buf.G, s[0:3], s[3:6],
                              gq=buf.gq, stream=stream)


# ---------------------------------------------------------------------------
# Multi-layer perceptron (all layers trainable).
# ---------------------------------------------------------------------------

@dataclass
class MLP:
    Ws: List[torch.Tensor]
    relu: List[bool]
    B: int
    acts: List[torch.Tensor] = field(default_factory=list)
    z32: List[torch.Tensor] = field(default_factory=list)
    d32: List[torch.Tensor] = field(default_factory=list)
    deltas: List[torch.Tensor] = field(default_factory=list)
    G: List[torch.Tensor] = field(default_factory=list)
    Gq: Optional[List[torch.Tensor]] = None   # with_gq: each layer's Gq of the last step
    e32: Optional[torch.Tensor] = None
    # per step: [fwd max x L | err max | dgrad max x L | G max x L] (uint32)
    # and shifts [fwd s x L | err s | dgrad s x L | (s, ws) x L]
    maxes: Optional[torch.Tensor] = None
    shifts: Optional[torch.Tensor] = None

    @staticmethod
    def make(Ws, B, relu=None, with_gq=False):
        L = len(Ws)
        dev = Ws[0].device
        m = MLP(list(Ws), relu if relu is not None else [l < L - 1 for l in range(L)], B)
        if with_gq:
            m.Gq = [_i32(*w.shape, device=dev) for w in Ws]
        sizes = [Ws[0].shape[1]] + [w.shape[0] for w in Ws]
        m.acts = [None] + [_i8(B, sizes[l + 1], device=dev) for l in range(L)]
        m.z32 = [_i32(B, sizes[l + 1], device=dev) for l in range(L)]
        m.d32 = [_i32(B, sizes[l], device=dev) for l in range(L)]
        m.deltas = [_i8(B, sizes[l], device=dev) for l in range(L + 1)]
        m.G = [_i32(*w.shape, device=dev) for w in Ws]
        m.e32 = _i32(B, sizes[-1], device=dev)
        m.maxes = torch.zeros(3 * L + 1, dtype=torch.int32, device=dev)
        m.shifts = torch.zeros(4 * L + 1, dtype=torch.int32, device=dev)
        return m

    def step(self, X, labels, target_mag=127, tb_w=TB_WEIGHT, mu=MU_WEIGHT, tb_a=TB_DELTA,
             tb_d=TB_DELTA, stream=None):
        L = len(self.Ws)
        mx, sh = self.maxes, self.shifts
        ops.ionn_fill_u32(mx, 0, stream=stream)
        self.acts[0] = X
        for l in range(L):
            ops.int_linear_fwd(self.acts[l], self.Ws[l], self.z32[l], absmax_Y=mx[l:l + 1],
                               stream=stream)
            ops.niti_quantize(self.z32[l], mx[l:l + 1], tb_a, self.relu[l], self.acts[l + 1],
                              shift_out=sh[l:l + 1], stream=stream)
        ops.int_output_error(self.acts[L], labels, target_mag, self.e32, absmax_e=mx[L:L + 1],
                             stream=stream)
        ops.niti_quantize(self.e32, mx[L:L + 1], tb_d, False, self.deltas[L],
                          shift_out=sh[L:L + 1], stream=stream)
        for l in range(L - 1, -1, -1):
            mask = self.acts[l] if (l >= 1 and self.relu[l - 1]) else None
            dm = mx[L + 1 + l:L + 2 + l]
            ops.int_linear_dgrad(self.deltas[l + 1], self.Ws[l], self.d32[l], relu_act=mask,
                                 absmax_dX=dm, stream=stream)
            ops.niti_quantize(self.d32[l], dm, tb_d, False, self.deltas[l],
                              shift_out=sh[L + 1 + l:L + 2 + l], stream=stream)
            gm = mx[2 * L + 1 + l:2 * L + 2 + l]
            ops.int_linear_wgrad(self.deltas[l + 1], self.acts[l], self.G[l], absmax_G=gm,
                                 stream=stream)
            ops.niti_quantize_update(self.G[l], gm, tb_w, mu, self.Ws[l],
                                     shifts_out=sh[2 * L + 1 + 2 * l:2 * L + 3 + 2 * l],
                                     gq_out=self.Gq[l] if self.Gq is not None else None,
                                     stream=stream)

    def shift_record(self):
        """Host copy of the last step's shifts in the oracle's record layout."""
        L = len(self.Ws)
        s = self.shifts.cpu().tolist()
        return dict(s_fwd=s[:L], s_err=s[L], s_dgrad=s[L + 1:2 * L + 1],
                    s_upd=[(s[2 * L + 1 + 2 * l], s[2 * L + 2 + 2 * l]) for l in range(L)])


# ---------------------------------------------------------------------------
# 3x3 conv layer.
# ---------------------------------------------------------------------------

@dataclass
class ConvStepBuffers:
    """Device buffers of one 3x3 conv step.

    scal, int32[16]: [0:3] the max |Y|, |dX|, |G|, [3] s_y, [4] s_dx,
    [5:7] the update's s, ws; [8:11] and [12:15] the two sets the maxima are
    max-combined into when steps alternate (alternate=True): each step's
    update clears the set the next step uses, so no fill kernel runs per
    step; the maxima of the step just taken are then in set `maxima()`."""
    Y: torch.Tensor
    y8: torch.Tensor
    dX: torch.Tensor
    dx8: torch.Tensor
    G: torch.Tensor
    scal: torch.Tensor
    gq: Optional[torch.Tensor] = None
    ws: Optional[torch.Tensor] = None   # weight-gradient workspace (None: no fast path)
    rws: Optional[torch.Tensor] = None  # one-pass requantisation workspace (None: two passes)
    alternate: bool = False
    phase: int = 0

    @staticmethod
    def make(N, H, W, Cin, Cout, device, with_gq=False, one_pass=True, alternate=False):
        d = ops.conv_desc(N, H, W, Cin, Cout)
        wsb = ops.int_conv_wgrad_workspace_bytes(d)
        rwb = ops.int_conv_requant_workspace_bytes(d) if one_pass else 0
        return ConvStepBuffers(_i32(N, H, W, Cout, device=device), _i8(N, H, W, Cout, device=device),
                               _i32(N, H, W, Cin, device=device), _i8(N, H, W, Cin, device=device),
                               _i32(Cout, 3, 3, Cin, device=device),
                               torch.zeros(16, dtype=torch.int32, device=device),
                               _i32(Cout, 3, 3, Cin, device=device) if with_gq else None,
                               torch.empty(wsb, dtype=torch.uint8, device=device) if wsb else None,
                               torch.empty(rwb, dtype=torch.uint8, device=device) if rwb else None,
                               alternate)

    def maxima(self):
        """The max |Y|, |dX|, |G| scalars of the last step (device view)."""
        if not self.alternate:
            return self.scal[0:3]
        o = 8 if self.phase == 1 else 12
        return self.scal[o:o + 3]

    def _sets(self, stream):
        """The maxima of this step and the set the update clears (None: a
        fill kernel cleared this step's set)."""
        s = self.scal
        if not self.alternate:
            ops.ionn_fill_u32(s[0:3], 0, stream=stream)
            return s[0:3], None
        m = s[8:11] if self.phase == 0 else s[12:15]
        nxt = s[12:15] if self.phase == 0 else s[8:11]
        self.phase ^= 1
        return m, nxt


def _conv_update(buf, m, nxt, tb_w, mu, Wt, stream):
    s = buf.scal
    if nxt is None:
        ops.niti_quantize_update(buf.G, m[2:3], tb_w, mu, Wt, shifts_out=s[5:7], gq_out=buf.gq, stream=stream)
    else:
        ops.niti_quantize_update_clear(buf.G, m[2:3], tb_w, mu, Wt, nxt, shifts_out=s[5:7], gq_out=buf.gq,
                                       stream=stream)


def conv_step(X, Wt, dY, buf: ConvStepBuffers, tb_a=TB_DELTA, tb_d=TB_DELTA, tb_w=TB_WEIGHT,
              mu=MU_WEIGHT, stream=None):
    N, H, W_, Cin = X.shape
    Cout = Wt.shape[0]
    d = ops.conv_desc(N, H, W_, Cin, Cout)
    s = buf.scal
    m, nxt = buf._sets(stream)
    ops.int_conv_fwd(X, Wt, buf.Y, d, absmax_Y=m[0:1], stream=stream)
    ops.niti_quantize(buf.Y, m[0:1], tb_a, False, buf.y8, shift_out=s[3:4], stream=stream)
    ops.int_conv_dgrad(dY, Wt, buf.dX, d, absmax_dX=m[1:2], stream=stream)
    ops.niti_quantize(buf.dX, m[1:2], tb_d, False, buf.dx8, shift_out=s[4:5], stream=stream)
    ops.int_conv_wgrad(dY, X, buf.G, d, absmax_G=m[2:3], workspace=buf.ws, stream=stream)
    _conv_update(buf, m, nxt, tb_w, mu, Wt, stream)


def conv_step_fused(X, Wt, dY, buf: ConvStepBuffers, tb_a=TB_DELTA, tb_d=TB_DELTA, tb_w=TB_WEIGHT,
                    mu=MU_WEIGHT, stream=None):
    """The same step with the requantisation fused into the contractions
    (64 -> 64 channels): y8, dx8, G, the update and every shift as in
    conv_step; buf.Y and buf.dX are not written (the int32 sums are never
    stored).  With buf.rws each requantising contraction is one pass plus a
    streaming pass over its int8 output, else two contraction passes.  With
    buf.alternate no fill kernel runs (a captured HIP graph must then hold
    an even number of steps)."""
    N, H, W_, Cin = X.shape
    Cout = Wt.shape[0]
    d = ops.conv_desc(N, H, W_, Cin, Cout)
    s = buf.scal
    m, nxt = buf._sets(stream)
    ops.int_conv_fwd_requant(X, Wt, buf.y8, d, tb_a, False, m[0:1], shift_out=s[3:4], workspace=buf.rws,
                             stream=stream)
    ops.int_conv_dgrad_requant(dY, Wt, buf.dx8, d, tb_d, m[1:2], shift_out=s[4:5], workspace=buf.rws,
                               stream=stream)
    ops.int_conv_wgrad(dY, X, buf.G, d, absmax_G=m[2:3], workspace=buf.ws, stream=stream)
    _conv_update(buf, m, nxt, tb_w, mu, Wt, stream)


# ---------------------------------------------------------------------------
# DFP-16 layer.
# ---------------------------------------------------------------------------

@dataclass
class DfpStepBuffers:
    Y: torch.Tensor
    dX: torch.Tensor
    G: torch.Tensor
    ws: torch.Tensor          # one workspace, reused by the three contractions
    exps: torch.Tensor        # int32[8]: eY, edX, eG, status x3
    gavg: torch.Tensor        # float64[1]

    @staticmethod
    def make(M, K, N, device):
        wsb = max(ops.dfp16_workspace_bytes(M, K, N, w) for w in range(3))
        return DfpStepBuffers(torch.empty(M, N, dtype=torch.int16, device=device),
                              torch.empty(M, K, dtype=torch.int16, device=device),
                              torch.empty(N, K, dtype=torch.int16, device=device),
                              torch.empty(wsb, dtype=torch.uint8, device=device),
                              torch.zeros(8, dtype=torch.int32, device=device),
                              torch.zeros(1, dtype=torch.float64, device=device))


def dfp16_step(X, eX, W, eW, dY, edY, buf: DfpStepBuffers, stream=None):
    """eX, eW, edY: device int32[1] exponents."""
    e = buf.exps
    ops.dfp16_gemm_fwd(X, eX, W, eW, buf.Y, e[0:1], buf.ws, status_out=e[3:4], stream=stream)
    ops.dfp16_gemm_dgrad(dY, edY, W, eW, buf.dX, e[1:2], buf.ws, status_out=e[4:5], stream=stream)
    ops.dfp16_gemm_wgrad(dY, edY, X, eX, buf.G, e[2:3], buf.ws, status_out=e[5:6], stream=stream)
    ops.dfp16_gavg(buf.G, e[2:3], eW, buf.gavg, stream=stream)


# ---------------------------------------------------------------------------
# Model-level driver (ionn_model_forward / ionn_model_backward).
# ---------------------------------------------------------------------------

class Model:
    """Device copy of a layer list and the driver's workspace.  Layers are
    dicts: kind "conv" or "linear", relu, geometry (conv: H, W, Cin, Cout, KH,
    KW, pad; linear: IN, OUT) and host arrays weight, offset, mult, k."""

    def __init__(self, layers, B, device):
        self.B = B
        self.dev = []
        for L in layers:
            conv = L["kind"] == "conv"
            t = (0 if conv else 2) + (1 if L["relu"] else 0)
            geo = dict(H=L["H"], W=L["W"], Cin=L["Cin"], Cout=L["Cout"], KH=L["KH"], KW=L["KW"], pad=L["pad"]) \
                if conv else dict(H=1, W=1, Cin=L["IN"], Cout=L["OUT"])
            self.dev.append(dict(type=t, **geo,
                                 weight=torch.from_numpy(L["weight"].copy()).to(device),
                                 offset=torch.from_numpy(L["offset"].copy()).to(device),
                                 mult=torch.from_numpy(L["mult"].copy()).to(device),
                                 k=torch.from_numpy(L["k"].copy()).to(device)))
        self.larr = ops.layer_array(self.dev)
        n = ops.ionn_model_workspace_bytes(self.larr, B)
        self.ws = torch.empty(n, dtype=torch.uint8, device=device)
        self.shifts = torch.zeros(1 + 5 * len(layers), dtype=torch.int32, device=device)
        last = self.dev[-1]
        n_out = last["Cout"]
        if last["type"] < 2:
            n_out *= (last["H"] + 2 * last["pad"] - last["KH"] + 1) * (last["W"] + 2 * last["pad"] - last["KW"] + 1)
        self.out = torch.empty(B, n_out, dtype=torch.int8, device=device)

    def forward(self, X, stream=None):
        ops.ionn_model_forward(self.larr, X, self.ws, out=self.out, stream=stream)

    def backward(self, X, labels, tmc, tmw, stream=None):
        ops.ionn_model_backward(self.larr, X, labels, tmc, tmw, self.ws, shifts_out=self.shifts, stream=stream)

    def step(self, X, labels, tmc, tmw, stream=None):
        self.forward(X, stream=stream)
        self.backward(X, labels, tmc, tmw, stream=stream)


# ---------------------------------------------------------------------------
# Adaptive per-layer precision (apt_update / apt_adjust).
# ---------------------------------------------------------------------------

class AptLayers:
    """Device state of adaptive per-layer precision over L int16 weight
    tensors: their precisions k, weight exponents e_w and the epoch's Gavg
    sums and counts, plus the workspace a sampling step needs.  The host
    never reads the state back unless asked to.  The ctypes argument arrays
    are built once (bind_grads for the gradient buffers), so a step costs
    one library call."""

    def __init__(self, Ws, ks, es, device, int8_layers=()):
        """int8_layers: indices of layers held in int8 (their k must be at
        most 8 and stays there: half the memory of int16)."""
        self.W = []
        for l, w in enumerate(Ws):
            if l in int8_layers:
                if int(ks[l]) > 8 or w.min(initial=0) < -128 or w.max(initial=0) > 127:
                    raise ValueError(f"layer {l}: int8 storage needs k <= 8 and mantissas in [-128, 127]")
                w = w.astype(np.int8)
            self.W.append(torch.from_numpy(np.ascontiguousarray(w).copy()).to(device))
        L = len(self.W)
        self._mixed = bool(int8_layers)
        self.k = torch.tensor(list(ks), dtype=torch.int32, device=device)
        self.e_w = torch.tensor(list(es), dtype=torch.int32, device=device)
        self.gsum = torch.zeros(L, dtype=torch.float64, device=device)
        self.gcnt = torch.zeros(L, dtype=torch.int32, device=device)
        self.dk = torch.zeros(L, dtype=torch.int32, device=device)
        self.ws = torch.empty(max(ops.apt_workspace_bytes([w.numel() for w in self.W]), 8),
                              dtype=torch.uint8, device=device)
        self._Wp = ops._ptr_array(self.W, None, "W")
        self._wb = ops._wbytes(self.W)
        self._n = ops._sizes(self.W)
        self._G = None

    def bind_grads(self, Gs):
        """Fix the gradient buffers (int16 device tensors, one per layer) that
        step() reads when it is given none."""
        if len(Gs) != len(self.W) or any(g.numel() != w.numel() for g, w in zip(Gs, self.W)):
            raise ValueError("one gradient per layer, of the layer's size")
        self._G = (list(Gs), ops._ptr_array(Gs, torch.int16, "G"))

    def step(self, Gs, e_g, lr_shift, sample=False, stream=None):
        """One update of every layer with gradients Gs (int16 device tensors;
        None: the bound buffers) and their exponents e_g (int32 device [L])."""
        if Gs is not None:
            self.bind_grads(Gs)
        if self._G is None:
            raise ValueError("no gradient buffers")
        L = len(self.W)
        args = (self._G[1], self._n, ops._p(self.k), ops._p(self.e_w), ops._p(e_g, torch.int32, L, "e_g"),
                int(lr_shift), ops._p(self.gsum) if sample else None, ops._p(self.gcnt) if sample else None,
                ops._p(self.ws) if sample else None, self.ws.numel() if sample else 0, ops._stream(stream))
        if self._mixed:
            ops.check(ops.lib().apt_update_mixed(L, self._Wp, self._wb, *args), "apt_update_mixed")
        else:
            ops.check(ops.lib().apt_update(L, self._Wp, *args), "apt_update")

    def end_epoch(self, t_min, t_max, k_min=2, k_max=16, stream=None):
        L = len(self.W)
        args = (self._n, ops._p(self.k), ops._p(self.e_w), ops._p(self.gsum), ops._p(self.gcnt), float(t_min),
                float(t_max), int(k_min), int(k_max), ops._p(self.dk), ops._stream(stream))
        if self._mixed:
            ops.check(ops.lib().apt_adjust_mixed(L, self._Wp, self._wb, *args), "apt_adjust_mixed")
        else:
            ops.check(ops.lib().apt_adjust(L, self._Wp, *args), "apt_adjust")


# ---------------------------------------------------------------------------
# AdamW over a model's tensors (ionn_adamw_step).
# ---------------------------------------------------------------------------

class AdamW:
    """The optimiser of a list of float32 master weights, updated in place.
    Ms and Vs: the moments, float32 tensors; or, with Ss (int8 [blocks][2] per
    tensor), codes of one byte of m and of sqrt(v).  Rs (int8, as the weights)
    carries what a code leaves of sqrt(v), so that the second moment follows
    its definition within about 2%; None: allocated as zeros, the codes' own values
    (keep them with the other states).  Rs=False: codes alone, whose v is right
    on average and scatters by about 30% per weight.  The ctypes arrays are
    built once (bind_grads for the gradient buffers), so a step costs one
    library call.

    t counts the steps taken.  With on_device the count and the learning rate
    live in device scalars (self.step_dev, advanced by each step, and
    self.lr_dev), so that steps can be captured in a graph and replayed."""

    def __init__(self, Ps, Ms, Vs, Ss=None, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, t=0,
                 on_device=False, Rs=None):
        self.P, self.M, self.V, self.S = list(Ps), list(Ms), list(Vs), None if Ss is None else list(Ss)
        self.lr, self.betas, self.eps, self.weight_decay, self.t = lr, betas, eps, weight_decay, int(t)
        bits = 32 if Ss is None else 8
        for xs in (self.M, self.V):
            ops._same(len(xs) == len(self.P) and all(x.numel() == p.numel() for x, p in zip(xs, self.P)),
                      "weights and states")
        self.R = None
        ops._same(not Rs or Ss is not None, "remainders without codes")
        if Ss is not None and Rs is not False:
            zeros = lambda p: torch.zeros(p.shape, dtype=torch.int8, device=p.device)  # noqa: E731
            self.R = [zeros(p) for p in self.P] if Rs is None else list(Rs)
            ops._same(len(self.R) == len(self.P) and all(r.numel() == p.numel() for r, p in zip(self.R, self.P)),
                      "weights and remainders")
        if Ss is not None:
            ops._same(len(self.S) == len(self.P) and
                      all(s.numel() == 2 * -(-p.numel() // ops.ADAMW_BLOCK) for s, p in zip(self.S, self.P)),
                      "weights and state exponents")
        self._Pp = ops._ptr_array(self.P, torch.float32, "P")
        self._states = [ops._state_ptrs(self.M, bits, "M"), ops._state_ptrs(self.V, bits, "V")]
        self._states += [None if Ss is None else ops._ptr_array(self.S, torch.int8, "S"),
                         bits if self.R is None else ops._ptr_array(self.R, torch.int8, "R")]
        self._n = ops._sizes(self.P)
        self._G = None
        self.step_dev = self.lr_dev = None
        if on_device:
            dev = self.P[0].device
            self.step_dev = torch.tensor([self.t], dtype=torch.int32, device=dev)
            self.lr_dev = torch.tensor([lr], dtype=torch.float32, device=dev)

    @staticmethod
    def make(Ps, bits=32, **kw):
        """Cleared states of 32 or 8 bits for these weights: 8 or 2 bytes per
        weight, 3 with remainders (bits=8, Rs=None)."""
        if bits == 32:
            return AdamW(Ps, [torch.zeros_like(p) for p in Ps], [torch.zeros_like(p) for p in Ps], **kw)
        if bits != 8:
            raise ValueError(f"bits = {bits} (8 or 32)")
        codes = lambda: [torch.zeros(p.shape, dtype=torch.uint8, device=p.device) for p in Ps]  # noqa: E731
        blocks = [torch.zeros(-(-p.numel() // ops.ADAMW_BLOCK), 2, dtype=torch.int8, device=p.device) for p in Ps]
        return AdamW(Ps, codes(), codes(), blocks, **{"Rs": False, **kw})

    def bind_grads(self, Gs):
        """Fix the gradient buffers (device tensors of one floating type, one
        per weight) that step() reads when it is given none."""
        if len(Gs) != len(self.P) or any(g.numel() != p.numel() for g, p in zip(Gs, self.P)):
            raise ValueError("one gradient per weight tensor, of its size")
        if self.P:
            self._G = (list(Gs), ops._ptr_array(Gs, Gs[0].dtype, "G"), ops._dtype(Gs[0], "G"))

    def step(self, Gs=None, grad_scale=None, absmax_P=None, stream=None):
        """One step with gradients Gs (None: the bound buffers)."""
        if not self.P:
            return
        if Gs is not None:
            self.bind_grads(Gs)
        if self._G is None:
            raise ValueError("no gradient buffers")
        name = "ionn_adamw_step" if self.R is None else "ionn_adamw_step_carried"
        call = getattr(ops.lib(), name)
        args = (len(self.P), self._Pp, self._G[1], self._G[2], *self._states, self._n, self.t + 1,
                self.lr, self.betas[0], self.betas[1], self.eps, self.weight_decay,
                ops._s(self.step_dev, torch.int32, "step"), ops._s(self.lr_dev, torch.float32, "lr_dev"),
                ops._s(grad_scale, torch.float32, "grad_scale"), ops._v(absmax_P, torch.int32, len(self.P), "absmax_P"),
                ops._on(stream, self.P[0]))
        self._count(1, stream)
        rc = call(*args)
        if rc:  # (not a step: neither count keeps it)
            self._count(-1, stream)
            ops.check(rc, name)
        self.t += 1

    def _count(self, by, stream):
        """Moves the count on the device, if there is one."""
        if self.step_dev is None:
            return
        if stream is None:
            self.step_dev.add_(by)
            return
        on = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))
        with torch.cuda.stream(on):
            self.step_dev.add_(by)


# ---------------------------------------------------------------------------
# The residual MLP block of a transformer on DFP-8 products.
# ---------------------------------------------------------------------------

class ResidualMlp:
    """y = x + W2 act(W1 norm(x) + b1) + b2 over a batch of B rows, trained as
    "Mixed Precision Training of Convolutional Neural Networks using Integer
    Operations" (section 4) lays out: integer products on DFP-8 copies of
    activations, weights and errors, everything around them in floating
    point, FP32 master weights.

    Activations and their gradients are of type dtype.  Weights decay, gains
    and biases do not; both groups keep their moments in state_bits bits (8:
    with remainders of the second moment, three bytes per weight).  All
    buffers are allocated here, so a step only enqueues kernels (and can be
    captured in a graph with on_device)."""

    def __init__(self, W1, b1, W2, b2, gamma, beta, B, dtype=torch.bfloat16, act="gelu", eps=1e-5, state_bits=8,
                 lr=1e-3, betas=(0.9, 0.999), weight_decay=0.01, on_device=False):
        """W1: [H][D], b1: [H], W2: [D][H], b2, gamma, beta: [D], float32 device tensors, updated in place."""
        H, D = W1.shape
        ops._same(W2.shape == (D, H) and b1.numel() == H and all(t.numel() == D for t in (b2, gamma, beta)),
                  "the block's weights")
        dev = W1.device
        new = lambda *shape, dt=dtype: torch.empty(shape, dtype=dt, device=dev)  # noqa: E731
        f32, i8, i32 = torch.float32, torch.int8, torch.int32
        self.B, self.act, self.eps = B, act, eps
        self.W1, self.b1, self.W2, self.b2, self.gamma, self.beta = W1, b1, W2, b2, gamma, beta
        self.W1_8, self.W2_8 = new(H, D, dt=i8), new(D, H, dt=i8)
        # exponents: norm output, hidden activation, W1, W2, the two errors
        self.e = torch.zeros(6, dtype=i32, device=dev)
        # largest magnitudes: norm output, hidden activation, W1, W2 (float32 bits)
        self.top = torch.zeros(4, dtype=i32, device=dev)
        # as dfp8_from_float leaves it: of the last backward's errors, and of
        # the last norm output, hidden activation, W1 and W2
        self.status = torch.zeros(2, dtype=i32, device=dev)
        self.operand_status = torch.zeros(4, dtype=i32, device=dev)
        self.h, self.h8, self.mean, self.rstd = new(B, D), new(B, D, dt=i8), new(B, dt=f32), new(B, dt=f32)
        self.z, self.a, self.a8, self.y = new(B, H), new(B, H), new(B, H, dt=i8), new(B, D)
        self.da, self.dh, self.dx = new(B, H), new(B, D), new(B, D)
        self.d2_8, self.d1_8 = new(B, D, dt=i8), new(B, H, dt=i8)
        self.gW1, self.gW2 = new(H, D), new(D, H)
        self.gb1, self.gb2, self.ggamma, self.gbeta = new(H, dt=f32), new(D, dt=f32), new(D, dt=f32), new(D, dt=f32)
        need = max(ops.dfp8_linear_fwd_workspace_bytes(B, D, H), ops.dfp8_linear_fwd_workspace_bytes(B, H, D),
                   ops.dfp8_linear_bwd_workspace_bytes(B, D, H), ops.dfp8_linear_bwd_workspace_bytes(B, H, D),
                   ops.ionn_layer_norm_bwd_workspace_bytes(B, D), ops.dfp8_from_float_workspace_bytes())
        self.ws = new(need, dt=torch.uint8)
        kw = dict(bits=state_bits, lr=lr, betas=betas, on_device=on_device, Rs=None)
        self.opt = AdamW.make([W1, W2], weight_decay=weight_decay, **kw)
        self.opt.bind_grads([self.gW1, self.gW2])
        self.opt_vectors = AdamW.make([b1, b2, gamma, beta], weight_decay=0.0, **kw)
        self.opt_vectors.bind_grads([self.gb1, self.gb2, self.ggamma, self.gbeta])
        st = self.operand_status
        ops.dfp8_from_float(W1, self.W1_8, self.e[2:3], workspace=self.ws, status_out=st[2:3])
        ops.dfp8_from_float(W2, self.W2_8, self.e[3:4], workspace=self.ws, status_out=st[3:4])

    def forward(self, x, stream=None):
        """y of a batch x [B][D]; keeps what backward() reads."""
        e, top, st, kw = self.e, self.top, self.operand_status, dict(stream=stream)
        ops.ionn_fill_u32(top[0:2], 0, **kw)
        ops.ionn_layer_norm_fwd(x, self.h, gamma=self.gamma, beta=self.beta, eps=self.eps, mean=self.mean,
                                rstd=self.rstd, absmax_y=top[0:1], **kw)
        ops.dfp8_from_float(self.h, self.h8, e[0:1], absmax=top[0:1], status_out=st[0:1], **kw)
        ops.dfp8_linear_fwd(self.h8, e[0:1], self.W1_8, e[2:3], self.a, bias=self.b1, act=self.act, Z=self.z,
                            absmax_Y=top[1:2], workspace=self.ws, **kw)
        ops.dfp8_from_float(self.a, self.a8, e[1:2], absmax=top[1:2], status_out=st[1:2], **kw)
        ops.dfp8_linear_fwd(self.a8, e[1:2], self.W2_8, e[3:4], self.y, bias=self.b2, residual=x, workspace=self.ws,
                            **kw)
        return self.y

    def backward(self, x, dy, stream=None):
        """dx, and every parameter's gradient, for the error dy of the last forward(x)."""
        e, kw = self.e, dict(workspace=self.ws, stream=stream)
        ops.dfp8_linear_bwd(dy, None, "none", self.a8, e[1:2], self.W2_8, e[3:4], self.d2_8, e[4:5], dX=self.da,
                            G=self.gW2, gb=self.gb2, status_out=self.status[0:1], **kw)
        ops.dfp8_linear_bwd(self.da, self.z, self.act, self.h8, e[0:1], self.W1_8, e[2:3], self.d1_8, e[5:6],
                            dX=self.dh, G=self.gW1, gb=self.gb1, status_out=self.status[1:2], **kw)
        ops.ionn_layer_norm_bwd(self.dh, x, self.mean, self.rstd, self.dx, gamma=self.gamma, dres=dy,
                                dgamma=self.ggamma, dbeta=self.gbeta, **kw)
        return self.dx

    def update(self, stream=None):
        """The optimiser step on the last backward's gradients, and the new DFP-8 weights."""
        ops.ionn_fill_u32(self.top[2:4], 0, stream=stream)
        self.opt.step(absmax_P=self.top[2:4], stream=stream)
        self.opt_vectors.step(stream=stream)
        st = self.operand_status
        ops.dfp8_from_float(self.W1, self.W1_8, self.e[2:3], absmax=self.top[2:3], status_out=st[2:3], stream=stream)
        ops.dfp8_from_float(self.W2, self.W2_8, self.e[3:4], absmax=self.top[3:4], status_out=st[3:4], stream=stream)
