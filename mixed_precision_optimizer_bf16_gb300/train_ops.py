"""Training operators from torch tensors: distillation loss, gated norms, expert balance, policy and
preference losses, activations kept in 8 bits, rotary positions.

Marshalling only (shapes, types, data_ptr()s, stream handles, status ->
exception); all arithmetic is in libbf16opt.so (the "training operators" of
include/bf16opt.h, where the formulas stand).  Outputs and workspaces are torch
allocations made on the stream that the kernels run on: the current one, or
`stream`.  Nothing synchronises, so a training step that uses these calls
can be captured in a CUDA graph.

  distill_forward / distill_backward / distill_loss_grad, distill_loss (autograd)
  norm_gate_forward / norm_gate_backward, norm_gate (autograd)
  balance_forward / balance_backward, balance (autograd)
  token_logp_forward / policy_forward / preference_forward, token_logp_backward (of all three),
  policy_loss_grad; token_logp, policy_loss, preference_loss (autograd)
  pack8 / unpack8; glu8_forward / glu8_backward, glu8 (autograd)
  rotary_forward / rotary_backward, rotary (autograd)

The autograd forms have first derivatives only: going through a gradient of theirs once more
is an error.
"""
import contextlib
import functools
import math
import struct

import torch

from . import bf16opt as C

_TYPE = {torch.bfloat16: C.BF16OPT_TYPE_BF16, torch.float32: C.BF16OPT_TYPE_F32}
_INDEX = {torch.int32: C.BF16OPT_INDEX_I32, torch.int64: C.BF16OPT_INDEX_I64}
_F32 = (torch.float32,)
_NORM = {None: C.BF16OPT_NORM_NONE, "none": C.BF16OPT_NORM_NONE, "rms": C.BF16OPT_NORM_RMS, "layer": C.BF16OPT_NORM_LAYER}
_ACT = {None: C.BF16OPT_GATE_IDENTITY, "none": C.BF16OPT_GATE_IDENTITY, "sigmoid": C.BF16OPT_GATE_SIGMOID}

# The descriptors of include/bf16opt.h as packed bytes, in the structs' own layout:
# a small call's cost is this file's, and packing takes a fraction of what a
# ctypes structure takes.  (The tests compare both.)
_DISTILL_T = struct.Struct("@QII4iPQPQPQPPPfff4x")
_NORM_GATE_T = struct.Struct("@QI6iIQPPPPPfff4x")
_BALANCE_T = struct.Struct("@QIIQiiPQPff")
_TOKENS_T = struct.Struct("@QIiifPQPP")
_POLICY_T = struct.Struct("@PPPfffI")
_PREFERENCE_T = struct.Struct("@QiiPPfffi")
_PACK_T = struct.Struct("@QIi")
_GLU_T = struct.Struct("@QIiii")
_ROTARY_T = struct.Struct("@QQIIIIiiiiPQqPfI12Q")

_empty, _empty_like = torch.empty, torch.empty_like
_Tensor = torch.Tensor


def _need(t, what, dtypes, shape, index, rows_apart=False):
    """A tensor that the library may reach through a raw pointer: on CUDA device
    `index`, of one of `dtypes`, of `shape`, contiguous -- or, with rows_apart,
    with contiguous rows that do not overlap."""
    if isinstance(t, _Tensor) and t.is_cuda and t.dtype in dtypes and t.shape == shape and t.get_device() == index and t.is_contiguous():
        return
    if not isinstance(t, _Tensor) or not t.is_cuda:
        raise ValueError(f"{what}: must be a CUDA tensor")
    if t.get_device() != index:
        raise ValueError(f"{what}: on {t.device}, expected cuda:{index}")
    if t.dtype not in dtypes:
        raise ValueError(f"{what}: dtype {t.dtype}, expected one of {[str(d) for d in dtypes]}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not rows_apart or (t.shape[1] > 1 and t.stride(1) != 1) or (t.shape[0] > 1 and t.stride(0) < t.shape[1]):
        raise ValueError(f"{what}: must be contiguous" + (" within rows that do not overlap" if rows_apart else ""))


def _matrix(t, what):
    """(rows, columns, device index) of a CUDA matrix."""
    if not isinstance(t, _Tensor) or not t.is_cuda or t.dim() != 2:
        raise ValueError(f"{what}: must be a CUDA tensor of two dimensions")
    rows, columns = t.shape
    return rows, columns, t.get_device()


def _writable(t, what):
    """An output of the caller's: autograd has to be able to do without its old values, and to see that they are gone."""
    if t.requires_grad and torch.is_grad_enabled() and (t.is_leaf or (t._is_view() and t._base.is_leaf)):
        raise ValueError(f"{what}: a leaf (or a view of one) that requires a gradient is not written in place")


def _written(*outs):
    """The caller's outputs of a call that has gone through: their versions move on, as under torch's own writes."""
    for t in outs:
        if t is not None:
            torch.autograd.graph.increment_version(t)


def _stride(t):
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _p(t):
    return t.data_ptr() if t is not None else 0


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _on_stream(call):
    """Gives a function `stream=None`: it runs on the device of its first tensor
    (by place or by name), on `stream` or on that device's current one.  Its inputs are marked as used
    on a stream that is not the current one, so that their memory outlives the
    kernels."""
    @functools.wraps(call)
    def run(*args, stream=None, **more):
        first = args[0] if args else None
        if not isinstance(first, _Tensor):
            first = next((t for t in (*args, *more.values()) if isinstance(t, _Tensor)), None)
        if first is None or not first.is_cuda or (stream is None and first.get_device() == _current_device()):
            return call(*args, **more)
        index = first.get_device()
        with contextlib.ExitStack() as stack:
            stack.enter_context(torch.cuda.device(index))
            if stream is not None and stream != torch.cuda.current_stream(index):
                for t in (*args, *more.values()):
                    if isinstance(t, _Tensor) and t.is_cuda:
                        t.record_stream(stream)
                stack.enter_context(torch.cuda.stream(stream))
            return call(*args, **more)
    return run


class _First(torch.autograd.Function):
    """A gradient as it is; to go through it once more is an error."""
    @staticmethod
    def forward(ctx, gradient):
        return gradient.detach()

    @staticmethod
    def backward(ctx, _):
        raise RuntimeError("train_ops: these operators have no second derivative")


def _first_only(backward):
    """For the backward of an autograd form: under create_graph its gradients, which come from raw
    pointers, would else pass for constants.  (once_differentiable sees only the incoming gradients, and lets
    those of a plain sum through.)"""
    @functools.wraps(backward)
    def run(ctx, *grads):
        with torch.no_grad():
            out = backward(ctx, *grads)
        if not torch.is_grad_enabled():
            return out
        return tuple(_First.apply(g.detach().requires_grad_()) if g is not None else None for g in out)
    return run


# ------------------------------------------------------------------ distillation

def _distill(logits, teacher_ids, teacher_logits, temperature, kl_weight, ce_weight, labels, row_weight, teacher_lse):
    """(descriptor, rows, device index)."""
    rows, vocab, index = _matrix(logits, "logits")
    k = _matrix(teacher_ids, "teacher_ids")[1]
    _need(logits, "logits", _TYPE, (rows, vocab), index, True)
    _need(teacher_ids, "teacher_ids", _INDEX, (rows, k), index, True)
    _need(teacher_logits, "teacher_logits", _TYPE, (rows, k), index, True)
    if labels is not None:
        _need(labels, "labels", _INDEX, (rows,), index)
    if row_weight is not None:
        _need(row_weight, "row_weight", _F32, (rows,), index)
    if teacher_lse is not None:
        _need(teacher_lse, "teacher_lse", _F32, (rows,), index)
    return _DISTILL_T.pack(
        rows, vocab, k, _TYPE[logits.dtype], _TYPE[teacher_logits.dtype], _INDEX[teacher_ids.dtype],
        _INDEX[labels.dtype] if labels is not None else 0, logits.data_ptr(), _stride(logits), teacher_ids.data_ptr(),
        _stride(teacher_ids), teacher_logits.data_ptr(), _stride(teacher_logits), _p(teacher_lse), _p(labels),
        _p(row_weight), temperature, kl_weight, ce_weight), rows, index


@_on_stream
def distill_forward(logits, teacher_ids, teacher_logits, *, temperature=1.0, kl_weight=1.0, ce_weight=0.0, labels=None,
                    row_weight=None, teacher_lse=None):
    """Per-row loss [rows] and log-sum-exps [rows, 2] (FP32) of student logits
    [rows, vocab] (bf16 or FP32) against a teacher's kept entries [rows, k]
    (ids int32 or int64, logits bf16 or FP32; an id outside the vocabulary is
    no entry) and, with ce_weight, labels [rows] (outside: no label)."""
    d, rows, index = _distill(logits, teacher_ids, teacher_logits, temperature, kl_weight, ce_weight, labels, row_weight, teacher_lse)
    loss = _empty(rows, dtype=torch.float32, device=logits.device)
    lse = _empty((rows, 2), dtype=torch.float32, device=logits.device)
    C.check(C.bf16opt_distill_forward(d, loss.data_ptr(), lse.data_ptr(), _raw_stream(index)))
    return loss, lse


def _dlogits(logits, out, index):
    if out is None:
        return _empty_like(logits, memory_format=torch.contiguous_format)
    _need(out, "out", (logits.dtype,), logits.shape, index, True)
    _writable(out, "out")
    return out


@_on_stream
def distill_backward(logits, teacher_ids, teacher_logits, lse, dloss=None, *, temperature=1.0, kl_weight=1.0, ce_weight=0.0,
                     labels=None, row_weight=None, teacher_lse=None, out=None):
    """Gradient of the logits from that of the rows' losses (dloss [rows]
    FP32; None: 1), with distill_forward's arguments and lse.  out may be
    logits itself."""
    d, rows, index = _distill(logits, teacher_ids, teacher_logits, temperature, kl_weight, ce_weight, labels, row_weight, teacher_lse)
    _need(lse, "lse", _F32, (rows, 2), index)
    if dloss is not None:
        _need(dloss, "dloss", _F32, (rows,), index)
    given, out = out, _dlogits(logits, out, index)
    C.check(C.bf16opt_distill_backward(d, lse.data_ptr(), _p(dloss), out.data_ptr(), _stride(out), _raw_stream(index)))
    _written(given)
    return out


@_on_stream
def distill_loss_grad(logits, teacher_ids, teacher_logits, dloss=None, *, temperature=1.0, kl_weight=1.0, ce_weight=0.0,
                      labels=None, row_weight=None, teacher_lse=None, out=None):
    """Per-row loss and the gradient of the logits in one pass over them (for a
    gradient dloss, or 1, of each row's loss).  out may be logits itself."""
    d, rows, index = _distill(logits, teacher_ids, teacher_logits, temperature, kl_weight, ce_weight, labels, row_weight, teacher_lse)
    if dloss is not None:
        _need(dloss, "dloss", _F32, (rows,), index)
    loss = _empty(rows, dtype=torch.float32, device=logits.device)
    given, out = out, _dlogits(logits, out, index)
    C.check(C.bf16opt_distill_loss_grad(d, _p(dloss), loss.data_ptr(), 0, out.data_ptr(), _stride(out), _raw_stream(index)))
    _written(given)
    return loss, out


class _Distill(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, teacher_ids, teacher_logits, how):
        loss, lse = distill_forward(logits, teacher_ids, teacher_logits, **how)
        ctx.save_for_backward(logits, teacher_ids, teacher_logits, lse, *[how[n] for n in _DISTILL_TENSORS])
        ctx.how = {n: v for n, v in how.items() if n not in _DISTILL_TENSORS}
        return loss

    @staticmethod
    @_first_only
    def backward(ctx, dloss):
        logits, ids, top, lse, *tensors = ctx.saved_tensors
        return (distill_backward(logits, ids, top, lse, dloss.float().contiguous(), **ctx.how,
                                 **dict(zip(_DISTILL_TENSORS, tensors))), None, None, None)


_DISTILL_TENSORS = ("labels", "row_weight", "teacher_lse")


def distill_loss(logits, teacher_ids, teacher_logits, *, temperature=1.0, kl_weight=1.0, ce_weight=0.0, labels=None,
                 row_weight=None, teacher_lse=None):
    """The rows' losses [rows] as distill_forward, differentiable in logits.
    The teacher is a constant: no gradient goes to teacher_logits or
    teacher_lse.  A row_weight that requires a gradient is refused (multiply the
    losses by it instead)."""
    if isinstance(row_weight, _Tensor) and row_weight.requires_grad and torch.is_grad_enabled():
        raise ValueError("row_weight: requires a gradient, which the loss does not give; multiply the losses by it, or detach it")
    return _Distill.apply(logits, teacher_ids, teacher_logits,
                          dict(temperature=temperature, kl_weight=kl_weight, ce_weight=ce_weight, labels=labels,
                               row_weight=row_weight, teacher_lse=teacher_lse))


# ------------------------------------------------------------------- gated norms

def _norm_gate(stream_t, what, y, pre, post, pre_weight, pre_bias, post_weight, post_bias, gate, gate_act, residual_scale,
               branch_scale, eps):
    """(descriptor, rows, device index)."""
    rows, hidden, index = _matrix(y, "y")
    _need(y, "y", _TYPE, (rows, hidden), index)
    _need(stream_t, what, _TYPE, (rows, hidden), index)
    if pre not in _NORM or post not in _NORM or gate_act not in _ACT:
        raise ValueError("pre, post: None, 'none', 'rms' or 'layer'; gate_act: None, 'none' or 'sigmoid'")
    wtypes = _TYPE
    for n, w in (("pre_weight", pre_weight), ("pre_bias", pre_bias), ("post_weight", post_weight), ("post_bias", post_bias)):
        if w is not None:
            _need(w, n, wtypes, (hidden,), index)
            wtypes = (w.dtype,)
    gate_rows = 0
    if gate is not None:
        gate_rows = _matrix(gate, "gate")[0]
        _need(gate, "gate", (y.dtype,), (gate_rows, hidden), index)
    return _NORM_GATE_T.pack(
        rows, hidden, _TYPE[y.dtype], _TYPE[stream_t.dtype], _TYPE[wtypes[0]] if wtypes is not _TYPE else 0, _NORM[pre],
        _NORM[post], _ACT[gate_act], 0, gate_rows, _p(gate), _p(pre_weight), _p(pre_bias), _p(post_weight), _p(post_bias),
        residual_scale, branch_scale, eps), rows, index


@_on_stream
def norm_gate_forward(x, y, *, pre="rms", post="rms", pre_weight=None, pre_bias=None, post_weight=None, post_bias=None,
                      gate=None, gate_act="none", residual_scale=1.0, branch_scale=1.0, eps=1e-5, out_r=None, out_h=None):
    """r = residual_scale x + branch_scale act(gate) N_post(y) and h = N_pre(r)
    for the residual stream x and the block's output y [rows, hidden].  gate
    [gate_rows, hidden]: rows / gate_rows consecutive rows share one.  Returns
    (r, h, stats): h None if pre is None; stats [rows, 4] FP32 for the backward
    call.  out_r may be x, out_h may be y."""
    d, rows, index = _norm_gate(x, "x", y, pre, post, pre_weight, pre_bias, post_weight, post_bias, gate, gate_act,
                                residual_scale, branch_scale, eps)
    if out_r is not None:
        _need(out_r, "out_r", (x.dtype,), x.shape, index)
        _writable(out_r, "out_r")
    if out_h is not None:
        _need(out_h, "out_h", (y.dtype,), y.shape, index)
        _writable(out_h, "out_h")
    r = out_r if out_r is not None else _empty_like(x)
    h = out_h if out_h is not None or not _NORM[pre] else _empty_like(y)
    stats = _empty((rows, 4), dtype=torch.float32, device=y.device)
    C.check(C.bf16opt_norm_gate_forward(d, x.data_ptr(), y.data_ptr(), r.data_ptr(), _p(h), stats.data_ptr(), _raw_stream(index)))
    _written(out_r, out_h)
    return r, h, stats


@functools.lru_cache(maxsize=4096)
def _norm_gate_workspace(rows, hidden, types, gate_rows, index):
    """Bytes, by what they depend on: the sizes, the element types and the device."""
    with torch.cuda.device(index):
        rc, nbytes = C.bf16opt_norm_gate_workspace(
            C.bf16opt_norm_gate_t(rows, hidden, *types, 0, 0, 0, 0, 0, gate_rows, 256 if gate_rows else None, None, None, None, None,
                                  1.0, 1.0, 1.0))
        C.check(rc)
    return nbytes


def norm_gate_backward(dr, dh, r, y, stats, *, pre="rms", post="rms", pre_weight=None, pre_bias=None, post_weight=None,
                       post_bias=None, gate=None, gate_act="none", residual_scale=1.0, branch_scale=1.0, eps=1e-5, stream=None):
    """Gradients of norm_gate_forward from those of r (dr, None: 0) and h (dh,
    None: 0): a dict of dx, dy, dgate, dpre_weight, dpre_bias, dpost_weight and
    dpost_bias, None for what is not there."""
    return _norm_gate_backward(dr, dh, r, y, stats, pre, post, pre_weight, pre_bias, post_weight, post_bias, gate, gate_act,
                               residual_scale, branch_scale, eps, stream=stream)


@_on_stream
def _norm_gate_backward(dr, dh, r, y, stats, pre, post, pre_weight, pre_bias, post_weight, post_bias, gate, gate_act,
                        residual_scale, branch_scale, eps, want=(True,) * 5):
    """want: whether the gradients of gate, pre_weight, pre_bias, post_weight and post_bias are asked for."""
    stream_t = r if r is not None else dr
    d, rows, index = _norm_gate(stream_t, "r", y, pre, post, pre_weight, pre_bias, post_weight, post_bias, gate, gate_act,
                                residual_scale, branch_scale, eps)
    hidden = y.shape[1]
    if dr is not None:
        _need(dr, "dr", (stream_t.dtype,), (rows, hidden), index)
    if dh is not None:
        _need(dh, "dh", (y.dtype,), (rows, hidden), index)
    _need(stats, "stats", _F32, (rows, 4), index)
    dx, dy = _empty_like(stream_t), _empty_like(y)
    dgate, dw1, db1, dw2, db2 = (_empty_like(t) if t is not None and w else None
                                 for t, w in zip((gate, pre_weight, pre_bias, post_weight, post_bias), want))
    nbytes = _norm_gate_workspace(rows, hidden, (_TYPE[y.dtype], _TYPE[stream_t.dtype]), gate.shape[0] if gate is not None else 0, index)
    ws = _empty(nbytes, dtype=torch.uint8, device=y.device)
    C.check(C.bf16opt_norm_gate_backward(d, _p(dr), _p(dh), _p(r), y.data_ptr(), stats.data_ptr(), dx.data_ptr(),
                                         dy.data_ptr(), _p(dgate), _p(dw1), _p(db1), _p(dw2), _p(db2), ws.data_ptr(),
                                         nbytes, _raw_stream(index)))
    return dict(dx=dx, dy=dy, dgate=dgate, dpre_weight=dw1, dpre_bias=db1, dpost_weight=dw2, dpost_bias=db2)


class _NormGate(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, y, pre_weight, pre_bias, post_weight, post_bias, gate, how):
        ctx.set_materialize_grads(False)
        r, h, stats = norm_gate_forward(x, y, pre_weight=pre_weight, pre_bias=pre_bias, post_weight=post_weight,
                                        post_bias=post_bias, gate=gate, **how)
        ctx.save_for_backward(r, y, stats, pre_weight, pre_bias, post_weight, post_bias, gate)
        ctx.how = how
        return r, h

    @staticmethod
    @_first_only
    def backward(ctx, dr, dh):
        if dr is None and dh is None:
            return (None,) * 8
        r, y, stats, pre_weight, pre_bias, post_weight, post_bias, gate = ctx.saved_tensors
        _, _, *weights, wants_gate, _ = ctx.needs_input_grad
        g = _norm_gate_backward(dr.contiguous() if dr is not None else None, dh.contiguous() if dh is not None else None,
                                r, y, stats, pre_weight=pre_weight, pre_bias=pre_bias, post_weight=post_weight,
                                post_bias=post_bias, gate=gate, want=(wants_gate, *weights), **ctx.how)
        return (g["dx"], g["dy"], g["dpre_weight"], g["dpre_bias"], g["dpost_weight"], g["dpost_bias"], g["dgate"], None)


def norm_gate(x, y, *, pre="rms", post="rms", pre_weight=None, pre_bias=None, post_weight=None, post_bias=None, gate=None,
              gate_act="none", residual_scale=1.0, branch_scale=1.0, eps=1e-5):
    """(r, h) as norm_gate_forward, differentiable in x, y, the weights and the gate."""
    return _NormGate.apply(x, y, pre_weight, pre_bias, post_weight, post_bias, gate,
                           dict(pre=pre, post=post, gate_act=gate_act, residual_scale=residual_scale,
                                branch_scale=branch_scale, eps=eps))


# ----------------------------------------------------------------- expert balance

def _balance(logits, k, mask, groups, balance_weight, z_weight, renormalise):
    """(descriptor, tokens, experts, device index)."""
    tokens, experts, index = _matrix(logits, "logits")
    _need(logits, "logits", _TYPE, (tokens, experts), index, True)
    if mask is not None:
        _need(mask, "mask", (torch.bool, torch.uint8), (tokens,), index)
    return _BALANCE_T.pack(tokens, experts, k, groups, _TYPE[logits.dtype], 1 if renormalise else 0, logits.data_ptr(),
                           _stride(logits), _p(mask), balance_weight, z_weight), tokens, experts, index


@functools.lru_cache(maxsize=4096)
def _balance_workspace(tokens, experts, k, groups, index):
    with torch.cuda.device(index):
        rc, nbytes = C.bf16opt_balance_workspace(
            C.bf16opt_balance_t(tokens, experts, k, groups, 0, 0, None, experts, None, 0.0, 0.0))
        C.check(rc)
    return nbytes


@_on_stream
def balance_forward(logits, k, *, mask=None, groups=1, balance_weight=1e-2, z_weight=0.0, renormalise=True):
    """A router's choice: (ids [tokens, k] int32, weights [tokens, k] FP32,
    counts [groups, experts] int32, loss FP32, saved) for logits [tokens,
    experts] (bf16 or FP32); mask [tokens] bool or uint8, 0: the token counts
    for nothing; groups: runs of tokens balanced each for itself."""
    d, tokens, experts, index = _balance(logits, k, mask, groups, balance_weight, z_weight, renormalise)
    nbytes = _balance_workspace(tokens, experts, k, groups, index)
    dev = logits.device
    ids = _empty((tokens, k), dtype=torch.int32, device=dev)
    weights = _empty((tokens, k), dtype=torch.float32, device=dev)
    counts = _empty((groups, experts), dtype=torch.int32, device=dev)
    loss = _empty((), dtype=torch.float32, device=dev)
    saved = _empty(tokens + groups, dtype=torch.float32, device=dev)
    ws = _empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    C.check(C.bf16opt_balance_forward(d, ids.data_ptr(), weights.data_ptr(), counts.data_ptr(), loss.data_ptr(),
                                      saved.data_ptr(), _p(ws), nbytes, _raw_stream(index)))
    return ids, weights, counts, loss, saved


@_on_stream
def balance_backward(logits, ids, counts, saved, dweights=None, dloss=None, *, mask=None, groups=1, balance_weight=1e-2,
                     z_weight=0.0, renormalise=True, out=None):
    """Gradient of the logits from those of the weights (None: 0) and of the
    loss (a tensor of one FP32; None: 1), with balance_forward's arguments and
    results.  out may be logits itself."""
    k = _matrix(ids, "ids")[1]
    d, tokens, experts, index = _balance(logits, k, mask, groups, balance_weight, z_weight, renormalise)
    _need(ids, "ids", (torch.int32,), (tokens, k), index)
    _need(counts, "counts", (torch.int32,), (groups, experts), index)
    _need(saved, "saved", _F32, (tokens + groups,), index)
    if dweights is not None:
        _need(dweights, "dweights", _F32, (tokens, k), index)
    if dloss is not None:
        _need(dloss, "dloss", _F32, dloss.shape if isinstance(dloss, _Tensor) and dloss.numel() == 1 else (1,), index)
    given, out = out, _dlogits(logits, out, index)
    C.check(C.bf16opt_balance_backward(d, ids.data_ptr(), counts.data_ptr(), saved.data_ptr(), _p(dweights), _p(dloss),
                                       out.data_ptr(), _stride(out), _raw_stream(index)))
    _written(given)
    return out


class _Balance(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k, mask, how):
        ctx.set_materialize_grads(False)
        ids, weights, counts, loss, saved = balance_forward(logits, k, mask=mask, **how)
        ctx.save_for_backward(logits, ids, counts, saved, mask)
        ctx.how = how
        ctx.mark_non_differentiable(ids, counts)
        return ids, weights, counts, loss

    @staticmethod
    @_first_only
    def backward(ctx, _ids, dweights, _counts, dloss):
        if dweights is None and dloss is None:
            return None, None, None, None
        logits, ids, counts, saved, mask = ctx.saved_tensors
        if dloss is None:
            dloss = torch.zeros((), dtype=torch.float32, device=logits.device)
        return (balance_backward(logits, ids, counts, saved, dweights.contiguous() if dweights is not None else None,
                                 dloss, mask=mask, **ctx.how), None, None, None)


def balance(logits, k, *, mask=None, groups=1, balance_weight=1e-2, z_weight=0.0, renormalise=True):
    """(ids, weights, counts, loss) as balance_forward, differentiable in logits
    through weights and loss."""
    return _Balance.apply(logits, k, mask, dict(groups=groups, balance_weight=balance_weight, z_weight=z_weight,
                                                renormalise=renormalise))


# ------------------------------------- log-probabilities, policy and preference losses

_PREFER = {"sigmoid": C.BF16OPT_PREFER_SIGMOID, "hinge": C.BF16OPT_PREFER_HINGE, "ipo": C.BF16OPT_PREFER_IPO}


def _tokens(logits, labels, temperature, row_weight):
    """(descriptor, rows, device index)."""
    rows, vocab, index = _matrix(logits, "logits")
    _need(logits, "logits", _TYPE, (rows, vocab), index, True)
    _need(labels, "labels", _INDEX, (rows,), index)
    if row_weight is not None:
        _need(row_weight, "row_weight", _F32, (rows,), index)
    return _TOKENS_T.pack(rows, vocab, _TYPE[logits.dtype], _INDEX[labels.dtype], temperature, logits.data_ptr(), _stride(logits),
                          labels.data_ptr(), _p(row_weight)), rows, index


def _policy(rows, index, advantage, old_logp, ref_logp, clip_low, clip_high, kl_weight):
    _need(advantage, "advantage", _F32, (rows,), index)
    if old_logp is not None:
        _need(old_logp, "old_logp", _F32, (rows,), index)
    if ref_logp is not None:
        _need(ref_logp, "ref_logp", _F32, (rows,), index)
    return _POLICY_T.pack(advantage.data_ptr(), _p(old_logp), _p(ref_logp), clip_low, clip_high, kl_weight, 0)


@_on_stream
def token_logp_forward(logits, labels, *, temperature=1.0, row_weight=None):
    """Log-probabilities [rows] (FP32) that softmax(logits / temperature) gives
    to labels [rows] (int32 or int64), and saved [rows, 4] for
    token_logp_backward.  logits: [rows, vocab] bf16 or FP32.  A row with row_weight 0 or
    with a label outside the vocabulary does not count: what stands in it has no effect, and it has 0."""
    d, rows, index = _tokens(logits, labels, temperature, row_weight)
    dev = logits.device
    logp = _empty(rows, dtype=torch.float32, device=dev)
    saved = _empty((rows, 4), dtype=torch.float32, device=dev)
    C.check(C.bf16opt_token_logp_forward(d, logp.data_ptr(), saved.data_ptr(), _raw_stream(index)))
    return logp, saved


@_on_stream
def policy_forward(logits, labels, advantage, *, old_logp=None, ref_logp=None, clip_low=0.2, clip_high=0.2, kl_weight=0.0,
                   temperature=1.0, row_weight=None):
    """Clipped policy loss of each token, with kl_weight times an estimate of the
    KL distance to a reference: (loss [rows], logp [rows], saved [rows, 4]), FP32.
    advantage, old_logp (None: the tokens are this model's own, ratio 1) and ref_logp (None: no
    KL term): [rows] FP32, constants."""
    d, rows, index = _tokens(logits, labels, temperature, row_weight)
    p = _policy(rows, index, advantage, old_logp, ref_logp, clip_low, clip_high, kl_weight)
    dev = logits.device
    loss = _empty(rows, dtype=torch.float32, device=dev)
    logp = _empty(rows, dtype=torch.float32, device=dev)
    saved = _empty((rows, 4), dtype=torch.float32, device=dev)
    C.check(C.bf16opt_policy_forward(d, p, loss.data_ptr(), logp.data_ptr(), saved.data_ptr(), _raw_stream(index)))
    return loss, logp, saved


@_on_stream
def policy_loss_grad(logits, labels, advantage, dloss=None, *, old_logp=None, ref_logp=None, clip_low=0.2, clip_high=0.2,
                     kl_weight=0.0, temperature=1.0, row_weight=None, out=None):
    """(loss [rows], logp [rows], gradient of the logits), for a gradient dloss
    [rows], or 1, of each row's loss, in one pass over the logits.  out may be logits itself."""
    d, rows, index = _tokens(logits, labels, temperature, row_weight)
    p = _policy(rows, index, advantage, old_logp, ref_logp, clip_low, clip_high, kl_weight)
    if dloss is not None:
        _need(dloss, "dloss", _F32, (rows,), index)
    dev = logits.device
    loss = _empty(rows, dtype=torch.float32, device=dev)
    logp = _empty(rows, dtype=torch.float32, device=dev)
    given, out = out, _dlogits(logits, out, index)
    C.check(C.bf16opt_policy_loss_grad(d, p, _p(dloss), loss.data_ptr(), logp.data_ptr(), out.data_ptr(), _stride(out), _raw_stream(index)))
    _written(given)
    return loss, logp, out


@_on_stream
def preference_forward(logits, labels, offsets, *, ref_logp=None, kind="sigmoid", beta=0.1, label_smoothing=0.0, margin=0.0,
                       length_normalise=False, temperature=1.0):
    """Loss of pairs of sequences, one preferred to the other: (loss [pairs], logp
    [2 pairs] (the sequences' log-probabilities), saved [rows, 4]), FP32.  offsets [2 pairs + 1] (int32 or
    int64): sequence i is rows offsets[i] to offsets[i + 1]; sequence i is preferred to sequence
    pairs + i.  Rows whose label is outside the vocabulary (prompts, padding) and rows outside the
    sequences do not count.  ref_logp [2 pairs] FP32: a reference's (None: 0).
    kind: 'sigmoid', 'hinge' or 'ipo'; label_smoothing is the sigmoid's, the others take no notice of it."""
    d, rows, index = _tokens(logits, labels, temperature, None)
    if kind not in _PREFER:
        raise ValueError("kind: 'sigmoid', 'hinge' or 'ipo'")
    entries = offsets.shape[0] if isinstance(offsets, _Tensor) and offsets.dim() == 1 else 0
    if entries % 2 == 0:
        raise ValueError("offsets: must be [2 pairs + 1]")
    _need(offsets, "offsets", _INDEX, (entries,), index)
    if ref_logp is not None:
        _need(ref_logp, "ref_logp", _F32, (entries - 1,), index)
    pairs = entries // 2
    p = _PREFERENCE_T.pack(pairs, _INDEX[offsets.dtype], _PREFER[kind], offsets.data_ptr(), _p(ref_logp), beta, label_smoothing, margin,
                           1 if length_normalise else 0)
    dev = logits.device
    loss = _empty(pairs, dtype=torch.float32, device=dev)
    logp = _empty(2 * pairs, dtype=torch.float32, device=dev)
    saved = _empty((rows, 4), dtype=torch.float32, device=dev)
    C.check(C.bf16opt_preference_forward(d, p, loss.data_ptr(), logp.data_ptr(), saved.data_ptr(), _raw_stream(index)))
    return loss, logp, saved


@_on_stream
def token_logp_backward(logits, labels, saved, dloss=None, *, temperature=1.0, out=None):
    """Gradient of the logits from that of the losses (or log-probabilities) of
    token_logp_forward, policy_forward or preference_forward, with its saved and the same
    logits, labels and temperature.  dloss: FP32, one for each loss; None: 1.  out may be
    logits itself."""
    d, rows, index = _tokens(logits, labels, temperature, None)
    _need(saved, "saved", _F32, (rows, 4), index)
    losses = 0
    if dloss is not None:
        losses = dloss.shape[0] if isinstance(dloss, _Tensor) and dloss.dim() == 1 else 0
        _need(dloss, "dloss", _F32, (losses,), index)
    given, out = out, _dlogits(logits, out, index)
    C.check(C.bf16opt_token_logp_backward(d, saved.data_ptr(), _p(dloss), losses, out.data_ptr(), _stride(out), _raw_stream(index)))
    _written(given)
    return out


def _constants(**tensors):
    """The losses are differentiable in the logits alone."""
    for n, t in tensors.items():
        if isinstance(t, _Tensor) and t.requires_grad and torch.is_grad_enabled():
            raise ValueError(f"{n}: requires a gradient, which the loss does not give; detach it")


class _TokenLoss(torch.autograd.Function):
    """The three forward calls: (losses, further results that are constants)."""
    @staticmethod
    def forward(ctx, logits, labels, temperature, call):
        loss, *more, saved = call()
        ctx.save_for_backward(logits, labels, saved)
        ctx.temperature = temperature
        ctx.mark_non_differentiable(*more)
        return (loss, *more)

    @staticmethod
    @_first_only
    def backward(ctx, dloss, *_):
        logits, labels, saved = ctx.saved_tensors
        return token_logp_backward(logits, labels, saved, dloss.float().contiguous(), temperature=ctx.temperature), None, None, None


def token_logp(logits, labels, *, temperature=1.0, row_weight=None):
    """Log-probabilities [rows] as token_logp_forward, differentiable in logits."""
    _constants(row_weight=row_weight)
    return _TokenLoss.apply(logits, labels, temperature,
                            lambda: token_logp_forward(logits, labels, temperature=temperature, row_weight=row_weight))[0]


def policy_loss(logits, labels, advantage, *, old_logp=None, ref_logp=None, clip_low=0.2, clip_high=0.2, kl_weight=0.0,
                temperature=1.0, row_weight=None):
    """(loss [rows], logp [rows]) as policy_forward, the loss differentiable in logits; logp is a constant."""
    _constants(advantage=advantage, old_logp=old_logp, ref_logp=ref_logp, row_weight=row_weight)
    return _TokenLoss.apply(logits, labels, temperature, lambda: policy_forward(
        logits, labels, advantage, old_logp=old_logp, ref_logp=ref_logp, clip_low=clip_low, clip_high=clip_high,
        kl_weight=kl_weight, temperature=temperature, row_weight=row_weight))


def preference_loss(logits, labels, offsets, *, ref_logp=None, kind="sigmoid", beta=0.1, label_smoothing=0.0, margin=0.0,
                    length_normalise=False, temperature=1.0):
    """(loss [pairs], logp [2 pairs]) as preference_forward, the loss differentiable in logits; logp is a constant."""
    _constants(ref_logp=ref_logp)
    return _TokenLoss.apply(logits, labels, temperature, lambda: preference_forward(
        logits, labels, offsets, ref_logp=ref_logp, kind=kind, beta=beta, label_smoothing=label_smoothing, margin=margin,
        length_normalise=length_normalise, temperature=temperature))


# -------------------------------------------------------- activations kept in 8 bits

_GLU = {"silu": C.BF16OPT_GLU_SILU, "gelu": C.BF16OPT_GLU_GELU}
_U8 = (torch.uint8,)


def _output(out, like, what, shape, index):
    if out is None:
        return _empty(shape, dtype=like.dtype, device=like.device)
    _need(out, what, (like.dtype,), shape, index, True)
    _writable(out, what)
    return out


@_on_stream
def pack8(x):
    """(codes [rows, 32 runs], scales [rows, runs]), uint8, of an activation x [rows,
    columns] (bf16 or FP32): each run of 32 columns as e4m3 numbers times the power of two
    2^(scale - 127)."""
    rows, columns, index = _matrix(x, "x")
    _need(x, "x", _TYPE, (rows, columns), index, True)
    runs = (columns + 31) // 32
    codes = _empty((rows, 32 * runs), dtype=torch.uint8, device=x.device)
    scales = _empty((rows, runs), dtype=torch.uint8, device=x.device)
    C.check(C.bf16opt_pack(_PACK_T.pack(rows, columns, _TYPE[x.dtype]), x.data_ptr(), _stride(x), codes.data_ptr(), scales.data_ptr(),
                           _raw_stream(index)))
    return codes, scales


@_on_stream
def unpack8(codes, scales, columns, *, dtype=torch.bfloat16, out=None):
    """[rows, columns] of what pack8 kept, rounded to dtype (bf16 holds it exactly but below its smallest normal
    number)."""
    rows, wide, index = _matrix(codes, "codes")
    runs = (columns + 31) // 32
    _need(codes, "codes", _U8, (rows, 32 * runs), index)
    _need(scales, "scales", _U8, (rows, runs), index)
    if dtype not in _TYPE:
        raise ValueError("dtype: bf16 or FP32")
    if out is None:
        x = _empty((rows, columns), dtype=dtype, device=codes.device)
    else:
        _need(out, "out", (dtype,), (rows, columns), index, True)
        _writable(out, "out")
        x = out
    C.check(C.bf16opt_unpack(_PACK_T.pack(rows, columns, _TYPE[dtype]), codes.data_ptr(), scales.data_ptr(), x.data_ptr(), _stride(x),
                             _raw_stream(index)))
    _written(out)
    return x


@_on_stream
def glu8_forward(gate, up=None, *, act="silu", keep=True, out=None):
    """(h, codes, scales): h = act(gate) up, or act(gate) without up, [rows, columns] bf16
    or FP32 (rows may be apart: halves of one projection); codes [parts, rows, 32 runs] and scales [parts, rows, runs],
    uint8: gate and up as pack8 keeps them, for glu8_backward (keep=False: None).
    act: 'silu' or 'gelu' (by tanh).  out may be gate or up."""
    rows, columns, index = _matrix(gate, "gate")
    _need(gate, "gate", _TYPE, (rows, columns), index, True)
    if up is not None:
        _need(up, "up", (gate.dtype,), (rows, columns), index, True)
    if act not in _GLU:
        raise ValueError("act: 'silu' or 'gelu'")
    parts, runs = 1 if up is None else 2, (columns + 31) // 32
    h = _output(out, gate, "out", (rows, columns), index)
    codes = _empty((parts, rows, 32 * runs), dtype=torch.uint8, device=gate.device) if keep else None
    scales = _empty((parts, rows, runs), dtype=torch.uint8, device=gate.device) if keep else None
    d = _GLU_T.pack(rows, columns, _TYPE[gate.dtype], _GLU[act], parts - 1)
    C.check(C.bf16opt_glu_forward(d, gate.data_ptr(), _stride(gate), _p(up), _stride(up) if up is not None else 0, h.data_ptr(), _stride(h),
                                  _p(codes), _p(scales), _raw_stream(index)))
    _written(out)
    return h, codes, scales


@_on_stream
def glu8_backward(dh, codes, scales, *, act="silu", out_gate=None, out_up=None, out_h=None):
    """(dgate, dup) of glu8_forward from the gradient of h and what was kept; dup None without up.  out_gate and
    out_up may be halves of one matrix; out_h: where act(gate) up of what was kept is wanted too.  One of
    them may be dh."""
    rows, columns, index = _matrix(dh, "dh")
    _need(dh, "dh", _TYPE, (rows, columns), index, True)
    runs = (columns + 31) // 32
    parts = codes.shape[0] if isinstance(codes, _Tensor) and codes.dim() == 3 and codes.shape[0] in (1, 2) else 2
    _need(codes, "codes", _U8, (parts, rows, 32 * runs), index)
    _need(scales, "scales", _U8, (parts, rows, runs), index)
    if act not in _GLU:
        raise ValueError("act: 'silu' or 'gelu'")
    if parts == 1 and out_up is not None:
        raise ValueError("out_up: there is no up")
    dgate = _output(out_gate, dh, "out_gate", (rows, columns), index)
    dup = _output(out_up, dh, "out_up", (rows, columns), index) if parts == 2 else None
    if out_h is not None:
        _output(out_h, dh, "out_h", (rows, columns), index)
    d = _GLU_T.pack(rows, columns, _TYPE[dh.dtype], _GLU[act], parts - 1)
    C.check(C.bf16opt_glu_backward(d, dh.data_ptr(), _stride(dh), codes.data_ptr(), scales.data_ptr(), dgate.data_ptr(), _stride(dgate),
                                   _p(dup), _stride(dup) if dup is not None else 0, _p(out_h), _stride(out_h) if out_h is not None else 0,
                                   _raw_stream(index)))
    _written(out_gate, out_up, out_h)
    return dgate, dup


class _Glu8(torch.autograd.Function):
    @staticmethod
    def forward(ctx, gate, up, act):
        h, codes, scales = glu8_forward(gate, up, act=act, keep=any(ctx.needs_input_grad))
        ctx.save_for_backward(codes, scales)
        ctx.act = act
        return h

    @staticmethod
    @_first_only
    def backward(ctx, dh):
        codes, scales = ctx.saved_tensors
        return (*glu8_backward(dh if dh.stride(1) == 1 and dh.stride(0) >= dh.shape[1] else dh.contiguous(), codes, scales, act=ctx.act), None)


def glu8(gate, up=None, *, act="silu"):
    """h as glu8_forward, differentiable in gate and up.  Autograd keeps 33 / 32 bytes for each of their elements, and
    their gradients are those at the values that were kept."""
    return _Glu8.apply(gate, up, act)


# ------------------------------------------------------------------ rotary positions

_LAYOUT = {"half": C.BF16OPT_ROTARY_HALF, "interleaved": C.BF16OPT_ROTARY_INTERLEAVED}
_NOWHERE = (0, 0, 0)


@functools.lru_cache(maxsize=256)
def _frequencies(rotary_dim, base, scaling, factor, original_length, slow, fast):
    """(radians per position as packed doubles, their address, factor on the turned pairs' length)."""
    import ctypes
    if not (isinstance(rotary_dim, int) and rotary_dim >= 2 and rotary_dim % 2 == 0):
        raise ValueError("rotary_dim: must be even and at least 2")
    if not (math.isfinite(base) and base > 0 and math.isfinite(factor) and factor > 0):
        raise ValueError("base, factor: must be finite and > 0")
    scale = 1.0
    if scaling == "ntk":
        if rotary_dim < 4:
            raise ValueError("scaling 'ntk': rotary_dim must be at least 4")
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    f = [base ** (-2 * i / rotary_dim) for i in range(rotary_dim // 2)]
    if scaling == "linear":
        f = [v / factor for v in f]
    elif scaling == "yarn":
        if not (original_length > 0 and 0 <= slow < fast):
            raise ValueError("scaling 'yarn': original_length > 0 and 0 <= slow < fast")
        keep = [min(1.0, max(0.0, (original_length * v / (2 * math.pi) - slow) / (fast - slow))) for v in f]
        f = [v * (k + (1 - k) / factor) for v, k in zip(f, keep)]
        scale = 0.1 * math.log(factor) + 1 if factor > 1 else 1.0
    elif scaling not in (None, "none", "ntk"):
        raise ValueError("scaling: None, 'linear', 'ntk' or 'yarn'")
    table = (ctypes.c_double * len(f))(*f)
    return table, ctypes.addressof(table), scale


def _heads(t, what, dtypes, like=None):
    """(shape, strides between batches, tokens and heads) of [tokens, heads, dim] or [batch, tokens, heads, dim]."""
    if not isinstance(t, _Tensor) or not t.is_cuda:
        raise ValueError(f"{what}: must be a CUDA tensor")
    shape, s = t.shape, t.stride()
    n = len(s)
    if (n != 3 and n != 4) or t.dtype not in dtypes or (s[-1] != 1 and shape[-1] > 1):
        raise ValueError(f"{what}: must be [tokens, heads, dim] or [batch, tokens, heads, dim], of {[str(d) for d in dtypes]}, contiguous within heads")
    if like is not None and (t.get_device() != like.get_device() or shape[:-2] != like.shape[:-2] or shape[-1] != like.shape[-1]):
        raise ValueError(f"{what}: shape {tuple(shape)} on {t.device} does not go with {tuple(like.shape)} on {like.device}")
    return shape, ((0, s[0], s[1]) if n == 3 else s[:3])


def _turned(x, out, what, dtypes, shape):
    """(a result of x's shape, its strides): the caller's or a new one."""
    if out is None:
        heads, dim = shape[-2:]
        return _empty(shape, dtype=x.dtype, device=x.device), (shape[-3] * heads * dim, heads * dim, dim)
    got, strides = _heads(out, what, dtypes, x)
    if got != shape:
        raise ValueError(f"{what}: shape {tuple(got)}, expected {tuple(shape)}")
    _writable(out, what)
    return out, strides


@_on_stream
def _rotary(q, k, positions, rotary_dim, layout, base, scaling, factor, original_length, slow, fast, offset, out_q, out_k, inverse):
    shape, sq = _heads(q, "q", _TYPE)
    index, dtypes = q.get_device(), (q.dtype,)
    *batch, seq, heads, dim = shape
    batch = batch[0] if batch else 1
    if layout not in _LAYOUT:
        raise ValueError("layout: 'half' or 'interleaved'")
    sk, kv = _NOWHERE, 0
    if k is not None:
        k_shape, sk = _heads(k, "k", dtypes, q)
        kv = k_shape[-2]
    elif out_k is not None:
        raise ValueError("out_k: there is no k")
    each = 0
    if positions is not None:
        shared = isinstance(positions, _Tensor) and positions.dim() == 1
        _need(positions, "positions", _INDEX, (seq,) if shared else (batch, seq), index)
        each = 0 if shared else seq
    rotary_dim = dim if rotary_dim is None else rotary_dim
    table, address, scale = _frequencies(rotary_dim, base, scaling, factor, original_length, slow, fast)
    rq, so_q = _turned(q, out_q, "out_q", dtypes, shape)
    rk, so_k = _turned(k, out_k, "out_k", dtypes, k_shape) if k is not None else (None, _NOWHERE)
    one, two = (q, rq, sq, so_q, heads), (k, rk, sk, so_k, kv)
    if heads == 0:   # nothing of q: k in its place
        one, two = two, (None, None, _NOWHERE, _NOWHERE, 0)
        if kv == 0:
            return rq, rk
    elif kv == 0:
        two = (None, None, _NOWHERE, _NOWHERE, 0)
    d = _ROTARY_T.pack(batch, seq, one[4], two[4], dim, rotary_dim, _TYPE[q.dtype], _LAYOUT[layout],
                       _INDEX[positions.dtype] if positions is not None else 0, inverse, _p(positions), each, offset, address, scale, 0,
                       *one[2], *two[2], *one[3], *two[3])
    C.check(C.bf16opt_rotary(d, one[0].data_ptr(), _p(two[0]), one[1].data_ptr(), _p(two[1]), _raw_stream(index)))
    _written(out_q, out_k)
    return rq, rk


def rotary_forward(q, k=None, positions=None, *, rotary_dim=None, layout="half", base=10000.0, scaling=None, factor=1.0,
                   original_length=2048, slow=1.0, fast=32.0, offset=0, out_q=None, out_k=None, stream=None):
    """(q, k) with positions turned into the first rotary_dim elements of each head
    (None: all).  q: [tokens, heads, dim] or [batch, tokens, heads, dim], k (or None) the same with its own number of
    heads; bf16 or FP32; any strides with contiguous heads.  positions: None (0, 1, ..), [tokens] or [batch, tokens],
    int32 or int64; offset is added.  layout: pairs are (i, i + rotary_dim / 2) ('half') or neighbours
    ('interleaved').  Pair i turns by base^(-2 i / rotary_dim), a 64-bit number, a position;
    scaling for longer contexts: 'linear' (frequencies / factor), 'ntk' (base factor^(d / (d - 2))), 'yarn'
    (pairs that turn less than `slow` times in original_length are slowed by factor, those above `fast` are
    not, between them a ramp; the turned pairs are 0.1 ln(factor) + 1 times as long).  out_q may be q, out_k may be k."""
    return _rotary(q, k, positions, rotary_dim, layout, base, scaling, factor, original_length, slow, fast, offset, out_q, out_k, 0,
                   stream=stream)


def rotary_backward(dq, dk=None, positions=None, *, rotary_dim=None, layout="half", base=10000.0, scaling=None, factor=1.0,
                    original_length=2048, slow=1.0, fast=32.0, offset=0, out_q=None, out_k=None, stream=None):
    """Gradients of rotary_forward's inputs from those of its results: the same, turned back."""
    return _rotary(dq, dk, positions, rotary_dim, layout, base, scaling, factor, original_length, slow, fast, offset, out_q, out_k, 1,
                   stream=stream)


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, positions, how):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(positions)
        ctx.how = how
        return rotary_forward(q, k, positions, **how)

    @staticmethod
    @_first_only
    def backward(ctx, dq, dk):
        positions, = ctx.saved_tensors
        grads = [g if g is None or g.shape[-1] < 2 or g.stride(-1) == 1 else g.contiguous() for g in (dq, dk)]
        if grads[0] is None:
            return None, rotary_backward(grads[1], None, positions, **ctx.how)[0] if grads[1] is not None else None, None, None
        return (*rotary_backward(grads[0], grads[1], positions, **ctx.how), None, None)


def rotary(q, k=None, positions=None, *, rotary_dim=None, layout="half", base=10000.0, scaling=None, factor=1.0,
           original_length=2048, slow=1.0, fast=32.0, offset=0):
    """(q, k) as rotary_forward, differentiable in both."""
    return _Rotary.apply(q, k, positions, dict(rotary_dim=rotary_dim, layout=layout, base=base, scaling=scaling, factor=factor,
                                               original_length=original_length, slow=slow, fast=fast, offset=offset))
