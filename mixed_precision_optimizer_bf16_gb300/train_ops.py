"""Training operators from torch tensors: distillation loss, gated norms, expert balance.

Marshalling only (shapes, types, data_ptr()s, stream handles, status ->
exception); all arithmetic is in libbf16opt.so (the "training operators" of
include/bf16opt.h, where the formulas stand).  Outputs and workspaces are torch
allocations made on the stream that the kernels run on: the current one, or
`stream`.  Nothing synchronises, so a training step that uses these calls
can be captured in a CUDA graph.

  distill_forward / distill_backward / distill_loss_grad, distill_loss (autograd)
  norm_gate_forward / norm_gate_backward, norm_gate (autograd)
  balance_forward / balance_backward, balance (autograd)

The autograd forms have first derivatives only: going through a gradient of theirs once more
is an error.
"""
import contextlib
import functools
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
