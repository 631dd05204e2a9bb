"""The routed-expert layer around the grouped GEMM: router, grouped order,
the rows' way to their experts and back, and the experts' activation with its
input kept in 8 bits.

Argument marshalling and autograd only: every step runs in the HIP kernels
behind the C ABI (``include/mxq_moe.h``, which defines each operation).
Tensors must be CUDA (ROCm) tensors on one device; calls are enqueued on the
current stream of that device, outputs and workspaces are allocated with
PyTorch's caching allocator.  There is no CPU path.

Everything can be captured into a graph, backward passes too; as with any
operator, a backward is captured with ``torch.autograd.grad``, or with leaves of
which no eager graph is alive.  Second derivatives and forward-mode derivatives
are refused.

A layer's pass, as :func:`mxfp4_moe` makes it::

    weights, experts = moe_route(logits, 8, score="sigmoid", bias=bias, groups=8, top_groups=4)
    plan = moe_plan(experts, num_experts)
    rows = moe_dispatch(x, plan)
    rows = MXFP4GroupedMM.apply(rows, gate_up, gate_up_scales, plan.offs)
    rows = swiglu(rows, plan.offs)
    rows = MXFP4GroupedMM.apply(rows, down, down_scales, plan.offs)
    out = moe_combine(rows, weights, plan)
"""

from typing import NamedTuple

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import _lib
from .ops import _DT, _E8M0, _FMT, _need_cuda
from .ops import MXFP4GroupedMM, mxfp4_grouped_mm_fwd_w4a4_quantized, mxfp4_grouped_mm_fwd_w4a8_quantized

CHECKPOINT_BLOCK = 32
_SCORE = {"softmax": 0, "sigmoid": 1}


class MoEPlan(NamedTuple):
    """Grouped order of the routed slots (slot t * top_k + j is token t's j-th expert).

    offs: int32 [local experts], cumulative row counts, what the grouped GEMM takes.
    rows: int32 [tokens, top_k], each slot's row r, or ~r (negative) for a slot
        that no local expert serves; such rows lie behind offs[-1].
    slots: int32 [tokens * top_k], the slot in each row.
    """
    offs: torch.Tensor
    rows: torch.Tensor
    slots: torch.Tensor


_entries = {}


def _call(name, device, *args):
    """Run entry point ``name`` on ``device``'s current stream (appended as the last argument).

    A decoding step makes these calls one after another, and a backward makes
    them on a thread that has just woken, so the host's part of each counts: the
    raw stream handle costs 0.1 us against 1.9 us for a Stream object (8 us on
    autograd's thread), and the device is only switched where it has to be
    (1.3 us)."""
    fn = _entries.get(name)
    if fn is None:
        fn = _entries[name] = getattr(_lib.moe_lib(), name)
    index = device.index
    if index == torch._C._cuda_getDevice():
        status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if status:
        _lib.check(status, name)


def _first_order(backward):
    """A Function's backward without a second derivative.  ``once_differentiable``
    says so to autograd, at 20 us a call on the autograd thread; it is only
    needed where a graph of the backward is being made (create_graph)."""
    guarded = once_differentiable(backward)

    def run(ctx, *grads):
        return guarded(ctx, *grads) if torch.is_grad_enabled() else backward(ctx, *grads)
    return run


def _differentiated(*tensors):
    """Whether autograd has to see a call on these tensors: one wants a gradient, or a forward-mode level is open and one
    carries a tangent (which the Functions refuse: they have no forward-mode derivative)."""
    if torch.is_grad_enabled():
        for t in tensors:
            if t.requires_grad:
                return True
    return forward_ad._current_level >= 0 and any(forward_ad.unpack_dual(t).tangent is not None for t in tensors)


def _float_type(t, name):
    code = _DT.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    return code


def _ptr(t):
    """Address of a tensor's first element; 0 (NULL) for None and for an empty tensor."""
    return 0 if t is None else t.data_ptr()


# ------------------------------------------------------------------- router
def _route(logits, top_k, score, bias, groups, top_groups, group_best, renormalize, scale, mask):
    T, E = logits.shape
    device = logits.device
    weights = torch.empty(T, top_k, dtype=torch.float32, device=device)
    experts = torch.empty(T, top_k, dtype=torch.int32, device=device)
    _call("moe_route", device, logits.data_ptr(), _DT[logits.dtype], T, E, top_k, score, _ptr(bias), groups,
          top_groups, group_best, renormalize, scale, _ptr(mask), weights.data_ptr(), experts.data_ptr())
    return weights, experts


class _MoERoute(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, top_k, score, bias, groups, top_groups, group_best, renormalize, scale, mask):
        weights, experts = _route(logits, top_k, score, bias, groups, top_groups, group_best, renormalize, scale, mask)
        ctx.save_for_backward(logits, experts)
        ctx.how = score, renormalize, scale
        ctx.mark_non_differentiable(experts)
        ctx.set_materialize_grads(False)      # no zeros for the experts' missing gradient
        return weights, experts

    @staticmethod
    @_first_order
    def backward(ctx, grad_weights, _):
        if grad_weights is None:
            return (None,) * 10
        logits, experts = ctx.saved_tensors
        score, renormalize, scale = ctx.how
        g = grad_weights.contiguous()
        grad = torch.empty_like(logits)
        T, E = logits.shape
        _call("moe_route_bwd", logits.device, logits.data_ptr(), _DT[logits.dtype], T, E, experts.shape[1], score,
              renormalize, scale, experts.data_ptr(), g.data_ptr(), grad.data_ptr())
        return (grad,) + (None,) * 9


def moe_route(logits, top_k, *, score="softmax", bias=None, groups=1, top_groups=1, group_best=2, renormalize=True,
              scale=1.0, token_mask=None):
    """Experts and weights of each token from its router logits [T, E].

    ``score``: "softmax" over the experts or "sigmoid" of each; ``bias``
    (float32 [E]) is added to the scores for the choice only; with ``groups``
    runs of experts only the ``top_groups`` best (by the sum of their
    ``group_best`` largest biased scores) are kept; the ``top_k`` best experts
    are taken, ties to the lower index.  The weights are the chosen scores,
    divided by their sum with ``renormalize``, times ``scale``.  Tokens with
    ``token_mask`` (bool [T]) false, and places for which no expert is left
    (logits or biases of -inf), get expert -1 and weight 0.

    Returns (weights float32 [T, top_k], experts int32 [T, top_k]); the weights
    have a gradient with respect to the logits."""
    if score not in _SCORE:
        raise ValueError("moe_route: score must be 'softmax' or 'sigmoid'")
    _need_cuda(logits)
    _float_type(logits, "moe_route")
    if logits.dim() != 2:
        raise ValueError("moe_route: logits must be [tokens, experts]")
    if bias is not None:
        _need_cuda(logits, bias)
        if bias.dtype != torch.float32 or bias.shape != logits.shape[1:]:
            raise TypeError("moe_route: bias must be float32 [experts]")
        bias = bias.detach().contiguous()
    if token_mask is not None:
        _need_cuda(logits, token_mask)
        if token_mask.dtype != torch.bool or token_mask.shape != logits.shape[:1]:
            raise TypeError("moe_route: token_mask must be bool [tokens]")
        token_mask = token_mask.contiguous()
    top_k = int(top_k)
    if not 1 <= top_k <= min(32, logits.shape[1]):
        raise ValueError("moe_route: top_k must be between 1 and 32 and no more than the experts")
    args = (logits.contiguous(), top_k, _SCORE[score], bias, int(groups), int(top_groups), int(group_best),
            int(bool(renormalize)), float(scale), token_mask)
    return _MoERoute.apply(*args) if _differentiated(logits) else _route(*args)


# ------------------------------------------------------------ grouped order
def moe_plan(experts, num_experts, first_expert=0, local_experts=None):
    """Grouped order of the slots of ``experts`` (int32 [T, top_k], as
    ``moe_route`` returns them) for the ``local_experts`` experts from
    ``first_expert`` on (default: all ``num_experts``): a stable sort by
    expert.  Every other value, -1 among them, is a slot that is not served."""
    _need_cuda(experts)
    num_experts, first_expert = int(num_experts), int(first_expert)
    local = num_experts - first_expert if local_experts is None else int(local_experts)
    if experts.dtype != torch.int32:
        raise TypeError("moe_plan: experts must be int32")
    if experts.dim() != 2:
        raise ValueError("moe_plan: experts must be [tokens, top_k]")
    if first_expert < 0 or local < 1 or first_expert + local > num_experts:
        raise ValueError("moe_plan: the local experts must lie within num_experts")
    e = experts.contiguous()
    T, k = e.shape
    need = _lib.moe_lib().moe_plan_workspace(T, k, local)
    if need < 0:
        raise ValueError("moe_plan: at most 1024 local experts and fewer than 2^31 - 2^16 slots, top_k at least 1")
    offs = torch.empty(local, dtype=torch.int32, device=e.device)
    rows = torch.empty_like(e)
    slots = torch.empty(T * k, dtype=torch.int32, device=e.device)
    work = torch.empty(need // 4, dtype=torch.int32, device=e.device) if need else None
    _call("moe_plan", e.device, e.data_ptr(), T, k, first_expert, local, offs.data_ptr(), rows.data_ptr(),
          slots.data_ptr(), _ptr(work), need)
    return MoEPlan(offs, rows, slots)


def _plan_rows(rows, tokens, device, name):
    if rows.dtype != torch.int32 or rows.dim() != 2:
        raise TypeError(f"{name}: plan.rows must be int32 [tokens, top_k]")
    if rows.device != device:
        raise ValueError("all tensors must be on the same device")
    if tokens is not None and rows.shape[0] != tokens:
        raise ValueError(f"{name}: the plan is of {rows.shape[0]} tokens, not {tokens}")
    if rows.shape[1] < 1:
        raise ValueError(f"{name}: the plan has no slot for a token")
    return rows.contiguous()


def _dispatch(x, rows):
    (T, H), k = x.shape, rows.shape[1]
    out = torch.empty(T * k, H, dtype=x.dtype, device=x.device)
    _call("moe_dispatch", x.device, x.data_ptr(), _DT[x.dtype], T, H, k, rows.data_ptr(), out.data_ptr())
    return out


class _MoEDispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, rows):
        ctx.save_for_backward(rows)
        return _dispatch(x, rows)

    @staticmethod
    @_first_order
    def backward(ctx, grad):
        rows, = ctx.saved_tensors
        g = grad.contiguous()
        (T, k), H = rows.shape, g.shape[1]
        out = g.new_empty((T, H))
        _call("moe_dispatch_bwd", g.device, g.data_ptr(), _DT[g.dtype], T, H, k, rows.data_ptr(), out.data_ptr())
        return out, None


def moe_dispatch(x, plan):
    """Tokens' rows in the grouped order: x [T, H] -> [T * top_k, H], zeros in
    the rows behind ``plan.offs[-1]``.  The gradient of x sums its served rows
    in float32."""
    _need_cuda(x)
    _float_type(x, "moe_dispatch")
    if x.dim() != 2:
        raise ValueError("moe_dispatch: x must be [tokens, hidden]")
    rows = _plan_rows(plan.rows, x.shape[0], x.device, "moe_dispatch")
    x = x.contiguous()
    return _MoEDispatch.apply(x, rows) if _differentiated(x) else _dispatch(x, rows)


def _quantized_rows(rows, width, format, device):
    """Codes and scale bytes of rows in the form that the products with low-bit activations take."""
    if format == "mxfp4":
        codes = torch.empty(rows, width // 2, dtype=torch.int8, device=device)
    else:
        codes = torch.empty(rows, width, dtype=torch.uint8, device=device)
    return codes, torch.empty(rows, width // 32, dtype=torch.uint8, device=device)


def _scale_view(scales, format):
    return scales.view(_E8M0) if format == "mxfp4" and _E8M0 is not None else scales


def moe_dispatch_quantized(x, plan, format):
    """``moe_dispatch`` with the rows quantized on the way, in the form that a
    grouped GEMM with low-bit activations takes (no gradient).

    "fp8": (codes uint8 [T * top_k, H], scales uint8 [T * top_k, H / 32]) as
    ``quantize_cache_packed(rows, "fp8", 32)`` gives them, for
    ``mxfp4_grouped_mm_fwd_w4a8_quantized``; "mxfp4": (int8 [T * top_k, H / 2],
    float8_e8m0fnu [T * top_k, H / 32]) as ``quantize_mxfp4(rows)``, for
    ``mxfp4_grouped_mm_fwd_w4a4_quantized``.  H % 32 == 0."""
    _need_cuda(x)
    dt = _float_type(x, "moe_dispatch_quantized")
    if format not in ("fp8", "mxfp4"):
        raise ValueError("moe_dispatch_quantized: format must be 'fp8' or 'mxfp4'")
    if x.dim() != 2 or x.shape[1] % 32:
        raise ValueError("moe_dispatch_quantized: x must be [tokens, hidden] with hidden a multiple of 32")
    rows = _plan_rows(plan.rows, x.shape[0], x.device, "moe_dispatch_quantized")
    x = x.detach().contiguous()
    (T, H), k = x.shape, rows.shape[1]
    codes, scales = _quantized_rows(T * k, H, format, x.device)
    _call("moe_dispatch_quantized", x.device, x.data_ptr(), dt, T, H, k, rows.data_ptr(), _FMT[format],
          codes.data_ptr(), scales.data_ptr())
    return codes, _scale_view(scales, format)


# ------------------------------------------------------------------ combine
def _combine(y, weights, rows):
    (T, k), H = rows.shape, y.shape[1]
    out = torch.empty(T, H, dtype=y.dtype, device=y.device)
    _call("moe_combine", y.device, y.data_ptr(), _DT[y.dtype], T, H, k, rows.data_ptr(), weights.data_ptr(),
          out.data_ptr())
    return out


class _MoECombine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, weights, rows):
        ctx.save_for_backward(y if ctx.needs_input_grad[1] else None, weights, rows)
        return _combine(y, weights, rows)

    @staticmethod
    @_first_order
    def backward(ctx, grad):
        y, weights, rows = ctx.saved_tensors
        want_y, want_weights, _ = ctx.needs_input_grad
        g = grad.contiguous()
        (T, k), H = rows.shape, g.shape[1]
        gy = g.new_empty((T * k, H)) if want_y else None
        gw = torch.empty_like(weights) if want_weights else None
        _call("moe_combine_bwd", g.device, g.data_ptr(), _ptr(y), _DT[g.dtype], T, H, k, rows.data_ptr(),
              weights.data_ptr(), _ptr(gy), _ptr(gw))
        return gy, gw, None


def moe_combine(y, weights, plan):
    """The experts' rows back to their tokens: out[t] = sum over the served
    slots of weights[t, j] * y[row of (t, j)], summed in float32 in slot
    order.  y [T * top_k, H], weights float32 [T, top_k]; both have
    gradients."""
    _need_cuda(y, weights)
    _float_type(y, "moe_combine")
    if weights.dtype != torch.float32:
        raise TypeError("moe_combine: weights must be float32")
    rows = _plan_rows(plan.rows, None, y.device, "moe_combine")
    if weights.shape != rows.shape:
        raise ValueError("moe_combine: weights must be [tokens, top_k] like plan.rows")
    if y.dim() != 2 or y.shape[0] != rows.numel():
        raise ValueError("moe_combine: y must be [tokens * top_k, hidden]")
    y, weights = y.contiguous(), weights.contiguous()
    if _differentiated(y, weights):
        return _MoECombine.apply(y, weights, rows)
    return _combine(y, weights, rows)


# ------------------------------------------------------------------- swiglu
def _gate_up_args(gate_up, offs, name):
    if gate_up.dim() != 2 or gate_up.shape[1] % 64:
        raise ValueError(f"{name}: gate_up must be [rows, 2 * inter] with inter a multiple of 32")
    if offs is not None:
        _need_cuda(gate_up, offs)
        if offs.dtype != torch.int32 or offs.dim() != 1 or offs.shape[0] == 0:
            raise TypeError(f"{name}: offs must be int32 [experts]")
        offs = offs.contiguous()
    return gate_up.contiguous(), offs


def _swiglu(x, offs, keep):
    R, I = x.shape[0], x.shape[1] // 2
    h = torch.empty(R, I, dtype=x.dtype, device=x.device)
    codes = scales = None
    if keep:
        codes = torch.empty(R, 2 * I, dtype=torch.uint8, device=x.device)
        scales = torch.empty(R, 2 * I // CHECKPOINT_BLOCK, dtype=torch.uint8, device=x.device)
    _call("swiglu_fwd", x.device, x.data_ptr(), _DT[x.dtype], R, I, _ptr(offs), 0 if offs is None else offs.shape[0],
          h.data_ptr(), _ptr(codes), _ptr(scales))
    return h, codes, scales


class _SwiGLU(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, offs, checkpoint):
        h, codes, scales = _swiglu(x, offs, checkpoint == "fp8")
        ctx.save_for_backward(None if checkpoint == "fp8" else x, codes, scales, offs)
        return h

    @staticmethod
    @_first_order
    def backward(ctx, grad):
        x, codes, scales, offs = ctx.saved_tensors
        g = grad.contiguous()
        R, I = g.shape
        out = g.new_empty((R, 2 * I))
        _call("swiglu_bwd", g.device, g.data_ptr(), _ptr(x), _ptr(codes), _ptr(scales), _DT[g.dtype], R, I, _ptr(offs),
              0 if offs is None else offs.shape[0], out.data_ptr())
        return out, None, None


def swiglu(gate_up, offs=None, checkpoint="fp8"):
    """h = silu(gate) * up of gate_up [rows, 2 * inter] = [gate | up], inter a
    multiple of 32.  With ``offs`` (int32 cumulative counts, as the grouped
    GEMM takes them) the rows from offs[-1] on are not read and come out as
    zeros, as do their gradients.

    Where a gradient is wanted, ``checkpoint="fp8"`` keeps gate_up for the
    backward as E4M3 codes with one power-of-two scale per 32 columns (what
    ``quantize_cache_packed(gate_up, "fp8", 32)`` gives), and the gradient is
    that of silu(gate) * up at the kept values, which are up to 2^-4 of their
    size (or 2^-10 of the block's power of two) from the true ones, whatever the
    type of gate_up.  ``checkpoint=None`` keeps gate_up itself: the gradient at the
    true values, for 2 or 4 bytes an element instead of 1.03.  An inf or a NaN
    reaches the gradients at its place either way; kept in 8 bits it takes the
    other values of its block with it."""
    _need_cuda(gate_up)
    _float_type(gate_up, "swiglu")
    if checkpoint not in ("fp8", None):
        raise ValueError("swiglu: checkpoint must be 'fp8' or None")
    x, offs = _gate_up_args(gate_up, offs, "swiglu")
    if _differentiated(x):
        return _SwiGLU.apply(x, offs, checkpoint)
    return _swiglu(x, offs, False)[0]


def swiglu_quantized(gate_up, format, offs=None):
    """``swiglu`` with h quantized on its way out, in the form that a grouped
    GEMM with low-bit activations takes (no gradient): the codes and scales that
    quantizing swiglu's output gives, bit for bit, as ``moe_dispatch_quantized``
    returns them for "fp8" and "mxfp4"."""
    _need_cuda(gate_up)
    dt = _float_type(gate_up, "swiglu_quantized")
    if format not in ("fp8", "mxfp4"):
        raise ValueError("swiglu_quantized: format must be 'fp8' or 'mxfp4'")
    x, offs = _gate_up_args(gate_up.detach(), offs, "swiglu_quantized")
    R, I = x.shape[0], x.shape[1] // 2
    codes, scales = _quantized_rows(R, I, format, x.device)
    _call("swiglu_quantized", x.device, x.data_ptr(), dt, R, I, _ptr(offs), 0 if offs is None else offs.shape[0],
          _FMT[format], codes.data_ptr(), scales.data_ptr())
    return codes, _scale_view(scales, format)


# -------------------------------------------------------------------- layer
def mxfp4_moe(x, weights, experts, gate_up, gate_up_scales, down, down_scales, *, num_experts=None, first_expert=0,
              activations="bf16", checkpoint="fp8"):
    """The routed experts of one layer on bf16 x [T, H]: gather, gate/up
    product, SwiGLU, down product, weighted sum.

    ``weights``, ``experts``: as ``moe_route`` returns them.  ``gate_up`` and
    ``gate_up_scales``: mxfp4 [E, 2 * inter, H] packed as int8 [E, 2 * inter,
    H / 2] with E8M0 [E, 2 * inter, H / 32]; ``down`` and ``down_scales``:
    [E, H, inter] likewise, of the E local experts, which are experts
    first_expert .. first_expert + E - 1 of ``num_experts`` (default: the last
    of them); slots of other experts add nothing.
    ``activations``: "bf16" (gradients for x and weights; ``checkpoint`` is
    swiglu's: "fp8" rounds what the activation's gradient is taken at, None does
    not), or "fp8" / "mxfp4" activations in both products (W4A8 / W4A4,
    no gradients; H and inter multiples of 512)."""
    if activations not in ("bf16", "fp8", "mxfp4"):
        raise ValueError("mxfp4_moe: activations must be 'bf16', 'fp8' or 'mxfp4'")
    if x.dtype != torch.bfloat16 or x.dim() != 2:
        raise TypeError("mxfp4_moe: x must be bfloat16 [tokens, hidden]")
    if activations != "bf16" and _differentiated(x, weights):
        raise ValueError("mxfp4_moe: low-bit activations have no gradient")
    local = gate_up.shape[0]
    plan = moe_plan(experts, first_expert + local if num_experts is None else num_experts, first_expert, local)
    if activations == "bf16":
        rows = MXFP4GroupedMM.apply(moe_dispatch(x, plan), gate_up, gate_up_scales, plan.offs)
        rows = MXFP4GroupedMM.apply(swiglu(rows, plan.offs, checkpoint), down, down_scales, plan.offs)
    else:
        mm = mxfp4_grouped_mm_fwd_w4a8_quantized if activations == "fp8" else mxfp4_grouped_mm_fwd_w4a4_quantized
        rows = mm(*moe_dispatch_quantized(x, plan, activations), gate_up, gate_up_scales, plan.offs)
        rows = mm(*swiglu_quantized(rows, activations, plan.offs), down, down_scales, plan.offs)
    return moe_combine(rows, weights, plan)
