"""GPU parity of swiglu, its 8-bit checkpoint and its gradients against the
float64 oracle."""

import numpy as np
import pytest
import torch

import nvfp4_quantization_grouped_amd as mxq
from nvfp4_quantization_grouped_amd import _lib
from oracle import moe
from tests.gpu_util import DTYPES, dev
from tests.moe_util import U, assert_rounded, f64, i32, values

pytestmark = pytest.mark.gpu

# sigmoid: exp(-|x|) by one hardware exponential (1 ulp = 2 roundings), its argument's error put back (1), 1 + a (1),
# the reciprocal (2), a product (1): 7 roundings; two products more in h.  16 leaves a factor of 1.7.
SIG = 16 * U


def bound_h(x):
    return SIG * np.abs(moe.swiglu(x)) + 2.0 ** -126 * np.abs(x).max(initial=0) ** 2


def bound_grad(x, gh):
    """d u s (1 + g (1 - s)) and d g s: relative errors of the factors; the bracket's is SIG (1 + |g|) absolute."""
    g, u = np.split(x, 2, axis=1)
    s = moe.sigmoid(g)
    tiny = 2.0 ** -126 * (1 + np.abs(x).max(initial=0)) ** 2 * np.abs(gh).max(initial=0)
    return np.concatenate([np.abs(gh * u * s) * (2 + 2 * np.abs(g)) * SIG, np.abs(gh * g * s) * SIG], 1) + tiny


def check(x, dtype, offs=None, checkpoint="fp8", seed=0):
    g = np.random.default_rng(seed)
    R, I = x.shape[0], x.shape[1] // 2
    n = R if offs is None else min(R, max(0, int(offs[-1])))
    leaf = x.detach().clone().requires_grad_(True)
    ot = None if offs is None else i32(offs)
    h = mxq.swiglu(leaf, ot, checkpoint=checkpoint)
    xs = f64(x)
    want = np.zeros((R, I))
    want[:n] = moe.swiglu(xs[:n])
    assert_rounded(h[:n], want[:n], dtype, bound_h(xs[:n]), "h")
    assert (f64(h[n:]) == 0).all()
    assert torch.equal(h, mxq.swiglu(x, ot)), "the call without a gradient gives the same"
    gh = values(g, (R, I), dtype, 0.5)
    gh[n:] = float("nan")
    grad, = torch.autograd.grad(h, leaf, gh)
    at = xs[:n] if checkpoint is None else moe.kept(xs[:n])
    gs = f64(gh)[:n]
    assert_rounded(grad[:n], moe.swiglu_grad(at, gs), dtype, bound_grad(at, gs), "grad")
    assert (f64(grad[n:]) == 0).all() and grad.dtype == x.dtype


@pytest.mark.parametrize("R,I", [(1, 32), (3, 64), (64, 2048), (257, 96), (33, 1408), (1000, 32), (2, 32 * 513)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("checkpoint", ["fp8", None])
def test_swiglu(R, I, dtype, checkpoint):
    check(values(np.random.default_rng(R + I), (R, 2 * I), dtype, 2.0), dtype, None, checkpoint, R)


@pytest.mark.parametrize("offs", [[10, 20, 37], [0, 0, 0], [5, 64, 64], [100, 90, 3], [1, 2, 1000], [0, 0, -4]])
@pytest.mark.parametrize("checkpoint", ["fp8", None])
def test_swiglu_rows_behind_the_last_expert(offs, checkpoint):
    """Rows from offs[-1] on hold NaN and are not read; offsets outside [0, rows] are clamped."""
    x = values(np.random.default_rng(1), (64, 256), "bf16")
    x[min(64, max(0, offs[-1])):] = float("nan")
    check(x, "bf16", np.array(offs, np.int32), checkpoint)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_swiglu_far_values(dtype):
    """Blocks of zeros, signed zeros, values that differ by 2^40 within a block, gates far out on both sides."""
    x = values(np.random.default_rng(2), (12, 128), dtype)
    x[0] = 0.0
    x[1] = -0.0
    x[2] *= torch.exp2(torch.arange(128, device=dev()).float() % 32 - 20).to(x.dtype)
    x[3, :64] = torch.linspace(-120, 120, 64, device=dev()).to(x.dtype)
    x[4] = 448.0
    x[5] = 449.0
    x[6] *= 2.0 ** -60
    x[7, :64] = -1.2784645
    check(x, dtype)
    check(x, dtype, checkpoint=None)


def test_swiglu_keeps_what_the_packed_cache_form_keeps():
    """Codes and scales are quantize_cache_packed's, bit for bit; rows that do not count stay as they were."""
    g = np.random.default_rng(3)
    L, s = _lib.moe_lib(), torch.cuda.current_stream().cuda_stream
    for dtype, R, I in (("bf16", 37, 160), ("f16", 5, 32), ("f32", 20, 2048)):
        x = values(g, (R, 2 * I), dtype, 3.0)
        x[1] *= 1e-4
        offs = i32([3, R - 2])
        h = torch.empty(R, I, dtype=x.dtype, device=dev())
        codes = torch.full((R, 2 * I), 77, dtype=torch.uint8, device=dev())
        scales = torch.full((R, I // 16), 78, dtype=torch.uint8, device=dev())
        assert L.swiglu_fwd(x.data_ptr(), {"f32": 0, "bf16": 1, "f16": 2}[dtype], R, I, offs.data_ptr(), 2, h.data_ptr(),
                            codes.data_ptr(), scales.data_ptr(), s) == 0
        want = mxq.quantize_cache_packed(x, "fp8", 32)
        assert torch.equal(codes[:R - 2], want[0][:R - 2]) and torch.equal(scales[:R - 2], want[1][:R - 2])
        assert (codes[R - 2:] == 77).all() and (scales[R - 2:] == 78).all()


@pytest.mark.parametrize("R,I", [(1, 32), (5, 96), (64, 2048), (33, 1408), (1000, 64), (2, 32 * 513)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("format", ["fp8", "mxfp4"])
def test_swiglu_quantized(R, I, dtype, format):
    """Bit for bit what quantizing swiglu's output gives, rows behind the last expert (which hold NaN) included."""
    x = values(np.random.default_rng(R + I + 1), (R, 2 * I), dtype, 2.0)
    x[0] = 0.0
    for offs in (None, i32([R // 2, max(0, R - 3)])):
        if offs is not None:
            x[max(0, R - 3):] = float("nan")
        codes, scales = mxq.swiglu_quantized(x, format, offs)
        h = mxq.swiglu(x, offs)
        want = mxq.quantize_cache_packed(h, "fp8", 32) if format == "fp8" else mxq.quantize_mxfp4(h)
        assert codes.dtype == want[0].dtype and scales.dtype == want[1].dtype
        assert torch.equal(codes, want[0]) and torch.equal(scales.view(torch.uint8), want[1].view(torch.uint8))


@pytest.mark.parametrize("format", ["fp8", "mxfp4"])
def test_swiglu_quantized_over_many_values(format):
    """One rounding of h more or less shows in about one code of ten million: 268 million of them."""
    x = torch.randn(32768, 2 * 8192, device=dev(), generator=torch.Generator(dev()).manual_seed(7)).mul_(3).half()
    codes, scales = mxq.swiglu_quantized(x, format)
    h = mxq.swiglu(x)
    want = mxq.quantize_cache_packed(h, "fp8", 32) if format == "fp8" else mxq.quantize_mxfp4(h)
    assert torch.equal(codes, want[0]) and torch.equal(scales.view(torch.uint8), want[1].view(torch.uint8))


def test_swiglu_past_32_bit_offsets():
    """Rows whose element offsets pass 2^31 and whose byte offsets pass 2^32: what the same rows give alone."""
    R, I = 600_000, 2048
    x = torch.randn(R, 2 * I, device=dev(), dtype=torch.bfloat16, generator=torch.Generator(dev()).manual_seed(8))
    offs = i32([R // 2, R - 5])
    at = torch.tensor([0, 1, 262143, 262144, 524287, 524288, R - 7, R - 6], device=dev())
    for checkpoint in ("fp8", None):
        leaf, few = x.detach().requires_grad_(True), x[at].requires_grad_(True)
        h = mxq.swiglu(leaf, offs, checkpoint)
        want = mxq.swiglu(few, None, checkpoint)
        assert torch.equal(h[at], want) and not h[R - 5:].any()
        go = x[:, :I].contiguous()
        got, = torch.autograd.grad(h, leaf, go)
        want, = torch.autograd.grad(want, few, go[at])
        assert torch.equal(got[at], want) and not got[R - 5:].any()
        del h, got, leaf
    for format in ("fp8", "mxfp4"):
        got, want = mxq.swiglu_quantized(x, format, offs), mxq.swiglu_quantized(x[at], format)
        assert torch.equal(got[0][at], want[0])
        assert torch.equal(got[1].view(torch.uint8)[at], want[1].view(torch.uint8))


def test_swiglu_holds_what_it_says():
    """With a gradient wanted, the graph keeps 8 bits an element (and a scale per 32), not the input."""
    x = values(np.random.default_rng(4), (4096, 4096), "bf16").requires_grad_(True)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    h = mxq.swiglu(x)
    held = torch.cuda.memory_allocated() - before - h.numel() * 2
    assert x.numel() <= held <= x.numel() * 1.04


def test_swiglu_strided_misaligned_and_empty():
    g = np.random.default_rng(5)
    base = values(g, (20, 300), "bf16")
    for x in (base[:, 3:131], base[:, ::2][:, :128], base.view(-1)[1:20 * 128 + 1].view(20, 128)):
        check(x, "bf16")
    e = torch.zeros(0, 64, device=dev(), requires_grad=True)
    assert torch.autograd.grad(mxq.swiglu(e).sum(), e)[0].shape == (0, 64)
    leaf = base[:, :128].contiguous().requires_grad_(True)
    a, = torch.autograd.grad(mxq.swiglu(leaf).sum(), leaf)                   # a broadcast gradient
    b, = torch.autograd.grad(mxq.swiglu(leaf), leaf, torch.ones(20, 64, device=dev(), dtype=torch.bfloat16))
    assert torch.equal(a, b)


def test_swiglu_refusals():
    x = torch.zeros(4, 128, device=dev())
    for call in (lambda: mxq.swiglu(x[:, :96]), lambda: mxq.swiglu(x, checkpoint="int8"),
                 lambda: mxq.swiglu(x.view(-1)), lambda: mxq.swiglu(x, torch.zeros(2, dtype=torch.int32)),
                 lambda: mxq.swiglu_quantized(x[:, :96], "fp8"), lambda: mxq.swiglu_quantized(x, "nvfp4")):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: mxq.swiglu(x.double()), lambda: mxq.swiglu(x, torch.zeros(2, device=dev())),
                 lambda: mxq.swiglu(x, torch.zeros(0, dtype=torch.int32, device=dev()))):
        with pytest.raises(TypeError):
            call()
