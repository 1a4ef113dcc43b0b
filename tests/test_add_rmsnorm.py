"""Residual addition + RMSNorm (csa_add_rmsnorm) vs its formula in 64 bits.

Tolerances, relative to |y|: the sum of squares is fp32 over runs of at most
64 products per thread and a tree of at most 10 levels, so it is off by at most
(64 + 10 + 1) 2^-24 and its root by half of that; with the division, the root,
the two products and the weight each off by 2^-24, y is within 48 * 2^-24. An output
rounding adds half a step of the output's type (bf16 2^-8, E4M3 2^-4, or half of
E4M3's smallest step, 2^-10, times the scale)."""
import ctypes

import pytest
import torch

from compressed_sparse_attention_15_b200 import _lib, ops
from compressed_sparse_attention_15_b200.build import build

gpu = pytest.mark.gpu
F32 = 48 * 2.0 ** -24


def _inputs(rows, D, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, D, generator=g) * scale).to(dtype)
    r = (torch.randn(rows, D, generator=g) * 2 * scale).to(dtype)
    w = 1 + 0.1 * torch.randn(D, generator=g)
    return x, r, w


def _reference(h, w, eps):
    h = h.double()
    return h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * w.double()


def _check(out, x, r, w, eps, fp8, group):
    out = [t.cpu() for t in out]
    if r is not None:
        h = out[-1]
        # one rounding of the fp32 sum (itself off by 2^-24)
        total = x.double() + r.double()
        step = 2.0 ** -8 + 2.0 ** -23 if x.dtype == torch.bfloat16 else 2.0 ** -24
        assert torch.all((h.double() - total).abs() <= step * total.abs())
    else:
        h = x
    y = _reference(h, w, eps)
    if not fp8:
        step = 2.0 ** -8 if x.dtype == torch.bfloat16 else 2.0 ** -24
        err = (out[0].double() - y).abs()
        assert torch.all(err <= (F32 + step * (1 + F32)) * y.abs() + 2.0 ** -133), err.max()
        return
    g = group or x.shape[-1]
    s = out[1].double()
    amax = y.reshape(*y.shape[:-1], -1, g).abs().amax(-1)
    want = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
    assert torch.all((s - want).abs() <= (F32 + 2.0 ** -23) * want)
    s = s.repeat_interleave(g, -1)
    v = out[0].view(torch.float8_e4m3fn).double() * s
    err = (v - y).abs()
    assert torch.all(err <= (2.0 ** -4 + 2 * F32) * y.abs() + 2.0 ** -10 * s), err.max()


CASES = [
    # rows, D, residual, fp8, group
    (1, 4096, True, True, 128),
    (3, 4096, True, True, 0),
    (5, 512, False, True, 32),
    (7, 256, True, True, 256),
    (9, 1024, False, False, 0),
    (2, 16384, True, False, 0),
    (2, 16384, True, True, 64),
    (4, 8200, True, True, 0),
    (33, 1, True, False, 0),
    (6, 7, True, False, 0),
    (6, 1023, True, True, 0),
    (3, 96, False, True, 32),
    (70, 264, True, False, 0),
    (4097, 128, True, True, 64),
]


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,D,residual,fp8,group", CASES)
def test_matches_the_formula(cuda_device, rows, D, residual, fp8, group, dtype):
    x, r, w = _inputs(rows, D, dtype, rows * 7 + D)
    r = r if residual else None
    out = ops.add_rmsnorm(x.to(cuda_device), w.to(cuda_device), residual=None if r is None else r.to(cuda_device),
                          fp8=fp8, group=group)
    assert len(out) == 1 + fp8 + residual
    _check(out, x, r, w, 1e-6, fp8, group)


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_unaligned_strided_and_in_place(cuda_device, dtype):
    # rows of a wider tensor (strides that are and are not multiples of 8 elements, an odd base), h over the residual
    for D, wide, off in ((256, 512, 0), (256, 300, 3), (40, 41, 1)):
        x, r, w = _inputs(11, wide, dtype, wide)
        xs = x[:, off:off + D]
        r = r[:, :D].contiguous()
        w = w[:D].contiguous()
        rd = r.to(cuda_device)
        out = ops.add_rmsnorm(x.to(cuda_device)[:, off:off + D], w.to(cuda_device), residual=rd, sum_out=rd, eps=1e-3)
        assert out[-1].data_ptr() == rd.data_ptr()
        _check(out, xs, r, w, 1e-3, False, 0)
        # y over x, h over the residual
        rd, xd = r.to(cuda_device), xs.contiguous().to(cuda_device)
        out = ops.add_rmsnorm(xd, w.to(cuda_device), residual=rd, sum_out=rd, out=xd, eps=1e-3)
        _check(out, xs, r, w, 1e-3, False, 0)


@gpu
def test_odd_output_base(cuda_device):
    x, r, w = _inputs(5, 256, torch.bfloat16, 3)
    buf = torch.full((5 * 256 + 16,), 7, dtype=torch.uint8, device=cuda_device)
    out = buf[3:3 + 5 * 256].view(5, 256)
    got = ops.add_rmsnorm(x.to(cuda_device), w.to(cuda_device), residual=r.to(cuda_device), fp8=True, group=64, out=out)
    _check(got, x, r, w, 1e-6, True, 64)
    assert torch.all(buf[:3] == 7) and torch.all(buf[3 + 5 * 256:] == 7)


@gpu
@pytest.mark.parametrize("D", [256, 250])
@pytest.mark.parametrize("fp8", [False, True])
def test_zero_infinite_and_nan_rows(cuda_device, D, fp8):
    x = torch.ones(5, D, dtype=torch.bfloat16)
    x[1] = 0
    x[2, 3] = float("nan")
    x[3, 5] = float("inf")
    w = torch.ones(D)
    out = [t.cpu() for t in ops.add_rmsnorm(x.to(cuda_device), w.to(cuda_device), fp8=fp8)]
    y = out[0].view(torch.float8_e4m3fn).float() * out[1] if fp8 else out[0].float()
    assert torch.all(y[1] == 0) and torch.isnan(y[2]).all()
    assert torch.isnan(y[3, 5]) and torch.all(y[3, :5] == 0) and torch.all(y[3, 6:] == 0)
    for i in (0, 4):  # neighbours of the odd rows
        assert torch.all((y[i] - 1).abs() < 0.01)
    if fp8:
        assert out[1][1] == 1


@gpu
def test_empty_captured_and_on_a_side_stream(cuda_device):
    w = torch.ones(64, device=cuda_device)
    y, = ops.add_rmsnorm(torch.zeros(0, 64, device=cuda_device), w)
    assert y.shape == (0, 64)
    x, r, wh = _inputs(8, 64, torch.float32, 5)
    xd, rd, wd = x.to(cuda_device), r.to(cuda_device), wh.to(cuda_device)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ops.add_rmsnorm(xd, wd, residual=rd)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out = ops.add_rmsnorm(xd, wd, residual=rd, fp8=True, group=32)
        xd.copy_(x.flip(0))
        g.replay()
    s.synchronize()
    _check(out, x.flip(0), r, wh, 1e-6, True, 32)


def test_entry_point_refuses_bad_arguments():
    build()
    L = _lib.lib()
    N, P = ctypes.c_void_p(0), ctypes.c_void_p(4096)  # P is never dereferenced

    def call(x=P, xs=0, res=N, w=P, eps=1e-6, out=P, sc=N, so=N, rows=2, D=64, group=0, dt=1, od=1):
        return L.csa_add_rmsnorm(x, xs, res, w, eps, out, sc, so, rows, D, group, dt, od, N)

    odd = ctypes.c_void_p(4097)
    bad = [dict(x=N), dict(w=N), dict(out=N), dict(xs=63), dict(res=P), dict(so=P), dict(eps=-1.0),
           dict(eps=float("nan")), dict(rows=-1), dict(D=0), dict(D=16385), dict(dt=2), dict(od=0), dict(group=32),
           dict(od=2), dict(od=2, sc=ctypes.c_void_p(4098)), dict(od=2, sc=P, group=16), dict(od=2, sc=P, group=48),
           dict(od=2, sc=P, group=128), dict(x=odd), dict(out=odd), dict(res=odd, so=P), dict(w=ctypes.c_void_p(4098))]
    for kw in bad:
        assert call(**kw) == 1, kw
    assert call(rows=0, x=N, out=N) == 0


def test_wrapper_refuses_host_tensors():
    with pytest.raises(ValueError, match="CUDA tensor"):
        ops.add_rmsnorm(torch.zeros(2, 64), torch.ones(64))


@gpu
def test_wrapper_refuses_bad_shapes(cuda_device):
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device=cuda_device)  # noqa: E731
    w = z(64, dtype=torch.float32)
    for kw in (dict(x=z(2, 32)), dict(x=z(64, 2).t()), dict(x=z(2, 2, 128)[:, :, :64]), dict(residual=z(3, 64)),
               dict(sum_out=z(2, 64)), dict(group=32), dict(fp8=True, group=48), dict(out_scales=z(2, 1)),
               dict(fp8=True, out_scales=z(2, 2, dtype=torch.float32)), dict(out=z(2, 32))):
        with pytest.raises((ValueError, TypeError)):
            ops.add_rmsnorm(**{"x": z(2, 64), "weight": w, **kw})
    with pytest.raises(TypeError):
        ops.add_rmsnorm(z(2, 64, dtype=torch.float16), w)
    with pytest.raises(TypeError):
        ops.add_rmsnorm(z(2, 64), z(64))
    with pytest.raises(_lib.CsaError):
        ops.add_rmsnorm(z(2, 64), w, eps=-1.0)


def test_refuses_one_tensor_for_both_outputs():
    build()
    N, P, P2 = ctypes.c_void_p(0), ctypes.c_void_p(4096), ctypes.c_void_p(8192)  # never dereferenced
    assert _lib.lib().csa_add_rmsnorm(P, 0, P, P, 1e-6, P2, N, P2, 2, 64, 0, 1, 1, N) == 1


def _nearest_e4m3(q):
    """The E4M3 value nearest to q (64 bits), ties to the even one."""
    step = torch.ldexp(torch.ones_like(q), torch.frexp(q)[1].clamp(min=-5) - 4)
    return torch.round(q / step) * step


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("group", [0, 32, 256])
def test_codes_at_and_next_to_ties_are_the_quotient_s(cuda_device, dtype, group):
    # Rows of +-1 without eps have a norm of 1: y is +- the weight, any fp32 number. Every group's scale s has 18
    # bits, its largest weight is 448 s, the others are the middles between two E4M3 values times s (exact), or one
    # fp32 step beside them: quotients that are ties, or at least 2^-24 of themselves away from one.
    D = 4096
    g = torch.Generator().manual_seed(group)
    n = group or D
    s = torch.randint(1 << 17, 1 << 18, (D // n, 1), generator=g).double() * 2.0 ** torch.randint(-40, 20, (D // n, 1), generator=g)
    t = torch.randint(16, 32, (D // n, n), generator=g).double() * 2.0 ** torch.randint(-10, 4, (D // n, n), generator=g)
    low = torch.randint(0, 16, (D // n, n), generator=g).double() * 2.0 ** -10  # among the subnormals, and zero
    w = (s * torch.where(torch.rand(D // n, n, generator=g) < 0.2, low, t)).float()
    w = torch.nextafter(w, w * torch.randint(0, 3, w.shape, generator=g))  # one step down, none or up
    w[:, 0] = (448 * s[:, 0]).float()
    sign = torch.randint(0, 2, (3, D), generator=g) * 2 - 1
    quotient = (w.double() / s).float()  # the fp32 quotient (53 bits are enough for its rounding to be that of y / s)
    want = _nearest_e4m3(quotient.double().flatten() * sign).clamp(-448, 448)
    x = sign.to(dtype).to(cuda_device)
    buf = torch.zeros(3 * D + 16, dtype=torch.uint8, device=cuda_device)
    for out in (buf[:3 * D].view(3, D), buf[3:3 + 3 * D].view(3, D)):  # 8-byte aligned, and not
        codes, scales = ops.add_rmsnorm(x, w.flatten().to(cuda_device), eps=0.0, fp8=True, group=group, out=out)
        assert torch.equal(scales.cpu().double(), s.T.expand(3, -1))
        got = codes.view(torch.float8_e4m3fn).cpu().double()
        assert torch.equal(got, want), f"{int((got != want).sum())} of {want.numel()} codes"
        assert torch.equal(codes.cpu() >> 7 != 0, sign < 0), "the sign stays, of zeros too"
