"""GPU tests of qlora_fmt4_linear_fwd: the product of a few tokens with an Int4 / FP4 E2M1 /
FP4 E3M0 weight straight from its codes, against the formula in 64 bits.

Tolerance, element by element, with S = sum_k |w_k| |x_k|:
  * the output's rounding: half a step, eps / 2 |y|;
  * inside a 64-block four mma add 16 exact products each to fp32: every term is cut to 24 bits
    at the largest's exponent, at most 17 2^-23 of the terms' sum each, 4 times: 2^-16 S covers it;
  * a constant and an addition per block, the sums over at most 16 warps, 8 CTAs and the final
    factor: (blocks + 32) 2^-24 S;
  * the split of x: inputs below 2^-31 of the largest of their 256 neighbours, 2^-39 of it each.
"""
import pytest
import torch

import bit_nf4_quantized_double_b200 as q
from oracle import formats as F

pytestmark = pytest.mark.gpu

FMTS = ("int4", "fp4_e2m1", "fp4_e3m0")


def weight64(codes, absmax, rows, cols, fmt):
    """|w| signs and all, fp64, from the packed codes."""
    S, mags = F.FORMATS[fmt]
    c = torch.stack((codes >> 4, codes & 15), 1).reshape(-1).long()
    table = torch.tensor(mags + [-m for m in mags], dtype=torch.float64, device=codes.device)
    return (table[c].view(-1, 64) * (absmax.double() / S)[:, None]).view(rows, cols)


def inputs(M, rows, cols, seed, x_std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    X = (torch.randn(M, cols, generator=g, device="cuda") * x_std).to(torch.bfloat16)
    codes = torch.randint(0, 256, (rows * cols // 2,), generator=g, device="cuda", dtype=torch.uint8)
    absmax = 0.05 * torch.exp(0.5 * torch.randn(rows * cols // 64, generator=g, device="cuda"))
    return X, codes, absmax


def check(Y, X, codes, absmax, rows, fmt):
    assert q.qlora_get_device_status() == q.QLORA_OK
    W = weight64(codes, absmax, rows, X.shape[1], fmt)
    X64 = X.double()
    ref, size = X64 @ W.t(), X64.abs() @ W.abs().t()
    blocks = X.shape[1] // 64
    tol = torch.finfo(Y.dtype).eps / 2 * ref.abs() * (1 + 2.0 ** -10) + (2.0 ** -16 + (blocks + 32) * 2.0 ** -24) * size
    bad = (Y.double() - ref).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, worst {float(((Y.double() - ref).abs() / tol.clamp_min(1e-300)).max()):.2f}"


# tokens 1..17 (a second group of sixteen), rows off the 16-row tile, odd block counts, one slice and
# less, tiles side by side (cols <= 2048), clusters along the row, several passes (cols > 32768)
SHAPES = [(1, 1, 64), (1, 16, 256), (3, 17, 128), (2, 33, 192), (8, 40, 320), (9, 31, 512), (5, 250, 1024), (16, 100, 2048),
          (17, 47, 2112), (4, 300, 4096), (7, 64, 4160), (1, 5000, 448), (12, 90, 8192), (3, 130, 11008), (2, 24, 33024),
          (16, 600, 33088), (1, 20000, 256), (33, 70, 704)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,rows,cols", SHAPES)
def test_against_64_bits(fmt, M, rows, cols):
    X, codes, absmax = inputs(M, rows, cols, seed=M * 7 + rows)
    for dt in (torch.float32, torch.bfloat16):
        Y = q.qlora_fmt4_linear_fwd(X, codes, absmax, rows, fmt, out_dtype=dt)
        assert Y.shape == (M, rows) and Y.dtype == dt
        check(Y, X, codes, absmax, rows, fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_every_code(fmt):
    # one weight at a time: X picks input k of row k of a weight whose rows hold each code in turn
    rows, cols = 64, 64
    code = (torch.arange(rows, device="cuda")[:, None] + torch.arange(cols, device="cuda")[None, :]) % 16
    codes = ((code[:, 0::2] << 4) | code[:, 1::2]).to(torch.uint8).reshape(-1).contiguous()
    absmax = torch.full((rows,), F.FORMATS[fmt][0], device="cuda")
    X = torch.eye(64, device="cuda", dtype=torch.bfloat16)
    Y = q.qlora_fmt4_linear_fwd(X, codes, absmax, rows, fmt, out_dtype=torch.float32)
    W = weight64(codes, absmax, rows, cols, fmt)
    # one rounding of the constant's factor 1 / S at most
    assert ((Y.double() - W.t()).abs() <= 2.0 ** -22 * W.t().abs()).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1e12, 1e30])
def test_magnitudes(fmt, scale):
    # far from fp16's range, and one token large where another is small
    X, codes, absmax = inputs(4, 48, 512, seed=11, x_std=scale)
    X[1] *= 1e-4
    X[2, ::7] *= 300.0
    X[3] = 0
    Y = q.qlora_fmt4_linear_fwd(X, codes, absmax, 48, fmt, out_dtype=torch.float32)
    check(Y, X, codes, absmax, 48, fmt)
    assert (Y[3] == 0).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_nan_and_infinity(fmt):
    X, codes, absmax = inputs(5, 40, 512, seed=3)
    X[1, 300] = float("nan")
    X[2, 5] = float("inf")
    X[3, 70] = float("-inf")
    absmax[8 * 7 + 2] = float("inf")                     # row 7, block 2
    absmax[8 * 9 + 1] = 0.0
    Y = q.qlora_fmt4_linear_fwd(X, codes, absmax, 40, fmt, out_dtype=torch.float32)
    # the formula: a block's constant times its sum (an infinite constant meets the sum, not each weight)
    v = weight64(codes, torch.full_like(absmax, F.FORMATS[fmt][0]), 40, 512, fmt).view(40, 8, 64)
    dots = torch.einsum("mbk,rbk->mrb", X.double().view(5, 8, 64), v)
    ref = (dots * (absmax.double() / F.FORMATS[fmt][0]).view(1, 40, 8)).sum(2)
    assert torch.equal(torch.isnan(Y), torch.isnan(ref))
    assert torch.equal(torch.isposinf(Y), torch.isposinf(ref)) and torch.equal(torch.isneginf(Y), torch.isneginf(ref))
    fin = torch.isfinite(ref)
    assert fin[0].sum() == 39 and ((Y.double() - ref)[fin].abs() <= 1e-4 * ref[fin].abs().max()).all()


def test_strides_alignment_and_guards():
    # a strided X, constants that start on 4 bytes only, outputs inside a larger buffer left as it was
    M, rows, cols = 3, 50, 1024
    X, codes, absmax = inputs(M, rows, cols, seed=5)
    wide = torch.zeros(M, 2 * cols, dtype=torch.bfloat16, device="cuda")
    wide[:, ::2] = X
    odd = torch.empty(absmax.numel() + 1, device="cuda")[1:]
    odd.copy_(absmax)
    assert odd.data_ptr() % 16 == 4
    for dt in (torch.float32, torch.bfloat16):
        buf = torch.full((M * rows + 32,), 7.0, dtype=dt, device="cuda")
        Y = buf[16:16 + M * rows].view(M, rows)
        out = q.qlora_fmt4_linear_fwd(wide[:, ::2], codes, odd, rows, "fp4_e2m1", Y=Y)
        assert out.data_ptr() == Y.data_ptr()
        check(Y, X, codes, absmax, rows, "fp4_e2m1")
        assert (buf[:16] == 7).all() and (buf[16 + M * rows:] == 7).all()


def test_repeatable_streams_and_graph():
    M, rows, cols = 6, 700, 8192
    X, codes, absmax = inputs(M, rows, cols, seed=8)
    Y = q.qlora_fmt4_linear_fwd(X, codes, absmax, rows, "int4", out_dtype=torch.float32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = q.qlora_fmt4_linear_fwd(X, codes, absmax, rows, "int4", out_dtype=torch.float32, stream=s)
    s.synchronize()
    assert torch.equal(Y, other)
    # captured twice in a row (the second call reads the first's output), replayed with new inputs
    codes2 = torch.randint(0, 256, (64 * 704 // 2,), device="cuda", dtype=torch.uint8)
    absmax2 = torch.rand(64 * 704 // 64, device="cuda")
    Xs, Yb = X.clone(), torch.empty(M, 704, dtype=torch.bfloat16, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        Y1 = q.qlora_fmt4_linear_fwd(Xs, codes, absmax, rows, "int4", out_dtype=torch.bfloat16)
        Yb.zero_()
        Yb[:, :rows] = Y1
        Y2 = q.qlora_fmt4_linear_fwd(Yb, codes2, absmax2, 64, "fp4_e3m0", out_dtype=torch.float32)
    for seed in (21, 22):
        Xs.copy_(inputs(M, rows, cols, seed)[0])
        g.replay()
        torch.cuda.synchronize()
        check(Y1, Xs, codes, absmax, rows, "int4")
        check(Y2, Yb, codes2, absmax2, 64, "fp4_e3m0")


@pytest.mark.parametrize("fmt", FMTS)
def test_quantised_weight(fmt):
    # with the formats' own entry points: the dequantised bf16 weight differs by its rounding only
    rows, cols = 96, 512
    W = torch.randn(rows, cols, device="cuda") * 0.02
    X = torch.randn(4, cols, device="cuda").to(torch.bfloat16)
    codes, absmax = q.qlora_fmt4_quantize(W, fmt)
    Y = q.qlora_fmt4_linear_fwd(X, codes, absmax, rows, fmt, out_dtype=torch.float32)
    check(Y, X, codes, absmax, rows, fmt)
    Wb = q.qlora_fmt4_dequant(codes, absmax, rows * cols, fmt).view(rows, cols).double()
    assert ((Y.double() - X.double() @ Wb.t()).abs() <= 2.0 ** -8 * 1.01 * (X.double().abs() @ Wb.abs().t())).all()


def test_large_offsets():
    # codes past 2^31 bytes: the last rows of a weight of 2^32 + weights
    cols, rows = 32768, 131072 + 48
    codes = torch.zeros(rows * cols // 2, dtype=torch.uint8, device="cuda")
    absmax = torch.zeros(rows * cols // 64, device="cuda")
    tail = 64
    codes[-tail * cols // 2:] = torch.randint(0, 256, (tail * cols // 2,), device="cuda", dtype=torch.uint8)
    absmax[-tail * cols // 64:] = 0.05
    X = torch.randn(1, cols, device="cuda").to(torch.bfloat16)
    Y = q.qlora_fmt4_linear_fwd(X, codes, absmax, rows, "int4", out_dtype=torch.float32)
    assert (Y[:, :-tail] == 0).all()
    check(Y[:, -tail:].contiguous(), X, codes[-tail * cols // 2:], absmax[-tail * cols // 64:], tail, "int4")


def test_output_of_another_stream_is_not_reused():
    # torch allocates Y on the current stream; dropped while the other stream still writes it, its block must not be
    # handed out again
    M, rows, cols = 5, 997, 512
    X, codes, absmax = inputs(M, rows, cols, seed=17)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
    Y = q.qlora_fmt4_linear_fwd(X, codes, absmax, rows, "int4", stream=s)
    used = Y.data_ptr()
    del Y
    fresh = torch.empty(M, rows, dtype=torch.bfloat16, device="cuda")
    assert fresh.data_ptr() != used
    s.synchronize()


# clusters with more tiles than a segment holds, an odd number of them, and a last tile of four rows
@pytest.mark.parametrize("M,rows,cols", [(2, 38500, 4352), (10, 19508, 4352), (1, 38500, 4160)])
def test_several_segments(M, rows, cols):
    X, codes, absmax = inputs(M, rows, cols, seed=M)
    Y = q.qlora_fmt4_linear_fwd(X, codes, absmax, rows, "fp4_e2m1", out_dtype=torch.float32)
    check(Y, X, codes, absmax, rows, "fp4_e2m1")


def test_timed_launches_give_the_same():
    # the profiling hooks launch without the overlap of neighbouring kernels
    X, codes, absmax = inputs(4, 300, 4096, seed=23)
    first = q.qlora_fmt4_linear_fwd(X, codes, absmax, 300, "int4")
    q.qlora_profile_enable(True)
    try:
        timed = q.qlora_fmt4_linear_fwd(X, codes, absmax, 300, "int4")
        torch.cuda.synchronize()
    finally:
        q.qlora_profile_enable(False)
    assert torch.equal(first, timed)


# Int4 with work for every CTA, which takes the codes from a table: one CTA or a cluster along the row, constants that do
# or do not start on 16 bytes, tiles side by side
@pytest.mark.parametrize("M,rows,cols", [(1, 2400, 4096), (8, 2500, 4032), (3, 1300, 4160), (5, 1250, 8192), (2, 20011, 1024)])
def test_int4_table(M, rows, cols):
    X, codes, absmax = inputs(M, rows, cols, seed=M + rows)
    Y = q.qlora_fmt4_linear_fwd(X, codes, absmax, rows, "int4", out_dtype=torch.float32)
    check(Y, X, codes, absmax, rows, "int4")
    # one input after the other: every code of a row by itself, and its constant's sign
    X1 = torch.zeros(M, cols, dtype=torch.bfloat16, device="cuda")
    X1[:, 7] = 1e30
    X1[:, cols - 3] = -1e-30
    check(q.qlora_fmt4_linear_fwd(X1, codes, -absmax, rows, "int4", out_dtype=torch.float32), X1, codes, -absmax, rows, "int4")
