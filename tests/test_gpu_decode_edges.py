"""GPU tests of what the decode-time products (qlora_fmt4_linear_fwd, qlora_moe_fwd) do at their
edges: waits that run out, the ends of the fp32 range, calls on another stream, refusals."""
import pytest
import torch

import bit_nf4_quantized_double_b200 as q
from oracle import formats as F

pytestmark = pytest.mark.gpu


def test_a_warps_wait_has_one_answer():
    # 24 waits that complete, 24 that are aborted, 48 that get both at nearly the same time, one that runs into its limit
    assert q.qlora_get_device_status() == q.QLORA_OK
    out = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    assert q.lib().qlora_selftest_wait_warp(out.data_ptr(), None) == q.QLORA_OK
    assert q.qlora_get_device_status() == q.QLORA_ERR_TIMEOUT
    split, wrong, gave_up, waits = out.tolist()
    assert split == 0 and wrong == 0 and waits == 97
    assert 25 <= gave_up <= 73


# Int4 takes its codes from a table for few tokens and many rows, by bit placement else
@pytest.mark.parametrize("fmt", ["int4", "fp4_e2m1", "fp4_e3m0"])
@pytest.mark.parametrize("M,rows", [(5, 40), (12, 40), (7, 4800)])
@pytest.mark.parametrize("ec,ex", [(63, 64), (-60, -66), (99, 28), (-100, 60), (40, -166)])
def test_ends_of_the_range(fmt, M, rows, ec, ex):
    # one input per token, so that Y = v c x / S: results up to 3.2e38 and down to subnormals, far constants and far tokens.
    # Roundings: the constant's product, the token's power of two (a half step if subnormal), 1 / S and its product; bf16's own
    S, mags = F.FORMATS[fmt]
    cols = 2048
    g = torch.Generator(device="cuda").manual_seed(M + rows + ec)
    X = torch.zeros(M, cols, dtype=torch.float64, device="cuda")
    at = torch.randint(0, cols, (M,), generator=g, device="cuda")
    sign = torch.randint(0, 2, (M,), generator=g, device="cuda").double() * 2 - 1
    top = max(ex, -126)
    X[torch.arange(M), at] = sign * 2.0 ** top
    codes = torch.randint(0, 256, (rows * cols // 2,), generator=g, device="cuda", dtype=torch.uint8)
    absmax = (1 + 0.9 * torch.rand(rows * cols // 64, generator=g, device="cuda")) * 2.0 ** (ec + ex - top)
    c = torch.stack((codes >> 4, codes & 15), 1).reshape(-1).long()
    table = torch.tensor(mags + [-m for m in mags], dtype=torch.float64, device="cuda")
    W = (table[c].view(-1, 64) * (absmax.double() / S)[:, None]).view(rows, cols)
    ref = X @ W.t()
    for dt in (torch.float32, torch.bfloat16):
        Y = q.qlora_fmt4_linear_fwd(X.to(torch.bfloat16), codes, absmax, rows, fmt, out_dtype=dt).double()
        tol = 2.0 ** -22 * ref.abs() + 2 * 2.0 ** -149
        if dt == torch.bfloat16:
            tol += 2.0 ** -8 * 1.001 * ref.abs() + 2.0 ** -134
        assert torch.isfinite(Y).all() and ((Y - ref).abs() <= tol).all()
    assert q.qlora_get_device_status() == q.QLORA_OK


def strided(t):
    """The same values in every second column of a wider tensor."""
    wide = torch.zeros(t.shape[0], 2 * t.shape[1], dtype=t.dtype, device=t.device)
    wide[:, ::2] = t
    return wide[:, ::2]


def test_strided_inputs_on_another_stream():
    # the copies that a call makes run where its kernels do, not behind what the current stream is busy with
    g = torch.Generator(device="cuda").manual_seed(5)
    M, rows, cols = 4, 320, 512
    X = torch.randn(M, cols, generator=g, device="cuda").to(torch.bfloat16)
    W = torch.randn(rows, cols, generator=g, device="cuda") * 0.02
    router = torch.randn(4, cols, generator=g, device="cuda")
    codes, absmax = q.qlora_fmt4_quantize(W, "int4")
    nf4 = q.qlora_nf4_quantize(W)
    gate, up = (q.qlora_nf4_quantize(torch.randn(4 * 64, cols, generator=g, device="cuda")) for _ in range(2))
    down = q.qlora_nf4_quantize(torch.randn(4 * cols, 64, generator=g, device="cuda"))
    Xs, Ws, rs = strided(X), strided(W), strided(router)

    def calls(X, W, router, stream):
        out = [q.qlora_fmt4_linear_fwd(X, codes, absmax, rows, "int4", stream=stream)]
        out += q.qlora_moe_fwd(X, router, gate, up, down, 2, stream=stream)
        out += q.qlora_fmt4_quantize(W, "int4", stream=stream)
        for t in (q.qlora_nf4_quantize(W, stream=stream), *q.qlora_nf4_quantize_grouped([W], stream=stream)):
            out += [t.codes, t.scale8, t.scale2, t.offset]
        return out

    want = calls(X, W, router, None)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    got = calls(Xs, Ws, rs, s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, [t.clone() for t in got]))
    assert torch.equal(nf4.codes, got[-4])


# one CTA along the row, clusters of short rows (made while there are fewer tiles than SMs) and of long ones, tiles side by
# side, the table and bit placement
@pytest.mark.parametrize("fmt", ["int4", "fp4_e2m1", "fp4_e3m0"])
@pytest.mark.parametrize("M,rows,cols", [(3, 1000, 256), (8, 300, 4096), (7, 640, 4160), (16, 500, 2048), (12, 600, 8192),
                                         (4, 2600, 4096), (2, 5000, 2048), (2, 300, 33024)])
def test_norm_of_the_error(fmt, M, rows, cols):
    # per token, over the rows. mma cuts its 17 terms to 24 bits at the largest (about three times their rms): 2^-24 6 / 4 =
    # 9e-8 of the norm; at most 4 + 15 + 7 additions after one another, each 2^-25 of a partial sum: 2^-25 sqrt(26 / 2) =
    # 1.1e-7; token's power of two none, 1 / S and its product 2^-24 each: 8e-8. Together 1.7e-7, three times that allowed
    S, mags = F.FORMATS[fmt]
    g = torch.Generator(device="cuda").manual_seed(rows)
    X = torch.randn(M, cols, generator=g, device="cuda").to(torch.bfloat16)
    codes = torch.randint(0, 256, (rows * cols // 2,), generator=g, device="cuda", dtype=torch.uint8)
    absmax = 0.05 * torch.exp(0.5 * torch.randn(rows * cols // 64, generator=g, device="cuda"))
    c = torch.stack((codes >> 4, codes & 15), 1).reshape(-1).long()
    table = torch.tensor(mags + [-m for m in mags], dtype=torch.float64, device="cuda")
    y = X.double() @ (table[c].view(-1, 64) * (absmax.double() / S)[:, None]).view(rows, cols).t()
    Y = q.qlora_fmt4_linear_fwd(X, codes, absmax, rows, fmt, out_dtype=torch.float32)
    assert q.qlora_get_device_status() == q.QLORA_OK
    assert ((Y.double() - y).norm(dim=1) <= 5e-7 * y.norm(dim=1)).all()


def test_a_strided_vector_is_quantised_by_its_values():
    W = torch.randn(2 * 16421, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    want = q.qlora_nf4_quantize(W[::2].clone())
    for got in (q.qlora_nf4_quantize(W[::2]), *q.qlora_nf4_quantize_grouped([W[::2]])):
        assert all(torch.equal(getattr(want, n), getattr(got, n)) for n in ("codes", "scale8", "scale2", "offset"))
