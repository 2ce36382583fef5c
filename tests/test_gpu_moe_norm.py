"""qlora_moe_fwd against the formula in 64 bits, by the norm of a token's output: the elementwise
bound of test_gpu_moe.py adds up absolute values through two products and is as large as the output
itself for wide layers, where a lost block would pass.

Tolerance: ||Y - y|| <= 4e-3 ||y|| for every token. Y's rounding to bf16 is uniform within half a step
2^(e - 8) of values in [2^e, 2^(e + 1)): at most 2^-7 / sqrt(12) = 2.3e-3 of the norm, and a quarter more
as four deviations of a sum over 64 outputs: 2.8e-3. The codebook and the hidden values are
fp16, 2^-11 / sqrt(3) = 2.8e-4 of the norm each and independent: gate and up (times at most 1.5 through
silu, whose relative slope is near 1), hidden values and down: 7e-4 together. fp32 sums: below 1e-5.
"""
import pytest
import torch

import bit_nf4_quantized_double_b200 as q
from test_gpu_moe import SHAPES, dense, layer

LIMIT = 4e-3


def norm_error(Y, y):
    """The largest ||Y - y|| / ||y|| of a token."""
    return float(((Y.double() - y).norm(dim=1) / y.norm(dim=1)).max())


def exact(X, router, gate, up, down, k, renorm=True):
    E, d, f = router.shape[0], X.shape[1], down.cols
    X64 = X.double()
    logits = X64 @ router.double().t()
    order = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
    p = torch.softmax(logits, 1).gather(1, order)
    if renorm:
        p = p / p.sum(1, keepdim=True)
    G, U, D = dense(gate).view(E, f, d), dense(up).view(E, f, d), dense(down).view(E, d, f)
    y = torch.zeros_like(X64)
    for e in order.unique().tolist():
        tok, slot = torch.nonzero(order == e, as_tuple=True)
        a, b = X64[tok] @ G[e].t(), X64[tok] @ U[e].t()
        y.index_add_(0, tok, p[tok, slot][:, None] * ((a / (1 + torch.exp(-a)) * b) @ D[e].t()))
    return y, order.to(torch.int32)


def check(a, k, renorm=True):
    Y, experts, _ = q.qlora_moe_fwd(*a, k, renorm=renorm)
    assert q.qlora_get_device_status() == q.QLORA_OK
    y, order = exact(*a, k, renorm)
    assert torch.equal(experts, order)
    assert norm_error(Y, y) <= LIMIT


def test_the_limit_tells_errors_from_roundings():
    y = torch.randn(64, 64, generator=torch.Generator().manual_seed(1), dtype=torch.float64)
    assert norm_error(y.to(torch.bfloat16), y) <= LIMIT - 7e-4
    for wrong in (1.01 * y, y * (torch.arange(64) != 63), y.roll(1, 0)):
        assert norm_error(wrong.to(torch.bfloat16), y) > LIMIT


@pytest.mark.gpu
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,d,f,E,k", SHAPES + [(1, 65536, 64, 2, 1), (3, 64, 65536, 1, 1), (64, 128, 128, 1, 1),
                                                (64, 256, 64, 2, 2), (32, 4160, 4224, 4, 2)])
def test_norm(T, d, f, E, k, renorm):
    check(layer(T, d, f, E, seed=T + d + f + E, rdt=torch.bfloat16 if renorm else torch.float32), k, renorm)


def ends(n):
    """Blocks of 64 of a row of n values at the ends of its slices of 256, chunks of 16 slices or the even shares that the
    kernel makes of them, and of the row."""
    blocks, slices = n // 64, -(-n // 256)
    chunks = -(-slices // 16)
    at = {0, blocks - 1}
    for c in range(chunks):
        first = c * (slices // chunks) + min(c, slices % chunks)
        at |= {4 * first - 1, 4 * first, 4 * first + 3}
    return sorted(b for b in at if 0 <= b < blocks)


# more than one chunk of either width, with odd block counts and a last slice of one to four blocks
WIDE = [(2, 4352, 256, 3, 2), (4, 8192, 128, 2, 1), (3, 4160, 192, 2, 2), (1, 12480, 64, 2, 1), (9, 1088, 64, 3, 2)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,d,f,E,k", WIDE)
def test_inputs_of_one_block(T, d, f, E, k):
    a = layer(T, d, f, E, seed=d)
    X = a[0].clone()
    for b in ends(d):
        a[0].zero_()
        a[0][:, 64 * b:64 * b + 64] = X[:, 64 * b:64 * b + 64]
        check(a, k)


@pytest.mark.gpu
@pytest.mark.parametrize("T,f,d,E,k", WIDE)
def test_hidden_values_of_one_block(T, f, d, E, k):
    # the up product's constants are zero but for the rows of one block of hidden values
    a = layer(T, d, f, E, seed=f)
    up, scale8 = a[3], a[3].scale8.clone().view(E, f, d // 64)
    up.offset.zero_()
    scale8[scale8 == 0] = 1
    for b in ends(f):
        up.scale8.zero_()
        up.scale8.view(E, f, d // 64)[:, 64 * b:64 * b + 64] = scale8[:, 64 * b:64 * b + 64]
        check(a, k)


@pytest.mark.gpu
def test_large_and_small_activations():
    for scale in (1e-3, 64.0):
        a = layer(3, 4352, 320, 6, seed=4)
        a[0].mul_(scale)
        a[0][1, 17] = 40.0 * scale
        check(a, 2)
