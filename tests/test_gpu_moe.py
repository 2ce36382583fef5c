"""GPU tests of qlora_moe_fwd: the mixture-of-experts layer with NF4 experts against the formula
in 64 bits.

Choices have to be equal. Weights: fp32 rounding and that of exp, 8 2^-24 relative, and a step of
2^-149 where a softmax value of less than 2^-126 leaves fp32's normal range. Outputs,
element by element and to first order, with u = 2^-11 (half a step of fp16) and all sums over
absolute values:
  * the codebook in fp16: u sum |G| |x| on g, the same on the up product, u sum |D| |h| on y;
  * |silu'| <= 1.1, so h is off by 1.1 dg |up| + |silu| dup, and by u |h| for its own rounding;
  * fp32 sums, constants and the inner cuts of mma: 2^-14 of each sum covers 4 mma a block and up
    to 1024 blocks (2^-16 + 1056 2^-24);
  * Y's rounding: 2^-8 |y|. Second-order terms: a factor of 1.05.
"""
import pytest
import torch

import bit_nf4_quantized_double_b200 as q

pytestmark = pytest.mark.gpu


def random_tensor(rows, cols, g):
    n = rows * cols
    nb = n // 64
    t = q.nf4_empty(rows, cols)
    t.codes.copy_(torch.randint(0, 256, (n // 2,), generator=g, device="cuda", dtype=torch.uint8))
    t.scale8.copy_((torch.randn(nb, generator=g, device="cuda") * 40).clamp(-127, 127).round().to(torch.int8))
    t.scale2.copy_(0.02 + 0.02 * torch.rand(t.scale2.numel(), generator=g, device="cuda"))
    t.offset.fill_(0.05)
    return t


def dense(t):
    """fp64 weight of a stored tensor, not rounded to bf16."""
    table = torch.tensor(q.qlora_nf4_codebook(), dtype=torch.float64, device="cuda")
    w = table[torch.stack((t.codes >> 4, t.codes & 15), 1).reshape(-1).long()]
    step = (t.scale2.double() / 127).repeat_interleave(256)[:t.scale8.numel()]
    return (w.view(-1, 64) * (t.scale8.double() * step + t.offset.double())[:, None]).view(t.rows, t.cols)


def layer(T, d, f, E, seed, rdt=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    X = torch.randn(T, d, generator=g, device="cuda").to(torch.bfloat16)
    router = (torch.randn(E, d, generator=g, device="cuda") / d ** 0.5).to(rdt)
    return X, router, random_tensor(E * f, d, g), random_tensor(E * f, d, g), random_tensor(E * d, f, g)


def reference(X, router, gate, up, down, k, renorm):
    """(y, tolerance of y, experts, weights) in 64 bits."""
    E, d, f = router.shape[0], X.shape[1], down.cols
    X64 = X.double()
    logits = X64 @ router.double().t()
    order = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
    p = torch.softmax(logits, 1).gather(1, order)
    if renorm:
        p = p / p.sum(1, keepdim=True)
    G, U, D = dense(gate).view(E, f, d), dense(up).view(E, f, d), dense(down).view(E, d, f)
    y, tol = torch.zeros_like(X64), torch.zeros_like(X64)
    u, s = 2.0 ** -11, 2.0 ** -14
    for e in order.unique().tolist():
        tok, slot = torch.nonzero(order == e, as_tuple=True)
        x, w = X64[tok], p[tok, slot][:, None]
        a, b = x @ G[e].t(), x @ U[e].t()
        da, db = (u + s) * (x.abs() @ G[e].abs().t()), (u + s) * (x.abs() @ U[e].abs().t())
        h = torch.nn.functional.silu(a) * b
        dh = 1.1 * da * (b.abs() + db) + torch.nn.functional.silu(a).abs() * db + (u + 2.0 ** -20) * h.abs()
        y.index_add_(0, tok, w * (h @ D[e].t()))
        tol.index_add_(0, tok, w.abs() * (dh @ D[e].abs().t() + (u + s) * (h.abs() @ D[e].abs().t())))
    return y, 1.05 * tol + 2.0 ** -8 * (y.abs() + tol), order.to(torch.int32), p


def check(out, ref):
    Y, experts, weights = out
    y, tol, order, p = ref
    assert q.qlora_get_device_status() == q.QLORA_OK
    assert torch.equal(experts, order)
    assert ((weights.double() - p).abs() <= 8 * 2.0 ** -24 * p + 2.0 ** -149).all()
    err = (Y.double() - y).abs()
    assert (err <= tol).all(), float((err / tol.clamp_min(1e-300)).max())


# one block to several chunks of either width, odd block counts, tiles side by side, one token to more
# than a job's eight per expert, one expert, all experts, many experts
SHAPES = [(1, 64, 64, 1, 1), (2, 128, 192, 4, 2), (5, 256, 320, 7, 3), (1, 2048, 512, 32, 8), (7, 1088, 704, 13, 3),
          (20, 512, 256, 4, 4), (64, 320, 448, 16, 8), (17, 4096, 512, 2, 1), (4, 8192, 1024, 3, 2), (2, 4352, 4352, 3, 2),
          (40, 576, 128, 256, 16), (64, 64, 64, 64, 16), (33, 192, 576, 3, 1), (9, 128, 8256, 5, 2)]


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,d,f,E,k", SHAPES)
def test_against_64_bits(T, d, f, E, k, renorm):
    a = layer(T, d, f, E, seed=T + d + f, rdt=torch.float32 if renorm else torch.bfloat16)
    check(q.qlora_moe_fwd(*a, k, renorm=renorm), reference(*a, k, renorm))


def test_ties_go_to_the_lower_expert():
    a = layer(6, 256, 64, 12, seed=1)
    a[1][3] = a[1][1]
    a[1][7] = a[1][1]
    a[1][8:] = 0
    a[0][2] = 0                                           # every logit of token 2 is zero
    out = q.qlora_moe_fwd(*a, 5)
    check(out, reference(*a, 5, True))
    assert out[1][2].tolist() == [0, 1, 2, 3, 4]


def test_close_logits():
    # neighbours 2^-40 apart: fp32 sums would order them by chance
    T, d, E = 4, 512, 16
    a = layer(T, d, 64, E, seed=2)
    a[1][:] = a[1][0]
    a[0][:, 0] = 1.0
    a[1][:, 0] = torch.tensor([2.0 ** -30 * ((5 * e) % E) for e in range(E)], device="cuda")
    out = q.qlora_moe_fwd(*a, 4)
    check(out, reference(*a, 4, True))


def test_large_and_small_activations():
    for scale in (1e-3, 64.0):
        a = layer(3, 512, 256, 6, seed=4)
        a[0].mul_(scale)
        a[0][1, 17] = 40.0 * scale
        check(q.qlora_moe_fwd(*a, 2), reference(*a, 2, True))


def test_nan_and_infinity_stay_in_their_token():
    a = layer(5, 256, 128, 8, seed=6)
    clean = q.qlora_moe_fwd(*a, 2)
    a[0][1, 9] = float("nan")
    a[0][3, 200] = float("inf")
    Y, experts, weights = q.qlora_moe_fwd(*a, 2)
    assert q.qlora_get_device_status() == q.QLORA_OK
    assert experts[1].tolist() == [0, 1] and torch.isnan(Y[1]).all() and torch.isnan(weights[1]).all()
    assert ((experts >= 0) & (experts < 8)).all() and not torch.isfinite(Y[3]).any()
    keep = [0, 2, 4]
    assert torch.equal(Y[keep], clean[0][keep]) and torch.equal(experts[keep], clean[1][keep])


def test_outputs_and_guards():
    T, d, k = 3, 128, 2
    a = layer(T, d, 64, 4, seed=7)
    buf = torch.full((T * d + 64,), 3.0, dtype=torch.bfloat16, device="cuda")
    Y = buf[32:32 + T * d].view(T, d)
    ws = torch.full((q.qlora_moe_fwd_workspace(T, d, 64, 4, k) + 256,), 255, dtype=torch.uint8, device="cuda")
    need = ws.numel() - 256
    out = q.qlora_moe_fwd(*a, k, Y=Y, ws=ws[:need])
    assert out[0].data_ptr() == Y.data_ptr()
    check(out, reference(*a, k, True))
    assert (buf[:32] == 3).all() and (buf[32 + T * d:] == 3).all() and (ws[need:] == 255).all()
    # the choice's outputs are optional in the C ABI
    Y2 = torch.empty_like(Y)
    import ctypes
    t = [w.ctype() for w in a[2:]]
    st = q.lib().qlora_moe_fwd(a[0].data_ptr(), T, a[1].data_ptr(), q.QLORA_F32, 4, ctypes.byref(t[0]), ctypes.byref(t[1]),
                               ctypes.byref(t[2]), k, 1, Y2.data_ptr(), None, None, ws.data_ptr(), need,
                               torch.cuda.current_stream().cuda_stream)
    assert st == q.QLORA_OK
    torch.cuda.synchronize()
    assert torch.equal(Y2, Y)


def test_repeatable_streams_and_graph():
    T, d, f, E, k = 6, 1024, 512, 16, 4
    a = layer(T, d, f, E, seed=9, rdt=torch.bfloat16)
    first = q.qlora_moe_fwd(*a, k)
    again = q.qlora_moe_fwd(*a, k)
    assert all(torch.equal(x, y) for x, y in zip(first, again))
    # two streams at once, a workspace each
    outs = []
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        outs.append([q.qlora_moe_fwd(*a, k, stream=s) for _ in range(5)])
    for s in streams:
        s.synchronize()
    assert all(torch.equal(x, y) for o in outs for r in o for x, y in zip(first, r))
    # captured, replayed with new tokens
    X = a[0].clone()
    ws = torch.empty(q.qlora_moe_fwd_workspace(T, d, f, E, k), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = q.qlora_moe_fwd(X, *a[1:], k, ws=ws)
        out2 = q.qlora_moe_fwd(out[0], *a[1:], k, ws=ws)   # the next layer in the same workspace
    for seed in (31, 32):
        X.copy_(layer(T, d, 64, E, seed)[0])
        g.replay()
        torch.cuda.synchronize()
        check(out, reference(X, *a[1:], k, True))
        check(out2, reference(out[0], *a[1:], k, True))


def test_decode_step_with_quantised_weights():
    # as a decode step uses them: experts quantised as one stacked tensor, the layer, a 4-bit output projection
    T, d, f, E, k, vocab = 4, 256, 384, 6, 2, 500
    g = torch.Generator(device="cuda").manual_seed(12)
    W = [torch.randn(r, c, generator=g, device="cuda") * 0.02 for r, c in ((E * f, d), (E * f, d), (E * d, f), (vocab, d))]
    gate, up, down = (q.qlora_nf4_quantize(w) for w in W[:3])
    codes, absmax = q.qlora_fmt4_quantize(W[3], "fp4_e2m1")
    X = torch.randn(T, d, generator=g, device="cuda").to(torch.bfloat16)
    router = torch.randn(E, d, generator=g, device="cuda") / 16
    out = q.qlora_moe_fwd(X, router, gate, up, down, k)
    logits = q.qlora_fmt4_linear_fwd(out[0], codes, absmax, vocab, "fp4_e2m1", out_dtype=torch.float32)
    ref = reference(X, router, gate, up, down, k, True)
    check(out, ref)
    Wh = q.qlora_fmt4_dequant(codes, absmax, vocab * d, "fp4_e2m1").view(vocab, d).double()
    err = (logits.double() - out[0].double() @ Wh.t()).abs()
    assert (err <= 1.01 * 2.0 ** -8 * (out[0].double().abs() @ Wh.abs().t())).all()
    # the stored experts are those of the layer's own dequantisation, up to its rounding to bf16
    assert ((q.qlora_nf4_dequant(gate).double() - dense(gate)).abs() <= 1.01 * 2.0 ** -8 * dense(gate).abs()).all()


def test_outputs_of_another_stream_are_not_reused():
    # torch allocates the outputs on the current stream; dropped while the other stream still writes them, their
    # blocks must not be handed out again
    T, d, f, E, k = 5, 768, 256, 4, 2
    a = layer(T, d, f, E, seed=15)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
    out = q.qlora_moe_fwd(*a, k, stream=s)
    used = {t.data_ptr() for t in out}
    del out
    fresh = [torch.empty(T, d, dtype=torch.bfloat16, device="cuda"), torch.empty(T, k, device="cuda"),
             torch.empty(T, k, device="cuda")]
    assert not used & {t.data_ptr() for t in fresh}
    s.synchronize()


# the widest layer either way (16 chunks of D, of F), every token at one expert (eight full jobs), all of two
@pytest.mark.parametrize("T,d,f,E,k", [(1, 65536, 64, 2, 1), (3, 64, 65536, 1, 1), (64, 128, 128, 1, 1), (64, 256, 64, 2, 2)])
def test_extremes(T, d, f, E, k):
    a = layer(T, d, f, E, seed=T + E)
    check(q.qlora_moe_fwd(*a, k), reference(*a, k, True))


def test_timed_launches_give_the_same():
    # the profiling hooks launch without the overlap of neighbouring kernels
    a = layer(5, 512, 320, 8, seed=19)
    first = q.qlora_moe_fwd(*a, 3)
    q.qlora_profile_enable(True)
    try:
        timed = q.qlora_moe_fwd(*a, 3)
        torch.cuda.synchronize()
    finally:
        q.qlora_profile_enable(False)
    assert all(torch.equal(x, y) for x, y in zip(first, timed))
    check(timed, reference(*a, 3, True))


def test_two_graphs_and_a_product_at_once():
    # replays on two streams, each with its own workspace, and the 4-bit product on a third: a layer that waits for its
    # CTAs shares the chip with the others
    T, d, f, E, k = 8, 1024, 512, 16, 4
    a = layer(T, d, f, E, seed=25)
    first = q.qlora_moe_fwd(*a, k)
    W = torch.randn(4096, d, device="cuda") * 0.02
    codes, absmax = q.qlora_fmt4_quantize(W, "int4")
    Y = q.qlora_fmt4_linear_fwd(a[0], codes, absmax, 4096, "int4")
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        ws = torch.empty(q.qlora_moe_fwd_workspace(T, d, f, E, k), dtype=torch.uint8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = [q.qlora_moe_fwd(*a, k, ws=ws) for _ in range(4)]
        graphs.append((g, outs, ws, torch.cuda.Stream()))
    third = torch.cuda.Stream()
    products = []
    for _ in range(5):
        for g, _, _, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(third):
            products += [q.qlora_fmt4_linear_fwd(a[0], codes, absmax, 4096, "int4") for _ in range(4)]
    torch.cuda.synchronize()
    assert q.qlora_get_device_status() == q.QLORA_OK
    assert all(torch.equal(x, y) for _, outs, _, _ in graphs for o in outs for x, y in zip(first, o))
    assert all(torch.equal(Y, p) for p in products)
