"""8-bit quantisation and products against the fp64 oracle.

Quantisation is exact: scales and e4m3 values must be equal. A product of e4m3 values is exact
in fp32; with S = sum over k of |sa a sb b|, a sum of 128 of them inside one block and of the
blocks after it rounds at most 128 + blocks times by one unit of 2^-23 of at most S (2^-23, not
half of it: the tensor core may cut instead of rounding), the two scales and their products by
3 * 2^-24 each: |error| <= (128 + blocks + 4) 2^-23 S, and the output's own rounding (half a step)."""
import numpy as np
import pytest
import torch

import linear_cross_entropy_chunked_gb300 as lce
from oracle import ops_oracle

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def rand(r, c, seed, dtype="bf16", spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(r, c, generator=g) * torch.exp(spread * torch.randn(r, 1, generator=g))
    return (x * torch.exp(spread * torch.randn(1, c, generator=g))).to(DTYPES[dtype])


def same(got, want):
    np.testing.assert_array_equal(got, want)


def check_quantized(pair, X64, tiles):
    q, scale = pair
    wq, ws = ops_oracle.quantize_fp8(X64, tiles)
    assert q.dtype == torch.float8_e4m3fn and q.shape == X64.shape and q.stride(0) % 16 == 0
    same(scale.double().cpu().numpy(), ws)
    same(q.float().double().cpu().numpy(), wq)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("r,c", [(1, 1), (1, 128), (2, 130), (5, 7), (127, 129), (128, 128), (129, 257),
                                 (300, 1000), (1, 4097), (4099, 3)])
def test_quantize(r, c, dtype):
    X = rand(r, c, r * 31 + c, dtype)
    d = X.cuda()
    x64 = X.double().numpy()
    for tiles in (False, True):
        check_quantized(lce.quantize_fp8(d, tiles=tiles), x64, tiles)
        check_quantized(lce.quantize_fp8(d, tiles=tiles, transpose=True), x64.T, tiles)
    w = lce.fp8_weight(d)
    check_quantized((w.q, w.scale), x64, True)
    check_quantized((w.q_t, w.scale_t), x64.T, True)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_quantize_strides(dtype):
    wide = rand(70, 700, 3, dtype).cuda()
    for at in (0, 1, 5, 8):
        v = wide[::2, at:at + 333]
        for tiles in (False, True):
            check_quantized(lce.quantize_fp8(v, tiles=tiles), v.double().cpu().numpy(), tiles)
            check_quantized(lce.quantize_fp8(v, tiles=tiles, transpose=True), v.double().cpu().numpy().T, tiles)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("r,c", [(128, 128), (256, 129), (300, 1001), (129, 263), (384, 392)])
def test_quantize_rows_that_start_anywhere(r, c, dtype):
    # every offset of a row's start within 16 bytes, and rows that begin and end with the memory
    for extra in range(0, 9):
        flat = torch.randn(r * (c + extra) + 8, generator=torch.Generator().manual_seed(extra)).to(DTYPES[dtype]).cuda()
        for at in (0, 1, 5):
            v = flat[at:at + r * (c + extra)].view(r, c + extra)[:, extra:] if extra else flat[at:at + r * c].view(r, c)
            check_quantized(lce.quantize_fp8(v), v.double().cpu().numpy(), False)
        check_quantized(lce.quantize_fp8(v, transpose=True), v.double().cpu().numpy().T, False)
        check_quantized(lce.quantize_fp8(v, tiles=True), v.double().cpu().numpy(), True)


@pytest.mark.parametrize("tiles", [False, True])
def test_quantize_special_values(tiles):
    X = torch.randn(260, 400)
    X[0] = 0.0
    X[1, :128] = 1e-44                     # below the smallest scale
    X[2, :128] = 2.0 ** -120
    X[3, 5] = float("inf")
    X[4, 6] = float("nan")
    X[5, :] = float("nan")
    X[6, 7] = 3.4e38
    X[7, :128] = 448.0                     # the border of a scale, and one step beyond
    X[8, :128] = float(np.nextafter(np.float32(448), np.float32(500)))
    X[9, :128] = torch.arange(128) * 3.5   # ties
    X[10, 128:] = -X[9, :128].repeat(3)[:272]
    for m in (X, X.t().contiguous()):
        check_quantized(lce.quantize_fp8(m.cuda(), tiles=tiles), m.double().numpy(), tiles)
        check_quantized(lce.quantize_fp8(m.cuda(), tiles=tiles, transpose=True), m.double().numpy().T, tiles)
    b = X.bfloat16()
    check_quantized(lce.quantize_fp8(b.cuda(), tiles=tiles), b.double().numpy(), tiles)


def operand(r, k, seed, tiles):
    """Random e4m3 values and fp32 scales that are no powers of two."""
    g = torch.Generator().manual_seed(seed)
    ld = -(-k // 16) * 16
    q = (torch.randn(r, ld, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
    s = torch.rand(-(-r // 128) if tiles else r, -(-k // 128), generator=g) + 0.25
    return q.cuda()[:, :k], (s * 10 ** (torch.rand(s.shape, generator=g) * 2 - 1)).cuda()


def full(q, s):
    v = q.float().double()
    s = s.double().repeat_interleave(128, 1)[:, :q.shape[1]]
    return v * (s if s.shape[0] == q.shape[0] else s.repeat_interleave(128, 0)[:q.shape[0]])


def check_product(got, A, B, K):
    want = A @ B.t()
    S = A.abs() @ B.abs().t()
    bound = (128 + -(-K // 128) + 4) * 2.0 ** -23 * S
    if got.dtype != torch.float32:
        bound = bound + torch.finfo(got.dtype).eps / 2 * (want.abs() + bound)
    if got.dtype == torch.float16:
        over = want.abs() > 65504
        assert torch.isinf(got[want.abs() > 65600]).all()
        want, got, bound = want[~over], got[~over], bound[~over]
        bound = bound + 2.0 ** -25
    err = (got.double() - want).abs()
    assert (err <= bound).all(), ((err - bound).max().item(), (err / S.clamp(min=1e-300)).max().item() if got.dtype == torch.float32 else None)


@pytest.mark.parametrize("b_rows", [False, True])
@pytest.mark.parametrize("m,n,k", [
    (1, 1, 1), (1, 7, 16), (1, 128, 128), (3, 129, 200), (8, 64, 127), (9, 1000, 129), (64, 1000, 1000),
    (127, 257, 384), (128, 128, 4096), (1, 4096, 4096), (129, 300, 512), (33, 5000, 640), (16, 20000, 256),
    (256, 256, 256), (300, 33, 8192), (1000, 3000, 100), (1025, 2050, 1300), (2048, 5000, 384),
    (200, 30000, 130), (20000, 300, 96)])
def test_product(m, n, k, b_rows):
    a, sa = operand(m, k, m + k, False)
    b, sb = operand(n, k, n * 3 + k, not b_rows)
    A, B = full(a, sa), full(b, sb)
    for dt in DTYPES.values():
        check_product(lce.fp8_matmul(a, sa, b, sb, out_dtype=dt), A, B, k)


def test_product_repeats_and_status():
    a, sa = operand(700, 2000, 1, False)
    b, sb = operand(6000, 2000, 2, True)
    ws = torch.full((1024,), 255, dtype=torch.uint8, device="cuda")
    first = lce.fp8_matmul(a, sa, b, sb, ws=ws)
    assert lce.read_status(ws) == 0
    for _ in range(3):
        assert torch.equal(first, lce.fp8_matmul(a, sa, b, sb))


@pytest.mark.parametrize("m,n", [(1, 100), (40, 1000), (300, 9001)])
def test_product_leaves_what_lies_beside(m, n):
    a, sa = operand(m, 300, 5, False)
    b, sb = operand(n, 300, 6, True)
    for dt in DTYPES.values():
        wide = torch.full((m + 3, n + 40), 7.0, dtype=dt, device="cuda")
        ld = -(-(n + 24) // 8) * 8
        wide = torch.full((m + 3, ld), 7.0, dtype=dt, device="cuda")
        out = wide[1:m + 1, 8:8 + n]
        got = lce.fp8_matmul(a, sa, b, sb, out=out)
        assert got is out
        check_product(out, full(a, sa), full(b, sb), 300)
        assert (wide[0] == 7).all() and (wide[m + 1:] == 7).all()
        assert (wide[:, :8] == 7).all() and (wide[:, 8 + n:] == 7).all()


def test_nan_stays_in_its_row_and_column():
    a, sa = operand(70, 300, 8, False)
    b, sb = operand(200, 300, 9, True)
    a.view(torch.uint8)[3, 5] = 0x7f
    b.view(torch.uint8)[11, 299] = 0x7f
    z = lce.fp8_matmul(a, sa, b, sb)
    bad = torch.isnan(z)
    want = torch.zeros_like(bad)
    want[3] = True
    want[:, 11] = True
    assert torch.equal(bad, want)


def dq(x, tiles=False):
    q, s = ops_oracle.quantize_fp8(x.double().cpu().numpy(), tiles)
    return torch.from_numpy(ops_oracle.dequantize_fp8(q, s)).cuda()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("m,v,d", [(1, 300, 64), (5, 1000, 100), (130, 257, 300), (700, 3000, 520)])
def test_linear_and_gradients(m, v, d, dtype):
    X = rand(m, d, 1, dtype, 0.5).cuda().requires_grad_()
    W = (rand(v, d, 2, dtype, 0.2) * 0.05).cuda().requires_grad_()
    dZ = (rand(m, v, 3, dtype, 0.5) * 0.01).cuda()
    Z = lce.fp8_linear(X, W)
    dX, dW = torch.autograd.grad(Z, (X, W), dZ)
    assert Z.dtype == X.dtype and dX.dtype == X.dtype and dW.dtype == W.dtype
    assert dX.shape == X.shape and dW.shape == W.shape
    x, w, z = dq(X.detach()), dq(W.detach(), True), dq(dZ)
    check_product(Z, x, w, d)
    check_product(dX, z, w.t(), v)
    check_product(dW, dq(dZ.t()), dq(X.detach().t()), m)
    # frozen: the same logits and gradient of X
    w8 = lce.fp8_weight(W.detach())
    Z2 = lce.fp8_linear(X, w8)
    (dX2,) = torch.autograd.grad(Z2, X, dZ)
    assert torch.equal(Z2, Z) and torch.equal(dX2, dX)
    with torch.no_grad():
        assert torch.equal(lce.fp8_linear(X, w8._replace(q_t=None, scale_t=None)), Z)
    # only one of the two
    (dX3,) = torch.autograd.grad(lce.fp8_linear(X, W.detach()), X, dZ)
    (dW3,) = torch.autograd.grad(lce.fp8_linear(X.detach(), W), W, dZ)
    assert torch.equal(dX3, dX) and torch.equal(dW3, dW)


def test_gradients_against_differences():
    # on the e4m3 grid (whole numbers up to 8 and one 448 in every block: scale 1) the function
    # is linear, and a difference is exact
    g = torch.Generator().manual_seed(4)

    def grid(r, c):
        x = torch.randint(-8, 9, (r, c), generator=g).float()
        x[:, ::128] = 448.0
        x[::128] = 448.0
        return x.cuda()
    m, v, d = 130, 260, 270
    X, W, dZ = grid(m, d), grid(v, d), grid(m, v)
    Xg, Wg = X.clone().requires_grad_(), W.clone().requires_grad_()
    dX, dW = torch.autograd.grad(lce.fp8_linear(Xg, Wg), (Xg, Wg), dZ)
    for i, j in ((1, 1), (129, 269), (17, 200), (100, 127)):
        for P, G, f in ((X, dX, lambda p: lce.fp8_linear(p, W)), (W, dW, lambda p: lce.fp8_linear(X, p))):
            up, down = P.clone(), P.clone()
            up[i, j], down[i, j] = 9.0, -9.0
            change = ((f(up).double() - f(down).double()) * dZ.double()).sum().item() / 18.0
            # all sums are whole numbers below 2^24 times a power of two
            assert abs(change - G[i, j].item()) <= 2.0 ** -20 * max(abs(change), 2.0 ** 20), (i, j)


def test_gradient_of_broadcast_and_strided_upstream():
    X = rand(40, 256, 1).cuda().requires_grad_()
    w8 = lce.fp8_weight(rand(1001, 256, 2).cuda())
    Z = lce.fp8_linear(X, w8)
    (a,) = torch.autograd.grad(Z.float().sum(), X, retain_graph=True)
    (b,) = torch.autograd.grad(Z, X, torch.ones(40, 1001, dtype=Z.dtype, device="cuda"), retain_graph=True)
    (c,) = torch.autograd.grad(Z, X, torch.ones(1, 1, dtype=Z.dtype, device="cuda").expand(40, 1001))
    assert torch.equal(a, b) and torch.equal(b, c)


def test_second_derivative_is_refused():
    X = rand(8, 128, 1).cuda().requires_grad_()
    W = rand(40, 128, 2).cuda().requires_grad_()
    dX, dW = torch.autograd.grad(lce.fp8_linear(X, W).float().square().sum(), (X, W), create_graph=True)
    with pytest.raises(RuntimeError, match="differentiate twice"):
        (dX.float().sum() + dW.float().sum()).backward()


def test_without_gradients():
    X, W = rand(33, 200, 1).cuda().requires_grad_(), rand(300, 200, 2).cuda().requires_grad_()
    Z = lce.fp8_linear(X, W)
    with torch.no_grad():
        Y = lce.fp8_linear(X, W)
    assert Z.requires_grad and not Y.requires_grad and torch.equal(Y, Z)


def test_graph_and_stream():
    a, sa = operand(64, 512, 1, False)
    b, sb = operand(5000, 512, 2, True)
    x = rand(64, 512, 7).cuda()
    w8 = lce.fp8_weight(rand(700, 512, 8).cuda(), transpose=False)
    out = torch.empty(64, 5000, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(1024, dtype=torch.uint8, device="cuda")
    want = lce.fp8_matmul(a, sa, b, sb)
    graphs = []
    for _ in range(2):                       # two graphs that share a workspace and an output
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lce.fp8_matmul(a, sa, b, sb, out=out, ws=ws)
            with torch.no_grad():
                z = lce.fp8_linear(x, w8)
        graphs.append((g, z))
    for g, z in graphs:
        out.zero_()
        z.zero_()
        x.copy_(rand(64, 512, 9))
        g.replay()
        assert torch.equal(out, want)
        with torch.no_grad():
            assert torch.equal(z, lce.fp8_linear(x, w8))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = lce.fp8_matmul(a, sa, b, sb, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)


def test_no_rows():
    w = rand(300, 64, 1).cuda().requires_grad_()
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    z = lce.fp8_linear(x, w)
    assert z.shape == (0, 300)
    dx, dw = torch.autograd.grad(z, (x, w), torch.empty(0, 300, dtype=torch.bfloat16, device="cuda"))
    assert dx.shape == (0, 64) and (dw == 0).all()


@pytest.mark.parametrize("out_dtype", list(DTYPES))
@pytest.mark.parametrize("m,n,k", [(1537, 1701, 20000), (700, 4001, 33001), (2049, 1290, 50000)])
def test_few_tiles_and_a_long_k(m, n, k, out_dtype):
    # parts of k, added from the workspace; a small workspace gives the product in one part
    (a, sa), (b, sb) = operand(m, k, 1, False), operand(n, k, 2, True)
    t = DTYPES[out_dtype]
    size = lce.fp8_matmul_workspace_size(m, n, k)
    assert size > 1024 and lce.fp8_matmul_workspace_size(m, n, k, rows=True) == 1024
    wide = torch.full((m, 4096), 7.0, dtype=t, device="cuda")
    out = wide[:, :n]
    guard = torch.full((size + 4096,), 85, dtype=torch.uint8, device="cuda")
    ws = guard[2048:2048 + size]
    lce.fp8_matmul(a, sa, b, sb, out=out, ws=ws)
    assert lce.read_status(ws) == 0 and (wide[:, n:] == 7).all()
    assert (guard[:2048] == 85).all() and (guard[2048 + size:] == 85).all()
    one = lce.fp8_matmul(a, sa, b, sb, out_dtype=t, ws=torch.empty(1024, dtype=torch.uint8, device="cuda"))
    assert torch.equal(out, lce.fp8_matmul(a, sa, b, sb, out_dtype=t))
    A = a.double() * sa.double().repeat_interleave(128, 1)[:, :k]
    B = b.double() * sb.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    want, S = A @ B.T, A.abs() @ B.abs().T
    blocks = -(-k // 128)
    # (the bound of the module's head: the parts' sums add up to as many blocks, and at most 8 more)
    bound = (128 + blocks + 4 + 8) * 2.0 ** -23 * S + torch.finfo(t).eps / 2 * want.abs()
    # rounding to nearest gives infinity from half a step past the type's largest value on; the bf16 and fp32
    # results lie far below theirs
    edge = torch.finfo(t).max * (1 + torch.finfo(t).eps / 4)
    over, finite = want.abs() - bound >= edge, want.abs() + bound < edge
    for got in (out, one):
        assert ((got.double() - want).abs() <= bound * (1 + 2.0 ** -10))[finite].all()
        assert (got.double()[over] == want[over].sign() * float("inf")).all()


def test_parts_in_a_graph_and_a_gradient():
    # the gradient of an input whose layer is narrow, eager and captured
    X = rand(1537, 1600, 1).cuda()
    w8 = lce.fp8_weight(rand(20000, 1600, 2).cuda())
    dZ = rand(1537, 20000, 3).cuda()
    Xg = X.clone().requires_grad_()
    (dX,) = torch.autograd.grad(lce.fp8_linear(Xg, w8), Xg, dZ)
    q, s = lce.quantize_fp8(dZ)
    want = lce.fp8_matmul(q, s, w8.q_t, w8.scale_t)
    assert torch.equal(dX, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = lce.fp8_matmul(q, s, w8.q_t, w8.scale_t)
    out.zero_()
    g.replay()
    assert torch.equal(out, want)


@pytest.mark.parametrize("m,d,v", [(1, 128, 300), (40, 200, 129), (300, 264, 1001)])
def test_either_gradient_alone(m, d, v):
    X, W, dZ = rand(m, d, 1).cuda(), rand(v, d, 2).cuda(), rand(m, v, 3).cuda()
    both = [t.clone().requires_grad_() for t in (X, W)]
    dX, dW = torch.autograd.grad(lce.fp8_linear(*both), both, dZ)
    Xg, Wg = X.clone().requires_grad_(), W.clone().requires_grad_()
    (a,) = torch.autograd.grad(lce.fp8_linear(Xg, W), Xg, dZ)
    (b,) = torch.autograd.grad(lce.fp8_linear(X, Wg), Wg, dZ)
    (c,) = torch.autograd.grad(lce.fp8_linear(Xg, lce.fp8_weight(W)), Xg, dZ)
    assert torch.equal(a, dX) and torch.equal(b, dW) and torch.equal(c, dX)


def test_training_on_another_stream_and_twice_through_one_graph():
    X, W, dZ = rand(64, 256, 1).cuda().requires_grad_(), rand(500, 256, 2).cuda().requires_grad_(), rand(64, 500, 3).cuda()
    want = torch.autograd.grad(lce.fp8_linear(X, W), (X, W), dZ)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        Z = lce.fp8_linear(X, W)
        first = torch.autograd.grad(Z, (X, W), dZ, retain_graph=True)
        second = torch.autograd.grad(Z, (X, W), dZ)
    torch.cuda.current_stream().wait_stream(side)
    for got in (first, second):
        assert all(torch.equal(g, w) for g, w in zip(got, want))
