"""The surrounding operators at the ends of their ranges: tails of the activations, activations far below and above
fp16, layers wider than one wave of byte tables, moments that are not numbers, temporaries on a stream that is not the
current one, gradients that are replaced between steps, every entry point in the form that expands the weights."""
import math

import numpy as np
import pytest
import torch

from residual_binarized_weight_b200 import build as rbw_build
from residual_binarized_weight_b200 import rbw
from tests.test_adamw_gpu import F32, make, reference, upload
from tests.test_epilogue_gpu import act64
from tests.test_linear_gpu import Case

gpu = pytest.mark.gpu
DEV = "cuda"


# ---------------------------------------------------------------- optimizer
@gpu
@pytest.mark.parametrize("n,at", [(600, 300), (256, 0), (700, 699)])
def test_a_second_moment_of_nan_stays(n, at):
    """8-bit states: NaN in a gradient is NaN in both moments, in this step and the next; the other elements of the
    block are as if that element were 0 (its moments start from 0), bit for bit."""
    t = make(n, 8, F32, F32, 6)
    for name in ("m", "v"):
        t[name].view(torch.uint8)[at] = 0
    t["g"][at] = 0
    want = reference(t, 3, 0, 11)
    t["g"][at] = np.nan
    T = upload(t)
    opt = rbw.AdamW([T], seed=11)
    opt.step(3)
    others = torch.arange(n) != at
    for got, name in ((T.exp_avg, "m"), (T.exp_avg_sq, "v")):
        assert bool(torch.isnan(got.float())[at]), name
        assert torch.equal(got.cpu().view(torch.uint8)[others], want[name].view(torch.uint8)[others]), name
    for got, name in ((T.exp_avg_scale, "ms"), (T.exp_avg_sq_scale, "vs")):
        assert np.array_equal(got.cpu().numpy(), want[name]), name
    T.grad.nan_to_num_(0.0)
    opt.step(4)
    for got in (T.exp_avg, T.exp_avg_sq, T.param):
        assert int(torch.isnan(got.float()).sum()) == 1 and bool(torch.isnan(got.float())[at])


@gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_replaced_gradients_are_the_ones_used(bits):
    """A gradient, rate or decay that is assigned between steps counts in the next one."""
    ts = [make(3000, bits, F32, F32, i) for i in range(3)]
    Ts, Rs = [upload(t) for t in ts], [upload(t) for t in ts]
    opt = rbw.AdamW(Ts, seed=2)
    opt.step(1)
    rbw.AdamW(Rs, seed=2).step(1)
    for T, R in zip(Ts[1:], Rs[1:]):
        new = torch.randn(3000, device=DEV)
        T.grad, R.grad = new, new
        T.lr = R.lr = 0.5
        T.weight_decay = R.weight_decay = 0.25
    opt.step(2)
    rbw.AdamW(Rs, seed=2).step(2)
    for T, R in zip(Ts, Rs):
        for a, b in ((T.param, R.param), (T.exp_avg, R.exp_avg), (T.exp_avg_sq, R.exp_avg_sq)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# ---------------------------------------------------------------- activations
# GELU is p Phi(p).  Below zero Phi's kernel form is a quotient (one unit of 2^-23), a polynomial (with its own
# roundings 4 units), two products and exp(-p^2 / 2), by CUDA's bound for the fast exponential 2 + 0.6 p^2 units, whose
# argument's rounding counts 0.25 p^2 more: less than (2 p^2 + 16) 2^-23, relative to the result wherever it lies.
def gelu_bound(p):
    return (2 * p * p + 16) * 2.0 ** -23


@gpu
@pytest.mark.parametrize("M", [1, 5, 70])
def test_gelu_relative_to_itself(M):
    """X is 0, so that P is the bias: the activation in fp32."""
    N = 3277
    c = Case(M, N, 64, 2)
    c.layer.h16.zero_()
    p = (torch.arange(N, device=DEV) - 1638) / 128.0           # -12.8 .. 12.8
    Y = rbw.linear(c.layer, c.X, bias=p, act="gelu", y_dtype=torch.float32).double()
    p = p.double()
    want = 0.5 * p * torch.special.erfc(-p / math.sqrt(2))
    assert bool(((Y - want).abs() <= gelu_bound(p) * want.abs()).all())


@gpu
@pytest.mark.parametrize("N", [200, 1640])
def test_gelu_slope_far_below_zero(N):
    """dP and dmul at p = 0 .. -12.8; the slope's two terms cancel near -0.75, so its bound goes by their sizes."""
    P = (-torch.arange(N, device=DEV) * (12.8 / N)).bfloat16().expand(9, N).contiguous()
    one = torch.ones_like(P)
    dP, dU, db = rbw.epilogue_backward(one, P, act="gelu", mul=one)
    p = P.double()
    c, t = 0.5 * torch.special.erfc(-p / math.sqrt(2)), p * torch.exp(-p * p / 2) / math.sqrt(2 * math.pi)
    a, d = act64(p, "gelu")
    assert bool(((dU.double() - a).abs() <= (2.0 ** -8 + gelu_bound(p)) * a.abs()).all())
    off = gelu_bound(p) * (c + t.abs())
    assert bool(((dP.double() - d).abs() <= 2.0 ** -8 * d.abs() + off).all())
    assert bool(((db.double() - d.sum(0)).abs() <= (off + 9 * 2.0 ** -24 * d.abs()).sum(0)).all())


# ---------------------------------------------------------------- activations out of fp16's range
def rescaled(c, scale):
    """The case with row m of X times scale[m]: X, the exact product and its bound.  The bound is Case's without its
    absolute part: planes' ratios and sums (k >= 2), the tensor core's sums; all in proportion to the row."""
    c.X = (c.X.double() * scale[:, None]).bfloat16()
    planes = rbw.planes_to_rowmajor(c.layer).cpu().numpy().view(np.uint8)
    b = torch.from_numpy(np.unpackbits(planes, bitorder="little").reshape(c.k, c.N, c.K)).to(DEV)
    x, h, g = c.X.double(), c.h.double(), c.g.double()
    c.z = sum(((x * h[i]) @ (b[i].double() * 2 - 1).T) * g[i] for i in range(c.k))
    size = sum((x.abs() @ h[i].abs())[:, None] * g[i].abs() for i in range(c.k))
    top = g.abs().amax(0) * x.abs().sum(1, keepdim=True)
    c.slack = ((c.k > 1) * (c.k + 1) * 2.0 ** -11 + (c.K / 16 + 16) * 2.0 ** -23) * size + \
        (c.k > 1) * 2 * c.k * 2.0 ** -21 * top
    return c


FORMS = [(1, 300, 544, 2), (2, 300, 544, 2), (9, 203, 320, 1), (64, 700, 4128, 2), (333, 264, 96, 3), (9, 128, 11008, 2),
         (5, 64, 20032, 2), (2600, 4104, 1056, 2), (2048, 8191, 160, 2)]


@gpu
@pytest.mark.parametrize("M,N,K,k", FORMS)
def test_rows_of_any_size(M, N, K, k):
    """Rows of X from 1e-37 to 1e5, as gradients and outliers have them."""
    c = Case(M, N, K, k, seed=M)
    e = torch.tensor([0.0, -4, -6, -9, -15, -25, -37, -8, -7, -5], device=DEV, dtype=torch.float64)
    rescaled(c, 10.0 ** e.repeat((M + 9) // 10)[:M])
    st = torch.zeros(4, dtype=torch.int32, device=DEV)
    Y = rbw.linear(c.layer, c.X, y_dtype=torch.float32, dev_status=st)
    off = (Y.double() - c.z).abs() - c.slack - 2.0 ** -23 * c.z.abs() - 2.0 ** -148
    assert bool((off <= 0).all()), float(off.max())
    assert int(st[0]) == 0
    Z = rbw.linear(c.layer, c.X, residual=Y, y_dtype=torch.float32)       # the epilogue goes on from the scaled row
    assert bool(((Z.double() - 2 * Y.double()).abs() <= 2.0 ** -23 * Y.double().abs()).all())
    wide = (c.X.double() * 1e4).bfloat16()
    ok = wide.float().abs().amax(1) > 65536
    rescaled(c, torch.full((M,), 1e4, device=DEV, dtype=torch.float64))
    Y = rbw.linear(c.layer, c.X, y_dtype=torch.float32, dev_status=st)
    off = (Y.double() - c.z).abs() - c.slack - 2.0 ** -23 * c.z.abs() - 2.0 ** -148
    assert bool((off <= 0).all()), float(off.max())
    if M == 1:
        assert int(st[0]) == 0
    elif bool(ok.any()):
        assert int(st[0]) == rbw.RB_DEV_RANGE                              # reported all the same


@gpu
@pytest.mark.parametrize("M,N,K,k", FORMS[1:])
def test_small_values_beside_a_large_one(M, N, K, k):
    """A row whose largest value meets weights of 0: what counts is 1e-8 of it."""
    c = Case(M, N, K, k, seed=M + 1)
    c.layer.h16[:, 5] = 0
    c.h = c.layer.h16
    c.X[:, 5] = 0
    scale = torch.full((M,), 1e-8, device=DEV, dtype=torch.float64)
    rescaled(c, scale)
    c.X[:, 5] = 1.0
    Y = rbw.linear(c.layer, c.X, y_dtype=torch.float32)
    # values keep their bits down to 2^-31 of the row's largest, and are off by at most 2^-39 of it below
    size = sum((c.h[i].double().abs().sum() * c.g[i].double().abs())[None] for i in range(k))
    off = (Y.double() - c.z).abs() - c.slack - 2.0 ** -23 * c.z.abs() - 2.0 ** -39 * size
    assert bool((off <= 0).all()), float(off.max())


@gpu
@pytest.mark.parametrize("M,N,K,k", FORMS[1:])
def test_rows_that_are_not_finite(M, N, K, k):
    """An infinity or NaN stays in its row; an infinity is reported, a NaN shows itself."""
    c = Case(M, N, K, k, seed=M + 2)
    c.layer.h16.abs_().clamp_min_(1e-3)
    clean = rbw.linear(c.layer, c.X, y_dtype=torch.float32)
    for bad, flag in ((float("inf"), rbw.RB_DEV_RANGE), (float("nan"), 0)):
        X = c.X.clone()
        X[1, K // 2] = bad
        X[1, K - 1] = 1e30
        st = torch.zeros(4, dtype=torch.int32, device=DEV)
        Y = rbw.linear(c.layer, X, y_dtype=torch.float32, dev_status=st)
        assert not bool(torch.isfinite(Y[1]).any())
        assert int(st[0]) == rbw.RB_DEV_RANGE                              # (1e30 is above fp16, too)
        keep = torch.arange(M, device=DEV) != 1
        assert torch.equal(Y[keep], clean[keep])
        if bad == bad:
            assert bool((Y[1] == float("inf")).logical_or(Y[1] == -float("inf")).all())
        X[1, K - 1] = 0
        st.zero_()
        rbw.linear(c.layer, X, dev_status=st)
        assert int(st[0]) == flag


@gpu
@pytest.mark.parametrize("M,N,K", [(70, 290, 480), (2600, 4100, 1056)])
def test_small_rows_of_a_training_forward(M, N, K):
    W = torch.randn(N, K, device=DEV) * 0.02
    g, h = rbw.svid_greedy(W, 2, 10)
    X = torch.randn(M, K, device=DEV).bfloat16()
    s = 2.0 ** -60
    pre = [torch.empty(M, N, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    a = rbw.qat_linear(W, g, h, 2, X, preact=pre[0], y_dtype=torch.float32)
    b = rbw.qat_linear(W, g, h, 2, X * s, preact=pre[1], y_dtype=torch.float32)
    assert torch.equal(a * s, b) and torch.equal(pre[0] * s, pre[1])       # scaled by a power of two: bit for bit


# ---------------------------------------------------------------- one token
@gpu
@pytest.mark.parametrize("N,K,k", [(128256, 4096, 3), (151936, 4096, 4), (400000, 4096, 2), (400000, 4096, 1),
                                   (1000000, 288, 2)])
def test_one_token_of_a_wide_layer(N, K, k):
    """Rows that one wave of the byte-table kernel cannot hold.  Against the product of two such tokens, both within
    their bounds of the definition: that of test_linear_gpu, and K 2^-23 of the magnitudes for the tables' fp32 sums."""
    L = rbw.PackedLayer(N, K, k)
    S, T = (K + 255) // 256, (N + 31) // 32
    p = L.planes.view(k, S, T, 8, 32)
    p.random_(-2 ** 31, 2 ** 31 - 1)
    rows = rbw.planes_to_rowmajor(L)                           # drops what stands for absent rows and columns
    L = rbw.planes_from_rowmajor(rows, N, K, k, out=L)
    L.g16.copy_((torch.rand(k, N, device=DEV) + 0.5) * 0.6 ** torch.arange(k, device=DEV)[:, None])
    L.h16.copy_(torch.randn(k, K, device=DEV) * 0.1)
    x = torch.randn(1, K, device=DEV).bfloat16()
    bias = torch.randn(N, device=DEV)
    res = torch.randn(1, N, device=DEV)
    y1 = rbw.linear(L, x, bias=bias, residual=res, y_dtype=torch.float32)
    y2 = rbw.linear(L, x.repeat(2, 1), bias=bias, residual=res.repeat(2, 1), y_dtype=torch.float32)
    g, h, xd = L.g16.double(), L.h16.double(), x.double()
    size = sum((xd.abs() @ h[i].abs())[:, None] * g[i].abs() for i in range(k))
    top = g.abs().amax(0) * xd.abs().sum()
    tol = ((k > 1) * (k + 1) * 2.0 ** -11 + (K / 16 + 16 + K) * 2.0 ** -23) * size + (k > 1) * 2 * k * 2.0 ** -25 * top
    tol = tol + 2.0 ** -22 * (y2[:1].double().abs() + bias.abs() + res.abs())
    assert bool(((y1.double() - y2[:1].double()).abs() <= tol).all())
    assert torch.equal(rbw.linear(L, x, y_dtype=torch.float32), rbw.gemv(L, x))


# ---------------------------------------------------------------- streams
def delay(cycles=40_000_000):
    """Some 20 ms of idling on the current stream."""
    torch.cuda._sleep(cycles)


def stream_case(which):
    """(call(stream), bytes of the workspace that it makes itself)"""
    if which == "backward":
        M, N = 3000, 1000
        d = torch.randn(M, N, device=DEV).bfloat16()
        return lambda s: rbw.epilogue_backward(d, d, act="silu", stream=s)[2], rbw.epilogue_backward_workspace_bytes(M, N)
    M, N, K = (2600, 4100, 1056) if which == "dense" else (300, 512, 1024)
    if which in ("qat", "forward"):
        W = torch.randn(N, K, device=DEV) * 0.02
        g, h = rbw.svid_greedy(W, 2, 5)
        X = torch.randn(M, K, device=DEV).bfloat16()
        if which == "forward":
            return lambda s: rbw.qat_forward(W, g, h, 2, X, stream=s), rbw.qat_forward_workspace_bytes(N, K, 2, M)
        return lambda s: rbw.qat_linear(W, g, h, 2, X, stream=s), rbw.qat_linear_workspace_bytes(N, K, 2, M)
    c = Case(M, N, K, 2)
    return lambda s: rbw.linear(c.layer, c.X, stream=s), rbw.linear_workspace_bytes(N, K, 2, M)


@gpu
@pytest.mark.parametrize("which", ["linear", "dense", "qat", "forward", "backward"])
def test_temporaries_belong_to_the_given_stream(which):
    """The workspace that a call on another stream makes for itself is not given to the current stream while that call
    is still to run: what the current stream then allocates and fills keeps its values."""
    call, nbytes = stream_case(which)
    want = call(None)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        delay()
    got = call(s)
    mine = [torch.full((max(nbytes // d, 16),), 77, dtype=torch.uint8, device=DEV) for d in (1, 1, 2, 4)]
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    for t in mine:
        assert bool((t == 77).all())


@gpu
@pytest.mark.parametrize("which", ["linear", "dense", "qat", "forward", "backward"])
def test_results_of_another_stream_outlive_their_readers(which):
    """A result made on another stream and dropped while the current stream still has to read it is not overwritten
    by the next call's."""
    call, _ = stream_case(which)
    want = call(None).clone()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    got = call(s)
    torch.cuda.current_stream().wait_stream(s)
    delay()
    copy = got.clone()
    del got
    with torch.cuda.stream(s):
        junk = [torch.full_like(want, 5.0) for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(copy, want) and all(bool((t == 5).all()) for t in junk)


# ---------------------------------------------------------------- weights expanded once
def expanded(N, K, k, M):
    """Whether the product runs on weights expanded in its workspace, by that workspace's size."""
    return rbw.linear_workspace_bytes(N, K, k, M) >= 2 * N * K + 2 * M * K


DENSE = [(2600, 4100, 1056), (2048, 8192, 160)]


@pytest.mark.parametrize("k", [1, 2, 4])
@pytest.mark.parametrize("M,N,K", DENSE)
def test_these_sizes_expand_the_weights(M, N, K, k):
    rbw_build.build()
    assert expanded(N, K, k, M) and not expanded(N, K, k, 64)


@gpu
@pytest.mark.parametrize("k", [1, 2, 4])
@pytest.mark.parametrize("M,N,K", DENSE)
def test_latent_weight_expanded(M, N, K, k):
    """As test_linear_gpu's test_latent_weight, with the expanded weights' subnormal step (2^-21 of the row's largest)."""
    assert expanded(N, K, k, M)
    W = torch.randn(N, K, generator=torch.Generator().manual_seed(k)).cuda() * 0.02
    g, h = rbw.svid_greedy(W, k, 10)
    c = Case(M, N, K, k, seed=4)
    r, What, size = W.clone(), 0, 0
    for i in range(k):
        t = g[i][:, None] * h[i]
        s = torch.where(r >= 0, 1.0, -1.0)
        What = What + s.double() * g[i].double()[:, None] * h[i].double()
        size = size + t.double().abs()
        r = r - s * t
    x = c.X.double()
    c.z = x @ What.T
    c.slack = ((k + 2) * 2.0 ** -11 + (K / 16 + 16) * 2.0 ** -23) * (x.abs() @ size.T) + \
        (k > 1) * k * 2.0 ** -21 * g.double().abs().amax(0) * x.abs().sum(1, keepdim=True)
    pre = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    ws = rbw.workspace(rbw.qat_linear_workspace_bytes(N, K, k, M))
    Y = rbw.qat_linear(W, g, h, k, c.X, bias=c.bias, act="gelu_tanh", mul=c.mul, residual=c.res16, preact=pre, ws=ws)
    c.check(Y, c.bias, "gelu_tanh", c.mul, c.res16, pre)
    c.check(rbw.qat_linear(W, g, h, k, c.X, ws=ws, y_dtype=torch.float32), norm=False)
    planes = rbw.pack(W, g, h, k).planes
    assert torch.equal(ws[:4 * planes.numel()].view(torch.int32), planes)


@gpu
@pytest.mark.parametrize("M,N,K", DENSE)
def test_planes_of_an_expanded_training_forward_feed_the_next_launch(M, N, K):
    k = 2
    assert expanded(N, K, k, M)
    gen = torch.Generator().manual_seed(M)
    Ws = [(torch.randn(N, K, generator=gen) * 0.02).cuda() for _ in range(3)]
    g, h = torch.full((k, N), 0.02, device=DEV), torch.full((k, K), 0.5, device=DEV)
    g[1] *= 0.5
    X = torch.randn(M, K, generator=gen).bfloat16().cuda()
    W = Ws[0].clone()
    ws = rbw.workspace(rbw.qat_linear_workspace_bytes(N, K, k, M))
    words = rbw.pack(W, g, h, k).planes.numel()
    L = rbw.PackedLayer(N, K, k, planes=ws[:4 * words].view(torch.int32), g16=g.half(), h16=h.half())
    few = X[:7]
    ws2 = [rbw.workspace(rbw.linear_workspace_bytes(N, K, k, m)) for m in (M, 7)]
    Y, Z = (torch.empty(M, N, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    z = torch.empty(7, N, dtype=torch.bfloat16, device=DEV)

    def chain():
        rbw.qat_linear(W, g, h, k, X, Y, ws=ws, flags=rbw.RB_LAUNCH_PDL)
        rbw.linear(L, few, z, ws=ws2[1], flags=rbw.RB_LAUNCH_PDL)          # reads the planes before it waits
        rbw.linear(L, X, Z, ws=ws2[0], flags=rbw.RB_LAUNCH_PDL)

    chain()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for i in range(9):
        W.copy_(Ws[i % 3])
        graph.replay() if i % 2 else chain()
        torch.cuda.synchronize()
        P = rbw.pack(Ws[i % 3], g, h, k)
        assert torch.equal(Z, rbw.linear(P, X)) and torch.equal(z, rbw.linear(P, few)), i


@gpu
@pytest.mark.parametrize("M,N,K", DENSE)
def test_expanded_weights_in_a_graph_and_on_streams(M, N, K):
    a, b = Case(M, N, K, 2, seed=1), Case(M, K, N // 32 * 32, 2, seed=2)
    assert expanded(N, K, 2, M)
    X = a.X.clone()
    mid, out = torch.empty(M, N // 32 * 32 + 32, dtype=torch.bfloat16, device=DEV), torch.empty(M, K, device=DEV)
    ws = [rbw.workspace(rbw.linear_workspace_bytes(N, K, 2, M)), rbw.workspace(rbw.linear_workspace_bytes(K, N // 32 * 32, 2, M))]

    def chain():
        rbw.linear(a.layer, X, mid[:, :N], act="silu", ws=ws[0], flags=rbw.RB_LAUNCH_PDL)
        rbw.linear(b.layer, mid[:, :N // 32 * 32], out, ws=ws[1], flags=rbw.RB_LAUNCH_PDL)

    chain()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):
            chain()
    for k in range(2):
        X.copy_(torch.randn(M, K, generator=torch.Generator().manual_seed(k)).bfloat16())
        g.replay()
        torch.cuda.synchronize()
        m = rbw.linear(a.layer, X, act="silu")
        assert torch.equal(m, mid[:, :N])
        assert torch.equal(rbw.linear(b.layer, m[:, :N // 32 * 32].contiguous(), y_dtype=torch.float32), out)
    want = [rbw.linear(c.layer, c.X) for c in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append(rbw.linear((a, b)[i % 2].layer, (a, b)[i % 2].X))
        torch.cuda.synchronize()
        assert all(torch.equal(y, want[i % 2]) for i, y in enumerate(got))


@gpu
@pytest.mark.parametrize("M,N,K", DENSE)
def test_expanded_weights_report_what_they_meet(M, N, K):
    k = 2
    c = Case(M, N, K, k, seed=3)
    st = torch.zeros(4, dtype=torch.int32, device=DEV)
    X = c.X.clone()
    X[M - 1, K - 1] = 1e6
    rbw.linear(c.layer, X, dev_status=st)
    assert int(st[0]) == rbw.RB_DEV_RANGE
    c.layer.g16[0, 5], c.layer.g16[1, 5] = 0, float("nan")
    bad = torch.isnan(rbw.linear(c.layer, c.X))
    assert bool(bad[:, 5].all()) and int(bad.sum()) == M
    W = torch.randn(N, K, device=DEV)
    for at in (0, 21, K - 1):
        for value, flag in ((1.0, 0), (7e4, rbw.RB_DEV_RANGE), (-float("inf"), rbw.RB_DEV_RANGE),
                            (float("nan"), rbw.RB_DEV_NONFINITE)):
            g, h = torch.ones(k, N, device=DEV), torch.ones(k, K, device=DEV)
            h[k - 1, at] = value
            st.zero_()
            rbw.qat_linear(W, g, h, k, c.X, dev_status=st)
            assert int(st[0]) & flag == flag and (flag or int(st[0]) == 0), (at, value, int(st[0]))


@gpu
@pytest.mark.parametrize("M,N,K", [(6000, 262176, 16416), (262200, 8192, 16416)])
def test_expanded_weights_with_large_offsets(M, N, K):
    """W16 past 2^32 elements, and X16."""
    k = 2
    assert expanded(N, K, k, M)
    L = rbw.PackedLayer(N, K, k)
    L.planes.zero_()                                         # -1 everywhere; the last rows' words are set below
    words = torch.zeros(k, 64, K // 32, dtype=torch.int32, device=DEV)
    words.random_(-2 ** 31, 2 ** 31 - 1)
    T, S = (N + 31) // 32, (K + 255) // 256
    small = rbw.planes_from_rowmajor(words, 64, K, k)
    L.planes.view(k, S, T, 256)[:, :, T - 2:] = small.planes.view(k, S, 2, 256)
    L.g16.copy_(torch.rand(k, N, device=DEV) + 0.5), L.h16.copy_(torch.randn(k, K, device=DEV) * 0.1)
    X = torch.randn(500, K, device=DEV).bfloat16().repeat((M + 499) // 500, 1)[:M]
    Y = rbw.linear(L, X)
    first = Y[:500].clone()
    assert bool((Y[:M // 500 * 500].view(-1, 500, N) == first).all())
    assert torch.equal(Y[M // 500 * 500:], first[:M % 500])
    del Y
    x = X[:500].double()
    bits = np.unpackbits(words.cpu().numpy().view(np.uint8), bitorder="little").reshape(k, 64, K)
    sign = torch.from_numpy(bits).to(DEV).double() * 2 - 1
    g, h = L.g16.double(), L.h16.double()
    for rows, s in ((slice(N - 64, N), sign), (slice(0, 64), -torch.ones_like(sign))):
        want = sum(((x * h[i]) @ s[i].T) * g[i, rows] for i in range(k))
        size = sum((x.abs() @ h[i].abs())[:, None] * g[i, rows].abs() for i in range(k))
        tol = ((k + 1) * 2.0 ** -11 + (K / 16 + 16) * 2.0 ** -23) * size + \
            k * 2.0 ** -21 * g[:, rows].amax(0) * x.abs().sum(1, keepdim=True)
        assert bool(((first[:, rows].double() - want).abs() <= tol + 2.0 ** -8 * want.abs()).all())
    torch.cuda.empty_cache()
