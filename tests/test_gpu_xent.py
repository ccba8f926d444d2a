"""GPU parity of the loss head (lin_xent, lin_xent_bwd) with a plain float64 implementation.

Bounds (u = 2^-24, the fp32 half step; h the operands' half step, 2^-8 or 2^-11):
  logits      |dz| <= gamma(K) * sum_k |x w|            (gpu_util.gamma: fp32 accumulation of exact products)
  lse         max_v |dz| + fp32 statistics: a term's 2^x has an argument error of at most 24u
              (terms below 2^-24 of the maximum do not count) and 2u of its own, a chain of 64
              additions within a wave and J joins of 26u each, then two roundings of the result
  G           |dG| <= |s| (h |p - t| + p (|dz| + |dlse| + 4u))  + fp16's subnormal step
  dX, dW      sum |dG| |w| + gamma(R) sum |G w| + h |result| (and fp16's subnormal step)
"""
import numpy as np
import pytest
import torch

import linear_layer_backward_bwd_amd as lb
from gpu_util import gamma

pytestmark = pytest.mark.gpu
DEV = "cuda"
T = {"bf16": torch.bfloat16, "f16": torch.float16}
H = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
U = 2.0 ** -24


def case(M, K, V, dtype, seed=0, ignored=0.2, w_std=None, offset=0):
    g = torch.Generator().manual_seed(seed * 7919 + M * 31 + K * 17 + V)
    X = torch.randn(M, K, generator=g).to(T[dtype])
    W = (torch.randn(K, V, generator=g) * (w_std if w_std is not None else 1.5 / K ** 0.5)).to(T[dtype])
    t = torch.randint(0, V, (M,), generator=g)
    t[torch.rand(M, generator=g) < ignored] = -100
    return place(X, offset), place(W, offset), t.to(DEV)


def place(t, offset):
    """t on the GPU, `offset` elements past a 16-byte boundary, canaries on both sides."""
    buf = torch.full((t.numel() + 128 + offset,), -123.0, dtype=t.dtype, device=DEV)
    v = buf[64 + offset:64 + offset + t.numel()].view(t.shape)
    v.copy_(t)
    v.whole = buf
    return v


def guarded(shape, dtype, offset=0):
    return place(torch.full(shape, float("nan"), dtype=dtype), offset)


def check_guards(v):
    n, lo = v.numel(), (v.data_ptr() - v.whole.data_ptr()) // v.element_size()
    assert bool((v.whole[:lo] == -123.0).all()) and bool((v.whole[lo + n:] == -123.0).all())


def plain(X, W, t):
    """float64 logits, lse, loss, and the magnitude sums of the logits."""
    x, w = X.double(), W.double()
    z = x @ w
    S = x.abs() @ w.abs()
    lse = torch.logsumexp(z, 1)
    loss = lse - z.gather(1, t.clamp(min=0)[:, None])[:, 0]
    keep = t >= 0
    return z, S, torch.where(keep, lse, 0.0), torch.where(keep, loss, 0.0), keep


def lse_bound(S, K, V, lse):
    dz = 1.01 * gamma(K) * S.amax(1)
    joins = V / 32 / 16 + 16
    return dz + U * (26 + 64 + 26 * joins) + 4 * U * lse.abs()


def check_forward(X, W, t, got):
    loss, lse, out = got
    z, S, rl, ro, keep = plain(X, W, t)
    b = lse_bound(S, X.shape[1], W.shape[1], rl)
    assert bool(((lse.double() - rl).abs() <= b * keep).all())
    zt = (S.gather(1, t.clamp(min=0)[:, None])[:, 0]) * 1.01 * gamma(X.shape[1])
    bl = (b + zt + 2 * U * ro.abs()) * keep
    assert bool(((loss.double() - ro).abs() <= bl).all())
    n = int(keep.sum())
    mean = float(ro.sum()) / n if n else 0.0
    assert abs(out[0].item() - mean) <= (float(bl.sum()) / n if n else 0.0) + 2 * U * abs(mean)
    assert out[1].item() == np.float32(1.0 / n if n else 0.0)


def check_backward(X, W, t, lse, dX, dW, dtype, scale=1.0, d_scale=None, row_scale=None):
    K, V, M = X.shape[1], W.shape[1], X.shape[0]
    keep = t >= 0
    x = torch.where(keep[:, None], X.double(), 0.0)
    w = W.double()
    s = torch.full((M,), float(scale), dtype=torch.float64, device=DEV) * keep
    if d_scale is not None:
        s = s * d_scale.double()
    if row_scale is not None:
        s = s * row_scale.double()
    z = x @ w
    S = x.abs() @ w.abs()
    p = torch.exp(z - lse.double()[:, None])
    g = p.clone()
    g.scatter_add_(1, t.clamp(min=0)[:, None], -torch.ones_like(g[:, :1]))
    dz = 1.01 * gamma(K) * S
    h, smax = H[dtype], float(s.abs().max()) if M else 0.0
    dG = s.abs()[:, None] * (h * g.abs() + p * (dz + 4 * U * (1 + lse.double().abs()[:, None]) + 8 * U) + 4 * U)
    G = g * s[:, None]
    if dtype == "f16":
        dG = dG + 2.0 ** -38 * smax
    tiny = 2.0 ** -24 if dtype == "f16" else 1e-38
    if dX is not None:
        ref = G @ w.T
        b = (dG @ w.abs().T) + gamma(V) * 1.01 * ((G.abs() + dG) @ w.abs().T)
        b = b + h * (ref.abs() + b) + tiny
        assert bool(((dX.double() - ref).abs() <= b).all()), float(((dX.double() - ref).abs() / b).max())
        assert bool((dX[~keep] == 0).all())
    if dW is not None:
        ref = x.T @ G
        b = (x.abs().T @ dG) + gamma(M) * 1.01 * (x.abs().T @ (G.abs() + dG))
        b = b + h * (ref.abs() + b) + tiny
        assert bool(((dW.double() - ref).abs() <= b).all()), float(((dW.double() - ref).abs() / b).max())


def both(X, W, t, dtype, offset=0, **kw):
    M, K = X.shape
    V = W.shape[1]
    loss, lse = guarded((M,), torch.float32), guarded((M,), torch.float32)
    out = guarded((2,), torch.float32)
    lb.lin_xent(X, W, t, loss, lse, out)
    dX, dW = guarded((M, K), T[dtype], offset), guarded((K, V), T[dtype], offset)
    lb.lin_xent_bwd(X, W, t, lse, dX, dW, **kw)
    torch.cuda.synchronize()
    for v in (loss, lse, out, dX, dW):
        check_guards(v)
    return loss, lse, out, dX, dW


SHAPES = [(1, 1, 1), (1, 8, 5), (1, 64, 1000), (2, 7, 127), (5, 100, 128), (31, 64, 129), (32, 264, 2056),
          (33, 65, 257), (64, 128, 640), (65, 96, 250), (100, 33, 1001), (128, 520, 384), (129, 64, 256),
          (255, 72, 999), (256, 128, 512), (257, 264, 2056), (300, 31, 1023), (513, 136, 768), (1000, 200, 3001)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,K,V", SHAPES)
def test_matches_float64(M, K, V, dtype):
    X, W, t = case(M, K, V, dtype)
    loss, lse, out, dX, dW = both(X, W, t, dtype)
    check_forward(X, W, t, (loss, lse, out))
    check_backward(X, W, t, lse, dX, dW, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("offset", [1, 2, 4])
@pytest.mark.parametrize("M,K,V", [(3, 64, 264), (40, 40, 520), (300, 136, 512), (2600, 64, 264)])
def test_unaligned(M, K, V, dtype, offset):
    X, W, t = case(M, K, V, dtype, offset=offset)
    loss, lse, out, dX, dW = both(X, W, t, dtype, offset=offset)
    check_forward(X, W, t, (loss, lse, out))
    check_backward(X, W, t, lse, dX, dW, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,K,V", [(1, 130, 333), (17, 64, 4097), (70, 96, 1027), (130, 520, 2051), (200, 64, 20001),
                                   (256, 40, 9001), (257, 72, 1025), (2570, 64, 515), (2559, 65, 517)])
def test_odd_vocabulary(M, K, V, dtype):
    """Rows of W that start at any element: read through registers (M up to 256 backward, 2559
    forward) or copied first, in each tile shape."""
    X, W, t = case(M, K, V, dtype, seed=16)
    loss, lse, out, dX, dW = both(X, W, t, dtype)
    check_forward(X, W, t, (loss, lse, out))
    check_backward(X, W, t, lse, dX, dW, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M", [20, 400])
def test_scales(M, dtype):
    """Loss scale, device scale (the forward's 1 / count) and row weights, some of them 0 or negative."""
    X, W, t = case(M, 64, 700, dtype, seed=3)
    w = torch.randn(M, device=DEV)
    w[::5] = 0.0
    loss, lse, out = lb.lin_xent(X, W, t)
    dX, dW = torch.empty_like(X), torch.empty_like(W)
    lb.lin_xent_bwd(X, W, t, lse, dX, dW, scale=1024.0, d_scale=out[1:], row_scale=w)
    check_backward(X, W, t, lse, dX, dW, dtype, 1024.0, out[1:], w)
    assert bool((dX[::5] == 0).all())


@pytest.mark.parametrize("M", [7, 300])
def test_one_product_only(M):
    X, W, t = case(M, 72, 520, "bf16", seed=4)
    _, lse, _ = lb.lin_xent(X, W, t)
    dX, dW, dX2, dW2 = (torch.empty_like(a) for a in (X, W, X, W))
    lb.lin_xent_bwd(X, W, t, lse, dX, dW)
    lb.lin_xent_bwd(X, W, t, lse, dX=dX2)
    lb.lin_xent_bwd(X, W, t, lse, dW=dW2)
    lb.lin_xent_bwd(X, W, t, lse)
    assert torch.equal(dX, dX2) and torch.equal(dW, dW2)


@pytest.mark.parametrize("M", [5, 70, 300])
def test_rows_out_of_the_loss_may_hold_anything(M):
    X, W, t = case(M, 64, 513, "bf16", seed=5)
    t[0] = -1
    out = t < 0
    clean = both(X, W, t, "bf16")
    X[out] = float("nan")
    X[0] = float("inf")
    got = both(X, W, t, "bf16")
    for a, b in zip(clean, got):
        assert torch.equal(a, b)


def test_no_row_counts():
    X, W, t = case(40, 64, 300, "bf16", seed=6)
    t.fill_(-100)
    loss, lse, out, dX, dW = both(X, W, t, "bf16", d_scale=torch.zeros(1, device=DEV))
    for a in (loss, lse, out, dX, dW):
        assert bool((a == 0).all())


def test_no_rows():
    X, W, t = case(0, 64, 300, "bf16")
    loss, lse, out, dX, dW = both(X, W, t, "bf16")
    assert bool((out == 0).all()) and bool((dW == 0).all())


def test_target_past_the_vocabulary_is_nan():
    X, W, t = case(10, 64, 300, "bf16", seed=8, ignored=0.0)
    t[3] = 300
    t[4] = 1 << 40
    loss, lse, out, dX, dW = both(X, W, t, "bf16")
    bad = torch.tensor([3, 4], device=DEV)
    assert bool(loss[bad].isnan().all()) and int(loss.isnan().sum()) == 2 and bool(out[0].isnan())
    assert bool(dX[bad].isnan().all()) and int(dX.isnan().sum()) == 128 and bool(dW.isnan().all())


def test_nan_and_inf_stay_in_their_rows():
    X, W, t = case(20, 64, 300, "bf16", seed=9, ignored=0.0)
    X[2, 5] = float("nan")
    X[7, 1] = float("inf")
    loss, lse, out, dX, dW = both(X, W, t, "bf16")
    assert int(loss.isfinite().sum()) == 18 and not bool(loss[2].isfinite()) and not bool(loss[7].isfinite())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("std", [0.0, 0.01, 30.0])
def test_flat_and_sharp_logits(std, dtype):
    """Uniform rows (all logits 0), nearly uniform ones, and logits of hundreds."""
    X, W, t = case(70, 64, 2056, dtype, seed=10, w_std=std)
    loss, lse, out, dX, dW = both(X, W, t, dtype)
    check_forward(X, W, t, (loss, lse, out))
    check_backward(X, W, t, lse, dX, dW, dtype)


@pytest.mark.parametrize("M,K,V,dtype", [(64, 4096, 50257, "bf16"),   # packed pieces of W, dX in ranges
                                         (300, 2050, 70001, "f16"),
                                         (9000, 64, 40000, "bf16"),   # two pieces of G
                                         (520, 8, 4000, "bf16")])
def test_pieces(M, K, V, dtype):
    X, W, t = case(M, K, V, dtype, seed=11)
    loss, lse, out, dX, dW = both(X, W, t, dtype)
    rows = torch.randperm(M, generator=torch.Generator().manual_seed(1))[:256].to(DEV)
    z, S, rl, ro, keep = plain(X[rows], W, t[rows])
    b = lse_bound(S, K, V, rl) * keep
    assert bool(((lse[rows].double() - rl).abs() <= b).all())
    assert bool(((loss[rows].double() - ro).abs() <= 2 * b + 1e-6 * ro.abs()).all())
    check_backward(X, W, t, lse, dX, dW, dtype)


def test_many_statistics_pieces():
    """Statistics of one piece of the vocabulary are bounded: rows x columns that take two."""
    M, K, V = 36000, 16, 65000
    X, W, t = case(M, K, V, "bf16", seed=12)
    loss, lse, out = lb.lin_xent(X, W, t)
    rows = torch.arange(0, M, 97, device=DEV)
    z, S, rl, ro, keep = plain(X[rows], W, t[rows])
    b = lse_bound(S, K, V, rl) * keep
    assert bool(((lse[rows].double() - rl).abs() <= b).all())
    assert bool(((loss[rows].double() - ro).abs() <= 2 * b + 1e-6 * ro.abs()).all())
    assert abs(out[0].item() - float(loss.double().sum() / (t >= 0).sum())) <= 1e-6 * out[0].item()


@pytest.mark.parametrize("M,K,V", [(9, 64, 1000), (300, 128, 777)])
def test_repeatable_bit_for_bit(M, K, V):
    X, W, t = case(M, K, V, "bf16", seed=13)
    a = both(X, W, t, "bf16")
    b = both(X, W, t, "bf16")
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_gradient_against_differences():
    """<dX, D> and <dW, E> against central differences of the float64 loss."""
    M, K, V = 48, 64, 500
    X, W, t = case(M, K, V, "bf16", seed=14)
    loss, lse, out, dX, dW = both(X, W, t, "bf16", scale=1.0)
    g = torch.Generator(device=DEV).manual_seed(2)
    D = torch.randn(M, K, dtype=torch.float64, device=DEV, generator=g)
    E = torch.randn(K, V, dtype=torch.float64, device=DEV, generator=g)

    def total(x, w):
        z = x @ w
        each = torch.logsumexp(z, 1) - z.gather(1, t.clamp(min=0)[:, None])[:, 0]
        return float((each * (t >= 0)).sum())

    eps = 1e-5
    x, w = X.double(), W.double()
    for got, move, a, b in ((dX, D, 1.0, 0.0), (dW, E, 0.0, 1.0)):
        num = (total(x + eps * a * D, w + eps * b * E) - total(x - eps * a * D, w - eps * b * E)) / (2 * eps)
        # every entry of dX and dW carries G's and its own rounding, of random sign: 4 sigma
        noise = 2 * H["bf16"] * float((got.double() * move).norm()) * 4
        assert abs(float((got.double() * move).sum()) - num) <= noise + 1e-6 * abs(num)


@pytest.mark.parametrize("M", [12, 300])
def test_captured_graph_replays(M):
    K, V = 64, 1001
    X, W, t = case(M, K, V, "bf16", seed=15)
    n = max(lb.lin_xent_workspace(M, K, V), lb.lin_xent_bwd_workspace(M, K, V))
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    loss, lse = (torch.empty(M, device=DEV) for _ in range(2))
    out = torch.empty(2, device=DEV)
    dX, dW = torch.empty_like(X), torch.empty_like(W)

    def step():
        lb.lin_xent(X, W, t, loss, lse, out, ws=ws)
        lb.lin_xent_bwd(X, W, t, lse, dX, dW, d_scale=out[1:], ws=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(4):
        X2, W2, t2 = case(M, K, V, "bf16", seed=20 + seed)
        X.copy_(X2)
        W.copy_(W2)
        t.copy_(t2)
        graph.replay()
        torch.cuda.synchronize()
        got = [a.clone() for a in (loss, lse, out, dX, dW)]
        l2, e2, o2 = lb.lin_xent(X2, W2, t2)
        gX, gW = torch.empty_like(X), torch.empty_like(W)
        lb.lin_xent_bwd(X2, W2, t2, e2, gX, gW, d_scale=o2[1:])
        torch.cuda.synchronize()
        for a, b in zip(got, (l2, e2, o2, gX, gW)):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    cases = [case(200, 128, 3000, "bf16", seed=s) for s in (30, 31)]
    want = [both(*c, "bf16") for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[None] * 5 for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, (c, st) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(st):
                X, W, t = c
                loss, lse, out = lb.lin_xent(X, W, t)
                dX, dW = torch.empty_like(X), torch.empty_like(W)
                lb.lin_xent_bwd(X, W, t, lse, dX, dW)
                got[i] = [loss, lse, out, dX, dW]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


@pytest.mark.parametrize("M,K,V", [(200001, 16, 40), (70000, 9, 130)])
def test_many_rows(M, K, V):
    X, W, t = case(M, K, V, "bf16", seed=40)
    loss, lse, out, dX, dW = both(X, W, t, "bf16")
    check_forward(X, W, t, (loss, lse, out))
    check_backward(X, W, t, lse, dX, dW, "bf16")


@pytest.mark.parametrize("M,V", [(3, 1 << 21), (3, (1 << 21) + 5), (300, 1 << 21)])
def test_weights_past_4_gib(M, V):
    """W and dW of 4.6 GB: every row of the loss and of dX, dW on sampled rows."""
    K = 1100
    g = torch.Generator(device=DEV).manual_seed(41)
    X = torch.randn(M, K, device=DEV, generator=g).bfloat16()
    W = torch.empty(K, V, dtype=torch.bfloat16, device=DEV).normal_(0, 0.03, generator=g)
    t = torch.randint(0, V, (M,), device=DEV, generator=g)
    t[0], t[1] = V - 1, -1
    loss, lse, out = lb.lin_xent(X, W, t)
    dX, dW = torch.full_like(X, float("nan")), torch.full_like(W, float("nan"))
    lb.lin_xent_bwd(X, W, t, lse, dX, dW)
    z = torch.cat([X.double() @ W[:, lo:lo + (1 << 18)].double() for lo in range(0, V, 1 << 18)], 1)
    keep = t >= 0
    rl = torch.where(keep, torch.logsumexp(z, 1), 0.0)
    ro = torch.where(keep, rl - z.gather(1, t.clamp(min=0)[:, None])[:, 0], 0.0)
    # |dz| <= gamma(K) sum |x w| < 2^-24 * 99 * K * 0.06 and the statistics of 2^21 columns
    bound = 99 * U * K * 0.06 + U * (90 + 26 * (V / 512 + 16)) + 4 * U * 16
    assert float((lse.double() - rl).abs().max()) <= bound and float((loss.double() - ro).abs().max()) <= 2 * bound
    G = torch.exp(z - rl[:, None])
    G.scatter_add_(1, t.clamp(min=0)[:, None], -torch.ones_like(G[:, :1]))
    G *= keep[:, None]
    ref = sum(G[:, lo:lo + (1 << 18)] @ W[:, lo:lo + (1 << 18)].double().T.contiguous() for lo in range(0, V, 1 << 18))
    # the roundings of G and of dX, each at most half a bf16 step of its terms
    assert float((dX.double() - ref).norm()) <= 2 * H["bf16"] * float(ref.norm())
    rows = torch.tensor([0, 1, 511, 1023, K - 1], device=DEV)
    ref = X[:, rows].double().T @ G
    assert float((dW[rows].double() - ref).norm()) <= 2 * H["bf16"] * float(ref.norm())
    assert bool(dW[rows].isfinite().all())


def test_strided_views_are_refused():
    X, W, t = case(8, 64, 128, "bf16", seed=42)
    with pytest.raises(ValueError):
        lb.lin_xent(X[:, :32], W[:32], t)
    with pytest.raises(ValueError):
        lb.lin_xent(X, W[:, ::2], t)
    with pytest.raises(ValueError):
        lb.lin_xent(X, W, t, ws=torch.empty(16, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("M,K,V", [(1, 3, 5), (17, 65, 1001), (33, 64, 256), (65, 130, 777), (200, 72, 520),
                                   (300, 100, 1025), (2600, 40, 333), (4097, 24, 200)])
@pytest.mark.parametrize("offset", [0, 1])
def test_workspace_of_exactly_the_size_asked_for(M, K, V, offset):
    X, W, t = case(M, K, V, "bf16", seed=50, offset=offset)
    loss, lse, out = lb.lin_xent(X, W, t)
    dX, dW = torch.empty_like(X), torch.empty_like(W)
    lb.lin_xent_bwd(X, W, t, lse, dX, dW)
    for need in (lb.lin_xent_workspace(M, K, V), lb.lin_xent_bwd_workspace(M, K, V)):
        whole = torch.full((need + 8192,), 90, dtype=torch.uint8, device=DEV)
        ws = whole[4096:4096 + need]
        if need == lb.lin_xent_workspace(M, K, V):
            got = lb.lin_xent(X, W, t, ws=ws)
            for a, b in zip(got, (loss, lse, out)):
                assert torch.equal(a, b)
        if need == lb.lin_xent_bwd_workspace(M, K, V):
            gX, gW = torch.empty_like(X), torch.empty_like(W)
            lb.lin_xent_bwd(X, W, t, lse, gX, gW, ws=ws)
            assert torch.equal(gX, dX) and torch.equal(gW, dW)
        assert bool((whole[:4096] == 90).all()) and bool((whole[4096 + need:] == 90).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,V", [(1, 40), (70, 1000), (300, 3001)])
def test_loss_of_a_nearly_sure_row(M, V, dtype):
    """Exact logits: 1000 for the target, 984 for the others, so loss = log1p((V − 1) e^-16).  The
    sum is 2^d (1 + (V − 1) e^-16), where d is what rounding the maximum's exponent left (up to
    2^-14) and cancels: 2^d and the logarithm are off by a few u, and each of up to 128 additions
    beside the 1 by u (lse − z is off by 1000 u)."""
    X = torch.zeros(M, 8, dtype=T[dtype], device=DEV)
    X[:, 3] = 1.0
    W = torch.full((8, V), 984.0, dtype=T[dtype], device=DEV)
    hit = V // 3
    W[:, hit] = 1000.0
    t = torch.full((M,), hit, dtype=torch.int64, device=DEV)
    loss, lse, out = lb.lin_xent(X, W, t)
    ref = float(np.log1p((V - 1) * np.exp(-16.0)))
    bound = (128 + 32) * U
    assert bool(((loss.double() - ref).abs() <= bound).all()), float((loss.double() - ref).abs().max())
    assert abs(out[0].item() - ref) <= bound
    assert bool(((lse.double() - 1000.0 - ref).abs() <= 4 * U * 1000 + bound).all())


@pytest.mark.parametrize("M", [50, 900, 5000])
def test_row_weights_of_many_rows(M):
    """The largest |s| from a wave, from the rows themselves and from a launch of its own; weights of rows out
    of the loss may hold anything."""
    X, W, t = case(M, 40, 300, "f16", seed=9)
    w = torch.rand(M, device=DEV) * 2e-5
    big = int(((t >= 0).nonzero())[-1])
    w[big] = -3.0
    lse = lb.lin_xent(X, W, t)[1]
    poison = torch.where(t < 0, torch.tensor(float("nan"), device=DEV), w)
    poison[int((t < 0).nonzero()[0])] = float("inf")
    dX, dW = torch.empty_like(X), torch.empty_like(W)
    lb.lin_xent_bwd(X, W, t, lse, dX, dW, scale=64.0, row_scale=poison)
    check_backward(X, W, t, lse, dX, dW, "f16", 64.0, None, torch.where(t < 0, torch.zeros_like(w), w))


@pytest.mark.parametrize("M,K,V", [(1, 3, 5), (17, 65, 1001), (33, 64, 256), (65, 130, 777), (200, 72, 520),
                                   (300, 100, 1025), (2600, 40, 333), (600, 24, 20011)])
def test_a_workspace_full_of_nan(M, K, V):
    """What a workspace held before the call reaches nothing."""
    X, W, t = case(M, K, V, "bf16", seed=51)
    got = []
    for fill in (0, 255):
        ws = torch.full((max(lb.lin_xent_workspace(M, K, V), lb.lin_xent_bwd_workspace(M, K, V)),), fill,
                        dtype=torch.uint8, device=DEV)
        loss, lse, out = lb.lin_xent(X, W, t, ws=ws)
        ws.fill_(fill)
        dX, dW = torch.empty_like(X), torch.empty_like(W)
        lb.lin_xent_bwd(X, W, t, lse, dX, dW, ws=ws)
        got.append((loss, lse, out, dX, dW))
    for a, b in zip(*got):
        assert torch.equal(a, b) and not bool(a.isnan().any())
