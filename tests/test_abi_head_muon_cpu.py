"""Refusals of the loss head and Muon entry points on the host, before anything is launched
(CPU only: no call here reaches the GPU), and their no-op cases."""
import ctypes

import pytest
import torch

import linear_layer_backward_bwd_amd as lb

NULL = None
P = ctypes.c_void_p(4096)        # never dereferenced: every call below is refused on the host
BIG = 1 << 40


def xent(M=8, K=64, V=100, dtype=1, X=P, W=P, target=P, loss=P, lse=P, out=P, ws=P, nbytes=BIG):
    return lb.library().lin_xent(X, W, target, loss, lse, out, M, K, V, dtype, ws, nbytes)


def xent_bwd(M=8, K=64, V=100, dtype=1, X=P, W=P, target=P, lse=P, dX=P, dW=P, ws=P, nbytes=BIG):
    return lb.library().lin_xent_bwd(X, W, target, lse, NULL, NULL, 1.0, dX, dW, M, K, V, dtype, ws, nbytes)


COMMON = [
    (dict(dtype=0), -2), (dict(dtype=3), -2), (dict(dtype=-1), -2),
    (dict(M=-1), -1), (dict(K=0), -1), (dict(V=0), -1), (dict(K=-4), -1), (dict(V=-4), -1),
    (dict(M=1 << 27), -1), (dict(K=1 << 22), -1), (dict(V=1 << 22), -1),
    (dict(X=NULL), -1), (dict(W=NULL), -1), (dict(target=NULL), -1), (dict(lse=NULL), -1),
    (dict(ws=NULL), -1), (dict(ws=ctypes.c_void_p(4104)), -1), (dict(nbytes=0), -1), (dict(nbytes=-1), -1),
]


@pytest.mark.parametrize("over,code", COMMON + [(dict(loss=NULL), -1), (dict(out=NULL), -1),
                                                (dict(M=0, out=NULL), -1)])
def test_lin_xent_rejects_on_host(over, code):
    assert xent(**over) == code
    assert lb.lb_last_error().startswith("lin_xent")


@pytest.mark.parametrize("over,code", COMMON)
def test_lin_xent_bwd_rejects_on_host(over, code):
    assert xent_bwd(**over) == code
    assert lb.lb_last_error().startswith("lin_xent_bwd")


def test_lin_xent_bwd_without_outputs_is_a_noop():
    assert xent_bwd(dX=NULL, dW=NULL, ws=NULL, nbytes=0) == 0
    assert lb.lb_last_error() == ""


@pytest.mark.parametrize("entry", [xent, xent_bwd])
@pytest.mark.parametrize("M,K,V", [(1, 1, 1), (8, 64, 100), (300, 128, 1001), (5000, 64, 40000)])
def test_a_byte_too_few_is_refused(entry, M, K, V):
    need = lb.lin_xent_workspace(M, K, V) if entry is xent else lb.lin_xent_bwd_workspace(M, K, V)
    assert need > 0
    assert entry(M=M, K=K, V=V, nbytes=need - 1) == -1
    assert str(need) in lb.lb_last_error()


def test_workspace_queries():
    assert lb.lin_xent_workspace(0, 64, 100) == 0 and lb.lin_xent_bwd_workspace(0, 64, 100) == 0
    for bad in ((-1, 4, 4), (4, 0, 4), (4, 4, 0), (4, 1 << 22, 4), (1 << 27, 4, 4)):
        with pytest.raises(RuntimeError):
            lb.lin_xent_workspace(*bad)
        with pytest.raises(RuntimeError):
            lb.lin_xent_bwd_workspace(*bad)
    # the gradient's workspace holds a bounded piece of the logits, not all of them
    assert lb.lin_xent_bwd_workspace(16384, 4096, 131072) < 2 * 16384 * 131072 * 2 // 3
    assert lb.lin_xent_workspace(16384, 4096, 131072) < 600 << 20
    for bad in ((-1, 4, 4), (1, -1, 4), (1, 4, 1 << 20), (65536, 4, 4)):
        with pytest.raises(RuntimeError):
            lb.muon_workspace(*bad)
    for empty in ((0, 4, 4), (2, 0, 4), (2, 4, 0)):
        assert lb.muon_workspace(*empty) == 0


def orth(G=P, gd=0, O=P, od=1, batch=2, K=64, N=32, steps=5, ws=P, nbytes=BIG):
    return lb.library().muon_orth(G, gd, O, od, batch, K, N, steps, ws, nbytes)


def step(W=P, g=P, gd=0, mom=ctypes.c_void_p(8192), batch=2, K=64, N=32, beta=0.9, steps=5, w16=NULL, wd16=0, ws=P,
         nbytes=BIG):
    return lb.library().muon_step(W, g, gd, mom, batch, K, N, 1e-3, beta, 0.1, 1.0, steps, 1, 1.0, NULL, NULL,
                                  w16, wd16, ws, nbytes)


SIZES = [(dict(batch=-1), -1), (dict(batch=65536), -1), (dict(K=-1), -1), (dict(N=-1), -1), (dict(K=1 << 20), -1),
         (dict(N=1 << 20), -1), (dict(steps=0), -1), (dict(steps=-3), -1), (dict(gd=3), -2), (dict(gd=-1), -2),
         (dict(ws=NULL), -1), (dict(ws=ctypes.c_void_p(4100)), -1), (dict(nbytes=0), -1)]


@pytest.mark.parametrize("over,code", SIZES + [(dict(od=0), -2), (dict(od=7), -2), (dict(G=NULL), -1),
                                               (dict(O=NULL), -1)])
def test_muon_orth_rejects_on_host(over, code):
    assert orth(**over) == code
    assert lb.lb_last_error().startswith("muon_orth")


@pytest.mark.parametrize("over,code", SIZES + [
    (dict(W=NULL), -1), (dict(g=NULL), -1), (dict(mom=NULL), -1), (dict(beta=1.0), -1), (dict(beta=-0.1), -1),
    (dict(beta=float("nan")), -1), (dict(w16=ctypes.c_void_p(64), wd16=0), -2), (dict(w16=P, wd16=1), -1)])
def test_muon_step_rejects_on_host(over, code):
    assert step(**over) == code
    assert lb.lb_last_error().startswith("muon_step")


@pytest.mark.parametrize("over", [dict(batch=0), dict(K=0), dict(N=0)])
def test_empty_muon_calls_are_noops(over):
    assert orth(**over) == 0 and step(**over) == 0
    assert orth(**over, ws=NULL, nbytes=0) == 0 and step(**over, ws=NULL, nbytes=0) == 0


def test_a_byte_too_few_is_refused_by_muon():
    need = lb.muon_workspace(2, 64, 32)
    assert orth(nbytes=need - 1) == -1 and step(nbytes=need - 1) == -1


def test_head_binding_checks_types_and_shapes():
    X, W = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(8, 10, dtype=torch.bfloat16)
    t, v = torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    for bad in (lambda: lb.lin_xent(X.float(), W.float(), t), lambda: lb.lin_xent(X, W.half(), t),
                lambda: lb.lin_xent(X, W, t, out=torch.zeros(3)),
                lambda: lb.lin_xent_bwd(X, W, t, v, X, W, d_scale=torch.zeros(2))):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: lb.lin_xent(X, W[:7], t), lambda: lb.lin_xent(X[0], W, t), lambda: lb.lin_xent(X, W, t.int()),
                lambda: lb.lin_xent(X, W, t[:3]), lambda: lb.lin_xent(X, W, t, loss=v.double()),
                lambda: lb.lin_xent_bwd(X, W, t, v[:2], X, W), lambda: lb.lin_xent_bwd(X, W, t, None, X, W),
                lambda: lb.lin_xent_bwd(X, W, t, v, X[:2], W), lambda: lb.lin_xent_bwd(X, W, t, v, X, W.half()),
                lambda: lb.lin_xent(X, W, t)):      # on the CPU
        with pytest.raises(ValueError):
            bad()


def test_muon_binding_checks_types_and_shapes():
    G = torch.zeros(2, 4, 6)
    for bad in (lambda: lb.muon_orth(G.int()), lambda: lb.muon_orth(G, out=torch.zeros(2, 4, 6)),
                lambda: lb.muon_orth(G, out=torch.zeros(2, 4, 6, dtype=torch.float16), dtype=torch.bfloat16),
                lambda: lb.muon_step(G.half(), G, G, 1e-3, 0.9, 0.1), lambda: lb.muon_step(G, G.int(), G, 1e-3, 0.9, 0.1),
                lambda: lb.muon_step(G, G, G.clone(), 1e-3, 0.9, 0.1, w16=G),
                lambda: lb.muon_step(G, G, G, 1e-3, 0.9, 0.1, clip=torch.zeros(2)),
                lambda: lb.muon_step(G, G, G, 1e-3, 0.9, 0.1, skip=torch.zeros(1))):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: lb.muon_orth(G[0, 0]), lambda: lb.muon_orth(G, out=torch.zeros(2, 4, 5, dtype=torch.float16)),
                lambda: lb.muon_step(G, G[0], G, 1e-3, 0.9, 0.1),
                lambda: lb.muon_step(G, G, G, 1e-3, 0.9, 0.1, w16=torch.zeros(4, 6, dtype=torch.float16)),
                lambda: lb.muon_orth(G)):           # on the CPU
        with pytest.raises(ValueError):
            bad()
