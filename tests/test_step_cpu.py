"""Refusals and sizes of the embedding and the layer norm (no GPU needed: every check comes before the first HIP call)."""
import ctypes
import os

import pytest
import torch

from bit_quantized_lora_02_amd import binding as B

bf = torch.bfloat16
OK = 0x10000  # aligned, never dereferenced: every check below fails first
MIS = 0x10008
ODD = 0x10002
BIG = 1 << 62


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from bit_quantized_lora_02_amd import build
        build.build()
    return B.load_library()


def embed(lib, tokens=OK, T=8, W=OK, V=100, D=64, scale=1.0, Y=OK):
    return lib.qlora_embed(tokens, T, W, V, D, scale, Y, None)


def embed_bwd(lib, tokens=OK, dY=OK, T=8, V=100, D=64, scale=1.0, acc=0, dW=OK, ws=OK, nb=BIG):
    return lib.qlora_embed_bwd(tokens, dY, T, V, D, scale, acc, dW, ws, nb, None)


def norm(lib, X=OK, T=8, D=64, w=OK, b=None, kind=1, eps=1e-5, Y=OK, mean=None, rstd=None):
    return lib.qlora_layer_norm(X, T, D, w, b, kind, eps, Y, mean, rstd, None)


def norm_bwd(lib, X=OK, dY=OK, T=8, D=64, w=OK, kind=1, mean=OK, rstd=OK, dX=OK, dw=OK, db=OK, ws=OK, nb=BIG):
    return lib.qlora_layer_norm_bwd(X, dY, T, D, w, kind, mean, rstd, dX, dw, db, ws, nb, None)


EMBED_SIZES = [(dict(T=-1), "T must"), (dict(T=(1 << 22) + 1), "T must"), (dict(V=0), "n_vocab"),
               (dict(V=(1 << 22) + 1), "n_vocab"), (dict(D=0), "multiple of 8"), (dict(D=60), "multiple of 8"),
               (dict(D=(1 << 22) + 8), "2^22"), (dict(V=1 << 21, D=1 << 14), "2^34"), (dict(T=1 << 20, D=1 << 12), "2^32"),
               (dict(tokens=None), "tokens"), (dict(tokens=0x10004), "8-byte")]
NORM_SIZES = [(dict(T=-1), "T must"), (dict(T=(1 << 22) + 1), "T must"), (dict(D=0), "multiple of 8"),
              (dict(D=60), "multiple of 8"), (dict(D=32776), "32768"), (dict(T=1 << 20, D=1 << 12), "2^32"),
              (dict(kind=2), "weight_type"), (dict(kind=-1), "weight_type"), (dict(X=None), "X"), (dict(X=MIS), "16-byte"),
              (dict(w=None), "weight"), (dict(w=MIS), "16-byte"), (dict(mean=ODD), "4-byte"), (dict(rstd=ODD), "4-byte")]


@pytest.mark.parametrize("call,kw,text", [(f, *c) for f, cases in (
    (embed, EMBED_SIZES + [(dict(W=None), "W must"), (dict(W=MIS), "16-byte"), (dict(Y=None), "Y"), (dict(Y=MIS), "16-byte")]),
    (embed_bwd, EMBED_SIZES + [(dict(dY=None), "dY"), (dict(dY=MIS), "16-byte"), (dict(dW=None), "dW"),
                               (dict(dW=MIS), "16-byte"), (dict(ws=None), "workspace"), (dict(ws=MIS), "workspace")]),
    (norm, NORM_SIZES + [(dict(Y=None), "Y"), (dict(Y=MIS), "16-byte"), (dict(b=MIS), "16-byte"), (dict(eps=-1.0), "eps"),
                         (dict(eps=float("nan")), "eps"), (dict(eps=float("inf")), "eps")]),
    (norm_bwd, NORM_SIZES + [(dict(dY=None), "dY"), (dict(dY=MIS), "16-byte"), (dict(dX=MIS), "16-byte"),
                             (dict(dw=MIS), "16-byte"), (dict(db=MIS), "16-byte"), (dict(mean=None), "mean"),
                             (dict(rstd=None), "rstd"), (dict(ws=None), "workspace"), (dict(ws=MIS), "workspace")]),
) for c in cases])
def test_refuses(lib, call, kw, text):
    assert call(lib, **kw) == B.QLORA_EINVAL
    assert text in lib.qlora_last_error().decode()


def test_workspaces(lib):
    c = ctypes.c_size_t()
    for T in (0, 1, 8, 9, 8192, 8193, 1 << 22):
        nb = B.embed_workspace_bytes(T, 64)
        assert nb >= T * (8 if T <= 8192 else 16)
        assert nb <= 16 * T + 2 * 64 * 4 * (T / (8 if T <= 2048 else 16) + 1) + 2048
        if nb:
            assert embed_bwd(lib, T=T, nb=nb - 1) == B.QLORA_EWORKSPACE
    for T, D in ((0, 8), (1, 32768), (1 << 20, 64), (4096, 4096)):
        nb = B.layer_norm_workspace_bytes(T, D)
        assert 0 < nb <= 256 * 2 * D * 4
        assert norm_bwd(lib, T=T, D=D, nb=nb - 1) == B.QLORA_EWORKSPACE
    assert lib.qlora_embed_workspace_bytes(8, 60, ctypes.byref(c)) == B.QLORA_EINVAL
    assert lib.qlora_embed_workspace_bytes(8, 64, None) == B.QLORA_EINVAL
    assert lib.qlora_layer_norm_workspace_bytes(8, 60, ctypes.byref(c)) == B.QLORA_EINVAL
    assert lib.qlora_layer_norm_workspace_bytes(8, 64, None) == B.QLORA_EINVAL


def test_valid_calls_reach_the_device_check(lib):
    if torch.cuda.is_available():
        pytest.skip("the fake addresses above must not reach a GPU")
    for rc in (embed(lib), embed_bwd(lib), norm(lib), norm_bwd(lib), embed(lib, T=0, tokens=None, Y=None),
               embed_bwd(lib, T=0, tokens=None, dY=None), norm(lib, T=0, X=None, Y=None),
               norm_bwd(lib, T=0, X=None, dY=None, mean=None, rstd=None), norm_bwd(lib, dw=None, db=None, ws=None, nb=0)):
        assert rc == B.QLORA_ENODEV


TOKENS, W, X, G, STAT = (torch.zeros(8, dtype=torch.int64), torch.zeros(100, 64, dtype=bf), torch.zeros(8, 64, dtype=bf),
                         torch.zeros(64), torch.zeros(8))


@pytest.mark.parametrize("fn,kw,exc", [
    (B.embed, dict(tokens=TOKENS.int()), TypeError), (B.embed, dict(tokens=TOKENS.view(2, 4)), TypeError),
    (B.embed, dict(tokens=[1, 2]), TypeError), (B.embed, dict(W=W.float()), TypeError), (B.embed, dict(W=W[0]), ValueError),
    (B.embed, dict(out=torch.zeros(8, 72, dtype=bf)), ValueError), (B.embed, dict(out=torch.zeros(8, 64)), TypeError),
    (B.embed, dict(out=torch.zeros(64, 8, dtype=bf).t()), ValueError), (B.embed, {}, TypeError),  # (not on a GPU)
    (B.embed_bwd, dict(tokens=TOKENS[:7]), ValueError), (B.embed_bwd, dict(dY=X.half()), TypeError),
    (B.embed_bwd, dict(accumulate=True), ValueError), (B.embed_bwd, dict(dW=torch.zeros(99, 64, dtype=bf)), ValueError),
    (B.embed_bwd, dict(ws=torch.zeros(64, 2, dtype=torch.uint8).t()), ValueError), (B.embed_bwd, {}, TypeError),
    (B.layer_norm, dict(X=X.float()), TypeError), (B.layer_norm, dict(X=X[0]), ValueError),
    (B.layer_norm, dict(weight=G[:63]), ValueError), (B.layer_norm, dict(weight=G.double()), TypeError),
    (B.layer_norm, dict(weight=None), TypeError), (B.layer_norm, dict(bias=G.to(bf)), TypeError),
    (B.layer_norm, dict(weight=torch.zeros(128)[::2]), ValueError),
    (B.layer_norm, dict(outs=(torch.zeros(9, 64, dtype=bf), None, None)), ValueError),
    (B.layer_norm, dict(outs=(X, STAT.double(), None)), TypeError), (B.layer_norm, {}, TypeError),
    (B.layer_norm_bwd, dict(dY=X[:7]), ValueError), (B.layer_norm_bwd, dict(mean=STAT[:7]), ValueError),
    (B.layer_norm_bwd, dict(rstd=STAT.to(bf)), TypeError), (B.layer_norm_bwd, dict(outs=(None, G.to(bf), None)), TypeError),
    (B.layer_norm_bwd, {}, TypeError),
])
def test_binding_refuses(lib, fn, kw, exc):
    base = {B.embed: dict(tokens=TOKENS, W=W), B.embed_bwd: dict(tokens=TOKENS, dY=X, n_vocab=100),
            B.layer_norm: dict(X=X, weight=G), B.layer_norm_bwd: dict(X=X, dY=X, weight=G, mean=STAT, rstd=STAT)}[fn]
    with pytest.raises(exc):
        fn(**(base | kw))


def test_functions_ask_for_the_gradients_that_are_needed(monkeypatch):
    asked = []
    monkeypatch.setattr(B, "layer_norm", lambda X, w, b, eps: (X.clone(), STAT, STAT))
    monkeypatch.setattr(B, "layer_norm_bwd", lambda X, dY, w, m, r, *need: asked.append(need) or tuple(
        torch.ones_like(t) if n else None for n, t in zip(need, (X, w, w))))
    monkeypatch.setattr(B, "embed", lambda tokens, W, scale: W[tokens] * scale)
    monkeypatch.setattr(B, "embed_bwd", lambda tokens, dY, V, scale: asked.append((V, scale)) or torch.ones(V, 64, dtype=bf))
    for need in ((True, True, True), (False, True, False), (True, False, False)):
        x, w, b = (t.clone().requires_grad_(n) for n, t in zip(need, (X, G, G)))
        B.LayerNormFn.apply(x, w, b).sum().backward()
        assert asked.pop() == need
        assert [t.grad is not None for t in (x, w, b)] == list(need)
    w = W.clone().requires_grad_(True)
    B.EmbedFn.apply(TOKENS, w, 2.0).sum().backward()
    assert asked.pop() == (100, 2.0) and (w.grad == 1).all()


def test_embed_function_refuses_a_scale_that_asks_for_a_gradient(monkeypatch):
    monkeypatch.setattr(B, "embed", lambda tokens, W, scale: W[tokens] * float(scale))
    w, scale = W.clone().requires_grad_(True), torch.tensor(2.0, requires_grad=True)
    with pytest.raises(ValueError, match="scale gets no gradient"):
        B.EmbedFn.apply(TOKENS, w, scale)
    assert B.EmbedFn.apply(TOKENS, w, scale.detach()).requires_grad
    with torch.no_grad():
        assert not B.EmbedFn.apply(TOKENS, w, scale).requires_grad


def test_embed_function_keeps_the_forwards_scale(monkeypatch):
    asked = []
    monkeypatch.setattr(B, "embed", lambda tokens, W, scale: W[tokens] * float(scale))
    monkeypatch.setattr(B, "embed_bwd", lambda tokens, dY, V, scale: asked.append(float(scale)) or torch.ones(V, 64, dtype=bf))
    scale = torch.tensor(2.0)
    Y = B.EmbedFn.apply(TOKENS, W.clone().requires_grad_(True), scale)
    scale.fill_(5.0)
    Y.sum().backward()
    assert asked == [2.0]


@pytest.mark.parametrize("T,D,f32", [(1, 8, True), (37, 264, True), (90, 72, False)])
def test_norm_references_are_the_definitions_gradients(T, D, f32):
    """The formulas that the kernels are held against, entry by entry against torch's gradients of the definition in
    binary64; a term that is left out, or has the other sign, is past the bounds."""
    from test_step_gpu import norm_bwd_reference, norm_inputs, norm_reference
    X, dY, w, b = norm_inputs(T, D, f32, T + D)
    leaves = [t.double().requires_grad_(True) for t in (X, w, b)]
    Y = torch.nn.functional.layer_norm(leaves[0], (D,), leaves[1], leaves[2], 1e-5)
    Y.backward(dY.double())
    y, mean, rstd, *_ = norm_reference(X, w, b, 1e-5)
    assert (y - Y).abs().max() <= 1e-11 * Y.abs().max()
    want, bounds = norm_bwd_reference(X, dY, w, mean, rstd, f32)
    for x, t in zip(want, leaves):
        assert (x - t.grad).abs().max() <= 1e-10 * t.grad.abs().max()
    xh = (X.double() - mean[:, None]) * rstd[:, None]
    g, r, bound = dY.double() * w.double(), rstd[:, None], 1.1 * bounds[0]
    one, two = r * g.mean(1, keepdim=True), r * xh * (g * xh).mean(1, keepdim=True)
    for off in (one, two, 2 * one, 2 * two):
        assert (off.abs() > bound).double().mean() > 0.5
    assert ((0.02 * want[1]).abs() > 1.1 * bounds[1]).double().mean() > 0.5
    assert ((0.02 * want[2]).abs() > 1.1 * bounds[2]).double().mean() > 0.5


@pytest.mark.parametrize("T,V,D,kind", [(37, 50, 264, "any"), (200, 7, 8, "runs")])
def test_embedding_reference_is_the_definitions_gradient(T, V, D, kind):
    from test_step_gpu import embed_bwd_reference, tokens_of
    tokens, dY = tokens_of(kind, T, V, T), torch.randn(T, D, generator=torch.Generator().manual_seed(T)).to(bf)
    w = torch.zeros(V, D, dtype=torch.float64, requires_grad=True)
    rows = torch.cat([w, torch.zeros(1, D, dtype=torch.float64)])[torch.where((tokens >= 0) & (tokens < V), tokens, V)]
    (rows * 1.5).backward(dY.double())
    dW, bound, named = embed_bwd_reference(tokens, dY, V, 1.5)
    assert (dW - w.grad).abs().max() <= 1e-12 * w.grad.abs().max()
    assert ((0.02 * dW).abs() > 1.1 * bound)[named].double().mean() > 0.5
