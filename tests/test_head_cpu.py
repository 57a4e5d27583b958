"""Refusals and sizes of the output layer's losses (no GPU needed: every check comes before the first HIP call)."""
import ctypes
import os

import pytest
import torch

from bit_quantized_lora_02_amd import binding as B

bf = torch.bfloat16
OK = ctypes.c_void_p(0x10000)  # aligned, never dereferenced: every check below fails first
MIS = ctypes.c_void_p(0x10008)
ODD = ctypes.c_void_p(0x10002)
BIG = 1 << 62


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from bit_quantized_lora_02_amd import build
        build.build()
    return B.load_library()


def ce(lib, X=OK, T=8, W=OK, V=100, K=64, labels=OK, weight=None, loss=OK, dX=OK, dW=None, ws=OK, nb=BIG):
    return lib.qlora_head_ce(X, T, W, V, K, labels, weight, loss, dX, dW, ws, nb, None)


def kd(lib, X=OK, T=8, W=OK, V=100, K=64, index=OK, logit=OK, k=4, tau=1.0, weight=None, loss=OK, dX=OK, dW=None, ws=OK,
       nb=BIG):
    return lib.qlora_head_distill(X, T, W, V, K, index, logit, k, tau, weight, loss, dX, dW, ws, nb, None)


SHARED = [
    (dict(T=-1), "T must"), (dict(T=(1 << 22) + 1), "T must"),
    (dict(V=0), "n_vocab"), (dict(V=(1 << 22) + 1), "n_vocab"),
    (dict(K=0), "multiple of 8"), (dict(K=60), "multiple of 8"), (dict(K=(1 << 22) + 8), "2^22"),
    (dict(V=1 << 21, K=1 << 14), "2^34"), (dict(T=1 << 20, K=1 << 11), "2^31"),
    (dict(X=None), "X and loss"), (dict(loss=None), "X and loss"), (dict(W=None), "W must"),
    (dict(X=MIS), "16-byte"), (dict(W=MIS), "16-byte"), (dict(dX=MIS), "16-byte"), (dict(dW=MIS), "16-byte"),
    (dict(loss=ODD), "4-byte"), (dict(weight=ODD), "4-byte"),
    (dict(ws=None), "workspace"), (dict(ws=MIS), "workspace"),
]


@pytest.mark.parametrize("kw,text", SHARED + [(dict(labels=None), "labels"), (dict(labels=ODD), "8-byte")])
def test_cross_entropy_refuses(lib, kw, text):
    assert ce(lib, **kw) == B.QLORA_EINVAL
    assert text in lib.qlora_last_error().decode()


@pytest.mark.parametrize("kw,text", SHARED + [
    (dict(index=None), "index"), (dict(logit=None), "logit"), (dict(index=ODD), "4-byte"), (dict(logit=ODD), "4-byte"),
    (dict(k=0), "k must"), (dict(k=257), "k must"), (dict(tau=0.0), "tau"), (dict(tau=-1.0), "tau"), (dict(tau=9e-5), "tau"), (dict(tau=1.1e4), "tau"),
    (dict(tau=float("nan")), "tau"), (dict(tau=float("inf")), "tau")])
def test_distillation_refuses(lib, kw, text):
    assert kd(lib, **kw) == B.QLORA_EINVAL
    assert text in lib.qlora_last_error().decode()


def test_workspace_is_checked_and_bounded(lib):
    nb = B.head_workspace_bytes(8, 100, 64, 0, True, False)
    assert ce(lib, nb=nb - 1) == B.QLORA_EWORKSPACE
    assert kd(lib, nb=nb) == B.QLORA_EWORKSPACE  # its targets need more
    c = ctypes.c_size_t()
    assert lib.qlora_head_workspace_bytes(8, 100, 64, -1, 1, 0, ctypes.byref(c)) == B.QLORA_EINVAL
    assert lib.qlora_head_workspace_bytes(8, 100, 64, 257, 1, 0, ctypes.byref(c)) == B.QLORA_EINVAL
    assert lib.qlora_head_workspace_bytes(8, 100, 60, 0, 1, 0, ctypes.byref(c)) == B.QLORA_EINVAL
    assert lib.qlora_head_workspace_bytes(8, 100, 64, 0, 1, 0, None) == B.QLORA_EINVAL
    # scoring keeps only statistics, 8 bytes per row and 64 columns, and a copy of X
    T, V = 8192, 131072
    assert B.head_workspace_bytes(T, V, 4096, 0, False, False) < T * V / 8 + 2 * T * 4096 + (1 << 20)
    # gradients hold a block of at most 1 GiB and the dX product's partial sums, however many rows there are
    for T in (4096, 65536, 1 << 18):
        assert B.head_workspace_bytes(T, V, 4096, 0, True, False) < (3 << 29) + (2 * 4096 + 32) * T


def test_no_rows_and_no_gpu(lib):
    """Valid arguments get as far as the device check (QLORA_ENODEV without a GPU)."""
    if torch.cuda.is_available():
        pytest.skip("the fake addresses above must not reach a GPU")
    assert ce(lib) == B.QLORA_ENODEV and kd(lib) == B.QLORA_ENODEV
    assert ce(lib, T=0, X=None, labels=None, loss=None, dX=None) == B.QLORA_ENODEV


def args(T=8, V=100, K=64):
    return torch.zeros(T, K, dtype=bf), torch.zeros(V, K, dtype=bf), torch.zeros(T, dtype=torch.int64)


@pytest.mark.parametrize("change,exc", [
    (dict(labels=torch.zeros(8, dtype=torch.int32)), TypeError),
    (dict(labels=torch.zeros(7, dtype=torch.int64)), TypeError),  # not on a GPU comes first
    (dict(labels=None), TypeError),
    (dict(W=torch.zeros(100, 72, dtype=bf)), ValueError),
    (dict(W=torch.zeros(100, 64)), TypeError),
    (dict(X=torch.zeros(8, 64, dtype=torch.float16)), TypeError),
    (dict(X=torch.zeros(64, dtype=bf)), ValueError),
    (dict(weight=torch.zeros(7)), ValueError),
    (dict(weight=torch.zeros(8, dtype=torch.float64)), TypeError),
    (dict(weight=torch.zeros(16)[::2]), ValueError),
    (dict(outs=(torch.zeros(9), None, None)), ValueError),
    (dict(outs=(torch.zeros(8), torch.zeros(8, 72, dtype=bf), None)), ValueError),
    (dict(outs=(torch.zeros(8), None, torch.zeros(100, 64))), TypeError),
    (dict(ws=torch.zeros(64, 2, dtype=torch.uint8).t()), ValueError),
    (dict(), TypeError),  # a valid call is refused as not on a GPU
])
def test_binding_refuses(lib, change, exc):
    X, W, y = args()
    kw = dict(X=X, W=W, labels=y) | change
    with pytest.raises(exc):
        B.head_ce(**kw)


@pytest.mark.parametrize("change,exc", [
    (dict(index=torch.zeros(8, 4, dtype=torch.int64)), TypeError),
    (dict(index=torch.zeros(8, dtype=torch.int32)), TypeError),
    (dict(logit=torch.zeros(8, 4, dtype=torch.float64)), TypeError),
    (dict(index=torch.zeros(8, 0, dtype=torch.int32), logit=torch.zeros(8, 0)), ValueError),
    (dict(index=torch.zeros(8, 257, dtype=torch.int32), logit=torch.zeros(8, 257)), ValueError),
    (dict(), TypeError),
])
def test_distill_binding_refuses(lib, change, exc):
    X, W, _ = args()
    kw = dict(X=X, W=W, index=torch.zeros(8, 4, dtype=torch.int32), logit=torch.zeros(8, 4)) | change
    with pytest.raises(exc):
        B.head_distill(**kw)


def test_distill_function_refuses_teacher_gradients():
    X, W = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(5, 64, dtype=torch.bfloat16)
    index, logit = torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 1, requires_grad=True)
    with pytest.raises(ValueError, match="teacher's logits get no gradient"):
        B.HeadDistillFn.apply(X, W, index, logit)


@pytest.mark.parametrize("op", ["ce", "kd"])
@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_functions_form_no_gradient_where_none_is_recorded(monkeypatch, op, mode):
    """Scoring with trained operands: neither dX nor dW is asked for with gradients off, both are with them on (head_ce and
    head_distill stand-ins on the CPU record what they are asked for)."""
    T, V, K = 3, 5, 8
    asked = []

    def call(X, W, *targets, need_dx=True, need_dw=False):
        asked.append((need_dx, need_dw))
        return torch.ones(T), torch.full((T, K), 2.0, dtype=bf) if need_dx else None, \
            torch.full((V, K), 3.0, dtype=bf) if need_dw else None

    monkeypatch.setattr(B, "head_ce", call)
    monkeypatch.setattr(B, "head_distill", call)
    X, W, weight = torch.zeros(T, K, dtype=bf), torch.zeros(V, K, dtype=bf), torch.full((T,), 0.5)
    for t in (X, W, weight):
        t.requires_grad_(True)
    index, logit = torch.zeros(T, 1, dtype=torch.int32), torch.zeros(T, 1)
    if op == "ce":
        calls = [lambda: B.HeadCEFn.apply(X, W, torch.zeros(T, dtype=torch.int64)),
                 lambda: B.HeadCEFn.apply(X, W, torch.zeros(T, dtype=torch.int64), weight)]
    else:
        calls = [lambda: B.HeadDistillFn.apply(X, W, index, logit),
                 lambda: B.HeadDistillFn.apply(X, W, index, logit, 2.0, weight)]
    for fn, total in zip(calls, (3.0, 1.5)):
        with mode():
            got, loss = fn()
        assert asked.pop() == (False, False) and not got.requires_grad and got == total and loss.shape == (T,)
        got, loss = fn()
        assert asked.pop() == (True, True) and got.requires_grad and not loss.requires_grad and got == total
        got.backward()
        assert (X.grad == 2.0).all() and (W.grad == 3.0).all()
        assert weight.grad is None if total == 3.0 else (weight.grad == 1.0).all()
        X.grad = W.grad = None
    if op == "kd":  # a teacher's logits that ask for a gradient are refused only where one would be recorded
        logit.requires_grad_(True)
        with mode():
            calls[0]()
        with pytest.raises(ValueError, match="teacher's logits get no gradient"):
            calls[0]()


@pytest.mark.parametrize("T", [1, 300, 4096, 8192, 65536, 1 << 18])
@pytest.mark.parametrize("V,K", [(1000, 256), (32000, 4096), (128256, 4096), (1 << 20, 1024)])
def test_workspace_holds_what_the_header_names(T, V, K):
    """Every part of the workspace, as the header lists it, with and without dX and dW."""
    lde, rows = -(-V // 128) * 128, T + 15
    most = min(T + 15, max(256, (1 << 30) // (2 * lde)) + 15)  # rows of a block of E
    x = -(-K // 128) * 256 * rows
    few = 40 << 20  # binary32 sums of a product with at most half as many output tiles as workgroups
    lists = 32 * T + 4096
    for dx in (False, True):
        for dw in (False, True):
            grad = dx or dw
            e = 2 * lde * most * grad
            stat = 8 * (V // 64 + 1) * most if grad else max(1 << 30, 256 * 8 * (V // 64 + 1))
            parts = 4 * min(32 * most * K, 4 * 256 * 384 * 256) * dx
            copy = 2 * (most + 128) * K * dw
            carried = 4 * V * K * (dw and T > most)
            bound = x + e + stat + lists + parts + copy + carried + few * (1 + dw)
            got = B.head_workspace_bytes(T, V, K, 0, dx, dw)
            assert got <= bound, (dx, dw, got, bound)
            if carried:
                assert got > carried
