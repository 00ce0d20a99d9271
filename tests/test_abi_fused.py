"""CPU: argument checks of the gated product, the cross entropy of a projection
and gradient clipping (everything is refused on the host before a launch), their
workspace queries, and the refusals of the torch forms."""
import ctypes

import pytest

import mixed_precision_matmul_gb300 as mpg

TOP = 2 ** 31 - 256


@pytest.fixture(scope="module", autouse=True)
def built():
    mpg.build()


def layer(tokens=40, hidden=64, inner=96, dtype=mpg.BF16, act=0, x=4096, wg=8192, wu=12288, ldx=None, ldwg=None, ldwu=None):
    return mpg.GatedLayer(tokens, hidden, inner, dtype, act, x, wg, wu, hidden if ldx is None else ldx,
                          hidden if ldwg is None else ldwg, hidden if ldwu is None else ldwu)


def forward(Y=4096, ldy=96, G=0, ldg=96, U=0, ldu=96, ws=4096, ws_bytes=1 << 40, **kw):
    return mpg.gated_gemm_raw(layer(**kw), Y, ldy, G, ldg, U, ldu, ws, ws_bytes, check=False)


def backward(dY=4096, lddy=96, G=0, ldg=96, U=0, ldu=96, dX=4096, lddx=64, dWg=4096, lddwg=64, dWu=4096, lddwu=64, ws=4096,
             ws_bytes=1 << 40, **kw):
    return mpg.gated_gemm_backward_raw(layer(**kw), dY, lddy, G, ldg, U, ldu, dX, lddx, dWg, lddwg, dWu, lddwu, ws, ws_bytes,
                                       check=False)


LAYER_FAULTS = [dict(tokens=-1), dict(hidden=-1), dict(inner=-1), dict(tokens=TOP + 1), dict(hidden=TOP + 1, ldx=TOP + 1),
                dict(inner=TOP + 1), dict(dtype=mpg.F32), dict(dtype=3), dict(act=3), dict(act=-1), dict(x=0), dict(wg=0),
                dict(wu=0), dict(x=4097), dict(ldx=63), dict(ldwg=63), dict(ldwu=63)]


@pytest.mark.parametrize("kw", LAYER_FAULTS + [dict(Y=0), dict(Y=4097), dict(ldy=95), dict(G=4096), dict(U=4096),
                                               dict(G=4096, U=4096, ldg=95), dict(G=4096, U=4096, ldu=95)])
def test_gated_gemm_refuses(kw):
    assert forward(**kw) == mpg.ERR_INVALID_ARG and mpg.last_error()


@pytest.mark.parametrize("kw", LAYER_FAULTS + [dict(dY=0), dict(dY=4097), dict(lddy=95), dict(G=4096), dict(dWg=0), dict(dWu=0),
                                               dict(dX=4097), dict(lddx=63), dict(lddwg=63), dict(lddwu=63),
                                               dict(G=4096, U=4096, ldu=95)])
def test_gated_backward_refuses(kw):
    assert backward(**kw) == mpg.ERR_INVALID_ARG and mpg.last_error()


def test_gated_workspaces():
    size = mpg.lib().mpg_gated_gemm_workspace_size
    back = mpg.lib().mpg_gated_gemm_backward_workspace_size
    assert size(ctypes.byref(layer())) == 0                                  # nothing has to be copied
    assert size(ctypes.byref(layer(hidden=65))) >= (40 + 2 * 96) * 72 * 2     # lines of 72 elements
    assert size(ctypes.byref(layer(tokens=1, hidden=65))) >= (1 + 2 * 96) * 72 * 2
    assert size(ctypes.byref(layer(tokens=1))) == 0
    assert size(None) == 0 and size(ctypes.byref(layer(tokens=-1))) == 0 and size(ctypes.byref(layer(tokens=0))) == 0
    need = back(ctypes.byref(layer()))
    assert need >= 2 * 40 * 96 * 2
    assert back(ctypes.byref(layer(tokens=0))) == 0
    for kw in (dict(ws=0), dict(ws_bytes=need - 1), dict(ws=4100)):
        assert backward(**kw) == mpg.ERR_WORKSPACE
    assert forward(hidden=65, ws=0) == mpg.ERR_WORKSPACE
    assert forward(hidden=65, ws_bytes=100) == mpg.ERR_WORKSPACE


def test_gated_without_elements():
    assert forward(tokens=0) == mpg.OK and forward(inner=0) == mpg.OK
    assert backward(hidden=0) == mpg.OK and backward(dX=0, dWg=0, dWu=0) == mpg.OK
    assert mpg.gated_gemm_raw(None, 4096, 64, check=False) == mpg.ERR_INVALID_ARG


def desc(tokens=40, hidden=64, vocab=100, dtype=mpg.BF16, x=4096, w=8192, ldx=None, ldw=None, target=4096, target_bytes=8,
         target_stride=1, ignore=-100):
    return mpg.VocabLoss(tokens, hidden, vocab, dtype, x, w, hidden if ldx is None else ldx, hidden if ldw is None else ldw,
                         target, target_bytes, target_stride, ignore)


def loss(out=4096, lse=4096, ws=4096, ws_bytes=1 << 40, **kw):
    return mpg.linear_cross_entropy_raw(desc(**kw), out, lse, ws, ws_bytes, check=False)


def loss_backward(lse=4096, dloss=4096, dX=4096, lddx=64, dW=4096, lddw=64, ws=4096, ws_bytes=1 << 40, **kw):
    return mpg.linear_cross_entropy_backward_raw(desc(**kw), lse, dloss, 1, dX, lddx, dW, lddw, ws, ws_bytes, check=False)


DESC_FAULTS = [dict(tokens=-1), dict(hidden=-1), dict(vocab=-1), dict(vocab=0), dict(hidden=0), dict(tokens=TOP + 1),
               dict(vocab=TOP + 1), dict(hidden=TOP + 1), dict(dtype=mpg.F32), dict(target=0), dict(target=4100), dict(x=0),
               dict(w=0), dict(w=4097), dict(ldx=63), dict(ldw=63), dict(target_bytes=2)]


@pytest.mark.parametrize("kw", DESC_FAULTS + [dict(out=0), dict(lse=0), dict(out=4097), dict(lse=4098)])
def test_loss_refuses(kw):
    assert loss(**kw) == mpg.ERR_INVALID_ARG and mpg.last_error()


@pytest.mark.parametrize("kw", DESC_FAULTS + [dict(lse=0), dict(dloss=0), dict(dloss=4097), dict(dX=4097), dict(lddx=63),
                                              dict(lddw=63)])
def test_loss_backward_refuses(kw):
    assert loss_backward(**kw) == mpg.ERR_INVALID_ARG and mpg.last_error()


def test_loss_workspaces():
    size = mpg.lib().mpg_linear_cross_entropy_workspace_size
    back = mpg.lib().mpg_linear_cross_entropy_backward_workspace_size
    need = size(ctypes.byref(desc()))
    assert need > 0 and loss(ws_bytes=need - 1) == mpg.ERR_WORKSPACE and loss(ws=0) == mpg.ERR_WORKSPACE
    need = back(ctypes.byref(desc()))
    assert need > 0 and loss_backward(ws_bytes=need - 1) == mpg.ERR_WORKSPACE and loss_backward(ws=0) == mpg.ERR_WORKSPACE
    # the logits' gradient is held in pieces, not whole: 2^14 tokens and 2^20 classes are 32 GB
    assert back(ctypes.byref(desc(tokens=2 ** 14, vocab=2 ** 20))) < 2 ** 30
    assert size(None) == 0 and back(ctypes.byref(desc(vocab=0))) == 0
    assert loss(tokens=0) == mpg.OK and loss_backward(dX=0, dW=0) == mpg.OK
    assert loss_backward(tokens=0, dW=0) == mpg.OK


def grad(g=4096, out=8192, count=16, g_dtype=mpg.F32, out_dtype=mpg.F32):
    return mpg.Grad(g, out, count, g_dtype, out_dtype)


def clip(grads, max_norm=1.0, norm=4096, eps=1e-6, ws=4096, ws_bytes=1 << 40):
    return mpg.clip_grad_norm_raw(grads, max_norm, norm, eps, ws, ws_bytes, check=False)


@pytest.mark.parametrize("grads,kw", [
    ([grad(count=-1)], {}), ([grad(g_dtype=3)], {}), ([grad(out_dtype=-1)], {}), ([grad(g=0)], {}), ([grad(out=0)], {}),
    ([grad(g=4098)], {}), ([grad(out=8193)], {}), ([grad(out=4096, out_dtype=mpg.BF16)], {}),
    ([grad()], dict(max_norm=-1.0)), ([grad()], dict(max_norm=float("nan"))), ([grad()], dict(eps=-1.0)),
    ([grad()], dict(eps=float("inf"))), ([grad()], dict(norm=0)), ([grad()], dict(norm=4098)),
    # results that overlap another's gradient or result, or a part of their own gradient
    ([grad(), grad()], {}), ([grad(out=4096), grad(out=4096)], {}), ([grad(out=4100)], {}),
    ([grad(), grad(g=8192 + 60, out=16384)], {}), ([grad(), grad(g=16384, out=8192 + 60)], {}),
    ([grad(g=16384, out=32768), grad(g=8192, out=16384 - 4)], {}),
])
def test_clip_refuses(grads, kw):
    assert clip(grads, **kw) == mpg.ERR_INVALID_ARG and mpg.last_error()


def test_clip_workspace_and_order():
    size = mpg.lib().mpg_clip_grad_norm_workspace_size
    table = (mpg.Grad * 2)(grad(), grad(g=16384, out=32768))
    need = size(2, table)
    assert need > 0
    assert clip(list(table), ws_bytes=need - 1) == mpg.ERR_WORKSPACE
    assert clip(list(table), ws=0) == mpg.ERR_WORKSPACE
    # neighbours, in any order, and one gradient read twice do not overlap
    for grads in ([grad(out=8192), grad(g=4096 + 64, out=8192 + 64)], [grad(g=4096 + 64, out=8192 + 64), grad()],
                  [grad(), grad(out=16384)], [grad(out=4096), grad(g=8192, out=8192)]):
        assert clip(grads, ws=0) == mpg.ERR_WORKSPACE
    assert size(-1, table) == 0


def test_torch_forms_refuse():
    import torch
    bf = torch.bfloat16
    x, w, t = torch.zeros(4, 8, dtype=bf), torch.zeros(6, 8, dtype=bf), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError):
        mpg.gated_gemm(x, w, w, act="relu")
    with pytest.raises(ValueError):
        mpg.gated_gemm(x, w, w)                       # not on a CUDA device
    with pytest.raises(ValueError):
        mpg.gated_gemm_backward(torch.zeros(4, 6, dtype=bf), x, w, w)
    with pytest.raises(ValueError):
        mpg.linear_cross_entropy(x, w, t)
    with pytest.raises(ValueError):
        mpg.linear_cross_entropy_backward(x, w, t, torch.zeros(4), torch.zeros(4))
    with pytest.raises(ValueError):
        mpg.clip_grad_norm([], 1.0)
    with pytest.raises(ValueError):
        mpg.clip_grad_norm([x], 1.0)
    with pytest.raises(ValueError):
        mpg.clip_grad_norm([x], 1.0, out=[])


def test_dense_memory_orders():
    import torch
    from mixed_precision_matmul_gb300.clip import _dense
    t = torch.zeros(4, 6, 8)
    assert _dense(t) and _dense(t.permute(2, 0, 1)) and _dense(t[:0]) and _dense(t[0, 0, 0]) and _dense(t[1:2].permute(1, 0, 2))
    assert not _dense(t[:, 1:]) and not _dense(t[:, :, ::2]) and not _dense(t[0].expand(4, 6, 8)) and not _dense(t[:, :, 0])
