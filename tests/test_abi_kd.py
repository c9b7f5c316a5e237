"""Host checks of the distillation from top logits (CPU only: no kernel is ever launched here)."""
import pytest
import torch

lx = pytest.importorskip("cross_entropy_tv_amd", reason="HIP library not built")
L = lx.lib

A = 1 << 32  # fake, never dereferenced device addresses
BAD, ALIAS, WS = lx.LX_ERR_INVALID_ARG, lx.LX_ERR_ALIAS, lx.LX_ERR_WORKSPACE
NEED = lx.lx_ce_kd_workspace_bytes(4, 100000, 1)
NEED_STEP = lx.lx_ce_kd_forward_backward_workspace_bytes(4, 100000, 1)


def forward(z=A, ld=100000, t=A * 2, ids=A * 3, top=A * 4, rest=A * 5, BT=4, V=100000, K=8, T=1.0, ce=A * 6, kd=A * 7,
            lse=A * 8, state=A * 9, dt=1, ws=A * 10, wsb=NEED):
    return L.lx_ce_kd_forward(z, ld, t, ids, top, rest, BT, V, K, -100, T, ce, kd, lse, state, dt, ws, wsb, None)


def backward(grad=A * 12, ldg=100000, z=A, ld=100000, t=A * 2, ids=A * 3, top=A * 4, BT=4, V=100000, K=8, T=1.0, lse=A * 8,
             state=A * 9, cr=None, kr=None, gs=None, dt=1):
    return L.lx_ce_kd_backward(grad, ldg, z, ld, t, ids, top, BT, V, K, -100, T, lse, state, 1.0, 1.0, cr, kr, gs, dt, None)


def step(z=A, ld=100000, t=A * 2, ids=A * 3, top=A * 4, rest=A * 5, BT=4, V=100000, K=8, T=1.0, ce=A * 6, kd=A * 7, lse=A * 8,
         state=A * 9, grad=A * 12, ldg=100000, cr=None, kr=None, gs=None, dt=1, ws=A * 10, wsb=NEED_STEP):
    return L.lx_ce_kd_forward_backward(z, ld, t, ids, top, rest, BT, V, K, -100, T, ce, kd, lse, state, grad, ldg, 1.0, 1.0,
                                       cr, kr, gs, dt, ws, wsb, None)


@pytest.mark.parametrize("call", [forward, backward, step])
def test_sizes_and_types(call):
    assert call(BT=0) == lx.LX_OK
    assert call(dt=3) == lx.LX_ERR_UNSUPPORTED_DTYPE
    for kw in (dict(BT=-1), dict(V=0), dict(V=2 ** 31), dict(K=0), dict(K=257), dict(T=0.0), dict(T=-1.0), dict(T=2048.0),
               dict(T=float("nan")), dict(T=float("inf")), dict(ld=99999), dict(ld=2 ** 62), dict(z=None), dict(z=A + 1),
               dict(t=None), dict(t=A * 2 + 4), dict(ids=None), dict(ids=A * 3 + 2), dict(top=None), dict(top=A * 4 + 1),
               dict(lse=None), dict(lse=A * 8 + 2), dict(state=None), dict(state=A * 9 + 8),
               dict(BT=2 ** 40, V=1, ld=1)):
        assert call(**kw) == BAD, kw


@pytest.mark.parametrize("call", [forward, step])
def test_outputs(call):
    for kw in (dict(ce=None), dict(kd=None), dict(ce=A * 6 + 2), dict(kd=A * 7 + 1), dict(rest=A * 5 + 2)):
        assert call(**kw) == BAD, kw
    for kw in (dict(ce=A + 8), dict(kd=A * 2), dict(lse=A * 3), dict(state=A * 4), dict(ce=A * 5), dict(kd=A * 6),
               dict(ws=A * 9), dict(ws=A)):
        assert call(**kw) == ALIAS, kw


def test_workspaces():
    assert NEED > 0 and NEED_STEP > 0
    for call in (forward, step):
        assert call(ws=None) == WS
        assert call(ws=A * 10 + 128) == WS
    assert forward(wsb=NEED - 1) == WS
    assert step(wsb=NEED_STEP - 1) == WS
    for q in (lx.lx_ce_kd_workspace_bytes, lx.lx_ce_kd_forward_backward_workspace_bytes):
        assert q(0, 1000, 1) == 0
        assert q(4, 0, 1) == 0
        assert q(4, 1000, 3) == 0
        assert q(8192, 151936, 1) < 8192 * 1000  # partial sums only


@pytest.mark.parametrize("call", [backward, step])
def test_gradient(call):
    for kw in (dict(grad=None), dict(grad=A * 12 + 1), dict(ldg=99999), dict(cr=A * 13 + 2), dict(kr=A * 13 + 2),
               dict(gs=A * 13 + 1)):
        assert call(**kw) == BAD, kw
    for kw in (dict(grad=A + 2), dict(grad=A, ldg=100008), dict(grad=A * 3), dict(grad=A * 8), dict(grad=A * 9),
               dict(cr=A * 12), dict(kr=A * 12 + 4), dict(gs=A * 12)):
        assert call(**kw) == ALIAS, kw


def test_the_package_checks_what_it_passes():
    """Every refusal comes before the library is called (CPU tensors: none is a device tensor)."""
    f = lambda *s: torch.zeros(*s)  # noqa: E731

    def call(**kw):
        a = dict(student=f(3, 50), target=torch.zeros(3, dtype=torch.int64), ignore_index=-100,
                 ids=torch.zeros(3, 4, dtype=torch.int32), top=f(3, 4), lse_rest=f(3), temperature=1.0, ce=f(3), kd=f(3),
                 lse=f(3), state=f(3, 4))
        a.update(kw)
        lx.lx_ce_kd_forward(**a)

    with pytest.raises(ValueError, match="device tensor"):
        call()


NEED_TOP = lx.lx_top_logits_workspace_bytes(4, 100000, 8)


def top(z=A, ld=100000, BT=4, V=100000, K=8, T=1.0, out=A * 2, ids=A * 3, lse=A * 4, rest=A * 5, dt=1, ws=A * 6, wsb=NEED_TOP):
    return L.lx_top_logits(z, ld, BT, V, K, T, out, ids, lse, rest, dt, ws, wsb, None)


def test_top_logits():
    assert top(BT=0) == lx.LX_OK
    assert top(dt=-1) == lx.LX_ERR_UNSUPPORTED_DTYPE
    for kw in (dict(BT=-1), dict(V=0), dict(V=2 ** 31), dict(K=0), dict(K=257), dict(T=0.0), dict(T=float("nan")),
               dict(T=2.0 ** -11), dict(ld=99999), dict(z=None), dict(z=A + 1), dict(out=None), dict(ids=None),
               dict(out=A * 2 + 2), dict(ids=A * 3 + 1), dict(lse=A * 4 + 2), dict(rest=A * 5 + 1)):
        assert top(**kw) == BAD, kw
    for kw in (dict(out=A + 4), dict(ids=A * 2), dict(lse=A * 3), dict(rest=A * 4), dict(ws=A)):
        assert top(**kw) == ALIAS, kw
    assert NEED_TOP > 0
    assert top(ws=None) == top(wsb=NEED_TOP - 1) == top(ws=A * 6 + 16) == WS
    q = lx.lx_top_logits_workspace_bytes
    assert q(0, 100, 8) == q(4, 0, 8) == q(4, 100, 0) == q(4, 100, 257) == 0
    assert q(1, 2 ** 31 - 1, 256) < 1 << 20


NEED_LIN = lx.lx_ce_kd_linear_workspace_bytes(4, 1000, 64, 8, 512, True)


def linear(x=A, w=A * 2, H=64, t=A * 3, ids=A * 4, top=A * 5, rest=A * 6, BT=4, V=1000, K=8, T=1.0, ce=A * 7, kd=A * 8,
           lse=A * 9, state=A * 10, gx=A * 11, gw=A * 12, gdt=1, cr=None, kr=None, gs=None, piece=512, ws=A * 13, wsb=NEED_LIN):
    return L.lx_ce_kd_linear_forward_backward(x, w, H, t, ids, top, rest, BT, V, K, -100, T, ce, kd, lse, state, gx, gw, gdt,
                                              1.0, 1.0, cr, kr, gs, piece, ws, wsb, None)


def test_linear():
    assert linear(BT=0, gw=None) == lx.LX_OK
    assert linear(gdt=2) == lx.LX_ERR_UNSUPPORTED_DTYPE
    for kw in (dict(BT=-1), dict(BT=2 ** 31), dict(V=0), dict(V=2 ** 31), dict(H=0), dict(H=60), dict(H=2 ** 22 + 8), dict(K=-1),
               dict(K=257), dict(T=0.0), dict(piece=0), dict(piece=2 ** 22 + 1), dict(x=None), dict(w=None), dict(x=A + 8),
               dict(w=A * 2 + 2), dict(t=None), dict(ids=None), dict(top=None), dict(ce=None), dict(kd=None), dict(lse=None),
               dict(state=None), dict(state=A * 10 + 8), dict(gx=A * 11 + 8), dict(gw=A * 12 + 4), dict(cr=A * 14 + 2),
               dict(kr=A * 14 + 2), dict(gs=A * 14 + 2), dict(BT=2 ** 30, V=2 ** 30), dict(BT=0, gw=A * 12 + 4),
               dict(K=0, ce=None), dict(K=0, lse=None), dict(K=0, t=None)):
        assert linear(**kw) == BAD, kw
    for kw in (dict(ce=A), dict(kd=A * 2), dict(lse=A * 3), dict(state=A * 4), dict(gx=A * 5), dict(gw=A * 6), dict(ce=A * 8),
               dict(gx=A * 12), dict(ws=A * 2), dict(cr=A * 11), dict(kr=A * 12), dict(gs=A * 12)):
        assert linear(**kw) == ALIAS, kw
    assert linear(ws=None) == linear(wsb=NEED_LIN - 1) == linear(ws=A * 13 + 128) == WS
    q = lx.lx_ce_kd_linear_workspace_bytes
    assert q(0, 1000, 64, 8, 512, True) == q(4, 0, 64, 8, 512, True) == q(4, 1000, 60, 8, 512, True) == 0
    assert q(4, 1000, 64, 8, 512, False) < q(4, 1000, 64, 8, 512, True)
    # one piece of the gradient of the logits, sums and grad_x: far below the logits
    assert q(8192, 151936, 4096, 64, 8192, True) < 8192 * 151936 * 2 // 4
    assert lx.lx_ce_kd_linear_piece(8192, 151936) * 8192 <= 1 << 27
    assert lx.lx_ce_kd_linear_piece(1, 100) == 100
    assert lx.lx_ce_kd_linear_piece(0, 2 ** 31 - 1) <= 1 << 22
