"""Host checks of the low-rank adapters (CPU only: no kernel is ever launched here)."""
import pytest
import torch

lx = pytest.importorskip("cross_entropy_tv_amd", reason="HIP library not built")
L = lx.lib

A = 1 << 40  # fake, never dereferenced device addresses
FW = lx.lx_lora_forward_workspace_bytes(100, 4, 256, 512, 16)
BW = lx.lx_lora_backward_workspace_bytes(100, 4, 3, 256, 512, 16)


def fwd(x=A, ldx=256, a=A * 2, b=A * 3, ad=A * 4, st=A * 5, sc=A * 6, rk=A * 7, T=100, R=4, n=3, H=256, N=512, r=16,
        base=A * 8, ldb=512, bdt=0, y=A * 9, ldy=512, ydt=1, ws=A * 10, wsb=FW):
    return L.lx_lora_forward(x, ldx, a, b, ad, st, sc, rk, T, R, n, H, N, r, base, ldb, bdt, y, ldy, ydt, ws, wsb, None)


def bwd(gy=A * 11, ldgy=512, x=A, ldx=256, a=A * 2, b=A * 3, ad=A * 4, st=A * 5, sc=A * 6, rk=A * 7, T=100, R=4, n=3,
        H=256, N=512, r=16, base=A * 8, ldb=256, gx=A * 9, ldgx=256, ga=A * 12, gb=A * 13, ws=A * 10, wsb=BW):
    return L.lx_lora_backward(gy, ldgy, x, ldx, a, b, ad, st, sc, rk, T, R, n, H, N, r, base, ldb, gx, ldgx, ga, gb, ws,
                              wsb, None)


@pytest.mark.parametrize("call", [fwd, bwd], ids=["forward", "backward"])
def test_shapes_and_pointers(call):
    bad = lx.LX_ERR_INVALID_ARG
    for kw in (dict(T=-1), dict(T=2 ** 22 + 1), dict(R=-1), dict(R=2 ** 24 + 1), dict(n=0), dict(n=2 ** 20 + 1),
               dict(H=252), dict(H=0), dict(N=516), dict(N=2 ** 22 + 8), dict(r=12), dict(r=0), dict(r=136),
               dict(n=2 ** 20, r=128, H=2 ** 20), dict(ldx=248), dict(ldx=260), dict(x=None), dict(a=None),
               dict(b=None), dict(ad=None), dict(st=None), dict(sc=None), dict(x=A + 8), dict(a=A * 2 + 8),
               dict(b=A * 3 + 2), dict(ad=A * 4 + 4), dict(st=A * 5 + 4), dict(sc=A * 6 + 2), dict(rk=A * 7 + 4),
               dict(base=A * 8 + 8), dict(ldb=100)):
        assert call(**kw) == bad, kw
    assert call(ws=None) == lx.LX_ERR_WORKSPACE
    assert call(wsb=63) == lx.LX_ERR_WORKSPACE
    assert call(ws=A * 10 + 128) == lx.LX_ERR_WORKSPACE
    assert call(ws=A + 512) == lx.LX_ERR_ALIAS         # workspace over x
    assert call(ws=A * 8) == lx.LX_ERR_ALIAS           # ... over base


def test_forward_only():
    assert fwd(T=0) == lx.LX_OK
    assert fwd(R=0) == lx.LX_OK
    assert fwd(ydt=2) == lx.LX_ERR_UNSUPPORTED_DTYPE
    assert fwd(bdt=2) == lx.LX_ERR_UNSUPPORTED_DTYPE
    assert fwd(y=None) == lx.LX_ERR_INVALID_ARG
    assert fwd(ldy=500) == lx.LX_ERR_INVALID_ARG
    assert fwd(y=A * 9 + 8) == lx.LX_ERR_INVALID_ARG
    assert fwd(y=A + 1024) == lx.LX_ERR_ALIAS           # inside x
    assert fwd(y=A * 3) == lx.LX_ERR_ALIAS              # over B
    assert fwd(y=A * 8) == lx.LX_ERR_ALIAS              # over base, of another type
    assert fwd(y=A * 8 + 16, ydt=0) == lx.LX_ERR_ALIAS
    assert fwd(y=A * 8, ydt=0, ldy=520) == lx.LX_ERR_ALIAS  # another row stride


def test_backward_only():
    assert bwd(gx=None, ga=None, gb=None) == lx.LX_ERR_INVALID_ARG
    assert bwd(gy=None) == lx.LX_ERR_INVALID_ARG
    assert bwd(ldgy=504) == lx.LX_ERR_INVALID_ARG
    assert bwd(ldgx=200) == lx.LX_ERR_INVALID_ARG
    assert bwd(ga=A * 12 + 4) == lx.LX_ERR_INVALID_ARG
    assert bwd(ga=A * 13) == lx.LX_ERR_ALIAS             # the two gradients
    assert bwd(T=0, ga=A * 13) == lx.LX_ERR_ALIAS
    assert bwd(gb=A * 11 + 4096) == lx.LX_ERR_ALIAS      # inside grad_y
    assert bwd(gx=A * 8, ldgx=264) == lx.LX_ERR_ALIAS     # over base with another row stride
    assert bwd(ga=A * 8) == lx.LX_ERR_ALIAS              # over base


def test_the_package_checks_what_it_passes():
    """CPU tensors: every refusal comes before the library is called."""
    z = torch.zeros
    bf, i64 = torch.bfloat16, torch.int64

    def call(**kw):
        a = dict(x=z(4, 16, dtype=bf), A=z(2, 8, 16, dtype=bf), B=z(2, 24, 8, dtype=bf), adapter=z(1, dtype=i64),
                 req_start=z(2, dtype=i64), scale=z(2), rank=None, base=None, y=z(4, 24))
        a.update(kw)
        lx.lx_lora_forward(**a)

    with pytest.raises(ValueError, match="device tensor"):
        call()
    with pytest.raises(ValueError, match="bfloat16"):
        call(x=z(4, 16))
    with pytest.raises(ValueError, match="n_adapters"):
        call(B=z(2, 24, 16, dtype=bf))


def test_workspace_sizes():
    assert lx.lx_lora_forward_workspace_bytes(0, 4, 256, 512, 16) == 0
    assert lx.lx_lora_forward_workspace_bytes(100, 4, 250, 512, 16) == 0
    assert lx.lx_lora_forward_workspace_bytes(64, 64, 4096, 4096, 16) < 1 << 20
    assert lx.lx_lora_backward_workspace_bytes(100, 0, 3, 256, 512, 16) == 0
