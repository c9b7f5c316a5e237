"""Host checks of the draft verification (CPU only: no kernel is ever launched here)."""
import pytest
import torch

lx = pytest.importorskip("cross_entropy_tv_amd", reason="HIP library not built")
L = lx.lib

A = 1 << 32  # fake, never dereferenced device addresses
NEED = lx.lx_draft_verify_workspace_bytes(4, 3, 1000)


def verify(target=A, ldt=1000, draft=A * 2, ldd=1000, tok=A * 3, start=A * 4, S=4, N=9, L_=3, V=1000, temp=A * 5,
           ua=A * 6, us=A * 7, n=A * 8, out=A * 9, lp=A * 10, dt=1, ws=A * 11, wsb=NEED):
    return L.lx_draft_verify(target, ldt, draft, ldd, tok, start, S, N, L_, V, temp, ua, us, n, out, lp, dt, ws, wsb,
                             None)


def test_validation():
    bad, alias = lx.LX_ERR_INVALID_ARG, lx.LX_ERR_ALIAS
    assert verify(S=0) == lx.LX_OK
    assert verify(dt=3) == lx.LX_ERR_UNSUPPORTED_DTYPE
    assert verify(S=-1) == bad
    assert verify(N=-1) == bad
    assert verify(N=13) == bad                     # more than S * max_draft
    assert verify(V=0) == bad
    assert verify(V=2 ** 31) == bad
    assert verify(L_=-1) == bad
    assert verify(S=2 ** 24, L_=3) == bad           # S * (max_draft + 1)
    assert verify(S=2 ** 20, L_=3, V=2 ** 24) == bad   # workgroups
    assert verify(ldt=999) == bad
    assert verify(ldd=999) == bad
    assert verify(ldt=2 ** 62) == bad
    for name in ("target", "tok", "start", "ua", "us", "n", "out"):
        assert verify(**{name: None}) == bad, name
    assert verify(target=A + 1) == bad
    assert verify(draft=A * 2 + 1) == bad
    assert verify(tok=A * 3 + 4) == bad
    assert verify(start=A * 4 + 4) == bad
    assert verify(temp=A * 5 + 2) == bad
    assert verify(out=A * 9 + 4) == bad
    assert verify(lp=A * 10 + 2) == bad
    assert verify(out=A + 8) == alias               # inside the target logits
    assert verify(lp=A * 9) == alias                # inside the tokens
    assert verify(n=A * 4) == alias                 # the starts
    assert verify(ws=A * 2) == alias                # the draft logits
    assert verify(ws=None) == lx.LX_ERR_WORKSPACE
    assert verify(wsb=NEED - 1) == lx.LX_ERR_WORKSPACE
    assert verify(ws=A * 11 + 128) == lx.LX_ERR_WORKSPACE


def test_workspace_sizes():
    assert lx.lx_draft_verify_workspace_bytes(0, 3, 1000) == 0
    assert lx.lx_draft_verify_workspace_bytes(4, 3, 0) == 0
    assert lx.lx_draft_verify_workspace_bytes(4, -1, 1000) == 0
    assert lx.lx_draft_verify_workspace_bytes(4, 0, 1000) > 0
    # partial sums only: far below the logits
    assert lx.lx_draft_verify_workspace_bytes(256, 8, 151936) < 256 * 8 * 151936 // 100


def test_the_package_checks_what_it_passes():
    """The binding refuses tensors that the C entry point could not tell from right ones (CPU tensors here: none is
    a device tensor, and every refusal comes before the library is called)."""
    f = lambda *s: torch.zeros(*s)  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int64)  # noqa: E731

    def call(**kw):
        a = dict(target=f(7, 50), draft=f(5, 50), draft_tokens=i(5), draft_start=i(3), max_draft=3, temperature=f(2),
                 u_accept=f(5), u_sample=f(2), n_accepted=i(2), tokens=i(2, 4), logprobs=f(2, 4))
        a.update(kw)
        lx.lx_draft_verify(**a)

    with pytest.raises(ValueError, match="device tensor"):
        call()
    with pytest.raises(ValueError, match="device tensor"):
        call(target=f(7, 50, 1))
