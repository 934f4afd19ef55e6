"""Refusals of the selective mixer's entry points, before any launch (no GPU needed): pointers here are numbers."""
import ctypes

import pytest
import torch

P = 1 << 20  # 16-byte aligned; never dereferenced
Q, R, S = P + 4096, P + 8192, P + 12288


@pytest.fixture(scope="module")
def lib(kda):
    return kda.lib()


def test_layer_norm(kda, lib):
    def fwd(x=P, ldx=64, w=None, b=None, y=Q, ldy=64, mean=None, rstd=None, M=4, N=64, dtype=0):
        return lib.kda_layer_norm_fwd(x, ldx, w, b, y, ldy, mean, rstd, M, N, dtype, 1e-5, None)
    bad = kda.KDA_ERR_INVALID_ARG
    assert fwd(dtype=2) == bad and fwd(M=-1) == bad and fwd(N=0) == bad and fwd(x=None) == bad and fwd(y=None) == bad
    assert fwd(ldx=63) == bad and fwd(ldy=63) == bad and fwd(y=P) == bad and fwd(x=P + 1) == bad and fwd(w=P + 2) == bad
    assert fwd(x=P + 2, dtype=1) == bad and fwd(M=0) == kda.KDA_OK
    assert fwd(M=0x7fffff01) == fwd(N=0x7fffff01, ldx=1 << 31, ldy=1 << 31) == kda.KDA_ERR_UNSUPPORTED

    def bwd(dy=P, x=Q, mean=S, rstd=S, dx=R, dw=S, ws=None, size=0, ld=64, M=4):
        return lib.kda_layer_norm_bwd(dy, ld, x, ld, None, mean, rstd, dx, ld, dw, None, M, 64, 0, ws, size, None)
    need = lib.kda_layer_norm_bwd_workspace(4, 64)
    assert need > 0 and lib.kda_layer_norm_bwd_workspace(-1, 64) == 0
    assert bwd() == kda.KDA_ERR_WORKSPACE and bwd(ws=P, size=need - 1) == kda.KDA_ERR_WORKSPACE
    assert bwd(ws=P + 16, size=need) == bad and bwd(mean=None) == bad and bwd(dx=P) == bad and bwd(dx=Q) == bad
    assert bwd(ld=60) == bad and bwd(dy=None) == bad


def test_linear(kda, lib):
    def fwd(x=P, ldx=64, W=Q, ldw=64, b=None, r=None, ldr=0, y=R, ldy=32, pre=None, ldp=0, M=8, N=32, K=64, act=0):
        return lib.kda_linear_act_bf16(x, ldx, W, ldw, b, r, ldr, y, ldy, pre, ldp, M, N, K, act, None)
    bad = kda.KDA_ERR_INVALID_ARG
    assert fwd(act=5) == bad and fwd(act=-1) == bad and fwd(M=-1) == bad and fwd(x=None) == bad and fwd(ldx=56) == bad
    assert fwd(ldx=68) == bad and fwd(y=R + 8) == bad and fwd(ldy=36) == bad and fwd(r=S, ldr=31) == bad
    assert fwd(pre=S, ldp=36) == bad and fwd(pre=S + 2, ldp=40) == bad and fwd(y=P) == bad and fwd(r=R, ldr=32) == bad
    assert fwd(pre=R, ldp=32) == bad and fwd(b=S + 2) == bad and fwd(r=S + 1, ldr=32) == bad
    assert fwd(M=0x7fffff01) == fwd(N=0x7fffff01) == fwd(K=0x7fffff01) == kda.KDA_ERR_UNSUPPORTED
    assert fwd(K=0, ldx=64) == kda.KDA_ERR_UNSUPPORTED and fwd(M=0) == kda.KDA_OK and fwd(N=0, K=0) == kda.KDA_OK

    def bwd(dy=P, lddy=32, x=Q, W=R, pre=S, dx=S + 4096, dW=S + 8192, act=3, ws=None, size=0, K=64, lddx=64):
        return lib.kda_linear_act_bwd_bf16(dy, lddy, x, 64, W, 64, pre, 32, dx, lddx, dW, 64, None, 8, 32, K, act, ws,
                                           size, None)
    need = lib.kda_linear_act_bwd_workspace(8, 32)
    assert bwd() == kda.KDA_ERR_WORKSPACE and bwd(ws=P, size=need - 1) == kda.KDA_ERR_WORKSPACE
    assert bwd(ws=P + 128, size=need) == bad and bwd(pre=None) == bad and bwd(x=None) == bad and bwd(W=None) == bad
    assert bwd(lddy=30) == bad and bwd(dx=P) == bad and bwd(dW=S + 4096) == bad and bwd(lddx=60) == bad
    assert bwd(lddx=68) == bad and bwd(act=9) == bad and bwd(x=Q + 8) == bad


def test_short_conv(kda, lib):
    def fwd(x=P, ldx=16, w=Q, y=R, ldy=16, cu=None, nseq=0, B=2, T=3, C=16, W=4, dtype=0, cin=None, cout=None):
        return lib.kda_short_conv_fwd(x, ldx, w, None, y, ldy, cin, cout, cu, nseq, B, T, C, W, dtype, 1, None)
    bad = kda.KDA_ERR_INVALID_ARG
    assert fwd(W=1) == fwd(W=5) == kda.KDA_ERR_UNSUPPORTED
    assert fwd(dtype=9) == bad and fwd(B=-1) == bad and fwd(C=-1) == bad and fwd(nseq=2) == bad and fwd(cu=S) == bad
    assert fwd(cu=S, nseq=2) == bad and fwd(cu=S + 2, nseq=2, B=1) == bad and fwd(cu=S, nseq=0, B=1) == bad
    assert fwd(x=None) == bad and fwd(ldx=15) == bad and fwd(ldy=15) == bad and fwd(y=P) == bad and fwd(w=Q + 1) == bad
    assert fwd(B=70000, T=70000) == kda.KDA_ERR_UNSUPPORTED
    assert fwd(C=0) == kda.KDA_OK and fwd(B=0) == kda.KDA_OK and fwd(T=0) == kda.KDA_OK

    def bwd(dx=S, ws=None, size=0, dci=None, dco=None, dy=P):
        return lib.kda_short_conv_bwd(dy, 16, Q, 16, R, None, None, dco, dx, 16, None, None, dci, None, 0, 2, 3, 16, 4,
                                      0, 1, ws, size, None)
    need = lib.kda_short_conv_bwd_workspace(6, 16, 4)
    assert bwd() == kda.KDA_ERR_WORKSPACE and bwd(ws=P + 8, size=need) == bad and bwd(dx=P) == bad and bwd(dx=Q) == bad
    assert bwd(dci=S + 64, dco=S + 64) == bad and bwd(dy=None) == bad
    assert lib.kda_short_conv_bwd_workspace(6, 16, 5) == 0

    def step(x=P, w=Q, st=R, y=S, B=2, C=16, W=4, ld=16):
        return lib.kda_short_conv_step(x, ld, w, None, st, y, ld, B, C, W, 0, 1, None)
    assert step(W=0) == kda.KDA_ERR_UNSUPPORTED and step(x=None) == bad and step(st=None) == bad and step(y=P) == bad
    assert step(st=P) == bad and step(ld=8) == bad and step(B=-1) == bad and step(B=0) == kda.KDA_OK


def _params(kda, A=P, D=None, bias=None, ch=32, G=1, N=16, sp=1):
    from gated_delta_rule_123_b200.mixer import ScanParams
    return ctypes.byref(ScanParams(A, D, bias, ch, G, N, sp))


def test_selective_scan(kda, lib):
    bad, uns = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED

    def fwd(u=P, dt=Q, Bm=R, C=R, z=None, y=S, ld=32, ldb=16, p=None, cu=None, nseq=0, B=2, T=40, dtype=0, h0=None, ws=None):
        return lib.kda_selective_scan_fwd(u, ld, dt, ld, Bm, ldb, C, ldb, z, ld, p or _params(kda), h0, None, y, ld, cu, nseq,
                                          B, T, dtype, ws, 0, None)
    assert fwd(p=ctypes.byref(__import__("gated_delta_rule_123_b200.mixer", fromlist=["x"]).ScanParams())) == bad  # no groups
    assert fwd(p=_params(kda, G=3)) == bad and fwd(p=_params(kda, N=0)) == bad and fwd(p=_params(kda, A=None)) == bad
    assert fwd(p=_params(kda, N=33), ldb=33) == uns and fwd(p=_params(kda, D=P + 2)) == bad
    assert fwd(dtype=3) == bad and fwd(u=None) == bad and fwd(Bm=None) == bad and fwd(ld=31) == bad and fwd(ldb=15) == bad
    assert fwd(y=P) == bad and fwd(z=S) == bad and fwd(u=P + 1) == bad and fwd(h0=P + 2) == bad
    assert fwd(nseq=1) == bad and fwd(cu=S, nseq=1) == bad and fwd(B=-1) == bad and fwd(B=1 << 16, T=1 << 16) == uns
    assert fwd(B=70000, T=1) == uns
    # long and narrow: segments need their workspace
    assert lib.kda_selective_scan_fwd_workspace(1, 8192, 32, 1, 16, 0) > 0
    assert fwd(B=1, T=8192) == kda.KDA_ERR_WORKSPACE
    assert fwd(B=0) == kda.KDA_OK and fwd(p=_params(kda, ch=0)) == kda.KDA_OK

    def bwd(dy=P, u=P + 64, dt=Q, du=S, ddt=S + 64, dA=S + 128, dB=S + 192, dC=S + 256, z=None, dz=None, ws=None, size=0,
            h0=None, dh=None, dh0=None):
        return lib.kda_selective_scan_bwd(dy, 32, u, 32, dt, 32, R, 16, R, 16, z, 32, _params(kda), h0, dh, du, 32, ddt, 32,
                                          dB, 16, dC, 16, dz, 32, dA, None, None, dh0, None, 0, 2, 40, 0, ws, size, None)
    need = lib.kda_selective_scan_bwd_workspace(2, 40, 32, 1, 16, 0)
    assert bwd() == kda.KDA_ERR_WORKSPACE and bwd(ws=P, size=need - 1) == kda.KDA_ERR_WORKSPACE
    assert bwd(ws=P + 4, size=need) == bad and bwd(dA=None) == bad and bwd(du=P) == bad and bwd(du=S + 64) == bad
    assert bwd(z=Q + 64) == bad and bwd(dh=P, dh0=P) == bad and bwd(h0=P, dh0=P) == bad and bwd(dC=R) == bad

    def step(u=P, dt=Q, st=S, y=S + 4096, ld=32, B=2, p=None):
        return lib.kda_selective_scan_step(u, ld, dt, ld, R, 16, R, 16, None, 0, p or _params(kda), st, y, ld, B, 0, None)
    assert step(st=None) == bad and step(y=P) == bad and step(y=S) == bad and step(ld=30) == bad and step(B=-1) == bad
    assert step(p=_params(kda, N=64)) == uns and step(st=S + 2) == bad and step(B=0) == kda.KDA_OK


def test_bindings_check_their_tensors(kda):
    """The bindings refuse CPU tensors and wrong types before the library sees a pointer."""
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        kda.layer_norm_fwd(x)
    with pytest.raises(ValueError):
        kda.linear_act(x.bfloat16(), x.bfloat16())
    with pytest.raises(ValueError):
        kda.short_conv_step(x, x, x)
    with pytest.raises(ValueError):
        kda.selective_scan_step(x, x, x, x[:, None], x[:, None], x)


def test_row_strides():
    from gated_delta_rule_123_b200.mixer import _ld
    t = torch.zeros(3, 5, 24)
    assert _ld(t, "t") == 24 and _ld(t[:, :, 8:16], "t") == 24 and _ld(t[:1], "t") == 24 and _ld(t.new_zeros(3, 0, 24), "t") == 24
    assert _ld(t.view(3, 5, 2, 12), "t", 2) == 24 and _ld(t[:, :, None, 3:7], "t", 2) == 24
    assert _ld(t[:1, :1, :17], "t") == 24  # one row: rounded up, never stepped over
    for bad in (t[:, :3], t.transpose(0, 1), t[:, :, ::2], t[:, :1].expand(3, 5, 24)):
        with pytest.raises(ValueError):
            _ld(bad, "t")
    with pytest.raises(ValueError):
        _ld(t.view(3, 5, 2, 12)[:, :, :, :6], "t", 2)


def test_sizes_and_strides_past_32_bits_are_refused(kda, monkeypatch):
    """The C entry points take int sizes (and the projection int row strides): what does not fit never reaches them."""
    from gated_delta_rule_123_b200 import mixer

    def reached(*args):
        raise AssertionError("reached the library")
    monkeypatch.setattr(mixer, "_first", lambda t, what, dtypes=(): t.device)  # tensors without storage stand in
    monkeypatch.setattr(mixer, "_run", reached)
    monkeypatch.setattr(mixer, "_query", reached)
    big, b16, f32 = (1 << 32) + 5, torch.bfloat16, torch.float32
    m = lambda *s, t=b16: torch.empty(s, device="meta", dtype=t)  # noqa: E731
    far = torch.empty_strided((2, 8), ((1 << 32) + 8, 1), device="meta", dtype=b16)
    w, x = m(8, 8), m(2, 8)
    A = m(1, 1, t=f32)
    calls = [
        lambda: mixer.layer_norm_fwd(m(big, 1)),
        lambda: mixer.layer_norm_bwd(m(big, 1), m(big, 1), None, m(big, t=f32), m(big, t=f32)),
        lambda: mixer.linear_act(m(big, 8), w), lambda: mixer.linear_act(far, w), lambda: mixer.linear_act(x, far),
        lambda: mixer.linear_act(x, w, residual=far), lambda: mixer.linear_act(x, w, out=far),
        lambda: mixer.linear_act_bwd(m(big, 8), m(big, 8), w), lambda: mixer.linear_act_bwd(far, x, w),
        lambda: mixer.linear_act_bwd(x, far, w), lambda: mixer.linear_act_bwd(x, x, w, far, "silu"),
        lambda: mixer.short_conv_fwd(m(1, big, 1), m(1, 4)), lambda: mixer.short_conv_fwd(m(big, 1, 1), m(1, 4)),
        lambda: mixer.short_conv_fwd(m(1 << 16, 1 << 16, 1), m(1, 4)),
        lambda: mixer.short_conv_bwd(m(1, big, 1), m(1, big, 1), m(1, 4)),
        lambda: mixer.short_conv_fwd(m(big, 0, 1), m(1, 4)),
        lambda: mixer.short_conv_fwd(m(1, 4, 1), m(1, 4), cu_seqlens=m(big, t=torch.int32)),
        lambda: mixer.short_conv_step(m(big, 1), m(1, 4), m(big, 3, 1)),
        lambda: mixer.selective_scan_fwd(m(1, big, 1), m(1, big, 1), A, m(1, big, 1, 1), m(1, big, 1, 1)),
        lambda: mixer.selective_scan_bwd(m(1, big, 1), m(1, big, 1), m(1, big, 1), A, m(1, big, 1, 1), m(1, big, 1, 1)),
        lambda: mixer.selective_scan_step(m(big, 1), m(big, 1), A, m(big, 1, 1), m(big, 1, 1), m(big, 1, 1, t=f32)),
    ]
    for i, f in enumerate(calls):
        with pytest.raises(ValueError, match="2\\^31"):
            f()
            raise AssertionError(i)
