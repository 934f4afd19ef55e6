"""The short convolution, its gradients and its step on the GPU against float64.

y: four products and a sum in fp32, then the fast exponential and division of the SiLU (about 2^-20 together, and up
to 2^-18 where the sum cancels).  dw and db sum the tokens' terms of random sign: 2^-18 sqrt(tokens)."""
import pytest
import torch

import mixer_reference as ref
from mixer_reference import assert_close

pytestmark = pytest.mark.gpu
TOL = 2.0 ** -18


def _case(B, T, C, W, cu, dtype, seed, state=True, bias=True):
    gen = torch.Generator().manual_seed(seed)
    n = B if cu is None else len(cu) - 1
    r = lambda *s, std=1.0: (std * torch.randn(s, generator=gen)).to(dtype)  # noqa: E731
    return dict(x=r(B, T, C), w=r(C, W, std=0.4), b=0.1 * torch.randn(C, generator=gen) if bias else None,
                st=r(n, W - 1, C) if state else None, dy=r(B, T, C), dst=r(n, W - 1, C) if state else None)


def _check(kda, c, cu, dtype, silu):
    d = {k: None if v is None else v.double() for k, v in c.items()}
    g = {k: None if v is None else v.cuda() for k, v in c.items()}
    cug = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    y, out = kda.short_conv_fwd(g["x"], g["w"], g["b"], cug, g["st"], silu, output_conv_state=True)
    yr, outr = ref.conv(d["x"], d["w"], d["b"], cu, d["st"], silu)
    assert_close(y, yr, dtype, TOL, "y")
    assert torch.equal(out.double().cpu(), outr)  # copies
    dx, dw, db, dst = kda.short_conv_bwd(g["dy"], g["x"], g["w"], g["b"], cug, g["st"], g["dst"], silu)
    dxr, dwr, dbr, dstr = ref.conv(d["x"], d["w"], d["b"], cu, d["st"], silu, d["dy"], d["dst"])
    M = c["x"].shape[0] * c["x"].shape[1]
    assert_close(dx, dxr, dtype, TOL, "dx")
    assert_close(dw, dwr, dtype, TOL * M ** 0.5, "dw")
    assert_close(db, dbr, torch.float32, TOL * M ** 0.5, "db")
    if c["st"] is None:
        assert dst is None
    else:
        assert_close(dst, dstr, dtype, TOL, "dstate")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("B,T,C", [(1, 1, 8), (2, 2, 33), (3, 3, 64), (1, 12, 1032), (2, 13, 40), (2, 300, 1), (3, 517, 136)])
def test_dense(kda, B, T, C, W, dtype):
    _check(kda, _case(B, T, C, W, None, dtype, 7 * T + C + W), None, dtype, True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("W", [2, 4])
@pytest.mark.parametrize("cu", [[0, 5], [0, 0, 1, 2, 2, 4, 7, 40, 40], [0, 1, 2, 3, 4, 5, 6, 7, 8], [0, 12, 24, 36, 37],
                                [0, 130, 131, 260, 300]])
def test_packed(kda, cu, W, dtype):
    T = cu[-1]
    _check(kda, _case(1, T, 72, W, cu, dtype, T + W), cu, dtype, True)
    _check(kda, _case(1, T, 20, W, cu, dtype, T + W + 1, state=False, bias=False), cu, dtype, False)


def test_long_runs(kda):
    """Many runs of the backward pass, each of 128 tokens."""
    cu = [0, 1000, 1001, 40000, 70000]
    _check(kda, _case(1, 70000, 32, 4, cu, torch.float32, 9), cu, torch.float32, True)


def test_slice_of_a_projection(kda):
    gen = torch.Generator().manual_seed(2)
    z = torch.randn((2, 50, 200), generator=gen).to(torch.bfloat16).cuda()
    w = torch.randn((64, 4), generator=gen).to(torch.bfloat16)
    for off in (64, 67):  # on a 16-byte boundary and off it
        x = z[:, :, off:off + 64]
        y, _ = kda.short_conv_fwd(x, w.cuda())
        assert_close(y, ref.conv(x.double().cpu(), w.double(), None, None, None, True)[0], torch.bfloat16, TOL)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("B,C", [(1, 8), (5, 33), (256, 512)])
def test_step_continues_the_sequence(kda, B, C, W, dtype):
    """Three steps from the cache of a prefill are the three next tokens of the whole sequence."""
    c = _case(B, 10, C, W, None, dtype, B + C)
    x, w, b = c["x"].cuda(), c["w"].cuda(), c["b"].cuda()
    _, cache = kda.short_conv_fwd(x[:, :7], w, b, output_conv_state=True) if B == 1 else \
        kda.short_conv_fwd(x[:, :7].contiguous(), w, b, output_conv_state=True)
    want = ref.conv(c["x"].double(), c["w"].double(), c["b"].double(), None, None, True)[0]
    for t in range(7, 10):
        y = kda.short_conv_step(x[:, t].contiguous(), w, cache, b)
        assert_close(y, want[:, t], dtype, TOL)
    assert torch.equal(cache, x[:, 10 - (W - 1):])


def test_in_place_cache_and_no_tokens(kda):
    c = _case(1, 9, 40, 4, [0, 2, 9], torch.bfloat16, 4)
    cu = torch.tensor([0, 2, 9], dtype=torch.int32, device="cuda")
    st = c["st"].cuda()
    y0, out = kda.short_conv_fwd(c["x"].cuda(), c["w"].cuda(), None, cu, st, output_conv_state=True)
    y1, same = kda.short_conv_fwd(c["x"].cuda(), c["w"].cuda(), None, cu, st, conv_state_out=st)
    assert same.data_ptr() == st.data_ptr() and torch.equal(y0, y1) and torch.equal(out, st)
    e = torch.empty((3, 0, 40), device="cuda", dtype=torch.bfloat16)
    st3 = torch.randn(3, 3, 40, device="cuda").to(torch.bfloat16)
    y, out = kda.short_conv_fwd(e, c["w"].cuda(), conv_state=st3, output_conv_state=True)
    assert torch.equal(out, st3)
    dx, dw, db, dst = kda.short_conv_bwd(e, e.clone(), c["w"].cuda(), conv_state=st3, d_conv_state_out=st3)
    assert torch.equal(dst, st3) and not dw.any() and not db.any()


def test_one_bad_sequence_leaves_the_others_alone(kda):
    c = _case(1, 30, 64, 4, [0, 10, 20, 30], torch.float32, 6, bias=False)
    cu = torch.tensor([0, 10, 20, 30], dtype=torch.int32, device="cuda")
    x, dy = c["x"].clone(), c["dy"].clone()
    x[0, 10:20], dy[0, 10:20] = float("nan"), float("inf")
    args = (c["w"].cuda(), None, cu, c["st"].cuda())
    good, bad = (kda.short_conv_fwd(t.cuda(), *args)[0] for t in (c["x"], x))
    dgood = kda.short_conv_bwd(c["dy"].cuda(), c["x"].cuda(), *args)[0]
    dbad = kda.short_conv_bwd(dy.cuda(), x.cuda(), *args)[0]
    for p, q in ((good, bad), (dgood, dbad)):
        assert torch.equal(p[:, :10], q[:, :10]) and torch.equal(p[:, 20:], q[:, 20:])
