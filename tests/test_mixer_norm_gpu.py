"""Layer norm on the GPU against float64, every register shape and the any-width kernel.

fp32 arithmetic: a sum over N terms by a tree of threads is off by at most (N / 256 + 16) half steps of its terms'
absolute sum (a thread adds at most N / 256 terms in a row in the widest loop, then 16 levels), and the mean, the
variance and the normalised value each carry a few more; 64 half steps, 2^-18, cover every width here.  Column sums
add up to M terms of random sign, whose absolute sum is about sqrt(M) times their sum: 2^-18 sqrt(M)."""
import pytest
import torch

import mixer_reference as ref
from mixer_reference import assert_close

pytestmark = pytest.mark.gpu
TOL = 2.0 ** -18


def _inputs(M, N, dtype, seed, ld=None, off=0):
    gen = torch.Generator().manual_seed(seed)

    def rows(std=1.0, mean=0.0):
        t = (mean + std * torch.randn((M, ld or N), generator=gen)).to(dtype)
        return t[:, off:off + N]
    return rows(1.5, 0.3), rows(), 1 + 0.2 * torch.randn(N, generator=gen), 0.1 * torch.randn(N, generator=gen)


def _check(kda, x, dy, w, b, dtype):
    d = lambda t: None if t is None else t.double()  # noqa: E731
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    xg, dyg = (torch.empty_strided(t.shape, t.stride(), dtype=dtype, device="cuda").copy_(t) for t in (x, dy))
    y, mean, rstd = kda.layer_norm_fwd(xg, cu(w), cu(b))
    yr, mr, rr = ref.norm_fwd(d(x), d(w), d(b), 1e-5)
    assert_close(y, yr, dtype, TOL, "y")
    assert_close(mean, mr, torch.float32, TOL * 8, "mean")  # the mean is small against the terms of its sum
    assert_close(rstd, rr, torch.float32, TOL, "rstd")
    dx, dw, db = kda.layer_norm_bwd(dyg, xg, cu(w), mean, rstd)
    dxr, dwr, dbr = ref.norm_bwd(d(dy), d(x), d(w), mean.double().cpu(), rstd.double().cpu())
    M = x.reshape(-1, x.shape[-1]).shape[0]
    assert_close(dx, dxr, dtype, TOL, "dx")
    assert_close(dw, dwr, torch.float32, TOL * M ** 0.5, "dw")
    assert_close(db, dbr, torch.float32, TOL * M ** 0.5, "db")
    again = kda.layer_norm_bwd(dyg, xg, cu(w), mean, rstd)
    for p, q in zip((dx, dw, db), again):
        assert torch.equal(p, q)  # the sums' order is fixed


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N", [(1, 8), (3, 64), (37, 256), (5, 384), (700, 520), (9, 1024), (4, 2048), (2000, 2048),
                                 (6, 4096), (3, 8192), (2, 16384), (5, 1), (9, 7), (33, 1603), (2, 20000)])
def test_norm(kda, M, N, dtype):
    if N == 1:  # x - mean is 0: y is the bias, every gradient but db is 0
        x, dy, w, b = _inputs(M, N, dtype, 1)
        y, mean, rstd = kda.layer_norm_fwd(x.cuda(), w.cuda(), b.cuda())
        assert torch.equal(y.cpu(), b.to(dtype).expand(M, 1))
        dx, dw, db = kda.layer_norm_bwd(dy.cuda(), x.cuda(), w.cuda(), mean, rstd)
        assert not dx.any() and not dw.any()
        assert_close(db, dy.double().sum(0), torch.float32, TOL)
        return
    x, dy, w, b = _inputs(M, N, dtype, M * 31 + N)
    _check(kda, x, dy, w, b, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N", [(4737, 536), (5001, 1024), (4800, 2048), (4741, 1800), (4739, 4096), (9001, 600)])
def test_norm_of_many_rows(kda, M, N, dtype):
    """Enough rows for the kernel whose blocks walk over them."""
    x, dy, w, b = _inputs(M, N, dtype, M + N)
    _check(kda, x, dy, w, b, dtype)


@pytest.mark.parametrize("N,ld,off", [(256, 264, 8), (256, 300, 0), (250, 257, 3)])
def test_norm_of_slices(kda, N, ld, off):
    x, dy, w, b = _inputs(19, N, torch.bfloat16, 5, ld, off)
    _check(kda, x, dy, w, b, torch.bfloat16)


def test_norm_without_weights_and_of_three_axes(kda):
    x, dy, w, b = _inputs(12, 128, torch.float32, 6)
    _check(kda, x, dy, None, None, torch.float32)
    y, mean, rstd = kda.layer_norm_fwd(x.cuda().reshape(3, 4, 128), w.cuda(), None, eps=0.1)
    yr, _, rr = ref.norm_fwd(x.double(), w.double(), None, 0.1)
    assert mean.shape == (3, 4)
    assert_close(y.reshape(12, 128), yr, torch.float32, TOL)
    assert_close(rstd.reshape(-1), rr, torch.float32, TOL)
    dx, dw, db = kda.layer_norm_bwd(dy.cuda().reshape(3, 4, 128), x.cuda().reshape(3, 4, 128), w.cuda(), mean, rstd,
                                    weight_grad=False, bias_grad=False)
    assert dw is None and db is None and dx.shape == (3, 4, 128)


def test_norm_rows_are_independent_and_constant_rows_are_fine(kda):
    x = torch.full((3, 512), 1000.0, device="cuda")
    x[1] = float("nan")
    y, mean, rstd = kda.layer_norm_fwd(x)
    assert not y[0].any() and not y[2].any() and y[1].isnan().all()  # no cancellation: 1000 - mean is exactly 0
    assert abs(float(rstd[0]) - 1e-5 ** -0.5) < 1e-4 * 1e-5 ** -0.5


def test_norm_of_no_rows(kda):
    x = torch.empty((0, 64), device="cuda")
    y, mean, rstd = kda.layer_norm_fwd(x)
    assert y.shape == (0, 64) and mean.shape == (0,)
    dx, dw, db = kda.layer_norm_bwd(x, x.clone(), None, mean, rstd)
    assert not dw.any() and not db.any()
