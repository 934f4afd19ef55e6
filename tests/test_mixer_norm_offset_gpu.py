"""Layer norm's gradients of rows whose mean is far above their spread, and of constant rows: xh = (x - mean) rstd must
come from the difference, not from x rstd and mean rstd, which cancel.

The difference is exact to half a step, so the tolerances of test_mixer_norm_gpu.py hold: 2^-18, and sqrt(rows) of it
for the column sums.  mean and rstd are inputs of the gradient: the float64 statement gets the same ones."""
import pytest
import torch

import mixer_reference as ref
from mixer_reference import assert_close

pytestmark = pytest.mark.gpu
TOL = 2.0 ** -18
# one size for every register shape, and (odd widths) the any-width kernels of a warp and of a block to a row
WIDTHS = [64, 256, 512, 1024, 2048, 4096, 8192, 16384, 250, 1603]


@pytest.mark.parametrize("N", WIDTHS)
@pytest.mark.parametrize("dtype,mean,std", [(torch.float32, 1000.0, 1.0), (torch.float32, -1000.0, 0.01),
                                            (torch.bfloat16, 1000.0, 30.0)])
def test_large_mean(kda, N, dtype, mean, std):
    gen = torch.Generator().manual_seed(N)
    M = 37
    x, dy = (mean + std * torch.randn((M, N), generator=gen)).to(dtype), torch.randn((M, N), generator=gen).to(dtype)
    w = 1 + 0.2 * torch.randn(N, generator=gen)
    xd = x.double()
    mu = xd.mean(1).float()
    rs = ((xd - mu.double()[:, None]) ** 2).mean(1).add(1e-5).rsqrt().float()
    dx, dw, db = kda.layer_norm_bwd(dy.cuda(), x.cuda(), w.cuda(), mu.cuda(), rs.cuda())
    dxr, dwr, dbr = ref.norm_bwd(dy.double(), xd, w.double(), mu.double(), rs.double())
    assert_close(dx, dxr, dtype, TOL, "dx")
    assert_close(dw, dwr, torch.float32, TOL * M ** 0.5, "dw")
    assert_close(db, dbr, torch.float32, TOL * M ** 0.5, "db")


@pytest.mark.parametrize("N", WIDTHS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_constant_rows(kda, N, dtype):
    """xh is exactly 0: so is the weight's gradient, and dx is rstd (c - mean(c))."""
    gen = torch.Generator().manual_seed(N + 1)
    M = 9
    mu = (1234.567 + 100 * torch.randn(M, generator=gen)).to(dtype).float()
    x, dy = mu[:, None].expand(M, N).to(dtype).contiguous(), torch.randn((M, N), generator=gen).to(dtype)
    w = 1 + 0.2 * torch.randn(N, generator=gen)
    rs = torch.full((M,), 1e-5 ** -0.5)
    dx, dw, db = kda.layer_norm_bwd(dy.cuda(), x.cuda(), w.cuda(), mu.cuda(), rs.cuda())
    assert not dw.any()
    dxr, _, dbr = ref.norm_bwd(dy.double(), x.double(), w.double(), mu.double(), rs.double())
    assert_close(dx, dxr, dtype, TOL, "dx")
    assert_close(db, dbr, torch.float32, TOL * M ** 0.5, "db")
