"""The projection's products with more tiles than the GPU has SMs, so that a block walks over several: the second
accumulator, the handing back of the first and the staging tile's reuse, for each tile width and each product.

On 148 SMs, 18944 rows are 148 tiles high and 19200 rows 150.  Columns: up to 64 take 64-wide tiles, 128 (at 150) take
128-wide ones, 512 (at 148) take 256-wide ones.  Tolerances as in test_mixer_linear_gpu.py."""
import pytest
import torch

import mixer_reference as ref
from mixer_reference import assert_close

pytestmark = pytest.mark.gpu
FP32, DS = 2.0 ** -12, 2.0 ** -8
# rows of the product (ragged at the end), columns, length of the sum
TILES = [(19173, 64, 200), (19173, 61, 72), (19200, 128, 72), (19173, 125, 200), (18944, 512, 136), (18907, 509, 72),
         (40000, 512, 64)]


def _t(gen, *shape, std=1.0):
    return (std * torch.randn(shape, generator=gen)).to(torch.bfloat16)


def _padded(t):
    """On the GPU, with rows on 16-byte boundaries."""
    full = torch.zeros((t.shape[0], (t.shape[1] + 7) // 8 * 8), device="cuda", dtype=t.dtype)
    full[:, :t.shape[1]] = t.cuda()
    return full[:, :t.shape[1]]


@pytest.mark.parametrize("M,N,K", TILES)
def test_forward(kda, M, N, K):
    gen = torch.Generator().manual_seed(M + N + K)
    x, W, r = _t(gen, M, K), _t(gen, N, K, std=K ** -0.5), _t(gen, M, N)
    b = 0.3 * torch.randn(N, generator=gen)
    s = x.double() @ W.double().T + b.double()
    y, pre = kda.linear_act(x.cuda(), W.cuda(), b.cuda(), r.cuda(), act="gelu", output_pre=True)
    y2 = kda.linear_act(x.cuda(), W.cuda(), b.cuda(), act="none")
    torch.cuda.synchronize()
    assert kda.device_status() == 0
    assert_close(y, ref.act(s, "gelu")[0] + r.double(), torch.bfloat16, FP32, "y")
    assert_close(pre, s, torch.bfloat16, FP32, "pre")
    assert_close(y2, s, torch.bfloat16, FP32, "y without the extras")


@pytest.mark.parametrize("rows,cols,length", TILES)
@pytest.mark.parametrize("product", ["dx", "dW"])
def test_gradients(kda, product, rows, cols, length):
    # dx is [M, K] summed over N, dW is [N, K] summed over M
    M, N, K = (rows, length, cols) if product == "dx" else (length, rows, cols)
    gen = torch.Generator().manual_seed(M + N + K + 1)
    x, W, dy, pre = _t(gen, M, K), _t(gen, N, K, std=K ** -0.5), _t(gen, M, N), _t(gen, M, N)
    dx, dW, db = kda.linear_act_bwd(dy.cuda(), _padded(x), _padded(W), pre.cuda(), "silu")
    torch.cuda.synchronize()
    assert kda.device_status() == 0
    ds = dy.double() * ref.act(pre.double(), "silu")[1]
    assert_close(dx, ds @ W.double(), torch.bfloat16, FP32 + DS, "dx")
    assert_close(dW, ds.T @ x.double(), torch.bfloat16, FP32 + DS, "dW")
    assert_close(db, ds.sum(0), torch.float32, 2.0 ** -18 * M ** 0.5, "db")
