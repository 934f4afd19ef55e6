"""linear_act and its gradients on the tensor cores against float64 products of the same bf16 values.

y and pre are rounded once from fp32 sums of K terms: K 2^-24 of their absolute sum, about sqrt(K) times the result
for random signs, so 2^-24 K^1.5 at the very most and 2^-13 at the K used here (the tensor cores' fp32 accumulation
may also cut low bits of aligned terms: 2^-22 each).  With a softplus or GELU the fast exponential and logarithm and
the error function add under 2^-18.  The gradients' operand ds is itself rounded to bf16 (2^-8 of each term): the
products of random signs keep that relative size, so dx and dW are within one more half step."""
import pytest
import torch

import mixer_reference as ref
from mixer_reference import assert_close

pytestmark = pytest.mark.gpu
FP32, DS = 2.0 ** -12, 2.0 ** -8


def _t(gen, *shape, std=1.0):
    return (std * torch.randn(shape, generator=gen)).to(torch.bfloat16)


def _fwd(kda, M, N, K, act, bias, residual, pre, seed=0):
    gen = torch.Generator().manual_seed(seed + M + 3 * N + 7 * K)
    x, W = _t(gen, M, K), _t(gen, N, K, std=K ** -0.5)
    b = 0.3 * torch.randn(N, generator=gen) if bias else None
    r = _t(gen, M, N) if residual else None
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    out = kda.linear_act(x.cuda(), W.cuda(), c(b), c(r), act=act, output_pre=pre)
    torch.cuda.synchronize()
    assert kda.device_status() == 0
    y, p = out if pre else (out, None)
    s = x.double() @ W.double().T + (b.double() if bias else 0)
    want = ref.act(s, act)[0] + (r.double() if residual else 0)
    assert_close(y, want, torch.bfloat16, FP32, "y")
    if pre:
        assert_close(p, s, torch.bfloat16, FP32, "pre")
    return y


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu", "softplus"])
@pytest.mark.parametrize("bias,residual,pre", [(True, True, True), (True, False, False), (False, True, False)])
def test_epilogues(kda, act, bias, residual, pre):
    _fwd(kda, 200, 264, 136, act, bias, residual, pre)


@pytest.mark.parametrize("M,N,K", [(1, 1, 8), (1, 256, 64), (2, 2048, 4096), (5, 17, 1312), (16, 2048, 4096), (16, 100, 72),
                                   (17, 33, 40), (32, 520, 1032), (33, 64, 256), (64, 4096, 2048), (100, 1000, 520),
                                   (128, 256, 64), (129, 257, 72), (700, 384, 2048), (3000, 1500, 264)])
def test_sizes(kda, M, N, K):
    _fwd(kda, M, N, K, "silu", True, True, False)
    _fwd(kda, M, N, K, "gelu", True, False, True)


def test_slices_and_odd_strides(kda):
    gen = torch.Generator().manual_seed(3)
    M, N, K = 150, 130, 64
    xb, Wb, rb = _t(gen, M, K + 24), _t(gen, N, K + 8, std=0.1), _t(gen, M, N + 5)
    x, W, r = xb.cuda()[:, 16:16 + K], Wb.cuda()[:, 8:], rb.cuda()[:, 3:3 + N]
    full = torch.full((M, 152), float("nan"), device="cuda", dtype=torch.bfloat16)
    y = kda.linear_act(x, W, None, r, out=full[:, :N])
    assert y.data_ptr() == full.data_ptr() and full[:, N:].isnan().all()  # nothing written past the columns
    want = x.double().cpu() @ W.double().cpu().T + r.double().cpu()
    assert_close(y, want, torch.bfloat16, FP32)


def test_infinities_and_nan_stay_in_their_rows(kda):
    gen = torch.Generator().manual_seed(4)
    x, W, r = _t(gen, 140, 64), _t(gen, 300, 64), _t(gen, 140, 300)
    r[3, 5], r[4, 6] = float("inf"), float("nan")
    x[7, 2] = float("nan")
    y = kda.linear_act(x.cuda(), W.cuda(), None, r.cuda(), act="relu").cpu().float()
    bad = ~y.isfinite()
    want = torch.zeros_like(bad)
    want[3, 5] = want[4, 6] = True
    want[7] = True
    assert torch.equal(bad, want) and y[3, 5] == float("inf")


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu", "softplus"])
@pytest.mark.parametrize("M,N,K", [(1, 8, 8), (40, 24, 64), (300, 264, 136), (1000, 17, 200), (257, 640, 2048), (4096, 128, 256)])
def test_gradients(kda, M, N, K, act):
    gen = torch.Generator().manual_seed(M + N + K)
    x, W, dy, pre = _t(gen, M, K), _t(gen, N, K, std=K ** -0.5), _t(gen, M, N), _t(gen, M, N)
    dx, dW, db = kda.linear_act_bwd(dy.cuda(), x.cuda(), W.cuda(), None if act == "none" else pre.cuda(), act)
    torch.cuda.synchronize()
    assert kda.device_status() == 0
    ds = dy.double() * ref.act(pre.double(), act)[1]
    assert_close(dx, ds @ W.double(), torch.bfloat16, FP32 + DS, "dx")
    assert_close(dW, ds.T @ x.double(), torch.bfloat16, FP32 + DS, "dW")
    # db: fp32 sums of the unrounded ds; M terms of random sign
    assert_close(db, ds.sum(0), torch.float32, 2.0 ** -18 * M ** 0.5, "db")
    again = kda.linear_act_bwd(dy.cuda(), x.cuda(), W.cuda(), None if act == "none" else pre.cuda(), act)
    assert all(torch.equal(p, q) for p, q in zip((dx, dW, db), again))


def test_gradients_of_no_rows(kda):
    e = lambda *s: torch.empty(s, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    dx, dW, db = kda.linear_act_bwd(e(0, 24), e(0, 16), torch.ones(24, 16, device="cuda", dtype=torch.bfloat16), e(0, 24), "silu")
    assert dx.shape == (0, 16) and not dW.any() and not db.any()
    assert kda.linear_act(e(0, 16), e(24, 16)).shape == (0, 24)


def _in_padding(t):
    """t [rows, n] as columns of a tensor whose rows go on with NaN to the next multiple of 8 and 8 more."""
    rows, n = t.shape
    full = torch.full((rows, (n + 7) // 8 * 8 + 8), float("nan"), device="cuda", dtype=t.dtype)
    full[:, :n] = t.cuda()
    return full[:, :n]


@pytest.mark.parametrize("M", [1, 7, 16, 32, 50, 64, 150, 300])
@pytest.mark.parametrize("N,K", [(24, 1), (40, 12), (17, 31), (264, 100), (33, 1029)])
def test_sums_that_end_inside_a_vector(kda, M, N, K):
    """K not a multiple of 8: what a row holds behind its K values takes no part."""
    gen = torch.Generator().manual_seed(M + N + K)
    x, W = _t(gen, M, K), _t(gen, N, K, std=K ** -0.5)
    y = kda.linear_act(_in_padding(x), _in_padding(W))
    torch.cuda.synchronize()
    assert kda.device_status() == 0
    assert_close(y, x.double() @ W.double().T, torch.bfloat16, FP32)


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (5, 12, 20), (40, 17, 12), (150, 100, 31), (300, 1029, 33)])
def test_gradients_whose_sums_end_inside_a_vector(kda, M, N, K, act):
    gen = torch.Generator().manual_seed(M + N + K)
    x, W, dy, pre = _t(gen, M, K), _t(gen, N, K, std=K ** -0.5), _t(gen, M, N), _t(gen, M, N)
    ws = torch.full((1 << 24,), 255, device="cuda", dtype=torch.uint8)  # NaN in every type
    dx, dW, db = kda.linear_act_bwd(_in_padding(dy), _in_padding(x), _in_padding(W),
                                    None if act == "none" else _in_padding(pre), act, workspace=ws)
    torch.cuda.synchronize()
    assert kda.device_status() == 0
    ds = dy.double() * ref.act(pre.double(), act)[1]
    assert_close(dx, ds @ W.double(), torch.bfloat16, FP32 + DS, "dx")
    assert_close(dW, ds.T @ x.double(), torch.bfloat16, FP32 + DS, "dW")
    assert_close(db, ds.sum(0), torch.float32, 2.0 ** -18 * M ** 0.5, "db")
