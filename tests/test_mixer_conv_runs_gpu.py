"""The short convolution where a thread's run of tokens is longer than the rows it keeps in flight (test_mixer_conv_gpu.py
has runs of 8 to 10 tokens): the refilled ring, its edge-free form and the sequences that start and end inside it.

A depthwise convolution's channels are independent, so a sample of them is compared, each with all of its tokens.
Tolerances as in test_mixer_conv_gpu.py: 2^-18 for the fp32 arithmetic of an output, sqrt(tokens) of it for the sums."""
import pytest
import torch

import mixer_reference as ref
from mixer_reference import assert_close

pytestmark = pytest.mark.gpu
TOL = 2.0 ** -18


def check(kda, B, T, C, W, cu, dtype, state, silu, seed):
    gen = torch.Generator().manual_seed(seed)
    n = B if cu is None else len(cu) - 1
    r = lambda *s, std=1.0: (std * torch.randn(s, generator=gen)).to(dtype)  # noqa: E731
    x, w, b, dy = r(B, T, C), r(C, W, std=0.4), 0.1 * torch.randn(C, generator=gen), r(B, T, C)
    st, dst = (r(n, W - 1, C), r(n, W - 1, C)) if state else (None, None)
    pick = torch.cat([torch.arange(0, C, 61), torch.tensor([C - 2, C - 1])])
    d = lambda t: None if t is None else t[..., pick].double()  # noqa: E731
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    cug = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    y, out = kda.short_conv_fwd(c(x), c(w), c(b), cug, c(st), silu, output_conv_state=True)
    args = (d(x), w[pick].double(), b[pick].double(), cu, d(st), silu)
    yr, outr = ref.conv(*args)
    assert_close(y.cpu()[..., pick], yr, dtype, TOL, "y")
    assert torch.equal(out.cpu()[..., pick].double(), outr)
    dx, dw, db, din = kda.short_conv_bwd(c(dy), c(x), c(w), c(b), cug, c(st), c(dst), silu)
    dxr, dwr, dbr, dinr = ref.conv(*args, d(dy), d(dst))
    assert_close(dx.cpu()[..., pick], dxr, dtype, TOL, "dx")
    assert_close(dw.cpu()[pick], dwr, dtype, TOL * (B * T) ** 0.5, "dw")
    assert_close(db.cpu()[pick], dbr, torch.float32, TOL * (B * T) ** 0.5, "db")
    if state:
        assert_close(din.cpu()[..., pick], dinr, dtype, TOL, "dstate")


def edges(run, ring, T):
    """Offsets at, one before and one behind a run's first row, a ring's first row in it and its last one; sequences of no,
    one, two and three tokens at each kind of place."""
    cu = [0, run - 1, run, run + 1, run + 1, run + ring, 2 * run + ring + 1, 2 * run + 2 * ring - 1, 2 * run + 2 * ring + 1,
          3 * run + ring // 2, 3 * run + ring // 2 + 3, 4 * run, 4 * run, 4 * run + 1, 5 * run - 3, 5 * run - 1, 6 * run + 2,
          10 * run, T - 2, T]
    assert cu == sorted(cu)
    return cu


# 6000 rows of 4096 channels (vectors of four): runs of 65 tokens in the forward pass, 10 rows in flight, and of 109 in the
# backward pass, 4 in flight.  6000 rows of 1025 channels (one at a time): 65 and 41.
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("C,back", [(4096, 109), (1025, 41)])
def test_packed(kda, C, back, W, dtype):
    check(kda, 1, 6000, C, W, edges(65, 10, 6000), dtype, True, True, C + W)
    check(kda, 1, 6000, C, W, edges(back, 4, 6000), dtype, False, W != 3, C + W + 1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_dense(kda, W, dtype):
    """3 sequences of 1999 tokens: their edges fall inside the runs (65 and 109 tokens)."""
    check(kda, 3, 1999, 4096, W, None, dtype, W != 3, W != 2, W)
    check(kda, 3, 1999, 1025, W, None, dtype, W == 3, W != 2, W + 10)
