"""The short convolution on a packed buffer that is longer than its sequences: the rows that an offset covers have their
outputs and gradients whatever the rows left out hold, for runs of every length.

Tolerances as in test_mixer_conv_gpu.py: 2^-18 for the fp32 arithmetic of an output, sqrt(tokens) of it for the sums."""
import pytest
import torch

import mixer_reference as ref
from mixer_reference import assert_close

pytestmark = pytest.mark.gpu
TOL = 2.0 ** -18


def check(kda, T, C, W, cu, dtype, state, behind, seed, columns=None):
    """``behind``: the gradient in the rows that the offsets leave out: 0, 1 (random), or NaN, there in the inputs too.  Sums
    are compared where it is 0."""
    gen = torch.Generator().manual_seed(seed)
    n = len(cu) - 1
    r = lambda *s, std=1.0: (std * torch.randn(s, generator=gen)).to(dtype)  # noqa: E731
    x, w, b, dy = r(1, T, C), r(C, W, std=0.4), 0.1 * torch.randn(C, generator=gen), r(1, T, C)
    st, dst = (r(n, W - 1, C), r(n, W - 1, C)) if state else (None, None)
    inside = torch.zeros(T, dtype=torch.bool)
    inside[cu[0]:cu[-1]] = True
    dy[0, ~inside] *= behind
    if behind != behind:
        x[0, ~inside] = behind
    pick = slice(None) if columns is None else columns
    d = lambda t: None if t is None else t[..., pick].double()  # noqa: E731  (channels are independent)
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    cug = torch.tensor(cu, dtype=torch.int32, device="cuda")
    y, out = kda.short_conv_fwd(c(x), c(w), c(b), cug, c(st), output_conv_state=True)
    args = (d(x), w[pick].double(), b[pick].double(), cu, d(st), True)
    yr, outr = ref.conv(*args)
    assert_close(y.cpu()[:, inside][..., pick], yr[:, inside], dtype, TOL, "y")
    assert torch.equal(out.cpu()[..., pick].double(), outr)
    dx, dw, db, din = kda.short_conv_bwd(c(dy), c(x), c(w), c(b), cug, c(st), c(dst))
    dxr, dwr, dbr, dinr = ref.conv(*args, d(dy), d(dst))
    assert_close(dx.cpu()[:, inside][..., pick], dxr[:, inside], dtype, TOL, "dx")
    if state:
        assert_close(din.cpu()[..., pick], dinr, dtype, TOL, "dstate")
    if behind == 0:
        assert_close(dw.cpu()[pick], dwr, dtype, TOL * T ** 0.5, "dw")
        assert_close(db.cpu()[pick], dbr, torch.float32, TOL * T ** 0.5, "db")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("behind", [0, 1, float("nan")])
@pytest.mark.parametrize("cu", [[0, 13, 29], [0, 32], [0, 31], [0, 33], [0, 30, 31], [0, 30, 30, 32, 32], [0, 1], [0, 0],
                                [0, 39]])
def test_rows_behind_the_last_sequence(kda, cu, behind, W, dtype):
    """40 rows in runs of 8 tokens: the last offset next to a run's edge, inside a run, one row before the buffer's end."""
    for C in (24, 9):  # vectors of channels, and one at a time
        for state in (False, True):
            check(kda, 40, C, W, cu, dtype, state, behind, 5 * cu[-1] + C + W)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("C", [4096, 1025])
@pytest.mark.parametrize("last", [5830, 5940, 5941, 5942, 5943, 5944])
def test_rows_behind_the_last_sequence_in_long_runs(kda, last, C, dtype):
    """6000 rows of 4096 channels: runs of 65 (forward) and 109 tokens; 1025 channels: 65 and 41."""
    columns = torch.arange(0, C, 41)
    for behind in (0, 1, float("nan")):
        check(kda, 6000, C, 4, [0, 700, last - 2, last], dtype, True, behind, last + C, columns)
