"""The selective scan on a packed buffer that is longer than its sequences: the rows that an offset covers, the final
states and the gradients of the initial ones do not depend on the rows left out.

Tolerances as in test_mixer_scan_gpu.py."""
import pytest
import torch

import mixer_reference as ref
from mixer_reference import assert_close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [4, 16, 32])
@pytest.mark.parametrize("T,cu", [(40, [0, 13, 29]), (40, [0, 0]), (70, [0, 31, 32, 32]), (1500, [0, 5, 600, 1203]),
                                  (1500, [0, 700, 1499]), (1500, [0, 17])])
def test_rows_behind_the_last_sequence(kda, T, cu, N):
    gen = torch.Generator().manual_seed(T + cu[-1] + N)
    ch, n, last = 40, len(cu) - 1, cu[-1]
    r = lambda *s, std=1.0: std * torch.randn(s, generator=gen)  # noqa: E731
    A = -torch.arange(1, N + 1).float().repeat(ch, 1) * torch.exp(0.1 * r(ch, N))
    t = dict(u=r(1, T, ch), dt=r(1, T, ch, std=0.5), A=A, Bm=r(1, T, 1, N), Cm=r(1, T, 1, N), D=r(ch), z=r(1, T, ch),
             bias=r(ch) - 2, h0=r(n, ch, N, std=0.3), dy=r(1, T, ch), dh=r(n, ch, N, std=0.3))
    t["dy"][0, last:] = 0
    cug = torch.tensor(cu, dtype=torch.int32, device="cuda")
    d = {k: v.double() for k, v in t.items()}
    names = ("u", "dt", "A", "Bm", "Cm", "D", "z", "bias")
    a64 = tuple(d[k] for k in names) + (True, d["h0"], cu)
    yr, finr = ref.scan(*a64)
    want = ref.scan(*a64, d["dy"], d["dh"])
    longest = max(b - a for a, b in zip(cu, cu[1:]))
    tol = (longest ** 0.5 + 16) * 2.0 ** -20
    for behind in (0, 1):  # what the rows left out hold: finite values without a gradient, then anything
        if behind:
            for k in ("u", "dt", "Bm", "Cm", "z", "dy"):
                t[k][0, last:] = float("nan")
        g = {k: v.cuda() for k, v in t.items()}
        args = tuple(g[k] for k in names) + (True, g["h0"], cug)
        y, fin = kda.selective_scan_fwd(*args)
        assert_close(y[:, :last], yr[:, :last], torch.float32, tol, "y")
        assert_close(fin, finr, torch.float32, tol, "final state")
        got = kda.selective_scan_bwd(g["dy"], *args, g["dh"])
        for i, name in enumerate(("du", "ddt", "dA", "dB", "dC", "dD", "dz", "dbias", "dh0")):
            if name in ("dA", "dD", "dbias"):
                if not behind:
                    assert_close(got[i], want[i], torch.float32, 2 * tol + T ** 0.5 * 2.0 ** -20, name)
            elif name == "dh0":
                assert_close(got[i], want[i], torch.float32, 2 * tol, name)
            else:
                assert_close(got[i][:, :last], want[i][:, :last], torch.float32, 2 * tol, name)
