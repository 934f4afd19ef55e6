"""The selective scan, its gradients and its step on the GPU against float64.

The state is a product of up to T decays, each off by 2^-22 (the fast exponential) and 2^-24 times its exponent (under
2^-22 at the exponents here), then a sum of T terms: at most T 2^-20 of the terms' absolute sum, and 16 half steps for
the sum over the states, the step size and the gate.  Outputs of random-sign terms are smaller than those sums by up
to a factor of about 8; errors of random sign grow with sqrt(T), not T.  So (sqrt(T) + 16) 2^-20 for outputs and
states, twice that for gradients (two recurrences), and sqrt(tokens) more for the sums over tokens (dA, dD, dbias)
at their share of 2^-20."""
import pytest
import torch

import mixer_reference as ref
from mixer_reference import assert_close

pytestmark = pytest.mark.gpu


def make(B, T, ch, G, N, cu, dtype, seed, gate=True, skip=True, bias=True, state=True):
    gen = torch.Generator().manual_seed(seed)
    n = B if cu is None else len(cu) - 1
    r = lambda *s, std=1.0: (std * torch.randn(s, generator=gen)).to(dtype)  # noqa: E731
    f = lambda *s, std=1.0: std * torch.randn(s, generator=gen)  # noqa: E731
    A = -torch.arange(1, N + 1).float().repeat(ch, 1) * torch.exp(f(ch, N, std=0.1))
    return dict(u=r(B, T, ch), dt=r(B, T, ch, std=0.5), A=A, Bm=r(B, T, G, N), Cm=r(B, T, G, N),
                D=f(ch) if skip else None, z=r(B, T, ch) if gate else None, bias=f(ch) - 2 if bias else None,
                h0=f(n, ch, N, std=0.3) if state else None, dy=r(B, T, ch), dh=f(n, ch, N, std=0.3) if state else None)


def check(kda, c, cu, dtype, sp=True):
    d = {k: None if v is None else v.double() for k, v in c.items()}
    g = {k: None if v is None else v.cuda() for k, v in c.items()}
    cug = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    B, T, _ = c["u"].shape
    longest = T if cu is None else max(b - a for a, b in zip(cu, cu[1:]))
    tol = (longest ** 0.5 + 16) * 2.0 ** -20
    y, fin = kda.selective_scan_fwd(g["u"], g["dt"], g["A"], g["Bm"], g["Cm"], g["D"], g["z"], g["bias"], sp, g["h0"], cug)
    yr, finr = ref.scan(d["u"], d["dt"], d["A"], d["Bm"], d["Cm"], d["D"], d["z"], d["bias"], sp, d["h0"], cu)
    assert_close(y, yr, dtype, tol, "y")
    assert_close(fin, finr, torch.float32, tol, "final state")
    got = kda.selective_scan_bwd(g["dy"], g["u"], g["dt"], g["A"], g["Bm"], g["Cm"], g["D"], g["z"], g["bias"], sp, g["h0"],
                                 cug, g["dh"])
    want = ref.scan(d["u"], d["dt"], d["A"], d["Bm"], d["Cm"], d["D"], d["z"], d["bias"], sp, d["h0"], cu, d["dy"], d["dh"])
    names = ("du", "ddt", "dA", "dB", "dC", "dD", "dz", "dbias", "dh0")
    given = dict(dD=c["D"], dz=c["z"], dbias=c["bias"], dh0=c["h0"])
    total = (B * T) ** 0.5
    for name, p, q in zip(names, got, want):
        if name in given and given[name] is None:
            assert p is None
            continue
        low = name in ("du", "ddt", "dB", "dC", "dz")
        extra = total * 2.0 ** -20 if name in ("dA", "dD", "dbias") else 0.0
        assert_close(p, q, dtype if low else torch.float32, 2 * tol + extra, name)
    return g, cug, y, got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N", [1, 5, 8, 16, 32])
@pytest.mark.parametrize("B,T,ch,G", [(1, 1, 8, 1), (2, 3, 33, 1), (1, 33, 64, 2), (2, 70, 120, 3), (1, 257, 40, 1)])
def test_dense(kda, B, T, ch, G, N, dtype):
    check(kda, make(B, T, ch, G, N, None, dtype, T + ch + N), None, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cu", [[0, 1], [0, 0, 0, 3, 3, 40, 41, 64, 64], [0, 32, 64, 96], [0, 31, 65, 200, 200, 700]])
def test_packed(kda, cu, dtype):
    check(kda, make(1, cu[-1], 48, 1, 16, cu, dtype, cu[-1]), cu, dtype)
    check(kda, make(1, cu[-1], 24, 2, 4, cu, dtype, cu[-1] + 1, state=False), cu, dtype)


@pytest.mark.parametrize("N", [4, 16, 32])
@pytest.mark.parametrize("cu", [None, [0, 5, 600, 600, 601, 1500], [0, 1499, 1500], [0, 512, 1024, 1500]])
def test_segments(kda, cu, N):
    """Long enough to be cut: segments that start inside, at and between sequences."""
    check(kda, make(1, 1500, 32, 1, N, cu, torch.float32, 11 + N), cu, torch.float32)


@pytest.mark.parametrize("gate,skip,bias,state,sp", [(False, False, False, False, True), (True, False, True, False, False),
                                                     (False, True, False, True, True)])
def test_options(kda, gate, skip, bias, state, sp):
    c = make(2, 45, 32, 1, 16, None, torch.float32, 21, gate, skip, bias, state)
    if not sp:  # the step size is used as it is: keep it small and positive, as such a caller does
        c["dt"] = c["dt"].abs() * 0.1
        c["bias"] = None if c["bias"] is None else c["bias"].abs() * 0.05
    check(kda, c, None, torch.float32, sp)


def test_slices_of_a_projection(kda):
    """x and z, and B and C, as slices of wider rows, on and off 16-byte boundaries."""
    gen = torch.Generator().manual_seed(8)
    for off in (0, 3):
        xz = torch.randn((2, 40, 2 * 64 + 8), generator=gen).to(torch.bfloat16).cuda()
        bc = torch.randn((2, 40, 8 + 32 + 8), generator=gen).to(torch.bfloat16).cuda()
        u, z = xz[:, :, off:off + 64], xz[:, :, off + 64:off + 128]
        Bm, Cm = (bc[:, :, None, 8 + off + k:8 + off + k + 16] for k in (0, 16))
        dt = torch.randn((2, 40, 64), generator=gen).to(torch.bfloat16).cuda()
        A = -torch.rand((64, 16), generator=gen).cuda() - 0.1
        d = lambda t: t.double().cpu()  # noqa: E731
        y, fin = kda.selective_scan_fwd(u, dt, A, Bm, Cm, z=z)
        yr, finr = ref.scan(d(u), d(dt), d(A), d(Bm), d(Cm), z=d(z))
        assert_close(y, yr, torch.bfloat16, 24 * 2.0 ** -20)
        assert_close(fin, finr, torch.float32, 24 * 2.0 ** -20)
        got = kda.selective_scan_bwd(u, u, dt, A, Bm, Cm, z=z)
        want = ref.scan(d(u), d(dt), d(A), d(Bm), d(Cm), z=d(z), dy=d(u))
        for i in (0, 1, 3, 4, 6):
            assert_close(got[i], want[i], torch.bfloat16, 48 * 2.0 ** -20, str(i))


def test_same_bits_every_time(kda):
    cu = [0, 100, 900, 2000]
    g, cug, y, got = check(kda, make(1, 2000, 64, 2, 16, cu, torch.bfloat16, 31), cu, torch.bfloat16)
    for _ in range(2):
        y2, _ = kda.selective_scan_fwd(g["u"], g["dt"], g["A"], g["Bm"], g["Cm"], g["D"], g["z"], g["bias"], True, g["h0"], cug)
        got2 = kda.selective_scan_bwd(g["dy"], g["u"], g["dt"], g["A"], g["Bm"], g["Cm"], g["D"], g["z"], g["bias"], True,
                                      g["h0"], cug, g["dh"])
        assert torch.equal(y, y2) and all(torch.equal(p, q) for p, q in zip(got, got2))


def test_one_bad_sequence_leaves_the_others_alone(kda):
    """Infinities and NaN of one packed sequence reach no other one, forward or backward, across segments too."""
    cu = [0, 400, 800, 1300]
    c = make(1, 1300, 32, 1, 16, cu, torch.float32, 41)
    bad = {k: None if v is None else v.clone() for k, v in c.items()}
    for k in ("u", "z", "dy"):
        bad[k][0, 400:800] = float("nan")
    bad["Bm"][0, 400:800] = float("inf")
    bad["Cm"][0, 400:800] = float("-inf")
    bad["h0"][1] = float("nan")
    cug = torch.tensor(cu, dtype=torch.int32, device="cuda")
    outs = []
    for s in (c, bad):
        g = {k: v.cuda() for k, v in s.items()}
        a = (g["u"], g["dt"], g["A"], g["Bm"], g["Cm"], g["D"], g["z"], g["bias"], True, g["h0"], cug)
        outs.append(kda.selective_scan_fwd(*a) + kda.selective_scan_bwd(g["dy"], *a, g["dh"]))
    keep = torch.cat([torch.arange(0, 400), torch.arange(800, 1300)]).cuda()
    for i in (0, 2, 3, 5, 6, 8):  # y, du, ddt, dB, dC, dz
        assert torch.equal(outs[0][i][:, keep], outs[1][i][:, keep]), i
    for i in (1, 10):             # final states, gradients of the initial ones
        assert torch.equal(outs[0][i][[0, 2]], outs[1][i][[0, 2]]), i


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,ch,G,N", [(1, 8, 1, 16), (3, 33, 1, 5), (7, 96, 3, 8), (64, 256, 1, 16), (2, 40, 2, 32), (1, 1, 1, 1)])
def test_step_continues_the_sequence(kda, B, ch, G, N, dtype):
    """Steps from the state of a prefill are the next tokens of the whole sequence."""
    c = make(B, 9, ch, G, N, None, dtype, B + ch + N)
    g = {k: None if v is None else v.cuda() for k, v in c.items()}
    d = {k: None if v is None else v.double() for k, v in c.items()}
    want, fin = ref.scan(d["u"], d["dt"], d["A"], d["Bm"], d["Cm"], d["D"], d["z"], d["bias"], True, d["h0"])
    part = lambda k, s: g[k][:, s].contiguous()  # noqa: E731
    s = slice(0, 6)
    y, state = kda.selective_scan_fwd(part("u", s), part("dt", s), g["A"], part("Bm", s), part("Cm", s), g["D"], part("z", s),
                                      g["bias"], True, g["h0"])
    tol = 20 * 2.0 ** -20
    assert_close(y, want[:, :6], dtype, tol)
    for t in range(6, 9):
        y = kda.selective_scan_step(part("u", t), part("dt", t), g["A"], part("Bm", t), part("Cm", t), state, g["D"],
                                    part("z", t), g["bias"])
        assert_close(y, want[:, t], dtype, tol)
    assert_close(state, fin, torch.float32, tol)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,ch,G,N", [(75, 4096, 1, 16), (73, 4096, 2, 8), (41, 4096, 1, 32), (150, 2080, 4, 16), (74, 4093, 1, 16)])
def test_step_of_many_sequences(kda, B, ch, G, N, dtype):
    """Enough sequences for the kernel whose threads walk over them; the last one goes without a gate."""
    c = make(B, 1, ch, G, N, None, dtype, B + N, gate=ch != 4093)
    d = {k: None if v is None else v.double() for k, v in c.items()}
    one = lambda k: None if c[k] is None else c[k][:, 0].cuda()  # noqa: E731
    state = c["h0"].cuda()
    y = kda.selective_scan_step(one("u"), one("dt"), c["A"].cuda(), one("Bm"), one("Cm"), state, c["D"].cuda(), one("z"),
                                c["bias"].cuda())
    want, fin = ref.scan(d["u"], d["dt"], d["A"], d["Bm"], d["Cm"], d["D"], d["z"], d["bias"], True, d["h0"])
    assert_close(y, want[:, 0], dtype, 20 * 2.0 ** -20)
    assert_close(state, fin, torch.float32, 20 * 2.0 ** -20)


def test_no_tokens_and_state_in_place(kda):
    e = torch.empty((2, 0, 16), device="cuda")
    A, bc = -torch.ones((16, 4), device="cuda"), torch.empty((2, 0, 1, 4), device="cuda")
    h = torch.randn((2, 16, 4), device="cuda")
    y, fin = kda.selective_scan_fwd(e, e.clone(), A, bc, bc.clone(), initial_state=h)
    assert y.shape == (2, 0, 16) and torch.equal(fin, h)
    got = kda.selective_scan_bwd(e, e.clone(), e.clone(), A, bc, bc.clone(), initial_state=h, d_final_state=h.clone())
    assert torch.equal(got[8], h) and not got[2].any()
    c = make(1, 700, 32, 1, 16, [0, 300, 700], torch.float32, 51)
    g = {k: v.cuda() for k, v in c.items()}
    cu = torch.tensor([0, 300, 700], dtype=torch.int32, device="cuda")
    a = (g["u"], g["dt"], g["A"], g["Bm"], g["Cm"])
    y0, f0 = kda.selective_scan_fwd(*a, initial_state=g["h0"], cu_seqlens=cu)
    y1, f1 = kda.selective_scan_fwd(*a, initial_state=g["h0"], cu_seqlens=cu, final_state=g["h0"])
    assert f1.data_ptr() == g["h0"].data_ptr() and torch.equal(y0, y1) and torch.equal(f0, f1)
