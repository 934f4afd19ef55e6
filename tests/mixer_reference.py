"""Plain float64 statements of the selective mixer's operators -- TEST INFRASTRUCTURE.

Loops over tokens and sequences, torch on the CPU in float64; gradients by the
formulas, which tests/test_mixer_reference.py compares with differences."""
import torch


def silu(x):
    return x * torch.sigmoid(x)


def dsilu(x):
    s = torch.sigmoid(x)
    return s + x * s * (1 - s)


def softplus(x):
    return torch.logaddexp(x, torch.zeros_like(x))


def act(x, kind):
    """Value and derivative."""
    if kind == "none":
        return x, torch.ones_like(x)
    if kind == "relu":
        return torch.clamp(x, min=0), (x > 0).to(x.dtype)
    if kind == "silu":
        return silu(x), dsilu(x)
    if kind == "softplus":
        return softplus(x), torch.sigmoid(x)
    cdf = 0.5 * torch.erfc(-x * 0.5 ** 0.5)
    return x * cdf, cdf + x * torch.exp(-0.5 * x * x) / (2 * torch.pi) ** 0.5


def norm_fwd(x, w, b, eps):
    mean = x.mean(-1, keepdim=True)
    rstd = ((x - mean) ** 2).mean(-1, keepdim=True).add(eps).rsqrt()
    y = (x - mean) * rstd
    y = y * w if w is not None else y
    y = y + b if b is not None else y
    return y, mean[..., 0], rstd[..., 0]


def norm_bwd(dy, x, w, mean, rstd):
    xh = (x - mean[..., None]) * rstd[..., None]
    c = dy * w if w is not None else dy
    dx = rstd[..., None] * (c - c.mean(-1, keepdim=True) - xh * (c * xh).mean(-1, keepdim=True))
    return dx, (dy * xh).reshape(-1, x.shape[-1]).sum(0), dy.reshape(-1, x.shape[-1]).sum(0)


def bounds(B, T, cu):
    return [b * T for b in range(B + 1)] if cu is None else [int(c) for c in cu]


def conv(x, w, b, cu, state, use_silu, dy=None, dstate=None):
    """Forward: (y, state out).  With dy: (dx, dw, db, gradient of the incoming state)."""
    B, T, C = x.shape
    W = w.shape[1]
    bd = bounds(B, T, cu)
    flat = x.reshape(B * T, C)
    y, tails = torch.zeros_like(flat), []
    dx, dw, db, din = torch.zeros_like(flat), torch.zeros_like(w), torch.zeros(C, dtype=x.dtype), []
    for n in range(len(bd) - 1):
        lo, hi = bd[n], bd[n + 1]
        old = state[n] if state is not None else torch.zeros(W - 1, C, dtype=x.dtype)
        full = torch.cat([old, flat[lo:hi]])
        s = torch.zeros(hi - lo, C, dtype=x.dtype) + (b if b is not None else 0)
        for j in range(W):
            s = s + full[j:j + hi - lo] * w[:, j]
        y[lo:hi] = silu(s) if use_silu else s
        tails.append(full[len(full) - (W - 1):])
        if dy is not None:
            ds = dy.reshape(B * T, C)[lo:hi] * (dsilu(s) if use_silu else 1)
            df = torch.zeros_like(full)
            for j in range(W):
                df[j:j + hi - lo] += ds * w[:, j]
                dw[:, j] += (ds * full[j:j + hi - lo]).sum(0)
            db += ds.sum(0)
            if dstate is not None:
                df[len(full) - (W - 1):] += dstate[n]
            dx[lo:hi] = df[W - 1:]
            din.append(df[:W - 1])
    if dy is not None:
        return dx.reshape(x.shape), dw, db, torch.stack(din)
    return y.reshape(x.shape), torch.stack(tails)


def scan(u, dt, A, Bm, Cm, D=None, z=None, bias=None, sp=True, h0=None, cu=None, dy=None, dhT=None):
    """Forward: (y, final states).  With dy: every gradient, in selective_scan_bwd's order."""
    B, T, ch = u.shape
    G, N = Bm.shape[-2:]
    bd = bounds(B, T, cu)
    M, nseq = B * T, len(bd) - 1
    uf, dtf = u.reshape(M, ch), dt.reshape(M, ch)
    Bf = Bm.reshape(M, G, N).repeat_interleave(ch // G, 1)
    Cf = Cm.reshape(M, G, N).repeat_interleave(ch // G, 1)
    raw = dtf + (bias if bias is not None else 0)
    step = softplus(raw) if sp else raw
    skip = D if D is not None else torch.zeros(ch, dtype=u.dtype)
    final = torch.zeros(nseq, ch, N, dtype=u.dtype)
    before, hs = torch.zeros(M, ch, N, dtype=u.dtype), torch.zeros(M, ch, N, dtype=u.dtype)
    a = torch.exp(step[..., None] * A)
    for n in range(nseq):
        h = h0[n].clone() if h0 is not None else torch.zeros(ch, N, dtype=u.dtype)
        for t in range(bd[n], bd[n + 1]):
            before[t] = h
            h = a[t] * h + (step[t] * uf[t])[:, None] * Bf[t]
            hs[t] = h
        final[n] = h
    ysum = (hs * Cf).sum(-1) + skip * uf
    gate = silu(z.reshape(M, ch)) if z is not None else 1.0
    if dy is None:
        return (ysum * gate).reshape(u.shape), final
    dyf = dy.reshape(M, ch)
    p = dyf * gate
    g_all, dh0 = torch.zeros_like(hs), torch.zeros(nseq, ch, N, dtype=u.dtype)
    for n in range(nseq):
        g = dhT[n].clone() if dhT is not None else torch.zeros(ch, N, dtype=u.dtype)
        for t in range(bd[n + 1] - 1, bd[n] - 1, -1):
            g = g + Cf[t] * p[t][:, None]
            g_all[t] = g
            g = a[t] * g
        dh0[n] = g
    e = g_all * a * before
    gb = (g_all * Bf).sum(-1)
    dstep = gb * uf + (e * A).sum(-1)
    ddt = dstep * torch.sigmoid(raw) if sp else dstep
    fold = lambda x: x.reshape(M, G, ch // G, N).sum(2).reshape(Bm.shape)  # noqa: E731
    return ((gb * step + skip * p).reshape(u.shape), ddt.reshape(u.shape), (e * step[..., None]).sum(0),
            fold(g_all * (step * uf)[..., None]), fold(hs * p[..., None]), (p * uf).sum(0),
            (dyf * ysum * dsilu(z.reshape(M, ch))).reshape(u.shape) if z is not None else None, ddt.sum(0), dh0)


# ---------------------------------------------------------------- tolerances
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # of one rounding, relative


def assert_close(got, want, out_dtype, fp32_rel, what=""):
    """Relative L2 of an output against float64: at most half a step of its own type for the one rounding of the
    result, plus fp32_rel for the fp32 arithmetic before it (each caller derives its own); and no element off by more
    than the rounding of its own size and 40 times that arithmetic's share of the largest.  Exact where want is zero
    everywhere."""
    assert got is not None, what
    got = got.detach().double().cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    if want.numel() == 0:
        return
    assert torch.isfinite(got).all(), what
    err, norm, big = (got - want), want.norm(), want.abs().max()
    half = HALF_STEP[out_dtype]
    rel = float(err.norm() / norm) if norm > 0 else float(err.norm())
    assert rel <= half + fp32_rel, (what, rel, half + fp32_rel)
    over = (err.abs() - half * want.abs() - 40 * fp32_rel * big).max()
    assert over <= 0, (what, float(over), float(big))
