"""Cases of the selective mixer's operators: layer norm, the projection with its epilogue, the short
causal convolution and the selective scan, each direction, for prompts, training and single tokens.

``run`` computes a case in its plain form (elementary torch operations in 32 bits), or, where ``own``
is true, by the framework's entry points.  ``exact`` states each operator in 64 bits, token by token."""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
ES = {"bf16": 2, "fp32": 4}


def listed():
    return [
        # pre-norm of the packed prefill that the layer runs: 65536 tokens of width 2048
        dict(name="norm prefill 65536x2048", op="norm", M=65536, N=2048, dtype="bf16"),
        # pre-norm of one decode step of a few sequences: the call's latency
        dict(name="norm decode 4x2048", op="norm", M=4, N=2048, dtype="bf16"),
        # its gradients in a training step
        dict(name="norm gradient 16384x2048", op="norm_bwd", M=16384, N=2048, dtype="bf16"),
        # a training forward pass of a wide projection: bias, GELU, residual, pre-activation kept
        dict(name="linear train 16384x8192x2048", op="linear", M=16384, N=8192, K=2048, act="gelu", bias=True,
             residual=True, pre=True),
        # the output projection of a decode step with its residual: bound by the weights
        dict(name="linear decode 16x2048x4096", op="linear", M=16, N=2048, K=4096, act="none", bias=True,
             residual=True, pre=False),
        # gradients of a projection with SiLU
        dict(name="linear gradient 8192x4096x2048", op="linear_bwd", M=8192, N=4096, K=2048, act="silu"),
        # the convolution in front of the scan, packed prefill
        dict(name="conv prefill 65536x4096", op="conv", B=1, T=65536, C=4096, W=4, seqs=8, dtype="bf16", cache=True),
        # its gradients, odd sizes, 32 bits
        dict(name="conv gradient 3x2047x2056", op="conv_bwd", B=3, T=2047, C=2056, W=4, seqs=0, dtype="fp32", cache=True),
        # one token for each of 256 sequences
        dict(name="conv decode 256x4096", op="conv_step", B=256, C=4096, W=4, dtype="bf16"),
        # the scan over a packed prompt of 8192 tokens, inner width 4096, 16 states a channel
        dict(name="scan prefill 8192x4096", op="scan", B=1, T=8192, D=4096, N=16, G=1, seqs=4, dtype="bf16", gate=True),
        # its gradients, odd length
        dict(name="scan gradient 2x2047x2048", op="scan_bwd", B=2, T=2047, D=2048, N=16, G=1, seqs=0, dtype="bf16",
             gate=True),
        # one token for each of 256 sequences: bound by the states
        dict(name="scan decode 256x4096", op="scan_step", B=256, D=4096, N=16, G=1, dtype="bf16", gate=True),
    ]


def draw(rng):
    def size(lo, hi):  # spread over the logarithm
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def width(lo, hi, step):  # mostly a multiple of `step`, sometimes odd
        n = size(lo, hi)
        return n if rng.random() < 0.25 else max(step, n // step * step)

    op = rng.choice(["norm", "norm_bwd", "linear", "linear_bwd", "conv", "conv_bwd", "conv_step", "scan", "scan_bwd",
                     "scan_step"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op in ("norm", "norm_bwd"):
        N = width(64, 8192, 8)
        return dict(op=op, M=size(1, 16384 * 2048 // N), N=N, dtype=dtype)
    if op == "linear":
        act = rng.choice(["none", "relu", "gelu", "silu", "softplus"])
        return dict(op=op, M=size(1, 16384), N=width(16, 8192, 16), K=size(8, 2048) // 8 * 8, act=act,
                    bias=rng.random() < 0.7, residual=rng.random() < 0.5, pre=rng.random() < 0.4)
    if op == "linear_bwd":
        return dict(op=op, M=size(8, 8192), N=size(16, 4096) // 8 * 8, K=size(8, 2048) // 8 * 8,
                    act=rng.choice(["none", "relu", "gelu", "silu", "softplus"]))
    if op in ("conv", "conv_bwd"):
        C, top = width(32, 4096, 8), 1 << (27 if op == "conv" else 23)
        seqs = rng.choice([0, size(1, 64)])
        B = 1 if seqs else rng.choice([1, 2, 3, 5])
        return dict(op=op, B=B, T=size(1, min(65536, max(1, top // (B * C)))), C=C, W=rng.choice([2, 3, 4, 4]), seqs=seqs,
                    dtype=dtype, cache=rng.random() < 0.5)
    if op == "conv_step":
        return dict(op=op, B=size(1, 256), C=width(32, 4096, 8), W=rng.choice([2, 3, 4, 4]), dtype=dtype)
    G, N = rng.choice([1, 1, 1, 2, 4]), rng.choice([16, 16, 16, 8, 32, 5])
    D = G * max(1, width(32, 4096 * 16 // max(N, 16), 8) // G)
    if op == "scan_step":
        return dict(op=op, B=size(1, 256), D=D, N=N, G=G, dtype=dtype, gate=rng.random() < 0.6)
    seqs = rng.choice([0, size(1, 32)])
    B = 1 if seqs else rng.choice([1, 2, 3, 5])
    top = (8192 * 4096 * 16 if op == "scan" else 2 * 2047 * 2048 * 16) // (B * D * N)
    return dict(op=op, B=B, T=size(1, max(1, min(16384, top))), D=D, N=N, G=G, seqs=seqs, dtype=dtype,
                gate=rng.random() < 0.6)


def prepare(case, seed):
    c, op = dict(case), case["op"]
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 1000 + 7)
    low = DT[c.get("dtype", "bf16")]

    def rnd(*shape, std=1.0, mean=0.0, t=low):
        return (mean + std * torch.randn(shape, generator=gen, device="cuda")).to(t)

    f32 = torch.float32
    s = dict(case=c)
    if op in ("norm", "norm_bwd"):
        M, N = c["M"], c["N"]
        s.update(x=rnd(M, N, std=1.5, mean=0.3), w=rnd(N, std=0.2, mean=1.0, t=f32), b=rnd(N, std=0.1, t=f32))
        if op == "norm_bwd":  # the statistics that the forward pass returned
            xf = s["x"].double()
            mean = xf.mean(1)
            rstd = 1.0 / torch.sqrt((xf - mean[:, None]).square().mean(1) + 1e-5)
            s.update(dy=rnd(M, N), mean=mean.float(), rstd=rstd.float())
    elif op in ("linear", "linear_bwd"):
        M, N, K = c["M"], c["N"], c["K"]
        s.update(x=rnd(M, K), W=rnd(N, K, std=1.0 / math.sqrt(K)))
        if op == "linear":
            s.update(b=rnd(N, std=0.3, t=f32) if c["bias"] else None, res=rnd(M, N) if c["residual"] else None)
        else:  # the pre-activation that the forward pass returned
            s.update(dy=rnd(M, N), pre=None if c["act"] == "none" else rnd(M, N))
    elif op == "conv_step":
        B, C, W = c["B"], c["C"], c["W"]
        s.update(x=rnd(B, C), w=rnd(C, W, std=0.4), b=rnd(C, std=0.1, t=f32), cache=rnd(B, W - 1, C))
    elif op in ("conv", "conv_bwd"):
        B, T, C, W = c["B"], c["T"], c["C"], c["W"]
        s["cu"], n = _offsets(c, seed)
        s.update(x=rnd(B, T, C), w=rnd(C, W, std=0.4), b=rnd(C, std=0.1, t=f32),
                 cache=rnd(n, W - 1, C) if c["cache"] else None)
        if op == "conv_bwd":
            s.update(dy=rnd(B, T, C), dcache=rnd(n, W - 1, C) if c["cache"] else None)
    else:
        B, D, N, G = c["B"], c["D"], c["N"], c["G"]
        lead = (B,) if op == "scan_step" else (B, c["T"])
        n = B
        if op != "scan_step":
            s["cu"], n = _offsets(c, seed)
        # step sizes log-uniform in [0.001, 0.1] through the inverse of softplus; A near -1 .. -N
        dt0 = torch.exp(torch.rand(D, generator=gen, device="cuda") * math.log(100.0) + math.log(1e-3))
        A = -torch.arange(1, N + 1, device="cuda", dtype=f32).repeat(D, 1) * torch.exp(0.1 * torch.randn((D, N), generator=gen, device="cuda"))
        s.update(u=rnd(*lead, D), dt=rnd(*lead, D, std=0.5), A=A, Bm=rnd(*lead, G, N), Cm=rnd(*lead, G, N),
                 skip=rnd(D, std=0.2, mean=1.0, t=f32), z=rnd(*lead, D) if c["gate"] else None,
                 bias=dt0 + torch.log(-torch.expm1(-dt0)), h0=rnd(n, D, N, std=0.1, t=f32))
        if op == "scan_bwd":
            s.update(dy=rnd(*lead, D), dh=rnd(n, D, N, std=0.1, t=f32))
    return s


def _offsets(c, seed):
    """Offsets of the packed sequences (now and then an empty one), or None for a dense batch; and how many sequences."""
    if not c["seqs"]:
        return None, c["B"]
    gen = torch.Generator().manual_seed(int(seed) + 99)
    cuts = torch.randint(0, c["T"] + 1, (c["seqs"] - 1,), generator=gen).sort().values
    cu = torch.cat([torch.zeros(1, dtype=torch.long), cuts, torch.full((1,), c["T"])])
    return cu.to(torch.int32).cuda(), c["seqs"]


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


def work(case):
    c, op = case, case["op"]
    e = ES[c.get("dtype", "bf16")]
    if op == "norm":
        return dict(bytes=2 * e * c["M"] * c["N"] + 8 * c["N"] + 8 * c["M"], flops=8 * c["M"] * c["N"])
    if op == "norm_bwd":
        return dict(bytes=3 * e * c["M"] * c["N"] + 12 * c["N"] + 8 * c["M"], flops=14 * c["M"] * c["N"])
    if op in ("linear", "linear_bwd"):
        M, N, K = c["M"], c["N"], c["K"]
        if op == "linear":
            b = 2 * (M * K + N * K + M * N * (1 + c["residual"] + c["pre"])) + 4 * N * c["bias"]
            return dict(bytes=b, flops=2 * M * N * K)
        return dict(bytes=2 * (2 * M * K + 2 * N * K + M * N * (1 + (c["act"] != "none"))) + 4 * N, flops=4 * M * N * K)
    if op == "conv_step":
        return dict(bytes=e * c["B"] * c["C"] * 2 * c["W"] + c["C"] * (e * c["W"] + 4), flops=c["B"] * c["C"] * (2 * c["W"] + 4))
    if op in ("conv", "conv_bwd"):
        M, C, W = c["B"] * c["T"], c["C"], c["W"]
        n = (c["seqs"] or c["B"]) * c["cache"] * (W - 1) * C * 2 * e
        back = op == "conv_bwd"
        return dict(bytes=(3 if back else 2) * M * C * e + n + (1 + back) * C * (e * W + 4), flops=M * C * ((6 if back else 2) * W + 4))
    B, D, N, G = c["B"], c["D"], c["N"], c["G"]
    if op == "scan_step":
        return dict(bytes=8 * B * D * N + e * B * (D * (3 + c["gate"]) + 2 * G * N) + 4 * D * (N + 2), flops=7 * B * D * N)
    M, n = B * c["T"], c["seqs"] or B
    if op == "scan":
        return dict(bytes=e * M * (D * (3 + c["gate"]) + 2 * G * N) + 8 * n * D * N + 4 * D * (N + 2), flops=7 * M * D * N)
    return dict(bytes=e * M * (D * (5 + 2 * c["gate"]) + 4 * G * N) + 12 * n * D * N + 8 * D * (N + 2), flops=24 * M * D * N)


# ---------------------------------------------------------------- the framework's calls
def _own(s):
    import gated_delta_rule_123_b200 as kda
    c, op = s["case"], s["case"]["op"]
    if op == "norm":
        return kda.layer_norm_fwd(s["x"], s["w"], s["b"], eps=1e-5)
    if op == "norm_bwd":
        return kda.layer_norm_bwd(s["dy"], s["x"], s["w"], s["mean"], s["rstd"])
    if op == "linear":
        return kda.linear_act(s["x"], s["W"], bias=s["b"], residual=s["res"], act=c["act"], output_pre=c["pre"])
    if op == "linear_bwd":
        return kda.linear_act_bwd(s["dy"], s["x"], s["W"], pre=s["pre"], act=c["act"])
    if op == "conv":
        return kda.short_conv_fwd(s["x"], s["w"], bias=s["b"], cu_seqlens=s["cu"], conv_state=s["cache"],
                                  output_conv_state=c["cache"])
    if op == "conv_bwd":
        return kda.short_conv_bwd(s["dy"], s["x"], s["w"], bias=s["b"], cu_seqlens=s["cu"], conv_state=s["cache"],
                                  d_conv_state_out=s["dcache"])
    if op == "conv_step":
        return kda.short_conv_step(s["x"], s["w"], s["cache"], bias=s["b"]), s["cache"]
    if op == "scan":
        return kda.selective_scan_fwd(s["u"], s["dt"], s["A"], s["Bm"], s["Cm"], D=s["skip"], z=s["z"], dt_bias=s["bias"],
                                      initial_state=s["h0"], cu_seqlens=s["cu"])
    if op == "scan_bwd":
        return kda.selective_scan_bwd(s["dy"], s["u"], s["dt"], s["A"], s["Bm"], s["Cm"], D=s["skip"], z=s["z"],
                                      dt_bias=s["bias"], initial_state=s["h0"], cu_seqlens=s["cu"], d_final_state=s["dh"])
    y = kda.selective_scan_step(s["u"], s["dt"], s["A"], s["Bm"], s["Cm"], s["h0"], D=s["skip"], z=s["z"], dt_bias=s["bias"])
    return y, s["h0"]


# ---------------------------------------------------------------- the plain forms, 32 bits
def _norm(s):
    x = s["x"].float()
    mean = x.mean(1)
    xc = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((xc * xc).mean(1) + 1e-5)
    return (xc * rstd[:, None] * s["w"] + s["b"]).to(s["x"].dtype), mean, rstd


def _norm_bwd(s):
    dy, r = s["dy"].float(), s["rstd"][:, None]
    xh = (s["x"].float() - s["mean"][:, None]) * r
    g = dy * s["w"]
    dx = r * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return dx.to(s["x"].dtype), (dy * xh).sum(0), dy.sum(0)


def _softplus(x):
    return torch.clamp(x, min=0.0) + torch.log1p(torch.exp(-torch.abs(x)))


def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _act(x, kind):
    if kind == "none":
        return x
    if kind == "relu":
        return torch.clamp(x, min=0.0)
    if kind == "gelu":
        return 0.5 * x * (1.0 + torch.erf(x * math.sqrt(0.5)))
    return x * _sigmoid(x) if kind == "silu" else _softplus(x)


def _dact(x, kind):
    if kind == "relu":
        return (x > 0).to(x.dtype)
    if kind == "gelu":
        return 0.5 * (1.0 + torch.erf(x * math.sqrt(0.5))) + x * torch.exp(-0.5 * x * x) / math.sqrt(2.0 * math.pi)
    g = _sigmoid(x)
    return g * (1.0 + x * (1.0 - g)) if kind == "silu" else g


def _linear(s):
    c, t = s["case"], s["x"].dtype
    pre = s["x"].float() @ s["W"].float().T
    pre = pre + s["b"] if s["b"] is not None else pre
    y = _act(pre, c["act"])
    y = (y + s["res"].float() if s["res"] is not None else y).to(t)
    return (y, pre.to(t)) if c["pre"] else y


def _linear_bwd(s):
    ds = s["dy"].float()
    if s["pre"] is not None:
        ds = ds * _dact(s["pre"].float(), s["case"]["act"])
    t = s["x"].dtype
    return (ds @ s["W"].float()).to(t), (ds.T @ s["x"].float()).to(t), ds.sum(0)


def _places(s, M, T):
    """For every token of the flattened batch: its sequence and that sequence's first token; and all bounds."""
    t = torch.arange(M, device="cuda")
    if s["cu"] is None:
        bounds = torch.arange(0, M + 1, T, device="cuda")
    else:
        bounds = s["cu"].long()
    seq = (t[:, None] >= bounds[None, 1:]).sum(1)
    return t, seq, bounds


def _window(s, x, t, seq, bounds, W):
    """Input j of every token's window, j = 0 .. W-1 (the last is the token itself): [W, M, C]."""
    src = t[None, :] - torch.arange(W - 1, -1, -1, device="cuda")[:, None]
    row = src - bounds[seq][None, :]
    win = x[src.clamp(min=0)]
    if s["cache"] is not None:
        old = s["cache"].float()[seq[None, :].expand(W, -1), (row + W - 1).clamp(max=W - 2)]
    else:
        old = torch.zeros_like(win)
    return torch.where((row >= 0)[..., None], win, old), src, row


def _tail(s, W, C, bounds):
    """Where each row of the cache after the call comes from: a token (>= 0 in `tok`), else a row of the old cache."""
    n = bounds.numel() - 1
    tok = bounds[1:, None] - (W - 1) + torch.arange(W - 1, device="cuda")
    return tok, tok - bounds[:-1, None], torch.arange(n, device="cuda")[:, None].expand(n, W - 1)


def _conv(s):
    B, T, C = s["x"].shape
    W, low = s["w"].shape[1], s["x"].dtype
    x = s["x"].reshape(B * T, C).float()
    t, seq, bounds = _places(s, B * T, T)
    win, _, _ = _window(s, x, t, seq, bounds, W)
    pre = (win * s["w"].float().T[:, None, :]).sum(0) + s["b"]
    y = (pre * _sigmoid(pre)).to(low).reshape(B, T, C)
    if s["cache"] is None:
        return y, None
    tok, row, n = _tail(s, W, C, bounds)
    new = torch.where((row >= 0)[..., None], s["x"].reshape(B * T, C)[tok.clamp(min=0)], s["cache"][n, (row + W - 1).clamp(max=W - 2)])
    return y, new


def _conv_bwd(s):
    B, T, C = s["x"].shape
    W, low = s["w"].shape[1], s["x"].dtype
    x, w = s["x"].reshape(B * T, C).float(), s["w"].float()
    t, seq, bounds = _places(s, B * T, T)
    win, src, row = _window(s, x, t, seq, bounds, W)
    pre = (win * w.T[:, None, :]).sum(0) + s["b"]
    g = _sigmoid(pre)
    ds = s["dy"].reshape(B * T, C).float() * g * (1.0 + pre * (1.0 - g))
    dwin = ds[None] * w.T[:, None, :]
    keep = (row >= 0)[..., None]
    dx = torch.zeros_like(x)
    dx.index_add_(0, src.clamp(min=0).reshape(-1), torch.where(keep, dwin, 0.0).reshape(-1, C))
    dcache = None
    if s["cache"] is not None:
        n_seq = bounds.numel() - 1
        dcache = torch.zeros(n_seq * (W - 1), C, device="cuda")
        at = seq[None, :] * (W - 1) + (row + W - 1).clamp(max=W - 2)
        dcache.index_add_(0, at.reshape(-1), torch.where(keep, 0.0, dwin).reshape(-1, C))
        tok, trow, n = _tail(s, W, C, bounds)
        dnew, inside = s["dcache"].float(), (trow >= 0)[..., None]
        dx.index_add_(0, tok.clamp(min=0).reshape(-1), torch.where(inside, dnew, 0.0).reshape(-1, C))
        at = n * (W - 1) + (trow + W - 1).clamp(max=W - 2)
        dcache.index_add_(0, at.reshape(-1), torch.where(inside, 0.0, dnew).reshape(-1, C))
        dcache = dcache.reshape(n_seq, W - 1, C).to(low)
    return dx.to(low).reshape(B, T, C), (ds[None] * win).sum(1).T.contiguous().to(low), ds.sum(0), dcache


def _conv_step(s):
    win = torch.cat([s["cache"], s["x"][:, None]], 1)
    pre = (win.float() * s["w"].float().T).sum(1) + s["b"]
    s["cache"].copy_(win[:, 1:])
    return (pre * _sigmoid(pre)).to(s["x"].dtype), s["cache"]


def _recur(a, b):
    """h_t = a_t h_{t-1} + b_t along dimension 0, from h = 0, by doubling."""
    k = 1
    while k < a.shape[0]:
        b = torch.cat([b[:k], torch.addcmul(b[k:], a[k:], b[:-k])])
        a = torch.cat([a[:k], a[k:] * a[:-k]])
        k *= 2
    return b


def _scan_parts(s):
    D, N = s["A"].shape
    M = s["u"].numel() // D
    G = s["Bm"].shape[-2]
    u, raw = s["u"].reshape(M, D).float(), s["dt"].reshape(M, D).float() + s["bias"]
    spread = lambda x: x.reshape(M, G, N).float().repeat_interleave(D // G, 1)  # noqa: E731
    step = _softplus(raw)
    return u, raw, step, torch.exp(step[..., None] * s["A"]), spread(s["Bm"]), spread(s["Cm"])


def _states(s, a, inp):
    """States after and before every token: [M, D, N] each; with the bounds of the sequences."""
    M = a.shape[0]
    t, seq, bounds = _places(s, M, s["u"].shape[1])
    first = (t == bounds[seq])[:, None, None]
    start = s["h0"][seq]
    h = _recur(torch.where(first, 0.0, a), torch.where(first, torch.addcmul(inp, a, start), inp))
    before = torch.where(first, start, torch.cat([start[:1], h[:-1]]))
    return h, before, t, seq, bounds


def _scan(s):
    u, raw, step, a, Bm, Cm = _scan_parts(s)
    h, _, _, _, bounds = _states(s, a, (step * u)[..., None] * Bm)
    y = (h * Cm).sum(-1) + s["skip"] * u
    if s["z"] is not None:
        z = s["z"].reshape(y.shape).float()
        y = y * z * _sigmoid(z)
    some = (bounds[1:] > bounds[:-1])[:, None, None]
    return y.to(s["u"].dtype).reshape(s["u"].shape), torch.where(some, h[(bounds[1:] - 1).clamp(min=0)], s["h0"])


def _scan_bwd(s):
    low, shape = s["u"].dtype, s["u"].shape
    D, N = s["A"].shape
    G = s["Bm"].shape[-2]
    u, raw, step, a, Bm, Cm = _scan_parts(s)
    M = u.shape[0]
    h, before, t, seq, bounds = _states(s, a, (step * u)[..., None] * Bm)
    dy, dz = s["dy"].reshape(M, D).float(), None
    if s["z"] is not None:
        z = s["z"].reshape(M, D).float()
        g = _sigmoid(z)
        dz = (dy * ((h * Cm).sum(-1) + s["skip"] * u) * g * (1.0 + z * (1.0 - g))).to(low).reshape(shape)
        dy = dy * z * g
    last = (t == bounds[seq + 1] - 1)[:, None, None]
    inp = Cm * dy[..., None]
    inp = torch.where(last, inp + s["dh"][seq], inp)
    nxt = torch.where(last, 0.0, torch.cat([a[1:], a[:1]]))
    grad = _recur(nxt.flip(0), inp.flip(0)).flip(0)
    dec = grad * a * before  # gradient of the exponent
    dstep = (grad * Bm).sum(-1) * u + (dec * s["A"]).sum(-1)
    ddt = dstep * _sigmoid(raw)
    du = (grad * Bm).sum(-1) * step + s["skip"] * dy
    fold = lambda x: x.reshape(M, G, D // G, N).sum(2).to(low).reshape(s["Bm"].shape)  # noqa: E731
    dh0 = torch.where((bounds[1:] > bounds[:-1])[:, None, None], (a * grad)[bounds[:-1].clamp(max=M - 1)], s["dh"])
    return (du.to(low).reshape(shape), ddt.to(low).reshape(shape), (dec * step[..., None]).sum(0),
            fold(grad * (step * u)[..., None]), fold(h * dy[..., None]), (dy * u).sum(0), dz, ddt.sum(0), dh0)


def _scan_step(s):
    u, raw, step, a, Bm, Cm = _scan_parts(s)
    s["h0"].copy_(a * s["h0"] + (step * u)[..., None] * Bm)
    y = (s["h0"] * Cm).sum(-1) + s["skip"] * u
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z * _sigmoid(z)
    return y.to(s["u"].dtype), s["h0"]


_PLAIN = dict(norm=_norm, norm_bwd=_norm_bwd, linear=_linear, linear_bwd=_linear_bwd, conv=_conv, conv_bwd=_conv_bwd,
              conv_step=_conv_step, scan=_scan, scan_bwd=_scan_bwd, scan_step=_scan_step)


# ---------------------------------------------------------------- the definitions, 64 bits
def exact(case, seed):
    c, op = case, case["op"]
    s = prepare(case, seed)
    d = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    if op == "norm":
        var, mean = torch.var_mean(d["x"], dim=1, correction=0)
        rstd = torch.pow(var + 1e-5, -0.5)
        return torch.addcmul(d["b"], (d["x"] - mean.unsqueeze(1)) * rstd.unsqueeze(1), d["w"]), mean, rstd
    if op == "norm_bwd":
        N, xc = c["N"], d["x"] - d["mean"].unsqueeze(1)
        xh = xc * d["rstd"].unsqueeze(1)
        g = d["dy"] * d["w"]
        dx = (g * N - g.sum(1, keepdim=True) - xh * torch.linalg.vecdot(g, xh).unsqueeze(1)) * (d["rstd"] / N).unsqueeze(1)
        return dx, torch.einsum("mn,mn->n", d["dy"], xh), torch.einsum("mn->n", d["dy"])
    if op == "linear":
        pre = torch.einsum("mk,nk->mn", d["x"], d["W"])
        if d["b"] is not None:
            pre += d["b"]
        y = _exact_act(pre, c["act"])[0]
        if d["res"] is not None:
            y = y + d["res"]
        return (y, pre) if c["pre"] else y
    if op == "linear_bwd":
        ds = d["dy"] if d["pre"] is None else d["dy"] * _exact_act(d["pre"], c["act"])[1]
        return torch.einsum("mn,nk->mk", ds, d["W"]), torch.einsum("mn,mk->nk", ds, d["x"]), torch.einsum("mn->n", ds)
    if op == "conv_step":
        pre, W = d["b"] + d["x"] * d["w"][:, -1], c["W"]
        for j in range(W - 1):
            pre = pre + d["cache"][:, j] * d["w"][:, j]
        return torch.nn.functional.silu(pre), torch.cat([d["cache"][:, 1:], d["x"].unsqueeze(1)], 1)
    bounds = _exact_bounds(c, s)
    if op in ("conv", "conv_bwd"):
        return _exact_conv(c, d, bounds, op == "conv_bwd")
    return _exact_scan(c, d, bounds, op)


def _exact_act(x, kind):
    """The activation and its derivative."""
    F = torch.nn.functional
    if kind == "none":
        return x, torch.ones_like(x)
    if kind == "relu":
        return F.relu(x), torch.heaviside(x, torch.zeros((), dtype=x.dtype, device=x.device))
    if kind == "softplus":
        return torch.logaddexp(x, torch.zeros_like(x)), torch.special.expit(x)
    if kind == "silu":
        p = torch.special.expit(x)
        return x * p, p + x * p * (1 - p)
    cdf = torch.special.ndtr(x)
    return x * cdf, cdf + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)


def _exact_bounds(c, s):
    if c["op"] == "scan_step":
        return list(range(c["B"] + 1))
    return s["cu"].tolist() if s["cu"] is not None else [b * c["T"] for b in range(c["B"] + 1)]


def _exact_conv(c, d, bounds, back):
    """Sequence by sequence: the padded inputs, the sum over the taps, and its transpose."""
    W, C = c["W"], c["C"]
    x, w, b = d["x"].reshape(-1, C), d["w"], d["b"]
    ys, tails, dxs, dold = [], [], [], []
    dw, db = torch.zeros_like(w), torch.zeros_like(b)
    for n in range(len(bounds) - 1):
        lo, hi = bounds[n], bounds[n + 1]
        old = d["cache"][n] if d["cache"] is not None else x.new_zeros(W - 1, C)
        full = torch.cat([old, x[lo:hi]])
        pre = b + sum(full[j:j + hi - lo] * w[:, j] for j in range(W))
        ys.append(_exact_act(pre, "silu")[0])
        tails.append(full[full.shape[0] - (W - 1):])
        if back:
            ds = d["dy"].reshape(-1, C)[lo:hi] * _exact_act(pre, "silu")[1]
            dfull = torch.zeros_like(full)
            for j in range(W):
                dfull[j:j + hi - lo] += ds * w[:, j]
                dw[:, j] += (ds * full[j:j + hi - lo]).sum(0)
            db += ds.sum(0)
            if d["cache"] is not None:
                dfull[full.shape[0] - (W - 1):] += d["dcache"][n]
            dxs.append(dfull[W - 1:])
            dold.append(dfull[:W - 1])
    shape = d["x"].shape
    if back:
        return torch.cat(dxs).reshape(shape), dw, db, torch.stack(dold) if d["cache"] is not None else None
    return torch.cat(ys).reshape(shape), torch.stack(tails) if d["cache"] is not None else None


def _exact_scan(c, d, bounds, op):
    """Token by token over all sequences of the batch at once (a dense batch), or one after the other (packed)."""
    D, N, G = c["D"], c["N"], c["G"]
    packed = op != "scan_step" and d["cu"] is not None
    T = 1 if op == "scan_step" else c["T"]
    rows = 1 if packed else c["B"]
    if rows * T * D * N > 9e8 or T > 20000:
        return None
    x = {k: d[k].reshape(rows, T, D) for k in ("u", "dt", "z", "dy") if d.get(k) is not None}
    wide = {k: d[k].reshape(rows, T, G, 1, N).expand(rows, T, G, D // G, N).reshape(rows, T, D, N) if G > 1
            else d[k].reshape(rows, T, 1, N) for k in ("Bm", "Cm")}
    raw = x["dt"] + d["bias"]
    step = torch.logaddexp(raw, torch.zeros_like(raw))
    starts = {}
    for n in range(len(bounds) - 1):
        if packed and bounds[n + 1] > bounds[n]:
            starts[bounds[n]] = n
    h = d["h0"] if not packed else None
    final = d["h0"].clone()
    y = torch.empty_like(step)
    back = op == "scan_bwd"
    keep = torch.empty((rows, T, D, N), dtype=torch.float64, device="cuda") if back else None
    prev = None
    for t in range(T):
        if t in starts:
            if prev is not None:
                final[prev] = h[0]
            prev = starts[t]
            h = d["h0"][prev:prev + 1]
        if back:
            keep[:, t] = h
        h = torch.exp(step[:, t, :, None] * d["A"]) * h + (step[:, t] * x["u"][:, t]).unsqueeze(-1) * wide["Bm"][:, t]
        y[:, t] = (h * wide["Cm"][:, t]).sum(-1)
    if packed:
        final[prev] = h[0]
    else:
        final = h
    y = y + d["skip"] * x["u"]
    if not back:
        if "z" in x:
            y = y * _exact_act(x["z"], "silu")[0]
        shape = d["u"].shape
        return y.reshape(shape), final.reshape(d["h0"].shape)
    p, dz = x["dy"], None
    if "z" in x:
        f, df = _exact_act(x["z"], "silu")
        dz, p = (x["dy"] * y * df).reshape(d["u"].shape), x["dy"] * f
    ends = {bounds[n + 1] - 1: n for n in range(len(bounds) - 1) if bounds[n + 1] > bounds[n]} if packed else {}
    dh0 = d["dh"].clone()
    du, ddt = torch.empty_like(step), torch.empty_like(step)
    dA = torch.zeros_like(d["A"])
    dB, dC = (torch.empty((rows, T, G, N), dtype=torch.float64, device="cuda") for _ in range(2))
    carry = None if packed else d["dh"]
    for t in range(T - 1, -1, -1):
        if t in ends:
            carry = d["dh"][ends[t]:ends[t] + 1]
        a = torch.exp(step[:, t, :, None] * d["A"])
        before, bm, cm = keep[:, t], wide["Bm"][:, t], wide["Cm"][:, t]
        su = (step[:, t] * x["u"][:, t]).unsqueeze(-1)
        g = carry + p[:, t].unsqueeze(-1) * cm
        dC[:, t] = ((a * before + su * bm) * p[:, t].unsqueeze(-1)).reshape(rows, G, D // G, N).sum(2)
        dB[:, t] = (g * su).reshape(rows, G, D // G, N).sum(2)
        gb, ge = (g * bm).sum(-1), g * a * before
        du[:, t] = gb * step[:, t] + d["skip"] * p[:, t]
        ddt[:, t] = gb * x["u"][:, t] + (ge * d["A"]).sum(-1)
        dA += (ge * step[:, t].unsqueeze(-1)).sum(0)
        carry = a * g
        if t in starts:
            dh0[starts[t]] = carry[0]
    if not packed:
        dh0 = carry
    ddt = ddt * torch.special.expit(raw)
    shape = d["u"].shape
    return (du.reshape(shape), ddt.reshape(shape), dA, dB.reshape(d["Bm"].shape), dC.reshape(d["Bm"].shape),
            (p * x["u"]).sum((0, 1)), dz, ddt.sum((0, 1)), dh0.reshape(d["h0"].shape))
