"""The mixer's operators together, as a pre-norm selective block uses them: a packed prompt, its gradients, then single
tokens from the caches that the prompt left; the same on side streams and replayed from a graph; and tensors of more
than 2^31 elements.

Block: h = norm(x); [u, z] = h W_in^T; c = SiLU(conv(u)); [r, B, C] = c W_x^T; dt = r W_dt^T;
       y = scan(c, dt, B, C; gate z); out = x + y W_out^T."""
import pytest
import torch
import torch.nn.functional as F

import mixer_reference as ref
from mixer_reference import assert_close

pytestmark = pytest.mark.gpu
D_MODEL, INNER, RANK, N = 64, 96, 8, 16


def weights(seed, dtype=torch.bfloat16):
    gen = torch.Generator().manual_seed(seed)
    w = lambda *s: (torch.randn(s, generator=gen) * s[-1] ** -0.5).to(dtype)  # noqa: E731
    f = lambda *s, std=1.0, mean=0.0: mean + std * torch.randn(s, generator=gen)  # noqa: E731
    return dict(norm_w=f(D_MODEL, std=0.2, mean=1.0), norm_b=f(D_MODEL, std=0.1), W_in=w(2 * INNER, D_MODEL),
                conv_w=(0.4 * torch.randn((INNER, 4), generator=gen)).to(dtype), conv_b=f(INNER, std=0.1),
                W_x=w(RANK + 2 * N, INNER), W_dt=w(INNER, RANK), dt_b=f(INNER, std=0.5, mean=-2.0),
                A=-torch.arange(1, N + 1).float().repeat(INNER, 1) * torch.exp(f(INNER, N, std=0.1)), D=f(INNER, mean=1.0),
                W_out=w(D_MODEL, INNER))


def prompt(kda, x, W, cu):
    """Forward over packed tokens x [M, d]; returns out, the caches, and what the backward pass needs."""
    M = x.shape[0]
    h, mean, rstd = kda.layer_norm_fwd(x, W["norm_w"], W["norm_b"])
    uz = kda.linear_act(h, W["W_in"])
    u, z = uz[None, :, :INNER], uz[None, :, INNER:]
    c, cache = kda.short_conv_fwd(u, W["conv_w"], W["conv_b"], cu, output_conv_state=True)
    rbc = kda.linear_act(c[0], W["W_x"])
    Bm, Cm = (rbc[None, :, None, RANK + k * N:RANK + (k + 1) * N] for k in (0, 1))
    dt = kda.linear_act(rbc[:, :RANK], W["W_dt"])
    y, state = kda.selective_scan_fwd(c, dt[None], W["A"], Bm, Cm, W["D"], z, W["dt_b"], cu_seqlens=cu)
    out = kda.linear_act(y[0], W["W_out"], residual=x)
    return out, (cache, state), (h, mean, rstd, u, z, c, rbc, dt, Bm, Cm, y, M)


def token(kda, x, W, caches):
    """One token for every sequence, x [n, d]."""
    cache, state = caches
    h, _, _ = kda.layer_norm_fwd(x, W["norm_w"], W["norm_b"])
    uz = kda.linear_act(h, W["W_in"])
    c = kda.short_conv_step(uz[:, :INNER], W["conv_w"], cache, W["conv_b"])
    rbc = kda.linear_act(c, W["W_x"])
    dt = kda.linear_act(rbc[:, :RANK], W["W_dt"])
    y = kda.selective_scan_step(c, dt, W["A"], rbc[:, None, RANK:RANK + N], rbc[:, None, RANK + N:], state, W["D"],
                                uz[:, INNER:], W["dt_b"])
    return kda.linear_act(y, W["W_out"], residual=x)


def gradients(kda, dout, x, W, cu, kept):
    h, mean, rstd, u, z, c, rbc, dt, Bm, Cm, y, M = kept
    g = {}
    dy, g["W_out"], _ = kda.linear_act_bwd(dout, y[0], W["W_out"], bias_grad=False)
    dc, ddt, g["A"], dB, dC, g["D"], dz, g["dt_b"], _ = kda.selective_scan_bwd(
        dy[None], c, dt[None], W["A"], Bm, Cm, W["D"], z, W["dt_b"], cu_seqlens=cu)
    dr, g["W_dt"], _ = kda.linear_act_bwd(ddt[0], rbc[:, :RANK], W["W_dt"], bias_grad=False)
    drbc = torch.cat([dr, dB.reshape(M, N), dC.reshape(M, N)], 1)
    dc2, g["W_x"], _ = kda.linear_act_bwd(drbc, c[0], W["W_x"], bias_grad=False)
    du, g["conv_w"], g["conv_b"], _ = kda.short_conv_bwd(dc + dc2, u, W["conv_w"], W["conv_b"], cu)
    dh, g["W_in"], _ = kda.linear_act_bwd(torch.cat([du[0], dz[0]], 1), h, W["W_in"], bias_grad=False)
    dx, g["norm_w"], g["norm_b"] = kda.layer_norm_bwd(dh, x, W["norm_w"], mean, rstd)
    g["x"] = dx + dout
    return g


def block64(x, W, cu):
    """The block in float64, differentiable by torch."""
    h = F.layer_norm(x, (D_MODEL,), W["norm_w"], W["norm_b"], 1e-5)
    u, z = (h @ W["W_in"].T).split(INNER, 1)
    outs = []
    for lo, hi in zip(cu, cu[1:]):
        pad = torch.cat([x.new_zeros(3, INNER), u[lo:hi]])
        c = F.silu(sum(pad[j:j + hi - lo] * W["conv_w"][:, j] for j in range(4)) + W["conv_b"])
        r, Bm, Cm = (c @ W["W_x"].T).split([RANK, N, N], 1)
        step = F.softplus(r @ W["W_dt"].T + W["dt_b"])
        s, ys = x.new_zeros(INNER, N), []
        for t in range(hi - lo):
            s = torch.exp(step[t][:, None] * W["A"]) * s + (step[t] * c[t])[:, None] * Bm[t]
            ys.append((s * Cm[t]).sum(1))
        if hi > lo:
            y = (torch.stack(ys) + W["D"] * c) * F.silu(z[lo:hi])
            outs.append(x[lo:hi] + y @ W["W_out"].T)
    return torch.cat(outs)


CU = [0, 1, 1, 40, 43, 130]


def _case(seed):
    gen = torch.Generator().manual_seed(seed)
    x, dout = (torch.randn((CU[-1], D_MODEL), generator=gen).to(torch.bfloat16) for _ in range(2))
    W = weights(seed + 1)
    return x, dout, W


def test_prompt_gradients_and_tokens(kda):
    x, dout, W = _case(3)
    Wg = {k: v.cuda() for k, v in W.items()}
    cu = torch.tensor(CU, dtype=torch.int32, device="cuda")
    out, caches, kept = prompt(kda, x.cuda(), Wg, cu)
    x64 = x.double().requires_grad_()
    W64 = {k: v.double().requires_grad_() for k, v in W.items()}
    want = block64(x64, W64, CU)
    (want * dout.double()).sum().backward()
    # seven tensors are rounded to bf16 on the way (h, uz, c, rbc, dt, y, out): at most half a step each, 7 x 2^-8
    # of what they feed, if none damped it
    assert_close(out, want.detach(), torch.bfloat16, 7 * 2.0 ** -8, "out")
    # and in the backward pass as many again (two of them to both operands' products)
    for name, g in gradients(kda, dout.cuda(), x.cuda(), Wg, cu, kept).items():
        w = x64.grad if name == "x" else W64[name].grad
        err = float((g.double().cpu() - w).norm() / w.norm())
        assert err <= 16 * 2.0 ** -8, (name, err)
    # three more tokens for each sequence, one at a time, against the whole sequences in one prompt
    gen = torch.Generator().manual_seed(9)
    more = torch.randn((3, len(CU) - 1, D_MODEL), generator=gen).to(torch.bfloat16)
    rows, cu2 = [], [0]
    for n, (lo, hi) in enumerate(zip(CU, CU[1:])):
        rows.append(torch.cat([x[lo:hi], more[:, n]]))
        cu2.append(cu2[-1] + hi - lo + 3)
    whole = block64(torch.cat(rows).double(), {k: v.double() for k, v in W.items()}, cu2)
    for t in range(3):
        got = token(kda, more[t].cuda(), Wg, caches)
        want = torch.stack([whole[cu2[n + 1] - 3 + t] for n in range(len(CU) - 1)])
        assert_close(got, want, torch.bfloat16, 7 * 2.0 ** -8, f"token {t}")
    assert kda.device_status() == 0


def test_side_streams_and_graph_replay_give_the_same_bits(kda):
    x, dout, W = _case(5)
    Wg, xg, dg = {k: v.cuda() for k, v in W.items()}, x.cuda(), dout.cuda()
    cu = torch.tensor(CU, dtype=torch.int32, device="cuda")

    def step():
        out, caches, kept = prompt(kda, xg, Wg, cu)
        g = gradients(kda, dg, xg, Wg, cu, kept)
        return [out, *caches, *g.values()]
    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(3):  # both streams busy at once
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(step())
    torch.cuda.synchronize()
    for got in outs:
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    # two graphs captured on their own streams and replayed in turn and at once
    graphs, held = [], []
    for s in streams:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            held.append(step())
        graphs.append(g)
    for t in [t for h in held for t in h]:
        t.zero_()
    torch.cuda.synchronize()
    for _ in range(2):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for got in held:
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    # a replay reads what is in its inputs then
    xg.copy_(x.flip(0))
    with torch.cuda.stream(streams[0]):
        graphs[0].replay()
    torch.cuda.synchronize()
    again = step()
    assert all(torch.equal(a, b) for a, b in zip(held[0], again)) and not torch.equal(again[0], want[0])


def test_bindings_refuse_what_does_not_fit(kda):
    c = lambda *s, t=torch.float32: torch.zeros(s, device="cuda", dtype=t)  # noqa: E731
    b16 = torch.bfloat16
    bad = [
        lambda: kda.layer_norm_fwd(c(4, 8), c(9)), lambda: kda.layer_norm_fwd(c(4, 8, t=torch.float16)),
        lambda: kda.layer_norm_fwd(c(4, 8).t()), lambda: kda.layer_norm_bwd(c(4, 8), c(4, 8), None, c(3), c(4)),
        lambda: kda.linear_act(c(4, 8), c(4, 8)), lambda: kda.linear_act(c(4, 8, t=b16), c(4, 16, t=b16)),
        lambda: kda.linear_act(c(4, 8, t=b16), c(4, 8, t=b16), act="tanh"),
        lambda: kda.linear_act(c(4, 12, t=b16), c(4, 12, t=b16)),  # rows not on 16-byte boundaries
        lambda: kda.linear_act_bwd(c(4, 8, t=b16), c(4, 16, t=b16), c(8, 16, t=b16), act="silu"),
        lambda: kda.short_conv_fwd(c(2, 4, 8), c(8, 5)), lambda: kda.short_conv_fwd(c(2, 4, 8), c(9, 4)),
        lambda: kda.short_conv_fwd(c(2, 4, 8), c(8, 4), cu_seqlens=torch.tensor([0, 4], dtype=torch.int32, device="cuda")),
        lambda: kda.short_conv_fwd(c(1, 4, 8), c(8, 4), cu_seqlens=torch.tensor([0, 4], device="cuda")),
        lambda: kda.short_conv_step(c(2, 8), c(8, 4), c(2, 2, 8)),
        lambda: kda.selective_scan_fwd(c(1, 4, 8), c(1, 4, 8), c(8, 33), c(1, 4, 1, 33), c(1, 4, 1, 33)),
        lambda: kda.selective_scan_fwd(c(1, 4, 8), c(1, 4, 8), c(8, 4), c(1, 4, 3, 4), c(1, 4, 3, 4)),
        lambda: kda.selective_scan_fwd(c(1, 4, 8), c(1, 4, 8), c(8, 4), c(1, 4, 1, 4), c(1, 4, 1, 4), z=c(1, 4, 9)),
        lambda: kda.selective_scan_step(c(2, 8), c(2, 8), c(8, 4), c(2, 1, 4), c(2, 1, 4), c(2, 8, 5)),
        lambda: kda.selective_scan_fwd(c(1, 4, 8), c(1, 4, 8), c(8, 4), c(1, 4, 1, 4), c(1, 4, 1, 4, t=b16)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError, kda.KDAError)):
            f()
            raise AssertionError(i)


@pytest.mark.slow
def test_more_than_2_31_elements(kda):
    """Row offsets past 32 bits: the last rows of norm and convolution, and sampled channels of the scan."""
    M, C = (1 << 31) // 4096 + 300, 4096
    x = torch.empty((1, M, C), device="cuda", dtype=torch.bfloat16)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x[0, -70:] = torch.randn((70, C), generator=gen, device="cuda").to(torch.bfloat16)
    x[0, :-70] = 0.5
    y, mean, rstd = kda.layer_norm_fwd(x[0])
    want = ref.norm_fwd(x[0, -64:].double().cpu(), None, None, 1e-5)
    assert_close(y[-64:], want[0], torch.bfloat16, 2.0 ** -18)
    w = (0.4 * torch.randn((C, 4), generator=gen, device="cuda")).to(torch.bfloat16)
    del y
    y, _ = kda.short_conv_fwd(x, w)
    want = ref.conv(x[:, -70:].double().cpu(), w.double().cpu(), None, None, None, True)[0]
    assert_close(y[:, -64:], want[:, -64:], torch.bfloat16, 2.0 ** -18)
    del x, y
    torch.cuda.empty_cache()
    T, ch = (1 << 31) // 65536 + 40, 65536
    u = torch.randn((1, T, ch), generator=gen, device="cuda", dtype=torch.bfloat16)
    dt = 0.5 * torch.randn((1, T, ch), generator=gen, device="cuda", dtype=torch.bfloat16)
    A = -torch.rand((ch, 4), generator=gen, device="cuda") - 0.5
    Bm, Cm = (torch.randn((1, T, 1, 4), generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    y, fin = kda.selective_scan_fwd(u, dt, A, Bm, Cm)
    pick = torch.tensor([0, 31, 40000, 65535], device="cuda")
    d = lambda t: t.double().cpu()  # noqa: E731
    # the last 3000 tokens: every decay is below exp(-0.3 x 0.5), so what came before is below exp(-450)
    sub = lambda t: d(t[:, -3000:, pick])  # noqa: E731
    small = dt[:, -3000:, pick].float().amin().item()
    assert torch.nn.functional.softplus(torch.tensor(small)) > 0.05
    yr, finr = ref.scan(sub(u), sub(dt), d(A[pick]), d(Bm[:, -3000:]), d(Cm[:, -3000:]))
    assert_close(y[:, -200:, pick], yr[:, -200:], torch.bfloat16, (3000 ** 0.5 + 16) * 2.0 ** -20)
    assert_close(fin[:, pick], finr, torch.float32, (3000 ** 0.5 + 16) * 2.0 ** -20)


@pytest.mark.slow
def test_almost_2_31_tokens(kda):
    """One channel, as many tokens as the convolution takes: the last run ends next to 2^31."""
    T = 0x7fffff00
    x = torch.full((1, T, 1), 0.5, device="cuda", dtype=torch.bfloat16)
    gen = torch.Generator(device="cuda").manual_seed(2)
    x[0, -70:] = torch.randn((70, 1), generator=gen, device="cuda").to(torch.bfloat16)
    w = (0.4 * torch.randn((1, 4), generator=gen, device="cuda")).to(torch.bfloat16)
    y = torch.full_like(x, float("nan"))
    kda.short_conv_fwd(x, w, out=y)
    want = ref.conv(x[:, -70:].double().cpu(), w.double().cpu(), None, None, None, True)[0]
    assert_close(y[:, -60:], want[:, 10:], torch.bfloat16, 2.0 ** -18)
    # 2^20 equal tokens before them: the window's sum is the same for each
    assert torch.equal(y[0, -(1 << 20):-70], y[0, 10:11].expand((1 << 20) - 70, 1))
