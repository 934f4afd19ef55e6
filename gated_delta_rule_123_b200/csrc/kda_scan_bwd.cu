// Selective state-space scan, backward (the notation of kda_scan.cu).
//
// With p_t = dy_t SiLU(z_t) and the gradient of the state
//   g_t = C_t p_t + a_{t+1} g_{t+1}            (after the last token: the final state's)
// and e_t = g_t a_t h_{t-1}, the gradient of the exponent D_t A:
//   dC_t = sum_d p_t h_t         dB_t = sum_d g_t D_t u_t       (over the group's channels)
//   du_t = D_t sum_n g_t B_t + Dskip p_t       dD_t = u_t sum_n g_t B_t + sum_n e_t A
//   dA = sum_t e_t D_t           ddt_t = dD_t sigmoid(dt_t + bias)   dbias = sum_t ddt_t
//   dDskip = sum_t p_t u_t       dz_t = dy_t (sum_n C_t h_t + Dskip u_t) SiLU'(z_t)     dh_0 = a_1 g_1
//
// States are needed in reverse order and are too many to keep, so a first pass
// writes the state before every few tokens, counted from a zero state at its
// segment's start, with the sum of D up to there: the decay from the segment's start
// to that token is exp(A sum(D)), so a checkpoint is completed by adding that times
// the segment's incoming state.  The same pass accumulates the reverse map of the
// segment, G = sum_t (a_1 .. a_t) C_t p_t: the gradient of the incoming state is G +
// exp(A sum(D)) times the gradient of the state at its end.  So both directions of
// the recurrence cross segments by a few operations per state, and the second pass
// runs every segment on its own: per run of KC tokens it computes the decays and
// states forward from the checkpoint into registers, then walks back.
//
// Layout as in the forward pass, a lane per channel, so every sum over the states and
// every sum over the tokens (dA, dDskip, dbias) stays in a lane.  The sums over the
// channels for dB and dC are the only exchange; they go through shared memory, then
// over the blocks in a fixed order: every result is the same on every run.  Bound by
// the latency of 8 warps an SM: the registers hold KC tokens' decays and states.
// Measured at 2 x 2047 tokens, 2048 channels, 16 states: 98 us the first pass, 285 us
// the second (a quad of lanes to a channel: 164 and 633 us).
#include "kda_scan.cuh"

namespace kda {
namespace scan {

__device__ __forceinline__ float dsilu(float z) {
    const float g = sigmoidf(z);
    return g * (1.f + z * (1.f - g));
}

// The flags of a tile's token: the sequence that starts at it and the one that ends with it.
__device__ __forceinline__ void edge_flags(const SArgs& a, long long t, bool here, int& first, int& last) {
    first = last = -1;
    if (here) {
        const int m = seq_of(a.cu, a.nseq, a.seq_len, int(t));
        const int end = seq_begin(a.cu, a.seq_len, m + 1, a.ntok);
        if (seq_begin(a.cu, a.seq_len, m, a.ntok) == t && end > t) first = m;  // (not an empty one before rows left out)
        if (end == t + 1) last = m;
    }
}

// Tokens between two checkpoints of a channel padded to NP states: as many as the
// second pass can hold in registers (decays and states of every token).
__host__ __device__ constexpr int ckpt_tokens(int NP) { return NP <= 8 ? 8 : 4; }

template <typename T, int NP>
struct MapSmem {
    T u[2][kFT][kCh], dt[2][kFT][kCh], z[2][kFT][kCh], dy[2][kFT][kCh];
    T b[2][kFT][NP], c[2][kFT][NP];
    float bc[kFT][2 * NP];
    int first[kFT], last[kFT];
};

// The first pass, in the forward pass's layout (a lane holds a channel): states before
// every KC tokens from a zero state, the sums of D up to there, the segment's end state
// and its reverse map.
template <typename T, int NP, int kCopy>
__global__ void __launch_bounds__(32) bwd_map_kernel(const SArgs a, bool bc_vec) {
    constexpr int kP = NP / 2, KC = ckpt_tokens(NP);
    __shared__ __align__(128) MapSmem<T, NP> sm;
    const int lane = threadIdx.x;
    const Place p = place(a);
    if (p.t0 >= p.t1) return;
    const int d = p.d0 + lane, valid = p.dend - p.d0;
    const bool live = lane < valid;
    f2 A2[kP], h[kP], P[kP], G[kP];
#pragma unroll
    for (int i = 0; i < kP; ++i) {
        A2[i] = h[i] = G[i] = 0ull;
        P[i] = dup2(1.f);
    }
    if (live) {
        load_pairs<NP>(A2, a.A + (size_t)d * a.N, a.N);
#pragma unroll
        for (int i = 0; i < kP; ++i) A2[i] = mul2(A2[i], dup2(kL2e));
    }
    const float bias = a.bias && live ? a.bias[d] : 0.f;
    const size_t at = (size_t)d * a.N, row = (size_t)a.D * a.N;
    bool open = true;  // no sequence has ended in the segment yet: later tokens do not see the incoming state
    float dsum = 0.f;
    int n = seq_of(a.cu, a.nseq, a.seq_len, int(p.t0));
    long long s_beg = seq_begin(a.cu, a.seq_len, n, a.ntok), s_end = seq_begin(a.cu, a.seq_len, n + 1, a.ntok);
    auto request = [&](long long tt, int w) {
        const int m = int(p.t1 - tt < kFT ? p.t1 - tt : kFT);
        stage_tile<T, kCopy>(sm.u[w], a.u, tt, m, a.ldu, p.d0, valid, lane);
        stage_tile<T, kCopy>(sm.dt[w], a.dt, tt, m, a.lddt, p.d0, valid, lane);
        stage_tile<T, kCopy>(sm.dy[w], a.dy, tt, m, a.lddy, p.d0, valid, lane);
        if (a.z) stage_tile<T, kCopy>(sm.z[w], a.z, tt, m, a.ldz, p.d0, valid, lane);
        stage_bc<T, NP>(sm.b[w], a.Bm, tt, m, a.ldb, (long long)p.g * a.N, a.N, bc_vec, lane);
        stage_bc<T, NP>(sm.c[w], a.Cm, tt, m, a.ldc, (long long)p.g * a.N, a.N, bc_vec, lane);
        cp_async_commit();
    };
    request(p.t0, 0);
    const long long chunk0 = ((long long)p.b * a.S + p.s) * (a.L / KC);
    int buf = 0;
    for (long long tt = p.t0; tt < p.t1; tt += kFT, buf ^= 1) {
        const int steps = int(p.t1 - tt < kFT ? p.t1 - tt : kFT);
        const bool edges = !(s_beg < tt && s_end > tt + kFT);
        if (edges && lane < kFT) edge_flags(a, tt + lane, lane < steps, sm.first[lane], sm.last[lane]);
        cp_async_wait0();
        __syncwarp();
        widen_rows<T, NP>(sm.bc, 0, sm.b[buf], lane);
        widen_rows<T, NP>(sm.bc, NP, sm.c[buf], lane);
        __syncwarp();
        if (tt + kFT < p.t1) request(tt + kFT, buf ^ 1);
        auto keep = [&](int k) {  // the checkpoint before token k
            const long long ck = chunk0 + (tt - p.t0 + k) / KC;
            if (live) {
                store_pairs<NP>(h, a.ckpt + (ck * a.D + d) * NP, NP);
                a.ckpt_d[ck * a.D + d] = dsum;
            }
        };
        auto token = [&](int k, auto reverse) {
            constexpr bool kOpen = decltype(reverse)::value;
            float D = to_f32<T>(sm.dt[buf][k][lane]) + bias;
            if (a.softplus) D = softplus_poly(D);
            float pv = to_f32<T>(sm.dy[buf][k][lane]);
            if (a.z) pv *= siluf(to_f32<T>(sm.z[buf][k][lane]));
            const f2 D2 = dup2(D), w2 = dup2(D * to_f32<T>(sm.u[buf][k][lane])), p2 = dup2(pv);
#pragma unroll
            for (int i = 0; i < kP; i += 2) {
                const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(&sm.bc[k][2 * i]);
                const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(&sm.bc[k][NP + 2 * i]);
                float x0, x1, x2, x3;
                upk(mul2(D2, A2[i]), x0, x1);
                upk(mul2(D2, A2[i + 1]), x2, x3);
                const f2 e0 = pk(ex2(x0), ex2(x1)), e1 = pk(ex2(x2), ex2(x3));
                h[i] = fma2(e0, h[i], mul2(w2, b.x));
                h[i + 1] = fma2(e1, h[i + 1], mul2(w2, b.y));
                if constexpr (kOpen) {
                    P[i] = mul2(P[i], e0);
                    P[i + 1] = mul2(P[i + 1], e1);
                    G[i] = fma2(P[i], mul2(c.x, p2), G[i]);
                    G[i + 1] = fma2(P[i + 1], mul2(c.y, p2), G[i + 1]);
                }
            }
            dsum += D;
        };
        auto run = [&](auto reverse) {
            int k = 0;
#pragma unroll 1
            for (; k + 4 <= steps; k += 4) {
                if (k % KC == 0) keep(k);
#pragma unroll
                for (int j = 0; j < 4; ++j) token(k + j, reverse);
            }
            if (k < steps && k % KC == 0) keep(k);
#pragma unroll 1
            for (; k < steps; ++k) token(k, reverse);
        };
        if (!edges) {
            if (open) run(std::true_type{});
            else run(std::false_type{});
        } else {
#pragma unroll 1
            for (int k = 0; k < steps; ++k) {
                if (k % KC == 0) keep(k);
                if (sm.first[k] >= 0) {
#pragma unroll
                    for (int i = 0; i < kP; ++i) h[i] = 0ull;
                    if (a.h0 && live) load_pairs<NP>(h, a.h0 + sm.first[k] * row + at, a.N);
                }
                if (open) token(k, std::true_type{});
                else token(k, std::false_type{});
                if (sm.last[k] >= 0) {
                    if (open && a.dhT && live) {
                        f2 e[kP];
                        load_pairs<NP>(e, a.dhT + sm.last[k] * row + at, a.N);
#pragma unroll
                        for (int i = 0; i < kP; ++i) G[i] = fma2(P[i], e[i], G[i]);
                    }
                    open = false;
                }
            }
        }
        if (s_end <= tt + kFT && tt + kFT < p.t1) {
            n = seq_of(a.cu, a.nseq, a.seq_len, int(tt + kFT));
            s_beg = seq_begin(a.cu, a.seq_len, n, a.ntok);
            s_end = seq_begin(a.cu, a.seq_len, n + 1, a.ntok);
        }
        __syncwarp();
    }
    if (live) {
        const long long i = (long long)p.b * a.S + p.s;
        store_pairs<NP>(h, a.seg_h + i * row + at, a.N);
        store_pairs<NP>(G, a.seg_g + i * row + at, a.N);
        a.seg_d[i * a.D + d] = dsum;
    }
}

// One value of 2 NP per lane and column, summed over the warp's lanes (channels): the
// lanes write their rows to shared memory, a lane adds 4 columns of a part of the rows
// and the parts are added by a halving exchange, which leaves 4 / halvings values with
// a lane.  Rows of 2 NP + 4 floats: no bank twice, writing or reading.
template <int NP>
struct ChannelSum {
    static constexpr int kCols = 2 * NP, kPitch = kCols + 4, kCG = kCols / 4, kRG = 32 / kCG;  // column and row groups
    static constexpr int kLeft = kRG >= 4 ? 1 : 2;
    float s[2][32][kPitch];
};
template <int NP>
__device__ __forceinline__ void channel_sum_write(ChannelSum<NP>& cs, int buf, int lane, int col, f2 v0, f2 v1) {
    ulonglong2 v;
    v.x = v0;
    v.y = v1;
    *reinterpret_cast<ulonglong2*>(&cs.s[buf][lane][col]) = v;
}
// To be called after a __syncwarp; writes the sums to out[0 .. 2N) (dB, then dC).
template <int NP>
__device__ __forceinline__ void channel_sum_read(const ChannelSum<NP>& cs, int buf, int lane, float* out, int N) {
    using C = ChannelSum<NP>;
    const int cg = lane % C::kCG, rg = lane / C::kCG;
    f2 a = 0ull, b = 0ull;
#pragma unroll
    for (int r = 0; r < 32 / C::kRG; ++r) {
        const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(&cs.s[buf][rg * (32 / C::kRG) + r][cg * 4]);
        a = add2(a, v.x);
        b = add2(b, v.y);
    }
    float v[4];
    upk(a, v[0], v[1]);
    upk(b, v[2], v[3]);
    int col = cg * 4;
    {
        const bool up = lane & 16;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float keep = up ? v[2 + i] : v[i], give = up ? v[i] : v[2 + i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, 16);
        }
        col += up ? 2 : 0;
    }
    if constexpr (C::kRG >= 4) {
        const bool up = lane & 8;
        const float keep = up ? v[1] : v[0], give = up ? v[0] : v[1];
        v[0] = keep + __shfl_xor_sync(0xffffffffu, give, 8);
        col += up ? 1 : 0;
    }
    if constexpr (C::kRG >= 8) v[0] += __shfl_xor_sync(0xffffffffu, v[0], 4);
#pragma unroll
    for (int i = 0; i < C::kLeft; ++i) {
        const int c = col + i, n = c % NP;
        if (n < N && (C::kRG < 8 || !(lane & 4))) out[(c / NP) * N + n] = v[i];
    }
}

constexpr int kMT = 8;  // tokens of a tile in the second pass: its shared memory lets the registers bound the warps of an SM

template <typename T, int NP>
struct MainSmem {
    static constexpr int kChunks = kMT / ckpt_tokens(NP);
    T u[2][kMT][kCh], dt[2][kMT][kCh], z[2][kMT][kCh], dy[2][kMT][kCh];
    T b[2][kMT][NP], c[2][kMT][NP];
    float ck[2][kChunks][32 * NP];  // the tile's checkpoints, a lane's 16-byte vectors swizzled
    float ckd[2][kChunks][32];
    float bc[kMT][2 * NP];
    float hin[32 * NP];  // the state that enters the segment, swizzled alike
    ChannelSum<NP> sum;
    int first[kMT], last[kMT];
};
// Place of vector i (4 states) of a lane's NP states: eight neighbouring lanes touch no bank twice.
template <int NP>
__device__ __forceinline__ int swz(int lane, int i) {
    constexpr int kV = NP / 4;  // vectors of a lane: 2 or 4
    return (lane * kV + (i ^ ((lane / (8 / kV)) & (kV - 1)))) * 4;
}

// The second pass for up to 16 states: a lane holds a channel.
template <typename T, int NP, int kCopy>
__global__ void __launch_bounds__(32) bwd_kernel(const SArgs a, bool bc_vec) {
    constexpr int kP = NP / 2, KC = ckpt_tokens(NP), kV = NP / 4;
    using Smem = MainSmem<T, NP>;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
    const int lane = threadIdx.x;
    const Place p = place(a);
    const int d = p.d0 + lane, valid = p.dend - p.d0;
    const bool live = lane < valid;
    const long long si = (long long)p.b * a.S + p.s;
    const size_t at = (size_t)d * a.N, row = (size_t)a.D * a.N;
    f2 A2[kP], g[kP], dA[kP];
#pragma unroll
    for (int i = 0; i < kP; ++i) A2[i] = g[i] = dA[i] = 0ull;
    if (live) {
        load_pairs<NP>(A2, a.A + (size_t)d * a.N, a.N);
#pragma unroll
        for (int i = 0; i < kP; ++i) A2[i] = mul2(A2[i], dup2(kL2e));
    }
    const float bias = a.bias && live ? a.bias[d] : 0.f, skip = a.skip && live ? a.skip[d] : 0.f;
    if (a.dh0)  // empty sequences hand the final state's gradient on
        for (int n = blockIdx.y; n < a.nseq; n += gridDim.y)
            if (live && seq_begin(a.cu, a.seq_len, n, a.ntok) == seq_begin(a.cu, a.seq_len, n + 1, a.ntok)) {
                f2 e[kP];
#pragma unroll
                for (int i = 0; i < kP; ++i) e[i] = 0ull;
                if (a.dhT) load_pairs<NP>(e, a.dhT + n * row + at, a.N);
                store_pairs<NP>(e, a.dh0 + n * row + at, a.N);
            }
    if (p.t0 >= p.t1) return;
    // the state that enters the segment, and the gradient that enters at its end
    const int nf = seq_of(a.cu, a.nseq, a.seq_len, int(p.t0));
    const long long f_beg = seq_begin(a.cu, a.seq_len, nf, a.ntok), f_end = seq_begin(a.cu, a.seq_len, nf + 1, a.ntok);
    {
        f2 h[kP];
#pragma unroll
        for (int i = 0; i < kP; ++i) h[i] = 0ull;
        const long long base = (long long)p.b * a.S;
        if (live && f_beg < p.t0) {
            chain_states<NP>(h, a, base + (f_beg - p.row0) / a.L, base + p.s, d, A2);
        }
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            ulonglong2 v;
            v.x = h[2 * i];
            v.y = h[2 * i + 1];
            *reinterpret_cast<ulonglong2*>(&sm.hin[swz<NP>(lane, i)]) = v;
        }
        const int nl = seq_of(a.cu, a.nseq, a.seq_len, int(p.t1 - 1));
        const long long l_end = seq_begin(a.cu, a.seq_len, nl + 1, a.ntok);
        if (live && l_end > p.t1) {
#pragma unroll
            for (int k = 0; k < kP; ++k) h[k] = dup2(1.f);  // the decay from t1 to the segment looked at
            // segments up to the one that holds the sequence's end, the next map on its way
            const int last = int((l_end - 1 - p.row0) / a.L);
            f2 next[kP];
            float nsd = 0.f;
            auto request = [&](int i) {
                load_pairs<NP>(next, a.seg_g + (base + i) * row + at, a.N);
                nsd = a.seg_d[(base + i) * a.D + d];
            };
            request(p.s + 1);
            for (int i = p.s + 1; i <= last; ++i) {
                f2 e[kP];
#pragma unroll
                for (int k = 0; k < kP; ++k) e[k] = next[k];
                const f2 sd = dup2(nsd);
                if (i < last) request(i + 1);
#pragma unroll
                for (int k = 0; k < kP; ++k) {
                    g[k] = fma2(h[k], e[k], g[k]);
                    h[k] = mul2(h[k], decay(A2[k], sd));
                }
            }
        }
    }
    if (!live)  // lanes without a channel take part in the sums over channels: their inputs are 0
        for (int w = 0; w < 2; ++w) {
            for (int k = 0; k < kMT; ++k)
                sm.u[w][k][lane] = sm.dt[w][k][lane] = sm.z[w][k][lane] = sm.dy[w][k][lane] = from_f32<T>(0.f);
            for (int j = 0; j < Smem::kChunks; ++j) {
                sm.ckd[w][j][lane] = 0.f;
                for (int i = 0; i < NP; ++i) sm.ck[w][j][lane * NP + i] = 0.f;
            }
        }
    const long long chunk0 = si * (a.L / KC);
    auto request = [&](long long tt, int w) {
        const int m = int(p.t1 - tt < kMT ? p.t1 - tt : kMT);
        stage_tile<T, kCopy>(sm.u[w], a.u, tt, m, a.ldu, p.d0, valid, lane);
        stage_tile<T, kCopy>(sm.dt[w], a.dt, tt, m, a.lddt, p.d0, valid, lane);
        stage_tile<T, kCopy>(sm.dy[w], a.dy, tt, m, a.lddy, p.d0, valid, lane);
        if (a.z) stage_tile<T, kCopy>(sm.z[w], a.z, tt, m, a.ldz, p.d0, valid, lane);
        stage_bc<T, NP>(sm.b[w], a.Bm, tt, m, a.ldb, (long long)p.g * a.N, a.N, bc_vec, lane);
        stage_bc<T, NP>(sm.c[w], a.Cm, tt, m, a.ldc, (long long)p.g * a.N, a.N, bc_vec, lane);
        if (live)
#pragma unroll
            for (int j = 0; j < Smem::kChunks; ++j)
                if (j * KC < m) {
                    const long long ck = (chunk0 + (tt - p.t0) / KC + j) * a.D + d;
#pragma unroll
                    for (int i = 0; i < kV; ++i) cp_async<16>(&sm.ck[w][j][swz<NP>(lane, i)], a.ckpt + ck * NP + 4 * i);
                    cp_async<4>(&sm.ckd[w][j][lane], a.ckpt_d + ck);
                }
        cp_async_commit();
    };
    float aD = 0.f, ab = 0.f;  // dDskip, dbias of the channel
    const int tiles = int((p.t1 - p.t0 + kMT - 1) / kMT);
    request(p.t0 + (long long)(tiles - 1) * kMT, 0);
    int buf = 0;
    float* const part = a.part_bc + ((((long long)(blockIdx.x % a.bpg) * a.rows * a.row_len) * a.G + p.g) * 2) * a.N;
    for (int ti = tiles - 1; ti >= 0; --ti, buf ^= 1) {
        const long long tt = p.t0 + (long long)ti * kMT;
        const int steps = int(p.t1 - tt < kMT ? p.t1 - tt : kMT);
        int ef = -1, el = -1;
        if (lane < kMT) {
            edge_flags(a, tt + lane, lane < steps, ef, el);
            sm.first[lane] = ef;
            sm.last[lane] = el;
        }
        const bool edges = __any_sync(0xffffffffu, ef >= 0 || el >= 0);
        cp_async_wait0();
        __syncwarp();
        widen_rows<T, NP>(sm.bc, 0, sm.b[buf], lane);
        widen_rows<T, NP>(sm.bc, NP, sm.c[buf], lane);
        if (steps < kMT) {  // tokens past the end: B = C = 0
            __syncwarp();
            for (int i = steps * 2 * NP + lane; i < kMT * 2 * NP; i += 32) (&sm.bc[0][0])[i] = 0.f;
        }
        __syncwarp();
        if (ti > 0) request(tt - kMT, buf ^ 1);
        auto walk = [&](auto has_edges) {
            constexpr bool kEdges = decltype(has_edges)::value;
#pragma unroll 1
            for (int k0 = (steps - 1) / KC * KC; k0 >= 0; k0 -= KC) {
                f2 h[kP], av[KC][kP], hp[KC][kP];
                float Dv[KC], uv[KC], pv[KC], ys[KC];
                // forward from the checkpoint
                {
                    const int j = k0 / KC;
#pragma unroll
                    for (int i = 0; i < kV; ++i) {
                        const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(&sm.ck[buf][j][swz<NP>(lane, i)]);
                        h[2 * i] = v.x;
                        h[2 * i + 1] = v.y;
                    }
                    if (f_beg < p.t0 && tt + k0 < f_end) {  // it counts from zero: add the incoming state's part
                        const f2 sd = dup2(sm.ckd[buf][j][lane]);
#pragma unroll
                        for (int i = 0; i < kV; ++i) {
                            const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(&sm.hin[swz<NP>(lane, i)]);
                            h[2 * i] = fma2(decay(A2[2 * i], sd), v.x, h[2 * i]);
                            h[2 * i + 1] = fma2(decay(A2[2 * i + 1], sd), v.y, h[2 * i + 1]);
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < KC; ++j) {
                    const int k = k0 + j;
                    const bool in = k < steps;  // tokens past the end: D = 0, p = 0
                    if (kEdges && sm.first[k] >= 0) {
#pragma unroll
                        for (int i = 0; i < kP; ++i) h[i] = 0ull;
                        if (a.h0 && live) load_pairs<NP>(h, a.h0 + sm.first[k] * row + at, a.N);
                    }
                    float D = to_f32<T>(sm.dt[buf][k][lane]) + bias;
                    if (a.softplus) D = softplus_poly(D);
                    Dv[j] = in ? D : 0.f;
                    uv[j] = in ? to_f32<T>(sm.u[buf][k][lane]) : 0.f;
                    pv[j] = in ? to_f32<T>(sm.dy[buf][k][lane]) : 0.f;
                    if (a.z && in) pv[j] *= siluf(to_f32<T>(sm.z[buf][k][lane]));
                    const f2 D2 = dup2(Dv[j]), w2 = dup2(Dv[j] * uv[j]);
                    f2 s = 0ull;
#pragma unroll
                    for (int i = 0; i < kP; i += 2) {
                        const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(&sm.bc[k][2 * i]);
                        const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(&sm.bc[k][NP + 2 * i]);
#pragma unroll
                        for (int v = 0; v < 2; ++v) {
                            av[j][i + v] = decay(A2[i + v], D2);
                            hp[j][i + v] = h[i + v];
                            h[i + v] = fma2(av[j][i + v], h[i + v], mul2(w2, v ? b.y : b.x));
                            s = fma2(h[i + v], v ? c.y : c.x, s);
                        }
                    }
                    ys[j] = lo2(s) + hi2(s);
                }
                // and back
#pragma unroll
                for (int j = KC - 1; j >= 0; --j) {
                    const int k = k0 + j;
                    if (k >= steps) continue;
                    if (kEdges && sm.last[k] >= 0) {
#pragma unroll
                        for (int i = 0; i < kP; ++i) g[i] = 0ull;
                        if (a.dhT && live) load_pairs<NP>(g, a.dhT + sm.last[k] * row + at, a.N);
                    }
                    const f2 D2 = dup2(Dv[j]), w2 = dup2(Dv[j] * uv[j]), p2 = dup2(pv[j]);
                    f2 sgb = 0ull, sea = 0ull;
#pragma unroll
                    for (int i = 0; i < kP; i += 2) {
                        const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(&sm.bc[k][2 * i]);
                        const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(&sm.bc[k][NP + 2 * i]);
                        f2 db[2], dc[2];
#pragma unroll
                        for (int v = 0; v < 2; ++v) {
                            const f2 bv = v ? b.y : b.x;
                            g[i + v] = fma2(v ? c.y : c.x, p2, g[i + v]);
                            const f2 ah = mul2(av[j][i + v], hp[j][i + v]);
                            const f2 e = mul2(g[i + v], ah);
                            db[v] = mul2(g[i + v], w2);
                            dc[v] = mul2(p2, fma2(w2, bv, ah));
                            sgb = fma2(g[i + v], bv, sgb);
                            sea = fma2(e, A2[i + v], sea);
                            dA[i + v] = fma2(e, D2, dA[i + v]);
                            g[i + v] = mul2(g[i + v], av[j][i + v]);
                        }
                        channel_sum_write<NP>(sm.sum, j & 1, lane, 2 * i, db[0], db[1]);
                        channel_sum_write<NP>(sm.sum, j & 1, lane, NP + 2 * i, dc[0], dc[1]);
                    }
                    if (kEdges && sm.first[k] >= 0 && a.dh0 && live) store_pairs<NP>(g, a.dh0 + sm.first[k] * row + at, a.N);
                    __syncwarp();  // (the next token writes the other buffer)
                    channel_sum_read<NP>(sm.sum, j & 1, lane, part + (tt + k) * a.G * 2 * a.N, a.N);
                    const float gb = lo2(sgb) + hi2(sgb), ea = (lo2(sea) + hi2(sea)) * 0.69314718055994531f;
                    float ddt = gb * uv[j] + ea;
                    if (a.softplus) ddt *= sigmoidf(to_f32<T>(sm.dt[buf][k][lane]) + bias);
                    aD += pv[j] * uv[j];
                    ab += ddt;
                    if (live) {
                        static_cast<T*>(a.du)[(tt + k) * a.lddu + d] = from_f32<T>(gb * Dv[j] + skip * pv[j]);
                        static_cast<T*>(a.ddt)[(tt + k) * a.ldddt + d] = from_f32<T>(ddt);
                        if (a.z)
                            static_cast<T*>(a.dz)[(tt + k) * a.lddz + d] = from_f32<T>(
                                to_f32<T>(sm.dy[buf][k][lane]) * (ys[j] + skip * uv[j]) * dsilu(to_f32<T>(sm.z[buf][k][lane])));
                    }
                }
            }
        };
        if (edges) walk(std::true_type{});
        else walk(std::false_type{});
        __syncwarp();
    }
    if (live) {
        store_pairs<NP>(dA, a.part_a + si * row + at, a.N);
        a.part_d[si * 2 * a.D + d] = aD;
        a.part_d[(si * 2 + 1) * a.D + d] = ab;
    }
}

// 2R values per lane summed over the 8 quads of a warp (lanes with the same q): each
// exchange hands half of the values to the partner, so lane (quad bits b4 b3 b2) is
// left with the values from number b4 R + b3 R/2 + b2 R/4 on, R/4 of them.
template <int R>
__device__ __forceinline__ void channel_sum(float (&v)[2 * R], int lane) {
    const bool b4 = lane & 16, b3 = lane & 8, b2 = lane & 4;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const float keep = b4 ? v[R + i] : v[i], give = b4 ? v[i] : v[R + i];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, give, 16);
    }
#pragma unroll
    for (int i = 0; i < R / 2; ++i) {
        const float keep = b3 ? v[R / 2 + i] : v[i], give = b3 ? v[i] : v[R / 2 + i];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, give, 8);
    }
#pragma unroll
    for (int i = 0; i < R / 4; ++i) {
        const float keep = b2 ? v[R / 4 + i] : v[i], give = b2 ? v[i] : v[R / 4 + i];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, give, 4);
    }
}

// The second pass for 17 to 32 states, which do not fit one lane's registers: a quad of
// lanes holds a channel, R = 8 states each; a block holds 32 channels.
template <int R>
struct BwdSmem {
    float4 s[kTT][kCh];  // D, D u, p
    float b[kTT][4 * R], c[kTT][4 * R];
    float gb[kTT][kYP], ea[kTT][kYP], hc[kTT][kYP];  // sums over n: g B, e A log2(e), h C
    float red[4][kTT][8 * R];                        // per warp: sums over its channels, [dB | dC]
    float bias[kCh], skip[kCh];
    int first[kTT], last[kTT];
};

template <typename T, int R, bool kVec>
__global__ void __launch_bounds__(128) bwd_quad_kernel(const SArgs a, bool bc_vec) {
    static_assert(R == 8, "what a lane is left with of the sums over channels");
    constexpr int KC = ckpt_tokens(4 * R);
    extern __shared__ __align__(16) uint8_t smem_raw[];
    BwdSmem<R>& sm = *reinterpret_cast<BwdSmem<R>*>(smem_raw);
    const int tid = threadIdx.x, q = tid & 3, c = tid >> 2, lane = tid & 31, warp = tid >> 5;
    const Place p = place(a);
    const int d = p.d0 + c, n0 = q * R;
    const bool live = d < p.dend;
    const long long si = (long long)p.b * a.S + p.s;
    float A2[R], g[R], hin[R], dA[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        A2[r] = live && n0 + r < a.N ? a.A[(size_t)d * a.N + n0 + r] * kL2e : 0.f;
        g[r] = hin[r] = dA[r] = 0.f;
    }
    if (tid < kCh) {
        const int e = p.d0 + tid;
        sm.bias[tid] = a.bias && e < p.dend ? a.bias[e] : 0.f;
        sm.skip[tid] = a.skip && e < p.dend ? a.skip[e] : 0.f;
    }
    if (a.dh0)  // empty sequences hand the final state's gradient on
        for (int n = blockIdx.y; n < a.nseq; n += gridDim.y)
            if (live && seq_begin(a.cu, a.seq_len, n, a.ntok) == seq_begin(a.cu, a.seq_len, n + 1, a.ntok)) {
                float e[R];
#pragma unroll
                for (int r = 0; r < R; ++r) e[r] = 0.f;
                if (a.dhT) load_h<R>(e, a.dhT + ((size_t)n * a.D + d) * a.N, n0, a.N);
                store_h<R>(e, a.dh0 + ((size_t)n * a.D + d) * a.N, n0, a.N);
            }
    if (p.t0 >= p.t1) return;  // (never: every segment has tokens)
    // the state that enters the segment, and the gradient that enters at its end
    const int nf = seq_of(a.cu, a.nseq, a.seq_len, int(p.t0));
    const long long f_beg = seq_begin(a.cu, a.seq_len, nf, a.ntok), f_end = seq_begin(a.cu, a.seq_len, nf + 1, a.ntok);
    if (live && f_beg < p.t0) state_before<R>(hin, a, p, f_beg, d, n0, A2);
    {
        const int nl = seq_of(a.cu, a.nseq, a.seq_len, int(p.t1 - 1));
        const long long l_end = seq_begin(a.cu, a.seq_len, nl + 1, a.ntok);
        if (live && l_end > p.t1) {
            float prod[R];
#pragma unroll
            for (int r = 0; r < R; ++r) prod[r] = 1.f;
            for (int i = p.s + 1; i < a.S; ++i) {
                float e[R];
                const long long at = (long long)p.b * a.S + i;
                load_h<R>(e, a.seg_g + (at * a.D + d) * a.N, n0, a.N);
                const float sd = a.seg_d[at * a.D + d];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    g[r] += prod[r] * e[r];
                    prod[r] *= ex2(A2[r] * sd);
                }
                if (l_end <= p.row0 + (long long)(i + 1) * a.L) break;
            }
        }
    }
    const int dv = p.d0 + 8 * q, valid = p.dend - dv;
    V8<T> ru, rd, rz, ry;
    VR<T, R> rb, rc;
    auto request = [&](long long tt) {
        const long long t = tt + c;
        if (t < p.t1) {
            load8<T, kVec>(ru, a.u, t, a.ldu, dv, valid);
            load8<T, kVec>(rd, a.dt, t, a.lddt, dv, valid);
            load8<T, kVec>(ry, a.dy, t, a.lddy, dv, valid);
            if (a.z) load8<T, kVec>(rz, a.z, t, a.ldz, dv, valid);
            load_states<T, R>(rb, a.Bm, t * a.ldb + (long long)p.g * a.N, n0, a.N, bc_vec);
            load_states<T, R>(rc, a.Cm, t * a.ldc + (long long)p.g * a.N, n0, a.N, bc_vec);
        } else {
            zero8<T>(ru);
            zero8<T>(rd);
            zero8<T>(ry);
            zero8<T>(rz);
#pragma unroll
            for (int r = 0; r < R; ++r) rb.v[r] = rc.v[r] = from_f32<T>(0.f);
        }
    };
    float aD[8], ab[8];  // this thread's part of dDskip and dbias: its tokens, 8 channels
#pragma unroll
    for (int i = 0; i < 8; ++i) aD[i] = ab[i] = 0.f;
    const long long chunk0 = si * (a.L / KC);
    const int tiles = int((p.t1 - p.t0 + kTT - 1) / kTT);
    request(p.t0 + (long long)(tiles - 1) * kTT);
    __syncthreads();
    for (int ti = tiles - 1; ti >= 0; --ti) {
        const long long tt = p.t0 + (long long)ti * kTT;
        const bool here = tt + c < p.t1;
        int ef = -1, el = -1;
        if (q == 0) {
            edge_flags(a, tt + c, here, ef, el);
            sm.first[c] = ef;
            sm.last[c] = el;
        }
        const V8<T> u8 = ru, d8 = rd, z8 = rz, y8 = ry;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float u = to_f32<T>(u8.v[i]);
            const float D = here ? step_size(to_f32<T>(d8.v[i]) + sm.bias[8 * q + i], a.softplus) : 0.f;
            float pv = to_f32<T>(y8.v[i]);
            if (a.z) {
                const float z = to_f32<T>(z8.v[i]);
                pv *= __fdividef(z, 1.f + __expf(-z));
            }
            sm.s[c][8 * q + i] = make_float4(D, D * u, pv, 0.f);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            sm.b[c][n0 + r] = to_f32<T>(rb.v[r]);
            sm.c[c][n0 + r] = to_f32<T>(rc.v[r]);
        }
        const bool edges = __syncthreads_or(ef >= 0 || el >= 0);
        if (ti > 0) request(tt - kTT);
        const int steps = int(p.t1 - tt < kTT ? p.t1 - tt : kTT);
        auto walk = [&](auto has_edges) {  // two bodies, as in the forward pass
        constexpr bool kEdges = decltype(has_edges)::value;
#pragma unroll 1
        for (int k0 = (steps - 1) / KC * KC; k0 >= 0; k0 -= KC) {
            const long long tc = tt + k0, ck = chunk0 + (tc - p.t0) / KC;
            float h[R], av[KC][R], hp[KC][R];
#pragma unroll
            for (int r = 0; r < R; ++r) h[r] = 0.f;
            if (live) {
                load_h<R>(h, a.ckpt + (ck * a.D + d) * (4 * R), n0, a.N);
                if (f_beg < p.t0 && tc < f_end) {  // the checkpoint counts from zero: add the incoming state's part
                    const float sd = a.ckpt_d[ck * a.D + d];
#pragma unroll
                    for (int r = 0; r < R; ++r) h[r] += ex2(A2[r] * sd) * hin[r];
                }
            }
#pragma unroll
            for (int j4 = 0; j4 < KC; j4 += 4) {
                float acc[4];
#pragma unroll
                for (int jj = 0; jj < 4; ++jj) {
                    const int j = j4 + jj, k = k0 + j;
                    if (kEdges && sm.first[k] >= 0) {
#pragma unroll
                        for (int r = 0; r < R; ++r) h[r] = 0.f;
                        if (a.h0 && live) load_h<R>(h, a.h0 + ((size_t)sm.first[k] * a.D + d) * a.N, n0, a.N);
                    }
                    const float4 s = sm.s[k][c];
                    acc[jj] = 0.f;
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        av[j][r] = ex2(s.x * A2[r]);
                        hp[j][r] = h[r];
                        h[r] = av[j][r] * h[r] + s.y * sm.b[k][n0 + r];
                        acc[jj] += h[r] * sm.c[k][n0 + r];
                    }
                }
                sm.hc[k0 + j4 + q][c] = lane_transpose_sum<4>(acc, q);
            }
#pragma unroll
            for (int j4 = KC - 4; j4 >= 0; j4 -= 4) {
                float agb[4], aea[4];
#pragma unroll
                for (int jj = 3; jj >= 0; --jj) {
                    const int j = j4 + jj, k = k0 + j;
                    const float4 s = sm.s[k][c];
                    if (kEdges && sm.last[k] >= 0) {
#pragma unroll
                        for (int r = 0; r < R; ++r) g[r] = 0.f;
                        if (a.dhT && live) load_h<R>(g, a.dhT + ((size_t)sm.last[k] * a.D + d) * a.N, n0, a.N);
                    }
                    agb[jj] = aea[jj] = 0.f;
                    float v[2 * R];
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const float Bv = sm.b[k][n0 + r], Cv = sm.c[k][n0 + r];
                        g[r] += Cv * s.z;
                        const float ah = av[j][r] * hp[j][r];
                        const float e = g[r] * ah;
                        v[r] = g[r] * s.y;
                        v[R + r] = s.z * (ah + s.y * Bv);
                        agb[jj] += g[r] * Bv;
                        aea[jj] += e * A2[r];
                        dA[r] += e * s.x;
                        g[r] *= av[j][r];
                    }
                    if (kEdges && sm.first[k] >= 0 && a.dh0 && live)
                        store_h<R>(g, a.dh0 + ((size_t)sm.first[k] * a.D + d) * a.N, n0, a.N);
                    channel_sum<R>(v, lane);
                    // value number b4 R + b3 R/2 + ... of the list [dB | dC] of this lane's states
                    float* o = sm.red[warp][k] + ((lane & 16) ? 4 * R : 0) + n0;
                    o[((lane >> 1) & 4) + ((lane >> 1) & 2)] = v[0];
                    o[((lane >> 1) & 4) + ((lane >> 1) & 2) + 1] = v[1];
                }
                sm.gb[k0 + j4 + q][c] = lane_transpose_sum<4>(agb, q);
                sm.ea[k0 + j4 + q][c] = lane_transpose_sum<4>(aea, q);
            }
        }
        };
        if (edges) walk(std::true_type{});
        else walk(std::false_type{});
        __syncthreads();
        if (here) {
            float odu[8], odt[8], odz[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int ch = 8 * q + i;
                const float4 s = sm.s[c][ch];
                const float u = to_f32<T>(u8.v[i]), gb = sm.gb[c][ch];
                odu[i] = gb * s.x + sm.skip[ch] * s.z;
                float dD = gb * u + sm.ea[c][ch] * 0.69314718055994531f;
                if (a.softplus) dD *= sigmoidf(to_f32<T>(d8.v[i]) + sm.bias[ch]);
                odt[i] = dD;
                aD[i] += s.z * u;
                ab[i] += dD;
                if (a.z) odz[i] = to_f32<T>(y8.v[i]) * (sm.hc[c][ch] + sm.skip[ch] * u) * dsilu(to_f32<T>(z8.v[i]));
            }
            store8<T, kVec>(a.du, tt + c, a.lddu, dv, valid, odu);
            store8<T, kVec>(a.ddt, tt + c, a.ldddt, dv, valid, odt);
            if (a.z) store8<T, kVec>(a.dz, tt + c, a.lddz, dv, valid, odz);
        }
        // the block's sums over its channels: [block of the group][token][group][dB | dC][N]
        for (int i = tid; i < steps * 8 * R; i += 128) {
            const int k = i / (8 * R), v = i % (8 * R), n = v % (4 * R);
            if (n < a.N) {
                const float t = sm.red[0][k][v] + sm.red[1][k][v] + sm.red[2][k][v] + sm.red[3][k][v];
                const long long tok = tt + k, ntok = (long long)a.rows * a.row_len;
                a.part_bc[((((long long)(blockIdx.x % a.bpg) * ntok + tok) * a.G + p.g) * 2 + v / (4 * R)) * a.N + n] = t;
            }
        }
        __syncthreads();
    }
    if (live) store_h<R>(dA, a.part_a + (si * a.D + d) * a.N, n0, a.N);
    // dDskip and dbias: sums over the 32 token slots of the block
    float* buf = &sm.gb[0][0];  // gb, ea and hc in a row: 2 x 32 x 33 floats fit
    static_assert(3 * kTT * kYP >= 2 * 32 * 33, "room for the final sums");
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        buf[c * 33 + 8 * q + i] = aD[i];
        buf[32 * 33 + c * 33 + 8 * q + i] = ab[i];
    }
    __syncthreads();
    if (tid < 64) {
        const int which = tid >> 5, ch = tid & 31;
        float t = 0.f;
        for (int k = 0; k < 32; ++k) t += buf[which * 32 * 33 + k * 33 + ch];
        if (p.d0 + ch < p.dend) a.part_d[(si * 2 + which) * a.D + p.d0 + ch] = t;
    }
}

// The last sums, each in a fixed order, in one launch: dB and dC from the blocks' sums
// [block][token][group][2][N] (1024 outputs a block, threads side by side), then 32
// columns a block of dA, dDskip and dbias from the segments'.
template <typename T>
__global__ void __launch_bounds__(1024) bwd_finish_kernel(const SArgs a, const BwdOut o, int bc_blocks, int a_blocks) {
    __shared__ float s[32][33];
    if (int(blockIdx.x) < bc_blocks) {
        const long long total = (long long)a.rows * a.row_len * a.G * 2 * a.N;
        const long long i = (long long)blockIdx.x * 1024 + threadIdx.x;
        if (i >= total) return;
        float t = 0.f;
#pragma unroll 8
        for (int k = 0; k < a.bpg; ++k) t += a.part_bc[k * total + i];
        const int n = int(i % a.N);
        const long long r = i / a.N, tg = r >> 1, tok = tg / a.G, g = tg % a.G;
        if (r & 1) static_cast<T*>(o.dC)[tok * o.lddc + g * a.N + n] = from_f32<T>(t);
        else static_cast<T*>(o.dB)[tok * o.lddb + g * a.N + n] = from_f32<T>(t);
        return;
    }
    const int lane = threadIdx.x & 31, row = threadIdx.x >> 5, b = blockIdx.x - bc_blocks;
    const int per = (a.D + 31) / 32;  // blocks of a vector of channels
    const float* part;
    float* out;
    long long n, stride, i;
    if (b < a_blocks) {
        part = a.part_a;
        out = o.dA;
        n = stride = (long long)a.D * a.N;
        i = (long long)b * 32 + lane;
    } else {
        const int which = (b - a_blocks) / per;
        part = a.part_d + which * a.D;
        out = which ? o.dbias : o.dskip;
        n = a.D;
        stride = 2ll * a.D;
        i = (long long)((b - a_blocks) % per) * 32 + lane;
    }
    if (!out) return;
    float t = 0.f;
    if (i < n) {
#pragma unroll 8
        for (int k = row; k < a.rows * a.S; k += 32) t += part[k * stride + i];
    }
    s[row][lane] = t;
    __syncthreads();
    if (row == 0 && i < n) {
        t = 0.f;
#pragma unroll
        for (int r = 0; r < 32; ++r) t += s[r][lane];
        out[i] = t;
    }
}

// Segments of the backward pass: the map pass runs in any case (checkpoints), so they
// may be shorter than the forward pass's.
static Cut bwd_cut(int B, int T, int D, int G, int N, bool packed) {
    Cut c{};
    c.rows = packed ? 1 : B;
    c.row_len = T;
    c.bpg = int(cdiv(D / G, kCh));
    const long long blocks = (long long)c.rows * G * c.bpg;
    // Up to 16 states the second pass holds 8 warps an SM (its registers): one full wave of
    // warps (8192 tokens of 4096 channels in all: 8 segments 380 us, 12 485 us, 16 394 us).
    // Above, 4 blocks of 4 warps an SM.
    long long S = N <= 16 ? 8ll * device_sm_count() / blocks : cdiv(4ll * device_sm_count(), blocks);
    cut_row(c, S);
    return c;
}

struct BwdPlan {
    Cut c;
    size_t off_segh, off_segd, off_segg, off_ckpt, off_ckptd, off_bc, off_a, off_d, total;
};
static BwdPlan bwd_plan(int B, int T, int D, int G, int N, bool packed) {
    BwdPlan p{};
    p.c = bwd_cut(B, T, D, G, N, packed);
    const int NP = padded_states(N);
    const size_t segs = size_t(p.c.rows) * p.c.S, chunks = segs * (p.c.L / ckpt_tokens(NP)), toks = size_t(p.c.rows) * T;
    size_t off = 0;
    auto take = [&](size_t floats) {
        const size_t at = off;
        off += mix::up256(floats * 4);
        return at;
    };
    p.off_segh = take(segs * D * N);
    p.off_segd = take(segs * D);
    p.off_segg = take(segs * D * N);
    p.off_ckpt = take(chunks * D * NP);
    p.off_ckptd = take(chunks * D);
    p.off_bc = take(size_t(p.c.bpg) * toks * G * 2 * N);
    p.off_a = take(segs * D * N);
    p.off_d = take(segs * 2 * D);
    p.total = off;
    return p;
}

template <typename T, int NP, int kCopy>
int bwd_run(const SArgs& a, const BwdOut& o, bool bc, bool vec, cudaStream_t st) {
    const dim3 grid(a.G * a.bpg, a.rows * a.S);
    bwd_map_kernel<T, NP, kCopy><<<grid, 32, 0, st>>>(a, bc);
    if constexpr (NP <= 16) {
        auto kern = bwd_kernel<T, NP, kCopy>;
        if (!set_smem_attr(kern, sizeof(MainSmem<T, NP>))) return KDA_ERR_CUDA;
        kern<<<grid, 32, sizeof(MainSmem<T, NP>), st>>>(a, bc);
    } else {
        auto kern = vec ? bwd_quad_kernel<T, NP / 4, true> : bwd_quad_kernel<T, NP / 4, false>;
        if (!set_smem_attr(kern, sizeof(BwdSmem<NP / 4>))) return KDA_ERR_CUDA;
        kern<<<grid, 128, sizeof(BwdSmem<NP / 4>), st>>>(a, states_ok(a, sizeof(T), NP / 4));
    }
    const long long bc_blocks = cdiv((long long)a.rows * a.row_len * a.G * 2 * a.N, 1024);
    const long long a_blocks = cdiv((long long)a.D * a.N, 32);
    bwd_finish_kernel<T><<<unsigned(bc_blocks + a_blocks + 2 * cdiv(a.D, 32)), 1024, 0, st>>>(a, o, int(bc_blocks), int(a_blocks));
    return cudaPeekAtLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

template <typename T, int NP>
int bwd_states(const SArgs& a, const BwdOut& o, cudaStream_t st) {
    const void* ptrs[] = {a.u, a.dt, a.z, a.dy, a.du, a.ddt, a.dz};
    const long long lds[] = {a.ldu, a.lddt, a.ldz, a.lddy, a.lddu, a.ldddt, a.lddz};
    const int copy = copy_bytes(a, sizeof(T), ptrs, lds, 4);  // of the inputs
    const bool vec = vec8_ok(a, sizeof(T), ptrs, lds, 7), bc = bc_whole(a, sizeof(T));
    if (copy == 16) return bwd_run<T, NP, 16>(a, o, bc, vec, st);
    return copy == 4 ? bwd_run<T, NP, 4>(a, o, bc, vec, st) : bwd_run<T, NP, 0>(a, o, bc, vec, st);
}
template <typename T>
int bwd(const SArgs& a, const BwdOut& o, cudaStream_t st) {
    if (a.N <= 8) return bwd_states<T, 8>(a, o, st);
    return a.N <= 16 ? bwd_states<T, 16>(a, o, st) : bwd_states<T, 32>(a, o, st);
}

}  // namespace scan

size_t selective_scan_bwd_workspace_bytes(int B, int T, int D, int G, int N, bool packed) {
    return scan::bwd_plan(B, T, D, G, N, packed).total;
}

int launch_selective_scan_bwd(scan::SArgs a, const scan::BwdOut& o, int B, int tokens, int dtype, void* ws,
                              cudaStream_t st) {
    const scan::BwdPlan p = scan::bwd_plan(B, tokens, a.D, a.G, a.N, a.cu != nullptr);
    scan_cut_args(a, p.c);
    uint8_t* b = static_cast<uint8_t*>(ws);
    a.seg_h = reinterpret_cast<float*>(b + p.off_segh);
    a.seg_d = reinterpret_cast<float*>(b + p.off_segd);
    a.seg_g = reinterpret_cast<float*>(b + p.off_segg);
    a.ckpt = reinterpret_cast<float*>(b + p.off_ckpt);
    a.ckpt_d = reinterpret_cast<float*>(b + p.off_ckptd);
    a.part_bc = reinterpret_cast<float*>(b + p.off_bc);
    a.part_a = reinterpret_cast<float*>(b + p.off_a);
    a.part_d = reinterpret_cast<float*>(b + p.off_d);
    return dtype == KDA_BF16 ? scan::bwd<__nv_bfloat16>(a, o, st) : scan::bwd<float>(a, o, st);
}

}  // namespace kda
