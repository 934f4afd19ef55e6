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
// writes the state before every KC = 32 / R tokens, counted from a zero state at
// its segment's start, with the sum of D up to there: the decay from the segment's
// start to that token is exp(A sum(D)), so a checkpoint is completed by adding that
// times the segment's incoming state.  The same pass accumulates the reverse map
// of the segment, G = sum_t (a_1 .. a_t) C_t p_t: the gradient of the incoming
// state is G + exp(A sum(D)) times the gradient of the state at its end.  So both
// directions of the recurrence cross segments by a few operations per state, and
// the second pass runs every segment on its own: per run of KC tokens it computes
// the states forward from the checkpoint into registers, then walks back.
//
// The sums over n of a channel are sums over a quad of lanes (four tokens at a
// time); the sums over the channels for dB and dC are sums over the eight quads of
// a warp by a halving exchange, then over the warps and blocks in a fixed order:
// every result is the same on every run.
#include "kda_mixer.cuh"

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
        if (seq_begin(a.cu, a.seq_len, m) == t) first = m;
        if (seq_begin(a.cu, a.seq_len, m + 1) == t + 1) last = m;
    }
}

template <typename T, int R, bool kVec>
__global__ void __launch_bounds__(128) bwd_map_kernel(const SArgs a, bool bc_vec) {
    constexpr int KC = 32 / R;
    __shared__ __align__(16) float2 sdu[2][kTT][kCh];
    __shared__ float sp[2][kTT][kCh + 8];
    __shared__ __align__(16) float sb[2][kTT][4 * R], sc[2][kTT][4 * R];
    __shared__ float sbias[kCh];
    __shared__ int sfirst[2][kTT], slast[2][kTT];
    const int tid = threadIdx.x, q = tid & 3, c = tid >> 2;
    const Place p = place(a);
    if (p.t0 >= p.t1) return;
    const int d = p.d0 + c, n0 = q * R;
    const bool live = d < p.dend;
    float A2[R], h[R], P[R], G[R], dsum = 0.f;
    bool open = true;  // no sequence has ended in the segment yet: later tokens do not see the incoming state
#pragma unroll
    for (int r = 0; r < R; ++r) {
        A2[r] = live && n0 + r < a.N ? a.A[(size_t)d * a.N + n0 + r] * kLog2e : 0.f;
        h[r] = G[r] = 0.f;
        P[r] = 1.f;
    }
    if (tid < kCh) sbias[tid] = a.bias && p.d0 + tid < p.dend ? a.bias[p.d0 + tid] : 0.f;
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
        }
    };
    request(p.t0);
    __syncthreads();
    const long long chunk0 = ((long long)p.b * a.S + p.s) * (a.L / KC);
    int buf = 0;
    for (long long tt = p.t0; tt < p.t1; tt += kTT, buf ^= 1) {
        const bool here = tt + c < p.t1;
        int ef = -1, el = -1;
        if (q == 0) {
            edge_flags(a, tt + c, here, ef, el);
            sfirst[buf][c] = ef;
            slast[buf][c] = el;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float u = here ? to_f32<T>(ru.v[i]) : 0.f;
            const float D = here ? step_size(to_f32<T>(rd.v[i]) + sbias[8 * q + i], a.softplus) : 0.f;
            float pv = here ? to_f32<T>(ry.v[i]) : 0.f;
            if (a.z && here) {
                const float z = to_f32<T>(rz.v[i]);
                pv *= __fdividef(z, 1.f + __expf(-z));
            }
            sdu[buf][c][8 * q + i] = make_float2(D, D * u);
            sp[buf][c][8 * q + i] = pv;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            sb[buf][c][n0 + r] = here ? to_f32<T>(rb.v[r]) : 0.f;
            sc[buf][c][n0 + r] = here ? to_f32<T>(rc.v[r]) : 0.f;
        }
        const bool edges = __syncthreads_or(ef >= 0 || el >= 0);
        if (tt + kTT < p.t1) request(tt + kTT);
        const int steps = int(p.t1 - tt < kTT ? p.t1 - tt : kTT);
#pragma unroll 1
        for (int k0 = 0; k0 < steps; k0 += KC) {
            const long long ck = chunk0 + (tt - p.t0 + k0) / KC;
            if (live) {
                store_h<R>(h, a.ckpt + (ck * a.D + d) * a.N, n0, a.N);
                if (q == 0) a.ckpt_d[ck * a.D + d] = dsum;
            }
#pragma unroll
            for (int j = 0; j < KC; ++j) {
                const int k = k0 + j;
                if (edges && sfirst[buf][k] >= 0) {
#pragma unroll
                    for (int r = 0; r < R; ++r) h[r] = 0.f;
                    if (a.h0 && live) load_h<R>(h, a.h0 + ((size_t)sfirst[buf][k] * a.D + d) * a.N, n0, a.N);
                }
                const float2 du = sdu[buf][k][c];
                const float pv = sp[buf][k][c];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float e = ex2(du.x * A2[r]);
                    h[r] = e * h[r] + du.y * sb[buf][k][n0 + r];
                    P[r] *= e;
                    if (open) G[r] += P[r] * (sc[buf][k][n0 + r] * pv);
                }
                dsum += du.x;
                if (edges && slast[buf][k] >= 0) {
                    if (open && a.dhT && live) {
                        float e[R];
                        load_h<R>(e, a.dhT + ((size_t)slast[buf][k] * a.D + d) * a.N, n0, a.N);
#pragma unroll
                        for (int r = 0; r < R; ++r) G[r] += P[r] * e[r];
                    }
                    open = false;
                }
            }
        }
    }
    if (live) {
        const long long i = (long long)p.b * a.S + p.s;
        store_h<R>(h, a.seg_h + (i * a.D + d) * a.N, n0, a.N);
        store_h<R>(G, a.seg_g + (i * a.D + d) * a.N, n0, a.N);
        if (q == 0) a.seg_d[i * a.D + d] = dsum;
    }
}

// 2R values per lane summed over the 8 quads of a warp (lanes with the same q): each
// exchange hands half of the values to the partner, so lane (quad bits b4 b3 b2) is
// left with value(s) number b4 R + b3 R/2 + ...; returns how many (kLeft).
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
    if constexpr (R >= 4) {
#pragma unroll
        for (int i = 0; i < R / 4; ++i) {
            const float keep = b2 ? v[R / 4 + i] : v[i], give = b2 ? v[i] : v[R / 4 + i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, 4);
        }
    } else {
        v[0] += __shfl_xor_sync(0xffffffffu, v[0], 4);
    }
}

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
__global__ void __launch_bounds__(128) bwd_kernel(const SArgs a, bool bc_vec) {
    constexpr int KC = 32 / R;
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
        A2[r] = live && n0 + r < a.N ? a.A[(size_t)d * a.N + n0 + r] * kLog2e : 0.f;
        g[r] = hin[r] = dA[r] = 0.f;
    }
    if (tid < kCh) {
        const int e = p.d0 + tid;
        sm.bias[tid] = a.bias && e < p.dend ? a.bias[e] : 0.f;
        sm.skip[tid] = a.skip && e < p.dend ? a.skip[e] : 0.f;
    }
    if (a.dh0)  // empty sequences hand the final state's gradient on
        for (int n = blockIdx.y; n < a.nseq; n += gridDim.y)
            if (live && seq_begin(a.cu, a.seq_len, n) == seq_begin(a.cu, a.seq_len, n + 1)) {
                float e[R];
#pragma unroll
                for (int r = 0; r < R; ++r) e[r] = 0.f;
                if (a.dhT) load_h<R>(e, a.dhT + ((size_t)n * a.D + d) * a.N, n0, a.N);
                store_h<R>(e, a.dh0 + ((size_t)n * a.D + d) * a.N, n0, a.N);
            }
    if (p.t0 >= p.t1) return;  // (never: every segment has tokens)
    // the state that enters the segment, and the gradient that enters at its end
    const int nf = seq_of(a.cu, a.nseq, a.seq_len, int(p.t0));
    const long long f_beg = seq_begin(a.cu, a.seq_len, nf), f_end = seq_begin(a.cu, a.seq_len, nf + 1);
    if (live && f_beg < p.t0) state_before<R>(hin, a, p, f_beg, d, n0, A2);
    {
        const int nl = seq_of(a.cu, a.nseq, a.seq_len, int(p.t1 - 1));
        const long long l_end = seq_begin(a.cu, a.seq_len, nl + 1);
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
#pragma unroll 1
        for (int k0 = (steps - 1) / KC * KC; k0 >= 0; k0 -= KC) {
            const long long tc = tt + k0, ck = chunk0 + (tc - p.t0) / KC;
            float h[R], av[KC][R], hp[KC][R];
#pragma unroll
            for (int r = 0; r < R; ++r) h[r] = 0.f;
            if (live) {
                load_h<R>(h, a.ckpt + (ck * a.D + d) * a.N, n0, a.N);
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
                    if (edges && sm.first[k] >= 0) {
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
                sm.hc[k0 + j4 + q][c] = quad_transpose_sum(acc, q);
            }
#pragma unroll
            for (int j4 = KC - 4; j4 >= 0; j4 -= 4) {
                float agb[4], aea[4];
#pragma unroll
                for (int jj = 3; jj >= 0; --jj) {
                    const int j = j4 + jj, k = k0 + j;
                    const float4 s = sm.s[k][c];
                    if (edges && sm.last[k] >= 0) {
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
                    if (edges && sm.first[k] >= 0 && a.dh0 && live)
                        store_h<R>(g, a.dh0 + ((size_t)sm.first[k] * a.D + d) * a.N, n0, a.N);
                    channel_sum<R>(v, lane);
                    // value number b4 R + b3 R/2 + ... of the list [dB | dC] of this lane's states
                    float* o = sm.red[warp][k] + ((lane & 16) ? 4 * R : 0) + n0;
                    if constexpr (R == 2) {
                        if (!(lane & 4)) o[(lane >> 3) & 1] = v[0];
                    } else if constexpr (R == 4) {
                        o[((lane >> 2) & 2) + ((lane >> 2) & 1)] = v[0];
                    } else {
                        o[((lane >> 1) & 4) + ((lane >> 1) & 2)] = v[0];
                        o[((lane >> 1) & 4) + ((lane >> 1) & 2) + 1] = v[1];
                    }
                }
                sm.gb[k0 + j4 + q][c] = quad_transpose_sum(agb, q);
                sm.ea[k0 + j4 + q][c] = quad_transpose_sum(aea, q);
            }
        }
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

// dB and dC from the blocks' sums [block][token][group][2][N].
template <typename T>
__global__ void __launch_bounds__(256) bwd_bc_sum_kernel(const float* __restrict__ part, int parts, long long total,
                                                         int G, int N, T* __restrict__ dB, long long lddb,
                                                         T* __restrict__ dC, long long lddc) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= total) return;
    float t = 0.f;
#pragma unroll 8
    for (int k = 0; k < parts; ++k) t += part[k * total + i];
    const int n = int(i % N);
    const long long r = i / N, tg = r >> 1;
    const long long tok = tg / G, g = tg % G;
    if (r & 1) dC[tok * lddc + g * N + n] = from_f32<T>(t);
    else dB[tok * lddb + g * N + n] = from_f32<T>(t);
}

// Segments of the backward pass: the map pass runs in any case (checkpoints), so they
// may be shorter than the forward pass's.
static Cut bwd_cut(int B, int T, int D, int G, bool packed) {
    Cut c{};
    c.rows = packed ? 1 : B;
    c.row_len = T;
    c.bpg = int(cdiv(D / G, kCh));
    const long long blocks = (long long)c.rows * G * c.bpg;
    long long S = cdiv((long long)device_sm_count() * 3, blocks);
    const long long most = T / 128 < 32 ? T / 128 : 32;
    if (S > most) S = most;
    if (S < 1) S = 1;
    c.L = int(cdiv(cdiv(T, S), kTT) * kTT);
    c.S = int(cdiv(T, c.L));
    return c;
}

struct BwdPlan {
    Cut c;
    size_t off_segh, off_segd, off_segg, off_ckpt, off_ckptd, off_bc, off_a, off_d, total;
};
static BwdPlan bwd_plan(int B, int T, int D, int G, int N, bool packed) {
    BwdPlan p{};
    p.c = bwd_cut(B, T, D, G, packed);
    const size_t segs = size_t(p.c.rows) * p.c.S, KC = 32 / states_per_lane(N);
    const size_t chunks = segs * (p.c.L / KC), toks = size_t(p.c.rows) * T;
    size_t off = 0;
    auto take = [&](size_t floats) {
        const size_t at = off;
        off += mix::up256(floats * 4);
        return at;
    };
    p.off_segh = take(segs * D * N);
    p.off_segd = take(segs * D);
    p.off_segg = take(segs * D * N);
    p.off_ckpt = take(chunks * D * N);
    p.off_ckptd = take(chunks * D);
    p.off_bc = take(size_t(p.c.bpg) * toks * G * 2 * N);
    p.off_a = take(segs * D * N);
    p.off_d = take(segs * 2 * D);
    p.total = off;
    return p;
}

struct BwdOut {
    void *dB, *dC;
    long long lddb, lddc;
    float *dA, *dskip, *dbias;
};

template <typename T, int R, bool kVec>
int bwd_vec(const SArgs& a, const BwdOut& o, bool bc, cudaStream_t st) {
    const dim3 grid(a.G * a.bpg, a.rows * a.S);
    bwd_map_kernel<T, R, kVec><<<grid, 128, 0, st>>>(a, bc);
    auto kern = bwd_kernel<T, R, kVec>;
    if (!set_smem_attr(kern, sizeof(BwdSmem<R>))) return KDA_ERR_CUDA;
    kern<<<grid, 128, sizeof(BwdSmem<R>), st>>>(a, bc);
    const long long total = (long long)a.rows * a.row_len * a.G * 2 * a.N;
    bwd_bc_sum_kernel<T><<<unsigned(cdiv(total, 256)), 256, 0, st>>>(a.part_bc, a.bpg, total, a.G, a.N,
                                                                     static_cast<T*>(o.dB), o.lddb,
                                                                     static_cast<T*>(o.dC), o.lddc);
    const int segs = a.rows * a.S;
    const long long dn = (long long)a.D * a.N;
    sum_parts_kernel<float><<<unsigned(cdiv(dn, 32)), 256, 0, st>>>(a.part_a, segs, dn, o.dA, dn);
    if (o.dskip) sum_parts_kernel<float><<<unsigned(cdiv(a.D, 32)), 256, 0, st>>>(a.part_d, segs, 2ll * a.D, o.dskip, a.D);
    if (o.dbias)
        sum_parts_kernel<float><<<unsigned(cdiv(a.D, 32)), 256, 0, st>>>(a.part_d + a.D, segs, 2ll * a.D, o.dbias, a.D);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

template <typename T, int R>
int bwd(const SArgs& a, const BwdOut& o, cudaStream_t st) {
    const void* ptrs[] = {a.u, a.dt, a.z, a.dy, a.du, a.ddt, a.dz};
    const long long lds[] = {a.ldu, a.lddt, a.ldz, a.lddy, a.lddu, a.ldddt, a.lddz};
    const bool bc = states_ok(a, sizeof(T), R);
    if (vec8_ok(a, sizeof(T), ptrs, lds, 7)) return bwd_vec<T, R, true>(a, o, bc, st);
    return bwd_vec<T, R, false>(a, o, bc, st);
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
    KDA_SCAN_DISPATCH(a.N, (scan::bwd<T, R>(a, o, st)))
}

}  // namespace kda
