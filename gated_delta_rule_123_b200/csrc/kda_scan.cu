// Selective state-space scan, forward: prompts and single tokens.
//
// Per channel d with N states, over the tokens t of a sequence:
//   D_t = softplus(dt_t + bias),  a_t[n] = exp(D_t A[n])
//   h_t[n] = a_t[n] h_{t-1}[n] + D_t u_t B_t[n]
//   y_t = (sum_n C_t[n] h_t[n] + Dskip u_t) SiLU(z_t)
// with B and C shared by the channels of a group.  A diagonal relative of the
// recurrences next to it: KDA's decay is per key channel and shared by the value
// columns, here every (channel, state) pair has its own, made from a step size
// per token, so the chunk form by matrix products does not apply.
//
// What bounds it: u, dt, z and y pass HBM once, but every (token, channel, state)
// needs one exponential, and the special-function unit gives 16 a clock and SM.
//
// Layout.  A quad of lanes holds one channel, R = N / 4 states a lane; a block of
// 128 threads holds 32 channels and walks its tokens in tiles of 32.  For each tile
// a thread loads one token's 16-byte vector of 8 channels of u, dt and z while the
// tile before is computed, turns them into (D, D u) pairs in shared memory, and
// after the tile's recurrence finishes the same 8 outputs, so global memory is read
// and written in whole vectors once.  Sums over n: four tokens of a quad are
// reduced together by a transposing exchange (3 shuffles for 4 tokens), which
// leaves each lane with one token's sum.
//
// Few sequences do not fill the SMs, so the token axis is cut into segments: a
// first pass runs all but the last one's recurrence from a zero state (no y) and
// leaves the end state and sum(D) of each; since the decay over a segment is
// exp(A sum(D)), the second pass starts each segment from the states before it.
#include "kda_mixer.cuh"

namespace kda {

namespace scan {

using namespace mix;

constexpr int kTT = 32;   // tokens of a tile
constexpr int kCh = 32;   // channels of a block
constexpr int kYP = 40;   // row pitch of the tile of sums: quads' four rows fall on different banks
constexpr float kLog2e = 1.4426950408889634f;

struct SArgs {
    const void *u, *dt, *z, *Bm, *Cm, *dy;
    const float *A, *skip, *bias, *h0;
    float* hT;
    void* y;
    const int32_t* cu;
    long long ldu, lddt, ldz, ldb, ldc, ldy, lddy;  // elements from token to token
    int nseq, seq_len;                              // sequences; dense: tokens of each
    int rows, row_len;  // dense: B rows of T tokens; packed: one row of all tokens
    int D, G, N, Dg, bpg;  // channels, groups, states, channels per group, blocks per group
    int softplus;
    int L, S;              // tokens per segment, segments per row
    float *seg_h, *seg_d;  // [rows S][D][N] end states from zero, [rows S][D] sums of D
    // backward
    const float* dhT;
    float *ckpt, *ckpt_d, *seg_g;  // states and sums of D at every chunk's start; the reverse maps
    float *part_bc, *part_a, *part_d;
    void *du, *ddt, *dz;
    float* dh0;
    long long lddu, ldddt, lddz;
};

template <typename T>
struct alignas(16) V8 {
    T v[8];
};
template <typename T, int R>
struct alignas(R * sizeof(T) < 16 ? R * sizeof(T) : 16) VR {
    T v[R];
};

// 8 channels of one token: whole vectors, or element by element up to `valid`.
template <typename T, bool kVec>
__device__ __forceinline__ void load8(V8<T>& r, const void* base, long long tok, long long ld, int d, int valid) {
    const T* p = static_cast<const T*>(base) + tok * ld + d;
    if constexpr (kVec) {
        if (valid >= 8) {
            r = *reinterpret_cast<const V8<T>*>(p);
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) r.v[i] = i < valid ? p[i] : from_f32<T>(0.f);
}
template <typename T, bool kVec>
__device__ __forceinline__ void store8(void* base, long long tok, long long ld, int d, int valid, const float* f) {
    T* p = static_cast<T*>(base) + tok * ld + d;
    if constexpr (kVec) {
        if (valid >= 8) {
            V8<T> r;
#pragma unroll
            for (int i = 0; i < 8; ++i) r.v[i] = from_f32<T>(f[i]);
            *reinterpret_cast<V8<T>*>(p) = r;
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < valid) p[i] = from_f32<T>(f[i]);
}
template <typename T>
__device__ __forceinline__ void zero8(V8<T>& r) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.v[i] = from_f32<T>(0.f);
}

// R states of one token's B or C (states n0 .. n0 + R - 1 of N).
template <typename T, int R>
__device__ __forceinline__ void load_states(VR<T, R>& r, const void* base, long long off, int n0, int N, bool vec) {
    const T* p = static_cast<const T*>(base) + off + n0;
    if (vec) {
        r = *reinterpret_cast<const VR<T, R>*>(p);
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i) r.v[i] = n0 + i < N ? p[i] : from_f32<T>(0.f);
    }
}

// 2^x on the special-function unit (relative error about 2^-22; below 2^-126 it gives 0).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float step_size(float raw, int softplus) { return softplus ? softplusf(raw) : raw; }

// R fp32 states of (row r of [..][N]) at n0; zero beyond N.
template <int R>
__device__ __forceinline__ void load_h(float (&h)[R], const float* p, int n0, int N) {
#pragma unroll
    for (int i = 0; i < R; ++i) h[i] = n0 + i < N ? p[n0 + i] : 0.f;
}
template <int R>
__device__ __forceinline__ void store_h(const float (&h)[R], float* p, int n0, int N) {
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (n0 + i < N) p[n0 + i] = h[i];
}

// v[j] of the quad's four lanes summed; lane q is left with the sum of v[q].
__device__ __forceinline__ float quad_transpose_sum(const float (&v)[4], int q) {
    const bool hi = q & 2, lo = q & 1;
    float a0 = hi ? v[2] : v[0], a1 = hi ? v[3] : v[1];
    a0 += __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[2], 2);
    a1 += __shfl_xor_sync(0xffffffffu, hi ? v[1] : v[3], 2);
    const float k = lo ? a1 : a0;
    return k + __shfl_xor_sync(0xffffffffu, lo ? a0 : a1, 1);
}

// What a block works on: segment s of row b, channels d0 .. of group g.
struct Place {
    int b, s, g, d0, dend;
    long long row0, t0, t1;  // tokens on the flattened axis
};
__device__ __forceinline__ Place place(const SArgs& a) {
    Place p;
    p.b = blockIdx.y / a.S;
    p.s = blockIdx.y % a.S;
    p.g = blockIdx.x / a.bpg;
    p.d0 = p.g * a.Dg + (blockIdx.x % a.bpg) * kCh;
    p.dend = (p.g + 1) * a.Dg;
    p.row0 = (long long)p.b * a.row_len;
    p.t0 = p.row0 + (long long)p.s * a.L;
    const long long e = p.row0 + a.row_len;
    p.t1 = p.t0 + a.L < e ? p.t0 + a.L : e;
    return p;
}

// State at the start of segment s (token t0, inside a sequence that began at s_beg
// before t0): the map of the segment that holds s_beg already starts from that
// sequence's initial state; the maps after it are applied in order.
template <int R>
__device__ __forceinline__ void state_before(float (&h)[R], const SArgs& a, const Place& p, long long s_beg, int d,
                                             int n0, const float (&A2)[R]) {
    const int sb = int((s_beg - p.row0) / a.L);
    const long long base = (long long)p.b * a.S;
    load_h<R>(h, a.seg_h + ((base + sb) * a.D + d) * a.N, n0, a.N);
    for (int i = sb + 1; i < p.s; ++i) {
        float e[R];
        load_h<R>(e, a.seg_h + ((base + i) * a.D + d) * a.N, n0, a.N);
        const float sd = a.seg_d[(base + i) * a.D + d];
#pragma unroll
        for (int r = 0; r < R; ++r) h[r] = ex2(A2[r] * sd) * h[r] + e[r];
    }
}

// kOut false: the map of a segment (end state from zero, sum of D).  kOut true: outputs.
template <typename T, int R, bool kVec, bool kOut>
__global__ void __launch_bounds__(128) fwd_kernel(const SArgs a, bool bc_vec) {
    __shared__ __align__(16) float2 sdu[2][kTT][kCh];
    __shared__ __align__(16) float sb[2][kTT][4 * R];
    __shared__ __align__(16) float sc[kOut ? 2 : 1][kOut ? kTT : 1][4 * R];
    __shared__ __align__(16) float sy[kOut ? kTT : 1][kYP];
    __shared__ float sbias[kCh], sskip[kCh];
    __shared__ int sfirst[kTT], slast[kTT];

    const int tid = threadIdx.x, q = tid & 3, c = tid >> 2;  // quad lane and channel; also: vector and token
    Place p = place(a);
    const int d = p.d0 + c, n0 = q * R;
    const bool live = d < p.dend;
    if (!kOut) {  // only what the segment after this one needs
        if (p.s == a.S - 1) return;
        const int n = seq_of(a.cu, a.nseq, a.seq_len, int(p.t1 - 1));
        const long long sbeg = seq_begin(a.cu, a.seq_len, n);
        if (sbeg > p.t0) p.t0 = sbeg;
    }
    float A2[R], h[R], dsum = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        A2[r] = live && n0 + r < a.N ? a.A[(size_t)d * a.N + n0 + r] * kLog2e : 0.f;
        h[r] = 0.f;
    }
    if (tid < kCh) {
        const int e = p.d0 + tid;
        sbias[tid] = a.bias && e < p.dend ? a.bias[e] : 0.f;
        sskip[tid] = a.skip && e < p.dend ? a.skip[e] : 0.f;
    }
    if (kOut && a.hT)  // empty sequences hand their initial state on
        for (int n = blockIdx.y; n < a.nseq; n += gridDim.y)
            if (live && seq_begin(a.cu, a.seq_len, n) == seq_begin(a.cu, a.seq_len, n + 1)) {
                float e[R];
#pragma unroll
                for (int r = 0; r < R; ++r) e[r] = 0.f;
                if (a.h0) load_h<R>(e, a.h0 + ((size_t)n * a.D + d) * a.N, n0, a.N);
                store_h<R>(e, a.hT + ((size_t)n * a.D + d) * a.N, n0, a.N);
            }
    if (p.t0 >= p.t1) return;
    int n = seq_of(a.cu, a.nseq, a.seq_len, int(p.t0));
    long long s_beg = seq_begin(a.cu, a.seq_len, n), s_end = seq_begin(a.cu, a.seq_len, n + 1);
    if (live) {
        if (kOut && s_beg < p.t0) state_before<R>(h, a, p, s_beg, d, n0, A2);
        else if (!kOut && s_beg == p.t0 && a.h0) load_h<R>(h, a.h0 + ((size_t)n * a.D + d) * a.N, n0, a.N);
    }

    // this thread's part of a tile: token c of the tile, channels d0 + 8 q .., states n0 ..
    const int dv = p.d0 + 8 * q, valid = p.dend - dv;
    V8<T> ru, rd, rz;
    VR<T, R> rb, rc;
    auto request = [&](long long tt) {
        const long long t = tt + c;
        if (t < p.t1) {
            load8<T, kVec>(ru, a.u, t, a.ldu, dv, valid);
            load8<T, kVec>(rd, a.dt, t, a.lddt, dv, valid);
            load_states<T, R>(rb, a.Bm, t * a.ldb + (long long)p.g * a.N, n0, a.N, bc_vec);
            if constexpr (kOut) {
                load_states<T, R>(rc, a.Cm, t * a.ldc + (long long)p.g * a.N, n0, a.N, bc_vec);
                if (a.z) load8<T, kVec>(rz, a.z, t, a.ldz, dv, valid);
            }
        }
    };
    request(p.t0);
    __syncthreads();  // sbias and sskip
    int buf = 0;
    for (long long tt = p.t0; tt < p.t1; tt += kTT, buf ^= 1) {
        const long long t = tt + c;
        const bool here = t < p.t1;
        // sequence starts and ends inside the tile
        const bool edges = kOut && !(s_beg < tt && s_end > tt + kTT);
        if (edges && q == 0) {
            int f = -1, l = -1;
            if (here) {
                const int m = seq_of(a.cu, a.nseq, a.seq_len, int(t));
                if (seq_begin(a.cu, a.seq_len, m) == t) f = m;
                if (seq_begin(a.cu, a.seq_len, m + 1) == t + 1) l = m;
            }
            sfirst[c] = f;
            slast[c] = l;
        }
        float u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // tokens past the end: D = 0, the state stays
            u[i] = here ? to_f32<T>(ru.v[i]) : 0.f;
            const float D = here ? step_size(to_f32<T>(rd.v[i]) + sbias[8 * q + i], a.softplus) : 0.f;
            sdu[buf][c][8 * q + i] = make_float2(D, D * u[i]);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            sb[buf][c][n0 + r] = here ? to_f32<T>(rb.v[r]) : 0.f;
            if constexpr (kOut) sc[buf][c][n0 + r] = here ? to_f32<T>(rc.v[r]) : 0.f;
        }
        V8<T> z = rz;
        __syncthreads();
        if (tt + kTT < p.t1) request(tt + kTT);
        const int steps = int(p.t1 - tt < kTT ? p.t1 - tt : kTT);
#pragma unroll 2
        for (int j4 = 0; j4 < steps; j4 += 4) {
            float acc[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = j4 + j;
                if (edges && sfirst[k] >= 0) {
#pragma unroll
                    for (int r = 0; r < R; ++r) h[r] = 0.f;
                    if (a.h0 && live) load_h<R>(h, a.h0 + ((size_t)sfirst[k] * a.D + d) * a.N, n0, a.N);
                }
                const float2 du = sdu[buf][k][c];
                acc[j] = 0.f;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    h[r] = ex2(du.x * A2[r]) * h[r] + du.y * sb[buf][k][n0 + r];
                    if constexpr (kOut) acc[j] += h[r] * sc[buf][k][n0 + r];
                }
                if (!kOut) dsum += du.x;
                if (edges && slast[k] >= 0 && a.hT && live)
                    store_h<R>(h, a.hT + ((size_t)slast[k] * a.D + d) * a.N, n0, a.N);
            }
            if constexpr (kOut) sy[j4 + q][c] = quad_transpose_sum(acc, q);
        }
        if constexpr (kOut) {
            __syncthreads();
            if (here) {
                float o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    o[i] = sy[c][8 * q + i] + sskip[8 * q + i] * u[i];
                    if (a.z) {
                        const float g = to_f32<T>(z.v[i]);
                        o[i] *= __fdividef(g, 1.f + __expf(-g));
                    }
                }
                store8<T, kVec>(a.y, t, a.ldy, dv, valid, o);
            }
            if (s_end <= tt + kTT && tt + kTT < p.t1) {
                n = seq_of(a.cu, a.nseq, a.seq_len, int(tt + kTT));
                s_beg = seq_begin(a.cu, a.seq_len, n);
                s_end = seq_begin(a.cu, a.seq_len, n + 1);
            }
        }
    }
    if (!kOut && live) {
        const long long i = (long long)p.b * a.S + p.s;
        store_h<R>(h, a.seg_h + (i * a.D + d) * a.N, n0, a.N);
        if (q == 0) a.seg_d[i * a.D + d] = dsum;
    }
}

// One token per sequence, the state in place.  Bound by HBM: the state is read and
// written once.  A quad of lanes holds one channel's states.
template <typename T, int R, bool kFull>
__global__ void __launch_bounds__(256) step_kernel(const SArgs a, float* __restrict__ state) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    const int q = int(i & 3), n0 = q * R;
    const long long cd = i >> 2;
    const bool live = cd < (long long)a.rows * a.D;
    const int d = live ? int(cd % a.D) : 0;
    const long long b = live ? cd / a.D : 0;
    const int g = d / a.Dg;
    float* hp = state + (size_t)(b * a.D + d) * a.N;
    float h[R], A[R];
    if constexpr (kFull) {
        const VR<float, R> hv = *reinterpret_cast<const VR<float, R>*>(hp + n0);
        const VR<float, R> av = *reinterpret_cast<const VR<float, R>*>(a.A + (size_t)d * a.N + n0);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            h[r] = hv.v[r];
            A[r] = av.v[r];
        }
    } else {
        load_h<R>(h, hp, n0, a.N);
        load_h<R>(A, a.A + (size_t)d * a.N, n0, a.N);
    }
    const float u = to_f32<T>(static_cast<const T*>(a.u)[b * a.ldu + d]);
    const float D = step_size(to_f32<T>(static_cast<const T*>(a.dt)[b * a.lddt + d]) + (a.bias ? a.bias[d] : 0.f),
                              a.softplus);
    const T* Bp = static_cast<const T*>(a.Bm) + b * a.ldb + (long long)g * a.N;
    const T* Cp = static_cast<const T*>(a.Cm) + b * a.ldc + (long long)g * a.N;
    float y = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const bool in = kFull || n0 + r < a.N;
        const float Bv = in ? to_f32<T>(Bp[n0 + r]) : 0.f, Cv = in ? to_f32<T>(Cp[n0 + r]) : 0.f;
        h[r] = ex2(D * A[r] * kLog2e) * h[r] + D * u * Bv;
        y += h[r] * Cv;
    }
    y += __shfl_xor_sync(0xffffffffu, y, 1);
    y += __shfl_xor_sync(0xffffffffu, y, 2);
    if (!live) return;
    if constexpr (kFull) {
        VR<float, R> hv;
#pragma unroll
        for (int r = 0; r < R; ++r) hv.v[r] = h[r];
        *reinterpret_cast<VR<float, R>*>(hp + n0) = hv;
    } else {
        store_h<R>(h, hp, n0, a.N);
    }
    if (q == 0) {
        y += (a.skip ? a.skip[d] : 0.f) * u;
        if (a.z) {
            const float g2 = to_f32<T>(static_cast<const T*>(a.z)[b * a.ldz + d]);
            y *= __fdividef(g2, 1.f + __expf(-g2));
        }
        static_cast<T*>(a.y)[b * a.ldy + d] = from_f32<T>(y);
    }
}

// ---------------------------------------------------------------- host side
static int states_per_lane(int N) { return N <= 8 ? 2 : (N <= 16 ? 4 : 8); }

// Segments: enough blocks for the SMs, from segments long enough to pay for the map
// pass, in whole tiles.
struct Cut {
    int rows, row_len, bpg, L, S;
};
static Cut fwd_cut(int B, int T, int D, int G, bool packed) {
    Cut c{};
    c.rows = packed ? 1 : B;
    c.row_len = T;
    c.bpg = int(cdiv(D / G, kCh));
    const long long blocks = (long long)c.rows * G * c.bpg;
    const long long want = (long long)device_sm_count() * 4;
    long long S = blocks >= device_sm_count() ? 1 : cdiv(want, blocks);
    const long long most = T / 256 < 32 ? T / 256 : 32;
    if (S > most) S = most;
    if (S < 1) S = 1;
    c.L = int(cdiv(cdiv(T, S), kTT) * kTT);
    c.S = int(cdiv(T, c.L));
    return c;
}

static bool vec8_ok(const SArgs& a, int es, const void* const* ptrs, const long long* lds, int n) {
    if (a.Dg % 8) return false;
    for (int i = 0; i < n; ++i)
        if (ptrs[i] && (!al16(ptrs[i]) || (lds[i] * es) % 16)) return false;
    return true;
}
// B and C in whole vectors of R states.
static bool states_ok(const SArgs& a, int es, int R) {
    const int bytes = R * es < 16 ? R * es : 16;
    return a.N == 4 * R && reinterpret_cast<uintptr_t>(a.Bm) % bytes == 0 && reinterpret_cast<uintptr_t>(a.Cm) % bytes == 0 &&
           (a.ldb * es) % bytes == 0 && (a.ldc * es) % bytes == 0;
}

template <typename T, int R>
int fwd(const SArgs& a, cudaStream_t st) {
    const void* ptrs[] = {a.u, a.dt, a.z, a.y};
    const long long lds[] = {a.ldu, a.lddt, a.ldz, a.ldy};
    const bool vec = vec8_ok(a, sizeof(T), ptrs, lds, 4), bc = states_ok(a, sizeof(T), R);
    const dim3 grid(a.G * a.bpg, a.rows * a.S);
    if (a.S > 1) {
        if (vec) fwd_kernel<T, R, true, false><<<grid, 128, 0, st>>>(a, bc);
        else fwd_kernel<T, R, false, false><<<grid, 128, 0, st>>>(a, bc);
    }
    if (vec) fwd_kernel<T, R, true, true><<<grid, 128, 0, st>>>(a, bc);
    else fwd_kernel<T, R, false, true><<<grid, 128, 0, st>>>(a, bc);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

template <typename T, int R>
int step(const SArgs& a, float* state, cudaStream_t st) {
    const unsigned grid = unsigned(cdiv((long long)a.rows * a.D * 4, 256));
    if (a.N == 4 * R && al16(state) && al16(a.A)) step_kernel<T, R, true><<<grid, 256, 0, st>>>(a, state);
    else step_kernel<T, R, false><<<grid, 256, 0, st>>>(a, state);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace scan

#define KDA_SCAN_DISPATCH(N, CALL)                             \
    if (dtype == KDA_BF16) {                                   \
        using T = __nv_bfloat16;                               \
        if ((N) <= 8) { constexpr int R = 2; return CALL; }    \
        if ((N) <= 16) { constexpr int R = 4; return CALL; }   \
        constexpr int R = 8;                                   \
        return CALL;                                           \
    }                                                          \
    using T = float;                                           \
    if ((N) <= 8) { constexpr int R = 2; return CALL; }        \
    if ((N) <= 16) { constexpr int R = 4; return CALL; }       \
    constexpr int R = 8;                                       \
    return CALL;

static void scan_cut_args(scan::SArgs& a, const scan::Cut& c) {
    a.rows = c.rows;
    a.row_len = c.row_len;
    a.bpg = c.bpg;
    a.L = c.L;
    a.S = c.S;
}

size_t selective_scan_fwd_workspace_bytes(int B, int T, int D, int G, int N, bool packed) {
    const scan::Cut c = scan::fwd_cut(B, T, D, G, packed);
    if (c.S <= 1) return 0;
    return mix::up256(size_t(c.rows) * c.S * D * N * 4) + mix::up256(size_t(c.rows) * c.S * D * 4);
}

int launch_selective_scan_fwd(scan::SArgs a, int B, int tokens, int dtype, void* ws, cudaStream_t st) {
    const scan::Cut c = scan::fwd_cut(B, tokens, a.D, a.G, a.cu != nullptr);
    scan_cut_args(a, c);
    a.seg_h = static_cast<float*>(ws);
    a.seg_d = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + mix::up256(size_t(c.rows) * c.S * a.D * a.N * 4));
    KDA_SCAN_DISPATCH(a.N, (scan::fwd<T, R>(a, st)))
}

int launch_selective_scan_step(scan::SArgs a, float* state, int dtype, cudaStream_t st) {
    KDA_SCAN_DISPATCH(a.N, (scan::step<T, R>(a, state, st)))
}

}  // namespace kda
