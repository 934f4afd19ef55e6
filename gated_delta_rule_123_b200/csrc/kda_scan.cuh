// The selective scan's arguments and the parts that its passes share (kda_scan.cu,
// kda_scan_bwd.cu).
#pragma once

#include "kda_mixer.cuh"

namespace kda {
namespace scan {

using namespace mix;

constexpr int kTT = 32;   // tokens of a tile
constexpr int kCh = 32;   // channels of a block
constexpr int kYP = 40;   // row pitch of the backward pass's tiles of sums (a quad's four rows on different banks)

struct SArgs {
    const void *u, *dt, *z, *Bm, *Cm, *dy;
    const float *A, *skip, *bias, *h0;
    float* hT;
    void* y;
    const int32_t* cu;
    long long ldu, lddt, ldz, ldb, ldc, ldy, lddy;  // elements from token to token
    int nseq, seq_len, ntok;                        // sequences; dense: tokens of each; all tokens
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

__device__ __forceinline__ float step_size(float raw, int softplus) { return softplus ? softplus_poly(raw) : raw; }

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

// v[j] summed over L neighbouring lanes; lane q of them is left with the sum of v[q].
template <int L>
__device__ __forceinline__ float lane_transpose_sum(float (&v)[L], int q) {
#pragma unroll
    for (int s = L / 2; s >= 1; s /= 2)
#pragma unroll
        for (int i = 0; i < s; ++i) {
            const float keep = q & s ? v[s + i] : v[i], give = q & s ? v[i] : v[s + i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, s);
        }
    return v[0];
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

constexpr int kFT = 16;  // tokens of a tile in the forward pass

// A tile of 32 channels of rows [tt, tt + n) into shared memory, by asynchronous copies of
// kCopy bytes (16 or 4) or element by element (0); columns past `valid` are left as they
// were or 0.
template <typename T, int kCopy, int kTok>
__device__ __forceinline__ void stage_tile(T (&dst)[kTok][kCh], const void* base, long long tt, int n, long long ld, int d0,
                                           int valid, int lane) {
    const T* p = static_cast<const T*>(base) + tt * ld + d0;
    if constexpr (kCopy > 0) {
        constexpr int kE = kCopy / sizeof(T), kRow = kCh / kE;  // copies of a row
#pragma unroll
        for (int i = 0; i < kTok * kRow / 32; ++i) {
            const int k = (lane + 32 * i) / kRow, v = (lane + 32 * i) % kRow;
            if (k < n && v * kE < valid) cp_async<kCopy>(&dst[k][v * kE], p + k * ld + v * kE);
        }
    } else {
        T r[kTok];
#pragma unroll
        for (int k = 0; k < kTok; ++k) r[k] = k < n && lane < valid ? p[k * ld + lane] : from_f32<T>(0.f);
#pragma unroll
        for (int k = 0; k < kTok; ++k) dst[k][lane] = r[k];
    }
}
// The same for a group's NP states of B or C (states past N are 0).
template <typename T, int NP, int kTok>
__device__ __forceinline__ void stage_bc(T (&dst)[kTok][NP], const void* base, long long tt, int n, long long ld, long long off,
                                         int N, bool vec, int lane) {
    const T* p = static_cast<const T*>(base) + tt * ld + off;
    if (vec) {
        constexpr int kE = 16 / sizeof(T), kRow = NP / kE;
#pragma unroll
        for (int i = 0; i < (kTok * kRow + 31) / 32; ++i) {
            const int k = (lane + 32 * i) / kRow, v = (lane + 32 * i) % kRow;
            if (k < n) cp_async<16>(&dst[k][v * kE], p + k * ld + v * kE);
        }
    } else {
#pragma unroll 4
        for (int i = lane; i < kTok * NP; i += 32) {
            const int k = i / NP, m = i % NP;
            dst[k][m] = k < n && m < N ? p[k * ld + m] : from_f32<T>(0.f);
        }
    }
}

// B (and C) of a tile as fp32, 8 (bf16) or 4 values a step.
template <typename T, int NP, int kW, int kTok>
__device__ __forceinline__ void widen_rows(float (&dst)[kTok][kW], int col, const T (&src)[kTok][NP], int lane) {
    constexpr int kE = 16 / sizeof(T), kAll = kTok * NP / kE;
#pragma unroll
    for (int i = 0; i < (kAll + 31) / 32; ++i) {
        const int e = (lane + 32 * i) * kE, k = e / NP, m = e % NP;
        if (kAll % 32 == 0 || k < kTok) {
            float f[kE];
            unpack16(*reinterpret_cast<const uint4*>(&src[k][m]), f, T());
#pragma unroll
            for (int u = 0; u < kE; u += 4)
                *reinterpret_cast<float4*>(&dst[k][col + m + u]) = make_float4(f[u], f[u + 1], f[u + 2], f[u + 3]);
        }
    }
}

// All NP states of a channel, in pairs; states past N are 0.
template <int NP>
__device__ __forceinline__ void load_pairs(f2 (&h)[NP / 2], const float* p, int N) {
    if (N == NP && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
#pragma unroll
        for (int i = 0; i < NP / 4; ++i) {
            const float4 v = reinterpret_cast<const float4*>(p)[i];
            h[2 * i] = pk(v.x, v.y);
            h[2 * i + 1] = pk(v.z, v.w);
        }
    } else {
#pragma unroll
        for (int i = 0; i < NP / 2; ++i) h[i] = pk(2 * i < N ? p[2 * i] : 0.f, 2 * i + 1 < N ? p[2 * i + 1] : 0.f);
    }
}
template <int NP>
__device__ __forceinline__ void store_pairs(const f2 (&h)[NP / 2], float* p, int N) {
    if (N == NP && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
#pragma unroll
        for (int i = 0; i < NP / 4; ++i) {
            float4 v;
            upk(h[2 * i], v.x, v.y);
            upk(h[2 * i + 1], v.z, v.w);
            reinterpret_cast<float4*>(p)[i] = v;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NP / 2; ++i) {
            float a, b;
            upk(h[i], a, b);
            if (2 * i < N) p[2 * i] = a;
            if (2 * i + 1 < N) p[2 * i + 1] = b;
        }
    }
}

// 2^(A2 x), a pair.
__device__ __forceinline__ f2 decay(f2 A2, f2 x) {
    float x0, x1;
    upk(mul2(A2, x), x0, x1);
    return pk(ex2(x0), ex2(x1));
}
// The state after segment `first` (its own end state) and the maps of the segments up to
// `last`, the next one's map on its way while one is applied.
template <int NP>
__device__ __forceinline__ void chain_states(f2 (&h)[NP / 2], const SArgs& a, long long first, long long last, int d,
                                             const f2 (&A2)[NP / 2]) {
    constexpr int kP = NP / 2;
    const size_t row = (size_t)a.D * a.N, at = (size_t)d * a.N;
    load_pairs<NP>(h, a.seg_h + first * row + at, a.N);
    f2 next[kP];
    float nsd = 0.f;
    if (first + 1 < last) {
        load_pairs<NP>(next, a.seg_h + (first + 1) * row + at, a.N);
        nsd = a.seg_d[(first + 1) * a.D + d];
    }
    for (long long i = first + 1; i < last; ++i) {
        f2 e[kP];
#pragma unroll
        for (int k = 0; k < kP; ++k) e[k] = next[k];
        const f2 sd = dup2(nsd);
        if (i + 1 < last) {
            load_pairs<NP>(next, a.seg_h + (i + 1) * row + at, a.N);
            nsd = a.seg_d[(i + 1) * a.D + d];
        }
#pragma unroll
        for (int k = 0; k < kP; ++k) h[k] = fma2(decay(A2[k], sd), h[k], e[k]);
    }
}

// ---------------------------------------------------------------- host side
// How the tokens are cut: segments of L tokens, S per row.
struct Cut {
    int rows, row_len, bpg, L, S;
};
// Segments of whole tiles of 16 tokens, S per row as far as there are tiles.  A warp
// alone takes about 0.27 us a token and 0.15 us a segment before its own, so few channels
// are cut down to one tile, and no row into more than 256.
inline void cut_row(Cut& c, long long S) {
    const long long tiles = cdiv(c.row_len, 16);
    if (S > tiles) S = tiles;
    if (S > 256) S = 256;
    if (S < 1) S = 1;
    c.L = int(cdiv(tiles, S) * 16);
    c.S = int(cdiv(c.row_len, c.L));
}

inline bool vec8_ok(const SArgs& a, int es, const void* const* ptrs, const long long* lds, int n) {
    if (a.Dg % 8) return false;
    for (int i = 0; i < n; ++i)
        if (ptrs[i] && (!al16(ptrs[i]) || (lds[i] * es) % 16)) return false;
    return true;
}
// Bytes that the inputs' rows and groups can be copied by: 16, 4 or (0) single elements.
inline int copy_bytes(const SArgs& a, int es, const void* const* ptrs, const long long* lds, int n) {
    if (vec8_ok(a, es, ptrs, lds, n)) return 16;
    if ((a.Dg * es) % 4) return 0;
    for (int i = 0; i < n; ++i)
        if (ptrs[i] && (reinterpret_cast<uintptr_t>(ptrs[i]) % 4 || (lds[i] * es) % 4)) return 0;
    return 4;
}
inline int padded_states(int N) { return N <= 8 ? 8 : (N <= 16 ? 16 : 32); }
// B and C by 16-byte vectors: N is what a lane is padded to, and every group's row is aligned.
inline bool bc_whole(const SArgs& a, int es) {
    return a.N == padded_states(a.N) && al16(a.Bm) && al16(a.Cm) && (a.ldb * es) % 16 == 0 && (a.ldc * es) % 16 == 0;
}
// B and C in whole vectors of n states.
inline bool states_ok(const SArgs& a, int es, int n) {
    const int bytes = n * es < 16 ? n * es : 16;
    return a.N == 4 * n && reinterpret_cast<uintptr_t>(a.Bm) % bytes == 0 && reinterpret_cast<uintptr_t>(a.Cm) % bytes == 0 &&
           (a.ldb * es) % bytes == 0 && (a.ldc * es) % bytes == 0;
}

struct BwdOut {
    void *dB, *dC;
    long long lddb, lddc;
    float *dA, *dskip, *dbias;
};

}  // namespace scan

inline void scan_cut_args(scan::SArgs& a, const scan::Cut& c) {
    a.rows = c.rows;
    a.row_len = c.row_len;
    a.bpg = c.bpg;
    a.L = c.L;
    a.S = c.S;
}

size_t selective_scan_fwd_workspace_bytes(int B, int T, int D, int G, int N, int num_seqs);
int launch_selective_scan_fwd(scan::SArgs a, int B, int tokens, int dtype, void* ws, cudaStream_t st);
size_t selective_scan_bwd_workspace_bytes(int B, int T, int D, int G, int N, bool packed);
int launch_selective_scan_bwd(scan::SArgs a, const scan::BwdOut& o, int B, int tokens, int dtype, void* ws,
                              cudaStream_t st);
int launch_selective_scan_step(scan::SArgs a, float* state, int dtype, cudaStream_t st);

}  // namespace kda
