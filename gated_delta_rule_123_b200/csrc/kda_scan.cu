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
// Layout.  A lane holds one channel with all its states, a warp 32 channels, and
// warps are independent blocks.  So the step size, its decays, the sum over the states
// and the gate of a (token, channel) stay in one lane, with no exchange between lanes;
// the N states are N independent chains, which hide each other's latency; and B and C
// are the same for the whole warp: one broadcast 16-byte read of shared memory serves
// four states of 32 channels.  (Four or eight lanes to a channel, for more warps from
// the same channels, measured 455 us at best at 8192 tokens x 4096 channels x 16 states
// where this layout takes 372: the exchange and the per-lane copies of D and D u made the
// shared-memory pipe and the instruction issue the bound.)  u, dt, z, B and C are
// copied a tile of 16 tokens ahead into shared memory by cp.async.
//
// Few sequences and channels do not fill the SMs, so the token axis is cut into
// segments: a first pass runs all but the last one's recurrence from a zero state (no
// y) and leaves the end state and sum(D) of each; since the decay over a segment is
// exp(A sum(D)), the second pass starts each segment from the states before it.
#include "kda_scan.cuh"

namespace kda {
namespace scan {

template <typename T, int NP, bool kOut>
struct FwdSmem {
    // this tile's and the next one's inputs
    T u[2][kFT][kCh], dt[2][kFT][kCh], z[kOut ? 2 : 1][kOut ? kFT : 1][kCh];
    T b[2][kFT][NP], c[kOut ? 2 : 1][kOut ? kFT : 1][NP];
    float bc[kFT][kOut ? 2 * NP : NP];  // this tile's B, then C, as fp32
    int first[kFT], last[kFT];
};

// kOut false: the map of a segment (end state from zero, sum of D).  kOut true: outputs.
template <typename T, int NP, int kCopy, bool kOut>
__global__ void __launch_bounds__(32, NP <= 16 ? 18 : 10) fwd_kernel(const SArgs a, bool bc_vec) {
    constexpr int kP = NP / 2;
    __shared__ __align__(128) FwdSmem<T, NP, kOut> sm;
    const int lane = threadIdx.x;
    Place p = place(a);
    const int d = p.d0 + lane, valid = p.dend - p.d0;
    const bool live = lane < valid;
    if (!kOut) {  // only what the segment after this one needs
        if (p.s == a.S - 1) return;
        const int n = seq_of(a.cu, a.nseq, a.seq_len, int(p.t1 - 1));
        const long long sbeg = seq_begin(a.cu, a.seq_len, n, a.ntok);
        if (sbeg > p.t0) p.t0 = sbeg;
    }
    f2 A2[kP], h[kP];
#pragma unroll
    for (int i = 0; i < kP; ++i) A2[i] = h[i] = 0ull;
    if (live) {
        load_pairs<NP>(A2, a.A + (size_t)d * a.N, a.N);
#pragma unroll
        for (int i = 0; i < kP; ++i) A2[i] = mul2(A2[i], dup2(kL2e));
    }
    const float bias = a.bias && live ? a.bias[d] : 0.f, skip = kOut && a.skip && live ? a.skip[d] : 0.f;
    const size_t at = (size_t)d * a.N, row = (size_t)a.D * a.N;  // of a [channels][N] state
    if (kOut && a.hT)  // empty sequences hand their initial state on
        for (int n = blockIdx.y; n < a.nseq; n += gridDim.y)
            if (live && seq_begin(a.cu, a.seq_len, n, a.ntok) == seq_begin(a.cu, a.seq_len, n + 1, a.ntok)) {
                f2 e[kP];
#pragma unroll
                for (int i = 0; i < kP; ++i) e[i] = 0ull;
                if (a.h0) load_pairs<NP>(e, a.h0 + n * row + at, a.N);
                store_pairs<NP>(e, a.hT + n * row + at, a.N);
            }
    if (p.t0 >= p.t1) return;
    int n = seq_of(a.cu, a.nseq, a.seq_len, int(p.t0));
    long long s_beg = seq_begin(a.cu, a.seq_len, n, a.ntok), s_end = seq_begin(a.cu, a.seq_len, n + 1, a.ntok);
    if (live && kOut && s_beg < p.t0) {
        // the state at t0: the map of the segment that holds the sequence's start begins
        // with that sequence's initial state; the maps after it are applied in order
        const long long base = (long long)p.b * a.S;
        const int sb = int((s_beg - p.row0) / a.L);
        chain_states<NP>(h, a, base + sb, base + p.s, d, A2);
    } else if (live && !kOut && s_beg == p.t0 && a.h0) {
        load_pairs<NP>(h, a.h0 + n * row + at, a.N);
    }

    float dsum = 0.f;
    int buf = 0;
    auto request = [&](long long tt, int w) {
        const int m = int(p.t1 - tt < kFT ? p.t1 - tt : kFT);
        stage_tile<T, kCopy>(sm.u[w], a.u, tt, m, a.ldu, p.d0, valid, lane);
        stage_tile<T, kCopy>(sm.dt[w], a.dt, tt, m, a.lddt, p.d0, valid, lane);
        stage_bc<T, NP>(sm.b[w], a.Bm, tt, m, a.ldb, (long long)p.g * a.N, a.N, bc_vec, lane);
        if constexpr (kOut) {
            stage_bc<T, NP>(sm.c[w], a.Cm, tt, m, a.ldc, (long long)p.g * a.N, a.N, bc_vec, lane);
            if (a.z) stage_tile<T, kCopy>(sm.z[w], a.z, tt, m, a.ldz, p.d0, valid, lane);
        }
        cp_async_commit();
    };
    request(p.t0, 0);
    for (long long tt = p.t0; tt < p.t1; tt += kFT, buf ^= 1) {
        const int steps = int(p.t1 - tt < kFT ? p.t1 - tt : kFT);
        // sequence starts and ends inside the tile
        const bool edges = kOut && !(s_beg < tt && s_end > tt + kFT);
        if (edges && lane < kFT) {
            int f = -1, l = -1;
            if (lane < steps) {
                const int m = seq_of(a.cu, a.nseq, a.seq_len, int(tt + lane));
                if (seq_begin(a.cu, a.seq_len, m, a.ntok) == tt + lane) f = m;
                if (seq_begin(a.cu, a.seq_len, m + 1, a.ntok) == tt + lane + 1) l = m;
            }
            sm.first[lane] = f;
            sm.last[lane] = l;
        }
        cp_async_wait0();
        __syncwarp();
        widen_rows<T, NP>(sm.bc, 0, sm.b[buf], lane);
        if constexpr (kOut) widen_rows<T, NP>(sm.bc, NP, sm.c[buf], lane);
        __syncwarp();
        if (tt + kFT < p.t1) request(tt + kFT, buf ^ 1);
        T* yp = kOut ? static_cast<T*>(a.y) + tt * a.ldy + d : nullptr;
        auto token = [&](int k) {
            float D = to_f32<T>(sm.dt[buf][k][lane]) + bias;
            if (a.softplus) D = softplus_poly(D);
            const float u = to_f32<T>(sm.u[buf][k][lane]);
            const f2 D2 = dup2(D), w2 = dup2(D * u);
            f2 s[2] = {0ull, 0ull};
#pragma unroll
            for (int i = 0; i < kP; i += 2) {
                const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(&sm.bc[k][2 * i]);
                float x0, x1, x2, x3;
                upk(mul2(D2, A2[i]), x0, x1);
                upk(mul2(D2, A2[i + 1]), x2, x3);
                h[i] = fma2(pk(ex2(x0), ex2(x1)), h[i], mul2(w2, b.x));
                h[i + 1] = fma2(pk(ex2(x2), ex2(x3)), h[i + 1], mul2(w2, b.y));
                if constexpr (kOut) {
                    const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(&sm.bc[k][NP + 2 * i]);
                    s[0] = fma2(h[i], c.x, s[0]);
                    s[1] = fma2(h[i + 1], c.y, s[1]);
                }
            }
            if constexpr (kOut) {
                const f2 t = add2(s[0], s[1]);
                float y = (lo2(t) + hi2(t)) + skip * u;
                if (a.z) y *= siluf(to_f32<T>(sm.z[buf][k][lane]));
                if (live) yp[k * a.ldy] = from_f32<T>(y);
            } else {
                dsum += D;
            }
        };
        if (!edges) {  // (tests for edges between the tokens would keep their loads and exponentials from overlapping)
            int k = 0;
#pragma unroll 1
            for (; k + 4 <= steps; k += 4) {
#pragma unroll
                for (int j = 0; j < 4; ++j) token(k + j);
            }
#pragma unroll 1
            for (; k < steps; ++k) token(k);
        } else {
#pragma unroll 1
            for (int k = 0; k < steps; ++k) {
                if (sm.first[k] >= 0) {
#pragma unroll
                    for (int i = 0; i < kP; ++i) h[i] = 0ull;
                    if (a.h0 && live) load_pairs<NP>(h, a.h0 + sm.first[k] * row + at, a.N);
                }
                token(k);
                if (sm.last[k] >= 0 && a.hT && live) store_pairs<NP>(h, a.hT + sm.last[k] * row + at, a.N);
            }
        }
        if (kOut && s_end <= tt + kFT && tt + kFT < p.t1) {
            n = seq_of(a.cu, a.nseq, a.seq_len, int(tt + kFT));
            s_beg = seq_begin(a.cu, a.seq_len, n, a.ntok);
            s_end = seq_begin(a.cu, a.seq_len, n + 1, a.ntok);
        }
        __syncwarp();
    }
    if (!kOut && live) {
        const long long i = (long long)p.b * a.S + p.s;
        store_pairs<NP>(h, a.seg_h + i * row + at, a.N);
        a.seg_d[i * a.D + d] = dsum;
    }
}

// One token per sequence, the state in place.  Bound by HBM: the state is read and
// written once.  A quad of lanes holds one channel, R states a lane, for one sequence.
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
#pragma unroll
        for (int r = 0; r < R; ++r) h[r] = hv.v[r];
    } else {
        load_h<R>(h, hp, n0, a.N);
    }
    load_h<R>(A, a.A + (size_t)d * a.N, n0, a.N);
    VR<T, R> B, C;
    load_states<T, R>(B, a.Bm, b * a.ldb + (long long)g * a.N, n0, a.N, kFull);
    load_states<T, R>(C, a.Cm, b * a.ldc + (long long)g * a.N, n0, a.N, kFull);
    const float u = to_f32<T>(static_cast<const T*>(a.u)[b * a.ldu + d]);
    const float D = step_size(to_f32<T>(static_cast<const T*>(a.dt)[b * a.lddt + d]) + (a.bias ? a.bias[d] : 0.f),
                              a.softplus);
    float y = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        h[r] = ex2(D * A[r] * kL2e) * h[r] + D * u * to_f32<T>(B.v[r]);
        y += h[r] * to_f32<T>(C.v[r]);
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
        if (a.z) y *= siluf(to_f32<T>(static_cast<const T*>(a.z)[b * a.ldz + d]));
        static_cast<T*>(a.y)[b * a.ldy + d] = from_f32<T>(y);
    }
}

// The same for many sequences (whole 16-byte vectors of states): a thread keeps its
// channel's A, bias and skip and walks the sequences b0 .. b1, the next kRing states on
// their way into a ring that only it reads and the next sequence's other inputs in
// registers.  256 x 4096 x 16 bf16: 28 us = 5.1 TB/s (a thread per sequence: 42 us).
// Blocks an SM: what the registers (and, at 8 states a lane, the ring) allow without spilling.
__host__ __device__ constexpr int step_blocks(int R) { return R <= 4 ? 4 : 2; }
template <typename T, int R>
__global__ void __launch_bounds__(256, R <= 4 ? 4 : 2) step_many_kernel(const SArgs a, float* __restrict__ state, int per) {
    constexpr int kRing = 4;
    using V = VR<float, R>;
    __shared__ __align__(16) V ring[kRing][256];
    const int tid = threadIdx.x;
    const long long i = (long long)blockIdx.x * 256 + tid;
    const int q = int(i & 3), n0 = q * R;
    const bool live = (i >> 2) < a.D;
    const int d = live ? int(i >> 2) : a.D - 1;  // (lanes past the last channel repeat it and store nothing)
    const int g = d / a.Dg;
    const int b0 = blockIdx.y * per, b1 = min(a.rows, b0 + per);
    float A2[R];
    load_h<R>(A2, a.A + (size_t)d * a.N, n0, a.N);
#pragma unroll
    for (int r = 0; r < R; ++r) A2[r] *= kL2e;
    const float bias = a.bias ? a.bias[d] : 0.f, skip = a.skip ? a.skip[d] : 0.f;
    const size_t row = (size_t)a.D * a.N;
    float *ahead = state + b0 * row + (size_t)d * a.N + n0, *hp = ahead;  // the state to request next, and this one's
    int left = b1 - b0;  // states still to request
    auto request = [&](int slot) {
        if (left > 0) {
            constexpr int kB = sizeof(V) < 16 ? sizeof(V) : 16;
#pragma unroll
            for (int k = 0; k < int(sizeof(V)) / kB; ++k)
                cp_async<kB>(reinterpret_cast<uint8_t*>(&ring[slot][tid]) + kB * k, reinterpret_cast<uint8_t*>(ahead) + kB * k);
            ahead += row;
            --left;
        }
        cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < kRing - 1; ++k) request(k);
    // Four sequences at a time: each lane of a quad makes one's step size and finishes one's
    // output, so that the four lanes share that work.
    auto mine = [&](int b) { return min(b + q, b1 - 1); };
    T nu, ndt, nz = from_f32<T>(0.f);
    auto load = [&](int b) {
        const long long m = mine(b);
        nu = static_cast<const T*>(a.u)[m * a.ldu + d];
        ndt = static_cast<const T*>(a.dt)[m * a.lddt + d];
        if (a.z) nz = static_cast<const T*>(a.z)[m * a.ldz + d];
    };
    const T *pB = static_cast<const T*>(a.Bm) + b0 * a.ldb + (long long)g * a.N + n0;
    const T *pC = static_cast<const T*>(a.Cm) + b0 * a.ldc + (long long)g * a.N + n0;
    VR<T, R> nB, nC;  // of the next sequence
    auto load_bc = [&]() {
        nB = *reinterpret_cast<const VR<T, R>*>(pB);
        nC = *reinterpret_cast<const VR<T, R>*>(pC);
        pB += a.ldb;
        pC += a.ldc;
    };
    if (b0 < b1) {
        load(b0);
        load_bc();
    }
    for (int b = b0; b < b1; b += 4) {
        const float u = to_f32<T>(nu), z = to_f32<T>(nz);
        const float Dq = step_size(to_f32<T>(ndt) + bias, a.softplus), wq = Dq * u;
        if (b + 4 < b1) load(b + 4);
        float y = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (b + j >= b1) break;  // the same for the whole block
            const VR<T, R> B = nB, C = nC;
            if (b + j + 1 < b1) load_bc();
            cp_async_wait<kRing - 2>();
            V h = ring[j][tid];
            request((j + 3) & 3);  // into the place of the state before this one
            const float D = __shfl_sync(0xffffffffu, Dq, j, 4), w = __shfl_sync(0xffffffffu, wq, j, 4);
            float s = 0.f;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                h.v[r] = ex2(D * A2[r]) * h.v[r] + w * to_f32<T>(B.v[r]);
                s += h.v[r] * to_f32<T>(C.v[r]);
            }
            s += __shfl_xor_sync(0xffffffffu, s, 1);
            s += __shfl_xor_sync(0xffffffffu, s, 2);
            if (q == j) y = s;
            if (live) *reinterpret_cast<V*>(hp) = h;
            hp += row;
        }
        if (live && b + q < b1) {
            y += skip * u;
            if (a.z) y *= siluf(z);
            static_cast<T*>(a.y)[(long long)(b + q) * a.ldy + d] = from_f32<T>(y);
        }
    }
}

static Cut fwd_cut(int B, int T, int D, int G, bool packed) {
    Cut c{};
    c.rows = packed ? 1 : B;
    c.row_len = T;
    c.bpg = int(cdiv(D / G, kCh));
    // Unsegmented, 512 / 1024 warps take 450 / 300 us where segments take 360 (8192 x 4096
    // x 16); with segments, 28 warps an SM measured best (14: 430 us, 56: 370 us).
    const long long warps = (long long)c.rows * G * c.bpg, sms = device_sm_count();
    long long S = warps >= 5 * sms ? 1 : cdiv(28 * sms, warps);
    cut_row(c, S);
    return c;
}

template <typename T, int NP, int kCopy>
int fwd_run(const SArgs& a, bool bc, cudaStream_t st) {
    const dim3 grid(a.G * a.bpg, a.rows * a.S);
    if (a.S > 1) fwd_kernel<T, NP, kCopy, false><<<grid, 32, 0, st>>>(a, bc);
    fwd_kernel<T, NP, kCopy, true><<<grid, 32, 0, st>>>(a, bc);
    return cudaPeekAtLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
template <typename T, int NP>
int fwd_states(const SArgs& a, cudaStream_t st) {
    const void* ptrs[] = {a.u, a.dt, a.z};
    const long long lds[] = {a.ldu, a.lddt, a.ldz};
    const int copy = copy_bytes(a, sizeof(T), ptrs, lds, 3);
    const bool bc = bc_whole(a, sizeof(T));
    if (copy == 16) return fwd_run<T, NP, 16>(a, bc, st);
    return copy == 4 ? fwd_run<T, NP, 4>(a, bc, st) : fwd_run<T, NP, 0>(a, bc, st);
}
template <typename T>
int fwd(const SArgs& a, cudaStream_t st) {
    if (a.N <= 8) return fwd_states<T, 8>(a, st);
    return a.N <= 16 ? fwd_states<T, 16>(a, st) : fwd_states<T, 32>(a, st);
}

template <typename T, int R>
int step(const SArgs& a, float* state, cudaStream_t st) {
    const bool full = al16(state) && states_ok(a, sizeof(T), R);
    // the walking form in one wave of blocks; it needs several sequences a block
    const long long cols = cdiv((long long)a.D * 4, 256), fit = (long long)step_blocks(R) * device_sm_count() / cols, splits = fit > 1 ? fit : 1;
    if (full && a.rows >= 8 * splits) {
        const int per = int(cdiv(a.rows, splits));
        step_many_kernel<T, R><<<dim3(unsigned(cols), unsigned(cdiv(a.rows, per))), 256, 0, st>>>(a, state, per);
    } else {
        const unsigned grid = unsigned(cdiv((long long)a.rows * a.D * 4, 256));
        if (full) step_kernel<T, R, true><<<grid, 256, 0, st>>>(a, state);
        else step_kernel<T, R, false><<<grid, 256, 0, st>>>(a, state);
    }
    return cudaPeekAtLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
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

// Workspace of a segmented call: the segments' end states and sums, and a copy of the
// initial states for a call that updates them in place (one segment's block writes a
// sequence's final state while another's may still have to read its initial one).
struct ScanFwdPlan {
    scan::Cut c;
    size_t off_d, off_h0, total;
};
static ScanFwdPlan scan_fwd_plan(int B, int T, int D, int G, int N, int num_seqs) {
    ScanFwdPlan p{};
    p.c = scan::fwd_cut(B, T, D, G, num_seqs > 0);
    if (p.c.S <= 1) return p;
    const size_t segs = size_t(p.c.rows) * p.c.S, nseq = num_seqs > 0 ? num_seqs : B;
    p.off_d = mix::up256(segs * D * N * 4);
    p.off_h0 = p.off_d + mix::up256(segs * D * 4);
    p.total = p.off_h0 + mix::up256(nseq * D * N * 4);
    return p;
}
size_t selective_scan_fwd_workspace_bytes(int B, int T, int D, int G, int N, int num_seqs) {
    return scan_fwd_plan(B, T, D, G, N, num_seqs).total;
}

int launch_selective_scan_fwd(scan::SArgs a, int B, int tokens, int dtype, void* ws, cudaStream_t st) {
    const ScanFwdPlan p = scan_fwd_plan(B, tokens, a.D, a.G, a.N, a.cu ? a.nseq : 0);
    scan_cut_args(a, p.c);
    if (p.c.S > 1) {
        uint8_t* b = static_cast<uint8_t*>(ws);
        a.seg_h = reinterpret_cast<float*>(b);
        a.seg_d = reinterpret_cast<float*>(b + p.off_d);
        if (a.h0 && a.h0 == a.hT) {
            if (cudaMemcpyAsync(b + p.off_h0, a.h0, size_t(a.nseq) * a.D * a.N * 4, cudaMemcpyDeviceToDevice, st) != cudaSuccess)
                return KDA_ERR_CUDA;
            a.h0 = reinterpret_cast<const float*>(b + p.off_h0);
        }
    }
    return dtype == KDA_BF16 ? scan::fwd<__nv_bfloat16>(a, st) : scan::fwd<float>(a, st);
}

int launch_selective_scan_step(scan::SArgs a, float* state, int dtype, cudaStream_t st) {
    KDA_SCAN_DISPATCH(a.N, (scan::step<T, R>(a, state, st)))
}

}  // namespace kda
