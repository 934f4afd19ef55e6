// Short causal depthwise convolution, the public form of the layer's ShortConv
// ("Kimi Linear: An Expressive, Efficient Attention Architecture", section "Neural
// Parameterization"), with a bias, gradients and a single-token step.
//
//   s_t = b + sum_j w_j x_{t-(W-1)+j},  y_t = SiLU(s_t) or s_t
//   with ds = dy SiLU'(s):  dx_t = sum_j w_j ds_{t+(W-1)-j},  dw_j = sum_t ds_t x_{t-(W-1)+j},  db = sum_t ds_t
//
// The inputs before a sequence's start come from its cache of W - 1 rows, oldest
// first, or are zero.  Dense batches and packed sequences are one axis of tokens,
// on which the window restarts at each sequence.  Bound by HBM: forward reads x
// and writes y, backward reads dy and x and writes dx.  A thread owns four
// channels (8 bytes of bf16, 16 of fp32) and slides over a run of tokens, so each row is read once
// but for the W - 1 rows next to the run.
#include "kda_mixer.cuh"

namespace kda {

namespace conv {

using namespace mix;

// Four channels of a row (8 bytes of bf16, 16 of fp32), or one.  (Eight bf16 channels a
// thread need twice the registers: half the warps, or more spills.)
template <typename T, bool kVec>
struct Row {
    static constexpr int kN = kVec ? 4 : 1;
    using type = typename std::conditional<kVec, typename std::conditional<sizeof(T) == 2, uint2, uint4>::type, T>::type;
    type v;
    __device__ __forceinline__ void load(const T* p) { v = *reinterpret_cast<const type*>(p); }
    __device__ __forceinline__ void load_stream(const T* p) { v = __ldcs(reinterpret_cast<const type*>(p)); }
    __device__ __forceinline__ void zero() {
        if constexpr (!kVec) v = from_f32<T>(0.f);
        else if constexpr (sizeof(T) == 2) v = make_uint2(0, 0);
        else v = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void get(float* f) const {
        if constexpr (!kVec) {
            f[0] = to_f32<T>(v);
        } else if constexpr (sizeof(T) == 2) {
            f[0] = __uint_as_float(v.x << 16);
            f[1] = __uint_as_float(v.x & 0xffff0000u);
            f[2] = __uint_as_float(v.y << 16);
            f[3] = __uint_as_float(v.y & 0xffff0000u);
        } else {
            unpack16(v, f, 0.f);
        }
    }
    __device__ __forceinline__ void set(const float* f) {
        if constexpr (!kVec) v = from_f32<T>(f[0]);
        else if constexpr (sizeof(T) == 2) v = make_uint2(pack2_rn(f[0], f[1]), pack2_rn(f[2], f[3]));
        else v = pack16(f, 0.f);
    }
    __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<type*>(p) = v; }
};

// Rows in flight a thread, blocks an SM: chosen for bf16, whose width 4 spills 16 bytes a
// thread; fp32 rows are twice as wide and spill 192 bytes at width 4 and 60 at width 3.
constexpr int kFwdRing = 10, kFwdBlocks = 5;

struct Args {
    const void *x, *w, *cache_in;
    const float* bias;
    void *y, *cache_out;
    const int32_t* cu;
    long long ldx, ldy;
    int nseq, seq_len, ntok, C, silu;
    // backward
    const void *dy, *dcache_out;
    void *dx, *dcache_in;
    float* part;
    long long lddy, lddx;
};

// Row j (0 oldest) of the cache that sequence [s0, e0) leaves: taken from its own
// tokens, and for a sequence shorter than W - 1 from its old cache.
template <typename T, int W>
__device__ void tail_rows(const Args& a, long long i0, long long step) {
    const T* x = static_cast<const T*>(a.x);
    const T* in = static_cast<const T*>(a.cache_in);
    T* out = static_cast<T*>(a.cache_out);
    const long long total = (long long)a.nseq * a.C;
    for (long long i = i0; i < total; i += step) {
        const int n = int(i / a.C), c = int(i % a.C);
        const int s0 = seq_begin(a.cu, a.seq_len, n, a.ntok), e0 = seq_begin(a.cu, a.seq_len, n + 1, a.ntok);
        T r[W - 1];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const int p = e0 - (W - 1) + j;
            r[j] = p >= s0 ? x[(long long)p * a.ldx + c]
                           : (in ? in[((size_t)n * (W - 1) + max(0, W - 1 + p - s0)) * a.C + c] : from_f32<T>(0.f));
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j) out[((size_t)n * (W - 1) + j) * a.C + c] = r[j];
    }
}

template <typename T, int W>
__global__ void __launch_bounds__(256) tail_kernel(const Args a) {
    tail_rows<T, W>(a, (long long)blockIdx.x * 256 + threadIdx.x, (long long)gridDim.x * 256);
}

// The taps of a thread's channels: w[u][j], j = 0 the oldest.
template <typename T, int W, int kE>
__device__ __forceinline__ void load_taps(const T* w, int c0, float (&f)[kE][W]) {
    if constexpr (kE > 1 && W == 4) {  // four channels' taps: 32 or 64 bytes in a row
        constexpr int kP = int(16 / sizeof(T));
#pragma unroll
        for (int i = 0; i < kE * W / kP; ++i) {
            float t[kP];
            unpack16(reinterpret_cast<const uint4*>(w + (size_t)c0 * W)[i], t, T());
#pragma unroll
            for (int k = 0; k < kP; ++k) f[(i * kP + k) / W][(i * kP + k) % W] = t[k];
        }
    } else {
#pragma unroll
        for (int u = 0; u < kE; ++u)
#pragma unroll
            for (int j = 0; j < W; ++j) f[u][j] = to_f32<T>(w[(size_t)(c0 + u) * W + j]);
    }
}

// A thread: a vector of channels by a run of tokens (neighbouring threads, neighbouring
// vectors; narrow channels put several runs into a block).  It keeps kRing rows in flight: each row's register is requested again, kRing
// tokens ahead, as soon as its value has been used.
template <typename T, int W, bool kVec, int kRing>
__global__ void __launch_bounds__(128, kFwdBlocks) fwd_kernel(const Args a, int run) {
    constexpr int kE = Row<T, kVec>::kN, kP = kE > 1 ? kE / 2 : 1;
    const long long id = (long long)blockIdx.x * 128 + threadIdx.x;
    const int nvec = a.C / kE, at = int(id / nvec), c0 = int(id % nvec) * kE;
    if ((long long)at * run >= a.ntok) return;
    const T* x = static_cast<const T*>(a.x) + c0;
    T* y = static_cast<T*>(a.y) + c0;
    const T* in = static_cast<const T*>(a.cache_in);
    const int t0 = at * run, t1 = run < a.ntok - t0 ? t0 + run : a.ntok;  // (t0 + run may pass 2^31)
    Row<T, kVec> ring[kRing];
#pragma unroll
    for (int j = 0; j < kRing; ++j)
        if (t0 + j < t1) ring[j].load_stream(x + (long long)(t0 + j) * a.ldx);
    // channels in pairs (one channel on its own in the scalar form)
    f2 w[W][kP], b[kP], h[W - 1][kP];  // h: inputs at t-(W-1) .. t-1
    {
        float wf[kE][W];
        load_taps<T, W, kE>(static_cast<const T*>(a.w), c0, wf);
#pragma unroll
        for (int u = 0; u < kP; ++u) {
            constexpr int o = kE > 1 ? 1 : 0;
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][u] = pk(wf[2 * u * o][j], wf[2 * u * o + o][j]);
            b[u] = a.bias ? pk(a.bias[c0 + 2 * u * o], a.bias[c0 + 2 * u * o + o]) : 0ull;
        }
    }
    auto get2 = [](const Row<T, kVec>& r, f2 (&v)[kP]) {
        float f[kE];
        r.get(f);
#pragma unroll
        for (int u = 0; u < kP; ++u) v[u] = kE > 1 ? pk(f[2 * u], f[kE > 1 ? 2 * u + 1 : 0]) : pk(f[0], 0.f);
    };
    int n = seq_of(a.cu, a.nseq, a.seq_len, t0);
    int s_beg = seq_begin(a.cu, a.seq_len, n, a.ntok), s_end = seq_begin(a.cu, a.seq_len, n + 1, a.ntok);
    auto history = [&](int t) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const int p = t - (W - 1) + j;
            Row<T, kVec> r;
            if (p >= s_beg) r.load(x + (long long)p * a.ldx);
            else if (in) r.load(in + ((size_t)n * (W - 1) + max(0, W - 1 + p - s_beg)) * a.C + c0);
            else r.zero();
            get2(r, h[j]);
        }
    };
    history(t0);
    // the next row to request and the next one to store, stepped from token to token
    const T* ahead = x + (long long)(t0 + kRing) * a.ldx;
    T* out = y + (long long)t0 * a.ldy;
    auto token = [&](int i, int t) {
        f2 v[kP];
        get2(ring[i], v);
        if (t + kRing < t1) ring[i].load_stream(ahead);
        ahead += a.ldx;
        float o[kE];
#pragma unroll
        for (int u = 0; u < kP; ++u) {
            f2 s = b[u];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) s = fma2(w[j][u], h[j][u], s);
            s = fma2(w[W - 1][u], v[u], s);
            float s0, s1;
            upk(s, s0, s1);
            if (a.silu) {
                s0 = siluf(s0);
                if (kE > 1) s1 = siluf(s1);
            }
            o[kE > 1 ? 2 * u : 0] = s0;
            if constexpr (kE > 1) o[2 * u + 1] = s1;
#pragma unroll
            for (int j = 0; j + 1 < W - 1; ++j) h[j][u] = h[j + 1][u];
            h[W - 2][u] = v[u];
        }
        Row<T, kVec> r;
        r.set(o);
        r.store(out);
        out += a.ldy;
    };
    for (int tb = t0; tb < t1; tb += kRing) {
        if (s_end >= tb + kRing && t1 >= tb + kRing && tb < s_end) {  // no edge in the ring: the window moves by renaming registers
#pragma unroll
            for (int i = 0; i < kRing; ++i) token(i, tb + i);
            continue;
        }
#pragma unroll
        for (int i = 0; i < kRing; ++i) {
            const int t = tb + i;
            if (t >= t1) break;
            if (t >= s_end) {  // a new sequence starts at t (empty ones are skipped)
                while (t >= s_end && n + 1 < a.nseq) {
                    ++n;
                    s_beg = s_end;
                    s_end = seq_begin(a.cu, a.seq_len, n + 1, a.ntok);
                }
                history(t);
            }
            token(i, t);
        }
    }
}

// d SiLU(s) / ds, finite for every finite s (sigmoid(s) (1 + s (1 - sigmoid(s)))).
__device__ __forceinline__ float dsilu(float s) {
    const float g = sigmoidf(s);
    return g * (1.f + s * (1.f - g));
}

// Blocks of the backward pass that an SM's registers hold.
__host__ __device__ constexpr int bwd_blocks(int kE) { return kE == 4 ? 3 : 8; }

// Backward.  A thread slides over its run of tokens and W - 1 more: ds of a
// token is formed once its window is complete, and the token W - 1 back then has
// its whole gradient.  The run's sums for dw and db stay in registers and are
// written as partial sums [run][W + 1][C].
template <typename T, int W, bool kVec>
__global__ void __launch_bounds__(128, bwd_blocks(Row<T, kVec>::kN))
    bwd_kernel(const Args a, int run) {
    constexpr int kE = Row<T, kVec>::kN;
    const long long id = (long long)blockIdx.x * 128 + threadIdx.x;
    const int nvec = a.C / kE, at = int(id / nvec), c0 = int(id % nvec) * kE;
    if ((long long)at * run >= a.ntok) return;
    const T* x = static_cast<const T*>(a.x) + c0;
    const T* dy = static_cast<const T*>(a.dy) + c0;
    T* dx = static_cast<T*>(a.dx) + c0;
    const T* in = static_cast<const T*>(a.cache_in);
    const T* dout = static_cast<const T*>(a.dcache_out);
    const int t0 = at * run, t1 = run < a.ntok - t0 ? t0 + run : a.ntok;  // (t0 + run may pass 2^31)
    float w[kE][W], b[kE], aw[W][kE], ab[kE];
    load_taps<T, W, kE>(static_cast<const T*>(a.w), c0, w);
#pragma unroll
    for (int u = 0; u < kE; ++u) {
        b[u] = a.bias ? a.bias[c0 + u] : 0.f;
        ab[u] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) aw[j][u] = 0.f;
    }
    int n = seq_of(a.cu, a.nseq, a.seq_len, t0);
    int s_beg = seq_begin(a.cu, a.seq_len, n, a.ntok), s_end = seq_begin(a.cu, a.seq_len, n + 1, a.ntok);
    float h[W - 1][kE];   // inputs at t-(W-1) .. t-1
    float g[W - 1][kE];   // gradients of the inputs at t-(W-1) .. t-1, as far as they are known
    auto history = [&](int t) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const int p = t - (W - 1) + j;
            Row<T, kVec> r;
            if (p >= s_beg) r.load(x + (long long)p * a.ldx);
            else if (in) r.load(in + ((size_t)n * (W - 1) + max(0, W - 1 + p - s_beg)) * a.C + c0);
            else r.zero();
            r.get(h[j]);
#pragma unroll
            for (int u = 0; u < kE; ++u) g[j][u] = 0.f;
        }
    };
    // the gradient of input p of the current sequence is complete: add what flows back
    // through the cache that the sequence leaves, and store it
    auto finish = [&](int p, const float* v) {
        if (p < s_beg || p < t0 || p >= t1) return;
        float f[kE];
#pragma unroll
        for (int u = 0; u < kE; ++u) f[u] = v[u];
        if (dout && p >= s_end - (W - 1) && p < s_end) {
            Row<T, kVec> r;
            float e[kE];
            r.load(dout + ((size_t)n * (W - 1) + (p - (s_end - (W - 1)))) * a.C + c0);
            r.get(e);
#pragma unroll
            for (int u = 0; u < kE; ++u) f[u] += e[u];
        }
        Row<T, kVec> r;
        r.set(f);
        r.store(dx + (long long)p * a.lddx);
    };
    history(t0);
    const int t2 = min(a.ntok, t1 + W - 1);
    constexpr int kRing = 4;  // rows in flight
    Row<T, kVec> nx[kRing], nd[kRing];
#pragma unroll
    for (int j = 0; j < kRing; ++j)
        if (t0 + j < t2) {
            nx[j].load(x + (long long)(t0 + j) * a.ldx);
            nd[j].load(dy + (long long)(t0 + j) * a.lddy);
        }
    bool done = false;  // the run's last sequence has ended before the extra tokens
    auto token = [&](int i, int t, auto whole) {
        float v[kE], d[kE], dn[kE];
        nx[i].get(v);
        nd[i].get(d);
        if (t + kRing < t2) {
            nx[i].load(x + (long long)(t + kRing) * a.ldx);
            nd[i].load(dy + (long long)(t + kRing) * a.lddy);
        }
        const bool mine = decltype(whole)::value || t < t1;  // the run's own tokens count for dw and db
#pragma unroll
        for (int u = 0; u < kE; ++u) {
            if (a.silu) {
                float s = b[u];
#pragma unroll
                for (int j = 0; j < W - 1; ++j) s += w[u][j] * h[j][u];
                s += w[u][W - 1] * v[u];
                d[u] *= dsilu(s);
            }
            if (mine) {
                ab[u] += d[u];
#pragma unroll
                for (int j = 0; j < W - 1; ++j) aw[j][u] += d[u] * h[j][u];
                aw[W - 1][u] += d[u] * v[u];
            }
#pragma unroll
            for (int j = 0; j < W - 1; ++j) g[j][u] += w[u][j] * d[u];
            dn[u] = w[u][W - 1] * d[u];
        }
        if constexpr (decltype(whole)::value) {  // token t - (W - 1) is the run's and inside the sequence
            Row<T, kVec> r;
            r.set(g[0]);
            r.store(dx + (long long)(t - (W - 1)) * a.lddx);
        } else {
            finish(t - (W - 1), g[0]);
        }
#pragma unroll
        for (int u = 0; u < kE; ++u) {
#pragma unroll
            for (int j = 0; j + 1 < W - 1; ++j) {
                h[j][u] = h[j + 1][u];
                g[j][u] = g[j + 1][u];
            }
            h[W - 2][u] = v[u];
            g[W - 2][u] = dn[u];
        }
    };
    for (int tb = t0; tb < t2 && !done; tb += kRing) {
        // inside one sequence and the run, with the W - 1 tokens before: the window moves by
        // renaming registers, and no token finished here reaches the sequence's last rows
        if (tb - (W - 1) >= s_beg && tb - (W - 1) >= t0 && tb + kRing <= s_end && tb + kRing <= t1) {
#pragma unroll
            for (int i = 0; i < kRing; ++i) token(i, tb + i, std::true_type{});
            continue;
        }
#pragma unroll
        for (int i = 0; i < kRing; ++i) {
            const int t = tb + i;
            if (t >= t2 || done) break;
            if (t >= s_end) {
                for (int j = 0; j < W - 1; ++j) finish(t - (W - 1) + j, g[j]);
                if (t >= t1) {
                    done = true;
                    break;
                }
                while (t >= s_end && n + 1 < a.nseq) {
                    ++n;
                    s_beg = s_end;
                    s_end = seq_begin(a.cu, a.seq_len, n + 1, a.ntok);
                }
                if (t < s_end) {
                    history(t);
                } else {  // rows behind the last offset: their window goes on, but the gradients before them are complete
                    s_beg = t;
                    s_end = 0x7fffffff;
#pragma unroll
                    for (int j = 0; j < W - 1; ++j)
#pragma unroll
                        for (int u = 0; u < kE; ++u) g[j][u] = 0.f;
                }
            }
            token(i, t, std::false_type{});
        }
    }
    if (t2 == a.ntok && !done)  // the axis ends here: the last inputs have no later token
        for (int j = 0; j < W - 1; ++j) finish(t2 - (W - 1) + j, g[j]);
    float* p = a.part + (size_t)at * (W + 1) * a.C + c0;
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
        for (int u = 0; u < kE; ++u) p[(size_t)j * a.C + u] = aw[j][u];
#pragma unroll
    for (int u = 0; u < kE; ++u) p[(size_t)W * a.C + u] = ab[u];
}

// Gradient of the incoming cache of sequence n, channel c: row r (position p = s0 - (W - 1)
// + r) fed the first tokens of its sequence, and a sequence shorter than W - 1 passes rows on.
template <typename T, int W>
__device__ void cache_gradient(const Args& a, int n, int c) {
    const T *x = static_cast<const T*>(a.x) + c, *dy = static_cast<const T*>(a.dy) + c;
    const T* in = static_cast<const T*>(a.cache_in);
    const T* dout = static_cast<const T*>(a.dcache_out);
    float w[W];
#pragma unroll
    for (int j = 0; j < W; ++j) w[j] = to_f32<T>(static_cast<const T*>(a.w)[(size_t)c * W + j]);
    const float b = a.bias ? a.bias[c] : 0.f;
    const int s0 = seq_begin(a.cu, a.seq_len, n, a.ntok), e0 = seq_begin(a.cu, a.seq_len, n + 1, a.ntok);
    float h[2 * W - 2], g[W - 1];  // inputs from position s0 - (W - 1) on; the cache's gradient
#pragma unroll
    for (int i = 0; i < 2 * W - 2; ++i) {
        if (i < W - 1) {
            h[i] = in ? to_f32<T>(in[((size_t)n * (W - 1) + i) * a.C + c]) : 0.f;
            g[i < W - 1 ? i : 0] = 0.f;
        } else {
            h[i] = s0 + i - (W - 1) < e0 ? to_f32<T>(x[(long long)(s0 + i - (W - 1)) * a.ldx]) : 0.f;
        }
    }
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {  // token s0 + k: its window is h[k .. k + W - 1]
        if (s0 + k < e0) {
            float d = to_f32<T>(dy[(long long)(s0 + k) * a.lddy]);
            if (a.silu) {
                float s = b;
#pragma unroll
                for (int j = 0; j < W; ++j) s += w[j] * h[k + j];
                d *= dsilu(s);
            }
#pragma unroll
            for (int j = 0; j < W; ++j)
                if (k + j < W - 1) g[k + j] += w[j] * d;
        }
    }
    if (dout) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const int p = e0 - (W - 1) + j;
            if (p < s0) {
                const float e = to_f32<T>(dout[((size_t)n * (W - 1) + j) * a.C + c]);
#pragma unroll
                for (int r = 0; r < W - 1; ++r)
                    if (r == W - 1 + p - s0) g[r] += e;
            }
        }
    }
#pragma unroll
    for (int r = 0; r < W - 1; ++r)
        static_cast<T*>(a.dcache_in)[((size_t)n * (W - 1) + r) * a.C + c] = from_f32<T>(g[r]);
}

// dw [C][W] and db [C] from the runs' partial sums [run][W + 1][C] (32 threads to a column,
// in a fixed order), and in the blocks after those the gradients of the incoming caches.
template <typename T, int W>
__global__ void __launch_bounds__(1024) bwd_finish_kernel(const Args a, int parts, T* __restrict__ dw,
                                                          float* __restrict__ db) {
    __shared__ float s[32][33];
    const int j = blockIdx.y;
    if (j > W) {
        const long long step = (long long)(gridDim.y - (W + 1)) * gridDim.x * 1024;
        for (long long i = ((long long)(j - (W + 1)) * gridDim.x + blockIdx.x) * 1024 + threadIdx.x;
             i < (long long)a.nseq * a.C; i += step)
            cache_gradient<T, W>(a, int(i / a.C), int(i % a.C));
        return;
    }
    const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    const size_t stride = (size_t)(W + 1) * a.C;
    float v = 0.f;
    if (c < a.C) {
        const float* q = a.part + (size_t)j * a.C + c;
#pragma unroll 8
        for (int p = row; p < parts; p += 32) v += q[p * stride];
    }
    s[row][lane] = v;
    __syncthreads();
    if (row == 0 && c < a.C) {
        float t = 0.f;
#pragma unroll
        for (int r = 0; r < 32; ++r) t += s[r][lane];
        if (j < W) {
            if (dw) dw[(size_t)c * W + j] = from_f32<T>(t);
        } else if (db) {
            db[c] = t;
        }
    }
}

// One token per sequence; the cache moves up one row in place.
template <typename T, int W, bool kVec>
__global__ void __launch_bounds__(128) step_kernel(const Args a, T* __restrict__ cache) {
    constexpr int kE = Row<T, kVec>::kN;
    const int nvec = a.C / kE;
    const long long i = (long long)blockIdx.x * 128 + threadIdx.x;
    if (i >= (long long)a.nseq * nvec) return;
    const int n = int(i / nvec), c0 = int(i % nvec) * kE;
    Row<T, kVec> h[W];
    T* cn = cache + (size_t)n * (W - 1) * a.C + c0;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) h[j].load(cn + (size_t)j * a.C);
    h[W - 1].load(static_cast<const T*>(a.x) + n * a.ldx + c0);
    float w[kE][W], s[kE];
    load_taps<T, W, kE>(static_cast<const T*>(a.w), c0, w);
#pragma unroll
    for (int u = 0; u < kE; ++u) s[u] = a.bias ? a.bias[c0 + u] : 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) {
        float v[kE];
        h[j].get(v);
#pragma unroll
        for (int u = 0; u < kE; ++u) s[u] += w[u][j] * v[u];
        if (j > 0) h[j].store(cn + (size_t)(j - 1) * a.C);
    }
    if (a.silu) {
#pragma unroll
        for (int u = 0; u < kE; ++u) s[u] = siluf(s[u]);
    }
    h[0].set(s);
    h[0].store(static_cast<T*>(a.y) + n * a.ldy + c0);
}


// Tokens of one thread in the forward pass: one wave of the blocks that the SMs hold
// (65536 x 4096 bf16 in 3.5 waves of shorter runs 224 us, in 7 waves 308 us, in one 194 us
// = 5.5 TB/s at best; other machines 223).
static int fwd_run(int ntok, int C, int kE) {
    const long long want = cdiv((long long)ntok * cdiv(C, kE), (long long)device_sm_count() * kFwdBlocks * 128);
    return int(want < 8 ? 8 : want);
}

// The same for the backward pass; long runs also write few partial sums, (W + 1) x 4 bytes
// per channel and run.
static int bwd_run(int ntok, int C, int kE) {
    const long long want = cdiv((long long)ntok * cdiv(C, kE), (long long)device_sm_count() * bwd_blocks(kE) * 128);
    return int(want < 8 ? 8 : want);
}

template <typename T, int W>
int fwd(const Args& a, bool vec, cudaStream_t st) {
    if (a.ntok > 0) {
        const int kE = vec ? 4 : 1;
        const int run = fwd_run(a.ntok, a.C, kE);
        const unsigned grid = unsigned(cdiv(cdiv(a.ntok, run) * (a.C / kE), 128));
        if (vec) fwd_kernel<T, W, true, kFwdRing><<<grid, 128, 0, st>>>(a, run);
        else fwd_kernel<T, W, false, kFwdRing><<<grid, 128, 0, st>>>(a, run);
    }
    if (a.cache_out) {  // after the main kernel on the stream, so cache_out may be cache_in
        const long long n = cdiv((long long)a.nseq * a.C, 256);
        tail_kernel<T, W><<<unsigned(n < 4096 ? n : 4096), 256, 0, st>>>(a);
    }
    return cudaPeekAtLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

template <typename T, int W>
int bwd(const Args& a, bool vec, void* dw, float* db, cudaStream_t st) {
    const int kE = vec ? 4 : 1;
    int parts = 0;
    if (a.ntok > 0) {
        const int run = bwd_run(a.ntok, a.C, kE);
        parts = int(cdiv(a.ntok, run));
        const unsigned grid = unsigned(cdiv((long long)parts * (a.C / kE), 128));
        if (vec) bwd_kernel<T, W, true><<<grid, 128, 0, st>>>(a, run);
        else bwd_kernel<T, W, false><<<grid, 128, 0, st>>>(a, run);
    }
    const unsigned cols = unsigned(cdiv(a.C, 32));
    long long more = a.dcache_in ? cdiv((long long)a.nseq * a.C, 1024ll * cols) : 0;
    if (more > 1024) more = 1024;
    if (dw || db || more)
        bwd_finish_kernel<T, W><<<dim3(cols, unsigned(W + 1 + more)), 1024, 0, st>>>(a, parts, static_cast<T*>(dw), db);
    return cudaPeekAtLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

template <typename T, int W>
int step(const Args& a, bool vec, void* cache, cudaStream_t st) {
    const int kE = vec ? 4 : 1;
    const unsigned grid = unsigned(cdiv((long long)a.nseq * (a.C / kE), 128));
    if (vec) step_kernel<T, W, true><<<grid, 128, 0, st>>>(a, static_cast<T*>(cache));
    else step_kernel<T, W, false><<<grid, 128, 0, st>>>(a, static_cast<T*>(cache));
    return cudaPeekAtLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace conv

size_t short_conv_bwd_workspace_bytes(int ntok, int C, int W) {
    // the shortest runs of any element type and alignment
    size_t parts = 0;
    for (int e = 1; e <= 4; e += 3) {
        const size_t p = size_t(mix::cdiv(ntok, conv::bwd_run(ntok, C, e)));
        if (p > parts) parts = p;
    }
    return mix::up256(parts * (W + 1) * C * sizeof(float));
}

// Four channels at a time: every row of every tensor starts on a boundary of four values
// (the taps on 16 bytes).
static bool short_conv_vec(int C, int dtype, const void* w, const void* const* ptrs, int np, const long long* lds, int nl) {
    const int bytes = dtype == KDA_BF16 ? 8 : 16;
    if (C % 4 || !mix::al16(w)) return false;
    for (int i = 0; i < np; ++i)
        if (reinterpret_cast<uintptr_t>(ptrs[i]) % bytes) return false;
    for (int i = 0; i < nl; ++i)
        if (lds[i] % 4) return false;
    return true;
}

#define KDA_CONV_DISPATCH(CALL)                                     \
    if (dtype == KDA_BF16) {                                        \
        using T = __nv_bfloat16;                                    \
        if (W == 2) { constexpr int kW = 2; return CALL; }          \
        if (W == 3) { constexpr int kW = 3; return CALL; }          \
        constexpr int kW = 4;                                       \
        return CALL;                                                \
    }                                                               \
    using T = float;                                                \
    if (W == 2) { constexpr int kW = 2; return CALL; }              \
    if (W == 3) { constexpr int kW = 3; return CALL; }              \
    constexpr int kW = 4;                                           \
    return CALL;

int launch_short_conv_fwd(const void* x, long long ldx, const void* w, const float* bias, void* y, long long ldy,
                          const void* cache_in, void* cache_out, const int32_t* cu, int nseq, int seq_len, int ntok,
                          int C, int W, int dtype, int silu, cudaStream_t st) {
    conv::Args a{};
    a.x = x; a.ldx = ldx; a.w = w; a.bias = bias; a.y = y; a.ldy = ldy;
    a.cache_in = cache_in; a.cache_out = cache_out;
    a.cu = cu; a.nseq = nseq; a.seq_len = seq_len; a.ntok = ntok; a.C = C; a.silu = silu;
    const void* ptrs[] = {x, y, cache_in, cache_out};
    const long long lds[] = {ldx, ldy};
    const bool vec = short_conv_vec(C, dtype, w, ptrs, 4, lds, 2);
    KDA_CONV_DISPATCH((conv::fwd<T, kW>(a, vec, st)))
}

int launch_short_conv_bwd(const void* dy, long long lddy, const void* x, long long ldx, const void* w,
                          const float* bias, const void* cache_in, const void* dcache_out, void* dx, long long lddx,
                          void* dw, float* db, void* dcache_in, const int32_t* cu, int nseq, int seq_len, int ntok,
                          int C, int W, int dtype, int silu, void* ws, cudaStream_t st) {
    conv::Args a{};
    a.x = x; a.ldx = ldx; a.w = w; a.bias = bias;
    a.cache_in = cache_in; a.dcache_out = dcache_out; a.dcache_in = dcache_in;
    a.dy = dy; a.lddy = lddy; a.dx = dx; a.lddx = lddx;
    a.part = static_cast<float*>(ws);
    a.cu = cu; a.nseq = nseq; a.seq_len = seq_len; a.ntok = ntok; a.C = C; a.silu = silu;
    const void* ptrs[] = {x, dy, dx, cache_in, dcache_out};
    const long long lds[] = {ldx, lddy, lddx};
    const bool vec = short_conv_vec(C, dtype, w, ptrs, 5, lds, 3);
    KDA_CONV_DISPATCH((conv::bwd<T, kW>(a, vec, dw, db, st)))
}

int launch_short_conv_step(const void* x, long long ldx, const void* w, const float* bias, void* cache, void* y,
                           long long ldy, int B, int C, int W, int dtype, int silu, cudaStream_t st) {
    conv::Args a{};
    a.x = x; a.ldx = ldx; a.w = w; a.bias = bias; a.y = y; a.ldy = ldy;
    a.nseq = B; a.seq_len = 1; a.ntok = B; a.C = C; a.silu = silu;
    const void* ptrs[] = {x, y, cache};
    const long long lds[] = {ldx, ldy};
    const bool vec = short_conv_vec(C, dtype, w, ptrs, 3, lds, 2);
    KDA_CONV_DISPATCH((conv::step<T, kW>(a, vec, cache, st)))
}

}  // namespace kda
