// Layer norm over the last axis, forward and backward.
//
//   mu = mean(x), r = 1 / sqrt(mean((x - mu)^2) + eps), y = (x - mu) r w + b
//   with xh = (x - mu) r and c = w dy:
//   dx = r (c - mean(c) - xh mean(c xh)),  dw = sum over rows of dy xh,  db = sum over rows of dy
//
// Both passes are bound by HBM: forward reads x and writes y, backward reads dy
// and x and writes dx.  A row therefore stays in registers from its load to its
// store (mean first, then the centred squares, so no cancellation), in 16-byte
// vectors held by one warp or by one block; widths that do not divide into
// 16-byte vectors, unaligned rows and rows beyond a block's registers take a
// kernel that walks the row again from the caches.  Statistics and sums are fp32.
#include "kda_mixer.cuh"

namespace kda {
namespace norm {

using namespace mix;

template <int kTpr>
__device__ __forceinline__ float row_sum(float v, float* sred) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (kTpr > 32) {
        constexpr int kW = kTpr / 32;
        if ((threadIdx.x & 31) == 0) sred[threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int w = 0; w < kW; ++w) v += sred[w];
    }
    return v;
}

// The values of a vector, two to a register pair.
template <typename T>
__device__ __forceinline__ void pairs(const Raw<T, true>& r, f2 (&v)[Pack<T, true>::kN / 2]) {
    float f[Pack<T, true>::kN];
    r.get(f);
#pragma unroll
    for (int u = 0; u < Pack<T, true>::kN / 2; ++u) v[u] = pk(f[2 * u], f[2 * u + 1]);
}

// kTpr threads hold one row, kVpt vectors each; a block of max(kTpr, 128) threads.
template <typename T, int kTpr, int kVpt>
__global__ void __launch_bounds__(kTpr == 32 ? 128 : kTpr)
    fwd_kernel(const T* __restrict__ x, long long ldx, const float* __restrict__ w, const float* __restrict__ b,
               T* __restrict__ y, long long ldy, float* __restrict__ mean, float* __restrict__ rstd, int M, int N,
               float eps) {
    constexpr int kE = Pack<T, true>::kN, kRows = kTpr == 32 ? 4 : 1;
    __shared__ float sred[2][kTpr > 32 ? kTpr / 32 : 1];
    const int t = threadIdx.x % kTpr, nvec = N / kE;
    long long row = (long long)blockIdx.x * kRows + threadIdx.x / kTpr;
    const long long step = (long long)gridDim.x * kRows;
    if (row >= M) return;  // whole warps; with one row per block the grid is exact
    for (; row < M; row += step) {
        Raw<T, true> raw[kVpt];
#pragma unroll
        for (int i = 0; i < kVpt; ++i) {
            const int j = t + i * kTpr;
            if (j < nvec) raw[i].load_stream(x + row * ldx + (size_t)j * kE);
            else raw[i].zero();
        }
        f2 f[kVpt][kE / 2], sum = 0ull;
#pragma unroll
        for (int i = 0; i < kVpt; ++i) {
            pairs(raw[i], f[i]);
#pragma unroll
            for (int u = 0; u < kE / 2; ++u) sum = add2(sum, f[i][u]);
        }
        const float mu = row_sum<kTpr>(lo2(sum) + hi2(sum), sred[0]) / float(N);
        const f2 nmu = dup2(-mu);
        sum = 0ull;
#pragma unroll
        for (int i = 0; i < kVpt; ++i) {
            if (t + i * kTpr >= nvec) break;
#pragma unroll
            for (int u = 0; u < kE / 2; ++u) {
                f[i][u] = add2(f[i][u], nmu);
                sum = fma2(f[i][u], f[i][u], sum);
            }
        }
        const float r = 1.f / sqrtf(row_sum<kTpr>(lo2(sum) + hi2(sum), sred[1]) / float(N) + eps);
        if (t == 0) {
            if (mean) mean[row] = mu;
            if (rstd) rstd[row] = r;
        }
        T* yr = y + row * ldy;
        const f2 r2 = dup2(r);
#pragma unroll
        for (int i = 0; i < kVpt; ++i) {
            const int j = t + i * kTpr;
            if (j >= nvec) break;
            float o[kE];
#pragma unroll
            for (int u = 0; u < kE; u += 4) {
                f2 v0 = mul2(f[i][u / 2], r2), v1 = mul2(f[i][u / 2 + 1], r2);
                if (w) {
                    const ulonglong2 ww = *reinterpret_cast<const ulonglong2*>(w + (size_t)j * kE + u);
                    const ulonglong2 bb = b ? *reinterpret_cast<const ulonglong2*>(b + (size_t)j * kE + u) : make_ulonglong2(0, 0);
                    v0 = fma2(v0, ww.x, bb.x);
                    v1 = fma2(v1, ww.y, bb.y);
                } else if (b) {
                    const ulonglong2 bb = *reinterpret_cast<const ulonglong2*>(b + (size_t)j * kE + u);
                    v0 = add2(v0, bb.x);
                    v1 = add2(v1, bb.y);
                }
                upk(v0, o[u], o[u + 1]);
                upk(v1, o[u + 2], o[u + 3]);
            }
            raw[i].set(o);
            raw[i].store(yr + (size_t)j * kE);
        }
    }
}

// Many rows of up to 512 vectors: kTpr threads own two vectors of columns each and keep
// those columns' weight and bias in registers for all the rows that the block walks
// (read from L1 for every row they are four times the row's own bytes, and the L1 pipe
// was the bound: 102 us at 65536 x 2048 bf16, now 90 us = 6.0 TB/s, in a graph's replays).  512 threads an SM
// measured best (384: 98, 640: 97, 768: 122 us).  kR rows at a time share the barriers;
// the rows to come are on their way into a ring by copies that each thread waits for on
// its own (it reads back only what it copied itself).
template <typename T, int kTpr>
__global__ void __launch_bounds__(kTpr)
    fwd_rows_kernel(const T* __restrict__ x, long long ldx, const float* __restrict__ w, const float* __restrict__ b,
                    T* __restrict__ y, long long ldy, float* __restrict__ mean, float* __restrict__ rstd, int M, int N,
                    float eps) {
    constexpr int kE = Pack<T, true>::kN, kVpt = 2, kR = 2, kDepth = kTpr < 256 ? 3 : 2, kW = kTpr / 32;
    __shared__ float sred[2][2][kW][kR];
    __shared__ __align__(16) uint4 ring[kDepth][kR][kVpt][kTpr];
    const int t = threadIdx.x, nvec = N / kE, warp = t >> 5;
    const bool have[kVpt] = {t < nvec, t + kTpr < nvec};
    f2 wv[kVpt][kE / 2], bv[kVpt][kE / 2];
#pragma unroll
    for (int i = 0; i < kVpt; ++i)
#pragma unroll
        for (int u = 0; u < kE / 2; ++u) {
            const int c = (t + i * kTpr) * kE + 2 * u;
            wv[i][u] = w && have[i] ? pk(w[c], w[c + 1]) : dup2(1.f);
            bv[i][u] = b && have[i] ? pk(b[c], b[c + 1]) : 0ull;
        }
    const long long step = (long long)gridDim.x * kR;
    auto request = [&](long long r0, int slot) {
#pragma unroll
        for (int r = 0; r < kR; ++r)
#pragma unroll
            for (int i = 0; i < kVpt; ++i)
                if (r0 + r < M && have[i]) cp_async<16>(&ring[slot][r][i][t], x + (r0 + r) * ldx + (size_t)(t + i * kTpr) * kE);
        cp_async_commit();
    };
    long long row = (long long)blockIdx.x * kR;
#pragma unroll
    for (int k = 0; k < kDepth - 1; ++k) request(row + k * step, k);
    int slot = 0, buf = 0;
    for (; row < M; row += step, buf ^= 1) {
        cp_async_wait<kDepth - 2>();
        f2 f[kR][kVpt][kE / 2];
        float s[kR];
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            f2 a = 0ull;
#pragma unroll
            for (int i = 0; i < kVpt; ++i) {
                Raw<T, true> raw;
                if (row + r < M && have[i]) raw.v = ring[slot][r][i][t];
                else raw.zero();
                pairs(raw, f[r][i]);
#pragma unroll
                for (int u = 0; u < kE / 2; ++u) a = add2(a, f[r][i][u]);
            }
            s[r] = lo2(a) + hi2(a);
        }
        request(row + (kDepth - 1) * step, slot == 0 ? kDepth - 1 : slot - 1);  // into the place used before this one
        if (++slot == kDepth) slot = 0;
        // (the two sums have buffers of their own, and a row's barriers come before its
        // successor but one writes them again)
        auto block_sum = [&](int which) {
#pragma unroll
            for (int r = 0; r < kR; ++r) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) s[r] += __shfl_xor_sync(0xffffffffu, s[r], o);
                if ((t & 31) == 0) sred[which][buf][warp][r] = s[r];
            }
            __syncthreads();
#pragma unroll
            for (int r = 0; r < kR; ++r) {
                s[r] = 0.f;
#pragma unroll
                for (int k = 0; k < kW; ++k) s[r] += sred[which][buf][k][r];
            }
        };
        block_sum(0);
        float mu[kR];
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            mu[r] = s[r] / float(N);
            const f2 nmu = dup2(-mu[r]);
            f2 a = 0ull;
#pragma unroll
            for (int i = 0; i < kVpt; ++i)
                if (have[i]) {
#pragma unroll
                    for (int u = 0; u < kE / 2; ++u) {
                        f[r][i][u] = add2(f[r][i][u], nmu);
                        a = fma2(f[r][i][u], f[r][i][u], a);
                    }
                }
            s[r] = lo2(a) + hi2(a);
        }
        block_sum(1);
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            if (row + r >= M) break;
            const float rs = 1.f / sqrtf(s[r] / float(N) + eps);
            if (t == 0) {
                if (mean) mean[row + r] = mu[r];
                if (rstd) rstd[row + r] = rs;
            }
            const f2 r2 = dup2(rs);
#pragma unroll
            for (int i = 0; i < kVpt; ++i) {
                float o[kE];
#pragma unroll
                for (int u = 0; u < kE / 2; ++u) upk(fma2(mul2(f[r][i][u], r2), wv[i][u], bv[i][u]), o[2 * u], o[2 * u + 1]);
                Raw<T, true> raw;
                raw.set(o);
                if (have[i]) raw.store(y + (row + r) * ldy + (size_t)(t + i * kTpr) * kE);
            }
        }
    }
}

// Any width and alignment: one block or (up to 1024) one warp per row, element by element; the second and
// third walk over the row hit the caches.
template <typename T, int kTpr>
__global__ void __launch_bounds__(256)
    fwd_any_kernel(const T* __restrict__ x, long long ldx, const float* __restrict__ w, const float* __restrict__ b,
                   T* __restrict__ y, long long ldy, float* __restrict__ mean, float* __restrict__ rstd, int M, int N,
                   float eps) {
    __shared__ float sred[2][8];
    const int t = threadIdx.x % kTpr;
    const long long row = (long long)blockIdx.x * (256 / kTpr) + threadIdx.x / kTpr;
    if (row >= M) return;  // whole warps; with one row per block the grid is exact
    const T* xr = x + row * ldx;
    float s = 0.f;
    for (int j = t; j < N; j += kTpr) s += to_f32<T>(xr[j]);
    const float mu = row_sum<kTpr>(s, sred[0]) / float(N);
    s = 0.f;
    for (int j = t; j < N; j += kTpr) {
        const float d = to_f32<T>(xr[j]) - mu;
        s += d * d;
    }
    const float r = 1.f / sqrtf(row_sum<kTpr>(s, sred[1]) / float(N) + eps);
    if (t == 0) {
        if (mean) mean[row] = mu;
        if (rstd) rstd[row] = r;
    }
    T* yr = y + row * ldy;
    for (int j = t; j < N; j += kTpr)
        yr[j] = from_f32<T>((to_f32<T>(xr[j]) - mu) * r * (w ? w[j] : 1.f) + (b ? b[j] : 0.f));
}

// Backward, rows in registers.  A block of kTpr threads owns every gridDim.x-th
// row and adds up its columns of dw and db in registers over its rows, so those
// sums cost no extra pass; the blocks' partial sums [block][2][N] are added in a
// fixed order by sum_parts_kernel.
template <typename T, int kTpr, int kVpt>
__global__ void __launch_bounds__(kTpr)
    bwd_kernel(const T* __restrict__ dy, long long lddy, const T* __restrict__ x, long long ldx,
               const float* __restrict__ w, const float* __restrict__ mean, const float* __restrict__ rstd,
               T* __restrict__ dx, long long lddx, float* __restrict__ part, int M, int N) {
    constexpr int kE = Pack<T, true>::kN;
    __shared__ float2 sred[2][kTpr / 32];
    const int t = threadIdx.x, nvec = N / kE;
    // the columns' weights: in registers where they fit (16 a thread)
    constexpr bool kHold = kVpt * kE <= 16;
    f2 wv[kHold ? kVpt : 1][kE / 2];
    if constexpr (kHold) {
#pragma unroll
        for (int i = 0; i < kVpt; ++i)
#pragma unroll
            for (int u = 0; u < kE / 2; ++u) {
                const int c = (t + i * kTpr) * kE + 2 * u;
                wv[i][u] = w && t + i * kTpr < nvec ? pk(w[c], w[c + 1]) : dup2(1.f);
            }
    }
    auto weights = [&](int i, int u) {
        if constexpr (kHold) return make_ulonglong2(wv[i][u], wv[i][u + 1]);
        else return w ? *reinterpret_cast<const ulonglong2*>(w + (t + i * kTpr) * kE + 2 * u) : make_ulonglong2(dup2(1.f), dup2(1.f));
    };
    f2 aw[kVpt][kE / 2], ab[kVpt][kE / 2];
#pragma unroll
    for (int i = 0; i < kVpt; ++i)
#pragma unroll
        for (int u = 0; u < kE / 2; ++u) aw[i][u] = ab[i][u] = 0ull;
    // the block's next row, requested one row ahead where the registers allow it (32
    // values a thread would spill)
    constexpr bool kAhead = kVpt * kE <= 16;
    Raw<T, true> nx[kVpt], nd[kVpt];
    float nmu = 0.f, nr = 0.f;
    auto request = [&](long long row) {
#pragma unroll
        for (int i = 0; i < kVpt; ++i) {
            const int j = t + i * kTpr;
            if (j < nvec) {
                nx[i].load(x + row * ldx + (size_t)j * kE);
                nd[i].load(dy + row * lddy + (size_t)j * kE);
            } else {
                nx[i].zero();
                nd[i].zero();
            }
        }
        nmu = mean[row];
        nr = rstd[row];
    };
    int buf = 0;
    if (kAhead && blockIdx.x < M) request(blockIdx.x);
    for (long long row = blockIdx.x; row < M; row += gridDim.x, buf ^= 1) {
        if (!kAhead) request(row);
        Raw<T, true> rx[kVpt], rd[kVpt];
#pragma unroll
        for (int i = 0; i < kVpt; ++i) {
            rx[i] = nx[i];
            rd[i] = nd[i];
        }
        const float mu = nmu, r = nr;
        if (kAhead && row + gridDim.x < M) request(row + gridDim.x);
        // (xh from the difference: x r - mu r would cancel where the mean is far above the spread)
        const f2 r2 = dup2(r), minus_mu = dup2(-mu);
        f2 p0 = 0ull, p1 = 0ull;  // sums of c and c xh
#pragma unroll
        for (int i = 0; i < kVpt; ++i) {
            const int j = t + i * kTpr;
            if (j >= nvec) break;
            f2 fx[kE / 2], fd[kE / 2];
            pairs(rx[i], fx);
            pairs(rd[i], fd);
#pragma unroll
            for (int u = 0; u < kE / 2; u += 2) {
                const ulonglong2 ww = weights(i, u);
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    const f2 xh = mul2(add2(fx[u + v], minus_mu), r2), c = mul2(fd[u + v], v ? ww.y : ww.x);
                    p0 = add2(p0, c);
                    p1 = fma2(c, xh, p1);
                    aw[i][u + v] = fma2(fd[u + v], xh, aw[i][u + v]);
                    ab[i][u + v] = add2(ab[i][u + v], fd[u + v]);
                }
            }
        }
        float s0 = lo2(p0) + hi2(p0), s1 = lo2(p1) + hi2(p1);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            s0 += __shfl_xor_sync(0xffffffffu, s0, o);
            s1 += __shfl_xor_sync(0xffffffffu, s1, o);
        }
        // two buffers: a block's next row writes the other one, and the barrier of that
        // row comes before this buffer is written again
        if ((t & 31) == 0) sred[buf][t >> 5] = make_float2(s0, s1);
        __syncthreads();
        s0 = s1 = 0.f;
#pragma unroll
        for (int k = 0; k < kTpr / 32; ++k) {
            s0 += sred[buf][k].x;
            s1 += sred[buf][k].y;
        }
        // dx = r c - r mean(c) - xh r mean(c xh)
        const f2 m0 = dup2(-r * (s0 / float(N))), m1 = dup2(-r * (s1 / float(N)));
#pragma unroll
        for (int i = 0; i < kVpt; ++i) {
            const int j = t + i * kTpr;
            if (j >= nvec) break;
            f2 fx[kE / 2], fd[kE / 2];
            pairs(rx[i], fx);
            pairs(rd[i], fd);
            float o[kE];
#pragma unroll
            for (int u = 0; u < kE / 2; u += 2) {
                const ulonglong2 ww = weights(i, u);
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    const f2 xh = mul2(add2(fx[u + v], minus_mu), r2), c = mul2(fd[u + v], v ? ww.y : ww.x);
                    upk(fma2(c, r2, fma2(xh, m1, m0)), o[2 * (u + v)], o[2 * (u + v) + 1]);
                }
            }
            rd[i].set(o);
            rd[i].store(dx + row * lddx + (size_t)j * kE);
        }
    }
    if (part) {
#pragma unroll
        for (int i = 0; i < kVpt; ++i) {
            const int j = t + i * kTpr;
            if (j >= nvec) break;
            float* p = part + (size_t)blockIdx.x * 2 * N + (size_t)j * kE;
#pragma unroll
            for (int u = 0; u < kE / 2; u += 2) {
                *reinterpret_cast<ulonglong2*>(p + 2 * u) = make_ulonglong2(aw[i][u], aw[i][u + 1]);
                *reinterpret_cast<ulonglong2*>(p + N + 2 * u) = make_ulonglong2(ab[i][u], ab[i][u + 1]);
            }
        }
    }
}

// Any width and alignment: dx row by row, then the column sums in a second walk.
template <typename T, int kTpr>
__global__ void __launch_bounds__(256)
    bwd_any_kernel(const T* __restrict__ dy, long long lddy, const T* __restrict__ x, long long ldx,
                   const float* __restrict__ w, const float* __restrict__ mean, const float* __restrict__ rstd,
                   T* __restrict__ dx, long long lddx, int M, int N) {
    __shared__ float sred[2][8];
    const int t = threadIdx.x % kTpr;
    const long long row = (long long)blockIdx.x * (256 / kTpr) + threadIdx.x / kTpr;
    if (row >= M) return;  // whole warps; with one row per block the grid is exact
    const T *xr = x + row * ldx, *dr = dy + row * lddy;
    const float mu = mean[row], r = rstd[row];
    float s0 = 0.f, s1 = 0.f;
    for (int j = t; j < N; j += kTpr) {
        const float c = __fmul_rn(to_f32<T>(dr[j]), w ? w[j] : 1.f);  // rounded as below: c - mean(c) is exactly 0 at N = 1
        s0 += c;
        s1 += c * (to_f32<T>(xr[j]) - mu) * r;
    }
    s0 = row_sum<kTpr>(s0, sred[0]) / float(N);
    s1 = row_sum<kTpr>(s1, sred[1]) / float(N);
    T* dxr = dx + row * lddx;
    for (int j = t; j < N; j += kTpr) {
        const float xh = (to_f32<T>(xr[j]) - mu) * r;
        dxr[j] = from_f32<T>(r * (__fmul_rn(to_f32<T>(dr[j]), w ? w[j] : 1.f) - s0 - xh * s1));
    }
}
// Thread = one column, block row = a run of rows: partial sums [gridDim.y][2][N].
template <typename T>
__global__ void __launch_bounds__(128)
    bwd_any_cols_kernel(const T* __restrict__ dy, long long lddy, const T* __restrict__ x, long long ldx,
                        const float* __restrict__ mean, const float* __restrict__ rstd, float* __restrict__ part, int M,
                        int N) {
    const int j = blockIdx.x * 128 + threadIdx.x;
    if (j >= N) return;
    float aw = 0.f, ab = 0.f;
#pragma unroll 4
    for (long long row = blockIdx.y; row < M; row += gridDim.y) {
        const float d = to_f32<T>(dy[row * lddy + j]);
        aw += d * (to_f32<T>(x[row * ldx + j]) - mean[row]) * rstd[row];
        ab += d;
    }
    part[(size_t)blockIdx.y * 2 * N + j] = aw;
    part[(size_t)blockIdx.y * 2 * N + N + j] = ab;
}

// Threads and vectors per thread that hold a row of nvec vectors.
struct Shape {
    int tpr, vpt;  // vpt 0: no fit
};
static Shape bwd_shape(int nvec) {
    if (nvec <= 64) return {32, nvec <= 32 ? 1 : 2};
    if (nvec <= 256) return {128, nvec <= 128 ? 1 : 2};
    if (nvec <= 512) return {256, 2};
    if (nvec <= 2048) return {512, nvec <= 1024 ? 2 : 4};
    return {0, 0};
}

static bool vec_ok(int N, int es, const void* const* ptrs, const long long* lds, int n) {
    if ((N * es) % 16) return false;
    for (int i = 0; i < n; ++i)
        if (!al16(ptrs[i]) || (lds[i] * es) % 16) return false;
    return true;
}

// Blocks of the backward pass: enough to fill the SMs at the register use of the
// shape, and no more than there are rows (each block writes 2 N partial sums).
static int bwd_blocks(int M, int tpr) {
    const long long want = (long long)device_sm_count() * (tpr >= 512 ? 1 : (tpr == 256 ? 2 : (tpr == 128 ? 4 : 12)));
    return int(M < want ? M : want);
}
static int any_blocks(int M) { return M < 256 ? M : 256; }

template <typename T>
int fwd(const T* x, long long ldx, const float* w, const float* b, T* y, long long ldy, float* mean, float* rstd, int M,
        int N, float eps, cudaStream_t st) {
    constexpr int es = sizeof(T), kE = 16 / es;
    const void* ptrs[] = {x, y, w, b};
    const long long lds[] = {ldx, ldy, 0, 0};
    const int nvec = N / kE;
    if (vec_ok(N, es, ptrs, lds, 4) && nvec <= 2048) {
#define KDA_LN_FWD(TPR, VPT)                                                                                   \
    fwd_kernel<T, TPR, VPT><<<unsigned(TPR == 32 ? cdiv(M, 4) : M), TPR == 32 ? 128 : TPR, 0, st>>>(           \
        x, ldx, w, b, y, ldy, mean, rstd, M, N, eps)
#define KDA_LN_ROWS(TPR)                                                                                       \
    fwd_rows_kernel<T, TPR><<<unsigned(device_sm_count()) * (512 / TPR), TPR, 0, st>>>(x, ldx, w, b, y, ldy, mean, \
                                                                                       rstd, M, N, eps)
        const bool many = M > 32 * device_sm_count();  // several rows for every block that the SMs hold
        if (nvec <= 32) KDA_LN_FWD(32, 1);
        else if (nvec <= 64) KDA_LN_FWD(32, 2);
        else if (nvec <= 128 && many) KDA_LN_ROWS(64);
        else if (nvec <= 128) KDA_LN_FWD(32, 4);
        else if (nvec <= 256 && many) KDA_LN_ROWS(128);
        else if (nvec <= 256) KDA_LN_FWD(128, 2);
        else if (nvec <= 512 && many) KDA_LN_ROWS(256);
        else if (nvec <= 512) KDA_LN_FWD(256, 2);
        else if (nvec <= 1024) KDA_LN_FWD(256, 4);
        else KDA_LN_FWD(512, 4);
#undef KDA_LN_ROWS
#undef KDA_LN_FWD
    } else {
        if (N <= 1024) fwd_any_kernel<T, 32><<<unsigned(cdiv(M, 8)), 256, 0, st>>>(x, ldx, w, b, y, ldy, mean, rstd, M, N, eps);
        else fwd_any_kernel<T, 256><<<unsigned(M), 256, 0, st>>>(x, ldx, w, b, y, ldy, mean, rstd, M, N, eps);
    }
    return cudaPeekAtLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

template <typename T>
int bwd(const T* dy, long long lddy, const T* x, long long ldx, const float* w, const float* mean, const float* rstd,
        T* dx, long long lddx, float* dw, float* db, int M, int N, float* part, cudaStream_t st) {
    constexpr int es = sizeof(T), kE = 16 / es;
    const void* ptrs[] = {dy, x, dx, w};
    const long long lds[] = {lddy, ldx, lddx, 0};
    const Shape sh = bwd_shape(N / kE);
    int parts;
    if (vec_ok(N, es, ptrs, lds, 4) && sh.vpt) {
        parts = bwd_blocks(M, sh.tpr);
        float* p = (dw || db) ? part : nullptr;
#define KDA_LN_BWD(TPR, VPT) \
    if (sh.tpr == TPR && sh.vpt == VPT) \
    bwd_kernel<T, TPR, VPT><<<parts, TPR, 0, st>>>(dy, lddy, x, ldx, w, mean, rstd, dx, lddx, p, M, N)
        KDA_LN_BWD(32, 1);
        KDA_LN_BWD(32, 2);
        KDA_LN_BWD(128, 1);
        KDA_LN_BWD(128, 2);
        KDA_LN_BWD(256, 2);
        KDA_LN_BWD(512, 2);
        KDA_LN_BWD(512, 4);
#undef KDA_LN_BWD
    } else {
        if (N <= 1024) bwd_any_kernel<T, 32><<<unsigned(cdiv(M, 8)), 256, 0, st>>>(dy, lddy, x, ldx, w, mean, rstd, dx, lddx, M, N);
        else bwd_any_kernel<T, 256><<<unsigned(M), 256, 0, st>>>(dy, lddy, x, ldx, w, mean, rstd, dx, lddx, M, N);
        parts = any_blocks(M);
        if (dw || db)
            bwd_any_cols_kernel<T><<<dim3(unsigned(cdiv(N, 128)), parts), 128, 0, st>>>(dy, lddy, x, ldx, mean, rstd,
                                                                                        part, M, N);
    }
    sum_parts<float>(part, parts, 2ll * N, dw, db, N, st);
    return cudaPeekAtLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace norm

size_t layer_norm_bwd_workspace_bytes(int M, int N) {
    // whichever path the call takes (its type and alignment decide): the most blocks of any
    int parts = norm::any_blocks(M);
    for (int e = 4; e <= 8; e += 4) {
        const norm::Shape sh = norm::bwd_shape(N / e);
        if (sh.vpt && norm::bwd_blocks(M, sh.tpr) > parts) parts = norm::bwd_blocks(M, sh.tpr);
    }
    return mix::up256(size_t(parts) * 2 * N * sizeof(float));
}

int launch_layer_norm_fwd(const void* x, long long ldx, const float* w, const float* b, void* y, long long ldy,
                          float* mean, float* rstd, int M, int N, int dtype, float eps, cudaStream_t st) {
    if (dtype == KDA_BF16)
        return norm::fwd(static_cast<const __nv_bfloat16*>(x), ldx, w, b, static_cast<__nv_bfloat16*>(y), ldy, mean,
                         rstd, M, N, eps, st);
    return norm::fwd(static_cast<const float*>(x), ldx, w, b, static_cast<float*>(y), ldy, mean, rstd, M, N, eps, st);
}

int launch_layer_norm_bwd(const void* dy, long long lddy, const void* x, long long ldx, const float* w,
                          const float* mean, const float* rstd, void* dx, long long lddx, float* dw, float* db, int M,
                          int N, int dtype, void* ws, cudaStream_t st) {
    float* part = static_cast<float*>(ws);
    if (dtype == KDA_BF16)
        return norm::bwd(static_cast<const __nv_bfloat16*>(dy), lddy, static_cast<const __nv_bfloat16*>(x), ldx, w,
                         mean, rstd, static_cast<__nv_bfloat16*>(dx), lddx, dw, db, M, N, part, st);
    return norm::bwd(static_cast<const float*>(dy), lddy, static_cast<const float*>(x), ldx, w, mean, rstd,
                     static_cast<float*>(dx), lddx, dw, db, M, N, part, st);
}

}  // namespace kda
