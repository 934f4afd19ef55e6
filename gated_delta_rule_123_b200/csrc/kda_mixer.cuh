// Device and host helpers shared by the selective mixer's kernels (layer norm,
// linear epilogue gradients, short convolution, selective scan).
#pragma once

#include <type_traits>

#include "kda_common.cuh"

namespace kda {

int device_sm_count();

namespace mix {

// A 16-byte vector of T (kVec) or one element, as floats.
template <typename T, bool kVec>
struct Pack {
    static constexpr int kN = kVec ? int(16 / sizeof(T)) : 1;
};

__device__ __forceinline__ void unpack16(const uint4& r, float* f, float) {
    f[0] = __uint_as_float(r.x);
    f[1] = __uint_as_float(r.y);
    f[2] = __uint_as_float(r.z);
    f[3] = __uint_as_float(r.w);
}
__device__ __forceinline__ void unpack16(const uint4& r, float* f, __nv_bfloat16) {
    // a bf16 is the upper half of the fp32 with the same value
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint32_t pack2_rn(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ uint4 pack16(const float* f, float) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
__device__ __forceinline__ uint4 pack16(const float* f, __nv_bfloat16) {
    return make_uint4(pack2_rn(f[0], f[1]), pack2_rn(f[2], f[3]), pack2_rn(f[4], f[5]), pack2_rn(f[6], f[7]));
}

// Raw storage of one Pack: loads are issued early and converted later.
template <typename T, bool kVec>
struct Raw {
    using type = typename std::conditional<kVec, uint4, T>::type;
    type v;
    __device__ __forceinline__ void load(const T* p) { v = *reinterpret_cast<const type*>(p); }
    __device__ __forceinline__ void load_stream(const T* p) { v = __ldcs(reinterpret_cast<const type*>(p)); }
    __device__ __forceinline__ void zero() {
        if constexpr (kVec) v = make_uint4(0, 0, 0, 0);
        else v = from_f32<T>(0.f);
    }
    __device__ __forceinline__ void get(float* f) const {
        if constexpr (kVec) unpack16(v, f, T());
        else f[0] = to_f32<T>(v);
    }
    __device__ __forceinline__ void set(const float* f) {
        if constexpr (kVec) v = pack16(f, T());
        else v = from_f32<T>(f[0]);
    }
    __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<type*>(p) = v; }
};

// Two fp32 values in one 64-bit register pair: Blackwell's packed instructions do both
// in one issue slot (the kernels here are bound by issue and by the special-function
// unit where they are not bound by HBM).
typedef unsigned long long f2;
__device__ __forceinline__ f2 pk(float lo, float hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void upk(f2 v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ float lo2(f2 v) {
    float a, b;
    upk(v, a, b);
    return a;
}
__device__ __forceinline__ float hi2(f2 v) {
    float a, b;
    upk(v, a, b);
    return b;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 dup2(float v) { return pk(v, v); }

// 2^x on the special-function unit (relative error about 2^-22; below 2^-126 it gives 0).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kL2e = 1.4426950408889634f;

__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// log(1 + e^x) = max(x, 0) + log1p(e^-|x|).  log1p(e) / e on [0, 1] is its Chebyshev
// interpolant of degree 9 (relative error 1.2e-7 with fp32 coefficients and steps, also
// where e is tiny): no second special function, and no branch.
__device__ __forceinline__ float softplus_poly(float x) {
    const float e = ex2(-fabsf(x) * kL2e);
    float r = fmaf(-0.0031760570127516985f, e, 0.019542526453733444f);
    r = fmaf(r, e, -0.056373611092567444f);
    r = fmaf(r, e, 0.10543623566627502f);
    r = fmaf(r, e, -0.1526966691017151f);
    r = fmaf(r, e, 0.1966327428817749f);
    r = fmaf(r, e, -0.24951615929603577f);
    r = fmaf(r, e, 0.33329710364341736f);
    r = fmaf(r, e, -0.49999892711639404f);
    r = fmaf(r, e, 1.f);
    return fmaf(r, e, fmaxf(x, 0.f));
}
// x / (1 + e^-x); -0 where e^-x overflows.  Like sigmoidf below it takes the fast
// exponential and division (relative error about 2^-21 + |x| 2^-24, for negative x; less
// for positive ones): they are one special function each, which is what bounds the scan.
// In fp32 outputs of the convolution 1.9e-7 is left where exact functions leave 1.3e-7.
__device__ __forceinline__ float siluf(float x) { return x * rcp(1.f + ex2(-x * kL2e)); }

// 16, 8 or 4 bytes of global memory into shared memory, asynchronously.
template <int kBytes>
__device__ __forceinline__ void cp_async(void* dst, const void* src) {
    static_assert(kBytes == 4 || kBytes == 8 || kBytes == 16, "cp.async size");
    if constexpr (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(dst)), "l"(src), "n"(kBytes) : "memory");
}
// 16 bytes, of which the first `bytes` are read and the others are 0.
__device__ __forceinline__ void cp_async_part(void* dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory"); }
__device__ __forceinline__ void cp_async_wait0() { cp_async_wait<0>(); }

__device__ __forceinline__ float sigmoidf(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }
// Sequence of token t, packed (cu[n] <= t < cu[n + 1]) or dense with seq_len tokens each,
// and a sequence's first token.  Offsets outside 0 .. ntok count as the nearer bound, so
// that no offsets lead to memory that is not the tensors'.
__device__ __forceinline__ int seq_of(const int32_t* cu, int nseq, int seq_len, int t) {
    if (!cu) return t / seq_len;
    int lo = 0, hi = nseq;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}
__device__ __forceinline__ int seq_begin(const int32_t* cu, int seq_len, int n, int ntok) {
    return cu ? max(0, min(cu[n], ntok)) : n * seq_len;
}

inline bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline size_t up256(size_t x) { return (x + 255) & ~size_t(255); }
inline long long cdiv(long long a, long long b) { return (a + b - 1) / b; }

// out[i] = sum over p of part[p * stride + i], i < n, in a fixed order: 32 threads
// add every 32nd part each, then their sums are added.  Two outputs of n columns side
// by side in the parts (n each, the second may be NULL) go in one launch.  Bound by
// the latency of a thread's chain of loads, so the chain is short and unrolled:
// 592 parts of 4096 columns take 6 us (with 8 threads a column, 20 us).
template <typename Out>
__global__ void __launch_bounds__(1024) sum_parts_kernel(const float* __restrict__ part, int parts, long long stride,
                                                         Out* __restrict__ out, Out* __restrict__ out2, long long n) {
    __shared__ float s[32][33];
    const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
    const long long blocks1 = (n + 31) / 32;
    const bool second = blockIdx.x >= blocks1;
    const long long i = (blockIdx.x - (second ? blocks1 : 0)) * 32 + lane;
    Out* o = second ? out2 : out;
    if (!o) return;
    float a = 0.f;
    if (i < n) {
        const float* q = part + (second ? n : 0) + i;
#pragma unroll 8
        for (int p = row; p < parts; p += 32) a += q[p * stride];
    }
    s[row][lane] = a;
    __syncthreads();
    if (row == 0 && i < n) {
        float t = 0.f;
#pragma unroll
        for (int r = 0; r < 32; ++r) t += s[r][lane];
        o[i] = from_f32<Out>(t);
    }
}
template <typename Out>
inline void sum_parts(const float* part, int parts, long long stride, Out* out, Out* out2, long long n, cudaStream_t st) {
    if (!out && !out2) return;
    sum_parts_kernel<Out><<<unsigned(cdiv(n, 32) * (out2 ? 2 : 1)), 1024, 0, st>>>(part, parts, stride, out, out2, n);
}

}  // namespace mix

// Launches of the mixer's kernels (argument checks: kda_mixer_api.cu).
size_t layer_norm_bwd_workspace_bytes(int M, int N);
int launch_layer_norm_fwd(const void* x, long long ldx, const float* w, const float* b, void* y, long long ldy,
                          float* mean, float* rstd, int M, int N, int dtype, float eps, cudaStream_t st);
int launch_layer_norm_bwd(const void* dy, long long lddy, const void* x, long long ldx, const float* w,
                          const float* mean, const float* rstd, void* dx, long long lddx, float* dw, float* db, int M,
                          int N, int dtype, void* ws, cudaStream_t st);
size_t short_conv_bwd_workspace_bytes(int ntok, int C, int W);
int launch_short_conv_fwd(const void* x, long long ldx, const void* w, const float* bias, void* y, long long ldy,
                          const void* cache_in, void* cache_out, const int32_t* cu, int nseq, int seq_len, int ntok,
                          int C, int W, int dtype, int silu, cudaStream_t st);
int launch_short_conv_bwd(const void* dy, long long lddy, const void* x, long long ldx, const void* w,
                          const float* bias, const void* cache_in, const void* dcache_out, void* dx, long long lddx,
                          void* dw, float* db, void* dcache_in, const int32_t* cu, int nseq, int seq_len, int ntok,
                          int C, int W, int dtype, int silu, void* ws, cudaStream_t st);
int launch_short_conv_step(const void* x, long long ldx, const void* w, const float* bias, void* cache, void* y,
                           long long ldy, int B, int C, int W, int dtype, int silu, cudaStream_t st);

}  // namespace kda
