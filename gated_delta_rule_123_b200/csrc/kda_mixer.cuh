// Device and host helpers shared by the selective mixer's kernels (layer norm,
// linear epilogue gradients, short convolution, selective scan).
#pragma once

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

__device__ __forceinline__ float sigmoidf(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }
// log(1 + e^x) without overflow, and with e^x's relative accuracy for very negative x.
__device__ __forceinline__ float softplusf(float x) { return fmaxf(x, 0.f) + log1pf(__expf(-fabsf(x))); }

inline bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline size_t up256(size_t x) { return (x + 255) & ~size_t(255); }
inline long long cdiv(long long a, long long b) { return (a + b - 1) / b; }

// out[i] = sum over p of part[p * stride + i], i < n, in a fixed order: 8 threads
// walk every 8th part each, then their sums are added.  Bound by reading the
// partial sums once.
template <typename Out>
__global__ void __launch_bounds__(256) sum_parts_kernel(const float* __restrict__ part, int parts, long long stride,
                                                        Out* __restrict__ out, long long n) {
    __shared__ float s[8][33];
    const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
    const long long i = (long long)blockIdx.x * 32 + lane;
    float a = 0.f, b = 0.f;
    if (i < n) {
        int p = row;
        for (; p + 8 < parts; p += 16) {
            a += part[p * stride + i];
            b += part[(p + 8) * stride + i];
        }
        if (p < parts) a += part[p * stride + i];
    }
    s[row][lane] = a + b;
    __syncthreads();
    if (row == 0 && i < n) {
        float t = 0.f;
#pragma unroll
        for (int r = 0; r < 8; ++r) t += s[r][lane];
        out[i] = from_f32<Out>(t);
    }
}

}  // namespace mix
}  // namespace kda
