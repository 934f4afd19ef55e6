// The projection GEMM with a bias, an activation and a residual in its epilogue,
// and its gradients, on sm_100a.
//
//   s = x W^T + b,  y = act(s) + residual          x [M, K], W [N, K], y [M, N]
//   ds = dy act'(s):  dx = ds W,  dW = ds^T x,  db = sum over rows of ds
//
// "Kimi Linear: An Expressive, Efficient Attention Architecture", section "Neural
// Parameterization", has bias-free projections (kda_linear_bf16); the mixers next
// to them have a bias, an activation or a residual after theirs, and training
// needs the gradients.  All three products run in one persistent tcgen05 kernel
// with the roles of kda_gemm.cu (a TMA producer warp, one MMA-issuing thread, two
// accumulators in TMEM, eight epilogue warps).  What differs by product is which
// axis of an operand is contiguous: x and W of the forward pass hold the summed
// axis contiguous (K-major tiles); in dx = ds W the summed axis is the row index
// of W, in dW = ds^T x it is the row index of both, so those tiles are loaded as
// 64-column by 64-row boxes and read as MN-major operands.  No operand is ever
// transposed in memory.  bf16 operands, fp32 accumulation; ds is rounded to bf16
// because it is an operand of two tensor-core products.
#include "kda_gemm.cuh"
#include "kda_mixer.cuh"

namespace kda {
namespace lin {

using namespace gemm;  // the GEMM's TMA, TMEM and staging helpers, and its tile BM x BK

enum Act { kNone = KDA_ACT_NONE, kRelu = KDA_ACT_RELU, kGelu = KDA_ACT_GELU, kSilu = KDA_ACT_SILU,
           kSoftplus = KDA_ACT_SOFTPLUS };

template <int kBN>
struct LPlan {
    static constexpr uint32_t kB = kBN * BK * 2, kStage = kABytes + kB;
    // per epilogue warp: one tile, for s and then for y (a tile for each would cost the
    // fourth stage: 516 us against 424 at 16384 x 8192 x 2048 with a bias and the pre-activation)
    static constexpr uint32_t kStagingBytes = 4096;
    // as many stages as fit beside the staging tiles and the barriers, at most 8
    static constexpr int kFit = int((232448 - 1280 - kEpiWarps * kStagingBytes) / kStage);
    static constexpr int kStages = kFit < 8 ? kFit : 8;
    static constexpr uint32_t OFF_STAGING = kStages * kStage;
    static constexpr uint32_t OFF_BARS = OFF_STAGING + kEpiWarps * kStagingBytes;
    static constexpr uint32_t kSmem = OFF_BARS + 256 + 1024;
    static_assert(kStages >= 3 && kSmem <= 232448, "shared-memory plan");
};

struct LArgs {
    int M, N, K, tiles_m, tiles_n;
    const float* bias;
    const __nv_bfloat16* res;
    int ldr, res_vec, act;
    __nv_bfloat16 *c, *pre;  // outputs, for the columns that no TMA store writes
    int ldc, ldp;
};

// A TMA store clips a row at whole 16-byte groups, so it would write past an N that is
// not a multiple of 8: the maps of the outputs end at the last whole group, and the
// N % 8 columns after it are stored by each row's thread.
template <int kN>
__device__ __forceinline__ void store_ragged(__nv_bfloat16* row, const float* v, int first, int cols) {
#pragma unroll
    for (int j = 0; j < kN; ++j)
        if (j >= first && j < cols) row[j] = __float2bfloat16_rn(v[j]);
}

// 1 - Phi(|x|) = erfc(|x| / sqrt 2) / 2 and e^{-x^2/2}.  erfc(z) = e^{-z^2} t S(t) with t =
// 1 / (1 + z / 2); S is a polynomial fitted to a relative 1.4e-6 over z in [0, 10], beyond
// which the product is below the smallest bf16.  z^2 is rounded before the exponential, so
// the whole is good to 2e-6 up to |x| = 3 and 1.8e-5 at 13; results are rounded to bf16
// (3.9e-3).  Relative accuracy in the tail matters
// (x Phi(x) for negative x), so erf's absolute error bounds would not do.  At
// 16384 x 8192 x 2048 with a bias, GELU takes 411 us where no activation takes 385.
__device__ __forceinline__ float phi_tail(float x, float& gauss) {
    const float z = fabsf(x) * 0.70710678118654752f;
    const float t = mix::rcp(fmaf(0.5f, z, 1.f));
    gauss = mix::ex2(z * z * -1.4426950408889634f);
    float s = fmaf(0.08820453f, t, -0.35673877f);
    s = fmaf(s, t, 0.38922512f);
    s = fmaf(s, t, 0.03789042f);
    s = fmaf(s, t, 0.28150379f);
    s = fmaf(s, t, 0.27758215f);
    s = fmaf(s, t, 0.28233141f);
    return 0.5f * gauss * t * s;
}
__device__ __forceinline__ float gelu(float x) {
    float g;
    const float q = phi_tail(x, g);
    return x * (x > 0.f ? 1.f - q : q);
}
// Outputs and the residual pass once: stored and loaded as the first lines to leave L2,
// which W and the rows of x in flight need.
__device__ __forceinline__ uint64_t policy_evict_first() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ void tma_store_2d_once(const CUtensorMap* map, const void* src, int c0, int c1, uint64_t policy) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group.L2::cache_hint [%0, {%2, %3}], [%1], %4;" ::"l"(map),
                 "r"(smem_u32(src)), "r"(c0), "r"(c1), "l"(policy)
                 : "memory");
}

template <int kN>
__device__ __forceinline__ void apply_act(float* v, int act) {
    switch (act) {
        case kRelu:
#pragma unroll
            for (int j = 0; j < kN; ++j) v[j] = v[j] < 0.f ? 0.f : v[j];  // keeps NaN
            break;
        case kGelu:
#pragma unroll
            for (int j = 0; j < kN; ++j) v[j] = gelu(v[j]);
            break;
        case kSilu:
#pragma unroll
            for (int j = 0; j < kN; ++j) v[j] = mix::siluf(v[j]);
            break;
        case kSoftplus:
#pragma unroll
            for (int j = 0; j < kN; ++j) v[j] = mix::softplus_poly(v[j]);
            break;
        default: break;
    }
}

template <int kBN, bool kAMN, bool kBMN, bool kPre>
__global__ void __launch_bounds__(gemm::kThreads, 1)
    kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
           const __grid_constant__ CUtensorMap map_c, const __grid_constant__ CUtensorMap map_p, const LArgs p) {
    using P = LPlan<kBN>;
    constexpr int kStages = P::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(sm);
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + P::OFF_BARS);
    uint64_t* empty = full + kStages;
    uint64_t* acc_full = empty + kStages;
    uint64_t* acc_empty = acc_full + 2;
    uint32_t* sTmem = reinterpret_cast<uint32_t*>(acc_empty + 2);
    volatile int* sAbort = reinterpret_cast<volatile int*>(sTmem + 1);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int total = p.tiles_m * p.tiles_n;
    const int nkb = (p.K + BK - 1) / BK;

    if (warp == 0) {
        tmem_alloc(sTmem, 2 * kBN);
        tmem_relinquish();
    }
    if (tid == 32) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], kEpiWarps);
        }
        *sAbort = 0;
        fence_mbar_init();
    }
    if (tid == 64) {
        prefetch_tmap(&map_a);
        prefetch_tmap(&map_b);
        prefetch_tmap(&map_c);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *sTmem;

    if (warp == 0) {
        // ---------------------------------------------------------------- TMA producer
        if (lane == 0) {
            int stage = 0, issued = 0;  // issued: loads whose full barrier may still be pending at exit
            uint32_t phase = 0;
            for (int t = blockIdx.x; t < total && !*sAbort; t += gridDim.x) {
                const int m0 = (t / p.tiles_n) * BM, n0 = (t % p.tiles_n) * kBN;
                for (int kb = 0; kb < nkb; ++kb) {
                    if (!mbar_wait(&empty[stage], phase ^ 1, 8)) {
                        *sAbort = 1;
                        break;
                    }
                    uint8_t* sa = sm + stage * P::kStage;
                    uint8_t* sb = sa + kABytes;
                    mbar_arrive_expect_tx(&full[stage], P::kStage);
                    if constexpr (kAMN) {
#pragma unroll
                        for (int i = 0; i < BM / 64; ++i) tma_load_2d(sa + i * 8192, &map_a, &full[stage], m0 + 64 * i, kb * BK);
                    } else {
                        tma_load_2d(sa, &map_a, &full[stage], kb * BK, m0);
                    }
                    if constexpr (kBMN) {
#pragma unroll
                        for (int i = 0; i < kBN / 64; ++i) tma_load_2d(sb + i * 8192, &map_b, &full[stage], n0 + 64 * i, kb * BK);
                    } else {
                        tma_load_2d(sb, &map_b, &full[stage], kb * BK, n0);
                    }
                    ++issued;
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            if (*sAbort) {  // let every load this thread issued land before the CTA exits
                for (int s = 0; s < kStages && issued > 0; ++s, --issued) {
                    if (--stage < 0) {
                        stage = kStages - 1;
                        phase ^= 1;
                    }
                    mbar_wait(&full[stage], phase, 9);
                }
            }
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer
        if (lane == 0) {
            int stage = 0, i = 0;
            uint32_t phase = 0;
            bool pending = false;  // a commit whose barrier may not have arrived yet
            for (int t = blockIdx.x; t < total && !*sAbort; t += gridDim.x, ++i) {
                const int buf = i & 1;
                const uint32_t aph = (i >> 1) & 1;
                int nw = p.N - (t % p.tiles_n) * kBN;
                nw = nw >= kBN ? kBN : ((nw + 15) & ~15);
                const uint32_t idesc = idesc_bf16(BM, nw, kAMN, kBMN);
                if (!mbar_wait(&acc_empty[buf], aph ^ 1, 10)) {
                    *sAbort = 1;
                    break;
                }
                tc_fence_after();
                const uint32_t dtm = tbase + uint32_t(buf * kBN);
                for (int kb = 0; kb < nkb; ++kb) {
                    if (!mbar_wait(&full[stage], phase, 11)) {
                        *sAbort = 1;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = sbase + stage * P::kStage, sb = sa + kABytes;
#pragma unroll
                    for (int k = 0; k < BK / 16; ++k) {
                        const uint64_t da = kAMN ? sdesc_sw128(sa + k * 2048, 8192, 1024) : sdesc_sw128(sa + k * 32, 16, 1024);
                        const uint64_t db = kBMN ? sdesc_sw128(sb + k * 2048, 8192, 1024) : sdesc_sw128(sb + k * 32, 16, 1024);
                        umma_bf16(dtm, da, db, idesc, (kb | k) != 0);
                    }
                    umma_commit(&empty[stage]);
                    pending = true;
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (*sAbort) break;
                umma_commit(&acc_full[buf]);
            }
            if (*sAbort && pending) {  // the last MMAs still read shared memory: let them finish
                const int last = (stage + kStages - 1) % kStages;
                mbar_wait(&empty[last], stage == 0 ? phase ^ 1 : phase, 12);
            }
        }
    } else {
        // ---------------------------------------------------------------- epilogue
        const int ew = warp - 2;
        const int quad = warp & 3;   // TMEM lane quadrant this warp may read
        const int half = ew >> 2;    // column half of the tile (a 64-wide tile has one)
        constexpr int kChunks = kBN >= 128 ? kBN / 128 : 1;
        const uint64_t policy = policy_evict_first();
        const uint32_t stg = sbase + P::OFF_STAGING + uint32_t(ew) * P::kStagingBytes;
        uint8_t* stg_p = sm + P::OFF_STAGING + ew * P::kStagingBytes;
        int i = 0;
        for (int t = blockIdx.x; t < total; t += gridDim.x, ++i) {
            const int buf = i & 1;
            const uint32_t aph = (i >> 1) & 1;
            const int m0 = (t / p.tiles_n) * BM, n0 = (t % p.tiles_n) * kBN;
            const int row = m0 + quad * 32 + lane;  // output row of this thread
            const int cols = min(kBN, p.N - n0);    // valid columns of this tile
            // this thread's 64 residual values of a chunk, requested before the accumulator
            // is waited for: 128 contiguous bytes of its row
            uint4 res[8];
            auto load_res = [&](int c0) {
                if (p.res && row < p.M && p.res_vec) {
                    const __nv_bfloat16* r = p.res + (size_t)row * p.ldr + n0 + c0;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (c0 + 8 * j + 8 <= cols) res[j] = __ldcs(reinterpret_cast<const uint4*>(r) + j);
                }
            };
            const int h0 = kBN >= 128 ? half * (kBN / 2) : 0;
            if (h0 < cols) load_res(h0);
            const bool ok = mbar_wait(&acc_full[buf], aph, 13);
            if (__any_sync(0xffffffffu, !ok) || *sAbort) {
                *sAbort = 1;
                break;
            }
            tc_fence_after();
            const uint32_t tacc = tbase + uint32_t(buf * kBN) + (uint32_t(quad * 32) << 16);
#pragma unroll 1
            for (int ch = 0; ch < kChunks; ++ch) {
                const int c0 = h0 + ch * 64;  // tile column of this 64-wide chunk
                if (c0 >= cols || (kBN < 128 && half)) break;
                float v[64];
                tmem_ld32(tacc + c0, v);
                tmem_ld32(tacc + c0 + 32, v + 32);
                tmem_wait_ld();
                if (p.bias) {
                    const float* b = p.bias + n0 + c0;
                    if (c0 + 64 <= cols && (reinterpret_cast<uintptr_t>(b) & 15) == 0) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const float4 q = __ldg(reinterpret_cast<const float4*>(b) + j);
                            v[4 * j] += q.x;
                            v[4 * j + 1] += q.y;
                            v[4 * j + 2] += q.z;
                            v[4 * j + 3] += q.w;
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 64; ++j)
                            if (c0 + j < cols) v[j] += __ldg(b + j);
                    }
                }
                if (lane == 0) gemm::bulk_wait_read0();  // the previous stores have read the staging tiles
                __syncwarp();
                const int whole = (p.N & ~7) - (n0 + c0);  // chunk columns that the TMA store covers
                const bool ragged = whole < 64 && (p.N & 7) && row < p.M;
                uint32_t w32[32];
                if constexpr (kPre) {
                    if (ragged) store_ragged<64>(p.pre + (size_t)row * p.ldp + n0 + c0, v, whole, cols - c0);
#pragma unroll
                    for (int j = 0; j < 32; ++j) w32[j] = bf16x2_rn(v[2 * j], v[2 * j + 1]);
                    stage_row(stg, lane, w32);
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0 && whole > 0) {
                        tma_store_2d_once(&map_p, stg_p, n0 + c0, m0 + quad * 32, policy);
                        gemm::bulk_commit();
                    }
                }
                apply_act<64>(v, p.act);
                if (p.res && row < p.M) {
                    if (p.res_vec) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            if (c0 + 8 * j + 8 <= cols) {
                                float f[8];
                                mix::unpack16(res[j], f, __nv_bfloat16());
#pragma unroll
                                for (int u = 0; u < 8; ++u) v[8 * j + u] += f[u];
                            } else {
#pragma unroll
                                for (int u = 0; u < 8; ++u)
                                    if (c0 + 8 * j + u < cols)
                                        v[8 * j + u] += __bfloat162float(p.res[(size_t)row * p.ldr + n0 + c0 + 8 * j + u]);
                            }
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 64; ++j)
                            if (c0 + j < cols) v[j] += __bfloat162float(p.res[(size_t)row * p.ldr + n0 + c0 + j]);
                    }
                }
                if (ch + 1 < kChunks && c0 + 64 < cols) load_res(c0 + 64);
                if (ragged) store_ragged<64>(p.c + (size_t)row * p.ldc + n0 + c0, v, whole, cols - c0);
#pragma unroll
                for (int j = 0; j < 32; ++j) w32[j] = bf16x2_rn(v[2 * j], v[2 * j + 1]);
                if constexpr (kPre) {
                    if (lane == 0) gemm::bulk_wait_read0();  // the store of s has read the tile
                    __syncwarp();
                }
                stage_row(stg, lane, w32);
                fence_async_smem();
                __syncwarp();
                if (lane == 0 && whole > 0) {
                    tma_store_2d_once(&map_c, stg_p, n0 + c0, m0 + quad * 32, policy);
                    gemm::bulk_commit();
                }
            }
            // this warp has read its part of the accumulator: hand it back to the MMA warp
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[buf]);
        }
        if (lane == 0) gemm::bulk_wait0();  // every store of this warp has completed
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tbase, 2 * kBN);
}

// C [M, N] = A B^T summed over K.  K-major operands: A [M, K], B [N, K]; MN-major
// ones hold the summed axis as rows: A [K, M], B [K, N].
template <int kBN, bool kAMN, bool kBMN, bool kPre>
static int launch_tile(const void* A, int lda, const void* B, int ldb, void* C, int ldc, void* pre, int ldp, LArgs a,
                       cudaStream_t st, const char** why) {
    CUtensorMap ma, mb, mc, mp;
    const bool ok = (kAMN ? map_2d(&ma, A, false, a.K, a.M, lda, 64, BK) : map_2d(&ma, A, false, a.M, a.K, lda, BK, BM)) &&
                    (kBMN ? map_2d(&mb, B, false, a.K, a.N, ldb, 64, BK) : map_2d(&mb, B, false, a.N, a.K, ldb, BK, kBN)) &&
                    map_2d(&mc, C, false, a.M, a.N < 8 ? 8 : a.N & ~7, ldc, 64, 32) &&
                    (kPre ? map_2d(&mp, pre, false, a.M, a.N < 8 ? 8 : a.N & ~7, ldp, 64, 32) : (mp = mc, true));
    if (!ok) {
        *why = "cuTensorMapEncodeTiled failed for a GEMM operand";
        return KDA_ERR_CUDA;
    }
    a.c = static_cast<__nv_bfloat16*>(C);
    a.ldc = ldc;
    a.pre = static_cast<__nv_bfloat16*>(pre);
    a.ldp = ldp;
    a.tiles_m = (a.M + BM - 1) / BM;
    a.tiles_n = (a.N + kBN - 1) / kBN;
    const long long tiles = (long long)a.tiles_m * a.tiles_n;
    const int sms = device_sm_count(), grid = int(tiles < sms ? tiles : sms);
    auto kern = kernel<kBN, kAMN, kBMN, kPre>;
    constexpr uint32_t smem = LPlan<kBN>::kSmem;
    if (!set_smem_attr(kern, smem)) {
        *why = "cudaFuncSetAttribute failed for the GEMM kernel";
        return KDA_ERR_CUDA;
    }
    kern<<<grid, gemm::kThreads, smem, st>>>(ma, mb, mc, mp, a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) {
        *why = cudaGetErrorString(e);
        return KDA_ERR_CUDA;
    }
    return KDA_OK;
}

// Tile width by the SMs it fills: the cost of a width is its waves of tiles times the
// columns of a tile, plus what a tile costs whatever its width (the A operand's share
// of the loads).
static int tile_width(int M, int N) {
    const long long sms = device_sm_count(), tm = (M + BM - 1) / BM;
    int best = 256;
    long long least = 0;
    for (int bn = 256; bn >= 64; bn /= 2) {
        const long long waves = mix::cdiv(tm * ((N + bn - 1) / bn), sms), cost = waves * (bn + 64);
        if (bn == 256 || cost < least) {
            best = bn;
            least = cost;
        }
    }
    return best;
}

template <bool kAMN, bool kBMN, bool kPre>
static int launch(const void* A, int lda, const void* B, int ldb, void* C, int ldc, void* pre, int ldp, const LArgs& a,
                  cudaStream_t st, const char** why) {
    switch (tile_width(a.M, a.N)) {
        case 256: return launch_tile<256, kAMN, kBMN, kPre>(A, lda, B, ldb, C, ldc, pre, ldp, a, st, why);
        case 128: return launch_tile<128, kAMN, kBMN, kPre>(A, lda, B, ldb, C, ldc, pre, ldp, a, st, why);
        default: return launch_tile<64, kAMN, kBMN, kPre>(A, lda, B, ldb, C, ldc, pre, ldp, a, st, why);
    }
}

__device__ __forceinline__ float act1(float x, int act) {
    float v[1] = {x};
    apply_act<1>(v, act);
    return v[0];
}

// Few rows of x (decode): bound by reading W once.  A block has 16 rows of W (outputs);
// its warps take slices of K and add their sums in shared memory, in order.  Warp MMAs
// (m16n8k16) with W as the 16-row operand and up to 8 kMT rows of x as columns: the sum
// over k has no order, so a thread's fragments are 8 neighbouring values of its rows,
// 16 bytes that it copies into a ring of kU steps and reads back itself, with no
// exchange between threads.  (Loads into registers do not stay in flight: the compiler
// sinks them to their MMAs, 54 registers where kU steps would need 96.)  128-row tiles of
// the kernel above leave most SMs idle and 112 of 128 rows empty: 32 us at 16 x 2048 x 4096, here 6 to 8.
constexpr int kSkinnyWarps = 8;
template <int kMT>
struct Skinny {
    static constexpr int kU = kMT <= 2 ? 6 : (kMT == 4 ? 4 : 3), kV = 2 + kMT;  // steps in flight; vectors a thread copies per step
    static constexpr int kRing = kSkinnyWarps * kU * kV * 32 * 16, kRed = kSkinnyWarps * 16 * (8 * kMT + 1) * 4;
    static constexpr int kSmem = kRing > kRed ? kRing : kRed;  // (the sums reuse the ring)
};

template <int kMT>
__global__ void __launch_bounds__(32 * kSkinnyWarps)
    skinny_kernel(const __nv_bfloat16* __restrict__ x, int ldx, const __nv_bfloat16* __restrict__ W, int ldw,
                  const LArgs p) {
    constexpr int kU = Skinny<kMT>::kU, kV = Skinny<kMT>::kV;
    extern __shared__ __align__(16) uint8_t skinny_smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    uint4* ring = reinterpret_cast<uint4*>(skinny_smem) + (size_t)warp * kU * kV * 32 + lane;
    const int n0 = blockIdx.x * 16;
    // K in steps of 32 (8 values a thread), dealt to the warps in runs
    const int steps = (p.K + 31) / 32, per = (steps + kSkinnyWarps - 1) / kSkinnyWarps;
    const int s0 = warp * per, s1 = min(steps, s0 + per);
    float acc[kMT][4];
#pragma unroll
    for (int m = 0; m < kMT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][i] = 0.f;
    const bool in0 = n0 + g < p.N, in1 = n0 + g + 8 < p.N;
    const __nv_bfloat16 *w0 = W + (size_t)(n0 + g) * ldw, *w1 = W + (size_t)(n0 + g + 8) * ldw;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    auto request = [&](int s, int slot) {
        const int k = s * 32 + t * 8;
        uint4* v = ring + slot * kV * 32;
        if (s < s1) {
            const bool in = k < p.K;
            const int bytes = min(16, 2 * (p.K - k));  // (what a row holds after its K values is not read)
            if (in && in0) mix::cp_async_part(v, w0 + k, bytes);
            else v[0] = zero;
            if (in && in1) mix::cp_async_part(v + 32, w1 + k, bytes);
            else v[32] = zero;
#pragma unroll
            for (int m = 0; m < kMT; ++m) {
                if (in && m * 8 + g < p.M) mix::cp_async_part(v + (2 + m) * 32, x + (size_t)(m * 8 + g) * ldx + k, bytes);
                else v[(2 + m) * 32] = zero;
            }
        }
        mix::cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kU - 1; ++i) request(s0 + i, i);
    int slot = 0;
    for (int s = s0; s < s1; ++s) {
        mix::cp_async_wait<kU - 2>();
        const uint4* v = ring + slot * kV * 32;
        const uint4 a0 = v[0], a1 = v[32];
        uint4 b[kMT];
#pragma unroll
        for (int m = 0; m < kMT; ++m) b[m] = v[(2 + m) * 32];
        request(s + kU - 1, slot == 0 ? kU - 1 : slot - 1);  // into the place of the step before this one
        if (++slot == kU) slot = 0;
#pragma unroll
        for (int m = 0; m < kMT; ++m) {
            asm volatile(
                "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                : "+f"(acc[m][0]), "+f"(acc[m][1]), "+f"(acc[m][2]), "+f"(acc[m][3])
                : "r"(a0.x), "r"(a1.x), "r"(a0.y), "r"(a1.y), "r"(b[m].x), "r"(b[m].y));
            asm volatile(
                "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                : "+f"(acc[m][0]), "+f"(acc[m][1]), "+f"(acc[m][2]), "+f"(acc[m][3])
                : "r"(a0.z), "r"(a1.z), "r"(a0.w), "r"(a1.w), "r"(b[m].z), "r"(b[m].w));
        }
    }
    __syncthreads();  // every warp has used its ring
    float (*red)[16][8 * kMT + 1] = reinterpret_cast<float (*)[16][8 * kMT + 1]>(skinny_smem);
#pragma unroll
    for (int m = 0; m < kMT; ++m) {  // sums: rows g, g + 8 of W; columns (rows of x) 2t, 2t + 1
        red[warp][g][m * 8 + 2 * t] = acc[m][0];
        red[warp][g][m * 8 + 2 * t + 1] = acc[m][1];
        red[warp][g + 8][m * 8 + 2 * t] = acc[m][2];
        red[warp][g + 8][m * 8 + 2 * t + 1] = acc[m][3];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * 8 * kMT; i += 32 * kSkinnyWarps) {
        const int n = n0 + (i & 15), row = i >> 4;
        if (n >= p.N || row >= p.M) continue;
        float v = p.bias ? p.bias[n] : 0.f;
#pragma unroll
        for (int w = 0; w < kSkinnyWarps; ++w) v += red[w][i & 15][row];
        if (p.pre) p.pre[(size_t)row * p.ldp + n] = __float2bfloat16_rn(v);
        v = act1(v, p.act);
        if (p.res) v += __bfloat162float(p.res[(size_t)row * p.ldr + n]);
        p.c[(size_t)row * p.ldc + n] = __float2bfloat16_rn(v);
    }
}

template <int kMT>
static int launch_skinny(const void* x, int ldx, const void* W, int ldw, const LArgs& a, cudaStream_t st,
                         const char** why) {
    if (!set_smem_attr(skinny_kernel<kMT>, Skinny<kMT>::kSmem)) {
        *why = "cudaFuncSetAttribute failed for the skinny kernel";
        return KDA_ERR_CUDA;
    }
    skinny_kernel<kMT><<<unsigned(mix::cdiv(a.N, 16)), 32 * kSkinnyWarps, Skinny<kMT>::kSmem, st>>>(
        static_cast<const __nv_bfloat16*>(x), ldx, static_cast<const __nv_bfloat16*>(W), ldw, a);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) return KDA_OK;
    *why = cudaGetErrorString(e);
    return KDA_ERR_CUDA;
}

__device__ __forceinline__ float dact(float x, int act) {
    switch (act) {
        case kRelu: return x > 0.f ? 1.f : 0.f;
        case kGelu: {
            float g;
            const float q = phi_tail(x, g);
            return (x > 0.f ? 1.f - q : q) + x * 0.39894228040143268f * g;
        }
        case kSilu: {
            const float g = mix::sigmoidf(x);
            return g * (1.f + x * (1.f - g));
        }
        case kSoftplus: return mix::sigmoidf(x);
        default: return 1.f;
    }
}

// ds = dy act'(s) in bf16 (when ds is not NULL) and its column sums over a run of
// rows, part[blockIdx.y][N], summed from the unrounded values.  A block: 32 vectors
// of 8 columns by 8 rows.  Bound by HBM.
template <bool kVec>
__global__ void __launch_bounds__(256)
    act_grad_kernel(const __nv_bfloat16* __restrict__ dy, long long lddy, const __nv_bfloat16* __restrict__ s,
                    long long lds, __nv_bfloat16* __restrict__ ds, long long ldds, float* __restrict__ part, int M, int N,
                    int rows_per_block, int act) {
    using V = mix::Raw<__nv_bfloat16, kVec>;
    constexpr int kE = kVec ? 8 : 1;
    __shared__ float red[8][32 * kE + 1];
    const int lane = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int c0 = (blockIdx.x * 32 + lane) * kE;
    const long long r0 = (long long)blockIdx.y * rows_per_block;
    const long long r1 = r0 + rows_per_block < M ? r0 + rows_per_block : M;
    float sum[kE];
#pragma unroll
    for (int u = 0; u < kE; ++u) sum[u] = 0.f;
    if (c0 < N) {
        // four rows' loads before the first is used
        constexpr int kU = 4;
        for (long long rb = r0 + ty; rb < r1; rb += 8 * kU) {
            V vd[kU], vs[kU];
#pragma unroll
            for (int i = 0; i < kU; ++i) {
                const long long r = rb + 8 * i;
                if (r < r1) {
                    vd[i].load_stream(dy + r * lddy + c0);
                    if (act != kNone) vs[i].load_stream(s + r * lds + c0);
                }
            }
#pragma unroll
            for (int i = 0; i < kU; ++i) {
                const long long r = rb + 8 * i;
                if (r >= r1) break;
                float d[kE], x[kE];
                vd[i].get(d);
                if (act != kNone) {
                    vs[i].get(x);
#pragma unroll
                    for (int u = 0; u < kE; ++u) d[u] *= dact(x[u], act);
                }
#pragma unroll
                for (int u = 0; u < kE; ++u) sum[u] += d[u];
                if (ds) {
                    vd[i].set(d);
                    vd[i].store(ds + r * ldds + c0);
                }
            }
        }
    }
    if (!part) return;
#pragma unroll
    for (int u = 0; u < kE; ++u) red[ty][u * 32 + lane] = sum[u];
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * kE; i += 256) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) t += red[k][i];
        const int c = (blockIdx.x * 32 + (i & 31)) * kE + (i >> 5);
        if (c < N) part[(size_t)blockIdx.y * N + c] = t;
    }
}

// Rows per block of act_grad_kernel: a multiple of 32 that makes one wave of 2 blocks an SM.
static int grad_rows(int M, int N, int kE) {
    const long long cols = mix::cdiv(N, 32 * kE), fit = (long long)device_sm_count() * 2 / cols;
    return int(mix::cdiv(mix::cdiv(M, fit > 0 ? fit : 1), 32) * 32);
}

}  // namespace lin

int launch_linear_act(const void* x, int ldx, const void* W, int ldw, const float* bias, const void* res, int ldr,
                      void* y, int ldy, void* pre, int ldp, int M, int N, int K, int act, cudaStream_t st,
                      const char** why) {
    lin::LArgs a{};
    a.M = M;
    a.N = N;
    a.K = K;
    a.bias = bias;
    a.res = static_cast<const __nv_bfloat16*>(res);
    a.ldr = ldr;
    a.res_vec = res && mix::al16(res) && ldr % 8 == 0;
    a.act = act;
    // Up to 32 rows: the skinny kernel.  Up to 64 it pays while 64-wide tiles leave half of the
    // SMs idle (64 x 2048 x 4096: 14 against 28 us; 64 x 8192 x 2048: 34 against 17 us).
    if (M <= 32 || (M <= 64 && 2 * mix::cdiv(N, 64) <= device_sm_count())) {
        a.c = static_cast<__nv_bfloat16*>(y);
        a.ldc = ldy;
        a.pre = static_cast<__nv_bfloat16*>(pre);
        a.ldp = ldp;
        if (M <= 8) return lin::launch_skinny<1>(x, ldx, W, ldw, a, st, why);
        if (M <= 16) return lin::launch_skinny<2>(x, ldx, W, ldw, a, st, why);
        if (M <= 32) return lin::launch_skinny<4>(x, ldx, W, ldw, a, st, why);
        return lin::launch_skinny<8>(x, ldx, W, ldw, a, st, why);
    }
    if (pre) return lin::launch<false, false, true>(x, ldx, W, ldw, y, ldy, pre, ldp, a, st, why);
    return lin::launch<false, false, false>(x, ldx, W, ldw, y, ldy, nullptr, 0, a, st, why);
}

struct LinearBwdPlan {
    int ldds;
    size_t off_part, total;
};
static LinearBwdPlan linear_bwd_plan(int M, int N) {
    LinearBwdPlan p{};
    p.ldds = (N + 7) & ~7;
    p.off_part = mix::up256(size_t(M) * p.ldds * 2);
    size_t parts = 0;  // the more blocks of either vector width
    for (int e = 1; e <= 8; e += 7) {
        const size_t n = size_t(mix::cdiv(M, lin::grad_rows(M, N, e)));
        if (n > parts) parts = n;
    }
    p.total = p.off_part + mix::up256(parts * N * sizeof(float));
    return p;
}
size_t linear_act_bwd_workspace_bytes(int M, int N) { return linear_bwd_plan(M, N).total; }

int launch_linear_act_bwd(const void* dy, int lddy, const void* x, int ldx, const void* W, int ldw, const void* pre,
                          int ldp, void* dx, int lddx, void* dW, int lddw, float* dbias, int M, int N, int K, int act,
                          void* ws, cudaStream_t st, const char** why) {
    using bf16 = __nv_bfloat16;
    const LinearBwdPlan pl = linear_bwd_plan(M, N);
    uint8_t* b = static_cast<uint8_t*>(ws);
    // dy itself is the operand when there is no activation and TMA can read it
    const bool direct = act == KDA_ACT_NONE && mix::al16(dy) && lddy % 8 == 0;
    bf16* ds = direct ? nullptr : reinterpret_cast<bf16*>(b);
    float* part = dbias ? reinterpret_cast<float*>(b + pl.off_part) : nullptr;
    const bool vec = N % 8 == 0 && mix::al16(dy) && lddy % 8 == 0 && (!pre || (mix::al16(pre) && ldp % 8 == 0));
    if (ds || part) {
        const int kE = vec ? 8 : 1, rows = lin::grad_rows(M, N, kE);
        const int parts = int(mix::cdiv(M, rows));
        const dim3 grid(unsigned(mix::cdiv(N, 32 * kE)), parts);
        const bf16 *d = static_cast<const bf16*>(dy), *s = static_cast<const bf16*>(pre);
        if (vec) lin::act_grad_kernel<true><<<grid, 256, 0, st>>>(d, lddy, s, ldp, ds, pl.ldds, part, M, N, rows, act);
        else lin::act_grad_kernel<false><<<grid, 256, 0, st>>>(d, lddy, s, ldp, ds, pl.ldds, part, M, N, rows, act);
        if (part)
            mix::sum_parts<float>(part, parts, N, dbias, nullptr, N, st);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) {
            *why = cudaGetErrorString(e);
            return KDA_ERR_CUDA;
        }
    }
    const void* op = direct ? dy : ds;
    const int ldop = direct ? lddy : pl.ldds;
    lin::LArgs a{};
    if (dx) {  // [M, K] = ds [M, N] W [N, K]
        a.M = M;
        a.N = K;
        a.K = N;
        const int rc = lin::launch<false, true, false>(op, ldop, W, ldw, dx, lddx, nullptr, 0, a, st, why);
        if (rc != KDA_OK) return rc;
    }
    if (dW) {  // [N, K] = ds^T [N, M] x [M, K]
        a.M = N;
        a.N = K;
        a.K = M;
        const int rc = lin::launch<true, true, false>(op, ldop, x, ldx, dW, lddw, nullptr, 0, a, st, why);
        if (rc != KDA_OK) return rc;
    }
    return KDA_OK;
}

}  // namespace kda
