// Hybrid dense / 2:4 product in 8-bit integers on single CTAs:
// Y[m,n] = (sum_k Xq[m,k] * (Wq (.) Mask)[n,k]) * x_scale[m] * w_scale[n].
//
// The bf16 kernels' method (dense slabs on tcgen05.mma, 2:4 slabs on
// tcgen05.mma.sp, the weight as operand A; PATCH abstract, "PATCH: Learnable
// Tile-level Hybrid Sparsity for LLMs") with kind::i8: int8 operands and
// int32 sums, which are exact (the host keeps K * 128 * 128 below 2^31). The
// two scales are applied once per output in fp32, before the one rounding to
// the output type.
//
// One persistent CTA per SM walks a list of output tiles (strip of 128 weight
// rows, block of up to 128 tokens): warp 0 streams each 128-column slab and its
// activation tile with TMA, warp 1 issues the MMAs into one of two TMEM
// accumulators, warps 2..5 drain the other one. All waits are bounded.
#include <cuda_fp16.h>

#include "q8.cuh"
#include "q8_mma.cuh"

namespace patch {

namespace {

constexpr int kThreads = 192;
constexpr int kBN = kGemmBN;                      // tokens per tile, at most
constexpr int kStageA = 18432;                    // 16 KB dense, or 8 KB codes + 2 KB metadata
constexpr int kStageB = kBN * 128;
constexpr int kStages = 6;
constexpr int kECol = 2 * kBN;                    // 4 metadata columns after the accumulators
constexpr int kTmemCols = 512;
constexpr int kSmemData = kStages * (kStageA + kStageB);
constexpr int kSmemBytes = kSmemData + 1024 /*align*/ + 256 /*barriers*/;

template <class T>
__device__ __forceinline__ T out_cast(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 out_cast(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half out_cast(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float out_cast(float v) { return v; }

template <class T>
__global__ void __launch_bounds__(kThreads, 1)
    q8_gemm_kernel(const __grid_constant__ GroupMaps maps, const __grid_constant__ Q8Args a, const int n_tok) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    uint8_t* sA = smem;
    uint8_t* sB = smem + kStages * kStageA;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kSmemData);
    uint64_t* full = bars;
    uint64_t* empty = bars + kStages;
    uint64_t* acc_full = bars + 2 * kStages;
    uint64_t* acc_empty = acc_full + 2;
    uint64_t* drain = acc_full + 4;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 4);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    auto raise = [&]() {
        *abort_flag = 1;
        atomicCAS(a.status, 0, kStatusTimeout);
    };
    const int w_begin = a.work_off[blockIdx.x];
    const int w_end = a.work_off[blockIdx.x + 1];

    if (warp == 0) {
        if (lane == 0) {
            // ---------------- producer ----------------
            int stage = 0, issued = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int it = w_begin; it < w_end && ok; ++it) {
                const int u = a.work[it];
                const int l = u >> kUnitShift, lu = u & kUnitMask;
                const LinDesc& L = a.lins[l];
                const int s = lu / a.MB, j = lu % a.MB, KB = L.KB;
                const uint32_t* trow = L.slab + (size_t)s * KB;
                const uint32_t* mrow = L.meta + (size_t)s * KB;
                uint32_t d_next = trow[0];
                for (int b = 0; b < KB; ++b) {
                    const uint32_t d = d_next;
                    if (b + 1 < KB) d_next = trow[b + 1];  // fetched one slab ahead
                    if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag)) {
                        raise();
                        ok = false;
                        break;
                    }
                    const bool sp = d & kSlabSparse;
                    mbar_arrive_expect_tx(&full[stage], (sp ? kSparseValBytes + kMetaBytes : kDenseSlabBytes) +
                                                            (uint32_t)n_tok * 128u);
                    tma_load_2d(sA + stage * kStageA, sp ? &maps.a8[l] : &maps.a16[l], &full[stage], 0,
                                (int)(slab_offset_bytes(d) >> 7));
                    if (sp)
                        tma_load_2d(sA + stage * kStageA + kSparseValBytes, &maps.e[l], &full[stage], 0,
                                    (int)(mrow[b] >> 3));
                    tma_load_2d(sB + stage * kStageB, &maps.x[l], &full[stage], b * kQ8SlabK, j * kBN);
                    ++issued;
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // Wait (bounded, whatever the abort flag says) for the copies still
            // in flight so none lands after this CTA exits.
            for (int i = 0; i < kStages && i < issued; ++i) {
                if (--stage < 0) {
                    stage = kStages - 1;
                    phase ^= 1u;
                }
                const uint64_t t0 = globaltimer();
                while (!mbar_try_wait(&full[stage], phase) && globaltimer() - t0 < kWaitLimitNs) {
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // ---------------- MMA issuer ----------------
            const uint32_t idesc_d = idesc_i8(128, n_tok, false);
            const uint32_t idesc_s = idesc_i8(128, n_tok, true);
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true, any_mma = false;
            int t = 0;
            for (int it = w_begin; it < w_end && ok; ++it, ++t) {
                const int u = a.work[it];
                const LinDesc& L = a.lins[u >> kUnitShift];
                const int KB = L.KB;
                const uint32_t* trow = L.slab + (size_t)((u & kUnitMask) / a.MB) * KB;
                const int acc = t & 1;
                if (!mbar_wait(&acc_empty[acc], ((t >> 1) & 1) ^ 1u, abort_flag)) {
                    raise();
                    break;
                }
                tc_fence_after();
                uint32_t d_next = trow[0];
                for (int b = 0; b < KB; ++b) {
                    const uint32_t d = d_next;
                    if (b + 1 < KB) d_next = trow[b + 1];
                    if (!mbar_wait(&full[stage], phase, abort_flag)) {
                        raise();
                        ok = false;
                        break;
                    }
                    const uint32_t a_addr = smem_u32(sA + stage * kStageA);
                    const bool sp = d & kSlabSparse;
                    if (sp)
                        tc_cp_128x128b(tmem_base + kECol, smem_desc(a_addr + kSparseValBytes, 16, 128, kLayoutNone));
                    issue_slab_i8(sp, b == 0, a_addr, smem_u32(sB + stage * kStageB), tmem_base + (uint32_t)(acc * kBN),
                                  tmem_base + kECol, idesc_d, idesc_s);
                    any_mma = true;
                    tc_commit(&empty[stage]);
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                tc_commit(&acc_full[acc]);
            }
            if (*abort_flag && any_mma) {
                // Let issued MMAs finish before TMEM is released.
                tc_commit(drain);
                const uint64_t t0 = globaltimer();
                while (!mbar_try_wait(drain, 0) && globaltimer() - t0 < kWaitLimitNs) {
                }
            }
        }
    } else {
        // ---------------- epilogue (warps 2..5) ----------------
        const int q = warp & 3;  // TMEM lane quadrant this warp may access
        int t = 0;
        for (int it = w_begin; it < w_end; ++it, ++t) {
            const int u = a.work[it];
            const int l = u >> kUnitShift, lu = u & kUnitMask;
            const int s = lu / a.MB, j = lu % a.MB, acc = t & 1;
            const int n = s * kStrip + q * 32 + lane;
            const float sw = a.w_scale[l][n];
            const float* xs = a.x_scale[l];
            T* yc = static_cast<T*>(a.Y[l]) + n;
            const int64_t ldy = a.ldy[l];
            if (!mbar_wait(&acc_full[acc], (t >> 1) & 1, abort_flag)) {
                if (lane == 0) raise();
                break;
            }
            tc_fence_after();
            const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * kBN);
#pragma unroll 1
            for (int c0 = 0; c0 < n_tok; c0 += 16) {
                const int m0 = j * kBN + c0;
                if (m0 >= a.M) break;
                uint32_t v[16];
                tmem_ld_32x32b_x16(taddr + c0, v);
                tc_wait_ld();
#pragma unroll
                for (int c = 0; c < 16; ++c)
                    if (m0 + c < a.M) yc[(m0 + c) * ldy] = out_cast<T>((float)(int)v[c] * xs[m0 + c] * sw);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[acc]);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, kTmemCols);
    }
}

}  // namespace

cudaError_t q8_prepare_single() {
    cudaError_t e = cudaFuncSetAttribute(q8_gemm_kernel<__nv_bfloat16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kSmemBytes);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(q8_gemm_kernel<__half>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(q8_gemm_kernel<float>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    return e;
}

cudaError_t launch_q8_gemm(const GroupMaps& maps, const Q8Args& a, int y_type, int n_tok, int grid, cudaStream_t st) {
    if (y_type == kBf16)
        q8_gemm_kernel<__nv_bfloat16><<<grid, kThreads, kSmemBytes, st>>>(maps, a, n_tok);
    else if (y_type == kFp16)
        q8_gemm_kernel<__half><<<grid, kThreads, kSmemBytes, st>>>(maps, a, n_tok);
    else
        q8_gemm_kernel<float><<<grid, kThreads, kSmemBytes, st>>>(maps, a, n_tok);
    return cudaGetLastError();
}

}  // namespace patch
