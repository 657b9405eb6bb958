// Hybrid dense / 2:4 product in 8-bit integers, K split over a cluster:
// Y[m,n] = (sum_k Xq[m,k] * (Wq (.) Mask)[n,k]) * x_scale[m] * w_scale[n].
//
// The bf16 kernels' method (dense slabs on tcgen05.mma, 2:4 slabs on
// tcgen05.mma.sp, the weight as operand A; PATCH abstract, "PATCH: Learnable
// Tile-level Hybrid Sparsity for LLMs") with kind::i8: int8 operands and
// int32 sums, which are exact (the host keeps K * 128 * 128 below 2^31). The
// two scales are applied once per output in fp32, before the one rounding to
// the output type.
//
// For few tokens the call is bound by the weight bytes it streams, and for one
// linear by latency: 12 MB arrive in 2 us, less than a launch takes. So every
// unit (strip of 128 weight rows, tile of up to BN tokens) is one cluster of P
// CTAs, each with 1/P of the K axis, enough of them that nearly all of the
// weight is in flight at once. There is no work list, no workspace and no
// counter: a CTA finds its unit from its block index, its slab records in one
// load, and the P partial sums meet in distributed shared memory, where each
// CTA adds up its share of the unit and stores it, 4 rows of a token at a time
// (whole 128-row runs per token). Integer sums do not depend on the order.
//
// With programmatic dependent launch the set-up and the first weight loads
// run while the previous kernel of the stream finishes; activations and
// scales are read, and Y written, after griddepcontrol.wait.
//
// Warp 0 streams slabs and activation tiles with TMA, warp 1 issues the MMAs,
// warps 2..5 move the accumulator to shared memory, all warps add up. All
// waits are bounded.
#include <cuda_fp16.h>

#include "q8.cuh"
#include "q8_mma.cuh"

namespace patch {

namespace {

constexpr int kThreads = 192;
constexpr int kStageA = 16384;  // a dense record, or a 2:4 one (10 KB)

template <int BN, int STAGES, int CTAS>
struct Cfg {
    static constexpr int kStage = kStageA + BN * 128;
    static constexpr int kSmemData = STAGES * kStage;
    static constexpr int kSmemBytes = kSmemData + 1024 /*align*/ + 256 /*barriers*/ + (BN + kStrip) * 4 /*scales*/;
    static constexpr int kTmemCols = BN + 4 <= 32 ? 32 : BN + 4 <= 64 ? 64 : BN + 4 <= 128 ? 128 : 256;
    static_assert(kStage % 1024 == 0, "stages keep the 1024-byte swizzle alignment");
    static_assert(BN * 128 * 4 <= kSmemData, "the partial sums fit in the stages");
    static_assert(kTmemCols * CTAS <= 512, "TMEM columns of the resident CTAs");
    static_assert(CTAS * (kSmemBytes + 1024) <= 228 * 1024, "shared memory of the resident CTAs");
};

__device__ __forceinline__ int4 ld_cluster(uint32_t addr) {
    int4 v;
    asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// Four consecutive rows of one token.
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void store4(__half* p, float4 v) {
    const __half2 a = __floats2half2_rn(v.x, v.y), b = __floats2half2_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }

// This CTA's share of a unit's items (int4 at the same place in every CTA of the
// cluster, at most ITEMS of them): their sums over the P CTAs, handed to store().
//
// No CTA leaves while another may still read its sums: a warp arrives at the last
// barrier of the cluster only once all that it reads is in its registers, and stores
// behind the arrival. Nothing has to be visible behind this barrier, so the arrival
// is a relaxed one, and what keeps it behind the reads is its predicate, which is
// computed from every word read (zero: an argument that is 0, which the compiler
// does not know). An arrival with release waits for a fence instead: 4.5 us for 4.0
// at 16 x 4096 x 4096, 3.3 for 2.9 at 16 x 512 x 2048, 11.9 for 11.3 at 100 x 4096 x 11008.
template <int P, int ITEMS, class Store>
__device__ __forceinline__ void join(uint32_t base, int rank, int items, uint32_t zero, Store store) {
    constexpr int kAtOnce = P <= 6 ? 12 / P : 1;  // up to twelve reads under way at a time
    constexpr int kStep = P * kThreads;
    constexpr int kEach = (ITEMS + kStep - 1) / kStep;
    uint32_t from[P];
#pragma unroll
    for (int p = 0; p < P; ++p) from[p] = map_to_rank(base, p);
    const int i0 = rank * kThreads + (int)threadIdx.x;
    int4 sum[kEach];
    uint32_t seen = 0;
#pragma unroll
    for (int k0 = 0; k0 < kEach; k0 += kAtOnce) {
        int4 v[kAtOnce][P];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const int i = i0 + (k0 + k) * kStep;
            if (k0 + k < kEach && i < items)
#pragma unroll
                for (int p = 0; p < P; ++p) v[k][p] = ld_cluster(from[p] + (uint32_t)i * 16u);
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            if (k0 + k >= kEach || i0 + (k0 + k) * kStep >= items) continue;
            int4 t = v[k][0];
#pragma unroll
            for (int p = 1; p < P; ++p) t = make_int4(t.x + v[k][p].x, t.y + v[k][p].y, t.z + v[k][p].z, t.w + v[k][p].w);
            sum[k0 + k] = t;
            seen |= (uint32_t)(t.x | t.y | t.z | t.w);
        }
    }
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.eq.u32 p, %0, 0;\n\t"
        "@p barrier.cluster.arrive.relaxed.aligned;\n\t}" ::"r"(__reduce_or_sync(0xffffffffu, seen & zero))
        : "memory");
#pragma unroll
    for (int k = 0; k < kEach; ++k)
        if (i0 + k * kStep < items) store(i0 + k * kStep, sum[k]);
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int BN, int STAGES, int CTAS, int G, class T>
__global__ void __launch_bounds__(kThreads, CTAS)
    q8_split_kernel(const __grid_constant__ Q8Maps<G> maps, const __grid_constant__ Q8SplitArgs<G> a) {
    using C = Cfg<BN, STAGES, CTAS>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kSmemData);
    uint64_t* empty = full + STAGES;
    uint64_t* acc_full = empty + STAGES;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_full + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    float* s_sw = reinterpret_cast<float*>(smem + C::kSmemData + 256);  // [kStrip] the rows' scales
    float* s_sx = s_sw + kStrip;                                        // [BN] the tokens' scales

    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);  // known to be uniform
    const int lane = threadIdx.x & 31;
    const int P = a.P;
    const int rank = (int)blockIdx.x % P;
    const int unit = (int)blockIdx.x / P;
    int l = 0;
    if (G > 1)
        while (l + 1 < a.n && unit >= a.m[l + 1].unit0) ++l;
    const Q8Member& L = a.m[l];
    const int lu = unit - L.unit0;
    const int s = lu / a.MB, m0 = (lu % a.MB) * a.n_tok;
    const int b0 = (int)((int64_t)rank * L.KB / P), nb = (int)((int64_t)(rank + 1) * L.KB / P) - b0;

    // the CTA's slab records, a lane each, fetched while the barriers are set up
    const uint32_t* drow = L.slab + (size_t)s * L.KB + b0;
    uint32_t d_now = 0, d_next = 0;
    if (warp <= 1) {
        if (lane < nb) d_now = drow[lane];
        if (32 + lane < nb) d_next = drow[32 + lane];
    }
    if (threadIdx.x == 64) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        mbar_init(acc_full, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    auto raise = [&]() {
        *abort_flag = 1;
        atomicCAS(a.status, 0, kStatusTimeout);
    };
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (warp == 0) {
        // ---------------- producer ----------------
        // Weights first out of L2, which leaves the activations in it, and what the
        // neighbours of this call left. Five layers' weights in turn, with the hint and
        // without: 100 x 11008 x 4096 9.9 and 11.0 us, 16 tokens 8.0 and 8.6; where the
        // five fit in L2 (4096 x 4096) it costs 1 %, but a model's weights do not.
        const uint64_t pol_w = policy_evict_first();
        auto load_w = [&](int i, uint32_t d) {
            const int st = i % STAGES;
            uint8_t* dst = smem + st * C::kStage;
            const bool sp = d & kSlabSparse;
            mbar_arrive_expect_tx(&full[st], q8_record_bytes(d) + (uint32_t)a.n_tok * 128u);
            const CUtensorMap* map = sp ? &maps.a10[l] : &maps.a16[l];
            const int at = (int)(slab_offset_bytes(d) >> 7);
            tma_load_2d_hint(dst, map, &full[st], 0, at, pol_w);
        };
        auto load_x = [&](int i) {
            const int st = i % STAGES;
            tma_load_2d(smem + st * C::kStage + kStageA, &maps.x[l], &full[st], (b0 + i) * kQ8SlabK, m0);
        };
        const int ahead = min(STAGES, nb);
        for (int i = 0; i < ahead; ++i) {
            const uint32_t d = __shfl_sync(0xffffffffu, d_now, i);
            if (lane == 0) load_w(i, d);
        }
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if (lane == 0)
            for (int i = 0; i < ahead; ++i) load_x(i);
        __syncwarp();
        int i = ahead;
        for (; i < nb; ++i) {
            if (i % 32 == 0) {
                d_now = d_next;
                if (i + 32 + lane < nb) d_next = drow[i + 32 + lane];
            }
            const uint32_t d = __shfl_sync(0xffffffffu, d_now, i % 32);
            const bool ok = mbar_wait(&empty[i % STAGES], (uint32_t)((i / STAGES) & 1) ^ 1u, abort_flag);
            if (!__all_sync(0xffffffffu, ok)) {
                if (lane == 0) raise();
                break;
            }
            if (lane == 0) {
                load_w(i, d);
                load_x(i);
            }
            __syncwarp();
        }
        // Wait (bounded, whatever the abort flag says) for the copies still in
        // flight so none lands after this CTA exits.
        if (lane == 0)
            for (int k = max(0, i - STAGES); k < i; ++k) {
                const uint64_t t0 = globaltimer();
                while (!mbar_try_wait(&full[k % STAGES], (uint32_t)((k / STAGES) & 1)) &&
                       globaltimer() - t0 < kWaitLimitNs) {
                }
            }
    } else if (warp == 1) {
        // ---------------- MMA issuer: the whole warp, one elected lane issuing ----------------
        const uint32_t el = elect();
        const uint32_t idesc_d = idesc_i8(128, a.n_tok, false);
        const uint32_t idesc_s = idesc_i8(128, a.n_tok, true);
        const uint32_t e_col = tmem_base + BN;
        const uint32_t ring0 = smem_u32(smem);
        uint32_t kinds = 0, st = 0, phase = 0;
        for (int i = 0; i < nb; ++i) {
            if (i % 32 == 0) {
                if (i > 0) {
                    d_now = d_next;
                    if (i + 32 + lane < nb) d_next = drow[i + 32 + lane];
                }
                kinds = __ballot_sync(0xffffffffu, d_now & kSlabSparse);
            }
            if (!__all_sync(0xffffffffu, mbar_wait(&full[st], phase, abort_flag))) {
                if (lane == 0) raise();
                break;
            }
            const uint32_t a_addr = ring0 + st * (uint32_t)C::kStage;
            issue_slab_i8<false>(el, (kinds >> (i % 32)) & 1u, i == 0, a_addr, a_addr + kStageA, tmem_base, e_col,
                                 idesc_d, idesc_s);
            commit_el(el, &empty[st]);
            if (++st == STAGES) {
                st = 0;
                phase ^= 1u;
            }
        }
        // after a timeout this still covers the MMAs that were issued
        commit_el(el, acc_full);
        __syncwarp();
        asm volatile("griddepcontrol.wait;" ::: "memory");
    } else {
        // ---------------- accumulator -> shared memory (the stages are free) ----------------
        asm volatile("griddepcontrol.wait;" ::: "memory");
        const int q = warp & 3;  // TMEM lane quadrant this warp may access
        const int tokens = min(a.n_tok, a.M - m0);
        {
            const int t = (int)threadIdx.x - 64;
            s_sw[t] = L.w_scale[s * kStrip + t];
            if (t < tokens) s_sx[t] = L.x_scale[m0 + t];
        }
        int* part = reinterpret_cast<int*>(smem) + q * 32 + lane;  // [token][row]
        bool ok = mbar_try_wait(acc_full, 0);
        const uint64_t t0 = globaltimer();
        while (!ok && globaltimer() - t0 < 2 * kWaitLimitNs) ok = mbar_try_wait(acc_full, 0);
        if (__all_sync(0xffffffffu, ok)) {  // (the limit may pass between two lanes' tries)
            tc_fence_after();
            for (int c0 = 0; c0 < tokens; c0 += 16) {
                uint32_t v[16];
                tmem_ld_32x32b_x16(tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)c0, v);
                tc_wait_ld();
#pragma unroll
                for (int c = 0; c < 16; ++c)
                    if (c0 + c < tokens) part[(c0 + c) * kStrip] = (int)v[c];
            }
        } else if (lane == 0) {
            raise();
        }
        tc_fence_before();
    }

    // ---------------- sum over the cluster ----------------
    __syncwarp();
    if (P > 1)
        cluster_sync();
    else
        __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, C::kTmemCols);
    }
    const int items = min(a.n_tok, a.M - m0) * (kStrip / 4);
    T* y0 = static_cast<T*>(L.Y) + (int64_t)m0 * L.ldy + (int64_t)s * kStrip;
    auto store = [&](int i, int4 sum) {
        const int tok = i / (kStrip / 4), row = (i % (kStrip / 4)) * 4;
        const float sx = s_sx[tok];
        const float4 sw = *reinterpret_cast<const float4*>(s_sw + row);
        store4(y0 + tok * L.ldy + row, make_float4((float)sum.x * sx * sw.x, (float)sum.y * sx * sw.y,
                                                   (float)sum.z * sx * sw.z, (float)sum.w * sx * sw.w));
    };
    if (P == 1) {
#pragma unroll 4
        for (int i = (int)threadIdx.x; i < items; i += kThreads)
            store(i, *reinterpret_cast<const int4*>(smem + (size_t)i * 16));
    } else {
        // (Reading, at about 20 bytes a cycle and SM, is the fastest way found: sums
        // stored straight to the CTA that joins them took 10 to 15 % longer, sums sent
        // by bulk copies 10 %, added in place by bulk copies 20 to 30 %.)
        const uint32_t base = smem_u32(smem);
        constexpr int kItems = BN * (kStrip / 4);
        switch (P) {
            case 2: join<2, kItems>(base, rank, items, a.zero, store); break;
            case 3: join<3, kItems>(base, rank, items, a.zero, store); break;
            case 4: join<4, kItems>(base, rank, items, a.zero, store); break;
            case 5: join<5, kItems>(base, rank, items, a.zero, store); break;
            case 6: join<6, kItems>(base, rank, items, a.zero, store); break;
            case 7: join<7, kItems>(base, rank, items, a.zero, store); break;
            default: join<8, kItems>(base, rank, items, a.zero, store); break;
        }
    }
}

template <int BN, int STAGES, int CTAS, int G, class T>
cudaError_t prepare() {
    return cudaFuncSetAttribute(q8_split_kernel<BN, STAGES, CTAS, G, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Cfg<BN, STAGES, CTAS>::kSmemBytes);
}

template <int BN, int STAGES, int CTAS, int G, class T>
cudaError_t launch(const Q8Maps<G>& maps, const Q8SplitArgs<G>& a, int grid, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = Cfg<BN, STAGES, CTAS>::kSmemBytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.P;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, q8_split_kernel<BN, STAGES, CTAS, G, T>, maps, a);
}

#define Q8_SPLIT_CONFIGS(X) X(0) X(1) X(2) X(3) X(4)
static_assert(sizeof(kQ8SplitConfigs) / sizeof(kQ8SplitConfigs[0]) == 5, "every form is listed");
#define Q8_PARAMS(I) kQ8SplitConfigs[I].bn, kQ8SplitConfigs[I].stages, kQ8SplitConfigs[I].ctas

template <int BN, int STAGES, int CTAS>
cudaError_t prepare_all() {
    cudaError_t e = cudaSuccess;
    if (e == cudaSuccess) e = prepare<BN, STAGES, CTAS, 1, __nv_bfloat16>();
    if (e == cudaSuccess) e = prepare<BN, STAGES, CTAS, 1, __half>();
    if (e == cudaSuccess) e = prepare<BN, STAGES, CTAS, 1, float>();
    if (e == cudaSuccess) e = prepare<BN, STAGES, CTAS, kMaxGroup, __nv_bfloat16>();
    if (e == cudaSuccess) e = prepare<BN, STAGES, CTAS, kMaxGroup, __half>();
    if (e == cudaSuccess) e = prepare<BN, STAGES, CTAS, kMaxGroup, float>();
    return e;
}

}  // namespace

cudaError_t q8_prepare_split() {
    cudaError_t e = cudaSuccess;
#define Q8_PREPARE(I) \
    if (e == cudaSuccess) e = prepare_all<Q8_PARAMS(I)>();
    Q8_SPLIT_CONFIGS(Q8_PREPARE)
#undef Q8_PREPARE
    return e;
}

template <int G>
cudaError_t launch_q8_split(const Q8Maps<G>& maps, const Q8SplitArgs<G>& a, int config, int y_type, int grid,
                            cudaStream_t st) {
#define Q8_LAUNCH(I)                                                                        \
    if (config == I)                                                                        \
        return y_type == kBf16   ? launch<Q8_PARAMS(I), G, __nv_bfloat16>(maps, a, grid, st) \
               : y_type == kFp16 ? launch<Q8_PARAMS(I), G, __half>(maps, a, grid, st)        \
                                 : launch<Q8_PARAMS(I), G, float>(maps, a, grid, st);
    Q8_SPLIT_CONFIGS(Q8_LAUNCH)
#undef Q8_LAUNCH
    return cudaErrorInvalidValue;
}
template cudaError_t launch_q8_split<1>(const Q8Maps<1>&, const Q8SplitArgs<1>&, int, int, int, cudaStream_t);
template cudaError_t launch_q8_split<kMaxGroup>(const Q8Maps<kMaxGroup>&, const Q8SplitArgs<kMaxGroup>&, int, int, int,
                                                cudaStream_t);

}  // namespace patch
