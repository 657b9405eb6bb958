// Pack and unpack kernels of the 8-bit integer path: bit-packed keep/prune
// mask + frozen weights (bf16, quantised here with one scale per output
// channel, or int8 codes) -> dense slabs or compressed 2:4 codes with their
// position codes, and dense images of 2:4 slabs whose partner strip is dense.
//
// Semantics as for the bf16 pack: the mask zeroes pruned weights and each
// tile is dense or 2:4 (PATCH model card "llama_3.2_1b-PATCH-45Sparse",
// method and release paragraphs). Layout: see q8.cuh. One pass over W bound
// by HBM, done once per weight.
#include "q8.cuh"

namespace patch {

namespace {

constexpr float kMinScale = 1.17549435e-38f;  // 2^-126

__device__ __forceinline__ int keep_bit(uint32_t byte, int e, int bitorder) {
    return bitorder == 0 ? (byte >> (7 - e)) & 1 : (byte >> e) & 1;
}

// Channel scales of bf16 weights: max |w| over the kept ones / 127, at least
// 2^-126. A channel that keeps a NaN or an infinity counts as a bad scale.
__global__ void __launch_bounds__(128) q8_scale_kernel(const Q8PackArgs a) {
    __shared__ uint32_t s_max[4];
    const int64_t n = blockIdx.x;
    const uint16_t* w = static_cast<const uint16_t*>(a.W) + n * a.K;
    uint32_t top = 0;
    for (int64_t k = 8 * (int64_t)threadIdx.x; k < a.K; k += 8 * 128) {
        const uint4 raw = *reinterpret_cast<const uint4*>(w + k);
        const uint32_t mb = a.bits[(n * a.K + k) >> 3];
        const uint32_t v[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (keep_bit(mb, e, a.bitorder)) top = max(top, (v[e >> 1] >> (16 * (e & 1))) & 0x7FFFu);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
        top = max(max(s_max[0], s_max[1]), max(s_max[2], s_max[3]));
        if (top >= 0x7F80u) atomicAdd(&a.counters[3], 1ull);
        a.w_scale[n] = fmaxf(__uint_as_float(top << 16) / 127.f, kMinScale);
    }
}

// 16 codes of row n from column k (a multiple of 16); zeros past K.
__device__ __forceinline__ void load_codes(const Q8PackArgs& a, int64_t n, int64_t k, int8_t* c) {
    if (k >= a.K) {
        *reinterpret_cast<uint4*>(c) = make_uint4(0, 0, 0, 0);
        return;
    }
    if (a.w_int8) {
        *reinterpret_cast<uint4*>(c) = *reinterpret_cast<const uint4*>(static_cast<const int8_t*>(a.W) + n * a.K + k);
        return;
    }
    const uint16_t* w = static_cast<const uint16_t*>(a.W) + n * a.K + k;
    const float scale = a.w_scale[n];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint4 raw = *reinterpret_cast<const uint4*>(w + 8 * h);
        const uint32_t v[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            // a pruned weight may be larger than the kept ones: its code is dropped, so it only has to fit
            const float y = __uint_as_float((v[e >> 1] >> (16 * (e & 1))) << 16) / scale;
            c[8 * h + e] = (int8_t)__float2int_rn(fminf(fmaxf(y, -127.f), 127.f));
        }
    }
}

// Mask bits of 16 columns from k as keep bits, lowest column in bit 0; zeros past K.
__device__ __forceinline__ uint32_t load_keep(const Q8PackArgs& a, int64_t n, int64_t k) {
    if (k >= a.K) return 0u;
    const int64_t e0 = n * a.K + k;
    uint32_t keep = 0;
#pragma unroll
    for (int e = 0; e < 16; ++e) keep |= (uint32_t)keep_bit(a.bits[(e0 + e) >> 3], e & 7, a.bitorder) << e;
    return keep;
}

// Dense image of slab (s, b) at dst. When `count` is set the validation
// counters are updated (groups of 2:4-flagged tiles, stray zeros, pruned).
__device__ void write_dense(const Q8PackArgs& a, int s, int b, uint8_t* dst, bool count, unsigned long long& bad,
                            unsigned long long& stray, unsigned long long& pruned) {
    const int tiles_k = (int)(a.K / a.C);
    for (int q = threadIdx.x; q < 1024; q += blockDim.x) {
        const int r = q >> 3, L = q & 7;
        const int64_t n = (int64_t)s * kStrip + r, k = (int64_t)b * kQ8SlabK + 16 * L;
        __align__(16) int8_t c[16];
        load_codes(a, n, k, c);
        const uint32_t keep = load_keep(a, n, k);
#pragma unroll
        for (int e = 0; e < 16; ++e)
            if (!((keep >> e) & 1u)) c[e] = 0;
        if (count && k < a.K) {
            const int kept = __popc(keep);
            pruned += 16 - kept;
            if (a.flags[(n / a.R) * tiles_k + (k / a.C)]) {
                for (int g = 0; g < 4; ++g) bad += __popc((keep >> (4 * g)) & 15u) != 2;
            } else {
                stray += 16 - kept;
            }
        }
        *reinterpret_cast<uint4*>(dst + sw128_off(r, L)) = *reinterpret_cast<uint4*>(c);
    }
}

// One block per slab (s, b).
__global__ void __launch_bounds__(256) q8_pack_kernel(const Q8PackArgs a) {
    __shared__ unsigned long long s_cnt[3];  // bad groups, stray zeros, pruned
    if (threadIdx.x < 3) s_cnt[threadIdx.x] = 0;
    __syncthreads();
    const int s = blockIdx.x / a.KB, b = blockIdx.x % a.KB;
    if (a.w_int8 && b == 0 && threadIdx.x < kStrip) {
        const float given = a.w_scale[s * kStrip + threadIdx.x];
        if (!(given >= 0.f && given < INFINITY)) atomicAdd(&a.counters[3], 1ull);
    }
    const uint32_t d = a.slab[blockIdx.x];
    uint8_t* base = a.out + slab_offset_bytes(d);
    unsigned long long bad = 0, stray = 0, pruned = 0;
    if (!(d & kSlabSparse)) {
        write_dense(a, s, b, base, true, bad, stray, pruned);
    } else {
        uint8_t* meta = base + kSparseValBytes;
        // 512 items: row r, 32 columns from 32 L (8 groups, 16 kept codes)
        for (int q = threadIdx.x; q < 512; q += blockDim.x) {
            const int r = q >> 2, L = q & 3;
            const int64_t n = (int64_t)s * kStrip + r, k = (int64_t)b * kQ8SlabK + 32 * L;
            __align__(16) int8_t c[32], kept[16];
            load_codes(a, n, k, c);
            load_codes(a, n, k + 16, c + 16);
            uint32_t code = 0x44444444u;  // positions 0 and 1, for the padding
            if (k >= a.K) {
                *reinterpret_cast<uint4*>(kept) = make_uint4(0, 0, 0, 0);
            } else {
                const uint32_t keep = load_keep(a, n, k) | load_keep(a, n, k + 16) << 16;
                code = 0;
#pragma unroll
                for (int g = 0; g < 8; ++g) {
                    int idx[2] = {0, 1}, m = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if ((keep >> (4 * g + i)) & 1u) {
                            if (m < 2) idx[m] = i;
                            ++m;
                        }
                    pruned += 4 - m;
                    if (m != 2) {
                        ++bad;
                        idx[0] = 0;
                        idx[1] = 1;
                    }
                    kept[2 * g] = c[4 * g + idx[0]];
                    kept[2 * g + 1] = c[4 * g + idx[1]];
                    code |= (uint32_t)(idx[0] | (idx[1] << 2)) << (4 * g);
                }
            }
            *reinterpret_cast<uint4*>(base + sw64_off(r, L)) = *reinterpret_cast<uint4*>(kept);
            *reinterpret_cast<uint32_t*>(meta + r * 16 + L * 4) = code;
        }
        // a 2:4 slab whose partner strip is dense also gets a dense image
        const uint32_t g = a.gemm[blockIdx.x];
        if (!(g & kSlabSparse)) {
            unsigned long long x0 = 0, x1 = 0, x2 = 0;
            write_dense(a, s, b, a.out + slab_offset_bytes(g), false, x0, x1, x2);
        }
    }
    for (int o = 16; o > 0; o >>= 1) {
        bad += __shfl_xor_sync(0xffffffffu, bad, o);
        stray += __shfl_xor_sync(0xffffffffu, stray, o);
        pruned += __shfl_xor_sync(0xffffffffu, pruned, o);
    }
    if ((threadIdx.x & 31) == 0) {
        atomicAdd(&s_cnt[0], bad);
        atomicAdd(&s_cnt[1], stray);
        atomicAdd(&s_cnt[2], pruned);
    }
    __syncthreads();
    if (threadIdx.x < 3 && s_cnt[threadIdx.x]) atomicAdd(&a.counters[threadIdx.x], s_cnt[threadIdx.x]);
}

// Decode the per-strip records back to the masked codes, row-major N x K.
__global__ void __launch_bounds__(256) q8_unpack_kernel(const uint8_t* __restrict__ packed,
                                                        const uint32_t* __restrict__ slab, int KB, int64_t K,
                                                        int8_t* __restrict__ W) {
    const int s = blockIdx.x / KB, b = blockIdx.x % KB;
    const uint32_t d = slab[blockIdx.x];
    const uint8_t* base = packed + slab_offset_bytes(d);
    for (int q = threadIdx.x; q < 1024; q += blockDim.x) {
        const int r = q >> 3, L = q & 7;
        const int64_t n = (int64_t)s * kStrip + r, k = (int64_t)b * kQ8SlabK + 16 * L;
        if (k >= K) continue;
        __align__(16) int8_t c[16];
        if (!(d & kSlabSparse)) {
            *reinterpret_cast<uint4*>(c) = *reinterpret_cast<const uint4*>(base + sw128_off(r, L));
        } else {
            // 16 columns: 4 groups, half of a 16-byte piece of kept codes
            __align__(8) int8_t kept[8];
            *reinterpret_cast<uint2*>(kept) = *reinterpret_cast<const uint2*>(base + sw64_off(r, L >> 1) + 8 * (L & 1));
            const uint32_t code = *reinterpret_cast<const uint16_t*>(base + kSparseValBytes + r * 16 + L * 2);
            *reinterpret_cast<uint4*>(c) = make_uint4(0, 0, 0, 0);
            for (int g = 0; g < 4; ++g) {
                const uint32_t p = (code >> (4 * g)) & 15u;
                c[4 * g + (p & 3u)] = kept[2 * g];
                c[4 * g + (p >> 2)] = kept[2 * g + 1];
            }
        }
        *reinterpret_cast<uint4*>(W + n * K + k) = *reinterpret_cast<uint4*>(c);
    }
}

}  // namespace

cudaError_t launch_q8_pack(const Q8PackArgs& a, int S, cudaStream_t st) {
    if (!a.w_int8) {
        q8_scale_kernel<<<S * kStrip, 128, 0, st>>>(a);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    q8_pack_kernel<<<S * a.KB, 256, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_q8_unpack(const uint8_t* packed, const uint32_t* slab, int S, int KB, int64_t K, int8_t* W, cudaStream_t st) {
    q8_unpack_kernel<<<S * KB, 256, 0, st>>>(packed, slab, KB, K, W);
    return cudaGetLastError();
}

}  // namespace patch
