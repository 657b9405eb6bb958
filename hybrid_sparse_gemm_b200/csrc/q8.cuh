// 8-bit integer path: packed-format constants, kernel argument structs and
// launch entry points shared by the host runtime.
//
// A slab is a strip (128 rows of W) times 128 columns: a dense record is the
// 128 x 128 block of codes, 128 bytes per row in the 128-byte-swizzled layout
// (16 KB); a 2:4 record is 64 kept codes per row in the 64-byte-swizzled layout
// (8 KB) followed by the slab's 2 KB of metadata, 16 bytes per row, so that one
// copy brings both: the 4-bit code of group g of the slab (columns 4g .. 4g+3)
// is at bit 4g of the row's 128 bits. One tcgen05.cp.128x128b puts the block
// into four TMEM columns, row r in lane r; each sparse MMA (K = 64) reads two of
// them. A last slab of 64 columns (K % 128 == 64) is padded with zero codes.
// Records lie strip-major, then the dense images of 2:4 slabs whose partner
// strip's slab is dense.
#pragma once

#include "kernels.cuh"

namespace patch {

constexpr int kQ8SlabK = 128;
constexpr int kQ8SparseBytes = kSparseValBytes + kMetaBytes;
__host__ __device__ inline uint32_t q8_record_bytes(uint32_t d) {
    return (d & kSlabSparse) ? kQ8SparseBytes : kDenseSlabBytes;
}

// Output element types (match patch_dtype).
constexpr int kBf16 = 0, kFp16 = 1, kFp32 = 2;

struct Q8PackArgs {
    const void* W;            // N x K, row-major: bf16 bits, or int8 codes
    int w_int8;
    const uint8_t* bits;      // bit-packed keep mask
    int bitorder;             // 0 MSB first, 1 LSB first
    const uint8_t* flags;     // tile flags on the device, (N/R) x (K/C)
    const uint32_t* slab;     // per-strip slab table, S x KB
    const uint32_t* gemm;     // CTA-pair slab table, S x KB
    float* w_scale;           // N channel scales (written for bf16 weights, checked for int8 codes)
    uint8_t* out;             // packed bytes
    int64_t K;
    int R, C, KB;
    unsigned long long* counters;  // [bad groups, stray zeros, pruned, bad scales]
};
cudaError_t launch_q8_pack(const Q8PackArgs& a, int S, cudaStream_t st);
cudaError_t launch_q8_unpack(const uint8_t* packed, const uint32_t* slab, int S, int KB, int64_t K, int8_t* W, cudaStream_t st);

// Tensor maps of G members: activation codes (per call), and the packed bytes
// viewed as 128-byte rows with boxes of a dense (128 rows) and a 2:4 record (80).
template <int G>
struct Q8Maps {
    CUtensorMap x[G], a16[G], a10[G];
};

// Split-K kernel: one cluster of P CTAs per unit (strip, token tile).
struct Q8Member {
    const uint32_t* slab;  // S x KB
    const float* x_scale;  // M
    const float* w_scale;  // N
    void* Y;
    int64_t ldy;           // row pitch of Y, elements
    int KB;
    int unit0;             // the member's first unit
};
template <int G>
struct Q8SplitArgs {
    Q8Member m[G];
    int* status;
    int n;      // members
    int M;
    int MB;     // token tiles
    int n_tok;  // tokens per tile, a multiple of 16
    int P;      // CTAs per unit
    uint32_t zero;  // 0 (see the kernel's join)
};
// The kernel's forms: tokens per unit (n_tok at most), pipeline stages, CTAs
// resident per SM. They share the SM's shared memory. One CTA with a deep pipeline
// streams its slabs faster than two shallow ones side by side and joins fewer sums,
// as long as one CTA per SM is the whole call; with more CTAs than that, one joins
// and stores while the other streams. Measured at 2:4 tiles 70 %, each at its P of
// the least estimate, one deep and two shallow: 100 x 4096 x 4096 6.8 and 8.4 us, 100 x
// 11008 x 4096 10.4 and 11.6, 64 x 4096 x 4096 5.8 and 6.0, 200 x 11008 x 4096 (172
// units) 18.1 and 14.9. 16 tokens, measured before the sums were joined in registers:
// 6 stages x 2 CTAs 4.4 us at 4096 x 4096, 4 x 3 4.5, 3 x 4 and 12 x 1 4.9; 4096 x
// 11008 8.4 (7.9 now), 8.7, 9.1 and 8.4.
struct Q8SplitConfig {
    int bn, stages, ctas;
};
constexpr Q8SplitConfig kQ8SplitConfigs[] = {{16, 6, 2}, {64, 9, 1}, {64, 4, 2}, {128, 6, 1}, {128, 3, 2}};
// grid: all units * P; config: index into kQ8SplitConfigs
template <int G>
cudaError_t launch_q8_split(const Q8Maps<G>& maps, const Q8SplitArgs<G>& a, int config, int y_type, int grid,
                            cudaStream_t st);
constexpr int kQ8MaxParts = 8;
cudaError_t q8_prepare_split();

// Kernel on CTA pairs with two strips per CTA (many tokens). A work unit is
// (member, strip quad, token tile); the MB tiles share M's 32-token granules,
// tile_gran each and one more for the first tile_extra.
struct Q8WideMember {
    const uint32_t* gemm;  // CTA-pair slab table, rows in pair-position order
    const int* order;      // strips by pair position
    const float* x_scale;
    const float* w_scale;
    void* Y;
    int64_t ldy;
    int S, KB;
    int unit0;             // the member's first unit
};
template <int G>
struct Q8WideArgs {
    Q8WideMember m[G];
    int* status;
    int n, units;          // members, units of all of them
    int M, MB;
    int tile_gran, tile_extra;
    int x_rows;            // rows of the activation boxes: half the largest tile
};
constexpr int kQ8WideBN = 224;  // tokens per tile: kind::i8 on a CTA pair takes multiples of 32
template <int G>
cudaError_t launch_q8_wide(const Q8Maps<G>& maps, const Q8WideArgs<G>& a, int y_type, int clusters, cudaStream_t st);
cudaError_t q8_prepare_wide(int* max_clusters);

// Row operators: one row of 8-bit codes and one scale per token.
enum RowMode { kRowQuantize = 0, kRowNorm = 1, kRowNormResidual = 2, kRowSiluMul = 3 };
struct RowArgs {
    const void* x;            // x, or gate
    const void* r;            // residual, or up
    void* ro;                 // x + residual
    const void* gamma;
    int64_t ldx, ldr, ldo, ldq;
    int64_t M;
    int K;
    float eps;
    int8_t* q;
    float* scale;
};
cudaError_t launch_rows_q8(const RowArgs& a, int mode, int type, int sms, cudaStream_t st);
cudaError_t launch_dequantize_q8(const int8_t* q, int64_t ldq, const float* scale, int64_t M, int K, void* out, int64_t ldo,
                                 int type, cudaStream_t st);

}  // namespace patch
