// Hybrid dense / 2:4 product in 8-bit integers on CTA pairs with two strips per
// CTA, for many tokens:
// Y[m,n] = (sum_k Xq[m,k] * (Wq (.) Mask)[n,k]) * x_scale[m] * w_scale[n].
//
// The arrangement of the bf16 kernel for large launches (PATCH abstract,
// "PATCH: Learnable Tile-level Hybrid Sparsity for LLMs", dense slabs on
// tcgen05.mma, 2:4 slabs on tcgen05.mma.sp) with kind::i8. A cluster of two
// CTAs owns a strip quad (pair positions 4c .. 4c+3) and a tile of up to 224
// tokens. Every 128-column slab issues two 256-row MMAs (cta_group::2), one per
// strip pair, so that each activation byte from L2 serves 512 weight rows: per
// slab and CTA 20 KB of 2:4 records and 14 KB of activations feed 448 cycles of
// the tensor pipe, 76 bytes a cycle. Stages lie in a ring sized by their records
// (six 2:4 stages in flight), a record and its metadata come in one copy, four
// warps issue copies and two issue MMAs, whole warps with an elected lane.
//
// Measured: one CTA pair alone takes 457 cycles a 2:4 stage and 905 a dense one, the
// pipe's own pace; all pairs together 1.0 to 1.15 times that. Between two tiles of a
// pair the accumulators are read for 3300 cycles, a sixth of a tile of 32 slabs,
// but taking the conversions out of it won 1 % of the time only: 2048 x 11008 x
// 4096 with 90 % 2:4 tiles of 128 x 128 takes 48 us at the clock of a short run (its
// MMAs 32 us at twice the bf16 matrix rate, 84 % of the pairs' slabs being 2:4), 8192 x
// 13824 x 5120 253 us, and in a run of seconds, where the card's power limit holds the
// clock near 1.4 GHz, 291 us (270 and 311 with tiles of 128 x 64, whose slabs are 2:4
// in 71 % of the pairs). fp32 outputs are stored before the accumulator is handed
// back: 54 us for 49, and 358 for 268.
//
// TMEM: accumulators in columns [0, 224) and [256, 480), metadata of strip pair
// 0 at 224 and of pair 1 at 232. All waits are bounded.
#include <cuda_fp16.h>

#include "q8.cuh"
#include "q8_mma.cuh"

namespace patch {

namespace {

constexpr int kProducers = 4;                   // TMA-issuing warps (stages dealt round robin)
constexpr int kMmaWarp = kProducers;            // MMA issuers (leader CTA), one per strip pair;
constexpr int kMmaWarps = 2;                    // the first also owns TMEM
constexpr int kEpiWarp0 = 8;                    // (two warps idle: register splits go by warpgroup)
constexpr int kEpiWarps = 16;                   // per accumulator, two warps per TMEM lane quarter
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
constexpr int kBN = kQ8WideBN;
constexpr int kStageX = kBN / 2 * 128;          // 14 KB of activations per slab and CTA
constexpr int kQ = 8;                           // per-stage barriers: more than the stages that fit in the ring
constexpr int kMinStage = 2 * kQ8SparseBytes + kStageX;
constexpr int kEpiCols = kBN / 2;               // columns of an epilogue warp
constexpr int kSmemScales = kEpiWarps * kEpiCols * 4;
constexpr int kRing = (232448 - kSmemScales - 1024 - 512) / 1024 * 1024;
constexpr int kSmemBytes = kRing + kSmemScales + 1024 + 512;
constexpr uint32_t kDenseStage = 2 * kDenseSlabBytes + kStageX;
constexpr uint32_t kSaved = kDenseSlabBytes - kQ8SparseBytes;  // by each 2:4 record of a stage
static_assert(kStageX % 1024 == 0 && kQ8SparseBytes % 1024 == 0, "every record starts 1024-byte aligned");
static_assert(kRing / kMinStage + 2 <= kQ, "stages in flight stay within the barrier window");
// A wait for stage j's phase by parity is right only once stage j - kQ is known
// to be consumed. A producer that loads stage g waits for a j <= g - 3 (a ring of
// at least four stages); its previous stage, g - kProducers, waited for one after
// g - kProducers - kQ.
static_assert(kProducers <= 4 && kRing / kDenseStage >= 4, "no wait is two phases ahead");
// Registers: launched with 80 a thread (768 threads); the producers' warpgroup
// gives up 24 of them and the issuers' 40, the four epilogue warpgroups take 16
// more: 128 * (56 + 40 + 4 * 96) = 61440, what the block was launched with.
constexpr int kRegsProduce = 56, kRegsIssue = 40, kRegsEpi = 96;
static_assert(128 * (kRegsProduce + kRegsIssue + 4 * kRegsEpi) <= kThreads * 80, "the register split adds up");
constexpr int kAcc1 = 256;                      // first column of accumulator 1
constexpr int kECol0 = kBN;                     // metadata columns of strip pair 0
constexpr int kECol1 = kBN + 8;                 // ... and of strip pair 1
constexpr int kTmemCols = 512;
static_assert(kECol1 + 4 <= kAcc1, "metadata columns fit between the accumulators");

template <class A>
__device__ __forceinline__ int tile_start(const A& a, int j) {
    return 32 * (j * a.tile_gran + min(j, a.tile_extra));
}
template <class A>
__device__ __forceinline__ int tile_tokens(const A& a, int j) {
    return 32 * (a.tile_gran + (j < a.tile_extra ? 1 : 0));
}

// Stages are placed one after another in a ring of kRing bytes; a stage that
// does not fit before the end starts again at 0. Producers and issuers keep track
// of all of them, in registers (with the ring's history in local memory a step of
// the walk took 470 cycles, more than the stage's MMAs). `pos` counts bytes up to the
// newest stage's end, skipped ends included (modulo 2^32: only differences are
// used); the tail is the oldest stage whose bytes are not known to be free.
struct Ring {
    uint32_t pos = 0, off = 0;            // end of the newest stage
    uint32_t tail_pos = 0, tail_off = 0;  // start of stage `tail`
    int tail = 0, next = 0;               // `next`: stages placed
    uint64_t kinds = 0;                   // 4 bits a stage, newest lowest: 2:4 records | started at 0 again << 2
    // Places a stage with `sparse` 2:4 records (0..2); returns its ring offset.
    __device__ __forceinline__ uint32_t place(uint32_t sparse) {
        const uint32_t size = kDenseStage - kSaved * sparse;
        const bool wrap = off + size > (uint32_t)kRing;
        if (wrap) {
            pos += (uint32_t)kRing - off;
            off = 0;
        }
        kinds = (kinds << 4) | sparse | (wrap ? 4u : 0u);
        const uint32_t at = off;
        pos += size;
        off += size;
        ++next;
        return at;
    }
    // Whether stages in the newest one's place have to be consumed first; then
    // the tail moves past them, and the last of them is stage tail - 1.
    __device__ __forceinline__ bool reclaim() {
        bool any = false;
        while ((int)(pos - (uint32_t)kRing - tail_pos) > 0) {
            const int age = 4 * (next - 1 - tail);  // at most 4 * 11
            const uint32_t size = kDenseStage - kSaved * ((uint32_t)(kinds >> age) & 3u);
            tail_pos += size;
            tail_off += size;
            ++tail;
            if ((uint32_t)(kinds >> (age - 4)) & 4u) {
                tail_pos += (uint32_t)kRing - tail_off;
                tail_off = 0;
            }
            any = true;
        }
        return any;
    }
};

// Two numbers as a pair of 16-bit ones, the first in the low half.
__device__ __forceinline__ uint32_t pack2(float x, float y, __nv_bfloat16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack2(float x, float y, __half) {
    const __half2 v = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Two products at once, each rounded as a * b is.
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t pair2(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
template <class T>
__device__ __forceinline__ uint32_t pack2(uint64_t v, T t) {
    float x, y;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
    return pack2(x, y, t);
}

template <int G, class T>
__global__ void __launch_bounds__(kThreads, 1)
    q8_wide_kernel(const __grid_constant__ Q8Maps<G> maps, const __grid_constant__ Q8WideArgs<G> a) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    float* scales = reinterpret_cast<float*>(smem + kRing);  // [epilogue warp][kEpiCols]
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kRing + kSmemScales);
    uint64_t* full = bars;                       // [kQ] leader: both CTAs' bytes of stage g (at g % kQ)
    uint64_t* empty = full + kQ;                 // [kQ] every CTA: stage g consumed by both issuers
    uint64_t* acc_full = empty + kQ;             // [2] both CTAs: accumulator h ready
    uint64_t* acc_empty = acc_full + 2;          // [2] leader: the 16 epilogue warps of accumulator h drained it
    uint64_t* drain = acc_empty + 2;             // [2]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 2);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);  // known to be uniform
    const int lane = threadIdx.x & 31;
    const uint32_t pr = cluster_rank();          // CTA within the pair (0 = leader)
    const int cl = blockIdx.x >> 1;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kQ; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kMmaWarps);
        }
        for (int h = 0; h < 2; ++h) {
            mbar_init(&acc_full[h], 1);
            mbar_init(&acc_empty[h], kEpiWarps);  // its 8 epilogue warps in each of the 2 CTAs
            mbar_init(&drain[h], 1);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc2(tmem_slot, kTmemCols);
        tmem_relinquish2();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // barriers of both CTAs initialised before any remote use
    tc_fence_after();
    const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    auto raise = [&]() {
        *abort_flag = 1;
        atomicCAS(a.status, 0, kStatusTimeout);
    };
    // Pair position of the strip this CTA loads for strip pair h of quad c.
    // Missing positions fall back to one whose partner relation is kept, so
    // both halves of every MMA stay one kind.
    auto pos_of = [&](int S, int c, int h) {
        int pos = 4 * c + 2 * h + (int)pr;
        if (pos >= S) pos = 4 * c + 2 * h;
        if (pos >= S) pos = 4 * c + (int)pr;
        if (pos >= S) pos = 4 * c;
        return pos;
    };
    // Unit u is (member, quad, token tile); pair cl takes units cl, cl + pairs, ...
    // Units of one wave share their quads' weights in L2; quads and members come in
    // the order of falling cost.
    const int pairs = gridDim.x >> 1;
    struct Unit {
        int l, c, j;
    };
    auto unit_of = [&](int u) {
        Unit x;
        x.l = 0;
        if (G > 1)
            while (x.l + 1 < a.n && u >= a.m[x.l + 1].unit0) ++x.l;
        u -= a.m[x.l].unit0;
        x.c = u / a.MB;
        x.j = u - x.c * a.MB;
        return x;
    };
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (warp < kProducers) {
        // ---------------- producers (both CTAs) ----------------
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsProduce));
        // Every producer walks the whole stage sequence to place each stage
        // in the ring; it loads the stages g with g % kProducers == me, whole
        // warps together, lane 0 issuing. Before, the stages that last used those
        // ring bytes must have been consumed (in order, so waiting for the latest
        // suffices).
        const int me = warp;
        Ring ring;
        int g = 0;
        int my_last = -1;    // sequence index of the last stage this producer loaded
        bool ok = true;
        // every strip quad of a member reads the same activation tiles, so
        // they are kept in L2 over the weight records (each read by one wave
        // of token tiles)
        const uint64_t pol_x = policy_evict_last();
        const uint32_t x_bytes = (uint32_t)a.x_rows * 128u;
        // Until the ring is full for the first time only weights are loaded: they
        // do not depend on the stream's previous kernel. Activations (at most two
        // of this warp's stages are then without theirs) follow once it is done.
        bool waited = false;
        int n_pend = 0, pend_l = 0, pend_tok = 0, pend_b0 = 0, pend_b1 = 0;
        uint32_t pend_dst0 = 0, pend_dst1 = 0, pend_bar0 = 0, pend_bar1 = 0;
        auto load_pending = [&]() {
            asm volatile("griddepcontrol.wait;" ::: "memory");
            waited = true;
            if (lane == 0 && n_pend > 0)
                tma_load_2d_pair_hint(pend_dst0, &maps.x[pend_l], pend_bar0, pend_b0 * kQ8SlabK, pend_tok, pol_x);
            if (lane == 0 && n_pend > 1)
                tma_load_2d_pair_hint(pend_dst1, &maps.x[pend_l], pend_bar1, pend_b1 * kQ8SlabK, pend_tok, pol_x);
        };
        for (int u = cl; u < a.units && ok; u += pairs) {
            const Unit un = unit_of(u);
            const int l = un.l, c = un.c, j = un.j;
            const Q8WideMember& L = a.m[l];
            const int KB = L.KB;
            const uint32_t* t0 = L.gemm + (size_t)pos_of(L.S, c, 0) * KB;
            const uint32_t* t1 = L.gemm + (size_t)pos_of(L.S, c, 1) * KB;
            const int tok = tile_start(a, j) + (int)pr * (tile_tokens(a, j) >> 1);
            // records of 32 slabs, a lane each, the next 32 on their way
            uint32_t r0 = 0, r1 = 0, m0 = 0, m1 = 0;
            uint32_t n0 = lane < KB ? t0[lane] : 0u, n1 = lane < KB ? t1[lane] : 0u;
            for (int b = 0; b < KB; ++b, ++g) {
                if ((b & 31) == 0) {
                    r0 = n0;
                    r1 = n1;
                    m0 = __ballot_sync(0xffffffffu, r0 & kSlabSparse);
                    m1 = __ballot_sync(0xffffffffu, r1 & kSlabSparse);
                    const int nb = b + 32 + lane;
                    n0 = nb < KB ? t0[nb] : 0u;
                    n1 = nb < KB ? t1[nb] : 0u;
                }
                const uint32_t s0 = (m0 >> (b & 31)) & 1u, s1 = (m1 >> (b & 31)) & 1u;
                const uint32_t off = ring.place(s0 + s1);
                if (g % kProducers != me) continue;
                const bool reuse = ring.reclaim();
                if (!waited && (reuse || u != cl || n_pend == 2)) load_pending();
                if (reuse) {
                    const int jl = ring.tail - 1;
                    const bool free = mbar_wait(&empty[jl % kQ], (uint32_t)((jl / kQ) & 1), abort_flag);
                    if (!__all_sync(0xffffffffu, free)) {
                        if (lane == 0) raise();
                        ok = false;
                        break;
                    }
                }
                const uint32_t d0 = __shfl_sync(0xffffffffu, r0, b & 31), d1 = __shfl_sync(0xffffffffu, r1, b & 31);
                const uint32_t b0 = q8_record_bytes(d0), b1 = q8_record_bytes(d1);
                const uint32_t bar = map_to_rank(smem_u32(&full[g % kQ]), 0);
                const uint32_t dst = smem_u32(smem) + off;
                if (lane == 0) {
                    if (pr == 0) mbar_arrive_expect_tx(&full[g % kQ], 2u * (b0 + b1 + x_bytes));
                    tma_load_2d_pair(dst, s0 ? &maps.a10[l] : &maps.a16[l], bar, 0, (int)(slab_offset_bytes(d0) >> 7));
                    tma_load_2d_pair(dst + b0, s1 ? &maps.a10[l] : &maps.a16[l], bar, 0,
                                     (int)(slab_offset_bytes(d1) >> 7));
                    if (waited)
                        tma_load_2d_pair_hint(dst + b0 + b1, &maps.x[l], bar, b * kQ8SlabK, tok, pol_x);
                }
                if (!waited) {
                    if (n_pend == 0) {
                        pend_dst0 = dst + b0 + b1;
                        pend_bar0 = bar;
                        pend_b0 = b;
                    } else {
                        pend_dst1 = dst + b0 + b1;
                        pend_bar1 = bar;
                        pend_b1 = b;
                    }
                    ++n_pend;
                    pend_l = l;
                    pend_tok = tok;
                }
                my_last = g;
            }
        }
        if (!waited) load_pending();
        if (pr == 0 && lane == 0) {
            // Bounded wait for the loads of my stages among the last kQ of
            // the sequence, whatever the abort flag says, so none lands
            // after the cluster exits.
            for (int gg = g - kQ; gg <= my_last; ++gg) {
                if (gg < 0 || gg % kProducers != me) continue;
                const uint64_t t0 = globaltimer();
                while (!mbar_try_wait(&full[gg % kQ], (uint32_t)((gg / kQ) & 1)) &&
                       globaltimer() - t0 < kWaitLimitNs) {
                }
            }
        }
    } else if (warp < kEpiWarp0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
        if (pr == 0 && warp < kMmaWarp + kMmaWarps) {
            // ---------------- MMA issuers (leader CTA), one per strip pair ----------------
            // Both read every stage; a stage's ring bytes are free once both have
            // committed it. Whole warps, one elected lane issuing.
            const int h = warp - kMmaWarp;
            const uint32_t el = elect();
            const uint32_t d_tmem = tmem_base + (uint32_t)(h * kAcc1);
            const uint32_t e_col = tmem_base + (uint32_t)(h ? kECol1 : kECol0);
            const uint32_t ring0 = smem_u32(smem);
            Ring ring;
            int g = 0, t = 0;
            bool ok = true, any_mma = false;
            for (int u = cl; u < a.units && ok; u += pairs, ++t) {
                const Unit un = unit_of(u);
                const Q8WideMember& L = a.m[un.l];
                const int KB = L.KB;
                const uint32_t* t0 = L.gemm + (size_t)pos_of(L.S, un.c, 0) * KB;
                const uint32_t* t1 = L.gemm + (size_t)pos_of(L.S, un.c, 1) * KB;
                const int nt = tile_tokens(a, un.j);
                const uint32_t idesc_d = idesc_i8(256, nt, false);
                const uint32_t idesc_s = idesc_i8(256, nt, true);
                uint32_t m0 = 0, m1 = 0;
                uint32_t n0 = lane < KB ? t0[lane] : 0u, n1 = lane < KB ? t1[lane] : 0u;
                for (int b = 0; b < KB; ++b, ++g) {
                    if ((b & 31) == 0) {
                        m0 = __ballot_sync(0xffffffffu, n0 & kSlabSparse);
                        m1 = __ballot_sync(0xffffffffu, n1 & kSlabSparse);
                        const int nb = b + 32 + lane;
                        n0 = nb < KB ? t0[nb] : 0u;
                        n1 = nb < KB ? t1[nb] : 0u;
                    }
                    const uint32_t s0 = (m0 >> (b & 31)) & 1u, s1 = (m1 >> (b & 31)) & 1u;
                    const uint32_t at = ring0 + ring.place(s0 + s1);
                    const uint32_t b0 = kDenseSlabBytes - kSaved * s0, b1 = kDenseSlabBytes - kSaved * s1;
                    ok = mbar_wait(&full[g % kQ], (uint32_t)((g / kQ) & 1), abort_flag);
                    // the first stage of a tile is at hand before the accumulator is
                    if (b == 0) ok = ok && mbar_wait(&acc_empty[h], (t & 1) ^ 1u, abort_flag);
                    if (!__all_sync(0xffffffffu, ok)) {
                        if (lane == 0) raise();
                        ok = false;
                        break;
                    }
                    if (b == 0) tc_fence_after();
                    issue_slab_i8<true>(el, h ? s1 : s0, b == 0, at + (h ? b0 : 0u), at + b0 + b1, d_tmem, e_col,
                                        idesc_d, idesc_s);
                    any_mma = true;
                    commit2_mask_el(el, &empty[g % kQ], 3);
                }
                if (!ok) break;
                commit2_mask_el(el, &acc_full[h], 3);
            }
            __syncwarp();
            if (*abort_flag && any_mma && el) {
                commit2_local(&drain[h]);
                const uint64_t t0 = globaltimer();
                while (!mbar_try_wait(&drain[h], 0) && globaltimer() - t0 < kWaitLimitNs) {
                }
            }
        }
    } else {
        // ---------------- epilogue (16 warps, both CTAs) ----------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsEpi));
        asm volatile("griddepcontrol.wait;" ::: "memory");
        const int w = warp - kEpiWarp0;
        const int h = w >> 3;                    // accumulator (strip pair) this warp drains
        const int q = warp & 3;                  // TMEM lane quarter this warp may access
        float* sx = scales + w * kEpiCols;       // the token scales of this warp's columns
        int t = 0;
        for (int u = cl; u < a.units; u += pairs, ++t) {
            const Unit un = unit_of(u);
            const int c = un.c, j = un.j;
            const Q8WideMember& L = a.m[un.l];
            const int pos = 4 * c + 2 * h + (int)pr;   // pair position of this CTA's strip
            const bool store = pos < L.S;
            const int row = (store ? L.order[pos] : 0) * kStrip + q * 32 + lane;
            const float sw = L.w_scale[row];
            const int cols = tile_tokens(a, j) / 2;    // half of the tile's columns, the first or the second
            const int tok0 = tile_start(a, j) + ((w >> 2) & 1) * cols;
            const int64_t ldy = L.ldy;
            for (int i = lane; i < cols; i += 32) sx[i] = tok0 + i < a.M ? L.x_scale[tok0 + i] : 0.f;
            __syncwarp();
            // (the lanes may see a limit or the abort flag at different times)
            if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[h], t & 1, abort_flag))) {
                if (lane == 0) raise();
                break;
            }
            tc_fence_after();
            const uint32_t taddr =
                tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(h * kAcc1 + ((w >> 2) & 1) * cols);
            auto release = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) remote_arrive(map_to_rank(smem_u32(&acc_empty[h]), 0));
            };
            if constexpr (sizeof(T) == 2) {
                // The whole half-tile is scaled, rounded and packed in registers
                // (two tokens each) and the accumulator handed back before the
                // first store: all CTAs finish a tile at about the same time,
                // and the burst of stores then overlaps the next tile's MMAs.
                // Eight columns at a time, the next eight on their way.
                const uint64_t sw2 = pair2(sw, sw);
                uint32_t p[kEpiCols / 8][4], buf[2][8];
                tmem_ld_32x32b_x8(taddr, buf[0]);
                tc_wait_ld();
#pragma unroll
                for (int k = 0; k < kEpiCols / 8; ++k) {
                    if (8 * k >= cols) break;
                    uint32_t* v = buf[k & 1];
                    if (8 * (k + 1) < cols) tmem_ld_32x32b_x8(taddr + 8 * (k + 1), buf[(k + 1) & 1]);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(sx + 8 * k + 4 * e);
                        const uint32_t* u = v + 4 * e;
                        p[k][2 * e] = pack2(mul2(mul2(pair2((float)(int)u[0], (float)(int)u[1]), f.x), sw2), T());
                        p[k][2 * e + 1] = pack2(mul2(mul2(pair2((float)(int)u[2], (float)(int)u[3]), f.y), sw2), T());
                    }
                    tc_wait_ld();
                }
                release();
                if (!store) continue;
                // lanes 2i and 2i+1 hold rows 2i and 2i+1 of tokens 2e and 2e+1;
                // after one swap each stores both rows of one token
                const bool odd = lane & 1;
                T* y = static_cast<T*>(L.Y) + (int64_t)(tok0 + odd) * ldy + (row & ~1);
                const int mrem = a.M - tok0 - odd;
#pragma unroll
                for (int k = 0; k < kEpiCols / 8; ++k) {
                    if (8 * k >= cols) break;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t got = __shfl_xor_sync(0xffffffffu, p[k][e], 1);
                        const uint32_t two = __byte_perm(p[k][e], got, odd ? 0x3276 : 0x5410);
                        if (8 * k + 2 * e < mrem) __stcs(reinterpret_cast<uint32_t*>(y + (8 * k + 2 * e) * ldy), two);
                    }
                }
            } else {
                T* y = static_cast<T*>(L.Y) + (int64_t)tok0 * ldy + row;
#pragma unroll 1
                for (int k = 0; k < cols && store; k += 16) {
                    uint32_t v[16];
                    tmem_ld_32x32b_x16(taddr + k, v);
                    tc_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (tok0 + k + e < a.M) y[(k + e) * ldy] = (float)(int)v[e] * sx[k + e] * sw;
                }
                release();
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();  // no CTA leaves while the other may still signal it
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc2(tmem_base, kTmemCols);
    }
}

cudaLaunchConfig_t config(int clusters, cudaLaunchAttribute* attr, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * clusters, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cfg;
}

template <int G, class T>
cudaError_t prepare() {
    return cudaFuncSetAttribute(q8_wide_kernel<G, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
}

}  // namespace

cudaError_t q8_prepare_wide(int* max_clusters) {
    cudaError_t e = prepare<1, __nv_bfloat16>();
    if (e == cudaSuccess) e = prepare<1, __half>();
    if (e == cudaSuccess) e = prepare<1, float>();
    if (e == cudaSuccess) e = prepare<kMaxGroup, __nv_bfloat16>();
    if (e == cudaSuccess) e = prepare<kMaxGroup, __half>();
    if (e == cudaSuccess) e = prepare<kMaxGroup, float>();
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = config(1, attr, nullptr);
    return cudaOccupancyMaxActiveClusters(max_clusters, q8_wide_kernel<1, __nv_bfloat16>, &cfg);
}

template <int G>
cudaError_t launch_q8_wide(const Q8Maps<G>& maps, const Q8WideArgs<G>& a, int y_type, int clusters, cudaStream_t st) {
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = config(clusters, attr, st);
    return y_type == kBf16   ? cudaLaunchKernelEx(&cfg, q8_wide_kernel<G, __nv_bfloat16>, maps, a)
           : y_type == kFp16 ? cudaLaunchKernelEx(&cfg, q8_wide_kernel<G, __half>, maps, a)
                             : cudaLaunchKernelEx(&cfg, q8_wide_kernel<G, float>, maps, a);
}
template cudaError_t launch_q8_wide<1>(const Q8Maps<1>&, const Q8WideArgs<1>&, int, int, cudaStream_t);
template cudaError_t launch_q8_wide<kMaxGroup>(const Q8Maps<kMaxGroup>&, const Q8WideArgs<kMaxGroup>&, int, int,
                                               cudaStream_t);

}  // namespace patch
