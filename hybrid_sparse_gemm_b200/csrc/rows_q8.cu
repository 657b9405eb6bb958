// Row operators that end in 8-bit codes: quantisation, RMS norm (with the
// residual's addition) and silu(gate) * up, each one pass over its inputs.
//
// A row y gets the scale s = max(max|y| / 127, 2^-126) and the codes
// round(y / s), ties to even. One reduction per row is enough: with
// y = h * gamma / rms(h), max|y| = max|h * gamma| / rms(h), so the sum of
// squares and the maximum are reduced together. The row stays in registers
// between the reduction and the codes, so every input byte is read once; rows of
// more than 16384 elements, and operands of more than about 8176 that lie at
// different offsets from their 16-byte boundaries, are read a second time for the
// codes. All sums are fp32. A row that holds a NaN or an infinity (or whose sum of
// squares or product with gamma overflows) gets the scale NaN and zero codes, so
// that a product over it is NaN instead of silently wrong.
//
// The kernels are bound by HBM for many rows and by latency for few. A row is
// spread over as many threads as give each one or two groups of eight
// elements (four where the values stay packed); blocks are persistent and read
// their next row before they reduce the present one, so that loads stay in
// flight across the barrier. For many rows the instructions count as much as
// the bytes: about ten an element fill the issue slots that 6.5 TB/s leave.
// Rows that do not lie on 16-byte boundaries are taken in groups that do, with
// the elements before the first and after the last group one to a lane; what
// lies at another offset is shifted into place.
#include <cuda_fp16.h>

#include <atomic>
#include <type_traits>

#include "q8.cuh"

namespace patch {

namespace {

constexpr float kMinScale = 1.17549435e-38f;  // 2^-126

template <class T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_float(float v) { return v; }
template <class T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_float(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_float(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float from_float(float v) { return v; }

// Eight elements as they lie in memory.
template <class T>
struct Raw {
    uint4 w[sizeof(T) / 2];
};
template <class T>
__device__ __forceinline__ Raw<T> load_raw(const T* p) {  // p on a 16-byte boundary
    Raw<T> r;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.w[i] = reinterpret_cast<const uint4*>(p)[i];
    return r;
}
template <class T>
__device__ __forceinline__ void unpack(const Raw<T>& r, float* v) {
    const T* e = reinterpret_cast<const T*>(r.w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_float(e[i]);
}

// Words w[0 .. N) shifted down by `bytes` (0..15, the same in a warp), from N + 4 words.
template <int N>
__device__ __forceinline__ void shift_down(uint32_t* w, int bytes) {
    if (bytes & 8) {
#pragma unroll
        for (int i = 0; i < N + 2; ++i) w[i] = w[i + 2];
    }
    if (bytes & 4) {
#pragma unroll
        for (int i = 0; i < N + 1; ++i) w[i] = w[i + 1];
    }
    if (bytes & 3) {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 8 * (bytes & 3));
    }
}

// Elements [e, e + 8) of a row of K at any alignment; zeros outside the row. No
// byte outside the row is read.
template <class T>
__device__ __forceinline__ void load_any(const T* row, int e, int K, float* v) {
    const int off = (int)(reinterpret_cast<uintptr_t>(row + e) & 15u);
    constexpr int kBytes = 8 * (int)sizeof(T);
    const int64_t at = (int64_t)e * (int)sizeof(T) - off;  // from the row's start, of the boundary below
    if (off == 0 && e >= 0 && e + 8 <= K) {
        unpack(load_raw(row + e), v);
    } else if (at >= 0 && at + kBytes + 16 <= (int64_t)K * (int)sizeof(T)) {
        __align__(16) uint32_t w[kBytes / 4 + 4];
        const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(row) + at);
#pragma unroll
        for (int i = 0; i < kBytes / 16 + 1; ++i) reinterpret_cast<uint4*>(w)[i] = p[i];
        shift_down<kBytes / 4>(w, off);
        const T* x = reinterpret_cast<const T*>(w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_float(x[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = e + i >= 0 && e + i < K ? to_float(row[e + i]) : 0.f;
    }
}
template <class T>
__device__ __forceinline__ void store_any(T* row, int e, int K, const float* v) {
    const bool whole = e >= 0 && e + 8 <= K;
    __align__(16) T x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = from_float<T>(v[i]);
    if (whole && (reinterpret_cast<uintptr_t>(row + e) & 15u) == 0) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i)
            reinterpret_cast<uint4*>(row + e)[i] = reinterpret_cast<const uint4*>(x)[i];
    } else if (whole && (reinterpret_cast<uintptr_t>(row + e) & 3u) == 0) {
#pragma unroll
        for (int i = 0; i < 2 * (int)sizeof(T); ++i)
            reinterpret_cast<uint32_t*>(row + e)[i] = reinterpret_cast<const uint32_t*>(x)[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (e + i >= 0 && e + i < K) row[e + i] = x[i];
    }
}

// What turns a row's values into codes: round(v * pre * up / step).
struct RowScale {
    float pre, up;  // both 1 unless the scale is very small
    float step, inv;  // inv: 1 / step, rounded
    bool finite;
};

// round(v / step), ties to even, as the low byte, the quotient being the one of an
// fp32 division: one Newton step on v * inv gives it (P. Markstein, IBM J. Res.
// Dev. 34, 1990), a sum with 1.5 * 2^23 rounds it into the low bits (it is at most
// 127). Tried on the CPU against rint(v / step) at every tie n + 1/2, n < 128, with
// every mantissa of the step and the nine values around the tie: no code differs;
// with the product v * inv alone, 6 in 100 of them do. Quotients near a tie are not
// rare, since half a row's maximum lies at 63.5. The remainder v - q * step has to be
// representable: row_scale lifts steps below 2^-64.
__device__ __forceinline__ uint32_t code_bits(float v, const RowScale& s) {
    const float q = __fmul_rn(v, s.inv);
    return __float_as_uint(__fadd_rn(__fmaf_rn(__fmaf_rn(-q, s.step, v), s.inv, q), 12582912.f));
}
// The same for two values at once: half the instructions.
__device__ __forceinline__ uint2 code_bits2(float v0, float v1, const RowScale& s) {
    uint32_t a, b;
    asm("{\n\t.reg .b64 v, q, r, i, d, m;\n\t"
        "mov.b64 v, {%2, %3};\n\t"
        "mov.b64 i, {%4, %4};\n\t"
        "mov.b64 d, {%5, %5};\n\t"
        "mov.b64 m, {%6, %6};\n\t"
        "mul.rn.f32x2 q, v, i;\n\t"
        "fma.rn.f32x2 r, q, d, v;\n\t"  // d: -step, so that (-q) * step = q * d
        "fma.rn.f32x2 q, r, i, q;\n\t"
        "add.rn.f32x2 q, q, m;\n\t"
        "mov.b64 {%0, %1}, q;\n\t}"
        : "=r"(a), "=r"(b)
        : "f"(v0), "f"(v1), "f"(s.inv), "f"(-s.step), "f"(12582912.f));
    return make_uint2(a, b);
}
__device__ __forceinline__ uint2 codes8(const float* v, const RowScale& s) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint2 a = code_bits2(v[4 * i], v[4 * i + 1], s), b = code_bits2(v[4 * i + 2], v[4 * i + 3], s);
        w[i] = s.finite ? __byte_perm(__byte_perm(a.x, a.y, 0x0040), __byte_perm(b.x, b.y, 0x0040), 0x5410) : 0u;
    }
    return make_uint2(w[0], w[1]);
}
// Codes off their rows' 8-byte boundaries by `off` (1..7): each lane stores the
// aligned word made of the last `off` codes of its group c and the first ones of
// the group after it (next); where there is none beside it, and before the
// first group, the codes go in pieces of 4, 2 and 1. p: the group's first code.
__device__ __forceinline__ void store_codes_off(int8_t* p, int off, uint2 c, uint2 next, bool has_prev, bool has_next) {
    const int skip = 8 - off;  // codes before the boundary
    uint32_t w[4] = {c.x, c.y, next.x, next.y};
    if (skip & 4) {
        w[0] = w[1];
        w[1] = w[2];
        w[2] = w[3];
    }
    w[0] = __funnelshift_r(w[0], w[1], 8 * (skip & 3));
    w[1] = __funnelshift_r(w[1], w[2], 8 * (skip & 3));
    if (has_next) {
        *reinterpret_cast<uint2*>(p + skip) = make_uint2(w[0], w[1]);
    } else {
        int8_t* t = p + skip;
        uint32_t left = w[0];
        if (off & 4) {
            *reinterpret_cast<uint32_t*>(t) = left;
            t += 4;
            left = w[1];
        }
        if (off & 2) {
            *reinterpret_cast<uint16_t*>(t) = (uint16_t)left;
            t += 2;
            left >>= 16;
        }
        if (off & 1) *t = (int8_t)left;
    }
    if (!has_prev) {
        int8_t* t = p;
        uint32_t lo = c.x, hi = c.y;
        if (skip & 1) {
            *t++ = (int8_t)lo;
            lo = __funnelshift_r(lo, hi, 8);
            hi >>= 8;
        }
        if (skip & 2) {
            *reinterpret_cast<uint16_t*>(t) = (uint16_t)lo;
            t += 2;
            lo = __funnelshift_r(lo, hi, 16);
        }
        if (skip & 4) *reinterpret_cast<uint32_t*>(t) = lo;
    }
}
// The codes of elements [e, e + 8) of a row of K, wherever they lie.
__device__ __forceinline__ void store_codes_any(int8_t* row, int e, int K, uint2 c) {
    int8_t* p = row + e;
    if (e >= 0 && e + 8 <= K) {
        const int off = (int)(reinterpret_cast<uintptr_t>(p) & 7u);
        if (off == 0) *reinterpret_cast<uint2*>(p) = c;
        else store_codes_off(p, off, c, c, false, false);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (e + i >= 0 && e + i < K) p[i] = (int8_t)((i < 4 ? c.x >> (8 * i) : c.y >> (8 * (i - 4))) & 0xFFu);
    }
}

// g / (1 + e^-g) * u. For g below -88 the exponential is infinite and the
// result zero (exactly, below 3e-37 * |u|).
__device__ __forceinline__ float silu_mul(float g, float u) {
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(1.f + __expf(-g)));  // within one unit; 0 for infinity
    return g * r * u;
}

// max(m, |v|), NaN if either is.
__device__ __forceinline__ float max_abs(float m, float v) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(v)));
    return r;
}

__host__ __device__ constexpr bool two_inputs(int mode) { return mode == kRowNormResidual || mode == kRowSiluMul; }
__host__ __device__ constexpr bool is_norm(int mode) { return mode == kRowNorm || mode == kRowNormResidual; }

// From the inputs x and r of a group: v = y (h * gamma for the norms), the sum
// of squares of h, and h in x's place where there is a residual. The sum of two
// 16-bit numbers is rounded once, as it would be from fp32.
__device__ __forceinline__ void add_raw(Raw<__nv_bfloat16>& x, const Raw<__nv_bfloat16>& r) {
    __nv_bfloat162* a = reinterpret_cast<__nv_bfloat162*>(x.w);
    const __nv_bfloat162* b = reinterpret_cast<const __nv_bfloat162*>(r.w);
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = __hadd2_rn(a[i], b[i]);
}
__device__ __forceinline__ void add_raw(Raw<__half>& x, const Raw<__half>& r) {
    __half2* a = reinterpret_cast<__half2*>(x.w);
    const __half2* b = reinterpret_cast<const __half2*>(r.w);
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = __hadd2_rn(a[i], b[i]);
}
__device__ __forceinline__ void add_raw(Raw<float>& x, const Raw<float>& r) {
    float* a = reinterpret_cast<float*>(x.w);
    const float* b = reinterpret_cast<const float*>(r.w);
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] += b[i];
}
template <class T, int MODE>
__device__ __forceinline__ void combine(Raw<T>& x, const Raw<T>& r, const float* gamma, float* v, float& ss) {
    if (MODE == kRowNormResidual) add_raw(x, r);
    unpack(x, v);
    if (MODE == kRowSiluMul) {
        float u[8];
        unpack(r, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = silu_mul(v[i], u[i]);
    }
    if (is_norm(MODE)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            ss = __fmaf_rn(v[i], v[i], ss);
            v[i] *= gamma[i];
        }
    }
}

// The same for one element.
template <class T, int MODE>
__device__ __forceinline__ float combine_one(T& x, T r, T gamma, float& ss) {
    if (MODE == kRowNormResidual) x = from_float<T>(to_float(x) + to_float(r));
    float v = to_float(x);
    if (MODE == kRowSiluMul) v = silu_mul(v, to_float(r));
    if (is_norm(MODE)) {
        ss = __fmaf_rn(v, v, ss);
        v *= to_float(gamma);
    }
    return v;
}

// Reduces the row's maximum and sum over the blockDim.x threads that hold it,
// and writes its scale. s: 64 words, another set for the row after this one.
template <int MODE>
__device__ __forceinline__ RowScale row_scale(const RowArgs& a, int64_t row, float largest, float ss, uint32_t* s) {
    // as bits: ordered like the values, NaN above infinity
    uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(largest));
    if (is_norm(MODE)) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
    if (blockDim.x > 32) {  // (then blockDim.y is 1)
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
        if (lane == 0) {
            s[warp] = top;
            s[32 + warp] = __float_as_uint(ss);
        }
        __syncthreads();
        top = __reduce_max_sync(0xffffffffu, lane < warps ? s[lane] : 0u);
        if (is_norm(MODE)) {
            ss = lane < warps ? __uint_as_float(s[32 + lane]) : 0.f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        }
    }
    // The norm is common to a row's values and its scale: codes come from v and
    // max|v| alone, so they do not depend on the order of the sum of squares
    // (unless the scale is at its least).
    RowScale x;
    x.finite = top < 0x7F800000u;
    const float most = __uint_as_float(top);
    float scale = most / 127.f;
    x.step = scale;
    x.pre = x.up = 1.f;
    if (is_norm(MODE)) {
        const float r = rsqrtf(ss / (float)a.K + a.eps);
        scale = most * r / 127.f;
        x.finite = x.finite && ss < INFINITY && scale < INFINITY;
        if (x.step < kMinScale || scale < kMinScale) {
            x.pre = r;
            x.step = scale;
        }
    }
    scale = fmaxf(scale, kMinScale);
    x.step = fmaxf(x.step, kMinScale);
    if (x.step < 0x1p-64f) {  // both lifted by the same power of two
        x.up = 0x1p62f;
        x.step *= x.up;
    }
    x.inv = 1.f / x.step;
    if (threadIdx.x == 0) a.scale[row] = x.finite ? scale : __uint_as_float(0x7FC00000u);
    return x;
}
__device__ __forceinline__ void look(const float* v, float& top) {
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max_abs(top, v[i]);
}
// The same for a group as it lies in memory.
__device__ __forceinline__ void look(const Raw<__nv_bfloat16>& x, float& top) {
    const __nv_bfloat162* e = reinterpret_cast<const __nv_bfloat162*>(x.w);
    __nv_bfloat162 m = __habs2(e[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) m = __hmax2_nan(m, __habs2(e[i]));
    top = max_abs(max_abs(top, __low2float(m)), __high2float(m));
}
__device__ __forceinline__ void look(const Raw<__half>& x, float& top) {
    const __half2* e = reinterpret_cast<const __half2*>(x.w);
    __half2 m = __habs2(e[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) m = __hmax2_nan(m, __habs2(e[i]));
    top = max_abs(max_abs(top, __low2float(m)), __high2float(m));
}
__device__ __forceinline__ void look(const Raw<float>& x, float& top) {
    look(reinterpret_cast<const float*>(x.w), top);
}
// all(lifted) makes a row's codes: in one go where the values are taken as they
// are, which nearly all rows' are. (A branch at every group keeps the compiler from
// mixing the groups' instructions.)
template <bool LIFTED>
__device__ __forceinline__ uint2 codes_of(float* v, const RowScale& s) {
    if (LIFTED) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] * s.pre * s.up;
    }
    return codes8(v, s);
}
template <class All>
__device__ __forceinline__ void make_codes(const RowScale& s, All all) {
    if (s.pre == 1.f && s.up == 1.f) all(std::false_type());
    else all(std::true_type());
}

// blockDim.x threads per row (one warp, then blockDim.y rows at a time; or the
// whole block), ITEMS groups each. All rows on 16-byte boundaries (the codes' on
// 8-byte ones), K % 8 == 0.
template <class T, int MODE, int ITEMS, int THREADS>
__global__ void __launch_bounds__(THREADS) rows_kernel(const RowArgs a) {
    __shared__ uint32_t s[2][64];
    // quantisation needs the values twice, but never as fp32 at once
    constexpr bool kPacked = MODE == kRowQuantize;
    const int n = blockDim.x;
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    auto group = [&](int i) { return (i * n + (int)threadIdx.x) * 8; };
    Raw<T> x[ITEMS], r[two_inputs(MODE) ? ITEMS : 1], gamma[is_norm(MODE) ? ITEMS : 1];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {  // zeros past the row
        x[i] = {};
        if constexpr (two_inputs(MODE)) r[i] = {};
        if constexpr (is_norm(MODE)) {
            gamma[i] = {};
            if (group(i) < a.K) gamma[i] = load_raw(static_cast<const T*>(a.gamma) + group(i));
        }
    }
    auto fetch = [&](int64_t m) {
        const T* px = static_cast<const T*>(a.x) + m * a.ldx;
        const T* pr = static_cast<const T*>(a.r) + m * a.ldr;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
            if (group(i) < a.K) {
                x[i] = load_raw(px + group(i));
                if constexpr (two_inputs(MODE)) r[i] = load_raw(pr + group(i));
            }
    };
    if (row < a.M) fetch(row);
    for (int turn = 0; row < a.M; row += step, turn ^= 1) {
        float v[kPacked ? 1 : ITEMS][8], ss = 0.f, top = 0.f;
        Raw<T> now[kPacked ? ITEMS : 1];
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            if constexpr (kPacked) {
                now[i] = x[i];
                look(x[i], top);
            } else {
                float g[8];
                if constexpr (is_norm(MODE)) unpack(gamma[i], g);
                combine<T, MODE>(x[i], r[two_inputs(MODE) ? i : 0], g, v[i], ss);
                if (MODE == kRowNormResidual && group(i) < a.K)
                    *reinterpret_cast<Raw<T>*>(static_cast<T*>(a.ro) + row * a.ldo + group(i)) = x[i];
                look(v[i], top);
                // (h stays in x past the row: zeros, as they were)
            }
        }
        if (row + step < a.M) fetch(row + step);
        const RowScale sc = row_scale<MODE>(a, row, top, ss, s[turn]);
        int8_t* q = a.q + row * a.ldq;
        make_codes(sc, [&](auto lifted) {
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                if constexpr (kPacked) unpack(now[i], v[0]);
                const uint2 c = codes_of<lifted>(v[kPacked ? 0 : i], sc);
                if (group(i) < a.K) *reinterpret_cast<uint2*>(q + group(i)) = c;
            }
        });
    }
}

// The same for rows at any alignment; x, r and ro lie at the same offset from a
// 16-byte boundary. A warp's groups are consecutive. gamma's copy in shared
// memory: it lies at another offset from the groups in every row.
template <class T, int MODE, int ITEMS, int THREADS>
__global__ void __launch_bounds__(THREADS) rows_edge_kernel(const RowArgs a) {
    __shared__ uint32_t s[2][64];
    extern __shared__ uint4 copy_of_gamma[];
    T* gamma = reinterpret_cast<T*>(copy_of_gamma);
    constexpr bool kPacked = MODE == kRowQuantize;
    const int lane = threadIdx.x & 31;
    const int first = ((int)threadIdx.x >> 5) * 32 * ITEMS + lane;  // this thread's first group
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // elements before the first group, groups, and this lane's element beside them (-1: none)
    struct Split {
        int head, groups, beside;
    };
    auto split = [&](int64_t m) {
        Split p;
        const int mis = (int)(reinterpret_cast<uintptr_t>(static_cast<const T*>(a.x) + m * a.ldx) & 15u);
        p.head = min(a.K, (16 - mis) % 16 / (int)sizeof(T));
        p.groups = (a.K - p.head) / 8;
        const int tail = a.K - p.head - 8 * p.groups, t = (int)threadIdx.x;
        p.beside = t < p.head ? t : t >= 8 && t < 8 + tail ? a.K - tail + t - 8 : -1;
        return p;
    };
    Raw<T> x[ITEMS], r[two_inputs(MODE) ? ITEMS : 1];
    T bx = from_float<T>(0.f), br = bx;  // the element beside the groups
    auto fetch = [&](int64_t m) {
        const Split p = split(m);
        const T* px = static_cast<const T*>(a.x) + m * a.ldx;
        const T* pr = static_cast<const T*>(a.r) + m * a.ldr;
        if (p.beside >= 0) {
            bx = px[p.beside];
            if (two_inputs(MODE)) br = pr[p.beside];
        }
        px += p.head;
        pr += p.head;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int g = first + 32 * i;
            if (g < p.groups) {
                x[i] = load_raw(px + 8 * g);
                if constexpr (two_inputs(MODE)) r[i] = load_raw(pr + 8 * g);
            } else {
                x[i] = {};
                if constexpr (two_inputs(MODE)) r[i] = {};
            }
        }
    };
    if (row < a.M) fetch(row);
    if constexpr (is_norm(MODE)) {
        const int all = blockDim.x * blockDim.y, t = threadIdx.y * blockDim.x + threadIdx.x;
        for (int k = t; k < a.K; k += all) gamma[k] = static_cast<const T*>(a.gamma)[k];
        __syncthreads();
    }
    for (int turn = 0; row < a.M; row += step, turn ^= 1) {
        const Split p = split(row);
        float v[kPacked ? 1 : ITEMS][8], ss = 0.f, top = 0.f, bv = 0.f;
        Raw<T> now[kPacked ? ITEMS : 1];
        T* ro = static_cast<T*>(a.ro) + row * a.ldo;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            if constexpr (kPacked) {
                now[i] = x[i];
                look(x[i], top);
            } else {
                const int g = first + 32 * i, e = p.head + 8 * g;
                float y[8];
                if constexpr (is_norm(MODE)) {
                    if (g < p.groups) {
                        // two boundaries' worth (the copy has room behind it), shifted
                        constexpr int kWords = 2 * (int)sizeof(T);
                        __align__(16) uint32_t w[kWords + 4];
                        const int at = e * (int)sizeof(T);
#pragma unroll
                        for (int k = 0; k < kWords / 4 + 1; ++k)
                            reinterpret_cast<uint4*>(w)[k] = copy_of_gamma[at / 16 + k];
                        shift_down<kWords>(w, at & 15);
                        const T* z = reinterpret_cast<const T*>(w);
#pragma unroll
                        for (int k = 0; k < 8; ++k) y[k] = to_float(z[k]);
                    } else {
#pragma unroll
                        for (int k = 0; k < 8; ++k) y[k] = 0.f;
                    }
                }
                combine<T, MODE>(x[i], r[two_inputs(MODE) ? i : 0], y, v[i], ss);
                if (MODE == kRowNormResidual && g < p.groups) *reinterpret_cast<Raw<T>*>(ro + e) = x[i];
                look(v[i], top);
            }
        }
        if (p.beside >= 0) {
            bv = combine_one<T, MODE>(bx, br, is_norm(MODE) ? gamma[p.beside] : bx, ss);
            if (MODE == kRowNormResidual) ro[p.beside] = bx;
            top = max_abs(top, bv);
        }
        if (row + step < a.M) fetch(row + step);
        const RowScale sc = row_scale<MODE>(a, row, top, ss, s[turn]);
        int8_t* q = a.q + row * a.ldq + p.head;
        const int off = (int)(reinterpret_cast<uintptr_t>(q) & 7u);  // of every group
        uint2 c[ITEMS];
        make_codes(sc, [&](auto lifted) {
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                if constexpr (kPacked) unpack(now[i], v[0]);
                c[i] = codes_of<lifted>(v[kPacked ? 0 : i], sc);
            }
        });
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int g = first + 32 * i;
            if (off == 0) {
                if (g < p.groups) *reinterpret_cast<uint2*>(q + 8 * g) = c[i];
            } else {
                // the next group: the next lane's, or the first lane's next
                const bool wrap = lane == 0 && i + 1 < ITEMS;
                const uint2 give = wrap ? c[i + 1 < ITEMS ? i + 1 : i] : c[i];
                uint2 next;
                next.x = __shfl_sync(0xffffffffu, give.x, lane + 1);
                next.y = __shfl_sync(0xffffffffu, give.y, lane + 1);
                const bool has_next = g + 1 < p.groups && (lane < 31 || i + 1 < ITEMS);
                const bool has_prev = g > 0 && (lane > 0 || i > 0);
                if (g < p.groups) store_codes_off(q + 8 * g, off, c[i], next, has_prev, has_next);
            }
        }
        if (p.beside >= 0) {
            bv = bv * sc.pre * sc.up;
            a.q[row * a.ldq + p.beside] = sc.finite ? (int8_t)(code_bits(bv, sc) & 0xFFu) : (int8_t)0;
        }
    }
}

// Inputs at any alignment, in groups that lie on x's 16-byte boundaries.
// ITEMS = 0: rows of any length, read a second time for the codes.
template <class T, int MODE, int ITEMS>
__global__ void __launch_bounds__(512) rows_any_kernel(const RowArgs a) {
    __shared__ uint32_t s[2][64];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    const int n = blockDim.x;
    int turn = 0;
    for (int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; row < a.M; row += step, turn ^= 1) {
        const T* xr = static_cast<const T*>(a.x) + row * a.ldx;
        const int off = (int)(reinterpret_cast<uintptr_t>(xr) & 15u) / (int)sizeof(T);
        auto group = [&](int e, float* v, float& ss, bool again) {
            float o[8], g[8];
            if (MODE == kRowNormResidual && again) {
                load_any(static_cast<const T*>(a.ro) + row * a.ldo, e, a.K, v);
            } else {
                load_any(xr, e, a.K, v);
                if (two_inputs(MODE)) load_any(static_cast<const T*>(a.r) + row * a.ldr, e, a.K, o);
            }
            if (is_norm(MODE)) load_any(static_cast<const T*>(a.gamma), e, a.K, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (MODE == kRowNormResidual && !again) v[i] = o[i] = to_float(from_float<T>(v[i] + o[i]));
                if (MODE == kRowSiluMul) v[i] = silu_mul(v[i], o[i]);
                if (is_norm(MODE)) {
                    ss = __fmaf_rn(v[i], v[i], ss);
                    v[i] *= g[i];
                }
            }
            if (MODE == kRowNormResidual && !again) store_any(static_cast<T*>(a.ro) + row * a.ldo, e, a.K, o);
        };
        float ss = 0.f, top = 0.f;
        if constexpr (ITEMS > 0) {
            float v[ITEMS][8];
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                group((i * n + (int)threadIdx.x) * 8 - off, v[i], ss, false);
                look(v[i], top);
            }
            const RowScale sc = row_scale<MODE>(a, row, top, ss, s[turn]);
            make_codes(sc, [&](auto lifted) {
#pragma unroll
                for (int i = 0; i < ITEMS; ++i)
                    store_codes_any(a.q + row * a.ldq, (i * n + (int)threadIdx.x) * 8 - off, a.K, codes_of<lifted>(v[i], sc));
            });
        } else {
            // whole warps take part to the end, for the exchange between lanes
            const int64_t end = ((int64_t)a.K + off + 8 * n - 1) / (8 * n) * (8 * n);
            float v[8], unused = 0.f;
            for (int64_t e = (int64_t)threadIdx.x * 8; e < end; e += 8 * n) {
                group((int)e - off, v, ss, false);
                look(v, top);
            }
            const RowScale sc = row_scale<MODE>(a, row, top, ss, s[turn]);
            for (int64_t e = (int64_t)threadIdx.x * 8; e < end; e += 8 * n) {
                group((int)e - off, v, unused, true);
                store_codes_any(a.q + row * a.ldq, (int)e - off, a.K, codes_of<true>(v, sc));
            }
        }
    }
}

// A launch whose set-up may overlap the stream's previous kernel (the kernels
// wait for it before they touch memory).
template <class... Params, class... Args>
cudaError_t go(void (*kernel)(Params...), dim3 grid, dim3 block, int smem, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Persistent blocks: as many as are resident, found once per kernel and block size (by warps per block).
template <class... Params>
cudaError_t resident(void (*kernel)(Params...), int threads, std::atomic<int>* known, int* per_sm) {
    int n = known[threads / 32].load(std::memory_order_relaxed);
    if (n == 0) {
        cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, 0);
        if (e != cudaSuccess) return e;
        n = n < 1 ? 1 : n;
        known[threads / 32].store(n, std::memory_order_relaxed);
    }
    *per_sm = n;
    return cudaSuccess;
}

constexpr int kGammaBytes = 200 * 1024;  // of an SM's shared memory for the blocks' copies of gamma

template <class T, int MODE, int ITEMS, bool EDGE, int THREADS>
cudaError_t launch_instance(const RowArgs& a, dim3 block, int sms, cudaStream_t st) {
    static std::atomic<int> known[33];
    void (*kernel)(RowArgs);
    if constexpr (EDGE) kernel = rows_edge_kernel<T, MODE, ITEMS, THREADS>;
    else kernel = rows_kernel<T, MODE, ITEMS, THREADS>;
    int per_sm = 1;
    const cudaError_t e = resident(kernel, (int)(block.x * block.y), known, &per_sm);
    if (e != cudaSuccess) return e;
    // gamma's copy, and room for the words read behind it
    int smem = 0;
    if constexpr (EDGE && is_norm(MODE)) {
        smem = (a.K * (int)sizeof(T) + 15) / 16 * 16 + 32;
        if (per_sm > kGammaBytes / smem) per_sm = kGammaBytes / smem;
    }
    const int64_t rows = (a.M + block.y - 1) / block.y, most = (int64_t)sms * per_sm;
    return go(kernel, dim3((unsigned)(rows < most ? rows : most)), block, smem, st, a);
}

template <class T, int MODE, int ITEMS>
cudaError_t launch_any(const RowArgs& a, dim3 block, int sms, cudaStream_t st) {
    static std::atomic<int> known[33];
    auto kernel = rows_any_kernel<T, MODE, ITEMS>;
    int per_sm = 1;
    const cudaError_t e = resident(kernel, (int)(block.x * block.y), known, &per_sm);
    if (e != cudaSuccess) return e;
    const int64_t rows = (a.M + block.y - 1) / block.y, most = (int64_t)sms * per_sm;
    return go(kernel, dim3((unsigned)(rows < most ? rows : most)), block, 0, st, a);
}

template <class T, int MODE>
cudaError_t launch_rows(const RowArgs& a, int sms, cudaStream_t st) {
    auto at = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
    auto pitch = [](int64_t ld) { return (uintptr_t)(ld * (int64_t)sizeof(T)); };
    // r and ro at x's offset from a 16-byte boundary in every row
    auto with_x = [&](const void* p, int64_t ld) {
        return !p || (((at(p) - at(a.x)) | (pitch(ld) - pitch(a.ldx))) & 15u) == 0;
    };
    const bool same = with_x(a.r, a.ldr) && with_x(a.ro, a.ldo);
    const bool aligned = same && a.K % 8 == 0 && ((at(a.x) | pitch(a.ldx) | at(a.gamma)) & 15u) == 0 &&
                         ((at(a.q) | (uintptr_t)a.ldq) & 7u) == 0;
    const int64_t groups = (a.K + 7) / 8;  // of eight elements in a row
    // gamma's copy has to fit what a block may use without asking
    const bool edge = same && !(is_norm(MODE) && (int64_t)a.K * (int)sizeof(T) > 47 * 1024);
    auto threads = [&](int items) { return (groups + items - 1) / items + 31 & ~(int64_t)31; };
    dim3 block(32, 1);
    int items = 0;
    // Four groups a thread halve what a row's reduction costs each element, two
    // leave room for more threads. Measured (bf16, us with four and with two): norm
    // 8192 x 5120 25.9 and 32.7, with residual 47.4 and 47.7, quantise 22.6 and 24.6,
    // silu * up 4096 x 8192 33.2 and 35.2, but 2048 x 13824 33.3 and 31.7 (norm with
    // residual 4096 x 12288 59.7 and 66.4: with 1024 threads it spills 48 bytes). Off
    // the boundaries four only: 2048 x 13823 38 (36, and 43 with two, when a code was
    // one product). fp32 (norm and residual, 4096 x 4096): 43.9 and 34.8.
    const bool four = sizeof(T) == 2 && threads(4) >= 64 && threads(4) <= (aligned ? 256 : 512);
    if (groups <= 64) {
        // a warp per row, eight rows per block
        items = groups <= 32 ? 1 : 2;
        block.y = (unsigned)(a.M < 8 ? a.M : 8);
    } else if (threads(1) <= 512 && a.M <= sms) {
        items = 1;  // few rows: the shortest way through one
    } else if (four) {
        items = 4;
    } else if (threads(2) <= (sizeof(T) == 2 ? 1024 : 512)) {
        items = 2;
    } else if (threads(4) <= 512) {
        items = 4;
    }
    if (groups > 64 && items > 0) block.x = (unsigned)threads(items);
    if (items == 0 || !(aligned || edge)) {
        // (groups on x's boundaries: one more, where the first is partial)
        const int64_t two = (groups + 2) / 2 + 31 & ~(int64_t)31;
        if (items == 0 || two > 512) return launch_any<T, MODE, 0>(a, dim3(512, 1), sms, st);
        if (two > 32) block = dim3((unsigned)two, 1);
        return launch_any<T, MODE, 2>(a, block, sms, st);
    }
#define PATCH_ROWS(ITEMS, THREADS)                                                  \
    (aligned ? launch_instance<T, MODE, ITEMS, false, THREADS>(a, block, sms, st) \
             : launch_instance<T, MODE, ITEMS, true, THREADS>(a, block, sms, st))
    if (items == 1) return PATCH_ROWS(1, 512);
    if (items == 4) return PATCH_ROWS(4, 512);
    // (off the boundaries, rows of that length took four groups)
    if constexpr (sizeof(T) == 2)
        if (aligned && block.x > 512) return launch_instance<T, MODE, 2, false, 1024>(a, block, sms, st);
    return PATCH_ROWS(2, 512);
#undef PATCH_ROWS
}

template <class T>
cudaError_t launch_rows_type(const RowArgs& a, int mode, int sms, cudaStream_t st) {
    return mode == kRowQuantize       ? launch_rows<T, kRowQuantize>(a, sms, st)
           : mode == kRowNorm         ? launch_rows<T, kRowNorm>(a, sms, st)
           : mode == kRowNormResidual ? launch_rows<T, kRowNormResidual>(a, sms, st)
                                      : launch_rows<T, kRowSiluMul>(a, sms, st);
}

// values = code * scale, the fp32 product rounded to the output's type, in groups
// on the output's 16-byte boundaries. A thread takes kDeq groups, a block's row
// apart: their loads are in flight together.
constexpr int kDeq = 2;
template <class T>
__global__ void __launch_bounds__(256) dequantize_kernel(const int8_t* q, int64_t ldq, const float* scale, int64_t M,
                                                         int K, int chunks, T* out, int64_t ldo) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t row = (int64_t)(blockIdx.x / chunks) * blockDim.y + threadIdx.y;
    if (row >= M) return;
    const float s = scale[row];
    const int8_t* qr = q + row * ldq;
    T* orow = out + row * ldo;
    const int first = (int)(blockIdx.x % chunks) * (int)blockDim.x * kDeq + (int)threadIdx.x;
    const int lead = (int)(reinterpret_cast<uintptr_t>(orow) & 15u) / (int)sizeof(T);
    uint32_t w[kDeq][4];
#pragma unroll
    for (int i = 0; i < kDeq; ++i) {
        const int e = (first + i * (int)blockDim.x) * 8 - lead;
        const int off = (int)(reinterpret_cast<uintptr_t>(qr + e) & 7u);
        if (e >= K) continue;
        if (off == 0 && e >= 0 && e + 8 <= K) {
            *reinterpret_cast<uint2*>(w[i]) = *reinterpret_cast<const uint2*>(qr + e);
        } else if (e - off >= 0 && e - off + 16 <= K) {
            *reinterpret_cast<uint2*>(w[i]) = *reinterpret_cast<const uint2*>(qr + e - off);
            *reinterpret_cast<uint2*>(w[i] + 2) = *reinterpret_cast<const uint2*>(qr + e - off + 8);
            if (off & 4) {
                w[i][0] = w[i][1];
                w[i][1] = w[i][2];
                w[i][2] = w[i][3];
            }
            if (off & 3) {
                w[i][0] = __funnelshift_r(w[i][0], w[i][1], 8 * (off & 3));
                w[i][1] = __funnelshift_r(w[i][1], w[i][2], 8 * (off & 3));
            }
        } else {
            w[i][0] = w[i][1] = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (e + k >= 0 && e + k < K) w[i][k >> 2] |= (uint32_t)(uint8_t)qr[e + k] << (8 * (k & 3));
        }
    }
#pragma unroll
    for (int i = 0; i < kDeq; ++i) {
        const int e = (first + i * (int)blockDim.x) * 8 - lead;
        if (e >= K) continue;
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = (float)(int8_t)(w[i][k >> 2] >> (8 * (k & 3))) * s;
        store_any(orow, e, K, v);
    }
}

template <class T>
cudaError_t launch_deq(const int8_t* q, int64_t ldq, const float* scale, int64_t M, int K, T* out, int64_t ldo,
                       cudaStream_t st) {
    // a row in as few blocks as hold it at kDeq groups a thread, all but full (rows
    // off the 16-byte boundaries may have a group more); short rows share a block
    const bool aligned = K % 8 == 0 && ((reinterpret_cast<uintptr_t>(out) | (uintptr_t)(ldo * (int64_t)sizeof(T))) & 15u) == 0;
    const int64_t groups = ((int64_t)K + 7) / 8 + (aligned ? 0 : 1);
    const int chunks = (int)((groups + 256 * kDeq - 1) / (256 * kDeq));
    const unsigned x = (unsigned)((groups + kDeq * chunks - 1) / (kDeq * chunks) + 31) / 32 * 32;
    const dim3 block(x, M < 256 / x ? (unsigned)M : 256 / x);
    // whole rows per launch, within the grid's limit of 2^31 - 1 blocks
    const int64_t most = 2147483647ll / chunks * block.y;
    for (int64_t m0 = 0; m0 < M; m0 += most) {
        const int64_t rows = M - m0 < most ? M - m0 : most;
        const cudaError_t e = go(dequantize_kernel<T>, dim3((unsigned)((rows + block.y - 1) / block.y * chunks)), block, 0, st,
                                 q + m0 * ldq, ldq, scale + m0, rows, K, chunks, out + m0 * ldo, ldo);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_rows_q8(const RowArgs& a, int mode, int type, int sms, cudaStream_t st) {
    return type == kBf16   ? launch_rows_type<__nv_bfloat16>(a, mode, sms, st)
           : type == kFp16 ? launch_rows_type<__half>(a, mode, sms, st)
                           : launch_rows_type<float>(a, mode, sms, st);
}

cudaError_t launch_dequantize_q8(const int8_t* q, int64_t ldq, const float* scale, int64_t M, int K, void* out, int64_t ldo,
                                 int type, cudaStream_t st) {
    return type == kBf16   ? launch_deq(q, ldq, scale, M, K, static_cast<__nv_bfloat16*>(out), ldo, st)
           : type == kFp16 ? launch_deq(q, ldq, scale, M, K, static_cast<__half*>(out), ldo, st)
                           : launch_deq(q, ldq, scale, M, K, static_cast<float*>(out), ldo, st);
}

}  // namespace patch
