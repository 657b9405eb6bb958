// Row operators that end in 8-bit codes: quantisation, RMS norm (with the
// residual's addition) and silu(gate) * up, each one pass over its inputs.
//
// A row y gets the scale s = max(max|y| / 127, 2^-126) and the codes
// round(y / s), ties to even. One reduction per row is enough: with
// y = h * gamma / rms(h), max|y| = max|h * gamma| / rms(h), so the sum of
// squares and the maximum are reduced together. The row stays in registers
// between the reduction and the codes, so every input byte is read once.
// All sums are fp32. A row that holds a NaN or an infinity (or whose sum of
// squares overflows) gets the scale NaN and zero codes, so that a product
// over it is NaN instead of silently wrong.
#include <cuda_fp16.h>

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

// VEC consecutive elements: 16-byte accesses for VEC = 8, single ones for VEC = 1.
template <class T, int VEC>
__device__ __forceinline__ void load(const T* p, float* v) {
    if constexpr (VEC == 1) {
        v[0] = to_float(*p);
    } else {
        constexpr int N = VEC * (int)sizeof(T) / 16;
        uint4 raw[N];
#pragma unroll
        for (int i = 0; i < N; ++i) raw[i] = reinterpret_cast<const uint4*>(p)[i];
        const T* e = reinterpret_cast<const T*>(raw);
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = to_float(e[i]);
    }
}
template <class T, int VEC>
__device__ __forceinline__ void store(T* p, const float* v) {
    if constexpr (VEC == 1) {
        *p = from_float<T>(v[0]);
    } else {
        constexpr int N = VEC * (int)sizeof(T) / 16;
        uint4 raw[N];
        T* e = reinterpret_cast<T*>(raw);
#pragma unroll
        for (int i = 0; i < VEC; ++i) e[i] = from_float<T>(v[i]);
#pragma unroll
        for (int i = 0; i < N; ++i) reinterpret_cast<uint4*>(p)[i] = raw[i];
    }
}

// round(v * inv), ties to even, as the low byte: the product is rounded once,
// into the mantissa of 1.5 * 2^23 (|v * inv| is at most 127 and a little).
__device__ __forceinline__ uint32_t code_bits(float v, float inv) {
    return __float_as_uint(__fmaf_rn(v, inv, 12582912.f));
}
template <int VEC>
__device__ __forceinline__ void store_codes(int8_t* p, const float* v, float inv, bool finite) {
    if constexpr (VEC == 1) {
        *p = finite ? (int8_t)(code_bits(v[0], inv) & 0xFFu) : (int8_t)0;
    } else {
        uint32_t w[VEC / 4];
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) {
            const uint32_t lo = __byte_perm(code_bits(v[4 * i], inv), code_bits(v[4 * i + 1], inv), 0x0040);
            const uint32_t hi = __byte_perm(code_bits(v[4 * i + 2], inv), code_bits(v[4 * i + 3], inv), 0x0040);
            w[i] = finite ? __byte_perm(lo, hi, 0x5410) : 0u;
        }
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    }
}

// g / (1 + e^-g) * u, with the exponential of a number below zero so that
// nothing overflows and the divisor stays in [1, 2].
__device__ __forceinline__ float silu_mul(float g, float u) {
    const float t = __expf(-fabsf(g));
    return g * __fdividef(g < 0.f ? t : 1.f, 1.f + t) * u;
}

// One item of a row: VEC values of y (of h * gamma for the norms), the sum of
// squares of h, and the sum h itself written where the mode has a residual.
template <class T, int MODE, int VEC>
__device__ __forceinline__ void item(const RowArgs& a, int64_t row, int e, float* v, float& ss, bool again) {
    const T* x = static_cast<const T*>(a.x) + row * a.ldx + e;
    if (MODE == kRowNormResidual) {
        T* ro = static_cast<T*>(a.ro) + row * a.ldo + e;
        if (again) {
            load<T, VEC>(ro, v);
        } else {
            float r[VEC];
            load<T, VEC>(x, v);
            load<T, VEC>(static_cast<const T*>(a.r) + row * a.ldr + e, r);
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] = to_float(from_float<T>(v[i] + r[i]));
            store<T, VEC>(ro, v);
        }
    } else {
        load<T, VEC>(x, v);
    }
    if (MODE == kRowSiluMul) {
        float u[VEC];
        load<T, VEC>(static_cast<const T*>(a.r) + row * a.ldr + e, u);
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = silu_mul(v[i], u[i]);
    }
    if (MODE == kRowNorm || MODE == kRowNormResidual) {
        float g[VEC];
        load<T, VEC>(static_cast<const T*>(a.gamma) + e, g);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            ss = __fmaf_rn(v[i], v[i], ss);
            v[i] *= g[i];
        }
    }
}

// blockDim.x threads per row (a warp, then blockDim.y rows per block; or the
// whole block), ITEMS vectors of VEC elements each, held in registers;
// ITEMS = 0: rows of any length, read a second time for the codes.
template <class T, int MODE, int VEC, int ITEMS>
__global__ void __launch_bounds__(1024) rows_kernel(const RowArgs a) {
    __shared__ uint32_t s_max[32];
    __shared__ float s_sum[32];
    const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (row >= a.M) return;  // whole warps: rows of a block's y share no barrier
    const int n = blockDim.x;
    float v[ITEMS > 0 ? ITEMS : 1][VEC];
    float ss = 0.f;
    uint32_t top = 0;  // largest |y| as bits: ordered like the values, NaN above infinity
    auto look = [&](const float* y) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) top = max(top, __float_as_uint(y[i]) & 0x7FFFFFFFu);
    };
    if constexpr (ITEMS > 0) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int e = (i * n + (int)threadIdx.x) * VEC;
            if (e < a.K) item<T, MODE, VEC>(a, row, e, v[i], ss, false);
            else
#pragma unroll
                for (int j = 0; j < VEC; ++j) v[i][j] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) look(v[i]);
    } else {
        for (int64_t e = (int64_t)threadIdx.x * VEC; e < a.K; e += (int64_t)n * VEC) {
            item<T, MODE, VEC>(a, row, (int)e, v[0], ss, false);
            look(v[0]);
        }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (MODE == kRowNorm || MODE == kRowNormResidual) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
    if (n > 32) {  // the block's warps in one row (blockDim.y == 1)
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = n >> 5;
        if (lane == 0) {
            s_max[warp] = top;
            s_sum[warp] = ss;
        }
        __syncthreads();
        top = __reduce_max_sync(0xffffffffu, lane < warps ? s_max[lane] : 0u);
        if (MODE == kRowNorm || MODE == kRowNormResidual) {
            ss = lane < warps ? s_sum[lane] : 0.f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        }
    }
    bool finite = top < 0x7F800000u;
    float most = __uint_as_float(top), r = 1.f;
    if (MODE == kRowNorm || MODE == kRowNormResidual) {
        finite = finite && ss < INFINITY;
        r = rsqrtf(ss / (float)a.K + a.eps);
        most *= r;
        finite = finite && most < INFINITY;
    }
    const float scale = fmaxf(most / 127.f, kMinScale);
    const float inv = 1.f / scale;  // at most 2^126
    auto norm = [&](float* y) {
        if (MODE == kRowNorm || MODE == kRowNormResidual) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) y[j] *= r;
        }
    };
    if (threadIdx.x == 0) a.scale[row] = finite ? scale : __uint_as_float(0x7FC00000u);
    int8_t* q = a.q + row * a.ldq;
    if constexpr (ITEMS > 0) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int e = (i * n + (int)threadIdx.x) * VEC;
            norm(v[i]);
            if (e < a.K) store_codes<VEC>(q + e, v[i], inv, finite);
        }
    } else {
        for (int64_t e = (int64_t)threadIdx.x * VEC; e < a.K; e += (int64_t)n * VEC) {
            item<T, MODE, VEC>(a, row, (int)e, v[0], ss, true);
            norm(v[0]);
            store_codes<VEC>(q + e, v[0], inv, finite);
        }
    }
}

// A launch whose set-up may overlap the stream's previous kernel (the kernels
// wait for it before they touch memory).
template <class... Params, class... Args>
cudaError_t go(void (*kernel)(Params...), dim3 grid, dim3 block, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <class T, int MODE>
cudaError_t launch_rows(const RowArgs& a, int sms, cudaStream_t st) {
    auto wide = [](const void* p, int64_t ld) {
        return !p || ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(ld * (int64_t)sizeof(T))) & 15u) == 0;
    };
    const bool vec = a.K % 8 == 0 && wide(a.x, a.ldx) && wide(a.r, a.ldr) && wide(a.ro, a.ldo) && wide(a.gamma, 0) &&
                     ((reinterpret_cast<uintptr_t>(a.q) | (uintptr_t)a.ldq) & 7u) == 0;
    const int64_t items = vec ? a.K / 8 : a.K;  // vectors in a row
    dim3 block(32, 1), grid((unsigned)a.M);
    cudaError_t e = cudaSuccess;
    auto per_row = [&](int each) { return (int)((items + each - 1) / each + 31) / 32 * 32; };
    if (vec) {
        if (items <= 128) {
            block.y = (unsigned)(a.M < 8 ? a.M : 8);
            grid.x = (unsigned)((a.M + block.y - 1) / block.y);
            if (items <= 32) e = go(rows_kernel<T, MODE, 8, 1>, grid, block, st, a);
            else if (items <= 64) e = go(rows_kernel<T, MODE, 8, 2>, grid, block, st, a);
            else e = go(rows_kernel<T, MODE, 8, 4>, grid, block, st, a);
            return e;
        }
        const int most = a.M <= sms ? 1024 : 512;
        if (per_row(1) <= most) {
            block.x = per_row(1);
            e = go(rows_kernel<T, MODE, 8, 1>, grid, block, st, a);
        } else if (per_row(2) <= most) {
            block.x = per_row(2);
            e = go(rows_kernel<T, MODE, 8, 2>, grid, block, st, a);
        } else if (per_row(4) <= 1024) {
            block.x = per_row(4);
            e = go(rows_kernel<T, MODE, 8, 4>, grid, block, st, a);
        } else {
            block.x = 1024;
            e = go(rows_kernel<T, MODE, 8, 0>, grid, block, st, a);
        }
    } else if (items <= 32 * 16) {
        block.y = (unsigned)(a.M < 8 ? a.M : 8);
        grid.x = (unsigned)((a.M + block.y - 1) / block.y);
        e = go(rows_kernel<T, MODE, 1, 16>, grid, block, st, a);
    } else if (items <= 1024 * 16) {
        block.x = per_row(16);
        e = go(rows_kernel<T, MODE, 1, 16>, grid, block, st, a);
    } else {
        block.x = 1024;
        e = go(rows_kernel<T, MODE, 1, 0>, grid, block, st, a);
    }
    return e;
}

template <class T>
cudaError_t launch_rows_type(const RowArgs& a, int mode, int sms, cudaStream_t st) {
    return mode == kRowQuantize       ? launch_rows<T, kRowQuantize>(a, sms, st)
           : mode == kRowNorm         ? launch_rows<T, kRowNorm>(a, sms, st)
           : mode == kRowNormResidual ? launch_rows<T, kRowNormResidual>(a, sms, st)
                                      : launch_rows<T, kRowSiluMul>(a, sms, st);
}

// values = code * scale, one product and one rounding per element.
template <class T, int VEC>
__global__ void __launch_bounds__(256) dequantize_kernel(const int8_t* q, int64_t ldq, const float* scale, int K,
                                                         int chunks, T* out, int64_t ldo) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t row = blockIdx.x / chunks;
    const int e = ((int)(blockIdx.x % chunks) * 256 + (int)threadIdx.x) * VEC;
    if (e >= K) return;
    const float s = scale[row];
    float v[VEC];
    if constexpr (VEC == 1) {
        v[0] = (float)q[row * ldq + e] * s;
    } else {
        const uint2 raw = *reinterpret_cast<const uint2*>(q + row * ldq + e);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = (float)(int8_t)(raw.x >> (8 * i)) * s;
            v[4 + i] = (float)(int8_t)(raw.y >> (8 * i)) * s;
        }
    }
    store<T, VEC>(out + row * ldo + e, v);
}

template <class T>
cudaError_t launch_deq(const int8_t* q, int64_t ldq, const float* scale, int64_t M, int K, T* out, int64_t ldo,
                       cudaStream_t st) {
    const bool vec = K % 8 == 0 && ((reinterpret_cast<uintptr_t>(q) | (uintptr_t)ldq) & 7u) == 0 &&
                     ((reinterpret_cast<uintptr_t>(out) | (uintptr_t)(ldo * (int64_t)sizeof(T))) & 15u) == 0;
    const int chunks = (int)(((int64_t)K + (vec ? 2047 : 255)) / (vec ? 2048 : 256));
    // whole rows per launch, within the grid's limit of 2^31 - 1 blocks
    const int64_t most = 2147483647ll / chunks;
    for (int64_t m0 = 0; m0 < M; m0 += most) {
        const unsigned grid = (unsigned)((M - m0 < most ? M - m0 : most) * chunks);
        const cudaError_t e = go(vec ? dequantize_kernel<T, 8> : dequantize_kernel<T, 1>, dim3(grid), dim3(256), st,
                                 q + m0 * ldq, ldq, scale + m0, K, chunks, out + m0 * ldo, ldo);
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
