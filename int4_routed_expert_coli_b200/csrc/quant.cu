// Rows to 8-bit floating point (e4m3), one fp32 scale per row and block of 128:
//   s[b][r] = max(max_k |x[r][k]| / 448, 2^-126),  q = e4m3(x / s)
// 448 is e4m3's largest value; the quotient is rounded to fp32, then to
// nearest even.  The lower bound keeps the division defined for a block of
// zeros (q = 0) and for one whose scale would be subnormal.  A NaN or an
// infinity in a block makes its scale NaN or infinite, so every product of
// that row is NaN: nothing is hidden.
//
// Moves 3 bytes per bf16 value: 4096 x 6144 18 us, 4.3 TB/s, 16384 x 6144 4.8 TB/s.
// Neither memory nor issue is full (2048 x 6144 under the profiler 2.2 TB/s, issue 48
// %): a warp loads once, reduces, stores and ends, so its loads pass only under other
// warps' conversions.  It holds 1024 values of a row in registers (one read), and the
// scales, stored block-major for the product that reads them, leave through shared
// memory in runs of 8 rows.
#include <cuda_fp8.h>

#include "coli_internal.cuh"
#include "launch.cuh"
#include "ptx.cuh"

namespace coli {
namespace {

constexpr int kQRows = 8;      // rows per CTA, one warp each
constexpr int kQBlocks = 8;    // 128-blocks per CTA

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// x / s rounded to nearest, from r = 1 / s rounded to nearest: one correction of
// x r by its exact remainder (Markstein's theorem, IBM J. Res. Dev. 34, 1990).  A
// division by the same s for every value of a block costs three instructions.
__device__ __forceinline__ float quotient(float x, float s, float r) {
    const float q = x * r;
    return fmaf(fmaf(-q, s, x), r, q);
}

// Two 16-byte halves of 8 fp32 values, or 8 bf16 values in the first.
template <bool kBf16>
struct Raw {
    uint4 u[kBf16 ? 1 : 2];
    __device__ __forceinline__ void load(const void* x, int64_t i) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(x) +
                                                        i * (kBf16 ? 2 : 4));
        u[0] = __ldcs(p);
        if constexpr (!kBf16) u[1] = __ldcs(p + 1);
    }
    __device__ __forceinline__ void values(float (&v)[8]) const {
        if constexpr (kBf16) {
            const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[2 * j] = __uint_as_float(w[j] << 16);
                v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                v[4 * j] = __uint_as_float(u[j].x);
                v[4 * j + 1] = __uint_as_float(u[j].y);
                v[4 * j + 2] = __uint_as_float(u[j].z);
                v[4 * j + 3] = __uint_as_float(u[j].w);
            }
        }
    }
};

// The loads of a thread's four vectors are all in flight and stay packed until
// their turn, so that six CTAs fit an SM (four, with every value unpacked first).
template <bool kBf16>
__global__ void __launch_bounds__(kQRows * 32, kBf16 ? 6 : 4)
quantize_rows_kernel(int R, int K, const void* __restrict__ x, uint8_t* __restrict__ q,
                     float* __restrict__ scales) {
    __shared__ float sc[kQBlocks][kQRows];
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t r0 = (int64_t)blockIdx.x * kQRows;
    const int b0 = blockIdx.y * kQBlocks;
    const int64_t row = r0 + warp;
    const int k0 = b0 * 128 + lane * 8;  // half a warp per block of 128
    if (row < R) {
        Raw<kBf16> raw[4] = {};
#pragma unroll
        for (int i = 0; i < 4; ++i)  // K is a multiple of 16: whole vectors
            if (k0 + i * 256 < K) raw[i].load(x, row * K + k0 + i * 256);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v[8];
            raw[i].values(v);
            float m = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max_nan(m, fabsf(v[j]));
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float s = max_nan(__fdiv_rn(m, 448.f), 1.17549435e-38f);
            const float inv = __frcp_rn(s);
            // the correction's terms are exact away from the ends of fp32's range
            const bool inner = s > 1e-30f && s < 1e30f;
            if (k0 + i * 256 < K) {
                uint32_t w[2];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float a = v[2 * j], b = v[2 * j + 1];
                    const float2 f = inner ? make_float2(quotient(a, s, inv), quotient(b, s, inv))
                                           : make_float2(__fdiv_rn(a, s), __fdiv_rn(b, s));
                    const __nv_fp8x2_storage_t p =
                        __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
                    if (j & 1) w[j >> 1] |= (uint32_t)p << 16;
                    else w[j >> 1] = p;
                }
                *reinterpret_cast<uint2*>(q + row * K + k0 + i * 256) = make_uint2(w[0], w[1]);
            }
            if ((lane & 15) == 0) sc[2 * i + (lane >> 4)][warp] = s;
        }
    }
    __syncthreads();
    const int b = threadIdx.x / kQRows, i = threadIdx.x % kQRows;
    if (b < kQBlocks && b0 + b < (K + 127) / 128 && r0 + i < R)
        scales[(int64_t)(b0 + b) * R + r0 + i] = sc[b][i];
}

}  // namespace
}  // namespace coli

using namespace coli;

extern "C" coli_status coli_moe_fp8_quantize_rows(int32_t R, int32_t K, const void* x,
                                                  coli_out_dtype x_dtype, uint8_t* q,
                                                  float* scales, void* stream) {
    if (R < 0 || K < 1 || !valid_dtype(x_dtype)) return COLI_ERR_INVALID_ARG;
    if (K % 16 || K > 65536 || R > 1 << 24) return COLI_ERR_SHAPE;
    if (R == 0) return COLI_OK;
    if (!x || !q || !scales) return COLI_ERR_INVALID_ARG;
    if (!ptr_aligned(x, 16) || !ptr_aligned(q, 16) || !ptr_aligned(scales, 16))
        return COLI_ERR_ALIGN;
    const int kb = (K + 127) / 128;
    const dim3 grid((R + kQRows - 1) / kQRows, (kb + kQBlocks - 1) / kQBlocks);
    const cudaError_t err = launch_serialized(
        x_dtype == COLI_OUT_BF16 ? quantize_rows_kernel<true> : quantize_rows_kernel<false>, grid,
        dim3(kQRows * 32), 0, static_cast<cudaStream_t>(stream), R, K, x, q, scales);
    return err == cudaSuccess ? COLI_OK : COLI_ERR_CUDA;
}
