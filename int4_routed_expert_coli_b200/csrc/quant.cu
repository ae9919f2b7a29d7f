// Rows to 8-bit floating point (e4m3), one fp32 scale per row and block of 128:
//   s[b][r] = max(max_k |x[r][k]| / 448, 2^-126),  q = e4m3(x / s)
// 448 is e4m3's largest value; the quotient is rounded to fp32, then to
// nearest even.  The lower bound keeps the division defined for a block of
// zeros (q = 0) and for one whose scale would be subnormal.  A NaN or an
// infinity in a block makes its scale NaN or infinite, so every product of
// that row is NaN: nothing is hidden.
//
// Bound by memory traffic (3 bytes per bf16 value): a warp holds 1024 values
// of a row in registers (one read), and the scales, stored block-major for the
// product that reads them, leave through shared memory in runs of 8 rows.
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

template <bool kBf16>
__global__ void __launch_bounds__(kQRows * 32)
quantize_rows_kernel(int R, int K, const void* __restrict__ x, uint8_t* __restrict__ q,
                     float* __restrict__ scales) {
    __shared__ float sc[kQBlocks][kQRows];
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kb_total = (K + 127) / 128;
    const int64_t r0 = (int64_t)blockIdx.x * kQRows;
    const int b0 = blockIdx.y * kQBlocks;
    const int64_t r = r0 + warp;
    float v[4][8];
    const int k0 = b0 * 128 + lane * 8;  // half a warp per block of 128
    if (r < R) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = k0 + i * 256;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
            if (k < K) {  // K is a multiple of 16: whole vectors
                if constexpr (kBf16) {
                    const uint4 u = __ldg(reinterpret_cast<const uint4*>(
                        static_cast<const uint16_t*>(x) + r * K + k));
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        v[i][2 * j] = __uint_as_float(w[j] << 16);
                        v[i][2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
                    }
                } else {
                    const float4* p =
                        reinterpret_cast<const float4*>(static_cast<const float*>(x) + r * K + k);
                    const float4 a = __ldg(p), b = __ldg(p + 1);
                    v[i][0] = a.x; v[i][1] = a.y; v[i][2] = a.z; v[i][3] = a.w;
                    v[i][4] = b.x; v[i][5] = b.y; v[i][6] = b.z; v[i][7] = b.w;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float m = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max_nan(m, fabsf(v[i][j]));
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float s = max_nan(__fdiv_rn(m, 448.f), 1.17549435e-38f);
            const int k = k0 + i * 256;
            if (k < K) {
                uint32_t w[2];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const __nv_fp8x2_storage_t p = __nv_cvt_float2_to_fp8x2(
                        make_float2(__fdiv_rn(v[i][2 * j], s), __fdiv_rn(v[i][2 * j + 1], s)),
                        __NV_SATFINITE, __NV_E4M3);
                    if (j & 1) w[j >> 1] |= (uint32_t)p << 16;
                    else w[j >> 1] = p;
                }
                *reinterpret_cast<uint2*>(q + r * K + k) = make_uint2(w[0], w[1]);
            }
            if ((lane & 15) == 0) sc[2 * i + (lane >> 4)][warp] = s;
        }
    }
    __syncthreads();
    const int b = threadIdx.x / kQRows, i = threadIdx.x % kQRows;
    if (b < kQBlocks && b0 + b < kb_total && r0 + i < R)
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
