// The norms around a block, fused with the block's gate, the residual scale
// and the residual sum (RMS norms; one pass over the rows):
//
//   n = y rsqrt(mean(y^2) + eps) post_w     (with post_w; otherwise n = y)
//   s = x + alpha g n                       (without a block output y: s = x)
//   o = s rsqrt(mean(s^2) + eps) pre_w      (the next block's input)
//
// g is 1, one value per channel or one per token.  Sums and the whole row are
// fp32; s and o are each rounded once, at their store, and o is computed from
// the unrounded s.
//
// Backward, from the stored s and y (r and ry: the two inverse RMS values,
// recomputed, a row is in hand anyway; A = alpha times a token's gate, cp = post_w
// times a channel's gate):
//   d  = ds + r do pre_w - r^3 mean(do pre_w s) s        dx = d
//   dy = ry A cp d - ry^3 mean(A cp d y) y               (no post_w: dy = A cp d)
//   dpre_w = sum_t do s r
//   C = sum_t gate_token d y ry:  dpost_w = alpha gate_channel C,
//   a channel gate's dgate = alpha post_w C, a token's = alpha ry sum_h cp d y
// so a row needs four sums (s^2, do pre_w s, y^2, cp d y) and a column two.
//
// Both directions move each value once: 8 and 12 bytes a bf16 value.  4096 x 6144
// bf16 with both norms and a channel gate takes 37.5 us forward (5.4 TB/s, 82 % of a
// copy's rate) and 66 us backward (4.6 TB/s; a row's chain of loads, sums and stores
// in few warps is what is left); 64 tokens 3.1 and 9.8 us, which is launches.  Rows
// that are no whole vectors of 8, or wider than 8192, are read one by one with
// nothing ahead of the one that reduces: 6140 wide 48 and 117 us, 6141 84 and 185,
// 8200 75 and 265 (8192: 49 and 88).
#include <algorithm>

#include "coli_internal.cuh"
#include "launch.cuh"
#include "ptx.cuh"

namespace coli {
namespace {

constexpr int kMaxNormH = 16384;

struct NormArgs {
    int T, H;
    const void *x, *y;        // forward: x; backward: unused
    const float *post_w, *gate, *pre_w;
    int gate_kind;
    float alpha, eps;
    int x_bf16, y_bf16, o_bf16;
    void *s_out, *o;
    // backward
    const void *go, *gs, *s;  // gradients of o and s (nullable), the stored s
    void *dx, *dy;
    float *dpre_w, *dpost_w, *dgate;
    float* part;              // [grid][2][H] column partials: dpre_w, C
};

// NCH vectors of VEC values as they lie in memory (whole vectors are aligned).
// The loads stand apart from the conversions: a load whose type's branch also
// converts it is waited for before the next one is issued (4096 x 1001 fp32
// backward 56 us with the conversions inside, 41 us so).
template <int VEC, int NCH>
struct Raw {
    uint32_t u[NCH][VEC];

    // vectors at h(c), of a row's H values at element `row`; zeros past its end
    // and where p is null
    __device__ __forceinline__ void load(const void* p, int64_t row, int bf16, int H) {
#pragma unroll
        for (int c = 0; c < NCH; ++c)
#pragma unroll
            for (int j = 0; j < VEC; ++j) u[c][j] = 0;
        if (!p) return;
        if (bf16) {
            const uint16_t* q = static_cast<const uint16_t*>(p) + row;
#pragma unroll
            for (int c = 0; c < NCH; ++c) {
                const int h = column(c);
                if (h >= H) continue;
                if constexpr (VEC == 8) {
                    const uint4 x = *reinterpret_cast<const uint4*>(q + h);
                    u[c][0] = x.x; u[c][1] = x.y; u[c][2] = x.z; u[c][3] = x.w;
                } else if constexpr (VEC == 4) {
                    const uint2 x = *reinterpret_cast<const uint2*>(q + h);
                    u[c][0] = x.x; u[c][1] = x.y;
                } else {
                    u[c][0] = q[h];
                }
            }
        } else {
            const uint32_t* q = static_cast<const uint32_t*>(p) + row;
#pragma unroll
            for (int c = 0; c < NCH; ++c) {
                const int h = column(c);
                if (h >= H) continue;
                if constexpr (VEC == 1) {
                    u[c][0] = q[h];
                } else {
#pragma unroll
                    for (int j = 0; j < VEC; j += 4) {
                        const uint4 x = *reinterpret_cast<const uint4*>(q + h + j);
                        u[c][j] = x.x; u[c][j + 1] = x.y; u[c][j + 2] = x.z; u[c][j + 3] = x.w;
                    }
                }
            }
        }
    }
    __device__ __forceinline__ void values(int bf16, float (&v)[NCH][VEC]) const {
#pragma unroll
        for (int c = 0; c < NCH; ++c)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const uint32_t w = u[c][j / 2];
                v[c][j] = __uint_as_float(!bf16 ? u[c][j] : j & 1 ? w & 0xFFFF0000u : w << 16);
            }
    }
    // first column of this thread's vector c
    static __device__ __forceinline__ int column(int c) {
        return (c * blockDim.x + threadIdx.x) * VEC;
    }
};

// VEC of the fp32 weights, from column h on.
template <int VEC>
__device__ __forceinline__ void load_w(const float* p, int h, float* w) {
    if constexpr (VEC == 1) {
        w[0] = __ldg(p + h);
    } else {
#pragma unroll
        for (int j = 0; j < VEC; j += 4) {
            const float4 x = __ldg(reinterpret_cast<const float4*>(p + h + j));
            w[j] = x.x; w[j + 1] = x.y; w[j + 2] = x.z; w[j + 3] = x.w;
        }
    }
}

template <int VEC>
__device__ __forceinline__ void store_vals(void* p, int64_t i, int bf16, const float* v) {
    if (bf16) {
        if constexpr (VEC == 1) {
            static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v[0]);
        } else {
            uint32_t w[VEC / 2];
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                w[j] = *reinterpret_cast<const uint32_t*>(&h);
            }
            uint16_t* q = static_cast<uint16_t*>(p) + i;
            if constexpr (VEC == 8) *reinterpret_cast<uint4*>(q) = make_uint4(w[0], w[1], w[2], w[3]);
            else *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
        }
    } else {
        float* q = static_cast<float*>(p) + i;
        if constexpr (VEC == 1) {
            q[0] = v[0];
        } else {
#pragma unroll
            for (int j = 0; j < VEC; j += 4)
                *reinterpret_cast<float4*>(q + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        }
    }
}

// Sums of N values over the block, in a fixed order; every thread gets them.
// `tmp` holds N * 32 floats; calls alternate between two of them.
template <int N>
__device__ __forceinline__ void block_sums(float (&v)[N], float* tmp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) tmp[i * 32 + warp] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float t = lane < nw ? tmp[i * 32 + lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
        v[i] = t;
    }
}

// Block sums of N = 2 or 4 values over at most WARPS warps, in a fixed order.  The
// first levels of the butterfly halve the values a lane carries instead of
// reducing each of them: N - 1 + 5 - log2(N) shuffles a stage and not 5 N.
template <int N, int WARPS>
__device__ __forceinline__ void packed_sums(float (&v)[N], float* tmp) {
    constexpr unsigned kAll = 0xffffffffu;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    float x;
    if constexpr (N == 4) {
        const bool b0 = lane & 1, b1 = lane & 2;
        const float k0 = (b0 ? v[1] : v[0]) + __shfl_xor_sync(kAll, b0 ? v[0] : v[1], 1);
        const float k1 = (b0 ? v[3] : v[2]) + __shfl_xor_sync(kAll, b0 ? v[2] : v[3], 1);
        x = (b1 ? k1 : k0) + __shfl_xor_sync(kAll, b1 ? k0 : k1, 2);
    } else {
        const bool b0 = lane & 1;
        x = (b0 ? v[1] : v[0]) + __shfl_xor_sync(kAll, b0 ? v[0] : v[1], 1);
    }
#pragma unroll
    for (int o = N; o < 32; o <<= 1) x += __shfl_xor_sync(kAll, x, o);
    if (lane < N) tmp[lane * 32 + warp] = x;  // value `lane` of this warp
    __syncthreads();
    // 32 / N lanes to a value, each with its share of the warps
    constexpr int kLanes = 32 / N;
    const int k = lane / kLanes, i = lane % kLanes;
    x = i < nw ? tmp[k * 32 + i] : 0.f;
#pragma unroll
    for (int j = kLanes; j < WARPS; j += kLanes)
        if (i + j < nw) x += tmp[k * 32 + i + j];
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) x += __shfl_xor_sync(kAll, x, o);
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = __shfl_sync(kAll, x, j * kLanes);
}

// One row per CTA, NCH chunks of VEC consecutive values per thread.
template <int VEC, int NCH>
__global__ void __launch_bounds__(VEC * NCH == 32 ? 512 : 1024)
block_norm_kernel(const NormArgs a) {
    __shared__ float tmp[2][32];
    pdl_wait();
    pdl_launch_dependents();
    const int H = a.H;
    const int64_t row = (int64_t)blockIdx.x * H;
    float v[NCH][VEC];
    float s[NCH][VEC];
    {
        Raw<VEC, NCH> ry, rx;
        ry.load(a.y, row, a.y_bf16, H);
        rx.load(a.x, row, a.x_bf16, H);
        ry.values(a.y_bf16, v);
        rx.values(a.x_bf16, s);
    }
    if (a.y) {
        float ry = 1.f;
        if (a.post_w) {
            float q[1] = {0.f};
#pragma unroll
            for (int c = 0; c < NCH; ++c)
#pragma unroll
                for (int j = 0; j < VEC; ++j) q[0] += v[c][j] * v[c][j];
            block_sums<1>(q, tmp[0]);
            ry = rsqrtf(q[0] / (float)H + a.eps);
        }
        const float gt = a.gate_kind == COLI_GATE_TOKEN ? a.alpha * a.gate[blockIdx.x] : a.alpha;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int h = (c * blockDim.x + threadIdx.x) * VEC;
            if (h >= H) continue;
            float w[VEC];
            if (a.post_w) {
                load_w<VEC>(a.post_w, h, w);
#pragma unroll
                for (int j = 0; j < VEC; ++j) v[c][j] *= ry * w[j];
            }
            if (a.gate_kind == COLI_GATE_CHANNEL) {
                load_w<VEC>(a.gate, h, w);
#pragma unroll
                for (int j = 0; j < VEC; ++j) v[c][j] *= w[j];
            }
#pragma unroll
            for (int j = 0; j < VEC; ++j) s[c][j] += gt * v[c][j];
        }
    }
    if (a.s_out) {
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int h = (c * blockDim.x + threadIdx.x) * VEC;
            if (h < H) store_vals<VEC>(a.s_out, row + h, a.x_bf16, s[c]);
        }
    }
    if (!a.o) return;
    float q[1] = {0.f};
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
        for (int j = 0; j < VEC; ++j) q[0] += s[c][j] * s[c][j];
    block_sums<1>(q, tmp[1]);
    const float r = rsqrtf(q[0] / (float)H + a.eps);
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
        const int h = (c * blockDim.x + threadIdx.x) * VEC;
        if (h >= H) continue;
        float w[VEC];
        load_w<VEC>(a.pre_w, h, w);
#pragma unroll
        for (int j = 0; j < VEC; ++j) w[j] *= s[c][j] * r;
        store_vals<VEC>(a.o, row + h, a.o_bf16, w);
    }
}

// A CTA takes rows blockIdx.x, blockIdx.x + gridDim.x, ...; a thread keeps the
// same columns for all of them, so the column sums stay in its registers and
// leave as one partial row per CTA, summed by the next kernel in CTA order.
template <int VEC, int NCH>
__global__ void __launch_bounds__(VEC * NCH == 8 && VEC == 1 ? 768 : 512)
block_norm_bwd_kernel(const NormArgs a) {
    __shared__ float tmp[2][4 * 32];
    pdl_wait();
    pdl_launch_dependents();
    const int H = a.H;
    const float inv_h = 1.f / (float)H;
    float c_pre[NCH][VEC], c_y[NCH][VEC];
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
        for (int j = 0; j < VEC; ++j) c_pre[c][j] = c_y[c][j] = 0.f;

    for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
        const int64_t row = (int64_t)t * H;
        float s[NCH][VEC], y[NCH][VEC], g[NCH][VEC], d[NCH][VEC];
        {
            Raw<VEC, NCH> rg, rs, rd, ry;
            rg.load(a.go, row, a.o_bf16, H);
            rs.load(a.go ? a.s : nullptr, row, a.x_bf16, H);
            rd.load(a.gs, row, a.x_bf16, H);
            ry.load(a.y, row, a.y_bf16, H);
            rg.values(a.o_bf16, g);
            rs.values(a.x_bf16, s);
            rd.values(a.x_bf16, d);
            ry.values(a.y_bf16, y);
        }
        float q[4] = {0.f, 0.f, 0.f, 0.f};  // sum s^2, sum do pre_w s, sum y^2
        if (a.go) {
#pragma unroll
            for (int c = 0; c < NCH; ++c) {
                const int h = (c * blockDim.x + threadIdx.x) * VEC;
                if (h >= H) continue;
                float w[VEC];
                load_w<VEC>(a.pre_w, h, w);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    q[0] += s[c][j] * s[c][j];
                    q[1] += g[c][j] * w[j] * s[c][j];
                }
            }
        }
        if (a.post_w) {
#pragma unroll
            for (int c = 0; c < NCH; ++c)
#pragma unroll
                for (int j = 0; j < VEC; ++j) q[2] += y[c][j] * y[c][j];
        }
        packed_sums<4, 32>(q, tmp[0]);
        const float r = rsqrtf(q[0] * inv_h + a.eps);
        const float ry = a.post_w ? rsqrtf(q[2] * inv_h + a.eps) : 1.f;
        const float rk = r * (r * r * (q[1] * inv_h));
        const float gt = a.gate_kind == COLI_GATE_TOKEN ? a.gate[t] : 1.f;
        const float A = a.alpha * gt, cy = gt * ry;
        float p[1] = {0.f};  // sum cp d y
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int h = (c * blockDim.x + threadIdx.x) * VEC;
            if (h >= H) continue;
            float w[VEC];
            if (a.go) {
                load_w<VEC>(a.pre_w, h, w);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    c_pre[c][j] += (g[c][j] * s[c][j]) * r;
                    d[c][j] += r * (g[c][j] * w[j]) - rk * s[c][j];
                }
            }
            if (a.dx) store_vals<VEC>(a.dx, row + h, a.x_bf16, d[c]);
            if (a.y) {
                float cp[VEC];
#pragma unroll
                for (int j = 0; j < VEC; ++j) cp[j] = 1.f;
                if (a.post_w) load_w<VEC>(a.post_w, h, cp);
                if (a.gate_kind == COLI_GATE_CHANNEL) {
                    load_w<VEC>(a.gate, h, w);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) cp[j] *= w[j];
                }
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    c_y[c][j] += (d[c][j] * y[c][j]) * cy;
                    d[c][j] *= cp[j];
                    p[0] += d[c][j] * y[c][j];
                }
            }
        }
        if (!a.y) {
            __syncthreads();  // tmp[0] is read by all before the next row writes it
            continue;
        }
        block_sums<1>(p, tmp[1]);
        const float c1 = ry * A, c2 = a.post_w ? ry * (ry * ry * (A * p[0] * inv_h)) : 0.f;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int h = (c * blockDim.x + threadIdx.x) * VEC;
            if (h >= H || !a.dy) continue;
#pragma unroll
            for (int j = 0; j < VEC; ++j) d[c][j] = c1 * d[c][j] - c2 * y[c][j];
            store_vals<VEC>(a.dy, row + h, a.y_bf16, d[c]);
        }
        if (a.dgate && a.gate_kind == COLI_GATE_TOKEN && threadIdx.x == 0)
            a.dgate[t] = a.alpha * ry * p[0];
    }
    if (!a.part) return;
    float* part = a.part + (int64_t)blockIdx.x * 2 * H;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
        const int h = (c * blockDim.x + threadIdx.x) * VEC;
        if (h >= H) continue;
        if (a.dpre_w) store_vals<VEC>(part, h, 0, c_pre[c]);
        if (a.y) store_vals<VEC>(part + H, h, 0, c_y[c]);
    }
}

// ---- many rows of whole 16-byte vectors ------------------------------------------
// A CTA walks rows blockIdx.x, + gridDim.x, ... .  Each thread owns kVpt vectors
// of 8 columns and copies them (cp.async) into its own places of a ring in
// shared memory, rows ahead of the one it works on, so that the memory system
// has rows in flight whatever the row reductions wait for; nobody else reads
// those places, so the copies need no barrier.  The weights of a thread's
// columns lie in its registers (up to 384 threads, H 6144) or in shared memory
// (wider rows): read from L2 for every row they would be more bytes than the row
// itself.  The types are template parameters and the loops have no branches (a
// vector past the row's end has places of its own that nothing fills; its sums
// are masked and its stores left out), so that a row's loads and sums interleave.
constexpr int kVpt = 2;                 // vectors per thread
constexpr int kRingMaxThreads = 512;
constexpr int kRingSmem = 222 * 1024;   // dynamic shared memory of a CTA, at most
constexpr int kRegThreads = 384;        // up to these, the weights fit in registers
constexpr int kRegPairThreads = 256;    // and, backward, two CTAs in an SM

// Pairs of fp32 values in one 64-bit register: one instruction for both.  (Issue
// slots bound the same kernels on single values: 52 and 91 us at 4096 x 6144 bf16.)
typedef unsigned long long f2;
__device__ __forceinline__ f2 pair(float lo, float hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unpair(f2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float sum2(f2 v) {
    const float2 f = unpair(v);
    return f.x + f.y;
}

// 8 values as four pairs.
template <bool BF16>
__device__ __forceinline__ void load_pairs(const char* p, f2 (&v)[4]) {
    if constexpr (BF16) {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = pair(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
    } else {
        const ulonglong2 x = reinterpret_cast<const ulonglong2*>(p)[0];
        const ulonglong2 z = reinterpret_cast<const ulonglong2*>(p)[1];
        v[0] = x.x; v[1] = x.y; v[2] = z.x; v[3] = z.y;
    }
}
template <bool BF16>
__device__ __forceinline__ void store_pairs(void* p, int64_t i, const f2 (&v)[4]) {
    if constexpr (BF16) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = unpair(v[j]);
            const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
            w[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
            make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        ulonglong2* q = reinterpret_cast<ulonglong2*>(static_cast<float*>(p) + i);
        q[0] = make_ulonglong2(v[0], v[1]);
        q[1] = make_ulonglong2(v[2], v[3]);
    }
}

struct RingPlan {
    int slots;            // rows in the ring
    const void* src[4];   // copied arrays (null: absent)
    uint32_t at[4];       // byte offset of each in a slot
    uint32_t slot;        // bytes of a slot
    uint32_t weights;     // bytes of the weights before the ring
};

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src)
                 : "memory");
}
// At most `n` of this thread's latest groups in flight (n <= 6).
__device__ __forceinline__ void cp_async_wait_n(int n) {
    switch (n) {
        case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
        case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
        case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
        case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
        case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
        case 5: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
        default: asm volatile("cp.async.wait_group 6;" ::: "memory"); break;
    }
}

// One thread's view of the ring.
struct RowRing {
    const RingPlan& p;
    char* base;
    int H, T;

    // column of vector c, and whether the row has it
    static __device__ __forceinline__ int col(int c) {
        return (c * blockDim.x + threadIdx.x) * 8;
    }
    __device__ __forceinline__ bool live(int c) const { return col(c) < H; }

    template <bool BF16>
    __device__ __forceinline__ void copy(int k, int64_t t, char* slot) const {
        constexpr int kSize = BF16 ? 2 : 4;
        if (!p.src[k]) return;
        const char* g = static_cast<const char*>(p.src[k]) + t * H * kSize;
#pragma unroll
        for (int c = 0; c < kVpt; ++c) {
            if (!live(c)) continue;
            cp_async16(slot + p.at[k] + col(c) * kSize, g + col(c) * kSize);
            if (!BF16) cp_async16(slot + p.at[k] + col(c) * kSize + 16, g + col(c) * kSize + 16);
        }
    }
    // This thread's copies of row t into slot i, one group (empty past the end).
    template <bool B0, bool B1, bool B2, bool B3>
    __device__ __forceinline__ void fetch(int64_t t, int i) const {
        if (t < T) {
            char* slot = base + (size_t)i * p.slot;
            copy<B0>(0, t, slot);
            copy<B1>(1, t, slot);
            copy<B2>(2, t, slot);
            copy<B3>(3, t, slot);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    template <bool BF16>
    __device__ __forceinline__ void load(int k, int i, int c, f2 (&v)[4]) const {
        load_pairs<BF16>(base + (size_t)i * p.slot + p.at[k] + col(c) * (BF16 ? 2 : 4), v);
    }
};

// The weights into shared memory: pre_w, and post_w times a channel's gate
// (ones where there is none), each [2][H / 2]: a vector's first four values in
// the first plane, the others in the second (a warp's 16-byte reads then fall
// on consecutive addresses).
__device__ __forceinline__ void stage_weights(float* w_pre, float* w_cp, const NormArgs& a) {
    const int H = a.H;
    for (int h = threadIdx.x * 4; h < H; h += blockDim.x * 4) {
        float4 v = make_float4(1.f, 1.f, 1.f, 1.f);
        const int at = (h & 4 ? H / 2 : 0) + h / 8 * 4;
        if (a.pre_w) v = __ldg(reinterpret_cast<const float4*>(a.pre_w + h));
        *reinterpret_cast<float4*>(w_pre + at) = v;
        v = make_float4(1.f, 1.f, 1.f, 1.f);
        if (a.post_w) v = __ldg(reinterpret_cast<const float4*>(a.post_w + h));
        if (a.gate_kind == COLI_GATE_CHANNEL) {
            const float4 g = __ldg(reinterpret_cast<const float4*>(a.gate + h));
            v.x *= g.x; v.y *= g.y; v.z *= g.z; v.w *= g.w;
        }
        *reinterpret_cast<float4*>(w_cp + at) = v;
    }
    __syncthreads();
}
__device__ __forceinline__ void load_weights(const float* w, int H, int col, f2 (&v)[4]) {
    const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(w + col / 2);
    const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(w + H / 2 + col / 2);
    v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
}

// A thread's weights (pre_w, and post_w times a channel's gate), in registers or
// in shared memory.
template <bool REG>
struct Weights {
    f2 v[REG ? 2 : 1][REG ? kVpt : 1][4];
    const float* at;
    int H;

    __device__ __forceinline__ Weights(const NormArgs& a, char* smem)
        : at(reinterpret_cast<const float*>(smem)), H(a.H) {
        if constexpr (REG) {
#pragma unroll
            for (int c = 0; c < kVpt; ++c) {
                const int h = min(RowRing::col(c), a.H - 8);
                float w[8], g[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = 1.f;
                if (a.pre_w) load_w<8>(a.pre_w, h, w);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[0][c][j] = pair(w[2 * j], w[2 * j + 1]);
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = 1.f;
                if (a.post_w) load_w<8>(a.post_w, h, w);
                if (a.gate_kind == COLI_GATE_CHANNEL) {
                    load_w<8>(a.gate, h, g);
#pragma unroll
                    for (int j = 0; j < 8; ++j) w[j] *= g[j];
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) v[1][c][j] = pair(w[2 * j], w[2 * j + 1]);
            }
        } else {
            stage_weights(reinterpret_cast<float*>(smem), reinterpret_cast<float*>(smem) + H, a);
        }
    }
    // k 0: pre_w, 1: post_w times the gate
    __device__ __forceinline__ void load(int k, int c, f2 (&w)[4]) const {
        if constexpr (REG) {
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = v[k][c][j];
        } else {
            load_weights(at + k * H, H, min(RowRing::col(c), H - 8), w);
        }
    }
};

template <bool REG, bool XB, bool YB, bool OB>
__global__ void __launch_bounds__(REG ? kRegThreads : kRingMaxThreads)
block_norm_ring_kernel(const __grid_constant__ NormArgs a, const __grid_constant__ RingPlan p) {
    extern __shared__ __align__(128) char smem[];
    __shared__ float tmp[2][2 * 32];
    const int H = a.H;
    const RowRing ring{p, smem + p.weights, H, a.T};
    const float inv_h = 1.f / (float)H;
    pdl_wait();
    pdl_launch_dependents();
    for (int i = 0; i < p.slots; ++i)
        ring.fetch<XB, YB, false, false>(blockIdx.x + (int64_t)i * gridDim.x, i);
    const Weights<REG> weights(a, smem);
    // this thread's share of the sum of y^2 of the row in slot i
    auto sum_y = [&](int i) {
        float q = 0.f;
#pragma unroll
        for (int c = 0; c < kVpt; ++c) {
            f2 y[4], z = 0;
            ring.load<YB>(1, i, c, y);
#pragma unroll
            for (int j = 0; j < 4; ++j) z = fma2(y[j], y[j], z);
            q += ring.live(c) ? sum2(z) : 0.f;
        }
        return q;
    };
    // One round of block sums a row: the y^2 of the next row joins the s^2 of
    // this one.
    float q[2] = {0.f, 0.f};
    if (a.post_w) {
        cp_async_wait_n(p.slots - 1);
        q[1] = sum_y(0);
        packed_sums<2, 16>(q, tmp[1]);
    }
    int slot = 0, odd = 0;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        cp_async_wait_n(p.slots - 2);  // this row and the next one are in the ring
        const int64_t row = t * H;
        const int after = slot + 1 == p.slots ? 0 : slot + 1;
        f2 s[kVpt][4];
#pragma unroll
        for (int c = 0; c < kVpt; ++c) ring.load<XB>(0, slot, c, s[c]);
        if (a.y) {
            float A = a.alpha;
            if (a.gate_kind == COLI_GATE_TOKEN) A *= __ldg(a.gate + t);
            if (a.post_w) A *= rsqrtf(q[1] * inv_h + a.eps);
            const f2 A2 = pair(A, A);
#pragma unroll
            for (int c = 0; c < kVpt; ++c) {
                f2 y[4], w[4];
                ring.load<YB>(1, slot, c, y);
                weights.load(1, c, w);
#pragma unroll
                for (int j = 0; j < 4; ++j) s[c][j] = fma2(A2, mul2(y[j], w[j]), s[c][j]);
            }
        }
        q[0] = 0.f;
#pragma unroll
        for (int c = 0; c < kVpt; ++c) {
            f2 z = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) z = fma2(s[c][j], s[c][j], z);
            q[0] += ring.live(c) ? sum2(z) : 0.f;
            if (a.s_out && ring.live(c)) store_pairs<XB>(a.s_out, row + ring.col(c), s[c]);
        }
        q[1] = a.post_w ? sum_y(after) : 0.f;
        // the slot is read: fetch the row that takes its place
        ring.fetch<XB, YB, false, false>(t + (int64_t)p.slots * gridDim.x, slot);
        if (a.o || a.post_w) packed_sums<2, 16>(q, tmp[odd]);
        if (a.o) {
            const float r = rsqrtf(q[0] * inv_h + a.eps);
            const f2 r2 = pair(r, r);
#pragma unroll
            for (int c = 0; c < kVpt; ++c) {
                f2 w[4];
                weights.load(0, c, w);
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = mul2(mul2(s[c][j], r2), w[j]);
                if (ring.live(c)) store_pairs<OB>(a.o, row + ring.col(c), w);
            }
        }
        slot = after;
        odd ^= 1;
    }
}

// THREADS: the most it is launched with.  Two CTAs of 256 threads fit an SM with 128
// registers each (4096 x 4096 bf16: 47 us, one CTA of 138 registers 58), one of 384
// is better off with all it can use (4096 x 6144: 66 us, with 128 registers 73).
template <int THREADS, bool XB, bool YB, bool OB>
__global__ void __launch_bounds__(THREADS, THREADS <= kRegPairThreads ? 2 : 1)
block_norm_bwd_ring_kernel(const __grid_constant__ NormArgs a,
                           const __grid_constant__ RingPlan p) {
    extern __shared__ __align__(128) char smem[];
    __shared__ float tmp[2][4 * 32];
    constexpr bool REG = THREADS <= kRegThreads;
    const int H = a.H;
    const RowRing ring{p, smem + p.weights, H, a.T};
    const float inv_h = 1.f / (float)H;
    constexpr int kGo = 0, kS = 1, kGs = 2, kY = 3;
    pdl_wait();
    pdl_launch_dependents();
    for (int i = 0; i < p.slots; ++i)
        ring.fetch<OB, XB, XB, YB>(blockIdx.x + (int64_t)i * gridDim.x, i);
    const Weights<REG> weights(a, smem);
    f2 c_pre[kVpt][4], c_y[kVpt][4];
#pragma unroll
    for (int c = 0; c < kVpt; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j) c_pre[c][j] = c_y[c][j] = 0;
    // This thread's shares of the first three sums of the row in slot i: s^2,
    // do pre_w s, y^2.
    auto first_sums = [&](int i, float (&q)[4]) {
        q[0] = q[1] = q[2] = 0.f;
#pragma unroll
        for (int c = 0; c < kVpt; ++c) {
            f2 z0 = 0, z1 = 0, z2 = 0;
            if (a.go) {
                f2 s[4], g[4], w[4];
                ring.load<OB>(kGo, i, c, g);
                ring.load<XB>(kS, i, c, s);
                weights.load(0, c, w);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    z0 = fma2(s[j], s[j], z0);
                    z1 = fma2(mul2(g[j], s[j]), w[j], z1);
                }
            }
            if (a.post_w) {
                f2 y[4];
                ring.load<YB>(kY, i, c, y);
#pragma unroll
                for (int j = 0; j < 4; ++j) z2 = fma2(y[j], y[j], z2);
            }
            if (ring.live(c)) {
                q[0] += sum2(z0);
                q[1] += sum2(z1);
                q[2] += sum2(z2);
            }
        }
    };
    // One round of block sums a row: the next row's first three join this row's
    // last.
    float q[4];
    cp_async_wait_n(p.slots - 1);
    first_sums(0, q);
    q[3] = 0.f;
    packed_sums<4, 16>(q, tmp[1]);
    int slot = 0, odd = 0;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const int64_t row = t * H;
        const int after = slot + 1 == p.slots ? 0 : slot + 1;
        float gt = 1.f;
        if (a.gate_kind == COLI_GATE_TOKEN) gt = __ldg(a.gate + t);
        const float r = rsqrtf(q[0] * inv_h + a.eps);
        const float ry = a.post_w ? rsqrtf(q[2] * inv_h + a.eps) : 1.f;
        const float rk = -r * (r * r * (q[1] * inv_h));
        const float A = a.alpha * gt, cy = gt * ry;
        const f2 r2 = pair(r, r), rk2 = pair(rk, rk), cy2 = pair(cy, cy);
        f2 e[kVpt][4];            // cp d
        q[3] = 0.f;               // sum cp d y
#pragma unroll
        for (int c = 0; c < kVpt; ++c) {
            f2 d[4] = {0, 0, 0, 0};
            if (a.gs) ring.load<XB>(kGs, slot, c, d);
            if (a.go) {
                f2 s[4], g[4], w[4];
                ring.load<OB>(kGo, slot, c, g);
                ring.load<XB>(kS, slot, c, s);
                weights.load(0, c, w);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    c_pre[c][j] = fma2(mul2(g[j], s[j]), r2, c_pre[c][j]);
                    d[j] = fma2(mul2(g[j], w[j]), r2, d[j]);
                    d[j] = fma2(s[j], rk2, d[j]);
                }
            }
            if (a.dx && ring.live(c)) store_pairs<XB>(a.dx, row + ring.col(c), d);
            if (a.y) {
                f2 y[4], w[4], z = 0;
                ring.load<YB>(kY, slot, c, y);
                weights.load(1, c, w);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    c_y[c][j] = fma2(mul2(d[j], y[j]), cy2, c_y[c][j]);
                    e[c][j] = mul2(d[j], w[j]);
                    z = fma2(e[c][j], y[j], z);
                }
                q[3] += ring.live(c) ? sum2(z) : 0.f;
            }
        }
        cp_async_wait_n(p.slots - 2);  // the next row is in the ring
        first_sums(after, q);
        packed_sums<4, 16>(q, tmp[odd]);
        if (a.y) {
            const float c1 = ry * A;
            const float c2 = a.post_w ? -ry * (ry * ry * (A * q[3] * inv_h)) : 0.f;
            const f2 c12 = pair(c1, c1), c22 = pair(c2, c2);
            if (a.dy) {
#pragma unroll
                for (int c = 0; c < kVpt; ++c) {
                    f2 y[4];
                    ring.load<YB>(kY, slot, c, y);
#pragma unroll
                    for (int j = 0; j < 4; ++j) y[j] = fma2(c12, e[c][j], mul2(c22, y[j]));
                    if (ring.live(c)) store_pairs<YB>(a.dy, row + ring.col(c), y);
                }
            }
            if (a.dgate && a.gate_kind == COLI_GATE_TOKEN && threadIdx.x == 0)
                a.dgate[t] = a.alpha * ry * q[3];
        }
        ring.fetch<OB, XB, XB, YB>(t + (int64_t)p.slots * gridDim.x, slot);
        slot = after;
        odd ^= 1;
    }
    if (!a.part) return;
    float* part = a.part + (int64_t)blockIdx.x * 2 * H;
#pragma unroll
    for (int c = 0; c < kVpt; ++c) {
        if (!ring.live(c)) continue;
        if (a.dpre_w) store_pairs<false>(part, ring.col(c), c_pre[c]);
        if (a.y) store_pairs<false>(part + H, ring.col(c), c_y[c]);
    }
}

// Column sums over the CTAs' partial rows, 32 columns per block, 16 warps over
// the CTAs; fixed order (each warp its strided share ascending, then the warps
// ascending).  A warp has kColBatch loads in flight (of the last row again where
// there are no more): one round of L2 latency for 160 partial rows.  blockIdx.y
// 0: dpre_w, 1: C, from which dpost_w and a channel gate's dgate follow.
constexpr int kColBatch = 10, kColWarps = 16;

__global__ void __launch_bounds__(kColWarps * 32)
norm_columns_kernel(const NormArgs a, int n_part) {
    __shared__ float acc[kColWarps][32];
    pdl_wait();
    pdl_launch_dependents();
    const bool channel = a.gate_kind == COLI_GATE_CHANNEL;
    float* dgate = channel ? a.dgate : nullptr;
    if (blockIdx.y == 0 ? !a.dpre_w : !(a.dpost_w || dgate)) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int h = blockIdx.x * 32 + lane;
    float v = 0.f;
    if (h < a.H) {
        const float* p = a.part + (int64_t)blockIdx.y * a.H + h;
        for (int i0 = warp; i0 < n_part; i0 += kColWarps * kColBatch) {
            float f[kColBatch];
#pragma unroll
            for (int j = 0; j < kColBatch; ++j)
                f[j] = p[(int64_t)min(i0 + kColWarps * j, n_part - 1) * 2 * a.H];
#pragma unroll
            for (int j = 0; j < kColBatch; ++j) v += i0 + kColWarps * j < n_part ? f[j] : 0.f;
        }
    }
    acc[warp][lane] = v;
    __syncthreads();
    if (warp != 0 || h >= a.H) return;
#pragma unroll
    for (int w = 1; w < kColWarps; ++w) v += acc[w][lane];
    if (blockIdx.y == 0) {
        a.dpre_w[h] = v;
    } else {
        v *= a.alpha;
        if (a.dpost_w) a.dpost_w[h] = channel ? v * a.gate[h] : v;
        if (dgate) dgate[h] = a.post_w ? v * a.post_w[h] : v;
    }
}

// ---- host ---------------------------------------------------------------------

coli_status check_norm(int32_t T, int32_t H, int32_t gate_kind, const void* gate, const void* y,
                       const void* post_w, float eps) {
    if (T < 0 || H <= 0) return COLI_ERR_INVALID_ARG;
    if (gate_kind != COLI_GATE_NONE && gate_kind != COLI_GATE_CHANNEL &&
        gate_kind != COLI_GATE_TOKEN)
        return COLI_ERR_INVALID_ARG;
    if (!(eps >= 0.f)) return COLI_ERR_INVALID_ARG;
    if (H > kMaxNormH || T > 1 << 24) return COLI_ERR_SHAPE;
    if (T == 0) return COLI_OK;  // tensors of no tokens have no address
    if ((gate != nullptr) != (gate_kind != COLI_GATE_NONE)) return COLI_ERR_INVALID_ARG;
    if (!y && (post_w || gate)) return COLI_ERR_INVALID_ARG;
    return COLI_OK;
}

// CTAs of the backward kernels, at most (each leaves one partial row per column
// sum in the workspace).  Narrow rows take more: 768, which keeps the workspace
// within 1536 rows of H floats.  888 are 0.8 us faster where they make five rows a
// CTA of six (4096 rows: 256 bf16 16.1 and 16.9, 500 fp32 17.1 and 18.0), 0.9 slower where
// 768 do as many (1200 x 256 fp32 11.1 and 10.2, 2000 x 33 12.7 and 11.8).
constexpr int kBwdNarrowH = 512, kBwdNarrowCtas = 768, kBwdCtas = 3 * 148;
int norm_bwd_ctas(int T, int H) {
    return std::max(1, std::min(T, H <= kBwdNarrowH ? kBwdNarrowCtas : kBwdCtas));
}

// Bytes that a call's partial rows take, behind the workspace's header.
size_t norm_bwd_bytes(int T, int H) {
    return sizeof(float) * 2 * (size_t)H * (size_t)norm_bwd_ctas(T, H);
}

// Where the ring kernels pay: enough values that the rows gain more than the
// ring's start costs.  bf16, ring against one row a CTA, forward: 450 rows of 2048
// 3.9 and 3.2 us, 900 of them 4.9 and 5.2; 300 of 4096 4.4 and 5.2, 200 of them 4.0
// and 3.3; 4096 rows of 768 10.4 and 7.0.  Backward: 300 rows of 768 7.7 and 6.6,
// 600 of them 8.7 and 9.1; 200 of 2048 7.7 and 10.3; 4096 of 6144 66 and 113.
constexpr int kRingMinH = 512, kRingFwdMinH = 1536;
constexpr int64_t kRingFwdValues = 1 << 20, kRingBwdValues = 400000;

// The ring kernels' launch for these arrays: threads, CTAs per SM and ring depth,
// or false where the row is too wide, not of whole vectors, or the values too few.
bool plan_ring(bool backward, const NormArgs& a, const void* const (&src)[4],
               const int (&bf16)[4], RingPlan* p, int* threads, int* grid, int* smem) {
    if (a.H % 8 || a.H < (backward ? kRingMinH : kRingFwdMinH) ||
        a.H > 8 * kVpt * kRingMaxThreads ||
        (int64_t)a.T * a.H < (backward ? kRingBwdValues : kRingFwdValues))
        return false;
    *threads = ((a.H + 8 * kVpt - 1) / (8 * kVpt) + 31) / 32 * 32;
    *p = RingPlan{};
    uint32_t slot = 0;
    for (int k = 0; k < 4; ++k) {
        if (!src[k]) continue;
        p->src[k] = src[k];
        p->at[k] = slot;
        slot += (uint32_t)(*threads * 8 * kVpt) * (bf16[k] ? 2 : 4);
    }
    p->slot = (slot + 127) / 128 * 128;
    p->weights =
        *threads <= kRegThreads ? 0 : (uint32_t)(2 * sizeof(float) * a.H + 127) / 128 * 128;
    // threads that the register file holds: 74 registers each, 128 backward
    const int resident = backward ? 512 : 768;
    for (int per_sm = std::max(1, std::min(3, resident / *threads)); per_sm >= 1; --per_sm) {
        const int room = (kRingSmem + 2048) / per_sm - 2048;
        const int slots = std::min(7, (room - (int)p->weights) / (int)p->slot);
        // two rows in hand, one on its way; one CTA of very wide rows does with two
        if (slots < (per_sm == 1 ? 2 : 3)) continue;
        p->slots = slots;
        *grid = 148 * per_sm;
        *smem = (int)(p->weights + slots * p->slot);
        // (backward, each CTA has partial sums to leave: 450 rows of 2048 take 10.3
        // us with 148 CTAs, 10.7 with 444; 900 of them 13.9 with 296, 12.9 with 444)
        if (a.T >= *grid * (backward && per_sm > 1 ? 2 : 1)) return true;
    }
    return false;
}

template <int THREADS, bool XB, bool YB, bool OB>
cudaError_t launch_ring(bool backward, const NormArgs& a, const RingPlan& p, int threads, int grid,
                        int smem, cudaStream_t st) {
    auto kernel = backward ? block_norm_bwd_ring_kernel<THREADS, XB, YB, OB>
                           : block_norm_ring_kernel<THREADS <= kRegThreads, XB, YB, OB>;
    // (always the same limit: host threads cannot lower it under each other)
    const cudaError_t err =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingSmem);
    if (err != cudaSuccess) return err;
    return launch_serialized(kernel, dim3(grid), dim3(threads), smem, st, a, p);
}

template <int THREADS>
cudaError_t dispatch_types(bool backward, const NormArgs& a, const RingPlan& p, int threads,
                           int grid, int smem, cudaStream_t st) {
    using Fn = cudaError_t (*)(bool, const NormArgs&, const RingPlan&, int, int, int, cudaStream_t);
    static const Fn fn[2][2][2] = {
        {{launch_ring<THREADS, false, false, false>, launch_ring<THREADS, false, false, true>},
         {launch_ring<THREADS, false, true, false>, launch_ring<THREADS, false, true, true>}},
        {{launch_ring<THREADS, true, false, false>, launch_ring<THREADS, true, false, true>},
         {launch_ring<THREADS, true, true, false>, launch_ring<THREADS, true, true, true>}}};
    return fn[a.x_bf16 != 0][a.y_bf16 != 0][a.o_bf16 != 0](backward, a, p, threads, grid, smem, st);
}

cudaError_t dispatch_ring(bool backward, const NormArgs& a, const RingPlan& p, int threads, int grid,
                          int smem, cudaStream_t st) {
    if (threads <= kRegPairThreads)
        return dispatch_types<kRegPairThreads>(backward, a, p, threads, grid, smem, st);
    if (threads <= kRegThreads)
        return dispatch_types<kRegThreads>(backward, a, p, threads, grid, smem, st);
    return dispatch_types<kRingMaxThreads>(backward, a, p, threads, grid, smem, st);
}

// Vectors and threads: 16-byte accesses where all rows start on 16 bytes whatever
// their type, 16 or 8 bytes where H is a multiple of 4, else one value at a time.
// Wider rows take more values a thread, up to what the registers hold (fp32, 4096
// rows, forward and backward: 2001 values by 8 a thread 24.8 and 59.5 us, by 4 28.5
// and 83.9; 1001 by 8 13.9 and 49.8, by 4 14.8 and 41.1; 2004 in 4 vectors a thread
// 21.1 and 43.9, in 2 19.9 and 60.4).  With 32 values a thread, backward, six arrays
// of them do not fit 128 registers: about 1 KB a thread spills (4096 x 16384 bf16
// forward 158 us, backward 427).
template <template <int, int> class Launch>
cudaError_t dispatch_width(int H, int max_threads, const NormArgs& a, int grid, cudaStream_t st) {
    auto threads = [&](int vec, int nch) { return ((H + vec * nch - 1) / (vec * nch) + 31) / 32 * 32; };
    if (H % 8 == 0) {
        if (threads(8, 1) <= max_threads) return Launch<8, 1>::run(a, grid, threads(8, 1), st);
        if (threads(8, 2) <= max_threads) return Launch<8, 2>::run(a, grid, threads(8, 2), st);
        return Launch<8, 4>::run(a, grid, threads(8, 4), st);
    }
    if (H % 4 == 0) {
        if (H <= 1024) return Launch<4, 2>::run(a, grid, threads(4, 2), st);
        if (threads(4, 4) <= 512) return Launch<4, 4>::run(a, grid, threads(4, 4), st);
        return Launch<4, 8>::run(a, grid, threads(4, 8), st);
    }
    if (H <= 1024) return Launch<1, 4>::run(a, grid, threads(1, 4), st);
    if (threads(1, 8) <= 768) return Launch<1, 8>::run(a, grid, threads(1, 8), st);
    return Launch<1, 32>::run(a, grid, threads(1, 32), st);
}

template <int VEC, int NCH>
struct Forward {
    static cudaError_t run(const NormArgs& a, int grid, int threads, cudaStream_t st) {
        return launch_serialized(block_norm_kernel<VEC, NCH>, dim3(grid), dim3(threads), 0, st, a);
    }
};
template <int VEC, int NCH>
struct Backward {
    static cudaError_t run(const NormArgs& a, int grid, int threads, cudaStream_t st) {
        return launch_serialized(block_norm_bwd_kernel<VEC, NCH>, dim3(grid), dim3(threads), 0, st,
                                 a);
    }
};

}  // namespace
}  // namespace coli

using namespace coli;

extern "C" {

coli_status coli_moe_block_norm(int32_t T, int32_t H, const void* x, coli_out_dtype x_dtype,
                                const void* y, coli_out_dtype y_dtype, const float* post_w,
                                const float* gate, int32_t gate_kind, float alpha,
                                const float* pre_w, float eps, void* s_out, void* o,
                                coli_out_dtype o_dtype, void* stream) {
    coli_status s = check_norm(T, H, gate_kind, gate, y, post_w, eps);
    if (s != COLI_OK) return s;
    if (!valid_dtype(x_dtype) || !valid_dtype(y_dtype) || !valid_dtype(o_dtype))
        return COLI_ERR_INVALID_ARG;
    if (T == 0) return COLI_OK;
    if ((!s_out && !o) || (o && !pre_w)) return COLI_ERR_INVALID_ARG;
    if (!x) return COLI_ERR_INVALID_ARG;
    const void* ptrs[7] = {x, y, post_w, gate, pre_w, s_out, o};
    for (const void* p : ptrs)
        if (!ptr_aligned(p, 16)) return COLI_ERR_ALIGN;
    NormArgs a = {};
    a.T = T; a.H = H; a.x = x; a.y = y; a.post_w = post_w; a.gate = gate; a.pre_w = pre_w;
    a.gate_kind = gate_kind; a.alpha = alpha; a.eps = eps;
    a.x_bf16 = x_dtype == COLI_OUT_BF16;
    a.y_bf16 = y_dtype == COLI_OUT_BF16;
    a.o_bf16 = o_dtype == COLI_OUT_BF16;
    a.s_out = s_out; a.o = o;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const void* const src[4] = {x, y, nullptr, nullptr};
    const int bf16[4] = {a.x_bf16, a.y_bf16, 0, 0};
    RingPlan p;
    int threads, grid, smem;
    cudaError_t err;
    if (plan_ring(false, a, src, bf16, &p, &threads, &grid, &smem))
        err = dispatch_ring(false, a, p, threads, grid, smem, st);
    else
        err = dispatch_width<Forward>(H, T <= 148 ? 1024 : 512, a, T, st);
    return err == cudaSuccess ? COLI_OK : COLI_ERR_CUDA;
}

size_t coli_moe_block_norm_workspace_size(int32_t T, int32_t H) {
    if (T < 0 || H <= 0) return 0;
    // never less than a narrower call's, whose rows have more CTAs: a workspace
    // of some T and H serves every call with no more of either
    return kHeaderBytes +
           std::max(norm_bwd_bytes(T, H), norm_bwd_bytes(T, std::min(H, kBwdNarrowH)));
}

coli_status coli_moe_block_norm_backward(
    int32_t T, int32_t H, const void* go, coli_out_dtype o_dtype, const void* gs, const void* s_in,
    coli_out_dtype x_dtype, const void* y, coli_out_dtype y_dtype, const float* post_w,
    const float* gate, int32_t gate_kind, float alpha, const float* pre_w, float eps, void* dx,
    void* dy, float* dpre_w, float* dpost_w, float* dgate, void* ws, size_t ws_bytes,
    void* stream) {
    coli_status s = check_norm(T, H, gate_kind, gate, y, post_w, eps);
    if (s != COLI_OK) return s;
    if (!valid_dtype(x_dtype) || !valid_dtype(y_dtype) || !valid_dtype(o_dtype))
        return COLI_ERR_INVALID_ARG;
    // no gradient of something the call does not have
    if (T > 0 && ((dpre_w && !go) || (dpost_w && !post_w) || (dgate && !gate) || (dy && !y)))
        return COLI_ERR_INVALID_ARG;
    const void* ptrs[12] = {go, gs, s_in, y, post_w, gate, pre_w, dx, dy, dpre_w, dpost_w, dgate};
    for (const void* p : ptrs)
        if (!ptr_aligned(p, 16)) return COLI_ERR_ALIGN;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) {  // sums over no tokens
        cudaError_t err = cudaSuccess;
        float* col[3] = {dpre_w, dpost_w, gate_kind == COLI_GATE_CHANNEL ? dgate : nullptr};
        for (float* p : col)
            if (p && err == cudaSuccess) err = cudaMemsetAsync(p, 0, sizeof(float) * H, st);
        return err == cudaSuccess ? COLI_OK : COLI_ERR_CUDA;
    }
    if (!go && !gs) return COLI_ERR_INVALID_ARG;
    if (go && (!s_in || !pre_w)) return COLI_ERR_INVALID_ARG;
    const bool columns = dpre_w || dpost_w || (dgate && gate_kind == COLI_GATE_CHANNEL);
    if (columns) {
        if (!ws) return COLI_ERR_INVALID_ARG;
        if (!ptr_aligned(ws, 256)) return COLI_ERR_ALIGN;
        if (ws_bytes < kHeaderBytes + norm_bwd_bytes(T, H)) return COLI_ERR_WORKSPACE;
    }
    NormArgs a = {};
    a.T = T; a.H = H; a.y = y; a.post_w = post_w; a.gate = gate; a.pre_w = pre_w;
    a.gate_kind = gate_kind; a.alpha = alpha; a.eps = eps;
    a.x_bf16 = x_dtype == COLI_OUT_BF16;
    a.y_bf16 = y_dtype == COLI_OUT_BF16;
    a.o_bf16 = o_dtype == COLI_OUT_BF16;
    a.go = go; a.gs = gs; a.s = s_in; a.dx = dx; a.dy = dy;
    a.dpre_w = dpre_w; a.dpost_w = dpost_w; a.dgate = dgate;
    a.part = columns ? reinterpret_cast<float*>(static_cast<char*>(ws) + kHeaderBytes) : nullptr;
    const void* const src[4] = {go, go ? s_in : nullptr, gs, y};
    const int bf16[4] = {a.o_bf16, a.x_bf16, a.x_bf16, a.y_bf16};
    RingPlan p;
    int threads, smem, grid;
    cudaError_t err;
    if (plan_ring(true, a, src, bf16, &p, &threads, &grid, &smem)) {
        err = dispatch_ring(true, a, p, threads, grid, smem, st);
    } else {
        grid = norm_bwd_ctas(T, H);
        err = dispatch_width<Backward>(H, 512, a, grid, st);
    }
    if (err == cudaSuccess && columns)
        err = launch_serialized(norm_columns_kernel, dim3((H + 31) / 32, 2), dim3(kColWarps * 32), 0,
                                st, a, grid);
    return err == cudaSuccess ? COLI_OK : COLI_ERR_CUDA;
}

}  // extern "C"
