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
// Backward, from the stored s and y (a = do pre_w, r and ry the two inverse
// RMS values, recomputed: a row is in hand anyway, so nothing is saved for it):
//   ds' = ds + r (a - s r^2 mean(a s))      dx = ds'
//   dpre_w = sum_t do s r
//   dgate = alpha sum (ds' n) over the tokens (channel) or channels (token)
//   dn = alpha g ds',  b = dn post_w
//   dpost_w = sum_t dn y ry,  dy = ry (b - y ry^2 mean(b y))   (no post_w: dy = dn)
//
// Both directions move each value once and are bound by memory traffic.
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
    float* part;              // [grid][3][H] column partials: pre_w, post_w, gate
};

// VEC consecutive values starting at element i (16-byte aligned for VEC = 8).
template <int VEC>
__device__ __forceinline__ void load_vals(const void* p, int64_t i, int bf16, float* v) {
    if constexpr (VEC == 8) {
        if (bf16) {
            const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[2 * j] = __uint_as_float(w[j] << 16);
                v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
            }
        } else {
            const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
            const float4 a = q[0], b = q[1];
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        }
    } else {
        v[0] = bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16)
                    : static_cast<const float*>(p)[i];
    }
}

template <int VEC>
__device__ __forceinline__ void store_vals(void* p, int64_t i, int bf16, const float* v) {
    if constexpr (VEC == 8) {
        if (bf16) {
            uint4 u;
            uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                w[j] = *reinterpret_cast<const uint32_t*>(&h);
            }
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = u;
        } else {
            float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
            q[0] = make_float4(v[0], v[1], v[2], v[3]);
            q[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
    } else {
        if (bf16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v[0]);
        else static_cast<float*>(p)[i] = v[0];
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
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
        const int h = (c * blockDim.x + threadIdx.x) * VEC;
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[c][j] = s[c][j] = 0.f;
        if (h < H) {
            if (a.y) load_vals<VEC>(a.y, row + h, a.y_bf16, v[c]);
            load_vals<VEC>(a.x, row + h, a.x_bf16, s[c]);
        }
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
                load_vals<VEC>(a.post_w, h, 0, w);
#pragma unroll
                for (int j = 0; j < VEC; ++j) v[c][j] *= ry * w[j];
            }
            if (a.gate_kind == COLI_GATE_CHANNEL) {
                load_vals<VEC>(a.gate, h, 0, w);
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
        load_vals<VEC>(a.pre_w, h, 0, w);
#pragma unroll
        for (int j = 0; j < VEC; ++j) w[j] *= s[c][j] * r;
        store_vals<VEC>(a.o, row + h, a.o_bf16, w);
    }
}

// A CTA takes rows blockIdx.x, blockIdx.x + gridDim.x, ...; a thread keeps the
// same columns for all of them, so the column sums stay in its registers and
// leave as one partial row per CTA, summed by the next kernel in CTA order.
template <int VEC, int NCH>
__global__ void __launch_bounds__(512)
block_norm_bwd_kernel(const NormArgs a) {
    __shared__ float tmp[2][3 * 32];
    pdl_wait();
    pdl_launch_dependents();
    const int H = a.H;
    float c_pre[NCH][VEC], c_post[NCH][VEC], c_gate[NCH][VEC];
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
        for (int j = 0; j < VEC; ++j) c_pre[c][j] = c_post[c][j] = c_gate[c][j] = 0.f;

    for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
        const int64_t row = (int64_t)t * H;
        float s[NCH][VEC], y[NCH][VEC], g[NCH][VEC], d[NCH][VEC];
        float q[3] = {0.f, 0.f, 0.f};  // sum s^2, sum a s, sum y^2
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int h = (c * blockDim.x + threadIdx.x) * VEC;
#pragma unroll
            for (int j = 0; j < VEC; ++j) s[c][j] = y[c][j] = g[c][j] = d[c][j] = 0.f;
            if (h < H) {
                if (a.go) {
                    load_vals<VEC>(a.go, row + h, a.o_bf16, g[c]);
                    load_vals<VEC>(a.s, row + h, a.x_bf16, s[c]);
                }
                if (a.gs) load_vals<VEC>(a.gs, row + h, a.x_bf16, d[c]);
                if (a.y) load_vals<VEC>(a.y, row + h, a.y_bf16, y[c]);
            }
        }
        if (a.go) {
#pragma unroll
            for (int c = 0; c < NCH; ++c) {
                const int h = (c * blockDim.x + threadIdx.x) * VEC;
                if (h >= H) continue;
                float w[VEC];
                load_vals<VEC>(a.pre_w, h, 0, w);
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
        block_sums<3>(q, tmp[0]);
        const float inv_h = 1.f / (float)H;
        const float r = rsqrtf(q[0] / (float)H + a.eps);
        const float ry = a.post_w ? rsqrtf(q[2] / (float)H + a.eps) : 1.f;
        const float k1 = r * r * (q[1] * inv_h);
        const float gt = a.gate_kind == COLI_GATE_TOKEN ? a.gate[t] : 1.f;
        float p[2] = {0.f, 0.f};  // sum b y, sum ds' n
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int h = (c * blockDim.x + threadIdx.x) * VEC;
            if (h >= H) continue;
            float w[VEC];
            if (a.go) {
                load_vals<VEC>(a.pre_w, h, 0, w);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    c_pre[c][j] += g[c][j] * (s[c][j] * r);
                    d[c][j] += r * (g[c][j] * w[j] - s[c][j] * k1);
                }
            }
            if (a.dx) store_vals<VEC>(a.dx, row + h, a.x_bf16, d[c]);
            if (a.y) {
                float pw[VEC], cg[VEC];
#pragma unroll
                for (int j = 0; j < VEC; ++j) pw[j] = cg[j] = 1.f;
                if (a.post_w) load_vals<VEC>(a.post_w, h, 0, pw);
                if (a.gate_kind == COLI_GATE_CHANNEL) load_vals<VEC>(a.gate, h, 0, cg);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float yh = y[c][j] * ry;       // normalised block output
                    const float ds = a.alpha * d[c][j];
                    const float dg = ds * (yh * pw[j]);
                    p[1] += dg;
                    c_gate[c][j] += dg;
                    const float dn = ds * (gt * cg[j]);
                    c_post[c][j] += dn * yh;
                    d[c][j] = dn * pw[j];                // b
                    p[0] += d[c][j] * y[c][j];
                }
            }
        }
        if (!a.y) {
            __syncthreads();  // tmp[0] is read by all before the next row writes it
            continue;
        }
        block_sums<2>(p, tmp[1]);
        const float k2 = a.post_w ? ry * ry * (p[0] * inv_h) : 0.f;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int h = (c * blockDim.x + threadIdx.x) * VEC;
            if (h >= H || !a.dy) continue;
#pragma unroll
            for (int j = 0; j < VEC; ++j) d[c][j] = ry * (d[c][j] - y[c][j] * k2);
            store_vals<VEC>(a.dy, row + h, a.y_bf16, d[c]);
        }
        if (a.dgate && a.gate_kind == COLI_GATE_TOKEN && threadIdx.x == 0) a.dgate[t] = p[1];
    }
    float* part = a.part + (int64_t)blockIdx.x * 3 * H;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
        const int h = (c * blockDim.x + threadIdx.x) * VEC;
        if (h >= H) continue;
        if (a.dpre_w) store_vals<VEC>(part, h, 0, c_pre[c]);
        if (a.dpost_w) store_vals<VEC>(part + H, h, 0, c_post[c]);
        if (a.dgate && a.gate_kind == COLI_GATE_CHANNEL) store_vals<VEC>(part + 2 * H, h, 0, c_gate[c]);
    }
}

// Column sums: out[h] = sum over the CTAs of part[cta][which][h], 32 columns
// per block, 8 warps over the CTAs; fixed order (each warp its strided share
// ascending, then the warps ascending).
__global__ void __launch_bounds__(256)
norm_columns_kernel(const float* part, int n_part, int H, float* dpre_w, float* dpost_w,
                    float* dgate) {
    __shared__ float acc[8][32];
    pdl_wait();
    pdl_launch_dependents();
    const int which = blockIdx.y;
    float* out = which == 0 ? dpre_w : which == 1 ? dpost_w : dgate;
    if (!out) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int h = blockIdx.x * 32 + lane;
    float v = 0.f;
    if (h < H) {
        const float* p = part + (int64_t)which * H + h;
#pragma unroll 4
        for (int i = warp; i < n_part; i += 8) v += p[(int64_t)i * 3 * H];
    }
    acc[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && h < H) {
#pragma unroll
        for (int w = 1; w < 8; ++w) v += acc[w][lane];
        out[h] = v;
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

// CTAs of the backward kernel: two per SM hide each other's row reductions.
int norm_bwd_ctas(int T) { return std::max(1, std::min(T, 2 * 148)); }

// Chunks per thread: rows of whole 8-value vectors use 16-byte accesses, other
// widths one value at a time.
template <template <int, int> class Launch>
cudaError_t dispatch_width(int H, int max_threads, const NormArgs& a, int grid, cudaStream_t st) {
    auto threads = [&](int vec, int nch) { return ((H + vec * nch - 1) / (vec * nch) + 31) / 32 * 32; };
    if (H % 8 == 0) {
        if (threads(8, 1) <= max_threads) return Launch<8, 1>::run(a, grid, threads(8, 1), st);
        if (threads(8, 2) <= max_threads) return Launch<8, 2>::run(a, grid, threads(8, 2), st);
        return Launch<8, 4>::run(a, grid, threads(8, 4), st);
    }
    if (threads(1, 4) <= 512) return Launch<1, 4>::run(a, grid, threads(1, 4), st);
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
    const cudaError_t err =
        dispatch_width<Forward>(H, T <= 148 ? 1024 : 512, a, T, static_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? COLI_OK : COLI_ERR_CUDA;
}

size_t coli_moe_block_norm_workspace_size(int32_t T, int32_t H) {
    if (T < 0 || H <= 0) return 0;
    return kHeaderBytes + sizeof(float) * 3 * (size_t)H * (size_t)norm_bwd_ctas(T);
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
        if (ws_bytes < coli_moe_block_norm_workspace_size(T, H)) return COLI_ERR_WORKSPACE;
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
    const int grid = norm_bwd_ctas(T);
    cudaError_t err = dispatch_width<Backward>(H, 512, a, grid, st);
    if (err == cudaSuccess && columns)
        err = launch_serialized(norm_columns_kernel, dim3((H + 31) / 32, 3), dim3(256), 0, st,
                                a.part, grid, H, dpre_w, dpost_w,
                                gate_kind == COLI_GATE_CHANNEL ? dgate : nullptr);
    return err == cudaSuccess ? COLI_OK : COLI_ERR_CUDA;
}

}  // extern "C"
