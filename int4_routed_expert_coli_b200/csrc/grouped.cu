// Matrix products of rows grouped by expert (ragged group sizes, read on the
// device from the batch-union's offsets), on the fifth-generation tensor
// cores, fp32 sums.  For expert e with the rows r of [offsets[e], offsets[e+1]):
//
//   kFwd  out[r][n]   = sum_k x[r][k] w[e][n][k]                 bf16 or e4m3
//   kDx   dx[r][k]    = sum_n dy[r][n] w[e][n][k]                bf16
//   kDw   dw[e][n][k] = sum_{r in e} dy[r][n] x[r][k]            bf16
//
// The long, regular dimension (weight rows; the weights' columns for kDx) is
// the MMA M (128 per CTA), the ragged rows are N (up to BN, in multiples of
// 16, so a group of 130 rows costs 144 and not two tiles of 128); kDw has
// n as M, k as N and the rows as the reduction.  Operands are read as they lie
// in memory: an operand whose reduction index is the slow one (w of kDx, both
// of kDw) is an MN-major tile, so no transposed copy exists.
//
// One CTA per SM, persistent; warp 0 loads (tensor copies, a ring of stages
// of 128 bytes x rows), warp 1 issues the MMAs, warps 4-11 drain the
// accumulators.  Tensor memory holds two accumulators; the MMAs of one run
// while the other is drained:
//   * a bf16 sum is drained into fp32 registers every kChunk K-blocks: the
//     tensor cores' fp32 accumulation truncates, and a chain of 6144 products
//     is 7e-6 off (16384: 2e-5), a chain of 2048 2e-6;
//   * an e4m3 sum is drained every block of 128, times the block's two scales
//     (the row's and the weight block's, whose product warps 2 and 3 put in
//     shared memory: a weight tile's 128 rows are one scale block).
//
// Tiles: whole waves of tiles are dealt to the CTAs in order; the tiles of the
// last, incomplete wave are dealt as one sequence of K-blocks, cut into equal
// ranges, so few tiles (one token's experts) still use every SM.  A tile cut
// by a range's end leaves fp32 partial sums in the workspace; the CTA that
// finishes last adds them in the order of the ranges (the same bits whoever
// is last) and writes the tile.
//
// Rows before offsets[0] and behind offsets[E] are neither read into a result
// nor written.  Every wait is bounded (COLI_ERR_TIMEOUT).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "coli_internal.cuh"
#include "launch.cuh"
#include "ptx.cuh"
#include "tcgen05.cuh"

namespace coli {
namespace {

enum Mode { kFwd = 0, kDx = 1, kDw = 2 };

constexpr int kBM = 128;               // M per CTA
constexpr int kRowBytes = 128;         // bytes of one operand row (or column) per stage
constexpr int kABytes = kBM * kRowBytes;
constexpr int kMaxStages = 12;
constexpr int kThreads = 384;
constexpr int kEpiWarp0 = 4, kEpiWarps = 8;
constexpr int kMaxGrid = 148;
constexpr int kChunk = 32;             // bf16 K-blocks per accumulator chain
constexpr int kScaleBufs = 4;
constexpr int kSmemMax = 227 * 1024;
constexpr int kMinRange = 4;           // K-blocks of a range of the last wave, at least

struct MmArgs {
    const int* offsets;   // [E + 1]
    int R, E;
    int M;                // rows of the M dimension (kFwd, kDw: N of the API; kDx: K)
    int red;              // reduction length (kFwd: K, kDx: N; kDw: per group)
    int cols;             // kDw: columns of dw
    void* out;
    int out_bf16, accumulate;
    const float* xs;      // fp8: [KB][R] scales of the rows
    const float* ws;      // fp8: [E][ceil(M/128)][KB] scales of the weights
    float* part;          // partial tiles, two per CTA
    int* counters;        // one per CTA, zero between calls
    int* status;
};

template <int MODE, bool FP8, int BN_>
struct Cfg {
    static constexpr int BN = BN_;
    static constexpr int BK = FP8 ? 128 : 64;              // reduction per stage
    static constexpr int kBoxRows = BN >= 256 ? 64 : 16;   // rows per B tensor copy
    static constexpr int kBBytes = BN * kRowBytes;
    static constexpr int kStage = kABytes + kBBytes;
    static constexpr int kTmemCols = 2 * BN;
    static constexpr bool kAMn = MODE != kFwd;
    static constexpr bool kBMn = MODE == kDw;
    static constexpr int kAcc = BN / 2;                    // accumulators per epilogue thread
};

// Everything of shared memory but the stages.
struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t sc_full[kScaleBufs], sc_empty[kScaleBufs];
    uint32_t tmem;
    int abort;
    int last;                              // this CTA finishes the cut tile
    long long scan[2][kThreads / 32 + 1];
    int tile0[kMaxExperts + 1];            // first tile (of the first M tile column) of each group
    long long step0[kMaxExperts + 1];      // K-block steps before each group
};
constexpr int kSharedBytes = (sizeof(Shared) + 127) / 128 * 128;

template <class C, bool FP8>
constexpr int scale_bytes() { return FP8 ? kScaleBufs * C::BN * 4 : 0; }
template <class C, bool FP8>
constexpr int stage_count() {
    return std::min(kMaxStages, (kSmemMax - 1024 - kSharedBytes - scale_bytes<C, FP8>()) / C::kStage);
}

// A piece of work: K-blocks [kb0, kb1) of one tile.
struct Piece {
    int e, m0;
    int row0, rows;      // kFwd, kDx: the tile's rows; kDw: the group's
    int col0;            // kDw: first column
    int n;               // valid columns of the MMA N dimension
    int kb0, kb1, kb;    // of kb
    long long step;      // of the tile's first K-block, relative to the last wave
};

// Where this CTA is in its sequence of pieces; every role walks its own copy.
template <int MODE, class C>
struct Walk {
    const MmArgs& a;
    const Shared& s;
    int m_tiles, c_tiles;
    long long full;              // tiles dealt whole
    long long tile;              // next of those
    long long cur, end, base;    // next step and end of this CTA's range; first step of the wave

    __device__ __forceinline__ Walk(const MmArgs& a_, const Shared& s_) : a(a_), s(s_) {
        m_tiles = (a.M + kBM - 1) / kBM;
        c_tiles = MODE == kDw ? (a.cols + C::BN - 1) / C::BN : 1;
        const long long per = (long long)m_tiles * c_tiles;
        const long long tiles = s.tile0[a.E] * per;
        full = tiles - tiles % gridDim.x;
        tile = blockIdx.x;
        const long long steps = s.step0[a.E] * per;
        base = full < tiles ? step_of(full) : steps;
        const long long q = range();
        cur = base + min(steps - base, q * blockIdx.x);
        end = base + min(steps - base, q * (blockIdx.x + 1));
    }
    // K-blocks of one CTA's range of the last wave
    __device__ __forceinline__ long long range() const {
        const long long n = s.step0[a.E] * ((long long)m_tiles * c_tiles) - base;
        return max((long long)kMinRange, (n + gridDim.x - 1) / gridDim.x);
    }
    __device__ __forceinline__ int group_kb(int e) const {
        if (MODE != kDw) return (a.red + C::BK - 1) / C::BK;
        const int rows = __ldg(a.offsets + e + 1) - __ldg(a.offsets + e);
        return max(1, (rows + C::BK - 1) / C::BK);
    }
    __device__ __forceinline__ int group_of_tile(long long t) const {
        const long long per = (long long)m_tiles * c_tiles;
        int lo = 0, hi = a.E;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s.tile0[mid] * per <= t) lo = mid;
            else hi = mid;
        }
        return lo;
    }
    __device__ __forceinline__ long long step_of(long long t) const {
        const long long per = (long long)m_tiles * c_tiles;
        const int e = group_of_tile(t);
        return s.step0[e] * per + (t - s.tile0[e] * per) * group_kb(e);
    }
    __device__ __forceinline__ void fill(Piece& p, int e, long long t, int kb) const {
        const int off = __ldg(a.offsets + e), rows = __ldg(a.offsets + e + 1) - off;
        p.e = e;
        p.kb = kb;
        if (MODE == kDw) {
            p.m0 = (int)(t / c_tiles) * kBM;
            p.col0 = (int)(t % c_tiles) * C::BN;
            p.n = min(C::BN, a.cols - p.col0);
            p.row0 = off;
            p.rows = rows;
        } else {
            // a group's rows are shared evenly by its row tiles (16-row grain)
            const int nt = s.tile0[e + 1] - s.tile0[e];
            const int bn = ((rows + nt - 1) / nt + 15) & ~15;
            const int i = (int)(t % nt) * bn;
            p.m0 = (int)(t / nt) * kBM;
            p.col0 = 0;
            p.row0 = off + i;
            p.rows = p.n = max(0, min(bn, rows - i));
        }
    }
    __device__ __forceinline__ bool next(Piece& p) {
        const long long per = (long long)m_tiles * c_tiles;
        if (tile < full) {
            const int e = group_of_tile(tile), kb = group_kb(e);
            fill(p, e, tile - s.tile0[e] * per, kb);
            p.kb0 = 0;
            p.kb1 = kb;
            p.step = -1;
            tile += gridDim.x;
            return true;
        }
        if (cur >= end) return false;
        int lo = 0, hi = a.E;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s.step0[mid] * per <= cur) lo = mid;
            else hi = mid;
        }
        const int kb = group_kb(lo);
        const long long in = cur - s.step0[lo] * per, t = in / kb;
        fill(p, lo, t, kb);
        p.kb0 = (int)(in - t * kb);
        p.kb1 = (int)min((long long)kb, p.kb0 + (end - cur));
        p.step = cur - p.kb0 - base;
        cur += p.kb1 - p.kb0;
        return true;
    }
};

// Columns of the MMA: the valid ones rounded up to 16.
__device__ __forceinline__ int mma_n(int n) { return max(16, (n + 15) & ~15); }

template <int MODE, bool FP8, int BN_>
__global__ void __launch_bounds__(kThreads, 1)
grouped_mm_kernel(const __grid_constant__ CUtensorMap amap,
                  const __grid_constant__ CUtensorMap bmap, const MmArgs a) {
    using C = Cfg<MODE, FP8, BN_>;
    constexpr int kStages = stage_count<C, FP8>();
    extern __shared__ uint8_t smem_raw[];
    uint8_t* stage0 = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* scale0 = reinterpret_cast<float*>(stage0 + (size_t)kStages * C::kStage);
    Shared& s = *reinterpret_cast<Shared*>(stage0 + (size_t)kStages * C::kStage +
                                           scale_bytes<C, FP8>());
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int* abort = &s.abort;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.acc_full[i], 1);
            mbar_init(&s.acc_empty[i], kEpiWarps);
        }
        for (int i = 0; i < kScaleBufs; ++i) {
            mbar_init(&s.sc_full[i], 1);
            mbar_init(&s.sc_empty[i], kEpiWarps);
        }
        s.abort = 0;
        fence_barrier_init();
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_addr(&s.tmem)),
                     "r"(C::kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    pdl_launch_dependents();
    pdl_wait();

    // Tiles and K-block steps before each group (of one M tile): a scan over
    // the groups, three per thread.  An impossible offset pair is reported and
    // gets no tile.
    {
        long long v[3], w[3], sum_v = 0, sum_w = 0;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const int e = threadIdx.x * 3 + i;
            v[i] = w[i] = 0;
            if (e < a.E) {
                const int lo = __ldg(a.offsets + e), hi = __ldg(a.offsets + e + 1);
                if (lo < 0 || hi < lo || hi > a.R) {
                    report(a.status, COLI_ERR_BAD_INDEX);
                } else if (MODE == kDw) {
                    v[i] = 1;
                    w[i] = max(1, (hi - lo + C::BK - 1) / C::BK);
                } else {
                    v[i] = (hi - lo + C::BN - 1) / C::BN;
                    w[i] = v[i] * ((a.red + C::BK - 1) / C::BK);
                }
            }
            sum_v += v[i];
            sum_w += w[i];
        }
        long long iv = sum_v, iw = sum_w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long nv = __shfl_up_sync(0xffffffffu, iv, o);
            const long long nw = __shfl_up_sync(0xffffffffu, iw, o);
            if (lane >= o) {
                iv += nv;
                iw += nw;
            }
        }
        if (lane == 31) {
            s.scan[0][warp] = iv;
            s.scan[1][warp] = iw;
        }
        __syncthreads();
        long long bv = iv - sum_v, bw = iw - sum_w;
        for (int i = 0; i < warp; ++i) {
            bv += s.scan[0][i];
            bw += s.scan[1][i];
        }
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const int e = threadIdx.x * 3 + i;
            if (e <= a.E) {
                s.tile0[e] = (int)bv;
                s.step0[e] = bw;
            }
            bv += v[i];
            bw += w[i];
        }
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&s.tmem);

    auto stage_ptr = [&](int i) { return stage0 + (size_t)i * C::kStage; };
    auto timeout = [&]() {
        report(a.status, COLI_ERR_TIMEOUT);
        *abort = 1;
    };
    Walk<MODE, C> walk(a, s);
    Piece p;

    if (warp == 0) {
        // ------------------------------- loads ---------------------------------
        if (lane == 0) {
            uint32_t it = 0;
            while (!*abort && walk.next(p)) {
                if (MODE == kDw && p.rows == 0) continue;  // nothing to add up
                const int boxes = MODE == kDw ? (p.n + 63) / 64
                                              : (p.n + C::kBoxRows - 1) / C::kBoxRows;
                const uint32_t bytes =
                    kABytes + boxes * (MODE == kDw ? 64 : C::kBoxRows) * kRowBytes;
                bool ok = true;
                for (int kb = p.kb0; kb < p.kb1; ++kb, ++it) {
                    const int i = it % kStages;
                    if (it >= kStages && !mbar_wait(&s.empty[i], (it / kStages - 1) & 1)) {
                        timeout();
                        ok = false;
                        break;
                    }
                    uint8_t* sa = stage_ptr(i);
                    uint8_t* sb = sa + kABytes;
                    mbar_arrive_expect_tx(&s.full[i], bytes);
                    if constexpr (MODE == kFwd) {
                        tc::tma_3d(sa, &amap, kb * C::BK, p.m0, p.e, &s.full[i]);
                    } else if constexpr (MODE == kDx) {
                        tc::tma_3d(sa, &amap, p.m0, kb * C::BK, p.e, &s.full[i]);
                        tc::tma_3d(sa + kABytes / 2, &amap, p.m0 + 64, kb * C::BK, p.e, &s.full[i]);
                    } else {
                        const int r = p.row0 + kb * C::BK;
                        tc::tma_2d(sa, &amap, p.m0, r, &s.full[i]);
                        tc::tma_2d(sa + kABytes / 2, &amap, p.m0 + 64, r, &s.full[i]);
                    }
                    if constexpr (MODE == kDw) {
                        for (int b = 0; b < boxes; ++b)
                            tc::tma_2d(sb + b * 64 * kRowBytes, &bmap, p.col0 + b * 64,
                                       p.row0 + kb * C::BK, &s.full[i]);
                    } else {
                        for (int b = 0; b < boxes; ++b)
                            tc::tma_2d(sb + b * C::kBoxRows * kRowBytes, &bmap, kb * C::BK,
                                       p.row0 + b * C::kBoxRows, &s.full[i]);
                    }
                }
                if (!ok) break;
            }
            // after a timeout nobody consumes the stages: the copies in flight
            // still end before this CTA does
            if (*abort)
                for (uint32_t j = it > kStages ? it - kStages : 0; j < it; ++j)
                    mbar_wait(&s.full[j % kStages], (j / kStages) & 1);
        }
    } else if (warp == 1) {
        // -------------------------------- MMAs ---------------------------------
        const uint64_t abase = C::kAMn ? tc::desc_base(64 * kRowBytes, 1024) : tc::desc_base(0, 1024);
        const uint64_t bbase = C::kBMn ? tc::desc_base(64 * kRowBytes, 1024) : tc::desc_base(0, 1024);
        constexpr uint32_t kAStep = C::kAMn ? 2048 / 16 : 2;  // one MMA along the reduction
        constexpr uint32_t kBStep = C::kBMn ? 2048 / 16 : 2;
        uint32_t it = 0, ch = 0;
        while (!*abort && walk.next(p)) {
            if (MODE == kDw && p.rows == 0) continue;
            const uint32_t id = tc::idesc(kBM, mma_n(p.n), FP8 ? 0 : 1, C::kAMn, C::kBMn);
            bool ok = true;
            for (int kb = p.kb0; kb < p.kb1; ++kb, ++it) {
                const bool first = FP8 || (kb - p.kb0) % kChunk == 0;
                const uint32_t buf = ch & 1;
                if (first && ch >= 2) {
                    if (!mbar_wait(&s.acc_empty[buf], (ch / 2 - 1) & 1)) ok = false;
                }
                const int i = it % kStages;
                if (!ok || !mbar_wait(&s.full[i], (it / kStages) & 1)) {
                    timeout();
                    ok = false;
                    break;
                }
                int steps = 4;
                if constexpr (MODE == kDw) {
                    // the group's last K-block: rows of the next group behind
                    // its end are cleared (in both operands: they may hold
                    // infinities), whole MMA steps of them are left out
                    const int valid = p.rows - kb * C::BK;
                    if (valid < C::BK) {
                        steps = (valid + 15) / 16;
                        const int boxes = 2 + (p.n + 63) / 64;
                        const int clear = (steps * 16 - valid) * 8;
                        uint8_t* sa = stage_ptr(i);
                        for (int b = 0; b < boxes; ++b)
                            for (int j = lane; j < clear; j += 32)
                                *reinterpret_cast<uint4*>(sa + b * 64 * kRowBytes +
                                                          valid * kRowBytes + j * 16) =
                                    make_uint4(0, 0, 0, 0);
                        fence_proxy_async();
                        __syncwarp();
                    }
                }
                tc::fence_after();
                const bool last = FP8 || kb + 1 == p.kb1 || (kb - p.kb0) % kChunk == kChunk - 1;
                if (lane == 0) {
                    const uint32_t sa = smem_addr(stage_ptr(i));
                    const uint64_t ad = tc::desc_at(abase, sa);
                    const uint64_t bd = tc::desc_at(bbase, sa + kABytes);
                    const uint32_t d = tmem + buf * C::BN;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (k < steps)
                            tc::mma<FP8, 1>(d, ad + k * kAStep, bd + k * kBStep, id,
                                            !first || k > 0);
                    tc::commit(&s.empty[i]);
                    if (last) tc::commit(&s.acc_full[buf]);
                }
                __syncwarp();
                if (last) ++ch;
            }
            if (!ok) break;
        }
    } else if (warp < kEpiWarp0) {
        // ---------------- fp8: products of the two scales, per column -------------
        if constexpr (FP8) {
            const int KB = (a.red + C::BK - 1) / C::BK;
            uint32_t ch = 0;
            while (!*abort && walk.next(p)) {
                const float* wsc = a.ws + ((int64_t)p.e * walk.m_tiles + p.m0 / kBM) * KB;
                bool ok = true;
                for (int kb = p.kb0; kb < p.kb1; ++kb, ++ch) {
                    if ((int)(ch & 1) != warp - 2) continue;  // the two warps alternate
                    const int b = ch % kScaleBufs;
                    const float sw = __ldg(wsc + kb);
                    const float* xs = a.xs + (int64_t)kb * a.R + p.row0;
                    float v[C::BN / 32];
#pragma unroll
                    for (int j = 0; j < C::BN / 32; ++j)
                        v[j] = j * 32 + lane < p.n ? __ldg(xs + j * 32 + lane) * sw : 0.f;
                    if (ch >= kScaleBufs && !mbar_wait(&s.sc_empty[b], (ch / kScaleBufs - 1) & 1)) {
                        if (lane == 0) timeout();
                        ok = false;
                        break;
                    }
#pragma unroll
                    for (int j = 0; j < C::BN / 32; ++j) scale0[b * C::BN + j * 32 + lane] = v[j];
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s.sc_full[b]);
                }
                if (!ok) break;
            }
        }
    } else {
        // ------------------------------ epilogue ---------------------------------
        const int q = warp & 3, half = (warp - kEpiWarp0) >> 2;
        const int mrow = q * 32 + lane;       // row of the tile
        const int c0 = half * C::kAcc;        // this thread's columns: [c0, c0 + kAcc)
        const uint32_t tq = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)c0;
        uint32_t ch = 0;
        while (!*abort && walk.next(p)) {
            float acc[C::kAcc];
#pragma unroll
            for (int j = 0; j < C::kAcc; ++j) acc[j] = 0.f;
            bool ok = true;
            if (!(MODE == kDw && p.rows == 0)) {
                const int n_ch = FP8 ? p.kb1 - p.kb0 : (p.kb1 - p.kb0 + kChunk - 1) / kChunk;
                for (int i = 0; i < n_ch; ++i, ++ch) {
                    const uint32_t buf = ch & 1, sb = ch % kScaleBufs;
                    if (!mbar_wait(&s.acc_full[buf], (ch / 2) & 1) ||
                        (FP8 && !mbar_wait(&s.sc_full[sb], (ch / kScaleBufs) & 1))) {
                        if (lane == 0) timeout();
                        ok = false;
                        break;
                    }
                    tc::fence_after();
#pragma unroll
                    for (int j0 = 0; j0 < C::kAcc; j0 += 16) {
                        if (c0 + j0 < p.n) {
                            uint32_t v[16];
                            tc::ld16(tq + buf * C::BN + j0, v);
                            tc::ld_wait(v);
                            if constexpr (FP8) {
                                const float4* sc =
                                    reinterpret_cast<const float4*>(scale0 + sb * C::BN + c0 + j0);
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    const float4 f = sc[j];
                                    acc[j0 + 4 * j] += __uint_as_float(v[4 * j]) * f.x;
                                    acc[j0 + 4 * j + 1] += __uint_as_float(v[4 * j + 1]) * f.y;
                                    acc[j0 + 4 * j + 2] += __uint_as_float(v[4 * j + 2]) * f.z;
                                    acc[j0 + 4 * j + 3] += __uint_as_float(v[4 * j + 3]) * f.w;
                                }
                            } else {
#pragma unroll
                                for (int j = 0; j < 16; ++j) acc[j0 + j] += __uint_as_float(v[j]);
                            }
                        }
                    }
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&s.acc_empty[buf]);
                        if (FP8) mbar_arrive(&s.sc_empty[sb]);
                    }
                }
            }
            if (!ok) break;

            if (p.kb1 - p.kb0 < p.kb) {
                // a cut tile: leave the partial sums; the last of its ranges adds them
                const long long rng = walk.range();
                const int c_first = (int)(p.step / rng);
                const int c_last = (int)((p.step + p.kb - 1) / rng);
                float* mine = a.part + ((int64_t)blockIdx.x * 2 + (p.kb0 == 0)) * (kBM * C::BN);
#pragma unroll
                for (int j = 0; j < C::kAcc; ++j)
                    if (c0 + j < p.n) __stcg(mine + (c0 + j) * kBM + mrow, acc[j]);
                __threadfence();
                named_barrier(1, kEpiWarps * 32);
                if (warp == kEpiWarp0 && lane == 0) {
                    const int before = atomicAdd(a.counters + c_first, 1);
                    s.last = before == c_last - c_first;
                    if (s.last) a.counters[c_first] = 0;
                }
                named_barrier(1, kEpiWarps * 32);
                if (!*const_cast<volatile int*>(&s.last)) continue;
                __threadfence();
#pragma unroll
                for (int j = 0; j < C::kAcc; ++j) acc[j] = 0.f;
                for (int c = c_first; c <= c_last; ++c) {
                    const float* src = a.part + ((int64_t)c * 2 + (c == c_first)) * (kBM * C::BN);
#pragma unroll
                    for (int j = 0; j < C::kAcc; ++j)
                        if (c0 + j < p.n) acc[j] += __ldcg(src + (c0 + j) * kBM + mrow);
                }
            }

            const int m = p.m0 + mrow;
            if (m >= a.M) {
                // a row of the last M tile that does not exist
            } else if constexpr (MODE == kDw) {
                // a thread's columns are consecutive in its row of dw; columns
                // come in whole vectors of 8
                const int64_t o = ((int64_t)p.e * a.M + m) * a.cols + p.col0;
#pragma unroll
                for (int j0 = 0; j0 < C::kAcc; j0 += 8) {
                    if (c0 + j0 >= p.n) continue;
                    float* v = acc + j0;
                    if (a.out_bf16) {
                        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + o +
                                                              c0 + j0);
                        uint32_t u[4];
                        if (a.accumulate) {
                            const uint4 old = *dst;
                            const uint32_t w[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                v[2 * j] += __uint_as_float(w[j] << 16);
                                v[2 * j + 1] += __uint_as_float(w[j] & 0xFFFF0000u);
                            }
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                            u[j] = *reinterpret_cast<const uint32_t*>(&h);
                        }
                        *dst = make_uint4(u[0], u[1], u[2], u[3]);
                    } else {
                        float4* dst =
                            reinterpret_cast<float4*>(static_cast<float*>(a.out) + o + c0 + j0);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            float4 f = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2],
                                                   v[4 * j + 3]);
                            if (a.accumulate) {
                                const float4 old = dst[j];
                                f.x += old.x; f.y += old.y; f.z += old.z; f.w += old.w;
                            }
                            dst[j] = f;
                        }
                    }
                }
            } else {
                // a warp writes 32 consecutive values of one row at a time
                const int64_t o = (int64_t)p.row0 * a.M + m;
                if (a.out_bf16) {
                    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + o;
#pragma unroll
                    for (int j = 0; j < C::kAcc; ++j)
                        if (c0 + j < p.n) dst[(int64_t)(c0 + j) * a.M] = __float2bfloat16_rn(acc[j]);
                } else {
                    float* dst = static_cast<float*>(a.out) + o;
#pragma unroll
                    for (int j = 0; j < C::kAcc; ++j)
                        if (c0 + j < p.n) dst[(int64_t)(c0 + j) * a.M] = acc[j];
                }
            }
            __syncwarp();
        }
    }

    tc::fence_before();
    __syncthreads();
    if (warp == 2) {
        tc::fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(C::kTmemCols)
                     : "memory");
    }
}

// ---- host -----------------------------------------------------------------------

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// [outer][rows][inner] elements (bf16 or bytes), boxes of 128 bytes x box_rows
// with the 128-byte swizzle; what lies outside reads as zero.
bool encode_operand(CUtensorMap* m, bool fp8, const void* base, int inner, int64_t rows, int outer,
                    int box_rows) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    const uint64_t size = fp8 ? 1 : 2;
    const cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)rows, (cuuint64_t)outer};
    const cuuint64_t strides[2] = {inner * size, inner * size * (uint64_t)rows};
    const cuuint32_t box[3] = {(cuuint32_t)(kRowBytes / size), (cuuint32_t)box_rows, 1};
    const cuuint32_t es[3] = {1, 1, 1};
    return enc(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
               outer > 0 ? 3 : 2, const_cast<void*>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE, bool FP8, int BN>
coli_status launch_mm(const void* A, const void* B, const MmArgs& a, int N, int K, cudaStream_t st) {
    using C = Cfg<MODE, FP8, BN>;
    CUtensorMap amap, bmap;
    bool ok;
    if constexpr (MODE == kDw)
        ok = encode_operand(&amap, false, A, N, a.R, 0, 64) &&
             encode_operand(&bmap, false, B, K, a.R, 0, 64);
    else
        ok = encode_operand(&amap, FP8, A, K, N, a.E, MODE == kFwd ? kBM : 64) &&
             encode_operand(&bmap, FP8, B, MODE == kFwd ? K : N, a.R, 0, C::kBoxRows);
    if (!ok) return COLI_ERR_CUDA;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return COLI_ERR_CUDA;
    constexpr int smem = 1024 + stage_count<C, FP8>() * C::kStage + scale_bytes<C, FP8>() +
                         kSharedBytes;
    static_assert(smem <= kSmemMax && stage_count<C, FP8>() >= 3, "shared memory");
    auto kernel = grouped_mm_kernel<MODE, FP8, BN>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
        cudaSuccess)
        return COLI_ERR_CUDA;
    const cudaError_t err =
        launch_serialized(kernel, dim3(std::min(sms, kMaxGrid)), dim3(kThreads), smem, st, amap,
                          bmap, a);
    return err == cudaSuccess ? COLI_OK : COLI_ERR_CUDA;
}

// Narrow row tiles when the groups average at most 32 rows: the loads of the
// weights bound such calls, and narrow tiles leave room for more of them.
bool narrow(int R, int E) { return (int64_t)R <= 32 * (int64_t)E; }

constexpr size_t kPartBytes = sizeof(float) * kMaxGrid * 2 * kBM * 256;

coli_status check_mm(int32_t R, int32_t E, int32_t N, int32_t K, int grain) {
    if (R < 0 || E < 1 || N < 1 || K < 1) return COLI_ERR_INVALID_ARG;
    if (E > kMaxExperts || R > 1 << 24 || N % 8 || K % grain || N > 65536 || K > 65536)
        return COLI_ERR_SHAPE;
    return COLI_OK;
}

// Pointer, alignment and workspace checks of a call with R > 0.
coli_status check_ptrs(const void* a, const void* b, const int32_t* offsets, const void* out,
                       int out_dtype, const void* ws, size_t ws_bytes) {
    if (!valid_dtype(out_dtype)) return COLI_ERR_INVALID_ARG;
    if (!a || !b || !offsets || !out || !ws) return COLI_ERR_INVALID_ARG;
    if (!ptr_aligned(a, 16) || !ptr_aligned(b, 16) || !ptr_aligned(out, 16) ||
        !ptr_aligned(offsets, 4) || !ptr_aligned(ws, 256))
        return COLI_ERR_ALIGN;
    if (ws_bytes < kHeaderBytes + kPartBytes) return COLI_ERR_WORKSPACE;
    return COLI_OK;
}

MmArgs make_mm_args(const int32_t* offsets, int R, int E, int M, int red, void* out,
                    coli_out_dtype od, void* ws) {
    MmArgs a = {};
    a.offsets = offsets;
    a.R = R;
    a.E = E;
    a.M = M;
    a.red = red;
    a.out = out;
    a.out_bf16 = od == COLI_OUT_BF16;
    a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + kHeaderBytes);
    a.counters = reinterpret_cast<int*>(static_cast<char*>(ws) + kTileCntOffset);
    a.status = static_cast<int*>(ws);
    return a;
}

}  // namespace
}  // namespace coli

using namespace coli;

extern "C" {

size_t coli_moe_grouped_workspace_size(int32_t R, int32_t E) {
    return R < 0 || E < 1 ? 0 : kHeaderBytes + kPartBytes;
}

coli_status coli_moe_grouped_mm(int32_t R, int32_t E, int32_t N, int32_t K, const void* x_bf16,
                                const void* w_bf16, const int32_t* offsets, void* out,
                                coli_out_dtype out_dtype, void* ws, size_t ws_bytes, void* stream) {
    coli_status s = check_mm(R, E, N, K, 8);
    if (s != COLI_OK || R == 0) return s;
    s = check_ptrs(x_bf16, w_bf16, offsets, out, out_dtype, ws, ws_bytes);
    if (s != COLI_OK) return s;
    const MmArgs a = make_mm_args(offsets, R, E, N, K, out, out_dtype, ws);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return narrow(R, E) ? launch_mm<kFwd, false, 64>(w_bf16, x_bf16, a, N, K, st)
                        : launch_mm<kFwd, false, 256>(w_bf16, x_bf16, a, N, K, st);
}

coli_status coli_moe_grouped_mm_dx(int32_t R, int32_t E, int32_t N, int32_t K, const void* dy_bf16,
                                   const void* w_bf16, const int32_t* offsets, void* dx,
                                   coli_out_dtype dx_dtype, void* ws, size_t ws_bytes,
                                   void* stream) {
    coli_status s = check_mm(R, E, N, K, 8);
    if (s != COLI_OK || R == 0) return s;
    s = check_ptrs(dy_bf16, w_bf16, offsets, dx, dx_dtype, ws, ws_bytes);
    if (s != COLI_OK) return s;
    const MmArgs a = make_mm_args(offsets, R, E, K, N, dx, dx_dtype, ws);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return narrow(R, E) ? launch_mm<kDx, false, 64>(w_bf16, dy_bf16, a, N, K, st)
                        : launch_mm<kDx, false, 256>(w_bf16, dy_bf16, a, N, K, st);
}

coli_status coli_moe_grouped_mm_dw(int32_t R, int32_t E, int32_t N, int32_t K, const void* dy_bf16,
                                   const void* x_bf16, const int32_t* offsets, void* dw,
                                   coli_out_dtype dw_dtype, int32_t accumulate, void* ws,
                                   size_t ws_bytes, void* stream) {
    coli_status s = check_mm(R, E, N, K, 8);
    if (s != COLI_OK) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (R == 0) {  // no rows: gradients of zero
        if (!dw || !valid_dtype(dw_dtype)) return COLI_ERR_INVALID_ARG;
        if (accumulate) return COLI_OK;
        const size_t n = (size_t)E * N * K * (dw_dtype == COLI_OUT_BF16 ? 2 : 4);
        return cudaMemsetAsync(dw, 0, n, st) == cudaSuccess ? COLI_OK : COLI_ERR_CUDA;
    }
    s = check_ptrs(dy_bf16, x_bf16, offsets, dw, dw_dtype, ws, ws_bytes);
    if (s != COLI_OK) return s;
    MmArgs a = make_mm_args(offsets, R, E, N, 0, dw, dw_dtype, ws);
    a.cols = K;
    a.accumulate = accumulate != 0;
    return launch_mm<kDw, false, 256>(dy_bf16, x_bf16, a, N, K, st);
}

coli_status coli_moe_fp8_grouped_mm(int32_t R, int32_t E, int32_t N, int32_t K, const uint8_t* xq,
                                    const float* x_scale, const uint8_t* wq, const float* w_scale,
                                    const int32_t* offsets, void* out, coli_out_dtype out_dtype,
                                    void* ws, size_t ws_bytes, void* stream) {
    coli_status s = check_mm(R, E, N, K, 16);
    if (s != COLI_OK || R == 0) return s;
    s = check_ptrs(xq, wq, offsets, out, out_dtype, ws, ws_bytes);
    if (s != COLI_OK) return s;
    if (!x_scale || !w_scale) return COLI_ERR_INVALID_ARG;
    if (!ptr_aligned(x_scale, 16) || !ptr_aligned(w_scale, 16)) return COLI_ERR_ALIGN;
    MmArgs a = make_mm_args(offsets, R, E, N, K, out, out_dtype, ws);
    a.xs = x_scale;
    a.ws = w_scale;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return narrow(R, E) ? launch_mm<kFwd, true, 64>(wq, xq, a, N, K, st)
                        : launch_mm<kFwd, true, 256>(wq, xq, a, N, K, st);
}

}  // extern "C"
