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
// 16 per CTA, so a group of 130 rows costs 160 and not two tiles of 128); kDw has
// n as M, k as N and the rows as the reduction.  Operands are read as they lie
// in memory: an operand whose reduction index is the slow one (w of kDx, both
// of kDw) is an MN-major tile, so no transposed copy exists.  Wide e4m3 products
// have the rows as M (kFwdRows): a thread then drains one row, with one scale a
// K-block, and not one for each of its columns (4096 rows of 32 experts of 4096 x
// 6144: 199 us, with the weights as M 291).
//
// One CTA per SM, persistent; one thread of warp 0 loads (tensor copies into a
// ring of stages of 128 bytes x rows), one of warp 1 issues the MMAs, warp 2 copies
// scales or clears rows, eight warps drain the accumulators, of which tensor
// memory holds two or more; the MMAs of one run while another is drained:
//   * a bf16 sum is drained into fp32 registers every kChunk K-blocks at most:
//     the tensor cores' fp32 accumulation truncates, and a chain of 6144
//     products is 7e-6 off (16384: 2e-5), one of 768 below 1e-6;
//   * an e4m3 sum is drained every block of 128, times the block's two scales
//     (the row's and the weight block's; 128 weight rows are one scale block),
//     which are copied ahead into shared memory.
// bf16 tiles are 256 x 256 by a pair of CTAs (each loads its half of both operands:
// a K-block of 64 is 32 KB a CTA for 128 x 256 x 64), or 128 x 64 by one where the
// weights' stream bounds the call or few tiles would leave SMs idle (`narrow`).
//
// What bounds them, and the measured times (B200, one call between L2 flushes):
//   * 8192 x 6144 x 6144 bf16 405 us, 1.53 PFLOP/s (a stream of calls, at the 1.3
//     GHz that the power limit leaves, 487): the tensor cores; e4m3 391 us: the
//     drain, whose round trip (commit, wait, read, release) a K-block of 128 pays
//     for, 0.76 us each, twice its MMAs;
//   * 4096 rows of 32 experts of 4096 x 6144 bf16 308 us (weights alone 245 at a
//     copy's rate), 8192 rows back to their gradient 365 (ten groups of more than
//     256 rows read their weights twice);
//   * weight gradients of 16384 rows of the same experts 1070 us in fp32 (3.2 GB
//     written: 490 at a copy's rate), 900 in bf16.  In 1, 8, 32, 64 equal groups,
//     with pauses, fp32 590, 625, 910, 1390 us, bf16 580, 580, 740, 1090: from 8 to
//     64 the added results take their own time, 7.4 and 5.5 TB/s of them, as if
//     nothing of it passed under the MMAs.  Added to what dw holds (32 groups):
//     fp32 1510; bf16, each thread at its own row, 16 bytes at a time, 2170;
//   * one token's eight experts: bf16 67 us (6.0 TB/s), e4m3 41 (4.9 TB/s): the
//     weights' stream, and its start and end.
//
// Tiles: whole waves of tiles are dealt to the workers in order; the tiles of the
// last, incomplete wave, where that pays, as one sequence of K-blocks, cut into
// equal ranges, so few tiles (one token's experts) still use every SM.  A tile cut
// by a range's end leaves fp32 partial sums in the workspace; of the warps that
// hold the same part of a tile, the one that finishes last adds them in the order
// of the ranges (the same bits whoever is last) and writes it.
//
// Rows before offsets[0] and behind offsets[E] are neither read into a result
// nor written.  Every wait is bounded (COLI_ERR_TIMEOUT): the roles of a CTA wait
// for each other at barriers in shared memory only, with a limit, and meet once,
// at the kernel's end, which each reaches when its own next wait runs out.
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

// kFwdRows: kFwd with the rows as M and the weight rows as N
enum Mode { kFwd = 0, kDx = 1, kDw = 2, kFwdRows = 3 };

constexpr int kBM = 128;               // M per CTA
constexpr int kRowBytes = 128;         // bytes of one operand row (or column) per stage
constexpr int kABytes = kBM * kRowBytes;
constexpr int kMaxStages = 12;
constexpr int kTmemAll = 512;          // tensor memory columns
constexpr int kMaxBufs = 8;
constexpr int kEpiWarps = 8;
constexpr int kMaxGrid = 148;
constexpr int kChunk = 12;             // bf16 K-blocks per accumulator chain, at most
constexpr int kScaleBufs = 4;          // handovers whose column scales are loaded ahead
constexpr int kScaleRing = 8;          // kFwdRows: K-blocks whose scales are loaded ahead
constexpr int kSmemMax = 227 * 1024;
constexpr uint64_t kSettleNs = 100000; // after a timeout, for copies that no barrier counts
// The last wave is cut into ranges of kMinRange K-blocks at least, and not at all
// where a whole tile costs a worker at most Cfg::kCutCost K-blocks more than its
// range.
constexpr int kMinRange = 12;
constexpr int kBand = 8;               // row tiles that share their weights' strips in L2
// kDw: a warp's stores leave through kStoreBufs stagings of 32 rows x 64 bytes
constexpr int kStoreBytes = 32 * 64, kStoreBufs = 3;

// Tensor maps of a call.  An MN-major operand is copied 64 columns at a time
// (a[0], b[0]), or 128 at once where its rows are whole runs of 64 columns
// (a[1], b[1]: the runs are a dimension of their own); b[i] of a K-major one has
// boxes of (i + 1) kBoxRows rows.
struct Maps {
    CUtensorMap a[2], b[4], out;
};

struct MmArgs {
    const int* offsets;   // [E + 1]
    int R, E;
    int M;                // rows of the M dimension (kFwd, kDw: N of the API; kDx: K)
    int red;              // reduction length (kFwd: K, kDx: N; kDw: per group)
    int cols;             // kDw: columns of dw
    void* out;
    int out_bf16, accumulate;
    int a_wide, b_wide;   // maps a[1], b[1] exist (MN-major operands)
    const float* xs;      // fp8: [KB][R] scales of the rows
    const float* ws;      // fp8: [E][ceil(M/128)][KB] scales of the weights
    float* part;          // partial tiles, two per CTA
    int* counters;        // one per epilogue warp, zero between calls
    int* status;
    uint64_t wait_ns;     // time limit of a wait
    int withhold;         // test hook: CTA 0's first stage never fills
};

// CTAS = 2: a pair of CTAs works on one tile of 256 M rows.  Each holds its
// 128 rows of A and half of the columns of B; the even one issues the MMAs of
// both (cta_group::2), each drains its own 128 rows.
template <int MODE, bool FP8, int BN_, int CTAS_>
struct Cfg {
    static constexpr int BN = BN_, CTAS = CTAS_;
    static constexpr int BK = FP8 ? 128 : 64;              // reduction per stage
    static constexpr bool kRows = MODE == kFwdRows;
    // A part of B is loaded by one tensor copy of its rows rounded up to this: a
    // box of 1 .. kBoxes times as many rows (with several copies of 32 rows 8192 x
    // 6144 x 6144 took 4 % longer).
    static constexpr int kBoxRows = kRows ? 128 : BN == 256 ? 32 : 16;
    [[maybe_unused]] static constexpr int kBoxes = MODE == kDw ? 0 : BN / CTAS / kBoxRows;
    static constexpr int kBBytes = BN / CTAS * kRowBytes;
    static constexpr int kStage = kABytes + kBBytes;
    static constexpr bool kColScale = FP8 && MODE != kFwdRows;  // scales per column
    // Accumulators per handover: a narrow e4m3 tile's K-block is little work, and
    // the round trip of its accumulator, paid for each, took 0.53 us of a K-block
    // whose weights come in 0.2 (one token's eight experts 52 us, with four 42).
    static constexpr int kBatch = kColScale ? 4 : 1;
    static constexpr int kBufs = kTmemAll / (BN * kBatch);      // handovers under way
    // What partial sums cost, in K-blocks: a narrow tile's are 32 KB a CTA, a wide
    // one's 128 KB, about 15 us to leave and be added up.  With 12 for all, whole
    // tiles being better: 2048 rows of 8 groups, N 512, K 2048 bf16 30.4 us and 20.2,
    // 600 rows of 3 groups of 4096 x 6144 54 and 44, 300 x 2048 x 2048 (narrow) 17.5
    // and 14.1, 512 x 4096 x 4096 e4m3 31 and 26.
    static constexpr int kCutCost = BN <= 64 ? 32 : FP8 ? 24 : 40;
    static constexpr int kNGrain = 16 * CTAS;              // MMA N in multiples of this
    static constexpr bool kAMn = MODE == kDx || MODE == kDw;
    static constexpr bool kBMn = MODE == kDw;
    static constexpr int kAcc = BN / 2;                    // accumulators per epilogue thread
    // Four front warps (loads, MMAs, one that copies scales or clears), eight of
    // the epilogue.  A wide tile's epilogue thread holds 128 sums and 32 loaded
    // values, more than 384 threads can have each (168 registers): the front
    // warpgroup gives registers to the epilogue's two.
    static constexpr int kFront = 4;
    static constexpr bool kSplitRegs = kAcc > 64;
    static constexpr int kFrontRegs = 72, kEpiRegs = 216;
    static_assert(128 * kFrontRegs + 256 * kEpiRegs <= 384 * 168, "register split");
    static constexpr int kThreads = (kFront + kEpiWarps) * 32;
    static constexpr int kStoreStage = MODE == kDw ? kEpiWarps * kStoreBufs * kStoreBytes : 0;
    static constexpr int kScaleSlot = BN + 4;              // floats (a multiple of 16 bytes)
    static constexpr int kScaleBytes =
        kColScale ? kScaleBufs * kBatch * kScaleSlot * 4 : kRows && FP8 ? kScaleRing * kEpiWarps * 32 * 8 : 0;
};

// Everything of shared memory but the stages.
struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t acc_full[kMaxBufs], acc_empty[kMaxBufs];
    uint64_t sc_full[kScaleBufs], sc_empty[kScaleBufs];
    // kDw, a group's cut last K-block: its copies are done; the rows behind the
    // group's end are cleared
    uint64_t tail_full[kMaxStages], tail_ready[kMaxStages];
    uint64_t mma_done;                     // after a timeout: no MMA is under way
    uint32_t tmem;
    uint32_t loaded;                       // kDw: K-blocks loaded, at the ring's last turn
    int bad;                               // an offset pair is impossible
    int abort;
    int kb_max;                            // K-blocks of the longest tile
    int whole, wave, range;                // whole tiles; steps of the last wave, of a range of it
    long long base;                        // first step of the last wave
    long long scan[2][16];
    int off[kMaxExperts + 1];              // the offsets (checked where a group has tiles)
    int tile0[kMaxExperts + 1];            // first tile (of the first M tile column) of each group
    long long step0[kMaxExperts + 1];      // K-block steps before each group
};
constexpr int kSharedBytes = (sizeof(Shared) + 127) / 128 * 128;

template <class C>
constexpr int fixed_smem() { return 1024 + kSharedBytes + C::kScaleBytes + C::kStoreStage; }
template <class C>
constexpr int stage_count() {
    return std::min(kMaxStages, (kSmemMax - fixed_smem<C>()) / C::kStage);
}

// A piece of work: K-blocks [kb0, kb1) of one tile.
struct Piece {
    int e, m0;           // expert; first M row of this CTA
    int row0, rows;      // the tile's rows; kDw: the group's
    int col0;            // kDw, kFwdRows: first column
    int n;               // valid columns of the MMA N dimension
    int kb0, kb1, kb;    // of kb
    int step;            // of the tile's first K-block in the last wave's sequence
};

// The sequence of pieces of one CTA (of a pair, CTAS = 2: both CTAs walk the
// same tiles, each with its own M rows); every role walks its own copy.  Tiles
// and the steps of one wave fit 32 bits for every size the host lets through
// (R at most 2^24, M and the columns at most 2^16); step0 counts in 64.
template <int MODE, class C>
struct Walk {
    const MmArgs& a;
    const Shared& s;
    int tile;        // next of the tiles dealt whole
    int cur, end;    // next step and end of this worker's range of the last wave

    static __device__ __forceinline__ int worker() { return blockIdx.x / C::CTAS; }
    static __device__ __forceinline__ int workers() { return gridDim.x / C::CTAS; }
    static __device__ __forceinline__ int rank() { return blockIdx.x % C::CTAS; }
    // tiles of one group (kDw) or of one row tile of it
    static __device__ __forceinline__ int m_tiles(const MmArgs& a) {
        const int per = C::kRows ? C::BN : kBM * C::CTAS;
        return (a.M + per - 1) / per;
    }
    static __device__ __forceinline__ int c_tiles(const MmArgs& a) {
        return MODE == kDw ? (a.cols + C::BN - 1) / C::BN : 1;
    }
    // rows of a row tile, at most
    static constexpr int kTileRows = C::kRows ? kBM * C::CTAS : C::BN;
    static __device__ __forceinline__ int group_kb(const MmArgs& a, const Shared& s, int e) {
        if (MODE != kDw) return (a.red + C::BK - 1) / C::BK;
        const int rows = s.off[e + 1] - s.off[e];
        return max(1, (rows + C::BK - 1) / C::BK);
    }
    // The last group with first[e] * per <= v.
    template <typename T>
    static __device__ __forceinline__ int group_of(const T* first, long long per, long long v, int E) {
        int lo = 0, hi = E;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (first[mid] * per <= v) lo = mid;
            else hi = mid;
        }
        return lo;
    }
    // Where the whole tiles end and how the last wave is cut (one thread).
    static __device__ __forceinline__ void plan(const MmArgs& a, Shared& s) {
        const long long per = (long long)m_tiles(a) * c_tiles(a);
        const long long tiles = s.tile0[a.E] * per, steps = s.step0[a.E] * per;
        const long long full = tiles - tiles % workers();
        long long base = steps;
        if (full < tiles) {
            const int e = group_of(s.tile0, per, full, a.E);
            base = s.step0[e] * per + (full - s.tile0[e] * per) * group_kb(a, s, e);
        }
        const int wave = (int)(steps - base);
        const int range = max(kMinRange, (wave + workers() - 1) / workers());
        const bool cut = s.kb_max > range + C::kCutCost;
        s.whole = (int)(cut ? full : tiles);
        s.base = base;
        s.wave = cut ? wave : 0;
        s.range = range;
    }
    __device__ __forceinline__ Walk(const MmArgs& a_, const Shared& s_) : a(a_), s(s_) {
        tile = worker();
        cur = (int)min((long long)s.wave, (long long)s.range * worker());
        end = min(s.wave, cur + s.range);
    }
    __device__ __forceinline__ void fill(Piece& p, int e, int t, int kb) const {
        const int off = s.off[e], rows = s.off[e + 1] - off;
        p.e = e;
        p.kb = kb;
        if (MODE == kDw) {
            const int ct = c_tiles(a);
            p.m0 = (t / ct * C::CTAS + rank()) * kBM;
            p.col0 = t % ct * C::BN;
            p.n = min(C::BN, a.cols - p.col0);
            p.row0 = off;
            p.rows = rows;
        } else {
            // bands of kBand row tiles, the row tiles of a band fastest: what
            // the workers have in hand at a time is few strips of both operands
            const int nt = s.tile0[e + 1] - s.tile0[e], mt = m_tiles(a);
            const int band = t / (kBand * mt), in = t - band * kBand * mt;
            const int bw = min(kBand, nt - band * kBand);
            const int ti = band * kBand + in % bw, tm = in / bw;
            if (C::kRows) {
                const int i = (ti * C::CTAS + rank()) * kBM;
                p.row0 = off + i;
                p.rows = max(0, min(kBM, rows - i));
                p.m0 = 0;
                p.col0 = tm * C::BN;
                p.n = min(C::BN, a.M - p.col0);
            } else {
                // a group's rows are shared evenly by its row tiles (16-row grain)
                const int bn = ((rows + nt - 1) / nt + 15) & ~15, i = ti * bn;
                p.m0 = (tm * C::CTAS + rank()) * kBM;
                p.col0 = 0;
                p.row0 = off + i;
                p.rows = p.n = max(0, min(bn, rows - i));
            }
        }
    }
    __device__ __forceinline__ bool next(Piece& p) {
        const long long per = (long long)m_tiles(a) * c_tiles(a);
        if (tile < s.whole) {
            const int e = group_of(s.tile0, per, tile, a.E), kb = group_kb(a, s, e);
            fill(p, e, (int)(tile - s.tile0[e] * per), kb);
            p.kb0 = 0;
            p.kb1 = kb;
            p.step = 0;
            tile += workers();
            return true;
        }
        if (cur >= end) return false;
        const long long at = s.base + cur;
        const int e = group_of(s.step0, per, at, a.E), kb = group_kb(a, s, e);
        const long long in = at - s.step0[e] * per;
        const int t = (int)(in / kb);
        fill(p, e, t, kb);
        p.kb0 = (int)(in - (long long)t * kb);
        p.kb1 = min(kb, p.kb0 + (end - cur));
        p.step = cur - p.kb0;
        cur += p.kb1 - p.kb0;
        return true;
    }
};

// K-blocks of one handover from the MMAs to the epilogue, of n.  bf16: one
// accumulator chain, as few as possible and of equal lengths (a short one behind
// a long one would leave the drain no time).  e4m3: kBatch K-blocks, each with
// its own accumulator.
template <class C, bool FP8>
__device__ __forceinline__ int chain_len(int n) {
    if (FP8) return C::kBatch;
    const int chains = (n + kChunk - 1) / kChunk;
    return (n + chains - 1) / chains;
}

// Columns of the MMA: the valid ones rounded up to its grain.
template <class C>
__device__ __forceinline__ int mma_n(int n) {
    return (max(n, 1) + C::kNGrain - 1) / C::kNGrain * C::kNGrain;
}

// Add one accumulator's columns (times their scales: `one` for all, and where
// there are some `sc` per column) to a thread's sums, and call `release` once they are all loaded.
// The loads of 16 columns run under the sums of the 16 before; a whole tile's
// loop has no branches, so its instructions interleave.
template <class C, bool FP8, bool WHOLE, class Release>
__device__ __forceinline__ void drain(uint32_t src, const float* sc, float one, int nc,
                                      float (&acc)[C::kAcc], Release release) {
    constexpr int kGroups = C::kAcc / 16;
    uint32_t v[2][16];
    tc::ld16(src, v[0]);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        if (!WHOLE && g * 16 >= nc) break;
        float4 f[4];
        if constexpr (C::kColScale) {
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = reinterpret_cast<const float4*>(sc + g * 16)[j];
        }
        uint32_t(&w)[16] = v[g & 1];
        tc::ld_wait(w);
        if (g + 1 < kGroups && (WHOLE || (g + 1) * 16 < nc))
            tc::ld16(src + (g + 1) * 16, v[(g + 1) & 1]);
        else
            release();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float* d = acc + g * 16 + 4 * j;
            if constexpr (C::kRows) {
                tc::fma2(d, w + 4 * j, one);
                tc::fma2(d + 2, w + 4 * j + 2, one);
            } else if constexpr (C::kColScale) {
                d[0] += __uint_as_float(w[4 * j]) * (f[j].x * one);
                d[1] += __uint_as_float(w[4 * j + 1]) * (f[j].y * one);
                d[2] += __uint_as_float(w[4 * j + 2]) * (f[j].z * one);
                d[3] += __uint_as_float(w[4 * j + 3]) * (f[j].w * one);
            } else {
                d[0] += __uint_as_float(w[4 * j]);
                d[1] += __uint_as_float(w[4 * j + 1]);
                d[2] += __uint_as_float(w[4 * j + 2]);
                d[3] += __uint_as_float(w[4 * j + 3]);
            }
        }
    }
}

template <int MODE, bool FP8, int BN_, int CTAS_>
__global__ void __launch_bounds__(Cfg<MODE, FP8, BN_, CTAS_>::kThreads, 1)
grouped_mm_kernel(const __grid_constant__ Maps maps, const MmArgs a) {
    using C = Cfg<MODE, FP8, BN_, CTAS_>;
    constexpr int kStages = stage_count<C>();
    constexpr int CTAS = C::CTAS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* stage0 = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* store0 = stage0 + (size_t)kStages * C::kStage;
    float* scale0 = reinterpret_cast<float*>(store0 + C::kStoreStage);
    Shared& s = *reinterpret_cast<Shared*>(store0 + C::kStoreStage + C::kScaleBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CTAS == 2 ? tc::cta_rank() : 0;
    volatile int* abort = &s.abort;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            // (an arrival that never comes withholds the stage)
            mbar_init(&s.full[i], i == 0 && blockIdx.x == 0 && a.withhold ? 2 : 1);
            mbar_init(&s.empty[i], 1);
            mbar_init(&s.tail_full[i], 1);
            mbar_init(&s.tail_ready[i], CTAS);
        }
        for (int i = 0; i < C::kBufs; ++i) {
            mbar_init(&s.acc_full[i], 1);
            mbar_init(&s.acc_empty[i], kEpiWarps * CTAS);
        }
        for (int i = 0; i < kScaleBufs; ++i) {
            mbar_init(&s.sc_full[i], 32);  // one arrival per copying lane
            mbar_init(&s.sc_empty[i], kEpiWarps);
        }
        mbar_init(&s.mma_done, 1);
        s.loaded = 0;
        s.bad = 0;
        s.abort = 0;
        s.kb_max = MODE == kDw ? 0 : (a.red + C::BK - 1) / C::BK;
        fence_barrier_init();
    }
    if (warp == 1) tc::alloc<CTAS>(&s.tmem, kTmemAll);
    if (threadIdx.x == 0) {
        tc::prefetch_map(&maps.a[0]);
        tc::prefetch_map(&maps.b[0]);
    }
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait();

    // Tiles and K-block steps before each group (of one M tile): a scan over
    // the groups, kPer per thread.  An impossible offset pair is reported and
    // gets no tile.
    auto group_tiles = [&](int rows) -> long long {
        constexpr int kTileRows = Walk<MODE, C>::kTileRows;
        return MODE == kDw ? 1 : (rows + kTileRows - 1) / kTileRows;
    };
    auto tile_kb = [&](int rows) {
        return MODE == kDw ? max(1, (rows + C::BK - 1) / C::BK) : (a.red + C::BK - 1) / C::BK;
    };
    {
        constexpr int kPer = (kMaxExperts + 1 + C::kThreads - 1) / C::kThreads;
        long long v[kPer], w[kPer], sum_v = 0, sum_w = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = threadIdx.x * kPer + i;
            v[i] = w[i] = 0;
            if (e < a.E) {
                const int lo = __ldg(a.offsets + e), hi = __ldg(a.offsets + e + 1);
                s.off[e] = lo;
                if (e + 1 == a.E) s.off[e + 1] = hi;
                if (lo < 0 || hi < lo || hi > a.R) {
                    report(a.status, COLI_ERR_BAD_INDEX);
                    s.bad = 1;
                } else {
                    v[i] = group_tiles(hi - lo);
                    w[i] = v[i] * tile_kb(hi - lo);
                    if (MODE == kDw) atomicMax(&s.kb_max, (int)w[i]);
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
        for (int i = 0; i < kPer; ++i) {
            const int e = threadIdx.x * kPer + i;
            if (e <= a.E) {
                s.tile0[e] = (int)bv;
                s.step0[e] = bw;
            }
            bv += v[i];
            bw += w[i];
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        // Behind a pair that descends, a group may start inside an earlier one: it
        // gets no tile either, or both would write its rows.  (Rare enough for one
        // thread.)
        if (s.bad) {
            long long tiles = 0, steps = 0;
            int end = 0;
            for (int e = 0; e < a.E; ++e) {
                const int lo = s.off[e], hi = s.off[e + 1];
                s.tile0[e] = (int)tiles;
                s.step0[e] = steps;
                if (lo < end || hi < lo || hi > a.R) continue;
                end = hi;
                tiles += group_tiles(hi - lo);
                steps += group_tiles(hi - lo) * tile_kb(hi - lo);
            }
            s.tile0[a.E] = (int)tiles;
            s.step0[a.E] = steps;
        }
        Walk<MODE, C>::plan(a, s);
    }
    tc::fence_before();
    __syncthreads();
    if constexpr (CTAS == 2) tc::cluster_sync();  // the pair's barriers are ready
    tc::fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&s.tmem);

    auto stage_ptr = [&](int i) { return stage0 + (size_t)i * C::kStage; };
    auto timeout = [&]() {
        report(a.status, COLI_ERR_TIMEOUT);
        *abort = 1;
    };
    // one answer for a whole warp
    auto warp_aborted = [&]() { return __shfl_sync(0xffffffffu, (int)*abort, 0) != 0; };
    Walk<MODE, C> walk(a, s);
    Piece p = {};

    if (warp < C::kFront) {
        if constexpr (C::kSplitRegs) tc::regs_dec<C::kFrontRegs>();
        if (warp == 0) {
            // ------------------------------ loads --------------------------------
            if (lane == 0) {
                uint32_t it = 0;
                uint32_t tails = 0;   // parity of the next use of each stage's tail barrier
                int last_tail = -1;
                // rows of B (kDw: columns, in runs of 64) that CTA `r` of the pair
                // loads, in boxes
                auto boxes_of = [&](int r) {
                    const int half = mma_n<C>(p.n) / CTAS;
                    const int n = max(0, min(half, p.n - r * half));
                    return MODE == kDw ? (n + 63) / 64 : (n + C::kBoxRows - 1) / C::kBoxRows;
                };
                auto bytes_of = [&](int boxes) {
                    return (uint32_t)(kABytes + boxes * (MODE == kDw ? 64 : C::kBoxRows) * kRowBytes);
                };
                // One thread runs this for every K-block, so the loop keeps to what
                // changes: the stage, its barriers' addresses, the coordinates.
                const uint32_t empty0 = smem_addr(&s.empty[0]), full0 = smem_addr(&s.full[0]);
                const uint32_t tail0 = smem_addr(&s.tail_full[0]);
                const uint32_t load0 = CTAS == 2 ? tc::cluster_addr(&s.full[0], 0) : full0;
                const uint32_t tload0 = CTAS == 2 ? tc::cluster_addr(&s.tail_full[0], rank) : tail0;
                const uint32_t data0 = smem_addr(stage0);
                uint32_t stage = 0, free = 1;  // parity of the stage's last release
                while (!*abort && walk.next(p)) {
                    if (MODE == kDw && p.rows == 0) continue;  // nothing to add up
                    const int boxes = boxes_of(rank);
                    const uint32_t bytes = bytes_of(boxes);
                    const uint32_t all =
                        CTAS == 2 ? bytes + bytes_of(boxes_of(1 - rank)) : bytes;
                    const int b0 = rank * (mma_n<C>(p.n) / CTAS);  // first column of this CTA
                    const CUtensorMap* bmap = &maps.b[MODE == kDw ? 0 : max(boxes, 1) - 1];
                    bool ok = true;
                    int k = p.kb0 * C::BK;
                    for (int kb = p.kb0; kb < p.kb1; ++kb, k += C::BK) {
                        if (!tc::wait(empty0 + stage * 8, free, a.wait_ns)) {
                            timeout();
                            ok = false;
                            break;
                        }
                        const uint32_t sa = data0 + stage * C::kStage, sb = sa + kABytes;
                        // copies complete on the barrier of the CTA that issues the
                        // MMAs; those of a group's cut last K-block on each CTA's own
                        // tail barrier, for the warp that clears rows of it
                        uint32_t bar = load0 + stage * 8;
                        if (MODE == kDw && p.rows - k < C::BK) {
                            if (rank == 0) tc::arrive(full0 + stage * 8);
                            tc::expect(tail0 + stage * 8, bytes);
                            bar = tload0 + stage * 8;
                            tails ^= 1u << stage;
                            last_tail = stage;
                        } else if (rank == 0) {
                            tc::expect(full0 + stage * 8, all);
                        }
                        if constexpr (MODE == kFwd) {
                            tc::tma_3d<CTAS>(sa, &maps.a[0], k, p.m0, p.e, bar);
                        } else if constexpr (C::kRows) {
                            tc::tma_2d<CTAS>(sa, &maps.a[0], k, p.row0, bar);
                        } else if constexpr (MODE == kDx) {
                            if (a.a_wide) {
                                tc::tma_4d<CTAS>(sa, &maps.a[1], 0, k, p.m0 / 64, p.e, bar);
                            } else {
                                tc::tma_3d<CTAS>(sa, &maps.a[0], p.m0, k, p.e, bar);
                                tc::tma_3d<CTAS>(sa + kABytes / 2, &maps.a[0], p.m0 + 64, k, p.e,
                                                 bar);
                            }
                        } else if (a.a_wide) {
                            tc::tma_3d<CTAS>(sa, &maps.a[1], 0, p.row0 + k, p.m0 / 64, bar);
                        } else {
                            tc::tma_2d<CTAS>(sa, &maps.a[0], p.m0, p.row0 + k, bar);
                            tc::tma_2d<CTAS>(sa + kABytes / 2, &maps.a[0], p.m0 + 64, p.row0 + k,
                                             bar);
                        }
                        if constexpr (MODE == kDw) {
                            // (a cut last tile's parts need not start at a run of 64)
                            if (a.b_wide && p.n == C::BN)
                                tc::tma_3d<CTAS>(sb, &maps.b[1], 0, p.row0 + k,
                                                 (p.col0 + b0) / 64, bar);
                            else
                                for (int b = 0; b < boxes; ++b)
                                    tc::tma_2d<CTAS>(sb + b * 64 * kRowBytes, bmap,
                                                     p.col0 + b0 + b * 64, p.row0 + k, bar);
                        } else if (boxes > 0) {
                            if constexpr (C::kRows)
                                tc::tma_3d<CTAS>(sb, bmap, k, p.col0 + b0, p.e, bar);
                            else
                                tc::tma_2d<CTAS>(sb, bmap, k, p.row0 + b0, bar);
                        }
                        ++it;
                        if (++stage == kStages) {
                            stage = 0;
                            free ^= 1;
                            if (MODE == kDw) *const_cast<volatile uint32_t*>(&s.loaded) = it;
                        }
                    }
                    if (!ok) break;
                }
                // Whoever consumes the stages may give up at any time: the copies in
                // flight end before this CTA does (those of the odd CTA complete on
                // the even one's barriers, and a pair ends together).
                if (rank == 0)
                    for (uint32_t j = it > kStages ? it - kStages : 0; j < it; ++j)
                        tc::wait(full0 + j % kStages * 8, (j / kStages) & 1, a.wait_ns);
                if (last_tail >= 0)
                    tc::wait(tail0 + last_tail * 8, (tails >> last_tail & 1) ^ 1, a.wait_ns);
                if (CTAS == 2 && *abort) {
                    // the other CTA may have filled a stage that this one did not
                    // arm: time enough for a stage's copies to land
                    const uint64_t t0 = global_timer_ns();
                    while (global_timer_ns() - t0 < kSettleNs) __nanosleep(1000);
                }
            }
        } else if (warp == 1) {
            // ------------------------------- MMAs --------------------------------
            // One thread, for every K-block: wait, four MMAs, one or two commits.
            // (By a whole warp, with stages found by division, this loop took 0.46 us
            // a K-block whatever its size, more than the MMAs.)
            if (rank == 0 && lane == 0) {
                constexpr uint32_t kAStep = C::kAMn ? 2048 / 16 : 2;  // along the reduction
                constexpr uint32_t kBStep = C::kBMn ? 2048 / 16 : 2;
                const uint64_t ad0 =
                    tc::desc_at(C::kAMn ? tc::desc_base(64 * kRowBytes, 1024) : tc::desc_base(0, 1024),
                                smem_addr(stage0));
                const uint64_t bd0 =
                    tc::desc_at(C::kBMn ? tc::desc_base(64 * kRowBytes, 1024) : tc::desc_base(0, 1024),
                                smem_addr(stage0) + kABytes);
                const uint32_t full0 = smem_addr(&s.full[0]), empty0 = smem_addr(&s.empty[0]);
                const uint32_t ready0 = smem_addr(&s.tail_ready[0]);
                const uint32_t afull0 = smem_addr(&s.acc_full[0]);
                const uint32_t aempty0 = smem_addr(&s.acc_empty[0]);
                uint32_t stage = 0, full = 0;    // parity of the stage's next filling
                uint32_t buf = 0, drained = 1;   // parity of the accumulator's last release
                uint32_t tails = 0;              // parity of each stage's next cut last K-block
                Piece nxt = {};
                bool more = walk.next(nxt);
                while (!*abort && more) {
                    p = nxt;
                    bool looked = false;  // the next piece is looked up under this one's MMAs
                    if (MODE == kDw && p.rows == 0) {
                        more = walk.next(nxt);
                        continue;
                    }
                    const uint32_t id =
                        tc::idesc(kBM * CTAS, mma_n<C>(p.n), FP8 ? 0 : 1, C::kAMn, C::kBMn);
                    const int len = chain_len<C, FP8>(p.kb1 - p.kb0);
                    for (int c0 = p.kb0; c0 < p.kb1; c0 += len) {
                        const int c1 = min(c0 + len, p.kb1);
                        if (!tc::wait(aempty0 + buf * 8, drained, a.wait_ns)) goto gave_up;
                        for (int kb = c0; kb < c1; ++kb) {
                            const uint32_t d =
                                tmem + (buf * C::kBatch + (C::kBatch > 1 ? kb - c0 : 0)) * C::BN;
                            if (!tc::wait(full0 + stage * 8, full, a.wait_ns)) goto gave_up;
                            const uint64_t ad = ad0 + stage * (C::kStage / 16);
                            const uint64_t bd = bd0 + stage * (C::kStage / 16);
                            if (MODE == kDw && p.rows - kb * C::BK < C::BK) {
                                // a group's cut last K-block: whole MMA steps behind its
                                // end are left out, warp 2 clears the rest of the last
                                if (!tc::wait_cluster(ready0 + stage * 8, tails >> stage & 1,
                                                      a.wait_ns))
                                    goto gave_up;
                                tails ^= 1u << stage;
                                tc::fence_after();
                                const int steps = (p.rows - kb * C::BK + 15) / 16;
                                for (int k = 0; k < steps; ++k)
                                    tc::mma<FP8, CTAS>(d, ad + k * kAStep, bd + k * kBStep, id,
                                                       kb > c0 || k > 0);
                            } else {
                                tc::fence_after();
                                tc::mma<FP8, CTAS>(d, ad, bd, id, !FP8 && kb > c0);
#pragma unroll
                                for (int k = 1; k < 4; ++k)
                                    tc::mma<FP8, CTAS>(d, ad + k * kAStep, bd + k * kBStep, id, 1);
                            }
                            tc::commit<CTAS>(empty0 + stage * 8);
                            if (++stage == kStages) {
                                stage = 0;
                                full ^= 1;
                            }
                        }
                        tc::commit<CTAS>(afull0 + buf * 8);
                        buf = buf + 1 == C::kBufs ? 0 : buf + 1;
                        drained ^= buf == 0;
                        if (!looked) {
                            more = walk.next(nxt);
                            looked = true;
                        }
                    }
                    continue;
                gave_up:  // no stage or accumulator of a failed wait is passed on
                    timeout();
                    break;
                }
                // after a timeout nobody waits for the last MMAs: they end before
                // tensor memory is freed
                if (*abort) {
                    tc::commit_here<CTAS>(smem_addr(&s.mma_done));
                    tc::wait(smem_addr(&s.mma_done), 0, a.wait_ns);
                }
            }
        } else if (MODE == kDw && warp == 2) {
            // ------ kDw: clear what lies behind a group's end in its last K-block ------
            // (rows of the next group, in both operands: they may hold infinities), up
            // to the next MMA step.  In a pair each CTA clears its own part.  Groups of
            // whole K-blocks need none, so a wait can span the work of many tiles: its
            // limit starts again whenever the loads go on.
            uint32_t it = 0, tails = 0;
            while (!warp_aborted() && walk.next(p)) {
                if (p.rows == 0) continue;
                it += p.kb1 - p.kb0;
                const int valid = p.rows - (p.kb1 - 1) * C::BK;
                if (valid >= C::BK) continue;
                const int i = (it - 1) % kStages;
                bool ok = tc::wait_warp(&s.tail_full[i], tails >> i & 1, a.wait_ns);
                for (uint32_t seen = 0; !ok;) {
                    const uint32_t now = __shfl_sync(
                        0xffffffffu, *const_cast<volatile uint32_t*>(&s.loaded), 0);
                    if (now == seen || warp_aborted()) break;
                    seen = now;
                    ok = tc::wait_warp(&s.tail_full[i], tails >> i & 1, a.wait_ns);
                }
                if (!ok) {
                    if (lane == 0) timeout();
                    break;
                }
                tails ^= 1u << i;
                const int half = mma_n<C>(p.n) / CTAS;
                const int n = max(0, min(half, p.n - (int)rank * half));
                const int boxes = 2 + (n + 63) / 64;
                const int chunks = ((valid + 15) / 16 * 16 - valid) * 8;
                for (int b = 0; b < boxes; ++b)
                    for (int j = lane; j < chunks; j += 32)
                        *reinterpret_cast<uint4*>(stage_ptr(i) + b * 64 * kRowBytes +
                                                  valid * kRowBytes + j * 16) =
                            make_uint4(0, 0, 0, 0);
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) {
                    if (CTAS == 2)
                        tc::arrive_release_cluster(tc::cluster_addr(&s.tail_ready[i], 0));
                    else mbar_arrive(&s.tail_ready[i]);
                }
            }
        } else if constexpr (C::kColScale) {
            // ----------- fp8: the rows' scales (one per column) and the weights' ----------
            // Copied ahead (cp.async), kScaleBufs handovers; a K-block's slot holds the
            // columns' scales and, behind them, the weights' scale.
            if (warp == 2) {
                const int KB = (a.red + C::BK - 1) / C::BK;
                const int w_tiles = (a.M + kBM - 1) / kBM;
                uint32_t ch = 0;
                while (!warp_aborted() && walk.next(p)) {
                    // (an odd CTA past the last weight rows computes nothing that is stored)
                    const int wt = min(p.m0 / kBM, w_tiles - 1);
                    const float* wsc = a.ws + ((int64_t)p.e * w_tiles + wt) * KB + p.kb0;
                    const float* xs = a.xs + (int64_t)p.kb0 * a.R + p.row0;
                    bool ok = true;
                    for (int k0 = p.kb0; k0 < p.kb1; k0 += C::kBatch, ++ch) {
                        const uint32_t b = ch % kScaleBufs;
                        if (!tc::wait_warp(&s.sc_empty[b], (ch / kScaleBufs & 1) ^ 1, a.wait_ns)) {
                            if (lane == 0) timeout();
                            ok = false;
                            break;
                        }
                        float* slot = scale0 + b * (C::kBatch * C::kScaleSlot);
                        const int n = min(C::kBatch, p.kb1 - k0);
                        for (int k = 0; k < n; ++k, ++wsc, xs += a.R, slot += C::kScaleSlot) {
#pragma unroll
                            for (int j = lane; j < C::BN; j += 32)
                                if (j < p.n) cp_async4(slot + j, xs + j);
                            if (lane == 0) cp_async4(slot + C::BN, wsc);
                        }
                        tc::cp_async_arrive(&s.sc_full[b]);
                    }
                    if (!ok) break;
                }
                tc::cp_async_wait<0>();
            }
        }
    } else {
        // ------------------------------ epilogue ---------------------------------
        if constexpr (C::kSplitRegs) tc::regs_inc<C::kEpiRegs>();
        const int q = warp & 3, half = (warp - C::kFront) >> 2;
        const int mrow = q * 32 + lane;       // row of this CTA's part of the tile
        uint8_t* stage_out = store0 + (warp - C::kFront) * kStoreBufs * kStoreBytes;
        int store_buf = 0;
        const uint32_t acc_empty =
            CTAS == 2 ? tc::cluster_addr(&s.acc_empty[0], 0) : smem_addr(&s.acc_empty[0]);
        uint32_t ch = 0;
        // (whoever gave up ends this loop too: the next accumulator does not come)
        while (walk.next(p)) {
            // the two warps of a lane quarter share the columns evenly
            // (kFwdRows: the columns of one weight scale each)
            const int hn = C::kRows ? 128 : (p.n + 63) / 64 * 32;
            const int c0 = half * hn;                       // first column of this thread
            const int nc = max(0, min(p.n - c0, hn));       // and how many
            const uint32_t tq = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)c0;
            float acc[C::kAcc];
#pragma unroll
            for (int j = 0; j < C::kAcc; ++j) acc[j] = 0.f;
            bool ok = true;
            if (MODE == kDw && p.rows == 0) {
                if (a.accumulate) continue;  // nothing to add
            } else {
                // kFwdRows: this thread's row has one scale per K-block, its columns
                // one weight scale.  Each thread copies its own two numbers into its
                // own ring in shared memory, kScaleRing - 1 K-blocks ahead.
                const float *xs = nullptr, *wsc = nullptr;
                float2* ring = reinterpret_cast<float2*>(scale0) + (threadIdx.x - C::kFront * 32);
                auto fetch = [&](int i) {
                    if (xs && i < p.kb1 - p.kb0) {
                        float2* slot = ring + (i & (kScaleRing - 1)) * (kEpiWarps * 32);
                        cp_async4(&slot->x, xs + (int64_t)i * a.R);
                        cp_async4(&slot->y, wsc + i);
                    }
                    cp_async_commit();
                };
                if constexpr (C::kRows) {
                    if (mrow < p.rows && nc > 0) {
                        xs = a.xs + (int64_t)p.kb0 * a.R + p.row0 + mrow;
                        wsc = a.ws +
                              ((int64_t)p.e * ((a.M + 127) / 128) + (p.col0 + c0) / 128) * p.kb +
                              p.kb0;
                    }
                    for (int i = 0; i < kScaleRing - 1; ++i) fetch(i);
                }
                const int len = chain_len<C, FP8>(p.kb1 - p.kb0);
                const int n_ch = (p.kb1 - p.kb0 + len - 1) / len;
                for (int i = 0; i < n_ch; ++i, ++ch) {
                    const uint32_t buf = ch % C::kBufs, sb = ch % kScaleBufs;
                    // what does not need the accumulator stays out of the way from
                    // one accumulator's MMAs over its drain to the next one's
                    float one = 0.f;
                    if constexpr (C::kRows) {
                        tc::cp_async_wait<kScaleRing - 2>();
                        const float2 f = ring[(i & (kScaleRing - 1)) * (kEpiWarps * 32)];
                        one = f.x * f.y;
                    }
                    if (!tc::wait_warp(&s.acc_full[buf], (ch / C::kBufs) & 1, a.wait_ns) ||
                        (C::kColScale &&
                         !tc::wait_warp(&s.sc_full[sb], (ch / kScaleBufs) & 1, a.wait_ns))) {
                        if (lane == 0) timeout();
                        ok = false;
                        break;
                    }
                    tc::fence_after();
                    const uint32_t src = tq + buf * (C::kBatch * C::BN);
                    const float* sc = scale0 + sb * (C::kBatch * C::kScaleSlot);
                    auto release = [&]() {
                        tc::fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            if (CTAS == 2) tc::arrive_cluster(acc_empty + buf * 8);
                            else tc::arrive(acc_empty + buf * 8);
                            if (C::kColScale) mbar_arrive(&s.sc_empty[sb]);
                        }
                    };
                    if constexpr (C::kColScale) {
                        const int n = min(C::kBatch, p.kb1 - p.kb0 - i * len);
                        if (nc > 0) {
#pragma unroll
                            for (int k = 0; k < C::kBatch; ++k)
                                if (k < n)
                                    drain<C, FP8, false>(src + k * C::BN, sc + k * C::kScaleSlot + c0,
                                                         sc[k * C::kScaleSlot + C::BN], nc, acc,
                                                         [] {});
                        }
                        release();
                    } else {
                        if (nc == C::kAcc) drain<C, FP8, true>(src, sc, one, nc, acc, release);
                        else if (nc > 0) drain<C, FP8, false>(src, sc, one, nc, acc, release);
                        else release();
                    }
                    if constexpr (C::kRows) fetch(i + kScaleRing - 1);
                }
            }
            if (!ok) break;

            if (p.kb1 - p.kb0 < p.kb) {
                // a cut tile: leave the partial sums; the last of its ranges adds
                // them, in the order of the ranges.  Each warp reads only what the
                // same warp of another CTA left, so it counts and goes on by itself.
                if (nc == 0) continue;
                const int c_first = p.step / s.range;
                const int c_last = (p.step + p.kb - 1) / s.range;
                constexpr int kPart = kBM * C::BN;
                auto part_of = [&](int worker, bool head) {
                    return a.part + (((int64_t)worker * 2 + head) * CTAS + rank) * kPart +
                           c0 * kBM + mrow;
                };
                float* mine = part_of(walk.worker(), p.kb0 == 0);
#pragma unroll
                for (int j = 0; j < C::kAcc; ++j)
                    if (j < nc) __stcg(mine + j * kBM, acc[j]);
                __threadfence();
                __syncwarp();
                int last = 0;
                if (lane == 0) {
                    int* count = a.counters + (c_first * CTAS + rank) * kEpiWarps + warp - C::kFront;
                    last = atomicAdd(count, 1) == c_last - c_first;
                    if (last) *count = 0;
                }
                if (!__shfl_sync(0xffffffffu, last, 0)) continue;
                __threadfence();
#pragma unroll
                for (int j = 0; j < C::kAcc; ++j) acc[j] = 0.f;
                // as many loads in flight as registers allow: wide tiles 32 columns
                // of a part at a time, narrow ones 8 columns of 8 parts (the padding
                // behind the last column is read too)
                constexpr int kCols = C::kAcc > 64 ? 32 : 8, kParts = C::kAcc > 64 ? 1 : 8;
#pragma unroll 1
                for (int c = c_first; c <= c_last; c += kParts) {
#pragma unroll
                    for (int j0 = 0; j0 < C::kAcc; j0 += kCols) {
                        if (j0 >= nc) break;
                        float f[kParts][kCols];
#pragma unroll
                        for (int i = 0; i < kParts; ++i) {
                            const float* src = part_of(c + i, c + i == c_first) + j0 * kBM;
#pragma unroll
                            for (int j = 0; j < kCols; ++j)
                                f[i][j] = kParts == 1 || c + i <= c_last ? __ldcg(src + j * kBM)
                                                                         : 0.f;
                        }
#pragma unroll
                        for (int i = 0; i < kParts; ++i)
#pragma unroll
                            for (int j = 0; j < kCols; ++j) acc[j0 + j] += f[i][j];
                    }
                }
            }

            const int m = p.m0 + mrow;
            if constexpr (MODE == kDw) {
                // 32 rows x 64 bytes at a time through shared memory to a tensor
                // store, which leaves out what lies outside dw; up to kStoreBufs of
                // them under way
                if (!(a.accumulate && a.out_bf16)) {
#pragma unroll
                    for (int g = 0; g < C::kAcc / 16; ++g) {
                        // 16 fp32 columns, or 32 bf16 ones of every other group
                        if (g * 16 >= nc || p.m0 + q * 32 >= a.M) break;
                        if (a.out_bf16 && (g & 1)) continue;
                        uint8_t* out = stage_out + store_buf * kStoreBytes;
                        store_buf = store_buf + 1 == kStoreBufs ? 0 : store_buf + 1;
                        if (lane == 0) tc::store_read_wait<kStoreBufs - 1>();
                        __syncwarp();
                        // 64-byte swizzle: rows in pairs of 128 bytes
                        uint8_t* row = out + lane * 64;
                        const int x = (lane >> 1) & 3;
                        if (a.out_bf16) {
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                uint32_t u[4];
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    constexpr int kLast = C::kAcc - 2;
                                    const float* f = acc + min(g * 16 + 8 * j + 2 * i, kLast);
                                    const __nv_bfloat162 h = __floats2bfloat162_rn(f[0], f[1]);
                                    u[i] = *reinterpret_cast<const uint32_t*>(&h);
                                }
                                *reinterpret_cast<uint4*>(row + ((j ^ x) << 4)) =
                                    make_uint4(u[0], u[1], u[2], u[3]);
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                *reinterpret_cast<float4*>(row + ((j ^ x) << 4)) =
                                    make_float4(acc[g * 16 + 4 * j], acc[g * 16 + 4 * j + 1],
                                                acc[g * 16 + 4 * j + 2], acc[g * 16 + 4 * j + 3]);
                        }
                        fence_proxy_async();
                        __syncwarp();
                        if (lane == 0)
                            tc::tma_store_3d(&maps.out, out, p.col0 + c0 + g * 16, p.m0 + q * 32,
                                             p.e, a.accumulate);
                    }
                } else if (m < a.M) {
                    // added to bf16 values: one rounding of the whole sum
                    uint4* dst = reinterpret_cast<uint4*>(
                        static_cast<uint16_t*>(a.out) + ((int64_t)p.e * a.M + m) * a.cols + p.col0 +
                        c0);
#pragma unroll
                    for (int j0 = 0; j0 < C::kAcc; j0 += 8) {
                        if (j0 >= nc) break;  // columns come in whole vectors of 8
                        const uint4 old = dst[j0 / 8];
                        const uint32_t w[4] = {old.x, old.y, old.z, old.w};
                        uint32_t u[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float* f = acc + j0 + 2 * j;
                            const __nv_bfloat162 h = __floats2bfloat162_rn(
                                f[0] + __uint_as_float(w[j] << 16),
                                f[1] + __uint_as_float(w[j] & 0xFFFF0000u));
                            u[j] = *reinterpret_cast<const uint32_t*>(&h);
                        }
                        dst[j0 / 8] = make_uint4(u[0], u[1], u[2], u[3]);
                    }
                }
            } else if constexpr (C::kRows) {
                // a thread's columns are consecutive in its row of the output
                if (mrow < p.rows) {
                    const int64_t o = (int64_t)(p.row0 + mrow) * a.M + p.col0 + c0;
#pragma unroll
                    for (int j0 = 0; j0 < C::kAcc; j0 += 8) {
                        if (j0 >= nc) break;  // columns come in whole vectors of 8
                        const float* f = acc + j0;
                        if (a.out_bf16) {
                            uint32_t u[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const __nv_bfloat162 h =
                                    __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
                                u[j] = *reinterpret_cast<const uint32_t*>(&h);
                            }
                            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + o + j0) =
                                make_uint4(u[0], u[1], u[2], u[3]);
                        } else {
                            float4* dst =
                                reinterpret_cast<float4*>(static_cast<float*>(a.out) + o + j0);
                            dst[0] = make_float4(f[0], f[1], f[2], f[3]);
                            dst[1] = make_float4(f[4], f[5], f[6], f[7]);
                        }
                    }
                }
            } else if (m < a.M) {
                // a warp writes 32 consecutive values of one row at a time
                const int64_t o = (int64_t)(p.row0 + c0) * a.M + m;
                if (a.out_bf16) {
                    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + o;
#pragma unroll
                    for (int j = 0; j < C::kAcc; ++j)
                        if (j < nc) dst[(int64_t)j * a.M] = __float2bfloat16_rn(acc[j]);
                } else {
                    float* dst = static_cast<float*>(a.out) + o;
#pragma unroll
                    for (int j = 0; j < C::kAcc; ++j)
                        if (j < nc) dst[(int64_t)j * a.M] = acc[j];
                }
            }
            __syncwarp();
        }
        if (MODE == kDw && lane == 0) tc::store_wait();
        if constexpr (C::kRows) tc::cp_async_wait<0>();
    }

    __syncwarp();
    tc::fence_before();
    __syncthreads();
    // a pair ends together: the even CTA's MMAs read the odd one's memory, the
    // odd one's epilogue arrives on the even one's barriers
    if constexpr (CTAS == 2) tc::cluster_sync();
    if (warp == 1) {
        tc::fence_after();
        tc::dealloc<CTAS>(tmem, kTmemAll);
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

enum Type { kBytes, kBf16, kF32 };

// A tensor map of `rank` dimensions (strides of all but the first, in bytes),
// boxes with the 128-byte swizzle (or the 64-byte one, for boxes that wide); what
// lies outside reads as zero.
bool encode(CUtensorMap* m, Type type, const void* base, int rank, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box,
            CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint32_t es[4] = {1, 1, 1, 1};
    const CUtensorMapDataType dt = type == kBytes  ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : type == kBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                   : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
    return enc(m, dt, rank, const_cast<void*>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [outer][rows][inner] (outer 0: two dimensions), boxes of 128 (or 64) bytes x
// box_rows.
bool encode_rows(CUtensorMap* m, Type type, const void* base, int inner, int64_t rows, int outer,
                 int box_rows, int box_bytes = kRowBytes) {
    const cuuint64_t size = type == kBytes ? 1 : type == kBf16 ? 2 : 4;
    const cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)rows, (cuuint64_t)outer};
    const cuuint64_t strides[2] = {inner * size, inner * size * (cuuint64_t)rows};
    const cuuint32_t box[3] = {(cuuint32_t)(box_bytes / size), (cuuint32_t)box_rows, 1};
    return encode(m, type, base, outer > 0 ? 3 : 2, dims, strides, box,
                  box_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
}

// The same bf16 array with its rows as runs of 64 columns, [outer][run][rows][64]:
// boxes of 64 rows of two runs, one behind the other.
bool encode_runs(CUtensorMap* m, const void* base, int inner, int64_t rows, int outer) {
    const cuuint64_t dims[4] = {64, (cuuint64_t)rows, (cuuint64_t)inner / 64, (cuuint64_t)outer};
    const cuuint64_t strides[3] = {(cuuint64_t)inner * 2, 128,
                                   (cuuint64_t)inner * 2 * (cuuint64_t)rows};
    const cuuint32_t box[4] = {64, 64, 2, 1};
    return encode(m, kBf16, base, outer > 0 ? 4 : 3, dims, strides, box);
}

template <int MODE, bool FP8, int BN, int CTAS>
coli_status launch_mm(const void* A, const void* B, MmArgs a, int N, int K, cudaStream_t st) {
    using C = Cfg<MODE, FP8, BN, CTAS>;
    const Type in = FP8 ? kBytes : kBf16;
    Maps maps = {};
    bool ok;
    if constexpr (MODE == kDw) {
        a.a_wide = N % 64 == 0;
        a.b_wide = K % 64 == 0;
        ok = encode_rows(&maps.a[0], in, A, N, a.R, 0, 64) &&
             encode_rows(&maps.b[0], in, B, K, a.R, 0, 64) &&
             (!a.a_wide || encode_runs(&maps.a[1], A, N, a.R, 0)) &&
             (!a.b_wide || encode_runs(&maps.b[1], B, K, a.R, 0)) &&
             encode_rows(&maps.out, a.out_bf16 ? kBf16 : kF32, a.out, K, N, a.E, 32, 64);
    } else {
        a.a_wide = MODE == kDx && K % 64 == 0;
        if constexpr (C::kRows)
            ok = encode_rows(&maps.a[0], in, A, K, a.R, 0, kBM);
        else
            ok = encode_rows(&maps.a[0], in, A, K, N, a.E, MODE == kFwd ? kBM : 64) &&
                 (!a.a_wide || encode_runs(&maps.a[1], A, K, N, a.E));
        for (int i = 0; i < C::kBoxes && ok; ++i)
            ok = encode_rows(&maps.b[i], in, B, MODE == kDx ? N : K, C::kRows ? N : a.R,
                             C::kRows ? a.E : 0, (i + 1) * C::kBoxRows);
    }
    if (!ok) return COLI_ERR_CUDA;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return COLI_ERR_CUDA;
    constexpr int smem = fixed_smem<C>() + stage_count<C>() * C::kStage;
    static_assert(smem <= kSmemMax && stage_count<C>() >= 4, "shared memory");
    auto kernel = grouped_mm_kernel<MODE, FP8, BN, CTAS>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
        cudaSuccess)
        return COLI_ERR_CUDA;
    const int grid = std::max(CTAS, std::min(sms, kMaxGrid) / CTAS * CTAS);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CTAS;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CTAS == 2 ? 2 : 1;
    const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, maps, a);
    return err == cudaSuccess ? COLI_OK : COLI_ERR_CUDA;
}

// Narrow row tiles (64 rows, one CTA) where the weights' loads bound the call.
// Measured at N 4096, K 6144, narrow against wide: one group of 64 rows 28.7 and
// 34.8 us, of 128 rows 38.9 (narrow 32.8); 32 groups of 32 rows on average 266 and
// 279 us, of 48 rows 276 and 283, of 64 rows 297 and 285 (e4m3: 156 and 167, 174
// and 170, 195 and 176).
// And where they make a wave at most: wide ones would leave SMs without work (1024
// x 1024 x 1024 narrow 9.7 us, wide 14.7; 2217 rows of 5 groups, N 472, K 1624 14.0
// and 20.3, with more than a wave, for their 1624 columns, 18.1 and 14.5; 2048 x
// 1024 x 2048, 1.7 waves, 23.7 and 20.1).  The host does not know the groups' sizes and
// goes by their average: where one of 128 groups holds all of 4096 rows, the call
// takes 410 us, with wide tiles 157.
bool narrow(int R, int E, int M) {
    const int64_t rows = (int64_t)R + 32 * (int64_t)E;  // half a tile lost per group
    return (int64_t)R <= 48 * (int64_t)E + 16 || rows * ((M + kBM - 1) / kBM) <= 64 * 160;
}

static_assert(sizeof(int) * kMaxGrid * kEpiWarps <= kHeaderBytes - kTileCntOffset, "counters");
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
    const GroupedHook hook = take_grouped_hook();
    a.wait_ns = hook.wait_ns;
    a.withhold = hook.withhold;
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
    return narrow(R, E, N) ? launch_mm<kFwd, false, 64, 1>(w_bf16, x_bf16, a, N, K, st)
                        : launch_mm<kFwd, false, 256, 2>(w_bf16, x_bf16, a, N, K, st);
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
    return narrow(R, E, K) ? launch_mm<kDx, false, 64, 1>(w_bf16, dy_bf16, a, N, K, st)
                        : launch_mm<kDx, false, 256, 2>(w_bf16, dy_bf16, a, N, K, st);
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
    return launch_mm<kDw, false, 256, 2>(dy_bf16, x_bf16, a, N, K, st);
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
    return narrow(R, E, N) ? launch_mm<kFwd, true, 64, 1>(wq, xq, a, N, K, st)
                        : launch_mm<kFwdRows, true, 256, 1>(xq, wq, a, N, K, st);
}

}  // extern "C"
