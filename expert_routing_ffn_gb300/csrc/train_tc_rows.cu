// The experts' products that give grouped rows, on the tensor cores (tcgen05,
// accumulators in tensor memory), fed by TMA.  With x, h, dy, dg, du the
// grouped rows and Wg, Wu, Wd [I, d] an expert's weights:
//   Up    g = x Wg^T, u = x Wu^T       K = d; epilogue h = SiLU(g) u
//   Down  y = h Wd                     K = I
//   Dh    dh = dy Wd^T                 K = d; epilogue dg, du from g, u
//   Dx    dx = dg Wg + du Wu           K = I twice, one accumulator
//
// The weights are the MMA's M side and the rows its N side: a tile is 256
// weight rows (or columns) on a CTA pair (2-CTA MMA, 128 accumulator lanes in
// each CTA) x up to 256 grouped rows.  N goes in steps of 32, so a segment's
// rows are split into nearly equal tiles and a ragged end costs at most 31
// rows, where rows on the M side cost up to 255: 384 rows an expert took 2
// tiles of 256 (DeepSeek-V2-Lite shape, 4096 tokens), a third of the MMA work.
// It also serves a decode-size batch, N = 32, as a pure stream of weights.
//
// The accumulator comes out transposed (a lane is a channel, a column a row of
// the output).  tcgen05.ld in the 16x256b shape hands it out in the layout of
// matrix fragments, and stmatrix with transposition writes it to shared memory
// as rows of 64 channels (128 bytes, swizzled), whence TMA stores it.  In Up
// a CTA's M side is 64 gate rows and 64 up rows; the warps that hold g and
// those that hold u of the same channels swap half of their values through
// shared memory, in fp32.  In Dh g and u come in by TMA and ldmatrix in the
// same layout, and dg, du overwrite them.
//
// PACKED: g and u are rows in 8 bits (the format stands in moe_train.h).  The
// 32 lanes of a warp are one block of 32 channels, so a row's largest magnitude
// takes three shuffles, and a thread's four channels of a row are one word of
// the block: eight threads write (Up) or read (Dh) its 32 bytes straight from
// registers, a whole sector, without shared memory.  Dh fetches a panel's words
// while it waits for the accumulator or works on the panel before, and gives h
// beside dg and du.  4096 tokens of the Qwen2-57B shape, skewed, Up: 0.83-0.88 ms, as
// with g and u in bf16; DeepSeek-V2-Lite shape, Dh: 160 us for 747 MB (without h and
// with g and u in bf16 140 us).
//
// The tiles of all experts form one list (expert by expert, row tiles
// innermost: a weight tile read by several of them comes from L2 after the
// first), taken round robin by the resident pairs; the tiles of the last,
// partial round are cut into parts.
//
// Block: warp 0 issues the TMA loads, warp 1 the MMAs (of the pair's leader),
// both converged with one lane picked for the issue; warps 2-9 the epilogue,
// in panels of 32 rows through a ring of buffers.  Accumulators are
// double-buffered.  Every wait is bounded.
//
// Bound and measurements (GB300; 76 pairs):
//   few rows an expert: HBM reads of the weights.  8 tokens, Mixtral-8x7B
//     shape, Down: 121 us for 846 MB, 1.03 of the measured copy bandwidth.
//   many rows: the tensor pipe at the clock that the power limit leaves.
//     1024 rows an expert, Up at d 4096, I 3584: 313 us, 1.54 PFLOP/s, 0.91 of
//     the measured sustained bf16 rate; 4096 tokens of the Qwen2-57B shape,
//     skewed, Up: 0.88-0.91 ms, 1.32-1.37 PFLOP/s.
//   between: both.  384 rows an expert (DeepSeek-V2-Lite shape, 4096 tokens),
//     Dx: 976 MB and 283 GFLOP take 144 and 146 us at the burst rates; 190 us
//     measured (218 in long runs).  With every load served by L2 it takes 155,
//     without loads 145, without stores 181: what is left is HBM latency beside
//     the stores that six stages do not cover (five: 202 us).
// Tried and left out: copies into L2 ahead of the loads (slower at every
// distance: 190 -> 200 us and worse, the weights came from HBM twice); two pairs
// sharing the rows by multicast (36 clusters of four instead of 76 pairs: no
// faster, though measured while the issue of the MMAs was still the bound);
// tiles of 512 rows over both accumulators, which load a third less but leave the
// epilogue beside no MMA (384 rows an expert, Up: 229 -> 249 us, Dx even); one
// epilogue buffer in Down and Dx (even); L2 policies on the stores (even); boxes
// of 16 rows for a ragged B (a copy costs its issuing warp some 100 cycles
// whatever its size: 247 -> 295 us before the issue was converged).
#include <cuda.h>

#include <array>
#include <cstring>
#include <mutex>
#include <vector>

#include "common.cuh"
#include "pack8.cuh"
#include "tma.h"
#include "train.h"
#include "train_tc.cuh"

namespace moe {

namespace {

using namespace train;

constexpr int kGroups = 2, kGroupThreads = 128;  // epilogue: two groups of four warps
constexpr int kThreads = 64 + kGroups * kGroupThreads;
constexpr int kStepN = 32;     // granularity of N on a CTA pair
constexpr int kPanel = 32;     // rows per epilogue panel
constexpr uint32_t kBK = kTcBK;
constexpr uint32_t kStageA = 128 * kBK * 2;
constexpr uint32_t kBox = kPanel * 128;  // 32 rows x 64 channels
constexpr int kBoxHeights = 8;

// MAXN: the most rows of a tile.
template <int FORM, int MAXN, bool PACKED>
struct Cfg {
    static constexpr bool kNT = FORM == kFormUp || FORM == kFormDh;  // weights K-major
    static constexpr int kChannels = FORM == kFormUp ? 64 : 128;     // output channels of one CTA
    static constexpr int kBoxes = FORM == kFormUp ? (PACKED ? 1 : 3) : FORM == kFormDh ? (PACKED ? 6 : 4) : 2;  // boxes of a panel
    static constexpr uint32_t kStage = kStageA + MAXN / 2 * kBK * 2;
    static constexpr uint32_t kBuffer = kBoxes * kBox;
    // Panel buffers of a group.  Large tiles of Up have one, which costs a barrier a panel and leaves room for a
    // sixth stage: 384 rows an expert (DeepSeek-V2-Lite shape) 239 -> 231 us, 4096 tokens of the Qwen2-57B shape
    // 900 -> 880; 200 rows (Granite shape) 37.4 -> 38.6; 64-row tiles, which have eight stages, 110 -> 112.
    // Dh, PACKED, has six boxes: one buffer and five stages 161 us (384 rows an expert) and 296 (Qwen2-57B shape, 2048
    // tokens), two and four 166 and 329; 64-row tiles 64 against 66.
    static constexpr int kBuffers = PACKED ? (FORM == kFormDh ? 1 : 2) : FORM == kFormUp && MAXN == 256 ? 1 : 2;
    static constexpr uint32_t kSwap = FORM == kFormUp ? kGroupThreads * 32 : 0;  // a group's room to swap values
    static constexpr uint32_t kEpi = kGroups * (kBuffers * kBuffer + kSwap);
    static constexpr int kStages = (int)((224 * 1024 - kEpi) / kStage);
    static constexpr uint32_t kPanels = (kStages * kStage + 1023) / 1024 * 1024;  // epilogue buffers
    static constexpr uint32_t kTable = kPanels + kEpi;
    static constexpr uint32_t kBars = kTable + ((kTrainMaxExperts + 1) * 4 + 15) / 16 * 16;
    static constexpr uint32_t kSmem = kBars + (2 * kStages + 5 + kGroups * kBuffers) * 8 + 16;
    static_assert(kSmem <= 232448, "227 KB of shared memory per block");
};

struct RowsParams {
    CUtensorMap a[2];         // weights
    CUtensorMap b[2][kBoxHeights];  // rows [M, K] in boxes of 16, 32, .. 128 rows
    CUtensorMap in[2];        // Dh: g, u
    CUtensorMap o[3];         // outputs (boxes of 32 rows x 64 channels)
    __nv_bfloat16* out[3];
    int8_t* q[2];             // PACKED: g, u (Up writes them, Dh reads them)
    uint8_t* scale[2];
    const int32_t* offsets;
    int M, N, d, I, nb;       // nb: blocks of a packed row
    DevError* err;
    MapParams dw;             // the maps of the weight gradients that follow this kernel
};

// 1 / (1 + e^-g) = e^g / (1 + e^g), of the two the one whose exponential is
// at most 1: from g = -87.34 on (e^-g past 2^126) the first form is flushed
// to zero, where h, dg and du are still bf16 numbers.  The fast exponential is
// within 2 + 1.173 |g| ulp of float32 (documented), 105 at |g| = 88, and the
// fast division within 2; bf16 rounds at 2^15 ulp.  Below 2^-126 a sigmoid has
// float32's absolute spacing of 2^-149, and below g = -104 it is zero.
__device__ __forceinline__ float fast_sigmoid(float g) {
    const float e = __expf(-fabsf(g));
    return __fdividef(g < 0.f ? e : 1.f, 1.f + e);
}

__device__ __forceinline__ uint32_t pack_f(uint32_t lo, uint32_t hi) {
    return pack_bf16x2(__uint_as_float(lo), __uint_as_float(hi));
}

struct Tile {
    int e, row0, rows, c0;  // expert, first row, rows of the tile, first channel of the pair
};

// The rows of a segment are cut into units of 32 (the last one ragged), the
// units into as few tiles of at most MAXN rows as possible, of sizes that
// differ by one unit at most.
template <int MAXN>
__device__ __forceinline__ int row_tiles(int rows) { return (rows + MAXN - 1) / MAXN; }

// Where the units' whole rounds end, the tiles left over are fewer than the
// units: each is cut into `cut` parts of its rows, so that the last round is
// as short as it can be with one part a unit (its weights come from L2 then).
struct Schedule {
    int whole, cut, total;  // tiles of whole rounds, parts of a later tile, list entries
};
__device__ __forceinline__ Schedule schedule(int n_tiles, int n_units) {
    Schedule s;
    const int left = n_tiles % n_units;
    s.whole = n_tiles - left;
    s.cut = left > 0 ? n_units / left : 1;
    if (s.cut > 8) s.cut = 8;
    s.total = s.whole + left * s.cut;
    return s;
}

// List entry t; rows = 0 for a part that its tile is too short for.
template <int FORM, int MAXN, bool PACKED>
__device__ __forceinline__ Tile decode(const RowsParams& p, const int* first, const Schedule& sc, int t) {
    int part = 0, cut = 1;
    if (t >= sc.whole) {
        cut = sc.cut;
        part = (t - sc.whole) % cut;
        t = sc.whole + (t - sc.whole) / cut;
    }
    int lo = 0, hi = p.N;
    while (hi - lo > 1) {  // the last expert whose tiles start at or before t
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= t) lo = mid;
        else hi = mid;
    }
    const int r0 = min(max(p.offsets[lo], 0), p.M), rows = min(max(p.offsets[lo + 1], 0), p.M) - r0;
    const int mts = row_tiles<MAXN>(rows), units = (rows + kStepN - 1) / kStepN;
    const int local = t - first[lo], c = local / mts, m = local - c * mts;
    const int base = units / mts, more = units - base * mts;          // the first `more` tiles have a unit more
    const int u0 = m * base + min(m, more), nu = base + (m < more);   // this tile's units
    const int a = u0 + part * nu / cut, b = u0 + (part + 1) * nu / cut;
    Tile x;
    x.e = lo;
    x.row0 = r0 + a * kStepN;
    x.rows = min(b * kStepN, rows) - a * kStepN;
    x.c0 = c * 2 * Cfg<FORM, MAXN, PACKED>::kChannels;
    return x;
}

// A panel's g and u in 8 bits, as a thread of the epilogue holds them: its four
// channels of eight rows, and the steps of row `lane`.
struct PackedPanel {
    uint32_t g[8], u[8];
    float sg, su;
};

template <int FORM, int MAXN, bool PACKED>
__global__ void __launch_bounds__(kThreads, 1) grouped_rows_kernel(const __grid_constant__ RowsParams p) {
    using C = Cfg<FORM, MAXN, PACKED>;
    constexpr int kS = C::kStages;
    extern __shared__ __align__(1024) unsigned char smem[];
    int* first = reinterpret_cast<int*>(smem + C::kTable);  // tiles before each expert
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBars);
    uint64_t *empty = full + kS, *tfull = empty + kS, *tempty = tfull + 2, *drain = tempty + 2, *pfull = drain + 1;
    uint32_t* tmem_s = reinterpret_cast<uint32_t*>(pfull + kGroups * C::kBuffers);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_s + 1);

    grid_dep_wait();  // the previous kernels' outputs; no tensor memory is taken before it
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = smem_u32(smem);
    const uint32_t rank = cluster_rank();
    const bool leader = rank == 0;
    const int unit = (int)(blockIdx.x >> 1), n_units = (int)(gridDim.x >> 1);
    const int n_cols = C::kNT ? p.I : p.d;                   // channels of the output
    const int K = C::kNT ? p.d : p.I;
    const int nk1 = (K + (int)kBK - 1) / (int)kBK, nk = FORM == kFormDx ? 2 * nk1 : nk1;

    auto row_at = [&](int e) { return min(max(p.offsets[e], 0), p.M); };
    if (tid == 32) {
        for (int s = 0; s < kS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], 2 * kGroups * 4);  // an arrival per epilogue warp of both CTAs
        }
        mbar_init(drain, 1);
        for (int b = 0; b < kGroups * C::kBuffers; ++b) mbar_init(&pfull[b], 1);
        fence_mbar_init();
        *abort_flag = 0;
        if (base & 1023u) {  // the swizzled tiles need it
            set_error(p.err, MOE_ERR_CAPACITY, 1023);
            *abort_flag = 1;
        }
    }
    if (warp == 0) {
        const int cts = (n_cols + 2 * C::kChannels - 1) / (2 * C::kChannels);
        int carry = 0;
        for (int b = 0; b < p.N; b += 32) {
            const int e = b + lane;
            const int v = e < p.N ? row_tiles<MAXN>(max(row_at(e + 1) - row_at(e), 0)) * cts : 0;
            int inc = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += x;
            }
            if (e < p.N) first[e] = carry + inc - v;
            carry += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0) first[p.N] = carry;
    }
    if (warp == 1) tmem_alloc(tmem_s);
    if (p.dw.maps && warp >= 2)
        for (int e = (int)blockIdx.x * 8 + warp - 2; e < p.N; e += (int)gridDim.x * 8) expert_maps(p.dw, e);
    {  // rows of no expert
        const int64_t v0 = (int64_t)row_at(p.N) * n_cols / 8, v1 = (int64_t)p.M * n_cols / 8;
        for (int64_t v = v0 + (int64_t)blockIdx.x * kThreads + tid; v < v1; v += (int64_t)gridDim.x * kThreads)
            for (int o = 0; o < 3; ++o)
                if (p.out[o]) reinterpret_cast<uint4*>(p.out[o])[v] = make_uint4(0, 0, 0, 0);
        if constexpr (FORM == kFormUp && PACKED) {
            const int64_t b1 = (int64_t)p.M * p.nb;
            for (int64_t b = (int64_t)row_at(p.N) * p.nb + (int64_t)blockIdx.x * kThreads + tid; b < b1; b += (int64_t)gridDim.x * kThreads)
                for (int o = 0; o < 2; ++o) {
                    uint4* q = reinterpret_cast<uint4*>(p.q[o]) + 2 * b;
                    q[0] = q[1] = make_uint4(0, 0, 0, 0);
                    p.scale[o][b] = 0;
                }
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // the peer's barriers are ready before any arrival from here
    tc_fence_after();
    const uint32_t tmem = *tmem_s;
    const Schedule sc = schedule(first[p.N], n_units);

    if (warp == 0) {
        // ---------------- loads (each CTA its own stages, on the leader's barrier)
        const uint32_t full0 = leader_address(&full[0]);
        // The rows are read for every tile of channels and by the products that follow: they stay in L2.  The
        // weights of few rows pass through it once (those of an expert that has more than 64 rows in such a batch
        // serve its other row tiles too; skewed batches were not measured apart).  DeepSeek-V2-Lite shape, Up: 8
        // tokens 63.8 -> 61.6 us, 64 tokens 111.5 -> 108.1; the weight gradients after Dx, 4096 tokens, 254 -> 246.
        // With many rows the weights are shared by row tiles, and any policy on them cost 2 %.
        const uint64_t keep = l2_evict_last_policy(), once = l2_evict_first_policy();
        int st = 0, it = 0;
        uint32_t phase = 1;
        for (int t = unit; t < sc.total; t += n_units) {
            if (__any_sync(0xffffffffu, *abort_flag)) break;
            const Tile x = decode<FORM, MAXN, PACKED>(p, first, sc, t);
            const int rows = __shfl_sync(0xffffffffu, x.rows, 0), e = __shfl_sync(0xffffffffu, x.e, 0);
            if (rows <= 0) continue;
            const int half = (rows + kStepN - 1) / kStepN * kStepN / 2;  // rows staged by each CTA
            const int brow = __shfl_sync(0xffffffffu, x.row0, 0) + (int)rank * half;
            const int ch = __shfl_sync(0xffffffffu, x.c0, 0) + (int)rank * C::kChannels;
            const uint32_t bytes = 2 * (kStageA + (uint32_t)half * 128);
            for (int kb = 0; kb < nk; ++kb, ++it) {
                // a wait that gives up raises the abort flag, which ends the later ones
                (void)wait<true>(&empty[st], phase, abort_flag, p.err, 1);
                __syncwarp();
                if (elect_one()) {
                    const uint32_t ad = base + st * C::kStage, bd = ad + kStageA, bar = full0 + st * 8;
                    auto weights = [&](uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t b) {
                        if constexpr (MAXN <= 64) load_3d_hint(dst, map, c0, c1, e, b, once);
                        else load_3d(dst, map, c0, c1, e, b);
                    };
                    if (leader) mbar_arrive_expect_tx(&full[st], bytes);
                    const int part = FORM == kFormDx && kb >= nk1;
                    const int k0 = (kb - part * nk1) * (int)kBK;
                    if constexpr (FORM == kFormUp) {
                        weights(ad, &p.a[0], k0, ch, bar);
                        weights(ad + 8192, &p.a[1], k0, ch, bar);
                    } else if constexpr (FORM == kFormDh) {
                        weights(ad, &p.a[0], k0, ch, bar);
                    } else {
                        weights(ad, &p.a[part], ch, k0, bar);
                        weights(ad + 8192, &p.a[part], ch + 64, k0, bar);
                    }
                    load_2d_hint(bd, &p.b[part][half / 16 - 1], k0, brow, bar, keep);
                }
                __syncwarp();
                if (++st == kS) { st = 0; phase ^= 1; }
            }
        }
        // the leader's MMAs have consumed this CTA's last stages before it may leave
        for (int k = it > kS ? it - kS : 0; k < it; ++k)
            (void)wait<true>(&empty[k % kS], (k / kS) & 1, abort_flag, p.err, 2, false);
    } else if (warp == 1) {
        // ---------------- MMAs (the pair's leader)
        if (leader) {
            // K-major: 16 values = 32 bytes along the swizzled row; MN-major: 16 rows of 128 bytes,
            // the next 64 channels 8 KB on
            const uint64_t da0 = C::kNT ? smem_desc(base, 16, 1024) : smem_desc(base, 8192, 1024);
            const uint64_t db0 = smem_desc(base + kStageA, 16, 1024);
            constexpr uint32_t kStepA = C::kNT ? 32 : 2048, kStepB = 32;
            int st = 0, local = 0;
            uint32_t phase = 0;
            for (int t = unit; t < sc.total; t += n_units) {
                if (__any_sync(0xffffffffu, *abort_flag)) break;
                const Tile x = decode<FORM, MAXN, PACKED>(p, first, sc, t);
                const int rows = __shfl_sync(0xffffffffu, x.rows, 0);
                if (rows <= 0) continue;
                const uint32_t idesc = tc_idesc(256, (rows + kStepN - 1) / kStepN * kStepN, 0, C::kNT ? 0 : 1);
                const int ab = local & 1;
                const uint32_t acc = tmem + ab * 256;
                // a wait that gives up raises the abort flag, which ends the later ones
                (void)wait<true>(&tempty[ab], ((local >> 1) & 1) ^ 1, abort_flag, p.err, 3);
                tc_fence_after();
                for (int kb = 0; kb < nk; ++kb) {
                    (void)wait<true>(&full[st], phase, abort_flag, p.err, 4);
                    tc_fence_after();
                    __syncwarp();
                    if (elect_one()) {
                        const uint64_t da = desc_at(da0, st * C::kStage), db = desc_at(db0, st * C::kStage);
#pragma unroll
                        for (int kk = 0; kk < (int)kBK / 16; ++kk)
                            mma(acc, desc_at(da, kk * kStepA), desc_at(db, kk * kStepB), idesc, (kb | kk) ? 1u : 0u);
                        commit(&empty[st]);
                        if (kb + 1 == nk) commit(&tfull[ab]);
                    }
                    __syncwarp();
                    if (++st == kS) { st = 0; phase ^= 1; }
                }
                ++local;
            }
            // every MMA issued here is done before tensor memory is released
            if (elect_one()) commit_local(drain);
            __syncwarp();
            (void)wait<true>(drain, 0, abort_flag, p.err, 6, false);
        }
    } else {
        // ---------------- epilogue: warp w on tensor-memory lanes 32 (w % 4) ..; a group of four
        // warps takes every other panel, with buffers and a barrier of its own
        const int quarter = warp & 3, group = (warp - 2) >> 2, etid = (tid - 64) & (kGroupThreads - 1);
        const int bar_id = 1 + group;
        const bool boss = etid == 0;  // issues the group's output stores (and Dh's input loads)
        const uint32_t panels = base + C::kPanels + group * C::kBuffers * C::kBuffer;
        uint64_t* const in_bar = pfull + group * C::kBuffers;
        const uint32_t free0 = leader_address(&tempty[0]), free1 = leader_address(&tempty[1]);
        // stmatrix / ldmatrix: lanes 8j .. 8j + 7 address matrix j, a row of 16 bytes each
        const int mj = lane >> 3, mr = lane & 7;
        // this warp's 32 channels: the box and the first 16-byte chunk in its rows
        const int my_box = quarter >> 1, my_chunk = (quarter & 1) * 4;
        int local = 0, pn = 0;
        uint32_t in_phase = 0;  // Dh: parity of each buffer's input barrier
        // Dh: g and u of 32 rows from q0 on into buffer `b`
        auto load_inputs = [&](const Tile& x, int ch, int q0, int b) {
            const uint32_t dst = panels + b * C::kBuffer, bar = smem_u32(&in_bar[b]);
            const int n_box = ch + 64 < n_cols ? 2 : 1;
            mbar_arrive_expect_tx(&in_bar[b], 2 * n_box * kBox);
            for (int j = 0; j < n_box; ++j) {
                load_2d<false>(dst + j * kBox, &p.in[0], ch + j * 64, x.row0 + q0, bar);
                load_2d<false>(dst + (2 + j) * kBox, &p.in[1], ch + j * 64, x.row0 + q0, bar);
            }
        };
        // Dh, PACKED: g and u of 32 rows from q0 on, 32 channels of this warp; what lies past the rows is not used
        PackedPanel ahead;
        auto load_packed = [&](const Tile& x, int ch, int q0) {
            const int block = (ch + quarter * 32) / 32;
#pragma unroll
            for (int i = 0; i < 8; ++i) ahead.g[i] = ahead.u[i] = 0;
            ahead.sg = ahead.su = 0.f;
            if (block >= p.nb) return;  // the same for the warp
            const int r0 = x.row0 + q0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int64_t at = ((int64_t)min(r0 + (i >> 1) * 8 + (lane & 3) * 2 + (i & 1), p.M - 1) * p.nb + block) * 32 + (lane >> 2) * 4;
                ahead.g[i] = *reinterpret_cast<const uint32_t*>(p.q[0] + at);
                ahead.u[i] = *reinterpret_cast<const uint32_t*>(p.q[1] + at);
            }
            const int64_t at = (int64_t)min(r0 + lane, p.M - 1) * p.nb + block;
            ahead.sg = pack8::step(p.scale[0][at]);
            ahead.su = pack8::step(p.scale[1][at]);
        };
        for (int t = unit; t < sc.total; t += n_units) {
            const Tile x = decode<FORM, MAXN, PACKED>(p, first, sc, t);
            if (x.rows <= 0) continue;
            const int ch = x.c0 + (int)rank * C::kChannels;
            const bool any = ch < n_cols && group * kPanel < x.rows;  // this group has a panel of this CTA's channels
            if (FORM == kFormDh && PACKED && any) load_packed(x, ch, group * kPanel);
            if (FORM == kFormDh && !PACKED && any && boss) {  // the first panel's inputs, beside the tile's MMAs
                stores_read<C::kBuffers - 1>();
                load_inputs(x, ch, group * kPanel, pn % C::kBuffers);
            }
            const int ab = local & 1;
            bool ok = true;
            if (lane == 0) ok = wait<true>(&tfull[ab], (local >> 1) & 1, abort_flag, p.err, 5);
            // the four warps share barriers: they leave together
            const bool stop = bar_any(bar_id, kGroupThreads, !ok || *abort_flag);
            ++local;
            tc_fence_after();
            const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + ab * 256;
            if (any) {
#pragma unroll 1
                for (int q0 = group * kPanel; q0 < x.rows; q0 += kGroups * kPanel, ++pn) {
                    const uint32_t buf = panels + (pn % C::kBuffers) * C::kBuffer;
                    PackedPanel in;
                    if constexpr (FORM == kFormDh && PACKED) {
                        in = ahead;
                        if (q0 + kGroups * kPanel < x.rows) load_packed(x, ch, q0 + kGroups * kPanel);
                    }
                    if (FORM == kFormDh && !PACKED && boss && q0 + kGroups * kPanel < x.rows) {
                        stores_read<0>();  // the last panel's store has left the other buffer
                        load_inputs(x, ch, q0 + kGroups * kPanel, (pn + 1) % C::kBuffers);
                    }
                    uint32_t lo[16], hi[16];  // lanes 0-15 and 16-31 of the warp's quarter
                    tmem_ld_16x32(taddr + q0, lo);
                    tmem_ld_16x32(taddr + (16u << 16) + q0, hi);
                    if constexpr (C::kBuffers == 1) {  // the last panel's store has read the buffer
                        if (boss) stores_read<0>();
                        bar_sync(bar_id, kGroupThreads);
                    }
                    tmem_ld_wait();
                    if constexpr (FORM == kFormUp) {
                        // warps of quarters 0, 1 hold g and those of 2, 3 hold u of the same channels, at the
                        // same registers.  Each pair of warps swaps 16 rows' values for the other 16's, in
                        // fp32, and forms h of the rows it then has both of.
                        const bool is_u = quarter >= 2;
                        if constexpr (PACKED) {
                            const int block = (ch + (quarter & 1) * 32) / 32;
                            int8_t* const q = p.q[is_u] + (lane >> 2) * 4;
#pragma unroll
                            for (int i = 0; i < 8; ++i) {  // a row: channels lane / 4 + 0, 8, 16, 24
                                const int k = (i >> 1) * 4 + (i & 1), r = q0 + (i >> 1) * 8 + (lane & 3) * 2 + (i & 1);
                                float v[4] = {__uint_as_float(lo[k]), __uint_as_float(lo[k + 2]), __uint_as_float(hi[k]), __uint_as_float(hi[k + 2])};
                                uint32_t m = max(max(pack8::magnitude(v[0]), pack8::magnitude(v[1])), max(pack8::magnitude(v[2]), pack8::magnitude(v[3])));
#pragma unroll
                                for (int o = 4; o < 32; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                                const uint32_t E = pack8::exponent(m);
                                const float inv = pack8::to_steps(E);
                                if (E == pack8::kTop)
#pragma unroll
                                    for (int j = 0; j < 4; ++j) v[j] = pack8::within(v[j], E);
                                uint32_t w = pack8::bytes4(pack8::quantise(v[0], inv), pack8::quantise(v[1], inv), pack8::quantise(v[2], inv),
                                                           pack8::quantise(v[3], inv));
                                if (E == 255u) w = 0;
                                if (r < x.rows && block < p.nb) {
                                    const int64_t at = (int64_t)(x.row0 + r) * p.nb + block;
                                    *reinterpret_cast<uint32_t*>(q + at * 32) = w;
                                    if (lane < 4) p.scale[is_u][at] = (uint8_t)E;
                                }
                            }
                        }
                        float4* mine = reinterpret_cast<float4*>(smem + C::kPanels + kGroups * C::kBuffers * C::kBuffer +
                                                                 group * C::kSwap) + etid;
                        const float4* theirs = mine + (((etid >> 5) ^ 2) - (etid >> 5)) * 32;
                        // g gives away rows 16-31 (blocks 2, 3), u rows 0-15, a block at a time
                        const uint32_t at = buf + mr * 128 + (((my_chunk + mj) ^ mr) << 4);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t* l = is_u ? lo + 4 * i : lo + 8 + 4 * i;
                            const uint32_t* h = is_u ? hi + 4 * i : hi + 8 + 4 * i;
                            if (i > 0) bar_sync(3 + group * 2 + (quarter & 1), 64);
                            mine[0] = make_float4(__uint_as_float(l[0]), __uint_as_float(l[1]), __uint_as_float(l[2]),
                                                  __uint_as_float(l[3]));
                            mine[kGroupThreads] = make_float4(__uint_as_float(h[0]), __uint_as_float(h[1]),
                                                              __uint_as_float(h[2]), __uint_as_float(h[3]));
                            if (!PACKED && p.out[0]) {  // g or u of 16 rows, beside the swap
#pragma unroll
                                for (int b = 2 * i; b < 2 * i + 2; ++b)
                                    stmatrix_x4_trans(at + (is_u ? kBox : 0) + b * 1024, pack_f(lo[4 * b], lo[4 * b + 1]),
                                                      pack_f(lo[4 * b + 2], lo[4 * b + 3]), pack_f(hi[4 * b], hi[4 * b + 1]),
                                                      pack_f(hi[4 * b + 2], hi[4 * b + 3]));
                            }
                            bar_sync(3 + group * 2 + (quarter & 1), 64);
                            uint32_t w[4];
#pragma unroll
                            for (int z = 0; z < 2; ++z) {
                                const float4 o = theirs[z * kGroupThreads];
                                const uint32_t* m = z ? (is_u ? hi + 8 + 4 * i : hi + 4 * i) : (is_u ? lo + 8 + 4 * i : lo + 4 * i);
                                const float of[4] = {o.x, o.y, o.z, o.w};
                                float v[4];
#pragma unroll
                                for (int q = 0; q < 4; ++q) {
                                    const float mf = __uint_as_float(m[q]);
                                    const float g = is_u ? of[q] : mf, u = is_u ? mf : of[q];
                                    v[q] = g * fast_sigmoid(g) * u;
                                }
                                w[2 * z] = pack_bf16x2(v[0], v[1]);
                                w[2 * z + 1] = pack_bf16x2(v[2], v[3]);
                            }
                            stmatrix_x4_trans(at + (PACKED ? 0 : 2 * kBox) + ((is_u ? 2 : 0) + i) * 1024, w[0], w[1], w[2], w[3]);
                        }
                    } else {
                        const uint32_t at = buf + my_box * kBox + mr * 128 + (((my_chunk + mj) ^ mr) << 4);
                        if constexpr (FORM == kFormDh && !PACKED) {
                            if (lane == 0)
                                (void)wait<false>(&in_bar[pn % C::kBuffers], (in_phase >> (pn % C::kBuffers)) & 1, abort_flag, p.err, 7, false);
                            __syncwarp();
                            in_phase ^= 1u << (pn % C::kBuffers);
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {  // 8 rows, 32 channels
                            const uint32_t* h[4] = {lo + 4 * i, lo + 4 * i + 2, hi + 4 * i, hi + 4 * i + 2};
                            if constexpr (FORM == kFormDh && PACKED) {
                                uint32_t a[4], b[4], hh[4];
                                float sg[2], su[2];
                                uint32_t gw[2], uw[2];
#pragma unroll
                                for (int z = 0; z < 2; ++z) {
                                    const int r = i * 8 + (lane & 3) * 2 + z;
                                    sg[z] = __shfl_sync(0xffffffffu, in.sg, r);
                                    su[z] = __shfl_sync(0xffffffffu, in.su, r);
                                    gw[z] = pack8::biased(in.g[2 * i + z]);
                                    uw[z] = pack8::biased(in.u[2 * i + z]);
                                }
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    float da[2], db[2], hv[2];
#pragma unroll
                                    for (int z = 0; z < 2; ++z) {
                                        const float gf = pack8::value(gw[z], j) * sg[z], uf = pack8::value(uw[z], j) * su[z];
                                        const float dh = __uint_as_float(h[j][z]), s = fast_sigmoid(gf), silu = gf * s;
                                        da[z] = dh * uf * s * (1.f + gf * (1.f - s));
                                        db[z] = dh * silu;
                                        hv[z] = silu * uf;
                                    }
                                    a[j] = pack_bf16x2(da[0], da[1]);
                                    b[j] = pack_bf16x2(db[0], db[1]);
                                    hh[j] = pack_bf16x2(hv[0], hv[1]);
                                }
                                stmatrix_x4_trans(at + i * 1024, a[0], a[1], a[2], a[3]);
                                stmatrix_x4_trans(at + 2 * kBox + i * 1024, b[0], b[1], b[2], b[3]);
                                stmatrix_x4_trans(at + 4 * kBox + i * 1024, hh[0], hh[1], hh[2], hh[3]);
                            } else if constexpr (FORM == kFormDh) {
                                uint32_t g[4], u[4], a[4], b[4];
                                ldmatrix_x4_trans(at + i * 1024, g[0], g[1], g[2], g[3]);
                                ldmatrix_x4_trans(at + 2 * kBox + i * 1024, u[0], u[1], u[2], u[3]);
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    float da[2], db[2];
#pragma unroll
                                    for (int z = 0; z < 2; ++z) {
                                        const float gf = z ? bf16_hi(g[j]) : bf16_lo(g[j]);
                                        const float uf = z ? bf16_hi(u[j]) : bf16_lo(u[j]);
                                        const float dh = __uint_as_float(h[j][z]), s = fast_sigmoid(gf);
                                        da[z] = dh * uf * s * (1.f + gf * (1.f - s));
                                        db[z] = dh * gf * s;
                                    }
                                    a[j] = pack_bf16x2(da[0], da[1]);
                                    b[j] = pack_bf16x2(db[0], db[1]);
                                }
                                stmatrix_x4_trans(at + i * 1024, a[0], a[1], a[2], a[3]);
                                stmatrix_x4_trans(at + 2 * kBox + i * 1024, b[0], b[1], b[2], b[3]);
                            } else {
                                uint32_t w[4];
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    w[j] = pack_bf16x2(__uint_as_float(h[j][0]), __uint_as_float(h[j][1]));
                                stmatrix_x4_trans(at + i * 1024, w[0], w[1], w[2], w[3]);
                            }
                        }
                    }
                    fence_proxy_async();
                    // the next panel's buffer is free once the store that last used it has read it
                    if ((FORM != kFormDh || PACKED) && C::kBuffers == 2 && boss) stores_read<0>();
                    bar_sync(bar_id, kGroupThreads);
                    // box b of the buffer: which output, and its first channel
                    auto out_of = [&](int b) { return FORM == kFormUp ? (PACKED ? 2 : b) : FORM == kFormDh ? b >> 1 : 0; };
                    auto col_of = [&](int b) { return ch + (FORM == kFormUp ? 0 : (b & 1) * 64); };
                    const int n_rows = x.rows - q0;
                    if (n_rows >= kPanel) {
                        if (boss) {
#pragma unroll
                            for (int b = 0; b < C::kBoxes; ++b)
                                if (p.out[out_of(b)] && col_of(b) < n_cols)
                                    store_2d(&p.o[out_of(b)], col_of(b), x.row0 + q0, buf + b * kBox);
                        }
                    } else {  // the rows after these are another expert's
                        for (int c = etid; c < C::kBoxes * n_rows * 8; c += kGroupThreads) {
                            const int b = c / (n_rows * 8), r = c / 8 % n_rows, q = c & 7;
                            const int col = col_of(b) + q * 8;
                            if (p.out[out_of(b)] && col < n_cols)
                                *reinterpret_cast<uint4*>(p.out[out_of(b)] + (int64_t)(x.row0 + q0 + r) * n_cols + col) =
                                    *reinterpret_cast<const uint4*>(smem + (buf - base) + b * kBox + r * 128 + ((q ^ (r & 7)) << 4));
                        }
                    }
                    if (boss) stores_commit();  // a group per panel, empty or not
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (!leader) arrive_cluster(ab ? free1 : free0);
                else mbar_arrive(&tempty[ab]);
            }
            if (stop) break;
        }
        // the buffers stay until the stores have read them, and the outputs are
        // complete when the grid ends
        if (boss) stores_done();
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    // the leader's MMAs, which read the peer's shared memory and write its
    // tensor memory, are done before either CTA frees or leaves
    cluster_sync();
    tc_fence_after();
    if (warp == 1) tmem_free(tmem);
    grid_dep_launch();
}

// ---------------------------------------------------------------- host

template <int FORM, int MAXN, bool PACKED>
cudaError_t launch_form(const RowsParams& p, int64_t units, int sms, cudaStream_t st) {
    auto kern = grouped_rows_kernel<FORM, MAXN, PACKED>;
    constexpr uint32_t kSmem = Cfg<FORM, MAXN, PACKED>::kSmem;
    cudaError_t e = allow_max_smem(kern);
    if (e != cudaSuccess) return e;
    int most = 0;
    e = resident_clusters(reinterpret_cast<const void*>(kern), 2, kThreads, kSmem, sms, &most);
    if (e != cudaSuccess) return e;
    if (most <= 0) return cudaErrorInvalidConfiguration;
    if (units > most) units = most;
    return note_launch(reinterpret_cast<const void*>(kern), kThreads, kSmem,
                       launch_units(kern, p, (int)units, 2, kThreads, kSmem, st));
}

template <int FORM, bool PACKED = false>
cudaError_t launch_rows(const RowsParams& p, bool few, int64_t units, int sms, cudaStream_t st) {
    return few ? launch_form<FORM, 64, PACKED>(p, units, sms, st) : launch_form<FORM, 256, PACKED>(p, units, sms, st);
}

}  // namespace

bool grouped_tc_shapes(bool bf16, int d, int I) {
    // rows on 16-byte boundaries; below 64 a K step or a box is mostly padding
    return bf16 && d % 8 == 0 && I % 8 == 0 && d >= 64 && I >= 64;
}

bool grouped_tc_usable(const GroupedArgs& a) {
    if (!grouped_tc_shapes(a.bf16, a.d, a.I) || a.M == 0) return false;
    for (const void* q : {a.a0, a.a1, a.b0, a.b1, a.g, a.u, (const void*)a.o0, (const void*)a.o1, (const void*)a.o2})
        if (reinterpret_cast<uintptr_t>(q) & 15u) return false;
    return true;
}

cudaError_t resident_clusters(const void* kernel, int size, int threads, uint32_t smem, int sms, int* clusters) {
    static std::mutex mu;
    static std::vector<std::array<int64_t, 3>> done;  // kernel, device, clusters
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    for (const auto& x : done)
        if (x[0] == (int64_t)reinterpret_cast<uintptr_t>(kernel) && x[1] == dev) { *clusters = (int)x[2]; return cudaSuccess; }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sms / size * size);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
    if (e != cudaSuccess) return e;
    *clusters = n < sms / size ? n : sms / size;
    done.push_back({(int64_t)reinterpret_cast<uintptr_t>(kernel), dev, *clusters});
    return cudaSuccess;
}

cudaError_t launch_grouped_rows_tc(const GroupedArgs& a, const GroupedArgs* dw, cudaStream_t st) {
    RowsParams p;
    std::memset(&p, 0, sizeof(p));
    p.offsets = a.offsets; p.err = a.err;
    p.M = a.M; p.N = a.N; p.d = a.d; p.I = a.I;
    const bool nt = a.form == kFormUp || a.form == kFormDh;
    const uint64_t d = (uint64_t)a.d, I = (uint64_t)a.I, M = (uint64_t)a.M;
    const uint64_t K = nt ? d : I, cols = nt ? I : d;
    // By the batch's average rows an expert, dropped slots included.  Tiles of up to 64 rows leave room for 8 or 9
    // stages instead of 5 or 6, which is what a stream of weights wants: 48 rows an expert (DeepSeek-V2-Lite
    // shape) took Up 121 us against 129 and Dh 73 against 77, 96 rows 149 against 132 and 92 against 84.
    const bool few = (long long)a.M <= 48LL * a.N;
    const int max_n = few ? 64 : 256;
    const int span = a.form == kFormUp ? 128 : 256;
    bool ok = true;
    const void* rows[2] = {a.a0, a.a1};
    const void* weights[2] = {a.b0, a.b1};
    const void* in[2] = {a.g, a.u};
    void* outs[3] = {a.o0, a.o1, a.o2};
    if (a.packed) {  // g and u without tensor maps
        const bool up = a.form == kFormUp;
        p.nb = pack_blocks(a.I);
        for (int i = 0; i < 2; ++i) {
            p.q[i] = static_cast<int8_t*>(up ? outs[i] : const_cast<void*>(in[i]));
            p.scale[i] = up ? (i ? a.s1 : a.s0) : const_cast<uint8_t*>(i ? a.us : a.gs);
            in[i] = nullptr;
            if (up) outs[i] = nullptr;
        }
    }
    auto rows_map = [&](CUtensorMap* m, const void* base, uint64_t width, uint32_t box_rows) {
        ok = ok && encode_bf16_2d(m, base, width, M, width * 2, 64, box_rows) == MOE_OK;
    };
    for (int i = 0; i < 2; ++i) {
        // a box height for every part of a tile that can occur (a tile has at most M rows, rounded up to 32)
        if (rows[i])
            for (int h = 0; h < max_n / kStepN && h * kStepN < a.M; ++h) rows_map(&p.b[i][h], rows[i], K, (h + 1) * 16);
        // K-major weights in boxes of the rows that a CTA takes of one matrix, MN-major in 64 x 64
        if (weights[i])
            ok = ok && encode_3d(&p.a[i], true, weights[i], d, I, (uint64_t)a.N, 64, a.form == kFormDh ? 128 : 64) == MOE_OK;
        if (in[i]) rows_map(&p.in[i], in[i], cols, kPanel);
    }
    for (int i = 0; i < 3; ++i) {
        p.out[i] = static_cast<__nv_bfloat16*>(outs[i]);
        if (outs[i]) rows_map(&p.o[i], outs[i], cols, kPanel);
    }
    if (dw) ok = ok && dw_map_params(*dw, p.dw);
    if (!ok) return cudaErrorInvalidValue;
    const int64_t col_tiles = ((int64_t)cols + span - 1) / span;
    // an upper bound of the tiles, each cut into up to eight parts where there are few
    const int64_t units = ((int64_t)a.M / max_n + (a.N < a.M ? a.N : a.M)) * col_tiles * 8;
    switch (a.form) {
        case kFormUp: return a.packed ? launch_rows<kFormUp, true>(p, few, units, a.sms, st) : launch_rows<kFormUp>(p, few, units, a.sms, st);
        case kFormDown: return launch_rows<kFormDown>(p, few, units, a.sms, st);
        case kFormDh: return a.packed ? launch_rows<kFormDh, true>(p, few, units, a.sms, st) : launch_rows<kFormDh>(p, few, units, a.sms, st);
        case kFormDx: return launch_rows<kFormDx>(p, few, units, a.sms, st);
        case kFormDw: break;
    }
    return cudaErrorInvalidValue;
}

}  // namespace moe
