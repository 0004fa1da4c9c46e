// The experts' grouped products on the tensor cores (tcgen05, accumulators in
// tensor memory), fed by TMA: bf16 layers whose rows start on 16-byte
// boundaries.  One persistent kernel per form; with x, h, dy, dg, du the
// grouped rows and Wg, Wu, Wd [I, d] an expert's weights:
//   Up    [g | u] = x [Wg ; Wu]^T      128 channels of each a tile, K = d;
//                                      epilogue h = SiLU(g) u, stores g, u, h
//   Down  y = h Wd                     K = I; Wd an MN-major operand
//   Dh    dh = dy Wd^T                 K = d; epilogue dg, du from g, u
//   Dx    dx = dg Wg + du Wu           K = I twice, one accumulator
//   Dw    dW = a^T b over the expert's rows: both operands MN-major, K = rows
// A tile is 128 rows (or channels) x 256 columns, or 256 x 256 on a CTA pair
// with the 2-CTA MMA, where each CTA stages half of either operand.
//
// The tiles of all experts form one list (expert by expert, row tiles
// innermost, so that a weight tile is read by consecutive units and comes from
// L2 after the first); every CTA forms the prefix sums of the counts itself.
// A row tile that runs past its segment reads the next expert's rows: rows do
// not mix in these products and those are not stored.  In Dw the rows are
// summed, so each expert has tensor maps of its own whose row count ends with
// its segment (map kernel): TMA fills the rest of the last K step with zeros.
//
// Block: warp 0 issues the TMA loads, warp 1 the MMAs (one thread), warps 2-5
// drain the accumulators (a thread owns a row), double-buffered so that the
// epilogue of a tile runs beside the next tile's MMAs.  Outputs go through
// 32 x 128-byte boxes in shared memory and TMA stores; a warp at the ragged
// end of a segment stores its rows directly.  Every wait is bounded.
#include <cuda.h>

#include <cstring>
#include <mutex>

#include "common.cuh"
#include "tma.h"
#include "train.h"
#include "train_tc.cuh"

namespace moe {

namespace {

using namespace train;

constexpr int kBM = 128, kBN = 256, kThreads = 192;
constexpr uint32_t kBK = kTcBK;
constexpr uint32_t kStageA = kBM * kBK * 2;  // 16 KB
constexpr uint32_t kBox = 32 * 128;          // 32 rows x 128 bytes
constexpr int kMapsPerExpert = 3;            // Dw: a0, a1, b

template <bool PAIR>
struct Cfg {
    static constexpr int kStages = PAIR ? 6 : 4;
    static constexpr uint32_t kStageB = (PAIR ? kBN / 2 : kBN) * kBK * 2;
    static constexpr uint32_t kStage = kStageA + kStageB;
    static constexpr uint32_t kBoxes = kStages * kStage;      // 8 boxes: two per epilogue warp
    static constexpr uint32_t kTable = kBoxes + 8 * kBox;     // tiles before each expert
    static constexpr uint32_t kBars = kTable + ((kTrainMaxExperts + 1) * 4 + 15) / 16 * 16;
    static constexpr uint32_t kSmem = kBars + (2 * kStages + 5) * 8 + 16;
    static_assert(kSmem <= 232448, "227 KB of shared memory per block");
};

struct TcGrouped {
    CUtensorMap a[2], b[2], o[3];
    const unsigned char* maps;  // Dw: [N][kMapsPerExpert] tensor maps
    const int32_t* offsets;
    __nv_bfloat16* out[3];      // row forms
    const __nv_bfloat16 *g, *u; // Dh
    int M, N, d, I, n_mat, accumulate;
    DevError* err;
};

// g s(g) u and its pieces with the fast exponential and division (a few ulp in
// fp32; the results are rounded to bf16).  e^-g overflows to infinity for very
// negative g and 1 / (1 + inf) = 0, the limit.
__device__ __forceinline__ float fast_sigmoid(float g) { return __fdividef(1.f, 1.f + __expf(-g)); }

// One tile: the expert, its rows, the tile's first row (channel in Dw) and
// column, which of two matrices (Dw), and the K steps
struct Tile {
    int e, row0, rows, m0, n0, mat, nk;
};

template <int FORM>
__device__ __forceinline__ int steps_of(const TcGrouped& p, int rows) {
    const int K = FORM == kFormDw ? rows : FORM == kFormUp || FORM == kFormDh ? p.d : p.I;
    return (K + (int)kBK - 1) / (int)kBK * (FORM == kFormDx ? 2 : 1);
}
template <int FORM>
__device__ __forceinline__ int col_tiles(const TcGrouped& p) {
    return FORM == kFormUp ? (p.I + 127) / 128 : ((FORM == kFormDh ? p.I : p.d) + kBN - 1) / kBN;
}

template <int FORM, bool PAIR>
__device__ __forceinline__ Tile decode(const TcGrouped& p, const int* first, int t) {
    constexpr int kRows = PAIR ? 2 * kBM : kBM;
    int lo = 0, hi = p.N;
    while (hi - lo > 1) {  // the last expert whose tiles start at or before t
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= t) lo = mid;
        else hi = mid;
    }
    Tile x;
    x.e = lo;
    x.row0 = min(max(p.offsets[lo], 0), p.M);
    x.rows = max(min(max(p.offsets[lo + 1], 0), p.M) - x.row0, 0);
    int local = t - first[lo];
    const int mts = ((FORM == kFormDw ? p.I : x.rows) + kRows - 1) / kRows;
    x.mat = 0;
    if (FORM == kFormDw && p.n_mat > 1) {
        const int per = mts * col_tiles<FORM>(p);
        x.mat = local / per;
        local -= x.mat * per;
    }
    x.m0 = local % mts * kRows;
    x.n0 = local / mts * (FORM == kFormUp ? 128 : kBN);
    x.nk = steps_of<FORM>(p, x.rows);
    return x;
}

template <int FORM, bool PAIR, bool F32>
__global__ void __launch_bounds__(kThreads, 1) grouped_tc_kernel(const __grid_constant__ TcGrouped p) {
    using C = Cfg<PAIR>;
    constexpr int kS = C::kStages;
    constexpr bool kRowForm = FORM != kFormDw;
    constexpr bool kNT = FORM == kFormUp || FORM == kFormDh;  // weights K-major
    extern __shared__ __align__(1024) unsigned char smem[];
    int* first = reinterpret_cast<int*>(smem + C::kTable);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBars);
    uint64_t *empty = full + kS, *tfull = empty + kS, *tempty = tfull + 2, *drain = tempty + 2;
    uint32_t* tmem_s = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_s + 1);

    grid_dep_wait();  // the previous kernels' outputs; no tensor memory is taken before it
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = smem_u32(smem);
    const uint32_t rank = PAIR ? cluster_rank() : 0;
    const bool leader = rank == 0;
    const int unit = PAIR ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
    const int n_units = PAIR ? (int)(gridDim.x >> 1) : (int)gridDim.x;
    constexpr int kRows = PAIR ? 2 * kBM : kBM;
    const int row_off = (int)rank * kBM;

    if (warp == 0) {  // tiles before each expert
        int carry = 0;
        for (int b = 0; b < p.N; b += 32) {
            const int e = b + lane;
            int v = 0;
            if (e < p.N) {
                const int r0 = min(max(p.offsets[e], 0), p.M), r1 = min(max(p.offsets[e + 1], 0), p.M);
                v = ((kRowForm ? max(r1 - r0, 0) : p.I) + kRows - 1) / kRows * col_tiles<FORM>(p) * (kRowForm ? 1 : p.n_mat);
            }
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
    if (tid == 32) {
        for (int s = 0; s < kS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], PAIR ? 8 : 4);  // an arrival per epilogue warp (of both CTAs)
        }
        mbar_init(drain, 1);
        fence_mbar_init();
        *abort_flag = 0;
        if (base & 1023u) {  // the swizzled tiles need it
            set_error(p.err, MOE_ERR_CAPACITY, 1023);
            *abort_flag = 1;
        }
    }
    if (warp == 1) tmem_alloc<PAIR>(tmem_s);
    if constexpr (kRowForm) {  // rows of no expert
        const int n_cols = kNT ? p.I : p.d;
        const int64_t v0 = (int64_t)min(max(p.offsets[p.N], 0), p.M) * n_cols / 8, v1 = (int64_t)p.M * n_cols / 8;
        for (int64_t v = v0 + (int64_t)blockIdx.x * kThreads + tid; v < v1; v += (int64_t)gridDim.x * kThreads)
            for (int o = 0; o < 3; ++o)
                if (p.out[o]) reinterpret_cast<uint4*>(p.out[o])[v] = make_uint4(0, 0, 0, 0);
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync();  // the peer's barriers are ready before any arrival from here
    tc_fence_after();
    const uint32_t tmem = *tmem_s;
    const int n_tiles = first[p.N];

    if (warp == 0) {
        // ---------------- loads (each CTA its own stages)
        if (lane == 0) {
            int it = 0, last_e = -1;
            for (int t = unit; t < n_tiles && !*abort_flag; t += n_units) {
                const Tile x = decode<FORM, PAIR>(p, first, t);
                const unsigned char* emaps = nullptr;
                if constexpr (FORM == kFormDw) {
                    emaps = p.maps + (size_t)x.e * kMapsPerExpert * 128;
                    if (x.e != last_e && x.nk > 0) {
                        for (int m = 0; m < kMapsPerExpert; ++m) map_acquire(emaps + m * 128);
                        last_e = x.e;
                    }
                }
                const int nk1 = FORM == kFormDx ? x.nk / 2 : x.nk;
                for (int kb = 0; kb < x.nk; ++kb, ++it) {
                    const int st = it % kS;
                    if (!wait<PAIR>(&empty[st], ((it / kS) & 1) ^ 1, abort_flag, p.err, 1)) break;
                    const uint32_t ad = base + st * C::kStage, bd = ad + kStageA;
                    const uint32_t bar = PAIR ? leader_address(&full[st]) : smem_u32(&full[st]);
                    if (leader) mbar_arrive_expect_tx(&full[st], (PAIR ? 2 : 1) * C::kStage);
                    const int part = FORM == kFormDx && kb >= nk1;
                    const int k0 = (kb - part * nk1) * (int)kBK;
                    if constexpr (FORM == kFormDw) {
                        const void* am = emaps + x.mat * 128;
                        const void* bm = emaps + 2 * 128;
#pragma unroll
                        for (int j = 0; j < kBM / 64; ++j)
                            load_2d<PAIR>(ad + j * 8192, am, x.m0 + row_off + j * 64, k0, bar);
#pragma unroll
                        for (int j = 0; j < (PAIR ? 2 : 4); ++j)
                            load_2d<PAIR>(bd + j * 8192, bm, x.n0 + (int)rank * 128 + j * 64, k0, bar);
                    } else {
                        load_2d<PAIR>(ad, &p.a[part], k0, x.row0 + x.m0 + row_off, bar);
                        if constexpr (FORM == kFormUp) {
                            // B = [gate rows ; up rows]; a pair's leader holds the gate rows, its peer the up rows
                            if (!PAIR || leader) load_3d<PAIR>(bd, &p.b[0], k0, x.n0, x.e, bar);
                            if (!PAIR) load_3d<PAIR>(bd + C::kStageB / 2, &p.b[1], k0, x.n0, x.e, bar);
                            else if (!leader) load_3d<PAIR>(bd, &p.b[1], k0, x.n0, x.e, bar);
                        } else if constexpr (FORM == kFormDh) {
#pragma unroll
                            for (int j = 0; j < (PAIR ? 1 : 2); ++j)
                                load_3d<PAIR>(bd + j * 16384, &p.b[0], k0, x.n0 + ((int)rank + j) * 128, x.e, bar);
                        } else {
#pragma unroll
                            for (int j = 0; j < (PAIR ? 2 : 4); ++j)
                                load_3d<PAIR>(bd + j * 8192, &p.b[part], x.n0 + (int)rank * 128 + j * 64, k0, x.e, bar);
                        }
                    }
                }
            }
            // the last stages' loads have landed (a pair: and were consumed by the
            // leader's MMAs) before the block may leave
            for (int k = it > kS ? it - kS : 0; k < it; ++k) {
                if constexpr (PAIR) (void)wait<true>(&empty[k % kS], (k / kS) & 1, abort_flag, p.err, 2, false);
                else (void)wait<false>(&full[k % kS], (k / kS) & 1, abort_flag, p.err, 2, false);
            }
        }
    } else if (warp == 1) {
        // ---------------- MMAs (the leader of a pair)
        if (lane == 0 && leader) {
            constexpr uint32_t idesc = tc_idesc(PAIR ? 2 * kBM : kBM, kBN, kNT ? 0 : 1, FORM == kFormDw ? 1 : 0);
            int it = 0, local = 0;
            for (int t = unit; t < n_tiles; t += n_units, ++local) {
                if (*abort_flag) break;
                const int nk = decode<FORM, PAIR>(p, first, t).nk;
                const int ab = local & 1;
                if (!wait<PAIR>(&tempty[ab], ((local >> 1) & 1) ^ 1, abort_flag, p.err, 3)) break;
                tc_fence_after();
                bool ok = true;
                for (int kb = 0; kb < nk; ++kb, ++it) {
                    const int st = it % kS;
                    if (!wait<PAIR>(&full[st], (it / kS) & 1, abort_flag, p.err, 4)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t ad = base + st * C::kStage, bd = ad + kStageA;
#pragma unroll
                    for (int kk = 0; kk < (int)kBK / 16; ++kk) {
                        // K-major: 16 values = 32 bytes along the swizzled row; MN-major: 16 rows of 128 bytes,
                        // the next 64 rows or columns 8 KB on
                        const uint64_t da = FORM == kFormDw ? smem_desc(ad + kk * 2048, 8192, 1024) : smem_desc(ad + kk * 32, 16, 1024);
                        const uint64_t db = kNT ? smem_desc(bd + kk * 32, 16, 1024) : smem_desc(bd + kk * 2048, 8192, 1024);
                        mma<PAIR>(tmem + ab * kBN, da, db, idesc, (kb | kk) ? 1u : 0u);
                    }
                    commit<PAIR>(&empty[st]);
                }
                if (!ok) break;
                commit<PAIR>(&tfull[ab]);
            }
            // every MMA issued here is done before tensor memory is released
            commit_local<PAIR>(drain);
            (void)wait<PAIR>(drain, 0, abort_flag, p.err, 6, false);
        }
    } else {
        // ---------------- epilogue: warps 2..5, a thread owns an accumulator row
        const int quarter = warp & 3;
        const uint32_t boxes = base + C::kBoxes + quarter * 2 * kBox;
        const uint32_t sw = lane & 7;  // 128-byte swizzle: chunk j of row i at chunk j ^ (i & 7)
        const uint32_t free0 = PAIR ? leader_address(&tempty[0]) : 0, free1 = PAIR ? leader_address(&tempty[1]) : 0;
        int local = 0, pn = 0;
        // 32 packed values (64 bytes) of this row to half `hh` of box `box`
        auto to_box = [&](uint32_t box, int hh, const uint32_t* w) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                st_shared16(box + lane * 128 + ((((uint32_t)(hh * 4 + q)) ^ sw) << 4), w[4 * q], w[4 * q + 1],
                            w[4 * q + 2], w[4 * q + 3]);
        };
        // the same to a row in global memory, columns below n_cols
        auto to_row = [&](__nv_bfloat16* row, int col, int n_cols, const uint32_t* w) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (col + q * 8 < n_cols)
                    *reinterpret_cast<uint4*>(row + col + q * 8) =
                        make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
        };
        for (int t = unit; t < n_tiles; t += n_units, ++local) {
            if (__shfl_sync(0xffffffffu, *abort_flag, 0)) break;
            const Tile x = decode<FORM, PAIR>(p, first, t);
            const int ab = local & 1;
            bool ok = true;
            if (lane == 0) ok = wait<PAIR>(&tfull[ab], (local >> 1) & 1, abort_flag, p.err, 5);
            if (!__shfl_sync(0xffffffffu, ok, 0)) break;
            tc_fence_after();
            const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + ab * kBN;
            const int m_first = x.m0 + row_off + quarter * 32;  // this warp's first row (channel) in the segment
            if constexpr (kRowForm) {
                const bool valid = m_first + lane < x.rows, boxed = m_first + 32 <= x.rows;
                const int n_cols = kNT ? p.I : p.d;
                const int64_t row = (int64_t)x.row0 + m_first + lane;
                if (m_first < x.rows) {
                    constexpr int kCols = FORM == kFormUp ? 128 : kBN;
#pragma unroll 1
                    for (int c = 0; c < kCols && x.n0 + c < n_cols; c += 64) {
                        const int col = x.n0 + c;
                        if constexpr (FORM == kFormDh) {
                            if (boxed) {
                                if (lane == 0) stores_read<0>();
                                __syncwarp();
                            }
#pragma unroll 1
                            for (int hh = 0; hh < 2; ++hh) {
                                float v[32];
                                tmem_ld32(taddr + c + hh * 32, v);
                                uint32_t wg[16], wu[16];
#pragma unroll
                                for (int q = 0; q < 4; ++q) {
                                    const int cc = col + hh * 32 + q * 8;
                                    uint4 gq = make_uint4(0, 0, 0, 0), uq = gq;
                                    if (valid && cc < n_cols) {
                                        gq = *reinterpret_cast<const uint4*>(p.g + row * n_cols + cc);
                                        uq = *reinterpret_cast<const uint4*>(p.u + row * n_cols + cc);
                                    }
                                    float gf[8], uf[8];
                                    unpack16(gq, gf, (__nv_bfloat16*)nullptr);
                                    unpack16(uq, uf, (__nv_bfloat16*)nullptr);
#pragma unroll
                                    for (int i = 0; i < 8; i += 2) {
                                        float a[2], b[2];
#pragma unroll
                                        for (int j = 0; j < 2; ++j) {
                                            const float g = gf[i + j], s = fast_sigmoid(g), dh = v[q * 8 + i + j];
                                            a[j] = dh * uf[i + j] * s * (1.f + g * (1.f - s));
                                            b[j] = dh * g * s;
                                        }
                                        wg[q * 4 + i / 2] = pack_bf16x2(a[0], a[1]);
                                        wu[q * 4 + i / 2] = pack_bf16x2(b[0], b[1]);
                                    }
                                }
                                if (boxed) {
                                    to_box(boxes, hh, wg);
                                    to_box(boxes + kBox, hh, wu);
                                } else if (valid) {
                                    to_row(p.out[0] + row * n_cols, col + hh * 32, n_cols, wg);
                                    to_row(p.out[1] + row * n_cols, col + hh * 32, n_cols, wu);
                                }
                            }
                            if (boxed) {
                                fence_proxy_async();
                                __syncwarp();
                                if (lane == 0) {
                                    store_2d(&p.o[0], col, x.row0 + m_first, boxes);
                                    store_2d(&p.o[1], col, x.row0 + m_first, boxes + kBox);
                                }
                            }
                        } else {
                            // Up: g, u, h (h alone where the pre-activations are not kept); else one output
#pragma unroll 1
                            for (int kind = FORM == kFormUp && !p.out[0] ? 2 : 0; kind < (FORM == kFormUp ? 3 : 1); ++kind) {
                                const uint32_t box = boxes + (pn & 1) * kBox;
                                if (boxed) {
                                    if (lane == 0) stores_read<1>();  // the store before the last has left this box
                                    __syncwarp();
                                    ++pn;
                                }
#pragma unroll 1
                                for (int hh = 0; hh < 2; ++hh) {
                                    float v[32];
                                    tmem_ld32(taddr + c + hh * 32 + (kind == 1 ? 128 : 0), v);
                                    if (FORM == kFormUp && kind == 2) {
                                        float u[32];
                                        tmem_ld32(taddr + 128 + c + hh * 32, u);
#pragma unroll
                                        for (int i = 0; i < 32; ++i) v[i] = v[i] * fast_sigmoid(v[i]) * u[i];
                                    }
                                    uint32_t w[16];
#pragma unroll
                                    for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
                                    if (boxed) to_box(box, hh, w);
                                    else if (valid) to_row(p.out[kind] + row * n_cols, col + hh * 32, n_cols, w);
                                }
                                if (boxed) {
                                    fence_proxy_async();
                                    __syncwarp();
                                    if (lane == 0) store_2d(&p.o[kind], col, x.row0 + m_first, box);
                                }
                            }
                        }
                    }
                }
            } else if (m_first < p.I && !(p.accumulate && x.nk == 0)) {
                constexpr int kW = F32 ? 32 : 64;  // columns of a box
#pragma unroll 1
                for (int c = 0; c < kBN && x.n0 + c < p.d; c += kW) {
                    const uint32_t box = boxes + (pn & 1) * kBox;
                    if (lane == 0) stores_read<1>();
                    __syncwarp();
                    ++pn;
#pragma unroll 1
                    for (int hh = 0; hh < kW / 32; ++hh) {
                        float v[32];
                        if (x.nk > 0) tmem_ld32(taddr + c + hh * 32, v);
                        else {
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] = 0.f;
                        }
                        uint32_t w[32];
                        if constexpr (F32) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(v[i]);
                            to_box(box, 0, w);
                            to_box(box, 1, w + 16);
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
                            to_box(box, hh, w);
                        }
                    }
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) {
                        if (F32 && p.accumulate) add_3d(&p.o[x.mat], x.n0 + c, m_first, x.e, box);
                        else store_3d(&p.o[x.mat], x.n0 + c, m_first, x.e, box);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (PAIR && !leader) arrive_cluster(ab ? free1 : free0);
                else mbar_arrive(&tempty[ab]);
            }
        }
        // the boxes stay until the stores have read them, and the outputs are
        // complete when the grid ends
        if (lane == 0) stores_done();
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    // the leader's MMAs, which read the peer's shared memory and write its
    // tensor memory, are done before either CTA frees or leaves
    if constexpr (PAIR) cluster_sync();
    tc_fence_after();
    if (warp == 1) tmem_free<PAIR>(tmem);
    grid_dep_launch();
}

// ---------------------------------------------------------------- per-expert maps
// Dw: expert e's rows of a0, a1 and b as tensor maps of their own, made from
// the maps of the whole tensors.  A warp per expert.
struct MapParams {
    CUtensorMap t[kMapsPerExpert];
    const unsigned char* rows[kMapsPerExpert];  // the tensors
    int64_t row_bytes[kMapsPerExpert];
    unsigned char* maps;
    const int32_t* offsets;
    int M, N, n_mat;
};

__global__ void __launch_bounds__(128) expert_maps_kernel(const __grid_constant__ MapParams p) {
    grid_dep_wait();
    const int e = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (e < p.N) {
        const int r0 = min(max(p.offsets[e], 0), p.M), rows = min(max(p.offsets[e + 1], 0), p.M) - r0;
        if (rows > 0) {
            for (int m = 0; m < kMapsPerExpert; ++m) {
                unsigned char* out = p.maps + ((size_t)e * kMapsPerExpert + m) * 128;
                reinterpret_cast<uint32_t*>(out)[lane] = reinterpret_cast<const uint32_t*>(&p.t[m])[lane];
                __syncwarp();
                if (lane == 0)
                    map_replace(out, reinterpret_cast<uint64_t>(p.rows[m]) + (uint64_t)r0 * (uint64_t)p.row_bytes[m],
                                (uint32_t)rows);
            }
            if (lane == 0) map_release();
        }
    }
    grid_dep_launch();
}

// ---------------------------------------------------------------- host

// CTA pairs of this kernel that can be resident at once; cached per device
template <typename K>
cudaError_t resident_pairs(K kern, int sms, int* pairs) {
    static std::mutex mu;
    static int cache[64];
    static bool have[64] = {false};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) { *pairs = 0; return cudaSuccess; }
    std::lock_guard<std::mutex> lock(mu);
    if (!have[dev]) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(sms & ~1);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = Cfg<true>::kSmem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
            (void)cudaGetLastError();
            n = 0;
        }
        cache[dev] = n < sms / 2 ? n : sms / 2;
        have[dev] = true;
    }
    *pairs = cache[dev];
    return cudaSuccess;
}

template <int FORM, bool PAIR, bool F32>
cudaError_t launch_form(const TcGrouped& p, int64_t units, int sms, cudaStream_t st) {
    auto kern = grouped_tc_kernel<FORM, PAIR, F32>;
    cudaError_t e = allow_max_smem(kern);
    if (e != cudaSuccess) return e;
    int most = sms;
    if constexpr (PAIR) {
        e = resident_pairs(kern, sms, &most);
        if (e != cudaSuccess) return e;
        if (most <= 0) return cudaErrorInvalidConfiguration;
    }
    if (units > most) units = most;
    if (units < 1) units = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)units * (PAIR ? 2 : 1));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Cfg<PAIR>::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = PAIR ? 2 : 1;
    return note_launch(reinterpret_cast<const void*>(kern), kThreads, Cfg<PAIR>::kSmem, cudaLaunchKernelEx(&cfg, kern, p));
}

template <int FORM, bool F32>
cudaError_t launch_pairs_or_not(const TcGrouped& p, bool pair, int64_t units, int sms, cudaStream_t st) {
    return pair ? launch_form<FORM, true, F32>(p, units, sms, st) : launch_form<FORM, false, F32>(p, units, sms, st);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

bool grouped_tc_shapes(bool bf16, int d, int I) {
    // rows on 16-byte boundaries; below 64 a K step or a box is mostly padding
    return bf16 && d % 8 == 0 && I % 8 == 0 && d >= 64 && I >= 64;
}

bool grouped_tc_usable(const GroupedArgs& a) {
    if (!grouped_tc_shapes(a.bf16, a.d, a.I) || a.M == 0) return false;
    for (const void* q : {a.a0, a.a1, a.b0, a.b1, a.g, a.u, (const void*)a.o0, (const void*)a.o1, (const void*)a.o2})
        if (!aligned16(q)) return false;
    return true;
}

cudaError_t launch_grouped_tc(const GroupedArgs& a, cudaStream_t st, int* launches) {
    TcGrouped p;
    std::memset(&p, 0, sizeof(p));
    p.maps = a.maps; p.offsets = a.offsets; p.err = a.err;
    p.M = a.M; p.N = a.N; p.d = a.d; p.I = a.I;
    p.n_mat = a.o1 && a.form == kFormDw ? 2 : 1;
    p.accumulate = a.accumulate;
    p.g = static_cast<const __nv_bfloat16*>(a.g);
    p.u = static_cast<const __nv_bfloat16*>(a.u);
    *launches = 1;
    // 256-row tiles of a pair once the segments average that many rows: below,
    // more of a tile is another expert's rows.  Dw's rows are the I channels.
    const bool pair = a.form == kFormDw ? a.I >= 256 : (long long)a.M >= 256LL * a.N;
    const int tile_rows = pair ? 2 * kBM : kBM;
    const uint64_t d = (uint64_t)a.d, I = (uint64_t)a.I, M = (uint64_t)a.M;
    bool ok = true;
    auto rows_map = [&](CUtensorMap* m, const void* base, uint64_t cols, uint32_t box_rows) {
        ok = ok && encode_bf16_2d(m, base, cols, M, cols * 2, 64, box_rows) == MOE_OK;
    };
    auto weight_map = [&](CUtensorMap* m, const void* base, uint32_t box_rows) {
        ok = ok && encode_3d(m, true, base, d, I, (uint64_t)a.N, 64, box_rows) == MOE_OK;
    };
    auto out_rows = [&](int i, void* o, uint64_t cols) {
        p.out[i] = static_cast<__nv_bfloat16*>(o);
        if (o) rows_map(&p.o[i], o, cols, 32);
    };
    const int64_t n_tiles = a.form == kFormUp ? (a.I + 127) / 128 : ((a.form == kFormDh ? a.I : a.d) + kBN - 1) / kBN;
    int64_t units = ((int64_t)a.M / tile_rows + (a.N < a.M ? a.N : a.M)) * n_tiles;
    switch (a.form) {
        case kFormUp:
            rows_map(&p.a[0], a.a0, d, kBM);
            weight_map(&p.b[0], a.b0, 128); weight_map(&p.b[1], a.b1, 128);
            out_rows(0, a.o0, I); out_rows(1, a.o1, I); out_rows(2, a.o2, I);
            return ok ? launch_pairs_or_not<kFormUp, false>(p, pair, units, a.sms, st) : cudaErrorInvalidValue;
        case kFormDown:
            rows_map(&p.a[0], a.a0, I, kBM);
            weight_map(&p.b[0], a.b0, 64);
            out_rows(0, a.o0, d);
            return ok ? launch_pairs_or_not<kFormDown, false>(p, pair, units, a.sms, st) : cudaErrorInvalidValue;
        case kFormDh:
            rows_map(&p.a[0], a.a0, d, kBM);
            weight_map(&p.b[0], a.b0, 128);
            out_rows(0, a.o0, I); out_rows(1, a.o1, I);
            return ok ? launch_pairs_or_not<kFormDh, false>(p, pair, units, a.sms, st) : cudaErrorInvalidValue;
        case kFormDx:
            rows_map(&p.a[0], a.a0, I, kBM); rows_map(&p.a[1], a.a1, I, kBM);
            weight_map(&p.b[0], a.b0, 64); weight_map(&p.b[1], a.b1, 64);
            out_rows(0, a.o0, d);
            return ok ? launch_pairs_or_not<kFormDx, false>(p, pair, units, a.sms, st) : cudaErrorInvalidValue;
        case kFormDw: break;
    }
    MapParams mp;
    std::memset(&mp, 0, sizeof(mp));
    const void* a1 = a.a1 ? a.a1 : a.a0;
    rows_map(&mp.t[0], a.a0, I, kBK); rows_map(&mp.t[1], a1, I, kBK); rows_map(&mp.t[2], a.b0, d, kBK);
    const void* rows[3] = {a.a0, a1, a.b0};
    for (int i = 0; i < 3; ++i) {
        mp.rows[i] = static_cast<const unsigned char*>(rows[i]);
        mp.row_bytes[i] = (int64_t)(i < 2 ? I : d) * 2;
    }
    mp.maps = a.maps; mp.offsets = a.offsets; mp.M = a.M; mp.N = a.N; mp.n_mat = p.n_mat;
    for (int i = 0; i < p.n_mat; ++i)
        ok = ok && encode_3d(&p.o[i], !a.out_f32, i ? a.o1 : a.o0, d, I, (uint64_t)a.N, a.out_f32 ? 32 : 64, 32) == MOE_OK;
    if (!ok) return cudaErrorInvalidValue;
    cudaError_t e = launch_pdl(expert_maps_kernel, dim3((a.N + 3) / 4), dim3(128), 0, st, mp);
    if (e != cudaSuccess) return e;
    *launches = 2;
    units = (int64_t)a.N * p.n_mat * ((a.I + tile_rows - 1) / tile_rows) * n_tiles;
    return a.out_f32 ? launch_pairs_or_not<kFormDw, true>(p, pair, units, a.sms, st)
                     : launch_pairs_or_not<kFormDw, false>(p, pair, units, a.sms, st);
}

}  // namespace moe
