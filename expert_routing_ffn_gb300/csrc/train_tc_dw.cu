// The weight gradients of the experts' products on the tensor cores: per
// expert, dW = a^T b over its grouped rows (a [M, I]: dg and du, or h; b
// [M, d]: x, or dy), one or two a in a launch.  tcgen05, accumulators in
// tensor memory, fed by TMA.
//
// A tile is 128 channels x 256 columns of one dW, or 256 x 256 on a CTA pair
// with the 2-CTA MMA where each CTA stages half of either operand.  The rows
// are the K axis, so both operands are MN-major as they lie in memory.  They
// are summed, so a step that ran past the segment would add the next expert's
// rows: each expert has tensor maps of its own whose row count ends with its
// segment (map kernel), and TMA fills the rest of the last step with zeros.
// Every dW is written once, those of experts without rows as zeros, so at the
// sizes of a training step (a few hundred rows an expert) the store of dW
// costs as much as the MMAs: the epilogue has four 4 KB boxes a warp, so that
// its stores queue up instead of waiting for one another.
//
// Tiles are taken round robin by the resident CTAs (pairs), experts with most
// rows first, so that the units end together when the load is skewed.
//
// Block: warp 0 issues the TMA loads, warp 1 the MMAs (one thread), warps 2-5
// drain the accumulators (a thread owns a channel), double-buffered.  Every
// wait is bounded.
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
constexpr int kBoxesPerWarp = 4;
constexpr uint32_t kBK = kTcBK;
constexpr uint32_t kStageA = kBM * kBK * 2;  // 16 KB
constexpr uint32_t kBox = 32 * 128;          // 32 channels x 128 bytes
constexpr int kMapsPerExpert = 3;            // a0, a1, b

template <bool PAIR>
struct Cfg {
    static constexpr int kStages = PAIR ? 5 : 3;
    static constexpr uint32_t kStageB = (PAIR ? kBN / 2 : kBN) * kBK * 2;
    static constexpr uint32_t kStage = kStageA + kStageB;
    static constexpr uint32_t kBoxes = kStages * kStage;
    static constexpr uint32_t kTable = kBoxes + 4 * kBoxesPerWarp * kBox;  // experts by rows, packed with their row counts
    static constexpr uint32_t kBars = kTable + (kTrainMaxExperts * 4 + 15) / 16 * 16;
    static constexpr uint32_t kSmem = kBars + (2 * kStages + 5) * 8 + 16;
    static_assert(kSmem <= 232448, "227 KB of shared memory per block");
};

struct DwParams {
    CUtensorMap o[2];
    const unsigned char* maps;  // [N][kMapsPerExpert] tensor maps
    const int32_t* offsets;
    int M, N, d, I, n_mat, accumulate;
    DevError* err;
};

struct Tile {
    int e, rows, m0, n0, mat;
};

template <bool PAIR, bool F32>
__global__ void __launch_bounds__(kThreads, 1) grouped_dw_kernel(const __grid_constant__ DwParams p) {
    using C = Cfg<PAIR>;
    constexpr int kS = C::kStages;
    constexpr int kRows = PAIR ? 2 * kBM : kBM;
    extern __shared__ __align__(1024) unsigned char smem[];
    int* order = reinterpret_cast<int*>(smem + C::kTable);  // rank -> expert
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
    const int row_off = (int)rank * kBM;

    auto rows_of = [&](int e) {
        const int r0 = min(max(p.offsets[e], 0), p.M);
        return max(min(max(p.offsets[e + 1], 0), p.M) - r0, 0);
    };
    {  // experts in order of falling row count (the lower index first among equals)
        int* rows_s = reinterpret_cast<int*>(smem);  // the stages are not in use yet
        for (int e = tid; e < p.N; e += kThreads) rows_s[e] = rows_of(e);
        __syncthreads();
        for (int e = tid; e < p.N; e += kThreads) {
            const int r = rows_s[e];
            int place = 0;
            for (int f = 0; f < p.N; ++f) {
                const int q = rows_s[f];
                place += q > r || (q == r && f < e);
            }
            order[place] = e;
        }
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
    fence_proxy_async();  // the row counts' shared memory becomes a stage that TMA writes
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync();  // the peer's barriers are ready before any arrival from here
    tc_fence_after();
    const uint32_t tmem = *tmem_s;
    const int mts = (p.I + kRows - 1) / kRows, nts = (p.d + kBN - 1) / kBN;
    const int per = mts * nts * p.n_mat, n_tiles = per * p.N;
    // channel tiles innermost: a column tile of b is read by consecutive units
    auto decode = [&](int t) {
        Tile x;
        const int place = t / per;
        int local = t - place * per;
        x.e = order[place];
        x.rows = rows_of(x.e);
        x.mat = local / (mts * nts);
        local -= x.mat * mts * nts;
        x.n0 = local / mts;
        x.m0 = (local - x.n0 * mts) * kRows;
        x.n0 *= kBN;
        return x;
    };

    if (warp == 0) {
        // ---------------- loads (each CTA its own stages)
        if (lane == 0) {
            int it = 0, last_e = -1;
            for (int t = unit; t < n_tiles && !*abort_flag; t += n_units) {
                const Tile x = decode(t);
                const unsigned char* emaps = p.maps + (size_t)x.e * kMapsPerExpert * 128;
                if (x.e != last_e && x.rows > 0) {
                    for (int m = 0; m < kMapsPerExpert; ++m) map_acquire(emaps + m * 128);
                    last_e = x.e;
                }
                for (int k0 = 0; k0 < x.rows; k0 += (int)kBK, ++it) {
                    const int st = it % kS;
                    if (!wait<PAIR>(&empty[st], ((it / kS) & 1) ^ 1, abort_flag, p.err, 1)) break;
                    const uint32_t ad = base + st * C::kStage, bd = ad + kStageA;
                    const uint32_t bar = PAIR ? leader_address(&full[st]) : smem_u32(&full[st]);
                    if (leader) mbar_arrive_expect_tx(&full[st], (PAIR ? 2 : 1) * C::kStage);
#pragma unroll
                    for (int j = 0; j < kBM / 64; ++j)
                        load_2d<PAIR>(ad + j * 8192, emaps + x.mat * 128, x.m0 + row_off + j * 64, k0, bar);
#pragma unroll
                    for (int j = 0; j < (PAIR ? 2 : 4); ++j)
                        load_2d<PAIR>(bd + j * 8192, emaps + 2 * 128, x.n0 + (int)rank * 128 + j * 64, k0, bar);
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
            constexpr uint32_t idesc = tc_idesc(PAIR ? 2 * kBM : kBM, kBN, 1, 1);
            int it = 0, local = 0;
            for (int t = unit; t < n_tiles; t += n_units, ++local) {
                if (*abort_flag) break;
                const int rows = decode(t).rows;
                const int ab = local & 1;
                if (!wait<PAIR>(&tempty[ab], ((local >> 1) & 1) ^ 1, abort_flag, p.err, 3)) break;
                tc_fence_after();
                bool ok = true;
                for (int k0 = 0; k0 < rows; k0 += (int)kBK, ++it) {
                    const int st = it % kS;
                    if (!wait<PAIR>(&full[st], (it / kS) & 1, abort_flag, p.err, 4)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t ad = base + st * C::kStage, bd = ad + kStageA;
                    // 16 rows of 128 bytes a step, the next 64 channels or columns 8 KB on;
                    // 16-row steps without a row of the segment are left out
                    const int steps = min((int)kBK / 16, (rows - k0 + 15) / 16);
                    for (int kk = 0; kk < steps; ++kk)
                        mma<PAIR>(tmem + ab * kBN, smem_desc(ad + kk * 2048, 8192, 1024), smem_desc(bd + kk * 2048, 8192, 1024),
                                  idesc, (k0 | kk) ? 1u : 0u);
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
        // ---------------- epilogue: warps 2..5, a thread owns a channel of dW
        const int quarter = warp & 3;
        const uint32_t boxes = base + C::kBoxes + quarter * kBoxesPerWarp * kBox;
        const uint32_t sw = lane & 7;  // 128-byte swizzle: chunk j of row i at chunk j ^ (i & 7)
        const uint32_t free0 = PAIR ? leader_address(&tempty[0]) : 0, free1 = PAIR ? leader_address(&tempty[1]) : 0;
        int local = 0, pn = 0;
        constexpr int kW = F32 ? 32 : 64;  // columns of a box
        for (int t = unit; t < n_tiles; t += n_units, ++local) {
            if (__shfl_sync(0xffffffffu, *abort_flag, 0)) break;
            const Tile x = decode(t);
            const int ab = local & 1;
            bool ok = true;
            if (lane == 0) ok = wait<PAIR>(&tfull[ab], (local >> 1) & 1, abort_flag, p.err, 5);
            if (!__shfl_sync(0xffffffffu, ok, 0)) break;
            tc_fence_after();
            const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + ab * kBN;
            const int m = x.m0 + row_off + quarter * 32;  // this warp's first channel
            if (m < p.I && !(p.accumulate && x.rows == 0)) {
#pragma unroll 1
                for (int c = 0; c < kBN && x.n0 + c < p.d; c += kW, ++pn) {
                    const uint32_t box = boxes + (pn % kBoxesPerWarp) * kBox;
                    if (lane == 0) stores_read<kBoxesPerWarp - 1>();  // the store that last used this box
                    __syncwarp();
#pragma unroll
                    for (int hh = 0; hh < kW / 32; ++hh) {
                        float v[32];
                        if (x.rows > 0) tmem_ld32(taddr + c + hh * 32, v);
                        else {
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] = 0.f;
                        }
                        // 64 bytes (32 bf16 values, or 16 of 32 floats) a half of the box's row
#pragma unroll
                        for (int q = 0; q < (F32 ? 8 : 4); ++q) {
                            uint32_t w[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                w[i] = F32 ? __float_as_uint(v[q * 4 + i]) : pack_bf16x2(v[q * 8 + 2 * i], v[q * 8 + 2 * i + 1]);
                            st_shared16(box + lane * 128 + ((((uint32_t)(hh * 4 + q)) ^ sw) << 4), w[0], w[1], w[2], w[3]);
                        }
                    }
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) {
                        if (F32 && p.accumulate) add_3d(&p.o[x.mat], x.n0 + c, m, x.e, box);
                        else store_3d(&p.o[x.mat], x.n0 + c, m, x.e, box);
                        stores_commit();
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
// Expert e's rows of a0, a1 and b as tensor maps of their own, made from the
// maps of the whole tensors.  A warp per expert.
struct MapParams {
    CUtensorMap t[kMapsPerExpert];
    const unsigned char* rows[kMapsPerExpert];  // the tensors
    int64_t row_bytes[kMapsPerExpert];
    unsigned char* maps;
    const int32_t* offsets;
    int M, N;
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

template <bool PAIR, bool F32>
cudaError_t launch_dw(const DwParams& p, int64_t units, int sms, cudaStream_t st) {
    auto kern = grouped_dw_kernel<PAIR, F32>;
    cudaError_t e = allow_max_smem(kern);
    if (e != cudaSuccess) return e;
    int most = sms;
    if constexpr (PAIR) {
        e = resident_pairs(reinterpret_cast<const void*>(kern), kThreads, Cfg<true>::kSmem, sms, &most);
        if (e != cudaSuccess) return e;
        if (most <= 0) return cudaErrorInvalidConfiguration;
    }
    if (units > most) units = most;
    return note_launch(reinterpret_cast<const void*>(kern), kThreads, Cfg<PAIR>::kSmem,
                       launch_units(kern, p, (int)units, PAIR, kThreads, Cfg<PAIR>::kSmem, st));
}

}  // namespace

cudaError_t launch_grouped_dw_tc(const GroupedArgs& a, cudaStream_t st) {
    DwParams p;
    std::memset(&p, 0, sizeof(p));
    p.maps = a.maps; p.offsets = a.offsets; p.err = a.err;
    p.M = a.M; p.N = a.N; p.d = a.d; p.I = a.I;
    p.n_mat = a.o1 ? 2 : 1;
    p.accumulate = a.accumulate;
    const uint64_t d = (uint64_t)a.d, I = (uint64_t)a.I, M = (uint64_t)a.M;
    MapParams mp;
    std::memset(&mp, 0, sizeof(mp));
    const void* rows[kMapsPerExpert] = {a.a0, a.a1 ? a.a1 : a.a0, a.b0};
    for (int i = 0; i < kMapsPerExpert; ++i) {
        const uint64_t cols = i < 2 ? I : d;
        if (encode_bf16_2d(&mp.t[i], rows[i], cols, M, cols * 2, 64, kBK) != MOE_OK) return cudaErrorInvalidValue;
        mp.rows[i] = static_cast<const unsigned char*>(rows[i]);
        mp.row_bytes[i] = (int64_t)cols * 2;
    }
    mp.maps = a.maps; mp.offsets = a.offsets; mp.M = a.M; mp.N = a.N;
    for (int i = 0; i < p.n_mat; ++i)
        if (encode_3d(&p.o[i], !a.out_f32, i ? a.o1 : a.o0, d, I, (uint64_t)a.N, a.out_f32 ? 32 : 64, 32) != MOE_OK)
            return cudaErrorInvalidValue;
    cudaError_t e = launch_pdl(expert_maps_kernel, dim3((a.N + 3) / 4), dim3(128), 0, st, mp);
    if (e != cudaSuccess) return e;
    // a pair's 256 channels, unless the expert has less
    const bool pair = a.I >= 2 * kBM;
    const int tile_rows = pair ? 2 * kBM : kBM;
    const int64_t units = (int64_t)a.N * p.n_mat * ((a.I + tile_rows - 1) / tile_rows) * ((a.d + kBN - 1) / kBN);
    if (pair) return a.out_f32 ? launch_dw<true, true>(p, units, a.sms, st) : launch_dw<true, false>(p, units, a.sms, st);
    return a.out_f32 ? launch_dw<false, true>(p, units, a.sms, st) : launch_dw<false, false>(p, units, a.sms, st);
}

}  // namespace moe
