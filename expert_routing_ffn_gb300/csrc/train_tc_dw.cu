// The weight gradients of the experts' products on the tensor cores: per
// expert, dW = a^T b over its grouped rows (a [M, I]: dg and du, or h; b
// [M, d]: x, or dy), one or two a in a launch.  tcgen05, accumulators in
// tensor memory, fed by TMA.
//
// The channels of all a form strips of 128; a tile is two strips x 256 columns
// on a CTA pair (2-CTA MMA), a strip each, where each CTA stages its strip and
// half of the columns.  (Two strips of different a share a tile at the seam:
// I = 1408 is 11 strips, and dWg and dWu together 11 tiles.)  The rows are the
// K axis, so both operands are MN-major as they lie in memory.  They
// are summed, so a step that ran past the segment would add the next expert's
// rows: each expert has tensor maps of its own whose row count ends with its
// segment (map kernel), and TMA fills the rest of the last step with zeros.
// Every dW is written once, so at the sizes of a training step (a few hundred
// rows an expert) storing it costs as much as the MMAs.  Eight epilogue warps,
// two to a quarter of the accumulator's lanes, take their part of a tile out
// of tensor memory in one go and give the accumulator back before they convert
// and store.  An expert without rows has no tiles: its dW is filled with zeros
// in contiguous pieces at the end.
//
// Tiles are taken round robin by the resident pairs, experts with most rows
// first, so that the pairs end together when the load is skewed.
//
// Block: warp 0 issues the TMA loads, warp 1 the MMAs (of the pair's leader),
// warps 2-9 the epilogue (a thread owns a channel).  Accumulators are
// double-buffered.  Every wait is bounded.
//
// Bound and measurements (GB300): few rows, HBM writes: dWg and dWu of 8 tokens
// in the Mixtral-8x7B shape 298 us for 1.88 GB, 0.93 of the measured copy
// bandwidth.  384 rows an expert (DeepSeek-V2-Lite shape, 4096 tokens), both:
// 976 MB and 283 GFLOP take 144 and 146 us at the burst rates; 235 us measured,
// of which the loads' latency beside the stream of stores is most (without the
// stores 169 us).  Zeroing the foreign rows in shared memory by a warp of its
// own instead of per-expert maps needs a release across the CTAs of a pair that
// costs more than the maps: 303 us.
#include <cuda.h>

#include <cstring>

#include "common.cuh"
#include "tma.h"
#include "train.h"
#include "train_tc.cuh"

namespace moe {

namespace {

using namespace train;

constexpr int kStrip = 128, kBN = 256, kEpiWarps = 8, kThreads = 64 + 32 * kEpiWarps;
constexpr uint32_t kBK = kTcBK;
constexpr uint32_t kStageA = kStrip * kBK * 2, kStageB = kBN / 2 * kBK * 2, kStage = kStageA + kStageB;
constexpr uint32_t kBox = 32 * 128;          // 32 channels x 128 bytes

// BOXES: store boxes of an epilogue warp.  One keeps fewer stores under way and leaves room for a sixth stage:
// 384 rows an expert (DeepSeek-V2-Lite shape), dWg and dWu 249 -> 235 us, one matrix 139 -> 131.  With few rows,
// where the stores are the work, two: 8 tokens 118 us against 125, 96 rows an expert 140 against 153, 160 rows
// 158 against 150.
template <int BOXES>
struct DwCfg {
    static constexpr int kS = BOXES == 1 ? 6 : 5;  // stages
    static constexpr uint32_t kBoxes = kS * kStage, kTable = kBoxes + kEpiWarps * BOXES * kBox;  // table: rank -> expert
    static constexpr uint32_t kBars = kTable + kTrainMaxExperts * 4 + 16;
    static constexpr uint32_t kSmem = kBars + (2 * kS + 5) * 8 + 16;
    static_assert(kSmem <= 232448, "227 KB of shared memory per block");
};

struct DwParams {
    CUtensorMap o[2];
    unsigned char* out[2];
    const unsigned char* maps;  // [N][kMapsPerExpert] tensor maps
    const int32_t* offsets;
    int M, N, d, I, n_mat, accumulate;
    DevError* err;
};

// The tiles of one pair in order: expert by expert (order[] of falling rows,
// those without rows left out), strips outermost, column tiles innermost: the
// rows of dW that consecutive pairs write at a time are contiguous.
struct Walk {
    int e, rows, strip, n0;  // expert, its rows, the pair's first strip, first column
    int place, n_live, mt, nt, mts, nts, d_place, d_mt, d_nt;

    __device__ __forceinline__ bool more() const { return place < n_live; }
    __device__ __forceinline__ void set(const DwParams& p, const int* order, bool new_expert) {
        strip = 2 * mt;
        n0 = nt * kBN;
        if (new_expert && place < n_live) {
            e = order[place];
            const int r0 = min(max(p.offsets[e], 0), p.M);
            rows = max(min(max(p.offsets[e + 1], 0), p.M) - r0, 0);
        }
    }
    __device__ __forceinline__ Walk(const DwParams& p, const int* order, int live, int unit, int n_units) {
        mts = ((p.I + kStrip - 1) / kStrip * p.n_mat + 1) / 2;
        nts = (p.d + kBN - 1) / kBN;
        n_live = live;
        const int per = mts * nts;
        place = unit / per;
        mt = unit % per / nts;
        nt = unit % nts;
        d_place = n_units / per;
        d_mt = n_units % per / nts;
        d_nt = n_units % nts;
        e = rows = 0;
        set(p, order, true);
    }
    __device__ __forceinline__ void next(const DwParams& p, const int* order) {
        const int was = place;
        nt += d_nt;
        mt += d_mt;
        place += d_place;
        if (nt >= nts) { nt -= nts; ++mt; }
        if (mt >= mts) { mt -= mts; ++place; }
        set(p, order, place != was);
    }
};

template <bool F32, int BOXES>
__global__ void __launch_bounds__(kThreads, 1) grouped_dw_kernel(const __grid_constant__ DwParams p) {
    using C = DwCfg<BOXES>;
    constexpr int kS = C::kS;
    extern __shared__ __align__(1024) unsigned char smem[];
    int* order = reinterpret_cast<int*>(smem + C::kTable);  // rank -> expert
    int* live_s = order + kTrainMaxExperts;               // experts with rows
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBars);
    uint64_t *empty = full + kS, *tfull = empty + kS, *tempty = tfull + 2, *drain = tempty + 2;
    uint32_t* tmem_s = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_s + 1);

    grid_dep_wait();  // the previous kernels' outputs; no tensor memory is taken before it
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = smem_u32(smem);
    const uint32_t rank = cluster_rank();
    const bool leader = rank == 0;
    const int unit = (int)(blockIdx.x >> 1), n_units = (int)(gridDim.x >> 1);

    auto rows_of = [&](int e) {
        const int r0 = min(max(p.offsets[e], 0), p.M);
        return max(min(max(p.offsets[e + 1], 0), p.M) - r0, 0);
    };
    {  // experts in order of falling row count (the lower index first among equals)
        int* rows_s = reinterpret_cast<int*>(smem);  // the stages are not in use yet
        for (int e = tid; e < p.N; e += kThreads) rows_s[e] = rows_of(e);
        if (tid == 0) *live_s = 0;
        __syncthreads();
        for (int e = tid; e < p.N; e += kThreads) {
            const int r = rows_s[e];
            int place = 0;
            for (int f = 0; f < p.N; ++f) {
                const int q = rows_s[f];
                place += q > r || (q == r && f < e);
            }
            order[place] = e;
            if (r > 0) atomicMax(live_s, place + 1);
        }
    }
    if (tid == 32) {
        for (int s = 0; s < kS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], 2 * kEpiWarps);  // an arrival per epilogue warp of both CTAs
        }
        mbar_init(drain, 1);
        fence_mbar_init();
        *abort_flag = 0;
        if (base & 1023u) {  // the swizzled tiles need it
            set_error(p.err, MOE_ERR_CAPACITY, 1023);
            *abort_flag = 1;
        }
    }
    if (warp == 1) tmem_alloc(tmem_s);
    fence_proxy_async();  // the row counts' shared memory becomes a stage that TMA writes
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // the peer's barriers are ready before any arrival from here
    tc_fence_after();
    const uint32_t tmem = *tmem_s;
    const int live = *live_s;
    const int strips = (p.I + kStrip - 1) / kStrip;  // of one a
    // this CTA's strip of a tile: which a, and its first channel (past I: no such strip)
    auto strip_of = [&](const Walk& x, int& mat, int& m0) {
        const int q = x.strip + (int)rank;
        mat = q >= strips && p.n_mat > 1;
        m0 = (q - (mat ? strips : 0)) * kStrip;
    };

    if (warp == 0) {
        // ---------------- loads (each CTA its own stages, on the leader's barrier)
        const uint32_t full0 = leader_address(&full[0]);
        int st = 0, it = 0;
        uint32_t phase = 1;
        // The maps of the experts that this pair takes tiles of, an expert a lane: all experts' made
        // the Granite-shaped down gradient 57.3 us instead of 55.0, and each expert's at its first tile, in the loads' way,
        // 11 us of 193 (8 tokens, DeepSeek-V2-Lite shape, up gradient).
        const int per = (strips * p.n_mat + 1) / 2 * ((p.d + kBN - 1) / kBN);  // tiles of an expert
        for (int j = lane; j < live; j += 32) {
            // the pair's first tile from that expert's first tile on
            const int t = unit + (max(j * per - unit, 0) + n_units - 1) / n_units * n_units;
            if (t < (j + 1) * per)
                for (int m = 0; m < kMapsPerExpert; ++m) map_acquire(p.maps + ((size_t)order[j] * kMapsPerExpert + m) * 128);
        }
        __syncwarp();
        for (Walk x(p, order, live, unit, n_units); x.more(); x.next(p, order)) {
            if (__any_sync(0xffffffffu, *abort_flag)) break;
            int mat, m0;
            strip_of(x, mat, m0);
            const int rows = __shfl_sync(0xffffffffu, x.rows, 0), e = __shfl_sync(0xffffffffu, x.e, 0);
            const int n0 = x.n0 + (int)rank * 128;
            const unsigned char* emaps = p.maps + (size_t)e * kMapsPerExpert * 128;
            Walk nx = x;
            nx.next(p, order);
            if (nx.more() && nx.e != x.e && lane < kMapsPerExpert)
                map_prefetch(p.maps + ((size_t)nx.e * kMapsPerExpert + lane) * 128);
            __syncwarp();
            for (int k0 = 0; k0 < rows; k0 += (int)kBK, ++it) {
                // a wait that gives up raises the abort flag, which ends the later ones
                (void)wait<true>(&empty[st], phase, abort_flag, p.err, 1);
                __syncwarp();
                if (elect_one()) {
                    const uint32_t ad = base + st * kStage, bd = ad + kStageA, bar = full0 + st * 8;
                    if (leader) mbar_arrive_expect_tx(&full[st], 2 * kStage);
#pragma unroll
                    for (int j = 0; j < 2; ++j) load_2d<true>(ad + j * 8192, emaps + mat * 128, m0 + j * 64, k0, bar);
#pragma unroll
                    for (int j = 0; j < 2; ++j) load_2d<true>(bd + j * 8192, emaps + 2 * 128, n0 + j * 64, k0, bar);
                }
                __syncwarp();
                if (++st == kS) { st = 0; phase ^= 1; }
            }
        }
        // the leader's MMAs have consumed this CTA's last stages before it may leave
        for (int k = it > kS ? it - kS : 0; k < it; ++k)
            (void)wait<true>(&empty[k % kS], (k / kS) & 1, abort_flag, p.err, 2, false);
    } else if (warp == 1) {
        // ---------------- MMAs (the leader of a pair)
        if (leader) {
            constexpr uint32_t idesc = tc_idesc(2 * kStrip, kBN, 1, 1);
            // 16 rows of 128 bytes a step, the next 64 channels or columns 8 KB on
            const uint64_t da0 = smem_desc(base, 8192, 1024), db0 = smem_desc(base + kStageA, 8192, 1024);
            int st = 0, local = 0;
            uint32_t phase = 0;
            for (Walk x(p, order, live, unit, n_units); x.more(); x.next(p, order), ++local) {
                if (__any_sync(0xffffffffu, *abort_flag)) break;
                const int rows = __shfl_sync(0xffffffffu, x.rows, 0);
                const int ab = local & 1;
                const uint32_t acc = tmem + ab * kBN;
                // a wait that gives up raises the abort flag, which ends the later ones
                (void)wait<true>(&tempty[ab], ((local >> 1) & 1) ^ 1, abort_flag, p.err, 3);
                tc_fence_after();
                for (int k0 = 0; k0 < rows; k0 += (int)kBK) {
                    (void)wait<true>(&full[st], phase, abort_flag, p.err, 4);
                    tc_fence_after();
                    __syncwarp();
                    if (elect_one()) {
                        const uint64_t da = desc_at(da0, st * kStage), db = desc_at(db0, st * kStage);
                        // 16-row steps without a row of the segment are left out
#pragma unroll
                        for (int kk = 0; kk < (int)kBK / 16; ++kk)
                            if (kk == 0 || k0 + kk * 16 < rows)
                                mma(acc, desc_at(da, kk * 2048), desc_at(db, kk * 2048), idesc, (k0 | kk) ? 1u : 0u);
                        commit(&empty[st]);
                    }
                    __syncwarp();
                    if (++st == kS) { st = 0; phase ^= 1; }
                }
                if (elect_one()) commit(&tfull[ab]);
                __syncwarp();
            }
            // every MMA issued here is done before tensor memory is released
            if (elect_one()) commit_local(drain);
            __syncwarp();
            (void)wait<true>(drain, 0, abort_flag, p.err, 6, false);
        }
    } else {
        // ---------------- epilogue: a thread owns a channel of dW, two warps share a quarter of
        // the lanes, 128 columns each
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        const uint32_t boxes = base + C::kBoxes + (warp - 2) * BOXES * kBox;
        const uint32_t sw = lane & 7;  // 128-byte swizzle: chunk j of row i at chunk j ^ (i & 7)
        const uint32_t free0 = leader_address(&tempty[0]), free1 = leader_address(&tempty[1]);
        int local = 0;
        constexpr int kW = F32 ? 32 : 64;  // columns of a box
        for (Walk x(p, order, live, unit, n_units); x.more(); x.next(p, order), ++local) {
            if (__any_sync(0xffffffffu, *abort_flag)) break;
            const int ab = local & 1;
            int mat, m;
            strip_of(x, mat, m);
            m += quarter * 32;  // this warp's first channel
            (void)wait<true>(&tfull[ab], (local >> 1) & 1, abort_flag, p.err, 5);
            tc_fence_after();
            __syncwarp();
            const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + ab * kBN + half * 128;
            uint32_t v[128];
#pragma unroll
            for (int i = 0; i < 4; ++i) tmem_ld32(taddr + i * 32, v + i * 32);
            tmem_ld_wait();
            // the accumulator is free
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (!leader) arrive_cluster(ab ? free1 : free0);
                else mbar_arrive(&tempty[ab]);
            }
            if (m >= p.I) continue;
            // a box at a time; of two, one is filled while the store of the other drains
#pragma unroll
            for (int r = 0; r < 128 / kW; ++r) {
                const uint32_t box = boxes + r % BOXES * kBox;
                if (lane == 0) stores_read<BOXES - 1>();
                __syncwarp();
#pragma unroll
                for (int q = 0; q < 8; ++q) {  // 16 bytes
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        w[i] = F32 ? v[r * kW + q * 4 + i]
                                   : pack_bf16x2(__uint_as_float(v[r * kW + q * 8 + 2 * i]),
                                                 __uint_as_float(v[r * kW + q * 8 + 2 * i + 1]));
                    st_shared16(box + lane * 128 + (((uint32_t)q ^ sw) << 4), w[0], w[1], w[2], w[3]);
                }
                fence_proxy_async();
                __syncwarp();
                const int col = x.n0 + half * 128 + r * kW;
                if (lane == 0) {
                    if (col >= p.d) {
                    } else if (F32 && p.accumulate) add_3d(&p.o[mat], col, m, x.e, box);
                    else store_3d(&p.o[mat], col, m, x.e, box);
                    stores_commit();
                }
            }
        }
        // zeros for the experts without rows, in contiguous pieces of this warp's boxes
        if (!p.accumulate && live < p.N) {
            constexpr uint32_t kPiece = BOXES * kBox;
            if (lane == 0) stores_read<0>();
            __syncwarp();
            for (uint32_t i = lane * 16; i < kPiece; i += 512) st_shared16(boxes + i, 0, 0, 0, 0);
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
                const uint64_t bytes = (uint64_t)p.I * p.d * (F32 ? 4 : 2), pieces = (bytes + kPiece - 1) / kPiece;
                const uint64_t n = pieces * (uint64_t)(p.N - live) * p.n_mat;
                for (uint64_t c = (uint64_t)blockIdx.x * kEpiWarps + (warp - 2); c < n; c += (uint64_t)gridDim.x * kEpiWarps) {
                    const uint64_t which = c / pieces, at = (c - which * pieces) * kPiece;
                    unsigned char* o = p.out[which % p.n_mat] + (uint64_t)order[live + which / p.n_mat] * bytes + at;
                    store_bulk(o, boxes, (uint32_t)min((uint64_t)kPiece, bytes - at));
                    stores_commit();
                }
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
    cluster_sync();
    tc_fence_after();
    if (warp == 1) tmem_free(tmem);
    grid_dep_launch();
}

// ---------------------------------------------------------------- per-expert maps
// By a launch of its own where no other kernel of the call has made them.
__global__ void __launch_bounds__(128) expert_maps_kernel(const __grid_constant__ MapParams p) {
    grid_dep_wait();
    const int e = blockIdx.x * 4 + (threadIdx.x >> 5);
    if (e < p.N) expert_maps(p, e);
    grid_dep_launch();
}

template <bool F32, int BOXES>
cudaError_t launch_dw(const DwParams& p, int sms, cudaStream_t st) {
    auto kern = grouped_dw_kernel<F32, BOXES>;
    constexpr uint32_t kSmem = DwCfg<BOXES>::kSmem;
    cudaError_t e = allow_max_smem(kern);
    if (e != cudaSuccess) return e;
    int most = 0;
    e = resident_clusters(reinterpret_cast<const void*>(kern), 2, kThreads, kSmem, sms, &most);
    if (e != cudaSuccess) return e;
    if (most <= 0) return cudaErrorInvalidConfiguration;
    const int64_t strips = (p.I + kStrip - 1) / kStrip;
    int64_t units = p.N * ((strips * p.n_mat + 1) / 2) * ((p.d + kBN - 1) / kBN);
    if (units > most) units = most;
    return note_launch(reinterpret_cast<const void*>(kern), kThreads, kSmem,
                       launch_units(kern, p, (int)units, 2, kThreads, kSmem, st));
}

}  // namespace

bool dw_map_params(const GroupedArgs& a, MapParams& mp) {
    const void* rows[kMapsPerExpert] = {a.a0, a.a1 ? a.a1 : a.a0, a.b0};
    std::memset(&mp, 0, sizeof(mp));
    for (int i = 0; i < kMapsPerExpert; ++i) {
        const uint64_t cols = (uint64_t)(i < 2 ? a.I : a.d);
        // The template is the map of a single row.  A map encodes more than the fields that are replaced on the
        // device: one bit depends on the tensor's size (clear below 128 KB), and a segment of a few rows under
        // the bit of the whole tensor was read beyond its end, past the allocation.  What is right for one row
        // is right for any segment, which contains it.
        if (encode_bf16_2d(&mp.t[i], rows[i], cols, 1, cols * 2, 64, kBK) != MOE_OK) return false;
        mp.rows[i] = static_cast<const unsigned char*>(rows[i]);
        mp.row_bytes[i] = (int64_t)cols * 2;
    }
    mp.maps = a.maps; mp.offsets = a.offsets; mp.M = a.M; mp.N = a.N;
    return true;
}

cudaError_t launch_grouped_dw_tc(const GroupedArgs& a, bool have_maps, cudaStream_t st) {
    DwParams p;
    std::memset(&p, 0, sizeof(p));
    p.maps = a.maps; p.offsets = a.offsets; p.err = a.err;
    p.M = a.M; p.N = a.N; p.d = a.d; p.I = a.I;
    p.n_mat = a.o1 ? 2 : 1;
    p.accumulate = a.accumulate;
    p.out[0] = static_cast<unsigned char*>(a.o0);
    p.out[1] = static_cast<unsigned char*>(a.o1);
    for (int i = 0; i < p.n_mat; ++i)
        if (encode_3d(&p.o[i], !a.out_f32, p.out[i], (uint64_t)a.d, (uint64_t)a.I, (uint64_t)a.N, a.out_f32 ? 32 : 64, 32) != MOE_OK)
            return cudaErrorInvalidValue;
    if (!have_maps) {
        MapParams mp;
        if (!dw_map_params(a, mp)) return cudaErrorInvalidValue;
        const cudaError_t e = launch_pdl(expert_maps_kernel, dim3((a.N + 3) / 4), dim3(128), 0, st, mp);
        if (e != cudaSuccess) return e;
    }
    const bool few = (long long)a.M <= 128LL * a.N;
    return few ? (a.out_f32 ? launch_dw<true, 2>(p, a.sms, st) : launch_dw<false, 2>(p, a.sms, st))
               : (a.out_f32 ? launch_dw<true, 1>(p, a.sms, st) : launch_dw<false, 1>(p, a.sms, st));
}

}  // namespace moe
