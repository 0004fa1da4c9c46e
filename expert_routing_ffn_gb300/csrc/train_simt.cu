// The experts' grouped products on the CUDA cores, in fp32 arithmetic: for
// fp32 layers, and for bf16 layers whose sizes or addresses TMA cannot take
// (rows that do not start on 16-byte boundaries).  Every size and alignment.
//
// A block of 8 warps computes tiles of 64 (or 16) rows x 128 columns, 16 deep
// at a time: a warp owns 8 (2) rows, a lane 4 columns.  A lane's values of the
// left operand are the warp's (broadcast reads), so per step of K a warp reads
// 6 wavefronts of shared memory for 32 FMAs a lane.  Both operands lie in
// shared memory as they do in global memory, so fp32 stages come by cp.async,
// three in flight, without passing through registers; bf16 ones are converted
// on the way.  Rows that hold K contiguously are padded to 20 floats, which
// puts the 16-byte reads of eight lanes on different banks.
//
// Bound: FMA rate.  The 16-row tiles serve segments that average so few rows
// that most of a 64-row tile would be padding; with fewer still, or without
// 16-byte loads, grouped_few_kernel streams the weights past eight rows.
// Measured, fp32: 128 rows an expert at d = I = 1024, 16 experts, Up: 297 us, 29
// TFLOP/s (ragged rows fill 0.8 of the tiles, the tiles 0.7 of three rounds).
// Tiles are numbered expert by expert; every block forms the prefix sums of the
// tile counts itself.
#include <cuda_bf16.h>

#include "common.cuh"
#include "pack8.cuh"
#include "train.h"

namespace moe {

namespace {

constexpr int kThreads = 256, kBN = 128, kBK = 16, kPitch = kBK + 4, kStages = 3;

struct SimtParams {
    const void *a0, *a1, *b0, *b1, *g, *u;
    void *o0, *o1, *o2;
    const uint8_t *gs, *us;  // PACKED: the scales of g, u (Dh) or of o0, o1 (Up)
    uint8_t *s0, *s1;
    const int32_t* offsets;
    int M, N, d, I, nb;      // nb: blocks of a packed row
    int out_f32, accumulate;
    int vec;  // fp32: every row of every operand starts on a 16-byte boundary
};

__device__ __forceinline__ float ld(const void* p, int64_t i, const float*) { return static_cast<const float*>(p)[i]; }
__device__ __forceinline__ float ld(const void* p, int64_t i, const __nv_bfloat16*) {
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ __forceinline__ void st(void* p, int64_t i, float v, const float*) { static_cast<float*>(p)[i] = v; }
__device__ __forceinline__ void st(void* p, int64_t i, float v, const __nv_bfloat16*) {
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// 1 / (1 + e^-g) = e^g / (1 + e^g), of the two the one whose exponential is at most 1: e^-g is infinite from
// g = -88.73 on, where h, dg and du are still numbers of the type
__device__ __forceinline__ float sigmoid(float g) {
    const float e = expf(-fabsf(g));
    return (g < 0.f ? e : 1.f) / (1.f + e);
}

// 16 or 4 bytes global -> shared, zeros where `in` is false (nothing is read then)
__device__ __forceinline__ void copy16(float* dst, const float* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(float* dst, const float* src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(in ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// FORM Up:   [C0 | C1] = a0 [b0 ; b1]^T   rows x I (64 columns of each a tile), K = d
//      Down: C = a0 b0                    rows x d, K = I
//      Dh:   C = a0 b0^T                  rows x I, K = d
//      Dx:   C = a0 b0 + a1 b1            rows x d, K = I twice
//      Dw:   C = a^T b0                   I x d, K = the expert's rows; one or two a
template <typename W, int FORM, int BM>
struct Cfg {
    static constexpr bool kNT = FORM == kFormUp || FORM == kFormDh;  // b holds K contiguously
    static constexpr bool kTN = FORM == kFormDw;                      // a holds its rows contiguously
    static constexpr int kA = kTN ? kBK * BM : BM * kPitch;            // floats of a stage
    static constexpr int kB = kNT ? kBN * kPitch : kBK * kBN;
    static constexpr int kStage = kA + kB;
    static constexpr int kSmem = kStages * kStage * 4;
};

// row_s: the experts' first rows, tile_s: the tiles before each expert, of(its rows) each
template <typename F>
__device__ __forceinline__ void count_tiles(const SimtParams& p, int* row_s, int* tile_s, F of) {
    const int tid = threadIdx.x;
    for (int e = tid; e <= p.N; e += kThreads) row_s[e] = min(max(p.offsets[e], 0), p.M);
    __syncthreads();
    if (tid < 32) {
        int carry = 0;
        for (int b = 0; b < p.N; b += 32) {
            const int e = b + tid;
            const int v = e < p.N ? of(max(row_s[e + 1] - row_s[e], 0)) : 0;
            int inc = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, inc, o);
                if (tid >= o) inc += x;
            }
            if (e < p.N) tile_s[e] = carry + inc - v;
            carry += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (tid == 0) tile_s[p.N] = carry;
    }
    __syncthreads();
}
// the last expert whose tiles start at or before this one
__device__ __forceinline__ int expert_of(const int* tile_s, int N, int tile) {
    int lo = 0, hi = N;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (tile_s[mid] <= tile) lo = mid;
        else hi = mid;
    }
    return lo;
}
// the products that give rows: value c (Up: g, and u) of a grouped row and a column
template <typename W, int FORM, bool PACKED>
__device__ __forceinline__ void emit(const SimtParams& p, int64_t row, int n, float c, float u) {
    const W* tag = nullptr;
    if constexpr (FORM == kFormUp) {
        static_assert(!PACKED, "a block at a time: emit_block");
        const int64_t at = row * p.I + n;
        if (p.o0) { st(p.o0, at, c, tag); st(p.o1, at, u, tag); }
        st(p.o2, at, c * sigmoid(c) * u, tag);
    } else if constexpr (FORM == kFormDh) {
        const int64_t at = row * p.I + n;
        float g, v;
        if constexpr (PACKED) {
            g = pack8::value_at(static_cast<const int8_t*>(p.g), p.gs, row, n, p.nb);
            v = pack8::value_at(static_cast<const int8_t*>(p.u), p.us, row, n, p.nb);
        } else {
            g = ld(p.g, at, tag);
            v = ld(p.u, at, tag);
        }
        const float sg = sigmoid(g);
        if constexpr (PACKED) st(p.o2, at, g * sg * v, tag);
        st(p.o0, at, c * v * sg * (1.f + g * (1.f - sg)), tag);
        st(p.o1, at, c * g * sg, tag);
    } else st(p.o0, row * p.d + n, c, tag);
}
// Up, PACKED: the g and u of one block of a row, a column a lane (zeros past the last column)
template <typename W>
__device__ __forceinline__ void emit_block(const SimtParams& p, int64_t row, int n, float g, float u) {
    const W* tag = nullptr;
    const int lane = threadIdx.x & 31;
    if (n - lane >= p.I) return;  // the same for the warp
    const int64_t at = row * p.nb + n / 32;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        const float v = which ? u : g;
        const uint32_t E = pack8::exponent(__reduce_max_sync(0xffffffffu, pack8::magnitude(v)));
        int8_t* q = static_cast<int8_t*>(which ? p.o1 : p.o0) + at * 32;
        q[4 * (lane & 7) + (lane >> 3)] = E == 255u ? 0 : (int8_t)pack8::quantise(pack8::within(v, E), pack8::to_steps(E));
        if (lane == 0) (which ? p.s1 : p.s0)[at] = (uint8_t)E;
    }
    if (n < p.I) st(p.o2, row * p.I + n, g * sigmoid(g) * u, tag);
}
// zeros for the rows of no expert
template <typename W, bool PACKED_UP>
__device__ __forceinline__ void zero_rest(const SimtParams& p, int first_row, int n_cols) {
    const W* tag = nullptr;
    const int64_t first = (int64_t)first_row * n_cols, last = (int64_t)p.M * n_cols;
    const int64_t start = (int64_t)blockIdx.x * kThreads + threadIdx.x, step = (int64_t)gridDim.x * kThreads;
    for (int64_t i = first + start; i < last; i += step) {
        if (p.o0 && !PACKED_UP) st(p.o0, i, 0.f, tag);
        if (p.o1 && !PACKED_UP) st(p.o1, i, 0.f, tag);
        if (p.o2) st(p.o2, i, 0.f, tag);
    }
    if constexpr (PACKED_UP) {
        for (int64_t i = (int64_t)first_row * p.nb + start; i < (int64_t)p.M * p.nb; i += step) {
            for (void* o : {p.o0, p.o1}) {
                uint4* q = static_cast<uint4*>(o) + 2 * i;
                q[0] = q[1] = make_uint4(0, 0, 0, 0);
            }
            p.s0[i] = p.s1[i] = 0;
        }
    }
}

template <typename W, int FORM, int BM, bool PACKED>
__global__ void __launch_bounds__(kThreads) grouped_simt_kernel(const SimtParams p) {
    using C = Cfg<W, FORM, BM>;
    constexpr int kR = BM / 8;  // rows of a lane
    constexpr bool kF32 = sizeof(W) == 4;
    extern __shared__ __align__(16) float stages[];
    __shared__ int row_s[kTrainMaxExperts + 1], tile_s[kTrainMaxExperts + 1];
    const W* tag = nullptr;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    grid_dep_wait();
    const int n_cols = C::kNT ? p.I : p.d;
    constexpr int kCols = FORM == kFormUp ? kBN / 2 : kBN;  // output columns of a tile
    const int nt = (n_cols + kCols - 1) / kCols;
    const int n_mat = FORM == kFormDw && p.o1 ? 2 : 1;
    const int mt_w = (p.I + BM - 1) / BM;
    count_tiles(p, row_s, tile_s,
                [&](int rows) { return FORM == kFormDw ? n_mat * mt_w * nt : (rows + BM - 1) / BM * nt; });
    for (int tile = blockIdx.x; tile < tile_s[p.N]; tile += gridDim.x) {
        const int e = expert_of(tile_s, p.N, tile), row0 = row_s[e], rows = max(row_s[e + 1] - row0, 0);
        int local = tile - tile_s[e];
        const int mts = FORM == kFormDw ? mt_w : (rows + BM - 1) / BM;
        const int mat = local / (mts * nt);
        local -= mat * mts * nt;
        const int m0 = local % mts * BM, n0 = local / mts * kCols;
        const int m_end = FORM == kFormDw ? p.I : rows;
        const int K = FORM == kFormDw ? rows : C::kNT ? p.d : p.I;
        const int64_t w0 = (int64_t)e * p.I * p.d;
        const int parts = FORM == kFormDx ? 2 : 1;
        const int steps1 = (K + kBK - 1) / kBK, steps = steps1 * parts;

        // stage `step` of the operands into buffer step % kStages
        auto fetch = [&](int step) {
            float* As = stages + step % kStages * C::kStage;
            float* Bs = As + C::kA;
            const int part = FORM == kFormDx && step >= steps1;
            const int k0 = (step - part * steps1) * kBK;
            const void* A = FORM == kFormDw ? (mat ? p.a1 : p.a0) : part ? p.a1 : p.a0;
            // element (i, k) of either operand: its place in global memory and in the stage, and whether it exists
            auto a_at = [&](int m, int k, int64_t& g, int& s) {
                g = C::kTN ? (int64_t)(row0 + k0 + k) * p.I + m0 + m : (int64_t)(row0 + m0 + m) * K + k0 + k;
                s = C::kTN ? k * BM + m : m * kPitch + k;
                return k0 + k < K && m0 + m < m_end;
            };
            auto b_at = [&](int n, int k, const void*& B, int64_t& g, int& s) {
                B = part ? p.b1 : p.b0;
                int c = n;
                if (FORM == kFormUp && n >= kCols) { B = p.b1; c = n - kCols; }
                g = C::kNT ? w0 + (int64_t)(n0 + c) * K + k0 + k
                  : C::kTN ? (int64_t)(row0 + k0 + k) * p.d + n0 + c : w0 + (int64_t)(k0 + k) * p.d + n0 + c;
                s = C::kNT ? n * kPitch + k : k * kBN + n;
                return k0 + k < K && n0 + c < n_cols;
            };
            if constexpr (kF32) {
                if (p.vec) {
#pragma unroll
                    for (int i = tid; i < BM * kBK / 4; i += kThreads) {
                        const int m = C::kTN ? i % (BM / 4) * 4 : i / (kBK / 4), k = C::kTN ? i / (BM / 4) : i % (kBK / 4) * 4;
                        int64_t g; int s;
                        const bool in = a_at(m, k, g, s);
                        copy16(As + s, static_cast<const float*>(A) + (in ? g : 0), in);
                    }
#pragma unroll
                    for (int i = tid; i < kBN * kBK / 4; i += kThreads) {
                        const int n = C::kNT ? i / (kBK / 4) : i % (kBN / 4) * 4, k = C::kNT ? i % (kBK / 4) * 4 : i / (kBN / 4);
                        int64_t g; int s; const void* B;
                        const bool in = b_at(n, k, B, g, s);
                        copy16(Bs + s, static_cast<const float*>(B) + (in ? g : 0), in);
                    }
                } else {
                    for (int i = tid; i < BM * kBK; i += kThreads) {
                        const int m = C::kTN ? i % BM : i / kBK, k = C::kTN ? i / BM : i % kBK;
                        int64_t g; int s;
                        const bool in = a_at(m, k, g, s);
                        copy4(As + s, static_cast<const float*>(A) + (in ? g : 0), in);
                    }
                    for (int i = tid; i < kBN * kBK; i += kThreads) {
                        const int n = C::kNT ? i / kBK : i % kBN, k = C::kNT ? i % kBK : i / kBN;
                        int64_t g; int s; const void* B;
                        const bool in = b_at(n, k, B, g, s);
                        copy4(Bs + s, static_cast<const float*>(B) + (in ? g : 0), in);
                    }
                }
            } else {
#pragma unroll 4
                for (int i = tid; i < BM * kBK; i += kThreads) {
                    const int m = C::kTN ? i % BM : i / kBK, k = C::kTN ? i / BM : i % kBK;
                    int64_t g; int s;
                    const bool in = a_at(m, k, g, s);
                    As[s] = in ? ld(A, g, tag) : 0.f;
                }
#pragma unroll 4
                for (int i = tid; i < kBN * kBK; i += kThreads) {
                    const int n = C::kNT ? i / kBK : i % kBN, k = C::kNT ? i % kBK : i / kBN;
                    int64_t g; int s; const void* B;
                    const bool in = b_at(n, k, B, g, s);
                    Bs[s] = in ? ld(B, g, tag) : 0.f;
                }
            }
        };

        float acc[kR][4];
#pragma unroll
        for (int i = 0; i < kR; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll
        for (int s = 0; s < kStages - 1; ++s) {
            if (s < steps) fetch(s);
            copies_commit();
        }
        for (int s = 0; s < steps; ++s) {
            copies_wait<kStages - 2>();
            __syncthreads();  // this stage has arrived for every thread, the last one has been read
            if (s + kStages - 1 < steps) fetch(s + kStages - 1);
            copies_commit();
            const float* As = stages + s % kStages * C::kStage;
            const float* Bs = As + C::kA;
#pragma unroll
            for (int k = 0; k < kBK; k += 4) {
                float a[kR][4], b[4][4];  // a[row][k], b[column][k]
                if constexpr (C::kTN) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int i = 0; i < kR; ++i) a[i][q] = As[(k + q) * BM + warp * kR + i];
                } else {
#pragma unroll
                    for (int i = 0; i < kR; ++i)
                        *reinterpret_cast<float4*>(a[i]) = *reinterpret_cast<const float4*>(As + (warp * kR + i) * kPitch + k);
                }
                if constexpr (C::kNT) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *reinterpret_cast<float4*>(b[j]) = *reinterpret_cast<const float4*>(Bs + (lane + 32 * j) * kPitch + k);
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float4 v = *reinterpret_cast<const float4*>(Bs + (k + q) * kBN + lane * 4);
                        b[0][q] = v.x; b[1][q] = v.y; b[2][q] = v.z; b[3][q] = v.w;
                    }
                }
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int i = 0; i < kR; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i][q], b[j][q], acc[i][j]);
            }
        }
        copies_wait<0>();
        __syncthreads();  // before the next tile's first stages
#pragma unroll
        for (int i = 0; i < kR; ++i) {
            const int m = m0 + warp * kR + i;
            if (m >= m_end) continue;
#pragma unroll
            for (int j = 0; j < (FORM == kFormUp ? 2 : 4); ++j) {
                const int n = n0 + (C::kNT ? lane + 32 * j : lane * 4 + j);
                if constexpr (FORM == kFormUp && PACKED) {
                    emit_block<W>(p, row0 + m, n, acc[i][j], acc[i][j + 2]);
                    continue;
                }
                if (n >= n_cols) continue;
                const float c = acc[i][j];
                if constexpr (FORM == kFormDw) {
                    const int64_t at = w0 + (int64_t)m * p.d + n;
                    void* o = mat ? p.o1 : p.o0;
                    if (p.out_f32) {
                        float* f = static_cast<float*>(o) + at;
                        *f = p.accumulate ? *f + c : c;
                    } else st(o, at, c, tag);
                } else if constexpr (!(FORM == kFormUp && PACKED))
                    emit<W, FORM, PACKED>(p, row0 + m, n, c, FORM == kFormUp ? acc[i][j + (FORM == kFormUp ? 2 : 0)] : 0.f);
            }
        }
    }
    if constexpr (FORM != kFormDw) zero_rest<W, FORM == kFormUp && PACKED>(p, row_s[p.N], n_cols);
    grid_dep_launch();
}

// ---------------------------------------------------------------- few rows an expert
// Eight rows against weights that are read once, straight into registers, each
// value for eight FMAs: a stream of the weights, where the tiles above spend
// their time on shared memory.  16 tokens of the tiny layer: Up 10.9 -> 7.9 us
// (the call's host time is 6.5), Dx 34 -> 10.5; 32 tokens of d 511, I 301 in
// bf16, Up 36 -> 7.6.  Bound: the loads' latency, a block an SM (4 rows an
// expert at d = I = 1024, Dh: 25 us for 67 MB, 0.39 of the copy bandwidth).
// The rows wait in shared memory, kFewK values of K at a time.
//   K contiguous (Up, Dh): a warp owns eight rows of the weights (Up: four of
//   either matrix), a lane every 32nd group of four values of K; the 64 sums
//   of a warp are added over its lanes by a halving exchange that leaves two to
//   a lane, in Up the g and u of one channel.
//   columns contiguous (Down, Dx): a half-warp owns every 16th value of K, a
//   lane four columns; the sixteen sums of an output are added in order.
constexpr int kFewRows = 8, kFewK = 512;

// four values of a weight row from i on; `left` of the row are there (VEC: none or four at least)
template <typename W, bool VEC>
__device__ __forceinline__ void load4(const void* p, int64_t i, int left, float (&v)[4]) {
    const W* tag = nullptr;
    if constexpr (VEC) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (left > 0) x = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = j < left ? ld(p, i + j, tag) : 0.f;
    }
}

template <typename W, int FORM, bool VEC, bool PACKED>
__global__ void __launch_bounds__(kThreads) grouped_few_kernel(const SimtParams p) {
    constexpr bool kNT = FORM == kFormUp || FORM == kFormDh;
    constexpr int kCols = FORM == kFormUp ? 32 : 64, kParts = FORM == kFormDx ? 2 : 1;
    constexpr int kSums = kThreads / 16;  // of an output (columns contiguous)
    __shared__ __align__(16) float sm[kNT ? kFewK * kFewRows : kSums * kFewRows * kCols];  // the rows, then the sums
    static_assert(kSums * kFewRows * 64 >= kFewK * kFewRows, "room for the rows");
    __shared__ int row_s[kTrainMaxExperts + 1], tile_s[kTrainMaxExperts + 1];
    const W* tag = nullptr;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n_cols = kNT ? p.I : p.d, K = kNT ? p.d : p.I, nt = (n_cols + kCols - 1) / kCols;
    grid_dep_wait();
    count_tiles(p, row_s, tile_s, [&](int rows) { return (rows + kFewRows - 1) / kFewRows * nt; });
    for (int tile = blockIdx.x; tile < tile_s[p.N]; tile += gridDim.x) {
        const int e = expert_of(tile_s, p.N, tile), rows = max(row_s[e + 1] - row_s[e], 0);
        const int local = tile - tile_s[e], mts = (rows + kFewRows - 1) / kFewRows;
        const int m0 = local % mts * kFewRows, n0 = local / mts * kCols, n_rows = min(rows - m0, kFewRows);
        const int64_t first = row_s[e] + m0, w0 = (int64_t)e * p.I * p.d;
        float acc[kNT ? 64 : 32];  // [row][weight row] or [row][column]
#pragma unroll
        for (int i = 0; i < (kNT ? 64 : 32); ++i) acc[i] = 0.f;
        for (int part = 0; part < kParts; ++part) {
            const void *A = part ? p.a1 : p.a0, *B = part ? p.b1 : p.b0;
            for (int k0 = 0; k0 < K; k0 += kFewK) {
                const int kc = min(kFewK, K - k0);
                __syncthreads();
#pragma unroll
                for (int j = 0; j < kFewK * kFewRows / kThreads; ++j) {
                    const int i = j * kThreads + tid, r = i / kFewK, k = i % kFewK;
                    sm[kNT ? i : k * kFewRows + r] = r < n_rows && k < kc ? ld(A, (first + r) * K + k0 + k, tag) : 0.f;
                }
                __syncthreads();
                if constexpr (kNT) {
#pragma unroll 1
                    for (int k = lane * 4; k < kc; k += 128) {
                        float w[8][4];
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const int n = n0 + (FORM == kFormUp ? warp * 4 + c / 2 : warp * 8 + c);
                            load4<W, VEC>(FORM == kFormUp && c % 2 ? p.b1 : B, w0 + (int64_t)n * K + k0 + k,
                                          n < n_cols ? kc - k : 0, w[c]);
                        }
#pragma unroll
                        for (int r = 0; r < kFewRows; ++r) {
                            const float4 x = *reinterpret_cast<const float4*>(sm + r * kFewK + k);
#pragma unroll
                            for (int c = 0; c < 8; ++c)
                                acc[r * 8 + c] = fmaf(x.w, w[c][3], fmaf(x.z, w[c][2], fmaf(x.y, w[c][1], fmaf(x.x, w[c][0], acc[r * 8 + c]))));
                        }
                    }
                } else {
                    const int n = n0 + lane % 16 * 4;
#pragma unroll 8
                    for (int k = tid / 16; k < kc; k += kSums) {
                        float w[4];
                        load4<W, VEC>(B, w0 + (int64_t)(k0 + k) * p.d + n, n_cols - n, w);
                        float x[kFewRows];
                        *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(sm + k * kFewRows);
                        *reinterpret_cast<float4*>(x + 4) = *reinterpret_cast<const float4*>(sm + k * kFewRows + 4);
#pragma unroll
                        for (int r = 0; r < kFewRows; ++r)
#pragma unroll
                            for (int j = 0; j < 4; ++j) acc[r * 4 + j] = fmaf(x[r], w[j], acc[r * 4 + j]);
                    }
                }
            }
        }
        if constexpr (kNT) {
            // lane L ends with sums 2 L and 2 L + 1: row L / 4
#pragma unroll
            for (int o = 16, n = 32; o > 0; o >>= 1, n >>= 1)
#pragma unroll
                for (int i = 0; i < n; ++i) {
                    const float keep = lane & o ? acc[i + n] : acc[i], give = lane & o ? acc[i] : acc[i + n];
                    acc[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                }
            const int r = lane / 4, n = n0 + warp * (FORM == kFormUp ? 4 : 8) + lane % 4 * (FORM == kFormUp ? 1 : 2);
            if constexpr (FORM == kFormUp && PACKED) {
                // the tile is one block of 32 channels: a row a warp, through shared memory
                static_assert(kCols == 32, "a block of packed values");
                __syncthreads();
                sm[r * 32 + n - n0] = acc[0];
                sm[kFewRows * 32 + r * 32 + n - n0] = acc[1];
                __syncthreads();
                if (warp < n_rows) emit_block<W>(p, first + warp, n0 + lane, sm[warp * 32 + lane], sm[kFewRows * 32 + warp * 32 + lane]);
            } else {
                if (r < n_rows && n < n_cols) emit<W, FORM, PACKED>(p, first + r, n, acc[0], acc[1]);
                if (FORM == kFormDh && r < n_rows && n + 1 < n_cols) emit<W, FORM, PACKED>(p, first + r, n + 1, acc[1], 0.f);
            }
        } else {
            __syncthreads();
#pragma unroll
            for (int r = 0; r < kFewRows; ++r)
                *reinterpret_cast<float4*>(sm + (tid / 16 * kFewRows + r) * kCols + lane % 16 * 4) =
                    make_float4(acc[r * 4], acc[r * 4 + 1], acc[r * 4 + 2], acc[r * 4 + 3]);
            __syncthreads();
            for (int i = tid; i < kFewRows * kCols; i += kThreads) {
                const int r = i / kCols, n = n0 + i % kCols;
                float c = 0.f;
#pragma unroll
                for (int q = 0; q < kSums; ++q) c += sm[q * kFewRows * kCols + i];
                if (r < n_rows && n < n_cols) emit<W, FORM, PACKED>(p, first + r, n, c, 0.f);
            }
        }
    }
    zero_rest<W, FORM == kFormUp && PACKED>(p, row_s[p.N], n_cols);
    grid_dep_launch();
}

template <typename W, int FORM, bool PACKED>
cudaError_t launch_few(const GroupedArgs& a, const SimtParams& p, cudaStream_t stream) {
    constexpr int kCols = FORM == kFormUp ? 32 : 64;
    const int64_t nt = ((FORM == kFormUp || FORM == kFormDh ? a.I : a.d) + kCols - 1) / kCols;
    int64_t tiles = ((int64_t)a.M / kFewRows + (a.N < a.M ? a.N : a.M)) * nt;
    if (tiles > (int64_t)a.sms * 8) tiles = (int64_t)a.sms * 8;
    const dim3 grid((unsigned)(tiles < 1 ? 1 : tiles));
    if constexpr (sizeof(W) == 4)
        if (p.vec) return launch_pdl(grouped_few_kernel<W, FORM, true, PACKED>, grid, dim3(kThreads), 0, stream, p);
    return launch_pdl(grouped_few_kernel<W, FORM, false, PACKED>, grid, dim3(kThreads), 0, stream, p);
}

template <typename W, int FORM, int BM, bool PACKED>
cudaError_t launch_tiles(const GroupedArgs& a, const SimtParams& p, cudaStream_t stream) {
    auto kern = grouped_simt_kernel<W, FORM, BM, PACKED>;
    constexpr int kSmem = Cfg<W, FORM, BM>::kSmem;
    cudaError_t e = allow_max_smem(kern);
    if (e != cudaSuccess) return e;
    const int n_cols = Cfg<W, FORM, BM>::kNT ? a.I : a.d, cols = FORM == kFormUp ? kBN / 2 : kBN;
    const int64_t nt = (n_cols + cols - 1) / cols;
    int64_t tiles = FORM == kFormDw ? (int64_t)a.N * (a.o1 ? 2 : 1) * ((a.I + BM - 1) / BM) * nt
                                    : ((int64_t)a.M / BM + (a.N < a.M ? a.N : a.M)) * nt;
    if (tiles > (int64_t)a.sms * 8) tiles = (int64_t)a.sms * 8;
    return note_launch(reinterpret_cast<const void*>(kern), kThreads, kSmem,
                       launch_pdl(kern, dim3((unsigned)(tiles < 1 ? 1 : tiles)), dim3(kThreads), kSmem, stream, p));
}

template <typename W, int FORM, bool PACKED = false>
cudaError_t launch_form(const GroupedArgs& a, const SimtParams& p, cudaStream_t stream) {
    // Dw's tile rows are channels, of which there are many.  Of the others, few rows an expert by the batch's
    // average, dropped slots included; the limits were measured at one size with 16-byte loads and one without, and
    // other sizes may cross over elsewhere.  fp32 at d = I = 1024, 16 experts, few against 16-row tiles, us, at 4, 8
    // and 16 rows: Up 47 60, 59 60, 96 76; Dx 49 73, 90 73, 125 118; Dh 25 53, 36 43, 56 66; 64-row tiles pass the
    // 16-row ones at 40 rows (Up 119 both, at 16 rows 119 against 79).  Without 16-byte loads, against 64-row tiles,
    // at 25, 64 and 128 rows of d 511, I 301: Up 14 60, 34 61, 60 62; Dx 20 63, 39 64, 69 64.
    if constexpr (FORM != kFormDw) {
        const int few = !p.vec ? 96 : FORM == kFormDh ? 16 : 6;
        if ((int64_t)a.M <= (int64_t)few * a.N) return launch_few<W, FORM, PACKED>(a, p, stream);
        if constexpr (sizeof(W) == 4)
            if (p.vec && (int64_t)a.M <= 24LL * a.N) return launch_tiles<W, FORM, 16, PACKED>(a, p, stream);
    }
    return launch_tiles<W, FORM, 64, PACKED>(a, p, stream);
}

template <typename W>
cudaError_t launch(const GroupedArgs& a, const SimtParams& p, cudaStream_t stream) {
    switch (a.form) {
        case kFormUp: return a.packed ? launch_form<W, kFormUp, true>(a, p, stream) : launch_form<W, kFormUp>(a, p, stream);
        case kFormDown: return launch_form<W, kFormDown>(a, p, stream);
        case kFormDh: return a.packed ? launch_form<W, kFormDh, true>(a, p, stream) : launch_form<W, kFormDh>(a, p, stream);
        case kFormDx: return launch_form<W, kFormDx>(a, p, stream);
        case kFormDw: return launch_form<W, kFormDw>(a, p, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_grouped_simt(const GroupedArgs& a, cudaStream_t stream) {
    SimtParams p;
    p.a0 = a.a0; p.a1 = a.a1; p.b0 = a.b0; p.b1 = a.b1; p.g = a.g; p.u = a.u;
    p.o0 = a.o0; p.o1 = a.o1; p.o2 = a.o2; p.offsets = a.offsets;
    p.gs = a.gs; p.us = a.us; p.s0 = a.s0; p.s1 = a.s1; p.nb = pack_blocks(a.I);
    p.M = a.M; p.N = a.N; p.d = a.d; p.I = a.I; p.out_f32 = a.out_f32; p.accumulate = a.accumulate;
    p.vec = !a.bf16 && a.d % 4 == 0 && a.I % 4 == 0;
    for (const void* q : {a.a0, a.a1, a.b0, a.b1}) p.vec = p.vec && (reinterpret_cast<uintptr_t>(q) & 15u) == 0;
    return a.bf16 ? launch<__nv_bfloat16>(a, p, stream) : launch<float>(a, p, stream);
}

}  // namespace moe
