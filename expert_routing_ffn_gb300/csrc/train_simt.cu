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
// that most of a 64-row tile would be padding.  Measured, fp32: 128 rows an
// expert at d = I = 1024, 16 experts, Up: 304 us, 28 TFLOP/s (ragged rows fill
// 0.8 of the tiles, the tiles 0.7 of three rounds); 16 tokens of the tiny
// layer: 11 us.  Tiles are numbered expert by
// expert; every block forms the prefix sums of the tile counts itself.
#include <cuda_bf16.h>

#include "common.cuh"
#include "train.h"

namespace moe {

namespace {

constexpr int kThreads = 256, kBN = 128, kBK = 16, kPitch = kBK + 4, kStages = 3;

struct SimtParams {
    const void *a0, *a1, *b0, *b1, *g, *u;
    void *o0, *o1, *o2;
    const int32_t* offsets;
    int M, N, d, I;
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

__device__ __forceinline__ float sigmoid(float g) { return 1.f / (1.f + expf(-g)); }

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

template <typename W, int FORM, int BM>
__global__ void __launch_bounds__(kThreads) grouped_simt_kernel(const SimtParams p) {
    using C = Cfg<W, FORM, BM>;
    constexpr int kR = BM / 8;  // rows of a lane
    constexpr bool kF32 = sizeof(W) == 4;
    extern __shared__ __align__(16) float stages[];
    __shared__ int row_s[kTrainMaxExperts + 1], tile_s[kTrainMaxExperts + 1];
    const W* tag = nullptr;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    grid_dep_wait();
    for (int e = tid; e <= p.N; e += kThreads) row_s[e] = min(max(p.offsets[e], 0), p.M);
    __syncthreads();
    const int n_cols = C::kNT ? p.I : p.d;
    constexpr int kCols = FORM == kFormUp ? kBN / 2 : kBN;  // output columns of a tile
    const int nt = (n_cols + kCols - 1) / kCols;
    const int n_mat = FORM == kFormDw && p.o1 ? 2 : 1;
    const int mt_w = (p.I + BM - 1) / BM;
    if (tid < 32) {  // tiles before each expert
        int carry = 0;
        for (int b = 0; b < p.N; b += 32) {
            const int e = b + tid;
            int v = 0;
            if (e < p.N) v = FORM == kFormDw ? n_mat * mt_w * nt : (max(row_s[e + 1] - row_s[e], 0) + BM - 1) / BM * nt;
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
    for (int tile = blockIdx.x; tile < tile_s[p.N]; tile += gridDim.x) {
        int lo = 0, hi = p.N;  // the last expert whose tiles start at or before this one
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (tile_s[mid] <= tile) lo = mid;
            else hi = mid;
        }
        const int e = lo, row0 = row_s[e], rows = max(row_s[e + 1] - row0, 0);
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
                if (n >= n_cols) continue;
                const float c = acc[i][j];
                if constexpr (FORM == kFormUp) {
                    const int64_t at = (int64_t)(row0 + m) * p.I + n;
                    const float u = acc[i][j + 2];
                    if (p.o0) { st(p.o0, at, c, tag); st(p.o1, at, u, tag); }
                    st(p.o2, at, c * sigmoid(c) * u, tag);
                } else if constexpr (FORM == kFormDh) {
                    const int64_t at = (int64_t)(row0 + m) * p.I + n;
                    const float g = ld(p.g, at, tag), u = ld(p.u, at, tag), sg = sigmoid(g);
                    st(p.o0, at, c * u * sg * (1.f + g * (1.f - sg)), tag);
                    st(p.o1, at, c * g * sg, tag);
                } else if constexpr (FORM == kFormDw) {
                    const int64_t at = w0 + (int64_t)m * p.d + n;
                    void* o = mat ? p.o1 : p.o0;
                    if (p.out_f32) {
                        float* f = static_cast<float*>(o) + at;
                        *f = p.accumulate ? *f + c : c;
                    } else st(o, at, c, tag);
                } else st(p.o0, (int64_t)(row0 + m) * p.d + n, c, tag);
            }
        }
    }
    if constexpr (FORM != kFormDw) {  // rows of no expert
        const int64_t first = (int64_t)row_s[p.N] * n_cols, last = (int64_t)p.M * n_cols;
        for (int64_t i = first + (int64_t)blockIdx.x * kThreads + tid; i < last; i += (int64_t)gridDim.x * kThreads) {
            if (p.o0) st(p.o0, i, 0.f, tag);
            if (p.o1) st(p.o1, i, 0.f, tag);
            if (p.o2) st(p.o2, i, 0.f, tag);
        }
    }
    grid_dep_launch();
}

template <typename W, int FORM, int BM>
cudaError_t launch_tiles(const GroupedArgs& a, const SimtParams& p, cudaStream_t stream) {
    auto kern = grouped_simt_kernel<W, FORM, BM>;
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

template <typename W, int FORM>
cudaError_t launch_form(const GroupedArgs& a, const SimtParams& p, cudaStream_t stream) {
    // Dw's tile rows are channels, of which there are many
    if (FORM != kFormDw && (int64_t)a.M <= 24LL * a.N) return launch_tiles<W, FORM, 16>(a, p, stream);
    return launch_tiles<W, FORM, 64>(a, p, stream);
}

template <typename W>
cudaError_t launch(const GroupedArgs& a, const SimtParams& p, cudaStream_t stream) {
    switch (a.form) {
        case kFormUp: return launch_form<W, kFormUp>(a, p, stream);
        case kFormDown: return launch_form<W, kFormDown>(a, p, stream);
        case kFormDh: return launch_form<W, kFormDh>(a, p, stream);
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
    p.M = a.M; p.N = a.N; p.d = a.d; p.I = a.I; p.out_f32 = a.out_f32; p.accumulate = a.accumulate;
    p.vec = !a.bf16 && a.d % 4 == 0 && a.I % 4 == 0;
    for (const void* q : {a.a0, a.a1, a.b0, a.b1}) p.vec = p.vec && (reinterpret_cast<uintptr_t>(q) & 15u) == 0;
    return a.bf16 ? launch<__nv_bfloat16>(a, p, stream) : launch<float>(a, p, stream);
}

}  // namespace moe
