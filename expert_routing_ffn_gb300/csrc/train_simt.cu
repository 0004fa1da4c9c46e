// The experts' grouped products on the CUDA cores, in fp32 arithmetic: for
// fp32 layers, and for bf16 layers whose sizes or addresses TMA cannot take
// (rows that do not start on 16-byte boundaries).  Every size and alignment.
//
// A block computes 64 x 64 tiles of the output, 256 threads with 4 x 4
// accumulators each, the operands staged through shared memory 16 deep with
// the next stage's loads in flight.  Tiles are numbered expert by expert
// (a segment of rows has ceil(rows / 64) row tiles); every block forms the
// prefix sums of the tile counts from expert_offsets itself.
#include <cuda_bf16.h>

#include "common.cuh"
#include "train.h"

namespace moe {

namespace {

constexpr int kThreads = 256, kBM = 64, kBN = 64, kBK = 16;

struct SimtParams {
    const void *a0, *a1, *b0, *b1, *g, *u;
    void *o0, *o1, *o2;
    const int32_t* offsets;
    int M, N, d, I;
    int out_f32, accumulate;
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

// FORM Up:   C0 = a0 b0^T, C1 = a0 b1^T        rows x I, K = d
//      Down: C0 = a0 b0                        rows x d, K = I
//      Dh:   C0 = a0 b0^T                      rows x I, K = d
//      Dx:   C0 = a0 b0 + a1 b1                rows x d, K = I twice
//      Dw:   C0 = a^T b0                       I x d, K = the expert's rows; one or two a
template <typename W, int FORM>
__global__ void __launch_bounds__(kThreads) grouped_simt_kernel(const SimtParams p) {
    constexpr bool kDual = FORM == kFormUp;
    constexpr int kPad = 4;  // rows of the stages stay 16-byte aligned
    __shared__ __align__(16) float As[kBK][kBM + kPad];
    __shared__ __align__(16) float Bs[kDual ? 2 : 1][kBK][kBN + kPad];
    __shared__ int row_s[kTrainMaxExperts + 1], tile_s[kTrainMaxExperts + 1];
    const W* tag = nullptr;
    const int tid = threadIdx.x;
    grid_dep_wait();
    for (int e = tid; e <= p.N; e += kThreads) row_s[e] = min(max(p.offsets[e], 0), p.M);
    __syncthreads();
    const int n_cols = FORM == kFormUp || FORM == kFormDh ? p.I : p.d;
    const int nt = (n_cols + kBN - 1) / kBN;
    const int n_mat = FORM == kFormDw && p.o1 ? 2 : 1;
    const int mt_w = (p.I + kBM - 1) / kBM;
    if (tid < 32) {  // tiles before each expert
        int carry = 0;
        for (int b = 0; b < p.N; b += 32) {
            const int e = b + tid;
            int v = 0;
            if (e < p.N) v = FORM == kFormDw ? n_mat * mt_w * nt : (max(row_s[e + 1] - row_s[e], 0) + kBM - 1) / kBM * nt;
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
    const int ty = tid / 16, tx = tid % 16;
    for (int tile = blockIdx.x; tile < tile_s[p.N]; tile += gridDim.x) {
        int lo = 0, hi = p.N;  // the last expert whose tiles start at or before this one
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (tile_s[mid] <= tile) lo = mid;
            else hi = mid;
        }
        const int e = lo, row0 = row_s[e], rows = max(row_s[e + 1] - row0, 0);
        int local = tile - tile_s[e];
        const int mts = FORM == kFormDw ? mt_w : (rows + kBM - 1) / kBM;
        const int mat = local / (mts * nt);
        local -= mat * mts * nt;
        const int m0 = local % mts * kBM, n0 = local / mts * kBN;
        const int m_end = FORM == kFormDw ? p.I : rows;
        const int K = FORM == kFormDw ? rows : FORM == kFormUp || FORM == kFormDh ? p.d : p.I;
        const int64_t w0 = (int64_t)e * p.I * p.d;
        float acc[kDual ? 2 : 1][4][4];
#pragma unroll
        for (int c = 0; c < (kDual ? 2 : 1); ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[c][i][j] = 0.f;
        const int parts = FORM == kFormDx ? 2 : 1;
        const int steps1 = (K + kBK - 1) / kBK;
        float ra[4], rb[kDual ? 2 : 1][4];
        // the four values of a stage that this thread brings, read along the
        // operand's contiguous axis
        auto fetch = [&](int step) {
            const int part = FORM == kFormDx && step >= steps1;
            const int k0 = (step - part * steps1) * kBK;
            const void* A = FORM == kFormDw ? (mat ? p.a1 : p.a0) : part ? p.a1 : p.a0;
            const void* B = part ? p.b1 : p.b0;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int i = q * kThreads + tid;
                {
                    const int k = FORM == kFormDw ? i / kBM : i % kBK, m = FORM == kFormDw ? i % kBM : i / kBK;
                    const bool in = k0 + k < K && m0 + m < m_end;
                    const int64_t at = FORM == kFormDw ? (int64_t)(row0 + k0 + k) * p.I + m0 + m
                                                       : (int64_t)(row0 + m0 + m) * K + k0 + k;
                    ra[q] = in ? ld(A, at, tag) : 0.f;
                }
                {
                    constexpr bool kNT = FORM == kFormUp || FORM == kFormDh;
                    const int k = kNT ? i % kBK : i / kBN, n = kNT ? i / kBK : i % kBN;
                    const bool in = k0 + k < K && n0 + n < n_cols;
                    const int64_t at = kNT ? w0 + (int64_t)(n0 + n) * K + k0 + k
                                     : FORM == kFormDw ? (int64_t)(row0 + k0 + k) * p.d + n0 + n
                                                       : w0 + (int64_t)(k0 + k) * p.d + n0 + n;
                    rb[0][q] = in ? ld(B, at, tag) : 0.f;
                    if constexpr (kDual) rb[1][q] = in ? ld(p.b1, at, tag) : 0.f;
                }
            }
        };
        auto stage = [&]() {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int i = q * kThreads + tid;
                if (FORM == kFormDw) As[i / kBM][i % kBM] = ra[q];
                else As[i % kBK][i / kBK] = ra[q];
                constexpr bool kNT = FORM == kFormUp || FORM == kFormDh;
                const int k = kNT ? i % kBK : i / kBN, n = kNT ? i / kBK : i % kBN;
                Bs[0][k][n] = rb[0][q];
                if constexpr (kDual) Bs[1][k][n] = rb[1][q];
            }
        };
        const int steps = steps1 * parts;
        if (steps > 0) fetch(0);
        for (int s = 0; s < steps; ++s) {
            __syncthreads();  // the last stage has been read
            stage();
            __syncthreads();
            if (s + 1 < steps) fetch(s + 1);
#pragma unroll
            for (int k = 0; k < kBK; ++k) {
                const float4 a = *reinterpret_cast<const float4*>(&As[k][ty * 4]);
                const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                for (int c = 0; c < (kDual ? 2 : 1); ++c) {
                    const float4 b = *reinterpret_cast<const float4*>(&Bs[c][k][tx * 4]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        acc[c][i][0] = fmaf(av[i], b.x, acc[c][i][0]);
                        acc[c][i][1] = fmaf(av[i], b.y, acc[c][i][1]);
                        acc[c][i][2] = fmaf(av[i], b.z, acc[c][i][2]);
                        acc[c][i][3] = fmaf(av[i], b.w, acc[c][i][3]);
                    }
                }
            }
        }
        __syncthreads();  // before the next tile's first stage
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int m = m0 + ty * 4 + i;
            if (m >= m_end) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = n0 + tx * 4 + j;
                if (n >= n_cols) continue;
                const float c0 = acc[0][i][j];
                if constexpr (FORM == kFormUp) {
                    const int64_t at = (int64_t)(row0 + m) * p.I + n;
                    const float c1 = acc[kDual ? 1 : 0][i][j];
                    if (p.o0) { st(p.o0, at, c0, tag); st(p.o1, at, c1, tag); }
                    st(p.o2, at, c0 * sigmoid(c0) * c1, tag);
                } else if constexpr (FORM == kFormDh) {
                    const int64_t at = (int64_t)(row0 + m) * p.I + n;
                    const float g = ld(p.g, at, tag), u = ld(p.u, at, tag), sg = sigmoid(g);
                    st(p.o0, at, c0 * u * sg * (1.f + g * (1.f - sg)), tag);
                    st(p.o1, at, c0 * g * sg, tag);
                } else if constexpr (FORM == kFormDw) {
                    const int64_t at = w0 + (int64_t)m * p.d + n;
                    void* o = mat ? p.o1 : p.o0;
                    if (p.out_f32) {
                        float* f = static_cast<float*>(o) + at;
                        *f = p.accumulate ? *f + c0 : c0;
                    } else st(o, at, c0, tag);
                } else st(p.o0, (int64_t)(row0 + m) * p.d + n, c0, tag);
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

template <typename W>
cudaError_t launch(const GroupedArgs& a, const SimtParams& p, cudaStream_t st) {
    const int n_cols = a.form == kFormUp || a.form == kFormDh ? a.I : a.d;
    const int64_t nt = (n_cols + kBN - 1) / kBN;
    int64_t tiles = a.form == kFormDw ? (int64_t)a.N * (a.o1 ? 2 : 1) * ((a.I + kBM - 1) / kBM) * nt
                                      : ((int64_t)a.M / kBM + (a.N < a.M ? a.N : a.M)) * nt;
    if (tiles > (int64_t)a.sms * 6) tiles = (int64_t)a.sms * 6;
    const dim3 grid((unsigned)(tiles < 1 ? 1 : tiles));
    switch (a.form) {
        case kFormUp: return launch_pdl(grouped_simt_kernel<W, kFormUp>, grid, dim3(kThreads), 0, st, p);
        case kFormDown: return launch_pdl(grouped_simt_kernel<W, kFormDown>, grid, dim3(kThreads), 0, st, p);
        case kFormDh: return launch_pdl(grouped_simt_kernel<W, kFormDh>, grid, dim3(kThreads), 0, st, p);
        case kFormDx: return launch_pdl(grouped_simt_kernel<W, kFormDx>, grid, dim3(kThreads), 0, st, p);
        case kFormDw: return launch_pdl(grouped_simt_kernel<W, kFormDw>, grid, dim3(kThreads), 0, st, p);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_grouped_simt(const GroupedArgs& a, cudaStream_t st) {
    SimtParams p;
    p.a0 = a.a0; p.a1 = a.a1; p.b0 = a.b0; p.b1 = a.b1; p.g = a.g; p.u = a.u;
    p.o0 = a.o0; p.o1 = a.o1; p.o2 = a.o2; p.offsets = a.offsets;
    p.M = a.M; p.N = a.N; p.d = a.d; p.I = a.I; p.out_f32 = a.out_f32; p.accumulate = a.accumulate;
    return a.bf16 ? launch<__nv_bfloat16>(a, p, st) : launch<float>(a, p, st);
}

}  // namespace moe
