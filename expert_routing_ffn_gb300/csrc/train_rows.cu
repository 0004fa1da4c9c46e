// Token rows of the training step: sorted by expert (dispatch), brought back
// with the gates applied (combine), and the gradients of both.
//
// All of it moves rows of d values whose place is an index: the work is bytes.
// Rows are moved in vectors of 16 bytes where every row starts on a 16-byte
// boundary, else of 4, else of single bf16 values.
#include <cuda_bf16.h>

#include "common.cuh"
#include "train.h"

namespace moe {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

template <int VB> struct VecOf;
template <> struct VecOf<16> { using T = uint4; };
template <> struct VecOf<4> { using T = uint32_t; };
template <> struct VecOf<2> { using T = uint16_t; };

template <int VB>
__device__ __forceinline__ typename VecOf<VB>::T zero_vec() {
    typename VecOf<VB>::T v;
    if constexpr (VB == 16) v = make_uint4(0, 0, 0, 0);
    else v = 0;
    return v;
}

// values of a vector as fp32, and back (one rounding, to nearest even)
template <typename W, int VB>
__device__ __forceinline__ void to_floats(const typename VecOf<VB>::T& v, float* f) {
    if constexpr (VB == 16) unpack16(v, f, (W*)nullptr);
    else if constexpr (VB == 4 && sizeof(W) == 4) f[0] = __uint_as_float(v);
    else if constexpr (VB == 4) { f[0] = bf16_lo(v); f[1] = bf16_hi(v); }
    else f[0] = __uint_as_float((uint32_t)v << 16);
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
}
template <typename W, int VB>
__device__ __forceinline__ typename VecOf<VB>::T from_floats(const float* f) {
    if constexpr (VB == 16 && sizeof(W) == 4)
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    else if constexpr (VB == 16)
        return make_uint4(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7]));
    else if constexpr (VB == 4 && sizeof(W) == 4) return __float_as_uint(f[0]);
    else if constexpr (VB == 4) return bf16_pair(f[0], f[1]);
    else { const __nv_bfloat16 b = __float2bfloat16_rn(f[0]); return *reinterpret_cast<const uint16_t*>(&b); }
}

// ---------------------------------------------------------------- dispatch
// One launch sorts and moves.  The slots form chunks of at most a block's
// threads (whole tokens); a block ranks the slots of its chunk, a slot a
// thread, and moves its share of the chunk's rows: each row of x is read once
// and written to the places of its k slots.  What comes before the chunk the
// block counts by itself (kDispAlone slots: 16 indices a thread); longer
// batches have a counting launch first (65536 slots: 32 us against 45 when
// every block counted half of them).
// Ranking is repeated by the blocks that share a chunk, so those are few and
// large: with 256-thread blocks, eight to an SM, 777 tokens of 1763 values
// took 18 us, with 1024-thread blocks 12.
// Bound: HBM writes.  4096 tokens of 3584 bf16 values, 8 slots each: 50 us for
// 265 MB, 0.78 of the measured copy bandwidth.
struct DispatchParams {
    const char* x; int64_t ldx;
    const int32_t* idx;
    int T, N, k, capacity, chunk_tokens, shares;
    int64_t row_bytes;
    char* xp; int32_t *offsets, *perm, *inv;
    int32_t* counts;  // [spans][N + 1], where there is more than one
    int spans, span_tokens;
    DevError* err;
};

__device__ __forceinline__ int dispatch_key(const DispatchParams& p, int64_t slot) {
    const int e = p.idx[slot];
    return (unsigned)e < (unsigned)p.N ? e : p.N;
}

__global__ void __launch_bounds__(1024) dispatch_count_kernel(const DispatchParams p) {
    extern __shared__ int hist[];
    for (int i = threadIdx.x; i <= p.N; i += blockDim.x) hist[i] = 0;
    __syncthreads();
    grid_dep_wait();
    const int64_t s0 = (int64_t)blockIdx.x * p.span_tokens * p.k;
    const int64_t s1 = min(s0 + (int64_t)p.span_tokens * p.k, (int64_t)p.T * p.k);
    for (int64_t s = s0 + threadIdx.x; s < s1; s += blockDim.x) atomicAdd(&hist[dispatch_key(p, s)], 1);
    __syncthreads();
    for (int i = threadIdx.x; i <= p.N; i += blockDim.x) p.counts[(size_t)blockIdx.x * (p.N + 1) + i] = hist[i];
    grid_dep_launch();
}

// vectors of a row that a lane moves at a time: more in long batches, whose
// items are plenty
__host__ __device__ constexpr int dispatch_vectors(int vb, int threads) { return vb < 16 || threads == 1024 ? 4 : 2; }

template <int VB, int THREADS>
__global__ void __launch_bounds__(THREADS) dispatch_move_kernel(const DispatchParams p) {
    using V = typename VecOf<VB>::T;
    constexpr int kW = THREADS / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int NK = p.N + 1;  // keys: the experts, then "no expert"
    extern __shared__ int sm[];
    int* tot = sm;                    // [NK] slots of the whole batch per key
    int* before = tot + NK;           // [NK] slots of earlier chunks per key
    int* off = before + NK;           // [NK] first row of each expert
    int* pos_s = off + NK;            // [THREADS]
    uint16_t* cnt = reinterpret_cast<uint16_t*>(pos_s + THREADS);  // [kW][NK] slots of a warp per key, then those before it
    __shared__ int wdrop[kW], s_kept, s_drop_before;

    const int chunk = blockIdx.x / p.shares, share = blockIdx.x % p.shares;
    const int t0 = chunk * p.chunk_tokens;
    const int n_tok = min(p.chunk_tokens, p.T - t0);
    const int n = n_tok * p.k;  // at most THREADS
    const int64_t slot0 = (int64_t)t0 * p.k;
    for (int i = tid; i < 2 * NK; i += THREADS) sm[i] = 0;
    for (int i = tid; i < kW * NK; i += THREADS) cnt[i] = 0;
    __syncthreads();
    grid_dep_wait();
    // this thread's slot, and its rank among the warp's slots of the same key
    int key = -1;
    if (tid < n) {
        key = p.idx[slot0 + tid];
        if (key >= p.N && share == 0) set_error(p.err, MOE_ERR_DEVICE_INDEX, (int)(slot0 + tid));
        if ((unsigned)key >= (unsigned)p.N) key = p.N;
    }
    const uint32_t peers = __match_any_sync(0xffffffffu, key);
    const int rank = __popc(peers & ((1u << lane) - 1u));
    if (key >= 0 && rank == 0) cnt[warp * NK + key] = (uint16_t)__popc(peers);
    // the slots of the batch and those before the chunk: spans that were
    // counted, the rest one by one (consecutive lanes take consecutive slots:
    // a token's experts differ, so few of them meet at one counter)
    const int span = p.spans > 1 ? t0 / p.span_tokens : 0;
    const int64_t all = p.spans > 1 ? slot0 : (int64_t)p.T * p.k;
#pragma unroll 8
    for (int64_t s = (int64_t)span * p.span_tokens * p.k + tid; s < all; s += THREADS) {
        const int e = dispatch_key(p, s);
        if (p.spans == 1) atomicAdd(&tot[e], 1);
        if (s < slot0) atomicAdd(&before[e], 1);
    }
    if (p.spans > 1) {
        const int n_cnt = p.spans * NK;
        for (int i = tid; i < n_cnt; i += THREADS) {
            const int v = __ldcg(p.counts + i);
            const int c = i / NK, e = i - c * NK;
            if (v) {
                atomicAdd(&tot[e], v);
                if (c < span) atomicAdd(&before[e], v);
            }
        }
    }
    __syncthreads();
    for (int e = tid; e < NK; e += THREADS) {
        int sum = 0;
        for (int w = 0; w < kW; ++w) {
            const int v = cnt[w * NK + e];
            cnt[w * NK + e] = (uint16_t)sum;
            sum += v;
        }
    }
    const int cap = p.capacity > 0 ? p.capacity : 0x7fffffff;
    if (warp == kW - 1) {  // first rows: exclusive scan of the kept slots
        int carry = 0, over = 0;
        for (int b = 0; b < p.N; b += 32) {
            const int e = b + lane;
            const int v = e < p.N ? min(tot[e], cap) : 0;
            if (e < p.N) over += max(0, before[e] - cap);
            int inc = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += u;
            }
            if (e < p.N) off[e] = carry + inc - v;
            carry += __shfl_sync(0xffffffffu, inc, 31);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) over += __shfl_xor_sync(0xffffffffu, over, o);
        if (lane == 0) { off[p.N] = carry; s_kept = carry; s_drop_before = before[p.N] + over; }
    }
    __syncthreads();
    const int r = key >= 0 && key < p.N ? before[key] + cnt[warp * NK + key] + rank : 0;
    const bool drop = key == p.N || (key >= 0 && r >= cap);
    const uint32_t dropped = __ballot_sync(0xffffffffu, drop);
    if (lane == 0) wdrop[warp] = __popc(dropped);
    __syncthreads();
    if (tid < n) {
        int q = off[key < p.N ? key : 0] + r;
        if (drop) {
            int d0 = s_kept + s_drop_before + __popc(dropped & ((1u << lane) - 1u));
            for (int w = 0; w < warp; ++w) d0 += wdrop[w];
            q = ~d0;
        }
        pos_s[tid] = q;
        if (share == 0) {
            p.inv[slot0 + tid] = q < 0 ? q - 1 : q;  // ~row - 1 = -2 - row
            p.perm[q < 0 ? ~q : q] = q < 0 ? -1 : (int)(slot0 + tid);
        }
    }
    if (blockIdx.x == 0)
        for (int e = tid; e <= p.N; e += THREADS) p.offsets[e] = off[e];
    __syncthreads();
    // an item: 32 x kU vectors of one token's row, read once, written k times
    constexpr int kU = dispatch_vectors(VB, THREADS);
    const int n_vec = (int)(p.row_bytes / VB);
    const int pieces = (n_vec + 32 * kU - 1) / (32 * kU);
    const int items = n_tok * pieces;
    for (int it = share * kW + warp; it < items; it += p.shares * kW) {
        const int t = it / pieces, v0 = (it - t * pieces) * 32 * kU + lane;
        const V* src = reinterpret_cast<const V*>(p.x + (int64_t)(t0 + t) * p.ldx);
        V v[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u)
            if (v0 + u * 32 < n_vec) v[u] = src[v0 + u * 32];
        for (int s = 0; s < p.k; ++s) {
            const int q = pos_s[t * p.k + s];
            V* dst = reinterpret_cast<V*>(p.xp + (int64_t)(q < 0 ? ~q : q) * p.row_bytes);
#pragma unroll
            for (int u = 0; u < kU; ++u)
                if (v0 + u * 32 < n_vec) dst[v0 + u * 32] = q < 0 ? zero_vec<VB>() : v[u];
        }
    }
    grid_dep_launch();
}

// ---------------------------------------------------------------- combine
// out[t] = add[t] + sum_s gate[t,s] y[inv[t,s]].  A warp takes `m` x 32
// vectors of one token's row; the rows of up to eight slots are loaded before
// any is used.  Slots are added in slot order, add last, in fp32.  Bound: HBM
// reads; 4096 tokens of 3584 bf16 values, 8 slots each: 52 us for 294 MB, 0.84
// of the measured copy bandwidth.
struct CombineParams {
    const char* y; const float* gate; const int32_t* inv;
    const char* add; int64_t ldadd; char* out; int64_t ldout;  // bytes
    int T, k, m, pieces, n_rows;
    int64_t row_bytes;
};

template <typename W, int VB>
__global__ void __launch_bounds__(kThreads) combine_rows_kernel(const CombineParams p) {
    using V = typename VecOf<VB>::T;
    constexpr int kE = VB / (int)sizeof(W);
    const int lane = threadIdx.x & 31;
    grid_dep_wait();
    const int n_vec = (int)(p.row_bytes / VB);
    const int64_t items = (int64_t)p.T * p.pieces;
    for (int64_t it = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); it < items; it += (int64_t)gridDim.x * kWarps) {
        const int64_t t = it / p.pieces;
        const int v0 = (int)(it - t * p.pieces) * 32 * p.m + lane;
        int my_row = -1;
        float my_gate = 1.f;
        if (lane < p.k) {
            my_row = p.inv[t * p.k + lane];
            if (my_row >= p.n_rows) my_row = -1;
            if (p.gate) my_gate = p.gate[t * p.k + lane];
        }
        for (int j = 0; j < p.m; ++j) {
            const int vi = v0 + j * 32;
            const bool in = vi < n_vec;
            float acc[kE];
#pragma unroll
            for (int i = 0; i < kE; ++i) acc[i] = 0.f;
            V base = zero_vec<VB>();
            if (in && p.add) base = reinterpret_cast<const V*>(p.add + t * p.ldadd)[vi];
            for (int s0 = 0; s0 < p.k; s0 += 8) {
                V v[8];
                int row[8];
#pragma unroll
                for (int s = 0; s < 8; ++s) {
                    row[s] = s0 + s < p.k ? __shfl_sync(0xffffffffu, my_row, s0 + s) : -1;
                    if (row[s] >= 0 && in)
                        v[s] = reinterpret_cast<const V*>(p.y + (int64_t)row[s] * p.row_bytes)[vi];
                }
#pragma unroll
                for (int s = 0; s < 8; ++s) {
                    const float g = __shfl_sync(0xffffffffu, my_gate, (s0 + s) & 31);
                    if (row[s] >= 0 && in) {
                        float f[kE];
                        to_floats<W, VB>(v[s], f);
#pragma unroll
                        for (int i = 0; i < kE; ++i) acc[i] = fmaf(g, f[i], acc[i]);
                    }
                }
            }
            if (in) {
                if (p.add) {
                    float f[kE];
                    to_floats<W, VB>(base, f);
#pragma unroll
                    for (int i = 0; i < kE; ++i) acc[i] += f[i];
                }
                reinterpret_cast<V*>(p.out + t * p.ldout)[vi] = from_floats<W, VB>(acc);
            }
        }
    }
    grid_dep_launch();
}

// ---------------------------------------------------------------- combine, gradient
// One block per token: dout's row is read once, every slot's y row is read
// (for dgate) and its dy row written in the same pass.  The k dot products
// are summed per thread, then over the warp, then over the warps, in fixed
// order.  Bound: HBM; 4096 tokens of 3584 bf16 values, 8 slots each: 77 us for
// 500 MB, 0.95 of the measured copy bandwidth.
constexpr int kGradMaxThreads = 512, kGradWarps = kGradMaxThreads / 32;

struct CombineGradParams {
    const char* dout; int64_t lddout; const char* y; const float* gate; const int32_t* inv;
    char* dy; float* dgate;
    int k, n_rows;
    int64_t row_bytes;
};

template <typename W, int VB, int KB>
__global__ void __launch_bounds__(VB == 16 ? 128 : kGradMaxThreads) combine_grad_kernel(const CombineGradParams p) {
    using V = typename VecOf<VB>::T;
    constexpr int kE = VB / (int)sizeof(W);
    __shared__ float part[kGradWarps][KB];
    __shared__ int row_s[KB];
    __shared__ float gate_s[KB];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t t = blockIdx.x;
    grid_dep_wait();
    if (tid < KB) {
        int r = tid < p.k ? p.inv[t * p.k + tid] : -1;
        if (r >= p.n_rows || r < -1 - p.n_rows) r = -1;  // out of range: no row
        row_s[tid] = r;
        gate_s[tid] = tid < p.k && p.gate ? p.gate[t * p.k + tid] : 1.f;
    }
    __syncthreads();
    const int n_vec = (int)(p.row_bytes / VB);
    float dot[KB];
#pragma unroll
    for (int s = 0; s < KB; ++s) dot[s] = 0.f;
    for (int vi = tid; vi < n_vec; vi += blockDim.x) {
        float g[kE];
        to_floats<W, VB>(reinterpret_cast<const V*>(p.dout + t * p.lddout)[vi], g);
#pragma unroll
        for (int s0 = 0; s0 < KB; s0 += 8) {
            V v[8];
            if (p.dgate) {
#pragma unroll
                for (int s = 0; s < 8; ++s)
                    if (row_s[s0 + s] >= 0)
                        v[s] = reinterpret_cast<const V*>(p.y + (int64_t)row_s[s0 + s] * p.row_bytes)[vi];
            }
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                const int row = row_s[s0 + s];
                if (row >= 0 && p.dgate) {
                    float f[kE];
                    to_floats<W, VB>(v[s], f);
#pragma unroll
                    for (int i = 0; i < kE; ++i) dot[s0 + s] = fmaf(g[i], f[i], dot[s0 + s]);
                }
                if (p.dy && row != -1) {
                    float f[kE];
                    const float w = gate_s[s0 + s];
#pragma unroll
                    for (int i = 0; i < kE; ++i) f[i] = w * g[i];
                    reinterpret_cast<V*>(p.dy + (int64_t)(row >= 0 ? row : -2 - row) * p.row_bytes)[vi] =
                        row >= 0 ? from_floats<W, VB>(f) : zero_vec<VB>();
                }
            }
        }
    }
    if (p.dgate) {
#pragma unroll
        for (int s = 0; s < KB; ++s) {
            const float v = warp_sum(dot[s]);
            if (lane == 0) part[warp][s] = v;
        }
        __syncthreads();
        if (tid < p.k) {
            float v = 0.f;
            for (int w = 0; w < (int)blockDim.x / 32; ++w) v += part[w][tid];
            p.dgate[t * p.k + tid] = row_s[tid] >= 0 ? v : 0.f;
        }
    }
    grid_dep_launch();
}

// bytes of the vectors that rows of `row_bytes` at these addresses and strides allow
int vec_bytes(int64_t row_bytes, std::initializer_list<int64_t> places) {
    int64_t bits = row_bytes;
    for (int64_t v : places) bits |= v;
    return bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 2;
}
int64_t at(const void* p) { return (int64_t)reinterpret_cast<uintptr_t>(p); }

}  // namespace

template <int THREADS>
static cudaError_t launch_move(const DispatchParams& p, int vb, int blocks, cudaStream_t st) {
    const size_t smem = (size_t)(3 * (p.N + 1) + THREADS) * 4 + (size_t)THREADS / 32 * (p.N + 1) * 2;
    const dim3 grid((unsigned)blocks), block(THREADS);
    return vb == 16 ? launch_pdl(dispatch_move_kernel<16, THREADS>, grid, block, smem, st, p)
         : vb == 4  ? launch_pdl(dispatch_move_kernel<4, THREADS>, grid, block, smem, st, p)
                    : launch_pdl(dispatch_move_kernel<2, THREADS>, grid, block, smem, st, p);
}

cudaError_t launch_dispatch_rows(const DispatchArgs& a, cudaStream_t st, int* launches) {
    DispatchParams p;
    p.x = static_cast<const char*>(a.x); p.ldx = a.ldx_bytes; p.idx = a.idx;
    p.T = a.T; p.N = a.N; p.k = a.k; p.capacity = a.capacity;
    p.row_bytes = a.row_bytes; p.xp = static_cast<char*>(a.x_perm);
    p.offsets = a.offsets; p.perm = a.perm; p.inv = a.inv; p.counts = a.counts; p.err = a.err;
    p.spans = dispatch_spans(a.T, a.k);
    p.span_tokens = dispatch_span_tokens(a.T, a.k);
    // a small batch: small blocks, which start sooner and synchronise faster
    const int64_t slots = (int64_t)a.T * a.k;
    const int threads = slots <= 256 ? 256 : slots <= 4096 ? 512 : 1024, warps = threads / 32;
    p.chunk_tokens = threads / a.k < a.T ? threads / a.k : a.T;
    const int chunks = (a.T + p.chunk_tokens - 1) / p.chunk_tokens;
    const int vb = vec_bytes(a.row_bytes, {at(a.x), at(a.x_perm), a.ldx_bytes});
    // blocks: a warp for every row piece, at most one wave
    const int piece = 32 * dispatch_vectors(vb, threads) * vb;
    const int64_t items = (int64_t)p.chunk_tokens * ((a.row_bytes + piece - 1) / piece);
    const int64_t need = (items + warps - 1) / warps, wave = (int64_t)a.sms * (2048 / threads) / chunks;
    p.shares = (int)(need < wave ? need : wave);
    if (p.shares < 1) p.shares = 1;
    *launches = 1;
    if (p.spans > 1) {
        const cudaError_t e = launch_pdl(dispatch_count_kernel, dim3(p.spans), dim3(1024), (size_t)(a.N + 1) * 4, st, p);
        if (e != cudaSuccess) return e;
        *launches = 2;
    }
    return threads == 256 ? launch_move<256>(p, vb, chunks * p.shares, st)
         : threads == 512 ? launch_move<512>(p, vb, chunks * p.shares, st)
                          : launch_move<1024>(p, vb, chunks * p.shares, st);
}

cudaError_t launch_combine_rows(const CombineRowsArgs& a, cudaStream_t st) {
    const int es = a.bf16 ? 2 : 4;
    CombineParams p;
    p.y = static_cast<const char*>(a.y); p.gate = a.gate; p.inv = a.inv;
    p.add = static_cast<const char*>(a.add); p.ldadd = a.ldadd * es;
    p.out = static_cast<char*>(a.out); p.ldout = a.ldout * es;
    p.T = a.T; p.k = a.k; p.n_rows = a.T * a.k; p.row_bytes = a.d * es;
    const int vb = vec_bytes(p.row_bytes, {at(a.y), at(a.out), p.ldout, a.add ? at(a.add) : 0, a.add ? p.ldadd : 0});
    const int n_vec = (int)(p.row_bytes / vb), groups = (n_vec + 31) / 32;
    // a warp takes more of a row only where the tokens fill the GPU by themselves
    const int64_t warps = (int64_t)a.sms * 64;
    p.m = (int)((int64_t)a.T * groups / warps);
    p.m = p.m < 1 ? 1 : p.m > 4 ? 4 : p.m;
    p.pieces = (groups + p.m - 1) / p.m;
    const int64_t blocks = ((int64_t)a.T * p.pieces + kWarps - 1) / kWarps;
    const dim3 grid((unsigned)(blocks < (1 << 20) ? blocks : (1 << 20)));
    if (a.bf16)
        return vb == 16 ? launch_pdl(combine_rows_kernel<__nv_bfloat16, 16>, grid, dim3(kThreads), 0, st, p)
             : vb == 4  ? launch_pdl(combine_rows_kernel<__nv_bfloat16, 4>, grid, dim3(kThreads), 0, st, p)
                        : launch_pdl(combine_rows_kernel<__nv_bfloat16, 2>, grid, dim3(kThreads), 0, st, p);
    return vb == 16 ? launch_pdl(combine_rows_kernel<float, 16>, grid, dim3(kThreads), 0, st, p)
                    : launch_pdl(combine_rows_kernel<float, 4>, grid, dim3(kThreads), 0, st, p);
}

template <typename W, int VB>
static cudaError_t launch_grad(const CombineGradParams& p, int T, cudaStream_t st) {
    // small vectors: more threads to a row, a few vectors each
    int threads = 128;
    if (VB < 16)
        while (threads < kGradMaxThreads && p.row_bytes / VB > 4 * threads) threads *= 2;
    return p.k <= 8 ? launch_pdl(combine_grad_kernel<W, VB, 8>, dim3(T), dim3(threads), 0, st, p)
                    : launch_pdl(combine_grad_kernel<W, VB, 16>, dim3(T), dim3(threads), 0, st, p);
}

cudaError_t launch_combine_rows_grad(const CombineRowsGradArgs& a, cudaStream_t st) {
    const int es = a.bf16 ? 2 : 4;
    CombineGradParams p;
    p.dout = static_cast<const char*>(a.dout); p.lddout = a.lddout * es;
    p.y = static_cast<const char*>(a.y); p.gate = a.gate; p.inv = a.inv;
    p.dy = static_cast<char*>(a.dy); p.dgate = a.dgate;
    p.k = a.k; p.n_rows = a.T * a.k; p.row_bytes = a.d * es;
    const int vb = vec_bytes(p.row_bytes, {at(a.dout), p.lddout, a.dgate ? at(a.y) : 0, a.dy ? at(a.dy) : 0});
    if (a.bf16)
        return vb == 16 ? launch_grad<__nv_bfloat16, 16>(p, a.T, st)
             : vb == 4  ? launch_grad<__nv_bfloat16, 4>(p, a.T, st)
                        : launch_grad<__nv_bfloat16, 2>(p, a.T, st);
    return vb == 16 ? launch_grad<float, 16>(p, a.T, st) : launch_grad<float, 4>(p, a.T, st);
}

}  // namespace moe
