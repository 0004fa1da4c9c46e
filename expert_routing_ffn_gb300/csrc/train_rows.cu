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
// The slots of one chunk of tokens are counted per expert (dispatch_count:
// one block per chunk), then every block of dispatch_move ranks the slots of
// its chunk again, which costs it a few thousand cycles and spares a third
// launch and a round trip of the positions through memory, and moves its
// share of the chunk's rows: each row of x is read once and written to the
// places of its k slots.  A batch of one chunk needs no counting launch.
struct DispatchParams {
    const char* x; int64_t ldx;
    const int32_t* idx;
    int T, N, k, capacity, chunk_tokens, shares, n_chunks;
    int64_t row_bytes;
    char* xp; int32_t *offsets, *perm, *inv;
    int32_t* counts;
    DevError* err;
};

__device__ __forceinline__ int dispatch_key(const DispatchParams& p, int64_t slot, bool report) {
    const int e = p.idx[slot];
    if (e >= p.N) {
        if (report) set_error(p.err, MOE_ERR_DEVICE_INDEX, (int)slot);
        return p.N;
    }
    return e < 0 ? p.N : e;
}

__global__ void __launch_bounds__(kThreads) dispatch_count_kernel(const DispatchParams p) {
    extern __shared__ int hist[];
    for (int i = threadIdx.x; i <= p.N; i += kThreads) hist[i] = 0;
    __syncthreads();
    grid_dep_wait();
    const int64_t s0 = (int64_t)blockIdx.x * p.chunk_tokens * p.k;
    const int64_t s1 = min(s0 + (int64_t)p.chunk_tokens * p.k, (int64_t)p.T * p.k);
    for (int64_t s = s0 + threadIdx.x; s < s1; s += kThreads) atomicAdd(&hist[dispatch_key(p, s, false)], 1);
    __syncthreads();
    for (int i = threadIdx.x; i <= p.N; i += kThreads) p.counts[(size_t)blockIdx.x * (p.N + 1) + i] = hist[i];
    grid_dep_launch();
}

template <int VB>
__global__ void __launch_bounds__(kThreads) dispatch_move_kernel(const DispatchParams p) {
    using V = typename VecOf<VB>::T;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int NK = p.N + 1;  // keys: the experts, then "no expert"
    extern __shared__ int sm[];
    int* cnt = sm;                    // [kWarps][NK] slots of a warp per key, then those before it
    int* tot = cnt + kWarps * NK;     // [NK] slots of the whole batch per key
    int* before = tot + NK;           // [NK] slots of earlier chunks per key
    int* off = before + NK;           // [NK] first row of each expert
    int* pos_s = off + NK;            // [slots of a chunk]
    __shared__ int wdrop[kWarps], s_kept, s_drop_before;

    const int chunk = blockIdx.x / p.shares, share = blockIdx.x % p.shares;
    const int t0 = chunk * p.chunk_tokens;
    const int n_tok = min(p.chunk_tokens, p.T - t0);
    const int n = n_tok * p.k;
    const int64_t slot0 = (int64_t)t0 * p.k;
    for (int i = tid; i < kWarps * NK + 2 * NK; i += kThreads) sm[i] = 0;
    __syncthreads();
    grid_dep_wait();
    // rank among the warp's slots of the same key; a warp owns a run of slots
    const int run = ((n + kWarps - 1) / kWarps + 31) / 32 * 32;
    const int r0 = min(warp * run, n), r1 = min(r0 + run, n);
    for (int b = r0; b < r1; b += 32) {
        const int i = b + lane;
        const int key = i < r1 ? dispatch_key(p, slot0 + i, share == 0) : -1;
        const uint32_t peers = __match_any_sync(0xffffffffu, key);
        const int ahead = __popc(peers & ((1u << lane) - 1u));
        const int seen = key >= 0 ? cnt[warp * NK + key] : 0;
        __syncwarp();
        if (key >= 0 && ahead == 0) cnt[warp * NK + key] = seen + __popc(peers);
        __syncwarp();
        if (key >= 0) pos_s[i] = (key << 16) | (seen + ahead);
    }
    if (p.n_chunks > 1) {
        const int n_cnt = p.n_chunks * NK;
        for (int i = tid; i < n_cnt; i += kThreads) {
            const int v = __ldcg(p.counts + i);
            const int c = i / NK, e = i - c * NK;
            if (v) {
                atomicAdd(&tot[e], v);
                if (c < chunk) atomicAdd(&before[e], v);
            }
        }
    }
    __syncthreads();
    for (int e = tid; e < NK; e += kThreads) {
        int sum = before[e];
        for (int w = 0; w < kWarps; ++w) {
            const int v = cnt[w * NK + e];
            cnt[w * NK + e] = sum;
            sum += v;
        }
        if (p.n_chunks == 1) tot[e] = sum;
    }
    __syncthreads();
    const int cap = p.capacity > 0 ? p.capacity : 0x7fffffff;
    if (warp == 0) {  // first rows: exclusive scan of the kept slots
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
    int drops = 0;
    for (int b = r0; b < r1; b += 32) {
        const int i = b + lane;
        bool drop = false;
        if (i < r1) {
            const int key = pos_s[i] >> 16, r = (pos_s[i] & 0xffff) + (key < p.N ? cnt[warp * NK + key] : 0);
            drop = key == p.N || r >= cap;
            if (!drop) pos_s[i] = off[key] + r;
        }
        const uint32_t m = __ballot_sync(0xffffffffu, drop);
        if (drop) pos_s[i] = ~(drops + __popc(m & ((1u << lane) - 1u)));  // its number among the warp's
        drops += __popc(m);
    }
    if (lane == 0) wdrop[warp] = drops;
    __syncthreads();
    int drop0 = s_kept + s_drop_before;
    for (int w = 0; w < warp; ++w) drop0 += wdrop[w];
    for (int i = r0 + lane; i < r1; i += 32) {
        if (pos_s[i] < 0) pos_s[i] = ~(drop0 + ~pos_s[i]);
        if (share == 0) {
            const int q = pos_s[i];
            p.inv[slot0 + i] = q < 0 ? q - 1 : q;  // ~row - 1 = -2 - row
            p.perm[q < 0 ? ~q : q] = q < 0 ? -1 : (int)(slot0 + i);
        }
    }
    if (blockIdx.x == 0)
        for (int e = tid; e <= p.N; e += kThreads) p.offsets[e] = off[e];
    __syncthreads();
    // an item: 32 x kU vectors of one token's row, read once, written k times
    constexpr int kU = VB == 16 ? 2 : 4;
    const int n_vec = (int)(p.row_bytes / VB);
    const int pieces = (n_vec + 32 * kU - 1) / (32 * kU);
    const int items = n_tok * pieces;
    for (int it = share * kWarps + warp; it < items; it += p.shares * kWarps) {
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
// any is used.  Slots are added in slot order, add last, in fp32.
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
// order.
constexpr int kGradThreads = 128, kGradWarps = kGradThreads / 32;

struct CombineGradParams {
    const char* dout; int64_t lddout; const char* y; const float* gate; const int32_t* inv;
    char* dy; float* dgate;
    int k, n_rows;
    int64_t row_bytes;
};

template <typename W, int VB, int KB>
__global__ void __launch_bounds__(kGradThreads) combine_grad_kernel(const CombineGradParams p) {
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
    for (int vi = tid; vi < n_vec; vi += kGradThreads) {
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
#pragma unroll
            for (int w = 0; w < kGradWarps; ++w) v += part[w][tid];
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

cudaError_t launch_dispatch_rows(const DispatchArgs& a, cudaStream_t st, int* launches) {
    DispatchParams p;
    p.x = static_cast<const char*>(a.x); p.ldx = a.ldx_bytes; p.idx = a.idx;
    p.T = a.T; p.N = a.N; p.k = a.k; p.capacity = a.capacity;
    p.chunk_tokens = dispatch_chunk_tokens(a.T, a.k);
    p.n_chunks = dispatch_chunks(a.T, a.k);
    p.row_bytes = a.row_bytes; p.xp = static_cast<char*>(a.x_perm);
    p.offsets = a.offsets; p.perm = a.perm; p.inv = a.inv; p.counts = a.counts; p.err = a.err;
    const int vb = vec_bytes(a.row_bytes, {at(a.x), at(a.x_perm), a.ldx_bytes});
    // blocks: enough for every row piece to have a warp, at most one wave
    const int piece = 32 * (vb == 16 ? 2 : 4) * vb;
    const int64_t items = (int64_t)p.chunk_tokens * ((a.row_bytes + piece - 1) / piece);
    int64_t shares = (items + kWarps - 1) / kWarps;
    const int64_t wave = ((int64_t)a.sms * 8 + p.n_chunks - 1) / p.n_chunks;
    p.shares = (int)(shares < wave ? shares : wave);
    if (p.shares < 1) p.shares = 1;
    *launches = 1;
    if (p.n_chunks > 1) {
        cudaError_t e = launch_pdl(dispatch_count_kernel, dim3(p.n_chunks), dim3(kThreads), (size_t)(a.N + 1) * 4, st, p);
        if (e != cudaSuccess) return e;
        *launches = 2;
    }
    const size_t smem = ((size_t)(kWarps + 3) * (a.N + 1) + (size_t)p.chunk_tokens * a.k) * 4;
    const dim3 grid((unsigned)(p.n_chunks * p.shares));
    return vb == 16 ? launch_pdl(dispatch_move_kernel<16>, grid, dim3(kThreads), smem, st, p)
         : vb == 4  ? launch_pdl(dispatch_move_kernel<4>, grid, dim3(kThreads), smem, st, p)
                    : launch_pdl(dispatch_move_kernel<2>, grid, dim3(kThreads), smem, st, p);
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
    return p.k <= 8 ? launch_pdl(combine_grad_kernel<W, VB, 8>, dim3(T), dim3(kGradThreads), 0, st, p)
                    : launch_pdl(combine_grad_kernel<W, VB, 16>, dim3(T), dim3(kGradThreads), 0, st, p);
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
