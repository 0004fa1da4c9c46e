// Rows kept in 8 bits: packed, restored (and gathered), and read by the
// combine's gradient.  The format stands in moe_train.h.
//
// The work is bytes.  A thread has eight columns of a row, four threads a
// block of 32: its largest magnitude takes two shuffles, and the turn from
// columns to the order of a matrix fragment two more.
#include "pack8.cuh"
#include "pairs.cuh"
#include "train.h"

namespace moe {

namespace {

using namespace pack8;

constexpr int kThreads = 256, kWarps = kThreads / 32, kCols = 256;  // columns of a warp

// A warp takes several pieces of kCols columns of a row at a time, all their loads
// before any use; a row's pieces are split evenly.  Gather of 4096 tokens, 8 slots
// each, in long runs over changing inputs, with at most four, five, seven, eight pieces:
// d 3584 56, 52, 49, 50 us; d 1536 26, 27, 23, 24; d 4096 59, 62, 60, 55; of 6 slots, d
// 2048, 25, 25, 27, 23.  Seven is half a row of 3584 and was taken there; it splits
// 2048 and 4096 into more turns than eight does.  At d 3584 the packing before it takes
// 12 us and the gather's bytes 37 at the copy bandwidth.
// The issue rate bounds the gather (74 % of the slots, DRAM at 0.58 of copy): a token is
// restored anew for each of its slots.
constexpr int kPackPieces = 4, kUnpackPieces = 7;

struct PackParams {
    const void* x; int64_t ldx;  // elements
    int8_t* q; uint8_t* scale;
    int64_t rows;
    int cols, nb, chunks, per;   // chunks of `per` pieces in a row
    const int32_t* index; int divisor;
    int64_t src_rows;
};

// f(row, first column of the chunk, the row's index) for the chunks of this warp,
// round robin; an index is fetched a chunk ahead
template <typename F>
__device__ __forceinline__ void each_chunk(const PackParams& p, F f) {
    const int64_t first = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5), stride = (int64_t)gridDim.x * kWarps;
    const int64_t dr = stride / p.chunks;
    const int dc = (int)(stride - dr * p.chunks);
    int64_t r = first / p.chunks;
    int c = (int)(first - r * p.chunks);
    int index = p.index && r < p.rows ? p.index[r] : 0;
    while (r < p.rows) {
        const int64_t r0 = r;
        const int c0 = c, i = index;
        r += dr;
        c += dc;
        if (c >= p.chunks) { c -= p.chunks; ++r; }
        if (p.index && r < p.rows) index = p.index[r];
        f(r0, c0 * p.per * kCols, i);
    }
}

template <typename W, bool VEC>
__global__ void __launch_bounds__(kThreads) pack_rows_kernel(const PackParams p) {
    const int lane = threadIdx.x & 31;
    grid_dep_wait();
    grid_dep_launch();
    each_chunk(p, [&](int64_t r, int c0, int) {
        float f[kPackPieces][8];
#pragma unroll
        for (int u = 0; u < kPackPieces; ++u)
            load8<W, VEC>(static_cast<const W*>(p.x) + r * p.ldx, c0 + u * kCols + lane * 8, u < p.per ? p.cols : 0, f[u]);
#pragma unroll
        for (int u = 0; u < kPackPieces; ++u) {
            if (u >= p.per || c0 + u * kCols >= p.cols) break;  // the same for the warp
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, magnitude(f[u][i]));
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
            const uint32_t E = exponent(m);
            const float inv = to_steps(E);
            uint32_t b[8];
            if (E == kTop)
#pragma unroll
                for (int i = 0; i < 8; ++i) f[u][i] = within(f[u][i], E);
#pragma unroll
            for (int i = 0; i < 8; ++i) b[i] = E == 255u ? 0u : quantise(f[u][i], inv);
            const uint2 w = to_packed(bytes4(b[0], b[1], b[2], b[3]), bytes4(b[4], b[5], b[6], b[7]));
            const int block = (c0 + u * kCols) / 32 + lane / 4;
            if (block < p.nb) {
                const int64_t at = r * p.nb + block;
                *reinterpret_cast<uint2*>(p.q + at * 32 + (lane & 3) * 8) = w;
                if ((lane & 3) == 0) p.scale[at] = (uint8_t)E;
            }
        }
    });
}

template <typename W, bool VEC>
__global__ void __launch_bounds__(kThreads) unpack_rows_kernel(const PackParams p) {
    const int lane = threadIdx.x & 31;
    grid_dep_wait();
    grid_dep_launch();
    each_chunk(p, [&](int64_t r, int c0, int index) {
        const int64_t src = !p.index ? r : index < 0 ? -1 : index / p.divisor;
        const bool there = src >= 0 && src < p.src_rows;
        uint2 w[kUnpackPieces];
        uint32_t E[kUnpackPieces];
#pragma unroll
        for (int u = 0; u < kUnpackPieces; ++u) {
            const int block = (c0 + u * kCols) / 32 + lane / 4;
            w[u] = make_uint2(0, 0);
            E[u] = 0;
            if (there && u < p.per && block < p.nb) {
                const int64_t at = src * p.nb + block;
                w[u] = *reinterpret_cast<const uint2*>(p.q + at * 32 + (lane & 3) * 8);
                E[u] = p.scale[at];
            }
        }
#pragma unroll
        for (int u = 0; u < kUnpackPieces; ++u) {
            if (u >= p.per || c0 + u * kCols >= p.cols) break;  // the same for the warp
            const float s = step(E[u]);
            const uint2 v = to_columns(w[u]);
            const uint32_t lo = biased(v.x), hi = biased(v.y);
            const float f[8] = {value<0>(lo) * s, value<1>(lo) * s, value<2>(lo) * s, value<3>(lo) * s,
                                value<0>(hi) * s, value<1>(hi) * s, value<2>(hi) * s, value<3>(hi) * s};
            store8<W, VEC>(static_cast<W*>(const_cast<void*>(p.x)) + r * p.ldx, c0 + u * kCols + lane * 8, p.cols, f);
        }
    });
}

// ---------------------------------------------------------------- combine, gradient
// A block takes a token at a time: dout's row, every slot's row of y in 8 bits for
// dgate, and its row of dy written.  A thread takes dout in two orders, by columns
// for dy and by the order of its two words for the products, so the words need no
// exchange.  Everything is fetched ahead: a token's rows and gates two tokens, dout
// one, the words of eight slots one piece of 256 columns.
// Bound: HBM, two thirds of it writes: 4096 tokens of 3584 values, 8 slots each: 71 us
// for 386 MB, 0.81 of the measured copy bandwidth, with three blocks of eight warps
// an SM.  Without the words ahead 78, with dout from global memory 76; two blocks 87,
// four (64 registers) 100; a branch a slot before its loads 171.  Two tokens a block
// (1001 of 1536 values, Granite shape) take 11.3 us, 11.9 with dout from global memory.
// Beyond eight slots 16 sums spill (170 to 220 bytes): 2048 tokens of 1536, 16 slots, 37
// us, 0.63.
constexpr int kGradWarps = 8, kGradBlocks = 3;  // a block's warps at most; blocks an SM

struct GradParams {
    const void* dout; int64_t lddout; const int8_t* q; const uint8_t* scale; const float* gate; const int32_t* inv;
    void* dy; float* dgate;
    int T, k, n_rows, d, nb;
};

// Eight slots' words of one piece, and their scales: lane l holds those of slot l / 4,
// blocks 2 (l % 4) and the next.
struct SlotWords {
    uint2 w[8];
    uint32_t scales;
};
__device__ __forceinline__ void load_slots(const GradParams& p, const int* rows, int c0, SlotWords& o) {
    const int lane = threadIdx.x & 31, block = min(c0 / 32 + lane / 4, p.nb - 1);  // past the last block dout has zeros
#pragma unroll
    for (int s = 0; s < 8; ++s)  // a slot without a row reads row 0, and its sum is not used
        o.w[s] = *reinterpret_cast<const uint2*>(p.q + ((int64_t)max(rows[s], 0) * p.nb + block) * 32 + (lane & 3) * 8);
    const uint8_t* e = p.scale + (int64_t)max(rows[lane >> 2], 0) * p.nb;
    const int b = c0 / 32 + (lane & 3) * 2;
    o.scales = e[min(b, p.nb - 1)] | (uint32_t)e[min(b + 1, p.nb - 1)] << 8;
}

// STAGED (with VEC): dout comes a token ahead by asynchronous copies to shared memory
template <typename W, bool VEC, bool STAGED, int KB>
__global__ void __launch_bounds__(kGradWarps * 32, kGradBlocks) combine_grad_packed_kernel(const GradParams p) {
    extern __shared__ __align__(16) unsigned char dout_s[];  // STAGED: [2][d]
    __shared__ float part[kGradWarps][KB];
    __shared__ int row_s[2][KB];  // this token's rows and the next one's
    __shared__ float gate_s[2][KB];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    int next_row = -1;
    float next_gate = 1.f;
    auto fetch = [&](int64_t t) {  // a token's rows and gates, two tokens ahead of their use
        if (tid < p.k && t < p.T) {
            const int r = p.inv[t * p.k + tid];
            next_row = r >= p.n_rows || r < -1 - p.n_rows ? -1 : r;  // out of range: no row
            if (p.gate) next_gate = p.gate[t * p.k + tid];
        }
    };
    auto keep = [&](int buf) {
        if (tid < KB) {
            row_s[buf][tid] = next_row;
            gate_s[buf][tid] = next_gate;
        }
    };
    auto fetch_dout = [&](int64_t t, int to) {
        if (STAGED && t < p.T) {
            const char* src = reinterpret_cast<const char*>(static_cast<const W*>(p.dout) + t * p.lddout);
            const int bytes = p.d * (int)sizeof(W);
            const uint32_t dst = smem_u32(dout_s) + to * bytes;
            for (int i = tid * 16; i < bytes; i += blockDim.x * 16)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + i), "l"(src + i) : "memory");
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    };
    grid_dep_wait();
    grid_dep_launch();
    fetch(blockIdx.x);
    fetch_dout(blockIdx.x, 0);
    keep(0);
    fetch(blockIdx.x + gridDim.x);
    __syncthreads();
    SlotWords ahead;  // of the next piece, eight slots at a time
    if (p.dgate) load_slots(p, row_s[0], warp * kCols, ahead);
    int buf = 0;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, buf ^= 1) {
        keep(buf ^ 1);
        if (STAGED) asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
        fetch(t + 2 * gridDim.x);
        fetch_dout(t + gridDim.x, buf ^ 1);
        const W* dout = STAGED ? reinterpret_cast<const W*>(dout_s) + buf * p.d : static_cast<const W*>(p.dout) + t * p.lddout;
        const int* rows = row_s[buf];
        float dot[KB];
#pragma unroll
        for (int s = 0; s < KB; ++s) dot[s] = 0.f;
        for (int c0 = warp * kCols; c0 < p.d; c0 += warps * kCols) {
            const int c = c0 + lane * 8;
            float g[8], h[8];
            load8<W, VEC>(dout, c, p.d, g);
            if (p.dgate) {
                load_interleaved<W, VEC>(dout, c, p.d, h);
#pragma unroll
                for (int s0 = 0; s0 < KB; s0 += 8) {
                    const SlotWords now = ahead;
                    if (s0 + 8 < KB) load_slots(p, rows + s0 + 8, c0, ahead);
                    else if (c0 + warps * kCols < p.d) load_slots(p, rows, c0 + warps * kCols, ahead);
                    else if (t + gridDim.x < p.T) load_slots(p, row_s[buf ^ 1], warp * kCols, ahead);
#pragma unroll
                    for (int s = 0; s < 8; ++s) {
                        const uint32_t lo = biased(now.w[s].x), hi = biased(now.w[s].y);
                        const uint32_t E = __shfl_sync(0xffffffffu, now.scales, s * 4 + lane / 8) >> (lane & 4 ? 8 : 0) & 0xffu;
                        // y itself, exact, before dout: a product of dout with whole steps can pass the range where dout y does not
                        const Pair f = pair(step(E));
                        auto y = [&](float a, float b) { return mul(add(pair(a, b), pair(-kRaw)), f); };
                        Pair v = mul(pair(h[0], h[1]), y(raw<0>(lo), raw<0>(hi)));
                        v = fma(pair(h[2], h[3]), y(raw<1>(lo), raw<1>(hi)), v);
                        v = fma(pair(h[4], h[5]), y(raw<2>(lo), raw<2>(hi)), v);
                        v = fma(pair(h[6], h[7]), y(raw<3>(lo), raw<3>(hi)), v);
                        dot[s0 + s] += both(v);
                    }
                }
            }
            if (p.dy) {
#pragma unroll
                for (int s = 0; s < KB; ++s) {
                    const int row = rows[s];
                    if (row == -1) continue;
                    float f[8] = {};
                    if (row >= 0) {
                        const Pair a = pair(gate_s[buf][s]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 v = halves(mul(pair(g[2 * i], g[2 * i + 1]), a));
                            f[2 * i] = v.x; f[2 * i + 1] = v.y;
                        }
                    }
                    store8<W, VEC>(static_cast<W*>(p.dy) + (int64_t)(row >= 0 ? row : -2 - row) * p.d, c, p.d, f);
                }
            }
        }
        if (p.dgate) {
#pragma unroll
            for (int s = 0; s < KB; ++s) {
                const float v = warp_sum(dot[s]);
                if (lane == 0) part[warp][s] = v;
            }
        }
        __syncthreads();
        if (p.dgate && tid < p.k) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < kGradWarps; ++w)
                if (w < warps) v += part[w][tid];
            p.dgate[t * p.k + tid] = rows[tid] >= 0 ? v : 0.f;
        }
    }
}

// rows that start on 16 bytes and hold whole vectors of them
bool vectors(const void* p, int64_t ld, int cols, bool bf16) {
    const int n = bf16 ? 8 : 4;
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % n == 0 && cols % n == 0;
}

void set_chunks(PackParams& p, int most) {
    const int pieces = (p.cols + kCols - 1) / kCols;
    p.chunks = (pieces + most - 1) / most;
    p.per = (pieces + p.chunks - 1) / p.chunks;
}

unsigned pack_grid(int64_t items, int sms) {
    const int64_t blocks = (items + kWarps - 1) / kWarps, most = (int64_t)sms * 8;
    return (unsigned)(blocks < most ? blocks : most);
}

}  // namespace

cudaError_t launch_pack_rows(int64_t rows, int cols, const void* x, int64_t ldx, bool bf16, int8_t* q, uint8_t* scale,
                             int sms, cudaStream_t st) {
    PackParams p = {};
    p.x = x; p.ldx = ldx; p.q = q; p.scale = scale; p.rows = rows; p.cols = cols; p.nb = pack_blocks(cols);
    set_chunks(p, kPackPieces);
    const dim3 grid(pack_grid(rows * p.chunks, sms)), block(kThreads);
    const bool vec = vectors(x, ldx, cols, bf16);
    if (bf16)
        return vec ? launch_pdl(pack_rows_kernel<__nv_bfloat16, true>, grid, block, 0, st, p)
                   : launch_pdl(pack_rows_kernel<__nv_bfloat16, false>, grid, block, 0, st, p);
    return vec ? launch_pdl(pack_rows_kernel<float, true>, grid, block, 0, st, p)
               : launch_pdl(pack_rows_kernel<float, false>, grid, block, 0, st, p);
}

cudaError_t launch_unpack_rows(int64_t src_rows, int cols, const int8_t* q, const uint8_t* scale, const int32_t* index,
                               int divisor, int64_t rows, void* out, int64_t ldo, bool bf16, int sms, cudaStream_t st) {
    PackParams p = {};
    p.x = out; p.ldx = ldo; p.q = const_cast<int8_t*>(q); p.scale = const_cast<uint8_t*>(scale); p.rows = rows;
    p.cols = cols; p.nb = pack_blocks(cols);
    set_chunks(p, kUnpackPieces);
    p.index = index; p.divisor = divisor; p.src_rows = src_rows;
    const dim3 grid(pack_grid(rows * p.chunks, sms)), block(kThreads);
    const bool vec = vectors(out, ldo, cols, bf16);
    if (bf16)
        return vec ? launch_pdl(unpack_rows_kernel<__nv_bfloat16, true>, grid, block, 0, st, p)
                   : launch_pdl(unpack_rows_kernel<__nv_bfloat16, false>, grid, block, 0, st, p);
    return vec ? launch_pdl(unpack_rows_kernel<float, true>, grid, block, 0, st, p)
               : launch_pdl(unpack_rows_kernel<float, false>, grid, block, 0, st, p);
}

template <typename W, bool VEC, bool STAGED>
static cudaError_t launch_grad(const GradParams& p, int sms, cudaStream_t st) {
    // as many warps as share a row's pieces evenly
    const int pieces = (p.d + kCols - 1) / kCols, turns = (pieces + kGradWarps - 1) / kGradWarps;
    const int warps = (pieces + turns - 1) / turns;
    const dim3 block(32 * warps);
    const size_t smem = STAGED ? 2 * (size_t)p.d * sizeof(W) : 0;
    int most = sms * (kGradWarps * kGradBlocks / warps);
    if (most > p.T) most = p.T;
    return p.k <= 8 ? launch_pdl(combine_grad_packed_kernel<W, VEC, STAGED, 8>, dim3(most), block, smem, st, p)
                    : launch_pdl(combine_grad_packed_kernel<W, VEC, STAGED, 16>, dim3(most), block, smem, st, p);
}

cudaError_t launch_combine_rows_grad_packed(const CombineRowsGradPackedArgs& a, cudaStream_t st) {
    GradParams p;
    p.dout = a.dout; p.lddout = a.lddout; p.q = a.q; p.scale = a.scale; p.gate = a.gate; p.inv = a.inv;
    p.dy = a.dy; p.dgate = a.dgate; p.T = a.T; p.k = a.k; p.n_rows = a.T * a.k; p.d = a.d; p.nb = pack_blocks(a.d);
    const bool vec = vectors(a.dout, a.lddout, a.d, a.bf16) && (!a.dy || vectors(a.dy, a.d, a.d, a.bf16));
    // two of dout's rows within the 48 KB that a block has without asking for more
    const bool staged = vec && 2LL * a.d * (a.bf16 ? 2 : 4) <= 40960;
    if (a.bf16)
        return staged ? launch_grad<__nv_bfloat16, true, true>(p, a.sms, st)
             : vec    ? launch_grad<__nv_bfloat16, true, false>(p, a.sms, st)
                      : launch_grad<__nv_bfloat16, false, false>(p, a.sms, st);
    return staged ? launch_grad<float, true, true>(p, a.sms, st)
         : vec    ? launch_grad<float, true, false>(p, a.sms, st)
                  : launch_grad<float, false, false>(p, a.sms, st);
}

}  // namespace moe
