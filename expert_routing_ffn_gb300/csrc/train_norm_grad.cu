// The gradient of a block's end (norm, gate, residual scale, residual, next
// norm) and of a norm alone.
//
// With xo = out b, g = dnext w_next', v = yn w_post' gate (post_norm) or y gate:
//   D = dout + b g - xo c,       c = b mean(g xo)
//   mean(D v) = mean((dout + b g) v) - c mean(xo v)
// so the three sums of a row, of g xo, (dout + b g) v and xo v, are taken at
// once; D and dy follow.  The error is that of D's own cancellation.
//
// Sums over the tokens: a group of threads that owns a row's columns takes
// many rows and keeps two sums a column, of dnext xo and of D v without the
// weights; dgate of a channel and dw_post are both multiples of the latter.
// A second launch adds the groups' sums in their order (8 us for the 152 blocks of
// a long batch, 3 in long runs).
//
// Bound: HBM beside the issue rate (53 % of the slots, DRAM at 0.72 of copy).  8192
// tokens of 3584 bf16 values, a gate a token: 75 us for 352 MB, both launches, on
// inputs that change (71 in long runs); rows from global memory to registers took 133,
// the ring without pairs and with a row's rstd fetched when it is needed 90.  16384
// tokens of 1536, a norm alone: 39 us for 201 MB (32 in long runs).  Eight values a
// thread instead of 16, 1024 threads of 64 registers: 105 us and 45.
//
// What does not take the ring is slower by far: rows whose inputs leave it no room, as
// 4096 tokens of 8192 with a float32 branch (245 us, 0.32 of copy; with a full gate,
// which also leaves the threads too few, 265, 0.37), for the register form spills there
// (92 and 132 bytes at two bf16 vectors a thread, 992 at four of float32: 300 tokens of
// 8192 33 us, 0.26); rows above 8192 (256 of 65536: 526 us, for 12 MB hold the column
// sums of 24 groups); value by value (8192 of 2001: 114 us, 0.25).  Many short rows
// leave most of the ring's threads without work: 65536 tokens of 256, a norm alone, 38 us,
// 0.39.
#include "train_norm.cuh"

namespace moe {

namespace {

using namespace norm;

struct BlockGradParams {
    const char* dout; int64_t lddout; const char* dnext; int64_t lddnext;
    const char* y; int64_t ldy; const char* out; int64_t ldo;
    const void* gate; int gate_kind;
    const void *w_post, *w_next;
    const float *rstd_post, *rstd_next;
    char* dr; int64_t lddr; char* dy; int64_t lddy;  // strides in bytes
    void* dgate;
    int T, d, n_vec, post, group, rows, columns;     // columns: sums over the tokens are asked for
    float offset, scale, inv_d;
    float* part;                                     // [groups][2][d]
    DevError* err;
};

// E values a vector; C > 0: a thread's C vectors of a row, and its columns' sums,
// stay in registers; C = 0: a row of any length, read twice, and sums that grow in
// the workspace.
template <typename W, typename Y, int E, int C>
__global__ void __launch_bounds__(kMaxGroup) block_grad_kernel(const BlockGradParams p) {
    constexpr bool kY = !std::is_same_v<Y, None>;
    constexpr int kN = C > 0 ? C : 1;
    __shared__ __align__(16) float red[kBlock / 32][2][kMaxGroupWarps][4];
    const int tid = threadIdx.x % p.group, grp = threadIdx.x / p.group;
    Sums sums = {red[grp], p.group / 32, tid / 32, 1 + grp, p.group, 0};
    // f(slot, i) for the vectors i of this thread
    auto each = [&](auto f) {
        if constexpr (C > 0) {
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (tid + c * p.group < p.n_vec) f(c, tid + c * p.group);
        } else
            for (int i = tid; i < p.n_vec; i += p.group) f(0, i);
    };
    Raw<W, E> dout[kN], dnext[kN], xo_[kN], wn[kN], wp[kN], gate[kN];
    Raw<Y, E> y[kN];
    float cn[kN][E], cp[kN][E];  // the columns' sums
#pragma unroll
    for (int c = 0; c < kN; ++c) {
        dout[c].zero(); dnext[c].zero(); xo_[c].zero(); wn[c].zero(); wp[c].zero();
#pragma unroll
        for (int j = 0; j < E; ++j) cn[c][j] = cp[c][j] = 0.f;
    }
    auto load_weights = [&](int c, int i) {
        if (p.w_next) wn[c].load(p.w_next, i);
        if (kY && p.w_post) wp[c].load(p.w_post, i);
        if (kY && p.gate_kind == MOE_GATE_CHANNEL) gate[c].load(p.gate, i);
    };
    grid_dep_wait();
    grid_dep_launch();
    if (C > 0) each(load_weights);
    const int64_t groups = (int64_t)gridDim.x * p.rows, first = (int64_t)blockIdx.x * p.rows + grp;
    float *col_next = p.part + first * 2 * p.d, *col_post = col_next + p.d;
    for (int64_t t = first; t < p.T; t += groups) {
        auto load_row = [&](int c, int i) {
            if (p.dout) dout[c].load(p.dout + t * p.lddout, i);
            if (p.dnext) {
                dnext[c].load(p.dnext + t * p.lddnext, i);
                xo_[c].load(p.out + t * p.ldo, i);
            }
            if constexpr (kY) {
                y[c].load(p.y + t * p.ldy, i);
                if (p.gate_kind == MOE_GATE_FULL) gate[c].load(static_cast<const char*>(p.gate) + t * p.d * (int64_t)sizeof(W), i);
            }
        };
        if (C > 0) each(load_row);
        const float a = kY && p.post ? p.rstd_post[t] : 1.f, b = p.dnext ? p.rstd_next[t] : 0.f;
        const float gt = kY && p.gate_kind == MOE_GATE_TOKEN ? static_cast<const float*>(p.gate)[t] : 1.f;
        float s[3] = {0.f, 0.f, 0.f};
        if (p.dnext || kY) {
            each([&](int c, int i) {
                if (C == 0) {
                    load_weights(c, i);
                    load_row(c, i);
                }
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    const float xo = xo_[c][j] * b, g = dnext[c][j] * (p.offset + wn[c][j]);
                    s[0] = fmaf(g, xo, s[0]);
                    if constexpr (kY) {
                        float v = y[c][j] * a;
                        if (p.post) v *= p.offset + wp[c][j];
                        if (p.gate_kind >= MOE_GATE_CHANNEL) v *= gate[c][j];
                        s[1] = fmaf(fmaf(b, g, dout[c][j]), v, s[1]);
                        s[2] = fmaf(xo, v, s[2]);
                    }
                }
            });
            sums.sum(s);
        }
        const float cc = b * (s[0] / (float)p.d);
        const float dv = s[1] - cc * s[2];                       // sum D v
        const float m = p.scale * gt * (dv / (float)p.d);        // mean(dp w_post' yn)
        if (kY && p.gate_kind == MOE_GATE_TOKEN && p.dgate && tid == 0) static_cast<float*>(p.dgate)[t] = p.scale * dv;
        each([&](int c, int i) {
            if (C == 0) {
                load_weights(c, i);
                load_row(c, i);
            }
            float D[E], dyv[E], dg[E];
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const float xo = xo_[c][j] * b, g = dnext[c][j] * (p.offset + wn[c][j]);
                D[j] = fmaf(b, g, dout[c][j]) - xo * cc;
                if (C == 0) cn[c][j] = cp[c][j] = 0.f;
                cn[c][j] = fmaf(dnext[c][j], xo, cn[c][j]);
                if constexpr (kY) {
                    const float yn = y[c][j] * a, w = p.post ? p.offset + wp[c][j] : 1.f;
                    const float ga = p.gate_kind >= MOE_GATE_CHANNEL ? gate[c][j] : gt, dq = p.scale * D[j];
                    dg[j] = dq * yn * w;
                    dyv[j] = dq * ga * w;
                    if (p.post) dyv[j] = a * (dyv[j] - yn * m);
                    const bool gated = p.gate_kind == MOE_GATE_TOKEN || p.gate_kind == MOE_GATE_FULL;
                    cp[c][j] = fmaf(D[j] * yn, gated ? ga : 1.f, cp[c][j]);
                }
            }
            if (p.dr) store<W, E>(p.dr + t * p.lddr, i, D);
            if constexpr (kY) {
                if (p.dy) store<Y, E>(p.dy + t * p.lddy, i, dyv);
                if (p.gate_kind == MOE_GATE_FULL && p.dgate)
                    store<W, E>(static_cast<char*>(p.dgate) + t * p.d * (int64_t)sizeof(W), i, dg);
            }
            if (C == 0 && p.columns) {
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    const int col = i * E + j;
                    col_next[col] = t == first ? cn[c][j] : col_next[col] + cn[c][j];
                    if constexpr (kY) col_post[col] = t == first ? cp[c][j] : col_post[col] + cp[c][j];
                }
            }
        });
    }
    if (C > 0 && p.columns && first < p.T)
        each([&](int c, int i) {
            store<float, E>(col_next, i, cn[c]);
            if constexpr (kY) store<float, E>(col_post, i, cp[c]);
        });
}

// The same for long batches, rows coming through shared memory.  The factors of
// the columns wait there too, in float32: w_next' and w_post' times the gate of a
// channel.  A row's values pass through registers once; of what the sums need,
// D without its projection (t), out and y stay.
enum { kInDout, kInDnext, kInOut, kInY, kInGate };
// Threads of a block, by the registers that 16 values of every input take.  A full
// gate at 512 threads spilled: 149 us and, in float32, 187, where 384 threads take
// 113 and 110 (8192 tokens, d 3584, and d 2048).
__host__ __device__ constexpr int ring_threads(bool branch, bool full) { return full ? 384 : branch ? 512 : 768; }

template <typename W, typename Y, int C, bool FULL>
__global__ void __launch_bounds__(ring_threads(!std::is_same_v<Y, None>, FULL), 1)
    block_grad_ring_kernel(const __grid_constant__ BlockGradParams p, const __grid_constant__ RingParams rp) {
    constexpr bool kY = !std::is_same_v<Y, None>;
    constexpr int E = 16 / (int)sizeof(W), P = E / 2, kSums = kY ? 2 : 1;  // sums of a column
    extern __shared__ __align__(128) char smem[];
    __shared__ __align__(16) float red[kMaxGroups][2][kMaxGroupWarps][4];
    const int tid = threadIdx.x % p.group, grp = threadIdx.x / p.group;
    Sums sums = {red[grp], p.group / 32, tid / 32, 1 + grp, p.group, 0};
    const int groups = (int)gridDim.x * p.rows, first = (int)blockIdx.x * p.rows + grp;
    float *f_next = reinterpret_cast<float*>(smem), *f_post = f_next + (p.dnext ? p.d : 0);
    Ring ring(rp, smem, grp, p.T, first, groups);
    if (tid == 0) ring.init();
    fence_mbar_init();
    grid_dep_wait();
    grid_dep_launch();
    __syncthreads();
    if (tid == 0)
        for (int s = 0; s < rp.stages; ++s) ring.issue();
    for (int c = threadIdx.x; c < p.d; c += blockDim.x) {
        if (p.dnext) put_factor<E>(f_next, p.n_vec, c, p.offset + (p.w_next ? to_f32(static_cast<const W*>(p.w_next)[c]) : 0.f));
        if constexpr (kY) {
            float w = p.post ? p.offset + (p.w_post ? to_f32(static_cast<const W*>(p.w_post)[c]) : 0.f) : 1.f;
            if (p.gate_kind == MOE_GATE_CHANNEL) w *= to_f32(static_cast<const W*>(p.gate)[c]);
            put_factor<E>(f_post, p.n_vec, c, w);
        }
    }
    // a row's own numbers, fetched a row ahead
    float a1 = 1.f, b1 = 0.f, gt1 = 1.f;
    auto fetch = [&](int t) {
        if (t >= p.T) return;
        if (kY && p.post) a1 = __ldg(p.rstd_post + t);
        if (p.dnext) b1 = __ldg(p.rstd_next + t);
        if (kY && p.gate_kind == MOE_GATE_TOKEN) gt1 = __ldg(static_cast<const float*>(p.gate) + t);
    };
    fetch(first);
    __syncthreads();
    Pair cn[C][P], cp[C][P];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int j = 0; j < P; ++j) cn[c][j] = cp[c][j] = 0;
    for (int t = first; t < p.T; t += groups) {
        const float lost = ring.wait(), a = a1, b = b1 + lost, gt = gt1 + lost;
        fetch(t + groups);
        Pair s0 = 0, s1 = 0, s2 = 0;
        Pair dt[C][P];  // dout + b dnext w_next'
        Raw<W, E> out[C], gate[C];
        Raw<Y, E> y[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = tid + c * p.group;
            if (i >= p.n_vec) continue;
#pragma unroll
            for (int j = 0; j < P; ++j) dt[c][j] = 0;
            if (p.dout) {
                Raw<W, E> v;
                v.load(ring.input(kInDout), i);
#pragma unroll
                for (int j = 0; j < P; ++j) dt[c][j] = v.pair_of(j);
            }
            out[c].zero();
            if (p.dnext) {
                Raw<W, E> v;
                v.load(ring.input(kInDnext), i);
                out[c].load(ring.input(kInOut), i);
                Pair w[P];
                get_factors<E>(f_next, p.n_vec, i, w);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const Pair dn = v.pair_of(j), xo = mul(out[c].pair_of(j), pair(b)), g = mul(dn, w[j]);
                    s0 = fma(g, xo, s0);
                    cn[c][j] = fma(dn, xo, cn[c][j]);
                    dt[c][j] = fma(pair(b), g, dt[c][j]);
                }
            }
            if constexpr (kY) {
                y[c].load(ring.input(kInY), i);
                Pair w[P];
                get_factors<E>(f_post, p.n_vec, i, w);
                if constexpr (FULL) {
                    gate[c].load(ring.input(kInGate), i);
#pragma unroll
                    for (int j = 0; j < P; ++j) w[j] = mul(w[j], gate[c].pair_of(j));
                }
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const Pair v = mul(mul(y[c].pair_of(j), pair(a)), w[j]);
                    s1 = fma(dt[c][j], v, s1);
                    s2 = fma(mul(out[c].pair_of(j), pair(b)), v, s2);
                }
            }
        }
        float cc, dv = 0.f;
        if constexpr (kY) {
            float s[3] = {both(s0), both(s1), both(s2)};
            sums.sum(s);
            cc = b * (s[0] * p.inv_d);
            dv = s[1] - cc * s[2];
        } else {
            float s[1] = {both(s0)};
            sums.sum(s);
            cc = b * (s[0] * p.inv_d);
        }
        if (p.group == 32) __syncwarp();
        if (tid == 0) ring.issue();  // into the stage that every thread has read
        ring.next();
        const float k2 = a * p.scale * gt, k3 = p.post ? -a * (p.scale * gt * (dv * p.inv_d)) : 0.f;
        if (kY && p.gate_kind == MOE_GATE_TOKEN && p.dgate && tid == 0) static_cast<float*>(p.dgate)[t] = p.scale * dv;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = tid + c * p.group;
            if (i >= p.n_vec) continue;
            Pair (&D)[P] = dt[c];
#pragma unroll
            for (int j = 0; j < P; ++j) D[j] = fma(mul(out[c].pair_of(j), pair(b)), pair(-cc), D[j]);
            if (p.dr) store<W, P>(p.dr + t * p.lddr, i, D);
            if constexpr (kY) {
                Pair w[P], dyv[P];
                get_factors<E>(f_post, p.n_vec, i, w);
                if constexpr (FULL) {
                    Pair dg[P];
#pragma unroll
                    for (int j = 0; j < P; ++j) {
                        const Pair yn = mul(y[c].pair_of(j), pair(a)), Dy = mul(D[j], yn), ga = gate[c].pair_of(j);
                        dg[j] = mul(mul(Dy, w[j]), pair(p.scale));
                        w[j] = mul(w[j], ga);
                        cp[c][j] = fma(Dy, ga, cp[c][j]);
                        dyv[j] = mul(mul(D[j], w[j]), pair(k2));
                        if (p.post) dyv[j] = fma(yn, pair(k3), dyv[j]);
                    }
                    if (p.dgate) store<W, P>(static_cast<char*>(p.dgate) + (int64_t)t * p.d * (int64_t)sizeof(W), i, dg);
                } else {
#pragma unroll
                    for (int j = 0; j < P; ++j) {
                        const Pair yn = mul(y[c].pair_of(j), pair(a));
                        cp[c][j] = fma(mul(D[j], yn), pair(gt), cp[c][j]);
                        dyv[j] = mul(mul(D[j], w[j]), pair(k2));
                        if (p.post) dyv[j] = fma(yn, pair(k3), dyv[j]);
                    }
                }
                if (p.dy) store<Y, P>(p.dy + t * p.lddy, i, dyv);
            }
        }
    }
    if (tid == 0) ring.drain();
    if (ring.dead) set_error(p.err, MOE_ERR_TIMEOUT, first);
    if (p.columns) {
        // the groups' sums meet in shared memory, where the rings were, and leave as one
        float* mine = reinterpret_cast<float*>(smem + rp.rings) + (size_t)grp * kSums * p.d;
        __syncthreads();
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = tid + c * p.group;
            if (i >= p.n_vec) continue;
            store<float, P>(mine, i, cn[c]);
            if constexpr (kY) store<float, P>(mine + p.d, i, cp[c]);
        }
        __syncthreads();
        const float* all = reinterpret_cast<const float*>(smem + rp.rings);
        for (int c = threadIdx.x; c < kSums * p.d; c += blockDim.x) {
            float v = all[c];
            for (int g = 1; g < p.rows; ++g) v += all[(size_t)g * kSums * p.d + c];
            p.part[(int64_t)blockIdx.x * 2 * p.d + c] = v;
        }
    }
}

// The groups' sums of 32 columns, added by the block's warps, each in the groups'
// order, then in the warps'.  A warp for every eight groups: 912 groups of 1536
// columns took eight warps 13 us.
struct ColumnParams {
    const float* part;
    int groups, d, gate_kind, post, accumulate;
    float offset, scale;
    const void *gate, *w_post;
    void *dw_next, *dw_post, *dgate;  // dgate: of a channel
};

template <typename W, typename G>
__global__ void __launch_bounds__(1024) column_sums_kernel(const ColumnParams p) {
    __shared__ float red[32][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, col = blockIdx.x * 32 + lane, which = blockIdx.y;
    grid_dep_wait();
    grid_dep_launch();
    float s = 0.f;
    if (col < p.d && (which || p.dw_next))
#pragma unroll 8
        for (int g = warp; g < p.groups; g += warps) s += __ldcg(p.part + ((int64_t)g * 2 + which) * p.d + col);
    red[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && col < p.d) {
        s = 0.f;
        for (int w = 0; w < warps; ++w) s += red[w][lane];
        auto put = [&](void* to, float v) {
            G* o = static_cast<G*>(to) + col;
            if constexpr (sizeof(G) == 4) *o = p.accumulate ? *o + v : v;
            else *o = __float2bfloat16_rn(v);
        };
        if (!which) {
            if (p.dw_next) put(p.dw_next, s);
        } else {
            s *= p.scale;
            if (p.dw_post) put(p.dw_post, p.gate_kind == MOE_GATE_CHANNEL ? s * to_f32(static_cast<const W*>(p.gate)[col]) : s);
            if (p.dgate) put(p.dgate, p.post ? s * (p.offset + (p.w_post ? to_f32(static_cast<const W*>(p.w_post)[col]) : 0.f)) : s);
        }
    }
}

template <typename W, typename Y, int E, int C>
cudaError_t launch(BlockGradParams p, int parts, int sms, int* groups, cudaStream_t st) {
    p.n_vec = p.d / E;
    const Shape s = shape_of(p.n_vec, C);
    p.group = s.group; p.rows = s.rows;
    int64_t blocks = ((int64_t)p.T + s.rows - 1) / s.rows, most = (int64_t)sms * 2;
    if (p.columns && most > parts / s.rows) most = parts / s.rows;
    if (most < 1) { most = 1; p.rows = 1; }
    if (blocks > most) blocks = most;
    const int64_t all = blocks * p.rows;
    *groups = (int)(all < p.T ? all : p.T);
    return launch_pdl(block_grad_kernel<W, Y, E, C>, dim3((unsigned)blocks), dim3(p.group * p.rows), 0, st, p);
}

template <typename W, typename Y>
cudaError_t launch_vectors(const BlockGradParams& p, int e, int parts, int sms, int* groups, cudaStream_t st) {
    constexpr int kWide = 16 / (int)sizeof(W);
    constexpr bool kY = !std::is_same_v<Y, None>;
    if (e == kWide) {
        constexpr int C = 16 / kWide;  // 16 values a thread
        BlockGradParams q = p;
        q.n_vec = p.d / e;
        RingParams r = {};
        const uint32_t row = (uint32_t)p.d * (uint32_t)sizeof(W);
        auto input = [&](int i, const char* src, int64_t stride, uint32_t bytes) { r.src[i] = src; r.stride[i] = stride; r.bytes[i] = bytes; };
        input(kInDout, p.dout, p.lddout, row);
        input(kInDnext, p.dnext, p.lddnext, row);
        input(kInOut, p.dnext ? p.out : nullptr, p.ldo, row);
        if constexpr (kY) input(kInY, p.y, p.ldy, (uint32_t)p.d * (uint32_t)sizeof(Y));
        if (kY && p.gate_kind == MOE_GATE_FULL) input(kInGate, static_cast<const char*>(p.gate), row, row);
        RingShape s;
        const uint32_t weights = ((p.dnext ? 1u : 0u) + (kY ? 1u : 0u)) * (uint32_t)p.d * 4;
        // The sums of a group (two float32 a column with y, else one) fit where its ring was: at least two stages of
        // two rows or more of at least two bytes a value.
        if (q.n_vec <= kMaxGroup * C && (!p.columns || parts >= sms) && ring_shape(r, p.T, q.n_vec, C, ring_threads(kY, p.gate_kind == MOE_GATE_FULL), kMaxGroups, weights, sms, s)) {
            q.group = s.group; q.rows = s.groups;
            auto kern = block_grad_ring_kernel<W, Y, C, false>;
            if constexpr (kY)
                if (p.gate_kind == MOE_GATE_FULL) kern = block_grad_ring_kernel<W, Y, C, true>;
            cudaError_t err = allow_max_smem(kern);
            if (err != cudaSuccess) return err;
            *groups = s.blocks;
            return launch_pdl(kern, dim3((unsigned)s.blocks), dim3(s.group * s.groups), s.smem, st, q, r);
        }
    }
    return with_chunks<kWide>(p.d, e, [&](auto E, auto C) { return launch<W, Y, E, C>(p, parts, sms, groups, st); });
}

}  // namespace

cudaError_t launch_block_out_grad(const NormGradArgs& a, cudaStream_t st, int* launches) {
    const int64_t es = a.bf16 ? 2 : 4, ys = a.y_f32 ? 4 : es;
    BlockGradParams p;
    p.dout = static_cast<const char*>(a.dout); p.lddout = a.lddout * es;
    p.dnext = static_cast<const char*>(a.dnext); p.lddnext = a.lddnext * es;
    p.y = static_cast<const char*>(a.y); p.ldy = a.ldy * ys;
    p.out = static_cast<const char*>(a.out); p.ldo = a.ldo * es;
    p.gate = a.gate; p.gate_kind = a.gate_kind; p.w_post = a.w_post; p.w_next = a.w_next;
    p.rstd_post = a.rstd_post; p.rstd_next = a.rstd_next;
    p.dr = static_cast<char*>(a.dresidual); p.lddr = a.lddr * es;
    p.dy = static_cast<char*>(a.dy); p.lddy = a.lddy * ys;
    const bool channel = a.gate_kind == MOE_GATE_CHANNEL;
    p.dgate = channel ? nullptr : a.dgate;
    p.T = a.T; p.d = a.d; p.post = a.post; p.offset = a.offset; p.scale = a.scale; p.part = a.part;
    p.inv_d = 1.f / (float)a.d;
    p.err = a.err;
    p.columns = a.dw_post || a.dw_next || (channel && a.dgate);
    const int parts = norm_parts(a.T, a.d);
    int groups = 0;
    *launches = 1;
    cudaError_t e;
    const int v = vector_values(a.bf16, a.d, {{a.dout, p.lddout}, {a.dnext, p.lddnext}, {a.y, p.ldy}, {a.dnext ? a.out : nullptr, p.ldo},
                                              {a.gate_kind == MOE_GATE_TOKEN ? nullptr : a.gate, 0}, {a.w_post, 0}, {a.w_next, 0},
                                              {a.dresidual, p.lddr}, {a.dy, p.lddy}, {a.gate_kind == MOE_GATE_FULL ? a.dgate : nullptr, 0}});
    if (!a.bf16) e = a.y ? launch_vectors<float, float>(p, v, parts, a.sms, &groups, st) : launch_vectors<float, None>(p, v, parts, a.sms, &groups, st);
    else if (!a.y) e = launch_vectors<__nv_bfloat16, None>(p, v, parts, a.sms, &groups, st);
    else if (a.y_f32) e = launch_vectors<__nv_bfloat16, float>(p, v, parts, a.sms, &groups, st);
    else e = launch_vectors<__nv_bfloat16, __nv_bfloat16>(p, v, parts, a.sms, &groups, st);
    if (e != cudaSuccess || !p.columns) return e;
    ColumnParams c;
    c.part = a.part; c.groups = groups; c.d = a.d; c.gate_kind = a.gate_kind; c.post = a.post; c.accumulate = a.accumulate;
    c.offset = a.offset; c.scale = a.scale; c.gate = a.gate; c.w_post = a.w_post;
    c.dw_next = a.dw_next; c.dw_post = a.dw_post; c.dgate = channel ? a.dgate : nullptr;
    const dim3 grid((unsigned)((a.d + 31) / 32), a.y ? 2 : 1), block(32 * (groups >= 256 ? 32 : (groups + 7) / 8));
    *launches = 2;
    if (!a.bf16) return launch_pdl(column_sums_kernel<float, float>, grid, block, 0, st, c);
    return a.grads_f32 ? launch_pdl(column_sums_kernel<__nv_bfloat16, float>, grid, block, 0, st, c)
                       : launch_pdl(column_sums_kernel<__nv_bfloat16, __nv_bfloat16>, grid, block, 0, st, c);
}

}  // namespace moe
