// The end of a block: norm, gate, residual scale and residual, and the norm
// before the next block, in one pass; and a norm alone.
//
// A row's d values stand on the threads of a group (whole warps), several
// groups to a block for short rows.  out depends on y's norm and the next norm
// on out, so a row takes two sums over its threads, one after the other.  The
// algebra that would give both at once, sum (r + a v)^2 from three sums, cancels
// where the branch undoes the residual, and is not used.
//
// Bound: a row's chain of waits for long batches, the call's host time for a few
// tokens.  Three forms (figures of long runs over changing inputs):
//   ring       long batches: 8192 tokens of 3584 bf16 values, a gate a token: 51 us
//              for 235 MB, 0.68 of the measured copy bandwidth (registers: 77);
//              a norm alone 29 us, 0.60.  Three rows are in work on an SM there, one
//              at 4096 tokens of 8192 (73 us, 0.54; 36, 0.55), and each goes through
//              wait, squares, barrier, root and stores on its own: 1.5 us.  Rows of
//              float32 have more bytes a step: 8192 tokens of 2048, 47 us, 0.84
//   registers  a thread's 16 values stay; 8 tokens of 4096: 5 us on the device
//   C = 0      rows beyond that (d above 8192; value by value above 4096), read three
//              times: 256 tokens of 65536, a norm alone 23 us, 0.42
// Rows whose length, stride or address is not of whole 16-byte vectors (8 bf16 or 4
// float32 values) are read value by value (8192 tokens of 2001: 80 us, 0.24): a vector
// across the end of an odd row would hold the neighbour's values, and narrower
// vectors for even rows are not built.
#include "train_norm.cuh"

namespace moe {

namespace {

using namespace norm;

struct BlockOutParams {
    const char* y; int64_t ldy;
    const char* r; int64_t ldr;
    const void* gate; int gate_kind;
    const void *w_post, *w_next;
    char* out; int64_t ldo; char* next; int64_t ldn;  // strides in bytes
    float *rstd_post, *rstd_next;
    int T, d, n_vec, post, group, rows;
    float eps, offset, scale;
};

// (sum x^2 / d + eps)^-1/2; `again` sums (x 2^-80)^2, for rows whose squares pass float32's range,
// beside eps at the same scale (zero unless eps is large)
template <typename F>
__device__ __forceinline__ float rstd_of(Sums& sums, float ss, int d, float eps, F again) {
    float s[1] = {ss};
    sums.sum(s);
    const float m = s[0] / (float)d + eps;
    if (!(m < INFINITY)) {  // the same for every thread of the row; NaN stays NaN
        s[0] = again();
        sums.sum(s);
        return 0x1p-80f / sqrtf(s[0] / (float)d + eps * 0x1p-80f * 0x1p-80f);
    }
    return 1.f / sqrtf(m);
}

// E values a vector; C > 0: a thread's C vectors of a row stay in registers,
// C = 0: a row of any length, read again for each sum and for the result.
template <typename W, typename Y, int E, int C>
__global__ void __launch_bounds__(kMaxGroup) block_out_kernel(const BlockOutParams p) {
    constexpr bool kY = !std::is_same_v<Y, None>;
    constexpr int kN = C > 0 ? C : 1;
    __shared__ __align__(16) float red[kBlock / 32][2][kMaxGroupWarps][4];
    const int tid = threadIdx.x % p.group, g = threadIdx.x / p.group;
    Sums sums = {red[g], p.group / 32, tid / 32, 1 + g, p.group, 0};
    // f(slot, i) for the vectors i of this thread
    auto each = [&](auto f) {
        if constexpr (C > 0) {
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (tid + c * p.group < p.n_vec) f(c, tid + c * p.group);
        } else
            for (int i = tid; i < p.n_vec; i += p.group) f(0, i);
    };
    Raw<W, E> r[kN], wp[kN], wn[kN], gate[kN];
    Raw<Y, E> y[kN];
    auto load_weights = [&](int c, int i) {
        wp[c].zero();
        wn[c].zero();
        if (kY && p.w_post) wp[c].load(p.w_post, i);
        if (p.w_next) wn[c].load(p.w_next, i);
        if (kY && p.gate_kind == MOE_GATE_CHANNEL) gate[c].load(p.gate, i);
    };
    grid_dep_wait();
    grid_dep_launch();
    if (C > 0) each(load_weights);
    for (int64_t t = (int64_t)blockIdx.x * p.rows + g; t < p.T; t += (int64_t)gridDim.x * p.rows) {
        auto load_row = [&](int c, int i) {
            y[c].load(p.y + t * p.ldy, i);
            r[c].load(p.r + t * p.ldr, i);
            if (kY && p.gate_kind == MOE_GATE_FULL) gate[c].load(static_cast<const char*>(p.gate) + t * p.d * (int64_t)sizeof(W), i);
        };
        if (C > 0) each(load_row);
        float a = 1.f, gt = p.scale;
        if (kY && p.gate_kind == MOE_GATE_TOKEN) gt *= static_cast<const float*>(p.gate)[t];
        if (kY && p.post) {
            auto squares = [&](float s) {
                float ss = 0.f;
                each([&](int c, int i) {
                    if (C == 0) y[c].load(p.y + t * p.ldy, i);
#pragma unroll
                    for (int j = 0; j < E; ++j) ss = fmaf(y[c][j] * s, y[c][j] * s, ss);
                });
                return ss;
            };
            a = rstd_of(sums, squares(1.f), p.d, p.eps, [&] { return squares(0x1p-80f); });
            if (tid == 0 && p.rstd_post) p.rstd_post[t] = a;
        }
        float v[kN][E];  // out before its rounding
        auto value = [&](int c, int i) {
            if (C == 0) {
                load_weights(c, i);
                load_row(c, i);
            }
#pragma unroll
            for (int j = 0; j < E; ++j) {
                v[c][j] = r[c][j];
                if constexpr (kY) {
                    float b = y[c][j];
                    if (p.post) b = b * a * (p.offset + wp[c][j]);
                    if (p.gate_kind >= MOE_GATE_CHANNEL) b *= gate[c][j];
                    v[c][j] = fmaf(gt, b, v[c][j]);
                }
            }
        };
        if (C > 0) {
            each([&](int c, int i) {
                value(c, i);
                if (p.out) store<W, E>(p.out + t * p.ldo, i, v[c]);
            });
        }
        float b = 1.f;
        if (p.next) {
            auto squares = [&](float s) {
                float ss = 0.f;
                each([&](int c, int i) {
                    if (C == 0) value(c, i);
#pragma unroll
                    for (int j = 0; j < E; ++j) ss = fmaf(v[c][j] * s, v[c][j] * s, ss);
                });
                return ss;
            };
            b = rstd_of(sums, squares(1.f), p.d, p.eps, [&] { return squares(0x1p-80f); });
            if (tid == 0 && p.rstd_next) p.rstd_next[t] = b;
        }
        if (C == 0 || p.next)
            each([&](int c, int i) {
                if (C == 0) {
                    value(c, i);
                    if (p.out) store<W, E>(p.out + t * p.ldo, i, v[c]);
                }
                if (p.next) {
#pragma unroll
                    for (int j = 0; j < E; ++j) v[c][j] = v[c][j] * b * (p.offset + wn[c][j]);
                    store<W, E>(p.next + t * p.ldn, i, v[c]);
                }
            });
    }
}

// The same for long batches, rows coming through shared memory and the factors of
// the columns waiting there in float32: w_post' times the gate of a channel, and
// w_next'.
enum { kInResidual, kInY, kInGate };

template <typename W, typename Y, int C, bool FULL>
__global__ void __launch_bounds__(768, 1)
    block_out_ring_kernel(const __grid_constant__ BlockOutParams p, const __grid_constant__ RingParams rp) {
    constexpr bool kY = !std::is_same_v<Y, None>;
    constexpr int E = 16 / (int)sizeof(W), P = E / 2;
    extern __shared__ __align__(128) char smem[];
    __shared__ __align__(16) float red[kMaxGroups][2][kMaxGroupWarps][4];
    const int tid = threadIdx.x % p.group, grp = threadIdx.x / p.group;
    Sums sums = {red[grp], p.group / 32, tid / 32, 1 + grp, p.group, 0};
    const int groups = (int)gridDim.x * p.rows, first = (int)blockIdx.x * p.rows + grp;
    float *f_next = reinterpret_cast<float*>(smem), *f_post = f_next + (p.next ? p.d : 0);
    Ring ring(rp, smem, grp, p.T, first, groups);
    if (tid == 0) ring.init();
    fence_mbar_init();
    grid_dep_wait();
    grid_dep_launch();
    __syncthreads();
    if (tid == 0)
        for (int s = 0; s < rp.stages; ++s) ring.issue();
    for (int c = threadIdx.x; c < p.d; c += blockDim.x) {
        if (p.next) put_factor<E>(f_next, p.n_vec, c, p.offset + (p.w_next ? to_f32(static_cast<const W*>(p.w_next)[c]) : 0.f));
        if constexpr (kY) {
            float w = p.post ? p.offset + (p.w_post ? to_f32(static_cast<const W*>(p.w_post)[c]) : 0.f) : 1.f;
            if (p.gate_kind == MOE_GATE_CHANNEL) w *= to_f32(static_cast<const W*>(p.gate)[c]);
            put_factor<E>(f_post, p.n_vec, c, w);
        }
    }
    float gt1 = 1.f;  // a token's gate, fetched a row ahead
    auto fetch = [&](int t) {
        if (kY && p.gate_kind == MOE_GATE_TOKEN && t < p.T) gt1 = __ldg(static_cast<const float*>(p.gate) + t);
    };
    fetch(first);
    __syncthreads();
    for (int t = first; t < p.T; t += groups) {
        const float lost = ring.wait();
        const float gt = p.scale * gt1 + lost;
        fetch(t + groups);
        Pair v[C][P];
        Raw<W, E> gate[C];
        Raw<Y, E> y[C];
        auto each = [&](auto f) {
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (tid + c * p.group < p.n_vec) f(c, tid + c * p.group);
        };
        each([&](int c, int i) {
            Raw<W, E> r;
            r.load(ring.input(kInResidual), i);
            if constexpr (kY) y[c].load(ring.input(kInY), i);
            if constexpr (FULL) gate[c].load(ring.input(kInGate), i);
#pragma unroll
            for (int j = 0; j < P; ++j) v[c][j] = r.pair_of(j);
        });
        // the stage is free when every thread has brought its part of the row's first sum
        bool held = true;
        auto release = [&](float rstd) {
            if (held) {
                if (p.group == 32) __syncwarp();
                if (tid == 0) ring.issue(isnan(rstd));  // a thread that gave up made the sum NaN
                ring.next();
                held = false;
            }
        };
        float a = 1.f;
        if (kY && p.post) {
            auto squares = [&](float k) {
                Pair ss = 0;
                each([&](int c, int) {
#pragma unroll
                    for (int j = 0; j < P; ++j) {
                        const Pair x = mul(y[c].pair_of(j), pair(k));
                        ss = fma(x, x, ss);
                    }
                });
                return both(ss) + lost;
            };
            a = rstd_of(sums, squares(1.f), p.d, p.eps, [&] { return squares(0x1p-80f); });
            release(a);
            if (tid == 0 && p.rstd_post) p.rstd_post[t] = a;
        }
        if constexpr (kY)
            each([&](int c, int i) {
                Pair w[P];
                get_factors<E>(f_post, p.n_vec, i, w);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    Pair b = mul(mul(y[c].pair_of(j), pair(a)), w[j]);
                    if constexpr (FULL) b = mul(b, gate[c].pair_of(j));
                    v[c][j] = fma(pair(gt), b, v[c][j]);
                }
                store<W, P>(p.out + t * p.ldo, i, v[c]);
            });
        if (p.next) {
            auto squares = [&](float k) {
                Pair ss = 0;
                each([&](int c, int) {
#pragma unroll
                    for (int j = 0; j < P; ++j) {
                        const Pair x = mul(v[c][j], pair(k));
                        ss = fma(x, x, ss);
                    }
                });
                return both(ss) + lost;
            };
            const float b = rstd_of(sums, squares(1.f), p.d, p.eps, [&] { return squares(0x1p-80f); });
            release(b);
            if (tid == 0 && p.rstd_next) p.rstd_next[t] = b;
            each([&](int c, int i) {
                Pair w[P];
                get_factors<E>(f_next, p.n_vec, i, w);
#pragma unroll
                for (int j = 0; j < P; ++j) v[c][j] = mul(mul(v[c][j], pair(b)), w[j]);
                store<W, P>(p.next + t * p.ldn, i, v[c]);
            });
        }
    }
    if (tid == 0) ring.drain();
}

template <typename W, typename Y, int E, int C>
cudaError_t launch(BlockOutParams p, int sms, cudaStream_t st) {
    p.n_vec = p.d / E;
    const Shape s = shape_of(p.n_vec, C);
    p.group = s.group; p.rows = s.rows;
    int64_t blocks = ((int64_t)p.T + s.rows - 1) / s.rows;
    const int64_t most = (int64_t)sms * (s.threads() > 256 ? 2 : 4);
    if (blocks > most) blocks = most;
    return launch_pdl(block_out_kernel<W, Y, E, C>, dim3((unsigned)blocks), dim3(s.threads()), 0, st, p);
}

template <typename W, typename Y>
cudaError_t launch_vectors(const BlockOutParams& p, int e, int sms, cudaStream_t st) {
    constexpr int kWide = 16 / (int)sizeof(W);
    constexpr bool kY = !std::is_same_v<Y, None>;
    if (e == kWide && (p.post || p.next)) {  // without a norm there is no sum to wait for: registers give 5.1 TB/s
        constexpr int C = 16 / kWide;  // 16 values a thread
        BlockOutParams q = p;
        q.n_vec = p.d / e;
        RingParams r = {};
        const uint32_t row = (uint32_t)p.d * (uint32_t)sizeof(W);
        auto input = [&](int i, const char* src, int64_t stride, uint32_t bytes) { r.src[i] = src; r.stride[i] = stride; r.bytes[i] = bytes; };
        input(kInResidual, p.r, p.ldr, row);
        if constexpr (kY) input(kInY, p.y, p.ldy, (uint32_t)p.d * (uint32_t)sizeof(Y));
        if (kY && p.gate_kind == MOE_GATE_FULL) input(kInGate, static_cast<const char*>(p.gate), row, row);
        RingShape s;
        const uint32_t weights = ((p.next ? 1u : 0u) + (kY ? 1u : 0u)) * (uint32_t)p.d * 4;
        // Rows of 64 vectors or fewer leave the ring's threads too few (d 256, 65536 tokens: 58 us against 30 in
        // registers; d 512 37 against 34; d 1024 29 against 34), and so does a norm alone with one group (d 8192,
        // 4096 tokens: 41 against 36; with a branch 74 against 88).
        if (q.n_vec > 64 && q.n_vec <= kMaxGroup * C && ring_shape(r, p.T, q.n_vec, C, 768, kMaxGroups, weights, sms, s) &&
            (kY || s.groups > 1)) {
            q.group = s.group; q.rows = s.groups;
            auto kern = block_out_ring_kernel<W, Y, C, false>;
            if constexpr (kY)
                if (p.gate_kind == MOE_GATE_FULL) kern = block_out_ring_kernel<W, Y, C, true>;
            const cudaError_t err = allow_max_smem(kern);
            if (err != cudaSuccess) return err;
            return launch_pdl(kern, dim3((unsigned)s.blocks), dim3(s.group * s.groups), s.smem, st, q, r);
        }
    }
    return with_chunks<kWide>(p.d, e, [&](auto E, auto C) { return launch<W, Y, E, C>(p, sms, st); });
}

}  // namespace

cudaError_t launch_block_out(const NormArgs& a, cudaStream_t st) {
    const int64_t es = a.bf16 ? 2 : 4, ys = a.y_f32 ? 4 : es;
    BlockOutParams p;
    p.y = static_cast<const char*>(a.y); p.ldy = a.ldy * ys;
    p.r = static_cast<const char*>(a.residual); p.ldr = a.ldr * es;
    p.gate = a.gate; p.gate_kind = a.gate_kind; p.w_post = a.w_post; p.w_next = a.w_next;
    p.out = static_cast<char*>(a.out); p.ldo = a.ldo * es;
    p.next = static_cast<char*>(a.next); p.ldn = a.ldn * es;
    p.rstd_post = a.rstd_post; p.rstd_next = a.rstd_next;
    p.T = a.T; p.d = a.d; p.post = a.post; p.eps = a.eps; p.offset = a.offset; p.scale = a.scale;
    const int e = vector_values(a.bf16, a.d, {{a.y, p.ldy}, {a.residual, p.ldr}, {a.out, p.ldo}, {a.next, p.ldn},
                                              {a.gate_kind == MOE_GATE_TOKEN ? nullptr : a.gate, 0}, {a.w_post, 0}, {a.w_next, 0}});
    if (!a.bf16) return a.y ? launch_vectors<float, float>(p, e, a.sms, st) : launch_vectors<float, None>(p, e, a.sms, st);
    return !a.y     ? launch_vectors<__nv_bfloat16, None>(p, e, a.sms, st)
         : a.y_f32 ? launch_vectors<__nv_bfloat16, float>(p, e, a.sms, st)
                   : launch_vectors<__nv_bfloat16, __nv_bfloat16>(p, e, a.sms, st);
}

}  // namespace moe
