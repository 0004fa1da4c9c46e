// The end of a block: norm, gate, residual scale and residual, and the norm
// before the next block, in one pass; and a norm alone.
//
// A row's d values stand on the threads of a group (whole warps), several
// groups to a block for short rows.  out depends on y's norm and the next norm
// on out, so a row takes two sums over its threads, one after the other.  The
// algebra that would give both at once, sum (r + a v)^2 from three sums, cancels
// where the branch undoes the residual, and is not used.
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

// (sum x^2 / d + eps)^-1/2; `again` sums (x 2^-80)^2, for rows whose squares pass float32's range
template <typename F>
__device__ __forceinline__ float rstd_of(Sums& sums, float ss, int d, float eps, F again) {
    float s[1] = {ss};
    sums.sum(s);
    if (!(s[0] < INFINITY)) {  // the same for every thread of the row; NaN stays NaN
        s[0] = again();
        sums.sum(s);
        return 0x1p-80f / sqrtf(s[0] / (float)d);
    }
    return 1.f / sqrtf(s[0] / (float)d + eps);
}

template <typename W, typename Y, int E>
__global__ void __launch_bounds__(kMaxGroup) block_out_kernel(const BlockOutParams p) {
    constexpr bool kY = !std::is_same_v<Y, None>;
    __shared__ float red[kBlock / 32][2][kMaxGroupWarps][4];
    const int tid = threadIdx.x % p.group, g = threadIdx.x / p.group;
    Sums sums = {red[g], p.group / 32, tid / 32, 1 + g, p.group, 0};
    grid_dep_wait();
    for (int64_t t = (int64_t)blockIdx.x * p.rows + g; t < p.T; t += (int64_t)gridDim.x * p.rows) {
        const char *yrow = p.y + t * p.ldy, *rrow = p.r + t * p.ldr;
        float a = 1.f, gt = p.scale;
        if (kY && p.gate_kind == MOE_GATE_TOKEN) gt *= static_cast<const float*>(p.gate)[t];
        if (kY && p.post) {
            auto squares = [&](float s) {
                float ss = 0.f;
                for (int i = tid; i < p.n_vec; i += p.group) {
                    Raw<Y, E> y;
                    y.load(yrow, i);
#pragma unroll
                    for (int j = 0; j < E; ++j) ss = fmaf(y[j] * s, y[j] * s, ss);
                }
                return ss;
            };
            a = rstd_of(sums, squares(1.f), p.d, p.eps, [&] { return squares(0x1p-80f); });
            if (tid == 0 && p.rstd_post) p.rstd_post[t] = a;
        }
        // vector i of out, before its rounding
        auto value = [&](int i, float (&v)[E]) {
            Raw<W, E> r, w, gate;
            Raw<Y, E> y;
            r.load(rrow, i);
            y.load(yrow, i);
            w.zero();
            if (kY && p.w_post) w.load(p.w_post, i);
            if (kY && p.gate_kind == MOE_GATE_CHANNEL) gate.load(p.gate, i);
            if (kY && p.gate_kind == MOE_GATE_FULL) gate.load(static_cast<const char*>(p.gate) + t * p.d * (int64_t)sizeof(W), i);
#pragma unroll
            for (int j = 0; j < E; ++j) {
                v[j] = r[j];
                if constexpr (kY) {
                    float b = y[j];
                    if (p.post) b = b * a * (p.offset + w[j]);
                    if (p.gate_kind >= MOE_GATE_CHANNEL) b *= gate[j];
                    v[j] = fmaf(gt, b, v[j]);
                }
            }
        };
        float b = 1.f;
        if (p.next) {
            auto squares = [&](float s) {
                float ss = 0.f;
                for (int i = tid; i < p.n_vec; i += p.group) {
                    float v[E];
                    value(i, v);
#pragma unroll
                    for (int j = 0; j < E; ++j) ss = fmaf(v[j] * s, v[j] * s, ss);
                }
                return ss;
            };
            b = rstd_of(sums, squares(1.f), p.d, p.eps, [&] { return squares(0x1p-80f); });
            if (tid == 0 && p.rstd_next) p.rstd_next[t] = b;
        }
        for (int i = tid; i < p.n_vec; i += p.group) {
            float v[E];
            value(i, v);
            if (p.out) store<W, E>(p.out + t * p.ldo, i, v);
            if (p.next) {
                Raw<W, E> w;
                w.zero();
                if (p.w_next) w.load(p.w_next, i);
#pragma unroll
                for (int j = 0; j < E; ++j) v[j] = v[j] * b * (p.offset + w[j]);
                store<W, E>(p.next + t * p.ldn, i, v);
            }
        }
    }
    grid_dep_launch();
}

template <typename W, typename Y, int E>
cudaError_t launch(BlockOutParams p, int sms, cudaStream_t st) {
    p.n_vec = p.d / E;
    const Shape s = shape_of(p.n_vec, 0);
    p.group = s.group; p.rows = s.rows;
    int64_t blocks = ((int64_t)p.T + s.rows - 1) / s.rows;
    if (blocks > (int64_t)sms * 8) blocks = (int64_t)sms * 8;
    return launch_pdl(block_out_kernel<W, Y, E>, dim3((unsigned)blocks), dim3(s.threads()), 0, st, p);
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
    if (!a.bf16) return a.y ? launch<float, float, 1>(p, a.sms, st) : launch<float, None, 1>(p, a.sms, st);
    return !a.y     ? launch<__nv_bfloat16, None, 1>(p, a.sms, st)
         : a.y_f32 ? launch<__nv_bfloat16, float, 1>(p, a.sms, st)
                   : launch<__nv_bfloat16, __nv_bfloat16, 1>(p, a.sms, st);
}

}  // namespace moe
