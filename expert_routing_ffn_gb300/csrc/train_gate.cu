// The router's gradient: from the gates of a token's slots back through the
// (optional) renormalisation and the softmax to the logits, with the
// load-balance loss.
//   v_e  = sum of d gate over the token's slots on e  +  c N f_e / T
//   dl_e = p_e (v_e - sum_j p_j v_j)
// Renormalised gates w_s = p_s / sum_j p_j have a gradient of their own form:
// through them dl_e gains sum over the slots on e of w_s (dgate_s - sum_j
// dgate_j w_j), whose sum over e is zero, and v_e keeps the load's term alone.
// The slots' sum may be as small as float32 goes, and 1 / 2^-128 is no float32
// number, while the w_s are ordinary: only they are formed.
//   loss = c N sum_e f_e P_e,  f_e = slots on e / (T k),  P_e = mean_t p_te
// T x N floats in and out: latency decides at every size (16384 tokens of 40
// experts, 6 MB: 14 us in two launches).  A warp owns a token, up to four at a
// time so that their loads are in flight together, a lane every 32nd expert.  f and P need the
// whole batch first; their sums are taken by at most kGateParts blocks in
// token order and added up by every block of the second launch, so no atomic
// decides an order.  Without a balance term that first launch is left out.
#include "common.cuh"
#include "train.h"

namespace moe {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32, kBlocksPerSm = 4;

struct GateParams {
    const float* prob; const int32_t* idx; const float* dgate;
    int T, N, k, parts, rows_per_part;
    float balance;
    float *dlogits, *loss, *part;
};

// part[b][0][e] = slots on e, part[b][1][e] = sum of p_te, over block b's tokens
__global__ void __launch_bounds__(kThreads) gate_load_kernel(const GateParams p) {
    extern __shared__ float gsm[];
    int* slots = reinterpret_cast<int*>(gsm);  // [N]
    float* psum = gsm + p.N;                   // [kWarps][N]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < p.N; i += kThreads) slots[i] = 0;
    __syncthreads();
    grid_dep_wait();
    const int64_t t0 = (int64_t)blockIdx.x * p.rows_per_part;
    const int64_t t1 = min(t0 + p.rows_per_part, (int64_t)p.T);
    for (int64_t i = t0 * p.k + tid; i < t1 * p.k; i += kThreads) {
        const int e = p.idx[i];
        if (e >= 0 && e < p.N) atomicAdd(&slots[e], 1);
    }
    for (int e = lane; e < p.N; e += 32) {
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        int64_t t = t0 + warp;
        for (; t + 3 * kWarps < t1; t += 4 * kWarps)
#pragma unroll
            for (int u = 0; u < 4; ++u) s[u] += p.prob[(t + u * kWarps) * p.N + e];
        for (; t < t1; t += kWarps) s[0] += p.prob[t * p.N + e];
        psum[warp * p.N + e] = (s[0] + s[1]) + (s[2] + s[3]);
    }
    __syncthreads();
    float* out = p.part + (size_t)blockIdx.x * 2 * p.N;
    for (int e = tid; e < p.N; e += kThreads) {
        float s = 0.f;
        for (int w = 0; w < kWarps; ++w) s += psum[w * p.N + e];
        out[e] = (float)slots[e];  // below 2^24: exact
        out[p.N + e] = s;
    }
    grid_dep_launch();
}

// NV: experts per lane.  Four blocks an SM, which is the grid's size: where the compiler took 78 registers (NV 16)
// a fourth of the blocks had to wait, and 16384 tokens of 500 experts took 71 us instead of 59.
template <int NV, bool RENORM>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) gate_grad_kernel(const GateParams p) {
    extern __shared__ float gsm[];
    float* load = gsm;            // [N] c N f_e / T
    float* lterm = gsm + p.N;     // [N] f_e P_e
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dep_wait();
    const bool bal = p.parts > 0;
    if (bal) {
        // the parts in kSlices runs, a run a thread, then the runs in order
        constexpr int kSlices = 8;
        float* run = gsm + 2 * p.N;  // [kSlices][2][N]
        for (int i = tid; i < kSlices * p.N; i += kThreads) {
            const int q = i / p.N, e = i - q * p.N;
            float c = 0.f, s = 0.f;
#pragma unroll 8
            for (int b = q; b < p.parts; b += kSlices) {
                c += __ldcg(p.part + (size_t)b * 2 * p.N + e);
                s += __ldcg(p.part + (size_t)b * 2 * p.N + p.N + e);
            }
            run[(q * 2) * p.N + e] = c;
            run[(q * 2 + 1) * p.N + e] = s;
        }
        __syncthreads();
        for (int e = tid; e < p.N; e += kThreads) {
            float c = 0.f, s = 0.f;
#pragma unroll
            for (int q = 0; q < kSlices; ++q) {
                c += run[(q * 2) * p.N + e];
                s += run[(q * 2 + 1) * p.N + e];
            }
            const float f = c / ((float)p.T * (float)p.k);
            load[e] = p.balance * (float)p.N / (float)p.T * f;
            lterm[e] = f * (s / (float)p.T);
        }
        __syncthreads();
    }
    if (blockIdx.x == 0 && tid == 0 && p.loss) {
        float l = 0.f;
        if (bal)
            for (int e = 0; e < p.N; ++e) l += lterm[e];
        p.loss[0] = p.balance * (float)p.N * l;
    }
    // kU tokens at a time: their loads are in flight together
    constexpr int kU = NV <= 2 ? 4 : NV <= 4 ? 2 : 1;
    const int64_t stride = (int64_t)gridDim.x * kWarps;
    for (int64_t t0 = (int64_t)blockIdx.x * kWarps + warp; t0 < p.T; t0 += kU * stride) {
        int my_e[kU];
        float my_d[kU], my_p[kU], q[kU][NV], v[kU][NV];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int64_t t = t0 + u * stride;
            my_e[u] = -1;
            my_d[u] = my_p[u] = 0.f;
            if (lane < p.k && t < p.T) {
                my_e[u] = p.idx[t * p.k + lane];
                my_d[u] = p.dgate[t * p.k + lane];
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int e = i * 32 + lane;
                q[u][i] = e < p.N && t < p.T ? p.prob[t * p.N + e] : 0.f;
                v[u][i] = bal && e < p.N ? load[e] : 0.f;
            }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            if (my_e[u] < 0 || my_e[u] >= p.N) my_e[u] = -1, my_d[u] = 0.f;
            else if (RENORM) my_p[u] = p.prob[(t0 + u * stride) * p.N + my_e[u]];
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            if (RENORM) {
                const float total = warp_sum(my_p[u]);
                const float w = total > 0.f ? my_p[u] / total : 0.f;
                const float mean = warp_sum(my_d[u] * w);
                my_d[u] = w * (my_d[u] - mean);
            }
            // the slots' terms: into v (gates that are probabilities), or into dl itself (renormalised)
            auto add_slots = [&] {
                for (int s = 0; s < p.k; ++s) {
                    const int e = __shfl_sync(0xffffffffu, my_e[u], s);
                    const float dg = __shfl_sync(0xffffffffu, my_d[u], s);
#pragma unroll
                    for (int i = 0; i < NV; ++i)
                        if (e == i * 32 + lane) v[u][i] += dg;
                }
            };
            if (!RENORM) add_slots();
            float dot = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i) dot = fmaf(q[u][i], v[u][i], dot);
            dot = warp_sum(dot);
#pragma unroll
            for (int i = 0; i < NV; ++i) v[u][i] = q[u][i] * (v[u][i] - dot);
            if (RENORM) add_slots();
            const int64_t t = t0 + u * stride;
            if (t < p.T) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (i * 32 + lane < p.N) p.dlogits[t * p.N + i * 32 + lane] = v[u][i];
            }
        }
    }
    grid_dep_launch();
}

template <bool RENORM>
cudaError_t launch_grad(const GateParams& p, int nv, dim3 grid, size_t smem, cudaStream_t st) {
    return nv <= 1 ? launch_pdl(gate_grad_kernel<1, RENORM>, grid, dim3(kThreads), smem, st, p)
         : nv <= 2 ? launch_pdl(gate_grad_kernel<2, RENORM>, grid, dim3(kThreads), smem, st, p)
         : nv <= 4 ? launch_pdl(gate_grad_kernel<4, RENORM>, grid, dim3(kThreads), smem, st, p)
         : nv <= 8 ? launch_pdl(gate_grad_kernel<8, RENORM>, grid, dim3(kThreads), smem, st, p)
                   : launch_pdl(gate_grad_kernel<16, RENORM>, grid, dim3(kThreads), smem, st, p);
}

}  // namespace

cudaError_t launch_gate_grad(const GateGradArgs& a, cudaStream_t st, int* launches) {
    GateParams p;
    p.prob = a.prob; p.idx = a.idx; p.dgate = a.dgate;
    p.T = a.T; p.N = a.N; p.k = a.k; p.balance = a.balance;
    p.dlogits = a.dlogits; p.loss = a.loss; p.part = a.part;
    p.parts = 0; p.rows_per_part = 0;
    *launches = 1;
    if (a.balance > 0.f) {
        // 32 tokens a block at least: shorter batches have fewer blocks to add up
        int parts = (a.T + 31) / 32;
        if (parts > kGateParts) parts = kGateParts;
        p.rows_per_part = (a.T + parts - 1) / parts;
        p.parts = (a.T + p.rows_per_part - 1) / p.rows_per_part;
        const size_t smem = (size_t)a.N * (1 + kWarps) * 4;
        cudaError_t e = launch_pdl(gate_load_kernel, dim3(p.parts), dim3(kThreads), smem, st, p);
        if (e != cudaSuccess) return e;
        *launches = 2;
    }
    int64_t blocks = ((int64_t)a.T + kWarps - 1) / kWarps;
    if (blocks > (int64_t)a.sms * kBlocksPerSm) blocks = (int64_t)a.sms * kBlocksPerSm;
    const dim3 grid((unsigned)blocks);
    const size_t smem = (size_t)a.N * 2 * 4 * (p.parts > 0 ? 9 : 1);
    const int nv = (a.N + 31) / 32;
    return a.renorm ? launch_grad<true>(p, nv, grid, smem, st) : launch_grad<false>(p, nv, grid, smem, st);
}

}  // namespace moe
