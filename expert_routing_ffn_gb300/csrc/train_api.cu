// C ABI of the training step (include/moe_train.h): argument checks,
// workspace layout and the launches of each call.
#include <cmath>
#include <initializer_list>

#include "common.cuh"
#include "train.h"

using namespace moe;

namespace moe {
void note_launches(int n);
}

namespace {

inline cudaStream_t S(void* s) { return reinterpret_cast<cudaStream_t>(s); }
bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

#define TRAIN_TRY(expr)                                    \
    do {                                                   \
        moe_status _st = (expr);                           \
        if (_st != MOE_OK) return _st;                     \
    } while (0)

#define TRAIN_CUDA(expr)                                   \
    do {                                                   \
        cudaError_t _e = (expr);                           \
        if (_e != cudaSuccess) return cuda_failed(_e, #expr); \
    } while (0)

moe_status check_dims(const moe_dims* D) {
    if (!D) return MOE_ERR_INVALID_ARG;
    if (D->T < 0 || D->d <= 0 || D->N <= 0 || D->k <= 0 || D->I <= 0) return MOE_ERR_INVALID_ARG;
    if (D->wtype != MOE_DTYPE_BF16 && D->wtype != MOE_DTYPE_F32) return MOE_ERR_UNSUPPORTED;
    if (D->N > kTrainMaxExperts || D->k > kTrainMaxTopK || D->k > D->N) return MOE_ERR_UNSUPPORTED;
    if (D->d > 65536 || D->I > 65536) return MOE_ERR_UNSUPPORTED;
    if ((long long)D->T * D->k > kTrainMaxSlots) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

// One region serves every call: the error word, then what the call needs
// (nothing is carried from one call to the next).
struct TrainWs {
    size_t err, counts, part, maps, total;
};

TrainWs train_ws(const moe_dims& D) {
    TrainWs L;
    L.err = 0;
    const size_t o = align_up(sizeof(DevError), kAlign);
    L.counts = L.part = L.maps = o;
    const size_t counts = (size_t)dispatch_spans(D.T, D.k) * (D.N + 1) * 4;
    const size_t part = (size_t)kGateParts * 2 * D.N * 4;
    const size_t maps = (size_t)D.N * 3 * 128;
    size_t most = counts > part ? counts : part;
    if (maps > most) most = maps;
    L.total = align_up(o + most, kAlign);
    return L;
}

moe_status check_ws(const moe_dims* D, void* ws, size_t ws_bytes) {
    if (!ws || !aligned(ws, kAlign)) return MOE_ERR_INVALID_ARG;
    return ws_bytes < train_ws(*D).total ? MOE_ERR_CAPACITY : MOE_OK;
}

size_t elem(const moe_dims* D) { return D->wtype == MOE_DTYPE_BF16 ? 2 : 4; }

// rows of the layer's type: present, aligned to an element, stride >= d
moe_status check_rows(const moe_dims* D, const void* p) {
    return p && aligned(p, elem(D)) ? MOE_OK : MOE_ERR_INVALID_ARG;
}
// indices and float32 values: present, or NULL where that is allowed, and aligned
bool words(std::initializer_list<const void*> needed, std::initializer_list<const void*> optional = {}) {
    for (const void* p : needed)
        if (!p || !aligned(p, 4)) return false;
    for (const void* p : optional)
        if (!aligned(p, 4)) return false;
    return true;
}
moe_status check_stride(const moe_dims* D, int64_t* ld) {
    if (*ld == 0) *ld = D->d;
    return *ld < D->d || *ld > ((int64_t)1 << 40) ? MOE_ERR_INVALID_ARG : MOE_OK;
}

GroupedArgs grouped(const moe_dims* D, TrainForm form, const int32_t* offsets, void* ws) {
    GroupedArgs a = {};
    a.form = form; a.offsets = offsets;
    a.M = D->T * D->k; a.N = D->N; a.d = D->d; a.I = D->I;
    a.bf16 = D->wtype == MOE_DTYPE_BF16;
    a.maps = ws_at<unsigned char>(ws, train_ws(*D).maps);
    a.err = ws_at<DevError>(ws, 0);
    a.sms = device_sms();
    return a;
}

moe_status run_grouped(const GroupedArgs& a, const GroupedArgs* dw, void* stream, const char* what) {
    // the row product of a gradient call, then its weight product, either of them optional (form = kFormNone)
    const bool rows = a.form != kFormNone, rows_tc = rows && grouped_tc_usable(a), dw_tc = dw && grouped_tc_usable(*dw);
    cudaError_t e = cudaSuccess;
    int launches = 0;
    if (rows) {
        e = rows_tc ? launch_grouped_rows_tc(a, dw_tc ? dw : nullptr, S(stream)) : launch_grouped_simt(a, S(stream));
        ++launches;
    }
    if (e == cudaSuccess && dw) {
        e = dw_tc ? launch_grouped_dw_tc(*dw, rows_tc, S(stream)) : launch_grouped_simt(*dw, S(stream));
        launches += dw_tc && !rows_tc ? 2 : 1;
    }
    if (e != cudaSuccess) return cuda_failed(e, what);
    note_launches(launches);
    return MOE_OK;
}

// accumulate: into weight gradients that are there
moe_status check_grads(const moe_dims* D, moe_dtype gtype, bool accumulate) {
    if (gtype != MOE_DTYPE_F32 && gtype != MOE_DTYPE_BF16) return MOE_ERR_UNSUPPORTED;
    if (gtype != MOE_DTYPE_F32 && gtype != D->wtype) return MOE_ERR_UNSUPPORTED;
    return accumulate && gtype != MOE_DTYPE_F32 ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

moe_status check_grad_buffer(moe_dtype gtype, const void* p) {
    return p && aligned(p, gtype == MOE_DTYPE_F32 ? 4 : 2) ? MOE_OK : MOE_ERR_INVALID_ARG;
}

}  // namespace

extern "C" {

moe_status moe_train_workspace_size(const moe_dims* dims, size_t* bytes) {
    TRAIN_TRY(check_dims(dims));
    if (!bytes) return MOE_ERR_INVALID_ARG;
    *bytes = train_ws(*dims).total;
    return MOE_OK;
}

moe_status moe_dispatch_rows(const moe_dims* dims, const void* x, int64_t ldx, const int32_t* expert_idx,
                             int capacity, void* x_perm, int32_t* expert_offsets, int32_t* perm,
                             int32_t* inv_perm, void* ws, size_t ws_bytes, void* stream) {
    TRAIN_TRY(check_dims(dims));
    TRAIN_TRY(check_ws(dims, ws, ws_bytes));
    TRAIN_TRY(check_stride(dims, &ldx));
    if (capacity < 0 || !words({expert_offsets})) return MOE_ERR_INVALID_ARG;
    if (dims->T == 0) {
        TRAIN_CUDA(cudaMemsetAsync(expert_offsets, 0, (size_t)(dims->N + 1) * 4, S(stream)));
        return MOE_OK;
    }
    TRAIN_TRY(check_rows(dims, x));
    TRAIN_TRY(check_rows(dims, x_perm));
    if (!words({expert_idx, perm, inv_perm})) return MOE_ERR_INVALID_ARG;
    DispatchArgs a;
    const int64_t es = (int64_t)elem(dims);
    a.x = x; a.ldx_bytes = ldx * es; a.idx = expert_idx;
    a.T = dims->T; a.N = dims->N; a.k = dims->k; a.capacity = capacity;
    a.row_bytes = dims->d * es; a.x_perm = x_perm;
    a.offsets = expert_offsets; a.perm = perm; a.inv = inv_perm;
    a.counts = ws_at<int32_t>(ws, train_ws(*dims).counts);
    a.sms = device_sms(); a.err = ws_at<DevError>(ws, 0);
    int launches = 0;
    TRAIN_CUDA(launch_dispatch_rows(a, S(stream), &launches));
    note_launches(launches);
    return MOE_OK;
}

moe_status moe_combine_rows(const moe_dims* dims, const void* y_perm, const float* gate,
                            const int32_t* inv_perm, const void* add, int64_t ldadd, void* out,
                            int64_t ldout, void* stream) {
    TRAIN_TRY(check_dims(dims));
    TRAIN_TRY(check_stride(dims, &ldadd));
    TRAIN_TRY(check_stride(dims, &ldout));
    if (dims->T == 0) return MOE_OK;
    TRAIN_TRY(check_rows(dims, y_perm));
    TRAIN_TRY(check_rows(dims, out));
    if (!words({inv_perm}, {gate}) || !aligned(add, elem(dims))) return MOE_ERR_INVALID_ARG;
    CombineRowsArgs a;
    a.y = y_perm; a.gate = gate; a.inv = inv_perm; a.add = add; a.ldadd = ldadd; a.out = out; a.ldout = ldout;
    a.T = dims->T; a.k = dims->k; a.d = dims->d; a.bf16 = dims->wtype == MOE_DTYPE_BF16; a.sms = device_sms();
    TRAIN_CUDA(launch_combine_rows(a, S(stream)));
    note_launches(1);
    return MOE_OK;
}

moe_status moe_dispatch_rows_grad(const moe_dims* dims, const void* dx_perm, const int32_t* inv_perm,
                                  const void* add, int64_t ldadd, void* dx, int64_t lddx, void* stream) {
    return moe_combine_rows(dims, dx_perm, nullptr, inv_perm, add, ldadd, dx, lddx, stream);
}

moe_status moe_combine_rows_grad(const moe_dims* dims, const void* dout, int64_t lddout, const void* y_perm,
                                 const float* gate, const int32_t* inv_perm, void* dy_perm, float* dgate,
                                 void* stream) {
    TRAIN_TRY(check_dims(dims));
    TRAIN_TRY(check_stride(dims, &lddout));
    if (dims->T == 0 || (!dy_perm && !dgate)) return MOE_OK;
    TRAIN_TRY(check_rows(dims, dout));
    if (dgate) TRAIN_TRY(check_rows(dims, y_perm));
    if (!words({inv_perm}, {gate, dgate}) || !aligned(dy_perm, elem(dims))) return MOE_ERR_INVALID_ARG;
    CombineRowsGradArgs a;
    a.dout = dout; a.lddout = lddout; a.y = y_perm; a.gate = gate; a.inv = inv_perm; a.dy = dy_perm;
    a.dgate = dgate; a.T = dims->T; a.k = dims->k; a.d = dims->d; a.bf16 = dims->wtype == MOE_DTYPE_BF16;
    TRAIN_CUDA(launch_combine_rows_grad(a, S(stream)));
    note_launches(1);
    return MOE_OK;
}

moe_status moe_gate_grad(const moe_dims* dims, const float* router_prob, const int32_t* topk_idx,
                         const float* dgate, float balance, float* dlogits, float* balance_loss, void* ws,
                         size_t ws_bytes, void* stream) {
    TRAIN_TRY(check_dims(dims));
    TRAIN_TRY(check_ws(dims, ws, ws_bytes));
    if (!(balance >= 0.f) || std::isinf(balance)) return MOE_ERR_INVALID_ARG;
    if (!words({}, {balance_loss})) return MOE_ERR_INVALID_ARG;
    if (dims->T == 0) {
        if (balance_loss) TRAIN_CUDA(cudaMemsetAsync(balance_loss, 0, 4, S(stream)));
        return MOE_OK;
    }
    if (!words({router_prob, topk_idx, dgate, dlogits})) return MOE_ERR_INVALID_ARG;
    GateGradArgs a;
    a.prob = router_prob; a.idx = topk_idx; a.dgate = dgate;
    a.T = dims->T; a.N = dims->N; a.k = dims->k; a.renorm = dims->renorm_topk != 0; a.balance = balance;
    a.dlogits = dlogits; a.loss = balance_loss; a.part = ws_at<float>(ws, train_ws(*dims).part);
    a.sms = device_sms();
    int launches = 0;
    TRAIN_CUDA(launch_gate_grad(a, S(stream), &launches));
    note_launches(launches);
    return MOE_OK;
}

moe_status moe_experts_up(const moe_dims* dims, const void* x_perm, const int32_t* expert_offsets,
                          const void* w_gate, const void* w_up, void* g, void* u, void* h, void* ws,
                          size_t ws_bytes, void* stream) {
    TRAIN_TRY(check_dims(dims));
    TRAIN_TRY(check_ws(dims, ws, ws_bytes));
    if (dims->T == 0) return MOE_OK;
    if (!words({expert_offsets}) || (g == nullptr) != (u == nullptr)) return MOE_ERR_INVALID_ARG;
    for (const void* p : {x_perm, w_gate, w_up, (const void*)h}) TRAIN_TRY(check_rows(dims, p));
    if (g) for (const void* p : {(const void*)g, (const void*)u}) TRAIN_TRY(check_rows(dims, p));
    GroupedArgs a = grouped(dims, kFormUp, expert_offsets, ws);
    a.a0 = x_perm; a.b0 = w_gate; a.b1 = w_up; a.o0 = g; a.o1 = u; a.o2 = h;
    return run_grouped(a, nullptr, stream, "moe_experts_up");
}

moe_status moe_experts_down(const moe_dims* dims, const void* h, const int32_t* expert_offsets,
                            const void* w_down, void* y_perm, void* ws, size_t ws_bytes, void* stream) {
    TRAIN_TRY(check_dims(dims));
    TRAIN_TRY(check_ws(dims, ws, ws_bytes));
    if (dims->T == 0) return MOE_OK;
    if (!words({expert_offsets})) return MOE_ERR_INVALID_ARG;
    for (const void* p : {h, w_down, (const void*)y_perm}) TRAIN_TRY(check_rows(dims, p));
    GroupedArgs a = grouped(dims, kFormDown, expert_offsets, ws);
    a.a0 = h; a.b0 = w_down; a.o0 = y_perm;
    return run_grouped(a, nullptr, stream, "moe_experts_down");
}

moe_status moe_experts_up_grad(const moe_dims* dims, const void* dg, const void* du, const void* x_perm,
                               const int32_t* expert_offsets, const void* w_gate, const void* w_up,
                               void* dx_perm, void* dw_gate, void* dw_up, moe_dtype gtype, int accumulate,
                               void* ws, size_t ws_bytes, void* stream) {
    TRAIN_TRY(check_dims(dims));
    TRAIN_TRY(check_ws(dims, ws, ws_bytes));
    TRAIN_TRY(check_grads(dims, gtype, accumulate && (dw_gate || dw_up)));
    if (!words({expert_offsets}) || (dw_gate == nullptr) != (dw_up == nullptr)) return MOE_ERR_INVALID_ARG;
    if (dims->T > 0) for (const void* p : {dg, du}) TRAIN_TRY(check_rows(dims, p));
    if (dw_gate) {
        for (const void* p : {(const void*)dw_gate, (const void*)dw_up}) TRAIN_TRY(check_grad_buffer(gtype, p));
        if (dims->T > 0) TRAIN_TRY(check_rows(dims, x_perm));
    }
    if (dx_perm && dims->T > 0)
        for (const void* p : {w_gate, w_up, (const void*)dx_perm}) TRAIN_TRY(check_rows(dims, p));
    GroupedArgs a = grouped(dims, kFormNone, expert_offsets, ws), w = grouped(dims, kFormDw, expert_offsets, ws);
    if (dx_perm && dims->T > 0) {
        a.form = kFormDx;
        a.a0 = dg; a.a1 = du; a.b0 = w_gate; a.b1 = w_up; a.o0 = dx_perm;
    }
    w.a0 = dg; w.a1 = du; w.b0 = x_perm; w.o0 = dw_gate; w.o1 = dw_up;
    w.out_f32 = gtype == MOE_DTYPE_F32; w.accumulate = accumulate != 0;
    const bool want = dw_gate && !(accumulate && dims->T == 0);
    return run_grouped(a, want ? &w : nullptr, stream, "moe_experts_up_grad");
}

moe_status moe_experts_down_grad(const moe_dims* dims, const void* dy_perm, const void* h, const void* g,
                                 const void* u, const int32_t* expert_offsets, const void* w_down, void* dg,
                                 void* du, void* dw_down, moe_dtype gtype, int accumulate, void* ws,
                                 size_t ws_bytes, void* stream) {
    TRAIN_TRY(check_dims(dims));
    TRAIN_TRY(check_ws(dims, ws, ws_bytes));
    TRAIN_TRY(check_grads(dims, gtype, accumulate && dw_down));
    if (!words({expert_offsets}) || (dg == nullptr) != (du == nullptr)) return MOE_ERR_INVALID_ARG;
    if (dims->T > 0) TRAIN_TRY(check_rows(dims, dy_perm));
    if (dw_down) {
        TRAIN_TRY(check_grad_buffer(gtype, dw_down));
        if (dims->T > 0) TRAIN_TRY(check_rows(dims, h));
    }
    if (dg && dims->T > 0)
        for (const void* p : {g, u, w_down, (const void*)dg, (const void*)du}) TRAIN_TRY(check_rows(dims, p));
    GroupedArgs a = grouped(dims, kFormNone, expert_offsets, ws), w = grouped(dims, kFormDw, expert_offsets, ws);
    if (dg && dims->T > 0) {
        a.form = kFormDh;
        a.a0 = dy_perm; a.b0 = w_down; a.g = g; a.u = u; a.o0 = dg; a.o1 = du;
    }
    w.a0 = h; w.b0 = dy_perm; w.o0 = dw_down;
    w.out_f32 = gtype == MOE_DTYPE_F32; w.accumulate = accumulate != 0;
    const bool want = dw_down && !(accumulate && dims->T == 0);
    return run_grouped(a, want ? &w : nullptr, stream, "moe_experts_down_grad");
}

const char* moe_experts_path(const moe_dims* dims) {
    if (check_dims(dims) != MOE_OK) return "unsupported";
    return grouped_tc_shapes(dims->wtype == MOE_DTYPE_BF16, dims->d, dims->I) ? "tc" : "simt";
}

}  // extern "C"
