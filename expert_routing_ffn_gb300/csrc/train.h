// Launch interfaces of the training step's kernels (train_*.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/moe_train.h"
#include "common.cuh"
#include "kernels.h"

namespace moe {

// moe_api.cu: records a failed CUDA call for moe_last_error_detail(), and the
// device's SM count
moe_status cuda_failed(cudaError_t e, const char* what);
int device_sms();

constexpr int kTrainMaxExperts = 512;
constexpr int kTrainMaxTopK = 16;
constexpr int kTrainMaxSlots = 1 << 24;

// ---------------------------------------------------------------- token rows
// Batches of up to kDispAlone slots are sorted in one launch, each block
// counting all slots; longer ones have a counting launch first, a block per
// span of whole tokens, about kDispSpan slots.
constexpr int kDispAlone = 1 << 14, kDispSpan = 1 << 12;
inline int dispatch_span_tokens(int T, int k) { return (long long)T * k <= kDispAlone ? (T > 0 ? T : 1) : kDispSpan / k; }
inline int dispatch_spans(int T, int k) {
    const int t = dispatch_span_tokens(T, k);
    return T > 0 ? (T + t - 1) / t : 1;
}

struct DispatchArgs {
    const void* x; int64_t ldx_bytes;
    const int32_t* idx;
    int T, N, k, capacity;
    int64_t row_bytes;
    void* x_perm; int32_t *offsets, *perm, *inv;
    int32_t* counts;  // workspace: spans x (N + 1)
    int sms;
    DevError* err;
};
cudaError_t launch_dispatch_rows(const DispatchArgs& a, cudaStream_t st, int* launches);

struct CombineRowsArgs {
    const void* y; const float* gate; const int32_t* inv;
    const void* add; int64_t ldadd; void* out; int64_t ldout;  // strides in elements
    int T, k; int64_t d;
    bool bf16;
    int sms;
};
cudaError_t launch_combine_rows(const CombineRowsArgs& a, cudaStream_t st);

struct CombineRowsGradArgs {
    const void* dout; int64_t lddout; const void* y; const float* gate; const int32_t* inv;
    void* dy; float* dgate;
    int T, k; int64_t d;
    bool bf16;
};
cudaError_t launch_combine_rows_grad(const CombineRowsGradArgs& a, cudaStream_t st);

// ---------------------------------------------------------------- router
constexpr int kGateParts = 128;  // blocks of the load and probability sums
struct GateGradArgs {
    const float* prob; const int32_t* idx; const float* dgate;
    int T, N, k, renorm; float balance;
    float *dlogits, *loss;
    float* part;  // workspace: kGateParts x 2 x N
    int sms;
};
cudaError_t launch_gate_grad(const GateGradArgs& a, cudaStream_t st, int* launches);

// ---------------------------------------------------------------- the block around the layer
struct NormArgs {
    const void* y; int64_t ldy; bool y_f32;  // NULL: a norm alone (x in residual, its norm in next)
    const void* residual; int64_t ldr;
    const void* gate; int gate_kind;         // moe_block_gate
    const void *w_post, *w_next;             // NULL: zeros
    void* out; int64_t ldo; void* next; int64_t ldn;
    float *rstd_post, *rstd_next;
    int T, d, post;
    float eps, offset, scale;
    bool bf16;
    int sms;
};
cudaError_t launch_block_out(const NormArgs& a, cudaStream_t st);
int lost_row();  // moe_testing_lose_row's

constexpr int kNormMaxParts = 2048;              // column sums of so many row groups
constexpr size_t kNormPartBytes = 12u << 20;     // and in so much of the workspace
// row groups whose column sums (two float32 [d]) the workspace holds
inline int norm_parts(int T, int d) {
    long long n = (long long)(kNormPartBytes / (8 * (size_t)d));
    if (n > kNormMaxParts) n = kNormMaxParts;
    return (int)(n < T ? n : T > 0 ? T : 1);
}
struct NormGradArgs {
    const void* dout; int64_t lddout; const void* dnext; int64_t lddnext;  // either may be NULL
    const void* y; int64_t ldy; bool y_f32;  // NULL: nothing of the branch is asked for
    const void* out; int64_t ldo;            // the next norm's input (with dnext)
    const void* gate; int gate_kind;
    const void *w_post, *w_next;
    const float *rstd_post, *rstd_next;
    void* dresidual; int64_t lddr; void* dy; int64_t lddy;
    void* dgate; void *dw_post, *dw_next;    // NULL: not asked for
    int T, d, post;
    float offset, scale;
    bool bf16, grads_f32, accumulate;
    float* part;                             // workspace: norm_parts x 2 x d
    DevError* err;
    int sms;
};
cudaError_t launch_block_out_grad(const NormGradArgs& a, cudaStream_t st, int* launches);

// ---------------------------------------------------------------- rows in 8 bits
constexpr int kPackBlock = 32;
inline int pack_blocks(int cols) { return (cols + kPackBlock - 1) / kPackBlock; }
cudaError_t launch_pack_rows(int64_t rows, int cols, const void* x, int64_t ldx, bool bf16, int8_t* q, uint8_t* scale,
                             int sms, cudaStream_t st);
cudaError_t launch_unpack_rows(int64_t src_rows, int cols, const int8_t* q, const uint8_t* scale, const int32_t* index,
                               int divisor, int64_t rows, void* out, int64_t ldo, bool bf16, int sms, cudaStream_t st);
struct CombineRowsGradPackedArgs {
    const void* dout; int64_t lddout; const int8_t* q; const uint8_t* scale; const float* gate; const int32_t* inv;
    void* dy; float* dgate;
    int T, k, d;
    bool bf16;
    int sms;
};
cudaError_t launch_combine_rows_grad_packed(const CombineRowsGradPackedArgs& a, cudaStream_t st);

// ---------------------------------------------------------------- grouped products
enum TrainForm {
    kFormUp = 0,    // g, u, h from x
    kFormDown = 1,  // y = h Wd
    kFormDh = 2,    // dg, du from dy (through SwiGLU)
    kFormDx = 3,    // dx = dg Wg + du Wu
    kFormDw = 4,    // dW = a^T b per expert, one or two a
    kFormNone = 5
};
struct GroupedArgs {
    TrainForm form;
    const void *a0, *a1;      // rows: [M, K] (Up: x; Down: h; Dh: dy; Dx: dg, du; Dw: [M, I], one or two)
    const void *b0, *b1;      // weights [N, I, d] (Up, Dx: gate, up; Down, Dh: down); Dw: b0 = rows [M, d]
    const void *g, *u;        // Dh: pre-activations [M, I]
    void *o0, *o1, *o2;       // Up: g, u, h; Down: y; Dh: dg, du (packed: and h); Dx: dx; Dw: dW of a0, a1
    bool packed;              // Up: g, u leave as packed rows, Dh: they come so; their scales
    const uint8_t *gs, *us;   // Dh
    uint8_t *s0, *s1;         // Up
    const int32_t* offsets;   // device [N + 1]
    int M, N, d, I;
    bool bf16, out_f32, accumulate;  // out_f32, accumulate: Dw
    unsigned char* maps;      // workspace: per-expert tensor maps (Dw on the tensor cores)
    DevError* err;
    int sms;
};
bool grouped_tc_shapes(bool bf16, int d, int I);
bool grouped_tc_usable(const GroupedArgs& a);
cudaError_t launch_grouped_simt(const GroupedArgs& a, cudaStream_t st);
// tensor cores: the forms that give rows (dw, or NULL: the weight-gradient
// product that follows, whose tensor maps this launch makes on the side), and
// Dw (one launch, or two without such maps)
cudaError_t launch_grouped_rows_tc(const GroupedArgs& a, const GroupedArgs* dw, cudaStream_t st);
cudaError_t launch_grouped_dw_tc(const GroupedArgs& a, bool have_maps, cudaStream_t st);
// clusters of `size` CTAs of a kernel that can be resident at once
cudaError_t resident_clusters(const void* kernel, int size, int threads, uint32_t smem, int sms, int* clusters);

// A persistent launch of `units` clusters of `size` CTAs behind the previous
// kernel of the stream.
template <typename P>
inline cudaError_t launch_units(void (*kern)(P), const std::remove_const_t<P>& p, int units, int size, int threads,
                                uint32_t smem, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units < 1 ? 1 : units) * (unsigned)size);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)size;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = size > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace moe
