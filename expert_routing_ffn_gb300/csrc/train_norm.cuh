// Building blocks of the block's norms (train_norm.cu, train_norm_grad.cu):
// rows as vectors of E values a thread, and sums over a row's threads.
#pragma once

#include <cuda_bf16.h>

#include <initializer_list>
#include <type_traits>

#include "common.cuh"
#include "pairs.cuh"
#include "train.h"

namespace moe {
namespace norm {

constexpr int kMaxGroup = 512, kMaxGroupWarps = kMaxGroup / 32, kBlock = 256;

struct None {};  // the type of a y that is not there

// E consecutive values of type W, as they lie in memory: whole 16 bytes, or one value
template <typename W, int E>
struct Raw {
    static constexpr int kBytes = E * (int)sizeof(W), kN = kBytes / 16;
    static_assert(kBytes % 16 == 0 || E == 1, "");
    uint4 v[(kBytes + 15) / 16];
    __device__ __forceinline__ void load(const void* row, int i) {
        const char* p = static_cast<const char*>(row) + (int64_t)i * kBytes;
        if constexpr (kN > 0) {
#pragma unroll
            for (int j = 0; j < kN; ++j) v[j] = reinterpret_cast<const uint4*>(p)[j];
        } else if constexpr (kBytes == 4) v[0].x = *reinterpret_cast<const uint32_t*>(p);
        else v[0].x = *reinterpret_cast<const uint16_t*>(p);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int j = 0; j < (kBytes + 15) / 16; ++j) v[j] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ uint32_t word(int i) const {
        const uint4& q = v[i / 4];
        return i % 4 == 0 ? q.x : i % 4 == 1 ? q.y : i % 4 == 2 ? q.z : q.w;
    }
    __device__ __forceinline__ Pair pair_of(int i) const {  // values 2 i and 2 i + 1
        if constexpr (sizeof(W) == 4) return pair(__uint_as_float(word(2 * i)), __uint_as_float(word(2 * i + 1)));
        else return pair(bf16_lo(word(i)), bf16_hi(word(i)));
    }
    __device__ __forceinline__ float operator[](int i) const {
        if constexpr (sizeof(W) == 4) return __uint_as_float(word(i));
        else return i % 2 ? bf16_hi(word(i / 2)) : bf16_lo(word(i / 2));
    }
};
template <int E>
struct Raw<None, E> {
    __device__ __forceinline__ void load(const void*, int) {}
    __device__ __forceinline__ void zero() {}
    __device__ __forceinline__ Pair pair_of(int) const { return 0; }
    __device__ __forceinline__ float operator[](int) const { return 0.f; }
};

// values to vector i of a row, each rounded once
template <typename W, int E>
__device__ __forceinline__ void store(void* row, int i, const float (&f)[E]) {
    if constexpr (!std::is_same_v<W, None>) {
        static_assert(E * sizeof(W) % 16 == 0 || E == 1, "");
        char* p = static_cast<char*>(row) + (int64_t)i * E * (int)sizeof(W);
        if constexpr (sizeof(W) == 4) {
            if constexpr (E % 4 == 0) {
#pragma unroll
                for (int j = 0; j < E / 4; ++j)
                    reinterpret_cast<float4*>(p)[j] = make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
            } else *reinterpret_cast<float*>(p) = f[0];
        } else {
            uint32_t w[(E + 1) / 2];
#pragma unroll
            for (int j = 0; j < E; j += 2) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(f[j], j + 1 < E ? f[j + 1 < E ? j + 1 : j] : 0.f);
                w[j / 2] = *reinterpret_cast<const uint32_t*>(&b);
            }
            if constexpr (E == 8) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
            else *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
        }
    }
}

// the same from pairs
template <typename W, int E>
__device__ __forceinline__ void store(void* row, int i, const Pair (&f)[E]) {
    float v[2 * E];
#pragma unroll
    for (int j = 0; j < E; ++j) {
        const float2 h = halves(f[j]);
        v[2 * j] = h.x;
        v[2 * j + 1] = h.y;
    }
    store<W, 2 * E>(row, i, v);
}

// Sums over the threads of a row: a group of G threads (whole warps), beside
// other groups of the block.  Every thread gets them, in an order that does not
// change.  Two buffers: a group's barrier for one sum also frees the buffer of
// the sum before it.
struct Sums {
    float (*buf)[kMaxGroupWarps][4];  // [2][warps][values], the group's own
    int warps, warp, bar, threads, at;
    __device__ __forceinline__ void sync() const { asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(threads) : "memory"); }
    template <int N>
    __device__ __forceinline__ void sum(float (&v)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
        if (warps == 1) return;
        float(*b)[4] = buf[at];
        at ^= 1;
        if ((threadIdx.x & 31) == 0)
            *reinterpret_cast<float4*>(b[warp]) = make_float4(v[0], N > 1 ? v[N > 1] : 0.f, N > 2 ? v[N > 2 ? 2 : 0] : 0.f, 0.f);
        sync();
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = 0.f;
#pragma unroll 4
        for (int w = 0; w < warps; ++w) {
            const float4 q = *reinterpret_cast<const float4*>(b[w]);
            v[0] += q.x;
            if constexpr (N > 1) v[1] += q.y;
            if constexpr (N > 2) v[2] += q.z;
        }
    }
};

// Threads of a row and rows of a block, for rows of n_vec vectors, `chunks` of
// them a thread (0: as many as it takes).
struct Shape {
    int group, rows;
    int threads() const { return group * rows; }
};
inline Shape shape_of(int n_vec, int chunks) {
    Shape s;
    const int per = 32 * (chunks > 0 ? chunks : 4);
    s.group = 32 * ((n_vec + per - 1) / per);
    if (s.group > kMaxGroup) s.group = kMaxGroup;  // with chunks > 0 the caller has seen to it
    s.rows = s.group >= kBlock ? 1 : kBlock / s.group;
    return s;
}

// ---------------------------------------------------------------- rows through shared memory
// Long batches: one block an SM, and a ring of stages for each of its groups,
// each stage a row of every input, brought by bulk copies that the group's first
// thread issues `stages` rows ahead.  A group reads its row into registers, and
// the barrier of the row's first sum tells that thread that the stage is free.
//
// A wait that gives up (mbar_wait's limit) is the group's matter: the thread says so in
// the group's word before that barrier, so behind it the issuing thread knows that
// every thread has seen the row arrive, or fetches no more.  A stage is therefore
// never filled while a copy into it may be on its way, and the copies in flight at
// the end are the last one of each stage, which drain waits for.  The results of that
// row and of the group's rows after it become NaN; the group goes on, because its
// threads meet at barriers.
constexpr int kMaxInputs = 5, kMaxStages = 8, kMaxGroups = 12;
struct RingParams {
    const char* src[kMaxInputs];  // rows, NULL: not there
    int64_t stride[kMaxInputs];   // bytes
    uint32_t bytes[kMaxInputs], at[kMaxInputs];  // of a row; its place in a stage
    uint32_t stage_bytes;
    int stages;
    uint32_t rings, barriers;     // offsets in shared memory (the weights come first)
    int lost;                     // moe_testing_lose_row's row: more is announced than comes (-1: none)
};
constexpr int kBarriers = kMaxStages + 1;  // of a group, and its word that a wait gave up
struct Ring {
    const RingParams& p;
    char* base;
    uint64_t* full;
    int T, first, step;
    uint64_t policy;
    int slot, issue_slot;
    uint32_t phase;
    int ahead;      // the next row to fetch
    bool dead;      // a wait of this thread gave up

    __device__ __forceinline__ Ring(const RingParams& p, char* smem, int group, int T, int first, int step)
        : p(p), base(smem + p.rings + (size_t)group * p.stages * p.stage_bytes),
          full(reinterpret_cast<uint64_t*>(smem + p.barriers) + group * kBarriers), T(T), first(first), step(step),
          policy(l2_evict_first_policy()), slot(0), issue_slot(0), phase(0), ahead(first), dead(false) {}
    __device__ __forceinline__ volatile int& gave_up() const { return *reinterpret_cast<volatile int*>(full + kMaxStages); }
    __device__ __forceinline__ void init() {
        for (int s = 0; s < p.stages; ++s) mbar_init(&full[s], 1);
        gave_up() = 0;
    }
    // One row more, by one thread, behind the barrier of the first sum of the row that had the
    // stage; none once a wait has given up (look: whether one may have).
    __device__ __forceinline__ void issue(bool look = true) {
        if (ahead >= T || (look && gave_up())) return;
        mbar_arrive_expect_tx(&full[issue_slot], p.stage_bytes + (ahead == p.lost ? 16u : 0u));
        char* dst = base + (size_t)issue_slot * p.stage_bytes;
#pragma unroll
        for (int i = 0; i < kMaxInputs; ++i)
            if (p.src[i]) bulk_g2s(dst + p.at[i], p.src[i] + (int64_t)ahead * p.stride[i], p.bytes[i], &full[issue_slot], policy);
        ahead += step;
        if (++issue_slot == p.stages) issue_slot = 0;
    }
    // The current row's stage has arrived: 0, or NaN where this thread gave up on it or on a row before.
    __device__ __forceinline__ float wait() {
        if (!dead && mbar_wait(&full[slot], phase)) return 0.f;
        dead = true;
        gave_up() = 1;
        return __int_as_float(0x7fc00000);
    }
    __device__ __forceinline__ const char* input(int i) const { return base + (size_t)slot * p.stage_bytes + p.at[i]; }
    __device__ __forceinline__ void next() {
        if (++slot == p.stages) { slot = 0; phase ^= 1; }
    }
    // at the end, by the thread that issues: no copy may land once the block is gone
    __device__ __forceinline__ void drain() {
        if (!gave_up()) return;  // every thread has seen every row arrive
        const int issued = (ahead - first) / step;
        for (int s = 0; s < p.stages && s < issued; ++s) (void)mbar_wait(&full[s], (uint32_t)((issued - 1 - s) / p.stages) & 1u);
    }
};

// float32 factors of a row's columns in shared memory, so that a warp's 16-byte
// reads of them do not meet: part h of vector i at 4 (h n_vec + i)
template <int E>
__device__ __forceinline__ void put_factor(float* f, int n_vec, int col, float v) {
    f[4 * (col % E / 4 * n_vec + col / E) + col % 4] = v;
}
template <int E>
__device__ __forceinline__ void get_factors(const float* f, int n_vec, int i, Pair (&v)[E / 2]) {
#pragma unroll
    for (int h = 0; h < E / 4; ++h) {
        const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(f + 4 * (h * n_vec + i));
        v[2 * h] = q.x;
        v[2 * h + 1] = q.y;
    }
}

// Whether a batch takes the ring, and its geometry: `groups` rows at a time of
// `group` threads each, at most `threads` and `most` groups in all; at least
// four rows a group.  More groups of two stages beat fewer of three: norm gradient
// of 16384 tokens, d 1536, eight against six 38 -> 35 us with warm caches, 41 -> 40 on
// inputs that change; of 8192 float32 tokens, d 2048, on inputs that change 70 -> 57,
// block gradient 87 -> 77; nothing measured got slower.
struct RingShape {
    int group, groups, blocks;
    uint32_t smem;
};
inline bool ring_shape(RingParams& r, int T, int n_vec, int chunks, int threads, int most, uint32_t weights, int sms, RingShape& s) {
    constexpr uint32_t kLimit = 232448 - kMaxGroups * 2 * kMaxGroupWarps * 16;  // shared memory of a block, less the sums'
    s.group = 32 * ((n_vec + 32 * chunks - 1) / (32 * chunks));
    r.stage_bytes = 0;
    for (int i = 0; i < kMaxInputs; ++i)
        if (r.src[i]) {
            r.at[i] = r.stage_bytes;
            r.stage_bytes += r.bytes[i];
        }
    const uint32_t bars = kMaxGroups * kBarriers * 8;
    r.rings = (weights + 127) / 128 * 128;
    r.lost = lost_row();
    if (most > kMaxGroups) most = kMaxGroups;
    if (most > threads / s.group) most = threads / s.group;
    for (s.groups = most; s.groups > 0; --s.groups) {
        const int64_t stages = ((int64_t)kLimit - r.rings - bars) / ((int64_t)s.groups * r.stage_bytes);
        r.stages = (int)(stages < kMaxStages ? stages : kMaxStages);
        if (r.stages >= 2) break;
    }
    // by the groups that the threads allow: which outputs are asked for does not choose the kernel
    if (s.groups <= 0 || T < 4LL * sms * most) return false;
    r.barriers = r.rings + (uint32_t)s.groups * r.stages * r.stage_bytes;
    s.smem = r.barriers + bars;
    s.blocks = sms;
    return true;
}

// Values of a vector that every row of these tensors allows: 16 bytes of the
// layer's type, or a single value.  A place: address (NULL = not there) and row
// stride in bytes.
struct Place {
    const void* p;
    int64_t stride;
};
inline int vector_values(bool bf16, int d, std::initializer_list<Place> places) {
    const int wide = bf16 ? 8 : 4;
    if (d % wide) return 1;
    for (const Place& x : places)
        if (x.p && ((reinterpret_cast<uintptr_t>(x.p) | (uintptr_t)x.stride) & 15u)) return 1;
    return wide;
}

// f(E, C) with the values of a vector and the vectors of a thread for rows of d
// values: up to 16 values a thread in registers, else C = 0.
template <int WIDE, typename F>
inline cudaError_t with_chunks(int d, int e, F f) {
    using std::integral_constant;
    const int n = d / e;
    if (e == WIDE) {
        if (n <= kMaxGroup) return f(integral_constant<int, WIDE>(), integral_constant<int, 1>());
        if (n <= 2 * kMaxGroup) return f(integral_constant<int, WIDE>(), integral_constant<int, 2>());
        if constexpr (WIDE == 4)
            if (n <= 4 * kMaxGroup) return f(integral_constant<int, WIDE>(), integral_constant<int, 4>());
        return f(integral_constant<int, WIDE>(), integral_constant<int, 0>());
    }
    if (n <= 8 * kMaxGroup) return f(integral_constant<int, 1>(), integral_constant<int, 8>());
    return f(integral_constant<int, 1>(), integral_constant<int, 0>());
}

}  // namespace norm
}  // namespace moe
