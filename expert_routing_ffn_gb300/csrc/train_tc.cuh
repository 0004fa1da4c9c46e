// Building blocks of the training step's tensor-core products beside those of
// tc_common.cuh: CTA pairs, 3-D tensor loads, tensor stores and reductions,
// and tensor maps changed on the device.
#pragma once

#include "tc_common.cuh"

namespace moe {
namespace train {

// ---------------------------------------------------------------- CTA pairs
// The even CTA of a cluster pair (the leader) issues the MMAs, which read
// both CTAs' shared memory at the same offsets and write each CTA's 128
// accumulator rows into its own tensor memory.
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t leader_address(const void* bar) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(bar)), "r"(cluster_rank() & ~1u));
    return a;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Arrive on another CTA's barrier.  What it tells the other CTA is that tensor
// memory has been read (ordered by the tcgen05 fence before it), so it carries
// no cluster-scope release: that one waited for the thread's stores under way,
// some 3000 cycles a tile in the weight-gradient kernel.
__device__ __forceinline__ void arrive_cluster(uint32_t bar_cl) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar_cl) : "memory");
}
__device__ __forceinline__ bool try_wait_cluster(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n"
        " mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    return ok != 0;
}

template <bool PAIR>
__device__ __forceinline__ bool try_wait(uint64_t* bar, uint32_t parity) {
    return PAIR ? try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity);
}
// The rest of a wait whose first try failed: gives up when another role has
// aborted (honor_abort) or after the clock budget (records MOE_ERR_TIMEOUT).
template <bool PAIR>
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort_flag, DevError* err,
                                       int where, bool honor_abort) {
    const long long t0 = clock64();
    for (uint32_t i = 0;; ++i) {
        if (try_wait<PAIR>(bar, parity)) return true;
        if ((i & 63) == 63) {
            if (honor_abort && *abort_flag) return false;
            if (clock64() - t0 > kTcWaitCycles) {
                set_error(err, MOE_ERR_TIMEOUT, where);
                *abort_flag = 1;
                return false;
            }
        }
    }
}
// Bounded wait; PAIR: cluster-scope acquire (another CTA signals the barrier).
// The thread that issues the MMAs waits once per 64 values of K, some 400
// cycles of MMAs: the common case is one instruction and a branch.
template <bool PAIR>
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, DevError* err,
                                     int where, bool honor_abort = true) {
    if (try_wait<PAIR>(bar, parity)) return true;
    return wait_slow<PAIR>(bar, parity, abort_flag, err, where, honor_abort);
}

// ---------------------------------------------------------------- loads, stores
// Tile loads; bar: the mbarrier's shared::cluster address (the leader's for a
// pair; 3-D loads are a pair's).
template <bool PAIR>
__device__ __forceinline__ void load_2d(uint32_t dst, const void* map, int c0, int c1, uint32_t bar) {
    if constexpr (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(bar) : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(bar) : "memory");
}
__device__ __forceinline__ void load_3d(uint32_t dst, const void* map, int c0, int c1, int c2, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar) : "memory");
}
// The pair's loads with an L2 policy.
__device__ __forceinline__ void load_2d_hint(uint32_t dst, const void* map, int c0, int c1, uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(bar), "l"(policy) : "memory");
}
__device__ __forceinline__ void load_3d_hint(uint32_t dst, const void* map, int c0, int c1, int c2, uint32_t bar,
                                             uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4}], [%5], %6;"
        ::"r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "l"(policy) : "memory");
}
__device__ __forceinline__ uint64_t l2_evict_last_policy() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ void store_2d(const void* map, int c0, int c1, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];"
                 ::"l"(map), "r"(c0), "r"(c1), "r"(src) : "memory");
}
__device__ __forceinline__ void store_3d(const void* map, int c0, int c1, int c2, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];"
                 ::"l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(src) : "memory");
}
// `bytes` (a multiple of 16) of shared memory to 16-byte aligned global memory
__device__ __forceinline__ void store_bulk(void* dst, uint32_t src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}
// global += shared, fp32
__device__ __forceinline__ void add_3d(const void* map, int c0, int c1, int c2, uint32_t src) {
    asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];"
                 ::"l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(src) : "memory");
}
__device__ __forceinline__ void stores_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// at most N committed groups of stores still read their shared memory
template <int N>
__device__ __forceinline__ void stores_read() { asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void stores_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// ---------------------------------------------------------------- MMA
// One lane of a converged warp.  The warp that issues MMAs runs its loop with
// all lanes and picks one for the issue alone: the loop's addresses and
// descriptors are then uniform, and an MMA takes them from uniform registers.
// From a branch of a single lane they had to be moved there one by one, some
// 100 cycles an MMA: 625 cycles per 64 values of K whatever N was, where a
// 256 x 256 tile's MMAs take 512.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
    return r != 0;
}

// A shared-memory matrix descriptor advanced by `bytes` (a multiple of 16):
// the address field is its low 14 bits, and no operand crosses 256 KB.
__device__ __forceinline__ uint64_t desc_at(uint64_t desc, uint32_t bytes) { return desc + (bytes >> 4); }

__device__ __forceinline__ void mma(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n"
        ::"r"(tmem_d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc) : "memory");
}
// arrive on `bar` of both CTAs when the MMAs issued so far are done
__device__ __forceinline__ void commit(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
        ::"r"(smem_u32(bar)), "h"((uint16_t)3) : "memory");
}
// the same, on this CTA's barrier alone
__device__ __forceinline__ void commit_local(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                 ::"r"(smem_u32(bar)) : "memory");
}
// all 512 columns, of both CTAs: by a warp of each
__device__ __forceinline__ void tmem_alloc(uint32_t* where) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(where)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t base) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(base));
}

// 32 consecutive accumulator columns of this thread's tensor-memory lane; the
// values are there after tmem_ld_wait
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
          "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
          "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}

// 16 tensor-memory lanes x 32 columns: four 16 x 8 blocks in the fragment
// layout of an m16n8 accumulator.  Of block i, thread T holds lane T / 4 (v[4i],
// v[4i + 1]) and T / 4 + 8 (v[4i + 2], v[4i + 3]) at columns 8i + 2 (T % 4), + 1.
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Four 8 x 8 matrices of 16-bit values, transposed on the way: lanes 8j .. 8j + 7
// give the addresses of matrix j's columns (16 bytes each).
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};"
                 ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(addr) : "memory");
}
__device__ __forceinline__ void bar_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// the same; whether any thread brought `pred`
__device__ __forceinline__ bool bar_any(int id, int threads, bool pred) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %3, 0;\n"
        " barrier.cta.red.or.pred q, %1, %2, p;\n selp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(r) : "r"(id), "r"(threads), "r"((int)pred) : "memory");
    return r != 0;
}

// ---------------------------------------------------------------- tensor maps changed on the device
// Rows [first, first + rows) of a 2-D map, as a map of its own: its address
// and its row count are replaced in global memory.  A kernel that uses the map
// acquires it first (map_acquire, by the warp that issues the copies).
__device__ __forceinline__ void map_replace(void* map, uint64_t address, uint32_t rows) {
    asm volatile("tensormap.replace.tile.global_address.global.b1024.b64 [%0], %1;" ::"l"(map), "l"(address) : "memory");
    asm volatile("tensormap.replace.tile.global_dim.global.b1024.b32 [%0], 1, %1;" ::"l"(map), "r"(rows) : "memory");
}
__device__ __forceinline__ void map_release() { asm volatile("fence.proxy.tensormap::generic.release.gpu;" ::: "memory"); }
__device__ __forceinline__ void map_prefetch(const void* map) { asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory"); }
__device__ __forceinline__ void map_acquire(const void* map) {
    asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(map) : "memory");
}

// The weight gradients' maps: an expert's rows of a0, a1 and b, made from a
// one-row map of each tensor by one warp (expert_maps), in the workspace.
constexpr int kMapsPerExpert = 3;
struct MapParams {
    CUtensorMap t[kMapsPerExpert];
    const unsigned char* rows[kMapsPerExpert];  // the tensors
    int64_t row_bytes[kMapsPerExpert];
    unsigned char* maps;                        // [N][kMapsPerExpert] of 128 bytes; NULL: none to make
    const int32_t* offsets;
    int M, N;
};
__device__ __forceinline__ void expert_maps(const MapParams& p, int e) {
    const int lane = threadIdx.x & 31;
    const int r0 = min(max(p.offsets[e], 0), p.M), rows = min(max(p.offsets[e + 1], 0), p.M) - r0;
    if (rows <= 0) return;
    for (int m = 0; m < kMapsPerExpert; ++m) {
        unsigned char* out = p.maps + ((size_t)e * kMapsPerExpert + m) * 128;
        reinterpret_cast<uint32_t*>(out)[lane] = reinterpret_cast<const uint32_t*>(&p.t[m])[lane];
        __syncwarp();
        if (lane == 0)
            map_replace(out, reinterpret_cast<uint64_t>(p.rows[m]) + (uint64_t)r0 * (uint64_t)p.row_bytes[m],
                        (uint32_t)rows);
    }
    if (lane == 0) map_release();
}

}  // namespace train

// train_tc_dw.cu: the maps' templates for a weight-gradient product
bool dw_map_params(const struct GroupedArgs& a, train::MapParams& mp);
}  // namespace moe
