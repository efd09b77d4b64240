// mxf8_mma.cuh -- the block-scaled tensor-core instructions (tcgen05
// kind::mxf8f6f4.block_scale), tensor-memory reads, barriers of a CTA pair and
// tensor maps that the MXFP8 products share.
#pragma once

#include "tma.cuh"

namespace mxq {
namespace {

constexpr int kBM = 128, kBK = 128;  // kBK elements = bytes of E4M3
constexpr uint32_t kSfTile = 512;    // one 128 x 4 scale tile
constexpr uint64_t kWaitNs = 1000000000ull;  // one second

enum GemmError : int32_t { kErrNone = 0, kErrFullWait = 1, kErrEmptyWait = 2, kErrAccumWait = 3 };

// Shared-memory matrix descriptor (tcgen05): start address, leading and
// stride byte offsets in 16-byte units, descriptor version 1, layout type.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo,
                                              uint32_t layout) {
  return uint64_t((addr >> 4) & 0x3fffu) | (uint64_t(lbo & 0x3fffu) << 16) |
         (uint64_t(sbo & 0x3fffu) << 32) | (1ull << 46) | (uint64_t(layout) << 61);
}

// K-major operand tile, rows of 128 bytes with the 128-byte swizzle: 8-row
// groups 1024 bytes apart (layout type 2).
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
  return smem_desc(addr, 1, 1024 >> 4, 2);
}

// The 512-byte scale tile seen as 32 rows of 16 bytes, no swizzle.
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr) {
  return smem_desc(addr, 1, 128 >> 4, 0);
}

// Instruction descriptor of kind::mxf8f6f4.block_scale: E4M3 x E4M3, both
// K-major, fp32 accumulator, M = 128, N = BN, E8M0 scales; the scale-factor
// ids pick byte `k` (the scale column of the k-th MMA of a K block) of the
// 32-bit scale columns of A and B.
template <int BN>
__device__ __forceinline__ uint32_t instr_desc(uint32_t k) {
  return (k << 4) | (uint32_t(BN >> 3) << 17) | (1u << 23) | (uint32_t(kBM >> 4) << 24) | (k << 29);
}

// The MMA, the scale copy and the commit for a converged warp: each is
// issued by the one lane that elect.sync picks, inside the same asm block.
// The MMA and the copy take their shared-memory descriptors as 32-bit words
// (low words of A and B, one high word), so the warp only adds offsets to
// precomputed words.
__device__ __forceinline__ void mma_mxf8(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t hi,
                                         uint32_t idesc, uint32_t sfa_tmem, uint32_t sfb_tmem,
                                         uint32_t accumulate) {
  asm volatile(
      "{ .reg .pred p, e; .reg .b64 da, db; elect.sync _|e, 0xffffffff; setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 da, {%1, %3}; mov.b64 db, {%2, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale [%0], da, db, %4, [%6], [%7], p; }"
      ::"r"(d_tmem), "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate), "r"(sfa_tmem),
        "r"(sfb_tmem)
      : "memory");
}

__device__ __forceinline__ void tmem_copy_scales(uint32_t taddr, uint32_t lo, uint32_t hi) {
  asm volatile("{ .reg .pred e; .reg .b64 d; elect.sync _|e, 0xffffffff; mov.b64 d, {%1, %2};\n\t"
               "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], d; }" ::"r"(taddr), "r"(lo), "r"(hi)
               : "memory");
}

__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile(
      "{ .reg .pred e; elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0]; }" ::"r"(bar)
      : "memory");
}

__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// 32 consecutive fp32 accumulator columns of this thread's lane.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
        "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
        "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// As tmem_ld32, without the wait: r is not valid before tmem_ld_wait(r).
__device__ __forceinline__ void tmem_ld32_start(uint32_t taddr, uint32_t (&r)[32]) {
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

// Waits for this thread's tensor-memory loads; r goes through the wait, so
// that nothing reads it before.
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),
                 "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]),
                 "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]),
                 "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// 16 consecutive fp32 accumulator columns of this thread's lane.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void sts128_u32(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

__device__ __forceinline__ uint4 lds128_u32(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ void record_error(int32_t* err, int32_t code) {
  if (err) atomicCAS(err, 0, code);
}

__device__ __forceinline__ uint32_t cluster_ctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// All threads of both CTAs of the cluster.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

// Shared::cluster address of the same shared variable in CTA `rank`.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t local, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
  return r;
}

__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

// As above, where the other CTA relies on what this one has written: ordered
// over the cluster, which takes a microsecond.
__device__ __forceinline__ void mbar_release_remote(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

// TMA load into this CTA's shared memory whose completion is counted on a
// barrier of the pair (given by its shared::cluster address).
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map,
                                                 uint32_t cluster_bar, int32_t x, int32_t y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(cluster_bar), "r"(x), "r"(y)
      : "memory");
}

// The same for a converged warp: issued by the lane that elect.sync picks.
__device__ __forceinline__ void tma_elect_2d_pair(uint32_t dst, const CUtensorMap* map, uint32_t cluster_bar, int32_t x,
                                                  int32_t y) {
  asm volatile(
      "{ .reg .pred e; elect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2]; }"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(cluster_bar), "r"(x), "r"(y)
      : "memory");
}

__device__ __forceinline__ void tma_elect_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y) {
  asm volatile(
      "{ .reg .pred e; elect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2]; }"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}

__device__ __forceinline__ void mbar_elect_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("{ .reg .pred e; elect.sync _|e, 0xffffffff;\n\t"
               "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1; }" ::"r"(bar), "r"(bytes)
               : "memory");
}

// The pair forms of mma_mxf8, tmem_copy_scales and mma_commit, for a
// converged warp: each instruction is issued by the one lane that elect.sync
// picks, inside the same asm block (no branch around it). The commit arrives
// on the barrier at this shared offset in both CTAs of the pair once the
// MMAs issued so far have completed.
__device__ __forceinline__ void mma_mxf8_pair(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo,
                                              uint32_t hi, uint32_t idesc, uint32_t sfa_tmem,
                                              uint32_t sfb_tmem, uint32_t accumulate) {
  asm volatile(
      "{ .reg .pred p, e; .reg .b64 da, db; elect.sync _|e, 0xffffffff; setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 da, {%1, %3}; mov.b64 db, {%2, %3};\n\t"
      "@e tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale [%0], da, db, %4, [%6], [%7], p; }"
      ::"r"(d_tmem), "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate), "r"(sfa_tmem),
        "r"(sfb_tmem)
      : "memory");
}
__device__ __forceinline__ void tmem_copy_scales_pair(uint32_t taddr, uint32_t lo, uint32_t hi) {
  asm volatile("{ .reg .pred e; .reg .b64 d; elect.sync _|e, 0xffffffff; mov.b64 d, {%1, %2};\n\t"
               "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], d; }" ::"r"(taddr), "r"(lo), "r"(hi)
               : "memory");
}
__device__ __forceinline__ void mma_commit_pair(uint32_t bar) {
  asm volatile(
      "{ .reg .pred e; elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1; }"
      ::"r"(bar), "h"(uint16_t(3))
      : "memory");
}

// A K block of the pair for a converged warp, issued by one lane: the scale
// copies (A's tile to sfa, B's one or two, side by side, to sfb, sfb + 4), four
// MMAs of K = 32 and the commit on `bar`. One elect.sync for all.
__device__ __forceinline__ void mma_block_pair(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t hi,
                                               uint32_t idesc, uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t sca_lo,
                                               uint32_t scb_lo, uint32_t sc_hi, uint32_t two, uint32_t accumulate, uint32_t bar) {
  asm volatile(
      "{ .reg .pred e, t, p; .reg .b64 da, db, sc; .reg .b32 al, bl, sl, id, ta, tb;\n\t"
      "elect.sync _|e, 0xffffffff; setp.ne.and.b32 t, %9, 0, e; setp.ne.b32 p, %10, 0;\n\t"
      "mov.b64 sc, {%13, %8};\n\t"
      "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%6], sc;\n\t"
      "add.u32 sl, %13, 32; add.u32 tb, %6, 4; mov.b64 sc, {sl, %8};\n\t"
      "@t tcgen05.cp.cta_group::2.32x128b.warpx4 [tb], sc;\n\t"
      "mov.b64 sc, {%7, %8};\n\t"
      "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%5], sc;\n\t"
      "mov.b64 da, {%1, %3}; mov.b64 db, {%2, %3};\n\t"
      "@e tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale [%0], da, db, %4, [%5], [%6], p;\n\t"
      "setp.eq.b32 p, 0, 0;\n\t"
      "add.u32 al, %1, 2; add.u32 bl, %2, 2; mov.b64 da, {al, %3}; mov.b64 db, {bl, %3};\n\t"
      "or.b32 id, %4, 0x20000010; or.b32 ta, %5, 0x40000000; or.b32 tb, %6, 0x40000000;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale [%0], da, db, id, [ta], [tb], p;\n\t"
      "add.u32 al, %1, 4; add.u32 bl, %2, 4; mov.b64 da, {al, %3}; mov.b64 db, {bl, %3};\n\t"
      "or.b32 id, %4, 0x40000020; or.b32 ta, %5, 0x80000000; or.b32 tb, %6, 0x80000000;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale [%0], da, db, id, [ta], [tb], p;\n\t"
      "add.u32 al, %1, 6; add.u32 bl, %2, 6; mov.b64 da, {al, %3}; mov.b64 db, {bl, %3};\n\t"
      "or.b32 id, %4, 0x60000030; or.b32 ta, %5, 0xc0000000; or.b32 tb, %6, 0xc0000000;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale [%0], da, db, id, [ta], [tb], p;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%11], %12; }"
      ::"r"(d_tmem), "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(sca_lo), "r"(sc_hi),
        "r"(two), "r"(accumulate), "r"(bar), "h"(uint16_t(3)), "r"(scb_lo)
      : "memory");
}

// Instruction descriptor as instr_desc<256> but for the pair's M = 256.
__device__ __forceinline__ uint32_t instr_desc_pair(uint32_t k) {
  return (k << 4) | (uint32_t(256 >> 3) << 17) | (1u << 23) | (uint32_t(256 >> 4) << 24) | (k << 29);
}

// ------------------------------------------------------------------ host

// [rows, K] bytes, row stride K, boxes of box_rows rows x 128 bytes,
// 128-byte swizzle; out-of-range rows and columns read as zero.
bool make_operand_map(CUtensorMap* map, const uint8_t* p, uint64_t rows, uint64_t K,
                      uint32_t box_rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {K, rows};
  const cuuint64_t strides[1] = {K};
  const cuuint32_t box[2] = {uint32_t(kBK), box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(p), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A swizzled scale array seen as rows of 128 bytes; one load takes a 512-byte
// 128 x 4 scale tile (4 rows), no swizzle.
bool make_scale_map(CUtensorMap* map, const uint8_t* p, uint64_t bytes) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {128, bytes / 128};
  const cuuint64_t strides[1] = {128};
  const cuuint32_t box[2] = {128, 4};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(p), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace mxq
