// Pieces that the tcgen05 attention kernels share: the 128 x 128 tile and its staging in
// swizzled shared memory, TMEM stores, the exponential, the product with its A operand in
// TMEM, and the copy into the other CTA of a pair.
#pragma once

#include "common.cuh"

namespace nf4ls {

constexpr int TT = 128;                   // query / key tile
constexpr int TILE_BYTES = TT * 128 * 2;  // 128 rows x 128 dims bf16 = 32 KB
constexpr int ATOM = TILE_BYTES / 2;      // one 64-dim (or 64-key) swizzle atom: 16 KB

// One thread's 32 fp32 values (columns 32 c .. 32 c + 31 of its row r of a 128 x 128 tile),
// times sc, as bf16 into the tile's two 128-byte swizzled 64-column atoms at tile.
__device__ __forceinline__ void stage_row32(uint32_t tile, int r, int c, const uint32_t (&v)[32], float sc) {
  const uint32_t row = tile + (uint32_t)(c >> 1) * (TT * 128) + (uint32_t)r * 128;
#pragma unroll
  for (int q4 = 0; q4 < 4; ++q4) {
    const int chunk = (c & 1) * 4 + q4;  // 16-byte chunk of the 128-byte row
    st_shared_v4(row + ((uint32_t)(chunk ^ (r & 7)) << 4),
                 pack_bf16x2(__uint_as_float(v[8 * q4]) * sc, __uint_as_float(v[8 * q4 + 1]) * sc),
                 pack_bf16x2(__uint_as_float(v[8 * q4 + 2]) * sc, __uint_as_float(v[8 * q4 + 3]) * sc),
                 pack_bf16x2(__uint_as_float(v[8 * q4 + 4]) * sc, __uint_as_float(v[8 * q4 + 5]) * sc),
                 pack_bf16x2(__uint_as_float(v[8 * q4 + 6]) * sc, __uint_as_float(v[8 * q4 + 7]) * sc));
  }
}

__device__ __forceinline__ void stage_row32(uint32_t tile, int r, int c, const float (&v)[32]) {
  uint32_t u[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(v[i]);
  stage_row32(tile, r, c, u, 1.0f);
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
      "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
      "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// 16 lanes x 32 columns of TMEM as the fragments of a warp-level product: registers 4 j + e of
// lane l are row l / 4 (+ 8 for e >= 2), column 8 j + 2 (l % 4) + (e & 1).
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// 16 lanes x 8 columns: registers 2 j + e of lane l are row l / 4 + 8 e, column 4 j + l % 4.
__device__ __forceinline__ void tmem_st_frag(uint32_t taddr, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st_cols(uint32_t taddr, const uint32_t (&r)[32]) { tmem_st32(taddr, r); }
__device__ __forceinline__ void tmem_st_cols(uint32_t taddr, const uint32_t (&r)[16]) { tmem_st16(taddr, r); }

// 2^x by the hardware approximation (ex2.approx, flush-to-zero): its relative error is
// far below the bf16 rounding that every probability gets next.
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// D[tmem] (+)= A[tmem] * B[smem desc]: A of M = 128 lanes x 16 bf16 (8 columns).
__device__ __forceinline__ void umma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// One lane of the (converged) warp: 1 in it, 0 in the others.
__device__ __forceinline__ uint32_t elect_lane() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}

// The products and the commit by one lane, executed by the whole warp under a predicate (el
// from elect_lane, once per kernel).  In a branch of one lane the descriptors have to be
// moved to uniform registers before each product: beside eight busy warps that took 93
// cycles per product of 128 x 128 x 16, more than the 64 the tensor core needs for it; this
// form takes 31.  The operands are the same in every lane.
__device__ __forceinline__ void umma_ss(uint32_t el, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(el)
      : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t el, uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(el)
      : "memory");
}
__device__ __forceinline__ void commit_by(uint32_t el, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "setp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(el)
      : "memory");
}
// The warp's number and a value of shared memory as the same in every lane.
__device__ __forceinline__ int warp_number() { return __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0); }

// mbar_wait (common.cuh) of a whole converged warp: its first lane asks the barrier, under a
// predicate, and every decision is voted, so that no lane ever runs apart from the others.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* err, int kid,
                                          int site) {
  const uint32_t a = smem_u32(bar), first = (threadIdx.x & 31) == 0 ? 1u : 0u;
  unsigned long long t0 = 0;
  for (int i = 0;; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 e, %3, 0;\n\t"
        "setp.ne.b32 p, %3, %3;\n\t"
        "@e mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(a), "r"(parity), "r"(first)
        : "memory");
    if (__any_sync(0xffffffffu, ok)) {
      __syncwarp();  // the vote orders no memory: this hands what the first lane acquired to the others
      return true;
    }
    if ((i & 15) == 15) {
      const unsigned long long t = global_ns();
      if (t0 == 0) t0 = t;
      const bool late = __any_sync(0xffffffffu, t - t0 > kWaitLimitNs);
      if (late && first) {
        *abort_flag = 1;
        record_error(err, 1, kid, site);
      }
      __syncwarp();
      if (__any_sync(0xffffffffu, late || *abort_flag != 0)) return false;
    }
  }
}

// Bulk copy of bytes (a multiple of 16) from this CTA's shared memory to another CTA's of
// the cluster, completing transaction bytes on that CTA's mbarrier (both given by their
// shared::cluster addresses).
__device__ __forceinline__ void bulk_copy_to_peer(uint32_t dst_cluster, uint32_t src, uint32_t bytes,
                                                  uint32_t bar_cluster) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   dst_cluster),
               "r"(src), "r"(bytes), "r"(bar_cluster)
               : "memory");
}

// TMEM column of the A operand of 16-row step ks (0-7) of a block whose first column is
// c0: warp half g packed its 64 rows' values to columns c0 + 64 g .. c0 + 64 g + 31.
__device__ __forceinline__ uint32_t packed_col(uint32_t c0, int ks) { return c0 + (ks >> 2) * 64 + (ks & 3) * 8; }

}  // namespace nf4ls
