// Causal grouped-query attention over a packed batch (forward and gradients) on the
// 5th-generation tensor cores: the sequences lie one behind the other and have any length.
#include <algorithm>
#include <cstring>
#include <type_traits>

#include "attention_tile.cuh"
#include "common.cuh"
#include "internal.h"

namespace nf4ls {

namespace {

struct FwdParams {
  CUtensorMap tq, tk, tv, to;  // [total, cols] bf16, box 64 cols x 128 rows, 128-byte swizzle (to: output)
  const PackTile* tiles;
  __nv_bfloat16* o;
  float* lse;
  int ldo, total, nq, nkv;
  float scale_log2;
  int* err;
};

struct BwdParams {
  CUtensorMap tq, tk, tv, tdo;  // inputs
  CUtensorMap tdq, tdk, tdv;        // the gradients, same boxes (TMA stores)
  const PackTile *query_tiles, *key_tiles;  // most work first
  float* stats;    // [nq, n_tiles, 2, 128]: -lse log2(e) and -delta
  unsigned* next;  // query side: items handed out beyond each block's first
  __nv_bfloat16 *dq, *dk, *dv;
  int ld_dq, ld_dk, ld_dv, total, n_tiles, nq, nkv;
  float scale, scale_log2;
  int* err;
};

struct StatsParams {
  const PackTile* tiles;
  const __nv_bfloat16 *o, *d_o;  // the forward's output and its gradient
  const float* lse;
  float* stats;    // as above
  unsigned* next;  // set to 0
  int ld_o, ld_do, total, n_tiles, nq;
};

// Zeros row r of a tile of NA 64-dim atoms (a whole row is the same under any swizzle).
template <int NA>
__device__ __forceinline__ void zero_row(uint32_t tile, int r) {
#pragma unroll
  for (int j = 0; j < NA; ++j)
#pragma unroll
    for (int c = 0; c < 8; ++c) st_shared_v4(tile + j * ATOM + r * 128 + c * 16, 0u, 0u, 0u, 0u);
}

// Two 32-bit values to an instruction.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  return (uint64_t)__float_as_uint(a) | ((uint64_t)__float_as_uint(b) << 32);
}
__device__ __forceinline__ float lo2(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi2(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t pack2(uint32_t a, uint32_t b) { return (uint64_t)a | ((uint64_t)b << 32); }

template <typename F>
__device__ __forceinline__ void either(bool c, F&& f) {  // two straight-line forms of f, not one with a select per value
  if (c)
    f(std::true_type{});
  else
    f(std::false_type{});
}

// The staged tile at `tile` to rows row .. row + n_rows - 1 and columns col .. col + D - 1 of
// the output: one TMA store per atom where the tile is whole, else 16 bytes a thread, so
// that the rows behind the sequence's end stay as they are.  All `threads` threads call.
template <int D>
__device__ __forceinline__ void store_tile(const CUtensorMap* map, __nv_bfloat16* out, int ld, uint32_t tile, int row,
                                           int col, int n_rows, int tid, int threads) {
  if (n_rows == TT) {
    if (tid == 0) {
      for (int j = 0; j < D / 64; ++j) tma_store_2d(map, tile + j * ATOM, col + 64 * j, row);
      tma_store_drain();
    }
    return;
  }
  for (int i = tid; i < n_rows * (D / 8); i += threads) {
    const int r = i / (D / 8), c = i % (D / 8);
    const uint4 v = ld_shared_v4(tile + (c >> 3) * ATOM + r * 128 + (((c & 7) ^ (r & 7)) << 4));
    *reinterpret_cast<uint4*>(out + (size_t)(row + r) * ld + col + c * 8) = v;
  }
}

// ------------------------------------------------------------------------------ forward
// One block per 128-query tile of one head and sequence, two blocks on an SM, online
// softmax over the key tiles up to the diagonal:
//   S = Q K^T; p = 2^(S scale log2e - m), the reference maximum m of a row moving only when a
//   tile's maximum exceeds it by more than 8, a factor of 2^8; O += P V, P as bf16 over the scores it came
//   from; o = O / sum p.
// Within a tile these depend on one another; the second block's products run meanwhile, and
// the first half of P V under the second half's exponentials.  16.4k rows of 8B heads, the
// tensor core's work 444 us: 647 us alone, 755 back to back under the power cap; 2048 rows:
// 26.7 us.  A tile is 1024 cycles of the tensor
// core and as many of the exponential unit; a block takes 3400 for it, since scores to
// registers, exponentials, P back and a wait at each hand-over follow one another, and two
// blocks keep both units 59% busy.  Built and measured beside it, when it took 740 and 25.8 us
// (long, short): two tiles of one block taking turns under one issuer, 751 and 31 us; blocks that go through a list of
// tiles, 801 and 25.6 us (the list's state spills the scores); a row shared by two warps,
// 854 and 28 us; three of eight exponentials by a cubic on the multiplier instead of the
// exponential unit, 3% slower (13 issue slots for 8 cycles of the unit).  Every lane
// waits on a barrier by itself here: one lane for its warp took 770 us, on the gradients'
// kernels it is the faster form.
// warps 0-3: softmax and epilogue (warp w owns TMEM lanes 32 w .. 32 w + 31, one query
// row per thread, its 128 scores in registers); warp 4: TMA producer; warp 5: MMA issuer
constexpr int F_THREADS = 192, F_PROD = 4, F_MMA = 5;
constexpr int F_OFF_Q = 0, F_OFF_K = TILE_BYTES, F_OFF_V = 2 * TILE_BYTES, F_OFF_BAR = 3 * TILE_BYTES;
constexpr int SMEM_TC = 1024 + F_OFF_BAR + 128;
constexpr float kRescaleLog2 = 8.0f;  // the reference maximum may trail the true one by this much
constexpr float kFarLog2 = 16384.0f;  // a scaled maximum of this size is rounded by up to 2^-10

template <int D>
__global__ void __launch_bounds__(F_THREADS, 2) k_packed_fwd(const __grid_constant__ FwdParams p) {
  constexpr int NA = D / 64, KS = D / 16, TB = NA * ATOM;  // swizzle atoms, k-steps and bytes of a tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + F_OFF_BAR);
  uint64_t* q_full = bars;
  uint64_t* k_full = bars + 1;
  uint64_t* k_empty = bars + 2;
  uint64_t* v_full = bars + 3;
  uint64_t* v_empty = bars + 4;
  uint64_t* s_full = bars + 5;
  uint64_t* p_half = bars + 6;   // 2: P of keys 64 h .. 64 h + 63 is in TMEM (one arrival per softmax warp)
  uint64_t* o_full = bars + 8;   // one phase per key tile: the P V product of that tile is done
  uint64_t* drain = bars + 9;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 10);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = warp_number(), lane = threadIdx.x & 31;
  // heads fastest, then the plan's tiles, most key tiles first
  const int h = blockIdx.x % p.nq;
  const PackTile pt = p.tiles[blockIdx.x / p.nq];
  const int qt = pt.tile, row0 = pt.row0;
  const int n_rows = min(TT, pt.len - qt * TT);  // rows of this tile (keys of the diagonal tile)
  const int kvh = h / (p.nq / p.nkv);
  const int nk = qt + 1;  // key tiles at or before the diagonal

  // by the producer: the MMA warp goes straight to the allocation, which takes a whole,
  // converged warp (beside a branch of its own first lane it faulted)
  if (warp == F_PROD && lane == 0) {
    tma_prefetch_desc(&p.tq);
    tma_prefetch_desc(&p.tk);
    tma_prefetch_desc(&p.tv);
    mbar_init(q_full, 1);
    mbar_init(k_full, 1);
    mbar_init(k_empty, 1);
    mbar_init(v_full, 1);
    mbar_init(v_empty, 1);
    mbar_init(s_full, 1);
    mbar_init(&p_half[0], 4);
    mbar_init(&p_half[1], 4);
    mbar_init(o_full, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == F_MMA) {
    __syncwarp();
    tmem_alloc(tmem_slot, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);  // [0, 128) S then P, [128, 256) O

  if (warp == F_PROD) {
    // ------------------------------------------------------------------ TMA producer
    if (lane == 0) {
      mbar_arrive_expect_tx(q_full, TB);
      for (int j = 0; j < NA; ++j) tma_load_2d(base + F_OFF_Q + j * ATOM, &p.tq, q_full, h * D + 64 * j, row0 + qt * TT);
      int issued_k = 0, issued_v = 0;
      for (int kt = 0; kt < nk; ++kt) {
        if (kt > 0 && !mbar_wait(k_empty, (kt - 1) & 1, abort_flag, p.err, KID_PACKED, 21)) break;
        mbar_arrive_expect_tx(k_full, TB);
        for (int j = 0; j < NA; ++j)
          tma_load_2d(base + F_OFF_K + j * ATOM, &p.tk, k_full, kvh * D + 64 * j, row0 + kt * TT);
        issued_k = kt + 1;
        if (kt > 0 && !mbar_wait(v_empty, (kt - 1) & 1, abort_flag, p.err, KID_PACKED, 22)) break;
        mbar_arrive_expect_tx(v_full, TB);
        for (int j = 0; j < NA; ++j)
          tma_load_2d(base + F_OFF_V + j * ATOM, &p.tv, v_full, kvh * D + 64 * j, row0 + kt * TT);
        issued_v = kt + 1;
      }
      if (*abort_flag) {  // let the copies already issued land before the CTA exits
        mbar_wait_drain(q_full, 0);
        if (issued_k > 0) mbar_wait_drain(k_full, (issued_k - 1) & 1);
        if (issued_v > 0) mbar_wait_drain(v_full, (issued_v - 1) & 1);
      }
    }
  } else if (warp == F_MMA) {
    // ------------------------------------------------------------------ MMA issuer
    constexpr uint32_t idesc_s = idesc_bf16(128, 128, false);  // Q K^T: both K-major
    constexpr uint32_t idesc_o = idesc_bf16(128, D, true);     // P V: V N-major
    const uint32_t sQ = smem_u32(base + F_OFF_Q), sK = smem_u32(base + F_OFF_K), sV = smem_u32(base + F_OFF_V);
    const uint32_t el = elect_lane();
    // every wait is agreed on by the whole warp , so that no lane goes on alone
    bool ok = __all_sync(0xffffffffu, mbar_wait(q_full, 0, abort_flag, p.err, KID_PACKED, 23));
    for (int kt = 0; ok && kt < nk; ++kt) {
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(k_full, kt & 1, abort_flag, p.err, KID_PACKED, 24)))) break;
      tc_fence_after();
      // tcgen05.mma of one thread run in issue order, so S may overwrite the P that the
      // previous tile's P V product reads
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const uint32_t off = (ks >> 2) * ATOM + (ks & 3) * 32;
        umma_ss(el, tmem, sdesc_sw128(sQ + off, 16, 1024), sdesc_sw128(sK + off, 16, 1024), idesc_s, ks ? 1u : 0u);
      }
      commit_by(el, s_full);
      commit_by(el, k_empty);
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(v_full, kt & 1, abort_flag, p.err, KID_PACKED, 26)))) break;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {  // the first half runs under the second half's exponentials
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&p_half[hf], kt & 1, abort_flag, p.err, KID_PACKED, 25)))) break;
        tc_fence_after();
#pragma unroll
        for (int ks = 4 * hf; ks < 4 * hf + 4; ++ks)  // 16 keys per step: P columns 8 ks .., V rows 16 ks ..
          umma_ts(el, tmem + 128, tmem + ks * 8, sdesc_sw128(sV + ks * 2048, ATOM, 1024), idesc_o, (kt | ks) ? 1u : 0u);
      }
      if (!ok) break;
      commit_by(el, v_empty);
      commit_by(el, o_full);
    }
  } else {
    // ------------------------------------------------------------------ softmax + epilogue
    const int r = warp * 32 + lane;  // query row in the tile = TMEM lane
    const uint32_t trow = tmem + ((uint32_t)(warp * 32) << 16);
    const float sl = p.scale_log2;
    float m_run = -INFINITY, ms = -INFINITY, l_run = 0.f;  // the reference maximum, that scaled, the sum
    bool ok = true;
    for (int kt = 0; kt < nk; ++kt) {
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(s_full, kt & 1, abort_flag, p.err, KID_PACKED, 27)))) break;
      tc_fence_after();
      const bool diag = kt == qt;
      // the row of scores, held in registers; masked ones (on the diagonal tile, which is
      // also the only one that the sequence may end in) become -inf whatever they were
      uint32_t v[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(trow + c * 32, v[c]);
      tmem_wait_ld();
      if (diag) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i) v[c][i] = c * 32 + i <= r ? v[c][i] : 0xFF800000u;
      }
      float m4[4];  // independent chains
#pragma unroll
      for (int e = 0; e < 4; ++e) m4[e] = fmaxf(__uint_as_float(v[0][e]), __uint_as_float(v[0][4 + e]));
#pragma unroll
      for (int i = 8; i < 128; i += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          m4[e] = fmaxf(fmaxf(m4[e], __uint_as_float(v[i / 32][i % 32 + e])), __uint_as_float(v[i / 32][i % 32 + 4 + e]));
      float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
      const float mxs = mx * sl, m_old = m_run, ms_old = ms;
      bool up = mxs > ms + kRescaleLog2;
      if (up) m_run = mx, ms = mxs;
      // no score above -inf so far (products beyond fp32): probabilities of 0, not NaN
      float ref = ms == -INFINITY ? 0.0f : ms;
      // (the branch of the far rows costs 1% for 16.4k rows, nothing for 2048)
      if (__builtin_expect(__any_sync(0xffffffffu, (kt > 0 && up) || fabsf(ms) >= kFarLog2), 0)) {  // out of line
        const bool far = fabsf(ms) >= kFarLog2 && m_run > -INFINITY;
        if (far && (mx - m_run) * sl > kRescaleLog2) up = true, m_run = mx, ms = mxs;
        const bool resc = kt > 0 && up;
        if (__any_sync(0xffffffffu, resc)) {
          // the previous tile's P V product must be in O before O is scaled
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(o_full, (kt - 1) & 1, abort_flag, p.err, KID_PACKED, 28)))) break;
          tc_fence_after();
          const float alpha = resc ? fast_exp2(far ? (m_old - m_run) * sl : ms_old - ms) : 1.0f;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {  // 16 columns at a time: the scores hold the registers
            uint32_t o[16];
            tmem_ld16(trow + 128 + c * 16, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st16(trow + 128 + c * 16, o);
          }
          tmem_wait_st();
          l_run *= alpha;
        }
        if (__any_sync(0xffffffffu, far)) {
          // the fused multiply-add below takes the rounded product of the maximum from the exact one of a score:
          // with such scores that would leave more than the exponential's range; the difference first
          const float sub = far ? m_run : 0.0f;
          ref = far ? 0.0f : ref;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i) v[c][i] = __float_as_uint(__uint_as_float(v[c][i]) - sub);
        }
      }
      if (diag && n_rows < TT) {
        // rows of V behind the sequence's end belong to others: zeros, so that a
        // non-finite value there times a probability of 0 stays out of O
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(v_full, kt & 1, abort_flag, p.err, KID_PACKED, 30)))) break;
        if (r >= n_rows) zero_row<NA>(smem_u32(base + F_OFF_V), r);
        fence_proxy_async_smem();
      }
      const uint64_t sl2 = pack2(sl, sl), nm2 = pack2(-ref, -ref);
      uint64_t acc[2] = {0, 0};
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
        for (int c = 2 * hf; c < 2 * hf + 2; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const uint64_t x = fma2(pack2(v[c][2 * j], v[c][2 * j + 1]), sl2, nm2);
            const float e0 = fast_exp2(lo2(x)), e1 = fast_exp2(hi2(x));
            acc[j & 1] = add2(acc[j & 1], pack2(e0, e1));
            pk[j] = pack_bf16x2(e0, e1);
          }
          tmem_st16(trow + c * 16, pk);  // over scores that this warp has read
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_half[hf]);
        __syncwarp();
      }
      acc[0] = add2(acc[0], acc[1]);
      l_run += lo2(acc[0]) + hi2(acc[0]);
    }
    // O / sum through the freed Q tile's shared memory and two TMA stores (coalesced rows);
    // all four warps reach the barrier, the store is issued only when no wait failed
    if (ok && __all_sync(0xffffffffu, mbar_wait(o_full, (nk - 1) & 1, abort_flag, p.err, KID_PACKED, 29))) {
      tc_fence_after();
      const float inv = 1.0f / l_run;
      const uint32_t tile = smem_u32(base + F_OFF_Q);
#pragma unroll
      for (int c = 0; c < D / 32; c += 2) {
        uint32_t v[2][32];
        tmem_ld32(trow + 128 + c * 32, v[0]);
        tmem_ld32(trow + 128 + c * 32 + 32, v[1]);
        tmem_wait_ld();
        stage_row32(tile, r, c, v[0], inv);
        stage_row32(tile, r, c + 1, v[1], inv);
      }
      if (r < n_rows)
        p.lse[(size_t)h * p.total + row0 + qt * TT + r] = (ms + log2f(l_run)) * 0.6931471805599453f;
    }
    fence_proxy_async_smem();
    asm volatile("bar.sync 1, 128;" ::: "memory");
    if (!*abort_flag)
      store_tile<D>(&p.to, p.o, p.ldo, smem_u32(base + F_OFF_Q), row0 + qt * TT, h * D, n_rows, threadIdx.x, 128);
  }

  // On an aborted run the products already issued must finish before TMEM is freed.
  __syncthreads();
  if (warp == F_MMA && *abort_flag) {
    commit_by(elect_lane(), drain);
    mbar_wait_drain(drain, 0);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == F_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// ------------------------------------------------------------------------------ backward
// dQ (per query tile and head) and dK, dV (per key tile and kv head), one 128 x 128 block
// ("item") at a time:
//   query side, item = one key tile:   S = Q K^T, dP = dO V^T; then dQ += dS K;
//   key side, item = one query tile:   S^T = K Q^T, dP^T = V dO^T; then dV += P^T dO and
//     dK += dS^T Q,
// P = 2^(S scale log2e - lse log2e), dS = P (dP - delta).  P and dS are written back as bf16
// (two per 32-bit column) over the scores they came from and are the A operand of their
// products from TMEM.  S, dP and the accumulators fill TMEM, so no second item fits
// beside them; what keeps the tensor core busy is the order of the products within the
// one that is there:
//   query side:  S(i+1) | dQ(i) | dP(i+1)          key side:  dV(i) | S(i+1) | dK(i) | dP(i+1)
// The exponentials of item i + 1 need only S(i+1) and run under the two products behind
// it, and dS(i), which needs dP(i), under the product behind that.  (With columns of its
// own for dS and dO left in shared memory, dP(i+1) need not wait for dQ(i), but dP then
// reads both operands from shared memory: 2% slower.)  The key side hands P and dS over in
// halves, so that the product of the first half runs under the making of the second.  The
// tiles come through two rings: those that the first and the last product of an item read
// (K; Q) live longest and have three stages, the others (V; dO) two.  12.2k rows of 8B heads,
// the tensor core's work of both sides 1258 us: 1555 us alone, 1850 back to back under the
// power cap.
// A small kernel before them forms delta = rowsum(dO * O) and puts it beside lse log2e.
// Accumulation runs in a fixed order (query side: key tiles in order; key side: query heads of
// the group, then query tiles), so results are bit-reproducible.

// warp 0: MMA issuer, warp 1: TMA producer (the scheduler prefers its oldest warp: as the last
// of the block they waited up to 600 cycles for an issue slot), warp 2: stores dQ; warps 4-19:
// elementwise and epilogue (TMEM lane quarter w % 4, columns 32 (w / 4 - 1) .. of a block;
// four on each scheduler hide one another's waits where two did not)
constexpr int B_THREADS = 640, B_MMA = 0, B_PROD = 1, B_STORE = 2, B_FIRST = 4, B_EW = 512;
constexpr int B_OFF_A = 0;                              // Q, dO (query side) or K, V (key side)
constexpr int B_OFF_R3 = 2 * TILE_BYTES;                // 3 stages: K (query side) or Q (key side)
constexpr int B_OFF_R2 = B_OFF_R3 + 3 * TILE_BYTES;     // 2 stages: V (query side) or dO (key side)
constexpr int B_OFF_X = B_OFF_R2 + 2 * TILE_BYTES;      // query side: delta quarters [4][128]; key side: 2 stages
                                                        // x (128 lse + 128 delta floats)
constexpr int B_OFF_BAR = B_OFF_X + 2048;
constexpr int SMEM_BWD = 232448;  // all of it: what lies behind the barriers is slack for the alignment
static_assert(B_OFF_BAR + 256 + 512 <= SMEM_BWD, "shared memory of the packed attention backward");

// TMEM column of the A operand of 16-row step ks (0-7) of a block whose first column is c0:
// column group g packed its 32 rows' values to columns c0 + 32 g .. c0 + 32 g + 15.
__device__ __forceinline__ uint32_t packed32(uint32_t c0, int ks) { return c0 + (ks >> 1) * 32 + (ks & 1) * 8; }

__device__ __forceinline__ void bar_ew() { asm volatile("bar.sync 1, %0;" ::"n"(B_EW) : "memory"); }

// The 1024-byte aligned start of the shared memory; false where the slack does not hold it
// (recorded, the same for every thread and block).
__device__ __forceinline__ bool smem_base(uint8_t* raw, uint8_t** base, int* err) {
  *base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  if (*base - raw + B_OFF_BAR + 256 <= SMEM_BWD) return true;
  if (threadIdx.x == 0) record_error(err, 2, KID_PACKED, 1);
  return false;
}

// STATISTICS of the query rows for both sides: delta = rowsum(dO * O), and lse log2(e) beside
// it, a block per query tile and head.  Bound by memory for long batches (12.2k rows of 8B
// heads 35 us, 70% of the DRAM rate), by the latency of its loads and reductions for short
// ones (2048 rows 10 us, 40%).  With them the two sides need nothing of one another and share
// the GPU; when the query side formed them, the key side stood behind it (2048 rows 70 us, 64 so).
template <int D>
__global__ void __launch_bounds__(256, 5) k_packed_stats(const StatsParams p) {
  constexpr int L = D / 8, STEP = 256 / L, N = TT / STEP;  // lanes of a row; rows at a time; rows of a thread
  next_may_start();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.next = 0;
  const PackTile pt = p.tiles[blockIdx.x];
  const int li = threadIdx.x % L, r0 = threadIdx.x / L, h = blockIdx.y, n_rows = min(TT, pt.len - pt.tile * TT);
  const size_t row0 = (size_t)pt.row0 + pt.tile * TT;
  float* st = p.stats + ((size_t)h * p.n_tiles + pt.index) * (2 * TT);
  uint4 a[N], d[N];  // all loads of a thread are in flight together
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int r = r0 + k * STEP;
    const bool there = r < n_rows;
    a[k] = there ? __ldg(reinterpret_cast<const uint4*>(p.o + (row0 + r) * p.ld_o + h * D) + li) : make_uint4(0u, 0u, 0u, 0u);
    d[k] = there ? __ldg(reinterpret_cast<const uint4*>(p.d_o + (row0 + r) * p.ld_do + h * D) + li) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int r = r0 + k * STEP;
    const uint32_t aw[4] = {a[k].x, a[k].y, a[k].z, a[k].w}, dw[4] = {d[k].x, d[k].y, d[k].z, d[k].w};
    float v = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) v += bf16_lo(aw[j]) * bf16_lo(dw[j]) + bf16_hi(aw[j]) * bf16_hi(dw[j]);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (li == 0 && r < n_rows) {
      st[r] = -p.lse[(size_t)h * p.total + row0 + r] * 1.4426950408889634f;
      st[TT + r] = -v;
    }
  }
}

// QUERY side: dQ of query tiles of one head each ("items").  A block takes an item as it comes
// to the end of its last one, most work first, so that the blocks that start late (behind key
// tiles) do less, and the next one's tiles land and its first products run under the end of
// this one.  (A block for each, whose first products wait 5 k cycles for its tiles, cost 13% of
// both sides' time for 2048 rows, 3% for 12.2k.)
// The Q and dO tiles are copied into TMEM (bf16 pairs, one query row per lane), so that S and
// dP read only K and V from shared memory: 4 KB per 64 tensor-core cycles instead of 8 KB,
// which is all that shared memory delivers, while the next tiles land in it.  The K ring's
// last entry of an item is the place through which its dQ leaves.
template <int D>
__device__ __forceinline__ void query_side(const BwdParams& p, int block, int blocks) {
  constexpr int NA = D / 64, KS = D / 16, TB = NA * ATOM;  // swizzle atoms, k-steps and bytes of a tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base;
  if (!smem_base(smem_raw, &base, p.err)) return;
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + B_OFF_BAR);
  uint64_t* q_full = bars;          // Q, dO
  uint64_t* q_read = bars + 1;      // ... and they have been read (one arrival per elementwise warp)
  uint64_t* qa_full = bars + 2;     // Q and dO are in TMEM (one arrival per elementwise warp)
  uint64_t* k_full = bars + 3;      // 3
  uint64_t* k_empty = bars + 6;     // 3
  uint64_t* v_full = bars + 9;      // 2
  uint64_t* v_empty = bars + 11;    // 2
  uint64_t* s_full = bars + 13;
  uint64_t* s_read = bars + 14;     // S is in registers (one arrival per elementwise warp)
  uint64_t* dp_full = bars + 15;
  uint64_t* ds_full = bars + 16;    // dS is in TMEM (one arrival per elementwise warp)
  uint64_t* acc_full = bars + 17;
  uint64_t* out_full = bars + 18;   // dQ is in its place in the K ring (one arrival per elementwise warp)
  uint64_t* drain = bars + 19;
  uint64_t* item_full = bars + 20;  // 2: this block's next item is known
  uint64_t* item_empty = bars + 22; // 2: every warp has it
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 24);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = warp_number(), lane = threadIdx.x & 31;
  volatile int* items = reinterpret_cast<volatile int*>(base + B_OFF_X);  // 2
  // Item number n of this block, by a whole warp, once for each n: heads fastest, then the
  // plan's tiles, most key tiles first; -1: no more (or a wait failed).
  auto take = [&](int n) -> int {
    if (!warp_wait(&item_full[n & 1], (n >> 1) & 1, abort_flag, p.err, KID_PACKED, 57)) return -1;
    const int item = items[n & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(&item_empty[n & 1]);
    __syncwarp();
    return item;
  };

  // by the producer: the MMA warp goes straight to the allocation, which takes a whole,
  // converged warp (beside a branch of its own first lane it faulted)
  if (warp == B_PROD && lane == 0) {
    tma_prefetch_desc(&p.tq);
    tma_prefetch_desc(&p.tk);
    tma_prefetch_desc(&p.tv);
    tma_prefetch_desc(&p.tdo);
    mbar_init(q_full, 1);
    mbar_init(q_read, B_EW / 32);
    mbar_init(qa_full, B_EW / 32);
    for (int i = 0; i < 3; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
      mbar_init(&item_full[i], 1);
      mbar_init(&item_empty[i], B_EW / 32 + 2);  // and the MMA and the storing warp
    }
    mbar_init(s_full, 1);
    mbar_init(s_read, B_EW / 32);
    mbar_init(dp_full, 1);
    mbar_init(ds_full, B_EW / 32);
    mbar_init(acc_full, 1);
    mbar_init(out_full, B_EW / 32);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == B_MMA) {
    __syncwarp();
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  constexpr uint32_t T_S = 0, T_DP = 128, T_DQ = 256, T_Q = 384, T_DO = 448;  // dS packed over dP
  // c: key tiles (entries of the V ring) before an item; c3: entries of the K ring, which has
  // one more an item, the place for its dQ

  if (warp == B_PROD) {
    if (lane == 0) {
      int n_q = 0, e3 = 0, e2 = 0;  // issued: items' Q and dO, entries of the rings
      // the next entry of the K ring is free: its stage, or -1
      auto ring3 = [&]() -> int {
        const int st = e3 % 3;
        return e3 < 3 || mbar_wait(&k_empty[st], (e3 / 3 - 1) & 1, abort_flag, p.err, KID_PACKED, 41) ? st : -1;
      };
      auto load = [&](const CUtensorMap* map, uint8_t* to, uint64_t* full, int col, int row) {
        mbar_arrive_expect_tx(full, TB);
        for (int j = 0; j < NA; ++j) tma_load_2d(to + j * ATOM, map, full, col + 64 * j, row);
      };
      const int n_items = p.n_tiles * p.nq;
      bool ok = true;
      for (int n = 0;; ++n) {
        if (n >= 2 && !mbar_wait(&item_empty[n & 1], ((n >> 1) - 1) & 1, abort_flag, p.err, KID_PACKED, 58)) break;
        if (n == 1) wait_for_previous();  // the counter
        const unsigned more = n == 0 ? block : blocks + atomicAdd(p.next, 1u);
        const int item = more < (unsigned)n_items ? (int)more : -1;
        items[n & 1] = item;
        mbar_arrive(&item_full[n & 1]);
        if (item < 0) break;
        const int h = item % p.nq, col = h * D, kvc = h / (p.nq / p.nkv) * D;
        const PackTile pt = p.query_tiles[item / p.nq];
        const int row = pt.row0 + pt.tile * TT, n_kt = pt.tile + 1;
        if (n > 0 && !mbar_wait(q_read, (n - 1) & 1, abort_flag, p.err, KID_PACKED, 40)) break;
        mbar_arrive_expect_tx(q_full, 2 * TB);
        for (int j = 0; j < NA; ++j) {
          tma_load_2d(base + B_OFF_A + j * ATOM, &p.tq, q_full, col + 64 * j, row);
          tma_load_2d(base + B_OFF_A + TILE_BYTES + j * ATOM, &p.tdo, q_full, col + 64 * j, row);
        }
        n_q = n + 1;
        int st = 0;
        for (int kt = 0; kt < n_kt; ++kt) {
          st = ring3();
          if (!(ok = st >= 0)) break;
          load(&p.tk, base + B_OFF_R3 + st * TILE_BYTES, &k_full[st], kvc, pt.row0 + kt * TT);
          ++e3;
          const int sv = e2 & 1;
          if (e2 >= 2 && !(ok = mbar_wait(&v_empty[sv], ((e2 >> 1) - 1) & 1, abort_flag, p.err, KID_PACKED, 42))) break;
          load(&p.tv, base + B_OFF_R2 + sv * TILE_BYTES, &v_full[sv], kvc, pt.row0 + kt * TT);
          ++e2;
        }
        if (!ok || (st = ring3()) < 0) break;  // the place for dQ
        mbar_arrive(&k_full[st]);
        ++e3;
      }
      if (*abort_flag) {  // let the copies already issued land before the CTA exits
        if (n_q > 0) mbar_wait_drain(q_full, (n_q - 1) & 1);
        for (int i = max(0, e3 - 3); i < e3; ++i) mbar_wait_drain(&k_full[i % 3], (i / 3) & 1);
        for (int i = max(0, e2 - 2); i < e2; ++i) mbar_wait_drain(&v_full[i & 1], (i >> 1) & 1);
      }
    }
  } else if (warp == B_MMA) {
    constexpr uint32_t idesc_s = idesc_bf16(128, 128, false);  // S, dP: N = 128 keys
    constexpr uint32_t idesc_a = idesc_bf16(128, D, true);     // dQ += dS K: K N-major
    const uint32_t s3 = smem_u32(base + B_OFF_R3), s2 = smem_u32(base + B_OFF_R2), el = elect_lane();
    // every wait is agreed on by the whole warp, so that no lane goes on alone
    auto wait = [&](uint64_t* bar, int parity, int site) -> bool {
      const bool ok = warp_wait(bar, parity & 1, abort_flag, p.err, KID_PACKED, site);
      tc_fence_after();
      return ok;
    };
    auto scores = [&](int e) -> bool {  // S of the K tile in entry e: over the head dim, Q in TMEM
      if (!wait(&k_full[e % 3], e / 3, 44)) return false;
      const uint32_t sK = s3 + (e % 3) * TILE_BYTES;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
        umma_ts(el, tmem + T_S, tmem + T_Q + ks * 8, sdesc_sw128(sK + (ks >> 2) * ATOM + (ks & 3) * 32, 16, 1024),
                idesc_s, ks ? 1u : 0u);
      commit_by(el, s_full);
      return true;
    };
    auto dprobs = [&](int e) -> bool {  // dP of the V tile in entry e
      if (!wait(&v_full[e & 1], e >> 1, 45)) return false;
      const uint32_t sV = s2 + (e & 1) * TILE_BYTES;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
        umma_ts(el, tmem + T_DP, tmem + T_DO + ks * 8, sdesc_sw128(sV + (ks >> 2) * ATOM + (ks & 3) * 32, 16, 1024),
                idesc_s, ks ? 1u : 0u);
      commit_by(el, dp_full);
      commit_by(el, &v_empty[e & 1]);
      return true;
    };
    bool ok = true;
    int c3 = 0, c = 0;
    for (int n = 0, item; ok && (item = take(n)) >= 0; ++n) {
      const int n_kt = p.query_tiles[item / p.nq].tile + 1;
      // (the elementwise warps have then read the last item's S; its dP(last) goes first)
      if (!(ok = wait(qa_full, n, 43) && !*abort_flag)) break;
      if (!(ok = scores(c3) && dprobs(c))) break;
      for (int i = 0; i < n_kt; ++i) {
        if (i + 1 < n_kt && !(ok = wait(s_read, c + i, 46) && scores(c3 + i + 1))) break;
        if (!(ok = wait(ds_full, c + i, 47))) break;
        const int e = c3 + i;
        const uint32_t sK = s3 + (e % 3) * TILE_BYTES;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)  // 16 keys per step
          umma_ts(el, tmem + T_DQ, tmem + packed32(T_DP, ks), sdesc_sw128(sK + ks * 2048, ATOM, 1024), idesc_a,
                  (i | ks) ? 1u : 0u);
        commit_by(el, &k_empty[e % 3]);
        if (i + 1 < n_kt && !(ok = dprobs(c + i + 1))) break;
      }
      if (ok) commit_by(el, acc_full);
      c3 += n_kt + 1;
      c += n_kt;
    }
  } else if (warp == B_STORE) {
    // dQ to memory by TMA stores, while the other warps are at the next item
    bool ok = true;
    int c3 = 0;
    for (int n = 0, item; ok && (item = take(n)) >= 0; ++n) {
      const PackTile pt = p.query_tiles[item / p.nq];
      const int e = c3 + pt.tile + 1;
      if (!(ok = warp_wait(out_full, n & 1, abort_flag, p.err, KID_PACKED, 56))) break;
      // nothing is stored once a wait has failed
      if (!*abort_flag)
        store_tile<D>(&p.tdq, p.dq, p.ld_dq, smem_u32(base + B_OFF_R3 + (e % 3) * TILE_BYTES), pt.row0 + pt.tile * TT,
                      item % p.nq * D, min(TT, pt.len - pt.tile * TT), lane, 32);
      __syncwarp();
      if (lane == 0) mbar_arrive(&k_empty[e % 3]);
      __syncwarp();
      c3 = e + 1;
    }
  } else if (warp >= B_FIRST) {
    // ------------------------------------------------------------------ elementwise + epilogue
    const int wq = warp & 3, g = (warp - B_FIRST) >> 2;
    const int r = wq * 32 + lane;  // query row = TMEM lane
    const uint32_t trow = tmem + ((uint32_t)(wq * 32) << 16);
    // An item begins with Q and dO into TMEM (the MMA warp starts on them): group g < D / 32
    // takes dims 32 g .. of its row, 16-byte chunks c0 .. c0 + 3 of swizzle atom g / 2 of the
    // tiles, to TMEM columns 16 g ..
    const bool has_dims = g < D / 32;
    const int atom = g >> 1, c0 = (g & 1) * 4;
    const uint8_t* q_row = base + B_OFF_A + atom * ATOM + r * 128;
    const uint8_t* dO_row = base + B_OFF_A + TILE_BYTES + atom * ATOM + r * 128;
    bool ok = true;
    auto to_tmem = [&](int n) {
      ok = ok && warp_wait(q_full, n & 1, abort_flag, p.err, KID_PACKED, 50);
      if (ok && has_dims) {
        uint32_t w[16];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint4 x = *reinterpret_cast<const uint4*>((t ? dO_row : q_row) + (((c0 + c) ^ (r & 7)) << 4));
            w[4 * c] = x.x, w[4 * c + 1] = x.y, w[4 * c + 2] = x.z, w[4 * c + 3] = x.w;
          }
          tmem_st16(trow + (t ? T_DO : T_Q) + g * 16, w);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(q_read);
        mbar_arrive(qa_full);  // also on failure: the MMA warp then sees the abort
      }
      __syncwarp();
    };
    // (rows behind the sequence's end have no statistics: their lanes compute values that
    // nothing stores)
    auto stats_of = [&](int item, const PackTile& pt) -> float2 {
      const float* st = p.stats + ((size_t)(item % p.nq) * p.n_tiles + pt.index) * (2 * TT);
      return make_float2(__ldcg(st + r), __ldcg(st + TT + r));  // written while this block may have run
    };
    const uint64_t sl2 = pack2(p.scale_log2, p.scale_log2);
    int item = take(0), c3 = 0, c = 0;
    PackTile pt = {};
    float2 stat = {};
    if (item >= 0) {
      pt = p.query_tiles[item / p.nq];
      to_tmem(0);
      wait_for_previous();  // the statistics
      stat = stats_of(item, pt);
    }
    for (int n = 0; item >= 0; ++n) {
      const int qt = pt.tile, n_kt = qt + 1, n_rows = min(TT, pt.len - qt * TT);
      const uint64_t nlse2 = pack2(stat.x, stat.x), ndl2 = pack2(stat.y, stat.y);
      for (int kt = 0; ok && kt < n_kt; ++kt) {
        const bool diag = kt == qt;
        if (!(ok = warp_wait(s_full, (c + kt) & 1, abort_flag, p.err, KID_PACKED, 52))) break;
        tc_fence_after();
        uint32_t sv[32];
        tmem_ld32(trow + T_S + g * 32, sv);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_read);
        if (diag && n_rows < TT) {
          // rows of K behind the sequence's end: zeros for the product dS K (S is done with them)
          if (r >= n_rows && g == 0)
            zero_row<NA>(smem_u32(base + B_OFF_R3 + ((c3 + kt) % 3) * TILE_BYTES), r);
          fence_proxy_async_smem();
        }
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          const uint64_t x = fma2(pack2(sv[j], sv[j + 1]), sl2, nlse2);
          sv[j] = __float_as_uint(fast_exp2(lo2(x)));
          sv[j + 1] = __float_as_uint(fast_exp2(hi2(x)));
        }
        if (!(ok = warp_wait(dp_full, (c + kt) & 1, abort_flag, p.err, KID_PACKED, 53))) break;
        tc_fence_after();
        uint32_t dp[32];
        tmem_ld32(trow + T_DP + g * 32, dp);
        tmem_wait_ld();
        either(diag, [&](auto masked) {  // keys 32 g .. of the tile
          uint32_t dd[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const uint64_t ds = mul2(pack2(sv[2 * j], sv[2 * j + 1]), add2(pack2(dp[2 * j], dp[2 * j + 1]), ndl2));
            float d0 = lo2(ds), d1 = hi2(ds);
            if (masked) {
              const int c = g * 32 + 2 * j;
              d0 = c <= r ? d0 : 0.f;
              d1 = c + 1 <= r ? d1 : 0.f;
            }
            dd[j] = pack_bf16x2(d0, d1);
          }
          tmem_st16(trow + T_DP + g * 32, dd);  // over dP values this warp has read
        });
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ds_full);
      }
      item = take(n + 1);
      if (item >= 0) {
        pt = p.query_tiles[item / p.nq];
        stat = stats_of(item, pt);
      }
      ok = ok && warp_wait(acc_full, n & 1, abort_flag, p.err, KID_PACKED, 54);
      tc_fence_after();
      if (item >= 0) to_tmem(n + 1);  // the next item's first products run under this one's end
      const int e = c3 + n_kt;
      const uint32_t out = smem_u32(base + B_OFF_R3 + (e % 3) * TILE_BYTES);
      ok = ok && warp_wait(&k_full[e % 3], (e / 3) & 1, abort_flag, p.err, KID_PACKED, 55);
      if (ok && has_dims) {
        uint32_t v[32];
        tmem_ld32(trow + T_DQ + g * 32, v);
        tmem_wait_ld();
        stage_row32(out, r, g, v, p.scale);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(out_full);
      __syncwarp();
      c3 += n_kt + 1;
      c += n_kt;
    }
  }
  __syncthreads();
  if (warp == B_MMA && *abort_flag) {  // products already issued finish before TMEM is freed
    commit_by(elect_lane(), drain);
    mbar_wait_drain(drain, 0);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == B_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// KEY side: dK, dV of one key tile of one kv head, by one CTA or (SPLIT) by a cluster of two
// that split the group's query heads (the first ceil(group / 2) heads and the rest).  Each then
// finishes one of the two tensors: it stages the other tensor's fp32 partial sums in its own
// shared memory and sends them in one bulk copy into the peer's, and adds the peer's to its
// own in the order first CTA + second CTA.
template <int D, bool SPLIT>
__device__ __forceinline__ void key_side(const BwdParams& p, int block) {
  constexpr int NA = D / 64, KS = D / 16, TB = NA * ATOM;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base;
  if (!smem_base(smem_raw, &base, p.err)) return;
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + B_OFF_BAR);
  uint64_t* kv_full = bars;         // K, V
  uint64_t* q_full = bars + 1;      // 3 stages
  uint64_t* q_empty = bars + 4;     // 3
  uint64_t* do_full = bars + 7;     // 2 stages (dO, lse, delta of one (head, query tile))
  uint64_t* do_empty = bars + 9;    // 2
  uint64_t* s_full = bars + 11;
  uint64_t* dp_full = bars + 12;
  uint64_t* p_half = bars + 13;     // 2: P^T of queries 16 h .. of each 32 is in TMEM (one arrival per elementwise warp)
  uint64_t* ds_half = bars + 15;    // 2: dS^T likewise
  uint64_t* acc_full = bars + 17;
  uint64_t* drain = bars + 18;
  uint64_t* peer_full = bars + 19;  // the peer CTA's partial sums of this CTA's tensor have landed
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 20);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = warp_number(), lane = threadIdx.x & 31;
  const int item = SPLIT ? block >> 1 : block, kvh = item % p.nkv;
  const PackTile pt = p.key_tiles[item / p.nkv];
  const int kt = pt.tile, row0 = pt.row0;
  const int n_keys = min(TT, pt.len - kt * TT);
  const uint32_t crank = SPLIT ? cluster_ctarank() : 0;
  const int grp = p.nq / p.nkv, n_qt = (pt.len + TT - 1) / TT;
  const int n_last = pt.len - (n_qt - 1) * TT;  // rows of the sequence's last query tile
  const int hpc = SPLIT ? (grp + 1) / 2 : grp, h_begin = (int)crank * hpc, h_count = min(grp, h_begin + hpc) - h_begin;
  // (head, query tile) items of this CTA
  const int per_head = n_qt - kt, n_st = h_count * per_head;

  // by the producer: the MMA warp goes straight to the allocation, which takes a whole,
  // converged warp (beside a branch of its own first lane it faulted)
  if (warp == B_PROD && lane == 0) {
    tma_prefetch_desc(&p.tq);
    tma_prefetch_desc(&p.tk);
    tma_prefetch_desc(&p.tv);
    tma_prefetch_desc(&p.tdo);
    mbar_init(kv_full, 1);
    for (int i = 0; i < 3; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&do_full[i], 1);
      mbar_init(&do_empty[i], 1);
    }
    mbar_init(s_full, 1);
    mbar_init(dp_full, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&p_half[i], B_EW / 32);
      mbar_init(&ds_half[i], B_EW / 32);
    }
    mbar_init(acc_full, 1);
    mbar_init(drain, 1);
    mbar_init(peer_full, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == B_MMA) {
    __syncwarp();
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  constexpr uint32_t T_S = 0, T_DP = 128, T_DV = 256, T_DK = 384;  // P^T packed over S^T, dS^T over dP^T

  if (warp == B_PROD) {
    if (lane == 0) {
      mbar_arrive_expect_tx(kv_full, 2 * TB);
      for (int j = 0; j < NA; ++j) {
        tma_load_2d(base + B_OFF_A + j * ATOM, &p.tk, kv_full, kvh * D + 64 * j, row0 + kt * TT);
        tma_load_2d(base + B_OFF_A + TILE_BYTES + j * ATOM, &p.tv, kv_full, kvh * D + 64 * j, row0 + kt * TT);
      }
      int issued_q = 0, issued_do = 0;
      for (int i = 0; i < n_st; ++i) {
        const int s3 = i % 3, s2 = i & 1;
        const int h = kvh * grp + h_begin + i / per_head, qt = kt + i % per_head;
        if (i >= 3 && !mbar_wait(&q_empty[s3], (i / 3 - 1) & 1, abort_flag, p.err, KID_PACKED, 31)) break;
        mbar_arrive_expect_tx(&q_full[s3], TB);
        for (int j = 0; j < NA; ++j)
          tma_load_2d(base + B_OFF_R3 + s3 * TILE_BYTES + j * ATOM, &p.tq, &q_full[s3], h * D + 64 * j, row0 + qt * TT);
        issued_q = i + 1;
        if (i >= 2 && !mbar_wait(&do_empty[s2], ((i >> 1) - 1) & 1, abort_flag, p.err, KID_PACKED, 32)) break;
        mbar_arrive_expect_tx(&do_full[s2], TB + 1024);
        for (int j = 0; j < NA; ++j)
          tma_load_2d(base + B_OFF_R2 + s2 * TILE_BYTES + j * ATOM, &p.tdo, &do_full[s2], h * D + 64 * j, row0 + qt * TT);
        if (i == 0) wait_for_previous();  // the statistics
        bulk_load(base + B_OFF_X + s2 * 1024, p.stats + ((size_t)h * p.n_tiles + pt.index - kt + qt) * (2 * TT), 1024,
                  &do_full[s2]);
        issued_do = i + 1;
      }
      if (*abort_flag) {  // let the copies already issued land before the CTA exits
        mbar_wait_drain(kv_full, 0);
        for (int i = max(0, issued_q - 3); i < issued_q; ++i) mbar_wait_drain(&q_full[i % 3], (i / 3) & 1);
        for (int i = max(0, issued_do - 2); i < issued_do; ++i) mbar_wait_drain(&do_full[i & 1], (i >> 1) & 1);
      }
    }
  } else if (warp == B_MMA) {
    constexpr uint32_t idesc_s = idesc_bf16(128, 128, false);  // S^T, dP^T: N = 128 queries
    constexpr uint32_t idesc_a = idesc_bf16(128, D, true);     // dV, dK: dO, Q N-major
    const uint32_t sK = smem_u32(base + B_OFF_A), sV = sK + TILE_BYTES;
    const uint32_t r3 = smem_u32(base + B_OFF_R3), r2 = smem_u32(base + B_OFF_R2);
    auto wait = [&](uint64_t* bar, int parity, int site) -> bool {
      const bool ok = warp_wait(bar, parity & 1, abort_flag, p.err, KID_PACKED, site);
      tc_fence_after();
      return ok;
    };
    const uint32_t el = elect_lane();
    // block = A B^T over the head dim, both from shared memory
    auto block = [&](uint32_t t, uint32_t a, uint32_t b, uint64_t* full) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const uint32_t off = (ks >> 2) * ATOM + (ks & 3) * 32;
        umma_ss(el, tmem + t, sdesc_sw128(a + off, 16, 1024), sdesc_sw128(b + off, 16, 1024), idesc_s, ks ? 1u : 0u);
      }
      commit_by(el, full);
    };
    // acc += (packed block)^T-side product over the 128 queries, 16 per step, each half of the
    // steps as soon as its part of the block is there
    auto accumulate = [&](uint32_t t, uint32_t packed, uint32_t b, int i, uint64_t* half, int site) -> bool {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        if (!wait(&half[hf], i, site)) return false;
#pragma unroll
        for (int ks = hf; ks < 8; ks += 2)
          umma_ts(el, tmem + t, tmem + packed32(packed, ks), sdesc_sw128(b + ks * 2048, ATOM, 1024), idesc_a,
                  (i | ks) ? 1u : 0u);
      }
      return true;
    };
    bool ok = n_st > 0 && wait(kv_full, 0, 33);
    if (ok && (ok = wait(&q_full[0], 0, 34))) block(T_S, sK, r3, s_full);
    if (ok && (ok = wait(&do_full[0], 0, 35))) block(T_DP, sV, r2, dp_full);
    for (int i = 0; ok && i < n_st; ++i) {
      const bool more = i + 1 < n_st;
      if (more && !(ok = wait(&q_full[(i + 1) % 3], (i + 1) / 3, 34))) break;
      if (!(ok = accumulate(T_DV, T_S, r2 + (i & 1) * TILE_BYTES, i, p_half, 36))) break;
      // in issue order: S^T(i+1) overwrites the P^T(i) that dV(i) has read
      if (more) block(T_S, sK, r3 + ((i + 1) % 3) * TILE_BYTES, s_full);
      if (more && !(ok = wait(&do_full[(i + 1) & 1], (i + 1) >> 1, 35))) break;
      if (!(ok = accumulate(T_DK, T_DP, r3 + (i % 3) * TILE_BYTES, i, ds_half, 37))) break;
      commit_by(el, &q_empty[i % 3]);
      commit_by(el, &do_empty[i & 1]);  // behind ds_half: the statistics have been read as well
      if (more) block(T_DP, sV, r2 + ((i + 1) & 1) * TILE_BYTES, dp_full);
    }
    if (ok) commit_by(el, acc_full);
  } else if (warp >= B_FIRST) {
    const int tid = threadIdx.x - B_FIRST * 32;
    const int wq = warp & 3, g = (warp - B_FIRST) >> 2;
    const int r = wq * 32 + lane;  // key row = TMEM lane
    const uint32_t trow = tmem + ((uint32_t)(wq * 32) << 16);
    const uint64_t sl2 = pack2(p.scale_log2, p.scale_log2);
    const int row_f = wq * 32 + (lane >> 2), col0 = g * 32 + 2 * (lane & 3);  // of the first fragment value
    bool ok = true;
    for (int i = 0; i < n_st; ++i) {
      const int qt = kt + i % per_head;
      const bool ragged = qt == n_qt - 1 && n_last < TT, masked = qt == kt || ragged;
      // The block in fragments, for the sake of the statistics, which belong to its columns:
      // a lane sees 8 of the warp's 32 columns, so a warp's loads of them take a quarter of
      // the shared-memory cycles that whole rows per lane take (those, beside the products'
      // own operands, held this pass up to 1850 cycles; it takes about half of that now).
      // Row l / 4 + 8 of lane half hl and column 8 j + 2 (l % 4) of the warp's 32 x 32 part;
      // queries lo <= c < hi are kept: those at or behind the key, in front of the end.
      const float* ld = reinterpret_cast<const float*>(base + B_OFF_X + (i & 1) * 1024) + col0;
      const int diag_row = qt == kt ? row_f - col0 : -TT, hi = ragged ? n_last - col0 : TT;
      if (!(ok = warp_wait(&do_full[i & 1], (i >> 1) & 1, abort_flag, p.err, KID_PACKED, 60)))
        break;
      if (!(ok = warp_wait(s_full, i & 1, abort_flag, p.err, KID_PACKED, 61))) break;
      tc_fence_after();
      uint32_t sv[2][16];
#pragma unroll
      for (int hl = 0; hl < 2; ++hl) tmem_ld_frag(trow + (uint32_t)(hl << 20) + T_S + g * 32, sv[hl]);
      tmem_wait_ld();
      if (ragged) {
        // rows of Q and dO behind the sequence's end: zeros for the products dS^T Q and P^T dO,
        // once S^T and dP^T are done with them
        if (!(ok = warp_wait(dp_full, i & 1, abort_flag, p.err, KID_PACKED, 62))) break;
        if (r >= n_last && g < 2)
          zero_row<NA>(smem_u32(g == 0 ? base + B_OFF_R3 + (i % 3) * TILE_BYTES : base + B_OFF_R2 + (i & 1) * TILE_BYTES), r);
        fence_proxy_async_smem();
      }
      // columns 16 hf .. of this warp's 32 as bf16 pairs over the block (which this warp has
      // read), then on to the product
      auto hand_over = [&](uint32_t t, int hf, const uint32_t (&w)[2][4], uint64_t* half) {
#pragma unroll
        for (int hl = 0; hl < 2; ++hl) tmem_st_frag(trow + (uint32_t)(hl << 20) + t + g * 32 + hf * 8, w[hl]);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&half[hf]);
        __syncwarp();
      };
      either(masked, [&](auto mask) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t pp[2][4];
#pragma unroll
          for (int j = 2 * hf; j < 2 * hf + 2; ++j) {
            const float2 l = *reinterpret_cast<const float2*>(ld + 8 * j);
#pragma unroll
            for (int k = 0; k < 4; ++k) {  // the four pairs of these two columns
              const int hl = k >> 1, e = 4 * j + 2 * (k & 1);
              const uint64_t x = fma2(pack2(sv[hl][e], sv[hl][e + 1]), sl2, pack2(l.x, l.y));
              float e0 = fast_exp2(lo2(x)), e1 = fast_exp2(hi2(x));
              if (mask) {
                const int lo = diag_row + 16 * hl + 8 * (k & 1);
                e0 = 8 * j >= lo && 8 * j < hi ? e0 : 0.f;
                e1 = 8 * j + 1 >= lo && 8 * j + 1 < hi ? e1 : 0.f;
              }
              sv[hl][e] = __float_as_uint(e0);
              sv[hl][e + 1] = __float_as_uint(e1);
              pp[hl][(e / 2) & 3] = pack_bf16x2(e0, e1);
            }
          }
          hand_over(T_S, hf, pp, p_half);
        }
      });
      if (!(ok = warp_wait(dp_full, i & 1, abort_flag, p.err, KID_PACKED, 62))) break;
      tc_fence_after();
      uint32_t dp[2][16];
#pragma unroll
      for (int hl = 0; hl < 2; ++hl) tmem_ld_frag(trow + (uint32_t)(hl << 20) + T_DP + g * 32, dp[hl]);
      tmem_wait_ld();
      either(masked, [&](auto mask) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t dd[2][4];
#pragma unroll
          for (int j = 2 * hf; j < 2 * hf + 2; ++j) {
            const float2 d = *reinterpret_cast<const float2*>(ld + 128 + 8 * j);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int hl = k >> 1, e = 4 * j + 2 * (k & 1);
              const uint64_t y = mul2(pack2(sv[hl][e], sv[hl][e + 1]), add2(pack2(dp[hl][e], dp[hl][e + 1]), pack2(d.x, d.y)));
              float e0 = lo2(y), e1 = hi2(y);
              if (mask) {  // not by the zero of p alone: dP of a masked place may be anything
                const int lo = diag_row + 16 * hl + 8 * (k & 1);
                e0 = 8 * j >= lo && 8 * j < hi ? e0 : 0.f;
                e1 = 8 * j + 1 >= lo && 8 * j + 1 < hi ? e1 : 0.f;
              }
              dd[hl][(e / 2) & 3] = pack_bf16x2(e0, e1);
            }
          }
          hand_over(T_DP, hf, dd, ds_half);
        }
      });
    }
    const bool have = n_st > 0 && ok && warp_wait(acc_full, 0, abort_flag, p.err, KID_PACKED, 63);
    if (have) tc_fence_after();
    const bool has_dims = g < D / 32;  // dims 32 g ..
    const uint32_t tile = smem_u32(base + B_OFF_A);
    if constexpr (!SPLIT) {
      // through the freed K and V tiles' shared memory and TMA stores; dK takes the softmax scale
      if (have && has_dims) {
        uint32_t v[32];
        tmem_ld32(trow + T_DV + g * 32, v);
        tmem_wait_ld();
        stage_row32(tile, r, g, v, 1.0f);
        tmem_ld32(trow + T_DK + g * 32, v);
        tmem_wait_ld();
        stage_row32(tile + TILE_BYTES, r, g, v, p.scale);
      }
      fence_proxy_async_smem();
      bar_ew();
      if (!*abort_flag) {  // the whole tiles' stores by one thread each
        store_tile<D>(&p.tdv, p.dv, p.ld_dv, tile, row0 + kt * TT, kvh * D, n_keys, tid, B_EW);
        store_tile<D>(&p.tdk, p.dk, p.ld_dk, tile + TILE_BYTES, row0 + kt * TT, kvh * D, n_keys, (tid + 32) % B_EW, B_EW);
      }
    } else {
      // The partial sums cross over: the first CTA finishes dV and the second dK, so each sends
      // the other tensor (fp32 rows of D floats, 16-byte chunks swizzled by row) from the start
      // of its freed rings into the space behind it in the peer's.
      constexpr uint32_t PB = 128u * D * 4u;  // one tensor's partial sums
      static_assert(2 * PB <= 5u * TILE_BYTES, "the rings hold both sides of the exchange");
      const uint32_t ring = smem_u32(base + B_OFF_R3);
      const uint32_t t_send = trow + (crank == 0 ? T_DK : T_DV), t_keep = trow + (crank == 0 ? T_DV : T_DK);
      const uint32_t prow = (uint32_t)r * (D * 4);
      if (has_dims) {
        uint32_t v[32];
        if (have) {
          tmem_ld32(t_send + g * 32, v);
          tmem_wait_ld();
        }
#pragma unroll
        for (int q4 = 0; q4 < 8; ++q4) {
          const uint32_t o = ring + prow + ((uint32_t)((g * 8 + q4) ^ (r & 7)) << 4);
          if (have)
            st_shared_v4(o, v[4 * q4], v[4 * q4 + 1], v[4 * q4 + 2], v[4 * q4 + 3]);
          else
            st_shared_v4(o, 0u, 0u, 0u, 0u);
        }
      }
      fence_proxy_async_smem();
      if (tid == 0) mbar_arrive_expect_tx(peer_full, PB);
      bar_ew();
      // both CTAs have finished their products: both rings are free
      cluster_sync_all();
      if (tid == 0) {
        const uint32_t other = crank ^ 1u;
        bulk_copy_to_peer(mapa_shared(ring + PB, other), ring, PB, mapa_shared(smem_u32(peer_full), other));
      }
      (void)warp_wait(peer_full, 0, abort_flag, p.err, KID_PACKED, 64);
      // this CTA's tensor (its sums plus the peer's) through the freed K tile's shared memory
      // and TMA stores; dK takes the softmax scale
      const float sc = crank == 0 ? 1.0f : p.scale;
      if (has_dims) {
        float v[32];
        uint32_t vr[32];
        if (have) {
          tmem_ld32(t_keep + g * 32, vr);
          tmem_wait_ld();
        }
#pragma unroll
        for (int q4 = 0; q4 < 8; ++q4) {
          const uint4 in = ld_shared_v4(ring + PB + prow + ((uint32_t)((g * 8 + q4) ^ (r & 7)) << 4));
          const float iv[4] = {__uint_as_float(in.x), __uint_as_float(in.y), __uint_as_float(in.z), __uint_as_float(in.w)};
#pragma unroll
          for (int e = 0; e < 4; ++e) v[4 * q4 + e] = ((have ? __uint_as_float(vr[4 * q4 + e]) : 0.f) + iv[e]) * sc;
        }
        stage_row32(tile, r, g, v);
      }
      fence_proxy_async_smem();
      bar_ew();
      if (!*abort_flag)
        store_tile<D>(crank == 0 ? &p.tdv : &p.tdk, crank == 0 ? p.dv : p.dk, crank == 0 ? p.ld_dv : p.ld_dk, tile,
                      row0 + kt * TT, kvh * D, n_keys, tid, B_EW);
      // the peer has its copy of this CTA's partial sums before this shared memory goes
      cluster_sync_all();
    }
  }
  if (SPLIT && warp < B_FIRST) {  // the other warps join the two cluster barriers too
    __syncwarp();
    cluster_sync_all();
    cluster_sync_all();
  }
  __syncthreads();
  if (warp == B_MMA && *abort_flag) {  // products already issued finish before TMEM is freed
    commit_by(elect_lane(), drain);
    mbar_wait_drain(drain, 0);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == B_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Both sides in one launch: the key side's blocks, whose items are the longest, then the query
// side's on the SMs that they leave free.  (In launches of their own, the second begun early,
// the same for 2048 rows; 256 rows 3 us more of the GPU's and 2 of the host's time.)
template <int D, bool SPLIT>
__global__ void __launch_bounds__(B_THREADS, 1) k_packed_bwd(const __grid_constant__ BwdParams p) {
  const int n_key = p.n_tiles * p.nkv * (SPLIT ? 2 : 1);
  if ((int)blockIdx.x < n_key)
    key_side<D, SPLIT>(p, blockIdx.x);
  else
    query_side<D>(p, blockIdx.x - n_key, gridDim.x - n_key);
}

template <typename K>
int allow_smem(K kernel, int bytes, int (&configured)[64]) {
  int dev = 0;
  NF4_CUDA_TRY(cudaGetDevice(&dev));
  if (dev >= 64 || !configured[dev]) {
    NF4_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
    if (dev < 64) configured[dev] = 1;
  }
  return NF4LS_OK;
}

template <int D>
int launch_fwd(const FwdParams& p, int n_tiles, cudaStream_t s) {
  static int configured[64] = {0};
  NF4_TRY(allow_smem(k_packed_fwd<D>, SMEM_TC, configured));
  k_packed_fwd<D><<<(unsigned)n_tiles * p.nq, F_THREADS, SMEM_TC, s>>>(p);
  note_launch();
  NF4_CUDA_TRY(cudaGetLastError());
  return NF4LS_OK;
}

// Two CTAs for a key tile, or one?  In tenths of an item of the key side (2.7 k cycles): a CTA
// takes 10 each and 25 of its own, or 40 with the exchange of a pair; the query side, which
// fills the SMs that the key side leaves, 9 a key tile and 11 an item.  What counts is the
// longest CTA, with a little to spare, or the sum over the SMs.  8 kv heads of 4 query heads,
// one CTA against two: 2048 rows in one sequence 117 and 113 us, in four 49 and 57, in eight 38
// and 48; one of 512 rows 31 and 22.
bool split_heads(const nf4ls_pack* pack, int nq, int nkv, int sms) {
  const int group = nq / nkv;
  if (group == 1) return false;
  const int64_t blocks = pack->n_blocks * nq, tiles = (int64_t)pack->n_tiles * nkv;
  auto time = [&](int heads, int64_t ctas, int own) -> int64_t {
    const int64_t longest = 10ll * heads * ((pack->max_len + TT - 1) / TT) + own;
    return std::max<int64_t>(longest * 17 / 16, (10 * blocks + ctas * own + 9 * blocks + 11ll * pack->n_tiles * nq) / sms);
  };
  return time((group + 1) / 2, 2 * tiles, 40) < time(group, tiles, 25);
}

template <int D, bool SPLIT>
int launch_sides(const BwdParams& p, int sms, cudaStream_t s) {
  static int configured[64] = {0};
  NF4_TRY(allow_smem(k_packed_bwd<D, SPLIT>, SMEM_BWD, configured));
  int64_t blocks = (int64_t)p.n_tiles * p.nkv * (SPLIT ? 2 : 1) + std::min<int64_t>((int64_t)p.n_tiles * p.nq, sms);
  if (SPLIT) blocks += blocks & 1;  // a query side's block may have nothing to do
  NF4_CUDA_TRY(launch_kernel(k_packed_bwd<D, SPLIT>, blocks, {B_THREADS, SMEM_BWD, true, SPLIT ? 2 : 1}, s, p));
  note_launch();
  return NF4LS_OK;
}

template <int D>
int launch_bwd(const BwdParams& p, const StatsParams& st, const nf4ls_pack* pack, cudaStream_t s) {
  int dev = 0, sms = 0;
  NF4_CUDA_TRY(cudaGetDevice(&dev));
  NF4_CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  // the statistics; the second launch may begin while they are formed, and waits for them
  NF4_CUDA_TRY(launch_kernel(k_packed_stats<D>, dim3((unsigned)p.n_tiles, (unsigned)p.nq), {256, 0, false, 1}, s, st));
  note_launch();
  return split_heads(pack, p.nq, p.nkv, sms) ? launch_sides<D, true>(p, sms, s) : launch_sides<D, false>(p, sms, s);
}

int check_heads(const nf4ls_pack* pack, const nf4ls_packed_heads* h, const char* who) {
  if (!h) return fail(NF4LS_INVALID_ARG, "%s: null heads", who);
  if (h->head_dim != 64 && h->head_dim != 128) return fail(NF4LS_SHAPE, "%s: head_dim must be 64 or 128", who);
  if (h->n_q < 1 || h->n_kv < 1 || h->n_q % h->n_kv || h->n_q > 1024)
    return fail(NF4LS_SHAPE, "%s: n_q %d, n_kv %d (n_q a multiple of n_kv, at most 1024)", who, h->n_q, h->n_kv);
  if (!(h->scale > 0.0f) || !(h->scale < 1e30f)) return fail(NF4LS_INVALID_ARG, "%s: scale must be positive", who);
  if ((int64_t)pack->n_tiles * h->n_q * 2 > 0x7FFFFFFF) return fail(NF4LS_SHAPE, "%s: too many tiles for one launch", who);
  return NF4LS_OK;
}

int check_rows(const void* p, int ld, int width, const char* name, const char* who) {
  if (!p) return fail(NF4LS_INVALID_ARG, "%s: null %s", who, name);
  if (!aligned(p, 16)) return fail(NF4LS_ALIGN, "%s: %s must be 16-byte aligned", who, name);
  if (ld < width || ld % 8) return fail(NF4LS_SHAPE, "%s: row stride %d of %s (a multiple of 8, at least %d)", who, ld, name, width);
  return NF4LS_OK;
}

int tile_map(CUtensorMap* map, const void* p, int width, int total, int ld) {
  return tma_map_bf16(map, p, (uint64_t)width, (uint64_t)total, (uint64_t)ld * 2, 64, TT);
}

const PackTile* tile_list(const nf4ls_pack* p, uint64_t off) {
  return reinterpret_cast<const PackTile*>(static_cast<const uint8_t*>(p->plan_dev) + off);
}

}  // namespace

}  // namespace nf4ls

using namespace nf4ls;

extern "C" size_t nf4ls_packed_attention_ws_bytes(const nf4ls_pack* pack, const nf4ls_packed_heads* heads) {
  if (!pack || !heads || pack->n_tiles < 0 || heads->n_q < 1) return 0;
  return (size_t)heads->n_q * pack->n_tiles * 2 * TT * sizeof(float) + 256;  // the query side's counter behind them
}

extern "C" int nf4ls_packed_attention_fwd(const nf4ls_pack* pack, const nf4ls_packed_heads* heads,
                                          const nf4ls_packed_attention* t, nf4ls_stream stream) {
  static_assert(SMEM_TC <= 232448, "shared memory of the packed attention");
  const char* who = "nf4ls_packed_attention_fwd";
  clear_error();
  NF4_TRY(check_pack(pack, who));
  NF4_TRY(check_heads(pack, heads, who));
  if (!t) return fail(NF4LS_INVALID_ARG, "%s: null tensors", who);
  const int d = heads->head_dim, qd = heads->n_q * d, kvd = heads->n_kv * d;
  NF4_TRY(check_rows(t->q, t->ld_q, qd, "q", who));
  NF4_TRY(check_rows(t->k, t->ld_k, kvd, "k", who));
  NF4_TRY(check_rows(t->v, t->ld_v, kvd, "v", who));
  NF4_TRY(check_rows(t->o, t->ld_o, qd, "o", who));
  if (!t->lse) return fail(NF4LS_INVALID_ARG, "%s: null lse", who);
  if (!aligned(t->lse, 16)) return fail(NF4LS_ALIGN, "%s: lse must be 16-byte aligned", who);
  if (pack->total == 0) return NF4LS_OK;
  FwdParams p;
  std::memset(&p, 0, sizeof(p));
  NF4_TRY(tile_map(&p.tq, t->q, qd, pack->total, t->ld_q));
  NF4_TRY(tile_map(&p.tk, t->k, kvd, pack->total, t->ld_k));
  NF4_TRY(tile_map(&p.tv, t->v, kvd, pack->total, t->ld_v));
  NF4_TRY(tile_map(&p.to, t->o, qd, pack->total, t->ld_o));
  p.tiles = tile_list(pack, pack->off_query_tiles);
  p.o = static_cast<__nv_bfloat16*>(t->o);
  p.lse = t->lse;
  p.ldo = t->ld_o;
  p.total = pack->total;
  p.nq = heads->n_q;
  p.nkv = heads->n_kv;
  p.scale_log2 = heads->scale * 1.4426950408889634f;
  p.err = device_error_ptr();
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return d == 64 ? launch_fwd<64>(p, pack->n_tiles, s) : launch_fwd<128>(p, pack->n_tiles, s);
}

extern "C" int nf4ls_packed_attention_bwd(const nf4ls_pack* pack, const nf4ls_packed_heads* heads,
                                          const nf4ls_packed_attention* t, void* ws_dev, size_t ws_bytes,
                                          nf4ls_stream stream) {
  const char* who = "nf4ls_packed_attention_bwd";
  clear_error();
  NF4_TRY(check_pack(pack, who));
  NF4_TRY(check_heads(pack, heads, who));
  if (!t) return fail(NF4LS_INVALID_ARG, "%s: null tensors", who);
  const int d = heads->head_dim, qd = heads->n_q * d, kvd = heads->n_kv * d;
  NF4_TRY(check_rows(t->q, t->ld_q, qd, "q", who));
  NF4_TRY(check_rows(t->k, t->ld_k, kvd, "k", who));
  NF4_TRY(check_rows(t->v, t->ld_v, kvd, "v", who));
  NF4_TRY(check_rows(t->o, t->ld_o, qd, "o", who));
  NF4_TRY(check_rows(t->d_o, t->ld_do, qd, "do", who));
  NF4_TRY(check_rows(t->dq, t->ld_dq, qd, "dq", who));
  NF4_TRY(check_rows(t->dk, t->ld_dk, kvd, "dk", who));
  NF4_TRY(check_rows(t->dv, t->ld_dv, kvd, "dv", who));
  if (!t->lse) return fail(NF4LS_INVALID_ARG, "%s: null lse", who);
  if (pack->total == 0) return NF4LS_OK;
  if (!ws_dev || ws_bytes < nf4ls_packed_attention_ws_bytes(pack, heads))
    return fail(NF4LS_INVALID_ARG, "%s: workspace too small", who);
  if (!aligned(ws_dev, 256)) return fail(NF4LS_ALIGN, "%s: the workspace must be 256-byte aligned", who);
  BwdParams p;
  std::memset(&p, 0, sizeof(p));
  NF4_TRY(tile_map(&p.tq, t->q, qd, pack->total, t->ld_q));
  NF4_TRY(tile_map(&p.tk, t->k, kvd, pack->total, t->ld_k));
  NF4_TRY(tile_map(&p.tv, t->v, kvd, pack->total, t->ld_v));
  NF4_TRY(tile_map(&p.tdo, t->d_o, qd, pack->total, t->ld_do));
  NF4_TRY(tile_map(&p.tdq, t->dq, qd, pack->total, t->ld_dq));
  NF4_TRY(tile_map(&p.tdk, t->dk, kvd, pack->total, t->ld_dk));
  NF4_TRY(tile_map(&p.tdv, t->dv, kvd, pack->total, t->ld_dv));
  p.stats = static_cast<float*>(ws_dev);
  p.next = reinterpret_cast<unsigned*>(p.stats + (size_t)heads->n_q * pack->n_tiles * 2 * TT);
  p.dq = static_cast<__nv_bfloat16*>(t->dq);
  p.dk = static_cast<__nv_bfloat16*>(t->dk);
  p.dv = static_cast<__nv_bfloat16*>(t->dv);
  p.ld_dq = t->ld_dq;
  p.ld_dk = t->ld_dk;
  p.ld_dv = t->ld_dv;
  p.total = pack->total;
  p.n_tiles = pack->n_tiles;
  p.nq = heads->n_q;
  p.nkv = heads->n_kv;
  p.scale = heads->scale;
  p.scale_log2 = heads->scale * 1.4426950408889634f;
  p.err = device_error_ptr();
  p.query_tiles = tile_list(pack, pack->off_query_tiles);
  p.key_tiles = tile_list(pack, pack->off_key_tiles);
  const StatsParams st = {p.query_tiles, static_cast<const __nv_bfloat16*>(t->o), static_cast<const __nv_bfloat16*>(t->d_o), t->lse,
                          p.stats, p.next, t->ld_o, t->ld_do, p.total, p.n_tiles, p.nq};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return d == 64 ? launch_bwd<64>(p, st, pack, s) : launch_bwd<128>(p, st, pack, s);
}
