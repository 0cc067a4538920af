// Rotary positions of queries and keys at given positions, forward and transposed: pairs in
// the rotate-half or the interleaved layout, the whole head or its first rot_dim dims,
// frequencies scaled for contexts longer than the trained one.
//
// The angle of a pair is position x frequency.  At positions of hundreds of thousands an
// fp32 product would be off by tenths of a radian, so the frequencies are held as 64-bit
// fractions of a turn (2^-64 turns per position, computed on the host): the integer product
// wraps around at whole turns by itself and its top 32 bits are the angle to 2^-32 turns.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace nf4ls {

namespace {

struct RopeParams {
  const uint64_t* turns;     // [rot_dim / 2]
  const int32_t* positions;  // [rows]
  const __nv_bfloat16 *q, *k;
  __nv_bfloat16 *qo, *ko;
  int ld_q, ld_k, ld_qo, ld_ko;
  int rows, n_q, n_heads;    // n_heads = query heads + key heads
  int d, rot;
  int heads_per_thread;
  int copy_q, copy_k;        // the dims behind rot are copied (not when in place)
  float mscale, sign;
};

// A thread owns one unit of 32 bytes per head (8 pairs, or 16 dims behind rot_dim) of one
// row, for heads_per_thread heads: the angles are computed once for all of them.  What
// bounds it is memory: every element is read and written once, neighbouring threads hold
// neighbouring units.  16.4k rows of 40 heads of 128: 57 us, 5.9 TB/s, 0.90 of the copy rate
// (one head's loads at a time 64).
constexpr int HB = 4;  // heads whose loads are in flight together
template <bool INTERLEAVED>
__global__ void __launch_bounds__(256) k_rope(const RopeParams p) {
  const int units = p.d / 16;
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  const int row = i / units, u = i - row * units;
  if (row >= p.rows) return;
  const int h0 = blockIdx.y * p.heads_per_thread, h1 = min(p.n_heads, h0 + p.heads_per_thread);
  const bool rotates = u * 16 < p.rot;
  float c[8], s[8];
  if (rotates) {
    const uint64_t pos = (uint64_t)(int64_t)p.positions[row];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int32_t half_turns = (int32_t)((pos * p.turns[u * 8 + j]) >> 32);  // of 2^-31 half turns
      const float a = (float)half_turns * (3.14159265358979f / 2147483648.0f);   // in [-pi, pi]
      // absolute error of the fast sine and cosine there: below 2^-21, far under the bf16
      // rounding of the result
      c[j] = __cosf(a) * p.mscale;
      s[j] = __sinf(a) * (p.mscale * p.sign);
    }
  }
  // offsets of the unit's two 16-byte pieces in a head
  const int o0 = !rotates || INTERLEAVED ? u * 16 : u * 8;
  const int o1 = !rotates || INTERLEAVED ? o0 + 8 : o0 + p.rot / 2;
  // the loads of HB heads, then their stores: heads are disjoint, also in place, which the
  // compiler cannot know
  for (int hb = h0; hb < h1; hb += HB) {
    uint4 v[HB][2];
#pragma unroll
    for (int i = 0; i < HB; ++i) {
      const int h = hb + i;
      const bool is_q = h < p.n_q;
      if (h >= h1 || (!rotates && !(is_q ? p.copy_q : p.copy_k))) continue;
      const __nv_bfloat16* x = is_q ? p.q + (size_t)row * p.ld_q + h * p.d : p.k + (size_t)row * p.ld_k + (h - p.n_q) * p.d;
      v[i][0] = *reinterpret_cast<const uint4*>(x + o0);
      v[i][1] = *reinterpret_cast<const uint4*>(x + o1);
    }
#pragma unroll
    for (int i = 0; i < HB; ++i) {
      const int h = hb + i;
      const bool is_q = h < p.n_q;
      if (h >= h1 || (!rotates && !(is_q ? p.copy_q : p.copy_k))) continue;
      __nv_bfloat16* y = is_q ? p.qo + (size_t)row * p.ld_qo + h * p.d : p.ko + (size_t)row * p.ld_ko + (h - p.n_q) * p.d;
      uint4 v0 = v[i][0], v1 = v[i][1];
      if (rotates) {
        uint32_t w0[4] = {v0.x, v0.y, v0.z, v0.w}, w1[4] = {v1.x, v1.y, v1.z, v1.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (INTERLEAVED) {  // a pair is the two halves of a 32-bit word
            const float a0 = bf16_lo(w0[j]), b0 = bf16_hi(w0[j]), a1 = bf16_lo(w1[j]), b1 = bf16_hi(w1[j]);
            w0[j] = pack_bf16x2(a0 * c[j] - b0 * s[j], b0 * c[j] + a0 * s[j]);
            w1[j] = pack_bf16x2(a1 * c[4 + j] - b1 * s[4 + j], b1 * c[4 + j] + a1 * s[4 + j]);
          } else {  // word j of the two pieces holds pairs 2 j and 2 j + 1
            const float a0 = bf16_lo(w0[j]), b0 = bf16_lo(w1[j]), a1 = bf16_hi(w0[j]), b1 = bf16_hi(w1[j]);
            const float c0 = c[2 * j], s0 = s[2 * j], c1 = c[2 * j + 1], s1 = s[2 * j + 1];
            w0[j] = pack_bf16x2(a0 * c0 - b0 * s0, a1 * c1 - b1 * s1);
            w1[j] = pack_bf16x2(b0 * c0 + a0 * s0, b1 * c1 + a1 * s1);
          }
        }
        v0 = make_uint4(w0[0], w0[1], w0[2], w0[3]);
        v1 = make_uint4(w1[0], w1[1], w1[2], w1[3]);
      }
      *reinterpret_cast<uint4*>(y + o0) = v0;
      *reinterpret_cast<uint4*>(y + o1) = v1;
    }
  }
}

int check_rope(const nf4ls_rope_cfg* c, const char* who) {
  if (!c) return fail(NF4LS_INVALID_ARG, "%s: null config", who);
  if (c->head_dim < 16 || c->head_dim > 512 || c->head_dim % 16)
    return fail(NF4LS_SHAPE, "%s: head_dim %d (a multiple of 16 up to 512)", who, c->head_dim);
  if (c->rot_dim < 16 || c->rot_dim > c->head_dim || c->rot_dim % 16)
    return fail(NF4LS_SHAPE, "%s: rot_dim %d (a multiple of 16, at most head_dim)", who, c->rot_dim);
  if (!(c->theta > 1.0) || !std::isfinite(c->theta)) return fail(NF4LS_INVALID_ARG, "%s: theta must be above 1", who);
  if (c->scaling < NF4LS_ROPE_NONE || c->scaling > NF4LS_ROPE_YARN)
    return fail(NF4LS_INVALID_ARG, "%s: unknown scaling %d", who, c->scaling);
  if (c->scaling != NF4LS_ROPE_NONE && (!(c->factor >= 1.0) || !std::isfinite(c->factor)))
    return fail(NF4LS_INVALID_ARG, "%s: the scaling factor must be at least 1", who);
  if (c->scaling >= NF4LS_ROPE_BANDED) {
    if (!(c->original > 0.0) || !std::isfinite(c->original))
      return fail(NF4LS_INVALID_ARG, "%s: the original context must be positive", who);
    if (!(c->low > 0.0) || !(c->high > c->low) || !std::isfinite(c->high))
      return fail(NF4LS_INVALID_ARG, "%s: turns low %g, high %g (0 < low < high)", who, c->low, c->high);
  }
  return NF4LS_OK;
}

int check_side(const void* x, const void* y, int ld_x, int ld_y, int width, int rows, const char* name, const char* who) {
  if (!x || !y) return fail(NF4LS_INVALID_ARG, "%s: null %s", who, name);
  if (!aligned(x, 16) || !aligned(y, 16)) return fail(NF4LS_ALIGN, "%s: %s must be 16-byte aligned", who, name);
  if (ld_x < width || ld_y < width || ld_x % 8 || ld_y % 8)
    return fail(NF4LS_SHAPE, "%s: row strides %d, %d of %s (multiples of 8, at least %d)", who, ld_x, ld_y, name, width);
  if (x == y && ld_x != ld_y && rows > 1)  // in place is the same rows; another stride is an overlap
    return fail(NF4LS_INVALID_ARG, "%s: %s in place with another row stride", who, name);
  return NF4LS_OK;
}

}  // namespace

}  // namespace nf4ls

using namespace nf4ls;

extern "C" int nf4ls_rope_table(const nf4ls_rope_cfg* c, uint64_t* turns_host, float* mscale) {
  clear_error();
  NF4_TRY(check_rope(c, "nf4ls_rope_table"));
  if (!turns_host || !mscale) return fail(NF4LS_INVALID_ARG, "nf4ls_rope_table: null output");
  const long double two_pi = 6.283185307179586476925286766559005768L;
  const int r = c->rot_dim;
  double low_pair = 0.0, high_pair = 0.0;
  if (c->scaling == NF4LS_ROPE_YARN) {
    // the pair that turns n times over the original context
    auto pair_of = [&](double n) {
      return r * std::log(c->original / (n * (double)two_pi)) / (2.0 * std::log(c->theta));
    };
    low_pair = std::fmax(std::floor(pair_of(c->high)), 0.0);
    high_pair = std::fmin(std::ceil(pair_of(c->low)), r - 1.0);
  }
  for (int i = 0; i < r / 2; ++i) {
    const double inv = std::pow(c->theta, -2.0 * i / r);
    double f = inv;
    if (c->scaling == NF4LS_ROPE_LINEAR) {
      f = inv / c->factor;
    } else if (c->scaling != NF4LS_ROPE_NONE) {
      double keep;  // the share of the unscaled frequency
      if (c->scaling == NF4LS_ROPE_BANDED)
        keep = (c->original * inv / (double)two_pi - c->low) / (c->high - c->low);
      else
        keep = 1.0 - (i - low_pair) / std::fmax(high_pair - low_pair, 0.001);
      keep = std::fmin(std::fmax(keep, 0.0), 1.0);
      f = inv * keep + inv / c->factor * (1.0 - keep);
    }
    turns_host[i] = (uint64_t)((long double)f / two_pi * 18446744073709551616.0L);  // f <= 1: below a turn
  }
  *mscale = c->scaling == NF4LS_ROPE_YARN ? (float)(0.1 * std::log(c->factor) + 1.0) : 1.0f;
  return NF4LS_OK;
}

extern "C" int nf4ls_rope_apply(const nf4ls_rope_cfg* c, const nf4ls_rope_rows* t, nf4ls_stream stream) {
  const char* who = "nf4ls_rope_apply";
  clear_error();
  NF4_TRY(check_rope(c, who));
  if (!t) return fail(NF4LS_INVALID_ARG, "%s: null rows", who);
  if (t->rows < 0 || t->n_q < 0 || t->n_kv < 0 || t->n_q + t->n_kv < 1 || t->n_q > 1024 || t->n_kv > 1024)
    return fail(NF4LS_SHAPE, "%s: rows %d, heads %d + %d", who, t->rows, t->n_q, t->n_kv);
  if (!t->turns_dev || (t->rows > 0 && !t->positions_dev)) return fail(NF4LS_INVALID_ARG, "%s: null table or positions", who);
  if (!aligned(t->turns_dev, 16)) return fail(NF4LS_ALIGN, "%s: the table must be 16-byte aligned", who);
  if (t->n_q) NF4_TRY(check_side(t->q, t->q_out, t->ld_q, t->ld_q_out, t->n_q * c->head_dim, t->rows, "q", who));
  if (t->n_kv) NF4_TRY(check_side(t->k, t->k_out, t->ld_k, t->ld_k_out, t->n_kv * c->head_dim, t->rows, "k", who));
  const int units = c->head_dim / 16;
  if ((int64_t)t->rows * units > 0x7FFFFFFFll - 256) return fail(NF4LS_SHAPE, "%s: too many rows for one launch", who);
  if (t->rows == 0) return NF4LS_OK;
  RopeParams p;
  p.turns = t->turns_dev;
  p.positions = t->positions_dev;
  p.q = static_cast<const __nv_bfloat16*>(t->q);
  p.k = static_cast<const __nv_bfloat16*>(t->k);
  p.qo = static_cast<__nv_bfloat16*>(t->q_out);
  p.ko = static_cast<__nv_bfloat16*>(t->k_out);
  p.ld_q = t->ld_q;
  p.ld_k = t->ld_k;
  p.ld_qo = t->ld_q_out;
  p.ld_ko = t->ld_k_out;
  p.rows = t->rows;
  p.n_q = t->n_q;
  p.n_heads = t->n_q + t->n_kv;
  p.d = c->head_dim;
  p.rot = c->rot_dim;
  p.copy_q = p.q != p.qo;
  p.copy_k = p.k != p.ko;
  p.mscale = t->mscale;
  p.sign = t->inverse ? -1.0f : 1.0f;
  // Four heads a thread, fewer where that does not fill the GPU (148 SMs, half their threads).
  const int64_t threads = (int64_t)t->rows * units, fill = 148 * 1024;
  const int splits = (int)std::min<int64_t>(p.n_heads, std::max<int64_t>((p.n_heads + 3) / 4, fill / threads));
  p.heads_per_thread = (p.n_heads + splits - 1) / splits;
  const dim3 grid((unsigned)((threads + 255) / 256), (unsigned)((p.n_heads + p.heads_per_thread - 1) / p.heads_per_thread));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (c->interleaved)
    k_rope<true><<<grid, 256, 0, s>>>(p);
  else
    k_rope<false><<<grid, 256, 0, s>>>(p);
  note_launch();
  NF4_CUDA_TRY(cudaGetLastError());
  return NF4LS_OK;
}
