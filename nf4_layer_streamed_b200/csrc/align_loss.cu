// Losses of preference and policy training on token logits, with the gradient of the logits.
//
// Both are functions of the log probability of each row's target token,
//   logp_t = x[target] - max - log(sum exp(x - max)),
// so the gradient of a row of logits is a coefficient times (onehot - softmax):
//   preference: the coefficient is that of the row's sequence, known only after every row of
//     both sequences of the pair: one pass that reads the logits for the statistics, one
//     that reads them again and writes the gradient;
//   policy: the coefficient follows from the row alone: statistics and gradient in one launch.
// What bounds them is memory (rows of up to 128 k logits are read and written once per pass)
// and, where a pass only reads, the exponential unit beside it (76% busy at 128 k).
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace nf4ls {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

// A block per row, as many as an SM's 2048 threads hold.  Short rows are latency (a block's
// loads, reduction and the row's own terms): blocks of 256 threads, eight an SM, against 512
// and four: 8000 rows of 16k logits 91 and 113 us (policy), 4000 rows 33 and 39 (statistics),
// 38 and 42 (gradient); 2048 rows of 49k 38 and 38, 57 and 54.  Rows so long that those in
// work do not stay in L2 from a policy row's first pass to its second: two blocks an SM of 768
// threads that hold 96 KB of their row in shared memory.  1999 rows, four blocks of 512 and
// two of 768: of 65k 98 and 102 us, 74k 110 and 105, 98k 148 and 134, 128k 195 and 175.  A call
// without a gradient takes the same blocks for the sake of the same bits, though the smaller
// ones are faster there (128k 70 and 82 us).
constexpr int kShortRow = 24576, kLongRow = 98304;  // logits

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// (m, s): the maximum of some values and the sum of exp(value - m); s = 0 and m = -inf for
// none.  Values of -inf (masked tokens) add nothing; NaN and +inf make s NaN.
struct Stat {
  float m, s;
};
__device__ __forceinline__ float safe_ref(float m) { return m == -INFINITY ? 0.0f : m; }

// The difference to the maximum is taken before the scaling by log2(e): a row whose values
// are all the type's lowest would overflow the other way round.  The exponential unit's
// values are too small by 5e-8 of themselves on average, which a mean over rows keeps: sums
// are rescaled by expf instead (on average within 1e-8), and only once behind the loop.
__device__ __forceinline__ void add8(Stat& st, const uint4& u) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  float x[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = bf16_lo(w[k]);
    x[2 * k + 1] = bf16_hi(w[k]);
  }
  const float cm = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
  if (cm > st.m) {
    st.s *= expf(st.m - cm);
    st.m = cm;
  }
  const float ref = safe_ref(st.m);
  float e[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) e[k] = exp2_fast((x[k] - ref) * kLog2e);
  st.s += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
}
__device__ __forceinline__ void add1(Stat& st, float x) {
  if (x > st.m) {
    st.s *= expf(st.m - x);
    st.m = x;
  }
  st.s += exp2_fast((x - safe_ref(st.m)) * kLog2e);
}

// A row of V bf16 values: `head` of them before the first 16-byte boundary, n16 pieces of
// eight, then a tail.
struct RowSplit {
  int head, n16, tail0;
  __device__ RowSplit(const __nv_bfloat16* row, int V) {
    head = min(V, (int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / 2);
    n16 = (V - head) / 8;
    tail0 = head + n16 * 8;
  }
};

// Statistics of a row by the whole block (fixed order: reruns give the same bits).  The
// threads' sums are short and their rounding errors average out; those of the last, sequential
// one would be most of a row's error (7e-8): it is taken in 64 bits.
struct RowStat {
  float m;
  double s;
};
template <int T>
__device__ __forceinline__ RowStat block_stats(const __nv_bfloat16* row, int V, uint4* keep = nullptr,
                                               int n_keep = 0) {
  __shared__ float red_m[T / 32], red_s[T / 32];
  const int t = threadIdx.x;
  const RowSplit sp(row, V);
  Stat st = {-INFINITY, 0.0f};
  if (t < sp.head) add1(st, __bfloat162float(row[t]));
  const uint4* v = reinterpret_cast<const uint4*>(row + sp.head);
  int j = t;
  for (; j + 3 * T < sp.n16; j += 4 * T) {
    const uint4 a = v[j], b = v[j + T], c = v[j + 2 * T], d = v[j + 3 * T];
    if (j < n_keep) {
      keep[j] = a;
      keep[j + T] = b;
      keep[j + 2 * T] = c;
      keep[j + 3 * T] = d;
    }
    add8(st, a);
    add8(st, b);
    add8(st, c);
    add8(st, d);
  }
  for (; j < sp.n16; j += T) add8(st, v[j]);
  if (sp.tail0 + t < V) add1(st, __bfloat162float(row[sp.tail0 + t]));
  // the row's maximum first, so that a thread's sum is scaled to it once
  float m = st.m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((t & 31) == 0) red_m[t >> 5] = m;
  __syncthreads();
  m = red_m[0];
#pragma unroll
  for (int i = 1; i < T / 32; ++i) m = fmaxf(m, red_m[i]);
  float s = st.s * expf(st.m - safe_ref(m));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((t & 31) == 0) red_s[t >> 5] = s;
  __syncthreads();
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < T / 32; ++i) sum += (double)red_s[i];
  return {m, sum};
}

// out = coef (onehot(target) - exp(x - m) / s) for the row; in may be out.
template <int T>
__device__ __forceinline__ void block_grad(const __nv_bfloat16* in, __nv_bfloat16* out, int V, float m, float sum,
                                           int target, float coef, const uint4* keep = nullptr, int n_keep = 0) {
  const int t = threadIdx.x;
  const float ref = safe_ref(m), k = -coef / sum;
  auto g = [&](float x, int i) {
    const float v = exp2_fast((x - ref) * kLog2e) * k;
    return i == target ? v + coef : v;
  };
  const RowSplit sp(in, V);
  if (((reinterpret_cast<uintptr_t>(in) ^ reinterpret_cast<uintptr_t>(out)) & 15) != 0) {
    // rows that start at different places within 16 bytes: element by element
    for (int i = t; i < V; i += T) out[i] = __float2bfloat16_rn(g(__bfloat162float(in[i]), i));
    return;
  }
  if (t < sp.head) out[t] = __float2bfloat16_rn(g(__bfloat162float(in[t]), t));
  const uint4* v = reinterpret_cast<const uint4*>(in + sp.head);
  uint4* o = reinterpret_cast<uint4*>(out + sp.head);
  auto piece = [&](const uint4& u, int j) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    const int i0 = sp.head + j * 8;
    uint32_t r[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = pack_bf16x2(g(bf16_lo(w[e]), i0 + 2 * e), g(bf16_hi(w[e]), i0 + 2 * e + 1));
    o[j] = make_uint4(r[0], r[1], r[2], r[3]);
  };
  // last pieces first: the statistics pass over the same row has left them in L2
  int j = t < sp.n16 ? t + (sp.n16 - 1 - t) / T * T : -1;  // this thread's last piece
  for (; j >= 0 && (j - t) / T % 4 != 3; j -= T) piece(v[j], j);  // behind the whole steps of four
  for (; j >= 0; j -= 4 * T) {
    const uint4* from = j < n_keep ? keep : v;
    const uint4 a = from[j], b = from[j - T], c = from[j - 2 * T], d = from[j - 3 * T];
    piece(a, j);
    piece(b, j - T);
    piece(c, j - 2 * T);
    piece(d, j - 3 * T);
  }
  const int i = sp.tail0 + t;
  if (i < V) out[i] = __float2bfloat16_rn(g(__bfloat162float(in[i]), i));
}

template <int T>
__device__ __forceinline__ void block_zero(__nv_bfloat16* out, int V) {
  const RowSplit sp(out, V);
  const int t = threadIdx.x;
  if (t < sp.head) out[t] = __float2bfloat16_rn(0.f);
  uint4* o = reinterpret_cast<uint4*>(out + sp.head);
  for (int j = t; j < sp.n16; j += T) o[j] = make_uint4(0u, 0u, 0u, 0u);
  if (sp.tail0 + t < V) out[sp.tail0 + t] = __float2bfloat16_rn(0.f);
}

// x[target] and m are bf16 values: the difference and the logarithm in 64 bits lose
// nothing that sums over long sequences would miss.
__device__ __forceinline__ double target_logp(float xt, RowStat st) { return (double)xt - (double)st.m - log(st.s); }

// A block per row.  (Clusters that share a row measured 140 us for 2048 rows of 128 k logits,
// this 73: small independent blocks, four to an SM, hide the reductions' waits best.)
template <int T>
__global__ void __launch_bounds__(T) k_token_logp(const __nv_bfloat16* __restrict__ logits, int64_t ld, int V,
                                                   const int32_t* __restrict__ targets, float4* __restrict__ stats,
                                                   float* __restrict__ logp) {
  next_may_start();
  const int row = blockIdx.x;
  const int target = targets[row];
  if (target < 0 || target >= V) {
    if (threadIdx.x == 0) {
      stats[row] = make_float4(0.f, 1.f, 0.f, 0.f);
      logp[row] = 0.f;
    }
    return;
  }
  const __nv_bfloat16* x = logits + (size_t)row * ld;
  const RowStat st = block_stats<T>(x, V);
  if (threadIdx.x == 0) {
    const double lp = target_logp(__bfloat162float(x[target]), st);
    const float hi = (float)lp;
    stats[row] = make_float4(st.m, (float)st.s, isfinite(hi) ? (float)(lp - (double)hi) : 0.f, 0.f);
    logp[row] = hi;
  }
}

// One block: sums of each sequence's log probabilities (a warp per sequence, in 64 bits),
// then every pair's loss and the coefficients of its two sequences.
constexpr int PT = 1024;
__global__ void __launch_bounds__(PT) k_preference(const int32_t* __restrict__ cu, int n_seqs,
                                                   const float* __restrict__ logp, const float4* __restrict__ stats,
                                                   const float* __restrict__ ref_logp,
                                                   float beta, float smoothing, int kind, float* __restrict__ seq_logp,
                                                   float* __restrict__ margin, float* __restrict__ coef,
                                                   float* __restrict__ loss) {
  __shared__ double red[PT / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n_pairs = n_seqs / 2;
  next_may_start();
  wait_for_previous();
  double total = 0.0;
  for (int pair = warp; pair < n_pairs; pair += PT / 32) {
    double sum[2];
    for (int e = 0; e < 2; ++e) {
      const int a = cu[2 * pair + e], b = cu[2 * pair + e + 1];
      double v = 0.0;
      for (int i = a + lane; i < b; i += 32) v += (double)logp[i] + (double)stats[i].z;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      sum[e] = v;
    }
    if (lane == 0) {
      const double gap = (sum[0] - sum[1]) - ((double)ref_logp[2 * pair] - (double)ref_logp[2 * pair + 1]);
      const double h = (double)beta * gap;
      double l, slope;  // of this pair's loss, and its derivative by gap
      if (kind == NF4LS_PREF_SIGMOID) {
        // -log sigmoid(h) = max(-h, 0) + log1p(exp(-|h|)); sigmoid(-h) without overflow
        const double e = exp(-fabs(h)), soft = log1p(e);
        const double away = h >= 0.0 ? e / (1.0 + e) : 1.0 / (1.0 + e);  // sigmoid(-h)
        l = (1.0 - smoothing) * (fmax(-h, 0.0) + soft);
        if (smoothing > 0.0f) l += smoothing * (fmax(h, 0.0) + soft);  // not 0 x inf for an infinite margin
        slope = beta * (smoothing * (1.0 - away) - (1.0 - smoothing) * away);
        if (isnan(h)) l = slope = h;
      } else if (kind == NF4LS_PREF_HINGE) {
        l = h < 1.0 ? 1.0 - h : 0.0;
        slope = h < 1.0 ? -(double)beta : 0.0;
        if (isnan(h)) l = slope = h;
      } else {
        const double z = gap - 0.5 / (double)beta;
        l = z * z;
        slope = 2.0 * z;
      }
      total += l;
      seq_logp[2 * pair] = (float)sum[0];
      seq_logp[2 * pair + 1] = (float)sum[1];
      margin[pair] = (float)h;
      coef[2 * pair] = (float)(slope / n_pairs);
      coef[2 * pair + 1] = (float)(-slope / n_pairs);
    }
  }
  if (lane == 0) red[warp] = total;
  __syncthreads();
  if (threadIdx.x == 0) {
    double v = 0.0;
    for (int i = 0; i < PT / 32; ++i) v += red[i];
    *loss = (float)(v / n_pairs);
  }
}

template <int T>
__global__ void __launch_bounds__(T, 2048 / T) k_logits_grad(const __nv_bfloat16* logits, int64_t ld, int V,
                                                    const int32_t* __restrict__ targets,
                                                    const float4* __restrict__ stats, const int32_t* __restrict__ seq,
                                                    const float* __restrict__ coef, float scale, __nv_bfloat16* dlogits,
                                                    int64_t ld_d) {
  // last rows first: they are what the forward's pass has left in L2
  const int row = gridDim.x - 1 - blockIdx.x;
  wait_for_previous();
  const int target = targets[row];
  __nv_bfloat16* out = dlogits + (size_t)row * ld_d;
  const float c = target >= 0 && target < V ? coef[seq[row]] * scale : 0.0f;
  if (c == 0.0f) {
    block_zero<T>(out, V);
    return;
  }
  const float4 st = stats[row];
  block_grad<T>(logits + (size_t)row * ld, out, V, st.x, st.y, target, c);
}

struct PolicyParams {
  const __nv_bfloat16* logits;
  __nv_bfloat16* dlogits;
  int64_t ld, ld_d;
  int V;
  const int32_t* targets;
  const float *old_logp, *ref_logp, *adv, *weights;
  float clip_low, clip_high, kl, scale;
  float *logp, *row_loss;
};

// By one thread: the row's loss, into memory, and the coefficient of its gradient; in 64 bits,
// since the terms of a mean over rows cancel.
__device__ __forceinline__ float policy_row(const PolicyParams& p, int row, float xt, RowStat st) {
  const double lp = target_logp(xt, st);
  const double a = p.adv[row], w = p.weights[row];
  const double r = exp(lp - (double)p.old_logp[row]);
  const double held_r = fmin(fmax(r, 1.0 - (double)p.clip_low), 1.0 + (double)p.clip_high);
  const double free_s = r * a, held = held_r * a;
  const bool passes = free_s <= held;  // the gradient flows through the unclipped term
  // no KL term where its coefficient is 0 (ref_logp may then be null)
  const double gap = p.kl > 0.0f ? (double)p.ref_logp[row] - lp : 0.0, e1 = expm1(gap);
  // the comparison drops a NaN of r or A (not 0 x inf, a row of no advantage): it goes into both
  const bool spoiled = isnan(r) || isnan(a);
  const double surrogate = spoiled ? r + a : (passes ? free_s : held), flows = spoiled ? r + a : (passes ? free_s : 0.0);
  p.logp[row] = (float)lp;
  p.row_loss[row] = (float)(w * (p.kl * (e1 - gap) - surrogate));
  return (float)(w * (-p.kl * e1 - flows) * p.scale);
}

// KEEP: pieces of 16 bytes of a row that stay in shared memory between its two passes.
template <int T, int KEEP>
__global__ void __launch_bounds__(T, 2048 / T) k_policy(const PolicyParams p) {
  __shared__ float c_sh;
  next_may_start();
  const int row = blockIdx.x;
  const int target = p.targets[row];
  __nv_bfloat16* out = p.dlogits ? p.dlogits + (size_t)row * p.ld_d : nullptr;
  if (target < 0 || target >= p.V) {
    if (threadIdx.x == 0) {
      p.logp[row] = 0.f;
      p.row_loss[row] = 0.f;
    }
    if (out) block_zero<T>(out, p.V);
    return;
  }
  const __nv_bfloat16* x = p.logits + (size_t)row * p.ld;
  const float xt = __bfloat162float(x[target]);
  extern __shared__ uint4 keep[];
  const int n_keep = out ? min(KEEP, RowSplit(x, p.V).n16) / (4 * T) * (4 * T) : 0;
  const RowStat st = block_stats<T>(x, p.V, keep, n_keep);
  if (threadIdx.x == 0) c_sh = policy_row(p, row, xt, st);
  if (!out) return;
  __syncthreads();
  const float c = c_sh;
  if (c == 0.0f)
    block_zero<T>(out, p.V);
  else
    block_grad<T>(x, out, p.V, st.m, (float)st.s, target, c, keep, n_keep);
}

__global__ void __launch_bounds__(PT) k_sum_rows(const float* __restrict__ v, int n, float* __restrict__ out) {
  __shared__ double red[PT / 32];
  double s = 0.0;
  wait_for_previous();
  for (int i = threadIdx.x; i < n; i += PT) s += (double)v[i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    double t = 0.0;
    for (int i = 0; i < PT / 32; ++i) t += red[i];
    *out = (float)t;
  }
}

template <typename... P, typename... A>
int launch(void (*k)(P...), int64_t blocks, int threads, bool early, cudaStream_t s, A... args) {
  NF4_CUDA_TRY(launch_kernel(k, blocks, {threads, 0, early, 1}, s, args...));
  note_launch();
  return NF4LS_OK;
}

int check_logits(const nf4ls_logits* t, int rows, const char* who) {
  if (!t) return fail(NF4LS_INVALID_ARG, "%s: null logits", who);
  if (t->vocab < 1 || t->vocab > (1 << 28)) return fail(NF4LS_SHAPE, "%s: vocab %d", who, t->vocab);
  if (t->ld < t->vocab || t->ld > (1ll << 40)) return fail(NF4LS_SHAPE, "%s: row stride %lld < vocab %d", who, (long long)t->ld, t->vocab);
  if (rows > 0 && (!t->logits_dev || !t->targets_dev)) return fail(NF4LS_INVALID_ARG, "%s: null logits or targets", who);
  if (!aligned(t->logits_dev, 2) || !aligned(t->targets_dev, 4)) return fail(NF4LS_ALIGN, "%s: misaligned logits or targets", who);
  return NF4LS_OK;
}

int check_grad(const nf4ls_logits* t, const void* d, int64_t ld, const char* who) {
  if (ld < t->vocab || ld > (1ll << 40)) return fail(NF4LS_SHAPE, "%s: row stride %lld of the gradient", who, (long long)ld);
  if (!aligned(d, 2)) return fail(NF4LS_ALIGN, "%s: misaligned gradient", who);
  if (d == t->logits_dev && ld != t->ld) return fail(NF4LS_INVALID_ARG, "%s: in place with another row stride", who);
  return NF4LS_OK;
}

}  // namespace

}  // namespace nf4ls

using namespace nf4ls;

extern "C" int nf4ls_preference_fwd(const nf4ls_pack* pack, const nf4ls_preference_cfg* c, const nf4ls_logits* t,
                                    const float* ref_logp_dev, const nf4ls_preference_out* out, nf4ls_stream stream) {
  const char* who = "nf4ls_preference_fwd";
  clear_error();
  NF4_TRY(check_pack(pack, who));
  if (!c || !out) return fail(NF4LS_INVALID_ARG, "%s: null config or outputs", who);
  if (pack->n_seqs % 2) return fail(NF4LS_SHAPE, "%s: %d sequences are not pairs", who, pack->n_seqs);
  if (c->kind < NF4LS_PREF_SIGMOID || c->kind > NF4LS_PREF_SQUARED) return fail(NF4LS_INVALID_ARG, "%s: unknown kind %d", who, c->kind);
  if (!(c->beta > 0.0f) || !std::isfinite(c->beta)) return fail(NF4LS_INVALID_ARG, "%s: beta must be positive", who);
  if (!(c->label_smoothing >= 0.0f && c->label_smoothing < 0.5f))
    return fail(NF4LS_INVALID_ARG, "%s: label_smoothing outside [0, 0.5)", who);
  NF4_TRY(check_logits(t, pack->total, who));
  if (!ref_logp_dev || !out->loss || !out->seq_logp || !out->margin || !out->coef ||
      (pack->total > 0 && (!out->logp || !out->row_stats)))
    return fail(NF4LS_INVALID_ARG, "%s: null reference or output", who);
  if (!aligned(out->row_stats, 16)) return fail(NF4LS_ALIGN, "%s: row_stats must be 16-byte aligned", who);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto* stats = reinterpret_cast<float4*>(out->row_stats);
  if (pack->total > 0) {
    const auto* x = static_cast<const __nv_bfloat16*>(t->logits_dev);
    const bool brief = t->vocab < kShortRow;
    NF4_TRY(launch(brief ? k_token_logp<256> : k_token_logp<512>, pack->total, brief ? 256 : 512, false, s, x, t->ld, t->vocab, t->targets_dev, stats, out->logp));
  }
  const int32_t* cu = reinterpret_cast<const int32_t*>(static_cast<const uint8_t*>(pack->plan_dev) + pack->off_cu);
  NF4_TRY(launch(k_preference, 1, PT, true, s, cu, pack->n_seqs, out->logp, stats, ref_logp_dev, c->beta,
                 c->label_smoothing, c->kind, out->seq_logp, out->margin, out->coef, out->loss));
  return NF4LS_OK;
}

extern "C" int nf4ls_preference_bwd(const nf4ls_pack* pack, const nf4ls_logits* t, const nf4ls_preference_out* saved,
                                    float grad_scale, void* dlogits_dev, int64_t ld_d, nf4ls_stream stream) {
  const char* who = "nf4ls_preference_bwd";
  clear_error();
  NF4_TRY(check_pack(pack, who));
  NF4_TRY(check_logits(t, pack->total, who));
  if (pack->total == 0) return NF4LS_OK;
  if (!saved || !saved->row_stats || !saved->coef || !dlogits_dev) return fail(NF4LS_INVALID_ARG, "%s: null argument", who);
  if (!aligned(saved->row_stats, 16)) return fail(NF4LS_ALIGN, "%s: row_stats must be 16-byte aligned", who);
  NF4_TRY(check_grad(t, dlogits_dev, ld_d, who));
  const int32_t* seq = reinterpret_cast<const int32_t*>(static_cast<const uint8_t*>(pack->plan_dev) + pack->off_seq);
  const bool brief = t->vocab < kShortRow;
  NF4_TRY(launch(brief ? k_logits_grad<256> : k_logits_grad<512>, pack->total, brief ? 256 : 512, true,
                 static_cast<cudaStream_t>(stream),
                 static_cast<const __nv_bfloat16*>(t->logits_dev), t->ld, t->vocab, t->targets_dev,
                 reinterpret_cast<const float4*>(saved->row_stats), seq, saved->coef, grad_scale,
                 static_cast<__nv_bfloat16*>(dlogits_dev), ld_d));
  return NF4LS_OK;
}

extern "C" int nf4ls_policy_loss(const nf4ls_policy_cfg* c, int32_t rows, const nf4ls_logits* t, const nf4ls_policy_rows* in,
                                 float* loss_dev, float* logp_dev, float* row_loss_dev, void* dlogits_dev, int64_t ld_d,
                                 nf4ls_stream stream) {
  const char* who = "nf4ls_policy_loss";
  clear_error();
  if (!c || !loss_dev) return fail(NF4LS_INVALID_ARG, "%s: null config or loss", who);
  if (rows < 0) return fail(NF4LS_INVALID_ARG, "%s: %d rows", who, rows);
  if (!(c->clip_low >= 0.0f && c->clip_low <= 1.0f) || !(c->clip_high >= 0.0f) || !std::isfinite(c->clip_high))
    return fail(NF4LS_INVALID_ARG, "%s: clip range %g, %g", who, c->clip_low, c->clip_high);
  if (!(c->kl_coef >= 0.0f) || !std::isfinite(c->kl_coef)) return fail(NF4LS_INVALID_ARG, "%s: kl_coef %g", who, c->kl_coef);
  if (!std::isfinite(c->grad_scale)) return fail(NF4LS_INVALID_ARG, "%s: grad_scale %g", who, c->grad_scale);
  NF4_TRY(check_logits(t, rows, who));
  if (rows > 0 && (!in || !in->old_logp || (c->kl_coef > 0.0f && !in->ref_logp) || !in->advantages || !in->weights || !logp_dev || !row_loss_dev))
    return fail(NF4LS_INVALID_ARG, "%s: null row argument", who);
  if (dlogits_dev) NF4_TRY(check_grad(t, dlogits_dev, ld_d, who));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows > 0) {
    PolicyParams p;
    p.logits = static_cast<const __nv_bfloat16*>(t->logits_dev);
    p.dlogits = static_cast<__nv_bfloat16*>(dlogits_dev);
    p.ld = t->ld;
    p.ld_d = ld_d;
    p.V = t->vocab;
    p.targets = t->targets_dev;
    p.old_logp = in->old_logp;
    p.ref_logp = in->ref_logp;
    p.adv = in->advantages;
    p.weights = in->weights;
    p.clip_low = c->clip_low;
    p.clip_high = c->clip_high;
    p.kl = c->kl_coef;
    p.scale = c->grad_scale;
    p.logp = logp_dev;
    p.row_loss = row_loss_dev;
    if (p.V < kShortRow) {
      NF4_TRY(launch(k_policy<256, 0>, rows, 256, false, s, p));
    } else if (p.V < kLongRow) {
      NF4_TRY(launch(k_policy<512, 0>, rows, 512, false, s, p));
    } else {
      constexpr int T = 768, KEEP = 8 * T;  // without a gradient too: the same bits
      static int configured[64] = {0};
      int dev = 0;
      NF4_CUDA_TRY(cudaGetDevice(&dev));
      if (dev >= 64 || !configured[dev]) {
        NF4_CUDA_TRY(cudaFuncSetAttribute(k_policy<T, KEEP>, cudaFuncAttributeMaxDynamicSharedMemorySize, KEEP * 16));
        if (dev < 64) configured[dev] = 1;
      }
      NF4_CUDA_TRY(launch_kernel(k_policy<T, KEEP>, rows, {T, p.dlogits ? (size_t)KEEP * 16 : 0, false, 1}, s, p));
      note_launch();
    }
  }
  NF4_TRY(launch(k_sum_rows, 1, PT, true, s, row_loss_dev, rows, loss_dev));
  return NF4LS_OK;
}
