// gate.cu -- the router: experts and weights of each token from its logits, the
// load-balance loss, and their gradients.
//
// Gate.  key_e = fl32(l_e + bias_e) (the bias steers selection alone), ids = the top_k
// largest keys, largest first, equal keys by the lower expert.  Selection is one fp32 add
// and comparisons, so the choice is the same bits on any machine and can be replayed.
// s = softmax(l) over the experts or sigmoid(l); weight of the i-th choice
//   w_i = c s_i / sum_j s_j (j over the choices)   or, not normalised,   c s_i.
//
// Gradient, g_i = dL/dw_i, sums over the choices:
//   softmax, normalised   dl_i = w_i (g_i - sum_j w_j g_j / c)
//   softmax               dl_e = p_e (c g_e [e chosen] - sum_j c p_j g_j)
//   sigmoid, normalised   dl_i = p_i (1 - s_i) (c g_i - sum_j p_j c g_j),  p_i = s_i / sum_j s_j
//   sigmoid               dl_i = c g_i s_i (1 - s_i)
//
// Balance loss.  p = softmax(l) or sigmoid(l) / Z.  Over the T_q counted tokens of each
// sequence q (empty ones left out, S of them are not):
//   L = alpha / S  sum_q  E / (K T_q^2)  sum_e count_qe  sum_t p_te
// The counts are constants to the gradient:
//   a_e = dL alpha / S  E / (K T_q^2) count_qe,   softmax: dl_e = p_e (a_e - sum_j p_j a_j),
//   sigmoid: dl_e = s_e (1 - s_e) / Z (a_e - sum_j p_j a_j).
//
// One warp a token, V experts a lane, VEC of them neighbours (one load of up to 16 bytes); all
// sums fp32.  Reads the logits once.  Few tokens: launch-bound.  Many: the instructions of the
// selection (393 a token of 256 experts, top 8) and of the probabilities (208 in the loss, 254 in its
// gradient), at 68 to 86% of the issue rate, take longer than its bytes.  32768 x 256, us, launched from a graph:
// gate (fp32, softmax) 13.1, gradient 7.0, without normalize 15.6; balance loss (bf16, sigmoid, 13 sequences)
// 17.5, gradient 13.2, added onto another 14.4.
#include "block128.cuh"

namespace fme {

namespace {

constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kGateWarps = 8;

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_float(float v) {
  if constexpr (sizeof(T) == 2)
    return __float2bfloat16_rn(v);
  else
    return v;
}

template <typename T, int VEC>
struct alignas(VEC * sizeof(T)) Pack {
  T v[VEC];
};

// Expert of a lane's j-th value.
template <int VEC>
__device__ __forceinline__ int expert_of(int j, int lane) {
  return (j / VEC) * (32 * VEC) + lane * VEC + j % VEC;
}

// A token's row, V values a lane; -inf past the experts (a multiple of VEC).
template <typename T, int V, int VEC>
__device__ __forceinline__ void load_row(const T *row, int experts, int lane, float (&l)[V]) {
#pragma unroll
  for (int j = 0; j < V; j += VEC) {
    const int e = expert_of<VEC>(j, lane);
    if (e < experts) {
      const Pack<T, VEC> p = *reinterpret_cast<const Pack<T, VEC> *>(row + e);
#pragma unroll
      for (int c = 0; c < VEC; ++c) l[j + c] = to_float(p.v[c]);
    } else {
#pragma unroll
      for (int c = 0; c < VEC; ++c) l[j + c] = -INFINITY;
    }
  }
}

template <typename T, int V, int VEC>
__device__ __forceinline__ void store_row(T *row, int experts, int lane, const float (&v)[V]) {
#pragma unroll
  for (int j = 0; j < V; j += VEC) {
    const int e = expert_of<VEC>(j, lane);
    if (e < experts) {
      Pack<T, VEC> p;
#pragma unroll
      for (int c = 0; c < VEC; ++c) p.v[c] = from_float<T>(v[j + c]);
      *reinterpret_cast<Pack<T, VEC> *>(row + e) = p;
    }
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int s = 16; s; s >>= 1) v += __shfl_xor_sync(kAll, v, s);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int s = 16; s; s >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, s));
  return v;
}

// sigmoid(l) and 1 - sigmoid(l) = sigmoid(-l) from one exponential that cannot overflow,
// t = e^-|l|: 1 / (1 + t) and t / (1 + t).  A NaN stays one.
__device__ __forceinline__ void sigmoids(float l, float &s, float &rest) {
  const float t = __expf(-fabsf(l));
  const float r = rcp_approx(1.0f + t);
  const float tr = t * r;
  s = l >= 0.0f ? r : tr;
  rest = l >= 0.0f ? tr : r;
}
__device__ __forceinline__ float sigmoid(float l) {
  float s, rest;
  sigmoids(l, s, rest);
  return s;
}

// Ratios of sigmoids, s_i / sum of s, of rows far below zero.  Sigmoids are subnormal from -87 and zero from -104 down,
// their ratios are not.  Where the sum is below this, every logit is negative, and e^(l - max) (1 - s), which is
// s e^-max, takes the place of s: the factor cancels.  2^-8: what the sigmoids themselves then lose is a ratio
// below 2^-118, next to fp32's own 2^-126.  Other rows keep their one exponential.
constexpr float kSmallSum = 0x1p-8f;

// Order of floats (no NaN) as unsigned integers: larger float, larger integer, none 0; -0 as +0.
__device__ __forceinline__ uint32_t order_key(float f) {
  const int32_t b = __float_as_int(f + 0.0f);
  return static_cast<uint32_t>(b) ^ (static_cast<uint32_t>(b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_order(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// The largest of a row held V values a lane, or 0 where nothing is above -inf: a finite offset for
// exponentials, so that such a row's are 0 and only +inf and NaN give NaN.
template <int V>
__device__ __forceinline__ float row_offset(const float (&l)[V]) {
  float m = l[0];
#pragma unroll
  for (int j = 1; j < V; ++j) m = fmaxf(m, l[j]);
  m = warp_max(m);
  return m == -INFINITY ? 0.0f : m;
}

// x = exp(l - m) of the row (lanes past the experts hold -inf) and its sum.
template <int V>
__device__ __forceinline__ float exp_row(const float (&l)[V], float m, float (&x)[V]) {
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    x[j] = __expf(l[j] - m);
    sum += x[j];
  }
  return warp_sum(sum);
}

template <typename T, int V, int VEC>
__global__ void __launch_bounds__(32 * kGateWarps) gate_kernel(const T *__restrict__ logits, int64_t tokens,
                                                               int experts, int top_k, bool softmax, bool normalize,
                                                               float scale, const float *__restrict__ bias,
                                                               int32_t *__restrict__ ids,
                                                               float *__restrict__ weights) {
  // candidates' keys and experts
  __shared__ alignas(16) float cand[kGateWarps][32];
  __shared__ int cand_id[kGateWarps][32];
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kGateWarps + warp;
  if (t >= tokens) return;
  const T *row = logits + t * experts;
  float l[V];
  load_row<T, V, VEC>(row, experts, lane, l);
  float denom = 1.0f, m_all = 0.0f;  // softmax over all experts, only where the weights need it
  if (softmax && !normalize) {
    float x[V];
    m_all = row_offset<V>(l);
    denom = exp_row<V>(l, m_all, x);
  }
  // Keys, a NaN as -inf; `live`: not past the experts (whole packs are or are not).
  float key[V];
  bool live[V];
#pragma unroll
  for (int j = 0; j < V; ++j) live[j] = expert_of<VEC>(j - j % VEC, lane) < experts;
  if (bias) {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (live[j]) l[j] += __ldg(bias + expert_of<VEC>(j, lane));
  }
#pragma unroll
  for (int j = 0; j < V; ++j) key[j] = fmaxf(l[j], -INFINITY);
  // A lower bound of the top_k-th key: the top_k-th largest of the lanes' largest keys (equal ones
  // taken together, which only lowers it).
  float bound = -INFINITY;
  if constexpr (V > 1) {
    float largest = key[0];
#pragma unroll
    for (int j = 1; j < V; ++j) largest = fmaxf(largest, key[j]);
    uint32_t m = order_key(largest), at_most = 0;
    for (int i = 0; i < top_k; ++i) {
      at_most = __reduce_max_sync(kAll, m);
      if (m == at_most) m = 0;
    }
    if (at_most) bound = from_order(at_most);
  }
  // The keys at or above it are the candidates, in any order: every lane hands in one at a time.
  uint32_t mine_set = 0;
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (key[j] >= bound && live[j]) mine_set |= 1u << j;
  int *ci = cand_id[warp];
  int n = 0;
  while (const uint32_t has = __ballot_sync(kAll, mine_set != 0)) {
    const int at = n + __popc(has & ((1u << lane) - 1));
    if (mine_set && at < 32) ci[at] = expert_of<VEC>(__ffs(mine_set) - 1, lane);
    mine_set &= mine_set - 1;
    n += __popc(has);
  }
  int pos = top_k, my_id = 0;  // this lane's choice: number and expert; none if pos >= top_k
  float my_l = -INFINITY;      // without the bias
  if (n <= 32) {
    float *ck = cand[warp];
    __syncwarp();
    if (lane < n) {
      my_id = ci[lane];
      my_l = to_float(row[my_id]);
    }
    const float me = fmaxf(bias && lane < n ? my_l + __ldg(bias + my_id) : my_l, -INFINITY);
    ck[lane] = me;
    __syncwarp();
    // every candidate counts the larger keys
    int before = 0;
    for (int q = 0; q < n; q += 4) {
      const float4 k = *reinterpret_cast<const float4 *>(ck + q);
      before += (k.x > me ? 1 : 0) + (k.y > me ? 1 : 0) + (k.z > me ? 1 : 0) + (k.w > me ? 1 : 0);
    }
    // Of two different keys one counts the other: fewer counts than pairs, and some are equal.
    if (__reduce_add_sync(kAll, lane < n ? before : 0) != n * (n - 1) / 2)
      for (int q = 0; q < n; ++q) before += ck[q] == me && ci[q] < my_id ? 1 : 0;
    if (lane < n) pos = before;
  } else {
    // many equal keys: one choice after the other
    uint32_t left[V];
#pragma unroll
    for (int j = 0; j < V; ++j) left[j] = live[j] ? order_key(key[j]) : 0u;
    for (int i = 0; i < top_k; ++i) {
      uint32_t best = 0;
#pragma unroll
      for (int j = 0; j < V; ++j) best = max(best, left[j]);
      best = __reduce_max_sync(kAll, best);
      int e = INT32_MAX;
#pragma unroll
      for (int j = V - 1; j >= 0; --j)
        if (left[j] == best) e = expert_of<VEC>(j, lane);
      e = __reduce_min_sync(kAll, e);
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (e == expert_of<VEC>(j, lane)) left[j] = 0;
      if (lane == i) {
        pos = i;
        my_id = e;
        my_l = to_float(row[e]);
      }
    }
  }
  const bool mine = pos < top_k;
  if (!mine) my_l = -INFINITY;
  float s;
  if (softmax) {
    float ref = normalize ? warp_max(my_l) : m_all;
    if (ref == -INFINITY) ref = 0.0f;
    s = mine ? __expf(my_l - ref) : 0.0f;
  } else {
    s = mine ? sigmoid(my_l) : 0.0f;
  }
  if (normalize) {
    denom = warp_sum(s);
    if (!softmax && denom < kSmallSum) {
      const float top = warp_max(my_l);
      s = __expf(my_l - (top == -INFINITY ? 0.0f : top)) * (1.0f - s);
      denom = warp_sum(s);
    }
  }
  if (mine) {
    ids[t * top_k + pos] = my_id;
    weights[t * top_k + pos] = denom == 0.0f ? 0.0f : scale * s / denom;
  }
}

// softmax without normalize: every expert has a share of the gradient.
template <typename T, int V, int VEC>
__global__ void __launch_bounds__(32 * kGateWarps) gate_backward_dense_kernel(
    const T *__restrict__ logits, const int32_t *__restrict__ ids, const float *__restrict__ d_weights, int64_t tokens,
    int experts, int top_k, float scale, T *__restrict__ d_logits, int32_t *status) {
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kGateWarps + (threadIdx.x >> 5);
  if (t >= tokens) return;
  const T *row = logits + t * experts;
  float l[V], x[V];
  load_row<T, V, VEC>(row, experts, lane, l);
  int id = lane < top_k ? __ldg(ids + t * top_k + lane) : -1;
  if (lane < top_k && (id < 0 || id >= experts)) {
    report(status, kDevBadIndex);
    id = -1;
  }
  const bool live = id >= 0;
  const float g = live ? scale * __ldg(d_weights + t * top_k + lane) : 0.0f;
  const float my_l = live ? to_float(row[id]) : -INFINITY;
  const float m = row_offset<V>(l);
  const float denom = exp_row<V>(l, m, x);
  const float inner = warp_sum(live && denom != 0.0f ? __expf(my_l - m) / denom * g : 0.0f);
  const float r = denom == 0.0f ? 0.0f : 1.0f / denom;
#pragma unroll
  for (int j = 0; j < V; ++j) l[j] = 0.0f;  // the choices' g
  for (int i = 0; i < top_k; ++i) {
    const int e = __shfl_sync(kAll, id, i);
    const float v = __shfl_sync(kAll, g, i);
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (e == expert_of<VEC>(j, lane)) l[j] = v;
  }
#pragma unroll
  for (int j = 0; j < V; ++j) l[j] = x[j] * r * (l[j] - inner);
  store_row<T, V, VEC>(d_logits + t * experts, experts, lane, l);
}

// The rest: only the choices' logits are read and only their gradients are not zero.  kWidth lanes
// (a power of two, at least top_k) take a token and a warp 32 / kWidth of them, so that their chains
// of dependent loads run side by side (top_k = 8, 32768 x 256: 10.8 -> 7.6 us); the warp writes zeros
// over its tokens' rows, then the choices' values.
template <typename T, int kWidth>
__global__ void __launch_bounds__(32 * kGateWarps) gate_backward_kernel(
    const T *__restrict__ logits, const int32_t *__restrict__ ids, const float *__restrict__ d_weights, int64_t tokens,
    int experts, int top_k, bool softmax, bool normalize, float scale, T *__restrict__ d_logits, int32_t *status) {
  constexpr int kTokens = 32 / kWidth;
  const int lane = threadIdx.x & 31;
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kGateWarps + (threadIdx.x >> 5)) * kTokens;
  if (t0 >= tokens) return;
  const int64_t t = t0 + lane / kWidth;
  const int i = lane % kWidth;
  auto group_sum = [](float v) {
#pragma unroll
    for (int s = kWidth / 2; s; s >>= 1) v += __shfl_xor_sync(kAll, v, s);
    return v;
  };
  const bool mine = t < tokens && i < top_k;
  int id = mine ? __ldg(ids + t * top_k + i) : -1;
  if (mine && (id < 0 || id >= experts)) {
    report(status, kDevBadIndex);
    id = -1;
  }
  const bool live = id >= 0;
  const float g = live ? scale * __ldg(d_weights + t * top_k + i) : 0.0f;
  const float l = live ? to_float(logits[t * experts + id]) : -INFINITY;
  // zeros while the logits are on their way
  const int64_t n = min(tokens - t0, static_cast<int64_t>(kTokens)) * experts;
  T *out = d_logits + t0 * experts;
  if (experts * sizeof(T) % 16 == 0) {
    for (int64_t c = lane; c < n * static_cast<int64_t>(sizeof(T)) / 16; c += 32)
      reinterpret_cast<uint4 *>(out)[c] = make_uint4(0, 0, 0, 0);
  } else {
    for (int64_t c = lane; c < n; c += 32) out[c] = from_float<T>(0.0f);
  }
  float d;
  if (softmax) {
    float ref = l;
#pragma unroll
    for (int s = kWidth / 2; s; s >>= 1) ref = fmaxf(ref, __shfl_xor_sync(kAll, ref, s));
    if (ref == -INFINITY) ref = 0.0f;
    const float s = live ? __expf(l - ref) : 0.0f;
    const float total = group_sum(s);
    const float p = total == 0.0f ? 0.0f : s / total;
    d = p * (g - group_sum(p * g));
  } else {
    float s = 0.0f, rest = 0.0f;
    if (live) sigmoids(l, s, rest);
    if (normalize) {
      float total = group_sum(s);
      if (__any_sync(kAll, total < kSmallSum)) {
        float top = l;
#pragma unroll
        for (int o = kWidth / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
        const float near = __expf(l - (top == -INFINITY ? 0.0f : top)) * rest;
        if (total < kSmallSum) s = near;
        total = group_sum(s);
      }
      const float p = total == 0.0f ? 0.0f : s / total;
      d = p * (g - group_sum(p * g)) * rest;
    } else {
      d = g * s * rest;
    }
  }
  __syncwarp();
  if (live) d_logits[t * experts + id] = from_float<T>(d);
}

// ------------------------------------------------------------- balance loss --
// Probabilities of one token's row, V a lane; also s and 1 - s scaled for the gradient.  A row far below zero is
// read again (kept for that, its logits would cost the other rows registers).
template <typename T, int V, int VEC>
__device__ __forceinline__ void probabilities(const float (&l)[V], const T *row, int experts, int lane, bool softmax,
                                              float (&p)[V], float (&slope)[V]) {
  if (softmax) {
    const float z = exp_row<V>(l, row_offset<V>(l), p);
    const float r = z == 0.0f ? 0.0f : 1.0f / z;
#pragma unroll
    for (int j = 0; j < V; ++j) slope[j] = p[j] = p[j] * r;
  } else {
    float z = 0.0f;  // lanes past the experts hold -inf: sigmoid 0
#pragma unroll
    for (int j = 0; j < V; ++j) {
      sigmoids(l[j], p[j], slope[j]);
      z += p[j];
    }
    z = warp_sum(z);
    if (z < kSmallSum) {  // slope: 1 - s
      load_row<T, V, VEC>(row, experts, lane, p);
      const float top = row_offset<V>(p);
      z = 0.0f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float s;
        sigmoids(p[j], s, slope[j]);
        p[j] = __expf(p[j] - top) * slope[j];
        z += p[j];
      }
      z = warp_sum(z);
    }
    const float r = z == 0.0f ? 0.0f : 1.0f / z;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      p[j] *= r;
      slope[j] *= p[j];
    }
  }
}

// The last sequence that starts at or before token t (so empty ones are passed over): halving down
// to 32 candidates, then all at once.  The whole warp calls it.
__device__ __forceinline__ int64_t find_sequence(const int32_t *offsets, int64_t num_seqs, int64_t t, int lane) {
  int64_t lo = 0, hi = num_seqs;
  while (hi - lo > 32) {
    const int64_t mid = (lo + hi) >> 1;
    if (__ldg(offsets + mid) <= t)
      lo = mid;
    else
      hi = mid;
  }
  const int64_t mine = lo + 1 + lane;
  return lo + __popc(__ballot_sync(kAll, mine < hi && __ldg(offsets + mine) <= t));
}

// One CTA for `chunk` consecutive tokens: for each sequence that has some of them, the sums of p and
// the counts of its counted tokens go to the workspace's slot chunk + sequence (along the tokens one
// of the two grows from piece to piece, so no two pieces share a slot).  Equal chunks of tokens
// rather than slices of each sequence, whose lengths may differ a hundredfold.  The order of every
// sum is fixed.
constexpr int kPartWarps = 16;

template <typename T, int V, int VEC>
__global__ void __launch_bounds__(32 * kPartWarps) balance_partial_kernel(LaunchBalance a) {
  extern __shared__ float smem[];  // [kPartWarps / 2][experts] sums, then [experts] counts
  constexpr int kHalf = kPartWarps / 2;
  start_next_kernel();
  const int experts = a.num_experts;
  int32_t *cnt = reinterpret_cast<int32_t *>(smem + kHalf * experts);
  __shared__ int32_t n_tokens;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * a.chunk;
  const int64_t c1 = min(a.tokens, c0 + a.chunk);
  if (blockIdx.x == 0) {  // once: are the sequences well formed?
    bool bad = false;
    if (a.seq_offsets)
      for (int64_t s = threadIdx.x; s <= a.num_seqs; s += blockDim.x) {
        const int32_t v = __ldg(a.seq_offsets + s);
        bad |= s == 0 ? v != 0 : v < __ldg(a.seq_offsets + s - 1);
        bad |= s == a.num_seqs && v != a.tokens;
      }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) {
      a.flags[0] = 0;  // CTAs of balance_final_kernel that are done
      a.flags[1] = bad;
      if (bad) report(a.status, kDevBadOffsets);
    }
  }
  const T *logits = static_cast<const T *>(a.logits);
  // the next token's row, mask and choice, loaded while this one is summed
  float next[V];
  bool next_on = false;
  int32_t next_id = 0;
  auto prefetch = [&](int64_t t) {
    load_row<T, V, VEC>(logits + t * experts, experts, lane, next);
    next_on = !a.token_mask || __ldg(a.token_mask + t);
    if (lane < a.top_k) next_id = __ldg(a.ids + t * a.top_k + lane);
  };
  if (c0 + warp < c1) prefetch(c0 + warp);
  for (int64_t t0 = c0; t0 < c1;) {
    int64_t seq = 0, t1 = c1;
    if (a.seq_offsets) {
      seq = find_sequence(a.seq_offsets, a.num_seqs, t0, lane);
      t1 = min(c1, static_cast<int64_t>(__ldg(a.seq_offsets + seq + 1)));
      if (t1 <= t0) break;  // malformed: no sequence holds t0
    }
    if (t0 > c0 && t0 + warp < t1) prefetch(t0 + warp);
    for (int e = threadIdx.x; e < experts; e += blockDim.x) cnt[e] = 0;
    if (threadIdx.x == 0) n_tokens = 0;
    __syncthreads();
    float sum[V];
#pragma unroll
    for (int j = 0; j < V; ++j) sum[j] = 0.0f;
    int mine = 0;
    for (int64_t t = t0 + warp; t < t1; t += kPartWarps) {
      float l[V], p[V], slope[V];
#pragma unroll
      for (int j = 0; j < V; ++j) l[j] = next[j];
      const bool on = next_on;
      const int32_t e = next_id;
      if (t + kPartWarps < t1) prefetch(t + kPartWarps);
      if (!on) continue;
      if (lane < a.top_k) {
        if (e >= 0 && e < experts)
          atomicAdd(&cnt[e], 1);
        else
          report(a.status, kDevBadIndex);
      }
      probabilities<T, V, VEC>(l, logits + t * experts, experts, lane, a.softmax, p, slope);
#pragma unroll
      for (int j = 0; j < V; ++j) sum[j] += p[j];
      ++mine;
    }
    if (lane == 0 && mine) atomicAdd(&n_tokens, mine);
    if (warp >= kHalf) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (expert_of<VEC>(j, lane) < experts) smem[(warp - kHalf) * experts + expert_of<VEC>(j, lane)] = sum[j];
    }
    __syncthreads();
    if (warp < kHalf) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (expert_of<VEC>(j, lane) < experts) smem[warp * experts + expert_of<VEC>(j, lane)] += sum[j];
    }
    __syncthreads();
    const int64_t slot = blockIdx.x + seq;
    for (int e = threadIdx.x; e < experts; e += blockDim.x) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kHalf; ++w) v += smem[w * experts + e];
      a.part_sum[slot * experts + e] = v;
      a.part_count[slot * experts + e] = cnt[e];
    }
    if (threadIdx.x == 0) a.part_tokens[slot] = n_tokens;
    t0 = t1;
    __syncthreads();  // before the next piece clears what was just read
  }
}

// Adds one and returns what was there; orders the thread's writes before it, and later reads after it.
__device__ __forceinline__ int32_t take_ticket(int32_t *counter) {
  int32_t old;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(old) : "l"(counter) : "memory");
  return old;
}

// One CTA for 32 experts of a sequence: lane = expert, each warp adds every 32nd piece, the warps'
// sums are added in order; then the experts' part of the sequence's term.  The last CTA to finish adds
// all parts in order; an only CTA has nothing to add (1023 tokens x 32 experts: the loss 8.5 -> 6.1 us).
__global__ void __launch_bounds__(1024) balance_final_kernel(LaunchBalance a) {
  __shared__ float sums[32][33];
  __shared__ int32_t cnts[32][33];
  __shared__ float2 red[32];
  __shared__ int last;
  __shared__ int32_t total_tokens;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int experts = a.num_experts;
  const int groups = (experts + 31) >> 5;
  const int64_t s = blockIdx.x / groups;
  const int e = static_cast<int>(blockIdx.x - s * groups) * 32 + lane;
  if (tid == 0) total_tokens = 0;
  // the sequence's pieces: slots first .. last
  wait_for_previous_kernel();
  const bool bad = __ldcg(a.flags + 1) != 0;  // malformed sequences: no token counts
  // (cut to the tokens, so that malformed ones stay inside the workspace until `bad` is known)
  const int64_t lo = a.seq_offsets ? max(0, __ldg(a.seq_offsets + s)) : 0;
  const int64_t hi = a.seq_offsets ? min(a.tokens, static_cast<int64_t>(__ldg(a.seq_offsets + s + 1))) : a.tokens;
  const bool none = hi <= lo;
  const int64_t first = none ? 0 : lo / a.chunk + s;
  const int64_t last_slot = none ? -1 : (hi - 1) / a.chunk + s;
  float v = 0.0f;
  int32_t c = 0;
  if (e < experts) {
#pragma unroll 4
    for (int64_t i = first + warp; i <= last_slot; i += 32) {
      v += a.part_sum[i * experts + e];
      c += a.part_count[i * experts + e];
    }
  }
  sums[warp][lane] = bad ? 0.0f : v;
  cnts[warp][lane] = bad ? 0 : c;
  int32_t n = 0;
  for (int64_t i = first + tid; i <= last_slot; i += 1024) n += a.part_tokens[i];
  __syncthreads();
  if (n && !bad) atomicAdd(&total_tokens, n);
  __syncthreads();
  if (warp == 0) {
    v = 0.0f;
    c = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      v += sums[i][lane];
      c += cnts[i][lane];
    }
    if (e < experts) a.counts[s * experts + e] = c;
    const float term = warp_sum(e < experts ? static_cast<float>(c) * v : 0.0f);
    if (lane == 0) {
      const int32_t t = total_tokens;
      const float tf = static_cast<float>(t);
      if (e < 32) a.seq_tokens[s] = t;
      const float all = t > 0 ? term / tf * (static_cast<float>(experts) / (static_cast<float>(a.top_k) * tf)) : 0.0f;
      if (gridDim.x == 1) {  // the only part
        a.loss[0] = a.alpha * all;
        last = 0;
      } else {
        a.term[blockIdx.x] = all;
        last = take_ticket(a.flags) == static_cast<int32_t>(gridDim.x) - 1;
      }
    }
  }
  __syncthreads();
  if (!last) return;
  float all = 0.0f, live = 0.0f;
  for (int64_t i = tid; i < gridDim.x; i += 1024) all += __ldcg(a.term + i);
  for (int64_t i = tid; i < a.num_seqs; i += 1024) live += __ldcg(a.seq_tokens + i) > 0 ? 1.0f : 0.0f;
  all = warp_sum(all);
  live = warp_sum(live);
  if (lane == 0) red[warp] = make_float2(all, live);
  __syncthreads();
  if (warp == 0) {
    all = warp_sum(red[lane].x);
    live = warp_sum(red[lane].y);
    if (lane == 0) a.loss[0] = live > 0.0f ? a.alpha * all / live : 0.0f;
  }
}

// A warp takes `per_warp` consecutive tokens; the sequence's coefficients stay in registers from
// one token to the next.  Four CTAs fit an SM, as the launch assumes (fp32, 8 values a lane: three
// without the bound, 13.8 -> 11.5 us for 32768 x 256).
template <typename T, int V, int VEC>
__global__ void __launch_bounds__(32 * kGateWarps, V <= 8 ? 4 : 1) balance_backward_kernel(LaunchBalance a, int per_warp) {
  const int lane = threadIdx.x & 31;
  const int experts = a.num_experts;
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kGateWarps + (threadIdx.x >> 5)) * per_warp;
  if (t0 >= a.tokens) return;
  const int64_t t1 = min(a.tokens, t0 + per_warp);
  const T *logits = static_cast<const T *>(a.logits);
  float l[V], w[V];
  load_row<T, V, VEC>(logits + t0 * experts, experts, lane, l);
  bool next_on = !a.token_mask || __ldg(a.token_mask + t0);
  int live = 0;  // sequences with tokens
  for (int64_t s = lane; s < a.num_seqs; s += 32) live += __ldg(a.seq_tokens + s) > 0;
  live = __reduce_add_sync(kAll, live);
  int64_t seq = 0, next_start = a.tokens;
  if (a.seq_offsets) {
    seq = find_sequence(a.seq_offsets, a.num_seqs, t0, lane);
    next_start = seq + 1 < a.num_seqs ? __ldg(a.seq_offsets + seq + 1) : a.tokens;
  }
  const float up = __ldg(a.d_loss) * a.alpha / static_cast<float>(live);
  int64_t loaded = -1;  // the sequence that w and n belong to
  int32_t n = 0;
  for (int64_t t = t0; t < t1; ++t) {
    while (t >= next_start && seq + 1 < a.num_seqs) {
      ++seq;
      next_start = seq + 1 < a.num_seqs ? __ldg(a.seq_offsets + seq + 1) : a.tokens;
    }
    if (seq != loaded) {
      n = __ldg(a.seq_tokens + seq);
      const float tn = static_cast<float>(n);
      const float c = n > 0 ? up * (static_cast<float>(experts) / (static_cast<float>(a.top_k) * tn)) / tn : 0.0f;
      // Counts above their mean: the same for all experts falls out of a_e - sum p a, and where every expert is chosen
      // (top_k = experts) nothing is left, not rounding noise.
      const int32_t mean = n / experts * a.top_k + n % experts * a.top_k / experts;  // of n top_k choices, in 32 bits
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int e = expert_of<VEC>(j, lane);
        w[j] = e < experts ? c * static_cast<float>(__ldg(a.counts + seq * experts + e) - mean) : 0.0f;
      }
      loaded = seq;
    }
    float cur[V];
#pragma unroll
    for (int j = 0; j < V; ++j) cur[j] = l[j];
    const bool on = next_on;
    if (t + 1 < t1) {
      load_row<T, V, VEC>(logits + (t + 1) * experts, experts, lane, l);
      next_on = !a.token_mask || __ldg(a.token_mask + t + 1);
    }
    T *out = static_cast<T *>(a.d_logits) + t * experts;
    if (!on || n <= 0) {
      if (!a.accumulate) {
#pragma unroll
        for (int j = 0; j < V; ++j) cur[j] = 0.0f;
        store_row<T, V, VEC>(out, experts, lane, cur);
      }
      continue;
    }
    float p[V], slope[V];
    probabilities<T, V, VEC>(cur, logits + t * experts, experts, lane, a.softmax, p, slope);
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) dot += p[j] * w[j];
    dot = warp_sum(dot);
    if (a.accumulate) {
      load_row<T, V, VEC>(out, experts, lane, cur);
#pragma unroll
      for (int j = 0; j < V; ++j) cur[j] += slope[j] * (w[j] - dot);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) cur[j] = slope[j] * (w[j] - dot);
    }
    store_row<T, V, VEC>(out, experts, lane, cur);
  }
}

// Calls f with the values a lane holds, V, and how many are neighbours: as many as fit a 16-byte
// load where the experts divide by it, else one.
template <typename T, typename F>
cudaError_t by_width(int experts, F f) {
  auto with = [&](auto v) {
    constexpr int V = decltype(v)::value;
    constexpr int kVec = V < 16 / static_cast<int>(sizeof(T)) ? V : 16 / static_cast<int>(sizeof(T));
    if (experts % kVec == 0) return f(v, std::integral_constant<int, kVec>{});
    return f(v, std::integral_constant<int, 1>{});
  };
  if (experts <= 32) return with(std::integral_constant<int, 1>{});
  if (experts <= 64) return with(std::integral_constant<int, 2>{});
  if (experts <= 128) return with(std::integral_constant<int, 4>{});
  if (experts <= 256) return with(std::integral_constant<int, 8>{});
  if (experts <= 512) return with(std::integral_constant<int, 16>{});
  return with(std::integral_constant<int, 32>{});
}

template <typename T>
cudaError_t gate(const LaunchGate &a) {
  const unsigned blocks = static_cast<unsigned>((a.tokens + kGateWarps - 1) / kGateWarps);
  return by_width<T>(a.num_experts, [&](auto v, auto vec) {
    gate_kernel<T, decltype(v)::value, decltype(vec)::value><<<blocks, 32 * kGateWarps, 0, a.stream>>>(
        static_cast<const T *>(a.logits), a.tokens, a.num_experts, a.top_k, a.softmax, a.normalize, a.scale, a.bias,
        a.ids, a.weights);
    return cudaGetLastError();
  });
}

template <typename T, int kWidth>
cudaError_t gate_backward(const LaunchGate &a) {
  const int64_t per = kGateWarps * (32 / kWidth);
  gate_backward_kernel<T, kWidth><<<static_cast<unsigned>((a.tokens + per - 1) / per), 32 * kGateWarps, 0, a.stream>>>(
      static_cast<const T *>(a.logits), a.ids, a.d_weights, a.tokens, a.num_experts, a.top_k, a.softmax, a.normalize,
      a.scale, static_cast<T *>(a.d_logits), a.status);
  return cudaGetLastError();
}

template <typename T>
cudaError_t gate_backward(const LaunchGate &a) {
  if (!a.softmax || a.normalize) {
    if (a.top_k <= 2) return gate_backward<T, 2>(a);
    if (a.top_k <= 4) return gate_backward<T, 4>(a);
    if (a.top_k <= 8) return gate_backward<T, 8>(a);
    if (a.top_k <= 16) return gate_backward<T, 16>(a);
    return gate_backward<T, 32>(a);
  }
  const unsigned blocks = static_cast<unsigned>((a.tokens + kGateWarps - 1) / kGateWarps);
  return by_width<T>(a.num_experts, [&](auto v, auto vec) {
    gate_backward_dense_kernel<T, decltype(v)::value, decltype(vec)::value>
        <<<blocks, 32 * kGateWarps, 0, a.stream>>>(static_cast<const T *>(a.logits), a.ids, a.d_weights, a.tokens,
                                                   a.num_experts, a.top_k, a.scale, static_cast<T *>(a.d_logits),
                                                   a.status);
    return cudaGetLastError();
  });
}

template <typename T>
cudaError_t balance_partial(const LaunchBalance &a) {
  const unsigned blocks = static_cast<unsigned>(a.tokens > 0 ? (a.tokens + a.chunk - 1) / a.chunk : 1);
  const size_t smem = static_cast<size_t>(kPartWarps / 2 + 1) * a.num_experts * 4;
  return by_width<T>(a.num_experts, [&](auto v, auto vec) {
    balance_partial_kernel<T, decltype(v)::value, decltype(vec)::value>
        <<<blocks, 32 * kPartWarps, smem, a.stream>>>(a);
    return cudaGetLastError();
  });
}

template <typename T>
cudaError_t balance_backward(const LaunchBalance &a) {
  // one wave: as many tokens a warp as 32 warps an SM leave (32768 x 256: 12.9 us; four a warp 13.7, two 15.8)
  const int64_t wave = 32 * static_cast<int64_t>(a.num_sms);
  const int per_warp = static_cast<int>((a.tokens + wave - 1) / wave);
  const int64_t warps = (a.tokens + per_warp - 1) / per_warp;
  const unsigned blocks = static_cast<unsigned>((warps + kGateWarps - 1) / kGateWarps);
  return by_width<T>(a.num_experts, [&](auto v, auto vec) {
    balance_backward_kernel<T, decltype(v)::value, decltype(vec)::value>
        <<<blocks, 32 * kGateWarps, 0, a.stream>>>(a, per_warp);
    return cudaGetLastError();
  });
}

}  // namespace

cudaError_t launch_gate(const LaunchGate &a) { return a.bf16 ? gate<__nv_bfloat16>(a) : gate<float>(a); }

cudaError_t launch_gate_backward(const LaunchGate &a) {
  return a.bf16 ? gate_backward<__nv_bfloat16>(a) : gate_backward<float>(a);
}

cudaError_t launch_balance_loss(const LaunchBalance &a) {
  cudaError_t err = a.bf16 ? balance_partial<__nv_bfloat16>(a) : balance_partial<float>(a);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.num_seqs * ((a.num_experts + 31) / 32)), 1, 1);
  cfg.blockDim = dim3(1024, 1, 1);
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, balance_final_kernel, a);
}

cudaError_t launch_balance_backward(const LaunchBalance &a) {
  return a.bf16 ? balance_backward<__nv_bfloat16>(a) : balance_backward<float>(a);
}

}  // namespace fme
