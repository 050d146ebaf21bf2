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
//   sigmoid, normalised   dl_i = (c g_i - sum_j (s_j / S) c g_j) / S  s_i (1 - s_i),  S = sum_j s_j
//   sigmoid               dl_i = c g_i s_i (1 - s_i)
//
// Balance loss.  p = softmax(l) or sigmoid(l) / Z.  Over the T_q counted tokens of each
// sequence q (empty ones left out, S of them are not):
//   L = alpha / S  sum_q  E / (K T_q^2)  sum_e count_qe  sum_t p_te
// The counts are constants to the gradient:
//   a_e = dL alpha / S  E / (K T_q^2) count_qe,   softmax: dl_e = p_e (a_e - sum_j p_j a_j),
//   sigmoid: dl_e = s_e (1 - s_e) / Z (a_e - sum_j p_j a_j).
//
// One warp a token, expert e in lane e % 32, so that loads are contiguous; all sums fp32.
// Reads the logits once: HBM-bound when there are many tokens, launch-bound when few.
#include "block128.cuh"

namespace fme {

namespace {

constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kGateWarps = 8;

__device__ __forceinline__ float load_logit(const float *p) { return __ldg(p); }
__device__ __forceinline__ float load_logit(const __nv_bfloat16 *p) { return __bfloat162float(__ldg(p)); }
__device__ __forceinline__ void store_grad(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_grad(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

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

__device__ __forceinline__ float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }

// Order of keys as unsigned integers: larger float, larger integer; -0 as +0; a NaN counts as
// the lowest.  0 is below every key (no expert here, or already taken).
__device__ __forceinline__ uint32_t order_key(float f) {
  if (f != f) return 1u;
  const uint32_t b = __float_as_uint(f + 0.0f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// exp(l - max) of a row held V values a lane; a row without a finite maximum gets zeros (all
// -inf: nothing is left of the row) or NaN (+inf or NaN among them).
template <int V>
__device__ __forceinline__ float exp_row(const float (&l)[V], float (&x)[V], int experts, int lane) {
  float m = -INFINITY, bad = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    m = fmaxf(m, l[j]);
    bad += l[j] == l[j] ? 0.0f : l[j];
  }
  m = warp_max(m);
  float sum = bad;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    x[j] = m == -INFINITY ? 0.0f : expf(l[j] - m);
    if (lane + 32 * j < experts) sum += x[j];
  }
  return warp_sum(sum);
}

template <typename T, int V>
__global__ void __launch_bounds__(32 * kGateWarps) gate_kernel(const T *__restrict__ logits, int64_t tokens,
                                                               int experts, int top_k, bool softmax, bool normalize,
                                                               float scale, const float *__restrict__ bias,
                                                               int32_t *__restrict__ ids,
                                                               float *__restrict__ weights) {
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kGateWarps + (threadIdx.x >> 5);
  if (t >= tokens) return;
  float l[V];
  uint32_t key[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = lane + 32 * j;
    l[j] = e < experts ? load_logit(logits + t * experts + e) : -INFINITY;
    key[j] = e < experts ? order_key(bias ? l[j] + __ldg(bias + e) : l[j]) : 0u;
  }
  float denom = 1.0f;  // softmax over all experts, only where the weights need it
  float m = 0.0f;
  if (softmax && !normalize) {
    float x[V];
    denom = exp_row<V>(l, x, experts, lane);
    m = -INFINITY;
#pragma unroll
    for (int j = 0; j < V; ++j) m = fmaxf(m, l[j]);
    m = warp_max(m);
  }
  int my_id = 0;
  float my_l = -INFINITY;
  for (int i = 0; i < top_k; ++i) {
    uint32_t best = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) best = max(best, key[j]);
    best = __reduce_max_sync(kAll, best);
    int at = INT32_MAX;
#pragma unroll
    for (int j = V - 1; j >= 0; --j)
      if (key[j] == best) at = lane + 32 * j;
    at = __reduce_min_sync(kAll, at);
    float lv = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (at == lane + 32 * j) {
        key[j] = 0;
        lv = l[j];
      }
    lv = __shfl_sync(kAll, lv, at & 31);
    if (lane == (i & 31)) {
      my_id = at;
      my_l = lv;
    }
  }
  // lane i holds choice i (top_k <= 32)
  const bool mine = lane < top_k;
  float s;
  if (softmax) {
    const float ref = normalize ? warp_max(mine ? my_l : -INFINITY) : m;
    s = !mine ? 0.0f : my_l != my_l ? my_l : ref == -INFINITY ? 0.0f : expf(my_l - ref);
  } else {
    s = mine ? sigmoid(my_l) : 0.0f;
  }
  if (normalize) denom = warp_sum(s);
  if (mine) {
    ids[t * top_k + lane] = my_id;
    weights[t * top_k + lane] = denom == 0.0f ? 0.0f : scale * s / denom;
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(32 * kGateWarps) gate_backward_kernel(
    const T *__restrict__ logits, const int32_t *__restrict__ ids, const float *__restrict__ d_weights, int64_t tokens,
    int experts, int top_k, bool softmax, bool normalize, float scale, T *__restrict__ d_logits, int32_t *status) {
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kGateWarps + (threadIdx.x >> 5);
  if (t >= tokens) return;
  const T *row = logits + t * experts;
  const bool mine = lane < top_k;
  int id = mine ? __ldg(ids + t * top_k + lane) : -1;
  if (mine && (id < 0 || id >= experts)) {
    report(status, kDevBadIndex);
    id = -1;
  }
  const bool live = id >= 0;
  const float g = live ? scale * __ldg(d_weights + t * top_k + lane) : 0.0f;
  const float my_l = live ? load_logit(row + id) : -INFINITY;
  float l[V], x[V];
  float d_mine, inner = 0.0f, denom = 1.0f;
  if (softmax && !normalize) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = lane + 32 * j;
      l[j] = e < experts ? load_logit(row + e) : -INFINITY;
    }
    denom = exp_row<V>(l, x, experts, lane);
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < V; ++j) m = fmaxf(m, l[j]);
    m = warp_max(m);
    const float p = !live ? 0.0f : denom == 0.0f ? 0.0f : expf(my_l - m) / denom;
    inner = warp_sum(p * g);
    d_mine = g;  // times p_e below
  } else if (softmax) {
    const float ref = warp_max(my_l);
    const float s = !live || ref == -INFINITY ? 0.0f : expf(my_l - ref);
    const float total = warp_sum(s);
    const float p = total == 0.0f ? 0.0f : s / total;
    d_mine = p * (g - warp_sum(p * g));
  } else {
    const float s = live ? sigmoid(my_l) : 0.0f;
    const float rest = live ? sigmoid(-my_l) : 0.0f;
    if (normalize) {
      const float total = warp_sum(s);
      const float mean = total == 0.0f ? 0.0f : warp_sum(s * g) / total;
      d_mine = total == 0.0f ? 0.0f : (g - mean) / total * s * rest;
    } else {
      d_mine = g * s * rest;
    }
  }
  float out[V];
#pragma unroll
  for (int j = 0; j < V; ++j) out[j] = 0.0f;
  for (int i = 0; i < top_k; ++i) {
    const int e = __shfl_sync(kAll, id, i);
    const float v = __shfl_sync(kAll, d_mine, i);
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (e == lane + 32 * j) out[j] = v;
  }
  if (softmax && !normalize) {
#pragma unroll
    for (int j = 0; j < V; ++j) out[j] = denom == 0.0f ? 0.0f : x[j] / denom * (out[j] - inner);
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = lane + 32 * j;
    if (e < experts) store_grad(d_logits + t * experts + e, out[j]);
  }
}

// ------------------------------------------------------------- balance loss --
// Probabilities of one token's row, V a lane; also s and 1 - s scaled for the gradient.
template <typename T, int V>
__device__ __forceinline__ void probabilities(const T *row, int experts, int lane, bool softmax, float (&p)[V],
                                              float (&slope)[V]) {
  float l[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = lane + 32 * j;
    l[j] = e < experts ? load_logit(row + e) : -INFINITY;
  }
  if (softmax) {
    const float z = exp_row<V>(l, p, experts, lane);
    const float r = z == 0.0f ? 0.0f : 1.0f / z;
#pragma unroll
    for (int j = 0; j < V; ++j) slope[j] = p[j] = p[j] * r;
  } else {
    float z = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      p[j] = lane + 32 * j < experts ? sigmoid(l[j]) : 0.0f;
      z += p[j];
    }
    z = warp_sum(z);
    const float r = z == 0.0f ? 0.0f : 1.0f / z;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      slope[j] = lane + 32 * j < experts ? p[j] * sigmoid(-l[j]) * r : 0.0f;
      p[j] *= r;
    }
  }
}

// One CTA for each (sequence, slice): sums of p and counts of the slice's counted tokens into
// the workspace, [sequence][slice][experts] each.  The order of every sum is fixed.
constexpr int kPartWarps = 16;

template <typename T, int V>
__global__ void __launch_bounds__(32 * kPartWarps) balance_partial_kernel(LaunchBalance a) {
  extern __shared__ float smem[];  // [kPartWarps / 2][experts] sums, then [experts] counts
  constexpr int kHalf = kPartWarps / 2;
  const int experts = a.num_experts;
  int32_t *cnt = reinterpret_cast<int32_t *>(smem + kHalf * experts);
  __shared__ int32_t n_tokens;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t seq = blockIdx.x / a.slices;
  const int slice = static_cast<int>(blockIdx.x - seq * a.slices);
  const int64_t lo = a.seq_offsets ? __ldg(a.seq_offsets + seq) : 0;
  const int64_t hi = a.seq_offsets ? __ldg(a.seq_offsets + seq + 1) : a.tokens;
  const bool bad = lo < 0 || hi < lo || hi > a.tokens || (seq == 0 && lo != 0) ||
                   (seq == a.num_seqs - 1 && hi != a.tokens);
  if (bad && threadIdx.x == 0) report(a.status, kDevBadOffsets);
  for (int e = threadIdx.x; e < experts; e += blockDim.x) cnt[e] = 0;
  if (threadIdx.x == 0) {
    n_tokens = 0;
    if (blockIdx.x == 0) *a.done = 0;  // of balance_final_kernel
  }
  __syncthreads();
  const int64_t per = (hi - lo + a.slices - 1) / a.slices;
  const int64_t t0 = lo + slice * per, t1 = bad ? t0 : min(hi, t0 + per);
  float sum[V];
#pragma unroll
  for (int j = 0; j < V; ++j) sum[j] = 0.0f;
  int mine = 0;
  for (int64_t t = t0 + warp; t < t1; t += kPartWarps) {
    if (a.token_mask && !__ldg(a.token_mask + t)) continue;
    float p[V], slope[V];
    probabilities<T, V>(static_cast<const T *>(a.logits) + t * experts, experts, lane, a.softmax, p, slope);
#pragma unroll
    for (int j = 0; j < V; ++j) sum[j] += p[j];
    ++mine;
    if (lane < a.top_k) {
      const int32_t e = __ldg(a.ids + t * a.top_k + lane);
      if (e >= 0 && e < experts)
        atomicAdd(&cnt[e], 1);
      else
        report(a.status, kDevBadIndex);
    }
  }
  if (lane == 0 && mine) atomicAdd(&n_tokens, mine);
  if (warp >= kHalf) {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (lane + 32 * j < experts) smem[(warp - kHalf) * experts + lane + 32 * j] = sum[j];
  }
  __syncthreads();
  if (warp < kHalf) {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (lane + 32 * j < experts) smem[warp * experts + lane + 32 * j] += sum[j];
  }
  __syncthreads();
  const int64_t at = static_cast<int64_t>(blockIdx.x) * experts;
  for (int e = threadIdx.x; e < experts; e += blockDim.x) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kHalf; ++w) v += smem[w * experts + e];
    a.part_sum[at + e] = v;
    a.part_count[at + e] = cnt[e];
  }
  if (threadIdx.x == 0) a.part_tokens[blockIdx.x] = n_tokens;
}

__device__ __forceinline__ float block_sum(float v, float *part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = warp_sum(v);
  __syncthreads();
  if (lane == 0) part[warp] = v;
  __syncthreads();
  return warp_sum(part[lane]);
}

// One CTA of 1024 threads a sequence: thread (part, e) adds every parts-th slice, the parts are
// added in order; then the sequence's term.  The last CTA to finish adds the terms.
__global__ void __launch_bounds__(1024) balance_final_kernel(LaunchBalance a) {
  __shared__ float sums[1024];
  __shared__ int32_t cnts[1024];
  __shared__ float red[32];
  __shared__ int last;
  __shared__ int32_t total_tokens;
  const int tid = threadIdx.x;
  const int experts = a.num_experts;
  const int width = (experts + 31) & ~31;
  const int parts = 1024 / width;
  const int64_t s = blockIdx.x;
  const int e = tid % width, part = tid / width;
  float v = 0.0f;
  int32_t c = 0;
  if (part < parts && e < experts) {
#pragma unroll 8
    for (int i = part; i < a.slices; i += parts) {
      const int64_t at = (s * a.slices + i) * experts + e;
      v += a.part_sum[at];
      c += a.part_count[at];
    }
  }
  sums[tid] = v;
  cnts[tid] = c;
  int32_t n = 0;
  for (int i = tid; i < a.slices; i += 1024) n += a.part_tokens[s * a.slices + i];
  if (tid == 0) total_tokens = 0;
  __syncthreads();
  if (n) atomicAdd(&total_tokens, n);
  float term = 0.0f;
  if (tid < experts) {
    v = 0.0f;
    c = 0;
    for (int i = 0; i < parts; ++i) {
      v += sums[i * width + tid];
      c += cnts[i * width + tid];
    }
    a.counts[s * experts + tid] = c;
    term = static_cast<float>(c) * v;
  }
  term = block_sum(term, red);
  if (tid == 0) {
    const int32_t t = total_tokens;
    const float tf = static_cast<float>(t);
    a.seq_tokens[s] = t;
    a.term[s] = t > 0 ? term / tf * (static_cast<float>(experts) / (static_cast<float>(a.top_k) * tf)) : 0.0f;
    __threadfence();
    last = atomicAdd(a.done, 1) == static_cast<int>(gridDim.x) - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  float all = 0.0f, live = 0.0f;
  for (int64_t i = tid; i < a.num_seqs; i += 1024) {
    all += __ldcg(a.term + i);
    live += __ldcg(a.seq_tokens + i) > 0 ? 1.0f : 0.0f;
  }
  all = block_sum(all, red);
  live = block_sum(live, red);
  if (tid == 0) a.loss[0] = live > 0.0f ? a.alpha * all / live : 0.0f;
}

template <typename T, int V>
__global__ void __launch_bounds__(32 * kGateWarps) balance_backward_kernel(LaunchBalance a) {
  const int lane = threadIdx.x & 31;
  const int experts = a.num_experts;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kGateWarps + (threadIdx.x >> 5);
  // sequences with tokens
  int live = 0;
  for (int64_t s = lane; s < a.num_seqs; s += 32) live += __ldg(a.seq_tokens + s) > 0;
  live = __reduce_add_sync(kAll, live);
  if (t >= a.tokens) return;
  int64_t seq = 0;
  if (a.seq_offsets) {  // the last sequence that starts at or before t
    int64_t lo = 0, hi = a.num_seqs;
    while (hi - lo > 1) {
      const int64_t mid = (lo + hi) >> 1;
      if (__ldg(a.seq_offsets + mid) <= t)
        lo = mid;
      else
        hi = mid;
    }
    seq = lo;
  }
  T *out = static_cast<T *>(a.d_logits) + t * experts;
  const bool on = !a.token_mask || __ldg(a.token_mask + t);
  const int32_t n = __ldg(a.seq_tokens + seq);
  if (!on || n <= 0) {
    if (!a.accumulate)
      for (int e = lane; e < experts; e += 32) store_grad(out + e, 0.0f);
    return;
  }
  const float tn = static_cast<float>(n);
  const float c = __ldg(a.d_loss) * a.alpha / static_cast<float>(live) *
                  (static_cast<float>(experts) / (static_cast<float>(a.top_k) * tn)) / tn;
  float p[V], slope[V], w[V];
  probabilities<T, V>(static_cast<const T *>(a.logits) + t * experts, experts, lane, a.softmax, p, slope);
  float dot = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = lane + 32 * j;
    w[j] = e < experts ? c * static_cast<float>(__ldg(a.counts + seq * experts + e)) : 0.0f;
    dot += p[j] * w[j];
  }
  dot = warp_sum(dot);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = lane + 32 * j;
    if (e >= experts) continue;
    float d = slope[j] * (w[j] - dot);
    if (a.accumulate) d += load_logit(out + e);
    store_grad(out + e, d);
  }
}

template <typename F>
cudaError_t by_width(int experts, F f) {
  if (experts <= 32) return f(std::integral_constant<int, 1>{});
  if (experts <= 64) return f(std::integral_constant<int, 2>{});
  if (experts <= 128) return f(std::integral_constant<int, 4>{});
  if (experts <= 256) return f(std::integral_constant<int, 8>{});
  if (experts <= 512) return f(std::integral_constant<int, 16>{});
  return f(std::integral_constant<int, 32>{});
}

}  // namespace

cudaError_t launch_gate(const LaunchGate &a) {
  const unsigned blocks = static_cast<unsigned>((a.tokens + kGateWarps - 1) / kGateWarps);
  return by_width(a.num_experts, [&](auto v) {
    constexpr int V = decltype(v)::value;
    if (a.bf16)
      gate_kernel<__nv_bfloat16, V><<<blocks, 32 * kGateWarps, 0, a.stream>>>(
          static_cast<const __nv_bfloat16 *>(a.logits), a.tokens, a.num_experts, a.top_k, a.softmax, a.normalize, a.scale,
          a.bias, a.ids, a.weights);
    else
      gate_kernel<float, V><<<blocks, 32 * kGateWarps, 0, a.stream>>>(static_cast<const float *>(a.logits), a.tokens,
                                                                     a.num_experts, a.top_k, a.softmax, a.normalize,
                                                                     a.scale, a.bias, a.ids, a.weights);
    return cudaGetLastError();
  });
}

cudaError_t launch_gate_backward(const LaunchGate &a) {
  const unsigned blocks = static_cast<unsigned>((a.tokens + kGateWarps - 1) / kGateWarps);
  return by_width(a.num_experts, [&](auto v) {
    constexpr int V = decltype(v)::value;
    if (a.bf16)
      gate_backward_kernel<__nv_bfloat16, V><<<blocks, 32 * kGateWarps, 0, a.stream>>>(
          static_cast<const __nv_bfloat16 *>(a.logits), a.ids, a.d_weights, a.tokens, a.num_experts, a.top_k, a.softmax,
          a.normalize, a.scale, static_cast<__nv_bfloat16 *>(a.d_logits), a.status);
    else
      gate_backward_kernel<float, V><<<blocks, 32 * kGateWarps, 0, a.stream>>>(
          static_cast<const float *>(a.logits), a.ids, a.d_weights, a.tokens, a.num_experts, a.top_k, a.softmax,
          a.normalize, a.scale, static_cast<float *>(a.d_logits), a.status);
    return cudaGetLastError();
  });
}

cudaError_t launch_balance_loss(const LaunchBalance &a) {
  const unsigned blocks = static_cast<unsigned>(a.num_seqs * a.slices);
  const size_t smem = static_cast<size_t>(kPartWarps / 2 + 1) * a.num_experts * 4;
  cudaError_t err = by_width(a.num_experts, [&](auto v) {
    constexpr int V = decltype(v)::value;
    if (a.bf16)
      balance_partial_kernel<__nv_bfloat16, V><<<blocks, 32 * kPartWarps, smem, a.stream>>>(a);
    else
      balance_partial_kernel<float, V><<<blocks, 32 * kPartWarps, smem, a.stream>>>(a);
    return cudaGetLastError();
  });
  if (err != cudaSuccess) return err;
  balance_final_kernel<<<static_cast<unsigned>(a.num_seqs), 1024, 0, a.stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_balance_backward(const LaunchBalance &a) {
  const unsigned blocks = static_cast<unsigned>((a.tokens + kGateWarps - 1) / kGateWarps);
  return by_width(a.num_experts, [&](auto v) {
    constexpr int V = decltype(v)::value;
    if (a.bf16)
      balance_backward_kernel<__nv_bfloat16, V><<<blocks, 32 * kGateWarps, 0, a.stream>>>(a);
    else
      balance_backward_kernel<float, V><<<blocks, 32 * kGateWarps, 0, a.stream>>>(a);
    return cudaGetLastError();
  });
}

}  // namespace fme
