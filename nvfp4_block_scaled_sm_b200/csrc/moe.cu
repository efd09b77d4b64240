// moe.cu -- routing of tokens to experts: scores, choice and weights (with
// their gradient), and the sort of the (token, choice) pairs by expert whose
// row offsets the grouped entry points take.
//
// Router. p = softmax(l) or sigmoid(l); an expert is chosen by p + bias, ties
// to the lowest index, among the experts of the best groups where groups are
// given (a group's score is the sum of its two best). One warp takes one
// token, lane i the experts i V .. i V + V - 1, all in registers: one read of
// the logits, no shared memory.
//
// The choice is that of the real numbers p + bias, not of their fp32 roundings
// (neighbouring scores are often closer than fp32's error, and the choice
// would then hang on the order of a sum). Without a bias the order of p is
// that of the logits, which are compared as they are. With one, keys are
// formed in fp32 with a bound on their error; a token whose choice some
// difference below that bound could turn takes the same steps again in fp64.
#include "common.cuh"

namespace mxq {
namespace {

constexpr int kMaxTopK = MXQ_ROUTE_MAX_TOP_K;
constexpr int kMaxGroups = MXQ_ROUTE_MAX_GROUPS;
constexpr int kSoftmax = MXQ_SCORE_SOFTMAX, kSigmoid = MXQ_SCORE_SIGMOID;

__device__ __forceinline__ float neg_inf() { return __uint_as_float(0xff800000u); }
__device__ __forceinline__ float pos_inf() { return __uint_as_float(0x7f800000u); }

// A logit as fp32; NaN counts as -inf, and -0 as +0.
__device__ __forceinline__ float clean(float v) { return v == v ? v + 0.f : neg_inf(); }
__device__ __forceinline__ float logit_at(const uint16_t* p, int64_t i) {
  return clean(__uint_as_float(uint32_t(p[i]) << 16));
}
__device__ __forceinline__ float logit_at(const float* p, int64_t i) { return clean(p[i]); }

// Unsigned order of fp32 values (0 is below every value).
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ uint64_t ordered(double v) {
  const uint64_t b = uint64_t(__double_as_longlong(v));
  return (b >> 63) ? ~b : b | (1ull << 63);
}
__device__ __forceinline__ double unordered(uint64_t k) {
  return __longlong_as_double(int64_t((k >> 63) ? k & ~(1ull << 63) : ~k));
}

__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(kFull, v); }
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
  const uint32_t hi = __reduce_max_sync(kFull, uint32_t(v >> 32));
  const uint32_t lo = __reduce_max_sync(kFull, uint32_t(v >> 32) == hi ? uint32_t(v) : 0u);
  return (uint64_t(hi) << 32) | lo;
}
template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

__device__ __forceinline__ float exp_of(float v) { return expf(v); }
__device__ __forceinline__ double exp_of(double v) { return exp(v); }

struct RouteArgs {
  const void* logits;
  const float* bias;
  float* weights;
  int32_t* experts;
  int64_t T, ld;
  int32_t E, top_k, groups, top_groups;
  int scoring, renormalize;
  float scale;
  int vector;               // rows can be read 16 bytes at a time
};

// e^(l - top) for the softmax, with equal infinities at distance 0.
template <typename F>
__device__ __forceinline__ F exp_from(F l, F top) { return l == top ? F(1) : exp_of(l - top); }

// The choice of one token: ordered keys of F's width (0: not there or left
// out) in key[V]; lane j gets the j-th chosen expert in *id. Returns the
// smallest difference of neighbouring keys among the chosen and the next one
// that is not an exact tie (same logit, same bias), +inf if there is none.
template <typename F, typename U, int V, bool GAPS>
__device__ __forceinline__ F choose(U (&key)[V], const float (&l)[V], const float* bias, int top_k, int lane,
                                    int* id) {
  U best = 0;
  int at = 0;
#pragma unroll
  for (int i = 0; i < V; i++)
    if (key[i] > best) { best = key[i]; at = i; }
  F gap = F(pos_inf()), last = 0;
  int last_id = -1;
  const int rounds = GAPS ? top_k + 1 : top_k;
  for (int j = 0; j < rounds; j++) {
    const U top = warp_max(best);
    if (top == 0) break;
    const int win = __ffs(__ballot_sync(kFull, best == top)) - 1;
    const int e = __shfl_sync(kFull, lane * V + at, win);
    if constexpr (GAPS) {
      const F v = unordered(top);
      if (j > 0) {
        // an exact tie has equal keys by construction; its order is the index
        F d = last - v;
        if (d == F(0)) {
          float mine = 0.f, other = 0.f;
#pragma unroll
          for (int i = 0; i < V; i++) {
            mine = lane * V + i == e ? l[i] : mine;
            other = lane * V + i == last_id ? l[i] : other;
          }
          mine = __shfl_sync(kFull, mine, e / V);
          other = __shfl_sync(kFull, other, last_id / V);
          if (mine == other && bias[e] == bias[last_id]) d = F(pos_inf());
        }
        gap = d < gap || d != d ? (d != d ? F(0) : d) : gap;
      }
      last = v;
      last_id = e;
    }
    if (j < top_k && lane == j) *id = e;
    if (lane == win) {
      best = 0;
#pragma unroll
      for (int i = 0; i < V; i++) {
        if (i == at) key[i] = 0;
      }
#pragma unroll
      for (int i = 0; i < V; i++)
        if (key[i] > best) { best = key[i]; at = i; }
    }
  }
  return gap;
}

// Leaves out (key 0) the experts of all but the best groups. Returns the
// difference between the last group kept and the first left out.
template <typename F, typename U, int V>
__device__ __forceinline__ F keep_groups(U (&key)[V], const F (&value)[V], int E, int groups, int top_groups,
                                         int lane) {
  const int size = E / groups;
  F score = F(neg_inf());                         // lane g: the score of group g
  auto two_best = [&](F& a, F& b, F v) {
    b = v > a ? a : (v > b ? v : b);
    a = v > a ? v : a;
  };
  const int lanes = size / V;
  if (size % V == 0 && (lanes & (lanes - 1)) == 0 && lanes <= 32) {
    // whole lanes make up a group: two best of the lane, then of its neighbours
    F a = F(neg_inf()), b = F(neg_inf());
#pragma unroll
    for (int i = 0; i < V; i++) two_best(a, b, value[i]);
    for (int o = 1; o < lanes; o <<= 1) {
      const F a2 = __shfl_xor_sync(kFull, a, o), b2 = __shfl_xor_sync(kFull, b, o);
      two_best(a, b, a2);
      two_best(a, b, b2);
    }
    const F mine = size == 1 ? a : a + b;
    score = __shfl_sync(kFull, mine, (lane * lanes) & 31);
  } else {
    for (int g = 0; g < groups; g++) {
      F a = F(neg_inf()), b = F(neg_inf());
#pragma unroll
      for (int i = 0; i < V; i++) {
        const int e = lane * V + i;
        if (e >= g * size && e < (g + 1) * size) two_best(a, b, value[i]);
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const F a2 = __shfl_xor_sync(kFull, a, o), b2 = __shfl_xor_sync(kFull, b, o);
        two_best(a, b, a2);
        two_best(a, b, b2);
      }
      if (lane == g) score = size == 1 ? a : a + b;
    }
  }
  if (score != score) score = F(neg_inf());
  U k = lane < groups ? ordered(score) : U(0);
  uint32_t kept = 0;
  F last = F(0);
  for (int j = 0; j < top_groups; j++) {
    const U top = warp_max(k);
    const int win = __ffs(__ballot_sync(kFull, k == top)) - 1;
    kept |= 1u << win;
    last = unordered(top);
    if (lane == win) k = 0;
  }
  const U next = warp_max(k);
  const F d = next == 0 ? F(pos_inf()) : last - unordered(next);
#pragma unroll
  for (int i = 0; i < V; i++) {
    const int e = lane * V + i;
    if (e < E && !(kept >> (e / size) & 1u)) key[i] = 0;
  }
  return d != d ? F(0) : d;
}

// Scores and keys of a token in F, and its choice. Returns false if the choice
// is in doubt at F's accuracy.
template <typename F, typename U, int V>
__device__ __forceinline__ bool route_token(const RouteArgs& a, const float (&l)[V], int lane, int* id) {
  F value[V];
  U key[V];
  const bool scores = a.bias || a.groups > 1;     // else the logits decide
  F sum = F(1);
  float top = neg_inf();
  if (scores && a.scoring == kSoftmax) {
#pragma unroll
    for (int i = 0; i < V; i++) top = fmaxf(top, l[i]);
    top = unordered(warp_max(ordered(top)));
    sum = F(0);
#pragma unroll
    for (int i = 0; i < V; i++)
      if (l[i] > neg_inf()) sum += exp_from(F(l[i]), F(top));
    sum = warp_sum(sum);
  }
  F most = F(0);                                  // the largest p + |bias|
#pragma unroll
  for (int i = 0; i < V; i++) {
    const int e = lane * V + i;
    F v = F(neg_inf());
    if (e < a.E) {
      if (!scores) {
        v = F(l[i]);
      } else {
        F p = F(0);
        if (l[i] > neg_inf())
          p = a.scoring == kSoftmax ? exp_from(F(l[i]), F(top)) / sum : F(1) / (F(1) + exp_of(-F(l[i])));
        const float b = a.bias ? a.bias[e] : 0.f;
        v = p + F(b);
        if (v != v) v = F(neg_inf());
        const F size = p + F(fabsf(b));
        if (size < F(pos_inf()) && size > most) most = size;
      }
    }
    value[i] = v;
    key[i] = e < a.E ? (v == F(0) ? ordered(F(0)) : ordered(v)) : U(0);
  }
  if (!scores) {
    choose<F, U, V, false>(key, l, nullptr, a.top_k, lane, id);
    return true;
  }
  F gap = F(pos_inf());
  if (a.groups > 1) gap = keep_groups<F, U, V>(key, value, a.E, a.groups, a.top_groups, lane);
  if (a.bias) {
    const F d = choose<F, U, V, true>(key, l, a.bias, a.top_k, lane, id);
    gap = d < gap ? d : gap;
  } else {
#pragma unroll
    for (int i = 0; i < V; i++)
      if (key[i]) key[i] = ordered(F(l[i]));      // the groups are known: the logits decide
    choose<F, U, V, false>(key, l, nullptr, a.top_k, lane, id);
  }
  if constexpr (sizeof(F) == 4) {
    // Error of a key: p to 8 roundings' size for the sigmoid (expf's two units
    // in the last place, the sum, the quotient, the addition of the bias);
    // for the softmax the exponent's rounding, at most 2^-24 in all, and the
    // sum's, (V + 5) roundings, besides. Keys differ by two errors, scores of
    // groups by four; twice that is asked for.
    const F most_all = unordered(warp_max(ordered(most)));
    const F unit = __uint_as_float(0x33800000u);  // 2^-24
    return gap > (a.scoring == kSoftmax ? F(8 * (V + 16)) : F(64)) * unit * most_all + 8 * unit;
  }
  return true;
}

template <typename T, int V>
__device__ __noinline__ void route_token_fp64(const RouteArgs& a, int64_t t, int lane, int* id) {
  float l[V];
#pragma unroll
  for (int i = 0; i < V; i++) {
    const int e = lane * V + i;
    l[i] = e < a.E ? logit_at(static_cast<const T*>(a.logits), t * a.ld + e) : neg_inf();
  }
  (void)route_token<double, uint64_t, V>(a, l, lane, id);
}

template <typename T, int V>
__device__ __forceinline__ void load_logits(const RouteArgs& a, int64_t t, int lane, float (&l)[V]) {
  const T* const row = static_cast<const T*>(a.logits) + t * a.ld;
  constexpr int kPer = 16 / sizeof(T);
  if (V % kPer == 0 && a.vector) {
#pragma unroll
    for (int i = 0; i < V / kPer; i++) {
      const int e = lane * V + i * kPer;
      uint4 q = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
      if (sizeof(T) == 4) q = make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u);
      if (e < a.E) q = ld_nc_v4(row + e);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int c = 0; c < kPer; c++)
        l[i * kPer + c] = clean(sizeof(T) == 4 ? __uint_as_float(w[c]) : (c & 1) ? bf16_hi(w[c >> 1]) : bf16_lo(w[c >> 1]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; i++) {
      const int e = lane * V + i;
      l[i] = e < a.E ? logit_at(row, e) : neg_inf();
    }
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) moe_route_kernel(const RouteArgs a) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int64_t step = int64_t(gridDim.x) * (kThreads / 32);
  for (int64_t t = int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); t < a.T; t += step) {
    float l[V];
    load_logits<T, V>(a, t, lane, l);
    int id = 0;
    if (!route_token<float, uint32_t, V>(a, l, lane, &id)) route_token_fp64<T, V>(a, t, lane, &id);

    // lane j holds the j-th choice
    const bool mine = lane < a.top_k;
    const float lj = mine ? logit_at(static_cast<const T*>(a.logits), t * a.ld + id) : neg_inf();
    float w = 0.f;
    if (a.scoring == kSoftmax) {
      // renormalized weights are the softmax of the chosen logits, whatever
      // the others are
      float top = lj;
      if (!a.renormalize) {
#pragma unroll
        for (int i = 0; i < V; i++) top = fmaxf(top, l[i]);
      }
      top = unordered(warp_max(ordered(top)));
      w = lj > neg_inf() ? exp_from(lj, top) : 0.f;
      float sum = w;
      if (!a.renormalize) {
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < V; i++)
          if (l[i] > neg_inf()) sum += exp_from(l[i], top);
      }
      sum = warp_sum(sum);
      w = sum > 0.f ? w / sum : 0.f;
    } else if (lj > neg_inf()) {
      w = 1.f / (1.f + expf(-lj));
    }
    if (a.scoring == kSigmoid && a.renormalize) {
      // where every chosen score is small, all are taken e^-top times larger
      // (their ratios stay, and none is lost below fp32's range)
      const float top = unordered(warp_max(ordered(lj)));
      if (top < 0.f && lj > neg_inf()) w = expf(lj - top) / (1.f + expf(lj));
      const float sum = warp_sum(w);
      w = sum > 0.f ? w / sum : 0.f;
    }
    if (mine) {
      a.weights[t * a.top_k + lane] = w * a.scale;
      a.experts[t * a.top_k + lane] = id;
    }
  }
}

// ---------------------------------------------------------------- gradient

// With q_j the score of choice j and g_j the gradient of its weight times the
// scale: weights q_j (renormalized: w_j = q_j / sum q) have
//   softmax                 dl_e = p_e (sum_{j chose e} g_j - sum_j g_j q_j)
//   softmax, renormalized   dl_e = sum_{j chose e} w_j (g_j - sum_i g_i w_i)
//   sigmoid                 dl_e = sum_{j chose e} g_j q_j (1 - q_j)
//   sigmoid, renormalized   dl_e = sum_{j chose e} w_j (g_j - sum_i g_i w_i) (1 - q_j)
// One warp per token; the choice itself has no gradient.
struct RouteGradArgs {
  RouteArgs r;
  const float* grad;
  const int32_t* chosen;
  void* out;
  int vector_out;
};

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) moe_route_backward_kernel(const RouteGradArgs b) {
  pdl_enter();
  const RouteArgs& a = b.r;
  const int lane = threadIdx.x & 31;
  const int64_t step = int64_t(gridDim.x) * (kThreads / 32);
  for (int64_t t = int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); t < a.T; t += step) {
    float l[V];
    load_logits<T, V>(a, t, lane, l);
    int id = -1;
    float g = 0.f, lj = neg_inf();
    if (lane < a.top_k) {
      id = b.chosen[t * a.top_k + lane];
      if (id < 0 || id >= a.E) id = -1;
      if (id >= 0) {
        g = b.grad[t * a.top_k + lane] * a.scale;
        lj = logit_at(static_cast<const T*>(a.logits), t * a.ld + id);
      }
    }
    const bool full = a.scoring == kSoftmax && !a.renormalize;   // every logit has a gradient
    float top = lj;
    if (full) {
#pragma unroll
      for (int i = 0; i < V; i++) top = fmaxf(top, l[i]);
    }
    top = unordered(warp_max(ordered(top)));
    float p[V], c = 0.f, minus = 0.f;                            // c: choice j's own part
    if (a.scoring == kSoftmax) {
      float q = lj > neg_inf() ? exp_from(lj, top) : 0.f;
      float sum = q;
      if (full) {
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < V; i++) {
          p[i] = l[i] > neg_inf() ? exp_from(l[i], top) : 0.f;
          sum += p[i];
        }
      }
      sum = warp_sum(sum);
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
      q *= inv;
      minus = warp_sum(g * q);
      if (full) {
#pragma unroll
        for (int i = 0; i < V; i++) p[i] *= inv;
        c = g;
      } else {
        c = q * (g - minus);
      }
    } else {
      const float q = 1.f / (1.f + expf(-lj)), other = 1.f / (1.f + expf(lj));   // p and 1 - p
      if (a.renormalize) {
        float w = lj > neg_inf() ? (top < 0.f ? expf(lj - top) * other : q) : 0.f;
        const float sum = warp_sum(w);
        w = sum > 0.f ? w / sum : 0.f;
        c = w * (g - warp_sum(g * w)) * other;
      } else {
        c = g * q * other;
      }
    }
    float d[V];
#pragma unroll
    for (int i = 0; i < V; i++) d[i] = 0.f;
    for (int j = 0; j < a.top_k; j++) {
      const int e = __shfl_sync(kFull, id, j);
      const float v = __shfl_sync(kFull, c, j);
      if (e >= 0 && e / V == lane) {
#pragma unroll
        for (int i = 0; i < V; i++)
          if (e % V == i) d[i] += v;
      }
    }
    if (full) {
#pragma unroll
      for (int i = 0; i < V; i++) d[i] = p[i] * (d[i] - minus);
    }
    T* const row = static_cast<T*>(b.out) + t * int64_t(a.E);
    constexpr int kPer = 16 / sizeof(T);
    if (V % kPer == 0 && b.vector_out) {
#pragma unroll
      for (int i = 0; i < V / kPer; i++) {
        const int e = lane * V + i * kPer;
        uint32_t w[4];
#pragma unroll
        for (int c4 = 0; c4 < 4; c4++) {
          if constexpr (sizeof(T) == 4) w[c4] = __float_as_uint(d[i * kPer + c4]);
          else w[c4] = cvt_bf16x2(d[(i * kPer + 2 * c4) % V], d[(i * kPer + 2 * c4 + 1) % V]);
        }
        if (e < a.E) st_v4(row + e, make_uint4(w[0], w[1], w[2], w[3]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; i++) {
        const int e = lane * V + i;
        if (e < a.E) {
          if constexpr (sizeof(T) == 4) row[e] = d[i];
          else row[e] = uint16_t(cvt_bf16x2(d[i], 0.f));
        }
      }
    }
  }
}

// ---------------------------------------------------------------- dispatch

// A stable counting sort of P expert ids into E buckets (and one for the ids
// outside [0, E)) by one cluster. Each of the cluster's warps takes a
// contiguous piece: it counts its ids (equal ids of 32 are found with
// match.any, so each bucket of the warp's own counters is added to by one
// lane), the counters become first places by a scan over the warps of a CTA,
// the CTAs of the cluster (through distributed shared memory) and the buckets,
// and a second walk over the piece hands the places out. No atomics: the order
// of equal ids is that of the pairs.
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortClusters = 8;

__global__ void __launch_bounds__(kSortThreads) moe_dispatch_kernel(const int32_t* experts, int64_t P, int E,
                                                                    int64_t* row_offsets, int32_t* order,
                                                                    int32_t* positions, uint32_t ctas,
                                                                    int64_t piece) {
  extern __shared__ uint32_t counts[];            // [kSortWarps][E + 1], then totals [E + 1]
  __shared__ uint32_t warp_totals[kSortWarps];
  pdl_enter();
  const int B = E + 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = blockIdx.x;
  uint32_t* const mine = counts + warp * B;
  uint32_t* const totals = counts + kSortWarps * B;
  for (int i = tid; i < kSortWarps * B; i += kSortThreads) counts[i] = 0;
  __syncthreads();

  const int64_t begin = min((int64_t(rank) * kSortWarps + warp) * piece, P);
  const int64_t end = min(begin + piece, P);
  auto bucket_at = [&](int64_t p) -> int {
    if (p >= end) return -1;
    const int e = experts[p];
    return e < 0 || e >= E ? E : e;
  };
  for (int64_t p0 = begin; p0 < end; p0 += 32) {
    const int b = bucket_at(p0 + lane);
    const uint32_t same = __match_any_sync(kFull, b);
    if (b >= 0 && lane == __ffs(same) - 1) mine[b] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  for (int b = tid; b < B; b += kSortThreads) {
    uint32_t at = 0;
    for (int w = 0; w < kSortWarps; w++) {
      const uint32_t n = counts[w * B + b];
      counts[w * B + b] = at;
      at += n;
    }
    totals[b] = at;
  }
  if (ctas > 1)
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
  else
    __syncthreads();

  // first place of each bucket in this CTA: the smaller buckets of every CTA,
  // and this bucket of the CTAs before
  const uint32_t totals_addr = static_cast<uint32_t>(__cvta_generic_to_shared(totals));
  uint32_t carry = 0;
  for (int b0 = 0; b0 < B; b0 += kSortThreads) {
    const int b = b0 + tid;
    uint32_t all = 0, before = 0;
    if (b < B) {
      for (uint32_t q = 0; q < ctas; q++) {
        uint32_t n;
        if (ctas == 1) {
          n = totals[b];
        } else {
          uint32_t addr;
          asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(totals_addr + b * 4), "r"(q));
          asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(n) : "r"(addr));
        }
        all += n;
        before += q < rank ? n : 0;
      }
    }
    uint32_t incl = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += up;
    }
    if (lane == 31) warp_totals[warp] = incl;
    __syncthreads();
    uint32_t first = carry + incl - all, sum = 0;
    for (int w = 0; w < kSortWarps; w++) {
      first += w < warp ? warp_totals[w] : 0;
      sum += warp_totals[w];
    }
    carry += sum;
    if (b < B) {
      if (rank == 0) row_offsets[b] = first;      // bucket E starts where expert E - 1 ends
      for (int w = 0; w < kSortWarps; w++) counts[w * B + b] += first + before;
    }
    __syncthreads();
  }

  for (int64_t p0 = begin; p0 < end; p0 += 32) {
    const int64_t p = p0 + lane;
    const int b = bucket_at(p);
    const uint32_t same = __match_any_sync(kFull, b);
    uint32_t at = 0;
    if (b >= 0) at = mine[b] + __popc(same & ((1u << lane) - 1));
    __syncwarp();
    if (b >= 0) {
      if (lane == __ffs(same) - 1) mine[b] += __popc(same);
      order[at] = int32_t(p);
      positions[p] = b == E ? -1 : int32_t(at);
    }
    __syncwarp();
  }
  if (ctas > 1)                                   // no CTA leaves while its totals are read
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// ------------------------------------------------------------------- host

template <typename Args, typename F>
mxq_status launch_tokens(F kernel, int64_t T, const Args& args, cudaStream_t stream) {
  const int64_t per = kThreads / 32;
  const int64_t grid = std::min<int64_t>((T + per - 1) / per, int64_t(sm_count()) * 16);
  return launched(launch_pdl(kernel, uint32_t(grid), stream, args));
}

template <typename T>
mxq_status launch_route(const RouteArgs& a, cudaStream_t s) {
  if (a.E <= 32) return launch_tokens(moe_route_kernel<T, 1>, a.T, a, s);
  if (a.E <= 64) return launch_tokens(moe_route_kernel<T, 2>, a.T, a, s);
  if (a.E <= 128) return launch_tokens(moe_route_kernel<T, 4>, a.T, a, s);
  if (a.E <= 256) return launch_tokens(moe_route_kernel<T, 8>, a.T, a, s);
  if (a.E <= 512) return launch_tokens(moe_route_kernel<T, 16>, a.T, a, s);
  return launch_tokens(moe_route_kernel<T, 32>, a.T, a, s);
}

template <typename T>
mxq_status launch_route_backward(const RouteGradArgs& b, cudaStream_t s) {
  const int32_t E = b.r.E;
  if (E <= 32) return launch_tokens(moe_route_backward_kernel<T, 1>, b.r.T, b, s);
  if (E <= 64) return launch_tokens(moe_route_backward_kernel<T, 2>, b.r.T, b, s);
  if (E <= 128) return launch_tokens(moe_route_backward_kernel<T, 4>, b.r.T, b, s);
  if (E <= 256) return launch_tokens(moe_route_backward_kernel<T, 8>, b.r.T, b, s);
  if (E <= 512) return launch_tokens(moe_route_backward_kernel<T, 16>, b.r.T, b, s);
  return launch_tokens(moe_route_backward_kernel<T, 32>, b.r.T, b, s);
}

mxq_status check_route(int dt, int64_t T, int32_t E, int64_t ld, int scoring, int32_t top_k, int32_t renormalize) {
  if (!valid_dtype(dt)) return MXQ_ERR_DTYPE;
  if (T < 0 || E < 1 || E > MXQ_GROUPED_MAX_EXPERTS || ld < E || top_k < 1 || top_k > E || top_k > kMaxTopK)
    return MXQ_ERR_SHAPE;
  if ((scoring != kSoftmax && scoring != kSigmoid) || (renormalize != 0 && renormalize != 1)) return MXQ_ERR_ARG;
  return MXQ_OK;
}

inline bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace
}  // namespace mxq

extern "C" {

mxq_status moe_route(const void* logits, int dt, int64_t T, int32_t E, int64_t ld, int scoring,
                     const float* bias, int32_t groups, int32_t top_groups, int32_t top_k, int32_t renormalize,
                     float scale, float* weights, int32_t* experts, mxq_stream_t stream) {
  using namespace mxq;
  const mxq_status st = check_route(dt, T, E, ld, scoring, top_k, renormalize);
  if (st != MXQ_OK) return st;
  if (groups < 1 || groups > kMaxGroups || E % groups != 0 || top_groups < 1 || top_groups > groups ||
      top_k > E / groups * top_groups)
    return MXQ_ERR_SHAPE;
  if (T == 0) return MXQ_OK;
  if (!logits || !weights || !experts) return MXQ_ERR_NULL;
  if (!aligned_to(logits, elem_size(dt)) || !aligned_to(bias, 4) || !aligned_to(weights, 4) ||
      !aligned_to(experts, 4))
    return MXQ_ERR_ALIGN;
  RouteArgs a{};
  a.logits = logits;
  a.bias = bias;
  a.weights = weights;
  a.experts = experts;
  a.T = T;
  a.ld = ld;
  a.E = E;
  a.top_k = top_k;
  a.groups = top_groups == groups ? 1 : groups;   // all groups kept: none to choose
  a.top_groups = top_groups;
  a.scoring = scoring;
  a.renormalize = renormalize;
  a.scale = scale;
  const int per = 16 / elem_size(dt);
  a.vector = aligned16(logits) && ld % per == 0 && E % per == 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dt == MXQ_BF16 ? launch_route<uint16_t>(a, s) : launch_route<float>(a, s);
}

mxq_status moe_route_backward(const float* grad_weights, const void* logits, int dt, int64_t T, int32_t E,
                              int64_t ld, const int32_t* experts, int scoring, int32_t top_k,
                              int32_t renormalize, float scale, void* grad_logits, mxq_stream_t stream) {
  using namespace mxq;
  const mxq_status st = check_route(dt, T, E, ld, scoring, top_k, renormalize);
  if (st != MXQ_OK) return st;
  if (T == 0) return MXQ_OK;
  if (!grad_weights || !logits || !experts || !grad_logits) return MXQ_ERR_NULL;
  if (!aligned_to(logits, elem_size(dt)) || !aligned_to(grad_logits, elem_size(dt)) ||
      !aligned_to(grad_weights, 4) || !aligned_to(experts, 4))
    return MXQ_ERR_ALIGN;
  RouteGradArgs b{};
  b.r.logits = logits;
  b.r.T = T;
  b.r.ld = ld;
  b.r.E = E;
  b.r.top_k = top_k;
  b.r.groups = b.r.top_groups = 1;
  b.r.scoring = scoring;
  b.r.renormalize = renormalize;
  b.r.scale = scale;
  const int per = 16 / elem_size(dt);
  b.r.vector = aligned16(logits) && ld % per == 0 && E % per == 0;
  b.vector_out = aligned16(grad_logits) && E % per == 0;
  b.grad = grad_weights;
  b.chosen = experts;
  b.out = grad_logits;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dt == MXQ_BF16 ? launch_route_backward<uint16_t>(b, s) : launch_route_backward<float>(b, s);
}

mxq_status moe_dispatch(const int32_t* experts, int64_t P, int32_t E, int64_t* row_offsets, int32_t* order,
                        int32_t* positions, mxq_stream_t stream) {
  using namespace mxq;
  if (P < 0 || P > 0x7fffffff || E < 1 || E > MXQ_GROUPED_MAX_EXPERTS) return MXQ_ERR_SHAPE;
  if (!row_offsets || (P > 0 && (!experts || !order || !positions))) return MXQ_ERR_NULL;
  if (!aligned_to(row_offsets, 8) || !aligned_to(experts, 4) || !aligned_to(order, 4) || !aligned_to(positions, 4))
    return MXQ_ERR_ALIGN;
  // at least four walks of 32 pairs for a warp before the next CTA pays for
  // the exchange
  uint32_t ctas = 1;
  while (ctas < uint32_t(kSortClusters) && P > int64_t(ctas) * kSortThreads * 4) ctas *= 2;
  const int64_t warps = int64_t(ctas) * kSortWarps;
  const int64_t piece = ((P + warps - 1) / warps + 31) / 32 * 32;
  const size_t smem = size_t(kSortWarps + 1) * size_t(E + 1) * 4;
  const cudaError_t attr_err =
      ensure_smem_limit<moe_dispatch_kernel>((kSortWarps + 1) * (MXQ_GROUPED_MAX_EXPERTS + 1) * 4);
  if (attr_err != cudaSuccess) {
    record_cuda_error(attr_err);
    return MXQ_ERR_CUDA;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return launched(cudaLaunchKernelEx(&cfg, moe_dispatch_kernel, experts, P, int(E), row_offsets, order, positions,
                                     ctas, piece));
}

}  // extern "C"
