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
// The choice is that of p + bias in fp64, not of its fp32 roundings (neighbouring
// scores are often closer than fp32's error, and the choice would then hang on
// the order of a sum). Without a bias the order of p is that of the logits, which
// are compared as they are. With one, keys are formed in fp32 with a bound on
// their error; a token whose choice some difference below that bound could turn
// takes the same steps again in fp64. So does a token with more than 32 keys
// above the bound of choose_quick: of random ones none at top_k = 8 of 64 to 1024
// or of 4 of 8 groups of 256, one in two thousand at 16 of 256, but most where the
// keys lie in few lanes or top_k is large (84 % at 16 of one group of two of 256,
// 92 % at 24 of 256, all at 32). 16384 tokens of 256 experts, sigmoid with a bias:
// 31 us at top_k = 8, 38 at 16, 86 at 16 of one group of two, 96 at 24, 116 at 32.
//
// Bound by instructions: 16384 tokens of 256 experts with a bias and 4 of 8
// groups take 34 us, 1090 instructions a token (0.5 TB/s of logits, where the
// read alone would take 2.8 us); choosing one expert a reduction, with full
// exponentials, took 2090 and 68 us.
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
  return b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
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

// Exponentials and reciprocals of the scores that a choice goes by: one
// instruction each in fp32 (their errors are in the bound on the keys), exact
// ones in fp64.
__device__ __forceinline__ float exp_of(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v * 1.4426950408889634f));
  return r;
}
__device__ __forceinline__ double exp_of(double v) { return exp(v); }
__device__ __forceinline__ float inverse(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ double inverse(double v) { return 1.0 / v; }
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ float smaller(float a, float b) { return fminf(a, b); }
__device__ __forceinline__ double larger(double a, double b) { return fmax(a, b); }
__device__ __forceinline__ double smaller(double a, double b) { return fmin(a, b); }

struct RouteArgs {
  const void* logits;
  const float* bias;
  float* weights;
  int32_t* experts;
  int64_t T, ld;
  int32_t E, top_k, groups, top_groups;
  int32_t group_size, group_lanes;   // experts of a group; lanes that hold just those, or 0
  int scoring, renormalize;
  float scale;
  int vector;               // rows can be read 16 bytes at a time
};

// e^(l - top) for the softmax, with equal infinities at distance 0.
template <typename F>
__device__ __forceinline__ F exp_from(F l, F top) { return l == top ? F(1) : exp_of(l - top); }
// The same for the weights and gradients.
__device__ __forceinline__ float weight_from(float l, float top) { return l == top ? 1.f : expf(l - top); }
// 1 / (1 + e^-l). Below -80 the 1 is far under e^-l's last bit, and e^-l soon has
// no fp32 value where e^l still has one.
__device__ __forceinline__ float sigmoid(float l) { return l < -80.f ? expf(l) : 1.f / (1.f + expf(-l)); }

// The choice of one token in fp64: ordered keys (0: not there or left out);
// lane j gets the j-th chosen expert in *id. One key a round.
template <int V>
__device__ __forceinline__ void choose(uint64_t (&key)[V], int top_k, int lane, int* id) {
  uint64_t best = 0;
  int at = 0;
#pragma unroll
  for (int i = 0; i < V; i++)
    if (key[i] > best) { best = key[i]; at = i; }
  for (int j = 0; j < top_k; j++) {
    const uint64_t top = warp_max(best);
    if (top == 0) break;
    const int win = __ffs(__ballot_sync(kFull, best == top)) - 1;
    const int e = __shfl_sync(kFull, lane * V + at, win);
    if (lane == j) *id = e;
    if (lane == win) {
      best = 0;
#pragma unroll
      for (int i = 0; i < V; i++)
        if (i == at) key[i] = 0;
#pragma unroll
      for (int i = 0; i < V; i++)
        if (key[i] > best) { best = key[i]; at = i; }
    }
  }
}

// The same in fp32, for `want` keys: the largest keys of the lanes give a bound
// that the want-th largest of all cannot be below; the few keys from there on
// (`list`, 32 words of this warp) are ranked against one another, one a lane.
// Lane j gets the j-th key and expert (key 0: there are fewer). Returns false,
// with nothing chosen, if more than 32 keys reach the bound.
template <int V>
__device__ __forceinline__ bool choose_quick(const uint32_t (&key)[V], int want, int lane, uint64_t* list,
                                             uint32_t* got, int* id) {
  uint32_t rest = key[0];
#pragma unroll
  for (int i = 1; i < V; i++) rest = max(rest, key[i]);
  uint32_t bound = 1;
  for (int j = 0; j < want; j++) {
    uint32_t top = warp_max(rest);
    if (top == 0 && bound > 1) {                  // every lane has given its largest: on to the next ones
#pragma unroll
      for (int i = 0; i < V; i++) rest = max(rest, key[i] < bound ? key[i] : 0u);
      top = warp_max(rest);
    }
    if (top == 0) {                               // fewer keys than wanted: all count
      bound = 1;
      break;
    }
    bound = top;
    rest = rest == top ? 0 : rest;
  }
  int n = 0;
  const uint32_t before = (1u << lane) - 1;
#pragma unroll
  for (int i = 0; i < V; i++) {
    const uint32_t m = __ballot_sync(kFull, key[i] >= bound);
    const int at = n + __popc(m & before);
    if (key[i] >= bound && at < 32) list[at] = (uint64_t(key[i]) << 32) | uint32_t(~(lane * V + i));
    n += __popc(m);
  }
  if (n > 32) return false;
  __syncwarp();
  const uint64_t mine = lane < n ? list[lane] : 0;   // the lower index is the larger of equal keys
  if (lane >= n && lane < ((n + 3) & ~3)) list[lane] = 0;
  __syncwarp();
  int rank = 0;
  for (int j = 0; j < n; j += 4) {
#pragma unroll
    for (int q = 0; q < 4; q++) rank += list[j + q] > mine ? 1 : 0;
  }
  __syncwarp();
  if (lane < n) list[rank] = mine;
  __syncwarp();
  const uint64_t chosen = lane < n ? list[lane] : 0;
  __syncwarp();
  *got = uint32_t(chosen >> 32);
  *id = lane < n ? int(~uint32_t(chosen)) : 0;
  return true;
}

// Leaves out (key 0) the experts of all but the best groups. Returns the
// difference between the last group kept and the first left out.
template <typename F, typename U, int V>
__device__ __forceinline__ F keep_groups(U (&key)[V], const F (&value)[V], const RouteArgs& a, int lane) {
  const int size = a.group_size, lanes = a.group_lanes;
  auto two_best = [&](F& x, F& y, F v) {
    y = larger(y, smaller(x, v));
    x = larger(x, v);
  };
  F score = F(neg_inf());
  int g = lane;                                   // the group whose score this lane holds
  bool holds = lane < a.groups;
  if (lanes > 0) {
    // whole lanes make up a group: two best of the lane, then of its neighbours
    F x = F(neg_inf()), y = F(neg_inf());
#pragma unroll
    for (int i = 0; i < V; i++) two_best(x, y, value[i]);
    for (int o = 1; o < lanes; o <<= 1) {
      const F x2 = __shfl_xor_sync(kFull, x, o), y2 = __shfl_xor_sync(kFull, y, o);
      y = larger(larger(y, y2), smaller(x, x2));
      x = larger(x, x2);
    }
    score = size == 1 ? x : x + y;
    holds = lane * V < a.E;                       // every lane of the group holds it
    g = lane;
  } else {
    for (int q = 0; q < a.groups; q++) {
      F x = F(neg_inf()), y = F(neg_inf());
#pragma unroll
      for (int i = 0; i < V; i++) {
        const int e = lane * V + i;
        if (e >= q * size && e < (q + 1) * size) two_best(x, y, value[i]);
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const F x2 = __shfl_xor_sync(kFull, x, o), y2 = __shfl_xor_sync(kFull, y, o);
        y = larger(larger(y, y2), smaller(x, x2));
        x = larger(x, x2);
      }
      if (lane == q) score = size == 1 ? x : x + y;
    }
  }
  if (score != score) score = F(neg_inf());
  U k = holds ? ordered(score) : U(0);
  uint32_t kept = 0;                              // lanes of the groups kept
  U last = 0;
  for (int j = 0; j < a.top_groups; j++) {
    const U top = warp_max(k);
    uint32_t win = __ballot_sync(kFull, k == top);
    win &= ~win + 1;                              // the lowest of equal scores
    if (lanes > 1) win *= (lanes >= 32 ? ~0u : (1u << lanes) - 1);   // all lanes of its group
    kept |= win;
    last = top;
    if (win >> g & 1u) k = 0;
  }
  const U next = warp_max(k);
  const F d = next == 0 ? F(pos_inf()) : unordered(last) - unordered(next);
  if (lanes > 0) {
    const bool out = !(kept >> lane & 1u);
#pragma unroll
    for (int i = 0; i < V; i++) key[i] = out ? 0 : key[i];
  } else {
    int q = lane * V / size, end = (q + 1) * size;   // the group of the lane's next expert, and where it ends
#pragma unroll
    for (int i = 0; i < V; i++) {
      const int e = lane * V + i;
      if (e >= end) {                             // (size >= 1: one step is enough)
        q++;
        end += size;
      }
      if (e < a.E && !(kept >> (q & 31) & 1u)) key[i] = 0;
    }
  }
  return d != d ? F(0) : d;
}

// Scores and keys of a token in F, and its choice, with the lane's biases.
// Returns false if the choice is in doubt at F's accuracy.
template <typename F, typename U, typename T, int V>
__device__ __forceinline__ bool route_token(const RouteArgs& a, const T* row, const float (&l)[V],
                                            const float (&bias)[V], float most_bias, int lane, uint64_t* list,
                                            int* id) {
  U key[V];
  F gap = F(pos_inf());
  F most = F(most_bias);                          // bound on p + |bias|
  if (a.bias || a.groups > 1) {
    F value[V];
    if (a.scoring == kSoftmax) {
      float top = neg_inf();
#pragma unroll
      for (int i = 0; i < V; i++) top = fmaxf(top, l[i]);
      top = unordered(warp_max(ordered(top)));
      F sum = F(0);
#pragma unroll
      for (int i = 0; i < V; i++) {
        value[i] = lane * V + i < a.E ? exp_from(F(l[i]), F(top)) : F(0);
        sum += value[i];
      }
      sum = warp_sum(sum);
      const F inv = top > neg_inf() ? inverse(sum) : F(0);   // (a row of -inf has no scores)
      most += inv;
#pragma unroll
      for (int i = 0; i < V; i++) value[i] *= inv;
    } else {
      most += F(1);
#pragma unroll
      for (int i = 0; i < V; i++) value[i] = inverse(F(1) + exp_of(-F(l[i])));
    }
#pragma unroll
    for (int i = 0; i < V; i++) {
      const bool there = lane * V + i < a.E;
      value[i] = there ? value[i] + F(bias[i]) : F(neg_inf());
      key[i] = there ? ordered(value[i]) : U(0);
    }
    if (a.groups > 1) gap = keep_groups<F, U, V>(key, value, a, lane);
  }
  if (!a.bias) {                                  // the logits decide among the groups that are kept
#pragma unroll
    for (int i = 0; i < V; i++) {
      const bool there = a.groups > 1 ? key[i] != 0 : lane * V + i < a.E;
      key[i] = there ? ordered(F(l[i])) : U(0);
    }
  }
  if constexpr (sizeof(F) == 8) {
    choose(key, a.top_k, lane, id);
    return true;
  } else {
    uint32_t got;
    if (!choose_quick(key, a.bias ? a.top_k + 1 : a.top_k, lane, list, &got, id)) return false;
    if (a.bias) {
      // neighbours in the order of the keys: an exact tie (same logit, same
      // bias) is in order as it is, any other difference has to be clear
      const float mine = logit_at(row, *id), b = a.bias[*id];
      const float next_l = __shfl_down_sync(kFull, mine, 1), next_b = __shfl_down_sync(kFull, b, 1);
      const uint32_t next = __shfl_down_sync(kFull, got, 1);
      if (lane < a.top_k && lane < 31 && next != 0 && !(mine == next_l && b == next_b)) {
        const float d = unordered(got) - unordered(next);
        gap = d < gap ? d : d == d ? gap : 0.f;
      }
      if (a.top_k == 32 && a.E > 32) gap = 0.f;   // the 33rd has no lane
    }
    if (a.bias || a.groups > 1) {
      // Error of a key, in units of 2^-24 of p + |bias|: for the sigmoid 2 for
      // the exponential, at most 1 for the rounding of its argument after the
      // factor p (1 - p), 1 for the sum, 2 for the reciprocal, 1 for the bias:
      // below 8. For the softmax 2 for the exponential, at most 2 for its
      // argument's two roundings after the factor p, V + 5 for the sum, 2 for
      // the reciprocal, 1 for the product, 1 for the bias: below V + 16. Keys
      // differ by two errors, scores of groups by four and two additions;
      // twice that is asked for.
      const float unit = __uint_as_float(0x33800000u);   // 2^-24
      return __all_sync(kFull, gap > (a.scoring == kSoftmax ? float(8 * (V + 16)) : 80.f) * unit * most + 8 * unit);
    }
    return true;
  }
}

// The lane's biases (NaN as -inf, 0 without a bias); returns the largest
// finite magnitude of all.
template <int V>
__device__ __forceinline__ float load_bias(const RouteArgs& a, int lane, float (&bias)[V]) {
  float most = 0.f;
#pragma unroll
  for (int i = 0; i < V; i++) {
    const int e = lane * V + i;
    bias[i] = a.bias && e < a.E ? a.bias[e] : 0.f;
    if (bias[i] != bias[i]) bias[i] = neg_inf();
    const float m = fabsf(bias[i]);
    most = fmaxf(most, m < pos_inf() ? m : 0.f);
  }
  return __uint_as_float(warp_max(__float_as_uint(most)));
}

template <typename T, int V>
__device__ __noinline__ int route_token_fp64(const RouteArgs& a, const T* row, int lane) {
  float l[V], bias[V];
#pragma unroll
  for (int i = 0; i < V; i++) {
    const int e = lane * V + i;
    l[i] = e < a.E ? logit_at(row, e) : neg_inf();
  }
  const float most = load_bias(a, lane, bias);
  int id = 0;
  (void)route_token<double, uint64_t, T, V>(a, row, l, bias, most, lane, nullptr, &id);
  return id;
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
__global__ void __launch_bounds__(kThreads, V <= 4 ? 4 : V <= 8 ? 3 : 2) moe_route_kernel(const RouteArgs a) {
  __shared__ uint64_t lists[kThreads / 32][32];
  pdl_enter();
  const int lane = threadIdx.x & 31;
  float bias[V];
  const float most_bias = load_bias(a, lane, bias);
  const int64_t step = int64_t(gridDim.x) * (kThreads / 32);
  for (int64_t t = int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); t < a.T; t += step) {
    const T* const row = static_cast<const T*>(a.logits) + t * a.ld;
    int id = 0;
    float top = 0.f, sum = 0.f;                   // of the whole row's softmax, where the weights need them
    {
      float l[V];
      load_logits<T, V>(a, t, lane, l);
      if (a.scoring == kSoftmax && !a.renormalize) {
        top = neg_inf();
#pragma unroll
        for (int i = 0; i < V; i++) top = fmaxf(top, l[i]);
        top = unordered(warp_max(ordered(top)));
#pragma unroll
        for (int i = 0; i < V; i++)
          if (l[i] > neg_inf()) sum += weight_from(l[i], top);
        sum = warp_sum(sum);
      }
      if (!route_token<float, uint32_t, T, V>(a, row, l, bias, most_bias, lane, lists[threadIdx.x >> 5], &id))
        id = route_token_fp64<T, V>(a, row, lane);
    }

    // lane j holds the j-th choice
    const bool mine = lane < a.top_k;
    const float lj = mine ? logit_at(row, id) : neg_inf();
    float w = 0.f;
    if (a.scoring == kSoftmax) {
      if (a.renormalize) top = unordered(warp_max(ordered(lj)));
      w = lj > neg_inf() ? weight_from(lj, top) : 0.f;
      // renormalized weights are the softmax of the chosen logits, whatever
      // the others are
      if (a.renormalize) sum = warp_sum(w);
      w = sum > 0.f ? w / sum : 0.f;
    } else if (lj > neg_inf()) {
      w = sigmoid(lj);
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
// One warp per token, the choices' parts joined to the experts' through shared
// memory (a walk over the choices in registers took 17.5 us for 15); the choice
// itself has no gradient. 16384 x 256 fp32: 13.6 us from memory (2.5 TB/s), 11.4
// where L2 holds the logits. Only the plain softmax needs the whole row; the
// other forms read it too (11.8 to 13.2 us).
struct RouteGradArgs {
  RouteArgs r;
  const float* grad;
  const int32_t* chosen;
  void* out;
  int vector_out;
};

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) moe_route_backward_kernel(const RouteGradArgs b) {
  __shared__ __align__(16) float rows[kThreads / 32][32 * V];
  pdl_enter();
  const RouteArgs& a = b.r;
  const int lane = threadIdx.x & 31;
  float* const mine = rows[threadIdx.x >> 5];     // the choices' parts, by expert
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
      float q = lj > neg_inf() ? weight_from(lj, top) : 0.f;
      float sum = q;
      if (full) {
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < V; i++) {
          p[i] = l[i] > neg_inf() ? weight_from(l[i], top) : 0.f;
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
      const float q = sigmoid(lj), other = sigmoid(-lj);         // p and 1 - p
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
    for (int i = 0; i < V; i++) mine[lane * V + i] = 0.f;
    __syncwarp();
    // one store a choice; where an expert is named twice, one choice after
    // another (the same sum every run)
    const uint32_t same = __match_any_sync(kFull, id < 0 ? -1 - lane : id);
    if (__all_sync(kFull, same == 1u << lane)) {
      if (id >= 0) mine[id] = c;
    } else {
      for (int j = 0; j < a.top_k; j++) {
        if (lane == j && id >= 0) mine[id] += c;
        __syncwarp();
      }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < V; i++) d[i] = mine[lane * V + i];
    __syncwarp();
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
// outside [0, E)). Up to 4096 ids one CTA does all of it; more are cut into
// chunks, one a CTA: a first kernel ranks each id among its chunk's and counts
// the chunk's buckets, a second adds up the counts of the chunks before and
// places the ids (131072 pairs of 256 experts on one cluster of 8 CTAs with
// the counts in distributed shared memory took 24 us, in two kernels 11.4).
//
// Inside a CTA each warp takes a contiguous piece, 32 ids a walk: lanes with
// the same id are found by a vote for each bit of it (11 votes at most;
// match.any made the walks half as fast), and an id's rank among its warp's is
// the warp's counter of its bucket plus the equal ids of the lanes before. The
// counters then become first places by a scan over the warps. No atomics: the
// order of equal ids is that of the pairs.
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortAhead = 4;              // walks whose ids are read together
constexpr int64_t kSortChunk = 32 * kSortWarps * kSortAhead;
constexpr int64_t kSortChunks = 128;       // at most; the second kernel reads all their counts

// Ids of a chunk (a multiple of 32 for each warp).
inline int64_t sort_chunk(int64_t P) {
  const int64_t per = (P + kSortChunks - 1) / kSortChunks;
  return std::max(kSortChunk, (per + kSortThreads - 1) / kSortThreads * kSortThreads);
}

// Exclusive sum over buckets b0 + threadIdx.x of `n`, on top of *carry, which
// goes on by the sum of all. `warp_totals`: kSortWarps words.
__device__ __forceinline__ uint32_t block_first(uint32_t n, uint32_t* warp_totals, uint32_t* carry) {
  static_assert(kSortWarps == 32, "one lane a warp below");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t incl = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t up = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) warp_totals[warp] = incl;
  __syncthreads();
  const uint32_t own = warp_totals[lane];
  uint32_t sum = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t up = __shfl_up_sync(kFull, sum, o);
    if (lane >= o) sum += up;
  }
  const uint32_t first = *carry + __shfl_sync(kFull, sum - own, warp) + incl - n;
  *carry += __shfl_sync(kFull, sum, 31);
  __syncthreads();
  return first;
}

// ONE: the whole sort; otherwise ranks within the chunk into `positions` and
// the chunk's counts into `chunk_counts` [chunks][E + 1].
template <bool ONE>
__global__ void __launch_bounds__(kSortThreads) moe_dispatch_kernel(const int32_t* experts, int64_t P, int E,
                                                                    int64_t chunk, int64_t* row_offsets,
                                                                    int32_t* order, int32_t* positions,
                                                                    uint32_t* chunk_counts) {
  extern __shared__ uint32_t counts[];            // [kSortWarps][E + 1], then places [E + 1]
  __shared__ uint32_t warp_totals[kSortWarps];
  pdl_enter();
  const int B = E + 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t* const mine = counts + warp * B;
  uint32_t* const places = counts + kSortWarps * B;
  const int64_t piece = chunk / kSortWarps;
  const int64_t begin = min(int64_t(blockIdx.x) * chunk + warp * piece, P);
  const int64_t end = min(begin + piece, P);
  const int bits = 32 - __clz(B);

  int id[kSortAhead];                             // B past the end
  uint32_t rank[kSortAhead];
  auto read = [&](int64_t p0) {
#pragma unroll
    for (int q = 0; q < kSortAhead; q++) {
      const int64_t p = p0 + q * 32 + lane;
      int e = B;
      if (p < end) {
        e = experts[p];
        e = e < 0 || e >= E ? E : e;
      }
      id[q] = e;
    }
  };
  auto count = [&](int64_t p0) {
#pragma unroll
    for (int q = 0; q < kSortAhead; q++) {
      if (p0 + q * 32 >= end) break;
      const int b = id[q];
      uint32_t same = kFull;
      for (int i = 0; i < bits; i++) {
        const bool set = b >> i & 1;
        const uint32_t m = __ballot_sync(kFull, set);
        same &= set ? m : ~m;
      }
      const uint32_t n = b < B ? mine[b] : 0;
      __syncwarp();
      if (b < B && lane == __ffs(same) - 1) mine[b] = n + __popc(same);
      rank[q] = n + __popc(same & ((1u << lane) - 1));
      __syncwarp();
    }
  };
  const bool once = piece <= 32 * kSortAhead;     // all ids and ranks of a warp stay in registers
  read(begin);
  for (int i = tid; i < kSortWarps * B; i += kSortThreads) counts[i] = 0;
  __syncthreads();
  for (int64_t p0 = begin; p0 < end; p0 += 32 * kSortAhead) {
    if (p0 > begin) read(p0);
    count(p0);
  }
  __syncthreads();

  // counters become the warps' first ranks of each bucket
  uint32_t carry = 0;
  for (int b0 = 0; b0 < B; b0 += kSortThreads) {
    const int b = b0 + tid;
    uint32_t at = 0;
    if (b < B) {
      uint32_t n[kSortWarps];
#pragma unroll
      for (int w = 0; w < kSortWarps; w++) n[w] = counts[w * B + b];
#pragma unroll
      for (int w = 0; w < kSortWarps; w++) {
        counts[w * B + b] = at;
        at += n[w];
      }
      if constexpr (!ONE) chunk_counts[int64_t(blockIdx.x) * B + b] = at;
    }
    if constexpr (ONE) {
      const uint32_t first = block_first(at, warp_totals, &carry);
      if (b < B) {
        row_offsets[b] = first;                   // bucket E starts where expert E - 1 ends
        places[b] = first;
      }
    }
  }
  __syncthreads();

  // (a second walk, where there is one, counts on from the first ranks)
  for (int64_t p0 = begin; p0 < end; p0 += 32 * kSortAhead) {
    if (!once) {
      read(p0);
      count(p0);
    }
#pragma unroll
    for (int q = 0; q < kSortAhead; q++) {
      const int64_t p = p0 + q * 32 + lane;
      if (p >= end) break;
      const int b = id[q];
      const uint32_t at = rank[q] + (once ? mine[b] : 0u);
      if constexpr (ONE) {
        order[places[b] + at] = int32_t(p);
        positions[p] = b == E ? -1 : int32_t(places[b] + at);
      } else {
        positions[p] = int32_t(at);
      }
    }
  }
}

__global__ void __launch_bounds__(kSortThreads) moe_dispatch_place_kernel(const int32_t* experts, int64_t P, int E,
                                                                          int64_t chunk, int chunks,
                                                                          int64_t* row_offsets, int32_t* order,
                                                                          int32_t* positions,
                                                                          const uint32_t* chunk_counts) {
  __shared__ uint32_t places[MXQ_GROUPED_MAX_EXPERTS + 1];
  __shared__ uint32_t warp_totals[kSortWarps];
  pdl_enter();
  const int B = E + 1, own = blockIdx.x;
  uint32_t carry = 0;
  for (int b0 = 0; b0 < B; b0 += kSortThreads) {
    const int b = b0 + threadIdx.x;
    uint32_t all = 0, before = 0;
    if (b < B) {
#pragma unroll 16
      for (int q = 0; q < chunks; q++) {
        const uint32_t n = chunk_counts[int64_t(q) * B + b];
        all += n;
        before += q < own ? n : 0;
      }
    }
    const uint32_t first = block_first(all, warp_totals, &carry);
    if (b < B) {
      places[b] = first + before;
      if (own == 0) row_offsets[b] = first;
    }
  }
  __syncthreads();
  const int64_t begin = int64_t(own) * chunk, end = min(begin + chunk, P);
#pragma unroll 4
  for (int64_t p = begin + threadIdx.x; p < end; p += kSortThreads) {
    int b = experts[p];
    b = b < 0 || b >= E ? E : b;
    const uint32_t at = places[b] + uint32_t(positions[p]);
    order[at] = int32_t(p);
    positions[p] = b == E ? -1 : int32_t(at);
  }
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
  a.group_size = E / a.groups;
  int V = 1;                                      // experts of a lane
  while (32 * V < E) V *= 2;
  a.group_lanes = a.group_size % V == 0 && ((a.group_size / V) & (a.group_size / V - 1)) == 0 ? a.group_size / V : 0;
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

size_t mxq_moe_dispatch_workspace_bytes(int64_t P, int32_t E) {
  using namespace mxq;
  if (P < 0 || P > 0x7fffffff || E < 1 || E > MXQ_GROUPED_MAX_EXPERTS) return 0;
  const int64_t chunk = sort_chunk(P), chunks = (P + chunk - 1) / chunk;
  return chunks <= 1 ? 0 : size_t(chunks) * size_t(E + 1) * 4;
}

mxq_status moe_dispatch(const int32_t* experts, int64_t P, int32_t E, int64_t* row_offsets, int32_t* order,
                        int32_t* positions, void* workspace, size_t ws_bytes, mxq_stream_t stream) {
  using namespace mxq;
  if (P < 0 || P > 0x7fffffff || E < 1 || E > MXQ_GROUPED_MAX_EXPERTS) return MXQ_ERR_SHAPE;
  if (!row_offsets || (P > 0 && (!experts || !order || !positions))) return MXQ_ERR_NULL;
  if (!aligned_to(row_offsets, 8) || !aligned_to(experts, 4) || !aligned_to(order, 4) || !aligned_to(positions, 4))
    return MXQ_ERR_ALIGN;
  const size_t need = mxq_moe_dispatch_workspace_bytes(P, E);
  if (need > 0 && (!workspace || ws_bytes < need)) return MXQ_ERR_WORKSPACE;
  if (need > 0 && !aligned_to(workspace, 4)) return MXQ_ERR_ALIGN;
  const int64_t chunk = sort_chunk(P);
  const uint32_t chunks = uint32_t(std::max<int64_t>(1, (P + chunk - 1) / chunk));
  const size_t smem = size_t(kSortWarps + 1) * size_t(E + 1) * 4;
  constexpr int kMost = (kSortWarps + 1) * (MXQ_GROUPED_MAX_EXPERTS + 1) * 4;
  cudaError_t attr_err = ensure_smem_limit<moe_dispatch_kernel<true>>(kMost);
  if (attr_err == cudaSuccess) attr_err = ensure_smem_limit<moe_dispatch_kernel<false>>(kMost);
  if (attr_err != cudaSuccess) {
    record_cuda_error(attr_err);
    return MXQ_ERR_CUDA;
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint32_t* const counts = static_cast<uint32_t*>(workspace);
  if (chunks == 1)
    return launched(launch_pdl_ex(moe_dispatch_kernel<true>, 1, kSortThreads, smem, s, experts, P, int(E), chunk,
                                  row_offsets, order, positions, counts));
  const mxq_status st = launched(launch_pdl_ex(moe_dispatch_kernel<false>, chunks, kSortThreads, smem, s, experts, P,
                                               int(E), chunk, row_offsets, order, positions, counts));
  if (st != MXQ_OK) return st;
  return launched(launch_pdl_ex(moe_dispatch_place_kernel, chunks, kSortThreads, 0, s, experts, P, int(E), chunk,
                                int(chunks), row_offsets, order, positions,
                                static_cast<const uint32_t*>(counts)));
}

}  // extern "C"
