// Routing by scores: softmax or sigmoid scores, a balance bias that enters the
// choice only, group-limited top-k with k up to 16, weights renormalised over
// the choices; and its gradient.
//
//   s[t, e] = softmax_e(h[t, :]) or 1 / (1 + exp(-h[t, e])),  c = s + bias
//   a group's value = the sum of its group_top largest c; top_groups groups stay
//   choices = the k largest c of the groups that stay (ties -> lower expert)
//   w[t, j] = scale * s[t, e_j] / (renorm ? sum_i s[t, e_i] : 1)
//
// The order is not that of fp32 roundings: without a bias and sums of two it is the
// logits' own order, else that of c and its sums in fp64, which ranks the candidates
// that fp32 cannot tell apart (scores that saturate in fp64 too are ties).
//
// Bound by instruction issue: 65536 x 256 fp32 logits, 8 experts in 4 of 8 groups by
// sigmoid scores with a bias, 40 us, 493 warp instructions a token; the
// logits' bytes alone would take 10.9.  4 tokens: 4.0 us.  Layers of few experts take
// a thread per token (route_few_kernel).
#include <cfloat>
#include <climits>
#include <cmath>
#include <type_traits>

#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 8;  // warps per block, a token each
constexpr int kFewThreads = 128;  // of route_few_kernel's blocks
constexpr int kMaxOpen = 512;  // tokens a block lists for its fp64 pass
constexpr int32_t kOpenMark = INT_MIN;  // in expert_idx until then: one that did not fit the list
// A logit at or below bf16's lowest value masks its expert, as -inf does.
constexpr float kLowest = -3.3895313892515355e38f;

// What decides a token's order: the logits, or the scores (plus bias).
enum RouteMode { kByLogit = 0, kBySigmoid = 1, kBySoftmax = 2 };

// Candidates whose keys (23-bit values, see route_kernel) are this close are
// not told apart by fp32.  In units of the key (at most 2^-23 of a score), for a pair:
//   logits: m - x and the key each rounded once, 0.75 a candidate: under 2;
//   sigmoid: the bias part of the key 1.5, the key's rounding 0.5, the score
//     s (1 - s) (2^-22 + 1.5 |x| 2^-24) + s 2^-23 <= 1.7 a candidate: under 8;
//   softmax: bias and key 2 a candidate, as above.  With u = 2^-24, z = m - x and p the
//     scores (the pair's sum to at most 1): the exponentials (4 u + 2.2 u z) p, 2.8 for both;
//     their products with 1 / sum, u p, 0.5; and 1 / sum itself, which moves the pair by at
//     most its relative error: V + 4 additions (V - 1 in a lane, 5 over the warp), the
//     terms' 4 u + 2.2 u z averaged by p (z averaged, times the larger p, is at most 1.5
//     for 256 experts), a reciprocal, (V + 12.3) u.  In all 17.5 for 8 logits a lane, 21.5
//     for 16.
__host__ __device__ constexpr unsigned near_units(int mode, int V) {
  return mode == kByLogit ? 4u : mode == kBySigmoid ? 12u : V <= 8 ? 24u : 28u;
}

struct RouteParams {
  int64_t T;
  int E, k;
  int G, gs;        // groups that are told apart (1: no group limit), experts each
  int lanes;        // lanes per group: 32 / (G rounded up to a power of two)
  int top_groups, group_top;
  int sigmoid, renorm;
  int by_logit;     // the logits' order decides (no bias, no sum of two scores)
  int per_warp;     // consecutive tokens of one warp
  int slots;        // of them, tokens whose weights are formed together
  int seg;          // lanes per such token: k rounded up to a power of two
  float scale;
  const void* logits;
  const float* bias;
  int32_t* idx;
  float* gate;
  int32_t* status;
};

MOE_DEV float to_float(float v) { return v; }
MOE_DEV float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

// A row's logit and an expert's bias, where the expert comes out of a key.  The
// bounds-checked build reports one outside 0..E-1 and does not read there.
MOE_DEV bool expert_ok(const RouteParams& p, int e) {
#if MOE_CHECK_BOUNDS
  if (e < 0 || e >= p.E) {
    if (p.status) atomicOr(p.status, MOE_STATUS_BAD_INDEX);
    return false;
  }
#else
  (void)p, (void)e;
#endif
  return true;
}
template <typename L>
MOE_DEV float logit_at(const RouteParams& p, const L* h, int e) {
  return expert_ok(p, e) ? to_float(h[e]) : 0.f;
}
MOE_DEV float bias_at(const RouteParams& p, int e) {
  return expert_ok(p, e) ? __ldg(p.bias + e) : 0.f;
}

MOE_DEV bool counts(float x) { return x > kLowest && x < INFINITY; }  // false for NaN

MOE_DEV float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}
MOE_DEV float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// W consecutive logits from p (aligned to W elements), as floats
template <int W>
MOE_DEV void load_logits(const float* p, float* x) {
  if constexpr (W == 4) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p));
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  } else {
    x[0] = __ldg(p);
  }
}
template <int W>
MOE_DEV void load_logits(const __nv_bfloat16* p, float* x) {
  if constexpr (W == 4) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    x[0] = __uint_as_float(v.x << 16); x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16); x[3] = __uint_as_float(v.y & 0xffff0000u);
  } else {
    x[0] = __bfloat162float(__ldg(p));
  }
}

// fp64 values as integers of the same order; 0 below all of them
MOE_DEV unsigned long long ordered(double v) {
  const long long b = __double_as_longlong(v);
  return static_cast<unsigned long long>(b ^ ((b >> 63) | LLONG_MIN));
}

// The token's choices decided in fp64: lane j < k returns choice j's expert, or
// -1.  buf: E entries of this warp's shared memory.  Called for the few
// tokens that settle_order and settle_groups leave open, by one warp while
// others are done, so its chain of dependent steps counts: a choice is three integer
// maxima (both halves of the value, then the lowest expert) and a search
// through the winner's own candidates, and the loads and exponentials of a
// lane's V candidates are independent.
template <typename L, int V>
__device__ int route_exact(const RouteParams& p, int64_t t, unsigned long long* buf) {
  const int lane = threadIdx.x & 31;
  const L* h = static_cast<const L*>(p.logits) + t * p.E;
  // lane's candidates: experts first + lanes * i of its group
  const int q = lane / p.lanes;
  const int first = q * p.gs + (lane & (p.lanes - 1));
  const int end = q < p.G ? (q + 1) * p.gs : 0;
  float x[V], bias[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = first + p.lanes * i;
    x[i] = e < end ? to_float(h[e]) : -INFINITY;
    bias[i] = e < end && p.bias ? __ldg(p.bias + e) : 0.f;
  }
  double c[V];
  if (p.by_logit) {
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = static_cast<double>(x[i]) + 0.0;  // -0 is +0
  } else if (p.sigmoid) {
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = 1.0 / (1.0 + exp(-static_cast<double>(x[i])));
  } else {
    float mf = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) mf = counts(x[i]) ? fmaxf(mf, x[i]) : mf;
    const double m = warp_max(mf);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      c[i] = counts(x[i]) ? exp(static_cast<double>(x[i]) - m) : 0.0;
      sum += c[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] /= sum;
  }
  double b1 = -INFINITY, b2 = -INFINITY;  // the lane's two best, then its group's
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = first + p.lanes * i;
    const bool can = counts(x[i]) && fabsf(bias[i]) < INFINITY;
    c[i] = can ? c[i] + static_cast<double>(bias[i]) : -INFINITY;
    if (e < end) buf[e] = can ? ordered(c[i]) : 0ull;
    b2 = fmax(b2, fmin(b1, c[i]));
    b1 = fmax(b1, c[i]);
  }
  bool stays = true;
  if (p.G > 1) {
    for (int o = 1; o < p.lanes; o <<= 1) {
      const double o1 = __shfl_xor_sync(kFull, b1, o), o2 = __shfl_xor_sync(kFull, b2, o);
      b2 = fmax(fmin(b1, o1), fmax(b2, o2));
      b1 = fmax(b1, o1);
    }
    const double v = p.group_top == 2 && b2 > -INFINITY ? b1 + b2 : b1;
    int rank = 0;
    for (int g = 0; g < p.G; ++g) {
      const double o = __shfl_sync(kFull, v, g * p.lanes);
      rank += o > v || (o == v && g < q);
    }
    stays = rank < p.top_groups;
  }
  int mine = -1;
  unsigned long long best = 0ull;
  int be = 0;
  bool look = stays;  // the lane's best is not known yet
  for (int j = 0; j < p.k; ++j) {
    if (look) {
      best = 0ull;
      for (int e = first; e < end; e += p.lanes)
        if (buf[e] > best) {
          best = buf[e];
          be = e;
        }
      look = false;
    }
    const unsigned hi = static_cast<unsigned>(best >> 32), lo = static_cast<unsigned>(best);
    const unsigned top_hi = __reduce_max_sync(kFull, hi);
    const unsigned top_lo = __reduce_max_sync(kFull, hi == top_hi ? lo : 0u);
    if (top_hi == 0u && top_lo == 0u) break;  // the same in every lane: nothing is left
    const bool among = hi == top_hi && lo == top_lo;
    const int e = static_cast<int>(__reduce_min_sync(kFull, among ? static_cast<unsigned>(be) : ~0u));
    if (lane == j) mine = e;
    if (among && be == e) {
      buf[e] = 0ull;
      look = true;
    }
  }
  __syncwarp();  // the buffer is free for the warp's next token
  return mine;
}

// sum and maximum over aligned segments of `seg` lanes (a power of two)
MOE_DEV float seg_sum(float v, int seg) {
  for (int o = seg >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
MOE_DEV float seg_max(float v, int seg) {
  for (int o = seg >> 1; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}

// Weight of this lane's choice from its logit (-inf: none); the choices of a
// token lie in one segment.  m, inv: the row's maximum and 1 / sum of
// exponentials, for softmax weights that are not renormalised.
MOE_DEV float choice_weight(const RouteParams& p, float x, float m, float inv) {
  const bool there = x > -INFINITY;
  if (!p.renorm) {
    if (!there) return 0.f;
    return p.scale * (p.sigmoid ? __fdividef(1.0f, 1.0f + expf(-x)) : expf(x - m) * inv);
  }
  // scaled by the largest choice so that small scores keep their ratio
  const float mx = seg_max(x, p.seg);
  const float ref = p.sigmoid ? fminf(mx, 0.f) : mx;
  float w = 0.f;
  if (there) {
    const bool up = p.sigmoid && x >= 0.f;
    w = expf(up ? -x : x - ref);
    if (p.sigmoid) w = __fdividef(up ? 1.0f : w, 1.0f + (up ? w : expf(x)));
  }
  const float sum = seg_sum(w, p.seg);
  return sum > 0.f ? p.scale * __fdividef(w, sum) : 0.f;
}

// A whole token through route_exact, by one warp.
template <typename L, int V>
__device__ __noinline__ void finish_exact(const RouteParams& p, int64_t t,
                                          unsigned long long* buf) {
  const int lane = threadIdx.x & 31;
  const L* h = static_cast<const L*>(p.logits) + t * p.E;
  const int e = route_exact<L, V>(p, t, buf);
  float m = -INFINITY, inv = 0.f;
  if (!p.sigmoid && !p.renorm) {
    for (int i = lane; i < p.E; i += 32) {
      const float x = to_float(h[i]);
      if (counts(x)) m = fmaxf(m, x);
    }
    m = warp_max(m);
    for (int i = lane; i < p.E; i += 32) {
      const float x = to_float(h[i]);
      if (counts(x)) inv += expf(x - m);
    }
    inv = warp_sum(inv);
    inv = inv > 0.f ? 1.0f / inv : 0.f;
  }
  const float w = choice_weight(p, e >= 0 ? logit_at(p, h, e) : -INFINITY, m, inv);
  if (lane < p.k) {
    p.idx[t * p.k + lane] = e;
    p.gate[t * p.k + lane] = w;
  }
}

// Descending sort of N register values (N a power of two): Batcher's odd-even
// merge network (1968), 19 exchanges for 8 values, 63 for 16.
template <int N>
MOE_DEV void sort_desc(uint32_t (&v)[N]) {
#pragma unroll
  for (int p = 1; p < N; p <<= 1) {
#pragma unroll
    for (int k = p; k >= 1; k >>= 1) {
#pragma unroll
      for (int lo = 0; lo < N; ++lo) {
        const int hi = lo + k;
        // pairs of the merge step: blocks of 2k from k % p on, inside one run of 2p
        if (hi < N && lo >= k % p && (lo - k % p) % (2 * k) < k && lo / (2 * p) == hi / (2 * p)) {
          const uint32_t a = max(v[lo], v[hi]);
          v[hi] = min(v[lo], v[hi]);
          v[lo] = a;
        }
      }
    }
  }
}

// A lane's sorted keys: the first in `head`, the others behind it in the lane's
// column of shared memory (its own reads and writes only, so nothing waits), and
// zeros behind those.  Taking the first away is then one predicated load; shifting V
// registers costs V instructions of the whole warp.
constexpr int kZeroRows = kMaxChoices + 1;  // what k takes from an empty list may read
template <int V>
struct KeyList {
  uint32_t head;
  uint32_t next;  // shared-memory address
  // out: none of the lane's keys may be chosen (its group is left out)
  MOE_DEV void fill(const uint32_t (&key)[V], uint32_t column, bool out) {
    head = out ? 0u : key[0];
#pragma unroll
    for (int i = 1; i < V; ++i)
      asm volatile("st.shared.u32 [%0], %1;" ::"r"(column + 128u * (i - 1)), "r"(key[i]) : "memory");
    next = out ? column + 128u * (V - 1) : column;
  }
  MOE_DEV void take(uint32_t top) {  // the first key, if it is `top` (the warp's largest), goes
    if (head == top) {
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(head) : "r"(next) : "memory");
      next += 128u;
    }
  }
};

MOE_DEV float exp2_fast(float x) {  // 2 units in the last place; ftz
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
MOE_DEV float rcp_fast(float x) {  // 1 unit in the last place; ftz
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
constexpr float kLog2e = 1.4426950408889634f;

MOE_DEV int expert_of(uint32_t key) { return 255 - static_cast<int>(key & 511u); }

MOE_DEV float warp_max_redux(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// Blocks that fit an SM: 64 registers a thread up to 8 logits a lane, 80 above.
__host__ __device__ constexpr int blocks_per_sm(int V) { return V <= 8 ? 4 : 3; }

// Keys of one lane's V logits (their experts: e0 + (i / W) * lanes * W + i % W),
// and for softmax weights the row's maximum and 1 / sum.  MASKED: some of
// them, here or in another lane, may not count.
template <typename L, int V, int W, int MODE, bool MASKED>
MOE_DEV void make_keys(const RouteParams& p, const float (&x)[V], const float (&off)[V],
                       float unit, int e0, bool sums, uint32_t (&key)[V], float& m, float& inv,
                       bool& bad) {
  constexpr bool kExactKey = MODE == kByLogit && sizeof(L) == 2;
  bool can[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    can[i] = true;
    if (MASKED) {
      const bool fine = x[i] < INFINITY;  // false for NaN
      bad |= !fine;
      can[i] = fine && x[i] > kLowest;
    }
  }
  if (sums || (MODE == kByLogit && !kExactKey)) {
    m = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) m = fmaxf(m, can[i] ? x[i] : -INFINITY);
    m = warp_max_redux(m);
  }
  float s[V];
  if (sums) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      s[i] = can[i] ? exp2_fast((x[i] - m) * kLog2e) : 0.f;
      sum += s[i];
    }
    sum = warp_sum(sum);
    inv = sum > 0.f ? __frcp_rn(sum) : 0.f;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const uint32_t low = static_cast<uint32_t>(255 - e0 - (i / W) * p.lanes * W - i % W);
    float v;
    if constexpr (kExactKey) {  // the bits of a bf16 in ascending order, 1..65535
      const uint32_t u = __float_as_uint(x[i] + 0.f) >> 16;  // -0 is +0
      v = __uint_as_float((u & 0x8000u ? 0xffffu ^ u : u | 0x8000u) + 1u);
    } else if constexpr (MODE == kByLogit) {
      v = fmaxf(fmaf(m - x[i], -262144.0f, 16777214.0f), 8388609.0f);
    } else {
      const float sc = MODE == kBySigmoid ? rcp_fast(1.0f + exp2_fast(-kLog2e * x[i])) : s[i] * inv;
      v = fmaf(sc, unit, off[i]);
      if (MASKED) can[i] = can[i] && v > 0.f;  // not the NaN of a masked expert
    }
    key[i] = can[i] ? (__float_as_uint(v) << 9) + low : 0u;
  }
}

// Whether keys that are close have unlike inputs: equal logits (and biases) are
// in their order already.  close: this lane's choice (at `rel`) and the next;
// edge: the last choice and one of those this lane has left.
template <typename L, int V>
MOE_DEV void check_inputs(const RouteParams& p, const L* h, bool has_bias, unsigned near,
                          uint32_t mine, int rel, uint32_t last, KeyList<V> list, bool& close,
                          bool& edge) {
  const bool there = rel >= 0 && rel < p.k && mine != 0u;
  const uint32_t after = __shfl_down_sync(kFull, mine, 1);
  const int e = there ? expert_of(mine) : 0;
  const float x = there ? logit_at(p, h, e) : 0.f, b = there && has_bias ? bias_at(p, e) : 0.f;
  const float xa = __shfl_down_sync(kFull, x, 1), ba = __shfl_down_sync(kFull, b, 1);
  close = close && after != 0u && !(x == xa && b == ba);
  // With nothing left here there is nothing to compare; `last` is then no expert's key
  // either where the whole row ran out before k choices.
  if (list.head == 0u) edge = false;
  if (edge) {
    const int el = expert_of(last);
    const float xl = logit_at(p, h, el), bl = has_bias ? bias_at(p, el) : 0.f;
    edge = false;
    while (list.head != 0u && (last >> 9) - (list.head >> 9) <= near) {
      const int en = expert_of(list.head);
      edge |= logit_at(p, h, en) != xl || (has_bias && bias_at(p, en) != bl);
      list.take(list.head);
    }
  }
}

// The order of the choices in fp64, where the groups are settled: the k choices and
// those left that are close to the last one, a candidate per lane, ranked by
// counting.  False if there are more candidates than lanes.
template <typename L, int V, int MODE>
MOE_DEV bool settle_order(const RouteParams& p, const L* h, bool has_bias, unsigned near, int at,
                          uint32_t last, KeyList<V> list, uint32_t& mine) {
  const int lane = threadIdx.x & 31;
  uint32_t cand = __shfl_sync(kFull, mine, (at + lane) & 31);
  if (lane >= p.k) cand = 0u;
  int n = p.k;
  for (;; ++n) {
    const uint32_t next = __reduce_max_sync(kFull, list.head);
    if (next == 0u || (last >> 9) - (next >> 9) > near) break;
    if (n == 32) return false;
    if (lane == n) cand = next;
    list.take(next);
  }
  const int e = expert_of(cand);
  double c = -INFINITY;
  if (cand != 0u) {
    const double x = logit_at(p, h, e);
    c = MODE == kByLogit ? x : 1.0 / (1.0 + exp(-x)) + (has_bias ? bias_at(p, e) : 0.f);
  }
  int rank = 0;
  for (int i = 0; i < n; ++i) {
    const double o = __shfl_sync(kFull, c, i);
    const int oe = __shfl_sync(kFull, e, i);
    rank += o > c || (o == c && oe < e);
  }
  for (int i = 0; i < n; ++i) {
    const int r = __shfl_sync(kFull, rank, i);
    const uint32_t key = __shfl_sync(kFull, cand, i);
    if (r < p.k && lane == at + r) mine = key;
  }
  return true;
}

// Which groups stay, in fp64.  a1, a2: the keys of the group's two best.  False
// where a third candidate is so close to them that they are not known.
template <typename L, int V, int MODE>
MOE_DEV bool settle_groups(const RouteParams& p, const L* h, bool has_bias, unsigned near, int q,
                           uint32_t a1, uint32_t a2, const uint32_t (&key)[V], bool& out) {
  const uint32_t least = p.group_top == 2 ? a2 : a1;
  bool third = false;
#pragma unroll
  for (int i = 0; i < (V < 3 ? V : 3); ++i)
    third |= key[i] != 0u && key[i] != a1 && key[i] != a2 && (least >> 9) - (key[i] >> 9) <= near;
  if (__any_sync(kFull, third)) return false;
  double v[2];
#pragma unroll 1
  for (int i = 0; i < 2; ++i) {
    const uint32_t a = i == 0 ? a1 : a2;
    const int e = expert_of(a);
    double c = -INFINITY;
    if (a != 0u) {
      const double x = logit_at(p, h, e);
      c = MODE == kByLogit ? x : 1.0 / (1.0 + exp(-x)) + (has_bias ? bias_at(p, e) : 0.f);
    }
    v[i] = c;
  }
  const double value = p.group_top == 2 ? v[0] + v[1] : fmax(v[0], v[1]);
  int rank = 0;
  for (int g = 0; g < p.G; ++g) {
    const double o = __shfl_sync(kFull, value, g * p.lanes);
    rank += o > value || (o == value && g < q);
  }
  out = q < p.G && rank >= p.top_groups;
  return true;
}

// A warp per token.  Lane l holds V logits of one group (of the whole row
// where there is no group limit).  Each candidate becomes a 32-bit key,
// (value in 23 bits) << 9 | (255 - expert): unique, larger is better, equal
// values to the lower expert; 0 marks an expert that cannot be chosen.  The
// value is the mantissa of a float between 2^23 and 2^24, so that a scale, an
// offset and the rounding to an integer are one fused multiply-add.  A lane
// sorts its keys once, and each choice is one warp-wide integer maximum over the
// lanes' first keys.  The rounding is checked afterwards: where neighbours in
// the order (or the last choice and one left out) are within near_units, and
// are not equal inputs, those candidates alone are ranked in fp64
// (settle_order, settle_groups).  What that leaves open (softmax scores with a
// bias, whose sum is needed in fp64 too; a third candidate close to a group's
// two) is listed, and the block's warps decide it at the end (finish_exact),
// side by side.  What that costs, 65536 x 256, us: by sigmoid scores and groups 40 for
// random logits, 67 where every expert has a twin one step away (candidates settled
// alone), 300 where every token goes to finish_exact (such as a group of which one
// expert is left, with sums of two); softmax scores with a bias 47 and, with twins,
// 290; by the logits 31 and 50.
//
// The scores here only decide, so they take the hardware's exp2 and reciprocal;
// the weights of the k choices are formed from their logits with expf.  That
// part uses k lanes, so a warp first collects the choices of `slots` tokens.
// A token is a chain of dependent steps behind a load from memory, so the next
// token's logits are on their way while one is decided.
template <typename L, int V, int W, int MODE>
__global__ void __launch_bounds__(kWarps * 32, blocks_per_sm(V))
route_kernel(const __grid_constant__ RouteParams p) {
  // per warp: the lanes' key lists, and after the loop route_exact's candidates
  __shared__ union {
    uint32_t column[V - 1 + kZeroRows][32];
    unsigned long long candidate[256];
  } s_warp[kWarps];
  __shared__ int32_t s_open[kMaxOpen];
  __shared__ int s_num_open;
  dev::pdl_trigger();
  if (threadIdx.x == 0) s_num_open = 0;
  dev::pdl_wait();
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int q = lane / p.lanes, li = lane & (p.lanes - 1);
  constexpr bool kExactKey = MODE == kByLogit && sizeof(L) == 2;  // a bf16 logit fits the key
  constexpr unsigned kNear = near_units(MODE, V);
  const bool has_bias = MODE != kByLogit && p.bias != nullptr;
  const bool sums = !p.sigmoid && (MODE == kBySoftmax || !p.renorm);  // weights need 1 / sum
  bool bad = false;

  // this lane's experts: first + (i / W) * lanes * W + li * W + i % W within group q
  const int first = q * p.gs;
  // the warp's tokens: tb .. tb + count - 1
  const int64_t tb = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * p.per_warp;
  const int count = tb < p.T ? static_cast<int>(min(static_cast<int64_t>(p.per_warp), p.T - tb)) : 0;
  const L* rows = static_cast<const L*>(p.logits) + tb * p.E;
  const L* from = rows + first + li * W;  // this lane's part of the next row to load
  bool has[V / W];
#pragma unroll
  for (int c = 0; c < V / W; ++c) has[c] = q < p.G && li * W + c * p.lanes * W < p.gs;
  auto load_row = [&](float (&x)[V]) {
#pragma unroll
    for (int c = 0; c < V / W; ++c) {
      if (has[c]) {
        load_logits<W>(from + c * p.lanes * W, x + c * W);
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i) x[c * W + i] = -INFINITY;
      }
    }
    from += p.E;
  };
  float ahead[V];  // the next token's logits: on their way during the set-up, and once a
                   // token's are keys during its choice
  if (count > 0) load_row(ahead);
  float off[V];    // score modes: the bias's part of the key; NaN masks the expert
  float unit = 0.f;
  if constexpr (MODE != kByLogit) {
    float bmin = INFINITY, bmax = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int o = (i / W) * p.lanes * W + li * W + i % W;
      off[i] = 0.f;
      if (q < p.G && o < p.gs) {
        if (has_bias) off[i] = __ldg(p.bias + first + o);
        if (fabsf(off[i]) < INFINITY) {
          bmin = fminf(bmin, off[i]);
          bmax = fmaxf(bmax, off[i]);
        } else {
          if (!(off[i] < 0.f)) bad = true;  // NaN or +inf; -inf masks the expert
          off[i] = NAN;
        }
      }
    }
    const float lo = -warp_max(-bmin);
    unit = 8388600.0f / (1.0f + (warp_max(bmax) - lo));
#pragma unroll
    for (int i = 0; i < V; ++i)  // a range past fp32's: unit is 0 and fp64 decides
      off[i] = off[i] == off[i] ? fminf(off[i] - lo, FLT_MAX) * unit + 8388610.0f : NAN;
  }
  // every lane holds V logits of experts that its bias does not mask
  bool whole = q < p.G && p.gs == p.lanes * V;
  if constexpr (MODE != kByLogit) {
#pragma unroll
    for (int i = 0; i < V; ++i) whole = whole && off[i] == off[i];
  }
  whole = __all_sync(kFull, whole);

  const uint32_t column = dev::smem_u32(&s_warp[warp].column[0][lane]);
  for (int i = 0; i < kZeroRows; ++i) s_warp[warp].column[V - 1 + i][lane] = 0u;
  // in the weights' part lane slot * seg + j works for choice j of a batch's token `slot`
  const int my_slot = lane / p.seg, my_j = lane & (p.seg - 1);

  for (int done = 0; done < count; done += p.slots) {
    const int in_batch = min(p.slots, count - done);
    uint32_t mine = 0u;
    float my_m = 0.f, my_inv = 0.f;
    unsigned open = 0u;      // slots whose order fp32 could not tell
    for (int slot = 0; slot < in_batch; ++slot) {
      // 0 unless a logit is masked, NaN or infinite (or above 2.3e38): the product
      // overflows for the lowest values too, and inf * 0 is NaN
      float odd = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) odd = fmaf(-kLog2e * ahead[i], 0.f, odd);
      uint32_t key[V];
      float m = 0.f, inv = 0.f;
      if (whole && __all_sync(kFull, odd == 0.f))
        make_keys<L, V, W, MODE, false>(p, ahead, off, unit, first + li * W, sums, key, m, inv, bad);
      else
        make_keys<L, V, W, MODE, true>(p, ahead, off, unit, first + li * W, sums, key, m, inv, bad);
      if (done + slot + 1 < count) load_row(ahead);
      sort_desc<V>(key);

      bool unsure = false, out = false;
      if (p.G > 1) {
        uint32_t a1 = key[0], a2 = V > 1 ? key[V > 1 ? 1 : 0] : 0u;
        for (int o = 1; o < p.lanes; o <<= 1) {
          const uint32_t o1 = __shfl_xor_sync(kFull, a1, o), o2 = __shfl_xor_sync(kFull, a2, o);
          a2 = max(min(a1, o1), max(a2, o2));
          a1 = max(a1, o1);
        }
        uint32_t v = a1 >> 9;
        if (p.group_top == 2) {
          v += a2 >> 9;
          unsure = a1 != 0u && a2 == 0u;  // a sum of one: its offset differs
        }
        uint32_t g = a1 ? (v << 5) | static_cast<uint32_t>(31 - q) : 0u;  // 0: stays, or is empty
        uint32_t last = 0u;
#pragma unroll 4
        for (int i = 0; i < p.top_groups; ++i) {
          last = __reduce_max_sync(kFull, g);
          if (g == last) g = 0u;
        }
        out = g != 0u;
        // a group left out that may be as good as the last one that stays
        const bool near_out = !kExactKey && out && last - g < (2 * kNear + 1) << 5;
        if (__any_sync(kFull, near_out || unsure)) {
          unsure = __any_sync(kFull, unsure);
          if constexpr (MODE != kBySoftmax && !kExactKey) {
            const L* h = rows + static_cast<int64_t>(done + slot) * p.E;
            unsure = unsure || !settle_groups<L, V, MODE>(p, h, has_bias, kNear, q, a1, a2, key, out);
          } else {
            unsure = true;
          }
        }
      }

      KeyList<V> list;
      list.fill(key, column, out);
      uint32_t last = 0u;
      const int rel = lane - slot * p.seg;
#pragma unroll 4
      for (int j = 0; j < p.k; ++j) {
        last = __reduce_max_sync(kFull, list.head);
        if (rel == j) mine = last;
        list.take(last);
      }
      if constexpr (!kExactKey) {
        // neighbours in the order, and the last choice against what this lane has left
        const uint32_t after = __shfl_down_sync(kFull, mine, 1);
        // (whole keys: the experts' bits only widen it, and check_inputs sorts out a 0 in
        // place of a key)
        bool close = static_cast<unsigned>(rel) < static_cast<unsigned>(p.k - 1) &&
                     mine - after < (kNear + 1) << 9;
        bool edge = last - list.head < (kNear + 1) << 9;
        if (__any_sync(kFull, close || edge)) {
          const L* h = rows + static_cast<int64_t>(done + slot) * p.E;
          check_inputs(p, h, has_bias, kNear, mine, rel, last, list, close, edge);
          if (__any_sync(kFull, close || edge)) {
            bool settled = false;
            if constexpr (MODE != kBySoftmax)
              settled = settle_order<L, V, MODE>(p, h, has_bias, kNear, slot * p.seg, last, list, mine);
            if (!settled) unsure = true;
          }
        }
      }
      if (__any_sync(kFull, unsure)) open |= 1u << slot;
      if (sums && my_slot == slot) {
        my_m = m;
        my_inv = inv;
      }
    }

    const bool in = my_slot < in_batch && my_j < p.k;
    const L* h = rows + static_cast<int64_t>(done) * p.E;
    const int e = in && mine ? expert_of(mine) : -1;
    const float xj = e >= 0 ? logit_at(p, h + my_slot * p.E, e) : -INFINITY;
    const float w = choice_weight(p, xj, my_m, my_inv);
    if (in && !((open >> my_slot) & 1u)) {
      const int64_t o = (tb + done) * p.k + my_slot * p.k + my_j;
      p.idx[o] = e;
      p.gate[o] = w;
    }
    for (; open; open &= open - 1u) {
      const int64_t to = tb + done + __ffs(open) - 1;
      if (lane == 0) {
        const int n = atomicAdd(&s_num_open, 1);
        if (n < kMaxOpen) s_open[n] = static_cast<int32_t>(to);
        else p.idx[to * p.k] = kOpenMark;  // no room: found again below
      }
    }
  }
  // (a call inside the loop above would keep its registers in local memory)
  __syncthreads();
  const int num_open = s_num_open;
  for (int i = warp; i < min(num_open, kMaxOpen); i += kWarps)
    finish_exact<L, V>(p, s_open[i], s_warp[warp].candidate);
  if (num_open > kMaxOpen) {
    for (int i = 0; i < count; ++i)
      if (*static_cast<volatile int32_t*>(p.idx + (tb + i) * p.k) == kOpenMark)
        finish_exact<L, V>(p, tb + i, s_warp[warp].candidate);
  }
  if (__any_sync(kFull, bad) && lane == 0 && p.status) atomicOr(p.status, MOE_STATUS_BAD_LOGIT);
}

// Few experts (E <= EM <= 16) and many tokens: a thread per token, everything in its
// registers.  The order is decided by the logits themselves or, with a bias or sums of
// two scores, by scores in fp64 for all of them: with so few it costs less than
// telling where fp32 would do.  launch_route_t says from how many tokens.
template <typename L, int EM, bool BY_LOGIT>
__global__ void __launch_bounds__(kFewThreads) route_few_kernel(const __grid_constant__ RouteParams p) {
  using C = typename std::conditional<BY_LOGIT, float, double>::type;
  constexpr C kNone = -INFINITY;
  dev::pdl_trigger();
  dev::pdl_wait();
  bool bad = false;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kFewThreads;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kFewThreads + threadIdx.x; t < p.T; t += stride) {
    const L* h = static_cast<const L*>(p.logits) + t * p.E;
    float x[EM];
    if (p.E % 4 == 0) {
#pragma unroll
      for (int i = 0; i < EM; i += 4) {
        if (i < p.E) load_logits<4>(h + i, x + i);
        else x[i] = x[i + 1] = x[i + 2] = x[i + 3] = -INFINITY;
      }
    } else {
#pragma unroll
      for (int i = 0; i < EM; ++i) x[i] = i < p.E ? to_float(h[i]) : -INFINITY;
    }
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < EM; ++i) {
      if (!counts(x[i])) {
        if (!(x[i] < 0.f)) bad = true;  // NaN or +inf
        x[i] = -INFINITY;
      }
      m = fmaxf(m, x[i]);
    }
    // what decides; an expert that cannot be chosen has kNone
    C c[EM];
    if constexpr (BY_LOGIT) {
#pragma unroll
      for (int i = 0; i < EM; ++i) c[i] = x[i];
    } else {
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < EM; ++i) {
        const double z = static_cast<double>(x[i]);
        c[i] = x[i] == -INFINITY ? 0.0 : p.sigmoid ? 1.0 / (1.0 + exp(-z)) : exp(z - m);
        sum += c[i];
      }
#pragma unroll
      for (int i = 0; i < EM; ++i) {
        if (!p.sigmoid) c[i] /= sum;
        bool can = x[i] > -INFINITY;
        if (p.bias && i < p.E) {
          const float b = __ldg(p.bias + i);
          if (!(fabsf(b) < INFINITY)) {
            if (!(b < 0.f)) bad = true;
            can = false;
          }
          c[i] += static_cast<double>(b);
        }
        if (!can) c[i] = kNone;
      }
    }
    unsigned allowed = (1u << EM) - 1u;
    if (p.G > 1) {
      C value[EM];
#pragma unroll
      for (int g = 0; g < EM; ++g) {
        value[g] = kNone;
        if (g < p.G) {
          C b1 = kNone, b2 = kNone;
#pragma unroll
          for (int i = 0; i < EM; ++i) {
            if (i >= g * p.gs && i < (g + 1) * p.gs) {
              if (c[i] > b1) {
                b2 = b1;
                b1 = c[i];
              } else if (c[i] > b2) {
                b2 = c[i];
              }
            }
          }
          value[g] = p.group_top == 2 && b2 > kNone ? b1 + b2 : b1;
        }
      }
      allowed = 0u;
      for (int n = 0; n < p.top_groups; ++n) {
        C best = kNone;
        int bg = -1;
#pragma unroll
        for (int g = 0; g < EM; ++g)
          if (value[g] > best) {
            best = value[g];
            bg = g;
          }
        if (bg < 0) break;
        allowed |= ((1u << p.gs) - 1u) << (bg * p.gs);
#pragma unroll
        for (int g = 0; g < EM; ++g)
          if (g == bg) value[g] = kNone;
      }
    }
    unsigned long long order = 0ull;  // 4 bits a choice
    int n = 0;
    unsigned taken = 0u;
    for (; n < p.k; ++n) {
      C best = kNone;
      int be = -1;
#pragma unroll
      for (int i = 0; i < EM; ++i)
        if (((allowed & ~taken) >> i & 1u) && c[i] > best) {
          best = c[i];
          be = i;
        }
      if (be < 0) break;
      order |= static_cast<unsigned long long>(be) << (4 * n);
      taken |= 1u << be;
    }
    // weights of the chosen experts, as in choice_weight
    float w[EM], sum = 0.f, ref = 0.f;
    if (p.renorm) {
      float mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < EM; ++i)
        if (taken >> i & 1u) mx = fmaxf(mx, x[i]);
      ref = p.sigmoid ? fminf(mx, 0.f) : mx;
    } else if (!p.sigmoid) {
      ref = m;
    }
#pragma unroll
    for (int i = 0; i < EM; ++i) {
      w[i] = 0.f;
      const bool chosen = taken >> i & 1u;
      if (chosen || (!p.renorm && !p.sigmoid && x[i] > -INFINITY)) {
        const bool up = p.sigmoid && x[i] >= 0.f;
        w[i] = expf(up ? -x[i] : x[i] - ref);
        if (p.sigmoid) w[i] = __fdividef(up ? 1.0f : w[i], 1.0f + (up ? w[i] : expf(x[i])));
        sum += w[i];
      }
    }
    const float f = p.renorm || !p.sigmoid ? (sum > 0.f ? __fdividef(1.0f, sum) : 0.f) : 1.0f;
    for (int j = 0; j < p.k; ++j) {
      const int e = j < n ? static_cast<int>(order >> (4 * j)) & 15 : -1;
      float wj = 0.f;
#pragma unroll
      for (int i = 0; i < EM; ++i)
        if (i == e) wj = w[i];
      p.idx[t * p.k + j] = e;
      p.gate[t * p.k + j] = p.scale * (f * wj);
    }
  }
  if (bad && p.status) atomicOr(p.status, MOE_STATUS_BAD_LOGIT);
}

struct RouteBwdParams {
  int64_t T;
  int E, k;
  int seg;  // lanes per token: a power of two, >= k and >= E / 8
  int sigmoid, renorm;
  float scale;
  const void* logits;
  const int32_t* idx;
  const float* dgate;
  void* dlogits;
  int32_t* status;
};

template <int W>
MOE_DEV void store_logits(float* p, const float* v) {
  if constexpr (W == 4) *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  else *p = v[0];
}
template <int W>
MOE_DEV void store_logits(__nv_bfloat16* p, const float* v) {
  if constexpr (W == 4) {
    __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
  } else {
    *p = __float2bfloat16_rn(v[0]);
  }
}

// `seg` lanes per token: each holds up to 8 entries of the row, lane j < k of
// them choice j.  The choices are constants of the gradient.  With
// a_j = scale * dw_j:
//   DENSE (softmax, not renormalised):  dh_e = s_e (a_e - sum_i a_i s_i)
//   softmax, renorm:  dh_j = q_j (a_j - sum_i a_i q_i), q = the choices' softmax
//   sigmoid:          dh_j = a_j s_j (1 - s_j)
//   sigmoid, renorm:  dh_j = q_j (1 - s_j)(a_j - sum_i a_i q_i), q_i = s_i / sum s
// What belongs to the chosen entries goes through a row of zeros in shared
// memory, which the same lanes clear again, so that every entry of dlogits is
// stored once, in vectors.  Short chains of shuffles behind two dependent loads:
// latency for the usual batches (32768 x 64, softmax gates of 6 choices, 18 MB: 8 us a
// call, 15.6 with a warp per token and a second store of the chosen entries).
template <typename L, int W, bool DENSE>
__global__ void __launch_bounds__(kWarps * 32) route_backward_kernel(const RouteBwdParams p) {
  __shared__ __align__(16) float s_rows[kWarps][256];
  dev::pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int seg = p.seg, li = lane & (seg - 1), sub = lane / seg;
  float* row = s_rows[warp] + sub * (seg * 8);
#pragma unroll
  for (int i = 0; i < 8; ++i) s_rows[warp][lane + 32 * i] = 0.f;
  dev::pdl_wait();
  __syncwarp();
  constexpr int kParts = 8 / W;  // vectors of W entries: at part * seg * W + li * W
  const int per_warp = 32 / seg;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps * per_warp;
  bool bad = false;
  for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * per_warp; t0 < p.T;
       t0 += step) {
    const int64_t t = t0 + sub;
    const bool live = t < p.T;
    const L* h = static_cast<const L*>(p.logits) + t * p.E;
    float v[8];
    if (DENSE) {
#pragma unroll
      for (int c = 0; c < kParts; ++c) {
        const int o = (c * seg + li) * W;
        if (live && o < p.E) {
          load_logits<W>(h + o, v + c * W);
        } else {
#pragma unroll
          for (int i = 0; i < W; ++i) v[c * W + i] = -INFINITY;
        }
      }
    }
    int e = -1;
    float a = 0.f, x = -INFINITY;
    if (live && li < p.k) {
      e = __ldg(p.idx + t * p.k + li);
      a = p.scale * __ldg(p.dgate + t * p.k + li);
      if (e < -1 || e >= p.E) {
        bad = true;
        e = -1;
      }
      if (e >= 0) x = to_float(h[e]);
      if (!counts(x)) e = -1;
      if (e < 0) {
        a = 0.f;
        x = -INFINITY;
      }
    }
    float dot = 0.f, inv = 0.f, mine = 0.f;  // mine: what this choice adds to its entry
    if (DENSE) {
      float m = -INFINITY;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = counts(v[i]) ? v[i] : -INFINITY;
        m = fmaxf(m, v[i]);
      }
      m = seg_max(m, seg);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = v[i] > -INFINITY ? expf(v[i] - m) : 0.f;
        sum += v[i];
      }
      sum = seg_sum(sum, seg);
      inv = sum > 0.f ? 1.0f / sum : 0.f;
      dot = seg_sum(e >= 0 ? a * (expf(x - m) * inv) : 0.f, seg);
      mine = a;
    } else {
      float s = 0.f, slope = 1.f;
      if (p.sigmoid) {
        const float mx = p.renorm ? fminf(seg_max(x, seg), 0.f) : 0.f;
        if (e >= 0) {
          const float z = expf(-fabsf(x));  // 1 / (1 + z) and z / (1 + z) are s and 1 - s
          const float big = __fdividef(1.0f, 1.0f + z), small = __fdividef(z, 1.0f + z);
          s = x >= 0.f ? big : expf(x - mx) * big;
          slope = x >= 0.f ? small : big;
        }
      } else {
        const float mx = seg_max(x, seg);
        if (e >= 0) s = expf(x - mx);
      }
      if (p.renorm) {
        const float sum = seg_sum(s, seg);
        s = sum > 0.f ? __fdividef(s, sum) : 0.f;
        dot = seg_sum(a * s, seg);
      }
      mine = s * slope * (a - dot);
    }
    // choices of the same expert (a caller's own indices) add up, in order
    const unsigned same = __match_any_sync(kFull, e >= 0 ? (sub << 9) | e : -1 - lane);
    if (__any_sync(kFull, __popc(same) > 1)) {
      float all = 0.f;
      for (int j = 0; j < p.k; ++j) {
        const int from = (lane & ~(seg - 1)) + j;
        const float o = __shfl_sync(kFull, mine, from);
        if ((same >> from) & 1u) all += o;
      }
      mine = all;
    }
    if (e >= 0) row[e] = mine;
    __syncwarp();
#pragma unroll
    for (int c = 0; c < kParts; ++c) {
      const int o = (c * seg + li) * W;
      if (live && o < p.E) {
        float r[W];
        if constexpr (W == 4) {
          const float4 q = *reinterpret_cast<const float4*>(row + o);
          r[0] = q.x; r[1] = q.y; r[2] = q.z; r[3] = q.w;
        } else {
          r[0] = row[o];
        }
        if (DENSE) {
#pragma unroll
          for (int i = 0; i < W; ++i) r[i] = (v[c * W + i] * inv) * (r[i] - dot);
        }
        store_logits<W>(static_cast<L*>(p.dlogits) + t * p.E + o, r);
      }
    }
    __syncwarp();
    if (e >= 0) row[e] = 0.f;
    __syncwarp();
  }
  if (__any_sync(kFull, bad) && lane == 0 && p.status) atomicOr(p.status, MOE_STATUS_BAD_INDEX);
}

template <typename L, int W>
void launch_route_backward_t(const RouteBwdParams& p, cudaStream_t s) {
  const int64_t per_block = static_cast<int64_t>(kWarps) * (32 / p.seg);
  const int64_t want = (p.T + per_block - 1) / per_block, most = static_cast<int64_t>(num_sms()) * 8;
  const dim3 grid(static_cast<unsigned>(want < most ? want : most)), block(kWarps * 32);
  if (!p.sigmoid && !p.renorm) launch_pdl(route_backward_kernel<L, W, true>, grid, block, 0, s, p);
  else launch_pdl(route_backward_kernel<L, W, false>, grid, block, 0, s, p);
}

template <typename L, int V, int W>
void launch_route_m(RouteParams p, cudaStream_t s) {
  // a wave of blocks, each warp a run of consecutive tokens
  const int64_t warps = static_cast<int64_t>(num_sms()) * blocks_per_sm(V) * kWarps;
  p.per_warp = static_cast<int>((p.T + warps - 1) / warps);
  p.slots = 32 / p.seg;
  while (p.slots > p.per_warp) p.slots >>= 1;
  const int64_t per_block = static_cast<int64_t>(p.per_warp) * kWarps;
  const dim3 g(static_cast<unsigned>((p.T + per_block - 1) / per_block)), block(kWarps * 32);
  if (p.by_logit) launch_pdl(route_kernel<L, V, W, kByLogit>, g, block, 0, s, p);
  else if (p.sigmoid) launch_pdl(route_kernel<L, V, W, kBySigmoid>, g, block, 0, s, p);
  else launch_pdl(route_kernel<L, V, W, kBySoftmax>, g, block, 0, s, p);
}

template <typename L, int V>
void launch_route_v(const RouteParams& p, bool vec, cudaStream_t s) {
  if constexpr (V >= 4) {
    if (vec) return launch_route_m<L, V, 4>(p, s);
  }
  launch_route_m<L, V, 1>(p, s);
}

template <typename L, int EM>
void launch_route_few(const RouteParams& p, cudaStream_t s) {
  const int64_t want = (p.T + kFewThreads - 1) / kFewThreads, most = static_cast<int64_t>(num_sms()) * 16;
  const dim3 grid(static_cast<unsigned>(want < most ? want : most)), block(kFewThreads);
  if (p.by_logit) launch_pdl(route_few_kernel<L, EM, true>, grid, block, 0, s, p);
  else launch_pdl(route_few_kernel<L, EM, false>, grid, block, 0, s, p);
}

template <typename L>
void launch_route_t(const RouteParams& p, cudaStream_t s) {
  // A thread per token, for a warp per token (us, fp32 logits, tokens x experts and choices):
  //   by the logits, softmax:        4096 x 8, 2: 2.4, 3.5; 65536 x 8, 2: 4.6, 17.0;
  //                                  1024 x 16, 4: 3.8, 2.9; 4096 x 16, 4: 3.9, 3.7
  //   by scores and a bias, sigmoid: 4096 x 8, 2: 5.9, 4.6; 65536 x 8, 2: 9.7, 18.7;
  //     4 groups:                    16384 x 16, 4: 15.0, 10.5; 65536 x 16, 4: 16.7, 27.9
  if (p.E <= 16 && p.T >= (p.by_logit ? 4096 : 32768)) {
    if (p.E <= 8) launch_route_few<L, 8>(p, s);
    else launch_route_few<L, 16>(p, s);
    return;
  }
  const bool vec = p.gs % 4 == 0;
  const int per = vec ? (p.gs + 4 * p.lanes - 1) / (4 * p.lanes) * 4
                      : (p.gs + p.lanes - 1) / p.lanes;
  if (per <= 1) launch_route_v<L, 1>(p, false, s);
  else if (per <= 2) launch_route_v<L, 2>(p, false, s);
  else if (per <= 4) launch_route_v<L, 4>(p, vec, s);
  else if (per <= 8) launch_route_v<L, 8>(p, vec, s);
  else launch_route_v<L, 16>(p, vec, s);
}

}  // namespace

int32_t launch_route(const moe_route_config& c, const void* logits, const float* bias,
                     int32_t* expert_idx, float* gate, int32_t* status, cudaStream_t s) {
  if (c.T == 0) return MOE_OK;
  RouteParams p{};
  p.T = c.T;
  p.E = c.E;
  p.k = c.k;
  p.G = c.top_groups < c.num_groups ? c.num_groups : 1;
  p.gs = c.E / p.G;
  int lanes = 32;
  while (lanes * p.G > 32) lanes >>= 1;  // groups padded to a power of two of lanes
  p.lanes = lanes;
  p.top_groups = c.top_groups;
  p.group_top = c.group_top;
  p.sigmoid = c.score == MOE_SCORE_SIGMOID;
  p.renorm = c.renorm;
  p.by_logit = !bias && (p.G == 1 || c.group_top == 1);
  p.scale = static_cast<float>(c.scale);
  p.logits = logits;
  p.bias = bias;
  p.idx = expert_idx;
  p.gate = gate;
  p.status = status;
  p.seg = 1;
  while (p.seg < c.k) p.seg <<= 1;
  if (c.dtype == MOE_DTYPE_BF16) launch_route_t<__nv_bfloat16>(p, s);
  else launch_route_t<float>(p, s);
  return check_launch("route_kernel");
}

int32_t launch_route_backward(const moe_route_config& c, const void* logits,
                              const int32_t* expert_idx, const float* dgate, void* dlogits,
                              int32_t* status, cudaStream_t s) {
  if (c.T == 0) return MOE_OK;
  RouteBwdParams p{};
  p.T = c.T;
  p.E = c.E;
  p.k = c.k;
  p.sigmoid = c.score == MOE_SCORE_SIGMOID;
  p.renorm = c.renorm;
  p.scale = static_cast<float>(c.scale);
  p.logits = logits;
  p.idx = expert_idx;
  p.dgate = dgate;
  p.dlogits = dlogits;
  p.status = status;
  p.seg = 1;
  while (p.seg < c.k || p.seg * 8 < c.E) p.seg <<= 1;
  const bool vec = c.E % 4 == 0;
  if (c.dtype == MOE_DTYPE_BF16) {
    if (vec) launch_route_backward_t<__nv_bfloat16, 4>(p, s);
    else launch_route_backward_t<__nv_bfloat16, 1>(p, s);
  } else {
    if (vec) launch_route_backward_t<float, 4>(p, s);
    else launch_route_backward_t<float, 1>(p, s);
  }
  return check_launch("route_backward_kernel");
}

}  // namespace moe
