// Routing by scores: softmax or sigmoid scores, a balance bias that enters the
// choice only, group-limited top-k with k up to 16, weights renormalised over
// the choices; and its gradient.
//
//   s[t, e] = softmax_e(h[t, :]) or 1 / (1 + exp(-h[t, e])),  c = s + bias
//   a group's value = the sum of its group_top largest c; top_groups groups stay
//   choices = the k largest c of the groups that stay (ties -> lower expert)
//   w[t, j] = scale * s[t, e_j] / (renorm ? sum_i s[t, e_i] : 1)
//
// The order is that of the real numbers, not of their fp32 roundings: without
// a bias it is the logits' own order, and where fp32 cannot tell two
// candidates apart the token is decided again in fp64 (route_exact).
#include <cmath>

#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 8;  // warps per block, a token each
// A logit at or below bf16's lowest value masks its expert, as -inf does.
constexpr float kLowest = -3.3895313892515355e38f;
// Key units (see make_key) within which two candidates are not told apart.
// The fp32 score is off by less than 8 * 2^-24 (expf 2 ulp, a sum and a
// division on values <= 1), the sum with the bias and the scaling to the key
// by one unit each; two candidates and a margin give 16 units of 2^-24.
constexpr unsigned kNear = 16;

struct RouteParams {
  int64_t T;
  int E, k;
  int G, gs;        // groups that are told apart (1: no group limit), experts each
  int lanes;        // lanes per group: 32 / (G rounded up to a power of two)
  int top_groups, group_top;
  int sigmoid, renorm;
  int by_logit;     // the logits' order decides (no bias, no sum of two scores)
  float scale;
  const void* logits;
  const float* bias;
  int32_t* idx;
  float* gate;
  int32_t* status;
};

MOE_DEV float to_float(float v) { return v; }
MOE_DEV float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

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

// The token's choices decided in fp64: lane j < k returns choice j's expert, or
// -1.  buf: E doubles of this warp's shared memory.
template <typename L>
__device__ __noinline__ int route_exact(const RouteParams& p, int64_t t, double* buf) {
  const int lane = threadIdx.x & 31;
  const L* h = static_cast<const L*>(p.logits) + t * p.E;
  double m = -INFINITY, sum = 0.0;
  if (!p.by_logit && !p.sigmoid) {
    float mf = -INFINITY;
    for (int e = lane; e < p.E; e += 32) {
      const float x = to_float(h[e]);
      if (counts(x)) mf = fmaxf(mf, x);
    }
    m = warp_max(mf);
    for (int e = lane; e < p.E; e += 32) {
      const float x = to_float(h[e]);
      if (counts(x)) sum += exp(static_cast<double>(x) - m);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  }
  for (int e = lane; e < p.E; e += 32) {
    const float x = to_float(h[e]);
    double c = -INFINITY;
    if (counts(x)) {
      const double xd = x;
      if (p.by_logit) c = xd;
      else c = p.sigmoid ? 1.0 / (1.0 + exp(-xd)) : exp(xd - m) / sum;
      if (p.bias) {
        const float b = __ldg(p.bias + e);
        c = fabsf(b) < INFINITY ? c + static_cast<double>(b) : -INFINITY;
      }
    }
    buf[e] = c;
  }
  __syncwarp();
  unsigned stay = kFull;
  if (p.G > 1) {
    double v = -INFINITY;
    if (lane < p.G) {  // a group per lane
      double b1 = -INFINITY, b2 = -INFINITY;
      for (int i = 0; i < p.gs; ++i) {
        const double c = buf[lane * p.gs + i];
        if (c > b1) { b2 = b1; b1 = c; }
        else if (c > b2) b2 = c;
      }
      v = p.group_top == 2 && b2 > -INFINITY ? b1 + b2 : b1;
    }
    int rank = 0;
    for (int q = 0; q < p.G; ++q) {
      const double o = __shfl_sync(kFull, v, q);
      rank += o > v || (o == v && q < lane);
    }
    stay = __ballot_sync(kFull, lane < p.G && rank < p.top_groups);
  }
  int mine = -1;
  for (int j = 0; j < p.k; ++j) {
    double bv = -INFINITY;
    int be = -1;
    for (int e = lane; e < p.E; e += 32)
      if (((stay >> (p.G > 1 ? e / p.gs : 0)) & 1u) && buf[e] > bv) { bv = buf[e]; be = e; }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double ov = __shfl_xor_sync(kFull, bv, o);
      const int oe = __shfl_xor_sync(kFull, be, o);
      if (oe >= 0 && (be < 0 || ov > bv || (ov == bv && oe < be))) { bv = ov; be = oe; }
    }
    if (be < 0) break;  // the same in every lane: nothing is left
    if (lane == j) mine = be;
    __syncwarp();
    if (lane == 0) buf[be] = -INFINITY;
    __syncwarp();
  }
  __syncwarp();  // the buffer is free for the warp's next token
  return mine;
}

// Descending sort of N register values (N a power of two), a bitonic network.
template <int N>
MOE_DEV void sort_desc(uint32_t (&v)[N]) {
#pragma unroll
  for (int size = 2; size <= N; size <<= 1) {
#pragma unroll
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int j = i ^ stride;
        if (j > i) {
          const bool down = (i & size) == 0;
          const uint32_t hi = max(v[i], v[j]), lo = min(v[i], v[j]);
          v[i] = down ? hi : lo;
          v[j] = down ? lo : hi;
        }
      }
    }
  }
}

// A warp per token.  Lane l holds V logits of one group (of the whole row
// where there is no group limit).  Each candidate becomes a 32-bit key,
// (rounded value in 24 bits) << 8 | (255 - expert): unique, larger is better,
// ties in the value to the lower expert; 0 marks an expert that cannot be
// chosen.  A lane sorts its keys once, and each choice is one warp-wide integer
// maximum over the lanes' first keys.  The rounding to 24 bits is checked
// afterwards: neighbours in the order (and the last choice against the first
// one left out) that are within kNear units, and are not equal inputs, send
// the token to route_exact.
template <typename L, int V, int W>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(const __grid_constant__ RouteParams p) {
  __shared__ double s_buf[kWarps][256];
  dev::pdl_trigger();
  dev::pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int q = lane / p.lanes, li = lane & (p.lanes - 1);
  const int64_t nwarps = static_cast<int64_t>(gridDim.x) * kWarps;
  const L* logits = static_cast<const L*>(p.logits);
  constexpr bool kBf16 = sizeof(L) == 2;
  const bool exact_key = kBf16 && p.by_logit;  // a bf16 logit fits the key
  const bool has_bias = p.bias != nullptr;
  bool bad = false;

  // this lane's experts: offset(i) = (i / W) * lanes * W + li * W + i % W within group q
  const int first = q * p.gs;
  float b[V];
  float lo = 0.f, unit = 0.f;
  if (!p.by_logit) {
    float bmin = INFINITY, bmax = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int o = (i / W) * p.lanes * W + li * W + i % W;
      b[i] = 0.f;
      if (q < p.G && o < p.gs) {
        if (has_bias) b[i] = __ldg(p.bias + first + o);
        if (!(fabsf(b[i]) < INFINITY)) {
          if (!(b[i] < 0.f)) bad = true;  // NaN or +inf; -inf masks the expert
          b[i] = -INFINITY;
        } else {
          bmin = fminf(bmin, b[i]);
          bmax = fmaxf(bmax, b[i]);
        }
      }
    }
    lo = -warp_max(-bmin);
    unit = 16777213.0f / (1.0f + warp_max(bmax) - lo);
  }

  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp; t < p.T; t += nwarps) {
    const L* h = logits + t * p.E;
    float x[V];
#pragma unroll
    for (int c = 0; c < V / W; ++c) {
      const int o = c * p.lanes * W + li * W;
      if (q < p.G && o < p.gs) {
        load_logits<W>(h + first + o, x + c * W);
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i) x[c * W + i] = -INFINITY;
      }
    }
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (!counts(x[i])) {
        if (!(x[i] < 0.f)) bad = true;  // NaN or +inf
        x[i] = -INFINITY;
      }
      m = fmaxf(m, x[i]);
    }
    const bool softmax_sum = !p.sigmoid && (!p.by_logit || !p.renorm);
    float inv = 0.f;
    if (softmax_sum || (p.by_logit && !exact_key)) m = warp_max(m);
    uint32_t key[V];
    float s[V];
    if (softmax_sum) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        s[i] = x[i] > -INFINITY ? expf(x[i] - m) : 0.f;
        sum += s[i];
      }
      sum = warp_sum(sum);
      inv = sum > 0.f ? 1.0f / sum : 0.f;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = first + (i / W) * p.lanes * W + li * W + i % W;
      uint32_t v;
      bool can = x[i] > -INFINITY;
      if (exact_key) {  // the bits of a bf16 in ascending order, 1..65535
        const uint32_t u = __float_as_uint(x[i] + 0.f) >> 16;  // -0 is +0
        v = (u & 0x8000u ? 0xffffu ^ u : u | 0x8000u) + 1u;
      } else if (p.by_logit) {
        v = 1u + static_cast<uint32_t>(fmaxf(16777213.0f - (m - x[i]) * 524288.0f, 0.f));
      } else {
        const float sc = p.sigmoid ? 1.0f / (1.0f + expf(-x[i])) : s[i] * inv;
        can = can && b[i] > -INFINITY;
        v = 1u + static_cast<uint32_t>(fminf(fmaxf((sc + b[i] - lo) * unit, 0.f), 16777213.0f));
      }
      key[i] = can ? (v << 8) | static_cast<uint32_t>(255 - e) : 0u;
    }
    sort_desc<V>(key);

    bool unsure = false;
    if (p.G > 1) {
      uint32_t a1 = key[0], a2 = V > 1 ? key[V > 1 ? 1 : 0] : 0u;
      for (int o = 1; o < p.lanes; o <<= 1) {
        const uint32_t o1 = __shfl_xor_sync(kFull, a1, o), o2 = __shfl_xor_sync(kFull, a2, o);
        a2 = max(min(a1, o1), max(a2, o2));
        a1 = max(a1, o1);
      }
      uint32_t v = a1 >> 8;
      if (p.group_top == 2) {
        v += a2 >> 8;
        unsure = __any_sync(kFull, a1 != 0u && a2 == 0u);  // a sum of one: its offset differs
      }
      uint32_t g = a1 ? (v << 5) | static_cast<uint32_t>(31 - q) : 0u;
      bool stays = false;
      uint32_t last = 0u;
      for (int i = 0; i < p.top_groups; ++i) {
        last = __reduce_max_sync(kFull, g);
        if (g == last) {
          stays = true;
          g = 0u;
        }
      }
      const uint32_t next = __reduce_max_sync(kFull, g);
      if (!exact_key && next != 0u && (last >> 5) - (next >> 5) <= 2 * kNear) unsure = true;
      if (!stays) {
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = 0u;
      }
    }

    uint32_t mine = 0u, last = 0u;
    for (int j = 0; j < p.k; ++j) {
      last = __reduce_max_sync(kFull, key[0]);
      if (lane == j) mine = last;
      if (key[0] == last) {
#pragma unroll
        for (int i = 0; i + 1 < V; ++i) key[i] = key[i + 1];
        key[V - 1] = 0u;
      }
    }
    int e = mine ? 255 - static_cast<int>(mine & 255u) : -1;
    float xj = e >= 0 ? to_float(h[e]) : -INFINITY;
    if (!exact_key && !unsure) {
      const float bj = e >= 0 && has_bias ? __ldg(p.bias + e) : 0.f;
      const uint32_t after = __shfl_down_sync(kFull, mine, 1);
      const float xa = __shfl_down_sync(kFull, xj, 1), ba = __shfl_down_sync(kFull, bj, 1);
      const bool close = lane + 1 < p.k && after != 0u && (mine >> 8) - (after >> 8) <= kNear &&
                         !(xj == xa && bj == ba);
      unsure = __any_sync(kFull, close);
      if (last != 0u && !unsure) {
        // the last choice against what was left out, past those equal to it
        const float xl = __shfl_sync(kFull, xj, p.k - 1), bl = __shfl_sync(kFull, bj, p.k - 1);
        for (;;) {
          const uint32_t next = __reduce_max_sync(kFull, key[0]);
          if (next == 0u || (last >> 8) - (next >> 8) > kNear) break;
          const int en = 255 - static_cast<int>(next & 255u);
          if (to_float(h[en]) != xl || (has_bias && __ldg(p.bias + en) != bl)) {
            unsure = true;
            break;
          }
          if (key[0] == next) {
#pragma unroll
            for (int i = 0; i + 1 < V; ++i) key[i] = key[i + 1];
            key[V - 1] = 0u;
          }
        }
      }
    }
    if (unsure) {
      e = route_exact<L>(p, t, s_buf[warp]);
      xj = e >= 0 ? to_float(h[e]) : -INFINITY;
    }

    // weights: lane j holds choice j
    float w;
    if (p.renorm) {
      // scaled by the largest choice so that small scores keep their ratio
      const float mx = warp_max(xj);
      const float ref = p.sigmoid ? fminf(mx, 0.f) : mx;
      w = 0.f;
      if (xj > -INFINITY) {
        if (!p.sigmoid) w = expf(xj - ref);
        else w = xj >= 0.f ? 1.0f / (1.0f + expf(-xj)) : expf(xj - ref) / (1.0f + expf(xj));
      }
      const float sum = warp_sum(w);
      w = sum > 0.f ? p.scale * (w / sum) : 0.f;
    } else {
      w = 0.f;
      if (xj > -INFINITY)
        w = p.scale * (p.sigmoid ? 1.0f / (1.0f + expf(-xj)) : expf(xj - m) * inv);
    }
    if (lane < p.k) {
      p.idx[t * p.k + lane] = e;
      p.gate[t * p.k + lane] = w;
    }
  }
  if (__any_sync(kFull, bad) && lane == 0 && p.status) atomicOr(p.status, MOE_STATUS_BAD_LOGIT);
}

struct RouteBwdParams {
  int64_t T;
  int E, k;
  int sigmoid, renorm;
  float scale;
  const void* logits;
  const int32_t* idx;
  const float* dgate;
  void* dlogits;
  int32_t* status;
};

MOE_DEV void store_logit(float* p, float v) { *p = v; }
MOE_DEV void store_logit(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// A warp per token; lane j < k holds choice j.  The choices are constants of
// the gradient.  With a_j = scale * dw_j (summed over equal choices):
//   softmax:         dh_e = s_e (a_e - sum_i a_i s_i), every expert
//   softmax, renorm: dh_j = q_j (a_j - sum_i a_i q_i), q = the choices' softmax
//   sigmoid:         dh_j = a_j s_j (1 - s_j)
//   sigmoid, renorm: dh_j = q_j (1 - s_j)(a_j - sum_i a_i q_i), q_i = s_i / sum s
// The dense part of a row is written first and the chosen entries over it, by
// the same warp.
template <typename L>
__global__ void __launch_bounds__(kWarps * 32) route_backward_kernel(const RouteBwdParams p) {
  dev::pdl_trigger();
  dev::pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t nwarps = static_cast<int64_t>(gridDim.x) * kWarps;
  const bool dense = !p.sigmoid && !p.renorm;
  bool bad = false;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp; t < p.T; t += nwarps) {
    const L* h = static_cast<const L*>(p.logits) + t * p.E;
    L* out = static_cast<L*>(p.dlogits) + t * p.E;
    int e = -1;
    float a = 0.f, x = -INFINITY;
    if (lane < p.k) {
      e = __ldg(p.idx + t * p.k + lane);
      if (e < -1 || e >= p.E) bad = true;
      if (e < 0 || e >= p.E) e = -1;
      if (e >= 0) {
        a = p.scale * __ldg(p.dgate + t * p.k + lane);
        x = to_float(h[e]);
        if (!counts(x)) {
          e = -1;
          a = 0.f;
          x = -INFINITY;
        }
      }
    }
    float d = 0.f;
    if (dense) {
      float m = -INFINITY;
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int o = lane + 32 * i;
        v[i] = o < p.E ? to_float(h[o]) : -INFINITY;
        if (!counts(v[i])) v[i] = -INFINITY;
        m = fmaxf(m, v[i]);
      }
      m = warp_max(m);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = v[i] > -INFINITY ? expf(v[i] - m) : 0.f;
        sum += v[i];
      }
      sum = warp_sum(sum);
      const float inv = sum > 0.f ? 1.0f / sum : 0.f;
      const float s = e >= 0 ? expf(x - m) * inv : 0.f;
      const float dot = warp_sum(a * s);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int o = lane + 32 * i;
        if (o < p.E) store_logit(out + o, -(v[i] * inv) * dot);
      }
      float all = 0.f;  // a summed over choices of the same expert
      for (int j = 0; j < p.k; ++j) {
        const float aj = __shfl_sync(kFull, a, j);
        if (__shfl_sync(kFull, e, j) == e) all += aj;
      }
      d = s * (all - dot);
    } else {
      for (int o = lane; o < p.E; o += 32) store_logit(out + o, 0.f);
      float s = 0.f, slope = 1.f;
      const float mx = warp_max(x);
      if (p.sigmoid) {
        const float ref = p.renorm ? fminf(mx, 0.f) : 0.f;
        if (e >= 0) {
          s = x >= 0.f ? 1.0f / (1.0f + expf(-x)) : expf(x - ref) / (1.0f + expf(x));
          slope = x >= 0.f ? expf(-x) / (1.0f + expf(-x)) : 1.0f / (1.0f + expf(x));
        }
      } else if (e >= 0) {
        s = expf(x - mx);
      }
      float part = 0.f;
      if (p.renorm) {
        const float sum = warp_sum(s);
        s = sum > 0.f ? s / sum : 0.f;
        const float dot = warp_sum(a * s);
        part = s * slope * (a - dot);
      } else {
        part = a * s * slope;
      }
      for (int j = 0; j < p.k; ++j) {  // choices of the same expert add up
        const float pj = __shfl_sync(kFull, part, j);
        if (__shfl_sync(kFull, e, j) == e) d += pj;
      }
    }
    __syncwarp();  // the row's dense part is written before its chosen entries
    if (e >= 0) store_logit(out + e, d);
  }
  if (__any_sync(kFull, bad) && lane == 0 && p.status) atomicOr(p.status, MOE_STATUS_BAD_INDEX);
}

template <typename L, int V>
void launch_route_v(const RouteParams& p, bool vec, unsigned grid, cudaStream_t s) {
  if constexpr (V >= 4) {
    if (vec) {
      launch_pdl(route_kernel<L, V, 4>, dim3(grid), dim3(kWarps * 32), 0, s, p);
      return;
    }
  }
  launch_pdl(route_kernel<L, V, 1>, dim3(grid), dim3(kWarps * 32), 0, s, p);
}

template <typename L>
void launch_route_t(const RouteParams& p, unsigned grid, cudaStream_t s) {
  const bool vec = p.gs % 4 == 0;
  const int per = vec ? (p.gs + 4 * p.lanes - 1) / (4 * p.lanes) * 4
                      : (p.gs + p.lanes - 1) / p.lanes;
  if (per <= 1) launch_route_v<L, 1>(p, false, grid, s);
  else if (per <= 2) launch_route_v<L, 2>(p, false, grid, s);
  else if (per <= 4) launch_route_v<L, 4>(p, vec, grid, s);
  else if (per <= 8) launch_route_v<L, 8>(p, vec, grid, s);
  else launch_route_v<L, 16>(p, vec, grid, s);
}

unsigned token_grid(int64_t T, int blocks_per_sm) {
  const int64_t want = (T + kWarps - 1) / kWarps;
  const int64_t most = static_cast<int64_t>(num_sms()) * blocks_per_sm;
  return static_cast<unsigned>(want < most ? want : most);
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
  const unsigned grid = token_grid(c.T, 8);
  if (c.dtype == MOE_DTYPE_BF16) launch_route_t<__nv_bfloat16>(p, grid, s);
  else launch_route_t<float>(p, grid, s);
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
  const unsigned grid = token_grid(c.T, 8);
  if (c.dtype == MOE_DTYPE_BF16)
    launch_pdl(route_backward_kernel<__nv_bfloat16>, dim3(grid), dim3(kWarps * 32), 0, s, p);
  else
    launch_pdl(route_backward_kernel<float>, dim3(grid), dim3(kWarps * 32), 0, s, p);
  return check_launch("route_backward_kernel");
}

}  // namespace moe
