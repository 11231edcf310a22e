// AdamW over many tensors in one call, with the moments in fp32 or in 8 bits,
// the gradients scaled by the SparseClip coefficient as they are read.
//
//   c  = min(1, max_norm / norm)                (norm: a device double, or c = 1)
//   m  = b1 m + (1 - b1) c g
//   v  = b2 v + (1 - b2) (c g)^2
//   p -= lr wd p + lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// 8-bit moments: every 256 consecutive elements of a tensor share one fp32
// scale per moment.  m is kept as e4m3 codes of m / scale with scale =
// max|m| / 448; v as e4m3 codes of sqrt(v) / scale, scale = max sqrt(v) / 448,
// so that its 18 binades cover 36 of v; a v > 0 never falls below the
// smallest code: a step divided by a second moment that was rounded to zero
// would be unbounded, one divided by a moment rounded up is only shorter.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <new>
#include <type_traits>
#include <vector>

#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kQBlock = 256;         // elements per scale: 8 per lane of one warp
constexpr int kRound = 2048;         // elements per block and round: 8 per thread
// A chunk of a tensor is what a block (fp32 moments) or a warp (8-bit) takes at a
// time: long where there are enough chunks for all of them, short where small
// tensors would leave SMs idle.
constexpr int kLongChunk = 4 * kRound;
constexpr int kLongChunk8 = 8 * kQBlock, kShortChunk8 = kQBlock;
constexpr int kMaxTensors = 4096;
// Tensors in a launch's parameter block: the large one is 26 KB of the 32 KB limit, and
// a launch copies all of it.
constexpr int kSmallBatch = 24, kMiddleBatch = 128, kLargeBatch = 384;
// An |m| maximum below this stores the block's m as zeros: its scale's
// reciprocal would leave fp32's range.
constexpr float kTiny = 1e-30f;

struct AdamTensor {
  float* p;
  const void* g;
  void* m;
  void* v;
  float* ms;
  float* vs;
  __nv_bfloat16* copy;
  int64_t len;
};

struct AdamHyper {
  float b1, nb1, b2, nb2, eps;      // nb = 1 - b, rounded from the double
  float one;                        // 1 (see add)
  float decay, rate, root;          // from the host's step and lr (see StepScalars)
  double wd;                        // the rest for the device's own
  double beta1, beta2;
  double max_norm;
  const double* norm;               // nullable
  const double* step_lr;            // nullable: {step, lr} on the device
  int32_t* status;
};

template <int N>
struct AdamBatch {
  AdamTensor t[N];
  int32_t first[N + 1];             // first chunk of each tensor; first[n] = chunks in all
  int32_t n;
  int32_t chunk;                    // elements per chunk
};

struct StepScalars {
  float clip, decay, rate, root;    // root = 1 / sqrt(1 - b2^t)
  int skip;
};

MOE_DEV float sqrt_fast(float x) {
  // off by at most 2^-23 relative, which changes the length of a step by as much
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

MOE_DEV float rcp_fast(float x) {  // 1 unit in the last place; x >= eps, a normal number
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// p, m, v (fp32) -> their next values
MOE_DEV void adam_one(float& p, float g, float& m, float& v, const AdamHyper& h,
                      const StepScalars& s) {
  g *= s.clip;
  m = fmaf(h.b1, m, h.nb1 * g);
  v = fmaf(h.b2, v, h.nb2 * g * g);
  p = fmaf(-s.rate, m * rcp_fast(fmaf(sqrt_fast(v), s.root, h.eps)), p * s.decay);
}

// (packed arithmetic: half the issue slots, and under the power cap the step's speed
// goes by its instructions)
using dev::Pair;
using dev::both;
using dev::fma2;
using dev::halves;
using dev::mul2;
using dev::pair;

// a + b, as a * one + b with a 1 that the compiler does not see: it contracts a packed
// add of a packed product, and a * 1.0f + b just so, into one fused operation in
// spite of the .rn (found as different last bits of the moments).
MOE_DEV Pair add(Pair a, Pair b, const AdamHyper& h) { return fma2(a, both(h.one), b); }

// The moments that are about to be rounded to 8 bits; v goes from sqrt(v) to v.
// A code is a step of 6 to 12 percent, so one that falls on the other side of a
// rounding border moves the next step visibly: every product and sum here is
// rounded by itself, as the formula is written, and the codes do not depend on
// how a compiler contracts it.  (The root is sqrtf's for the same reason; the fp32
// moments take the approximate one.)
MOE_DEV void moments8(Pair g, Pair& m, Pair& v, const AdamHyper& h, const StepScalars& s) {
  g = mul2(g, both(s.clip));
  m = add(mul2(both(h.b1), m), mul2(both(h.nb1), g), h);
  v = add(mul2(both(h.b2), mul2(v, v)), mul2(mul2(both(h.nb2), g), g), h);
}

// a / b rounded to nearest from inv = 1 / b rounded to nearest (Markstein, "Computation
// of elementary functions on the IBM RISC System/6000 processor", 1990): one
// reciprocal serves a whole block.  Exact while a's residual is representable,
// a > 1e-31; below that the codes may be off by one.
MOE_DEV Pair quotient(Pair a, float b, float inv) {
  const Pair q = mul2(a, both(inv));
  return fma2(fma2(q, both(-b), a), both(inv), q);
}

MOE_DEV Pair step_param(Pair p, Pair m, Pair r, const AdamHyper& h, const StepScalars& s) {
  const float2 d = halves(fma2(r, both(s.root), both(h.eps)));
  const Pair u = mul2(m, pair(rcp_fast(d.x), rcp_fast(d.y)));
  return fma2(both(-s.rate), u, mul2(p, both(s.decay)));
}

MOE_DEV void load4(const float* p, float (&f)[4]) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
}
MOE_DEV void load4(const __nv_bfloat16* p, float (&f)[4]) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  f[0] = __uint_as_float(v.x << 16); f[1] = __uint_as_float(v.x & 0xffff0000u);
  f[2] = __uint_as_float(v.y << 16); f[3] = __uint_as_float(v.y & 0xffff0000u);
}
MOE_DEV void store4(float* p, const float (&f)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
}
MOE_DEV void store4(__nv_bfloat16* p, const float (&f)[4]) {
  __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
  *reinterpret_cast<uint2*>(p) =
      make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
}
MOE_DEV float load1(const float* p) { return *p; }
MOE_DEV float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// four e4m3 codes <-> four floats
MOE_DEV void of_e4m3x4(uint32_t q, float (&f)[4]) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(q));
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f[0]), "=f"(f[1])
      : "r"(lo));
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f[2]), "=f"(f[3])
      : "r"(hi));
}
MOE_DEV uint32_t to_e4m3x4(const float (&f)[4]) {
  uint32_t q;
  asm("{\n\t.reg .b16 a, b;\n\tcvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\tmov.b32 %0, {a, b};\n\t}"
      : "=r"(q)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]));
  return q;
}

struct Rates {
  float decay, rate, root;
};
// In fp64: 1 - b^t loses its leading digits for b near 1 and small t.
__host__ __device__ inline Rates step_rates(double t, double lr, double wd, double beta1, double beta2) {
  return Rates{static_cast<float>(1.0 - lr * wd), static_cast<float>(lr / (1.0 - pow(beta1, t))),
               static_cast<float>(1.0 / sqrt(1.0 - pow(beta2, t)))};
}

// The step's scalars, the same in every block: the host's, unless the norm or the
// step come from the device.  Every thread of the block calls it.
MOE_DEV StepScalars step_scalars(const AdamHyper& h, StepScalars* shared) {
  if (!h.norm && !h.step_lr) return StepScalars{1.0f, h.decay, h.rate, h.root, 0};
  if (threadIdx.x == 0) {
    StepScalars s{1.0f, h.decay, h.rate, h.root, 0};
    if (h.step_lr) {
      const double t = h.step_lr[0], lr = h.step_lr[1];
      if (!(t >= 1.0) || !isfinite(t) || !isfinite(lr)) s.skip = 1;
      const Rates r = step_rates(t, lr, h.wd, h.beta1, h.beta2);
      s.decay = r.decay;
      s.rate = r.rate;
      s.root = r.root;
    }
    if (h.norm) {
      const double n = *h.norm;
      if (!isfinite(n)) s.skip = 1;
      if (n > h.max_norm) s.clip = static_cast<float>(h.max_norm / n);
    }
    *shared = s;
  }
  __syncthreads();
  return *shared;
}

// tensor of chunk c (last i with first[i] <= c)
template <int N>
MOE_DEV int tensor_of(const AdamBatch<N>& b, int c) {
  int lo = 0, hi = b.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (b.first[mid] <= c) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// In a round thread i takes the 4 elements at 4 i and the 4 at 1024 + 4 i, so that
// every load of a warp is one contiguous run; 8 loads in flight a thread and five
// blocks an SM (48 registers; with 59 and four it was 909 us) keep HBM busy: 184 M
// parameters with a bf16 copy, 5.5 GB, 872 us, 0.97 of the copy rate.
template <typename G, int N>
__global__ void __launch_bounds__(kThreads, 5)
adamw_kernel(const __grid_constant__ AdamBatch<N> b, const AdamHyper h) {
  __shared__ StepScalars s_step;
  dev::pdl_trigger();
  dev::pdl_wait();
  const StepScalars s = step_scalars(h, &s_step);
  if (s.skip) {
    if (blockIdx.x == 0 && threadIdx.x == 0 && h.status) atomicOr(h.status, MOE_STATUS_NONFINITE);
    return;
  }
  for (int c = blockIdx.x; c < b.first[b.n]; c += gridDim.x) {
    const int n = tensor_of(b, c);
    const AdamTensor& t = b.t[n];
    const int64_t chunk = static_cast<int64_t>(c - b.first[n]) * b.chunk;
    const int64_t end = min(chunk + b.chunk, t.len);
    float* p = t.p;
    const G* g = static_cast<const G*>(t.g);
    float* m = static_cast<float*>(t.m);
    float* v = static_cast<float*>(t.v);
    int64_t base = chunk;
    for (; base + kRound <= end; base += kRound) {
      float fp[2][4], fg[2][4], fm[2][4], fv[2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int64_t i = base + u * (kThreads * 4) + threadIdx.x * 4;
        load4(p + i, fp[u]);
        load4(g + i, fg[u]);
        load4(m + i, fm[u]);
        load4(v + i, fv[u]);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int64_t i = base + u * (kThreads * 4) + threadIdx.x * 4;
#pragma unroll
        for (int k = 0; k < 4; ++k) adam_one(fp[u][k], fg[u][k], fm[u][k], fv[u][k], h, s);
        store4(p + i, fp[u]);
        store4(m + i, fm[u]);
        store4(v + i, fv[u]);
        if (t.copy) store4(t.copy + i, fp[u]);
      }
    }
    for (int64_t i = base + threadIdx.x; i < end; i += kThreads) {
      float x = p[i], y = m[i], z = v[i];
      adam_one(x, load1(g + i), y, z, h, s);
      p[i] = x;
      m[i] = y;
      v[i] = z;
      if (t.copy) t.copy[i] = __float2bfloat16_rn(x);
    }
  }
}

// 8-bit moments: a warp owns the 256 elements of one scale, 4 at 4 l and 4 at
// 128 + 4 l per lane l.
template <typename G>
struct Block8 {
  float p[2][4], g[2][4];
  uint32_t qm[2], qv[2];
  float ms, vs;

  // p, the codes and the scales of the next step
  MOE_DEV void step(const AdamHyper& h, const StepScalars& s) {
    Pair m[4], r[4];  // of elements 2 k, 2 k + 1 of the lane's eight
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float dm[4], dr[4];
      of_e4m3x4(qm[u], dm);
      of_e4m3x4(qv[u], dr);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        Pair& mk = m[2 * u + k];
        Pair& rk = r[2 * u + k];
        mk = mul2(pair(dm[2 * k], dm[2 * k + 1]), both(ms));
        rk = mul2(pair(dr[2 * k], dr[2 * k + 1]), both(vs));
        moments8(pair(g[u][2 * k], g[u][2 * k + 1]), mk, rk, h, s);
        const float2 v = halves(rk);
        rk = pair(sqrtf(v.x), sqrtf(v.y));
      }
    }
    // magnitudes keep their order as integers, and a NaN is above all of them
    uint32_t bits_m = 0u, bits_r = 0u;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float* pk = &p[k / 2][2 * (k % 2)];
      const float2 np = halves(step_param(pair(pk[0], pk[1]), m[k], r[k], h, s));
      pk[0] = np.x;
      pk[1] = np.y;
      const float2 fm = halves(m[k]), fr = halves(r[k]);
      bits_m = max(bits_m, max(__float_as_uint(fabsf(fm.x)), __float_as_uint(fabsf(fm.y))));
      bits_r = max(bits_r, max(__float_as_uint(fr.x), __float_as_uint(fr.y)));
    }
    const float top_m = __uint_as_float(__reduce_max_sync(0xffffffffu, bits_m));
    const float top_r = __uint_as_float(__reduce_max_sync(0xffffffffu, bits_r) & 0x7fffffffu);
    // (a NaN fails the comparison: it becomes the scale)
    ms = top_m < kTiny ? 0.f : top_m * (1.0f / 448.0f);
    vs = top_r * (1.0f / 448.0f);
    const float im = ms == 0.f ? 0.f : __frcp_rn(ms);
    const float ir = vs == 0.f ? 0.f : __frcp_rn(vs);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float cm[4], cr[4];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float2 fm = halves(quotient(m[2 * u + k], ms, im));
        const float2 fr = halves(quotient(r[2 * u + k], vs, ir));
        const float2 old = halves(r[2 * u + k]);
        cm[2 * k] = fm.x;
        cm[2 * k + 1] = fm.y;
        // 2^-9, the smallest code, unless v is 0
        cr[2 * k] = fmaxf(fr.x, old.x > 0.f ? 0.001953125f : 0.f);
        cr[2 * k + 1] = fmaxf(fr.y, old.y > 0.f ? 0.001953125f : 0.f);
      }
      qm[u] = to_e4m3x4(cm);
      qv[u] = to_e4m3x4(cr);
    }
  }

  // a block behind whose 256 elements the tensor ends: one element at a time
  MOE_DEV void load_tail(const AdamTensor& t, int64_t base, int lane) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      qm[u] = qv[u] = 0u;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t i = base + u * 128 + lane * 4 + k;
        p[u][k] = g[u][k] = 0.f;
        if (i < t.len) {
          p[u][k] = t.p[i];
          g[u][k] = load1(static_cast<const G*>(t.g) + i);
          qm[u] |= static_cast<uint32_t>(static_cast<const uint8_t*>(t.m)[i]) << (8 * k);
          qv[u] |= static_cast<uint32_t>(static_cast<const uint8_t*>(t.v)[i]) << (8 * k);
        }
      }
    }
  }

  MOE_DEV void store(const AdamTensor& t, int64_t base, int lane) const {
    uint8_t* m_ = static_cast<uint8_t*>(t.m);
    uint8_t* v_ = static_cast<uint8_t*>(t.v);
    const bool full = base + kQBlock <= t.len;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t i = base + u * 128 + lane * 4;
      if (full) {
        store4(t.p + i, p[u]);
        *reinterpret_cast<uint32_t*>(m_ + i) = qm[u];
        *reinterpret_cast<uint32_t*>(v_ + i) = qv[u];
        if (t.copy) store4(t.copy + i, p[u]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (i + k < t.len) {
            t.p[i + k] = p[u][k];
            m_[i + k] = static_cast<uint8_t>(qm[u] >> (8 * k));
            v_[i + k] = static_cast<uint8_t>(qv[u] >> (8 * k));
            if (t.copy) t.copy[i + k] = __float2bfloat16_rn(p[u][k]);
          }
        }
      }
    }
  }
};

template <int BYTES>
MOE_DEV void copy_async(void* smem, const void* global) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dev::smem_u32(smem)), "l"(global),
               "n"(BYTES)
               : "memory");
}
MOE_DEV void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
MOE_DEV void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory"); }

// The arithmetic on a block takes as long as its loads, and loads held in registers
// would leave too few warps to overlap them.  So a thread copies its part of the
// next block into its own places in shared memory (asynchronous copies, waited
// for by the thread that issued them: no barrier) while it works on one.
template <typename G>
struct Stage8 {
  float4 p[2][kThreads];
  typename std::conditional<sizeof(G) == 4, float4, uint2>::type g[2][kThreads];
  uint32_t m[2][kThreads], v[2][kThreads];
};

// A warp takes a chunk of up to 8 consecutive blocks: their scales are one
// 32-byte sector, loaded and stored at once by 8 lanes.  (One 4-byte store per
// block cost 80 of 522 us on 184 M parameters: partial sectors.)  With bf16
// gradients, 2.6 GB: 440 us at full clocks, 0.9 of the copy rate; issue-bound (0.75 of
// the slots), and 490 once the board's power cap lowers the clock.
template <typename G, int N>
__global__ void __launch_bounds__(kThreads, 3)
adamw8_kernel(const __grid_constant__ AdamBatch<N> b, const AdamHyper h) {
  extern __shared__ __align__(16) uint8_t s_mem[];
  Stage8<G>* stage = reinterpret_cast<Stage8<G>*>(s_mem);  // [2]
  __shared__ StepScalars s_step;
  dev::pdl_trigger();
  dev::pdl_wait();
  const StepScalars s = step_scalars(h, &s_step);
  if (s.skip) {
    if (blockIdx.x == 0 && threadIdx.x == 0 && h.status) atomicOr(h.status, MOE_STATUS_NONFINITE);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 31;
  const int stride = gridDim.x * (kThreads / 32);
  const int chunks = b.first[b.n];
  const int run = b.chunk / kQBlock;  // 8 or 1

  // a place in the warp's sequence of blocks
  struct Place {
    int c, n, i;        // chunk, its tensor, block in the chunk
    int64_t start, end;  // elements of the chunk in the tensor
  };
  auto enter = [&](Place& q) {  // chunk q.c; the tensors are met in order
    if (q.c >= chunks) return;
    while (b.first[q.n + 1] <= q.c) ++q.n;
    q.i = 0;
    q.start = static_cast<int64_t>(q.c - b.first[q.n]) * b.chunk;
    q.end = min(q.start + b.chunk, b.t[q.n].len);
  };
  auto advance = [&](Place& q) {
    if (q.start + (++q.i) * kQBlock < q.end) return;
    q.c += stride;
    enter(q);
  };
  Place ahead{static_cast<int>(blockIdx.x) * (kThreads / 32) + (tid >> 5), 0, 0, 0, 0};
  enter(ahead);
  Place now = ahead;
  float ms_ahead = 0.f, vs_ahead = 0.f;  // lane i: scale of the chunk's block i
  auto fetch = [&](Stage8<G>& st) {
    if (ahead.c < chunks) {
      const AdamTensor& t = b.t[ahead.n];
      if (ahead.i == 0 && lane < run && ahead.start + lane * kQBlock < ahead.end) {
        ms_ahead = t.ms[ahead.start / kQBlock + lane];
        vs_ahead = t.vs[ahead.start / kQBlock + lane];
      }
      const int64_t base = ahead.start + ahead.i * kQBlock;
      if (base + kQBlock <= t.len) {
        const int64_t i = base + lane * 4;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          copy_async<16>(&st.p[u][tid], t.p + i + u * 128);
          copy_async<sizeof(st.g[u][tid])>(&st.g[u][tid], static_cast<const G*>(t.g) + i + u * 128);
          copy_async<4>(&st.m[u][tid], static_cast<const uint8_t*>(t.m) + i + u * 128);
          copy_async<4>(&st.v[u][tid], static_cast<const uint8_t*>(t.v) + i + u * 128);
        }
      }
      advance(ahead);
    }
    copy_commit();
  };
  fetch(stage[0]);
  float ms = 0.f, vs = 0.f;
  for (int slot = 0; now.c < chunks; slot ^= 1) {
    if (now.i == 0) {
      ms = ms_ahead;
      vs = vs_ahead;
    }
    fetch(stage[slot ^ 1]);
    copy_wait<1>();
    const AdamTensor& t = b.t[now.n];
    const int64_t base = now.start + now.i * kQBlock;
    Block8<G> x;
    if (base + kQBlock <= t.len) {
      const Stage8<G>& st = stage[slot];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        load4(reinterpret_cast<const float*>(&st.p[u][tid]), x.p[u]);
        load4(reinterpret_cast<const G*>(&st.g[u][tid]), x.g[u]);
        x.qm[u] = st.m[u][tid];
        x.qv[u] = st.v[u][tid];
      }
    } else {
      x.load_tail(t, base, lane);
    }
    x.ms = __shfl_sync(0xffffffffu, ms, now.i);
    x.vs = __shfl_sync(0xffffffffu, vs, now.i);
    x.step(h, s);
    x.store(t, base, lane);
    if (lane == now.i) {
      ms = x.ms;
      vs = x.vs;
    }
    if (base + kQBlock >= now.end && lane <= now.i) {
      t.ms[now.start / kQBlock + lane] = ms;
      t.vs[now.start / kQBlock + lane] = vs;
    }
    advance(now);
  }
  copy_wait<0>();
}

struct Lists {
  const int64_t* len;
  float* const* param;
  const void* const* grad;
  void* const* m;
  void* const* v;
  float* const* ms;
  float* const* vs;
  void* const* copy;
};

int32_t bad_arg(const std::string& what) {
  return fail(MOE_ERR_INVALID_ARGUMENT, "moe_adamw: " + what);
}

int32_t check_lists(const moe_adamw_config* c, int32_t n, const Lists& l) {
  if (!c) return bad_arg("config is null");
  if (n < 0) return bad_arg("negative tensor count");
  if (n > kMaxTensors)
    return fail(MOE_ERR_UNSUPPORTED, "moe_adamw: more than " + std::to_string(kMaxTensors) + " tensors");
  if (c->grad_dtype != MOE_DTYPE_BF16 && c->grad_dtype != MOE_DTYPE_F32)
    return bad_arg("unknown gradient dtype");
  if (c->state_bits != 32 && c->state_bits != 8) return bad_arg("state_bits must be 32 or 8");
  if (n > 0 && (!l.len || !l.param || !l.grad || !l.m || !l.v)) return bad_arg("null tensor array");
  if (n > 0 && c->state_bits == 8 && (!l.ms || !l.vs)) return bad_arg("null scale array");
  int64_t chunks = 0;
  for (int32_t i = 0; i < n; ++i) {
    if (l.len[i] < 0) return bad_arg("negative length");
    if (l.len[i] == 0) continue;
    const void* need[6] = {l.param[i], l.grad[i], l.m[i], l.v[i],
                           c->state_bits == 8 ? l.ms[i] : l.param[i],
                           c->state_bits == 8 ? l.vs[i] : l.param[i]};
    for (int q = 0; q < 4; ++q) {
      if (!need[q]) return bad_arg("null tensor");
      if (!aligned16(need[q])) return fail(MOE_ERR_ALIGNMENT, "moe_adamw: tensor not 16-byte aligned");
    }
    for (int q = 4; q < 6; ++q) {
      if (!need[q]) return bad_arg("null scales");
      if (reinterpret_cast<uintptr_t>(need[q]) & 3u)
        return fail(MOE_ERR_ALIGNMENT, "moe_adamw: scales not 4-byte aligned");
    }
    if (l.copy && l.copy[i] && !aligned16(l.copy[i]))
      return fail(MOE_ERR_ALIGNMENT, "moe_adamw: bf16 copy not 16-byte aligned");
    chunks += (l.len[i] + kRound - 1) / kRound;  // (the short 8-bit chunk is not used for that many)
    if (chunks > (1 << 30)) return fail(MOE_ERR_UNSUPPORTED, "moe_adamw: more than 2^41 elements");
  }
  return MOE_OK;
}

int32_t check_hyper(const moe_adamw_config* c, const double* norm, const double* step_lr) {
  auto fraction = [](double b) { return b >= 0.0 && b < 1.0; };
  if (!fraction(c->beta1) || !fraction(c->beta2)) return bad_arg("beta outside [0, 1)");
  // 0 / 0 for a parameter whose gradients were all zero
  if (!(c->eps >= FLT_MIN) || !(c->eps <= FLT_MAX)) return bad_arg("eps must be a normal positive fp32 number");
  if (!(c->weight_decay >= 0.0) || !std::isfinite(c->weight_decay))
    return bad_arg("weight_decay must be >= 0 and finite");
  if (!step_lr && (c->step < 1 || !std::isfinite(c->lr))) return bad_arg("step must be >= 1, lr finite");
  if (norm && (!(c->max_norm > 0.0) || !std::isfinite(c->max_norm)))
    return bad_arg("max_norm must be positive and finite");
  for (const double* q : {norm, step_lr})
    if (reinterpret_cast<uintptr_t>(q) & 7u)
      return fail(MOE_ERR_ALIGNMENT, "moe_adamw: norm / step_lr not 8-byte aligned");
  return MOE_OK;
}

template <typename G, int N>
void launch_batch(const AdamBatch<N>& b, const AdamHyper& h, bool bits8, cudaStream_t s) {
  const int chunks = b.first[b.n];
  if (bits8) {
    constexpr size_t kSmem = 2 * sizeof(Stage8<G>);
    const int blocks = (chunks + kThreads / 32 - 1) / (kThreads / 32);
    const dim3 grid(static_cast<unsigned>(std::min(blocks, num_sms() * 3)));
    cudaFuncSetAttribute(adamw8_kernel<G, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
    launch_pdl(adamw8_kernel<G, N>, grid, dim3(kThreads), kSmem, s, b, h);
    return;
  }
  const dim3 grid(static_cast<unsigned>(std::min(chunks, num_sms() * 8)));
  launch_pdl(adamw_kernel<G, N>, grid, dim3(kThreads), 0, s, b, h);
}

template <int N>
int32_t run_batches(const moe_adamw_config& c, int32_t n, const Lists& l, const AdamHyper& h,
                    cudaStream_t s) {
  AdamBatch<N> b;
  const bool bits8 = c.state_bits == 8;
  int64_t all = 0;
  for (int32_t i = 0; i < n; ++i) all += l.len[i];
  if (bits8) b.chunk = all >= static_cast<int64_t>(num_sms()) * 64 * kLongChunk8 ? kLongChunk8 : kShortChunk8;
  else b.chunk = all >= static_cast<int64_t>(num_sms()) * 32 * kLongChunk ? kLongChunk : kRound;
  for (int32_t i = 0; i < n;) {
    b.n = 0;
    b.first[0] = 0;
    for (; i < n && b.n < N; ++i) {
      if (l.len[i] == 0) continue;
      b.t[b.n] = AdamTensor{l.param[i], l.grad[i], l.m[i], l.v[i], bits8 ? l.ms[i] : nullptr,
                            bits8 ? l.vs[i] : nullptr,
                            l.copy ? static_cast<__nv_bfloat16*>(l.copy[i]) : nullptr, l.len[i]};
      b.first[b.n + 1] = b.first[b.n] + static_cast<int32_t>((l.len[i] + b.chunk - 1) / b.chunk);
      ++b.n;
    }
    if (b.n == 0) break;
    if (c.grad_dtype == MOE_DTYPE_BF16) launch_batch<__nv_bfloat16, N>(b, h, bits8, s);
    else launch_batch<float, N>(b, h, bits8, s);
    const int32_t rc = check_launch("adamw_kernel");
    if (rc != MOE_OK) return rc;
  }
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_adamw_config_size(void) { return sizeof(moe_adamw_config); }

extern "C" int32_t moe_adamw_check(const moe_adamw_config* cfg, int32_t n, const int64_t* len,
                                   float* const* param, const void* const* grad, void* const* m,
                                   void* const* v, float* const* m_scale, float* const* v_scale,
                                   void* const* bf16_copy) {
  set_last_error("");
  const Lists l{len, param, grad, m, v, m_scale, v_scale, bf16_copy};
  int32_t rc = check_lists(cfg, n, l);
  if (rc != MOE_OK) return rc;
  // what the step writes must not overlap anything else it reads or writes
  struct Range {
    uintptr_t lo, hi;
    bool written;
  };
  std::vector<Range> r;
  try {
    r.reserve(7 * static_cast<size_t>(n));
  } catch (const std::bad_alloc&) {
    return bad_arg("no host memory for the check");
  }
  const bool bits8 = cfg->state_bits == 8;
  const int64_t es = bits8 ? 1 : 4;
  auto add = [&](const void* q, int64_t bytes, bool written) {
    if (q) r.push_back(Range{reinterpret_cast<uintptr_t>(q), reinterpret_cast<uintptr_t>(q) + bytes, written});
  };
  for (int32_t i = 0; i < n; ++i) {
    if (len[i] == 0) continue;
    add(param[i], 4 * len[i], true);
    add(grad[i], (cfg->grad_dtype == MOE_DTYPE_BF16 ? 2 : 4) * len[i], false);
    add(m[i], es * len[i], true);
    add(v[i], es * len[i], true);
    if (bits8) {
      const int64_t blocks = (len[i] + kQBlock - 1) / kQBlock;
      add(m_scale[i], 4 * blocks, true);
      add(v_scale[i], 4 * blocks, true);
    }
    if (bf16_copy) add(bf16_copy[i], 2 * len[i], true);
  }
  std::sort(r.begin(), r.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
  uintptr_t end_any = 0, end_written = 0;
  for (const Range& q : r) {
    if (q.lo < (q.written ? end_any : end_written))
      return bad_arg("a tensor that the step writes overlaps another one");
    end_any = std::max(end_any, q.hi);
    if (q.written) end_written = std::max(end_written, q.hi);
  }
  return MOE_OK;
}

extern "C" int32_t moe_adamw_step(const moe_adamw_config* cfg, int32_t n, const int64_t* len,
                                  float* const* param, const void* const* grad, void* const* m,
                                  void* const* v, float* const* m_scale, float* const* v_scale,
                                  void* const* bf16_copy, const double* norm,
                                  const double* step_lr, int32_t* status, moe_stream_t stream) {
  CallRange range_("moe_adamw_step");
  set_last_error("");
  const Lists l{len, param, grad, m, v, m_scale, v_scale, bf16_copy};
  int32_t rc = check_lists(cfg, n, l);
  if (rc != MOE_OK) return rc;
  rc = check_hyper(cfg, norm, step_lr);
  if (rc != MOE_OK) return rc;
  AdamHyper h{};
  h.b1 = static_cast<float>(cfg->beta1);
  h.nb1 = static_cast<float>(1.0 - cfg->beta1);
  h.b2 = static_cast<float>(cfg->beta2);
  h.nb2 = static_cast<float>(1.0 - cfg->beta2);
  h.eps = static_cast<float>(cfg->eps);
  h.one = 1.0f;
  if (!step_lr) {
    const Rates r = step_rates(static_cast<double>(cfg->step), cfg->lr, cfg->weight_decay,
                               cfg->beta1, cfg->beta2);
    h.decay = r.decay;
    h.rate = r.rate;
    h.root = r.root;
  }
  h.wd = cfg->weight_decay;
  h.beta1 = cfg->beta1;
  h.beta2 = cfg->beta2;
  h.max_norm = cfg->max_norm;
  h.norm = norm;
  h.step_lr = step_lr;
  h.status = status;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (n <= kSmallBatch) return run_batches<kSmallBatch>(*cfg, n, l, h, s);
  if (n <= kMiddleBatch) return run_batches<kMiddleBatch>(*cfg, n, l, h, s);
  return run_batches<kLargeBatch>(*cfg, n, l, h, s);
}
