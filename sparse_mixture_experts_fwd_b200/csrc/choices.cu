// The row exchange around the experts for up to 16 choices a token, and its
// gradients (the one- and two-choice forward copies are in permute.cu):
//   dispatch            xe[e_j, s_j, :] = x[t, :]
//   dispatch, backward  dx[t, :] = sum over kept j of dxe[e_j, s_j, :]
//   combine             y[t, :] = sum over kept j of w_j ye[e_j, s_j, :]
//   combine, backward   dye[e_j, s_j, :] = w_j dy[t, :],  dw_j = <dy[t], ye[e_j, s_j]>
// A kept choice owns its expert row, so no two tokens touch the same one and
// nothing is added atomically.
#include <algorithm>
#include <type_traits>

#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

struct ChoiceParams {
  int64_t T;
  int k, E, C, row_vec;  // row_vec: 16-byte vectors per row
  int team;              // threads per token: 32, 64, 128 or 256
  const int32_t* expert_idx;
  const float* gate;     // null: 1
  const int32_t* slot;
  const uint8_t* kept;
  const uint4* tok_in;   // x or dy, [T, d]
  uint4* tok_out;        // dx or y
  const uint4* row_in;   // dxe or ye, [E, C, d]
  uint4* row_out;        // xe or dye
  float* dgate;          // [T, k]
  int32_t* status;
};

// Expert row (in vectors) of this lane's choice of token t; -1 if it was dropped.
// The slot and expert of a kept choice come from the assignment; a row outside
// the buffer is skipped in the bounds-checked build.
MOE_DEV int64_t choice_row(const ChoiceParams& p, int64_t t, int lane, bool* bad) {
  if (lane >= p.k || !__ldg(p.kept + t * p.k + lane)) return -1;
  const int e = __ldg(p.expert_idx + t * p.k + lane), s = __ldg(p.slot + t * p.k + lane);
#if MOE_CHECK_BOUNDS
  if (e < 0 || e >= p.E || s < 0 || s >= p.C) {
    *bad = true;
    return -1;
  }
#else
  (void)bad;
#endif
  return (static_cast<int64_t>(e) * p.C + s) * p.row_vec;
}

struct Bf16Vec {
  static constexpr int kN = 8;
  static MOE_DEV void unpack(const uint4& u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static MOE_DEV uint4 pack(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
struct F32Vec {
  static constexpr int kN = 4;
  static MOE_DEV void unpack(const uint4& u, float (&f)[4]) {
    f[0] = __uint_as_float(u.x);
    f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z);
    f[3] = __uint_as_float(u.w);
  }
  static MOE_DEV uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
};

MOE_DEV void report(const ChoiceParams& p, bool bad) {
  if (MOE_CHECK_BOUNDS && __any_sync(0xffffffffu, bad) && (threadIdx.x & 31) == 0 && p.status)
    atomicOr(p.status, MOE_STATUS_BAD_INDEX);
}

// K >= k: the choices a thread keeps in registers.
template <int K>
__global__ void __launch_bounds__(kThreads) scatter_kernel(const ChoiceParams p) {
  dev::pdl_trigger();
  dev::pdl_wait();
  const int lane = threadIdx.x & 31, member = threadIdx.x % p.team;
  const int per = kThreads / p.team;
  bool bad = false;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * per + threadIdx.x / p.team; t < p.T;
       t += static_cast<int64_t>(gridDim.x) * per) {
    const int64_t mine = choice_row(p, t, lane, &bad);
    int64_t row[K];
#pragma unroll
    for (int j = 0; j < K; ++j) row[j] = __shfl_sync(0xffffffffu, mine, j);
    const uint4* src = p.tok_in + t * p.row_vec;
#pragma unroll 4
    for (int v = member; v < p.row_vec; v += p.team) {
      const uint4 val = __ldg(src + v);
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (row[j] >= 0) p.row_out[row[j] + v] = val;
    }
  }
  report(p, bad);
}

// y or dx: the kept rows (times the gate), summed in choice order in fp32 and
// rounded once.
template <int K, class V>
__global__ void __launch_bounds__(kThreads) gather_kernel(const ChoiceParams p) {
  dev::pdl_trigger();
  dev::pdl_wait();
  constexpr int N = V::kN;
  const int lane = threadIdx.x & 31, member = threadIdx.x % p.team;
  const int per = kThreads / p.team;
  bool bad = false;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * per + threadIdx.x / p.team; t < p.T;
       t += static_cast<int64_t>(gridDim.x) * per) {
    const int64_t mine = choice_row(p, t, lane, &bad);
    const float gate = mine >= 0 && p.gate ? __ldg(p.gate + t * p.k + lane) : 1.0f;
    int64_t row[K];
    float g[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
      row[j] = __shfl_sync(0xffffffffu, mine, j);
      g[j] = __shfl_sync(0xffffffffu, gate, j);
    }
    uint4* dst = p.tok_out + t * p.row_vec;
    for (int v = member; v < p.row_vec; v += p.team) {
      uint4 r[K];
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (row[j] >= 0) r[j] = __ldg(p.row_in + row[j] + v);
      float acc[N];
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] = 0.f;
#pragma unroll
      for (int j = 0; j < K; ++j) {
        if (row[j] >= 0) {
          float f[N];
          V::unpack(r[j], f);
#pragma unroll
          for (int i = 0; i < N; ++i) acc[i] = fmaf(g[j], f[i], acc[i]);
        }
      }
      dst[v] = V::pack(acc);
    }
  }
  report(p, bad);
}

template <int K, class V>
__global__ void __launch_bounds__(kThreads) combine_backward_kernel(const ChoiceParams p) {
  __shared__ float s_part[kThreads / 32][K];
  dev::pdl_trigger();
  dev::pdl_wait();
  constexpr int N = V::kN;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, member = threadIdx.x % p.team;
  const int per = kThreads / p.team;
  bool bad = false;
  // every team of a block runs the same number of rounds (a block barrier is inside)
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * per; t0 < p.T;
       t0 += static_cast<int64_t>(gridDim.x) * per) {
    const int64_t t = t0 + threadIdx.x / p.team;
    const bool there = t < p.T;
    const int64_t mine = there ? choice_row(p, t, lane, &bad) : -1;
    const float gate = mine >= 0 ? __ldg(p.gate + t * p.k + lane) : 0.f;
    int64_t row[K];
    float g[K], dot[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
      row[j] = __shfl_sync(0xffffffffu, mine, j);
      g[j] = __shfl_sync(0xffffffffu, gate, j);
      dot[j] = 0.f;
    }
    if (there) {
      const uint4* src = p.tok_in + t * p.row_vec;
      for (int v = member; v < p.row_vec; v += p.team) {
        const uint4 dyv = __ldg(src + v);
        uint4 r[K];
#pragma unroll
        for (int j = 0; j < K; ++j)
          if (row[j] >= 0) r[j] = p.row_in[row[j] + v];  // dye may be ye
        float dy[N];
        V::unpack(dyv, dy);
#pragma unroll
        for (int j = 0; j < K; ++j) {
          if (row[j] >= 0) {
            float f[N];
            V::unpack(r[j], f);
#pragma unroll
            for (int i = 0; i < N; ++i) {
              dot[j] = fmaf(dy[i], f[i], dot[j]);
              f[i] = g[j] * dy[i];
            }
            p.row_out[row[j] + v] = V::pack(f);
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < K; ++j) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
      if (lane == 0) s_part[warp][j] = dot[j];
    }
    __syncthreads();
    if (there && member < p.k) {
      float sum = 0.f;
      const int w0 = warp;  // member < 16: this is the team's first warp
      for (int w = 0; w < p.team / 32; ++w) sum += s_part[w0 + w][member];
      p.dgate[t * p.k + member] = sum;
    }
    __syncthreads();
  }
  report(p, bad);
}

// Threads per token: a warp where there are tokens for every SM's warps, else
// more, so that a few tokens' rows are still spread over many lanes.
int team_size(int64_t T, int row_vec) {
  int team = 32;
  while (team < kThreads && T * team < static_cast<int64_t>(num_sms()) * 1024 && team < row_vec)
    team *= 2;
  return team;
}

unsigned grid_for(int64_t T, int team) {
  const int per = kThreads / team;
  return static_cast<unsigned>(
      std::max<int64_t>(1, std::min<int64_t>((T + per - 1) / per, int64_t(num_sms()) * 16)));
}

ChoiceParams base_params(const moe_config& c, const int32_t* expert_idx, const float* gate,
                         const int32_t* slot, const uint8_t* kept, int32_t* status) {
  ChoiceParams p{};
  p.T = c.T;
  p.k = c.k;
  p.E = c.E;
  p.C = c.capacity;
  p.row_vec = static_cast<int>(c.d_model * elem_size(c.dtype) / 16);
  p.team = team_size(c.T, p.row_vec);
  p.expert_idx = expert_idx;
  p.gate = gate;
  p.slot = slot;
  p.kept = kept;
  p.status = status;
  return p;
}

// calls f with the register width for k choices as a template argument
template <class F>
void with_width(int k, F&& f) {
  if (k <= 1) f(std::integral_constant<int, 1>{});
  else if (k <= 2) f(std::integral_constant<int, 2>{});
  else if (k <= 4) f(std::integral_constant<int, 4>{});
  else if (k <= 8) f(std::integral_constant<int, 8>{});
  else f(std::integral_constant<int, 16>{});
}

int32_t launch_gather(const moe_config& c, const ChoiceParams& p, cudaStream_t s) {
  const unsigned grid = grid_for(c.T, p.team);
  with_width(c.k, [&](auto w) {
    constexpr int K = decltype(w)::value;
    if (c.dtype == MOE_DTYPE_BF16)
      launch_pdl(gather_kernel<K, Bf16Vec>, dim3(grid), dim3(kThreads), 0, s, p);
    else
      launch_pdl(gather_kernel<K, F32Vec>, dim3(grid), dim3(kThreads), 0, s, p);
  });
  return check_launch("gather_kernel");
}

}  // namespace

int32_t launch_scatter_choices(const moe_config& c, const void* x, const int32_t* expert_idx,
                               const int32_t* slot, const uint8_t* kept, void* xe, int32_t* status,
                               cudaStream_t s) {
  ChoiceParams p = base_params(c, expert_idx, nullptr, slot, kept, status);
  p.tok_in = static_cast<const uint4*>(x);
  p.row_out = static_cast<uint4*>(xe);
  const dim3 grid(grid_for(c.T, p.team)), block(kThreads);
  if (c.k <= 4) launch_pdl(scatter_kernel<4>, grid, block, 0, s, p);
  else if (c.k <= 8) launch_pdl(scatter_kernel<8>, grid, block, 0, s, p);
  else launch_pdl(scatter_kernel<16>, grid, block, 0, s, p);
  return check_launch("scatter_kernel");
}

int32_t launch_gather_choices(const moe_config& c, const void* rows, const int32_t* expert_idx,
                              const float* gate, const int32_t* slot, const uint8_t* kept,
                              void* out, int32_t* status, cudaStream_t s) {
  ChoiceParams p = base_params(c, expert_idx, gate, slot, kept, status);
  p.row_in = static_cast<const uint4*>(rows);
  p.tok_out = static_cast<uint4*>(out);
  return launch_gather(c, p, s);
}

int32_t launch_combine_backward(const moe_config& c, const void* dy, const void* ye,
                                const int32_t* expert_idx, const float* gate, const int32_t* slot,
                                const uint8_t* kept, void* dye, float* dgate, int32_t* status,
                                cudaStream_t s) {
  ChoiceParams p = base_params(c, expert_idx, gate, slot, kept, status);
  p.tok_in = static_cast<const uint4*>(dy);
  p.row_in = static_cast<const uint4*>(ye);
  p.row_out = static_cast<uint4*>(dye);
  p.dgate = dgate;
  const unsigned grid = grid_for(c.T, p.team);
  with_width(c.k, [&](auto w) {
    constexpr int K = decltype(w)::value;
    if (c.dtype == MOE_DTYPE_BF16)
      launch_pdl(combine_backward_kernel<K, Bf16Vec>, dim3(grid), dim3(kThreads), 0, s, p);
    else
      launch_pdl(combine_backward_kernel<K, F32Vec>, dim3(grid), dim3(kThreads), 0, s, p);
  });
  return check_launch("combine_backward_kernel");
}

}  // namespace moe
