// The row exchange around the experts for up to 16 choices a token, and its
// gradients (the one- and two-choice forward copies are in permute.cu):
//   dispatch            xe[e_j, s_j, :] = x[t, :]
//   dispatch, backward  dx[t, :] = sum over kept j of dxe[e_j, s_j, :]
//   combine             y[t, :] = sum over kept j of w_j ye[e_j, s_j, :]
//   combine, backward   dye[e_j, s_j, :] = w_j dy[t, :],  dw_j = <dy[t], ye[e_j, s_j]>
// A kept choice owns its expert row, so no two tokens touch the same one and
// nothing is added atomically.  All of them are copies of rows by 16-byte vectors,
// bound by HBM and the bytes in flight.  16384 tokens, 8 kept choices, rows of
// 2 KB, 302 MB one way (46 us at the copy rate): dispatch 54 us, combine 49,
// dispatch's gradient 49, combine's (570 MB, 87 us) 98.  5 tokens: 3.6 us.
#include <algorithm>
#include <type_traits>

#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

struct ChoiceParams {
  int64_t T;
  int k, E, C, row_vec;  // row_vec: 16-byte vectors per row
  int team;              // threads per token: 16, 32, 64, 128 or 256
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

// Expert row (in vectors) and gate of choice j of token t; -1 if it was dropped.
// The slot and expert of a kept choice come from the assignment; a row outside
// the buffer is skipped in the bounds-checked build.
struct Choice {
  int64_t row;
  float gate;
};
MOE_DEV Choice choice_of(const ChoiceParams& p, int64_t t, int j, bool* bad) {
  Choice c{-1, 0.f};
  if (t >= p.T || j >= p.k) return c;
  const int64_t a = t * p.k + j;
  const bool kept = __ldg(p.kept + a) != 0;
  const int e = __ldg(p.expert_idx + a), s = __ldg(p.slot + a);
  const float g = p.gate ? __ldg(p.gate + a) : 1.0f;
  if (!kept) return c;
#if MOE_CHECK_BOUNDS
  if (e < 0 || e >= p.E || s < 0 || s >= p.C) {
    *bad = true;
    return c;
  }
#else
  (void)bad;
#endif
  c.row = (static_cast<int64_t>(e) * p.C + s) * p.row_vec;
  c.gate = g;
  return c;
}

// A team's place in the grid.  Teams of one warp or less hold a choice per
// lane; wider ones hold the same choices in each of their warps.  The sums load
// the next token's choices while the rows of one are on their way: they are a
// chain of their own in front of the rows' addresses.
template <int LANES>
struct Walk {
  int64_t t, step;
  int member, team, first;  // place in the team, its size, its first lane
  MOE_DEV explicit Walk(const ChoiceParams& p) {
    team = LANES < 32 ? LANES : p.team;
    const int per = kThreads / team;
    t = static_cast<int64_t>(blockIdx.x) * per + threadIdx.x / team;
    step = static_cast<int64_t>(gridDim.x) * per;
    member = threadIdx.x % team;
    first = (threadIdx.x & 31) & ~(LANES - 1);
  }
};

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

// Warps whose lanes work for different tokens walk together: a round is done while
// any of them has a token.
template <int LANES>
MOE_DEV bool any_left(const Walk<LANES>& w, const ChoiceParams& p) {
  if (LANES == 32) return w.t < p.T;
  return __any_sync(0xffffffffu, w.t < p.T);
}

// K >= k: the choices a thread keeps in registers.
template <int K, int LANES>
__global__ void __launch_bounds__(kThreads) scatter_kernel(const ChoiceParams p) {
  dev::pdl_trigger();
  dev::pdl_wait();
  Walk<LANES> w(p);
  const int j0 = (threadIdx.x & 31) - w.first;
  bool bad = false;
  for (; any_left(w, p); w.t += w.step) {
    const Choice mine = choice_of(p, w.t, j0, &bad);
    int64_t row[K];
#pragma unroll
    for (int j = 0; j < K; ++j) row[j] = __shfl_sync(0xffffffffu, mine.row, w.first + j);
    if (w.t < p.T) {
      const uint4* src = p.tok_in + w.t * p.row_vec;
#pragma unroll(LANES == 32 ? 4 : 1)
      for (int v = w.member; v < p.row_vec; v += w.team) {
        const uint4 val = __ldg(src + v);
#pragma unroll
        for (int j = 0; j < K; ++j)
          if (row[j] >= 0) p.row_out[row[j] + v] = val;
      }
    }
  }
  report(p, bad);
}

// y or dx: the kept rows (times the gate), summed in choice order in fp32 and
// rounded once.  Up to 8 rows are in flight: 16 would leave room for one block
// an SM (65536 tokens x 16 rows of 256 bytes: 175 us then, 0.25 of the copy rate).
// Bound by the bytes in flight, so for 8 rows 64 registers and four blocks an SM
// (8191 tokens, rows of 5 KB: 59.2 us, 64.6 with the compiler's 70 registers and
// three blocks) and for fewer rows 48 and five (16384 tokens, 4 rows of 2 KB: 30.9 us,
// 42.1 with as many registers as the unrolled loads would take).
template <int K, class V, int LANES>
__global__ void __launch_bounds__(kThreads, K == 16 ? 3 : K == 8 ? 4 : 5) gather_kernel(const ChoiceParams p) {
  dev::pdl_trigger();
  dev::pdl_wait();
  constexpr int N = V::kN;
  constexpr int B = K < 8 ? K : 8;
  Walk<LANES> w(p);
  const int j0 = (threadIdx.x & 31) - w.first;
  bool bad = false;
  Choice next = choice_of(p, w.t, j0, &bad);
  for (; any_left(w, p); w.t += w.step) {
    const Choice mine = next;
    next = choice_of(p, w.t + w.step, j0, &bad);
    uint4* dst = p.tok_out + w.t * p.row_vec;
    float acc[N];
    // choices b .. b + B - 1: their rows' vector v, then its part of the sum
    auto fetch = [&](const int64_t* row, uint4 (&r)[B], int v) {
#pragma unroll
      for (int j = 0; j < B; ++j)
        if (row[j] >= 0) r[j] = __ldg(p.row_in + row[j] + v);
    };
    auto add = [&](const int64_t* row, const float* g, const uint4 (&r)[B]) {
#pragma unroll
      for (int j = 0; j < B; ++j) {
        if (row[j] >= 0) {
          float f[N];
          V::unpack(r[j], f);
#pragma unroll
          for (int i = 0; i < N; ++i) acc[i] = fmaf(g[j], f[i], acc[i]);
        }
      }
    };
    if constexpr (LANES == 32) {  // the choices are the same for the whole warp
      int64_t row[K];
      float g[K];
#pragma unroll
      for (int j = 0; j < K; ++j) {
        row[j] = __shfl_sync(0xffffffffu, mine.row, j);
        g[j] = __shfl_sync(0xffffffffu, mine.gate, j);
      }
      constexpr int U = K >= 8 ? 1 : K >= 4 ? 2 : 4;  // up to 8 vectors ahead of the sums
      for (int v0 = w.member; v0 < p.row_vec; v0 += U * w.team) {
        uint4 r[U][B];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (v0 + u * w.team < p.row_vec) fetch(row, r[u], v0 + u * w.team);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int v = v0 + u * w.team;
          if (v < p.row_vec) {
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] = 0.f;
            add(row, g, r[u]);
#pragma unroll
            for (int b = B; b < K; b += B) {  // (K = 16: U is 1)
              fetch(row + b, r[u], v);
              add(row + b, g + b, r[u]);
            }
            dst[v] = V::pack(acc);
          }
        }
      }
    } else {  // rows of at most LANES vectors: one each
      const bool on = w.t < p.T && w.member < p.row_vec;
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] = 0.f;
#pragma unroll
      for (int b = 0; b < K; b += B) {
        int64_t row[B];
        float g[B];
#pragma unroll
        for (int j = 0; j < B; ++j) {
          row[j] = __shfl_sync(0xffffffffu, mine.row, w.first + b + j);
          g[j] = __shfl_sync(0xffffffffu, mine.gate, w.first + b + j);
        }
        if (on) {
          uint4 r[B];
          fetch(row, r, w.member);
          add(row, g, r);
        }
      }
      if (on) dst[w.member] = V::pack(acc);
    }
  }
  report(p, bad);
}

// K sums over LANES lanes at once, by halves: in each step a lane gives away the
// half of its values that its partner keeps, so K = 8 takes 9 shuffles and not
// 40.  Afterwards lane l holds sum (l / spread) % K, spread = LANES / K (K <= LANES).
template <int K, int LANES>
MOE_DEV float reduce_many(float (&v)[K]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = LANES / 2, n = K; o > 0; o >>= 1) {
    if (n > 1) {
      n >>= 1;
      const bool upper = (lane & o) != 0;
#pragma unroll
      for (int i = 0; i < K / 2; ++i) {
        if (i < n) {
          const float give = upper ? v[i] : v[i + n], keep = upper ? v[i + n] : v[i];
          v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
      }
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
    }
  }
  return v[0];
}

template <int K, class V, int LANES>
__global__ void __launch_bounds__(kThreads) combine_backward_kernel(const ChoiceParams p) {
  __shared__ float s_part[kThreads / 32][K];
  dev::pdl_trigger();
  dev::pdl_wait();
  constexpr int N = V::kN;
  constexpr int B = K < 8 ? K : 8;
  constexpr int kSpread = LANES / K;
  Walk<LANES> w(p);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int j0 = lane - w.first;
  bool bad = false;
  Choice next = choice_of(p, w.t, j0, &bad);
  // a team of several warps meets at a block barrier, so then every team of the
  // block runs the same number of rounds
  const int64_t first_t = static_cast<int64_t>(blockIdx.x) * (kThreads / w.team);
  for (int64_t t0 = first_t; w.team > 32 ? t0 < p.T : any_left(w, p); t0 += w.step, w.t += w.step) {
    const Choice mine = next;
    next = choice_of(p, w.t + w.step, j0, &bad);
    float dot[K];
#pragma unroll
    for (int j = 0; j < K; ++j) dot[j] = 0.f;
    const bool there = w.t < p.T;
    const uint4* src = p.tok_in + w.t * p.row_vec;
    // choices b .. b + B - 1: their rows' vector v, then what becomes of it
    auto fetch = [&](const int64_t* row, uint4 (&r)[B], int v) {
#pragma unroll
      for (int j = 0; j < B; ++j)
        if (row[j] >= 0) r[j] = p.row_in[row[j] + v];  // dye may be ye
    };
    auto work = [&](const int64_t* row, const float* g, float* sums, const uint4 (&r)[B],
                    const float (&dy)[N], int v) {
#pragma unroll
      for (int j = 0; j < B; ++j) {
        if (row[j] >= 0) {
          float f[N];
          V::unpack(r[j], f);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            sums[j] = fmaf(dy[i], f[i], sums[j]);
            f[i] = g[j] * dy[i];
          }
          p.row_out[row[j] + v] = V::pack(f);
        }
      }
    };
    if constexpr (LANES == 32) {  // the choices are the same for the whole warp
      int64_t row[K];
      float g[K];
#pragma unroll
      for (int j = 0; j < K; ++j) {
        row[j] = __shfl_sync(0xffffffffu, mine.row, j);
        g[j] = __shfl_sync(0xffffffffu, mine.gate, j);
      }
      if (there) {
        // up to 8 rows' vectors are loaded before any is stored: the compiler may not
        // move loads over the stores by itself
        constexpr int U = K >= 8 ? 1 : K >= 4 ? 2 : 4;
        for (int v0 = w.member; v0 < p.row_vec; v0 += U * w.team) {
          uint4 dv[U], r[U][B];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int v = v0 + u * w.team;
            if (v < p.row_vec) {
              dv[u] = __ldg(src + v);
              fetch(row, r[u], v);
            }
          }
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int v = v0 + u * w.team;
            if (v < p.row_vec) {
              float dy[N];
              V::unpack(dv[u], dy);
              work(row, g, dot, r[u], dy, v);
#pragma unroll
              for (int b = B; b < K; b += B) {  // (K = 16: U is 1)
                fetch(row + b, r[u], v);
                work(row + b, g + b, dot + b, r[u], dy, v);
              }
            }
          }
        }
      }
    } else {  // rows of at most LANES vectors: one each
      const bool on = there && w.member < p.row_vec;
      float dy[N];
      if (on) V::unpack(__ldg(src + w.member), dy);
#pragma unroll
      for (int b = 0; b < K; b += B) {
        int64_t row[B];
        float g[B];
#pragma unroll
        for (int j = 0; j < B; ++j) {
          row[j] = __shfl_sync(0xffffffffu, mine.row, w.first + b + j);
          g[j] = __shfl_sync(0xffffffffu, mine.gate, w.first + b + j);
        }
        if (on) {
          uint4 r[B];
          fetch(row, r, w.member);
          work(row, g, dot + b, r, dy, w.member);
        }
      }
    }
    const float sum = reduce_many<K, LANES>(dot);
    const int j = (j0 / kSpread) % K;
    const bool writes = j0 % kSpread == 0;
    if (w.team <= 32) {
      if (there && writes && j < p.k) p.dgate[w.t * p.k + j] = sum;
    } else {
      if (writes) s_part[warp][j] = sum;
      __syncthreads();
      if (there && w.member < p.k) {
        float all = 0.f;  // member < 16: `warp` is the team's first
        for (int q = 0; q < w.team / 32; ++q) all += s_part[warp + q][w.member];
        p.dgate[w.t * p.k + w.member] = all;
      }
      __syncthreads();
    }
  }
  report(p, bad);
}

// Threads per token: half a warp for rows of at most 16 vectors (a whole one would
// idle by half), a warp where there are tokens for every SM's warps, else more, so
// that a few tokens' rows are still spread over many lanes.
int team_size(int64_t T, int row_vec) {
  if (row_vec <= 16) return 16;
  int team = 32;
  while (team < kThreads && T * team < static_cast<int64_t>(num_sms()) * 1024 && team < row_vec)
    team *= 2;
  return team;
}

unsigned grid_for(int64_t T, int team, int blocks_per_sm) {
  const int per = kThreads / team;
  return static_cast<unsigned>(std::max<int64_t>(
      1, std::min<int64_t>((T + per - 1) / per, int64_t(num_sms()) * blocks_per_sm)));
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

// calls f with the register width for k choices and the lanes of a team in a warp as
// template arguments
template <int LANES, class F>
void with_width(int k, F&& f) {
  using std::integral_constant;
  integral_constant<int, LANES> lanes;
  if (k <= 1) f(integral_constant<int, 1>{}, lanes);
  else if (k <= 2) f(integral_constant<int, 2>{}, lanes);
  else if (k <= 4) f(integral_constant<int, 4>{}, lanes);
  else if (k <= 8) f(integral_constant<int, 8>{}, lanes);
  else f(integral_constant<int, 16>{}, lanes);
}
template <class F>
void with_shape(const ChoiceParams& p, F&& f) {
  if (p.team == 16) with_width<16>(p.k, f);
  else with_width<32>(p.k, f);
}

}  // namespace

int32_t launch_scatter_choices(const moe_config& c, const void* x, const int32_t* expert_idx,
                               const int32_t* slot, const uint8_t* kept, void* xe, int32_t* status,
                               cudaStream_t s) {
  ChoiceParams p = base_params(c, expert_idx, nullptr, slot, kept, status);
  p.tok_in = static_cast<const uint4*>(x);
  p.row_out = static_cast<uint4*>(xe);
  const dim3 grid(grid_for(c.T, p.team, 16)), block(kThreads);
  with_shape(p, [&](auto w, auto lanes) {
    constexpr int K = decltype(w)::value < 4 ? 4 : decltype(w)::value;  // called for k > 2
    launch_pdl(scatter_kernel<K, decltype(lanes)::value>, grid, block, 0, s, p);
  });
  return check_launch("scatter_kernel");
}

int32_t launch_gather_choices(const moe_config& c, const void* rows, const int32_t* expert_idx,
                              const float* gate, const int32_t* slot, const uint8_t* kept,
                              void* out, int32_t* status, cudaStream_t s) {
  ChoiceParams p = base_params(c, expert_idx, gate, slot, kept, status);
  p.row_in = static_cast<const uint4*>(rows);
  p.tok_out = static_cast<uint4*>(out);
  const dim3 grid(grid_for(c.T, p.team, 16)), block(kThreads);
  with_shape(p, [&](auto w, auto lanes) {
    constexpr int K = decltype(w)::value, kLanes = decltype(lanes)::value;
    if (c.dtype == MOE_DTYPE_BF16) launch_pdl(gather_kernel<K, Bf16Vec, kLanes>, grid, block, 0, s, p);
    else launch_pdl(gather_kernel<K, F32Vec, kLanes>, grid, block, 0, s, p);
  });
  return check_launch("gather_kernel");
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
  // its 100 to 150 registers leave two blocks an SM: a longer grid is a ragged tail
  // (65536 tokens, 8 rows of 512 bytes: 109 us with 16, 102 with 4)
  const dim3 grid(grid_for(c.T, p.team, 4)), block(kThreads);
  with_shape(p, [&](auto w, auto lanes) {
    constexpr int K = decltype(w)::value, kLanes = decltype(lanes)::value;
    if (c.dtype == MOE_DTYPE_BF16)
      launch_pdl(combine_backward_kernel<K, Bf16Vec, kLanes>, grid, block, 0, s, p);
    else
      launch_pdl(combine_backward_kernel<K, F32Vec, kLanes>, grid, block, 0, s, p);
  });
  return check_launch("combine_backward_kernel");
}

}  // namespace moe
