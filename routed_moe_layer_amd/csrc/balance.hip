// The router's balance: how evenly a batch loads the experts, as a loss on the gate's
// probabilities, and its gradient.
//   p[t] = softmax(logits[t]),  c_e = unmasked routed rows of expert e,  S_e = sum_t p[t, e],
//   N = unmasked tokens,  loss = coef * E * sum_e (c_e / sum c) * (S_e / N);
//   d loss / d logits[t, e] = coef * E / (N sum c) * p[t, e] * (c_e - sum_i p[t, i] c_i)
// with the counts taken as constants.  The gradient uses c_e - mean(c), which changes nothing as
// the probabilities sum to one: nearly equal counts keep their differences, equal ones give 0.
//
// A row is held in registers by LPR lanes (4, 16 or 64 by the number of experts), V values each,
// so it is read once; the next row's loads are under way meanwhile, and the mask of the one behind
// it.  The sums over tokens stay in the same lanes, then go over the workgroup's wavefronts in LDS
// and over the workgroups in a second launch, each in a fixed order, so a call's result never
// depends on timing.
#include "common.h"
#include "kernels.h"

namespace rmoe {

// Wavefronts of a workgroup, and rows of sums that they share in LDS: with more than 1024 experts a
// row's registers leave room for half as many wavefronts, and LDS for fewer rows.
constexpr int balance_waves(int V) { return V <= 16 ? 16 : 8; }
constexpr int balance_slots(int V) { return V <= 16 ? 8 : 2; }

template <int CTRL, int ROW_MASK>
__device__ __forceinline__ float dppf(float old, float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(old), __float_as_int(x), CTRL,
                                                    ROW_MASK, 0xF, false));
}
__device__ __forceinline__ float read_last(float x) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 63));
}
// Maximum and sum over the LPR lanes of a row, returned to all of them.
template <int LPR>
__device__ __forceinline__ float row_max(float x) {
  x = fmaxf(x, dppf<0xB1, 0xF>(x, x));                 // quad_perm [1,0,3,2]
  x = fmaxf(x, dppf<0x4E, 0xF>(x, x));                 // quad_perm [2,3,0,1]
  if constexpr (LPR >= 16) {
    x = fmaxf(x, dppf<0x141, 0xF>(x, x));              // row_half_mirror
    x = fmaxf(x, dppf<0x140, 0xF>(x, x));              // row_mirror
  }
  if constexpr (LPR == 64) {
    x = fmaxf(x, dppf<0x142, 0xA>(x, x));              // row_bcast:15 into rows 1, 3
    x = fmaxf(x, dppf<0x143, 0xC>(x, x));              // row_bcast:31 into rows 2, 3
    x = read_last(x);
  }
  return x;
}
template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
  x += dppf<0xB1, 0xF>(0.0f, x);
  x += dppf<0x4E, 0xF>(0.0f, x);
  if constexpr (LPR >= 16) {
    x += dppf<0x141, 0xF>(0.0f, x);
    x += dppf<0x140, 0xF>(0.0f, x);
  }
  if constexpr (LPR == 64) {
    x += dppf<0x142, 0xA>(0.0f, x);
    x += dppf<0x143, 0xC>(0.0f, x);
    x = read_last(x);
  }
  return x;
}

// Expert of a lane's value v.  VEC: groups of four consecutive experts.
template <int LPR, bool VEC>
__device__ __forceinline__ int expert_of(int sub, int v) {
  return VEC ? 4 * (sub + LPR * (v >> 2)) + (v & 3) : sub + LPR * v;
}

// A lane's V values of a row, `pad` past the last expert.  VEC needs E a multiple of 4 and rows
// aligned to four values.
// NT: past the caches.
template <bool BF16, int LPR, int V, bool VEC, bool NT>
__device__ __forceinline__ void load_row(const void* base, int64_t row, int E, int sub, float pad,
                                         float (&z)[V]) {
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      const int e = 4 * (sub + LPR * i);
      if (e < E) {
        if constexpr (BF16) {
          const u32x2* p = reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(base) + row * E + e);
          const u32x2 w = NT ? __builtin_nontemporal_load(p) : *p;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            z[4 * i + 2 * j] = __uint_as_float(w[j] << 16);
            z[4 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
          }
        } else {
          const f32x4* p = reinterpret_cast<const f32x4*>(static_cast<const float*>(base) + row * E + e);
          const f32x4 w = NT ? __builtin_nontemporal_load(p) : *p;
#pragma unroll
          for (int j = 0; j < 4; ++j) z[4 * i + j] = w[j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) z[4 * i + j] = pad;
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = sub + LPR * v;
      z[v] = pad;
      if (e < E) {
        if constexpr (BF16) z[v] = bf16_to_f32(static_cast<const uint16_t*>(base)[row * E + e]);
        else z[v] = static_cast<const float*>(base)[row * E + e];
      }
    }
  }
}

// exp(x), x <= 0, to a step and a half.  The exponential of 2 takes y = x / ln 2 rounded, which alone
// would be off by up to |x| half steps of the result; x - y ln 2, ln 2 in two parts, is what that
// rounding left, and is multiplied in.  The factor is 1 / ln 2 rounded up: y is never above
// x / ln 2, so the rest lies in [0, 1], and the bounds (a modifier of the instruction) only
// make 0 of the NaN or infinity that an infinite or very large -x leaves.  Three more instructions a
// value than the bare exponential: one workgroup's 64 x 896 logits 11.2 -> 12.3 us, 16384 x 896 19.5
// -> 20.2, their gradient as before.
__device__ __forceinline__ float exp_nonpositive(float x) {
  const float y = x * 1.442695140838623046875f, e = __builtin_amdgcn_exp2f(y);
  const float rest = __builtin_fmaf(y, 1.9046542999577674e-9f,
                                    __builtin_fmaf(y, -0.693147182464599609375f, x));
  return __builtin_fmaf(e, __builtin_amdgcn_fmed3f(rest, 0.0f, 1.0f), e);
}

// exp(z - max) in place; returns 1 / their sum.  A row of -inf has probabilities 0 (factor 0); a
// NaN or +inf makes the factor NaN.
template <int LPR, int V>
__device__ __forceinline__ float softmax_parts(float (&z)[V]) {
  float m = z[0];
#pragma unroll
  for (int v = 1; v < V; ++v) m = fmaxf(m, z[v]);
  m = row_max<LPR>(m);
  if (m == -__builtin_inff()) m = 0.0f;
  float s = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    z[v] = exp_nonpositive(z[v] - m);
    s += z[v];
  }
  s = row_sum<LPR>(s);
  return s == 0.0f ? 0.0f : 1.0f / s;
}

template <bool BF16, int LPR, int V, bool VEC>
__global__ __launch_bounds__(balance_waves(V) * 64) void balance_stats_kernel(BalanceArgs a) {
  constexpr int kRows = 64 / LPR, kWaves = balance_waves(V), kSlots = balance_slots(V);
  constexpr int kThreads = kWaves * 64;
  extern __shared__ char s_raw[];
  float* s_sum = reinterpret_cast<float*>(s_raw);      // [kSlots][E]
  int32_t* s_count = reinterpret_cast<int32_t*>(s_raw) + kSlots * a.E;
  __shared__ int32_t s_tokens, s_routed;
  __shared__ double s_dot[kWaves];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, sub = lane % LPR;
  const int step = static_cast<int>(gridDim.x) * kWaves * kRows;
  int t = (static_cast<int>(blockIdx.x) * kWaves + wave) * kRows + lane / LPR;
  float z[V], acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.0f;
  auto counted = [&](int row) { return row < a.T && (!a.mask || a.mask[row]); };
  // rows that do not count are never read
  auto fetch = [&](int row, bool live, float (&to)[V]) {
    // (one row a wavefront: the same for its lanes, and no lane fills what it then loads)
    if (LPR == 64 ? __builtin_amdgcn_readfirstlane(live) != 0 : live) {
      load_row<BF16, LPR, V, VEC, false>(a.logits, row, a.E, sub, -__builtin_inff(), to);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) to[v] = -__builtin_inff();
    }
  };
  bool live = counted(t + step);                       // of the row behind the one under way
  fetch(t, counted(t), z);
  for (int e = tid; e < a.E; e += kThreads) s_count[e] = 0;
  if (tid == 0) s_tokens = s_routed = 0;
  __syncthreads();
  // the experts' counts, while the first rows are on their way
  int tokens = 0;
  const int ids = a.T * a.k;
  for (int f = static_cast<int>(blockIdx.x) * kThreads + tid; f < ids; f += static_cast<int>(gridDim.x) * kThreads) {
    const int row = f / a.k, e = a.ids[f];
    if (!counted(row)) continue;
    if (f == row * a.k) ++tokens;
    if (e >= 0 && e < a.E) atomicAdd(&s_count[e], 1);
  }
  if (tokens) atomicAdd(&s_tokens, tokens);
  // a row under way in z and the one behind it in next, which then change places
  auto add_row = [&](float (&row)[V]) {
    const float inv = softmax_parts<LPR, V>(row);
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = __builtin_fmaf(row[v], inv, acc[v]);
  };
  auto fetch_next = [&](float (&to)[V]) {
    t += step;
    fetch(t, live, to);
    live = counted(t + step);
  };
  float next[V];
  for (int base = t - lane / LPR; base < a.T; base += step) {              // whole wavefronts
    fetch_next(next);
    add_row(z);
    base += step;
    if (base >= a.T) break;
    fetch_next(z);
    add_row(next);
  }
  if constexpr (LPR < 64) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int off = LPR; off < 64; off <<= 1) acc[v] += __shfl_xor(acc[v], off);
    }
  }
#pragma unroll
  for (int w = 0; w < kWaves; w += kSlots) {
    if (wave / kSlots == w / kSlots && lane < LPR) {
      float* to = s_sum + (wave % kSlots) * a.E;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = expert_of<LPR, VEC>(sub, v);
        if (e < a.E) to[e] = w == 0 ? acc[v] : to[e] + acc[v];
      }
    }
    __syncthreads();
  }
  for (int e = tid; e < a.E; e += kThreads) {          // (each thread the experts it goes on with)
    float sum = s_sum[e];
#pragma unroll
    for (int i = 1; i < kSlots; ++i) sum += s_sum[i * a.E + e];
    s_sum[e] = sum;
  }

  if (gridDim.x > 1) {
    float* sums = a.part_sums + static_cast<int64_t>(blockIdx.x) * a.E;
    int32_t* counts = a.part_counts + static_cast<int64_t>(blockIdx.x) * a.E;
    for (int e = tid; e < a.E; e += kThreads) {
      sums[e] = s_sum[e];
      counts[e] = s_count[e];
    }
    if (tid == 0) {
      a.part_tokens[blockIdx.x] = s_tokens;
      if (blockIdx.x == 0) *a.ticket = 0u;
    }
    return;
  }
  // one workgroup: it has everything
  double dot = 0.0;
  int routed = 0;
  for (int e = tid; e < a.E; e += kThreads) {
    const float s = s_sum[e];
    const int c = s_count[e];
    a.sums[e] = s;
    a.counts[e] = c;
    dot += static_cast<double>(c) * s;
    routed += c;
  }
  if (routed) atomicAdd(&s_routed, routed);
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) dot += __shfl_xor(dot, off);
  if (lane == 0) s_dot[wave] = dot;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kWaves; ++w) dot += s_dot[w];
    const int n = s_tokens;
    a.tokens[0] = n;
    a.loss[0] = n > 0 && s_routed > 0
                    ? static_cast<float>(static_cast<double>(a.coef) * a.E * dot /
                                         (static_cast<double>(n) * s_routed))
                    : 0.0f;
  }
}

// The workgroups' sums and counts into the call's: sixteen experts per workgroup, its 64 groups of
// sixteen lanes over the G parts.  The workgroup that comes last adds up the loss.
constexpr int kJoinGroups = 64, kJoinExperts = kBalanceJoinExperts;
__global__ __launch_bounds__(kJoinGroups * kJoinExperts) void balance_join_kernel(BalanceArgs a, int G) {
  __shared__ double s_sum[kJoinGroups][kJoinExperts];
  __shared__ int32_t s_count[kJoinGroups][kJoinExperts];
  __shared__ int32_t s_tokens[16];
  const int tid = threadIdx.x, group = tid / kJoinExperts, col = tid % kJoinExperts;
  const int e = static_cast<int>(blockIdx.x) * kJoinExperts + col;
  double sum = 0.0;
  int32_t count = 0;
  if (e < a.E) {
#pragma unroll 4
    for (int g = group; g < G; g += kJoinGroups) {
      sum += a.part_sums[static_cast<int64_t>(g) * a.E + e];
      count += a.part_counts[static_cast<int64_t>(g) * a.E + e];
    }
  }
  s_sum[group][col] = sum;
  s_count[group][col] = count;
  if (blockIdx.x == 0) {
    int32_t tokens = 0;
    for (int g = tid; g < G; g += kJoinGroups * kJoinExperts) tokens += a.part_tokens[g];
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) tokens += __shfl_xor(tokens, off);
    if ((tid & 63) == 0) s_tokens[tid >> 6] = tokens;
  }
  __syncthreads();
  if (tid >= 64) return;
  // four quarters of the groups, then those
#pragma unroll
  for (int i = 4; i < kJoinGroups; i += 4) {
    sum += s_sum[group + i][col];
    count += s_count[group + i][col];
  }
#pragma unroll
  for (int off = kJoinExperts; off < 64; off <<= 1) {
    sum += __shfl_xor(sum, off);
    count += __shfl_xor(count, off);
  }
  const float s = static_cast<float>(sum);
  if (group == 0 && e < a.E) {
    a.sums[e] = s;
    a.counts[e] = count;
  }
  double dot = static_cast<double>(count) * s;
  int64_t routed = count;
#pragma unroll
  for (int off = kJoinExperts / 2; off > 0; off >>= 1) {
    dot += __shfl_xor(dot, off);
    routed += __shfl_xor(routed, off);
  }
  bool last = false;
  if (tid == 0) {
    a.part_dot[blockIdx.x] = dot;
    a.part_routed[blockIdx.x] = routed;
    if (blockIdx.x == 0) {
      int32_t n = 0;
      for (int w = 0; w < 16; ++w) n += s_tokens[w];
      a.tokens[0] = n;
    }
    __threadfence();
    last = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
    __threadfence();
  }
  if (!__shfl(static_cast<int>(last), 0)) return;
  dot = 0.0;
  routed = 0;
  for (unsigned b = tid; b < gridDim.x; b += 64) {
    dot += __hip_atomic_load(a.part_dot + b, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    routed += __hip_atomic_load(a.part_routed + b, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    dot += __shfl_xor(dot, off);
    routed += __shfl_xor(routed, off);
  }
  if (tid == 0) {
    const int32_t n = __hip_atomic_load(a.tokens, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    a.loss[0] = n > 0 && routed > 0
                    ? static_cast<float>(static_cast<double>(a.coef) * a.E * dot /
                                         (static_cast<double>(n) * static_cast<double>(routed)))
                    : 0.0f;
  }
}

template <bool BF16, int LPR, int V, bool VEC>
__global__ __launch_bounds__(256) void balance_grad_kernel(BalanceGradArgs a) {
  constexpr int kRows = 64 / LPR;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, sub = lane % LPR;
  const int step = static_cast<int>(gridDim.x) * 4 * kRows;
  int t = (static_cast<int>(blockIdx.x) * 4 + wave) * kRows + lane / LPR;
  auto counted = [&](int row) { return row < a.T && (!a.mask || a.mask[row]); };
  auto fetch = [&](int row, bool live, float (&to)[V]) {
    if (live) {
      load_row<BF16, LPR, V, VEC, true>(a.logits, row, a.E, sub, -__builtin_inff(), to);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) to[v] = -__builtin_inff();
    }
  };
  float z[V], d[V];
  bool live = counted(t), live_next = counted(t + step);
  fetch(t, live, z);
  // centred counts
  double all = 0.0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = expert_of<LPR, VEC>(sub, v);
    if (e < a.E) all += a.counts[e];
  }
#pragma unroll
  for (int off = 1; off < LPR; off <<= 1) all += __shfl_xor(all, off);
  const double mean = all / a.E;
  const double n = a.tokens[0];
  const bool some = n > 0.0 && all > 0.0;              // without, NaN rows have no gradient either
  // The scale may lie far outside fp32's range where the gradient does not: half of its power of two
  // goes to the counts (at most 2^80, so that sums over 4096 of 31 bits stay below 2^127), and what
  // then is still above 2^80 to the result.  (Below 2^-190 nothing is left of any gradient.)
  const double whole = some ? static_cast<double>(a.coef) * a.E / (n * all) *
                                  (a.grad_loss ? a.grad_loss[0] : 1.0f)
                            : 0.0;
  const int power = __builtin_amdgcn_frexp_exp(whole), half = min(max(power / 2, -80), 80);
  const int above = __builtin_amdgcn_readfirstlane(max(power - 160, 0));
  const float scale = static_cast<float>(ldexp(whole, -half - above));
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = expert_of<LPR, VEC>(sub, v);
    d[v] = e < a.E ? ldexpf(static_cast<float>(a.counts[e] - mean), half) : 0.0f;
  }
  for (int base = t - lane / LPR; base < a.T; base += step, t += step) {   // whole wavefronts
    float next[V], more[V];
    if (a.add && t < a.T) {
      load_row<BF16, LPR, V, VEC, true>(a.add, t, a.E, sub, 0.0f, more);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) more[v] = 0.0f;
    }
    fetch(t + step, live_next, next);
    const bool live_then = counted(t + 2 * step);
    const float inv = softmax_parts<LPR, V>(z);
    float dot = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) dot = __builtin_fmaf(z[v], d[v], dot);
    dot = row_sum<LPR>(dot) * inv;
    if (t < a.T) {
      const float f = scale * inv;
      float o[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float p = f * z[v], c = d[v] - dot;
        const float sum = above == 0 ? __builtin_fmaf(p, c, more[v]) : ldexpf(p * c, above) + more[v];
        o[v] = live && some ? sum : more[v];
      }
      const int64_t at = static_cast<int64_t>(t) * a.E;
      if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
          const int e = 4 * (sub + LPR * i);
          if (e >= a.E) continue;
          if constexpr (BF16)
            __builtin_nontemporal_store(
                u32x2{pack_bf16x2(o[4 * i], o[4 * i + 1]), pack_bf16x2(o[4 * i + 2], o[4 * i + 3])},
                reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.grad) + at + e));
          else
            __builtin_nontemporal_store(f32x4{o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]},
                                        reinterpret_cast<f32x4*>(static_cast<float*>(a.grad) + at + e));
        }
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int e = sub + LPR * v;
          if (e >= a.E) continue;
          if constexpr (BF16) static_cast<uint16_t*>(a.grad)[at + e] = f32_to_bf16(o[v]);
          else static_cast<float*>(a.grad)[at + e] = o[v];
        }
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) z[v] = next[v];
    live = live_next;
    live_next = live_then;
  }
}

// f(IntC<LPR>, IntC<V>) for the lanes and registers that a row of E experts takes.
template <int V>
struct RowC { static constexpr int value = V; };
template <class F>
static void for_experts(int E, F f) {
  if (E <= 16) f(RowC<4>{}, RowC<4>{});
  else if (E <= 64) f(RowC<16>{}, RowC<4>{});
  else if (E <= 256) f(RowC<64>{}, RowC<4>{});
  else if (E <= 512) f(RowC<64>{}, RowC<8>{});
  else if (E <= 1024) f(RowC<64>{}, RowC<16>{});
  else if (E <= 2048) f(RowC<64>{}, RowC<32>{});
  else f(RowC<64>{}, RowC<64>{});
}

// Workgroups of the first launch.  One that takes all rows, up to four a wavefront, is a call of
// one launch.  us with one and with two launches: 48 x 896 10.1 / 11.5, 64 x 896 11.8 / 11.4 (BF16
// 12.6 / 11.6), 64 x 512 8.9 / 11.4, 256 x 64 8.3 / 11.3, 32 x 2048 15.4 / 17.7, 32 x 4096 26.9 / 30.0
// (BF16 31.2 / 31.4).  One workgroup is bound by what its CU issues: 64 x 896 are 16 rows a SIMD, about
// 240 instructions each.  16384 x 896 logits take 20 us, 15.5 the first launch (3.8 TB/s) and 5.3 the
// second; in BF16 21, which the same instructions bound and not the half as many bytes.
int balance_parts(int T, int E) {
  const int rows = balance_waves(E <= 1024 ? 16 : 64) * (E <= 16 ? 16 : E <= 64 ? 4 : 1);
  if (T <= 4 * rows) return 1;
  const int G = (T + rows - 1) / rows, most = E <= 1024 ? kBalanceMaxParts / 2 : kBalanceMaxParts;
  return G < most ? G : most;
}

hipError_t launch_balance_loss(const BalanceArgs& a, hipStream_t stream) {
  const int G = balance_parts(a.T, a.E);
  const bool vec = a.E % 4 == 0 && reinterpret_cast<uintptr_t>(a.logits) % (a.bf16 ? 8 : 16) == 0;
  for_experts(a.E, [&](auto lpr, auto v) {
    constexpr int L = decltype(lpr)::value, V = decltype(v)::value;
    const dim3 grid(static_cast<unsigned>(G)), block(balance_waves(V) * 64);
    const size_t lds = static_cast<size_t>(a.E) * 4 * (balance_slots(V) + 1);
    if (a.bf16) {
      if (vec) balance_stats_kernel<true, L, V, true><<<grid, block, lds, stream>>>(a);
      else balance_stats_kernel<true, L, V, false><<<grid, block, lds, stream>>>(a);
    } else {
      if (vec) balance_stats_kernel<false, L, V, true><<<grid, block, lds, stream>>>(a);
      else balance_stats_kernel<false, L, V, false><<<grid, block, lds, stream>>>(a);
    }
  });
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || G == 1) return err;
  const unsigned joins = static_cast<unsigned>((a.E + kJoinExperts - 1) / kJoinExperts);
  balance_join_kernel<<<dim3(joins), dim3(kJoinGroups * kJoinExperts), 0, stream>>>(a, G);
  return hipGetLastError();
}

// Bound by the bytes: 16384 x 896 logits and as many values added (170 MB) 37 us, 4.6 TB/s (a large
// copy on the same card 5.1).  As many workgroups as the CUs hold at once (each goes on to further
// rows), and the rows go past the caches both ways: with eight workgroups per CU whatever the
// registers 42 us, through the caches 46; 8192 x 2048 logits 34 us and 58.  More than 2048 experts are
// 64 values a lane in four arrays, one wavefront a SIMD, and where E is no multiple of four they come
// one by one: 4096 x 4096 logits 41 us (BF16 58), 4096 x 4095 55 (BF16 115); the loss 59 and 62.
hipError_t launch_balance_loss_grad(const BalanceGradArgs& a, hipStream_t stream) {
  const int rows = 4 * (a.E <= 16 ? 16 : a.E <= 64 ? 4 : 1), blocks = (a.T + rows - 1) / rows;
  const uintptr_t all = reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.add) |
                        reinterpret_cast<uintptr_t>(a.grad);
  const bool vec = a.E % 4 == 0 && all % (a.bf16 ? 8 : 16) == 0;
  for_experts(a.E, [&](auto lpr, auto v) {
    constexpr int L = decltype(lpr)::value, V = decltype(v)::value;
    const int most = a.cus * (V <= 8 ? 8 : V <= 16 ? 5 : V <= 32 ? 3 : 1);
    const dim3 grid(static_cast<unsigned>(blocks < most ? blocks : most)), block(256);
    if (a.bf16) {
      if (vec) balance_grad_kernel<true, L, V, true><<<grid, block, 0, stream>>>(a);
      else balance_grad_kernel<true, L, V, false><<<grid, block, 0, stream>>>(a);
    } else {
      if (vec) balance_grad_kernel<false, L, V, true><<<grid, block, 0, stream>>>(a);
      else balance_grad_kernel<false, L, V, false><<<grid, block, 0, stream>>>(a);
    }
  });
  return hipGetLastError();
}

}  // namespace rmoe
