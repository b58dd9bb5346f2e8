// moe.hip - the mixture-of-experts operators around the grouped GEMMs: routing (forward and
// backward), the layouts of the routed rows, the move of tokens into them with the per-token FP8
// cast, and the weighted way back (forward and backward).
//
// All of them are bound by HBM or, for small batches, by latency. No atomics on global memory
// and no order that depends on timing: every result is the same on every run.
#include <math.h>

#include <utility>

#include "dg_device.h"
#include "dg_launch.h"

namespace dg {
namespace {

template <int N>
struct Const {
  static constexpr int value = N;
};

// ---------------------------------------------------------------------------------
// routing
// ---------------------------------------------------------------------------------
// Order of the selection keys as unsigned integers: larger float, larger integer; -0 as +0; NaN
// below -infinity. 0 is left free for "not a candidate".
__device__ __forceinline__ uint32_t key_order(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  const uint32_t order = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
  return x != x ? 1u : order;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  if (k <= 1u) return -INFINITY;
  return __uint_as_float((k >> 31) ? (k & 0x7FFFFFFFu) : ~k);
}

// Reductions over the wave on the vector ALU: quads, halves and wholes of a row of 16 lanes by DPP,
// rows and halves of the wave by gfx950's lane swaps; every lane gets the result. `lanes` (a power
// of two) limits them to aligned runs of that many lanes.
template <typename Op>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t v, Op op, int lanes = 64) {
  if (lanes > 1) v = op(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));   // quad: 1 0 3 2
  if (lanes > 2) v = op(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));   // quad: 2 3 0 1
  if (lanes > 4) v = op(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, true));  // half row mirrored
  if (lanes > 8) v = op(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, true));  // row mirrored
  if (lanes > 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = op(r[0], r[1]);
  }
  if (lanes > 32) {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = op(r[0], r[1]);
  }
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
  return __uint_as_float(wave_reduce(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

template <bool kBf16>
__device__ __forceinline__ float load1(const void* base, int64_t elem) {
  if constexpr (kBf16) return bf16_to_f32(static_cast<const uint16_t*>(base)[elem]);
  else return static_cast<const float*>(base)[elem];
}
template <bool kBf16>
__device__ __forceinline__ void store1(void* base, int64_t elem, float v) {
  if constexpr (kBf16) static_cast<uint16_t*>(base)[elem] = (uint16_t)bf16_rne(v);
  else static_cast<float*>(base)[elem] = v;
}

// A token's row is held by L lanes (32: two tokens to a wave; 64), NPER consecutive experts each,
// -infinity past the last one. Rows whose length is a multiple of 4, held in runs of 4, are read and
// written in whole vectors.
template <int L>
__device__ __forceinline__ int seg_lane() {
  return threadIdx.x & (L - 1);
}
template <bool kBf16, int L, int NPER>
__device__ __forceinline__ void load_row(const void* base, int64_t t, int E, float (&x)[NPER]) {
  const int e0 = seg_lane<L>() * NPER;
  if (NPER % 4 == 0 && E % 4 == 0) {
    if constexpr (NPER % 4 == 0) {
#pragma unroll
      for (int i = 0; i < NPER; i += 4) {
        x[i] = x[i + 1] = x[i + 2] = x[i + 3] = -INFINITY;
        if (e0 + i < E) load4<kBf16>(base, t * E + e0 + i, &x[i]);
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < NPER; ++i) x[i] = e0 + i < E ? load1<kBf16>(base, t * E + e0 + i) : -INFINITY;
}
template <bool kBf16, int L, int NPER>
__device__ __forceinline__ void store_row(void* base, int64_t t, int E, const float (&x)[NPER]) {
  const int e0 = seg_lane<L>() * NPER;
  if (NPER % 4 == 0 && E % 4 == 0) {
    if constexpr (NPER % 4 == 0) {
#pragma unroll
      for (int i = 0; i < NPER; i += 4) {
        if (e0 + i >= E) break;
        if constexpr (kBf16)
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + t * E + e0 + i) =
              make_uint2(bf16_rne(x[i]) | (bf16_rne(x[i + 1]) << 16), bf16_rne(x[i + 2]) | (bf16_rne(x[i + 3]) << 16));
        else
          *reinterpret_cast<float4*>(static_cast<float*>(base) + t * E + e0 + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < NPER; ++i)
    if (e0 + i < E) store1<kBf16>(base, t * E + e0 + i, x[i]);
}

template <int L>
__device__ __forceinline__ uint32_t seg_max(uint32_t v) {
  return wave_reduce(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; }, L);
}
template <int L>
__device__ __forceinline__ float seg_max(float v) {
  return __uint_as_float(wave_reduce(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }, L));
}
template <int L>
__device__ __forceinline__ float seg_sum(float v) {
  return __uint_as_float(wave_reduce(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }, L));
}
// The value that lane l of this lane's row holds; l is the same throughout the wave.
template <int L>
__device__ __forceinline__ uint32_t seg_value(uint32_t v, int l) {
  const uint32_t a = (uint32_t)__builtin_amdgcn_readlane((int)v, l);
  if constexpr (L == 64) return a;
  const uint32_t b = (uint32_t)__builtin_amdgcn_readlane((int)v, l + 32);
  return (threadIdx.x & 32) ? b : a;
}

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// Softmax over the row: its maximum (0 for a row of -infinity alone) and the sum of e^(x - maximum).
template <int L, int NPER>
__device__ __forceinline__ void softmax_sums(const float (&x)[NPER], int E, float& mx, float& sum) {
  const int e0 = seg_lane<L>() * NPER;
  mx = x[0];
#pragma unroll
  for (int i = 1; i < NPER; ++i) mx = fmaxf(mx, x[i]);
  mx = seg_max<L>(mx);
  if (mx == -INFINITY) mx = 0.0f;
  sum = 0.0f;
#pragma unroll
  for (int i = 0; i < NPER; ++i) sum += e0 + i < E ? expf(x[i] - mx) : 0.0f;
  sum = seg_sum<L>(sum);
}
__device__ __forceinline__ float softmax_at(float x, float mx, float sum) { return sum == 0.0f ? 0.0f : expf(x - mx) / sum; }

// A row whose softmax is NaN: one that holds a NaN or +infinity.
template <int L, int NPER>
__device__ __forceinline__ bool row_is_nan(const float (&x)[NPER]) {
  bool found = false;
#pragma unroll
  for (int i = 0; i < NPER; ++i) found = found || !(x[i] < INFINITY);
  uint64_t any = __ballot(found);
  if (L == 32) any = (threadIdx.x & 32) ? any >> 32 : any & 0xFFFFFFFFu;
  return any != 0;
}

// A wave's LDS operations run in order; this keeps the compiler from moving others across, and waits.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// The best topk_groups groups of experts where groups are no whole runs of lanes: the keys of the
// others become 0. Keys and group values meet in LDS (E + 64 words a row); a lane takes every L-th group.
template <int L, int NPER>
__device__ __forceinline__ void keep_groups(uint32_t (&k)[NPER], const RouteProblem& p, uint32_t* lds) {
  const int sl = seg_lane<L>(), e0 = sl * NPER;
  const int per = p.E / p.groups;
  uint32_t* value = lds + p.E;
#pragma unroll
  for (int i = 0; i < NPER; ++i)
    if (e0 + i < p.E) lds[e0 + i] = k[i];
  wave_lds_fence();
  for (int g = sl; g < p.groups; g += L) {
    uint32_t first = 0, second = 0;
    for (int e = g * per; e < (g + 1) * per; ++e) {
      const uint32_t key = lds[e];
      second = max(second, min(first, key));
      first = max(first, key);
    }
    value[g] = key_order(key_value(first) + (p.group_top == 2 ? key_value(second) : 0.0f));
  }
  wave_lds_fence();
  uint64_t kept = 0;  // this lane's groups, at bit i for group sl + i * L
  for (int g = sl, i = 0; g < p.groups; g += L, ++i) {
    const uint32_t mine = value[g];
    int place = 0;
    for (int h = 0; h < p.groups; ++h) place += value[h] > mine || (value[h] == mine && h < g) ? 1 : 0;
    if (place < p.topk_groups) kept |= 1ull << i;
  }
  wave_lds_fence();
  for (int g = sl, i = 0; g < p.groups; g += L, ++i) value[g] = (uint32_t)(kept >> i) & 1;
  wave_lds_fence();
#pragma unroll
  for (int i = 0; i < NPER; ++i)
    if (e0 + i < p.E && value[(uint32_t)(e0 + i) / (uint32_t)per] == 0) k[i] = 0;
}

// Merge exchange (Batcher): the compare-exchange steps that sort n values, in order.
template <int N>
struct SortSteps {
  int count = 0;
  int a[64] = {}, b[64] = {};
  constexpr SortSteps() {
    int top = 1;
    while (top * 2 < N) top *= 2;
    for (int p = top; N > 1 && p > 0; p /= 2) {
      int q = top, r = 0, d = p;
      while (true) {
        for (int i = 0; i + d < N; ++i)
          if ((i & p) == r) {
            a[count] = i;
            b[count++] = i + d;
          }
        if (q == p) break;
        d = q - p;
        q /= 2;
        r = p;
      }
    }
  }
};
template <int N, int... I>
__device__ __forceinline__ void sort_steps(uint64_t (&v)[N], std::integer_sequence<int, I...>) {
  constexpr SortSteps<N> steps;
  const auto exchange = [&](auto a, auto b) {
    constexpr int x = decltype(a)::value, y = decltype(b)::value;
    const bool swap = v[y] > v[x];
    const uint64_t hi = swap ? v[y] : v[x], lo = swap ? v[x] : v[y];
    v[x] = hi;
    v[y] = lo;
  };
  (exchange(Const<steps.a[I]>(), Const<steps.b[I]>()), ...);
}
// A lane's keys in falling order, equal ones by index, and their indices at 4 bits each. An index
// travels below its key, turned round: one comparison orders both.
template <int N>
__device__ __forceinline__ void sort_run(uint32_t (&k)[N], uint64_t& order) {
  uint64_t v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = (uint64_t)k[i] << 32 | (uint32_t)(15 - i);
  sort_steps<N>(v, std::make_integer_sequence<int, SortSteps<N>().count>());
  order = 0;
#pragma unroll
  for (int i = N - 1; i >= 0; --i) {
    k[i] = (uint32_t)(v[i] >> 32);
    order = order << 4 | (15 - ((uint32_t)v[i] & 15));
  }
}

// L lanes per token; the row stays in registers. Each lane sorts its NPER keys once, so that the
// row's best key is the largest of L first ones: per choice a reduction, and a shift in the first lane that
// holds it. Bound by the vector ALU (a row of 256 is 1 KB but some 450 instructions, a fifth of them the
// sigmoids): two tokens to a wave share those of the reductions and the choices. 16384 tokens x 256
// experts, 8 of 4 of 8 groups: 14.8 us, 13.9 replayed (18.5 with one token to a wave and a second reduction for the
// holder, 16.4 with that alone); 5001 x 160 softmax: 6.4 us (10.2 with powers of two only as runs); one
// token: 4.3 us.
template <bool kBf16, int L, int NPER>
__global__ __launch_bounds__(256) void route_kernel(RouteProblem p, int64_t wg0) {
  extern __shared__ uint32_t lds[];
  __shared__ int picks[256 / L][kMaxTopk];
  const int sl = seg_lane<L>(), e0 = sl * NPER;
  const int64_t t = (wg0 + blockIdx.x) * (256 / L) + threadIdx.x / L;
  const int64_t wave_t = (wg0 + blockIdx.x) * (256 / L) + __builtin_amdgcn_readfirstlane(threadIdx.x / 64) * (64 / L);
  if (wave_t >= p.T) return;
  const bool live = t < p.T;  // the second token of the last wave may not be there: it repeats the last one
  const int64_t tt = live ? t : p.T - 1;
  const int E = p.E;
  float x[NPER];
  load_row<kBf16, L, NPER>(p.logits, tt, E, x);
  // selection keys: score + bias; without a bias the scores' order is the logits' own
  const bool by_logit = p.bias == nullptr && (p.groups == 1 || p.group_top == 1);
  float mx = 0.0f, sum = 0.0f;
  if (!p.sigmoid && !(by_logit && p.renormalise)) softmax_sums<L, NPER>(x, E, mx, sum);
  float key[NPER];
#pragma unroll
  for (int i = 0; i < NPER; ++i) key[i] = x[i];
  if (!by_logit) {
    float b[NPER];
#pragma unroll
    for (int i = 0; i < NPER; ++i) b[i] = 0.0f;
    if (p.bias != nullptr) load_row<false, L, NPER>(p.bias, 0, E, b);
    if (p.sigmoid) {
#pragma unroll
      for (int i = 0; i < NPER; ++i) key[i] = sigmoid(x[i]) + b[i];
    } else {
#pragma unroll
      for (int i = 0; i < NPER; ++i) key[i] = softmax_at(x[i], mx, sum) + b[i];
    }
  }
  uint32_t k[NPER];
#pragma unroll
  for (int i = 0; i < NPER; ++i) k[i] = e0 + i < E ? key_order(key[i]) : 0;
  const int per = E / p.groups, run = per / NPER;  // lanes of a group
  const bool whole_runs = per % NPER == 0 && (run & (run - 1)) == 0;
  if (p.groups > 1 && !whole_runs) keep_groups<L, NPER>(k, p, lds + (threadIdx.x / L) * (E + 64));
  uint64_t order;  // 4 bits each: which of the lane's experts
  sort_run<NPER>(k, order);
  if (p.groups > 1 && whole_runs) {
    uint32_t first = k[0], second = NPER > 1 ? k[NPER > 1 ? 1 : 0] : 0;
    const auto merge = [&](uint32_t f, uint32_t s) {
      second = max(min(first, f), max(second, s));
      first = max(first, f);
    };
    const auto dpp = [&](auto ctrl) {
      constexpr int c = decltype(ctrl)::value;
      merge((uint32_t)__builtin_amdgcn_mov_dpp((int)first, c, 0xF, 0xF, true),
            (uint32_t)__builtin_amdgcn_mov_dpp((int)second, c, 0xF, 0xF, true));
    };
    if (run > 1) dpp(Const<0xB1>());
    if (run > 2) dpp(Const<0x4E>());
    if (run > 4) dpp(Const<0x141>());
    if (run > 8) dpp(Const<0x140>());
    if (L == 64 && run > 16) {  // two groups; a whole row of lanes is one group
      const auto f = __builtin_amdgcn_permlane16_swap(first, first, false, false);
      const auto s = __builtin_amdgcn_permlane16_swap(second, second, false, false);
      first = f[0], second = s[0];
      merge(f[1], s[1]);
    }
    const float value = key_value(first) + (p.group_top == 2 ? key_value(second) : 0.0f);
    const uint32_t mine = key_order(value);
    const int g = sl / run;
    int place = 0;
    for (int h = 0; h < p.groups; ++h) {
      const uint32_t other = seg_value<L>(mine, h * run);
      place += other > mine || (other == mine && h < g) ? 1 : 0;
    }
    if (place >= p.topk_groups)
#pragma unroll
      for (int i = 0; i < NPER; ++i) k[i] = 0;
  }
  // of the lanes that hold the best key, the first has the lowest expert
  int* mine = picks[threadIdx.x / L];
  for (int j = 0; j < p.topk; ++j) {
    const uint32_t best = seg_max<L>(k[0]);
    bool first = k[0] == best;
    const uint64_t holders = __ballot(first);
    if (__popcll(holders) != 64 / L) {  // a tie somewhere
      const uint64_t row = L == 64 ? holders : (threadIdx.x & 32) ? holders >> 32 : holders & 0xFFFFFFFFu;
      first = first && (row & ((1ull << sl) - 1)) == 0;
    }
    if (first) {
      mine[j] = e0 + ((int)order & 15);
#pragma unroll
      for (int i = 0; i < NPER - 1; ++i) k[i] = k[i + 1];
      k[NPER - 1] = 0;
      order >>= 4;
    }
  }
  wave_lds_fence();
  // lane j of the row takes choice j (and choice j + 32 where the row has 32 lanes)
  constexpr int PICKS = 64 / L;
  int id[PICKS];
  float w[PICKS];
#pragma unroll
  for (int q = 0; q < PICKS; ++q) id[q] = sl + q * L < p.topk ? mine[sl + q * L] : 0;
  float total = 0.0f;
  if (p.sigmoid || !p.renormalise) {
#pragma unroll
    for (int q = 0; q < PICKS; ++q) {
      w[q] = 0.0f;
      if (sl + q * L < p.topk) {
        const float xj = load1<kBf16>(p.logits, tt * E + id[q]);
        w[q] = p.sigmoid ? sigmoid(xj) : softmax_at(xj, mx, sum);
      }
      total += w[q];
    }
  } else {
    // the softmax's own sum cancels: e^x over the chosen alone, without its underflow. A NaN or +infinity
    // anywhere in the row makes that sum NaN, and so the weights
    float top = -INFINITY;
#pragma unroll
    for (int q = 0; q < PICKS; ++q) {
      w[q] = sl + q * L < p.topk ? load1<kBf16>(p.logits, tt * E + id[q]) : -INFINITY;
      top = fmaxf(top, w[q]);
    }
    top = seg_max<L>(top);
    if (top == -INFINITY) top = 0.0f;
    const bool nan = row_is_nan<L, NPER>(x);
#pragma unroll
    for (int q = 0; q < PICKS; ++q) {
      w[q] = sl + q * L < p.topk ? (nan ? NAN : expf(w[q] - top)) : 0.0f;
      total += w[q];
    }
  }
  if (p.renormalise) {
    total = seg_sum<L>(total);
#pragma unroll
    for (int q = 0; q < PICKS; ++q)
      if (sl + q * L < p.topk) w[q] = total == 0.0f ? 0.0f : w[q] / total;
  }
#pragma unroll
  for (int q = 0; q < PICKS; ++q)
    if (live && sl + q * L < p.topk) {
      p.ids[t * p.topk + sl + q * L] = id[q];
      p.weights[t * p.topk + sl + q * L] = w[q] * p.scale;
    }
}

// d loss / d logits from d loss / d weights. With s the scores, C the chosen experts and
// S = sum of s over C: renormalised w_i = scale s_i / S gives ds_i = scale/S (g_i - sum_j g_j s_j / S),
// else ds_i = scale g_i. Sigmoid: dx = ds s (1 - s) on C, 0 elsewhere, 1 - s as the sigmoid of -x (the
// difference is 6 % off at x = 16 and 0 from 17 on); softmax:
// dx_j = s_j (ds_j - sum_C ds_i s_i). Renormalised, that last sum is 0 and s_i ds_i depends on
// s_i / S alone: of a softmax row the rest is then read only for a NaN or +infinity, which makes the whole
// row's scores, weights and gradient NaN. Of a sigmoid row the chosen logits are all that is read. The chosen experts' parts reach the lanes that write them through LDS.
// 16384 tokens x 256 experts: sigmoid 8.4 us, 17 MB written, bound by the chain of the ids, the logits that
// they name, and the row, more than by HBM; softmax 9.1 us renormalised, 10.0 not. 5001 x 160 softmax, not
// renormalised: 4.9 us.
template <bool kBf16, int L, int NPER>
__global__ __launch_bounds__(256) void route_backward_kernel(RouteProblem p, int64_t wg0) {
  __shared__ __attribute__((aligned(16))) float row[256 / L][L * NPER];
  const int sl = seg_lane<L>(), e0 = sl * NPER;
  const int64_t t = (wg0 + blockIdx.x) * (256 / L) + threadIdx.x / L;
  const int64_t wave_t = (wg0 + blockIdx.x) * (256 / L) + __builtin_amdgcn_readfirstlane(threadIdx.x / 64) * (64 / L);
  if (wave_t >= p.T) return;
  const bool live = t < p.T;
  const int64_t tt = live ? t : p.T - 1;
  const int E = p.E;
  float* mine = row[threadIdx.x / L];
  float x[NPER];
  if (!p.sigmoid) load_row<kBf16, L, NPER>(p.logits, tt, E, x);
  constexpr int PICKS = 64 / L;
  int id[PICKS];
  float xj[PICKS], g[PICKS], s[PICKS], own[PICKS];
#pragma unroll
  for (int q = 0; q < PICKS; ++q) {
    const int j = sl + q * L;
    id[q] = j < p.topk ? p.ids[tt * p.topk + j] : -1;
    if (id[q] < 0 || id[q] >= E) id[q] = -1;  // no expert: no gradient
    xj[q] = id[q] >= 0 ? load1<kBf16>(p.logits, tt * E + id[q]) : -INFINITY;
    g[q] = id[q] >= 0 ? p.dweights[tt * p.topk + j] * p.scale : 0.0f;
  }
  float dx[NPER];  // what every expert of the row gets, then with the chosen ones' own parts
  if (p.sigmoid || p.renormalise) {
    if (p.sigmoid) {
#pragma unroll
      for (int q = 0; q < PICKS; ++q) s[q] = id[q] >= 0 ? sigmoid(xj[q]) : 0.0f;
    } else {
      float top = -INFINITY;
#pragma unroll
      for (int q = 0; q < PICKS; ++q) top = fmaxf(top, xj[q]);
      top = seg_max<L>(top);
      if (top == -INFINITY) top = 0.0f;
#pragma unroll
      for (int q = 0; q < PICKS; ++q) s[q] = id[q] >= 0 ? expf(xj[q] - top) : 0.0f;
    }
    if (p.renormalise) {
      float S = 0.0f, gs = 0.0f;
#pragma unroll
      for (int q = 0; q < PICKS; ++q) S += s[q];
      S = seg_sum<L>(S);
      if (p.sigmoid) {
        // S may be 1e-38, and 1 / S or a product past fp32: only ratios of scores count, so a smaller S and all
        // of them times the power of two that brings it to [1/2, 1), which is exact
        const int up = max(-__builtin_amdgcn_frexp_expf(S), 0);
        S = ldexpf(S, up);
#pragma unroll
        for (int q = 0; q < PICKS; ++q) s[q] = ldexpf(s[q], up);
      }
#pragma unroll
      for (int q = 0; q < PICKS; ++q) gs += g[q] * s[q];
      gs = seg_sum<L>(gs);
#pragma unroll
      for (int q = 0; q < PICKS; ++q) g[q] = S == 0.0f || id[q] < 0 ? 0.0f : (g[q] - gs / S) / S;
    }
#pragma unroll
    for (int q = 0; q < PICKS; ++q) own[q] = p.sigmoid ? g[q] * s[q] * sigmoid(-xj[q]) : g[q] * s[q];
    const float rest = !p.sigmoid && row_is_nan<L, NPER>(x) ? NAN : 0.0f;
#pragma unroll
    for (int i = 0; i < NPER; ++i) dx[i] = rest;
  } else {
    float mx, sum;
    softmax_sums<L, NPER>(x, E, mx, sum);
    float inner = 0.0f;
#pragma unroll
    for (int q = 0; q < PICKS; ++q) {
      own[q] = id[q] >= 0 ? g[q] * softmax_at(xj[q], mx, sum) : 0.0f;
      inner += own[q];
    }
    inner = seg_sum<L>(inner);
#pragma unroll
    for (int i = 0; i < NPER; ++i) dx[i] = e0 + i < E ? -softmax_at(x[i], mx, sum) * inner : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < NPER; ++i) mine[e0 + i] = dx[i];
  wave_lds_fence();
#pragma unroll
  for (int q = 0; q < PICKS; ++q)
    if (id[q] >= 0) atomicAdd(&mine[id[q]], own[q]);  // in the order of the lanes, should an id come twice
  wave_lds_fence();
#pragma unroll
  for (int i = 0; i < NPER; ++i) dx[i] = mine[e0 + i];
  if (live) store_row<kBf16, L, NPER>(p.dlogits, t, E, dx);
}

// ---------------------------------------------------------------------------------
// layouts
// ---------------------------------------------------------------------------------
// A stable counting sort of the T * topk pairs (token, choice) by expert, one workgroup per
// expert and no exchange between them: a workgroup counts every expert's pairs itself (LDS
// integer atomics), which gives it its first row, and then places its own pairs in order. Waves take
// consecutive stretches of the ids, four ids a lane and kLayoutBatch loads in flight; ids that fit
// one batch per wave (32768 pairs) are read once.
// 32768 pairs over 32 experts: 11.5 us, bound by the vector ALU (some 150 instructions per 256 ids).
constexpr int kLayoutThreads = 1024, kLayoutWaves = kLayoutThreads / 64, kLayoutBatch = 8;

// Bits of a wave mask below this lane, added to `more`.
__device__ __forceinline__ int bits_below(uint64_t m, int more) {
  return (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, (uint32_t)more));
}

__global__ __launch_bounds__(kLayoutThreads) void layout_kernel(LayoutProblem p) {
  constexpr int kCopies = 4;  // of the counts, by lane: neighbouring pairs often go to the same expert
  __shared__ __attribute__((aligned(16))) int hist[kMaxExperts][kCopies];
  constexpr int kList = 8192;
  __shared__ int counts[kLayoutWaves];
  __shared__ int list[kList];
  const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int g = blockIdx.x, G = p.G;
  const int P = (int)p.pairs;
  constexpr int kStep = 256 * kLayoutBatch;  // ids of a wave's batch
  const int batches = (P + kLayoutWaves * kStep - 1) / (kLayoutWaves * kStep);
  // wave w takes the ids [w, w + 1) * stretch
  const int stretch = batches > 1 ? batches * kStep : ((P + kLayoutWaves - 1) / kLayoutWaves + 255) / 256 * 256;
  const int64_t lo = (int64_t)w * stretch;
  const int hi = (int)(lo + stretch < P ? lo + stretch : P);
  v4i ids[kLayoutBatch];
  auto load = [&](int b) {
#pragma unroll
    for (int u = 0; u < kLayoutBatch; ++u) {
      const int64_t i = lo + (int64_t)b * kStep + u * 256 + lane * 4;
      ids[u] = v4i{-1, -1, -1, -1};
      if (i - lane * 4 >= hi) break;  // the same for every lane
      if (i + 4 <= hi) ids[u] = *reinterpret_cast<const v4i*>(p.ids + i);
      else
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (i + k < hi) ids[u][k] = p.ids[i + k];
    }
  };
  if (!p.masked)
    for (int e = t; e < G * kCopies; e += kLayoutThreads) hist[e / kCopies][e % kCopies] = 0;
  __syncthreads();
  int count = 0;
  for (int b = 0; b < batches; ++b) {
    load(b);
#pragma unroll
    for (int u = 0; u < kLayoutBatch; ++u) {
      if (lo + (int64_t)b * kStep + u * 256 >= hi) break;  // the same for every lane
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int e = ids[u][k];
        count += __popcll(__ballot(e == g));
        if (!p.masked && e >= 0 && e < G) atomicAdd(&hist[e][lane % kCopies], 1);
      }
    }
  }
  if (lane == 0) counts[w] = count;
  __syncthreads();
  // every wave for itself: the pairs of the waves before it and of all; the rows of the experts
  // before this one and of all
  const auto add = [](uint32_t a, uint32_t b) { return a + b; };
  const int of_wave = lane < kLayoutWaves ? counts[lane] : 0;
  const int total = (int)wave_reduce((uint32_t)of_wave, add);
  int rank = (int)wave_reduce((uint32_t)(lane < w ? of_wave : 0), add);
  int mine = 0, used = 0;
  if (!p.masked) {
    for (int e = lane; e < G; e += 64) {
      const v4i c = *reinterpret_cast<const v4i*>(hist[e]);
      const int padded = (c[0] + c[1] + c[2] + c[3] + kQ - 1) / kQ * kQ;
      used += padded;
      if (e < g) mine += padded;
    }
    mine = (int)wave_reduce((uint32_t)mine, add);
    used = (int)wave_reduce((uint32_t)used, add);
  }
  const int64_t first = p.masked ? (int64_t)g * p.rows : mine;
  const int held = p.masked && total > p.rows ? (int)p.rows : total;  // the masked layout holds p.rows rows per expert
  const int my_rank = rank;
  // the expert's pairs in order, kList at a time (nearly always all of them), through LDS: written from
  // where they are found, a store instruction would carry the one or two lanes that match
  for (int start = 0; start == 0 || start < total; start += kList) {
    rank = my_rank - start;
    for (int b = 0; b < batches; ++b) {
      if (batches > 1) load(b);
#pragma unroll
      for (int u = 0; u < kLayoutBatch; ++u) {
        const int64_t i0 = lo + (int64_t)b * kStep + u * 256;
        if (i0 >= hi) break;
        int r = rank;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint64_t m = __ballot(ids[u][k] == g);
          r = bits_below(m, r);  // this expert's pairs of the lanes below
          rank += __popcll(m);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int e = ids[u][k];
          const int i = (int)i0 + lane * 4 + k;
          if (e == g) {
            if (r >= 0 && r < kList) list[r] = i;
            ++r;
          }
          if (g == 0 && start == 0 && (e < 0 || e >= G) && i < hi) p.pos[i] = -1;
        }
      }
    }
    __syncthreads();
    for (int r = start + t; r < total && r < start + kList; r += kLayoutThreads) {
      const int i = list[r - start];
      if (r < held) {
        p.row_pair[first + r] = i;
        if (!p.masked) p.m_indices[first + r] = g;
      }
      p.pos[i] = r < held ? (int)(first + r) : -1;
    }
    __syncthreads();
  }
  if (p.masked) {
    for (int64_t r = held + t; r < p.rows; r += kLayoutThreads) p.row_pair[first + r] = -1;
    if (t == 0) p.masked_m[g] = held;
    return;
  }
  const int64_t end = first + (int64_t)(total + kQ - 1) / kQ * kQ;
  for (int64_t r = first + total + t; r < end; r += kLayoutThreads) p.row_pair[r] = p.m_indices[r] = -1;
  for (int64_t r = used + (int64_t)g * kLayoutThreads + t; r < p.rows; r += (int64_t)G * kLayoutThreads)
    p.row_pair[r] = p.m_indices[r] = -1;
  if (t == 0) {
    p.offsets[g] = (int)first;
    if (g == 0) p.offsets[G] = used;
  }
}

// 16 bytes, past the caches (kStream) or through them.
template <bool kStream>
__device__ __forceinline__ v4i load16(const void* p) {
  if constexpr (kStream) return __builtin_nontemporal_load(static_cast<const v4i*>(p));
  else return *static_cast<const v4i*>(p);
}
template <bool kStream>
__device__ __forceinline__ void store16(void* p, v4i v) {
  if constexpr (kStream) __builtin_nontemporal_store(v, static_cast<v4i*>(p));
  else *static_cast<v4i*>(p) = v;
}

// The same sort for many pairs, in three launches over chunks of the ids: 131072 pairs take 17 us over
// 32 experts and 20 over 256, where every expert's workgroup looking at every id takes 36 and 35; 1048576
// over 256 take 104 (the second launch walks 1024 chunks in one workgroup). Until
// the last launch overwrites it, a chunk's own part of `pos` holds its counts.
constexpr int kLayoutChunk = 1024;
static_assert(kLayoutChunk >= kMaxExperts, "a chunk's counts fit in its part of pos");
constexpr int kChunkLoads = (2 * kLayoutChunk - 1 + 255) / 256;  // of 64 ids a wave; the last chunk may be nearly twice as long

__device__ __forceinline__ void chunk_range(const LayoutProblem& p, int chunks, int64_t& lo, int64_t& hi) {
  lo = (int64_t)blockIdx.x * kLayoutChunk;  // the last chunk takes what is left over
  hi = (int)blockIdx.x == chunks - 1 ? p.pairs : lo + kLayoutChunk;
}

// 1. Pairs per expert of each chunk; every row empty.
__global__ __launch_bounds__(256) void layout_count_kernel(LayoutProblem p, int chunks) {
  __shared__ int hist[kMaxExperts];
  for (int e = threadIdx.x; e < p.G; e += 256) hist[e] = 0;
  __syncthreads();
  int64_t lo, hi;
  chunk_range(p, chunks, lo, hi);
  int ids[kChunkLoads];  // all loads in flight at once
#pragma unroll
  for (int u = 0; u < kChunkLoads; ++u) {
    const int64_t i = lo + u * 256 + threadIdx.x;
    ids[u] = i < hi ? p.ids[i] : -1;
  }
#pragma unroll
  for (int u = 0; u < kChunkLoads; ++u)
    if (ids[u] >= 0 && ids[u] < p.G) atomicAdd(&hist[ids[u]], 1);
  const int64_t rows = p.masked ? p.rows * p.G : p.rows;
  for (int64_t r = (int64_t)blockIdx.x * 256 + threadIdx.x; r < rows; r += (int64_t)chunks * 256) {
    p.row_pair[r] = -1;
    if (!p.masked) p.m_indices[r] = -1;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.G; e += 256) p.pos[lo + e] = hist[e];
}

// 2. One workgroup, a thread per expert: its pairs in the chunks before each, its total, and the
// contiguous layout's offsets.
__global__ __launch_bounds__(kMaxExperts) void layout_scan_kernel(LayoutProblem p, int chunks) {
  __shared__ int wave_rows[kMaxExperts / 64];
  const int e = threadIdx.x, lane = e & 63, w = e >> 6;
  int total = 0;
  if (e < p.G) {
    constexpr int kBatch = 16;  // loads in flight
    for (int c0 = 0; c0 < chunks; c0 += kBatch) {
      int v[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) v[u] = c0 + u < chunks ? p.pos[(int64_t)(c0 + u) * kLayoutChunk + e] : 0;
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (c0 + u < chunks) p.pos[(int64_t)(c0 + u) * kLayoutChunk + e] = total;
        total += v[u];
      }
    }
  }
  if (p.masked) {
    if (e < p.G) p.masked_m[e] = total < p.rows ? total : (int)p.rows;
    return;
  }
  const int padded = (total + kQ - 1) / kQ * kQ;
  int upto = padded;  // inclusive sum over the wave
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int t = __shfl_up(upto, d, 64);
    if (lane >= d) upto += t;
  }
  if (lane == 63) wave_rows[w] = upto;
  __syncthreads();
  for (int k = 0; k < w; ++k) upto += wave_rows[k];
  if (e < p.G) p.offsets[e] = upto - padded;
  if (e == p.G - 1) p.offsets[p.G] = upto;
}

// 3. The chunk's pairs in order: a wave takes a stretch of it, 64 ids at a time; the lanes with one
// expert find each other by its bits.
__global__ __launch_bounds__(256) void layout_place_kernel(LayoutProblem p, int chunks) {
  __shared__ int next[4][kMaxExperts];  // next row in the expert, for each wave's pairs
  const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6), G = p.G;
  int64_t lo, hi;
  chunk_range(p, chunks, lo, hi);
  const int stretch = ((int)(hi - lo) + 255) / 256 * 64;
  const int64_t from = lo + (int64_t)w * stretch, to = from + stretch < hi ? from + stretch : hi;
  int ids[kChunkLoads];
#pragma unroll
  for (int u = 0; u < kChunkLoads; ++u) {
    const int64_t i = from + u * 64 + lane;
    ids[u] = i < to ? p.ids[i] : -1;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    for (int e = t; e < G; e += 256) next[k][e] = 0;
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kChunkLoads; ++u)
    if (ids[u] >= 0 && ids[u] < G) atomicAdd(&next[w][ids[u]], 1);
  __syncthreads();
  for (int e = t; e < G; e += 256) {
    int row = p.pos[lo + e];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int n = next[k][e];
      next[k][e] = row;
      row += n;
    }
  }
  __syncthreads();
  const int bits = 32 - __clz(G - 1 | 1);
#pragma unroll
  for (int u = 0; u < kChunkLoads; ++u) {
    if (from + u * 64 >= to) break;  // the same for every lane
    const int64_t i = from + u * 64 + lane;
    const int e = ids[u];
    const bool here = e >= 0 && e < G;
    uint64_t same = __ballot(here);
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot((e >> b) & 1);
      same &= (e >> b) & 1 ? set : ~set;
    }
    if (here) {
      const int before = bits_below(same, 0);
      const int r = next[w][e] + before;  // row in the expert
      if (!p.masked || r < p.rows) {
        const int64_t row = (p.masked ? (int64_t)e * p.rows : p.offsets[e]) + r;
        p.row_pair[row] = (int)i;
        if (!p.masked) p.m_indices[row] = e;
        p.pos[i] = (int)row;
      } else {
        p.pos[i] = -1;
      }
      wave_lds_fence();  // every lane has read before the first of each expert moves on
      if (before == 0) next[w][e] += __popcll(same);
    } else if (i < to) {
      p.pos[i] = -1;
    }
    wave_lds_fence();
  }
}

// ---------------------------------------------------------------------------------
// dispatch: gather and per-token FP8 cast
// ---------------------------------------------------------------------------------
// One wave per token and run of 8 K blocks: 16 consecutive values a lane, 8 lanes a block. The token
// is read and cast once, and its codes go to the row of each of its choices as 1 KB stores (by layout
// row instead, every token was read topk times: 192 against 74 us on 4096 tokens x 8 choices of 7168).
// Consecutive tokens stay on one XCD: rows that share a line of scales then meet in one L2 (60 against
// 84 us without). Codes too large for the caches are written past them (60 against 74 us), so that
// those lines stay; 4096 tokens x 8 choices of 7168 then move at 5.0 TB/s.
// The workgroups past the tokens (contiguous layout) write zero codes and scales into the rows
// without a token of one block in use each, which the GEMM reads.
template <bool kBf16, bool kPow2, bool kStream>
__global__ __launch_bounds__(256) void dispatch_kernel(DispatchProblem p, uint32_t token_wgs, int64_t wg0) {
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t nseg = (uint32_t)(p.kblocks + 7) / 8;
  const int64_t H = (int64_t)p.kblocks * kQ;
  const uint32_t wg = (uint32_t)wg0 + blockIdx.x;
  if (wg < token_wgs) {
    const uint32_t u = xcd_remap(wg, token_wgs) * 4 + (uint32_t)w;
    const uint32_t t = u / nseg, seg = u - t * nseg;
    if (t >= p.T) return;
    const int kb = (int)seg * 8 + (lane >> 3);  // this lane's K block
    const bool in = kb < p.kblocks;
    const int64_t col = (int64_t)seg * 1024 + lane * 16;
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      v[i] = v[i + 1] = v[i + 2] = v[i + 3] = 0.0f;
      if (in) load4<kBf16>(p.x, (int64_t)t * H + col + i, &v[i]);
    }
    float amax = fabsf(v[0]);
#pragma unroll
    for (int i = 1; i < 16; ++i) amax = fmaxf(amax, fabsf(v[i]));
    amax = seg_max<8>(amax);  // of numbers: NaN only for a chunk of NaN alone
    const float s = kPow2 ? pow2_ceil(amax / 448.0f) : amax / 448.0f;
    const v4i codes = quant16<kPow2>(v, s);
    const int64_t first = (int64_t)t * p.topk;
    for (int j = 0; j < p.topk; ++j) {
      const int64_t row = p.pos[first + j];
      if (row < 0 || row >= p.groups * p.rows) continue;
      if (!in) continue;
      store16<kStream>(p.q + row * H + col, codes);
      if ((lane & 7) == 0) {
        const int64_t g = p.masked ? (uint32_t)row / (uint32_t)p.rows : 0;
        p.sf[(g * p.kblocks + kb) * p.rows + (row - g * p.rows)] = s;
      }
    }
    return;
  }
  const int64_t block = wg - token_wgs, r0 = block * kQ + w * 32;
  if (p.row_pair[block * kQ] < 0) return;  // not in use
  uint64_t empty = __ballot(lane < 32 && p.row_pair[r0 + (lane & 31)] < 0);
  while (empty != 0) {
    const int64_t row = r0 + __ffsll((unsigned long long)empty) - 1;
    empty &= empty - 1;
    for (int64_t col = lane * 16; col < H; col += 1024) *reinterpret_cast<v4i*>(p.q + row * H + col) = v4i{0, 0, 0, 0};
    for (int kb = lane; kb < p.kblocks; kb += 64) p.sf[kb * p.rows + row] = 0.0f;
  }
}

// ---------------------------------------------------------------------------------
// combine
// ---------------------------------------------------------------------------------
__device__ __forceinline__ void unpack8(const v4i& raw, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_to_f32((uint32_t)raw[i] & 0xFFFFu);
    v[2 * i + 1] = bf16_to_f32((uint32_t)raw[i] >> 16);
  }
}
__device__ __forceinline__ v4i pack8(const float (&v)[8]) {
  v4i o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = (int)(bf16_rne(v[2 * i]) | (bf16_rne(v[2 * i + 1]) << 16));
  return o;
}

// Rows past the Infinity Cache's size are read and written past the caches (kStream): 4096 tokens x 8
// choices of 7168 (470 MB) forward 96 against 110 us, backward 188 against 204 us (5.3 TB/s; a plain copy
// runs at 5.1). Smaller ones are still there from the kernel that wrote them: 512 tokens, forward 12.7 us
// against 14.7 streamed, backward 24 against 30.
// out[t] = sum_j w[t,j] y[pos[t,j]], summed in fp32 in the order of the choices and rounded once.
// One wave per token and 512 columns.
template <bool kStream>
__global__ __launch_bounds__(256) void combine_kernel(CombineProblem p, int64_t wg0) {
  const int lane = threadIdx.x & 63;
  const int64_t u = (wg0 + blockIdx.x) * 4 + (threadIdx.x >> 6);
  const int64_t nseg = (p.H + 511) / 512;
  if (u >= p.T * nseg) return;
  const int64_t t = u / nseg, col = (u - t * nseg) * 512 + lane * 8;
  if (col >= p.H) return;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < p.topk; ++j) {
    const int64_t r = p.pos[t * p.topk + j];
    if (r < 0 || r >= p.rows) continue;
    const float w = p.weights ? p.weights[t * p.topk + j] : 1.0f;
    float v[8];
    unpack8(load16<kStream>(p.y + r * p.H + col), v);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = fmaf(w, v[i], acc[i]);
  }
  store16<kStream>(p.out + t * p.H + col, pack8(acc));
}

// dy[pos[t,j]] = w[t,j] dout[t], dweights[t,j] = <dout[t], y[pos[t,j]]>: one wave per pair. The
// workgroups past the pairs (contiguous layout, row_pair given) write zeros into the rows without a
// token of the used blocks.
template <bool kStream>
__global__ __launch_bounds__(256) void combine_backward_kernel(CombineProblem p, int64_t wg0) {
  const int lane = threadIdx.x & 63;
  const int64_t pairs = p.T * p.topk;
  const int64_t pair_wgs = (pairs + 3) / 4;
  const int64_t H = p.H, wg = wg0 + blockIdx.x;
  if (wg < pair_wgs) {
    const int64_t i = wg * 4 + (threadIdx.x >> 6);
    if (i >= pairs) return;
    const int64_t r = p.pos[i], t = i / p.topk;
    if (r < 0 || r >= p.rows) {
      if (lane == 0) p.dweights[i] = 0.0f;
      return;
    }
    const float w = p.weights[i];
    float dot = 0.0f;
    for (int64_t col = lane * 8; col < H; col += 512) {
      float d[8], v[8];
      unpack8(*reinterpret_cast<const v4i*>(p.dout + t * H + col), d);
      unpack8(load16<kStream>(p.y + r * H + col), v);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        dot = fmaf(d[k], v[k], dot);
        d[k] *= w;
      }
      store16<kStream>(p.dy + r * H + col, pack8(d));
    }
    dot = wave_sum(dot);
    if (lane == 0) p.dweights[i] = dot;
    return;
  }
  const int64_t r = (wg - pair_wgs) * 4 + (threadIdx.x >> 6);
  if (r >= p.rows || p.row_pair[r] >= 0 || p.row_pair[r & ~(int64_t)(kQ - 1)] < 0) return;
  for (int64_t col = lane * 8; col < H; col += 512) *reinterpret_cast<v4i*>(p.dy + r * H + col) = v4i{0, 0, 0, 0};
}

}  // namespace

// Lanes and experts per lane by the number of experts: 32 lanes a token up to 512, where a lane's
// sorted run is at most 16 long, else 64. Runs of 3, 5, 6, 10 and 12 beside the powers of two keep groups
// of experts in whole runs of lanes for 96, 160, 192, 320 and 384 experts.
#define DG_ROUTE_CONFIGS(X) \
  X(32, 1) X(32, 2) X(32, 3) X(32, 4) X(32, 5) X(32, 6) X(32, 8) X(32, 10) X(32, 12) X(32, 16) X(64, 10) X(64, 12) X(64, 16)

hipError_t launch_route(const RouteProblem& p, hipStream_t stream) {
#define DG_X(l, n)                                                                                               \
  if (p.E <= l * n) {                                                                                            \
    const int64_t wgs = (p.T + 256 / l - 1) / (256 / l);                                                         \
    const int per = p.E / p.groups, run = per / n;                                                               \
    const bool in_lds = p.groups > 1 && (per % n != 0 || (run & (run - 1)) != 0);                                \
    const size_t bytes = in_lds ? (size_t)(256 / l) * (p.E + 64) * 4 : 0;                                        \
    return launch_in_pieces(wgs, [&](dim3 grid, int64_t wg0) {                                                   \
      if (p.bf16) route_kernel<true, l, n><<<grid, dim3(256), bytes, stream>>>(p, wg0);                          \
      else route_kernel<false, l, n><<<grid, dim3(256), bytes, stream>>>(p, wg0);                                \
    });                                                                                                          \
  }
  DG_ROUTE_CONFIGS(DG_X)
#undef DG_X
  return hipErrorInvalidValue;
}

hipError_t launch_route_backward(const RouteProblem& p, hipStream_t stream) {
#define DG_X(l, n)                                                                                               \
  if (p.E <= l * n) {                                                                                            \
    return launch_in_pieces((p.T + 256 / l - 1) / (256 / l), [&](dim3 grid, int64_t wg0) {                       \
      if (p.bf16) route_backward_kernel<true, l, n><<<grid, dim3(256), 0, stream>>>(p, wg0);                     \
      else route_backward_kernel<false, l, n><<<grid, dim3(256), 0, stream>>>(p, wg0);                           \
    });                                                                                                          \
  }
  DG_ROUTE_CONFIGS(DG_X)
#undef DG_X
  return hipErrorInvalidValue;
}

hipError_t launch_layout(const LayoutProblem& p, hipStream_t stream) {
  // one launch up to about where three take no longer (32768 pairs: 11.3 us either way)
  if (p.pairs < 49152) {
    layout_kernel<<<dim3((unsigned)p.G), dim3(kLayoutThreads), 0, stream>>>(p);
    return hipGetLastError();
  }
  const int chunks = (int)(p.pairs / kLayoutChunk);
  layout_count_kernel<<<dim3((unsigned)chunks), dim3(256), 0, stream>>>(p, chunks);
  layout_scan_kernel<<<dim3(1), dim3(kMaxExperts), 0, stream>>>(p, chunks);
  layout_place_kernel<<<dim3((unsigned)chunks), dim3(256), 0, stream>>>(p, chunks);
  return hipGetLastError();
}

hipError_t launch_dispatch(const DispatchProblem& p, int bf16, int pow2, hipStream_t stream) {
  const int64_t token_wgs = (p.T * ((p.kblocks + 7) / 8) + 3) / 4;
  const int64_t wgs = token_wgs + (p.masked ? 0 : p.rows / kQ);
  if (wgs > 0x1FFFFFFF) return hipErrorInvalidValue;  // 2^31 waves: terabytes of tokens
  const uint32_t n = (uint32_t)token_wgs;
  // more codes than the chip's L2s (32 MB) hold
  const bool past = p.T * p.topk * p.kblocks * kQ > (int64_t)32 << 20;
  return launch_in_pieces(wgs, [&](dim3 grid, int64_t wg0) {
    const dim3 block(256);
    switch ((bf16 ? 4 : 0) + (pow2 ? 2 : 0) + (past ? 1 : 0)) {
      case 0: dispatch_kernel<false, false, false><<<grid, block, 0, stream>>>(p, n, wg0); break;
      case 1: dispatch_kernel<false, false, true><<<grid, block, 0, stream>>>(p, n, wg0); break;
      case 2: dispatch_kernel<false, true, false><<<grid, block, 0, stream>>>(p, n, wg0); break;
      case 3: dispatch_kernel<false, true, true><<<grid, block, 0, stream>>>(p, n, wg0); break;
      case 4: dispatch_kernel<true, false, false><<<grid, block, 0, stream>>>(p, n, wg0); break;
      case 5: dispatch_kernel<true, false, true><<<grid, block, 0, stream>>>(p, n, wg0); break;
      case 6: dispatch_kernel<true, true, false><<<grid, block, 0, stream>>>(p, n, wg0); break;
      default: dispatch_kernel<true, true, true><<<grid, block, 0, stream>>>(p, n, wg0); break;
    }
  });
}

// The rows that these pairs can name are more than the 256 MB of the Infinity Cache.
static bool past_caches(const CombineProblem& p) {
  const int64_t pairs = p.T * p.topk;
  return (pairs < p.rows ? pairs : p.rows) * p.H * 2 > (int64_t)256 << 20;
}

hipError_t launch_combine(const CombineProblem& p, hipStream_t stream) {
  return launch_in_pieces((p.T * ((p.H + 511) / 512) + 3) / 4, [&](dim3 grid, int64_t wg0) {
    if (past_caches(p)) combine_kernel<true><<<grid, dim3(256), 0, stream>>>(p, wg0);
    else combine_kernel<false><<<grid, dim3(256), 0, stream>>>(p, wg0);
  });
}

hipError_t launch_combine_backward(const CombineProblem& p, hipStream_t stream) {
  const int64_t wgs = (p.T * p.topk + 3) / 4 + (p.row_pair ? (p.rows + 3) / 4 : 0);
  return launch_in_pieces(wgs, [&](dim3 grid, int64_t wg0) {
    if (past_caches(p)) combine_backward_kernel<true><<<grid, dim3(256), 0, stream>>>(p, wg0);
    else combine_backward_kernel<false><<<grid, dim3(256), 0, stream>>>(p, wg0);
  });
}

}  // namespace dg
