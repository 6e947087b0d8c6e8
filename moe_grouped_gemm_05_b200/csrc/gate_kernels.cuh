// Routing of tokens to experts, and its gradient: the step that makes the
// topk_ids of the MoE permutation and the weights of the combine.
//
//   s = softmax(l) or sigmoid(l);  c = s + bias
//   a group's score is the sum of its `group_top` best c; the topk_group best
//   groups stay; the topk best c among their experts are chosen, ties to the
//   lowest index; w_j = scale * s_j, or scale * s_j / sum_j s_j.
//
// Order.  The choice is that of a comparison in 64 bits.  Without a bias the
// experts are compared by their logits, which is exact.  Where scores are
// compared (a bias, or groups by sums of two), the kernel computes them in 32
// bits with a bound on their error, and a row in which two values that matter
// lie within twice that bound is decided again in 64 bits by the same warp.
//
// Backward, with g the gradient of w, r_j = s_j / sum s and ids fixed:
//   softmax, renormalised   dl_j = scale r_j (g_j - sum_i r_i g_i)
//   sigmoid, renormalised   dl_j = scale r_j (1 - s_j) (g_j - sum_i r_i g_i)
//   sigmoid                 dl_j = scale s_j (1 - s_j) g_j
//   softmax                 dl_e = scale p_e (G_e - sum_i p_i g_i),  G_e = g of e's slot or 0
// (every form but the last is zero outside the chosen experts).
#pragma once
#include <cuda_bf16.h>
#include <cfloat>
#include <cstdint>

#include "ptx.cuh"

namespace dg {

constexpr int kGateMaxTopk = 32;    // lane j of the warp holds slot j
constexpr int kGateMaxGroups = 32;  // lane g holds group g
constexpr int kGateWarps = 4;       // tokens of a block, one warp each

struct GateArgs {
  const void* logits;   // [T][E]
  const float* bias;    // [E] or nullptr
  int T, E, topk;
  int n_group, topk_group, group_top;
  int sigmoid, renorm;
  float scale;
  int32_t* ids;         // [T][topk]
  float* weights;       // [T][topk]
};

struct GateBackwardArgs {
  const void* logits;   // [T][E]
  const int32_t* ids;   // [T][topk]
  const float* d_weights;
  int T, E, topk;
  int sigmoid, renorm;
  float scale;
  void* d_logits;       // [T][E]
};

// ---------------------------------------------------------------- rows in registers
// Lane t of the warp holds elements [t*V, t*V + V) of a row; those behind its
// end read as `fill`.  With E % V == 0 a lane's elements are one aligned run,
// moved in accesses of up to 16 bytes.

template <int V>
__device__ __forceinline__ void gate_load_row(const float* row, int E, int lane, float fill, float (&l)[V]) {
  const int e0 = lane * V;
  if (E % V == 0) {
    if (e0 >= E) {
#pragma unroll
      for (int i = 0; i < V; ++i) l[i] = fill;
    } else if constexpr (V >= 4) {
#pragma unroll
      for (int i = 0; i < V / 4; ++i) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(row + e0) + i);
        l[4 * i] = v.x;
        l[4 * i + 1] = v.y;
        l[4 * i + 2] = v.z;
        l[4 * i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) l[i] = __ldg(row + e0 + i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = e0 + i < E ? __ldg(row + e0 + i) : fill;
  }
}

template <int V>
__device__ __forceinline__ void gate_load_row(const __nv_bfloat16* row, int E, int lane, float fill, float (&l)[V]) {
  const int e0 = lane * V;
  if (E % V == 0) {
    if (e0 >= E) {
#pragma unroll
      for (int i = 0; i < V; ++i) l[i] = fill;
    } else if constexpr (V >= 8) {
#pragma unroll
      for (int i = 0; i < V / 8; ++i) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(row + e0) + i);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          l[8 * i + 2 * j] = __uint_as_float(u[j] << 16);
          l[8 * i + 2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
        }
      }
    } else if constexpr (V >= 2) {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        const uint32_t u = __ldg(reinterpret_cast<const uint32_t*>(row + e0) + i);
        l[2 * i] = __uint_as_float(u << 16);
        l[2 * i + 1] = __uint_as_float(u & 0xFFFF0000u);
      }
    } else {
      l[0] = __bfloat162float(row[e0]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = e0 + i < E ? __bfloat162float(row[e0 + i]) : fill;
  }
}

template <int V>
__device__ __forceinline__ void gate_store_row(float* row, int E, int lane, const float (&l)[V]) {
  const int e0 = lane * V;
  if (E % V == 0) {
    if (e0 >= E) return;
    if constexpr (V >= 4) {
#pragma unroll
      for (int i = 0; i < V / 4; ++i)
        reinterpret_cast<float4*>(row + e0)[i] = make_float4(l[4 * i], l[4 * i + 1], l[4 * i + 2], l[4 * i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) row[e0 + i] = l[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (e0 + i < E) row[e0 + i] = l[i];
  }
}

__device__ __forceinline__ uint32_t gate_bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int V>
__device__ __forceinline__ void gate_store_row(__nv_bfloat16* row, int E, int lane, const float (&l)[V]) {
  const int e0 = lane * V;
  if (E % V == 0) {
    if (e0 >= E) return;
    if constexpr (V >= 8) {
#pragma unroll
      for (int i = 0; i < V / 8; ++i)
        reinterpret_cast<uint4*>(row + e0)[i] =
            make_uint4(gate_bf16x2(l[8 * i], l[8 * i + 1]), gate_bf16x2(l[8 * i + 2], l[8 * i + 3]),
                       gate_bf16x2(l[8 * i + 4], l[8 * i + 5]), gate_bf16x2(l[8 * i + 6], l[8 * i + 7]));
    } else if constexpr (V >= 2) {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) reinterpret_cast<uint32_t*>(row + e0)[i] = gate_bf16x2(l[2 * i], l[2 * i + 1]);
    } else {
      row[e0] = __float2bfloat16_rn(l[0]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (e0 + i < E) row[e0 + i] = __float2bfloat16_rn(l[i]);
  }
}

__device__ __forceinline__ float gate_at(const float* row, int e) { return __ldg(row + e); }
__device__ __forceinline__ float gate_at(const __nv_bfloat16* row, int e) { return __bfloat162float(row[e]); }

// ---------------------------------------------------------------- warp reductions

// A float's bits as an unsigned key in the same order (no NaN; -0 and +0 differ).
__device__ __forceinline__ uint32_t ordered_key(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

__device__ __forceinline__ float warp_max(float x) {
  return key_value(__reduce_max_sync(0xffffffffu, ordered_key(x)));
}
template <typename R>
__device__ __forceinline__ R warp_sum(R x) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// The two largest of {a1 >= a2} and {b1 >= b2}, in a1 >= a2.
template <typename R>
__device__ __forceinline__ void merge_top2(R& a1, R& a2, R b1, R b2) {
  const R lo = a1 < b1 ? a1 : b1;
  const R hi2 = a2 > b2 ? a2 : b2;
  a1 = a1 > b1 ? a1 : b1;
  a2 = lo > hi2 ? lo : hi2;
}

// A group's score from its two best values: the best, or the sum of both (of
// one where only one expert of the group can be chosen); -inf where none can.
template <typename R>
__device__ __forceinline__ R group_score(R a1, R a2, int group_top) {
  return group_top == 1 || a2 == -INFINITY ? a1 : a1 + a2;
}

// Scores of all groups for any group size: lane g gets group g's (-inf behind
// the last).  v: the lane's V values, -inf where an expert cannot be chosen.
template <typename R, int V>
__device__ __forceinline__ R group_scores_any(const R (&v)[V], int lane, int n_group, int gsize, int group_top) {
  R mine = -INFINITY;
  for (int g = 0; g < n_group; ++g) {
    R a1 = -INFINITY, a2 = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int rel = lane * V + i - g * gsize;
      if (rel >= 0 && rel < gsize) merge_top2(a1, a2, v[i], static_cast<R>(-INFINITY));
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
      const R b1 = __shfl_xor_sync(0xffffffffu, a1, o), b2 = __shfl_xor_sync(0xffffffffu, a2, o);
      merge_top2(a1, a2, b1, b2);
    }
    if (lane == g) mine = group_score(a1, a2, group_top);
  }
  return mine;
}

// ---------------------------------------------------------------- the choice in 64 bits

// Chooses the experts of one row in 64 bits; lane j returns the expert of slot
// j, or -1.  Rows come here when 32 bits cannot tell two values apart, so it
// is kept out of line and written for size, not speed.
template <typename LT, int V>
__device__ __noinline__ int gate_choose64(const GateArgs& p, const LT* row, int lane) {
  double c[V], k[V];
  double top = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane * V + i;
    c[i] = e < p.E ? static_cast<double>(gate_at(row, e)) : -INFINITY;
    k[i] = c[i];
    top = c[i] > top ? c[i] : top;
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    const double b = __shfl_xor_sync(0xffffffffu, top, o);
    top = b > top ? b : top;
  }
  double total = 0.0;
  if (!p.sigmoid) {
#pragma unroll
    for (int i = 0; i < V; ++i) total += exp(c[i] - top);
    total = warp_sum(total);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane * V + i;
    const bool dead = c[i] == -INFINITY || (p.bias && __ldg(p.bias + e) == -INFINITY);
    const double s = p.sigmoid ? 1.0 / (1.0 + exp(-c[i])) : exp(c[i] - top) / total;
    c[i] = dead ? -INFINITY : (p.bias ? s + static_cast<double>(__ldg(p.bias + e)) : s);
    k[i] = p.bias || dead ? c[i] : k[i];  // without a bias the experts go by their logits
  }
  if (p.n_group > 1) {
    const int gsize = p.E / p.n_group;
    const double mine = group_scores_any<double, V>(c, lane, p.n_group, gsize, p.group_top);
    int rank = 0;
    for (int j = 0; j < p.n_group; ++j) {
      const double o = __shfl_sync(0xffffffffu, mine, j);
      rank += o > mine || (o == mine && j < lane);
    }
    const uint32_t kept = __ballot_sync(0xffffffffu, lane < p.n_group && rank < p.topk_group);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (!((kept >> min(31, (lane * V + i) / gsize)) & 1)) k[i] = -INFINITY;
  }
  int mine_id = -1;
  for (int j = 0; j < p.topk; ++j) {
    double best = -INFINITY;
    int at = 0x7FFFFFFF;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (k[i] > best) {
        best = k[i];
        at = lane * V + i;
      }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
      const double b = __shfl_xor_sync(0xffffffffu, best, o);
      const int a = __shfl_xor_sync(0xffffffffu, at, o);
      if (b > best || (b == best && a < at)) {
        best = b;
        at = a;
      }
    }
    if (best == -INFINITY) break;
    if (lane == j) mine_id = at;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (lane * V + i == at) k[i] = -INFINITY;
  }
  return mine_id;
}

// ---------------------------------------------------------------- forward

// One warp a token.
//
// Error of a 32-bit score (u = 2^-24, __expf within 2 + 1.173|x| units of 2u):
//   sigmoid  s(1-s)(2 + 1.173|l|) 2u <= (0.5 + 0.27) 2u, with the sum and the
//            division at most 4u = 2^-22; c adds |c| u, |c| <= 1 + |bias|.
//   softmax  p (2^-18 + 2^-21) from the sum over at most 1024 terms and the
//            quotient, 0.61 * 2u from the exponent's argument: <= p 2^-17 + 2^-23.
// Two values closer than `near` (both errors, rounded up) are not told apart;
// a sum of two has twice the error.
template <typename LT, int V>
__global__ void __launch_bounds__(32 * kGateWarps) moe_gate_kernel(const GateArgs p) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kGateWarps + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const LT* row = static_cast<const LT*>(p.logits) + static_cast<size_t>(t) * p.E;
  int32_t* ids = p.ids + static_cast<size_t>(t) * p.topk;
  float* weights = p.weights + static_cast<size_t>(t) * p.topk;

  float l[V];
  gate_load_row<V>(row, p.E, lane, -INFINITY, l);
  bool bad = false;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    bad |= !(l[i] < INFINITY);  // +inf or NaN
    l[i] += 0.0f;               // -0 becomes +0, so that equal logits have equal keys
  }
  const bool sums = p.n_group > 1 && p.group_top > 1;
  const bool scored = p.bias != nullptr || sums;
  float top = 0.0f, total = 1.0f;
  if (!p.sigmoid && (scored || !p.renorm)) {
    float m = l[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = fmaxf(m, l[i]);
    top = warp_max(m);
    if (top == -INFINITY) top = 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) sum += expf(l[i] - top);
    total = warp_sum(sum);
  }
  // c: what groups are ranked by; key: what experts are ranked by (0: cannot be chosen)
  float c[V];
  uint32_t key[V];
  float near = 0.0f;
  if (scored) {
    float big = 0.0f;
    float b[V];
    if (p.bias) gate_load_row<V>(p.bias, p.E, lane, 0.0f, b);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float s = p.sigmoid ? __frcp_rn(1.0f + __expf(-l[i])) : __fdividef(__expf(l[i] - top), total);
      c[i] = s;
      if (p.bias) {
        bad |= !(b[i] < INFINITY);
        c[i] = s + b[i] + 0.0f;
        if (b[i] > -INFINITY) big = fmaxf(big, fabsf(b[i]));
        if (l[i] == -INFINITY) c[i] = -INFINITY;
      } else if (l[i] == -INFINITY) {
        c[i] = -INFINITY;
      }
      const float by = p.bias ? c[i] : l[i];
      key[i] = by == -INFINITY ? 0u : ordered_key(by);
    }
    near = 0x1p-21f + (p.sigmoid ? 0.0f : __fdividef(0x1p-16f, total));
    if (p.bias) near += 0x1p-22f * (1.0f + warp_max(big));
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      c[i] = l[i];
      key[i] = l[i] == -INFINITY ? 0u : ordered_key(l[i]);
    }
  }
  if (__any_sync(0xffffffffu, bad)) {
    // NaN or +inf among the logits or the bias: the token is not routed
    if (lane == 0) atomicOr(&g_dg_error, 0x20);
    if (lane < p.topk) {
      ids[lane] = -1;
      weights[lane] = 0.0f;
    }
    return;
  }

  bool unsure = false;
  if (p.n_group > 1) {
    const int gsize = p.E / p.n_group;
    const int span = gsize / V;  // lanes of a group, where its experts are whole lanes of a power of two
    const bool whole = gsize % V == 0 && (span & (span - 1)) == 0;
    float mine;
    int at;  // the group whose score this lane holds
    if (whole) {
      float a1 = c[0], a2 = -INFINITY;
#pragma unroll
      for (int i = 1; i < V; ++i) merge_top2(a1, a2, c[i], -INFINITY);
      for (int o = 1; o < span; o <<= 1) {
        const float b1 = __shfl_xor_sync(0xffffffffu, a1, o), b2 = __shfl_xor_sync(0xffffffffu, a2, o);
        merge_top2(a1, a2, b1, b2);
      }
      mine = group_score(a1, a2, p.group_top);
      at = lane / span;
    } else {
      mine = group_scores_any<float, V>(c, lane, p.n_group, gsize, p.group_top);
      at = lane;
    }
    // near for groups: twice an expert's, and the rounding of the sum
    const float gnear = scored ? (sums ? 2.0f * near + 0x1p-22f : near) : 0.0f;
    int above = 0, sure_above = 0, maybe_above = 0;
    for (int j = 0; j < p.n_group; ++j) {
      const float o = __shfl_sync(0xffffffffu, mine, whole ? j * span : j);
      above += o > mine || (o == mine && j < at);
      sure_above += o > mine + gnear;
      maybe_above += o >= mine - gnear && j != at;
    }
    const bool mine_kept = at < p.n_group && above < p.topk_group && mine > -INFINITY;
    if (scored && at < p.n_group && mine > -INFINITY)
      unsure = !(maybe_above < p.topk_group || sure_above >= p.topk_group);
    if (whole) {
      if (!mine_kept) {
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = 0u;
      }
    } else {
      const uint32_t kept = __ballot_sync(0xffffffffu, mine_kept);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (!((kept >> min(31, (lane * V + i) / gsize)) & 1)) key[i] = 0u;
    }
    unsure = __any_sync(0xffffffffu, unsure);
  }

  // The best key of the warp, topk times; one more shows whether the last
  // place was a close one.
  int mine_id = -1;
  if (!unsure) {
    const int rounds = p.bias ? p.topk + 1 : p.topk;
    float before = INFINITY;
    int before_id = -1;
    for (int j = 0; j < rounds; ++j) {
      uint32_t best = key[0];
#pragma unroll
      for (int i = 1; i < V; ++i) best = max(best, key[i]);
      const uint32_t all = __reduce_max_sync(0xffffffffu, best);
      if (all == 0u) break;
      const int src = __ffs(__ballot_sync(0xffffffffu, best == all)) - 1;
      int at = 0;
      if (lane == src) {
        bool found = false;
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (!found && key[i] == all) {
            found = true;
            key[i] = 0u;
            at = lane * V + i;
          }
      }
      at = __shfl_sync(0xffffffffu, at, src);
      if (p.bias) {
        const float v = key_value(all);
        if (before - v <= near &&
            !(gate_at(row, at) == gate_at(row, before_id) && __ldg(p.bias + at) == __ldg(p.bias + before_id))) {
          unsure = true;
          break;
        }
        before = v;
        before_id = at;
      }
      if (lane == j && j < p.topk) mine_id = at;
    }
  }
  if (unsure) mine_id = gate_choose64<LT, V>(p, row, lane);

  const bool has = mine_id >= 0;
  const float x = has ? gate_at(row, mine_id) : -INFINITY;
  float w;
  if (p.renorm) {
    // s_j / sum s from the ratios to the largest: no under- or overflow however small the scores
    const float m = warp_max(x);
    float v;
    if (p.sigmoid) v = x < 0.0f ? expf(x - fminf(m, 0.0f)) / (1.0f + expf(x)) : 1.0f / (1.0f + expf(-x));
    else v = expf(x - m);
    if (!has) v = 0.0f;
    w = v / warp_sum(v);
  } else if (p.sigmoid) {
    w = x < 0.0f ? expf(x) / (1.0f + expf(x)) : 1.0f / (1.0f + expf(-x));
  } else {
    w = expf(x - top) / total;
  }
  if (lane < p.topk) {
    ids[lane] = mine_id;
    weights[lane] = has ? p.scale * w : 0.0f;
  }
}

// ---------------------------------------------------------------- backward

// One warp a token: lane j holds slot j, the row is put together in shared
// memory and written once.
template <typename LT, int V>
__global__ void __launch_bounds__(32 * kGateWarps) moe_gate_backward_kernel(const GateBackwardArgs p) {
  __shared__ __align__(16) float rows[kGateWarps][32 * V];
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kGateWarps + (threadIdx.x >> 5);
  if (t >= p.T) return;
  float* acc = rows[threadIdx.x >> 5];
  const LT* row = static_cast<const LT*>(p.logits) + static_cast<size_t>(t) * p.E;
  LT* out = static_cast<LT*>(p.d_logits) + static_cast<size_t>(t) * p.E;

  int id = lane < p.topk ? __ldg(p.ids + static_cast<size_t>(t) * p.topk + lane) : -1;
  if (id < -1 || id >= p.E) {
    atomicOr(&g_dg_error, 0x2);
    id = -1;
  }
  const bool has = id >= 0;
  const float g = has ? __ldg(p.d_weights + static_cast<size_t>(t) * p.topk + lane) : 0.0f;
  const bool dense = !p.sigmoid && !p.renorm;
  float v = g;  // what the slot adds to its expert's place in `acc`
  if (!dense) {
    const float x = has ? gate_at(row, id) : -INFINITY;
    // 1 - s, and s / sum s as in the forward pass
    const float rest = x < 0.0f ? 1.0f / (1.0f + expf(x)) : expf(-x) / (1.0f + expf(-x));
    if (p.renorm) {
      float m = warp_max(x);
      if (m == -INFINITY) m = 0.0f;
      float r;
      if (p.sigmoid) r = x < 0.0f ? expf(x - fminf(m, 0.0f)) / (1.0f + expf(x)) : 1.0f / (1.0f + expf(-x));
      else r = expf(x - m);
      if (!has) r = 0.0f;
      const float sum = warp_sum(r);
      r = sum > 0.0f ? r / sum : 0.0f;
      const float mean = warp_sum(r * g);
      v = p.scale * r * (p.sigmoid ? rest : 1.0f) * (g - mean);
    } else {
      const float s = x < 0.0f ? expf(x) / (1.0f + expf(x)) : 1.0f / (1.0f + expf(-x));
      v = p.scale * s * rest * g;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) acc[lane + 32 * i] = 0.0f;
  __syncwarp();
  // an expert named twice in a row takes both slots' share, in slot order
  const uint32_t same = __match_any_sync(0xffffffffu, has ? id : -1 - lane);
  if (__all_sync(0xffffffffu, (same & (same - 1)) == 0u)) {
    if (has) acc[id] = v;
  } else {
    for (int j = 0; j < p.topk; ++j) {
      if (lane == j && has) acc[id] += v;
      __syncwarp();
    }
  }
  __syncwarp();
  float o[V];
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = acc[lane * V + i];
  if (dense && __any_sync(0xffffffffu, has)) {
    float l[V];
    gate_load_row<V>(row, p.E, lane, -INFINITY, l);
    float m = l[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = fmaxf(m, l[i]);
    m = warp_max(m);
    if (m == -INFINITY) m = 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      l[i] = expf(l[i] - m);
      sum += l[i];
    }
    sum = warp_sum(sum);
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    float mean = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      l[i] *= inv;
      mean += l[i] * o[i];
    }
    mean = warp_sum(mean);
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = p.scale * l[i] * (o[i] - mean);
  }
  gate_store_row<V>(out, p.E, lane, o);
}

}  // namespace dg
