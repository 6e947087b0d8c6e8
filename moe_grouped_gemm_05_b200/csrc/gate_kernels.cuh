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
//
// A token belongs to a team of L lanes, half a warp or a whole one.  All lanes
// of a warp take part in every shuffle and vote, whatever their team decides.
#pragma once
#include <cuda_bf16.h>
#include <cfloat>
#include <cstdint>

#include "ptx.cuh"

namespace dg {

constexpr int kGateMaxTopk = 32;    // lane j of the team holds slot j
constexpr int kGateMaxGroups = 32;  // lane g holds group g
constexpr int kGateWarps = 4;       // warps of a block (8 and 16 measured the same)
constexpr int kGateList = 32;       // listed experts of a token that are ranked at once

struct GateArgs {
  const void* logits;   // [T][E]
  const float* bias;    // [E] or nullptr
  int T, E, topk;
  int n_group, topk_group, group_top;
  int gsize;            // experts of a group
  int span_log2;        // a group belongs to 2^span_log2 lanes of its own, `width` experts each; or -1
  int width;
  int vec, full;        // every lane holds one aligned run of V experts or none; every lane holds V
  int deal;             // the kept groups' experts are dealt out over all lanes
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
// A lane holds `live` <= V elements of a row, from `first` on and `step` apart; the
// others read as `fill`.  vec: every lane has V of them or none, in aligned runs,
// which are moved in accesses of up to 16 bytes.

template <int V>
__device__ __forceinline__ void gate_load_row(const float* row, int first, int step, int live, bool vec,
                                              float fill, float (&l)[V]) {
  if (vec) {
    if (live == 0) {
#pragma unroll
      for (int i = 0; i < V; ++i) l[i] = fill;
    } else if constexpr (V >= 4) {
#pragma unroll
      for (int i = 0; i < V / 4; ++i) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(row + first) + i);
        l[4 * i] = v.x;
        l[4 * i + 1] = v.y;
        l[4 * i + 2] = v.z;
        l[4 * i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) l[i] = __ldg(row + first + i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = i < live ? __ldg(row + first + i * step) : fill;
  }
}

template <int V>
__device__ __forceinline__ void gate_load_row(const __nv_bfloat16* row, int first, int step, int live, bool vec,
                                              float fill, float (&l)[V]) {
  if (vec) {
    if (live == 0) {
#pragma unroll
      for (int i = 0; i < V; ++i) l[i] = fill;
    } else if constexpr (V >= 8) {
#pragma unroll
      for (int i = 0; i < V / 8; ++i) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(row + first) + i);
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
        const uint32_t u = __ldg(reinterpret_cast<const uint32_t*>(row + first) + i);
        l[2 * i] = __uint_as_float(u << 16);
        l[2 * i + 1] = __uint_as_float(u & 0xFFFF0000u);
      }
    } else {
      l[0] = __bfloat162float(row[first]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = i < live ? __bfloat162float(row[first + i * step]) : fill;
  }
}

template <int V>
__device__ __forceinline__ void gate_store_row(float* row, int first, int step, int live, bool vec,
                                               const float (&l)[V]) {
  if (vec) {
    if (live == 0) return;
    if constexpr (V >= 4) {
#pragma unroll
      for (int i = 0; i < V / 4; ++i)
        reinterpret_cast<float4*>(row + first)[i] = make_float4(l[4 * i], l[4 * i + 1], l[4 * i + 2], l[4 * i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) row[first + i] = l[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < live) row[first + i * step] = l[i];
  }
}

__device__ __forceinline__ uint32_t gate_bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int V>
__device__ __forceinline__ void gate_store_row(__nv_bfloat16* row, int first, int step, int live, bool vec,
                                               const float (&l)[V]) {
  if (vec) {
    if (live == 0) return;
    if constexpr (V >= 8) {
#pragma unroll
      for (int i = 0; i < V / 8; ++i)
        reinterpret_cast<uint4*>(row + first)[i] =
            make_uint4(gate_bf16x2(l[8 * i], l[8 * i + 1]), gate_bf16x2(l[8 * i + 2], l[8 * i + 3]),
                       gate_bf16x2(l[8 * i + 4], l[8 * i + 5]), gate_bf16x2(l[8 * i + 6], l[8 * i + 7]));
    } else if constexpr (V >= 2) {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) reinterpret_cast<uint32_t*>(row + first)[i] = gate_bf16x2(l[2 * i], l[2 * i + 1]);
    } else {
      row[first] = __float2bfloat16_rn(l[0]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < live) row[first + i * step] = __float2bfloat16_rn(l[i]);
  }
}

__device__ __forceinline__ float gate_at(const float* row, int e) { return __ldg(row + e); }
__device__ __forceinline__ float gate_at(const __nv_bfloat16* row, int e) { return __bfloat162float(row[e]); }

// ---------------------------------------------------------------- reductions over a team

// Largest of the team's values (no NaN among them).
template <int L>
__device__ __forceinline__ float team_max(float x) {
  if constexpr (L == 32) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
  } else {
#pragma unroll
    for (int o = L / 2; o >= 1; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
  }
}
template <int L, typename R>
__device__ __forceinline__ R team_sum(R x) {
#pragma unroll
  for (int o = L / 2; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
// The lanes of the team on which p holds, and whether it holds on some.
template <int L>
__device__ __forceinline__ uint32_t team_ballot(bool p, int lane) {
  const uint32_t b = __ballot_sync(0xffffffffu, p);
  return L == 32 ? b : b >> (lane & ~(L - 1)) & ((1u << (L & 31)) - 1u);
}
template <int L>
__device__ __forceinline__ bool team_any(bool p, int lane) {
  return team_ballot<L>(p, lane) != 0;
}

// The k-th largest of the team's values.  Of a whole warp, equal values count
// once (which gives a smaller one, or -inf).
template <int L>
__device__ __forceinline__ float team_kth(float x, int k, int lane) {
  if constexpr (L == 32) {
    float kth = -INFINITY;
    for (int j = 0; j < k; ++j) {
      kth = team_max<L>(x);
      x = x == kth ? -INFINITY : x;
    }
    return kth;
  } else {
    // a bitonic sorting network, descending
#pragma unroll
    for (int size = 2; size <= L; size <<= 1)
#pragma unroll
      for (int o = size / 2; o >= 1; o >>= 1) {
        const float y = __shfl_xor_sync(0xffffffffu, x, o);
        const bool upper = (lane & o) != 0, up = size < L && (lane & size) != 0;
        x = upper == up ? fmaxf(x, y) : fminf(x, y);
      }
    return __shfl_sync(0xffffffffu, x, k - 1, L);
  }
}

// max(a, |b|), a NaN's place taken by NaN.
__device__ __forceinline__ float max_abs_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
  return r;
}

// 2^x (within 2^-22 relative) and 1/x (within 2^-23) by the approximate
// instructions; subnormals are taken as zero.
__device__ __forceinline__ float fast_exp2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float fast_rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
constexpr float kLog2e = 1.4426950408889634f;

// n += (x >= bound); and, where x >= bound, (x, e) to the shared list at `to`,
// which moves on.  Written out, since the compiler makes branches of them.
__device__ __forceinline__ void count_from(int& n, float x, float bound) {
  asm("{\n\t.reg .pred p;\n\tsetp.ge.f32 p, %1, %2;\n\t@p add.s32 %0, %0, 1;\n\t}" : "+r"(n) : "f"(x), "f"(bound));
}
__device__ __forceinline__ void list_from(uint32_t& to, float x, int e, float bound) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ge.f32 p, %1, %3;\n\t@p st.shared.v2.b32 [%0], {%1, %2};\n\t"
      "@p add.u32 %0, %0, 8;\n\t}"
      : "+r"(to)
      : "f"(x), "r"(e), "f"(bound)
      : "memory");
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
// A sum beyond the type's range is its largest value, so that a group of two
// experts with the lowest bias can still be kept.
__device__ __forceinline__ float group_score(float a1, float a2, int group_top) {
  return group_top == 1 || a2 == -INFINITY ? a1 : fminf(fmaxf(a1 + a2, -FLT_MAX), FLT_MAX);
}
__device__ __forceinline__ double group_score(double a1, double a2, int group_top) {
  return group_top == 1 || a2 == -INFINITY ? a1 : a1 + a2;  // (of 32-bit biases: within range)
}

// The two best values of each group for any group size: lane g of the team gets
// group g's in m1 >= m2 (-inf behind the last).  v: the lane's V values, -inf
// where an expert cannot be chosen.
template <typename R, int L, int V>
__device__ __forceinline__ void group_best_any(const R (&v)[V], int tl, int n_group, int gsize, R& m1, R& m2) {
  m1 = m2 = -INFINITY;
  for (int g = 0; g < n_group; ++g) {
    R a1 = -INFINITY, a2 = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int rel = tl * V + i - g * gsize;
      if (rel >= 0 && rel < gsize) merge_top2(a1, a2, v[i], static_cast<R>(-INFINITY));
    }
#pragma unroll
    for (int o = L / 2; o >= 1; o >>= 1) {
      const R b1 = __shfl_xor_sync(0xffffffffu, a1, o), b2 = __shfl_xor_sync(0xffffffffu, a2, o);
      merge_top2(a1, a2, b1, b2);
    }
    if (tl == g) {
      m1 = a1;
      m2 = a2;
    }
  }
}

// ---------------------------------------------------------------- the choice in 64 bits

// Sum of exp(l - top) over the row in 64 bits (every lane of the team returns it).
template <typename LT, int L>
__device__ __noinline__ double gate_total64(const LT* row, int E, int tl, float top) {
  double sum = 0.0;
  for (int e = tl; e < (E + L - 1) / L * L; e += L)
    sum += e < E ? exp(static_cast<double>(gate_at(row, e)) - static_cast<double>(top)) : 0.0;
  return team_sum<L>(sum);
}

// c of expert e in 64 bits; total64 from gate_total64 (softmax only).
template <typename LT>
__device__ __noinline__ double gate_score64(const GateArgs& p, const LT* row, int e, float top, double total64) {
  const double x = gate_at(row, e);
  const double s = p.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - static_cast<double>(top)) / total64;
  return p.bias ? s + static_cast<double>(__ldg(p.bias + e)) : s;
}

// Chooses the experts of a row in 64 bits; lane j of the team returns the
// expert of slot j, or -1.  Rows come here when 32 bits cannot tell values
// apart and more than the listed candidates are in question, so it is kept out
// of line and written for size, not speed.
template <typename LT, int L, int V>
__device__ __noinline__ int gate_choose64(const GateArgs& p, const LT* row, int tl, float top) {
  double c[V], k[V];
  const double total = p.sigmoid ? 1.0 : gate_total64<LT, L>(row, p.E, tl, top);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = tl * V + i;
    const double x = e < p.E ? static_cast<double>(gate_at(row, e)) : -INFINITY;
    const bool dead = x == -INFINITY || (p.bias && __ldg(p.bias + e) == -INFINITY);
    c[i] = dead ? -INFINITY : gate_score64(p, row, e, top, total);
    k[i] = p.bias || dead ? c[i] : x;  // without a bias the experts go by their logits
  }
  if (p.n_group > 1) {
    double m1, m2;
    group_best_any<double, L, V>(c, tl, p.n_group, p.gsize, m1, m2);
    const double mine = group_score(m1, m2, p.group_top);
    int rank = 0;
    for (int j = 0; j < p.n_group; ++j) {
      const double o = __shfl_sync(0xffffffffu, mine, j, L);
      rank += o > mine || (o == mine && j < tl);
    }
    const bool kept = tl < p.n_group && rank < p.topk_group;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (!__shfl_sync(0xffffffffu, kept, min(L - 1, (tl * V + i) / p.gsize), L)) k[i] = -INFINITY;
  }
  int mine_id = -1;
  for (int j = 0; j < p.topk; ++j) {
    double best = -INFINITY;
    int at = 0x7FFFFFFF;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (k[i] > best) {
        best = k[i];
        at = tl * V + i;
      }
#pragma unroll
    for (int o = L / 2; o >= 1; o >>= 1) {
      const double b = __shfl_xor_sync(0xffffffffu, best, o);
      const int a = __shfl_xor_sync(0xffffffffu, at, o);
      if (b > best || (b == best && a < at)) {
        best = b;
        at = a;
      }
    }
    if (tl == j && best > -INFINITY) mine_id = at;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (tl * V + i == at) k[i] = -INFINITY;
  }
  return mine_id;
}

// ---------------------------------------------------------------- forward

// Error of a 32-bit score (u = 2^-24).  ex2.approx is within 2^-22 = 4u
// relative, rcp.approx within 2^-23 = 2u; the argument x log2(e) of ex2 is off
// by 2u |x| log2(e) (the constant's rounding and the product's), which is 2u |x|
// relative in the exponential.
//   sigmoid  s(1-s)(4 + 2|l|) u <= (1 + 0.45) u, the sum u, the quotient 2u:
//            below 5u.
//   softmax  p |x| 2u <= 0.74u and 4u p from the exponential; from the sum (at
//            most 1024 terms, in 64 bits (2 + 2 * 6.94) u of their own and 37 u
//            of additions) and the quotient 60u p: <= p 2^-17 + u.
// That is `e0`.  c = s + b adds |c| u, and at most 1, since b itself lies within 1 of
// s + b: a bias of any size, the type's lowest among them, leaves values at a distance
// told apart.  Values a < k can be out of order only where k - a is at most both errors
// together, and then |a| <= |k| + (k - a): so within `gate_near` of k, which k alone
// decides.  A sum of two has both terms' errors and its own, at most u |sum| and at
// most the smaller term (the larger one is a 32-bit number too; so with the sum cut off
// at the type's range).
//
// The choice.  The topk-th largest of the lanes' best values is a lower bound
// of the topk-th best value of the row, since so many values reach it, and few
// values do (for 256 experts, topk 8: about eleven).  Those (and the ones
// within `gate_near` below it) are put together in shared memory, and each
// lane counts the ones before its own.  That takes the place of topk rounds of
// finding and removing the best (which serve the rows with more than 32).
//
// Measured, 16384 tokens: 256 experts in 8 groups, topk 8, 16.2 us (topk rounds
// 37.9), the same with a whole group or all but one of its experts pushed out by a
// bias of -1e9 or the type's lowest value, 18.9 us with a group masked; without groups
// 13.4, without bias 11.6; 64 experts, softmax, topk 6, 6.2 us (a whole warp a token
// 9.4); 160 experts in 8 groups, 3 kept, 18.8 us (47.6 before groups of any size had
// lanes of their own and few kept experts were dealt out).  Bound by issue, some 740
// instructions a token of 256 experts in groups; more resident warps or larger blocks
// change nothing.
__device__ __forceinline__ float gate_near(float e0, float k) {
  return 2.0f * e0 + fminf(0x1.001p-23f * (1.0f + fabsf(k)), 3.0f);
}
// Error of a group's score, made of a1 or of a1 >= a2.
__device__ __forceinline__ float group_error(float e0, float a1, float a2, int group_top) {
  constexpr float u = 0x1.001p-24f;
  const float x1 = fabsf(a1), x2 = fabsf(a2), err = e0 + fminf(u * x1, 1.0f);
  if (group_top == 1 || a2 == -INFINITY) return err;
  const float sum = fabsf(a1 + a2);
  return err + e0 + fminf(u * x2, 1.0f) + fminf(sum < INFINITY ? u * sum : INFINITY, fminf(x1, x2));
}
// No less than group_error but for a sum that was cut off at the type's range, in fewer
// steps; with two units of `mine` for the roundings of mine + and - the margin.  (A cut off
// sum is right where this is used: the true one of a group that is not kept is lower still,
// at the top of the range groups are equal, and at its bottom none that is left out has a
// score.)  Taken for each group by itself, so that one with experts pushed out by a bias of
// any size brings no other into question.
__device__ __forceinline__ float group_margin(float e0, float a1, float a2, float mine, int group_top) {
  const float x2 = group_top == 1 || a2 == -INFINITY ? 0.0f : fabsf(a2);
  return 2.0f * e0 + fminf(0x1.01p-24f * (fabsf(a1) + x2), 2.0f) + 0x1.81p-23f * fabsf(mine);
}

template <typename LT, int L, int V, bool SIGMOID, bool BIAS>
__global__ void __launch_bounds__(32 * kGateWarps) moe_gate_kernel(const __grid_constant__ GateArgs p) {
  constexpr int kTeams = 32 * kGateWarps / L;
  constexpr int kOwn = kGateList / L;            // listed experts of a lane
  __shared__ float2 lists[kTeams][L * V];        // value, expert
  __shared__ int counts[kTeams];
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int tl = threadIdx.x & (L - 1);
  const int team = threadIdx.x / L;
  float2* list = lists[team];
  int* count = counts + team;
  const int t0 = blockIdx.x * kTeams + (threadIdx.x >> 5) * (32 / L);  // the warp's first token
  if (t0 >= p.T) return;
  const int t = t0 + (L == 32 ? 0 : lane / L);
  const bool mine_is = t < p.T;  // (a last odd token leaves a team without one)
  const LT* row = static_cast<const LT*>(p.logits) + static_cast<size_t>(mine_is ? t : t0) * p.E;

  const bool sums = p.n_group > 1 && p.group_top > 1;
  const bool scored = BIAS || sums;
  // This lane's experts.  With groups, each group has lanes of its own (where its
  // experts fit into them); without, a row of whole runs of V is cut into those,
  // and any other is dealt out an expert at a time.  (vec: the first line has it in
  // both ways, since groups then fill their lanes.)
  int first = tl * V, step = 1, live = first < p.E ? V : 0;
  if (!p.vec) {
    if (p.n_group == 1) {
      first = tl;
      step = L;
      live = max(0, (p.E - tl + L - 1) / L);
    } else if (p.span_log2 >= 0) {
      const int g = tl >> p.span_log2, part = (tl & ((1 << p.span_log2) - 1)) * p.width;
      first = g * p.gsize + part;
      live = g < p.n_group ? min(p.width, max(0, p.gsize - part)) : 0;
    } else {
      live = min(V, max(0, p.E - first));
    }
  }
  float l[V], c[V];
  gate_load_row<V>(row, first, step, live, p.vec, -FLT_MAX, l);
  if (BIAS) gate_load_row<V>(p.bias, first, step, live, p.vec, 0.0f, c);
  float big = 0.0f, largest = 0.0f;  // the largest |logit| and |bias|: below infinity when nothing is masked or bad
#pragma unroll
  for (int i = 0; i < V; ++i) {
    big = max_abs_nan(big, l[i]);
    if (BIAS) largest = max_abs_nan(largest, c[i]);
  }
  float top = 0.0f, total = 1.0f;
  if (!SIGMOID && (scored || !p.renorm)) {
    float m = l[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = fmaxf(m, l[i]);
    top = team_max<L>(m);
    if (top == -INFINITY) top = 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) sum += i < live ? expf(l[i] - top) : 0.0f;
    total = team_sum<L>(sum);
  }
  float e0 = 0.0f;
  if (scored) {
    const float inv = SIGMOID ? 1.0f : fast_rcp(total);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float s = SIGMOID ? fast_rcp(1.0f + fast_exp2(-kLog2e * l[i])) : fast_exp2(kLog2e * (l[i] - top)) * inv;
      c[i] = BIAS ? s + c[i] : s;
    }
    e0 = 0x1.4p-22f + (SIGMOID ? 0.0f : 0x1p-17f * inv);  // 5u
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = l[i];
  }
  // masks, and rows that are not numbers
  if (__any_sync(0xffffffffu, !(big < INFINITY) || !(largest < INFINITY))) {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      bad |= i < live && !(l[i] < INFINITY);
      if (l[i] == -INFINITY) c[i] = -INFINITY;
      if (BIAS) {
        const float b = i < live ? __ldg(p.bias + first + i * step) : 0.0f;
        bad |= !(b < INFINITY);
        if (b == -INFINITY) c[i] = -INFINITY;
      }
    }
    if (team_any<L>(bad, lane)) {
      // NaN or +inf among the logits or the bias: no expert can be chosen
      if (tl == 0) atomicOr(&g_dg_error, 0x20);
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] = -INFINITY;
    }
  }
  if (!p.full) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i >= live) c[i] = -INFINITY;
  }
  int expert[V];
#pragma unroll
  for (int i = 0; i < V; ++i) expert[i] = first + i * step;

  bool unsure = false;  // the token needs the choice in 64 bits (the team agrees)
  if (p.n_group > 1) {
    const bool whole = p.span_log2 >= 0;
    const int span = whole ? 1 << p.span_log2 : 1;
    const int at = whole ? tl >> p.span_log2 : tl;  // the group whose score this lane holds
    float a1 = c[0], a2 = -INFINITY;  // the group's two best values
    if (whole) {
#pragma unroll
      for (int i = 1; i < V; ++i) {
        a2 = fmaxf(a2, fminf(a1, c[i]));
        a1 = fmaxf(a1, c[i]);
      }
      for (int o = 1; o < span; o <<= 1) {
        const float b1 = __shfl_xor_sync(0xffffffffu, a1, o), b2 = __shfl_xor_sync(0xffffffffu, a2, o);
        a2 = fmaxf(fminf(a1, b1), fmaxf(a2, b2));
        a1 = fmaxf(a1, b1);
      }
    } else {
      group_best_any<float, L, V>(c, tl, p.n_group, p.gsize, a1, a2);
    }
    const float mine = group_score(a1, a2, p.group_top);
    // lanes behind the last group have -inf, as groups without an expert to choose
    const bool some = mine > -INFINITY;
    // the topk_group-th best score
    const float kth = team_kth<L>(mine, L == 32 ? p.topk_group : p.topk_group * span, lane);
    bool kept = some && mine >= kth;
    const float err = scored ? group_margin(e0, a1, a2, mine, p.group_top) : 0.0f;
    // what the lowest kept score may be at least, and the highest of the others at most
    const float least_kept = -team_max<L>(kept ? err - mine : -INFINITY);
    const float most_other = team_max<L>(some && !kept ? mine + err : -INFINITY);
    // (every lane votes, whatever its team found: no vote behind a condition that teams may differ in)
    const int lanes_kept = __popc(team_ballot<L>(kept, lane));
    const bool slow = (most_other > -INFINITY && most_other >= least_kept) || lanes_kept > p.topk_group * span;
    if (__any_sync(0xffffffffu, slow)) {
      // a close call, or equal scores: rank the groups one by one
      const float gerr = scored && some ? group_error(e0, a1, a2, p.group_top) : 0.0f;
      int above = 0, sure_above = 0, maybe_above = 0;
      for (int j = 0; j < p.n_group; ++j) {
        const float o = __shfl_sync(0xffffffffu, mine, j * span, L);
        const float both = gerr + __shfl_sync(0xffffffffu, gerr, j * span, L);
        above += o > mine || (o == mine && j < at);
        sure_above += o - mine > both;
        maybe_above += j != at && mine - o <= both;
      }
      if (slow) kept = some && above < p.topk_group;
      // is a kept group too close to one that is not?
      unsure = team_any<L>(scored && some && maybe_above >= p.topk_group && sure_above < p.topk_group, lane);
      if (__any_sync(0xffffffffu, unsure) && whole) {
        // The groups' scores in 64 bits, from the one or two experts that each
        // is made of, if 32 bits tell those from the group's others.
        const float least = p.group_top == 1 || a2 == -INFINITY ? a1 : a2, lowest = least - gate_near(e0, least);
        int n = 0, e1 = -1, e2 = -1;
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (c[i] >= lowest && c[i] > -INFINITY) {
            e2 = e1;
            e1 = first + i;
            ++n;
          }
        for (int o = 1; o < span; o <<= 1) {
          const int f1 = __shfl_xor_sync(0xffffffffu, e1, o), f2 = __shfl_xor_sync(0xffffffffu, e2, o);
          n += __shfl_xor_sync(0xffffffffu, n, o);
          // (right when there are two of them in all, and not used otherwise)
          const int x1 = e1 >= 0 ? e1 : f1, x2 = e1 >= 0 ? (e2 >= 0 ? e2 : f1) : f2;
          e1 = x1;
          e2 = x2;
        }
        const int want = p.group_top == 1 || a2 == -INFINITY ? 1 : 2;
        const bool told = !team_any<L>(some && n != want, lane);
        const double total64 = SIGMOID ? 1.0 : gate_total64<LT, L>(row, p.E, tl, top);
        // of two experts, one by the odd lanes and one by the even ones
        const bool use = some && unsure && told;
        const bool second = want == 2 && span > 1 && (tl & 1);
        double exact = use ? gate_score64(p, row, second ? max(e1, e2) : want == 2 ? min(e1, e2) : e1, top, total64)
                           : -INFINITY;
        __syncwarp();
        const double other = __shfl_xor_sync(0xffffffffu, exact, 1);
        if (use && want == 2) exact += span > 1 ? other : gate_score64(p, row, max(e1, e2), top, total64);
        __syncwarp();
        above = 0;
        for (int j = 0; j < p.n_group; ++j) {
          const double o = __shfl_sync(0xffffffffu, exact, j * span, L);
          above += o > exact || (o == exact && j < at);
        }
        if (unsure && told) {
          kept = some && above < p.topk_group;
          unsure = false;
        }
      }
    }
    if (!BIAS && sums) {  // the groups went by scores, their experts go by the logits
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] = c[i] == -INFINITY ? c[i] : l[i];
    }
    if (p.deal) {
      // Few lanes have experts left: these, in order, are dealt out over all lanes,
      // so that the best of the lanes tell more about the best of the row.
      const uint32_t heads = team_ballot<L>(kept && (tl & (span - 1)) == 0, lane);
      const int to = __popc(heads & ((1u << (at << p.span_log2)) - 1u)) * p.gsize + (first - at * p.gsize);
      if (kept) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (i < live) list[to + i] = make_float2(c[i], __int_as_float(first + i));
      }
      const int left = __popc(heads) * p.gsize;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float2 x = tl + L * i < left ? list[tl + L * i] : make_float2(-INFINITY, 0.0f);
        c[i] = x.x;
        expert[i] = __float_as_int(x.y);
      }
      __syncwarp();
    } else if (whole) {
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] = kept ? c[i] : -INFINITY;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (!__shfl_sync(0xffffffffu, kept, min(L - 1, (tl * V + i) / p.gsize), L)) c[i] = -INFINITY;
    }
  }

  int mine_id = -1;
  float best = c[0];
#pragma unroll
  for (int i = 1; i < V; ++i) best = fmaxf(best, c[i]);
  if (tl == 0) *count = 0;
  const float kth = team_kth<L>(best, p.topk, lane);
  // (-FLT_MAX where fewer lanes than topk have an expert: every one is in question)
  const float bound = kth == -INFINITY ? -FLT_MAX : BIAS ? kth - gate_near(e0, kth) : kth;
  int n = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) count_from(n, c[i], bound);
  __syncwarp();
  uint32_t to = smem_u32(list) + 8 * (n > 0 ? atomicAdd(count, n) : 0);
#pragma unroll
  for (int i = 0; i < V; ++i) list_from(to, c[i], expert[i], bound);
  __syncwarp();
  const int all = *count;
  const int m = min(all, kGateList);
  const float2 none = make_float2(-INFINITY, __int_as_float(-1));
  float2 x[kOwn];
  int rank[kOwn];
  if constexpr (L == 32) {
    // the place of candidate `lane`, or of lane % 16 from half of the others where no more than 16 are
    const bool two = m <= 16;
    const int own = two ? tl & 15 : tl;
    x[0] = own < m ? list[own] : none;
    rank[0] = 0;
    for (int j = two ? tl >> 4 : 0; j < m; j += two ? 2 : 1) {
      const float2 o = list[j];
      rank[0] += o.x > x[0].x || (o.x == x[0].x && __float_as_int(o.y) < __float_as_int(x[0].y));
    }
    if (two) rank[0] += __shfl_xor_sync(0xffffffffu, rank[0], 16);
  } else {
    // both teams count to the longer list, the shorter one filled up
    const int longest = __reduce_max_sync(0xffffffffu, m);
#pragma unroll
    for (int r = 0; r < kOwn; ++r) {
      const int own = tl + L * r;
      x[r] = own < m ? list[own] : none;
      if (own >= m && own < longest) list[own] = none;
      rank[r] = 0;
    }
    __syncwarp();
#pragma unroll
    for (int r = 0; r < kOwn; ++r)
      if (r == 0 || longest > L * r)
        for (int j = 0; j < longest; ++j) {
          const float2 o = list[j];
          rank[r] += o.x > x[r].x || (o.x == x[r].x && __float_as_int(o.y) < __float_as_int(x[r].y));
        }
  }
  __syncwarp();
#pragma unroll
  for (int r = 0; r < kOwn; ++r)
    if (tl + L * r < m) list[rank[r]] = x[r];
  __syncwarp();
  const float2 y = tl < m ? list[tl] : none;
  mine_id = tl < p.topk ? __float_as_int(y.y) : -1;
  if (BIAS) {
    // neighbours in the order, down to the first behind the chosen ones
    const bool near_one = tl < p.topk && tl + 1 < m && y.x - list[tl + 1].x <= gate_near(e0, y.x);
    if (__any_sync(0xffffffffu, near_one)) {
      const bool found_near = team_any<L>(near_one, lane);
      const bool redo = found_near && all <= kGateList;
      const double total64 = SIGMOID ? 1.0 : gate_total64<LT, L>(row, p.E, tl, top);
      double z[kOwn];
#pragma unroll
      for (int r = 0; r < kOwn; ++r) {
        z[r] = redo && tl + L * r < m ? gate_score64(p, row, __float_as_int(x[r].y), top, total64) : -INFINITY;
        rank[r] = 0;
      }
      __syncwarp();
      const int longest = __reduce_max_sync(0xffffffffu, m);
#pragma unroll
      for (int q = 0; q < kOwn; ++q)
        for (int j = 0; j < min(L, longest - L * q); ++j) {
          const double o = __shfl_sync(0xffffffffu, z[q], j, L);
          const int oe = __shfl_sync(0xffffffffu, __float_as_int(x[q].y), j, L);
#pragma unroll
          for (int r = 0; r < kOwn; ++r) rank[r] += o > z[r] || (o == z[r] && oe < __float_as_int(x[r].y));
        }
#pragma unroll
      for (int r = 0; r < kOwn; ++r)
        if (redo && tl + L * r < m) list[rank[r]] = x[r];
      __syncwarp();
      if (redo && tl < min(m, p.topk)) mine_id = __float_as_int(list[tl].y);
    }
  }
  if (__any_sync(0xffffffffu, all > kGateList)) {
    // more than 32 in question: the best of the team, topk times; one more
    // shows whether the last place was a close one
    const int rounds = BIAS ? p.topk + 1 : p.topk;
    float before = INFINITY;
    int before_e = -1;
    bool close = false;
    int found_id = -1;
    for (int j = 0; j < rounds; ++j) {
      float lead = c[0];
#pragma unroll
      for (int i = 1; i < V; ++i) lead = fmaxf(lead, c[i]);
      const float next = team_max<L>(lead);
      // of equal ones the expert with the lowest index (a lane's experts are in order)
      int e = 0x7FFFFFFF;
#pragma unroll
      for (int i = V - 1; i >= 0; --i)
        if (next > -INFINITY && c[i] == next) e = expert[i];
      int lowest = e;
#pragma unroll
      for (int o = L / 2; o >= 1; o >>= 1) lowest = min(lowest, __shfl_xor_sync(0xffffffffu, lowest, o));
      const bool found = lowest != 0x7FFFFFFF;
      if (found && e == lowest) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (expert[i] == e) c[i] = -INFINITY;
      }
      e = lowest;
      // equal logits with equal biases tie whatever the precision
      if (BIAS && found && before - next <= gate_near(e0, before) &&
          !(gate_at(row, e) == gate_at(row, before_e) && __ldg(p.bias + e) == __ldg(p.bias + before_e)))
        close = true;
      before = next;
      before_e = e;
      if (tl == j && j < p.topk && found) found_id = e;
    }
    if (all > kGateList) {
      mine_id = found_id;
      unsure |= close;
    }
  }
  if (__any_sync(0xffffffffu, unsure)) {
    const int id = gate_choose64<LT, L, V>(p, row, tl, top);
    if (unsure) mine_id = id;
  }

  const bool has = mine_id >= 0;
  const float s = has ? gate_at(row, mine_id) : -INFINITY;  // the chosen expert's logit
  float w;
  if (p.renorm) {
    // s_j / sum s, from e^(s - hi) or e^(min(s, 0) - min(hi, 0)) / (1 + e^-|s|): ratios to the
    // largest, so no share that is itself a normal number underflows on the way
    const float hi = team_max<L>(s);
    float v = SIGMOID ? __fdiv_rn(expf(fminf(s, 0.0f) - fminf(hi, 0.0f)), 1.0f + expf(-fabsf(s))) : expf(s - hi);
    v = has ? v : 0.0f;
    w = __fdiv_rn(v, team_sum<L>(v));
  } else if (SIGMOID) {
    w = __fdiv_rn(expf(fminf(s, 0.0f)), 1.0f + expf(-fabsf(s)));
  } else {
    w = __fdiv_rn(expf(s - top), total);
  }
  if (mine_is && tl < p.topk) {
    p.ids[static_cast<size_t>(t) * p.topk + tl] = mine_id;
    p.weights[static_cast<size_t>(t) * p.topk + tl] = has ? p.scale * w : 0.0f;
  }
}

// ---------------------------------------------------------------- backward

// One warp a token: lane j holds slot j, the row is put together in shared
// memory and written once.  16384 x 256 FP32, topk 8: 6.8 us (2.7 TB/s, the rows
// coming from L2), dense softmax 7.7 us; bound by the latency of the gathered
// logits and of the sums, which one row's warp cannot overlap.
// VEC: E % V == 0, whole runs of V experts a lane; else one expert after another.
template <typename LT, int V, bool VEC>
__global__ void __launch_bounds__(32 * kGateWarps) moe_gate_backward_kernel(const GateBackwardArgs p) {
  __shared__ __align__(16) float rows[kGateWarps][32 * V];
  __shared__ int owner[kGateWarps][32 * V];
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kGateWarps + (threadIdx.x >> 5);
  if (t >= p.T) return;
  float* acc = rows[threadIdx.x >> 5];
  int* slot = owner[threadIdx.x >> 5];
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
    // s = e^min(x,0) / (1 + e^-|x|) and 1 - s = e^-max(x,0) / (1 + e^-|x|)
    const float tail = expf(-fabsf(x));
    const float inv = __fdiv_rn(1.0f, 1.0f + tail);
    const float rest = (x < 0.0f ? 1.0f : tail) * inv;
    if (p.renorm) {
      float m = team_max<32>(x);
      if (m == -INFINITY) m = 0.0f;
      // s / sum s as in the forward pass
      float r = p.sigmoid ? expf(fminf(x, 0.0f) - fminf(m, 0.0f)) * inv : expf(x - m);
      r = has ? r : 0.0f;
      const float sum = team_sum<32>(r);
      r = sum > 0.0f ? __fdiv_rn(r, sum) : 0.0f;
      const float mean = team_sum<32>(r * g);
      v = p.scale * r * (p.sigmoid ? rest : 1.0f) * (g - mean);
    } else {
      v = p.scale * ((x < 0.0f ? tail : 1.0f) * inv) * rest * g;
    }
  }
  const int first = VEC ? lane * V : lane;
  constexpr int step = VEC ? 1 : 32;
  const int live = VEC ? (first < p.E ? V : 0) : max(0, (p.E - lane + 31) / 32);
  float o[V];
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = 0.0f;
  gate_store_row<V>(acc, lane * V, 1, V, true, o);
  __syncwarp();
  if (has) {
    acc[id] = v;
    slot[id] = lane;
  }
  __syncwarp();
  if (__any_sync(0xffffffffu, has && slot[id] != lane)) {
    // an expert named twice in a row takes both slots' share, in slot order
    if (has) acc[id] = 0.0f;
    __syncwarp();
    for (int j = 0; j < p.topk; ++j) {
      if (lane == j && has) acc[id] += v;
      __syncwarp();
    }
  }
  if constexpr (V >= 4 && VEC) {
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      const float4 q = reinterpret_cast<const float4*>(acc + first)[i];
      o[4 * i] = q.x, o[4 * i + 1] = q.y, o[4 * i + 2] = q.z, o[4 * i + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = acc[first + i * step];
  }
  if (dense && __any_sync(0xffffffffu, has)) {
    float l[V];
    gate_load_row<V>(row, first, step, live, VEC, -INFINITY, l);
    float m = l[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = fmaxf(m, l[i]);
    m = team_max<32>(m);
    if (m == -INFINITY) m = 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      l[i] = expf(l[i] - m);
      sum += l[i];
    }
    sum = team_sum<32>(sum);
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    float mean = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      l[i] *= inv;
      mean += l[i] * o[i];
    }
    mean = team_sum<32>(mean);
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = p.scale * l[i] * (o[i] - mean);
  }
  gate_store_row<V>(out, first, step, live, VEC, o);
}

}  // namespace dg
