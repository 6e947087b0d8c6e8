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
  int gsize;            // experts of a group
  int span_log2;        // a group is 2^span_log2 whole lanes, or -1
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

// Largest of the warp's values (no NaN among them).
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
template <typename R>
__device__ __forceinline__ R warp_sum(R x) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// max(a, |b|), a NaN's place taken by NaN.
__device__ __forceinline__ float max_abs_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
  return r;
}

// 2^x and 1/x by the approximate instructions, each within one unit in the
// last place of 2^-22 or better, subnormals taken as zero.
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
    const int gsize = p.gsize;
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

// Sum of exp(l - top) over the row in 64 bits (every lane returns it).
template <typename LT, int V>
__device__ __noinline__ double gate_total64(const LT* row, int E, int lane, float top) {
  double sum = 0.0;
  for (int i = 0; i < V; ++i) {
    const int e = lane + 32 * i;
    if (e < E) sum += exp(static_cast<double>(gate_at(row, e)) - static_cast<double>(top));
  }
  return warp_sum(sum);
}

// c of expert e in 64 bits; total64 from gate_total64 (softmax only).
template <typename LT>
__device__ __noinline__ double gate_score64(const GateArgs& p, const LT* row, int e, float top, double total64) {
  const double x = gate_at(row, e);
  const double s = p.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - static_cast<double>(top)) / total64;
  return p.bias ? s + static_cast<double>(__ldg(p.bias + e)) : s;
}

// One warp a token.
//
// Error of a 32-bit score (u = 2^-24).  ex2.approx and rcp.approx are within
// 2^-22 = 4u relative; the argument x log2(e) of ex2 is off by 2u |x| log2(e)
// (the constant's rounding and the product's), which is 2u |x| relative in the
// exponential.
//   sigmoid  s(1-s)(4 + 2|l|) u <= (1 + 0.45) u, the sum u, the quotient 4u:
//            below 7u.
//   softmax  p |x| 2u <= 0.74u and 4u p from the exponential; from the sum (at
//            most 1024 terms, in 64 bits (2 + 2 * 6.94) u of their own and 37 u
//            of additions) and the quotient 60u p: <= p 2^-17 + u.
// c = s + b adds |c| u <= (1 + B) u, B the largest |b|.  Two values closer than
// both errors together (`near`) are not told apart; a sum of two has both
// terms' errors and its own rounding, 2 (1 + B) u.
//
// The choice.  The topk-th largest of the lanes' best values is a lower bound
// of the topk-th best value of the row, since so many values reach it, and few
// values do (for 256 experts, topk 8: about ten).  Those (and the ones closer
// below it than `near`) are put together in shared memory, one a lane, and each
// lane counts the ones before its own.  That takes the place of topk rounds of
// finding and removing the best (which serve the rows with more than 32).
template <typename LT, int V, bool SIGMOID, bool BIAS>
__global__ void __launch_bounds__(32 * kGateWarps) moe_gate_kernel(const __grid_constant__ GateArgs p) {
  __shared__ float2 cand[kGateWarps][32 * V];  // value, expert
  __shared__ int count[kGateWarps];
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  float2* list = cand[warp];
  const int t = blockIdx.x * kGateWarps + warp;
  if (t >= p.T) return;
  const LT* row = static_cast<const LT*>(p.logits) + static_cast<size_t>(t) * p.E;

  const bool sums = p.n_group > 1 && p.group_top > 1;
  const bool scored = BIAS || sums;
  const bool full = p.E == 32 * V;  // every lane holds V experts
  const int live = full ? V : min(V, max(0, p.E - lane * V));
  float l[V], c[V];
  gate_load_row<V>(row, p.E, lane, -FLT_MAX, l);
  if (BIAS) gate_load_row<V>(p.bias, p.E, lane, 0.0f, c);
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
    top = warp_max(m);
    if (top == -INFINITY) top = 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) sum += i < live ? expf(l[i] - top) : 0.0f;
    total = warp_sum(sum);
  }
  float near = 0.0f;
  if (scored) {
    const float inv = SIGMOID ? 1.0f : fast_rcp(total);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float s = SIGMOID ? fast_rcp(1.0f + fast_exp2(-kLog2e * l[i])) : fast_exp2(kLog2e * (l[i] - top)) * inv;
      c[i] = BIAS ? s + c[i] : s;
    }
    near = 0x1p-20f + (SIGMOID ? 0.0f : 0x1p-16f * inv);
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
        const float b = i < live ? __ldg(p.bias + lane * V + i) : 0.0f;
        bad |= !(b < INFINITY);
        if (b == -INFINITY) c[i] = -INFINITY;
        largest = fmaxf(i == 0 ? 0.0f : largest, b > -INFINITY ? fabsf(b) : 0.0f);
      }
    }
    if (__any_sync(0xffffffffu, bad)) {
      // NaN or +inf among the logits or the bias: the token is not routed
      if (lane == 0) atomicOr(&g_dg_error, 0x20);
      if (lane < p.topk) {
        p.ids[static_cast<size_t>(t) * p.topk + lane] = -1;
        p.weights[static_cast<size_t>(t) * p.topk + lane] = 0.0f;
      }
      return;
    }
  }
  if (BIAS) {
    largest = warp_max(largest);
    near += 0x1p-23f * (1.0f + largest);
  }
  if (!full) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i >= live) c[i] = -INFINITY;
  }

  bool unsure = false;  // the row needs the choice in 64 bits (all lanes agree)
  if (p.n_group > 1) {
    const bool whole = p.span_log2 >= 0;
    const int span = whole ? 1 << p.span_log2 : 1;  // lanes that hold the same group
    float mine;
    float a1 = c[0], a2 = -INFINITY;
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
      mine = group_score(a1, a2, p.group_top);
    } else {
      mine = group_scores_any<float, V>(c, lane, p.n_group, p.gsize, p.group_top);
    }
    // lanes behind the last group have -inf, as groups without an expert to choose
    const float gnear = scored ? 2.0f * near + 0x1p-21f * (1.0f + largest) : 0.0f;
    // the topk_group-th best score (equal ones once), and the best below it
    float rest = mine, kth = -INFINITY;
    for (int j = 0; j < p.topk_group; ++j) {
      kth = warp_max(rest);
      rest = rest == kth ? -INFINITY : rest;
    }
    bool kept = mine >= kth && mine > -INFINITY;
    const bool close = scored && kth - warp_max(rest) <= gnear;  // (-inf - -inf is NaN: not close)
    if (close || __popc(__ballot_sync(0xffffffffu, kept)) > p.topk_group * span) {
      // a close call or equal scores: rank the groups one by one
      const int at = whole ? lane >> p.span_log2 : lane;
      const bool some = mine > -INFINITY;
      int above = 0, sure_above = 0, maybe_above = 0;
      for (int j = 0; j < p.n_group; ++j) {
        const float o = __shfl_sync(0xffffffffu, mine, j * span);
        above += o > mine || (o == mine && j < at);
        sure_above += o > mine + gnear;
        maybe_above += j != at && o >= mine - gnear;
      }
      kept = some && above < p.topk_group;
      unsure = scored && __any_sync(0xffffffffu, some && maybe_above >= p.topk_group && sure_above < p.topk_group);
      if (unsure && whole) {
        // The groups' scores in 64 bits, from the one or two experts that each
        // is made of, if 32 bits tell those from the group's others.
        const float lowest = (p.group_top == 1 || a2 == -INFINITY ? a1 : a2) - near;
        int n = 0, e1 = -1, e2 = -1;
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (c[i] >= lowest && c[i] > -INFINITY) {
            e2 = e1;
            e1 = lane * V + i;
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
        if (__all_sync(0xffffffffu, !some || n == want)) {
          const double total64 = SIGMOID ? 1.0 : gate_total64<LT, V>(row, p.E, lane, top);
          double exact = -INFINITY;
          if (some) {
            exact = gate_score64(p, row, e1, top, total64);
            if (want == 2) exact += gate_score64(p, row, e2, top, total64);
          }
          __syncwarp();
          above = 0;
          for (int j = 0; j < p.n_group; ++j) {
            const double o = __shfl_sync(0xffffffffu, exact, j * span);
            above += o > exact || (o == exact && j < at);
          }
          kept = some && above < p.topk_group;
          unsure = false;
        }
      }
    }
    if (whole) {
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] = kept ? c[i] : -INFINITY;
    } else {
      const uint32_t all_kept = __ballot_sync(0xffffffffu, kept);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (!((all_kept >> min(31, (lane * V + i) / p.gsize)) & 1)) c[i] = -INFINITY;
    }
    if (!BIAS && sums) {  // the groups went by scores, their experts go by the logits
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] = c[i] == -INFINITY ? c[i] : l[i];
    }
  }

  int mine_id = -1;
  if (!unsure) {
    float best = c[0];
#pragma unroll
    for (int i = 1; i < V; ++i) best = fmaxf(best, c[i]);
    if (lane == 0) count[warp] = 0;
    float kth = -INFINITY;
    for (int j = 0; j < p.topk; ++j) {
      kth = warp_max(best);
      best = best == kth ? -INFINITY : best;
    }
    // (-FLT_MAX where fewer lanes than topk have an expert: every one is in question)
    const float bound = kth == -INFINITY ? -FLT_MAX : BIAS ? kth - near : kth;
    int n = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) n += c[i] >= bound;
    __syncwarp();
    int pos = n > 0 ? atomicAdd(&count[warp], n) : 0;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (c[i] >= bound) list[pos++] = make_float2(c[i], __int_as_float(lane * V + i));
    __syncwarp();
    const int m = count[warp];
    if (m <= 32) {
      // the place of candidate `lane` (of lane % 16, from half of the others, where no more than 16 are)
      const bool two = m <= 16;
      const int own = two ? lane & 15 : lane;
      const float2 x = own < m ? list[own] : make_float2(-INFINITY, 0.0f);
      int rank = 0;
      for (int j = two ? lane >> 4 : 0; j < m; j += two ? 2 : 1) {
        const float2 o = list[j];
        rank += o.x > x.x || (o.x == x.x && __float_as_int(o.y) < __float_as_int(x.y));
      }
      __syncwarp();
      if (two) rank += __shfl_xor_sync(0xffffffffu, rank, 16);
      if (lane < m) list[rank] = x;
      __syncwarp();
      float2 y = lane < m ? list[lane] : make_float2(-INFINITY, __int_as_float(-1));
      if (BIAS) {
        // neighbours in the order, down to the first behind the chosen ones
        const float next = __shfl_down_sync(0xffffffffu, y.x, 1);
        if (__any_sync(0xffffffffu, lane < p.topk && lane + 1 < m && y.x - next <= near)) {
          const int e = __float_as_int(y.y);
          const double total64 = SIGMOID ? 1.0 : gate_total64<LT, V>(row, p.E, lane, top);
          const double z = lane < m ? gate_score64(p, row, e, top, total64) : -INFINITY;
          __syncwarp();
          rank = 0;
          for (int j = 0; j < m; ++j) {
            const double o = __shfl_sync(0xffffffffu, z, j);
            const int oe = __shfl_sync(0xffffffffu, e, j);
            rank += o > z || (o == z && oe < e);
          }
          if (lane < m) list[rank] = y;
          __syncwarp();
          if (lane < m) y = list[lane];
        }
      }
      mine_id = lane < p.topk ? __float_as_int(y.y) : -1;
    } else {
      // more than 32 in question: the best of the warp, topk times; one more
      // shows whether the last place was a close one
      const int rounds = BIAS ? p.topk + 1 : p.topk;
      float before = INFINITY;
      for (int j = 0; j < rounds; ++j) {
        float lead = c[0];
#pragma unroll
        for (int i = 1; i < V; ++i) lead = fmaxf(lead, c[i]);
        const float all = warp_max(lead);
        if (all == -INFINITY) break;
        if (BIAS && before - all <= near) {
          unsure = true;
          break;
        }
        before = all;
        const int src = __ffs(__ballot_sync(0xffffffffu, lead == all)) - 1;
        int at = 0;
        if (lane == src) {
          bool found = false;
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (!found && c[i] == all) {
              found = true;
              c[i] = -INFINITY;
              at = lane * V + i;
            }
        }
        at = __shfl_sync(0xffffffffu, at, src);
        if (lane == j && j < p.topk) mine_id = at;
      }
    }
  }
  if (unsure) mine_id = gate_choose64<LT, V>(p, row, lane);

  const bool has = mine_id >= 0;
  const float x = has ? gate_at(row, mine_id) : -INFINITY;
  float w;
  if (p.renorm) {
    // s_j / sum s; from the ratios to the largest, where the scores might underflow
    const float m = warp_max(x);
    float v;
    if (!SIGMOID) v = expf(x - m);
    else if (m > -60.0f) v = __fdiv_rn(1.0f, 1.0f + expf(-x));
    else v = __fdiv_rn(expf(x - m), 1.0f + expf(x));
    v = has ? v : 0.0f;
    w = __fdiv_rn(v, warp_sum(v));
  } else if (SIGMOID) {
    w = __fdiv_rn(expf(fminf(x, 0.0f)), 1.0f + expf(-fabsf(x)));
  } else {
    w = __fdiv_rn(expf(x - top), total);
  }
  if (lane < p.topk) {
    p.ids[static_cast<size_t>(t) * p.topk + lane] = mine_id;
    p.weights[static_cast<size_t>(t) * p.topk + lane] = has ? p.scale * w : 0.0f;
  }
}

// ---------------------------------------------------------------- backward

// One warp a token: lane j holds slot j, the row is put together in shared
// memory and written once.
template <typename LT, int V>
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
      float m = warp_max(x);
      if (m == -INFINITY) m = 0.0f;
      // s / sum s as in the forward pass
      float r = p.sigmoid ? expf(fminf(x, 0.0f) - fminf(m, 0.0f)) * inv : expf(x - m);
      r = has ? r : 0.0f;
      const float sum = warp_sum(r);
      r = sum > 0.0f ? __fdiv_rn(r, sum) : 0.0f;
      const float mean = warp_sum(r * g);
      v = p.scale * r * (p.sigmoid ? rest : 1.0f) * (g - mean);
    } else {
      v = p.scale * ((x < 0.0f ? tail : 1.0f) * inv) * rest * g;
    }
  }
  float o[V];
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = 0.0f;
  gate_store_row<V>(acc, 32 * V, lane, o);
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
  if constexpr (V >= 4) {
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      const float4 q = reinterpret_cast<const float4*>(acc + lane * V)[i];
      o[4 * i] = q.x, o[4 * i + 1] = q.y, o[4 * i + 2] = q.z, o[4 * i + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = acc[lane * V + i];
  }
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
