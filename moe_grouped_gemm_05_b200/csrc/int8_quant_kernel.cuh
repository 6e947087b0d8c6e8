// Per-token int8 quantisation: x[M][K] (BF16 or FP32) -> codes q[M][K] and one
// FP32 scale a row, and the same for routed tokens, written to the rows of
// their experts in the contiguous layout.
//
//   amax = max|x|;  scale = fp32(amax / 127), at least 2^-126 (1 for a row of zeros)
//   q = the integer nearest to x * fp32(127 / amax), ties to even
//
// The product is not rounded before the integer is taken: one fused
// multiply-add onto 1.5 * 2^23, whose last place is 1, rounds it once, and the
// code is the low byte of the sum.  So the codes are those of the definition
// evaluated in 64 bits.  A row that holds a NaN or an infinity gets scale NaN
// and codes 0, which makes its products NaN.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "ptx.cuh"
#include "quant_kernel.cuh"

namespace dg {

// Largest |x| of a unit of 16 elements as the bits of a float; a NaN's bits are
// above infinity's, so it wins.
template <typename T>
struct QuantUnit;

template <>
struct QuantUnit<__nv_bfloat16> {
  uint32_t u[8];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(p)), b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
    u[0] = a.x, u[1] = a.y, u[2] = a.z, u[3] = a.w;
    u[4] = b.x, u[5] = b.y, u[6] = b.z, u[7] = b.w;
  }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, u[i] & 0x7FFF7FFFu);
    return max(m << 16, m & 0xFFFF0000u);
  }
  __device__ __forceinline__ float value(int i) const {
    return __uint_as_float(i & 1 ? u[i >> 1] & 0xFFFF0000u : u[i >> 1] << 16);
  }
};

template <>
struct QuantUnit<float> {
  uint32_t u[16];
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 a = __ldg(reinterpret_cast<const uint4*>(p) + i);
      u[4 * i] = a.x, u[4 * i + 1] = a.y, u[4 * i + 2] = a.z, u[4 * i + 3] = a.w;
    }
  }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, u[i] & 0x7FFFFFFFu);
    return m;
  }
  __device__ __forceinline__ float value(int i) const { return __uint_as_float(u[i]); }
};

constexpr float kInt8Least = 0x1p-126f;  // the smallest scale

// Scale of a row with largest |x| amax, and its inverse (0 for a row that is not finite).
__device__ __forceinline__ void int8_scale(uint32_t amax_bits, float& scale, float& inverse) {
  const float amax = __uint_as_float(amax_bits);
  if (amax_bits == 0u) {
    scale = inverse = 1.0f;
  } else if (amax_bits >= 0x7F800000u) {
    scale = __uint_as_float(0x7FC00000u);
    inverse = 0.0f;
  } else if (amax < 127.0f * kInt8Least) {
    scale = kInt8Least;
    inverse = 1.0f / kInt8Least;
  } else {
    scale = __fdiv_rn(amax, 127.0f);
    inverse = __fdiv_rn(127.0f, amax);
  }
}

template <typename T>
__device__ __forceinline__ uint4 int8_codes(const QuantUnit<T>& v, float inverse) {
  if (inverse == 0.0f) return make_uint4(0, 0, 0, 0);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t n[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) n[j] = __float_as_uint(fmaf(v.value(4 * i + j), inverse, 12582912.0f));
    w[i] = __byte_perm(__byte_perm(n[0], n[1], 0x0040), __byte_perm(n[2], n[3], 0x0040), 0x5410);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

struct QuantArgs {
  const void* x;
  int M, K;
  uint8_t* q;             // [M][K], or the permuted codes [M_cap][K]
  float* scale;           // [M], or the permuted scales [M_cap]
  // permuted form only
  const int32_t* ids;     // [M][topk]
  const int32_t* row_of;  // [M][topk]
  int topk;
  int32_t* m_indices;
  int32_t* src_of;
  // the permuted form of few slots: it routes as well
  int G, M_cap;
  int32_t* row_of_out;
};

// One row a team of W warps (W = blockDim.y warps; blockDim.z teams of one warp
// when W == 1), each thread U units of 16 elements.  U == 0: a row of any
// length, read twice.
// PERM: every routed slot of the token gets the row's codes.
template <typename T, int U, bool PERM>
__global__ void __launch_bounds__(U == 4 && sizeof(T) == 4 ? 512 : 1024) quantize_int8_kernel(const QuantArgs p) {
  __shared__ uint32_t part[32];
  const int lane = threadIdx.x;
  const int W = blockDim.y;
  const int warp = threadIdx.y;
  const long long row = static_cast<long long>(blockIdx.x) * blockDim.z + threadIdx.z;
  const int units = p.K / 16;
  grid_dep_wait();
  grid_dep_launch();
  if (row >= p.M) return;  // whole warps: a block of several teams has one warp a team
  const T* x = static_cast<const T*>(p.x) + static_cast<size_t>(row) * p.K;
  const int step = 32 * W;
  const int u0 = 32 * warp + lane;
  constexpr int kU = U == 0 ? 1 : U;
  QuantUnit<T> v[kU] = {};
  uint32_t amax = 0;
  if constexpr (U == 0) {
    for (int u = u0; u < units; u += step) {
      v[0].load(x + 16 * static_cast<size_t>(u));
      amax = max(amax, v[0].top());
    }
  } else {
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (u0 + i * step < units) v[i].load(x + 16 * (u0 + i * step));
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (u0 + i * step < units) amax = max(amax, v[i].top());
  }
  // lane s holds the destination of slot s
  const int slot_row = PERM && lane < p.topk ? __ldg(p.row_of + row * p.topk + lane) : -1;
  amax = __reduce_max_sync(0xffffffffu, amax);
  if (W > 1) {
    if (lane == 0) part[warp] = amax;
    __syncthreads();
    amax = __reduce_max_sync(0xffffffffu, lane < W ? part[lane] : 0u);
  }
  float scale, inverse;
  int8_scale(amax, scale, inverse);
  if constexpr (!PERM) {
    if (warp == 0 && lane == 0) p.scale[row] = scale;
  } else if (warp == 0) {
    for (int s = lane; s < p.topk; s += 32) {
      const int r = s < 32 ? slot_row : __ldg(p.row_of + row * p.topk + s);
      if (r < 0) continue;
      p.scale[r] = scale;
      p.m_indices[r] = __ldg(p.ids + row * p.topk + s);
      p.src_of[r] = static_cast<int32_t>(row);
    }
  }
  if constexpr (U == 0) {
    for (int u = u0; u - lane < units; u += step) {
      const bool in = u < units;
      if (in) v[0].load(x + 16 * static_cast<size_t>(u));
      const uint4 c = int8_codes(v[0], inverse);
      if constexpr (PERM) {
        for (int s = 0; s < p.topk; ++s) {
          const int r = s < 32 ? __shfl_sync(0xffffffffu, slot_row, s) : __ldg(p.row_of + row * p.topk + s);
          if (in && r >= 0) reinterpret_cast<uint4*>(p.q + static_cast<size_t>(r) * p.K)[u] = c;
        }
      } else if (in) {
        reinterpret_cast<uint4*>(p.q + static_cast<size_t>(row) * p.K)[u] = c;
      }
    }
  } else {
    uint4 c[U];
#pragma unroll
    for (int i = 0; i < U; ++i) c[i] = int8_codes(v[i], inverse);
    for (int s = 0; s < (PERM ? p.topk : 1); ++s) {
      long long r = row;
      if constexpr (PERM) r = s < 32 ? __shfl_sync(0xffffffffu, slot_row, s) : __ldg(p.row_of + row * p.topk + s);
      if (r < 0) continue;
      uint4* to = reinterpret_cast<uint4*>(p.q + static_cast<size_t>(r) * p.K);
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (u0 + i * step < units) to[u0 + i * step] = c[i];
    }
  }
}

// Routing, quantisation and scattering of few slots (a decode batch) in one
// launch: 64 tokens, top-8 of 256, K = 2048 3.4 us against 10.4.  The routing
// kernel's cluster takes 7 to 10 us whatever the batch (its counting passes, two
// cluster barriers, a table of 32 counts an expert);
// here every block counts the experts of all slots and scans the segments for
// itself, and ranks only its own token's slots among the earlier ones.  Blocks
// behind the last token only mark padding rows.  Its time grows with slots times
// tokens; measured for K = 2048, this form against the cluster's:
//   slots   top-2 of 8      top-3 of 64     top-8 of 256
//    1024   4.4 /  7.6 us    4.0 /  8.5 us   3.3 / 10.5 us
//    2048   7.1 /  8.3       5.8 /  9.8      4.3 / 10.9
//    4096  16.4 /  9.3      13.0 / 11.3      8.6 / 12.3
// (K = 7168 and FP32 rows alike), so it takes up to 2048, where it wins for each.
constexpr int kFewSlots = 2048;
constexpr int kFewThreads = 256;

template <typename T, int U>
__global__ void __launch_bounds__(kFewThreads) quantize_permute_few_kernel(const QuantArgs p) {
  __shared__ int id[kFewSlots];
  __shared__ int count[kMoeMaxExperts];
  __shared__ int segment[kMoeMaxExperts];
  __shared__ int slot_row[kFewSlots];
  __shared__ int part[kFewThreads / 32];
  __shared__ uint32_t top[kFewThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t = blockIdx.x;
  const int n = p.M * p.topk;
  const int units = p.K / 16;
  const bool has = t < p.M;
  grid_dep_wait();
  grid_dep_launch();
  // this token's values are on their way while the experts are counted
  const T* x = static_cast<const T*>(p.x) + static_cast<size_t>(has ? t : 0) * p.K;
  constexpr int kU = U == 0 ? 1 : U;
  QuantUnit<T> v[kU] = {};
  if constexpr (U > 0) {
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (has && tid + i * kFewThreads < units) v[i].load(x + 16 * (tid + i * kFewThreads));
  }
  for (int e = tid; e < p.G; e += kFewThreads) count[e] = 0;
  __syncthreads();
  bool bad = false;
  for (int i = tid; i < n; i += kFewThreads) {
    const int e = __ldg(p.ids + i);
    const bool valid = e >= 0 && e < p.G;
    bad |= !valid && e != -1;
    id[i] = valid ? e : -1;
    if (valid) atomicAdd(&count[e], 1);
  }
  if (bad && t == 0) atomicOr(&g_dg_error, 0x2);
  __syncthreads();
  // segment offsets: exclusive scan of the counts rounded up to 128, four experts a thread
  constexpr int kEach = kMoeMaxExperts / kFewThreads;
  int sum = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int e = kEach * tid + i;
    sum += e < p.G ? (count[e] + 127) & ~127 : 0;
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) part[warp] = incl;
  uint32_t amax = 0;
  if constexpr (U > 0) {
#pragma unroll
    for (int i = 0; i < U; ++i) amax = max(amax, v[i].top());
  } else if (has) {
    for (int u = tid; u < units; u += kFewThreads) {
      v[0].load(x + 16 * static_cast<size_t>(u));
      amax = max(amax, v[0].top());
    }
  }
  amax = __reduce_max_sync(0xffffffffu, amax);
  if (lane == 0) top[warp] = amax;
  __syncthreads();
  int at = incl - sum, total = 0;
#pragma unroll
  for (int w = 0; w < kFewThreads / 32; ++w) {
    at += w < warp ? part[w] : 0;
    total += part[w];
    amax = max(amax, top[w]);
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int e = kEach * tid + i;
    if (e < p.G) {
      segment[e] = at;
      at += (count[e] + 127) & ~127;
    }
  }
  __syncthreads();
  float scale, inverse;
  int8_scale(amax, scale, inverse);
  if (has) {
    // a slot's row: its expert's segment, behind the earlier slots of the same expert
    for (int s = warp; s < p.topk; s += kFewThreads / 32) {
      const int pos = t * p.topk + s;
      const int e = id[pos];
      int before = 0;
      for (int i = lane; i < pos; i += 32) before += id[i] == e;
      before = __reduce_add_sync(0xffffffffu, before);
      const int r = e < 0 ? -1 : segment[e] + before;
      if (lane == 0) {
        slot_row[s] = r;
        p.row_of_out[pos] = r;
        if (r >= 0) {
          p.scale[r] = scale;
          p.m_indices[r] = e;
          p.src_of[r] = t;
        }
      }
    }
    __syncthreads();
    if constexpr (U > 0) {
      uint4 c[U];
#pragma unroll
      for (int i = 0; i < U; ++i) c[i] = int8_codes(v[i], inverse);
      for (int s = 0; s < p.topk; ++s) {
        const int r = slot_row[s];
        if (r < 0) continue;
        uint4* to = reinterpret_cast<uint4*>(p.q + static_cast<size_t>(r) * p.K);
#pragma unroll
        for (int i = 0; i < U; ++i)
          if (tid + i * kFewThreads < units) to[tid + i * kFewThreads] = c[i];
      }
    } else {
      for (int u = tid; u < units; u += kFewThreads) {
        v[0].load(x + 16 * static_cast<size_t>(u));
        const uint4 c = int8_codes(v[0], inverse);
        for (int s = 0; s < p.topk; ++s)
          if (slot_row[s] >= 0) reinterpret_cast<uint4*>(p.q + static_cast<size_t>(slot_row[s]) * p.K)[u] = c;
      }
    }
  }
  // padding rows of the segments, an expert a warp, and the rows behind the last segment
  const int warps = gridDim.x * (kFewThreads / 32);
  for (int e = t * (kFewThreads / 32) + warp; e < p.G; e += warps)
    for (int r = segment[e] + count[e] + lane; r < segment[e] + ((count[e] + 127) & ~127); r += 32) {
      p.m_indices[r] = -1;
      p.src_of[r] = -1;
      p.scale[r] = 0.0f;
    }
  for (int r = total + t * kFewThreads + tid; r < p.M_cap; r += gridDim.x * kFewThreads) {
    p.m_indices[r] = -1;
    p.src_of[r] = -1;
    p.scale[r] = 0.0f;
  }
}

}  // namespace dg
