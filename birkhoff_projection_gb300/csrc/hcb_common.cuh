// hcb_common.cuh -- pieces shared by the hyper-connection block kernels
// (hcb_enter.cu, hcb_leave.cu, hcb_leave_bwd.cu): row vectors in fp32 and
// bf16, the sums over a row, gates, and the launch shape.
//
// Mapping.  A group of G threads (a power of two, a warp at least) takes one
// token at a time; a CTA holds NG groups, and the grid is persistent (SMs x
// resident CTAs), so that a thread meets the same channels in every token
// and can keep its share of the weight gradients in shared memory until its
// last token.  Thread l of a group owns the channels [(k G + l) V, + V) for
// k = 0, 1, ...; what a row's second pass needs again is kept in fp32 in
// shared memory by the thread that wrote it (no barrier), while the barriers
// of the sums are between the threads of one group only.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "b4_device.cuh"
#include "b4_types.h"
#include "hc_block.h"

namespace b4 {
int record_cuda_error(cudaError_t e);  // birkhoff4_api.cu
}  // namespace b4

namespace hcb {

using b4::bf16_t;

constexpr int kThreads = 256;   // threads of a CTA with many short rows
constexpr int kMaxGroup = 512;  // threads of a group at most
constexpr int kMaxRows = 640;   // CTAs of a backward pass at most (rows of partial weight gradients)

// ---------------------------------------------------------------------------
// V consecutive elements of a row as floats
// ---------------------------------------------------------------------------
template <class T, int V>
struct Row;

template <int V>
struct Row<float, V> {
  static_assert(V == 1 || V == 4, "");
  __device__ __forceinline__ static void load(const float* p, float (&v)[V]) {
    if constexpr (V == 4) {
      const float4 q = *reinterpret_cast<const float4*>(p);
      v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
    } else {
      v[0] = *p;
    }
  }
  __device__ __forceinline__ static void store(float* p, const float (&v)[V]) {
    if constexpr (V == 4) {
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      *p = v[0];
    }
  }
  __device__ __forceinline__ static float round(float x) { return x; }
};

template <int V>
struct Row<bf16_t, V> {
  static_assert(V == 1 || V == 4 || V == 8, "");
  __device__ __forceinline__ static void load(const bf16_t* p, float (&v)[V]) {
    if constexpr (V == 8) {
      const uint4 q = *reinterpret_cast<const uint4*>(p);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) v[2 * i] = b4::bf16lo(w[i]), v[2 * i + 1] = b4::bf16hi(w[i]);
    } else if constexpr (V == 4) {
      const uint2 q = *reinterpret_cast<const uint2*>(p);
      v[0] = b4::bf16lo(q.x), v[1] = b4::bf16hi(q.x), v[2] = b4::bf16lo(q.y), v[3] = b4::bf16hi(q.y);
    } else {
      v[0] = b4::bf16lo(p->bits);
    }
  }
  __device__ __forceinline__ static void store(bf16_t* p, const float (&v)[V]) {
    if constexpr (V == 8) {
      *reinterpret_cast<uint4*>(p) = make_uint4(b4::pack_bf16(v[0], v[1]), b4::pack_bf16(v[2], v[3]),
                                                b4::pack_bf16(v[4], v[5]), b4::pack_bf16(v[6], v[7]));
    } else if constexpr (V == 4) {
      *reinterpret_cast<uint2*>(p) = make_uint2(b4::pack_bf16(v[0], v[1]), b4::pack_bf16(v[2], v[3]));
    } else {
      p->bits = static_cast<uint16_t>(b4::pack_bf16(v[0], 0.0f));
    }
  }
  __device__ __forceinline__ static float round(float x) {
    return b4::bf16lo(b4::pack_bf16(x, 0.0f));
  }
};

// fp32 scratch of a row in shared memory (V floats at a multiple of V)
template <int V>
__device__ __forceinline__ void keep(float* s, const float (&v)[V]) {
  if constexpr (V >= 4) {
#pragma unroll
    for (int i = 0; i < V; i += 4)
      *reinterpret_cast<float4*>(s + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  } else {
    s[0] = v[0];
  }
}
template <int V>
__device__ __forceinline__ void kept(const float* s, float (&v)[V]) {
  if constexpr (V >= 4) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 q = *reinterpret_cast<const float4*>(s + i);
      v[i] = q.x, v[i + 1] = q.y, v[i + 2] = q.z, v[i + 3] = q.w;
    }
  } else {
    v[0] = s[0];
  }
}

// A pointer to fp32 or bf16 values, told apart at run time: coefficients and
// weights, which are few beside the rows.
struct Any {
  const void* p;
  int32_t bf16;
  __device__ __forceinline__ float at(int64_t i) const {
    return bf16 ? b4::bf16lo(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
  }
  template <int V>
  __device__ __forceinline__ void load(int64_t i, float (&v)[V]) const {  // 1 where absent
    if (p == nullptr) {
#pragma unroll
      for (int k = 0; k < V; ++k) v[k] = 1.0f;
    } else if (bf16) {
      Row<bf16_t, V>::load(static_cast<const bf16_t*>(p) + i, v);
    } else if constexpr (V == 8) {
      float lo[4], hi[4];
      Row<float, 4>::load(static_cast<const float*>(p) + i, lo);
      Row<float, 4>::load(static_cast<const float*>(p) + i + 4, hi);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = lo[k], v[4 + k] = hi[k];
    } else {
      Row<float, V>::load(static_cast<const float*>(p) + i, v);
    }
  }
};

__device__ __forceinline__ void put_any(void* p, int32_t bf16, int64_t i, float v) {
  if (bf16)
    static_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(b4::pack_bf16(v, 0.0f));
  else
    static_cast<float*>(p)[i] = v;
}

// ---------------------------------------------------------------------------
// Kernel arguments
// ---------------------------------------------------------------------------
struct Params {
  int64_t T;
  int32_t S, C;
  int32_t G;  // threads of a group
  int32_t act, norm;
  float eps, eps_next, scale;
  const void *x, *y, *gate, *dout, *dh, *dres, *out_in;
  Any P, a, b, w, wn;
  int64_t x_ts, x_ss, y_ts, gate_ts, P_ts, a_ts, b_ts, dout_ts, dout_ss, dh_ts, dres_ts, dres_ss,
      out_ts, out_ss;
  void *h, *out, *dx, *dy, *dgate, *dP, *da, *db;
  float *dw, *dwn;  // partial weight gradients [CTAs, C]
};

// ---------------------------------------------------------------------------
// Sums over the threads of a group
// ---------------------------------------------------------------------------
__device__ __forceinline__ void group_sync(int G, int group) {
  if (G == 32)
    __syncwarp();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(G) : "memory");
}

// One warp's sums of up to 32 values in 31 shuffles: each exchange with the
// lane `o` away halves the values that a lane carries, so lane l ends with
// the sum of value l (0 from R on).
template <int R>
__device__ __forceinline__ float warp_sums(const float (&in)[R], int lane) {
  static_assert(R >= 1 && R <= 32, "");
  constexpr int N = R <= 1 ? 1 : R <= 2 ? 2 : R <= 4 ? 4 : R <= 8 ? 8 : R <= 16 ? 16 : 32;
  float v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = i < R ? in[i] : 0.0f;
  int o = 16;
#pragma unroll
  for (int n = N; n > 1; n >>= 1, o >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const float give = up ? v[i] : v[i + n / 2];
      const float stay = up ? v[i + n / 2] : v[i];
      v[i] = stay + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
#pragma unroll
  for (; o > 0; o >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
  // lane l now has the sum of value l / (32 / N)
  if constexpr (N == 32) return v[0];
  return __shfl_sync(0xffffffffu, v[0], (lane * (32 / N)) & 31);
}

// Sums of R values over a group of G threads: on return lane l of every warp
// has value l + 32 c in total[c].  `red` holds [2][G / 32][R] floats of the
// group; `turn` alternates between calls, so that one barrier a call is
// enough (a warp can be one call ahead of another, not two).
template <int R>
struct GroupSum {
  static constexpr int CH = (R + 31) / 32;
  static __host__ __device__ constexpr int floats(int G) { return 2 * (G / 32) * R; }
  __device__ __forceinline__ static void run(const float (&v)[R], float (&total)[CH], float* red,
                                             int& turn, int G, int group, int lane, int warp) {
    sums<0>(v, total, lane);
    if (G == 32) return;
    float* r = red + turn * (G / 32) * R;
    turn ^= 1;
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (c * 32 + lane < R) r[warp * R + c * 32 + lane] = total[c];
    group_sync(G, group);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float s = 0.0f;
      if (c * 32 + lane < R)
        for (int w = 0; w < G / 32; ++w) s += r[w * R + c * 32 + lane];
      total[c] = s;
    }
  }

 private:
  template <int K>
  __device__ __forceinline__ static void sums(const float (&v)[R], float (&total)[CH], int lane) {
    if constexpr (K < CH) {
      constexpr int N = R - 32 * K < 32 ? R - 32 * K : 32;
      float part[N];
#pragma unroll
      for (int i = 0; i < N; ++i) part[i] = v[32 * K + i];
      total[K] = warp_sums<N>(part, lane);
      sums<K + 1>(v, total, lane);
    }
  }
};

// Value i of a GroupSum's totals, in every lane.
template <int CH>
__device__ __forceinline__ float of_total(const float (&total)[CH], int i) {
  float r = 0.0f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const float t = __shfl_sync(0xffffffffu, total[c], i & 31);
    if (i / 32 == c) r = t;
  }
  return r;
}

// ---------------------------------------------------------------------------
// Gates: value and slope of act(g).  e = exp(-|g|) keeps 1 - sigmoid exact
// to fp32 on both sides and never overflows.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void gate_of(int act, float g, float& value, float& slope) {
  if (act == HCB_ACT_LINEAR) {
    value = g, slope = 1.0f;
    return;
  }
  const float e = __expf(-fabsf(g));
  const float inv = __fdividef(1.0f, 1.0f + e);
  const float s = g >= 0.0f ? inv : e * inv;
  const float rest = g >= 0.0f ? e * inv : inv;  // 1 - s
  // NaN: both comparisons are false and e is NaN, so s and rest are NaN
  if (act == HCB_ACT_SIGMOID)
    value = s, slope = s * rest;
  else
    value = g * s, slope = s * (1.0f + g * rest);
}

// ---------------------------------------------------------------------------
// Launch shape
// ---------------------------------------------------------------------------
struct Shape {
  int G, NG;
};

int sms();  // SMs of the current device (hcb_api.cu)

inline int padded(int C) { return (C + 3) / 4 * 4; }  // floats of a kept row

// Threads of a group: two vectors of a row to a thread where the tokens fill
// the GPU, one where they do not (a longer group shortens a token's path).
inline Shape shape_of(int64_t T, int C, int V, int max_group) {
  const int vecs = (C + V - 1) / V;
  const int per = T < sms() ? 1 : 2;
  int G = 32;
  while (G < max_group && G * per < vecs) G *= 2;
  return {G, std::max(1, kThreads / G)};
}

// Resident CTAs per SM of a kernel at (threads, shared bytes), remembered per
// kernel for the last such pair: the occupancy query is a host call that
// would show in the smallest launches.
template <auto KERN>
cudaError_t resident(int threads, size_t smem, int* out) {
  static std::atomic<uint64_t> last[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t key = (static_cast<uint64_t>(smem) << 24) | (static_cast<uint64_t>(threads) << 8);
  if (dev < 64) {
    const uint64_t got = last[dev].load(std::memory_order_acquire);
    if ((got & ~0xffull) == key && (got & 0xff) != 0) {
      *out = static_cast<int>(got & 0xff);
      return cudaSuccess;
    }
  }
  // the opt-in limit of a CTA, less the kernel's static shared memory
  cudaFuncAttributes fa;
  e = cudaFuncGetAttributes(&fa, KERN);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           232448 - static_cast<int>(fa.sharedSizeBytes));
  if (e != cudaSuccess) return e;
  int occ = 0;
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, KERN, threads, smem);
  if (e != cudaSuccess) return e;
  *out = std::max(1, std::min(occ, 255));
  if (dev < 64) last[dev].store(key | static_cast<uint64_t>(*out), std::memory_order_release);
  return cudaSuccess;
}

// Persistent launch of KERN: NG tokens to a CTA, `smem` bytes for each token's
// group.  At most max_grid CTAs; the grid is returned in *grid.
template <auto KERN>
cudaError_t launch(Params p, Shape sh, size_t smem_group, int max_grid, int* grid, cudaStream_t s) {
  p.G = sh.G;
  const size_t smem = smem_group * sh.NG;
  int occ = 0;
  const cudaError_t e = resident<KERN>(sh.G * sh.NG, smem, &occ);
  if (e != cudaSuccess) return e;
  const int64_t want = (p.T + sh.NG - 1) / sh.NG;
  *grid = static_cast<int>(std::min<int64_t>(want, std::min<int64_t>(max_grid, int64_t(sms()) * occ)));
  KERN<<<*grid, sh.G * sh.NG, smem, s>>>(p);
  return cudaGetLastError();
}

// Call F.operator()<SP, TX, TY, V>() for the streams (rounded up to 1, 2, 4
// or 8; the missing ones count as zeros), the row types and the vector width:
// 16 bytes of the wider row type (8 bytes of bf16 at 8 streams, for the
// registers), or single elements where rows do not allow vectors.
template <int SP, class F>
cudaError_t by_type(int x_bf16, int y_bf16, bool vec, F&& f) {
  constexpr int VB = SP == 8 ? 4 : 8;
  if (x_bf16) return vec ? f.template operator()<SP, bf16_t, bf16_t, VB>() : f.template operator()<SP, bf16_t, bf16_t, 1>();
  if (y_bf16) return vec ? f.template operator()<SP, float, bf16_t, 4>() : f.template operator()<SP, float, bf16_t, 1>();
  return vec ? f.template operator()<SP, float, float, 4>() : f.template operator()<SP, float, float, 1>();
}
template <class F>
cudaError_t by_streams(int S, int x_bf16, int y_bf16, bool vec, F&& f) {
  if (S == 1) return by_type<1>(x_bf16, y_bf16, vec, f);
  if (S == 2) return by_type<2>(x_bf16, y_bf16, vec, f);
  if (S <= 4) return by_type<4>(x_bf16, y_bf16, vec, f);
  return by_type<8>(x_bf16, y_bf16, vec, f);
}

// Sum the partial weight gradients [rows, C] and write them (hcb_api.cu).
cudaError_t finish_weights(const float* part, const float* part_next, int rows, int C, void* dw,
                           int dw_bf16, void* dwn, int dwn_bf16, cudaStream_t s);

// The pass launchers, one translation unit each: enqueue on `s`.
cudaError_t enter_forward(const Params& p, int x_bf16, int y_bf16, bool vec, cudaStream_t s);
cudaError_t enter_backward(const Params& p, int x_bf16, int y_bf16, bool vec, int* rows, cudaStream_t s);
cudaError_t leave_forward(const Params& p, int x_bf16, int y_bf16, bool vec, cudaStream_t s);
cudaError_t leave_backward(const Params& p, int x_bf16, int y_bf16, bool vec, int* rows, cudaStream_t s);

}  // namespace hcb
