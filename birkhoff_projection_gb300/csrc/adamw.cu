// adamw.cu -- one AdamW step over many tensors (adamw_step of
// include/adamw.h).
//
// A launch takes up to kTable tensors; their pointers travel in the launch's
// argument, so nothing is copied to the device and a captured launch replays.
// The elements are cut into chunks of kChunk that never cross a tensor; a
// CTA finds its chunk's tensor by bisection in the running count of chunks.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "adamw.h"
#include "b4_device.cuh"
#include "b4_types.h"

namespace b4 {
int record_cuda_error(cudaError_t e);  // birkhoff4_api.cu
}

namespace adamw {

using b4::bf16_t;

constexpr int kThreads = 256;
constexpr int kVec = 8;                    // elements of a thread at a time
constexpr int kChunk = kThreads * kVec;    // elements of a CTA
constexpr int kTable = 256;                // tensors of a launch at most
constexpr float kTop = 448.0f;             // e4m3's largest number
constexpr float kLeast = 0.001953125f;     // its smallest positive one, 2^-9
static_assert(ADAMW_BLOCK % kVec == 0 && kChunk % ADAMW_BLOCK == 0 && ADAMW_BLOCK / kVec == 16, "");

struct Entry {
  void* p;
  const void* g;
  void *m, *v;
  float *m_scale, *v_scale, *master;
  int64_t n;
  int64_t vec;  // on 16-byte boundaries
};
// N tensors of a launch: a launch's arguments are copied on every call, so
// few tensors take a smaller table.
template <int N>
struct Table {
  int32_t count;
  uint32_t first[N + 1];  // chunks before each tensor
  Entry at[N];
};

struct Hyper {
  float beta1, rest1, beta2, rest2;  // beta and 1 - beta
  float keep, rate, inv_root2, eps;  // 1 - lr wd, lr / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
  const float* grad_scale;
};

// One element: the new moments (every product and sum rounded by itself) and
// the new weight.
__device__ __forceinline__ void update(const Hyper& h, float g, float& p, float& m, float& v, float& r) {
  m = __fadd_rn(__fmul_rn(h.beta1, m), __fmul_rn(h.rest1, g));
  v = __fadd_rn(__fmul_rn(h.beta2, v), __fmul_rn(h.rest2, __fmul_rn(g, g)));
  r = __fsqrt_rn(v);
  p = p * h.keep - h.rate * m / (r * h.inv_root2 + h.eps);
}

template <class T>
__device__ __forceinline__ void load8(const void* base, int64_t i, int left, bool vec, float (&x)[kVec]) {
  const T* p = static_cast<const T*>(base) + i;
  if constexpr (sizeof(T) == 4) {
    if (vec && left >= kVec) {
      const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
      x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    } else {
#pragma unroll
      for (int k = 0; k < kVec; ++k) x[k] = k < left ? p[k] : 0.0f;
    }
  } else {
    if (vec && left >= kVec) {
      const uint4 q = *reinterpret_cast<const uint4*>(p);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) x[2 * k] = b4::bf16lo(w[k]), x[2 * k + 1] = b4::bf16hi(w[k]);
    } else {
#pragma unroll
      for (int k = 0; k < kVec; ++k) x[k] = k < left ? b4::bf16lo(p[k].bits) : 0.0f;
    }
  }
}
template <class T>
__device__ __forceinline__ void store8(void* base, int64_t i, int left, bool vec, const float (&x)[kVec]) {
  T* p = static_cast<T*>(base) + i;
  if constexpr (sizeof(T) == 4) {
    if (vec && left >= kVec) {
      reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
#pragma unroll
      for (int k = 0; k < kVec; ++k)
        if (k < left) p[k] = x[k];
    }
  } else {
    if (vec && left >= kVec) {
      *reinterpret_cast<uint4*>(p) = make_uint4(b4::pack_bf16(x[0], x[1]), b4::pack_bf16(x[2], x[3]),
                                                b4::pack_bf16(x[4], x[5]), b4::pack_bf16(x[6], x[7]));
    } else {
#pragma unroll
      for (int k = 0; k < kVec; ++k)
        if (k < left) p[k].bits = static_cast<uint16_t>(b4::pack_bf16(x[k], 0.0f));
    }
  }
}

// Eight e4m3 codes
__device__ __forceinline__ void load_codes(const void* base, int64_t i, int left, bool vec, float scale,
                                           float (&x)[kVec]) {
  const uint8_t* p = static_cast<const uint8_t*>(base) + i;
  uint32_t w[2] = {0, 0};
  if (vec && left >= kVec) {
    const uint2 q = *reinterpret_cast<const uint2*>(p);
    w[0] = q.x, w[1] = q.y;
  } else {
#pragma unroll
    for (int k = 0; k < kVec; ++k)
      if (k < left) w[k / 4] |= static_cast<uint32_t>(p[k]) << (8 * (k % 4));
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t h;  // two fp16, exact
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w[k / 2] >> (16 * (k % 2)))));
    float lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(h));
    x[2 * k] = __fmul_rn(lo, scale), x[2 * k + 1] = __fmul_rn(hi, scale);
  }
}
__device__ __forceinline__ void store_codes(void* base, int64_t i, int left, bool vec, const float (&q)[kVec]) {
  uint32_t w[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(q[4 * k + 1]), "f"(q[4 * k]));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(q[4 * k + 3]), "f"(q[4 * k + 2]));
    w[k] = static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
  }
  uint8_t* p = static_cast<uint8_t*>(base) + i;
  if (vec && left >= kVec) {
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int k = 0; k < kVec; ++k)
      if (k < left) p[k] = static_cast<uint8_t>(w[k / 4] >> (8 * (k % 4)));
  }
}

// The scale of a block from the magnitudes of its 16 threads, and its
// values' codes before rounding.
__device__ __forceinline__ float encode(float (&x)[kVec], bool root) {
  float most = 0.0f;
#pragma unroll
  for (int k = 0; k < kVec; ++k) {
    const float a = fabsf(x[k]);
    most = fmaxf(most, a < INFINITY ? a : 0.0f);  // NaN and infinities do not count
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  // below about 2^-119 the factor would overflow: held at 3e38, it stores such a block's values smaller
  const float inv = most > 0.0f ? fminf(__fmul_rn(kTop, __frcp_rn(most)), 3.0e38f) : 0.0f;
#pragma unroll
  for (int k = 0; k < kVec; ++k) {
    float q = __fmul_rn(x[k], inv);
    if (root && x[k] > 0.0f) q = fmaxf(q, kLeast);
    if (!(fabsf(x[k]) < INFINITY)) q = NAN;
    x[k] = q;
  }
  return __fmul_rn(most, 1.0f / kTop);
}

template <class TP, class TG, bool MASTER, bool EIGHT, int N>
__global__ void __launch_bounds__(kThreads) step_kernel(const __grid_constant__ Table<N> t, const Hyper h) {
  const uint32_t chunk = blockIdx.x;
  int lo = 0, hi = t.count;  // the last tensor whose first chunk is at most `chunk`
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (t.first[mid] <= chunk)
      lo = mid;
    else
      hi = mid;
  }
  const Entry& x = t.at[lo];
  const bool vec = x.vec != 0;
  const int64_t i = int64_t(chunk - t.first[lo]) * kChunk + threadIdx.x * kVec;
  const int64_t rest = x.n - i;
  const int left = rest > kVec ? kVec : rest < 0 ? 0 : static_cast<int>(rest);
  float g[kVec], p[kVec], m[kVec], v[kVec];
  load8<TG>(x.g, i, left, vec, g);
  if constexpr (MASTER)
    load8<float>(x.master, i, left, vec, p);
  else
    load8<TP>(x.p, i, left, vec, p);
  if constexpr (EIGHT) {
    const int64_t block = i / ADAMW_BLOCK;
    load_codes(x.m, i, left, vec, left > 0 ? x.m_scale[block] : 0.0f, m);
    load_codes(x.v, i, left, vec, left > 0 ? x.v_scale[block] : 0.0f, v);
#pragma unroll
    for (int j = 0; j < kVec; ++j) v[j] = __fmul_rn(v[j], v[j]);
  } else {
    load8<float>(x.m, i, left, vec, m);
    load8<float>(x.v, i, left, vec, v);
  }
  if (h.grad_scale) {
    const float s = *h.grad_scale;
#pragma unroll
    for (int j = 0; j < kVec; ++j) g[j] *= s;
  }
  float r[kVec];
#pragma unroll
  for (int j = 0; j < kVec; ++j) update(h, g[j], p[j], m[j], v[j], r[j]);
  if constexpr (MASTER) store8<float>(x.master, i, left, vec, p);
  store8<TP>(x.p, i, left, vec, p);
  if constexpr (EIGHT) {
    const float ms = encode(m, false), vs = encode(r, true);
    store_codes(x.m, i, left, vec, m);
    store_codes(x.v, i, left, vec, r);
    if (left > 0 && threadIdx.x % (ADAMW_BLOCK / kVec) == 0) {
      x.m_scale[i / ADAMW_BLOCK] = ms;
      x.v_scale[i / ADAMW_BLOCK] = vs;
    }
  } else {
    store8<float>(x.m, i, left, vec, m);
    store8<float>(x.v, i, left, vec, v);
  }
}

namespace {

bool placed(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

constexpr int kSmallTable = 48;

template <class TP, class TG, bool MASTER, bool EIGHT>
cudaError_t launch(const Table<kTable>& t, const Hyper& h, cudaStream_t s) {
  const uint32_t grid = t.first[t.count];
  if (t.count <= kSmallTable) {
    Table<kSmallTable> u;
    u.count = t.count;
    memcpy(u.first, t.first, sizeof(uint32_t) * (t.count + 1));
    memcpy(u.at, t.at, sizeof(Entry) * t.count);
    step_kernel<TP, TG, MASTER, EIGHT, kSmallTable><<<grid, kThreads, 0, s>>>(u, h);
  } else {
    step_kernel<TP, TG, MASTER, EIGHT, kTable><<<grid, kThreads, 0, s>>>(t, h);
  }
  return cudaGetLastError();
}
template <class TP, class TG, bool MASTER>
cudaError_t launch(const Table<kTable>& t, const Hyper& h, bool eight, cudaStream_t s) {
  return eight ? launch<TP, TG, MASTER, true>(t, h, s) : launch<TP, TG, MASTER, false>(t, h, s);
}

cudaError_t launch_any(const Table<kTable>& t, const Hyper& h, const adamw_opts* o, bool master, cudaStream_t s) {
  const bool eight = o->state_bits == 8, gb = o->g_dtype == B4_BF16;
  if (o->p_dtype == B4_F32)
    return gb ? launch<float, bf16_t, false>(t, h, eight, s) : launch<float, float, false>(t, h, eight, s);
  if (master)
    return gb ? launch<bf16_t, bf16_t, true>(t, h, eight, s) : launch<bf16_t, float, true>(t, h, eight, s);
  return gb ? launch<bf16_t, bf16_t, false>(t, h, eight, s) : launch<bf16_t, float, false>(t, h, eight, s);
}

}  // namespace
}  // namespace adamw

extern "C" int adamw_step(const adamw_tensor* x, int32_t count, const adamw_opts* o,
                          birkhoff4_stream_t stream) {
  using namespace adamw;
  if (o == nullptr || count < 0 || (count > 0 && x == nullptr)) return B4_EINVAL;
  if ((o->p_dtype != B4_F32 && o->p_dtype != B4_BF16) || (o->g_dtype != B4_F32 && o->g_dtype != B4_BF16))
    return B4_EINVAL;
  if (o->state_bits != 32 && o->state_bits != 8) return B4_EINVAL;
  for (double b : {o->beta1, o->beta2})
    if (!(b >= 0.0 && b < 1.0)) return B4_EINVAL;
  for (double b : {o->lr, o->eps, o->weight_decay})
    if (!(b >= 0.0) || std::isinf(b)) return B4_EINVAL;
  if (o->step < 1 || !placed(o->grad_scale, 4)) return B4_EINVAL;
  const bool eight = o->state_bits == 8;
  const int pb = o->p_dtype == B4_F32 ? 4 : 2, gb = o->g_dtype == B4_F32 ? 4 : 2;
  bool master = false;
  for (int32_t k = 0; k < count; ++k) {
    if (x[k].n < 0) return B4_EINVAL;
    if (k == 0)
      master = x[k].master != nullptr;
    else if (master != (x[k].master != nullptr))
      return B4_EINVAL;
    if (x[k].n == 0) continue;
    if (x[k].p == nullptr || x[k].g == nullptr || x[k].m == nullptr || x[k].v == nullptr) return B4_EINVAL;
    if (!placed(x[k].p, pb) || !placed(x[k].g, gb) || !placed(x[k].master, 4)) return B4_EINVAL;
    if (!eight && (!placed(x[k].m, 4) || !placed(x[k].v, 4))) return B4_EINVAL;
    if (eight && (x[k].m_scale == nullptr || x[k].v_scale == nullptr || !placed(x[k].m_scale, 4) ||
                  !placed(x[k].v_scale, 4)))
      return B4_EINVAL;
    if (x[k].n > (int64_t(1) << 40)) return B4_EINVAL;
  }
  if (master && o->p_dtype == B4_F32) return B4_ENOTIMPL;

  Hyper h;
  h.beta1 = static_cast<float>(o->beta1), h.rest1 = static_cast<float>(1.0 - o->beta1);
  h.beta2 = static_cast<float>(o->beta2), h.rest2 = static_cast<float>(1.0 - o->beta2);
  const double t = static_cast<double>(o->step);
  h.keep = static_cast<float>(1.0 - o->lr * o->weight_decay);
  h.rate = static_cast<float>(o->lr / (1.0 - std::pow(o->beta1, t)));
  h.inv_root2 = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(o->beta2, t)));
  h.eps = static_cast<float>(o->eps);
  h.grad_scale = o->grad_scale;

  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  Table<kTable> tab;
  tab.count = 0;
  for (int32_t k = 0; k < count; ++k) {
    if (x[k].n == 0) continue;
    // a tensor of more chunks than a grid holds is taken in pieces
    constexpr int64_t kMost = (int64_t(1) << 30) * kChunk;
    for (int64_t at = 0; at < x[k].n; at += kMost) {
      const int64_t n = std::min(x[k].n - at, kMost);
      const uint32_t chunks = static_cast<uint32_t>((n + kChunk - 1) / kChunk);
      if (tab.count == kTable || (tab.count > 0 && uint64_t(tab.first[tab.count]) + chunks > 0x7fffffffu)) {
        const cudaError_t e = launch_any(tab, h, o, master, s);
        if (e != cudaSuccess) return b4::record_cuda_error(e);
        tab.count = 0;
      }
      const int c = tab.count++;
      Entry& q = tab.at[c];
      q.p = static_cast<char*>(x[k].p) + at * pb;
      q.g = static_cast<const char*>(x[k].g) + at * gb;
      q.m = static_cast<char*>(x[k].m) + at * (eight ? 1 : 4);
      q.v = static_cast<char*>(x[k].v) + at * (eight ? 1 : 4);
      q.m_scale = eight ? x[k].m_scale + at / ADAMW_BLOCK : nullptr;
      q.v_scale = eight ? x[k].v_scale + at / ADAMW_BLOCK : nullptr;
      q.master = master ? x[k].master + at : nullptr;
      q.n = n;
      q.vec = placed(q.p, 16) && placed(q.g, 16) && placed(q.m, eight ? 8 : 16) && placed(q.v, eight ? 8 : 16) &&
              placed(q.master, 16);
      if (c == 0) tab.first[0] = 0;
      tab.first[c + 1] = tab.first[c] + chunks;
    }
  }
  if (tab.count == 0) return B4_OK;
  return b4::record_cuda_error(launch_any(tab, h, o, master, s));
}
