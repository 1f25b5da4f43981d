// adamw.cu -- one AdamW step over many tensors (adamw_step of
// include/adamw.h).
//
// A launch takes up to kTable tensors; their pointers travel in the launch's
// argument, so nothing is copied to the device and a captured launch replays.
// The elements are cut into chunks of kChunk that never cross a tensor; a
// CTA finds its chunk's tensor by bisection in the running count of chunks.
//
// Every element is read and written once.  Bound by memory: two layers of
// 2048 wide fp32 matrices, 3.8 GB, take 530 us with fp32 moments (7.1 TB/s;
// more than a copy reaches, as reads outnumber writes), 324 us with 8-bit ones
// (99% of the copy's rate), bf16 with fp32 masters and 8-bit moments 320 us
// (100%).  Of bf16 weights alone with 8-bit moments, 10 bytes to an element,
// the instructions that find a block's scale and make the codes take as long
// (262 us, 77%).  CTAs that the registers have to leave room for: 8-bit
// moments hide their conversions behind more warps (four 320 us, three 348,
// five, spilt, 346), fp32 ones need the registers for loads (three 532, four
// 599, five 769).
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "adamw.h"
#include "b4_device.cuh"
#include "b4_pairs.cuh"
#include "b4_types.h"

namespace b4 {
int record_cuda_error(cudaError_t e);  // birkhoff4_api.cu
}

namespace adamw {

using namespace b4::pairs;
using b4::bf16_t;

constexpr int kThreads = 256;
constexpr int kVec = 8;                          // neighbouring elements of a thread
constexpr int kRuns = 2;                         // runs of kThreads kVec elements of a CTA
constexpr int kChunk = kRuns * kThreads * kVec;  // elements of a CTA
constexpr int kTable = 256;                      // tensors of a launch at most
constexpr float kTop = 448.0f;                   // e4m3's largest number
constexpr float kLeast = 0.001953125f;           // its smallest positive one, 2^-9
static_assert(ADAMW_BLOCK % kVec == 0 && kThreads * kVec % ADAMW_BLOCK == 0 && ADAMW_BLOCK / kVec == 16, "");

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
  float one;                         // 1
  const float* grad_scale;
};

// Eight elements as they are in memory: 16 bytes to an fp32 quadruple, a bf16
// octuple or (half of them) eight codes.  The loads of all of a thread's
// arrays and runs are issued before the first is used.
template <class T>
struct Eight {
  static constexpr int WORDS = 2 * sizeof(T);
  uint32_t w[WORDS];

  __device__ __forceinline__ void load(const void* base, int64_t i, int left, bool vec) {
    const T* p = static_cast<const T*>(base) + i;
    if (vec && left >= kVec) {
      if constexpr (WORDS == 2) {
        const uint2 q = *reinterpret_cast<const uint2*>(p);
        w[0] = q.x, w[1] = q.y;
      } else {
#pragma unroll
        for (int k = 0; k < WORDS / 4; ++k) {
          const uint4 q = reinterpret_cast<const uint4*>(p)[k];
          w[4 * k] = q.x, w[4 * k + 1] = q.y, w[4 * k + 2] = q.z, w[4 * k + 3] = q.w;
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < WORDS; ++k) w[k] = 0;
#pragma unroll
      for (int k = 0; k < kVec; ++k) {
        if (k < left) {
          uint32_t x;
          if constexpr (sizeof(T) == 4)
            x = reinterpret_cast<const uint32_t*>(p)[k];
          else if constexpr (sizeof(T) == 2)
            x = reinterpret_cast<const uint16_t*>(p)[k];
          else
            x = reinterpret_cast<const uint8_t*>(p)[k];
          w[k * sizeof(T) / 4] |= x << (8 * (k * sizeof(T) % 4));
        }
      }
    }
  }
  __device__ __forceinline__ void store(void* base, int64_t i, int left, bool vec) const {
    T* p = static_cast<T*>(base) + i;
    if (vec && left >= kVec) {
      if constexpr (WORDS == 2) {
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
      } else {
#pragma unroll
        for (int k = 0; k < WORDS / 4; ++k)
          reinterpret_cast<uint4*>(p)[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < kVec; ++k) {
        if (k < left) {
          const uint32_t x = w[k * sizeof(T) / 4] >> (8 * (k * sizeof(T) % 4));
          if constexpr (sizeof(T) == 4)
            reinterpret_cast<uint32_t*>(p)[k] = x;
          else if constexpr (sizeof(T) == 2)
            reinterpret_cast<uint16_t*>(p)[k] = static_cast<uint16_t>(x);
          else
            reinterpret_cast<uint8_t*>(p)[k] = static_cast<uint8_t>(x);
        }
      }
    }
  }
  __device__ __forceinline__ void values(P2 (&x)[4]) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (sizeof(T) == 4)
        x[k] = pair(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1]));
      else
        x[k] = pair(b4::bf16lo(w[k]), b4::bf16hi(w[k]));
    }
  }
  __device__ __forceinline__ void round(const P2 (&x)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float lo, hi;
      split(x[k], lo, hi);
      if constexpr (sizeof(T) == 4)
        w[2 * k] = __float_as_uint(lo), w[2 * k + 1] = __float_as_uint(hi);
      else
        w[k] = b4::pack_bf16(lo, hi);
    }
  }
};

// Eight e4m3 codes and their values.
__device__ __forceinline__ void decode(const Eight<uint8_t>& c, float scale, P2 (&x)[4]) {
  const P2 s = twice(scale);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t h;  // two fp16, exact
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(c.w[k / 2] >> (16 * (k % 2)))));
    float lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(h));
    x[k] = mul2(pair(lo, hi), s);
  }
}

// Maximum of magnitudes; NaN if one of them is.
__device__ __forceinline__ float most_of(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
  return r;
}

// The codes and the scale of a block of which this thread has eight values,
// 15 neighbours the others.
template <bool ROOT>
__device__ __forceinline__ float encode(const P2 (&x)[4], Eight<uint8_t>& c) {
  float v[kVec];
#pragma unroll
  for (int k = 0; k < 4; ++k) split(x[k], v[2 * k], v[2 * k + 1]);
  float most = 0.0f;
#pragma unroll
  for (int k = 0; k < kVec; ++k) most = most_of(most, v[k]);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) most = most_of(most, __shfl_xor_sync(0xffffffffu, most, o));
  const bool finite = most < INFINITY;
  if (__any_sync(0xffffffffu, !finite)) {  // NaN and infinities do not count
    float some = 0.0f;
#pragma unroll
    for (int k = 0; k < kVec; ++k) some = fmaxf(some, fabsf(v[k]) < INFINITY ? fabsf(v[k]) : 0.0f);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) some = fmaxf(some, __shfl_xor_sync(0xffffffffu, some, o));
    most = some;
  }
  // below about 2^-119 the factor would overflow: held at 3e38, it stores such a block's values smaller
  const float inv = most > 0.0f ? fminf(__fmul_rn(kTop, __frcp_rn(most)), 3.0e38f) : 0.0f;
  float q[kVec];
#pragma unroll
  for (int k = 0; k < 4; ++k) split(mul2(x[k], twice(inv)), q[2 * k], q[2 * k + 1]);
#pragma unroll
  for (int k = 0; k < kVec; ++k) {
    if constexpr (ROOT) q[k] = v[k] > 0.0f ? fmaxf(q[k], kLeast) : q[k];
    if (!finite && !(fabsf(v[k]) < INFINITY)) q[k] = NAN;
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(q[4 * k + 1]), "f"(q[4 * k]));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(q[4 * k + 3]), "f"(q[4 * k + 2]));
    c.w[k] = static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
  }
  return __fmul_rn(most, 1.0f / kTop);
}

// New moments and weights of eight elements.  The moments' products and sums
// are each rounded: a packed product and a packed sum are fused where they
// meet, so the sum is one product times 1 (a 1 that only the launch knows)
// plus the other, which rounds once and is the same number.  r is sqrt(v).
__device__ __forceinline__ void update(const Hyper& h, P2 (&g)[4], P2 (&p)[4], P2 (&m)[4], P2 (&v)[4], P2 (&r)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    m[k] = fma2(mul2(twice(h.beta1), m[k]), twice(h.one), mul2(twice(h.rest1), g[k]));
    v[k] = fma2(mul2(twice(h.beta2), v[k]), twice(h.one), mul2(twice(h.rest2), mul2(g[k], g[k])));
    float lo, hi;
    split(v[k], lo, hi);
    r[k] = pair(__fsqrt_rn(lo), __fsqrt_rn(hi));
    split(fma2(r[k], twice(h.inv_root2), twice(h.eps)), lo, hi);
    const P2 up = mul2(mul2(m[k], twice(-h.rate)), pair(b4::rcp(lo), b4::rcp(hi)));
    p[k] = fma2(p[k], twice(h.keep), up);
  }
}

template <class TP, class TG, bool MASTER, bool EIGHT, int N>
__global__ void __launch_bounds__(kThreads, EIGHT ? 4 : 3) step_kernel(const __grid_constant__ Table<N> t, const Hyper h) {
  using TW = std::conditional_t<MASTER, float, TP>;        // what the step is taken on
  using TS = std::conditional_t<EIGHT, uint8_t, float>;    // a moment's elements
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
  const int64_t i0 = int64_t(chunk - t.first[lo]) * kChunk + threadIdx.x * kVec;
  void* weights = MASTER ? static_cast<void*>(x.master) : x.p;

  Eight<TG> g8[kRuns];
  Eight<TW> p8[kRuns];
  Eight<TS> m8[kRuns], v8[kRuns];
  float ms[kRuns], vs[kRuns];
  int left[kRuns];
#pragma unroll
  for (int a = 0; a < kRuns; ++a) {
    const int64_t i = i0 + a * kThreads * kVec, rest = x.n - i;
    left[a] = rest > kVec ? kVec : rest < 0 ? 0 : static_cast<int>(rest);
    g8[a].load(x.g, i, left[a], vec);
    p8[a].load(weights, i, left[a], vec);
    m8[a].load(x.m, i, left[a], vec);
    v8[a].load(x.v, i, left[a], vec);
    if constexpr (EIGHT) {
      ms[a] = left[a] > 0 ? x.m_scale[i / ADAMW_BLOCK] : 0.0f;
      vs[a] = left[a] > 0 ? x.v_scale[i / ADAMW_BLOCK] : 0.0f;
    }
  }
  const float gs = h.grad_scale ? *h.grad_scale : 1.0f;
#pragma unroll
  for (int a = 0; a < kRuns; ++a) {
    const int64_t i = i0 + a * kThreads * kVec;
    P2 g[4], p[4], m[4], v[4], r[4];
    g8[a].values(g);
    p8[a].values(p);
    if constexpr (EIGHT) {
      decode(m8[a], ms[a], m);
      decode(v8[a], vs[a], v);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = mul2(v[k], v[k]);
    } else {
      m8[a].values(m);
      v8[a].values(v);
    }
    if (h.grad_scale) {
#pragma unroll
      for (int k = 0; k < 4; ++k) g[k] = mul2(g[k], twice(gs));
    }
    update(h, g, p, m, v, r);
    p8[a].round(p);
    p8[a].store(weights, i, left[a], vec);
    if constexpr (MASTER) {
      Eight<TP> copy;
      copy.round(p);
      copy.store(x.p, i, left[a], vec);
    }
    if constexpr (EIGHT) {
      const float mscale = encode<false>(m, m8[a]), vscale = encode<true>(r, v8[a]);
      m8[a].store(x.m, i, left[a], vec);
      v8[a].store(x.v, i, left[a], vec);
      if (left[a] > 0 && threadIdx.x % (ADAMW_BLOCK / kVec) == 0) {
        x.m_scale[i / ADAMW_BLOCK] = mscale;
        x.v_scale[i / ADAMW_BLOCK] = vscale;
      }
    } else {
      m8[a].round(m);
      v8[a].round(v);
      m8[a].store(x.m, i, left[a], vec);
      v8[a].store(x.v, i, left[a], vec);
    }
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
    if (x[k].n < 0 || x[k].n > ADAMW_MAX_ELEMENTS) return B4_EINVAL;
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
  h.one = 1.0f;
  h.grad_scale = o->grad_scale;

  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  Table<kTable> tab;
  tab.count = 0;
  for (int32_t k = 0; k < count; ++k) {
    if (x[k].n == 0) continue;
    const uint32_t chunks = static_cast<uint32_t>((x[k].n + kChunk - 1) / kChunk);  // 2^28 at most
    if (tab.count == kTable || (tab.count > 0 && uint64_t(tab.first[tab.count]) + chunks > 0x7fffffffu)) {
      const cudaError_t e = launch_any(tab, h, o, master, s);
      if (e != cudaSuccess) return b4::record_cuda_error(e);
      tab.count = 0;
    }
    const int c = tab.count++;
    Entry& q = tab.at[c];
    q.p = x[k].p, q.g = x[k].g, q.m = x[k].m, q.v = x[k].v;
    q.m_scale = eight ? x[k].m_scale : nullptr;
    q.v_scale = eight ? x[k].v_scale : nullptr;
    q.master = x[k].master;
    q.n = x[k].n;
    q.vec = placed(q.p, 16) && placed(q.g, 16) && placed(q.m, eight ? 8 : 16) && placed(q.v, eight ? 8 : 16) &&
            placed(q.master, 16);
    if (c == 0) tab.first[0] = 0;
    tab.first[c + 1] = tab.first[c] + chunks;
  }
  if (tab.count == 0) return B4_OK;
  return b4::record_cuda_error(launch_any(tab, h, o, master, s));
}
