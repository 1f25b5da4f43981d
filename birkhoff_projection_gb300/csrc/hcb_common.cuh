// hcb_common.cuh -- pieces shared by the hyper-connection block kernels
// (hcb_enter.cu, hcb_leave.cu, hcb_leave_bwd.cu): rows that travel through
// shared memory ahead of their use, the sums over a row, gates, and the
// launch shape.
//
// Mapping.  A group of G threads (whole warps, 16 at most) takes one
// token at a time; a CTA holds NG groups, and the grid is persistent (SMs x
// resident CTAs).  A warp owns the same blocks of 32 V channels of every
// token, k = 0 .. K - 1, where V elements are 16 bytes of the wider row type.
// Where rows allow vectors (ODD 0), lane l has the V channels from l V on in a
// block; where they do not, a warp's accesses of 4 bytes are to neighbouring
// words: it has the pairs of channels 64 i + 2 l (ODD 1), or, where all rows
// are fp32, the channels 32 i + l (ODD 2).  (With V channels to a lane they
// were 16 bytes apart, and leave at 5001 x 4 x 1001 took 41 us.)
//
// Loads.  All of these kernels are bound by memory, and a row's sums keep a
// group waiting at a barrier; loads into registers then left the memory idle
// (40% of its rate).  So a thread copies its own vectors of the rows that it
// will need next (cp.async) into its own slots of shared memory, DEPTH items
// ahead of its work and across the end of a token: bytes in flight cost no
// registers, and since only the thread that copied a slot reads it, the ring
// needs no barrier and no wait other than the thread's own copies.  That asks
// of every layout of a slot that a byte belongs to the same thread in all
// kinds of items that pass through it.
//
// What a row's second pass needs again is kept in shared memory by the thread
// that will read it; so are a thread's shares of the weight gradients, which
// it holds until its last token.
//
// A warp's slots and kept values are one run of bytes of its own, in planes of
// its 32 lanes: a copy of 512 contiguous bytes lands contiguously, a warp's
// accesses are conflict-free, and every plane is a constant of the kernel
// away from the lane's base.  Measured on leave's gradient at 16384 x 4 x
// 4096 bf16: planes of the group's threads 570 us (their address arithmetic
// was a third of all instructions), one run to a thread 661 us (the copies
// scatter).
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <type_traits>

#include "b4_device.cuh"
#include "b4_pairs.cuh"
#include "b4_types.h"
#include "hc_block.h"

namespace b4 {
int record_cuda_error(cudaError_t e);  // birkhoff4_api.cu
}  // namespace b4

namespace hcb {

using namespace b4::pairs;
using b4::bf16_t;

constexpr int kThreads = 256;   // threads of a CTA with many short rows
constexpr int kMaxGroup = 512;  // threads of a group at most (16 warps: GroupSum)
constexpr int kMaxRows = 640;   // CTAs of a backward pass at most (rows of partial weight gradients)

// ---------------------------------------------------------------------------
// A lane's V elements of a block of a row, and their way through shared
// memory.  `row` is the row's first element and c the lane's first channel
// (ODD: the block's).  From C on there are zeros, and nothing is written, so
// that the lanes and blocks behind a row's end need no branches of their own.
//
// ODD rows need not lie on 16-byte boundaries (any alignment of the element
// type) and end with C wherever that is.  They are copied in 4-byte words.
// Where a bf16 block begins in the middle of a word, that word is read whole
// (no allocation begins inside a word) and a pair is the upper half of one
// word and the lower half of the next; past the row's last element nothing is
// read (the copy's source size), and the slot holds zeros.
// ---------------------------------------------------------------------------
// Copies to shared memory, D and S bytes behind d and p: constants of the
// instruction, not additions to an address.  n < the size: the rest are zeros;
// nothing is read for n <= 0, wherever p points.
template <int D, int S>
__device__ __forceinline__ void copy4(uint32_t d, const void* p) {
  asm volatile("cp.async.ca.shared.global [%0+%2], [%1+%3], 4;" ::"r"(d), "l"(p), "n"(D), "n"(S) : "memory");
}
template <int D, int S>
__device__ __forceinline__ void copy4_of(uint32_t d, const void* p, int n) {
  asm volatile("cp.async.ca.shared.global [%0+%3], [%1+%4], 4, %2;" ::"r"(d), "l"(p), "r"(max(0, min(4, n))), "n"(D), "n"(S)
               : "memory");
}
template <int D>
__device__ __forceinline__ void copy8(uint32_t d, const void* p, int n) {
  asm volatile("cp.async.ca.shared.global [%0+%3], [%1], 8, %2;" ::"r"(d), "l"(p), "r"(n), "n"(D) : "memory");
}
template <int D>
__device__ __forceinline__ void copy16(uint32_t d, const void* p, int n) {
  asm volatile("cp.async.cg.shared.global [%0+%3], [%1], 16, %2;" ::"r"(d), "l"(p), "r"(n), "n"(D) : "memory");
}
// f(0), ... f(N - 1), each with its number as a constant.
template <int N, int I = 0, class F>
__device__ __forceinline__ void each(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>());
    each<N, I + 1>(f);
  }
}
// The next launch of the stream may be set up now, if it waits by itself for
// this one's results (the sums of the partial weight gradients do).
__device__ __forceinline__ void let_next_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void copy_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Channel of a lane's element e in a block that begins at c (ODD 1 and 2).
template <int ODD>
__device__ __forceinline__ int channel(int c, int lane, int e) {
  return ODD == 1 ? c + 64 * (e / 2) + 2 * lane + e % 2 : c + 32 * e + lane;
}
// Whether a block lies within its row, with one word behind it.
template <int V>
__device__ __forceinline__ bool inside(int c, int C) {
  return c + 32 * V + 2 <= C;
}

template <class T, int V, int ODD>
struct Row {
  static constexpr int H = V / 2;
  static constexpr int BYTES = V * static_cast<int>(sizeof(T));
  static constexpr bool SPLIT = ODD && sizeof(T) == 2;               // pairs may straddle words
  static constexpr int SLOT = 32 * BYTES + (SPLIT ? 16 : 0);         // bytes of a warp in a slot
  static constexpr int KEPT = 32 * BYTES;                            // and of what it keeps in this type
  static_assert(BYTES == 16 || BYTES == 8, "");

  __device__ __forceinline__ static int straddles(const T* row, int c) {
    return SPLIT ? static_cast<int>(reinterpret_cast<uintptr_t>(row + c) & 2) : 0;
  }
  // Begin the copy of the lane's elements into the slot `OFF` bytes behind s
  // (the shared address of an item's slots).  FULL: the block is inside the
  // row (any block where rows allow vectors).
  template <bool FULL, int OFF>
  __device__ __forceinline__ static void copy(uint32_t s, int lane, const T* row, int c, int C) {
    if constexpr (ODD == 0) {
      const T* p = row + min(c, C - V);
      if constexpr (BYTES == 16)
        copy16<OFF>(s + lane * 16, p, c < C ? 16 : 0);
      else
        copy8<OFF>(s + lane * 8, p, c < C ? 8 : 0);
    } else if constexpr (SPLIT) {
      const int before = straddles(row, c);
      const char* p = reinterpret_cast<const char*>(row + c) - before + 4 * lane;
      const uint32_t to = s + 4 * lane;
      constexpr int LAST = 128 * (H - 1) + 4;
      if constexpr (FULL) {
        each<H>([&](auto i) { copy4<OFF + 128 * i.value, 128 * i.value>(to, p); });
        if (lane == 31) copy4<OFF + LAST, LAST>(to, p);
      } else {
        const int end = 2 * (C - c) + before - 4 * lane;  // bytes from p to the row's end
        each<H>([&](auto i) { copy4_of<OFF + 128 * i.value, 128 * i.value>(to, p, end - 128 * i.value); });
        if (lane == 31) copy4_of<OFF + LAST, LAST>(to, p, end - LAST);
      }
    } else {
      // four bytes to an element, in the order of the lane's elements: planes
      // of pairs (ODD 1) or of words
      const T* p = row + channel<ODD>(c, lane, 0);
      const uint32_t to = s + (ODD == 1 ? 8 : 4) * lane;
      const int left = 4 * (C - channel<ODD>(c, lane, 0));
      each<V>([&](auto e) {
        constexpr int E = e.value, TO = OFF + (ODD == 1 ? 256 * (E / 2) + 4 * (E % 2) : 128 * E);
        constexpr int FROM = ODD == 1 ? 256 * (E / 2) + 4 * (E % 2) : 128 * E;
        if constexpr (FULL)
          copy4<TO, FROM>(to, p);
        else
          copy4_of<TO, FROM>(to, p, left - FROM);
      });
    }
  }
  // The arrived slot's elements.
  __device__ __forceinline__ static void arrived(const char* s, int lane, const T* row, int c, P2 (&v)[H]) {
    uint32_t w[BYTES / 4];
    raw(s, lane, row, c, w);
    unpack(w, v);
  }
  // The same as they are in memory, and their values.
  __device__ __forceinline__ static void arrived_raw(const char* s, int lane, const T* row, int c,
                                                     uint32_t (&w)[BYTES / 4]) {
    raw(s, lane, row, c, w);
  }
  __device__ __forceinline__ static void values(const uint32_t (&w)[BYTES / 4], P2 (&v)[H]) { unpack(w, v); }
  // The same, and kept as they are at `to`.
  __device__ __forceinline__ static void arrived_kept(const char* s, int lane, const T* row, int c, P2 (&v)[H],
                                                      char* to) {
    uint32_t w[BYTES / 4];
    raw(s, lane, row, c, w);
    unpack(w, v);
    if constexpr (BYTES == 16)
      *reinterpret_cast<uint4*>(to + lane * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    else
      *reinterpret_cast<uint2*>(to + lane * 8) = make_uint2(w[0], w[1]);
  }
  __device__ __forceinline__ static void kept(const char* s, int lane, P2 (&v)[H]) {
    uint32_t w[BYTES / 4];
    words(s + lane * BYTES, w);
    unpack(w, v);
  }
  // The lane's elements read directly, zeros past C.
  __device__ __forceinline__ static void load(const T* row, int c, int lane, int C, P2 (&v)[H]) {
    if constexpr (ODD != 0) {
#pragma unroll
      for (int i = 0; i < H; ++i) {
        const int a = channel<ODD>(c, lane, 2 * i), b = channel<ODD>(c, lane, 2 * i + 1);
        v[i] = pair(a < C ? value(row + a) : 0.0f, b < C ? value(row + b) : 0.0f);
      }
    } else {
      uint32_t w[BYTES / 4];
      words(reinterpret_cast<const char*>(row + min(c, C - V)), w);
      unpack(w, v);
    }
  }
  // Round and write v; store_rounded leaves in v what was written.
  __device__ __forceinline__ static void store(T* row, int c, int lane, int C, const P2 (&v)[H]) {
    uint32_t w[BYTES / 4];
    pack(v, w);
    put(row, c, lane, C, w);
  }
  __device__ __forceinline__ static void store_rounded(T* row, int c, int lane, int C, P2 (&v)[H]) {
    uint32_t w[BYTES / 4];
    pack(v, w);
    put(row, c, lane, C, w);
    if constexpr (sizeof(T) == 2) unpack(w, v);
  }

 private:
  __device__ __forceinline__ static float value(const T* p) {
    if constexpr (sizeof(T) == 4)
      return *p;
    else
      return b4::bf16lo(p->bits);
  }
  __device__ __forceinline__ static void raw(const char* s, int lane, const T* row, int c, uint32_t (&w)[BYTES / 4]) {
    if constexpr (SPLIT) {
      const uint32_t* q = reinterpret_cast<const uint32_t*>(s) + lane;
      const bool split = straddles(row, c) != 0;
      const uint32_t which = split ? 0x5432 : 0x3210;
#pragma unroll
      for (int i = 0; i < H; ++i) w[i] = __byte_perm(q[32 * i], split ? q[32 * i + 1] : 0, which);
    } else if constexpr (ODD == 1) {
#pragma unroll
      for (int i = 0; i < H; ++i) {
        const uint2 q = *reinterpret_cast<const uint2*>(s + 256 * i + 8 * lane);
        w[(2 * i) % (BYTES / 4)] = q.x, w[(2 * i + 1) % (BYTES / 4)] = q.y;
      }
    } else if constexpr (ODD == 2) {
#pragma unroll
      for (int e = 0; e < V; ++e) w[e % (BYTES / 4)] = *reinterpret_cast<const uint32_t*>(s + 128 * e + 4 * lane);
    } else {
      words(s + lane * BYTES, w);
    }
  }
  __device__ __forceinline__ static void words(const char* s, uint32_t (&w)[BYTES / 4]) {
    if constexpr (BYTES == 16) {
      const uint4 q = *reinterpret_cast<const uint4*>(s);
      w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
    } else {
      const uint2 q = *reinterpret_cast<const uint2*>(s);
      w[0] = q.x, w[1] = q.y;
    }
  }
  __device__ __forceinline__ static void unpack(const uint32_t (&w)[BYTES / 4], P2 (&v)[H]) {
#pragma unroll
    for (int i = 0; i < H; ++i)
      v[i] = sizeof(T) == 4 ? pair(__uint_as_float(w[(2 * i) % (BYTES / 4)]), __uint_as_float(w[(2 * i + 1) % (BYTES / 4)]))
                            : pair(b4::bf16lo(w[i]), b4::bf16hi(w[i]));
  }
  __device__ __forceinline__ static void pack(const P2 (&v)[H], uint32_t (&w)[BYTES / 4]) {
#pragma unroll
    for (int i = 0; i < H; ++i) {
      float lo, hi;
      split(v[i], lo, hi);
      if constexpr (sizeof(T) == 4)
        w[2 * i] = __float_as_uint(lo), w[2 * i + 1] = __float_as_uint(hi);
      else
        w[i] = b4::pack_bf16(lo, hi);
    }
  }
  __device__ __forceinline__ static void put(T* row, int c, int lane, int C, const uint32_t (&w)[BYTES / 4]) {
    if constexpr (ODD == 0) {
      if (c >= C) return;
      if constexpr (BYTES == 16)
        *reinterpret_cast<uint4*>(row + c) = make_uint4(w[0], w[1], w[2], w[3]);
      else
        *reinterpret_cast<uint2*>(row + c) = make_uint2(w[0], w[1]);
    } else if constexpr (SPLIT) {
      uint16_t* p = reinterpret_cast<uint16_t*>(row + c + 2 * lane);
      if (inside<V>(c, C) && !straddles(row, c)) {
#pragma unroll
        for (int i = 0; i < H; ++i) reinterpret_cast<uint32_t*>(p)[32 * i] = w[i];
      } else {
        const int left = C - c - 2 * lane;
#pragma unroll
        for (int i = 0; i < H; ++i) {
          if (64 * i < left) p[64 * i] = static_cast<uint16_t>(w[i]);
          if (64 * i + 1 < left) p[64 * i + 1] = static_cast<uint16_t>(w[i] >> 16);
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int at = channel<ODD>(c, lane, e);
        if (at < C) reinterpret_cast<uint32_t*>(row)[at] = w[e % (BYTES / 4)];
      }
    }
  }
};

// All of the thread's copies, or the oldest of DEPTH, have arrived; a slot has been read and may be
// copied to again.  A lane of an ODD kernel reads a word of its neighbour's,
// so there the warp waits for each other (all of its branches are the warp's).
template <int ODD>
__device__ __forceinline__ void slots_ready() {
  copy_wait_all();
  if constexpr (ODD != 0) __syncwarp();
}
template <int DEPTH, int ODD>
__device__ __forceinline__ void slot_ready() {
  copy_wait<DEPTH - 1>();
  if constexpr (ODD != 0) __syncwarp();
}
template <int ODD>
__device__ __forceinline__ void slot_read() {
  if constexpr (ODD != 0) __syncwarp();
}

// V floats that a thread keeps for itself, in its warp's planes of four.
template <int V>
constexpr int kFloats = 128 * V;  // bytes of a warp
template <int V>
__device__ __forceinline__ void keep(char* s, int lane, const P2 (&v)[V / 2]) {
#pragma unroll
  for (int i = 0; i < V / 4; ++i) put16(s + lane * 16 + i * 512, v[2 * i], v[2 * i + 1]);
}
template <int V>
__device__ __forceinline__ void kept(const char* s, int lane, P2 (&v)[V / 2]) {
#pragma unroll
  for (int i = 0; i < V / 4; ++i) get16(s + lane * 16 + i * 512, v[2 * i], v[2 * i + 1]);
}

// A lane's elements of a row of partial weight gradients (whole vectors, see
// pitch).
template <int V, int ODD>
struct PartRow {
  __device__ __forceinline__ static void put(float* row, int c, int lane, int C, const P2 (&v)[V / 2]) {
    if constexpr (ODD != 0) {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        float lo, hi;
        split(v[i], lo, hi);
        if (channel<ODD>(c, lane, 2 * i) < C) row[channel<ODD>(c, lane, 2 * i)] = lo;
        if (channel<ODD>(c, lane, 2 * i + 1) < C) row[channel<ODD>(c, lane, 2 * i + 1)] = hi;
      }
    } else if (c < C) {
#pragma unroll
      for (int i = 0; i < V / 4; ++i) put16(row + c + 4 * i, v[2 * i], v[2 * i + 1]);
    }
  }
  __device__ __forceinline__ static void get(const float* row, int c, int lane, int C, P2 (&v)[V / 2]) {
    if constexpr (ODD != 0) {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        const int a = channel<ODD>(c, lane, 2 * i), b = channel<ODD>(c, lane, 2 * i + 1);
        v[i] = pair(a < C ? row[a] : 0.0f, b < C ? row[b] : 0.0f);
      }
    } else {
#pragma unroll
      for (int i = 0; i < V / 4; ++i) get16(row + min(c, C - V) + 4 * i, v[2 * i], v[2 * i + 1]);
    }
  }
};

// Add a b to a thread's share of a weight gradient: in shared memory at s,
// or, where rows are too long for that, in the group's row of the partial
// sums (global memory that only this thread touches; such groups are CTAs).
template <int V, int ODD>
__device__ __forceinline__ void add_share(char* s, float* row, int c, int lane, int C, const P2 (&a)[V / 2],
                                          const P2 (&b)[V / 2]) {
  P2 d[V / 2];
  if (row == nullptr) {
    kept<V>(s, lane, d);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) d[i] = fma2(a[i], b[i], d[i]);
    keep<V>(s, lane, d);
  } else {
    PartRow<V, ODD>::get(row, c, lane, C, d);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) d[i] = fma2(a[i], b[i], d[i]);
    PartRow<V, ODD>::put(row, c, lane, C, d);
  }
}

// A pointer to fp32 or bf16 values, told apart at run time: coefficients and
// weights, which are few beside the rows.
struct Any {
  const void* p;
  int32_t bf16;
  __device__ __forceinline__ float at_far(int64_t i) const {
    return bf16 ? b4::bf16lo(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
  }
  __device__ __forceinline__ float at(int i) const {
    return bf16 ? b4::bf16lo(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
  }
  // A lane's elements of a block of a weight (as Row has them; from C on any
  // of its values), 1 where there is none.  W says what is known of it: nothing (0), or that it is there, on
  // 16 bytes, and fp32 (1) or bf16 (2).  Told apart at run time, both types'
  // loads, conversions and choices between them are issued every time.
  template <int V, int ODD, int W>
  __device__ __forceinline__ void load(int c, int lane, int C, P2 (&v)[V / 2]) const {
    if (W == 0 && p == nullptr) {
#pragma unroll
      for (int k = 0; k < V / 2; ++k) v[k] = twice(1.0f);
    } else if constexpr (ODD != 0) {
#pragma unroll
      for (int k = 0; k < V / 2; ++k) {
        const int a = channel<ODD>(c, lane, 2 * k), b = channel<ODD>(c, lane, 2 * k + 1);
        if constexpr (W == 1) {  // the nearest of its values where there is none
          const float* q = static_cast<const float*>(p);
          v[k] = pair(q[min(a, C - 1)], q[min(b, C - 1)]);
        } else {
          v[k] = pair(a < C ? at(a) : 0.0f, b < C ? at(b) : 0.0f);
        }
      }
    } else if (W == 2 || (W == 0 && bf16)) {
#pragma unroll
      for (int k = 0; k < V / 4; ++k) {
        const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + min(c, C - V) + 4 * k);
        v[2 * k] = pair(b4::bf16lo(q.x), b4::bf16hi(q.x)), v[2 * k + 1] = pair(b4::bf16lo(q.y), b4::bf16hi(q.y));
      }
    } else {
#pragma unroll
      for (int k = 0; k < V / 4; ++k) get16(static_cast<const float*>(p) + min(c, C - V) + 4 * k, v[2 * k], v[2 * k + 1]);
    }
  }
};

// What W above a pass's weights (null where it has no such weight) allow: the
// type that both have, 0 where they differ, are missing or off 16 bytes.
struct Weights {
  static int kind(const Any& w) {
    return w.p == nullptr || (reinterpret_cast<uintptr_t>(w.p) & 15) != 0 ? 0 : w.bf16 ? 2 : 1;
  }
  static int kind(const Any& w, const Any& wn) { return kind(w) == kind(wn) ? kind(w) : 0; }
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
  uint32_t T;  // below 2^31, as are the strides: a row's offset is one 32 x 32 -> 64 bit product
  int32_t S, C;
  int32_t G;            // threads of a group
  int32_t group_bytes;  // shared memory of a group
  int32_t warp_bytes;   // and of a warp, within it
  int32_t act, norm;
  float eps, eps_next, scale;
  const void *x, *y, *gate, *dout, *dh, *dres, *out_in;
  Any P, a, b, w, wn;
  uint32_t x_ts, y_ts, gate_ts, P_ts, a_ts, b_ts, dout_ts, dh_ts, dres_ts, out_ts;
  uint32_t x_ss, dout_ss, dres_ss, out_ss;
  void *h, *out, *dx, *dy, *dgate, *dP, *da, *db;
  float *dw, *dwn;  // partial weight gradients [CTAs, pitch(C)]
  int32_t direct;   // rows too long to keep all of: the shares lie there from
                    // the start, and y and dh are read a second time
};

// Row t of an array with `stride` elements between its rows.
template <class T>
__device__ __forceinline__ const T* at_row(const void* p, uint32_t t, uint32_t stride) {
  return static_cast<const T*>(p) + uint64_t(t) * stride;
}

// The channel that a thread of a group has in its first block (ODD: its
// warp's first channel there).
template <int V, int ODD>
__device__ __forceinline__ int first_channel(int l) {
  return ODD != 0 ? l / 32 * 32 * V : l * V;
}

// Floats of a row of partial weight gradients: whole vectors.
__host__ __device__ constexpr int pitch(int C) { return (C + 7) / 8 * 8; }

// Write a CTA's sums of its NG groups' shares to its row (group 0's threads).
// `first`: where the first item of this thread's warp is in group 0.
template <int V, int ODD>
__device__ __forceinline__ void sum_shares(const char* first, const Params& p, int NG, int item, float* row) {
  if (threadIdx.x >= p.G) return;
  const int lane = threadIdx.x & 31;
  for (int c = first_channel<V, ODD>(threadIdx.x); c < p.C; c += p.G * V, first += item) {
    P2 d[V / 2];
    kept<V>(first, lane, d);
    for (int g = 1; g < NG; ++g) {
      P2 more[V / 2];
      kept<V>(first + g * p.group_bytes, lane, more);
#pragma unroll
      for (int j = 0; j < V / 2; ++j) d[j] = add2(d[j], more[j]);
    }
    PartRow<V, ODD>::put(row, c, lane, p.C, d);
  }
}

// ---------------------------------------------------------------------------
// A token's coefficients, fetched one token ahead: lane l of every warp loads
// value l (and l + 32, ...), and the warp spreads them through a few floats
// of shared memory of its own, each twice, to be read as pairs.  Order: P
// [SP, SP] (TP: transposed), then b [SP], then a [SP]; streams that are not
// there have zeros, absent arrays ones.
// ---------------------------------------------------------------------------
template <int SP, bool P, bool B, bool A, bool TP = false>
struct Coefficients {
  static constexpr int NP = P ? SP * SP : 0, NB = NP + (B ? SP : 0), N = NB + (A ? SP : 0);
  static constexpr int CH = (N + 31) / 32;
  static constexpr int FLOATS = (2 * N + 3) / 4 * 4;
  // what this lane fetches is the same for every token: an address (or none,
  // and then a constant), a stride in bytes, a type
  const char* src[CH];
  uint32_t stride[CH];
  bool bf16[CH];
  float next[CH];
  __device__ __forceinline__ void init(const Params& p, int lane) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int n = c * 32 + lane;
      src[c] = nullptr, stride[c] = 0, bf16[c] = false, next[c] = 0.0f;
      const Any* from = nullptr;
      int at = 0;
      if (n < NP) {
        const int i = TP ? n % SP : n / SP, j = TP ? n / SP : n % SP;
        if (i < p.S && j < p.S) from = p.P.p ? &p.P : nullptr, at = i * p.S + j, stride[c] = p.P_ts;
      } else if (n < NB) {
        if (n - NP < p.S) from = &p.b, at = n - NP, stride[c] = p.b_ts;
      } else if (n < N) {
        if (n - NB < p.S) from = &p.a, at = n - NB, stride[c] = p.a_ts;
      }
      if (from != nullptr) {
        bf16[c] = from->bf16 != 0;
        const int size = bf16[c] ? 2 : 4;
        next[c] = 1.0f;
        if (from->p != nullptr) src[c] = static_cast<const char*>(from->p) + at * size, stride[c] *= size;
      }
    }
  }
  __device__ __forceinline__ void fetch(uint32_t t) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (src[c] == nullptr) continue;
      const char* q = src[c] + uint64_t(t) * stride[c];
      next[c] = bf16[c] ? b4::bf16lo(*reinterpret_cast<const uint16_t*>(q)) : *reinterpret_cast<const float*>(q);
    }
  }
  // Put the fetched values where the warp reads them.
  __device__ __forceinline__ void spread(float* s, int lane) const {
    __syncwarp();  // the last token's readers are done
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (c * 32 + lane < N) reinterpret_cast<P2*>(s)[c * 32 + lane] = twice(next[c]);
    __syncwarp();
  }
  // SP of them, from place `from` on.
  __device__ __forceinline__ static void read(const float* s, int from, P2 (&v)[SP]) {
    if constexpr (SP >= 2) {
#pragma unroll
      for (int i = 0; i < SP; i += 2) get16(s + 2 * (from + i), v[i], v[i + 1]);
    } else {
      v[0] = *reinterpret_cast<const P2*>(s + 2 * from);
    }
  }
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
// has value l + 32 c in total[c].  `red` holds [2][R][20] floats of the group
// (16 warps at most; 20 keeps the reads of a warp conflict-free), zeros where
// there are no warps; `turn` alternates between calls, so that one barrier a
// call is enough (a warp can be one call ahead of another, not two).
template <int R>
struct GroupSum {
  static constexpr int CH = (R + 31) / 32;
  static constexpr __host__ __device__ int floats(int G) { return G == 32 ? 0 : 2 * R * 20; }
  __device__ __forceinline__ static void clear(float* red, int G, int l) {
    for (int i = l; i < floats(G); i += G) red[i] = 0.0f;
  }
  __device__ __forceinline__ static void run(const float (&v)[R], float (&total)[CH], float* red,
                                             int& turn, int G, int group, int lane, int warp) {
    sums<0>(v, total, lane);
    if (G == 32) return;
    float* r = red + turn;
    turn = R * 20 - turn;
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (c * 32 + lane < R) r[(c * 32 + lane) * 20 + warp] = total[c];
    group_sync(G, group);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float s = 0.0f;
      if (c * 32 + lane < R) {
        const float4* q = reinterpret_cast<const float4*>(r + (c * 32 + lane) * 20);
        for (int w = 0; w < G; w += 128) {
          const float4 x = *q++;
          s += (x.x + x.y) + (x.z + x.w);
        }
      }
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

// The sums that enter's gradient takes over a row: <G, x_s>, then <u, x_s>,
// then <G, u> and <u, u>.  Those are also sum_s a_s <G, x_s> and sum_s a_s
// <u, x_s>, but where the streams nearly cancel in u that keeps the rounding
// of the streams' sums: two streams alike to 1/1000 with the coefficients 1 and
// -0.999 leave <u, u> an error of 1e-4, and 1e-7 summed from u.  Of one stream,
// u = a x, nothing cancels.
__host__ __device__ constexpr int next_sums(int SP) { return SP > 1 ? 2 * SP + 2 : 2; }
template <int SP>
__device__ __forceinline__ void sums_of_u(const float (&total)[1], float a, float& gu, float& uu) {
  if constexpr (SP > 1)
    gu = of_total(total, 2 * SP), uu = of_total(total, 2 * SP + 1);
  else
    gu = a * of_total(total, 0), uu = a * of_total(total, 1);
}

// ---------------------------------------------------------------------------
// Gates: value and slope of act(g).  e = exp(-|g|) keeps 1 - sigmoid exact
// to fp32 on both sides and never overflows.  EXACT (gates of fp32 rows): expf,
// whose error is an ulp for any g.  The fast exponential's grows with |g| to 88
// 2^-24 where sigmoid is still a normal number: nothing beside the half step
// of 2^-9 by which bf16 rows are off, and fewer instructions.
// ---------------------------------------------------------------------------
template <bool EXACT>
__device__ __forceinline__ void gate_of(int act, float g, float& value, float& slope) {
  const float e = EXACT ? expf(-fabsf(g)) : __expf(-fabsf(g));
  const float inv = __fdividef(1.0f, 1.0f + e);
  const float s = g >= 0.0f ? inv : e * inv;
  const float rest = g >= 0.0f ? e * inv : inv;  // 1 - s
  // NaN: both comparisons are false and e is NaN, so s and rest are NaN
  if (act == HCB_ACT_SIGMOID)
    value = s, slope = s * rest;
  else
    value = g * s, slope = s * (1.0f + g * rest);
}
// The values of V gates, elements of rows of T, replace them; their slopes, if wanted.
template <class T, int V, bool SLOPE>
__device__ __forceinline__ void gates(int act, P2 (&g)[V / 2], P2 (&slope)[V / 2]) {
  constexpr bool EXACT = sizeof(T) == 4;
  if (act == HCB_ACT_LINEAR) {
    if constexpr (SLOPE) {
#pragma unroll
      for (int j = 0; j < V / 2; ++j) slope[j] = twice(1.0f);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < V / 2; ++j) {
    float lo, hi, slo, shi;
    split(g[j], lo, hi);
    gate_of<EXACT>(act, lo, lo, slo);
    gate_of<EXACT>(act, hi, hi, shi);
    g[j] = pair(lo, hi);
    if constexpr (SLOPE) slope[j] = pair(slo, shi);
  }
}

// ---------------------------------------------------------------------------
// Launch shape
// ---------------------------------------------------------------------------
constexpr size_t kSmemMax = 232448;  // shared memory of a CTA

struct Shape {
  int G, NG;
};

int sms();  // SMs of the current device (hcb_api.cu)


inline int items(int C, int V, int G) { return (C + V * G - 1) / (V * G); }  // K

// Threads of a group: `per` vectors of a row to a thread where the tokens
// fill the GPU, one where they do not (a longer group shortens a token's
// path).
inline Shape shape_of(int64_t T, int C, int V, int per, int max_group) {
  const int vecs = (C + V - 1) / V;
  if (T < sms()) per = 1;
  const int K = std::max((vecs + max_group - 1) / max_group, std::min(per, (vecs + 31) / 32));
  const int G = ((vecs + K - 1) / K + 31) / 32 * 32;
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
                           static_cast<int>(kSmemMax) - static_cast<int>(fa.sharedSizeBytes));
  if (e != cudaSuccess) return e;
  int occ = 0;
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, KERN, threads, smem);
  if (e != cudaSuccess) return e;
  *out = std::max(1, std::min(occ, 255));
  if (dev < 64) last[dev].store(key | static_cast<uint64_t>(*out), std::memory_order_release);
  return cudaSuccess;
}

// What a kernel's groups need: bytes of a warp in its slots and in a kept
// item, and of a group beside that.
struct Need {
  int ring, item, group;
  int of_warp(int C, int V, int G) const { return ring + items(C, V, G) * item; }
  size_t bytes(int C, int V, int G) const { return (size_t(G / 32) * of_warp(C, V, G) + group + 15) / 16 * 16; }
};

// The shape of a pass: need(G, direct) is a Need; a shape that does not fit is
// shrunk, and made direct (Params) where no group of 128 threads would do
// otherwise.  Fills in what a kernel has to know of it.
template <class N>
Shape plan(Params& p, Shape sh, int V, N&& need) {
  auto bytes = [&] { return need(sh.G, p.direct).bytes(p.C, V, sh.G); };
  p.direct = 0;
  while (bytes() * sh.NG > kSmemMax && sh.NG > 1) sh.NG /= 2;
  while (bytes() > kSmemMax && sh.G > 128) sh.G = (sh.G / 2 + 31) / 32 * 32;
  if (bytes() > kSmemMax) {
    p.direct = 1;
    while (bytes() > kSmemMax && sh.G > 32) sh.G = (sh.G / 2 + 31) / 32 * 32;
  }
  p.G = sh.G, p.group_bytes = static_cast<int32_t>(bytes());
  p.warp_bytes = need(sh.G, p.direct).of_warp(p.C, V, sh.G);
  return sh;
}

// Persistent launch of KERN, at most max_grid CTAs (the grid goes to *grid).
template <auto KERN>
cudaError_t launch(const Params& p, Shape sh, int max_grid, int* grid, cudaStream_t s) {
  const size_t smem = size_t(p.group_bytes) * sh.NG;
  int occ = 0;
  const cudaError_t e = resident<KERN>(sh.G * sh.NG, smem, &occ);
  if (e != cudaSuccess) return e;
  const int64_t want = (int64_t(p.T) + sh.NG - 1) / sh.NG;
  *grid = static_cast<int>(std::min<int64_t>(want, std::min<int64_t>(max_grid, int64_t(sms()) * occ)));
  KERN<<<*grid, sh.G * sh.NG, smem, s>>>(p);
  return cudaGetLastError();
}

// Runs f(FULL) for a block of a row's copies: FULL (a true_type) where rows
// allow vectors or the block is inside its row, so that all rows of an item
// share one branch.
template <int V, int ODD, class F>
__device__ __forceinline__ void by_block(int c, int C, F&& f) {
  if (ODD == 0 || inside<V>(c, C))
    f(std::true_type());
  else
    f(std::false_type());
}

// Call F.operator()<SP, EXACT, TX, TY, V, ODD>() for the streams (SP of them:
// 1, 2, 4 or 8; fewer, !EXACT, are rounded up, and the missing ones count as
// zeros), the row types and alignment.  An EXACT kernel takes it further that
// a mixing matrix comes with more than one stream and only with them, and
// that the pass is not direct; a launcher takes the other kernel where that
// does not hold.  V elements are 16 bytes of the wider
// row type (8 bytes of bf16 at 8 streams, for the registers).
template <int SP, bool EXACT, class F>
cudaError_t by_type(int x_bf16, int y_bf16, bool vec, F&& f) {
  constexpr int VB = SP == 8 ? 4 : 8;
  if (x_bf16)
    return vec ? f.template operator()<SP, EXACT, bf16_t, bf16_t, VB, 0>()
               : f.template operator()<SP, EXACT, bf16_t, bf16_t, VB, 1>();
  if (y_bf16)
    return vec ? f.template operator()<SP, EXACT, float, bf16_t, 4, 0>()
               : f.template operator()<SP, EXACT, float, bf16_t, 4, 1>();
  return vec ? f.template operator()<SP, EXACT, float, float, 4, 0>()
             : f.template operator()<SP, EXACT, float, float, 4, 2>();
}
template <class F>
cudaError_t by_streams(int S, int x_bf16, int y_bf16, bool vec, F&& f) {
  switch (S) {
    case 1: return by_type<1, true>(x_bf16, y_bf16, vec, f);
    case 2: return by_type<2, true>(x_bf16, y_bf16, vec, f);
    case 3: return by_type<4, false>(x_bf16, y_bf16, vec, f);
    case 4: return by_type<4, true>(x_bf16, y_bf16, vec, f);
    case 8: return by_type<8, true>(x_bf16, y_bf16, vec, f);
    default: return by_type<8, false>(x_bf16, y_bf16, vec, f);
  }
}

// The pass launchers, one translation unit each: enqueue on `s`.
cudaError_t enter_forward(const Params& p, int x_bf16, int y_bf16, bool vec, cudaStream_t s);
cudaError_t enter_backward(const Params& p, int x_bf16, int y_bf16, bool vec, int* rows, cudaStream_t s);
cudaError_t leave_forward(const Params& p, int x_bf16, int y_bf16, bool vec, cudaStream_t s);
cudaError_t leave_backward(const Params& p, int x_bf16, int y_bf16, bool vec, int* rows, cudaStream_t s);
cudaError_t leave_enter_backward(const Params& p, int x_bf16, int y_bf16, bool vec, int* rows, cudaStream_t s);
// One stream without a mixing matrix, rows of one item to a thread
// (hcb_residual.cu); false where a pass is not that.
bool residual_forward(const Params& p, int x_bf16, int y_bf16, bool vec, cudaStream_t s, cudaError_t* e);
bool residual_backward(const Params& p, int x_bf16, int y_bf16, bool vec, int* rows, cudaStream_t s, cudaError_t* e);

}  // namespace hcb
