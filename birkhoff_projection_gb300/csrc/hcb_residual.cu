// hcb_residual.cu -- leave and leave_enter and their gradients for one stream
// without a mixing matrix (the residual of an ordinary network), where a row
// is no longer than one vector to each of 512 threads.
//
// A thread then has the same V channels of every token, and everything that a
// row's later passes need stays in its registers: the rows themselves, both
// weights, and its shares of their gradients.  In hcb_leave_bwd.cuh that all
// goes through shared memory, 76 bytes to a channel of 12 bytes in memory,
// and the kernel was bound by that (255 us at 16384 x 4096 bf16, against a
// floor of 119; 63% of the shared-memory pipe's rate).  A barrier leaves a
// CTA of 512 threads idle, so it takes TOKENS tokens at a time: their sums
// share the barriers.
#include "hcb_common.cuh"

namespace hcb {

template <class TX, class TY, int V, int ODD, bool NEXT, bool GATED>
struct Residual {
  using RX = Row<TX, V, ODD>;
  using RY = Row<TY, V, ODD>;
  // a gate's slopes take the registers of a second token (8192 x 2048 bf16
  // with a gate: 63 us with one, 82 with two; 16384 x 4096 without: 193, 151)
  static constexpr int TOKENS = GATED && V == 8 ? 1 : 2;
  using Sum = GroupSum<2 * TOKENS>;
  // a token's slots: NEXT's stored result and dh, then dout, y and the gate
  static constexpr int DH = RX::SLOT, REST = NEXT ? DH + RY::SLOT : 0, Y = REST + RX::SLOT, GATE = Y + RY::SLOT;
  static constexpr int SLOT = GATED ? GATE + RY::SLOT : GATE;
};

template <class TX, class TY, int V, int ODD, bool NEXT, bool GATED, int W>
__global__ void __launch_bounds__(kMaxGroup, 1) residual_backward_kernel(const Params p) {
  using E = Residual<TX, TY, V, ODD, NEXT, GATED>;
  using RX = typename E::RX;
  using RY = typename E::RY;
  using Sum = typename E::Sum;
  constexpr int H = V / 2, N = E::TOKENS, SLOT = E::SLOT;
  extern __shared__ __align__(16) char smem[];
  const int G = p.G, NG = blockDim.x / G, group = threadIdx.x / G, l = threadIdx.x % G;
  const int lane = threadIdx.x & 31, warp = l / 32, C = p.C, c = first_channel<V, ODD>(l);
  char* of_group = smem + group * p.group_bytes;
  char* ring = of_group + warp * p.warp_bytes;
  float* red = reinterpret_cast<float*>(of_group + G / 32 * p.warp_bytes);
  float* red_next = red + Sum::floats(G);
  Sum::clear(red, G, l);
  if constexpr (NEXT) Sum::clear(red_next, G, l);
  let_next_launch();
  group_sync(G, group);
  int turn = 0, turn_next = 0;
  const float inv_c = 1.0f / static_cast<float>(C);
  const uint32_t step = gridDim.x * NG;

  auto copy_next = [&](uint32_t t, char* slot) {
    const uint32_t to = b4::smem_addr(slot);
    by_block<V, ODD>(c, C, [&](auto full) {
      constexpr bool FULL = decltype(full)::value;
      RX::template copy<FULL, 0>(to, lane, at_row<TX>(p.out_in, t, p.out_ts), c, C);
      RY::template copy<FULL, E::DH>(to, lane, at_row<TY>(p.dh, t, p.dh_ts), c, C);
    });
  };
  auto copy_rest = [&](uint32_t t, char* slot) {
    const uint32_t to = b4::smem_addr(slot);
    by_block<V, ODD>(c, C, [&](auto full) {
      constexpr bool FULL = decltype(full)::value;
      RX::template copy<FULL, E::REST>(to, lane, at_row<TX>(p.dout, t, p.dout_ts), c, C);
      RY::template copy<FULL, E::Y>(to, lane, at_row<TY>(p.y, t, p.y_ts), c, C);
      if (GATED) RY::template copy<FULL, E::GATE>(to, lane, at_row<TY>(p.gate, t, p.gate_ts), c, C);
    });
  };
  uint32_t t0 = blockIdx.x * NG + group;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const uint32_t t = t0 + n * step;
    if (t >= p.T) continue;
    if (NEXT) copy_next(t, ring + n * SLOT);
    copy_rest(t, ring + n * SLOT);
  }
  P2 w[H], wn[H], dw[H] = {}, dwn[H] = {};
  p.w.load<V, ODD, W>(c, lane, C, w);
  if (NEXT) p.wn.load<V, ODD, W>(c, lane, C, wn);

#pragma unroll 1
  for (; t0 < p.T; t0 += N * step) {
    slots_ready<ODD>();
    uint32_t o_raw[NEXT ? N : 1][RX::BYTES / 4], h_raw[NEXT ? N : 1][RY::BYTES / 4];
    float a[N], r_next[N], k_next[N];
    if constexpr (NEXT) {
      float sum[2 * N];
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const uint32_t t = t0 + n * step;
        sum[2 * n] = sum[2 * n + 1] = 0.0f;
        a[n] = 0.0f;
        if (t >= p.T) continue;
        a[n] = p.a.p ? p.a.at_far(int64_t(t) * p.a_ts) : 1.0f;
        P2 o[H], h[H], go = 0, oo = 0;
        RX::arrived_raw(ring + n * SLOT, lane, at_row<TX>(p.out_in, t, p.out_ts), c, o_raw[n]);
        RY::arrived_raw(ring + n * SLOT + E::DH, lane, at_row<TY>(p.dh, t, p.dh_ts), c, h_raw[n]);
        RX::values(o_raw[n], o);
        RY::values(h_raw[n], h);
#pragma unroll
        for (int j = 0; j < H; ++j) {
          go = fma2(mul2(h[j], wn[j]), o[j], go);
          oo = fma2(o[j], o[j], oo);
        }
        sum[2 * n] = both(go), sum[2 * n + 1] = both(oo);
      }
      slot_read<ODD>();
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const uint32_t t = t0 + (N + n) * step;
        if (t < p.T) copy_next(t, ring + n * SLOT);
      }
      float total[1];
      Sum::run(sum, total, red_next, turn_next, G, group, lane, warp);
#pragma unroll
      for (int n = 0; n < N; ++n) {
        // u = a o
        const float go = of_total(total, 2 * n), oo = of_total(total, 2 * n + 1);
        r_next[n] = rsqrtf(a[n] * a[n] * oo * inv_c + p.eps_next);
        k_next[n] = a[n] * go * inv_c * r_next[n] * r_next[n];
        const uint32_t t = t0 + n * step;
        if (p.da && l == 0 && t < p.T) put_any(p.da, p.a.bf16, t, r_next[n] * (go - k_next[n] * a[n] * oo));
      }
    }
    P2 dv[N][H], slope[GATED ? N : 1][H];
    uint32_t y_raw[N][RY::BYTES / 4];
    float b[N], sum[2 * N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const uint32_t t = t0 + n * step;
      sum[2 * n] = sum[2 * n + 1] = 0.0f;
      b[n] = 0.0f;
      if (t >= p.T) continue;
      b[n] = p.b.p ? p.b.at_far(int64_t(t) * p.b_ts) : 1.0f;
      P2 D[H], e[H], yy = 0, de = 0;
      RX::arrived(ring + n * SLOT + E::REST, lane, at_row<TX>(p.dout, t, p.dout_ts), c, D);
      if constexpr (NEXT) {
        // D = dout + a du, du = r (wn dh - k u)
        P2 o[H], h[H];
        RX::values(o_raw[n], o);
        RY::values(h_raw[n], h);
        const P2 ra = twice(r_next[n] * a[n]), minus_k = twice(-k_next[n] * a[n]);
#pragma unroll
        for (int j = 0; j < H; ++j) {
          const P2 ru = mul2(ra, o[j]);
          dwn[j] = fma2(h[j], ru, dwn[j]);
          D[j] = fma2(ra, mul2(h[j], wn[j]), fma2(minus_k, ru, D[j]));
        }
      }
      if (p.dx) RX::store(static_cast<TX*>(p.dx) + uint64_t(t) * uint32_t(C), c, lane, C, D);
      RY::arrived_raw(ring + n * SLOT + E::Y, lane, at_row<TY>(p.y, t, p.y_ts), c, y_raw[n]);
      RY::values(y_raw[n], e);
      const P2 b2 = twice(b[n]);
#pragma unroll
      for (int j = 0; j < H; ++j) {
        yy = fma2(e[j], e[j], yy);
        e[j] = mul2(e[j], w[j]);
        dv[n][j] = mul2(b2, D[j]);
      }
      if constexpr (GATED) {
        P2 g[H];
        RY::arrived(ring + n * SLOT + E::GATE, lane, at_row<TY>(p.gate, t, p.gate_ts), c, g);
        gates<TY, V, true>(p.act, g, slope[n]);
#pragma unroll
        for (int j = 0; j < H; ++j) {
          slope[n][j] = mul2(slope[n][j], mul2(e[j], dv[n][j]));
          e[j] = mul2(e[j], g[j]);
          dv[n][j] = mul2(dv[n][j], g[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < H; ++j) de = fma2(D[j], e[j], de);
      sum[2 * n] = both(de), sum[2 * n + 1] = both(yy);
    }
    slot_read<ODD>();
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const uint32_t t = t0 + (N + n) * step;
      if (t < p.T) copy_rest(t, ring + n * SLOT);
    }
    float total[1];
    Sum::run(sum, total, red, turn, G, group, lane, warp);
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const uint32_t t = t0 + n * step;
      const float de = of_total(total, 2 * n), yy = of_total(total, 2 * n + 1);
      if (t >= p.T) continue;
      const float rho = p.norm ? rsqrtf(yy * inv_c + p.eps) : 1.0f, sr = p.scale * rho;
      const P2 sr2 = twice(sr), minus_k = twice(p.norm ? -sr * (b[n] * de) * inv_c * rho * rho : 0.0f);
      if (p.db && l == 0) put_any(p.db, p.b.bf16, t, sr * de);
      P2 y[H];
      RY::values(y_raw[n], y);
#pragma unroll
      for (int j = 0; j < H; ++j) {
        dv[n][j] = mul2(dv[n][j], sr2);
        dw[j] = fma2(dv[n][j], y[j], dw[j]);
        y[j] = fma2(dv[n][j], w[j], mul2(minus_k, y[j]));
      }
      if (p.dy) RY::store(static_cast<TY*>(p.dy) + uint64_t(t) * uint32_t(C), c, lane, C, y);
      if constexpr (GATED) {
        if (p.dgate) {
#pragma unroll
          for (int j = 0; j < H; ++j) slope[n][j] = mul2(slope[n][j], sr2);
          RY::store(static_cast<TY*>(p.dgate) + uint64_t(t) * uint32_t(C), c, lane, C, slope[n]);
        }
      }
    }
  }
  copy_wait_all();
  // the shares of a CTA's groups, one after the other through shared memory
  if (p.dw == nullptr && (!NEXT || p.dwn == nullptr)) return;
  __syncthreads();
  const int64_t row = int64_t(blockIdx.x) * pitch(C);
  if (NG > 1) {
    keep<V>(ring, lane, dw);
    if (NEXT) keep<V>(ring + kFloats<V>, lane, dwn);
    __syncthreads();
    if (group > 0) return;
    for (int g = 1; g < NG; ++g) {
      P2 more[H];
      kept<V>(ring + g * p.group_bytes, lane, more);
#pragma unroll
      for (int j = 0; j < H; ++j) dw[j] = add2(dw[j], more[j]);
      if (NEXT) {
        kept<V>(ring + g * p.group_bytes + kFloats<V>, lane, more);
#pragma unroll
        for (int j = 0; j < H; ++j) dwn[j] = add2(dwn[j], more[j]);
      }
    }
  }
  if (p.dw) PartRow<V, ODD>::put(p.dw + row, c, lane, C, dw);
  if (NEXT && p.dwn) PartRow<V, ODD>::put(p.dwn + row, c, lane, C, dwn);
}

// leave and leave_enter likewise: the row, w act y and the result stay in
// registers between the sums.  leave_enter at 16384 x 4096 bf16, tokens at a
// time x CTAs on an SM: 1x2 103 us, 2x1 95, 2x2 105 (spilt), 3x1 86, 4x1 82.6
// (6.5 TB/s, 96% of the copy's rate; 117 through shared memory in
// hcb_leave.cu); fp32 vectors are half as many channels to a thread: 8192 x
// 2048 with bf16 y and a gate 2x2 42 us, 4x1 44, 2x1 50.  Odd rows with bf16
// ones among them are bound by their copies of single words and gain nothing
// (4001 x 4001 bf16 44 us there, 50 here; 4096 x 1431 fp32 27 and 22.6).
template <class TX, class TY, int V, int ODD, bool GATED>
struct ResidualForward {
  using RX = Row<TX, V, ODD>;
  using RY = Row<TY, V, ODD>;
  // tokens at a time, and CTAs that the registers have to leave room for
  static constexpr int TOKENS = V == 8 ? 4 : 2, MINB = V == 8 ? 1 : 2;
  using Sum = GroupSum<TOKENS>;
  static constexpr int Y = RX::SLOT, GATE = Y + RY::SLOT, SLOT = GATED ? GATE + RY::SLOT : GATE;
};

template <class TX, class TY, int V, int ODD, bool NEXT, bool GATED, int W>
__global__ void __launch_bounds__(kMaxGroup, ResidualForward<TX, TY, V, ODD, GATED>::MINB) residual_kernel(const Params p) {
  using E = ResidualForward<TX, TY, V, ODD, GATED>;
  using RX = typename E::RX;
  using RY = typename E::RY;
  using Sum = typename E::Sum;
  constexpr int H = V / 2, N = E::TOKENS, SLOT = E::SLOT;
  extern __shared__ __align__(16) char smem[];
  const int G = p.G, NG = blockDim.x / G, group = threadIdx.x / G, l = threadIdx.x % G;
  const int lane = threadIdx.x & 31, warp = l / 32, C = p.C, c = first_channel<V, ODD>(l);
  char* of_group = smem + group * p.group_bytes;
  char* ring = of_group + warp * p.warp_bytes;
  float* red = reinterpret_cast<float*>(of_group + G / 32 * p.warp_bytes);
  float* red_next = red + Sum::floats(G);
  Sum::clear(red, G, l);
  if constexpr (NEXT) Sum::clear(red_next, G, l);
  group_sync(G, group);
  int turn = 0, turn_next = 0;
  const float inv_c = 1.0f / static_cast<float>(C);
  const uint32_t step = gridDim.x * NG;

  auto copy = [&](uint32_t t, char* slot) {
    const uint32_t to = b4::smem_addr(slot);
    by_block<V, ODD>(c, C, [&](auto full) {
      constexpr bool FULL = decltype(full)::value;
      RX::template copy<FULL, 0>(to, lane, at_row<TX>(p.x, t, p.x_ts), c, C);
      RY::template copy<FULL, E::Y>(to, lane, at_row<TY>(p.y, t, p.y_ts), c, C);
      if (GATED) RY::template copy<FULL, E::GATE>(to, lane, at_row<TY>(p.gate, t, p.gate_ts), c, C);
    });
  };
  uint32_t t0 = blockIdx.x * NG + group;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const uint32_t t = t0 + n * step;
    if (t < p.T) copy(t, ring + n * SLOT);
  }
  P2 w[H], wn[H];
  p.w.load<V, ODD, W>(c, lane, C, w);
  if (NEXT) p.wn.load<V, ODD, W>(c, lane, C, wn);

#pragma unroll 1
  for (; t0 < p.T; t0 += N * step) {
    slots_ready<ODD>();
    uint32_t x_raw[N][RX::BYTES / 4];
    P2 v[N][H];
    float a[N], b[N], sum[N], total[1];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const uint32_t t = t0 + n * step;
      sum[n] = a[n] = b[n] = 0.0f;
      if (t >= p.T) continue;
      b[n] = p.b.p ? p.b.at_far(int64_t(t) * p.b_ts) : 1.0f;
      if (NEXT) a[n] = p.a.p ? p.a.at_far(int64_t(t) * p.a_ts) : 1.0f;
      RX::arrived_raw(ring + n * SLOT, lane, at_row<TX>(p.x, t, p.x_ts), c, x_raw[n]);
      RY::arrived(ring + n * SLOT + E::Y, lane, at_row<TY>(p.y, t, p.y_ts), c, v[n]);
      P2 yy = 0;
#pragma unroll
      for (int j = 0; j < H; ++j) {
        yy = fma2(v[n][j], v[n][j], yy);
        v[n][j] = mul2(v[n][j], w[j]);
      }
      sum[n] = both(yy);
      if constexpr (GATED) {
        P2 g[H], none[H];
        RY::arrived(ring + n * SLOT + E::GATE, lane, at_row<TY>(p.gate, t, p.gate_ts), c, g);
        gates<TY, V, false>(p.act, g, none);
#pragma unroll
        for (int j = 0; j < H; ++j) v[n][j] = mul2(v[n][j], g[j]);
      }
    }
    slot_read<ODD>();
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const uint32_t t = t0 + (N + n) * step;
      if (t < p.T) copy(t, ring + n * SLOT);
    }
    if (p.norm) Sum::run(sum, total, red, turn, G, group, lane, warp);
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const uint32_t t = t0 + n * step;
      const float rho = p.norm ? p.scale * rsqrtf(of_total(total, n) * inv_c + p.eps) : p.scale;
      sum[n] = 0.0f;
      if (t >= p.T) continue;
      TX* out = static_cast<TX*>(p.out) + uint64_t(t) * uint32_t(C);
      const P2 b2 = twice(b[n] * rho);
      P2 x[H];
      RX::values(x_raw[n], x);
#pragma unroll
      for (int j = 0; j < H; ++j) v[n][j] = fma2(b2, v[n][j], x[j]);
      if constexpr (NEXT) {
        P2 uu = 0;
        const P2 a2 = twice(a[n]);
        RX::store_rounded(out, c, lane, C, v[n]);
#pragma unroll
        for (int j = 0; j < H; ++j) {
          v[n][j] = mul2(a2, v[n][j]);
          uu = fma2(v[n][j], v[n][j], uu);
        }
        sum[n] = both(uu);
      } else {
        RX::store(out, c, lane, C, v[n]);
      }
    }
    if constexpr (NEXT) {
      Sum::run(sum, total, red_next, turn_next, G, group, lane, warp);
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const uint32_t t = t0 + n * step;
        const P2 r = twice(rsqrtf(of_total(total, n) * inv_c + p.eps_next));
        if (t >= p.T) continue;
#pragma unroll
        for (int j = 0; j < H; ++j) v[n][j] = mul2(v[n][j], mul2(r, wn[j]));
        RY::store(static_cast<TY*>(p.h) + uint64_t(t) * uint32_t(C), c, lane, C, v[n]);
      }
    }
  }
  copy_wait_all();
}

namespace {

template <class TX, class TY, int V, int ODD, bool NEXT, bool GATED>
bool forward(const Params& p, cudaStream_t s, cudaError_t* e) {
  using E = ResidualForward<TX, TY, V, ODD, GATED>;
  const int w = Weights::kind(p.w, NEXT ? p.wn : p.w);
  if (w == 0 || (w == 2 && ODD) || (p.C + V - 1) / V > kMaxGroup) return false;
  Params q = p;
  const Shape sh = plan(q, shape_of(p.T, p.C, V, 1, kMaxGroup), V,
                        [&](int G, int) { return Need{E::TOKENS * E::SLOT, 0, 4 * E::Sum::floats(G) * (NEXT ? 2 : 1)}; });
  if (q.direct || items(p.C, V, sh.G) != 1) return false;
  int grid;
  *e = w == 1 ? launch<residual_kernel<TX, TY, V, ODD, NEXT, GATED, 1>>(q, sh, 1 << 30, &grid, s)
              : launch<residual_kernel<TX, TY, V, ODD, NEXT, GATED, ODD ? 1 : 2>>(q, sh, 1 << 30, &grid, s);
  return true;
}

template <class TX, class TY, int V, int ODD>
bool forward(const Params& p, cudaStream_t s, cudaError_t* e) {
  if (p.h)
    return p.gate ? forward<TX, TY, V, ODD, true, true>(p, s, e) : forward<TX, TY, V, ODD, true, false>(p, s, e);
  return p.gate ? forward<TX, TY, V, ODD, false, true>(p, s, e) : forward<TX, TY, V, ODD, false, false>(p, s, e);
}

template <class TX, class TY, int V, int ODD, bool NEXT, bool GATED>
bool backward(const Params& p, int* rows, cudaStream_t s, cudaError_t* e) {
  using E = Residual<TX, TY, V, ODD, NEXT, GATED>;
  const int w = Weights::kind(p.w, NEXT ? p.wn : p.w);
  if (w == 0 || (w == 2 && ODD) || (p.C + V - 1) / V > kMaxGroup) return false;
  Params q = p;
  // a warp's slots are also where its shares pass
  constexpr int slots = E::TOKENS * E::SLOT > 2 * kFloats<V> ? E::TOKENS * E::SLOT : 2 * kFloats<V>;
  const Shape sh = plan(q, shape_of(p.T, p.C, V, 1, kMaxGroup), V,
                        [&](int G, int) { return Need{slots, 0, 4 * E::Sum::floats(G) * (NEXT ? 2 : 1)}; });
  if (q.direct || items(p.C, V, sh.G) != 1) return false;
  const int most = p.dw || p.dwn ? kMaxRows : 1 << 30;
  *e = w == 1 ? launch<residual_backward_kernel<TX, TY, V, ODD, NEXT, GATED, 1>>(q, sh, most, rows, s)
              : launch<residual_backward_kernel<TX, TY, V, ODD, NEXT, GATED, ODD ? 1 : 2>>(q, sh, most, rows, s);
  return true;
}

template <class TX, class TY, int V, int ODD>
bool backward(const Params& p, int* rows, cudaStream_t s, cudaError_t* e) {
  if (p.dh)
    return p.gate ? backward<TX, TY, V, ODD, true, true>(p, rows, s, e) : backward<TX, TY, V, ODD, true, false>(p, rows, s, e);
  return p.gate ? backward<TX, TY, V, ODD, false, true>(p, rows, s, e) : backward<TX, TY, V, ODD, false, false>(p, rows, s, e);
}

}  // namespace

bool residual_forward(const Params& p, int x_bf16, int y_bf16, bool vec, cudaStream_t s, cudaError_t* e) {
  if (p.S != 1 || p.P.p != nullptr) return false;
  if (!vec && y_bf16) return false;
  if (x_bf16) return forward<bf16_t, bf16_t, 8, 0>(p, s, e);
  if (y_bf16) return forward<float, bf16_t, 4, 0>(p, s, e);
  return vec ? forward<float, float, 4, 0>(p, s, e) : forward<float, float, 4, 2>(p, s, e);
}

bool residual_backward(const Params& p, int x_bf16, int y_bf16, bool vec, int* rows, cudaStream_t s, cudaError_t* e) {
  if (p.S != 1 || p.P.p != nullptr) return false;
  if (x_bf16) return vec ? backward<bf16_t, bf16_t, 8, 0>(p, rows, s, e) : backward<bf16_t, bf16_t, 8, 1>(p, rows, s, e);
  if (y_bf16) return vec ? backward<float, bf16_t, 4, 0>(p, rows, s, e) : backward<float, bf16_t, 4, 1>(p, rows, s, e);
  return vec ? backward<float, float, 4, 0>(p, rows, s, e) : backward<float, float, 4, 2>(p, rows, s, e);
}

}  // namespace hcb
