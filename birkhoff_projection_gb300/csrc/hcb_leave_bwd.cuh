// hcb_leave_bwd.cuh -- the gradient of leave and of leave_enter
// (hcb_leave_backward of include/hc_block.h); instantiated in hcb_leave_bwd.cu
// and hcb_leave_enter_bwd.cu.
#pragma once

#include "hcb_common.cuh"

namespace hcb {

// Every sum that the gradient needs is linear in what is read, up to the
// factor rho of y's norm: with q = act(gate) and e = w q y,
//   dP_ij = <D_i, x_j>,  db_i = scale rho <D_i, e>,  <g, y> = scale <dv, e>
// with dv = sum_i b_i D_i, so one pass over the row finds S^2 + S + 2 sums and
// writes dx.  It keeps q dv and act'(gate) w y dv, of which a second one
// writes dy, dgate and the weight's shares.  <dv, e> is also sum_i b_i <D_i, e>,
// but where the D_i nearly cancel in dv that would keep the rounding of the
// larger sums (next_sums in hcb_common.cuh).
// 16384 x 4 x 4096 bf16 with a gate: 374 us, 5.8 TB/s, 85% of the copy's rate;
// 4096 x 4 x 4096 fp32 with bf16 rows: 149 us, 93%.  The 22 sums to a thread
// take the registers of all but two CTAs of 256 threads, and the shares of dw
// the shared memory of deeper rings; four items to a thread instead of two
// take 415 us.
// NEXT adds a run of items before it: D_i = dout_i + a_i du with du from dh,
// as in enter_backward_kernel.  With what that keeps, four bf16 streams and a
// gate ask for 129 KB to a CTA of 256 threads, and an SM has one: 16384 x 4 x
// 4096 758 us, 55% of the copy's rate (enter's and leave's gradients apart 665);
// without a gate 482 us, 78%.
template <int SP, class TX, class TY, int V, int ODD, bool NEXT>
struct LeaveBackward {
  using RX = Row<TX, V, ODD>;
  using RY = Row<TY, V, ODD>;
  using Co = Coefficients<SP, true, true, NEXT, true>;
  // the sums: dP (by column), <D_i, e>, <y, y>, and of several streams <dv, e>
  static constexpr int YY = SP * SP + SP, DV = YY + 1, R = SP > 1 ? DV + 1 : DV;
  // dP's sums as pairs of channels, where the registers hold twice as many
  static constexpr bool PAIRS = SP <= 2 || (SP == 4 && V == 4);
  using Sum = GroupSum<R>;
  using SumNext = GroupSum<next_sums(SP)>;
  // CTAs that the registers have to leave room for on an SM
  static constexpr int minb(int gate) { return SP == 1 && gate == 0 ? 3 : SP <= 4 ? 2 : 1; }
  // a slot: dout, y, gate and x; or the stored result, and dh where y would be
  static constexpr int Y = SP * RX::SLOT, GATE = Y + RY::SLOT, X = GATE + RY::SLOT;
  __host__ __device__ static constexpr int slot(bool mix, bool gated) {
    return mix ? X + SP * RX::SLOT : gated ? X : GATE;
  }
  // kept: q dv (before it, NEXT: the next block's u); y; NEXT: dh; the shares
  // of dw and of dw_next; act' w y dv.  direct: the first and the last only.
  static constexpr int F = kFloats<V>, KY = F, KH = KY + RY::KEPT, KW = KH + (NEXT ? RY::KEPT : 0), KN = KW + F,
                       KB = KN + (NEXT ? F : 0);
  __host__ __device__ static constexpr int kb(int direct) { return direct ? F : KB; }
  __host__ __device__ static constexpr int item(bool gated, int direct) { return kb(direct) + (gated ? F : 0); }
};

// GATE: 0 no gate, 1 a gate, 2 told at run time.
template <int SP, bool EXACT, class TX, class TY, int V, int ODD, bool NEXT, int GATE, int W>
__global__ void __launch_bounds__(256, LeaveBackward<SP, TX, TY, V, ODD, NEXT>::minb(GATE)) leave_backward_kernel(const Params p) {
  using E = LeaveBackward<SP, TX, TY, V, ODD, NEXT>;
  using RX = typename E::RX;
  using RY = typename E::RY;
  using Co = typename E::Co;
  using Sum = typename E::Sum;
  // WHOLE, as in leave_kernel: a slot to every item, each copied to again as
  // soon as it is read.  For more streams the slots would leave room for fewer
  // threads: there is one, for the next item.
  constexpr bool WHOLE = EXACT && SP <= 2;
  constexpr int R = E::R, H = V / 2;
  extern __shared__ __align__(16) char smem[];
  const int G = p.G, NG = blockDim.x / G, group = threadIdx.x / G, l = threadIdx.x % G;
  const int lane = threadIdx.x & 31, warp = l / 32, C = p.C, S = EXACT ? SP : p.S, GV = G * V;
  const int K = (C + GV - 1) / GV, c0 = first_channel<V, ODD>(l), c1 = c0 + K * GV;
  const bool direct = !EXACT && p.direct;
  const bool mix = EXACT ? SP > 1 : p.P.p != nullptr, gated = GATE == 2 ? p.gate != nullptr : GATE != 0;
  const int SLOT = E::slot(mix, gated), ITEM = E::item(gated, direct), KB = E::kb(direct);
  const int NEXT_SLOT = WHOLE ? SLOT : 0;
  char* of_group = smem + group * p.group_bytes;
  char* ring = of_group + warp * p.warp_bytes;
  char* item0 = ring + (WHOLE ? K : 1) * SLOT;
  float* co_all = reinterpret_cast<float*>(of_group + G / 32 * p.warp_bytes);
  float* co_s = co_all + warp * Co::FLOATS;
  float* red = co_all + G / 32 * Co::FLOATS;
  float* red_next = red + Sum::floats(G);
  Sum::clear(red, G, l);
  if constexpr (NEXT) E::SumNext::clear(red_next, G, l);
  let_next_launch();
  group_sync(G, group);
  float* row_dw = direct && p.dw ? p.dw + int64_t(blockIdx.x) * pitch(C) : nullptr;
  float* row_dwn = NEXT && direct && p.dwn ? p.dwn + int64_t(blockIdx.x) * pitch(C) : nullptr;
  int turn = 0, turn_next = 0;
  const float inv_c = 1.0f / static_cast<float>(C);
  const uint32_t step = gridDim.x * NG;
  uint32_t t = blockIdx.x * NG + group;

  // The two kinds of items: `first`, NEXT's stored result and dh, and the
  // rest.  (One copy in the code for both: more would cost registers.)
  auto copy = [&](bool first, uint32_t t, int c, char* slot) {
    first = NEXT && first;
    const TX* d = first ? at_row<TX>(p.out_in, t, p.out_ts) : at_row<TX>(p.dout, t, p.dout_ts);
    const uint32_t ss = first ? p.out_ss : p.dout_ss;
    const uint32_t to = b4::smem_addr(slot);
    by_block<V, ODD>(c, C, [&](auto full) {
      constexpr bool FULL = decltype(full)::value;
      each<SP>([&](auto i) {
        if (EXACT || i.value < S) RX::template copy<FULL, i.value * RX::SLOT>(to, lane, d + i.value * ss, c, C);
      });
      RY::template copy<FULL, E::Y>(to, lane, first ? at_row<TY>(p.dh, t, p.dh_ts) : at_row<TY>(p.y, t, p.y_ts), c, C);
      if (first) return;
      if (gated) RY::template copy<FULL, E::GATE>(to, lane, at_row<TY>(p.gate, t, p.gate_ts), c, C);
      if (mix) {
        const TX* x = at_row<TX>(p.x, t, p.x_ts);
        each<SP>([&](auto i) {
          if (EXACT || i.value < S)
            RX::template copy<FULL, E::X + i.value * RX::SLOT>(to, lane, x + i.value * p.x_ss, c, C);
        });
      }
    });
  };
  Co co;
  co.init(p, lane);
  if (t < p.T) {
    co.fetch(t);
    char* slot = ring;
    for (int c = c0; c < (WHOLE ? c1 : c0 + 1); c += GV, slot += NEXT_SLOT) copy(true, t, c, slot);
  }
  {
    const P2 z[H] = {};
    char* item = item0;
#pragma unroll 1
    for (int c = c0; c < c1; c += GV, item += ITEM) {
      if (direct) {
        if (row_dw) PartRow<V, ODD>::put(row_dw, c, lane, C, z);
        if (NEXT && row_dwn) PartRow<V, ODD>::put(row_dwn, c, lane, C, z);
      } else {
        keep<V>(item + E::KW, lane, z);
        if constexpr (NEXT) keep<V>(item + E::KN, lane, z);
      }
    }
  }

#pragma unroll 1
  for (; t < p.T; t += step) {
    co.spread(co_s, lane);
    const bool more = t + step < p.T;
    if (more) co.fetch(t + step);
    float r_next = 0.0f, k_next = 0.0f;
    if constexpr (NEXT) {
      const TX* o = at_row<TX>(p.out_in, t, p.out_ts);
      const TY* dh = at_row<TY>(p.dh, t, p.dh_ts);
      P2 a[SP], sum2[next_sums(SP)] = {};
      Co::read(co_s, Co::NB, a);
      char *item = item0, *slot = ring;
      if (WHOLE) slots_ready<ODD>();
#pragma unroll 1
      for (int c = c0; c < c1; c += GV, item += ITEM, slot += NEXT_SLOT) {
        P2 xv[SP][H], g[H], w[H], u[H] = {};
        p.wn.load<V, ODD, W>(c, lane, C, w);
        if (!WHOLE) slots_ready<ODD>();
#pragma unroll
        for (int i = 0; i < SP; ++i) {
          if (EXACT || i < S) {
            RX::arrived(slot + i * RX::SLOT, lane, o + i * p.out_ss, c, xv[i]);
#pragma unroll
            for (int j = 0; j < H; ++j) u[j] = fma2(a[i], xv[i][j], u[j]);
          }
        }
        if (direct)
          RY::arrived(slot + E::Y, lane, dh, c, g);
        else
          RY::arrived_kept(slot + E::Y, lane, dh, c, g, item + E::KH);
        slot_read<ODD>();
        const bool same = !WHOLE && c + GV < c1;
        copy(same, t, WHOLE ? c : same ? c + GV : c0, slot);
#pragma unroll
        for (int j = 0; j < H; ++j) g[j] = mul2(g[j], w[j]);
#pragma unroll
        for (int i = 0; i < SP; ++i) {
          if (EXACT || i < S) {
#pragma unroll
            for (int j = 0; j < H; ++j) {
              sum2[i] = fma2(g[j], xv[i][j], sum2[i]);
              sum2[SP + i] = fma2(u[j], xv[i][j], sum2[SP + i]);
            }
          }
        }
        if constexpr (SP > 1) {
#pragma unroll
          for (int j = 0; j < H; ++j) {
            sum2[2 * SP] = fma2(g[j], u[j], sum2[2 * SP]);
            sum2[2 * SP + 1] = fma2(u[j], u[j], sum2[2 * SP + 1]);
          }
        }
        keep<V>(item, lane, u);
      }
      float sum[next_sums(SP)], total[1], gu, uu;
#pragma unroll
      for (int i = 0; i < next_sums(SP); ++i) sum[i] = both(sum2[i]);
      E::SumNext::run(sum, total, red_next, turn_next, G, group, lane, warp);
      sums_of_u<SP>(total, low(a[0]), gu, uu);
      r_next = rsqrtf(uu * inv_c + p.eps_next);
      k_next = gu * inv_c * r_next * r_next;
      if (p.da) {
        const float u_x = __shfl_sync(0xffffffffu, total[0], (lane + SP) & 31);
        if (warp == 0 && lane < S)
          put_any(p.da, p.a.bf16, int64_t(t) * S + lane, r_next * (total[0] - k_next * u_x));
      }
    }
    const TX* dout = at_row<TX>(p.dout, t, p.dout_ts);
    const TX* x = at_row<TX>(p.x, t, p.x_ts);
    const TY* y = at_row<TY>(p.y, t, p.y_ts);
    const TY* gate = at_row<TY>(p.gate, t, p.gate_ts);
    P2 sum_dP2[E::PAIRS ? SP * SP : 1] = {}, sum_e2[SP] = {}, sum_y2 = 0, sum_dv2 = 0;
    float sum_dP[E::PAIRS ? 1 : SP * SP] = {};
    TX* dx = p.dx ? static_cast<TX*>(p.dx) + uint64_t(t) * uint32_t(S * C) : nullptr;
    char *item = item0, *slot = ring;
    if (WHOLE) slots_ready<ODD>();
#pragma unroll 1
    for (int c = c0; c < c1; c += GV, item += ITEM, slot += NEXT_SLOT) {
      P2 du[H];
      if constexpr (NEXT) {
        P2 h[H], wn[H];
        const P2 r2 = twice(r_next), minus_k = twice(-k_next);
        kept<V>(item, lane, du);
        if (direct)
          RY::load(at_row<TY>(p.dh, t, p.dh_ts), c, lane, C, h);
        else
          RY::kept(item + E::KH, lane, h);
        p.wn.load<V, ODD, W>(c, lane, C, wn);
#pragma unroll
        for (int j = 0; j < H; ++j) du[j] = mul2(r2, du[j]);
        if (p.dwn) add_share<V, ODD>(item + E::KN, row_dwn, c, lane, C, h, du);
#pragma unroll
        for (int j = 0; j < H; ++j) du[j] = fma2(mul2(r2, wn[j]), h[j], mul2(minus_k, du[j]));
      }
      if (!WHOLE) slots_ready<ODD>();
      P2 D[SP][H], e[H], g[H];
#pragma unroll
      for (int i = 0; i < SP; ++i) {
        if (EXACT || i < S) {
          RX::arrived(slot + i * RX::SLOT, lane, dout + i * p.dout_ss, c, D[i]);
        } else {
#pragma unroll
          for (int j = 0; j < H; ++j) D[i][j] = 0;
        }
      }
      if constexpr (NEXT) {
        P2 a[SP];
        Co::read(co_s, Co::NB, a);
#pragma unroll
        for (int i = 0; i < SP; ++i)
#pragma unroll
          for (int j = 0; j < H; ++j) D[i][j] = fma2(a[i], du[j], D[i][j]);
      }
      if (mix) {
#pragma unroll
        for (int q = 0; q < SP; ++q) {
          if (EXACT || q < S) {
            P2 xv[H];
            RX::arrived(slot + E::X + q * RX::SLOT, lane, x + q * p.x_ss, c, xv);
#pragma unroll
            for (int i = 0; i < SP; ++i)
#pragma unroll
              for (int j = 0; j < H; ++j) {
                if constexpr (E::PAIRS) {
                  sum_dP2[q * SP + i] = fma2(D[i][j], xv[j], sum_dP2[q * SP + i]);
                } else {
                  float dl, dh, xl, xh;
                  split(D[i][j], dl, dh);
                  split(xv[j], xl, xh);
                  sum_dP[q * SP + i] = fmaf(dh, xh, fmaf(dl, xl, sum_dP[q * SP + i]));
                }
              }
          }
        }
      }
      if (direct)
        RY::arrived(slot + E::Y, lane, y, c, e);
      else
        RY::arrived_kept(slot + E::Y, lane, y, c, e, item + E::KY);
      if (gated) RY::arrived(slot + E::GATE, lane, gate, c, g);
      slot_read<ODD>();
      {
        const bool same = !WHOLE && c + GV < c1;
        if (same || more) copy(!same, same ? t : t + step, WHOLE ? c : same ? c + GV : c0, slot);
      }
      if (dx) {
#pragma unroll
        for (int q = 0; q < SP; ++q) {
          if (EXACT || q < S) {
            if (mix) {
              P2 d[H], P[SP];
              Co::read(co_s, q * SP, P);
#pragma unroll
              for (int j = 0; j < H; ++j) {
                d[j] = mul2(P[0], D[0][j]);
#pragma unroll
                for (int i = 1; i < SP; ++i) d[j] = fma2(P[i], D[i][j], d[j]);
              }
              RX::store(dx + q * C, c, lane, C, d);
            } else {
              RX::store(dx + q * C, c, lane, C, D[q]);
            }
          }
        }
      }
      P2 dv[H], b[SP];
      Co::read(co_s, Co::NP, b);
#pragma unroll
      for (int j = 0; j < H; ++j) {
        dv[j] = mul2(b[0], D[0][j]);
#pragma unroll
        for (int i = 1; i < SP; ++i) dv[j] = fma2(b[i], D[i][j], dv[j]);
        sum_y2 = fma2(e[j], e[j], sum_y2);
      }
      {
        P2 w[H];
        p.w.load<V, ODD, W>(c, lane, C, w);
#pragma unroll
        for (int j = 0; j < H; ++j) e[j] = mul2(e[j], w[j]);
      }
      if (gated) {
        P2 slope[H];
        gates<TY, V, true>(p.act, g, slope);
#pragma unroll
        for (int j = 0; j < H; ++j) {
          slope[j] = mul2(slope[j], mul2(e[j], dv[j]));
          e[j] = mul2(e[j], g[j]);
          if (SP > 1) sum_dv2 = fma2(dv[j], e[j], sum_dv2);
          dv[j] = mul2(dv[j], g[j]);
        }
        keep<V>(item + KB, lane, slope);
      } else if (SP > 1) {
#pragma unroll
        for (int j = 0; j < H; ++j) sum_dv2 = fma2(dv[j], e[j], sum_dv2);
      }
      keep<V>(item, lane, dv);
#pragma unroll
      for (int i = 0; i < SP; ++i)
#pragma unroll
        for (int j = 0; j < H; ++j) sum_e2[i] = fma2(D[i][j], e[j], sum_e2[i]);
    }
    float sum[R], total[Sum::CH];
#pragma unroll
    for (int i = 0; i < SP * SP; ++i) sum[i] = E::PAIRS ? both(sum_dP2[E::PAIRS ? i : 0]) : sum_dP[E::PAIRS ? 0 : i];
#pragma unroll
    for (int i = 0; i < SP; ++i) sum[SP * SP + i] = both(sum_e2[i]);
    sum[E::YY] = both(sum_y2);
    if constexpr (SP > 1) sum[E::DV] = both(sum_dv2);
    Sum::run(sum, total, red, turn, G, group, lane, warp);
    const float rho = p.norm ? rsqrtf(of_total(total, E::YY) * inv_c + p.eps) : 1.0f;
    float gy;
    if constexpr (SP > 1) {
      gy = of_total(total, E::DV);
    } else {
      P2 b[1];
      Co::read(co_s, Co::NP, b);
      gy = low(b[0]) * of_total(total, SP * SP);
    }
    const float sr = p.scale * rho;
    const P2 sr2 = twice(sr), minus_k = twice(p.norm ? -sr * gy * inv_c * rho * rho : 0.0f);
    if (warp == 0) {
#pragma unroll
      for (int ch = 0; ch < Sum::CH; ++ch) {
        const int n = ch * 32 + lane, i = n % SP, j = n / SP;
        if (n < SP * SP) {
          if (p.dP && i < S && j < S) put_any(p.dP, p.P.bf16, (int64_t(t) * S + i) * S + j, total[ch]);
        } else if (n < SP * SP + S) {
          if (p.db) put_any(p.db, p.b.bf16, int64_t(t) * S + n - SP * SP, sr * total[ch]);
        }
      }
    }
    TY* dy = p.dy ? static_cast<TY*>(p.dy) + uint64_t(t) * uint32_t(C) : nullptr;
    TY* dgate = gated && p.dgate ? static_cast<TY*>(p.dgate) + uint64_t(t) * uint32_t(C) : nullptr;
    item = item0;
#pragma unroll 1
    for (int c = c0; c < c1; c += GV, item += ITEM) {
      P2 yv[H], w[H], d[H];
      if (direct)
        RY::load(y, c, lane, C, yv);
      else
        RY::kept(item + E::KY, lane, yv);
      if (dgate) {
        P2 g[H];
        kept<V>(item + KB, lane, g);
#pragma unroll
        for (int j = 0; j < H; ++j) g[j] = mul2(g[j], sr2);
        RY::store(dgate, c, lane, C, g);
      }
      p.w.load<V, ODD, W>(c, lane, C, w);
      kept<V>(item, lane, d);
#pragma unroll
      for (int j = 0; j < H; ++j) d[j] = mul2(d[j], sr2);
      if (p.dw) add_share<V, ODD>(item + E::KW, row_dw, c, lane, C, d, yv);
      if (dy) {
#pragma unroll
        for (int j = 0; j < H; ++j) d[j] = fma2(d[j], w[j], mul2(minus_k, yv[j]));
        RY::store(dy, c, lane, C, d);
      }
    }
  }
  copy_wait_all();
  if (!direct && (p.dw || (NEXT && p.dwn))) {
    __syncthreads();
    const int64_t row = int64_t(blockIdx.x) * pitch(C);
    const char* first = smem + warp * p.warp_bytes + (WHOLE ? K : 1) * SLOT;
    if (p.dw) sum_shares<V, ODD>(first + E::KW, p, NG, ITEM, p.dw + row);
    if (NEXT && p.dwn) sum_shares<V, ODD>(first + E::KN, p, NG, ITEM, p.dwn + row);
  }
}

template <bool NEXT>
struct Backward {
  const Params& p;
  int* rows;
  cudaStream_t s;
  template <int SP, bool EXACT, class TX, class TY, int V, int ODD>
  cudaError_t operator()() const {
    using E = LeaveBackward<SP, TX, TY, V, ODD, NEXT>;
    Params q = p;
    const bool mix = p.P.p != nullptr, gated = p.gate != nullptr;
    auto need = [&](bool whole) {
      return [&, whole](int G, int direct) {
        const int slot = E::slot(mix, gated);
        return Need{whole ? 0 : slot, E::item(gated, direct) + (whole ? slot : 0),
                    4 * (G / 32 * E::Co::FLOATS + E::Sum::floats(G) + (NEXT ? E::SumNext::floats(G) : 0))};
      };
    };
    const Shape want = shape_of(p.T, p.C, V, 2, 256);
    const int most = p.dw || p.dwn ? kMaxRows : 1 << 30;
    int w = EXACT && mix == (SP > 1) ? Weights::kind(p.w, NEXT ? p.wn : p.w) : 0;
    if (w == 2 && ODD) w = 0;
    Shape sh = plan(q, want, V, need(w != 0 && SP <= 2));
    if (w != 0 && q.direct) w = 0;
    if (w == 0) sh = plan(q, want, V, need(false));
    constexpr int W1 = EXACT ? 1 : 0, W2 = EXACT && ODD == 0 ? 2 : 0;
    if (w == 1 && gated)
      return launch<leave_backward_kernel<SP, EXACT, TX, TY, V, ODD, NEXT, W1 ? 1 : 2, W1>>(q, sh, most, rows, s);
    if (w == 1)
      return launch<leave_backward_kernel<SP, EXACT, TX, TY, V, ODD, NEXT, W1 ? 0 : 2, W1>>(q, sh, most, rows, s);
    if (w == 2 && gated)
      return launch<leave_backward_kernel<SP, W2 != 0, TX, TY, V, ODD, NEXT, W2 ? 1 : 2, W2>>(q, sh, most, rows, s);
    if (w == 2)
      return launch<leave_backward_kernel<SP, W2 != 0, TX, TY, V, ODD, NEXT, W2 ? 0 : 2, W2>>(q, sh, most, rows, s);
    return launch<leave_backward_kernel<SP, false, TX, TY, V, ODD, NEXT, 2, 0>>(q, sh, most, rows, s);
  }
};

}  // namespace hcb
