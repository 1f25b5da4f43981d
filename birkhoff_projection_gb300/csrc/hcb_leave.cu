// hcb_leave.cu -- the block's output, normalised, gated and scaled, written
// back into the mixed residual streams, and the next block's input from the
// result (hcb_leave of include/hc_block.h).
#include "hcb_common.cuh"

namespace hcb {

// The output's norm has to be known before the first stream is written, so a
// token is two runs of items: y (and the gate), of which w act(gate) y is
// kept in fp32 while its square is summed, then the streams.
// 16384 x 4 x 4096 bf16 with a gate: 225 us, 5.96 TB/s, 88% of the copy's
// rate; 6734 x 4 x 2624 fp32: 104 us, 90%.  Bound by the waits for the copies
// at the beginning of each run: registers (118) leave room for 16 warps on an
// SM, and the shared-memory pipe, through which everything passes twice, is
// busy for 42% of the time.
// Up to four items to a thread: with one 304 us, with two 237, with eight 233.
template <int SP, bool WHOLE, class TX, class TY, int V, int ODD>
struct Leave {
  using RX = Row<TX, V, ODD>;
  using RY = Row<TY, V, ODD>;
  using Co = Coefficients<SP, true, true, true>;
  using Sum = GroupSum<1>;
  // CTAs that the registers have to leave room for on an SM
  static constexpr int MINB = SP <= 2 || (SP == 4 && V == 4 && ODD == 0) ? 3 : SP == 4 ? 2 : 1;
  // a slot: the streams, or y and the gate; in one place only where both have
  // planes of one size, so that a lane's bytes are its own in both
  static constexpr int Y = RX::SLOT == RY::SLOT ? 0 : SP * RX::SLOT;
  static constexpr int SLOT = SP * RX::SLOT > Y + 2 * RY::SLOT ? SP * RX::SLOT : Y + 2 * RY::SLOT;
  static constexpr int ITEM = kFloats<V>;  // kept: w act y, then u
  static Need need(int G, int) {
    return {WHOLE ? 0 : SLOT, ITEM + (WHOLE ? SLOT : 0), 4 * (G / 32 * Co::FLOATS + 2 * Sum::floats(G))};
  }
};

// WHOLE: a slot to every item.  While a thread works through a token's y it
// copies the token's streams into the slots that it has read, and while it
// works through those the next token's y, so that it only waits once a run.
// Otherwise (rows too long for that) there is one slot, for the next item.
template <int SP, bool EXACT, class TX, class TY, int V, int ODD, int W>
__global__ void __launch_bounds__(256, Leave<SP, EXACT, TX, TY, V, ODD>::MINB) leave_kernel(const Params p) {
  constexpr bool WHOLE = EXACT;
  using E = Leave<SP, WHOLE, TX, TY, V, ODD>;
  using RX = typename E::RX;
  using RY = typename E::RY;
  using Co = typename E::Co;
  constexpr int H = V / 2, NEXT_SLOT = WHOLE ? E::SLOT : 0;
  extern __shared__ __align__(16) char smem[];
  const int G = p.G, NG = blockDim.x / G, group = threadIdx.x / G, l = threadIdx.x % G;
  const int lane = threadIdx.x & 31, warp = l / 32, C = p.C, S = EXACT ? SP : p.S, GV = G * V;
  const int K = (C + GV - 1) / GV, c0 = first_channel<V, ODD>(l), c1 = c0 + K * GV;
  char* of_group = smem + group * p.group_bytes;
  char* ring = of_group + warp * p.warp_bytes;
  char* item0 = ring + (WHOLE ? K : 1) * E::SLOT;
  float* co_all = reinterpret_cast<float*>(of_group + G / 32 * p.warp_bytes);
  float* co_s = co_all + warp * Co::FLOATS;
  float* red = co_all + G / 32 * Co::FLOATS;
  float* red_next = red + GroupSum<1>::floats(G);
  E::Sum::clear(red, G, l);
  E::Sum::clear(red_next, G, l);
  group_sync(G, group);
  int turn = 0, turn_next = 0;
  const float inv_c = 1.0f / static_cast<float>(C);
  const bool mix = EXACT ? SP > 1 : p.P.p != nullptr, gated = p.gate != nullptr;
  const uint32_t step = gridDim.x * NG;
  uint32_t t = blockIdx.x * NG + group;

  auto copy_y = [&](uint32_t t, int c, char* slot) {
    const uint32_t to = b4::smem_addr(slot);
    by_block<V, ODD>(c, C, [&](auto full) {
      constexpr bool FULL = decltype(full)::value;
      RY::template copy<FULL, E::Y>(to, lane, at_row<TY>(p.y, t, p.y_ts), c, C);
      if (gated) RY::template copy<FULL, E::Y + RY::SLOT>(to, lane, at_row<TY>(p.gate, t, p.gate_ts), c, C);
    });
  };
  auto copy_x = [&](uint32_t t, int c, char* slot) {
    const TX* x = at_row<TX>(p.x, t, p.x_ts);
    const uint32_t to = b4::smem_addr(slot);
    by_block<V, ODD>(c, C, [&](auto full) {
      constexpr bool FULL = decltype(full)::value;
      each<SP>([&](auto i) {
        if (EXACT || i.value < S) RX::template copy<FULL, i.value * RX::SLOT>(to, lane, x + i.value * p.x_ss, c, C);
      });
    });
  };
  Co co;
  co.init(p, lane);
  if (t < p.T) {
    co.fetch(t);
    char* slot = ring;
    for (int c = c0; c < (WHOLE ? c1 : c0 + 1); c += GV, slot += NEXT_SLOT) copy_y(t, c, slot);
  }

#pragma unroll 1
  for (; t < p.T; t += step) {
    co.spread(co_s, lane);
    const bool more = t + step < p.T;
    if (more) co.fetch(t + step);
    const TX* x = at_row<TX>(p.x, t, p.x_ts);
    const TY* y = at_row<TY>(p.y, t, p.y_ts);
    const TY* gate = at_row<TY>(p.gate, t, p.gate_ts);
    P2 ss = 0;
    char *item = item0, *slot = ring;
    if (WHOLE) slots_ready<ODD>();
#pragma unroll 1
    for (int c = c0; c < c1; c += GV, item += E::ITEM, slot += NEXT_SLOT) {
      P2 v[H], w[H];
      p.w.load<V, ODD, W>(c, lane, C, w);
      if (!WHOLE) slots_ready<ODD>();
      RY::arrived(slot + E::Y, lane, y, c, v);
#pragma unroll
      for (int j = 0; j < H; ++j) {
        ss = fma2(v[j], v[j], ss);
        v[j] = mul2(v[j], w[j]);
      }
      if (gated) {
        P2 g[H];
        RY::arrived(slot + E::Y + RY::SLOT, lane, gate, c, g);
        gates<TY, V, false>(p.act, g, w);
#pragma unroll
        for (int j = 0; j < H; ++j) v[j] = mul2(v[j], g[j]);
      }
      keep<V>(item, lane, v);
      slot_read<ODD>();
      if (WHOLE)
        copy_x(t, c, slot);
      else if (c + GV < c1)
        copy_y(t, c + GV, slot);
      else
        copy_x(t, c0, slot);
    }
    float rho = p.scale;
    if (p.norm) {
      const float sum[1] = {both(ss)};
      float total[1];
      GroupSum<1>::run(sum, total, red, turn, G, group, lane, warp);
      rho *= rsqrtf(of_total(total, 0) * inv_c + p.eps);
    }
    P2 b[SP];
    Co::read(co_s, Co::NP, b);
#pragma unroll
    for (int i = 0; i < SP; ++i) b[i] = mul2(b[i], twice(rho));
    TX* out = static_cast<TX*>(p.out) + uint64_t(t) * uint32_t(S * C);
    ss = 0;
    item = item0, slot = ring;
    if (WHOLE) slots_ready<ODD>();
#pragma unroll 1
    for (int c = c0; c < c1; c += GV, item += E::ITEM, slot += NEXT_SLOT) {
      if (!WHOLE) slots_ready<ODD>();
      P2 v[H], xv[SP][H], u[H] = {};
      kept<V>(item, lane, v);
#pragma unroll
      for (int i = 0; i < SP; ++i) {
        if (EXACT || i < S) {
          RX::arrived(slot + i * RX::SLOT, lane, x + i * p.x_ss, c, xv[i]);
        } else {
#pragma unroll
          for (int j = 0; j < H; ++j) xv[i][j] = 0;
        }
      }
      slot_read<ODD>();
      if (WHOLE) {
        if (more) copy_y(t + step, c, slot);
      } else if (c + GV < c1) {
        copy_x(t, c + GV, slot);
      } else if (more) {
        copy_y(t + step, c0, slot);
      }
      P2 a[SP];
      if (p.h) Co::read(co_s, Co::NB, a);
#pragma unroll
      for (int i = 0; i < SP; ++i) {
        if (EXACT || i < S) {
          P2 o[H];
          if (mix) {
            P2 P[SP];
            Co::read(co_s, i * SP, P);
#pragma unroll
            for (int j = 0; j < H; ++j) {
              o[j] = mul2(b[i], v[j]);
#pragma unroll
              for (int q = 0; q < SP; ++q) o[j] = fma2(P[q], xv[q][j], o[j]);
            }
          } else {
#pragma unroll
            for (int j = 0; j < H; ++j) o[j] = fma2(b[i], v[j], xv[i][j]);
          }
          if (p.h) {
            RX::store_rounded(out + i * C, c, lane, C, o);
#pragma unroll
            for (int j = 0; j < H; ++j) u[j] = fma2(a[i], o[j], u[j]);
          } else {
            RX::store(out + i * C, c, lane, C, o);
          }
        }
      }
      if (p.h) {
#pragma unroll
        for (int j = 0; j < H; ++j) ss = fma2(u[j], u[j], ss);  // past C: y, x and so u are zeros
        keep<V>(item, lane, u);
      }
    }
    if (p.h) {
      const float sum[1] = {both(ss)};
      float total[1];
      GroupSum<1>::run(sum, total, red_next, turn_next, G, group, lane, warp);
      const P2 r = twice(rsqrtf(of_total(total, 0) * inv_c + p.eps_next));
      TY* h = static_cast<TY*>(p.h) + uint64_t(t) * uint32_t(C);
      item = item0;
#pragma unroll 1
      for (int c = c0; c < c1; c += GV, item += E::ITEM) {
        P2 u[H], w[H];
        kept<V>(item, lane, u);
        p.wn.load<V, ODD, W>(c, lane, C, w);
#pragma unroll
        for (int j = 0; j < H; ++j) u[j] = mul2(u[j], mul2(r, w[j]));
        RY::store(h, c, lane, C, u);
      }
    }
  }
  copy_wait_all();
}

namespace {

struct Forward {
  const Params& p;
  cudaStream_t s;
  template <int SP, bool EXACT, class TX, class TY, int V, int ODD>
  cudaError_t operator()() const {
    Params q = p;
    int grid;
    const Shape want = shape_of(p.T, p.C, V, 4, 256);
    const int w = EXACT && (p.P.p != nullptr) == (SP > 1) ? Weights::kind(p.w, p.h ? p.wn : p.w) : 0;
    if (w == 1 || (w == 2 && ODD == 0)) {
      const Shape sh = plan(q, want, V, Leave<SP, true, TX, TY, V, ODD>::need);
      if (!q.direct && w == 1)
        return launch<leave_kernel<SP, EXACT, TX, TY, V, ODD, EXACT ? 1 : 0>>(q, sh, 1 << 30, &grid, s);
      if (!q.direct)
        return launch<leave_kernel<SP, EXACT && ODD == 0, TX, TY, V, ODD, EXACT && ODD == 0 ? 2 : 0>>(q, sh, 1 << 30, &grid, s);
    }
    const Shape sh = plan(q, want, V, Leave<SP, false, TX, TY, V, ODD>::need);
    return launch<leave_kernel<SP, false, TX, TY, V, ODD, 0>>(q, sh, 1 << 30, &grid, s);
  }
};

}  // namespace

cudaError_t leave_forward(const Params& p, int x_bf16, int y_bf16, bool vec, cudaStream_t s) {
  return by_streams(p.S, x_bf16, y_bf16, vec, Forward{p, s});
}

}  // namespace hcb
