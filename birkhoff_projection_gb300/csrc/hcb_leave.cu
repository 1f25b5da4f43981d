// hcb_leave.cu -- the block's output, normalised, gated and scaled, written
// back into the mixed residual streams, and the next block's input from the
// result (hcb_leave of include/hc_block.h).
#include "hcb_common.cuh"

#ifndef HCB_LEAVE_DEPTH
#define HCB_LEAVE_DEPTH 2
#endif
#ifndef HCB_LEAVE_PER
#define HCB_LEAVE_PER 2
#endif

namespace hcb {

// The output's norm has to be known before the first stream is written, so a
// token is two runs of items: y (and the gate), of which w act(gate) y is
// kept in fp32 while its square is summed, then the streams.
template <int SP, class TX, class TY, int V, bool ODD>
struct Leave {
  using RX = Row<TX, V, ODD>;
  using RY = Row<TY, V, ODD>;
  using Co = Coefficients<SP, true, true, true>;
  using Sum = GroupSum<1>;
  static constexpr int DEPTH = HCB_LEAVE_DEPTH;
  // a slot: the streams, or y and the gate; in one place only where both have
  // planes of one size, so that a lane's bytes are its own in both
  static constexpr int Y = RX::SLOT == RY::SLOT ? 0 : SP * RX::SLOT;
  static constexpr int SLOT = SP * RX::SLOT > Y + 2 * RY::SLOT ? SP * RX::SLOT : Y + 2 * RY::SLOT;
  static constexpr int ITEM = kFloats<V>;  // kept: w act y, then u
  static Need need(int G, int) {
    return {DEPTH * SLOT, ITEM, 4 * (G / 32 * Co::FLOATS + 2 * Sum::floats(G))};
  }
};

template <int SP, bool EXACT, class TX, class TY, int V, bool ODD, int W>
__global__ void __launch_bounds__(SP == 8 ? 256 : kMaxGroup, 1) leave_kernel(const Params p) {
  using E = Leave<SP, TX, TY, V, ODD>;
  using RX = typename E::RX;
  using RY = typename E::RY;
  using Co = typename E::Co;
  constexpr int DEPTH = E::DEPTH, H = V / 2;
  extern __shared__ __align__(16) char smem[];
  const int G = p.G, NG = blockDim.x / G, group = threadIdx.x / G, l = threadIdx.x % G;
  const int lane = threadIdx.x & 31, warp = l / 32, C = p.C, S = EXACT ? SP : p.S, GV = G * V;
  const int K = (C + GV - 1) / GV, c0 = first_channel<V, ODD>(l);
  char* of_group = smem + group * p.group_bytes;
  char* ring = of_group + warp * p.warp_bytes;
  char* item0 = ring + DEPTH * E::SLOT;
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

  uint32_t ta = t;
  int ca = c0, ia = 0;
  char* slot_a = ring;
  auto copy_next = [&] {
    slot_read<ODD>();
    if (ta < p.T && ca < C) {
      if (ia >= K) {
        const TX* x = at_row<TX>(p.x, ta, p.x_ts);
#pragma unroll
        for (int i = 0; i < SP; ++i)
          if (EXACT || i < S) RX::copy(slot_a + i * RX::SLOT, lane, x + i * p.x_ss, ca, C);
      } else {
        RY::copy(slot_a + E::Y, lane, at_row<TY>(p.y, ta, p.y_ts), ca, C);
        if (gated) RY::copy(slot_a + E::Y + RY::SLOT, lane, at_row<TY>(p.gate, ta, p.gate_ts), ca, C);
      }
    }
    copy_commit();
    ca += GV;
    ++ia;
    if (ia == K) ca = c0;
    if (ia == 2 * K) ia = 0, ca = c0, ta += step;
    slot_a = slot_a == ring + (DEPTH - 1) * E::SLOT ? ring : slot_a + E::SLOT;
  };
  Co co;
  co.init(p, lane);
  if (t < p.T) co.fetch(t);
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) copy_next();

  const char* slot = ring;
#pragma unroll 1
  for (; t < p.T; t += step) {
    co.spread(co_s, lane);
    if (t + step < p.T) co.fetch(t + step);
    const TX* x = at_row<TX>(p.x, t, p.x_ts);
    const TY* y = at_row<TY>(p.y, t, p.y_ts);
    const TY* gate = at_row<TY>(p.gate, t, p.gate_ts);
    P2 ss = 0;
    char* item = item0;
#pragma unroll 1
    for (int c = c0, k = 0; k < K; ++k, c += GV, item += E::ITEM) {
      P2 w[H];
      if (c < C) p.w.load<V, ODD, W>(c, lane, C, w);
      slot_ready<DEPTH, ODD>();
      if (c < C) {
        P2 v[H];
        RY::arrived(slot + E::Y, lane, y, c, v);
#pragma unroll
        for (int j = 0; j < H; ++j) {
          ss = fma2(v[j], v[j], ss);
          v[j] = mul2(v[j], w[j]);
        }
        if (gated) {
          P2 g[H];
          RY::arrived(slot + E::Y + RY::SLOT, lane, gate, c, g);
          gates<V, false>(p.act, g, w);
#pragma unroll
          for (int j = 0; j < H; ++j) v[j] = mul2(v[j], g[j]);
        }
        keep<V>(item, lane, v);
      }
      copy_next();
      slot = slot == ring + (DEPTH - 1) * E::SLOT ? ring : slot + E::SLOT;
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
    item = item0;
#pragma unroll 1
    for (int c = c0, k = 0; k < K; ++k, c += GV, item += E::ITEM) {
      slot_ready<DEPTH, ODD>();
      if (c < C) {
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
      copy_next();
      slot = slot == ring + (DEPTH - 1) * E::SLOT ? ring : slot + E::SLOT;
    }
    if (p.h) {
      const float sum[1] = {both(ss)};
      float total[1];
      GroupSum<1>::run(sum, total, red_next, turn_next, G, group, lane, warp);
      const P2 r = twice(rsqrtf(of_total(total, 0) * inv_c + p.eps_next));
      TY* h = static_cast<TY*>(p.h) + uint64_t(t) * uint32_t(C);
      item = item0;
#pragma unroll 1
      for (int c = c0; c < C; c += GV, item += E::ITEM) {
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
  template <int SP, bool EXACT, class TX, class TY, int V, bool ODD>
  cudaError_t operator()() const {
    Params q = p;
    int grid;
    const Shape sh =
        plan(q, shape_of(p.T, p.C, V, HCB_LEAVE_PER, SP == 8 ? 256 : kMaxGroup), V, Leave<SP, TX, TY, V, ODD>::need);
    const int w = EXACT && (p.P.p != nullptr) == (SP > 1) ? Weights::kind(p.w, p.h ? p.wn : p.w) : 0;
    if (w == 1) return launch<leave_kernel<SP, EXACT, TX, TY, V, ODD, EXACT ? 1 : 0>>(q, sh, 1 << 30, &grid, s);
    if (w == 2 && !ODD) return launch<leave_kernel<SP, EXACT && !ODD, TX, TY, V, ODD, EXACT && !ODD ? 2 : 0>>(q, sh, 1 << 30, &grid, s);
    return launch<leave_kernel<SP, false, TX, TY, V, ODD, 0>>(q, sh, 1 << 30, &grid, s);
  }
};

}  // namespace

cudaError_t leave_forward(const Params& p, int x_bf16, int y_bf16, bool vec, cudaStream_t s) {
  return by_streams(p.S, x_bf16, y_bf16, vec, Forward{p, s});
}

}  // namespace hcb
