// hcb_leave_bwd.cu -- the gradient of leave and of leave_enter
// (hcb_leave_backward of include/hc_block.h).
#include "hcb_common.cuh"

#ifndef HCB_LEAVE_BWD_DEPTH
#define HCB_LEAVE_BWD_DEPTH 1
#endif
#ifndef HCB_LEAVE_BWD_PER
#define HCB_LEAVE_BWD_PER 2
#endif

namespace hcb {

// Every sum that the gradient needs is linear in what is read, up to the
// factor rho of y's norm: with q = act(gate) and e = w q y,
//   dP_ij = <D_i, x_j>,  db_i = scale rho <D_i, e>,
//   <g, y> = scale sum_i b_i <D_i, e>
// so one pass over the row finds S^2 + S + 1 sums and writes dx.  It keeps
// q dv and act'(gate) w y dv (dv = sum_i b_i D_i), of which a second one
// writes dy, dgate and the weight's shares.
// NEXT adds a run of items before it: D_i = dout_i + a_i du with du from dh,
// as in enter_backward_kernel.
template <int SP, class TX, class TY, int V, bool ODD, bool NEXT>
struct LeaveBackward {
  using RX = Row<TX, V, ODD>;
  using RY = Row<TY, V, ODD>;
  using Co = Coefficients<SP, true, true, NEXT>;
  static constexpr int R = SP * SP + SP + 1;
  using Sum = GroupSum<R>;
  using SumNext = GroupSum<2 * SP>;
  static constexpr int DEPTH = HCB_LEAVE_BWD_DEPTH;
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

template <int SP, bool EXACT, class TX, class TY, int V, bool ODD, bool NEXT>
__global__ void __launch_bounds__(SP == 8 ? 256 : kMaxGroup, 1) leave_backward_kernel(const Params p) {
  using E = LeaveBackward<SP, TX, TY, V, ODD, NEXT>;
  using RX = typename E::RX;
  using RY = typename E::RY;
  using Co = typename E::Co;
  using Sum = typename E::Sum;
  constexpr int R = E::R, DEPTH = E::DEPTH;
  extern __shared__ __align__(16) char smem[];
  const int G = p.G, NG = blockDim.x / G, group = threadIdx.x / G, l = threadIdx.x % G;
  const int lane = threadIdx.x & 31, warp = l / 32, C = p.C, S = EXACT ? SP : p.S, GV = G * V;
  const int K = (C + GV - 1) / GV;
  const bool mix = p.P.p != nullptr, gated = p.gate != nullptr;
  const int SLOT = E::slot(mix, gated), ITEM = E::item(gated, p.direct), KB = E::kb(p.direct);
  char* of_group = smem + group * p.group_bytes;
  char* ring = of_group + warp * p.warp_bytes;
  char* item0 = ring + DEPTH * SLOT;
  float* co_all = reinterpret_cast<float*>(of_group + G / 32 * p.warp_bytes);
  float* co_s = co_all + warp * Co::FLOATS;
  float* red = co_all + G / 32 * Co::FLOATS;
  float* red_next = red + Sum::floats(G);
  Sum::clear(red, G, l);
  if constexpr (NEXT) E::SumNext::clear(red_next, G, l);
  group_sync(G, group);
  float* row_dw = p.direct && p.dw ? p.dw + int64_t(blockIdx.x) * pitch(C) : nullptr;
  float* row_dwn = NEXT && p.direct && p.dwn ? p.dwn + int64_t(blockIdx.x) * pitch(C) : nullptr;
  int turn = 0, turn_next = 0;
  const float inv_c = 1.0f / static_cast<float>(C);
  const uint32_t step = gridDim.x * NG;
  uint32_t t = blockIdx.x * NG + group;

  const int NI = NEXT ? 2 * K : K;
  uint32_t ta = t;
  int ca = l * V, ia = 0;
  char* slot_a = ring;
  auto copy_next = [&] {
    if (ta < p.T && ca < C) {
      if (NEXT && ia < K) {
        const TX* o = at_row<TX>(p.out_in, ta, p.out_ts) + ca;
#pragma unroll
        for (int i = 0; i < SP; ++i)
          if (EXACT || i < S) RX::copy(slot_a + i * RX::SLOT, lane, o + i * p.out_ss, C - ca);
        RY::copy(slot_a + E::Y, lane, at_row<TY>(p.dh, ta, p.dh_ts) + ca, C - ca);
      } else {
        const TX* d = at_row<TX>(p.dout, ta, p.dout_ts) + ca;
#pragma unroll
        for (int i = 0; i < SP; ++i)
          if (EXACT || i < S) RX::copy(slot_a + i * RX::SLOT, lane, d + i * p.dout_ss, C - ca);
        RY::copy(slot_a + E::Y, lane, at_row<TY>(p.y, ta, p.y_ts) + ca, C - ca);
        if (gated) RY::copy(slot_a + E::GATE, lane, at_row<TY>(p.gate, ta, p.gate_ts) + ca, C - ca);
        if (mix) {
          const TX* x = at_row<TX>(p.x, ta, p.x_ts) + ca;
#pragma unroll
          for (int i = 0; i < SP; ++i)
            if (EXACT || i < S) RX::copy(slot_a + E::X + i * RX::SLOT, lane, x + i * p.x_ss, C - ca);
        }
      }
    }
    copy_commit();
    ca += GV;
    ++ia;
    if (NEXT && ia == K) ca = l * V;
    if (ia == NI) ia = 0, ca = l * V, ta += step;
    if constexpr (DEPTH > 1) slot_a = slot_a == ring + (DEPTH - 1) * SLOT ? ring : slot_a + SLOT;
  };
  Co co;
  co.init(p, lane);
  if (t < p.T) co.fetch(t);
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) copy_next();
  {
    const float z[V] = {};
    char* item = item0;
    for (int c = l * V; c < C; c += GV, item += ITEM) {
      if (p.direct) {
        if (row_dw) keep<V, 16>(reinterpret_cast<char*>(row_dw + c), 0, z);
        if (NEXT && row_dwn) keep<V, 16>(reinterpret_cast<char*>(row_dwn + c), 0, z);
      } else {
        keep<V>(item + E::KW, lane, z);
        if constexpr (NEXT) keep<V>(item + E::KN, lane, z);
      }
    }
  }

  const char* slot = ring;
  for (; t < p.T; t += step) {
    co.spread(co_s, lane);
    if (t + step < p.T) co.fetch(t + step);
    float a[SP], r_next = 0.0f, k_next = 0.0f;
    const TY* dh = nullptr;
    if constexpr (NEXT) {
      const TX* o = at_row<TX>(p.out_in, t, p.out_ts);
      dh = at_row<TY>(p.dh, t, p.dh_ts);
      Co::read(co_s, Co::NB, a);
      float sum[2 * SP];
#pragma unroll
      for (int s = 0; s < 2 * SP; ++s) sum[s] = 0.0f;
      char* item = item0;
      for (int c = l * V, k = 0; k < K; ++k, c += GV, item += ITEM) {
        float w[V];
        if (c < C) p.wn.load<V, ODD>(c, C - c, w);
        copy_wait<DEPTH - 1>();
        if (c < C) {
          float xv[SP][V], g[V], u[V];
#pragma unroll
          for (int i = 0; i < SP; ++i) {
            if (EXACT || i < S) {
              RX::arrived(slot + i * RX::SLOT, lane, o + i * p.out_ss + c, xv[i]);
            } else {
#pragma unroll
              for (int j = 0; j < V; ++j) xv[i][j] = 0.0f;
            }
          }
          if (p.direct)
            RY::arrived(slot + E::Y, lane, dh + c, g);
          else
            RY::arrived_kept(slot + E::Y, lane, dh + c, g, item + E::KH);
#pragma unroll
          for (int j = 0; j < V; ++j) {
            g[j] *= w[j];
            u[j] = 0.0f;
#pragma unroll
            for (int s = 0; s < SP; ++s) u[j] += a[s] * xv[s][j];
#pragma unroll
            for (int s = 0; s < SP; ++s) {
              sum[s] += g[j] * xv[s][j];
              sum[SP + s] += u[j] * xv[s][j];
            }
          }
          keep<V>(item, lane, u);
        }
        copy_next();
        if constexpr (DEPTH > 1) slot = slot == ring + (DEPTH - 1) * SLOT ? ring : slot + SLOT;
      }
      float total[1];
      E::SumNext::run(sum, total, red_next, turn_next, G, group, lane, warp);
      float gu = 0.0f, uu = 0.0f;
#pragma unroll
      for (int s = 0; s < SP; ++s) {
        gu += a[s] * of_total(total, s);
        uu += a[s] * of_total(total, SP + s);
      }
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
    float P[SP][SP], b[SP], sum[R];
    Co::read(co_s, Co::NP, b);
#pragma unroll
    for (int i = 0; i < SP; ++i) Co::read(co_s, i * SP, P[i]);
#pragma unroll
    for (int i = 0; i < R; ++i) sum[i] = 0.0f;
    TX* dx = p.dx ? static_cast<TX*>(p.dx) + uint64_t(t) * uint32_t(S * C) : nullptr;
    char* item = item0;
    for (int c = l * V, k = 0; k < K; ++k, c += GV, item += ITEM) {
      float w[V];
      if (c < C) p.w.load<V, ODD>(c, C - c, w);
      copy_wait<DEPTH - 1>();
      if (c >= C) {
        copy_next();
        if constexpr (DEPTH > 1) slot = slot == ring + (DEPTH - 1) * SLOT ? ring : slot + SLOT;
        continue;
      }
      float D[SP][V], e[V], g[V];
#pragma unroll
      for (int i = 0; i < SP; ++i) {
        if (EXACT || i < S) {
          RX::arrived(slot + i * RX::SLOT, lane, dout + i * p.dout_ss + c, D[i]);
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j) D[i][j] = 0.0f;
        }
      }
      if (p.direct)
        RY::arrived(slot + E::Y, lane, y + c, e);
      else
        RY::arrived_kept(slot + E::Y, lane, y + c, e, item + E::KY);
      if (gated) RY::arrived(slot + E::GATE, lane, gate + c, g);
      if constexpr (NEXT) {
        float u[V], h[V], wn[V];
        kept<V>(item, lane, u);
        if (p.direct)
          RY::load(dh + c, h, C - c);
        else
          RY::kept(item + E::KH, lane, h);
        p.wn.load<V, ODD>(c, C - c, wn);
        if (p.dwn) {
          float d[V];
#pragma unroll
          for (int j = 0; j < V; ++j) d[j] = h[j] * (u[j] * r_next);
          add_share<V>(item + E::KN, lane, row_dwn ? row_dwn + c : nullptr, d);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
          u[j] = r_next * (h[j] * wn[j] - k_next * u[j]);
#pragma unroll
          for (int i = 0; i < SP; ++i) D[i][j] += a[i] * u[j];
        }
      }
      if (mix) {
#pragma unroll
        for (int q = 0; q < SP; ++q) {
          if (EXACT || q < S) {
            float xv[V];
            RX::arrived(slot + E::X + q * RX::SLOT, lane, x + q * p.x_ss + c, xv);
#pragma unroll
            for (int i = 0; i < SP; ++i)
#pragma unroll
              for (int j = 0; j < V; ++j) sum[i * SP + q] += D[i][j] * xv[j];
          }
        }
      }
      copy_next();
      if constexpr (DEPTH > 1) slot = slot == ring + (DEPTH - 1) * SLOT ? ring : slot + SLOT;
      if (dx) {
#pragma unroll
        for (int q = 0; q < SP; ++q) {
          if (EXACT || q < S) {
            if (mix) {
              float d[V];
#pragma unroll
              for (int j = 0; j < V; ++j) {
                d[j] = P[0][q] * D[0][j];
#pragma unroll
                for (int i = 1; i < SP; ++i) d[j] += P[i][q] * D[i][j];
              }
              RX::store(dx + q * C + c, d, C - c);
            } else {
              RX::store(dx + q * C + c, D[q], C - c);
            }
          }
        }
      }
      float dv[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        dv[j] = 0.0f;
#pragma unroll
        for (int i = 0; i < SP; ++i) dv[j] += b[i] * D[i][j];
      }
#pragma unroll
      for (int j = 0; j < V; ++j) {
        sum[SP * SP + SP] += e[j] * e[j];
        e[j] *= w[j];
      }
      if (gated) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          float q, slope;
          gate_of(p.act, g[j], q, slope);
          g[j] = slope * e[j] * dv[j];
          e[j] *= q;
          dv[j] *= q;
        }
        keep<V>(item + KB, lane, g);
      }
      keep<V>(item, lane, dv);
#pragma unroll
      for (int i = 0; i < SP; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) sum[SP * SP + i] += D[i][j] * e[j];
    }
    float total[Sum::CH];
    Sum::run(sum, total, red, turn, G, group, lane, warp);
    const float rho = p.norm ? rsqrtf(of_total(total, SP * SP + SP) * inv_c + p.eps) : 1.0f;
    float gy = 0.0f;
#pragma unroll
    for (int i = 0; i < SP; ++i) gy += b[i] * of_total(total, SP * SP + i);
    const float sr = p.scale * rho;
    const float k_y = p.norm ? sr * gy * inv_c * rho * rho : 0.0f;
    if (warp == 0) {
#pragma unroll
      for (int ch = 0; ch < Sum::CH; ++ch) {
        const int i = ch * 32 + lane;
        if (i < SP * SP) {
          if (p.dP && i / SP < S && i % SP < S)
            put_any(p.dP, p.P.bf16, (int64_t(t) * S + i / SP) * S + i % SP, total[ch]);
        } else if (i < SP * SP + S) {
          if (p.db) put_any(p.db, p.b.bf16, int64_t(t) * S + i - SP * SP, sr * total[ch]);
        }
      }
    }
    TY* dy = p.dy ? static_cast<TY*>(p.dy) + uint64_t(t) * uint32_t(C) : nullptr;
    TY* dgate = p.dgate ? static_cast<TY*>(p.dgate) + uint64_t(t) * uint32_t(C) : nullptr;
    item = item0;
    for (int c = l * V; c < C; c += GV, item += ITEM) {
      float yv[V], w[V], d[V];
      if (p.direct)
        RY::load(y + c, yv, C - c);
      else
        RY::kept(item + E::KY, lane, yv);
      p.w.load<V, ODD>(c, C - c, w);
      kept<V>(item, lane, d);
#pragma unroll
      for (int j = 0; j < V; ++j) d[j] *= sr;
      if (dgate) {
        float g[V];
        kept<V>(item + KB, lane, g);
#pragma unroll
        for (int j = 0; j < V; ++j) g[j] *= sr;
        RY::store(dgate + c, g, C - c);
      }
      if (p.dw) {
        float z[V];
#pragma unroll
        for (int j = 0; j < V; ++j) z[j] = d[j] * yv[j];
        add_share<V>(item + E::KW, lane, row_dw ? row_dw + c : nullptr, z);
      }
      if (dy) {
#pragma unroll
        for (int j = 0; j < V; ++j) d[j] = d[j] * w[j] - k_y * yv[j];
        RY::store(dy + c, d, C - c);
      }
    }
  }
  copy_wait_all();
  if (!p.direct && (p.dw || (NEXT && p.dwn))) {
    __syncthreads();
    const int64_t row = int64_t(blockIdx.x) * pitch(C);
    const char* first = smem + warp * p.warp_bytes + DEPTH * SLOT;
    if (p.dw) sum_shares<V>(first + E::KW, p, NG, ITEM, p.dw + row);
    if (NEXT && p.dwn) sum_shares<V>(first + E::KN, p, NG, ITEM, p.dwn + row);
  }
}

namespace {

template <bool NEXT>
struct Backward {
  const Params& p;
  int* rows;
  cudaStream_t s;
  template <int SP, bool EXACT, class TX, class TY, int V, bool ODD>
  cudaError_t operator()() const {
    using E = LeaveBackward<SP, TX, TY, V, ODD, NEXT>;
    const bool mix = p.P.p != nullptr, gated = p.gate != nullptr;
    return launch<leave_backward_kernel<SP, EXACT, TX, TY, V, ODD, NEXT>>(
        p, shape_of(p.T, p.C, V, HCB_LEAVE_BWD_PER, SP == 8 ? 256 : kMaxGroup), V,
        [&](int G, int direct) {
          return Need{E::DEPTH * E::slot(mix, gated), E::item(gated, direct),
                      4 * (G / 32 * E::Co::FLOATS + E::Sum::floats(G) + (NEXT ? E::SumNext::floats(G) : 0))};
        },
        p.dw || p.dwn ? kMaxRows : 1 << 30, rows, s);
  }
};

}  // namespace

cudaError_t leave_backward(const Params& p, int x_bf16, int y_bf16, bool vec, int* rows, cudaStream_t s) {
  if (p.dh) return by_streams(p.S, x_bf16, y_bf16, vec, Backward<true>{p, rows, s});
  return by_streams(p.S, x_bf16, y_bf16, vec, Backward<false>{p, rows, s});
}

}  // namespace hcb
