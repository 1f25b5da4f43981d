// hcb_leave_bwd.cu -- the gradient of leave and of leave_enter
// (hcb_leave_backward of include/hc_block.h).
#include "hcb_common.cuh"

#ifndef HCB_LEAVE_BWD_DEPTH
#define HCB_LEAVE_BWD_DEPTH 1
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
  static __host__ __device__ constexpr int slot(int S, bool mix, bool gate) {
    return (mix ? 2 : 1) * S * RX::SLOT + (gate ? 2 : 1) * RY::SLOT;
  }
  static size_t bytes(int S, int C, int G, bool mix, bool gate, int weights, bool direct) {
    const int kept = 4 + (gate ? 4 : 0) + (direct ? 0 : sizeof(TY) + (NEXT ? sizeof(TY) : 0) + 4 * weights);
    return size_t(G) * (DEPTH * slot(S, mix, gate) + items(C, V, G) * V * kept) +
           4 * (G / 32 * Co::FLOATS + (Sum::floats(G) + 3) / 4 * 4 + (NEXT ? (SumNext::floats(G) + 3) / 4 * 4 : 0));
  }
};

template <int SP, class TX, class TY, int V, bool ODD, bool NEXT>
__global__ void __launch_bounds__(SP == 8 ? 256 : kMaxGroup, 1) leave_backward_kernel(const Params p) {
  using E = LeaveBackward<SP, TX, TY, V, ODD, NEXT>;
  using RX = typename E::RX;
  using RY = typename E::RY;
  using Co = typename E::Co;
  using Sum = typename E::Sum;
  constexpr int R = E::R, DEPTH = E::DEPTH;
  extern __shared__ __align__(16) char smem[];
  const int G = p.G, NG = blockDim.x / G, group = threadIdx.x / G, l = threadIdx.x % G;
  const int lane = threadIdx.x & 31, warp = l / 32, C = p.C, S = p.S;
  const int K = (C + V * G - 1) / (V * G);
  const bool mix = p.P.p != nullptr, gated = p.gate != nullptr;
  const int slot_bytes = G * E::slot(S, mix, gated);
  char* ring = smem + size_t(group) * p.group_bytes;
  float* a_s = reinterpret_cast<float*>(ring + DEPTH * slot_bytes);  // NEXT: u first; then q dv
  float* b_s = a_s + K * V * G;                                     // act' w y dv
  char* y_s = reinterpret_cast<char*>(b_s + (gated ? K * V * G : 0));
  const int row_kept = p.direct ? 0 : K * V * G * static_cast<int>(sizeof(TY));
  char* dh_s = y_s + row_kept;
  float* co_all = reinterpret_cast<float*>(dh_s + (NEXT ? row_kept : 0));
  float* co_s = co_all + warp * Co::FLOATS;
  float* red = co_all + G / 32 * Co::FLOATS;
  float* red_next = red + (Sum::floats(G) + 3) / 4 * 4;
  float* shares = red_next + (NEXT ? (E::SumNext::floats(G) + 3) / 4 * 4 : 0);
  WeightShare<V> dw = {shares, p.direct ? p.dw + int64_t(blockIdx.x) * pitch(C) : nullptr};
  WeightShare<V> dwn = {shares + (p.dw ? K * V * G : 0), p.direct ? p.dwn + int64_t(blockIdx.x) * pitch(C) : nullptr};
  int turn = 0, turn_next = 0;
  const float inv_c = 1.0f / static_cast<float>(C);
  const int64_t step = int64_t(gridDim.x) * NG;
  int64_t t = int64_t(blockIdx.x) * NG + group;

  const int NI = NEXT ? 2 * K : K;
  int64_t ta = t;
  int ia = 0, slot_a = 0;
  auto copy_next = [&] {
    const bool first = NEXT && ia < K;
    const int c = ((NEXT && !first ? ia - K : ia) * G + l) * V;
    if (ta < p.T && c < C) {
      char* s = ring + slot_a * slot_bytes;
      if (first) {
        const TX* o = static_cast<const TX*>(p.out_in) + ta * p.out_ts + c;
#pragma unroll
        for (int i = 0; i < SP; ++i)
          if (i < S) RX::copy(s + i * G * RX::SLOT, G, l, o + i * p.out_ss, C - c);
        RY::copy(s + S * G * RX::SLOT, G, l, static_cast<const TY*>(p.dh) + ta * p.dh_ts + c, C - c);
      } else {
        const TX* d = static_cast<const TX*>(p.dout) + ta * p.dout_ts + c;
#pragma unroll
        for (int i = 0; i < SP; ++i)
          if (i < S) RX::copy(s + i * G * RX::SLOT, G, l, d + i * p.dout_ss, C - c);
        s += S * G * RX::SLOT;
        RY::copy(s, G, l, static_cast<const TY*>(p.y) + ta * p.y_ts + c, C - c);
        s += G * RY::SLOT;
        if (gated) {
          RY::copy(s, G, l, static_cast<const TY*>(p.gate) + ta * p.gate_ts + c, C - c);
          s += G * RY::SLOT;
        }
        if (mix) {
          const TX* x = static_cast<const TX*>(p.x) + ta * p.x_ts + c;
#pragma unroll
          for (int i = 0; i < SP; ++i)
            if (i < S) RX::copy(s + i * G * RX::SLOT, G, l, x + i * p.x_ss, C - c);
        }
      }
    }
    copy_commit();
    if (++ia == NI) ia = 0, ta += step;
    if (++slot_a == DEPTH) slot_a = 0;
  };
  Co co;
  if (t < p.T) co.fetch(p, t, lane);
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) copy_next();
  if (p.dw) dw.zero(G, l, K, C);
  if (NEXT && p.dwn) dwn.zero(G, l, K, C);

  int slot = 0;
  for (; t < p.T; t += step) {
    co.spread(co_s, lane);
    if (t + step < p.T) co.fetch(p, t + step, lane);
    float a[SP], r_next = 0.0f, k_next = 0.0f;
    if constexpr (NEXT) {
      const TX* o = static_cast<const TX*>(p.out_in) + t * p.out_ts;
      const TY* dh = static_cast<const TY*>(p.dh) + t * p.dh_ts;
      Co::read(co_s, Co::NB, a);
      float sum[2 * SP];
#pragma unroll
      for (int s = 0; s < 2 * SP; ++s) sum[s] = 0.0f;
      for (int k = 0; k < K; ++k) {
        const int c = (k * G + l) * V;
        float xv[SP][V], g[V], w[V], u[V];
        if (c < C) p.wn.load<V, ODD>(c, C - c, w);
        copy_wait<DEPTH - 1>();
        if (c < C) {
          const char* s = ring + slot * slot_bytes;
#pragma unroll
          for (int i = 0; i < SP; ++i) {
            if (i < S) {
              RX::arrived(s + i * G * RX::SLOT, G, l, o + i * p.out_ss + c, xv[i]);
            } else {
#pragma unroll
              for (int j = 0; j < V; ++j) xv[i][j] = 0.0f;
            }
          }
          RY::arrived(s + S * G * RX::SLOT, G, l, dh + c, g);
        }
        copy_next();
        if (++slot == DEPTH) slot = 0;
        if (c < C) {
          if (!p.direct) keep_row<TY, V>(dh_s, G, l, k, g);
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
          keep<V>(a_s, G, l, k, u);
        }
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
          put_any(p.da, p.a.bf16, t * S + lane, r_next * (total[0] - k_next * u_x));
      }
    }
    const TX* dout = static_cast<const TX*>(p.dout) + t * p.dout_ts;
    const TX* x = static_cast<const TX*>(p.x) + t * p.x_ts;
    const TY* y = static_cast<const TY*>(p.y) + t * p.y_ts;
    const TY* gate = static_cast<const TY*>(p.gate) + t * p.gate_ts;
    float P[SP][SP], b[SP], sum[R];
    Co::read(co_s, Co::NP, b);
#pragma unroll
    for (int i = 0; i < SP; ++i) Co::read(co_s, i * SP, P[i]);
#pragma unroll
    for (int i = 0; i < R; ++i) sum[i] = 0.0f;
    TX* dx = p.dx ? static_cast<TX*>(p.dx) + t * S * C : nullptr;
    for (int k = 0; k < K; ++k) {
      const int c = (k * G + l) * V;
      float w[V];
      if (c < C) p.w.load<V, ODD>(c, C - c, w);
      copy_wait<DEPTH - 1>();
      if (c >= C) {
        copy_next();
        if (++slot == DEPTH) slot = 0;
        continue;
      }
      float D[SP][V], e[V], g[V];
      const char* s = ring + slot * slot_bytes;
#pragma unroll
      for (int i = 0; i < SP; ++i) {
        if (i < S) {
          RX::arrived(s + i * G * RX::SLOT, G, l, dout + i * p.dout_ss + c, D[i]);
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j) D[i][j] = 0.0f;
        }
      }
      s += S * G * RX::SLOT;
      RY::arrived(s, G, l, y + c, e);
      s += G * RY::SLOT;
      if (gated) {
        RY::arrived(s, G, l, gate + c, g);
        s += G * RY::SLOT;
      }
      if constexpr (NEXT) {
        float u[V], h[V], wn[V];
        kept<V>(a_s, G, l, k, u);
        if (p.direct)
          RY::load(static_cast<const TY*>(p.dh) + t * p.dh_ts + c, h, C - c);
        else
          kept_row<TY, V>(dh_s, G, l, k, h);
        p.wn.load<V, ODD>(c, C - c, wn);
        if (p.dwn) {
          float d[V];
#pragma unroll
          for (int j = 0; j < V; ++j) d[j] = h[j] * (u[j] * r_next);
          dwn.add(G, l, k, d);
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
          if (q < S) {
            float xv[V];
            RX::arrived(s + q * G * RX::SLOT, G, l, x + q * p.x_ss + c, xv);
#pragma unroll
            for (int i = 0; i < SP; ++i)
#pragma unroll
              for (int j = 0; j < V; ++j) sum[i * SP + q] += D[i][j] * xv[j];
          }
        }
      }
      copy_next();
      if (++slot == DEPTH) slot = 0;
      if (dx) {
#pragma unroll
        for (int q = 0; q < SP; ++q) {
          if (q < S) {
            float d[V];
            if (mix) {
#pragma unroll
              for (int j = 0; j < V; ++j) {
                d[j] = P[0][q] * D[0][j];
#pragma unroll
                for (int i = 1; i < SP; ++i) d[j] += P[i][q] * D[i][j];
              }
            } else {
#pragma unroll
              for (int j = 0; j < V; ++j) d[j] = D[q][j];
            }
            RX::store(dx + int64_t(q) * C + c, d, C - c);
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
      if (!p.direct) keep_row<TY, V>(y_s, G, l, k, e);
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
        keep<V>(b_s, G, l, k, g);
      }
      keep<V>(a_s, G, l, k, dv);
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
            put_any(p.dP, p.P.bf16, (t * S + i / SP) * S + i % SP, total[ch]);
        } else if (i < SP * SP + S) {
          if (p.db) put_any(p.db, p.b.bf16, t * S + i - SP * SP, sr * total[ch]);
        }
      }
    }
    TY* dy = p.dy ? static_cast<TY*>(p.dy) + t * C : nullptr;
    TY* dgate = p.dgate ? static_cast<TY*>(p.dgate) + t * C : nullptr;
    for (int k = 0; k < K; ++k) {
      const int c = (k * G + l) * V;
      if (c >= C) break;
      float yv[V], w[V], d[V];
      if (p.direct)
        RY::load(y + c, yv, C - c);
      else
        kept_row<TY, V>(y_s, G, l, k, yv);
      p.w.load<V, ODD>(c, C - c, w);
      kept<V>(a_s, G, l, k, d);
#pragma unroll
      for (int j = 0; j < V; ++j) d[j] *= sr;
      if (dgate) {
        float g[V];
        kept<V>(b_s, G, l, k, g);
#pragma unroll
        for (int j = 0; j < V; ++j) g[j] *= sr;
        RY::store(dgate + c, g, C - c);
      }
      if (p.dw) {
        float z[V];
#pragma unroll
        for (int j = 0; j < V; ++j) z[j] = d[j] * yv[j];
        dw.add(G, l, k, z);
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
    const size_t back = size_t(group) * p.group_bytes;
    if (p.dw)
      sum_shares<V>(reinterpret_cast<float*>(reinterpret_cast<char*>(dw.s) - back), p.group_bytes / 4, G, NG, C, p.dw + row);
    if (NEXT && p.dwn)
      sum_shares<V>(reinterpret_cast<float*>(reinterpret_cast<char*>(dwn.s) - back), p.group_bytes / 4, G, NG, C, p.dwn + row);
  }
}

namespace {

template <bool NEXT>
struct Backward {
  const Params& p;
  int* rows;
  cudaStream_t s;
  template <int SP, class TX, class TY, int V, bool ODD>
  cudaError_t operator()() const {
    using E = LeaveBackward<SP, TX, TY, V, ODD, NEXT>;
    Params q = p;
    const int weights = (p.dw != nullptr) + (NEXT && p.dwn != nullptr);
    const bool mix = p.P.p != nullptr, gate = p.gate != nullptr;
    const Shape sh = fitted(shape_of(p.T, p.C, V, SP == 8 ? 256 : kMaxGroup), true, &q.direct,
                            [&](int G, bool direct) { return E::bytes(p.S, p.C, G, mix, gate, weights, direct); });
    return launch<leave_backward_kernel<SP, TX, TY, V, ODD, NEXT>>(
        q, sh, E::bytes(p.S, p.C, sh.G, mix, gate, weights, q.direct), weights ? kMaxRows : 1 << 30, rows, s);
  }
};

}  // namespace

cudaError_t leave_backward(const Params& p, int x_bf16, int y_bf16, bool vec, int* rows, cudaStream_t s) {
  if (p.dh) return by_streams(p.S, x_bf16, y_bf16, vec, Backward<true>{p, rows, s});
  return by_streams(p.S, x_bf16, y_bf16, vec, Backward<false>{p, rows, s});
}

}  // namespace hcb
