// hcb_leave.cu -- the block's output, normalised, gated and scaled, written
// back into the mixed residual streams, and the next block's input from the
// result (hcb_leave of include/hc_block.h).
#include "hcb_common.cuh"

#ifndef HCB_LEAVE_DEPTH
#define HCB_LEAVE_DEPTH 2
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
  // y and the gate take the streams' place in a slot where both have vectors
  // of one size; otherwise a thread's part of a slot would not be its own for
  // both kinds of items, and they lie behind the streams
  static constexpr bool SHARED = RX::SLOT == RY::SLOT;
  static __host__ __device__ constexpr int y_at(int S) { return SHARED ? 0 : S * RX::SLOT; }
  static __host__ __device__ constexpr int slot(int S) {
    return SHARED && S >= 2 ? S * RX::SLOT : y_at(S) + 2 * RY::SLOT;
  }
  static size_t bytes(int S, int C, int G) {
    return size_t(G) * (DEPTH * slot(S) + items(C, V, G) * V * 4) +
           4 * (G / 32 * Co::FLOATS + 2 * ((Sum::floats(G) + 3) / 4 * 4));
  }
};

template <int SP, class TX, class TY, int V, bool ODD>
__global__ void __launch_bounds__(SP == 8 ? 256 : kMaxGroup, 1) leave_kernel(const Params p) {
  using E = Leave<SP, TX, TY, V, ODD>;
  using RX = typename E::RX;
  using RY = typename E::RY;
  using Co = typename E::Co;
  constexpr int DEPTH = E::DEPTH;
  extern __shared__ __align__(16) char smem[];
  const int G = p.G, NG = blockDim.x / G, group = threadIdx.x / G, l = threadIdx.x % G;
  const int lane = threadIdx.x & 31, warp = l / 32, C = p.C, S = p.S;
  const int K = (C + V * G - 1) / (V * G);
  const int slot_bytes = G * E::slot(S);
  char* ring = smem + size_t(group) * p.group_bytes;
  float* u_s = reinterpret_cast<float*>(ring + DEPTH * slot_bytes);  // w act y, then u
  float* co_s = u_s + K * V * G + warp * Co::FLOATS;
  float* red = u_s + K * V * G + G / 32 * Co::FLOATS;
  float* red_next = red + (GroupSum<1>::floats(G) + 3) / 4 * 4;
  int turn = 0, turn_next = 0;
  const float inv_c = 1.0f / static_cast<float>(C);
  const bool mix = p.P.p != nullptr;
  const int64_t step = int64_t(gridDim.x) * NG;
  int64_t t = int64_t(blockIdx.x) * NG + group;

  int64_t ta = t;
  int ia = 0, slot_a = 0;
  auto copy_next = [&] {
    const bool second = ia >= K;
    const int c = ((second ? ia - K : ia) * G + l) * V;
    if (ta < p.T && c < C) {
      char* s = ring + slot_a * slot_bytes;
      if (second) {
        const TX* x = static_cast<const TX*>(p.x) + ta * p.x_ts + c;
#pragma unroll
        for (int i = 0; i < SP; ++i)
          if (i < S) RX::copy(s + i * G * RX::SLOT, G, l, x + i * p.x_ss, C - c);
      } else {
        s += G * E::y_at(S);
        RY::copy(s, G, l, static_cast<const TY*>(p.y) + ta * p.y_ts + c, C - c);
        if (p.gate)
          RY::copy(s + G * RY::SLOT, G, l, static_cast<const TY*>(p.gate) + ta * p.gate_ts + c, C - c);
      }
    }
    copy_commit();
    if (++ia == 2 * K) ia = 0, ta += step;
    if (++slot_a == DEPTH) slot_a = 0;
  };
  Co co;
  if (t < p.T) co.fetch(p, t, lane);
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) copy_next();

  int slot = 0;
  for (; t < p.T; t += step) {
    co.spread(co_s, lane);
    if (t + step < p.T) co.fetch(p, t + step, lane);
    const TX* x = static_cast<const TX*>(p.x) + t * p.x_ts;
    const TY* y = static_cast<const TY*>(p.y) + t * p.y_ts;
    const TY* gate = p.gate ? static_cast<const TY*>(p.gate) + t * p.gate_ts : nullptr;
    float ss[1] = {0.0f};
    for (int k = 0; k < K; ++k) {
      const int c = (k * G + l) * V;
      float v[V], g[V], w[V];
      if (c < C) p.w.load<V, ODD>(c, C - c, w);
      copy_wait<DEPTH - 1>();
      if (c < C) {
        const char* s = ring + slot * slot_bytes + G * E::y_at(S);
        RY::arrived(s, G, l, y + c, v);
        if (gate) RY::arrived(s + G * RY::SLOT, G, l, gate + c, g);
      }
      copy_next();
      if (++slot == DEPTH) slot = 0;
      if (c < C) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          ss[0] += v[j] * v[j];
          v[j] *= w[j];
        }
        if (gate) {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            float q, slope;
            gate_of(p.act, g[j], q, slope);
            v[j] *= q;
          }
        }
        keep<V>(u_s, G, l, k, v);
      }
    }
    float rho = p.scale;
    if (p.norm) {
      float total[1];
      GroupSum<1>::run(ss, total, red, turn, G, group, lane, warp);
      rho *= rsqrtf(of_total(total, 0) * inv_c + p.eps);
    }
    float P[SP][SP], b[SP], a[SP];
    Co::read(co_s, Co::NP, b);
    Co::read(co_s, Co::NB, a);
#pragma unroll
    for (int i = 0; i < SP; ++i) {
      Co::read(co_s, i * SP, P[i]);
      b[i] *= rho;
    }
    TX* out = static_cast<TX*>(p.out) + t * S * C;
    ss[0] = 0.0f;
    for (int k = 0; k < K; ++k) {
      const int c = (k * G + l) * V;
      float v[V], xv[SP][V];
      if (c < C) kept<V>(u_s, G, l, k, v);
      copy_wait<DEPTH - 1>();
      if (c < C) {
        const char* s = ring + slot * slot_bytes;
#pragma unroll
        for (int i = 0; i < SP; ++i) {
          if (i < S) {
            RX::arrived(s + i * G * RX::SLOT, G, l, x + i * p.x_ss + c, xv[i]);
          } else {
#pragma unroll
            for (int j = 0; j < V; ++j) xv[i][j] = 0.0f;
          }
        }
      }
      copy_next();
      if (++slot == DEPTH) slot = 0;
      if (c < C) {
        float u[V];
#pragma unroll
        for (int j = 0; j < V; ++j) u[j] = 0.0f;
#pragma unroll
        for (int i = 0; i < SP; ++i) {
          if (i < S) {
            float o[V];
#pragma unroll
            for (int j = 0; j < V; ++j) o[j] = b[i] * v[j];
            if (mix) {
#pragma unroll
              for (int q = 0; q < SP; ++q)
#pragma unroll
                for (int j = 0; j < V; ++j) o[j] += P[i][q] * xv[q][j];
            } else {
#pragma unroll
              for (int j = 0; j < V; ++j) o[j] += xv[i][j];
            }
            RX::store(out + int64_t(i) * C + c, o, C - c);
            if (p.h) {
#pragma unroll
              for (int j = 0; j < V; ++j) u[j] += a[i] * RX::round(o[j]);
            }
          }
        }
        if (p.h) {
#pragma unroll
          for (int j = 0; j < V; ++j) ss[0] += u[j] * u[j];  // past C: y, x and so u are zeros
          keep<V>(u_s, G, l, k, u);
        }
      }
    }
    if (p.h) {
      float total[1];
      GroupSum<1>::run(ss, total, red_next, turn_next, G, group, lane, warp);
      const float r = rsqrtf(of_total(total, 0) * inv_c + p.eps_next);
      TY* h = static_cast<TY*>(p.h) + t * C;
      for (int k = 0; k < K; ++k) {
        const int c = (k * G + l) * V;
        if (c >= C) break;
        float u[V], w[V];
        kept<V>(u_s, G, l, k, u);
        p.wn.load<V, ODD>(c, C - c, w);
#pragma unroll
        for (int j = 0; j < V; ++j) u[j] *= r * w[j];
        RY::store(h + c, u, C - c);
      }
    }
  }
  copy_wait_all();
}

namespace {

struct Forward {
  const Params& p;
  cudaStream_t s;
  template <int SP, class TX, class TY, int V, bool ODD>
  cudaError_t operator()() const {
    using E = Leave<SP, TX, TY, V, ODD>;
    int direct, grid;
    const Shape sh = fitted(shape_of(p.T, p.C, V, SP == 8 ? 256 : kMaxGroup), false, &direct,
                            [&](int G, bool) { return E::bytes(p.S, p.C, G); });
    return launch<leave_kernel<SP, TX, TY, V, ODD>>(p, sh, E::bytes(p.S, p.C, sh.G), 1 << 30, &grid, s);
  }
};

}  // namespace

cudaError_t leave_forward(const Params& p, int x_bf16, int y_bf16, bool vec, cudaStream_t s) {
  return by_streams(p.S, x_bf16, y_bf16, vec, Forward{p, s});
}

}  // namespace hcb
