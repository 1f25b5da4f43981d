// hcb_leave.cu -- the block's output, normalised, gated and scaled, written
// back into the mixed residual streams, and the next block's input from the
// result (hcb_leave of include/hc_block.h).
#include "hcb_common.cuh"

namespace hcb {

template <int SP, class TX, class TY, int V>
__global__ void __launch_bounds__(kMaxGroup) leave_kernel(const Params p) {
  extern __shared__ __align__(16) float smem[];
  const int G = p.G, NG = blockDim.x / G, group = threadIdx.x / G, l = threadIdx.x % G;
  const int lane = threadIdx.x & 31, warp = l / 32, C = p.C;
  const int CP = p.h ? (C + 3) / 4 * 4 : 0;
  float* u_s = smem + group * CP;
  float* red = smem + NG * CP + group * 2 * GroupSum<1>::floats(G);
  float* red_next = red + GroupSum<1>::floats(G);
  int turn = 0, turn_next = 0;
  const float inv_c = 1.0f / static_cast<float>(C);
  const bool mix = p.P.p != nullptr;
  for (int64_t t = int64_t(blockIdx.x) * NG + group; t < p.T; t += int64_t(gridDim.x) * NG) {
    const TX* x = static_cast<const TX*>(p.x) + t * p.x_ts;
    const TY* y = static_cast<const TY*>(p.y) + t * p.y_ts;
    const TY* gate = p.gate ? static_cast<const TY*>(p.gate) + t * p.gate_ts : nullptr;
    float rho = 1.0f;
    if (p.norm) {
      float ss[1] = {0.0f};
#pragma unroll 2
      for (int c = l * V; c < C; c += G * V) {
        float yv[V];
        Row<TY, V>::load(y + c, yv);
#pragma unroll
        for (int k = 0; k < V; ++k) ss[0] += yv[k] * yv[k];
      }
      float total[1];
      GroupSum<1>::run(ss, total, red, turn, G, group, lane, warp);
      rho = rsqrtf(of_total(total, 0) * inv_c + p.eps);
    }
    float b[SP], P[SP][SP], a[SP];
#pragma unroll
    for (int i = 0; i < SP; ++i) {
      b[i] = i < p.S ? (p.b.p ? p.b.at(t * p.b_ts + i) : 1.0f) : 0.0f;
      a[i] = i < p.S && p.h ? (p.a.p ? p.a.at(t * p.a_ts + i) : 1.0f) : 0.0f;
#pragma unroll
      for (int j = 0; j < SP; ++j)
        P[i][j] = mix && i < p.S && j < p.S ? p.P.at(t * p.P_ts + i * p.S + j) : 0.0f;
    }
    TX* out = static_cast<TX*>(p.out) + t * p.S * C;
    float ss[1] = {0.0f};
#pragma unroll 1
    for (int c = l * V; c < C; c += G * V) {
      float v[V], w[V], xv[SP][V];
#pragma unroll
      for (int j = 0; j < SP; ++j) {
        if (j < p.S) {
          Row<TX, V>::load(x + j * p.x_ss + c, xv[j]);
        } else {
#pragma unroll
          for (int k = 0; k < V; ++k) xv[j][k] = 0.0f;
        }
      }
      Row<TY, V>::load(y + c, v);
      p.w.load<V>(c, w);
#pragma unroll
      for (int k = 0; k < V; ++k) v[k] *= p.scale * rho * w[k];
      if (gate) {
        float g[V];
        Row<TY, V>::load(gate + c, g);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          float q, slope;
          gate_of(p.act, g[k], q, slope);
          v[k] *= q;
        }
      }
      float u[V];
#pragma unroll
      for (int k = 0; k < V; ++k) u[k] = 0.0f;
#pragma unroll
      for (int i = 0; i < SP; ++i) {
        if (i < p.S) {
          float o[V];
#pragma unroll
          for (int k = 0; k < V; ++k) o[k] = b[i] * v[k];
          if (mix) {
#pragma unroll
            for (int j = 0; j < SP; ++j)
#pragma unroll
              for (int k = 0; k < V; ++k) o[k] += P[i][j] * xv[j][k];
          } else {
#pragma unroll
            for (int k = 0; k < V; ++k) o[k] += xv[i][k];
          }
          Row<TX, V>::store(out + int64_t(i) * C + c, o);
#pragma unroll
          for (int k = 0; k < V; ++k) u[k] += a[i] * Row<TX, V>::round(o[k]);
        }
      }
      if (p.h) {
#pragma unroll
        for (int k = 0; k < V; ++k) ss[0] += u[k] * u[k];
        keep<V>(u_s + c, u);
      }
    }
    if (p.h) {
      float total[1];
      GroupSum<1>::run(ss, total, red_next, turn_next, G, group, lane, warp);
      const float r = rsqrtf(of_total(total, 0) * inv_c + p.eps_next);
      TY* h = static_cast<TY*>(p.h) + t * C;
#pragma unroll 2
      for (int c = l * V; c < C; c += G * V) {
        float u[V], w[V];
        kept<V>(u_s + c, u);
        p.wn.load<V>(c, w);
#pragma unroll
        for (int k = 0; k < V; ++k) u[k] *= r * w[k];
        Row<TY, V>::store(h + c, u);
      }
    }
  }
}

namespace {

struct Forward {
  const Params& p;
  cudaStream_t s;
  template <int SP, class TX, class TY, int V>
  cudaError_t operator()() const {
    const Shape sh = shape_of(p.T, p.C, V, SP == 8 ? 256 : kMaxGroup);
    int grid;
    return launch<leave_kernel<SP, TX, TY, V>>(
        p, sh, sizeof(float) * ((p.h ? padded(p.C) : 0) + 2 * GroupSum<1>::floats(sh.G)), 1 << 30,
        &grid, s);
  }
};

}  // namespace

cudaError_t leave_forward(const Params& p, int x_bf16, int y_bf16, bool vec, cudaStream_t s) {
  return by_streams(p.S, x_bf16, y_bf16, vec, Forward{p, s});
}

}  // namespace hcb
