// hcb_enter.cu -- the block's input from the residual streams and its
// gradient (hcb_enter, hcb_enter_backward of include/hc_block.h).
#include "hcb_common.cuh"

namespace hcb {

// u = sum_s a_s x_s and its mean square in one pass over the row's streams;
// u stays in shared memory (fp32) until r is known, then h = w u r.
template <int SP, class TX, class TY, int V>
__global__ void __launch_bounds__(kMaxGroup) enter_kernel(const Params p) {
  extern __shared__ __align__(16) float smem[];
  const int G = p.G, NG = blockDim.x / G, group = threadIdx.x / G, l = threadIdx.x % G;
  const int lane = threadIdx.x & 31, warp = l / 32, C = p.C;
  const int CP = (C + 3) / 4 * 4;
  float* u_s = smem + group * CP;
  float* red = smem + NG * CP + group * GroupSum<1>::floats(G);
  int turn = 0;
  const float inv_c = 1.0f / static_cast<float>(C);
  for (int64_t t = int64_t(blockIdx.x) * NG + group; t < p.T; t += int64_t(gridDim.x) * NG) {
    const TX* x = static_cast<const TX*>(p.x) + t * p.x_ts;
    float a[SP];
#pragma unroll
    for (int s = 0; s < SP; ++s) a[s] = s < p.S ? (p.a.p ? p.a.at(t * p.a_ts + s) : 1.0f) : 0.0f;
    float ss[1] = {0.0f};
#pragma unroll 2
    for (int c = l * V; c < C; c += G * V) {
      float u[V];
#pragma unroll
      for (int k = 0; k < V; ++k) u[k] = 0.0f;
#pragma unroll
      for (int s = 0; s < SP; ++s) {
        if (s < p.S) {
          float xv[V];
          Row<TX, V>::load(x + s * p.x_ss + c, xv);
#pragma unroll
          for (int k = 0; k < V; ++k) u[k] += a[s] * xv[k];
        }
      }
#pragma unroll
      for (int k = 0; k < V; ++k) ss[0] += u[k] * u[k];
      keep<V>(u_s + c, u);
    }
    float total[1];
    GroupSum<1>::run(ss, total, red, turn, G, group, lane, warp);
    const float r = rsqrtf(of_total(total, 0) * inv_c + p.eps);
    TY* h = static_cast<TY*>(p.h) + t * C;
#pragma unroll 2
    for (int c = l * V; c < C; c += G * V) {
      float u[V], w[V];
      kept<V>(u_s + c, u);
      p.w.load<V>(c, w);
#pragma unroll
      for (int k = 0; k < V; ++k) u[k] *= r * w[k];
      Row<TY, V>::store(h + c, u);
    }
  }
}

// With G = w dh all sums of the gradient are linear in <G, x_s> and <u, x_s>:
// <G, u> = sum a_s <G, x_s>, <u, u> = sum a_s <u, x_s> and
// da_s = r (<G, x_s> - k <u, x_s>), so one pass over the row finds them and
// a second, over what the first kept, writes.
template <int SP, class TX, class TY, int V>
__global__ void __launch_bounds__(kMaxGroup) enter_backward_kernel(const Params p) {
  extern __shared__ __align__(16) float smem[];
  const int G = p.G, NG = blockDim.x / G, group = threadIdx.x / G, l = threadIdx.x % G;
  const int lane = threadIdx.x & 31, warp = l / 32, C = p.C;
  const int CP = (C + 3) / 4 * 4;
  float* u_s = smem + group * 2 * CP;
  float* dw_s = u_s + CP;
  float* red = smem + NG * 2 * CP + group * GroupSum<2 * SP>::floats(G);
  int turn = 0;
  const float inv_c = 1.0f / static_cast<float>(C);
  if (p.dw)
    for (int c = l; c < C; c += G) dw_s[c] = 0.0f;
  group_sync(G, group);
  for (int64_t t = int64_t(blockIdx.x) * NG + group; t < p.T; t += int64_t(gridDim.x) * NG) {
    const TX* x = static_cast<const TX*>(p.x) + t * p.x_ts;
    const TY* dh = static_cast<const TY*>(p.dh) + t * p.dh_ts;
    float a[SP];
#pragma unroll
    for (int s = 0; s < SP; ++s) a[s] = s < p.S ? (p.a.p ? p.a.at(t * p.a_ts + s) : 1.0f) : 0.0f;
    float sum[2 * SP];
#pragma unroll
    for (int s = 0; s < 2 * SP; ++s) sum[s] = 0.0f;
#pragma unroll 1
    for (int c = l * V; c < C; c += G * V) {
      float xv[SP][V], g[V], w[V], u[V];
#pragma unroll
      for (int s = 0; s < SP; ++s) {
        if (s < p.S) {
          Row<TX, V>::load(x + s * p.x_ss + c, xv[s]);
        } else {
#pragma unroll
          for (int k = 0; k < V; ++k) xv[s][k] = 0.0f;
        }
      }
      Row<TY, V>::load(dh + c, g);
      p.w.load<V>(c, w);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        g[k] *= w[k];
        u[k] = 0.0f;
#pragma unroll
        for (int s = 0; s < SP; ++s) u[k] += a[s] * xv[s][k];
#pragma unroll
        for (int s = 0; s < SP; ++s) {
          sum[s] += g[k] * xv[s][k];
          sum[SP + s] += u[k] * xv[s][k];
        }
      }
      keep<V>(u_s + c, u);
    }
    float total[1];
    GroupSum<2 * SP>::run(sum, total, red, turn, G, group, lane, warp);
    float gu = 0.0f, uu = 0.0f;
#pragma unroll
    for (int s = 0; s < SP; ++s) {
      gu += a[s] * of_total(total, s);
      uu += a[s] * of_total(total, SP + s);
    }
    const float r = rsqrtf(uu * inv_c + p.eps);
    const float k_u = gu * inv_c * r * r;
    if (p.da) {
      const float u_x = __shfl_sync(0xffffffffu, total[0], (lane + SP) & 31);
      if (warp == 0 && lane < p.S) put_any(p.da, p.a.bf16, t * p.S + lane, r * (total[0] - k_u * u_x));
    }
    const TX* dres = p.dres ? static_cast<const TX*>(p.dres) + t * p.dres_ts : nullptr;
    TX* dx = static_cast<TX*>(p.dx) + t * p.S * C;
#pragma unroll 1
    for (int c = l * V; c < C; c += G * V) {
      float u[V], g[V], w[V];
      kept<V>(u_s + c, u);
      Row<TY, V>::load(dh + c, g);
      p.w.load<V>(c, w);
      if (p.dw) {
        float d[V];
        kept<V>(dw_s + c, d);
#pragma unroll
        for (int k = 0; k < V; ++k) d[k] += g[k] * (u[k] * r);
        keep<V>(dw_s + c, d);
      }
      if (p.dx == nullptr) continue;
#pragma unroll
      for (int k = 0; k < V; ++k) u[k] = r * (g[k] * w[k] - k_u * u[k]);
#pragma unroll
      for (int s = 0; s < SP; ++s) {
        if (s < p.S) {
          float d[V];
          if (dres) {
            Row<TX, V>::load(dres + s * p.dres_ss + c, d);
#pragma unroll
            for (int k = 0; k < V; ++k) d[k] += a[s] * u[k];
          } else {
#pragma unroll
            for (int k = 0; k < V; ++k) d[k] = a[s] * u[k];
          }
          Row<TX, V>::store(dx + int64_t(s) * C + c, d);
        }
      }
    }
  }
  if (p.dw) {
    __syncthreads();
    for (int c = threadIdx.x; c < C; c += blockDim.x) {
      float d = 0.0f;
      for (int g = 0; g < NG; ++g) d += smem[(g * 2 + 1) * CP + c];
      p.dw[int64_t(blockIdx.x) * C + c] = d;
    }
  }
}

namespace {

struct Forward {
  const Params& p;
  cudaStream_t s;
  template <int SP, class TX, class TY, int V>
  cudaError_t operator()() const {
    const Shape sh = shape_of(p.T, p.C, V, kMaxGroup);
    int grid;
    return launch<enter_kernel<SP, TX, TY, V>>(
        p, sh, sizeof(float) * (padded(p.C) + GroupSum<1>::floats(sh.G)), 1 << 30, &grid, s);
  }
};
struct Backward {
  const Params& p;
  int* rows;
  cudaStream_t s;
  template <int SP, class TX, class TY, int V>
  cudaError_t operator()() const {
    const Shape sh = shape_of(p.T, p.C, V, kMaxGroup);
    return launch<enter_backward_kernel<SP, TX, TY, V>>(
        p, sh, sizeof(float) * (2 * padded(p.C) + GroupSum<2 * SP>::floats(sh.G)),
        p.dw ? kMaxRows : 1 << 30, rows, s);
  }
};

}  // namespace

cudaError_t enter_forward(const Params& p, int x_bf16, int y_bf16, bool vec, cudaStream_t s) {
  return by_streams(p.S, x_bf16, y_bf16, vec, Forward{p, s});
}
cudaError_t enter_backward(const Params& p, int x_bf16, int y_bf16, bool vec, int* rows, cudaStream_t s) {
  return by_streams(p.S, x_bf16, y_bf16, vec, Backward{p, rows, s});
}

}  // namespace hcb
