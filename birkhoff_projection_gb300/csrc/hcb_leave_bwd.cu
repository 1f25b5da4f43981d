// hcb_leave_bwd.cu -- the gradient of leave and of leave_enter
// (hcb_leave_backward of include/hc_block.h).
#include "hcb_common.cuh"

namespace hcb {

// Every sum that the gradient needs is linear in what is read, up to the
// factor rho of y's norm: with e = w act(gate) y,
//   dP_ij = <D_i, x_j>,  db_i = scale rho <D_i, e>,
//   <g, y> = scale sum_i b_i <D_i, e>
// so one pass over the row finds S^2 + S + 1 sums and writes dx, and a
// second one, over dv = sum_i b_i D_i kept in fp32, writes dy and dgate.
// NEXT adds a pass before it: D_i = dout_i + a_i du with du from dh, as in
// enter_backward_kernel.
template <int SP, class TX, class TY, int V, bool NEXT>
__global__ void __launch_bounds__(SP == 8 ? 256 : kMaxGroup) leave_backward_kernel(const Params p) {
  extern __shared__ __align__(16) float smem[];
  constexpr int R = SP * SP + SP + 1;
  const int G = p.G, NG = blockDim.x / G, group = threadIdx.x / G, l = threadIdx.x % G;
  const int lane = threadIdx.x & 31, warp = l / 32, C = p.C;
  const int CP = (C + 3) / 4 * 4;
  constexpr int KEPT = NEXT ? 3 : 2;
  float* dv_s = smem + group * KEPT * CP;  // u of the next block first, then dv
  float* dw_s = dv_s + CP;
  float* dwn_s = dw_s + CP;  // NEXT
  float* red = smem + NG * KEPT * CP +
               group * (GroupSum<R>::floats(G) + (NEXT ? GroupSum<2 * SP>::floats(G) : 0));
  float* red_next = red + GroupSum<R>::floats(G);
  int turn = 0, turn_next = 0;
  const float inv_c = 1.0f / static_cast<float>(C);
  const bool mix = p.P.p != nullptr;
  for (int c = l; c < C; c += G) {
    dw_s[c] = 0.0f;
    if constexpr (NEXT) dwn_s[c] = 0.0f;
  }
  group_sync(G, group);
  for (int64_t t = int64_t(blockIdx.x) * NG + group; t < p.T; t += int64_t(gridDim.x) * NG) {
    const TX* dout = static_cast<const TX*>(p.dout) + t * p.dout_ts;
    const TX* x = static_cast<const TX*>(p.x) + t * p.x_ts;
    const TY* y = static_cast<const TY*>(p.y) + t * p.y_ts;
    const TY* gate = p.gate ? static_cast<const TY*>(p.gate) + t * p.gate_ts : nullptr;
    float a[SP], r_next = 0.0f, k_next = 0.0f;
    const TY* dh = nullptr;
    if constexpr (NEXT) {
      const TX* o = static_cast<const TX*>(p.out_in) + t * p.out_ts;
      dh = static_cast<const TY*>(p.dh) + t * p.dh_ts;
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
            Row<TX, V>::load(o + s * p.out_ss + c, xv[s]);
          } else {
#pragma unroll
            for (int k = 0; k < V; ++k) xv[s][k] = 0.0f;
          }
        }
        Row<TY, V>::load(dh + c, g);
        p.wn.load<V>(c, w);
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
        keep<V>(dv_s + c, u);
      }
      float total[1];
      GroupSum<2 * SP>::run(sum, total, red_next, turn_next, G, group, lane, warp);
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
        if (warp == 0 && lane < p.S)
          put_any(p.da, p.a.bf16, t * p.S + lane, r_next * (total[0] - k_next * u_x));
      }
    }
    float b[SP], P[SP][SP], sum[R];
#pragma unroll
    for (int i = 0; i < SP; ++i) {
      b[i] = i < p.S ? (p.b.p ? p.b.at(t * p.b_ts + i) : 1.0f) : 0.0f;
#pragma unroll
      for (int j = 0; j < SP; ++j)
        P[i][j] = mix && i < p.S && j < p.S ? p.P.at(t * p.P_ts + i * p.S + j) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < R; ++i) sum[i] = 0.0f;
    TX* dx = p.dx ? static_cast<TX*>(p.dx) + t * p.S * C : nullptr;
#pragma unroll 1
    for (int c = l * V; c < C; c += G * V) {
      float D[SP][V], e[V], w[V];
#pragma unroll
      for (int i = 0; i < SP; ++i) {
        if (i < p.S) {
          Row<TX, V>::load(dout + i * p.dout_ss + c, D[i]);
        } else {
#pragma unroll
          for (int k = 0; k < V; ++k) D[i][k] = 0.0f;
        }
      }
      if constexpr (NEXT) {
        float u[V], g[V], d[V];
        kept<V>(dv_s + c, u);
        kept<V>(dwn_s + c, d);
        Row<TY, V>::load(dh + c, g);
        p.wn.load<V>(c, w);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          d[k] += g[k] * (u[k] * r_next);
          u[k] = r_next * (g[k] * w[k] - k_next * u[k]);
#pragma unroll
          for (int i = 0; i < SP; ++i) D[i][k] += a[i] * u[k];
        }
        keep<V>(dwn_s + c, d);
      }
      Row<TY, V>::load(y + c, e);
      p.w.load<V>(c, w);
      float dv[V];
#pragma unroll
      for (int k = 0; k < V; ++k) {
        sum[SP * SP + SP] += e[k] * e[k];
        e[k] *= w[k];
        dv[k] = 0.0f;
#pragma unroll
        for (int i = 0; i < SP; ++i) dv[k] += b[i] * D[i][k];
      }
      keep<V>(dv_s + c, dv);
      if (gate) {
        float g[V];
        Row<TY, V>::load(gate + c, g);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          float q, slope;
          gate_of(p.act, g[k], q, slope);
          e[k] *= q;
        }
      }
#pragma unroll
      for (int i = 0; i < SP; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) sum[SP * SP + i] += D[i][k] * e[k];
      if (mix) {
#pragma unroll
        for (int j = 0; j < SP; ++j) {
          if (j < p.S) {
            float xv[V];
            Row<TX, V>::load(x + j * p.x_ss + c, xv);
#pragma unroll
            for (int i = 0; i < SP; ++i)
#pragma unroll
              for (int k = 0; k < V; ++k) sum[i * SP + j] += D[i][k] * xv[k];
          }
        }
        if (dx) {
#pragma unroll
          for (int j = 0; j < SP; ++j) {
            if (j < p.S) {
              float d[V];
#pragma unroll
              for (int k = 0; k < V; ++k) {
                d[k] = 0.0f;
#pragma unroll
                for (int i = 0; i < SP; ++i) d[k] += P[i][j] * D[i][k];
              }
              Row<TX, V>::store(dx + int64_t(j) * C + c, d);
            }
          }
        }
      } else if (dx) {
#pragma unroll
        for (int j = 0; j < SP; ++j)
          if (j < p.S) Row<TX, V>::store(dx + int64_t(j) * C + c, D[j]);
      }
    }
    float total[GroupSum<R>::CH];
    GroupSum<R>::run(sum, total, red, turn, G, group, lane, warp);
    const float rho = p.norm ? rsqrtf(of_total(total, SP * SP + SP) * inv_c + p.eps) : 1.0f;
    float gy = 0.0f;
#pragma unroll
    for (int i = 0; i < SP; ++i) gy += b[i] * of_total(total, SP * SP + i);
    const float k_y = p.norm ? p.scale * gy * inv_c * rho * rho : 0.0f;
    if (warp == 0) {
#pragma unroll
      for (int ch = 0; ch < GroupSum<R>::CH; ++ch) {
        const int i = ch * 32 + lane;
        if (i < SP * SP) {
          if (p.dP && i / SP < p.S && i % SP < p.S)
            put_any(p.dP, p.P.bf16, (t * p.S + i / SP) * p.S + i % SP, total[ch]);
        } else if (i < SP * SP + p.S) {
          if (p.db) put_any(p.db, p.b.bf16, t * p.S + i - SP * SP, p.scale * rho * total[ch]);
        }
      }
    }
    TY* dy = p.dy ? static_cast<TY*>(p.dy) + t * C : nullptr;
    TY* dgate = p.dgate ? static_cast<TY*>(p.dgate) + t * C : nullptr;
#pragma unroll 1
    for (int c = l * V; c < C; c += G * V) {
      float yv[V], w[V], dz[V], d[V];
      Row<TY, V>::load(y + c, yv);
      p.w.load<V>(c, w);
      kept<V>(dv_s + c, dz);
#pragma unroll
      for (int k = 0; k < V; ++k) dz[k] *= p.scale;
      if (gate) {
        float g[V];
        Row<TY, V>::load(gate + c, g);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          float q, slope;
          gate_of(p.act, g[k], q, slope);
          g[k] = dz[k] * slope * (yv[k] * rho * w[k]);
          dz[k] *= q;
        }
        if (dgate) Row<TY, V>::store(dgate + c, g);
      }
      kept<V>(dw_s + c, d);
#pragma unroll
      for (int k = 0; k < V; ++k) d[k] += dz[k] * (yv[k] * rho);
      keep<V>(dw_s + c, d);
      if (dy) {
#pragma unroll
        for (int k = 0; k < V; ++k) dz[k] = rho * (dz[k] * w[k] - k_y * yv[k]);
        Row<TY, V>::store(dy + c, dz);
      }
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < C; c += blockDim.x) {
    if (p.dw) {
      float d = 0.0f;
      for (int g = 0; g < NG; ++g) d += smem[(g * KEPT + 1) * CP + c];
      p.dw[int64_t(blockIdx.x) * C + c] = d;
    }
    if (NEXT && p.dwn) {
      float d = 0.0f;
      for (int g = 0; g < NG; ++g) d += smem[(g * KEPT + 2) * CP + c];
      p.dwn[int64_t(blockIdx.x) * C + c] = d;
    }
  }
}

namespace {

template <bool NEXT>
struct Backward {
  const Params& p;
  int* rows;
  cudaStream_t s;
  template <int SP, class TX, class TY, int V>
  cudaError_t operator()() const {
    const Shape sh = shape_of(p.T, p.C, V, SP == 8 ? 256 : kMaxGroup);
    const int fl = GroupSum<SP * SP + SP + 1>::floats(sh.G) + (NEXT ? GroupSum<2 * SP>::floats(sh.G) : 0);
    return launch<leave_backward_kernel<SP, TX, TY, V, NEXT>>(
        p, sh, sizeof(float) * ((NEXT ? 3 : 2) * padded(p.C) + fl),
        p.dw || p.dwn ? kMaxRows : 1 << 30, rows, s);
  }
};

}  // namespace

cudaError_t leave_backward(const Params& p, int x_bf16, int y_bf16, bool vec, int* rows, cudaStream_t s) {
  if (p.dh) return by_streams(p.S, x_bf16, y_bf16, vec, Backward<true>{p, rows, s});
  return by_streams(p.S, x_bf16, y_bf16, vec, Backward<false>{p, rows, s});
}

}  // namespace hcb
