// hcb_enter.cu -- the block's input from the residual streams and its
// gradient (hcb_enter, hcb_enter_backward of include/hc_block.h).
#include "hcb_common.cuh"

#ifndef HCB_ENTER_DEPTH
#define HCB_ENTER_DEPTH 2
#endif
#ifndef HCB_ENTER_BWD_DEPTH
#define HCB_ENTER_BWD_DEPTH 2
#endif

namespace hcb {

// u = sum_s a_s x_s and its mean square in one pass over the row's streams;
// u stays in shared memory (fp32) until r is known, then h = w u r.
template <int SP, class TX, class TY, int V, bool ODD>
struct Enter {
  using RX = Row<TX, V, ODD>;
  using RY = Row<TY, V, ODD>;
  using Co = Coefficients<SP, false, false, true>;
  using Sum = GroupSum<1>;
  static constexpr int DEPTH = HCB_ENTER_DEPTH;
  static size_t bytes(int S, int C, int G) {
    return size_t(G) * (DEPTH * S * RX::SLOT + items(C, V, G) * V * 4) +
           4 * (G / 32 * Co::FLOATS + (Sum::floats(G) + 3) / 4 * 4);
  }
};

template <int SP, class TX, class TY, int V, bool ODD>
__global__ void __launch_bounds__(kMaxGroup) enter_kernel(const Params p) {
  using E = Enter<SP, TX, TY, V, ODD>;
  using RX = typename E::RX;
  using RY = typename E::RY;
  using Co = typename E::Co;
  constexpr int DEPTH = E::DEPTH;
  extern __shared__ __align__(16) char smem[];
  const int G = p.G, NG = blockDim.x / G, group = threadIdx.x / G, l = threadIdx.x % G;
  const int lane = threadIdx.x & 31, warp = l / 32, C = p.C, S = p.S;
  const int K = (C + V * G - 1) / (V * G);
  char* ring = smem + size_t(group) * p.group_bytes;
  float* u_s = reinterpret_cast<float*>(ring + DEPTH * G * S * RX::SLOT);
  float* co_s = u_s + K * V * G + warp * Co::FLOATS;
  float* red = u_s + K * V * G + G / 32 * Co::FLOATS;
  int turn = 0;
  const float inv_c = 1.0f / static_cast<float>(C);
  const int64_t step = int64_t(gridDim.x) * NG;
  int64_t t = int64_t(blockIdx.x) * NG + group;

  int64_t ta = t;  // the next item to copy
  int ka = 0, slot_a = 0;
  auto copy_next = [&] {
    const int c = (ka * G + l) * V;
    if (ta < p.T && c < C) {
      const TX* x = static_cast<const TX*>(p.x) + ta * p.x_ts + c;
      char* s = ring + slot_a * G * S * RX::SLOT;
#pragma unroll
      for (int i = 0; i < SP; ++i)
        if (i < S) RX::copy(s + i * G * RX::SLOT, G, l, x + i * p.x_ss, C - c);
    }
    copy_commit();
    if (++ka == K) ka = 0, ta += step;
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
    float a[SP];
    Co::read(co_s, Co::NB, a);
    const TX* x = static_cast<const TX*>(p.x) + t * p.x_ts;
    float ss[1] = {0.0f};
    for (int k = 0; k < K; ++k) {
      const int c = (k * G + l) * V;
      copy_wait<DEPTH - 1>();
      float u[V];
#pragma unroll
      for (int j = 0; j < V; ++j) u[j] = 0.0f;
      if (c < C) {
        const char* s = ring + slot * G * S * RX::SLOT;
#pragma unroll
        for (int i = 0; i < SP; ++i) {
          if (i < S) {
            float xv[V];
            RX::arrived(s + i * G * RX::SLOT, G, l, x + i * p.x_ss + c, xv);
#pragma unroll
            for (int j = 0; j < V; ++j) u[j] += a[i] * xv[j];
          }
        }
      }
      copy_next();
      if (++slot == DEPTH) slot = 0;
#pragma unroll
      for (int j = 0; j < V; ++j) ss[0] += u[j] * u[j];
      keep<V>(u_s, G, l, k, u);
    }
    float total[1];
    GroupSum<1>::run(ss, total, red, turn, G, group, lane, warp);
    const float r = rsqrtf(of_total(total, 0) * inv_c + p.eps);
    TY* h = static_cast<TY*>(p.h) + t * C;
    for (int k = 0; k < K; ++k) {
      const int c = (k * G + l) * V;
      if (c >= C) break;
      float u[V], w[V];
      kept<V>(u_s, G, l, k, u);
      p.w.load<V, ODD>(c, C - c, w);
#pragma unroll
      for (int j = 0; j < V; ++j) u[j] *= r * w[j];
      RY::store(h + c, u, C - c);
    }
  }
}

// With G = w dh all sums of the gradient are linear in <G, x_s> and <u, x_s>:
// <G, u> = sum a_s <G, x_s>, <u, u> = sum a_s <u, x_s> and
// da_s = r (<G, x_s> - k <u, x_s>), so one pass over the row finds them and
// a second, over what the first kept and over dres, writes.
template <int SP, class TX, class TY, int V, bool ODD>
struct EnterBackward {
  using RX = Row<TX, V, ODD>;
  using RY = Row<TY, V, ODD>;
  using Co = Coefficients<SP, false, false, true>;
  using Sum = GroupSum<2 * SP>;
  static constexpr int DEPTH = HCB_ENTER_BWD_DEPTH;
  static __host__ __device__ constexpr int slot(int S) { return S * RX::SLOT + RY::SLOT; }
  static size_t bytes(int S, int C, int G, bool dw) {
    return size_t(G) * (DEPTH * slot(S) + items(C, V, G) * V * (4 + sizeof(TY) + (dw ? 4 : 0))) +
           4 * (G / 32 * Co::FLOATS + (Sum::floats(G) + 3) / 4 * 4);
  }
};

template <int SP, class TX, class TY, int V, bool ODD>
__global__ void __launch_bounds__(kMaxGroup, 1) enter_backward_kernel(const Params p) {
  using E = EnterBackward<SP, TX, TY, V, ODD>;
  using RX = typename E::RX;
  using RY = typename E::RY;
  using Co = typename E::Co;
  using Sum = typename E::Sum;
  constexpr int DEPTH = E::DEPTH;
  extern __shared__ __align__(16) char smem[];
  const int G = p.G, NG = blockDim.x / G, group = threadIdx.x / G, l = threadIdx.x % G;
  const int lane = threadIdx.x & 31, warp = l / 32, C = p.C, S = p.S;
  const int K = (C + V * G - 1) / (V * G);
  const int slot_bytes = G * E::slot(S);
  char* ring = smem + size_t(group) * p.group_bytes;
  float* u_s = reinterpret_cast<float*>(ring + DEPTH * slot_bytes);
  char* dh_s = reinterpret_cast<char*>(u_s + K * V * G);
  float* co_all = reinterpret_cast<float*>(dh_s + K * V * G * sizeof(TY));
  float* co_s = co_all + warp * Co::FLOATS;
  float* red = co_all + G / 32 * Co::FLOATS;
  WeightShare<V> dw = {red + (Sum::floats(G) + 3) / 4 * 4,
                       p.direct ? p.dw + int64_t(blockIdx.x) * pitch(C) : nullptr};
  int turn = 0;
  const float inv_c = 1.0f / static_cast<float>(C);
  const int64_t step = int64_t(gridDim.x) * NG;
  int64_t t = int64_t(blockIdx.x) * NG + group;

  // items of a token: x and dh for every k, then, if there is one, dres
  const int NI = p.dres ? 2 * K : K;
  int64_t ta = t;
  int ia = 0, slot_a = 0;
  auto copy_next = [&] {
    const bool second = ia >= K;
    const int c = ((second ? ia - K : ia) * G + l) * V;
    if (ta < p.T && c < C) {
      char* s = ring + slot_a * slot_bytes;
      const TX* x = second ? static_cast<const TX*>(p.dres) + ta * p.dres_ts + c
                           : static_cast<const TX*>(p.x) + ta * p.x_ts + c;
      const int64_t ss = second ? p.dres_ss : p.x_ss;
#pragma unroll
      for (int i = 0; i < SP; ++i)
        if (i < S) RX::copy(s + i * G * RX::SLOT, G, l, x + i * ss, C - c);
      if (!second)
        RY::copy(s + S * G * RX::SLOT, G, l, static_cast<const TY*>(p.dh) + ta * p.dh_ts + c, C - c);
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

  int slot = 0;
  for (; t < p.T; t += step) {
    co.spread(co_s, lane);
    if (t + step < p.T) co.fetch(p, t + step, lane);
    float a[SP];
    Co::read(co_s, Co::NB, a);
    const TX* x = static_cast<const TX*>(p.x) + t * p.x_ts;
    const TY* dh = static_cast<const TY*>(p.dh) + t * p.dh_ts;
    float sum[2 * SP];
#pragma unroll
    for (int s = 0; s < 2 * SP; ++s) sum[s] = 0.0f;
    for (int k = 0; k < K; ++k) {
      const int c = (k * G + l) * V;
      float xv[SP][V], g[V], w[V], u[V];
      if (c < C) p.w.load<V, ODD>(c, C - c, w);
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
        RY::arrived(s + S * G * RX::SLOT, G, l, dh + c, g);
      }
      copy_next();
      if (++slot == DEPTH) slot = 0;
      if (c < C) {
        keep_row<TY, V>(dh_s, G, l, k, g);
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
        keep<V>(u_s, G, l, k, u);
      }
    }
    float total[1];
    Sum::run(sum, total, red, turn, G, group, lane, warp);
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
      if (warp == 0 && lane < S) put_any(p.da, p.a.bf16, t * S + lane, r * (total[0] - k_u * u_x));
    }
    const TX* dres = p.dres ? static_cast<const TX*>(p.dres) + t * p.dres_ts : nullptr;
    TX* dx = static_cast<TX*>(p.dx) + t * S * C;
    for (int k = 0; k < K; ++k) {
      const int c = (k * G + l) * V;
      float u[V], g[V], w[V];
      if (c < C) {
        kept<V>(u_s, G, l, k, u);
        kept_row<TY, V>(dh_s, G, l, k, g);
        p.w.load<V, ODD>(c, C - c, w);
        if (p.dw) {
          float d[V];
#pragma unroll
          for (int j = 0; j < V; ++j) d[j] = g[j] * (u[j] * r);
          dw.add(G, l, k, d);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) u[j] = r * (g[j] * w[j] - k_u * u[j]);
      }
      if (dres) {
        copy_wait<DEPTH - 1>();
        if (c < C) {
          const char* s = ring + slot * slot_bytes;
          float d[SP][V];
#pragma unroll
          for (int i = 0; i < SP; ++i)
            if (i < S) RX::arrived(s + i * G * RX::SLOT, G, l, dres + i * p.dres_ss + c, d[i]);
          copy_next();
#pragma unroll
          for (int i = 0; i < SP; ++i) {
            if (i < S) {
#pragma unroll
              for (int j = 0; j < V; ++j) d[i][j] += a[i] * u[j];
              RX::store(dx + int64_t(i) * C + c, d[i], C - c);
            }
          }
        } else {
          copy_next();
        }
        if (++slot == DEPTH) slot = 0;
      } else if (c < C && p.dx) {
#pragma unroll
        for (int i = 0; i < SP; ++i) {
          if (i < S) {
            float d[V];
#pragma unroll
            for (int j = 0; j < V; ++j) d[j] = a[i] * u[j];
            RX::store(dx + int64_t(i) * C + c, d, C - c);
          }
        }
      }
    }
  }
  copy_wait_all();
  if (p.dw && !p.direct) {
    __syncthreads();
    sum_shares<V>(reinterpret_cast<float*>(reinterpret_cast<char*>(dw.s) - size_t(group) * p.group_bytes),
                  p.group_bytes / 4, G, NG, C, p.dw + int64_t(blockIdx.x) * pitch(C));
  }
}

namespace {

struct Forward {
  const Params& p;
  cudaStream_t s;
  template <int SP, class TX, class TY, int V, bool ODD>
  cudaError_t operator()() const {
    using E = Enter<SP, TX, TY, V, ODD>;
    int direct, grid;
    const Shape sh = fitted(shape_of(p.T, p.C, V, kMaxGroup), false, &direct,
                            [&](int G, bool) { return E::bytes(p.S, p.C, G); });
    return launch<enter_kernel<SP, TX, TY, V, ODD>>(p, sh, E::bytes(p.S, p.C, sh.G), 1 << 30, &grid, s);
  }
};
struct Backward {
  const Params& p;
  int* rows;
  cudaStream_t s;
  template <int SP, class TX, class TY, int V, bool ODD>
  cudaError_t operator()() const {
    using E = EnterBackward<SP, TX, TY, V, ODD>;
    Params q = p;
    const bool dw = p.dw != nullptr;
    const Shape sh = fitted(shape_of(p.T, p.C, V, kMaxGroup), dw, &q.direct,
                            [&](int G, bool direct) { return E::bytes(p.S, p.C, G, dw && !direct); });
    return launch<enter_backward_kernel<SP, TX, TY, V, ODD>>(
        q, sh, E::bytes(p.S, p.C, sh.G, dw && !q.direct), dw ? kMaxRows : 1 << 30, rows, s);
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
