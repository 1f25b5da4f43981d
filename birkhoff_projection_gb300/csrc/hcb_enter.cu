// hcb_enter.cu -- the block's input from the residual streams and its
// gradient (hcb_enter, hcb_enter_backward of include/hc_block.h).
#include "hcb_common.cuh"

namespace hcb {

// u = sum_s a_s x_s and its mean square in one pass over the row's streams;
// u stays in shared memory (fp32) until r is known, then h = w u r.  Bound by
// memory: 16384 x 4 x 4096 bf16 in 99.7 us, 6.73 TB/s, 99% of the copy's rate.
// With few channels the sums' barriers and the instructions to a token show
// (16384 x 4 x 500 bf16: 26.6 us, 3.1 TB/s), and odd rows move in single words.
template <int SP, class TX, class TY, int V, int ODD>
struct Enter {
  using RX = Row<TX, V, ODD>;
  using RY = Row<TY, V, ODD>;
  using Co = Coefficients<SP, false, false, true>;
  using Sum = GroupSum<1>;
  static constexpr int DEPTH = 2;
  static constexpr int SLOT = SP * RX::SLOT;    // the streams
  static constexpr int ITEM = kFloats<V>;       // u
  static Need need(int G, int) {
    return {DEPTH * SLOT, ITEM, 4 * (G / 32 * Co::FLOATS + Sum::floats(G))};
  }
};

template <int SP, bool EXACT, class TX, class TY, int V, int ODD, int W>
__global__ void __launch_bounds__(kMaxGroup) enter_kernel(const Params p) {
  using E = Enter<SP, TX, TY, V, ODD>;
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
  E::Sum::clear(red, G, l);
  group_sync(G, group);
  int turn = 0;
  const float inv_c = 1.0f / static_cast<float>(C);
  const uint32_t step = gridDim.x * NG;
  uint32_t t = blockIdx.x * NG + group;

  uint32_t ta = t;  // the next item to copy
  int ca = c0, ka = 0;
  char* slot_a = ring;
  const TX* xa = at_row<TX>(p.x, ta, p.x_ts);
  auto copy_next = [&] {
    slot_read<ODD>();
    if (ta < p.T && ca < C) {
      const uint32_t to = b4::smem_addr(slot_a);
      by_block<V, ODD>(ca, C, [&](auto full) {
        constexpr bool FULL = decltype(full)::value;
        each<SP>([&](auto i) {
          if (EXACT || i.value < S)
            RX::template copy<FULL, i.value * RX::SLOT>(to, lane, xa + i.value * p.x_ss, ca, C);
        });
      });
    }
    copy_commit();
    ca += GV;
    if (++ka == K) ka = 0, ca = c0, ta += step, xa = at_row<TX>(p.x, ta, p.x_ts);
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
    P2 a[SP];
    Co::read(co_s, Co::NB, a);
    const TX* x = at_row<TX>(p.x, t, p.x_ts);
    P2 ss = 0;
    char* item = item0;
#pragma unroll 1
    for (int c = c0, k = 0; k < K; ++k, c += GV, item += E::ITEM) {
      slot_ready<DEPTH, ODD>();
      P2 u[H] = {};
      if (c < C) {
#pragma unroll
        for (int i = 0; i < SP; ++i) {
          if (EXACT || i < S) {
            P2 xv[H];
            RX::arrived(slot + i * RX::SLOT, lane, x + i * p.x_ss, c, xv);
#pragma unroll
            for (int j = 0; j < H; ++j) u[j] = fma2(a[i], xv[j], u[j]);
          }
        }
      }
      copy_next();
      slot = slot == ring + (DEPTH - 1) * E::SLOT ? ring : slot + E::SLOT;
#pragma unroll
      for (int j = 0; j < H; ++j) ss = fma2(u[j], u[j], ss);
      keep<V>(item, lane, u);
    }
    const float sum[1] = {both(ss)};
    float total[1];
    GroupSum<1>::run(sum, total, red, turn, G, group, lane, warp);
    const P2 r = twice(rsqrtf(of_total(total, 0) * inv_c + p.eps));
    TY* h = static_cast<TY*>(p.h) + uint64_t(t) * uint32_t(C);
    item = item0;
#pragma unroll 1
    for (int c = c0; c < C; c += GV, item += E::ITEM) {
      P2 u[H], w[H];
      kept<V>(item, lane, u);
      p.w.load<V, ODD, W>(c, lane, C, w);
#pragma unroll
      for (int j = 0; j < H; ++j) u[j] = mul2(u[j], mul2(r, w[j]));
      RY::store(h, c, lane, C, u);
    }
  }
  copy_wait_all();
}

// With G = w dh the gradient needs the sums <G, x_s>, <u, x_s> (for da_s =
// r (<G, x_s> - k <u, x_s>)), <G, u> and <u, u>; one pass over the row finds
// them and a second, over what the first kept and over dres, writes.  The last
// two are summed from u itself (next_sums in hcb_common.cuh).
// 16384 x 4 x 4096 bf16: 290 us, 6.0 TB/s, 89% of the copy's rate (fp32
// streams with bf16 rows 95%).  Two slots to a warp and two CTAs on an SM: one
// slot 322 us, three 305, three CTAs (spilt) 399; half as many threads with
// two items each 322.
template <int SP, class TX, class TY, int V, int ODD>
struct EnterBackward {
  using RX = Row<TX, V, ODD>;
  using RY = Row<TY, V, ODD>;
  using Co = Coefficients<SP, false, false, true>;
  using Sum = GroupSum<next_sums(SP)>;
  static constexpr int DEPTH = 2;
  // a slot: the streams (or dres), then dh
  static constexpr int DH = SP * RX::SLOT, SLOT = DH + RY::SLOT;
  // kept: u, dh, and the weight's share
  static constexpr int KH = kFloats<V>, KW = KH + RY::KEPT, ITEM = KW + kFloats<V>;
  static Need need(int G, int direct) {
    return {DEPTH * SLOT, direct ? KW : ITEM, 4 * (G / 32 * Co::FLOATS + Sum::floats(G))};
  }
};

template <int SP, bool EXACT, class TX, class TY, int V, int ODD, int W>
__global__ void __launch_bounds__(256, SP == 8 ? 1 : 2) enter_backward_kernel(const Params p) {
  using E = EnterBackward<SP, TX, TY, V, ODD>;
  using RX = typename E::RX;
  using RY = typename E::RY;
  using Co = typename E::Co;
  using Sum = typename E::Sum;
  constexpr int DEPTH = E::DEPTH, H = V / 2;
  extern __shared__ __align__(16) char smem[];
  const int G = p.G, NG = blockDim.x / G, group = threadIdx.x / G, l = threadIdx.x % G;
  const int lane = threadIdx.x & 31, warp = l / 32, C = p.C, S = EXACT ? SP : p.S, GV = G * V;
  const int K = (C + GV - 1) / GV, c0 = first_channel<V, ODD>(l);
  const bool direct = !EXACT && p.direct;
  const int ITEM = direct ? E::KW : E::ITEM;
  char* of_group = smem + group * p.group_bytes;
  char* ring = of_group + warp * p.warp_bytes;
  char* item0 = ring + DEPTH * E::SLOT;
  float* co_all = reinterpret_cast<float*>(of_group + G / 32 * p.warp_bytes);
  float* co_s = co_all + warp * Co::FLOATS;
  float* red = co_all + G / 32 * Co::FLOATS;
  Sum::clear(red, G, l);
  let_next_launch();
  group_sync(G, group);
  float* row_dw = direct && p.dw ? p.dw + int64_t(blockIdx.x) * pitch(C) : nullptr;
  int turn = 0;
  const float inv_c = 1.0f / static_cast<float>(C);
  const uint32_t step = gridDim.x * NG;
  uint32_t t = blockIdx.x * NG + group;

  // items of a token: x and dh for every k, then, if there is one, dres
  const int NI = p.dres ? 2 * K : K;
  uint32_t ta = t;
  int ca = c0, ia = 0;
  char* slot_a = ring;
  auto copy_next = [&] {
    slot_read<ODD>();
    const bool second = ia >= K;
    if (ta < p.T && ca < C) {
      const TX* x = second ? at_row<TX>(p.dres, ta, p.dres_ts)
                           : at_row<TX>(p.x, ta, p.x_ts);
      const int64_t ss = second ? p.dres_ss : p.x_ss;
      const uint32_t to = b4::smem_addr(slot_a);
      by_block<V, ODD>(ca, C, [&](auto full) {
        constexpr bool FULL = decltype(full)::value;
        each<SP>([&](auto i) {
          if (EXACT || i.value < S) RX::template copy<FULL, i.value * RX::SLOT>(to, lane, x + i.value * ss, ca, C);
        });
        if (!second) RY::template copy<FULL, E::DH>(to, lane, at_row<TY>(p.dh, ta, p.dh_ts), ca, C);
      });
    }
    copy_commit();
    ca += GV;
    ++ia;
    if (ia == K) ca = c0;
    if (ia == NI) ia = 0, ca = c0, ta += step;
    slot_a = slot_a == ring + (DEPTH - 1) * E::SLOT ? ring : slot_a + E::SLOT;
  };
  Co co;
  co.init(p, lane);
  if (t < p.T) co.fetch(t);
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) copy_next();
  if (p.dw) {
    const P2 z[H] = {};
    char* item = item0;
#pragma unroll 1
    for (int c = c0; c < C; c += GV, item += ITEM) {
      if (row_dw)
        PartRow<V, ODD>::put(row_dw, c, lane, C, z);
      else
        keep<V>(item + E::KW, lane, z);
    }
  }

  const char* slot = ring;
#pragma unroll 1
  for (; t < p.T; t += step) {
    co.spread(co_s, lane);
    if (t + step < p.T) co.fetch(t + step);
    P2 a[SP];
    Co::read(co_s, Co::NB, a);
    const TX* x = at_row<TX>(p.x, t, p.x_ts);
    const TY* dh = at_row<TY>(p.dh, t, p.dh_ts);
    P2 sum2[next_sums(SP)] = {};
    char* item = item0;
#pragma unroll 1
    for (int c = c0, k = 0; k < K; ++k, c += GV, item += ITEM) {
      P2 w[H];
      if (c < C) p.w.load<V, ODD, W>(c, lane, C, w);
      slot_ready<DEPTH, ODD>();
      if (c < C) {
        P2 xv[SP][H], g[H], u[H] = {};
#pragma unroll
        for (int i = 0; i < SP; ++i) {
          if (EXACT || i < S) {
            RX::arrived(slot + i * RX::SLOT, lane, x + i * p.x_ss, c, xv[i]);
#pragma unroll
            for (int j = 0; j < H; ++j) u[j] = fma2(a[i], xv[i][j], u[j]);
          }
        }
        RY::arrived_kept(slot + E::DH, lane, dh, c, g, item + E::KH);
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
      copy_next();
      slot = slot == ring + (DEPTH - 1) * E::SLOT ? ring : slot + E::SLOT;
    }
    float sum[next_sums(SP)], total[1], gu, uu;
#pragma unroll
    for (int i = 0; i < next_sums(SP); ++i) sum[i] = both(sum2[i]);
    Sum::run(sum, total, red, turn, G, group, lane, warp);
    sums_of_u<SP>(total, low(a[0]), gu, uu);
    const float r = rsqrtf(uu * inv_c + p.eps);
    const float k_u = gu * inv_c * r * r;
    if (p.da) {
      const float u_x = __shfl_sync(0xffffffffu, total[0], (lane + SP) & 31);
      if (warp == 0 && lane < S) put_any(p.da, p.a.bf16, int64_t(t) * S + lane, r * (total[0] - k_u * u_x));
    }
    // r u is what the weight's share takes, and du = r w dh - k (r u)
    const P2 r2 = twice(r), minus_k = twice(-k_u);
    const TX* dres = p.dres ? at_row<TX>(p.dres, t, p.dres_ts) : nullptr;
    TX* dx = p.dx ? static_cast<TX*>(p.dx) + uint64_t(t) * uint32_t(S * C) : nullptr;
    item = item0;
#pragma unroll 1
    for (int c = c0, k = 0; k < K; ++k, c += GV, item += ITEM) {
      if (dres) slot_ready<DEPTH, ODD>();
      if (c < C) {
        P2 u[H], g[H], w[H];
        kept<V>(item, lane, u);
        RY::kept(item + E::KH, lane, g);
        p.w.load<V, ODD, W>(c, lane, C, w);
#pragma unroll
        for (int j = 0; j < H; ++j) u[j] = mul2(r2, u[j]);
        if (p.dw) add_share<V, ODD>(item + E::KW, row_dw, c, lane, C, g, u);
#pragma unroll
        for (int j = 0; j < H; ++j) u[j] = fma2(mul2(r2, w[j]), g[j], mul2(minus_k, u[j]));
        if (dx) {
#pragma unroll
          for (int i = 0; i < SP; ++i) {
            if (EXACT || i < S) {
              P2 d[H] = {};
              if (dres) RX::arrived(slot + i * RX::SLOT, lane, dres + i * p.dres_ss, c, d);
#pragma unroll
              for (int j = 0; j < H; ++j) d[j] = fma2(a[i], u[j], d[j]);
              RX::store(dx + i * C, c, lane, C, d);
            }
          }
        }
      }
      if (dres) {
        copy_next();
        slot = slot == ring + (DEPTH - 1) * E::SLOT ? ring : slot + E::SLOT;
      }
    }
  }
  copy_wait_all();
  if (p.dw && !direct) {
    __syncthreads();
    sum_shares<V, ODD>(smem + warp * p.warp_bytes + DEPTH * E::SLOT + E::KW, p, NG, ITEM,
                  p.dw + int64_t(blockIdx.x) * pitch(C));
  }
}

namespace {

struct Forward {
  const Params& p;
  cudaStream_t s;
  template <int SP, bool EXACT, class TX, class TY, int V, int ODD>
  cudaError_t operator()() const {
    Params q = p;
    int grid;
    const Shape sh = plan(q, shape_of(p.T, p.C, V, 2, kMaxGroup), V, Enter<SP, TX, TY, V, ODD>::need);
    const int w = EXACT ? Weights::kind(p.w) : 0;
    if (w == 1) return launch<enter_kernel<SP, EXACT, TX, TY, V, ODD, EXACT ? 1 : 0>>(q, sh, 1 << 30, &grid, s);
    if (w == 2 && ODD == 0) return launch<enter_kernel<SP, EXACT && ODD == 0, TX, TY, V, ODD, EXACT && ODD == 0 ? 2 : 0>>(q, sh, 1 << 30, &grid, s);
    return launch<enter_kernel<SP, false, TX, TY, V, ODD, 0>>(q, sh, 1 << 30, &grid, s);
  }
};
struct Backward {
  const Params& p;
  int* rows;
  cudaStream_t s;
  template <int SP, bool EXACT, class TX, class TY, int V, int ODD>
  cudaError_t operator()() const {
    Params q = p;
    const Shape sh =
        plan(q, shape_of(p.T, p.C, V, 2, 256), V, EnterBackward<SP, TX, TY, V, ODD>::need);
    const int most = p.dw ? kMaxRows : 1 << 30;
    const int w = EXACT && !q.direct ? Weights::kind(p.w) : 0;
    if (w == 1) return launch<enter_backward_kernel<SP, EXACT, TX, TY, V, ODD, EXACT ? 1 : 0>>(q, sh, most, rows, s);
    if (w == 2 && ODD == 0)
      return launch<enter_backward_kernel<SP, EXACT && ODD == 0, TX, TY, V, ODD, EXACT && ODD == 0 ? 2 : 0>>(q, sh, most, rows, s);
    return launch<enter_backward_kernel<SP, false, TX, TY, V, ODD, 0>>(q, sh, most, rows, s);
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
