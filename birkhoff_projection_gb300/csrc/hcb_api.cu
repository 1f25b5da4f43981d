// hcb_api.cu -- the entry points of include/hc_block.h: argument checks on
// the host, the choice between vector and element-wise rows, and the sum of
// the partial weight gradients.
#include <cmath>
#include <cstring>

#include "b4_launch.cuh"
#include "hcb_common.cuh"

namespace hcb {

int sms() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  return b4::sm_count(dev);
}

namespace {

bool dtype_ok(int32_t d) { return d == B4_F32 || d == B4_BF16; }
bool eps_ok(float e) { return e >= 0.0f && !std::isinf(e); }
uintptr_t mask(int32_t dtype) { return dtype == B4_BF16 ? 1 : 3; }
bool placed(const void* p, int32_t dtype) { return (reinterpret_cast<uintptr_t>(p) & mask(dtype)) == 0; }

// What every entry point asks of sizes and types.
int check_sizes(const hcb_args* a) {
  if (a == nullptr || a->T < 0 || a->T > INT32_MAX) return B4_EINVAL;
  if (a->S < 1 || a->S > HCB_MAX_STREAMS || a->C < 1 || a->C > HCB_MAX_CHANNELS) return B4_EINVAL;
  for (int32_t d : {a->x_dtype, a->y_dtype, a->w_dtype, a->wn_dtype, a->p_dtype, a->a_dtype, a->b_dtype})
    if (!dtype_ok(d)) return B4_EINVAL;
  if (!eps_ok(a->eps) || !eps_ok(a->eps_next) || !std::isfinite(a->scale)) return B4_EINVAL;
  if (a->act < HCB_ACT_NONE || a->act > HCB_ACT_LINEAR) return B4_EINVAL;
  for (int64_t s : {a->x_ts, a->x_ss, a->y_ts, a->gate_ts, a->P_ts, a->a_ts, a->b_ts, a->dout_ts,
                    a->dout_ss, a->dh_ts, a->dres_ts, a->dres_ss, a->out_ts, a->out_ss})
    if (s < 0 || s > INT32_MAX / 4) return B4_EINVAL;
  for (const void* q : {a->x, a->dout, a->dres, a->out_in, static_cast<const void*>(a->out),
                        static_cast<const void*>(a->dx)})
    if (!placed(q, a->x_dtype)) return B4_EINVAL;
  for (const void* q : {a->y, a->gate, a->dh, static_cast<const void*>(a->h),
                        static_cast<const void*>(a->dy), static_cast<const void*>(a->dgate)})
    if (!placed(q, a->y_dtype)) return B4_EINVAL;
  if (!placed(a->P, a->p_dtype) || !placed(a->dP, a->p_dtype) || !placed(a->a, a->a_dtype) ||
      !placed(a->da, a->a_dtype) || !placed(a->b, a->b_dtype) || !placed(a->db, a->b_dtype) ||
      !placed(a->w, a->w_dtype) || !placed(a->dw, a->w_dtype) || !placed(a->w_next, a->wn_dtype) ||
      !placed(a->dw_next, a->wn_dtype))
    return B4_EINVAL;
  if (a->x_dtype == B4_BF16 && a->y_dtype == B4_F32) return B4_ENOTIMPL;
  return B4_OK;
}

Params params_of(const hcb_args* a) {
  Params p;
  memset(&p, 0, sizeof(p));
  p.T = static_cast<uint32_t>(a->T), p.S = a->S, p.C = a->C, p.act = a->act, p.norm = a->norm != 0;
  p.eps = a->eps, p.eps_next = a->eps_next, p.scale = a->scale;
  p.P = {a->P, a->p_dtype == B4_BF16}, p.a = {a->a, a->a_dtype == B4_BF16};
  p.b = {a->b, a->b_dtype == B4_BF16};
  p.w = {a->w, a->w_dtype == B4_BF16}, p.wn = {a->w_next, a->wn_dtype == B4_BF16};
  auto u = [](int64_t v) { return static_cast<uint32_t>(v); };
  p.x_ts = u(a->x_ts), p.x_ss = u(a->x_ss), p.y_ts = u(a->y_ts), p.gate_ts = u(a->gate_ts);
  p.P_ts = u(a->P_ts), p.a_ts = u(a->a_ts), p.b_ts = u(a->b_ts);
  p.dout_ts = u(a->dout_ts), p.dout_ss = u(a->dout_ss), p.dh_ts = u(a->dh_ts);
  p.dres_ts = u(a->dres_ts), p.dres_ss = u(a->dres_ss), p.out_ts = u(a->out_ts), p.out_ss = u(a->out_ss);
  return p;
}

// Whether every row can be read and written in 16-byte vectors: bases on 16
// bytes, strides and C whole vectors of the wider row type.
bool vectors(const hcb_args* a, const Params& p) {
  const int V = a->x_dtype == B4_F32 ? 4 : 8;
  if (a->C % V != 0) return false;
  for (const void* q : {p.x, p.y, p.gate, p.dout, p.dh, p.dres, p.out_in, p.w.p, p.wn.p,
                        static_cast<const void*>(p.h), static_cast<const void*>(p.out),
                        static_cast<const void*>(p.dx), static_cast<const void*>(p.dy),
                        static_cast<const void*>(p.dgate)})
    if (!b4::aligned16(q)) return false;
  const bool x = p.x != nullptr, y = p.y != nullptr, g = p.gate != nullptr, d = p.dout != nullptr;
  const bool h = p.dh != nullptr, r = p.dres != nullptr, o = p.out_in != nullptr, s = p.S > 1;
  const uint32_t strides[] = {x ? p.x_ts : 0,         x && s ? p.x_ss : 0,    y ? p.y_ts : 0,
                             g ? p.gate_ts : 0,      d ? p.dout_ts : 0,      d && s ? p.dout_ss : 0,
                             h ? p.dh_ts : 0,        r ? p.dres_ts : 0,      r && s ? p.dres_ss : 0,
                             o ? p.out_ts : 0,       o && s ? p.out_ss : 0};
  for (uint32_t v : strides)
    if (v % V != 0) return false;
  return true;
}

// Column sums of partial weight gradients part [rows, C]; blockIdx.y picks
// the weight.  32 columns to a CTA, kFinishRows rows at a time, a fixed order.
// At most 10 MB that are still in L2: what it costs is the launch and the
// loads' latency.  So it is launched while the pass before it still runs and
// waits for its results inside (let_next_launch), and has kFinishAhead loads
// in flight.  leave's gradient at 5001 x 4 x 1001 bf16, both launches: 16 rows
// of 4 loads behind the pass 60.9 us, 32 of 8 59.6, with the early launch
// 57.6; leave_enter's at 16384 x 1 x 512: 25.3, 25.0, 23.2.
struct Finish {
  const float* part[2];
  void* out[2];
  int bf16[2];
  int rows, C;
};
constexpr int kFinishRows = 32, kFinishAhead = 8;
__global__ void __launch_bounds__(32 * kFinishRows) finish_weights_kernel(const Finish f) {
  __shared__ float s[kFinishRows][33];
  const int which = blockIdx.y, c = blockIdx.x * 32 + threadIdx.x;
  const float* part = f.part[which];
  float d = 0.0f;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (c < f.C) {
#pragma unroll kFinishAhead
    for (int r = threadIdx.y; r < f.rows; r += kFinishRows) d += part[int64_t(r) * pitch(f.C) + c];
  }
  s[threadIdx.y][threadIdx.x] = d;
  __syncthreads();
  if (threadIdx.y != 0 || c >= f.C) return;
#pragma unroll
  for (int r = 1; r < kFinishRows; ++r) d += s[r][threadIdx.x];
  put_any(f.out[which], f.bf16[which], c, d);
}

// The scratch of a backward pass, split into rows for dw and dw_next.
int place_workspace(const hcb_args* a, Params* p) {
  const int n = (a->dw != nullptr) + (a->dw_next != nullptr && a->dh != nullptr && a->dout != nullptr);
  if (n == 0) return B4_OK;
  if (a->workspace == nullptr || !b4::aligned16(a->workspace) ||
      a->workspace_bytes < hcb_workspace_bytes(a->T, a->C, n))
    return B4_EINVAL;
  float* w = static_cast<float*>(a->workspace);
  const int64_t row = std::min<int64_t>(a->T, kMaxRows) * pitch(a->C);
  if (a->dw != nullptr) p->dw = w, w += row;
  if (n == 2 || a->dw == nullptr) p->dwn = w;
  return B4_OK;
}

cudaError_t finish(const hcb_args* a, const Params& p, int rows, cudaStream_t s) {
  Finish f;
  memset(&f, 0, sizeof(f));
  int n = 0;
  const bool next = a->dw_next != nullptr && a->dh != nullptr && a->dout != nullptr;
  if (a->dw != nullptr) f.part[n] = p.dw, f.out[n] = a->dw, f.bf16[n++] = p.w.bf16;
  if (next) f.part[n] = p.dwn, f.out[n] = a->dw_next, f.bf16[n++] = p.wn.bf16;
  if (n == 0) return cudaSuccess;
  f.rows = rows, f.C = a->C;
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t how;
  memset(&how, 0, sizeof(how));
  how.gridDim = dim3((a->C + 31) / 32, n), how.blockDim = dim3(32, kFinishRows), how.stream = s;
  how.attrs = &early, how.numAttrs = 1;
  return cudaLaunchKernelEx(&how, finish_weights_kernel, f);
}

}  // namespace
}  // namespace hcb

using namespace hcb;

extern "C" {

size_t hcb_workspace_bytes(int64_t T, int32_t C, int32_t weights) {
  if (T <= 0 || C < 1 || C > HCB_MAX_CHANNELS || weights < 1 || weights > 2) return 0;
  return static_cast<size_t>(std::min<int64_t>(T, kMaxRows)) * pitch(C) * weights * sizeof(float);
}

int hcb_enter(const hcb_args* a, birkhoff4_stream_t stream) {
  const int st = check_sizes(a);
  if (st != B4_OK) return st;
  if (a->T == 0) return B4_OK;
  if (a->x == nullptr || a->h == nullptr) return B4_EINVAL;
  Params p = params_of(a);
  p.x = a->x, p.h = a->h;
  p.wn.p = nullptr;
  return b4::record_cuda_error(enter_forward(p, a->x_dtype == B4_BF16, a->y_dtype == B4_BF16,
                                             vectors(a, p), reinterpret_cast<cudaStream_t>(stream)));
}

int hcb_enter_backward(const hcb_args* a, birkhoff4_stream_t stream) {
  int st = check_sizes(a);
  if (st != B4_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  Params p = params_of(a);
  p.wn.p = nullptr;
  if (a->T > 0) {
    if (a->x == nullptr || a->dh == nullptr) return B4_EINVAL;
    if (a->da != nullptr && a->a == nullptr) return B4_EINVAL;
    if (a->dres != nullptr && a->dx == nullptr) return B4_EINVAL;
    hcb_args only = *a;  // enter has one weight
    only.dw_next = nullptr;
    st = place_workspace(&only, &p);
    if (st != B4_OK) return st;
    p.x = a->x, p.dh = a->dh, p.dres = a->dres, p.dx = a->dx, p.da = a->da;
    int rows = 0;
    cudaError_t e = enter_backward(p, a->x_dtype == B4_BF16, a->y_dtype == B4_BF16, vectors(a, p), &rows, s);
    if (e == cudaSuccess) e = finish(&only, p, rows, s);
    return b4::record_cuda_error(e);
  }
  hcb_args only = *a;
  only.dw_next = nullptr;
  return b4::record_cuda_error(finish(&only, p, 0, s));
}

int hcb_leave(const hcb_args* a, birkhoff4_stream_t stream) {
  const int st = check_sizes(a);
  if (st != B4_OK) return st;
  if ((a->act == HCB_ACT_NONE) != (a->gate == nullptr) && a->T > 0) return B4_EINVAL;
  if (a->T == 0) return B4_OK;
  if (a->x == nullptr || a->y == nullptr || a->out == nullptr) return B4_EINVAL;
  Params p = params_of(a);
  p.x = a->x, p.y = a->y, p.gate = a->gate, p.out = a->out, p.h = a->h;
  if (a->h == nullptr) p.wn.p = nullptr;
  const int xb = a->x_dtype == B4_BF16, yb = a->y_dtype == B4_BF16;
  const bool vec = vectors(a, p);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (!residual_forward(p, xb, yb, vec, s, &e)) e = leave_forward(p, xb, yb, vec, s);
  return b4::record_cuda_error(e);
}

int hcb_leave_backward(const hcb_args* a, birkhoff4_stream_t stream) {
  int st = check_sizes(a);
  if (st != B4_OK) return st;
  if ((a->act == HCB_ACT_NONE) != (a->gate == nullptr) && a->T > 0) return B4_EINVAL;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  Params p = params_of(a);
  const bool next = a->dh != nullptr;
  if (a->T == 0) {
    // no rows: the weight gradients are sums of nothing
    hcb_args zero = *a;
    static const char any = 0;
    zero.dh = zero.dout = a->dw_next != nullptr ? &any : nullptr;
    return b4::record_cuda_error(finish(&zero, p, 0, s));
  }
  if (a->dout == nullptr || a->y == nullptr) return B4_EINVAL;
  if (a->P != nullptr && a->x == nullptr) return B4_EINVAL;
  if (a->dP != nullptr && a->P == nullptr) return B4_EINVAL;
  if (a->db != nullptr && a->b == nullptr) return B4_EINVAL;
  if (a->dgate != nullptr && a->gate == nullptr) return B4_EINVAL;
  if (next && (a->out_in == nullptr || a->dx == nullptr)) return B4_EINVAL;
  if (next && a->da != nullptr && a->a == nullptr) return B4_EINVAL;
  st = place_workspace(a, &p);
  if (st != B4_OK) return st;
  p.dout = a->dout, p.y = a->y, p.gate = a->gate, p.dx = a->dx, p.dy = a->dy, p.dgate = a->dgate;
  p.dP = a->dP, p.db = a->db;
  if (a->P != nullptr) p.x = a->x;
  if (next) {
    p.dh = a->dh, p.out_in = a->out_in, p.da = a->da;
  } else {
    p.wn.p = nullptr;
  }
  int rows = 0;
  const int xb = a->x_dtype == B4_BF16, yb = a->y_dtype == B4_BF16;
  const bool vec = vectors(a, p);
  cudaError_t e;
  if (!residual_backward(p, xb, yb, vec, &rows, s, &e))
    e = (next ? leave_enter_backward : leave_backward)(p, xb, yb, vec, &rows, s);
  if (e == cudaSuccess) e = finish(a, p, rows, s);
  return b4::record_cuda_error(e);
}

}  // extern "C"
