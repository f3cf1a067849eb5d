// C ABI of the residual block's operators (layer norm, linear, gated
// feed-forward): argument validation on the host, before any HIP call,
// workspace layout and dispatch.  Specified in include/mamba3_ssm.h.
#include "../../include/mamba3_ssm.h"

#include <hip/hip_runtime.h>

#include "m3_launch.hpp"

namespace {

constexpr int64_t kMaxWidth = int64_t(1) << 20;
constexpr int64_t kMaxRows = (int64_t(1) << 24) - 1;  // a block of 256 threads each stays under 2^32

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool aligned_all(std::initializer_list<const void*> ps, uintptr_t a) {
  for (const void* p : ps)
    if (!aligned(p, a)) return false;
  return true;
}

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

// A width and the row strides that go with it (0: contiguous).
m3_status check_width(int64_t width, std::initializer_list<int64_t> strides) {
  if (width <= 0) return M3_ERR_SHAPE;
  for (int64_t s : strides)
    if (s != 0 && s < width) return M3_ERR_SHAPE;
  if (width > kMaxWidth) return M3_ERR_UNSUPPORTED;
  for (int64_t s : strides)
    if (s > kMaxWidth) return M3_ERR_UNSUPPORTED;
  return M3_OK;
}

int64_t or_width(int64_t stride, int64_t width) { return stride ? stride : width; }

m3_status check_rows_type(int64_t rows, int32_t io_dtype, int32_t flags) {
  if (rows < 0) return M3_ERR_SHAPE;
  if (io_dtype != M3_F32 && io_dtype != M3_BF16) return M3_ERR_UNSUPPORTED;
  if (flags != 0 || rows > kMaxRows) return M3_ERR_UNSUPPORTED;
  return M3_OK;
}

m3_status check_norm(const m3_norm_dims* d) {
  if (!d) return M3_ERR_NULL;
  const m3_status st = check_rows_type(d->rows, d->io_dtype, d->flags);
  return st != M3_OK ? st : check_width(d->width, {d->x_stride, d->y_stride, d->skip_stride});
}

// The smallest tile any product kernel uses is 64 x 64.
bool tiles_fit(int64_t m, int64_t n) { return ((m + 63) / 64) * ((n + 63) / 64) < (int64_t(1) << 24); }

m3_status check_linear(const m3_linear_dims* d, bool gated, bool backward) {
  if (!d) return M3_ERR_NULL;
  m3_status st = check_rows_type(d->rows, d->io_dtype, d->flags & ~M3_FLAG_UNALIGNED);
  if (st != M3_OK) return st;
  if (d->reserved != 0 || d->act < M3_ACT_NONE || d->act > M3_ACT_SIGMOID) return M3_ERR_UNSUPPORTED;
  st = check_width(d->d_in, {d->x_stride});
  if (st == M3_OK) st = check_width(d->d_out, {d->y_stride, gated || backward ? 0 : d->residual_stride});
  if (st != M3_OK) return st;
  const int64_t n = gated ? 2 * d->d_out : d->d_out;
  if (n > kMaxWidth) return M3_ERR_UNSUPPORTED;
  if (!tiles_fit(d->rows, n) || (backward && (!tiles_fit(d->rows, d->d_in) || !tiles_fit(n, d->d_in))))
    return M3_ERR_UNSUPPORTED;
  return M3_OK;
}

int bf16(int32_t io_dtype) { return io_dtype == M3_BF16 ? 1 : 0; }
uintptr_t esize(int32_t io_dtype) { return io_dtype == M3_BF16 ? 2 : 4; }

m3_status hip_status(hipError_t e) { return e == hipSuccess ? M3_OK : M3_ERR_HIP; }

// Rows that the tiled products read 16 bytes at a time from 16-byte
// boundaries; others are first copied into rows padded with zeros.
int64_t padded(int64_t width, int32_t io_dtype) {
  const int64_t v = io_dtype == M3_BF16 ? 8 : 4;
  return (width + v - 1) / v * v;
}
bool off16(int64_t width, int64_t stride, const m3_linear_dims* d) {
  const int64_t es = (int64_t)esize(d->io_dtype);
  return (d->flags & M3_FLAG_UNALIGNED) || width * es % 16 != 0 || stride * es % 16 != 0;
}
// Without the flag, rows on 16 bytes have to start there.
bool base_ok(const void* p, bool packed) { return packed || aligned(p, 16); }

// A copy of rows x width into the workspace at `at` bytes, when needed.
struct Packer {
  m3::PackArgs args{};
  char* ws;
  int32_t io_dtype;
  void add(const void*& src, int64_t& ld, int64_t rows, int64_t width, size_t at) {
    auto& m = args.m[args.count++];
    m.src = src; m.dst = ws + at; m.rows = rows; m.width = width; m.src_ld = ld; m.ld = padded(width, io_dtype);
    src = m.dst;
    ld = m.ld;
  }
};

// Workspace of the forward: copies of x and W where their rows need them,
// then the split tiles' parts.
struct FwdWs {
  m3::MmPlan plan;
  bool pack_x, pack_w;
  size_t x, w, part, bytes;
};
FwdWs fwd_ws(const m3_linear_dims* d, bool gated) {
  FwdWs w{};
  if (d->rows == 0) return w;
  const size_t es = esize(d->io_dtype), n = (size_t)(gated ? 2 : 1) * d->d_out, row = padded(d->d_in, d->io_dtype) * es;
  w.plan = m3::mm_plan(bf16(d->io_dtype), gated ? m3::MM_GATED : m3::MM_LINEAR, d->rows, d->d_out, d->d_in);
  if (w.plan.tile != 0) {
    w.pack_x = off16(d->d_in, d->x_stride, d);
    w.pack_w = off16(d->d_in, 0, d);
  }
  w.w = w.pack_x ? up256(d->rows * row) : 0;
  w.part = w.w + (w.pack_w ? up256(n * row) : 0);
  w.bytes = w.part + w.plan.part_bytes;
  return w;
}

m3_status linear_fwd(const m3_linear_dims* d, bool gated, const void* x, const void* W, const float* bias,
                     const void* residual, void* y, void* pre, void* workspace, size_t workspace_bytes,
                     void* stream) {
  const m3_status st = check_linear(d, gated, false);
  if (st != M3_OK) return st;
  if (d->rows > 0 && (!x || !W || !y)) return M3_ERR_NULL;
  if (!aligned_all({x, W, residual, y, pre}, esize(d->io_dtype)) || !aligned(bias, 4) || !aligned(workspace, 16))
    return M3_ERR_ALIGN;
  const FwdWs w = fwd_ws(d, gated);
  if (w.plan.tile != 0 && (!base_ok(x, w.pack_x) || !base_ok(W, w.pack_w))) return M3_ERR_ALIGN;
  if (w.bytes > 0 && (!workspace || workspace_bytes < w.bytes)) return M3_ERR_WORKSPACE;
  if (d->rows == 0) return M3_OK;
  const hipStream_t s = (hipStream_t)stream;
  const int io = bf16(d->io_dtype);
  m3::MmArgs a{};
  a.P = x; a.ldp = or_width(d->x_stride, d->d_in);
  a.Q = W; a.ldq = d->d_in;
  a.M = d->rows; a.N = d->d_out; a.K = d->d_in;
  a.out = y; a.ldo = or_width(d->y_stride, d->d_out);
  a.bias = bias; a.res = residual; a.ldr = or_width(d->residual_stride, d->d_out);
  a.pre = pre; a.act = d->act;
  a.part = (float*)((char*)workspace + w.part);
  Packer pk{{}, (char*)workspace, d->io_dtype};
  if (w.pack_x) pk.add(a.P, a.ldp, a.M, a.K, w.x);
  if (w.pack_w) pk.add(a.Q, a.ldq, gated ? 2 * a.N : a.N, a.K, w.w);
  if (m3::launch_pack(io, pk.args, s) != hipSuccess) return M3_ERR_HIP;
  return hip_status(m3::launch_mm(io, m3::MM_PQ_K, gated ? m3::MM_GATED : m3::MM_LINEAR, a, w.plan, s));
}

// Workspace of the backward: dP in the io type (or the copy of dy where dP is
// dy itself), copies of x and W, the partial column sums, the split tiles'
// parts (of one product at a time).
struct BwdWs {
  m3::MmPlan dx, dw;
  bool has_dp, pack_dy, pack_x, pack_w;
  size_t dp, x, w, cols, part, bytes;
};
BwdWs bwd_ws(const m3_linear_dims* d, bool gated) {
  BwdWs w{};
  if (d->rows == 0) return w;
  const int io = bf16(d->io_dtype);
  const int64_t n = gated ? 2 * d->d_out : d->d_out, K = d->d_in;
  const size_t es = esize(d->io_dtype);
  w.dx = m3::mm_plan(io, m3::MM_STORE, d->rows, K, n);
  w.dw = m3::mm_plan(io, m3::MM_STORE, n, K, d->rows);
  w.has_dp = gated || d->act != M3_ACT_NONE;
  w.pack_dy = !w.has_dp && off16(d->d_out, d->y_stride, d);
  w.pack_x = off16(K, d->x_stride, d);
  w.pack_w = off16(K, 0, d);
  w.x = w.has_dp || w.pack_dy ? up256(d->rows * padded(n, d->io_dtype) * es) : 0;
  w.w = w.x + (w.pack_x ? up256(d->rows * padded(K, d->io_dtype) * es) : 0);
  w.cols = w.w + (w.pack_w ? up256(n * padded(K, d->io_dtype) * es) : 0);
  w.part = w.cols + up256(4 * n * (size_t)m3::act_bwd_parts(d->rows, d->d_out));
  w.bytes = w.part + (w.dx.part_bytes > w.dw.part_bytes ? w.dx.part_bytes : w.dw.part_bytes);
  return w;
}

m3_status linear_bwd(const m3_linear_dims* d, bool gated, const void* x, const void* W, const void* pre,
                     const void* dy, void* dx, void* dW, float* dbias, void* workspace, size_t workspace_bytes,
                     void* stream) {
  const m3_status st = check_linear(d, gated, true);
  if (st != M3_OK) return st;
  const bool has_dp = gated || d->act != M3_ACT_NONE, any = dx || dW || dbias;
  if (d->rows > 0 && ((dx && !W) || (dW && !x) || (any && (!dy || (has_dp && !pre))))) return M3_ERR_NULL;
  if (!aligned_all({x, W, pre, dy, dx, dW}, esize(d->io_dtype)) || !aligned(dbias, 4) || !aligned(workspace, 16))
    return M3_ERR_ALIGN;
  const BwdWs w = bwd_ws(d, gated);
  if (d->rows > 0 && ((dx && !base_ok(W, w.pack_w)) || (dW && !base_ok(x, w.pack_x)) ||
                      ((dx || dW) && !has_dp && !base_ok(dy, w.pack_dy))))
    return M3_ERR_ALIGN;
  if (!any) return M3_OK;
  if (w.bytes > 0 && (!workspace || workspace_bytes < w.bytes)) return M3_ERR_WORKSPACE;
  const hipStream_t s = (hipStream_t)stream;
  const int64_t n = gated ? 2 * d->d_out : d->d_out;
  const int io = bf16(d->io_dtype);
  if (d->rows == 0) {
    hipError_t e = hipSuccess;
    if (dW) e = m3::launch_zero(dW, n * d->d_in * (int64_t)esize(d->io_dtype), s);
    if (dbias && e == hipSuccess) e = m3::launch_zero(dbias, 4 * n, s);
    return hip_status(e);
  }
  char* ws = (char*)workspace;
  m3::MmArgs a{}, b{};
  a.P = dy; a.ldp = or_width(d->y_stride, d->d_out);
  a.part = b.part = (float*)(ws + w.part);
  a.Q = W; a.ldq = d->d_in;                             // dx[m][k] = sum_n dP[m][n] W[n][k]
  b.Q = x; b.ldq = or_width(d->x_stride, d->d_in);      // dW[n][k] = sum_m dP[m][n] x[m][k]
  const bool store_dp = has_dp && (dx || dW);
  if (store_dp || dbias) {
    m3::ActBwdArgs e{};
    e.pre = pre; e.dy = dy; e.ldy = a.ldp;
    e.ldp = padded(n, d->io_dtype);
    e.dp = store_dp ? ws + w.dp : nullptr;
    e.dbias = dbias;
    e.part = (float*)(ws + w.cols);
    e.rows = d->rows; e.cols = d->d_out; e.act = d->act; e.gated = gated;
    if (m3::launch_act_bwd(io, e, s) != hipSuccess) return M3_ERR_HIP;
    if (store_dp) {
      a.P = e.dp;
      a.ldp = e.ldp;
    }
  }
  Packer pk{{}, ws, d->io_dtype};
  if (w.pack_dy && (dx || dW)) pk.add(a.P, a.ldp, d->rows, n, w.dp);
  if (w.pack_x && dW) pk.add(b.Q, b.ldq, d->rows, d->d_in, w.x);
  if (w.pack_w && dx) pk.add(a.Q, a.ldq, n, d->d_in, w.w);
  if (m3::launch_pack(io, pk.args, s) != hipSuccess) return M3_ERR_HIP;
  b.P = a.P; b.ldp = a.ldp;
  a.M = d->rows; a.N = d->d_in; a.K = n;
  a.out = dx; a.ldo = d->d_in;
  b.M = n; b.N = d->d_in; b.K = d->rows;
  b.out = dW; b.ldo = d->d_in;
  hipError_t e = hipSuccess;
  if (dx && dW) e = m3::launch_mm_pair(io, a, w.dx, b, w.dw, s);
  else if (dx) e = m3::launch_mm(io, m3::MM_P_K, m3::MM_STORE, a, w.dx, s);
  else if (dW) e = m3::launch_mm(io, m3::MM_NONE_K, m3::MM_STORE, b, w.dw, s);
  return hip_status(e);
}

}  // namespace

extern "C" {

m3_status mamba3_layer_norm_fwd(const m3_norm_dims* d, const void* x, const float* gain, const float* bias,
                                float eps, void* y, float* mean, float* rstd, void* stream) {
  const m3_status st = check_norm(d);
  if (st != M3_OK) return st;
  if (!(eps >= 0.0f) || eps > 3.0e38f) return M3_ERR_UNSUPPORTED;
  if ((mean == nullptr) != (rstd == nullptr)) return M3_ERR_NULL;
  if (d->rows > 0 && (!x || !y)) return M3_ERR_NULL;
  if (!aligned_all({x, y}, esize(d->io_dtype)) || !aligned_all({gain, bias, mean, rstd}, 4)) return M3_ERR_ALIGN;
  if (d->rows == 0) return M3_OK;
  m3::NormArgs a{};
  a.x = x; a.gain = gain; a.bias = bias; a.y = y; a.mean = mean; a.rstd = rstd; a.eps = eps;
  a.rows = d->rows; a.width = d->width;
  a.x_stride = or_width(d->x_stride, d->width);
  a.y_stride = or_width(d->y_stride, d->width);
  return hip_status(m3::launch_norm_fwd(bf16(d->io_dtype), a, (hipStream_t)stream));
}

size_t mamba3_layer_norm_bwd_workspace_size(const m3_norm_dims* d) {
  if (check_norm(d) != M3_OK) return 0;
  return sizeof(float) * 2 * (size_t)d->width * (size_t)m3::norm_bwd_parts(bf16(d->io_dtype), d->rows, d->width);
}

m3_status mamba3_layer_norm_bwd(const m3_norm_dims* d, const void* x, const float* gain, const float* mean,
                                const float* rstd, const void* dy, const void* dskip, void* dx, float* dgain,
                                float* dbias, void* workspace, size_t workspace_bytes, void* stream) {
  const m3_status st = check_norm(d);
  if (st != M3_OK) return st;
  if (d->rows > 0 && (!x || !mean || !rstd || !dy)) return M3_ERR_NULL;
  if (!aligned_all({x, dy, dskip, dx}, esize(d->io_dtype)) ||
      !aligned_all({gain, mean, rstd, dgain, dbias, workspace}, 4))
    return M3_ERR_ALIGN;
  const hipStream_t s = (hipStream_t)stream;
  if (d->rows == 0) {
    hipError_t e = hipSuccess;
    if (dgain) e = m3::launch_zero(dgain, 4 * d->width, s);
    if (dbias && e == hipSuccess) e = m3::launch_zero(dbias, 4 * d->width, s);
    return hip_status(e);
  }
  const bool cols = dgain || dbias;
  if (cols && (!workspace || workspace_bytes < mamba3_layer_norm_bwd_workspace_size(d))) return M3_ERR_WORKSPACE;
  if (!cols && !dx) return M3_OK;
  m3::NormBwdArgs a{};
  a.x = x; a.gain = gain; a.mean = mean; a.rstd = rstd; a.dy = dy; a.dskip = dskip; a.dx = dx;
  a.dgain = dgain; a.dbias = dbias; a.part = (float*)workspace;
  a.rows = d->rows; a.width = d->width;
  a.x_stride = or_width(d->x_stride, d->width);
  a.y_stride = or_width(d->y_stride, d->width);
  a.skip_stride = or_width(d->skip_stride, d->width);
  return hip_status(m3::launch_norm_bwd(bf16(d->io_dtype), a, s));
}

size_t mamba3_linear_fwd_workspace_size(const m3_linear_dims* d) {
  return check_linear(d, false, false) == M3_OK ? fwd_ws(d, false).bytes : 0;
}

m3_status mamba3_linear_fwd(const m3_linear_dims* d, const void* x, const void* W, const float* bias,
                            const void* residual, void* y, void* pre, void* workspace, size_t workspace_bytes,
                            void* stream) {
  return linear_fwd(d, false, x, W, bias, residual, y, pre, workspace, workspace_bytes, stream);
}

size_t mamba3_linear_bwd_workspace_size(const m3_linear_dims* d) {
  return check_linear(d, false, true) == M3_OK ? bwd_ws(d, false).bytes : 0;
}

m3_status mamba3_linear_bwd(const m3_linear_dims* d, const void* x, const void* W, const void* pre, const void* dy,
                            void* dx, void* dW, float* dbias, void* workspace, size_t workspace_bytes,
                            void* stream) {
  return linear_bwd(d, false, x, W, pre, dy, dx, dW, dbias, workspace, workspace_bytes, stream);
}

size_t mamba3_gated_ffn_fwd_workspace_size(const m3_linear_dims* d) {
  return check_linear(d, true, false) == M3_OK ? fwd_ws(d, true).bytes : 0;
}

m3_status mamba3_gated_ffn_fwd(const m3_linear_dims* d, const void* x, const void* W, const float* bias, void* h,
                               void* pre, void* workspace, size_t workspace_bytes, void* stream) {
  return linear_fwd(d, true, x, W, bias, nullptr, h, pre, workspace, workspace_bytes, stream);
}

size_t mamba3_gated_ffn_bwd_workspace_size(const m3_linear_dims* d) {
  return check_linear(d, true, true) == M3_OK ? bwd_ws(d, true).bytes : 0;
}

m3_status mamba3_gated_ffn_bwd(const m3_linear_dims* d, const void* x, const void* W, const void* pre,
                               const void* dh, void* dx, void* dW, float* dbias, void* workspace,
                               size_t workspace_bytes, void* stream) {
  return linear_bwd(d, true, x, W, pre, dh, dx, dW, dbias, workspace, workspace_bytes, stream);
}

}  // extern "C"
