// C ABI of the attention layer's operators (head norms with rotation, windowed
// attention with sinks, that over a cache): argument validation on the host,
// before any HIP call, workspace layout and dispatch.  Specified in
// include/mamba3_ssm.h.
#include "../../include/mamba3_ssm.h"

#include <hip/hip_runtime.h>

#include "m3_common.hpp"
#include "m3_launch.hpp"

namespace {

constexpr int64_t kMaxWidth = int64_t(1) << 20;
constexpr int64_t kMaxRows = (int64_t(1) << 24) - 1;  // a block of 256 threads each stays under 2^32

bool aligned_all(std::initializer_list<const void*> ps, uintptr_t a) {
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) & (a - 1)) return false;
  return true;
}
int bf16(int32_t io_dtype) { return io_dtype == M3_BF16 ? 1 : 0; }
int64_t esize(int32_t io_dtype) { return io_dtype == M3_BF16 ? 2 : 4; }
int64_t or_width(int64_t stride, int64_t width) { return stride ? stride : width; }
size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }
m3_status hip_status(hipError_t e) { return e == hipSuccess ? M3_OK : M3_ERR_HIP; }
// a * b, or kMaxRows + 1 for anything above kMaxRows (a, b >= 0)
int64_t times(int64_t a, int64_t b) { return a != 0 && b > kMaxRows / a ? kMaxRows + 1 : a * b; }

// Heads side by side, and the row strides that go with them (0: contiguous).
m3_status check_row(int64_t heads, int64_t dim, std::initializer_list<int64_t> strides) {
  if (heads > kMaxWidth / dim) return M3_ERR_UNSUPPORTED;
  for (int64_t s : strides)
    if (s != 0 && s < heads * dim) return M3_ERR_SHAPE;
  for (int64_t s : strides)
    if (s > kMaxWidth) return M3_ERR_UNSUPPORTED;
  return M3_OK;
}

m3_status check(const m3_norm_rope_dims* d, bool backward) {
  if (!d) return M3_ERR_NULL;
  if (d->rows < 0 || d->seqlen < 0 || d->q_heads < 0 || d->k_heads < 0 || d->head_dim <= 0 || d->rope_dim < 0 ||
      d->rope_dim % 2 != 0 || d->rope_dim > d->head_dim)
    return M3_ERR_SHAPE;
  if (d->io_dtype != M3_F32 && d->io_dtype != M3_BF16) return M3_ERR_UNSUPPORTED;
  if ((d->flags & ~M3_FLAG_ROPE_HALVES) != 0 || d->rows > kMaxRows || d->head_dim > 256) return M3_ERR_UNSUPPORTED;
  m3_status st = check_row(d->q_heads, d->head_dim, {d->q_stride, d->q_out_stride, backward ? d->dq_stride : 0});
  if (st == M3_OK)
    st = check_row(d->k_heads, d->head_dim, {d->k_stride, d->k_out_stride, backward ? d->dk_stride : 0});
  return st;
}

m3::NormRopeArgs args_of(const m3_norm_rope_dims* d) {
  m3::NormRopeArgs a{};
  const int64_t wq = d->q_heads * d->head_dim, wk = d->k_heads * d->head_dim;
  a.rows = d->rows;
  a.seqlen = d->seqlen < d->rows ? (int)d->seqlen : 0;
  a.q_heads = (int)d->q_heads;
  a.k_heads = (int)d->k_heads;
  a.dim = (int)d->head_dim;
  a.rope = (int)d->rope_dim;
  a.halves = d->flags & M3_FLAG_ROPE_HALVES ? 1 : 0;
  a.q_stride = or_width(d->q_stride, wq);
  a.k_stride = or_width(d->k_stride, wk);
  a.q_out_stride = or_width(d->q_out_stride, wq);
  a.k_out_stride = or_width(d->k_out_stride, wk);
  a.dq_stride = or_width(d->dq_stride, wq);
  a.dk_stride = or_width(d->dk_stride, wk);
  return a;
}

// The parts of the dims that the three attention entry points share.
m3_status check_heads(int64_t batch, int64_t q_heads, int64_t kv_heads, int64_t dim, int64_t window, int64_t sinks,
                      float scale, int32_t io_dtype, int32_t reserved) {
  if (batch < 0 || q_heads <= 0 || kv_heads <= 0 || q_heads % kv_heads != 0 || dim <= 0 || window < 0 || sinks < 0)
    return M3_ERR_SHAPE;
  if (io_dtype != M3_F32 && io_dtype != M3_BF16) return M3_ERR_UNSUPPORTED;
  if (reserved != 0 || batch > kMaxRows || dim > 128 || dim % 8 != 0) return M3_ERR_UNSUPPORTED;
  if (!(scale > 0.0f) || scale > 2.35e38f) return M3_ERR_UNSUPPORTED;  // scale log2(e) is finite
  return M3_OK;
}
bool off16(std::initializer_list<int64_t> strides, int32_t io_dtype) {
  for (int64_t s : strides)
    if (s * esize(io_dtype) % 16 != 0) return true;
  return false;
}

bool packed(const m3_attn_dims* d) { return (d->flags & M3_FLAG_PACKED) != 0; }

m3_status check(const m3_attn_dims* d, bool backward) {
  if (!d) return M3_ERR_NULL;
  m3_status st = check_heads(d->batch, d->q_heads, d->kv_heads, d->head_dim, d->window, d->sinks, d->scale, d->io_dtype,
                             d->reserved);
  if (st != M3_OK) return st;
  if ((d->flags & ~M3_FLAG_PACKED) != 0) return M3_ERR_UNSUPPORTED;
  st = check_row(d->q_heads, d->head_dim,
                 {d->q_stride, d->o_stride, backward ? d->do_stride : 0, backward ? d->dq_stride : 0});
  if (st == M3_OK)
    st = check_row(d->kv_heads, d->head_dim,
                   {d->k_stride, d->v_stride, backward ? d->dk_stride : 0, backward ? d->dv_stride : 0});
  if (st != M3_OK) return st;
  if (off16({d->q_stride, d->k_stride, d->v_stride, d->o_stride}, d->io_dtype) ||
      (backward && off16({d->do_stride, d->dq_stride, d->dk_stride, d->dv_stride}, d->io_dtype)))
    return M3_ERR_ALIGN;
  if (packed(d)) {
    if (d->rows < 0) return M3_ERR_SHAPE;
    const int64_t tiles = d->rows / 128 + (d->batch < d->rows ? d->batch : d->rows);
    if (d->rows > kMaxRows || times(tiles, d->q_heads) > kMaxRows - 32768)
      return M3_ERR_UNSUPPORTED;
  } else {
    if (d->q_len < 0 || d->kv_len < 0 || (d->kv_rows != 0 && d->kv_rows < d->kv_len)) return M3_ERR_SHAPE;
    if (d->q_len > kMaxRows || d->kv_len > kMaxRows || times(d->batch, d->q_len) > kMaxRows ||
        times(times(d->batch, (d->q_len + 127) / 128), d->q_heads) > kMaxRows ||
        times(d->batch, d->kv_len) > kMaxRows ||
        times(times(d->batch, (d->kv_len + 127) / 128), d->kv_heads) > kMaxRows - 32768 ||
        d->kv_rows > (int64_t(1) << 40))
      return M3_ERR_UNSUPPORTED;
  }
  // the backward's rows of statistics, sixteen to a block
  if (backward && times(packed(d) ? d->rows : d->batch * d->q_len, (d->q_heads + 15) / 16) > kMaxRows)
    return M3_ERR_UNSUPPORTED;
  return M3_OK;
}

int64_t q_rows(const m3_attn_dims* d) { return packed(d) ? d->rows : d->batch * d->q_len; }
int64_t k_rows(const m3_attn_dims* d) { return packed(d) ? d->rows : d->batch * d->kv_len; }
int window_of(int64_t w) { return w == 0 || w >= m3::kNoWindow ? m3::kNoWindow : (int)w; }

// starts: only whether there are any, for the sizes.
m3::AttnArgs args_of(const m3_attn_dims* d, const int64_t* starts) {
  m3::AttnArgs a{};
  const int64_t wq = d->q_heads * d->head_dim, wk = d->kv_heads * d->head_dim;
  a.batch = d->batch;
  a.rows = q_rows(d);
  a.starts = packed(d) ? starts : nullptr;
  if (!packed(d)) {
    a.q_len = (int)d->q_len;
    a.kv_len = (int)d->kv_len;
    a.kv_rows = or_width(d->kv_rows, d->kv_len);
  }
  a.q_heads = (int)d->q_heads;
  a.kv_heads = (int)d->kv_heads;
  a.dim = (int)d->head_dim;
  a.window = window_of(d->window);
  const int64_t longest = packed(d) ? d->rows : d->kv_len;  // what is no key is no sink
  a.sinks = a.window == m3::kNoWindow ? 0 : (int)(d->sinks < longest ? d->sinks : longest);
  a.scale = d->scale;
  a.q_stride = or_width(d->q_stride, wq);
  a.k_stride = or_width(d->k_stride, wk);
  a.v_stride = or_width(d->v_stride, wk);
  a.o_stride = or_width(d->o_stride, wq);
  a.do_stride = or_width(d->do_stride, wq);
  a.dq_stride = or_width(d->dq_stride, wq);
  a.dk_stride = or_width(d->dk_stride, wk);
  a.dv_stride = or_width(d->dv_stride, wk);
  a.piece = m3::attn_bwd_piece(a);
  a.splits = m3::attn_bwd_splits(bf16(d->io_dtype), a);
  return a;
}

// Workspace of the backward: lse2, delta, the pieces' sums.
struct AttnBwdWs {
  size_t delta, part, bytes;
};
AttnBwdWs bwd_ws(const m3_attn_dims* d) {
  static const int64_t some = 0;
  AttnBwdWs w{};
  w.delta = up256(4 * (size_t)d->q_heads * (size_t)q_rows(d));
  w.part = 2 * w.delta;
  w.bytes = w.part + m3::attn_bwd_part_bytes(args_of(d, &some));
  return w;
}

m3_status check(const m3_attn_decode_dims* d) {
  if (!d) return M3_ERR_NULL;
  m3_status st = check_heads(d->batch, d->q_heads, d->kv_heads, d->head_dim, d->window, d->sinks, d->scale, d->io_dtype,
                             d->reserved);
  if (st != M3_OK) return st;
  if (d->tokens <= 0 || d->capacity <= 0) return M3_ERR_SHAPE;
  if (d->flags != 0 || d->tokens > 16 || d->capacity > (int64_t(1) << 30)) return M3_ERR_UNSUPPORTED;
  if (d->sinks >= d->capacity || d->capacity - d->sinks < d->tokens ||
      (d->window > 0 && d->capacity - d->sinks - d->tokens + 1 < d->window))
    return M3_ERR_SHAPE;
  st = check_row(d->q_heads, d->head_dim, {d->q_stride, d->o_stride});
  if (st == M3_OK)
    st = check_row(d->kv_heads, d->head_dim, {d->k_stride, d->v_stride, d->k_cache_stride, d->v_cache_stride});
  if (st != M3_OK) return st;
  if (off16({d->q_stride, d->k_stride, d->v_stride, d->o_stride, d->k_cache_stride, d->v_cache_stride}, d->io_dtype))
    return M3_ERR_ALIGN;
  const int64_t groups = (d->q_heads / d->kv_heads * d->tokens + 31) / 32;
  if (times(times(d->batch, d->kv_heads), groups) > kMaxRows ||
      times(times(d->batch, d->tokens), d->q_heads) > kMaxRows)
    return M3_ERR_UNSUPPORTED;
  return M3_OK;
}

m3::AttnDecodeArgs args_of(const m3_attn_decode_dims* d) {
  m3::AttnDecodeArgs a{};
  const int64_t wq = d->q_heads * d->head_dim, wk = d->kv_heads * d->head_dim;
  a.batch = d->batch;
  a.capacity = d->capacity;
  a.tokens = (int)d->tokens;
  a.q_heads = (int)d->q_heads;
  a.kv_heads = (int)d->kv_heads;
  a.dim = (int)d->head_dim;
  a.window = window_of(d->window);
  a.sinks = (int)d->sinks;
  a.scale = d->scale;
  a.q_stride = or_width(d->q_stride, wq);
  a.k_stride = or_width(d->k_stride, wk);
  a.v_stride = or_width(d->v_stride, wk);
  a.o_stride = or_width(d->o_stride, wq);
  a.kc_stride = or_width(d->k_cache_stride, wk);
  a.vc_stride = or_width(d->v_cache_stride, wk);
  a.splits = m3::attn_decode_splits(bf16(d->io_dtype), a);
  return a;
}

bool good_eps(float eps) { return eps >= 0.0f && eps <= 3.0e38f; }

}  // namespace

extern "C" {

m3_status mamba3_qk_norm_rope_fwd(const m3_norm_rope_dims* d, const void* q, const void* k, const float* gain_q,
                                  const float* gain_k, float eps, const float* theta, const int64_t* pos, void* q_out,
                                  void* k_out, void* stream) {
  const m3_status st = check(d, false);
  if (st != M3_OK) return st;
  if (!good_eps(eps)) return M3_ERR_UNSUPPORTED;
  if (d->rows > 0 && ((d->q_heads > 0 && (!q || !q_out)) || (d->k_heads > 0 && (!k || !k_out)) ||
                      (d->rope_dim > 0 && !theta)))
    return M3_ERR_NULL;
  if (!aligned_all({q, k, q_out, k_out}, esize(d->io_dtype)) || !aligned_all({gain_q, gain_k, theta}, 4) ||
      !aligned_all({pos}, 8))
    return M3_ERR_ALIGN;
  if (d->rows == 0 || d->q_heads + d->k_heads == 0) return M3_OK;
  m3::NormRopeArgs a = args_of(d);
  a.q = q; a.k = k; a.q_out = q_out; a.k_out = k_out;
  a.gain_q = gain_q; a.gain_k = gain_k; a.theta = theta; a.pos = pos; a.eps = eps;
  return hip_status(m3::launch_norm_rope(bf16(d->io_dtype), false, a, (hipStream_t)stream));
}

size_t mamba3_qk_norm_rope_bwd_workspace_size(const m3_norm_rope_dims* d) {
  if (check(d, true) != M3_OK || d->rows == 0 || d->q_heads + d->k_heads == 0) return 0;
  return sizeof(float) * 2 * (size_t)d->head_dim *
         (size_t)m3::norm_rope_parts(bf16(d->io_dtype), d->rows, d->q_heads + d->k_heads, d->head_dim, d->rope_dim);
}

m3_status mamba3_qk_norm_rope_bwd(const m3_norm_rope_dims* d, const void* q, const void* k, const void* dq_out,
                                  const void* dk_out, const float* gain_q, const float* gain_k, float eps,
                                  const float* theta, const int64_t* pos, void* dq, void* dk, float* dgain_q,
                                  float* dgain_k, void* workspace, size_t workspace_bytes, void* stream) {
  const m3_status st = check(d, true);
  if (st != M3_OK) return st;
  if (!good_eps(eps)) return M3_ERR_UNSUPPORTED;
  if (d->rows > 0 && ((d->q_heads > 0 && (!q || !dq_out || !dq)) || (d->k_heads > 0 && (!k || !dk_out || !dk)) ||
                      (d->rope_dim > 0 && !theta)))
    return M3_ERR_NULL;
  if (!aligned_all({q, k, dq_out, dk_out, dq, dk}, esize(d->io_dtype)) ||
      !aligned_all({gain_q, gain_k, theta, dgain_q, dgain_k, workspace}, 4) || !aligned_all({pos}, 8))
    return M3_ERR_ALIGN;
  const hipStream_t s = (hipStream_t)stream;
  if (d->rows == 0 || d->q_heads + d->k_heads == 0) {
    hipError_t e = hipSuccess;
    if (dgain_q) e = m3::launch_zero(dgain_q, 4 * d->head_dim, s);
    if (dgain_k && e == hipSuccess) e = m3::launch_zero(dgain_k, 4 * d->head_dim, s);
    return hip_status(e);
  }
  const bool gains = dgain_q || dgain_k;
  if (gains && (!workspace || workspace_bytes < mamba3_qk_norm_rope_bwd_workspace_size(d))) return M3_ERR_WORKSPACE;
  m3::NormRopeArgs a = args_of(d);
  a.q = q; a.k = k; a.dq_out = dq_out; a.dk_out = dk_out; a.q_out = dq; a.k_out = dk;
  a.gain_q = gain_q; a.gain_k = gain_k; a.theta = theta; a.pos = pos; a.eps = eps;
  a.part = gains ? (float*)workspace : nullptr;
  a.dgain_q = dgain_q; a.dgain_k = dgain_k;
  return hip_status(m3::launch_norm_rope(bf16(d->io_dtype), true, a, s));
}

m3_status mamba3_window_attn_fwd(const m3_attn_dims* d, const void* q, const void* k, const void* v,
                                 const int64_t* starts, void* o, float* lse, void* stream) {
  const m3_status st = check(d, false);
  if (st != M3_OK) return st;
  if ((q_rows(d) > 0 && (!q || !o || (k_rows(d) > 0 && (!k || !v)))) || (packed(d) && d->batch > 0 && !starts))
    return M3_ERR_NULL;
  if (!aligned_all({q, k, v, o}, 16) || !aligned_all({lse}, 4) || !aligned_all({starts}, 8)) return M3_ERR_ALIGN;
  if (d->batch == 0 || q_rows(d) == 0) return M3_OK;
  m3::AttnArgs a = args_of(d, starts);
  a.q = q; a.k = k; a.v = v; a.o = o; a.lse = lse;
  const hipStream_t s = (hipStream_t)stream;
  return hip_status(bf16(d->io_dtype) ? m3::launch_attn_fwd<m3::bf16_t>(a, s) : m3::launch_attn_fwd<float>(a, s));
}

size_t mamba3_window_attn_bwd_workspace_size(const m3_attn_dims* d) {
  return check(d, true) == M3_OK && d->batch > 0 && q_rows(d) > 0 ? bwd_ws(d).bytes : 0;
}

m3_status mamba3_window_attn_bwd(const m3_attn_dims* d, const void* q, const void* k, const void* v, const void* o,
                                 const float* lse, const void* dout, const int64_t* starts, void* dq, void* dk,
                                 void* dv, void* workspace, size_t workspace_bytes, void* stream) {
  const m3_status st = check(d, true);
  if (st != M3_OK) return st;
  const bool any = dq || dk || dv, queries = q_rows(d) > 0 && any;
  if ((queries && (!q || !o || !lse || !dout)) || (k_rows(d) > 0 && any && (!k || !v)) ||
      (packed(d) && d->batch > 0 && any && !starts))
    return M3_ERR_NULL;
  if (!aligned_all({q, k, v, o, dout, dq, dk, dv, workspace}, 16) || !aligned_all({lse}, 4) ||
      !aligned_all({starts}, 8))
    return M3_ERR_ALIGN;
  if (d->batch == 0 || !any) return M3_OK;
  const AttnBwdWs w = bwd_ws(d);
  if (queries && (!workspace || workspace_bytes < w.bytes)) return M3_ERR_WORKSPACE;
  m3::AttnArgs a = args_of(d, starts);
  a.q = q; a.k = k; a.v = v; a.o = (void*)o; a.lse = (float*)lse; a.dout = dout;
  a.dq = dq; a.dk = dk; a.dv = dv;
  a.lse2 = (float*)workspace;
  a.delta = (float*)((char*)workspace + w.delta);
  a.part = (float*)((char*)workspace + w.part);
  const hipStream_t s = (hipStream_t)stream;
  return hip_status(bf16(d->io_dtype) ? m3::launch_attn_bwd<m3::bf16_t>(a, s) : m3::launch_attn_bwd<float>(a, s));
}

size_t mamba3_window_attn_decode_workspace_size(const m3_attn_decode_dims* d) {
  return check(d) == M3_OK && d->batch > 0 ? m3::attn_decode_part_bytes(args_of(d)) : 0;
}

m3_status mamba3_window_attn_decode(const m3_attn_decode_dims* d, const void* q, const void* k, const void* v,
                                    void* k_cache, void* v_cache, const int64_t* lens, void* o, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  const m3_status st = check(d);
  if (st != M3_OK) return st;
  if (d->batch > 0 && (!q || !k || !v || !k_cache || !v_cache || !lens || !o)) return M3_ERR_NULL;
  if (!aligned_all({q, k, v, k_cache, v_cache, o, workspace}, 16) || !aligned_all({lens}, 8)) return M3_ERR_ALIGN;
  if (d->batch == 0) return M3_OK;
  m3::AttnDecodeArgs a = args_of(d);
  const size_t need = m3::attn_decode_part_bytes(a);
  if (need > 0 && (!workspace || workspace_bytes < need)) return M3_ERR_WORKSPACE;
  a.q = q; a.k = k; a.v = v; a.k_cache = k_cache; a.v_cache = v_cache; a.lens = lens; a.o = o;
  a.part = (float*)workspace;
  const hipStream_t s = (hipStream_t)stream;
  return hip_status(bf16(d->io_dtype) ? m3::launch_attn_decode<m3::bf16_t>(a, s)
                                      : m3::launch_attn_decode<float>(a, s));
}

}  // extern "C"
