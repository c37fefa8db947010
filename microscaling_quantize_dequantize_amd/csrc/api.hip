// C ABI of libmxqdq: argument validation and kernel selection.  Everything
// here runs on the host before the single kernel launch of each call; no
// call allocates, frees or synchronizes.
#include <stdint.h>

#include <atomic>

#include "../../include/libmxqdq.h"
#include "launch.h"

namespace {

thread_local hipStream_t tl_stream = nullptr;

// Largest accepted element count (2^46); far beyond any device memory, and it
// keeps every 64-bit index computation in range.
constexpr int64_t MAX_ELEMS = (int64_t)1 << 46;

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

int check_fmt(int fmt) { return (fmt == MX_FMT_E2M1 || fmt == MX_FMT_E4M3) ? MX_OK : MX_EFMT; }

int check_dtype(int dt) { return (dt == MX_DTYPE_BF16 || dt == MX_DTYPE_F32) ? MX_OK : MX_EDTYPE; }

int check_shape(int64_t M, int64_t K) {
  if (M < 0 || K < 0 || K % 32 != 0) return MX_ESHAPE;
  if (K > 0 && M > MAX_ELEMS / K) return MX_ESHAPE;
  return MX_OK;
}

int check_rot(const void *rot, int r, int64_t K, bool allow_none) {
  if (r == 0) return allow_none ? MX_OK : MX_EROT;
  if (r != 16 && r != 32 && r != 64 && r != 128) return MX_EROT;
  if (K % r != 0) return MX_EROT;
  if (rot == nullptr) return MX_EROT;
  return MX_OK;
}

int launched(hipError_t e) { return e == hipSuccess ? MX_OK : MX_ELAUNCH; }

}  // namespace

namespace mx {

int device_cu_count() {
  // per device, filled on first use (threads that race here store the same value)
  static std::atomic<int> cache[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
  int n = cache[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0) n = 256;
    cache[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

}  // namespace mx

extern "C" {

MX_API int mx_qdq(int fmt, const void *src, int src_dtype, int64_t M, int64_t K, const void *rot,
                  int rot_size, void *dst) {
  int st;
  if ((st = check_fmt(fmt)) || (st = check_dtype(src_dtype)) || (st = check_shape(M, K)) ||
      (st = check_rot(rot, rot_size, K, true)))
    return st;
  if (M == 0 || K == 0) return MX_OK;
  if (!src || !dst) return MX_ENULL;
  if (!aligned(src, 16) || !aligned(dst, 16) || (rot_size && !aligned(rot, 16))) return MX_EALIGN;
  const int64_t n = M * K;
  if (rot_size == 0)
    return launched(mx::launch_unrot(fmt, mx::OP_QDQ, src_dtype, src, dst, nullptr, nullptr, n, tl_stream));
  return launched(mx::launch_rot(fmt, mx::OP_QDQ, src_dtype, src, rot, rot_size, dst, nullptr, nullptr, n,
                                 tl_stream));
}

MX_API int mx_quantize(int fmt, const void *src, int64_t M, int64_t K, const void *rot, int rot_size,
                       uint8_t *codes, uint8_t *scales) {
  int st;
  if ((st = check_fmt(fmt)) || (st = check_shape(M, K)) || (st = check_rot(rot, rot_size, K, true)))
    return st;
  if (M == 0 || K == 0) return MX_OK;
  if (!src || !codes || !scales) return MX_ENULL;
  if (!aligned(src, 16) || !aligned(codes, 16) || !aligned(scales, 4) || (rot_size && !aligned(rot, 16)))
    return MX_EALIGN;
  const int64_t n = M * K;
  if (rot_size == 0)
    return launched(mx::launch_unrot(fmt, mx::OP_QUANT, MX_DTYPE_BF16, src, nullptr, codes, scales, n,
                                     tl_stream));
  return launched(mx::launch_rot(fmt, mx::OP_QUANT, MX_DTYPE_BF16, src, rot, rot_size, nullptr, codes, scales,
                                 n, tl_stream));
}

MX_API int mx_dequantize(int fmt, const uint8_t *codes, const uint8_t *scales, int64_t M, int64_t K,
                         int dst_dtype, void *dst) {
  int st;
  if ((st = check_fmt(fmt)) || (st = check_dtype(dst_dtype)) || (st = check_shape(M, K))) return st;
  if (M == 0 || K == 0) return MX_OK;
  if (!codes || !scales || !dst) return MX_ENULL;
  if (!aligned(codes, 16) || !aligned(dst, 16)) return MX_EALIGN;
  return launched(mx::launch_dequant(fmt, dst_dtype, codes, scales, dst, M * K, tl_stream));
}

MX_API int mx_rotate(const void *src, int src_dtype, int64_t M, int64_t K, const void *rot, int rot_size,
                     float *dst) {
  int st;
  if ((st = check_dtype(src_dtype)) || (st = check_shape(M, K)) || (st = check_rot(rot, rot_size, K, false)))
    return st;
  if (M == 0 || K == 0) return MX_OK;
  if (!src || !dst) return MX_ENULL;
  if (!aligned(src, 16) || !aligned(dst, 16) || !aligned(rot, 16)) return MX_EALIGN;
  return launched(mx::launch_rot(0, mx::OP_ROTATE, src_dtype, src, rot, rot_size, dst, nullptr, nullptr, M * K,
                                 tl_stream));
}

MX_API int64_t mx_blocked_scales_bytes(int64_t M, int64_t K) {
  if (check_shape(M, K) != MX_OK) return MX_ESHAPE;
  return ((M + 31) / 32) * ((K / 32 + 7) / 8) * 256;
}

MX_API int mx_scales_to_blocked(const uint8_t *scales, int64_t M, int64_t K, uint8_t *blocked) {
  int st;
  if ((st = check_shape(M, K))) return st;
  if (M == 0 || K == 0) return MX_OK;
  if (!scales || !blocked) return MX_ENULL;
  if (!aligned(blocked, 4)) return MX_EALIGN;
  const mx::BlockedScales bl{M, K / 32, (K / 32 + 7) / 8};
  if ((M + 31) / 32 > (int64_t)INT32_MAX || (bl.gblocks + 7) / 8 > 65535) return MX_ESHAPE;  // grid limits
  return launched(mx::launch_scales_to_blocked(scales, bl, blocked, tl_stream));
}

MX_API int mx_quantize_blocked(int fmt, const void *src, int64_t M, int64_t K, const void *rot, int rot_size,
                               uint8_t *codes, uint8_t *blocked_scales) {
  int st;
  if ((st = check_fmt(fmt)) || (st = check_shape(M, K)) || (st = check_rot(rot, rot_size, K, true)))
    return st;
  if (M == 0 || K == 0) return MX_OK;
  if (!src || !codes || !blocked_scales) return MX_ENULL;
  if (!aligned(src, 16) || !aligned(codes, 16) || !aligned(blocked_scales, 4) || (rot_size && !aligned(rot, 16)))
    return MX_EALIGN;
  const mx::BlockedScales bl{M, K / 32, (K / 32 + 7) / 8};
  const int64_t n = M * K;
  if (rot_size == 0)
    return launched(mx::launch_unrot(fmt, mx::OP_QUANT, MX_DTYPE_BF16, src, nullptr, codes, blocked_scales, n,
                                     tl_stream, &bl));
  return launched(mx::launch_rot(fmt, mx::OP_QUANT, MX_DTYPE_BF16, src, rot, rot_size, nullptr, codes,
                                 blocked_scales, n, tl_stream, &bl));
}

MX_API int mx_matmul(int fmt, const uint8_t *a_codes, const uint8_t *a_scales, const uint8_t *b_codes,
                     const uint8_t *b_scales, int scale_layout, int64_t M, int64_t N, int64_t K, float alpha,
                     int out_dtype, void *c) {
  int st;
  if ((st = check_fmt(fmt)) || (st = check_dtype(out_dtype)) || (st = check_shape(M, K)) ||
      (st = check_shape(N, K)))
    return st;
  if (scale_layout != MX_SCALES_ROWMAJOR && scale_layout != MX_SCALES_BLOCKED) return MX_ELAYOUT;
  if (M > ((int64_t)65535 << 7) || (N + 127) / 128 > (int64_t)INT32_MAX) return MX_ESHAPE;  // grid limits
  if ((fmt == MX_FMT_E2M1 ? K / 2 : K) > ((int64_t)1 << 23)) return MX_ESHAPE;  // 32-bit buffer offsets
  if (M == 0 || N == 0) return MX_OK;
  if (!c) return MX_ENULL;
  if (K > 0 && (!a_codes || !a_scales || !b_codes || !b_scales)) return MX_ENULL;
  if (!aligned(a_codes, 16) || !aligned(b_codes, 16) || !aligned(c, 16)) return MX_EALIGN;
  if (scale_layout == MX_SCALES_BLOCKED && (!aligned(a_scales, 4) || !aligned(b_scales, 4))) return MX_EALIGN;
  return launched(mx::launch_gemm(fmt, a_codes, a_scales, b_codes, b_scales, scale_layout, M, N, K, alpha,
                                  out_dtype, c, tl_stream));
}

namespace {

int check_nv(int64_t M, int64_t K, const void *rot, int r) {
  if (M < 0 || K < 0 || K % 16 != 0) return MX_ESHAPE;
  if (K > 0 && M > MAX_ELEMS / K) return MX_ESHAPE;
  if (r != 0 && K % 32 != 0) return MX_EROT;  // rotation blocks hold whole 32-element tiles
  return check_rot(rot, r, K, true);
}

}  // namespace

MX_API int mx_nvfp4_quantize(const void *src, int64_t M, int64_t K, const void *rot, int rot_size,
                             const float *global_scale, uint8_t *codes, uint8_t *scales) {
  int st;
  if ((st = check_nv(M, K, rot, rot_size))) return st;
  if (M == 0 || K == 0) return MX_OK;
  if (!src || !global_scale || !codes || !scales) return MX_ENULL;
  if (!aligned(src, 16) || !aligned(codes, 16) || !aligned(scales, 4) || !aligned(global_scale, 4) ||
      (rot_size && !aligned(rot, 16)))
    return MX_EALIGN;
  if (rot_size == 0)
    return launched(mx::launch_nv_unrot(mx::OP_QUANT, src, nullptr, codes, scales, global_scale, M * K, tl_stream));
  return launched(mx::launch_nv_rot(mx::OP_QUANT, src, rot, rot_size, nullptr, codes, scales, global_scale, M * K,
                                    tl_stream));
}

MX_API int mx_nvfp4_qdq(const void *src, int64_t M, int64_t K, const void *rot, int rot_size,
                        const float *global_scale, void *dst) {
  int st;
  if ((st = check_nv(M, K, rot, rot_size))) return st;
  if (M == 0 || K == 0) return MX_OK;
  if (!src || !global_scale || !dst) return MX_ENULL;
  if (!aligned(src, 16) || !aligned(dst, 16) || !aligned(global_scale, 4) || (rot_size && !aligned(rot, 16)))
    return MX_EALIGN;
  if (rot_size == 0)
    return launched(mx::launch_nv_unrot(mx::OP_QDQ, src, dst, nullptr, nullptr, global_scale, M * K, tl_stream));
  return launched(mx::launch_nv_rot(mx::OP_QDQ, src, rot, rot_size, dst, nullptr, nullptr, global_scale, M * K,
                                    tl_stream));
}

MX_API int mx_nvfp4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t M, int64_t K,
                               const float *global_scale, int dst_dtype, void *dst) {
  int st;
  if ((st = check_dtype(dst_dtype)) || (st = check_nv(M, K, nullptr, 0))) return st;
  if (M == 0 || K == 0) return MX_OK;
  if (!codes || !scales || !global_scale || !dst) return MX_ENULL;
  if (!aligned(codes, 16) || !aligned(dst, 16) || !aligned(global_scale, 4)) return MX_EALIGN;
  return launched(mx::launch_nv_dequant(dst_dtype, codes, scales, global_scale, dst, M * K, tl_stream));
}

namespace {

bool fits(int64_t v, int64_t most) { return v >= 0 && v <= most; }

int check_rotary(int64_t dim, const int64_t *positions, const double *inv_freq, int64_t rot, int layout) {
  if (rot < 0 || rot % 2 != 0 || rot > dim) return MX_EARG;
  if (layout != MX_ROTARY_HALF && layout != MX_ROTARY_INTERLEAVED) return MX_ELAYOUT;
  if (rot > 0 && (!aligned(positions, 8) || !aligned(inv_freq, 8))) return MX_EALIGN;
  return MX_OK;
}

int check_cache(const mx_cache *c) {
  if (!c) return MX_ENULL;
  int st = check_fmt(c->fmt);
  if (st) return st;
  if (c->dim < 32 || c->dim > 256 || c->dim % 32 != 0 || c->heads < 1 || c->heads > 65535 || c->page < 16 ||
      c->page > 65536 || (c->page & (c->page - 1)) != 0 || c->pages < 0 || c->pages > INT32_MAX ||
      c->pages > MAX_ELEMS / ((int64_t)c->heads * c->page * c->dim))
    return MX_ESHAPE;
  if (!aligned(c->k_codes, 16) || !aligned(c->k_scales, 16) || !aligned(c->v_codes, 16) || !aligned(c->v_scales, 16))
    return MX_EALIGN;
  return MX_OK;
}

bool empty_cache(const mx_cache *c) { return !c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales; }

mx::CacheView view(const mx_cache *c) {
  return mx::CacheView{{c->k_codes, c->v_codes}, {c->k_scales, c->v_scales}, c->pages, c->fmt, c->heads, c->dim,
                       __builtin_ctz((unsigned)c->page)};
}

int check_attention(const mx_cache *c, int64_t q_heads, int64_t batch, int64_t total_q, int64_t max_q,
                    int64_t max_kv) {
  int st = check_cache(c);
  if (st) return st;
  if (c->dim != 64 && c->dim != 96 && c->dim != 128 && c->dim != 192 && c->dim != 256) return MX_EARG;
  if (q_heads < 1 || q_heads % c->heads != 0 || q_heads > 65535) return MX_ESHAPE;
  if (!fits(batch, 1 << 24) || !fits(total_q, INT32_MAX / q_heads) || !fits(max_q, INT32_MAX / q_heads) ||
      !fits(max_kv, INT32_MAX - 65536))
    return MX_ESHAPE;
  // rows of the batch with every sequence at its longest, the bound of the division's numbers
  if ((double)batch * q_heads * (double)(max_q < total_q ? max_q : total_q) > 4294967296.0) return MX_ESHAPE;
  return MX_OK;
}

}  // namespace

MX_API int mx_rope(const void *src, int64_t src_token_stride, int64_t src_head_stride, int dtype, int64_t tokens,
                   int64_t heads, int64_t dim, const int64_t *positions, const double *inv_freq, int64_t rot,
                   int layout, double scale, int inverse, void *dst, int64_t dst_token_stride,
                   int64_t dst_head_stride) {
  int st;
  if ((st = check_dtype(dtype))) return st;
  if (tokens < 0 || !fits(heads, 65535) || !fits(dim, 4096) || tokens > INT32_MAX) return MX_ESHAPE;
  if ((st = check_rotary(dim, positions, inv_freq, rot, layout))) return st;
  // grid limits: tokens of a workgroup at least, and their angles in its table
  if ((tokens + mx::MAX_GROUPS_256 - 1) / mx::MAX_GROUPS_256 * (rot / 2) > mx::ROPE_TABLE) return MX_ESHAPE;
  if (tokens == 0 || heads == 0 || dim == 0) return MX_OK;
  if (!src || !dst || (rot > 0 && (!positions || !inv_freq))) return MX_ENULL;
  const uintptr_t size = dtype == MX_DTYPE_F32 ? 4 : 2;
  if (!aligned(src, size) || !aligned(dst, size)) return MX_EALIGN;
  if (src == dst) {
    if (src_token_stride != dst_token_stride || src_head_stride != dst_head_stride) return MX_EARG;
    if (rot == 0) return MX_OK;
  }
  const int64_t strides[4] = {src_token_stride, src_head_stride, dst_token_stride, dst_head_stride};
  return launched(mx::launch_rope(dtype, src, dst, tokens, heads, dim, strides, positions, inv_freq, rot, layout, scale,
                                  inverse, tl_stream));
}

MX_API int mx_cache_write(const mx_cache *cache, const void *k, int64_t k_token_stride, int64_t k_head_stride,
                          const void *v, int64_t v_token_stride, int64_t v_head_stride, const int64_t *slots,
                          int64_t tokens, const int64_t *positions, const double *inv_freq, int64_t rot, int layout,
                          double scale) {
  int st;
  if ((st = check_cache(cache))) return st;
  if (!fits(tokens, mx::MAX_GROUPS_256 * mx::CACHE_WRITE_TILE)) return MX_ESHAPE;
  if ((st = check_rotary(cache->dim, positions, inv_freq, rot, layout))) return st;
  if (tokens == 0 || cache->pages == 0) return MX_OK;
  if (empty_cache(cache) || !k || !v || !slots || (rot > 0 && (!positions || !inv_freq))) return MX_ENULL;
  if (!aligned(k, 2) || !aligned(v, 2) || !aligned(slots, 8)) return MX_EALIGN;
  const int64_t ks[2] = {k_token_stride, k_head_stride}, vs[2] = {v_token_stride, v_head_stride};
  return launched(mx::launch_cache_write(view(cache), k, ks, v, vs, slots, tokens, positions, inv_freq, rot, layout,
                                         scale, tl_stream));
}

MX_API int mx_cache_read(const mx_cache *cache, const int64_t *slots, int64_t tokens, void *k, void *v) {
  int st;
  if ((st = check_cache(cache))) return st;
  if (!fits(tokens, mx::MAX_GROUPS_256 * mx::CACHE_READ_TILE)) return MX_ESHAPE;
  if (tokens == 0) return MX_OK;
  if ((cache->pages > 0 && empty_cache(cache)) || !slots || !k || !v) return MX_ENULL;
  if (!aligned(slots, 8) || !aligned(k, 16) || !aligned(v, 16)) return MX_EALIGN;
  return launched(mx::launch_cache_read(view(cache), slots, tokens, k, v, tl_stream));
}

MX_API int64_t mx_cache_attention_workspace(const mx_cache *cache, int64_t q_heads, int64_t batch, int64_t total_q,
                                            int64_t max_q, int64_t max_kv) {
  const int st = check_attention(cache, q_heads, batch, total_q, max_q, max_kv);
  if (st) return st;
  if (max_q > total_q) max_q = total_q;
  return mx::attention_workspace(cache->fmt, cache->dim, cache->heads, (int)(q_heads / cache->heads), (int)batch,
                                 total_q, max_q, max_kv);
}

MX_API int mx_cache_attention(const mx_cache *cache, const void *q, int64_t q_token_stride, int64_t q_head_stride,
                              int64_t q_heads, const int32_t *q_starts, const int32_t *kv_lens, int64_t batch,
                              const int32_t *block_table, int64_t table_stride, int64_t table_pages, int64_t total_q,
                              int64_t max_q, int64_t max_kv, const int64_t *tree, int64_t tree_words, float scale,
                              void *out, void *workspace, int64_t workspace_bytes) {
  int st;
  if ((st = check_attention(cache, q_heads, batch, total_q, max_q, max_kv))) return st;
  if (!fits(table_pages, INT32_MAX / cache->page) || table_stride < table_pages || !fits(tree_words, INT32_MAX))
    return MX_ESHAPE;
  if (!(scale > 0.0f && scale * mx::LOG2_E <= 3.402823466e38f)) return MX_EARG;  // the kernels' factor is finite
  if (tree && (max_q < total_q ? max_q : total_q) > 64 * tree_words) return MX_EARG;
  if (total_q == 0) return MX_OK;
  const bool none = batch == 0 || max_q == 0;  // no sequence has queries: zeros, if there is an output
  if (none && !out) return MX_OK;
  if (!out || (!none && (!q || !q_starts || !kv_lens))) return MX_ENULL;
  if (!none && max_kv > 0 && table_pages > 0 && (!block_table || cache->pages == 0 || empty_cache(cache)))
    return MX_ENULL;
  if (!aligned(q, 16) || !aligned(out, 16) || q_token_stride % 8 != 0 || q_head_stride % 8 != 0 ||
      !aligned(q_starts, 4) || !aligned(kv_lens, 4) || !aligned(block_table, 4) || !aligned(tree, 8))
    return MX_EALIGN;
  const int group = (int)(q_heads / cache->heads);
  if (max_q > total_q) max_q = total_q;
  const int64_t need = mx::attention_workspace(cache->fmt, cache->dim, cache->heads, group, (int)batch, total_q, max_q,
                                               max_kv);
  if (need > 0 && !workspace) return MX_ENULL;
  if (workspace_bytes < need) return MX_EARG;
  if (need > 0 && !aligned(workspace, 16)) return MX_EALIGN;
  const mx::AttentionArgs a{view(cache), (const unsigned short *)q, (unsigned short *)out, q_token_stride,
                            q_head_stride, q_starts, kv_lens, block_table, tree, table_stride, (float *)workspace,
                            (int)batch, group, (int)table_pages, (int)total_q, (int)max_q, (int)max_kv,
                            (int)tree_words, scale};
  return launched(mx::launch_cache_attention(a, tl_stream));
}

MX_API void mx_set_stream(void *stream) { tl_stream = (hipStream_t)stream; }

MX_API void *mx_get_stream(void) { return (void *)tl_stream; }

MX_API const char *mx_status_string(int status) {
  switch (status) {
    case MX_OK: return "ok";
    case MX_EFMT: return "invalid format (expected MX_FMT_E2M1 or MX_FMT_E4M3)";
    case MX_EDTYPE: return "invalid dtype (expected MX_DTYPE_BF16 or MX_DTYPE_F32)";
    case MX_ESHAPE: return "invalid shape (M, K >= 0, K a multiple of 32, M*K <= 2^46)";
    case MX_EROT: return "invalid rotation (size 16/32/64/128 dividing K, non-NULL matrix)";
    case MX_ENULL: return "a required pointer is NULL";
    case MX_EALIGN: return "misaligned pointer (16 bytes; scales 4 bytes)";
    case MX_ELAUNCH: return "kernel launch failed";
    case MX_ELAYOUT:
      return "invalid layout (expected MX_SCALES_ROWMAJOR or MX_SCALES_BLOCKED; rotary: MX_ROTARY_HALF or "
             "MX_ROTARY_INTERLEAVED)";
    case MX_EARG: return "invalid rotary, cache or attention argument";
    default: return "unknown status";
  }
}

}  // extern "C"
