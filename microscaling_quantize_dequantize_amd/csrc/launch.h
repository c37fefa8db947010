// Internal launchers (host side).  Arguments are validated by the C ABI in
// api.hip before any of these is called; n is the element count M*K (> 0,
// a multiple of 32 and of the rotation block).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_device.h"

namespace mx {

enum Op { OP_QDQ = 0, OP_QUANT = 1, OP_ROTATE = 2 };

// Number of compute units of the current device (cached per device).
int device_cu_count();

// Workgroups of 256 threads that a launch holds in x: fewer than 2^32 threads.
constexpr int64_t MAX_GROUPS_256 = ((int64_t)1 << 24) - 1;
constexpr int CACHE_WRITE_TILE = 8, CACHE_READ_TILE = 16;  // tokens of a workgroup
constexpr int ROPE_TABLE = 2048;                           // angles of a workgroup: (token, pair) entries

// bl == nullptr: row-major scales; otherwise the blocked layout it describes.
hipError_t launch_unrot(int fmt, int op, int dtype, const void *src, void *dst, uint8_t *codes,
                        uint8_t *scales, int64_t n, hipStream_t stream, const BlockedScales *bl = nullptr);

hipError_t launch_dequant(int fmt, int dtype, const uint8_t *codes, const uint8_t *scales,
                          void *dst, int64_t n, hipStream_t stream);

hipError_t launch_rot(int fmt, int op, int dtype, const void *src, const void *rot, int r,
                      void *dst, uint8_t *codes, uint8_t *scales, int64_t n, hipStream_t stream,
                      const BlockedScales *bl = nullptr);

// bf16 source, any rotation size: the lane-owned kernels of rotl.hip.  fmt
// 0 MXFP4 and 1 MXFP8, quantize only (op OP_QUANT; anything else returns
// hipErrorInvalidValue; bl: blocked scales, or nullptr for row-major), 2
// NVFP4, QDQ or quantize (g: device pointer to the per-tensor multiplier).
hipError_t launch_rot_lanes(int fmt, int op, const void *src, const void *rot, int r, void *dst, uint8_t *codes,
                            uint8_t *scales, int64_t n, hipStream_t stream, const BlockedScales *bl,
                            const float *g = nullptr);

// NVFP4 (g: device pointer to the per-tensor fp32 multiplier; n = M*K).
hipError_t launch_nv_unrot(int op, const void *src, void *dst, uint8_t *codes, uint8_t *scales, const float *g,
                           int64_t n, hipStream_t stream);
hipError_t launch_nv_dequant(int dtype, const uint8_t *codes, const uint8_t *scales, const float *g, void *dst,
                             int64_t n, hipStream_t stream);
hipError_t launch_nv_rot(int op, const void *src, const void *rot, int r, void *dst, uint8_t *codes,
                         uint8_t *scales, const float *g, int64_t n, hipStream_t stream);

hipError_t launch_scales_to_blocked(const uint8_t *scales, const BlockedScales &bl, uint8_t *out,
                                    hipStream_t stream);

// scale_layout 0: row-major [rows x K/32]; 1: the blocked layout.
hipError_t launch_gemm(int fmt, const uint8_t *a, const uint8_t *as, const uint8_t *b, const uint8_t *bs,
                       int scale_layout, int64_t M, int64_t N, int64_t K, float alpha, int out_dtype, void *c,
                       hipStream_t stream);

// Rotary positions (strides: src token, src head, dst token, dst head, in elements).
hipError_t launch_rope(int dtype, const void *src, void *dst, int64_t tokens, int64_t heads, int64_t dim,
                       const int64_t strides[4], const int64_t *positions, const double *inv_freq, int64_t rot,
                       int layout, double scale, int inverse, hipStream_t stream);

// The paged cache as the kernels take it: [0] keys, [1] values.
struct CacheView {
  uint8_t *codes[2], *scales[2];
  int64_t pages;
  int fmt, heads, dim, page_log2;
};

// Strides: token, head, in elements.
hipError_t launch_cache_write(const CacheView &cache, const void *k, const int64_t k_strides[2], const void *v,
                              const int64_t v_strides[2], const int64_t *slots, int64_t tokens,
                              const int64_t *positions, const double *inv_freq, int64_t rot, int layout, double scale,
                              hipStream_t stream);
hipError_t launch_cache_read(const CacheView &cache, const int64_t *slots, int64_t tokens, void *k, void *v,
                             hipStream_t stream);

constexpr float LOG2_E = 1.4426950408889634f;  // weights are powers of two: the scores' factor is scale * LOG2_E

struct AttentionArgs {
  CacheView cache;
  const unsigned short *q;
  unsigned short *out;
  int64_t q_token, q_head;  // strides in elements
  const int *q_starts, *kv_lens, *table;
  const int64_t *tree;  // nullptr: causal
  int64_t table_stride;
  float *partial;  // workspace
  int batch, group, table_pages, total_q, max_q, max_kv, tree_words;
  float scale;
};

int64_t attention_workspace(int fmt, int dim, int heads, int group, int batch, int64_t total_q, int64_t max_q,
                            int64_t max_kv);
hipError_t launch_cache_attention(const AttentionArgs &a, hipStream_t stream);

}  // namespace mx
