// The paged MX cache: keys (rotated on the way, if asked) and values are
// quantised to MXFP4 or MXFP8 into their slots, and slots are read back.
//
// Layout, for `pages` pages of `page` tokens (a power of two, 16 at least)
// and H heads of D dimensions, kept apart for keys and values:
//   codes   [pages, H, page, D] bytes (MXFP8) or [pages, H, page, D/2] (MXFP4)
//   scales  [pages, H, D/32, page] E8M0 bytes
// so that a head's tokens of a page are contiguous, and so are the scales that
// consecutive tokens have for the same 32 dimensions: attention reads both in
// whole lines, and a lane of it four or sixteen tokens' scales in one load.
// Token slots are page * page_size + row.
//
// A lane owns 8 neighbouring dimensions of a (token, head), so four lanes hold
// the 32 of a scale and agree on it with two DPP permutations, as in the
// quantise kernels.  Keys are rotated in fp64 and rounded to bf16 before the
// scale is taken: the bf16 rounding and the element rounding after it have
// borders, and a rotation in fp32 would put some values on their wrong side.  The
// rounding to bf16 goes by way of fp32, as a conversion of fp64 commonly does: it
// differs from a single rounding for one value in some 10^5.
//
// Bound: HBM for reading (16384 tokens of 8 heads of 128 out of MXFP4 17 us, 71004
// of 5 heads of 96 out of MXFP8 33 us: 5.0 and 6.2 TB/s on MI355X).  Writing the
// former takes 27 us, 3.1 TB/s, and 17 without the rotation: the rest goes to
// forming the angles, in fp64 and before a row is loaded, and to the rotation.
// Loading the first rows before the angles (29 us), tiles of 16 tokens (27) and
// both pieces of a pair in one thread (26-27) were no faster.  64 tokens take 4 us.
#include "launch.h"
#include "rotary.h"

namespace mx {

constexpr int WRITE_THREADS = 256;
constexpr int WRITE_TABLE = CACHE_WRITE_TILE * 128;  // (token, pair) entries of up to 128 pairs: 16 KiB of LDS

struct WriteArgs {
  CacheView cache;
  const unsigned short *src[2];  // keys, values
  int64_t token_stride[2], head_stride[2];
  const int64_t *slots;
  Positions positions;
  const double *inv_freq;
  double scale;
  int64_t tokens;
  int half, tile, heads_per_wg;  // pairs rotated; tokens and heads of a workgroup
};

__device__ __forceinline__ double bf16_f64(unsigned short b) { return (double)__uint_as_float((unsigned)b << 16); }

template <bool VEC>
__device__ __forceinline__ u32x4 load8(const unsigned short *p) {
  if (VEC) return *(const u32x4 *)p;
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = (unsigned)p[2 * i] | ((unsigned)p[2 * i + 1] << 16);
  return o;
}

// Where the partners of dimensions d .. d + 7 are, if they are one aligned piece (half layout, half a multiple of 8).
__device__ __forceinline__ int partner_of(int d, int half) { return d < half ? d + half : d < 2 * half ? d - half : d; }

// The 8 dimensions w from d of a key x (a whole head), rotated; q: their partners if ALIGNED; tc, ts: cosines and
// sines of the token's pairs.
template <int LAYOUT, bool ALIGNED>
__device__ __forceinline__ u32x4 rotate8(const unsigned short *x, u32x4 w, u32x4 q, int d, int half, const double *tc,
                                         const double *ts) {
  if (d >= 2 * half) return w;
  double y[8];
  unsigned short own[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) own[e] = (unsigned short)(w[e / 2] >> (16 * (e & 1)));
  if (LAYOUT == ROTARY_INTERLEAVED) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const double a = bf16_f64(own[e]), b = bf16_f64(own[e + 1]);
      const int p = (d + e) / 2;
      const bool in = p < half;
      const double c = in ? tc[p] : 1.0, s = in ? ts[p] : 0.0;
      y[e] = in ? __builtin_fma(a, c, -(b * s)) : a;
      y[e + 1] = in ? __builtin_fma(b, c, a * s) : b;
    }
  } else if (ALIGNED) {
    const bool low = d < half;
    const int p = low ? d : d - half;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const double a = bf16_f64(own[e]), b = bf16_f64((unsigned short)(q[e / 2] >> (16 * (e & 1))));
      const double s = low ? -ts[p + e] : ts[p + e];
      y[e] = __builtin_fma(a, tc[p + e], b * s);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const double a = bf16_f64(own[e]);
      y[e] = a;
      if (d + e < 2 * half) {
        const bool low = d + e < half;
        const int p = low ? d + e : d + e - half;
        const double b = bf16_f64(x[low ? d + e + half : d + e - half]);
        y[e] = __builtin_fma(a, tc[p], b * (low ? -ts[p] : ts[p]));
      }
    }
  }
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = bf16x2_rne((float)y[2 * i], (float)y[2 * i + 1]);
  return o;
}

// A thread keeps its piece of 8 dimensions and takes (token, head) rows, WRITE_ROWS of them at a time so that their
// loads are under way together.
constexpr int WRITE_ROWS = 4;

// VEC: 16-byte loads (strides and pointers allow them).  ALIGNED: half layout whose partners are whole pieces.
template <int FMT, int LAYOUT, bool VEC, bool ALIGNED, bool AXES>
__global__ __launch_bounds__(WRITE_THREADS) void k_cache_write(WriteArgs a) {
  __shared__ double tc[WRITE_TABLE], ts[WRITE_TABLE];
  const CacheView &cv = a.cache;
  const bool value = blockIdx.z == 1;
  const int half = value ? 0 : a.half;
  const int64_t t0 = (int64_t)blockIdx.x * a.tile;
  const int nt = (int)(a.tokens - t0 < a.tile ? a.tokens - t0 : a.tile);
  const int h0 = blockIdx.y * a.heads_per_wg;
  const int nh = cv.heads - h0 < a.heads_per_wg ? cv.heads - h0 : a.heads_per_wg;
  for (int i = threadIdx.x; i < nt * half; i += WRITE_THREADS) {
    const int t = i / half, p = i - t * half;
    double s, c;
    sine_cosine(position_of<AXES>(a.positions, t0 + t, p) * a.inv_freq[p], s, c);
    tc[i] = c * a.scale;
    ts[i] = s * a.scale;
  }
  if (half) __syncthreads();
  const unsigned short *src = value ? a.src[1] : a.src[0];
  const int64_t st = value ? a.token_stride[1] : a.token_stride[0];
  const int64_t sh = value ? a.head_stride[1] : a.head_stride[0];
  uint8_t *codes = value ? cv.codes[1] : cv.codes[0], *scales = value ? cv.scales[1] : cv.scales[0];
  // rows: token fastest, then head, as neighbouring tokens of a head are neighbours in their page.  A row's pieces are
  // a multiple of 4, so the four lanes of a scale are in the loop together; threads past the last whole row have none.
  const int pieces = cv.dim / 8, pass = WRITE_THREADS / pieces;
  const int d = 8 * ((int)threadIdx.x % pieces), first = threadIdx.x / pieces, rows = nh * nt;
  if (first >= pass) return;
  for (int row0 = first; row0 < rows; row0 += pass * WRITE_ROWS) {
    u32x4 w[WRITE_ROWS], q[WRITE_ROWS];
    int64_t slot[WRITE_ROWS];
    const unsigned short *x[WRITE_ROWS];
#pragma unroll
    for (int k = 0; k < WRITE_ROWS; ++k) {
      int row = row0 + k * pass;
      row = row < rows ? row : rows - 1;
      const int h = row / nt, t = row - h * nt;
      x[k] = src + (t0 + t) * st + (h0 + h) * sh;
      w[k] = load8<VEC>(x[k] + d);
      q[k] = ALIGNED ? load8<VEC>(x[k] + partner_of(d, half)) : w[k];
      slot[k] = a.slots[t0 + t];
    }
#pragma unroll
    for (int k = 0; k < WRITE_ROWS; ++k) {
      const int row = row0 + k * pass;
      if (row >= rows) break;
      const int h = row / nt, t = row - h * nt;
      u32x4 v = w[k];
      if (half) v = rotate8<LAYOUT, ALIGNED>(x[k], v, q[k], d, half, tc + t * half, ts + t * half);
      unsigned m = piece_amax_bf16(v);
      m = umax(m, dpp<DPP_QUAD_1032>(m));
      m = umax(m, dpp<DPP_QUAD_2301>(m));
      const unsigned sb = scale_byte<FMT>(m << 16);
      const float sc = scale_operand(sb);
      if (slot[k] < 0 || slot[k] >= cv.pages << cv.page_log2) continue;  // padding: nothing is written
      const int64_t ph = (slot[k] >> cv.page_log2) * cv.heads + h0 + h;
      const int r = (int)(slot[k] & ((1 << cv.page_log2) - 1));
      if (FMT == 0) {
        unsigned c = fp4_from_bf16x8(v, sc);
        if (sb == 255u) c = 0u;
        *(unsigned *)(codes + ((ph << cv.page_log2) + r) * (cv.dim / 2) + d / 2) = c;
      } else {
        const unsigned c2 = e4m3_clamp_bf16x2(sb);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = clamp_bf16x2(v[i], c2);
        u32x2 c = fp8_from_bf16x8(v, sc);
        if (sb == 255u) c = u32x2{0x7F7F7F7Fu, 0x7F7F7F7Fu};
        *(u32x2 *)(codes + ((ph << cv.page_log2) + r) * cv.dim + d) = c;
      }
      if ((d & 31) == 0) scales[((ph * (cv.dim / 32) + d / 32) << cv.page_log2) + r] = (uint8_t)sb;
    }
  }
}

template <int FMT, int LAYOUT, bool VEC, bool ALIGNED>
static void write_start(dim3 grid, const WriteArgs &a, hipStream_t stream) {
  if (a.positions.axes) k_cache_write<FMT, LAYOUT, VEC, ALIGNED, true><<<grid, WRITE_THREADS, 0, stream>>>(a);
  else k_cache_write<FMT, LAYOUT, VEC, ALIGNED, false><<<grid, WRITE_THREADS, 0, stream>>>(a);
}

hipError_t launch_cache_write(const CacheView &cache, const void *k, const int64_t k_strides[2], const void *v,
                              const int64_t v_strides[2], const int64_t *slots, int64_t tokens,
                              const Positions &positions, const double *inv_freq, int64_t rot, int layout, double scale,
                              hipStream_t stream) {
  WriteArgs a{cache, {(const unsigned short *)k, (const unsigned short *)v}, {k_strides[0], v_strides[0]},
              {k_strides[1], v_strides[1]}, slots, positions, inv_freq, scale, tokens, (int)(rot / 2), 0, 0};
  a.tile = CACHE_WRITE_TILE;
  // all heads of a tile share its angles, unless there are too few tiles to fill the CUs
  const int64_t tiles = (tokens + a.tile - 1) / a.tile;
  int parts = 1;
  while (parts < cache.heads && tiles * parts < 2 * device_cu_count()) parts *= 2;
  a.heads_per_wg = (cache.heads + parts - 1) / parts;
  const dim3 grid((unsigned)tiles, (unsigned)((cache.heads + a.heads_per_wg - 1) / a.heads_per_wg), 2);
  bool vec = ((uintptr_t)k | (uintptr_t)v) % 16 == 0;
  for (int i = 0; i < 2; ++i) vec = vec && k_strides[i] % 8 == 0 && v_strides[i] % 8 == 0;
#define MX_WRITE(F, L, V, A) write_start<F, L, V, A>(grid, a, stream)
#define MX_FORMAT(F)                                                        \
  if (layout == ROTARY_INTERLEAVED) {                                       \
    if (vec) MX_WRITE(F, ROTARY_INTERLEAVED, true, false);                  \
    else MX_WRITE(F, ROTARY_INTERLEAVED, false, false);                     \
  } else if (vec && a.half % 8 == 0) MX_WRITE(F, ROTARY_HALF, true, true);  \
  else if (vec) MX_WRITE(F, ROTARY_HALF, true, false);                      \
  else MX_WRITE(F, ROTARY_HALF, false, false)
  if (cache.fmt == 0) {
    MX_FORMAT(0);
  } else {
    MX_FORMAT(1);
  }
#undef MX_FORMAT
#undef MX_WRITE
  return hipGetLastError();
}

// Slots back to bf16 [tokens, H, D]: the same pieces of 8 dimensions, rounded
// to nearest-even where a value is below bf16's range.  Slots outside the
// cache (padding) give zeros.
constexpr int READ_THREADS = 256, READ_TILE = CACHE_READ_TILE;

template <int FMT>
__global__ __launch_bounds__(READ_THREADS) void k_cache_read(CacheView cv, const int64_t *__restrict__ slots,
                                                             int64_t tokens, u32x4 *__restrict__ k,
                                                             u32x4 *__restrict__ v, int heads_per_wg) {
  const bool value = blockIdx.z == 1;
  const uint8_t *codes = value ? cv.codes[1] : cv.codes[0], *scales = value ? cv.scales[1] : cv.scales[0];
  u32x4 *dst = value ? v : k;
  const int64_t t0 = (int64_t)blockIdx.x * READ_TILE;
  const int nt = (int)(tokens - t0 < READ_TILE ? tokens - t0 : READ_TILE);
  const int h0 = blockIdx.y * heads_per_wg;
  const int nh = cv.heads - h0 < heads_per_wg ? cv.heads - h0 : heads_per_wg;
  const int pieces = cv.dim / 8, total = nh * nt * pieces;
  for (int i = threadIdx.x; i < total; i += READ_THREADS) {
    const int row = i / pieces, piece = i - row * pieces;
    const int h = row / nt, t = row - h * nt;
    const int64_t slot = slots[t0 + t];
    u32x4 o{0u, 0u, 0u, 0u};
    if (slot >= 0 && slot < cv.pages << cv.page_log2) {
      const int64_t ph = (slot >> cv.page_log2) * cv.heads + h0 + h;
      const int r = (int)(slot & ((1 << cv.page_log2) - 1));
      const unsigned sb = scales[((ph * (cv.dim / 32) + piece / 4) << cv.page_log2) + r];
      const int64_t at = ((ph << cv.page_log2) + r) * pieces + piece;
      const float sc = scale_operand(sb);
      o = FMT == 0 ? bf16x8_from_fp4(((const unsigned *)codes)[at], sc)
                   : bf16x8_from_fp8(((const u32x2 *)codes)[at], sc);
      if (sb == 255u) {
        const unsigned nn = BF16_NAN | (BF16_NAN << 16);
        o = u32x4{nn, nn, nn, nn};
      }
    }
    __builtin_nontemporal_store(o, dst + ((t0 + t) * cv.heads + h0 + h) * pieces + piece);
  }
}

hipError_t launch_cache_read(const CacheView &cache, const int64_t *slots, int64_t tokens, void *k, void *v,
                             hipStream_t stream) {
  const int64_t tiles = (tokens + READ_TILE - 1) / READ_TILE;
  int parts = 1;
  while (parts < cache.heads && tiles * parts < 4 * device_cu_count()) parts *= 2;
  const int per = (cache.heads + parts - 1) / parts;
  const dim3 grid((unsigned)tiles, (unsigned)((cache.heads + per - 1) / per), 2);
  if (cache.fmt == 0)
    k_cache_read<0><<<grid, READ_THREADS, 0, stream>>>(cache, slots, tokens, (u32x4 *)k, (u32x4 *)v, per);
  else
    k_cache_read<1><<<grid, READ_THREADS, 0, stream>>>(cache, slots, tokens, (u32x4 *)k, (u32x4 *)v, per);
  return hipGetLastError();
}

}  // namespace mx
