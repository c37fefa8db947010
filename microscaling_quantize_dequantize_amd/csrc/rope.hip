// Rotary positions: y = R(position) x on the first `rot` dimensions of every
// head, the rest copied, and the inverse rotation for gradients.
//
//   pair p of rot/2:  a' = a c - b s,  b' = b c + a s,
//   c, s = scale cos, scale sin of position * inv_freq[p];  the inverse takes
//   -s, which is the transposed rotation, so it gives the gradient of x from
//   that of y.
//
// Bound: HBM, one read and one write of x (3 flops a rotated element).  The
// angles are formed once for each (token, pair) in fp64, rounded once to fp32
// and kept in LDS for all heads of the token, whose pairs are rotated in fp32
// whatever the type of x.  Measured on MI355X: 8192 x 64 heads of 128 in bf16
// 43 us, 6.3 TB/s; in fp32 104 us, 5.2 TB/s; 4111 x 16 heads of 96 in fp32 9.4 us,
// 5.4 TB/s; 8 tokens 3.4 us.
//
// Split: a workgroup owns whole tokens (one, or several while their heads are
// few), a thread VEC neighbouring pairs of one head, so that both elements of
// a pair are read before either is written and dst may be src.
#include "launch.h"
#include "rotary.h"

namespace mx {

constexpr int ROPE_THREADS = 256;

struct RopeArgs {
  int64_t tokens, src_token, src_head, dst_token, dst_head;  // strides in elements
  const int64_t *positions;
  const double *inv_freq;
  double scale;
  int heads, dim, half, per_wg, inverse, copy;  // half: pairs; copy: the rest is copied too (dst is not src)
};

template <typename T, int N> struct Piece {
  T v[N];
} __attribute__((aligned(sizeof(T) * N)));

__device__ __forceinline__ float to_f32(unsigned short b) { return __uint_as_float((unsigned)b << 16); }
__device__ __forceinline__ float to_f32(float f) { return f; }
__device__ __forceinline__ void from_f32(unsigned short &d, float f) { d = (unsigned short)bf16x2_rne(f, 0.0f); }
__device__ __forceinline__ void from_f32(float &d, float f) { d = f; }

constexpr int ROPE_ROWS = 2;  // rows whose loads a thread has under way together, the first ones before the angles

// src and dst may be one tensor (no __restrict__): a thread reads all of a piece's pairs before it writes them.
template <typename T, int VEC, int LAYOUT>
__global__ __launch_bounds__(ROPE_THREADS) void k_rope(const T *src, T *dst, RopeArgs a) {
  __shared__ float tc[ROPE_TABLE], ts[ROPE_TABLE];
  // items of a head: pieces of VEC pairs (HALF and single pairs) or of VEC elements, then the pieces that are copied
  constexpr bool PAIRS = LAYOUT == ROTARY_HALF || VEC == 1;
  constexpr int V = VEC;
  const int turned = PAIRS ? a.half / V : (2 * a.half + V - 1) / V;
  const int rest0 = PAIRS ? 2 * a.half : turned * V;  // first element that is copied
  const int items = turned + (a.copy ? (a.dim - rest0) / V : 0);
  const int64_t t0 = (int64_t)blockIdx.x * a.per_wg;
  const int nt = (int)(a.tokens - t0 < a.per_wg ? a.tokens - t0 : a.per_wg);
  const int total = nt * a.heads;
  // a thread keeps its place in the head while the heads fit a pass of the workgroup
  const int step = items < ROPE_THREADS ? ROPE_THREADS / items : 1;
  const int first = items < ROPE_THREADS ? threadIdx.x / items : 0;
  const int item0 = threadIdx.x - first * items;
  const bool active = first < step && item0 < items;  // not so: threads past the last whole head

  Piece<T, V> u[ROPE_ROWS], w[ROPE_ROWS];
  auto offsets = [&](int item, int &da, int &db) {  // of the piece, and of the pairs' second elements
    const int p = item * V;
    da = item >= turned ? rest0 + (item - turned) * V : !PAIRS || LAYOUT == ROTARY_HALF ? p : 2 * p;
    db = LAYOUT == ROTARY_HALF ? p + a.half : 2 * p + 1;
  };
  auto load = [&](int item, int base) {
    int da, db;
    offsets(item, da, db);
#pragma unroll
    for (int k = 0; k < ROPE_ROWS; ++k) {
      const int row = base + k * step;
      if (row >= total) break;
      const int t = row / a.heads, h = row - t * a.heads;
      const T *x = src + (t0 + t) * a.src_token + h * a.src_head;
      u[k] = *(const Piece<T, V> *)(x + da);
      if (PAIRS && item < turned) w[k] = *(const Piece<T, V> *)(x + db);
    }
  };
  auto finish = [&](int item, int base) {
    int da, db;
    offsets(item, da, db);
#pragma unroll
    for (int k = 0; k < ROPE_ROWS; ++k) {
      const int row = base + k * step;
      if (row >= total) break;
      const int t = row / a.heads, h = row - t * a.heads;
      T *y = dst + (t0 + t) * a.dst_token + h * a.dst_head;
      if (item < turned) {
        const float *c = tc + t * a.half, *s = ts + t * a.half;
        if (PAIRS) {
          const int p = item * V;
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float f = to_f32(u[k].v[e]), g = to_f32(w[k].v[e]);
            from_f32(u[k].v[e], f * c[p + e] - g * s[p + e]);
            from_f32(w[k].v[e], g * c[p + e] + f * s[p + e]);
          }
          *(Piece<T, V> *)(y + db) = w[k];
        } else {
          const int p = da / 2;
#pragma unroll
          for (int e = 0; e < V / 2; ++e) {
            if (p + e < a.half) {  // the last piece may hold elements that are not rotated
              const float f = to_f32(u[k].v[2 * e]), g = to_f32(u[k].v[2 * e + 1]);
              from_f32(u[k].v[2 * e], f * c[p + e] - g * s[p + e]);
              from_f32(u[k].v[2 * e + 1], g * c[p + e] + f * s[p + e]);
            }
          }
        }
      }
      *(Piece<T, V> *)(y + da) = u[k];
    }
  };

  if (active) load(item0, first);
  for (int i = threadIdx.x; i < nt * a.half; i += ROPE_THREADS) {
    const int t = i / a.half, p = i - t * a.half;
    double s, c;
    sine_cosine((double)a.positions[t0 + t] * a.inv_freq[p], s, c);
    tc[i] = (float)(c * a.scale);
    ts[i] = (float)(a.inverse ? -s * a.scale : s * a.scale);
  }
  __syncthreads();
  if (!active) return;
  for (int item = item0; item < items; item += ROPE_THREADS)
    for (int base = first; base < total; base += ROPE_ROWS * step) {
      if (item != item0 || base != first) load(item, base);
      finish(item, base);
    }
}

// Half layout whose halves are not whole pieces: a thread has a piece of the row as it lies in memory, and takes the
// partners of its elements out of LDS, where the workgroup has put the rows' pieces.  (62 of 128 dimensions of 8192 x
// 64 heads in bf16: 66-69 us; 140 in pieces of single pairs; 43 with whole pieces.)  Every row is in LDS before any of
// it is written, so dst may be src.
template <typename T, int VEC>
__global__ __launch_bounds__(ROPE_THREADS) void k_rope_staged(const T *src, T *dst, RopeArgs a) {
  __shared__ float tc[ROPE_TABLE], ts[ROPE_TABLE];
  __shared__ Piece<T, VEC> rows[2][ROPE_THREADS];
  const int64_t t0 = (int64_t)blockIdx.x * a.per_wg;
  const int nt = (int)(a.tokens - t0 < a.per_wg ? a.tokens - t0 : a.per_wg);
  for (int i = threadIdx.x; i < nt * a.half; i += ROPE_THREADS) {
    const int t = i / a.half, p = i - t * a.half;
    double s, c;
    sine_cosine((double)a.positions[t0 + t] * a.inv_freq[p], s, c);
    tc[i] = (float)(c * a.scale);
    ts[i] = (float)(a.inverse ? -s * a.scale : s * a.scale);
  }
  const int items = a.dim / VEC, step = ROPE_THREADS / items;
  const int first = threadIdx.x / items, d = (threadIdx.x - first * items) * VEC, total = nt * a.heads;
  float c[VEC], s[VEC];
  int with = -1;  // the token whose angles these are
  for (int base = 0, turn = 0; base < total; base += step, turn ^= 1) {
    const int row = base + first;
    const bool in = first < step && row < total;
    const int t = in ? row / a.heads : 0, h = row - t * a.heads;
    Piece<T, VEC> u;
    if (in) rows[turn][threadIdx.x] = u = *(const Piece<T, VEC> *)(src + (t0 + t) * a.src_token + h * a.src_head + d);
    __syncthreads();  // (the other turn's rows are read until the barrier after this one)
    if (!in) continue;
    if (t != with) {
      with = t;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int p = d + e < a.half ? d + e : d + e - a.half;
        const bool turned = d + e < 2 * a.half;
        c[e] = turned ? tc[t * a.half + p] : 1.0f;
        s[e] = turned ? (d + e < a.half ? -ts[t * a.half + p] : ts[t * a.half + p]) : 0.0f;
      }
    }
    const T *mine = (const T *)&rows[turn][first * items];
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (d + e < 2 * a.half) {
        const float f = to_f32(u.v[e]), g = to_f32(mine[d + e < a.half ? d + e + a.half : d + e - a.half]);
        from_f32(u.v[e], f * c[e] + g * s[e]);
      }
    *(Piece<T, VEC> *)(dst + (t0 + t) * a.dst_token + h * a.dst_head + d) = u;
  }
}

template <typename T, int VEC, int LAYOUT>
static void rope_start(const void *src, void *dst, const RopeArgs &a, hipStream_t stream) {
  const unsigned grid = (unsigned)((a.tokens + a.per_wg - 1) / a.per_wg);
  k_rope<T, VEC, LAYOUT><<<grid, ROPE_THREADS, 0, stream>>>((const T *)src, (T *)dst, a);
}

template <typename T, int VEC>
static void rope_staged(const void *src, void *dst, const RopeArgs &a, hipStream_t stream) {
  const unsigned grid = (unsigned)((a.tokens + a.per_wg - 1) / a.per_wg);
  k_rope_staged<T, VEC><<<grid, ROPE_THREADS, 0, stream>>>((const T *)src, (T *)dst, a);
}

template <typename T, int LAYOUT>
static void rope_vec(int vec, const void *src, void *dst, const RopeArgs &a, hipStream_t stream) {
  switch (vec) {
    case 8:
      if constexpr (sizeof(T) == 2) return rope_start<T, 8, LAYOUT>(src, dst, a, stream);
    case 4: return rope_start<T, 4, LAYOUT>(src, dst, a, stream);
    case 2: return rope_start<T, 2, LAYOUT>(src, dst, a, stream);
    default: return rope_start<T, 1, LAYOUT>(src, dst, a, stream);
  }
}

hipError_t launch_rope(int dtype, const void *src, void *dst, int64_t tokens, int64_t heads, int64_t dim,
                       const int64_t strides[4], const int64_t *positions, const double *inv_freq, int64_t rot,
                       int layout, double scale, int inverse, hipStream_t stream) {
  const int size = dtype == 1 ? 4 : 2;
  RopeArgs a{tokens, strides[0], strides[1], strides[2], strides[3], positions, inv_freq, scale,
             (int)heads, (int)dim, (int)(rot / 2), 1, inverse, src != dst};
  // the widest piece, up to 16 bytes, at which every access is aligned and no head is cut; in the half layout the
  // halves should not be cut either
  int wide = 16 / size;
  for (; wide > 1; wide /= 2) {
    bool ok = dim % wide == 0 && (uintptr_t)src % (wide * size) == 0 && (uintptr_t)dst % (wide * size) == 0;
    for (int i = 0; i < 4; ++i) ok = ok && strides[i] % wide == 0;
    if (ok) break;
  }
  int vec = wide;
  while (layout == ROTARY_HALF && a.half % vec != 0) vec /= 2;
  const bool staged = vec < wide && wide >= 4 && dim / wide <= ROPE_THREADS;
  // tokens of a workgroup: about four 16-byte pieces for each of its threads, as long as the table holds them and
  // there are four workgroups for every CU
  const int64_t row = heads * dim * size;
  int64_t per = 4 * 16 * ROPE_THREADS / row;
  if (a.half && per > ROPE_TABLE / a.half) per = ROPE_TABLE / a.half;  // 16 KiB of LDS
  const int64_t spread = tokens / (4 * device_cu_count());
  if (per > spread) per = spread;
  const int64_t least = (tokens + MAX_GROUPS_256 - 1) / MAX_GROUPS_256;  // the table holds it: checked by the caller
  if (per < least) per = least;
  a.per_wg = per < 1 ? 1 : (int)per;
  if (staged) {
    if (dtype == 1) rope_staged<float, 4>(src, dst, a, stream);
    else if (wide == 8) rope_staged<unsigned short, 8>(src, dst, a, stream);
    else rope_staged<unsigned short, 4>(src, dst, a, stream);
  } else if (dtype == 1) {
    if (layout == ROTARY_HALF) rope_vec<float, ROTARY_HALF>(vec, src, dst, a, stream);
    else rope_vec<float, ROTARY_INTERLEAVED>(vec, src, dst, a, stream);
  } else {
    if (layout == ROTARY_HALF) rope_vec<unsigned short, ROTARY_HALF>(vec, src, dst, a, stream);
    else rope_vec<unsigned short, ROTARY_INTERLEAVED>(vec, src, dst, a, stream);
  }
  return hipGetLastError();
}

}  // namespace mx
