// Attention over the paged MX cache for many rows of a key/value head: trees
// of drafted tokens and chunks of a prompt.
//
// Bound: the matrix cores (4 D flops a pair of row and token, on bf16) and, as
// much, the vector units (an exponential a pair, which takes four issues).  So
// keys and values are converted once for a workgroup's 128 or 256 rows: tiles
// of 64 tokens are widened to bf16 on their way into LDS, two tiles in turn,
// while the codes of the tile after them are on their way from memory.
//
// S^T = K Q^T and O^T = V^T P^T on v_mfma_f32_32x32x16_bf16: lane l holds for
// row or column l % 32 of an operand the 8 elements k = 8 (l / 32) .., and of
// the result column l % 32, rows 8 (r / 4) + 4 (l / 32) + r % 4 in register r.
// A lane's scores are therefore of one row, and eight registers of them are,
// as they lie, the operand of the second product for 16 tokens if its k goes
// over the tokens in the same order; V^T comes in that order out of LDS by
// transposing reads of four tokens by 16 dimensions.  Row statistics need one
// exchange between the wave's halves.
//
// A wave takes 32 RB rows.  With RB = 2 an operand read from LDS serves two
// products, which halves the LDS traffic (64 bytes a clock of its 128 at full
// rate of the matrix cores).
//
// LDS rows are padded so that the reads are free of bank conflicts: K rows by
// 16 bytes (16 lanes' 16-byte reads of one column are then 4 banks apart),
// V rows to 16 or 48 banks past a multiple of 64 (four tokens' 64 bytes are
// then apart).
#include "attention.h"

namespace mx {

typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
typedef __attribute__((address_space(3))) uint8_t lds_u8;

template <int FMT, int D, int RB, int WAVES> struct Tiled {
  static constexpr int THREADS = 64 * WAVES;
  static constexpr int ROWS = 32 * RB * WAVES;
  static constexpr int CODE = FMT == 0 ? 8 : 16;                       // bytes of 16 dimensions
  static constexpr int ROW = D / 16;                                   // such units of a row
  static constexpr int ALL = 2 * TILE * ROW;                           // of a tile: keys, then values
  static constexpr int UNITS = (ALL + THREADS - 1) / THREADS;          // of a thread
  static constexpr int KS = 2 * D + 16;                                // bytes of an LDS row
  static constexpr int VS = 2 * D + (D == 96 ? 0 : 64);
  static constexpr int BUFFER = TILE * (KS + VS);
  static constexpr int LDS = 2 * BUFFER + 16;
};

__device__ __forceinline__ f32x16 mma32(u32x4 a, u32x4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                 0);
}

// Eight tokens of a dimension: two transposing reads, `far` bytes apart.
__device__ __forceinline__ u32x4 read_v(const lds_u8 *p, int far) {
  const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)p));
  const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)(p + far)));
  return u32x4{a.x, a.y, b.x, b.y};
}

template <int FMT, int D, int RB, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_attention_tiles(AttentionArgs a, Division dv) {
  using T = Tiled<FMT, D, RB, WAVES>;
  extern __shared__ __align__(16) uint8_t lds[];
  const CacheView &cv = a.cache;
  const int wave = uniform(threadIdx.x / 64), lane = threadIdx.x % 64, n32 = lane % 32, h = lane / 32;
  const int page_mask = (1 << cv.page_log2) - 1;
  volatile int *flags = (volatile int *)(lds + 2 * T::BUFFER);  // [0]: a page outside the cache, [1]: values that are not finite in a masked tile
  const float to_log2 = a.scale * 1.4426950408889634f;

  for (Pieces pc(a, dv); pc.next(a, dv);) {
    const Sequence sq = pc.s;
    const int b = pc.b, head = pc.head, rb = pc.block, t0 = pc.t0, t1 = pc.t1, tiles = pc.tiles, slot = pc.slot;
    const int q0 = sq.q0, len = sq.len, rows = sq.nq * a.group;
    const int first_new = len - sq.nq;                           // may be negative
    const int seen_by_all = a.tree ? first_new : first_new + 1;  // tokens before this need no mask
    const int tail0 = (seen_by_all < 0 ? 0 : seen_by_all) / TILE;  // the first tile that needs a mask
    const int *table = a.table + (int64_t)b * a.table_stride;
    const int row0 = rb * T::ROWS + wave * 32 * RB;

    u32x4 q[RB][D / 16];
    int node[RB];
#pragma unroll
    for (int n = 0; n < RB; ++n) {
      const int row = row0 + 32 * n + n32;
      const bool in = row < rows;
      node[n] = in ? row / a.group : 0;
      const unsigned short *x = a.q + (int64_t)(q0 + node[n]) * a.q_token +
                                (int64_t)(head * a.group + (in ? row - node[n] * a.group : 0)) * a.q_head + 8 * h;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) q[n][i] = in ? *(const u32x4 *)(x + 16 * i) : u32x4{0u, 0u, 0u, 0u};
    }

    f32x16 o[RB][D / 32];
    float m[RB], l[RB];
#pragma unroll
    for (int n = 0; n < RB; ++n) {
      m[n] = -__builtin_inff();
      l[n] = 0.0f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[n][i][r] = 0.0f;
    }

    // codes on their way: the thread's units of a tile
    unsigned code[T::UNITS][T::CODE / 4], scale[T::UNITS];
    int page[T::UNITS];
    auto unit_row = [&](int u, int &row, int &col) {  // which of keys (rows 0 ..) and values (TILE ..), 16 dimensions
      const int i = threadIdx.x + u * T::THREADS;
      row = i / T::ROW;
      col = i - row * T::ROW;
      return T::ALL % T::THREADS == 0 || i < T::ALL;
    };
    auto token_of = [&](int t, int row) {  // past the end: the last one again
      const int tok = t * TILE + row % TILE;
      return tok < len ? tok : len - 1;
    };
    auto look_up = [&](int t) {
#pragma unroll
      for (int u = 0; u < T::UNITS; ++u) {
        int row, col;
        if (!unit_row(u, row, col)) break;
        page[u] = table[token_of(t, row) >> cv.page_log2];
      }
    };
    auto fetch = [&](int t) {
#pragma unroll
      for (int u = 0; u < T::UNITS; ++u) {
        int row, col;
        if (!unit_row(u, row, col)) break;
        const int r = token_of(t, row) & page_mask;
        const bool ok = (unsigned)page[u] < (uint64_t)cv.pages;
        const int64_t ph = (int64_t)(ok ? page[u] : 0) * cv.heads + head;
        const bool value = row >= TILE;
        const uint8_t *c = value ? cv.codes[1] : cv.codes[0], *s = value ? cv.scales[1] : cv.scales[0];
        load_bytes<T::CODE>(code[u], c + (((ph << cv.page_log2) + r) * T::ROW + col) * T::CODE);
        scale[u] = s[((ph * (D / 32) + col / 2) << cv.page_log2) + r];
        if (!ok) scale[u] |= 0x100u;
      }
    };
    auto store = [&](int t) {
      uint8_t *buf = lds + (t & 1) * T::BUFFER;
      const bool tail = t >= tail0;
      bool outside_any = false;
      unsigned odd_any = 0u;
#pragma unroll
      for (int u = 0; u < T::UNITS; ++u) {
        int row, col;
        if (!unit_row(u, row, col)) break;
        const bool value = row >= TILE, outside = scale[u] > 0xFFu;
        unsigned w[8];
        widen<FMT, 16>(w, code[u], scale[u] & 0xFFu);
        outside_any |= outside;
        if (tail) {
          const unsigned keep = value && (outside || t * TILE + row - TILE >= len) ? 0u : 0xFFFFFFFFu;
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] &= keep;
          if (value) odd_any |= clear_not_finite<8>(w);
        } else if (outside) {
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = 0u;
        }
        u32x4 *d = (u32x4 *)(buf + (value ? TILE * T::KS + (row - TILE) * T::VS : row * T::KS) + 32 * col);
        d[0] = u32x4{w[0], w[1], w[2], w[3]};
        d[1] = u32x4{w[4], w[5], w[6], w[7]};
      }
      if (outside_any) flags[0] = 1;
      if (odd_any) flags[1] = 1;
    };

    if (threadIdx.x < 2) flags[threadIdx.x] = 0;
    __syncthreads();
    if (len > 0) {
      look_up(t0);
      fetch(t0);
      look_up(t0 + 1);
      store(t0);
      fetch(t0 + 1);
      look_up(t0 + 2);
    }
    __syncthreads();
    for (int t = t0; t < t1 && len > 0; ++t) {
      const lds_u8 *kb = (const lds_u8 *)(lds + (t & 1) * T::BUFFER + n32 * T::KS + 16 * h);
      const lds_u8 *vb = (const lds_u8 *)(lds + (t & 1) * T::BUFFER + TILE * T::KS + (4 * h + lane % 16 / 4) * T::VS +
                                          32 * (lane / 16 % 2) + 8 * (lane % 4));
      f32x16 s[RB][2];
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const u32x4 k = *(const __attribute__((address_space(3))) u32x4 *)(kb + u * 32 * T::KS + 32 * i);
#pragma unroll
          for (int n = 0; n < RB; ++n) s[n][u] = mma32(k, q[n][i], i == 0 ? f32x16{} : s[n][u]);
          if (u == 1 && i % 2 == 1) __builtin_amdgcn_sched_barrier(0);
        }

      const bool masked = t >= tail0 || flags[0];
      unsigned vis[RB][2];
      if (masked) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int tok = t * TILE + 32 * u;
          unsigned in = first_bits<32>(len - tok);
          if (flags[0]) {
            // pages hold 16 tokens at least
            if (tok < len && (unsigned)table[tok >> cv.page_log2] >= (uint64_t)cv.pages) in &= 0xFFFF0000u;
            if (tok + 16 < len && (unsigned)table[(tok + 16) >> cv.page_log2] >= (uint64_t)cv.pages) in &= 0xFFFFu;
          }
#pragma unroll
          for (int n = 0; n < RB; ++n) {
            vis[n][u] = (seen_bits<32>(a, q0 + node[n], node[n], tok - first_new) & in) >> (4 * h);
#pragma unroll
            for (int r = 0; r < 16; ++r)
              s[n][u][r] = (vis[n][u] >> (8 * (r / 4) + r % 4)) & 1u ? s[n][u][r] : -__builtin_inff();
          }
        }
      }

      // weights: registers 8 s .. of a half are the operand for its tokens 16 s ..
      u32x4 p[RB][4];
#pragma unroll
      for (int n = 0; n < RB; ++n) {
        float top = s[n][0][0];
#pragma unroll
        for (int k = 1; k < 32; ++k) top = fmaxf(top, s[n][k / 16][k % 16]);
        top = max_halves(top * to_log2);
        if (__builtin_amdgcn_ballot_w64(top > m[n] + LAG)) {
          const float big = fmaxf(m[n], top);
          const float f = big == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(m[n] - big);
          m[n] = big;
          l[n] *= f;
#pragma unroll
          for (int i = 0; i < D / 32; ++i) o[n][i] *= f;
        }
        const float base = m[n] == -__builtin_inff() ? 0.0f : m[n];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const float w0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][k / 8][2 * k % 16], to_log2, -base));
          const float w1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][k / 8][2 * k % 16 + 1], to_log2, -base));
          p[n][k / 4][k % 4] = bf16x2_rne(w0, w1);
          l[n] = add_pair(p[n][k / 4][k % 4], l[n]);
        }
      }

#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            const u32x4 v = read_v(vb + 16 * k * T::VS + 64 * i, 8 * T::VS);
#pragma unroll
            for (int n = 0; n < RB; ++n) o[n][i] = mma32(v, p[n][k], o[n][i]);
            if (i % 2 == 1) __builtin_amdgcn_sched_barrier(0);
          }

      if (t + 1 < t1) {
        store(t + 1);
        fetch(t + 2);
        look_up(t + 3);
      }
      __syncthreads();
    }

#pragma unroll
    for (int n = 0; n < RB; ++n) {
      const int row = row0 + 32 * n + n32;
      l[n] = sum_halves(l[n]);
      if (row >= rows) continue;
      if (flags[1]) {
        const int from = tail0 * TILE > t0 * TILE ? tail0 * TILE : t0 * TILE;
        const int to = t1 * TILE < len ? t1 * TILE : len;
        seen_tokens(a, table, head, q0 + node[n], node[n], first_new, from, to, [&](int64_t ph, int r) {
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            const unsigned sb = cv.scales[1][((ph * (D / 32) + i) << cv.page_log2) + r];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              unsigned code, w[2];
              load_bytes<T::CODE / 4>(&code, cv.codes[1] + (((ph << cv.page_log2) + r) * T::ROW * T::CODE) +
                                                 (32 * i + 8 * c + 4 * h) * T::CODE / 16);
              widen<FMT, 4>(w, &code, sb);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if ((not_finite(w[e / 2]) >> (16 * (e & 1))) & 1u) o[n][i][4 * c + e] = __uint_as_float(F32_NAN);
            }
          }
        });
      }
      if (t1 - t0 == tiles) {
        const int64_t at = (int64_t)(q0 + node[n]) * cv.heads * a.group + head * a.group + (row - node[n] * a.group);
        const float inv = reciprocal(l[n]);
        unsigned short *d = a.out + at * D + 4 * h;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            *(u32x2 *)(d + 32 * i + 8 * r) = u32x2{bf16x2_rne(o[n][i][4 * r] * inv, o[n][i][4 * r + 1] * inv),
                                                   bf16x2_rne(o[n][i][4 * r + 2] * inv, o[n][i][4 * r + 3] * inv)};
      } else {
        const int64_t part = 2 * (int64_t)blockIdx.x + slot;
        const int r0 = wave * 32 * RB + 32 * n + n32;  // of the block
        float *d = part_sums(a, dv, part, D) + (int64_t)r0 * D + 4 * h;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            *(f32x4 *)(d + 32 * i + 8 * r) =
                f32x4{o[n][i][4 * r], o[n][i][4 * r + 1], o[n][i][4 * r + 2], o[n][i][4 * r + 3]};
        if (h == 0) {
          float *ml = part_stats(a, dv, part, D) + 2 * r0;
          ml[0] = m[n];
          ml[1] = l[n];
        }
      }
    }
  }
}

template <int FMT, int D, int RB, int WAVES>
static hipError_t start(const AttentionArgs &a, const Division &d, hipStream_t stream) {
  using T = Tiled<FMT, D, RB, WAVES>;
  const int64_t grid = d.workers ? d.workers : (int64_t)a.batch * a.cache.heads * d.blocks;
  const hipError_t e = hipFuncSetAttribute((const void *)k_attention_tiles<FMT, D, RB, WAVES>,
                                           hipFuncAttributeMaxDynamicSharedMemorySize, T::LDS);
  if (e != hipSuccess) return e;
  k_attention_tiles<FMT, D, RB, WAVES><<<(unsigned)grid, T::THREADS, T::LDS, stream>>>(a, d);
  return hipGetLastError();
}

template <int FMT, int D>
static hipError_t by_rows(const AttentionArgs &a, const Division &d, hipStream_t stream) {
  if (d.rows == 128) return start<FMT, D, 1, 4>(a, d, stream);
  return start<FMT, D, 1, 8>(a, d, stream);
}

hipError_t launch_attention_tiles(const AttentionArgs &a, const Division &d, hipStream_t stream) {
#define MX_DIM(D) case D: return a.cache.fmt == 0 ? by_rows<0, D>(a, d, stream) : by_rows<1, D>(a, d, stream)
  switch (a.cache.dim) {
    MX_DIM(64);
    MX_DIM(96);
    MX_DIM(128);
    MX_DIM(192);
    MX_DIM(256);
    default: return hipErrorInvalidValue;
  }
#undef MX_DIM
}

}  // namespace mx
