// Attention over the paged MX cache for many rows of a key/value head: trees
// of drafted tokens and chunks of a prompt.
//
// Bound: the matrix cores (4 D flops a pair of row and token, on bf16) and, as
// much, the vector units (an exponential a pair, which takes four issues).  So
// keys and values are converted once for a workgroup's 128 or 256 rows: tiles
// of 64 tokens are widened to bf16 on their way into LDS, two tiles in turn,
// while the codes of the tile after them are on their way from memory.  The
// conversion of a tile is issued between the products of the scores before it,
// the weights of 16 tokens between the products of the 16 before them.
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
// A wave takes 32 rows: heads of up to 128 dimensions then fit the 256
// registers of two waves a SIMD, larger ones have one wave and keep the sums
// in accumulation registers.  (64 rows a wave halve the LDS reads, and measured
// the same or slower: 4 waves of 64 rows 125 us where 8 of 32 took 108.)
//
// LDS rows are padded so that the reads are free of bank conflicts: K rows by
// 16 bytes (16 lanes' 16-byte reads of one column are then 4 banks apart),
// V rows to 16 or 48 banks past a multiple of 64 (four tokens' 64 bytes are
// then apart).
//
// Measured on MI355X: 8 sequences x 64 heads over 8 of 128 (MXFP8), 64 new
// tokens over 32768: 625-640 us, 0.86-0.88 PFLOP/s (a library product of 16384^3
// in bf16 1.37), its clock falling to 1.85 GHz from 2.2; with 8192 tokens 0.74,
// heads of 256 0.71.  2 us a tile of 64 tokens by 256 rows; a piece costs some 15 us
// beside its tiles (plan, first loads, writing and joining the sums).
#include "attention.h"

namespace mx {

typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef __attribute__((address_space(3))) int lds_int;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;

template <int FMT, int D, int WAVES> struct Tiled {
  static constexpr int THREADS = 64 * WAVES;
  static constexpr int ROWS = 32 * WAVES;
  static constexpr int CODE = FMT == 0 ? 8 : 16;                       // bytes of 16 dimensions
  static constexpr int ROW = D / 16;                                   // such units of a row
  static constexpr int SHARE = THREADS / TILE;                         // threads of a token
  static constexpr int UNITS = (ROW + SHARE - 1) / SHARE;              // units of a thread, of the key and of the value
  static constexpr int KS = 2 * D + 16;                                // bytes of an LDS row
  static constexpr int VS = 2 * D + (D == 96 ? 0 : 64);
  static constexpr int BUFFER = TILE * (KS + VS);
  static constexpr int LDS = 2 * BUFFER + 16;
};

__device__ __forceinline__ f32x16 mma32(u32x4 a, u32x4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                 0);
}

// Kinds of instructions for the order that the compiler is asked for.
constexpr int SCHED_VALU = 0x2, SCHED_MFMA = 0x8, SCHED_LDS_READ = 0x100;
template <int KIND, int N> __device__ __forceinline__ void order() { __builtin_amdgcn_sched_group_barrier(KIND, N, 0); }

// Keeps what is computed of a loaded value behind this point: where a loop loads it for its next turn, the compiler
// would compute it, and wait for it, at once.
template <typename T> __device__ __forceinline__ void held(T &v) { asm volatile("" : "+v"(v)); }

// Eight tokens of a dimension: two transposing reads, `far` bytes apart.
__device__ __forceinline__ u32x4 read_v(const lds_u8 *p, int far) {
  const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)p));
  const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)(p + far)));
  return u32x4{a.x, a.y, b.x, b.y};
}

template <int FMT, int D, int WAVES>
__global__ __launch_bounds__(64 * WAVES, D <= 128 ? 2 : 1) void k_attention_tiles(AttentionArgs a, Division dv) {
  using T = Tiled<FMT, D, WAVES>;
  extern __shared__ __align__(16) uint8_t lds[];
  const CacheView &cv = a.cache;
  const int wave = uniform((int)threadIdx.x / 64), lane = threadIdx.x % 64, n32 = lane % 32, h = lane / 32;
  const int page_mask = (1 << cv.page_log2) - 1;
  // [0]: a page outside the cache was met, [1]: values that are not finite in a tile that needs a mask
  lds_int *flags = (lds_int *)(lds + 2 * T::BUFFER);
  constexpr bool ACC = D > 128 && WAVES == 4;  // one wave a SIMD: the sums are in accumulation registers
  constexpr int VG = D % 128 == 0 ? 4 : D % 96 == 0 ? 3 : 2;  // V operands of a group
  constexpr int PARTS = D / 32 / VG;                           // groups for 16 tokens
  const float to_log2 = a.scale * LOG2_E;

  Pieces pc(a, dv);
  while (pc.next(a, dv)) {
    const int nq = uniform(pc.s.nq), len = uniform(pc.s.len), q0 = uniform(pc.s.q0), b = uniform(pc.b);
    const int head = uniform(pc.head), rb = uniform(pc.block);
    const int t0 = uniform(pc.t0), t1 = uniform(pc.t1), tiles = uniform(pc.tiles), slot = uniform(pc.slot);
    const int rows = nq * a.group;
    const int first_new = uniform(pc.s.first_new);
    const int seen_by_all = a.tree ? first_new : first_new + 1;  // tokens before this need no mask
    // the first tile that needs a mask, or ends behind the tokens
    const int tail0 = (seen_by_all < 0 ? 0 : seen_by_all < len ? seen_by_all : len) / TILE;
    const int *table = a.table + (int64_t)b * a.table_stride;

    const int row = rb * T::ROWS + wave * 32 + n32;
    const bool in = row < rows;
    const int node = in ? row / a.group : 0;
    u32x4 q[D / 16];
    {
      const unsigned short *x = a.q + (int64_t)(q0 + node) * a.q_token +
                                (int64_t)(head * a.group + (in ? row - node * a.group : 0)) * a.q_head + 8 * h;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) q[i] = in ? *(const u32x4 *)(x + 16 * i) : u32x4{0u, 0u, 0u, 0u};
    }

    f32x16 o[D / 32];
    float m = -__builtin_inff(), l = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] = f32x16{};

    // codes on their way: a thread has one token of a tile, and of its key and its value (index 0 and 1 below) every
    // SHARE-th unit of 16 dimensions
    const int my_row = threadIdx.x / T::SHARE, my_col = threadIdx.x % T::SHARE;
    unsigned code[2][T::UNITS][T::CODE / 4], scale[2][T::UNITS];
    int page = 0;
    bool outside = false;  // the page is not in the cache
    auto has = [&](int u) { return T::ROW % T::SHARE == 0 || my_col + u * T::SHARE < T::ROW; };
    auto token_of = [&](int t) {  // past the end: the last one again
      const int tok = t * TILE + my_row;
      return tok < len ? tok : len - 1;
    };
    auto look_up = [&](int t) { page = table[token_of(t) >> cv.page_log2]; };
    auto fetch = [&](int t) {
      held(page);
      outside = (unsigned)page >= (uint64_t)cv.pages;
      const int r = token_of(t) & page_mask;
      const int64_t ph = (int64_t)(outside ? 0 : page) * cv.heads + head;
      const int64_t c0 = ((ph << cv.page_log2) + r) * (T::ROW * T::CODE) + my_col * T::CODE;
      const int64_t s0 = ((ph * (D / 32)) << cv.page_log2) + (r & ~3);
#pragma unroll
      for (int v = 0; v < 2; ++v)
#pragma unroll
        for (int u = 0; u < T::UNITS; ++u) {
          if (!has(u)) break;
          load_bytes<T::CODE>(code[v][u], cv.codes[v] + c0 + u * (T::SHARE * T::CODE));
          // four tokens' bytes: a byte would be masked, and so waited for, where it is loaded
          scale[v][u] = *(const unsigned *)(cv.scales[v] + s0 + ((my_col + u * T::SHARE) / 2 << cv.page_log2));
        }
    };
    auto place = [&](int t, int v, int u) {
      return (u32x4 *)(lds + (t & 1) * T::BUFFER + (v ? TILE * T::KS + my_row * T::VS : my_row * T::KS) + 32 * my_col +
                       32 * T::SHARE * u);
    };
    auto scale_of = [&](int t, int v, int u) { return scale[v][u] >> (8 * (token_of(t) & 3)) & 0xFFu; };
    auto store = [&](int t, int v, int u) {
      if (!has(u)) return;
      held(scale[v][u]);
      unsigned w[8];
      widen<FMT, 16>(w, code[v][u], scale_of(t, v, u));
      u32x4 *d = place(t, v, u);
      d[0] = u32x4{w[0], w[1], w[2], w[3]};
      d[1] = u32x4{w[4], w[5], w[6], w[7]};
    };
    // The values of a tile that needs a mask, or has pages outside the cache, once more: tokens that are not there
    // become zero, and so does what is not finite.
    auto clean = [&](int t) {
      unsigned odd = 0u;
#pragma unroll
      for (int u = 0; u < T::UNITS; ++u) {
        if (!has(u)) break;
        unsigned w[8];
        widen<FMT, 16>(w, code[1][u], scale_of(t, 1, u));
        const unsigned keep = outside || t * TILE + my_row >= len ? 0u : 0xFFFFFFFFu;
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] &= keep;
        if (t >= tail0) odd |= clear_not_finite<8>(w);
        u32x4 *d = place(t, 1, u);
        d[0] = u32x4{w[0], w[1], w[2], w[3]};
        d[1] = u32x4{w[4], w[5], w[6], w[7]};
      }
      if (outside) flags[0] = 1;
      if (odd) flags[1] = 1;
    };
    auto needs_clean = [&](int t) { return t >= tail0 || __builtin_amdgcn_ballot_w64(outside) != 0; };

    __syncthreads();  // the flags of the piece before have been read
    if (threadIdx.x < 2) flags[threadIdx.x] = 0;
    __syncthreads();
    if (len > 0) {
      look_up(t0);
      fetch(t0);
      look_up(t0 + 1);
#pragma unroll
      for (int u = 0; u < T::UNITS; ++u) store(t0, 0, u), store(t0, 1, u);
      if (needs_clean(t0)) clean(t0);
      fetch(t0 + 1);
      look_up(t0 + 2);
    }
    __builtin_amdgcn_s_waitcnt(0);  // the queries' loads too: none is left for the loop to wait for
    __syncthreads();
    for (int t = t0; t < t1 && len > 0; ++t) {
      const lds_u8 *kb = (const lds_u8 *)(lds + (t & 1) * T::BUFFER + n32 * T::KS + 16 * h);
      const lds_u8 *vb = (const lds_u8 *)(lds + (t & 1) * T::BUFFER + TILE * T::KS + (4 * h + lane % 16 / 4) * T::VS +
                                          32 * (lane / 16 % 2) + 8 * (lane % 4));
      const int outside_seen = flags[0];
      // operands are read one group ahead of the products that take them
      u32x4 kf[2][4], vf[2][VG];
      auto read_k = [&](int g) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          kf[g & 1][i] = *(const lds_u32x4 *)(kb + (i & 1) * 32 * T::KS + 64 * g + 32 * (i / 2));
      };
      auto read_values = [&](int g) {
#pragma unroll
        for (int i = 0; i < VG; ++i) {
          const int k = (g * VG + i) / (D / 32), d = (g * VG + i) % (D / 32);
          vf[g & 1][i] = read_v(vb + 16 * k * T::VS + 64 * d, 8 * T::VS);
        }
      };
      f32x16 s[2];
      read_k(0);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int g = 0; g < D / 32; ++g) {
        if (g + 1 < D / 32) read_k(g + 1);
        else read_values(0);
        // the next tile's conversion under the products
        if (g < 2 * T::UNITS) store(t + 1, g % 2, g / 2);
        if (g == D / 32 - 1)
#pragma unroll
          for (int k = D / 32; k < 2 * T::UNITS; ++k) store(t + 1, k % 2, k / 2);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            s[i & 1] = mma32(kf[g & 1][i], q[2 * g + i / 2], g == 0 && i < 2 ? f32x16{} : s[i & 1]);
        order<SCHED_LDS_READ, 4>();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          order<SCHED_MFMA, 1>();
          order<SCHED_VALU, 5>();
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (needs_clean(t + 1) && t + 1 < t1) clean(t + 1);
      fetch(t + 2);  // not under a condition: its registers would be copied, which waits for the loads
      look_up(t + 3);

      if (t >= tail0 || uniform(outside_seen)) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int tok = t * TILE + 32 * u;
          unsigned in = first_bits<32>(len - tok);
          if (outside_seen) {
            // pages hold 16 tokens at least
            if (tok < len && (unsigned)table[tok >> cv.page_log2] >= (uint64_t)cv.pages) in &= 0xFFFF0000u;
            if (tok + 16 < len && (unsigned)table[(tok + 16) >> cv.page_log2] >= (uint64_t)cv.pages) in &= 0xFFFFu;
          }
          const unsigned vis = (seen_bits<32>(a, q0 + node, node, tok - first_new) & in) >> (4 * h);
#pragma unroll
          for (int r = 0; r < 16; ++r) s[u][r] = (vis >> (8 * (r / 4) + r % 4)) & 1u ? s[u][r] : -__builtin_inff();
        }
      }

      float top = s[0][0];
#pragma unroll
      for (int k = 1; k < 32; ++k) top = fmaxf(top, s[k / 16][k % 16]);
      top = max_halves(top * to_log2);
      if (__builtin_amdgcn_ballot_w64(top > m + LAG)) {
        const float big = fmaxf(m, top);
        const float f = big == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(m - big);
        m = big;
        l *= f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) rescale<ACC>(o[i], f);
      }
      const float base = m == -__builtin_inff() ? 0.0f : m;

      // weights: registers 8 k .. of the scores are the operand for the tokens 16 k ..; those of the next 16 tokens
      // are computed under the products of these
      u32x4 p[4];
      auto weigh = [&](int k, int from, int to) {
#pragma unroll
        for (int i = from; i < to; ++i) {
          const int r = 8 * (k & 1) + 2 * i;
          const float w0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[k / 2][r], to_log2, -base));
          const float w1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[k / 2][r + 1], to_log2, -base));
          p[k][i] = bf16x2_rne(w0, w1);
          l = add_pair(p[k][i], l);
        }
      };
      weigh(0, 0, 4);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int g = 0; g < D / 8 / VG; ++g) {
        const int k = g / PARTS, part = g % PARTS;
        if (g + 1 < D / 8 / VG) read_values(g + 1);
        if (k < 3) weigh(k + 1, 4 * part / PARTS, 4 * (part + 1) / PARTS);
#pragma unroll
        for (int i = 0; i < VG; ++i) o[part * VG + i] = mma32(vf[g & 1][i], p[k], o[part * VG + i]);
#pragma unroll
        for (int i = 0; i < VG; ++i) {
          order<SCHED_LDS_READ, 2>();
          order<SCHED_MFMA, 1>();
          order<SCHED_VALU, (24 / PARTS + VG - 1) / VG>();
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      __syncthreads();
    }

    l = sum_halves(l);
    if (in) {
      if (flags[1]) {
        const int from = tail0 * TILE > t0 * TILE ? tail0 * TILE : t0 * TILE;
        const int to = t1 * TILE < len ? t1 * TILE : len;
        seen_tokens(a, table, head, q0 + node, node, first_new, from, to, [&](int64_t ph, int r) {
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
              for (int e = 0; e < 4; ++e) o[i][4 * c + e] += not_finite_or_zero(w[e / 2], e & 1);
            }
          }
        });
      }
      if (t1 - t0 == tiles) {
        const int64_t at = (int64_t)(q0 + node) * cv.heads * a.group + head * a.group + (row - node * a.group);
        const float inv = reciprocal(l);
        unsigned short *d = a.out + at * D + 4 * h;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            *(u32x2 *)(d + 32 * i + 8 * r) = u32x2{bf16x2_rne(o[i][4 * r] * inv, o[i][4 * r + 1] * inv),
                                                   bf16x2_rne(o[i][4 * r + 2] * inv, o[i][4 * r + 3] * inv)};
      } else {
        const int64_t part = 2 * (int64_t)blockIdx.x + slot;
        const int r0 = wave * 32 + n32;  // of the block
        float *d = part_sums(a, dv, part, D) + (int64_t)r0 * D + 4 * h;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            *(f32x4 *)(d + 32 * i + 8 * r) =
                f32x4{o[i][4 * r], o[i][4 * r + 1], o[i][4 * r + 2], o[i][4 * r + 3]};
        if (h == 0) {
          float *ml = part_stats(a, dv, part, D) + 2 * r0;
          ml[0] = m;
          ml[1] = l;
        }
      }
    }
  }
  pc.finish(a, dv);
  zero_padding(a);
}

template <int FMT, int D, int WAVES>
static hipError_t start(const AttentionArgs &a, const Division &d, hipStream_t stream) {
  using T = Tiled<FMT, D, WAVES>;
  const int64_t grid = d.workers ? d.workers : (int64_t)a.batch * a.cache.heads * d.blocks;
  static std::atomic<uint64_t> done{0};
  const hipError_t e = allow_lds((const void *)k_attention_tiles<FMT, D, WAVES>, T::LDS, done);
  if (e != hipSuccess) return e;
  k_attention_tiles<FMT, D, WAVES><<<(unsigned)grid, T::THREADS, T::LDS, stream>>>(a, d);
  return hipGetLastError();
}

template <int FMT, int D>
static hipError_t by_rows(const AttentionArgs &a, const Division &d, hipStream_t stream) {
  if (d.rows == 128) return start<FMT, D, 4>(a, d, stream);
  if constexpr (D <= 128) return start<FMT, D, 8>(a, d, stream);
  return hipErrorInvalidValue;
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
