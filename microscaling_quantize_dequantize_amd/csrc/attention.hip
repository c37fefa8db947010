// Attention of new tokens over the paged MX cache.
//
//   out[i] = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i . k_j - m_i)
//   over the tokens j that row i sees: all before the sequence's new tokens,
//   and of those the ones up to its own (causal) or those that its bits name
//   (a tree of drafted tokens).  A row that sees nothing gives zeros.
//
// Rows: the queries of the `group` heads that share a key/value head, for all
// new tokens of the sequence, are the rows of one product: row = token * group
// + head in the group.  A workgroup takes 16 NT rows and a span of the
// sequence's tokens, its four waves take units of 64 tokens of it in turn, each
// with a running maximum and sum of its own, and join in LDS at the end.  Long
// spans are split over workgroups, whose unnormalised fp32 sums are joined by a
// second kernel.
//
// Everything between the loads and the end stays in the lane that it is in.
// S^T = K Q^T and O^T = V^T P^T on v_mfma_f32_16x16x32_bf16 (lane l holds for
// column or row l % 16 of an operand the 8 elements of k = 8 (l / 16) ..; and
// of the result column l % 16, rows 4 (l / 16) ..).  Which token or dimension
// an index of k means is free as long as both operands agree:
//   - tile t of a unit takes tokens 4 m + t as its rows m, so that a lane's
//     four K rows are neighbours, with one 32-bit load for their scales, and
//     the lane holds the scores of the 16 tokens 16 (l / 16) .. of its row;
//   - a lane's share of a K row is D/4 neighbouring dimensions;
//   - the scores, as they lie, are the operand of the second product for 16
//     neighbouring tokens of V, whose scales are one 16-byte load;
//   - a lane's D/16 dimensions of V (neighbours) go to D/16 products, so only
//     pairs of tokens have to be exchanged within the lane (v_perm_b32).
// Keys and values are converted to bf16 with their scales, which is exact down
// to bf16's smallest normal, queries are bf16, products are accumulated in
// fp32, the maximum, the sum and the output's sums are fp32.  The weights p are
// rounded to bf16 (at most 2^-8 of each, independent of one another) for
// the second product; their sum takes them unrounded.
#include "launch.h"

namespace mx {

constexpr int ATT_WAVES = 4;
constexpr int UNIT = 64;  // tokens a wave takes at a time

template <int FMT, int D> struct Att {
  static constexpr int G = D / 32;                   // scales of a row
  static constexpr int RB = FMT == 0 ? D / 2 : D;    // bytes of a row
  static constexpr int KB = RB / 4;                  // bytes of a lane's share of a K row
  static constexpr int KW = KB / 4;
  static constexpr int STEPS = D / 32;               // products for a score tile
  static constexpr int NB = D == 64 || D == 128 ? 1 : 2;  // scales a share of a K row touches
  // V: a lane's dimensions, in one or two runs of neighbours (C0 from C0 * lane, C1 from B1 + C1 * lane)
  static constexpr int C0 = D == 96 ? 4 : D == 192 ? 8 : D / 16;
  static constexpr int C1 = D == 96 ? 2 : D == 192 ? 4 : 0;
  static constexpr int B1 = 16 * C0;
  static constexpr int VB0 = FMT == 0 ? C0 / 2 : C0, VB1 = FMT == 0 ? C1 / 2 : C1;  // bytes
  static constexpr int VW0 = (VB0 + 3) / 4, VW1 = (VB1 + 3) / 4;
};

// N bytes at p (aligned to the largest power of two that divides N) into words
template <int N>
__device__ __forceinline__ void load_bytes(unsigned *w, const uint8_t *p) {
  if constexpr (N % 16 == 0) {
#pragma unroll
    for (int i = 0; i < N / 16; ++i) {
      const u32x4 v = ((const u32x4 *)p)[i];
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  } else if constexpr (N % 8 == 0) {
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
      const u32x2 v = ((const u32x2 *)p)[i];
      w[2 * i] = v.x, w[2 * i + 1] = v.y;
    }
  } else if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) w[i] = ((const unsigned *)p)[i];
  } else if constexpr (N == 2) {
    w[0] = *(const unsigned short *)p;
  } else if constexpr (N == 1) {
    w[0] = *p;
  }
}

// Pairs of neighbouring dimensions of CNT codes as bf16.
template <int FMT, int CNT>
__device__ __forceinline__ void widen(unsigned *o, const unsigned *c, float sc) {
#pragma unroll
  for (int p = 0; p < CNT / 2; ++p) {
    if constexpr (FMT == 0) {
      const unsigned w = c[p / 4];
      bf16x2 r;
      switch (p & 3) {
        case 0: r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 0); break;
        case 1: r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 1); break;
        case 2: r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 2); break;
        default: r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 3); break;
      }
      o[p] = __builtin_bit_cast(unsigned, r);
    } else {
      const unsigned w = c[p / 2];
      o[p] = __builtin_bit_cast(unsigned, (p & 1) ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, sc, true)
                                                  : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, sc, false));
    }
  }
}

// The conversions' scale of an E8M0 byte: 2^(b-127), NaN for 0xFF (its exponent field with a mantissa).
__device__ __forceinline__ float e8m0(unsigned b) { return scale_operand(b); }

__device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                 0);
}

// Maximum and sum over the four lanes that hold a row (l, l ^ 16, l ^ 32, l ^ 48).
__device__ __forceinline__ float row_max(float v) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float row_sum(float v) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// What a wave keeps for its rows.
template <int D, int NT> struct RowState {
  f32x4 o[NT][D / 16];
  float m[NT], l[NT];  // maximum in units of log2, the same in the four lanes of a row; this lane's part of the sum
};

// The weights' maximum may lag behind the scores' by this many powers of two before the sums are rescaled.
constexpr float LAG = 8.0f;

// PV for one run of CNT dimensions (8 tokens a step, 2 steps): acc[i] += V^T[dims] P^T.
// MASKED: codes of tokens past the sequence are cleared, and values that are not finite reach only the rows
// that see them: they are taken out, and where a row sees one (a count by the same product) the result is NaN.
template <int FMT, int CNT, int NT, bool MASKED, int W, int CW>
__device__ __forceinline__ void accumulate(f32x4 (*acc)[W], int base, unsigned (*codes)[CW], const unsigned *scales,
                                           const u32x4 (*p)[2], const unsigned *vis,
                                           int valid) {
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    unsigned w[8][CNT / 2];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int tok = 8 * s + j;
      unsigned sb = (scales[tok / 4] >> (8 * (tok & 3))) & 0xFFu;
      unsigned c[CW];
#pragma unroll
      for (int i = 0; i < CW; ++i) c[i] = MASKED && tok >= valid ? 0u : codes[tok][i];
      if (MASKED && tok >= valid) sb = 0u;
      widen<FMT, CNT>(w[j], c, e8m0(sb));
      if (sb == 255u) {
#pragma unroll
        for (int i = 0; i < CNT / 2; ++i) w[j][i] = BF16_NAN | (BF16_NAN << 16);
      }
    }
    unsigned odd[8][CNT / 2];  // 1.0 where a value is not finite
    bool any = false;
    if (MASKED) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int i = 0; i < CNT / 2; ++i) {
          const bool lo = (w[j][i] & 0x7F80u) == 0x7F80u, hi = (w[j][i] & 0x7F800000u) == 0x7F800000u;
          odd[j][i] = (lo ? 0x3F80u : 0u) | (hi ? 0x3F800000u : 0u);
          w[j][i] &= (lo ? 0u : 0xFFFFu) | (hi ? 0u : 0xFFFF0000u);
          any |= lo | hi;
        }
      any = __builtin_amdgcn_ballot_w64(any) != 0;
    }
#pragma unroll
    for (int i = 0; i < CNT / 2; ++i)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const unsigned sel = half ? 0x07060302u : 0x05040100u;
        const u32x4 a{__builtin_amdgcn_perm(w[1][i], w[0][i], sel), __builtin_amdgcn_perm(w[3][i], w[2][i], sel),
                      __builtin_amdgcn_perm(w[5][i], w[4][i], sel), __builtin_amdgcn_perm(w[7][i], w[6][i], sel)};
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[n][base + 2 * i + half] = mma(a, p[n][s], acc[n][base + 2 * i + half]);
        if (MASKED && any) {
          const u32x4 b{__builtin_amdgcn_perm(odd[1][i], odd[0][i], sel), __builtin_amdgcn_perm(odd[3][i], odd[2][i], sel),
                        __builtin_amdgcn_perm(odd[5][i], odd[4][i], sel), __builtin_amdgcn_perm(odd[7][i], odd[6][i], sel)};
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            u32x4 sees;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              sees[k] = ((vis[n] >> (8 * s + 2 * k)) & 1u ? 0x3F80u : 0u) |
                        ((vis[n] >> (8 * s + 2 * k + 1)) & 1u ? 0x3F800000u : 0u);
            const f32x4 count = mma(b, sees, f32x4{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (count[r] > 0.0f) acc[n][base + 2 * i + half][r] = __uint_as_float(F32_NAN);
          }
        }
      }
  }
}

struct Span {  // host's choice of the split
  int chunk, splits, row_blocks;
};

template <int FMT, int D, int NT>
__global__ __launch_bounds__(64 * ATT_WAVES) void k_attention(AttentionArgs a, Span sp) {
  using A = Att<FMT, D>;
  extern __shared__ float lds[];
  const CacheView &cv = a.cache;
  // Consecutive workgroups go to the eight XCDs in turn: the row blocks of the same tokens are put on one, whose L2
  // then holds the tokens.
  const int items = sp.splits * a.batch * cv.heads;
  const int xcd = blockIdx.x % 8, local = blockIdx.x / 8;
  const int rb = local % sp.row_blocks, item = local / sp.row_blocks * 8 + xcd;
  if (item >= items) return;
  const int head = item % cv.heads, b = item / cv.heads % a.batch, split = item / cv.heads / a.batch;

  int q0 = a.q_starts[b], q1 = a.q_starts[b + 1];
  q0 = q0 < 0 ? 0 : q0;
  q1 = q1 > a.total_q ? a.total_q : q1;
  const int nq = q1 - q0, rows = nq * a.group;
  if (nq <= 0 || rb * 16 * NT >= rows) return;
  int len = a.kv_lens[b];
  len = len < 0 ? 0 : len > a.max_kv ? a.max_kv : len;
  const int cap = a.table_pages << cv.page_log2;
  len = len > cap ? cap : len;
  const int lo = split * sp.chunk;
  if (lo >= len && split > 0) return;  // (a sequence of no tokens still writes its zeros)
  const int hi = len - lo < sp.chunk ? len : lo + sp.chunk;
  const int first_new = len - nq;                                   // may be negative
  const int seen_by_all = a.tree ? first_new : first_new + 1;       // tokens before this need no mask

  const int wave = threadIdx.x / 64, lane = threadIdx.x % 64, n16 = lane % 16, g = lane / 16;
  const int page_mask = (1 << cv.page_log2) - 1;
  const int *table = a.table + (int64_t)b * a.table_stride;

  // queries: row n16 of each tile, the lane's D/4 dimensions
  u32x4 q[NT][A::STEPS];
  int node[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int row = (rb * NT + n) * 16 + n16;
    const bool in = row < rows;
    node[n] = in ? row / a.group : 0;
    const unsigned short *x = a.q + (int64_t)(q0 + node[n]) * a.q_token +
                              (int64_t)(head * a.group + (in ? row - node[n] * a.group : 0)) * a.q_head + g * (D / 4);
#pragma unroll
    for (int i = 0; i < A::STEPS; ++i) q[n][i] = in ? *(const u32x4 *)(x + 8 * i) : u32x4{0u, 0u, 0u, 0u};
  }

  RowState<D, NT> st;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    st.m[n] = -__builtin_inff();
    st.l[n] = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) st.o[n][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  unsigned kc[4][A::KW], ks[A::NB];
  unsigned vc0[16][A::VW0], vc1[16][A::VW1 > 0 ? A::VW1 : 1];
  unsigned vs0[4], vs1[4];
  bool bad = false;  // the page of the lane's 16 tokens is not in the cache

  // a page, or page 0 in place of one that is not in the cache (its tokens are masked)
  auto page_of = [&](int tok) {
    const unsigned p = (unsigned)table[tok >> cv.page_log2];
    return p < (uint64_t)cv.pages ? (int)p : -1;
  };
  auto load_k = [&](int base) {
    int tok = base + 4 * n16;
    const int last = (len - 1) & ~3;
    tok = tok > last ? last : tok;
    const int p = page_of(tok);
    const int64_t ph = (int64_t)(p < 0 ? 0 : p) * cv.heads + head;
    const int r = tok & page_mask;
    const uint8_t *c = cv.codes[0] + ((ph << cv.page_log2) + r) * A::RB + g * A::KB;
#pragma unroll
    for (int t = 0; t < 4; ++t) load_bytes<A::KB>(kc[t], c + t * A::RB);
    const int b0 = g * (D / 4) / 32;
#pragma unroll
    for (int i = 0; i < A::NB; ++i) {
      const int blk = b0 + i < A::G ? b0 + i : A::G - 1;
      ks[i] = *(const unsigned *)(cv.scales[0] + ((ph * A::G + blk) << cv.page_log2) + r);
    }
  };
  auto load_v = [&](int base) {
    int tok = base + 16 * g;
    const int last = (len - 1) & ~15;
    tok = tok > last ? last : tok;
    const int p = page_of(tok);
    bad = p < 0;
    const int64_t ph = (int64_t)(p < 0 ? 0 : p) * cv.heads + head;
    const int r = tok & page_mask;
    const uint8_t *c = cv.codes[1] + ((ph << cv.page_log2) + r) * A::RB;
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      load_bytes<A::VB0>(vc0[t], c + t * A::RB + n16 * A::VB0);
      if constexpr (A::C1 > 0) load_bytes<A::VB1>(vc1[t], c + t * A::RB + 16 * A::VB0 + n16 * A::VB1);
    }
    const uint8_t *s = cv.scales[1] + ((ph * A::G) << cv.page_log2) + r;
    load_bytes<16>(vs0, s + ((n16 * A::C0 / 32) << cv.page_log2));
    if constexpr (A::C1 > 0) load_bytes<16>(vs1, s + (((A::B1 + n16 * A::C1) / 32) << cv.page_log2));
  };

  const float to_log2 = a.scale * 1.4426950408889634f;
  const int first = lo + UNIT * wave;
  if (first < hi) {
    load_k(first);
    load_v(first);
  }
  for (int base = first; base < hi; base += UNIT * ATT_WAVES) {
    // scores: tile t holds tokens base + 4 m + t
    f32x4 s[NT][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
      for (int n = 0; n < NT; ++n) s[n][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < A::STEPS; ++i) {
        unsigned sb = (ks[0] >> (8 * t)) & 0xFFu;
        if (A::NB > 1) {
          const int rel = (g * (D / 4) % 32 + 8 * i) / 32;
          const unsigned s1 = (ks[A::NB - 1] >> (8 * t)) & 0xFFu;
          sb = rel ? s1 : sb;
        }
        u32x4 k;
        unsigned w[4];
        if constexpr (FMT == 0) widen<0, 8>(w, &kc[t][i], e8m0(sb));
        else widen<1, 8>(w, &kc[t][2 * i], e8m0(sb));
        k = u32x4{w[0], w[1], w[2], w[3]};
        if (sb == 255u) k = u32x4{BF16_NAN, BF16_NAN, BF16_NAN, BF16_NAN};
#pragma unroll
        for (int n = 0; n < NT; ++n) s[n][t] = mma(k, q[n][i], s[n][t]);
      }
    }
    const int next = base + UNIT * ATT_WAVES;
    if (next < hi) load_k(next);

    // the tokens of this lane that each row sees: bit 4 r + t
    const int tok0 = base + 16 * g;
    const bool masked = __builtin_amdgcn_ballot_w64(bad || base + UNIT > seen_by_all || base + UNIT > hi) != 0;
    unsigned vis[NT];
    int valid = 16;
    if (masked) {
      valid = bad ? 0 : hi - tok0;
      valid = valid < 0 ? 0 : valid > 16 ? 16 : valid;
      const unsigned in = (1u << valid) - 1u;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int j0 = tok0 - first_new;  // the first token's place among the new ones
        unsigned see = 0xFFFFu;
        if (a.tree == nullptr) {
          const int count = node[n] + 1 - j0;
          see = count >= 16 ? 0xFFFFu : count <= 0 ? 0u : (1u << count) - 1u;
        } else if (j0 > -16) {
          const int64_t *words = a.tree + (int64_t)(q0 + node[n]) * a.tree_words;
          const int at = j0 < 0 ? 0 : j0;
          const uint64_t w0 = at / 64 < a.tree_words ? (uint64_t)words[at / 64] : 0;
          const uint64_t w1 = at / 64 + 1 < a.tree_words ? (uint64_t)words[at / 64 + 1] : 0;
          uint64_t bits = w0 >> (at % 64);
          if (at % 64) bits |= w1 << (64 - at % 64);
          see = j0 < 0 ? ((unsigned)(bits << -j0) | ((1u << -j0) - 1u)) : (unsigned)bits;
        }
        vis[n] = see & in;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (!((vis[n] >> (4 * r + t)) & 1u)) s[n][t][r] = -__builtin_inff();
      }
    }

    // weights
    u32x4 p[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float top = s[n][0][0];
#pragma unroll
      for (int k = 1; k < 16; ++k) top = fmaxf(top, s[n][k / 4][k % 4]);
      top = row_max(top * to_log2);
      if (__builtin_amdgcn_ballot_w64(top > st.m[n] + LAG)) {
        const float m = fmaxf(st.m[n], top);
        const float f = m == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(st.m[n] - m);
        st.m[n] = m;
        st.l[n] *= f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) st.o[n][i] *= f;
      }
      const float m = st.m[n] == -__builtin_inff() ? 0.0f : st.m[n];
      float w[16];  // by token
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          w[4 * r + t] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][t][r], to_log2, -m));
          st.l[n] += w[4 * r + t];
        }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < 4; ++k) p[n][h][k] = bf16x2_rne(w[8 * h + 2 * k], w[8 * h + 2 * k + 1]);
    }

    if (masked) {
      accumulate<FMT, A::C0, NT, true>(st.o, 0, vc0, vs0, p, vis, valid);
      if constexpr (A::C1 > 0) accumulate<FMT, A::C1, NT, true>(st.o, A::C0, vc1, vs1, p, vis, valid);
    } else {
      accumulate<FMT, A::C0, NT, false>(st.o, 0, vc0, vs0, p, vis, valid);
      if constexpr (A::C1 > 0) accumulate<FMT, A::C1, NT, false>(st.o, A::C0, vc1, vs1, p, vis, valid);
    }
    if (next < hi) load_v(next);
  }

  // join the waves: two give theirs to two, one to one
#pragma unroll
  for (int n = 0; n < NT; ++n) st.l[n] = row_sum(st.l[n]);
  constexpr int WORDS = NT * (D / 4 + 2);  // of a lane
#pragma unroll
  for (int step = 2; step > 0; step /= 2) {
    float *mine = lds + (wave % step) * WORDS * 64 + lane;
    if (wave >= step && wave < 2 * step) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < D / 4; ++i) mine[(n * (D / 4 + 2) + i) * 64] = st.o[n][i / 4][i % 4];
        mine[(n * (D / 4 + 2) + D / 4) * 64] = st.m[n];
        mine[(n * (D / 4 + 2) + D / 4 + 1) * 64] = st.l[n];
      }
    }
    __syncthreads();
    if (wave < step) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float m2 = mine[(n * (D / 4 + 2) + D / 4) * 64], l2 = mine[(n * (D / 4 + 2) + D / 4 + 1) * 64];
        const float m = fmaxf(st.m[n], m2);
        const float f1 = m == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(st.m[n] - m);
        const float f2 = m == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(m2 - m);
        st.m[n] = m;
        st.l[n] = st.l[n] * f1 + l2 * f2;
#pragma unroll
        for (int i = 0; i < D / 4; ++i)
          st.o[n][i / 4][i % 4] = st.o[n][i / 4][i % 4] * f1 + mine[(n * (D / 4 + 2) + i) * 64] * f2;
      }
    }
    __syncthreads();
  }
  if (wave) return;

  const bool whole = len <= sp.chunk;  // nothing to join with
  const int64_t all_rows = (int64_t)a.total_q * cv.heads * a.group;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int row = (rb * NT + n) * 16 + n16;
    if (row >= rows) continue;
    const int64_t at = (int64_t)(q0 + node[n]) * cv.heads * a.group + head * a.group + (row - node[n] * a.group);
    // lane chunk 4 g + r of run 0 (C0 dimensions from C0 (4 g + r)) and of run 1
    if (whole) {
      const float inv = st.l[n] > 0.0f || st.l[n] != st.l[n] ? 1.0f / st.l[n] : 0.0f;
      unsigned short *o = a.out + at * D;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        unsigned *o0 = (unsigned *)(o + A::C0 * (4 * g + r));
#pragma unroll
        for (int i = 0; i < A::C0 / 2; ++i)
          o0[i] = bf16x2_rne(st.o[n][2 * i][r] * inv, st.o[n][2 * i + 1][r] * inv);
        unsigned *o1 = (unsigned *)(o + A::B1 + A::C1 * (4 * g + r));
#pragma unroll
        for (int i = 0; i < A::C1 / 2; ++i)
          o1[i] = bf16x2_rne(st.o[n][A::C0 + 2 * i][r] * inv, st.o[n][A::C0 + 2 * i + 1][r] * inv);
      }
    } else {
      float *o = a.partial + 2 * sp.splits * all_rows + (split * all_rows + at) * D;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
#pragma unroll
        for (int i = 0; i < A::C0; ++i) o[A::C0 * (4 * g + r) + i] = st.o[n][i][r];
#pragma unroll
        for (int i = 0; i < A::C1; ++i) o[A::B1 + A::C1 * (4 * g + r) + i] = st.o[n][A::C0 + i][r];
      }
      if (g == 0) {
        a.partial[2 * (split * all_rows + at)] = st.m[n];
        a.partial[2 * (split * all_rows + at) + 1] = st.l[n];
      }
    }
  }
}

// Joins the splits of a row: out = sum_s 2^(m_s - m) o_s / sum_s 2^(m_s - m) l_s.  One workgroup for a row; its waves
// take every fourth split.
template <int D>
__global__ __launch_bounds__(256) void k_join(AttentionArgs a, Span sp) {
  __shared__ float part[4][D + 2];
  const int heads = a.cache.heads * a.group;
  const int64_t at = blockIdx.x;
  const int token = (int)(at / heads);
  // the sequence of the token
  int lo = 0, hi = a.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.q_starts[mid] <= token) lo = mid; else hi = mid;
  }
  if (token < a.q_starts[lo] || token >= a.q_starts[lo + 1]) return;
  int len = a.kv_lens[lo];
  const int cap = a.table_pages << a.cache.page_log2;
  len = len > a.max_kv ? a.max_kv : len;
  len = len > cap ? cap : len;
  if (len <= sp.chunk) return;  // already written
  const int splits = (len + sp.chunk - 1) / sp.chunk;
  const int64_t all_rows = (int64_t)a.total_q * heads;
  const float *ml = a.partial, *o = a.partial + 2 * sp.splits * all_rows;
  const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
  constexpr int N = (D + 63) / 64;
  float m = -__builtin_inff(), l = 0.0f, acc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.0f;
  for (int s = wave; s < splits; s += 4) m = fmaxf(m, ml[2 * (s * all_rows + at)]);
  const float base = m == -__builtin_inff() ? 0.0f : m;
  for (int s = wave; s < splits; s += 4) {
    const float f = __builtin_amdgcn_exp2f(ml[2 * (s * all_rows + at)] - base);
    l += f * ml[2 * (s * all_rows + at) + 1];
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (D % 64 == 0 || 64 * i + lane < D) acc[i] += f * o[(s * all_rows + at) * D + 64 * i + lane];
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (64 * i + lane < D) part[wave][64 * i + lane] = acc[i];
  if (lane == 0) part[wave][D] = m, part[wave][D + 1] = l;
  __syncthreads();
  const int d = threadIdx.x;
  if (d >= D) return;
  float top = -__builtin_inff(), sum = 0.0f, v = 0.0f;
#pragma unroll
  for (int w = 0; w < 4; ++w) top = fmaxf(top, part[w][D]);
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float f = part[w][D] == -__builtin_inff() ? (part[w][D + 1] != 0.0f ? 1.0f : 0.0f) : __builtin_amdgcn_exp2f(part[w][D] - top);
    sum += f * part[w][D + 1];
    v += f * part[w][d];
  }
  const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
  a.out[at * D + d] = (unsigned short)bf16x2_rne(v * inv, 0.0f);
}

// Rows of a workgroup and the split of the tokens, from what the host knows (the longest sequence, the most new
// tokens).
struct Plan {
  int nt;
  Span span;
};

static Plan attention_plan(int dim, int heads, int group, int batch, int64_t max_q, int64_t max_kv) {
  const int64_t rows = max_q * group;
  Plan p;
  p.nt = rows <= 16 ? 1 : rows <= 32 || dim > 128 ? 2 : 4;
  p.span.row_blocks = (int)((rows + 16 * p.nt - 1) / (16 * p.nt));
  const int64_t unit = UNIT * ATT_WAVES;
  const int64_t units = max_kv > 0 ? (max_kv + unit - 1) / unit : 1;
  // enough workgroups to fill the CUs a few times over, so that ragged lengths even out
  const int64_t want = 8 * (int64_t)device_cu_count(), have = (int64_t)batch * heads * p.span.row_blocks;
  int64_t splits = (want + have - 1) / have;
  splits = splits < 1 ? 1 : splits > units ? units : splits;
  const int64_t chunk = (units + splits - 1) / splits * unit;
  p.span.chunk = (int)chunk;
  p.span.splits = (int)(max_kv > 0 ? (max_kv + chunk - 1) / chunk : 1);
  return p;
}

int64_t attention_workspace(int fmt, int dim, int heads, int group, int batch, int64_t total_q, int64_t max_q,
                            int64_t max_kv) {
  if (batch == 0 || max_q == 0) return 0;
  const Plan p = attention_plan(dim, heads, group, batch, max_q, max_kv);
  return p.span.splits < 2 ? 0 : p.span.splits * total_q * heads * group * (dim + 2) * 4;
}

template <int FMT, int D, int NT>
static hipError_t start(const AttentionArgs &a, const Span &sp, hipStream_t stream) {
  const int64_t items = (int64_t)sp.splits * a.batch * a.cache.heads;
  const unsigned grid = (unsigned)((items + 7) / 8 * 8 * sp.row_blocks);
  constexpr int bytes = 2 * NT * (D / 4 + 2) * 64 * 4;
  if (bytes > 65536) {
    const hipError_t e = hipFuncSetAttribute((const void *)k_attention<FMT, D, NT>,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
  }
  k_attention<FMT, D, NT><<<grid, 64 * ATT_WAVES, bytes, stream>>>(a, sp);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || sp.splits < 2) return e;
  k_join<D><<<(unsigned)((int64_t)a.total_q * a.cache.heads * a.group), 256, 0, stream>>>(a, sp);
  return hipGetLastError();
}

template <int FMT, int D>
static hipError_t by_rows(const AttentionArgs &a, hipStream_t stream) {
  const Plan p = attention_plan(D, a.cache.heads, a.group, a.batch, a.max_q, a.max_kv);
  if (p.nt == 1) return start<FMT, D, 1>(a, p.span, stream);
  if (p.nt == 2) return start<FMT, D, 2>(a, p.span, stream);
  if constexpr (D <= 128) return start<FMT, D, 4>(a, p.span, stream);
  return hipErrorInvalidValue;
}

hipError_t launch_cache_attention(const AttentionArgs &a, hipStream_t stream) {
#define MX_DIM(D) case D: return a.cache.fmt == 0 ? by_rows<0, D>(a, stream) : by_rows<1, D>(a, stream)
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
