// Attention of new tokens over the paged MX cache, for up to 32 rows of a
// key/value head (16 where heads have more than 128 dimensions): single tokens,
// small trees.
//
//   out[i] = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i . k_j - m_i)
//   over the tokens j that row i sees: all before the sequence's new tokens,
//   and of those the ones up to its own (causal) or those that its bits name
//   (a tree of drafted tokens).  A row that sees nothing gives zeros.
//
// Bound: HBM, every code and scale once (FETCH: TCC misses of 128 bytes equal
// the bytes of the case).  Measured on MI355X: 64 sequences of 16384, 8 heads of
// 128, 4 query heads each: MXFP8 381-384 us, 5.8 TB/s; MXFP4 227-235 us, 5.0 TB/s,
// where conversions and softmax of half the bytes take the vector units over half
// of the time; one sequence of 500000 in MXFP4 111 us, 4.9 TB/s.
//
// Rows: the queries of the `group` heads that share a key/value head, for all
// new tokens of the sequence, are the rows of one product: row = token * group
// + head in the group.  A workgroup takes a run of tiles of 64 tokens (see the
// division in attention.h), its four waves every fourth of them, each with a
// running maximum and sum of its own, and join in LDS at the end of an item.
//
// Everything between the loads and the end stays in the lane that it is in.
// S^T = K Q^T and O^T = V^T P^T on v_mfma_f32_16x16x32_bf16 (lane l holds for
// column or row l % 16 of an operand the 8 elements of k = 8 (l / 16) ..; and
// of the result column l % 16, rows 4 (l / 16) ..).  Which token or dimension
// an index of k means is free as long as both operands agree:
//   - a tile's score products t = 0 .. 3 take tokens 4 m + t as their rows m, so that a lane's
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
// the second product, and their sum takes them rounded, so that the weights add
// up to one.
#include "attention.h"

namespace mx {

constexpr int ATT_WAVES = 4;

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

__device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                 0);
}

// What a wave keeps for its rows.
template <int D, int NT> struct RowState {
  f32x4 o[NT][D / 16];
  float m[NT], l[NT];  // maximum in units of log2, the same in the four lanes of a row; this lane's part of the sum
};

// PV for one run of CNT dimensions (8 tokens a step, 2 steps): acc[i] += V^T[dims] P^T.
template <int FMT, int CNT, int NT, int W, int CW>
__device__ __forceinline__ void accumulate(f32x4 (*acc)[W], int base, unsigned (*codes)[CW], const unsigned *scales,
                                           const u32x4 (*p)[2]) {
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    unsigned w[8][CNT / 2];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int tok = 8 * s + j;
      widen<FMT, CNT>(w[j], codes[tok], (scales[tok / 4] >> (8 * (tok & 3))) & 0xFFu);
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
      }
    __builtin_amdgcn_sched_barrier(0);  // one step's widened values at a time
  }
}

// In a tile that needs a mask: codes of the tokens from `valid` on become zero, and where rows differ in what they see
// (`differ`, all ones or zero) so do the codes of values that are not finite (`odd` tells of these).
template <int FMT, int CNT, int CW>
__device__ __forceinline__ void clear_codes(unsigned (*codes)[CW], unsigned *scales, int valid, unsigned differ,
                                            unsigned &odd) {
  constexpr int BITS = FMT == 0 ? 4 : 8;
  constexpr unsigned ONE = (1u << BITS) - 1u;
#pragma unroll
  for (int tok = 0; tok < 16; ++tok) {
    const int at = 8 * (tok & 3);
    const unsigned sb = (scales[tok / 4] >> at) & 0xFFu;
    unsigned w[CNT / 2];
    widen<FMT, CNT>(w, codes[tok], sb);
    const unsigned in = tok < valid ? 0xFFFFFFFFu : 0u;
    unsigned clear[CW] = {};
#pragma unroll
    for (int i = 0; i < CNT / 2; ++i) {
      const unsigned bad = not_finite(w[i]) & in & differ;
      odd |= bad;
      clear[2 * i * BITS / 32] |= ((bad & 1u) * ONE | (bad >> 16) * (ONE << BITS)) << (2 * i * BITS % 32);
    }
#pragma unroll
    for (int i = 0; i < CW; ++i) codes[tok][i] &= in & ~clear[i];
    if ((sb == 255u && differ) || !in) scales[tok / 4] &= ~(0xFFu << at);
    __builtin_amdgcn_sched_barrier(0);
  }
}

// Adds a token's values that are not finite to the sums of one run of dimensions.
template <int FMT, int CNT, int W>
__device__ __forceinline__ void spoil(f32x4 (&acc)[W], int base, const uint8_t *codes, const uint8_t *scales, int first,
                                      int page_log2) {
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int d = first + CNT * r;
    unsigned code[(CNT + 3) / 4], w[CNT / 2];
    load_bytes<FMT == 0 ? CNT / 2 : CNT>(code, codes + (FMT == 0 ? d / 2 : d));
    widen<FMT, CNT>(w, code, scales[(d / 32) << page_log2]);
#pragma unroll
    for (int i = 0; i < CNT; ++i) acc[base + i][r] += not_finite_or_zero(w[i / 2], i & 1);
  }
}

template <int FMT, int D, int NT>
__global__ __launch_bounds__(64 * ATT_WAVES, rows_held(D, NT)) void k_attention_rows(AttentionArgs a, Division dv) {
  using A = Att<FMT, D>;
  constexpr bool ACC = NT > 1 || D > 128;  // one wave a SIMD: the sums are in accumulation registers
  extern __shared__ float lds[];
  const CacheView &cv = a.cache;
  const int wave = uniform((int)threadIdx.x / 64), lane = threadIdx.x % 64, n16 = lane % 16, g = lane / 16;
  const int page_mask = (1 << cv.page_log2) - 1;
  Pieces pc(a, dv);
  while (pc.next(a, dv)) {
    const int nq = uniform(pc.s.nq), len = uniform(pc.s.len), q0 = uniform(pc.s.q0), b = uniform(pc.b);
    const int head = uniform(pc.head), rb = uniform(pc.block);
    const int t0 = uniform(pc.t0), t1 = uniform(pc.t1), tiles = uniform(pc.tiles), slot = uniform(pc.slot);
  const int rows = nq * a.group;
  const int lo = t0 * TILE, hi = t1 * TILE < len ? t1 * TILE : len;
  const int first_new = uniform(pc.s.first_new);
  const int seen_by_all = a.tree ? first_new : first_new + 1;       // tokens before this need no mask
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
  unsigned odd = 0u;  // values that are not finite were taken out of a tile
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

  const float to_log2 = a.scale * LOG2_E;
  // rows may differ in what they see of the tile, or it ends behind the tokens
  auto differs = [&](int base) { return base + TILE > seen_by_all || base + TILE > hi; };
  const int first = lo + TILE * wave;
  if (first < hi) {
    load_k(first);
    load_v(first);
  }
  for (int base = first; base < hi; base += TILE * ATT_WAVES) {
    // scores: tile t holds tokens base + 4 m + t
    f32x4 s[NT][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
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
        if constexpr (FMT == 0) widen<0, 8>(w, &kc[t][i], sb);
        else widen<1, 8>(w, &kc[t][2 * i], sb);
        k = u32x4{w[0], w[1], w[2], w[3]};
#pragma unroll
        for (int n = 0; n < NT; ++n) s[n][t] = mma(k, q[n][i], i == 0 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : s[n][t]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    const int next = base + TILE * ATT_WAVES;
    if (next < hi) load_k(next);

    // the tokens of this lane that each row sees: bit 4 r + t
    const int tok0 = base + 16 * g;
    const bool masked = __builtin_amdgcn_ballot_w64(bad || differs(base)) != 0;
    int valid = 16;
    if (masked) {
      valid = bad ? 0 : hi - tok0;
      valid = valid < 0 ? 0 : valid > 16 ? 16 : valid;
      const unsigned in = first_bits<16>(valid);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const unsigned vis = seen_bits<16>(a, q0 + node[n], node[n], tok0 - first_new) & in;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            s[n][t][r] = (vis >> (4 * r + t)) & 1u ? s[n][t][r] : -__builtin_inff();
      }
    }

    // weights
    u32x4 p[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float top = s[n][0][0];
#pragma unroll
      for (int k = 1; k < 16; ++k) top = fmaxf(top, s[n][k / 4][k % 4]);
      top = max_rows16(max_halves(top * to_log2));
      if (__builtin_amdgcn_ballot_w64(top > st.m[n] + LAG)) {
        const float m = fmaxf(st.m[n], top);
        const float f = m == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(st.m[n] - m);
        st.m[n] = m;
        st.l[n] *= f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) rescale<ACC>(st.o[n][i], f);
      }
      const float m = st.m[n] == -__builtin_inff() ? 0.0f : st.m[n];
      float w[16];  // by token
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          w[4 * r + t] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][t][r], to_log2, -m));
        }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          p[n][h][k] = bf16x2_rne(w[8 * h + 2 * k], w[8 * h + 2 * k + 1]);
          st.l[n] = add_pair(p[n][h][k], st.l[n]);
        }
    }

    if (masked) {
      const unsigned differ = differs(base) ? 0xFFFFFFFFu : 0u;
      clear_codes<FMT, A::C0>(vc0, vs0, valid, differ, odd);
      if constexpr (A::C1 > 0) clear_codes<FMT, A::C1>(vc1, vs1, valid, differ, odd);
    }
    accumulate<FMT, A::C0, NT>(st.o, 0, vc0, vs0, p);
    if constexpr (A::C1 > 0) accumulate<FMT, A::C1, NT>(st.o, A::C0, vc1, vs1, p);
    if (next < hi) load_v(next);
  }

  if (__builtin_amdgcn_ballot_w64(odd != 0u)) {
    // of this wave's tiles, the ones they were taken out of
    for (int base = first; base < hi; base += TILE * ATT_WAVES) {
      if (!differs(base)) continue;
      const int to = base + TILE < hi ? base + TILE : hi;
#pragma unroll
      for (int n = 0; n < NT; ++n)
        seen_tokens(a, table, head, q0 + node[n], node[n], first_new, base, to, [&](int64_t ph, int r) {
          const uint8_t *c = cv.codes[1] + ((ph << cv.page_log2) + r) * A::RB;
          const uint8_t *sc = cv.scales[1] + ((ph * A::G) << cv.page_log2) + r;
          spoil<FMT, A::C0>(st.o[n], 0, c, sc, 4 * A::C0 * g, cv.page_log2);
          if constexpr (A::C1 > 0) spoil<FMT, A::C1>(st.o[n], A::C0, c, sc, A::B1 + 4 * A::C1 * g, cv.page_log2);
        });
    }
  }

  // join the waves: two give theirs to two, one to one
#pragma unroll
  for (int n = 0; n < NT; ++n) st.l[n] = sum_rows16(sum_halves(st.l[n]));
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
  if (wave) continue;

#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int row = (rb * NT + n) * 16 + n16;
    if (row >= rows) continue;
    // lane chunk 4 g + r of run 0 (C0 dimensions from C0 (4 g + r)) and of run 1
    if (t1 - t0 == tiles) {
      const int64_t at = (int64_t)(q0 + node[n]) * cv.heads * a.group + head * a.group + (row - node[n] * a.group);
      const float inv = reciprocal(st.l[n]);
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
      const int r16 = n * 16 + n16;  // of the block
      float *o = part_sums(a, dv, 2 * (int64_t)blockIdx.x + slot, D) + (int64_t)r16 * D;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
#pragma unroll
        for (int i = 0; i < A::C0; ++i) o[A::C0 * (4 * g + r) + i] = st.o[n][i][r];
#pragma unroll
        for (int i = 0; i < A::C1; ++i) o[A::B1 + A::C1 * (4 * g + r) + i] = st.o[n][A::C0 + i][r];
      }
      if (g == 0) {
        float *ml = part_stats(a, dv, 2 * (int64_t)blockIdx.x + slot, D) + 2 * r16;
        ml[0] = st.m[n];
        ml[1] = st.l[n];
      }
    }
  }
  }
  pc.finish(a, dv);
  zero_padding(a);
}

template <int FMT, int D, int NT>
static hipError_t start(const AttentionArgs &a, const Division &d, hipStream_t stream) {
  const int64_t grid = d.workers ? d.workers : (int64_t)a.batch * a.cache.heads * d.blocks;
  constexpr int bytes = 2 * NT * (D / 4 + 2) * 64 * 4;
  static_assert(bytes <= 65536, "more LDS than a kernel has without asking");
  k_attention_rows<FMT, D, NT><<<(unsigned)grid, 64 * ATT_WAVES, bytes, stream>>>(a, d);
  return hipGetLastError();
}

template <int FMT, int D>
static hipError_t by_rows(const AttentionArgs &a, const Division &d, hipStream_t stream) {
  if (d.rows == 16) return start<FMT, D, 1>(a, d, stream);
  if constexpr (D <= 128) return start<FMT, D, 2>(a, d, stream);
  return hipErrorInvalidValue;
}

hipError_t launch_attention_rows(const AttentionArgs &a, const Division &d, hipStream_t stream) {
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
