// What the attention kernels share: sequences and the division of their work,
// conversions, row statistics.
#pragma once

#include <atomic>

#include "launch.h"

namespace mx {

constexpr int TILE = 64;  // tokens of a tile, the unit of the division

// How the work is divided.  An item is a block of rows of one key/value head of one sequence, its work the tiles of
// 64 tokens that it reads; items follow one another by sequence, head and block.  `workers` workgroups take equal
// runs of tiles (not less than min_tiles), so that ragged sequences need no host copy of their lengths to be spread
// evenly.  A run that covers an item whole writes the result; pieces of an item go to the worker's two slots of the
// workspace and are joined by k_join.  Slot 0 is for a piece that continues its item, which only the run's first can;
// slot 1 for one that begins its item, which then is the run's last.  workers == 0: one workgroup for each item,
// nothing to join.
//
// What k_join goes by: a record for each item that the host's bounds allow, or, where these are more than the workers
// (one long sequence among many gives every one of them its blocks), a record for each worker, of the divided item that
// its run ends with.
struct Division {
  int workers, min_tiles, rows;  // rows: of a block
  int blocks, tiles;             // host's bounds on an item's blocks and tiles
  int records;                   // of items, or of workers
  bool by_worker;
};
struct Record {
  int first, last;  // workers that have the item's pieces
  int b, part;      // the item: sequence, head * blocks + block (of a worker's record)
};

// What is computed of a sequence: queries q0 .. q0 + nq, tokens 0 .. len.  first_new is the place of its first new
// token, from the lengths as they are: bounds below them leave queries and tokens out, and move no mask.  It is negative
// where there are more queries than tokens.
struct Sequence {
  int q0, nq, len, first_new;
};

// Values that are the same in every lane of a wave, told to the compiler: they stay in scalar registers, and branches
// on them cost no exec mask.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
  return (int64_t)(((uint64_t)(unsigned)uniform((int)(v >> 32)) << 32) | (unsigned)uniform((int)v));
}
__device__ __forceinline__ Sequence uniform(const Sequence &s) {
  return Sequence{uniform(s.q0), uniform(s.nq), uniform(s.len), uniform(s.first_new)};
}

__device__ __forceinline__ Sequence sequence_of(const AttentionArgs &a, int b) {
  Sequence s;
  const int q0 = a.q_starts[b], q1 = a.q_starts[b + 1];
  s.q0 = q0 < 0 ? 0 : q0;
  s.nq = (q1 > a.total_q ? a.total_q : q1) - s.q0;
  s.nq = s.nq < 0 ? 0 : s.nq;
  const int64_t cap = (int64_t)a.table_pages << a.cache.page_log2;
  int len = a.kv_lens[b];
  len = len < 0 ? 0 : len;
  s.first_new = len - s.nq;
  s.nq = s.nq > a.max_q ? a.max_q : s.nq;
  len = len > a.max_kv ? a.max_kv : len;
  s.len = len > cap ? (int)cap : len;
  return s;
}

// Zeros for the queries from `from` on, written by the last `groups` workgroups (of which `mine` is the place).
__device__ __forceinline__ void zero_rows(const AttentionArgs &a, int from, int groups, int mine) {
  const int64_t row = (int64_t)a.cache.heads * a.group * (a.cache.dim / 8), step = (int64_t)groups * blockDim.x;
  const int64_t first = from * row + (int64_t)mine * blockDim.x + threadIdx.x;
  for (int64_t i = first; i < a.total_q * row; i += step) ((u32x4 *)a.out)[i] = u32x4{0u, 0u, 0u, 0u};
}

// Queries of no sequence, from q_starts[batch] on (a batch may be padded at its end), give zeros.  The last 64
// workgroups see to it when their runs are done: where there is little work these have none.  (A load for it in every
// workgroup cost small trees 0.3 of 29 us.)
__device__ __forceinline__ void zero_padding(const AttentionArgs &a) {
  const int groups = gridDim.x < 64 ? gridDim.x : 64, mine = (int)(blockIdx.x - (gridDim.x - groups));
  if (mine < 0) return;
  const int end = uniform(a.q_starts[a.batch]);
  zero_rows(a, end < 0 ? 0 : end, groups, mine);
}

// Tiles of an item (one at least: rows without tokens get their zeros) and blocks of a head.
__device__ __forceinline__ int item_tiles(const Sequence &s) { return s.len > 0 ? (s.len + TILE - 1) / TILE : 1; }
__device__ __forceinline__ int item_blocks(const AttentionArgs &a, const Sequence &s, int rows) {
  return (s.nq * a.group + rows - 1) / rows;
}
__device__ __forceinline__ int64_t sequence_work(const AttentionArgs &a, int b, int rows) {
  const Sequence s = sequence_of(a, b);
  return (int64_t)item_blocks(a, s, rows) * a.cache.heads * item_tiles(s);
}

// All of these are computed by a whole wave, with the same result in every lane.
__device__ __forceinline__ int64_t wave_sum(int64_t v) {
#pragma unroll
  for (int d = 32; d > 0; d /= 2) v += __shfl_xor(v, d);
  return v;
}
__device__ __forceinline__ int64_t wave_prefix(int64_t v, int lane) {  // inclusive
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int64_t u = __shfl_up(v, d);
    if (lane >= d) v += u;
  }
  return v;
}

// Pairs of neighbouring dimensions of CNT codes as bf16.  The conversions take the scale from the exponent field of
// an fp32; 0xFF there makes NaN of every code (checked on gfx950 for all of them).
template <int FMT, int CNT>
__device__ __forceinline__ void widen(unsigned *o, const unsigned *c, unsigned scale_byte) {
  const float sc = scale_operand(scale_byte);
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

// N bytes at p (aligned to the largest power of two up to 16 that divides N) into words
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

// Sum of a packed bf16 pair onto c.
__device__ __forceinline__ float add_pair(unsigned pair, float c) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, pair), __builtin_bit_cast(bf16x2, 0x3F803F80u), c,
                                         false);
}

// Maximum and sum with lane ^ 32, and with lane ^ 16.
__device__ __forceinline__ float max_halves(float v) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ __forceinline__ float sum_halves(float v) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}
__device__ __forceinline__ float max_rows16(float v) {
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ __forceinline__ float sum_rows16(float v) {
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

// Which of N (up to 32) tokens from j0 (the first one's place among the sequence's new tokens, negative before them)
// a new token sees: bit i for place j0 + i.
template <int N>
__device__ __forceinline__ unsigned seen_bits(const AttentionArgs &a, int query, int node, int j0) {
  constexpr unsigned ALL = 0xFFFFFFFFu >> (32 - N);
  if (j0 <= -N) return ALL;
  if (a.tree == nullptr) {
    const int count = node + 1 - j0;
    return count >= N ? ALL : count <= 0 ? 0u : (1u << count) - 1u;
  }
  const int64_t *words = a.tree + (int64_t)query * a.tree_words;
  const int at = j0 < 0 ? 0 : j0, i0 = at / 64, last = a.tree_words - 1;
  uint64_t w0 = words[i0 < last ? i0 : last], w1 = words[i0 < last ? i0 + 1 : last];  // one wait for both
  if (i0 > last) w0 = 0;
  if (i0 + 1 > last) w1 = 0;
  uint64_t bits = w0 >> (at % 64);
  if (at % 64) bits |= w1 << (64 - at % 64);
  return (j0 < 0 ? ((unsigned)(bits << -j0) | ((1u << -j0) - 1u)) : (unsigned)bits) & ALL;
}

// Bits of the first n of N tokens.
template <int N>
__device__ __forceinline__ unsigned first_bits(int n) {
  constexpr unsigned ALL = 0xFFFFFFFFu >> (32 - N);
  return n >= N ? ALL : n <= 0 ? 0u : (1u << n) - 1u;
}

// The maximum that weights refer to may lag behind the scores' by this many powers of two before the sums are
// rescaled: weights stay below 2^8, and most tiles need no rescaling.
constexpr float LAG = 8.0f;

// Sums times f.  ACC: they are in accumulation registers, which the vector units do not reach, and are moved for this
// here and nowhere else (left to itself the compiler moves them in every tile, for the branch's sake).
template <bool ACC, typename V>
__device__ __forceinline__ void rescale(V &o, float f) {
  if (ACC) asm volatile("" : "+a"(o));
  o *= f;
  if (ACC) asm volatile("" : "+a"(o));
}

// Which sums of exponentials give a result (none: the row saw nothing) and its reciprocal; NaN stays NaN.
__device__ __forceinline__ float reciprocal(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }

// The workspace: D sums for each row of a slot, the slots' maxima and sums, and the records.
__device__ __forceinline__ float *part_sums(const AttentionArgs &a, const Division &d, int64_t slot, int dim) {
  return a.partial + slot * d.rows * dim;
}
__device__ __forceinline__ float *part_stats(const AttentionArgs &a, const Division &d, int64_t slot, int dim) {
  return a.partial + 2 * (int64_t)d.workers * d.rows * dim + slot * d.rows * 2;
}

__device__ __forceinline__ Record *records_of(const AttentionArgs &a, const Division &d) {
  return (Record *)(a.partial + 2 * (int64_t)d.workers * d.rows * (a.cache.dim + 2));
}

// A worker's run, piece by piece.
struct Pieces {
  // the piece: tiles t0 .. t1 of the item's `tiles`, and the slot for a part
  Sequence s;
  int b, head, block, t0, t1, tiles, slot;
  // the run
  int64_t at, end, in, per;  // of the work; in: of the sequence

  __device__ __forceinline__ Pieces(const AttentionArgs &a, const Division &d) {
    if (d.workers == 0) {  // one item: the run is found without the others' work
      const int item = blockIdx.x;
      const int heads = a.cache.heads;
      b = item / d.blocks / heads;
      s = uniform(sequence_of(a, b));
      const int blocks = item_blocks(a, s, d.rows), tiles = item_tiles(s);
      in = ((int64_t)(item / d.blocks % heads) * blocks + item % d.blocks) * tiles;
      at = 0;
      end = per = item % d.blocks < blocks ? tiles : 0;
    } else {
      const int lane = threadIdx.x % 64;
      int64_t work = lane < a.batch ? sequence_work(a, lane, d.rows) : 0;
      const int64_t upto = wave_prefix(work, lane);
      int64_t total = __shfl(upto, 63);
      for (int b0 = 64; b0 < a.batch; b0 += 64)
        total += wave_sum(b0 + lane < a.batch ? sequence_work(a, b0 + lane, d.rows) : 0);
      total = uniform(total);
      per = (total + d.workers - 1) / d.workers;
      per = per < d.min_tiles ? d.min_tiles : per;
      at = blockIdx.x * per;
      end = at + per < total ? at + per : total;
      if (at >= end) return;
      // the sequence in which the run starts
      int64_t base = 0, end_of = upto;
      for (int b0 = 0;; b0 += 64) {
        const uint64_t hit = __builtin_amdgcn_ballot_w64(at >= end_of - work && at < end_of);
        if (hit) {
          const int l = __builtin_ctzll(hit);
          b = uniform(b0 + l);
          in = at - uniform(__shfl(end_of - work, l));
          break;
        }
        base = __shfl(end_of, 63);
        work = b0 + 64 + lane < a.batch ? sequence_work(a, b0 + 64 + lane, d.rows) : 0;
        end_of = base + wave_prefix(work, lane);
      }
    }
  }
  __device__ __forceinline__ bool next(const AttentionArgs &a, const Division &d) {
    if (at >= end) return false;
    int item, blocks;
    for (;; ++b, in = 0) {  // to the next sequence that has rows
      s = uniform(sequence_of(a, b));
      tiles = item_tiles(s);
      blocks = item_blocks(a, s, d.rows);
      item = uniform((int)(in / tiles));
      if (item < blocks * a.cache.heads) break;
    }
    head = item / blocks;
    block = item % blocks;
    t0 = uniform((int)(in - (int64_t)item * tiles));
    t1 = uniform(end - at < tiles - t0 ? t0 + (int)(end - at) : tiles);
    slot = t0 > 0 ? 0 : 1;
    if (slot && d.workers && threadIdx.x == 0) {
      // who has the rest: read by k_join
      const Record r{(int)blockIdx.x, (int)((at + tiles - 1) / per), b, head * d.blocks + block};
      records_of(a, d)[d.by_worker ? blockIdx.x : (int64_t)b * a.cache.heads * d.blocks + r.part] = r;
    }
    at += t1 - t0;
    in += t1 - t0;
    return true;
  }
  // After the last piece: a worker's record where no item began.
  __device__ __forceinline__ void finish(const AttentionArgs &a, const Division &d) {
    if (d.by_worker && d.workers && (at == blockIdx.x * per || slot == 0) && threadIdx.x == 0)
      records_of(a, d)[blockIdx.x] = Record{(int)blockIdx.x, (int)blockIdx.x, 0, 0};
  }
};

// Values that are not finite, of tokens that some rows see and others do not, are left out of the products; afterwards
// they are added to their dimensions' sums in the rows that see them (a weight is above zero, so NaN and infinities of
// either sign come out as if they had been in the products).  For a row (query `query`, place `node` among the new
// tokens) and the tokens from .. to of its sequence: not_finite(codes, scales, row of the head's page) is asked for
// every token that the row sees.
template <typename Ask>
__device__ __forceinline__ void seen_tokens(const AttentionArgs &a, const int *table, int head, int query, int node,
                                            int first_new, int from, int to, Ask ask) {
  const CacheView &cv = a.cache;
#pragma unroll 1
  for (int tok = from; tok < to; ++tok) {
    const unsigned page = (unsigned)table[tok >> cv.page_log2];
    if (page >= (uint64_t)cv.pages || !(seen_bits<1>(a, query, node, tok - first_new) & 1u)) continue;
    ask((int64_t)page * cv.heads + head, tok & ((1 << cv.page_log2) - 1));
  }
}

// 1 in bit 0 and bit 16 for the values of a packed pair that are not finite (all ones in the exponent carry into the
// sign's place).
__device__ __forceinline__ unsigned not_finite(unsigned pair) {
  return (((pair & 0x7F807F80u) + 0x00800080u) >> 15) & 0x00010001u;
}

// The low or high half of a packed pair as fp32 if it is not finite, zero otherwise.
__device__ __forceinline__ float not_finite_or_zero(unsigned pair, int high) {
  const unsigned v = high ? pair & 0xFFFF0000u : pair << 16;
  return (v & 0x7F800000u) == 0x7F800000u ? __uint_as_float(v) : 0.0f;
}

// Takes values that are not finite out of N packed pairs; non-zero if there were any.
template <int N>
__device__ __forceinline__ unsigned clear_not_finite(unsigned *w) {
  unsigned any = 0u;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const unsigned bad = not_finite(w[i]);
    w[i] &= ~((bad << 16) - bad);
    any |= bad;
  }
  return any;
}

// Workgroups of the few-rows kernel that a CU holds at once (waves of a SIMD): what its registers allow.
constexpr int rows_held(int dim, int nt) { return nt > 1 || dim > 128 ? 1 : dim <= 64 ? 3 : 2; }

// ---- host ----

// More than 64 KiB of LDS for a kernel, asked for once on each device (`done`: a bit for each).
inline hipError_t allow_lds(const void *kernel, int bytes, std::atomic<uint64_t> &done) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = (uint64_t)1 << (dev & 63);
  if (done.load(std::memory_order_relaxed) & bit) return hipSuccess;
  e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

Division attention_division_rows(int dim, int heads, int group, int batch, int64_t max_q, int64_t max_kv);
Division attention_division_tiles(int dim, int heads, int group, int batch, int64_t max_q, int64_t max_kv);
hipError_t launch_attention_rows(const AttentionArgs &a, const Division &d, hipStream_t stream);
hipError_t launch_attention_tiles(const AttentionArgs &a, const Division &d, hipStream_t stream);

}  // namespace mx
