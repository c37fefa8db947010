// Attention over the paged MX cache: choice of the kernel, division of the
// work, and the kernel that joins the pieces of divided items.
#include "attention.h"

namespace mx {

// Joins the pieces of items: out = sum_s 2^(m_s - m) o_s / sum_s 2^(m_s - m) l_s, in the order of the workers.
//
// A lane has four dimensions of a row, so that its pieces come in loads of 16 bytes, and a wave several rows side by side;
// a workgroup of four waves has join_rows() rows of an item, P of them for each lane, all of whose first loads are under
// way together.  (A wave with one row at a time, its lanes two dimensions apart: 29 us against 14 for 248 items of 256
// rows, heads of 128, in two or three pieces.)
constexpr int join_side(int dim) { return 64 / (dim / 4); }  // rows of a wave's pass
constexpr int join_rows(int dim, int passes) { return 4 * passes * join_side(dim); }

template <int D, bool BY_WORKER, int P>
__global__ __launch_bounds__(256) void k_join(AttentionArgs a, Division dv, int row_groups) {
  constexpr int LANES = D / 4, SIDE = join_side(D);
  const int wave = uniform((int)threadIdx.x / 64), lane = threadIdx.x % 64;
  const int at = blockIdx.x / row_groups, row0 = (blockIdx.x - at * row_groups) * join_rows(D, P);
  const Record rec = records_of(a, dv)[at];
  // the item's record is where it belongs, so its sequence is read without waiting for it
  const int item = BY_WORKER ? uniform(rec.part) : at;
  const int block = item % dv.blocks, head = item / dv.blocks % a.cache.heads;
  const int b = BY_WORKER ? uniform(rec.b) : item / dv.blocks / a.cache.heads;
  const Sequence s = uniform(sequence_of(a, b));
  const int rows = s.nq * a.group - block * dv.rows;  // of this block, if not more than it holds
  if (row0 >= rows) return;                           // (also for items that are not there, whose workers are not set)
  const int w0 = uniform(rec.first), w1 = uniform(rec.last);
  if (w0 == w1) return;  // one worker had all of it and has written the result
  const int last = rows < dv.rows ? rows : dv.rows;
  const int side = lane / LANES, d = 4 * (lane - side * LANES);
  auto slot = [&](int w) { return 2 * (int64_t)w + (w == w0); };
  int r[P];
  float m[P], l[P];
  f32x4 acc[P];
  if (side >= SIDE) return;  // lanes behind the last whole row
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int row = row0 + (4 * p + wave) * SIDE + side;
    r[p] = row < last ? row : last - 1;  // (not written)
    m[p] = -__builtin_inff();
    l[p] = 0.0f;
    acc[p] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  if (row0 + wave * SIDE >= last) return;
  for (int w = w0; w <= w1; ++w) {
    const float *ml = part_stats(a, dv, slot(w), D);
#pragma unroll
    for (int p = 0; p < P; ++p) m[p] = fmaxf(m[p], ml[2 * r[p]]);
  }
#pragma unroll 4 / P
  for (int w = w0; w <= w1; ++w) {
    const float *ml = part_stats(a, dv, slot(w), D), *o = part_sums(a, dv, slot(w), D) + d;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const f32x4 v = *(const f32x4 *)(o + (int64_t)r[p] * D);
      const float f = __builtin_amdgcn_exp2f(ml[2 * r[p]] - (m[p] == -__builtin_inff() ? 0.0f : m[p]));
      l[p] += f * ml[2 * r[p] + 1];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[p][i] += f * v[i];
    }
  }
#pragma unroll
  for (int p = 0; p < P; ++p) {
    if (row0 + (4 * p + wave) * SIDE + side >= last) continue;
    const int row = block * dv.rows + r[p], node = row / a.group;
    unsigned short *out = a.out + ((int64_t)(s.q0 + node) * a.cache.heads * a.group + head * a.group + row -
                                   node * a.group) * D + d;
    const float inv = reciprocal(l[p]);
    *(u32x2 *)out = u32x2{bf16x2_rne(acc[p][0] * inv, acc[p][1] * inv), bf16x2_rne(acc[p][2] * inv, acc[p][3] * inv)};
  }
}

// The same for a row of few items with many pieces: sixteen waves share it.
template <int D>
__global__ __launch_bounds__(1024) void k_join_wide(AttentionArgs a, Division dv, int row_groups) {
  constexpr int WAVES = 16, N = (D + 63) / 64;
  __shared__ float waves[WAVES][D + 2];
  const int wave = uniform((int)threadIdx.x / 64), lane = threadIdx.x % 64;
  const int item = blockIdx.x / row_groups, r = blockIdx.x - item * row_groups;
  const Record rec = records_of(a, dv)[item];
  const int block = item % dv.blocks, head = item / dv.blocks % a.cache.heads;
  const Sequence s = uniform(sequence_of(a, item / dv.blocks / a.cache.heads));
  const int rows = s.nq * a.group - block * dv.rows;
  if (r >= rows) return;
  const int w0 = uniform(rec.first), w1 = uniform(rec.last);
  if (w0 == w1) return;
  if (r >= dv.rows) return;
  float m = -__builtin_inff(), l = 0.0f, acc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.0f;
  auto slot = [&](int w) { return 2 * (int64_t)w + (w == w0); };
  for (int w = w0 + wave; w <= w1; w += WAVES) m = fmaxf(m, part_stats(a, dv, slot(w), D)[2 * r]);
  const float base = m == -__builtin_inff() ? 0.0f : m;
#pragma unroll 4
  for (int w = w0 + wave; w <= w1; w += WAVES) {
    const float *ml = part_stats(a, dv, slot(w), D) + 2 * r, *o = part_sums(a, dv, slot(w), D) + (int64_t)r * D;
    const float f = __builtin_amdgcn_exp2f(ml[0] - base);
    l += f * ml[1];
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (D % 64 == 0 || 64 * i + lane < D) acc[i] += f * o[64 * i + lane];
  }
  const int row = block * dv.rows + r, node = row / a.group;
  unsigned short *out = a.out + ((int64_t)(s.q0 + node) * a.cache.heads * a.group + head * a.group + row -
                                 node * a.group) * D;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (D % 64 == 0 || 64 * i + lane < D) waves[wave][64 * i + lane] = acc[i];
  if (lane == 0) waves[wave][D] = m, waves[wave][D + 1] = l;
  __syncthreads();
  if (threadIdx.x < D) {
    float top = -__builtin_inff(), sum = 0.0f, v = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) top = fmaxf(top, waves[w][D]);
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      // a wave without a maximum has sums of zero, or NaN, which has to stay
      const float f = waves[w][D] == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(waves[w][D] - top);
      sum += f * waves[w][D + 1];
      v += f * waves[w][threadIdx.x];
    }
    out[threadIdx.x] = (unsigned short)bf16x2_rne(v * reciprocal(sum), 0.0f);
  }
}

// The few-rows kernel as far as its registers go: a row more and a tile's conversion serves 128.
static Division division_of(int dim, int heads, int group, int batch, int64_t max_q, int64_t max_kv, bool all,
                            bool *tiled) {
  *tiled = max_q * group > (dim > 128 ? 16 : 32);
  return *tiled ? attention_division_tiles(dim, heads, group, batch, max_q, max_kv, all)
                : attention_division_rows(dim, heads, group, batch, max_q, max_kv, all);
}

int64_t attention_workspace(int fmt, int dim, int heads, int group, int batch, int64_t total_q, int64_t max_q,
                            int64_t max_kv, bool all) {
  if (batch == 0 || total_q == 0 || max_q == 0) return 0;
  bool tiled;
  const Division d = division_of(dim, heads, group, batch, max_q, max_kv, all, &tiled);
  if (d.workers == 0) return 0;
  return 2 * (int64_t)d.workers * d.rows * (dim + 2) * 4 + (int64_t)d.records * (int64_t)sizeof(Record);
}

template <int D>
static hipError_t join(const AttentionArgs &a, const Division &d, hipStream_t stream) {
  const int most = a.max_q * a.group < d.rows ? a.max_q * a.group : d.rows;  // rows of a block
  // eight pieces or more of every item on the average and few rows: one row for sixteen waves
  if (d.workers / d.records >= 8 && d.records * most <= 2 * device_cu_count()) {
    k_join_wide<D><<<d.records * most, 1024, 0, stream>>>(a, d, most);
  } else {
    // Two passes of rows a wave, but one for the few rows of single tokens and small trees, whose loads are spread over more
    // workgroups so (heads of 128: 64 sequences of one token, 4 rows each, 6.0 us and 6.7 with two; blocks of 256 rows 11.6
    // and 10.6).
    const int passes = most <= 32 ? 1 : 2;
    const int groups = (most + join_rows(D, passes) - 1) / join_rows(D, passes), grid = d.records * groups;
    if (passes == 1) {
      if (d.by_worker) k_join<D, true, 1><<<grid, 256, 0, stream>>>(a, d, groups);
      else k_join<D, false, 1><<<grid, 256, 0, stream>>>(a, d, groups);
    } else {
      if (d.by_worker) k_join<D, true, 2><<<grid, 256, 0, stream>>>(a, d, groups);
      else k_join<D, false, 2><<<grid, 256, 0, stream>>>(a, d, groups);
    }
  }
  return hipGetLastError();
}

__global__ __launch_bounds__(256) void k_zero_padding(AttentionArgs a) {
  zero_rows(a, 0, gridDim.x, blockIdx.x);
}

hipError_t launch_cache_attention(const AttentionArgs &a, hipStream_t stream) {
  if (a.batch == 0 || a.max_q == 0) {  // no sequence has queries
    k_zero_padding<<<4 * device_cu_count(), 256, 0, stream>>>(a);
    return hipGetLastError();
  }
  bool tiled;
  const Division d =
      division_of(a.cache.dim, a.cache.heads, a.group, a.batch, a.max_q, a.max_kv, a.all, &tiled);
  const hipError_t e = tiled ? launch_attention_tiles(a, d, stream) : launch_attention_rows(a, d, stream);
  if (e != hipSuccess || d.workers == 0) return e;
  switch (a.cache.dim) {
    case 64: return join<64>(a, d, stream);
    case 96: return join<96>(a, d, stream);
    case 128: return join<128>(a, d, stream);
    case 192: return join<192>(a, d, stream);
    case 256: return join<256>(a, d, stream);
    default: return hipErrorInvalidValue;
  }
}

constexpr int WHOLE_TILES = 64;  // up to which items are not divided where queries see all tokens

// The division for a kernel of `rows` rows a block, with this many workers as long as they have runs of min_tiles.
static Division divide(int rows, int64_t workers, int min_tiles, int heads, int group, int batch, int64_t max_q,
                       int64_t max_kv, bool all, int64_t held, int cost) {
  Division d;
  d.rows = rows;
  d.min_tiles = min_tiles;
  d.blocks = (int)((max_q * group + rows - 1) / rows);
  d.tiles = (int)(max_kv > 0 ? (max_kv + TILE - 1) / TILE : 1);
  const int64_t items = (int64_t)batch * heads * d.blocks;
  const double most = __builtin_ceil((double)items * d.tiles / min_tiles);
  // a launch has fewer than 2^32 threads: with too many items of up to 512 the work is divided all the same
  // Where all of a sequence's tokens are seen (states of an encoder, a few thousand as a rule) items are alike, and what a
  // division costs, `cost` tiles of a workgroup, is often more than the rounds of whole items lose.  (256 items of 224
  // rows, heads of 64: 44 us undivided and 58 divided for 1500 tokens, 80 and 91 for 3000; 64 such items 41 and 34, 73
  // and 47.)  Up to 4096 tokens: one long sequence may be among short ones.
  //
  // Items of few rows are so never divided up to 2048 tokens, whatever the heads.  Single tokens in MXFP8, us a call whole
  // and divided (all are whole up to 2048):
  //   tokens                                512       1024       1500       2048
  //   512 items of 1 row, heads of 64    11 / 18    16 / 29    21 / 29    25 / 38
  //   512 items of 4, 128                17 / 25    26 / 35    36 / 46    45 / 54
  //   512 items of 4, 256                36 / 37    56 / 57    93 / 93   110 / 110
  //   64 items of 4, 128                 10 / 14    14 / 14    20 / 17    25 / 15
  //   8 items of 4, 256                  14 / 16    21 / 16    30 / 20    33 / 16
  // Few items with large heads lose by it: a tile's time grows with the head, the cost here does not.
  const int64_t rounds = (items + held - 1) / held;
  const bool whole = all && d.tiles <= WHOLE_TILES && (rounds * held - items) * d.tiles <= cost * held;
  d.workers = (d.tiles <= min_tiles || whole) && items < ((int64_t)1 << 32) / 512
                  ? 0
                  : (int)((double)workers < most ? workers : (int64_t)most);
  d.by_worker = items > d.workers;
  d.records = d.by_worker ? d.workers : (int)items;
  return d;
}

Division attention_division_rows(int dim, int heads, int group, int batch, int64_t max_q, int64_t max_kv, bool all) {
  const int rows = max_q * group <= 16 ? 16 : 32;
  // One run for every workgroup that the CUs hold at once (rows_held); of several sequences,
  // whose lengths differ as a rule, two, so that a CU that has finished early takes another: 64 ragged sequences in
  // MXFP8 224 us against 235 with one run each, 64 equal ones 384 against 381, one of 500000 tokens 129 against 120.
  const int64_t held = rows_held(dim, rows / 16) * (int64_t)device_cu_count();
  return divide(rows, batch > 1 ? 2 * held : held, 4, heads, group, batch, max_q, max_kv, all, held, 32);
}

Division attention_division_tiles(int dim, int heads, int group, int batch, int64_t max_q, int64_t max_kv, bool all) {
  // More rows share a tile's conversion in blocks of 256 (the 512 rows of 8192 tokens: 184 us against 196 in blocks of
  // 128), for which heads of more than 128 dimensions have no registers.  One workgroup for every CU, or two of the
  // small ones (64 rows over 32768 tokens: 201 us against 309 with one), in runs of eight tiles at least: a piece costs
  // as much as seven of them (512 tokens 30 us against 45 in runs of two tiles).
  // Whole items are better smaller: 320 of up to 224 rows, heads of 64, 1500 tokens 63 us and 84 in blocks of 256; 96 of
  // 800, 128, 1500 tokens 95 and 112.  So are most of those that are divided after all, but not all (32 of 2800, 128, 4000
  // tokens 226 and 214).
  const bool small = all && max_kv <= WHOLE_TILES * TILE;
  const int rows = max_q * group <= 128 || dim > 128 || small ? 128 : 256;
  const int two = rows == 128 && dim <= 128;
  const int64_t held = (1 + two) * (int64_t)device_cu_count();
  return divide(rows, held, 8, heads, group, batch, max_q, max_kv, all, held, two ? 20 : 13);
}

}  // namespace mx
