// Attention over the paged MX cache: choice of the kernel, division of the
// work, and the kernel that joins the pieces of divided items.
#include "attention.h"

namespace mx {

// Joins the pieces of items: out = sum_s 2^(m_s - m) o_s / sum_s 2^(m_s - m) l_s.  A workgroup of four waves (sixteen
// if WIDE) has ROWS rows of an item; WIDE: all waves share one row, as a row of few items has many pieces.
constexpr int JOIN_ROWS = 4;

template <int D, bool WIDE, bool BY_WORKER>
__global__ __launch_bounds__(WIDE ? 1024 : 256) void k_join(AttentionArgs a, Division dv, int row_groups) {
  constexpr int WAVES = WIDE ? 16 : 4;
  __shared__ float waves[WIDE ? WAVES : 1][D + 2];
  const int wave = uniform((int)threadIdx.x / 64), lane = threadIdx.x % 64;
  const int at = blockIdx.x / row_groups, row0 = (blockIdx.x - at * row_groups) * (WIDE ? 1 : JOIN_ROWS);
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
  constexpr int N = (D + 63) / 64;
  const int last = rows < dv.rows ? rows : dv.rows;
  for (int r = row0 + (WIDE ? 0 : wave); r < last && r < row0 + (WIDE ? 1 : JOIN_ROWS); r += WIDE ? 1 : WAVES) {
    float m = -__builtin_inff(), l = 0.0f, acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.0f;
    auto slot = [&](int w) { return 2 * (int64_t)w + (w == w0); };
    const int step = WIDE ? WAVES : 1;
    for (int w = w0 + (WIDE ? wave : 0); w <= w1; w += step) m = fmaxf(m, part_stats(a, dv, slot(w), D)[2 * r]);
    const float base = m == -__builtin_inff() ? 0.0f : m;
#pragma unroll 4
    for (int w = w0 + (WIDE ? wave : 0); w <= w1; w += step) {
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
    if (!WIDE) {
      const float inv = reciprocal(l);
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (D % 64 == 0 || 64 * i + lane < D) out[64 * i + lane] = (unsigned short)bf16x2_rne(acc[i] * inv, 0.0f);
      continue;
    }
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
}

// The few-rows kernel as far as its registers go: a row more and a tile's conversion serves 128.
static Division division_of(int dim, int heads, int group, int batch, int64_t max_q, int64_t max_kv, bool *tiled) {
  *tiled = max_q * group > (dim > 128 ? 16 : 32);
  return *tiled ? attention_division_tiles(dim, heads, group, batch, max_q, max_kv)
                : attention_division_rows(dim, heads, group, batch, max_q, max_kv);
}

int64_t attention_workspace(int fmt, int dim, int heads, int group, int batch, int64_t total_q, int64_t max_q,
                            int64_t max_kv) {
  if (batch == 0 || total_q == 0 || max_q == 0) return 0;
  bool tiled;
  const Division d = division_of(dim, heads, group, batch, max_q, max_kv, &tiled);
  if (d.workers == 0) return 0;
  return 2 * (int64_t)d.workers * d.rows * (dim + 2) * 4 + (int64_t)d.records * (int64_t)sizeof(Record);
}

template <int D>
static hipError_t join(const AttentionArgs &a, const Division &d, hipStream_t stream) {
  const int most = a.max_q * a.group < d.rows ? a.max_q * a.group : d.rows;  // rows of a block
  // eight pieces or more of every item on the average and few rows: one row for sixteen waves
  if (d.workers / d.records >= 8 && d.records * most <= 2 * device_cu_count()) {
    k_join<D, true, false><<<d.records * most, 1024, 0, stream>>>(a, d, most);
  } else {
    const int groups = (most + JOIN_ROWS - 1) / JOIN_ROWS;
    if (d.by_worker) k_join<D, false, true><<<d.records * groups, 256, 0, stream>>>(a, d, groups);
    else k_join<D, false, false><<<d.records * groups, 256, 0, stream>>>(a, d, groups);
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
      division_of(a.cache.dim, a.cache.heads, a.group, a.batch, a.max_q, a.max_kv, &tiled);
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

// The division for a kernel of `rows` rows a block, with this many workers as long as they have runs of min_tiles.
static Division divide(int rows, int64_t workers, int min_tiles, int heads, int group, int batch, int64_t max_q,
                       int64_t max_kv) {
  Division d;
  d.rows = rows;
  d.min_tiles = min_tiles;
  d.blocks = (int)((max_q * group + rows - 1) / rows);
  d.tiles = (int)(max_kv > 0 ? (max_kv + TILE - 1) / TILE : 1);
  const int64_t items = (int64_t)batch * heads * d.blocks;
  const double most = __builtin_ceil((double)items * d.tiles / min_tiles);
  // a launch has fewer than 2^32 threads: with too many items of up to 512 the work is divided all the same
  d.workers = d.tiles <= min_tiles && items < ((int64_t)1 << 32) / 512
                  ? 0
                  : (int)((double)workers < most ? workers : (int64_t)most);
  d.by_worker = items > d.workers;
  d.records = d.by_worker ? d.workers : (int)items;
  return d;
}

Division attention_division_rows(int dim, int heads, int group, int batch, int64_t max_q, int64_t max_kv) {
  const int rows = max_q * group <= 16 ? 16 : 32;
  // One run for every workgroup that the CUs hold at once (rows_held); of several sequences,
  // whose lengths differ as a rule, two, so that a CU that has finished early takes another: 64 ragged sequences in
  // MXFP8 224 us against 235 with one run each, 64 equal ones 384 against 381, one of 500000 tokens 129 against 120.
  const int64_t held = rows_held(dim, rows / 16) * (int64_t)device_cu_count();
  return divide(rows, batch > 1 ? 2 * held : held, 4, heads, group, batch, max_q, max_kv);
}

Division attention_division_tiles(int dim, int heads, int group, int batch, int64_t max_q, int64_t max_kv) {
  // More rows share a tile's conversion in blocks of 256 (the 512 rows of 8192 tokens: 184 us against 196 in blocks of
  // 128), for which heads of more than 128 dimensions have no registers.  One workgroup for every CU, or two of the
  // small ones (64 rows over 32768 tokens: 201 us against 309 with one), in runs of eight tiles at least: a piece costs
  // as much as seven of them (512 tokens 30 us against 45 in runs of two tiles).
  const int rows = max_q * group <= 128 || dim > 128 ? 128 : 256;
  const int64_t held = (rows == 128 && dim <= 128 ? 2 : 1) * (int64_t)device_cu_count();
  return divide(rows, held, 8, heads, group, batch, max_q, max_kv);
}

}  // namespace mx
