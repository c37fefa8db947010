// Attention over the paged MX cache: choice of the kernel, division of the
// work, and the kernel that joins the pieces of divided items.
#include "attention.h"

namespace mx {

// Joins the pieces of a row: out = sum_s 2^(m_s - m) o_s / sum_s 2^(m_s - m) l_s.  A workgroup of WAVES waves takes a
// row (the waves take pieces in turn) and finds its pieces from the same division as the workers.
template <int D, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_join(AttentionArgs a, Division dv) {
  __shared__ float part[WAVES][D + 2];
  const int wave = uniform(threadIdx.x / 64), lane = threadIdx.x % 64;
  const int heads = a.cache.heads * a.group;
  const int64_t at = blockIdx.x;
  const int token = (int)(at / heads), qh = (int)(at - (int64_t)token * heads);
  int b = 0, past = a.batch;  // the sequence of the token: the last that starts at or before it
  while (past - b > 1) {
    const int mid = (b + past) / 2;
    if (a.q_starts[mid] <= token) b = mid; else past = mid;
  }
  const Sequence s = sequence_of(a, b);
  const int node = token - s.q0;
  if (node < 0 || node >= s.nq) return;
  const int64_t per = run_tiles(dv, total_work(a, dv.rows));
  const int tiles = item_tiles(s), blocks = item_blocks(a, s, dv.rows);
  const int head = qh / a.group, row = node * a.group + qh - head * a.group;
  const int64_t begin = find_place(a, dv.rows, 0, b).first + ((int64_t)head * blocks + row / dv.rows) * tiles;
  const int w0 = (int)(begin / per), w1 = (int)((begin + tiles - 1) / per);
  if (w0 == w1) return;  // one worker had all of it and has written the result
  const int r = row % dv.rows;
  constexpr int N = (D + 63) / 64;
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
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (D % 64 == 0 || 64 * i + lane < D) part[wave][64 * i + lane] = acc[i];
  if (lane == 0) part[wave][D] = m, part[wave][D + 1] = l;
  __syncthreads();
  for (int d = threadIdx.x; d < D; d += 64 * WAVES) {
    float top = -__builtin_inff(), sum = 0.0f, v = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) top = fmaxf(top, part[w][D]);
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      // a wave without a maximum has sums of zero, or NaN, which has to stay
      const float f = part[w][D] == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(part[w][D] - top);
      sum += f * part[w][D + 1];
      v += f * part[w][d];
    }
    a.out[at * D + d] = (unsigned short)bf16x2_rne(v * reciprocal(sum), 0.0f);
  }
}

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
  return 2 * (int64_t)d.workers * d.rows * (dim + 2) * 4;
}

template <int D>
static hipError_t join(const AttentionArgs &a, const Division &d, hipStream_t stream) {
  const unsigned rows = (unsigned)((int64_t)a.total_q * a.cache.heads * a.group);
  // the more pieces a row can have, the more waves share them
  const int64_t items = (int64_t)a.batch * a.cache.heads * d.blocks;
  if (d.workers / items > 16) k_join<D, 16><<<rows, 1024, 0, stream>>>(a, d);
  else if (d.workers / items > 4) k_join<D, 4><<<rows, 256, 0, stream>>>(a, d);
  else k_join<D, 1><<<rows, 64, 0, stream>>>(a, d);
  return hipGetLastError();
}

hipError_t launch_cache_attention(const AttentionArgs &a, hipStream_t stream) {
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
  d.workers = d.tiles <= min_tiles && items <= INT32_MAX ? 0 : (int)((double)workers < most ? workers : (int64_t)most);
  return d;
}

Division attention_division_rows(int dim, int heads, int group, int batch, int64_t max_q, int64_t max_kv) {
  return divide(max_q * group <= 16 ? 16 : 32, 4 * (int64_t)device_cu_count(), 4, heads, group, batch, max_q, max_kv);
}

Division attention_division_tiles(int dim, int heads, int group, int batch, int64_t max_q, int64_t max_kv) {
  const int rows = max_q * group <= 128 ? 128 : 256;
  return divide(rows, (int64_t)device_cu_count(), 2, heads, group, batch, max_q, max_kv);
}

}  // namespace mx
