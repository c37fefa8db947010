// The cache's pages: whole pages copied, sequences forked, pages taken and
// freed, and a sequence's tokens compacted to those that are kept.
//
// refs[page] counts the rows of tables that hold a page; a page is free while
// it is zero.  Free pages are handed out lowest first, in the order of the
// rows and columns that lack one, so that the same tables give the same pages.
//
//   resize   row r holds ceil(kv_lens[r] / page) pages: those behind them are
//            released first, in all rows, then missing ones are taken.
//   fork     a child row shares its parent's full pages and has the tokens of
//            the last page, if it is not full, in a page of its own.
//   compact  token i of what is kept comes from place keep[i] >= i.
//
// Bound: HBM for what is moved (each byte read and written once), latency for
// the tables: one small kernel for the rows, one workgroup that hands out
// pages.
#include "launch.h"

namespace mx {

namespace {

struct BookArgs {
  int *refs;
  const int *kv_lens, *parents;  // parents: of a fork
  const int *table;              // of a fork: the parents'
  int64_t stride, out_stride;
  int *out, *missing;
  int pages, page_log2, rows, cols, out_rows;
};

// What a row of the result holds: `keep` pages of the row it comes from, `need` in all.
struct Row {
  int from, keep, need;
};

template <bool FORK>
__device__ __forceinline__ Row row_of(const BookArgs &a, int r) {
  const int from = FORK ? a.parents[r] : r;
  int len = FORK && (unsigned)from >= (unsigned)a.rows ? 0 : a.kv_lens[from];
  len = len < 0 ? 0 : len;
  const int full = len >> a.page_log2, need = full + ((len & ((1 << a.page_log2) - 1)) != 0);
  return Row{from, FORK ? full : need, need};
}

// Entry `j` of row `r`, of which `was` is what the row that it comes from holds there: the page is released or shared.
// True if the row lacks a page there.
template <bool FORK>
__device__ __forceinline__ bool settle(const BookArgs &a, const Row &row, int r, int j, int was) {
  const bool held = (unsigned)was < (unsigned)a.pages;
  int *dst = a.out + (int64_t)r * a.out_stride + j;
  if (FORK) {
    if (held) atomicAdd(a.refs + was, 1);
    *dst = held ? was : -1;
    return j < row.need && !held;
  }
  if (j < row.need) {
    if (!held && was != -1) *dst = -1;
    return !held;
  }
  // (a page that nobody holds stays free)
  if (held && atomicSub(a.refs + was, 1) <= 0) atomicAdd(a.refs + was, 1);
  if (was != -1) *dst = -1;
  return false;
}

template <bool FORK>
__device__ __forceinline__ int entry_of(const BookArgs &a, const Row &row, int j) {
  return FORK && j >= row.keep ? -1 : a.table[(int64_t)row.from * a.stride + j];
}

__device__ __forceinline__ int beyond(const BookArgs &a, const Row &row) {  // pages that the row has no column for
  return row.need > a.cols ? row.need - a.cols : 0;
}

// A wave has a row; missing[row] is what the row lacks.
template <bool FORK>
__global__ __launch_bounds__(256) void k_page_rows(BookArgs a) {
  const int r = blockIdx.x * 4 + threadIdx.x / 64, lane = threadIdx.x % 64;
  if (r >= a.out_rows) return;
  const Row row = row_of<FORK>(a, r);
  int lack = 0;
#pragma unroll 4
  for (int j = lane; j < a.cols; j += 64) lack += settle<FORK>(a, row, r, j, entry_of<FORK>(a, row, j));
#pragma unroll
  for (int d = 32; d > 0; d /= 2) lack += __shfl_xor(lack, d);
  if (lane == 0) a.missing[r] = lack + beyond(a, row);
}

constexpr int TAKE_THREADS = (int)TAKE_ROWS, TAKE_ITEMS = 4;  // entries of a table that a step of the workgroup looks at: 4096
constexpr int SCAN_ITEMS = 8, SKIP_ITEMS = 32;      // counts of holders: 8192, and 32768 where none is free
constexpr int queue_of(int items) { return TAKE_THREADS * (items + SCAN_ITEMS); }  // pages, for steps of so many items a thread

// The sum of v over the threads before this one, and over all of them (total).
__device__ __forceinline__ int block_prefix(int v, int *waves, int &total) {
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  int sum = v;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int u = __shfl_up(sum, d);
    if (lane >= d) sum += u;
  }
  __syncthreads();  // waves[] of the call before has been read
  if (lane == 63) waves[wave] = sum;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < TAKE_THREADS / 64; ++w) {
    before += w < wave ? waves[w] : 0;
    total += waves[w];
  }
  return before + sum - v;
}

// Free pages, found from the lowest on, for steps that want ITEMS for each thread at most.
template <int ITEMS>
struct FreePages {
  static constexpr int QUEUE = queue_of(ITEMS);
  int *queue;                          // in LDS
  int head = 0, size = 0, cursor = 0;  // of the queue; the first page that was not looked at

  // How many holders a page has: atomic, as the changes of this kernel are, which a barrier has put before it.
  static __device__ __forceinline__ int holders(const BookArgs &a, unsigned page) {
    return __hip_atomic_load(a.refs + page, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }

  // At least `wanted`, if there are so many.
  __device__ __forceinline__ void find(const BookArgs &a, int wanted, int *waves) {
    // the pool's low pages are taken as a rule: runs of them are passed over in large steps
    while (size == 0 && wanted > 0 && a.pages - cursor >= TAKE_THREADS * SKIP_ITEMS) {
      bool any = false;
#pragma unroll
      for (int k = 0; k < SKIP_ITEMS; ++k) any |= holders(a, (unsigned)cursor + k * TAKE_THREADS + threadIdx.x) == 0;
      if (__syncthreads_or(any)) break;
      cursor += TAKE_THREADS * SKIP_ITEMS;
    }
    while (size < wanted && cursor < a.pages) {
      int found = 0;
      unsigned free = 0;
      const unsigned p0 = (unsigned)cursor + threadIdx.x * SCAN_ITEMS;
#pragma unroll
      for (int k = 0; k < SCAN_ITEMS; ++k) {
        const unsigned p = p0 + k;
        const bool is = p < (unsigned)a.pages && holders(a, p) == 0;
        free |= (unsigned)is << k;
        found += is;
      }
      int all;
      int at = head + size + block_prefix(found, waves, all);
      for (; free; free &= free - 1, ++at) queue[at % QUEUE] = (int)(p0 + __builtin_ctz(free));
      size += all;
      cursor = cursor > a.pages - TAKE_THREADS * SCAN_ITEMS ? a.pages : cursor + TAKE_THREADS * SCAN_ITEMS;
    }
    __syncthreads();
  }
  // The page of this rank, or -1.
  __device__ __forceinline__ int operator[](int rank) const { return rank < size ? queue[(head + rank) % QUEUE] : -1; }
  __device__ __forceinline__ void drop(int count) {
    count = count < size ? count : size;
    head = (head + count) % QUEUE;
    size -= count;
    __syncthreads();  // the places that are free now are written by the next step
  }
};

// Small tables: one workgroup sees to the rows and hands out pages.  (64 rows of 256 entries take it 10 us where nothing
// is to be done, and two kernels 5; 64 rows of 63 entries 6 us.)
constexpr int SMALL_ROWS = 1024, SMALL_ITEMS = 4;  // rows; entries of a thread

template <bool FORK>
__global__ __launch_bounds__(TAKE_THREADS) void k_pages_small(BookArgs a) {
  __shared__ int waves[TAKE_THREADS / 64], queue[queue_of(1)], lacks[SMALL_ROWS];
  __shared__ Row rows[SMALL_ROWS];
  __shared__ unsigned any;  // OR of the threads' wants
  const int t = threadIdx.x, entries = a.out_rows * a.cols;
  if (t < a.out_rows) {
    rows[t] = row_of<FORK>(a, t);
    lacks[t] = 0;
  }
  if (t == 0) any = 0u;
  __syncthreads();
  unsigned wants = 0;  // bit k: this thread's entry k lacks a page
  int was[SMALL_ITEMS];
#pragma unroll
  for (int k = 0; k < SMALL_ITEMS; ++k) {
    const int e = k * TAKE_THREADS + t, r = e < entries ? e / a.cols : 0;
    was[k] = e < entries ? entry_of<FORK>(a, rows[r], e - r * a.cols) : -1;
  }
#pragma unroll
  for (int k = 0; k < SMALL_ITEMS; ++k) {
    const int e = k * TAKE_THREADS + t, r = e < entries ? e / a.cols : 0;
    if (e >= entries || !settle<FORK>(a, rows[r], r, e - r * a.cols, was[k])) continue;
    atomicAdd(lacks + r, 1);
    wants |= 1u << k;
  }
  FreePages<1> free{queue};
  if (FORK) {  // a page each for the rows whose last one is not full
    const bool want = t < a.out_rows && rows[t].keep < rows[t].need && rows[t].keep < a.cols;
    int total;
    const int rank = block_prefix(want, waves, total);
    free.find(a, total, waves);
    const int page = want ? free[rank] : -1;
    if (page >= 0) {
      a.out[t * a.out_stride + rows[t].keep] = page;
      a.refs[page] = 1;
    }
    if (t < a.out_rows) a.missing[t] = lacks[t] - (page >= 0) + beyond(a, rows[t]);
    return;
  }
  if (wants) atomicOr(&any, wants);
  __syncthreads();
  for (unsigned left = any; left; left &= left - 1) {  // in the order of the entries
    const int k = __builtin_ctz(left);
    const bool want = wants >> k & 1u;
    int total;
    const int rank = block_prefix(want, waves, total);
    free.find(a, total, waves);
    const int page = want ? free[rank] : -1;
    if (page >= 0) {
      const int e = k * TAKE_THREADS + t, r = e / a.cols;
      a.out[(int64_t)r * a.out_stride + (e - r * a.cols)] = page;
      a.refs[page] = 1;
      atomicSub(lacks + r, 1);
    }
    free.drop(total);
  }
  __syncthreads();
  if (t < a.out_rows) a.missing[t] = lacks[t] + beyond(a, rows[t]);
}

// Some row has a page behind one that it lacks: all entries are gone over.
__device__ __forceinline__ void take_holes(const BookArgs &a, FreePages<TAKE_ITEMS> &free, int *waves) {
  const int t = threadIdx.x;
  const int64_t entries = (int64_t)a.out_rows * a.cols;
  for (int64_t base = 0; base < entries; base += TAKE_THREADS * TAKE_ITEMS) {
    int *place[TAKE_ITEMS], *miss[TAKE_ITEMS];
    int wants = 0, total;
#pragma unroll
    for (int k = 0; k < TAKE_ITEMS; ++k) {
      const int64_t e = base + t * TAKE_ITEMS + k;
      place[k] = nullptr;
      if (e >= entries) continue;
      const int r = entries >> 32 ? (int)(e / a.cols) : (int)((unsigned)e / (unsigned)a.cols);
      miss[k] = a.missing + r;
      if (a.missing[r] == 0) continue;
      const Row row = row_of<false>(a, r);
      const int64_t j = e - (int64_t)r * a.cols;
      int *at = a.out + (int64_t)r * a.out_stride + j;
      if (j >= row.need || *at != -1) continue;
      place[k] = at;
      ++wants;
    }
    int rank = block_prefix(wants, waves, total);
    free.find(a, total, waves);
#pragma unroll
    for (int k = 0; k < TAKE_ITEMS; ++k) {
      if (place[k] == nullptr) continue;
      const int page = free[rank++];
      if (page < 0) continue;
      *place[k] = page;
      a.refs[page] = 1;
      atomicSub(miss[k], 1);
    }
    free.drop(total);
  }
}

// One workgroup hands out pages, to the entries that lack one in the order of rows and columns.  Of rows of a fork that is
// the one behind the full pages; of others as a rule the last ones that the row needs, which is looked at first.
template <bool FORK>
__global__ __launch_bounds__(TAKE_THREADS) void k_page_take(BookArgs a) {
  __shared__ int waves[TAKE_THREADS / 64], queue[queue_of(TAKE_ITEMS)];
  __shared__ int before[TAKE_THREADS + 1], end[TAKE_THREADS];  // of a step's rows: entries that lack a page, in sum; ends
  const int t = threadIdx.x;
  FreePages<TAKE_ITEMS> free{queue};

  // rows row0 .. row0 + TAKE_THREADS: what they lack within their columns; the sum
  auto look = [&](int row0) {
    const int r = row0 + t;
    int lack = 0;
    if (r < a.out_rows && (lack = a.missing[r]) != 0) {
      const Row row = row_of<FORK>(a, r);
      const int need = row.need < a.cols ? row.need : a.cols;
      end[t] = need;
      if (FORK) lack = row.keep < need;  // (its parent's holes are not filled)
      else lack -= beyond(a, row);
    }
    int total;
    const int rank = block_prefix(lack, waves, total);
    before[t] = rank;
    if (t == 0) before[TAKE_THREADS] = total;
    __syncthreads();
    return total;
  };
  // the entry of this rank, of rows that lack their last ones
  auto entry = [&](int row0, int rank, int &r) {
    int lo = 0, hi = TAKE_THREADS;  // before[lo] <= rank < before[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (before[mid] <= rank) lo = mid;
      else hi = mid;
    }
    r = row0 + lo;
    return a.out + (int64_t)r * a.out_stride + (end[lo] - (before[lo + 1] - rank));
  };
  if constexpr (!FORK) {
    bool tails = true, none = true;
    for (int row0 = 0; row0 < a.out_rows && tails; row0 += TAKE_THREADS) {
      const int total = look(row0);
      none = none && total == 0;
      bool other = false;
      for (int rank = t; rank < total; rank += TAKE_THREADS) {
        int r;
        other |= *entry(row0, rank, r) != -1;
      }
      tails = !__syncthreads_or(other);
    }
    if (!tails) return take_holes(a, free, waves);
    if (none) return;
  }
  for (int row0 = 0; row0 < a.out_rows; row0 += TAKE_THREADS) {
    const int total = look(row0);
    for (int base = 0; base < total; base += TAKE_THREADS * TAKE_ITEMS) {
      const int some = total - base < TAKE_THREADS * TAKE_ITEMS ? total - base : TAKE_THREADS * TAKE_ITEMS;
      free.find(a, some, waves);
      for (int rank = t; rank < some; rank += TAKE_THREADS) {
        const int page = free[rank];
        if (page < 0) continue;
        int r;
        *entry(row0, base + rank, r) = page;
        a.refs[page] = 1;
        atomicSub(a.missing + r, 1);
      }
      free.drop(some);
    }
    __syncthreads();  // before[] and end[] have been read
  }
}

// ---- moving ----

// The cache's four tensors as pieces of 16 bytes: codes and scales of a head's page.
struct Moved {
  u32x4 *codes[2], *scales[2];
  int code_pieces, scale_pieces;  // of a page of one head
};

Moved moved(const CacheView &cv) {
  const int page = 1 << cv.page_log2;
  return Moved{{(u32x4 *)cv.codes[0], (u32x4 *)cv.codes[1]}, {(u32x4 *)cv.scales[0], (u32x4 *)cv.scales[1]},
               page * (cv.fmt == 0 ? cv.dim / 2 : cv.dim) / 16, page * (cv.dim / 32) / 16};
}

constexpr int MOVE_THREADS = 256, MOVE_UNROLL = 4;

// A workgroup copies the pieces from .. to of one tensor's page.  PAST: what is written is not kept in the caches.
template <bool PAST>
__device__ __forceinline__ void copy_pieces(const u32x4 *src, u32x4 *dst, int64_t from, int64_t to) {
  for (int64_t i = from + threadIdx.x; i < to; i += MOVE_THREADS * MOVE_UNROLL) {
    u32x4 v[MOVE_UNROLL];
#pragma unroll
    for (int u = 0; u < MOVE_UNROLL; ++u)
      if (i + u * MOVE_THREADS < to) v[u] = src[i + u * MOVE_THREADS];
#pragma unroll
    for (int u = 0; u < MOVE_UNROLL; ++u)
      if (i + u * MOVE_THREADS < to) {
        if (PAST) __builtin_nontemporal_store(v[u], dst + i + u * MOVE_THREADS);
        else dst[i + u * MOVE_THREADS] = v[u];
      }
  }
}

// Part of `parts` workgroups of a page: each has its share of the codes and of the scales.
template <bool PAST>
__global__ __launch_bounds__(MOVE_THREADS) void k_copy_pages(Moved m, int64_t pages, int heads, const int *src,
                                                             const int *dst, int parts) {
  const int64_t n = blockIdx.x / parts;
  const int part = blockIdx.x - n * parts;
  const int from = src[n], to = dst[n];
  if ((unsigned)from >= (uint64_t)pages || (unsigned)to >= (uint64_t)pages || from == to) return;
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    const int64_t codes = (int64_t)heads * m.code_pieces, scales = (int64_t)heads * m.scale_pieces;
    const u32x4 *c = m.codes[v] + from * codes, *s = m.scales[v] + from * scales;
    copy_pieces<PAST>(c, m.codes[v] + to * codes, codes * part / parts, codes * (part + 1) / parts);
    copy_pieces<PAST>(s, m.scales[v] + to * scales, scales * part / parts, scales * (part + 1) / parts);
  }
}

// The last, partly filled page of each child: its parent's tokens and nothing behind them.
__global__ __launch_bounds__(MOVE_THREADS) void k_copy_last(Moved m, BookArgs a, int heads, int scale_rows) {
  const int child = blockIdx.x / heads, head = blockIdx.x - child * heads;
  const Row row = row_of<true>(a, child);
  if (row.keep == row.need || row.keep >= a.cols) return;
  const int from = a.table[(int64_t)row.from * a.stride + row.keep];
  const int to = a.out[(int64_t)child * a.out_stride + row.keep];
  if ((unsigned)from >= (unsigned)a.pages || (unsigned)to >= (unsigned)a.pages) return;
  const int tokens = a.kv_lens[row.from] & ((1 << a.page_log2) - 1);
  const int v = blockIdx.y, codes = m.code_pieces >> a.page_log2;  // pieces of a token
  const int64_t f = (int64_t)from * heads + head, t = (int64_t)to * heads + head;
  copy_pieces<false>(m.codes[v] + f * m.code_pieces, m.codes[v] + t * m.code_pieces, 0, tokens * codes);
  const uint8_t *s = (const uint8_t *)(m.scales[v] + f * m.scale_pieces);
  uint8_t *d = (uint8_t *)(m.scales[v] + t * m.scale_pieces);
  for (int g = 0; g < scale_rows; ++g)
    for (int i = threadIdx.x; i < tokens; i += MOVE_THREADS)
      d[(g << a.page_log2) + i] = s[(g << a.page_log2) + i];
}

struct CompactArgs {
  CacheView cache;
  const int *kv_starts, *keep, *counts, *table;
  int64_t keep_stride, stride;
  int *kv_lens;
  int max_keep, cols, code_parts, scale_parts;  // parts: workgroups that share a head's tokens
};

// Threads of a workgroup and tokens that each has under way.  Long lists have the large workgroups, whose groups are
// fewer, and two of them on a CU; short ones, of whole batches, the small ones: 64 sequences of up to 60 new tokens, 8
// heads of 128, 7.7 us against 15 with large ones, one of 8000 tokens 30 against 18.
constexpr int LARGE_THREADS = 1024, LARGE_UNROLL = 2, SMALL_THREADS = 256, SMALL_UNROLL = 4;
constexpr int COMPACT_TABLE = 4096;  // entries of the table in LDS

// A workgroup has some of the pieces of one head's tokens of one sequence, its keys' or values' codes or scales, and
// takes the tokens in groups: all of a group is read before any of it is written, and as keep[i] >= i no group writes
// what a later one reads.  So the tokens may be moved within their own pages, and every place has what place keep[i] held
// at the beginning.
// T: what a thread moves of a token, of which there are `per` pieces; this workgroup has those from piece0 to piece1.
template <int COMPACT_THREADS, int COMPACT_UNROLL, typename T>
__device__ __forceinline__ void compact(const CompactArgs &a, T *data, int per, int piece0, int piece1, bool planes,
                                        int b, int head) {
  __shared__ int near[COMPACT_TABLE];
  const CacheView &cv = a.cache;
  const int64_t start = a.kv_starts[b];
  const int *table = a.table + (int64_t)b * a.stride, *keep = a.keep + (int64_t)b * a.keep_stride;
  int count = a.counts[b];
  count = count < a.max_keep ? count : a.max_keep;
  const int mine = piece1 - piece0, group = COMPACT_THREADS / mine;
  const int token = threadIdx.x / mine, piece = piece0 + threadIdx.x - token * mine;
  const int64_t room = (int64_t)a.cols << cv.page_log2;
  const int mask = (1 << cv.page_log2) - 1;
  int next[COMPACT_UNROLL];  // entries of `keep` for the next group
  auto look_up = [&](int64_t base) {
#pragma unroll
    for (int u = 0; u < COMPACT_UNROLL; ++u) {
      const int64_t i = base + (int64_t)u * group + token;
      next[u] = token < group && i < count ? keep[i] : -1;
    }
  };
  look_up(0);
  // the table from the first place on, as far as it goes
  const int page0 = start < 0 ? 0 : start >= room ? a.cols : (int)(start >> cv.page_log2);
  for (int j = threadIdx.x; j < COMPACT_TABLE && j < a.cols - page0; j += COMPACT_THREADS) near[j] = table[page0 + j];
  __syncthreads();
  auto at = [&](int64_t place) -> int64_t {  // -1: no such place
    if (place < 0 || place >= room) return -1;
    const int j = (int)(place >> cv.page_log2) - page0;
    const int page = (unsigned)j < COMPACT_TABLE ? near[j] : table[page0 + j];
    if ((unsigned)page >= (uint64_t)cv.pages) return -1;
    const int64_t ph = (int64_t)page * cv.heads + head;
    const int r = (int)place & mask;
    return planes ? ((ph * per + piece) << cv.page_log2) + r : ((ph << cv.page_log2) + r) * per + piece;
  };
  for (int64_t base = 0; base < count; base += group * COMPACT_UNROLL) {
    T v[COMPACT_UNROLL];
    int64_t to[COMPACT_UNROLL];
#pragma unroll
    for (int u = 0; u < COMPACT_UNROLL; ++u) {
      const int64_t i = base + (int64_t)u * group + token;
      to[u] = -1;
      if (next[u] <= i) continue;  // it is where it belongs, or cannot be moved
      const int64_t from = at(start + next[u]);
      to[u] = from < 0 ? -1 : at(start + i);
      if (to[u] >= 0) v[u] = data[from];
    }
    look_up(base + group * COMPACT_UNROLL);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // what this wave reads has arrived
    __syncthreads();
#pragma unroll
    for (int u = 0; u < COMPACT_UNROLL; ++u)
      if (to[u] >= 0) data[to[u]] = v[u];
  }
}

template <int THREADS, int UNROLL>
__global__ __launch_bounds__(THREADS) void k_compact(CompactArgs a) {
  const CacheView &cv = a.cache;
  const int b = blockIdx.x / cv.heads, head = blockIdx.x - b * cv.heads, v = blockIdx.y % 2, part = blockIdx.y / 2;
  if (part >= a.code_parts) {
    const int per = cv.dim / 32, p = part - a.code_parts;
    compact<THREADS, UNROLL, uint8_t>(a, cv.scales[v], per, per * p / a.scale_parts, per * (p + 1) / a.scale_parts, true, b, head);
  } else {
    const int per = (cv.fmt == 0 ? cv.dim / 2 : cv.dim) / 16;
    compact<THREADS, UNROLL, u32x4>(a, (u32x4 *)cv.codes[v], per, per * part / a.code_parts, per * (part + 1) / a.code_parts, false, b,
                   head);
    if (blockIdx.y == 0 && head == 0 && threadIdx.x == 0) {
      const int count = a.counts[b] < a.max_keep ? a.counts[b] : a.max_keep;
      a.kv_lens[b] = a.kv_starts[b] + (count < 0 ? 0 : count);
    }
  }
}

BookArgs book(const CacheView &cv, int *refs, const int *table, int64_t stride, int cols, const int *kv_lens, int rows,
              const int *parents, int *out, int64_t out_stride, int out_rows, int *missing) {
  return BookArgs{refs, kv_lens, parents, table, stride, out_stride, out, missing, (int)cv.pages, cv.page_log2, rows,
                  cols, out_rows};
}

template <bool FORK>
hipError_t hand_out(const BookArgs &a, hipStream_t stream) {
  if (a.out_rows <= SMALL_ROWS && (int64_t)a.out_rows * a.cols <= TAKE_THREADS * SMALL_ITEMS) {
    k_pages_small<FORK><<<1, TAKE_THREADS, 0, stream>>>(a);
    return hipGetLastError();
  }
  k_page_rows<FORK><<<(a.out_rows + 3) / 4, 256, 0, stream>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_page_take<FORK><<<1, TAKE_THREADS, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_cache_resize(const CacheView &cache, int *refs, int *table, int64_t stride, int pages,
                               const int *kv_lens, int rows, int *missing, hipStream_t stream) {
  return hand_out<false>(book(cache, refs, table, stride, pages, kv_lens, rows, nullptr, table, stride, rows, missing),
                         stream);
}

hipError_t launch_cache_fork(const CacheView &cache, int *refs, const int *table, int64_t stride, int pages,
                             const int *kv_lens, int rows, const int *parents, int children, int *child_table,
                             int64_t child_stride, int *missing, hipStream_t stream) {
  const BookArgs a = book(cache, refs, table, stride, pages, kv_lens, rows, parents, child_table, child_stride,
                          children, missing);
  const hipError_t e = hand_out<true>(a, stream);
  if (e != hipSuccess) return e;
  k_copy_last<<<dim3((unsigned)(children * cache.heads), 2), MOVE_THREADS, 0, stream>>>(moved(cache), a, cache.heads,
                                                                                        cache.dim / 32);
  return hipGetLastError();
}

// Copies of so many bytes are written past the caches, which they would empty: 94 MB (keys and values, read) take 32 us so
// and 41 otherwise, 67 MB 20 and 30, 53 MB 16 and 22, 27 MB 9 either way.  What reads the copies at once has them from
// memory then: with a compaction behind it a copy of 94 MB takes 105 us so and 82 otherwise, one of 27 MB 31 and 26.
constexpr int64_t PAST_BYTES = (int64_t)64 << 20;

hipError_t launch_cache_copy(const CacheView &cache, const int *src, const int *dst, int64_t count, hipStream_t stream) {
  const Moved m = moved(cache);
  // a workgroup's share: 4 pieces for each thread, while the grid holds them
  int64_t parts = ((int64_t)cache.heads * m.code_pieces + MOVE_THREADS * MOVE_UNROLL - 1) / (MOVE_THREADS * MOVE_UNROLL);
  if (parts > MAX_GROUPS_256 / count) parts = MAX_GROUPS_256 / count;
  const unsigned grid = (unsigned)(count * parts);
  if (2 * 16 * (int64_t)cache.heads * (m.code_pieces + m.scale_pieces) * count >= PAST_BYTES)
    k_copy_pages<true><<<grid, MOVE_THREADS, 0, stream>>>(m, cache.pages, cache.heads, src, dst, (int)parts);
  else
    k_copy_pages<false><<<grid, MOVE_THREADS, 0, stream>>>(m, cache.pages, cache.heads, src, dst, (int)parts);
  return hipGetLastError();
}

hipError_t launch_cache_compact(const CacheView &cache, const int *kv_starts, const int *keep, int64_t keep_stride,
                                int max_keep, const int *counts, const int *table, int64_t stride, int pages, int batch,
                                int *kv_lens, hipStream_t stream) {
  const int codes = (cache.fmt == 0 ? cache.dim / 2 : cache.dim) / 16, scales = cache.dim / 32;
  CompactArgs a{cache, kv_starts, keep, counts, table, keep_stride, stride, kv_lens, max_keep, pages, 1, 1};
  const int64_t heads = (int64_t)batch * cache.heads;
  if ((int64_t)max_keep * codes <= 4 * SMALL_THREADS * SMALL_UNROLL) {
    k_compact<SMALL_THREADS, SMALL_UNROLL><<<dim3((unsigned)heads, 4), SMALL_THREADS, 0, stream>>>(a);
    return hipGetLastError();
  }
  // long lists of few heads are shared by the pieces of a token, down to one each, until every CU has a workgroup
  const auto parts = [&](int pieces) {
    int n = 1;
    while (n < pieces && 2 * heads * n < device_cu_count() && (int64_t)max_keep * pieces > LARGE_THREADS * LARGE_UNROLL * n)
      n = 2 * n < pieces ? 2 * n : pieces;
    return n;
  };
  a.code_parts = parts(codes);
  a.scale_parts = parts(scales);
  k_compact<LARGE_THREADS, LARGE_UNROLL>
      <<<dim3((unsigned)heads, (unsigned)(2 * (a.code_parts + a.scale_parts))), LARGE_THREADS, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace mx
