// Verification of drafted tokens against the target's probabilities.
//
// Node 0 of a sequence is its last settled token, the others are drafted, each
// a child of a node before it.  The walk starts at node c = 0 with weights
// w = p_c and W = 1, and asks the children of c in their order: child i with
// token x is kept if  u_i W q_c(x) < w(x),  and then c = i.  A child that is
// not kept leaves  w = max(w - W q_c, 0),  W = sum w.  The token after the last
// kept one is sampled from w: the first whose cumulative sum is above
// u_0 sum(w).  So what is put out is distributed as the target's own tokens,
// whatever the drafts were (q_c: the distribution the children of c were drawn
// from; without one, 1 for the child's token and 0 for the others).
// A refusal that would leave no weight at all leaves w as it is.  Tokens outside
// the vocabulary are not asked.
//
// As q is not negative, all that was taken from w is one factor:
//   w = max(p - F q, 0),  F the sum of the W that were taken,
// so no row is ever written; without a draft's row it is the tokens refused.
// Weights and sums are fp64, as the test and the sample have borders that fp32
// sums of 10^5 entries would miss.  Probabilities that are negative or NaN count
// as zero, infinite ones as the largest number of fp32.
//
// Three kernels.  k_branch (trees only) finds for each node what follows it:
// which child is kept, or the factors with which the walk ends there.  That does
// not depend on the way to the node, so nodes are worked on side by side, a
// workgroup each, and only those that a walk can reach and that have a child
// behind a refused one need the sum of a row.  k_sums follows the walk and sums
// the weights at its end in shares of 1024 entries; k_pick finds the token in one
// of them, with one wave.  Short rows are one workgroup's, which does both.
//
// Bound: HBM for large batches (64 rows of p and q of 128001 entries in fp32 on MI355X:
// k_sums 14.4 us, 4.5 TB/s, on inputs that change from call to call, and 12.4, 5.3
// TB/s, out of the last-level cache, which holds them; k_pick 4.9); else the chain of
// dependent loads (starts, tokens, points of rows, rows, sums: 6 us for small rows); of
// a node with several refused children the vector units of its one CU: 7 instructions
// an entry (two medians, two conversions, three of fp64 arithmetic), 5 us a refusal
// for 50001 entries and 10 for 128000, whatever their type.
// (A refusal's sum in fp32 would be quicker, but its error would move every border
// of the sample: one token in some thousand would be another.)
#include "launch.h"

namespace mx {

namespace {

// The median of a number, zero and the largest one; of NaN it is the smaller of the other two.
__device__ __forceinline__ double weight_of(float f) {
  return (double)__builtin_amdgcn_fmed3f(f, 0.0f, 3.402823466e38f);
}
__device__ __forceinline__ double weight_of(unsigned short b) { return weight_of(__uint_as_float((unsigned)b << 16)); }

template <typename T> struct Chunk {
  static constexpr int N = 16 / sizeof(T);
  T v[N];
} __attribute__((aligned(16)));
template <typename T> struct Loose {  // the same at any element
  T v[16 / sizeof(T)];
} __attribute__((packed, aligned(sizeof(T))));

// A node's rows, cut where the target's has 16-byte boundaries: chunk k holds the entries k N - off ..., of which those
// outside 0 .. vocab are zero; the chunks whole0 .. whole1 have none of these.  DRAFT: there is a row q, whose chunks may
// lie across boundaries (one load all the same).
template <typename T, bool DRAFT> struct Rows {
  static constexpr int N = Chunk<T>::N;
  const T *p, *q;
  int vocab, off, chunks, whole0, whole1;

  __device__ __forceinline__ Rows(const VerifyArgs &a, int64_t row) {
    p = (const T *)a.target + row * a.target_stride;
    q = DRAFT ? (const T *)a.draft + row * a.draft_stride : p;
    vocab = a.vocab;
    off = (int)((uintptr_t)p % 16 / sizeof(T));
    chunks = (vocab + off + N - 1) / N;
    whole0 = off > 0;
    whole1 = (vocab + off) / N;
  }
  // A chunk that is whole.
  __device__ __forceinline__ void read_whole(int64_t k, Chunk<T> &cp, Chunk<T> &cq) const {
    const int64_t e = k * N - off;
    cp = *(const Chunk<T> *)(p + e);
    if (DRAFT) cq = __builtin_bit_cast(Chunk<T>, *(const Loose<T> *)(q + e));
  }
  __device__ __forceinline__ void read(int k, Chunk<T> &cp, Chunk<T> &cq) const {
    if (k >= whole0 && k < whole1) return read_whole(k, cp, cq);
    const int64_t e = (int64_t)k * N - off;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool in = e + i >= 0 && e + i < vocab;
      cp.v[i] = in ? p[e + i] : T(0);
      if (DRAFT) cq.v[i] = in ? q[e + i] : T(0);
    }
  }
};

// What was taken from the weights: F q, or without a draft's row the tokens of a list.
struct Taken {
  double factor;
  const int *tokens;
  int count;
};

// The weights of chunk k.
template <typename T, bool DRAFT>
__device__ __forceinline__ void weigh(const Rows<T, DRAFT> &rows, const Taken &taken, int k, const Chunk<T> &p,
                                      const Chunk<T> &q, double *w) {
  constexpr int N = Chunk<T>::N;
#pragma unroll
  for (int i = 0; i < N; ++i) w[i] = weight_of(p.v[i]);
  if (DRAFT) {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = fmax(__builtin_fma(-taken.factor, weight_of(q.v[i]), w[i]), 0.0);
  } else {
    for (int j = 0; j < taken.count; ++j) {
      const int64_t at = taken.tokens[j] - ((int64_t)k * N - rows.off);
      if ((uint64_t)at < N) {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = at == i ? 0.0 : w[i];
      }
    }
  }
}

// Sums over the lanes of a wave go by row shifts and row broadcasts, which take a tenth of the time of exchanges by way
// of LDS; every lane is active.
template <int CTRL, int ROWS> __device__ __forceinline__ double shifted(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const unsigned lo = __builtin_amdgcn_update_dpp(0, (int)(unsigned)b, CTRL, ROWS, 0xF, false);
  const unsigned hi = __builtin_amdgcn_update_dpp(0, (int)(unsigned)(b >> 32), CTRL, ROWS, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Of the lanes up to this one.
__device__ __forceinline__ double wave_scan_f64(double v) {
  v += shifted<0x111, 0xF>(v);  // by 1, 2, 4 and 8 within rows of 16
  v += shifted<0x112, 0xF>(v);
  v += shifted<0x114, 0xF>(v);
  v += shifted<0x118, 0xF>(v);
  v += shifted<0x142, 0xA>(v);  // the last of rows 0 and 2 to rows 1 and 3
  v += shifted<0x143, 0xC>(v);  // the last of row 1 to rows 2 and 3
  return v;
}

__device__ __forceinline__ double lane_value(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const unsigned lo = __builtin_amdgcn_readlane((int)(unsigned)b, lane);
  const unsigned hi = __builtin_amdgcn_readlane((int)(unsigned)(b >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ double wave_sum_f64(double v) { return lane_value(wave_scan_f64(v), 63); }

// The sum of v over the workgroup, in the order of its waves; waves[] has a place for each.
template <int THREADS>
__device__ __forceinline__ double block_sum(double v, double *waves) {
  v = wave_sum_f64(v);
  __syncthreads();  // what the call before left there has been read
  if (threadIdx.x % 64 == 0) waves[threadIdx.x / 64] = v;
  __syncthreads();
  double total = 0.0;
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) total += waves[w];
  return total;
}

// The sum of the weights of the chunks from .. to that `lanes` lanes have among them, of which this is `lane`; each has
// its own part of it.
template <typename T, bool DRAFT>
__device__ __forceinline__ double add_weights(const Rows<T, DRAFT> &rows, const Taken &taken, int from, int to, int lanes,
                                              int lane) {
  constexpr int N = Chunk<T>::N, UNROLL = 4;
  double sum = 0.0;
  auto add = [&](int k, const Chunk<T> &p, const Chunk<T> &q) {
    double w[N];
    weigh<T, DRAFT>(rows, taken, k, p, q, w);
#pragma unroll
    for (int i = 0; i < N; ++i) sum += w[i];
  };
  auto add_cut = [&](int k) {
    Chunk<T> p, q;
    rows.read(k, p, q);
    add(k, p, q);
  };
  const int k0 = from > rows.whole0 ? from : rows.whole0, k1 = to < rows.whole1 ? to : rows.whole1;
  for (int64_t k = k0 + (int64_t)lane; k < k1; k += UNROLL * lanes) {
    Chunk<T> p[UNROLL], q[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u)
      // behind the end the last chunk, which is not added: no load waits for a branch
      rows.read_whole(k + u * lanes < k1 ? k + u * lanes : k1 - 1, p[u], q[u]);
#pragma unroll
    for (int u = 0; u < UNROLL; ++u)
      if (k + u * lanes < k1) add((int)k + u * lanes, p[u], q[u]);
  }
  // the ends, if they are cut (one lane each)
  if (lane == 0 && from < rows.whole0 && to > 0) add_cut(0);
  if (lane == lanes - 1 && to > rows.whole1 && to > rows.whole0 && from <= rows.whole1) add_cut(rows.whole1);
  return sum;
}

struct Nodes {
  int first, count;  // of a sequence
};

__device__ __forceinline__ Nodes nodes_of(const VerifyArgs &a, int b) {
  const int q0 = a.q_starts[b], q1 = a.q_starts[b + 1];
  const int first = q0 < 0 ? 0 : q0;
  int n = (q1 > a.total_q ? a.total_q : q1) - first;
  n = n < 0 ? 0 : n > a.max_q ? a.max_q : n;
  return Nodes{first, n};
}

// The workspace: sums of shares, and where each sequence's walk ends; of trees, what follows each node.
struct End {
  int node, kept;  // kept: drafted tokens
  double before, after;  // the factor without and with the last refusal
};
struct Follow {
  int next, pad;  // the child that is kept, or -1
  double before, after;
};
struct Space {
  End *ends;        // [batch]
  Follow *follow;   // [total_q], trees
  int *gone;        // [total_q], trees without a draft's rows: the node's token was taken from its parent's weights
  double *sums;     // [batch][shares]
};

int64_t ends_bytes(int batch) { return (int64_t)batch * (int64_t)sizeof(End); }
int64_t follow_bytes(int64_t total_q) { return total_q * (int64_t)sizeof(Follow); }
int64_t gone_bytes(int64_t total_q) { return (total_q * 4 + 7) / 8 * 8; }

// Whether the test of a point passes, with the weights as they are at first (what k_sums and k_branch ask alike).
__device__ __forceinline__ bool passes(double u, double W, double q, double w) { return u * W * q < w; }

// The point of a drafted token in its parent's rows.
template <typename T, bool DRAFT>
__device__ __forceinline__ void point_of(const VerifyArgs &a, int64_t row, int64_t x, double &p, double &q) {
  p = weight_of(((const T *)a.target)[row * a.target_stride + x]);
  q = DRAFT ? weight_of(((const T *)a.draft)[row * a.draft_stride + x]) : 1.0;
}

// ---- trees: what follows each node ----

constexpr int BRANCH_THREADS = VERIFY_NODES;

// The number of threads before this one for which v holds, and of all.
__device__ __forceinline__ int block_rank(bool v, int *waves, int &total) {
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const uint64_t mask = __builtin_amdgcn_ballot_w64(v);
  __syncthreads();
  if (lane == 0) waves[wave] = __builtin_popcountll(mask);
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < BRANCH_THREADS / 64; ++w) {
    before += w < wave ? waves[w] : 0;
    total += waves[w];
  }
  return before + __builtin_popcountll(mask & (((uint64_t)1 << lane) - 1));
}

template <typename T, bool DRAFT>
__global__ __launch_bounds__(BRANCH_THREADS) void k_branch(VerifyArgs a, Space space, int groups) {
  __shared__ double u[VERIFY_NODES], wp[VERIFY_NODES], wq[VERIFY_NODES], sums[BRANCH_THREADS / 64];
  __shared__ int token[VERIFY_NODES], parent[VERIFY_NODES], first[VERIFY_NODES], kids[VERIFY_NODES], list[VERIFY_NODES];
  __shared__ int ranks[BRANCH_THREADS / 64];
  __shared__ bool passed[VERIFY_NODES], open[VERIFY_NODES];
  const int b = blockIdx.x / groups, group = blockIdx.x - b * groups, t = threadIdx.x;
  const Nodes nodes = nodes_of(a, b);
  if (nodes.count == 0) return;
  Follow *follow = space.follow + nodes.first;
  int *gone = space.gone + nodes.first;

  bool asked = false;  // this thread's node has a parent that may ask it
  first[t] = VERIFY_NODES;
  kids[t] = 0;
  parent[t] = -1;
  if (t > 0 && t < nodes.count) {
    const int64_t x = a.tokens[nodes.first + t];
    const int up = a.parents[nodes.first + t];
    u[t] = a.uniforms[nodes.first + t];
    asked = up >= 0 && up < t && x >= 0 && x < a.vocab;
    if (asked) {
      double p, q;
      point_of<T, DRAFT>(a, nodes.first + up, x, p, q);
      wp[t] = p;
      wq[t] = q;
      token[t] = (int)x;
      parent[t] = up;
      passed[t] = passes(u[t], 1.0, q, p);
    }
  }
  __syncthreads();
  if (asked) {
    atomicMin(first + parent[t], t);
    atomicAdd(kids + parent[t], 1);
  }
  __syncthreads();
  // whether a walk can come from the parent to here: as its first child that is kept, or behind a first that is not
  if (asked) open[t] = first[parent[t]] == t ? passed[t] : !passed[first[parent[t]]];
  __syncthreads();
  int up = t;
  while (up > 0 && parent[up] >= 0 && open[up]) up = parent[up];
  const bool reached = t < nodes.count && up == 0;
  const bool refused = kids[t] > 0 && !passed[first[t]];
  const bool wanted = reached && refused && kids[t] > 1;
  if (group == 0 && reached && !wanted) {
    follow[t] = Follow{kids[t] > 0 && !refused ? first[t] : -1, 0, 0.0, refused ? 1.0 : 0.0};
    if (!DRAFT && refused) gone[first[t]] = 1;
  }
  int count;
  const int rank = block_rank(wanted, ranks, count);
  if (wanted) list[rank] = t;
  __syncthreads();

  for (int l = group; l < count; l += groups) {
    const int c = list[l];
    const bool mine = asked && parent[t] == c;
    int n;
    const int place = block_rank(mine, ranks, n);
    __syncthreads();
    if (mine) kids[place] = t;  // the children of c in their order (numbers of children are not read any more)
    __syncthreads();
    const Rows<T, DRAFT> rows(a, nodes.first + c);
    int next = -1;
    double before = 0.0, after = 0.0, W = 1.0;
    if (DRAFT) {
      for (int k = 0; k < n; ++k) {
        const int i = kids[k];
        if (passes(u[i], W, wq[i], fmax(__builtin_fma(-before, wq[i], wp[i]), 0.0))) {
          next = i;
          break;
        }
        after = before + W;
        if (k + 1 == n) break;
        const double left = block_sum<BRANCH_THREADS>(
            add_weights(rows, Taken{after, nullptr, 0}, 0, rows.chunks, BRANCH_THREADS, t), sums);
        if (left > 0.0) before = after, W = left;
      }
    } else {
      // the weights beside the children's tokens, once; W is that and those of the tokens that are left
      __shared__ int tokens[VERIFY_NODES];
      if (t < n) tokens[t] = token[kids[t]];
      __syncthreads();
      int *same = first;   // the first child (in the order) with the same token
      bool *taken = open;  // by that child: its token was taken
      if (t < n) {
        int j = 0;
        while (tokens[j] != tokens[t]) ++j;
        same[t] = j;
        taken[t] = false;
      }
      __syncthreads();
      const bool counts = t < n && same[t] == t;
      const double weight = counts ? wp[kids[t]] : 0.0;
      const double others = block_sum<BRANCH_THREADS>(
          add_weights(rows, Taken{0.0, tokens, n}, 0, rows.chunks, BRANCH_THREADS, t), sums);
      for (int k = 0; k < n; ++k) {
        const int i = kids[k], j = same[k];
        if (passes(u[i], W, 1.0, taken[j] ? 0.0 : wp[i])) {
          next = i;
          break;
        }
        const double rest = others + block_sum<BRANCH_THREADS>(counts && !taken[t] && t != j ? weight : 0.0, sums);
        const bool goes = rest > 0.0 || k + 1 == n;  // of the last one k_pick sees to it
        if (goes) W = rest, after = 1.0;
        if (t == 0) {
          if (goes) taken[j] = true;
          gone[i] = goes;
        }
        __syncthreads();
      }
    }
    if (t == 0) follow[c] = Follow{next, 0, before, after};
    __syncthreads();
  }
}

// ---- the walk, and the sums at its end ----

constexpr int SUM_THREADS = 256, ONE_THREADS = 1024;  // of k_sums beside k_pick, and of the kernel that is both
constexpr int SHARE = 1024;                           // entries of a share, a wave's unit, unless there are too many
constexpr int MOST_SHARES = 4096;

// A row's chunks in `shares` runs, of which a wave has `each`.
struct Cut {
  int shares, each;
  __device__ __forceinline__ int at(int chunks, int s) const { return (int)((int64_t)chunks * s / shares); }
};

// What was taken from the weights at a sequence's end node; !all: without its last refusal.  A wave puts the tokens into
// list[VERIFY_NODES] (LDS).
template <bool DRAFT, bool TREE>
__device__ __forceinline__ Taken taken_at(const VerifyArgs &a, const Space &space, int b, const Nodes &nodes,
                                          const End &end, bool all, int *list) {
  if (DRAFT) return Taken{all ? end.after : end.before, nullptr, 0};
  Taken taken{0.0, list, 0};
  if (!(end.after > 0.0)) return taken;
  const int lane = threadIdx.x % 64;
  if (!TREE) {
    if (lane == 0 && all) list[0] = (int)a.tokens[nodes.first + end.node + 1];
    taken.count = all;
  } else {
    const int *gone = space.gone + nodes.first;
    for (int base = end.node + 1; base < nodes.count; base += 64) {
      const int i = base + lane;
      int64_t x = -1;
      if (i < nodes.count && a.parents[nodes.first + i] == end.node) x = a.tokens[nodes.first + i];
      const bool asked = x >= 0 && x < a.vocab;
      const uint64_t mask = __builtin_amdgcn_ballot_w64(asked && gone[asked ? i : 0]);
      if (mask >> lane & 1) list[taken.count + __builtin_popcountll(mask & (((uint64_t)1 << lane) - 1))] = (int)x;
      taken.count += __builtin_popcountll(mask);
    }
    taken.count -= !all;  // the last child's, which is always there
  }
  return taken;
}

// The walk of sequence b; `write`: this workgroup puts out what is known from it.
template <int THREADS, typename T, bool DRAFT, bool TREE>
__device__ __forceinline__ End walk(const VerifyArgs &a, const Space &space, int b, const Nodes &nodes, bool write,
                                    int *next) {
  const int t = threadIdx.x, wave = t / 64, lane = t % 64;
  int *path = a.path + (int64_t)b * a.max_q;
  int64_t *out = a.out + (int64_t)b * a.max_q;
  End end{0, 0, 0.0, 0.0};
  if (TREE) {
    const Follow *follow = space.follow + nodes.first;
    for (int i = t; i < nodes.count; i += THREADS) next[i] = follow[i].next;
    __syncthreads();
    // what follows nodes that no walk reaches is not set, and not looked at.  A node's next one is behind it, unless
    // starts that do not ascend give it to several sequences: then the walk ends.
    for (int i = nodes.count > 0 ? next[0] : -1; i > end.node && i < nodes.count; i = next[i]) {
      end.node = i;
      ++end.kept;
      if (write && t == 0) {
        path[end.kept] = i;
        out[end.kept - 1] = a.tokens[nodes.first + i];
      }
    }
    if (nodes.count > 0) end.before = follow[end.node].before, end.after = follow[end.node].after;
  } else {
    // the first node that is not kept, in each wave its own first; bit 0: its token was refused, and is not outside
    // the vocabulary
    int key = 2 * nodes.count;
    for (int base = 1 + 64 * wave; base < nodes.count; base += THREADS) {
      const int i = base + lane;
      const int64_t x = i < nodes.count ? a.tokens[nodes.first + i] : -1;
      const bool in = x >= 0 && x < a.vocab;
      bool keep = i >= nodes.count;
      if (in) {
        double p, q;
        point_of<T, DRAFT>(a, nodes.first + i - 1, x, p, q);
        keep = passes(a.uniforms[nodes.first + i], 1.0, q, p);
      }
      const uint64_t stop = __builtin_amdgcn_ballot_w64(!keep), there = __builtin_amdgcn_ballot_w64(in);
      if (stop) {
        const int l = __builtin_ctzll(stop);
        key = 2 * (base + l) + (int)(there >> l & 1);
        break;
      }
    }
    if (lane == 0) next[wave] = key;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) key = next[w] < key ? next[w] : key;
    end.node = end.kept = nodes.count > 0 ? key / 2 - 1 : 0;
    end.after = key & 1;
    if (write)
      for (int i = 1 + t; i <= end.kept; i += THREADS) {
        path[i] = i;
        out[i - 1] = a.tokens[nodes.first + i];
      }
  }
  if (write) {
    if (t == 0) a.counts[b] = nodes.count > 0 ? end.kept + 1 : 0;
    for (int i = t; i < a.max_q; i += THREADS) {
      if (i == 0) path[0] = nodes.count > 0 ? 0 : -1;
      else if (i > end.kept) path[i] = -1;
      if (i > end.kept || nodes.count == 0) out[i] = -1;
    }
  }
  return end;
}

// The first lane whose running sum, after `before`, is above target (a lane without weight is not), the last one with
// weight if rounding leaves none, -1 without any; `before` becomes the sum before it.
__device__ __forceinline__ int first_above(double v, double target, double &before) {
  const double after = before + wave_scan_f64(v);
  const uint64_t any = __builtin_amdgcn_ballot_w64(v > 0.0), above = __builtin_amdgcn_ballot_w64(v > 0.0 && after > target);
  if (!any) return -1;
  const int lane = above ? __builtin_ctzll(above) : 63 - __builtin_clzll(any);
  before = lane_value(after - v, lane);
  return lane;
}

// The sampled token, by one wave: the share that the goal lies in, then each lane's run of its chunks, then that run.
// sums[] (LDS) has the shares' sums.
template <typename T, bool DRAFT, bool TREE>
__device__ __forceinline__ void pick(const VerifyArgs &a, const Space &space, int b, const Nodes &nodes, const End &end,
                                     Cut cut, double u, Taken taken, double *sums, int *list) {
  constexpr int N = Chunk<T>::N, HELD = 4;  // chunks of a lane that are read together
  const int lane = threadIdx.x % 64;
  const Rows<T, DRAFT> rows(a, nodes.first + end.node);
  const int some = (cut.shares + 63) / 64, s0 = lane * some;
  auto shares = [&]() {
    double v = 0.0;
    for (int s = s0; s < s0 + some && s < cut.shares; ++s) v += sums[s];
    return v;
  };
  double mine = shares(), total = wave_sum_f64(mine);
  if (!(total > 0.0) && end.after > end.before) {  // the last refusal would leave nothing: it takes nothing
    taken = taken_at<DRAFT, TREE>(a, space, b, nodes, end, false, list);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
    for (int s = 0; s < cut.shares; ++s) {
      const double v = wave_sum_f64(add_weights(rows, taken, cut.at(rows.chunks, s), cut.at(rows.chunks, s + 1), 64, lane));
      if (lane == 0) sums[s] = v;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
    mine = shares();
    total = wave_sum_f64(mine);
  }
  int64_t *out = a.out + (int64_t)b * a.max_q + end.kept;
  if (!(total > 0.0)) {
    if (lane == 0) *out = -1;
    return;
  }
  const double target = u * total;
  double before = 0.0, sum;
  int share = first_above(mine, target, before) * some;
  sum = before;
  for (int s = share, last = s + some < cut.shares ? s + some : cut.shares; s < last; ++s) {
    if (!(sums[s] > 0.0)) continue;
    share = s;
    before = sum;
    sum += sums[s];
    if (sum > target) break;
  }
  const int k0 = cut.at(rows.chunks, share), k1 = cut.at(rows.chunks, share + 1);
  const int run = (k1 - k0 + 63) / 64;
  const int f = (int64_t)k0 + (int64_t)lane * run < k1 ? k0 + lane * run : k1, l = k1 - f > run ? f + run : k1;
  mine = 0.0;
  for (int k = f; k < l; k += HELD) {
    Chunk<T> p[HELD], q[HELD];
#pragma unroll
    for (int h = 0; h < HELD; ++h) {
      rows.read(k + h < l ? k + h : l - 1, p[h], q[h]);
    }
#pragma unroll
    for (int h = 0; h < HELD; ++h) {
      if (k + h >= l) continue;
      double w[N];
      weigh<T, DRAFT>(rows, taken, k + h, p[h], q[h], w);
#pragma unroll
      for (int i = 0; i < N; ++i) mine += w[i];
    }
  }
  if (lane != first_above(mine, target, before)) return;
  sum = before;
  int64_t chosen = -1;
  bool done = false;
  for (int k = f; k < l && !done; ++k) {
    double w[N];
    Chunk<T> p, q;
    rows.read(k, p, q);
    weigh<T, DRAFT>(rows, taken, k, p, q, w);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      sum += w[i];
      if (w[i] > 0.0 && !done) {
        chosen = (int64_t)k * N - rows.off + i;
        done = sum > target;
      }
    }
  }
  *out = chosen;
}

template <int THREADS, typename T, bool DRAFT, bool TREE, bool ONE>
__global__ __launch_bounds__(THREADS) void k_sums(VerifyArgs a, Space space, Cut cut) {
  constexpr int WAVES = THREADS / 64;
  __shared__ double sums[ONE ? 2 * WAVES : 1];
  __shared__ int next[VERIFY_NODES], list[DRAFT ? 1 : VERIFY_NODES], held;
  const int groups = cut.shares / (WAVES * cut.each), b = blockIdx.x / groups, group = blockIdx.x - b * groups;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / 64), lane = threadIdx.x % 64;
  const Nodes nodes = nodes_of(a, b);
  const double u = ONE && nodes.count > 0 ? a.uniforms[nodes.first] : 0.0;
  const End end = walk<THREADS, T, DRAFT, TREE>(a, space, b, nodes, group == 0, next);
  if (!ONE && group == 0 && threadIdx.x == 0) space.ends[b] = end;
  if (nodes.count == 0) return;
  const Rows<T, DRAFT> rows(a, nodes.first + end.node);
  Taken taken{end.after, list, 0};
  if (!DRAFT) {
    if (wave == 0) {
      taken = taken_at<DRAFT, TREE>(a, space, b, nodes, end, true, list);
      if (lane == 0) held = taken.count;
    }
    __syncthreads();
    taken.count = held;
  }
  for (int e = 0; e < cut.each; ++e) {
    const int s = (group * WAVES + wave) * cut.each + e;
    const double sum =
        wave_sum_f64(add_weights(rows, taken, cut.at(rows.chunks, s), cut.at(rows.chunks, s + 1), 64, lane));
    if (lane == 0) (ONE ? sums[ONE ? s : 0] : space.sums[(int64_t)b * cut.shares + s]) = sum;
  }
  if (!ONE) return;
  __syncthreads();
  if (wave == 0) pick<T, DRAFT, TREE>(a, space, b, nodes, end, cut, u, taken, sums, list);
}

template <typename T, bool DRAFT, bool TREE>
__global__ __launch_bounds__(64) void k_pick(VerifyArgs a, Space space, Cut cut) {
  __shared__ double sums[MOST_SHARES];
  __shared__ int list[DRAFT ? 1 : VERIFY_NODES];
  const int b = blockIdx.x;
  for (int s = threadIdx.x; s < cut.shares; s += 64) sums[s] = space.sums[(int64_t)b * cut.shares + s];
  const End end = space.ends[b];
  const Nodes nodes = nodes_of(a, b);
  if (nodes.count == 0) return;
  const double u = a.uniforms[nodes.first];
  const Taken taken = taken_at<DRAFT, TREE>(a, space, b, nodes, end, true, list);
  __syncthreads();
  pick<T, DRAFT, TREE>(a, space, b, nodes, end, cut, u, taken, sums, list);
}

// Short rows are the work of one workgroup: a launch less, of 2.5 us for the host.  (Chains over 32000 entries: kernels
// 8.8 us against 7.6 of two for one sequence, 17 against 19 for 256.)  Longer ones have a share for each wave, or two
// where that is four workgroups for every CU.
constexpr int ONE_ENTRIES = 1 << 15;

Cut cut_of(int batch, int vocab) {
  constexpr int WAVES = SUM_THREADS / 64;
  if (vocab <= ONE_ENTRIES) {
    constexpr int waves = ONE_THREADS / 64;
    static_assert(ONE_ENTRIES <= 2 * waves * SHARE, "sums of k_sums");
    return vocab <= waves * SHARE ? Cut{waves, 1} : Cut{2 * waves, 2};
  }
  int64_t groups = ((int64_t)vocab + SHARE * WAVES - 1) / (SHARE * WAVES);
  const int each = batch * groups >= 4 * device_cu_count() ? 2 : 1;
  groups = (groups + each - 1) / each;
  if (groups > MOST_SHARES / (WAVES * each)) groups = MOST_SHARES / (WAVES * each);
  if (batch > 0 && groups > MAX_GROUPS_256 / batch) groups = MAX_GROUPS_256 / batch;
  return Cut{WAVES * each * (int)(groups < 1 ? 1 : groups), each};
}

template <typename T, bool DRAFT, bool TREE>
hipError_t verify(const VerifyArgs &a, const Space &space, hipStream_t stream) {
  if (TREE && a.max_q > 0 && a.total_q > 0) {
    // a workgroup for each node of a sequence, fewer of many sequences
    int64_t per = 2 * device_cu_count() / a.batch;
    per = per < 4 ? 4 : per;
    if (per > a.max_q) per = a.max_q;
    if (per > MAX_VERIFY / a.batch) per = MAX_VERIFY / a.batch;
    k_branch<T, DRAFT><<<(unsigned)(per * a.batch), BRANCH_THREADS, 0, stream>>>(a, space, (int)per);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const Cut cut = cut_of(a.batch, a.vocab);
  if (a.vocab <= ONE_ENTRIES) {
    k_sums<ONE_THREADS, T, DRAFT, TREE, true><<<(unsigned)a.batch, ONE_THREADS, 0, stream>>>(a, space, cut);
    return hipGetLastError();
  }
  const unsigned grid = (unsigned)(cut.shares / (SUM_THREADS / 64 * cut.each) * (int64_t)a.batch);
  k_sums<SUM_THREADS, T, DRAFT, TREE, false><<<grid, SUM_THREADS, 0, stream>>>(a, space, cut);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_pick<T, DRAFT, TREE><<<(unsigned)a.batch, 64, 0, stream>>>(a, space, cut);
  return hipGetLastError();
}

template <typename T>
hipError_t verify(const VerifyArgs &a, const Space &space, hipStream_t stream) {
  if (a.draft)
    return a.parents ? verify<T, true, true>(a, space, stream) : verify<T, true, false>(a, space, stream);
  return a.parents ? verify<T, false, true>(a, space, stream) : verify<T, false, false>(a, space, stream);
}

}  // namespace

int64_t verify_workspace(int batch, int64_t total_q, int vocab) {
  return ends_bytes(batch) + follow_bytes(total_q) + gone_bytes(total_q) +
         (int64_t)batch * cut_of(batch, vocab).shares * 8;
}

hipError_t launch_verify(int dtype, const VerifyArgs &a, hipStream_t stream) {
  char *at = (char *)a.workspace;
  Space space;
  space.ends = (End *)at;
  space.follow = (Follow *)(at += ends_bytes(a.batch));
  space.gone = (int *)(at += follow_bytes(a.total_q));
  space.sums = (double *)(at += gone_bytes(a.total_q));
  return dtype == 1 ? verify<float>(a, space, stream) : verify<unsigned short>(a, space, stream);
}

}  // namespace mx
