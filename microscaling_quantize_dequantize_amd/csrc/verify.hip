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
// A refusal that would leave no weight at all leaves w as it is.  Tokens outside the vocabulary are not asked.
//
// Weights are computed in fp64 from the rows, entry by entry: what a refusal
// takes away is remembered by its factor W alone (or its token), so that no row
// is ever written.  Probabilities that are negative or not finite count as zero.
//
// Bound: HBM, the rows of the node where the walk ends; only a refusal with
// another sibling behind it needs the sum of a row before that.
#include "launch.h"

namespace mx {

namespace {

constexpr int VERIFY_THREADS = 1024, VERIFY_WAVES = VERIFY_THREADS / 64;

__device__ __forceinline__ double weight_of(unsigned short b) {
  const float f = __uint_as_float((unsigned)b << 16);
  return f > 0.0f && f < __builtin_inff() ? (double)f : 0.0;
}
__device__ __forceinline__ double weight_of(float f) { return f > 0.0f && f < __builtin_inff() ? (double)f : 0.0; }

template <typename T> struct Chunk {
  static constexpr int N = 16 / sizeof(T);
  T v[N];
} __attribute__((aligned(16)));

// A node's rows, cut at 16-byte boundaries: chunk k holds the entries k N - off ..., of which those outside 0 .. vocab
// are zero.  DRAFT: there is a row q, which is cut like p; wide says that it lies to the boundaries as p does.
template <typename T, bool DRAFT> struct Rows {
  static constexpr int N = Chunk<T>::N;
  const T *p, *q;
  int vocab, off, chunks;
  bool wide;

  __device__ __forceinline__ Rows(const VerifyArgs &a, int64_t row) {
    p = (const T *)a.target + row * a.target_stride;
    q = DRAFT ? (const T *)a.draft + row * a.draft_stride : nullptr;
    vocab = a.vocab;
    off = (int)((uintptr_t)p % 16 / sizeof(T));
    wide = !DRAFT || (uintptr_t)q % 16 / sizeof(T) == (unsigned)off;
    chunks = (vocab + off + N - 1) / N;
  }
  __device__ __forceinline__ Chunk<T> read(const T *x, int k, bool whole) const {
    Chunk<T> c;
    const int64_t e = (int64_t)k * N - off;
    if (whole && k < chunks && e >= 0 && e + N <= vocab) return *(const Chunk<T> *)(x + e);
#pragma unroll
    for (int i = 0; i < N; ++i) c.v[i] = e + i >= 0 && e + i < vocab ? x[e + i] : T(0);
    return c;
  }
};

// What refusals have taken from the weights at the walk's node.
struct Taken {
  double *factor;  // with a draft's row: the W of each
  int *token;      // without: the tokens
  int count;
};

// The weights of a chunk.
template <typename T, bool DRAFT>
__device__ __forceinline__ void weigh(const Rows<T, DRAFT> &rows, const Taken &taken, int k, const Chunk<T> &p,
                                      const Chunk<T> &q, double *w) {
  constexpr int N = Chunk<T>::N;
#pragma unroll
  for (int i = 0; i < N; ++i) w[i] = weight_of(p.v[i]);
  for (int j = 0; j < taken.count; ++j) {
    if (DRAFT) {
      const double f = taken.factor[j];
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = fmax(w[i] - f * weight_of(q.v[i]), 0.0);
    } else {
      const int at = taken.token[j] - (k * N - rows.off);
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = at == i ? 0.0 : w[i];
    }
  }
}

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int d = 32; d > 0; d /= 2) v += __shfl_xor(v, d);
  return v;
}

// Sums of w over each wave's share of the chunks from .. to into sums[], and their sum (in the order of the waves).
template <typename T, bool DRAFT>
__device__ double sum_weights(const Rows<T, DRAFT> &rows, const Taken &taken, int from, int to, double *sums) {
  constexpr int N = Chunk<T>::N, UNROLL = 4;
  const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
  const int per = (to - from + VERIFY_WAVES - 1) / VERIFY_WAVES;
  const int k0 = from + wave * per, k1 = k0 + per < to ? k0 + per : to;
  double sum = 0.0;
  for (int k = k0 + lane; k < k1; k += 64 * UNROLL) {
    Chunk<T> p[UNROLL], q[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int at = k + 64 * u < k1 ? k + 64 * u : rows.chunks;  // behind the row: zeros
      p[u] = rows.read(rows.p, at, true);
      if (DRAFT) q[u] = rows.read(rows.q, at, rows.wide);
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      double w[N];
      weigh<T, DRAFT>(rows, taken, k + 64 * u, p[u], q[u], w);
#pragma unroll
      for (int i = 0; i < N; ++i) sum += w[i];
    }
  }
  sum = wave_sum_f64(sum);
  __syncthreads();  // sums of the call before have been read
  if (lane == 0) sums[wave] = sum;
  __syncthreads();
  double total = 0.0;
  for (int w = 0; w < VERIFY_WAVES; ++w) total += sums[w];
  return total;
}

// The first of n places whose running sum, after `before`, is above `target`, with `before` taken to what lies before
// it; the last one that has any weight if rounding leaves none; -1 if nothing has weight.
__device__ __forceinline__ int first_above(const double *sums, int n, double target, double &before) {
  int at = -1;
  double sum = before;
  for (int i = 0; i < n; ++i) {
    if (sums[i] > 0.0) {
      at = i;
      before = sum;
      sum += sums[i];
      if (sum > target) return at;
    }
  }
  return at;
}

template <typename T, bool DRAFT, bool TREE>
__global__ __launch_bounds__(VERIFY_THREADS) void k_verify(VerifyArgs a) {
  __shared__ double u[VERIFY_NODES], wp[VERIFY_NODES], wq[VERIFY_NODES], factor[VERIFY_NODES];
  __shared__ int64_t token[VERIFY_NODES];
  __shared__ int parent[VERIFY_NODES], refused[VERIFY_NODES];
  __shared__ double sums[VERIFY_THREADS];
  const int b = blockIdx.x, t = threadIdx.x;
  const int q0 = a.q_starts[b] < 0 ? 0 : a.q_starts[b];
  int nq = (a.q_starts[b + 1] > a.total_q ? a.total_q : a.q_starts[b + 1]) - q0;
  nq = nq < 0 ? 0 : nq > a.max_q ? a.max_q : nq;
  int *path = a.path + (int64_t)b * a.max_q;
  int64_t *out = a.out + (int64_t)b * a.max_q;

  if (t < nq) {
    const int64_t x = a.tokens[q0 + t];
    const int up = t == 0 ? -1 : TREE ? a.parents[q0 + t] : t - 1;
    u[t] = a.uniforms[q0 + t];
    token[t] = x;
    parent[t] = up;
    wp[t] = wq[t] = 0.0;
    if (up >= 0 && up < t && x >= 0 && x < a.vocab) {
      wp[t] = weight_of(((const T *)a.target)[(q0 + up) * a.target_stride + x]);
      wq[t] = DRAFT ? weight_of(((const T *)a.draft)[(q0 + up) * a.draft_stride + x]) : 1.0;
    }
  }
  __syncthreads();

  // the walk, the same in every thread
  int c = 0, kept = 0;
  double W = 1.0;
  Taken taken{factor, refused, 0};
  bool open = false;  // the last refusal's sum is not known yet
  auto settle = [&]() {
    const Rows<T, DRAFT> rows(a, q0 + c);
    const double left = sum_weights<T, DRAFT>(rows, taken, 0, rows.chunks, sums);
    if (left > 0.0) W = left;
    else --taken.count;
    open = false;
  };
  for (int i = 1; i < nq; ++i) {
    const int64_t x = token[i];
    if (parent[i] != c || x < 0 || x >= a.vocab) continue;
    if (open) settle();
    double w = wp[i];
    for (int j = 0; j < taken.count; ++j)
      w = DRAFT ? fmax(w - factor[j] * wq[i], 0.0) : refused[j] == x ? 0.0 : w;
    if (u[i] * W * wq[i] < w) {
      if (t == 0) {
        path[kept + 1] = i;
        out[kept] = x;
      }
      c = i;
      ++kept;
      W = 1.0;
      taken.count = 0;
    } else {
      __syncthreads();
      if (t == 0) {
        factor[taken.count] = W;
        refused[taken.count] = (int)x;
      }
      __syncthreads();
      ++taken.count;
      open = true;
    }
  }

  // the token after the last kept one
  int64_t chosen = -1;
  if (nq > 0) {
    const Rows<T, DRAFT> rows(a, q0 + c);
    double total = sum_weights<T, DRAFT>(rows, taken, 0, rows.chunks, sums);
    if (!(total > 0.0) && open) {
      --taken.count;
      total = sum_weights<T, DRAFT>(rows, taken, 0, rows.chunks, sums);
    }
    if (total > 0.0) {
      const double target = u[0] * total;
      double before = 0.0;
      const int wave = first_above(sums, VERIFY_WAVES, target, before);
      const int per = (rows.chunks + VERIFY_WAVES - 1) / VERIFY_WAVES;
      const int k0 = wave * per, k1 = k0 + per < rows.chunks ? k0 + per : rows.chunks;
      // that wave's share again, a run of chunks for each thread
      constexpr int N = Chunk<T>::N;
      const int run = (k1 - k0 + VERIFY_THREADS - 1) / VERIFY_THREADS;
      const int f = k0 + t * run, l = f + run < k1 ? f + run : k1;
      double mine = 0.0;
      for (int k = f; k < l; ++k) {
        double w[N];
        const Chunk<T> p = rows.read(rows.p, k, true), q = DRAFT ? rows.read(rows.q, k, rows.wide) : p;
        weigh<T, DRAFT>(rows, taken, k, p, q, w);
#pragma unroll
        for (int i = 0; i < N; ++i) mine += w[i];
      }
      __syncthreads();
      sums[t] = mine;
      __syncthreads();
      if (t == 0) {
        const int who = first_above(sums, VERIFY_THREADS, target, before);
        const int g = k0 + who * run, h = g + run < k1 ? g + run : k1;
        double sum = before;
        bool found = false;
        for (int k = g; k < h && !found; ++k) {
          double w[N];
          const Chunk<T> p = rows.read(rows.p, k, true), q = DRAFT ? rows.read(rows.q, k, rows.wide) : p;
          weigh<T, DRAFT>(rows, taken, k, p, q, w);
          for (int i = 0; i < N && !found; ++i) {
            sum += w[i];
            if (w[i] > 0.0) chosen = (int64_t)k * N - rows.off + i;
            found = sum > target && w[i] > 0.0;
          }
        }
      }
    }
  }
  if (t == 0) a.counts[b] = nq > 0 ? kept + 1 : 0;
  for (int i = t; i < a.max_q; i += VERIFY_THREADS) {
    if (i == 0) path[0] = nq > 0 ? 0 : -1;
    else if (i > kept || nq == 0) path[i] = -1;
    if (i > kept || nq == 0) out[i] = -1;
  }
  if (t == 0 && nq > 0) out[kept] = chosen;
}

template <typename T, bool DRAFT>
hipError_t verify(const VerifyArgs &a, hipStream_t stream) {
  if (a.parents) k_verify<T, DRAFT, true><<<a.batch, VERIFY_THREADS, 0, stream>>>(a);
  else k_verify<T, DRAFT, false><<<a.batch, VERIFY_THREADS, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

int64_t verify_workspace(int, int, int) { return 0; }

hipError_t launch_verify(int dtype, const VerifyArgs &a, hipStream_t stream) {
  if (dtype == 1) return a.draft ? verify<float, true>(a, stream) : verify<float, false>(a, stream);
  return a.draft ? verify<unsigned short, true>(a, stream) : verify<unsigned short, false>(a, stream);
}

}  // namespace mx
