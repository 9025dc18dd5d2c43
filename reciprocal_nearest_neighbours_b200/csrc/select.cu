// The pages of the store that are worth a query's attention.
//
//     score[t, g, p] = sum over the group's heads h of <q[t, h], mean[p, g]>
//                    = < sum_h q[t, h], mean[p, g] >
//
// The choice among nearly equal scores has to be the definition's, not the
// summation order's, so scores are formed in fp64: the sum of the group's
// queries is exact or nearly so, the products are, and the sums agree to about
// 1e-16 whatever their order. They become order-preserving 64-bit keys (0: not
// a candidate, all ones: taken whatever its score); a row's keys are held in
// registers, the select-th largest is found bit by bit (from the highest bit
// in which they differ), and the pages are written in ascending order.
//   steps (a few tokens a sequence): half a warp scores a page; for one token and
//       up to 512 pages in the block that picks, else in blocks of 64 pages before
//       the choice.
//       Bound by latency, then by reading the means once. (A cluster of 8 blocks
//       that shares the pages and picks in one kernel took 30 us for 16
//       sequences of up to 1024 pages; the two kernels take 24.)
//   chunks: the groups' sums once, then tiles of 64 tokens x 64 pages, 4 x 4 a
//       thread, both operands as fp64 in shared memory (bound by the fp64 units
//       and the shared memory that feeds them), then the choice. The keys of a
//       slab of tokens stay below kSlabBytes, about half of L2.
// Measured: one token of 16 sequences of 1024 pages, 4 key heads, 25 us; 2048 tokens
// over 256 pages 70 (scores 50).
#include "store.cuh"

namespace fastnn {

namespace {

constexpr int kThreads = 256;
constexpr int kTile = 64;      // tokens, pages of a score tile
constexpr int kDepth = 32;     // elements of d in shared memory at a time
constexpr int kStepTokens = 8; // fewer new tokens a sequence: the step kernel
constexpr int kWholeWidth = 512;  // pages that a single token's block scores and picks from by itself
constexpr int kShare = 64;        // pages that it scores where the table is wider
constexpr int64_t kSlabBytes = 64 << 20;

__device__ __forceinline__ uint64_t key_of(double x) {
  if (x != x) return 1;  // NaN: behind every number
  x += 0.0;              // -0 and 0 are equal
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x));
  const uint64_t k = (u >> 63) ? ~u : (u | 0x8000000000000000ull);
  return k < 2 ? 2 : k == ~0ull ? k - 1 : k;
}

__device__ __forceinline__ int seen_pages(const SelectArgs& a, const SeqView& w, int i) {
  return (visible(w, i) + a.st.page - 1) >> a.st.page_log2;
}

// The key row of token i (of the slab) of sequence s and key head g.
__device__ __forceinline__ uint64_t* key_row(const SelectArgs& a, int s, int i, int g) {
  return a.keys + ((static_cast<int64_t>(s) * a.slab + i) * a.st.heads + g) * a.st.width;
}

__device__ __forceinline__ uint64_t candidate(const SelectArgs& a, int p, int seen, bool there, double x) {
  if (!there) return 0;
  return p < a.keep_first || p >= seen - a.keep_last ? ~0ull : key_of(x);
}

__device__ __forceinline__ int page_of(const SelectArgs& a, int s, int p) {
  const int id = __ldg(a.st.table + static_cast<int64_t>(s) * a.st.width + p);
  return id < a.st.n_pages ? id : -1;
}

// Picks the pages of one row from its keys. W warps a row; thread r of the row
// holds keys [r * K, r * K + K) in registers (K == 0: any number, read again and
// again from `keys`).
template <int W, int K>
__device__ __forceinline__ void pick_row(const SelectArgs& a, const uint64_t* keys,
                                         const uint64_t (&held)[K ? K : 1], int seen, int64_t token, int g) {
  constexpr int kRow = 32 * W;
  __shared__ int parts[2][8];
  __shared__ uint64_t ends[2][8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = W == 1 ? lane : tid;
  const int per = K ? K : (seen + kRow - 1) / kRow;
  const int p0 = r * per;
  auto key = [&](int k) -> uint64_t { return p0 + k < seen ? keys[p0 + k] : 0; };
  int turn = 0;
  auto total = [&](int c) {  // over the row
    c = __reduce_add_sync(0xffffffffu, c);
    if (W > 1) {
      if (lane == 0) parts[turn][warp] = c;
      __syncthreads();
      c = 0;
#pragma unroll
      for (int q = 0; q < W; ++q) c += parts[turn][q];
      turn ^= 1;
    }
    return c;
  };
  auto before = [&](int c) {  // over the threads of the row before this one
    int x = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const int all = __shfl_sync(0xffffffffu, x, 31);
    x -= c;
    if (W > 1) {
      if (lane == 0) parts[turn][warp] = all;
      __syncthreads();
      for (int q = 0; q < warp; ++q) x += parts[turn][q];
      turn ^= 1;
    }
    return x;
  };
  auto count = [&](uint64_t level) {
    int c = 0;
    if (K) {
#pragma unroll
      for (int k = 0; k < (K ? K : 1); ++k) c += held[k] >= level;
    } else {
      for (int k = 0; k < per; ++k) c += key(k) >= level;
    }
    return total(c);
  };
  // The largest level that at least `select` keys reach (1: every candidate is
  // taken), and how many of the keys equal to it are (room < 0: all).
  uint64_t level = 1;
  int room = -1;
  if (count(1) > a.select) {
    // Bits above the highest one in which the candidates by score differ are common.
    uint64_t lo = ~0ull, hi = 0;
    for (int k = 0; k < per; ++k) {
      const uint64_t x = K ? held[K ? k : 0] : key(k);
      if (x && x != ~0ull) {  // those taken in any case reach every level
        lo = x < lo ? x : lo;
        hi = x > hi ? x : hi;
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const uint64_t l2 = __shfl_xor_sync(0xffffffffu, lo, o), h2 = __shfl_xor_sync(0xffffffffu, hi, o);
      lo = l2 < lo ? l2 : lo;
      hi = h2 > hi ? h2 : hi;
    }
    if (W > 1) {
      if (lane == 0) {
        ends[0][warp] = lo;
        ends[1][warp] = hi;
      }
      __syncthreads();
      for (int q = 0; q < W; ++q) {
        lo = ends[0][q] < lo ? ends[0][q] : lo;
        hi = ends[1][q] > hi ? ends[1][q] : hi;
      }
    }
    level = hi;
    int reach = a.select;
    if (lo != hi) {
      const int top = 63 - __clzll(static_cast<long long>(lo ^ hi));
      level = top == 63 ? 0 : (hi >> (top + 1)) << (top + 1);
      reach = a.select + 1;  // more than select keys reach the common bits
      for (int b = top; b >= 0; --b) {
        const uint64_t up = level | (1ull << b);
        const int c = count(up);
        if (c >= a.select) {
          level = up;
          reach = c;
          if (c == a.select) break;
        }
      }
    } else {
      reach = a.select + 1;
    }
    if (reach > a.select) room = a.select - (level == ~0ull ? 0 : count(level + 1));
  }
  int ties = 0, more = 0;
  if (room >= 0) {
    for (int k = 0; k < per; ++k) ties += (K ? held[K ? k : 0] : key(k)) == level;
    ties = before(ties);  // equal keys in the threads before
  }
  int t = ties;
  for (int k = 0; k < per; ++k) {
    const uint64_t x = K ? held[K ? k : 0] : key(k);
    more += x > level || (x == level && (room < 0 || t < room));
    t += x == level;
  }
  int at = before(more);
  int32_t* out = a.out + (token * a.st.heads + g) * a.select;
  t = ties;
  for (int k = 0; k < per; ++k) {
    const uint64_t x = K ? held[K ? k : 0] : key(k);
    const bool take = x > level || (x == level && (room < 0 || t < room));
    t += x == level;
    if (take && at < a.select) out[at++] = p0 + k;
  }
  const int taken = total(more);
  for (int k = taken + r; k < a.select; k += kRow) out[k] = -1;
}

template <int W, int K>
__global__ void __launch_bounds__(kThreads)
pick_kernel(SelectArgs a) {
  cudaGridDependencySynchronize();
  const StoreArgs& st = a.st;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = W == 1 ? static_cast<int64_t>(blockIdx.x) * 8 + warp : blockIdx.x;
  const int g = static_cast<int>(row % st.heads);
  const int64_t si = row / st.heads;
  const int s = static_cast<int>(si / a.slab), i = static_cast<int>(si - static_cast<int64_t>(s) * a.slab);
  if (s >= st.n_seqs) return;
  const SeqView w = seq_view(st, s, a.n, a.max_new, a.causal);
  if (a.first + i >= w.n) return;
  const int seen = seen_pages(a, w, a.first + i);
  const uint64_t* keys = key_row(a, s, i, g);
  uint64_t held[K ? K : 1];
  if (K) {
    const int p0 = (W == 1 ? lane : tid) * K;
#pragma unroll
    for (int k = 0; k < K; ++k) held[k] = p0 + k < seen ? keys[p0 + k] : 0;
  }
  pick_row<W, K>(a, keys, held, seen, static_cast<int64_t>(w.t0) + a.first + i, g);
}

// Steps: half a warp a page, lane l % 16 elements 8 (l % 16) and on, for each of the
// (fewer than kStepTokens) tokens. WHOLE (one token): a block scores all pages of
// its sequence and key head and picks from them; else it scores kShare pages, and
// pick_kernel follows.
template <typename T, bool WHOLE>
__global__ void __launch_bounds__(kThreads)
step_kernel(SelectArgs a) {
  __shared__ uint64_t held_keys[WHOLE ? kWholeWidth : 1];
  __shared__ __align__(16) double qs[kStepTokens][128];
  const StoreArgs& st = a.st;
  const int s = blockIdx.z, g = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const SeqView w = seq_view(st, s, a.n, a.max_new, a.causal);
  if (w.n <= 0) return;
  const int last = seen_pages(a, w, w.n - 1);
  const int share = WHOLE ? kWholeWidth : kShare, first = static_cast<int>(blockIdx.x) * share;
  if (!WHOLE && first >= last) return;
  const int e0 = (lane & 15) * 8;
  constexpr int kFly = 4;  // pages in flight a half warp
  uint4 mean[kFly];
  int id[kFly];
  auto fetch = [&](int k, int p) {
    id[k] = p < first + share && p < last ? page_of(a, s, p) : -1;
    mean[k] = make_uint4(0, 0, 0, 0);
    if (id[k] >= 0 && e0 < st.d)
      mean[k] = __ldg(reinterpret_cast<const uint4*>(
          st.mean + (static_cast<int64_t>(id[k]) * st.heads + g) * st.d + e0));
  };
  const int half = lane >> 4;
  int pw = first + warp * 2;  // the warp's first page: its two halves go through the loop together
#pragma unroll
  for (int k = 0; k < kFly; ++k) fetch(k, pw + half + 16 * k);
  for (int x = tid; x < w.n * 128; x += kThreads) {
    const int i = x >> 7, e = x & 127;
    double sum = 0.0;
    if (e < st.d) {
      const uint16_t* q = a.q + (static_cast<int64_t>(w.t0) + i) * a.q_stride +
                          static_cast<int64_t>(g) * a.group * st.d + e;
      for (int h = 0; h < a.group; ++h) sum += static_cast<double>(Half16<T>::one(__ldg(q + h * st.d)));
    }
    qs[i][e] = sum;
  }
  __syncthreads();
  for (; pw < first + share && pw < last; pw += 16 * kFly) {
    uint4 x[kFly];
    bool there[kFly];
#pragma unroll
    for (int k = 0; k < kFly; ++k) {
      x[k] = mean[k];
      there[k] = id[k] >= 0;
      fetch(k, pw + half + 16 * (kFly + k));
    }
    for (int i = 0; i < w.n; ++i) {
      // The pages' sums side by side: their chains of additions overlap.
      double acc[kFly] = {};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const double2 q = *reinterpret_cast<const double2*>(&qs[i][e0 + 2 * e]);
#pragma unroll
        for (int k = 0; k < kFly; ++k) {
          const uint32_t xs[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
          const float2 y = Half16<T>::unpack(xs[e]);
          acc[k] += static_cast<double>(y.x) * q.x;
          acc[k] += static_cast<double>(y.y) * q.y;
        }
      }
#pragma unroll
      for (int o = 8; o; o >>= 1)
#pragma unroll
        for (int k = 0; k < kFly; ++k) acc[k] += __shfl_xor_sync(0xffffffffu, acc[k], o);
      const int seen = seen_pages(a, w, i);
#pragma unroll
      for (int k = 0; k < kFly; ++k) {
        const int p = pw + half + 16 * k;
        if ((lane & 15) == k && p < first + share && p < seen) {
          const uint64_t key = candidate(a, p, seen, there[k], acc[k]);
          if (WHOLE) {
            held_keys[p] = key;
          } else {
            key_row(a, s, i, g)[p] = key;
          }
        }
      }
    }
  }
  if constexpr (WHOLE) {
    __syncthreads();
    constexpr int K = kWholeWidth / kThreads;
    const int seen = seen_pages(a, w, 0);
    uint64_t held[K];
#pragma unroll
    for (int k = 0; k < K; ++k) held[k] = tid * K + k < seen ? held_keys[tid * K + k] : 0;
    pick_row<8, K>(a, nullptr, held, seen, w.t0, g);
  }
}

// The sums of the groups' queries in fp64, 8 elements a thread: every page tile
// reads them, and widening is slow (a few elements a clock and SM).
template <typename T>
__global__ void __launch_bounds__(kThreads)
sum_kernel(SelectArgs a) {
  const StoreArgs& st = a.st;
  const int s = blockIdx.y, per = st.heads * (st.d / 8);
  const SeqView w = seq_view(st, s, a.n, a.max_new, a.causal);
  const int n = w.n - a.first < a.slab ? w.n - a.first : a.slab;
  for (int64_t x = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
       x < static_cast<int64_t>(n) * per; x += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int i = static_cast<int>(x / per), c = static_cast<int>(x - static_cast<int64_t>(i) * per);
    const int g = c / (st.d / 8), e = (c - g * (st.d / 8)) * 8;
    const uint16_t* q = a.q + (static_cast<int64_t>(w.t0) + a.first + i) * a.q_stride +
                        static_cast<int64_t>(g) * a.group * st.d + e;
    double sum[8] = {};
#pragma unroll 4
    for (int h = 0; h < a.group; ++h) {
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(q + h * st.d));
      const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = Half16<T>::unpack(xs[k]);
        sum[2 * k] += static_cast<double>(f.x);
        sum[2 * k + 1] += static_cast<double>(f.y);
      }
    }
    double2* out = reinterpret_cast<double2*>(
        a.sums + ((static_cast<int64_t>(s) * a.slab + i) * st.heads + g) * st.d + e);
#pragma unroll
    for (int k = 0; k < 4; ++k) out[k] = make_double2(sum[2 * k], sum[2 * k + 1]);
  }
}

// Block: 64 tokens x 64 pages of one sequence and key head.
template <typename T>
__global__ void __launch_bounds__(kThreads)
score_chunk_kernel(SelectArgs a) {
  cudaGridDependencySynchronize();
  __shared__ double qs[kDepth][kTile + 1], ms[kDepth][kTile + 1];
  __shared__ int ids[kTile];
  const StoreArgs& st = a.st;
  const int tiles = (a.slab + kTile - 1) / kTile;
  const int s = blockIdx.z / tiles, i0 = (blockIdx.z - s * tiles) * kTile, g = blockIdx.y, tid = threadIdx.x;
  const SeqView w = seq_view(st, s, a.n, a.max_new, a.causal);
  const int n = (w.n - a.first < a.slab ? w.n - a.first : a.slab) - i0;
  if (n <= 0) return;
  const int m = n < kTile ? n : kTile;
  const int pb = blockIdx.x * kTile;
  const int last = seen_pages(a, w, a.first + i0 + m - 1);
  if (pb >= last) return;
  if (tid < kTile) ids[tid] = pb + tid < last ? page_of(a, s, pb + tid) : -1;
  __syncthreads();
  // A thread fetches 8 elements of one token and of one page at a time, a step
  // ahead of the products.
  const int row = tid >> 2, e = (tid & 3) * 8;
  const double* q0 = a.sums + ((static_cast<int64_t>(s) * a.slab + i0 + row) * st.heads + g) * st.d + e;
  const uint16_t* m0 = st.mean + (static_cast<int64_t>(ids[row]) * st.heads + g) * st.d + e;
  double2 qn[4];
  uint4 mn;
  auto fetch = [&](int e0) {
    const bool in = e0 + e < st.d;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      qn[k] = in && row < m ? __ldcg(reinterpret_cast<const double2*>(q0 + e0) + k) : make_double2(0.0, 0.0);
    mn = in && ids[row] >= 0 ? __ldg(reinterpret_cast<const uint4*>(m0 + e0)) : make_uint4(0, 0, 0, 0);
  };
  fetch(0);
  double acc[4][4] = {};
  const int tx = tid & 15, ty = (tid >> 4) * 4;  // pages tx + 16 c, tokens ty + t
  for (int e0 = 0; e0 < st.d; e0 += kDepth) {
    __syncthreads();
    const uint32_t xs[4] = {mn.x, mn.y, mn.z, mn.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = Half16<T>::unpack(xs[k]);
      qs[e + 2 * k][row] = qn[k].x;
      qs[e + 2 * k + 1][row] = qn[k].y;
      ms[e + 2 * k][row] = f.x;
      ms[e + 2 * k + 1][row] = f.y;
    }
    __syncthreads();
    if (e0 + kDepth < st.d) fetch(e0 + kDepth);
#pragma unroll 8
    for (int k = 0; k < kDepth; ++k) {
      double q[4], p[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) q[c] = qs[k][ty + c];
#pragma unroll
      for (int c = 0; c < 4; ++c) p[c] = ms[k][tx + 16 * c];
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[t][c] += q[t] * p[c];
    }
  }
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    if (ty + t >= m) break;
    const int seen = seen_pages(a, w, a.first + i0 + ty + t);
    uint64_t* keys = key_row(a, s, i0 + ty + t, g);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int p = pb + tx + 16 * c;
      if (p < seen) keys[p] = candidate(a, p, seen, ids[tx + 16 * c] >= 0, acc[t][c]);
    }
  }
}

// Tokens of one slab: their keys stay below kSlabBytes (at least one tile).
int64_t slab_tokens(const StoreArgs& st, int max_new) {
  int64_t n = kSlabBytes / (static_cast<int64_t>(st.n_seqs) * st.heads * st.width * 8);
  n = n / kTile * kTile;
  if (n < kTile) n = kTile;
  return n < max_new ? n : max_new;
}

template <int W, int K>
cudaError_t pick(const SelectArgs& a, cudaStream_t st) {
  const int64_t rows = static_cast<int64_t>(a.st.n_seqs) * a.slab * a.st.heads;
  const int64_t blocks = W == 1 ? (rows + 7) / 8 : rows;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  return launch_after(pick_kernel<W, K>, dim3(static_cast<unsigned>(blocks)), dim3(W == 1 ? kThreads : 32 * W), st, a);
}

bool is_step(int max_new) { return max_new < kStepTokens; }
// A single token over few pages needs no scratch and one launch. (16 sequences of
// 400 pages, 4 key heads: 1 token 19.5 us by one block, 19.8 by two kernels; 7 tokens
// 80 and 38. Chunk kernels instead of the step's: 50 and 54. The table's width stands
// for the number of pages: measured with tables no wider than the need.)
bool is_whole(const StoreArgs& st, int max_new) { return max_new == 1 && st.width <= kWholeWidth; }

template <typename T>
int select_t(const SelectArgs& all, cudaStream_t st) {
  SelectArgs a = all;
  const int width = a.st.width;
  a.first = 0;
  if (is_whole(a.st, a.max_new)) {
    step_kernel<T, true><<<dim3(1, a.st.heads, a.st.n_seqs), kThreads, 0, st>>>(a);
    FASTNN_CUDA_TRY(cudaGetLastError());
    return FASTNN_OK;
  }
  a.slab = static_cast<int>(slab_tokens(a.st, a.max_new));
  const int page_blocks = (width + kTile - 1) / kTile;
  // Too many tiles for one grid dimension: a tile of tokens at a time.
  if (static_cast<int64_t>((a.slab + kTile - 1) / kTile) * a.st.n_seqs > 65535) a.slab = kTile;
  for (; a.first < a.max_new; a.first += a.slab) {
    if (is_step(a.max_new)) {
      step_kernel<T, false><<<dim3((width + kShare - 1) / kShare, a.st.heads, a.st.n_seqs), kThreads, 0, st>>>(a);
      FASTNN_CUDA_TRY(cudaGetLastError());
    } else {
      const int64_t items = static_cast<int64_t>(a.slab) * a.st.heads * (a.st.d / 8);
      const int64_t blocks = (items + kThreads - 1) / kThreads;
      sum_kernel<T><<<dim3(blocks < 4096 ? static_cast<unsigned>(blocks) : 4096u, a.st.n_seqs), kThreads, 0, st>>>(a);
      FASTNN_CUDA_TRY(cudaGetLastError());
      const unsigned z = static_cast<unsigned>((a.slab + kTile - 1) / kTile) * a.st.n_seqs;
      FASTNN_CUDA_TRY(launch_after(score_chunk_kernel<T>, dim3(page_blocks, a.st.heads, z), dim3(kThreads), st, a));
    }
    FASTNN_CUDA_TRY(width <= 128    ? (pick<1, 4>(a, st))
                    : width <= 256  ? (pick<1, 8>(a, st))
                    : width <= 512  ? (pick<1, 16>(a, st))
                    : width <= 1024 ? (pick<8, 4>(a, st))
                    : width <= 4096 ? (pick<8, 16>(a, st))
                                    : (pick<8, 0>(a, st)));
  }
  return FASTNN_OK;
}

}  // namespace

size_t select_key_bytes(const StoreArgs& st, int max_new) {
  return is_whole(st, max_new)
             ? 0 : static_cast<size_t>(st.n_seqs) * slab_tokens(st, max_new) * st.heads * st.width * 8;
}

size_t select_sum_bytes(const StoreArgs& st, int max_new) {
  return is_step(max_new)
             ? 0 : static_cast<size_t>(st.n_seqs) * slab_tokens(st, max_new) * st.heads * st.d * 8;
}

int launch_select(const SelectArgs& a, int dtype, cudaStream_t st) {
  return dtype == FASTNN_BF16 ? select_t<__nv_bfloat16>(a, st) : select_t<__half>(a, st);
}

}  // namespace fastnn
