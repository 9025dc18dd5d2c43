// The pages of the store that are worth a query's attention.
//
//     score[t, g, p] = sum over the group's heads h of <q[t, h], mean[p, g]>
//                    = < sum_h q[t, h], mean[p, g] >
//
// The choice among nearly equal scores has to be the definition's, not the
// summation order's, so scores are formed in fp64: the sum of the group's
// queries is exact or nearly so, the products are, and the sums agree to about
// 1e-16 whatever their order. A block takes up to kTok tokens of one sequence and key
// head; a thread scores one page for all of them, so that a mean is read and
// widened once for the block's tokens. The scores become order-preserving
// 64-bit keys in shared memory (0: not a candidate, all ones: taken whatever
// its score), and a warp per token finds the select-th largest key bit by bit
// and writes the pages in ascending order.
#include "store.cuh"

namespace fastnn {

namespace {

constexpr int kThreads = 256;
constexpr int kTok = 8;
constexpr int kSmemKeys = 196608;  // bytes of keys a block may hold

__device__ __forceinline__ uint64_t key_of(double x) {
  if (x != x) return 1;  // NaN: behind every number
  x += 0.0;              // -0 and 0 are equal
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x));
  const uint64_t k = (u >> 63) ? ~u : (u | 0x8000000000000000ull);
  return k < 2 ? 2 : k == ~0ull ? k - 1 : k;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
select_kernel(SelectArgs a, int tok_per_block, int key_stride) {
  extern __shared__ __align__(16) uint8_t smem[];
  const StoreArgs& st = a.st;
  const int s = blockIdx.z, g = blockIdx.y, tid = threadIdx.x;
  const SeqView w = seq_view(st, s, a.n, a.max_new, a.causal);
  const int i0 = static_cast<int>(blockIdx.x) * tok_per_block;
  if (i0 >= w.n) return;
  const int m = w.n - i0 < tok_per_block ? w.n - i0 : tok_per_block;
  double* qs = reinterpret_cast<double*>(smem);                    // [d][kTok]
  uint64_t* keys = reinterpret_cast<uint64_t*>(qs + st.d * kTok);  // [tok_per_block][key_stride]

  for (int i = tid; i < st.d * kTok; i += kThreads) {
    const int t = i / st.d, e = i - t * st.d;
    double sum = 0.0;
    if (t < m) {
      const uint16_t* q = a.q + (static_cast<int64_t>(w.t0) + i0 + t) * a.q_stride +
                          static_cast<int64_t>(g) * a.group * st.d + e;
      for (int h = 0; h < a.group; ++h) sum += static_cast<double>(Half16<T>::one(__ldg(q + h * st.d)));
    }
    qs[e * kTok + t] = sum;
  }
  __syncthreads();
  const int vlast = visible(w, i0 + m - 1);
  const int pages = (vlast + st.page - 1) >> st.page_log2;  // of the block's last token
  for (int p = tid; p < pages; p += kThreads) {
    const int id = __ldg(st.table + static_cast<int64_t>(s) * st.width + p);
    const bool there = id >= 0 && id < st.n_pages;
    double acc[kTok] = {};
    if (there) {
      const uint4* row = reinterpret_cast<const uint4*>(
          st.mean + (static_cast<int64_t>(id) * st.heads + g) * st.d);
      for (int c = 0; c < st.d / 8; ++c) {
        const uint4 x = __ldg(row + c);
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = Half16<T>::unpack(xs[i]);
          const double lo = f.x, hi = f.y;
          const double* q = qs + (c * 8 + 2 * i) * kTok;
#pragma unroll
          for (int t = 0; t < kTok; ++t) acc[t] += lo * q[t];
#pragma unroll
          for (int t = 0; t < kTok; ++t) acc[t] += hi * q[kTok + t];
        }
      }
    }
#pragma unroll
    for (int t = 0; t < kTok; ++t) {
      if (t >= m) break;
      const int seen = (visible(w, i0 + t) + st.page - 1) >> st.page_log2;
      uint64_t key = 0;
      if (there && p < seen)
        key = p < a.keep_first || p >= seen - a.keep_last ? ~0ull : key_of(acc[t]);
      keys[t * key_stride + p] = key;
    }
  }
  __syncthreads();
  const int warp = tid >> 5, lane = tid & 31;
  for (int t = warp; t < m; t += kThreads / 32) {
    const uint64_t* k = keys + t * key_stride;
    const int seen = (visible(w, i0 + t) + st.page - 1) >> st.page_log2;
    auto count = [&](uint64_t level) {
      int c = 0;
      for (int p = lane; p < seen; p += 32) c += k[p] >= level;
      return __reduce_add_sync(0xffffffffu, c);
    };
    // The largest level that at least `select` keys reach (or 1: every
    // candidate is taken), and how many of the keys equal to it are.
    uint64_t level = 1;
    int room = INT32_MAX;
    if (count(1) > a.select) {
      level = 0;
      int reach = 0;
      for (int b = 63; b >= 0; --b) {
        const uint64_t up = level | (1ull << b);
        const int c = count(up);
        if (c >= a.select) {
          level = up;
          reach = c;
          if (c == a.select) break;
        }
      }
      if (reach > a.select) room = a.select - (level == ~0ull ? 0 : count(level + 1));
    }
    int32_t* out = a.out + ((static_cast<int64_t>(w.t0) + i0 + t) * st.heads + g) * a.select;
    int done = 0, ties = 0;
    for (int p0 = 0; p0 < seen && done < a.select; p0 += 32) {
      const uint64_t key = p0 + lane < seen ? k[p0 + lane] : 0;
      const bool tie = room != INT32_MAX && key == level;
      const unsigned tied = __ballot_sync(0xffffffffu, tie);
      const int before = ties + __popc(tied & ((1u << lane) - 1u));
      const bool take = key >= level && key > 0 && (!tie || before < room);
      const unsigned taken = __ballot_sync(0xffffffffu, take);
      const int at = done + __popc(taken & ((1u << lane) - 1u));
      if (take && at < a.select) out[at] = p0 + lane;
      ties += __popc(tied);
      done += __popc(taken);
    }
    for (int i = done + lane; i < a.select; i += 32) out[i] = -1;
  }
}

template <typename T>
int select_t(const SelectArgs& a, cudaStream_t st) {
  const int key_stride = a.st.width;
  int tok = kSmemKeys / 8 / key_stride;
  if (tok > kTok) tok = kTok;
  if (tok > a.max_new) tok = a.max_new;
  if (tok < 1) return FASTNN_ERR_UNSUPPORTED;
  const size_t smem = static_cast<size_t>(a.st.d) * kTok * 8 + static_cast<size_t>(tok) * key_stride * 8;
  FASTNN_CUDA_TRY(cudaFuncSetAttribute(select_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kSmemKeys + 128 * kTok * 8));
  const int blocks = (a.max_new + tok - 1) / tok;
  select_kernel<T><<<dim3(blocks, a.st.heads, a.st.n_seqs), kThreads, smem, st>>>(a, tok, key_stride);
  FASTNN_CUDA_TRY(cudaGetLastError());
  return FASTNN_OK;
}

}  // namespace

int select_max_width() { return kSmemKeys / 8; }

int launch_select(const SelectArgs& a, int dtype, cudaStream_t st) {
  return dtype == FASTNN_BF16 ? select_t<__nv_bfloat16>(a, st) : select_t<__half>(a, st);
}

}  // namespace fastnn
