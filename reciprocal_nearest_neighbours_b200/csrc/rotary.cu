// Position rotation of rows, and the append of rotated keys and values to the
// paged token store.
//
// Pair j of axis a turns by t = pos[a] * freq[j]:
//     (u, w) -> scale * (u cos t - w sin t, w cos t + u sin t).
// The angle is formed as a number of turns in fp64 and reduced to half a turn
// either way before it is rounded to fp32 (a position of 2^20 at one radian a
// step would lose four decimal digits of its angle in an fp32 product); sine
// and cosine are then sincospif's. Both are computed once for a token and
// shared by its heads through shared memory. Everything else is two reads and
// two writes of 2 bytes a pair: the kernels are bound by memory. Measured: 24576
// tokens of 16 heads of 64 21.4 us, 4.7 TB/s; the append of 24k tokens of 8 heads of
// 128 in 12 ragged prompts, with means, 55 us, 3.8 TB/s (a block's phases follow
// one another: more warps an SM helped, more work a thread did not).
#include "store.cuh"

namespace fastnn {

namespace {

constexpr int kThreads = 256;
constexpr int kAppendThreads = 128;
constexpr int kAppendRows = 32;       // rows whose angles are held at a time
constexpr double kTurnsPerRadian = 0.15915494309189533577;  // 1 / (2 pi)

template <int V>
struct Vec;
template <> struct Vec<8> { using type = uint4; };
template <> struct Vec<4> { using type = uint2; };
template <> struct Vec<2> { using type = uint32_t; };
template <> struct Vec<1> { using type = uint16_t; };

template <int V>
union Pack {
  typename Vec<V>::type v;
  uint16_t h[V];
  uint32_t w[(V + 1) / 2];
};

template <typename T, int V>
__device__ __forceinline__ void unpack(const Pack<V>& p, float (&f)[V]) {
  if constexpr (V == 1) {
    f[0] = Half16<T>::one(p.h[0]);
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float2 x = Half16<T>::unpack(p.w[i]);
      f[2 * i] = x.x;
      f[2 * i + 1] = x.y;
    }
  }
}
template <typename T, int V>
__device__ __forceinline__ void repack(const float (&f)[V], Pack<V>& p) {
  if constexpr (V == 1) {
    p.h[0] = static_cast<uint16_t>(Half16<T>::pack(f[0], 0.f));
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) p.w[i] = Half16<T>::pack(f[2 * i], f[2 * i + 1]);
  }
}

// i / n and i % n of i = start, start + stride, ...: a division at the start, an
// addition and a carry a step (the append's loops are bound by
// instructions, and an integer division takes some thirty of them).
struct Split {
  int q, r, n, dq, dr;
  __device__ __forceinline__ Split(int start, int stride, int n_) : n(n_) {
    q = start / n;
    r = start - q * n;
    dq = stride / n;
    dr = stride - dq * n;
  }
  __device__ __forceinline__ void step() {
    q += dq;
    r += dr;
    if (r >= n) {
      r -= n;
      ++q;
    }
  }
};

__device__ __forceinline__ float2 turn_of(const RotaryArgs& r, int pos, int j) {
  double t = static_cast<double>(pos) * (__ldg(r.freq + j) * kTurnsPerRadian);
  t -= rint(t);
  float s, c;
  sincospif(static_cast<float>(2.0 * t), &s, &c);
  return make_float2(c * r.scale, s * r.scale * r.sign);
}

// V pairs of one row: two vectors of V elements. Half layout: the vectors hold
// the first and the second elements of the pairs; interleaved: whole pairs,
// V / 2 in each (V == 1: the two elements of one pair).
template <typename T, int V>
__device__ __forceinline__ void rotate_item(const uint16_t* row, uint16_t* out, int item,
                                            const float2* turns, const RotaryArgs& r) {
  const int per_axis = r.nf / V;
  const int a = item >= per_axis ? 1 : 0;
  const int j = (item - a * per_axis) * V;
  const float2* t = turns + a * r.nf + j;
  const int base = a * 2 * r.nf;
  const int o1 = r.interleaved ? base + 2 * j : base + j;
  const int o2 = r.interleaved ? o1 + V : o1 + r.nf;
  Pack<V> p1, p2;
  p1.v = *reinterpret_cast<const typename Vec<V>::type*>(row + o1);
  p2.v = *reinterpret_cast<const typename Vec<V>::type*>(row + o2);
  float x[V], y[V];
  unpack<T, V>(p1, x);
  unpack<T, V>(p2, y);
  if (V == 1 || !r.interleaved) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float2 cs = t[i];
      const float u = x[i], w = y[i];
      x[i] = u * cs.x - w * cs.y;
      y[i] = w * cs.x + u * cs.y;
    }
  } else if constexpr (V > 1) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float2 c1 = t[i], c2 = t[i + V / 2];
      const float u1 = x[2 * i], w1 = x[2 * i + 1], u2 = y[2 * i], w2 = y[2 * i + 1];
      x[2 * i] = u1 * c1.x - w1 * c1.y;
      x[2 * i + 1] = w1 * c1.x + u1 * c1.y;
      y[2 * i] = u2 * c2.x - w2 * c2.y;
      y[2 * i + 1] = w2 * c2.x + u2 * c2.y;
    }
  }
  repack<T, V>(x, p1);
  repack<T, V>(y, p2);
  *reinterpret_cast<typename Vec<V>::type*>(out + o1) = p1.v;
  *reinterpret_cast<typename Vec<V>::type*>(out + o2) = p2.v;
}

// A block takes `tokens` consecutive tokens with all their heads.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads)
rotary_kernel(const uint16_t* x, int64_t x_stride, int64_t n, int heads, int d, RotaryArgs r,
              uint16_t* out, int64_t out_stride, int tokens) {
  extern __shared__ float2 turns[];
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tokens;
  const int m = n - t0 < tokens ? static_cast<int>(n - t0) : tokens;
  const int nt = r.axes * r.nf;
  for (int i = threadIdx.x; i < m * nt; i += kThreads) {
    const int t = i / nt, j = i - t * nt, a = j >= r.nf ? 1 : 0;
    turns[i] = turn_of(r, __ldg(r.pos + (t0 + t) * r.axes + a), j - a * r.nf);
  }
  __syncthreads();
  const int items = nt / V, per_token = heads * items;
  for (int i = threadIdx.x; i < m * per_token; i += kThreads) {
    const int t = i / per_token, j = i - t * per_token;
    const int h = j / items, item = j - h * items;
    rotate_item<T, V>(x + (t0 + t) * x_stride + static_cast<int64_t>(h) * d,
                      out + (t0 + t) * out_stride + static_cast<int64_t>(h) * d, item,
                      turns + t * nt, r);
  }
  const int rest = (d - r.rot) / V;  // elements behind the rotated part
  if (rest > 0 && out != x) {
    for (int i = threadIdx.x; i < m * heads * rest; i += kThreads) {
      const int t = i / (heads * rest), j = i - t * heads * rest;
      const int h = j / rest, e = r.rot + (j - h * rest) * V;
      *reinterpret_cast<typename Vec<V>::type*>(out + (t0 + t) * out_stride + static_cast<int64_t>(h) * d + e) =
          *reinterpret_cast<const typename Vec<V>::type*>(x + (t0 + t) * x_stride + static_cast<int64_t>(h) * d + e);
    }
  }
}

// One block writes the new rows of one page of one sequence and one head, and
// then that page's mean. Block (0, 0, n_seqs), if there is one, writes the status
// word.
template <typename T, int V>
__global__ void __launch_bounds__(kAppendThreads)
append_kernel(StoreArgs st, const uint16_t* k, int64_t k_stride, const uint16_t* v,
              int64_t v_stride, int64_t n, int max_new, RotaryArgs r, int* status) {
  extern __shared__ float2 turns[];  // [kAppendRows][axes * nf]
  __shared__ float sums[kAppendThreads * 8];
  const int tid = threadIdx.x;
  const int s = blockIdx.z, h = blockIdx.y;
  if (s == st.n_seqs) {
    if (blockIdx.x != 0 || h != 0) return;
    bool bad = false;
    for (int q = tid; q < st.n_seqs; q += kAppendThreads) {
      const int64_t m = static_cast<int64_t>(st.cu[q + 1]) - st.cu[q], len = st.lens[q];
      bad = bad || m < 0 || m > max_new || st.cu[q] < 0 || st.cu[q + 1] > n || len < 0 ||
            (m > 0 && len + m > static_cast<int64_t>(st.width) * st.page);
      if (bad || m == 0) continue;
      for (int64_t p = len >> st.page_log2; p <= (len + m - 1) >> st.page_log2; ++p) {
        const int id = st.table[static_cast<int64_t>(q) * st.width + p];
        bad = bad || id < 0 || id >= st.n_pages;
      }
    }
    bad = __syncthreads_or(bad);
    if (tid == 0) *status = bad ? kStatusStoreIndex : 0;
    return;
  }
  const int len = __ldg(st.lens + s);
  const SeqView w = seq_view(st, s, n, max_new, 0);
  if (len < 0 || w.n == 0) return;
  const int64_t end = static_cast<int64_t>(len) + w.n;  // positions after the call
  const int64_t lp = (len >> st.page_log2) + static_cast<int64_t>(blockIdx.x);
  const int64_t p0 = lp << st.page_log2;
  if (p0 >= end || lp >= st.width) return;
  const int id = __ldg(st.table + static_cast<int64_t>(s) * st.width + lp);
  if (id < 0 || id >= st.n_pages) return;
  const int first = len > p0 ? static_cast<int>(len - p0) : 0;  // new rows [first, fill)
  const int fill = end - p0 < st.page ? static_cast<int>(end - p0) : st.page;
  const int64_t tok0 = w.t0 + (p0 + first - len);               // token of row `first`
  const int64_t slab = (static_cast<int64_t>(id) * st.heads + h) * st.page;
  uint16_t* kp = st.k + slab * st.d;
  uint16_t* vp = st.v + slab * st.dv;
  const uint16_t* ks = k + tok0 * k_stride + static_cast<int64_t>(h) * st.d;
  const uint16_t* vs = v + tok0 * v_stride + static_cast<int64_t>(h) * st.dv;
  const int rows = fill - first;

  // The page's rows of one head lie one after the other.
  const int vc = st.dv / 8;
  uint4* v_out = reinterpret_cast<uint4*>(vp + static_cast<int64_t>(first) * st.dv);
  Split at_v(tid, kAppendThreads, vc);
#pragma unroll 4
  for (int i = tid; i < rows * vc; i += kAppendThreads, at_v.step())
    v_out[i] = __ldg(reinterpret_cast<const uint4*>(vs + at_v.q * v_stride) + at_v.r);
  const int nt = r.rot ? r.axes * r.nf : 0;
  const int items = nt / V, rest = (st.d - r.rot) / V;
  for (int b = 0; b < rows; b += kAppendRows) {
    const int m = rows - b < kAppendRows ? rows - b : kAppendRows;
    if (b) __syncthreads();
    if (nt) {
      Split at(tid, kAppendThreads, nt);
      for (int i = tid; i < m * nt; i += kAppendThreads, at.step()) {
        const int a = at.r >= r.nf ? 1 : 0;
        turns[i] = turn_of(r, __ldg(r.pos + (tok0 + b + at.q) * r.axes + a), at.r - a * r.nf);
      }
    }
    __syncthreads();
    if (nt) {
      Split at(tid, kAppendThreads, items);
      for (int i = tid; i < m * items; i += kAppendThreads, at.step())
        rotate_item<T, V>(ks + (b + at.q) * k_stride, kp + (first + b + at.q) * st.d, at.r, turns + at.q * nt, r);
    }
    if (rest) {
      Split at(tid, kAppendThreads, rest);
#pragma unroll 4
      for (int i = tid; i < m * rest; i += kAppendThreads, at.step()) {
        const int e = r.rot + at.r * V;
        *reinterpret_cast<typename Vec<V>::type*>(kp + (first + b + at.q) * st.d + e) =
            __ldg(reinterpret_cast<const typename Vec<V>::type*>(ks + (b + at.q) * k_stride + e));
      }
    }
  }
  if (!st.mean) return;
  // The mean over the page's rows as stored: the rows this block has written
  // come back from L2. Each thread sums every groups-th row of one 8-element
  // column; the groups are then added in order, so the sum does not depend on
  // the schedule.
  __syncthreads();
  const int cols = st.d / 8;
  const int groups = kAppendThreads / cols < 16 ? kAppendThreads / cols : 16;
  const int g = tid / cols, c = tid - g * cols;
  if (g < groups) {
    float acc[8] = {};
    for (int row = g; row < fill; row += groups) {
      Pack<8> p;
      p.v = *reinterpret_cast<const uint4*>(kp + static_cast<int64_t>(row) * st.d + c * 8);
      float f[8];
      unpack<T, 8>(p, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += f[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[(g * cols + c) * 8 + i] = acc[i];
  }
  __syncthreads();
  if (tid < st.d / 2) {
    float a0 = 0.f, a1 = 0.f;
    for (int q = 0; q < groups; ++q) {
      a0 += sums[q * st.d + 2 * tid];
      a1 += sums[q * st.d + 2 * tid + 1];
    }
    const float inv = static_cast<float>(fill);
    reinterpret_cast<uint32_t*>(st.mean + (static_cast<int64_t>(id) * st.heads + h) * st.d)[tid] =
        Half16<T>::pack(a0 / inv, a1 / inv);
  }
}

bool fits(const void* p, int64_t stride, int d, int v) {
  return reinterpret_cast<uintptr_t>(p) % (2 * v) == 0 && stride % v == 0 && d % v == 0;
}

template <typename T, int V>
int rotary_v(const uint16_t* x, int64_t x_stride, int64_t n, int heads, int d, const RotaryArgs& r,
             uint16_t* out, int64_t out_stride, cudaStream_t st) {
  const int nt = r.axes * r.nf;
  // About four items a thread, so that the angles of few heads are still
  // computed by a full block; at most 16 KB of angles.
  const int64_t per_token = static_cast<int64_t>(heads) * (nt / V);
  int64_t tokens = 4 * kThreads / (per_token > 0 ? per_token : 1);
  const int64_t most = 2048 / nt;
  if (tokens > most) tokens = most;
  // ... unless that leaves SMs without a block.
  if (tokens > n / 148) tokens = n / 148;
  if (tokens < 1) tokens = 1;
  const int64_t blocks = (n + tokens - 1) / tokens;
  if (blocks > INT32_MAX) return FASTNN_ERR_INVALID;
  rotary_kernel<T, V><<<static_cast<unsigned>(blocks), kThreads, tokens * nt * sizeof(float2), st>>>(
      x, x_stride, n, heads, d, r, out, out_stride, static_cast<int>(tokens));
  FASTNN_CUDA_TRY(cudaGetLastError());
  return FASTNN_OK;
}

template <typename T>
int rotary_t(const uint16_t* x, int64_t x_stride, int64_t n, int heads, int d, const RotaryArgs& r,
             uint16_t* out, int64_t out_stride, cudaStream_t st) {
  for (int v = 8; v > 1; v /= 2) {
    if (r.nf % v || !fits(x, x_stride, d, v) || !fits(out, out_stride, d, v)) continue;
    if (v == 8) return rotary_v<T, 8>(x, x_stride, n, heads, d, r, out, out_stride, st);
    if (v == 4) return rotary_v<T, 4>(x, x_stride, n, heads, d, r, out, out_stride, st);
    return rotary_v<T, 2>(x, x_stride, n, heads, d, r, out, out_stride, st);
  }
  return rotary_v<T, 1>(x, x_stride, n, heads, d, r, out, out_stride, st);
}

template <typename T, int V>
int append_v(const StoreArgs& a, const uint16_t* k, int64_t k_stride, const uint16_t* v,
             int64_t v_stride, int64_t n, int max_new, const RotaryArgs& r, int* status,
             cudaStream_t st) {
  const unsigned touched = static_cast<unsigned>((static_cast<int64_t>(max_new) + a.page - 2) / a.page + 1);
  const size_t smem = r.rot ? kAppendRows * r.axes * r.nf * sizeof(float2) : 0;
  append_kernel<T, V><<<dim3(touched, a.heads, a.n_seqs + (status != nullptr)), kAppendThreads, smem, st>>>(
      a, k, k_stride, v, v_stride, n, max_new, r, status);
  FASTNN_CUDA_TRY(cudaGetLastError());
  return FASTNN_OK;
}

template <typename T>
int append_t(const StoreArgs& a, const uint16_t* k, int64_t k_stride, const uint16_t* v,
             int64_t v_stride, int64_t n, int max_new, const RotaryArgs& r, int* status,
             cudaStream_t st) {
  const int nf = r.rot ? r.nf : 8;  // rows are 16-byte aligned: only the pairs' runs decide
  if (nf % 8 == 0) return append_v<T, 8>(a, k, k_stride, v, v_stride, n, max_new, r, status, st);
  if (nf % 4 == 0) return append_v<T, 4>(a, k, k_stride, v, v_stride, n, max_new, r, status, st);
  if (nf % 2 == 0) return append_v<T, 2>(a, k, k_stride, v, v_stride, n, max_new, r, status, st);
  return append_v<T, 1>(a, k, k_stride, v, v_stride, n, max_new, r, status, st);
}

}  // namespace

int launch_rotary(const uint16_t* x, int64_t x_stride, int64_t n, int heads, int d, int dtype,
                  const RotaryArgs& r, uint16_t* out, int64_t out_stride, cudaStream_t st) {
  return dtype == FASTNN_BF16
             ? rotary_t<__nv_bfloat16>(x, x_stride, n, heads, d, r, out, out_stride, st)
             : rotary_t<__half>(x, x_stride, n, heads, d, r, out, out_stride, st);
}

int launch_store_append(const StoreArgs& a, int dtype, const uint16_t* k, int64_t k_stride,
                        const uint16_t* v, int64_t v_stride, int64_t n, int max_new,
                        const RotaryArgs& r, int* status, cudaStream_t st) {
  return dtype == FASTNN_BF16
             ? append_t<__nv_bfloat16>(a, k, k_stride, v, v_stride, n, max_new, r, status, st)
             : append_t<__half>(a, k, k_stride, v, v_stride, n, max_new, r, status, st);
}

}  // namespace fastnn
