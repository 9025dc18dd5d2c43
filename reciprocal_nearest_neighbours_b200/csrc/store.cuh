// The token store: what its kernels share (arguments, index arithmetic,
// 16-bit float conversions). Entry points: store_api.cu.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "common.cuh"

namespace fastnn {

constexpr int kStatusStoreIndex = 2;  // bit set in the device status word: a token without a place

// fastnn_store as the kernels take it.
struct StoreArgs {
  uint16_t* k;
  uint16_t* v;
  uint16_t* mean;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* cu;
  int64_t n_pages;
  int n_seqs, width, page, page_log2, heads, d, dv;
};

struct RotaryArgs {
  const int32_t* pos;
  const double* freq;
  int axes, rot, nf;  // nf: frequencies of one axis, rot / (2 * axes)
  int interleaved;
  float scale;
  float sign;         // -1: the inverse
};

struct AttendArgs {
  StoreArgs st;
  const uint16_t* q;
  int64_t q_stride, n;
  int hq, group, max_new, causal;
  float scale_log2;      // scale * log2(e)
  const int32_t* pages;  // [n][heads][select] or nullptr
  int select;
  uint16_t* out;
  float* lse;
  float* part;           // [splits][n][hq][dv] partial outputs, normalised
  float* part_lse;       // [splits][n][hq] log2 of the partial sums
  int splits;
  int split_len;         // positions of one split (a multiple of 128); selected pages: entries
  int* status;
  uint64_t wait_ns;
};

struct SelectArgs {
  StoreArgs st;
  const uint16_t* q;
  int64_t q_stride, n;
  int hq, group, max_new, causal;
  int keep_first, keep_last, select;
  int32_t* out;
  uint64_t* keys;   // [n_seqs][slab][heads][width] of the slab's tokens
  double* sums;     // [n_seqs][slab][heads][d], chunks only
  int slab, first;  // tokens of a slab; first token (of each sequence) of this one
};

// The new tokens of sequence s: first token, how many are taken, and the
// length that the i-th of them sees is min(see0 + i * step, cap).
struct SeqView {
  int t0, n;
  int64_t see0;
  int step;
  int cap;
};
__device__ __forceinline__ SeqView seq_view(const StoreArgs& st, int s, int64_t n, int max_new,
                                            int causal) {
  SeqView w;
  const int a = __ldg(st.cu + s), b = __ldg(st.cu + s + 1), len = __ldg(st.lens + s);
  const int64_t m = static_cast<int64_t>(b) - a;
  w.t0 = a;
  int64_t take = m < max_new ? m : max_new;
  if (a < 0) take = 0;
  if (take > n - a) take = n - a;
  w.n = take > 0 ? static_cast<int>(take) : 0;
  w.cap = st.width * st.page;
  w.see0 = causal ? static_cast<int64_t>(len) - m + 1 : len;
  w.step = causal ? 1 : 0;
  return w;
}
__device__ __forceinline__ int visible(const SeqView& w, int i) {
  const int64_t v = w.see0 + static_cast<int64_t>(i) * w.step;
  return v < 0 ? 0 : v < w.cap ? static_cast<int>(v) : w.cap;
}

template <typename T>
struct Half16;
template <>
struct Half16<__nv_bfloat16> {
  static __device__ __forceinline__ float2 unpack(uint32_t x) {
    return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
  }
  static __device__ __forceinline__ float one(uint16_t x) {
    return __uint_as_float(static_cast<uint32_t>(x) << 16);
  }
  // Round to nearest, ties to even; lo in the low half.
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
};
template <>
struct Half16<__half> {
  static __device__ __forceinline__ float2 unpack(uint32_t x) {
    return __half22float2(*reinterpret_cast<const __half2*>(&x));
  }
  static __device__ __forceinline__ float one(uint16_t x) {
    return __half2float(*reinterpret_cast<const __half*>(&x));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
};

// Lets a kernel use `bytes` of dynamic shared memory on the current device; the
// attribute is set once a device (setting it takes as long as a small launch's
// other host work).
template <auto kKernel>
cudaError_t allow_smem(int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Launches a kernel that starts with cudaGridDependencySynchronize(): its
// blocks may be brought up while the stream's previous kernel drains.
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, dim3 block, cudaStream_t st, A&&... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// Launches clusters of `width` blocks along x.
template <typename... P, typename... A>
cudaError_t launch_cluster(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, unsigned width,
                           cudaStream_t st, A&&... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = width;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

int launch_rotary(const uint16_t* x, int64_t x_stride, int64_t n, int heads, int d, int dtype,
                  const RotaryArgs& r, uint16_t* out, int64_t out_stride, cudaStream_t st);
int launch_store_append(const StoreArgs& a, int dtype, const uint16_t* k, int64_t k_stride,
                        const uint16_t* v, int64_t v_stride, int64_t n, int max_new,
                        const RotaryArgs& r, int* status, cudaStream_t st);
// Splits of the few-rows kernel for a call; device-independent.
void attend_plan(AttendArgs& a);
int launch_attend_rows(const AttendArgs& a, int dtype, cudaStream_t st);
// The tensor-core kernel for chunks: which calls it takes (at least kTcRows query
// rows a sequence and key head; the caller's scale must be positive), and the
// floats of a.part that it needs. Rows 32 / 64 / 128, 16 sequences of 4096 positions, 8
// key heads of 128: 76 / 79 / 83 us, the few-rows kernel 77 / 126 / 186; one of 8192: 34 /
// 34 / 36 and 28 / 32 / 43; 8 of 4096, 12 heads of 64: 55 / 56 / 59 and 42 / 63 / 105.
// (Sequences of one batch had equally many rows; a long one takes the others along.)
constexpr int kTcRows = 64;
bool attend_tc_takes(const AttendArgs& a);
size_t attend_tc_floats(const AttendArgs& a);
int launch_attend_tc(const AttendArgs& a, int dtype, cudaStream_t st);
int launch_select(const SelectArgs& a, int dtype, cudaStream_t st);
size_t select_key_bytes(const StoreArgs& st, int max_new);
size_t select_sum_bytes(const StoreArgs& st, int max_new);
uint64_t wait_timeout_ns();  // the limit set by fastnn_set_wait_timeout_ns (0: the default)

}  // namespace fastnn
