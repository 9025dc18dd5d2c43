// Attention over the paged token store for chunks of new tokens, on the
// 5th-generation tensor cores.
//
// The mathematics is that of attend.cu: one pass over the keys with a running
// maximum and sum. Two things differ. The maximum m that the exponentials
// refer to need not be the largest score so far: O / l does not depend on m,
// and weights up to kMostSum are as exact in 16-bit floats as weights up to 1.
// So a tile's weights are formed with the m in force, and only if their sum is
// above kMostSum is the tile's maximum sought, m raised and O (in tensor
// memory) rescaled. The sum of that tile is then at most its 128 keys, so m
// rises by more than 1 each time and soon no more. And the tiles run from the
// last key to the first: those with masked places come first, the others run
// unmasked.
//
// One CTA per SM, warp-specialised. An item is 2 x 128 query rows (rows are
// (token, query head of the group), whole tokens only) of one sequence and key
// head with all their key tiles of 128:
//   warps 0-3, 4-7: softmax of query tile 0, 1. A thread owns a row: it reads
//       its 128 scores from tensor memory, and writes the 16-bit weights over
//       them (heads of up to 64: beside them), as the A operand of the second
//       product; no shuffles.
//   warp 8: loads. Query tiles by one TMA box (64 elements x group x tokens);
//       K and V tiles page by page (a lane each) into a ring of 128-row tiles.
//       Pages that do not exist and V rows behind the last visible position
//       are zeroed in shared memory (their scores are masked).
//   warp 10: walks the CTA's share of the work, a few items ahead of the others.
//   warp 9: one thread issues S = Q K^T (both operands K-major in shared
//       memory) and O += P V (P from tensor memory, V as an MN-major operand,
//       so that its rows are used as they lie in the store). While one query
//       tile is in its softmax the other's products run.
// The work is the sequence of all items' key tiles, cut into equal shares, one
// per CTA (an item costs kItemCost tiles extra). An item that a cut divides
// leaves normalised partial outputs, which merge_kernel joins.
// Bound by: exponentials (16 a clock and SM: 1024 clocks a tile of 128 x 128) and,
// at 128 elements a head, products (1024 clocks a tile too), whose phases overlap
// between the two query tiles in part. Measured: 2048 tokens over 16384, 32 / 8
// heads of 128, 431 us (1.2 PFLOP/s, tensor pipe 60% busy; 490 to 500 us under the
// power cap of a long run); 12288 rows over 196608 keys of 24, values of 8, 708 us
// (exponentials 70% busy); 8 x 576 tokens over up to 9792, 12 heads of 64, 174 us.
// The weights are rounded to the store's 16-bit type: the operands of a
// product have one type, and a second product for what the rounding loses would
// take half as much tensor time again.
// Every wait is bounded; on expiry the kernel records FASTNN_ERR_TIMEOUT,
// drains what it issued, frees its tensor memory and returns.
#include <cuda.h>

#include <type_traits>

#include "nn_tc.cuh"
#include "ptx.cuh"
#include "store.cuh"

namespace fastnn {

namespace {

constexpr int kLoadWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kPlanWarp = 10;
constexpr int kThreads = 384;      // three warpgroups: two of softmax, one of loads and products
// Registers of a softmax thread and of the others after the split:
// 256 x 216 + 128 x 72 = 384 x 168, the block's registers at launch.
constexpr int kSoftRegs = 216;
constexpr int kOtherRegs = 72;
constexpr int kBlk = 128;          // rows of a tile (queries, keys)
// An item's fixed cost (its queries, the first scores, the output), in key tiles.
// 8 images of 576 tokens, with 1 / 2 / 4 / 6: 181 / 177 / 174 / 176 us.
constexpr int kItemCost = 4;
constexpr int kLeastShare = 2;     // a CTA's share is at least this many tiles and that cost
constexpr float kMostSum = 256.f;
constexpr int kMaxCtas = 160;
constexpr int kHoleRing = 16;      // tiles whose missing pages are remembered

template <int DP>
struct Tc {
  static constexpr int kTile = kBlk * DP * 2;      // bytes of a Q, K or V tile
  static constexpr int kStages = DP == 128 ? 5 : 8;
  static constexpr int kRing = 2 * kTile;          // after the two query tiles
  static constexpr int kCtl = kRing + kStages * kTile;
  static constexpr int kBlock = kBlk * 128;        // bytes of a 64-element column block
  // Of every 16 pairs of weights, so many by polynomial (14 instructions a pair
  // against 16 clocks of the special-function unit). Measured with 0 / 1 / 2 /
  // 3 / 5: 12288 queries over 196608 keys of 24 731 / 731 / 706 / 712 / 749 us; 2048
  // over 16384, 32 heads of 128, 436 / 433 / 431 / 436 / 441 us. (Its upper bound
  // costs 10 to 15 us of the former; the largest argument by a maximum of three
  // instead took 4 more.)
  static constexpr int kPolyPairs = 2;
  // Tensor memory columns of query tile w: scores at 128 w, O at kO + DP w, the
  // weights (packed in pairs, 64 columns) at kP + kPStep w: over the scores where
  // all 512 columns are in use (DP = 128), else by themselves, so that the
  // next scores need not wait for the weights' product.
  static constexpr bool kOwnP = DP == 64;
  static constexpr uint32_t kO = 256, kP = kOwnP ? 384 : 0, kPStep = kOwnP ? 64 : 128;
};


constexpr int kMaxStages = 8;
constexpr int kSegRing = 4;        // segments the planning warp is ahead of the others
constexpr int kSegReaders = 10;    // warps that read a segment: softmax, loads, products

// A CTA's part of one item: key tiles [ja, jb) of its query rows.
struct Seg {
  int s, g;
  int tok, n;        // first token of the batch; the sequence's tokens from it on
  int ja, jb;        // jb < 0: no more segments
  int whole, first;  // all of the item's tiles; the share starts with it
  int64_t see;       // token i of the segment sees positions below see + i * step, at most cap
  int step, cap, vmax;
};
__device__ __forceinline__ int seg_visible(const Seg& e, int i) {
  const int64_t v = e.see + static_cast<int64_t>(i) * e.step;
  return v < 0 ? 0 : v < e.cap ? static_cast<int>(v) : e.cap;
}

// Where the loading warp stands at its end.
struct Loads {
  int stage, phase, fix_phase, segs;
  uint32_t open;  // stages that it has loaded; bit 31: a load on `fix` is under way
};

struct TcCtl {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t q_full, q_empty, fix, done;
  uint64_t s_full[2];   // scores are there
  uint64_t s_free[2];   // kOwnP: the scores have been read
  uint64_t p_full[2];   // the weights are there
  uint64_t pv_done[2];  // a tile's second product is complete (!kOwnP: a segment's last)
  uint64_t seg_full[kSegRing], seg_empty[kSegRing];
  Seg seg[kSegRing];
  uint32_t holes[kHoleRing];
  Loads loads;
  uint32_t tmem;
  int abort;
};

struct TcArgs {
  AttendArgs a;
  int tt;         // tokens of a query tile: floor(128 / group)
  int ppt_log2;   // log2 of a key tile's pages
  int ctas;
  float* part;    // [2 * ctas][256][dv]
  float* part_lse;
  struct Cut* cuts;  // [ctas]
};

// Where a CTA's share begins, for the merge.
struct alignas(16) Cut {
  int64_t u0, u1;    // the share
  int64_t base, end; // units of the item that it begins in
  int s, g, tile, pad;
};

// ---- the plan: items and shares ------------------------------------------------

__device__ __forceinline__ int item_count(const SeqView& w, int tt) { return (w.n + 2 * tt - 1) / (2 * tt); }
__device__ __forceinline__ int item_tiles(const SeqView& w, int tt, int tile) {
  int last = (tile + 1) * 2 * tt - 1;
  if (last >= w.n) last = w.n - 1;
  const int t = (visible(w, last) + kBlk - 1) / kBlk;
  return t > 0 ? t : 1;
}
// Key tiles among the first x units of an item (the fixed cost comes first).
__device__ __forceinline__ int tiles_of(int64_t x) { return x > kItemCost ? static_cast<int>(x - kItemCost) : 0; }

// Units of one key head of sequence s, by a whole warp.
__device__ __forceinline__ int64_t head_units(const SeqView& w, int tt, int lane) {
  int64_t sum = 0;
  const int items = item_count(w, tt);
  for (int i = lane; i < items; i += 32) sum += item_tiles(w, tt, i) + kItemCost;
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

struct Spot {
  int s, g, tile;
  int64_t at;  // units into the item
};

// The item that unit u lies in; totals[s]: inclusive prefix sums of the
// sequences' units. By a whole warp; every lane gets the answer.
__device__ Spot locate(const TcArgs& p, const int64_t* totals, int64_t u, int lane) {
  const AttendArgs& a = p.a;
  Spot r{a.st.n_seqs, 0, 0, 0};
  for (int s0 = 0; s0 < a.st.n_seqs; s0 += 32) {
    const bool past = s0 + lane < a.st.n_seqs && totals[s0 + lane] > u;
    const unsigned b = __ballot_sync(0xffffffffu, past);
    if (b) {
      r.s = s0 + __ffs(b) - 1;
      break;
    }
  }
  if (r.s >= a.st.n_seqs) return r;
  int64_t off = u - (r.s ? totals[r.s - 1] : 0);
  const SeqView w = seq_view(a.st, r.s, a.n, a.max_new, a.causal);
  const int64_t per = (totals[r.s] - (r.s ? totals[r.s - 1] : 0)) / a.st.heads;
  r.g = static_cast<int>(off / per);
  off -= r.g * per;
  const int items = item_count(w, p.tt);
  for (int i0 = 0; i0 < items; i0 += 32) {
    int64_t c = i0 + lane < items ? item_tiles(w, p.tt, i0 + lane) + kItemCost : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, c, o);
      if (lane >= o) c += y;
    }
    const unsigned b = __ballot_sync(0xffffffffu, c > off);
    if (b) {
      const int at = __ffs(b) - 1;
      const int64_t before = __shfl_sync(0xffffffffu, c, at > 0 ? at - 1 : 0);
      r.tile = i0 + at;
      r.at = off - (at > 0 ? before : 0);
      return r;
    }
    off -= __shfl_sync(0xffffffffu, c, 31);
  }
  return r;
}

// Prefix sums of the sequences' units into totals, by `warps` warps of the
// block; returns the number of CTAs that share the work.
__device__ int plan(const TcArgs& p, int64_t* totals, int warp, int warps, int lane) {
  const AttendArgs& a = p.a;
  for (int s = warp; s < a.st.n_seqs; s += warps) {
    const SeqView w = seq_view(a.st, s, a.n, a.max_new, a.causal);
    const int64_t u = head_units(w, p.tt, lane) * a.st.heads;
    if (lane == 0) totals[s] = u;
  }
  __syncthreads();
  if (warp == 0) {
    int64_t base = 0;
    for (int s0 = 0; s0 < a.st.n_seqs; s0 += 32) {
      int64_t c = s0 + lane < a.st.n_seqs ? totals[s0 + lane] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, c, o);
        if (lane >= o) c += y;
      }
      if (s0 + lane < a.st.n_seqs) totals[s0 + lane] = base + c;
      base += __shfl_sync(0xffffffffu, c, 31);
    }
  }
  __syncthreads();
  const int64_t units = totals[a.st.n_seqs - 1];
  const int64_t most = units / (kLeastShare + kItemCost);
  return most < 1 ? 1 : most < p.ctas ? static_cast<int>(most) : p.ctas;
}
__device__ __forceinline__ int64_t share_start(int64_t units, int c, int ctas) {
  return units * c / ctas;
}

// ---- instructions ---------------------------------------------------------------

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ float2 halves(uint64_t x) {
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(x));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// 2^x of two numbers without the special-function unit: x = j + f with j the
// nearest whole number (the sum with 1.5 * 2^23 leaves it in the low mantissa
// bits), 2^f by its minimax polynomial of degree 5 on [-1/2, 1/2] (found by
// Remez exchange on the relative error; in fp32 2^-22.2, as good as the unit's),
// and j added to the exponent, which holds for x in [-126, 127]. Below, the result
// is 2^-126, nothing beside a row's largest weight of at least 2^-8. Above 8 =
// log2(kMostSum) any large result serves, since the tile's weights are formed
// anew by the unit then: 2^kPolyMost stands for all x beyond (a key may score any
// amount above the maximum in force), and for NaN, which fminf drops.
constexpr float kPolyMost = 64.f;
__device__ __forceinline__ float2 ex2_pair(uint64_t x) {
  float2 v = halves(x);
  x = pair(fmaxf(fminf(v.x, kPolyMost), -126.f), fmaxf(fminf(v.y, kPolyMost), -126.f));
  const uint64_t magic = pair(12582912.f, 12582912.f);
  const uint64_t t = add2(x, magic);
  const uint64_t f = sub2(x, sub2(t, magic));
  uint64_t q = pair(0.0013276472454890609f, 0.0013276472454890609f);
  q = fma2(q, f, pair(0.009675540961325169f, 0.009675540961325169f));
  q = fma2(q, f, pair(0.05550713092088699f, 0.05550713092088699f));
  q = fma2(q, f, pair(0.24022120237350464f, 0.24022120237350464f));
  q = fma2(q, f, pair(0.6931469440460205f, 0.6931469440460205f));
  q = fma2(q, f, pair(1.0000001192092896f, 1.0000001192092896f));
  const float2 w = halves(q), e = halves(t);
  return make_float2(__uint_as_float(__float_as_uint(w.x) + (__float_as_uint(e.x) << 23)),
                     __uint_as_float(__float_as_uint(w.y) + (__float_as_uint(e.y) << 23)));
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, int x, int y, int z,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem], 16-bit floats -> fp32.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// This thread's row, 16 (32) consecutive 32-bit columns.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31])
      : "memory");
}
// True in one lane of the (converged) warp, always the same one.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Descriptor of an MN-major operand in 128-byte swizzled 64-element column
// blocks: rows (the K index) of 128 bytes, 8-row groups 1024 bytes apart, column
// blocks kBlock bytes apart.
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t saddr, uint32_t block) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFF) | (static_cast<uint64_t>(block >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// Bounded wait for a phase; false, with the abort flag and the status set, if
// `limit` ns pass or another role has given up. A suspended test may take
// longer than a short limit; POLL: such limits (below kPolledLimit) are watched by
// polling, in a kernel of their own.
// (Inlined: a call would have to be possible within either register share.)
constexpr uint64_t kPolledLimit = 10000000;
template <bool POLL>
__device__ __forceinline__ bool phase_done(uint32_t bar, uint32_t parity) {
  return POLL ? ptx::mbar_test_wait(bar, parity) : ptx::mbar_try_wait(bar, parity);
}
template <bool POLL>
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, TcCtl* ctl, int* status,
                                         uint64_t limit) {
  if (phase_done<POLL>(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer_ns();
  for (uint32_t n = 1;; ++n) {
    if (phase_done<POLL>(bar, parity)) return true;
    if (POLL || (n & 63) == 0 || n == 8) {
      if (*reinterpret_cast<volatile int*>(&ctl->abort)) return false;
      if (ptx::globaltimer_ns() - t0 > limit) {
        *reinterpret_cast<volatile int*>(&ctl->abort) = 1;
        atomicOr(status, kStatusTimeout);
        return false;
      }
    }
  }
}

// ---- the kernel -----------------------------------------------------------------

template <typename T, int DP, bool POLL>
__global__ void __launch_bounds__(kThreads, 1)
attend_tc_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                 const __grid_constant__ CUtensorMap vmap, const __grid_constant__ TcArgs p) {
  using C = Tc<DP>;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t{1023});
  TcCtl* ctl = reinterpret_cast<TcCtl*>(smem + C::kCtl);
  const AttendArgs& a = p.a;
  const StoreArgs& st = a.st;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sbase = ptx::smem_u32(smem);
  const uint64_t limit = wait_limit(a.wait_ns);
  auto bar = [&](uint64_t& b) { return ptx::smem_u32(&b); };

  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      ptx::mbar_init(bar(ctl->full[i]), 1);
      ptx::mbar_init(bar(ctl->empty[i]), 1);
    }
    ptx::mbar_init(bar(ctl->q_full), 1);
    ptx::mbar_init(bar(ctl->q_empty), 1);
    ptx::mbar_init(bar(ctl->fix), 1);
    ptx::mbar_init(bar(ctl->done), 1);
    for (int w = 0; w < 2; ++w) {
      ptx::mbar_init(bar(ctl->s_full[w]), 1);
      ptx::mbar_init(bar(ctl->p_full[w]), 4);
      ptx::mbar_init(bar(ctl->s_free[w]), 4);
      ptx::mbar_init(bar(ctl->pv_done[w]), 1);
    }
    for (int i = 0; i < kSegRing; ++i) {
      ptx::mbar_init(bar(ctl->seg_full[i]), 1);
      ptx::mbar_init(bar(ctl->seg_empty[i]), kSegReaders);
    }
    ctl->abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(ptx::smem_u32(&ctl->tmem), 512);
    ptx::tmem_relinquish();
  }
  // The plan's prefix sums lie where the ring will be.
  int64_t* totals = reinterpret_cast<int64_t*>(smem + C::kRing);
  const int ctas = plan(p, totals, warp, kThreads / 32, lane);
  // The plan warp finds this CTA's share before the ring is written to.
  int64_t u = 0, left = 0;
  Spot at{};
  if (warp == kPlanWarp) {
    const int64_t units = totals[st.n_seqs - 1];
    const int c = blockIdx.x;
    if (c < ctas) {
      u = share_start(units, c, ctas);
      left = share_start(units, c + 1, ctas) - u;
    }
    if (left > 0) at = locate(p, totals, u, lane);
    if (lane == 0) {
      Cut cut{u, u + left, u - at.at, 0, at.s, at.g, at.tile, 0};
      if (left > 0)
        cut.end = cut.base + kItemCost +
                  item_tiles(seq_view(st, at.s, a.n, a.max_new, a.causal), p.tt, at.tile);
      p.cuts[blockIdx.x] = cut;
    }
  }
  ptx::fence_proxy_async_smem();  // totals are read; TMA writes there next
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  // The same in every lane, and told so to the compiler: the MMA issuer's
  // descriptors can then stay in uniform registers.
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl->tmem, 0);
  // Segment k of the share, copied from the ring; false at the end of the
  // share (or when a wait ran out).
  auto segment = [&](int k, Seg& e) {
    const int i = k & (kSegRing - 1);
    if (!__all_sync(0xffffffffu, wait_for<POLL>(bar(ctl->seg_full[i]), (k / kSegRing) & 1, ctl, a.status, limit)))
      return false;
    e = ctl->seg[i];
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(bar(ctl->seg_empty[i]));
    return e.jb >= 0;
  };
  const int ppt = 1 << p.ppt_log2;
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    const int w = warp >> 2, r = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + w * 128, to = tmem + lanes + C::kO + w * DP;
    const uint32_t tp = tmem + lanes + C::kP + w * C::kPStep;
    const int nvb = (st.dv + 63) / 64;
    const uint64_t scale2 = pair(a.scale_log2, a.scale_log2);
    uint32_t sp = 0, pd = 1;  // parities: of s_full, and of pv_done's last completed phase
    int tiles = 0;
    Seg e;
    for (int k = 0; segment(k, e); ++k) {
      const int nt = e.jb - e.ja;
      if (w * p.tt >= e.n) {  // this query tile has no row
        tiles += nt;
        continue;
      }
      const int tok = w * p.tt + r / a.group;
      const bool real = r < p.tt * a.group && tok < e.n;
      const int vis = real ? seg_visible(e, tok) : e.vmax;
      const int vmin = __reduce_min_sync(0xffffffffu, vis);
      bool ok = true;
      float m = -INFINITY, l = 0.f;
      for (int t = 0; t < nt; ++t, ++tiles) {
        const int k0 = (e.jb - 1 - t) * kBlk;
        ok = __all_sync(0xffffffffu, wait_for<POLL>(bar(ctl->s_full[w]), sp, ctl, a.status, limit));
        sp ^= 1;
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t holes = ctl->holes[tiles & (kHoleRing - 1)];
        const bool edge = k0 + kBlk > vmin || holes;
        uint32_t x[4][32];
        uint32_t pk[4][16];
        auto load = [&]() {
#pragma unroll
          for (int c = 0; c < 4; ++c) ptx::tmem_ld32(ts + c * 32, x[c]);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < 4; ++c) ptx::pin_regs(x[c]);
        };
        // The weights with the maximum in force, packed; returns their sum.
        auto weigh = [&](auto poly) {
          const float z = m == -INFINITY ? 0.f : -m;
          const uint64_t z2 = pair(z, z);
          uint64_t sum[2] = {0, 0};
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const uint64_t u = fma2(pair(__uint_as_float(x[c][2 * i]), __uint_as_float(x[c][2 * i + 1])),
                                      scale2, z2);
              float2 v;
              if (i < decltype(poly)::value) {
                v = ex2_pair(u);
              } else {
                v = halves(u);
                v = make_float2(ex2(v.x), ex2(v.y));
              }
              sum[i & 1] = add2(sum[i & 1], pair(v.x, v.y));
              pk[c][i] = Half16<T>::pack(v.x, v.y);
            }
          const float2 y = halves(add2(sum[0], sum[1]));
          return y.x + y.y;
        };
        load();
        // Most tiles need no maximum of their own: while their weights, by the
        // maximum in force, sum to no more than kMostSum, none of them is larger.
        // Rows that are no token's have no say: what lies there (another
        // sequence's queries, whatever shared memory held) must not decide how
        // the others' weights are formed.
        float sum = 0.f;
        bool again = edge || t == 0;
        if (!again) {
          sum = weigh(std::integral_constant<int, C::kPolyPairs>{});
          again = __any_sync(0xffffffffu, real && (sum > kMostSum || m == -INFINITY));
        }
        if (again) {
          load();  // the scores are still there: the weights have not been stored
          if (edge) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const int key = c * 32 + i;
                if (k0 + key >= vis || ((holes >> (key >> st.page_log2)) & 1u))
                  x[c][i] = __float_as_uint(-INFINITY);
              }
          }
          float top[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            top[c] = fmaxf(__uint_as_float(x[c][0]), __uint_as_float(x[c][1]));
#pragma unroll
            for (int i = 2; i < 32; i += 2)
              top[c] = ptx::fmax3(top[c], __uint_as_float(x[c][i]), __uint_as_float(x[c][i + 1]));
          }
          const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * a.scale_log2;
          if (__any_sync(0xffffffffu, real && mx > m)) {
            // Raise the maximum, and scale what was summed with the one before.
            const float up = fmaxf(m, mx);
            const float f = m == up ? 1.f : ex2(m - up);
            l *= f;
            m = up;
            if (t > 0) {
              if (C::kOwnP)
                ok = __all_sync(0xffffffffu, wait_for<POLL>(bar(ctl->pv_done[w]), pd, ctl, a.status, limit));
              ptx::tc_fence_after();
              for (int c = 0; c < nvb * 2; ++c) {
                uint32_t o[32];
                ptx::tmem_ld32(to + c * 32, o);
                ptx::tmem_ld_wait_regs(o);
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                tmem_st32(to + c * 32, o);
              }
            }
          }
          sum = weigh(std::integral_constant<int, 0>{});
        }
        l += sum;
        if (C::kOwnP) {
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar(ctl->s_free[w]));
          if (t > 0) {  // the weights before these have been used
            ok = ok && __all_sync(0xffffffffu, wait_for<POLL>(bar(ctl->pv_done[w]), pd, ctl, a.status, limit));
            ptx::tc_fence_after();
          }
          if (!ok) break;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_st16(tp + c * 16, pk[c]);
        tmem_st_wait();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(ctl->p_full[w]));
        if (C::kOwnP) pd ^= 1;
      }
      if (!ok) break;
      if (!C::kOwnP) pd ^= 1;
      ok = __all_sync(0xffffffffu, wait_for<POLL>(bar(ctl->pv_done[w]), pd, ctl, a.status, limit));
      if (!ok) break;
      ptx::tc_fence_after();
      const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
      const float lse2 = l > 0.f ? m + log2f(l) : l == 0.f ? -INFINITY : l;
      const bool whole = e.whole;
      const int64_t row = (static_cast<int64_t>(e.tok) + tok) * a.hq + e.g * a.group + r % a.group;
      const int slot = 2 * blockIdx.x + (e.first ? 0 : 1);
      float* part = p.part + (static_cast<int64_t>(slot) * 256 + w * 128 + r) * st.dv;
      for (int c = 0; c < nvb * 2; ++c) {
        uint32_t o[32];
        ptx::tmem_ld32(to + c * 32, o);
        ptx::tmem_ld_wait_regs(o);
        if (!real) continue;
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
          if (c * 32 + i >= st.dv) break;
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(o[i + e]) * inv;
          if (whole) {
            *reinterpret_cast<uint4*>(a.out + row * st.dv + c * 32 + i) =
                make_uint4(Half16<T>::pack(f[0], f[1]), Half16<T>::pack(f[2], f[3]),
                           Half16<T>::pack(f[4], f[5]), Half16<T>::pack(f[6], f[7]));
          } else {
            *reinterpret_cast<float4*>(part + c * 32 + i) = make_float4(f[0], f[1], f[2], f[3]);
            *reinterpret_cast<float4*>(part + c * 32 + i + 4) = make_float4(f[4], f[5], f[6], f[7]);
          }
        }
      }
      if (real) {
        if (!whole) {
          p.part_lse[slot * 256 + w * 128 + r] = lse2;
        } else if (a.lse) {
          a.lse[row] = lse2 * 0.69314718055994530942f;
        }
      }
      ptx::tc_fence_before();  // O is read before this thread hands over the next weights
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kLoadWarp) {
      int stage = 0;
      uint32_t phase = 0, fix_phase = 0, q_phase = 0;
      int tiles = 0, segs = 0;
      const int nkb = (st.d + 63) / 64, nvb = (st.dv + 63) / 64;
      uint32_t open_stages = 0;  // see Loads
      bool ok = true;
      Seg e;
      while (segment(segs, e)) {
        const bool two = p.tt < e.n;
        const int vmax = e.vmax;
        if (segs > 0) {
          ok = __all_sync(0xffffffffu, wait_for<POLL>(bar(ctl->q_empty), q_phase, ctl, a.status, limit));
          q_phase ^= 1;
          if (!ok) break;
        }
        if (lane == 0) {
          const uint32_t rows = static_cast<uint32_t>(p.tt * a.group);
          ptx::mbar_arrive_expect_tx(bar(ctl->q_full), (two ? 2u : 1u) * nkb * rows * 128u);
          for (int q = 0; q < (two ? 2 : 1); ++q)
            for (int b = 0; b < nkb; ++b)
              tma_load_3d(sbase + q * C::kTile + b * C::kBlock, &qmap, b * 64, e.g * a.group,
                          e.tok + q * p.tt, bar(ctl->q_full));
        }
        ++segs;
        // Lane i < ppt has page i of a tile; -1: no such page, or none of its
        // positions is visible. Read a tile ahead.
        auto page_id = [&](int j) {
          const int lp = (j << p.ppt_log2) + lane;
          return j >= e.ja && lane < ppt && lp < st.width && (lp << st.page_log2) < vmax
                     ? __ldg(st.table + static_cast<int64_t>(e.s) * st.width + lp)
                     : -1;
        };
        int id_next = page_id(e.jb - 1);
        for (int j = e.jb - 1; j >= e.ja; --j, ++tiles) {
          int id = id_next;
          if (id >= st.n_pages) id = -1;
          id_next = page_id(j - 1);
          const unsigned there = __ballot_sync(0xffffffffu, lane < ppt && id >= 0);
          const unsigned every = ppt == 32 ? 0xffffffffu : (1u << ppt) - 1u;
          const bool fix = there != every || (j + 1) * kBlk > vmax;
          const int pages = __popc(there);
          if (lane == 0) ctl->holes[tiles & (kHoleRing - 1)] = ~there & every;
          for (int kv = 0; kv < 2; ++kv) {
            ok = __all_sync(0xffffffffu,
                            wait_for<POLL>(bar(ctl->empty[stage]), phase ^ 1u, ctl, a.status, limit));
            if (!ok) break;
            const uint32_t dst = sbase + C::kRing + stage * C::kTile;
            const int blocks = kv ? nvb : nkb;
            const bool mend = kv && fix;  // V rows that no score may reach with NaN
            const uint32_t mb = mend ? bar(ctl->fix) : bar(ctl->full[stage]);
            if (lane == 0) ptx::mbar_arrive_expect_tx(mb, pages * blocks * st.page * 128u);
            __syncwarp();
            if (lane < ppt && id >= 0)
              for (int b = 0; b < blocks; ++b)
                tma_load_3d(dst + b * C::kBlock + ((lane << st.page_log2) * 128), kv ? &vmap : &kmap,
                            b * 64, 0, id * st.heads + e.g, mb);
            if (!mend) {
              open_stages |= 1u << stage;
            } else {
              ok = __all_sync(0xffffffffu, wait_for<POLL>(mb, fix_phase, ctl, a.status, limit));
              if (!ok) {  // the copies in flight are waited for before the kernel ends
                open_stages |= 1u << 31;
                break;
              }
              fix_phase ^= 1;
              // Four rows of 128 bytes at a time, 16 bytes a lane.
              const int from = there == every ? (vmax > j * kBlk ? vmax - j * kBlk : 0) : 0;
              for (int r = (from & ~3) + (lane >> 3); r < kBlk; r += 4) {
                if (j * kBlk + r < vmax && ((there >> (r >> st.page_log2)) & 1u)) continue;
                for (int b = 0; b < blocks; ++b)
                  *reinterpret_cast<uint4*>(smem + C::kRing + stage * C::kTile + b * C::kBlock + r * 128 +
                                            (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
              }
              ptx::fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) ptx::mbar_arrive(bar(ctl->full[stage]));
            }
            if (++stage == C::kStages) {
              stage = 0;
              phase ^= 1;
            }
          }
          if (!ok) break;
        }
        if (!ok) break;
      }
      if (lane == 0) ctl->loads = Loads{stage, static_cast<int>(phase), static_cast<int>(fix_phase), segs, open_stages};
    } else if (warp == kMmaWarp) {
      // The whole warp waits; one elected lane issues.
      const bool leader = elect_one();
      constexpr uint32_t kFmt = std::is_same<T, __half>::value ? 0u : 1u;
      const uint32_t nvb = (st.dv + 63) / 64;
      const uint32_t idesc_s = (1u << 4) | (kFmt << 7) | (kFmt << 10) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
      const uint32_t idesc_o = (1u << 4) | (kFmt << 7) | (kFmt << 10) | (1u << 16) |
                               ((nvb * 64u >> 3) << 17) | ((128u >> 4) << 24);
      const int ksteps = (st.d + 15) / 16;
      int stage = 0;
      uint32_t phase = 0;
      uint32_t pp = 0;  // bit w: the parity that p_full[w] (and s_free[w]) completes next
      auto await = [&](uint64_t& b, uint32_t parity) {
        return __all_sync(0xffffffffu, wait_for<POLL>(bar(b), parity, ctl, a.status, limit));
      };
      auto product_s = [&](int w, int kstage) {
        const uint64_t qd = ptx::smem_desc_kmajor(sbase + w * C::kTile, 128);
        const uint64_t kd = ptx::smem_desc_kmajor(sbase + C::kRing + kstage * C::kTile, 128);
  #pragma unroll
        for (int ks = 0; ks < DP / 16; ++ks) {
          if (ks >= ksteps) break;
          const uint32_t off = ((ks >> 2) * C::kBlock + (ks & 3) * 32) >> 4;
          ptx::mma_bf16(tmem + w * 128, qd + off, kd + off, idesc_s, ks > 0 ? 1u : 0u);
        }
        ptx::mma_commit(bar(ctl->s_full[w]));
      };
      auto product_o = [&](int w, int vstage, bool fresh) {
        const uint64_t vd = smem_desc_mn(sbase + C::kRing + vstage * C::kTile, C::kBlock);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          mma_ts(tmem + C::kO + w * DP, tmem + C::kP + w * C::kPStep + ks * 8, vd + ks * (2048 >> 4), idesc_o,
                 (fresh && ks == 0) ? 0u : 1u);
      };
      auto step = [&]() {
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1;
        }
      };
      Seg e;
      for (int k = 0; segment(k, e); ++k) {
        const int nw = p.tt < e.n ? 2 : 1, nt = e.jb - e.ja;
        if (!await(ctl->q_full, k & 1) || !await(ctl->full[stage], phase)) break;
        ptx::tc_fence_after();
        if (leader) {
          for (int w = 0; w < nw; ++w) product_s(w, stage);
          ptx::mma_commit(bar(ctl->empty[stage]));
          if (nt == 1) ptx::mma_commit(bar(ctl->q_empty));
        }
        step();
        bool ok = true;
        for (int t = 0; t < nt; ++t) {
          if (!(ok = await(ctl->full[stage], phase))) break;
          const int vstage = stage;
          step();
          const bool more = t + 1 < nt;
          if (more && !(ok = await(ctl->full[stage], phase))) break;
          for (int w = 0; w < nw; ++w) {
            if (C::kOwnP) {
              if (!(ok = await(ctl->s_free[w], (pp >> w) & 1u))) break;
              ptx::tc_fence_after();
              if (leader && more) product_s(w, stage);
            }
            if (!(ok = await(ctl->p_full[w], (pp >> w) & 1u))) break;
            pp ^= 1u << w;
            ptx::tc_fence_after();
            if (leader) {
              product_o(w, vstage, t == 0);
              if (C::kOwnP || !more) ptx::mma_commit(bar(ctl->pv_done[w]));
              if (!C::kOwnP && more) product_s(w, stage);
            }
          }
          if (!ok) break;
          if (leader) {
            ptx::mma_commit(bar(ctl->empty[vstage]));
            if (more) {
              ptx::mma_commit(bar(ctl->empty[stage]));
              if (t + 2 == nt) ptx::mma_commit(bar(ctl->q_empty));
            }
          }
          if (more) step();
        }
        if (!ok) break;
      }
      // Everything issued is complete before the tensor memory goes back.
      if (leader) {
        ptx::mma_commit(bar(ctl->done));
        const uint64_t t0 = ptx::globaltimer_ns();
        while (!ptx::mbar_try_wait(bar(ctl->done), 0) && ptx::globaltimer_ns() - t0 < kTimeoutNs) {
        }
      }
      __syncwarp();
    } else if (warp == kPlanWarp) {
      // Walks the share's items and hands out their segments.
      if (lane == 0) {
        SeqView w{};
        int items = 0, k = 0;
        if (left > 0) {
          w = seq_view(st, at.s, a.n, a.max_new, a.causal);
          items = item_count(w, p.tt);
        }
        bool first = true;
        for (bool more = true; more;) {
          Seg e;
          e.jb = -1;
          more = left > 0;
          if (more) {
            const int kt = item_tiles(w, p.tt, at.tile);
            const int64_t cost = kt + kItemCost;
            const int64_t end = at.at + left < cost ? at.at + left : cost;
            const int i0 = at.tile * 2 * p.tt;
            e.s = at.s;
            e.g = at.g;
            e.tok = w.t0 + i0;
            e.n = w.n - i0;
            e.ja = tiles_of(at.at);
            e.jb = tiles_of(end);
            e.whole = e.ja == 0 && e.jb == kt;
            e.first = first;
            e.see = w.see0 + static_cast<int64_t>(i0) * w.step;
            e.step = w.step;
            e.cap = w.cap;
            e.vmax = seg_visible(e, (e.n < 2 * p.tt ? e.n : 2 * p.tt) - 1);
            first = false;
            left -= end - at.at;
            at.at = 0;
            if (left > 0 && ++at.tile == items) {  // the next head, the next sequence with tokens
              at.tile = 0;
              if (++at.g == st.heads) {
                at.g = 0;
                do {
                  ++at.s;
                  w = seq_view(st, at.s, a.n, a.max_new, a.causal);
                  items = item_count(w, p.tt);
                } while (items == 0 && at.s + 1 < st.n_seqs);
              }
            }
            if (e.jb <= e.ja) continue;  // the item's fixed cost alone
          }
          const int i = k & (kSegRing - 1);
          if (!wait_for<POLL>(bar(ctl->seg_empty[i]), ((k / kSegRing) & 1) ^ 1, ctl, a.status, limit)) break;
          ctl->seg[i] = e;
          ptx::mbar_arrive(bar(ctl->seg_full[i]));
          ++k;
        }
      }
      __syncwarp();
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (tid == 0 && ctl->abort) {
    // Some role has given up, and copies may be under way that nobody waits for
    // any more: the block stays until their bytes are there (within the default
    // limit). A stage's last load completes the phase after its last wait on `empty`.
    const Loads d = ctl->loads;
    const uint64_t t0 = ptx::globaltimer_ns();
    auto drain = [&](uint64_t& b, uint32_t parity) {
      while (!ptx::mbar_test_wait(bar(b), parity) && ptx::globaltimer_ns() - t0 < kTimeoutNs) {
      }
    };
    for (int i = 0; i < C::kStages; ++i)
      if ((d.open >> i) & 1u) drain(ctl->full[i], static_cast<uint32_t>(i < d.stage ? d.phase : d.phase ^ 1));
    if (d.open >> 31) drain(ctl->fix, static_cast<uint32_t>(d.fix_phase));
    if (d.segs > 0) drain(ctl->q_full, static_cast<uint32_t>((d.segs - 1) & 1));
  }
  __syncthreads();
  if (warp == kMmaWarp) ptx::tmem_dealloc(tmem, 512);
}

// Joins the partial outputs of the items that a share's border divides. Block
// (c, i) looks at the border before CTA c + 1 and takes every gridDim.y-th group
// of rows of its item, if the item's first cut is there. A warp takes a row; its
// lanes look at the CTAs c, c + 1, ... that may have a part, 32 at a time.
template <typename T>
__global__ void __launch_bounds__(256)
merge_kernel(const __grid_constant__ TcArgs p) {
  cudaGridDependencySynchronize();
  const AttendArgs& a = p.a;
  const StoreArgs& st = a.st;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x;
  const Cut sp = p.cuts[c + 1];
  if (sp.u0 >= sp.u1 || sp.u0 == sp.base || p.cuts[c].u0 > sp.base) return;
  const SeqView w = seq_view(st, sp.s, a.n, a.max_new, a.causal);
  const int64_t base = sp.base, end = sp.end;
  // Lane's slot of partial outputs among CTAs k0 .. k0 + 31, -1: none.
  auto slot_of = [&](int k0) {
    const int k = k0 + lane;
    if (k >= p.ctas) return -1;
    const Cut cut = p.cuts[k];
    const bool part = cut.u0 < end && cut.u0 < cut.u1 &&
                      tiles_of((cut.u1 < end ? cut.u1 : end) - base) > tiles_of(cut.u0 > base ? cut.u0 - base : 0);
    return part ? 2 * k + (cut.u0 < base ? 1 : 0) : -1;
  };
  int windows = 0, parts = 0;
  const int first = slot_of(c);
  for (int k0 = c; k0 < p.ctas; k0 += 32) {
    const int found = __popc(__ballot_sync(0xffffffffu, (k0 == c ? first : slot_of(k0)) >= 0));
    if (found) {
      parts += found;
      windows = (k0 - c) / 32 + 1;
    }
  }
  if (parts <= 1) return;  // one CTA had all its tiles
  const int i0 = sp.tile * 2 * p.tt;
  for (int rr = blockIdx.y * 8 + warp; rr < 256; rr += gridDim.y * 8) {
    const int q = rr >> 7, r = rr & 127;
    const int tok = i0 + q * p.tt + r / a.group;
    if (r >= p.tt * a.group || tok >= w.n) continue;
    const int64_t row = (static_cast<int64_t>(w.t0) + tok) * a.hq + sp.g * a.group + r % a.group;
    float top = -INFINITY, sum = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int x = 0; x < windows; ++x) {
      const int slot = x == 0 ? first : slot_of(c + 32 * x);
      const float z = slot >= 0 ? p.part_lse[slot * 256 + rr] : -INFINITY;
      float up = fmaxf(top, z);
#pragma unroll
      for (int o = 16; o; o >>= 1) up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, o));
      if (!__any_sync(0xffffffffu, z != -INFINITY)) continue;  // NaN is a part, too: fmaxf drops it
      const float old = top == -INFINITY ? 0.f : ex2(top - up);
      sum *= old;
      v.x *= old;
      v.y *= old;
      v.z *= old;
      v.w *= old;
      top = up;
      const float f = z == -INFINITY ? 0.f : ex2(z - up);
      unsigned some = __ballot_sync(0xffffffffu, slot >= 0);
      while (some) {
        const int k = __ffs(some) - 1;
        some &= some - 1;
        const float fk = __shfl_sync(0xffffffffu, f, k);
        const int sk = __shfl_sync(0xffffffffu, slot, k);
        sum += fk;
        if (lane * 4 < st.dv) {
          const float4 y = *reinterpret_cast<const float4*>(
              p.part + (static_cast<int64_t>(sk) * 256 + rr) * st.dv + lane * 4);
          v.x += fk * y.x;
          v.y += fk * y.y;
          v.z += fk * y.z;
          v.w += fk * y.w;
        }
      }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    if (lane * 4 < st.dv)
      *reinterpret_cast<uint2*>(a.out + row * st.dv + lane * 4) =
          make_uint2(Half16<T>::pack(v.x * inv, v.y * inv), Half16<T>::pack(v.z * inv, v.w * inv));
    if (lane == 0 && a.lse)
      a.lse[row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994530942f;
  }
}

// ---- host ------------------------------------------------------------------------

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn get_encode() {
  static const EncodeFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeFn>(f);
  }();
  return fn;
}

// Boxes of 64 x b1 x b2 elements of a [n2][n1][n0] array of 16-bit floats.
int make_map(CUtensorMap* m, bool bf16, const void* base, uint64_t n0, uint64_t n1, uint64_t n2,
             uint64_t stride1, uint64_t stride2, uint32_t b1, uint32_t b2) {
  EncodeFn enc = get_encode();
  if (!enc) return FASTNN_ERR_CUDA;
  const cuuint64_t dims[3] = {n0, n1, n2};
  const cuuint64_t strides[2] = {stride1 * 2, stride2 * 2};
  const cuuint32_t box[3] = {64, b1, b2};
  const cuuint32_t one[3] = {1, 1, 1};
  const CUresult r = enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                         3, const_cast<void*>(base), dims, strides, box, one,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FASTNN_OK : FASTNN_ERR_CUDA;
}

constexpr int kMaxSeqs = 512;  // of one launch: the plan's sums fit beside the queries

template <typename T, int DP>
int tc_launch(const AttendArgs& all, cudaStream_t stream) {
  using C = Tc<DP>;
  constexpr int kSmem = 1024 + C::kCtl + static_cast<int>(sizeof(TcCtl));
  static_assert(kSmem <= 227 * 1024, "shared memory of an SM");
  static_assert(C::kStages <= kMaxStages && kMaxSeqs * 8 <= C::kTile, "layout");
  const bool bf16 = std::is_same<T, __nv_bfloat16>::value;
  int sms = 0;
  const int rc = device_sm_count(&sms);
  if (rc != FASTNN_OK) return rc;
  TcArgs p{};
  p.a = all;
  p.tt = kBlk / all.group;
  p.ppt_log2 = 7 - all.st.page_log2;
  p.ctas = sms < kMaxCtas ? sms : kMaxCtas;
  p.part = all.part;
  p.part_lse = all.part + static_cast<int64_t>(2) * kMaxCtas * 256 * all.st.dv;
  p.cuts = reinterpret_cast<Cut*>(p.part_lse + 2 * kMaxCtas * 256);
  const StoreArgs& st = all.st;
  CUtensorMap qm, km, vm;
  int e = make_map(&qm, bf16, all.q, st.d, all.hq, all.n, st.d, all.q_stride, all.group, p.tt);
  if (e == FASTNN_OK)
    e = make_map(&km, bf16, st.k, st.d, st.page, static_cast<uint64_t>(st.n_pages) * st.heads, st.d,
                 static_cast<uint64_t>(st.page) * st.d, st.page, 1);
  if (e == FASTNN_OK)
    e = make_map(&vm, bf16, st.v, st.dv, st.page, static_cast<uint64_t>(st.n_pages) * st.heads, st.dv,
                 static_cast<uint64_t>(st.page) * st.dv, st.page, 1);
  if (e != FASTNN_OK) return e;
  FASTNN_CUDA_TRY(cudaMemsetAsync(all.status, 0, sizeof(int), stream));
  const bool poll = wait_limit(all.wait_ns) < kPolledLimit;
  FASTNN_CUDA_TRY(poll ? (allow_smem<attend_tc_kernel<T, DP, true>>(kSmem))
                       : (allow_smem<attend_tc_kernel<T, DP, false>>(kSmem)));
  for (int s0 = 0; s0 < st.n_seqs; s0 += kMaxSeqs) {
    TcArgs q = p;
    q.a.st.n_seqs = st.n_seqs - s0 < kMaxSeqs ? st.n_seqs - s0 : kMaxSeqs;
    q.a.st.table += static_cast<int64_t>(s0) * st.width;
    q.a.st.lens += s0;
    q.a.st.cu += s0;
    if (poll) {
      attend_tc_kernel<T, DP, true><<<p.ctas, kThreads, kSmem, stream>>>(qm, km, vm, q);
    } else {
      attend_tc_kernel<T, DP, false><<<p.ctas, kThreads, kSmem, stream>>>(qm, km, vm, q);
    }
    FASTNN_CUDA_TRY(cudaGetLastError());
    FASTNN_CUDA_TRY(launch_after(merge_kernel<T>, dim3(p.ctas - 1, 32), dim3(256), stream, q));
  }
  return FASTNN_OK;
}

template <typename T>
int tc_width(const AttendArgs& a, cudaStream_t st) {
  const int wide = a.st.d > a.st.dv ? a.st.d : a.st.dv;
  return wide <= 64 ? tc_launch<T, 64>(a, st) : tc_launch<T, 128>(a, st);
}

}  // namespace

bool attend_tc_takes(const AttendArgs& a) {
  return !a.pages && a.group <= kBlk && static_cast<int64_t>(a.max_new) * a.group >= kTcRows &&
         a.st.n_pages * a.st.heads <= INT32_MAX;
}

size_t attend_tc_floats(const AttendArgs& a) {
  return static_cast<size_t>(2) * kMaxCtas * 256 * (a.st.dv + 1) + kMaxCtas * sizeof(Cut) / sizeof(float);
}

int launch_attend_tc(const AttendArgs& a, int dtype, cudaStream_t st) {
  return dtype == FASTNN_BF16 ? tc_width<__nv_bfloat16>(a, st) : tc_width<__half>(a, st);
}

}  // namespace fastnn
