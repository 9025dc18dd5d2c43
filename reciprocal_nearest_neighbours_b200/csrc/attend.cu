// Attention over the paged token store, few query rows at a time.
//
//     out[t, h] = sum_p exp2(x_p - lse2) value[p],  x_p = scale * log2(e) * <q[t, h], key[p]>
//
// in one pass over the keys: a running reference m, sum l and output O per row,
//     l' = l 2^(m - m') + sum 2^(x - m'),  O' = O 2^(m - m') + 2^(x - m') V,
// all in fp32. A block takes 8 or 16 rows of one sequence and key head (the rows
// are (token, query head of the group), so a group's heads share the keys' read)
// and one split of the positions. Its warps do not wait for one another: each
// streams every kWarps-th unit of 16 positions through its own cp.async ring,
// keeps its own (m, l, O), and the warps merge once at the end. Splits leave
// normalised partial outputs with their log2 sums, which combine_kernel weighs;
// of selected pages, which are few, the splits are one cluster.
// The products are mma.sync m16n8k16 with the KEYS as the 16 rows of the first
// operand and the query rows as its 8 columns: S^T = K Q^T, O^T = V^T P^T. A group
// of up to 8 heads then wastes no product, O takes half the registers that a
// 16-row tile of queries would need, and up to 12 warps fit an SM. With few rows
// the work is bound by reading K and V once. Measured (32 / 8 heads of 128): one
// token of 96 sequences of 17 to 8192 positions 245 us, 6.5 TB/s; of 3 sequences of up to
// 65k 100 us, 6.2 TB/s, and 5 for the join; 16 listed pages of 64 for each of
// 2048 tokens and 4 key heads 280 us, 15 TB/s out of L2.
#include <type_traits>

#include "store.cuh"
#include "ptx.cuh"

namespace fastnn {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kUnit = 16;    // positions of a unit: the smallest page
// Units in a warp's ring, and blocks an SM holds. At 128 elements two blocks with
// deeper rings stream single tokens' keys faster (3 long sequences 120 us against
// 125 with three blocks of two units), three serve many tokens' pages out of L2
// faster (2k tokens 280 us against 360).
template <int DP, bool MANY>
struct Depth {
  static constexpr int kStages = DP == 128 ? (MANY ? 2 : 3) : 4;
  static constexpr int kBlocks = DP == 128 && !MANY ? 2 : 3;
};
constexpr float kMostSum = 256.f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool real) {
  const int bytes = real ? 16 : 0;  // 0: the 16 bytes are zero-filled, nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Transposes an 8 x 8 matrix of 16-bit elements held by the warp (lane: row lane /
// 4, elements 2 (lane % 4) and the next one).
__device__ __forceinline__ uint32_t turn8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if constexpr (sizeof(T) == 2 && std::is_same<T, __half>::value) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
}

// Byte offset of 16-byte chunk c of row r in a tile of DP 16-bit elements a
// row. Chunks are permuted so that eight consecutive rows of one chunk column
// (an ldmatrix access) fall into eight different bank groups.
template <int DP>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  if constexpr (DP >= 64) return static_cast<uint32_t>(r * DP * 2 + ((c ^ (r & 7)) << 4));
  return static_cast<uint32_t>(r * DP * 2 + ((c ^ ((r >> 1) & 3)) << 4));
}

// NT: groups of 8 query rows of a block.
template <int DP, int NT, int kStages>
struct RowsSmem {
  static constexpr int kRows = 8 * NT;
  static constexpr int kTile = kUnit * DP * 2;       // bytes of one K or V unit
  static constexpr int kStage = 2 * kTile;
  static constexpr int kRing = kStages * kStage;     // a warp's ring
  static constexpr int kMl = kWarps * kRing;         // then [kWarps][16] m and l
  static constexpr int kTotal = kMl + kWarps * kRows * 2 * 4;
  static constexpr int kOutPitch = DP + 4;           // floats of a row in the merge
  static_assert(kRing >= kRows * kOutPitch * 4, "the merge reuses the ring");
};

// DP: head width padded to 32, 64 or 128. SEL: the positions are those of
// a.pages' entries for the block's (single) token. FULL: d == dv == DP, so a
// unit's K and V are 16 * DP consecutive elements each.
// With SEL the a.splits blocks of a row tile are a cluster and join their
// parts through one another's shared memory.
template <typename T, int DP, int NT, bool SEL, bool FULL, bool MANY>
__global__ void __launch_bounds__(kThreads, Depth<DP, MANY>::kBlocks)
attend_rows_kernel(AttendArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int kStages = Depth<DP, MANY>::kStages;
  using S = RowsSmem<DP, NT, kStages>;
  constexpr int kRows = S::kRows;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int s = blockIdx.z, g = blockIdx.y;
  const int split = static_cast<int>(blockIdx.x) % a.splits;
  const int tile = static_cast<int>(blockIdx.x) / a.splits;
  if (a.status && blockIdx.x == 0 && g == 0 && s == 0 && tid == 0) *a.status = 0;
  const StoreArgs& st = a.st;
  const SeqView w = seq_view(st, s, a.n, a.max_new, a.causal);

  // The block's rows: row r is token tok(r) of the sequence, query head
  // head(r); nrows of kRows exist.
  int r0, nrows, tok_first;
  if constexpr (SEL) {
    const int per_tok = (a.group + kRows - 1) / kRows;
    tok_first = tile / per_tok;
    if (tok_first >= w.n) return;
    r0 = (tile - tok_first * per_tok) * kRows;
    nrows = a.group - r0 < kRows ? a.group - r0 : kRows;
  } else {
    r0 = tile * kRows;
    const int64_t all = static_cast<int64_t>(w.n) * a.group;
    if (r0 >= all) return;
    nrows = all - r0 < kRows ? static_cast<int>(all - r0) : kRows;
    tok_first = r0 / a.group;
  }
  const int last = SEL ? tok_first : (r0 + nrows - 1) / a.group;
  const int vmax = visible(w, last);  // visible() grows with the token

  int u_count;      // units of the whole block
  int u_first = 0;  // SEL: the first of them
  int k0 = 0;       // first position (not SEL)
  const int32_t* list = nullptr;
  const int upp = st.page / kUnit;
  if constexpr (SEL) {
    list = a.pages + ((static_cast<int64_t>(w.t0) + tok_first) * st.heads + g) * a.select;
    const int u1 = a.select * upp;  // split_len counts units here
    u_first = split * a.split_len;
    u_count = u1 - u_first < a.split_len ? u1 - u_first : a.split_len;
  } else {
    k0 = split * a.split_len;
    if (split > 0 && k0 >= vmax) return;  // no row of the tile reads this split
    const int k1 = vmax - k0 < a.split_len ? vmax : k0 + a.split_len;
    u_count = (k1 - k0 + kUnit - 1) / kUnit;
  }

  // Query fragments: row lane / 4 of each group of 8, zero beyond d and beyond
  // nrows. The scores of a thread belong to rows 2 (lane % 4) and the next one.
  uint32_t qb[DP / 16][NT][2];
  int vis[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = (lane >> 2) + 8 * n;
    const bool real = r < nrows;
    const int rr = r0 + (real ? r : 0);
    const int tok = SEL ? tok_first : rr / a.group;
    const int hd = g * a.group + (SEL ? rr : rr - tok * a.group);
    const uint16_t* qr = a.q + (static_cast<int64_t>(w.t0) + tok) * a.q_stride +
                         static_cast<int64_t>(hd) * st.d;
#pragma unroll
    for (int ks = 0; ks < DP / 16; ++ks)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int col = ks * 16 + c * 8 + (lane & 3) * 2;
        qb[ks][n][c] = real && col < st.d ? __ldg(reinterpret_cast<const uint32_t*>(qr + col)) : 0u;
      }
#pragma unroll
    for (int e = 0; e < 2; ++e) {  // a row that is not there has zero queries and masks nothing more
      const int q = (lane & 3) * 2 + e + 8 * n;
      vis[n][e] = SEL || q >= nrows ? vmax : visible(w, (r0 + q) / a.group);
    }
  }
  const int vmin = SEL ? vmax : visible(w, tok_first);

  const uint32_t ring = ptx::smem_u32(smem) + warp * S::kRing;
  const int mine = u_count > warp ? (u_count - warp + kWarps - 1) / kWarps : 0;

  // Page ids of 32 of this warp's units at a time, one a lane: the physical
  // page (-1: hole) and, for SEL, the logical page.
  int ids = -1, lps = 0;
  auto fetch_ids = [&](int j) {
    const int u = warp + (j + lane) * kWarps;
    ids = -1;
    if (u < u_count) {
      int lp;
      if constexpr (SEL) {
        lp = __ldg(list + (u_first + u) / upp);
      } else {
        lp = (k0 + u * kUnit) >> st.page_log2;
      }
      lps = lp;
      if (lp >= 0 && lp < st.width) {
        const int id = __ldg(st.table + static_cast<int64_t>(s) * st.width + lp);
        if (id >= 0 && id < st.n_pages) ids = id;
      }
    }
  };
  // First position of unit j of this warp; its id decides whether it exists.
  auto unit_pos = [&](int j, int lp) {
    const int u = warp + j * kWarps;
    if constexpr (SEL) return lp * st.page + ((u_first + u) & (upp - 1)) * kUnit;
    return k0 + u * kUnit;
  };
  // Copies of one unit, 16 bytes a lane and step: step i takes chunk c of row
  // row0 + i * kRowStep.
  constexpr int kChunks = DP / 8, kSteps = kUnit * kChunks / 32, kRowStep = 32 / kChunks;
  const int row0 = lane / kChunks, c0 = lane % kChunks;
  const int64_t k_page = static_cast<int64_t>(st.page) * st.d, v_page = static_cast<int64_t>(st.page) * st.dv;
  // Positions of the ring's stages (-1: nothing there), as the warp knows them.
  int pos_ring[kStages];
  auto issue = [&](int j, int stage) {
    int pos = -1;
    if (j < mine) {
      if ((j & 31) == 0) fetch_ids(j);
      const int id = __shfl_sync(0xffffffffu, ids, j & 31);
      const int lp = SEL ? __shfl_sync(0xffffffffu, lps, j & 31) : 0;
      if (id >= 0) pos = unit_pos(j, lp);
      if (pos >= vmax) pos = -1;
      if (pos >= 0) {
        const int64_t slab = static_cast<int64_t>(id) * st.heads + g;
        const int in_page = pos & (st.page - 1);
        const uint32_t kd = ring + stage * S::kStage, vd = kd + S::kTile;
        if (FULL && pos + kUnit <= vmax) {
          const int64_t off = slab * k_page + in_page * DP + lane * 8;
          const uint16_t* kp = st.k + off;
          const uint16_t* vp = st.v + off;
#pragma unroll
          for (int i = 0; i < kSteps; ++i) {
            cp16(kd + chunk_at<DP>(row0 + i * kRowStep, c0), kp + i * 256, true);
            cp16(vd + chunk_at<DP>(row0 + i * kRowStep, c0), vp + i * 256, true);
          }
        } else {
          const uint16_t* kp = st.k + slab * k_page + in_page * st.d;
          const uint16_t* vp = st.v + slab * v_page + in_page * st.dv;
#pragma unroll
          for (int i = 0; i < kSteps; ++i) {
            const int r = row0 + i * kRowStep;
            const bool there = pos + r < vmax;  // what lies behind the length is not read
            const bool kr = there && c0 * 8 < st.d, vr = there && c0 * 8 < st.dv;
            cp16(kd + chunk_at<DP>(r, c0), kr ? kp + r * st.d + c0 * 8 : st.k, kr);
            cp16(vd + chunk_at<DP>(r, c0), vr ? vp + r * st.dv + c0 * 8 : st.v, vr);
          }
        }
      }
    }
    cp_commit();
    return pos;
  };

  float o[DP / 16][NT][4] = {};  // dims lane / 4 and + 8 of each 16, rows as the scores'
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) m[n][0] = m[n][1] = -INFINITY, l[n][0] = l[n][1] = 0.f;
  // Byte offsets of this lane's ldmatrix rows within a tile; the 16-column step
  // ks of a row lies at this offset with ks * 32 exclusive-or'ed in.
  const uint32_t k_off = chunk_at<DP>(lane & 15, lane >> 4);
  const uint32_t v_off = chunk_at<DP>((lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1);
#pragma unroll
  for (int j = 0; j < kStages - 1; ++j) pos_ring[j] = issue(j, j);
  for (int jb = 0; jb < mine; jb += kStages) {
#pragma unroll
    for (int st_i = 0; st_i < kStages; ++st_i) {
      const int j = jb + st_i;
      if (j >= mine) break;
      cp_wait<kStages - 2>();
      __syncwarp();
      const int pos = pos_ring[st_i];
      // The stage read at step j - 1 is free again: fill it before computing.
      constexpr int kBack = kStages - 1;
      pos_ring[(st_i + kBack) % kStages] = issue(j + kBack, (st_i + kBack) % kStages);
      if (pos < 0) continue;
      const uint32_t kd = ring + st_i * S::kStage + k_off, vd = ring + st_i * S::kStage + S::kTile + v_off;
      // Scores: positions lane / 4 (x[n][0], x[n][1]) and + 8, two rows each. Even
      // and odd steps add up apart: half as long a chain of dependent products.
      float x[NT][4] = {}, x2[NT][4] = {};
#pragma unroll
      for (int ks = 0; ks < DP / 16; ks += 2) {
        uint32_t k1[4], k2[4];
        ldsm4(kd ^ (ks * 32), k1);
        ldsm4(kd ^ (ks * 32 + 32), k2);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma16816<T>(x[n], k1, qb[ks][n][0], qb[ks][n][1]);
          mma16816<T>(x2[n], k2, qb[ks + 1][n][0], qb[ks + 1][n][1]);
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[n][e] += x2[n][e];
      const bool edge = pos + kUnit > vmin;
      if (edge) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (pos + (lane >> 2) + (e >> 1) * 8 >= vis[n][e & 1]) x[n][e] = -INFINITY;
      }
      // Weights by the reference in force, and each thread's share of their sums.
      // The reference need not be the largest score so far (O / l does not depend
      // on it): a maximum is sought, with the shuffles that takes, only when a
      // thread's sum says that a weight may be far above 1.
      float y[NT][4], sum[NT][2];
      auto weigh = [&]() {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float z = m[n][e] == -INFINITY ? 0.f : -m[n][e];
            y[n][e] = ex2(fmaf(x[n][e], a.scale_log2, z));
            y[n][e + 2] = ex2(fmaf(x[n][e + 2], a.scale_log2, z));
            sum[n][e] = y[n][e] + y[n][e + 2];
          }
      };
      weigh();
      bool raise = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) raise = raise || sum[n][e] > kMostSum || m[n][e] == -INFINITY;
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = m[n][e];  // a masked place stays out for a scale of any sign
            if (x[n][e] != -INFINITY) top = fmaxf(top, x[n][e] * a.scale_log2);
            if (x[n][e + 2] != -INFINITY) top = fmaxf(top, x[n][e + 2] * a.scale_log2);
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            // A row that has seen nothing yet has m = -inf: l and O are 0 then.
            const float f = m[n][e] == top ? 1.f : ex2(m[n][e] - top);
            l[n][e] *= f;
            m[n][e] = top;
#pragma unroll
            for (int t = 0; t < DP / 16; ++t) {
              o[t][n][e] *= f;
              o[t][n][e + 2] *= f;
            }
          }
        weigh();
      }
      if (edge) {  // and its weight is 0
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (x[n][e] == -INFINITY) y[n][e] = 0.f;
          sum[n][0] = y[n][0] + y[n][2];
          sum[n][1] = y[n][1] + y[n][3];
        }
      }
      // The weights go to the tensor cores rounded to the store's 16-bit type (the
      // operands of a product have one type), turned from (position, row) to the (row, position) fragments of an operand.
      uint32_t p[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        l[n][0] += sum[n][0];
        l[n][1] += sum[n][1];
        p[n][0] = turn8x8(Half16<T>::pack(y[n][0], y[n][1]));
        p[n][1] = turn8x8(Half16<T>::pack(y[n][2], y[n][3]));
      }
#pragma unroll
      for (int t = 0; t < DP / 16; ++t) {
        uint32_t v[4];
        ldsm4t(vd ^ (t * 32), v);
#pragma unroll
        for (int n = 0; n < NT; ++n) mma16816<T>(o[t][n], v, p[n][0], p[n][1]);
      }
    }
  }
  cp_wait<0>();
  __syncwarp();

  // Merge the warps: each leaves its rows' O (over its own ring), m and l.
  float* mine_o = reinterpret_cast<float*>(smem + warp * S::kRing);
  float* ml = reinterpret_cast<float*>(smem + S::kMl);
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float sum = l[n][e];
      sum += __shfl_xor_sync(0xffffffffu, sum, 4);
      sum += __shfl_xor_sync(0xffffffffu, sum, 8);
      sum += __shfl_xor_sync(0xffffffffu, sum, 16);
      const int q = n * 8 + (lane & 3) * 2 + e;
      if (lane < 4) {
        ml[(warp * kRows + q) * 2] = m[n][e];
        ml[(warp * kRows + q) * 2 + 1] = sum;
      }
#pragma unroll
      for (int t = 0; t < DP / 16; ++t) {
        mine_o[q * S::kOutPitch + t * 16 + (lane >> 2)] = o[t][n][e];
        mine_o[q * S::kOutPitch + t * 16 + (lane >> 2) + 8] = o[t][n][e + 2];
      }
    }
  __syncthreads();
  constexpr int kPerRow = kThreads / kRows;  // threads a row
  constexpr int kVec = (DP + kPerRow * 4 - 1) / (kPerRow * 4);
  const int r = tid / kPerRow, c_first = (tid % kPerRow) * 4;
  float top = -INFINITY;
#pragma unroll
  for (int q = 0; q < kWarps; ++q) top = fmaxf(top, ml[(q * kRows + r) * 2]);
  float sum = 0.f;
  float4 v[kVec];
#pragma unroll
  for (int k = 0; k < kVec; ++k) v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int q = 0; q < kWarps; ++q) {
    const float mq = ml[(q * kRows + r) * 2];
    const float f = mq == -INFINITY ? 0.f : mq == top ? 1.f : ex2(mq - top);
    sum += f * ml[(q * kRows + r) * 2 + 1];
#pragma unroll
    for (int k = 0; k < kVec; ++k) {
      const int c = c_first + k * kPerRow * 4;
      if (c >= DP) break;
      const float4 y = *reinterpret_cast<const float4*>(
          reinterpret_cast<const float*>(smem + q * S::kRing) + r * S::kOutPitch + c);
      v[k].x += f * y.x;
      v[k].y += f * y.y;
      v[k].z += f * y.z;
      v[k].w += f * y.w;
    }
  }
  if (SEL && a.splits > 1) {
    // This block's part goes where the first warp's was; then each thread joins
    // the parts of its places, the blocks taking turns at the columns.
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kVec; ++k) {
      const int c = c_first + k * kPerRow * 4;
      if (c < DP) *reinterpret_cast<float4*>(reinterpret_cast<float*>(smem) + r * S::kOutPitch + c) = v[k];
    }
    if (tid % kPerRow == 0) {
      ml[r * 2] = top;
      ml[r * 2 + 1] = sum;
    }
    ptx::cluster_sync();
    const uint32_t base = ptx::smem_u32(smem), mls = ptx::smem_u32(ml) + r * 8;
    top = -INFINITY;
    for (int q = 0; q < a.splits; ++q) top = fmaxf(top, ptx::cluster_ld2(ptx::cluster_map(mls, q)).x);
    sum = 0.f;
#pragma unroll
    for (int k = 0; k < kVec; ++k) v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int q = 0; q < a.splits; ++q) {
      const float2 part = ptx::cluster_ld2(ptx::cluster_map(mls, q));
      const float f = part.x == -INFINITY ? 0.f : part.x == top ? 1.f : ex2(part.x - top);
      sum += f * part.y;
      const uint32_t from = ptx::cluster_map(base, q) + r * S::kOutPitch * 4;
#pragma unroll
      for (int k = 0; k < kVec; ++k) {
        const int c = c_first + k * kPerRow * 4;
        if (c >= st.dv || (c / 4) % a.splits != split) continue;
        const float4 y = ptx::cluster_ld4(from + c * 4);
        v[k].x += f * y.x;
        v[k].y += f * y.y;
        v[k].z += f * y.z;
        v[k].w += f * y.w;
      }
    }
    ptx::cluster_sync();  // no block leaves while others read its part
  }
  if (r >= nrows) return;
  const float inv = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;
  const float lse2 = sum > 0.f ? top + log2f(sum) : sum == 0.f ? -INFINITY : sum;
  const int rr = r0 + r;
  const int tok = SEL ? tok_first : rr / a.group;
  const int hd = g * a.group + (SEL ? rr : rr - tok * a.group);
  const int64_t row = (static_cast<int64_t>(w.t0) + tok) * a.hq + hd;
  const bool whole = SEL || visible(w, tok) <= a.split_len;
  if (!SEL && whole && split > 0) return;
#pragma unroll
  for (int k = 0; k < kVec; ++k) {
    const int c = c_first + k * kPerRow * 4;
    if (c >= st.dv || (SEL && a.splits > 1 && (c / 4) % a.splits != split)) continue;
    const float4 y = make_float4(v[k].x * inv, v[k].y * inv, v[k].z * inv, v[k].w * inv);
    if (whole) {
      *reinterpret_cast<uint2*>(a.out + row * st.dv + c) =
          make_uint2(Half16<T>::pack(y.x, y.y), Half16<T>::pack(y.z, y.w));
    } else {
      *reinterpret_cast<float4*>(a.part + (split * a.n * a.hq + row) * st.dv + c) = y;
    }
  }
  if (tid % kPerRow == 0) {
    if (!whole) {
      a.part_lse[split * a.n * a.hq + row] = lse2;
    } else if (a.lse && (!SEL || split == 0)) {
      a.lse[row] = lse2 * 0.69314718055994530942f;  // ln 2
    }
  }
}

// Joins the splits of a row: out = sum_i 2^(lse2_i - lse2) out_i. A block takes one
// row, its warps every fourth split each (a warp alone would wait for some tens
// of them one after the other: 3 long sequences 119 us against 106).
template <typename T>
__global__ void __launch_bounds__(kThreads)
combine_kernel(AttendArgs a) {
  cudaGridDependencySynchronize();
  __shared__ float tops[kWarps], sums[kWarps];
  __shared__ float4 parts_v[kWarps][32];
  const StoreArgs& st = a.st;
  const int s = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const SeqView w = seq_view(st, s, a.n, a.max_new, a.causal);
  const int64_t r = blockIdx.x;
  if (r >= static_cast<int64_t>(w.n) * a.hq) return;
  const int vis = visible(w, static_cast<int>(r / a.hq));
  const int parts = (vis + a.split_len - 1) / a.split_len;
  if (parts <= 1) return;  // its one split has written the result
  const int64_t row = static_cast<int64_t>(w.t0) * a.hq + r;
  const int64_t step = a.n * a.hq;
  float top = -INFINITY;
  for (int i = threadIdx.x; i < parts; i += kThreads) top = fmaxf(top, a.part_lse[i * step + row]);
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) tops[warp] = top;
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kWarps; ++q) top = fmaxf(top, tops[q]);
  float sum = 0.f;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  const int c = lane * 4;
#pragma unroll 4
  for (int i = warp; i < parts; i += kWarps) {
    const float z = a.part_lse[i * step + row];  // NaN makes the row NaN, though fmaxf drops it
    const float f = z == -INFINITY ? 0.f : ex2(z - top);
    const float4 y = c < st.dv ? *reinterpret_cast<const float4*>(a.part + (i * step + row) * st.dv + c)
                               : make_float4(0.f, 0.f, 0.f, 0.f);
    sum += f;
    v.x += f * y.x;
    v.y += f * y.y;
    v.z += f * y.z;
    v.w += f * y.w;
  }
  parts_v[warp][lane] = v;
  if (lane == 0) sums[warp] = sum;
  __syncthreads();
  if (warp > 0) return;
#pragma unroll
  for (int q = 1; q < kWarps; ++q) {
    const float4 y = parts_v[q][lane];
    sum += sums[q];
    v.x += y.x;
    v.y += y.y;
    v.z += y.z;
    v.w += y.w;
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  if (c < st.dv)
    *reinterpret_cast<uint2*>(a.out + row * st.dv + c) =
        make_uint2(Half16<T>::pack(v.x * inv, v.y * inv), Half16<T>::pack(v.z * inv, v.w * inv));
  if (lane == 0 && a.lse) a.lse[row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994530942f;
}

// Groups of 8 query rows of a block: one if no block would have more rows.
int row_groups(const AttendArgs& a) {
  const int64_t rows = a.pages ? a.group : static_cast<int64_t>(a.max_new) * a.group;
  return rows <= 8 ? 1 : 2;
}
// Row tiles of a sequence and key head.
int64_t row_tiles(const AttendArgs& a) {
  const int per = 8 * row_groups(a);
  return a.pages ? static_cast<int64_t>(a.max_new) * ((a.group + per - 1) / per)
                 : (static_cast<int64_t>(a.max_new) * a.group + per - 1) / per;
}

template <typename T, int DP, int NT, bool SEL, bool FULL, bool MANY>
int rows_launch(const AttendArgs& a, cudaStream_t st) {
  using D = Depth<DP, MANY>;
  using S = RowsSmem<DP, NT, D::kStages>;
  static_assert(D::kBlocks * (S::kTotal + 1024) <= 228 * 1024, "the blocks fit an SM");
  FASTNN_CUDA_TRY((allow_smem<attend_rows_kernel<T, DP, NT, SEL, FULL, MANY>>(S::kTotal)));
  const int64_t tiles = row_tiles(a);
  if (tiles * a.splits > INT32_MAX) return FASTNN_ERR_INVALID;
  const dim3 grid(static_cast<unsigned>(tiles * a.splits), a.st.heads, a.st.n_seqs);
  if (SEL && a.splits > 1) {
    FASTNN_CUDA_TRY(launch_cluster(attend_rows_kernel<T, DP, NT, SEL, FULL, MANY>, grid, dim3(kThreads), S::kTotal,
                                   a.splits, st, a));
    return FASTNN_OK;
  }
  attend_rows_kernel<T, DP, NT, SEL, FULL, MANY><<<grid, kThreads, S::kTotal, st>>>(a);
  FASTNN_CUDA_TRY(cudaGetLastError());
  if (a.splits > 1) {
    const int64_t rows = static_cast<int64_t>(a.max_new) * a.hq;  // few: there are fewer tiles than blocks wanted
    if (rows > INT32_MAX) return FASTNN_ERR_INVALID;
    FASTNN_CUDA_TRY(launch_after(combine_kernel<T>, dim3(static_cast<unsigned>(rows), a.st.n_seqs),
                                 dim3(kThreads), st, a));
  }
  return FASTNN_OK;
}

template <typename T, int DP, int NT, bool SEL, bool FULL>
int rows_many(const AttendArgs& a, cudaStream_t st) {
  // More row tiles than the deeper rings' blocks fill twice: their keys are
  // shared, and come out of L2.
  if constexpr (DP == 128)
    if (row_tiles(a) * a.st.heads * a.st.n_seqs > 4 * 148 && a.max_new > 1)
      return rows_launch<T, DP, NT, SEL, FULL, true>(a, st);
  return rows_launch<T, DP, NT, SEL, FULL, false>(a, st);
}

template <typename T, int DP, bool SEL>
int rows_full(const AttendArgs& a, cudaStream_t st) {
  const bool full = a.st.d == DP && a.st.dv == DP;
  if (row_groups(a) == 1)
    return full ? rows_many<T, DP, 1, SEL, true>(a, st) : rows_many<T, DP, 1, SEL, false>(a, st);
  return full ? rows_many<T, DP, 2, SEL, true>(a, st) : rows_many<T, DP, 2, SEL, false>(a, st);
}

template <typename T, bool SEL>
int rows_width(const AttendArgs& a, cudaStream_t st) {
  const int wide = a.st.d > a.st.dv ? a.st.d : a.st.dv;
  if (wide <= 32) return rows_full<T, 32, SEL>(a, st);
  if (wide <= 64) return rows_full<T, 64, SEL>(a, st);
  return rows_full<T, 128, SEL>(a, st);
}

}  // namespace

// How many blocks share the positions of a row tile. The lengths are on the
// device; the table's width bounds them (and is taken for them: under a table far
// wider than its longest sequence fewer blocks have work). About four waves of blocks (two a SM)
// even out ragged lengths, a split is at least 256 positions long, and splits
// beyond a row's length cost an empty block each.
void attend_plan(AttendArgs& a) {
  const bool sel = a.pages != nullptr;
  const int64_t tiles = row_tiles(a);
  const int64_t base = tiles * a.st.heads * a.st.n_seqs;
  if (sel) {
    // One wave of blocks (units are of one length), joined as clusters of up to 8.
    const int units = a.select * (a.st.page / kUnit);
    int64_t splits = base >= 2 * 148 ? 1 : 2 * 148 / base;
    if (splits > 8) splits = 8;
    if (splits > (units + 15) / 16) splits = (units + 15) / 16;  // four units a warp at least
    a.split_len = static_cast<int>((units + splits - 1) / splits);
    a.splits = (units + a.split_len - 1) / a.split_len;
    return;
  }
  const int64_t want = 4 * 2 * 148;
  const int64_t splits = base >= want ? 1 : (want + base - 1) / base;
  const int64_t cap = static_cast<int64_t>(a.st.width) * a.st.page;
  int64_t len = (cap + splits - 1) / splits;
  if (len < 256) len = 256;
  len = (len + 127) / 128 * 128;
  if (len > (int64_t{1} << 30)) len = int64_t{1} << 30;
  a.split_len = static_cast<int>(len);
  a.splits = static_cast<int>((cap + len - 1) / len);
}

int launch_attend_rows(const AttendArgs& a, int dtype, cudaStream_t st) {
  if (dtype == FASTNN_BF16)
    return a.pages ? rows_width<__nv_bfloat16, true>(a, st) : rows_width<__nv_bfloat16, false>(a, st);
  return a.pages ? rows_width<__half, true>(a, st) : rows_width<__half, false>(a, st);
}

}  // namespace fastnn
