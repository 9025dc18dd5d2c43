// C ABI entry points of the token store (declared in include/fastnn.h):
// argument checks, workspace carving and the launches. Nothing is allocated
// and nothing is enqueued when an argument is refused.
#include <cmath>

#include "store.cuh"

using namespace fastnn;

namespace {

constexpr size_t kAlign = 256;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

bool dtype16(int dtype) { return dtype == FASTNN_BF16 || dtype == FASTNN_F16; }

// FASTNN_OK if the store's sizes are ones the kernels take.
int store_sizes(const fastnn_store* s) {
  if (!s) return FASTNN_ERR_INVALID;
  if (!dtype16(s->dtype)) return FASTNN_ERR_UNSUPPORTED;
  if (s->d < 8 || s->d > 128 || s->d % 8 || s->dv < 8 || s->dv > 128 || s->dv % 8)
    return FASTNN_ERR_UNSUPPORTED;
  if (s->page != 16 && s->page != 32 && s->page != 64 && s->page != 128)
    return FASTNN_ERR_UNSUPPORTED;
  if (s->n_seqs < 1 || s->n_seqs > 65534 || s->heads < 1 || s->heads > 1024 || s->n_pages < 1 ||
      s->n_pages > INT32_MAX || s->table_width < 1 ||
      static_cast<int64_t>(s->table_width) * s->page > INT32_MAX - 256)
    return FASTNN_ERR_INVALID;
  return FASTNN_OK;
}

StoreArgs store_args(const fastnn_store* s) {
  StoreArgs a{};
  a.k = static_cast<uint16_t*>(s->k_pages);
  a.v = static_cast<uint16_t*>(s->v_pages);
  a.mean = static_cast<uint16_t*>(s->k_mean);
  a.table = s->page_table;
  a.lens = s->lens;
  a.cu = s->cu;
  a.n_pages = s->n_pages;
  a.n_seqs = s->n_seqs;
  a.width = s->table_width;
  a.page = s->page;
  a.page_log2 = s->page == 16 ? 4 : s->page == 32 ? 5 : s->page == 64 ? 6 : 7;
  a.heads = s->heads;
  a.d = s->d;
  a.dv = s->dv;
  return a;
}

int rotation_args(const fastnn_rotation* r, int d, int inverse, RotaryArgs& a) {
  if (r->axes < 1 || r->axes > 2 || r->rot < 0 || r->rot > d || r->rot % (2 * r->axes))
    return FASTNN_ERR_INVALID;
  if (r->layout != FASTNN_ROTARY_HALF && r->layout != FASTNN_ROTARY_INTERLEAVED)
    return FASTNN_ERR_UNSUPPORTED;
  if (!std::isfinite(r->scale)) return FASTNN_ERR_INVALID;
  a.pos = r->pos;
  a.freq = r->freq;
  a.axes = r->axes;
  a.rot = r->rot;
  a.nf = r->rot / (2 * r->axes);
  a.interleaved = r->layout == FASTNN_ROTARY_INTERLEAVED;
  a.scale = r->scale;
  a.sign = inverse ? -1.f : 1.f;
  return FASTNN_OK;
}

// Checks of a ragged batch of new tokens. The kernels count tokens in 32 bits, up to
// a tile or a slab (at most 2^23 tokens) past the last one.
constexpr int64_t kMaxTokens = int64_t{1} << 30;
int batch_sizes(int64_t n, int max_new) {
  if (n < 0 || n > kMaxTokens) return FASTNN_ERR_INVALID;
  if (n > 0 && (max_new < 1 || max_new > n)) return FASTNN_ERR_INVALID;
  return FASTNN_OK;
}

int row_checks(const void* x, int64_t stride, int64_t width) {
  if (!x || !aligned(x, 16) || stride < width || stride % 8) return FASTNN_ERR_INVALID;
  return FASTNN_OK;
}

bool index_arrays(const fastnn_store* s) {
  return s->page_table && s->lens && s->cu && aligned(s->page_table, 4) && aligned(s->lens, 4) && aligned(s->cu, 4);
}
bool rotation_arrays(const RotaryArgs& r) { return r.pos && r.freq && aligned(r.pos, 4) && aligned(r.freq, 8); }

#define FASTNN_TRY(expr)              \
  do {                                \
    int rc_ = (expr);                 \
    if (rc_ != FASTNN_OK) return rc_; \
  } while (0)

AttendArgs attend_args(const fastnn_store* s, int64_t n, int heads_q, int max_new,
                       const int32_t* pages, int select) {
  AttendArgs a{};
  a.st = store_args(s);
  a.n = n;
  a.hq = heads_q;
  a.group = heads_q / s->heads;
  a.max_new = max_new;
  a.pages = pages;
  a.select = select;
  attend_plan(a);
  return a;
}

int attend_sizes(const fastnn_store* s, int64_t n, int heads_q, int max_new, int select) {
  FASTNN_TRY(store_sizes(s));
  FASTNN_TRY(batch_sizes(n, max_new));
  if (heads_q < 1 || heads_q % s->heads || heads_q > 65535 || select < 0 || select > 65535)
    return FASTNN_ERR_INVALID;
  return FASTNN_OK;
}

// fastnn_attend alone: the rows (token, head of a group) of a sequence, which are
// counted in 32 bits, up to a tile past the last one.
int attend_rows(const fastnn_store* s, int heads_q, int max_new) {
  return static_cast<int64_t>(max_new) * (heads_q / s->heads) > INT32_MAX - 16 ? FASTNN_ERR_INVALID : FASTNN_OK;
}

size_t part_bytes(const AttendArgs& a) {
  return a.splits > 1 && !a.pages ? static_cast<size_t>(a.splits) * a.n * a.hq * sizeof(float) : 0;
}
// Either kernel's partial outputs: which one runs also depends on the scale.
size_t attend_bytes(const AttendArgs& a) {
  const size_t rows = align_up(part_bytes(a) * a.st.dv) + align_up(part_bytes(a));
  const size_t tc = attend_tc_takes(a) ? align_up(attend_tc_floats(a) * sizeof(float)) : 0;
  return kAlign + (rows > tc ? rows : tc);
}

}  // namespace

extern "C" {

int fastnn_rotary(const void* x, int64_t x_stride, int64_t n, int heads, int d, int dtype,
                  const fastnn_rotation* rotation, int inverse, void* out, int64_t out_stride,
                  fastnn_stream_t stream) {
  if (!dtype16(dtype) || d < 1 || d > 1024) return FASTNN_ERR_UNSUPPORTED;
  if (n < 0 || heads < 1 || heads > 65535 || !rotation) return FASTNN_ERR_INVALID;
  RotaryArgs r{};
  FASTNN_TRY(rotation_args(rotation, d, inverse, r));
  if (r.rot == 0) return FASTNN_ERR_INVALID;
  if (n == 0) return FASTNN_OK;
  const int64_t width = static_cast<int64_t>(heads) * d;
  if (!rotation_arrays(r)) return FASTNN_ERR_INVALID;
  if (!x || !out || !aligned(x, 2) || !aligned(out, 2) || x_stride < width || out_stride < width)
    return FASTNN_ERR_INVALID;
  if (x == out && x_stride != out_stride) return FASTNN_ERR_INVALID;
  return launch_rotary(static_cast<const uint16_t*>(x), x_stride, n, heads, d, dtype, r,
                       static_cast<uint16_t*>(out), out_stride,
                       reinterpret_cast<cudaStream_t>(stream));
}

int fastnn_store_append(const fastnn_store* store, const void* k, int64_t k_stride, const void* v,
                        int64_t v_stride, int64_t n, int max_new, const fastnn_rotation* rotation,
                        void* workspace, size_t workspace_bytes, fastnn_stream_t stream) {
  FASTNN_TRY(store_sizes(store));
  FASTNN_TRY(batch_sizes(n, max_new));
  RotaryArgs r{};
  if (rotation) FASTNN_TRY(rotation_args(rotation, store->d, 0, r));
  if (n == 0) return FASTNN_OK;
  if (r.rot > 0 && !rotation_arrays(r)) return FASTNN_ERR_INVALID;
  FASTNN_TRY(row_checks(k, k_stride, static_cast<int64_t>(store->heads) * store->d));
  FASTNN_TRY(row_checks(v, v_stride, static_cast<int64_t>(store->heads) * store->dv));
  if (!store->k_pages || !aligned(store->k_pages, 16) || !store->v_pages ||
      !aligned(store->v_pages, 16) || !aligned(store->k_mean, 16) || !index_arrays(store) ||
      !aligned(workspace, kAlign))
    return FASTNN_ERR_INVALID;
  if (workspace && workspace_bytes < FASTNN_STORE_APPEND_WORKSPACE) return FASTNN_ERR_CAPACITY;
  return launch_store_append(store_args(store), store->dtype, static_cast<const uint16_t*>(k),
                             k_stride, static_cast<const uint16_t*>(v), v_stride, n, max_new, r,
                             static_cast<int*>(workspace), reinterpret_cast<cudaStream_t>(stream));
}

size_t fastnn_attend_workspace_size(const fastnn_store* store, int64_t n, int heads_q, int max_new,
                                    int select) {
  if (attend_sizes(store, n, heads_q, max_new, select) != FASTNN_OK) return 0;
  if (n == 0) return kAlign;
  if (attend_rows(store, heads_q, max_new) != FASTNN_OK) return 0;
  static const int32_t some = 0;
  return attend_bytes(attend_args(store, n, heads_q, max_new, select ? &some : nullptr, select));
}

int fastnn_attend(const fastnn_store* store, const void* q, int64_t q_stride, int64_t n,
                  int heads_q, int max_new, int causal, float scale, const int32_t* pages,
                  int select, void* out, float* lse, void* workspace, size_t workspace_bytes,
                  fastnn_stream_t stream) {
  FASTNN_TRY(attend_sizes(store, n, heads_q, max_new, select));
  if (!std::isfinite(scale) || (pages != nullptr) != (select > 0)) return FASTNN_ERR_INVALID;
  if (n == 0) return FASTNN_OK;
  FASTNN_TRY(attend_rows(store, heads_q, max_new));
  FASTNN_TRY(row_checks(q, q_stride, static_cast<int64_t>(heads_q) * store->d));
  if (!store->k_pages || !aligned(store->k_pages, 16) || !store->v_pages ||
      !aligned(store->v_pages, 16) || !index_arrays(store) || !aligned(pages, 4) || !out ||
      !aligned(out, 16) || !aligned(lse, 4) || !aligned(workspace, kAlign))
    return FASTNN_ERR_INVALID;
  AttendArgs a = attend_args(store, n, heads_q, max_new, pages, select);
  const size_t need = attend_bytes(a);
  if (!workspace && need > kAlign) return FASTNN_ERR_INVALID;
  if (workspace && workspace_bytes < need) return FASTNN_ERR_CAPACITY;
  a.q = static_cast<const uint16_t*>(q);
  a.q_stride = q_stride;
  a.causal = causal ? 1 : 0;
  a.scale_log2 = scale * 1.44269504088896340736f;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.status = reinterpret_cast<int*>(ws);
  a.part = reinterpret_cast<float*>(ws + kAlign);
  a.part_lse = reinterpret_cast<float*>(ws + kAlign + align_up(part_bytes(a) * a.st.dv));
  a.wait_ns = wait_timeout_ns();
  if (scale > 0.f && attend_tc_takes(a))
    return launch_attend_tc(a, store->dtype, reinterpret_cast<cudaStream_t>(stream));
  return launch_attend_rows(a, store->dtype, reinterpret_cast<cudaStream_t>(stream));
}

size_t fastnn_select_workspace_size(const fastnn_store* store, int64_t n, int heads_q, int max_new) {
  if (attend_sizes(store, n, heads_q, max_new, 1) != FASTNN_OK) return 0;
  if (n == 0) return kAlign;
  const StoreArgs a = store_args(store);
  return kAlign + align_up(select_key_bytes(a, max_new)) + align_up(select_sum_bytes(a, max_new));
}

int fastnn_select_pages(const fastnn_store* store, const void* q, int64_t q_stride, int64_t n,
                        int heads_q, int max_new, int causal, int keep_first, int keep_last,
                        int select, int32_t* out_pages, void* workspace, size_t workspace_bytes,
                        fastnn_stream_t stream) {
  FASTNN_TRY(attend_sizes(store, n, heads_q, max_new, select));
  if (keep_first < 0 || keep_last < 1 || select > 256 || keep_first > select - keep_last)
    return FASTNN_ERR_INVALID;
  if (n == 0) return FASTNN_OK;
  FASTNN_TRY(row_checks(q, q_stride, static_cast<int64_t>(heads_q) * store->d));
  if (!store->k_mean || !aligned(store->k_mean, 16) || !index_arrays(store) || !out_pages ||
      !aligned(out_pages, 4) || !aligned(workspace, kAlign))
    return FASTNN_ERR_INVALID;
  const size_t need = fastnn_select_workspace_size(store, n, heads_q, max_new);
  if (!workspace && need > kAlign) return FASTNN_ERR_INVALID;
  if (workspace && workspace_bytes < need) return FASTNN_ERR_CAPACITY;
  SelectArgs a{};
  a.st = store_args(store);
  a.q = static_cast<const uint16_t*>(q);
  a.q_stride = q_stride;
  a.n = n;
  a.hq = heads_q;
  a.group = heads_q / store->heads;
  a.max_new = max_new;
  a.causal = causal ? 1 : 0;
  a.keep_first = keep_first;
  a.keep_last = keep_last;
  a.select = select;
  a.out = out_pages;
  a.keys = reinterpret_cast<uint64_t*>(static_cast<uint8_t*>(workspace) + kAlign);
  a.sums = reinterpret_cast<double*>(static_cast<uint8_t*>(workspace) + kAlign +
                                     align_up(select_key_bytes(a.st, max_new)));
  return launch_select(a, store->dtype, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
