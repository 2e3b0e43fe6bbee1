// The C ABI of the event-history operators (include/dlrm.h): argument checks
// and launches.
#include <atomic>

#include "history.cuh"

namespace {

std::atomic<int64_t> stall_limit_ns{0};
std::atomic<int32_t> stall_withhold{0};

using dlrm::aligned_to;

// Rows are counted in int32, and rounded up to tiles of at most 256.
constexpr int64_t kRowLimit = (int64_t(1) << 31) - 256;

bool head_dim_ok(int d) { return d == 32 || d == 64 || d == 128; }

dlrm_status_t check_shape(const dlrm_history_t* h) {
  if (!h || h->n_pages < 1 || h->n_heads < 1 || h->n_slots < 1 || h->max_pages < 1 ||
      h->page_tokens < 1 || h->head_dim < 1)
    return DLRM_ERR_INVALID_ARG;
  if ((h->page_tokens != 32 && h->page_tokens != 64 && h->page_tokens != 128) ||
      !head_dim_ok(h->head_dim))
    return DLRM_ERR_UNSUPPORTED;
  // page numbers, table entries and a history's events are counted in int32
  const int64_t limit = int64_t(1) << 31;
  if (static_cast<int64_t>(h->n_slots) * h->max_pages >= limit ||
      static_cast<int64_t>(h->max_pages) * h->page_tokens >= limit / 2 ||
      static_cast<int64_t>(h->n_pages) + h->n_slots >= limit ||
      static_cast<int64_t>(h->n_heads) * h->page_tokens * h->head_dim >= limit)
    return DLRM_ERR_UNSUPPORTED;
  return DLRM_OK;
}

dlrm_status_t check_pool(const dlrm_history_t* h) {
  const dlrm_status_t s = check_shape(h);
  if (s != DLRM_OK) return s;
  if (!h->k_codes || !h->v_codes || !h->k_scales || !h->v_scales || !h->table || !h->lengths ||
      !h->refs || !h->free_pages || !h->n_free || !h->err || !h->work)
    return DLRM_ERR_INVALID_ARG;
  if (!aligned_to(h->k_codes, 16) || !aligned_to(h->v_codes, 16) || !aligned_to(h->work, 16) ||
      !aligned_to(h->k_scales, 4) || !aligned_to(h->v_scales, 4) || !aligned_to(h->table, 4) ||
      !aligned_to(h->lengths, 4) || !aligned_to(h->refs, 4) || !aligned_to(h->free_pages, 4) ||
      !aligned_to(h->n_free, 4) || !aligned_to(h->err, 4))
    return DLRM_ERR_INVALID_ARG;
  if (h->work_bytes < dlrm::history_work(*h).total) return DLRM_ERR_INVALID_ARG;
  return DLRM_OK;
}

dlrm_status_t check_slots(const dlrm_history_t* h, const int32_t* slots, int32_t batch) {
  if (batch < 0 || batch > h->n_slots) return DLRM_ERR_INVALID_ARG;
  if (batch > 0 && (!slots || !aligned_to(slots, 4))) return DLRM_ERR_INVALID_ARG;
  return DLRM_OK;
}

bool dtype_ok(int dtype) {
  return dtype == DLRM_DTYPE_FP32 || dtype == DLRM_DTYPE_BF16 || dtype == DLRM_DTYPE_FP16;
}

dlrm_status_t status_of(cudaError_t e) { return e == cudaSuccess ? DLRM_OK : DLRM_ERR_CUDA; }

// What both attention calls share; *run is false where there is nothing to do.
dlrm_status_t check_attention(const dlrm_attention_t* a, int kv_heads, bool* run) {
  *run = false;
  if (!a || a->batch < 0 || a->q_rows < 0 || a->n_heads < 1 || kv_heads < 1 ||
      a->n_heads % kv_heads != 0 || !dtype_ok(a->dtype) || a->window < 0 || a->sinks < 0 ||
      !(a->scale == a->scale))
    return DLRM_ERR_INVALID_ARG;
  if (a->q_rows >= kRowLimit || a->q_rows * (a->n_heads / kv_heads) >= kRowLimit) return DLRM_ERR_UNSUPPORTED;
  if (a->batch == 0 || a->q_rows == 0) return DLRM_OK;
  const size_t eb = static_cast<size_t>(dlrm::dtype_bytes(a->dtype));
  if (!a->q || !a->out || !a->q_starts || !aligned_to(a->q, eb) || !aligned_to(a->out, eb) ||
      !aligned_to(a->q_starts, 4) || !aligned_to(a->lse, 4) || !aligned_to(a->err, 4))
    return DLRM_ERR_INVALID_ARG;
  if (a->ld_q < 0 || a->ld_q_head < 0 || a->ld_out < 0 || a->ld_out_head < 0)
    return DLRM_ERR_INVALID_ARG;
  *run = true;
  return DLRM_OK;
}

// Whether rows and heads of an output lie over one another.
bool rows_overlap(int64_t rows, int64_t ld, int64_t heads, int64_t ld_head, int64_t dim) {
  if ((rows > 1 && ld < dim) || (heads > 1 && ld_head < dim)) return true;
  if (rows <= 1 || heads <= 1) return false;
  const bool inner = ld_head <= ld;                // the smaller stride is the heads'
  const int64_t a = inner ? ld_head : ld, na = inner ? heads : rows;
  const int64_t b = inner ? ld : ld_head, nb = inner ? rows : heads;
  // step j of the larger stride falls between steps i and i + 1 of the smaller
  for (int64_t j = 1; j < nb && j * b < a * (na - 1) + dim; ++j) {
    const int64_t i = j * b / a, r = j * b % a;
    if ((r < dim && i < na) || (a - r < dim && i + 1 < na)) return true;
  }
  return false;
}

}  // namespace

namespace dlrm {
WaitCfg attention_wait() {
  WaitCfg w;
  w.limit_ns = static_cast<uint64_t>(stall_limit_ns.load(std::memory_order_relaxed));
  w.withhold_last = stall_withhold.load(std::memory_order_relaxed);
  return w;
}
}  // namespace dlrm

extern "C" {

dlrm_status_t attention_test_stall(int64_t wait_limit_ns, int32_t withhold) {
  if (wait_limit_ns < 0) return DLRM_ERR_INVALID_ARG;
  stall_limit_ns.store(wait_limit_ns, std::memory_order_relaxed);
  stall_withhold.store(withhold, std::memory_order_relaxed);
  return DLRM_OK;
}

int64_t history_work_bytes(const dlrm_history_t* h) {
  return check_shape(h) == DLRM_OK ? dlrm::history_work(*h).total : -1;
}

dlrm_status_t history_reset(const dlrm_history_t* h, void* stream) {
  const dlrm_status_t s = check_pool(h);
  if (s != DLRM_OK) return s;
  return status_of(dlrm::launch_history_reset(*h, static_cast<cudaStream_t>(stream)));
}

dlrm_status_t history_append(const dlrm_history_t* h, const int32_t* slots, const int32_t* starts,
                             int32_t batch, const void* k, int64_t ld_k, int64_t ld_k_head,
                             const void* v, int64_t ld_v, int64_t ld_v_head, int64_t rows,
                             int32_t dtype, void* stream) {
  dlrm_status_t s = check_pool(h);
  if (s == DLRM_OK) s = check_slots(h, slots, batch);
  if (s != DLRM_OK) return s;
  if (rows < 0 || !dtype_ok(dtype) || ld_k < 0 || ld_k_head < 0 || ld_v < 0 || ld_v_head < 0)
    return DLRM_ERR_INVALID_ARG;
  if (rows >= (int64_t(1) << 31)) return DLRM_ERR_UNSUPPORTED;
  if (batch == 0 || rows == 0) return DLRM_OK;
  const size_t eb = static_cast<size_t>(dlrm::dtype_bytes(dtype));
  if (!starts || !aligned_to(starts, 4) || !k || !v || !aligned_to(k, eb) || !aligned_to(v, eb))
    return DLRM_ERR_INVALID_ARG;
  return status_of(dlrm::launch_history_append(*h, slots, starts, batch, k, ld_k, ld_k_head, v,
                                               ld_v, ld_v_head, rows, dtype,
                                               static_cast<cudaStream_t>(stream)));
}

dlrm_status_t history_fork(const dlrm_history_t* h, const int32_t* src, const int32_t* dst,
                           int32_t batch, void* stream) {
  dlrm_status_t s = check_pool(h);
  if (s == DLRM_OK) s = check_slots(h, src, batch);
  if (s == DLRM_OK) s = check_slots(h, dst, batch);
  if (s != DLRM_OK || batch == 0) return s;
  return status_of(
      dlrm::launch_history_fork(*h, src, dst, batch, true, static_cast<cudaStream_t>(stream)));
}

dlrm_status_t history_copy(const dlrm_history_t* h, const int32_t* src, const int32_t* dst,
                           int32_t batch, void* stream) {
  dlrm_status_t s = check_pool(h);
  if (s == DLRM_OK) s = check_slots(h, src, batch);
  if (s == DLRM_OK) s = check_slots(h, dst, batch);
  if (s != DLRM_OK || batch == 0) return s;
  return status_of(
      dlrm::launch_history_fork(*h, src, dst, batch, false, static_cast<cudaStream_t>(stream)));
}

dlrm_status_t history_free(const dlrm_history_t* h, const int32_t* slots, int32_t batch,
                           void* stream) {
  dlrm_status_t s = check_pool(h);
  if (s == DLRM_OK) s = check_slots(h, slots, batch);
  if (s != DLRM_OK || batch == 0) return s;
  return status_of(
      dlrm::launch_history_free(*h, slots, batch, 0, 0, static_cast<cudaStream_t>(stream)));
}

dlrm_status_t history_trim(const dlrm_history_t* h, const int32_t* slots, int32_t batch,
                           int32_t window, int32_t sinks, void* stream) {
  dlrm_status_t s = check_pool(h);
  if (s == DLRM_OK) s = check_slots(h, slots, batch);
  if (s != DLRM_OK) return s;
  if (window < 1 || sinks < 0) return DLRM_ERR_INVALID_ARG;
  if (batch == 0) return DLRM_OK;
  return status_of(dlrm::launch_history_free(*h, slots, batch, window, sinks,
                                             static_cast<cudaStream_t>(stream)));
}

dlrm_status_t history_compact(const dlrm_history_t* h, void* stream) {
  const dlrm_status_t s = check_pool(h);
  if (s != DLRM_OK) return s;
  return status_of(dlrm::launch_history_compact(*h, static_cast<cudaStream_t>(stream)));
}

dlrm_status_t history_attention(const dlrm_history_t* h, const dlrm_attention_t* a, void* stream) {
  dlrm_status_t s = check_pool(h);
  if (s != DLRM_OK) return s;
  bool run;
  s = check_attention(a, h->n_heads, &run);
  if (s != DLRM_OK || !run) return s;
  if (!a->slots || !aligned_to(a->slots, 4)) return DLRM_ERR_INVALID_ARG;
  // work units (8 rows of a kv head, 128 events) are counted in int32
  const int64_t tiles = a->q_rows * (a->n_heads / h->n_heads) / 8 + a->batch;
  const int64_t events = static_cast<int64_t>(h->max_pages) * h->page_tokens;
  if (tiles * h->n_heads >= (int64_t(1) << 31) / (events / 128 + 2)) return DLRM_ERR_UNSUPPORTED;
  if (rows_overlap(a->q_rows, a->ld_out, a->n_heads, a->ld_out_head, h->head_dim))
    return DLRM_ERR_INVALID_ARG;
  return status_of(dlrm::launch_history_attention(*h, *a, static_cast<cudaStream_t>(stream)));
}

dlrm_status_t window_attention(const dlrm_attention_t* a, void* stream) {
  if (!a) return DLRM_ERR_INVALID_ARG;
  bool run;
  const dlrm_status_t s = check_attention(a, a->n_kv_heads, &run);
  if (s != DLRM_OK) return s;
  if (!head_dim_ok(a->head_dim)) return a->head_dim < 1 ? DLRM_ERR_INVALID_ARG : DLRM_ERR_UNSUPPORTED;
  if (a->k_rows < 0 || a->ld_k < 0 || a->ld_k_head < 0 || a->ld_v < 0 || a->ld_v_head < 0)
    return DLRM_ERR_INVALID_ARG;
  if (a->k_rows >= kRowLimit) return DLRM_ERR_UNSUPPORTED;
  if (!run) return DLRM_OK;
  const size_t eb = static_cast<size_t>(dlrm::dtype_bytes(a->dtype));
  if (!a->k_starts || !aligned_to(a->k_starts, 4)) return DLRM_ERR_INVALID_ARG;
  if (a->k_rows > 0 && (!a->k || !a->v || !aligned_to(a->k, eb) || !aligned_to(a->v, eb)))
    return DLRM_ERR_INVALID_ARG;
  // CTAs of one launch
  const int64_t group = a->n_heads / a->n_kv_heads;
  if ((a->q_rows * group / 64 + a->batch) * a->n_kv_heads >= (int64_t(1) << 31))
    return DLRM_ERR_UNSUPPORTED;
  if (rows_overlap(a->q_rows, a->ld_out, a->n_heads, a->ld_out_head, a->head_dim))
    return DLRM_ERR_INVALID_ARG;
  return status_of(dlrm::launch_window_attention(*a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
