// Host side of the rotary and paged-cache entry points: argument checks, handles, launches.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <new>

#include "../../include/spa.h"
#include "spa_paged.cuh"

struct spa_rope {
  spa::RopeTabAny tab;
};

struct spa_paged {
  spa_paged_config cfg;
  spa::RopeTab128 tab;
  int G;
  int device;
  int num_sms;
  int grid;             // CTAs of the attention kernel
  int64_t capacity;     // tokens of a sequence
  void* mem;
  float* part;
  unsigned* ticket;
  unsigned* err;
};

namespace {

spa_status fail(spa_status code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return spa::set_last_error(code, buf);
}
spa_status cuda_fail(cudaError_t e, const char* what) {
  return fail(SPA_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}
bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

constexpr double kPi = 3.141592653589793238462643383279502884;

spa_status fill_table(const spa_rope_config& c, spa::RopeTabAny* t) {
  const int n = c.rot_dim / 2;
  double theta = c.theta;
  if (c.scaling == SPA_ROPE_BASE) theta *= std::pow(c.factor, (double)c.rot_dim / (c.rot_dim - 2));
  if (!std::isfinite(theta)) return fail(SPA_ERR_INVALID_ARG, "theta * factor^(rot_dim / (rot_dim - 2)) is not finite");
  double first = 0, last = 0;
  if (c.scaling == SPA_ROPE_RAMP) {
    auto dim = [&](double turns) { return c.rot_dim * std::log((double)c.orig_ctx / (2 * kPi * turns)) / (2 * std::log(theta)); };
    const double top = c.rot_dim - 1;
    first = std::fmin(std::fmax(std::floor(dim(c.high)), 0.0), top);
    last = std::fmin(std::fmax(std::ceil(dim(c.low)), 0.0), top);
    if (last <= first) last = first + 0.001;
  }
  for (int i = 0; i < n; ++i) {
    double f = std::pow(theta, -2.0 * i / c.rot_dim), keep = 1.0;
    if (c.scaling == SPA_ROPE_LINEAR) f /= c.factor;
    if (c.scaling == SPA_ROPE_BANDS) keep = ((double)c.orig_ctx * f / (2 * kPi) - c.low) / (c.high - c.low);
    if (c.scaling == SPA_ROPE_RAMP) keep = 1.0 - (i - first) / (last - first);
    keep = std::fmin(std::fmax(keep, 0.0), 1.0);
    if (c.scaling == SPA_ROPE_BANDS || c.scaling == SPA_ROPE_RAMP) f *= keep + (1.0 - keep) / c.factor;
    t->f_pi[i] = f / kPi;
  }
  t->rot = c.rot_dim;
  t->interleaved = c.layout == SPA_ROPE_INTERLEAVED;
  t->mag = c.magnitude != 0.0 ? c.magnitude : 1.0;
  for (int i = 0; i < n; ++i)
    if (!std::isfinite(t->f_pi[i])) return fail(SPA_ERR_INVALID_ARG, "the configuration gives frequency %d no finite value", i);
  return SPA_OK;
}

// (batch, token, head) strides of a call's tensor: the caller's, or dense [B][heads][T][d].
spa::Strides3 strides_of(const int64_t* s, int T, int heads, int d) {
  if (s) return {s[0], s[1], s[2]};
  return {(int64_t)heads * T * d, d, (int64_t)T * d};
}
bool strides_aligned(const spa::Strides3& s, int elem_size) {
  return ((s.b * elem_size) | (s.t * elem_size) | (s.h * elem_size)) % 16 == 0;
}

spa_status check_paged_config(const spa_paged_config* c) {
  if (!c) return fail(SPA_ERR_INVALID_ARG, "config is NULL");
  if (c->head_dim != 128) return fail(SPA_ERR_UNSUPPORTED, "head_dim must be 128 (got %d)", c->head_dim);
  if (c->kv_dtype != SPA_BF16 && c->kv_dtype != SPA_F32)
    return fail(SPA_ERR_UNSUPPORTED, "kv_dtype must be SPA_BF16 or SPA_F32 (got %d)", c->kv_dtype);
  if (c->page_format != SPA_PAGE_INT4 && c->page_format != SPA_PAGE_BF16)
    return fail(SPA_ERR_UNSUPPORTED, "page_format must be SPA_PAGE_INT4 or SPA_PAGE_BF16 (got %d)", c->page_format);
  if (c->n_kv_heads < 1 || c->n_kv_heads > spa::kMaxKvHeads)
    return fail(SPA_ERR_UNSUPPORTED, "n_kv_heads must be in [1, %d] (got %d)", spa::kMaxKvHeads, c->n_kv_heads);
  if (c->n_q_heads < 1 || c->n_q_heads % c->n_kv_heads != 0)
    return fail(SPA_ERR_INVALID_ARG, "n_q_heads (%d) must be a positive multiple of n_kv_heads (%d)", c->n_q_heads,
                c->n_kv_heads);
  if (c->n_q_heads / c->n_kv_heads > spa::kMaxGroup)
    return fail(SPA_ERR_UNSUPPORTED, "GQA group size must be in [1, %d] (got %d)", spa::kMaxGroup,
                c->n_q_heads / c->n_kv_heads);
  if (c->max_batch < 1 || (int64_t)c->max_batch * c->n_kv_heads > spa::kMaxPagedSlices)
    return fail(SPA_ERR_INVALID_ARG, "max_batch must be >= 1 with max_batch*n_kv_heads <= %d (got %d)",
                spa::kMaxPagedSlices, c->max_batch);
  if (c->page_size < 16 || c->page_size % 16 != 0 || c->page_size > 65536)
    return fail(SPA_ERR_INVALID_ARG, "page_size must be a multiple of 16 in [16, 65536] (got %d)", c->page_size);
  if (c->n_pages < 1) return fail(SPA_ERR_INVALID_ARG, "n_pages must be >= 1 (got %d)", c->n_pages);
  if (c->max_pages < 1 || (int64_t)c->max_pages * c->page_size > spa::kMaxCtx)
    return fail(SPA_ERR_INVALID_ARG, "max_pages must be >= 1 with max_pages*page_size <= 2^24 (got %d)", c->max_pages);
  return SPA_OK;
}

struct PagedPlan {
  size_t part, ticket, err, total;
};
PagedPlan plan(const spa_paged_config& c, int grid) {
  const size_t slices = (size_t)c.max_batch * c.n_kv_heads;
  PagedPlan p;
  p.part = 0;
  p.ticket = (grid + slices) * spa::kMergeWords * 4;
  p.err = (p.ticket + slices * 4 + 255) / 256 * 256;
  p.total = p.err + 256;
  return p;
}

spa_status check_device(const spa_paged* h) {
  int dev = -1;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev != h->device)
    return fail(SPA_ERR_INVALID_ARG, "the handle was created on device %d, the current device is %d", h->device, dev);
  return SPA_OK;
}
// Checks that every call on a paged cache shares.
spa_status check_call(const spa_paged* h, const void* pages, const int32_t* block_table, int B) {
  if (!h) return fail(SPA_ERR_INVALID_ARG, "handle is NULL");
  if (!pages || !block_table) return fail(SPA_ERR_INVALID_ARG, "pages and block_table must be non-NULL");
  if (!aligned(pages, 16) || !aligned(block_table, 4))
    return fail(SPA_ERR_INVALID_ARG, "pages must be 16-byte aligned, block_table 4-byte aligned");
  if (B < 1 || B > h->cfg.max_batch)
    return fail(SPA_ERR_INVALID_ARG, "B must be in [1, max_batch=%d] (got %d)", h->cfg.max_batch, B);
  return check_device(h);
}
spa::PagePool pool_of(const spa_paged* h, const void* pages, const int32_t* table) {
  const spa_paged_config& c = h->cfg;
  spa::PagePool p;
  p.pages = static_cast<unsigned char*>(const_cast<void*>(pages));
  p.table = table;
  p.Hkv = c.n_kv_heads;
  p.n_pages = c.n_pages;
  p.max_pages = c.max_pages;
  p.page_blocks = c.page_size / spa::kBlockTok;
  p.page_size = c.page_size;
  p.head_bytes = (int64_t)p.page_blocks * (c.page_format == SPA_PAGE_INT4 ? spa::kBlockBytes4 : spa::kBlockBytes16);
  p.err = h->err;
  return p;
}
// Row tensors of an append or a read.
spa_status check_rows(const spa_paged* h, const void* k, const void* v, const int64_t* start, const int64_t* n, int T,
                      const spa::Strides3& ks, const spa::Strides3& vs) {
  if (!k || !v || !start) return fail(SPA_ERR_INVALID_ARG, "the key rows, value rows and start_pos must be non-NULL");
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(start, 8) || !aligned(n, 8))
    return fail(SPA_ERR_INVALID_ARG, "key and value rows must be 16-byte aligned, start_pos and the row counts 8-byte aligned");
  const int es = h->cfg.kv_dtype == SPA_BF16 ? 2 : 4;
  if (!strides_aligned(ks, es) || !strides_aligned(vs, es))
    return fail(SPA_ERR_INVALID_ARG, "strides must be multiples of 16 bytes");
  if (T < 1 || T > h->capacity)
    return fail(SPA_ERR_INVALID_ARG, "T must be in [1, max_pages*page_size=%lld] (got %d)", (long long)h->capacity, T);
  return SPA_OK;
}

}  // namespace

extern "C" {

spa_status spa_rope_create(spa_rope** out, const spa_rope_config* c) {
  if (!out) return fail(SPA_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (!c) return fail(SPA_ERR_INVALID_ARG, "config is NULL");
  if (c->rot_dim < 2 || c->rot_dim % 2 != 0 || c->rot_dim > 2 * spa::kMaxRopePairs)
    return fail(SPA_ERR_INVALID_ARG, "rot_dim must be even in [2, %d] (got %d)", 2 * spa::kMaxRopePairs, c->rot_dim);
  if (c->layout != SPA_ROPE_HALF && c->layout != SPA_ROPE_INTERLEAVED)
    return fail(SPA_ERR_INVALID_ARG, "layout must be SPA_ROPE_HALF or SPA_ROPE_INTERLEAVED (got %d)", c->layout);
  if (c->scaling < SPA_ROPE_PLAIN || c->scaling > SPA_ROPE_RAMP)
    return fail(SPA_ERR_INVALID_ARG, "scaling must be one of SPA_ROPE_PLAIN .. SPA_ROPE_RAMP (got %d)", c->scaling);
  if (!(c->theta > 0.0) || !std::isfinite(c->theta)) return fail(SPA_ERR_INVALID_ARG, "theta must be positive and finite");
  if (!(c->magnitude >= 0.0) || !(c->magnitude <= 1e4))
    return fail(SPA_ERR_INVALID_ARG, "magnitude must be in [0, 1e4] (0 selects 1)");
  if (c->scaling != SPA_ROPE_PLAIN && (!(c->factor > 0.0) || !std::isfinite(c->factor)))
    return fail(SPA_ERR_INVALID_ARG, "factor must be positive and finite");
  if (c->scaling == SPA_ROPE_BASE && c->rot_dim < 4) return fail(SPA_ERR_INVALID_ARG, "SPA_ROPE_BASE needs rot_dim >= 4");
  if (c->scaling == SPA_ROPE_BANDS || c->scaling == SPA_ROPE_RAMP) {
    if (c->orig_ctx < 1) return fail(SPA_ERR_INVALID_ARG, "orig_ctx must be >= 1 (got %lld)", (long long)c->orig_ctx);
    if (!(c->low > 0.0) || !(c->high > c->low) || !std::isfinite(c->high))
      return fail(SPA_ERR_INVALID_ARG, "need 0 < low < high, finite");
    if (c->scaling == SPA_ROPE_RAMP && !(c->theta > 1.0)) return fail(SPA_ERR_INVALID_ARG, "SPA_ROPE_RAMP needs theta > 1");
  }
  spa_rope* r = new (std::nothrow) spa_rope;
  if (!r) return fail(SPA_ERR_WORKSPACE, "out of host memory");
  std::memset(&r->tab, 0, sizeof r->tab);
  const spa_status s = fill_table(*c, &r->tab);
  if (s) {
    delete r;
    return s;
  }
  *out = r;
  return SPA_OK;
}

spa_status spa_rope_destroy(spa_rope* r) {
  delete r;
  return SPA_OK;
}

spa_status spa_rope_inv_freq(const spa_rope* r, double* inv_freq, int n) {
  if (!r || !inv_freq) return fail(SPA_ERR_INVALID_ARG, "the table and inv_freq must be non-NULL");
  if (n != r->tab.rot / 2) return fail(SPA_ERR_INVALID_ARG, "n must be rot_dim / 2 = %d (got %d)", r->tab.rot / 2, n);
  for (int i = 0; i < n; ++i) inv_freq[i] = r->tab.f_pi[i] * kPi;
  return SPA_OK;
}

spa_status spa_rope_apply(const spa_rope* r, const void* x, const int64_t* x_strides, void* y, const int64_t* y_strides,
                          const int64_t* start_pos, const int64_t* positions, int B, int T, int n_heads, int head_dim,
                          int dtype, int transpose, spa_stream stream) {
  if (!r) return fail(SPA_ERR_INVALID_ARG, "the rotation is NULL");
  if (!x || !y) return fail(SPA_ERR_INVALID_ARG, "x and y must be non-NULL");
  if ((start_pos != nullptr) == (positions != nullptr))
    return fail(SPA_ERR_INVALID_ARG, "exactly one of start_pos and positions must be non-NULL");
  if (dtype != SPA_BF16 && dtype != SPA_F32) return fail(SPA_ERR_UNSUPPORTED, "dtype must be SPA_BF16 or SPA_F32 (got %d)", dtype);
  const unsigned es = dtype == SPA_BF16 ? 2 : 4;
  if (!aligned(x, es) || !aligned(y, es) || !aligned(start_pos, 8) || !aligned(positions, 8))
    return fail(SPA_ERR_INVALID_ARG, "x and y must be aligned to their elements, the positions 8-byte aligned");
  if (B < 1 || T < 1 || n_heads < 1) return fail(SPA_ERR_INVALID_ARG, "B, T and n_heads must be >= 1 (got %d, %d, %d)", B, T, n_heads);
  if (head_dim < r->tab.rot || head_dim > 65536)
    return fail(SPA_ERR_INVALID_ARG, "head_dim must be in [rot_dim=%d, 65536] (got %d)", r->tab.rot, head_dim);
  const cudaError_t e = spa::launch_rope(x, y, strides_of(x_strides, T, n_heads, head_dim), strides_of(y_strides, T, n_heads, head_dim),
                                         start_pos, positions, B, T, n_heads, head_dim, dtype, transpose, r->tab,
                                         reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "rope");
  return SPA_OK;
}

spa_status spa_paged_page_bytes(const spa_paged_config* cfg, size_t* bytes) {
  const spa_status r = check_paged_config(cfg);
  if (r) return r;
  if (!bytes) return fail(SPA_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = (size_t)cfg->n_kv_heads * (cfg->page_size / spa::kBlockTok) *
           (cfg->page_format == SPA_PAGE_INT4 ? spa::kBlockBytes4 : spa::kBlockBytes16);
  return SPA_OK;
}

spa_status spa_paged_create(spa_paged** out, const spa_paged_config* cfg, const spa_rope* rope) {
  if (!out) return fail(SPA_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  const spa_status r = check_paged_config(cfg);
  if (r) return r;
  if (rope && rope->tab.rot > cfg->head_dim)
    return fail(SPA_ERR_INVALID_ARG, "the rotation's rot_dim (%d) exceeds head_dim", rope->tab.rot);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  int major = 0, minor = 0;
  cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
  if (major != 10 || minor != 0)
    return fail(SPA_ERR_UNSUPPORTED, "libspa is built for sm_100a (B200); device %d is sm_%d%d", dev, major, minor);
  spa_paged* h = new (std::nothrow) spa_paged;
  if (!h) return fail(SPA_ERR_WORKSPACE, "out of host memory");
  std::memset(h, 0, sizeof *h);
  h->cfg = *cfg;
  h->G = cfg->n_q_heads / cfg->n_kv_heads;
  h->device = dev;
  h->capacity = (int64_t)cfg->max_pages * cfg->page_size;
  if (rope) {
    h->tab.rot = rope->tab.rot;
    h->tab.interleaved = rope->tab.interleaved;
    h->tab.mag = rope->tab.mag;
    std::memcpy(h->tab.f_pi, rope->tab.f_pi, sizeof h->tab.f_pi);
  } else {
    h->tab.mag = 1.0;
  }
  cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, dev);
  h->grid = h->num_sms < spa::kMaxAttendCtas ? h->num_sms : spa::kMaxAttendCtas;
  if (!spa::page_attend_setup(cfg->page_format)) {
    e = cudaGetLastError();
    delete h;
    return cuda_fail(e, "spa_paged_create: attention kernel set-up");
  }
  const PagedPlan p = plan(*cfg, h->grid);
  if ((e = cudaMalloc(&h->mem, p.total)) != cudaSuccess) {
    delete h;
    return fail(SPA_ERR_WORKSPACE, "cudaMalloc of %zu workspace bytes failed: %s", p.total, cudaGetErrorString(e));
  }
  char* base = static_cast<char*>(h->mem);
  h->part = reinterpret_cast<float*>(base + p.part);
  h->ticket = reinterpret_cast<unsigned*>(base + p.ticket);
  h->err = reinterpret_cast<unsigned*>(base + p.err);
  if ((e = cudaMemset(h->ticket, 0, p.total - p.ticket)) != cudaSuccess || (e = cudaDeviceSynchronize()) != cudaSuccess) {
    cudaFree(h->mem);
    delete h;
    return cuda_fail(e, "spa_paged_create: clearing the workspace");
  }
  *out = h;
  return SPA_OK;
}

spa_status spa_paged_destroy(spa_paged* h) {
  if (!h) return SPA_OK;
  int dev = h->device;
  cudaGetDevice(&dev);
  if (dev != h->device) cudaSetDevice(h->device);
  cudaDeviceSynchronize();
  const cudaError_t e = cudaFree(h->mem);
  if (dev != h->device) cudaSetDevice(dev);
  delete h;
  if (e != cudaSuccess) return cuda_fail(e, "cudaFree");
  return SPA_OK;
}

spa_status spa_paged_status(spa_paged* h, spa_stream stream) {
  if (!h) return fail(SPA_ERR_INVALID_ARG, "handle is NULL");
  const spa_status r = check_device(h);
  if (r) return r;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  unsigned w = 0;
  cudaError_t e;
  if ((e = cudaMemcpyAsync(&w, h->err, 4, cudaMemcpyDeviceToHost, st)) != cudaSuccess ||
      (e = cudaStreamSynchronize(st)) != cudaSuccess)
    return cuda_fail(e, "spa_paged_status");
  if (w == 0) return SPA_OK;
  // Only what was read: appends and reads of other streams may have set more since.
  if ((e = spa::launch_clear_bits(h->err, w, st)) != cudaSuccess || (e = cudaStreamSynchronize(st)) != cudaSuccess)
    return cuda_fail(e, "spa_paged_status");
  if (w & spa::kErrTimeout) return fail(SPA_ERR_DEVICE_TIMEOUT, "a copy into shared memory did not arrive in time; outputs are not valid");
  return fail(SPA_ERR_DEVICE_RANGE, "out of range on the device:%s%s%s%s", w & spa::kErrSeqLen ? " a length (clamped);" : "",
              w & spa::kErrStartPos ? " a position (row skipped);" : "", w & spa::kErrPage ? " a block_table entry (rows skipped);" : "",
              w & spa::kErrList ? " a selected count or position (skipped);" : "");
}

spa_status spa_kv_append_paged(spa_paged* h, const void* k_pre, const int64_t* k_strides, const void* v_new,
                               const int64_t* v_strides, const int64_t* start_pos, const int64_t* n_new_opt, int B, int T,
                               const int32_t* block_table, void* pages, spa_stream stream) {
  spa_status r = check_call(h, pages, block_table, B);
  if (r) return r;
  spa::AppendArgs a{};
  a.ks = strides_of(k_strides, T, h->cfg.n_kv_heads, 128);
  a.vs = strides_of(v_strides, T, h->cfg.n_kv_heads, 128);
  if ((r = check_rows(h, k_pre, v_new, start_pos, n_new_opt, T, a.ks, a.vs))) return r;
  a.k = k_pre;
  a.v = v_new;
  a.start = start_pos;
  a.n_new = n_new_opt;
  a.B = B;
  a.T = T;
  const cudaError_t e = spa::launch_page_append(pool_of(h, pages, block_table), a, h->cfg.kv_dtype, h->cfg.page_format, h->tab,
                                                h->num_sms, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "page append");
  return SPA_OK;
}

spa_status spa_kv_read_paged(spa_paged* h, const void* pages, const int32_t* block_table, const int64_t* start_pos,
                             const int64_t* n_rows_opt, int B, int T, void* k_rows, const int64_t* k_strides, void* v_rows,
                             const int64_t* v_strides, spa_stream stream) {
  spa_status r = check_call(h, pages, block_table, B);
  if (r) return r;
  spa::ReadArgs a{};
  a.ks = strides_of(k_strides, T, h->cfg.n_kv_heads, 128);
  a.vs = strides_of(v_strides, T, h->cfg.n_kv_heads, 128);
  if ((r = check_rows(h, k_rows, v_rows, start_pos, n_rows_opt, T, a.ks, a.vs))) return r;
  a.k = k_rows;
  a.v = v_rows;
  a.start = start_pos;
  a.n_rows = n_rows_opt;
  a.B = B;
  a.T = T;
  const cudaError_t e = spa::launch_page_read(pool_of(h, pages, block_table), a, h->cfg.kv_dtype, h->cfg.page_format,
                                              reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "page read");
  return SPA_OK;
}

spa_status spa_attend_paged(spa_paged* h, const void* q_pre, const void* pages, const int32_t* block_table,
                            const int64_t* seq_lens, int B, int64_t max_seq_len, const uint8_t* head_mask_opt, int n_sink,
                            int window, const int32_t* sel_idx_opt, const int32_t* sel_count_opt, int64_t sel_stride,
                            float* out, float* lse_opt, spa_stream stream) {
  spa_status r = check_call(h, pages, block_table, B);
  if (r) return r;
  if (!q_pre || !seq_lens || !out) return fail(SPA_ERR_INVALID_ARG, "q_pre, seq_lens and out must be non-NULL");
  if (!aligned(q_pre, 16) || !aligned(out, 16) || !aligned(seq_lens, 8) || !aligned(lse_opt, 4))
    return fail(SPA_ERR_INVALID_ARG, "q_pre and out must be 16-byte aligned, seq_lens 8-byte, lse_opt 4-byte aligned");
  if (max_seq_len < 0 || max_seq_len > h->capacity)
    return fail(SPA_ERR_INVALID_ARG, "max_seq_len must be in [0, max_pages*page_size=%lld] (got %lld)", (long long)h->capacity,
                (long long)max_seq_len);
  if ((sel_idx_opt != nullptr) != (sel_count_opt != nullptr))
    return fail(SPA_ERR_INVALID_ARG, "sel_idx and sel_count come together");
  if (sel_idx_opt && !head_mask_opt) return fail(SPA_ERR_INVALID_ARG, "a selection needs the head mask");
  if (sel_idx_opt && (!aligned(sel_idx_opt, 4) || !aligned(sel_count_opt, 4) || sel_stride < 1 || sel_stride > spa::kMaxCtx))
    return fail(SPA_ERR_INVALID_ARG, "sel_idx and sel_count must be 4-byte aligned, sel_stride in [1, 2^24] (got %lld)",
                (long long)sel_stride);
  if (head_mask_opt && (n_sink < 0 || window < 0 || (int64_t)n_sink + window < 1))
    return fail(SPA_ERR_INVALID_ARG, "n_sink, window must be >= 0 with n_sink + window >= 1");
  spa::PagedAttendArgs a;
  std::memset(&a, 0, sizeof a);
  a.pool = pool_of(h, pages, block_table);
  a.q = q_pre;
  a.seq_lens = seq_lens;
  a.list = sel_idx_opt;
  a.list_count = sel_count_opt;
  a.list_stride = sel_stride;
  a.out = out;
  a.lse = lse_opt;
  a.part = h->part;
  a.ticket = h->ticket;
  a.B = B;
  a.Hq = h->cfg.n_q_heads;
  a.G = h->G;
  a.n_slices = B * h->cfg.n_kv_heads;
  a.cap = max_seq_len ? max_seq_len : h->capacity;
  a.q_f32 = h->cfg.kv_dtype == SPA_F32;
  a.n_sink = n_sink;
  a.window = window;
  a.by_heads = (unsigned)(((1ull << 32) + h->cfg.n_kv_heads - 1) / h->cfg.n_kv_heads);
  a.by_blocks = (unsigned)(((1ull << 32) + a.pool.page_blocks - 1) / a.pool.page_blocks);
  a.scale_log2 = (float)(1.4426950408889634 / std::sqrt(128.0));
  for (int g = 0; g < h->cfg.n_kv_heads; ++g) {
    const bool ret = !head_mask_opt || head_mask_opt[g];
    a.all_rows[g] = ret && !sel_idx_opt;
    a.has_list[g] = ret && sel_idx_opt;
  }
  const cudaError_t e = spa::launch_page_attend(a, h->cfg.page_format, h->grid, h->tab, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "page attend");
  return SPA_OK;
}

}  // extern "C"
