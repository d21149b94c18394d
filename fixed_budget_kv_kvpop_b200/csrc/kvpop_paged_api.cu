// Host side of the paged cache and of kvpop_qk_norm_rope (include/kvpop.h):
// validation, device buffer layout, launches.
#include <atomic>
#include <cmath>
#include <new>

#include "kvpop_paged.cuh"

using namespace kvpop;

namespace {

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int element_size(int dtype) { return dtype == KVPOP_DTYPE_F32 ? 4 : 2; }

struct PagedLayout {
  size_t pages_off, pages_stride, scales_off, scales_stride, scratch_off, err_off, total;
};

int validate(const kvpop_paged_config* c) {
  if (!c) return KVPOP_ERR_INVALID_ARG;
  if (c->dtype != KVPOP_DTYPE_F32 && c->dtype != KVPOP_DTYPE_BF16) return KVPOP_ERR_INVALID_ARG;
  if (c->cache_format != KVPOP_CACHE_NATIVE && c->cache_format != KVPOP_CACHE_E4M3) return KVPOP_ERR_INVALID_ARG;
  if (c->cache_format == KVPOP_CACHE_E4M3 && c->dtype != KVPOP_DTYPE_BF16) return KVPOP_ERR_INVALID_ARG;
  if (c->n_layers < 1 || c->n_pages < 1 || c->max_batch < 1 || c->max_batch > 1024) return KVPOP_ERR_BAD_SHAPE;
  if (c->n_kv_heads < 1 || c->n_kv_heads > 1024 || c->n_q_heads < 1) return KVPOP_ERR_BAD_SHAPE;
  if (c->n_q_heads % c->n_kv_heads != 0 || c->n_q_heads / c->n_kv_heads > kMaxGroup) return KVPOP_ERR_BAD_SHAPE;
  if (c->head_dim != 64 && c->head_dim != 128) return KVPOP_ERR_BAD_SHAPE;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128 && c->page_size != 256)
    return KVPOP_ERR_BAD_SHAPE;
  if (static_cast<int64_t>(c->n_pages) * c->page_size > 2147483647) return KVPOP_ERR_BAD_SHAPE;
  if (static_cast<int64_t>(c->n_pages) * c->n_kv_heads > 2147483647) return KVPOP_ERR_BAD_SHAPE;   // a copy's coordinate
  // the bytes of all layers stay far below 2^63
  const double bytes = static_cast<double>(c->n_layers) * c->n_pages * c->page_size * c->n_kv_heads * 2.0 *
                       c->head_dim * 4.0;
  if (bytes > 1e18) return KVPOP_ERR_BAD_SHAPE;
  return KVPOP_OK;
}

PagedLayout make_layout(const kvpop_paged_config* c) {
  PagedLayout L{};
  const size_t rows = static_cast<size_t>(c->n_pages) * c->n_kv_heads * 2 * c->page_size;
  const bool e8 = c->cache_format == KVPOP_CACHE_E4M3;
  size_t off = 0;
  L.pages_stride = align256(rows * c->head_dim * (e8 ? 1 : element_size(c->dtype)));
  L.pages_off = off; off += c->n_layers * L.pages_stride;
  L.scales_stride = e8 ? align256(rows * 4) : 0;
  L.scales_off = e8 ? off : 0; off += c->n_layers * L.scales_stride;
  L.scratch_off = off;
  off += align256(attend_scratch_bytes(c->n_q_heads / c->n_kv_heads, c->head_dim, c->max_batch * c->n_kv_heads));
  L.err_off = off; off += 256;
  L.total = off;
  return L;
}

// Makes a device current for the scope of a call.
class DeviceScope {
 public:
  explicit DeviceScope(int device) {
    ok_ = cudaGetDevice(&before_) == cudaSuccess;
    if (ok_ && before_ != device) {
      ok_ = cudaSetDevice(device) == cudaSuccess;
      changed_ = ok_;
    }
  }
  ~DeviceScope() { if (changed_) cudaSetDevice(before_); }
  bool ok() const { return ok_; }
 private:
  int before_ = 0;
  bool ok_ = false, changed_ = false;
};

// The device that p's memory belongs to; false when it is not device memory.
bool device_of(const void* p, int* device) {
  cudaPointerAttributes at;
  if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  *device = at.device;
  return at.type == cudaMemoryTypeDevice || at.type == cudaMemoryTypeManaged;
}

// Checks rows of [batch][n_tokens][heads][d] and converts them.
bool rows_view(const kvpop_rows* r, int batch, int n_tokens, int heads, int esize, bool written, RowsView* out) {
  if (!r || !r->data || !aligned(r->data, 16)) return false;
  const int64_t stride[3] = {r->batch_stride, r->token_stride, r->head_stride};
  const int64_t n[3] = {batch, n_tokens, heads};
  for (int i = 0; i < 3; ++i) {
    if (n[i] <= 1) continue;
    if (stride[i] < 0 || (stride[i] * esize) % 16 != 0 || stride[i] > (INT64_C(1) << 40)) return false;
    if (written && stride[i] == 0) return false;
  }
  *out = RowsView{static_cast<uint8_t*>(r->data), r->batch_stride, r->token_stride, r->head_stride};
  return true;
}

bool rope_args(const kvpop_rope* r, int head_dim, RopeArgs* out, int* status) {
  *status = KVPOP_ERR_INVALID_ARG;
  if (!r) return false;
  if (r->rot_dim < 0 || r->rot_dim > head_dim || r->rot_dim % 8 != 0) {
    *status = KVPOP_ERR_BAD_SHAPE;
    return false;
  }
  if (!(r->eps >= 0.f) || !std::isfinite(r->eps) || !std::isfinite(r->rot_scale)) return false;
  if (r->interleaved != 0 && r->interleaved != 1) return false;
  if (!aligned(r->q_weight, 16) || !aligned(r->k_weight, 16) || !aligned(r->inv_freq, 8)) return false;
  if (r->rot_dim > 0 && !r->inv_freq) return false;
  *out = RopeArgs{r->q_weight, r->k_weight, r->inv_freq, r->eps, r->rot_scale, r->rot_dim, r->interleaved};
  return true;
}

int sm_count(int device) {
  static std::atomic<int> known[64];     // a device's count does not change
  int sms = device < 64 ? known[device].load(std::memory_order_relaxed) : 0;
  if (sms != 0) return sms;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) return 0;
  if (device < 64) known[device].store(sms, std::memory_order_relaxed);
  return sms;
}

// A CUDA call failed.  Its error is taken back: it belongs to this call alone, and the fixed-budget calls ask for the
// thread's last error after their launches.
int cuda_failed() {
  cudaGetLastError();
  return KVPOP_ERR_CUDA;
}

int status_of(int r) { return r == 0 ? KVPOP_OK : r == -2 ? KVPOP_ERR_BAD_SHAPE : cuda_failed(); }

}  // namespace

struct kvpop_paged_handle {
  kvpop_paged_config cfg;
  PagedLayout lay;
  uint8_t* mem;
  int device, num_sms, page_shift;
  CUtensorMap* maps = nullptr;   // per layer
  ~kvpop_paged_handle() { delete[] maps; }
};

namespace {

PagedLayer paged_layer(const kvpop_paged_handle* h, int layer) {
  PagedLayer p{};
  p.pages = h->mem + h->lay.pages_off + layer * h->lay.pages_stride;
  if (h->cfg.cache_format == KVPOP_CACHE_E4M3)
    p.scales = reinterpret_cast<float*>(h->mem + h->lay.scales_off + layer * h->lay.scales_stride);
  p.err = reinterpret_cast<int32_t*>(h->mem + h->lay.err_off);
  p.n_pages = h->cfg.n_pages;
  p.page_shift = h->page_shift;
  p.Hkv = h->cfg.n_kv_heads;
  return p;
}

// 0 (the default) or a factor whose products and reciprocals with the kernel's constants stay normal numbers.
bool factor_ok(float x) { return x == 0.f || (x >= 0x1p-100f && x <= 0x1p100f); }

bool bad_layer(const kvpop_paged_handle* h, int32_t layer) { return !h || layer < 0 || layer >= h->cfg.n_layers; }

// Page table and lengths of `batch` sequences.
bool tables_ok(const int32_t* table, int64_t stride, int32_t width, const int32_t* lens, int32_t batch) {
  if ((!table && width > 0) || !lens || !aligned(table, 4) || !aligned(lens, 4)) return false;
  return batch <= 1 || (stride >= width && stride <= (INT64_C(1) << 40));
}

}  // namespace

extern "C" {

int kvpop_qk_norm_rope(int32_t dtype, int32_t head_dim, int32_t n_q_heads, int32_t n_kv_heads,
                       const kvpop_rope* rope, int32_t batch, int32_t n_tokens, const kvpop_rows* q,
                       const kvpop_rows* k, const int32_t* positions, const kvpop_rows* q_out,
                       const kvpop_rows* k_out, void* stream) {
  if (dtype != KVPOP_DTYPE_F32 && dtype != KVPOP_DTYPE_BF16) return KVPOP_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return KVPOP_ERR_BAD_SHAPE;
  if (n_q_heads < 1 || n_q_heads > 16384 || n_kv_heads < 1 || n_kv_heads > 1024) return KVPOP_ERR_BAD_SHAPE;
  if (batch < 0 || n_tokens < 0) return KVPOP_ERR_INVALID_ARG;
  HeadsArgs a{};
  int status;
  if (!rope_args(rope, head_dim, &a.rope, &status)) return status;
  if (batch == 0 || n_tokens == 0) return KVPOP_OK;
  if (static_cast<int64_t>(batch) * n_tokens > (1 << 30)) return KVPOP_ERR_BAD_SHAPE;
  const int es = element_size(dtype);
  if (!positions || !aligned(positions, 4)) return KVPOP_ERR_INVALID_ARG;
  if (!rows_view(q, batch, n_tokens, n_q_heads, es, false, &a.q) ||
      !rows_view(k, batch, n_tokens, n_kv_heads, es, false, &a.k) ||
      !rows_view(q_out, batch, n_tokens, n_q_heads, es, true, &a.qo) ||
      !rows_view(k_out, batch, n_tokens, n_kv_heads, es, true, &a.ko))
    return KVPOP_ERR_INVALID_ARG;
  int device = 0;
  if (!device_of(q->data, &device)) return KVPOP_ERR_INVALID_ARG;
  DeviceScope scope(device);
  if (!scope.ok()) return cuda_failed();
  const int sms = sm_count(device);
  if (sms == 0) return cuda_failed();
  a.pos = positions;
  a.batch = batch; a.n_tokens = n_tokens; a.Hq = n_q_heads; a.Hkv = n_kv_heads;
  return status_of(launch_heads(a, dtype, head_dim, HEADS_DENSE, sms, static_cast<cudaStream_t>(stream)));
}

int kvpop_paged_bytes(const kvpop_paged_config* cfg, size_t* bytes) {
  if (!bytes) return KVPOP_ERR_INVALID_ARG;
  const int v = validate(cfg);
  if (v != KVPOP_OK) return v;
  *bytes = make_layout(cfg).total;
  return KVPOP_OK;
}

int kvpop_paged_create(const kvpop_paged_config* cfg, void* dev_mem, size_t bytes, kvpop_paged_handle** out) {
  if (!out) return KVPOP_ERR_INVALID_ARG;
  *out = nullptr;
  const int v = validate(cfg);
  if (v != KVPOP_OK) return v;
  const PagedLayout L = make_layout(cfg);
  if (!dev_mem || bytes < L.total || !aligned(dev_mem, 256)) return KVPOP_ERR_INVALID_ARG;
  int dev = 0, at = 0;
  if (!device_of(dev_mem, &at)) return KVPOP_ERR_INVALID_ARG;
  if (cudaGetDevice(&dev) != cudaSuccess) return cuda_failed();
  if (at != dev) return KVPOP_ERR_INVALID_ARG;
  const int sms = sm_count(dev);
  if (sms == 0) return cuda_failed();
  kvpop_paged_handle* h = new (std::nothrow) kvpop_paged_handle();
  if (!h) return KVPOP_ERR_INVALID_ARG;
  h->cfg = *cfg;
  h->lay = L;
  h->mem = static_cast<uint8_t*>(dev_mem);
  h->device = dev;
  h->num_sms = sms;
  for (h->page_shift = 4; (1 << h->page_shift) < cfg->page_size;) ++h->page_shift;
  const bool e8 = cfg->cache_format == KVPOP_CACHE_E4M3;
  h->maps = new (std::nothrow) CUtensorMap[cfg->n_layers];
  bool ok = h->maps != nullptr && prepare_attend(cfg->dtype, cfg->head_dim, e8, cfg->n_q_heads / cfg->n_kv_heads) == 0;
  for (int l = 0; ok && l < cfg->n_layers; ++l)
    ok = make_attend_map(&h->maps[l], h->mem + L.pages_off + l * L.pages_stride, cfg->dtype, cfg->head_dim, e8,
                         cfg->page_size, static_cast<int64_t>(cfg->n_pages) * cfg->n_kv_heads) == 0;
  // The default stream's clearing does not wait for non-blocking streams: what is queued there, and may still write
  // to memory that an allocator has handed on, ends first.
  ok = ok && cudaDeviceSynchronize() == cudaSuccess;
  if (!ok || cudaMemset(h->mem, 0, L.total) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) {
    delete h;
    return cuda_failed();
  }
  *out = h;
  return KVPOP_OK;
}

int kvpop_paged_append(kvpop_paged_handle* h, int32_t layer, const kvpop_rows* k, const kvpop_rows* v,
                       const int32_t* slots, int32_t batch, int32_t n_tokens, void* stream) {
  if (bad_layer(h, layer) || batch < 0 || n_tokens < 0) return KVPOP_ERR_INVALID_ARG;
  if (batch == 0 || n_tokens == 0) return KVPOP_OK;
  if (static_cast<int64_t>(batch) * n_tokens > (1 << 30)) return KVPOP_ERR_BAD_SHAPE;
  const kvpop_paged_config& c = h->cfg;
  const int es = element_size(c.dtype);
  HeadsArgs a{};
  if (!slots || !aligned(slots, 4)) return KVPOP_ERR_INVALID_ARG;
  if (!rows_view(k, batch, n_tokens, c.n_kv_heads, es, false, &a.k) ||
      !rows_view(v, batch, n_tokens, c.n_kv_heads, es, false, &a.v))
    return KVPOP_ERR_INVALID_ARG;
  a.pg = paged_layer(h, layer);
  a.slots = slots;
  a.batch = batch; a.n_tokens = n_tokens; a.Hq = c.n_q_heads; a.Hkv = c.n_kv_heads;
  DeviceScope scope(h->device);
  if (!scope.ok()) return cuda_failed();
  return status_of(launch_heads(a, c.dtype, c.head_dim, HEADS_APPEND, h->num_sms, static_cast<cudaStream_t>(stream)));
}

int kvpop_paged_append_qkv(kvpop_paged_handle* h, int32_t layer, const kvpop_rope* rope, const kvpop_rows* q,
                           const kvpop_rows* k, const kvpop_rows* v, const int32_t* positions,
                           const int32_t* slots, const kvpop_rows* q_out, int32_t batch, int32_t n_tokens,
                           void* stream) {
  if (bad_layer(h, layer) || batch < 0 || n_tokens < 0) return KVPOP_ERR_INVALID_ARG;
  const kvpop_paged_config& c = h->cfg;
  const int es = element_size(c.dtype);
  HeadsArgs a{};
  int status;
  if (!rope_args(rope, c.head_dim, &a.rope, &status)) return status;
  if (batch == 0 || n_tokens == 0) return KVPOP_OK;
  if (static_cast<int64_t>(batch) * n_tokens > (1 << 30)) return KVPOP_ERR_BAD_SHAPE;
  if (!slots || !aligned(slots, 4) || !positions || !aligned(positions, 4)) return KVPOP_ERR_INVALID_ARG;
  if (!rows_view(q, batch, n_tokens, c.n_q_heads, es, false, &a.q) ||
      !rows_view(k, batch, n_tokens, c.n_kv_heads, es, false, &a.k) ||
      !rows_view(v, batch, n_tokens, c.n_kv_heads, es, false, &a.v) ||
      !rows_view(q_out, batch, n_tokens, c.n_q_heads, es, true, &a.qo))
    return KVPOP_ERR_INVALID_ARG;
  a.pg = paged_layer(h, layer);
  a.pos = positions;
  a.slots = slots;
  a.batch = batch; a.n_tokens = n_tokens; a.Hq = c.n_q_heads; a.Hkv = c.n_kv_heads;
  DeviceScope scope(h->device);
  if (!scope.ok()) return cuda_failed();
  return status_of(launch_heads(a, c.dtype, c.head_dim, HEADS_STEP, h->num_sms, static_cast<cudaStream_t>(stream)));
}

int kvpop_paged_gather(kvpop_paged_handle* h, int32_t layer, const int32_t* page_table, int64_t table_stride,
                       int32_t table_width, const int32_t* lens, int32_t batch, int32_t n_tokens,
                       const kvpop_rows* k_out, const kvpop_rows* v_out, void* stream) {
  if (bad_layer(h, layer) || batch < 0 || n_tokens < 0 || table_width < 0) return KVPOP_ERR_INVALID_ARG;
  if (batch > 65535) return KVPOP_ERR_BAD_SHAPE;
  if (batch == 0 || n_tokens == 0) return KVPOP_OK;
  const kvpop_paged_config& c = h->cfg;
  const int es = element_size(c.dtype);
  GatherArgs a{};
  if (!tables_ok(page_table, table_stride, table_width, lens, batch)) return KVPOP_ERR_INVALID_ARG;
  if (!rows_view(k_out, batch, n_tokens, c.n_kv_heads, es, true, &a.k) ||
      !rows_view(v_out, batch, n_tokens, c.n_kv_heads, es, true, &a.v))
    return KVPOP_ERR_INVALID_ARG;
  a.pg = paged_layer(h, layer);
  a.table = page_table; a.lens = lens; a.table_stride = table_stride;
  a.batch = batch; a.width = table_width; a.n_tokens = n_tokens;
  DeviceScope scope(h->device);
  if (!scope.ok()) return cuda_failed();
  return status_of(launch_gather(a, c.dtype, c.head_dim, static_cast<cudaStream_t>(stream)));
}

int kvpop_paged_attend(kvpop_paged_handle* h, int32_t layer, const void* q, const int32_t* page_table,
                       int64_t table_stride, int32_t table_width, const int32_t* lens, int32_t batch,
                       const kvpop_attend_options* options, void* out, float* lse, void* stream) {
  if (bad_layer(h, layer) || batch < 0 || table_width < 0) return KVPOP_ERR_INVALID_ARG;
  const kvpop_paged_config& c = h->cfg;
  if (batch > c.max_batch) return KVPOP_ERR_BAD_SHAPE;
  const kvpop_attend_options o = options ? *options : kvpop_attend_options{0.f, 0.f, 0};
  if (!factor_ok(o.scale) || !factor_ok(o.softcap) || o.window < 0) return KVPOP_ERR_INVALID_ARG;
  if (batch == 0) return KVPOP_OK;
  if (!q || !out || !aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4)) return KVPOP_ERR_INVALID_ARG;
  if (!tables_ok(page_table, table_stride, table_width, lens, batch)) return KVPOP_ERR_INVALID_ARG;
  if (static_cast<int64_t>(table_width) * c.page_size > (1 << 30)) return KVPOP_ERR_BAD_SHAPE;
  AttendArgs a{};
  a.pg = paged_layer(h, layer);
  a.q = q; a.table = page_table; a.lens = lens; a.table_stride = table_stride;
  a.out = out; a.lse = lse;
  a.batch = batch; a.width = table_width; a.Hq = c.n_q_heads; a.G = c.n_q_heads / c.n_kv_heads;
  a.scale = o.scale > 0.f ? o.scale : 1.f / std::sqrt(static_cast<float>(c.head_dim));
  a.softcap = o.softcap;
  a.window = o.window;
  DeviceScope scope(h->device);
  if (!scope.ok()) return cuda_failed();
  return status_of(launch_attend(h->maps[layer], a, h->mem + h->lay.scratch_off, c.dtype, c.head_dim,
                                 h->num_sms, static_cast<cudaStream_t>(stream)));
}

int kvpop_paged_get_layout(const kvpop_paged_handle* h, kvpop_paged_layout_info* o) {
  if (!h || !o) return KVPOP_ERR_INVALID_ARG;
  o->pages_offset = h->lay.pages_off; o->pages_layer_stride = h->lay.pages_stride;
  o->scales_offset = h->lay.scales_off; o->scales_layer_stride = h->lay.scales_stride;
  return KVPOP_OK;
}

int kvpop_paged_get_error(kvpop_paged_handle* h, int32_t* device_bits) {
  if (!h) return KVPOP_ERR_INVALID_ARG;
  DeviceScope scope(h->device);
  if (!scope.ok() || cudaDeviceSynchronize() != cudaSuccess) return cuda_failed();
  int32_t bits = 0;
  if (cudaMemcpy(&bits, h->mem + h->lay.err_off, 4, cudaMemcpyDeviceToHost) != cudaSuccess) return cuda_failed();
  if (device_bits) *device_bits = bits;
  if (bits == 0) return KVPOP_OK;
  return (bits & DEVERR_TIMEOUT) ? KVPOP_ERR_TIMEOUT : KVPOP_ERR_DEVICE;
}

int kvpop_paged_clear_error(kvpop_paged_handle* h, void* stream) {
  if (!h) return KVPOP_ERR_INVALID_ARG;
  DeviceScope scope(h->device);
  if (!scope.ok()) return cuda_failed();
  return cudaMemsetAsync(h->mem + h->lay.err_off, 0, 4, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? KVPOP_OK
             : cuda_failed();
}

int kvpop_paged_destroy(kvpop_paged_handle* h) {
  if (!h) return KVPOP_ERR_INVALID_ARG;
  delete h;
  return KVPOP_OK;
}

}  // extern "C"
