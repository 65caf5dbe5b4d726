// kv_write.cu -- K and V rows into the drafter's 16-bit paged cache
// (include/stv.h, stv_kv_write).
//
// A copy: every element is read and written once, so HBM bounds it for
// prompts and the launch for a round's rows.  An item is 16 bytes of one row
// (one element where a view's strides or address allow no wide loads); the
// CTAs take kPer x kThreads adjacent items each, in order, so that what is in
// flight lies close together, and a thread's loads are all issued before its
// first store.
#include <string.h>

#include "stv_device.cuh"

namespace stv {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 4;  // (32,768 rows of 4 x 256 fp16: 43.6 us; 45.8 with 2 or 8)

struct WriteParams {
  const uint8_t* in[2];  // k, v
  int64_t row[2], head[2];  // strides in bytes
  const int32_t* slots;
  uint8_t* pool;
  int64_t page_bytes;
  int n_pages;
  int hkv;
  int per_head;  // items of one head's row
  int per_row;   // of a row of k and v
  int64_t items;
  int32_t* status;
};

template <typename V>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(const __grid_constant__ WriteParams p) {
  grid_dep_wait();
  grid_dep_launch();
  // (one 64-bit division for the CTA, short ones from there)
  const int64_t base = (int64_t)blockIdx.x * (kThreads * kPer), row0 = base / p.per_row;
  const uint32_t from = (uint32_t)(base - row0 * p.per_row) + threadIdx.x;
  V v[kPer];
  V* dst[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    dst[k] = nullptr;
    if (base + threadIdx.x + k * kThreads >= p.items) continue;
    const uint32_t i = from + k * kThreads, rows = i / (uint32_t)p.per_row;
    const int64_t row = row0 + rows;
    const int in_row = (int)(i - rows * (uint32_t)p.per_row);
    const int h2 = in_row / p.per_head, e = in_row - h2 * p.per_head;
    const int which = h2 >= p.hkv, h = h2 - which * p.hkv;
    const int slot = __ldg(p.slots + row);
    if (slot < 0 || slot / kPageTok >= p.n_pages) {
      if (slot != -1 && in_row == 0) report(p.status, STV_DEV_BAD_PAGE);
      continue;
    }
    const int64_t head_bytes = (int64_t)p.per_head * sizeof(V);
    dst[k] = reinterpret_cast<V*>(p.pool + slot / kPageTok * p.page_bytes +
                                  (((int64_t)h * 2 + which) * kPageTok + slot % kPageTok) * head_bytes) + e;
    v[k] = __ldg(reinterpret_cast<const V*>(p.in[which] + row * p.row[which] + h * p.head[which]) + e);
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k)
    if (dst[k]) *dst[k] = v[k];
}

}  // namespace
}  // namespace stv

extern "C" int stv_kv_write(const stv_shape* shape, const stv_layer_cache* layer, const stv_rows* k, const stv_rows* v,
                            const int32_t* slots, int n_rows, int32_t* dev_status, stv_stream_t stream) {
  using namespace stv;
  RowShape sh;
  int rc = check_row_shape(shape, &sh);
  if (rc || (rc = check_row_layer(layer, sh))) return rc;
  if (n_rows < 0 || !k || !v) return STV_ERR_INVALID_ARG;
  if (n_rows == 0) return STV_OK;
  if (!slots) return STV_ERR_INVALID_ARG;
  WriteParams p;
  memset(&p, 0, sizeof(p));
  bool wide = true;
  const stv_rows* in[2] = {k, v};
  for (int t = 0; t < 2; ++t) {
    const stv_rows* x = in[t];
    if (!rows_view_ok(x, sh.hd, n_rows) || x->heads != sh.hkv || (uintptr_t)x->data % 2) return STV_ERR_INVALID_ARG;
    if (rows_meet_pool(x, sh.hd, n_rows, layer)) return STV_ERR_INVALID_ARG;
    wide = wide && (uintptr_t)x->data % 16 == 0 && (x->heads == 1 || x->head_stride % 8 == 0) &&
           (n_rows == 1 || x->row_stride % 8 == 0);
    p.in[t] = static_cast<const uint8_t*>(x->data);
    p.row[t] = x->row_stride * 2;
    p.head[t] = x->head_stride * 2;
  }
  p.slots = slots;
  p.pool = layer->pool;
  p.page_bytes = layer->page_bytes;
  p.n_pages = layer->n_pages;
  p.hkv = sh.hkv;
  p.per_head = sh.hd / (wide ? 8 : 1);
  p.per_row = 2 * sh.hkv * p.per_head;
  p.items = (int64_t)n_rows * p.per_row;
  p.status = dev_status;
  const int64_t ctas = (p.items + kThreads * kPer - 1) / (kThreads * kPer);
  if (ctas > 0x7fffffff) return STV_ERR_SHAPE_UNSUPPORTED;
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = wide ? launch_pdl(kv_write_kernel<uint4>, (int)ctas, kThreads, 0, st, p)
                             : launch_pdl(kv_write_kernel<uint16_t>, (int)ctas, kThreads, 0, st, p);
  return e == cudaSuccess ? STV_OK : STV_ERR_CUDA;
}
