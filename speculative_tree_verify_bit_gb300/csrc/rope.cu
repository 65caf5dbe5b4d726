// rope.cu -- rotary positions with several axes on the q and k rows that
// precede the append (include/stv.h, stv_rope).
//
// Angles.  A frequency is kept in turns as a 64-bit fixed-point fraction F =
// f / (2 pi) * 2^64, so pos * F mod 2^64 is the phase without any range
// reduction and without loss at far positions: its top 32 bits, a signed
// fraction of half a turn, go to sincospif.  An fp32 product pos * f would be
// off by up to 2^-7 rad at a position of 262,144.
//
// One thread turns the same VE channel pairs (one 16-byte load from each half
// of the rotary channels) of kHeads heads of one row, so the VE sines and
// cosines are computed once for kHeads heads and stay in registers; the
// channels past rotary_dim are copied by threads of the same shape.  The call
// reads and writes each element once: bound by HBM for prompts, by the launch
// for a round's tree rows.
#include <cuda_bf16.h>
#include <math.h>
#include <string.h>

#include "stv_device.cuh"

namespace stv {
namespace {

constexpr int kMaxPairs = 256;
constexpr int kThreads = 256;

struct RopeParams {
  uint64_t turn[kMaxPairs];  // frequency of each pair, 2^64 per turn
  uint8_t axis[kMaxPairs];
  const void* in[2];  // q, k
  void* out[2];
  int64_t in_row[2], in_head[2], out_row[2], out_head[2];
  int heads[2];
  const int32_t* pos;
  int n_rows, n_axes, head_groups;
  int half, head_dim;
  int rot_items, items;  // per head: items that turn pairs, and those plus the ones that copy
  int negate;
};

template <typename T> __device__ __forceinline__ float to_f(T x);
template <> __device__ __forceinline__ float to_f(float x) { return x; }
template <> __device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f(float x) { return x; }
template <> __device__ __forceinline__ __half from_f(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float x) { return __float2bfloat16_rn(x); }

// VE elements: 16 bytes, or one element where the views allow no wide loads.
template <typename T, int VE>
struct alignas(sizeof(T) * VE) Vec {
  T e[VE];
};

template <typename T, int VE, int kHeads>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  using V = Vec<T, VE>;
  __shared__ uint64_t turn_s[kMaxPairs];
  __shared__ uint8_t axis_s[kMaxPairs];
  for (int i = threadIdx.x; i < p.half; i += kThreads) {
    turn_s[i] = p.turn[i];
    axis_s[i] = p.axis[i];
  }
  __syncthreads();
  grid_dep_wait();
  grid_dep_launch();
  const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t unit = id / p.items;
  const int j = (int)(id - unit * p.items);
  const int row = (int)(unit / p.head_groups);
  if (row >= p.n_rows) return;
  const int h0 = (int)(unit - (int64_t)row * p.head_groups) * kHeads;
  const int n_heads = p.heads[0] + p.heads[1];

  const bool turns = j < p.rot_items;
  // channels of the item: (c0, c1) = a pair of the two halves, or two pieces to copy
  const int c0 = turns ? j * VE : 2 * p.half + (j - p.rot_items) * 2 * VE;
  const int c1 = turns ? c0 + p.half : c0 + VE;
  const bool has1 = c1 < p.head_dim;

  V a[kHeads], b[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int h = h0 + i;
    if (h < n_heads) {
      const int t = h >= p.heads[0];
      const T* src = static_cast<const T*>(p.in[t]) + row * p.in_row[t] + (h - (t ? p.heads[0] : 0)) * p.in_head[t];
      a[i] = *reinterpret_cast<const V*>(src + c0);
      if (has1) b[i] = *reinterpret_cast<const V*>(src + c1);
    }
  }
  if (turns) {
    float c[VE], s[VE];
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      const uint64_t f = turn_s[c0 + e];
      const int32_t ps = __ldg(p.pos + (int64_t)axis_s[c0 + e] * p.n_rows + row);
      const uint64_t ph = (uint64_t)((int64_t)ps) * f;  // modulo a turn
      const float x = (float)(int32_t)(ph >> 32) * 4.656612873077393e-10f;  // half turns, [-1, 1]
      sincospif(x, &s[e], &c[e]);
      if (p.negate) s[e] = -s[e];
    }
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const float x = to_f(a[i].e[e]), y = to_f(b[i].e[e]);
        a[i].e[e] = from_f<T>(x * c[e] - y * s[e]);
        b[i].e[e] = from_f<T>(y * c[e] + x * s[e]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int h = h0 + i;
    if (h < n_heads) {
      const int t = h >= p.heads[0];
      T* dst = static_cast<T*>(p.out[t]) + row * p.out_row[t] + (h - (t ? p.heads[0] : 0)) * p.out_head[t];
      *reinterpret_cast<V*>(dst + c0) = a[i];
      if (has1) *reinterpret_cast<V*>(dst + c1) = b[i];
    }
  }
}

template <typename T, int VE>
cudaError_t launch_rope(RopeParams& p, bool copy_rest, cudaStream_t s) {
  const int rest = copy_rest ? p.head_dim - 2 * p.half : 0;
  p.rot_items = p.half / VE;
  p.items = p.rot_items + (rest / VE + 1) / 2;
  const int n_heads = p.heads[0] + p.heads[1];
  p.head_groups = n_heads;
  const int64_t ids = (int64_t)p.n_rows * p.head_groups * p.items;
  const int64_t grid = (ids + kThreads - 1) / kThreads;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_pdl(rope_kernel<T, VE, 1>, (int)grid, kThreads, 0, s, p);
}

// Every pair's frequency in turns per position, 2^64 a turn.  The last ones
// this thread made are kept: a model's layers ask for the same ones.
const uint64_t* turns_of(double theta, int rotary_dim) {
  static thread_local struct {
    double theta;
    int rotary_dim = 0;
    uint64_t turn[kMaxPairs];
  } memo;
  if (memo.rotary_dim != rotary_dim || memo.theta != theta) {
    for (int i = 0; i < rotary_dim / 2; ++i)
      memo.turn[i] = (uint64_t)ldexp(pow(theta, -2.0 * i / rotary_dim) * 0.15915494309189533577, 64);
    memo.theta = theta;
    memo.rotary_dim = rotary_dim;
  }
  return memo.turn;
}

bool rows_ok(const stv_rows* v, int head_dim, int n_rows) {
  if (!v->data || v->heads < 1 || v->heads > 1 << 16 || v->head_stride < head_dim) return false;
  // an extent of at most 2^50 bytes, so that no offset below overflows
  if (v->head_stride > ((int64_t)1 << 48) / v->heads || (n_rows > 1 && v->row_stride > ((int64_t)1 << 48) / n_rows))
    return false;
  return n_rows <= 1 || v->row_stride >= (v->heads - 1) * v->head_stride + head_dim;
}

// Whether elements of two views can meet: their extents do, and they are not
// different columns of rows with one stride.
bool may_meet(const stv_rows* a, const stv_rows* b, int head_dim, int n_rows, int64_t es) {
  const int64_t wa = ((a->heads - 1) * a->head_stride + head_dim) * es;
  const int64_t wb = ((b->heads - 1) * b->head_stride + head_dim) * es;
  const uintptr_t a0 = (uintptr_t)a->data, b0 = (uintptr_t)b->data;
  const uintptr_t a1 = a0 + (n_rows - 1) * a->row_stride * es + wa;
  const uintptr_t b1 = b0 + (n_rows - 1) * b->row_stride * es + wb;
  if (a1 <= b0 || b1 <= a0) return false;
  if (n_rows == 1 || a->row_stride != b->row_stride) return true;
  const int64_t st = a->row_stride * es;
  int64_t d = (int64_t)(b0 - a0) % st;  // column of b's row 0 against a's
  if (d < 0) d += st;
  return !(d >= wa && d + wb <= st);
}

bool same_view(const stv_rows* a, const stv_rows* b, int n_rows) {
  return a->data == b->data && (a->head_stride == b->head_stride || a->heads == 1) &&
         (a->row_stride == b->row_stride || n_rows == 1);
}

}  // namespace
}  // namespace stv

extern "C" int stv_rope(const stv_rope_spec* spec, int dtype, int head_dim, const int32_t* pos, int n_rows,
                        const stv_rows* q, const stv_rows* q_out, const stv_rows* k, const stv_rows* k_out,
                        int inverse, stv_stream_t stream) {
  using namespace stv;
  if (!spec || n_rows < 0 || (!q && !k) || !q != !q_out || !k != !k_out) return STV_ERR_INVALID_ARG;
  if (dtype != STV_F32 && dtype != STV_F16 && dtype != STV_BF16) return STV_ERR_INVALID_ARG;
  if (head_dim < 2 || head_dim > 2 * kMaxPairs || head_dim % 2) return STV_ERR_SHAPE_UNSUPPORTED;
  if (spec->rotary_dim < 2 || spec->rotary_dim > head_dim || spec->rotary_dim % 2) return STV_ERR_SHAPE_UNSUPPORTED;
  if (spec->n_axes < 1 || spec->n_axes > 4) return STV_ERR_SHAPE_UNSUPPORTED;
  if (!(spec->theta >= 1.0) || isinf(spec->theta)) return STV_ERR_INVALID_ARG;
  if (spec->interleaved != 0 && spec->interleaved != 1) return STV_ERR_INVALID_ARG;
  const int half = spec->rotary_dim / 2, na = spec->n_axes;
  int64_t sum = 0;
  for (int a = 0; a < na; ++a) {
    const int32_t n = spec->sections[a];
    if (n < 0) return STV_ERR_INVALID_ARG;
    sum += n;
    // interleaved: the last pair dealt to axis a exists
    if (spec->interleaved && a > 0 && n > 0 && a + (int64_t)na * (n - 1) >= half) return STV_ERR_INVALID_ARG;
  }
  if (sum != half) return STV_ERR_INVALID_ARG;
  if (n_rows == 0) return STV_OK;
  if (!pos) return STV_ERR_INVALID_ARG;

  RopeParams p;
  memset(&p, 0, sizeof(p));
  const stv_rows* in[2] = {q, k};
  const stv_rows* out[2] = {q_out, k_out};
  const int64_t es = dtype == STV_F32 ? 4 : 2;
  const int ve = (int)(16 / es);
  bool wide = half % ve == 0 && (head_dim - spec->rotary_dim) % ve == 0;
  bool in_place = true;
  for (int t = 0; t < 2; ++t) {
    if (!in[t]) continue;
    if (!rows_ok(in[t], head_dim, n_rows) || !rows_ok(out[t], head_dim, n_rows) || in[t]->heads != out[t]->heads)
      return STV_ERR_INVALID_ARG;
    in_place = in_place && same_view(in[t], out[t], n_rows);
    p.in[t] = in[t]->data;
    p.out[t] = out[t]->data;
    p.heads[t] = in[t]->heads;
    p.in_row[t] = in[t]->row_stride;
    p.in_head[t] = in[t]->head_stride;
    p.out_row[t] = out[t]->row_stride;
    p.out_head[t] = out[t]->head_stride;
    for (const stv_rows* v : {in[t], out[t]}) {
      if ((uintptr_t)v->data % es) return STV_ERR_INVALID_ARG;
      wide = wide && (uintptr_t)v->data % 16 == 0 && (v->heads == 1 || v->head_stride % ve == 0) &&
             (n_rows == 1 || v->row_stride % ve == 0);
    }
  }
  for (int t = 0; t < 2; ++t)
    for (int u = 0; u < 2; ++u) {
      if (out[t] && in[u] && !(t == u && same_view(in[u], out[t], n_rows)) &&
          may_meet(out[t], in[u], head_dim, n_rows, es))
        return STV_ERR_INVALID_ARG;
      if (t < u && out[t] && out[u] && may_meet(out[t], out[u], head_dim, n_rows, es)) return STV_ERR_INVALID_ARG;
    }

  memcpy(p.turn, turns_of(spec->theta, spec->rotary_dim), (size_t)half * sizeof(uint64_t));
  for (int i = 0; i < half; ++i) {
    int axis = 0;
    if (spec->interleaved) {
      axis = i % na;
      if (axis && i >= na * spec->sections[axis]) axis = 0;
    } else {
      for (int left = i; axis < na - 1 && left >= spec->sections[axis]; ++axis) left -= spec->sections[axis];
    }
    p.axis[i] = (uint8_t)axis;
  }
  p.pos = pos;
  p.n_rows = n_rows;
  p.n_axes = na;
  p.half = half;
  p.head_dim = head_dim;
  p.negate = inverse != 0;
  cudaStream_t st = (cudaStream_t)stream;
  const bool rest = !in_place;
  cudaError_t e;
  if (dtype == STV_F32)
    e = wide ? launch_rope<float, 4>(p, rest, st) : launch_rope<float, 1>(p, rest, st);
  else if (dtype == STV_F16)
    e = wide ? launch_rope<__half, 8>(p, rest, st) : launch_rope<__half, 1>(p, rest, st);
  else
    e = wide ? launch_rope<__nv_bfloat16, 8>(p, rest, st) : launch_rope<__nv_bfloat16, 1>(p, rest, st);
  return e == cudaSuccess ? STV_OK : STV_ERR_CUDA;
}
