// rope.cu -- rotary positions with several axes on the q and k rows that
// precede the append (include/stv.h, stv_rope).
//
// Angles.  A frequency is kept in turns as a 64-bit fixed-point fraction F =
// f / (2 pi) * 2^64, so pos * F mod 2^64 is the phase without any range
// reduction: its top 32 bits, a signed fraction of half a turn, go to sincospif.
// F is formed in pairs of doubles and is right to half its last place, 2^-34 of
// a turn at a position of 2^31 (with a frequency in one double, 2^-24); the
// conversion to fp32 costs 2^-26 of a turn, the cut to 32 bits 2^-32.  An fp32
// product pos * f would be off by up to 2^-7 rad at a position of 262,144.
//
// A CTA takes a few rows and some of their heads.  It computes each row's sines
// and cosines once, into shared memory (a thread that turned its own channels
// would compute them again for every head), while the loads of its first items
// are on their way.  An item is two 16-byte loads and stores of one head: a
// piece of the first half of the rotary channels and its partner in the
// second, or two pieces past them to copy, half of what lies there apart, so
// that neighbouring threads read neighbouring pieces.
//
// The call reads and writes each element once: bound by HBM for prompts, by
// the launch for a round's tree rows.
#include <cuda_bf16.h>
#include <math.h>
#include <string.h>

#include <algorithm>

#include "stv_device.cuh"

namespace stv {
namespace {

constexpr int kMaxPairs = 256;
constexpr int kThreads = 256;  // at least kMaxPairs
constexpr int kCtasPerSm = 5;  // by registers
constexpr int kShare = 14;     // items of a thread, for a prompt
constexpr int kMaxRowsPer = 8;
constexpr int kMaxHeadsPer = 64;

struct RopeParams {
  uint64_t turn[kMaxPairs];  // frequency of each pair, 2^64 per turn
  uint8_t axis[kMaxPairs];
  const void* in[2];  // q, k
  void* out[2];
  int64_t in_row[2], in_head[2], out_row[2], out_head[2];
  int heads[2];
  const int32_t* pos;
  int n_rows;
  int half, head_dim;
  int rot_items, items;  // per head: items that turn pairs, and those plus the ones that copy (<= kThreads)
  int rows_per, heads_per, head_blocks;  // a CTA's rows and heads; CTAs per block of rows
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

template <typename T, int VE>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) rope_kernel(const __grid_constant__ RopeParams p) {
  using V = Vec<T, VE>;
  extern __shared__ __align__(16) float table[];  // [rows][half] cosines, then as many sines
  grid_dep_wait();
  grid_dep_launch();
  const int hb = blockIdx.x % p.head_blocks;
  const int row0 = (int)(blockIdx.x / p.head_blocks) * p.rows_per;
  const int n_rows = min(p.rows_per, p.n_rows - row0);
  const int h0 = hb * p.heads_per, n_heads = min(p.heads_per, p.heads[0] + p.heads[1] - h0);
  float* sines = table + p.rows_per * p.half;

  // A thread keeps to one item of a head, its two pieces c0 and c1 (c1 past the
  // head: one piece only), and steps over the (row, head) pairs.
  const int at_once = kThreads / p.items;  // pairs
  const int u0 = (int)threadIdx.x / p.items, j = (int)threadIdx.x - u0 * p.items;
  const bool turns = j < p.rot_items;
  const int c0 = turns ? j * VE : 2 * p.half + (j - p.rot_items) * VE;
  const int c1 = c0 + (turns ? p.half : (p.items - p.rot_items) * VE);
  const bool two = c1 < p.head_dim;
  int row = u0 / n_heads, h = u0 - row * n_heads;
  const int row_step = at_once / n_heads, h_step = at_once - row_step * n_heads;
  if (u0 >= at_once) row = n_rows;

  auto load = [&](int r, int hh, V& a, V& b) {
    if (r < n_rows) {
      hh += h0;
      const int t = hh >= p.heads[0];
      const T* src = static_cast<const T*>(p.in[t]) + (row0 + r) * p.in_row[t] +
                     (hh - (t ? p.heads[0] : 0)) * p.in_head[t];
      a = *reinterpret_cast<const V*>(src + c0);
      if (two) b = *reinterpret_cast<const V*>(src + c1);
    }
  };
  V x, y;
  load(row, h, x, y);
  {
    // the table: a thread keeps to one pair of channels, whose parameters it reads once
    const int rows_at_once = kThreads / p.half;
    const int r0 = (int)threadIdx.x / p.half, pair = (int)threadIdx.x - r0 * p.half;
    if (r0 < rows_at_once) {
      const uint64_t turn = p.turn[pair];
      const int32_t* pos = p.pos + (int64_t)p.axis[pair] * p.n_rows + row0;
      for (int r = r0; r < n_rows; r += rows_at_once) {
        const uint64_t ph = (uint64_t)((int64_t)__ldg(pos + r)) * turn;  // modulo a turn
        const float x = (float)(int32_t)(ph >> 32) * 4.656612873077393e-10f;  // half turns, [-1, 1]
        float sn, cs;
        sincospif(x, &sn, &cs);
        table[r * p.half + pair] = cs;
        sines[r * p.half + pair] = p.negate ? -sn : sn;
      }
    }
    __syncthreads();
  }
#pragma unroll 1
  while (row < n_rows) {
    const int r = row, hh = h0 + h;
    row += row_step;
    h += h_step;
    if (h >= n_heads) {
      h -= n_heads;
      ++row;
    }
    V x1, y1;
    load(row, h, x1, y1);  // before this item's own loads are waited for
    if (turns) {
      const Vec<float, VE>& c = *reinterpret_cast<const Vec<float, VE>*>(table + r * p.half + c0);
      const Vec<float, VE>& s = *reinterpret_cast<const Vec<float, VE>*>(sines + r * p.half + c0);
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const float u = to_f(x.e[i]), v = to_f(y.e[i]);
        x.e[i] = from_f<T>(u * c.e[i] - v * s.e[i]);
        y.e[i] = from_f<T>(v * c.e[i] + u * s.e[i]);
      }
    }
    const int t = hh >= p.heads[0];
    T* dst = static_cast<T*>(p.out[t]) + (row0 + r) * p.out_row[t] + (hh - (t ? p.heads[0] : 0)) * p.out_head[t];
    *reinterpret_cast<V*>(dst + c0) = x;
    if (two) *reinterpret_cast<V*>(dst + c1) = y;
    x = x1;
    y = y1;
  }
}

template <typename T, int VE>
cudaError_t launch_rope(RopeParams& p, bool copy_rest, cudaStream_t s) {
  const int rest = copy_rest ? p.head_dim - 2 * p.half : 0;
  p.rot_items = p.half / VE;
  p.items = p.rot_items + (rest / VE + 1) / 2;
  int sm = 0;
  if (device_sm_count(&sm) != STV_OK) return cudaErrorUnknown;
  const int n_heads = p.heads[0] + p.heads[1];
  const int64_t all = (int64_t)p.n_rows * n_heads * p.items;
  // A CTA's share: up to kShare items per thread (32,768 rows of 28 heads: 148
  // us at 14, 152 at 8, 168 at 5), but three waves of CTAs at least (4,097 fp32
  // rows: 39 us in five waves, 47 in one and a third), and one item per thread
  // where that leaves SMs idle.
  const int64_t share = std::max<int64_t>(kThreads, std::min<int64_t>(all / (16 * sm), kShare * kThreads));
  const int64_t row_items = (int64_t)n_heads * p.items;
  p.rows_per = (int)std::max<int64_t>(1, std::min<int64_t>({share / row_items, kMaxRowsPer, p.n_rows}));
  p.heads_per = (int)std::max<int64_t>(1, std::min<int64_t>({share / p.items, n_heads, kMaxHeadsPer}));
  if (p.rows_per > 1) p.heads_per = std::min(n_heads, kMaxHeadsPer);
  p.head_blocks = (n_heads + p.heads_per - 1) / p.heads_per;
  p.heads_per = (n_heads + p.head_blocks - 1) / p.head_blocks;
  const int64_t grid = (int64_t)((p.n_rows + p.rows_per - 1) / p.rows_per) * p.head_blocks;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  const size_t smem = (size_t)p.rows_per * p.half * 2 * sizeof(float);
  return launch_pdl(rope_kernel<T, VE>, (int)grid, kThreads, smem, s, p);
}

// A sum of two doubles, some 104 bits (Dekker's arithmetic; the product's
// remainder by fma).
struct Twofold {
  double hi, lo;
};
Twofold mul(Twofold a, Twofold b) {
  const double p = a.hi * b.hi;
  const double e = fma(a.hi, b.hi, -p) + (a.hi * b.lo + a.lo * b.hi);
  const double s = p + e;
  return {s, e - (s - p)};
}

// theta^(-1 / n): the double nearby, and one step of Newton's method for
// r^n theta = 1, whose relative residual is formed in two doubles.
Twofold root_of_inverse(double theta, int n) {
  const double r = pow(theta, -1.0 / n);
  Twofold y = {theta, 0.0}, s = {r, 0.0};
  for (int m = n; m; m >>= 1) {
    if (m & 1) y = mul(y, s);
    s = mul(s, s);
  }
  return {r, -r * (((y.hi - 1.0) + y.lo) / n)};
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
    const Twofold step = root_of_inverse(theta, rotary_dim / 2);
    Twofold f = {0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57};  // 1 / (2 pi)
    for (int i = 0; i < rotary_dim / 2; ++i, f = mul(f, step)) {
      const double hi = ldexp(f.hi, 64), whole = floor(hi);
      memo.turn[i] = (uint64_t)whole + (uint64_t)llrint((hi - whole) + ldexp(f.lo, 64));
    }
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
          views_may_meet(out[t], in[u], head_dim, n_rows, es))
        return STV_ERR_INVALID_ARG;
      if (t < u && out[t] && out[u] && views_may_meet(out[t], out[u], head_dim, n_rows, es)) return STV_ERR_INVALID_ARG;
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
