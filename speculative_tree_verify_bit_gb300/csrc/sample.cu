// sample.cu -- sampling from the target's logits with temperature, top-k,
// top-p and min-p from given random numbers (include/stv.h, stv_sample).
//
// Every filter and the draw itself is a cut of one order (logit descending,
// then index ascending) at a given count or a given mass, so no sort of the
// vocabulary is needed.  A cluster of CTAs shares a row, each CTA a stretch of
// it:
//   1. One pass over the stretch finds the maximum (a NaN shows in it).
//   2. How far down the order do the cuts lie?  With top-k, the maxima of some
//      thousand groups of tokens tell: as many tokens at least exceed a value as
//      groups whose maximum does.  Otherwise a sample of some 8,192 tokens,
//      counted by quarter octaves of w, tells how much mass lies below a value.
//   3. A second pass (from L2) adds up the mass of all (unless top-k or min-p
//      alone make that unneeded), and takes the tokens above that value, the
//      head: gathers them when they are few, else counts them and adds their
//      masses in bins; then a third pass gathers the tokens of the few
//      bins that the cuts lie in.
//   4. The first CTA merges and sorts the gathered tokens and makes the cuts
//      exactly.  Where one lies past the head, the bins are filled once more,
//      with every token that has any mass.
// What is chosen by groups and samples is only how much is gathered.
//
// Masses.  w = exp((x - max) / T) as an integer of scale 2^45.  With C =
// T ln 2 / 64, k = rint(x / C) and z = x - k C (C in two floats; the first
// product's remainder is exact), w is 2^(k / 64) from a table of 64 entries
// times e^(z / T), |z / T| <= ln 2 / 128, whose cubic is rounded to 2^-29 of w.
// With the table, the constants and the products that is less than 2^-28 of w,
// and cutting w to a whole number adds up to a unit, at most 2^-44 of the
// largest: from 2^-16 of the largest down, the unit is what counts.  2^19
// tokens of scale 2^45 are all that 64 bits add up; finer units would take sums
// of two words, in the loop with the most instructions.  Integer sums do not depend on their order, so masses, bins and tokens depend
// neither on the cluster's size nor on the batch.
//
// What bounds it.  16 bf16 rows of 248,320 tokens (8 MB, 1.2 us at the copy
// bandwidth) take 21.5 us: a chain of steps of one to four microseconds with a
// barrier after each (first pass 2.8, groups 2, second pass 4.7, merge and sort
// 3.2, cuts and barriers 4; 41 % of the warps' time is spent waiting at
// barriers).  512 fp32 rows (508 MB, 75 us) take 318 us, of which no one limit
// accounts for all: 942 MB come from HBM (139 us; L2 does not hold the rows
// between the passes), the instructions fill 63 % of the issue slots of busy SMs
// (166 us spread over all; the sum of all weights, 24 instructions a token in
// the 216 rows that need it, is a fifth of them), and a quarter of the warps'
// time goes to barriers and loads.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <math.h>
#include <string.h>

#include <algorithm>
#include <utility>

#include "stv_device.cuh"

namespace cg = cooperative_groups;

namespace stv {
namespace {

using u64 = unsigned long long;

constexpr int kCoarse = 256;     // quarter octaves of the sample
constexpr int kMaxVocab = 1 << 19;
constexpr int kShift = 14;       // w < 2^45: 2^19 tokens stay below 2^64
constexpr int kMaxCluster = 8;
constexpr int kNarrowVocab = 16384;
constexpr int kStages = 7;       // one being read, six on their way
constexpr int kBinnedStages = 4; // where the bins' totals take the place of the others

struct SampleParams {
  const void* x;
  int64_t row_stride;
  int n_rows, vocab, rows_per_param;
  int stretch;       // tokens per CTA of a cluster
  int sample_every;  // 1: the sample is everything
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* u;
  int32_t* ids;
  float* logprob;
  int32_t* status;
  uint32_t table[64];  // 2^30 * 2^(j / 64)
};

// A row in the CTAs of a cluster, 512 threads each, two on an SM.
namespace wide {
constexpr int kThreads = 512, kCtasPerSm = 2, kBins = 2048, kBinBits = 11, kList = 2048, kDirect = 1600;
constexpr float kLeastHead = 512.f;
#include "sample_rows.cuh"
}  // namespace wide

// Many short rows, one in each of seven CTAs on an SM.
namespace narrow {
constexpr int kThreads = 128, kCtasPerSm = 7, kBins = 512, kBinBits = 9, kList = 512, kDirect = 400;
constexpr float kLeastHead = 128.f;
#include "sample_rows.cuh"
}  // namespace narrow

template <typename T>
cudaError_t launch_sample(SampleParams& p, cudaStream_t st) {
  int sm = 0;
  if (device_sm_count(&sm) != STV_OK) return cudaErrorUnknown;
  constexpr int VE = 16 / sizeof(T);
  // CTAs per row, of 2,048 tokens at least: as many as make up to four waves of
  // two CTAs per SM.  A row's last steps are one CTA's, and rows differ in
  // length several times over (see the bins), so short stretches pay: 128 fp16
  // rows of 248,320 take 121 us with two, 92 with four, 93 with eight; 512 fp32
  // rows, which L2 does not hold, 454 us with one, 318 with two, 326 with four.
  int c = 1;
  while (c < kMaxCluster && p.vocab / (2 * c) >= 2048 && (int64_t)p.n_rows * 2 * c <= 8 * sm) c *= 2;
  // More short rows than the wide CTAs take at a time: seven narrow ones hold an
  // SM's steps apart from one another (1,984 rows of 1,901 tokens 61 us, 138
  // with wide CTAs; 2,048 of 8,000 76 and 172; 644 of 14,442 58 and 82; but
  // 1,216 of 24,506 165 and 162, 2,048 of 50,000 366 and 302).
  const bool narrow = p.vocab <= kNarrowVocab && p.n_rows > wide::kCtasPerSm * sm;
  if (narrow) c = 1;
  p.stretch = ((p.vocab + c - 1) / c + VE - 1) / VE * VE;
  p.sample_every = std::max(1, p.vocab / 8192);
  const auto kernel = narrow ? narrow::sample_kernel<T> : wide::sample_kernel<T>;
  const size_t smem = narrow ? sizeof(narrow::Smem) : sizeof(wide::Smem);
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.n_rows * c));
    cfg.blockDim = dim3(narrow ? narrow::kThreads : wide::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)c;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, kernel, p);
  }
  if (e != cudaSuccess) (void)cudaGetLastError();
  return e;
}

}  // namespace
}  // namespace stv

extern "C" int stv_sample(const void* logits, int dtype, int64_t row_stride, int n_rows, int vocab,
                          const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                          int rows_per_param, const float* u, int32_t* ids, float* logprob, int32_t* dev_status,
                          stv_stream_t stream) {
  using namespace stv;
  if (dtype != STV_F32 && dtype != STV_F16 && dtype != STV_BF16) return STV_ERR_INVALID_ARG;
  if (n_rows < 0 || rows_per_param < 1 || vocab < 1) return STV_ERR_INVALID_ARG;
  if (vocab > kMaxVocab) return STV_ERR_SHAPE_UNSUPPORTED;
  if (n_rows == 0) return STV_OK;
  if (n_rows > 0x7fffffff / kMaxCluster) return STV_ERR_SHAPE_UNSUPPORTED;
  if (!logits || !u || !ids || (n_rows > 1 && row_stride < vocab)) return STV_ERR_INVALID_ARG;
  if ((uintptr_t)logits % (dtype == STV_F32 ? 4 : 2)) return STV_ERR_INVALID_ARG;
  SampleParams p;
  memset(&p, 0, sizeof(p));
  p.x = logits;
  p.row_stride = row_stride;
  p.n_rows = n_rows;
  p.vocab = vocab;
  p.rows_per_param = rows_per_param;
  p.temperature = temperature;
  p.top_k = top_k;
  p.top_p = top_p;
  p.min_p = min_p;
  p.u = u;
  p.ids = ids;
  p.logprob = logprob;
  p.status = dev_status;
  for (int j = 0; j < 64; ++j) p.table[j] = (uint32_t)llround(ldexp(exp2(j / 64.0), 30));
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = dtype == STV_F32   ? launch_sample<float>(p, st)
                        : dtype == STV_F16 ? launch_sample<__half>(p, st)
                                           : launch_sample<__nv_bfloat16>(p, st);
  return e == cudaSuccess ? STV_OK : STV_ERR_CUDA;
}
