// kd_gradnorm.cu -- the global norm of a list of gradients and their clipping:
//   norm = sqrt(sum x^2),  c = min(1, max_norm / (norm + 1e-6)),  out = c x.
//
// Memory-bound: every gradient is read for the norm and, unless the L2 still
// holds it, once more for the scaling, and written once.  A list is cut into
// units of 32 KB that a resident grid takes in turn, so that many small tensors
// and one large one both spread over the device in one launch; the list itself
// travels in the kernel's parameters (a graph captures it by value).
#include <math.h>
#include <stdlib.h>

#include <algorithm>

#include "kd_common.cuh"
#include "kd_internal.h"

namespace kd {

constexpr int GRAD_THREADS = 256;
constexpr int GRAD_BLOCKS_PER_SM = 3;
constexpr int GRAD_VECS = 8;                                        // 16-byte vectors per thread
constexpr int64_t GRAD_UNIT = 16 * GRAD_VECS * GRAD_THREADS;        // bytes

struct GradEntry {
  const unsigned char* src;
  unsigned char* dst;
  int64_t bytes;
  uint32_t first;                   // first unit of this tensor
  int32_t dtype;
};
template <int N>
struct GradTable {
  uint32_t n, units;
  GradEntry e[N];
};
// A launch takes the smaller table where the list fits it (4 KB of parameters;
// copying the larger one to the device costs more than a short kernel).
constexpr int GRAD_FEW = 100, GRAD_MANY = GRAD_MIN_TENSORS;
static_assert(sizeof(GradTable<GRAD_MANY>) + 128 <= 32764, "kernel parameter limit");

// One unit: a window of GRAD_UNIT bytes that starts on a 16-byte boundary, of
// which the bytes [lo, hi) belong to the tensor.  Windows follow the source's
// alignment, so that a tensor that begins inside a 16-byte line (a view into a
// flat buffer) is still read in whole lines, but for its first and last.
struct GradUnit {
  const unsigned char* src;         // window
  unsigned char* dst;               // the same place of the output
  int lo, hi, dtype;
};

template <int N>
__device__ __forceinline__ GradUnit grad_unit(const GradTable<N>& t, uint32_t u) {
  uint32_t i = 0, hi = t.n - 1;
  while (i < hi) {
    const uint32_t mid = (i + hi + 1) / 2;
    if (t.e[mid].first <= u) i = mid; else hi = mid - 1;
  }
  const GradEntry& e = t.e[i];
  const int64_t pad = static_cast<int64_t>(reinterpret_cast<uintptr_t>(e.src) & 15);
  const int64_t at = static_cast<int64_t>(u - e.first) * GRAD_UNIT - pad;   // of the window
  GradUnit g;
  g.src = e.src + at;
  g.dst = e.dst + at;
  g.lo = at < 0 ? static_cast<int>(-at) : 0;
  g.hi = static_cast<int>(min(e.bytes - at, static_cast<int64_t>(GRAD_UNIT)));
  g.dtype = e.dtype;
  return g;
}

// This thread's vectors of a unit, 0 where the window leaves the tensor.
__device__ __forceinline__ void grad_load(const GradUnit& g, uint4 (&r)[GRAD_VECS]) {
  if (g.lo == 0 && g.hi == GRAD_UNIT) {
#pragma unroll
    for (int i = 0; i < GRAD_VECS; ++i)
      r[i] = *reinterpret_cast<const uint4*>(g.src + 16 * (threadIdx.x + i * GRAD_THREADS));
    return;
  }
#pragma unroll
  for (int i = 0; i < GRAD_VECS; ++i) {
    const int o = 16 * (threadIdx.x + i * GRAD_THREADS);
    r[i] = make_uint4(0u, 0u, 0u, 0u);
    if (o >= g.lo && o + 16 <= g.hi) {
      r[i] = *reinterpret_cast<const uint4*>(g.src + o);
    } else if (o + 16 > g.lo && o < g.hi) {
      uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int k = 0; k < 8; ++k)            // two bytes at a time: lo and hi are even
        if (o + 2 * k >= g.lo && o + 2 * k < g.hi)
          w[k / 2] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(g.src + o + 2 * k))
                      << (16 * (k & 1));
      r[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Sum of squares.  The 4 (bf16: 8) squares of a vector are added in fp32 and the
// vectors in fp64: a conversion for each value kept the sums of 2.2 GB at 430 us,
// one for each vector leaves them to the memory (314 us, 7.0 TB/s).  All terms are
// positive, so the fp32 part is off by at most 8 roundings, 2^-21 of the sum.  A
// vector whose sum comes near the ends of fp32's range, where squares over- or
// underflow, is added in fp64 throughout.
__device__ __forceinline__ double grad_square(const GradUnit& g, const uint4 (&r)[GRAD_VECS]) {
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < GRAD_VECS; ++i) {
    const uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
    const bool bf16 = g.dtype == KD_DTYPE_BF16;
    float f = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float x = bf16 ? bf16_hi(w[k]) : __uint_as_float(w[k]);
      f = fmaf(x, x, f);
      if (bf16) f = fmaf(bf16_lo(w[k]), bf16_lo(w[k]), f);
    }
    if (f >= 1e-30f && f <= 1e37f) {
      sum += f;
    } else {
      for (int k = 0; k < 4; ++k) {
        const double x = bf16 ? bf16_hi(w[k]) : __uint_as_float(w[k]);
        const double y = bf16 ? bf16_lo(w[k]) : 0.f;
        sum = fma(x, x, fma(y, y, sum));
      }
    }
  }
  return sum;
}

template <int N>
__global__ void __launch_bounds__(GRAD_THREADS, GRAD_BLOCKS_PER_SM)
grad_sumsq_kernel(const __grid_constant__ GradTable<N> t, double* __restrict__ partials,
                  uint32_t* status) {
  __shared__ double sm[GRAD_THREADS / 32];
  griddep_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0) clear_status(status);      // nothing here can fail later
  double v[1] = {0.0};
  uint4 r[GRAD_VECS];
  for (uint32_t u = blockIdx.x; u < t.units; u += gridDim.x) {
    const GradUnit g = grad_unit(t, u);
    grad_load(g, r);
    v[0] += grad_square(g, r);
  }
  block_sum(v, sm);
  if (threadIdx.x == 0) partials[blockIdx.x] = v[0];
}

// Sum of the partials, in one order whatever the grid; thread 0's result.
__device__ __forceinline__ double grad_total(const double* p, int n, double* sm) {
  double v[1] = {0.0};
  for (int i = threadIdx.x; i < n; i += GRAD_THREADS) v[0] += __ldcg(p + i);
  block_sum(v, sm);
  return v[0];
}

__global__ void __launch_bounds__(GRAD_THREADS)
grad_total_kernel(const double* __restrict__ partials, int n, double* __restrict__ sumsq) {
  __shared__ double sm[GRAD_THREADS / 32];
  griddep_wait();
  const double s = grad_total(partials, n, sm);
  if (threadIdx.x == 0) *sumsq = s;
}

__device__ __forceinline__ uint32_t scale_bf16x2(uint32_t w, float c) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(bf16_lo(w) * c, bf16_hi(w) * c);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// Units in the reverse order of the sums: what the L2 holds is then read first.
// 2.2 GB into other tensors: 730 us, 6.0 TB/s.
template <int N>
__global__ void __launch_bounds__(GRAD_THREADS, GRAD_BLOCKS_PER_SM)
grad_scale_kernel(const __grid_constant__ GradTable<N> t, const double* __restrict__ partials,
                  int n_partials, double max_norm, float* __restrict__ norm, uint32_t* status) {
  __shared__ double sm[GRAD_THREADS / 32];
  __shared__ float factor;
  uint4 r[GRAD_VECS];
  GradUnit g;
  // the first unit's loads need not wait for the norm: the sums only read it
  const bool any = blockIdx.x < t.units;
  if (any) {
    g = grad_unit(t, t.units - 1 - blockIdx.x);
    grad_load(g, r);
  }
  griddep_wait();
  const double total = grad_total(partials, n_partials, sm);
  if (threadIdx.x == 0) {
    const double x = sqrt(total);
    const double c = isinf(max_norm) ? 1.0 : max_norm / (x + 1e-6);
    factor = c >= 1.0 ? 1.f : static_cast<float>(c);          // NaN stays NaN
    if (norm && blockIdx.x == 0) {
      *norm = static_cast<float>(x);
      clear_status(status);
    }
  }
  __syncthreads();
  const float c = factor;
  for (uint32_t u = blockIdx.x; u < t.units; u += gridDim.x) {
    if (u != blockIdx.x) {
      g = grad_unit(t, t.units - 1 - u);
      if (c == 1.f && g.src == g.dst) continue;               // in place, and nothing to scale
      grad_load(g, r);
    } else if (c == 1.f && g.src == g.dst) {
      continue;
    }
    const bool whole = ((reinterpret_cast<uintptr_t>(g.dst) & 15) == 0);
#pragma unroll
    for (int i = 0; i < GRAD_VECS; ++i) {
      const int o = 16 * (threadIdx.x + i * GRAD_THREADS);
      uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = g.dtype == KD_DTYPE_BF16 ? scale_bf16x2(w[k], c)
                                        : __float_as_uint(__uint_as_float(w[k]) * c);
      if (whole && o >= g.lo && o + 16 <= g.hi) {
        *reinterpret_cast<uint4*>(g.dst + o) = make_uint4(w[0], w[1], w[2], w[3]);
      } else if (o + 16 > g.lo && o < g.hi) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (o + 2 * k >= g.lo && o + 2 * k < g.hi)
            *reinterpret_cast<uint16_t*>(g.dst + o + 2 * k) =
                static_cast<uint16_t>(w[k / 2] >> (16 * (k & 1)));
      }
    }
  }
}

// ----------------------------------------------------------------------------
// Host side
// ----------------------------------------------------------------------------
namespace {

int64_t units_of(const void* p, int64_t bytes) {
  const int64_t pad = static_cast<int64_t>(reinterpret_cast<uintptr_t>(p) & 15);
  return (pad + bytes + GRAD_UNIT - 1) / GRAD_UNIT;
}

// Fills a table from the tensors [i, n) that have elements, as many as fit;
// returns the first one that is left.
template <int N>
int fill(GradTable<N>* t, const GradList& l, int i) {
  t->n = t->units = 0;
  for (; i < l.n && t->n < N; ++i) {
    if (l.numels[i] == 0) continue;
    const int64_t bytes = l.numels[i] * (l.dtypes[i] == KD_DTYPE_F32 ? 4 : 2);
    GradEntry& e = t->e[t->n];
    e.src = static_cast<const unsigned char*>(l.grads[i]);
    e.dst = l.outs ? static_cast<unsigned char*>(l.outs[i]) : nullptr;
    e.bytes = bytes;
    e.first = t->units;
    e.dtype = l.dtypes[i];
    t->units += static_cast<uint32_t>(units_of(e.src, bytes));
    ++t->n;
  }
  return i;
}

template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kern)(KArgs...), unsigned blocks, cudaStream_t s, bool pdl,
                   const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(GRAD_THREADS);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  count_launch();
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

unsigned grid_for(uint32_t units, int num_sms) {
  const unsigned cap = static_cast<unsigned>(std::min<int64_t>(
      static_cast<int64_t>(num_sms) * GRAD_BLOCKS_PER_SM, GRAD_MAX_BLOCKS));
  return std::max(1u, std::min(units, cap));
}

// One pass over the list, a launch for each table of it: the sums (the launches'
// partials one after the other, *n_partials of them), or the scaling.
template <int N>
cudaError_t sum_pass(const GradList& l, double* partials, int* n_partials, uint32_t* status,
                     cudaStream_t s, int num_sms) {
  GradTable<N> t;
  int i = 0;
  *n_partials = 0;
  do {
    i = fill(&t, l, i);
    const unsigned blocks = grid_for(t.units, num_sms);
    const cudaError_t e =
        launch(grad_sumsq_kernel<N>, blocks, s, false, t, partials + *n_partials, status);
    if (e != cudaSuccess) return e;
    *n_partials += static_cast<int>(blocks);
  } while (i < l.n);
  return cudaSuccess;
}

template <int N>
cudaError_t scale_pass(const GradList& l, const double* partials, int n_partials, double max_norm,
                       float* norm, uint32_t* status, cudaStream_t s, int num_sms, bool pdl) {
  GradTable<N> t;
  int i = 0;
  do {
    i = fill(&t, l, i);
    const cudaError_t e = launch(grad_scale_kernel<N>, grid_for(t.units, num_sms), s, pdl, t,
                                 partials, n_partials, max_norm, norm, status);
    if (e != cudaSuccess) return e;
    norm = nullptr;
    pdl = false;
  } while (i < l.n);
  return cudaSuccess;
}

}  // namespace

kd_status check_grads(const GradList& l, bool writes) {
  if (l.n < 1 || !l.grads || !l.numels || !l.dtypes || (writes && !l.outs))
    return KD_ERR_INVALID_ARG;
  int64_t units = 0;
  for (int i = 0; i < l.n; ++i) {
    if (l.numels[i] < 0) return KD_ERR_INVALID_ARG;
    if (l.dtypes[i] != KD_DTYPE_F32 && l.dtypes[i] != KD_DTYPE_BF16) return KD_ERR_UNSUPPORTED;
    if (l.numels[i] == 0) continue;
    const uintptr_t low = l.dtypes[i] == KD_DTYPE_F32 ? 3 : 1;
    if (!l.grads[i] || (reinterpret_cast<uintptr_t>(l.grads[i]) & low)) return KD_ERR_INVALID_ARG;
    if (writes && (!l.outs[i] || (reinterpret_cast<uintptr_t>(l.outs[i]) & low)))
      return KD_ERR_INVALID_ARG;
    if (l.numels[i] >= (int64_t(1) << 40)) return KD_ERR_UNSUPPORTED;
    units += units_of(l.grads[i], l.numels[i] * (low + 1));
    if (units >= (int64_t(1) << 31)) return KD_ERR_UNSUPPORTED;
  }
  if (!writes) return KD_OK;

  // Blocks read and write the list in any order, so no output may share memory with
  // another output, nor with a gradient other than its own.
  struct Range {
    uintptr_t begin, end;
    bool out;
    bool operator<(const Range& o) const { return begin < o.begin; }
  };
  Range* r = static_cast<Range*>(malloc(2 * sizeof(Range) * static_cast<size_t>(l.n)));
  if (!r) return KD_ERR_INTERNAL;
  size_t n_out = 0, n_in = 0;
  Range* in = r + l.n;
  for (int i = 0; i < l.n; ++i) {
    if (l.numels[i] == 0) continue;
    const uintptr_t bytes =
        static_cast<uintptr_t>(l.numels[i]) * (l.dtypes[i] == KD_DTYPE_F32 ? 4 : 2);
    const uintptr_t o = reinterpret_cast<uintptr_t>(l.outs[i]);
    const uintptr_t g = reinterpret_cast<uintptr_t>(l.grads[i]);
    r[n_out++] = Range{o, o + bytes, true};
    if (g != o) in[n_in++] = Range{g, g + bytes, false};
  }
  if (!std::is_sorted(r, r + n_out)) std::sort(r, r + n_out);
  if (!std::is_sorted(in, in + n_in)) std::sort(in, in + n_in);
  bool clash = false;
  uintptr_t end_out = 0, end_in = 0;
  for (size_t a = 0, b = 0; (a < n_out || b < n_in) && !clash;) {
    if (b >= n_in || (a < n_out && r[a].begin < in[b].begin)) {
      clash = r[a].begin < end_out || r[a].begin < end_in;
      end_out = std::max(end_out, r[a++].end);
    } else {
      clash = in[b].begin < end_out;
      end_in = std::max(end_in, in[b++].end);
    }
  }
  free(r);
  return clash ? KD_ERR_INVALID_ARG : KD_OK;
}

kd_status grad_sumsq(const GradList& l, double* sumsq, uint32_t* status, double* partials,
                     cudaStream_t s, int num_sms) {
  int n = 0;
  const cudaError_t e = l.n <= GRAD_FEW ? sum_pass<GRAD_FEW>(l, partials, &n, status, s, num_sms)
                                        : sum_pass<GRAD_MANY>(l, partials, &n, status, s, num_sms);
  if (e != cudaSuccess) return KD_ERR_CUDA;
  return launch(grad_total_kernel, 1, s, true, static_cast<const double*>(partials), n, sumsq) ==
                 cudaSuccess
             ? KD_OK
             : KD_ERR_CUDA;
}

kd_status grad_clip(const GradList& l, double max_norm, const double* sumsq, float* norm,
                    uint32_t* status, double* partials, cudaStream_t s, int num_sms) {
  int n = 1;
  cudaError_t e = cudaSuccess;
  if (!sumsq)
    e = l.n <= GRAD_FEW ? sum_pass<GRAD_FEW>(l, partials, &n, status, s, num_sms)
                        : sum_pass<GRAD_MANY>(l, partials, &n, status, s, num_sms);
  if (e != cudaSuccess) return KD_ERR_CUDA;
  const double* p = sumsq ? sumsq : partials;
  e = l.n <= GRAD_FEW
          ? scale_pass<GRAD_FEW>(l, p, n, max_norm, norm, status, s, num_sms, !sumsq)
          : scale_pass<GRAD_MANY>(l, p, n, max_norm, norm, status, s, num_sms, !sumsq);
  return e == cudaSuccess ? KD_OK : KD_ERR_CUDA;
}

}  // namespace kd
