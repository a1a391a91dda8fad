// The global norm of many gradient tensors, and clipping by it:
//
//   norm = sqrt(sum_i sum_j g_ij^2)     c = min(1, max_norm / (norm + 1e-6))
//   out_ij = g_ij * c                   (out may be g itself)
//
// The tensors are cut into chunks of 8192 elements; each CTA takes a
// contiguous run of chunks. The first kernel leaves one partial sum of
// squares per CTA, the second adds them (every CTA the same sum, in the same
// order) and scales. No atomics: the norm is the same in every run.
//
// Squares are summed 8 at a time in fp32 and then in fp64, so that the sum's
// error does not grow with the number of elements; 8 squares that leave the
// range in which fp32 holds them exactly enough are summed again in fp64.
//
// Bound by HBM: one read for the norm, one read and one write for the
// scaling, of which the second read finds in L2 what the first read last.
#include <algorithm>
#include <type_traits>

#include "kernels.cuh"

namespace moe {

namespace {

constexpr int kChunk = 8192;
constexpr int kClipThreads = 256;
constexpr int kParts = MOE_GRAD_PARTIALS;
constexpr int kMaxTensors = 256;  // per launch: the table travels as kernel arguments

// `chunk0[i]` is the tensor's first chunk. Its first chunk also holds the
// elements before its first 16-byte boundary.
template <int kCap>
struct GradTable {
  const void* g[kCap];
  void* out[kCap];
  int64_t size[kCap];
  int32_t chunk0[kCap + 1];
  uint8_t type[kCap];
  int32_t n;
  int32_t in_place;  // every tensor's output is the tensor itself
};

struct Span {
  int64_t begin, end;
};

MOE_DEV int elements_to_boundary(const void* p, int es) {
  return (int)((16u - (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) / es;
}

template <int kCap>
MOE_DEV Span span_of(const GradTable<kCap>& t, int i, int chunk) {
  const int es = t.type[i] == MOE_FP32 ? 4 : 2;
  const int64_t head = elements_to_boundary(t.g[i], es);
  const int64_t k = chunk - t.chunk0[i];
  Span s;
  s.begin = k == 0 ? 0 : head + k * kChunk;
  s.end = min(head + (k + 1) * kChunk, t.size[i]);
  return s;
}

template <int kCap>
MOE_DEV int tensor_of(const GradTable<kCap>& t, int chunk) {
  int lo = 0, hi = t.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.chunk0[mid] <= chunk) lo = mid; else hi = mid;
  }
  return lo;
}

template <typename T>
MOE_DEV float grad_f(T v) {
  if constexpr (std::is_same_v<T, float>) return v;
  else if constexpr (std::is_same_v<T, __half>) return __half2float(v);
  else return __bfloat162float(v);
}
template <typename T>
MOE_DEV T grad_t(float v) {
  if constexpr (std::is_same_v<T, float>) return v;
  else if constexpr (std::is_same_v<T, __half>) return __float2half_rn(v);
  else return __float2bfloat16_rn(v);
}

template <typename T>
struct alignas(16) Vec {
  T v[16 / sizeof(T)];
};

// The squares of one 16-byte vector. fp32 keeps them to 2^-22 unless their
// sum is outside [2^-80, 2^100], where a square may have been lost or have
// overflowed.
template <typename T>
MOE_DEV double squares(const Vec<T>& x) {
  constexpr int kV = 16 / sizeof(T);
  float s = 0.0f, any = 0.0f;
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    const float f = grad_f<T>(x.v[i]);
    s = fmaf(f, f, s);
    any = fmaxf(any, fabsf(f));
  }
  if ((s > 0x1p-80f && s < 0x1p100f) || (s == 0.0f && any == 0.0f)) return (double)s;
  double d = 0.0;
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    const double f = (double)grad_f<T>(x.v[i]);
    d = fma(f, f, d);
  }
  return d;
}

template <typename T>
MOE_DEV double span_squares(const T* g, const Span& s) {
  constexpr int kV = 16 / sizeof(T);
  constexpr int kStep = kClipThreads * kV;
  double sum = 0.0;
  int64_t at = min(s.begin + elements_to_boundary(g + s.begin, sizeof(T)), s.end);
  if (s.begin + threadIdx.x < at) {
    const double f = (double)grad_f<T>(g[s.begin + threadIdx.x]);
    sum = fma(f, f, sum);
  }
  for (; at + kStep <= s.end; at += kStep)
    sum += squares<T>(*reinterpret_cast<const Vec<T>*>(g + at + threadIdx.x * kV));
  for (int64_t i = at + threadIdx.x; i < s.end; i += kClipThreads) {
    const double f = (double)grad_f<T>(g[i]);
    sum = fma(f, f, sum);
  }
  return sum;
}

template <int kCap>
__global__ void __launch_bounds__(kClipThreads)
    grad_sumsq_kernel(const __grid_constant__ GradTable<kCap> t, double* partials, int add) {
  __shared__ double red[kClipThreads / 32];
  const int total = t.chunk0[t.n];
  const int c0 = (int)((int64_t)total * blockIdx.x / gridDim.x);
  const int c1 = (int)((int64_t)total * (blockIdx.x + 1) / gridDim.x);
  double sum = 0.0;
  int i = c0 < c1 ? tensor_of(t, c0) : 0;
  for (int c = c0; c < c1; ++c) {
    while (c >= t.chunk0[i + 1]) ++i;
    const Span s = span_of(t, i, c);
    if (t.type[i] == MOE_FP32) sum += span_squares(static_cast<const float*>(t.g[i]), s);
    else if (t.type[i] == MOE_BF16) sum += span_squares(static_cast<const __nv_bfloat16*>(t.g[i]), s);
    else sum += span_squares(static_cast<const __half*>(t.g[i]), s);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kClipThreads / 32; ++w) sum += red[w];
    partials[blockIdx.x] = add ? partials[blockIdx.x] + sum : sum;
  }
  // the places that no CTA has are zero
  if (blockIdx.x == 0 && !add)
    for (int j = gridDim.x + threadIdx.x; j < kParts; j += kClipThreads) partials[j] = 0.0;
}

template <typename T>
MOE_DEV void span_scale(const T* g, T* out, const Span& s, float c) {
  constexpr int kV = 16 / sizeof(T);
  constexpr int kStep = kClipThreads * kV;
  int64_t at = s.begin;
  if (((reinterpret_cast<uintptr_t>(g) ^ reinterpret_cast<uintptr_t>(out)) & 15u) == 0) {
    at = min(s.begin + elements_to_boundary(g + s.begin, sizeof(T)), s.end);
    if (s.begin + threadIdx.x < at)
      out[s.begin + threadIdx.x] = grad_t<T>(grad_f<T>(g[s.begin + threadIdx.x]) * c);
    for (; at + kStep <= s.end; at += kStep) {
      Vec<T> x = *reinterpret_cast<const Vec<T>*>(g + at + threadIdx.x * kV);
#pragma unroll
      for (int i = 0; i < kV; ++i) x.v[i] = grad_t<T>(grad_f<T>(x.v[i]) * c);
      *reinterpret_cast<Vec<T>*>(out + at + threadIdx.x * kV) = x;
    }
  }
  for (int64_t i = at + threadIdx.x; i < s.end; i += kClipThreads)
    out[i] = grad_t<T>(grad_f<T>(g[i]) * c);
}

template <int kCap>
__global__ void __launch_bounds__(kClipThreads)
    grad_clip_kernel(const __grid_constant__ GradTable<kCap> t, const double* partials,
                     float max_norm, float* norm) {
  __shared__ double red[kClipThreads / 32];
  __shared__ float factor;
  double sum = 0.0;
  for (int j = threadIdx.x; j < kParts; j += kClipThreads) sum += partials[j];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kClipThreads / 32; ++w) sum += red[w];
    const double root = sqrt(sum);
    const double q = (double)max_norm / (root + 1e-6);
    factor = q >= 1.0 ? 1.0f : (float)q;  // a NaN stays one
    if (blockIdx.x == 0) *norm = (float)root;
  }
  __syncthreads();
  const float c = factor;
  if (c == 1.0f && t.in_place) return;
  const int total = t.chunk0[t.n];
  const int c0 = (int)((int64_t)total * blockIdx.x / gridDim.x);
  const int c1 = (int)((int64_t)total * (blockIdx.x + 1) / gridDim.x);
  if (c0 >= c1) return;
  // backwards: the last chunks that the norm read are still in L2
  int i = tensor_of(t, c1 - 1);
  for (int k = c1 - 1; k >= c0; --k) {
    while (k < t.chunk0[i]) --i;
    const Span s = span_of(t, i, k);
    if (t.type[i] == MOE_FP32)
      span_scale(static_cast<const float*>(t.g[i]), static_cast<float*>(t.out[i]), s, c);
    else if (t.type[i] == MOE_BF16)
      span_scale(static_cast<const __nv_bfloat16*>(t.g[i]), static_cast<__nv_bfloat16*>(t.out[i]), s, c);
    else
      span_scale(static_cast<const __half*>(t.g[i]), static_cast<__half*>(t.out[i]), s, c);
  }
}

int element_size(int type) { return type == MOE_FP32 ? 4 : 2; }

int chunks_of(const void* g, int64_t size, int es) {
  if (size == 0) return 0;
  const int64_t head = (int64_t)((16 - (reinterpret_cast<uintptr_t>(g) & 15)) & 15) / es;
  const int64_t rest = size > head ? size - head : 1;
  return (int)((rest + kChunk - 1) / kChunk);
}

// Runs f(table) over the list's tensors, kCap at a time; tensors without
// elements are left out.
template <int kCap, typename F>
cudaError_t over_tables(const moe_grad_list& l, F&& f) {
  int at = 0;
  bool first = true;
  do {
    GradTable<kCap> t;
    t.n = 0;
    t.chunk0[0] = 0;
    t.in_place = 1;
    for (; at < l.n && t.n < kCap; ++at) {
      if (l.sizes[at] == 0) continue;
      const int i = t.n++;
      t.g[i] = l.grads[at];
      t.out[i] = l.out ? l.out[at] : const_cast<void*>(l.grads[at]);
      if (t.out[i] != t.g[i]) t.in_place = 0;
      t.size[i] = l.sizes[at];
      t.type[i] = (uint8_t)l.types[at];
      t.chunk0[i + 1] = t.chunk0[i] + chunks_of(t.g[i], t.size[i], element_size(l.types[at]));
    }
    const cudaError_t e = f(t, first);
    if (e != cudaSuccess) return e;
    first = false;
  } while (at < l.n);
  return cudaSuccess;
}

int clip_grid(int sms) { return std::min(kParts, 4 * sms); }

int check_list(const moe_grad_list* l) {
  if (!l) return MOE_ERR_NULL;
  if (l->n < 0) return MOE_ERR_SHAPE;
  if (l->n > 0 && (!l->grads || !l->sizes || !l->types)) return MOE_ERR_NULL;
  int64_t total = 0;
  for (int i = 0; i < l->n; ++i) {
    if (l->sizes[i] < 0 || l->sizes[i] > (1ll << 42)) return MOE_ERR_SHAPE;
    if (l->types[i] < MOE_BF16 || l->types[i] > MOE_FP32) return MOE_ERR_SHAPE;
    total += l->sizes[i] / kChunk + 2;
    if (total >= (1ll << 31)) return MOE_ERR_SHAPE;
    if (l->sizes[i] == 0) continue;
    if (!l->grads[i] || (l->out && !l->out[i])) return MOE_ERR_NULL;
    const int es = element_size(l->types[i]);
    if (!aligned(l->grads[i], es) || (l->out && !aligned(l->out[i], es))) return MOE_ERR_ALIGN;
  }
  return MOE_OK;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

int moe_grad_sumsq(const moe_grad_list* list, double* partials, void* stream) {
  const int bad = check_list(list);
  if (bad != MOE_OK) return bad;
  if (!partials) return MOE_ERR_NULL;
  if (!aligned(partials, 8)) return MOE_ERR_ALIGN;
  NvtxRange range("moe_grad_sumsq");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int most = clip_grid(moe_device_sm_count());
  auto go = [&](const auto& t, bool first) {
    const int total = t.chunk0[t.n];
    const int grid = total < 1 ? 1 : std::min(most, total);
    grad_sumsq_kernel<<<grid, kClipThreads, 0, s>>>(t, partials, first ? 0 : 1);
    return cudaGetLastError();
  };
  return cuda_status(list->n <= 32 ? over_tables<32>(*list, go)
                                   : over_tables<kMaxTensors>(*list, go));
}

int moe_grad_clip(const moe_grad_list* list, const double* partials, float max_norm, float* norm,
                  void* stream) {
  const int bad = check_list(list);
  if (bad != MOE_OK) return bad;
  if (!(max_norm >= 0.0f)) return MOE_ERR_SHAPE;
  if (!partials || !norm) return MOE_ERR_NULL;
  if (!aligned(partials, 8) || !aligned(norm, 4)) return MOE_ERR_ALIGN;
  NvtxRange range("moe_grad_clip");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int most = clip_grid(moe_device_sm_count());
  auto go = [&](const auto& t, bool) {
    const int total = t.chunk0[t.n];
    const int grid = total < 1 ? 1 : std::min(most, total);
    grad_clip_kernel<<<grid, kClipThreads, 0, s>>>(t, partials, max_norm, norm);
    return cudaGetLastError();
  };
  return cuda_status(list->n <= 32 ? over_tables<32>(*list, go)
                                   : over_tables<kMaxTensors>(*list, go));
}

}  // extern "C"
