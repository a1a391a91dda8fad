// The global norm of many gradient tensors, and clipping by it:
//
//   norm = sqrt(sum_i sum_j g_ij^2)     c = min(1, max_norm / (norm + 1e-6))
//   out_ij = g_ij * c                   (out may be g itself)
//
// The tensors are cut into chunks of at most 32 KiB; the CTAs
// go through them side by side, and a thread has 4 x 16 bytes in flight. The first kernel leaves one partial sum of
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

constexpr int kClipThreads = 256;
constexpr int kVectors = 8;       // 16-byte vectors of a chunk per thread
constexpr int kAtOnce = 4;        // of them in flight
constexpr int kCtasPerSm = 6;
constexpr int kParts = MOE_GRAD_PARTIALS;
constexpr int kMaxTensors = 1024;  // per launch: the table travels as kernel arguments

// `chunk0[i]` is the tensor's first chunk. Its first chunk also holds the
// elements before its first 128-byte boundary.
template <int kCap>
struct GradTable {
  static constexpr int cap = kCap;
  const void* g[kCap];
  void* out[kCap];
  int64_t size[kCap];
  int32_t chunk0[kCap + 1];
  uint8_t type[kCap];
  int32_t n;
  int32_t in_place;  // every tensor's output is the tensor itself
  int32_t vectors;   // 16-byte vectors per thread and chunk, 1 to kVectors
};

struct Span {
  int64_t begin, end;
};

MOE_DEV int elements_to_boundary(const void* p, int es, uint32_t boundary = 16u) {
  return (int)((0u - (uint32_t)reinterpret_cast<uintptr_t>(p)) & (boundary - 1u)) / es;
}

template <int kCap>
MOE_DEV Span span_of(const GradTable<kCap>& t, int i, int chunk) {
  const int es = t.type[i] == MOE_FP32 ? 4 : 2;
  const int64_t head = elements_to_boundary(t.g[i], es, 128u);
  const int64_t k = chunk - t.chunk0[i], len = t.vectors * (kClipThreads * 16 / es);
  Span s;
  s.begin = k == 0 ? 0 : head + k * len;
  s.end = min(head + (k + 1) * len, t.size[i]);
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

// the elements of a 32-bit word as fp32, and back
template <typename T>
MOE_DEV void word_to_f(uint32_t w, float (&f)[4 / sizeof(T)]) {
  if constexpr (std::is_same_v<T, float>) {
    f[0] = __uint_as_float(w);
  } else if constexpr (std::is_same_v<T, __half>) {
    f[0] = __half2float(__ushort_as_half((unsigned short)(w & 0xFFFFu)));
    f[1] = __half2float(__ushort_as_half((unsigned short)(w >> 16)));
  } else {
    f[0] = bf16_lo(w);
    f[1] = bf16_hi(w);
  }
}
template <typename T>
MOE_DEV uint32_t word_scaled(uint32_t w, float c) {
  float f[4 / sizeof(T)];
  word_to_f<T>(w, f);
  if constexpr (std::is_same_v<T, float>) {
    return __float_as_uint(f[0] * c);
  } else if constexpr (std::is_same_v<T, __half>) {
    return (uint32_t)__half_as_ushort(__float2half_rn(f[0] * c)) |
           ((uint32_t)__half_as_ushort(__float2half_rn(f[1] * c)) << 16);
  } else {
    return pack_bf16x2(f[0] * c, f[1] * c);
  }
}

template <typename T>
MOE_DEV uint4 vector_scaled(const uint4& x, float c) {
  return make_uint4(word_scaled<T>(x.x, c), word_scaled<T>(x.y, c), word_scaled<T>(x.z, c),
                    word_scaled<T>(x.w, c));
}

// the squares of one 16-byte vector, out of line: zeros and extremes only
template <typename T>
__device__ __noinline__ double squares_in_fp64(uint4 x) {
  constexpr int kE = 4 / sizeof(T);
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  double d = 0.0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float f[kE];
    word_to_f<T>(w[i], f);
#pragma unroll
    for (int j = 0; j < kE; ++j) d = fma((double)f[j], (double)f[j], d);
  }
  return d;
}

// The squares of one 16-byte vector. fp32 keeps them to 2^-22 unless their
// sum is outside [2^-80, 2^100], where a square may have been lost or have
// overflowed.
template <typename T>
MOE_DEV double squares(const uint4& x) {
  constexpr int kE = 4 / sizeof(T);
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float f[kE];
    word_to_f<T>(w[i], f);
#pragma unroll
    for (int j = 0; j < kE; ++j) s = fmaf(f[j], f[j], s);
  }
  return s > 0x1p-80f && s < 0x1p100f ? (double)s : squares_in_fp64<T>(x);
}

template <typename T>
MOE_DEV double span_squares(const T* g, const Span& s) {
  constexpr int kV = 16 / sizeof(T);
  double sum = 0.0;
  const int64_t at = min(s.begin + elements_to_boundary(g + s.begin, sizeof(T)), s.end);
  if (s.begin + threadIdx.x < at) {
    const double f = (double)grad_f<T>(g[s.begin + threadIdx.x]);
    sum = fma(f, f, sum);
  }
  const int n = (int)(s.end - at) / kV;
  const uint4* const v = reinterpret_cast<const uint4*>(g + at);
  int q = threadIdx.x;
  for (; q + (kAtOnce - 1) * kClipThreads < n; q += kAtOnce * kClipThreads) {
    uint4 x[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) x[i] = v[q + i * kClipThreads];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) sum += squares<T>(x[i]);
  }
  for (; q < n; q += kClipThreads) sum += squares<T>(v[q]);
  const int64_t rest = at + (int64_t)n * kV + threadIdx.x;
  if (rest < s.end) {
    const double f = (double)grad_f<T>(g[rest]);
    sum = fma(f, f, sum);
  }
  return sum;
}

template <int kCap>
__global__ void __launch_bounds__(kClipThreads, kCtasPerSm)
    grad_sumsq_kernel(const __grid_constant__ GradTable<kCap> t, double* partials, int add) {
  __shared__ double red[kClipThreads / 32];
  const int total = t.chunk0[t.n];
  double sum = 0.0;
  cudaTriggerProgrammaticLaunchCompletion();
  int i = (int)blockIdx.x < total ? tensor_of(t, blockIdx.x) : 0;
  for (int c = blockIdx.x; c < total; c += gridDim.x) {
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
  if (((reinterpret_cast<uintptr_t>(g) ^ reinterpret_cast<uintptr_t>(out)) & 15u) != 0) {
    for (int64_t i = s.begin + threadIdx.x; i < s.end; i += kClipThreads)
      out[i] = grad_t<T>(grad_f<T>(g[i]) * c);
    return;
  }
  const int64_t at = min(s.begin + elements_to_boundary(g + s.begin, sizeof(T)), s.end);
  if (s.begin + threadIdx.x < at)
    out[s.begin + threadIdx.x] = grad_t<T>(grad_f<T>(g[s.begin + threadIdx.x]) * c);
  const int n = (int)(s.end - at) / kV;
  const uint4* const v = reinterpret_cast<const uint4*>(g + at);
  uint4* const o = reinterpret_cast<uint4*>(out + at);
  int q = threadIdx.x;
  for (; q + (kAtOnce - 1) * kClipThreads < n; q += kAtOnce * kClipThreads) {
    uint4 x[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) x[i] = __ldcs(v + q + i * kClipThreads);
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) __stcs(o + q + i * kClipThreads, vector_scaled<T>(x[i], c));
  }
  for (; q < n; q += kClipThreads) __stcs(o + q, vector_scaled<T>(__ldcs(v + q), c));
  const int64_t rest = at + (int64_t)n * kV + threadIdx.x;
  if (rest < s.end) out[rest] = grad_t<T>(grad_f<T>(g[rest]) * c);
}

template <int kCap>
__global__ void __launch_bounds__(kClipThreads, kCtasPerSm)
    grad_clip_kernel(const __grid_constant__ GradTable<kCap> t, const double* partials,
                     float max_norm, float* norm) {
  __shared__ double red[kClipThreads / 32];
  __shared__ float factor;
  double sum = 0.0;
  cudaGridDependencySynchronize();
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
  // backwards: the last chunks that the norm read are still in L2
  int k = total - 1 - (int)blockIdx.x;
  int i = k >= 0 ? tensor_of(t, k) : 0;
  for (; k >= 0; k -= gridDim.x) {
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

int chunks_of(const void* g, int64_t size, int es, int vectors) {
  if (size == 0) return 0;
  const int64_t head = (int64_t)((0 - reinterpret_cast<uintptr_t>(g)) & 127) / es;
  const int64_t rest = size > head ? size - head : 1, len = vectors * (kClipThreads * 16 / es);
  return (int)((rest + len - 1) / len);
}

// Vectors per thread and chunk: fewer where the tensors are small, so that
// the chunks still go round the CTAs that fit on the device.
int vectors_of(const moe_grad_list& l, int ctas) {
  int64_t bytes = 0;
  for (int i = 0; i < l.n; ++i) bytes += l.sizes[i] * element_size(l.types[i]);
  const int64_t each = bytes / ((int64_t)ctas * kClipThreads * 16);
  return each >= kVectors ? kVectors : each < 1 ? 1 : (int)each;
}

// Runs f(table) over the list's tensors, kCap at a time; tensors without
// elements are left out.
template <int kCap, typename F>
cudaError_t over_tables(const moe_grad_list& l, int ctas, F&& f) {
  int at = 0;
  bool first = true;
  do {
    GradTable<kCap> t;
    t.n = 0;
    t.chunk0[0] = 0;
    t.in_place = 1;
    t.vectors = vectors_of(l, ctas);
    for (; at < l.n && t.n < kCap; ++at) {
      if (l.sizes[at] == 0) continue;
      const int i = t.n++;
      t.g[i] = l.grads[at];
      t.out[i] = l.out ? l.out[at] : const_cast<void*>(l.grads[at]);
      if (t.out[i] != t.g[i]) t.in_place = 0;
      t.size[i] = l.sizes[at];
      t.type[i] = (uint8_t)l.types[at];
      t.chunk0[i + 1] = t.chunk0[i] + chunks_of(t.g[i], t.size[i], element_size(l.types[at]), t.vectors);
    }
    const cudaError_t e = f(t, first);
    if (e != cudaSuccess) return e;
    first = false;
  } while (at < l.n);
  return cudaSuccess;
}

template <typename F>
cudaError_t over_list(const moe_grad_list& l, int ctas, F&& f) {
  // the table is copied to the device with every launch: no larger than needed
  if (l.n <= 16) return over_tables<16>(l, ctas, f);
  if (l.n <= 128) return over_tables<128>(l, ctas, f);
  if (l.n <= 512) return over_tables<512>(l, ctas, f);
  return over_tables<kMaxTensors>(l, ctas, f);
}

int clip_grid(int sms) { return std::min(kParts, kCtasPerSm * sms); }

int check_list(const moe_grad_list* l) {
  if (!l) return MOE_ERR_NULL;
  if (l->n < 0) return MOE_ERR_SHAPE;
  if (l->n > 0 && (!l->grads || !l->sizes || !l->types)) return MOE_ERR_NULL;
  int64_t total = 0;
  for (int i = 0; i < l->n; ++i) {
    if (l->sizes[i] < 0 || l->sizes[i] > (1ll << 42)) return MOE_ERR_SHAPE;
    if (l->types[i] < MOE_BF16 || l->types[i] > MOE_FP32) return MOE_ERR_SHAPE;
    // chunks: of kVectors vectors a thread, but for lists that are small
    total += l->sizes[i] * element_size(l->types[i]) / (kVectors * kClipThreads * 16) + 4;
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
  return cuda_status(over_list(*list, most, go));
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
    using Table = std::decay_t<decltype(t)>;
    void (*kernel)(const Table, const double*, float, float*) = grad_clip_kernel<Table::cap>;
    return launch_dependent(kernel, (unsigned)grid, kClipThreads, 0, s, t, partials, max_norm, norm);
  };
  return cuda_status(over_list(*list, most, go));
}

}  // extern "C"
