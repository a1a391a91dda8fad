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
// 0.7 G fp32 elements out of place take 1395 us (three passes at the copy
// rate: 1302), 512 mixed tensors of 150 M elements below the limit 70 (70).
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
constexpr int kSmall = MOE_GRAD_SMALL;  // lists that travel as kernel arguments
constexpr int kSearch = 4096;           // tensors whose first chunks fit in shared memory

// One tensor: `chunk0` is its first chunk in the list. That chunk also holds
// the elements before the tensor's first 128-byte boundary.
struct Entry {
  const void* g;
  void* out;
  int64_t size;
  int32_t chunk0;
  int32_t type;
};
static_assert(sizeof(Entry) == 32, "table entry");

// A list's tensors (those with elements), in the kernel's arguments, or in
// device memory for longer lists: a table of some hundred entries as arguments
// would cost more than the launch, and its look-ups, which go through the
// constant cache, more than the work (22 us against 5 for 471 tensors).
struct Small {
  Entry e[kSmall];
};
struct Table {
  const Entry* entries;  // device, or NULL: `small`
  int32_t n;
  int32_t chunks;
  int32_t in_place;      // every tensor's output is the tensor itself
  int32_t vectors;       // 16-byte vectors per thread and chunk, 1 to kVectors
};

struct Span {
  int64_t begin, end;
};

MOE_DEV int elements_to_boundary(const void* p, int es, uint32_t boundary = 16u) {
  return (int)((0u - (uint32_t)reinterpret_cast<uintptr_t>(p)) & (boundary - 1u)) / es;
}

MOE_DEV Span span_of(const Table& t, const Entry& e, int chunk) {
  const int es = e.type == MOE_FP32 ? 4 : 2;
  const int64_t head = elements_to_boundary(e.g, es, 128u);
  const int64_t k = chunk - e.chunk0, len = t.vectors * (kClipThreads * 16 / es);
  Span s;
  s.begin = k == 0 ? 0 : head + k * len;
  s.end = min(head + (k + 1) * len, e.size);
  return s;
}

// Finds a chunk's tensor: the last one whose first chunk is not after it.
template <bool kInArgs>
struct Finder {
  const Small& small;
  const Table& t;
  const int32_t* first;  // shared copy of the first chunks, or NULL
  MOE_DEV int chunk0(int i) const {
    if (kInArgs) return small.e[i].chunk0;
    return first != nullptr ? first[i] : t.entries[i].chunk0;
  }
  MOE_DEV Entry find(int chunk) const {
    int lo = 0, hi = t.n;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (chunk0(mid) <= chunk) lo = mid; else hi = mid;
    }
    return kInArgs ? small.e[lo] : t.entries[lo];
  }
};

// the first chunks into shared memory (lists of up to kSearch tensors)
template <bool kInArgs>
MOE_DEV const int32_t* load_first(const Table& t, int32_t* shared) {
  if constexpr (kInArgs) {
    return nullptr;
  } else {
    if (t.n > kSearch) return nullptr;
    for (int i = threadIdx.x; i < t.n; i += kClipThreads) shared[i] = t.entries[i].chunk0;
    __syncthreads();
    return shared;
  }
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

template <bool kInArgs>
__global__ void __launch_bounds__(kClipThreads, kCtasPerSm)
    grad_sumsq_kernel(const __grid_constant__ Small small, const Table t, double* partials) {
  __shared__ double red[kClipThreads / 32];
  extern __shared__ int32_t first[];
  double sum = 0.0;
  cudaTriggerProgrammaticLaunchCompletion();
  const Finder<kInArgs> finder{small, t, load_first<kInArgs>(t, first)};
  for (int c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const Entry e = finder.find(c);
    const Span s = span_of(t, e, c);
    if (e.type == MOE_FP32) sum += span_squares(static_cast<const float*>(e.g), s);
    else if (e.type == MOE_BF16) sum += span_squares(static_cast<const __nv_bfloat16*>(e.g), s);
    else sum += span_squares(static_cast<const __half*>(e.g), s);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kClipThreads / 32; ++w) sum += red[w];
    partials[blockIdx.x] = sum;
  }
  // the places that no CTA has are zero
  if (blockIdx.x == 0)
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

template <bool kInArgs>
__global__ void __launch_bounds__(kClipThreads, kCtasPerSm)
    grad_clip_kernel(const __grid_constant__ Small small, const Table t, const double* partials,
                     float max_norm, float* norm) {
  __shared__ double red[kClipThreads / 32];
  __shared__ float factor;
  extern __shared__ int32_t first[];
  double sum = 0.0;
  const Finder<kInArgs> finder{small, t, load_first<kInArgs>(t, first)};
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
  // backwards: the last chunks that the norm read are still in L2
  for (int k = t.chunks - 1 - (int)blockIdx.x; k >= 0; k -= gridDim.x) {
    const Entry e = finder.find(k);
    const Span s = span_of(t, e, k);
    if (e.type == MOE_FP32)
      span_scale(static_cast<const float*>(e.g), static_cast<float*>(e.out), s, c);
    else if (e.type == MOE_BF16)
      span_scale(static_cast<const __nv_bfloat16*>(e.g), static_cast<__nv_bfloat16*>(e.out), s, c);
    else
      span_scale(static_cast<const __half*>(e.g), static_cast<__half*>(e.out), s, c);
  }
}

int element_size(int type) { return type == MOE_FP32 ? 4 : 2; }

int clip_grid() { return std::min(kParts, kCtasPerSm * moe_device_sm_count()); }

// Vectors per thread and chunk: fewer where the tensors are small, so that
// the chunks still go round the CTAs that fit on a device.
int vectors_of(const moe_grad_list& l) {
  int64_t bytes = 0;
  for (int i = 0; i < l.n; ++i) bytes += l.sizes[i] * element_size(l.types[i]);
  const int64_t each = bytes / ((int64_t)kParts * kClipThreads * 16);
  return each >= kVectors ? kVectors : each < 1 ? 1 : (int)each;
}

// Runs over the list's tensors with elements: put(entry index, entry). Fills
// the sizes of *t.
template <typename F>
void entries_of(const moe_grad_list& l, Table* t, F&& put) {
  t->n = 0;
  t->chunks = 0;
  t->in_place = 1;
  t->vectors = vectors_of(l);
  for (int i = 0; i < l.n; ++i) {
    if (l.sizes[i] == 0) continue;
    const int es = element_size(l.types[i]);
    void* const out = l.out ? l.out[i] : const_cast<void*>(l.grads[i]);
    if (out != l.grads[i]) t->in_place = 0;
    put(t->n++, Entry{l.grads[i], out, l.sizes[i], t->chunks, l.types[i]});
    const int64_t head = (int64_t)((0 - reinterpret_cast<uintptr_t>(l.grads[i])) & 127) / es;
    const int64_t rest = l.sizes[i] > head ? l.sizes[i] - head : 1;
    const int64_t len = t->vectors * (kClipThreads * 16 / es);
    t->chunks += (int)((rest + len - 1) / len);
  }
}

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

// The kernels' arguments for a list. A table was checked when it was made.
struct Launch {
  Small small;
  Table t;
  size_t smem;
};
int launch_of(const moe_grad_list& l, Launch* a) {
  if (l.n <= kSmall) {
    const int bad = check_list(&l);
    if (bad != MOE_OK) return bad;
    a->t.entries = nullptr;
    entries_of(l, &a->t, [&](int i, const Entry& e) { a->small.e[i] = e; });
    a->smem = 0;
    return MOE_OK;
  }
  if (!l.table) return MOE_ERR_NULL;
  if (!aligned(l.table, 16)) return MOE_ERR_ALIGN;
  a->t = Table{static_cast<const Entry*>(l.table), l.plan[0], l.plan[1], l.plan[2], l.plan[3]};
  a->smem = a->t.n <= kSearch ? (size_t)a->t.n * 4 : 0;
  return MOE_OK;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_grad_table_size(const moe_grad_list* list) {
  if (check_list(list) != MOE_OK || list->n <= kSmall) return 0;
  return (size_t)list->n * sizeof(Entry);
}

int moe_grad_table(moe_grad_list* list, void* host_table) {
  const int bad = check_list(list);
  if (bad != MOE_OK) return bad;
  if (list->n <= kSmall) return MOE_OK;
  if (!host_table) return MOE_ERR_NULL;
  Entry* const e = static_cast<Entry*>(host_table);
  Table t{};
  entries_of(*list, &t, [&](int i, const Entry& x) { e[i] = x; });
  list->plan[0] = t.n;
  list->plan[1] = t.chunks;
  list->plan[2] = t.in_place;
  list->plan[3] = t.vectors;
  return MOE_OK;
}

int moe_grad_sumsq(const moe_grad_list* list, double* partials, void* stream) {
  if (!list || !partials) return MOE_ERR_NULL;
  if (!aligned(partials, 8)) return MOE_ERR_ALIGN;
  Launch a;
  const int r = launch_of(*list, &a);
  if (r != MOE_OK) return r;
  NvtxRange range("moe_grad_sumsq");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int grid = std::max(1, std::min(clip_grid(), a.t.chunks));
  if (a.t.entries)
    grad_sumsq_kernel<false><<<grid, kClipThreads, a.smem, s>>>(a.small, a.t, partials);
  else
    grad_sumsq_kernel<true><<<grid, kClipThreads, a.smem, s>>>(a.small, a.t, partials);
  return cuda_status(cudaGetLastError());
}

int moe_grad_clip(const moe_grad_list* list, const double* partials, float max_norm, float* norm,
                  void* stream) {
  if (!(max_norm >= 0.0f)) return MOE_ERR_SHAPE;
  if (!list || !partials || !norm) return MOE_ERR_NULL;
  if (!aligned(partials, 8) || !aligned(norm, 4)) return MOE_ERR_ALIGN;
  Launch a;
  const int r = launch_of(*list, &a);
  if (r != MOE_OK) return r;
  NvtxRange range("moe_grad_clip");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int grid = std::max(1, std::min(clip_grid(), a.t.chunks));
  void (*kernel)(const Small, const Table, const double*, float, float*) =
      a.t.entries ? grad_clip_kernel<false> : grad_clip_kernel<true>;
  return cuda_status(launch_dependent(kernel, (unsigned)grid, kClipThreads, a.smem, s, a.small, a.t,
                                      partials, max_norm, norm));
}

}  // extern "C"
