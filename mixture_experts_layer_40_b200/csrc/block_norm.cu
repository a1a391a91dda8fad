// Norms before and after a block, with its gate and residual scale, and their
// gradients: the Transformer block around the layer ("DeepSeek-V3:
// Auxiliary-Loss-Free MoE Load Balancing, ...").
//
//   N(v; w) = v * rsqrt(mean(v^2) + eps) * w
//   r = x + alpha * scale * gate * N(z; post)     u = N(r; pre)
//
// One pass over the rows: a team of warps holds a row in registers, so x and
// z are read once and r and u written once, whatever the number of norms.
// The backward recomputes both statistics from the rows it has to read
// anyway (one more term in a reduction it needs for the gradient), so the
// forward saves nothing. All arithmetic is fp32; r is rounded when it is
// stored, and u is computed from the unrounded row.
//
// Bound by HBM: a few operations per byte.
#include <atomic>
#include <type_traits>

#include "kernels.cuh"

namespace moe {

namespace {

constexpr int kNormThreads = 512;   // most threads of a CTA
constexpr int kTeamsMax = 8;        // rows in flight per CTA
constexpr int kMaxParts = 1024;     // partial column sums

enum Gate : int { kGateNone = 0, kGateRow = 1, kGateFull = 2 };

struct NormArgs {
  const void* x;      // Res [T, H] (backward: r)
  const void* z;      // Act [T, H] or NULL
  const void* gate;   // float [T], Act [T, H] or NULL
  const void* pre;    // weights: float or Act [H]
  const void* post;
  const void* scale;
  void* r;            // Res [T, H]
  void* u;            // Act [T, H]
  int64_t T;
  int32_t H;
  int32_t gate_kind;
  int32_t w_f32;
  int32_t team_warps;
  float alpha, eps;
  // backward
  const void* dr;     // Res
  const void* du;     // Act
  void* dx;           // Res
  void* dz;           // Act
  void* dgate;        // float [T] or Act [T, H]
  float* part;        // [parts, 2, H]
};

// up to 8 elements from p as fp32; kVec: all 8, 16-byte aligned
template <typename T>
MOE_DEV float to_f(T v) {
  if constexpr (std::is_same_v<T, float>) return v;
  else if constexpr (std::is_same_v<T, __half>) return __half2float(v);
  else return __bfloat162float(v);
}
template <typename T>
MOE_DEV T from_f(float v) {
  if constexpr (std::is_same_v<T, float>) return v;
  else if constexpr (std::is_same_v<T, __half>) return __float2half_rn(v);
  else return __float2bfloat16_rn(v);
}

template <typename T, bool kVec>
MOE_DEV void load8(const void* base, int64_t at, int n, float (&v)[8]) {
  const T* p = static_cast<const T*>(base) + at;
  if constexpr (kVec) {
    constexpr int kWords = sizeof(T) * 2;
    if (n > 0) {
      uint32_t w[kWords];
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const uint4 q = reinterpret_cast<const uint4*>(p)[i];
        w[4 * i] = q.x; w[4 * i + 1] = q.y; w[4 * i + 2] = q.z; w[4 * i + 3] = q.w;
      }
      const T* e = reinterpret_cast<const T*>(w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = to_f<T>(e[i]);
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? to_f<T>(p[i]) : 0.0f;
  }
}

template <typename T, bool kVec>
MOE_DEV void store8(void* base, int64_t at, int n, const float (&v)[8]) {
  T* p = static_cast<T*>(base) + at;
  if constexpr (kVec) {
    if (n > 0) {
      alignas(16) T e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = from_f<T>(v[i]);
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i)
        reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<const uint4*>(e)[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = from_f<T>(v[i]);
  }
}

template <typename Act, bool kVec>
MOE_DEV void load_w8(const void* w, bool f32, int at, int n, float (&v)[8]) {
  if (f32) load8<float, kVec>(w, at, n, v);
  else load8<Act, kVec>(w, at, n, v);
}

// Sums over a team of warps. Two buffers in turn: a thread writes one again
// only after a barrier that every reader of its last use has passed.
template <int kN>
MOE_DEV void team_sum(float (&v)[kN], int warps, int team, int wid, int lane,
                      float (*buf)[kTeamsMax][3][16], int& turn) {
#pragma unroll
  for (int i = 0; i < kN; ++i)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (warps == 1) return;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < kN; ++i) buf[turn][team][i][wid] = v[i];
  }
  asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(warps * 32) : "memory");
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    float s = 0.0f;
    for (int j = 0; j < warps; ++j) s += buf[turn][team][i][j];
    v[i] = s;
  }
  turn ^= 1;
}

template <typename Res, typename Act, int kNC, bool kVec>
__global__ void __launch_bounds__(kNormThreads) block_norm_kernel(const NormArgs p) {
  __shared__ float buf[2][kTeamsMax][3][16];
  const int W = p.team_warps, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int team = warp / W, wid = warp - team * W;
  const int teams = (blockDim.x >> 5) / W;
  const int H = p.H;
  const float inv_h = 1.0f / (float)H;
  int turn = 0;
  int col[kNC], n[kNC];
  float pre[kNC][8], post[kNC][8];  // post: alpha * scale * post
#pragma unroll
  for (int c = 0; c < kNC; ++c) {
    col[c] = ((c * W + wid) * 32 + lane) * 8;
    n[c] = min(max(H - col[c], 0), 8);
    if (p.pre) load_w8<Act, kVec>(p.pre, p.w_f32, col[c], n[c], pre[c]);
#pragma unroll
    for (int i = 0; i < 8; ++i) post[c][i] = p.alpha;
    float w[8];
    if (p.post) {
      load_w8<Act, kVec>(p.post, p.w_f32, col[c], n[c], w);
#pragma unroll
      for (int i = 0; i < 8; ++i) post[c][i] *= w[i];
    }
    if (p.scale) {
      load_w8<Act, kVec>(p.scale, p.w_f32, col[c], n[c], w);
#pragma unroll
      for (int i = 0; i < 8; ++i) post[c][i] *= w[i];
    }
  }
  for (int64_t row = (int64_t)blockIdx.x * teams + team; row < p.T;
       row += (int64_t)gridDim.x * teams) {
    const int64_t at = row * H;
    float r[kNC][8];
#pragma unroll
    for (int c = 0; c < kNC; ++c) load8<Res, kVec>(p.x, at + col[c], n[c], r[c]);
    if (p.z) {
      float z[kNC][8];
#pragma unroll
      for (int c = 0; c < kNC; ++c) load8<Act, kVec>(p.z, at + col[c], n[c], z[c]);
      float f = 1.0f;
      if (p.gate_kind == kGateRow) f = static_cast<const float*>(p.gate)[row];
      if (p.post) {
        float s[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < kNC; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) s[0] = fmaf(z[c][i], z[c][i], s[0]);
        team_sum(s, W, team, wid, lane, buf, turn);
        f *= rsqrtf(fmaf(s[0], inv_h, p.eps));
      }
#pragma unroll
      for (int c = 0; c < kNC; ++c) {
        if (p.gate_kind == kGateFull) {
          float g[8];
          load8<Act, kVec>(p.gate, at + col[c], n[c], g);
#pragma unroll
          for (int i = 0; i < 8; ++i) z[c][i] *= g[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) r[c][i] = fmaf(post[c][i] * f, z[c][i], r[c][i]);
        store8<Res, kVec>(p.r, at + col[c], n[c], r[c]);
      }
    }
    if (p.pre) {
      float s[1] = {0.0f};
#pragma unroll
      for (int c = 0; c < kNC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[0] = fmaf(r[c][i], r[c][i], s[0]);
      team_sum(s, W, team, wid, lane, buf, turn);
      const float f = rsqrtf(fmaf(s[0], inv_h, p.eps));
#pragma unroll
      for (int c = 0; c < kNC; ++c) {
#pragma unroll
        for (int i = 0; i < 8; ++i) r[c][i] *= f * pre[c][i];
        store8<Act, kVec>(p.u, at + col[c], n[c], r[c]);
      }
    }
  }
}

// The backward. With h = r R (R = rsqrt(mean r^2 + eps)) and y = z Z:
//   e  = dr + R (du pre - h mean(du pre h))          dx = e
//   q  = alpha scale gate e
//   dz = Z (q post - y mean(q post y))               (without post: dz = q)
//   dpre = sum_t du h;  c = sum_t alpha gate e y;  dpost = scale c;
//   dscale = post c;    dgate = alpha scale post y e (summed over the row)
// Two rounds of row sums: (r^2, du pre r, z^2), then alpha scale post y e,
// which gives both the row's gate gradient and the mean in dz. Each thread
// keeps its columns' sums over the rows of its CTA in registers; the CTAs'
// sums are added in a fixed order by a second kernel.
template <typename Res, typename Act, int kNC, bool kVec>
__global__ void __launch_bounds__(kNormThreads) block_norm_backward_kernel(const NormArgs p) {
  __shared__ float buf[2][kTeamsMax][3][16];
  const int W = p.team_warps, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int team = warp / W, wid = warp - team * W;
  const int teams = (blockDim.x >> 5) / W;
  const int H = p.H;
  const float inv_h = 1.0f / (float)H;
  int turn = 0;
  int col[kNC], n[kNC];
  float s_pre[kNC][8], s_c[kNC][8];
#pragma unroll
  for (int c = 0; c < kNC; ++c) {
    col[c] = ((c * W + wid) * 32 + lane) * 8;
    n[c] = min(max(H - col[c], 0), 8);
#pragma unroll
    for (int i = 0; i < 8; ++i) s_pre[c][i] = s_c[c][i] = 0.0f;
  }
  for (int64_t row = (int64_t)blockIdx.x * teams + team; row < p.T;
       row += (int64_t)gridDim.x * teams) {
    const int64_t at = row * H;
    float r[kNC][8], du[kNC][8], z[kNC][8], e[kNC][8];
    float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < kNC; ++c) {
      if (p.dr) {
        load8<Res, kVec>(p.dr, at + col[c], n[c], e[c]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) e[c][i] = 0.0f;
      }
      if (p.pre) {
        load8<Res, kVec>(p.x, at + col[c], n[c], r[c]);
        load8<Act, kVec>(p.du, at + col[c], n[c], du[c]);
        float w[8];
        load_w8<Act, kVec>(p.pre, p.w_f32, col[c], n[c], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          s[0] = fmaf(r[c][i], r[c][i], s[0]);
          s[1] = fmaf(du[c][i] * w[i], r[c][i], s[1]);
        }
      }
      if (p.z) {
        load8<Act, kVec>(p.z, at + col[c], n[c], z[c]);
        if (p.post) {
#pragma unroll
          for (int i = 0; i < 8; ++i) s[2] = fmaf(z[c][i], z[c][i], s[2]);
        }
      }
    }
    team_sum(s, W, team, wid, lane, buf, turn);
    if (p.pre) {
      const float R = rsqrtf(fmaf(s[0], inv_h, p.eps));
      const float mean = s[1] * R * inv_h;
#pragma unroll
      for (int c = 0; c < kNC; ++c) {
        float w[8];
        load_w8<Act, kVec>(p.pre, p.w_f32, col[c], n[c], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float h = r[c][i] * R;
          s_pre[c][i] = fmaf(du[c][i], h, s_pre[c][i]);
          e[c][i] = fmaf(R, fmaf(du[c][i], w[i], -h * mean), e[c][i]);
        }
        if (p.dx) store8<Res, kVec>(p.dx, at + col[c], n[c], e[c]);
      }
    }
    if (!p.z) continue;
    const float Z = p.post ? rsqrtf(fmaf(s[2], inv_h, p.eps)) : 1.0f;
    float row_gate = 1.0f;
    if (p.gate_kind == kGateRow) row_gate = static_cast<const float*>(p.gate)[row];
    float t[1] = {0.0f};
    // e becomes q post; with a full gate its gradient goes out here
#pragma unroll
    for (int c = 0; c < kNC; ++c) {
      float post[8], sc[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) post[i] = sc[i] = 1.0f;
      if (p.post) load_w8<Act, kVec>(p.post, p.w_f32, col[c], n[c], post);
      if (p.scale) load_w8<Act, kVec>(p.scale, p.w_f32, col[c], n[c], sc);
      float g[8], dg[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = row_gate;
      if (p.gate_kind == kGateFull) load8<Act, kVec>(p.gate, at + col[c], n[c], g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = z[c][i] * Z;
        const float ae = p.alpha * e[c][i];
        s_c[c][i] = fmaf(ae * g[i], y, s_c[c][i]);
        const float b = ae * sc[i] * post[i];
        dg[i] = b * y;
        t[0] += p.gate_kind == kGateFull ? dg[i] * g[i] : dg[i];
        e[c][i] = b * g[i];
        z[c][i] = y;
      }
      if (p.gate_kind == kGateFull) store8<Act, kVec>(p.dgate, at + col[c], n[c], dg);
    }
    float mean = 0.0f;
    if (p.post || p.gate_kind == kGateRow) {
      team_sum(t, W, team, wid, lane, buf, turn);
      if (p.gate_kind == kGateRow && wid == 0 && lane == 0)
        static_cast<float*>(p.dgate)[row] = t[0];
      mean = p.post ? t[0] * row_gate * inv_h : 0.0f;
    }
#pragma unroll
    for (int c = 0; c < kNC; ++c) {
#pragma unroll
      for (int i = 0; i < 8; ++i) e[c][i] = Z * fmaf(-z[c][i], mean, e[c][i]);
      store8<Act, kVec>(p.dz, at + col[c], n[c], e[c]);
    }
  }
  // the CTA's column sums: its teams' in turn, through shared memory
  if (teams == 1) {
#pragma unroll
    for (int c = 0; c < kNC; ++c) {
      if (n[c] > 0) {
        float* dst = p.part + (int64_t)blockIdx.x * 2 * H + col[c];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < n[c]) {
            dst[i] = s_pre[c][i];
            dst[H + i] = s_c[c][i];
          }
      }
    }
    return;
  }
  __shared__ float sum[2][kNormThreads * 8];
  for (int t = 0; t < teams; ++t) {
    if (team == t) {
#pragma unroll
      for (int c = 0; c < kNC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < n[c]) {
            const int h = col[c] + i;
            sum[0][h] = s_pre[c][i] + (t > 0 ? sum[0][h] : 0.0f);
            sum[1][h] = s_c[c][i] + (t > 0 ? sum[1][h] : 0.0f);
          }
    }
    __syncthreads();
  }
  for (int h = threadIdx.x; h < H; h += blockDim.x) {
    p.part[(int64_t)blockIdx.x * 2 * H + h] = sum[0][h];
    p.part[(int64_t)blockIdx.x * 2 * H + H + h] = sum[1][h];
  }
}

struct ColumnArgs {
  const float* part;
  int32_t parts, H, w_f32;
  const void* post;
  const void* scale;
  float* dpre;
  float* dpost;
  float* dscale;
};

// Sums of the CTAs' column sums, in a fixed order: 32 columns x 8 strands.
template <typename Act>
__global__ void __launch_bounds__(256) block_norm_columns_kernel(const ColumnArgs p) {
  __shared__ float sh[2][8][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int h = blockIdx.x * 32 + x;
  float a = 0.0f, b = 0.0f;
  if (h < p.H) {
    for (int i = y; i < p.parts; i += 8) {
      a += p.part[(int64_t)i * 2 * p.H + h];
      b += p.part[(int64_t)i * 2 * p.H + p.H + h];
    }
  }
  sh[0][y][x] = a;
  sh[1][y][x] = b;
  __syncthreads();
  if (y != 0 || h >= p.H) return;
  for (int i = 1; i < 8; ++i) {
    a += sh[0][i][x];
    b += sh[1][i][x];
  }
  auto weight = [&](const void* w) {
    if (w == nullptr) return 1.0f;
    return p.w_f32 ? static_cast<const float*>(w)[h] : to_f<Act>(static_cast<const Act*>(w)[h]);
  };
  if (p.dpre) p.dpre[h] = a;
  if (p.dpost) p.dpost[h] = b * weight(p.scale);
  if (p.dscale) p.dscale[h] = b * weight(p.post);
}

struct Plan {
  int nc, team_warps, teams, threads;
};

// Columns per thread (8 nc) and warps per row: a row within 4096 columns is
// spread over up to 16 warps with 8 columns a thread; wider rows take 16 or
// 32 columns a thread. Narrow rows share a CTA of 8 warps.
Plan plan_of(int H) {
  Plan q;
  const int chunks = (H + 7) / 8;
  q.nc = chunks <= kNormThreads ? 1 : chunks <= 2 * kNormThreads ? 2 : 4;
  q.team_warps = (chunks + 32 * q.nc - 1) / (32 * q.nc);
  q.teams = q.team_warps <= 4 ? kTeamsMax / q.team_warps : 1;
  q.threads = 32 * q.team_warps * q.teams;
  return q;
}

template <typename F>
cudaError_t by_types(int res, int act, F&& f) {
  auto act_is = [&](auto r) {
    using R = decltype(r);
    if (act == MOE_BF16) return f(r, __nv_bfloat16{});
    if (act == MOE_FP16) return f(r, __half{});
    if constexpr (std::is_same_v<R, float>) return f(r, float{});
    return cudaErrorInvalidValue;
  };
  if (res == MOE_FP32) return act_is(float{});
  if (res == MOE_BF16 && act == MOE_BF16) return f(__nv_bfloat16{}, __nv_bfloat16{});
  if (res == MOE_FP16 && act == MOE_FP16) return f(__half{}, __half{});
  return cudaErrorInvalidValue;
}

template <typename F>
cudaError_t by_plan(const Plan& q, bool vec, F&& f) {
  using std::integral_constant;
  auto go = [&](auto v) {
    if (q.nc == 1) return f(integral_constant<int, 1>{}, v);
    if (q.nc == 2) return f(integral_constant<int, 2>{}, v);
    return f(integral_constant<int, 4>{}, v);
  };
  return vec ? go(std::true_type{}) : go(std::false_type{});
}

// CTAs that are resident together on the whole device, by CTA size
template <typename K>
struct Resident {
  std::atomic<int> by_warps[kNormThreads / 32 + 1] = {};
  int get(K kernel, int threads, int sms) {
    std::atomic<int>& known = by_warps[threads / 32];
    int per = known.load(std::memory_order_relaxed);
    if (per == 0) {
      if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, 0) != cudaSuccess ||
          per < 1)
        per = 1;
      known.store(per, std::memory_order_relaxed);
    }
    return per * sms;
  }
};

bool norm_vec(const NormArgs& a) {
  const void* const all[] = {a.x, a.z, a.pre, a.post, a.scale, a.r, a.u, a.dr, a.du, a.dx, a.dz,
                             a.gate_kind == kGateFull ? a.gate : nullptr,
                             a.gate_kind == kGateFull ? a.dgate : nullptr};
  for (const void* q : all)
    if (!aligned(q, 16)) return false;
  return a.H % 8 == 0;
}

}  // namespace

}  // namespace moe

using namespace moe;

static int norm_args(int64_t T, int32_t H, int32_t res_type, int32_t act_type, int32_t w_type,
                     int32_t gate_kind, float eps) {
  if (T < 0 || H < 1 || H > MOE_BLOCK_NORM_MAX_H || T > (1ll << 40) / H) return MOE_ERR_SHAPE;
  if (act_type < MOE_BF16 || act_type > MOE_FP32) return MOE_ERR_SHAPE;
  if (res_type != act_type && res_type != MOE_FP32) return MOE_ERR_SHAPE;
  if (w_type != act_type && w_type != MOE_FP32) return MOE_ERR_SHAPE;
  if (gate_kind < kGateNone || gate_kind > kGateFull) return MOE_ERR_SHAPE;
  if (!(eps >= 0.0f)) return MOE_ERR_SHAPE;
  return MOE_OK;
}

static bool elements_aligned(const void* p, int type) { return aligned(p, type == MOE_FP32 ? 4 : 2); }

extern "C" {

int moe_block_norm(int64_t T, int32_t H, int32_t res_type, int32_t act_type, int32_t w_type,
                   int32_t gate_kind, float alpha, float eps, const void* x, const void* z,
                   const void* gate, const void* pre, const void* post, const void* scale, void* r,
                   void* u, void* stream) {
  const int bad = norm_args(T, H, res_type, act_type, w_type, gate_kind, eps);
  if (bad != MOE_OK) return bad;
  if (T == 0) return MOE_OK;  // nothing to do; empty tensors may carry NULL
  if (!z && (gate_kind != kGateNone || post || scale)) return MOE_ERR_SHAPE;
  if (!z && !pre) return MOE_ERR_SHAPE;
  if (!x || (z && !r) || (pre && !u) || (gate_kind != kGateNone && !gate)) return MOE_ERR_NULL;
  const int gate_type = gate_kind == kGateRow ? (int)MOE_FP32 : act_type;
  if (!elements_aligned(x, res_type) || !elements_aligned(r, res_type) ||
      !elements_aligned(z, act_type) || !elements_aligned(u, act_type) ||
      !elements_aligned(gate, gate_type) || !elements_aligned(pre, w_type) ||
      !elements_aligned(post, w_type) || !elements_aligned(scale, w_type))
    return MOE_ERR_ALIGN;
  NvtxRange range("moe_block_norm");
  NormArgs a{};
  a.x = x;
  a.z = z;
  a.gate = gate;
  a.pre = pre;
  a.post = post;
  a.scale = scale;
  a.r = z ? r : nullptr;
  a.u = pre ? u : nullptr;
  a.T = T;
  a.H = H;
  a.gate_kind = gate_kind;
  a.w_f32 = w_type == MOE_FP32;
  a.alpha = alpha;
  a.eps = eps;
  const Plan q = plan_of(H);
  a.team_warps = q.team_warps;
  const cudaError_t e = by_types(res_type, act_type, [&](auto res, auto act) {
    using Res = decltype(res);
    using Act = decltype(act);
    return by_plan(q, norm_vec(a), [&](auto nc, auto vec) {
      auto* kernel = block_norm_kernel<Res, Act, decltype(nc)::value, decltype(vec)::value>;
      static Resident<decltype(kernel)> resident;
      const int all = resident.get(kernel, q.threads, moe_device_sm_count());
      const int64_t need = (T + q.teams - 1) / q.teams;
      kernel<<<(unsigned)(need < all ? need : all), q.threads, 0,
               static_cast<cudaStream_t>(stream)>>>(a);
      return cudaGetLastError();
    });
  });
  return cuda_status(e);
}

size_t moe_block_norm_backward_workspace_size(int32_t H) {
  if (H < 1 || H > MOE_BLOCK_NORM_MAX_H) return 0;
  return (size_t)kMaxParts * 2 * (size_t)H * sizeof(float);
}

int moe_block_norm_backward(int64_t T, int32_t H, int32_t res_type, int32_t act_type,
                            int32_t w_type, int32_t gate_kind, float alpha, float eps,
                            const void* r, const void* z, const void* gate, const void* pre,
                            const void* post, const void* scale, const void* dr, const void* du,
                            void* dx, void* dz, void* dgate, float* dpre, float* dpost,
                            float* dscale, void* ws, size_t ws_bytes, void* stream) {
  const int bad = norm_args(T, H, res_type, act_type, w_type, gate_kind, eps);
  if (bad != MOE_OK) return bad;
  if (T > 0 && !z && (gate_kind != kGateNone || post || scale || !pre)) return MOE_ERR_SHAPE;
  if ((pre && !dpre) || (post && !dpost) || (scale && !dscale)) return MOE_ERR_NULL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) {  // no rows (their tensors may carry NULL): zero weight gradients
    cudaError_t e = cudaSuccess;
    if (pre) e = cudaMemsetAsync(dpre, 0, (size_t)H * 4, s);
    if (post && e == cudaSuccess) e = cudaMemsetAsync(dpost, 0, (size_t)H * 4, s);
    if (scale && e == cudaSuccess) e = cudaMemsetAsync(dscale, 0, (size_t)H * 4, s);
    return cuda_status(e);
  }
  if (!ws || (!dr && !pre)) return MOE_ERR_NULL;
  if (pre && (!r || !du || !dx)) return MOE_ERR_NULL;
  if (z && !dz) return MOE_ERR_NULL;
  if (gate_kind != kGateNone && (!gate || !dgate)) return MOE_ERR_NULL;
  const int gate_type = gate_kind == kGateRow ? (int)MOE_FP32 : act_type;
  if (!elements_aligned(r, res_type) || !elements_aligned(dr, res_type) ||
      !elements_aligned(dx, res_type) || !elements_aligned(z, act_type) ||
      !elements_aligned(du, act_type) || !elements_aligned(dz, act_type) ||
      !elements_aligned(gate, gate_type) || !elements_aligned(dgate, gate_type) ||
      !elements_aligned(pre, w_type) || !elements_aligned(post, w_type) ||
      !elements_aligned(scale, w_type) || !aligned(dpre, 4) || !aligned(dpost, 4) ||
      !aligned(dscale, 4) || !aligned(ws, 256))
    return MOE_ERR_ALIGN;
  if (ws_bytes < moe_block_norm_backward_workspace_size(H)) return MOE_ERR_WORKSPACE;
  NvtxRange range("moe_block_norm_backward");
  NormArgs a{};
  a.x = pre ? r : nullptr;
  a.z = z;
  a.gate = gate;
  a.pre = pre;
  a.post = post;
  a.scale = scale;
  a.dr = dr;
  a.du = pre ? du : nullptr;
  a.dx = pre ? dx : nullptr;
  a.dz = z ? dz : nullptr;
  a.dgate = dgate;
  a.T = T;
  a.H = H;
  a.gate_kind = gate_kind;
  a.w_f32 = w_type == MOE_FP32;
  a.alpha = alpha;
  a.eps = eps;
  a.part = static_cast<float*>(ws);
  const Plan q = plan_of(H);
  a.team_warps = q.team_warps;
  const cudaError_t e = by_types(res_type, act_type, [&](auto res, auto act) {
    using Res = decltype(res);
    using Act = decltype(act);
    return by_plan(q, norm_vec(a), [&](auto nc, auto vec) {
      auto* kernel = block_norm_backward_kernel<Res, Act, decltype(nc)::value,
                                                decltype(vec)::value>;
      static Resident<decltype(kernel)> resident;
      const int all = resident.get(kernel, q.threads, moe_device_sm_count());
      int64_t grid = (T + q.teams - 1) / q.teams;
      if (grid > all) grid = all;
      if (grid > kMaxParts) grid = kMaxParts;
      kernel<<<(unsigned)grid, q.threads, 0, s>>>(a);
      const cudaError_t r1 = cudaGetLastError();
      if (r1 != cudaSuccess || (!pre && !post && !scale)) return r1;
      const ColumnArgs c{a.part, (int32_t)grid, H, a.w_f32, post, scale,
                         pre ? dpre : nullptr, post ? dpost : nullptr, scale ? dscale : nullptr};
      block_norm_columns_kernel<Act><<<(H + 31) / 32, 256, 0, s>>>(c);
      return cudaGetLastError();
    });
  });
  return cuda_status(e);
}

}  // extern "C"
