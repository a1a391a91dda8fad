// Norms before and after a block, with its gate and residual scale, and their
// gradients: the Transformer block around the layer ("DeepSeek-V3:
// Auxiliary-Loss-Free MoE Load Balancing, ...").
//
//   N(v; w) = v * rsqrt(mean(v^2) + eps) * w
//   r = x + alpha * scale * gate * N(z; post)     u = N(r; pre)
//
// One pass over the rows: a team of warps holds a row on the SM, so x and
// z are read once and r and u written once, whatever the number of norms.
// The backward recomputes both statistics from the rows it has to read
// anyway (one more term in a reduction it needs for the gradient), so the
// forward saves nothing. All arithmetic is fp32; r is rounded when it is
// stored, and u is computed from the unrounded row.
//
// A few operations per byte, so HBM is the floor; what bounds it is the
// latency of the row sums (two in the forward, which takes two rows a step;
// three phases in the backward, one row a team at a time). 4096 rows of 7168
// in bf16, x and z to r and u: 47 us, 77% of the copy rate; backward of
// 16384 rows with an fp32 residual stream: 492 to 498 us, 66%. Odd widths go
// element by element and are bound by instructions: 777 rows of 1409 in fp16,
// backward, 17 us (floor 2.7).
#include <type_traits>

#include "kernels.cuh"

namespace moe {

namespace {

constexpr int kNormThreads = 896;  // most threads of a CTA (with 8 columns a thread)
constexpr int kBackThreads = 512;  // and of the kernels that hold more in registers
constexpr int kMaxParts = 1024;     // partial column sums
constexpr size_t kRing = 208 * 1024;
constexpr int kMaxStages = 6;       // rows asked for ahead, per team

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
  int32_t stages;     // vector form: rows in the ring
  float alpha, eps;
  // backward
  const void* dr;     // Res
  const void* du;     // Act
  void* dx;           // Res
  void* dz;           // Act
  void* dgate;        // float [T] or Act [T, H]
  float* part;        // [parts, 2, H]
};

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

// Two fp32 values in a register pair: two-lane multiplies and FMAs (each lane
// rounded once) halve the instructions of these row loops, which a few warps
// per scheduler could not issue fast enough one by one.
typedef uint64_t F2;
MOE_DEV F2 pack2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
MOE_DEV F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
MOE_DEV F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
MOE_DEV float lanes_sum(F2 a) {
  float lo, hi;
  unpack_f32x2(a, lo, hi);
  return lo + hi;
}

// 8 packed elements to and from fp32 pairs
template <typename T>
MOE_DEV void unpack8(const uint32_t (&w)[sizeof(T) * 2], F2 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (std::is_same_v<T, float>) {
      v[i] = pack2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    } else if constexpr (std::is_same_v<T, __half>) {
      v[i] = pack2(__half2float(__ushort_as_half((unsigned short)(w[i] & 0xFFFFu))),
                   __half2float(__ushort_as_half((unsigned short)(w[i] >> 16))));
    } else {
      v[i] = pack2(bf16_lo(w[i]), bf16_hi(w[i]));
    }
  }
}
template <typename T>
MOE_DEV void pack8(const F2 (&v)[4], uint32_t (&w)[sizeof(T) * 2]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    unpack_f32x2(v[i], lo, hi);
    if constexpr (std::is_same_v<T, float>) {
      w[2 * i] = __float_as_uint(lo);
      w[2 * i + 1] = __float_as_uint(hi);
    } else if constexpr (std::is_same_v<T, __half>) {
      w[i] = (uint32_t)__half_as_ushort(__float2half_rn(lo)) |
             ((uint32_t)__half_as_ushort(__float2half_rn(hi)) << 16);
    } else {
      w[i] = pack_bf16x2(lo, hi);
    }
  }
}

// A thread's 8 columns of one chunk. kVec: consecutive (n is 0 or 8; 16-byte
// accesses); otherwise `stride` columns apart, so that a warp's accesses are
// consecutive, and the first n of them exist.
template <typename T, bool kVec>
MOE_DEV void load8(const void* base, int64_t at, int n, int stride, F2 (&v)[4]) {
  const T* p = static_cast<const T*>(base) + at;
  if constexpr (kVec) {
    uint32_t w[sizeof(T) * 2] = {};
    if (n > 0) {
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
        const uint4 q = reinterpret_cast<const uint4*>(p)[i];
        w[4 * i] = q.x; w[4 * i + 1] = q.y; w[4 * i + 2] = q.z; w[4 * i + 3] = q.w;
      }
    }
    unpack8<T>(w, v);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = pack2(2 * i < n ? to_f<T>(p[2 * i * stride]) : 0.0f,
                   2 * i + 1 < n ? to_f<T>(p[(2 * i + 1) * stride]) : 0.0f);
  }
}

template <typename T, bool kVec>
MOE_DEV void store8(void* base, int64_t at, int n, int stride, const F2 (&v)[4]) {
  T* p = static_cast<T*>(base) + at;
  if constexpr (kVec) {
    if (n > 0) {
      uint32_t w[sizeof(T) * 2];
      pack8<T>(v, w);
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i)
        reinterpret_cast<uint4*>(p)[i] =
            make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo, hi;
      unpack_f32x2(v[i], lo, hi);
      if (2 * i < n) p[2 * i * stride] = from_f<T>(lo);
      if (2 * i + 1 < n) p[(2 * i + 1) * stride] = from_f<T>(hi);
    }
  }
}

template <typename Act, bool kVec>
MOE_DEV void load_w8(const void* w, bool f32, int at, int n, int stride, F2 (&v)[4]) {
  if (f32) load8<float, kVec>(w, at, n, stride, v);
  else load8<Act, kVec>(w, at, n, stride, v);
}

// One row tensor in the ring: every thread asks for its own columns of the
// rows ahead with asynchronous 16-byte copies into slots that only it reads,
// so waiting for its own copies is enough and no barrier guards the ring.
// A slot is read as often as wanted until the row is done, which keeps the
// row out of registers across the row sums.
template <typename T>
struct Slot {
  uint32_t base;  // this thread's first 16-byte slot of the tensor in stage 0
  static constexpr int pieces = sizeof(T) / 2;
  static constexpr int bytes(int threads, int nc) { return threads * nc * 8 * (int)sizeof(T); }
  MOE_DEV void ask(const void* g, int64_t at, int c, uint32_t stage) const {
    const T* p = static_cast<const T*>(g) + at;
#pragma unroll
    for (int j = 0; j < pieces; ++j)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                       base + stage + (uint32_t)((c * pieces + j) * blockDim.x * 16)),
                   "l"(p + j * (16 / sizeof(T)))
                   : "memory");
  }
  MOE_DEV void put(int c, const F2 (&v)[4]) const {
    uint32_t w[sizeof(T) * 2];
    pack8<T>(v, w);
#pragma unroll
    for (int j = 0; j < pieces; ++j)
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                       base + (uint32_t)((c * pieces + j) * blockDim.x * 16)),
                   "r"(w[4 * j]), "r"(w[4 * j + 1]), "r"(w[4 * j + 2]), "r"(w[4 * j + 3])
                   : "memory");
  }
  MOE_DEV void get(int c, uint32_t stage, F2 (&v)[4]) const {
    uint32_t w[sizeof(T) * 2];
#pragma unroll
    for (int j = 0; j < pieces; ++j)
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[4 * j]), "=r"(w[4 * j + 1]), "=r"(w[4 * j + 2]), "=r"(w[4 * j + 3])
                   : "r"(base + stage + (uint32_t)((c * pieces + j) * blockDim.x * 16))
                   : "memory");
    unpack8<T>(w, v);
  }
};

MOE_DEV void ask_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// this thread's copies have landed, but for the youngest `n` groups
MOE_DEV void ask_wait(int n) {
  switch (n) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
  }
}

// Where a thread stands: its team (the warps that share a row) and columns.
template <int kNC, bool kVec>
struct Place {
  int W, team, wid, lane, teams, stride, H;
  int col[kNC], n[kNC];
  MOE_DEV explicit Place(const NormArgs& p) {
    W = p.team_warps;
    H = p.H;
    lane = threadIdx.x & 31;
    team = (threadIdx.x >> 5) / W;
    wid = (threadIdx.x >> 5) - team * W;
    teams = (blockDim.x >> 5) / W;
    stride = kVec ? 1 : W * 32;
    const int me = wid * 32 + lane;
#pragma unroll
    for (int c = 0; c < kNC; ++c) {
      if (kVec) {
        col[c] = (c * W * 32 + me) * 8;
        n[c] = col[c] < H ? 8 : 0;
      } else {
        col[c] = c * 8 * stride + me;
        n[c] = min(max((H - col[c] + stride - 1) / stride, 0), 8);
      }
    }
  }
  MOE_DEV int64_t first() const { return (int64_t)blockIdx.x * teams + team; }
  MOE_DEV int64_t step() const { return (int64_t)gridDim.x * teams; }
};

typedef float TeamBuf[2][3][32];

// Sums over a team of warps. Two buffers in turn: a thread writes one again
// only after a barrier that every reader of its last use has passed.
template <int kN, typename P>
MOE_DEV void team_sum(float (&v)[kN], const P& at, TeamBuf& buf, int& turn) {
#pragma unroll
  for (int i = 0; i < kN; ++i)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (at.W == 1) return;
  if (at.lane == 0) {
#pragma unroll
    for (int i = 0; i < kN; ++i) buf[turn][i][at.team * at.W + at.wid] = v[i];
  }
  asm volatile("bar.sync %0, %1;" ::"r"(at.teams == 1 ? 0 : 1 + at.team), "r"(at.W * 32) : "memory");
  // the warps' sums, one to a lane, added in a tree: the same in every warp
#pragma unroll
  for (int i = 0; i < kN; ++i) v[i] = at.lane < at.W ? buf[turn][i][at.team * at.W + at.lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  turn ^= 1;
}

// alpha * post * scale of a thread's columns (absent weights are 1, columns
// beyond the row anything finite: their values are zeros)
template <typename Act, int kNC, bool kVec>
MOE_DEV void branch_weights(const NormArgs& p, const Place<kNC, kVec>& at, F2 (&wq)[kNC][4]) {
#pragma unroll
  for (int c = 0; c < kNC; ++c) {
    F2 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) wq[c][i] = pack2(p.alpha, p.alpha);
    if (p.post) {
      load_w8<Act, kVec>(p.post, p.w_f32, at.col[c], at.n[c], at.stride, w);
#pragma unroll
      for (int i = 0; i < 4; ++i) wq[c][i] = mul2(wq[c][i], w[i]);
    }
    if (p.scale) {
      load_w8<Act, kVec>(p.scale, p.w_f32, at.col[c], at.n[c], at.stride, w);
#pragma unroll
      for (int i = 0; i < 4; ++i) wq[c][i] = mul2(wq[c][i], w[i]);
    }
  }
}

template <typename Act, int kNC, bool kVec>
MOE_DEV void pre_weights(const NormArgs& p, const Place<kNC, kVec>& at, F2 (&w)[kNC][4]) {
#pragma unroll
  for (int c = 0; c < kNC; ++c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[c][i] = 0ull;
    if (p.pre) load_w8<Act, kVec>(p.pre, p.w_f32, at.col[c], at.n[c], at.stride, w[c]);
  }
}

// kR rows a step: their sums meet at the same barriers, which leaves half of
// the waiting of one row a step.
template <typename Res, typename Act, int kNC, int kR, bool kVec>
__global__ void __launch_bounds__(kNC == 1 ? kNormThreads : kBackThreads, 1)
    block_norm_kernel(const NormArgs p) {
  __shared__ TeamBuf buf;
  extern __shared__ __align__(16) uint8_t ring[];
  const Place<kNC, kVec> at(p);
  const float inv_h = 1.0f / (float)p.H;
  const bool full = p.gate_kind == kGateFull;
  int turn = 0;
  const Slot<Res> sx{smem_u32(ring) + threadIdx.x * 16};
  const Slot<Act> sz{sx.base + Slot<Res>::bytes(blockDim.x, kNC)};
  const Slot<Act> sg{sz.base + Slot<Act>::bytes(blockDim.x, kNC)};
  const uint32_t row_bytes = (uint32_t)(Slot<Res>::bytes(blockDim.x, kNC) +
                                        (p.z ? Slot<Act>::bytes(blockDim.x, kNC) : 0) +
                                        (full ? Slot<Act>::bytes(blockDim.x, kNC) : 0));
  const uint32_t stage_bytes = kR * row_bytes;
  // the kR rows of step i: i * step() apart, side by side over the teams
  const int64_t step = at.step();
  auto ask = [&](int64_t row, int s) {
#pragma unroll
    for (int q = 0; q < kR; ++q, row += step) {
      if (row >= p.T) break;
#pragma unroll
      for (int c = 0; c < kNC; ++c) {
        if (at.n[c] == 0) continue;
        const int64_t e = row * p.H + at.col[c];
        const uint32_t stage = s * stage_bytes + q * row_bytes;
        if (p.z) sz.ask(p.z, e, c, stage);
        sx.ask(p.x, e, c, stage);
        if (full) sg.ask(p.gate, e, c, stage);
      }
    }
    ask_commit();
  };
  if (kVec)
    for (int s = 0; s < p.stages - 1; ++s) ask(at.first() + s * kR * step, s);
  F2 pre[kNC][4], wq[kNC][4];
  pre_weights<Act>(p, at, pre);
  if (p.z) branch_weights<Act>(p, at, wq);
  int slot = 0;
  for (int64_t row = at.first(); row < p.T; row += kR * step) {
    const uint32_t stage = slot * stage_bytes;
    float gate[kR], s[kR];
#pragma unroll
    for (int q = 0; q < kR; ++q) {
      gate[q] = 1.0f;
      s[q] = 0.0f;
      if (p.gate_kind == kGateRow && row + q * step < p.T)
        gate[q] = static_cast<const float*>(p.gate)[row + q * step];
    }
    if (kVec) {
      const int ahead = p.stages - 1;
      ask(row + ahead * kR * step, slot + ahead < p.stages ? slot + ahead : slot - 1);
      ask_wait(ahead);
      slot = slot + 1 == p.stages ? 0 : slot + 1;
    }
    // columns beyond the row, and rows beyond the last, hold zeros throughout
    auto here = [&](int q, int c) { return at.n[c] > 0 && (kR == 1 || row + q * step < p.T); };
    auto get_x = [&](int q, int c, F2 (&v)[4]) {
      if (kVec) sx.get(c, stage + q * row_bytes, v);
      else load8<Res, kVec>(p.x, (row + q * step) * p.H + at.col[c], at.n[c], at.stride, v);
    };
    auto get_act = [&](const Slot<Act>& sl, const void* g, int q, int c, F2 (&v)[4]) {
      if (kVec) sl.get(c, stage + q * row_bytes, v);
      else load8<Act, kVec>(g, (row + q * step) * p.H + at.col[c], at.n[c], at.stride, v);
    };
    if (p.post) {
#pragma unroll
      for (int q = 0; q < kR; ++q) {
        F2 sum = 0ull;
#pragma unroll
        for (int c = 0; c < kNC; ++c) {
          if (!here(q, c)) continue;
          F2 z[4];
          get_act(sz, p.z, q, c, z);
#pragma unroll
          for (int i = 0; i < 4; ++i) sum = fma2(z[i], z[i], sum);
        }
        s[q] = lanes_sum(sum);
      }
      team_sum(s, at, buf, turn);
#pragma unroll
      for (int q = 0; q < kR; ++q) gate[q] *= rsqrtf(fmaf(s[q], inv_h, p.eps));
    }
    F2 r[kR][kNC][4];
#pragma unroll
    for (int q = 0; q < kR; ++q) {
      F2 sum = 0ull;
      const F2 g2 = pack2(gate[q], gate[q]);
#pragma unroll
      for (int c = 0; c < kNC; ++c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) r[q][c][i] = 0ull;
        if (!here(q, c)) continue;
        get_x(q, c, r[q][c]);
        if (p.z) {
          F2 z[4];
          get_act(sz, p.z, q, c, z);
          if (full) {
            F2 g[4];
            get_act(sg, p.gate, q, c, g);
#pragma unroll
            for (int i = 0; i < 4; ++i) z[i] = mul2(z[i], g[i]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) r[q][c][i] = fma2(mul2(g2, z[i]), wq[c][i], r[q][c][i]);
          store8<Res, kVec>(p.r, (row + q * step) * p.H + at.col[c], at.n[c], at.stride, r[q][c]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) sum = fma2(r[q][c][i], r[q][c][i], sum);
      }
      s[q] = lanes_sum(sum);
    }
    if (!p.pre) continue;
    team_sum(s, at, buf, turn);
#pragma unroll
    for (int q = 0; q < kR; ++q) {
      const float f = rsqrtf(fmaf(s[q], inv_h, p.eps));
      const F2 f2 = pack2(f, f);
#pragma unroll
      for (int c = 0; c < kNC; ++c) {
        if (!here(q, c)) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) r[q][c][i] = mul2(r[q][c][i], mul2(f2, pre[c][i]));
        store8<Act, kVec>(p.u, (row + q * step) * p.H + at.col[c], at.n[c], at.stride, r[q][c]);
      }
    }
  }
}

// The backward. With h = r R (R = rsqrt(mean r^2 + eps)) and y = z Z:
//   e  = dr + R (du pre - h mean(du pre h))          dx = e
//   q  = alpha scale gate e
//   dz = Z (q post - y mean(q post y))               (without post: dz = q)
//   dpre = sum_t du h;  c = sum_t gate e y;          dpost = alpha scale c;
//   dscale = alpha post c;   dgate = alpha scale post y e (summed over the row)
// Two rounds of row sums: (r^2, du pre r, z^2), then w z e with w = alpha
// scale post, which gives both the row's gate gradient and the mean in dz.
// Each thread keeps its columns' sums over the rows of its CTA in registers;
// the CTAs' sums are added in a fixed order by a second kernel.
template <typename Res, typename Act, int kNC, bool kVec, bool kFull>
__global__ void __launch_bounds__(kBackThreads, 1) block_norm_backward_kernel(const NormArgs p) {
  __shared__ TeamBuf buf;
  extern __shared__ __align__(16) uint8_t ring[];
  const Place<kNC, kVec> at(p);
  const int H = p.H;
  const float inv_h = 1.0f / (float)H;
  int turn = 0;
  F2 s_pre[kNC][4], s_c[kNC][4];
#pragma unroll
  for (int c = 0; c < kNC; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) s_pre[c][i] = s_c[c][i] = 0ull;

  const uint32_t act_bytes = Slot<Act>::bytes(blockDim.x, kNC);
  const uint32_t res_bytes = Slot<Res>::bytes(blockDim.x, kNC);
  uint32_t next = smem_u32(ring) + threadIdx.x * 16;
  // the first norm's weights stand in slots too: registers are short
  const Slot<float> sw{next};
  next += Slot<float>::bytes(blockDim.x, kNC);
  const uint32_t ring0 = next;
  const Slot<Res> sr{next};
  if (p.pre) next += res_bytes;
  const Slot<Res> sd{next};
  if (p.dr) next += res_bytes;
  const Slot<Act> su{next};
  if (p.pre) next += act_bytes;
  const Slot<Act> sz{next};
  if (p.z) next += act_bytes;
  const Slot<Act> sg{next};
  if (kFull) next += act_bytes;
  const uint32_t stage_bytes = next - ring0;
  auto ask = [&](int64_t row, int s) {
    if (row < p.T) {
#pragma unroll
      for (int c = 0; c < kNC; ++c) {
        if (at.n[c] == 0) continue;
        const int64_t e = row * H + at.col[c];
        if (p.pre) {
          sr.ask(p.x, e, c, s * stage_bytes);
          su.ask(p.du, e, c, s * stage_bytes);
        }
        if (p.z) sz.ask(p.z, e, c, s * stage_bytes);
        if (p.dr) sd.ask(p.dr, e, c, s * stage_bytes);
        if (kFull) sg.ask(p.gate, e, c, s * stage_bytes);
      }
    }
    ask_commit();
  };
  if (kVec)
    for (int s = 0; s < p.stages - 1; ++s) ask(at.first() + s * at.step(), s);
  F2 wq[kNC][4];
  pre_weights<Act>(p, at, wq);
#pragma unroll
  for (int c = 0; c < kNC; ++c) sw.put(c, wq[c]);
  branch_weights<Act>(p, at, wq);
  cudaTriggerProgrammaticLaunchCompletion();
  int slot = 0;
  for (int64_t row = at.first(); row < p.T; row += at.step()) {
    const int64_t e0 = row * H;
    const uint32_t stage = slot * stage_bytes;
    float row_gate = 1.0f;
    if (p.gate_kind == kGateRow) row_gate = static_cast<const float*>(p.gate)[row];
    if (kVec) {
      const int ahead = p.stages - 1;
      ask(row + ahead * at.step(), slot + ahead < p.stages ? slot + ahead : slot - 1);
      ask_wait(ahead);
      slot = slot + 1 == p.stages ? 0 : slot + 1;
    }
    auto get = [&](const auto& s, const void* g, int c, F2 (&v)[4]) {
      using S = std::decay_t<decltype(s)>;
      if (kVec) s.get(c, stage, v);
      else if constexpr (std::is_same_v<S, Slot<Res>>)
        load8<Res, kVec>(g, e0 + at.col[c], at.n[c], at.stride, v);
      else
        load8<Act, kVec>(g, e0 + at.col[c], at.n[c], at.stride, v);
    };
    F2 sum[3] = {0ull, 0ull, 0ull};
#pragma unroll
    for (int c = 0; c < kNC; ++c) {
      if (at.n[c] == 0) continue;
      if (p.pre) {
        F2 r[4], du[4], w[4];
        get(sr, p.x, c, r);
        get(su, p.du, c, du);
        sw.get(c, 0, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sum[0] = fma2(r[i], r[i], sum[0]);
          sum[1] = fma2(mul2(du[i], w[i]), r[i], sum[1]);
        }
      }
      if (p.post) {
        F2 z[4];
        get(sz, p.z, c, z);
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[2] = fma2(z[i], z[i], sum[2]);
      }
    }
    float s[3] = {lanes_sum(sum[0]), lanes_sum(sum[1]), lanes_sum(sum[2])};
    if (p.pre || p.post) team_sum(s, at, buf, turn);
    const float R = rsqrtf(fmaf(s[0], inv_h, p.eps));
    // of r in dx; the mean of du pre h first, since R to the third leaves fp32
    // for rows of 1e14 (or, without eps, of 1e-13)
    const float r_part = -(s[1] * inv_h * R) * R * R;
    const float Z = p.post ? rsqrtf(fmaf(s[2], inv_h, p.eps)) : 1.0f;
    F2 e[kNC][4];  // dx, then w e (times a full gate)
    F2 t2 = 0ull;
#pragma unroll
    for (int c = 0; c < kNC; ++c) {
      if (at.n[c] == 0) continue;
      if (p.dr) {
        get(sd, p.dr, c, e[c]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) e[c][i] = 0ull;
      }
      if (p.pre) {
        const F2 R2 = pack2(R, R), rp2 = pack2(r_part, r_part);
        F2 r[4], du[4], w[4];
        get(sr, p.x, c, r);
        get(su, p.du, c, du);
        sw.get(c, 0, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const F2 d = mul2(du[i], R2);
          s_pre[c][i] = fma2(d, r[i], s_pre[c][i]);
          e[c][i] = fma2(d, w[i], fma2(r[i], rp2, e[c][i]));
        }
        store8<Res, kVec>(p.dx, e0 + at.col[c], at.n[c], at.stride, e[c]);
      }
      if (!p.z) continue;
      F2 z[4];
      get(sz, p.z, c, z);
      if (kFull) {
        const F2 Z2 = pack2(Z, Z);
        F2 g[4], dg[4];
        get(sg, p.gate, c, g);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const F2 y = mul2(z[i], Z2);
          s_c[c][i] = fma2(mul2(e[c][i], g[i]), y, s_c[c][i]);
          e[c][i] = mul2(e[c][i], wq[c][i]);
          dg[i] = mul2(e[c][i], y);
          e[c][i] = mul2(e[c][i], g[i]);
          t2 = fma2(e[c][i], z[i], t2);
        }
        store8<Act, kVec>(p.dgate, e0 + at.col[c], at.n[c], at.stride, dg);
      } else {
        const F2 zg2 = pack2(Z * row_gate, Z * row_gate);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s_c[c][i] = fma2(e[c][i], mul2(z[i], zg2), s_c[c][i]);
          e[c][i] = mul2(e[c][i], wq[c][i]);
          t2 = fma2(e[c][i], z[i], t2);
        }
      }
    }
    if (!p.z) continue;
    float z_part = 0.0f;  // of z in dz
    if (p.post || p.gate_kind == kGateRow) {
      float t[1] = {lanes_sum(t2)};
      team_sum(t, at, buf, turn);
      if (p.gate_kind == kGateRow && at.wid == 0 && at.lane == 0)
        static_cast<float*>(p.dgate)[row] = t[0] * Z;
      if (p.post) z_part = -(t[0] * inv_h * Z) * (Z * row_gate) * Z;
    }
    const F2 zp2 = pack2(z_part, z_part), zg2 = pack2(Z * row_gate, Z * row_gate);
#pragma unroll
    for (int c = 0; c < kNC; ++c) {
      if (at.n[c] == 0) continue;
      F2 z[4];
      get(sz, p.z, c, z);
#pragma unroll
      for (int i = 0; i < 4; ++i) e[c][i] = fma2(e[c][i], zg2, mul2(z[i], zp2));
      store8<Act, kVec>(p.dz, e0 + at.col[c], at.n[c], at.stride, e[c]);
    }
  }
  // the CTA's column sums: each team's through shared memory, over the slots
  // (every thread has read its own; the others' are behind the barrier)
  if (kVec) ask_wait(0);
  __syncthreads();
  float* const sum = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int c = 0; c < kNC; ++c) {
    float a[8], b[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      unpack_f32x2(s_pre[c][i], a[2 * i], a[2 * i + 1]);
      unpack_f32x2(s_c[c][i], b[2 * i], b[2 * i + 1]);
    }
    float* const dst = sum + at.team * 2 * H + at.col[c];
    if (kVec) {
      if (at.n[c] > 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          reinterpret_cast<float4*>(dst)[i] =
              make_float4(a[4 * i], a[4 * i + 1], a[4 * i + 2], a[4 * i + 3]);
          reinterpret_cast<float4*>(dst + H)[i] =
              make_float4(b[4 * i], b[4 * i + 1], b[4 * i + 2], b[4 * i + 3]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < at.n[c]) {
          dst[i * at.stride] = a[i];
          dst[H + i * at.stride] = b[i];
        }
    }
  }
  __syncthreads();
  for (int h = threadIdx.x; h < 2 * H; h += blockDim.x) {
    float v = sum[h];
    for (int t = 1; t < at.teams; ++t) v += sum[t * 2 * H + h];
    p.part[(int64_t)blockIdx.x * 2 * H + h] = v;
  }
}

struct ColumnArgs {
  const float* part;
  int32_t parts, H, w_f32;
  float alpha;
  const void* post;
  const void* scale;
  float* dpre;
  float* dpost;
  float* dscale;
};

// Sums of the CTAs' column sums, in a fixed order: 32 columns x 32 strands.
template <typename Act>
__global__ void __launch_bounds__(1024) block_norm_columns_kernel(const ColumnArgs p) {
  __shared__ float sh[2][32][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  int h = blockIdx.x * 32 + x;
  float a = 0.0f, b = 0.0f;
  cudaGridDependencySynchronize();
  if (h < p.H) {
#pragma unroll 4
    for (int i = y; i < p.parts; i += 32) {
      a += p.part[(int64_t)i * 2 * p.H + h];
      b += p.part[(int64_t)i * 2 * p.H + p.H + h];
    }
  }
  sh[0][y][x] = a;
  sh[1][y][x] = b;
  __syncthreads();
  // each warp adds one column's strands
  a = sh[0][x][y];
  b = sh[1][x][y];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  h = blockIdx.x * 32 + y;
  if (x != 0 || h >= p.H) return;
  auto weight = [&](const void* w) {
    if (w == nullptr) return 1.0f;
    return p.w_f32 ? static_cast<const float*>(w)[h] : to_f<Act>(static_cast<const Act*>(w)[h]);
  };
  if (p.dpre) p.dpre[h] = a;
  if (p.dpost) p.dpost[h] = p.alpha * b * weight(p.scale);
  if (p.dscale) p.dscale[h] = p.alpha * b * weight(p.post);
}

// How rows are spread over threads, and the rows asked for ahead.
struct Plan {
  int nc, rows, team_warps, teams, threads, stages;
  bool vec;
  size_t smem;
};

// 8 columns a thread up to 7168 columns (the backward: 4096), 16 up to 8192
// and 32 above. The weights and column sums of 8 and 16 columns fit in registers
// beside the row's (but for 4 to 52 bytes in some backwards of 16); of 32 they
// do not: those backwards spill 550 to 670 bytes a thread, the forwards 40 to
// 190. One CTA per SM, with fewer teams where there are not rows
// enough for every SM's; the forward takes two rows a step where every team
// has more. per_column: bytes of the row tensors per column.
Plan plan_of(int64_t T, int H, int per_column, bool vec, int sms, bool backward) {
  Plan q;
  const int chunks = (H + 7) / 8;
  const int most1 = backward ? kBackThreads : kNormThreads;
  q.nc = chunks <= most1 ? 1 : chunks <= 2 * kBackThreads ? 2 : 4;
  // Where the backward has many rows, 16 columns a thread from 264 columns on:
  // twice the rows in flight (8192 rows of 512, 2048, 4096 columns: 16.7, 47.2,
  // 85.1 us against 18.8, 58.1, 109.1; at 148 rows 8 columns take 7.0, 7.6,
  // 9.2 against 8.4, 9.0, 9.6).
  if (backward && q.nc == 1 && chunks > 32 && T > 6 * sms) q.nc = 2;
  const int threads = q.nc == 1 ? most1 : kBackThreads;
  q.team_warps = (chunks + 32 * q.nc - 1) / (32 * q.nc);
  const int fit = threads / 32 / q.team_warps;
  // teams of more than a warp meet at a barrier of their own, of which there are 15
  const int most = q.team_warps > 1 && fit > 15 ? 15 : fit;
  const int64_t want = (T + sms - 1) / sms;
  q.teams = (int)(want < most ? want : most);
  q.threads = 32 * q.team_warps * q.teams;
  const size_t row = (size_t)q.threads * q.nc * 8 * per_column;
  q.rows = !backward && vec && T > (int64_t)q.teams * sms && 4 * row <= kRing && q.nc < 4 ? 2 : 1;
  const size_t stage = q.rows * row;
  // the backward's first weights are in shared memory as well
  const size_t fixed = backward ? (size_t)q.threads * q.nc * 8 * 4 : 0, room = kRing - fixed;
  q.vec = vec && stage <= room;
  q.stages = q.vec ? (int)(room / stage < kMaxStages ? room / stage : kMaxStages) : 0;
  q.smem = fixed + q.stages * stage;
  // the backward's column sums of the teams meet in the same memory
  const size_t sums = (size_t)q.teams * 2 * H * 4;
  if (backward && q.smem < sums) q.smem = sums;
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
cudaError_t by_plan(const Plan& q, F&& f) {
  using std::integral_constant;
  auto go = [&](auto v) {
    if (q.nc == 1) return f(integral_constant<int, 1>{}, v);
    if (q.nc == 2) return f(integral_constant<int, 2>{}, v);
    return f(integral_constant<int, 4>{}, v);
  };
  return q.vec ? go(std::true_type{}) : go(std::false_type{});
}

// the ring may take most of an SM's shared memory
template <typename K>
cudaError_t allow_smem(DeviceOnce& once, K kernel) {
  return once.run([&] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRing);
  });
}

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
  const int sms = moe_device_sm_count();
  const int res_size = res_type == MOE_FP32 ? 4 : 2, act_size = act_type == MOE_FP32 ? 4 : 2;
  const int per_column = res_size + (z ? act_size : 0) + (gate_kind == kGateFull ? act_size : 0);
  const Plan q = plan_of(T, H, per_column, norm_vec(a), sms, false);
  a.team_warps = q.team_warps;
  a.stages = q.stages;
  const cudaError_t e = by_types(res_type, act_type, [&](auto res, auto act) {
    using Res = decltype(res);
    using Act = decltype(act);
    return by_plan(q, [&](auto nc, auto vec) {
      constexpr int kNC = decltype(nc)::value;
      constexpr bool kVec = decltype(vec)::value;
      auto go = [&](auto* kernel, DeviceOnce& once) {
        const cudaError_t r0 = allow_smem(once, kernel);
        if (r0 != cudaSuccess) return r0;
        const int64_t need = (T + q.teams - 1) / q.teams;
        kernel<<<(unsigned)(need < sms ? need : sms), q.threads, q.smem,
                 static_cast<cudaStream_t>(stream)>>>(a);
        return cudaGetLastError();
      };
      static DeviceOnce once1, once2;
      if constexpr (kVec && kNC < 4) {
        if (q.rows == 2) return go(block_norm_kernel<Res, Act, kNC, 2, kVec>, once2);
      }
      return go(block_norm_kernel<Res, Act, kNC, 1, kVec>, once1);
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
  const int sms = moe_device_sm_count();
  const int res_size = res_type == MOE_FP32 ? 4 : 2, act_size = act_type == MOE_FP32 ? 4 : 2;
  const int per_column = (pre ? res_size + act_size : 0) + (dr ? res_size : 0) +
                         (z ? act_size : 0) + (gate_kind == kGateFull ? act_size : 0);
  const Plan q = plan_of(T, H, per_column, norm_vec(a), sms, true);
  a.team_warps = q.team_warps;
  a.stages = q.stages;
  const cudaError_t e = by_types(res_type, act_type, [&](auto res, auto act) {
    using Res = decltype(res);
    using Act = decltype(act);
    return by_plan(q, [&](auto nc, auto vec) {
      constexpr int kNC = decltype(nc)::value;
      constexpr bool kVec = decltype(vec)::value;
      const bool full = gate_kind == kGateFull;
      auto* kernel = full ? block_norm_backward_kernel<Res, Act, kNC, kVec, true>
                          : block_norm_backward_kernel<Res, Act, kNC, kVec, false>;
      static DeviceOnce once[2];
      const cudaError_t r0 = allow_smem(once[full], kernel);
      if (r0 != cudaSuccess) return r0;
      int64_t grid = (T + q.teams - 1) / q.teams;
      if (grid > sms) grid = sms;
      if (grid > kMaxParts) grid = kMaxParts;
      kernel<<<(unsigned)grid, q.threads, q.smem, s>>>(a);
      const cudaError_t r1 = cudaGetLastError();
      if (r1 != cudaSuccess || (!pre && !post && !scale)) return r1;
      const ColumnArgs c{a.part, (int32_t)grid, H, a.w_f32, alpha, post, scale,
                         pre ? dpre : nullptr, post ? dpost : nullptr, scale ? dscale : nullptr};
      return launch_dependent(block_norm_columns_kernel<Act>, (unsigned)((H + 31) / 32), 1024, 0, s, c);
    });
  });
  return cuda_status(e);
}

}  // extern "C"
