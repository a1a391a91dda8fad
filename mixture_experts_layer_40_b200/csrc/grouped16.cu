// Products grouped by expert in 16 bits (bf16 or fp16) with ragged groups, on
// tcgen05 tensor cores: the forward, the input gradient and the weight
// gradient of per-expert linear maps. Group g owns rows s_g .. s_g + r_g - 1
// of the row buffers, at any alignment:
//
//   forward        out[r, n] = sum_k a[r, k] W_g[n, k]     W [G, N, K]
//   input gradient out[r, n] = sum_k a[r, k] W_g[k, n]     W [G, K, N]
//   weight grad    dw_g[n, k] (+)= sum_{r in g} dy[r, n] x[r, k]
//
// 16-bit products are exact in fp32; sums are fp32 in TMEM, rounded once.
//
// The tensor cores take either operand with its reduction index fastest
// (K-major) or slowest (MN-major), so all three products read the tensors as
// they lie: no transposed copy of the weights or of the rows is made.
//
// One persistent CTA per SM, 256 threads:
//   warp 0     TMA producer: 64-deep k-blocks of A (128 rows) and B (kBN
//              columns) into a ring of shared-memory stages
//   warp 1     MMA issuer, M=128, N=kBN, K=16 into one of two TMEM buffers
//   warp 2     TMEM allocator; scans the groups into a tile prefix
//   warps 4-7  epilogue: TMEM -> registers -> global memory, while the next
//              tile's MMAs fill the other buffer
// Rows of a tile beyond its group are another group's rows or padding: each
// row of the accumulator depends on its own row of A alone, so whatever they
// hold stays in accumulator rows that are never stored. In the weight
// gradient the rows are the reduction: the last k-block's rows beyond the
// group are cleared in shared memory, in both operands (a NaN or infinity
// there would survive a product with zero), and 16-row steps past them are
// not issued.
#include <type_traits>

#include "kernels.cuh"

namespace moe {

namespace {

constexpr int kBM = 128;
constexpr int kBK = 64;
constexpr int kThreads16 = 256;
constexpr int kABytes = kBM * kBK * 2;
constexpr int kMaxGroups16 = 1025;
constexpr int kSmemBudget = 200 * 1024;

enum Way : int { kForward = 0, kInputGrad = 1, kWeightGrad = 2 };

template <int kBN>
struct Tile {
  static constexpr int b_bytes = kBN * kBK * 2;
  static constexpr int stage_bytes = kABytes + b_bytes;
  static constexpr int stages = kSmemBudget / stage_bytes < 8 ? kSmemBudget / stage_bytes : 8;
  static constexpr size_t dyn_smem = (size_t)stages * stage_bytes + 1024;
};

struct Args16 {
  const int32_t* group_rows;
  const int32_t* group_start;
  int32_t n_groups;
  int32_t kblocks;   // forward, input gradient: ceil(K / 64)
  int32_t n_tiles;   // kBN-wide column tiles per group
  int32_t m_tiles;   // weight gradient: 128-high row tiles of dw per group
  int64_t rows;      // rows of the row buffers
  int32_t M;         // weight gradient: rows of dw per group
  int32_t N;         // columns of the output
  void* out;
  int32_t out_type;  // MOE_BF16, MOE_FP16, MOE_FP32
  int32_t accumulate;
  uint32_t idesc;
  uint32_t* status;
};

struct alignas(8) Shared16 {
  uint64_t full[8];
  uint64_t empty[8];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t drained;
  uint32_t tmem_base;
  int abort;
  int prefix[kMaxGroups16 + 1];
  int rows[kMaxGroups16];
  int start[kMaxGroups16];
};

MOE_DEV void tma_load_3d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z,
                         uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// Descriptor of an MN-major tile with 128-byte swizzling, as 64-wide TMA boxes
// of kBK rows lay it out: 8 reduction rows of 128 bytes per 1024-byte group
// (the stride offset), the next 64 columns one box further (the leading
// offset).
MOE_DEV uint64_t smem_desc_mn_sw128(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)((kBK * 128) >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

struct TileAt {
  int g, m, n;
};

MOE_DEV TileAt tile_at(int tile, const int* prefix, int n_groups, int n_tiles) {
  int lo = 0, hi = n_groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if ((int64_t)prefix[mid] * n_tiles <= tile) lo = mid; else hi = mid;
  }
  const int local = tile - prefix[lo] * n_tiles;
  TileAt t;
  t.g = lo;
  t.m = local / n_tiles;
  t.n = local - t.m * n_tiles;
  return t;
}

// Group table into shared memory, by one warp: each group's rows and start
// (zero rows for a group that fails its check, which is flagged), and the
// running number of row tiles. Starts must ascend without overlap, so that no
// row of the output has two writers.
MOE_DEV void scan_groups(const Args16& p, Shared16& sh, int lane, bool weight_grad) {
  int carry = 0;
  int64_t end = 0;
  if (lane == 0) sh.prefix[0] = 0;
  for (int base = 0; base < p.n_groups; base += 32) {
    const int g = base + lane;
    int r = 0, st = 0;
    if (g < p.n_groups) {
      r = p.group_rows[g];
      st = p.group_start[g];
    }
    bool ok = r >= 0 && (r == 0 || (st >= 0 && (int64_t)st + r <= p.rows));
    // the largest end before this group
    int64_t upto = ok && r > 0 ? (int64_t)st + r : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o && v > upto) upto = v;
    }
    int64_t before = __shfl_up_sync(0xffffffffu, upto, 1);
    if (lane == 0 || before < end) before = end;
    ok = ok && (r == 0 || st >= before);
    if (!ok) {
      flag_status(p.status, kStatusBounds);
      r = 0;
    }
    const int64_t last = __shfl_sync(0xffffffffu, upto, 31);
    if (last > end) end = last;
    const int mt = weight_grad ? (g < p.n_groups ? p.m_tiles : 0) : (r + kBM - 1) / kBM;
    int incl = mt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (g < p.n_groups) {
      sh.rows[g] = r;
      sh.start[g] = st;
      sh.prefix[g + 1] = carry + incl;
    }
    carry += __shfl_sync(0xffffffffu, incl, 31);
  }
}

MOE_DEV uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

MOE_DEV void unpack16(uint32_t w, bool f16, float& lo, float& hi) {
  if (f16) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    lo = f.x;
    hi = f.y;
  } else {
    lo = bf16_lo(w);
    hi = bf16_hi(w);
  }
}

// 8 consecutive output columns of one row; added to what is there first when
// accumulating
MOE_DEV void store8(const Args16& p, int64_t at, const float* v) {
  if (p.out_type == MOE_FP32) {
    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.out) + at);
    float4 a = make_float4(v[0], v[1], v[2], v[3]), b = make_float4(v[4], v[5], v[6], v[7]);
    if (p.accumulate) {
      const float4 c = dst[0], d = dst[1];
      a.x += c.x; a.y += c.y; a.z += c.z; a.w += c.w;
      b.x += d.x; b.y += d.y; b.z += d.z; b.w += d.w;
    }
    dst[0] = a;
    dst[1] = b;
    return;
  }
  const bool f16 = p.out_type == MOE_FP16;
  uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at);
  float o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = v[i];
  if (p.accumulate) {
    const uint4 c = *dst;
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo, hi;
      unpack16(w[i], f16, lo, hi);
      o[2 * i] += lo;
      o[2 * i + 1] += hi;
    }
  }
  *dst = f16 ? make_uint4(pack_f16x2(o[0], o[1]), pack_f16x2(o[2], o[3]), pack_f16x2(o[4], o[5]),
                          pack_f16x2(o[6], o[7]))
             : make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]),
                          pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7]));
}

template <int kWay, int kBN>
__global__ void __launch_bounds__(kThreads16, 1)
    grouped16_kernel(const __grid_constant__ CUtensorMap tm_a,
                     const __grid_constant__ CUtensorMap tm_a32,
                     const __grid_constant__ CUtensorMap tm_b, const Args16 p) {
  using C = Tile<kBN>;
  constexpr bool kWgrad = kWay == kWeightGrad;
  __shared__ Shared16 sh;
  extern __shared__ uint8_t dyn_smem[];
  const uint32_t ring = (smem_u32(dyn_smem) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::stages; ++s) {
      mbar_init(smem_u32(&sh.full[s]), 1);
      mbar_init(smem_u32(&sh.empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&sh.tfull[b]), 1);
      mbar_init(smem_u32(&sh.tempty[b]), 4);
    }
    mbar_init(smem_u32(&sh.drained), 1);
    sh.abort = 0;
    fence_mbar_init();
    prefetch_tensormap(&tm_a);
    prefetch_tensormap(&tm_a32);
    prefetch_tensormap(&tm_b);
  }
  if (warp == 2) {
    tmem_alloc(smem_u32(&sh.tmem_base), 2 * kBN);
    scan_groups(p, sh, lane, kWgrad);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  const uint32_t tmem_base = sh.tmem_base;
  const int64_t total = (int64_t)sh.prefix[p.n_groups] * p.n_tiles;
  volatile int* abort = &sh.abort;

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ producer
      int it = 0;
      bool ok = true;
      for (int64_t tile = blockIdx.x; ok && tile < total; tile += gridDim.x) {
        const TileAt t = tile_at((int)tile, sh.prefix, p.n_groups, p.n_tiles);
        const int rows = sh.rows[t.g], start = sh.start[t.g];
        const int kb_n = kWgrad ? (rows + kBK - 1) / kBK : p.kblocks;
        const int live = rows - t.m * kBM;
        const int pieces = live > 96 ? 4 : (live + 31) / 32;
        const uint32_t bytes = (kWgrad ? kABytes : pieces * (kABytes / 4)) + C::b_bytes;
        for (int kb = 0; kb < kb_n; ++kb, ++it) {
          const int s = it % C::stages;
          if (!mbar_wait(smem_u32(&sh.empty[s]), ((uint32_t)(it / C::stages) & 1u) ^ 1u, abort,
                         p.status)) {
            ok = false;
            break;
          }
          const uint32_t full = smem_u32(&sh.full[s]);
          mbar_arrive_expect_tx(full, bytes);
          const uint32_t sa = ring + s * C::stage_bytes, sb = sa + kABytes;
          if (kWgrad) {
            const int r = start + kb * kBK;
#pragma unroll
            for (int i = 0; i < kBM / 64; ++i)
              tma_load_2d(sa + i * kBK * 128, &tm_a, t.m * kBM + i * 64, r, full);
#pragma unroll
            for (int i = 0; i < kBN / 64; ++i)
              tma_load_2d(sb + i * kBK * 128, &tm_b, t.n * kBN + i * 64, r, full);
          } else {
            const int r = start + t.m * kBM;
            if (pieces == 4) {
              tma_load_2d(sa, &tm_a, kb * kBK, r, full);
            } else {
              for (int i = 0; i < pieces; ++i)
                tma_load_2d(sa + i * (kABytes / 4), &tm_a32, kb * kBK, r + 32 * i, full);
            }
            if (kWay == kForward) {
              tma_load_3d(sb, &tm_b, kb * kBK, t.n * kBN, t.g, full);
            } else {
#pragma unroll
              for (int i = 0; i < kBN / 64; ++i)
                tma_load_3d(sb + i * kBK * 128, &tm_b, t.n * kBN + i * 64, kb * kBK, t.g, full);
            }
          }
        }
      }
      if (!ok) {
        // drain: every armed stage must land before the CTA may exit
        for (int s = 0; s < C::stages && s < it; ++s) {
          const int last = s + ((it - 1 - s) / C::stages) * C::stages;
          mbar_wait(smem_u32(&sh.full[s]), (uint32_t)(last / C::stages) & 1u, nullptr, p.status);
        }
      }
    }
  } else if (warp == 1) {
    // -------------------------------------------------------------- MMA issuer
    int it = 0, used = 0;
    bool ok = true;
    for (int64_t tile = blockIdx.x; ok && tile < total; tile += gridDim.x) {
      const TileAt t = tile_at((int)tile, sh.prefix, p.n_groups, p.n_tiles);
      const int rows = sh.rows[t.g];
      const int kb_n = kWgrad ? (rows + kBK - 1) / kBK : p.kblocks;
      if (kb_n == 0) continue;
      const int buf = used & 1;
      ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&sh.tempty[buf]),
                                             ((uint32_t)(used >> 1) & 1u) ^ 1u, abort, p.status));
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem_base + (uint32_t)(buf * kBN);
      for (int kb = 0; kb < kb_n; ++kb, ++it) {
        const int s = it % C::stages;
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&sh.full[s]),
                                               (uint32_t)(it / C::stages) & 1u, abort, p.status));
        if (!ok) break;
        tc_fence_after();
        const uint32_t sa = ring + s * C::stage_bytes, sb = sa + kABytes;
        int steps = kBK / 16;
        if (kWgrad && rows - kb * kBK < kBK) {
          // rows beyond the group, up to the next 16-row step: cleared in
          // every 64-column box (a swizzled row stays within its 128 bytes)
          const int live = rows - kb * kBK;
          steps = (live + 15) / 16;
          const int dead = steps * 16 - live;
          for (int i = lane; i < dead * 8 * (kBM + kBN) / 64; i += 32) {
            const int box = i / (dead * 8), q = i - box * dead * 8;
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                             sa + (uint32_t)(box * kBK * 128 + live * 128 + q * 16)),
                         "r"(0)
                         : "memory");
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (lane == 0) {
          const uint64_t da = kWgrad ? smem_desc_mn_sw128(sa) : smem_desc_sw128(sa);
          const uint64_t db = kWay == kForward ? smem_desc_sw128(sb) : smem_desc_mn_sw128(sb);
          constexpr uint64_t step_a = kWgrad ? 2048 >> 4 : 32 >> 4;
          constexpr uint64_t step_b = kWay == kForward ? 32 >> 4 : 2048 >> 4;
          for (int i = 0; i < steps; ++i)
            mma_bf16(d, da + step_a * i, db + step_b * i, p.idesc, (kb | i) > 0 ? 1u : 0u);
          mma_commit(smem_u32(&sh.empty[s]));
          if (kb == kb_n - 1) mma_commit(smem_u32(&sh.tfull[buf]));
        }
        __syncwarp();
      }
      ++used;
    }
    if (!ok && it > 0 && lane == 0) {
      // every issued MMA has completed before TMEM is released
      mma_commit(smem_u32(&sh.drained));
      mbar_wait(smem_u32(&sh.drained), 0u, nullptr, p.status);
    }
  } else if (warp >= 4) {
    // -------------------------------------------------------------- epilogue
    const int quarter = warp & 3;  // TMEM lanes 32 * quarter ..
    const int row = quarter * 32 + lane;
    const uint32_t lane_addr = tmem_base + ((uint32_t)(quarter * 32) << 16);
    int used = 0;
    for (int64_t tile = blockIdx.x; tile < total; tile += gridDim.x) {
      const TileAt t = tile_at((int)tile, sh.prefix, p.n_groups, p.n_tiles);
      const int rows = sh.rows[t.g];
      const bool empty = kWgrad && rows == 0;
      if (empty && p.accumulate) continue;
      const int buf = used & 1;
      if (!empty) {
        if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&sh.tfull[buf]),
                                               (uint32_t)(used >> 1) & 1u, abort, p.status)))
          break;
        tc_fence_after();
      }
      const int in_group = t.m * kBM + row;
      const bool live = in_group < (kWgrad ? p.M : rows);
      const int64_t out_row = kWgrad ? (int64_t)t.g * p.M + in_group
                                     : (int64_t)sh.start[t.g] + in_group;
      const int cols = min(kBN, p.N - t.n * kBN);
      const int64_t at = out_row * p.N + (int64_t)t.n * kBN;
      for (int c = 0; c < cols; c += 32) {
        float v[32];
        if (empty) {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0.0f;
        } else {
          tmem_ld32(lane_addr + (uint32_t)(buf * kBN + c), v);
          tmem_wait_ld();
        }
        if (live) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (c + 8 * j < cols) store8(p, at + c + 8 * j, v + 8 * j);
        }
        __syncwarp();
      }
      if (!empty) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.tempty[buf]));
        ++used;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 2) tmem_dealloc(tmem_base, 2 * kBN);
}

template <int kWay, int kBN>
cudaError_t launch16(const Args16& a, const CUtensorMap& ma, const CUtensorMap& ma32,
                     const CUtensorMap& mb, int64_t tile_bound, cudaStream_t stream, int sms) {
  static DeviceOnce once;
  cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(grouped16_kernel<kWay, kBN>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)Tile<kBN>::dyn_smem);
  });
  if (e != cudaSuccess) return e;
  if (tile_bound <= 0) return cudaSuccess;
  const int grid = (int)(tile_bound < sms ? tile_bound : sms);
  grouped16_kernel<kWay, kBN><<<grid, kThreads16, Tile<kBN>::dyn_smem, stream>>>(ma, ma32, mb, a);
  return cudaGetLastError();
}

uint32_t idesc16(int bn, bool f16, bool a_mn, bool b_mn) {
  const uint32_t fmt = f16 ? 0u : 1u;
  return make_idesc(kBM, bn, fmt, fmt) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u);
}

}  // namespace

cudaError_t launch_grouped_matmul(const Groups16& gr, bool f16, int out_type, int K, int N,
                                  const void* a, const void* b, bool trans_b, void* out,
                                  cudaStream_t stream, int sms) {
  if (gr.rows == 0) return cudaSuccess;
  Args16 p{};
  p.group_rows = gr.group_rows;
  p.group_start = gr.group_start;
  p.n_groups = gr.n_groups;
  p.rows = gr.rows;
  p.kblocks = (K + kBK - 1) / kBK;
  p.N = N;
  p.out = out;
  p.out_type = out_type;
  p.status = gr.status;
  CUtensorMap ma, ma32, mb;
  cudaError_t e = make_tmap_bf16(&ma, a, K, gr.rows, 1, kBK, kBM);
  if (e == cudaSuccess) e = make_tmap_bf16(&ma32, a, K, gr.rows, 1, kBK, 32);
  if (e != cudaSuccess) return e;
  // the row tiles there can be: every full one, and a partial one per group
  const int64_t m_bound = gr.rows / kBM + (gr.rows < gr.n_groups ? gr.rows : gr.n_groups);
  auto go = [&](auto bn_tag, auto launch_fwd, auto launch_dx) {
    constexpr int bn = decltype(bn_tag)::value;
    p.n_tiles = (N + bn - 1) / bn;
    p.idesc = idesc16(bn, f16, false, !trans_b);
    e = trans_b ? make_tmap_16b_3d(&mb, b, K, N, gr.n_groups, kBK, bn)
                : make_tmap_16b_3d(&mb, b, N, K, gr.n_groups, 64, kBK);
    if (e != cudaSuccess) return e;
    const int64_t bound = m_bound * p.n_tiles;
    if (bound >= (1ll << 31)) return cudaErrorInvalidValue;
    return trans_b ? launch_fwd(bound) : launch_dx(bound);
  };
#define MOE_GO(BN)                                                                        \
  go(std::integral_constant<int, BN>{},                                                   \
     [&](int64_t t) { return launch16<kForward, BN>(p, ma, ma32, mb, t, stream, sms); },  \
     [&](int64_t t) { return launch16<kInputGrad, BN>(p, ma, ma32, mb, t, stream, sms); })
  if (m_bound * ((N + 255) / 256) >= 4 * sms) return MOE_GO(256);
  if (m_bound * ((N + 127) / 128) >= 4 * sms) return MOE_GO(128);
  return MOE_GO(64);
#undef MOE_GO
}

cudaError_t launch_grouped_wgrad(const Groups16& gr, bool f16, int out_type, int N, int K,
                                 const void* dy, const void* x, void* dw, bool accumulate,
                                 cudaStream_t stream, int sms) {
  Args16 p{};
  p.group_rows = gr.group_rows;
  p.group_start = gr.group_start;
  p.n_groups = gr.n_groups;
  p.rows = gr.rows;
  p.M = N;
  p.N = K;
  p.m_tiles = (N + kBM - 1) / kBM;
  p.out = dw;
  p.out_type = out_type;
  p.accumulate = accumulate ? 1 : 0;
  p.status = gr.status;
  CUtensorMap ma, mb;
  // without rows nothing is loaded, and the row buffers may be NULL
  cudaError_t e = make_tmap_bf16(&ma, gr.rows > 0 ? dy : dw, N, gr.rows, 1, 64, kBK);
  if (e == cudaSuccess) e = make_tmap_bf16(&mb, gr.rows > 0 ? x : dw, K, gr.rows, 1, 64, kBK);
  if (e != cudaSuccess) return e;
  const int64_t m_all = (int64_t)gr.n_groups * p.m_tiles;
  auto go = [&](auto bn_tag) {
    constexpr int bn = decltype(bn_tag)::value;
    p.n_tiles = (K + bn - 1) / bn;
    p.idesc = idesc16(bn, f16, true, true);
    const int64_t bound = m_all * p.n_tiles;
    if (bound >= (1ll << 31)) return cudaErrorInvalidValue;
    return launch16<kWeightGrad, bn>(p, ma, ma, mb, bound, stream, sms);
  };
  if (m_all * ((K + 255) / 256) >= 2 * sms) return go(std::integral_constant<int, 256>{});
  return go(std::integral_constant<int, 128>{});
}

}  // namespace moe

using namespace moe;

static int grouped_args(int32_t type, int32_t out_type, int32_t n_groups, const int32_t* rows_of,
                        const int32_t* starts, int64_t rows, int32_t N, int32_t K) {
  if (type != MOE_BF16 && type != MOE_FP16) return MOE_ERR_SHAPE;
  if (out_type != type && out_type != MOE_FP32) return MOE_ERR_SHAPE;
  if (n_groups < 1 || n_groups > kMaxGroups16 || rows < 0 || rows >= (1ll << 31) - 256)
    return MOE_ERR_SHAPE;
  if (N < 8 || N % 8 != 0 || K < 8 || K % 8 != 0) return MOE_ERR_SHAPE;
  if (N > (1 << 20) || K > (1 << 20)) return MOE_ERR_SHAPE;
  if (!rows_of || !starts) return MOE_ERR_NULL;
  return MOE_OK;
}

extern "C" {

int moe_grouped_matmul(int32_t type, int32_t out_type, int32_t n_groups, const int32_t* group_rows,
                       const int32_t* group_start, int64_t rows, int32_t K, int32_t N,
                       const void* a, const void* b, int32_t trans_b, void* out,
                       uint32_t* status_ws, void* stream) {
  const int r = grouped_args(type, out_type, n_groups, group_rows, group_start, rows, N, K);
  if (r != MOE_OK) return r;
  if (rows == 0) return MOE_OK;  // nothing to do; empty tensors may carry NULL
  if (!a || !b || !out) return MOE_ERR_NULL;
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(out, 16)) return MOE_ERR_ALIGN;
  NvtxRange range("moe_grouped_matmul");
  const Groups16 gr{n_groups, group_rows, group_start, rows, status_ws};
  return cuda_status(launch_grouped_matmul(gr, type == MOE_FP16, out_type, K, N, a, b,
                                           trans_b != 0, out, static_cast<cudaStream_t>(stream),
                                           moe_device_sm_count()));
}

int moe_grouped_wgrad(int32_t type, int32_t out_type, int32_t n_groups, const int32_t* group_rows,
                      const int32_t* group_start, int64_t rows, int32_t N, int32_t K,
                      const void* dy, const void* x, void* dw, int32_t accumulate,
                      uint32_t* status_ws, void* stream) {
  const int r = grouped_args(type, out_type, n_groups, group_rows, group_start, rows, N, K);
  if (r != MOE_OK) return r;
  if (!dw || (rows > 0 && (!dy || !x))) return MOE_ERR_NULL;
  if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(dw, 16)) return MOE_ERR_ALIGN;
  NvtxRange range("moe_grouped_wgrad");
  const Groups16 gr{n_groups, group_rows, group_start, rows, status_ws};
  return cuda_status(launch_grouped_wgrad(gr, type == MOE_FP16, out_type, N, K, dy, x, dw,
                                          accumulate != 0, static_cast<cudaStream_t>(stream),
                                          moe_device_sm_count()));
}

}  // extern "C"
