// Products grouped by expert in 16 bits (bf16 or fp16) with ragged groups, on
// tcgen05 tensor cores: the forward, the input gradient and the weight
// gradient of per-expert linear maps. Group g owns rows s_g .. s_g + r_g - 1
// of the row buffers, at any alignment:
//
//   forward        out[r, n] = sum_k a[r, k] W_g[n, k]     W [G, N, K]
//   input gradient out[r, n] = sum_k a[r, k] W_g[k, n]     W [G, K, N]
//   weight grad    dw_g[n, k] (+)= sum_{r in g} dy[r, n] x[r, k]
//
// 16-bit products are exact in fp32; sums are fp32 in TMEM, in segments where
// they are long (below), rounded once.
//
// The tensor cores take either operand with its reduction index fastest
// (K-major) or slowest (MN-major), so all three products read the tensors as
// they lie: no transposed copy of the weights or of the rows is made.
//
// Forward and input gradient put the weights on the M side of the MMA (128
// output columns a CTA) and the group's rows on the N side, whose size goes
// in steps of 16: a ragged group costs its own rows rounded up to 16, not to
// a tile of 128, and a decoded token's weights stream through shared memory
// beside a few KB of rows. The accumulator is then out^T, which the epilogue
// turns round in shared memory.
//
// Kernels of two CTAs (cta_group::2) share a tile of M = 256: each SM holds
// half of either operand, so it reads 32 KB of L2 per 64-deep k-block instead
// of the 48 KB of a single SM's 128 x 256 tile.
//
// Bound by HBM where groups are short (the weights, once): 8 rows of 64 groups
// at 4096 x 7168 take 77 us (floor 69), 1024 rows at 7168 x 2048 take 295
// (294). Long groups are bound by the tensor cores at the clock that the power
// limit leaves: 32768 rows of 32 groups at 4096 x 7168 take 1402 us in short
// bursts (1.37 PFLOP/s) and 1830 in a run of seconds (1.05), where the clock
// falls to 1000 MHz and the MMAs of the groups' rows fill 87% of its cycles.
//
// One persistent CTA per SM:
//   warp 0     TMA producer: 64-deep k-blocks into a ring of stages
//   warp 1     MMA issuer (of the pair's first CTA), K=16 steps into one of
//              two TMEM buffers
//   warp 2     TMEM allocator; scans the groups into a tile prefix
//   warp 3     weight gradient: clears rows behind a group (below)
//   warps 4-   epilogue: TMEM -> registers -> shared memory -> global memory,
//              while the next tile's MMAs fill the other buffer
// Single-CTA kernels also come with a tile's reduction split over a cluster of
// 2, 4 or 8 CTAs: a tile by itself is bound by what one SM takes in (100 bytes
// a ns) or by the time of a small k-block (225 ns), however idle the others.
// Rows of a tile beyond its group are another group's rows or padding: each
// column of out^T depends on its own row alone, so whatever they hold stays
// in accumulator columns that are never stored. In the weight gradient the
// rows are the reduction: the last k-block's rows beyond the group are
// cleared in shared memory, in both operands (a NaN or infinity there would
// survive a product with zero), and 16-row steps past them are not issued.
#include <type_traits>

#include "kernels.cuh"

namespace moe {

namespace {

constexpr int kBM = 128;  // rows of the M operand per CTA
constexpr int kBK = 64;
constexpr int kABytes = kBM * kBK * 2;
constexpr int kMaxGroups16 = 1025;
constexpr int kMaxStages16 = 10;

enum Way : int { kForward = 0, kInputGrad = 1 };

struct Args16 {
  const int32_t* group_rows;
  const int32_t* group_start;
  int32_t n_groups;
  int32_t kblocks;   // matmul: ceil(K / 64)
  int32_t segment;   // matmul: k-blocks of one TMEM sum, at most
  int32_t n_tiles;   // weight gradient: column tiles of dw per group
  int32_t m_tiles;   // weight gradient: row tiles of dw per group
  int64_t rows;      // rows of the row buffers
  int32_t M;         // weight gradient: rows of dw per group
  int32_t N;         // columns of the output
  void* out;
  int32_t out_type;  // MOE_BF16, MOE_FP16, MOE_FP32
  int32_t accumulate;
  uint32_t idesc;    // without the N size where that varies
  uint32_t* status;
};

struct alignas(8) Shared16 {
  uint64_t full[kMaxStages16];
  uint64_t empty[kMaxStages16];
  uint64_t part[kMaxStages16];   // weight gradient: this CTA's own loads of a
                                 // stage whose last rows are to be cleared
  uint64_t ready[kMaxStages16];  // and both CTAs have cleared them
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t drained;
  uint64_t joined;               // split sums: all parts of a chunk are written
  uint64_t freed;                // and read
  uint32_t tmem_base;
  int abort;
  int asked;                     // weight gradient: k-blocks that the producer has asked for
  int prefix[kMaxGroups16 + 1];
  int rows[kMaxGroups16];
  int start[kMaxGroups16];
};

// ------------------------------------------------------ pairs of CTAs
MOE_DEV uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
MOE_DEV void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// the same shared-memory address in the pair's first CTA
MOE_DEV uint32_t in_leader(uint32_t addr) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
  return r;
}
// and in the cluster's CTA of this rank
MOE_DEV uint32_t in_cta(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
MOE_DEV float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
// Arrival on a barrier of the pair's first CTA. The releasing form, which
// also publishes the thread's stores to the other CTA, costs a memory barrier
// (a microsecond and more in the MMA's path); where only tcgen05 reads are
// done and nothing was stored, the relaxed one is enough.
MOE_DEV void mbar_arrive_release(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
MOE_DEV void mbar_arrive_relaxed(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// mbar_wait for a barrier on which the pair's other CTA arrives as well
template <int kCtas>
MOE_DEV bool mbar_wait_pair(uint32_t bar, uint32_t parity, volatile int* abort, uint32_t* status) {
  if constexpr (kCtas == 1) return mbar_wait(bar, parity, abort, status);
  unsigned long long t0 = 0;
  for (uint32_t i = 0;; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
    if (i == 0) t0 = global_ns();
    if ((i & 63u) == 63u) {
      if (*abort) return false;
      if (global_ns() - t0 > kWaitLimitNs) {
        flag_status(status, kStatusTimeout);
        *abort = 1;
        return false;
      }
    }
  }
}

// mbar_wait for a block that the producer may ask for much later, behind tiles
// that the waiting warp has no part in: the time limit runs from the last block
// that was asked for.
MOE_DEV bool mbar_wait_behind(uint32_t bar, uint32_t parity, const volatile int* asked,
                              volatile int* abort, uint32_t* status) {
  unsigned long long t0 = global_ns();
  int seen = *asked;
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63u) != 0u) continue;
    if (*abort) return false;
    const int now = *asked;
    if (now != seen) {
      seen = now;
      t0 = global_ns();
    } else if (global_ns() - t0 > kWaitLimitNs) {
      flag_status(status, kStatusTimeout);
      *abort = 1;
      return false;
    }
  }
}

template <int kCtas>
MOE_DEV void load_2d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, uint32_t bar) {
  if constexpr (kCtas == 1) {
    tma_load_2d(dst, map, x, y, bar);
  } else {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
  }
}
template <int kCtas>
MOE_DEV void load_3d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z,
                     uint32_t bar) {
  if constexpr (kCtas == 1) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
  } else {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
  }
}
template <int kCtas>
MOE_DEV void alloc16(uint32_t dst, uint32_t cols) {
  if constexpr (kCtas == 1) {
    tmem_alloc(dst, cols);
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int kCtas>
MOE_DEV void dealloc16(uint32_t taddr, uint32_t cols) {
  if constexpr (kCtas == 1) {
    tmem_dealloc(taddr, cols);
  } else {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols)
                 : "memory");
  }
}
template <int kCtas>
MOE_DEV void mma16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (kCtas == 1) {
    mma_bf16(d, a, b, idesc, accumulate);
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  }
}
// arrives on `bar` in every CTA of the tile when the MMAs issued so far are done
template <int kCtas>
MOE_DEV void commit16(uint32_t bar) {
  if constexpr (kCtas == 1) {
    mma_commit(bar);
  } else {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
  }
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
// 16 reduction steps further, in the descriptor's 16-byte address units
constexpr uint64_t kStepK = 32 >> 4;
constexpr uint64_t kStepMN = 16 * 128 >> 4;

// The producer and the MMA issuer run as whole warps of which one elected lane
// issues: so their loops stay uniform, and addresses, coordinates and
// descriptors in uniform registers, which the copy and MMA instructions take
// (run by a single lane, their instructions bounded small tiles: 620 cycles a
// k-block).
MOE_DEV bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}
MOE_DEV int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }
MOE_DEV bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort, uint32_t* status) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, status));
}

// A place in the ring of stages.
template <int kStages, int kStageBytes>
struct Cursor {
  uint32_t full, empty;   // this stage's barriers
  uint32_t offset = 0;    // and its bytes
  uint32_t phase = 0;
  int left = kStages;
  MOE_DEV Cursor(uint32_t full0, uint32_t empty0) : full(full0), empty(empty0) {}
  MOE_DEV void next() {
    full += 8;
    empty += 8;
    offset += kStageBytes;
    if (--left == 0) {
      left = kStages;
      full -= 8 * kStages;
      empty -= 8 * kStages;
      offset = 0;
      phase ^= 1u;
    }
  }
  MOE_DEV int stage() const { return kStages - left; }
};

struct TileAt {
  int g, m, n;
};

// tile -> (group, row tile of the group, column tile), columns fastest: the
// column tiles of one row tile run side by side and share its rows in L2.
// Called by whole warps.
MOE_DEV TileAt tile_at(uint32_t tile, const int* prefix, int n_groups, int n_tiles) {
  const int row_tile = (int)(tile / (uint32_t)n_tiles);
  int lo = 0, hi = n_groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= row_tile) lo = mid; else hi = mid;
  }
  TileAt t;
  t.g = uniform(lo);
  t.m = uniform(row_tile - prefix[lo]);
  t.n = uniform((int)(tile - (uint32_t)row_tile * (uint32_t)n_tiles));
  return t;
}

// The groups' rows and starts into shared memory, by the whole CTA
MOE_DEV void load_groups(const Args16& p, Shared16& sh) {
  for (int g = threadIdx.x; g < p.n_groups; g += blockDim.x) {
    sh.rows[g] = p.group_rows[g];
    sh.start[g] = p.group_start[g];
  }
}

// Checks them, by one warp (a group that fails is flagged and gets no rows),
// and adds up the row tiles (tile_rows rows each; 0: m_tiles for every
// group). Starts must ascend without overlap, so that no row of the output
// has two writers.
MOE_DEV void scan_groups(const Args16& p, Shared16& sh, int lane, int tile_rows) {
  int carry = 0;
  int64_t end = 0;
  if (lane == 0) sh.prefix[0] = 0;
  for (int base = 0; base < p.n_groups; base += 32) {
    const int g = base + lane;
    int r = 0, st = 0;
    if (g < p.n_groups) {
      r = sh.rows[g];
      st = sh.start[g];
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
    const int mt = tile_rows == 0 ? (g < p.n_groups ? p.m_tiles : 0)
                                  : (r + tile_rows - 1) / tile_rows;
    int incl = mt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (g < p.n_groups) {
      sh.rows[g] = r;
      sh.prefix[g + 1] = carry + incl;
    }
    carry += __shfl_sync(0xffffffffu, incl, 31);
  }
}

MOE_DEV uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// ============================================ forward and input gradient
//
// kNT: the most rows of a tile (N of the MMA). A group's rows are cut into
// equal tiles, so that none is nearly empty.
// kSub: tiles of kSub x 128 columns of the output a CTA, one accumulator each.
template <int kCtas, int kNT, int kSub>
struct MatCfg {
  // epilogue warpgroups: one for each accumulator, or two that share the rows
  // of one (a group alone takes as long as 10 k-blocks of its tile)
  static constexpr int groups = kSub == 2 || kNT >= 128 ? 2 : 1;
  static constexpr int threads = 128 + 128 * groups;
  // k-blocks of a stage: two where the tile is so small that waiting and
  // issuing for one (400 cycles) would take longer than its copies and MMAs
  static constexpr int depth = kNT >= 256 ? 1 : 2;
  static constexpr int x_bytes = kNT / kCtas * kBK * 2;  // one k-block of rows
  static constexpr int a_bytes = depth * kSub * kABytes;
  static constexpr int b_bytes = depth * x_bytes;
  static constexpr int stage_bytes = a_bytes + b_bytes;
  // a warp's 32 (fp32: 16) rows x 32 columns of the output, each row padded
  // by 16 bytes against bank conflicts
  static constexpr int turn_bytes = 32 * (32 * 2 + 16);
  static constexpr int room = 213 * 1024 - 4 * groups * turn_bytes;
  static constexpr int stages =
      room / stage_bytes < kMaxStages16 ? room / stage_bytes : kMaxStages16;
  static constexpr size_t dyn_smem = (size_t)stages * stage_bytes + 4 * groups * turn_bytes + 1024;
  // accumulators: two tiles of one (the next tile's MMAs run while one is
  // read), or the two of one tile
  static constexpr int tmem_cols = 2 * kNT;
  // rows of the boxes that fetch less than 128 rows of the groups
  static constexpr int x_box = kNT >= 128 ? 32 : 16;
  // a single CTA's tiles may be lower than 128 columns of the output
  static constexpr bool low = kCtas == 1 && kSub == 1;
  // split sums: rows of a part that lie in the turn buffers at a time, fp32
  static constexpr int part_rows = 16;
  // whether a tile's sum may be taken in segments, which the epilogue adds up
  // in registers: at most 64 a thread, beside the 32 of a load
  static constexpr bool cuts = kSub == 1 && kNT <= 128;
  static_assert(!low || part_rows * kBM * 4 <= 4 * groups * turn_bytes, "a part's rows");
};

// The tensor core's fp32 sums round towards zero at every step of 16 products:
// where all products are positive they are too small by about 2^-24 a step (448
// steps 2.7e-5, 4096 3.5e-4). So one TMEM sum runs only as far as that stays
// under a tenth of half a step of the output's type, and the segments are added
// up in registers, rounded to nearest: 8192 products for fp16, 65536 for bf16,
// and for fp32 outputs the 512 of the weight gradient.
inline int segment_blocks(int out_type) {
  return out_type == MOE_FP32 ? 8 : out_type == MOE_FP16 ? 128 : 1024;
}

// Rates for choosing tiles, in bytes per ns, measured with these kernels: what
// one SM takes in, what all take in from L2 together, and HBM; and the least
// time of a k-block, ns, that a single-CTA kernel needs from its few KB in flight.
constexpr float kSmIn = 100.0f, kL2 = 8900.0f, kHbm = 6450.0f, kLowBlock = 225.0f;
constexpr float kPairBlock = 370.0f;  // the same of a pair's 256 x 256 weight gradient
// ns, joining `split` parts of up to 16 rows (measured: 1.6 us for 2, 1.8 for
// 4, 2.8 for 8)
inline float join_ns(int split) { return 1500.0f + 250.0f * (float)split; }

// Time of a k-block of which each of `active` SMs takes in w bytes of weights,
// which `share` tiles need at the same time, and x bytes of rows.
__host__ __device__ inline float block_ns(float w, float x, float active, float share) {
  const float sm = (w + x) / kSmIn, l2 = (w + x) * active / kL2, hbm = w * active / (share * kHbm);
  const float in = sm > l2 ? sm : l2;
  return in > hbm ? in : hbm;
}
// the same for a round of `tiles` single-CTA tiles of height h
__host__ __device__ inline float low_block_ns(int h, int x_rows, int64_t tiles, int units, int share) {
  const float t = block_ns((float)(h * kBK * 2), (float)(x_rows * kBK * 2),
                           (float)(tiles < units ? tiles : units), (float)share);
  return t > kLowBlock ? t : kLowBlock;
}
// heights that the loads come in: boxes of 32 weight rows, or of 64 columns
__host__ __device__ constexpr int low_step(bool k_major) { return k_major ? 32 : 64; }
// clusters of `split` CTAs that run at a time: those of 4 and 8 do not fill
// every GPC (the occupancy query gives 33 and 15 on 148 SMs)
inline int split_units(int sms, int split) {
  const int units = split <= 2 ? sms / split : sms * (split == 4 ? 33 : 15) / 148;
  return units > 0 ? units : 1;
}
static_assert(16 * (32 * 4 + 16) <= 32 * (32 * 2 + 16), "fp32 rows in the turn buffer");

struct RowTile {
  int first, live, cols;  // first row, rows of the group, N of the MMA
};

// the group's rows in ceil(rows / kNT) tiles of equal size (multiples of 16)
template <int kNT>
MOE_DEV RowTile row_tile(int start, int rows, int m) {
  const int tiles = (rows + kNT - 1) / kNT;
  const int size = ((rows + tiles - 1) / tiles + 15) & ~15;
  RowTile t;
  t.first = uniform(start + m * size);
  t.live = uniform(min(size, rows - m * size));
  t.cols = (max(t.live, 1) + 15) & ~15;
  return t;
}

// kSplit (single CTAs): a tile's sum over K is split over a cluster of that
// many CTAs, for few tiles over a long K: each takes its share of the
// k-blocks, leaves its fp32 part in shared memory, and adds its share of the
// outputs up from all parts, in the order of the ranks.
template <int kWay, int kCtas, int kNT, int kSub, int kSplit>
__global__ void __cluster_dims__(kCtas * kSplit, 1, 1)
    __launch_bounds__(MatCfg<kCtas, kNT, kSub>::threads, 1) grouped_matmul_kernel(const __grid_constant__ CUtensorMap tm_w,
                          const __grid_constant__ CUtensorMap tm_x,
                          const __grid_constant__ CUtensorMap tm_x32, const Args16 p) {
  using C = MatCfg<kCtas, kNT, kSub>;
  static_assert(kSplit == 1 || (C::low && C::groups == 1 && kNT <= 32), "split tiles");
  __shared__ Shared16 sh;
  extern __shared__ uint8_t dyn_smem[];
  const uint32_t ring = (smem_u32(dyn_smem) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = kCtas == 1 ? 0 : (int)cluster_rank();
  const int part = kSplit == 1 ? 0 : (int)cluster_rank();

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::stages; ++s) {
      mbar_init(smem_u32(&sh.full[s]), 1);
      mbar_init(smem_u32(&sh.empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&sh.tfull[b]), 1);
      mbar_init(smem_u32(&sh.tempty[b]), 4 * kCtas * (C::groups / kSub));
    }
    mbar_init(smem_u32(&sh.drained), 1);
    if (kSplit > 1) {
      mbar_init(smem_u32(&sh.joined), 4 * kSplit);
      mbar_init(smem_u32(&sh.freed), 4 * kSplit);
    }
    sh.abort = 0;
    fence_mbar_init();
    prefetch_tensormap(&tm_w);
    prefetch_tensormap(&tm_x);
    prefetch_tensormap(&tm_x32);
  }
  if (warp == 2) alloc16<kCtas>(smem_u32(&sh.tmem_base), C::tmem_cols);
  load_groups(p, sh);
  __syncthreads();
  if (warp == 2) {
    scan_groups(p, sh, lane, kNT);
  }
  tc_fence_before();
  if constexpr (kCtas * kSplit > 1) cluster_sync();
  else __syncthreads();
  tc_fence_after();

  const uint32_t tmem_base = sh.tmem_base;
  const int row_tiles = sh.prefix[p.n_groups];
  const int team = blockIdx.x / (kCtas * kSplit), teams = gridDim.x / (kCtas * kSplit);
  // Output columns per tile. With few tiles a round of tiles of 128 would
  // leave SMs idle, and each SM takes in only so much: lower tiles spread the
  // weights over more of them.
  int height = kBM * kCtas * kSub;
  if (C::low) {
    float best = 0.0f;
    for (int h = kBM; h > 0; h -= low_step(kWay == kForward)) {
      const uint32_t tiles = (uint32_t)row_tiles * (uint32_t)((p.N + h - 1) / h);
      const uint32_t rounds = (tiles + teams - 1) / (uint32_t)teams;
      const float cost = (float)rounds * low_block_ns(h, C::x_box, (int64_t)tiles * kSplit, teams * kSplit, 1);
      if (h == kBM || cost < best) {
        best = cost;
        height = h;
      }
      if (rounds > 16) break;  // an idle share under a sixteenth
    }
  }
  const int n_tiles = (p.N + height - 1) / height;
  const uint32_t total = (uint32_t)row_tiles * (uint32_t)n_tiles;  // checked by the host
  volatile int* abort = &sh.abort;
  const int kb_all = (p.kblocks + C::depth - 1) / C::depth;  // (at least kSplit: the host)
  const int kb_0 = part * kb_all / kSplit, kb_n = (part + 1) * kb_all / kSplit - kb_0;
  const int cut = C::cuts ? p.segment / C::depth : kb_n;  // stages of one TMEM sum

  if (warp == 0) {
    {
      // ------------------------------------------------------------ producer
      const bool elected = elect_one();
      int it = 0;
      bool ok = true;
      Cursor<C::stages, C::stage_bytes> at(smem_u32(sh.full), smem_u32(sh.empty));
      // a pair's loads all count on its first CTA's barrier
      const uint32_t to_leader = kCtas == 2 ? in_leader(at.full) - at.full : 0;
      for (uint32_t tile = team; ok && tile < total; tile += teams) {
        const TileAt t = tile_at(tile, sh.prefix, p.n_groups, n_tiles);
        const RowTile rt = row_tile<kNT>(sh.start[t.g], sh.rows[t.g], t.m);
        const int half = rt.cols / kCtas;
        const int pieces = (half + C::x_box - 1) / C::x_box;
        const bool whole = kNT / kCtas >= 128 && pieces == 4;
        // the weights' boxes: all of 128 rows, or as many as the height takes
        const int w_pieces = !C::low ? 1 : kWay == kForward ? (height + 31) / 32 : (height + 63) / 64;
        const int w_bytes = !C::low ? kSub * kABytes : w_pieces * (kWay == kForward ? 32 : 64) * kBK * 2;
        const int row = rt.first + rank * half;
        const int n0 = t.n * height + rank * kBM;
        const uint32_t bytes = kCtas * C::depth * (w_bytes + pieces * C::x_box * kBK * 2);
        // (a second k-block may lie beyond K: zeros)
        const int k_end = (kb_0 + kb_n) * C::depth * kBK;
        for (int k0 = kb_0 * C::depth * kBK; k0 < k_end; k0 += C::depth * kBK, ++it, at.next()) {
          if (!warp_wait(at.empty, at.phase ^ 1u, abort, p.status)) {
            ok = false;
            break;
          }
          if (!elected) continue;
          if (rank == 0) mbar_arrive_expect_tx(at.full, bytes);
          const uint32_t full = at.full + to_leader;
#pragma unroll
          for (int j = 0; j < C::depth; ++j) {
            const int k = k0 + j * kBK;
            const uint32_t sa = ring + at.offset + j * kSub * kABytes;
            const uint32_t sb = ring + at.offset + C::a_bytes + j * C::x_bytes;
#pragma unroll
            for (int u = 0; u < kSub; ++u) {
              const int n = n0 + u * kBM * kCtas;
              if (C::low && kWay == kForward) {
                for (int i = 0; i < w_pieces; ++i)
                  load_3d<kCtas>(sa + i * 32 * kBK * 2, &tm_w, k, n + i * 32, t.g, full);
              } else if (C::low) {
                for (int i = 0; i < w_pieces; ++i)
                  load_3d<kCtas>(sa + i * kBK * 128, &tm_w, n + i * 64, k, t.g, full);
              } else if (kWay == kForward) {
                load_3d<kCtas>(sa + u * kABytes, &tm_w, k, n, t.g, full);
              } else {
#pragma unroll
                for (int i = 0; i < kBM / 64; ++i)
                  load_3d<kCtas>(sa + u * kABytes + i * kBK * 128, &tm_w, n + i * 64, k, t.g, full);
              }
            }
            if (whole) {
              load_2d<kCtas>(sb, &tm_x, k, row, full);
            } else {
              for (int i = 0; i < pieces; ++i)
                load_2d<kCtas>(sb + i * C::x_box * kBK * 2, &tm_x32, k, row + C::x_box * i, full);
            }
          }
        }
      }
      if (!ok && rank == 0) {
        // drain: every armed stage must land before the CTA may exit
        for (int s = 0; s < C::stages && s < it; ++s) {
          const int last = s + ((it - 1 - s) / C::stages) * C::stages;
          mbar_wait(smem_u32(&sh.full[s]), (uint32_t)(last / C::stages) & 1u, nullptr, p.status);
        }
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {
      // ------------------------------------------------------------ MMA issuer
      const bool elected = elect_one();
      int it = 0, used = 0;
      bool ok = true;
      Cursor<C::stages, C::stage_bytes> at(smem_u32(sh.full), smem_u32(sh.empty));
      const uint64_t desc_w = kWay == kForward ? smem_desc_sw128(ring) : smem_desc_mn_sw128(ring);
      const uint64_t desc_x = smem_desc_sw128(ring + C::a_bytes);
      constexpr uint64_t step_w = kWay == kForward ? kStepK : kStepMN;
      for (uint32_t tile = team; ok && tile < total; tile += teams) {
        const TileAt t = tile_at(tile, sh.prefix, p.n_groups, n_tiles);
        const RowTile rt = row_tile<kNT>(sh.start[t.g], sh.rows[t.g], t.m);
        const uint32_t idesc = p.idesc | ((uint32_t)(rt.cols >> 3) << 17);
        int in_sum = 0;  // stages in this TMEM sum
        for (int kb = 0; kb < kb_n; ++kb, ++it, at.next()) {
          // accumulators in use: sum by sum in turn, or both by each tile
          const int buf = kSub == 1 ? used & 1 : 0;
          const uint32_t free_phase = ((uint32_t)(kSub == 1 ? used >> 1 : used) & 1u) ^ 1u;
          const uint32_t d0 = tmem_base + (uint32_t)(buf * kNT);
          const bool last = kb == kb_n - 1 || in_sum == cut - 1;
          ok = warp_wait(at.full, at.phase, abort, p.status);
          if (!ok) break;
          tc_fence_after();
          const uint64_t off = at.offset >> 4;
#pragma unroll
          for (int u = 0; u < kSub; ++u) {
            if (in_sum == 0) {
              ok = warp_wait(smem_u32(&sh.tempty[buf + u]), free_phase, abort, p.status);
              if (!ok) break;
              tc_fence_after();
            }
            if (!elected) continue;
#pragma unroll
            for (int j = 0; j < C::depth; ++j) {
              const uint64_t dw = desc_w + off + (uint64_t)((j * kSub + u) * (kABytes >> 4));
              const uint64_t dx = desc_x + off + (uint64_t)(j * (C::x_bytes >> 4));
#pragma unroll
              for (int i = 0; i < kBK / 16; ++i)
                mma16<kCtas>(d0 + (uint32_t)(u * kNT), dw + step_w * i, dx + kStepK * i, idesc,
                             j + i > 0 ? 1u : (uint32_t)in_sum);
            }
            if (last) commit16<kCtas>(smem_u32(&sh.tfull[buf + u]));
          }
          if (!ok) break;
          if (elected) commit16<kCtas>(at.empty);
          if (last) ++used;
          in_sum = last ? 0 : in_sum + 1;
        }
      }
      if (!ok && it > 0) {
        // every issued MMA has completed before TMEM is released
        if (elected) commit16<kCtas>(smem_u32(&sh.drained));
        mbar_wait(smem_u32(&sh.drained), 0u, nullptr, p.status);
      }
    }
  } else if (warp >= 4) {
    // -------------------------------------------------------------- epilogue
    const int quarter = warp & 3;  // TMEM lanes 32 * quarter .. = output columns
    const int group = (warp - 4) >> 2;
    const int sub = kSub == 2 ? group : 0;
    constexpr int kShare = C::groups / kSub;  // groups that share an accumulator
    const int first = kShare == 2 ? 32 * group : 0;
    const uint32_t lane_addr = tmem_base + ((uint32_t)(quarter * 32) << 16);
    const uint32_t turn = ring + (uint32_t)(C::stages * C::stage_bytes + (warp - 4) * C::turn_bytes);
    const bool wide = p.out_type == MOE_FP32;
    const bool f16 = p.out_type == MOE_FP16;
    const int es = wide ? 4 : 2;
    const int pitch = 32 * es + 16;
    const int per_row = 32 * es / 16;  // 16-byte pieces of a row's 32 columns
    const int piece = lane % per_row, row0 = lane / per_row, row_step = 32 / per_row;
    int used = 0;
    uint32_t chunks = 0;  // of split sums
    for (uint32_t tile = team; tile < total; tile += teams) {
      const TileAt t = tile_at(tile, sh.prefix, p.n_groups, n_tiles);
      const RowTile rt = row_tile<kNT>(sh.start[t.g], sh.rows[t.g], t.m);
      // the next TMEM sum is in accumulator buf
      int buf = 0;
      auto wait_sum = [&] {
        buf = kSub == 1 ? used & 1 : sub;
        const uint32_t full_phase = (uint32_t)(kSub == 1 ? used >> 1 : used) & 1u;
        ++used;
        const bool full = __all_sync(
            0xffffffffu, mbar_wait(smem_u32(&sh.tfull[buf]), full_phase, abort, p.status));
        if (full) tc_fence_after();
        return full;
      };
      // this tile's output columns end where the next tile's begin
      const int n0 = t.n * height + (sub * kCtas + rank) * kBM + quarter * 32;
      const int n_end = min(t.n * height + height, p.N);
      const int n = n0 + piece * (16 / es);
      uint8_t* const out = static_cast<uint8_t*>(p.out) + ((int64_t)rt.first * p.N + n) * es;
      // the rows from c on in the turn buffer, 32 or (fp32) 16, to global memory
      auto copy_out = [&](int c) {
        __syncwarp();
        if (n < n_end) {
          // (count / row_step is 4 in both types)
          uint32_t q[4][4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(q[k][0]), "=r"(q[k][1]), "=r"(q[k][2]), "=r"(q[k][3])
                         : "r"(turn + (row0 + k * row_step) * pitch + piece * 16)
                         : "memory");
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int j = c + row0 + k * row_step;
            if (j < rt.live)
              *reinterpret_cast<uint4*>(out + (int64_t)j * p.N * es) =
                  make_uint4(q[k][0], q[k][1], q[k][2], q[k][3]);
          }
        }
        __syncwarp();
      };
      auto release = [&] {  // all read: the next MMAs may overwrite
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (kCtas == 2) mbar_arrive_relaxed(in_leader(smem_u32(&sh.tempty[buf])));
          else mbar_arrive(smem_u32(&sh.tempty[buf]));
        }
      };
      // 32 rows of the sum in accumulator buf, from row c on
      auto load_sum = [&](int c, float (&v)[32]) {
        tmem_ld32(lane_addr + (uint32_t)(buf * kNT + c), v);
        tmem_wait_ld();
      };
      // the same added to v
      auto add_sum = [&](int c, float (&v)[32]) {
        float more[32];
        load_sum(c, more);
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] += more[j];
      };
      if (!wait_sum()) break;
      if constexpr (kSplit > 1) {
        float v[32];
        load_sum(0, v);
        release();
        bool ok = true;
        for (int done = cut; done < kb_n; done += cut) {
          ok = wait_sum();
          if (!ok) break;
          add_sum(0, v);
          release();
        }
        if (!ok) break;
        const uint32_t joined = smem_u32(&sh.joined), freed = smem_u32(&sh.freed);
        const uint32_t parts = ring + (uint32_t)(C::stages * C::stage_bytes);
#pragma unroll
        for (int c = 0; c < kNT; c += C::part_rows) {
          if (c >= rt.live) break;
          ok = __all_sync(0xffffffffu,
                          mbar_wait_pair<2>(freed, (chunks & 1u) ^ 1u, abort, p.status));
          if (!ok) break;
#pragma unroll
          for (int j = 0; j < C::part_rows; ++j)
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(
                             parts + (uint32_t)((j * kBM + quarter * 32 + lane) * 4)),
                         "f"(v[c + j])
                         : "memory");
          __syncwarp();
          if (lane < kSplit) mbar_arrive_release(in_cta(joined, lane));
          ok = __all_sync(0xffffffffu, mbar_wait_pair<2>(joined, chunks & 1u, abort, p.status));
          if (!ok) break;
          // 8 columns of a row at a time
          const int rows = min(C::part_rows, rt.live - c);
          for (int i = part * 128 + quarter * 32 + lane; i < rows * (kBM / 8); i += kSplit * 128) {
            const int row = i / (kBM / 8), col = i % (kBM / 8) * 8;
            if (t.n * height + col >= n_end) continue;
            float4 lo = make_float4(0.0f, 0.0f, 0.0f, 0.0f), hi = lo;
#pragma unroll
            for (int q = 0; q < kSplit; ++q) {
              const uint32_t from = in_cta(parts + (uint32_t)((row * kBM + col) * 4), q);
              const float4 a = ld_cluster_f4(from), b = ld_cluster_f4(from + 16);
              lo.x += a.x, lo.y += a.y, lo.z += a.z, lo.w += a.w;
              hi.x += b.x, hi.y += b.y, hi.z += b.z, hi.w += b.w;
            }
            uint4* const dst = reinterpret_cast<uint4*>(
                static_cast<uint8_t*>(p.out) +
                ((int64_t)(rt.first + c + row) * p.N + t.n * height + col) * es);
            if (wide) {
              reinterpret_cast<float4*>(dst)[0] = lo;
              reinterpret_cast<float4*>(dst)[1] = hi;
            } else if (f16) {
              *dst = make_uint4(pack_f16x2(lo.x, lo.y), pack_f16x2(lo.z, lo.w),
                                pack_f16x2(hi.x, hi.y), pack_f16x2(hi.z, hi.w));
            } else {
              *dst = make_uint4(pack_bf16x2(lo.x, lo.y), pack_bf16x2(lo.z, lo.w),
                                pack_bf16x2(hi.x, hi.y), pack_bf16x2(hi.z, hi.w));
            }
          }
          __syncwarp();
          if (lane < kSplit) mbar_arrive_release(in_cta(freed, lane));
          ++chunks;
        }
        if (!ok) break;
        continue;
      }
      // 32 rows from c on to global memory, by way of the turn buffer
      auto put = [&](int c, const float (&v)[32]) {
        if (n0 >= n_end) return;
        if (wide) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              asm volatile("st.shared.f32 [%0], %1;" ::"r"(turn + j * pitch + lane * 4),
                           "f"(v[16 * h + j])
                           : "memory");
            copy_out(c + 16 * h);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const uint32_t w = f16 ? pack_f16x2(v[j], v[j + 1]) : pack_bf16x2(v[j], v[j + 1]);
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(turn + j * pitch + lane * 2),
                         "h"((uint16_t)w)
                         : "memory");
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(turn + (j + 1) * pitch + lane * 2),
                         "h"((uint16_t)(w >> 16))
                         : "memory");
          }
          copy_out(c);
        }
      };
      if (C::cuts && cut < kb_n) {
        constexpr int kPieces = kNT / (32 * kShare);
        float sum[kPieces][32];
        bool ok = true;
        for (int done = 0;;) {
#pragma unroll
          for (int i = 0; i < kPieces; ++i) {
            const int c = first + 32 * kShare * i;
            if (c >= rt.live) continue;
            if (done == 0) load_sum(c, sum[i]);
            else add_sum(c, sum[i]);
          }
          release();
          done += cut;
          if (done >= kb_n) break;
          ok = wait_sum();
          if (!ok) break;
        }
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
          if (first + 32 * kShare * i < rt.live) put(first + 32 * kShare * i, sum[i]);
        continue;
      }
      if (first >= rt.live) release();  // nothing for this group
      for (int c = first; c < rt.live; c += 32 * kShare) {
        float v[32];
        load_sum(c, v);
        if (c + 32 * kShare >= rt.live) release();
        put(c, v);
      }
    }
  }

  tc_fence_before();
  if constexpr (kCtas * kSplit > 1) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  if (warp == 2) dealloc16<kCtas>(tmem_base, C::tmem_cols);
}

// ====================================================== weight gradient
//
// dw_g = dy_g^T x_g: both operands MN-major, the reduction over the group's
// rows. The tensor core's fp32 sums round towards zero at every step, an error
// that grows with the steps of one sum; so the sums are taken over at most 512
// rows and added up in registers, rounded to nearest (one group of 512, 2048,
// 8192, 65536 rows: off by 4.7e-7, 4.8e-7, 4.8e-7, 5.2e-7 of the result).
//
// Measured: 32 groups of 16384 rows in all, dw 7168 x 2048 in fp32, take 617
// to 1033 us from process to process (floor 338). What bounds it is what SMs and L2 exchange: 3.8 GB of
// operand tiles in and 1.9 GB of dw out, 9.1 TB/s in 617 us; without the
// stores it takes 438 (8.6 TB/s), with a stage less 639.
constexpr int kSegment = 8;  // k-blocks per TMEM sum
constexpr int kWThreads = 384;
constexpr int kWRegsLaunch = 168, kWRegsCtl = 40, kWRegsEpi = 232;
static_assert(128 * kWRegsCtl + 256 * kWRegsEpi <= kWThreads * kWRegsLaunch, "register split");

template <int kCtas, int kBN>
struct WgCfg {
  static constexpr int b_bytes = kBN / kCtas * kBK * 2;
  static constexpr int stage_bytes = kABytes + b_bytes;
  static constexpr int buf_bytes = 32 * 128;  // a warp's 32 rows x 128 bytes
  static constexpr int room = 213 * 1024 - 8 * buf_bytes;
  static constexpr int stages = room / stage_bytes < 6 ? room / stage_bytes : 6;
  static constexpr size_t dyn_smem = (size_t)stages * stage_bytes + 8 * buf_bytes + 1024;
};

// the shared-memory sources of this thread's committed stores may be reused
MOE_DEV void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

MOE_DEV void store_3d(const CUtensorMap* map, uint32_t src, int32_t x, int32_t y, int32_t z,
                      bool add) {
  if (add)
    asm volatile(
        "cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group"
        " [%0, {%2, %3, %4}], [%1];" ::"l"(reinterpret_cast<uint64_t>(map)),
        "r"(src), "r"(x), "r"(y), "r"(z)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
            reinterpret_cast<uint64_t>(map)),
        "r"(src), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// 16 consecutive TMEM columns of this warp's 32 lanes
MOE_DEV void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// 32 consecutive columns of a warp's 32 rows (one row a lane) of dw, out
// through shared memory and a TMA store that clips at dw's edges; 16-bit
// outputs gather two calls' 32 columns in one 128-byte row.
struct DwOut {
  const CUtensorMap* map;
  uint32_t buf;
  MOE_DEV void put(const Args16& p, const float (&v)[32], int x, int y, int g, int lane) {
    const bool wide = p.out_type == MOE_FP32;
    const uint32_t swz = (uint32_t)(lane & 7);
    const int part = wide ? 0 : (x >> 5) & 1;  // which half of the 128-byte row
    if (part == 0) {
      if (lane == 0) bulk_wait_read();  // the last store has read the buffer
      __syncwarp();
    }
    const uint32_t row = buf + (uint32_t)(lane * 128);
    if (wide) {
#pragma unroll
      for (int c = 0; c < 8; ++c)
        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(row + (((uint32_t)c ^ swz) << 4)),
                     "f"(v[4 * c]), "f"(v[4 * c + 1]), "f"(v[4 * c + 2]), "f"(v[4 * c + 3])
                     : "memory");
    } else {
      const bool f16 = p.out_type == MOE_FP16;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = f16 ? pack_f16x2(v[8 * c + 2 * i], v[8 * c + 2 * i + 1])
                     : pack_bf16x2(v[8 * c + 2 * i], v[8 * c + 2 * i + 1]);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                         row + (((uint32_t)(4 * part + c) ^ swz) << 4)),
                     "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                     : "memory");
      }
    }
    if (wide || part == 1) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        store_3d(map, buf, wide ? x : x - 32, y, g, p.accumulate != 0);
        bulk_commit();
      }
    }
  }
};

// 32 consecutive columns of one row added to the 16-bit values at dst, rounded
// once (a TMA add would round the addend first); out of line, since its
// registers would be taken from the sums of the common paths
__device__ __noinline__ void add16(uint16_t* out, bool f16, const float* v, int columns) {
  for (int c = 0; c < 4 && 8 * c < columns; ++c) {
    uint4* dst = reinterpret_cast<uint4*>(out + 8 * c);
    const uint4 q = *dst;
    uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo = bf16_lo(w[i]), hi = bf16_hi(w[i]);
      if (f16) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        lo = f.x;
        hi = f.y;
      }
      lo += v[8 * c + 2 * i];
      hi += v[8 * c + 2 * i + 1];
      w[i] = f16 ? pack_f16x2(lo, hi) : pack_bf16x2(lo, hi);
    }
    *dst = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Joins a warp's 32 rows (one a lane) x 32 columns of dw at (y, x) with those
// of the same warp in the cluster's other CTAs, and writes this CTA's share.
// False where a wait ran out.
template <int kSplit>
MOE_DEV bool join_parts(const Args16& p, Shared16& sh, const float (&v)[32], uint32_t buf, int part,
                        int lane, uint32_t chunk, int g, int y, int x, volatile int* abort) {
  const uint32_t joined = smem_u32(&sh.joined), freed = smem_u32(&sh.freed);
  if (!__all_sync(0xffffffffu, mbar_wait_pair<2>(freed, (chunk & 1u) ^ 1u, abort, p.status)))
    return false;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                     buf + (uint32_t)(lane * 128 + ((i ^ (lane & 7)) << 4))),
                 "f"(v[4 * i]), "f"(v[4 * i + 1]), "f"(v[4 * i + 2]), "f"(v[4 * i + 3])
                 : "memory");
  __syncwarp();
  if (lane < kSplit) mbar_arrive_release(in_cta(joined, lane));
  if (!__all_sync(0xffffffffu, mbar_wait_pair<2>(joined, chunk & 1u, abort, p.status))) return false;
#pragma unroll
  for (int k = 0; k < 8 / kSplit; ++k) {
    // 4 columns of a row
    const int i = (part * (8 / kSplit) + k) * 32 + lane, row = i / 8, col = i % 8 * 4;
    if (y + row >= p.M || x + col >= p.N) continue;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int q = 0; q < kSplit; ++q) {
      const float4 a =
          ld_cluster_f4(in_cta(buf + (uint32_t)(row * 128 + (((col / 4) ^ (row & 7)) << 4)), q));
      s.x += a.x, s.y += a.y, s.z += a.z, s.w += a.w;
    }
    const int64_t at = ((int64_t)g * p.M + y + row) * p.N + x + col;
    if (p.out_type == MOE_FP32) {
      float4* const dst = reinterpret_cast<float4*>(static_cast<float*>(p.out) + at);
      if (p.accumulate) {
        const float4 d = *dst;
        s.x += d.x, s.y += d.y, s.z += d.z, s.w += d.w;
      }
      *dst = s;
    } else {
      const bool f16 = p.out_type == MOE_FP16;
      uint2* const dst = reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at);
      if (p.accumulate) {
        const uint2 d = *dst;
        if (f16) {
          const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&d.x));
          const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&d.y));
          s.x += lo.x, s.y += lo.y, s.z += hi.x, s.w += hi.y;
        } else {
          s.x += bf16_lo(d.x), s.y += bf16_hi(d.x), s.z += bf16_lo(d.y), s.w += bf16_hi(d.y);
        }
      }
      *dst = f16 ? make_uint2(pack_f16x2(s.x, s.y), pack_f16x2(s.z, s.w))
                 : make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
    }
  }
  __syncwarp();
  if (lane < kSplit) mbar_arrive_release(in_cta(freed, lane));
  return true;
}

// whether k-block kb of a group ends inside a 16-row step
MOE_DEV bool to_clear(int rows, int kb) {
  const int live = rows - kb * kBK;
  return live < kBK && (live & 15) != 0;
}

// this CTA's share of a group's k-blocks: all of them, or where tiles are
// split one of kSplit shares
struct Share {
  int begin, end;
};
template <int kSplit>
MOE_DEV Share share_of(int blocks, int part) {
  return kSplit == 1 ? Share{0, blocks}
                     : Share{part * blocks / kSplit, (part + 1) * blocks / kSplit};
}

// kSplit (single CTAs): a tile's rows are split over a cluster of that many
// CTAs, for few tiles over long groups: each sums its share, leaves the fp32
// part in shared memory, and adds its share of the tile up from all parts, in
// the order of the ranks.
template <int kCtas, int kBN, int kSplit>
__global__ void __cluster_dims__(kCtas * kSplit, 1, 1) __launch_bounds__(kWThreads, 1)
    grouped_wgrad_kernel(const __grid_constant__ CUtensorMap tm_a,
                         const __grid_constant__ CUtensorMap tm_b,
                         const __grid_constant__ CUtensorMap tm_a16,
                         const __grid_constant__ CUtensorMap tm_b16,
                         const __grid_constant__ CUtensorMap tm_out, const Args16 p) {
  using C = WgCfg<kCtas, kBN>;
  constexpr int kHalf = kBN / kCtas;     // columns of x this CTA loads
  constexpr int kEpiCols = kBN / 2;      // accumulator columns of an epilogue warp
  __shared__ Shared16 sh;
  extern __shared__ uint8_t dyn_smem[];
  const uint32_t ring = (smem_u32(dyn_smem) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  static_assert(kCtas == 1 || kSplit == 1, "single CTAs are split");
  const int rank = kCtas == 1 ? 0 : (int)cluster_rank();
  const int part = kSplit == 1 ? 0 : (int)cluster_rank();

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::stages; ++s) {
      mbar_init(smem_u32(&sh.full[s]), 1);
      mbar_init(smem_u32(&sh.empty[s]), 1);
      mbar_init(smem_u32(&sh.part[s]), 1);
      mbar_init(smem_u32(&sh.ready[s]), kCtas);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&sh.tfull[b]), 1);
      mbar_init(smem_u32(&sh.tempty[b]), 8 * kCtas);
    }
    mbar_init(smem_u32(&sh.drained), 1);
    if (kSplit > 1) {
      mbar_init(smem_u32(&sh.joined), 8 * kSplit);
      mbar_init(smem_u32(&sh.freed), 8 * kSplit);
    }
    sh.abort = 0;
    sh.asked = 0;
    fence_mbar_init();
    prefetch_tensormap(&tm_a);
    prefetch_tensormap(&tm_b);
    prefetch_tensormap(&tm_out);
  }
  if (warp == 2) alloc16<kCtas>(smem_u32(&sh.tmem_base), 2 * kBN);
  load_groups(p, sh);
  __syncthreads();
  if (warp == 2) {
    scan_groups(p, sh, lane, 0);
  }
  tc_fence_before();
  if constexpr (kCtas * kSplit > 1) cluster_sync();
  else __syncthreads();
  tc_fence_after();

  const uint32_t tmem_base = sh.tmem_base;
  const int team = blockIdx.x / (kCtas * kSplit), teams = gridDim.x / (kCtas * kSplit);
  const uint32_t total = (uint32_t)sh.prefix[p.n_groups] * (uint32_t)p.n_tiles;  // checked by the host
  volatile int* abort = &sh.abort;

  if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kWRegsCtl));
  if (warp == 0) {
    {
      // ------------------------------------------------------------ producer
      const bool elected = elect_one();
      int it = 0;
      uint32_t part_phase = 0;  // a bit per stage
      bool ok = true;
      Cursor<C::stages, C::stage_bytes> at(smem_u32(sh.full), smem_u32(sh.empty));
      const uint32_t to_leader = kCtas == 2 ? in_leader(at.full) - at.full : 0;
      for (uint32_t tile = team; ok && tile < total; tile += teams) {
        const TileAt t = tile_at(tile, sh.prefix, p.n_groups, p.n_tiles);
        const int rows = uniform(sh.rows[t.g]);
        const int kb_n = (rows + kBK - 1) / kBK;
        const int a0 = (t.m * kCtas + rank) * kBM, b0 = t.n * kBN + rank * kHalf;
        const Share of = share_of<kSplit>(kb_n, part);
        int r = uniform(sh.start[t.g]) + of.begin * kBK;
        for (int kb = of.begin; kb < of.end; ++kb, ++it, at.next(), r += kBK) {
          if (!warp_wait(at.empty, at.phase ^ 1u, abort, p.status)) {
            ok = false;
            break;
          }
          // A pair's loads count on its first CTA's barrier. Each CTA's loads
          // of a block to be cleared count on a barrier of its own, and the
          // first CTA's full barrier completes at once.
          uint32_t bar = at.full;
          const bool clear = kb == kb_n - 1 && to_clear(rows, kb);
          if (clear) part_phase ^= 1u << at.stage();
          if (!elected) continue;
          *static_cast<volatile int*>(&sh.asked) = it + 1;
          // the last block only as far as its 16-row steps go
          const int steps = min((rows - kb * kBK + 15) / 16, kBK / 16);
          const uint32_t bytes = (uint32_t)(C::stage_bytes / (kBK / 16) * steps);
          if (clear) {
            if (rank == 0) mbar_arrive(bar);
            bar = smem_u32(&sh.part[at.stage()]);
            mbar_arrive_expect_tx(bar, bytes);
          } else {
            if (rank == 0) mbar_arrive_expect_tx(bar, kCtas * bytes);
            bar += to_leader;
          }
          const uint32_t sa = ring + at.offset, sb = sa + kABytes;
          if (steps == kBK / 16) {
#pragma unroll
            for (int i = 0; i < kBM / 64; ++i)
              load_2d<kCtas>(sa + i * kBK * 128, &tm_a, a0 + i * 64, r, bar);
#pragma unroll
            for (int i = 0; i < kHalf / 64; ++i)
              load_2d<kCtas>(sb + i * kBK * 128, &tm_b, b0 + i * 64, r, bar);
          } else {
            for (int j = 0; j < steps; ++j) {
#pragma unroll
              for (int i = 0; i < kBM / 64; ++i)
                load_2d<kCtas>(sa + i * kBK * 128 + j * 16 * 128, &tm_a16, a0 + i * 64, r + 16 * j, bar);
#pragma unroll
              for (int i = 0; i < kHalf / 64; ++i)
                load_2d<kCtas>(sb + i * kBK * 128 + j * 16 * 128, &tm_b16, b0 + i * 64, r + 16 * j, bar);
            }
          }
        }
      }
      if (!ok) {
        // drain: every armed stage must land before the CTA may exit
        for (int s = 0; s < C::stages && s < it; ++s) {
          const int last = s + ((it - 1 - s) / C::stages) * C::stages;
          if (rank == 0)
            mbar_wait(smem_u32(&sh.full[s]), (uint32_t)(last / C::stages) & 1u, nullptr, p.status);
          mbar_wait(smem_u32(&sh.part[s]), ((part_phase >> s) & 1u) ^ 1u, nullptr, p.status);
        }
      }
    }
  } else if (warp == 3) {
    // ---------------------------------------------- rows behind a group cleared
    int it = 0;
    uint32_t part_phase = 0;
    for (uint32_t tile = team; tile < total; tile += teams) {
      const TileAt t = tile_at(tile, sh.prefix, p.n_groups, p.n_tiles);
      const int rows = sh.rows[t.g];
      const int kb_n = (rows + kBK - 1) / kBK;
      const Share of = share_of<kSplit>(kb_n, part);
      it += of.end - of.begin;
      if (of.begin == of.end || of.end < kb_n || !to_clear(rows, kb_n - 1)) continue;
      const int s = (it - 1) % C::stages;
      if (!__all_sync(0xffffffffu, mbar_wait_behind(smem_u32(&sh.part[s]), (part_phase >> s) & 1u,
                                                    &sh.asked, abort, p.status)))
        break;
      part_phase ^= 1u << s;
      // up to the next 16-row step, in every 64-column box (a swizzled row
      // stays within its 128 bytes)
      const uint32_t sa = ring + s * C::stage_bytes;
      const int live = rows - (kb_n - 1) * kBK;
      const int dead = ((live + 15) & ~15) - live;
      for (int i = lane; i < dead * 8 * (kBM + kHalf) / 64; i += 32) {
        const int box = i / (dead * 8), q = i - box * dead * 8;
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                         sa + (uint32_t)(box * kBK * 128 + live * 128 + q * 16)),
                     "r"(0)
                     : "memory");
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (rank > 0) mbar_arrive_release(in_leader(smem_u32(&sh.ready[s])));
        else mbar_arrive(smem_u32(&sh.ready[s]));
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {
      // ------------------------------------------------------------ MMA issuer
      const bool elected = elect_one();
      int it = 0, used = 0;
      uint32_t ready_phase = 0;
      bool ok = true;
      Cursor<C::stages, C::stage_bytes> at(smem_u32(sh.full), smem_u32(sh.empty));
      const uint64_t desc_a = smem_desc_mn_sw128(ring), desc_b = smem_desc_mn_sw128(ring + kABytes);
      for (uint32_t tile = team; ok && tile < total; tile += teams) {
        const TileAt t = tile_at(tile, sh.prefix, p.n_groups, p.n_tiles);
        const int rows = uniform(sh.rows[t.g]);
        const int kb_n = (rows + kBK - 1) / kBK;
        const Share of = share_of<kSplit>(kb_n, part);
        int in_segment = 0;
        for (int kb = of.begin; kb < of.end; ++kb, ++it, at.next()) {
          const int buf = used & 1;
          if (in_segment == 0) {
            ok = warp_wait(smem_u32(&sh.tempty[buf]), ((uint32_t)(used >> 1) & 1u) ^ 1u, abort,
                           p.status);
            if (!ok) break;
            tc_fence_after();
          }
          const uint32_t d = tmem_base + (uint32_t)(buf * kBN);
          ok = warp_wait(at.full, at.phase, abort, p.status);
          const bool last = kb == of.end - 1;
          int steps = kBK / 16;
          if (ok && kb == kb_n - 1) {
            steps = (rows - kb * kBK + 15) / 16;
            if (to_clear(rows, kb)) {
              ok = __all_sync(0xffffffffu,
                              mbar_wait_pair<kCtas>(smem_u32(&sh.ready[at.stage()]),
                                                    (ready_phase >> at.stage()) & 1u, abort, p.status));
              ready_phase ^= 1u << at.stage();
            }
          }
          if (!ok) break;
          tc_fence_after();
          const uint64_t off = at.offset >> 4;
#pragma unroll
          for (int i = 0; i < kBK / 16; ++i)
            if (i < steps && elected)
              mma16<kCtas>(d, desc_a + off + kStepMN * i, desc_b + off + kStepMN * i, p.idesc,
                           i > 0 ? 1u : (uint32_t)in_segment);
          if (elected) commit16<kCtas>(at.empty);
          if (++in_segment == kSegment || last) {
            if (elected) commit16<kCtas>(smem_u32(&sh.tfull[buf]));
            ++used;
            in_segment = 0;
          }
        }
      }
      if (!ok && it > 0) {
        // every issued MMA has completed before TMEM is released
        if (elected) commit16<kCtas>(smem_u32(&sh.drained));
        mbar_wait(smem_u32(&sh.drained), 0u, nullptr, p.status);
      }
    }
  } else if (warp >= 4) {
    // -------------------------------------------------------------- epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kWRegsEpi));
    const int ew = warp - 4;
    const int quarter = warp & 3;  // TMEM lanes 32 * quarter .. = rows of dw
    const int c0 = (ew >> 2) * kEpiCols;
    const uint32_t lane_addr = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)c0;
    DwOut out{&tm_out, ring + (uint32_t)(C::stages * C::stage_bytes + ew * C::buf_bytes)};
    const bool direct = p.accumulate && p.out_type != MOE_FP32;
    int used = 0;
    uint32_t chunks = 0;  // of split tiles
    bool ok = true;
    for (uint32_t tile = team; ok && tile < total; tile += teams) {
      const TileAt t = tile_at(tile, sh.prefix, p.n_groups, p.n_tiles);
      const int kb_n = (sh.rows[t.g] + kBK - 1) / kBK;
      if (kb_n == 0 && p.accumulate) continue;
      const Share of = share_of<kSplit>(kb_n, part);
      const int segments = (of.end - of.begin + kSegment - 1) / kSegment;
      const int y = (t.m * kCtas + rank) * kBM + quarter * 32, x0 = t.n * kBN + c0;
      auto emit = [&](const float (&v)[32], int c) {
        const int x = x0 + c;
        // a 16-bit row is stored when its second half is in: beyond the last
        // column both halves are skipped, or neither
        if (y >= p.M || (p.out_type == MOE_FP32 ? x : x & ~63) >= p.N) return;
        if (direct) {
          float w[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) w[i] = v[i];
          if (y + lane < p.M)
            add16(static_cast<uint16_t*>(p.out) + ((int64_t)t.g * p.M + y + lane) * p.N + x,
                  p.out_type == MOE_FP16, w, p.N - x);
        } else {
          out.put(p, v, x, y, t.g, lane);
        }
      };
      auto wait_segment = [&] {
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&sh.tfull[used & 1]),
                                               (uint32_t)(used >> 1) & 1u, abort, p.status));
        if (ok) tc_fence_after();
        return ok;
      };
      auto release_segment = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          const uint32_t bar = smem_u32(&sh.tempty[used & 1]);
          if (kCtas == 2) mbar_arrive_relaxed(in_leader(bar));
          else mbar_arrive(bar);
        }
        ++used;
      };
      if (kSplit == 1 && segments <= 1) {
        if (segments == 1 && !wait_segment()) break;
#pragma unroll 1
        for (int c = 0; c < kEpiCols; c += 32) {
          float v[32];
          if (segments == 1) {
            tmem_ld32(lane_addr + (uint32_t)((used & 1) * kBN + c), v);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0.0f;
          }
          emit(v, c);
        }
        if (segments == 1) release_segment();
      } else {
        float sum[kEpiCols / 32][32];
#pragma unroll
        for (int c = 0; c < kEpiCols / 32; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i) sum[c][i] = 0.0f;
        for (int seg = 0; seg < segments; ++seg) {
          if (!wait_segment()) break;
#pragma unroll
          for (int c = 0; c < kEpiCols / 16; ++c) {
            float v[16];
            tmem_ld16(lane_addr + (uint32_t)((used & 1) * kBN + 16 * c), v);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) sum[c / 2][(c & 1) * 16 + i] += v[i];
          }
          release_segment();
        }
        if (!ok) break;
        if constexpr (kSplit == 1) {
#pragma unroll
          for (int c = 0; c < kEpiCols / 32; ++c) emit(sum[c], 32 * c);
        } else {
#pragma unroll
          for (int c = 0; c < kEpiCols / 32; ++c) {
            ok = join_parts<kSplit>(p, sh, sum[c], out.buf, part, lane, chunks++, t.g, y,
                                    x0 + 32 * c, abort);
            if (!ok) break;
          }
        }
      }
    }
    if (lane == 0) bulk_wait_all();
  }

  tc_fence_before();
  if constexpr (kCtas * kSplit > 1) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  if (warp == 2) dealloc16<kCtas>(tmem_base, 2 * kBN);
}

// ================================================================ launches
template <int kWay, int kCtas, int kNT, int kSub, int kSplit>
cudaError_t launch_mat(Args16 a, const CUtensorMap& mw, const CUtensorMap& mx,
                       const CUtensorMap& mx32, int64_t row_tiles, cudaStream_t stream, int sms) {
  using C = MatCfg<kCtas, kNT, kSub>;
  static DeviceOnce once;
  cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(grouped_matmul_kernel<kWay, kCtas, kNT, kSub, kSplit>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::dyn_smem);
  });
  if (e != cudaSuccess) return e;
  a.idesc = make_idesc(kBM * kCtas, 0, a.idesc, a.idesc) | (kWay == kInputGrad ? 1u << 15 : 0u);
  // the most tiles there can be
  const int lowest = C::low ? low_step(kWay == kForward) : kBM * kCtas * kSub;
  const int64_t tiles = row_tiles * ((a.N + lowest - 1) / lowest);
  if (tiles >= (1ll << 31)) return cudaErrorInvalidValue;
  constexpr int kCluster = kCtas * kSplit;
  const int64_t units = kSplit == 1 ? sms / kCtas : split_units(sms, kSplit);
  const int64_t grid = (tiles < units ? tiles : units) * kCluster;
  grouped_matmul_kernel<kWay, kCtas, kNT, kSub, kSplit><<<(unsigned)grid, C::threads, C::dyn_smem, stream>>>(mw, mx, mx32, a);
  return cudaGetLastError();
}

template <int kCtas, int kBN, int kSplit>
cudaError_t launch_wg(Args16 a, const CUtensorMap& ma, const CUtensorMap& mb,
                      const CUtensorMap& ma16, const CUtensorMap& mb16, const CUtensorMap& mo,
                      cudaStream_t stream, int sms) {
  using C = WgCfg<kCtas, kBN>;
  static DeviceOnce once;
  cudaError_t e = once.run([] {
    // the register split is only safe if the kernel was built for it
    cudaFuncAttributes fa;
    cudaError_t r = cudaFuncGetAttributes(&fa, grouped_wgrad_kernel<kCtas, kBN, kSplit>);
    if (r != cudaSuccess) return r;
    if (fa.numRegs != kWRegsLaunch) return cudaErrorInvalidConfiguration;
    return cudaFuncSetAttribute(grouped_wgrad_kernel<kCtas, kBN, kSplit>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::dyn_smem);
  });
  if (e != cudaSuccess) return e;
  a.m_tiles = (a.M + kBM * kCtas - 1) / (kBM * kCtas);
  a.n_tiles = (a.N + kBN - 1) / kBN;
  a.idesc = make_idesc(kBM * kCtas, kBN, a.idesc, a.idesc) | 1u << 15 | 1u << 16;
  const int64_t tiles = (int64_t)a.n_groups * a.m_tiles * a.n_tiles;
  if (tiles >= (1ll << 31)) return cudaErrorInvalidValue;
  const int64_t units = kSplit == 1 ? sms / kCtas : split_units(sms, kSplit);
  const int64_t grid = (tiles < units ? tiles : units) * kCtas * kSplit;
  grouped_wgrad_kernel<kCtas, kBN, kSplit><<<(unsigned)grid, kWThreads, C::dyn_smem, stream>>>(ma, mb, ma16, mb16, mo, a);
  return cudaGetLastError();
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
  p.segment = segment_blocks(out_type);
  p.N = N;
  p.out = out;
  p.out_type = out_type;
  p.idesc = f16 ? 0u : 1u;
  p.status = gr.status;
  // The kernel whose rounds of tiles take the least time, if the groups were
  // alike: CTAs x rows x accumulators of 2x256x2, 2x128, 2x256 and 1x32, the
  // last also with its sums split over 2, 4 or 8 CTAs. Over 43 shapes the
  // choice was within 3% of the best of the first four in the mean. Some of
  // them (us, K-major weights; groups x rows, N x K):
  //   32 x 384, 4096 x 4096    322   372   348  1669
  //   16 x 800, 1024 x 1024     31    31    28   102
  //   2 x 821, 920 x 1184     17.4  10.1  11.7  21.2
  //   1 x 1, 4096 x 7168      35.8  20.2  28.8  29.7
  //   8 x 1, 4096 x 7168      75.5  74.3  77.6  73.7
  //   1 x 310, 728 x 936      15.3  10.5  11.3   9.2
  // and where splitting counts:
  //   1 x 1, 144 x 6320        31.6  18.6  26.0  26.9  16.8  11.9   9.4
  //   1 x 1, 4096 x 7168       35.7  20.1  28.9  29.8  18.2  12.3  16.3
  //   1 x 128, 1024 x 7168     38.2  23.5  32.1  31.5  20.8  15.6  24.9
  //   1 x 64, 2048 x 2048      14.7   9.7  12.1  13.0  11.7  11.0  20.5
  //   8 x 1, 7168 x 2048       41.0  41.9  45.9  45.8  47.7  53.1  87.3
  const int64_t busy = gr.rows < gr.n_groups ? gr.rows : gr.n_groups;
  const int64_t each = (gr.rows + busy - 1) / busy;
  auto cost = [&](int ctas, int nt, int sub, int parts) {
    const int64_t split = (each + nt - 1) / nt, rows = (each + split - 1) / split;
    const int units = parts == 1 ? sms / ctas : split_units(sms, parts);
    const float x = (float)((rows + 15) / 16 * 16 / ctas * kBK * 2);
    float best = 1e30f;
    const int step = ctas == 1 ? low_step(trans_b) : kBM * ctas * sub;
    for (int h = kBM * ctas * sub; h > 0; h -= step) {
      const int64_t tiles = busy * split * ((N + h - 1) / h), rounds = (tiles + units - 1) / units;
      if (parts > 1 && rounds > 1) break;  // a join in every round costs more than it gives
      const float active = (float)(tiles < units ? tiles : units) * (float)(ctas * parts);
      float kb = block_ns((float)(h / ctas * kBK * 2), x, active, (float)split);
      const float issue = ctas == 1 ? kLowBlock : nt == 128 ? 135.0f : sub == 1 ? 210.0f : 270.0f;
      kb = kb > issue ? kb : issue;
      const float mma = 2.0f * (float)(rows * sub) / 1.4f;  // cycles at the clock under load
      const float main = (float)((p.kblocks + parts - 1) / parts) * (kb > mma ? kb : mma);
      // the epilogue, beside the next tile's MMAs unless the tile has both
      // accumulators
      const float out = (sub == 1 && nt >= 128 ? 5.0f : 10.0f) * (float)rows + 500.0f +
                        (parts > 1 ? (rows > 16 ? 2.0f : 1.0f) * join_ns(parts) : 0.0f);
      const float t = sub == 2 ? (float)rounds * (main + out)
                               : (float)rounds * (main > out ? main : out) + out;
      if (t < best) best = t;
    }
    return best;
  };
  struct Choice {
    int ctas, nt, sub, parts;
  };
  constexpr Choice all[] = {{2, 256, 2, 1}, {2, 128, 1, 1}, {2, 256, 1, 1}, {1, 32, 1, 1},
                            {1, 32, 1, 2},  {1, 32, 1, 4},  {1, 32, 1, 8}};
  int pick = 1;
  float least = 1e30f;
  for (int i = 0; i < 7; ++i) {
    if (p.kblocks < 4 * all[i].parts && all[i].parts > 1) break;  // two stages a part
    // sums in segments take registers that tiles of 256 rows do not leave
    if (p.kblocks > p.segment && all[i].nt > 128) continue;
    const float t = cost(all[i].ctas, all[i].nt, all[i].sub, all[i].parts);
    if (t < least) {
      least = t;
      pick = i;
    }
  }
  CUtensorMap mw, mx, mx32;
  cudaError_t e = make_tmap_bf16(&mx, a, K, gr.rows, 1, kBK, kBM);
  if (e == cudaSuccess) e = make_tmap_bf16(&mx32, a, K, gr.rows, 1, kBK, pick >= 3 ? 16 : 32);
  if (e == cudaSuccess)
    e = trans_b ? make_tmap_16b_3d(&mw, b, K, N, gr.n_groups, kBK, pick >= 3 ? 32 : kBM)
                : make_tmap_16b_3d(&mw, b, N, K, gr.n_groups, 64, kBK);
  if (e != cudaSuccess) return e;
  auto go = [&](auto ctas, auto nt, auto sub, auto parts) {
    constexpr int kCtas = decltype(ctas)::value, kNT = decltype(nt)::value;
    constexpr int kSub = decltype(sub)::value, kSplit = decltype(parts)::value;
    static_assert(MatCfg<kCtas, kNT, kSub>::x_box == (kNT == 32 ? 16 : 32), "boxes of the maps");
    const int64_t row_tiles = gr.rows / kNT + busy;
    return trans_b ? launch_mat<kForward, kCtas, kNT, kSub, kSplit>(p, mw, mx, mx32, row_tiles, stream, sms)
                   : launch_mat<kInputGrad, kCtas, kNT, kSub, kSplit>(p, mw, mx, mx32, row_tiles, stream, sms);
  };
  using std::integral_constant;
  constexpr integral_constant<int, 1> one{};
  constexpr integral_constant<int, 2> two{};
  constexpr integral_constant<int, 32> low{};
  if (pick == 0) return go(two, integral_constant<int, 256>{}, two, one);
  if (pick == 1) return go(two, integral_constant<int, 128>{}, one, one);
  if (pick == 2) return go(two, integral_constant<int, 256>{}, one, one);
  if (pick == 3) return go(one, low, one, one);
  if (pick == 4) return go(one, low, one, two);
  if (pick == 5) return go(one, low, one, integral_constant<int, 4>{});
  return go(one, low, one, integral_constant<int, 8>{});
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
  p.out = dw;
  p.out_type = out_type;
  p.accumulate = accumulate ? 1 : 0;
  p.idesc = f16 ? 0u : 1u;
  p.status = gr.status;
  CUtensorMap ma, mb, ma16, mb16, mo;
  // without rows nothing is loaded, and the row buffers may be NULL
  cudaError_t e = make_tmap_bf16(&ma, gr.rows > 0 ? dy : dw, N, gr.rows, 1, 64, kBK);
  if (e == cudaSuccess) e = make_tmap_bf16(&mb, gr.rows > 0 ? x : dw, K, gr.rows, 1, 64, kBK);
  if (e == cudaSuccess) e = make_tmap_bf16(&ma16, gr.rows > 0 ? dy : dw, N, gr.rows, 1, 64, 16);
  if (e == cudaSuccess) e = make_tmap_bf16(&mb16, gr.rows > 0 ? x : dw, K, gr.rows, 1, 64, 16);
  if (e == cudaSuccess)
    e = out_type == MOE_FP32 ? make_tmap_f32_3d(&mo, dw, K, N, gr.n_groups, 32, 32)
                             : make_tmap_16b_3d(&mo, dw, K, N, gr.n_groups, 64, 32);
  if (e != cudaSuccess) return e;
  // Pairs of CTAs on 256 x 256 of dw, or single ones on 128 x 128, also with
  // the rows split over clusters of 2, 4 or 8, by the time of their rounds:
  // each SM takes in 32 KB a k-block, but the pair's covers four times as much
  // for two SMs; dw goes out at the SM's share of HBM while the next tile's
  // blocks come in. Splitting is for tiles that all run at once (us, fp32 dw;
  // groups x rows, N x K; unsplit and split):
  //   1 x 20000, 512 x 512     93.5  33.8     4 x 3000, 1360 x 112    19.7  17.0
  //   1 x 20000, 256 x 256     93.1  22.0     1 x 4000, 1024 x 1024   23.7  19.0
  //   1 x 1294, 504 x 160      12.1  11.2     1 x 2000, 4096 x 128    15.0  12.7
  const int es = out_type == MOE_FP32 ? 4 : 2;
  const int64_t blocks = (gr.rows / gr.n_groups + kBK - 1) / kBK;
  auto cost = [&](int side, int ctas, int split) {
    const int units = split == 1 ? sms / ctas : split_units(sms, split);
    const int64_t tiles = (int64_t)gr.n_groups * ((N + side - 1) / side) * ((K + side - 1) / side);
    const int64_t rounds = (tiles + units - 1) / units;
    if (split > 1 && (rounds > 1 || blocks < 2 * split)) return 1e30f;
    const float active = (float)((tiles < units ? tiles : units) * ctas * split);
    float kb = block_ns(0.0f, 32768.0f, active, 1.0f);
    if (ctas == 2 && kb < kPairBlock) kb = kPairBlock;
    const float in = (float)((blocks + split - 1) / split) * kb;
    const float out = (float)(side * side / ctas * es) / (kHbm / 148.0f);
    return (float)rounds * (in > out ? in : out) + (split > 1 ? 2.0f * join_ns(split) : out);
  };
  struct Choice {
    int side, ctas, split;
  };
  constexpr Choice all[] = {{128, 1, 1}, {128, 1, 2}, {128, 1, 4}, {128, 1, 8}, {256, 2, 1}};
  int pick = 0;
  float least = 1e30f;
  for (int i = 0; i < (N > kBM ? 5 : 4); ++i) {
    const float t = cost(all[i].side, all[i].ctas, all[i].split);
    if (t < least) {
      least = t;
      pick = i;
    }
  }
  if (pick == 0) return launch_wg<1, 128, 1>(p, ma, mb, ma16, mb16, mo, stream, sms);
  if (pick == 1) return launch_wg<1, 128, 2>(p, ma, mb, ma16, mb16, mo, stream, sms);
  if (pick == 2) return launch_wg<1, 128, 4>(p, ma, mb, ma16, mb16, mo, stream, sms);
  if (pick == 3) return launch_wg<1, 128, 8>(p, ma, mb, ma16, mb16, mo, stream, sms);
  return launch_wg<2, 256, 1>(p, ma, mb, ma16, mb16, mo, stream, sms);
}

}  // namespace moe

using namespace moe;

static int grouped_args(int32_t type, int32_t out_type, int32_t n_groups, const int32_t* rows_of,
                        const int32_t* starts, int64_t rows, int32_t N, int32_t K,
                        const uint32_t* status) {
  if (type != MOE_BF16 && type != MOE_FP16) return MOE_ERR_SHAPE;
  if (out_type != type && out_type != MOE_FP32) return MOE_ERR_SHAPE;
  if (n_groups < 1 || n_groups > kMaxGroups16 || rows < 0 || rows >= (1ll << 31) - 256)
    return MOE_ERR_SHAPE;
  if (N < 8 || N % 8 != 0 || K < 8 || K % 8 != 0) return MOE_ERR_SHAPE;
  if (N > (1 << 20) || K > (1 << 20)) return MOE_ERR_SHAPE;
  if (!rows_of || !starts) return MOE_ERR_NULL;
  // the kernels read and write them as words
  if (!aligned(rows_of, 4) || !aligned(starts, 4) || !aligned(status, 4)) return MOE_ERR_ALIGN;
  return MOE_OK;
}

extern "C" {

int moe_grouped_matmul(int32_t type, int32_t out_type, int32_t n_groups, const int32_t* group_rows,
                       const int32_t* group_start, int64_t rows, int32_t K, int32_t N,
                       const void* a, const void* b, int32_t trans_b, void* out,
                       uint32_t* status_ws, void* stream) {
  const int r =
      grouped_args(type, out_type, n_groups, group_rows, group_start, rows, N, K, status_ws);
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
  const int r =
      grouped_args(type, out_type, n_groups, group_rows, group_start, rows, N, K, status_ws);
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
