// Grouped-query decode attention over the 8-bit block-scaled cache (e4m3
// codes, one float32 scale per physical block and KV head).
//
// For query head h of sequence s (KV head h / G), over the positions p that
// the window and the holes leave:
//   t_p = scale * sum_i q_i c^K_pi * sK(p),  o = sum_p e^{t_p - m} c^V_p sV(p) / l,
//   l = sum_p e^{t_p - m},  m = max_p t_p,  lse = m + log l
// with codes c and the scales sK, sV of the block that holds p.
//
// Bound: HBM (2 * head_dim bytes a position and KV head against 4 * G *
// head_dim operations). Design:
//  * Work is the stream of all (sequence, head group, 16-position step)
//    units, cut into equal ranges, one per CTA; every CTA derives its range
//    from the context lengths. Going over to the next (sequence, head group)
//    costs a CTA the time of about 5 steps (the ring runs empty), so each
//    counts that many more (without: 118 for 115 us with 64 sequences, 17.8 for
//    15.5 us with 8 short ones; 3 or 8 steps instead: within 1 %). A CTA's
//    warps take the KV heads of the same steps (and, with few KV heads,
//    interleaved steps), so the lines they read together form whole blocks of
//    the pool.
//  * The cells of a step, all heads, arrive by one bulk copy each of K and V
//    (tensor copies with the 128-byte swizzle where rows are whole 128-byte
//    lines, so that the lanes' reads spread over the banks), into a ring that the
//    first warp of the heads' warps fills. (Copies by every lane of the bytes it
//    uses, a head's 128 bytes of every row apart, reached 4.3 TB/s with or
//    without the arithmetic: the accesses, not the work, were the bound.)
//  * A warp computes 16 positions of one KV head with mma.sync.m16n8k16:
//      S = Q K^T: rows 0..7 of A are the high f16 parts of the group's
//      queries, rows 8..15 the low parts. The k index of the product may run
//      over the dims in any order, so k step j of lane group c stands for
//      dims 16c + 4j .. + 3: a lane's 16 bytes of a row are four k steps.
//      O^T += V^T P^T: rows g and g + 8 of A stand for dims 2m and 2m + 1 of
//      16g .. 16g + 15 in tile m, so a lane's 16 bytes of a row are its rows
//      of eight tiles; two positions' bytes pair by byte permutes; P comes
//      from the lane's own scores.
//  * Codes become f16 by one conversion per pair (exact). sK multiplies the
//    scores. sV multiplies the probabilities, relative to the largest sV so
//    far: the accumulators are kept in units of that largest scale and the
//    probabilities carry a factor 2^7, so that with the lazy rescaling
//    (running maximum up to 2^8 behind) their f16 stay below 2^15 and a
//    probability of 1 has 2^31 steps below it.
//  * Partial results of a (CTA, sequence, head group) are merged by a second
//    kernel.
// Measured: Llama-3 heads (8 of 128, groups of 4), 64 sequences of 512..16384
// positions 111 us (610 MB, 5.5 TB/s: 5 us until the first bytes are used, CTAs
// that end between 87 and 103 us, 4 us of merging); 16 of 32768 at 4 heads of 256
// 160 us (6.4 TB/s); 8 windows of 3 heads of 64, float32, 14.6 us (latency).
#include <limits.h>
#include <math.h>

#include <algorithm>

#include "f8.cuh"
#include "f8.h"
#include "mma.cuh"
#include "tmap.h"

namespace mtkv {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kStep = 16;           // positions of a step
constexpr int kMaxG = 8;            // query heads per KV head
constexpr int kBatch = 8;           // step records read at a time
constexpr int kMeta = 2 * kBatch;   // step records per warp
constexpr int kMaxStages = 8;
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int kMinSteps = 4;        // units of a CTA's range, at least (8: 15.2 for 14.6 us below)
constexpr int kSegSteps = 5;        // what starting a (sequence, head group) costs, in steps
constexpr int kHdrBytes = 256;      // status word and padding at the workspace's start

// How a step's cells are copied: all rows as one tensor copy (rows of whole
// 128-byte lines, staged with an odd number of lines), all rows as one bulk copy
// (other rows, at their own pitch), or row by row (a head group of several: its
// part of each row, 16 bytes between them).
enum : int { kTensor = 0, kWhole = 1, kRowwise = 2 };

struct DecodeParams {
  CUtensorMap map_k, map_v;  // kTensor
  const uint8_t *k_pool, *v_pool;
  const float *k_scales, *v_scales;
  const int32_t *table, *ctx, *spans, *kv_map;
  const void *q;
  void *out;
  float *lse;
  float *part_o;   // [slot][head of the group][D]
  float2 *part_ml;  // [slot][head of the group]
  uint32_t *status;
  int B, Hq, H, G, max_blocks, bs_shift;
  int hc, n_hg;      // KV heads of a head group, head groups
  int slices;        // warps that share a KV head's steps
  int copy;          // kTensor, kWhole or kRowwise
  int pitch;         // staged bytes of a row
  int stages, stage_bytes;
  int whole;         // 1: CTA i takes all steps of (sequence, head group) i
  int n_ctas;
  long long n_phys;
  float qscale;      // softmax scale * log2(e)
};

template <int D>
struct Cfg {
  static constexpr int KP = D >= 64 ? D / 64 : 1;  // 16-byte K pieces per 8 positions
  static constexpr int VB = D / 8 < 16 ? D / 8 : 16;  // bytes of a V piece
  static constexpr int VP = D / 8 / VB;            // V pieces per position of a lane
  static constexpr int KS = D / 16;                // k steps of Q K^T
  static constexpr int MT = D / 16;                // dim tiles of O
  static constexpr int CTAS = D == 256 ? 1 : 2;    // per SM
  // shared memory of a CTA: the ring, then the step records
  // (two CTAs of 111 KB, their barriers and the system's 1 KB each fill the SM)
  static constexpr int SMEM = CTAS == 1 ? 224 * 1024 : 111 * 1024;
  static constexpr int META = kWarps * kMeta * 16;
};

struct Meta {
  int phys;       // physical block, or -1
  uint32_t mask;  // positions of the step that are read
  float ks, vs;
};

// Window [lo, hi) of sequence s, empty as (0, 0); with kv_map the span of its runs.
__device__ __forceinline__ void window(const DecodeParams &p, int s, int &lo, int &hi) {
  const int cmax = p.max_blocks << p.bs_shift;
  int c = p.ctx[s];
  if (c < 0 || c > cmax) {
    report(p.status, MT_STATUS_BIT_DEVICE_CHECK);
    c = c < 0 ? 0 : cmax;
  }
  lo = 0;
  hi = c;
  if (p.spans) {
    lo = max(p.spans[2 * s], 0);
    hi = min(p.spans[2 * s + 1], c);
  } else if (p.kv_map) {
    lo = INT_MAX;
    hi = 0;
#pragma unroll
    for (int r = 0; r < MT_KV_MAP_MAX_SPANS; ++r) {
      const int32_t *run = p.kv_map + ((size_t)s * MT_KV_MAP_MAX_SPANS + r) * 2;
      const int a = max(run[0], 0);
      const int e = (int)min((long long)run[0] + run[1], (long long)c);
      if (run[1] > 0 && e > a) {
        lo = min(lo, a);
        hi = max(hi, e);
      }
    }
  }
  if (hi <= lo) lo = hi = 0;
}

__device__ __forceinline__ int steps_of(int lo, int hi) {
  return hi > lo ? (hi - 1) / kStep - lo / kStep + 1 : 0;
}

// Units of a sequence in the stream: its steps, behind kSegSteps that stand for the
// time a CTA takes to go over to it.
__device__ __forceinline__ int units_of(int steps) { return steps ? steps + kSegSteps : 0; }

__device__ __forceinline__ long long warp_incl(long long v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(kAll, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

// Units of all sequences before s, and of all sequences: the whole warp takes part.
__device__ __forceinline__ void count_units(const DecodeParams &p, int s, long long &before,
                                            long long &total) {
  const int lane = threadIdx.x & 31;
  before = total = 0;
  for (int t = lane; t < p.B; t += 32) {
    int lo, hi;
    window(p, t, lo, hi);
    const int n = units_of(steps_of(lo, hi));
    total += n;
    if (t < s) before += n;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    before += __shfl_xor_sync(kAll, before, o);
    total += __shfl_xor_sync(kAll, total, o);
  }
}

// CTAs that a launch's ranges use: none with less than kMinSteps of work.
__device__ __forceinline__ int ctas_used(const DecodeParams &p, long long total) {
  return (int)max(1LL, min((long long)p.n_ctas, total / kMinSteps));
}

// 16 rows of all heads (kTensor): box (64, lines, 16) of [cell][line][64 x 16 bit].
__device__ __forceinline__ void copy_tensor(uint32_t dst, const CUtensorMap *map, int cell,
                                            uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(0), "r"(cell), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void copy_bulk(uint32_t dst, const void *src, uint32_t bytes,
                                          uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 4 consecutive dense elements as floats.
template <int DT>
__device__ __forceinline__ float4 load4(const void *p, size_t i) {
  if constexpr (DT == MT_F32) {
    return __ldg(reinterpret_cast<const float4 *>(p) + i / 4);
  } else {
    const uint2 w = __ldg(reinterpret_cast<const uint2 *>(p) + i / 4);
    if constexpr (DT == MT_F16) {
      const float2 a = h2_to_f2(w.x), b = h2_to_f2(w.y);
      return make_float4(a.x, a.y, b.x, b.y);
    } else {
      return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                         __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
    }
  }
}

template <int D, int DT>
__global__ void __launch_bounds__(kThreads, Cfg<D>::CTAS)
    decode_f8_kernel(const __grid_constant__ DecodeParams p) {
  using C = Cfg<D>;
  constexpr bool PLO = DT == MT_F32;  // low parts of the probabilities too
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kWarps * kMaxStages], empty[kWarps * kMaxStages];
  __shared__ int abort_s;
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int head_l = warp % p.hc, slice = warp / p.hc;  // within the head group
  const bool leader = head_l == 0 && slice < p.slices;  // fills its slice's ring
  const int ST = p.stages;
  const uint32_t ring_a = smem_u32(smem) + (uint32_t)(slice * ST * p.stage_bytes);
  uint64_t *full_r = full + slice * ST, *empty_r = empty + slice * ST;
  Meta *meta = reinterpret_cast<Meta *>(smem + C::SMEM - 1024 - C::META) + warp * kMeta;
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.slices * ST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], p.hc);
    }
    abort_s = 0;
    fence_mbar_init();
  }
  __syncthreads();
  // this lane's bytes of a staged step: K rows 8 t + g, dims 64 j + 16 c ..; V rows
  // 2c, 2c + 1, 8 + 2c, 9 + 2c, dims 128 j + VB g ..
  auto staged = [&](int row, int byte) -> uint32_t {
    if (p.copy != kTensor) return (uint32_t)(row * p.pitch + byte);
    const int line = row * (p.pitch >> 7) + (byte >> 7);
    return (uint32_t)(line * 128 + ((((byte >> 4) & 7) ^ (line & 7)) << 4) + (byte & 15));
  };
  uint32_t k_at[2][C::KP], v_at[4][C::VP];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int j = 0; j < C::KP; ++j) k_at[t][j] = staged(8 * t + g, head_l * D + 64 * j + 16 * c);
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int j = 0; j < C::VP; ++j)
      v_at[t][j] = p.stage_bytes / 2 +
                   staged(2 * c + (t & 1) + 8 * (t >> 1), head_l * D + 128 * j + C::VB * g);
  bool fine = true;            // false once a bounded wait ran out: no more waits or copies
  int u_slot = 0, u_par = 0;   // ring place of the next step to use, and its parity
  int i_slot = 0, i_par = 1;   // of the next step to fill (parity of its emptying)
  pdl_enter();

  // ---- this CTA's range of the stream (sequence, head group, step)
  long long r0 = 0, r1 = 0;
  int s = 0, hg = 0;       // where it starts
  long long skip = 0;      // units of (s, hg) before the range
  int w_lo = 0, w_hi = 0;  // sequence `lane`'s window (B <= 32)
  if (p.whole) {
    s = blockIdx.x / p.n_hg;
    hg = blockIdx.x % p.n_hg;
    r1 = INT_MAX;
  } else {
    long long total = 0, before = 0, incl;
    int k = 0;
    if (p.B <= 32) {
      // every window is loaded once, and kept: lane t has sequence t's
      if (lane < p.B) window(p, lane, w_lo, w_hi);
      k = units_of(steps_of(w_lo, w_hi));
      incl = warp_incl(k);
      total = __shfl_sync(kAll, incl, 31);
    } else {
      count_units(p, 0, before, total);
    }
    total *= p.n_hg;
    const int n = ctas_used(p, total);
    if ((int)blockIdx.x >= n) return;
    r0 = total * blockIdx.x / n;
    r1 = total * (blockIdx.x + 1) / n;
    if (r0 >= r1) return;
    // the sequence that holds unit r0: prefix sums of 32 sequences at a time
    long long run = 0;
    for (int b0 = 0;; b0 += 32) {
      if (p.B > 32) {
        k = 0;
        if (b0 + lane < p.B) {
          int lo, hi;
          window(p, b0 + lane, lo, hi);
          k = units_of(steps_of(lo, hi));
        }
        incl = warp_incl(k);
      }
      const uint32_t past = __ballot_sync(kAll, run + incl * p.n_hg > r0);
      if (past) {
        const int l = __ffs(past) - 1;
        s = b0 + l;
        const int ks = __shfl_sync(kAll, k, l);
        const long long off = r0 - run - (__shfl_sync(kAll, incl, l) - ks) * p.n_hg;
        hg = (int)(off / ks);
        skip = off % ks;
        break;
      }
      run += __shfl_sync(kAll, incl, 31) * p.n_hg;
    }
  }
  auto window_of = [&](int t, int &lo, int &hi) {
    if (!p.whole && p.B <= 32) {
      lo = __shfl_sync(kAll, w_lo, t);
      hi = __shfl_sync(kAll, w_hi, t);
    } else {
      window(p, t, lo, hi);
    }
  };

  long long left = r1 - r0;
  int slot_cta = blockIdx.x;
  while (left > 0 && s < p.B) {
    // ---- a segment: steps [a, b) of (s, hg)
    int lo, hi;
    window_of(s, lo, hi);
    const int n_all = steps_of(lo, hi);
    const int a = max((int)skip - kSegSteps, 0);
    const int b = (int)min((long long)n_all, max(skip + left - kSegSteps, 0LL));
    const int kvh = hg * p.hc + head_l;
    const bool mine = slice < p.slices && kvh < p.H;
    // steps of this warp's slice, and its own (none without a head)
    const int n_slice = a + slice < b ? (b - a - slice + p.slices - 1) / p.slices : 0;
    const int n_mine = mine ? n_slice : 0;
    const int step0 = lo / kStep + a + slice;
    // a step's data are in place / no longer needed by this warp; every warp of
    // the slice, with a head or without, takes part in every step, so none can be
    // a ring's round ahead of the others
    auto await_step = [&]() {
      if (fine)
        fine = __all_sync(kAll, mbar_wait_bounded(&full_r[u_slot], u_par, &abort_s, kWaitNs));
      if (!fine) abort_s = 1;  // the others' waits end too
    };
    auto next_step = [&]() {
      if (++u_slot == ST) {
        u_slot = 0;
        u_par ^= 1;
      }
    };
    if (!mine && slice < p.slices) {
#pragma unroll 1
      for (int k = 0; k < n_slice; ++k) {
        await_step();
        if (lane == 0 && fine) mbar_arrive(&empty_r[u_slot]);
        next_step();
      }
    }

    float oacc[C::MT][4];
#pragma unroll
    for (int m = 0; m < C::MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) oacc[m][i] = 0.f;
    float m_run = -INFINITY, l_run = 0.f, v_ref = 0.f;

    if (n_mine > 0) {
      // ---- step records: id, mask and scales of 8 steps at a time (a lane
      // each), a batch ahead: ids 8 steps before their use, scales 4 before
      const int bps = p.bs_shift == 5 ? 1 : 0;
      auto fetch_id = [&](int k) -> int {  // of this warp's step k
        if (k >= n_mine || lane >= kBatch) return -1;
        const int blk = (step0 + k * p.slices) >> bps;
        return p.table[(size_t)s * p.max_blocks + blk];
      };
      auto check_id = [&](int &id) {
        if (id < -1 || (long long)id >= p.n_phys) {
          report(p.status, MT_STATUS_BIT_DEVICE_CHECK);
          id = -1;
        }
      };
      auto mask_of = [&](int k, int id) -> uint32_t {
        if (id < 0) return 0u;
        const int pos = (step0 + k * p.slices) * kStep;
        auto bits = [&](int x, int y) -> uint32_t {  // positions [x, y)
          x = max(x - pos, 0);
          y = min(y - pos, kStep);
          return y > x ? ((1u << y) - 1u) & ~((1u << x) - 1u) : 0u;
        };
        if (!p.kv_map) return bits(lo, hi);
        uint32_t m = 0;
        for (int r = 0; r < MT_KV_MAP_MAX_SPANS; ++r) {
          const int32_t *run = p.kv_map + ((size_t)s * MT_KV_MAP_MAX_SPANS + r) * 2;
          if (run[1] > 0)
            m |= bits(max(run[0], 0), (int)min((long long)run[0] + run[1], (long long)hi));
        }
        return m;
      };
      auto put = [&](int k, int id, float ks, float vs) {
        if (lane < kBatch) meta[k & (kMeta - 1)] = Meta{id, mask_of(k, id), ks, vs};
      };
      auto scale_of = [&](const float *sc, int id) -> float {
        return id >= 0 ? __ldg(sc + (size_t)id * p.H + kvh) : 0.f;
      };
      int id_0 = fetch_id(lane);
      // (the queries' loads are on their way while the first ids are)
      const bool row_ok = g < p.G;
      const size_t qrow = ((size_t)s * p.Hq + (size_t)kvh * p.G + (row_ok ? g : 0)) * D;
      float4 x[C::KS];
#pragma unroll
      for (int j = 0; j < C::KS; ++j) {
          const int d = (j >> 2) * 64 + 16 * c + 4 * (j & 3);
          x[j] = row_ok ? load4<DT>(p.q, qrow + d) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      check_id(id_0);
      put(lane, id_0, 0.f, 0.f);
      int id_n = fetch_id(kBatch + lane);
      float ks_n = 0.f, vs_n = 0.f;
      __syncwarp();

      // ---- the copies of step k, by the ring's leader
      auto issue = [&](int k) {
        if (!leader || !fine || k >= n_mine) return;
        const Meta &mt = meta[k & (kMeta - 1)];
        fine = __all_sync(kAll, mbar_wait_bounded(&empty_r[i_slot], i_par, &abort_s, kWaitNs));
        if (!fine) {
          abort_s = 1;  // the others' waits end too
          return;
        }
        const uint32_t dst = ring_a + (uint32_t)(i_slot * p.stage_bytes);
        uint64_t *bar = &full_r[i_slot];
        const int half = p.bs_shift == 5 ? ((step0 + k * p.slices) & 1) * kStep : 0;
        const long long cell = ((long long)mt.phys << p.bs_shift) + half;
        const size_t row = (size_t)p.H * D;
        if (mt.mask == 0u) {
          if (lane == 0) mbar_arrive(bar);
        } else if (p.copy == kRowwise) {
          // lane: a row of K (0..15) or of V
          const uint32_t bytes = (uint32_t)(min(p.hc, p.H - hg * p.hc) * D);
          if (lane == 0) mbar_arrive_expect_tx(bar, 32 * bytes);
          __syncwarp();
          copy_bulk(dst + (lane >> 4) * (p.stage_bytes / 2) + (lane & 15) * p.pitch,
                    (lane < 16 ? p.k_pool : p.v_pool) + (size_t)(cell + (lane & 15)) * row +
                        (size_t)hg * p.hc * D,
                    bytes, bar);
        } else if (lane == 0) {
          mbar_arrive_expect_tx(bar, 2 * kStep * p.pitch);
          if (p.copy == kTensor) {
            copy_tensor(dst, &p.map_k, (int)cell, bar);
            copy_tensor(dst + p.stage_bytes / 2, &p.map_v, (int)cell, bar);
          } else {
            copy_bulk(dst, p.k_pool + (size_t)cell * row, kStep * p.pitch, bar);
            copy_bulk(dst + p.stage_bytes / 2, p.v_pool + (size_t)cell * row, kStep * p.pitch, bar);
          }
        }
        __syncwarp();
        if (++i_slot == ST) {
          i_slot = 0;
          i_par ^= 1;
        }
      };
      for (int k = 0; k < ST - 1; ++k) issue(k);
      // scales of the first batch, once its copies are under way
      if (lane < kBatch) {
        meta[lane].ks = scale_of(p.k_scales, id_0);
        meta[lane].vs = scale_of(p.v_scales, id_0);
      }
      if (ST - 1 > kBatch / 2) {  // the loop's first look is past this batch's scales
        check_id(id_n);
        ks_n = scale_of(p.k_scales, id_n);
        vs_n = scale_of(p.v_scales, id_n);
      }
      __syncwarp();

      // ---- the group's queries as A fragments: q / 2^e in high and low f16
      // parts, 2^e bringing the row's largest value to [2^11, 2^12)
      uint32_t qa[C::KS][4];
      float qfac;  // the row's factor on scores, 2^e * scale * log2(e)
      {
        float qmax = 0.f;
#pragma unroll
        for (int j = 0; j < C::KS; ++j) {
          qmax = fmaxf(fmaxf(qmax, fmaxf(fabsf(x[j].x), fabsf(x[j].y))),
                       fmaxf(fabsf(x[j].z), fabsf(x[j].w)));
        }
        qmax = fmaxf(qmax, __shfl_xor_sync(kAll, qmax, 1));
        qmax = fmaxf(qmax, __shfl_xor_sync(kAll, qmax, 2));
        // f = 2^(138 - exponent field), so qmax * f lies in [2^11, 2^12); its
        // own exponent kept within the normal range
        const int ef = (int)(__float_as_uint(qmax) >> 23);
        const int fe = min(max(265 - ef, 1), 253);
        const float f = qmax > 0.f ? __uint_as_float((uint32_t)fe << 23) : 1.f;
        qfac = p.qscale / f;
#pragma unroll
        for (int j = 0; j < C::KS; ++j) {
          split_h2(x[j].x * f, x[j].y * f, qa[j][0], qa[j][1]);
          split_h2(x[j].z * f, x[j].w * f, qa[j][2], qa[j][3]);
        }
      }

      float v_inv = 0.f;  // 1 / v_ref
#pragma unroll 1
      for (int k = 0; k < n_mine; ++k) {
        const int ki = k + ST - 1;  // the step whose copies start now
        if ((ki & (kBatch - 1)) == kBatch / 2) {
          check_id(id_n);
          ks_n = scale_of(p.k_scales, id_n);
          vs_n = scale_of(p.v_scales, id_n);
        } else if ((ki & (kBatch - 1)) == kBatch - 1) {
          const int k0 = (ki & ~(kBatch - 1)) + kBatch;
          if (k0 < n_mine) {
            put(k0 + lane, id_n, ks_n, vs_n);
            id_n = fetch_id(k0 + kBatch + lane);
          }
          __syncwarp();
        }
        issue(ki);
        await_step();
        const Meta mt = meta[k & (kMeta - 1)];
        const uint32_t st = ring_a + (uint32_t)(u_slot * p.stage_bytes);
        uint64_t *done = &empty_r[u_slot];
        next_step();
        // (once a wait has run out nothing is freed either, so nothing is refilled)
        if (mt.mask == 0u || !fine) {
          __syncwarp();
          if (lane == 0 && fine) mbar_arrive(done);
          continue;
        }

        // ---- scores
        uint4 kw[2][C::KP];
#pragma unroll
        for (int j = 0; j < C::KP; ++j)
#pragma unroll
          for (int t = 0; t < 2; ++t) kw[t][j] = lds16(st + k_at[t][j]);
        float sc[2][4];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < C::KP; ++j) {
            const uint4 w = kw[t][j];
            uint32_t b0, b1;
            f8::code4_to_h2(w.x, b0, b1);
            mma_f16(s0, qa[4 * j], b0, b1);
            f8::code4_to_h2(w.y, b0, b1);
            mma_f16(s1, qa[4 * j + 1], b0, b1);
            f8::code4_to_h2(w.z, b0, b1);
            mma_f16(s0, qa[4 * j + 2], b0, b1);
            f8::code4_to_h2(w.w, b0, b1);
            mma_f16(s1, qa[4 * j + 3], b0, b1);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[t][i] = s0[i] + s1[i];
        }
        // V's first piece, on its way while the softmax runs
        uint32_t w[4][C::VB / 4];
        auto load_v = [&](int j) {
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            if constexpr (C::VB == 16) {
              const uint4 u = lds16(st + v_at[t][j]);
              w[t][0] = u.x;
              w[t][1] = u.y;
              w[t][2] = u.z;
              w[t][3] = u.w;
            } else {
              const uint2 u = lds8(st + v_at[t][j]);
              w[t][0] = u.x;
              w[t][1] = u.y;
            }
            // positions that are not read: their codes may be anything, and a
            // NaN times a probability of 0 would reach the row
            if (mt.mask != 0xffffu && !((mt.mask >> (2 * c + (t & 1) + 8 * (t >> 1))) & 1u)) {
#pragma unroll
              for (int i = 0; i < C::VB / 4; ++i) w[t][i] = 0u;
            }
          }
          if (j == C::VP - 1) {  // the step's last read
            __syncwarp();
            if (lane == 0) mbar_arrive(done);
          }
        };
        load_v(0);
        // head g's scores at positions 2c, 2c + 1, 8 + 2c, 9 + 2c
        const float f = qfac * mt.ks;
        float x[4] = {(sc[0][0] + sc[0][2]) * f, (sc[0][1] + sc[0][3]) * f,
                      (sc[1][0] + sc[1][2]) * f, (sc[1][1] + sc[1][3]) * f};
        if (mt.mask != 0xffffu) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = 2 * c + (i & 1) + 8 * (i >> 1);
            if (!((mt.mask >> r) & 1u)) x[i] = -INFINITY;
          }
        }
        // ---- running maximum: rescaled only when a row grows past 2^8 (or
        // has its first position) or a larger V scale comes
        float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
        if (__any_sync(kAll, mx > m_run + 8.f || (m_run == -INFINITY && mx != -INFINITY) ||
                                 mt.vs > v_ref)) {
          mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 2));
          const float m_new = fmaxf(m_run, mx);
          float al = m_run == -INFINITY ? 0.f : ex2(m_run - m_new);
          m_run = m_new;
          l_run *= al;
          const float v_new = fmaxf(v_ref, mt.vs);
          al *= v_new > 0.f ? v_ref / v_new : 1.f;
          v_ref = v_new;
          v_inv = 1.f / fmaxf(v_new, 1.17549435e-38f);
          const float a0 = __shfl_sync(kAll, al, 8 * c), a1 = __shfl_sync(kAll, al, 8 * c + 4);
#pragma unroll
          for (int m = 0; m < C::MT; ++m) {
            oacc[m][0] *= a0;
            oacc[m][1] *= a1;
            oacc[m][2] *= a0;
            oacc[m][3] *= a1;
          }
        }
        // ---- probabilities
        const float mr = m_run == -INFINITY ? 0.f : m_run;
        const float wv = mt.vs * v_inv * 128.f;
        float pr[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          pr[i] = ex2(x[i] - mr);
          l_run += pr[i];
          pr[i] *= wv;
        }
        uint32_t ph[2], pl[2];
        split_h2(pr[0], pr[1], ph[0], pl[0]);
        split_h2(pr[2], pr[3], ph[1], pl[1]);
        // ---- O^T += V^T P^T
#pragma unroll
        for (int j = 0; j < C::VP; ++j) {
          if (j > 0) load_v(j);
#pragma unroll
          for (int i = 0; i < C::VB / 4; ++i) {
            uint32_t a0[4], a1[4];
            f8::code4_to_h2(__byte_perm(w[0][i], w[1][i], 0x5140), a0[0], a0[1]);
            f8::code4_to_h2(__byte_perm(w[2][i], w[3][i], 0x5140), a0[2], a0[3]);
            f8::code4_to_h2(__byte_perm(w[0][i], w[1][i], 0x7362), a1[0], a1[1]);
            f8::code4_to_h2(__byte_perm(w[2][i], w[3][i], 0x7362), a1[2], a1[3]);
            const int m = j * 8 + 2 * i;
            mma_f16(oacc[m], a0, ph[0], ph[1]);
            mma_f16(oacc[m + 1], a1, ph[0], ph[1]);
            if constexpr (PLO) {
              mma_f16(oacc[m], a0, pl[0], pl[1]);
              mma_f16(oacc[m + 1], a1, pl[0], pl[1]);
            }
          }
        }
      }
      l_run += __shfl_xor_sync(kAll, l_run, 1);
      l_run += __shfl_xor_sync(kAll, l_run, 2);
    }

    // ---- the accumulators in units of 1, relative to m
    {
      const float u = v_ref * (1.f / 128.f);
#pragma unroll
      for (int m = 0; m < C::MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) oacc[m][i] *= u;
    }
    // ---- warps that shared a KV head's steps: merged by the first of them
    if (p.slices > 1) {
      // every copy has landed and been read: the ring is scratch here
      __syncthreads();
      constexpr int OWN = 8 * D * 4;  // a warp's [8 heads][D]
      float *own = reinterpret_cast<float *>(smem + warp * OWN);
      float2 *ml = reinterpret_cast<float2 *>(meta);  // m, l of the 8 heads
      if (slice > 0) {
#pragma unroll
        for (int m = 0; m < C::MT; ++m) {
#pragma unroll
          for (int i = 0; i < 4; ++i) own[(m * 4 + i) * 32 + lane] = oacc[m][i];
        }
        if (c == 0) ml[g] = make_float2(m_run, l_run);
      }
      __syncthreads();
      if (slice == 0 && mine) {
        for (int w = 1; w < p.slices; ++w) {
          const int ow = warp + w * p.hc;
          const float *oo = reinterpret_cast<const float *>(smem + ow * OWN);
          const float2 o_ml = reinterpret_cast<const float2 *>(meta + (w * p.hc) * kMeta)[g];
          if (__any_sync(kAll, o_ml.x != -INFINITY || o_ml.y != 0.f)) {
            const float m_new = fmaxf(m_run, o_ml.x);
            const float f0 = m_run == -INFINITY ? 0.f : ex2(m_run - m_new);
            const float f1 = o_ml.x == -INFINITY ? 0.f : ex2(o_ml.x - m_new);
            l_run = l_run * f0 + o_ml.y * f1;
            m_run = m_new;
            const float x0 = __shfl_sync(kAll, f0, 8 * c), x1 = __shfl_sync(kAll, f0, 8 * c + 4);
            const float y0 = __shfl_sync(kAll, f1, 8 * c), y1 = __shfl_sync(kAll, f1, 8 * c + 4);
#pragma unroll
            for (int m = 0; m < C::MT; ++m) {
              const float *ov = oo + m * 128 + lane;
              oacc[m][0] = oacc[m][0] * x0 + ov[0] * y0;
              oacc[m][1] = oacc[m][1] * x1 + ov[32] * y1;
              oacc[m][2] = oacc[m][2] * x0 + ov[64] * y0;
              oacc[m][3] = oacc[m][3] * x1 + ov[96] * y1;
            }
          }
        }
      }
      // (ordered before the next segment's copies into the same bytes)
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncthreads();
    }
    // ---- heads 2c and 2c + 1: dims 16 g + 2 m + (0, 1) of each 128-dim part
    if (mine && slice == 0 && (b > a || p.whole)) {
      const bool done = a == 0 && b == n_all;  // the whole (sequence, head group)
      const float l0 = __shfl_sync(kAll, l_run, 8 * c), l1 = __shfl_sync(kAll, l_run, 8 * c + 4);
      const size_t slot = (size_t)slot_cta + (size_t)s * p.n_hg + hg;
      constexpr int SPAN = C::VB;  // consecutive dims of a lane
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int hd = 2 * c + e;
        if (hd >= p.G) continue;
        const float l = e ? l1 : l0;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const size_t orow = ((size_t)s * p.Hq + (size_t)kvh * p.G + hd) * D;
        float *prow = p.part_o + (slot * (p.hc * p.G) + head_l * p.G + hd) * D;
#pragma unroll
        for (int m = 0; m < C::MT; m += 2) {
          const int d = (m * 2 / SPAN) * 128 + SPAN * g + (m * 2) % SPAN;
          const float v0 = oacc[m][e], v1 = oacc[m][2 + e], v2 = oacc[m + 1][e],
                      v3 = oacc[m + 1][2 + e];
          if (done)
            f8::store4<DT>(p.out, orow + d, v0 * inv, v1 * inv, v2 * inv, v3 * inv);
          else
            f8::store4<MT_F32>(prow, d, v0, v1, v2, v3);
        }
      }
      if (c == 0 && g < p.G) {
        if (!done)
          p.part_ml[slot * (p.hc * p.G) + head_l * p.G + g] = make_float2(m_run, l_run);
        else if (p.lse)
          p.lse[(size_t)s * p.Hq + (size_t)kvh * p.G + g] =
              l_run == 0.f ? -INFINITY : (m_run + log2f(l_run)) * 0.69314718055994530942f;
      }
    }
    if (p.whole) break;
    left -= units_of(n_all) - skip;
    skip = 0;
    if (++hg == p.n_hg) {
      hg = 0;
      // the next sequence with work
      do {
        ++s;
        if (s >= p.B) break;
        window_of(s, lo, hi);
      } while (hi <= lo);
    }
  }
  if (!fine) {
    if (lane == 0) report(p.status, MT_STATUS_BIT_TIMEOUT);
    if (leader) {
      // copies still in flight land before the CTA leaves
      int never = 0;
      for (int i = 0; i < ST; ++i)
        mbar_wait_bounded(&full_r[i], i < i_slot ? i_par ^ 1 : i_par, &never, kWaitNs);
    }
  }
}

// Merge the partial results of split (sequence, head group)s: MW warps for each
// (sequence, query head) take its pieces in turn, then merge through shared
// memory. A CTA has one row, or with MW = 1 kMergeRows. Sequences that see
// nothing get 0 and -infinity here; those that one CTA finished are left alone.
constexpr int kMergeRows = 8;
constexpr int merge_threads(int mw) { return 32 * (mw == 1 ? kMergeRows : mw); }

template <int D, int DT, int MW>
__global__ void __launch_bounds__(merge_threads(MW))
    merge_f8_kernel(const __grid_constant__ DecodeParams p) {
  constexpr int DV = D / 32;
  __shared__ float o_s[MW > 1 ? MW : 1][MW > 1 ? D : 1];
  __shared__ float2 ml_s[MW];
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wi = MW == 1 ? 0 : warp;  // of this row's warps
  const int row = MW == 1 ? blockIdx.x * kMergeRows + warp : blockIdx.x;
  const bool live = row < p.B * p.Hq;
  const int s = live ? row / p.Hq : 0, h = live ? row % p.Hq : 0;
  const int kvh = h / p.G, hg = kvh / p.hc;
  // lengths and windows are inputs: read before the decode kernel has ended
  long long before, total;
  count_units(p, s, before, total);
  int lo, hi;
  window(p, s, lo, hi);
  const int n_all = steps_of(lo, hi);
  int c0 = 0, c1 = -1;  // CTAs that hold pieces
  if (n_all > 0) {
    total *= p.n_hg;
    const int n = ctas_used(p, total);
    const long long u0 = before * p.n_hg + (long long)hg * units_of(n_all) + kSegSteps;
    const long long u1 = u0 + n_all - 1;
    // CTA i holds units [total i / n, total (i + 1) / n)
    c0 = (int)(((u0 + 1) * n - 1) / total);
    c1 = (int)(((u1 + 1) * n - 1) / total);
  }
  // every CTA waits, also one with nothing to merge: this grid must not
  // complete before the decode has, or the stream's next kernel could start
  pdl_wait();
  if (!live || c0 == c1) return;  // (with MW > 1 the whole CTA is this row's)
  const int hin = (kvh - hg * p.hc) * p.G + h % p.G, per = p.hc * p.G;
  float M = -INFINITY, L = 0.f, acc[DV];
#pragma unroll
  for (int e = 0; e < DV; ++e) acc[e] = 0.f;
  const size_t slot0 = (size_t)s * p.n_hg + hg;
#pragma unroll 8
  for (int i = c0 + wi; i <= c1; i += MW) {
    const size_t rec = (slot0 + i) * per + hin;
    const float2 ml = __ldcg(p.part_ml + rec);
    float v[DV];
#pragma unroll
    for (int e = 0; e < DV; e += 2) {
      const float2 x = __ldcg(reinterpret_cast<const float2 *>(p.part_o + rec * D + lane * DV + e));
      v[e] = x.x;
      v[e + 1] = x.y;
    }
    if (ml.x == -INFINITY && ml.y == 0.f) continue;  // a piece that saw nothing
    const float m_new = fmaxf(M, ml.x);
    const float f0 = M == -INFINITY ? (L == 0.f ? 0.f : 1.f) : ex2(M - m_new);
    const float f1 = ml.x == -INFINITY ? 1.f : ex2(ml.x - m_new);  // (its sum is a NaN)
    M = m_new;
    L = L * f0 + ml.y * f1;
#pragma unroll
    for (int e = 0; e < DV; ++e) acc[e] = acc[e] * f0 + v[e] * f1;
  }
  if constexpr (MW > 1) {
    if (lane == 0) ml_s[wi] = make_float2(M, L);
#pragma unroll
    for (int e = 0; e < DV; ++e) o_s[wi][lane * DV + e] = acc[e];
    __syncthreads();
    if (wi > 0) return;
#pragma unroll
    for (int w = 1; w < MW; ++w) M = fmaxf(M, ml_s[w].x);
    L = 0.f;
#pragma unroll
    for (int e = 0; e < DV; ++e) acc[e] = 0.f;
#pragma unroll
    for (int w = 0; w < MW; ++w) {
      const float2 ml = ml_s[w];
      const float f = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : ex2(ml.x - M);
      L += ml.y * f;
#pragma unroll
      for (int e = 0; e < DV; ++e) acc[e] += o_s[w][lane * DV + e] * f;
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  const size_t o = ((size_t)s * p.Hq + h) * D + lane * DV;
#pragma unroll
  for (int e = 0; e < DV; e += 2) {
    if constexpr (DT == MT_F32)
      *reinterpret_cast<float2 *>(reinterpret_cast<float *>(p.out) + o + e) =
          make_float2(acc[e] * inv, acc[e + 1] * inv);
    else
      reinterpret_cast<uint32_t *>(p.out)[(o + e) / 2] =
          f8::pack2<DT>(acc[e] * inv, acc[e + 1] * inv);
  }
  if (p.lse && lane == 0)
    p.lse[(size_t)s * p.Hq + h] =
        L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994530942f;
}

// --------------------------------------------------------------------- host

struct Plan {
  DecodeParams p;
  long long ctas, slots;
  size_t ws;
};

mt_status make_plan(const mt_f8_attn_args *a, const char *where, Plan *pl) {
  const std::string w = std::string(where) + ": ";
  if (!a) return fail(MT_ERR_INVALID_ARG, w + "null args");
  mt_status st = check_f8_cache(&a->cache, where);
  if (st != MT_OK) return st;
  const mt_f8_cache &c = a->cache;
  if (!dtype_bytes(a->dtype)) return fail(MT_ERR_INVALID_ARG, w + "unknown dtype");
  if (a->n_heads <= 0 || a->n_heads % c.n_kv_heads)
    return fail(MT_ERR_INVALID_ARG, w + "n_heads must be a positive multiple of n_kv_heads");
  if (a->n_heads / c.n_kv_heads > kMaxG)
    return fail(MT_ERR_UNSUPPORTED, w + "more than 8 query heads per KV head");
  if (a->n_tokens != c.n_seqs)
    return fail(MT_ERR_INVALID_ARG, w + "n_tokens must equal n_seqs");
  if (a->q_start) return fail(MT_ERR_INVALID_ARG, w + "q_start is for prefill");
  if (a->spans && a->kv_map)
    return fail(MT_ERR_INVALID_ARG, w + "at most one of spans and kv_map");
  if (c.n_seqs > 0 && (!a->q || !a->out)) return fail(MT_ERR_INVALID_ARG, w + "null pointer");
  if (!aligned16(a->q) || !aligned16(a->out))
    return fail(MT_ERR_INVALID_ARG, w + "q and out must be 16-byte aligned");
  if ((long long)c.n_seqs * a->n_heads > 0x7fffffffLL)
    return fail(MT_ERR_UNSUPPORTED, w + "too many query rows");
  DeviceInfo di;
  st = device_info(&di);
  if (st != MT_OK) return st;
  DecodeParams &p = pl->p;
  p = DecodeParams{};
  p.k_pool = c.k_pool;
  p.v_pool = c.v_pool;
  p.k_scales = c.k_scales;
  p.v_scales = c.v_scales;
  p.table = c.block_table;
  p.ctx = c.context_lens;
  p.spans = a->spans;
  p.kv_map = a->kv_map;
  p.q = a->q;
  p.out = a->out;
  p.lse = a->lse;
  p.B = c.n_seqs;
  p.Hq = a->n_heads;
  p.H = c.n_kv_heads;
  p.G = a->n_heads / c.n_kv_heads;
  p.max_blocks = c.max_blocks;
  p.bs_shift = c.block_size == 32 ? 5 : 4;
  p.n_phys = c.n_phys_blocks;
  p.qscale = a->scale * 1.44269504088896340736f;
  p.hc = std::min(p.H, kWarps);
  p.n_hg = (p.H + p.hc - 1) / p.hc;
  p.slices = kWarps / p.hc;
  // staging: the head group's part of a row; a whole row of 128-byte lines takes
  // an odd number of them
  const int row = p.hc * c.head_dim;
  const long long cells = c.n_phys_blocks * c.block_size;
  const bool cells32 = cells > 0 && cells <= 0x7fffffffLL;  // a tensor map's range
  p.copy = p.n_hg > 1 ? kRowwise : row % 128 ? kWhole : cells32 ? kTensor : kRowwise;
  p.pitch = p.copy == kRowwise ? row + 16 : p.copy == kTensor ? (row / 128 | 1) * 128 : row;
  p.stage_bytes = (2 * kStep * p.pitch + 1023) / 1024 * 1024;
  const int ring = (c.head_dim == 64    ? Cfg<64>::SMEM - Cfg<64>::META
                    : c.head_dim == 128 ? Cfg<128>::SMEM - Cfg<128>::META
                                        : Cfg<256>::SMEM - Cfg<256>::META) -
                   1024;
  p.stages = std::min(kMaxStages, ring / (p.slices * p.stage_bytes));
  const long long rows = (long long)p.B * p.n_hg;
  // One CTA for each (sequence, head group), without pieces and a second launch, when
  // that is a few steps a warp (2 sequences of 100 positions, 2 steps a warp: 5.7 us
  // for 6.9; 250 positions, 16 steps a warp: 21.8 for 11.9), or when there are CTAs
  // enough and steps not too many (256 sequences of 8 heads: 250 positions 30 us for
  // 38, 500 52 for 57, 1000 96 for 92; 64 sequences of 250: 22.5 for 17.0).
  const long long grid = (long long)(c.head_dim == 256 ? 1 : 2) * di.n_sm;
  const long long steps = ((long long)p.max_blocks * c.block_size + kStep - 1) / kStep;
  p.whole = rows <= 0x7fffffffLL &&
            (steps <= 6 * p.slices || (steps <= 32 && 4 * rows >= 3 * grid));
  pl->ctas = p.whole ? rows : grid;
  p.n_ctas = (int)pl->ctas;
  pl->slots = p.whole ? 0 : pl->ctas + rows;
  pl->ws = kHdrBytes + (size_t)pl->slots * p.hc * p.G * (c.head_dim + 2) * sizeof(float);
  return MT_OK;
}

template <int D, int DT>
mt_status launch(const Plan &pl, cudaStream_t s) {
  auto kern = decode_f8_kernel<D, DT>;
  constexpr int smem = Cfg<D>::SMEM;
  static_assert(Cfg<D>::SMEM - 1024 - Cfg<D>::META >= kWarps * 8 * D * 4, "the merge's scratch");
  mt_status st = kernel_smem(reinterpret_cast<const void *>(kern), smem,
                             "cudaFuncSetAttribute(f8 decode smem)", true);
  if (st != MT_OK) return st;
  st = cuda_check(launch_pdl(kern, dim3((unsigned)pl.ctas), dim3(kThreads), smem, s, pl.p),
                  "f8 decode launch");
  if (st != MT_OK || pl.p.whole) return st;
  // Warps of a row by its pieces, which are the grid's CTAs over the (sequence, head
  // group)s on average: of the Llama-3 heads, 64 sequences (4.8 pieces) took 111.8
  // us with two warps and 114.7 with one, 256 sequences (1.2) 119.9 and 112.9.
  const long long groups = (long long)pl.p.B * pl.p.n_hg, rows = (long long)pl.p.B * pl.p.Hq;
  const int mw = pl.ctas <= 2 * groups ? 1 : pl.ctas <= 8 * groups ? 2 : 8;
  auto merge = mw == 1   ? merge_f8_kernel<D, DT, 1>
               : mw == 2 ? merge_f8_kernel<D, DT, 2>
                         : merge_f8_kernel<D, DT, 8>;
  const long long grid = mw == 1 ? (rows + kMergeRows - 1) / kMergeRows : rows;
  return cuda_check(launch_pdl(merge, dim3((unsigned)grid), dim3(merge_threads(mw)), 0, s, pl.p),
                    "f8 decode merge launch");
}

template <int D>
mt_status launch_dt(const Plan &pl, mt_dtype t, cudaStream_t s) {
  if (t == MT_F32) return launch<D, MT_F32>(pl, s);
  if (t == MT_F16) return launch<D, MT_F16>(pl, s);
  return launch<D, MT_BF16>(pl, s);
}

}  // namespace
}  // namespace mtkv

using namespace mtkv;

extern "C" size_t mt_paged_attn_decode_f8_workspace_bytes(const mt_f8_attn_args *a) {
  Plan pl;
  return make_plan(a, "mt_paged_attn_decode_f8_workspace_bytes", &pl) == MT_OK ? pl.ws : 0;
}

extern "C" mt_status mt_paged_attn_decode_f8(const mt_f8_attn_args *a, void *workspace,
                                             size_t workspace_bytes, mt_stream stream) {
  Plan pl;
  mt_status st = make_plan(a, "mt_paged_attn_decode_f8", &pl);
  if (st != MT_OK) return st;
  if (!workspace || workspace_bytes < pl.ws || !aligned16(workspace))
    return fail(MT_ERR_INVALID_ARG,
                "mt_paged_attn_decode_f8: workspace missing, too small or not 16-byte aligned");
  if (a->cache.n_seqs == 0) return ok();
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  pl.p.status = reinterpret_cast<uint32_t *>(ws);
  pl.p.part_o = reinterpret_cast<float *>(ws + kHdrBytes);
  pl.p.part_ml = reinterpret_cast<float2 *>(
      pl.p.part_o + (size_t)pl.slots * pl.p.hc * pl.p.G * a->cache.head_dim);
  if (pl.p.copy == kTensor) {
    const long long cells = (long long)a->cache.n_phys_blocks * a->cache.block_size;
    const size_t rb = (size_t)pl.p.H * a->cache.head_dim;
    st = encode_pool_map_3d(&pl.p.map_k, pl.p.k_pool, cells, rb, pl.p.pitch / 128, kStep);
    if (st != MT_OK) return st;
    st = encode_pool_map_3d(&pl.p.map_v, pl.p.v_pool, cells, rb, pl.p.pitch / 128, kStep);
    if (st != MT_OK) return st;
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  st = a->cache.head_dim == 64    ? launch_dt<64>(pl, a->dtype, s)
       : a->cache.head_dim == 128 ? launch_dt<128>(pl, a->dtype, s)
                                  : launch_dt<256>(pl, a->dtype, s);
  return st == MT_OK ? ok() : st;
}
