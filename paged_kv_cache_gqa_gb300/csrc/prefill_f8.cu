// Multi-query (prefill, chunked prefill) attention over the 8-bit
// block-scaled cache, on the 5th-generation tensor cores.
//
// Query j of sequence s (n queries, context c) sits at position c - n + j and
// reads the positions up to its own that the window and the holes leave:
//   t_p = scale * sum_i q_i c^K_pi * sK(p),  o = sum_p e^{t_p - m} c^V_p sV(p) / l,
//   lse = m + log l   (codes c, scales sK and sV of the block that holds p).
//
// Bound: the tensor pipe and, close behind it, the softmax (2 products of 128
// x 128 x head_dim and 128 exponentials a row for each chunk of 128
// positions). Design: a CTA works on two tiles of 128 (query, head) rows at a
// time, "streams" A and B, each with its own softmax warps, so one stream's
// softmax runs while the tensor cores compute the other's products.
//  * 16-bit queries: the streams are two row tiles over the same chunks, so
//    every converted chunk serves 256 rows. float32 queries: the streams are
//    the even and the odd chunks of one row tile, whose Q (and P) come as a
//    high and a low f16 part; the two results merge at the end (each thread
//    reads both accumulators of its row).
//  * 4 converter warps for K and 4 for V read a chunk's codes from global
//    memory into registers (16 bytes a lane, a chunk ahead), turn them into f16
//    (exact) and write them as swizzled operand tiles; rows of holes and past
//    the context become zeros. (One group for both had V's load latency in
//    every chunk: float32 1.10x, long f16 contexts 1.09x slower.)
//  * A warp per stream issues S = Q K^T (both from shared memory), another O +=
//    P V (P from tensor memory, over the scores it came from), in tiles of 64
//    positions: a stream has two score tiles, so S of the next is there when
//    the softmax of this one ends. (One warp for all products took about 4000
//    clocks a tile pair, four times the products themselves; one score tile of
//    128 positions a stream ran 1.15x longer.)
//  * 2 x 4 softmax warps, a thread per row: sK and the row's factor multiply
//    the scores inside the exponent's fused multiply-add; sV enters as an
//    addend of the exponent, log2(sV / v_ref), so neither costs an operation
//    per element; the row's sum takes it out again once per 16 columns.
//    O is rescaled only when the running maximum grows by more than 2^8 or
//    sV passes 4 v_ref, so probabilities stay below 2^15 as f16. At a unit's
//    end they bring the next unit's Q, then write the rows.
//  * Few units (one long context): a unit's chunks are cut into pieces whose
//    records a second kernel merges.
#include <limits.h>
#include <math.h>

#include <algorithm>

#include "f8.cuh"
#include "f8.h"
#include "mma.cuh"
#include "tc.cuh"

namespace mtkv {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kRows = 128;            // rows of a stream = tensor-memory lanes
constexpr int kChunk = 128;           // positions of a chunk
constexpr int kGroups = kChunk / 16;  // groups of 16 positions: one block's scales each
constexpr int kHalf = kChunk / 2;     // positions of a score tile
// warps 0..3: softmax of stream A, 4..7: of B (a thread per row); 8..11:
// converters of K, 12..15: of V; 16, 17 issue S, 18, 19 P V of A and B
constexpr int kConvWarp = 8;
constexpr int kMmaWarp = 16;
constexpr int kThreads = 32 * 20;
// registers a thread: the launch's 96 (65536 / 640, a multiple of 8) are shared
// out anew among the five warpgroups
constexpr int kLaunchRegs = 96, kSoftRegs = 144, kConvRegs = 72, kMmaRegs = 48;
static_assert(2 * kSoftRegs + 2 * kConvRegs + kMmaRegs <= 5 * kLaunchRegs, "registers of a CTA");
constexpr int kPvWarp = 18;
constexpr int kMetaSlots = 8;
constexpr int kUnitSlots = 4;
// tensor memory: two score tiles of stream A, then of B, in [0, 256); outputs
// of A, then of B, in [256, 512)
constexpr uint32_t kTmemCols = 512;
constexpr int kOCol = 256;
constexpr int kMaxSplit = 16;
constexpr int kMaxG = 8;
constexpr int kHdrBytes = 256;
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr float kPBits = 5.f;         // probabilities carry a factor 2^5 (2^8 * 2^2 * 2^5 = 2^15)
constexpr float kNoScale = -1000.f;   // log2 of a V scale of zero

struct PrefillF8Params {
  const uint8_t *k_pool, *v_pool;
  const float *k_scales, *v_scales;
  const int32_t *table, *ctx, *q_start, *spans, *kv_map;
  const void *q;
  void *out;
  float *lse;
  float *rec;       // [unit piece][row][D + 4]: max, sum, destination row, -, outputs
  int *rec_hdr;     // units and pieces per unit
  uint32_t *status;
  int B, Hq, H, G, n_tok, max_blocks, bs_shift;
  int tq;           // queries of a unit
  int g_inv;        // ceil(65536 / G): i / G = i * g_inv >> 16 for i < 256
  int rec_units;    // records the workspace holds
  long long n_phys;
  float qscale;     // softmax scale * log2(e)
};

template <int D, bool PAIR>
struct Cfg {
  static constexpr int HALVES = D / 64;                // 64-dim halves: 128-byte operand rows
  static constexpr int TILE = HALVES * kRows * 128;    // one f16 operand tile of 128 rows
  static constexpr int STAGES = D == 64 ? 3 : 2;       // of K and of V
  static constexpr int UNIT_ROWS = PAIR ? kRows : 2 * kRows;
  static constexpr int SMEM = 1024 + 2 * TILE + 2 * STAGES * TILE + 8 * 32 * 80;
};
static_assert(Cfg<128, false>::SMEM + 6144 <= 227 * 1024, "shared memory");
// one CTA per SM at every head size: the tensor-memory columns are for one
static_assert(2 * Cfg<64, false>::SMEM > 227 * 1024, "two CTAs would share tensor memory");

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3f(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Barrier of the 256 softmax threads that ANDs a flag.
__device__ __forceinline__ bool softmax_sync_and(bool v) {
  uint32_t r;
  asm volatile(
      "{ .reg .pred p, q; setp.ne.u32 p, %1, 0; barrier.red.and.pred q, 1, 256, p; "
      "selp.u32 %0, 1, 0, q; }"
      : "=r"(r)
      : "r"(v ? 1u : 0u)
      : "memory");
  return r != 0;
}

// 32 consecutive f32 columns of this thread's lane.
__device__ __forceinline__ void ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// The loads have landed: no use of v moves above this.
__device__ __forceinline__ void landed(float (&v)[32]) {
  tc::wait_ld();
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+f"(v[i]));
}

// A unit of work: up to UNIT_ROWS rows of one KV head, half chunks [sb, se) of
// chunks [cb, ce).
struct Unit {
  int s, h, qt;    // sequence, KV head, tile of tq queries
  int n, c, q0;    // queries and (clamped) context of the sequence, its first row
  int cb, ce, sb, se;
  int id;          // unit * pieces + piece; -1: no unit is left
  int pieces;      // pieces a unit is cut into
};

struct Walk {
  int s = 0, base = 0;  // sequence s starts with tile `base`
};

__device__ __forceinline__ int tiles_of(const PrefillF8Params &p, int s, bool flag) {
  const int q0 = p.q_start[s], q1 = p.q_start[s + 1];
  const bool bad = q1 < q0 || (q1 > q0 && (q0 < 0 || q1 > p.n_tok));
  const int n = bad ? 0 : q1 - q0;
  if (flag && (bad || (n > 0 && (n > p.ctx[s] || p.ctx[s] > (p.max_blocks << p.bs_shift)))))
    report(p.status, MT_STATUS_BIT_DEVICE_CHECK);
  return (n + p.tq - 1) / p.tq;
}

// Tiles of all sequences, and the most chunks any of them has: whole warp.
__device__ __forceinline__ void count_tiles(const PrefillF8Params &p, int &tiles, int &chunks) {
  const int lane = threadIdx.x & 31;
  long long t = 0;
  int m = 0;
  for (int s = lane; s < p.B; s += 32) {
    const int k = tiles_of(p, s, true);
    t += k;
    if (k) m = max(m, (min(max(p.ctx[s], 0), p.max_blocks << p.bs_shift) + kChunk - 1) / kChunk);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    t += __shfl_xor_sync(kAll, t, o);
    m = max(m, __shfl_xor_sync(kAll, m, o));
  }
  tiles = (int)t;
  chunks = m;
}

// Pieces of a unit's chunks when units are fewer than CTAs: the number whose
// waves of (chunks / pieces, and about 3 chunks' time to start and end) cost
// least.
__device__ __forceinline__ int pieces_of(const PrefillF8Params &p, int n_units, int chunks,
                                         int ctas) {
  if (n_units <= 0 || n_units >= ctas) return 1;
  int best = 1, cost = INT_MAX;
#pragma unroll 1
  for (int k = 1; k <= kMaxSplit && n_units * k <= p.rec_units; ++k) {
    const int waves = (n_units * k + ctas - 1) / ctas;
    const int c = waves * ((chunks + k - 1) / k + 3) + (k > 1 ? 2 : 0);
    if (c < cost) {
      cost = c;
      best = k;
    }
  }
  return best;
}

// The window of query row i at position pos, as a span (0, 0 when empty).
__device__ __forceinline__ void row_span(const PrefillF8Params &p, int i, int end, int &lo,
                                         int &hi) {
  lo = 0;
  hi = end;
  if (p.spans) {
    lo = max(p.spans[2 * (size_t)i], 0);
    hi = min(p.spans[2 * (size_t)i + 1], end);
  } else if (p.kv_map) {
    lo = INT_MAX;
    hi = 0;
#pragma unroll 1
    for (int r = 0; r < MT_KV_MAP_MAX_SPANS; ++r) {
      const int32_t *run = p.kv_map + ((size_t)i * MT_KV_MAP_MAX_SPANS + r) * 2;
      const int a = max(run[0], 0);
      const int e = (int)min((long long)run[0] + run[1], (long long)end);
      if (run[1] > 0 && e > a) {
        lo = min(lo, a);
        hi = max(hi, e);
      }
    }
  }
  if (hi <= lo) lo = hi = 0;
}

// Unit piece `u` of the launch: whole warp. w walks on (u never falls).
__device__ __forceinline__ void unit_at(const PrefillF8Params &p, Walk &w, int u, int n_units,
                                        int pieces, Unit &un) {
  un.id = -1;
  un.pieces = pieces;
  un.cb = un.ce = un.sb = un.se = 0;
  if (u >= n_units * pieces) return;
  const int lane = threadIdx.x & 31;
  const int tile = u / pieces / p.H;
  un.h = u / pieces % p.H;
  un.id = u;
#pragma unroll 1
  for (int b = w.s;; b += 32) {
    const int nt = b + lane < p.B ? tiles_of(p, b + lane, false) : 0;
    int incl = nt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kAll, incl, o);
      if (lane >= o) incl += y;
    }
    const uint32_t past = __ballot_sync(kAll, w.base + incl > tile);
    if (past) {
      const int l = __ffs(past) - 1;
      w.s = b + l;
      w.base += __shfl_sync(kAll, incl - nt, l);
      break;
    }
    w.base += __shfl_sync(kAll, incl, 31);
  }
  un.s = w.s;
  un.qt = tile - w.base;
  un.q0 = p.q_start[un.s];
  un.n = p.q_start[un.s + 1] - un.q0;
  un.c = min(max(p.ctx[un.s], 0), p.max_blocks << p.bs_shift);
  // chunks any query of the unit may read
  const int j0 = un.qt * p.tq, j1 = min(un.n, j0 + p.tq);
  int lo = 0, hi = min(un.c, un.c - un.n + j1);
  if (p.spans || p.kv_map) {
    lo = INT_MAX;
    hi = 0;
#pragma unroll 1
    for (int j = j0 + lane; j < j1; j += 32) {
      int a, e;
      row_span(p, un.q0 + j, min(un.c, un.c - un.n + j + 1), a, e);
      if (e > a) {
        lo = min(lo, a);
        hi = max(hi, e);
      }
    }
    lo = __reduce_min_sync(kAll, lo);
    hi = __reduce_max_sync(kAll, hi);
  }
  const int c0 = hi > lo ? lo / kChunk : 0, nch = hi > lo ? (hi - 1) / kChunk + 1 - c0 : 0;
  const int piece = u % pieces;
  un.cb = c0 + piece * nch / pieces;
  un.ce = c0 + (piece + 1) * nch / pieces;
  un.sb = max(2 * un.cb, lo / kHalf);
  un.se = min(2 * un.ce, (hi + kHalf - 1) / kHalf);
}

// What the converters tell the softmax about a chunk.
struct __align__(16) ChunkMeta {
  float ks[kGroups];   // K scale of each group of 16 positions
  float lv[kGroups];   // log2 of the V scale
  struct __align__(16) {
    uint32_t ok[2];    // positions of this half that hold data
    uint8_t nan[8];    // positions whose V holds a NaN (staged as zeros); byte 4 k +
                       // w, positions 32 k + 8 w .. + 7, is converter warp w's
  } half[2];
};

template <int D, int DT>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_f8_kernel(const __grid_constant__ PrefillF8Params p) {
  constexpr bool PAIR = DT == MT_F32;
  using C = Cfg<D, PAIR>;
  constexpr int ST = C::STAGES, TILE = C::TILE, HALVES = C::HALVES;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ uint32_t tmem_slot;
  __shared__ __align__(8) uint64_t q_full[2], q_free, k_full[ST], k_free[ST], v_full[ST], v_free[ST],
      s_full[2][2], p_full[2][2], pv_done[2][2], o_full[2], u_full[kUnitSlots],
      u_free[kUnitSlots], drain;
  __shared__ Unit units_s[kUnitSlots];     // the scheduler's units, in order
  __shared__ __align__(16) ChunkMeta meta[kMetaSlots];
  __shared__ float qfac_s[2][2 * kRows];   // by live unit parity: the row's factor on scores
  __shared__ float4 ml_s[kRows];           // stream B's max, sum, log2 v_ref, NaN flag
  __shared__ int abort_s;
  uint8_t *base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t *q_sm = base;                    // two tiles: streams A, B; or high, low parts
  uint8_t *k_sm = base + 2 * TILE, *v_sm = k_sm + ST * TILE;
  pdl_enter();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    // Q of a stream's rows, or (PAIR) of both: by the warps that wrote it
    mbar_init(&q_full[0], PAIR ? 8 : 4);
    mbar_init(&q_full[1], PAIR ? 8 : 4);
    mbar_init(&q_free, 2);  // PAIR: both streams' last scores of the unit
    for (int k = 0; k < ST; ++k) {
      mbar_init(&k_full[k], 4);
      mbar_init(&k_free[k], PAIR ? 1 : 2);  // the streams that read a chunk
      mbar_init(&v_full[k], 4);
      mbar_init(&v_free[k], PAIR ? 1 : 2);
    }
    for (int t = 0; t < 2; ++t) {
      for (int b = 0; b < 2; ++b) {
        mbar_init(&s_full[t][b], 2);  // the products' commit and the issuing thread
        mbar_init(&p_full[t][b], 4);
        mbar_init(&pv_done[t][b], 2);  // as for s_full
      }
      mbar_init(&o_full[t], 2);
    }
    for (int k = 0; k < kUnitSlots; ++k) {
      mbar_init(&u_full[k], 1);
      mbar_init(&u_free[k], 20);  // every warp
    }
    mbar_init(&drain, 4);
    abort_s = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tc::alloc(&tmem_slot, kTmemCols);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = tmem_slot;
  bool fine = true;
  // the converters work a chunk ahead and may sleep longer
  const unsigned nap = warp >= kConvWarp && warp < kMmaWarp ? 256 : 20;
  // Wait for a phase (bounded; false: it ran out, or another role gave up), by
  // one thread, which sleeps between its polls so that the waiting warps leave the
  // issue slots to the others (naps of 0 to 256 ns take the same time).
  auto wait1 = [&](uint64_t *bar, uint32_t parity) -> bool {
    if (mbar_try_wait(bar, parity & 1u)) return true;
    const uint64_t t0 = global_ns();
#pragma unroll 1
    do {
#pragma unroll 1
      for (int i = 0; i < 16; ++i) {
        __nanosleep(nap);
        if (mbar_try_wait(bar, parity & 1u)) return true;
      }
    } while (!*(volatile int *)&abort_s && global_ns() - t0 < kWaitNs);
    return false;
  };
  // The same for a warp, with the same answer in every lane.
  auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
    return __all_sync(kAll, wait1(bar, parity));
  };
  // Unit i of this CTA (false: none is left, or a wait ran out).
  auto next_unit = [&](int i, Unit &un) -> bool {
    const int k = i & (kUnitSlots - 1);
    if (!wait(&u_full[k], i / kUnitSlots)) {
      fine = false;
      return false;
    }
    un = units_s[k];
    __syncwarp();
    if (lane == 0) mbar_arrive(&u_free[k]);
    return un.id >= 0;
  };
  // Unit i has been found (or there is no such): no wait.
  auto unit_there = [&](int i) -> bool {
    return __all_sync(kAll, mbar_try_wait(&u_full[i & (kUnitSlots - 1)], (i / kUnitSlots) & 1));
  };
  // The next unit from number i on that has chunks; i moves past it.
  auto live_unit = [&](int &i, Unit &un) -> bool {
#pragma unroll 1
    while (next_unit(i, un)) {
      ++i;
      if (un.ce > un.cb) return true;
    }
    return false;
  };
  // The first half chunk of stream t at or after s, in a unit whose first
  // chunk is the CTA's chunk g0: with float32 queries chunk g is stream g % 2's.
  auto seek = [&](const int t, int g0, int cb, int s) -> int {
    return PAIR && ((g0 + (s >> 1) - cb) & 1) != t ? (s | 1) + 1 : s;
  };

  if (warp >= kConvWarp && warp < kMmaWarp) {
    // =========================================================== converters
    regs_down<kConvRegs>();
    // four warps for K, four for V, each a chunk ahead of what it stages
    const int kv = (warp - kConvWarp) >> 2, cw = warp & 3;
    const uint8_t *pool = kv ? p.v_pool : p.k_pool;
    uint8_t *ring = kv ? v_sm : k_sm;
    uint64_t *full = kv ? v_full : k_full, *empty = kv ? v_free : k_free;
    const bool noter = kv == 0 && cw == 0;  // also passes on scales and positions
    const int r_l = 8 * cw + (lane >> 2);  // rows r_l + 32 k
    const int piece = lane & 3;            // 16 bytes of a 64-byte half row
    const size_t row = (size_t)p.H * D;
    uint4 buf[4 * HALVES];
    int g = 0;                             // chunks converted so far
    // physical blocks of a chunk: lane l holds that of positions 16 l .. 16 l + 15
    auto fetch_ids = [&](int s, int c, int chunk) -> int {
      const int pos = chunk * kChunk + lane * 16;
      if (lane >= kGroups || pos >= c) return -1;
      const int id = p.table[(size_t)s * p.max_blocks + (pos >> p.bs_shift)];
      return id;
    };
    auto check_id = [&](int id) -> int {
      if (id >= -1 && (long long)id < p.n_phys) return id;
      report(p.status, MT_STATUS_BIT_DEVICE_CHECK);
      return -1;
    };
    auto load = [&](int h, int c, int chunk, int ids) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = r_l + 32 * k, pos = chunk * kChunk + r;
        const int id = __shfl_sync(kAll, ids, r >> 4);
        const bool have = id >= 0 && pos < c;
        const uint8_t *src = pool +
                             (((size_t)max(id, 0) << p.bs_shift) + (pos & ((1 << p.bs_shift) - 1))) *
                                 row +
                             (size_t)h * D + piece * 16;
#pragma unroll
        for (int hf = 0; hf < HALVES; ++hf)
          buf[k * HALVES + hf] = have ? __ldg(reinterpret_cast<const uint4 *>(src + 64 * hf))
                                      : make_uint4(0, 0, 0, 0);
      }
    };
    // codes -> f16 operand rows: 16 codes are the 16-byte units 2 piece, 2
    // piece + 1 of a 128-byte row, swizzled
    auto put = [&](uint8_t *tile) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = r_l + 32 * k;
#pragma unroll
        for (int hf = 0; hf < HALVES; ++hf) {
          const uint4 w = buf[k * HALVES + hf];
          uint4 x, y;
          f8::code4_to_h2(w.x, x.x, x.y);
          f8::code4_to_h2(w.y, x.z, x.w);
          f8::code4_to_h2(w.z, y.x, y.y);
          f8::code4_to_h2(w.w, y.z, y.w);
          uint8_t *t = tile + hf * (kRows * 128);
          *reinterpret_cast<uint4 *>(t + tc::sw128(r, 2 * piece)) = x;
          *reinterpret_cast<uint4 *>(t + tc::sw128(r, 2 * piece + 1)) = y;
        }
      }
    };
    Unit un;
    int iu = 0;
    bool have = live_unit(iu, un);
    int ids = -1;
    float ks = 0.f, vs = 0.f;
    auto load_scales = [&](int h) {
      ks = vs = 0.f;
      if (noter && ids >= 0) {
        ks = __ldg(p.k_scales + (size_t)ids * p.H + h);
        vs = __ldg(p.v_scales + (size_t)ids * p.H + h);
      }
    };
    if (have) {
      ids = check_id(fetch_ids(un.s, un.c, un.cb));
      load(un.h, un.c, un.cb, ids);
      load_scales(un.h);
    }
    while (have && fine) {
      // The unit after this one that has chunks, if the scheduler has found it by
      // now. (It runs no further than two units past the one whose products it
      // issues, so behind units without chunks it may still need this one's.)
      Unit nx = un;
      bool have2 = false, known = false;
#pragma unroll 1
      while (!known && unit_there(iu)) {
        have2 = next_unit(iu, nx);
        if (have2) {
          ++iu;
          known = have2 = nx.ce > nx.cb;
        } else {
          known = true;  // there is none
        }
      }
      for (int c = un.cb; c < un.ce; ++c, ++g) {
        const int st = g % ST;
        const bool more = c + 1 < un.ce;
        int h1 = more ? un.h : nx.h;
        int c1 = more ? un.c : have2 ? nx.c : 0;  // 0: nothing to load
        int chunk1 = more ? c + 1 : nx.cb;
        int raw1 = fetch_ids(more ? un.s : nx.s, c1, chunk1);
        if (g >= ST && !wait(&empty[st], g / ST - 1)) {
          fine = false;
          break;
        }
        // what the softmax needs to know, with K (this slot's last readers, eight
        // chunks back, have passed)
        ChunkMeta &m = meta[g & (kMetaSlots - 1)];
        if (noter) {
          const float lv = vs > 0.f ? log2f(vs) : vs == 0.f ? kNoScale : vs;
          const int rows = ids >= 0 ? min(un.c - c * kChunk - lane * 16, 16) : 0;
          const uint32_t bits = rows > 0 ? (1u << rows) - 1u : 0u;
          const uint32_t pair = bits << (16 * (lane & 1));
          const uint32_t both = pair | __shfl_xor_sync(kAll, pair, 1);
          if (lane < kGroups) {
            m.ks[lane] = ks;
            m.lv[lane] = lv;
            if ((lane & 1) == 0) m.half[lane >> 2].ok[(lane >> 1) & 1] = both;
          }
        }
        if (kv) {
          // V's NaN codes become zeros (times a probability of 0 they would reach
          // every row of the tile) and their positions are noted, for the softmax
          // to read once these products are issued
          uint32_t bad = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t hit = 0;
#pragma unroll
            for (int hf = 0; hf < HALVES; ++hf) {
              const uint4 w = buf[k * HALVES + hf];
              hit |= ((w.x & 0x7f7f7f7fu) + 0x01010101u) | ((w.y & 0x7f7f7f7fu) + 0x01010101u) |
                     ((w.z & 0x7f7f7f7fu) + 0x01010101u) | ((w.w & 0x7f7f7f7fu) + 0x01010101u);
            }
            bad |= ((hit & 0x80808080u) ? 1u : 0u) << k;
          }
          uint32_t nan_byte = 0;  // lane k < 4: that of rows 8 cw + 32 k .. + 7
          if (__any_sync(kAll, bad != 0)) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t b = __ballot_sync(kAll, (bad >> k) & 1u);
              if ((b >> (lane & ~3)) & 15u) {  // the row's four lanes
#pragma unroll
                for (int hf = 0; hf < HALVES; ++hf) buf[k * HALVES + hf] = make_uint4(0, 0, 0, 0);
              }
              if (lane == k) {
#pragma unroll
                for (int i = 0; i < 8; ++i) nan_byte |= ((b >> (4 * i)) & 15u ? 1u : 0u) << i;
              }
            }
          }
          if (lane < 4) m.half[lane >> 1].nan[4 * (lane & 1) + cw] = (uint8_t)nan_byte;
        }
        put(ring + st * TILE);
        tc::fence_proxy_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[st]);
        if (!more && !known) {
          have2 = live_unit(iu, nx);
          h1 = nx.h;
          c1 = have2 ? nx.c : 0;
          chunk1 = nx.cb;
          raw1 = fetch_ids(nx.s, c1, chunk1);
        }
        ids = check_id(raw1);
        load(h1, c1, chunk1, ids);
        load_scales(h1);
      }
      un = nx;
      have = have2;
    }
  } else if (warp >= kMmaWarp) {
    regs_down<kMmaRegs>();
    const int t = warp & 1;
    const uint32_t s_col = tmem + t * kChunk, o_col = tmem + kOCol + t * D;
    Unit un;
    int iu = 0, live = 0, g0 = 0, n = 0;  // n: half chunks of this stream so far
    if (warp < kPvWarp) {
      // =============================================================== scores
      // a warp per stream, one thread of it: S of half chunk n into score tile n
      // % 2 once P V of half chunk n - 2 has read it
      constexpr uint32_t idesc = tc::idesc_f16(kRows, kHalf, false);
      const uint64_t d_q = tc::desc_sw128(smem_u32(q_sm) + (PAIR ? 0 : t * TILE), 16, 1024);
      const uint64_t d_k = tc::desc_sw128(smem_u32(k_sm), 16, 1024);
      while (fine && live_unit(iu, un)) {
        if (lane == 0) {
          const int se = un.se;
          int j = seek(t, g0, un.cb, un.sb);
          fine = wait1(&q_full[PAIR ? 0 : t], live);
          if (PAIR && j >= se) mbar_arrive(&q_free);
#pragma unroll 1
          while (fine && j < se) {
            const int g = g0 + (j >> 1) - un.cb, st = g % ST, b = n & 1;
            fine = wait1(&k_full[st], g / ST) && (n < 2 || wait1(&pv_done[t][b], (n >> 1) - 1));
            if (!fine) break;
            tc::fence_after();
            const uint64_t kd = tc::desc_advance(d_k, st * TILE + (j & 1) * kHalf * 128);
            const uint32_t sc = s_col + b * kHalf;
#pragma unroll
            for (int hf = 0; hf < HALVES; ++hf)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                const uint32_t off = hf * (kRows * 128) + kk * 32;
                const uint64_t bd = tc::desc_advance(kd, off);
                tc::mma_f16(sc, tc::desc_advance(d_q, off), bd, idesc, hf + kk > 0);
                if constexpr (PAIR)
                  tc::mma_f16(sc, tc::desc_advance(d_q, off + TILE), bd, idesc, true);
              }
            tc::commit(&s_full[t][b]);
            if ((j & 1) || j + 1 >= se) tc::commit(&k_free[st]);
            j = seek(t, g0, un.cb, j + 1);
            if (PAIR && j >= se) tc::commit(&q_free);
            mbar_arrive(&s_full[t][b]);
            ++n;
          }
        }
        fine = __all_sync(kAll, fine);
        g0 += un.ce - un.cb;
        ++live;
      }
    } else {
      // ================================================================= P V
      // a warp per stream, one thread of it; the first one also finds the
      // CTA's units, two ahead of its own
      constexpr uint32_t idesc = tc::idesc_f16(kRows, D, true);
      const uint64_t d_v = tc::desc_sw128(smem_u32(v_sm), kRows * 128, 1024);
      Walk walk;
      int n_units = 0, pieces = 1, i_pub = 0;
      bool all_pub = false;
      auto publish_unit = [&]() {
        if (all_pub || !fine) return;
        Unit nu;
        unit_at(p, walk, blockIdx.x + i_pub * gridDim.x, n_units, pieces, nu);
        const int k = i_pub & (kUnitSlots - 1);
        if (i_pub >= kUnitSlots && !wait(&u_free[k], i_pub / kUnitSlots - 1)) {
          fine = false;
          return;
        }
        if (lane == 0) {
          units_s[k] = nu;
          mbar_arrive(&u_full[k]);
        }
        __syncwarp();
        ++i_pub;
        all_pub = nu.id < 0;
      };
      if (t == 0) {
        int n_tiles, max_chunks;
        count_tiles(p, n_tiles, max_chunks);
        n_units = n_tiles * p.H;
        pieces = pieces_of(p, n_units, max_chunks, gridDim.x);
        if (blockIdx.x == 0 && lane == 0 && p.rec_units > 0) {
          p.rec_hdr[0] = n_units;
          p.rec_hdr[1] = pieces;
        }
      }
#pragma unroll 1
      for (;; ++iu) {
        // units up to two past this one are known to the other roles
        if (t == 0) {
#pragma unroll 1
          while (i_pub < iu + 3 && !all_pub && fine) publish_unit();
        }
        if (!fine || !next_unit(iu, un)) break;
        if (lane == 0) {
          const int se = un.se;
          int j = seek(t, g0, un.cb, un.sb);
          bool acc = false;
#pragma unroll 1
          while (fine && j < se) {
            const int g = g0 + (j >> 1) - un.cb, st = g % ST, b = n & 1;
            fine = wait1(&v_full[st], g / ST) && wait1(&p_full[t][b], n >> 1);
            if (!fine) break;
            tc::fence_after();
            const uint64_t vd = tc::desc_advance(d_v, st * TILE + (j & 1) * kHalf * 128);
            const uint32_t pc = s_col + b * kHalf;
#pragma unroll
            for (int kk = 0; kk < kHalf / 16; ++kk) {
              // P of positions [16 kk, 16 kk + 16): 8 columns of its 32-column piece
              const uint32_t pk = pc + (kk >> 1) * 32 + (kk & 1) * 8;
              const uint64_t bd = tc::desc_advance(vd, kk * 2048);
              tc::mma_f16_ts(o_col, pk, bd, idesc, acc || kk > 0);
              if constexpr (PAIR) tc::mma_f16_ts(o_col, pk + 16, bd, idesc, true);
            }
            acc = true;
            tc::commit(&pv_done[t][b]);
            mbar_arrive(&pv_done[t][b]);
            if ((j & 1) || j + 1 >= se) tc::commit(&v_free[st]);
            j = seek(t, g0, un.cb, j + 1);
            if (j >= se) {
              tc::commit(&o_full[t]);
              mbar_arrive(&o_full[t]);
            }
            ++n;
          }
        }
        fine = __all_sync(kAll, fine);
        g0 += un.ce - un.cb;
      }
    }
    // every product has completed before tensor memory is released
    if (lane == 0) tc::commit(&drain);
    __syncwarp();
    if (!wait(&drain, 0)) fine = false;
  } else {
    regs_up<kSoftRegs>();
    // ================================================================ softmax
    const int t = warp >> 2, r = tid & (kRows - 1);
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_t = tmem + lanes + t * kChunk, o_t = tmem + lanes + kOCol + t * D;
    const int ur = PAIR ? r : t * kRows + r;  // row of the unit
    const int ur_q = ur * p.g_inv >> 16, ur_h = ur - ur_q * p.G;
    int n_s = 0;                              // score tiles of this stream so far
    int live = 0, g0 = 0, n_o = 0;
    Unit un;
    // The unit's Q as operand rows, D / 8 lanes a row: rows 32 warp .. + 31 of
    // the unit (PAIR: 16 warp .. + 15, for both streams). The elements are
    // copied asynchronously to where their f16 parts go (8 16-bit elements take
    // the room of 8 f16, 8 float32 that of two parts) and converted there, each
    // by the lane that copied it. Each row is scaled by a power of two that
    // brings its largest value to [2^11, 2^12), as in the decode, and by the sign
    // of the softmax scale, so the factor on scores is not negative.
    auto put_q = [&](const Unit &un, int parity) {
      constexpr int LPR = D / 8, RPI = 32 / LPR, NB = (PAIR ? 16 : 32) / RPI;
      constexpr int ES = PAIR ? 4 : 2;
      const int l = lane % LPR, r0 = (PAIR ? 16 : 32) * warp + lane / LPR;
      const uint8_t *q_l = reinterpret_cast<const uint8_t *>(p.q) +
                           (((size_t)un.q0 * p.Hq + (size_t)un.h * p.G) * D + 8 * l) * ES;
      uint8_t *d_l = q_sm + (l >> 3) * (kRows * 128);
      auto at = [&](int qr) -> uint8_t * {
        return d_l + (qr >> 7) * TILE + tc::sw128(qr & (kRows - 1), l & 7);
      };
#pragma unroll 1
      for (int i = 0; i < NB; ++i) {
        const int qr = r0 + i * RPI, uj = qr * p.g_inv >> 16, j = un.qt * p.tq + uj;
        const int ok = uj < p.tq && j < un.n ? 16 : 0;  // else zero-filled
        const uint8_t *src = ok ? q_l + ((size_t)j * p.Hq + (qr - uj * p.G)) * (D * ES) : q_l;
        const uint32_t dst = smem_u32(at(qr));
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok)
                     : "memory");
        if constexpr (PAIR)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + TILE),
                       "l"(src + 16), "r"(ok)
                       : "memory");
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll 1
      for (int i = 0; i < NB; ++i) {
        const int qr = r0 + i * RPI;
        uint8_t *d = at(qr);
        f8::Raw8<DT> x;
        x.w[0] = *reinterpret_cast<const uint4 *>(d);
        if constexpr (PAIR) x.w[1] = *reinterpret_cast<const uint4 *>(d + TILE);
        float v[8];
        x.get(v);
        float qmax = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) qmax = fmaxf(qmax, fabsf(v[e]));
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1) qmax = fmaxf(qmax, __shfl_xor_sync(kAll, qmax, o));
        const int ef = (int)(__float_as_uint(qmax) >> 23);
        const int fe = min(max(265 - ef, 1), 253);
        float f = qmax > 0.f ? __uint_as_float((uint32_t)fe << 23) : 1.f;
        if (l == 0) qfac_s[parity][qr] = fabsf(p.qscale) / f;
        if (p.qscale < 0.f) f = -f;
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (PAIR)
            split_h2(v[2 * e] * f, v[2 * e + 1] * f, hi[e], lo[e]);
          else
            hi[e] = h2_bits(__floats2half2_rn(v[2 * e] * f, v[2 * e + 1] * f));
        }
        *reinterpret_cast<uint4 *>(d) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        if constexpr (PAIR)
          *reinterpret_cast<uint4 *>(d + TILE) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
      tc::fence_proxy_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[PAIR ? 0 : t]);
    };
    // 32 rows x 64 bytes a warp, at a pitch of 80 bytes (8 lanes' 16-byte parts
    // on distinct banks): output rows pass through it so that a store
    // instruction covers 64 consecutive bytes of 8 rows
    uint8_t *o_sm = v_sm + ST * TILE + warp * (32 * 80);
    // a first round without a unit brings the first unit's Q
    int iu = -1;
    bool more = true;
    un.id = -1;
    un.n = un.cb = un.ce = un.sb = un.se = un.s = un.h = un.qt = un.c = un.q0 = 0;
    un.pieces = 1;
#pragma unroll 1
    while (fine && more) {
      const int j_q = un.qt * p.tq + ur_q, hd = un.h * p.G + ur_h;
      const bool row_in = ur_q < p.tq && j_q < un.n;
      const int i_row = un.q0 + j_q;
      int lo = 0, hi = 0;
      if (row_in) row_span(p, i_row, max(min(un.c - un.n + j_q + 1, un.c), 0), lo, hi);
      const int nch = un.ce - un.cb, cb = un.cb, id = un.id, pieces = un.pieces;
      const int sb_u = un.sb, se_u = un.se;
      const int j0_q = un.qt * p.tq, n_q = un.n;
      const size_t obase = ((size_t)un.q0 * p.Hq + (size_t)un.h * p.G) * D;
      float m_run = -INFINITY, l_run = 0.f, lv_ref = kNoScale;
      bool poison = false;
      const int se = se_u, first = seek(t, g0, cb, sb_u);
      float qfac = 0.f;
      // the scores of the n-th tile: once it is complete, then half by half
      float v[2][32];
      auto scores = [&](int n, int i) {
        if (i == 0) {
          fine = wait(&s_full[t][n & 1], n >> 1) && fine;
          tc::fence_after();
        }
        ld32(s_t + (n & 1) * kHalf + 32 * i, v[i]);
      };
      // this row's readable positions among [pos0, pos0 + 32), holes apart
      auto row_mask = [&](int pos0) -> uint32_t {
        uint32_t mk = 0u;
        auto add = [&](int x, int y) {  // positions [x, y)
          const int a = max(x - pos0, 0), b = min(y - pos0, 32);
          if (b > a) mk |= (0xffffffffu >> (32 - b)) & (0xffffffffu << a);
        };
        if (!p.kv_map) {
          add(lo, hi);
        } else if (row_in) {
#pragma unroll 1
          for (int q = 0; q < MT_KV_MAP_MAX_SPANS; ++q) {
            const int32_t *run = p.kv_map + ((size_t)i_row * MT_KV_MAP_MAX_SPANS + q) * 2;
            if (run[1] > 0)
              add(max(run[0], 0), (int)min((long long)run[0] + run[1], (long long)hi));
          }
        }
        return mk;
      };
      // half chunk jx (-1: none): a NaN among the V that this row reads there.
      // The note is there once the half chunk's P V has been issued, which the
      // scores of two tiles later, or the end of the unit's products, tell
      auto check_nan = [&](int jx) {
        if (jx < 0) return;
        const auto &hf = meta[(g0 + (jx >> 1) - cb) & (kMetaSlots - 1)].half[jx & 1];
        const uint2 nan = *reinterpret_cast<const uint2 *>(hf.nan);
        if (nan.x | nan.y)
          poison = poison || (nan.x & row_mask(jx * kHalf)) || (nan.y & row_mask(jx * kHalf + 32));
      };
      int j1 = -1, j2 = -1;  // this stream's half chunks one and two back
      // 16-bit: loaded a tile ahead, each half into the registers that the same
      // half of the tile before has just left (float32 has none to spare)
      if (!PAIR && first < se) {
        scores(n_s, 0);
        scores(n_s, 1);
      }
#pragma unroll 1
      for (int j = first, j_n; fine && j < se; j = j_n, ++n_s) {
        j_n = seek(t, g0, cb, j + 1);
        if constexpr (PAIR) {
          scores(n_s, 0);
          scores(n_s, 1);
        }
        if (j == first) qfac = qfac_s[live & 1][ur];
        const uint32_t s_j = s_t + (n_s & 1) * kHalf;
        const ChunkMeta &m = meta[(g0 + (j >> 1) - cb) & (kMetaSlots - 1)];
        const float4 ks4 = reinterpret_cast<const float4 *>(m.ks)[j & 1];
        const float4 lv4 = reinterpret_cast<const float4 *>(m.lv)[j & 1];
        const uint2 hf2 = *reinterpret_cast<const uint2 *>(m.half[j & 1].ok);
        // factors of the four groups' scores; not zero, so that the -inf of masked
        // positions stays -inf
        const float f[4] = {fmaxf(qfac * ks4.x, 1e-37f), fmaxf(qfac * ks4.y, 1e-37f),
                            fmaxf(qfac * ks4.z, 1e-37f), fmaxf(qfac * ks4.w, 1e-37f)};
        const float lv[4] = {lv4.x, lv4.y, lv4.z, lv4.w};
        const float lv_max = fmaxf(max3f(lv[0], lv[1], lv[2]), lv[3]);
        const int pos0 = j * kHalf;
        // every position readable for this row
        const bool open = (hf2.x & hf2.y) == 0xffffffffu && lo <= pos0 && hi >= pos0 + kHalf &&
                          !p.kv_map;
        check_nan(j2);
        j2 = j1;
        j1 = j;
        landed(v[0]);
        landed(v[1]);
        if (!open) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t mk = row_mask(pos0 + 32 * i) & (i ? hf2.y : hf2.x);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[i][e] = (mk >> e) & 1u ? v[i][e] : -INFINITY;
          }
        }
        // ---- running maximum
        float mx = -INFINITY;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float *x = v[q >> 1] + 16 * (q & 1);
          float a = max3f(x[0], x[1], x[2]), b = max3f(x[3], x[4], x[5]);
          a = max3f(a, x[6], x[7]);
          b = max3f(b, x[8], x[9]);
          a = max3f(a, x[10], x[11]);
          b = max3f(b, x[12], x[13]);
          a = max3f(a, x[14], x[15]);
          mx = fmaxf(mx, fmaxf(a, b) * f[q]);
        }
        // O is rescaled when a row's maximum grows past 2^8 (or it has its first
        // finite score), or when sV passes 4 v_ref
        const bool grow = mx > m_run + 8.f || (m_run == -INFINITY && mx != -INFINITY) ||
                          lv_max > lv_ref + 2.f;
        if (__any_sync(kAll, grow)) {
          const float m_new = fmaxf(m_run, mx), lv_new = fmaxf(lv_ref, lv_max);
          const float al = m_run == -INFINITY ? 0.f : ex2(m_run - m_new);
          l_run *= al;
          const float so = al * ex2(lv_ref - lv_new);
          m_run = m_new;
          lv_ref = lv_new;
          if (j > first) {
            // the products of the half chunk before have completed
            fine = wait(&pv_done[t][(n_s - 1) & 1], (n_s - 1) >> 1) && fine;
            tc::fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              float o[16];
              tc::ld16(o_t + c, o);
              tc::wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] *= so;
              tc::st16(o_t + c, o);
            }
            tc::wait_st();
          }
        }
        // ---- probabilities over the scores. Exponent: score * f + log2(sV /
        // v_ref) + 5 - max; the row's sum takes the V scale out again
        const float mr = m_run == -INFINITY ? 0.f : m_run;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t h[16], l[PAIR ? 16 : 1];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const float lw = fmaxf(lv[2 * i + q] - lv_ref, -60.f) + kPBits;
            const float2 ff = make_float2(f[2 * i + q], f[2 * i + q]);
            const float2 ad = make_float2(lw - mr, lw - mr);
            float2 s0 = make_float2(0.f, 0.f), s1 = s0;
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              float2 y = f2_fma(make_float2(v[i][16 * q + e], v[i][16 * q + e + 1]), ff, ad);
              y.x = ex2(y.x);
              y.y = ex2(y.y);
              if (e & 2)
                s1 = f2_add(s1, y);
              else
                s0 = f2_add(s0, y);
              if constexpr (PAIR)
                split_h2x(y, h[8 * q + e / 2], l[8 * q + e / 2]);
              else
                h[8 * q + e / 2] = h2_bits(__floats2half2_rn(y.x, y.y));
            }
            s0 = f2_add(s0, s1);
            l_run = fmaf(s0.x + s0.y, ex2(-lw), l_run);
          }
          tc::st16u(s_j + 32 * i, h);
          if constexpr (PAIR) tc::st16u(s_j + 32 * i + 16, l);
          if (!PAIR && j_n < se) scores(n_s + 1, i);
        }
        tc::wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[t][n_s & 1]);
      }
      // ---- the next unit's Q, while the last products run (its rows' last
      // scores have been read: this stream's, or (PAIR) both streams')
      const bool had = first < se;
      if (nch > 0) ++live;
      if (fine) more = next_unit(++iu, un);
      if (fine && more && un.ce > un.cb) {
        if (PAIR && live > 0) fine = wait(&q_free, live - 1);
        if (fine) put_q(un, live & 1);
      }
      // ---- the unit's rows
      if (had && fine) {
        fine = wait(&o_full[t], n_o);
        ++n_o;
        tc::fence_after();
        check_nan(j2);
        check_nan(j1);
      }
      if (!PAIR && !fine) break;
      if (poison) l_run = __int_as_float(0x7fffffff);
      float m_row = m_run, l_row = l_run;
      // factors of the two accumulators (stream A's thread writes the row when
      // the streams share it)
      float fa = had ? ex2(lv_ref - kPBits) : 0.f, fb = 0.f;
      bool writer = true, b_has = false;
      if constexpr (PAIR) {
        if (t == 1) ml_s[r] = make_float4(m_run, l_run, lv_ref, 0.f);
        // (a wait that ran out in any warp ends the loop of all)
        fine = softmax_sync_and(fine);
        if (!fine) break;
        if (t == 0) {
          const float4 o = ml_s[r];
          b_has = seek(1, g0, cb, sb_u) < se;
          m_row = fmaxf(m_run, o.x);
          // a part without a position has sum 0 (or NaN): weight 1 keeps it
          const float wa = m_run == -INFINITY ? (l_run == 0.f ? 0.f : 1.f) : ex2(m_run - m_row);
          const float wb = o.x == -INFINITY ? (o.y == 0.f ? 0.f : 1.f) : ex2(o.x - m_row);
          l_row = l_run * wa + o.y * wb;
          fa *= wa;
          fb = b_has ? wb * ex2(o.z - kPBits) : 0.f;
        } else {
          writer = false;
        }
      }
      if (writer && id >= 0) {
        const bool split = pieces > 1;
        const float inv = split ? 1.f : l_row == 0.f ? 0.f : 1.f / l_row;
        fa *= inv;
        fb *= inv;
        float *rr = split ? p.rec + ((size_t)id * C::UNIT_ROWS + ur) * (D + 4) : nullptr;
        // 64 bytes of every row a step; this lane stores part lane % 4 of rows
        // lane / 4 + 8 i of its warp
        constexpr int NC = PAIR ? 16 : 32, ES = PAIR ? 4 : 2;
        uint8_t *dst[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int rr2 = (ur & ~31) + 8 * i + (lane >> 2);
          const int uj = rr2 * p.g_inv >> 16, jq = j0_q + uj;
          dst[i] = uj < p.tq && jq < n_q
                       ? reinterpret_cast<uint8_t *>(p.out) +
                             (obase + ((size_t)jq * p.Hq + (rr2 - uj * p.G)) * D) * ES +
                             (lane & 3) * 16
                       : nullptr;
        }
#pragma unroll 1
        for (int c = 0; c < D; c += NC) {
          float o[NC], w[PAIR ? NC : 1];
          if constexpr (PAIR) {
            tc::ld16(o_t + c, o);
            tc::ld16(o_t + D + c, w);
          } else {
            ld32(o_t + c, o);
          }
          tc::wait_ld();
          // an accumulator that no product wrote in this unit is not used
#pragma unroll
          for (int e = 0; e < NC; ++e) {
            o[e] = had ? o[e] * fa : 0.f;
            if constexpr (PAIR) o[e] = b_has ? o[e] + w[e] * fb : o[e];
          }
          if (split) {
#pragma unroll
            for (int e = 0; e < NC; e += 4)
              f8::store4<MT_F32>(rr + 4, c + e, o[e], o[e + 1], o[e + 2], o[e + 3]);
          } else {
            uint4 *so = reinterpret_cast<uint4 *>(o_sm + lane * 80);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float *x = o + i * (NC / 4);
              if constexpr (PAIR)
                so[i] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]),
                                   __float_as_uint(x[2]), __float_as_uint(x[3]));
              else
                so[i] = make_uint4(f8::pack2<DT>(x[0], x[1]), f8::pack2<DT>(x[2], x[3]),
                                   f8::pack2<DT>(x[4], x[5]), f8::pack2<DT>(x[6], x[7]));
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (dst[i])
                *reinterpret_cast<uint4 *>(dst[i] + c * ES) = *reinterpret_cast<const uint4 *>(
                    o_sm + (8 * i + (lane >> 2)) * 80 + (lane & 3) * 16);
            __syncwarp();
          }
        }
        if (split)
          *reinterpret_cast<float4 *>(rr) = make_float4(
              m_row, l_row, __int_as_float(row_in ? i_row * p.Hq + hd : -1), 0.f);
        else if (row_in && p.lse)
          p.lse[(size_t)i_row * p.Hq + hd] =
              l_row == 0.f ? -INFINITY : (m_row + log2f(l_row)) * 0.69314718055994530942f;
      }
      // the accumulators have been read before the next unit's first P
      tc::fence_before();
      if constexpr (PAIR) softmax_sync_and(true);
      g0 += nch;
    }
  }
  if (!fine) {
    abort_s = 1;  // the other roles stop waiting within a few polls
    if (lane == 0) report(p.status, MT_STATUS_BIT_TIMEOUT);
  }
  tc::fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after();
    tc::dealloc(tmem, kTmemCols);
  }
}

// Merge the pieces of split units: a warp per row, a lane per D / 32 dims.
template <int D, int DT>
__global__ void __launch_bounds__(256)
    prefill_f8_merge_kernel(const __grid_constant__ PrefillF8Params p, int unit_rows) {
  constexpr int DV = D / 32;
  pdl_enter();
  const int n_units = p.rec_hdr[0], pieces = p.rec_hdr[1];
  if (pieces <= 1) return;
  const int lane = threadIdx.x & 31;
  const size_t pitch = (size_t)unit_rows * (D + 4);
  const long long rows = (long long)n_units * unit_rows;
  for (long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); w < rows;
       w += (long long)gridDim.x * 8) {
    const long long unit = w / unit_rows;
    const int row = (int)(w % unit_rows);
    const float *rr = p.rec + (size_t)unit * pieces * pitch + (size_t)row * (D + 4);
    float m = -INFINITY, l = 0.f;
    int dst = -1;
    if (lane < pieces) {
      const float4 hd = __ldcg(reinterpret_cast<const float4 *>(rr + lane * pitch));
      m = hd.x;
      l = hd.y;
      dst = __float_as_int(hd.z);
    }
    dst = __shfl_sync(kAll, dst, 0);
    if (dst < 0) continue;
    float M = m;
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kAll, M, o));
    // a piece that saw nothing weighs 0; one whose sum is NaN keeps it
    const float f = m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : ex2(m - M);
    float L = l * f;
#pragma unroll
    for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(kAll, L, o);
    float acc[DV];
#pragma unroll
    for (int e = 0; e < DV; ++e) acc[e] = 0.f;
#pragma unroll 4
    for (int k = 0; k < pieces; ++k) {
      const float fk = __shfl_sync(kAll, f, k);
#pragma unroll
      for (int e = 0; e < DV; e += 2) {
        const float2 x =
            __ldcg(reinterpret_cast<const float2 *>(rr + k * pitch + 4 + lane * DV + e));
        acc[e] += fk != 0.f ? fk * x.x : 0.f;
        acc[e + 1] += fk != 0.f ? fk * x.y : 0.f;
      }
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const size_t o = (size_t)dst * D + lane * DV;
    if constexpr (DT == MT_F32) {
#pragma unroll
      for (int e = 0; e < DV; e += 2)
        *reinterpret_cast<float2 *>(reinterpret_cast<float *>(p.out) + o + e) =
            make_float2(acc[e] * inv, acc[e + 1] * inv);
    } else {
#pragma unroll
      for (int e = 0; e < DV; e += 2)
        reinterpret_cast<uint32_t *>(p.out)[(o + e) / 2] =
            f8::pack2<DT>(acc[e] * inv, acc[e + 1] * inv);
    }
    if (p.lse && lane == 0)
      p.lse[dst] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994530942f;
  }
}

// --------------------------------------------------------------------- host

struct Plan {
  PrefillF8Params p;
  int ctas, unit_rows;
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
  if (c.head_dim == 256) return fail(MT_ERR_UNSUPPORTED, w + "head_dim must be 64 or 128");
  if (a->n_tokens < 0) return fail(MT_ERR_INVALID_ARG, w + "negative n_tokens");
  if (a->spans && a->kv_map)
    return fail(MT_ERR_INVALID_ARG, w + "at most one of spans and kv_map");
  if (c.n_seqs > 0 && a->n_tokens > 0 && (!a->q || !a->out || !a->q_start))
    return fail(MT_ERR_INVALID_ARG, w + "null pointer");
  if (!aligned16(a->q) || !aligned16(a->out))
    return fail(MT_ERR_INVALID_ARG, w + "q and out must be 16-byte aligned");
  DeviceInfo di;
  st = device_info(&di);
  if (st != MT_OK) return st;
  PrefillF8Params &p = pl->p;
  p = PrefillF8Params{};
  p.k_pool = c.k_pool;
  p.v_pool = c.v_pool;
  p.k_scales = c.k_scales;
  p.v_scales = c.v_scales;
  p.table = c.block_table;
  p.ctx = c.context_lens;
  p.q_start = a->q_start;
  p.spans = a->spans;
  p.kv_map = a->kv_map;
  p.q = a->q;
  p.out = a->out;
  p.lse = a->lse;
  p.B = c.n_seqs;
  p.Hq = a->n_heads;
  p.H = c.n_kv_heads;
  p.G = a->n_heads / c.n_kv_heads;
  p.n_tok = a->n_tokens;
  p.max_blocks = c.max_blocks;
  p.bs_shift = c.block_size == 32 ? 5 : 4;
  p.n_phys = c.n_phys_blocks;
  p.qscale = a->scale * 1.44269504088896340736f;
  pl->unit_rows = a->dtype == MT_F32 ? kRows : 2 * kRows;
  p.tq = pl->unit_rows / p.G;
  p.g_inv = (65536 + p.G - 1) / p.G;
  // units: at most n_tokens / tq + n_seqs tiles (and no more than rows) a head
  const long long tiles = std::min<long long>(a->n_tokens, a->n_tokens / p.tq + (long long)p.B);
  const long long units = tiles * p.H;
  if (units > (0x7fffffffLL / kMaxSplit) || (long long)a->n_tokens * p.Hq > 0x7fffffffLL)
    return fail(MT_ERR_UNSUPPORTED, w + "too many query rows");
  pl->ctas = di.n_sm;
  // units are cut only when full tiles are fewer than CTAs and contexts may
  // have several chunks
  const long long longest = ((long long)p.max_blocks * c.block_size + kChunk - 1) / kChunk;
  const bool few = (long long)(a->n_tokens / p.tq) * p.H < pl->ctas;
  p.rec_units = longest > 1 && few ? 4 * pl->ctas : 0;
  pl->ws = kHdrBytes + (size_t)p.rec_units * pl->unit_rows * (c.head_dim + 4) * sizeof(float);
  return MT_OK;
}

template <int D, int DT>
mt_status launch(const Plan &pl, cudaStream_t s) {
  auto kern = prefill_f8_kernel<D, DT>;
  constexpr int smem = Cfg<D, DT == MT_F32>::SMEM;
  mt_status st = kernel_smem(reinterpret_cast<const void *>(kern), smem,
                             "cudaFuncSetAttribute(f8 prefill smem)");
  if (st != MT_OK) return st;
  // the warpgroups' register shares are drawn from what the launch allocates
  static const int regs = [kern] {
    cudaFuncAttributes at;
    return cudaFuncGetAttributes(&at, kern) == cudaSuccess ? at.numRegs : 0;
  }();
  if (regs < kLaunchRegs) return fail(MT_ERR_UNSUPPORTED, "f8 prefill: built with too few registers");
  st = cuda_check(launch_pdl(kern, dim3(pl.ctas), dim3(kThreads), smem, s, pl.p),
                  "f8 prefill launch");
  if (st != MT_OK || pl.p.rec_units == 0) return st;
  return cuda_check(launch_pdl(prefill_f8_merge_kernel<D, DT>, dim3(4 * pl.ctas), dim3(256), 0, s,
                               pl.p, pl.unit_rows),
                    "f8 prefill merge launch");
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

extern "C" size_t mt_paged_attn_prefill_f8_workspace_bytes(const mt_f8_attn_args *a) {
  Plan pl;
  return make_plan(a, "mt_paged_attn_prefill_f8_workspace_bytes", &pl) == MT_OK ? pl.ws : 0;
}

extern "C" mt_status mt_paged_attn_prefill_f8(const mt_f8_attn_args *a, void *workspace,
                                              size_t workspace_bytes, mt_stream stream) {
  Plan pl;
  mt_status st = make_plan(a, "mt_paged_attn_prefill_f8", &pl);
  if (st != MT_OK) return st;
  if (!workspace || workspace_bytes < pl.ws || !aligned16(workspace))
    return fail(MT_ERR_INVALID_ARG,
                "mt_paged_attn_prefill_f8: workspace missing, too small or not 16-byte aligned");
  if (a->cache.n_seqs == 0 || a->n_tokens == 0) return ok();
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  pl.p.status = reinterpret_cast<uint32_t *>(ws);
  pl.p.rec_hdr = reinterpret_cast<int *>(ws + 128);
  pl.p.rec = reinterpret_cast<float *>(ws + kHdrBytes);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  st = a->cache.head_dim == 64 ? launch_dt<64>(pl, a->dtype, s) : launch_dt<128>(pl, a->dtype, s);
  return st == MT_OK ? ok() : st;
}
