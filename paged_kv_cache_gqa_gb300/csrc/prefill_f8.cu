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
//  * 4 converter warps read a chunk's codes from global memory into registers
//    (16 bytes a lane, a chunk ahead), turn them into f16 (exact) and write
//    them as swizzled operand tiles; rows of holes and past the context
//    become zeros. They also lay out the next unit's Q, each row scaled by a
//    power of two so that its largest value lies in [2^11, 2^12).
//  * One warp issues all products: S = Q K^T (both from shared memory) into
//    the stream's score columns of tensor memory, O += P V with P from tensor
//    memory over the scores it came from.
//  * 2 x 4 softmax warps, a thread per row: sK and the row's factor multiply
//    the scores inside the exponent's fused multiply-add; sV enters as an
//    addend of the exponent, log2(sV / v_ref), so neither costs an operation
//    per element; the row's sum takes it out again once per 16 columns.
//    O is rescaled only when the running maximum grows by more than 2^8 or
//    sV passes 4 v_ref, so probabilities stay below 2^15 as f16.
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
constexpr int kConvWarp = 8;          // warps 0..3: stream A, 4..7: B, 8..11: converters
constexpr int kMmaWarp = 12;
constexpr int kThreads = 32 * 13;
constexpr int kMetaSlots = 4;
constexpr uint32_t kTmemCols = 512;   // scores A, B: [0, 256); outputs A, B: [256, 512)
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
  static constexpr int SMEM = 1024 + 2 * TILE + 2 * STAGES * TILE;
};
static_assert(Cfg<128, false>::SMEM + 4096 <= 227 * 1024, "shared memory");
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

// Whether the phase with `parity` has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; "
      "selp.u32 %0, 1, 0, p; }"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
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

// A unit of work: up to UNIT_ROWS rows of one KV head, chunks [cb, ce).
struct Unit {
  int s, h, qt;    // sequence, KV head, tile of tq queries
  int n, c, q0;    // queries and (clamped) context of the sequence, its first row
  int cb, ce;
  int id;          // unit * pieces + piece
};

// Walks the units of one CTA in order; every warp keeps its own.
struct Walk {
  int s = 0, base = 0;  // sequence s starts with tile `base`
};

__device__ __forceinline__ int tiles_of(const PrefillF8Params &p, int s, bool flag) {
  const int q0 = p.q_start[s], q1 = p.q_start[s + 1], n = q1 - q0;
  const bool bad = n < 0 || (n > 0 && (q0 < 0 || q1 > p.n_tok));
  if (flag && (bad || (n > 0 && (n > p.ctx[s] || p.ctx[s] > (p.max_blocks << p.bs_shift)))))
    report(p.status, MT_STATUS_BIT_DEVICE_CHECK);
  return bad || n == 0 ? 0 : (n + p.tq - 1) / p.tq;
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

// Unit piece `u` of the launch (false: none): whole warp, same in every warp.
__device__ __forceinline__ bool unit_at(const PrefillF8Params &p, Walk &w, int u, int n_units,
                                        int pieces, Unit &un) {
  if (u >= n_units * pieces) return false;
  const int lane = threadIdx.x & 31;
  const int tile = u / pieces / p.H;
  un.h = u / pieces % p.H;
  un.id = u;
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
  un.cb = c0 + (int)((long long)piece * nch / pieces);
  un.ce = c0 + (int)((long long)(piece + 1) * nch / pieces);
  return true;
}

// What the converters tell the softmax about a chunk.
struct ChunkMeta {
  float ks[kGroups];   // K scale of each group of 16 positions
  float lv[kGroups];   // log2 of the V scale
  uint32_t ok[4];      // positions that hold data
  uint8_t nan[16];     // positions whose V holds a NaN (staged as zeros): byte 4 k + w
                       // is positions 32 k + 8 w .. + 7, written by converter warp w
};

template <int D, int DT>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_f8_kernel(const __grid_constant__ PrefillF8Params p) {
  constexpr bool PAIR = DT == MT_F32;
  using C = Cfg<D, PAIR>;
  constexpr int ST = C::STAGES, TILE = C::TILE, HALVES = C::HALVES;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ uint32_t tmem_slot;
  __shared__ __align__(8) uint64_t q_full, q_free, k_full[ST], k_free[ST], v_full[ST], v_free[ST],
      s_full[2], p_full[2], o_full[2], drain;
  __shared__ __align__(16) ChunkMeta meta[kMetaSlots];
  __shared__ float qfac_s[2][2 * kRows];   // by live unit parity: the row's factor on scores
  __shared__ float4 ml_s[kRows];           // stream B's max, sum, log2 v_ref, NaN flag
  __shared__ int abort_s;
  uint8_t *base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t *q_sm = base;                    // two tiles: streams A, B; or high, low parts
  uint8_t *k_sm = base + 2 * TILE, *v_sm = k_sm + ST * TILE;
  pdl_enter();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  int n_tiles, max_chunks;
  count_tiles(p, n_tiles, max_chunks);
  const int n_units = n_tiles * p.H;
  const int pieces = pieces_of(p, n_units, max_chunks, gridDim.x);
  if (blockIdx.x == 0 && tid == 0 && p.rec_units > 0) {
    p.rec_hdr[0] = n_units;
    p.rec_hdr[1] = pieces;
  }
  if ((int)blockIdx.x >= n_units * pieces) return;
  if (tid == 0) {
    mbar_init(&q_full, 4);
    mbar_init(&q_free, 1);
    for (int k = 0; k < ST; ++k) {
      mbar_init(&k_full[k], 4);
      mbar_init(&k_free[k], 1);
      mbar_init(&v_full[k], 4);
      mbar_init(&v_free[k], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 2);  // the products' commit and the issuing thread
      mbar_init(&p_full[t], 4);
      mbar_init(&o_full[t], 1);
    }
    mbar_init(&drain, 1);
    abort_s = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tc::alloc(&tmem_slot, kTmemCols);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = tmem_slot;
  Walk walk;
  bool fine = true;
  // the same answer in every lane of the warp
  auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
    return __all_sync(kAll, mbar_wait_bounded(bar, parity & 1u, &abort_s, kWaitNs));
  };
  // jobs (products of one stream with one chunk) of a unit; job j is stream j % 2
  auto jobs_of = [&](const Unit &un) -> int { return (un.ce - un.cb) * (PAIR ? 1 : 2); };
  auto chunk_of = [&](int j) -> int { return PAIR ? j : j >> 1; };

  if (warp >= kConvWarp && warp < kMmaWarp) {
    // =========================================================== converters
    const int cw = warp - kConvWarp;
    const int r_l = 8 * cw + (lane >> 2);  // rows r_l + 32 k
    const int piece = lane & 3;            // 16 bytes of a 64-byte half row
    const size_t row = (size_t)p.H * D;
    uint4 kb[4 * HALVES], vb[4 * HALVES];
    int g = 0;                             // chunks converted so far
    int live = 0;                          // units with chunks so far
    // physical blocks of a chunk: lane l holds that of positions 16 l .. 16 l + 15
    auto fetch_ids = [&](const Unit &un, int c) -> int {
      const int pos = c * kChunk + lane * 16;
      if (lane >= kGroups || pos >= un.c) return -1;
      const int id = p.table[(size_t)un.s * p.max_blocks + (pos >> p.bs_shift)];
      if (id < -1 || (long long)id >= p.n_phys) {
        report(p.status, MT_STATUS_BIT_DEVICE_CHECK);
        return -1;
      }
      return id;
    };
    auto load = [&](const uint8_t *pool, const Unit &un, int c, int ids, uint4 (&b)[4 * HALVES]) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = r_l + 32 * k, pos = c * kChunk + r;
        const int id = __shfl_sync(kAll, ids, r >> 4);
        const bool have = id >= 0 && pos < un.c;
        const uint8_t *src = pool +
                             (((size_t)max(id, 0) << p.bs_shift) + (pos & ((1 << p.bs_shift) - 1))) *
                                 row +
                             (size_t)un.h * D + piece * 16;
#pragma unroll
        for (int hf = 0; hf < HALVES; ++hf)
          b[k * HALVES + hf] = have ? __ldg(reinterpret_cast<const uint4 *>(src + 64 * hf))
                                    : make_uint4(0, 0, 0, 0);
      }
    };
    // codes -> f16 operand rows: 16 codes are the 16-byte units 2 piece, 2
    // piece + 1 of a 128-byte row, swizzled
    auto put = [&](uint8_t *tile, const uint4 (&b)[4 * HALVES]) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = r_l + 32 * k;
#pragma unroll
        for (int hf = 0; hf < HALVES; ++hf) {
          const uint4 w = b[k * HALVES + hf];
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
    auto publish = [&](uint64_t *bar) {
      tc::fence_proxy_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    // Q of a unit: a thread per row (two rows when the streams are row tiles)
    auto put_q = [&](const Unit &un, int parity) {
      const int jq = un.qt * p.tq;
#pragma unroll 1
      for (int t = 0; t < (PAIR ? 1 : 2); ++t) {
        const int r = 32 * cw + lane, ur = t * kRows + r;  // row of the tile, of the unit
        const int j = jq + ur / p.G;
        const bool have = ur < p.tq * p.G && j < un.n;
        const size_t off =
            ((size_t)(un.q0 + (have ? j : 0)) * p.Hq + (size_t)un.h * p.G + ur % p.G) * D;
        const uint8_t *src = reinterpret_cast<const uint8_t *>(p.q) + off * (PAIR ? 4 : 2);
        float qmax = 0.f;
        if (have) {
#pragma unroll 4
          for (int e = 0; e < D; e += 8) {
            f8::Raw8<DT> x;
            x.load(src + e * (PAIR ? 4 : 2));
            float f[8];
            x.get(f);
#pragma unroll
            for (int i = 0; i < 8; ++i) qmax = fmaxf(qmax, fabsf(f[i]));
          }
        }
        // as in the decode: largest value to [2^11, 2^12); the softmax scale's
        // sign goes with it, so the factor on scores is not negative
        const int ef = (int)(__float_as_uint(qmax) >> 23);
        const int fe = min(max(265 - ef, 1), 253);
        float f = qmax > 0.f ? __uint_as_float((uint32_t)fe << 23) : 1.f;
        qfac_s[parity][ur] = fabsf(p.qscale) / f;
        if (p.qscale < 0.f) f = -f;
        uint8_t *tile = q_sm + t * TILE;
#pragma unroll 4
        for (int e = 0; e < D; e += 8) {
          uint32_t hi[4] = {0, 0, 0, 0}, lo[4] = {0, 0, 0, 0};
          if (have) {
            f8::Raw8<DT> x;
            x.load(src + e * (PAIR ? 4 : 2));
            float v[8];
            x.get(v);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if constexpr (PAIR)
                split_h2(v[2 * i] * f, v[2 * i + 1] * f, hi[i], lo[i]);
              else
                hi[i] = h2_bits(__floats2half2_rn(v[2 * i] * f, v[2 * i + 1] * f));
            }
          }
          uint8_t *d = tile + (e >> 6) * (kRows * 128) + tc::sw128(r, (e >> 3) & 7);
          *reinterpret_cast<uint4 *>(d) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          if constexpr (PAIR)
            *reinterpret_cast<uint4 *>(d + TILE) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
    };

    Unit un;
    int u = blockIdx.x;
    bool have = unit_at(p, walk, u, n_units, pieces, un);
    while (have && un.ce <= un.cb) have = unit_at(p, walk, u += gridDim.x, n_units, pieces, un);
    int ids = have ? fetch_ids(un, un.cb) : -1;
    if (have) {
      load(p.k_pool, un, un.cb, ids, kb);
      load(p.v_pool, un, un.cb, ids, vb);
    }
    while (have && fine) {
      // the unit's Q, once the last unit's scores are computed
      if (live > 0 && !wait(&q_free, live - 1)) {
        fine = false;
        break;
      }
      put_q(un, live & 1);
      publish(&q_full);
      // the unit after this one
      Unit nx;
      int u2 = u + gridDim.x;
      bool have2 = unit_at(p, walk, u2, n_units, pieces, nx);
      while (have2 && nx.ce <= nx.cb)
        have2 = unit_at(p, walk, u2 += gridDim.x, n_units, pieces, nx);
      for (int c = un.cb; c < un.ce; ++c, ++g) {
        const int st = g % ST;
        const bool more = c + 1 < un.ce;
        const int ids_n = more ? fetch_ids(un, c + 1) : have2 ? fetch_ids(nx, nx.cb) : -1;
        // ---- what the softmax needs to know (its slot's last reader has
        // passed: four chunks back)
        ChunkMeta &m = meta[g & (kMetaSlots - 1)];
        if (cw == 0) {
          float ks = 0.f, lv = kNoScale;
          int rows = 0;
          if (ids >= 0) {
            ks = __ldg(p.k_scales + (size_t)ids * p.H + un.h);
            const float vs = __ldg(p.v_scales + (size_t)ids * p.H + un.h);
            lv = vs > 0.f ? log2f(vs) : vs == 0.f ? kNoScale : vs;
            rows = min(un.c - c * kChunk - lane * 16, 16);
          }
          const uint32_t bits = rows > 0 ? (1u << rows) - 1u : 0u;
          const uint32_t pair = bits << (16 * (lane & 1));
          const uint32_t both = pair | __shfl_xor_sync(kAll, pair, 1);
          if (lane < kGroups) {
            m.ks[lane] = ks;
            m.lv[lane] = lv;
            if ((lane & 1) == 0) m.ok[lane >> 1] = both;
          }
        }
        // V's NaN codes become zeros (times a probability of 0 they would
        // reach every row of the tile) and their positions are noted, before
        // K is published: the softmax reads the note with the scores
        uint32_t bad = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t hit = 0;
#pragma unroll
          for (int hf = 0; hf < HALVES; ++hf) {
            const uint4 w = vb[k * HALVES + hf];
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
              for (int hf = 0; hf < HALVES; ++hf) vb[k * HALVES + hf] = make_uint4(0, 0, 0, 0);
            }
            if (lane == k) {
#pragma unroll
              for (int i = 0; i < 8; ++i) nan_byte |= ((b >> (4 * i)) & 15u ? 1u : 0u) << i;
            }
          }
        }
        if (lane < 4) m.nan[4 * lane + cw] = (uint8_t)nan_byte;
        // ---- K
        if (g >= ST && !wait(&k_free[st], g / ST - 1)) {
          fine = false;
          break;
        }
        put(k_sm + st * TILE, kb);
        publish(&k_full[st]);
        if (more)
          load(p.k_pool, un, c + 1, ids_n, kb);
        else if (have2)
          load(p.k_pool, nx, nx.cb, ids_n, kb);
        // ---- V
        if (g >= ST && !wait(&v_free[st], g / ST - 1)) {
          fine = false;
          break;
        }
        put(v_sm + st * TILE, vb);
        publish(&v_full[st]);
        if (more)
          load(p.v_pool, un, c + 1, ids_n, vb);
        else if (have2)
          load(p.v_pool, nx, nx.cb, ids_n, vb);
        ids = ids_n;
      }
      ++live;
      un = nx;
      u = u2;
      have = have2;
    }
  } else if (warp == kMmaWarp) {
    // =============================================================== products
    constexpr uint32_t idesc_s = tc::idesc_f16(kRows, kChunk, false);
    constexpr uint32_t idesc_o = tc::idesc_f16(kRows, D, true);
    const uint64_t d_q = tc::desc_sw128(smem_u32(q_sm), 16, 1024);
    const uint64_t d_k = tc::desc_sw128(smem_u32(k_sm), 16, 1024);
    const uint64_t d_v = tc::desc_sw128(smem_u32(v_sm), kRows * 128, 1024);
    int n_p[2] = {0, 0};  // products P V issued so far, by stream
    auto issue_s = [&](const Unit &un, int g0, int j, int nj) -> bool {
      const int t = j & 1, g = g0 + chunk_of(j), st = g % ST;
      if (!wait(&k_full[st], g / ST)) return false;
      tc::fence_after();
      if (lane == 0) {
        const uint64_t kd = tc::desc_advance(d_k, st * TILE);
        const uint64_t qd = tc::desc_advance(d_q, PAIR ? 0 : t * TILE);
#pragma unroll
        for (int hf = 0; hf < HALVES; ++hf)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint32_t off = hf * (kRows * 128) + kk * 32;
            const uint64_t b = tc::desc_advance(kd, off);
            tc::mma_f16(tmem + t * kChunk, tc::desc_advance(qd, off), b, idesc_s, hf + kk > 0);
            if constexpr (PAIR)
              tc::mma_f16(tmem + t * kChunk, tc::desc_advance(qd, off + TILE), b, idesc_s, true);
          }
        tc::commit(&s_full[t]);
        if (PAIR || t == 1) tc::commit(&k_free[st]);
        if (j == nj - 1) tc::commit(&q_free);
        mbar_arrive(&s_full[t]);
      }
      __syncwarp();
      return true;
    };
    auto issue_pv = [&](const Unit &un, int g0, int j, int nj) -> bool {
      const int t = j & 1, g = g0 + chunk_of(j), st = g % ST;
      if (!wait(&v_full[st], g / ST) || !wait(&p_full[t], n_p[t])) return false;
      ++n_p[t];
      tc::fence_after();
      if (lane == 0) {
        const uint64_t vd = tc::desc_advance(d_v, st * TILE);
#pragma unroll
        for (int kk = 0; kk < kChunk / 16; ++kk) {
          // P of positions [16 kk, 16 kk + 16): 8 columns of its 32-column piece
          const uint32_t pc = tmem + t * kChunk + (kk >> 1) * 32 + (kk & 1) * 8;
          const uint64_t b = tc::desc_advance(vd, kk * 2048);
          tc::mma_f16_ts(tmem + kOCol + t * D, pc, b, idesc_o, j >= 2 || kk > 0);
          if constexpr (PAIR) tc::mma_f16_ts(tmem + kOCol + t * D, pc + 16, b, idesc_o, true);
        }
        if (PAIR || t == 1) tc::commit(&v_free[st]);
        if (j + 2 >= nj) tc::commit(&o_full[t]);
      }
      __syncwarp();
      return true;
    };
    Unit un;
    int u = blockIdx.x, g0 = 0, live = 0;
    bool have = unit_at(p, walk, u, n_units, pieces, un);
    while (have && un.ce <= un.cb) have = unit_at(p, walk, u += gridDim.x, n_units, pieces, un);
    int issued = 0;  // bits: the unit's first S of stream A, of stream B
    while (have && fine) {
      const int nj = jobs_of(un);
      if (issued == 0 && !wait(&q_full, live)) {
        fine = false;
        break;
      }
      for (int j = 0; j < min(2, nj) && fine; ++j)
        if (!((issued >> j) & 1)) fine = issue_s(un, g0, j, nj);
      issued = 0;
      Unit nx;
      int u2 = u + gridDim.x;
      bool have2 = unit_at(p, walk, u2, n_units, pieces, nx);
      while (have2 && nx.ce <= nx.cb)
        have2 = unit_at(p, walk, u2 += gridDim.x, n_units, pieces, nx);
      const int nj2 = have2 ? jobs_of(nx) : 0, g2 = g0 + un.ce - un.cb;
      for (int j = 0; j < nj && fine; ++j) {
        fine = issue_pv(un, g0, j, nj);
        if (fine && j + 2 < nj) {
          fine = issue_s(un, g0, j + 2, nj);
        } else if (fine && (j & 1) < nj2) {
          // the next unit's first scores of this stream, if they can start
          // now (else after this unit): its order of streams is kept
          const int t = j & 1, g = g2 + chunk_of(t);
          const bool ready = (issued || mbar_test(&q_full, (uint32_t)(live + 1) & 1u)) &&
                             mbar_test(&k_full[g % ST], (uint32_t)(g / ST) & 1u);
          if ((t == 0 || (issued & 1)) && __all_sync(kAll, ready)) {
            fine = issue_s(nx, g2, t, nj2);
            issued |= 1 << t;
          }
        }
      }
      g0 = g2;
      ++live;
      un = nx;
      u = u2;
      have = have2;
    }
    // every product has completed before tensor memory is released
    if (lane == 0) tc::commit(&drain);
    __syncwarp();
    if (!wait(&drain, 0)) fine = false;
  } else {
    // ================================================================ softmax
    const int t = warp >> 2, r = tid & (kRows - 1);
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_t = tmem + lanes + t * kChunk, o_t = tmem + lanes + kOCol + t * D;
    const int ur = PAIR ? r : t * kRows + r;  // row of the unit
    int n_s = 0;                              // score tiles of this stream so far
    int live = 0, g0 = 0, n_o = 0;
    Unit un;
    for (int u = blockIdx.x; fine && unit_at(p, walk, u, n_units, pieces, un); u += gridDim.x) {
      const int j_q = un.qt * p.tq + ur / p.G, hd = un.h * p.G + ur % p.G;
      const bool row_in = ur < p.tq * p.G && j_q < un.n;
      const int i_row = un.q0 + j_q;
      int lo = 0, hi = 0;
      if (row_in) row_span(p, i_row, max(min(un.c - un.n + j_q + 1, un.c), 0), lo, hi);
      const int nch = un.ce - un.cb;
      float m_run = -INFINITY, l_run = 0.f, lv_ref = kNoScale;
      bool poison = false;
      const int first = PAIR ? t : 0, stride = PAIR ? 2 : 1;
      float qfac = 0.f;
      for (int k = first; k < nch; k += stride, ++n_s) {
        if (!wait(&s_full[t], n_s)) {
          fine = false;
          break;
        }
        tc::fence_after();
        if (k == first) qfac = qfac_s[live & 1][ur];
        const ChunkMeta &m = meta[(g0 + k) & (kMetaSlots - 1)];
        const int pos0 = (un.cb + k) * kChunk;
        // ---- the row's readable positions
        uint32_t mk[4];
        bool full = true, vnan = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int a = pos0 + 32 * i;
          auto bits = [&](int x, int y) -> uint32_t {
            x = max(x - a, 0);
            y = min(y - a, 32);
            return y > x ? (0xffffffffu >> (32 - y)) & (0xffffffffu << x) : 0u;
          };
          uint32_t b = 0;
          if (p.kv_map) {
            if (row_in) {
              for (int q = 0; q < MT_KV_MAP_MAX_SPANS; ++q) {
                const int32_t *run = p.kv_map + ((size_t)i_row * MT_KV_MAP_MAX_SPANS + q) * 2;
                if (run[1] > 0)
                  b |= bits(max(run[0], 0), (int)min((long long)run[0] + run[1], (long long)hi));
              }
            }
          } else {
            b = bits(lo, hi);
          }
          mk[i] = b & m.ok[i];
          full = full && mk[i] == 0xffffffffu;
          vnan = vnan || (mk[i] & reinterpret_cast<const uint32_t *>(m.nan)[i]);
        }
        poison = poison || vnan;
        // ---- running maximum
        float f[kGroups], lv_max = kNoScale;
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
          // not zero: -inf scores of masked positions stay -inf
          f[i] = fmaxf(qfac * m.ks[i], 1e-37f);
          lv_max = fmaxf(lv_max, m.lv[i]);
        }
        float mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float v[32];
          ld32(s_t + 32 * i, v);
          tc::wait_ld();
          if (!full) {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = (mk[i] >> e) & 1u ? v[e] : -INFINITY;
          }
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const float *x = v + 16 * q;
            float a = max3f(x[0], x[1], x[2]), b = max3f(x[3], x[4], x[5]);
            a = max3f(a, x[6], x[7]);
            b = max3f(b, x[8], x[9]);
            a = max3f(a, x[10], x[11]);
            b = max3f(b, x[12], x[13]);
            a = max3f(a, x[14], x[15]);
            mx = fmaxf(mx, fmaxf(a, b) * f[2 * i + q]);
          }
        }
        // ---- O rescaled when the maximum grows past 2^8, or on a row's first
        // finite score, or when V's scale passes 4 v_ref (the products of the
        // chunk before have completed: they were issued before these scores)
        const bool grow = mx > m_run + 8.f || (m_run == -INFINITY && mx != -INFINITY);
        if (__any_sync(kAll, grow || lv_max > lv_ref + 2.f)) {
          const float m_new = fmaxf(m_run, mx), lv_new = fmaxf(lv_ref, lv_max);
          const float al = m_run == -INFINITY ? 0.f : ex2(m_run - m_new);
          l_run *= al;
          const float so = al * ex2(lv_ref - lv_new);
          m_run = m_new;
          lv_ref = lv_new;
          if (k > first) {
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              float v[16];
              tc::ld16(o_t + c, v);
              tc::wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) v[e] *= so;
              tc::st16(o_t + c, v);
            }
            tc::wait_st();
          }
        }
        // ---- probabilities over the scores
        const float mr = m_run == -INFINITY ? 0.f : m_run;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float v[32];
          ld32(s_t + 32 * i, v);
          tc::wait_ld();
          if (!full) {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = (mk[i] >> e) & 1u ? v[e] : -INFINITY;
          }
          uint32_t h[16], l[16];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            // exponent: score * f + log2(sV / v_ref) + 5 - max; the sum takes
            // the V scale out again
            const float lw = fmaxf(m.lv[2 * i + q] - lv_ref, -60.f) + kPBits;
            const float2 ff = make_float2(f[2 * i + q], f[2 * i + q]);
            const float2 ad = make_float2(lw - mr, lw - mr);
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              float2 x = f2_fma(make_float2(v[16 * q + e], v[16 * q + e + 1]), ff, ad);
              x.x = ex2(x.x);
              x.y = ex2(x.y);
              sum = f2_add(sum, x);
              if constexpr (PAIR)
                split_h2x(x, h[8 * q + e / 2], l[8 * q + e / 2]);
              else
                h[8 * q + e / 2] = h2_bits(__floats2half2_rn(x.x, x.y));
            }
            l_run = fmaf(sum.x + sum.y, ex2(-lw), l_run);
          }
          tc::st16u(s_t + 32 * i, h);
          if constexpr (PAIR) tc::st16u(s_t + 32 * i + 16, l);
        }
        tc::wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[t]);
      }
      // ---- the unit's rows
      const bool had = first < nch;
      if (had && fine) {
        fine = wait(&o_full[t], n_o);
        ++n_o;
        tc::fence_after();
      }
      if (!PAIR && !fine) break;
      if (nch > 0) {
        ++live;
        g0 += nch;
      }
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
          b_has = nch > 1;
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
      if (writer) {
        const bool split = pieces > 1;
        const float inv = split ? 1.f : l_row == 0.f ? 0.f : 1.f / l_row;
        fa *= inv;
        fb *= inv;
        float *rr = split ? p.rec + ((size_t)un.id * C::UNIT_ROWS + ur) * (D + 4) : nullptr;
        const size_t orow = ((size_t)i_row * p.Hq + hd) * D;
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          float v[16];
          if (had) {
            tc::ld16(o_t + c, v);
            tc::wait_ld();
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = had && (fa != 0.f) ? v[e] * fa : 0.f;
          if constexpr (PAIR) {
            if (b_has) {
              float w[16];
              tc::ld16(o_t + D + c, w);
              tc::wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) v[e] += fb != 0.f ? w[e] * fb : 0.f;
            }
          }
          if (split) {
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              f8::store4<MT_F32>(rr + 4, c + e, v[e], v[e + 1], v[e + 2], v[e + 3]);
          } else if (row_in) {
            if constexpr (PAIR) {
#pragma unroll
              for (int e = 0; e < 16; e += 4)
                f8::store4<DT>(p.out, orow + c + e, v[e], v[e + 1], v[e + 2], v[e + 3]);
            } else {
              uint32_t w[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) w[e] = f8::pack2<DT>(v[2 * e], v[2 * e + 1]);
              uint4 *o4 = reinterpret_cast<uint4 *>(p.out) + (orow + c) / 8;
              o4[0] = make_uint4(w[0], w[1], w[2], w[3]);
              o4[1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
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
