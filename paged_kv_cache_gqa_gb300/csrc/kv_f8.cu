// Storing rows into the 8-bit block-scaled cache, and reading rows back.
//
// Store. For a (block, head) that the call touches, with rows r of the call
// and kept rows k (rows of the block before the call's first position):
//   s  = max(s_old if there are kept rows, pow2(max |x_r|))
//   c_r = e4m3(x_r / s),   c_k = e4m3(c_k * s_old / s) when s > s_old.
// A unit of work is one (block, head) of K or of V, so the maximum, the scale
// and the codes need no other unit: one pass over the rows, which stay in
// registers between the maximum and the conversion (at most 8 groups of 8
// values a thread; wider units are shared by 2 or 4 warps that exchange the
// maximum through shared memory). Units are found without a plan: sequence s
// may touch blocks for at most floor(n / bs) + 2, so it owns the unit slots
// from floor(q_start[s] / bs) + 2 s on, and a warp finds its sequence by a
// search over q_start: with up to 32 sequences one round trip, a lane each. The
// rows are on their way before the block's id has come. Bound: HBM for prompts
// (139 MB of f16 prompts, 8 heads of 128, in 26.1 us: 5.33 TB/s; their float32
// form in 40.3 us: 5.76 TB/s), the call's latency for a decode step.
//
// Load. y = code * scale, each row's block looked up once per tile of rows.
// Bound: HBM.
#include <math.h>

#include <algorithm>

#include "f8.cuh"
#include "f8.h"

namespace mtkv {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct StoreParams {
  uint8_t *pool[2];
  float *scales[2];
  const void *x[2];
  const int32_t *table, *ctx, *q_start;
  uint32_t *status;
  int n_seqs, n_tok, H, max_blocks;
  long long n_phys;
};

template <int D, int BS, int DT>
__global__ void __launch_bounds__(kThreads, DT == MT_F32 ? 2 : 4)
    store_f8_kernel(const __grid_constant__ StoreParams p) {
  constexpr int LPR = D / 8;                           // lanes per row, 8 values each
  constexpr int RPP = 32 / LPR;                        // rows per pass of a warp
  constexpr int PASSES = BS / RPP;                     // passes of one warp over a block
  constexpr int WPU = PASSES > 8 ? PASSES / 8 : 1;     // warps that share a unit
  constexpr int NP = PASSES / WPU;                     // passes of each
  constexpr int UPC = kWarps / WPU;                    // units of a CTA
  constexpr int ES = DT == MT_F32 ? 4 : 2;
  __shared__ float amax_s[kWarps];
  pdl_enter();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = warp % WPU;
  const int upb = 2 * p.H;  // units of a block
  const long long unit = (long long)blockIdx.x * UPC + warp / WPU;
  const int slot = (int)(unit / upb), kv = (int)(unit % upb) / p.H, h = (int)(unit % upb) % p.H;

  // the unit's sequence, block and rows [a, z) of the block, block row a being row i0
  auto first_slot = [](int t, int q) { return max(q, 0) / BS + 2 * t; };
  int s, q0, q1, c;
  if (p.n_seqs <= 32) {
    // a lane has each sequence's first row and length: one round trip (by the search,
    // which takes three, a step of 32 sequences 2.8 us for 2.4)
    const int t = min(lane, p.n_seqs - 1);
    const int q_l = p.q_start[t], c_l = p.ctx[t], q_end = p.q_start[p.n_seqs];
    s = 31 - __clz(__ballot_sync(kAll, lane < p.n_seqs && first_slot(t, q_l) <= slot) | 1u);
    q0 = __shfl_sync(kAll, q_l, s);
    q1 = __shfl_sync(kAll, q_l, (s + 1) & 31);
    if (s + 1 == p.n_seqs) q1 = q_end;
    c = __shfl_sync(kAll, c_l, s);
  } else {
    s = f8::warp_search(p.n_seqs, slot, [&](int t) { return first_slot(t, p.q_start[t]); });
    q0 = p.q_start[s];
    q1 = p.q_start[s + 1];
    c = p.ctx[s];
  }
  const int n = q1 - q0;
  bool live = n > 0;
  if (n < 0 || (n > 0 && (q0 < 0 || q1 > p.n_tok || n > c || c > (long long)p.max_blocks * BS))) {
    if (lane == 0) report(p.status, MT_STATUS_BIT_DEVICE_CHECK);
    live = false;
  }
  const int first = c - n;  // the call's first position in the sequence
  const long long blk = (long long)(live ? first / BS : 0) + slot - (max(q0, 0) / BS + 2 * s);
  live = live && blk >= 0 && blk <= (c - 1) / BS;
  const int phys_raw = live ? p.table[(size_t)s * p.max_blocks + blk] : -1;
  const int a = live ? max(first - (int)blk * BS, 0) : 0;
  const int z = live ? min(c - (int)blk * BS, BS) : 0;
  const long long i0 = (long long)q0 + (int)blk * BS + a - first;
  if (WPU == 1 && !live) return;

  // rows of this warp's passes: row = (sub * NP + k) * RPP + lane / LPR. They are on
  // their way while the block's id is (a hole's rows are loaded for nothing)
  const int r_lane = lane / LPR, e0 = (lane % LPR) * 8;
  const uint8_t *x =
      reinterpret_cast<const uint8_t *>(p.x[kv]) + ((size_t)h * D + e0) * ES;
  const size_t row_bytes = (size_t)p.H * D * ES;
  f8::Raw8<DT> v[NP];
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const int r = (sub * NP + k) * RPP + r_lane;
    if (r >= a && r < z)
      v[k].load(x + (size_t)(i0 + r - a) * row_bytes);
    else
      v[k].zero();
  }
  int phys = phys_raw;
  if (phys < -1 || (long long)phys >= p.n_phys) {
    if (lane == 0) report(p.status, MT_STATUS_BIT_DEVICE_CHECK);
    phys = -1;
  }
  live = live && phys >= 0;
  if (WPU == 1 && !live) return;
  float *scale_p = p.scales[kv] + (live ? (size_t)phys * p.H + h : 0);
  float s_old = (live && a > 0) ? *scale_p : 0.f;
  if (!(s_old > 0.f && s_old < INFINITY)) s_old = 0.f;
  float amax = 0.f;
  bool finite = false;
  if constexpr (DT != MT_F32) {
    // 16-bit magnitudes order as integers, two at a time. (Through floats the
    // compiler kept all 64 of them for the conversion below: 94 registers, two
    // CTAs an SM instead of four, and 36.6 us for the prompts above.)
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < NP; ++k)
      top = __vmaxu2(
          __vmaxu2(top, v[k].w[0].x & 0x7fff7fffu),
          __vmaxu2(__vmaxu2(v[k].w[0].y & 0x7fff7fffu, v[k].w[0].z & 0x7fff7fffu),
                        v[k].w[0].w & 0x7fff7fffu));
    top = __reduce_max_sync(kAll, max(top & 0xffffu, top >> 16));
    finite = top < (DT == MT_F16 ? 0x7c00u : 0x7f80u);
    amax = DT == MT_F16 ? h2_to_f2(top).x : __uint_as_float(top << 16);
  }
  if (!finite) {
    amax = 0.f;
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      float f[8];
      v[k].get(f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float m = fabsf(f[i]);
        amax = fmaxf(amax, m < INFINITY ? m : 0.f);  // NaN compares false
      }
    }
    amax = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(amax)));  // not negative
  }
  if constexpr (WPU > 1) {
    if (lane == 0) amax_s[warp] = amax;
    __syncthreads();  // also: every warp of the unit has read s_old
#pragma unroll
    for (int w = 0; w < WPU; ++w) amax = fmaxf(amax, amax_s[warp - sub + w]);
    if (!live) return;
  }
  const float s_new = fmaxf(s_old, f8::pow2_scale(amax));
  if (sub == 0 && lane == 0) *scale_p = s_new;

  uint8_t *codes = p.pool[kv] + ((size_t)phys * BS * p.H + h) * D + e0;
  const size_t pitch = (size_t)p.H * D;
  if (a > 0 && s_new != s_old) {
    // kept rows under the grown scale (a kept scale of 0: its rows are 0)
    const float g = s_old / s_new;
#pragma unroll 1
    for (int k = 0; k < NP; ++k) {
      const int r = (sub * NP + k) * RPP + r_lane;
      if (r >= a) continue;
      uint2 *cp = reinterpret_cast<uint2 *>(codes + (size_t)r * pitch);
      uint2 w = *cp;
      uint32_t h0, h1, h2, h3;
      f8::code4_to_h2(w.x, h0, h1);
      f8::code4_to_h2(w.y, h2, h3);
      const float2 x0 = h2_to_f2(h0), x1 = h2_to_f2(h1), x2 = h2_to_f2(h2), x3 = h2_to_f2(h3);
      w.x = f8::to_code4(x0.x * g, x0.y * g, x1.x * g, x1.y * g);
      w.y = f8::to_code4(x2.x * g, x2.y * g, x3.x * g, x3.y * g);
      *cp = w;
    }
  }
  // x / s: a power of two that pow2_scale gave is inverted exactly; a kept
  // scale of another kind, which a caller may have written, divides. With s = 0
  // every finite value is 0, and an infinity keeps its saturated code.
  const bool pow2 = (__float_as_uint(s_new) & 0x7fffffu) == 0 && s_new >= 1.17549435e-38f &&
                    s_new <= 1.329228e36f;
  const float inv = pow2 ? f8::pow2_inv(s_new) : 1.f;
  const bool divide = !pow2 && s_new > 0.f;
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const int r = (sub * NP + k) * RPP + r_lane;
    if (r < a || r >= z) continue;
    float f[8];
    v[k].get(f);
    if (divide) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] /= s_new;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] *= inv;
    }
    uint2 w;
    w.x = f8::to_code4(f[0], f[1], f[2], f[3]);
    w.y = f8::to_code4(f[4], f[5], f[6], f[7]);
    *reinterpret_cast<uint2 *>(codes + (size_t)r * pitch) = w;
  }
}

// --------------------------------------------------------------------- load

struct LoadParams {
  const uint8_t *pool[2];
  const float *scales[2];
  void *y[2];
  const int32_t *table, *ctx, *q_start, *pos0;
  uint32_t *status;
  int n_seqs, n_tok, H, D, max_blocks;
  int bs_shift, d_shift;  // log2 of the block size and of D
  long long n_phys;
  int rows;  // rows per CTA
};

constexpr int kLoadRows = 32;  // most rows per CTA

template <int DT>
__global__ void __launch_bounds__(kThreads) load_f8_kernel(const __grid_constant__ LoadParams p) {
  // cell of each row, -1: reads 0, -2: not a row of any sequence
  __shared__ long long cell_s[kLoadRows];
  pdl_enter();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long r0 = (long long)blockIdx.x * p.rows;
  const int nr = (int)min((long long)p.rows, (long long)p.n_tok - r0);
  for (int r = warp; r < nr; r += kWarps) {
    const int i = (int)r0 + r;
    const int s = f8::warp_search(p.n_seqs, i, [&](int t) { return p.q_start[t]; });
    if (lane == 0) {
      const int q0 = p.q_start[s], q1 = p.q_start[s + 1], c = p.ctx[s];
      long long cell = -2;
      if (i >= q0 && i < q1) {
        const long long pos = (p.pos0 ? (long long)p.pos0[s] : (long long)c - (q1 - q0)) + (i - q0);
        cell = -1;
        bool bad = pos < 0 || pos >= c || pos >= ((long long)p.max_blocks << p.bs_shift);
        if (!bad) {
          const int phys = p.table[(size_t)s * p.max_blocks + (size_t)(pos >> p.bs_shift)];
          bad = phys < -1 || (long long)phys >= p.n_phys;
          if (!bad && phys >= 0)
            cell = ((long long)phys << p.bs_shift) + (pos & ((1 << p.bs_shift) - 1));
        }
        if (bad) report(p.status, MT_STATUS_BIT_DEVICE_CHECK);
      }
      cell_s[r] = cell;
    }
  }
  __syncthreads();
  // 8 codes a thread and step
  const int row_elems = p.H * p.D, gpr = row_elems >> 3, total = nr * gpr;
#pragma unroll 2
  for (int t = tid; t < total; t += kThreads) {
    const int r = t / gpr, e = (t - r * gpr) << 3;
    const long long cell = cell_s[r];
    if (cell == -2) continue;
    uint2 w[2] = {make_uint2(0, 0), make_uint2(0, 0)};
    float sc[2] = {0.f, 0.f};
    if (cell >= 0) {
      const size_t sp = (size_t)(cell >> p.bs_shift) * p.H + (e >> p.d_shift);
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        w[kv] = __ldg(reinterpret_cast<const uint2 *>(p.pool[kv] + (size_t)cell * row_elems + e));
        sc[kv] = __ldg(p.scales[kv] + sp);
      }
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      uint32_t h[4];
      f8::code4_to_h2(w[kv].x, h[0], h[1]);
      f8::code4_to_h2(w[kv].y, h[2], h[3]);
      float f[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 x = h2_to_f2(h[i]);
        f[2 * i] = cell >= 0 ? x.x * sc[kv] : 0.f;
        f[2 * i + 1] = cell >= 0 ? x.y * sc[kv] : 0.f;
      }
      const size_t o = (size_t)(r0 + r) * row_elems + e;
      if constexpr (DT == MT_F32) {
        f8::store4<DT>(p.y[kv], o, f[0], f[1], f[2], f[3]);
        f8::store4<DT>(p.y[kv], o + 4, f[4], f[5], f[6], f[7]);
      } else {
        reinterpret_cast<uint4 *>(p.y[kv])[o / 8] =
            make_uint4(f8::pack2<DT>(f[0], f[1]), f8::pack2<DT>(f[2], f[3]),
                       f8::pack2<DT>(f[4], f[5]), f8::pack2<DT>(f[6], f[7]));
      }
    }
  }
}

// ------------------------------------------------------------------- launch

template <int D, int BS, int DT>
mt_status launch_store(const StoreParams &p, long long slots, cudaStream_t s) {
  constexpr int passes = BS / (32 / (D / 8)), wpu = passes > 8 ? passes / 8 : 1;
  constexpr int upc = kWarps / wpu;
  const long long ctas = (slots * 2 * p.H + upc - 1) / upc;
  if (ctas > 0x7fffffffLL) return fail(MT_ERR_UNSUPPORTED, "mt_kv_store_f8: too many rows");
  return cuda_check(launch_pdl(store_f8_kernel<D, BS, DT>, dim3((unsigned)ctas), dim3(kThreads), 0,
                               s, p),
                    "mt_kv_store_f8 launch");
}

template <int D, int BS>
mt_status store_dt(const StoreParams &p, mt_dtype t, long long slots, cudaStream_t s) {
  if (t == MT_F32) return launch_store<D, BS, MT_F32>(p, slots, s);
  if (t == MT_F16) return launch_store<D, BS, MT_F16>(p, slots, s);
  return launch_store<D, BS, MT_BF16>(p, slots, s);
}

template <int D>
mt_status store_bs(const StoreParams &p, int bs, mt_dtype t, long long slots, cudaStream_t s) {
  return bs == 16 ? store_dt<D, 16>(p, t, slots, s) : store_dt<D, 32>(p, t, slots, s);
}

}  // namespace

mt_status check_f8_cache(const mt_f8_cache *c, const char *where) {
  const std::string w = std::string(where) + ": ";
  if (!c) return fail(MT_ERR_INVALID_ARG, w + "null cache");
  if (c->n_seqs < 0 || c->max_blocks < 0 || c->n_phys_blocks < 0 || c->n_kv_heads <= 0 ||
      c->head_dim <= 0 || c->block_size <= 0)
    return fail(MT_ERR_INVALID_ARG, w + "negative size or bad head shape");
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return fail(MT_ERR_UNSUPPORTED, w + "head_dim must be 64, 128 or 256");
  if (c->block_size != 16 && c->block_size != 32)
    return fail(MT_ERR_UNSUPPORTED, w + "block_size must be 16 or 32");
  if (c->n_kv_heads > kMaxF8KvHeads)
    return fail(MT_ERR_UNSUPPORTED, w + "more than 256 KV heads");
  // (the end of any kernel's tile, past the last position, is an int too)
  if ((long long)c->max_blocks * c->block_size > 0x7fffffffLL - 1023)
    return fail(MT_ERR_UNSUPPORTED, w + "max_blocks * block_size beyond 2^31 - 1024");
  if (c->n_phys_blocks > 0x7fffffffLL)
    return fail(MT_ERR_UNSUPPORTED, w + "more than 2^31 - 1 blocks");
  if (c->n_seqs == 0) return MT_OK;
  if (!c->context_lens || (c->max_blocks > 0 && !c->block_table) ||
      (c->n_phys_blocks > 0 && (!c->k_pool || !c->v_pool || !c->k_scales || !c->v_scales)))
    return fail(MT_ERR_INVALID_ARG, w + "null pointer in the cache");
  if (!aligned16(c->k_pool) || !aligned16(c->v_pool))
    return fail(MT_ERR_INVALID_ARG, w + "pools must be 16-byte aligned");
  return MT_OK;
}

}  // namespace mtkv

using namespace mtkv;

extern "C" mt_status mt_kv_store_f8(const mt_f8_cache *c, mt_dtype dtype, const void *k_new,
                                    const void *v_new, const int32_t *q_start, int n_tokens,
                                    uint32_t *status, mt_stream stream) {
  mt_status st = check_f8_cache(c, "mt_kv_store_f8");
  if (st != MT_OK) return st;
  if (!dtype_bytes(dtype)) return fail(MT_ERR_INVALID_ARG, "mt_kv_store_f8: unknown dtype");
  if (n_tokens < 0) return fail(MT_ERR_INVALID_ARG, "mt_kv_store_f8: negative n_tokens");
  if (n_tokens == 0 || c->n_seqs == 0) return ok();
  if (!k_new || !v_new || !q_start)
    return fail(MT_ERR_INVALID_ARG, "mt_kv_store_f8: null pointer");
  if (!aligned16(k_new) || !aligned16(v_new))
    return fail(MT_ERR_INVALID_ARG, "mt_kv_store_f8: rows must be 16-byte aligned");
  StoreParams p = {{c->k_pool, c->v_pool}, {c->k_scales, c->v_scales}, {k_new, v_new},
                   c->block_table, c->context_lens, q_start, status, c->n_seqs, n_tokens,
                   c->n_kv_heads, c->max_blocks, (long long)c->n_phys_blocks};
  const long long slots = n_tokens / c->block_size + 2LL * c->n_seqs;
  if (slots > 0x7fffffffLL) return fail(MT_ERR_UNSUPPORTED, "mt_kv_store_f8: too many sequences");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  st = c->head_dim == 64    ? store_bs<64>(p, c->block_size, dtype, slots, s)
       : c->head_dim == 128 ? store_bs<128>(p, c->block_size, dtype, slots, s)
                            : store_bs<256>(p, c->block_size, dtype, slots, s);
  return st == MT_OK ? ok() : st;
}

extern "C" mt_status mt_kv_load_f8(const mt_f8_cache *c, mt_dtype dtype, void *k_out, void *v_out,
                                   const int32_t *q_start, const int32_t *pos0, int n_tokens,
                                   uint32_t *status, mt_stream stream) {
  mt_status st = check_f8_cache(c, "mt_kv_load_f8");
  if (st != MT_OK) return st;
  if (!dtype_bytes(dtype)) return fail(MT_ERR_INVALID_ARG, "mt_kv_load_f8: unknown dtype");
  if (n_tokens < 0) return fail(MT_ERR_INVALID_ARG, "mt_kv_load_f8: negative n_tokens");
  if (n_tokens == 0 || c->n_seqs == 0) return ok();
  if (!k_out || !v_out || !q_start)
    return fail(MT_ERR_INVALID_ARG, "mt_kv_load_f8: null pointer");
  if (!aligned16(k_out) || !aligned16(v_out))
    return fail(MT_ERR_INVALID_ARG, "mt_kv_load_f8: rows must be 16-byte aligned");
  LoadParams p = {{c->k_pool, c->v_pool}, {c->k_scales, c->v_scales}, {k_out, v_out},
                  c->block_table, c->context_lens, q_start, pos0, status, c->n_seqs, n_tokens,
                  c->n_kv_heads, c->head_dim, c->max_blocks, c->block_size == 32 ? 5 : 4,
                  c->head_dim == 64 ? 6 : c->head_dim == 128 ? 7 : 8, (long long)c->n_phys_blocks, 0};
  // a CTA takes about 8192 values of K and of V (4 steps a thread), 1 to 32 rows
  p.rows = std::max(1, std::min(kLoadRows, 8192 / (c->n_kv_heads * c->head_dim)));
  const long long ctas = ((long long)n_tokens + p.rows - 1) / p.rows;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  auto kern = dtype == MT_F32 ? load_f8_kernel<MT_F32>
                              : dtype == MT_F16 ? load_f8_kernel<MT_F16> : load_f8_kernel<MT_BF16>;
  st = cuda_check(launch_pdl(kern, dim3((unsigned)ctas), dim3(kThreads), 0, s, p),
                  "mt_kv_load_f8 launch");
  return st == MT_OK ? ok() : st;
}
