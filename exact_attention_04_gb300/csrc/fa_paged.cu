// Decoding over a paged key/value cache, and writing tokens into its pages.
//
// Decode: one new query token per sequence, so each K and V row is used by
// the H / h_kv query heads of its group and then never again: 4 d bytes a
// token and K/V head against 4 d G flops, far below the tensor core's
// balance.  The bound is HBM, and the kernel is built to keep loads in
// flight: cp.async into per-warp rings in shared memory, no barrier between
// the warps while they stream.  The products run on mma.sync m16n8k16 with
// the group's heads as the 16 rows of a tile (a tcgen05 tile would be 128
// rows, of which a group fills 1 to 16, and its tensor-memory round trip
// costs more than the products).
//
//   s_j = scale q.k_j,  m = max s_j,  l = sum exp(s_j - m),
//   O = sum exp(s_j - m) v_j / l,  LSE = m + ln l
// over the visible keys, in one pass with the running m and l (fp32); P is
// rounded to bf16 for the P V product (half a step, at most 2^-8 of a weight),
// l adds the unrounded values, O stays in fp32 registers.
//
// Work split.  A tile is 64 token positions (128 at d = 64) of one (sequence,
// K/V head, 16 query heads; 32 where a group has more than 16).  Every CTA
// computes the same prefix sums over kv_len and takes tiles [c T / G,
// (c + 1) T / G) of the T there are: equal shares whatever the lengths, a pure
// function of kv_len.  A share may end inside a (sequence, head): such a part
// leaves its normalised O and LSE (base 2) in the workspace (at most two parts
// a CTA: slot 2c for the one that an earlier CTA began, 2c + 1 for the one
// that it begins and does not end), and a second kernel, a block per border
// between two shares, joins them,
//   LSE = log2 sum 2^LSE_i,  O = sum 2^(LSE_i - LSE) O_i,
// in the order of the CTAs; the blocks of an item that several borders cut
// share its rows (one row of 16000 tokens, h_kv = 1, H = 8: 32.5 -> 11.7 us
// against one block for all).  Loads run ahead across the boundary between two
// heads or sequences.  Calls with few tiles take a cluster of eight CTAs for
// each (sequence, head) instead, which joins its parts through shared memory
// (use_clusters).
#include <climits>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/fa.h"
#include "fa_internal.h"
#include "fa_paged.cuh"
#include "fa_window.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

using namespace ptx;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kRows = 16;                         // rows of the mma: query heads
constexpr int kCluster = 8;                       // CTAs of a cluster

struct DecodeParams {
  PagePool pool;
  const __nv_bfloat16* q;       // [B, H, d]
  __nv_bfloat16* o;             // [B, H, d]
  float* lse;                   // [B, H]
  const int* table;             // [B, max_pages]
  const int* kv_len;            // [B]
  int max_pages, max_len;       // max_len = max_pages * page_size
  int B, H, group, row_tiles;   // group = H / h_kv, row_tiles = ceil(group / (16 RT))
  int wl, sinks;
  int page16;                   // the page size is a multiple of 16
  float scale_log2;
  int parts;                    // CTAs of the split kernel
  float* o_part;                // [2 parts, 16 RT, d]
  float* lse_part;              // [2 parts, 16 RT]
  int2* meta;                   // [parts]: the (sequence, head) that a CTA's share starts in,
                                // and whether it cuts it
};

// The visible tiles of a sequence: `first` tiles from position 0 (the sinks),
// then the tiles from `shift` further on (the window) to the end.
struct Span {
  int len, lo;                  // visible: pos < len and (pos >= lo or pos < sinks)
  int first, shift, tiles;
};

template <int TILE>
__device__ __forceinline__ Span span_of(const DecodeParams& p, int b) {
  Span s;
  int len = __ldg(p.kv_len + b);
  len = len < 0 ? 0 : (len > p.max_len ? p.max_len : len);
  s.len = len;
  s.lo = len - 1 - p.wl > 0 ? len - 1 - p.wl : 0;
  const int send = p.sinks < s.lo ? p.sinks : s.lo;
  const int w0 = s.lo / TILE;
  const int ns = (send + TILE - 1) / TILE;
  s.first = ns < w0 ? ns : w0;
  s.shift = w0 - s.first;
  s.tiles = len > 0 ? s.first + (len + TILE - 1) / TILE - w0 : 0;
  return s;
}

// A place in the order of tiles: sequence, then (K/V head, row tile), then
// tile.
struct Cursor {
  int b, hr, tile;
  Span s;
};

template <int TILE>
__device__ __forceinline__ void cursor_at(const DecodeParams& p, int b, long long rem, Cursor& c) {
  c.b = b;
  c.s = span_of<TILE>(p, b);
  c.hr = static_cast<int>(rem / c.s.tiles);
  c.tile = static_cast<int>(rem - static_cast<long long>(c.hr) * c.s.tiles);
}

// The next tile; the caller knows that there is one.
template <int TILE>
__device__ __forceinline__ void cursor_next(const DecodeParams& p, Cursor& c) {
  if (++c.tile < c.s.tiles) return;
  c.tile = 0;
  if (++c.hr < p.pool.h_kv * p.row_tiles) return;
  c.hr = 0;
  do {
    ++c.b;
    c.s = span_of<TILE>(p, c.b);
  } while (c.s.tiles == 0 && c.b + 1 < p.B);
}

// Sum over the block of v (and the sum before this thread), through `warp_sum`.
template <int THREADS>
__device__ __forceinline__ long long block_scan(long long v, long long* warp_sum,
                                                long long& before) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  long long total = 0, pre = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) pre += warp_sum[w];
    total += warp_sum[w];
  }
  before = pre + x - v;
  return total;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t* a, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D, int RT = 1>
struct DecodeCfg {
  static constexpr int ROWS = kRows * RT;                  // query heads of a tile
  static constexpr int ROW = 2 * D;                        // bytes of a token's K or V row
  // Tokens of a warp's stage: what a stage costs besides its bytes (the page
  // lookup, the maximum's exchange, the loop) bounds d = 64, where 32 tokens
  // and one lookup for 16 took 87 us against 99 with 16 and one each (64 rows of 4096
  // tokens, h_kv = 8, 537 MB).
  static constexpr int TOK = D == 64 ? 32 : 16;
  static constexpr int TILE = kWarps * TOK;                // tokens of a CTA's stage
  static constexpr int HALF = TOK * ROW;                   // K (or V) of a stage
  static constexpr int STAGE = 2 * HALF;
  // 96 KB of loads in flight a CTA and two CTAs an SM (d = 256: 192 KB, one)
  static constexpr int STAGES = 3;
  static constexpr int CTAS = D == 256 ? 1 : 2;
  static constexpr bool QREG = D * RT <= 128;              // Q fragments in registers
  static constexpr int RCOLS = D * RT > 128 && D < 256 ? 16 : 32;   // columns merged at a time
  static constexpr int RED = RCOLS + 8;                    // floats of a reduction row
};

template <int D, int RT>
struct DecodeSmem {
  using C = DecodeCfg<D, RT>;
  alignas(128) uint8_t ring[kWarps][C::STAGES][C::STAGE];
  alignas(128) uint8_t q[C::ROWS * C::ROW];
  float red[kWarps][kRows][C::RED];
  float ml[kWarps][C::ROWS][2];
  uint32_t vis[kWarps][C::STAGES];
  long long warp_sum[kWarps];
  long long start_rem;
  int start_b;
};

__device__ __forceinline__ float cluster_load(uint32_t a) {
  float x;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(a) : "memory");
  return x;
}
__device__ __forceinline__ float4 cluster_load4(uint32_t a) {
  float4 x;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
               : "r"(a)
               : "memory");
  return x;
}

// CL: a cluster of CTAs takes each (sequence, head, row tile), an eighth of
// its tiles a CTA, and joins the parts through its shared memory.
template <int D, int RT, bool CL>
__global__ void __launch_bounds__(kThreads, DecodeCfg<D, RT>::CTAS)
    paged_decode_kernel(const __grid_constant__ DecodeParams p) {
  using C = DecodeCfg<D, RT>;
  constexpr int TILE = C::TILE;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  DecodeSmem<D, RT>& sm = *reinterpret_cast<DecodeSmem<D, RT>*>(smem_raw);
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int heads = p.pool.h_kv * p.row_tiles;
  Cursor next;
  int count;                     // the share's tiles
  const int cta = blockIdx.x;
  // sequences without a tile: O = 0, LSE = -inf
  auto write_empty = [&]() {
    for (int b = cta; b < p.B; b += gridDim.x) {
      if (span_of<TILE>(p, b).tiles > 0) continue;
      const size_t row0 = static_cast<size_t>(b) * p.H;
      uint4* o = reinterpret_cast<uint4*>(p.o + row0 * D);
      for (int e = threadIdx.x; e < p.H * (D / 8); e += kThreads) o[e] = make_uint4(0, 0, 0, 0);
      for (int h = threadIdx.x; h < p.H; h += kThreads) p.lse[row0 + h] = -INFINITY;
    }
  };
  if constexpr (CL) {
    const int item = cta / kCluster, rank = cta % kCluster;
    next.b = item / heads;
    next.hr = item - next.b * heads;
    next.s = span_of<TILE>(p, next.b);
    next.tile = next.s.tiles * rank / kCluster;
    count = next.s.tiles * (rank + 1) / kCluster - next.tile;
  } else {
    launch_dependents();
    // ---- this CTA's share of the tiles
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b_lo = min(p.B, static_cast<int>(threadIdx.x) * per), b_hi = min(p.B, b_lo + per);
    long long mine = 0;          // (64 bits: 2^31 rows and heads of 2^24 tiles)
    for (int b = b_lo; b < b_hi; ++b) mine += span_of<TILE>(p, b).tiles;
    long long before;
    const long long total = block_scan<kThreads>(mine, sm.warp_sum, before) * heads;
    const int parts = static_cast<int>(min(static_cast<long long>(p.parts), total));
    if (cta >= parts) {
      if (threadIdx.x == 0) p.meta[cta] = make_int2(-1, 0);
      write_empty();
      return;
    }
    const long long ta = cta * total / parts, tb = (cta + 1) * total / parts;
    if (ta >= before * heads && ta < (before + mine) * heads) {
      int b = b_lo;
      long long base = before * heads;
      for (;; ++b) {
        const long long n = static_cast<long long>(span_of<TILE>(p, b).tiles) * heads;
        if (ta < base + n) break;
        base += n;
      }
      sm.start_b = b;
      sm.start_rem = ta - base;
    }
    __syncthreads();
    count = static_cast<int>(tb - ta);       // the host keeps the largest an int
    cursor_at<TILE>(p, sm.start_b, sm.start_rem, next);
  }
  Cursor cur = next;

  // ---- the loading side: one tile ahead, the page of this lane's token
  const int tok = lane % C::TOK;
  int page = -1;                 // page number of the prefetched token
  long long part_off = 0;        // its slot's and head's offset
  auto look_up = [&]() {
    const int t = next.tile < next.s.first ? next.tile : next.tile + next.s.shift;
    const int pos = t * TILE + warp * C::TOK + tok;
    page = -1;
    if (pos < next.s.len && (pos >= next.s.lo || pos < p.sinks)) {
      const int j = static_cast<int>(static_cast<unsigned>(pos) /
                                     static_cast<unsigned>(p.pool.page_size));
      page = __ldg(p.table + static_cast<size_t>(next.b) * p.max_pages + j);
      part_off = static_cast<long long>(pos - j * p.pool.page_size) * p.pool.token_stride +
                 static_cast<long long>(next.hr / p.row_tiles) * p.pool.head_stride;
    }
  };
  const uint32_t ring = smem_u32(sm.ring[warp][0]);
  int looked = 0, issued = 0;
  look_up();
  looked = 1;
  // issues the prefetched tile's loads into its stage and prefetches the next
  auto issue = [&]() {
    if (issued < count) {
      const int slot = issued % C::STAGES;
      const bool ok = page >= 0 && page < p.pool.num_pages;
      const long long off = ok ? page * p.pool.page_stride + part_off : 0;
      const uint32_t vis = __ballot_sync(0xffffffffu, ok) & (C::TOK == 32 ? ~0u : 0xffffu);
      if (lane == 0) sm.vis[warp][slot] = vis;
      if (looked < count) {
        cursor_next<TILE>(p, next);
        look_up();
        ++looked;
      }
      if (vis) {
        constexpr int CH = C::ROW / 16;             // 16-byte chunks of a row
        constexpr int RPI = 32 / CH;                // rows of one warp instruction
        const int sub = RPI > 1 ? lane / CH : 0, ch = lane % CH;
        const uint32_t dst = ring + slot * C::STAGE + sub * C::ROW;
        auto copy = [&](int row0, const __nv_bfloat16* kp, const __nv_bfloat16* vp) {
          const int row = row0 + sub;
          const int bytes = (vis >> row) & 1u ? 16 : 0;    // 0: the row is filled with zeros
          const uint32_t d = dst + row0 * C::ROW + ((ch ^ (row & 7)) << 4);
          cp_async16(d, kp, bytes);
          cp_async16(d + C::HALF, vp, bytes);
        };
        if (p.page16) {
          // 16 tokens lie in one page: one lookup's offset (of any visible
          // one) serves them, and hidden ones have their slots there as well
          const long long stride = p.pool.token_stride;
          const long long mine = sub * stride + ch * 8;
#pragma unroll
          for (int g16 = 0; g16 < C::TOK; g16 += 16) {
            const uint32_t part = (vis >> g16) & 0xffffu;
            const int first = part ? __ffs(part) - 1 : 0;
            const long long base =
                part ? __shfl_sync(0xffffffffu, off, g16 + first) - first * stride : 0;
            const __nv_bfloat16* kp = p.pool.k + base + mine;
            const __nv_bfloat16* vp = p.pool.v + base + mine;
#pragma unroll
            for (int r = 0; r < 16; r += RPI, kp += RPI * stride, vp += RPI * stride)
              copy(g16 + r, kp, vp);
          }
        } else {
#pragma unroll
          for (int r = 0; r < C::TOK; r += RPI) {
            const long long ro = __shfl_sync(0xffffffffu, off, r + sub) + ch * 8;
            copy(r, p.pool.k + ro, p.pool.v + ro);
          }
        }
      }
      ++issued;
    }
    cp_async_commit();
  };
#pragma unroll 1
  for (int i = 0; i < C::STAGES - 1; ++i) issue();

  // ---- the computing side
  // the first tile of the current (sequence, head, row tile), from the share's
  // first on: negative where an earlier CTA began it
  int seg0 = -cur.tile;
  if (!CL && threadIdx.x == 0) p.meta[cta] = make_int2(cur.b * heads + cur.hr, seg0 < 0);
  const int g = lane / 4, t4 = lane % 4;
  float acc[RT][D / 8][4];
  float m[RT][2], l[RT][2];
  uint32_t qf[RT][C::QREG ? D / 16 : 1][4];
  const uint32_t qs = smem_u32(sm.q);
  auto q_addr = [&](int t, int ks) {
    const int row = kRows * t + (lane & 15);
    return qs + row * C::ROW + (((2 * ks + lane / 16) ^ (row & 7)) << 4);
  };
  // CL: this CTA's part, where warp 0's ring was (the merge's first barrier
  // is behind the last read of it, and no load is on its way)
  float* const o_smem = reinterpret_cast<float*>(sm.ring[0][0]);
  float* const lse_smem = o_smem + C::ROWS * D;
  static_assert((C::ROWS * D + C::ROWS) * 4 <= C::STAGES * C::STAGE, "the part fits the ring");
  bool fresh = true;
#pragma unroll 1
  for (int i = 0; i < count; ++i) {
    const int kvh = cur.hr / p.row_tiles, rt = cur.hr - kvh * p.row_tiles;
    const int rows = min(C::ROWS, p.group - rt * C::ROWS);
    const size_t row0 = static_cast<size_t>(cur.b) * p.H + kvh * p.group + rt * C::ROWS;
    if (fresh) {
      fresh = false;
      // Q of the group into shared memory (rows past it zero), then registers
      for (int e = threadIdx.x; e < C::ROWS * (C::ROW / 16); e += kThreads) {
        const int row = e / (C::ROW / 16), ch = e % (C::ROW / 16);
        uint4 x = make_uint4(0, 0, 0, 0);
        if (row < rows) x = __ldg(reinterpret_cast<const uint4*>(p.q + (row0 + row) * D) + ch);
        *reinterpret_cast<uint4*>(sm.q + row * C::ROW + ((ch ^ (row & 7)) << 4)) = x;
      }
      __syncthreads();
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        if constexpr (C::QREG) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) ldsm_x4(qf[t][ks], q_addr(t, ks));
        }
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[t][n][e] = 0.f;
        m[t][0] = m[t][1] = -INFINITY;
        l[t][0] = l[t][1] = 0.f;
      }
    }
    cp_async_wait<C::STAGES - 2>();
    __syncwarp();
    const int slot = i % C::STAGES;
    const uint32_t vis = sm.vis[warp][slot];
    issue();                     // into the stage that the previous tile left
    if (vis) {
      const uint32_t kb = ring + slot * C::STAGE;
      constexpr int NT = C::TOK / 8;                       // 8-token column tiles of S
      // two tiles take two accumulators each, so that four chains of products
      // run beside each other as with four tiles
      constexpr int CH2 = NT * RT == 2 ? 2 : 1;
      float x[RT][NT * CH2][4];
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int n = 0; n < NT * CH2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[t][n][e] = 0.f;
      {
        const int row = (lane / 16) * 8 + (lane & 7);
        const uint32_t ka = kb + row * C::ROW;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t af[RT][4];
          if constexpr (!C::QREG) {
#pragma unroll
            for (int t = 0; t < RT; ++t) ldsm_x4(af[t], q_addr(t, ks));
          }
          const uint32_t a = ka + (((2 * ks + ((lane / 8) & 1)) ^ (row & 7)) << 4);
#pragma unroll
          for (int n = 0; n < NT; n += 2) {
            uint32_t bf[4];
            ldsm_x4(bf, a + n * 8 * C::ROW);
            const int o = n + (CH2 == 2 ? NT * (ks & 1) : 0);
#pragma unroll
            for (int t = 0; t < RT; ++t) {
              const uint32_t* a4 = C::QREG ? qf[t][C::QREG ? ks : 0] : af[t];
              mma16816(x[t][o], a4, bf[0], bf[1]);
              mma16816(x[t][o + 1], a4, bf[2], bf[3]);
            }
          }
        }
      }
      uint32_t pf[RT][NT / 2][4];
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        float (&y)[NT * CH2][4] = x[t];
        if constexpr (CH2 == 2) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) y[n][e] += y[NT + n][e];
        }
        // rows g (elements 0, 1) and g + 8 (2, 3); columns 8 n + 2 t4 + {0, 1}
        if (vis != (C::TOK == 32 ? ~0u : 0xffffu)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!((vis >> (8 * n + 2 * t4 + (e & 1))) & 1u)) y[n][e] = -INFINITY;
        }
        float base[2];             // scale m, subtracted in the exponent
        bool moved = false;
        float alpha[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float mx = fmaxf(y[0][2 * r], y[0][2 * r + 1]);
#pragma unroll
          for (int n = 1; n < NT; ++n) mx = fmax3(mx, y[n][2 * r], y[n][2 * r + 1]);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          mx *= p.scale_log2;
          const float mn = fmaxf(m[t][r], mx);
          alpha[r] = m[t][r] == -INFINITY ? 0.f : ex2_approx(m[t][r] - mn);
          moved = moved || mn > m[t][r];
          m[t][r] = mn;
          base[r] = mn == -INFINITY ? 0.f : mn;
        }
        if (__any_sync(0xffffffffu, moved)) {
          l[t][0] *= alpha[0];
          l[t][1] *= alpha[1];
#pragma unroll
          for (int n = 0; n < D / 8; ++n) {
            acc[t][n][0] *= alpha[0];
            acc[t][n][1] *= alpha[0];
            acc[t][n][2] *= alpha[1];
            acc[t][n][3] *= alpha[1];
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            y[n][e] = ex2_approx(fmaf(y[n][e], p.scale_log2, -base[e / 2]));
            l[t][e / 2] += y[n][e];
          }
#pragma unroll
        for (int n = 0; n < NT / 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            pf[t][n][e] =
                pack_bf16x2(y[2 * n + e / 2][2 * (e & 1)], y[2 * n + e / 2][2 * (e & 1) + 1]);
      }
      {
        const int row = ((lane / 8) & 1) * 8 + (lane & 7);
        const uint32_t va = kb + C::HALF + row * C::ROW;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          const uint32_t a = va + (((2 * j + lane / 16) ^ (row & 7)) << 4);
#pragma unroll
          for (int n = 0; n < NT / 2; ++n) {
            uint32_t bf[4];
            ldsm_x4_t(bf, a + n * 16 * C::ROW);
#pragma unroll
            for (int t = 0; t < RT; ++t) {
              mma16816(acc[t][2 * j], pf[t][n], bf[0], bf[1]);
              mma16816(acc[t][2 * j + 1], pf[t][n], bf[2], bf[3]);
            }
          }
        }
      }
    }
    __syncwarp();                // every lane has read the stage
    const bool ends = cur.tile + 1 == cur.s.tiles;
    if (!ends && i + 1 < count) {
      ++cur.tile;
      continue;
    }
    // ---- the end of a (sequence, head) or of the share: merge the warps
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        l[t][r] += __shfl_xor_sync(0xffffffffu, l[t][r], 1);
        l[t][r] += __shfl_xor_sync(0xffffffffu, l[t][r], 2);
        if (t4 == 0) {
          sm.ml[warp][kRows * t + g + 8 * r][0] = m[t][r];
          sm.ml[warp][kRows * t + g + 8 * r][1] = l[t][r];
        }
      }
    const bool whole = !CL && seg0 >= 0 && ends;
    const int part = 2 * cta + (seg0 < 0 ? 0 : 1);
    constexpr int PC = C::RCOLS / 8;           // columns of a thread
    const int trow = threadIdx.x / 8, col = threadIdx.x % 8 * PC;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int row = kRows * t + trow;
      float w[kWarps], lse2 = 0.f;
#pragma unroll
      for (int c = 0; c < D / C::RCOLS; ++c) {
#pragma unroll
        for (int n = 0; n < C::RCOLS / 8; ++n) {
          const float* a = acc[t][C::RCOLS / 8 * c + n];
          *reinterpret_cast<float2*>(&sm.red[warp][g][8 * n + 2 * t4]) = make_float2(a[0], a[1]);
          *reinterpret_cast<float2*>(&sm.red[warp][g + 8][8 * n + 2 * t4]) =
              make_float2(a[2], a[3]);
        }
        __syncthreads();
        if (row < rows) {
          if (c == 0) {
            float mx = -INFINITY, sum = 0.f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) mx = fmaxf(mx, sm.ml[k][row][0]);
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
              const float mk = sm.ml[k][row][0];
              w[k] = mk == -INFINITY ? 0.f : ex2_approx(mk - mx);
              sum += w[k] * sm.ml[k][row][1];
            }
            // a NaN sum (a NaN score) stays one
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) w[k] *= inv;
            lse2 = sum == 0.f ? -INFINITY : mx + log2f(sum);
          }
          float y[PC];
#pragma unroll
          for (int e = 0; e < PC; ++e) y[e] = 0.f;
#pragma unroll
          for (int k = 0; k < kWarps; ++k)
#pragma unroll
            for (int e = 0; e < PC; e += 2) {
              const float2 z = *reinterpret_cast<const float2*>(&sm.red[k][trow][col + e]);
              y[e] = fmaf(w[k], z.x, y[e]);
              y[e + 1] = fmaf(w[k], z.y, y[e + 1]);
            }
          const int at = C::RCOLS * c + col;
          if (whole) {
            uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + (row0 + row) * D + at);
#pragma unroll
            for (int e = 0; e < PC; e += 2) dst[e / 2] = pack_bf16x2(y[e], y[e + 1]);
          } else {
            float* dst = CL ? o_smem + row * D + at
                            : p.o_part + (static_cast<size_t>(part) * C::ROWS + row) * D + at;
#pragma unroll
            for (int e = 0; e < PC; e += 2)
              *reinterpret_cast<float2*>(dst + e) = make_float2(y[e], y[e + 1]);
          }
        }
        __syncthreads();
      }
      if (row < rows && col == 0) {
        if (whole)
          p.lse[row0 + row] = lse2 * 0.69314718055994531f;
        else
          (CL ? lse_smem + row : p.lse_part + part * C::ROWS + row)[0] = lse2;
      }
    }
    if (i + 1 < count) {
      seg0 = i + 1;
      cursor_next<TILE>(p, cur);
      fresh = true;
    }
  }
  cp_async_wait<0>();
  if constexpr (CL) {
    if (count == 0 && threadIdx.x < C::ROWS) lse_smem[threadIdx.x] = -INFINITY;
    cluster_sync();
    const int rank = cta % kCluster;
    const int kvh = cur.hr / p.row_tiles, rt = cur.hr - kvh * p.row_tiles;
    const int rows = min(C::ROWS, p.group - rt * C::ROWS);
    const size_t row0 = static_cast<size_t>(cur.b) * p.H + kvh * p.group + rt * C::ROWS;
    const uint32_t o_at = smem_u32(o_smem), lse_at = smem_u32(lse_smem);
    for (int e = rank * kThreads + threadIdx.x; e < rows * (D / 4); e += kCluster * kThreads) {
      const int row = e / (D / 4), col = e % (D / 4) * 4;
      float lse[kCluster], mx = -INFINITY;
      float4 x[kCluster];
#pragma unroll
      for (int c = 0; c < kCluster; ++c) {
        lse[c] = cluster_load(in_cta(lse_at + row * 4, c));
        x[c] = cluster_load4(in_cta(o_at + (row * D + col) * 4, c));
      }
#pragma unroll
      for (int c = 0; c < kCluster; ++c) mx = fmaxf(mx, lse[c]);
      const float base = mx == -INFINITY ? 0.f : mx;
      float sum = 0.f;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int c = 0; c < kCluster; ++c) {
        if (lse[c] == -INFINITY) continue;      // (of a part without a tile, O was never written)
        const float w = ex2_approx(lse[c] - base);
        sum += w;
        y.x = fmaf(w, x[c].x, y.x);
        y.y = fmaf(w, x[c].y, y.y);
        y.z = fmaf(w, x[c].z, y.z);
        y.w = fmaf(w, x[c].w, y.w);
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      *reinterpret_cast<uint2*>(p.o + (row0 + row) * D + col) =
          make_uint2(pack_bf16x2(y.x * inv, y.y * inv), pack_bf16x2(y.z * inv, y.w * inv));
      if (col == 0)
        p.lse[row0 + row] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * 0.69314718055994531f;
    }
    __syncwarp();
    cluster_sync();              // no CTA leaves while its part is read
  } else {
    write_empty();
  }
}

// Joins the parts of the (sequence, head, row tile) that the border before CTA
// blockIdx.x + 1 cuts; where several borders cut it, their blocks share its
// rows.
constexpr int kJoinThreads = 512;             // at least as many as CTAs of the split kernel

template <int D, int RT>
__global__ void __launch_bounds__(kJoinThreads)
    paged_join_kernel(const __grid_constant__ DecodeParams p) {
  constexpr int WARPS = kJoinThreads / 32;
  constexpr int ROWS = kRows * RT;
  constexpr int PER = D / 32;                 // columns of a lane
  constexpr int AHEAD = D == 256 ? 4 : 8;     // parts whose loads are in flight together
  __shared__ int first, last;    // the borders that cut it
  __shared__ float w_max[WARPS], w_sum[WARPS];
  __shared__ float w_acc[WARPS][D];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int heads = p.pool.h_kv * p.row_tiles;
  const int c = blockIdx.x + 1;
  grid_dependency_wait();
  const int2 cut = p.meta[c];
  if (!cut.y) return;
  if (threadIdx.x == 0) first = last = c;
  __syncthreads();
  if (threadIdx.x < p.parts) {   // the launch keeps parts at or below the threads
    const int2 x = p.meta[threadIdx.x];
    if (x.y && x.x == cut.x) {
      atomicMin(&first, threadIdx.x);
      atomicMax(&last, threadIdx.x);
    }
  }
  __syncthreads();
  const int c0 = first - 1;      // the CTA of the first part
  const int blocks = last - c0, n = blocks + 1;   // parts
  const int b = cut.x / heads, hr = cut.x % heads;
  const int kvh = hr / p.row_tiles, rt = hr - kvh * p.row_tiles;
  const int rows = min(ROWS, p.group - rt * ROWS);
  const size_t row0 = static_cast<size_t>(b) * p.H + kvh * p.group + rt * ROWS;
  // this block's rows: from `row_lo` every `blocks`-th
  const int row_lo = c - first;
  if (row_lo >= rows) return;
  const int own = (rows - row_lo + blocks - 1) / blocks;
  // a warp takes a row (and with more rows than warps another), or with fewer
  // rows than warps every k-th part of one
  const int k = own > 8 ? 1 : (own > 4 ? 2 : (own > 2 ? 4 : (own == 2 ? 8 : 16)));
  const int sub = warp % k;
  for (int at = 0; at < (RT == 1 ? 1 : own); at += WARPS) {   // k = 1 where it goes round
    const int row = row_lo + (at + warp / k) * blocks;
    float mx = -INFINITY, sum = 0.f, acc[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] = 0.f;
    if (row < rows) {
      auto slot = [&](int i) {
        return static_cast<size_t>(2 * (c0 + i) + (i == 0 ? 1 : 0)) * ROWS + row;
      };
      for (int i0 = sub; i0 < n; i0 += AHEAD * k) {
        float lse[AHEAD], x[AHEAD][PER];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
          const int i = i0 + u * k;
          lse[u] = -INFINITY;
          if (i < n) {
            lse[u] = p.lse_part[slot(i)];
            const float* src = p.o_part + slot(i) * D + lane * PER;
#pragma unroll
            for (int e = 0; e < PER; ++e) x[u][e] = src[e];
          }
        }
        float m = mx;
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) m = fmaxf(m, lse[u]);
        const float base = m == -INFINITY ? 0.f : m;
        const float alpha = mx == -INFINITY ? 0.f : ex2_approx(mx - base);
        mx = m;
        sum *= alpha;
#pragma unroll
        for (int e = 0; e < PER; ++e) acc[e] *= alpha;
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
          if (i0 + u * k < n) {
            const float w = ex2_approx(lse[u] - base);
            sum += w;
#pragma unroll
            for (int e = 0; e < PER; ++e) acc[e] = fmaf(w, x[u][e], acc[e]);
          }
        }
      }
    }
    if (k > 1) {
      if (lane == 0) {
        w_max[warp] = mx;
        w_sum[warp] = sum;
      }
#pragma unroll
      for (int e = 0; e < PER; ++e) w_acc[warp][lane * PER + e] = acc[e];
      __syncthreads();
      if (sub == 0) {
        float m = mx;
        for (int o = 1; o < k; ++o) m = fmaxf(m, w_max[warp + o]);
        const float base = m == -INFINITY ? 0.f : m;
        const float a0 = mx == -INFINITY ? 0.f : ex2_approx(mx - base);
        mx = m;
        sum *= a0;
#pragma unroll
        for (int e = 0; e < PER; ++e) acc[e] *= a0;
        for (int o = 1; o < k; ++o) {
          const float mo = w_max[warp + o];
          const float a = mo == -INFINITY ? 0.f : ex2_approx(mo - base);
          sum = fmaf(a, w_sum[warp + o], sum);
#pragma unroll
          for (int e = 0; e < PER; ++e) acc[e] = fmaf(a, w_acc[warp + o][lane * PER + e], acc[e]);
        }
      }
    }
    if (sub == 0 && row < rows) {
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + (row0 + row) * D + lane * PER);
#pragma unroll
      for (int e = 0; e < PER / 2; ++e) dst[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
      if (lane == 0)
        p.lse[row0 + row] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * 0.69314718055994531f;
    }
  }
}

template <int D, int RT>
cudaError_t launch_decode_t(const DecodeParams& p, bool clusters, cudaStream_t stream) {
  constexpr int smem = sizeof(DecodeSmem<D, RT>);
  const auto kernel =
      clusters ? paged_decode_kernel<D, RT, true> : paged_decode_kernel<D, RT, false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  if (clusters) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kCluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.B * p.pool.h_kv * p.row_tiles * kCluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
  }
  kernel<<<p.parts, kThreads, smem, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (p.parts < 2) return cudaSuccess;        // nothing is cut
  return launch_dependent(paged_join_kernel<D, RT>, dim3(p.parts - 1), kJoinThreads, stream, p);
}

// CTAs of the split kernel: as many as are resident at once.
int decode_parts(int d, int num_sms) {
  const int n = num_sms * (d == 256 ? DecodeCfg<256>::CTAS : DecodeCfg<128>::CTAS);
  return n < kJoinThreads ? n : kJoinThreads;
}
static_assert(DecodeCfg<64>::CTAS == DecodeCfg<128>::CTAS &&
                  2 * (sizeof(DecodeSmem<128, 2>) + 1024) <= 233472 &&
                  2 * (sizeof(DecodeSmem<64, 2>) + 1024) <= 233472,
              "decode_parts");

// 16-row tiles that a CTA takes from one pass over K and V: two where a group
// has more than 16 heads, since a pass that reads K and V out of L2 takes its
// time too (64 rows of 8192 tokens, h_kv = 1, one tile / two: 32 heads, d =
// 128 89 / 64 us, d = 64 42 / 37; 64 heads 163 / 105, 70 / 56), and one at d =
// 256, where two tiles of O are more than the registers.
int decode_tiles(int d, int group) { return group > kRows && d < 256 ? 2 : 1; }

// Few tiles: a cluster an item and no join kernel.  All clusters resident at
// once, and of the tiles that a row can see (the table's width and the window
// bound them; kv_len is on the device) at most four a CTA, or eight where the
// clusters fill half of the GPU: past that the shares' even split over all SMs
// is worth more than the second kernel.  Shares / clusters, d = 128, ten calls
// a graph over rows that L2 holds: one row, h_kv = 8, of 1000 tokens 8.2 / 6.2
// us, 2000 9.0 / 8.3, 4000 10.3 / 12.0; four rows of 1000 10.1 / 7.4, 4000 16.4
// / 13.7; one row, h_kv = 1, of 2000 7.9 / 7.8, 4000 8.4 / 11.6 (and the host
// launches once).
bool use_clusters(int d, int B, int h_kv, int group, int num_sms, long long positions, int left,
                  int sinks) {
  const int rows = kRows * decode_tiles(d, group), resident = decode_parts(d, num_sms);
  const int tile = d == 64 ? DecodeCfg<64>::TILE : DecodeCfg<128>::TILE;
  const long long items = static_cast<long long>(B) * h_kv * ((group + rows - 1) / rows);
  long long tiles = (positions + tile - 1) / tile;
  if (left >= 0) {
    const long long near = (left + 1ll + tile - 1) / tile + 1 + (sinks + (tile - 1ll)) / tile;
    tiles = near < tiles ? near : tiles;
  }
  const int each = 2 * items * kCluster >= resident ? 8 : 4;
  return items * kCluster <= resident && tiles <= each * kCluster;
}

size_t part_floats(int d, int group, int num_sms) {
  return static_cast<size_t>(2) * decode_parts(d, num_sms) * kRows * decode_tiles(d, group);
}

// New tokens into pages: a thread copies 16 bytes of K and of V.  Bound by
// the copied bytes; every row is contiguous on both sides (8 rows of up to
// 8192 tokens, h_kv = 8, d = 128: 41 us for 2 x 134 MB, 6.5 TB/s).  Launched
// as a dependent of whatever is before it (the reservation of its pages, in a
// serving step): it reads nothing before the wait, and nothing through the
// read-only path, which may keep what was there when the grid started.
template <int D>
__global__ void __launch_bounds__(256)
    paged_append_kernel(const __grid_constant__ PagePool pool, const uint4* k_new,
                        const uint4* v_new, const int* table, int max_pages, const int* start,
                        const int* kv_len, int Nq, int bh_count) {
  grid_dependency_wait();
  constexpr int CH = D / 8;
  const unsigned e = blockIdx.x * 256u + threadIdx.x;   // the launch keeps Nq * CH below 2^31
  const int t = static_cast<int>(e / CH), ch = static_cast<int>(e % CH);
  if (t >= Nq) return;
  for (int bh = blockIdx.y; bh < bh_count; bh += gridDim.y) {
    const int b = bh / pool.h_kv, h = bh - b * pool.h_kv;
    const long long at = static_cast<long long>(start[b]) + t;
    if (at < 0 || at >= kv_len[b]) continue;
    const int pos = static_cast<int>(at);
    const int j = pos / pool.page_size;
    if (j >= max_pages) continue;
    const int page = table[static_cast<size_t>(b) * max_pages + j];
    if (page < 0 || page >= pool.num_pages) continue;
    const long long dst = page * pool.page_stride + h * pool.head_stride +
                          (pos - j * pool.page_size) * pool.token_stride + ch * 8;
    const size_t src = (static_cast<size_t>(bh) * Nq + t) * CH + ch;
    const uint4 a = k_new[src], c = v_new[src];
    *reinterpret_cast<uint4*>(pool.k + dst) = a;
    *reinterpret_cast<uint4*>(pool.v + dst) = c;
  }
}

}  // namespace
}  // namespace fa

extern "C" {

size_t fa_decode_paged_workspace_bytes(int H, int h_kv, int d) {
  if (H < 1 || h_kv < 1 || H % h_kv || (d != 64 && d != 128 && d != 256)) return 0;
  int sms = 0;
  if (fa::device_facts(&sms) != FA_OK) sms = 152;
  const size_t rows = fa::part_floats(d, H / h_kv, sms);
  return rows * d * sizeof(float) + (rows * sizeof(float) + 255) / 256 * 256 +
         (fa::decode_parts(d, sms) * sizeof(int2) + 255) / 256 * 256;
}

size_t fa_decode_paged_call_bytes(const fa_paged_kv_t* cache, int max_pages, int B, int H,
                                  int window_left, int sinks) {
  if (!cache || cache->page_size < 1 || max_pages < 1 || B < 1 || sinks < 0) return 0;
  const size_t all = fa_decode_paged_workspace_bytes(H, cache->h_kv, cache->d);
  if (all == 0) return 0;
  int sms = 0;
  if (fa::device_facts(&sms) != FA_OK) sms = 152;
  return fa::use_clusters(cache->d, B, cache->h_kv, H / cache->h_kv, sms,
                          static_cast<long long>(max_pages) * cache->page_size, window_left, sinks)
             ? 0
             : all;
}

fa_status_t fa_decode_paged(const void* q, const fa_paged_kv_t* cache, int layer,
                            const int* block_table, int max_pages, const int* kv_len, void* o,
                            float* lse, int B, int H, float scale, int window_left, int sinks,
                            void* workspace, size_t workspace_bytes, void* stream) {
  if (!q || !o || !lse || !kv_len || layer < 0) return FA_ERR_INVALID_ARG;
  if (!fa::aligned_to(q, 16) || !fa::aligned_to(o, 16) || !fa::aligned_to(lse, 4) ||
      !fa::aligned_to(kv_len, 4) || !fa::aligned_to(workspace, 256))
    return FA_ERR_INVALID_ARG;
  fa::DecodeParams p;
  const fa_status_t ps = fa::resolve_pool(cache, layer, &p.pool);
  if (ps != FA_OK) return ps;
  if (!fa::table_ok(block_table, max_pages, p.pool.page_size)) return FA_ERR_INVALID_ARG;
  if (B < 1 || H < 1 || H % p.pool.h_kv || window_left < -1 || sinks < 0) return FA_ERR_INVALID_ARG;
  if (!(scale > 0.f && scale <= 3.402823466e38f)) return FA_ERR_INVALID_ARG;
  p.group = H / p.pool.h_kv;
  const int rt = fa::decode_tiles(p.pool.d, p.group);
  p.row_tiles = (p.group + fa::kRows * rt - 1) / (fa::kRows * rt);
  p.max_len = max_pages * p.pool.page_size;
  const long long heads = static_cast<long long>(p.pool.h_kv) * p.row_tiles;
  const int tile = p.pool.d == 64 ? fa::DecodeCfg<64>::TILE : fa::DecodeCfg<128>::TILE;
  const long long tiles = (p.max_len + tile - 1ll) / tile;
  if (static_cast<long long>(B) * H >= INT_MAX) return FA_ERR_INVALID_ARG;
  const size_t need = fa_decode_paged_call_bytes(cache, max_pages, B, H, window_left, sinks);
  if (need > 0 && (!workspace || workspace_bytes < need)) return FA_ERR_INVALID_ARG;
  int sms = 0;
  const fa_status_t ds = fa::device_facts(&sms);
  if (ds != FA_OK) return ds;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.table = block_table;
  p.kv_len = kv_len;
  p.max_pages = max_pages;
  p.B = B;
  p.H = H;
  p.wl = window_left < 0 || window_left > fa::kUnbounded ? fa::kUnbounded : window_left;
  p.sinks = sinks;
  p.page16 = p.pool.page_size % 16 == 0;
  p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  const int most = fa::decode_parts(p.pool.d, sms);
  if (B * heads * tiles / most >= INT_MAX) return FA_ERR_INVALID_ARG;   // a share's tiles
  p.parts = B * heads * tiles < most ? static_cast<int>(B * heads * tiles) : most;
  p.o_part = static_cast<float*>(workspace);
  const size_t rows = fa::part_floats(p.pool.d, p.group, sms);
  p.lse_part = p.o_part + rows * p.pool.d;
  p.meta = reinterpret_cast<int2*>(reinterpret_cast<char*>(p.lse_part) +
                                   (rows * sizeof(float) + 255) / 256 * 256);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool cl = need == 0;
  cudaError_t e;
  switch (p.pool.d) {
    case 64:
      e = rt == 2 ? fa::launch_decode_t<64, 2>(p, cl, s) : fa::launch_decode_t<64, 1>(p, cl, s);
      break;
    case 128:
      e = rt == 2 ? fa::launch_decode_t<128, 2>(p, cl, s) : fa::launch_decode_t<128, 1>(p, cl, s);
      break;
    default: e = fa::launch_decode_t<256, 1>(p, cl, s); break;
  }
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status_t fa_paged_append(const void* k_new, const void* v_new, const fa_paged_kv_t* cache,
                            int layer, const int* block_table, int max_pages, const int* start,
                            const int* kv_len, int B, int Nq, void* stream) {
  if (!k_new || !v_new || !start || !kv_len || layer < 0) return FA_ERR_INVALID_ARG;
  if (!fa::aligned_to(k_new, 16) || !fa::aligned_to(v_new, 16) || !fa::aligned_to(start, 4) ||
      !fa::aligned_to(kv_len, 4))
    return FA_ERR_INVALID_ARG;
  fa::PagePool pool;
  const fa_status_t ps = fa::resolve_pool(cache, layer, &pool);
  if (ps != FA_OK) return ps;
  if (!fa::table_ok(block_table, max_pages, pool.page_size)) return FA_ERR_INVALID_ARG;
  if (B < 1 || Nq < 1 || Nq >= fa::kMaxPositions) return FA_ERR_INVALID_ARG;
  const long long bh = static_cast<long long>(B) * pool.h_kv;
  const long long vec = static_cast<long long>(Nq) * (pool.d / 8);
  if (vec >= INT_MAX - 256 || bh >= INT_MAX) return FA_ERR_INVALID_ARG;
  const fa_status_t ds = fa::device_facts(nullptr);
  if (ds != FA_OK) return ds;
  const uint4* kn = static_cast<const uint4*>(k_new);
  const uint4* vn = static_cast<const uint4*>(v_new);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int rows = static_cast<int>(bh);
  const dim3 grid(static_cast<unsigned>((vec + 255) / 256), rows < 65535 ? rows : 65535);
  const auto launch = [&](auto kernel) {
    return fa::launch_dependent(kernel, grid, 256, s, pool, kn, vn, block_table, max_pages, start,
                                kv_len, Nq, rows);
  };
  const cudaError_t e = pool.d == 64    ? launch(fa::paged_append_kernel<64>)
                        : pool.d == 128 ? launch(fa::paged_append_kernel<128>)
                                        : launch(fa::paged_append_kernel<256>);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
