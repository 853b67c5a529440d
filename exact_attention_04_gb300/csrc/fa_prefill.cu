// Attention of a chunk of new tokens per row over the paged cache.
//
// Work: a tile is up to 128 query rows - the heads of one K/V head's group
// times as many tokens of one row of the batch as fit - against the tiles of
// up to 128 keys that any of them sees.  The lengths are on the device, so a
// first kernel of one block lists the pieces (tile, range of key tiles): whole
// tiles where there are many, and ranges where few tiles would leave SMs idle
// (see plan_kernel).  The main kernel is persistent and takes the next piece
// from a counter, K/V heads innermost, so that the tiles that run at the same
// time share their keys through L2; a cut tile's pieces leave fp32 partial
// outputs and log-sum-exps that a third kernel joins.  What a piece computes
// does not depend on who takes it or when: results repeat bit for bit.
//
// Main kernel, one CTA per SM, roles by warp:
//   0        producer: takes pieces, looks pages up, loads Q and K by TMA.  A key
//            tile is whole pages (page_size <= 128: as many as fit; else up to
//            128 slots of one).  A page that does not exist is a box outside the
//            pool: TMA fills in zeros, and a bit mask of the tile's keys hides
//            them.
//   1        S = Q K^T on tcgen05 into tensor memory, running ahead
//   2        O += P V, P from tensor memory
//   3..      softmax: a row of the tile a thread; with d <= 128 two warps share
//            a row, each over half of every tile's keys with a maximum, sum
//            and O of its own
//   then 4   epilogue: merge the halves, divide, store O and LSE
//   last     V producer (K and V from one warp: N = 8192, d = 128, pages of 16
//            1.44 times as long, of 128 1.03 times)
// The recurrence and its roundings are those of the forward (fa_fwd.cu): S in
// base-2 units, a reference maximum that moves only when a block exceeds it by
// 2^24, P rounded to bf16 for the product (half a step, 2^-8 of a weight) and
// summed unrounded.
//
// What bounds it.  Many query rows: the softmax's instructions and the tensor
// pipe, as in the forward (N = 8192, not causal, pages of 16 / of 128 / the forward
// over contiguous K and V: d = 128, H = 32, h_kv = 8 713 / 712 / 678 us, 0.80 of the
// bf16 peak; d = 256, H = 16, h_kv = 4 695 / 672 / 668; d = 64, B = 2, H = 16 612 /
// 595 / 593, where eight copies a tile of 16-token pages keep the producers busy).
// Few rows: HBM (32 rows of 4 tokens after 8192, H = 32, h_kv = 8, d = 128: 1077 MB
// in 166 us, 0.95 of the copy bandwidth).  Short calls: the chain plan (4 us), first
// loads (4), a tile or two, and join (3 where something is cut): one row of 5
// tokens after 500 / 1000 / 1050, H = 32, h_kv = 8, d = 128 15 / 18 / 15 us, of which
// only the last, of nine key tiles, is cut by the estimate.
#include <climits>
#include <cmath>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_internal.h"
#include "fa_paged.cuh"
#include "fa_strided.cuh"
#include "fa_window.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

using namespace ptx;

constexpr int BM = 128;
constexpr int BN = 128;
constexpr int CHUNK = 128 * 128;   // bytes of 128 rows x 64 columns
constexpr float kRescaleSlack = 24.0f;
constexpr int kPlanThreads = 256;
constexpr int kPlanRows = 1024;    // rows whose tiles the plan counts in shared memory
constexpr float kJoinTiles = 2.f;  // what joining takes, in key tiles
constexpr int kMostRounds = 4;     // pieces of a cut call: at most so many a CTA, by its sum
constexpr int kItems = 4;          // pieces announced ahead
constexpr int kMostTail = 8;       // pieces of a tile behind the last whole round
// What a cut tile's piece takes beside its own key tiles (3 / 6 / 9: 512 tokens
// after 16000, d = 256, H = 16, h_kv = 4 217 / 164 / 168 us, d = 64, H = 16 86 / 72
// / 74; four chunks of 300 138 / 132 / 149; two of 1024 305 / 305 / 288).
constexpr float kCutTiles = 6.f;
constexpr int kRing = 8;           // key tiles whose masks are kept
// The epilogue's wait for a piece: 2^23 key tiles of up to 17 us (d = 256, pages
// of one).  The roles that work tile by tile give up after kWaitTimeoutNs, and
// raise the flag that ends this wait too.  (A limit by the piece's tiles: d = 64,
// N = 8192, pages of 128 594 / 602 us.)
constexpr unsigned long long kPieceTimeoutNs = 200000000000ull;

// A piece as the plan lists it, for every unit (K/V head, part of its group).
struct alignas(16) Entry {
  int row, n0, ntok, pos0;   // batch row; the tile's first token on the token axis, tokens,
                             // position of the first
  int len, s0, s1, slot;     // the row's keys; key tiles of the walk; partial output (times
                             // units + unit), or -1
  int jlo, ns, rlo, rhi;     // the walk: ns tiles of sinks, then from jlo on; [rlo, rhi): the
                             // keys that the row's tokens see, beside the sinks
};

struct JoinEntry {
  int batch, n0, ntok, slot0, pieces, pad[3];
};

struct Counters {
  unsigned items;      // pieces times units
  unsigned next;       // the next one to take
  int joins, most;     // cut tiles; most pieces of one
};

struct PrefillParams {
  CUtensorMap tq, tk, tv;
  __nv_bfloat16* o;
  long long ob, oh, ot;            // strides of o
  float* lse;                      // [batch, H, N]
  const int* table;
  const int* start;
  const int* kv_len;
  const int* offsets;              // nullptr: padded rows
  int B, H, N, h_kv;
  int group, gh, parts, units;     // query heads of a K/V head, of a tile; tiles a group; units
  int tpt;                         // tokens of a tile
  FastDiv fd_units, fd_parts, fd_gh, fd_tn, fd_grid;
  int max_pages, num_pages, page_size;
  int ppt, tpp, kt;                // pages of a key tile (0: tpp tiles a page), keys of one
  int groups, eights;              // eights of slots from page to page in tk, tv, and in all; or 0
  FastDiv fd_kt, fd_ps, fd_tpp;
  int wl, wr, sinks, causal;
  float scale_log2;
  int* status;
  Counters* counters;
  int* row_tiles;                  // [B + 1] tiles before a row (offsets)
  Entry* entries;
  JoinEntry* joins;
  int cap_tiles, cap_slots;        // (slots: times units)
  int slot_rows;
  float* o_part;
  float* lse_part;
  int grid;
};

// What a row's tokens are and see.
struct Row {
  int n0, ntok;        // its tokens on the token axis
  int start, len;
};

__device__ __forceinline__ Row row_at(const PrefillParams& p, int b) {
  Row r;
  int end;
  row_tokens(p.offsets, b, p.N, r.n0, end);
  r.ntok = end - r.n0;
  // (every token's position is an int: starts within 2^30, N below)
  r.start = min(max(p.start[b], -kUnbounded), kUnbounded - 1);
  r.len = min(max(p.kv_len[b], 0), p.max_pages * p.page_size);
  return r;
}

__device__ __forceinline__ int key_tile(const PrefillParams& p, int x) {
  if (p.ppt) return p.fd_kt.div(x);
  const int page = p.fd_ps.div(x);
  return page * p.tpp + ((x - page * p.page_size) >> 7);
}

// The position of a key tile's first key.
__device__ __forceinline__ int tile_pos(const PrefillParams& p, int j) {
  if (p.ppt) return j * p.kt;
  const int page = p.fd_tpp.div(j);
  return page * p.page_size + (j - page * p.tpp) * BN;
}

// Keys [lo, hi) of the tokens at positions pos0 .. pos0 + ntok - 1 (left of lo:
// the sinks).
__device__ __forceinline__ void tile_keys(const PrefillParams& p, int pos0, int ntok, int len,
                                          int& lo, int& hi) {
  long long last = static_cast<long long>(pos0) + ntok - 1;
  if (p.causal) last = last < len ? last : len - 1;   // tokens at or past len are not there
  if (p.causal && pos0 >= len) last = -1ll - kUnbounded;
  const long long h = last + p.wr + 1;
  hi = static_cast<int>(h < 0 ? 0 : (h > len ? len : h));
  const long long l = static_cast<long long>(pos0) - p.wl;
  lo = static_cast<int>(l < 0 ? 0 : (l > hi ? hi : l));
}

// The tile's walk: `ns` key tiles of sinks from 0, then from jlo; returns their
// number.
__device__ __forceinline__ int tile_walk(const PrefillParams& p, int pos0, int ntok, int len,
                                         int& jlo, int& ns) {
  int lo, hi;
  tile_keys(p, pos0, ntok, len, lo, hi);
  const int first = min(p.sinks, hi);
  ns = first > 0 ? key_tile(p, first - 1) + 1 : 0;
  jlo = 0;
  if (hi <= lo) return ns;
  jlo = key_tile(p, lo);
  ns = min(ns, jlo);
  return ns + key_tile(p, hi - 1) + 1 - jlo;
}

// ---------------------------------------------------------------- the plan

// Exclusive prefix sum over the block; total to every thread.
template <class T>
__device__ __forceinline__ T block_scan(T x, T* sm, T& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T v = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();
  if (lane == 31) sm[warp] = v;
  __syncthreads();
  T before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    const T y = sm[w];
    if (w < warp) before += y;
    total += y;
  }
  return v - x + before;
}

// Tile i of the call: rows in order, in a row the last tokens (under causality
// the most keys) first.
// rows: the tiles before each row.
__device__ __forceinline__ void plan_tile(const PrefillParams& p, const int* rows, int i, Entry& e,
                                          int& n) {
  int b, k, tiles;
  if (p.offsets) {
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
      const int m = (lo + hi) / 2;
      if (rows[m] <= i)
        lo = m;
      else
        hi = m;
    }
    b = lo;
    k = i - rows[b];
    tiles = rows[b + 1] - rows[b];
  } else {
    tiles = (p.N + p.tpt - 1) / p.tpt;
    b = p.fd_tn.div(i);
    k = i - b * tiles;
  }
  const Row r = row_at(p, b);
  const int t0 = (tiles - 1 - k) * p.tpt;
  e.row = b;
  e.n0 = r.n0 + t0;
  e.ntok = min(p.tpt, r.ntok - t0);
  e.pos0 = r.start + t0;
  e.len = r.len;
  n = tile_walk(p, e.pos0, e.ntok, e.len, e.jlo, e.ns);
  tile_keys(p, r.start, r.ntok, r.len, e.rlo, e.rhi);
}

// Lists the pieces.  With W key tiles to walk over all units, cutting the
// walks into equal pieces of about W / (k CTAs) tiles, k = 1 .. kMostRounds; or,
// where the walks are about alike, those behind the last whole round of tiles
// over the CTAs into 2 .. kMostTail pieces; or not at all: whichever ends first
// by the estimate below.  The code runs once, from instruction caches that hold
// none of it, so it is kept short: three passes over the tiles through one loop
// body.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ PrefillParams p) {
  __shared__ long long sm_long[kPlanThreads / 32];
  __shared__ int sm_rows[kPlanRows + 1];
  __shared__ unsigned long long sum;
  __shared__ int most, cut, cut_from, slots, joins, join_most;
  __shared__ int most_of[kMostRounds], pieces_of[kMostRounds], longest_of[kMostRounds];
  launch_dependents();
  grid_dependency_wait();
  const int tid = threadIdx.x, lane = tid & 31;
  if (tid < kMostRounds) pieces_of[tid] = longest_of[tid] = 0;
  if (tid == 0) {
    sum = 0;
    most = cut_from = slots = joins = join_most = 0;
    cut = INT_MAX;
  }
  // tiles of the rows
  int tiles;
  int* rows = p.B <= kPlanRows ? sm_rows : p.row_tiles;
  if (p.offsets) {
    // (offsets that do not rise may name a token again and again: tiles past
    // those that rising ones can make are left out, so that there is room for
    // every piece of the others; prefill_shape)
    long long before = 0;
    for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
      const int b = b0 + tid;
      long long n = 0, total;
      if (b < p.B) {
        int begin, end;
        row_tokens(p.offsets, b, p.N, begin, end);
        n = (end - begin + p.tpt - 1) / p.tpt;
      }
      const long long at = before + block_scan(n, sm_long, total);
      if (b < p.B) rows[b] = static_cast<int>(min(at, static_cast<long long>(p.cap_tiles)));
      before += total;
    }
    tiles = static_cast<int>(min(before, static_cast<long long>(p.cap_tiles)));
    if (tid == 0) rows[p.B] = tiles;
  } else {
    tiles = p.B * ((p.N + p.tpt - 1) / p.tpt);
  }
  __syncthreads();
  const bool once = tiles <= kPlanThreads;   // a tile a thread: looked at once
  int n = 0, before = 0;
  Entry e;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {     // the sum; the cuts; the list
    unsigned long long s = 0;
    int longest = 0;
#pragma unroll 1
    for (int i0 = 0; i0 < tiles; i0 += kPlanThreads) {
      const bool in = i0 + tid < tiles;
      if (in && (pass == 0 || !once)) plan_tile(p, rows, i0 + tid, e, n);
      if (pass == 0) {
        if (in) {
          s += n;
          longest = max(longest, n);
        }
      } else if (pass == 1) {
#pragma unroll
        for (int k = 0; k < kMostRounds; ++k) {
          // (an estimate: quotients in fp32)
          const float c = fmaxf(ceilf(__fdividef(n, most_of[k])), 1.f);
          const int a = __reduce_add_sync(0xffffffffu, in ? static_cast<int>(c) : 0);
          const int b = __reduce_max_sync(
              0xffffffffu, in ? static_cast<int>(ceilf(__fdividef(n, c))) : 0);
          if (lane == 0) {
            atomicAdd(&pieces_of[k], a);
            atomicMax(&longest_of[k], b);
          }
        }
      } else {
        const int c = !in ? 0 : (n > cut && i0 + tid >= cut_from ? (n + cut - 1) / cut : 1);
        // Where a thread has one tile, the longest pieces go first, by quarters of
        // the longest: the short ones level the CTAs (in the tiles' order / so: two
        // chunks of 512 beside fourteen single tokens 95 / 87 us, three of 1000 245
        // / 212, four of 300 140 / 132; four prompts from 0 on alike).  More tiles
        // level themselves, and their rows' keys should stay together in L2.  16
        // bits a quarter: cuts make at most kMostRounds CTAs' pieces beside a
        // tile's first.
        int quarter = 0;
        if (once && c > 0) {
          const float m = static_cast<float>(cut_from > 0 ? most : min(most, cut));
          quarter = static_cast<int>(fminf(fmaxf(4.f - __fdividef(4.f * n, c * m), 0.f), 3.f));
        }
        long long total;
        const long long ahead =
            block_scan(static_cast<long long>(c) << (16 * quarter), sm_long, total);
        int at = before + static_cast<int>(ahead);
        if (once) {
          at = static_cast<int>(ahead >> (16 * quarter) & 0xffff);
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            const int x = static_cast<int>(total & 0xffff);
            if (k < quarter) at += x;
            before += x;
            total >>= 16;
          }
        }
        before += static_cast<int>(total);
        int slot = -1;
        if (c > 1) {
          slot = atomicAdd(&slots, c);
          if (slot + c <= p.cap_slots) {
            JoinEntry j = {p.offsets ? 0 : e.row, e.n0, e.ntok, slot, c, {0, 0, 0}};
            p.joins[atomicAdd(&joins, 1)] = j;
            atomicMax(&join_most, c);
          } else {                           // (never: cap_slots holds every cut)
            slot = -1;
          }
        }
        // the first n % c pieces have a key tile more; a tile's thread writes a
        // few pieces, its warp many
        const auto put = [&](Entry x, int n, int c, int k, int slot, int at) {
          const int each = n / c, more = n - each * c;
          x.s0 = k * each + min(k, more);
          x.s1 = x.s0 + each + (k < more);
          x.slot = slot < 0 ? -1 : slot + k;
          p.entries[at + k] = x;
        };
        constexpr int OWN = 6;
        if (c <= OWN) {
#pragma unroll 1
          for (int k = 0; k < c; ++k) put(e, n, c, k, slot, at);
        }
        for (unsigned m = __ballot_sync(0xffffffffu, c > OWN); m; m &= m - 1) {
          const int l = __ffs(m) - 1;
          const auto from = [&](int v) { return __shfl_sync(0xffffffffu, v, l); };
          const Entry x = {from(e.row), from(e.n0), from(e.ntok), from(e.pos0), from(e.len), 0, 0,
                           0, from(e.jlo), from(e.ns), from(e.rlo), from(e.rhi)};
          const int xn = from(n), xc = from(c), xs = from(slot), xa = from(at);
          for (int k = lane; k < xc; k += 32) put(x, xn, xc, k, xs, xa);
        }
      }
    }
    if (pass == 0) {
      longest = __reduce_max_sync(0xffffffffu, longest);
#pragma unroll
      for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (lane == 0) {
        atomicAdd(&sum, s);
        atomicMax(&most, longest);
      }
      __syncthreads();
      if (tid < kMostRounds) {
        // (never less than the share, so that there is room for the cut tiles'
        // pieces, which are at most twice their key tiles by this)
        const float x = static_cast<float>(sum) * p.units / (p.grid * (tid + 1)) * 1.000001f + 1.f;
        most_of[tid] = x < 2e9f ? static_cast<int>(x) : INT_MAX;
      }
      __syncthreads();
      if (most <= most_of[kMostRounds - 1]) ++pass;      // nothing to cut
    } else if (pass == 1) {
      __syncthreads();
      if (tid < 32) {
        // key tiles that a CTA walks to the end: a whole tile costs one more, a
        // piece kCutTiles, the joins kJoinTiles.  Lane 0: no cuts; then the
        // kMostRounds cuts of all; then the tails.
        const float W = static_cast<float>(sum) * p.units, longest = most;
        const int k = lane - 1, c = lane - kMostRounds + 1;
        int from = 0, limit = INT_MAX;
        int pieces = tiles * p.units;
        float whole = 0.f, length = longest, rest = W, extra = 1.f;
        // (within 2 / 10 / 30 / 100 %: 2048 tokens after 14336 386 / 345 / 345 / 345 us,
        // after 30720 728 / 686 / 686 / 686; other chunks are one or the other by far)
        const bool alike = W * 1.1f > longest * pieces;
        bool can = k < 0;
        if (k >= 0 && k < kMostRounds) {
          limit = most_of[k];
          can = most > limit;
          pieces = pieces_of[k] * p.units;
          length = longest_of[k];
        } else if (k >= kMostRounds && c <= kMostTail) {
          const int rounds = p.fd_grid.div(pieces);
          from = p.fd_units.div(rounds * p.grid);
          limit = static_cast<int>(__fdividef(longest, c) * 1.000001f) + 1;
          can = rounds > 0 && limit < most && alike;
          pieces = (tiles - from) * p.units * c;
          length = limit;
          rest = W - __fdividef(W, tiles) * from;
          whole = rounds * (longest + 1.f);
        }
        if (k >= 0) extra = kCutTiles;
        // (level but for the last pieces: of any length, or short ones, of which half
        // the longest is left: none of it / a quarter / half / three quarters / all, 32
        // rows of which four bring 300 tokens, H = 16, h_kv = 4 138 / 137 / 126 / 125 /
        // 124 us, four chunks of 300 73 / 73 / 73 / 68 / 73, two of 1024 289 / 289 / 306 /
        // 306 / 306; others alike)
        const float even = fmaxf(__fdividef(rest + pieces * extra, p.grid) +
                                     (once && !alike ? 0.5f * length : length),
                                 length + extra);
        float end = whole + fminf((p.fd_grid.div(pieces - 1) + 1) * (length + extra), even);
        if (k >= 0) end += kJoinTiles + __fdividef(0.5f * pieces, p.grid);   // (its parts' bytes)
        if (!can) end = INFINITY;
        float best = end;
#pragma unroll
        for (int o = 16; o; o >>= 1) best = fminf(best, __shfl_xor_sync(0xffffffffu, best, o));
        if (lane == __ffs(__ballot_sync(0xffffffffu, end == best)) - 1) {
          cut = limit;
          cut_from = from;
        }
      }
      __syncthreads();
    }
  }
  __syncthreads();
  if (tid == 0) {
    Counters c;
    c.items = static_cast<unsigned>(before) * p.units;
    c.next = p.grid;
    c.joins = joins;
    c.most = join_most;
    *p.counters = c;
  }
}

// ---------------------------------------------------------------- the main kernel

static_assert(kMostTail <= 2 * kMostRounds, "room for a tail's pieces");

// GROUPED: how the boxes of a key tile land (Boxes).
template <int D, bool GROUPED>
struct Cfg {
  static constexpr int NCH = D / 64;
  static constexpr int TILE_BYTES = NCH * CHUNK;
  // of a K or V tile, in 16 bytes: from 64 columns to 64, from 8 keys to 8
  static constexpr uint32_t CHUNK16 = GROUPED ? 64 : CHUNK / 16, GROUP16 = GROUPED ? D : 64;
  static constexpr int STAGES = D == 64 ? 4 : (D == 128 ? 3 : 1);
  // d = 256: O takes 256 columns of tensor memory, and P buffers of their own
  // let the one S buffer be refilled once the softmax has loaded it.
  static constexpr bool SEP = D == 256;
  // key halves a warp (d = 128, N = 8192, pages of 16 / 128: 713 / 712 us; one warp
  // a row, with three S buffers, 882 / 958.  d = 256: one warp a row, since two O
  // parts would not fit)
  static constexpr int NHALF = D <= 128 ? 2 : 1;
  static constexpr int NSB = D == 64 ? 3 : (D == 128 ? 2 : 1);
  static constexpr int NPB = SEP ? 2 : NSB;
  static constexpr uint32_t TM_S = 0;
  static constexpr uint32_t TM_P = SEP ? 128 * NSB : TM_S;
  static constexpr uint32_t P_STRIDE = SEP ? 64 : 128;
  static constexpr uint32_t TM_O = SEP ? TM_P + 64 * NPB : 128 * NSB;
  static constexpr int OCOLS = D * NHALF;
  static constexpr uint32_t TM_COLS = 512;
  static_assert(TM_O + OCOLS <= TM_COLS, "tensor memory budget");
  static constexpr int EPI_WARP0 = 3 + 4 * NHALF;
  static constexpr int WARPS = EPI_WARP0 + 4 + 1;
  static constexpr int THREADS = 32 * WARPS;
  // a tile's mask slot is free again before the producer reaches the tile
  // kRing further on: it writes tile g's mask, at the earliest, once K of tile
  // g - 1 is on its way, when S of g - 1 - STAGES is done, so that the softmax
  // has read the mask of g - 1 - STAGES - NSB (before it lets go of the S buffer)
  static_assert(1 + STAGES + NSB <= kRing, "mask ring");
};

// A piece as the roles see it.
struct alignas(16) Item {
  int n0, ntok, pos0, len;      // n0 < 0: no more pieces
  int s0, nst, slot, jlo;
  int ns, rlo, rhi, batch;      // [rlo, rhi): the keys that the row's tokens see, beside the sinks
  int kvh, h0, nh, row;
};

template <class C>
struct Smem {
  alignas(1024) uint8_t q[C::TILE_BYTES];
  alignas(1024) uint8_t k[C::STAGES][C::TILE_BYTES];
  alignas(1024) uint8_t v[C::STAGES][C::TILE_BYTES];
  Item item[kItems];
  alignas(16) uint32_t mask[kRing][4];    // a key tile's keys that exist
  uint64_t item_full[kItems], item_empty[kItems];
  uint64_t q_full, q_empty;
  uint64_t k_full[C::STAGES], k_empty[C::STAGES];
  uint64_t v_full[C::STAGES], v_empty[C::STAGES];
  uint64_t s_full[C::NSB], s_free[C::NSB];
  uint64_t p_full[C::NPB * C::NHALF];
  uint64_t pv_done[C::NPB];
  uint64_t o_free, o_done, stats_full;
  uint64_t mma_done, pv_mma_done;
  float ostat[2 * C::NHALF][BM];
  uint32_t tmem_base;
  int abort;
};

static_assert(sizeof(Smem<Cfg<64, false>>) <= 232448 && sizeof(Smem<Cfg<128, true>>) <= 232448 &&
                  sizeof(Smem<Cfg<256, true>>) <= 232448,
              "shared memory of a block");

enum Site {
  kSiteItem = 41, kSiteItemSlot, kSiteQ, kSiteK, kSiteV, kSiteMmaQ, kSiteMmaK, kSiteMmaS,
  kSiteMmaP, kSiteMmaV, kSiteMmaO, kSiteSmS, kSiteSmP, kSiteSmO, kSiteEpi, kSiteDrain
};

__device__ __forceinline__ void fail(int* status, volatile int* abort, int site) {
  if ((threadIdx.x & 31) == 0) {
    atomicCAS(status, 0, status_code(site));
    *abort = 1;
  }
}

// 4-D tiled load global -> shared.
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int c0, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int c0, int c1, int c2, int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3),
      "r"(c4)
      : "memory");
}

// The next announced piece; false at the end, or after a wait that gave up.
template <class S>
__device__ __forceinline__ bool next_item(S& sm, uint32_t& k, Item& t, int* status) {
  const uint32_t b = k % kItems;
  if (!mbar_wait_warp(&sm.item_full[b], (k / kItems) & 1, &sm.abort, kWaitTimeoutNs)) {
    fail(status, &sm.abort, kSiteItem);
    return false;
  }
  t = sm.item[b];
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&sm.item_empty[b]);
  ++k;
  return t.n0 >= 0;
}

// The key tiles of a piece, one after the other.
struct Walk {
  int s, j;                    // step of the tile's walk, key tile
  __device__ explicit Walk(const Item& t) : s(t.s0), j(s < t.ns ? s : t.jlo + (s - t.ns)) {}
  __device__ __forceinline__ void next(const Item& t) { j = ++s == t.ns ? t.jlo : j + 1; }
};

// A place in a ring of N barriers.
template <int N>
struct Ring {
  int at = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++at == N) {
      at = 0;
      phase ^= 1;
    }
  }
};

// The boxes of a key tile.  Whole groups of eight slots (GROUPED): a box a
// page, which lands as [group][64 columns][slot].  Else a box a page (or 128
// slots of one) and 64 columns, which lands as [64 columns][slot]; box x is
// columns 64 (x % EACH) of page x / EACH.  A lane issues the boxes lane, lane +
// 32, ..  A page's number is asked for a tile ahead and not looked at before:
// the producer is the kernel's pace maker, and a look costs it the load's
// 700 cycles.
template <int D, bool GROUPED>
struct Boxes {
  static constexpr int EACH = GROUPED ? 1 : D / 64;   // boxes of a page
  const PrefillParams& p;
  const int* row;              // the row's pages
  int head;
  int pages;                   // of the row
  int count;                   // boxes of a tile
  int m, to;                   // this lane's (first) page of a tile, and where it lands
  __device__ Boxes(const PrefillParams& p_, const Item& t)
      : p(p_), row(p_.table + static_cast<long long>(t.row) * p_.max_pages), head(t.kvh) {
    pages = min(p.max_pages, (t.len + p.page_size - 1) / p.page_size);
    count = (p.ppt ? p.ppt : 1) * EACH;
    m = (threadIdx.x & 31) / EACH;
    to = place(threadIdx.x & 31);
  }
  __device__ __forceinline__ int place(int x) const {
    return GROUPED ? x * p.page_size * (D * 2)
                   : x % (D / 64) * CHUNK + x / (D / 64) * p.page_size * 128;
  }
  // the tile's first slot in its page
  __device__ __forceinline__ int slot0(int j) const {
    return p.ppt ? 0 : (j - p.fd_tpp.div(j) * p.tpp) * BN;
  }
  // the table's entry of page m of key tile j, -1 where there is none
  __device__ __forceinline__ int entry(int j, int m) const {
    const int i = p.ppt ? j * p.ppt + m : p.fd_tpp.div(j);
    return i < pages ? row[i] : -1;
  }
  __device__ __forceinline__ bool exists(int entry) const {
    return static_cast<unsigned>(entry) < static_cast<unsigned>(p.num_pages);
  }
  __device__ __forceinline__ void box(int x, int entry, int slot0, uint8_t* dst,
                                      const CUtensorMap* map, uint64_t* bar) const {
    // a page that does not exist lies outside the pool
    if constexpr (GROUPED)
      tma_load_5d(dst, map, bar, 0, 0, 0,
                  exists(entry) ? entry * p.groups + slot0 / 8 : p.eights, head);
    else
      tma_load_4d(dst, map, bar, 64 * (x % (D / 64)), slot0, head,
                  exists(entry) ? entry : p.num_pages);
  }
  // first: entry(j, m)
  __device__ __forceinline__ void load(int j, int first, uint8_t* dst, const CUtensorMap* map,
                                       uint64_t* bar) const {
    const int lane = threadIdx.x & 31;
    if (lane < count) box(lane, first, slot0(j), dst + to, map, bar);
    if (count > 32) {
      for (int x = lane + 32; x < count; x += 32)
        box(x, entry(j, x / EACH), slot0(j), dst + place(x), map, bar);
    }
  }
};

// A key tile's mask where pages may be missing, or its boxes are more than the
// lanes.
template <class B>
__device__ __forceinline__ void key_words(const PrefillParams& p, const B& boxes, int j,
                                          uint32_t* words) {
  const int lane = threadIdx.x & 31;
  for (int w = 0; w < 4; ++w) {
    const int x = 32 * w + lane;               // the lane's key of the tile
    const int m = p.ppt ? p.fd_ps.div(x) : 0;
    bool on = p.ppt ? x < p.kt
                    : x < p.page_size - (j - p.fd_tpp.div(j) * p.tpp) * BN;
    on = on && boxes.exists(boxes.entry(j, m));
    const uint32_t word = __ballot_sync(0xffffffffu, on);
    if (lane == 0) words[w] = word;
  }
}

// A key tile's mask; whole: the slots whose masks hide nothing.
template <class B>
__device__ __forceinline__ void set_mask(const PrefillParams& p, const B& boxes, int j, int page,
                                         uint32_t& whole, int slot, uint32_t* words) {
  const int lane = threadIdx.x & 31;
  const int keys = p.ppt ? p.kt : p.page_size - boxes.slot0(j);
  if (boxes.count <= 32 && keys >= p.kt &&
      __all_sync(0xffffffffu, lane >= boxes.count || boxes.exists(page))) {
    if (lane < 4) words[lane] = bits_below(p.kt - 32 * lane);
    whole |= 1u << slot;
  } else {
    key_words(p, boxes, j, words);
    whole &= ~(1u << slot);
  }
  __syncwarp();
}

// 16 bytes (part e % 8 of key e / 8, whatever the swizzle's order) of the 64
// columns c of a tile.
template <class C>
__device__ __forceinline__ uint4& v_part(uint8_t* tile, int c, int e) {
  return *reinterpret_cast<uint4*>(tile + 16 * (c * C::CHUNK16 + (e >> 6) * C::GROUP16 + (e & 63)));
}

template <int D, bool GROUPED>
__global__ void __launch_bounds__(Cfg<D, GROUPED>::THREADS, 1)
    prefill_kernel(const __grid_constant__ PrefillParams p) {
  using C = Cfg<D, GROUPED>;
  using S = Smem<C>;
  extern __shared__ uint8_t smem_raw[];
  const uintptr_t raw = reinterpret_cast<uintptr_t>(smem_raw);
  const uintptr_t aligned = (raw + 1023) & ~static_cast<uintptr_t>(1023);
  if (aligned - raw + sizeof(S) > dynamic_smem_size()) {
    if (threadIdx.x == 0) atomicCAS(p.status, 0, status_code(kSiteSmemLayout));
    return;
  }
  S& sm = *reinterpret_cast<S*>(aligned);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  volatile int* abort = &sm.abort;
  launch_dependents();
  if (threadIdx.x == 0) {
    sm.abort = 0;
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&sm.item_full[i], 1);
      mbar_init(&sm.item_empty[i], C::WARPS - 1);
    }
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, 1);
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&sm.k_full[s], 1);
      mbar_init(&sm.k_empty[s], 1);
      mbar_init(&sm.v_full[s], 1);
      mbar_init(&sm.v_empty[s], 1);
    }
    for (int b = 0; b < C::NSB; ++b) {
      mbar_init(&sm.s_full[b], 1);
      mbar_init(&sm.s_free[b], 4);
    }
    for (int b = 0; b < C::NPB; ++b) {
      for (int h = 0; h < C::NHALF; ++h) mbar_init(&sm.p_full[b * C::NHALF + h], 4);
      mbar_init(&sm.pv_done[b], 1);
    }
    mbar_init(&sm.o_free, 4);
    mbar_init(&sm.o_done, 1);
    mbar_init(&sm.stats_full, 32 * 4 * C::NHALF);
    mbar_init(&sm.mma_done, 1);
    mbar_init(&sm.pv_mma_done, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&sm.tmem_base, C::TM_COLS);
    tmem_relinquish();
  }
  // Rows of V that no load writes (a tile of fewer than 128 keys): zeros, since
  // P is 0 there and 0 NaN is NaN.
  if (p.kt < BN) {
    for (int s = 0; s < C::STAGES; ++s)
      for (int c = 0; c < C::NCH; ++c)
        for (int e = p.kt * 8 + threadIdx.x; e < BN * 8; e += C::THREADS)
          v_part<C>(sm.v[s], c, e) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = sm.tmem_base;
  // (every warp: the waits on barriers are bounded, this one is not)
  grid_dependency_wait();

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      prefetch_tmap(&p.tq);
      prefetch_tmap(&p.tk);
      prefetch_tmap(&p.tv);
    }
    const uint32_t items = p.counters->items;
    uint32_t i = blockIdx.x, q_it = 0, g = 0, whole = 0;   // whole: masks that hide nothing
    Ring<C::STAGES> st;
    bool ok = true;
    for (uint32_t k = 0; ok; ++k) {
      const uint32_t b = k % kItems;
      Item t;
      uint32_t next = 0;
      const int e = p.fd_units.div(i), u = static_cast<int>(i) - e * p.units;
      if (i < items) {
        const Entry en = p.entries[e];
        if (lane == 0) next = atomicAdd(&p.counters->next, 1u);   // (used after this piece)
        t.n0 = en.n0;
        t.ntok = en.ntok;
        t.pos0 = en.pos0;
        t.len = en.len;
        t.s0 = en.s0;
        t.nst = en.s1 - en.s0;
        t.slot = en.slot < 0 ? -1 : en.slot * p.units + u;
        t.jlo = en.jlo;
        t.ns = en.ns;
        t.rlo = en.rlo;
        t.rhi = en.rhi;
        t.batch = p.offsets ? 0 : en.row;
        t.kvh = p.fd_parts.div(u);
        const int part = u - t.kvh * p.parts;
        t.h0 = t.kvh * p.group + part * p.gh;
        t.nh = min(p.gh, p.group - part * p.gh);
        t.row = en.row;
      } else {
        t.n0 = -1;
        t.nst = 0;
      }
      if (!mbar_wait_warp(&sm.item_empty[b], ((k / kItems) & 1) ^ 1, abort, kWaitTimeoutNs)) {
        fail(p.status, abort, kSiteItemSlot);
        break;
      }
      if (lane == 0) {
        sm.item[b] = t;
        mbar_arrive(&sm.item_full[b]);
      }
      if (t.n0 < 0) break;
      const Boxes<D, GROUPED> boxes(p, t);
      Walk walk(t);
      int ahead = t.nst > 0 ? boxes.entry(walk.j, boxes.m) : 0;
      // the keys of every tile are all there if its pages are (asking tile by tile
      // where a page's last tile is smaller: 685 us where 624 stand below, for 36.8
      // instead of 37.2 with pages of 1500)
      const bool plain = boxes.count <= 32 && (p.ppt || p.page_size % BN == 0);
      for (int j = 0; j < t.nst; ++j) {
        const int jt = walk.j, page = ahead;
        walk.next(t);
        if (j + 1 < t.nst) ahead = boxes.entry(walk.j, boxes.m);
        // which keys exist: mostly all, as the mask's slot says already.  One vote
        // on this and on the wait, with all it takes ready before: with a vote each
        // d = 64, N = 8192, pages of 16 take 709 us, not 624.  With one stage the
        // wait is what everyone waits for, and nothing follows it (d = 256, two
        // sequences of 3001: 296 us, with one vote 304).
        const int slot = g % kRing;
        int fine = plain && (whole >> slot & 1u) && (lane >= boxes.count || boxes.exists(page));
        if constexpr (C::STAGES == 1) {
          if (!__all_sync(0xffffffffu, fine))
            set_mask(p, boxes, jt, page, whole, slot, sm.mask[slot]);
          if (!mbar_wait_warp(&sm.k_empty[st.at], st.phase ^ 1, abort, kWaitTimeoutNs)) {
            fail(p.status, abort, kSiteK);
            ok = false;
            break;
          }
        } else {
          asm volatile("" : "+r"(fine));
          const bool got = mbar_wait(&sm.k_empty[st.at], st.phase ^ 1, abort, kWaitTimeoutNs);
          if (!__all_sync(0xffffffffu, got && fine)) {
            if (!__all_sync(0xffffffffu, got)) {
              fail(p.status, abort, kSiteK);
              ok = false;
              break;
            }
            set_mask(p, boxes, jt, page, whole, slot, sm.mask[slot]);
          }
        }
        if (lane == 0) mbar_arrive_expect_tx(&sm.k_full[st.at], p.kt * (D * 2));
        boxes.load(jt, page, sm.k[st.at], &p.tk, &sm.k_full[st.at]);
        __syncwarp();
        ++g;
        st.next();
        if (j == 0) {
          // Q after the first keys: its buffer is free only when the piece
          // before has no more products to issue
          if (!mbar_wait_warp(&sm.q_empty, (q_it & 1) ^ 1, abort, kWaitTimeoutNs)) {
            fail(p.status, abort, kSiteQ);
            ok = false;
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(&sm.q_full, p.gh * p.tpt * (D * 2));
          if (lane < C::NCH)
            tma_load_4d(sm.q + lane * CHUNK, &p.tq, &sm.q_full, 64 * lane, t.h0, t.n0, t.batch);
          __syncwarp();
          ++q_it;
        }
      }
      i = __shfl_sync(0xffffffffu, next, 0);
    }
    // no copy may still be landing when the CTA exits
    if (q_it > 0 && !mbar_wait_warp(&sm.q_full, (q_it - 1) & 1, nullptr, kWaitTimeoutNs))
      fail(p.status, abort, kSiteDrain);
    for (int s = 0; s < C::STAGES; ++s) {
      if (g > static_cast<uint32_t>(s) &&
          !mbar_wait_warp(&sm.k_full[s], ((g - 1 - s) / C::STAGES) & 1, nullptr, kWaitTimeoutNs))
        fail(p.status, abort, kSiteDrain);
    }
  } else if (warp == C::WARPS - 1) {
    // ------------------------------------------------------------ V producer
    uint32_t k = 0, v_it = 0;
    Ring<C::STAGES> st;
    bool ok = true;
    for (Item t; ok && next_item(sm, k, t, p.status);) {
      const Boxes<D, GROUPED> boxes(p, t);
      Walk walk(t);
      int ahead = t.nst > 0 ? boxes.entry(walk.j, boxes.m) : 0;
      for (int j = 0; j < t.nst; ++j) {
        const int jt = walk.j, page = ahead;
        walk.next(t);
        if (j + 1 < t.nst) ahead = boxes.entry(walk.j, boxes.m);
        if (!mbar_wait_warp(&sm.v_empty[st.at], st.phase ^ 1, abort, kWaitTimeoutNs)) {
          fail(p.status, abort, kSiteV);
          ok = false;
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(&sm.v_full[st.at], p.kt * (D * 2));
        boxes.load(jt, page, sm.v[st.at], &p.tv, &sm.v_full[st.at]);
        __syncwarp();
        ++v_it;
        st.next();
      }
    }
    for (int s = 0; s < C::STAGES; ++s)
      if (v_it > static_cast<uint32_t>(s) &&
          !mbar_wait_warp(&sm.v_full[s], ((v_it - 1 - s) / C::STAGES) & 1, nullptr, kWaitTimeoutNs))
        fail(p.status, abort, kSiteDrain);
  } else if (warp == 1) {
    // ------------------------------------------------------------ S issuer
    constexpr uint32_t kIdescS = idesc_bf16_f32(BM, BN, 0, 0);
    const uint64_t dq0 = sdesc_sw128(smem_u32(sm.q), 16, 1024);
    uint32_t k = 0, q_it = 0, g = 0;
    bool ok = true;
    for (Item t; ok && next_item(sm, k, t, p.status);) {
      for (int j = 0; j < t.nst; ++j, ++g) {
        const uint32_t b = g % C::NSB;
        if (j == 0) {
          if (!mbar_wait_warp(&sm.q_full, q_it & 1, abort, kWaitTimeoutNs)) {
            fail(p.status, abort, kSiteMmaQ);
            ok = false;
            break;
          }
          ++q_it;
        }
        if (g >= static_cast<uint32_t>(C::NSB) &&
            !mbar_wait_warp(C::SEP ? &sm.s_free[b] : &sm.pv_done[b], ((g / C::NSB) & 1) ^ 1, abort,
                            kWaitTimeoutNs)) {
          fail(p.status, abort, kSiteMmaS);
          ok = false;
          break;
        }
        const int st = g % C::STAGES;
        if (!mbar_wait_warp(&sm.k_full[st], (g / C::STAGES) & 1, abort, kWaitTimeoutNs)) {
          fail(p.status, abort, kSiteMmaK);
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint64_t dk0 = sdesc_sw128(smem_u32(sm.k[st]), 16, C::GROUP16 * 16);
#pragma unroll
        for (int kk = 0; kk < C::NCH * 4; ++kk)
          mma_bf16_ss_w(tmem + C::TM_S + 128 * b, dq0 + ((kk / 4) * CHUNK + (kk % 4) * 32) / 16,
                        dk0 + ((kk / 4) * C::CHUNK16 + (kk % 4) * 2), kIdescS, kk > 0 ? 1u : 0u);
        mma_commit_w(&sm.k_empty[st]);
        mma_commit_w(&sm.s_full[b]);
        if (j == t.nst - 1) mma_commit_w(&sm.q_empty);
      }
    }
    // every product issued by this thread must finish before exit
    mma_commit_w(&sm.mma_done);
    if (!mbar_wait_warp(&sm.mma_done, 0, nullptr, kWaitTimeoutNs))
      fail(p.status, abort, kSiteDrain);
  } else if (warp == 2) {
    // ------------------------------------------------------------ P V issuer
    constexpr uint32_t kIdescPV = idesc_bf16_f32(BM, D, 0, 1);
    uint32_t k = 0, g = 0, o_it = 0;
    bool ok = true;
    for (Item t; ok && next_item(sm, k, t, p.status);) {
      // the tiles that may hold keys which no token of the row sees
      const int edge_hi = key_tile(p, t.rhi), edge_lo = key_tile(p, t.rlo);
      Walk walk(t);
      for (int j = 0; j < t.nst; ++j, ++g, walk.next(t)) {
        const uint32_t b = g % C::NPB;
        const int st = g % C::STAGES;
        if (!mbar_wait_warp(&sm.v_full[st], (g / C::STAGES) & 1, abort, kWaitTimeoutNs)) {
          fail(p.status, abort, kSiteMmaV);
          ok = false;
          break;
        }
        // slots that no token of the row sees may hold anything, and 0 NaN is
        // NaN: zeros in their place
        if (walk.j >= edge_hi || (walk.j <= edge_lo && t.rlo > 0)) {
          const int pos = tile_pos(p, walk.j);
          for (int e = lane; e < p.kt * 8; e += 32) {
            const int x = pos + e / 8;
            if (x >= t.rhi || (x < t.rlo && x >= p.sinks)) {
#pragma unroll
              for (int c = 0; c < C::NCH; ++c)
                v_part<C>(sm.v[st], c, e) = make_uint4(0, 0, 0, 0);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (j == 0) {
          if (!mbar_wait_warp(&sm.o_free, (o_it & 1) ^ 1, abort, kWaitTimeoutNs)) {
            fail(p.status, abort, kSiteMmaO);
            ok = false;
            break;
          }
          ++o_it;
        }
        const uint64_t dv0 = sdesc_sw128(smem_u32(sm.v[st]), C::CHUNK16 * 16, C::GROUP16 * 16);
#pragma unroll
        for (int h = 0; h < C::NHALF; ++h) {
          if (!mbar_wait_warp(&sm.p_full[b * C::NHALF + h], (g / C::NPB) & 1, abort,
                              kWaitTimeoutNs)) {
            fail(p.status, abort, kSiteMmaP);
            ok = false;
            break;
          }
          tc_fence_after_sync();
          constexpr int KH = BN / 16 / C::NHALF;
#pragma unroll
          for (int kk = 0; kk < KH; ++kk)
            mma_bf16_ts_w(tmem + C::TM_O + D * h,
                          tmem + C::TM_P + C::P_STRIDE * b + (BN / C::NHALF) * h + kk * 8,
                          dv0 + (h * KH + kk) * 2 * C::GROUP16, kIdescPV,
                          (j == 0 && kk == 0) ? 0u : 1u);
        }
        if (!ok) break;
        mma_commit_w(&sm.v_empty[st]);
        mma_commit_w(&sm.pv_done[b]);
        if (j == t.nst - 1) mma_commit_w(&sm.o_done);
      }
    }
    mma_commit_w(&sm.pv_mma_done);
    if (!mbar_wait_warp(&sm.pv_mma_done, 0, nullptr, kWaitTimeoutNs))
      fail(p.status, abort, kSiteDrain);
  } else if (warp >= C::EPI_WARP0) {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;           // the thread's row of the tile
    const int tr = p.fd_gh.div(r), hr = r - tr * p.gh;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const bool st32 = ((reinterpret_cast<uintptr_t>(p.o) | (p.ob * 2) | (p.oh * 2) | (p.ot * 2)) & 31) == 0;
    uint32_t k = 0, e_it = 0;
    for (Item t; next_item(sm, k, t, p.status);) {
      const bool valid = tr < t.ntok && hr < t.nh;
      __nv_bfloat16* out = p.o + t.batch * p.ob + (t.h0 + hr) * p.oh + (t.n0 + tr) * p.ot;
      float* lse = p.lse + (static_cast<long long>(t.batch) * p.H + t.h0 + hr) * p.N + t.n0 + tr;
      const long long part = static_cast<long long>(t.slot) * p.slot_rows + r;
      if (t.nst == 0) {                          // nothing to see: O = 0, LSE = -inf
        if (valid) {
#pragma unroll 4
          for (int i = 0; i < D / 8; ++i) reinterpret_cast<uint4*>(out)[i] = make_uint4(0, 0, 0, 0);
          *lse = -INFINITY;
        }
        continue;
      }
      const uint32_t ph = e_it & 1;
      ++e_it;
      if (!mbar_wait_warp(&sm.stats_full, ph, abort, kPieceTimeoutNs) ||
          !mbar_wait_warp(&sm.o_done, ph, abort, kPieceTimeoutNs)) {
        fail(p.status, abort, kSiteEpi);
        break;
      }
      tc_fence_after_sync();
      // the halves against the larger maximum: O = sum_h a_h O_h / sum_h a_h l_h
      float a[C::NHALF], m = -INFINITY, l = 0.f;
#pragma unroll
      for (int h = 0; h < C::NHALF; ++h) m = fmaxf(m, sm.ostat[C::NHALF + h][r]);
#pragma unroll
      for (int h = 0; h < C::NHALF; ++h) {
        const float mh = sm.ostat[C::NHALF + h][r];
        a[h] = mh == -INFINITY ? 0.f : ex2_approx(mh - m);
        l += a[h] * sm.ostat[h][r];
      }
      // (a sum that is not a number stays one)
      const float inv_l = l == 0.f ? 0.f : 1.f / l;
      const float lse_row = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
#pragma unroll
      for (int h = 0; h < C::NHALF; ++h) a[h] *= inv_l;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t orr[C::NHALF][32];
#pragma unroll
        for (int h = 0; h < C::NHALF; ++h) tmem_ld_x32(t_lane + C::TM_O + D * h + 32 * c, orr[h]);
        tmem_wait_ld();
#pragma unroll
        for (int h = 0; h < C::NHALF; ++h) reg_fence<32>(orr[h]);
        if (c == D / 32 - 1) {
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.o_free);
        }
        float o[32];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const auto pair = [&](int h) {
            return f2_make(__uint_as_float(orr[h][e]), __uint_as_float(orr[h][e + 1]));
          };
          uint64_t x = f2_mul(pair(0), f2_make(a[0], a[0]));
#pragma unroll
          for (int h = 1; h < C::NHALF; ++h) x = f2_fma(pair(h), f2_make(a[h], a[h]), x);
          f2_split(x, o[e], o[e + 1]);
        }
        if (!valid) continue;
        if (t.slot >= 0) {
          float* dst = p.o_part + part * D + 32 * c;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t r8[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) r8[e] = __float_as_uint(o[8 * i + e]);
            st_global_v8(dst + 8 * i, r8);
          }
        } else {
          __nv_bfloat16* dst = out + 32 * c;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t pk8[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
              pk8[e] = pack_bf16x2(o[16 * i + 2 * e], o[16 * i + 2 * e + 1]);
            if (st32) {
              st_global_v8(dst + 16 * i, pk8);
            } else {
              uint4* d4 = reinterpret_cast<uint4*>(dst + 16 * i);
              d4[0] = make_uint4(pk8[0], pk8[1], pk8[2], pk8[3]);
              d4[1] = make_uint4(pk8[4], pk8[5], pk8[6], pk8[7]);
            }
          }
        }
      }
      if (valid) {
        if (t.slot >= 0)
          p.lse_part[part] = lse_row;
        else
          *lse = lse_row;
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int quarter = warp & 3;
    const int hf = (warp - 3) >> 2;
    constexpr int NC = BN / C::NHALF;            // keys of a tile that this warp takes
    const int r = quarter * 32 + lane;
    const int tr = p.fd_gh.div(r);
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t t_o = t_lane + C::TM_O + D * hf;
    const float c2 = p.scale_log2;
    uint32_t k = 0, kv_it = 0, e_it = 0;
    bool ok = true;
    for (Item t; ok && next_item(sm, k, t, p.status);) {
      if (t.nst == 0) continue;
      // this row sees keys [.., hi] from lo on or below the sinks (a row behind
      // the tile's last counts as that one)
      const auto last_key = [&](int pos) {
        if (p.causal && pos >= t.len) return -1;
        const long long h = static_cast<long long>(pos) + p.wr;
        return static_cast<int>(h < t.len - 1 ? (h < -1 ? -1 : h) : t.len - 1);
      };
      const int pos = t.pos0 + min(tr, t.ntok - 1), pos_last = t.pos0 + t.ntok - 1;
      const int hi = last_key(pos), lo = max(pos, p.wl) - p.wl;
      // the tiles in between have nothing that some row does not see
      const int edge_hi = key_tile(p, min(last_key(t.pos0), last_key(pos_last)) + 1);
      const int all_lo = max(pos_last, p.wl) - p.wl;
      const int edge_lo = all_lo > 0 ? key_tile(p, min(all_lo, t.len)) : -1;
      float m_ref = -INFINITY, l = 0.f;
      Walk walk(t);
      for (int j = 0; j < t.nst; ++j, walk.next(t)) {
        const uint32_t b = kv_it % C::NSB;
        const uint32_t t_s = t_lane + C::TM_S + 128 * b;
        if (!mbar_wait_warp(&sm.s_full[b], (kv_it / C::NSB) & 1, abort, kWaitTimeoutNs)) {
          fail(p.status, abort, kSiteSmS);
          ok = false;
          break;
        }
        tc_fence_after_sync();
        uint32_t sr[NC];
#pragma unroll
        for (int c = 0; c < NC / 32; ++c) tmem_ld_x32(t_s + NC * hf + 32 * c, sr + 32 * c);
        uint32_t word[NC / 32], whole = ~0u;
#pragma unroll
        for (int w = 0; w < NC / 32; ++w) {
          word[w] = sm.mask[kv_it % kRing][NC / 32 * hf + w];
          whole &= word[w];
        }
        tmem_wait_ld();
        reg_fence<NC>(sr);
        if constexpr (C::SEP) {
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.s_free[b]);
        }
        float s[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) s[c] = __uint_as_float(sr[c]);
        if (whole != ~0u || walk.j >= edge_hi || walk.j <= edge_lo) {
          const int key0 = tile_pos(p, walk.j) + NC * hf;
          const int c_hi = hi - key0, c_lo = lo - key0;
#pragma unroll
          for (int w = 0; w < NC / 32; ++w) {
            const uint32_t on = word[w] & bits_below(c_hi + 1 - 32 * w) &
                                (~bits_below(c_lo - 32 * w) | bits_below(p.sinks - key0 - 32 * w));
            if (__any_sync(0xffffffffu, on != ~0u)) {
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (!((on >> c) & 1u)) s[32 * w + c] = -INFINITY;
            }
          }
        }
        float mx0 = s[0], mx1 = s[1], mx2 = s[2], mx3 = s[3];
#pragma unroll
        for (int c = 4; c + 8 <= NC; c += 8) {
          mx0 = fmax3(mx0, s[c], s[c + 1]);
          mx1 = fmax3(mx1, s[c + 2], s[c + 3]);
          mx2 = fmax3(mx2, s[c + 4], s[c + 5]);
          mx3 = fmax3(mx3, s[c + 6], s[c + 7]);
        }
        mx0 = fmax3(mx0, s[NC - 4], s[NC - 3]);
        mx1 = fmax3(mx1, s[NC - 2], s[NC - 1]);
        const float m_blk = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)) * c2;
        float alpha = 1.f;
        bool rescale = false;
        if (m_ref == -INFINITY) {
          if (m_blk != -INFINITY) {
            alpha = 0.f;
            m_ref = m_blk;
          }
        } else if (m_blk > m_ref + kRescaleSlack) {
          alpha = ex2_approx(m_ref - m_blk);
          m_ref = m_blk;
          rescale = true;
        }
        const float base = m_ref == -INFINITY ? 0.f : m_ref;
        const uint64_t c2x2 = f2_make(c2, c2), nbx2 = f2_make(-base, -base);
        uint64_t rsa = f2_make(0.f, 0.f), rsb = f2_make(0.f, 0.f);
        uint32_t pk[NC / 2];
#pragma unroll
        for (int c = 0; c < NC / 2; c += 2) {
          float a0, a1, a2, a3;
          f2_split(f2_fma(f2_make(s[2 * c], s[2 * c + 1]), c2x2, nbx2), a0, a1);
          f2_split(f2_fma(f2_make(s[2 * c + 2], s[2 * c + 3]), c2x2, nbx2), a2, a3);
          const float p0 = ex2_approx(a0), p1 = ex2_approx(a1);
          const float p2 = ex2_approx(a2), p3 = ex2_approx(a3);
          rsa = f2_add(rsa, f2_make(p0, p1));
          rsb = f2_add(rsb, f2_make(p2, p3));
          pk[c] = pack_bf16x2(p0, p1);
          pk[c + 1] = pack_bf16x2(p2, p3);
        }
        float rs0, rs1, rs2, rs3;
        f2_split(rsa, rs0, rs1);
        f2_split(rsb, rs2, rs3);
        l = l * alpha + ((rs0 + rs1) + (rs2 + rs3));
        const uint32_t pb = kv_it % C::NPB;
        if constexpr (C::SEP) {
          if (kv_it >= static_cast<uint32_t>(C::NPB) &&
              !mbar_wait_warp(&sm.pv_done[pb], ((kv_it / C::NPB) & 1) ^ 1, abort,
                              kWaitTimeoutNs)) {
            fail(p.status, abort, kSiteSmP);
            ok = false;
            break;
          }
          tc_fence_after_sync();
        }
        const uint32_t t_p = t_lane + C::TM_P + C::P_STRIDE * pb + NC * hf;
        tmem_st_x32(t_p, pk);
        if constexpr (NC == 128) tmem_st_x32(t_p + 32, pk + 32);
        if (__any_sync(0xffffffffu, rescale)) {
          // O holds every earlier product before it is scaled
          const uint32_t prev = kv_it - 1;
          if (!mbar_wait_warp(&sm.pv_done[prev % C::NPB], (prev / C::NPB) & 1, abort,
                              kWaitTimeoutNs)) {
            fail(p.status, abort, kSiteSmO);
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint64_t a2 = f2_make(alpha, alpha);
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t orr[32];
            tmem_ld_x32(t_o + 32 * c, orr);
            tmem_wait_ld();
            reg_fence<32>(orr);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float x0, x1;
              f2_split(f2_mul(f2_make(__uint_as_float(orr[2 * i]), __uint_as_float(orr[2 * i + 1])), a2), x0, x1);
              orr[2 * i] = __float_as_uint(x0);
              orr[2 * i + 1] = __float_as_uint(x1);
            }
            tmem_st_x32(t_o + 32 * c, orr);
          }
        }
        tmem_wait_st();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[pb * C::NHALF + hf]);
        ++kv_it;
      }
      if (!ok) break;
      // hand the rows' sums and maxima over, once the epilogue of the piece
      // before has read its own
      ++e_it;
      if (!mbar_wait_warp(&sm.o_free, ((e_it - 1) & 1) ^ 1, abort, kWaitTimeoutNs)) {
        fail(p.status, abort, kSiteEpi);
        break;
      }
      sm.ostat[hf][r] = l;
      sm.ostat[C::NHALF + hf][r] = m_ref;
      mbar_arrive(&sm.stats_full);
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, C::TM_COLS);
  }
}

// ---------------------------------------------------------------- the join

// Cut tiles: per row LSE = log sum_s exp(LSE_s) and O = sum_s exp(LSE_s - LSE)
// O_s, pieces in order of a tree.  Bound by L2's and HBM's latency.  Up to eight
// pieces: a warp has all the pieces of 1, 2 or 4 rows in flight together (eight
// rows piece after piece / so: 64 tokens after 4000, d = 64 24 / 19 us, 128 after
// 8000, d = 128 41 / 37, 32 rows of 4 tokens 183 / 180, 2048 tokens after 30720 691
// / 688); more: a block a row, its warps every fourth piece each.  A kernel of its
// own: the last CTA to finish a tile joining it ran cold code on one SM (one row
// of 5 tokens after some 1000, when a call took 17 us, 40).
template <int D>
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ PrefillParams p) {
  grid_dependency_wait();
  constexpr int PER = D / 32, V = PER == 2 ? 2 : 4, W = 4, SLOTS = 8;
  __shared__ float sm_o[W][D];
  __shared__ float sm_w[W];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const Counters c = *p.counters;
  const bool wide = c.most > SLOTS;
  const int shift = c.most <= 2 ? 2 : (c.most <= 4 ? 1 : 0);
  const int per = 1 << (wide ? 0 : shift);               // rows of a warp (or block)
  const int groups = (p.slot_rows + per - 1) / per;      // of a tile and unit
  const long long total = static_cast<long long>(c.joins) * p.units * groups;
  const long long step = wide ? gridDim.x : gridDim.x * W;
  for (long long x = wide ? blockIdx.x : blockIdx.x * W + warp; x < total; x += step) {
    const int item = static_cast<int>(x / groups);       // (joins times units: below 2^31)
    const int r0 = static_cast<int>(x - static_cast<long long>(item) * groups) * per;
    const int je = p.fd_units.div(item), u = item - je * p.units;
    const JoinEntry j = p.joins[je];
    const int kvh = p.fd_parts.div(u), pt = u - kvh * p.parts;
    const int nh = min(p.gh, p.group - pt * p.gh), h0 = kvh * p.group + pt * p.gh;
    // row r of piece s
    const auto at = [&](int s, int r) {
      return ((j.slot0 + s) * static_cast<long long>(p.units) + u) * p.slot_rows +
             min(r, p.slot_rows - 1);
    };
    const auto load = [&](int s, int r, float* v) {
      const float* src = p.o_part + at(s, r) * D + lane * PER;
#pragma unroll
      for (int i = 0; i < PER; i += V) {
        if constexpr (V == 2) {
          const float2 y = *reinterpret_cast<const float2*>(src + i);
          v[i] = y.x;
          v[i + 1] = y.y;
        } else {
          const float4 y = *reinterpret_cast<const float4*>(src + i);
          v[i] = y.x;
          v[i + 1] = y.y;
          v[i + 2] = y.z;
          v[i + 3] = y.w;
        }
      }
    };
    const auto store = [&](int r, const float* acc, float lse) {
      const int tr = p.fd_gh.div(r), h = r - tr * p.gh;
      if (r >= p.slot_rows || tr >= j.ntok || h >= nh) return;
      const long long tok = j.n0 + tr;
      uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + j.batch * p.ob + (h0 + h) * p.oh +
                                                  tok * p.ot + lane * PER);
#pragma unroll
      for (int i = 0; i < PER / 2; ++i) dst[i] = pack_bf16x2(acc[2 * i], acc[2 * i + 1]);
      if (lane == 0)
        p.lse[(static_cast<long long>(j.batch) * p.H + h0 + h) * p.N + tok] = lse;
    };
    if (!wide) {
      // slot i (lane, and of v): row i % per, piece i / per
      const int i8 = lane % SLOTS, s = i8 >> shift;
      const float a = s < j.pieces ? p.lse_part[at(s, r0 + (i8 & (per - 1)))] : -INFINITY;
      float v[SLOTS][PER];
#pragma unroll
      for (int i = 0; i < SLOTS; ++i) {
        if ((i >> shift) < j.pieces) {
          load(i >> shift, r0 + (i & (per - 1)), v[i]);
        } else {
#pragma unroll
          for (int e = 0; e < PER; ++e) v[i][e] = 0.f;
        }
      }
      float m = a;
#pragma unroll
      for (int o = SLOTS / 2; o; o >>= 1) {
        const float y = __shfl_xor_sync(0xffffffffu, m, o);
        if (o >= per) m = fmaxf(m, y);
      }
      const float base = m == -INFINITY ? 0.f : m;
      // (a NaN stays one: the sum is taken over the values themselves)
      float w = expf(a - base), sum = w;
#pragma unroll
      for (int o = SLOTS / 2; o; o >>= 1) {
        const float y = __shfl_xor_sync(0xffffffffu, sum, o);
        if (o >= per) sum += y;
      }
      w *= sum == 0.f ? 0.f : 1.f / sum;
      const float lse = sum == 0.f ? -INFINITY : base + logf(sum);
#pragma unroll
      for (int i = 0; i < SLOTS; ++i) {
        const float wi = __shfl_sync(0xffffffffu, w, i);
#pragma unroll
        for (int e = 0; e < PER; ++e) v[i][e] *= wi;
      }
#pragma unroll
      for (int o = SLOTS / 2; o; o >>= 1) {
        if (o >= per) {
#pragma unroll
          for (int i = 0; i < o; ++i) {
#pragma unroll
            for (int e = 0; e < PER; ++e) v[i][e] += v[i + o][e];
          }
        }
      }
#pragma unroll
      for (int i = 0; i < SLOTS / 2; ++i) {
        const float x = __shfl_sync(0xffffffffu, lse, i);
        if (i < per) store(r0 + i, v[i], x);
      }
      continue;
    }
    float m = -INFINITY;
    for (int s = lane; s < j.pieces; s += 32) m = fmaxf(m, p.lse_part[at(s, r0)]);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float base = m == -INFINITY ? 0.f : m;
    float acc[PER] = {}, sum = 0.f;
#pragma unroll 4
    for (int s = warp; s < j.pieces; s += W) {
      float v[PER];
      load(s, r0, v);
      const float w = expf(p.lse_part[at(s, r0)] - base);
      sum += w;
#pragma unroll
      for (int i = 0; i < PER; ++i) acc[i] = fmaf(w, v[i], acc[i]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i) sm_o[warp][lane * PER + i] = acc[i];
    if (lane == 0) sm_w[warp] = sum;
    __syncthreads();
    if (warp > 0) continue;
#pragma unroll
    for (int w = 1; w < W; ++w) {
      sum += sm_w[w];
#pragma unroll
      for (int i = 0; i < PER; ++i) acc[i] += sm_o[w][lane * PER + i];
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] *= inv;
    store(r0, acc, sum == 0.f ? -INFINITY : base + logf(sum));
  }
}

// ---------------------------------------------------------------- the host's side

size_t up256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

}  // namespace

// Everything that the sizes determine.
struct PrefillShape {
  int group, gh, parts, units, tpt, slot_rows;
  long long tiles, entries, slots;       // at most; (slots: of all units)
};

// False for sizes that no call takes.  The list has room for every piece of
// `tiles` tiles: in pieces of more than W / (k CTAs), k <= kMostRounds, with W
// the key tiles of all units, they have less than k CTAs / units pieces beside
// the first of each, and less than twice that in tiles that are cut; behind the
// last whole round less than CTAs / units + 1 tiles have kMostTail at most.
bool prefill_shape(int B, int H, int N, int h_kv, bool packed, int num_sms, PrefillShape* s) {
  if (B < 1 || H < 1 || N < 1 || h_kv < 1 || H % h_kv || N >= kMaxPositions) return false;
  s->group = H / h_kv;
  s->parts = (s->group + BM - 1) / BM;
  s->gh = (s->group + s->parts - 1) / s->parts;
  s->units = h_kv * s->parts;
  s->tpt = BM / s->gh;
  s->slot_rows = s->gh * (N < s->tpt ? N : s->tpt);
  s->tiles = packed ? N / s->tpt + static_cast<long long>(B)
                    : static_cast<long long>(B) * ((N + s->tpt - 1) / s->tpt);
  const long long cut = 2ll * kMostRounds * num_sms / s->units + kMostTail + 1;
  s->entries = s->tiles + cut;
  s->slots = cut * s->units;
  return s->entries * s->units < INT_MAX - 4096 && static_cast<long long>(B) * H < INT_MAX &&
         (packed || static_cast<long long>(B) * N < INT_MAX);
}

namespace {

struct Layout {
  size_t rows, entries, joins, o_part, lse_part, total;
};

Layout layout_of(const PrefillShape& s, int B, int d) {
  Layout l;
  l.rows = 256;
  l.entries = l.rows + up256((static_cast<size_t>(B) + 1) * sizeof(int));
  l.joins = l.entries + up256(static_cast<size_t>(s.entries) * sizeof(Entry));
  l.o_part = l.joins + up256(static_cast<size_t>(s.slots / s.units) * sizeof(JoinEntry));
  const size_t rows = static_cast<size_t>(s.slots) * s.slot_rows;
  l.lse_part = l.o_part + up256(rows * d * sizeof(float));
  l.total = l.lse_part + up256(rows * sizeof(float));
  return l;
}

template <int D, bool GROUPED>
cudaError_t launch_main(PrefillParams& p, int max_smem, cudaStream_t stream) {
  using C = Cfg<D, GROUPED>;
  const size_t smem = smem_request(sizeof(Smem<C>), max_smem);
  cudaError_t e = cudaFuncSetAttribute(prefill_kernel<D, GROUPED>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e == cudaSuccess) e = launch_dependent(plan_kernel, dim3(1), kPlanThreads, stream, p);
  if (e == cudaSuccess) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.grid);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, prefill_kernel<D, GROUPED>, p);
  }
  if (e == cudaSuccess) e = launch_dependent(join_kernel<D>, dim3(p.grid * 8), 128, stream, p);
  return e;
}

template <int D>
cudaError_t launch(PrefillParams& p, int max_smem, cudaStream_t stream) {
  if constexpr (D > 64)
    if (p.groups) return launch_main<D, true>(p, max_smem, stream);
  return launch_main<D, false>(p, max_smem, stream);
}

}  // namespace
}  // namespace fa

extern "C" {

size_t fa_prefill_paged_workspace_bytes(int B, int H, int N, int h_kv, int d, int packed) {
  int sms = 0;
  if (fa::device_facts(&sms) != FA_OK) sms = 152;
  fa::PrefillShape s;
  if ((d != 64 && d != 128 && d != 256) || !fa::prefill_shape(B, H, N, h_kv, packed != 0, sms, &s))
    return 0;
  return fa::layout_of(s, B, d).total;
}

fa_status_t fa_prefill_paged(const fa_strided_t* q, const fa_paged_kv_t* cache, int layer,
                             const int* block_table, int max_pages, const int* start,
                             const int* kv_len, const int* offsets, const fa_strided_t* o,
                             float* lse, int B, int H, int N, float scale, int causal,
                             int window_left, int window_right, int sinks, void* workspace,
                             size_t workspace_bytes, void* stream) {
  if (!lse || !start || !kv_len || layer < 0) return FA_ERR_INVALID_ARG;
  if (!fa::aligned_to(lse, 4) || !fa::aligned_to(start, 4) || !fa::aligned_to(kv_len, 4) ||
      !fa::aligned_to(offsets, 4) || !workspace || !fa::aligned_to(workspace, 256))
    return FA_ERR_INVALID_ARG;
  fa::PagePool pool;
  const fa_status_t ps = fa::resolve_pool(cache, layer, &pool);
  if (ps != FA_OK) return ps;
  if (!fa::table_ok(block_table, max_pages, pool.page_size)) return FA_ERR_INVALID_ARG;
  if (window_left < -1 || window_right < -1 || sinks < 0) return FA_ERR_INVALID_ARG;
  if (!(scale > 0.f && scale <= 3.402823466e38f)) return FA_ERR_INVALID_ARG;
  int sms = 0, max_smem = 0;
  int* status = nullptr;
  fa::PrefillShape s;
  // (the sizes are checked before the device is asked)
  if (!fa::prefill_shape(B, H, N, pool.h_kv, offsets != nullptr, 1, &s)) return FA_ERR_INVALID_ARG;
  const int batch = offsets ? 1 : B;
  if (!fa::strided_ok(q, batch, H, N, pool.d, true) ||
      !fa::strided_ok(o, batch, H, N, pool.d, true) || o->p == q->p)
    return FA_ERR_INVALID_ARG;
  const fa_status_t ds = fa::device_facts(&sms, &max_smem, &status);
  if (ds != FA_OK) return ds;
  if (!fa::prefill_shape(B, H, N, pool.h_kv, offsets != nullptr, sms, &s))
    return FA_ERR_INVALID_ARG;
  const fa::Layout l = fa::layout_of(s, B, pool.d);
  if (workspace_bytes < l.total) return FA_ERR_INVALID_ARG;
  fa::PrefillParams p = {};
  const long long qd[3] = {H, N, batch};
  const long long qs[3] = {q->head_stride, q->token_stride, q->batch_stride};
  const int qb[3] = {s.gh, s.tpt, 1};
  // Pages of whole eights whose step is whole eights too may come in one box
  // each, with the keys' eights outermost: a copy holds its warp for some 56
  // cycles, and tiles of few slots a page take many.  Pages past 32 slots take few
  // enough in boxes of 64 columns, which land sooner (whole / by 64 columns, N =
  // 8192: d = 128, H = 32, h_kv = 8, pages of 8 808 / 1287 us, 16 712 / 846, 32 719
  // / 713, 64 733 / 718; d = 256, H = 16, h_kv = 4, 8 767 / 1409, 16 695 / 957, 32
  // 677 / 769; 2048 tokens after 8000, 32 254 / 277, 40 271 / 265, 56 290 / 271).
  const long long eight = 8 * pool.token_stride;
  const long long step = pool.num_pages > 1 ? pool.page_stride / eight : pool.page_size / 8;
  const long long last = (pool.num_pages - 1) * step + pool.page_size / 8;   // eights in all
  const bool grouped = pool.d > 64 && pool.page_size % 8 == 0 && pool.page_size <= 32 &&
                       (pool.num_pages == 1 || pool.page_stride % eight == 0) && last < INT_MAX;
  const int slots = pool.page_size < fa::BN ? pool.page_size : fa::BN;
  if (grouped) {
    const long long gd[4] = {8, pool.d / 64, last, pool.h_kv};
    const long long gs[4] = {pool.token_stride, 64, eight, pool.head_stride};
    const int gb[4] = {8, pool.d / 64, slots / 8, 1};
    if (!fa::make_map_5d(&p.tk, pool.k, gd, gs, gb) || !fa::make_map_5d(&p.tv, pool.v, gd, gs, gb))
      return FA_ERR_CUDA;
  } else {
    const long long kd[3] = {pool.page_size, pool.h_kv, pool.num_pages};
    const long long ks[3] = {pool.token_stride, pool.head_stride, pool.page_stride};
    const int kb[3] = {slots, 1, 1};
    if (!fa::make_map_4d(&p.tk, pool.k, pool.d, kd, ks, kb) ||
        !fa::make_map_4d(&p.tv, pool.v, pool.d, kd, ks, kb))
      return FA_ERR_CUDA;
  }
  if (!fa::make_map_4d(&p.tq, q->p, pool.d, qd, qs, qb)) return FA_ERR_CUDA;
  p.groups = grouped ? static_cast<int>(step) : 0;
  p.eights = static_cast<int>(grouped ? last : 0);
  p.o = static_cast<__nv_bfloat16*>(o->p);
  p.ob = batch > 1 ? o->batch_stride : 0;
  p.oh = H > 1 ? o->head_stride : 0;
  p.ot = N > 1 ? o->token_stride : 0;
  p.lse = lse;
  p.table = block_table;
  p.start = start;
  p.kv_len = kv_len;
  p.offsets = offsets;
  p.B = B;
  p.H = H;
  p.N = N;
  p.h_kv = pool.h_kv;
  p.group = s.group;
  p.gh = s.gh;
  p.parts = s.parts;
  p.units = s.units;
  p.tpt = s.tpt;
  p.fd_units = fa::FastDiv::of(s.units);
  p.fd_grid = fa::FastDiv::of(sms);
  p.fd_parts = fa::FastDiv::of(s.parts);
  p.fd_gh = fa::FastDiv::of(s.gh);
  p.fd_tn = fa::FastDiv::of((N + s.tpt - 1) / s.tpt);
  p.max_pages = max_pages;
  p.num_pages = pool.num_pages;
  p.page_size = pool.page_size;
  p.ppt = pool.page_size <= fa::BN ? fa::BN / pool.page_size : 0;
  p.tpp = (pool.page_size + fa::BN - 1) / fa::BN;
  p.kt = p.ppt ? p.ppt * pool.page_size : fa::BN;
  p.fd_kt = fa::FastDiv::of(p.kt);
  p.fd_ps = fa::FastDiv::of(pool.page_size);
  p.fd_tpp = fa::FastDiv::of(p.tpp);
  p.causal = causal != 0;
  // (an unbounded side reaches past every position)
  p.wl = window_left < 0 ? INT_MAX : window_left;
  p.wr = p.causal ? 0 : (window_right < 0 ? INT_MAX : window_right);
  p.sinks = sinks;
  p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  p.status = status;
  char* ws = static_cast<char*>(workspace);
  p.counters = reinterpret_cast<fa::Counters*>(ws);
  p.row_tiles = reinterpret_cast<int*>(ws + l.rows);
  p.entries = reinterpret_cast<fa::Entry*>(ws + l.entries);
  p.joins = reinterpret_cast<fa::JoinEntry*>(ws + l.joins);
  p.o_part = reinterpret_cast<float*>(ws + l.o_part);
  p.lse_part = reinterpret_cast<float*>(ws + l.lse_part);
  p.cap_tiles = static_cast<int>(s.tiles);
  p.cap_slots = static_cast<int>(s.slots / s.units);
  p.slot_rows = s.slot_rows;
  p.grid = sms;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = pool.d == 64    ? fa::launch<64>(p, max_smem, st)
                        : pool.d == 128 ? fa::launch<128>(p, max_smem, st)
                                        : fa::launch<256>(p, max_smem, st);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
