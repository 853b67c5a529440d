// Pieces of the backward main kernel that keeps dQ transposed (fa_bwd_dt.cu):
// tile sizes, warp roles, the persistent schedule over key blocks, the
// visible query range of a key block, and failure reporting.
#pragma once
#include <cuda_runtime.h>

#include "fa_internal.h"
#include "fa_order.cuh"
#include "fa_window.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

using namespace ptx;

constexpr int BQ = 64;             // queries per step
constexpr int BK = 128;            // keys per work item
constexpr int DH = 128;            // head-dimension columns of dK, dV, dQ per work item
constexpr int KCH = 128 * 128;     // 128 rows x 128 bytes
constexpr int QCH = 64 * 128;      // 64 rows x 128 bytes
constexpr int kRowWarps = 8;       // two per sub-partition, one per 32-query half
constexpr int kDrainWarp0 = 3 + kRowWarps;   // four dQ drain warps
constexpr int kReduceWarp = kDrainWarp0 + 4; // d = 256: issues the dQ bulk reduce-adds
constexpr int kThreads = 32 * (kDrainWarp0 + 4);   // 15 warps (16 with the reduce warp)
// With 15 warps one sub-partition holds four: 128 registers a thread at most
// (the compiler is told 512 threads so that it plans for that).
constexpr int kRegThreads = 512;

enum Site {
  kSiteProdKV = 64, kSiteProdQ, kSiteMmaKV, kSiteMmaQ, kSiteMmaP, kSiteMmaDs, kSiteMmaDq,
  kSiteMmaAcc, kSiteRowS, kSiteRowDp, kSiteRowDsFree, kSiteRowAcc, kSiteDrainDq, kSiteDtDrain,
  kSiteStageFree, kSiteStageFull, kSiteRowV, kSiteMmaV, kSiteProdDo, kSiteMmaDo
};

__device__ __forceinline__ void record_failure(int* status, volatile int* abort, int site) {
  atomicCAS(status, 0, status_code(site));
  *abort = 1;
}

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  bool ok = mbar_wait(bar, parity, abort, kWaitTimeoutNs);
  return __all_sync(0xffffffffu, ok);
}

// Column of the packed bf16 P^T / dS^T for K-step kk (16 queries) within its
// 64-column buffer: queries 32h .. 32h+31 sit in columns 32h .. 32h+15.
__device__ __forceinline__ constexpr uint32_t pcol(int kk) {
  return static_cast<uint32_t>((kk >> 1) * 32 + (kk & 1) * 8);
}

// Issuer warps wait as a whole warp (mbar_wait_warp) and report a failure
// from lane 0.
__device__ __forceinline__ void issuer_fail(int* status, volatile int* abort, int lane, int site) {
  if (lane == 0) record_failure(status, abort, site);
}

// Units are (K/V head kvbh, key-block pair or key block, half); a work item
// (one key block) steps over the query heads of kvbh's group and, for each,
// the query blocks its keys are visible to.  Plain causal: key block n meets
// query blocks from its diagonal on, so blocks p and T-1-p are paired,
// longest first.  The halves of one key block are adjacent units so they run
// at the same time and share K, V, Q, dO in L2.
// This CTA's place in the schedule: its round-robin units (and the key
// blocks of a causal pair), then its row of the tail table.
struct DtIter {
  int u, kt, k;
};

// A block mask without a host copy (order != nullptr): the items (K/V head,
// key block; the halves of d adjacent) go in the cost-sorted turning deal of
// fa_order.cuh instead, from the order planned into the workspace.
struct DtSched {
  int T, P, per_bh, units, causal, nsplit;   // units: the round-robin units
  int BH;
  const uint32_t* order;                     // the cost-sorted order, or nullptr
  __device__ DtSched(int BH_, int N, int causal_, int nsplit_, int tail_heads,
                     const uint32_t* order_)
      : causal(causal_), nsplit(nsplit_), BH(BH_), order(order_) {
    T = (N + BK - 1) / BK;
    P = (T + 1) / 2;
    per_bh = causal ? P : T;
    units = (BH - tail_heads) * per_bh * nsplit;
  }
  __device__ void decode(int u, int& bh, int& pp, int& h) const {
    bh = u / (per_bh * nsplit);
    const int rem = u % (per_bh * nsplit);
    pp = rem / nsplit;
    h = rem % nsplit;
  }
  __device__ int nitems(int pp) const {
    if (!causal) return 1;
    return (pp == T - 1 - pp) ? 1 : 2;
  }
  __device__ int block(int pp, int k) const {
    if (!causal) return pp;
    return (k == 0) ? pp : (T - 1 - pp);
  }
  // The next work item of this CTA (K/V head, half of d, key block); false
  // when it has none left.  Every role walks the same sequence.
  __device__ bool next(const TailTable& tail, DtIter& it, int& kvbh, int& h, int& n) const {
    if (order) {   // round it.k of the cost-sorted deal
      const long long k = order_deal(it.k, gridDim.x, blockIdx.x);
      if (k >= static_cast<long long>(BH) * T * nsplit) return false;
      ++it.k;
      h = static_cast<int>(k % nsplit);
      order_item(order, BH, k / nsplit, kvbh, n);
      return true;
    }
    while (it.u < units) {
      int pp;
      decode(it.u, kvbh, pp, h);
      if (it.kt < nitems(pp)) {
        n = block(pp, it.kt);
        ++it.kt;
        return true;
      }
      it.u += gridDim.x;
      it.kt = 0;
    }
    if (tail.heads == 0 || blockIdx.x >= kTailCtas || it.k >= kTailItems) return false;
    const int e = tail.item[blockIdx.x][it.k];
    if (e < 0) return false;
    ++it.k;
    kvbh = tail_head(e);
    h = tail_half(e);
    n = tail_block(e);
    return true;
  }
};

// kv_len of K/V head kvbh's batch entry.
__device__ __forceinline__ int dt_len(const BwdParams& p, int kvbh) {
  int len = p.N;
  if (p.kv_len) {
    len = __ldg(p.kv_len + kvbh / p.H_kv);
    len = len < 0 ? 0 : (len > p.N ? p.N : len);
  }
  return len;
}

// Steps [i0, i1) of STEP query rows that see key block n (empty when none
// does).  With sinks, a block that holds some is seen to the last query.
template <int MK, int STEP>
__device__ __forceinline__ void step_range(const BwdParams& p, int n, int len, int& i0, int& i1) {
  int q_lo, q_hi;
  visible_queries(n * BK, BK, len, p.N, p.wl, p.wr, q_lo, q_hi);
  if (MK == kMaskSinks && n * BK < p.sinks && n * BK < len) q_hi = p.N;
  if (q_hi <= q_lo) {
    i0 = i1 = 0;
    return;
  }
  i0 = q_lo / STEP;
  i1 = (q_hi + STEP - 1) / STEP;
}

// Sinks.  The few key blocks that hold sinks are seen by every later query of
// a whole group, many times a window's worth, and whole key blocks per CTA
// leave the last round part-empty.  So of the items (K/V head, key block,
// half of d) without sinks as many as fill whole rounds go round-robin (so
// that CTAs working at the same time share Q, dO and the dQ accumulator
// through L2); the pool of the others, those with sinks and then the last
// part of a round, is laid end to end, an item taking its steps plus
// kItemCost (its start-up and epilogue, in steps), and CTA c of G takes
// [c total / G, (c + 1) total / G) of it.  A pool item within one share goes
// to dV, dK as any item; the pieces of a cut one leave fp32 rows in sk_part,
// slot 2c for the piece that starts past the item's first step (CTA c's
// first) and 2c + 1 for the one that starts at it (CTA c's last), and
// bwd_sinks_post_kernel adds them in the CTAs' order.  All of it is a
// function of the sizes and kv_len.  H = 16, h_kv = 4, N = 16384, d = 128,
// window 2047, 4 sinks: 694 us (700 when it was compared with whole items, the
// sinks' far queries as items of their own, 789, and with all items end to
// end, 1012: each CTA elsewhere in the sequence, and the dQ accumulator falls
// out of L2).
struct SkPlan {
  int whole;                    // the round-robin items are 0 .. whole - 1
  int j;                        // this CTA's first pool item
  long long p0;                 // where it starts
  long long xs, xe;             // this CTA's share of the pool
};

struct SkScratch {
  SkPlan plan;
  long long warp_sum[32];
};

// Shared memory for it, in the kernels with sinks.
struct SkNothing {};
template <int MK>
struct SkForT {
  using type = SkNothing;
};
template <>
struct SkForT<kMaskSinks> {
  using type = SkScratch;
};
template <int MK>
using SkFor = typename SkForT<MK>::type;

constexpr int kItemCost = 4;

// Sum over the block and, in `before`, over the earlier threads.
__device__ __forceinline__ long long sk_scan(long long v, long long* warp_sum, long long& before) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  long long total = 0, pre = 0;
  for (int w = 0; w < warps; ++w) {
    if (w < warp) pre += warp_sum[w];
    total += warp_sum[w];
  }
  before = pre + x - v;
  return total;
}

// Steps that item (kvbh, n) takes in all.
template <int STEP>
__device__ __forceinline__ long long sk_steps(const BwdParams& p, int kvbh, int n, int G) {
  int i0, i1;
  step_range<kMaskSinks, STEP>(p, n, dt_len(p, kvbh), i0, i1);
  return static_cast<long long>(i1 - i0) * G;
}

// The whole block; ends with a barrier.  Writes sc.plan and, for the join,
// sk_meta[c] = {the pool item that CTA c starts in, whether its share cuts
// it}.
template <int STEP>
__device__ __forceinline__ void sk_plan(const BwdParams& p, int G, SkScratch& sc) {
  const SkItems items(p);
  const int tid = threadIdx.x, threads = blockDim.x;
  const int rounds = items.plain / gridDim.x;
  const int whole = rounds * gridDim.x;
  const int pool = items.sunk + items.plain - whole;
  const int per = (pool + threads - 1) / threads;
  const int lo = min(pool, tid * per), hi = min(pool, lo + per);
  auto cost = [&](int j) {
    int kvbh, n, h;
    items.pool_item(p, j, whole, kvbh, n, h);
    return sk_steps<STEP>(p, kvbh, n, G) + kItemCost;
  };
  long long sum = 0, before;
  for (int j = lo; j < hi; ++j) sum += cost(j);
  const long long total = sk_scan(sum, sc.warp_sum, before);
  const long long ctas = min(static_cast<long long>(gridDim.x), total);   // no share is empty
  const bool idle = blockIdx.x >= ctas;
  const long long xs = idle ? 0 : total * blockIdx.x / ctas;
  const long long xe = idle ? 0 : total * (blockIdx.x + 1) / ctas;
  if (idle ? tid == 0 : xs >= before && xs < before + sum) {
    int j = lo;
    long long z = xs - before;                // how far xs lies in its item
    if (!idle)
      for (long long c = cost(j); z >= c; c = cost(++j)) z -= c;
    sc.plan = SkPlan{whole, j, idle ? 0 : xs - z, xs, xe};
    p.sk_meta[2 * blockIdx.x] = idle ? -1 : j;
    p.sk_meta[2 * blockIdx.x + 1] = !idle && z > kItemCost;
  }
  __syncthreads();
}

// The dV (0) or dK (1) rows of a piece: [128, cols] floats, cols = min(d, 128).
__device__ __forceinline__ float* sink_rows(const BwdParams& p, int slot, int cols, int which) {
  return p.sk_part + (static_cast<size_t>(slot) * 2 + which) * BK * cols;
}

// A work item as every role sees it: steps [a, b) of its nst a query head,
// head after head; none: a key block that no query sees (its gradients are
// written as zeros), or with sinks the empty end of one.
template <int MK>
struct Item {
  int kvbh, h, n, len;
  int i0, i1, nst, b;
  StepMask sk;
  static constexpr int a = 0, slot = -1;
  static constexpr bool zero = true;
  __device__ __forceinline__ bool empty() const { return b == 0; }
  __device__ __forceinline__ StepWalk walk(int bh0) const { return StepWalk(i0, i1, bh0, sk); }
};

template <>
struct Item<kMaskSinks> {
  int kvbh, h, n, len;
  int i0, i1, nst;
  int a, b;
  int slot;                     // of sk_part, or -1: dV and dK
  bool zero;                    // no query sees it, and this CTA writes the zeros
  __device__ __forceinline__ bool empty() const { return a >= b; }
  __device__ __forceinline__ StepWalk walk(int bh0) const {
    StepWalk w(i0, i1, bh0);
    if (a > 0) {
      w.bh += a / nst;
      w.i += a % nst;
    }
    return w;
  }
};

template <int MK, int STEP>
struct ItemWalk {
  const BwdParams& p;
  const TailTable& tail;
  const DtSched& sched;
  int G;                        // query heads per K/V head
  DtIter it;
  int turn;                     // sinks: how far this CTA's place in the next round is off
  const SkScratch* sc;          // it.u is the next round-robin item, then
  int j;                        // the pool's next item and where it starts
  long long p0;
  bool whole;                   // the item placed last is a round-robin one
  __device__ __forceinline__ ItemWalk(const BwdParams& p_, const TailTable& tail_,
                                      const DtSched& sched_, int G_, const SkScratch* sc_)
      : p(p_), tail(tail_), sched(sched_), G(G_), it{static_cast<int>(blockIdx.x), 0, 0},
        sc(sc_) {
    if constexpr (MK == kMaskSinks) {
      // every other round from the far end
      turn = p.sk_turn ? static_cast<int>(gridDim.x) - 1 - 2 * static_cast<int>(blockIdx.x) : 0;
      j = sc->plan.j;
      p0 = sc->plan.p0;
    }
  }
  // The next item's place, false when this CTA has none left, and what it
  // takes there.
  __device__ __forceinline__ bool place(int& kvbh, int& h, int& n) {
    if constexpr (MK == kMaskSinks) {
      const SkItems items(p);
      const int end = sc->plan.whole;
      whole = it.u < end;
      if (whole) {
        items.plain_item(p, it.u, kvbh, n, h);
        it.u += static_cast<int>(gridDim.x) + turn;
        turn = -turn;
      } else {
        if (p0 >= sc->plan.xe) return false;
        items.pool_item(p, j++, end, kvbh, n, h);
      }
      return true;
    } else {
      return sched.next(tail, it, kvbh, h, n);
    }
  }
  __device__ __forceinline__ void fill(int kvbh, int h, int n, Item<MK>& w) {
    w.kvbh = kvbh;
    w.h = h;
    w.n = n;
    if constexpr (MK == kMaskSinks) {
      w.slot = -1;
      w.len = p.kv_len ? max(0, min(p.N, __ldg(p.kv_len + p.fd_hkv.div(kvbh)))) : p.N;
      step_range<MK, STEP>(p, n, w.len, w.i0, w.i1);
      w.nst = w.i1 - w.i0;
      const long long steps = static_cast<long long>(w.nst) * G;
      w.a = 0;
      w.b = static_cast<int>(steps);
      w.zero = steps == 0;
      if (!whole) {
        const long long first = p0 + kItemCost, xs = sc->plan.xs;
        w.a = static_cast<int>(max(0ll, xs - first));
        w.b = static_cast<int>(max(0ll, min(steps, sc->plan.xe - first)));
        w.zero = steps == 0 && p0 >= xs;
        if (w.a > 0)
          w.slot = 2 * blockIdx.x;
        else if (w.b < steps)
          w.slot = 2 * blockIdx.x + 1;
        p0 = first + steps;
      }
    } else {
      w.len = dt_len(p, kvbh);
      step_range<MK, STEP>(p, n, w.len, w.i0, w.i1);
      w.sk = StepMask{MK == kMaskBlocks ? p.block_mask + n : nullptr, p.bm_t, BK / STEP};
      w.nst = count_steps(w.sk, w.i0, w.i1);
      if (w.nst == 0) w.i1 = w.i0;
      w.b = w.nst * G;
    }
  }
  __device__ __forceinline__ bool next(Item<MK>& w) {
    if (!place(w.kvbh, w.h, w.n)) return false;
    fill(w.kvbh, w.h, w.n, w);
    return true;
  }
};

// Rows [left, 128) of a tile of `chunks` 128-byte column chunks become
// zero, by a whole warp: keys past the sequence may hold anything, and their
// zero weights times NaN would be NaN.
__device__ __forceinline__ void zero_rows(uint8_t* tile, int chunks, int left, int lane) {
  for (int c = 0; c < chunks; ++c)
    for (int e = left * 8 + lane; e < BK * 8; e += 32)
      *reinterpret_cast<uint4*>(tile + c * KCH + e * 16) = make_uint4(0, 0, 0, 0);
}

}  // namespace
}  // namespace fa
