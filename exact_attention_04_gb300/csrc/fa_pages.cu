// The metadata of a paged cache and the copies it asks for: reserving, forking
// and freeing, trimming and compacting pages.
//
// Each call first settles the integers (which page goes where), then moves
// what has to move.
//
// The integers: one cluster of 8 CTAs of 1024 threads.  Ranks (the k-th free
// page, the k-th request) are prefix sums: a thread counts a contiguous
// run of pages or rows, the block scans the counts, and the 8 block totals
// are read from the other CTAs' shared memory.  The cluster's barriers order
// the phases; a grid of separate launches would pay a launch for each.
// Reference counts change by integer atomics, whose order does not matter.
// The bound is latency: a chain of two to five dependent passes over arrays
// that fit the L2.
//
// The copies: a grid of warps, a task of 16 slots of one (page, layer, head)
// each, K and V, every load of a task in flight before its first store.  The
// bound is HBM: each moved byte is read once and written once (compacting
// 0.85 GB: 265 us with its metadata, 6.4 TB/s).
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

constexpr int kCluster = 8;
constexpr int kMetaThreads = 1024;
constexpr int kMeta = kCluster * kMetaThreads;

__device__ __forceinline__ int remote_load(const int* p, int cta) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];"
               : "=r"(v)
               : "r"(in_cta(smem_u32(p), cta))
               : "memory");
  return v;
}

// Sums over the cluster.  add() leaves this block's total of v in the slot
// and returns the sum over the block's earlier threads; after a cluster_sync,
// total() is the whole sum and before() that of the earlier blocks.
struct ClusterScan {
  int warp_sum[kMetaThreads / 32];
  int block_total;

  __device__ int add(int v) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    if (warp == 0) {
      const int own = warp_sum[lane];
      int w = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
      }
      warp_sum[lane] = w - own;
      if (lane == 31) block_total = w;
    }
    __syncthreads();
    return warp_sum[warp] + x - v;
  }
  __device__ void sums(int& before, int& total) const {
    before = total = 0;
#pragma unroll
    for (int c = 0; c < kCluster; ++c) {
      const int t = remote_load(&block_total, c);
      if (c < static_cast<int>(blockIdx.x)) before += t;
      total += t;
    }
  }
};

// This thread's contiguous run of n items.
__device__ __forceinline__ void run_of(int n, int& lo, int& hi) {
  const long long g = static_cast<long long>(blockIdx.x) * kMetaThreads + threadIdx.x;
  const long long per = (static_cast<long long>(n) + kMeta - 1) / kMeta;
  lo = static_cast<int>(g * per < n ? g * per : n);
  hi = static_cast<int>((g + 1) * per < n ? (g + 1) * per : n);
}

__device__ __forceinline__ int clamp_len(int len, long long cap) {
  return len < 0 ? 0 : (len > cap ? static_cast<int>(cap) : len);
}

__device__ __forceinline__ int pages_of(int len, int page_size) {
  return len / page_size + (len % page_size != 0);
}

// ------------------------------------------------------------------ reserve

struct ReserveParams {
  int* table;
  int max_pages, page_size, num_pages, rows;
  const int* kv_len;
  const int* n_new;
  const int* ref;
  int* kv_len_out;
  int* ref_out;
  int* info;
  int* off;         // workspace [rows]: requests of the earlier rows
  int* fresh;       // workspace [num_pages]: the free pages in order
};

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kMetaThreads, 1)
    pages_reserve_kernel(const __grid_constant__ ReserveParams p) {
  __shared__ ClusterScan asked, free_pages;
  launch_dependents();
  const long long cap = static_cast<long long>(p.max_pages) * p.page_size;
  auto want_of = [&](int r, int& have) {
    have = clamp_len(p.kv_len[r], cap);
    const int n = p.n_new[r];
    const long long w = static_cast<long long>(have) + (n > 0 ? n : 0);
    return static_cast<int>(w < cap ? w : cap);
  };
  int r_lo, r_hi, p_lo, p_hi;
  run_of(p.rows, r_lo, r_hi);
  run_of(p.num_pages, p_lo, p_hi);
  int n = 0;
  for (int r = r_lo; r < r_hi; ++r) {
    int have;
    const int want = want_of(r, have);
    n += pages_of(want, p.page_size) - pages_of(have, p.page_size);
  }
  const int my_rows = asked.add(n);
  n = 0;
  for (int i = p_lo; i < p_hi; ++i) n += p.ref[i] == 0;
  const int my_pages = free_pages.add(n);
  cluster_sync();
  int before, requests, free_before, free_total;
  asked.sums(before, requests);
  free_pages.sums(free_before, free_total);
  const int served = requests < free_total ? requests : free_total;
  int at = before + my_rows;
  for (int r = r_lo; r < r_hi; ++r) {
    int have;
    const int want = want_of(r, have);
    p.off[r] = at;
    at += pages_of(want, p.page_size) - pages_of(have, p.page_size);
  }
  at = free_before + my_pages;
  for (int i = p_lo; i < p_hi; ++i) {
    const int v = p.ref[i];
    if (v == 0) {
      if (at < served) p.fresh[at] = i;
      p.ref_out[i] = at < served ? 1 : 0;
      ++at;
    } else {
      p.ref_out[i] = v;
    }
  }
  cluster_sync();
  const int lane = threadIdx.x % 32;
  for (int r = (blockIdx.x * kMetaThreads + threadIdx.x) / 32; r < p.rows; r += kMeta / 32) {
    int have;
    const int want = want_of(r, have);
    const int a = pages_of(have, p.page_size), b = pages_of(want, p.page_size);
    const int off = p.off[r];
    __syncwarp();
    for (int j = a + lane; j < b; j += 32) {
      const int k = off + (j - a);
      p.table[static_cast<size_t>(r) * p.max_pages + j] = k < served ? p.fresh[k] : -1;
    }
    if (lane == 0) {
      const int got = served - off < 0 ? 0 : (served - off < b - a ? served - off : b - a);
      const long long room = static_cast<long long>(a + got) * p.page_size;
      p.kv_len_out[r] = static_cast<int>(want < room ? want : room);
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    p.info[0] = free_total - served;
    p.info[1] = requests - served;
  }
}

// ------------------------------------------------------------------ copies

// Slots slot0 .. slot0 + 15 (those below `slots`) of one (layer, head) of
// page src, K and V, to each of the n pages dst[0 .. n).
template <int D>
__device__ __forceinline__ void copy_task(const PagePool& pool, int src, const int* dst, int n,
                                          int slots, int layer, int head, int slot0) {
  constexpr int CH = D / 8;                  // 16-byte vectors of a row
  constexpr int N = 16 * CH / 32;            // of a lane, K and V each
  const int lane = threadIdx.x % 32;
  const long long base = layer * pool.layer_stride + head * pool.head_stride;
  const long long s = base + src * pool.page_stride;
  uint4 a[N], b[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = i * 32 + lane, slot = slot0 + e / CH;
    if (slot < slots) {
      const long long o = s + slot * pool.token_stride + e % CH * 8;
      a[i] = *reinterpret_cast<const uint4*>(pool.k + o);
      b[i] = *reinterpret_cast<const uint4*>(pool.v + o);
    }
  }
  for (int c = 0; c < n; ++c) {
    const long long d = base + dst[c] * pool.page_stride;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = i * 32 + lane, slot = slot0 + e / CH;
      if (slot < slots) {
        const long long o = d + slot * pool.token_stride + e % CH * 8;
        *reinterpret_cast<uint4*>(pool.k + o) = a[i];
        *reinterpret_cast<uint4*>(pool.v + o) = b[i];
      }
    }
  }
}

constexpr int kCopyThreads = 256;

// All pairs' tasks over the grid's warps.  run(i, src, slots) says what pair
// i copies and returns for how many pairs from i on it does (their pages are
// dst[i ..]), 0 where an earlier pair does pair i's as well.
template <int D, class Run>
__device__ __forceinline__ void copy_pairs(const PagePool& pool, const int* dst, int pairs,
                                           Run run) {
  const int blocks = (pool.page_size + 15) / 16;
  const long long inner = static_cast<long long>(pool.layers) * pool.h_kv * blocks;
  const long long tasks = inner * pairs;
  const long long warps = static_cast<long long>(gridDim.x) * (kCopyThreads / 32);
  for (long long t = (static_cast<long long>(blockIdx.x) * kCopyThreads + threadIdx.x) / 32;
       t < tasks; t += warps) {
    const int i = static_cast<int>(t / inner);
    const long long rem = t - i * inner;
    const int lh = static_cast<int>(rem / blocks);
    const int slot0 = static_cast<int>(rem - static_cast<long long>(lh) * blocks) * 16;
    const int layer = lh / pool.h_kv;
    int src, slots;
    const int n = run(i, src, slots);
    if (n > 0 && slot0 < slots)
      copy_task<D>(pool, src, dst + i, n, slots, layer, lh - layer * pool.h_kv, slot0);
  }
}

// ------------------------------------------------------------------ fork

struct ForkParams {
  PagePool pool;
  const int* table;
  int max_pages, rows, new_rows;
  const int* kv_len;
  const int* ref;
  const int* parent;
  int* table_out;
  int* kv_len_out;
  int* ref_out;
  int* info;
  int* first;       // workspace [rows]: the first row that continues each
  int* count;       // workspace [rows]: how many continue it
  int* rank;        // workspace [new_rows]: place among the requests, or -1
  int2* ask;        // workspace [new_rows]: each request's source page and filled slots
  int* fresh;       // workspace [num_pages]
  int* served;      // workspace [1]
};

// What row r of the new table continues: the parent's length (0: nothing).
__device__ __forceinline__ int parent_of(const ForkParams& p, int r, int& len) {
  const int par = __ldg(p.parent + r);
  len = 0;
  if (par < 0 || par >= p.rows) return -1;
  len = clamp_len(__ldg(p.kv_len + par), static_cast<long long>(p.max_pages) * p.pool.page_size);
  return par;
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kMetaThreads, 1)
    pages_fork_kernel(const __grid_constant__ ForkParams p) {
  __shared__ ClusterScan asked, free_pages;
  launch_dependents();
  const int ps = p.pool.page_size, num_pages = p.pool.num_pages;
  const int gid = blockIdx.x * kMetaThreads + threadIdx.x;
  for (int r = gid; r < p.rows; r += kMeta) {
    p.first[r] = INT_MAX;
    p.count[r] = 0;
  }
  for (int i = gid; i < num_pages; i += kMeta) p.ref_out[i] = p.ref[i];
  cluster_sync();
  for (int r = gid; r < p.new_rows; r += kMeta) {
    int len;
    const int par = parent_of(p, r, len);
    if (par >= 0) {
      atomicMin(p.first + par, r);
      atomicAdd(p.count + par, 1);
    }
  }
  cluster_sync();
  // an old row's entries lose one reference and gain one for each row that
  // continues it (the partly filled page: for the first of them)
  const int lane = threadIdx.x % 32;
  for (int r = gid / 32; r < p.rows; r += kMeta / 32) {
    const int n = __ldcg(p.count + r);
    if (n == 1) continue;
    const int len = clamp_len(__ldg(p.kv_len + r), static_cast<long long>(p.max_pages) * ps);
    const int full = len / ps, np = pages_of(len, ps);
    for (int j = lane; j < np; j += 32) {
      const int page = __ldg(p.table + static_cast<size_t>(r) * p.max_pages + j);
      const int delta = j < full ? n - 1 : (n > 0 ? 0 : -1);
      if (page >= 0 && page < num_pages && delta != 0) atomicAdd(p.ref_out + page, delta);
    }
  }
  // requests: the further rows of a parent with a partly filled page
  int r_lo, r_hi;
  run_of(p.new_rows, r_lo, r_hi);
  auto asks = [&](int r, int2& what) {
    int len;
    const int par = parent_of(p, r, len);
    if (par < 0 || len % ps == 0 || __ldcg(p.first + par) == r) return false;
    what.x = __ldg(p.table + static_cast<size_t>(par) * p.max_pages + len / ps);
    what.y = len % ps;
    return what.x >= 0 && what.x < num_pages;
  };
  int n = 0;
  int2 what;
  for (int r = r_lo; r < r_hi; ++r) n += asks(r, what);
  const int my_rows = asked.add(n);
  cluster_sync();                           // and every reference has changed
  int p_lo, p_hi;
  run_of(num_pages, p_lo, p_hi);
  n = 0;
  for (int i = p_lo; i < p_hi; ++i) n += __ldcg(p.ref_out + i) == 0;
  const int my_pages = free_pages.add(n);
  cluster_sync();
  int before, requests, free_before, free_total;
  asked.sums(before, requests);
  free_pages.sums(free_before, free_total);
  const int served = requests < free_total ? requests : free_total;
  int at = before + my_rows;
  for (int r = r_lo; r < r_hi; ++r) {
    const bool a = asks(r, what);
    p.rank[r] = a ? at : -1;
    if (a) p.ask[at++] = what;
  }
  at = free_before + my_pages;
  for (int i = p_lo; i < p_hi && at < served; ++i)
    if (__ldcg(p.ref_out + i) == 0) {
      p.fresh[at++] = i;
      p.ref_out[i] = 1;
    }
  if (gid == 0) {
    *p.served = served;
    p.info[0] = free_total - served;
    p.info[1] = requests - served;
  }
  cluster_sync();                           // no block leaves while its totals are read
}

// The new table, the new lengths, and the copies of partly filled pages.
template <int D>
__global__ void __launch_bounds__(kCopyThreads)
    pages_fork_copy_kernel(const __grid_constant__ ForkParams p) {
  grid_dependency_wait();
  const int ps = p.pool.page_size;
  const int served = *p.served;
  // Rows that continue one parent are often neighbours: one read of its page
  // then serves up to kRun of them (seven copies of 32 pages over 8 layers: 105 us
  // against 117 to 152 with a read each).
  constexpr int kRun = 8;
  copy_pairs<D>(p.pool, p.fresh, served, [&](int i, int& src, int& slots) {
    const int2 what = p.ask[i];
    src = what.x;
    slots = what.y;
    const auto same = [&](int k) {
      const int2 x = p.ask[k];
      return x.x == what.x && x.y == what.y;
    };
    if (i % kRun && same(i - 1)) return 0;
    int n = 1;
    while ((i + n) % kRun && i + n < served && same(i + n)) ++n;
    return n;
  });
  const long long n = static_cast<long long>(p.new_rows) * p.max_pages;
  for (long long e = static_cast<long long>(blockIdx.x) * kCopyThreads + threadIdx.x; e < n;
       e += static_cast<long long>(gridDim.x) * kCopyThreads) {
    const int r = static_cast<int>(e / p.max_pages);
    const int j = static_cast<int>(e - static_cast<long long>(r) * p.max_pages);
    int len;
    const int par = parent_of(p, r, len);
    const int rank = p.rank[r], full = len / ps;
    int page = -1;
    if (j < pages_of(len, ps)) {
      page = __ldg(p.table + static_cast<size_t>(par) * p.max_pages + j);
      if (page < 0 || page >= p.pool.num_pages) page = -1;
      if (j == full && rank >= 0) page = rank < served ? p.fresh[rank] : -1;
    }
    p.table_out[e] = page;
    if (j == 0) p.kv_len_out[r] = rank >= served ? full * ps : len;
  }
}

// ------------------------------------------------------------------ trim

struct TrimParams {
  const int* table;
  int max_pages, page_size, num_pages, rows;
  const int* kv_len;
  int wl, sinks;
  int* table_out;
  int* ref_out;
};

// Table entry e: out of the table and the reference counts, or kept.
__device__ __forceinline__ void trim_entry(const TrimParams& p, long long e, long long cap) {
  const int r = static_cast<int>(e / p.max_pages);
  const int j = static_cast<int>(e - static_cast<long long>(r) * p.max_pages);
  const int len = clamp_len(__ldg(p.kv_len + r), cap);
  const long long lo = static_cast<long long>(j) * p.page_size;
  const bool drop = lo >= p.sinks && lo + p.page_size <= static_cast<long long>(len) - p.wl;
  const int page = p.table[e];
  p.table_out[e] = drop ? -1 : page;
  if (drop && page >= 0 && page < p.num_pages) atomicSub(p.ref_out + page, 1);
}

// Both steps in one cluster, where they are small (see fa_pages_trim).
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kMetaThreads, 1)
    pages_trim_small_kernel(const __grid_constant__ TrimParams p, const int* ref) {
  const int gid = blockIdx.x * kMetaThreads + threadIdx.x;
  for (int i = gid; i < p.num_pages; i += kMeta) p.ref_out[i] = ref[i];
  cluster_sync();
  const long long n = static_cast<long long>(p.rows) * p.max_pages;
  const long long cap = static_cast<long long>(p.max_pages) * p.page_size;
  for (long long e = gid; e < n; e += kMeta) trim_entry(p, e, cap);
}

__global__ void __launch_bounds__(256) pages_ref_copy_kernel(const int* ref, int* ref_out, int n) {
  launch_dependents();
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i < n) ref_out[i] = ref[i];
}

__global__ void __launch_bounds__(256) pages_trim_kernel(const __grid_constant__ TrimParams p) {
  grid_dependency_wait();
  const long long n = static_cast<long long>(p.rows) * p.max_pages;
  const long long cap = static_cast<long long>(p.max_pages) * p.page_size;
  for (long long e = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; e < n;
       e += static_cast<long long>(gridDim.x) * 256)
    trim_entry(p, e, cap);
}

// ------------------------------------------------------------------ compact

struct CompactParams {
  PagePool pool;
  const int* table;
  int max_pages, rows;
  const int* ref;
  int* table_out;
  int* ref_out;
  int* info;
  int* to;          // workspace [num_pages]: where each page goes
  int* hole;        // workspace [num_pages]: free pages before n
  int* mover;       // workspace [num_pages]: pages in use at n or later
  int* moved;       // workspace [1]
};

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kMetaThreads, 1)
    pages_compact_kernel(const __grid_constant__ CompactParams p) {
  __shared__ ClusterScan live, low;
  launch_dependents();
  const int num_pages = p.pool.num_pages;
  int lo, hi;
  run_of(num_pages, lo, hi);
  int n = 0;
  for (int i = lo; i < hi; ++i) n += p.ref[i] > 0;
  const int mine = live.add(n);
  cluster_sync();
  int before, total;
  live.sums(before, total);
  n = 0;
  for (int i = lo; i < hi && i < total; ++i) n += p.ref[i] > 0;
  low.add(n);
  cluster_sync();
  int skip, kept;                           // pages in use before `total` stay
  low.sums(skip, kept);
  const int moves = total - kept;
  int at = before + mine;                   // pages in use before i
  for (int i = lo; i < hi; ++i) {
    const int v = p.ref[i];
    const bool used = v > 0;
    if (used && i >= total) {
      p.mover[at - kept] = i;
    } else {
      p.to[i] = i;
      if (!used && i < total) p.hole[i - at] = i;
      if (p.ref_out != p.ref) p.ref_out[i] = v;
    }
    at += used;
  }
  cluster_sync();
  for (int k = blockIdx.x * kMetaThreads + threadIdx.x; k < moves; k += kMeta) {
    const int h = __ldcg(p.hole + k), m = __ldcg(p.mover + k);
    p.to[m] = h;
    p.ref_out[h] = p.ref[m];
    p.ref_out[m] = 0;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *p.moved = moves;
    p.info[0] = total;
    p.info[1] = moves;
  }
}

template <int D>
__global__ void __launch_bounds__(kCopyThreads)
    pages_compact_copy_kernel(const __grid_constant__ CompactParams p) {
  grid_dependency_wait();
  copy_pairs<D>(p.pool, p.hole, *p.moved, [&](int i, int& src, int& slots) {
    src = p.mover[i];
    slots = p.pool.page_size;
    return 1;
  });
  const long long n = static_cast<long long>(p.rows) * p.max_pages;
  for (long long e = static_cast<long long>(blockIdx.x) * kCopyThreads + threadIdx.x; e < n;
       e += static_cast<long long>(gridDim.x) * kCopyThreads) {
    const int page = p.table[e];
    p.table_out[e] = page >= 0 && page < p.pool.num_pages ? p.to[page] : -1;
  }
}

// ------------------------------------------------------------------ launches

// CTAs of a copy kernel: one a task of 8 warps and one for 256 table entries,
// at most 8 an SM.
unsigned copy_grid(const PagePool& pool, long long pairs, long long entries, int num_sms) {
  const long long blocks = (pool.page_size + 15) / 16;
  const long long tasks = pairs * pool.layers * pool.h_kv;      // below 2^31 times 2^31
  const long long cap = 8ll * num_sms;
  if (tasks >= cap * 8) return static_cast<unsigned>(cap);
  const long long want = (tasks * blocks + 7) / 8 + (entries + 255) / 256;
  return static_cast<unsigned>(want < 1 ? 1 : (want < cap ? want : cap));
}

size_t ints_bytes(long long n) { return (static_cast<size_t>(n) * sizeof(int) + 255) / 256 * 256; }

// The workspace in regions of 256 bytes' alignment.
struct Regions {
  char* at;
  int* take(long long n) {
    int* r = reinterpret_cast<int*>(at);
    at += ints_bytes(n);
    return r;
  }
};

bool ints_ok(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!p || !aligned_to(p, 4)) return false;
  return true;
}

constexpr int kMaxRows = 1 << 24;

}  // namespace
}  // namespace fa

extern "C" {

size_t fa_pages_workspace_bytes(int num_pages, int rows) {
  if (num_pages < 1 || rows < 1 || rows > fa::kMaxRows) return 0;
  return 3 * fa::ints_bytes(num_pages) + 3 * fa::ints_bytes(rows) + fa::ints_bytes(2ll * rows) +
         fa::ints_bytes(1);
}

fa_status_t fa_pages_reserve(int* block_table, int max_pages, int page_size, const int* kv_len,
                             const int* n_new, const int* ref, int num_pages, int rows,
                             int* kv_len_out, int* ref_out, int* info, void* workspace,
                             size_t workspace_bytes, void* stream) {
  if (!fa::ints_ok({kv_len, n_new, ref, kv_len_out, ref_out, info}) || !workspace ||
      !fa::aligned_to(workspace, 256) || page_size < 1 ||
      !fa::table_ok(block_table, max_pages, page_size))
    return FA_ERR_INVALID_ARG;
  if (num_pages < 1 || rows < 1 || rows > fa::kMaxRows ||
      static_cast<long long>(rows) * max_pages >= INT_MAX)
    return FA_ERR_INVALID_ARG;
  if (workspace_bytes < fa_pages_workspace_bytes(num_pages, rows)) return FA_ERR_INVALID_ARG;
  const fa_status_t ds = fa::device_facts(nullptr);
  if (ds != FA_OK) return ds;
  fa::Regions w{static_cast<char*>(workspace)};
  int* off = w.take(rows);
  int* fresh = w.take(num_pages);
  const fa::ReserveParams p{block_table, max_pages, page_size, num_pages, rows, kv_len, n_new,
                            ref, kv_len_out, ref_out, info, off, fresh};
  fa::pages_reserve_kernel<<<fa::kCluster, fa::kMetaThreads, 0,
                             static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status_t fa_pages_fork(const fa_paged_kv_t* cache, const int* block_table, int max_pages,
                          const int* kv_len, const int* ref, int rows, const int* parent,
                          int new_rows, int* table_out, int* kv_len_out, int* ref_out, int* info,
                          void* workspace, size_t workspace_bytes, void* stream) {
  if (!fa::ints_ok({kv_len, ref, parent, table_out, kv_len_out, ref_out, info}) || !workspace ||
      !fa::aligned_to(workspace, 256))
    return FA_ERR_INVALID_ARG;
  fa::ForkParams p;
  const fa_status_t ps = fa::resolve_pool(cache, -1, &p.pool);
  if (ps != FA_OK) return ps;
  if (!fa::table_ok(block_table, max_pages, p.pool.page_size)) return FA_ERR_INVALID_ARG;
  if (rows < 1 || rows > fa::kMaxRows || new_rows < 1 || new_rows > fa::kMaxRows ||
      table_out == block_table || kv_len_out == kv_len || ref_out == ref)
    return FA_ERR_INVALID_ARG;
  const int most = rows > new_rows ? rows : new_rows;
  if (workspace_bytes < fa_pages_workspace_bytes(p.pool.num_pages, most)) return FA_ERR_INVALID_ARG;
  int sms = 0;
  const fa_status_t ds = fa::device_facts(&sms);
  if (ds != FA_OK) return ds;
  p.table = block_table;
  p.max_pages = max_pages;
  p.rows = rows;
  p.new_rows = new_rows;
  p.kv_len = kv_len;
  p.ref = ref;
  p.parent = parent;
  p.table_out = table_out;
  p.kv_len_out = kv_len_out;
  p.ref_out = ref_out;
  p.info = info;
  fa::Regions w{static_cast<char*>(workspace)};
  p.first = w.take(rows);
  p.count = w.take(rows);
  p.rank = w.take(new_rows);
  p.ask = reinterpret_cast<int2*>(w.take(2ll * new_rows));
  p.fresh = w.take(p.pool.num_pages);
  p.served = w.take(1);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  fa::pages_fork_kernel<<<fa::kCluster, fa::kMetaThreads, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return FA_ERR_CUDA;
  const unsigned grid =
      fa::copy_grid(p.pool, new_rows, static_cast<long long>(new_rows) * max_pages, sms);
  switch (p.pool.d) {
    case 64:
      e = fa::launch_dependent(fa::pages_fork_copy_kernel<64>, grid, fa::kCopyThreads, s, p);
      break;
    case 128:
      e = fa::launch_dependent(fa::pages_fork_copy_kernel<128>, grid, fa::kCopyThreads, s, p);
      break;
    default: e = fa::launch_dependent(fa::pages_fork_copy_kernel<256>, grid, fa::kCopyThreads, s, p);
  }
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status_t fa_pages_trim(const int* block_table, int max_pages, int page_size,
                          const int* kv_len, const int* ref, int num_pages, int rows,
                          int window_left, int sinks, int* table_out, int* ref_out,
                          void* stream) {
  if (!fa::ints_ok({kv_len, ref, table_out, ref_out}) || page_size < 1 ||
      !fa::table_ok(block_table, max_pages, page_size))
    return FA_ERR_INVALID_ARG;
  if (num_pages < 1 || rows < 1 || rows > fa::kMaxRows || window_left < 0 || sinks < 0)
    return FA_ERR_INVALID_ARG;
  int sms = 0;
  const fa_status_t ds = fa::device_facts(&sms);
  if (ds != FA_OK) return ds;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const fa::TrimParams p{block_table, max_pages, page_size, num_pages, rows, kv_len,
                         window_left, sinks, table_out, ref_out};
  const long long n = static_cast<long long>(rows) * max_pages;
  const long long want = (n + 255) / 256, cap = 8ll * sms;
  const unsigned grid = static_cast<unsigned>(want < cap ? want : cap);
  // one launch where both arrays are small (4 x 100 entries: 2.2 us against
  // 2.4 in two, and a launch less for the host; 32 x 256: 3.0 / 2.4)
  if (n + num_pages <= 4096 && ref_out != ref) {
    fa::pages_trim_small_kernel<<<fa::kCluster, fa::kMetaThreads, 0, s>>>(p, ref);
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
  }
  if (ref_out == ref) {
    fa::pages_trim_kernel<<<grid, 256, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
  }
  fa::pages_ref_copy_kernel<<<static_cast<unsigned>((num_pages + 255ll) / 256), 256, 0, s>>>(
      ref, ref_out, num_pages);
  if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
  return fa::launch_dependent(fa::pages_trim_kernel, grid, 256, s, p) == cudaSuccess ? FA_OK
                                                                                     : FA_ERR_CUDA;
}

fa_status_t fa_pages_compact(const fa_paged_kv_t* cache, const int* block_table, int max_pages,
                             const int* ref, int rows, int* table_out, int* ref_out, int* info,
                             void* workspace, size_t workspace_bytes, void* stream) {
  if (!fa::ints_ok({ref, table_out, ref_out, info}) || !workspace ||
      !fa::aligned_to(workspace, 256))
    return FA_ERR_INVALID_ARG;
  fa::CompactParams p;
  const fa_status_t ps = fa::resolve_pool(cache, -1, &p.pool);
  if (ps != FA_OK) return ps;
  if (!fa::table_ok(block_table, max_pages, p.pool.page_size)) return FA_ERR_INVALID_ARG;
  if (rows < 1 || rows > fa::kMaxRows) return FA_ERR_INVALID_ARG;
  if (workspace_bytes < fa_pages_workspace_bytes(p.pool.num_pages, rows)) return FA_ERR_INVALID_ARG;
  int sms = 0;
  const fa_status_t ds = fa::device_facts(&sms);
  if (ds != FA_OK) return ds;
  p.table = block_table;
  p.max_pages = max_pages;
  p.rows = rows;
  p.ref = ref;
  p.table_out = table_out;
  p.ref_out = ref_out;
  p.info = info;
  fa::Regions w{static_cast<char*>(workspace)};
  p.to = w.take(p.pool.num_pages);
  p.hole = w.take(p.pool.num_pages);
  p.mover = w.take(p.pool.num_pages);
  p.moved = w.take(1);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  fa::pages_compact_kernel<<<fa::kCluster, fa::kMetaThreads, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return FA_ERR_CUDA;
  const unsigned grid = fa::copy_grid(p.pool, p.pool.num_pages / 2,
                                      static_cast<long long>(rows) * max_pages, sms);
  switch (p.pool.d) {
    case 64:
      e = fa::launch_dependent(fa::pages_compact_copy_kernel<64>, grid, fa::kCopyThreads, s, p);
      break;
    case 128:
      e = fa::launch_dependent(fa::pages_compact_copy_kernel<128>, grid, fa::kCopyThreads, s, p);
      break;
    default:
      e = fa::launch_dependent(fa::pages_compact_copy_kernel<256>, grid, fa::kCopyThreads, s, p);
  }
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
