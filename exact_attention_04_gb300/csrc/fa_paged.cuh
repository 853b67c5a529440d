// What the paged-cache kernels share: the pool's layout as the kernels see it
// and the host checks of the public structure.
#pragma once
#include <algorithm>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_internal.h"

namespace fa {

// One layer of the pool, or (layers > 1) all of them.
struct PagePool {
  __nv_bfloat16* k;
  __nv_bfloat16* v;
  long long layer_stride, page_stride, head_stride, token_stride;   // elements
  int layers, num_pages, page_size, h_kv, d;
};

constexpr long long kMaxPositions = 1ll << 30;   // max_pages * page_size stays below

inline bool aligned_to(const void* p, unsigned n) {
  return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

// Whether no two values of the pool share a place: taken from the smallest
// stride up, each axis steps past everything inside it, and the whole stays
// below 2^60 values.
inline bool axes_apart(const fa_paged_kv_t& c) {
  struct Axis {
    long long stride, n;
  };
  Axis a[4] = {{c.layer_stride, c.num_layers},
               {c.page_stride, c.num_pages},
               {c.head_stride, c.h_kv},
               {c.token_stride, c.page_size}};
  std::sort(a, a + 4, [](const Axis& x, const Axis& y) { return x.stride < y.stride; });
  long long extent = c.d;
  for (const Axis& x : a) {
    if (x.n == 1) continue;
    if (x.stride < extent || x.stride > ((1ll << 60) - extent) / (x.n - 1)) return false;
    extent += x.stride * (x.n - 1);
  }
  return true;
}

// The structure's own rules (see fa.h); *out is layer `layer`, or the whole
// pool when layer < 0.
inline fa_status_t resolve_pool(const fa_paged_kv_t* c, int layer, PagePool* out) {
  if (!c || !c->k || !c->v || !aligned_to(c->k, 16) || !aligned_to(c->v, 16))
    return FA_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128 && c->d != 256) return FA_ERR_UNSUPPORTED;
  if (c->num_layers < 1 || c->num_pages < 1 || c->page_size < 1 || c->h_kv < 1 ||
      c->page_size >= kMaxPositions || layer >= c->num_layers ||
      static_cast<long long>(c->num_layers) * c->h_kv > 0x7fffffffll)
    return FA_ERR_INVALID_ARG;
  const long long st[4] = {c->layer_stride, c->page_stride, c->head_stride, c->token_stride};
  for (long long s : st)
    if (s < 0 || (s & 7)) return FA_ERR_INVALID_ARG;
  if (!axes_apart(*c)) return FA_ERR_INVALID_ARG;
  const long long off = layer > 0 ? layer * c->layer_stride : 0;
  *out = PagePool{static_cast<__nv_bfloat16*>(c->k) + off, static_cast<__nv_bfloat16*>(c->v) + off,
                  c->layer_stride, c->page_stride, c->head_stride, c->token_stride,
                  layer < 0 ? c->num_layers : 1, c->num_pages, c->page_size, c->h_kv, c->d};
  return FA_OK;
}

// All threads of a cluster meet; what they wrote before is seen after.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

// The shared address a of this CTA in CTA `rank` of its cluster.
__device__ __forceinline__ uint32_t in_cta(uint32_t a, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}

// Launches a kernel that waits for the one before it in its own code
// (griddepcontrol.wait), so that its launch overlaps that one's run.
template <class... Args, class... Given>
cudaError_t launch_dependent(void (*kernel)(Args...), dim3 grid, unsigned threads,
                             cudaStream_t stream, Given... given) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args>(given)...);
}

// A block table over the pool: its width and address.
inline bool table_ok(const int* table, int max_pages, int page_size) {
  return table && aligned_to(table, 4) && max_pages >= 1 &&
         static_cast<long long>(max_pages) * page_size < kMaxPositions;
}

}  // namespace fa
