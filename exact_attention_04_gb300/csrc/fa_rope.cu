// Rotary positions: pair i of a head's first 2 P values, (a, b), becomes
//   (a cos t - b sin t, a sin t + b cos t) m,   t = position w_i,
// the other values stay.  A pair is (x_i, x_{i+P}), or (x_2i, x_2i+1) when
// interleaved.  The gradient is the turn by -t.
//
// Bound by memory: each value is read and written once (268 MB in 41.3 us, 0.96
// of the copy bandwidth; 906 MB of new tokens into pages in 135.3, 0.98).  A lane
// owns 16 bytes of a head, a warp 32 / (d / 8) tokens, and sine and cosine of a
// lane's pairs serve all the heads that the warp walks, kUnroll heads at a time,
// the next ones' loads in flight meanwhile.  The other half of a pair comes from
// the lane that owns it (shuffles; where P is no multiple of 8, through shared
// memory), so the turn may be in place.
#include <climits>
#include <cmath>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_internal.h"
#include "fa_paged.cuh"
#include "fa_strided.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

using namespace ptx;

// Warps of a block, and heads whose loads are in flight together: small blocks
// even the last wave out (H = 16 + 16, N = 8192, B = 2, d = 128: 4 / 8 / 16 warps
// 41.3 / 45.9 / 78.0 us; 2 / 4 / 8 heads 44.8 / 41.3 / 44.9; 36864 new tokens, 32 + 8
// + 8 heads, into pages 141 / 137 / 139).
constexpr int kWarps = 4;
constexpr int kUnroll = 4;

// How the pairs lie: halves whose length is a multiple of 8, neighbours, or
// halves of any length.
enum Pairs { kHalves, kNeighbours, kAnyHalves };

// One tensor of the walk: `heads` heads from x to y.
struct RotTensor {
  const __nv_bfloat16* x;
  __nv_bfloat16* y;
  long long xb, xh, xt, yb, yh, yt;   // strides of batch, head, token (values)
  int heads;
};

struct RotParams {
  RotTensor t[2];              // queries, keys (paged: y unused)
  const unsigned long long* turns;
  float magnitude;
  int half;                    // pairs P
  int back;                    // turn by -t
  int copy;                    // the values behind the pairs are copied
  const int* start;            // position of a row's first token, or nullptr (0)
  const int* pos;              // position of every token, or nullptr
  int N;                       // tokens of a row, or (offsets) of all rows
  int tokens;                  // B N, or N
  FastDiv fd_n;
  int chunk;                   // heads of a block's walk
  int heads;                   // of the whole walk
  // paged
  PagePool pool;
  const __nv_bfloat16* v;
  long long vb, vh, vt;
  const int* table;
  const int* kv_len;
  const int* offsets;
  int B, max_pages;
};

// The row of packed token i, the last one that begins at or before it, by a
// whole warp: 32 borders a look, so that few of the memory's latencies follow
// one another.  (Offsets that do not rise give some row.)
__device__ __forceinline__ int row_of(const int* offsets, int B, int i) {
  const int lane = threadIdx.x & 31;
  int lo = 0, len = B;
  while (len > 1) {
    const int step = (len + 31) / 32, at = lane * step;
    const bool here = at < len && offsets[lo + at] <= i;
    const int n = max(__popc(__ballot_sync(0xffffffffu, here)), 1) - 1;
    lo += n * step;
    len = min(step, len - n * step);
  }
  return lo;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// A lane's 8 values turned.  c, s: of its values (halves: s with the sign of
// the value's side) or of its four pairs (neighbours).
template <int D, int PAIRS>
__device__ __forceinline__ uint4 turn(uint4 x, const float* c, const float* s, int shift, int half,
                                      uint32_t* row, int ch) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t r[4];
  if constexpr (PAIRS == kNeighbours) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = bf16_lo(w[i]), b = bf16_hi(w[i]);
      r[i] = pack_bf16x2(fmaf(a, c[i], -(b * s[i])), fmaf(a, s[i], b * c[i]));
    }
  } else {
    float other[8];
    if constexpr (PAIRS == kHalves) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t o = __shfl_sync(0xffffffffu, w[i], (threadIdx.x & 31) + shift);
        other[2 * i] = bf16_lo(o);
        other[2 * i + 1] = bf16_hi(o);
      }
    } else {
      __syncwarp();
      *reinterpret_cast<uint4*>(row + ch * 4) = x;
      __syncwarp();
      const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(row);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = ch * 8 + i;
        const int o = e < half ? e + half : (e < 2 * half ? e - half : e);
        other[i] = __bfloat162float(v[o]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r[i] = pack_bf16x2(fmaf(bf16_lo(w[i]), c[2 * i], other[2 * i] * s[2 * i]),
                         fmaf(bf16_hi(w[i]), c[2 * i + 1], other[2 * i + 1] * s[2 * i + 1]));
  }
  if constexpr (PAIRS != kHalves) {
    // values behind the pairs stay: as numbers turned by nothing, an infinity
    // would become 0 inf, and in its neighbour too
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (4 * ch + i >= half) r[i] = w[i];
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

template <int D, int PAIRS, bool PAGED>
__global__ void __launch_bounds__(kWarps * 32)
    rope_kernel(const __grid_constant__ RotParams p) {
  constexpr int LPR = D / 8;             // lanes of a head
  constexpr int TPW = 32 / LPR;          // tokens of a warp
  constexpr int NC = PAIRS == kNeighbours ? 4 : 8;
  __shared__ uint4 rows[PAIRS == kAnyHalves ? kWarps * 32 : 1];
  // (paged: the rows' lengths may be what the kernel before writes)
  if constexpr (PAGED) grid_dependency_wait();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int ch = lane % LPR;             // the lane's 8 values of a head
  uint32_t* row_sm = reinterpret_cast<uint32_t*>(rows + warp * 32 + lane / LPR * LPR);
  const long long tok = (static_cast<long long>(blockIdx.x) * kWarps + warp) * TPW + lane / LPR;
  bool there = tok < p.tokens;
  int b = 0, n = there ? static_cast<int>(tok) : 0, at = 0, limit = 0;
  const bool packed = PAGED && p.offsets;
  if (!packed) {
    b = p.fd_n.div(n);
    n -= b * p.N;
    at = n;
  }
  // The lane's values of the heads of the walk: queries, keys, (paged) values.
  // The first heads are asked for before the token's row and position are
  // known, and each group before the one in hand is turned.
  const int bt = packed ? 0 : b;               // the batch entry of the token's address
  const __nv_bfloat16* x[3] = {p.t[0].x + bt * p.t[0].xb + n * p.t[0].xt + 8 * ch,
                               p.t[1].x + bt * p.t[1].xb + n * p.t[1].xt + 8 * ch,
                               p.v + bt * p.vb + n * p.vt + 8 * ch};
  const int hq = p.t[0].heads, hk = p.t[1].heads;
  const int h0 = blockIdx.y * p.chunk, h1 = min(h0 + p.chunk, p.heads);
  const auto load = [&](int h, uint4* v) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = h + u;
      v[u] = make_uint4(0, 0, 0, 0);
      if (there && i < h1) {
        const __nv_bfloat16* from = i < hq ? x[0] + i * p.t[0].xh
                                    : !PAGED || i < hq + hk
                                        ? x[1] + (i - hq) * p.t[1].xh
                                        : x[2] + (i - hq - hk) * p.vh;
        v[u] = *reinterpret_cast<const uint4*>(from);
      }
    }
  };
  uint4 v[kUnroll];
  load(h0, v);
  unsigned long long turns[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int e = NC * ch + i;           // a pair (neighbours) or a value
    const int pair = PAIRS != kNeighbours && e >= p.half ? e - p.half : e;
    turns[i] = pair < p.half ? p.turns[pair] : 0;
  }
  if (packed) {
    // the warp's first token's row; the other tokens' rows follow it
    const int first = static_cast<int>(
        min((static_cast<long long>(blockIdx.x) * kWarps + warp) * TPW, p.tokens - 1ll));
    b = row_of(p.offsets, p.B, first);
    // (tokens before the first row and behind the last are no row's)
    there = there && n >= p.offsets[0] && n < p.offsets[p.B];
    if (there) {
      while (b + 1 < p.B && p.offsets[b + 1] <= n) ++b;
      at = n - p.offsets[b];
    }
  }
  long long where = 0;                   // the position
  if (there) {
    where = p.pos ? p.pos[static_cast<long long>(b) * p.N + n]
                  : (p.start ? static_cast<long long>(p.start[b]) : 0) + at;
    if constexpr (PAGED) limit = p.kv_len[b];
  }
  // where a token's keys and values go
  long long slot = -1;
  if constexpr (PAGED) {
    if (there && where >= 0 && where < limit) {
      const int j = static_cast<int>(where) / p.pool.page_size;
      if (j < p.max_pages) {
        const int page = p.table[static_cast<long long>(b) * p.max_pages + j];
        if (page >= 0 && page < p.pool.num_pages)
          slot = page * p.pool.page_stride +
                 (static_cast<int>(where) - j * p.pool.page_size) * p.pool.token_stride + 8 * ch;
      }
    }
  }
  float c[NC], s[NC];
  const bool turned = 8 * ch < 2 * p.half;
  // halves: the other value of a pair lies `shift` lanes on
  const int shift =
      PAIRS != kHalves || !turned ? 0 : (8 * ch < p.half ? p.half / 8 : -(p.half / 8));
  if constexpr (PAIRS == kHalves) {
    // both lanes of a pair have the same eight angles: each takes four
    const int mine = shift < 0 ? 4 : 0;
    float sc[8];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      rotary_angle(shift < 0 ? turns[i + 4] : turns[i], where, p.magnitude, sc[2 * i],
                   sc[2 * i + 1]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float so = __shfl_sync(0xffffffffu, sc[2 * i], lane + shift);
      const float co = __shfl_sync(0xffffffffu, sc[2 * i + 1], lane + shift);
      s[i] = mine ? so : sc[2 * i];
      c[i] = mine ? co : sc[2 * i + 1];
      s[i + 4] = mine ? sc[2 * i] : so;
      c[i + 4] = mine ? sc[2 * i + 1] : co;
    }
    // the first half's values take the other's times -sin, back the other way
    const bool minus = (p.back != 0) == (shift < 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = minus ? -s[i] : s[i];
  } else {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int e = NC * ch + i;
      const bool second = PAIRS != kNeighbours && e >= p.half;
      c[i] = 1.f;
      s[i] = 0.f;
      if ((second ? e - p.half : e) < p.half) {
        rotary_angle(turns[i], where, p.magnitude, s[i], c[i]);
        if ((p.back != 0) != (PAIRS != kNeighbours && !second)) s[i] = -s[i];
      }
    }
  }
  const bool write = there && (turned || p.copy);
  __nv_bfloat16* const yq = p.t[0].y + bt * p.t[0].yb + n * p.t[0].yt + 8 * ch;
  __nv_bfloat16* const yk =
      PAGED ? p.pool.k + slot : p.t[1].y + bt * p.t[1].yb + n * p.t[1].yt + 8 * ch;
  const long long ykh = PAGED ? p.pool.head_stride : p.t[1].yh;
#pragma unroll 1
  for (int h = h0; h < h1; h += kUnroll) {
    uint4 next[kUnroll];
    if (h + kUnroll < h1) load(h + kUnroll, next);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = h + u;
      const uint4 r = turn<D, PAIRS>(v[u], c, s, shift, p.half, row_sm, ch);
      if (i < h1) {
        if (i < hq) {
          if (write) *reinterpret_cast<uint4*>(yq + i * p.t[0].yh) = turned ? r : v[u];
        } else if (!PAGED || i < hq + hk) {
          if (PAGED ? slot >= 0 : write)
            *reinterpret_cast<uint4*>(yk + (i - hq) * ykh) = turned ? r : v[u];
        } else if (slot >= 0) {
          *reinterpret_cast<uint4*>(p.pool.v + slot + (i - hq - hk) * p.pool.head_stride) = v[u];
        }
      }
      v[u] = next[u];
    }
  }
}

template <bool PAGED>
cudaError_t launch_rope(RotParams& p, int d, bool interleaved, int num_sms, cudaStream_t stream) {
  // Few tokens: the heads are shared out too (down to kUnroll a warp), until
  // there are 32 blocks an SM (16 / 32: gradients of 32 + 8 heads, N = 16384, B = 2
  // 100.3 / 99.2 us); each part computes its tokens' angles again.
  const long long groups = (p.tokens + static_cast<long long>(kWarps) * (256 / d) - 1) /
                           (kWarps * (256 / d));
  const long long most = (p.heads + kUnroll - 1) / kUnroll;
  long long parts = (num_sms * 32ll + groups - 1) / groups;
  parts = std::min(std::max(parts, 1ll), std::min(most, 65535ll));
  p.chunk = static_cast<int>(((p.heads + parts - 1) / parts + kUnroll - 1) / kUnroll * kUnroll);
  const dim3 grid(static_cast<unsigned>(groups),
                  static_cast<unsigned>((p.heads + p.chunk - 1) / p.chunk));
  const int pairs = interleaved ? kNeighbours : (p.half % 8 ? kAnyHalves : kHalves);
  const auto go = [&](auto kernel) {
    return PAGED ? launch_dependent(kernel, grid, kWarps * 32, stream, p)
                 : (kernel<<<grid, kWarps * 32, 0, stream>>>(p), cudaGetLastError());
  };
  const auto of_d = [&](auto dim) {
    constexpr int D = decltype(dim)::value;
    return pairs == kHalves       ? go(rope_kernel<D, kHalves, PAGED>)
           : pairs == kNeighbours ? go(rope_kernel<D, kNeighbours, PAGED>)
                                  : go(rope_kernel<D, kAnyHalves, PAGED>);
  };
  return d == 64    ? of_d(std::integral_constant<int, 64>())
         : d == 128 ? of_d(std::integral_constant<int, 128>())
                    : of_d(std::integral_constant<int, 256>());
}

fa_status_t rotary_ok(const fa_rotary_t* r, int d, RotParams* p) {
  if (d != 64 && d != 128 && d != 256) return FA_ERR_UNSUPPORTED;
  if (!r || !r->turns || !aligned_to(r->turns, 8) || r->dims < 2 || r->dims > d || r->dims % 2 ||
      !std::isfinite(r->magnitude))
    return FA_ERR_INVALID_ARG;
  p->turns = r->turns;
  p->magnitude = r->magnitude;
  p->half = r->dims / 2;
  return FA_OK;
}

RotTensor rot_tensor(const fa_strided_t* x, const fa_strided_t* y, int heads) {
  return RotTensor{static_cast<const __nv_bfloat16*>(x->p),
                   static_cast<__nv_bfloat16*>(y ? y->p : nullptr),
                   x->batch_stride, x->head_stride, x->token_stride,
                   y ? y->batch_stride : 0, y ? y->head_stride : 0, y ? y->token_stride : 0, heads};
}

// Whether b is a itself, seen alike (turned in place).
bool same(const fa_strided_t* a, const fa_strided_t* b, int B, int H, int N) {
  return a->p == b->p && (B == 1 || a->batch_stride == b->batch_stride) &&
         (H == 1 || a->head_stride == b->head_stride) &&
         (N == 1 || a->token_stride == b->token_stride);
}

// An output at its input's address, but seen through other strides.
bool crossed(const fa_strided_t* a, const fa_strided_t* b, int B, int H, int N) {
  return a->p == b->p && !same(a, b, B, H, N);
}

}  // namespace
}  // namespace fa

extern "C" {

fa_status_t fa_rotate(const fa_strided_t* q, const fa_strided_t* q_out, int H,
                      const fa_strided_t* k, const fa_strided_t* k_out, int h_kv, int B, int N,
                      int d, const int* start, const int* pos, const fa_rotary_t* rotary, int back,
                      void* stream) {
  fa::RotParams p = {};
  const fa_status_t rs = fa::rotary_ok(rotary, d, &p);
  if (rs != FA_OK) return rs;
  if (B < 1 || N < 1 || H < 1 || h_kv < 0 || static_cast<long long>(H) + h_kv > 65535 ||
      static_cast<long long>(B) * N >= INT_MAX)
    return FA_ERR_INVALID_ARG;
  if (!fa::strided_ok(q, B, H, N, d, false) || !fa::strided_ok(q_out, B, H, N, d, true) ||
      fa::crossed(q, q_out, B, H, N))
    return FA_ERR_INVALID_ARG;
  if (h_kv > 0 && (!fa::strided_ok(k, B, h_kv, N, d, false) ||
                   !fa::strided_ok(k_out, B, h_kv, N, d, true) || q_out->p == k_out->p ||
                   q_out->p == k->p || k_out->p == q->p || fa::crossed(k, k_out, B, h_kv, N)))
    return FA_ERR_INVALID_ARG;
  if (!fa::aligned_to(start, 4) || !fa::aligned_to(pos, 4) || (start && pos))
    return FA_ERR_INVALID_ARG;
  int sms = 0;
  const fa_status_t ds = fa::device_facts(&sms);
  if (ds != FA_OK) return ds;
  p.t[0] = fa::rot_tensor(q, q_out, H);
  if (h_kv > 0) p.t[1] = fa::rot_tensor(k, k_out, h_kv);
  p.copy = !(fa::same(q, q_out, B, H, N) && (h_kv == 0 || fa::same(k, k_out, B, h_kv, N)));
  p.back = back != 0;
  p.start = start;
  p.pos = pos;
  p.N = N;
  p.tokens = B * N;
  p.fd_n = fa::FastDiv::of(N);
  p.heads = H + h_kv;
  return fa::launch_rope<false>(p, d, rotary->interleaved != 0, sms,
                                static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

fa_status_t fa_paged_append_rotated(const fa_strided_t* q, const fa_strided_t* q_out, int H,
                                    const fa_strided_t* k_new, const fa_strided_t* v_new,
                                    const fa_paged_kv_t* cache, int layer, const int* block_table,
                                    int max_pages, const int* start, const int* kv_len,
                                    const int* offsets, int B, int N, const fa_rotary_t* rotary,
                                    void* stream) {
  if (!start || !kv_len || layer < 0 || !fa::aligned_to(start, 4) || !fa::aligned_to(kv_len, 4) ||
      !fa::aligned_to(offsets, 4))
    return FA_ERR_INVALID_ARG;
  fa::RotParams p = {};
  const fa_status_t ps = fa::resolve_pool(cache, layer, &p.pool);
  if (ps != FA_OK) return ps;
  const int d = p.pool.d, h_kv = p.pool.h_kv;
  const fa_status_t rs = fa::rotary_ok(rotary, d, &p);
  if (rs != FA_OK) return rs;
  if (!fa::table_ok(block_table, max_pages, p.pool.page_size)) return FA_ERR_INVALID_ARG;
  const int rows = offsets ? 1 : B;         // batch entries of the tensors
  if (B < 1 || B >= INT_MAX || N < 1 || N >= fa::kMaxPositions || H < 0 ||
      H + 2ll * h_kv > 65535 || static_cast<long long>(rows) * N >= INT_MAX)
    return FA_ERR_INVALID_ARG;
  if (!fa::strided_ok(k_new, rows, h_kv, N, d, false) ||
      !fa::strided_ok(v_new, rows, h_kv, N, d, false))
    return FA_ERR_INVALID_ARG;
  if (H > 0 && (!fa::strided_ok(q, rows, H, N, d, false) ||
                !fa::strided_ok(q_out, rows, H, N, d, true) || q_out->p == k_new->p ||
                q_out->p == v_new->p || fa::crossed(q, q_out, rows, H, N)))
    return FA_ERR_INVALID_ARG;
  int sms = 0;
  const fa_status_t ds = fa::device_facts(&sms);
  if (ds != FA_OK) return ds;
  if (H > 0) p.t[0] = fa::rot_tensor(q, q_out, H);
  p.t[1] = fa::rot_tensor(k_new, nullptr, h_kv);
  p.v = static_cast<const __nv_bfloat16*>(v_new->p);
  p.vb = v_new->batch_stride;
  p.vh = v_new->head_stride;
  p.vt = v_new->token_stride;
  p.copy = H > 0 && !fa::same(q, q_out, rows, H, N);
  p.start = start;
  p.kv_len = kv_len;
  p.offsets = offsets;
  p.table = block_table;
  p.max_pages = max_pages;
  p.B = B;
  p.N = N;
  p.tokens = rows * N;
  p.fd_n = fa::FastDiv::of(N);
  p.heads = H + 2 * h_kv;
  return fa::launch_rope<true>(p, d, rotary->interleaved != 0, sms,
                               static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

}  // extern "C"
