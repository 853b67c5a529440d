// [B, H, N, d] tensors seen through strides, rows of tokens that lie one
// after the other, and rotary angles: what the rotary and the chunk kernels
// share.
#pragma once
#include <algorithm>
#include <cstdint>

#include <cuda_bf16.h>

#include "fa_internal.h"
#include "fa_paged.cuh"

namespace fa {

// device_facts (fa_internal.h) with the largest dynamic shared memory of a block
// and the device's status word.
fa_status_t device_facts(int* num_sms, int* max_smem, int** status);

// bf16 [n[2], n[1], n[0], d] through strides s (values, multiples of 8) as a
// 4-D tensor (d, n[0], n[1], n[2]): a box of 64 columns and box[i] of each
// axis, 128-byte swizzle, zeros outside.
bool make_map_4d(CUtensorMap* m, const void* base, int d, const long long* n, const long long* s,
                 const int* box);
// The same of 64 columns (64, n[0], .., n[3]).
bool make_map_5d(CUtensorMap* m, const void* base, const long long* n, const long long* s,
                 const int* box);

// A public fa_strided_t over [B, H, N, d]: 16-byte aligned, strides that are
// multiples of 8 and reach less than 2^60 values; written tensors also have no
// two values in one place.  The stride of an axis of one does not count.
inline bool strided_ok(const fa_strided_t* t, int B, int H, int N, int d, bool written) {
  if (!t || !t->p || !aligned_to(t->p, 16)) return false;
  struct Axis {
    long long stride, n;
  };
  Axis a[3] = {{t->batch_stride, B}, {t->head_stride, H}, {t->token_stride, N}};
  std::sort(a, a + 3, [](const Axis& x, const Axis& y) { return x.stride < y.stride; });
  long long extent = d;
  for (const Axis& x : a) {
    if (x.n <= 1) continue;
    if (x.stride < 0 || (x.stride & 7) || (written && x.stride < extent) ||
        x.stride > ((1ll << 60) - extent) / (x.n - 1))
      return false;
    extent += x.stride * (x.n - 1);
  }
  return true;
}

// The tokens of row b: [begin, end) of the token axis (offsets: the rows lie
// one after the other in N tokens; a border outside them counts as the
// nearest), or all N of batch entry b.
__device__ __forceinline__ void row_tokens(const int* offsets, int b, int N, int& begin, int& end) {
  begin = 0;
  end = N;
  if (offsets) {
    begin = min(max(offsets[b], 0), N);
    end = min(max(offsets[b + 1], begin), N);
  }
}

// The angle of `pos` at `turns` 2^-64 turns a position, as sine and cosine
// times `magnitude`.  The product modulo 2^64 is the angle's exact fraction of
// a turn at any position (a product in fp32 would lose it from some thousands
// on).  Its upper 32 bits (what is cut off is below 2^-32 turns) become a float
// of half turns in [-1, 1], rounded by at most 2^-24 of itself and 2^-25 in
// all: together below 2^-26 + 2^-32 turns, 2^-23.3 radians.
__device__ __forceinline__ void rotary_angle(unsigned long long turns, long long pos, float magnitude,
                                             float& s, float& c) {
  const unsigned long long a = turns * static_cast<unsigned long long>(pos);
  sincospif(static_cast<float>(static_cast<int>(a >> 32)) * 4.656612873077393e-10f, &s, &c);
  s *= magnitude;
  c *= magnitude;
}

}  // namespace fa
