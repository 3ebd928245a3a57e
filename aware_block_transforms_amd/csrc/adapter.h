// Device helpers shared by the adapter kernels: matrix operands out of rows as
// they lie in memory, and which adapter a run of tokens belongs to.
#pragma once

#include "vec.h"

namespace wush {

// 16x16x32 product: lane 16 g + j holds row (or column) j and the eight k
// values 8 g .. 8 g + 7 of either operand; of the result it holds column j,
// rows 4 g .. 4 g + 3.
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                 0);
}

// An fp32 value as the sum of three bf16 values, exactly (8 + 8 + 8
// significant bits, truncated in turn; exact down to the subnormal range), so
// that a product with a bf16 operand rounds nowhere but in the fp32 sums.  The
// other way, one bf16 term, costs two thirds of the matrix work less and loses
// two bytes of every intermediate; these kernels wait for memory instead.  An
// infinity splits into an infinity and NaN: results it reaches are NaN.
__device__ __forceinline__ void split3(float v, uint32_t& a, uint32_t& b, uint32_t& c) {
  a = __builtin_bit_cast(uint32_t, v) & 0xffff0000u;
  const float r1 = v - __builtin_bit_cast(float, a);
  b = __builtin_bit_cast(uint32_t, r1) & 0xffff0000u;
  c = __builtin_bit_cast(uint32_t, r1 - __builtin_bit_cast(float, b));
}

__device__ __forceinline__ uint32_t top_halves(uint32_t lo, uint32_t hi) {
  return __builtin_amdgcn_perm(hi, lo, 0x07060302u);
}

// Eight fp32 k values of a lane as the three bf16 operands of split3.
__device__ __forceinline__ void split8(const float* v, u32x4 (&t)[3]) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    uint32_t a0, b0, c0, a1, b1, c1;
    split3(v[2 * p], a0, b0, c0);
    split3(v[2 * p + 1], a1, b1, c1);
    t[0][p] = top_halves(a0, a1);
    t[1][p] = top_halves(b0, b1);
    t[2][p] = top_halves(c0, c1);
  }
}

// Requests are runs of tokens: request s owns [off[s], off[s + 1]), where
// off[0] is 0 and off[nseg] is n (both are taken as such, not read).  They are
// cut into tiles of T tokens, numbered so that a workgroup finds its request
// without a table: tile j of request s has the number off[s] / T + s + j.
// These numbers rise with s and never meet, whatever the lengths, and all lie
// below n / T + nseg; the unused ones find an empty tile.
struct Tile {
  int begin, end;   // tokens, empty if begin >= end
  int adapter;      // -1: none
};

__device__ __forceinline__ int request_start(const int* __restrict__ off, int s, int nseg, int n) {
  return s <= 0 ? 0 : s >= nseg ? n : min(max(off[s], 0), n);
}

template <int T>
__device__ __forceinline__ Tile find_tile(int number, int n, int nseg, const int* __restrict__ off,
                                          const int* __restrict__ ids, int nad) {
  // every wave counts the requests whose first tile is not past `number`; the
  // count's last request is the tile's.  Of up to 64 requests the lanes hold
  // everything needed, one load after another is saved.
  const int lane = threadIdx.x & 63;
  Tile t{0, 0, -1};
  int s, first, last, a;
  if (nseg <= 64) {
    const int start = request_start(off, lane, nseg, n);
    const int id = lane < nseg ? ids[lane] : -1;
    s = __popcll(__ballot(lane < nseg && start / T + lane <= number)) - 1;
    if (s < 0) return t;
    s = __builtin_amdgcn_readfirstlane(s);
    first = __builtin_amdgcn_readlane(start, s);
    last = s + 1 < nseg ? __builtin_amdgcn_readlane(start, s + 1) : n;
    a = __builtin_amdgcn_readlane(id, s);
  } else {
    int count = 0;
    for (int b = 0; b < nseg; b += 64) {
      const int q = b + lane;
      count += __popcll(__ballot(q < nseg && request_start(off, q, nseg, n) / T + q <= number));
    }
    s = __builtin_amdgcn_readfirstlane(count - 1);
    if (s < 0) return t;
    first = request_start(off, s, nseg, n);
    last = request_start(off, s + 1, nseg, n);
    a = ids[s];
  }
  const int j = number - (first / T + s);
  // 64 bits: j runs far past the request's end on unused numbers
  const int64_t begin = first + static_cast<int64_t>(j) * T;
  if (j < 0 || begin >= last) return t;
  t.begin = static_cast<int>(begin);
  t.end = last - t.begin < T ? last : t.begin + T;
  t.adapter = a >= 0 && a < nad ? a : -1;
  return t;
}

inline int64_t tile_numbers(int n, int T, int nseg) { return static_cast<int64_t>(n / T) + nseg; }

}  // namespace wush
