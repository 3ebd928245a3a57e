// The grad kernel of the adapters: dF[a][r][c] = sum over the tokens t of
// adapter a of S[t][r] X[t][c], for (S, X, F) = (dV, X, A) and (V, dY, Bt).
//
// The sum runs over tokens, which lie along the slow axis of both operands, and
// an adapter's tokens may be spread over many requests.  A first small kernel
// lists the tokens of each adapter in order (`tokens`), and cuts each list into
// chunks; the grad kernel takes one chunk and 128 columns per workgroup.
//
// In a 16x16x32 product the eight k values of a lane are eight tokens.  A lane
// therefore loads the same eight columns of eight token rows, 16 bytes each
// (16 lanes read 256 contiguous bytes of a row), and exchanges halves between
// its own registers; no LDS and no lane exchange is needed, since which column
// a result belongs to is free to choose: operand c of lane j is column 8 j + c.
// The same holds for the rows: S is read as RT neighbouring values per lane, and
// row tile rt holds the rows RT j + rt.
//
// Chunks of one adapter are summed in order by a third kernel, so the result
// does not depend on scheduling; an adapter of one chunk is written directly.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "adapter.h"
#include "common.h"

using namespace wush;

namespace {

constexpr int kWaves = 4;
constexpr int kCols = 128;

// tokens [n]: the tokens of adapter 0, 1, ... in request order
// start [nad + 1]: where an adapter's tokens begin in that list
// chunk [nad + 1]: the number of its first chunk
// place [nseg]: where a request's tokens begin
struct Lists {
  int* tokens;
  int* start;
  int* chunk;
  int* place;
};

__device__ __forceinline__ int lane_prefix(int v) {   // inclusive
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const int o = __shfl_up(v, m, 64);
    if (lane >= m) v += o;
  }
  return v;
}

__global__ __launch_bounds__(1024) void adapter_list_kernel(int n, int nseg, const int* __restrict__ off,
                                                            const int* __restrict__ ids, int nad,
                                                            const int* __restrict__ rank, int span, Lists l) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  auto length = [&](int s, int a) {
    if (s >= nseg || ids[s] != a) return 0;
    return max(request_start(off, s + 1, nseg, n) - request_start(off, s, nseg, n), 0);
  };
  // one wave per adapter: its tokens (none where its rank is zero)
  for (int a = wave; a < nad; a += 16) {
    int sum = 0;
    if (rank[a] > 0)
      for (int b = 0; b < nseg; b += 64) sum = min(sum + length(b + lane, a), n);
    sum = __shfl(lane_prefix(sum), 63, 64);
    if (lane == 0) l.start[a] = min(sum, n);
  }
  __syncthreads();
  if (wave == 0) {
    int tokens = 0, chunks = 0;
    for (int b = 0; b < nad; b += 64) {
      const int a = b + lane;
      // capped at n, which offsets that do not rise could pass
      const int64_t past = tokens + static_cast<int64_t>(lane_prefix(a < nad ? l.start[a] : 0));
      const int to = static_cast<int>(min(past, static_cast<int64_t>(n)));
      const int before = __shfl_up(to, 1, 64), from = lane == 0 ? tokens : before;
      const int parts = (to - from + span - 1) / span, c = lane_prefix(parts);
      if (a < nad) {
        l.start[a] = from;
        l.chunk[a] = chunks + c - parts;
      }
      tokens = __shfl(to, 63, 64);
      chunks += __shfl(c, 63, 64);
    }
    if (lane == 0) {
      l.start[nad] = tokens;
      l.chunk[nad] = chunks;
    }
  }
  __syncthreads();
  for (int a = wave; a < nad; a += 16) {
    if (rank[a] <= 0) continue;
    int at = l.start[a];
    for (int b = 0; b < nseg; b += 64) {
      const int m = length(b + lane, a), p = lane_prefix(m);
      if (m > 0) l.place[b + lane] = at + p - m;
      at = min(at + __shfl(p, 63, 64), n);
    }
  }
  __syncthreads();
  for (int s = wave; s < nseg; s += 16) {
    const int a = ids[s];
    if (a < 0 || a >= nad || rank[a] <= 0) continue;
    const int first = request_start(off, s, nseg, n), m = request_start(off, s + 1, nseg, n) - first;
    if (m <= 0) continue;
    const int at = l.place[s];
    for (int i = lane; i < m; i += 64)
      if (at + i < n) l.tokens[at + i] = first + i;
  }
}

// Eight columns of eight token rows, and the matrix operands of each column.
struct act8_t {};

template <class X>
struct Rows;

template <>
struct Rows<bf16_t> {
  static constexpr int kTerms = 1;
  u32x4 v[8];
  __device__ __forceinline__ void load(int i, const void* x, const uint8_t*, int64_t row, int64_t ld, int c) {
    v[i] = *reinterpret_cast<const u32x4*>(static_cast<const bf16_t*>(x) + row * ld + c);
  }
  __device__ __forceinline__ void clear(int i) { v[i] = u32x4{0u, 0u, 0u, 0u}; }
  __device__ __forceinline__ void prepare() {}
  __device__ __forceinline__ void column(int c, u32x4 (&t)[3]) const {
#pragma unroll
    for (int p = 0; p < 4; ++p)
      t[0][p] = __builtin_amdgcn_perm(v[2 * p + 1][c / 2], v[2 * p][c / 2], c & 1 ? 0x07060302u : 0x05040100u);
  }
};

template <>
struct Rows<float> {
  static constexpr int kTerms = 3;
  raw8<float> v[8];
  __device__ __forceinline__ void load(int i, const void* x, const uint8_t*, int64_t row, int64_t ld, int c) {
    load8(v[i], static_cast<const float*>(x) + row * ld + c);
  }
  __device__ __forceinline__ void clear(int i) { v[i] = raw8<float>{}; }
  __device__ __forceinline__ void prepare() {}
  __device__ __forceinline__ void column(int c, u32x4 (&t)[3]) const {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = c < 4 ? v[i].a[c & 3] : v[i].b[c & 3];
    split8(x, t);
  }
};

// act8 codes: every value is a bf16 number, so one operand holds it exactly.
template <>
struct Rows<act8_t> {
  static constexpr int kTerms = 1;
  u32x2 v[8];
  uint32_t byte[8];
  float m[8];
  __device__ __forceinline__ void load(int i, const void* x, const uint8_t* scales, int64_t row, int64_t ld, int c) {
    v[i] = *reinterpret_cast<const u32x2*>(static_cast<const uint8_t*>(x) + row * ld + c);
    byte[i] = scales[row * (ld / 32) + c / 32];
  }
  __device__ __forceinline__ void clear(int i) {
    v[i] = u32x2{0u, 0u};
    byte[i] = 127u;
  }
  __device__ __forceinline__ void prepare() {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t s = byte[i] == 255u ? 0x7fc00000u : (max(byte[i], 6u) - 6u) << 23;
      m[i] = __builtin_bit_cast(float, s);
    }
  }
  __device__ __forceinline__ void column(int c, u32x4 (&t)[3]) const {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = static_cast<float>(static_cast<int8_t>(v[i][c / 4] >> (8 * (c & 3)))) * m[i];
#pragma unroll
    for (int p = 0; p < 4; ++p)
      t[0][p] = top_halves(__builtin_bit_cast(uint32_t, x[2 * p]), __builtin_bit_cast(uint32_t, x[2 * p + 1]));
  }
};

template <int RT>
__device__ __forceinline__ void load_rank(const float* p, float* v) {
  if constexpr (RT >= 4) {
#pragma unroll
    for (int q = 0; q < RT / 4; ++q) {
      const f32x4 r = reinterpret_cast<const f32x4*>(p)[q];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * q + i] = r[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < RT; ++i) v[i] = p[i];
  }
}

struct Side {
  const void* x;
  const uint8_t* scales;
  const float* s;   // [n][R]
  float* out;       // [nad][R][d]
  float* part;      // [chunks][R][d]
  int64_t ld;
  int d;
};

template <class X, int RT>
__device__ __forceinline__ void grad_tile(const Side& side, int col_wg, int begin, int end, int rk,
                                          const int* __restrict__ tokens, float* __restrict__ out,
                                          float (*red)[RT * 4 * 64]) {
  constexpr int R = 16 * RT;
  const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = col_wg * kCols + 8 * j;
  const int c = min(col, side.d - 8);
  f32x4 acc[RT][8];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[r][q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int t0 = begin + 32 * wave; t0 < end; t0 += 32 * kWaves) {
    Rows<X> x;
    float s[8][RT];
    const bool whole = t0 + 32 <= end;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t row = tokens[min(t0 + 8 * g + i, end - 1)];
      x.load(i, side.x, side.scales, row, side.ld, c);
      load_rank<RT>(side.s + row * R + RT * j, s[i]);
    }
    if (!whole) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (t0 + 8 * g + i >= end) {
          x.clear(i);
#pragma unroll
          for (int r = 0; r < RT; ++r) s[i][r] = 0.0f;
        }
    }
    x.prepare();
    u32x4 st[RT][3];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = s[i][r];
      split8(v, st[r]);
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      u32x4 xt[3];
      x.column(q, xt);
      // of three terms by three, those above 2^-24 of the product
#pragma unroll
      for (int m = 0; m < 3; ++m)
#pragma unroll
        for (int k = 0; k < Rows<X>::kTerms; ++k) {
          if (m + k > 2) continue;
#pragma unroll
          for (int r = 0; r < RT; ++r) acc[r][q] = mfma(st[r][m], xt[k], acc[r][q]);
        }
    }
  }
  // the four waves' sums, one column operand at a time: wave w writes its
  // share of every column, then sums two of the eight columns over the waves
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    __syncthreads();
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) red[wave][(r * 4 + e) * 64 + lane] = acc[r][q][e];
    __syncthreads();
    for (int i = threadIdx.x; i < RT * 4 * 64; i += 64 * kWaves) {
      const int l = i & 63, re = i >> 6;
      const int row = RT * (4 * (l >> 4) + (re & 3)) + (re >> 2), cc = col_wg * kCols + 8 * (l & 15) + q;
      float sum = red[0][i];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) sum += red[w][i];
      if (cc < side.d) out[static_cast<int64_t>(row) * side.d + cc] = row < rk ? sum : 0.0f;
    }
  }
}

template <class X, class G, int RT>
__global__ __launch_bounds__(64 * kWaves) void adapter_grad_kernel(Side a, Side b, int wgs_a, int nad,
                                                                   const int* __restrict__ rank, int span, Lists l) {
  constexpr int R = 16 * RT;
  __shared__ float red[kWaves][RT * 4 * 64];
  const int number = blockIdx.y;
  if (number >= l.chunk[nad]) return;
  int count = 0;
  for (int base = 0; base < nad; base += 64) {
    const int i = base + (threadIdx.x & 63);
    count += __popcll(__ballot(i < nad && l.chunk[i < nad ? i : 0] <= number));
  }
  const int ad = __builtin_amdgcn_readfirstlane(count - 1);
  const int first = l.chunk[ad], chunks = l.chunk[ad + 1] - first;
  const int begin = l.start[ad] + (number - first) * span, end = min(l.start[ad + 1], begin + span);
  const int rk = min(rank[ad], R);
  const bool left = blockIdx.x < wgs_a;
  const int64_t size = static_cast<int64_t>(R) * (left ? a.d : b.d);
  float* out = chunks == 1 ? (left ? a.out : b.out) + ad * size : (left ? a.part : b.part) + number * size;
  if (left)
    grad_tile<X, RT>(a, blockIdx.x, begin, end, rk, l.tokens, out, red);
  else
    grad_tile<G, RT>(b, blockIdx.x - wgs_a, begin, end, rk, l.tokens, out, red);
}

// Sums the chunks of the adapters that have several, clears those of none.
__global__ __launch_bounds__(256) void adapter_join_kernel(Side a, Side b, int R, int nad, Lists l) {
  const int ad = blockIdx.y;
  const int first = l.chunk[ad], last = l.chunk[ad + 1];
  if (last - first == 1) return;
  const bool left = blockIdx.z == 0;
  const float* part = left ? a.part : b.part;
  float* out = left ? a.out : b.out;
  const int64_t count = static_cast<int64_t>(R) * (left ? a.d : b.d);
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4; i < count;
       i += static_cast<int64_t>(gridDim.x) * 1024) {
    f32x4 s{0.0f, 0.0f, 0.0f, 0.0f};
    for (int k = first; k < last; ++k) s += *reinterpret_cast<const f32x4*>(part + k * count + i);
    *reinterpret_cast<f32x4*>(out + ad * count + i) = s;
  }
}

// Tokens per chunk: so many that the grid has about four workgroups for every
// compute unit, in whole turns of the four waves (128 tokens).
int span_of(int n, int d_in, int d_out) {
  const int wgs = (d_in + kCols - 1) / kCols + (d_out + kCols - 1) / kCols;
  const int chunks = (1024 + wgs - 1) / wgs;
  const int span = (n + chunks - 1) / chunks;
  return (span + 127) / 128 * 128 > 0 ? (span + 127) / 128 * 128 : 128;
}

int64_t chunk_numbers(int n, int span, int nad) { return static_cast<int64_t>(n / span) + nad; }

size_t round256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }

template <class X, class G, int RT>
void launch(dim3 grid, const Side& a, const Side& b, int wgs_a, int nad, const int* rank, int span, const Lists& l,
            hipStream_t s) {
  hipLaunchKernelGGL((adapter_grad_kernel<X, G, RT>), grid, dim3(64 * kWaves), 0, s, a, b, wgs_a, nad, rank, span, l);
}

template <class X, class G>
auto by_rank(int rmax) {
  return rmax == 16 ? launch<X, G, 1> : rmax == 32 ? launch<X, G, 2> : rmax == 64 ? launch<X, G, 4> : launch<X, G, 8>;
}

}  // namespace

namespace wush {

size_t adapter_grads_ws_bytes(int n, int d_in, int d_out, int nseg, int nad, int rmax) {
  const int span = span_of(n, d_in, d_out);
  return round256(static_cast<size_t>(n) * 4) + 2 * round256((static_cast<size_t>(nad) + 1) * 4) +
         round256(static_cast<size_t>(nseg) * 4) +
         static_cast<size_t>(chunk_numbers(n, span, nad)) * rmax * (static_cast<size_t>(d_in) + d_out) * sizeof(float);
}

bool adapter_grads_fit(int n, int d_in, int d_out, int nad) {
  return chunk_numbers(n, span_of(n, d_in, d_out), nad) <= 0xffff;
}

wush_status adapter_grads(const char* who, wush_dtype gdt, int xkind, int n, int d_in, int d_out, const void* dY,
                          int64_t ldg, const void* X, const uint8_t* x_scales, int64_t ldx, int nseg,
                          const int* seg_off, const int* seg_adapter, int nad, int rmax, const int* rank,
                          const float* V, const float* dV, float* dA, float* dBt, void* ws, hipStream_t s) {
  const int span = span_of(n, d_in, d_out);
  const int64_t numbers = chunk_numbers(n, span, nad);
  char* p = static_cast<char*>(ws);
  Lists l;
  l.tokens = reinterpret_cast<int*>(p);
  p += round256(static_cast<size_t>(n) * 4);
  l.start = reinterpret_cast<int*>(p);
  p += round256((static_cast<size_t>(nad) + 1) * 4);
  l.chunk = reinterpret_cast<int*>(p);
  p += round256((static_cast<size_t>(nad) + 1) * 4);
  l.place = reinterpret_cast<int*>(p);
  p += round256(static_cast<size_t>(nseg) * 4);
  float* part = reinterpret_cast<float*>(p);
  const Side a{X, x_scales, dV, dA, part, ldx, d_in};
  const Side b{dY, nullptr, V, dBt, part + numbers * rmax * d_in, ldg, d_out};
  hipLaunchKernelGGL(adapter_list_kernel, dim3(1), dim3(1024), 0, s, n, nseg, seg_off, seg_adapter, nad, rank, span, l);
  const int wgs_a = (d_in + kCols - 1) / kCols, wgs_b = (d_out + kCols - 1) / kCols;
  if (n > 0) {
    const dim3 grid(wgs_a + wgs_b, static_cast<unsigned>(numbers));
    const bool g32 = gdt == WUSH_F32;
    auto f = xkind == WUSH_F32 ? (g32 ? by_rank<float, float>(rmax) : by_rank<float, bf16_t>(rmax))
             : xkind == WUSH_BF16 ? (g32 ? by_rank<bf16_t, float>(rmax) : by_rank<bf16_t, bf16_t>(rmax))
                                  : (g32 ? by_rank<act8_t, float>(rmax) : by_rank<act8_t, bf16_t>(rmax));
    f(grid, a, b, wgs_a, nad, rank, span, l, s);
  }
  const int most = d_in > d_out ? d_in : d_out;
  const int64_t wide = (static_cast<int64_t>(rmax) * most + 1023) / 1024;
  hipLaunchKernelGGL(adapter_join_kernel, dim3(static_cast<unsigned>(wide < 2048 ? wide : 2048), nad, 2), dim3(256), 0,
                     s, a, b, rmax, nad, l);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? WUSH_OK : fail(WUSH_E_HIP, "%s launch: %s", who, hipGetErrorString(e));
}

}  // namespace wush
