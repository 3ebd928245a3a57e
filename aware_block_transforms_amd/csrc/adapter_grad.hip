// The grad kernel of the adapters: dF[a][r][c] = sum over the tokens t of
// adapter a of S[t][r] X[t][c], for (S, X, F) = (dV, X, A) and (V, dY, Bt).
//
// The sum runs over tokens, which lie along the slow axis of both operands, and
// an adapter's tokens may be spread over many requests.  So the tokens of each
// adapter are listed in order first (list_tokens), each list padded to whole
// steps of 32 tokens, and cut into chunks of several steps; a last kernel adds
// up the chunks of an adapter in order, so that results do not depend on scheduling
// (an adapter of one chunk is written directly).
//
// In a 16x16x32 product the eight k values of a lane are eight tokens.  A lane
// therefore loads the same eight columns of eight token rows, 16 bytes each
// (16 lanes read 256 contiguous bytes of a row), and exchanges halves between
// its own registers; no lane exchange is needed, since which column a result
// belongs to is free to choose: operand c of lane j is column 8 j + c.  A wave
// owns 128 columns.  The four waves of a workgroup walk over the same tokens
// and share the operands of S, which they split into three bf16 terms together,
// one step ahead, through two LDS buffers.  The rows of a bf16 or act8 X are loaded
// one step ahead too, into the registers that the step's operands have just left.
// Those of an fp32 X (or dY), of three terms, are loaded inside their step: there
// are no registers for more, and at rank 64 the kernel spills 92 to 100 bytes a
// lane wherever one side is fp32.
//
// Bound by the loads' latency at two waves a SIMD (one at rank 128), whose
// accumulators (16 RT x 128 fp32 a wave) leave no room for more.  4096 tokens,
// 4096 + 12288 bf16 columns at rank 32: 30 us and 6.5 us of join, 5.6 TB/s with
// the parts.  16384 tokens, 17408 act8 + 5120 bf16 columns at rank 64, 70% of the tokens with an
// adapter: 86 us and 11 us, 4.4 TB/s; the matrix cores are busy for 22 us of it,
// turning codes into values takes as long (each wave splitting all of S by
// itself: 147 us).  An order of the workgroups that keeps a chunk's columns on
// one XCD reads S once but takes 96 us.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "adapter.h"
#include "common.h"

using namespace wush;

namespace {

constexpr int kWaves = 4;
constexpr int kCols = 128 * kWaves;

// The lists of no tokens.
__global__ __launch_bounds__(256) void adapter_list_kernel(int nseg, const int* off, const int* ids, int nad,
                                                           const int* rank, int rmax, Lists l) {
  list_tokens<4>(0, nseg, off, ids, nad, rank, rmax, 1, nullptr, 0, l);
}

// Adapter of a step or chunk `number`: the last one whose first is not past it.
__device__ __forceinline__ int owner(const int* __restrict__ firsts, int nad, int number) {
  int count = 0;
  for (int b = 0; b < nad; b += 64) {
    const int i = b + (threadIdx.x & 63);
    count += __popcll(__ballot(i < nad && firsts[i < nad ? i : 0] <= number));
  }
  return __builtin_amdgcn_readfirstlane(count - 1);
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
  __device__ __forceinline__ void prepare() {}
  __device__ __forceinline__ void column(int c, u32x4 (&t)[1]) const {
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
  __device__ __forceinline__ void load(int i, const void* x, const uint8_t* scales, int64_t row, int64_t ld, int c) {
    v[i] = *reinterpret_cast<const u32x2*>(static_cast<const uint8_t*>(x) + row * ld + c);
    byte[i] = scales[row * (ld / 32) + c / 32];
  }
  // The scale bytes as 2^(e-6).  A byte of 255 stands for NaN, and is rare: one
  // look at the largest decides.
  __device__ __forceinline__ void prepare() {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, byte[i]);
    const bool bad = __ballot(top == 255u) != 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t unit = (byte[i] << 23) - (6u << 23);
      byte[i] = bad && byte[i] == 255u ? 0x7fc00000u : unit;
    }
  }
  __device__ __forceinline__ void column(int c, u32x4 (&t)[1]) const {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = static_cast<float>(static_cast<int8_t>(v[i][c / 4] >> (8 * (c & 3)))) * __builtin_bit_cast(float, byte[i]);
#pragma unroll
    for (int p = 0; p < 4; ++p)
      t[0][p] = top_halves(__builtin_bit_cast(uint32_t, x[2 * p]), __builtin_bit_cast(uint32_t, x[2 * p + 1]));
  }
};

struct Side {
  const void* x;
  const uint8_t* scales;
  const float* s;   // [n][R]
  float* out;       // [nad][R][d]
  float* part;      // [parts][R][d]
  int64_t ld;
  int d;
};

// Keeps the scheduler from moving loads and operands of one part of a step into
// another, which costs more registers than there are.
__device__ __forceinline__ void fence() { __builtin_amdgcn_sched_barrier(0); }

// Operands of S for one step: row tile, term, lane.
template <int RT>
using Shared = u32x4[RT][3][64];

// Steps [first, last) of an adapter whose list ends at `end`, for NT of the RT
// row tiles.
template <class X, int NT, int RT>
__device__ __forceinline__ void grad_steps(const Side& side, int c, int first, int last, int end,
                                           const int* __restrict__ tokens, Shared<RT>* ops, f32x4 (&acc)[RT][8]) {
  constexpr int R = 16 * RT, kTerms = Rows<X>::kTerms, kShare = (NT + kWaves - 1) / kWaves;
  const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Rows<X> x;
  float v[kShare][8];
  // a step's tokens are one per lane (twice); a lane's own are 8 g .. 8 g + 7
  auto list = [&](int step) { return tokens[32 * step + (lane & 31)]; };
  auto load_x = [&](int token) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x.load(i, side.x, side.scales, __shfl(token, 8 * g + i, 64), side.ld, c);
  };
  // S of the row tiles that this wave prepares
  auto load_s = [&](int token) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float* p = side.s + static_cast<int64_t>(__shfl(token, 8 * g + i, 64)) * R + j;
#pragma unroll
      for (int w = 0; w < kShare; ++w)
        if (wave + w * kWaves < NT) v[w][i] = p[16 * (wave + w * kWaves)];
    }
  };
  auto share = [&](int step, Shared<RT>& to) {
#pragma unroll
    for (int w = 0; w < kShare; ++w) {
      const int r = wave + w * kWaves;
      if (r >= NT) break;
      if (32 * (step + 1) > end) {   // padding
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (32 * step + 8 * g + i >= end) v[w][i] = 0.0f;
      }
      u32x4 o[3];
      split8(v[w], o);
#pragma unroll
      for (int m = 0; m < 3; ++m) to[r][m][lane] = o[m];
    }
  };
  int token = list(first), ahead = first + 1 < last ? list(first + 1) : 0;
  load_s(token);
  if constexpr (kTerms == 1) load_x(token);
  share(first, ops[0]);
  __syncthreads();
  for (int step = first, buf = 0; step < last; ++step, buf ^= 1) {
    const bool more = step + 1 < last;
    u32x4 xt[8][1];
    if constexpr (kTerms == 1) {
      x.prepare();
#pragma unroll
      for (int q = 0; q < 8; ++q) x.column(q, xt[q]);
      fence();
    } else {
      load_x(token);
    }
    if (more) {
      token = ahead;
      load_s(token);
      if constexpr (kTerms == 1) load_x(token);
      if (step + 2 < last) ahead = list(step + 2);
    }
    if constexpr (kTerms == 1) {
#pragma unroll
      for (int m = 0; m < 3; ++m) {
        fence();
        u32x4 st[NT];
#pragma unroll
        for (int r = 0; r < NT; ++r) st[r] = ops[buf][r][m][lane];
#pragma unroll
        for (int q = 0; q < 8; ++q)
#pragma unroll
          for (int r = 0; r < NT; ++r) acc[r][q] = mfma(st[r], xt[q][0], acc[r][q]);
      }
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        u32x4 t[3];
        x.column(q, t);
        // of three terms by three, those above 2^-24 of the product
#pragma unroll
        for (int m = 0; m < 3; ++m)
#pragma unroll
          for (int r = 0; r < NT; ++r) {
            const u32x4 st = ops[buf][r][m][lane];
#pragma unroll
            for (int k = 0; k < 3 - m; ++k) acc[r][q] = mfma(st, t[k], acc[r][q]);
          }
      }
    }
    fence();
    if (more) share(step + 1, ops[buf ^ 1]);
    __syncthreads();
  }
}

// `where` gives the place of the results: it is looked up after the steps, which
// have no registers to spare for it.
template <class X, int RT, class F>
__device__ __forceinline__ void grad_tile(const Side& side, int c0, int first, int last, int end, int rk,
                                          int rows, const int* __restrict__ tokens, Shared<RT>* ops, F where) {
  const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
  // waves and lanes past the last column repeat it: they still share the work
  // on S, and store nothing
  const int col = c0 + 8 * j, c = min(col, side.d - 8);
  f32x4 acc[RT][8];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[r][q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  // row tiles in use, rounded up to a power of two; the extra ones are zero in S
  const int tiles = (rk + 15) / 16;
  if (RT > 4 && tiles > 4)
    grad_steps<X, RT, RT>(side, c, first, last, end, tokens, ops, acc);
  else if (RT > 2 && tiles > 2)
    grad_steps<X, (RT > 4 ? 4 : RT), RT>(side, c, first, last, end, tokens, ops, acc);
  else if (RT > 1 && tiles > 1)
    grad_steps<X, (RT > 2 ? 2 : RT), RT>(side, c, first, last, end, tokens, ops, acc);
  else
    grad_steps<X, 1, RT>(side, c, first, last, end, tokens, ops, acc);
  if (col >= side.d) return;
  float* __restrict__ out = where();
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int row = 16 * r + 4 * g + e;
      if (row >= rows) continue;
      float v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = row < rk ? acc[r][q][e] : 0.0f;
      store8(out + static_cast<int64_t>(row) * side.d + col, v);
    }
}

// Two waves a SIMD up to rank 64, whose accumulators take half of the registers.
template <class X, class G, int RT>
__global__ __launch_bounds__(64 * kWaves, RT > 4 ? 1 : 2) void adapter_grad_kernel(Side a, Side b, int wgs_a, int nad,
                                                                   const int* __restrict__ rank, Lists l) {
  constexpr int R = 16 * RT;
  __shared__ Shared<RT> ops[2];
  const int number = blockIdx.y;
  if (number >= l.chunk[nad]) return;
  const int ad = owner(l.chunk, nad, number);
  const int before = l.chunk[ad], chunks = l.chunk[ad + 1] - before;
  const int span = l.span[ad];
  const int first = l.start[ad] + (number - before) * span, last = min(l.start[ad + 1], first + span);
  const int rk = min(rank[ad], R);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool left = blockIdx.x < wgs_a;
  auto where = [&]() {
    const int64_t size = static_cast<int64_t>(R) * (left ? a.d : b.d);
    return chunks == 1 ? (left ? a.out : b.out) + ad * size
                       : (left ? a.part : b.part) + (l.part[ad] + number - l.chunk[ad]) * size;
  };
  const int c0 = (left ? blockIdx.x : blockIdx.x - wgs_a) * kCols + 128 * wave;
  const int end = l.start[ad] + l.count[ad];
  // rows that do not count are left out of the chunks' parts
  const int rows = chunks == 1 ? R : rk;
  if (left)
    grad_tile<X, RT>(a, c0, first / 32, last / 32, end, rk, rows, l.tokens, ops, where);
  else
    grad_tile<G, RT>(b, c0, first / 32, last / 32, end, rk, rows, l.tokens, ops, where);
}

// Sums the chunks of the adapters that have several, clears those of none and
// the rows that do not count.
__global__ __launch_bounds__(256) void adapter_join_kernel(Side a, Side b, int R, int nad,
                                                           const int* __restrict__ rank, Lists l) {
  const int ad = blockIdx.y;
  const int chunks = l.chunk[ad + 1] - l.chunk[ad], first = l.part[ad], last = first + chunks;
  if (chunks == 1) return;
  const bool left = blockIdx.z == 0;
  const float* part = left ? a.part : b.part;
  float* out = left ? a.out : b.out;
  const int d = left ? a.d : b.d;
  const int64_t count = static_cast<int64_t>(R) * d, used = static_cast<int64_t>(min(max(rank[ad], 0), R)) * d;
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4; i < count;
       i += static_cast<int64_t>(gridDim.x) * 1024) {
    f32x4 s{0.0f, 0.0f, 0.0f, 0.0f};
    if (i < used) {
#pragma unroll 4
      for (int k = first; k < last; ++k) s += *reinterpret_cast<const f32x4*>(part + k * count + i);
    }
    *reinterpret_cast<f32x4*>(out + ad * count + i) = s;
  }
}

// Chunks wanted: so many that the workgroups fit the compute units once (two on
// each, one at rank 128), since a second round for the last few would take as
// long as the first.  The backward call without dX, two adapters, 4096 tokens of
// 4096 + 12288 and 16384 of 5120 + 5120 bf16 columns: 54 and 100 us at rank 16
// (with 256 more workgroups, which still fit, 56 and 105), 61 and 110 at rank 32,
// 79 and 143 at rank 64, 130 and 254 at rank 128; at ranks 32 to 128 with half as
// many 66 to 180 and 136 to 389, with twice as many 71 to 158 and 123 to 275.
int chunks_wanted(int n, int d_in, int d_out, int rmax) {
  const int wgs = (d_in + kCols - 1) / kCols + (d_out + kCols - 1) / kCols;
  const int slots = rmax == 128 ? 256 : 512;
  const int least = n / (32 * kMinSteps) + 1;
  const int c = slots / wgs;
  return c < 1 ? 1 : c < least ? c : least;
}

// Chunks there may be: each list's last may be short.
int64_t chunk_numbers(int n, int d_in, int d_out, int nad, int rmax) {
  return static_cast<int64_t>(chunks_wanted(n, d_in, d_out, rmax)) + nad;
}
// Partial sums there may be: chunks of adapters that have several.  Such an
// adapter has less than twice as many as its tokens fill, and all together fill
// no more than the chunks wanted.
int64_t part_numbers(int n, int d_in, int d_out, int nad, int rmax) {
  const int64_t all = chunk_numbers(n, d_in, d_out, nad, rmax), most = 2 * static_cast<int64_t>(chunks_wanted(n, d_in, d_out, rmax));
  return all < most ? all : most;
}
int64_t step_numbers(int n, int nad) { return static_cast<int64_t>(n / 32) + nad; }

size_t round256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }

size_t list_bytes(int n, int nseg, int nad) {
  return round256(static_cast<size_t>(step_numbers(n, nad)) * 32 * 4) + 5 * round256((static_cast<size_t>(nad) + 1) * 4) +
         round256(static_cast<size_t>(nseg) * 4);
}

template <class X, class G, int RT>
void launch(dim3 grid, const Side& a, const Side& b, int wgs_a, int nad, const int* rank, const Lists& l,
            hipStream_t s) {
  hipLaunchKernelGGL((adapter_grad_kernel<X, G, RT>), grid, dim3(64 * kWaves), 0, s, a, b, wgs_a, nad, rank, l);
}

template <class X, class G>
auto by_rank(int rmax) {
  return rmax == 16 ? launch<X, G, 1> : rmax == 32 ? launch<X, G, 2> : rmax == 64 ? launch<X, G, 4> : launch<X, G, 8>;
}

}  // namespace

namespace wush {

size_t adapter_grads_ws_bytes(int n, int d_in, int d_out, int nseg, int nad, int rmax) {
  return list_bytes(n, nseg, nad) +
         static_cast<size_t>(part_numbers(n, d_in, d_out, nad, rmax)) * rmax * (static_cast<size_t>(d_in) + d_out) * sizeof(float);
}

ListJob adapter_lists(int n, int d_in, int d_out, int nseg, int nad, int rmax, void* ws) {
  char* p = static_cast<char*>(ws);
  auto take = [&](size_t count) {
    int* at = reinterpret_cast<int*>(p);
    p += round256(count * 4);
    return at;
  };
  ListJob job{true, chunks_wanted(n, d_in, d_out, rmax), {}};
  job.l.tokens = take(static_cast<size_t>(step_numbers(n, nad)) * 32);
  job.l.count = take(static_cast<size_t>(nad) + 1);
  job.l.start = take(static_cast<size_t>(nad) + 1);
  job.l.chunk = take(static_cast<size_t>(nad) + 1);
  job.l.part = take(static_cast<size_t>(nad) + 1);
  job.l.span = take(static_cast<size_t>(nad) + 1);
  job.l.place = take(nseg);
  return job;
}

bool adapter_grads_fit(int n, int d_in, int d_out, int nad, int rmax) {
  return chunk_numbers(n, d_in, d_out, nad, rmax) <= 0xffff;
}

wush_status adapter_grads(const char* who, wush_dtype gdt, int xkind, int n, int d_in, int d_out, const void* dY,
                          int64_t ldg, const void* X, const uint8_t* x_scales, int64_t ldx, int nseg,
                          const int* seg_off, const int* seg_adapter, int nad, int rmax, const int* rank,
                          const float* V, const float* dV, float* dA, float* dBt, void* ws, hipStream_t s) {
  const int64_t numbers = chunk_numbers(n, d_in, d_out, nad, rmax);
  const ListJob job = adapter_lists(n, d_in, d_out, nseg, nad, rmax, ws);
  const Lists& l = job.l;
  float* part = reinterpret_cast<float*>(static_cast<char*>(ws) + list_bytes(n, nseg, nad));
  const Side a{X, x_scales, dV, dA, part, ldx, d_in};
  const Side b{dY, nullptr, V, dBt, part + part_numbers(n, d_in, d_out, nad, rmax) * rmax * d_in, ldg, d_out};
  // with tokens, the low kernel has made the lists
  if (n == 0)
    hipLaunchKernelGGL(adapter_list_kernel, dim3(1), dim3(256), 0, s, nseg, seg_off, seg_adapter, nad, rank, rmax, l);
  const int wgs_a = (d_in + kCols - 1) / kCols, wgs_b = (d_out + kCols - 1) / kCols;
  if (n > 0) {
    const dim3 grid(wgs_a + wgs_b, static_cast<unsigned>(numbers));
    const bool g32 = gdt == WUSH_F32;
    auto f = xkind == WUSH_F32 ? (g32 ? by_rank<float, float>(rmax) : by_rank<float, bf16_t>(rmax))
             : xkind == WUSH_BF16 ? (g32 ? by_rank<bf16_t, float>(rmax) : by_rank<bf16_t, bf16_t>(rmax))
                                  : (g32 ? by_rank<act8_t, float>(rmax) : by_rank<act8_t, bf16_t>(rmax));
    f(grid, a, b, wgs_a, nad, rank, l, s);
  }
  const int most = d_in > d_out ? d_in : d_out;
  const int64_t wide = (static_cast<int64_t>(rmax) * most + 1023) / 1024;
  hipLaunchKernelGGL(adapter_join_kernel, dim3(static_cast<unsigned>(wide < 2048 ? wide : 2048), nad, 2), dim3(256), 0,
                     s, a, b, rmax, nad, rank, l);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? WUSH_OK : fail(WUSH_E_HIP, "%s launch: %s", who, hipGetErrorString(e));
}

}  // namespace wush
