// Low-rank adapters of many requests beside a shared projection.
//
// Adapter a has A [R][d_in] and Bt [R][d_out] (the transpose of the usual B),
// of which the first rank[a] rows count, and a factor alpha[a].  For the tokens
// of a request with adapter a
//   V = alpha X A^T,   Y = Y0 + V Bt,
// and backward, from dY and the V of the forward call,
//   dV = alpha dY Bt^T,   dX = dX0 + dV A,   dA = dV^T X,   dBt = V^T dY.
// With both factors stored as rows of d values, three kernels do all of it:
//   low     V  = alpha X A^T   (also dV from dY and Bt)
//   spread  Y  = Y0 + V Bt     (also dX from dV and A)
//   grad    dA = dV^T X        (also dBt from V and dY), in adapter_grad.hip
// All are bound by memory at ranks up to 64: a pass over bf16 rows at rank r does
// r flops per byte of them, against a matrix rate of some 230 per byte that a
// large copy moves.  So X, Y0, Y and dY are read once by each kernel, and the
// operands of fp32 values are split into three bf16 terms (split3), which keeps V
// and all results at fp32 accuracy.  dY is read twice by a backward call, by the
// low and the grad kernel: dBt needs V of all tokens, dV a whole row of dY.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "adapter.h"
#include "common.h"

using namespace wush;

namespace wush {
wush_status adapter_grads(const char* who, wush_dtype gdt, int xkind, int n, int d_in, int d_out, const void* dY,
                          int64_t ldg, const void* X, const uint8_t* x_scales, int64_t ldx, int nseg,
                          const int* seg_off, const int* seg_adapter, int nad, int rmax, const int* rank,
                          const float* V, const float* dV, float* dA, float* dBt, void* ws, hipStream_t s);
ListJob adapter_lists(int n, int d_in, int d_out, int nseg, int nad, int rmax, void* ws);
bool adapter_grads_fit(int n, int d_in, int d_out, int nad, int rmax);
size_t adapter_grads_ws_bytes(int n, int d_in, int d_out, int nseg, int nad, int rmax);
}  // namespace wush

namespace {

constexpr int kWaves = 4;

// ---------------------------------------------------------------------------
// low: V[t][r] = alpha sum_k X[t][k] A[r][k], by 16x16x32 products of token
// rows with factor rows, both with k along the row.  A workgroup takes 16 TT
// tokens; its four waves and the grid's y share k in pieces of 64.  The waves'
// sums are joined through LDS, those of the y workgroups lie in `part`
// [gridDim.y][n][R] and are added by whoever reads V.
//
// An operand wants 16 rows side by side in neighbouring lanes, and loaded that
// way every lane is an access of its own to the first-level cache, which then
// bounds the kernel.  So a wave loads its pieces in whole 128-byte lines (eight
// lanes a row) and takes the operands out of its own part of LDS, where the
// 16-byte chunks of row r are kept in the order c ^ (r mod the row's chunks), so
// that the eight or sixteen rows of a read fall into different banks.  The next
// piece is on its way, in registers, during the products of the one in LDS.  The
// lanes of a wave read what others of its lanes wrote: its LDS instructions take
// effect in order, so no barrier is needed, only an order that the compiler keeps
// (lds_order).  Rows past the tile's tokens or the rank, and columns past
// d, lie outside the buffer resources and come as zeros.
//
// 16384 x 5120 in bf16 at rank 64: 42 us, 4.0 TB/s of X (55 us with operands
// loaded row by row); 4096 x 12288 at rank 32: 28 us, 3.7 TB/s.  Waits for loads
// are what is left: two pieces ahead in registers were slower (88 us, they cost
// half of the waves), and so were other orders of k.

// A piece of 64 columns of 16 N rows: C 16-byte chunks a row.
template <class T, int N>
struct Piece {
  static constexpr int C = is_f32<T> ? 16 : 8, kRows = 64 / C, kLoads = 16 * N / kRows, kBytes = 16 * N * C * 16;
  static constexpr int kValues = 16 / sizeof(T);   // of a chunk
  __amdgpu_buffer_rsrc_t from;
  uint32_t lane_at, stride, columns;
  u32x4 v[kLoads];

  // `rows` rows of d values, ld apart
  __device__ __forceinline__ void open(const T* p, int rows, int d, int64_t ld) {
    const int lane = threadIdx.x & 63;
    from = __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(p), static_cast<short>(0),
                                             ((rows - 1) * static_cast<int>(ld) + d) * static_cast<int>(sizeof(T)), 0x00020000);
    stride = static_cast<uint32_t>(kRows * ld * sizeof(T));
    lane_at = static_cast<uint32_t>((lane / C) * ld * sizeof(T)) + lane % C * 16;
    columns = d;
  }
  // the used row tiles' loads, at column k; the rows count in the vector offset,
  // which is what the range check is sure to see
  template <int USED>
  __device__ __forceinline__ void load(int k) {
#pragma unroll
    for (int i = 0; i < USED * 16 / kRows; ++i)
      v[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(from, lane_at + i * stride, k * sizeof(T), 0));
  }
  // the same for a piece that runs past the last column
  template <int USED>
  __device__ __forceinline__ void load_tail(int k) {
    const uint32_t at = k + (threadIdx.x & 63) % C * kValues < columns ? lane_at : 0x80000000u;
#pragma unroll
    for (int i = 0; i < USED * 16 / kRows; ++i)
      v[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(from, at + i * stride, k * sizeof(T), 0));
  }
  template <int USED>
  __device__ __forceinline__ void put(u32x4* lds) const {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < USED * 16 / kRows; ++i) {
      const int r = i * kRows + lane / C;
      lds[r * C + (lane % C ^ r % C)] = v[i];
    }
  }
};

// Between a wave's writes to its part of LDS and its other lanes' reads of it,
// both ways.  No instruction comes of it.
__device__ __forceinline__ void lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
}

// The operand of row tile i and k half h, lane 16 g + j: columns 8 (4 h + g) ..
// of row 16 i + j.
__device__ __forceinline__ void low_operand(const u32x4* lds, int i, int h, u32x4 (&t)[1], bf16_t) {
  const int lane = threadIdx.x & 63, r = 16 * i + (lane & 15), c = 4 * h + (lane >> 4);
  t[0] = lds[r * 8 + (c ^ r % 8)];
}
__device__ __forceinline__ void low_operand(const u32x4* lds, int i, int h, u32x4 (&t)[3], float) {
  const int lane = threadIdx.x & 63, r = 16 * i + (lane & 15), c = 2 * (4 * h + (lane >> 4));
  const f32x4 a = __builtin_bit_cast(f32x4, lds[r * 16 + (c ^ r % 16)]);
  const f32x4 b = __builtin_bit_cast(f32x4, lds[r * 16 + ((c + 1) ^ r % 16)]);
  const float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  split8(v, t);
}

// The products of a wave's pieces of k, for NT row tiles of the factor.
template <class X, int NT, int RT, int TT>
__device__ __forceinline__ void low_pieces(Piece<X, TT>& x, Piece<bf16_t, RT>& f, int k, int d, int step, u32x4* lds,
                                           f32x4 (&acc)[TT][RT]) {
  constexpr int kTerms = is_f32<X> ? 3 : 1;
  u32x4 *xl = lds, *fl = lds + Piece<X, TT>::kBytes / 16;
  auto multiply = [&]() {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      u32x4 ft[NT][1];
#pragma unroll
      for (int r = 0; r < NT; ++r) low_operand(fl, r, h, ft[r], bf16_t());
#pragma unroll
      for (int i = 0; i < TT; ++i) {
        u32x4 xt[kTerms];
        low_operand(xl, i, h, xt, X());
#pragma unroll
        for (int m = 0; m < kTerms; ++m)
#pragma unroll
          for (int r = 0; r < NT; ++r) acc[i][r] = mfma(xt[m], ft[r][0], acc[i][r]);
      }
    }
  };
  const int whole = k + 64 <= d ? (d - 64 - k) / step + 1 : 0;
  if (whole > 0) {
    x.template load<TT>(k);
    f.template load<NT>(k);
    for (int i = 0; i < whole; ++i) {
      x.template put<TT>(xl);
      f.template put<NT>(fl);
      lds_order();
      // past the last piece it is loaded again: a branch would cost a wait
      const int next = k + min(i + 1, whole - 1) * step;
      x.template load<TT>(next);
      f.template load<NT>(next);
      multiply();
      lds_order();
    }
  }
  k += whole * step;
  if (k < d) {
    x.template load_tail<TT>(k);
    f.template load_tail<NT>(k);
    x.template put<TT>(xl);
    f.template put<NT>(fl);
    lds_order();
    multiply();
  }
  lds_order();
}

template <class X, int RT, int TT>
__global__ __launch_bounds__(64 * kWaves) void adapter_low_kernel(int n, int d, const X* __restrict__ x, int64_t ldx,
                                                                  int nseg, const int* __restrict__ off,
                                                                  const int* __restrict__ ids, int nad,
                                                                  const bf16_t* __restrict__ factor,
                                                                  const int* __restrict__ rank,
                                                                  const float* __restrict__ alpha,
                                                                  float* __restrict__ part, ListJob job) {
  constexpr int R = 16 * RT, T = 16 * TT;
  // a wave's pieces, and after the products its sums of one token tile
  constexpr int kPieces = (Piece<X, TT>::kBytes + Piece<bf16_t, RT>::kBytes) / 16, kSums = 16 * R / 4;
  __shared__ u32x4 lds[kWaves][kPieces > kSums ? kPieces : kSums];
  if (job.on && blockIdx.x == 0) {
    if (blockIdx.y == 0)
      list_tokens<kWaves>(n, nseg, off, ids, nad, rank, R, job.chunks_wanted, reinterpret_cast<int*>(lds),
                          sizeof(lds) / sizeof(int), job.l);
    return;
  }
  const Tile t = find_tile<T>(blockIdx.x - job.on, n, nseg, off, ids, nad);
  if (t.begin >= t.end) return;
  float* out = part + (static_cast<int64_t>(blockIdx.y) * n + t.begin) * R;
  const int rows = t.end - t.begin;
  const int rk = t.adapter < 0 ? 0 : min(max(rank[t.adapter], 0), R);
  if (rk == 0) {
    for (int i = threadIdx.x; i < rows * R; i += 64 * kWaves) out[i] = 0.0f;
    return;
  }
  const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Piece<X, TT> xp;
  Piece<bf16_t, RT> fp;
  xp.open(x + t.begin * ldx, rows, d, ldx);
  fp.open(factor + static_cast<int64_t>(t.adapter) * R * d, rk, d, d);
  f32x4 acc[TT][RT];
#pragma unroll
  for (int i = 0; i < TT; ++i)
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[i][r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const int step = 64 * kWaves * gridDim.y, k = 64 * (kWaves * blockIdx.y + wave);
  // row tiles in use, rounded up to a power of two
  const int tiles = (rk + 15) / 16;
  if (RT > 4 && tiles > 4)
    low_pieces<X, RT, RT, TT>(xp, fp, k, d, step, lds[wave], acc);
  else if (RT > 2 && tiles > 2)
    low_pieces<X, (RT > 4 ? 4 : RT), RT, TT>(xp, fp, k, d, step, lds[wave], acc);
  else if (RT > 1 && tiles > 1)
    low_pieces<X, (RT > 2 ? 2 : RT), RT, TT>(xp, fp, k, d, step, lds[wave], acc);
  else
    low_pieces<X, 1, RT, TT>(xp, fp, k, d, step, lds[wave], acc);
  const float f = alpha[t.adapter];
  auto sums = [&](int w) { return reinterpret_cast<float*>(lds[w]); };
#pragma unroll
  for (int i = 0; i < TT; ++i) {
    if (16 * i >= rows) break;
    if (i > 0) __syncthreads();
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) sums(wave)[(4 * g + e) * R + 16 * r + j] = acc[i][r][e];
    __syncthreads();
    const int count = min(rows - 16 * i, 16) * R;
    for (int q = threadIdx.x; q < count; q += 64 * kWaves) {
      float s = sums(0)[q];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) s += sums(w)[q];
      out[16 * i * R + q] = q % R < rk ? f * s : 0.0f;
    }
  }
}

// ---------------------------------------------------------------------------
// spread: Y[t][c] = Y0[t][c] + sum_r V[t][r] Bt[r][c].  A wave owns 16 CW
// columns: its lane j those from CW j on, so that a row of Y0 and Y is read and
// written in whole 256-byte runs, 16 bytes a lane.  The factor's rows lie along
// the columns, so a lane reads eight rows (k) of its CW columns and exchanges
// halves between them to get CW operands; they stay in registers while the
// workgroup walks over its 16 TT tokens.  V's operands are the same for every
// column: the workgroup adds up the low kernel's parts and splits them once,
// into LDS, in the order the matrix instructions take them.  The sums start
// from Y0, whose next rows are loaded before the products of those in hand.
//
// 16384 x 17408 in fp32 at rank 64: 393 us, 5.8 TB/s of Y0 and Y, what a copy of
// that size reaches or more.  64 requests of one token on 12288 columns: 14 us,
// which the start of a workgroup (its request, the parts of V, the first factor
// rows) and five column blocks in turn take.  More and shorter workgroups do not
// help (16 us with 1152, 23 us with 3264, against 704), nor does an order that
// keeps requests of one column block on one XCD.

template <class T>
struct YRow;
template <>
struct YRow<float> {
  static constexpr int CW = 4;
  using raw = f32x4;
  using factors = u32x2;
  f32x4 v;
  __device__ __forceinline__ float at(int c) const { return v[c]; }
  __device__ __forceinline__ void put(const float* s) { v = f32x4{s[0], s[1], s[2], s[3]}; }
};
template <>
struct YRow<bf16_t> {
  static constexpr int CW = 8;
  using raw = u32x4;
  using factors = u32x4;
  u32x4 v;
  __device__ __forceinline__ float at(int c) const {
    return __builtin_bit_cast(float, c & 1 ? v[c / 2] & 0xffff0000u : v[c / 2] << 16);
  }
  __device__ __forceinline__ void put(const float* s) {
    v = u32x4{pack_bf16(s[0], s[1]), pack_bf16(s[2], s[3]), pack_bf16(s[4], s[5]), pack_bf16(s[6], s[7])};
  }
};

// What a spread workgroup knows of its tile.
struct SpreadTile {
  int begin, rows, rank, col_wg;
  int c0, stride;   // the wave's first columns, and the step to its next ones
};

// Operands of one 16-token tile and 32 ranks: three terms.  At rank 16 the
// upper half of k is free, and the first two terms share one operand (against
// the factor's rows twice).
template <int RT, int TT>
using SpreadOps = u32x4[TT][(RT + 1) / 2][RT == 1 ? 2 : 3][64];

// Where lane 16 g + j's 16 bytes of an operand lie.  Neighbouring threads of
// stage_v write neighbouring lane groups, which without the exchange would fall
// into the same banks.
template <int RT>
__device__ __forceinline__ int spread_slot(int ks, int g, int j) {
  return 16 * g + (j ^ (RT == 1 ? 4 * (g & 1) : 2 * g + (ks & 1)));
}

__device__ __forceinline__ void add8(float* v, const raw8<float>& r, bool counts) {
  float w[8];
  widen8(r, w);
#pragma unroll
  for (int x = 0; x < 8; ++x) v[x] += counts ? w[x] : 0.0f;
}

// Adds up the parts of V for the tile's tokens and puts its operands into LDS.
template <int RT, int TT>
__device__ __forceinline__ void stage_v(const SpreadTile& t, int n, const float* __restrict__ part, int splits,
                                        float* __restrict__ V, SpreadOps<RT, TT>& vop) {
  constexpr int R = 16 * RT;
  const int tiles = (t.rows + 15) / 16;
  const int64_t v_step = static_cast<int64_t>(n) * R;
  for (int q = threadIdx.x; q < tiles * 16 * (R / 8); q += 64 * kWaves) {
    const int row = q / (R / 8), r8 = q % (R / 8);
    float v[8] = {};
    if (row < t.rows) {
      const int64_t at = (static_cast<int64_t>(t.begin) + row) * R + 8 * r8;
      // four loads in flight, then those left together: each turn through memory
      // costs most of a microsecond
      raw8<float> o[4];
      int i = 0;
      for (; i + 3 < splits; i += 4) {
#pragma unroll
        for (int k = 0; k < 4; ++k) load8(o[k], part + at + (i + k) * v_step);
#pragma unroll
        for (int k = 0; k < 4; ++k) add8(v, o[k], true);
      }
      if (i < splits) {
#pragma unroll
        for (int k = 0; k < 3; ++k) load8(o[k], part + at + min(i + k, splits - 1) * v_step);
#pragma unroll
        for (int k = 0; k < 3; ++k) add8(v, o[k], i + k < splits);
      }
      // V itself, where the caller keeps it
      if (V && t.col_wg == 0) store8(V + at, v);
    }
    u32x4 o[3];
    split8(v, o);
    u32x4(*to)[64] = vop[row / 16][r8 / 4];
    const int at = spread_slot<RT>(r8 / 4, r8 & 3, row & 15);
    if constexpr (RT == 1) {
      to[0][at] = o[0];
      to[0][at + 32] = o[1];
      to[1][at] = o[2];
      to[1][at + 32] = u32x4{0u, 0u, 0u, 0u};
    } else {
#pragma unroll
      for (int m = 0; m < 3; ++m) to[m][at] = o[m];
    }
  }
}

// A wave's columns for KS operands of 32 ranks (0: no adapter, Y = Y0).  Y0 and
// Y are reached through buffer resources of the tile's rows, whose range check
// makes zeros of loads, and nothing of stores, past the last row; lanes past the
// last column use an offset outside.  So no branch stands between a load ahead
// and its use, and every wait covers only what it is for.
template <class Y, int RT, int TT, int KS, bool BASE, bool PAST>
__device__ __forceinline__ void spread_columns(const SpreadTile& t, int n, int d, const float* __restrict__ part,
                                               int splits, const bf16_t* __restrict__ factor, const Y* y0,
                                               int64_t ld0, Y* y, int64_t ldy, float* __restrict__ V,
                                               SpreadOps<RT, TT>& vop) {
  constexpr int CW = YRow<Y>::CW, TERMS = RT == 1 ? 2 : 3, F = KS > 0 ? KS : 1, B = sizeof(Y);
  constexpr uint32_t kOutside = 0x80000000u;
  constexpr int kAux = PAST ? 2 : 0;   // the non-temporal bit
  // the factor rows of the next columns too, where the registers hold both
  constexpr bool kAhead = TT == 1 && KS * CW <= 16;
  using raw = typename YRow<Y>::raw;
  using factors = typename YRow<Y>::factors;
  const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
  const int tiles = TT == 1 ? 1 : (t.rows + 15) / 16;
  auto resource = [&](const Y* p, int64_t ld) {
    return __builtin_amdgcn_make_buffer_rsrc(
        const_cast<Y*>(p + t.begin * ld), static_cast<short>(0),
        static_cast<int>(((t.rows - 1) * static_cast<int>(ld) + d) * B), 0x00020000);
  };
  const __amdgpu_buffer_rsrc_t to = resource(y, ldy);
  const __amdgpu_buffer_rsrc_t base = resource(BASE ? y0 : y, BASE ? ld0 : ldy);
  factors fr[F][8];
  auto load_factor = [&](int c0) {
    const int c = min(c0 + CW * j, d - CW);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = RT == 1 ? 8 * (g & 1) + i : 32 * ks + 8 * g + i;
        fr[ks][i] = *reinterpret_cast<const factors*>(factor + static_cast<int64_t>(min(r, t.rank - 1)) * d + c);
      }
  };
  // the lane's byte offset in a row; opaque, since the compiler would make a
  // branch of every access out of the choice
  auto place = [&](int c0) {
    uint32_t p = c0 + CW * j < d ? static_cast<uint32_t>((c0 + CW * j) * B) : kOutside;
    asm("" : "+v"(p));
    return p;
  };
  auto row = [&](int i, int e, int64_t ld) { return static_cast<uint32_t>((16 * i + 4 * g + e) * static_cast<int>(ld) * B); };
  raw in[4];
  auto load_rows = [&](int i, uint32_t at) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      in[e] = BASE ? __builtin_bit_cast(raw, __builtin_amdgcn_raw_buffer_load_b128(base, row(i, e, ld0) + at, 0, kAux))
                   : raw{0, 0, 0, 0};
  };
  int c0 = t.c0;
  load_factor(c0);
  uint32_t at = place(c0);
  load_rows(0, at);
  if (KS > 0 || V) stage_v<RT, TT>(t, n, part, splits, V, vop);
  if (KS > 0) __syncthreads();
  if (c0 >= d) return;
  // everything so far has come (s_waitcnt vmcnt(0)): otherwise the loop's first
  // wait, which all its turns share, would also cover the stores of the turn
  // before
  __builtin_amdgcn_s_waitcnt(0x0F70);
  do {
    if constexpr (TT == 1 && !kAhead) {
      if (c0 != t.c0) load_factor(c0);
    }
    u32x4 w[F][CW];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = RT == 1 ? 8 * (g & 1) + i : 32 * ks + 8 * g + i;
#pragma unroll
        for (int q = 0; q < CW / 2; ++q)
          if (r >= t.rank) fr[ks][i][q] = 0u;
      }
#pragma unroll
      for (int i = 0; i < CW; ++i)
#pragma unroll
        for (int p = 0; p < 4; ++p)
          w[ks][i][p] = __builtin_amdgcn_perm(fr[ks][2 * p + 1][i / 2], fr[ks][2 * p][i / 2],
                                              i & 1 ? 0x07060302u : 0x05040100u);
    }
    const uint32_t now = at;
    if constexpr (TT == 1) {
      c0 += t.stride;
      at = place(c0);
      if constexpr (kAhead) load_factor(c0);
    }
    for (int i = 0; i < tiles; ++i) {
      f32x4 acc[CW];
      YRow<Y> b[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) b[e].v = in[e];
#pragma unroll
      for (int q = 0; q < CW; ++q) acc[q] = f32x4{b[0].at(q), b[1].at(q), b[2].at(q), b[3].at(q)};
      load_rows(TT == 1 ? 0 : i + 1, at);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int m = 0; m < TERMS; ++m) {
          const u32x4 v = vop[i][ks][m][spread_slot<RT>(ks, g, j)];
#pragma unroll
          for (int q = 0; q < CW; ++q) acc[q] = mfma(v, w[ks][q], acc[q]);
        }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float s[CW];
#pragma unroll
        for (int q = 0; q < CW; ++q) s[q] = acc[q][e];
        YRow<Y> o;
        o.put(s);
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, o.v), to, row(i, e, ldy) + now, 0, kAux);
      }
    }
  } while (TT == 1 && c0 < d);
}

// Short requests live on the number of waves: three a SIMD, where the factor's
// operands leave the registers for it (64 requests on 12288 columns: 13.6 against 16.5 us).
template <class Y, int RT, int TT, bool BASE, bool PAST>
__global__ __launch_bounds__(64 * kWaves, TT == 1 && RT * YRow<Y>::CW <= 16 ? 3 : 1) void adapter_spread_kernel(int n, int d, int col_wgs,
                                                                     const float* __restrict__ part, int splits,
                                                                     int nseg, const int* __restrict__ off,
                                                                     const int* __restrict__ ids, int nad,
                                                                     const bf16_t* __restrict__ factor,
                                                                     const int* __restrict__ rank, const Y* y0,
                                                                     int64_t ld0, Y* y, int64_t ldy,
                                                                     float* __restrict__ V) {
  constexpr int R = 16 * RT, T = 16 * TT, KS = (R + 31) / 32, CW = YRow<Y>::CW;
  __shared__ SpreadOps<RT, TT> vop;
  // The column blocks of a tile read the same V: on one XCD (workgroups go to the
  // eight in turn, each has an L2 of its own), eight tiles side by side.  4096 x
  // 4096 at rank 32: 20 against 23 us.  Not where Y goes past the caches: memory
  // wants a row's column blocks side by side (16384 x 17408: 393 against 418 us).
  int number = blockIdx.x / col_wgs, col_wg = blockIdx.x % col_wgs;
  if constexpr (TT > 1 && !PAST) {
    const int turn = blockIdx.x / 8;
    number = turn / col_wgs * 8 + blockIdx.x % 8;
    col_wg = turn % col_wgs;
  }
  const Tile t = find_tile<T>(number, n, nseg, off, ids, nad);
  if (t.begin >= t.end) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rk = t.adapter < 0 ? 0 : min(max(rank[t.adapter], 0), R);
  const SpreadTile st{t.begin, t.end - t.begin, rk, col_wg, (col_wg * kWaves + wave) * 16 * CW,
                      col_wgs * kWaves * 16 * CW};
  const bf16_t* f = factor + static_cast<int64_t>(max(t.adapter, 0)) * R * d;
  if (rk == 0)
    spread_columns<Y, RT, TT, 0, BASE, PAST>(st, n, d, part, splits, f, y0, ld0, y, ldy, V, vop);
  else if (KS > 2 && rk > 64)
    spread_columns<Y, RT, TT, KS, BASE, PAST>(st, n, d, part, splits, f, y0, ld0, y, ldy, V, vop);
  else if (KS > 1 && rk > 32)
    spread_columns<Y, RT, TT, (KS > 2 ? 2 : KS), BASE, PAST>(st, n, d, part, splits, f, y0, ld0, y, ldy, V, vop);
  else
    spread_columns<Y, RT, TT, 1, BASE, PAST>(st, n, d, part, splits, f, y0, ld0, y, ldy, V, vop);
}

// V = the sum of the low kernel's parts, where no spread kernel writes it.
__global__ __launch_bounds__(256) void adapter_sum_kernel(int64_t count, const float* __restrict__ part, int splits,
                                                          float* __restrict__ V) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= count) return;
  float s = part[i];
  for (int p = 1; p < splits; ++p) s += part[p * count + i];
  V[i] = s;
}

// Token tiles of the low kernel: as many rows as the average request fills, so
// that the factor's rows are read once for them; at most 64, 32 at rank 128
// (the sums take 64 registers per lane at either limit).  16384 x 5120 at rank
// 64: 42 us with 64 rows, 58 with 32 or 16; 4096 x 12288 at rank 32: 27 us with
// 64, 29 with 32, 37 with 16.
int low_tiles(int n, int nseg, int rmax) {
  const int avg = n / (nseg > 0 ? nseg : 1);
  const int most = rmax > 64 ? 2 : 4;
  const int want = avg > 32 ? 4 : avg > 16 ? 2 : 1;
  return want < most ? want : most;
}

// Tokens a spread workgroup walks over: 64, so that the factor's operands are
// built once for four tiles (16384 x 17408: 393 us, with 16 tokens 519); 16 where
// requests are short (64 of one token on 12288 columns: 14 us, with 64 tokens 19).
bool short_requests(int n, int nseg) { return n / nseg <= 16; }

// Workgroups along k: three for every compute unit over the whole grid, in one
// round (16384 x 5120, rank 64: 42 us in two parts, 48 in five, 57 in one).  Not
// more than the root of the pieces that k has for them, since every workgroup
// that reads V adds their parts up (low and spread kernel together: one token of
// 4096 in 4 parts 7.8 us, in 9 parts 8.5; 4096 x 12288 at rank 32 in 7 parts 49.6
// us, in 11 parts 51.8, in 3 parts 50.5).
int low_splits(int n, int d, int nseg, int rmax) {
  const int64_t tiles = tile_numbers(n, 16 * low_tiles(n, nseg, rmax), nseg);
  const int pieces = (d + 64 * kWaves - 1) / (64 * kWaves);
  int s = static_cast<int>(768 / tiles), most = 1;
  while (most < s && most * most < pieces) ++most;
  return s < 1 ? 1 : most;
}

template <class X, int RT>
void low_by_tiles(int tt, int splits, int n, int d, const void* x, int64_t ldx, int nseg, const int* off,
                  const int* ids, int nad, const void* factor, const int* rank, const float* alpha, float* part,
                  const ListJob& job, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(tile_numbers(n, 16 * tt, nseg) + job.on), splits);
  auto k = adapter_low_kernel<X, RT, 1>;
  if (tt == 2) k = adapter_low_kernel<X, RT, 2>;
  if (tt == 4) k = adapter_low_kernel<X, RT, RT == 8 ? 2 : 4>;
  hipLaunchKernelGGL(k, grid, dim3(64 * kWaves), 0, s, n, d, static_cast<const X*>(x), ldx, nseg, off, ids, nad,
                     static_cast<const bf16_t*>(factor), rank, alpha, part, job);
}

template <class X>
void low(int n, int d, const void* x, int64_t ldx, int nseg, const int* off, const int* ids, int nad, int rmax,
         const void* factor, const int* rank, const float* alpha, float* part, const ListJob& job, hipStream_t s) {
  auto f = rmax == 16 ? low_by_tiles<X, 1> : rmax == 32 ? low_by_tiles<X, 2> : rmax == 64 ? low_by_tiles<X, 4>
                                                                                         : low_by_tiles<X, 8>;
  f(low_tiles(n, nseg, rmax), low_splits(n, d, nseg, rmax), n, d, x, ldx, nseg, off, ids, nad, factor, rank, alpha,
    part, job, s);
}

template <class Y, int RT>
void spread_by_tiles(bool one, int n, int d, const float* part, int splits, int nseg, const int* off, const int* ids,
                     int nad, const void* factor, const int* rank, const void* y0, int64_t ld0, void* y, int64_t ldy,
                     float* V, hipStream_t s) {
  const int cols = 16 * YRow<Y>::CW * kWaves, tokens = one ? 16 : 64;
  // short requests: a workgroup takes several column blocks in turn, so that
  // the three that fit every compute unit do it all in one round
  const int64_t tiles = tile_numbers(n, tokens, nseg);
  const int all = (d + cols - 1) / cols, few = tiles < 768 ? static_cast<int>(768 / tiles) : 1;
  const int col_wgs = one && few < all ? few : all;
  // Y beyond the 256 MB of the last-level cache goes past the caches, which keep
  // the inputs of the next call instead (16384 x 17408 fp32: 437 against 459 us
  // for both kernels)
  const bool far = static_cast<int64_t>(n) * d * static_cast<int64_t>(sizeof(Y)) > (int64_t{256} << 20);
  const dim3 grid(static_cast<unsigned>(col_wgs * (one || far ? tiles : (tiles + 7) / 8 * 8)));
  auto k = one ? (y0 ? adapter_spread_kernel<Y, RT, 1, true, false> : adapter_spread_kernel<Y, RT, 1, false, false>)
           : far ? (y0 ? adapter_spread_kernel<Y, RT, 4, true, true> : adapter_spread_kernel<Y, RT, 4, false, true>)
                 : (y0 ? adapter_spread_kernel<Y, RT, 4, true, false> : adapter_spread_kernel<Y, RT, 4, false, false>);
  hipLaunchKernelGGL(k, grid, dim3(64 * kWaves), 0, s, n, d, col_wgs, part, splits, nseg, off, ids, nad,
                     static_cast<const bf16_t*>(factor), rank, static_cast<const Y*>(y0), ld0, static_cast<Y*>(y), ldy,
                     V);
}

template <class Y>
void spread(int n, int d, const float* part, int splits, int nseg, const int* off, const int* ids, int nad, int rmax,
            const void* factor, const int* rank, const void* y0, int64_t ld0, void* y, int64_t ldy, float* V,
            hipStream_t s) {
  auto f = rmax == 16 ? spread_by_tiles<Y, 1> : rmax == 32 ? spread_by_tiles<Y, 2>
                                              : rmax == 64 ? spread_by_tiles<Y, 4> : spread_by_tiles<Y, 8>;
  f(short_requests(n, nseg), n, d, part, splits, nseg, off, ids, nad, factor, rank, y0, ld0, y, ldy, V, s);
}

bool rank_ok(int rmax) { return rmax == 16 || rmax == 32 || rmax == 64 || rmax == 128; }

size_t part_bytes(int n, int d, int nseg, int rmax) {
  return static_cast<size_t>(low_splits(n, d, nseg, rmax)) * n * rmax * sizeof(float);
}

size_t round256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }

constexpr int kMaxSeg = 1 << 20;
constexpr int kMaxTokens = 1 << 24;   // so that sums over 64 requests stay in 32 bits
// Row strides: the 64 rows of a workgroup stay below 2^31 bytes.
constexpr int64_t kMaxStride = 1 << 22;

// X as the grad kernel sees it: the two float types and the act8 codes.
constexpr int kAct8 = 2;

wush_status check(const char* who, wush_dtype a, wush_dtype b, wush_dtype c, int n, int d_in, int d_out, int nseg,
                  int nad, int rmax) {
  for (wush_dtype t : {a, b, c})
    if (t != WUSH_F32 && t != WUSH_BF16) return fail(WUSH_E_ARG, "%s: bad dtype", who);
  if (n < 0 || n > kMaxTokens || d_in < 8 || d_in % 8 || d_out < 8 || d_out % 8)
    return fail(WUSH_E_SHAPE, "%s: need n in 0..%d and d_in, d_out positive multiples of 8 (n=%d d_in=%d d_out=%d)", who,
                kMaxTokens, n, d_in, d_out);
  if (!rank_ok(rmax)) return fail(WUSH_E_SHAPE, "%s: rmax must be 16, 32, 64 or 128 (got %d)", who, rmax);
  if (nad < 1 || nseg < 1 || nseg > kMaxSeg)
    return fail(WUSH_E_SHAPE, "%s: need at least one adapter and 1..%d requests (nad=%d nseg=%d)", who, kMaxSeg, nad, nseg);
  // short requests launch no more workgroups than they have tiles (or 768)
  const int64_t d = d_in > d_out ? d_in : d_out;
  if (!short_requests(n, nseg) && (tile_numbers(n, 64, nseg) + 7) * ((d + 255) / 256) >= (int64_t{1} << 32) / (64 * kWaves))
    return fail(WUSH_E_SHAPE, "%s: n=%d with nseg=%d passes the launch limit", who, n, nseg);
  return WUSH_OK;
}

wush_status launched(const char* who) {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? WUSH_OK : fail(WUSH_E_HIP, "%s launch: %s", who, hipGetErrorString(e));
}

}  // namespace

extern "C" size_t wush_adapter_ws_bytes(int n, int d_in, int nseg, int rmax) {
  if (n < 1 || n > kMaxTokens || d_in < 8 || d_in % 8 || nseg < 1 || nseg > kMaxSeg || !rank_ok(rmax)) return 0;
  return part_bytes(n, d_in, nseg, rmax);
}

extern "C" wush_status wush_adapter_forward(wush_dtype xdt, wush_dtype ydt, int n, int d_in, int d_out, const void* X,
                                            int64_t ldx, int nseg, const int* seg_off, const int* seg_adapter, int nad,
                                            int rmax, const void* A, const void* Bt, const int* rank,
                                            const float* alpha, const void* Y0, int64_t ldy0, void* Y, int64_t ldy,
                                            float* V, void* ws, size_t ws_bytes, void* stream) {
  const char* who = "wush_adapter_forward";
  const wush_status st = check(who, xdt, ydt, ydt, n, d_in, d_out, nseg, nad, rmax);
  if (st != WUSH_OK) return st;
  if (ldx < d_in || ldx % 8 || ldy < d_out || ldy % 8 || (Y0 && (ldy0 < d_out || ldy0 % 8)))
    return fail(WUSH_E_SHAPE, "%s: row strides must be multiples of 8, at least the row's length", who);
  if (ldx > kMaxStride || ldy > kMaxStride || (Y0 && ldy0 > kMaxStride))
    return fail(WUSH_E_SHAPE, "%s: row strides above %lld values", who, static_cast<long long>(kMaxStride));
  if (n == 0) return WUSH_OK;
  if (!X || !seg_off || !seg_adapter || !A || !Bt || !rank || !alpha || !Y) return fail(WUSH_E_ARG, "%s: null pointer", who);
  for (const void* p : {X, A, Bt, Y0, static_cast<const void*>(Y), static_cast<const void*>(V), static_cast<const void*>(ws)})
    if (!aligned16(p)) return fail(WUSH_E_ARG, "%s: pointers must be 16-byte aligned", who);
  const size_t need = part_bytes(n, d_in, nseg, rmax);
  if (ws && ws_bytes < need) return fail(WUSH_E_ARG, "%s: workspace of %zu bytes, need %zu", who, ws_bytes, need);
  hipStream_t s = static_cast<hipStream_t>(stream);
  float* part = static_cast<float*>(ws);
  if (!ws) {
    const hipError_t e = hipMallocAsync(reinterpret_cast<void**>(&part), need, s);
    if (e != hipSuccess) return fail(WUSH_E_HIP, "%s: scratch: %s", who, hipGetErrorString(e));
  }
  auto f = xdt == WUSH_F32 ? low<float> : low<bf16_t>;
  f(n, d_in, X, ldx, nseg, seg_off, seg_adapter, nad, rmax, A, rank, alpha, part, ListJob{}, s);
  wush_status out = launched(who);
  if (out == WUSH_OK) {
    auto g = ydt == WUSH_F32 ? spread<float> : spread<bf16_t>;
    g(n, d_out, part, low_splits(n, d_in, nseg, rmax), nseg, seg_off, seg_adapter, nad, rmax, Bt, rank, Y0, ldy0, Y,
      ldy, V, s);
    out = launched(who);
  }
  if (!ws) (void)hipFreeAsync(part, s);
  return out;
}

extern "C" size_t wush_adapter_backward_ws_bytes(int n, int d_in, int d_out, int nseg, int nad, int rmax) {
  if (n < 0 || n > kMaxTokens || d_in < 8 || d_in % 8 || d_out < 8 || d_out % 8 || nseg < 1 || nseg > kMaxSeg || nad < 1 || !rank_ok(rmax))
    return 0;
  return round256(part_bytes(n, d_out, nseg, rmax)) + round256(static_cast<size_t>(n) * rmax * sizeof(float)) +
         adapter_grads_ws_bytes(n, d_in, d_out, nseg, nad, rmax);
}

extern "C" wush_status wush_adapter_backward(wush_dtype gdt, wush_dtype xdt, wush_dtype ydt, int n, int d_in, int d_out,
                                             const void* dY, int64_t ldg, const void* X, const uint8_t* x_scales,
                                             int64_t ldx, int nseg, const int* seg_off, const int* seg_adapter,
                                             int nad, int rmax, const void* A, const void* Bt, const int* rank,
                                             const float* alpha, const float* V, const void* dX0, int64_t lddx0,
                                             void* dX, int64_t lddx, float* dA, float* dBt, void* ws, size_t ws_bytes,
                                             void* stream) {
  const char* who = "wush_adapter_backward";
  const wush_status st = check(who, gdt, xdt, ydt, n, d_in, d_out, nseg, nad, rmax);
  if (st != WUSH_OK) return st;
  if (ldg < d_out || ldg % 8 || ldx < d_in || ldx % 8 || (dX && (lddx < d_in || lddx % 8)) ||
      (dX && dX0 && (lddx0 < d_in || lddx0 % 8)))
    return fail(WUSH_E_SHAPE, "%s: row strides must be multiples of 8, at least the row's length", who);
  if (ldg > kMaxStride || (dX && (lddx > kMaxStride || (dX0 && lddx0 > kMaxStride))))
    return fail(WUSH_E_SHAPE, "%s: row strides above %lld values", who, static_cast<long long>(kMaxStride));
  if (!adapter_grads_fit(n, d_in, d_out, nad, rmax)) return fail(WUSH_E_SHAPE, "%s: nad=%d passes the launch limit", who, nad);
  if (x_scales && (d_in % 32 || ldx != d_in))
    return fail(WUSH_E_SHAPE, "%s: an act8 checkpoint has whole groups of 32 and no row stride of its own", who);
  if (!seg_off || !seg_adapter || !A || !Bt || !rank || !alpha || !dA || !dBt || (n > 0 && (!dY || !X || !V)))
    return fail(WUSH_E_ARG, "%s: null pointer", who);
  for (const void* p : {dY, X, A, Bt, static_cast<const void*>(V), dX0, static_cast<const void*>(dX),
                        static_cast<const void*>(dA), static_cast<const void*>(dBt), static_cast<const void*>(ws)})
    if (!aligned16(p)) return fail(WUSH_E_ARG, "%s: pointers must be 16-byte aligned", who);
  const size_t need = wush_adapter_backward_ws_bytes(n, d_in, d_out, nseg, nad, rmax);
  if (ws && ws_bytes < need) return fail(WUSH_E_ARG, "%s: workspace of %zu bytes, need %zu", who, ws_bytes, need);
  hipStream_t s = static_cast<hipStream_t>(stream);
  void* base = ws;
  if (!ws) {
    const hipError_t e = hipMallocAsync(&base, need, s);
    if (e != hipSuccess) return fail(WUSH_E_HIP, "%s: scratch: %s", who, hipGetErrorString(e));
  }
  float* part = static_cast<float*>(base);
  float* dV = reinterpret_cast<float*>(static_cast<char*>(base) + round256(part_bytes(n, d_out, nseg, rmax)));
  char* rest = reinterpret_cast<char*>(dV) + round256(static_cast<size_t>(n) * rmax * sizeof(float));
  const int splits = low_splits(n, d_out, nseg, rmax);
  wush_status out = WUSH_OK;
  if (n > 0) {
    auto f = gdt == WUSH_F32 ? low<float> : low<bf16_t>;
    f(n, d_out, dY, ldg, nseg, seg_off, seg_adapter, nad, rmax, Bt, rank, alpha, part,
      adapter_lists(n, d_in, d_out, nseg, nad, rmax, rest), s);
    out = launched(who);
    if (out == WUSH_OK && dX) {
      auto g = ydt == WUSH_F32 ? spread<float> : spread<bf16_t>;
      g(n, d_in, part, splits, nseg, seg_off, seg_adapter, nad, rmax, A, rank, dX0, lddx0, dX, lddx, dV, s);
      out = launched(who);
    } else if (out == WUSH_OK) {
      const int64_t count = static_cast<int64_t>(n) * rmax;
      hipLaunchKernelGGL(adapter_sum_kernel, dim3(static_cast<unsigned>((count + 255) / 256)), dim3(256), 0, s, count,
                         part, splits, dV);
      out = launched(who);
    }
  }
  if (out == WUSH_OK)
    out = adapter_grads(who, gdt, x_scales ? kAct8 : static_cast<int>(xdt), n, d_in, d_out, dY, ldg, X, x_scales, ldx,
                        nseg, seg_off, seg_adapter, nad, rmax, rank, V, dV, dA, dBt, rest, s);
  if (!ws) (void)hipFreeAsync(base, s);
  return out;
}
