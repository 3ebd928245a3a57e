// act8: activations kept in 8 bits for the backward pass.
//
// One checkpoint holds 32 consecutive values of a row as int8 codes q under
// one power-of-two scale byte, the E8M0 convention of the MXFP4 scales:
//   a = max|x|, e = clamp(floor(log2 a), -120, 127), byte e + 127,
//   q = clamp(rint(x 2^(6-e)), -127, 127), value q 2^(e-6).
// The scaling and the read-back are exact (power of two), so the only rounding
// is the one to the nearest code, and every value is a bf16 number (seven
// significant bits): a matrix product reads a checkpoint without a further
// rounding.  A group with a NaN or an infinity gets byte 0xFF and zero codes
// and reads back as NaN, as the other formats' blocks do.
//
// All four kernels move bytes and do little else.  A wave owns a 512-value piece
// of a row, so that rows of any length lose at most part of one wave.  A lane
// holds eight of its values: eight neighbours where everything is bf16 (16 bytes
// an access), two runs of four where something is fp32, so that each access of
// the wave covers whole lines either way; a group is then four or eight
// neighbouring lanes, and its maximum takes two or three DPP steps.  Results
// that a later pass reads are written past the caches where they are larger
// than those (non-temporal stores).
//
// Gated activation on 16384 x 17408, fp32 in, bf16 and both checkpoints out: 597
// us, 5.8 TB/s; its backward, bf16 in, fp32 out: 581 us, 5.9 TB/s.  A copy of 1
// GiB moves 5.0 TB/s here.  Storing 4099 x 5120 in bf16 takes 12 us and reading
// back 12 us, 5.3 TB/s.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "common.h"
#include "vec.h"

using namespace wush;

namespace {

constexpr int kWaves = 4;   // per workgroup

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return __builtin_amdgcn_update_dpp(0u, v, CTRL, 0xf, 0xf, true);
}

// N neighbouring values of a row, as fp32.
template <class T, int N>
struct Run;
template <>
struct Run<float, 4> {
  f32x4 r;
  __device__ __forceinline__ void load(const float* p) { r = *reinterpret_cast<const f32x4*>(p); }
  __device__ __forceinline__ void widen(float* v) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = r[i];
  }
};
template <>
struct Run<bf16_t, 4> {
  u32x2 r;
  __device__ __forceinline__ void load(const bf16_t* p) { r = *reinterpret_cast<const u32x2*>(p); }
  __device__ __forceinline__ void widen(float* v) const {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = __builtin_bit_cast(float, i & 1 ? r[i / 2] & 0xffff0000u : r[i / 2] << 16);
  }
};
template <>
struct Run<bf16_t, 8> {
  raw8<bf16_t> r;
  __device__ __forceinline__ void load(const bf16_t* p) { load8(r, p); }
  __device__ __forceinline__ void widen(float* v) const { widen8(r, v); }
};

template <bool PAST, class V>
__device__ __forceinline__ void put(V v, V* p) {
  if constexpr (PAST)
    __builtin_nontemporal_store(v, p);
  else
    *p = v;
}

template <bool PAST, int N>
__device__ __forceinline__ void put_run(float* p, const float* v) {
  static_assert(N == 4, "fp32 runs are 16 bytes");
  put<PAST>(f32x4{v[0], v[1], v[2], v[3]}, reinterpret_cast<f32x4*>(p));
}
template <bool PAST, int N>
__device__ __forceinline__ void put_run(bf16_t* p, const float* v) {
  if constexpr (N == 4)
    put<PAST>(u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])}, reinterpret_cast<u32x2*>(p));
  else
    put<PAST>(u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])},
              reinterpret_cast<u32x4*>(p));
}

template <int N>
struct Codes {
  uint32_t q[N / 4];
  uint32_t byte;
};

// Codes of the lane's N values and its group's scale byte.
template <int N>
__device__ __forceinline__ Codes<N> encode(const float* v) {
  // |x| as bits: integer order is the order of magnitudes, and NaN and
  // infinities are those from 0x7f800000 on
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) a = max(a, __builtin_bit_cast(uint32_t, v[i]) & 0x7fffffffu);
  a = max(a, dpp<0xB1>(a));    // lanes 1 0 3 2
  a = max(a, dpp<0x4E>(a));    // lanes 2 3 0 1
  if constexpr (N == 4) a = max(a, dpp<0x141>(a));   // lanes 7 6 5 4 3 2 1 0
  const bool bad = a >= 0x7f800000u;
  const uint32_t byte = max(a >> 23, 7u);   // e + 127
  const float m = __builtin_bit_cast(float, (260u - byte) << 23);   // 2^(6-e)
  // adding 1.5 * 2^23 rounds to the nearest integer (ties to even) and leaves
  // its two's complement in the low bits; x m is exact inside the fma
  constexpr float kRound = 12582912.0f;
  uint32_t b[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float r = __builtin_fmaf(v[i], m, kRound);
    b[i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_fmed3f(r, kRound - 127.0f, kRound + 127.0f));
  }
  Codes<N> c;
#pragma unroll
  for (int h = 0; h < N / 4; ++h) {
    const uint32_t lo = __builtin_amdgcn_perm(b[4 * h + 1], b[4 * h], 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(b[4 * h + 3], b[4 * h + 2], 0x04000c0cu);
    c.q[h] = bad ? 0u : lo | hi;
  }
  c.byte = bad ? 255u : byte;
  return c;
}

template <int N>
__device__ __forceinline__ void decode(const Codes<N>& c, float* v) {
  // 2^(e-6); bytes below 7 do not occur in a checkpoint and read as zero
  const uint32_t s = c.byte == 255u ? 0x7fc00000u : (max(c.byte, 6u) - 6u) << 23;
  const float m = __builtin_bit_cast(float, s);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = static_cast<float>(static_cast<int8_t>(c.q[i / 4] >> (8 * (i & 3)))) * m;
}

// The wave's row and the lane's runs of N columns; a run may lie past the end.
template <int N>
struct Place {
  static constexpr int kRuns = 8 / N;
  int64_t row;
  int col[kRuns];
  bool in[kRuns];
};
template <int N>
__device__ __forceinline__ Place<N> place(int64_t n, int d, int per_row) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t piece = static_cast<int64_t>(blockIdx.x) * kWaves + wave;
  Place<N> p;
  p.row = piece / per_row;
#pragma unroll
  for (int r = 0; r < Place<N>::kRuns; ++r) {
    p.col[r] = static_cast<int>(piece - p.row * per_row) * 512 + r * 64 * N + (threadIdx.x & 63) * N;
    p.in[r] = p.row < n && p.col[r] < d;
  }
  return p;
}

template <int N>
__device__ __forceinline__ void put_codes(const Codes<N>& c, int64_t row, int col, int d, uint8_t* codes,
                                          uint8_t* scales) {
  if constexpr (N == 4)
    *reinterpret_cast<uint32_t*>(codes + row * d + col) = c.q[0];
  else
    *reinterpret_cast<u32x2*>(codes + row * d + col) = u32x2{c.q[0], c.q[1]};
  if ((threadIdx.x & (32 / N - 1)) == 0) scales[row * (d / 32) + col / 32] = static_cast<uint8_t>(c.byte);
}

template <int N>
__device__ __forceinline__ void get_codes(int64_t row, int col, int d, const uint8_t* codes, const uint8_t* scales,
                                          Codes<N>& c) {
  if constexpr (N == 4) {
    c.q[0] = *reinterpret_cast<const uint32_t*>(codes + row * d + col);
  } else {
    const u32x2 q = *reinterpret_cast<const u32x2*>(codes + row * d + col);
    c.q[0] = q[0];
    c.q[1] = q[1];
  }
  c.byte = scales[row * (d / 32) + col / 32];
}

// Values per run: eight bf16 values or four fp32 ones fill a lane's 16 bytes.
// Eight fp32 values a lane, two accesses that each skip every other 16 bytes,
// took 1272 instead of 1226 us on 16384 x 17408, forward and backward, with all
// outputs through the caches.
template <class A, class B>
constexpr int run_of = is_f32<A> || is_f32<B> ? 4 : 8;

template <class T, int N = run_of<T, T>>
__global__ __launch_bounds__(64 * kWaves) void act8_pack_kernel(int64_t n, int d, int per_row, const T* __restrict__ X,
                                                                uint8_t* __restrict__ codes,
                                                                uint8_t* __restrict__ scales) {
  const auto p = place<N>(n, d, per_row);
  Run<T, N> x[p.kRuns];
#pragma unroll
  for (int r = 0; r < p.kRuns; ++r)
    if (p.in[r]) x[r].load(X + p.row * d + p.col[r]);
#pragma unroll
  for (int r = 0; r < p.kRuns; ++r) {
    if (!p.in[r]) continue;
    float v[N];
    x[r].widen(v);
    put_codes<N>(encode<N>(v), p.row, p.col[r], d, codes, scales);
  }
}

template <class T, bool PAST, int N = run_of<T, T>>
__global__ __launch_bounds__(64 * kWaves) void act8_unpack_kernel(int64_t n, int d, int per_row,
                                                                  const uint8_t* __restrict__ codes,
                                                                  const uint8_t* __restrict__ scales,
                                                                  T* __restrict__ Y) {
  const auto p = place<N>(n, d, per_row);
  Codes<N> c[p.kRuns];
#pragma unroll
  for (int r = 0; r < p.kRuns; ++r)
    if (p.in[r]) get_codes<N>(p.row, p.col[r], d, codes, scales, c[r]);
#pragma unroll
  for (int r = 0; r < p.kRuns; ++r) {
    if (!p.in[r]) continue;
    float v[N];
    decode<N>(c[r], v);
    put_run<PAST, N>(Y + p.row * d + p.col[r], v);
  }
}

// 1 / (1 + exp(-x)) on the transcendental unit.  For positive x 1 to 2 ulp.  For
// negative x the rounding of 1.44 x shows: some |x| ulp (4 at -5, 15 at -16), and
// below -88 the result, at most 1e-38, becomes zero.  Splitting the product in two
// would remove it; results that are kept as bf16 or 8-bit codes do not see it.
__device__ __forceinline__ float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504088896341f * x));
}

template <class T, class H, bool KEEP, bool PAST, int N = run_of<T, H>>
__global__ __launch_bounds__(64 * kWaves) void act8_swiglu_kernel(int64_t n, int d, int per_row,
                                                                  const T* __restrict__ G, const T* __restrict__ U,
                                                                  int64_t ld, H* __restrict__ out,
                                                                  uint8_t* __restrict__ gc, uint8_t* __restrict__ gs,
                                                                  uint8_t* __restrict__ uc, uint8_t* __restrict__ us) {
  const auto p = place<N>(n, d, per_row);
  Run<T, N> rg[p.kRuns], ru[p.kRuns];
#pragma unroll
  for (int r = 0; r < p.kRuns; ++r)
    if (p.in[r]) {
      rg[r].load(G + p.row * ld + p.col[r]);
      ru[r].load(U + p.row * ld + p.col[r]);
    }
#pragma unroll
  for (int r = 0; r < p.kRuns; ++r) {
    if (!p.in[r]) continue;
    float g[N], u[N], h[N];
    rg[r].widen(g);
    ru[r].widen(u);
#pragma unroll
    for (int i = 0; i < N; ++i) h[i] = g[i] * sigmoid(g[i]) * u[i];
    put_run<PAST, N>(out + p.row * d + p.col[r], h);
    if (KEEP) {
      put_codes<N>(encode<N>(g), p.row, p.col[r], d, gc, gs);
      put_codes<N>(encode<N>(u), p.row, p.col[r], d, uc, us);
    }
  }
}

// With s = sigmoid(g): dU = dH g s, dG = dH u s (1 + g (1 - s)).
template <class H, class T, bool PAST, int N = run_of<T, H>>
__global__ __launch_bounds__(64 * kWaves) void act8_swiglu_bwd_kernel(
    int64_t n, int d, int per_row, const H* __restrict__ dH, const uint8_t* __restrict__ gc,
    const uint8_t* __restrict__ gs, const uint8_t* __restrict__ uc, const uint8_t* __restrict__ us,
    T* __restrict__ dG, T* __restrict__ dU, int64_t ld) {
  const auto p = place<N>(n, d, per_row);
  Run<H, N> rh[p.kRuns];
  Codes<N> cg[p.kRuns], cu[p.kRuns];
#pragma unroll
  for (int r = 0; r < p.kRuns; ++r)
    if (p.in[r]) {
      rh[r].load(dH + p.row * d + p.col[r]);
      get_codes<N>(p.row, p.col[r], d, gc, gs, cg[r]);
      get_codes<N>(p.row, p.col[r], d, uc, us, cu[r]);
    }
#pragma unroll
  for (int r = 0; r < p.kRuns; ++r) {
    if (!p.in[r]) continue;
    float dh[N], g[N], u[N];
    rh[r].widen(dh);
    decode<N>(cg[r], g);
    decode<N>(cu[r], u);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float s = sigmoid(g[i]), hs = dh[i] * s;
      u[i] = hs * u[i] * __builtin_fmaf(g[i], 1.0f - s, 1.0f);
      g[i] = hs * g[i];
    }
    put_run<PAST, N>(dG + p.row * ld + p.col[r], u);
    put_run<PAST, N>(dU + p.row * ld + p.col[r], g);
  }
}

// Columns are counted in 31 bits, to the end of a row's last piece.
constexpr int kMaxD = 0x7fffffff - 511;

int per_row(int d) { return (d + 511) / 512; }

// Whether an output of n x d values passes the 256 MB of the last-level cache:
// then it is written past the caches, which keeps them for the inputs (16384 x
// 17408, forward and backward: 1183 against 1226 us).
bool past(int n, int d, wush_dtype t) {
  return static_cast<int64_t>(n) * d * (t == WUSH_F32 ? 4 : 2) > (int64_t{256} << 20);
}

// Workgroups of n rows, 0 if they pass the launch limit of 2^32 threads.
unsigned blocks(int n, int d) {
  const int64_t b = (static_cast<int64_t>(n) * per_row(d) + kWaves - 1) / kWaves;
  return b < (int64_t{1} << 32) / (64 * kWaves) ? static_cast<unsigned>(b) : 0u;
}

wush_status check(const char* who, wush_dtype a, wush_dtype b, int n, int d) {
  if ((a != WUSH_F32 && a != WUSH_BF16) || (b != WUSH_F32 && b != WUSH_BF16))
    return fail(WUSH_E_ARG, "%s: bad dtype", who);
  if (n < 0 || d < 32 || d % 32 || d > kMaxD)
    return fail(WUSH_E_SHAPE, "%s: need n >= 0 and d a multiple of 32 in 32..%d (n=%d d=%d)", who, kMaxD, n, d);
  if (n > 0 && blocks(n, d) == 0) return fail(WUSH_E_SHAPE, "%s: n=%d d=%d passes the launch limit", who, n, d);
  return WUSH_OK;
}

wush_status launched(const char* who) {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? WUSH_OK : fail(WUSH_E_HIP, "%s launch: %s", who, hipGetErrorString(e));
}

}  // namespace

extern "C" wush_status wush_act8_pack(wush_dtype xdt, int n, int d, const void* X, int8_t* codes, uint8_t* scales,
                                      void* stream) {
  const wush_status st = check("wush_act8_pack", xdt, xdt, n, d);
  if (st != WUSH_OK) return st;
  if (n == 0) return WUSH_OK;
  if (!X || !codes || !scales) return fail(WUSH_E_ARG, "wush_act8_pack: null pointer");
  if (!aligned16(X) || !aligned16(codes)) return fail(WUSH_E_ARG, "wush_act8_pack: X and codes must be 16-byte aligned");
  hipStream_t s = static_cast<hipStream_t>(stream);
  uint8_t* c = reinterpret_cast<uint8_t*>(codes);
  const dim3 grid(blocks(n, d)), wg(64 * kWaves);
  if (xdt == WUSH_F32)
    hipLaunchKernelGGL(act8_pack_kernel<float>, grid, wg, 0, s, n, d, per_row(d), static_cast<const float*>(X), c, scales);
  else
    hipLaunchKernelGGL(act8_pack_kernel<bf16_t>, grid, wg, 0, s, n, d, per_row(d), static_cast<const bf16_t*>(X), c, scales);
  return launched("wush_act8_pack");
}

extern "C" wush_status wush_act8_unpack(wush_dtype ydt, int n, int d, const int8_t* codes, const uint8_t* scales,
                                        void* Y, void* stream) {
  const wush_status st = check("wush_act8_unpack", ydt, ydt, n, d);
  if (st != WUSH_OK) return st;
  if (n == 0) return WUSH_OK;
  if (!Y || !codes || !scales) return fail(WUSH_E_ARG, "wush_act8_unpack: null pointer");
  if (!aligned16(Y) || !aligned16(codes)) return fail(WUSH_E_ARG, "wush_act8_unpack: Y and codes must be 16-byte aligned");
  hipStream_t s = static_cast<hipStream_t>(stream);
  const uint8_t* c = reinterpret_cast<const uint8_t*>(codes);
  const dim3 grid(blocks(n, d)), wg(64 * kWaves);
  const bool far = past(n, d, ydt);
  if (ydt == WUSH_F32)
    hipLaunchKernelGGL((far ? act8_unpack_kernel<float, true> : act8_unpack_kernel<float, false>), grid, wg, 0, s, n, d, per_row(d), c, scales, static_cast<float*>(Y));
  else
    hipLaunchKernelGGL((far ? act8_unpack_kernel<bf16_t, true> : act8_unpack_kernel<bf16_t, false>), grid, wg, 0, s, n, d, per_row(d), c, scales, static_cast<bf16_t*>(Y));
  return launched("wush_act8_unpack");
}

namespace {

template <class T, class H>
void swiglu(bool keep, int n, int d, const void* G, const void* U, int64_t ld, void* out, uint8_t* gc, uint8_t* gs,
            uint8_t* uc, uint8_t* us, hipStream_t s) {
  const dim3 grid(blocks(n, d)), wg(64 * kWaves);
  const bool far = past(n, d, is_f32<H> ? WUSH_F32 : WUSH_BF16);
  auto k = keep ? (far ? act8_swiglu_kernel<T, H, true, true> : act8_swiglu_kernel<T, H, true, false>)
                : (far ? act8_swiglu_kernel<T, H, false, true> : act8_swiglu_kernel<T, H, false, false>);
  hipLaunchKernelGGL(k, grid, wg, 0, s, n, d, per_row(d), static_cast<const T*>(G), static_cast<const T*>(U), ld,
                     static_cast<H*>(out), gc, gs, uc, us);
}

template <class H, class T>
void swiglu_bwd(int n, int d, const void* dH, const uint8_t* gc, const uint8_t* gs, const uint8_t* uc,
                const uint8_t* us, void* dG, void* dU, int64_t ld, hipStream_t s) {
  const dim3 grid(blocks(n, d)), wg(64 * kWaves);
  const bool far = past(n, d, is_f32<T> ? WUSH_F32 : WUSH_BF16);
  hipLaunchKernelGGL((far ? act8_swiglu_bwd_kernel<H, T, true> : act8_swiglu_bwd_kernel<H, T, false>), grid, wg, 0, s, n, d, per_row(d), static_cast<const H*>(dH), gc,
                     gs, uc, us, static_cast<T*>(dG), static_cast<T*>(dU), ld);
}

}  // namespace

extern "C" wush_status wush_act8_swiglu(wush_dtype xdt, wush_dtype hdt, int n, int d, const void* G, const void* U,
                                        int64_t ld, void* H, int8_t* g_codes, uint8_t* g_scales, int8_t* u_codes,
                                        uint8_t* u_scales, void* stream) {
  const wush_status st = check("wush_act8_swiglu", xdt, hdt, n, d);
  if (st != WUSH_OK) return st;
  if (ld < d || ld % 8) return fail(WUSH_E_SHAPE, "wush_act8_swiglu: the row stride must be a multiple of 8, at least d");
  if (n == 0) return WUSH_OK;
  if (!G || !U || !H) return fail(WUSH_E_ARG, "wush_act8_swiglu: null pointer");
  const bool keep = g_codes != nullptr;
  if (keep != (g_scales != nullptr) || keep != (u_codes != nullptr) || keep != (u_scales != nullptr))
    return fail(WUSH_E_ARG, "wush_act8_swiglu: the four checkpoint pointers are given together or not at all");
  if (!aligned16(G) || !aligned16(U) || !aligned16(H) || !aligned16(g_codes) || !aligned16(u_codes))
    return fail(WUSH_E_ARG, "wush_act8_swiglu: G, U, H and the codes must be 16-byte aligned");
  hipStream_t s = static_cast<hipStream_t>(stream);
  auto f = xdt == WUSH_F32 ? (hdt == WUSH_F32 ? swiglu<float, float> : swiglu<float, bf16_t>)
                           : (hdt == WUSH_F32 ? swiglu<bf16_t, float> : swiglu<bf16_t, bf16_t>);
  f(keep, n, d, G, U, ld, H, reinterpret_cast<uint8_t*>(g_codes), g_scales, reinterpret_cast<uint8_t*>(u_codes),
    u_scales, s);
  return launched("wush_act8_swiglu");
}

extern "C" wush_status wush_act8_swiglu_bwd(wush_dtype hdt, wush_dtype xdt, int n, int d, const void* dH,
                                            const int8_t* g_codes, const uint8_t* g_scales, const int8_t* u_codes,
                                            const uint8_t* u_scales, void* dG, void* dU, int64_t ld, void* stream) {
  const wush_status st = check("wush_act8_swiglu_bwd", xdt, hdt, n, d);
  if (st != WUSH_OK) return st;
  if (ld < d || ld % 8)
    return fail(WUSH_E_SHAPE, "wush_act8_swiglu_bwd: the row stride must be a multiple of 8, at least d");
  if (n == 0) return WUSH_OK;
  if (!dH || !g_codes || !g_scales || !u_codes || !u_scales || !dG || !dU)
    return fail(WUSH_E_ARG, "wush_act8_swiglu_bwd: null pointer");
  if (!aligned16(dH) || !aligned16(dG) || !aligned16(dU) || !aligned16(g_codes) || !aligned16(u_codes))
    return fail(WUSH_E_ARG, "wush_act8_swiglu_bwd: dH, dG, dU and the codes must be 16-byte aligned");
  hipStream_t s = static_cast<hipStream_t>(stream);
  auto f = hdt == WUSH_F32 ? (xdt == WUSH_F32 ? swiglu_bwd<float, float> : swiglu_bwd<float, bf16_t>)
                           : (xdt == WUSH_F32 ? swiglu_bwd<bf16_t, float> : swiglu_bwd<bf16_t, bf16_t>);
  f(n, d, dH, reinterpret_cast<const uint8_t*>(g_codes), g_scales, reinterpret_cast<const uint8_t*>(u_codes), u_scales,
    dG, dU, ld, s);
  return launched("wush_act8_swiglu_bwd");
}
