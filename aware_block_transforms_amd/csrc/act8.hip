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
// All four kernels move bytes and do little else.  A lane owns eight values, a
// group is four neighbouring lanes (its maximum takes two DPP steps), and a
// wave one 512-value piece of a row, so that rows of any length lose at most
// part of one wave.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "common.h"
#include "vec.h"

using namespace wush;

namespace {

constexpr int kWaves = 4;   // per workgroup

template <int CTRL>
__device__ __forceinline__ uint32_t quad(uint32_t v) {
  return __builtin_amdgcn_update_dpp(0u, v, CTRL, 0xf, 0xf, true);
}

struct Codes {
  u32x2 q;
  uint32_t byte;
};

// Codes of the lane's eight values and the group's scale byte.
__device__ __forceinline__ Codes encode(const float* v) {
  // |x| as bits: integer order is the order of magnitudes, and NaN and
  // infinities are those from 0x7f800000 on
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = max(a, __builtin_bit_cast(uint32_t, v[i]) & 0x7fffffffu);
  a = max(a, quad<0xB1>(a));   // lanes 1 0 3 2
  a = max(a, quad<0x4E>(a));   // lanes 2 3 0 1
  const bool bad = a >= 0x7f800000u;
  const uint32_t byte = max(a >> 23, 7u);   // e + 127
  const float m = __builtin_bit_cast(float, (260u - byte) << 23);   // 2^(6-e)
  // adding 1.5 * 2^23 rounds to the nearest integer (ties to even) and leaves
  // its two's complement in the low bits; x m is exact inside the fma
  constexpr float kRound = 12582912.0f;
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float r = __builtin_fmaf(v[i], m, kRound);
    b[i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_fmed3f(r, kRound - 127.0f, kRound + 127.0f));
  }
  Codes c;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = __builtin_amdgcn_perm(b[4 * h + 1], b[4 * h], 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(b[4 * h + 3], b[4 * h + 2], 0x04000c0cu);
    c.q[h] = bad ? 0u : lo | hi;
  }
  c.byte = bad ? 255u : byte;
  return c;
}

__device__ __forceinline__ void decode(u32x2 q, uint32_t byte, float* v) {
  // 2^(e-6); bytes below 7 do not occur in a checkpoint and read as zero
  const uint32_t s = byte == 255u ? 0x7fc00000u : (max(byte, 6u) - 6u) << 23;
  const float m = __builtin_bit_cast(float, s);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = static_cast<float>(static_cast<int8_t>(q[i / 4] >> (8 * (i & 3)))) * m;
}

// The wave's row and the lane's first column; false past the end.
struct Place {
  int64_t row;
  int col;
};
__device__ __forceinline__ bool place(int64_t n, int d, int per_row, Place& p) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t piece = static_cast<int64_t>(blockIdx.x) * kWaves + wave;
  p.row = piece / per_row;
  p.col = static_cast<int>(piece - p.row * per_row) * 512 + (threadIdx.x & 63) * 8;
  return p.row < n && p.col < d;
}

__device__ __forceinline__ void put_codes(const Codes& c, const Place& p, int d, uint8_t* codes, uint8_t* scales) {
  *reinterpret_cast<u32x2*>(codes + p.row * d + p.col) = c.q;
  if ((threadIdx.x & 3) == 0) scales[p.row * (d / 32) + p.col / 32] = static_cast<uint8_t>(c.byte);
}

__device__ __forceinline__ void get_codes(const Place& p, int d, const uint8_t* codes, const uint8_t* scales, u32x2& q,
                                          uint32_t& byte) {
  q = *reinterpret_cast<const u32x2*>(codes + p.row * d + p.col);
  byte = scales[p.row * (d / 32) + p.col / 32];
}

template <class T>
__global__ __launch_bounds__(64 * kWaves) void act8_pack_kernel(int64_t n, int d, int per_row, const T* __restrict__ X,
                                                                uint8_t* __restrict__ codes,
                                                                uint8_t* __restrict__ scales) {
  Place p;
  if (!place(n, d, per_row, p)) return;
  raw8<T> r;
  load8(r, X + p.row * d + p.col);
  float v[8];
  widen8(r, v);
  put_codes(encode(v), p, d, codes, scales);
}

template <class T>
__global__ __launch_bounds__(64 * kWaves) void act8_unpack_kernel(int64_t n, int d, int per_row,
                                                                  const uint8_t* __restrict__ codes,
                                                                  const uint8_t* __restrict__ scales,
                                                                  T* __restrict__ Y) {
  Place p;
  if (!place(n, d, per_row, p)) return;
  u32x2 q;
  uint32_t byte;
  get_codes(p, d, codes, scales, q, byte);
  float v[8];
  decode(q, byte, v);
  store8(Y + p.row * d + p.col, v);
}

// 1 / (1 + exp(-x)) on the transcendental unit: 1 to 2 ulp where it matters
// (for x below -20 the relative error grows with |x|, on values below 1e-8).
__device__ __forceinline__ float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504088896341f * x));
}

template <class T, class H, bool KEEP>
__global__ __launch_bounds__(64 * kWaves) void act8_swiglu_kernel(int64_t n, int d, int per_row,
                                                                  const T* __restrict__ G, const T* __restrict__ U,
                                                                  int64_t ld, H* __restrict__ out,
                                                                  uint8_t* __restrict__ gc, uint8_t* __restrict__ gs,
                                                                  uint8_t* __restrict__ uc, uint8_t* __restrict__ us) {
  Place p;
  if (!place(n, d, per_row, p)) return;
  raw8<T> rg, ru;
  load8(rg, G + p.row * ld + p.col);
  load8(ru, U + p.row * ld + p.col);
  float g[8], u[8], h[8];
  widen8(rg, g);
  widen8(ru, u);
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = g[i] * sigmoid(g[i]) * u[i];
  store8(out + p.row * d + p.col, h);
  if (KEEP) {
    put_codes(encode(g), p, d, gc, gs);
    put_codes(encode(u), p, d, uc, us);
  }
}

// With s = sigmoid(g): dU = dH g s, dG = dH u s (1 + g (1 - s)).
template <class H, class T>
__global__ __launch_bounds__(64 * kWaves) void act8_swiglu_bwd_kernel(
    int64_t n, int d, int per_row, const H* __restrict__ dH, const uint8_t* __restrict__ gc,
    const uint8_t* __restrict__ gs, const uint8_t* __restrict__ uc, const uint8_t* __restrict__ us,
    T* __restrict__ dG, T* __restrict__ dU, int64_t ld) {
  Place p;
  if (!place(n, d, per_row, p)) return;
  raw8<H> rh;
  u32x2 qg, qu;
  uint32_t bg, bu;
  load8(rh, dH + p.row * d + p.col);
  get_codes(p, d, gc, gs, qg, bg);
  get_codes(p, d, uc, us, qu, bu);
  float dh[8], g[8], u[8];
  widen8(rh, dh);
  decode(qg, bg, g);
  decode(qu, bu, u);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float s = sigmoid(g[i]), hs = dh[i] * s;
    u[i] = hs * u[i] * __builtin_fmaf(g[i], 1.0f - s, 1.0f);
    g[i] = hs * g[i];
  }
  store8(dG + p.row * ld + p.col, u);
  store8(dU + p.row * ld + p.col, g);
}

int per_row(int d) { return (d + 511) / 512; }

// Workgroups of n rows, 0 if they pass the launch limit.
unsigned blocks(int n, int d) {
  const int64_t b = (static_cast<int64_t>(n) * per_row(d) + kWaves - 1) / kWaves;
  return b <= 0x7fffffff ? static_cast<unsigned>(b) : 0u;
}

wush_status check(const char* who, wush_dtype a, wush_dtype b, int n, int d) {
  if ((a != WUSH_F32 && a != WUSH_BF16) || (b != WUSH_F32 && b != WUSH_BF16))
    return fail(WUSH_E_ARG, "%s: bad dtype", who);
  if (n < 0 || d < 32 || d % 32) return fail(WUSH_E_SHAPE, "%s: need n >= 0 and d a positive multiple of 32 (n=%d d=%d)", who, n, d);
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
  if (ydt == WUSH_F32)
    hipLaunchKernelGGL(act8_unpack_kernel<float>, grid, wg, 0, s, n, d, per_row(d), c, scales, static_cast<float*>(Y));
  else
    hipLaunchKernelGGL(act8_unpack_kernel<bf16_t>, grid, wg, 0, s, n, d, per_row(d), c, scales, static_cast<bf16_t*>(Y));
  return launched("wush_act8_unpack");
}

namespace {

template <class T, class H>
void swiglu(bool keep, int n, int d, const void* G, const void* U, int64_t ld, void* out, uint8_t* gc, uint8_t* gs,
            uint8_t* uc, uint8_t* us, hipStream_t s) {
  const dim3 grid(blocks(n, d)), wg(64 * kWaves);
  auto k = keep ? act8_swiglu_kernel<T, H, true> : act8_swiglu_kernel<T, H, false>;
  hipLaunchKernelGGL(k, grid, wg, 0, s, n, d, per_row(d), static_cast<const T*>(G), static_cast<const T*>(U), ld,
                     static_cast<H*>(out), gc, gs, uc, us);
}

template <class H, class T>
void swiglu_bwd(int n, int d, const void* dH, const uint8_t* gc, const uint8_t* gs, const uint8_t* uc,
                const uint8_t* us, void* dG, void* dU, int64_t ld, hipStream_t s) {
  const dim3 grid(blocks(n, d)), wg(64 * kWaves);
  hipLaunchKernelGGL((act8_swiglu_bwd_kernel<H, T>), grid, wg, 0, s, n, d, per_row(d), static_cast<const H*>(dH), gc,
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
