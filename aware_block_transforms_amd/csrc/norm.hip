// Block norm: what stands between two blocks of a model, in one pass.
//
// Per token, with y the block's output and r the residual stream:
//   b  = y rsqrt(mean(y^2) + eps) * w_post * gate      (norm after the block)
//   r' = res r + branch b                              (gate and residual scale)
//   u  = r' rsqrt(mean(r'^2) + eps) * w_pre            (norm before the next)
// The gate is absent, one value per channel, per token or per element.  u is
// computed from r' before r' is rounded to its storage type.
//
// Backward, with k1, k2 the two rsqrt values kept by the forward call, and y
// and r' as stored:
//   x  = k2 r',  q = dU w_pre,   t = dR' + k2 (q - x mean(q x)),   dw_pre = sum dU x
//   z  = k1 y,   g = branch t,   dgate = g z w_post,               dw_post = sum g gate z
//   p  = g gate w_post,          dY = k1 (p - z mean(p z)),        dR = res t
// All sums are fp32.
//
// Both directions read and write every value once, and large calls up to 8192
// columns are bound by HBM.  Forward on 16384 x 5120, y fp32, the rest bf16: 151
// us, 5.5 TB/s.  Backward on 4096 x 4096: 50 us and 5 us for the column sums, 4.9
// TB/s; a copy of 256 MB moves 5.4 TB/s here, one of 1 GiB 5.0.  One row of 4096 takes 3.2 us, a turn
// through memory for the loads, one for the weights, and the launch.  A
// workgroup owns a row, a thread VPT pieces of eight values of it, which stay
// in registers between the two means.  In the backward kernel a workgroup
// walks over rows and keeps its columns' weight gradients in registers; the
// workgroups' sums are written once and added in a fixed order by a second
// kernel, so results do not depend on scheduling.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "common.h"
#include "vec.h"

using namespace wush;

namespace {

// Sum of each of N values over the workgroup, in every thread; `slot` holds 16
// floats per value and is not reused before the next barrier but one.
template <int N>
__device__ __forceinline__ void block_sums(float* v, float* slot) {
  const int wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if (waves == 1) return;
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) slot[i * 16 + wave] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float s = 0.0f;
    for (int w = 0; w < waves; ++w) s += slot[i * 16 + w];
    v[i] = s;
  }
}

__device__ __forceinline__ void load_weights(const float* w, int col, float* v) {
  raw8<float> r;
  load8(r, w + col);
  widen8(r, v);
}

struct NormArgs {
  int n, d;
  const float* w_post;
  const float* w_pre;
  const void* gate;
  float branch, res, eps;
  float* k1;
  float* k2;
};

// Stores of eight values, past the caches where PAST.
template <bool PAST>
__device__ __forceinline__ void put8(float* p, const float* v) {
  store8(p, v);   // two halves of lines: left to the caches to join
}
template <bool PAST>
__device__ __forceinline__ void put8(bf16_t* p, const float* v) {
  if constexpr (PAST)
    __builtin_nontemporal_store(
        u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])},
        reinterpret_cast<u32x4*>(p));
  else
    store8(p, v);
}

template <class Y, class R, class U, int VPT, bool PAST>
__global__ __launch_bounds__(1024) void norm_fwd_kernel(NormArgs a, int gate_kind, const Y* __restrict__ y,
                                                        const R* r, R* rout, U* __restrict__ u) {
  __shared__ float slots[2][16];
  const int64_t row = blockIdx.x, base = row * a.d;
  raw8<Y> ry[VPT];
  raw8<R> rr[VPT];
  raw8<Y> rg[VPT];
  int col[VPT];
  bool in[VPT];
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    col[v] = (v * blockDim.x + threadIdx.x) * 8;
    in[v] = col[v] < a.d;
    if (in[v]) {
      if (y) load8(ry[v], y + base + col[v]);
      load8(rr[v], r + base + col[v]);
      if (gate_kind == WUSH_GATE_ELEMENT) load8(rg[v], static_cast<const Y*>(a.gate) + base + col[v]);
    }
  }
  float x[VPT][8];
  float k1 = 1.0f;
  if (y) {
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      if (!in[v]) continue;
      widen8(ry[v], x[v]);
#pragma unroll
      for (int i = 0; i < 8; ++i) s = __builtin_fmaf(x[v][i], x[v][i], s);
    }
    if (a.w_post) {
      block_sums<1>(&s, slots[0]);
      k1 = 1.0f / __builtin_sqrtf(s / a.d + a.eps);
      if (a.k1 && threadIdx.x == 0) a.k1[row] = k1;
    }
  }
  float scale = a.branch * k1;
  if (gate_kind == WUSH_GATE_TOKEN) scale *= static_cast<const float*>(a.gate)[row];
  float s = 0.0f;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    if (!in[v]) continue;
    float t[8];
    widen8(rr[v], t);
    if (y) {
      float w[8];
      if (a.w_post) {
        load_weights(a.w_post, col[v], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[v][i] *= w[i];
      }
      if (gate_kind == WUSH_GATE_CHANNEL) {
        load_weights(static_cast<const float*>(a.gate), col[v], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[v][i] *= w[i];
      } else if (gate_kind == WUSH_GATE_ELEMENT) {
        widen8(rg[v], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[v][i] *= w[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) x[v][i] = __builtin_fmaf(x[v][i], scale, a.res * t[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[v][i] = a.res * t[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) s = __builtin_fmaf(x[v][i], x[v][i], s);
    if (rout) put8<PAST>(rout + base + col[v], x[v]);
  }
  if (!a.w_pre) return;
  block_sums<1>(&s, slots[1]);
  const float k2 = 1.0f / __builtin_sqrtf(s / a.d + a.eps);
  if (a.k2 && threadIdx.x == 0) a.k2[row] = k2;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    if (!in[v]) continue;
    float w[8];
    load_weights(a.w_pre, col[v], w);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] *= x[v][i] * k2;
    put8<PAST>(u + base + col[v], w);
  }
}

// Partial column sums of one workgroup: [3][d] (dw_pre, dw_post, dgate).  A
// thread owns eight columns of rows up to 8 MAXT.  The next row is loaded, into
// a second buffer, before the sums over the one in hand.  Loads return in order,
// so nothing may be loaded and waited for in between: the weights lie in LDS,
// the two rsqrt values come through the scalar cache, threads past the last
// column read the last columns again, and tensors that the caller left out are
// read as one that is there and replaced by zeros, not skipped by a branch.
// Where a branch or a weight load cut the row's loads off, 4096 x 4096 took 71 us
// against 59 with as many workgroups.  Five variants of 1024 threads with an fp32
// r spill 12 to 40 bytes a lane (rows of 4104 to 8192 columns; 4096 x 8192 with bf16 r 114
// us, a copy 100).  What the threads past the last column
// would add to a row's sums is dropped by a select on the sum: a factor of zero
// would make NaN of a row whose gradient holds an infinity there.
template <class Y, class R, class U, int MAXT, int GATE>
__global__ __launch_bounds__(MAXT) void norm_bwd_kernel(NormArgs a, const float* __restrict__ k1s,
                                                        const float* __restrict__ k2s, const U* __restrict__ du,
                                                        const R* drout, bool has_drout, const Y* __restrict__ y,
                                                        bool has_y, const R* __restrict__ rout, Y* __restrict__ dy,
                                                        R* dr, void* __restrict__ dgate, float* __restrict__ part) {
  constexpr bool CHANNEL = GATE == WUSH_GATE_CHANNEL, ELEMENT = GATE == WUSH_GATE_ELEMENT;
  __shared__ float slots[2][2 * 16];
  __shared__ f32x4 weights[CHANNEL ? 3 : 2][MAXT][2];
  const int me = threadIdx.x, col = min(8 * me, a.d - 8);
  const bool in = 8 * me < a.d, has_pre = a.w_pre != nullptr, has_post = a.w_post != nullptr;
  auto keep = [&](int which, const float* from, float otherwise) {
    f32x4 w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      w[h] = from ? reinterpret_cast<const f32x4*>(from + col)[h] : f32x4{otherwise, otherwise, otherwise, otherwise};
      weights[which][me][h] = w[h];
    }
  };
  keep(0, a.w_pre, 0.0f);
  keep(1, a.w_post, 1.0f);
  if constexpr (CHANNEL) keep(2, static_cast<const float*>(a.gate), 1.0f);
  // no barrier: a thread reads what it wrote itself
  auto weight = [&](int which, float* v) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x4 w = weights[which][me][h];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * h + i] = w[i];
    }
  };
  float s_pre[8], s_post[8], s_gate[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) s_pre[i] = s_post[i] = s_gate[i] = 0.0f;
  const float inv_d = 1.0f / a.d;
  struct Row {
    raw8<U> u;
    raw8<R> r, d;
    raw8<Y> y, g;
  };
  auto load = [&](Row& to, int64_t row) {
    const int64_t at = row * a.d + col;
    load8(to.u, du + at);
    load8(to.r, rout + at);
    load8(to.d, drout + at);
    load8(to.y, y + at);
    if constexpr (ELEMENT) load8(to.g, static_cast<const Y*>(a.gate) + at);
  };
  auto process = [&](const Row& now, int64_t row) {
    const int64_t at = row * a.d + col;
    const float k1 = has_post ? k1s[row] : 1.0f, k2 = has_pre ? k2s[row] : 0.0f;
    float q[8], x[8], w[8], m = 0.0f;
    widen8(now.u, q);
    widen8(now.r, x);
    weight(0, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = has_pre ? x[i] * k2 : 0.0f;
      q[i] = has_pre ? q[i] : 0.0f;
      s_pre[i] = __builtin_fmaf(q[i], x[i], s_pre[i]);
      q[i] *= w[i];
      m = __builtin_fmaf(q[i], x[i], m);
    }
    m = in ? m : 0.0f;
    block_sums<1>(&m, slots[0]);
    m *= inv_d;
    float t[8], z[8], g[8], o[8], sums[2] = {0.0f, 0.0f};   // p z, and the token gate's gradient
    widen8(now.d, t);
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = __builtin_fmaf(k2, __builtin_fmaf(-x[i], m, q[i]), has_drout ? t[i] : 0.0f);
    if (dr && in) {
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = a.res * t[i];
      store8(dr + at, o);
    }
    if (!has_y) {
      __syncthreads();   // slots[0] is read before the next row writes it
      return;
    }
    const float gate_t = GATE == WUSH_GATE_TOKEN && a.gate ? static_cast<const float*>(a.gate)[row] : 1.0f;
    widen8(now.y, z);
    weight(1, w);
    if constexpr (CHANNEL)
      weight(2, g);
    else if constexpr (ELEMENT)
      widen8(now.g, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (!CHANNEL && !ELEMENT) g[i] = gate_t;
      const float h = a.branch * t[i];
      z[i] *= k1;
      const float hz = h * z[i];
      o[i] = hz * w[i];
      if (CHANNEL) s_gate[i] += o[i];
      sums[1] += o[i];
      s_post[i] = __builtin_fmaf(hz, g[i], s_post[i]);
      t[i] = h * g[i] * w[i];   // p
      sums[0] = __builtin_fmaf(t[i], z[i], sums[0]);
    }
    if constexpr (ELEMENT)
      if (in) store8(static_cast<Y*>(dgate) + at, o);
    sums[0] = in ? sums[0] : 0.0f;
    sums[1] = in ? sums[1] : 0.0f;
    block_sums<2>(sums, slots[1]);
    if (GATE == WUSH_GATE_TOKEN && dgate && me == 0) static_cast<float*>(dgate)[row] = sums[1];
    // without a norm after the block dY is p itself
    const float mz = has_post ? sums[0] * inv_d : 0.0f;
    if (in) {
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = k1 * __builtin_fmaf(-z[i], mz, t[i]);
      store8(dy + at, o);
    }
  };
  // two buffers in turn; past the last row the last one is loaded again
  const int64_t last = a.n - 1, step = gridDim.x;
  int64_t row = blockIdx.x;
  Row p, q;
  load(p, row);
  for (;;) {
    load(q, min(row + step, last));
    process(p, row);
    if ((row += step) > last) break;
    load(p, min(row + step, last));
    process(q, row);
    if ((row += step) > last) break;
  }
  if (!in) return;
  float* out = part + static_cast<int64_t>(blockIdx.x) * 3 * a.d + col;
  if (has_pre) store8(out, s_pre);
  if (has_y && has_post) store8(out + a.d, s_post);
  if (CHANNEL) store8(out + 2 * a.d, s_gate);
}

// The same for rows above 8192 columns, VPT pieces a thread.  A row stays in
// registers as it lies in memory and is widened where it is used.  Even so every
// variant spills, 84 to 276 bytes a lane with two pieces and 380 to 808 with four;
// nor is a row loaded ahead.  That is what bounds it: 4096 x 12288, y fp32, the
// rest bf16, 326 us, 4096 x 16384 387 and 4096 x 17408 795, where a copy of the
// bytes takes 151, 203 and 223.
template <class Y, class R, class U, int VPT, int MAXT, int GATE>
__global__ __launch_bounds__(MAXT) void norm_bwd_wide_kernel(NormArgs a, const U* __restrict__ du,
                                                        const R* drout, const Y* __restrict__ y,
                                                        const R* __restrict__ rout, Y* __restrict__ dy, R* dr,
                                                        void* __restrict__ dgate, float* __restrict__ part) {
  constexpr bool CHANNEL = GATE == WUSH_GATE_CHANNEL, ELEMENT = GATE == WUSH_GATE_ELEMENT;
  __shared__ float slots[2][2 * 16];
  int col[VPT];
  bool in[VPT];
  float s_pre[VPT][8], s_post[VPT][8], s_gate[CHANNEL ? VPT : 1][8];
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    col[v] = (v * blockDim.x + threadIdx.x) * 8;
    in[v] = col[v] < a.d;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s_pre[v][i] = s_post[v][i] = 0.0f;
      if (CHANNEL) s_gate[v][i] = 0.0f;
    }
  }
  const float inv_d = 1.0f / a.d;
  struct Row {
    raw8<Y> y[VPT], g[ELEMENT ? VPT : 1];
    raw8<R> r[VPT], d[VPT];
    raw8<U> u[VPT];
  };
  auto load = [&](Row& to, int64_t row) {
    const int64_t base = row * a.d;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      if (!in[v]) continue;
      if (a.w_pre) {
        load8(to.u[v], du + base + col[v]);
        load8(to.r[v], rout + base + col[v]);
      }
      if (drout) load8(to.d[v], drout + base + col[v]);
      if (y) load8(to.y[v], y + base + col[v]);
      if (ELEMENT) load8(to.g[v], static_cast<const Y*>(a.gate) + base + col[v]);
    }
  };
  auto process = [&](const Row& in_row, int64_t row) {
    const auto& [ry, rg, rr, rd, ru] = in_row;
    const int64_t base = row * a.d;
    const float k1 = y && a.w_post ? a.k1[row] : 1.0f;
    const float k2 = a.w_pre ? a.k2[row] : 0.0f;
    float m = 0.0f;
    if (a.w_pre) {
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        if (!in[v]) continue;
        float w[8], q[8], x[8];
        widen8(ru[v], q);
        widen8(rr[v], x);
        load_weights(a.w_pre, col[v], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float qx = q[i] * (x[i] * k2);
          s_pre[v][i] += qx;
          m = __builtin_fmaf(qx, w[i], m);
        }
      }
      block_sums<1>(&m, slots[0]);
      m *= inv_d;
    }
    float sums[2] = {0.0f, 0.0f};   // p z, and the token gate's gradient
    float p[VPT][8];
    const float gate_t = GATE == WUSH_GATE_TOKEN && a.gate ? static_cast<const float*>(a.gate)[row] : 1.0f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      if (!in[v]) continue;
      float t[8], w[8], o[8];
      if (drout) {
        widen8(rd[v], t);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = 0.0f;
      }
      if (a.w_pre) {
        float q[8], x[8];
        widen8(ru[v], q);
        widen8(rr[v], x);
        load_weights(a.w_pre, col[v], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = __builtin_fmaf(k2, __builtin_fmaf(-x[i] * k2, m, q[i] * w[i]), t[i]);
      }
      if (dr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = a.res * t[i];
        store8(dr + base + col[v], o);
      }
      if (!y) continue;
      float z[8], g[8];
      widen8(ry[v], z);
      if (a.w_post) {
        load_weights(a.w_post, col[v], w);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = 1.0f;
      }
      if (CHANNEL) {
        load_weights(static_cast<const float*>(a.gate), col[v], g);
      } else if (ELEMENT) {
        widen8(rg[v], g);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = gate_t;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float h = a.branch * t[i];
        z[i] *= k1;
        const float hz = h * z[i], dg = hz * w[i];
        o[i] = dg;
        if (CHANNEL) s_gate[v][i] += dg;
        sums[1] += dg;
        s_post[v][i] = __builtin_fmaf(hz, g[i], s_post[v][i]);
        p[v][i] = h * g[i] * w[i];
        sums[0] = __builtin_fmaf(p[v][i], z[i], sums[0]);
      }
      if (ELEMENT) store8(static_cast<Y*>(dgate) + base + col[v], o);
    }
    if (!y) {
      if (a.w_pre) __syncthreads();   // slots[0] is read before the next row writes it
      return;
    }
    block_sums<2>(sums, slots[1]);
    if (GATE == WUSH_GATE_TOKEN && dgate && threadIdx.x == 0) static_cast<float*>(dgate)[row] = sums[1];
    // without a norm after the block dY is p itself
    const float mz = a.w_post ? k1 * sums[0] * inv_d : 0.0f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      if (!in[v]) continue;
      float z[8];
      widen8(ry[v], z);
#pragma unroll
      for (int i = 0; i < 8; ++i) p[v][i] = k1 * __builtin_fmaf(-z[i], mz, p[v][i]);
      store8(dy + base + col[v], p[v]);
    }
    if (!a.w_pre) __syncthreads();   // slots[1] likewise, where one barrier a row is all there is
  };
  for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
    Row p;
    load(p, row);
    process(p, row);
  }
  float* out = part + static_cast<int64_t>(blockIdx.x) * 3 * a.d;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    if (!in[v]) continue;
    if (a.w_pre) store8(out + col[v], s_pre[v]);
    if (y && a.w_post) store8(out + a.d + col[v], s_post[v]);
    if (CHANNEL) store8(out + 2 * a.d + col[v], s_gate[v]);
  }
}

// Adds the workgroups' column sums: 64 columns a workgroup.  A wave reads four
// partials at a time (16 lanes 256 bytes of each), its 16 waves every 64th.
__global__ __launch_bounds__(1024) void norm_cols_kernel(int d, int parts, const float* __restrict__ part,
                                                         float* __restrict__ dw_pre, float* __restrict__ dw_post,
                                                         float* __restrict__ dgate) {
  __shared__ f32x4 sh[16][16];
  float* out = blockIdx.y == 0 ? dw_pre : blockIdx.y == 1 ? dw_post : dgate;
  if (!out) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, j = lane & 15, c = blockIdx.x * 64 + 4 * j;
  f32x4 s{0.0f, 0.0f, 0.0f, 0.0f};
  if (c < d) {
#pragma unroll 4
    for (int i = 4 * wave + (lane >> 4); i < parts; i += 64)
      s += *reinterpret_cast<const f32x4*>(part + (static_cast<int64_t>(i) * 3 + blockIdx.y) * d + c);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    s[k] += __shfl_xor(s[k], 16, 64);
    s[k] += __shfl_xor(s[k], 32, 64);
  }
  if (lane < 16) sh[wave][j] = s;
  __syncthreads();
  if (wave != 0 || lane >= 16 || c >= d) return;
  s = sh[0][j];
#pragma unroll
  for (int w = 1; w < 16; ++w) s += sh[w][j];
  *reinterpret_cast<f32x4*>(out + c) = s;
}

constexpr int kMaxD = 24576;

// Pieces of eight values per thread of the forward kernel.  Few rows: one, up to
// 8192 columns, since only the number of waves hides latency there.  Many: two,
// whose loads are in flight together, four past 16384 columns.  One against two
// pieces in us, y fp32, the rest bf16, at 1, 256, 512, 1024 and 2048 rows: 4096
// columns 3.2/3.9, 4.1/4.7, 5.1/5.6, 8.5/8.4, 16.0/14.5; 5120 columns 3.6/4.1,
// 4.7/5.2, 6.2/6.3, 12.1/10.0, 20.2/19.8; 8192 columns 4.0/4.1, 5.7/5.7, 9.0/8.4,
// 17.3/14.7, 28.8/27.3.  16384 rows of 5120: 171/156.
int fwd_vpt(int n, int d) { return n < 512 && d <= 8192 ? 1 : d <= 16384 ? 2 : 4; }

// The backward kernel's: one up to 8192 columns.  Wider rows take more per
// thread, and so many registers that only twelve waves (of 168) fit beyond 16384.
int bwd_vpt(int d) { return d <= 8192 ? 1 : d <= 16384 ? 2 : 4; }

int threads(int d, int vpt) {
  const int per = 8 * vpt * 64;
  return 64 * ((d + per - 1) / per);
}

// Workgroups of the backward kernel: one for each of the 256 compute units, or
// eight waves of narrow rows.  Twice as many fit, but write twice the column
// sums (4096 x 4096: 55 against 59 us, 1021 x 2600 in fp32: 24 against 28).
int bwd_groups(int n, int d) {
  const int waves = threads(d, bwd_vpt(d)) / 64;
  const int fit = 256 * (waves > 8 ? 1 : 8 / waves);
  return n < fit ? n : fit;
}

wush_status check(const char* who, wush_dtype ydt, wush_dtype rdt, wush_dtype udt, int n, int d, wush_gate gate_kind,
                  const void* Y, const void* gate, const float* w_post, const float* w_pre, float branch, float res) {
  for (wush_dtype t : {ydt, rdt, udt})
    if (t != WUSH_F32 && t != WUSH_BF16) return fail(WUSH_E_ARG, "%s: bad dtype", who);
  if (rdt == WUSH_BF16 && udt == WUSH_F32)
    return fail(WUSH_E_UNSUPPORTED, "%s: an fp32 norm output beside a bf16 residual", who);
  if (n < 0 || d < 8 || d % 8 || d > kMaxD)
    return fail(WUSH_E_SHAPE, "%s: need n >= 0 and d a multiple of 8 in 8..%d (n=%d d=%d)", who, kMaxD, n, d);
  if (gate_kind < WUSH_GATE_NONE || gate_kind > WUSH_GATE_ELEMENT) return fail(WUSH_E_ARG, "%s: bad gate kind", who);
  if (n == 0) return WUSH_OK;   // an empty tensor may have no address
  if ((gate_kind != WUSH_GATE_NONE) != (gate != nullptr)) return fail(WUSH_E_ARG, "%s: a gate needs its kind and its pointer", who);
  if (!Y && (gate || w_post)) return fail(WUSH_E_ARG, "%s: w_post and the gate need Y", who);
  if (!Y && !w_pre) return fail(WUSH_E_ARG, "%s: nothing to do without Y and w_pre", who);
  if (!__builtin_isfinite(branch) || !__builtin_isfinite(res)) return fail(WUSH_E_ARG, "%s: scales must be finite", who);
  return WUSH_OK;
}

template <class F>
wush_status by_types(wush_dtype ydt, wush_dtype rdt, wush_dtype udt, F f) {
  const bool y = ydt == WUSH_F32, r = rdt == WUSH_F32, u = udt == WUSH_F32;
  if (y) {
    if (r) return u ? f(float(), float(), float()) : f(float(), float(), bf16_t());
    return f(float(), bf16_t(), bf16_t());
  }
  if (r) return u ? f(bf16_t(), float(), float()) : f(bf16_t(), float(), bf16_t());
  return f(bf16_t(), bf16_t(), bf16_t());
}

wush_status launched(const char* who) {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? WUSH_OK : fail(WUSH_E_HIP, "%s launch: %s", who, hipGetErrorString(e));
}

}  // namespace

extern "C" wush_status wush_block_norm(wush_dtype ydt, wush_dtype rdt, wush_dtype udt, int n, int d, const void* Y,
                                       const float* w_post, wush_gate gate_kind, const void* gate, float branch_scale,
                                       const void* R, float res_scale, const float* w_pre, float eps, void* Rout,
                                       void* U, float* rstd_post, float* rstd_pre, void* stream) {
  const char* who = "wush_block_norm";
  const wush_status st =
      check(who, ydt, rdt, udt, n, d, gate_kind, Y, gate, w_post, w_pre, branch_scale, res_scale);
  if (st != WUSH_OK) return st;
  if (!(eps > 0.0f) || !__builtin_isfinite(eps)) return fail(WUSH_E_ARG, "%s: eps must be positive and finite", who);
  if (n == 0) return WUSH_OK;
  if (static_cast<int64_t>(n) * threads(d, fwd_vpt(n, d)) >= int64_t{1} << 32)
    return fail(WUSH_E_SHAPE, "%s: n=%d d=%d passes the launch limit", who, n, d);
  if ((w_pre != nullptr) != (U != nullptr)) return fail(WUSH_E_ARG, "%s: w_pre and U are given together", who);
  if (!R || (!U && !Rout)) return fail(WUSH_E_ARG, "%s: null pointer", who);
  for (const void* p : {Y, static_cast<const void*>(w_post), R, static_cast<const void*>(w_pre),
                        static_cast<const void*>(Rout), static_cast<const void*>(U)})
    if (!aligned16(p)) return fail(WUSH_E_ARG, "%s: pointers must be 16-byte aligned", who);
  if (!aligned16(gate) && gate_kind != WUSH_GATE_TOKEN) return fail(WUSH_E_ARG, "%s: pointers must be 16-byte aligned", who);
  const NormArgs a{n, d, w_post, w_pre, gate, branch_scale, res_scale, eps, rstd_post, rstd_pre};
  hipStream_t s = static_cast<hipStream_t>(stream);
  return by_types(ydt, rdt, udt, [&](auto y, auto r, auto u) {
    using YT = decltype(y);
    using RT = decltype(r);
    using UT = decltype(u);
    const int vpt = fwd_vpt(n, d);
    // outputs beyond the 256 MB of the last-level cache are written past it
    // (16384 x 5120, both in bf16: 150 against 157 us)
    const int64_t out = static_cast<int64_t>(n) * d * ((Rout ? sizeof(RT) : 0) + (U ? sizeof(UT) : 0));
    const bool far = out > (int64_t{256} << 20);
    auto k = vpt == 1   ? norm_fwd_kernel<YT, RT, UT, 1, false>
             : vpt == 2 ? (far ? norm_fwd_kernel<YT, RT, UT, 2, true> : norm_fwd_kernel<YT, RT, UT, 2, false>)
                        : (far ? norm_fwd_kernel<YT, RT, UT, 4, true> : norm_fwd_kernel<YT, RT, UT, 4, false>);
    hipLaunchKernelGGL(k, dim3(n), dim3(threads(d, vpt)), 0, s, a, static_cast<int>(gate_kind), static_cast<const YT*>(Y),
                       static_cast<const RT*>(R), static_cast<RT*>(Rout), static_cast<UT*>(U));
    return launched(who);
  });
}

extern "C" size_t wush_block_norm_bwd_ws_bytes(int n, int d) {
  if (n < 1 || d < 8 || d % 8 || d > kMaxD) return 0;
  return static_cast<size_t>(bwd_groups(n, d)) * 3 * d * sizeof(float);
}

extern "C" wush_status wush_block_norm_bwd(wush_dtype ydt, wush_dtype rdt, wush_dtype udt, int n, int d,
                                           const void* dU, const void* dRout, const void* Y, const float* w_post,
                                           wush_gate gate_kind, const void* gate, float branch_scale, const void* Rout,
                                           float res_scale, const float* w_pre, const float* rstd_post,
                                           const float* rstd_pre, void* dY, void* dR, void* dgate, float* dw_post,
                                           float* dw_pre, void* ws, size_t ws_bytes, void* stream) {
  const char* who = "wush_block_norm_bwd";
  const wush_status st =
      check(who, ydt, rdt, udt, n, d, gate_kind, Y, gate, w_post, w_pre, branch_scale, res_scale);
  if (st != WUSH_OK) return st;
  if (n > 0) {
    if ((w_pre != nullptr) != (dU != nullptr) || (w_pre != nullptr) != (dw_pre != nullptr))
      return fail(WUSH_E_ARG, "%s: w_pre, dU and dw_pre are given together", who);
    if ((w_post != nullptr) != (dw_post != nullptr)) return fail(WUSH_E_ARG, "%s: w_post and dw_post are given together", who);
    if ((Y != nullptr) != (dY != nullptr)) return fail(WUSH_E_ARG, "%s: Y and dY are given together", who);
    if ((gate != nullptr) != (dgate != nullptr)) return fail(WUSH_E_ARG, "%s: gate and dgate are given together", who);
    if (!dU && !dRout) return fail(WUSH_E_ARG, "%s: no gradient given", who);
    if ((w_pre && (!Rout || !rstd_pre)) || (w_post && !rstd_post)) return fail(WUSH_E_ARG, "%s: null pointer", who);
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  for (const void* p : {dU, dRout, Y, static_cast<const void*>(w_post), Rout, static_cast<const void*>(w_pre),
                        static_cast<const void*>(dY), static_cast<const void*>(dR), static_cast<const void*>(dw_post),
                        static_cast<const void*>(dw_pre), static_cast<const void*>(ws)})
    if (!aligned16(p)) return fail(WUSH_E_ARG, "%s: pointers must be 16-byte aligned", who);
  if ((!aligned16(gate) || !aligned16(dgate)) && gate_kind != WUSH_GATE_TOKEN)
    return fail(WUSH_E_ARG, "%s: pointers must be 16-byte aligned", who);
  float* gate_cols = gate_kind == WUSH_GATE_CHANNEL ? static_cast<float*>(dgate) : nullptr;
  const bool cols = dw_pre || dw_post || gate_cols;
  const size_t need = cols ? wush_block_norm_bwd_ws_bytes(n, d) : 0;
  if (ws && ws_bytes < need) return fail(WUSH_E_ARG, "%s: workspace of %zu bytes, need %zu", who, ws_bytes, need);
  float* part = static_cast<float*>(ws);
  if (need && !ws) {
    const hipError_t e = hipMallocAsync(reinterpret_cast<void**>(&part), need, s);
    if (e != hipSuccess) return fail(WUSH_E_HIP, "%s: scratch: %s", who, hipGetErrorString(e));
  }
  const NormArgs a{n, d, w_post, w_pre, gate, branch_scale, res_scale, 0.0f, const_cast<float*>(rstd_post),
                   const_cast<float*>(rstd_pre)};
  const int groups = n > 0 ? bwd_groups(n, d) : 0;
  wush_status out = WUSH_OK;
  if (n > 0)
    out = by_types(Y ? ydt : rdt, rdt, dU ? udt : rdt, [&](auto y, auto r, auto u) {
      using YT = decltype(y);
      using RT = decltype(r);
      using UT = decltype(u);
      const YT* Yp = static_cast<const YT*>(Y);
      const RT* dRp = static_cast<const RT*>(dRout);
      const RT* Rp = static_cast<const RT*>(Rout);
      const UT* dUp = static_cast<const UT*>(dU);
      auto run = [&](auto gate) {
        constexpr int G = decltype(gate)::value;
        if (d > 8192) {
          auto k = d <= 16384 ? norm_bwd_wide_kernel<YT, RT, UT, 2, 1024, G> : norm_bwd_wide_kernel<YT, RT, UT, 4, 768, G>;
          hipLaunchKernelGGL(k, dim3(groups), dim3(threads(d, bwd_vpt(d))), 0, s, a, dUp, dRp, Yp, Rp,
                             static_cast<YT*>(dY), static_cast<RT*>(dR), dgate, part);
          return;
        }
        // stand-ins for what is left out: at least one of dRout and the pair
        // dU, Rout is there, and no type but Y's may be wider than R's
        const RT* some = dRp ? dRp : Rp;
        auto k = d <= 1024   ? norm_bwd_kernel<YT, RT, UT, 128, G>
                 : d <= 4096 ? norm_bwd_kernel<YT, RT, UT, 512, G>
                             : norm_bwd_kernel<YT, RT, UT, 1024, G>;
        hipLaunchKernelGGL(k, dim3(groups), dim3(threads(d, bwd_vpt(d))), 0, s, a, rstd_post, rstd_pre,
                           dUp ? dUp : reinterpret_cast<const UT*>(some), some, dRp != nullptr,
                           Yp ? Yp : reinterpret_cast<const YT*>(some), Yp != nullptr, w_pre ? Rp : some,
                           static_cast<YT*>(dY), static_cast<RT*>(dR), dgate, part);
      };
      using std::integral_constant;
      if (gate_kind == WUSH_GATE_CHANNEL)
        run(integral_constant<int, WUSH_GATE_CHANNEL>());
      else if (gate_kind == WUSH_GATE_ELEMENT)
        run(integral_constant<int, WUSH_GATE_ELEMENT>());
      else
        run(integral_constant<int, WUSH_GATE_TOKEN>());
      return launched(who);
    });
  if (out == WUSH_OK && cols) {
    hipLaunchKernelGGL(norm_cols_kernel, dim3((d + 63) / 64, 3), dim3(1024), 0, s, d, groups, part, dw_pre, dw_post,
                       gate_cols);
    out = launched(who);
  }
  if (need && !ws) (void)hipFreeAsync(part, s);
  return out;
}
