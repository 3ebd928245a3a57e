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
// infinity splits into an infinity and NaN, and one in the other operand meets
// terms that are zero: results that either reaches are NaN.
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

// The last of `count` items whose first(item) is not past `number`, -1 if there is
// none; first must rise.  A wave looks at 64 items that lie evenly apart at a
// time, and a 64th is left: two turns for 4096.
template <class F>
__device__ __forceinline__ int last_not_past(int count, int number, F first) {
  int s = 0, below = count;   // it lies in [s, below)
  for (;;) {
    const int step = (below - s + 63) / 64, q = s + (threadIdx.x & 63) * step;
    const int c = __popcll(__ballot(q < below && first(q) <= number));
    if (c == 0) return -1;
    s = __builtin_amdgcn_readfirstlane(s + (c - 1) * step);
    if (step == 1) return s;
    below = min(s + step, below);
  }
}

template <int T>
__device__ __forceinline__ Tile find_tile(int number, int n, int nseg, const int* __restrict__ off,
                                          const int* __restrict__ ids, int nad) {
  // the tile's request is the last one whose first tile is not past `number`.  Of
  // up to 64 requests the lanes hold everything needed; one load after another is
  // saved.  65536 requests of a token, 64 -> 64 at rank 16: 0.38 ms, 22 where every
  // workgroup looked at all of them; 4096 requests 29 us and 112.
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
    s = last_not_past(nseg, number, [&](int q) { return request_start(off, q, nseg, n) / T + q; });
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

// What the grad kernel walks over, made once per backward call.
// tokens [whole steps]: the tokens of adapter 0, 1, ..., each list in request
//   order and padded to a multiple of 32 by its last token
// count [nad]: an adapter's tokens (0 where its rank is)
// start [nad + 1]: where its list begins, a multiple of 32
// chunk [nad + 1]: the number of its first chunk
// part [nad]: the number of its first partial sum, where it has several chunks
// span [nad]: tokens of its chunks, whole steps
// place [nseg]: where a request's tokens begin
struct Lists {
  int* tokens;
  int* count;
  int* start;
  int* chunk;
  int* part;
  int* span;
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

// Steps of a chunk at least, so that its start and its part of the join stay
// small beside it (it matters only to short calls), and the relative cost of a
// step: what the rows take, and the products of each row tile.  Four adapters of
// ranks between 8 and rmax, all steps taken as equal against these costs: the grad
// kernel on 16384 tokens with act8 X at 64 94 and 85 us; the backward call without
// dX on 16384 tokens, 5120 + 5120 bf16 columns, 110 and 109 us at rmax 32, 125 and
// 120 at 64, 241 and 203 at 128, on 4096 tokens, 4096 + 12288, 59 and 58, 73 and 70,
// 123 and 108.
constexpr int kMinSteps = 4;
__device__ __forceinline__ float step_cost(int rank, int rmax) {
  const int tiles = (min(max(rank, 1), rmax) + 15) / 16;
  return tiles > 4 ? 9.0f : tiles > 2 ? 6.0f : tiles > 1 ? 5.0f : 4.5f;
}

// Makes the lists; one workgroup of WAVES waves, to which the low kernel of the
// backward call gives a place beside its own.  The work grows with the requests
// and with the adapters, not with their product: one wave goes over the requests,
// 64 at a time, and counts the tokens of every adapter as it finds each request's
// place among them; the lists' lengths then give the chunks, and all waves write
// the tokens.  Up to 64 requests stay in the lanes of every wave, and the counts of
// few adapters in `lds` (of `room` integers), since each turn through memory costs
// most of a microsecond: so few hide behind the low kernel.  Many do not: some 6
// us for each 64 requests (16384 tokens, 4096 + 4096 columns at rank 16, the whole
// backward call: 153 us for 12 requests of 4 adapters, 169 for 128 of 32, 206 for
// 512 of 128, 556 for 4096 of 256; with a wave that went over all requests for
// each adapter, and workgroups that looked at all requests, 158, 204, 440 and
// 3097).
template <int WAVES>
__device__ __forceinline__ void list_tokens(int n, int nseg, const int* off, const int* ids, int nad, const int* rank,
                                            int rmax, int chunks_wanted, int* lds, int room, const Lists& l) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const bool few = nseg <= 64;
  int* found = nad <= room ? lds : l.count;
  // a request's adapter (-1: none), first token and tokens, and how many tokens of
  // its adapter come before it
  struct Request {
    int adapter, first, tokens, place;
  };
  auto request = [&](int s) {
    Request r{-1, 0, 0, 0};
    if (s >= nseg) return r;
    const int a = ids[s];
    r.first = request_start(off, s, nseg, n);
    r.tokens = max(request_start(off, s + 1, nseg, n) - r.first, 0);
    if (a >= 0 && a < nad && r.tokens > 0) r.adapter = a;
    return r;
  };
  Request next = request(lane);
  for (int a = threadIdx.x; a < nad; a += 64 * WAVES) found[a] = 0;
  __syncthreads();
  Request r = next;
  if (few || wave == 0) {
    for (int b = 0; b < nseg; b += 64) {
      r = next;
      if (!few) next = request(b + 64 + lane);
      int at = b > 0 && r.adapter >= 0 ? found[r.adapter] : 0;
      bool last = true;   // of its adapter's requests among the 64
      for (int first = 0; first < min(nseg - b, 64); first += 8) {
#pragma unroll
        for (int i = first; i < first + 8; ++i) {
          const bool same = __builtin_amdgcn_readlane(r.adapter, i) == r.adapter;
          at += same && i < lane ? __builtin_amdgcn_readlane(r.tokens, i) : 0;
          last = last && !(same && i > lane);
        }
      }
      // counts end at n, which offsets that do not rise could pass
      r.place = min(at, n);
      if (r.adapter >= 0 && wave == 0) {
        if (!few) l.place[b + lane] = r.place;
        if (last) found[r.adapter] = min(at + r.tokens, n);
      }
      __threadfence_block();   // other lanes read these counts
    }
  }
  if (wave == 0) {
    // a list's cost: its tokens (none where its rank is zero) times the cost of a
    // step at its rank
    auto listed = [&](int a) { return a < nad && rank[a] > 0 ? found[a] : 0; };
    float cost = 0.0f;
    int busy = 0;
    for (int b = 0; b < nad; b += 64) {
      const int mine = listed(b + lane);
      if (mine > 0) cost += mine * step_cost(rank[b + lane], rmax);
      busy += __popcll(__ballot(mine > 0));
    }
    cost = wave_sum(cost);
    // every list ends inside a chunk, half of one wasted on average
    const float share = cost / max(1, chunks_wanted - busy / 2);
    int tokens = 0, chunks = 0, several = 0, steps = 0;   // tokens: those that are not padding
    for (int b = 0; b < nad; b += 64) {
      const int a = b + lane;
      // capped at n together too
      const int64_t past = tokens + static_cast<int64_t>(lane_prefix(listed(a)));
      const int to = static_cast<int>(min(past, static_cast<int64_t>(n)));
      const int before = __shfl_up(to, 1, 64);
      const int mine = to - (lane == 0 ? tokens : before);
      const int span = a < nad ? 32 * max(kMinSteps, static_cast<int>(ceilf(share / (32.0f * step_cost(rank[a], rmax))))) : 32;
      // chunks and those of adapters with several: at most 2^16 - 1 in all (the
      // launch's limit), and fewer, in the halves of one sum
      const int parts = (mine + span - 1) / span, kept = parts > 1 ? parts : 0;
      const int both = lane_prefix(parts | kept << 16), c = both & 0xffff, k = both >> 16;
      const int turns = (mine + 31) / 32, t = lane_prefix(turns);
      if (a < nad) {
        l.count[a] = mine;
        l.span[a] = span;
        l.start[a] = 32 * (steps + t - turns);
        l.chunk[a] = chunks + c - parts;
        l.part[a] = several + k - kept;
      }
      tokens = __builtin_amdgcn_readlane(to, 63);
      steps += __builtin_amdgcn_readlane(t, 63);
      chunks += __builtin_amdgcn_readlane(c, 63);
      several += __builtin_amdgcn_readlane(k, 63);
    }
    if (lane == 0) {
      l.start[nad] = 32 * steps;
      l.chunk[nad] = chunks;
    }
  }
  __syncthreads();
  // few requests: every wave a share of each one's tokens; many: of the requests
  const int turn = few ? 64 * WAVES : 64;
  for (int b = few ? 0 : 64 * wave; b < nseg; b += 64 * WAVES) {
    if (!few) {
      r = request(b + lane);
      r.place = r.adapter >= 0 ? l.place[b + lane] : 0;
    }
    int to = 0, tokens = 0;
    if (r.adapter >= 0) {
      const int count = l.count[r.adapter], start = l.start[r.adapter];
      to = start + r.place;
      tokens = max(min(r.tokens, count - r.place), 0);
      // the list's last token fills up its last step
      if (tokens > 0 && r.place + tokens == count && (wave == 0 || !few))
        for (int q = count; q % 32 != 0; ++q) l.tokens[start + q] = r.first + tokens - 1;
    }
    for (uint64_t left = __ballot(tokens > 0); left != 0; left &= left - 1) {
      const int i = __builtin_ctzll(left), first = __builtin_amdgcn_readlane(r.first, i);
      const int to_i = __builtin_amdgcn_readlane(to, i), tokens_i = __builtin_amdgcn_readlane(tokens, i);
      for (int q = few ? threadIdx.x : lane; q < tokens_i; q += turn) l.tokens[to_i + q] = first + q;
    }
  }
}

// The lists wanted from a launch that has a workgroup to spare for them.
struct ListJob {
  bool on;
  int chunks_wanted;
  Lists l;
};

inline int64_t tile_numbers(int n, int T, int nseg) { return static_cast<int64_t>(n / T) + nseg; }

}  // namespace wush
