// The routed experts' gated MLP on microscaled 4-bit weights:
//
//   y_t = sum_s w_ts D_e (silu(G_e x_t) * (V_e x_t)),  e = ids[t][s].
//
// Products run on the bfloat16 matrix instructions.  A weight, 4-bit float
// times power of two, is exact in bfloat16, and one conversion instruction
// turns two codes and their block's scale into two bfloat16 values, so the
// weights stay 4.25 bits wide up to the registers that feed the matrix unit.
// An activation is split into bfloat16 terms that add up to it exactly (one
// for bfloat16, two for float16, three for float32), each multiplied on its
// own into the same float32 accumulators.  (The block-scaled matrix
// instructions would take the codes unconverted, but their sums of 128
// products hold only about 14 bits, measured: 4e-5 of the result after one
// instruction.)
//
// Weight layout.  A matrix of R rows and K columns (zero-padded to multiples
// of 256) is cut into tiles of 32 rows by 64 columns, 1 KB of codes each: the
// 16 bytes of (half h of the columns, row r) hold the 32 codes of one scale
// block.  With lane = 32 h + r a wave loads a tile as one contiguous
// kilobyte, 16 bytes per lane, every lane's codes share one scale, and dword
// m of a lane is its operand of the m-th 32x32x16 instruction; both operands
// use the same order of columns, which is all a sum over columns asks for.
// Scale bytes of four column steps form one dword per lane.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <memory>
#include <new>

#include "device_util.h"
#include "hip_util.h"
#include "value_util.h"

struct cfr_experts {
  cfr_experts_config cfg;
  int sh = 0, si = 0;  // 64-column steps of a gate/up row and of a down row, multiples of 4
  int hp = 0, ip = 0;  // 64 sh and 64 si: padded hidden and inter
  void* mem = nullptr;
  // weights: codes [E][rows / 32][steps][1024], scales [E][rows / 32][steps / 4][64] dwords
  uint8_t *gate = nullptr, *up = nullptr, *down = nullptr;
  uint32_t *gate_s = nullptr, *up_s = nullptr, *down_s = nullptr;
  // workspace, written anew by every call
  int32_t* order = nullptr;   // [tokens * top] routed slots sorted by expert, in slot order
  int4* tiles = nullptr;      // [1 + tokens * top / 32 + E] number of tiles, then their entries (find_work)
  uint16_t* xt = nullptr;     // [terms][tokens][hp] bfloat16 terms of x
  uint16_t* h = nullptr;      // [terms][tokens * top][ip] bfloat16 terms of silu(g) u, sorted as order (of w silu(g) u,
                              // in slot order, in a call with few slots)
  float* yp = nullptr;        // [tokens * top][hp] w_ts D_e h of each slot: float32, or float16 with
  uint8_t* ye = nullptr;      // [tokens * top][hp / 64] powers of two (bfloat16 tokens)
  int32_t* status = nullptr;  // [1]
};

namespace cfr {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));

union Frag {  // eight bfloat16 values of one lane: its operand of a matrix instruction
  bf16x8_t v;
  bf16x2_t p[4];
  uint32_t u[4];
  u32x4_t w;
};

constexpr int kFewSlots = 64;  // calls with at most this many slots go without sorting (one ballot sees them all)
constexpr int kThreads = 256;

// Eight weights of one dword of codes, times their block's scale.
__device__ __forceinline__ Frag weights8(uint32_t codes, float scale) {
  Frag f;
  f.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
  f.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
  f.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
  f.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
  return f;
}

// 2^(byte - 127) of scale byte b of a dword (byte 0: the denormal 2^-127).
__device__ __forceinline__ float scale_of(uint32_t dword, int b) {
  return __uint_as_float(max(((dword >> (8 * b)) & 255u) << 23, 0x00400000u));
}

// v as N bfloat16 terms: each term but the last takes the leading eight bits
// of what is left (exact), the last is rounded.  Three terms hold a float32
// exactly, two a float16.  A non-finite v is its first term.
template <int N>
__device__ __forceinline__ void split(float v, uint16_t* t) {
  const bool odd = !(fabsf(v) < INFINITY);
  const uint16_t whole = f32_bf16(v);
#pragma unroll
  for (int i = 0; i < N - 1; ++i) {
    t[i] = (uint16_t)(__float_as_uint(v) >> 16);
    v -= bf16_f32(t[i]);
  }
  t[N - 1] = f32_bf16(v);
  if (N > 1 && odd) {
    t[0] = whole;
#pragma unroll
    for (int i = 1; i < N; ++i) t[i] = 0;
  }
}

// Eight values as N fragments of terms.
template <int N>
__device__ __forceinline__ void split8(const float* v, Frag* f) {
  uint16_t t[8][N];
#pragma unroll
  for (int j = 0; j < 8; ++j) split<N>(v[j], t[j]);
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) f[i].u[j] = t[2 * j][i] | (uint32_t)t[2 * j + 1][i] << 16;
}

template <int DT>
constexpr int terms() { return DT == CFR_F32 ? 3 : DT == CFR_F16 ? 2 : 1; }

// ---------------------------------------------------------------- layout ---

// One thread per lane of a tile: 16 bytes of codes and their scale byte.
__global__ __launch_bounds__(kThreads) void k_experts_layout(const uint8_t* __restrict__ codes,
                                                             const uint8_t* __restrict__ scales, int64_t rows,
                                                             int64_t cols, int tiles, int steps, int64_t total,
                                                             uint8_t* __restrict__ out, uint8_t* __restrict__ out_s,
                                                             int32_t* __restrict__ nan_seen) {
  const int64_t code_row = (cols + 1) / 2, scale_row = (cols + 31) / 32;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
    const int lane = (int)(i & 63);
    const int64_t tile_step = i >> 6;
    const int s = (int)(tile_step % steps);
    const int64_t te = tile_step / steps;  // expert * tiles + tile
    const int tile = (int)(te % tiles);
    const int64_t e = te / tiles;
    const int64_t row = (int64_t)tile * 32 + (lane & 31), blk = 2 * (int64_t)s + (lane >> 5);
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    uint8_t sb = 127;
    if (row < rows && blk * 32 < cols) {
      const uint8_t* src = codes + (e * rows + row) * code_row + blk * 16;
#pragma unroll
      for (int b = 0; b < 16; ++b) {
        const int64_t c = blk * 32 + 2 * b;
        uint32_t v = c < cols ? src[b] : 0u;
        if (c + 1 >= cols) v &= 15u;
        w[b >> 2] |= v << (8 * (b & 3));
      }
      sb = scales[(e * rows + row) * scale_row + blk];
      if (sb == 255) atomicOr(nan_seen, 1);
    }
    *reinterpret_cast<uint4*>(out + i * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    out_s[((te * (steps / 4) + (s >> 2)) * 64 + lane) * 4 + (s & 3)] = sb;
  }
}

// ------------------------------------------------------------------ plan ---

constexpr int kPlanThreads = 1024;

// Sum of v over the workgroup's threads below `limit`, in every thread.
__device__ __forceinline__ int sum_below(int v, int limit, int* sh) {
  v = wave_scan((int)threadIdx.x < limit ? v : 0);
  if ((threadIdx.x & 63) == 63) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  int s = 0;
  for (int k = 0; k < kPlanThreads / 64; ++k) s += sh[k];
  return s;
}

// Workgroups 0 .. E-1: each counts the slots of all experts in LDS (whole
// numbers, so the order of the additions does not matter), sums those of the
// experts below its own, and writes its own expert's slots, in slot order, and
// one entry of the tile list per `tile` slots of it.  The workgroups after them
// split x into terms.  Bound by its chain of reads: 4.6 us for 6216 slots, 11 us
// for 32768 (128 experts, bfloat16 tokens read in place).
template <int DT>
__global__ __launch_bounds__(kPlanThreads) void k_experts_plan(const int32_t* __restrict__ ids, int64_t slots, int E, int tile,
                                                               int32_t* __restrict__ order, int4* __restrict__ tiles,
                                                               int32_t* __restrict__ status,
                                                               const void* __restrict__ x, int64_t xs, int tokens, int H,
                                                               int hp, uint16_t* __restrict__ xt) {
  constexpr int N = terms<DT>(), kWaves = kPlanThreads / 64;
  if ((int)blockIdx.x >= E) {
    const int64_t per = hp / 8, total = (int64_t)tokens * per;
    for (int64_t i = (int64_t)(blockIdx.x - E) * kPlanThreads + threadIdx.x; i < total;
         i += (int64_t)(gridDim.x - E) * kPlanThreads) {
      const int64_t t = i / per;
      const int c = (int)(i - t * per) * 8;
      float v[8];
      Raw8 r;
      r.load(x, DT, t * xs + c, H - c);  // zeros past the row's end
      r.vals(DT, v);
      Frag f[N];
      split8<N>(v, f);
#pragma unroll
      for (int k = 0; k < N; ++k)
        *reinterpret_cast<u32x4_t*>(xt + ((int64_t)k * tokens + t) * hp + c) = f[k].w;
    }
    return;
  }
  __shared__ int hist[kPlanThreads], eq_of[kWaves], sums[2][kWaves];
  const int e = blockIdx.x, lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t seg = ((slots + kWaves - 1) / kWaves + 63) / 64 * 64;
  const int64_t lo = w * seg, hi = min(lo + seg, slots);
  hist[threadIdx.x] = 0;
  __syncthreads();
  constexpr int kBatch = 8;  // ids of a lane in flight together
  int id[kBatch], eq = 0;
  bool beyond = false;
  const auto read = [&](int64_t i0) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) id[k] = i0 + 64 * k + lane < hi ? ids[i0 + 64 * k + lane] : -1;
  };
  for (int64_t i0 = lo; i0 < hi; i0 += 64 * kBatch) {
    read(i0);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      eq += __popcll(__ballot(id[k] == e));
      beyond |= id[k] >= E;
      if (id[k] >= 0 && id[k] < E) atomicAdd(&hist[id[k]], 1);
    }
  }
  if (e == 0 && beyond) atomicOr(status, 1);
  if (lane == 0) eq_of[w] = eq;
  __syncthreads();
  const int c = hist[threadIdx.x], t = (c + tile - 1) / tile, mine = hist[e];
  const int start = sum_below(c, e, sums[0]), first = sum_below(t, e, sums[1]);
  for (int i = threadIdx.x; i < (mine + tile - 1) / tile; i += kPlanThreads)
    tiles[1 + first + i] = make_int4(e, first, start, mine);
  if (e == E - 1 && threadIdx.x == 0) tiles[0].x = first + (mine + tile - 1) / tile;  // their number
  if (eq == 0) return;
  int at = start;
  for (int k = 0; k < w; ++k) at += eq_of[k];
  for (int64_t i0 = lo; i0 < hi; i0 += 64 * kBatch) {
    if (hi - lo > 64 * kBatch) read(i0);  // otherwise they are still here
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const unsigned long long m = __ballot(id[k] == e);
      if (id[k] == e) order[at + __popcll(m & ((1ull << lane) - 1ull))] = (int32_t)(i0 + 64 * k + lane);
      at += __popcll(m);
    }
  }
}

// -------------------------------------------------------------- products ---

// Which (expert, first slot, slots) a workgroup works on, and which group of
// rows.
struct Work {
  int expert, first, n, group;
};

// An expert's work items are its groups of rows, each with all its tiles side
// by side, so that tiles which read the same weights run together.  Workgroups
// go to the eight XCDs in turn, and each XCD takes a contiguous range of the
// items: its L2 then holds those weights once.  Entry 1 + i of the list belongs
// to tile i: its expert, that expert's first tile, first slot and slots.
template <int BM>
__device__ __forceinline__ bool find_work(const int4* tiles, int groups, Work& w) {
  const int64_t total = (int64_t)__builtin_amdgcn_readfirstlane(tiles[0].x) * groups, per = (total + 7) / 8;
  const int64_t idx = blockIdx.x >> 3, item = (blockIdx.x & 7) * per + idx;
  if (idx >= per || item >= total) return false;
  const int4 t = tiles[1 + (int)(item / groups)];
  const int n = __builtin_amdgcn_readfirstlane(t.w), te = (n + BM - 1) / BM;
  const int r = (int)(item - (int64_t)__builtin_amdgcn_readfirstlane(t.y) * groups);
  w.expert = __builtin_amdgcn_readfirstlane(t.x);
  w.group = r / te;
  w.first = (r - w.group * te) * BM;
  w.n = min(BM, n - w.first);
  w.first += __builtin_amdgcn_readfirstlane(t.z);
  return true;
}

// A 32x32 product leaves lane (col, q) rows 8 j + 4 q + 0..3 of its column at
// 4 j .. 4 j + 3; d holds them as 16 bits each, two to a dword.  Exchanged with
// the lane of the other q: rows 16 j + 8 q + 0..7 in r[j], 16 bytes of a row.
__device__ __forceinline__ void eights(const uint32_t (&d)[8], u32x4_t (&r)[2]) {
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const auto x = __builtin_amdgcn_permlane32_swap(d[4 * j + i], d[4 * j + 2 + i], false, false);
      r[j][i] = x[0];
      r[j][2 + i] = x[1];
    }
}

// One wave's two 32-row weight tiles times 32 CF tokens: acc += W X^T over all
// steps.  The workgroup's W waves hold different rows and share the tokens'
// terms through LDS, two stages of KU column steps.  16-byte pieces of a
// token's 128 bytes are stored at place (piece ^ (token / 2 & 7)): two tokens
// span the 64 banks, so the 16 tokens that one cycle of a 16-byte LDS read
// touches lie in different banks (piece ^ (token & 7) cost a second cycle).
// Weights go from memory to registers one stage ahead, tokens two.
template <int N, int CF, int KU, int W>
struct Product {
  static constexpr int kRows = 32 * CF;
  static constexpr int kPass = 8 * W;  // tokens whose pieces the workgroup moves at a time
  static constexpr int kStage = N * KU * kRows * 128;  // bytes

  // base addresses are the same in every lane of a wave; offsets are in bytes
  const uint8_t* w[2];
  const uint32_t* ws[2];
  const uint8_t* x;
  int64_t term_stride;  // bytes
  uint32_t row[kRows / kPass];  // this thread's token rows, at its piece
  static_assert(kRows % kPass == 0, "whole passes");

  struct Weights {
    u32x4_t c[2][KU];
  };
  struct Operands {
    Frag a[2];
  };

  __device__ __forceinline__ void load_weights(Weights& r, int stage) const {
    const uint32_t at = (threadIdx.x & 63) * 16;
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int k = 0; k < KU; ++k)
        r.c[a][k] = *reinterpret_cast<const u32x4_t*>(w[a] + (int64_t)(stage * KU + k) * 1024 + at);
  }
  __device__ __forceinline__ void load_scales(uint32_t (&s)[2], int group) const {
#pragma unroll
    for (int a = 0; a < 2; ++a) s[a] = (ws[a] + group * 64)[threadIdx.x & 63];
  }
  // Passes over the 32 F tokens of a stage, and 16-byte pieces per thread.
  template <int F>
  static constexpr int passes() { return (32 * F + kPass - 1) / kPass; }
  template <int F>
  static constexpr int pieces() { return N * KU * passes<F>(); }

  template <int F>
  __device__ __forceinline__ void load_tokens(u32x4_t (&r)[pieces<F>()], int stage) const {
    constexpr int P = passes<F>();
#pragma unroll
    for (int i = 0; i < pieces<F>(); ++i) {
      const int f = i % P, k = (i / P) % KU, t = i / (P * KU);
      r[i] = *reinterpret_cast<const u32x4_t*>(x + t * term_stride + (stage * KU + k) * 128 + row[f]);
    }
  }
  template <int F>
  __device__ __forceinline__ void store_tokens(char* lds, const u32x4_t (&r)[pieces<F>()]) const {
    constexpr int P = passes<F>();
    const int tok = threadIdx.x >> 3, piece = (threadIdx.x & 7) ^ ((tok >> 1) & 7);
#pragma unroll
    for (int i = 0; i < pieces<F>(); ++i) {
      const int f = i % P, tk = i / P;  // tk = term * KU + step
      *reinterpret_cast<u32x4_t*>(lds + (tk * kRows + f * kPass + tok) * 128 + piece * 16) = r[i];
    }
  }
  // A stage is KU * 4 * N positions (step k, quarter m of its columns, term
  // t).  Each position requests the next one's tokens and converts the next
  // quarter's weights before its own products, so neither is waited for.
  // first: the stage's first step within its group of four.
  template <int F>
  __device__ __forceinline__ void multiply(f32x16_t (*acc)[CF], const char* lds, const Weights& r, const uint32_t (&s)[2],
                                           int first) const {
    const int col = threadIdx.x & 31, h = (threadIdx.x >> 5) & 1;
    const auto tokens = [&](Frag (&f)[F], int pos) {
      const int t = pos % N, m = pos / N % 4, k = pos / (4 * N);
#pragma unroll
      for (int i = 0; i < F; ++i)
        f[i].w = *reinterpret_cast<const u32x4_t*>(lds + ((t * KU + k) * kRows + i * 32 + col) * 128 +
                                                   (((h * 4 + m) ^ ((col >> 1) & 7)) * 16));
    };
    const auto convert = [&](Operands& o, int pos) {
      const int m = pos / N % 4, k = pos / (4 * N);
#pragma unroll
      for (int a = 0; a < 2; ++a) o.a[a] = weights8(r.c[a][k][m], scale_of(s[a], first + k));
    };
    constexpr int kPos = KU * 4 * N;
    Frag f[2][F];
    Operands o[2];
    tokens(f[0], 0);
    convert(o[0], 0);
#pragma unroll
    for (int pos = 0; pos < kPos; ++pos) {
      if (pos + 1 < kPos) {
        tokens(f[(pos + 1) & 1], pos + 1);
        if ((pos + 1) % N == 0) convert(o[((pos + 1) / N) & 1], pos + 1);
      }
#pragma unroll
      for (int i = 0; i < F; ++i)
#pragma unroll
        for (int a = 0; a < 2; ++a)
          acc[a][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(o[(pos / N) & 1].a[a].v, f[pos & 1][i].v, acc[a][i], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  // lds: two stages.  steps is a multiple of 4.  Loads past the last stage
  // read it again, so the loop has no branches around its loads.
  template <int F>
  __device__ __forceinline__ void run_as(f32x16_t (*acc)[CF], char* lds, int steps) const {
    constexpr int kStages = 4 / KU;  // of a group of four steps, which share a dword of scales
    const int last = steps / KU - 1, groups = steps / 4;
    Weights cur, next;
    u32x4_t xr[pieces<F>()];
    uint32_t s[2];
    load_scales(s, 0);
    load_tokens<F>(xr, 0);
    load_weights(cur, 0);
    store_tokens<F>(lds, xr);
    load_tokens<F>(xr, min(1, last));
    for (int g = 0; g < groups; ++g) {
      uint32_t sn[2];
#pragma unroll
      for (int j = 0; j < kStages; ++j) {
        const int st = g * kStages + j;
        load_weights(next, min(st + 1, last));
        if (j == 0) load_scales(sn, min(g + 1, groups - 1));
        lds_barrier();  // this stage is written, and the other one is no longer read
        store_tokens<F>(lds + ((st + 1) & 1) * kStage, xr);
        load_tokens<F>(xr, min(st + 2, last));
        multiply<F>(acc, lds + (st & 1) * kStage, cur, s, j * KU);
        cur = next;
      }
      s[0] = sn[0], s[1] = sn[1];
    }
  }
  // A tile that is not full does the work of its 32s of tokens only.
  __device__ __forceinline__ void run(f32x16_t (*acc)[CF], char* lds, int steps, int n) const {
    if constexpr (CF == 4) {
      if (n <= 32) return run_as<1>(acc, lds, steps);
      if (n > 32 && n <= 64) return run_as<2>(acc, lds, steps);
      if (n > 64 && n <= 96) return run_as<3>(acc, lds, steps);
    } else if constexpr (CF == 2) {
      if (n <= 32) return run_as<1>(acc, lds, steps);
    }
    run_as<CF>(acc, lds, steps);
  }
};

// h = silu(G x) * (V x) of a tile's slots and 32 W channels: each wave holds 32
// gate rows and the same 32 up rows, so the join needs no exchange.  Measured:
// 41 us at 64 float16 tokens of the Qwen3-30B-A3B layer (5.2 TB/s of weights), 53
// at 777 bfloat16 tokens (0.24 GB through memory at 4.5 TB/s), both bound by
// memory; 750 us at 4096 tokens of the Qwen3-235B-A22B layer (1.1 PFLOP/s, the
// matrix units 60% busy at a clock that falls to 1.75 GHz under them).
template <int N, int CF, int KU, int W>
__global__ __launch_bounds__(W * 64, 2) void k_experts_up(cfr_experts p, int64_t slots, const uint16_t* __restrict__ x,
                                                            int64_t xs, int64_t term_stride) {
  using P = Product<N, CF, KU, W>;
  __shared__ __align__(16) char lds[2 * P::kStage];
  Work wk;
  if (!find_work<P::kRows>(p.tiles, p.ip / (32 * W), wk)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t tile = (int64_t)wk.expert * (p.ip / 32) + wk.group * W + wave;
  P g;
  g.w[0] = p.gate + tile * p.sh * 1024;
  g.w[1] = p.up + tile * p.sh * 1024;
  g.ws[0] = p.gate_s + tile * (p.sh / 4) * 64;
  g.ws[1] = p.up_s + tile * (p.sh / 4) * 64;
  g.x = reinterpret_cast<const uint8_t*>(x);
  g.term_stride = term_stride * 2;
#pragma unroll
  for (int f = 0; f < P::template passes<CF>(); ++f) {
    const int r = min(f * P::kPass + ((int)threadIdx.x >> 3), wk.n - 1);  // past the tile's end: any row of it
    // below 2^32: in_place() and the workspace's limits see to it
    g.row[f] = (uint32_t)(p.order[wk.first + r] / p.cfg.top) * (uint32_t)(xs * 2) + (threadIdx.x & 7) * 16;
  }
  f32x16_t acc[2][CF] = {};
  g.run(acc, lds, p.sh, wk.n);
  const int col = lane & 31, q = lane >> 5, tile0 = (wk.group * W + wave) * 32;
#pragma unroll
  for (int f = 0; f < CF; ++f) {
    if (f * 32 >= wk.n) break;
    f32x16_t h;
#pragma unroll
    for (int i = 0; i < 16; ++i) h[i] = silu(acc[0][f][i]) * acc[1][f][i];
    if (tile0 + 32 > p.cfg.inter) {  // channels past the last one stay zero, whatever x holds
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (tile0 + 2 * (i & ~3) + 4 * q + (i & 3) >= p.cfg.inter) h[i] = 0.f;
    }
    uint16_t t[16][N];
#pragma unroll
    for (int i = 0; i < 16; ++i) split<N>(h[i], t[i]);
    uint16_t* out = p.h + (int64_t)(wk.first + f * 32 + col) * p.ip + tile0 + 8 * q;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      uint32_t d[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] = t[2 * i][k] | (uint32_t)t[2 * i + 1][k] << 16;
      u32x4_t r[2];
      eights(d, r);
      if (f * 32 + col < wk.n) {
        *reinterpret_cast<u32x4_t*>(out + (int64_t)k * slots * p.ip) = r[0];
        *reinterpret_cast<u32x4_t*>(out + (int64_t)k * slots * p.ip + 16) = r[1];
      }
    }
  }
}

// Values stored as float16 over a power of two that puts the block's largest
// finite one, of biased exponent e, at 2^14 or above: e is kept within 15 ..
// 254, so that both powers are normal floats.
__device__ __forceinline__ float to_half(uint32_t e) { return __uint_as_float((268u - e) << 23); }    // 2^(141 - e)
__device__ __forceinline__ float from_half(uint32_t e) { return __uint_as_float((e - 14u) << 23); }  // 2^(e - 141)

// w D h of a tile's slots and 64 W rows, to each slot's own place, in float32;
// for bfloat16 tokens, whose h was rounded to 2^-8 already, as float16 with one
// power of two per 64 values, at half the bytes through memory, written and read
// again (0.5 GB instead of 1 GB at 4096 tokens of the Qwen3-235B-A22B layer).
// That rounds each value to 2^-11 of itself, an eighth of y's own rounding,
// whatever stands beside it: half a step of the smallest float16 numbers is
// 2^-39 of the largest finite value of the 64, so down to 2^-28 of that the
// rounding is relative.  An infinity or a NaN is stored as itself.
// Measured as above: 28, 37 and 409 us; its rows are short, so a workgroup's
// start and end weigh more than in k_experts_up.
template <int N, int CF, int KU, int W>
__global__ __launch_bounds__(W * 64, 2) void k_experts_down(cfr_experts p, int64_t slots,
                                                              const float* __restrict__ gate_w) {
  using P = Product<N, CF, KU, W>;
  __shared__ __align__(16) char lds[2 * P::kStage];
  __shared__ int slot_of[P::kRows];
  __shared__ float weight_of[P::kRows];
  Work wk;
  if (!find_work<P::kRows>(p.tiles, (p.hp + 64 * W - 1) / (64 * W), wk)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // read now, used after the products; the barriers of run() come between
  if ((int)threadIdx.x < P::kRows) {
    const int slot = p.order[wk.first + min((int)threadIdx.x, wk.n - 1)];
    slot_of[threadIdx.x] = slot;
    weight_of[threadIdx.x] = gate_w[slot];
  }
  const int pair = wk.group * W + wave;  // of 32-row tiles; past the last one a wave repeats it and writes nothing
  const bool live = pair < p.hp / 64;
  const int64_t tile = (int64_t)wk.expert * (p.hp / 32) + min(pair, p.hp / 64 - 1) * 2;
  P g;
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    g.w[a] = p.down + (tile + a) * p.si * 1024;
    g.ws[a] = p.down_s + (tile + a) * (p.si / 4) * 64;
  }
  g.x = reinterpret_cast<const uint8_t*>(p.h + (int64_t)wk.first * p.ip);
  g.term_stride = slots * p.ip * 2;
#pragma unroll
  for (int f = 0; f < P::template passes<CF>(); ++f)
    g.row[f] = (uint32_t)min(f * P::kPass + ((int)threadIdx.x >> 3), wk.n - 1) * (uint32_t)(p.ip * 2) + (threadIdx.x & 7) * 16;
  f32x16_t acc[2][CF] = {};
  g.run(acc, lds, p.si, wk.n);
  if (!live) return;
  const int col = lane & 31, q = lane >> 5;
#pragma unroll
  for (int f = 0; f < CF; ++f) {
    if (f * 32 >= wk.n) break;
    const bool mine = f * 32 + col < wk.n;
    const int64_t slot = slot_of[f * 32 + col];
    const float w = weight_of[f * 32 + col];
    if constexpr (N > 1) {
      float* out = p.yp + slot * p.hp + pair * 64 + 4 * q;
      if (mine) {
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<float4*>(out + a * 32 + 2 * i) =
                make_float4(w * acc[a][f][i], w * acc[a][f][i + 1], w * acc[a][f][i + 2], w * acc[a][f][i + 3]);
      }
    } else {
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        top = max(top, max(__float_as_uint(acc[0][f][i]) & 0x7FFFFFFFu, __float_as_uint(acc[1][f][i]) & 0x7FFFFFFFu));
      // rows 4 q + .. of the other lane's half go out in this lane's eights: one power for both
      top = max(top, (uint32_t)xor_lane<32>((int)top));
      uint32_t e = __float_as_uint(__uint_as_float(top) * w) >> 23 & 255u;
      float sc = w;
      // values that are not finite, or so small that sc would not be (sc < 2^15
      // / top): w goes in first, and the largest of the finite ones counts.  The
      // two lanes of a column have one top and one w, so both come here or none.
      if (e == 255u || top < 15u << 23) {
        top = 0;
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            acc[a][f][i] *= w;
            const uint32_t m = __float_as_uint(acc[a][f][i]) & 0x7FFFFFFFu;
            top = max(top, m < 0x7F800000u ? m : 0u);
          }
        e = max(top, (uint32_t)xor_lane<32>((int)top)) >> 23;
        sc = 1.0f;
      }
      e = max(e, 15u);
      sc *= to_half(e);
      uint16_t* out = reinterpret_cast<uint16_t*>(p.yp) + slot * p.hp + pair * 64 + 8 * q;
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        uint32_t d[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          d[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{sc * acc[a][f][2 * i], sc * acc[a][f][2 * i + 1]}, f16x2_t));
        u32x4_t r[2];
        eights(d, r);
        if (mine) {
          *reinterpret_cast<u32x4_t*>(out + a * 32) = r[0];
          *reinterpret_cast<u32x4_t*>(out + a * 32 + 16) = r[1];
        }
      }
      if (mine && q == 0) p.ye[slot * (p.hp / 64) + pair] = (uint8_t)e;
    }
  }
}

// y_t = sum over its slots, in slot order, rounded once.  Bound by memory: 50 us
// at 4096 tokens of the Qwen3-235B-A22B layer (6 TB/s, part of it from the
// last-level cache), 6 us at 777 of the Qwen3-30B-A3B layer.
template <int DT>
__global__ __launch_bounds__(kThreads) void k_experts_combine(cfr_experts p, const int32_t* __restrict__ ids, int tokens,
                                                              void* __restrict__ y, int64_t ys) {
  const int H = p.cfg.hidden, top = p.cfg.top;
  const int64_t per = (H + 7) / 8, total = tokens * per;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
    const int64_t t = i / per;
    const int c = (int)(i - t * per) * 8;
    float v[8] = {};
    constexpr int kBatch = DT == CFR_BF16 ? 8 : 4;  // slots in flight together
    for (int s0 = 0; s0 < top; s0 += kBatch) {
      bool live[kBatch];
      u32x4_t q[kBatch][DT == CFR_BF16 ? 1 : 2];
      uint32_t e[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int64_t slot = t * top + s0 + k;
        const int id = s0 + k < top ? ids[slot] : -1;
        live[k] = id >= 0 && id < p.cfg.n_experts;
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (!live[k]) continue;
        const int64_t slot = t * top + s0 + k;
        if constexpr (DT == CFR_BF16) {
          q[k][0] = *reinterpret_cast<const u32x4_t*>(reinterpret_cast<const uint16_t*>(p.yp) + slot * p.hp + c);
          e[k] = p.ye[slot * (p.hp / 64) + (c >> 6)];
        } else {
          const u32x4_t* src = reinterpret_cast<const u32x4_t*>(p.yp + slot * p.hp + c);
          q[k][0] = src[0], q[k][1] = src[1];
        }
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (!live[k]) continue;
        if constexpr (DT == CFR_BF16) {
          const float sc = from_half(e[k]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t two = q[k][0][j];  // (a bit cast of the element itself reads the vector's first)
            const f16x2_t h = __builtin_bit_cast(f16x2_t, two);
            v[2 * j] = fmaf((float)h.x, sc, v[2 * j]);
            v[2 * j + 1] = fmaf((float)h.y, sc, v[2 * j + 1]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] += __uint_as_float(q[k][j >> 2][j & 3]);
        }
      }
    }
    store8(y, DT, t * ys + c, H - c, v);
  }
}

// ------------------------------------------------------------- few slots ---
//
// At most 64 slots: nothing is sorted; the two kernels below read the routing
// themselves, so a decode is two launches.  Both use 16x16x32 instructions on
// 16 rows of a tile (lane = 16 q + r holds block q of 128 columns) and split
// the columns over the waves of a workgroup.

// This lane's 16 bytes of codes and scale of rows r16 .. r16+15 of a tile at
// 128-column unit u.  The tile is the same for the wave, so addresses are a
// uniform base and a lane's own 32-bit offset.
struct Unit {
  u32x4_t c;
  uint32_t s;
  __device__ __forceinline__ void load(const uint8_t* codes, const uint32_t* scales, int64_t tile, int steps, int r16,
                                       int u) {
    const uint32_t lane = threadIdx.x & 63, row = r16 + (lane & 15), q = lane >> 4;
    const uint32_t at = (q >> 1) * 1024 + (q & 1) * 512 + row * 16, at_s = (q & 1) * 32 + row;
    c = *reinterpret_cast<const u32x4_t*>(codes + (tile * steps + 2 * u) * 1024 + at);
    s = (scales + (tile * (steps / 4) + (u >> 1)) * 64)[at_s];
  }
  __device__ __forceinline__ float scale(int u) const {
    const int q = (threadIdx.x & 63) >> 4;
    return scale_of(s, (2 * u + (q >> 1)) & 3);
  }
};

// w h of all slots of one expert and 16 channels, split into the terms that
// k_few_down multiplies: two at least, for its matrix unit idles and
// bfloat16's rounding of h can be had away for nothing.  One workgroup per
// (channel group, slot); the first slot of each expert does the work for all
// of them, kCols at a time.
// x: N bfloat16 terms, 16-byte aligned rows of whole 128-column units.  Few of
// the product's 16 columns are in use as a rule, and a load costs the path
// through the cache 16 bytes for every lane, used or not; so a wave loads the
// slots' own pieces only (a unit of one slot and term is 16 of 16 bytes, a
// quarter of a load), and spreads them to the columns through its own part of
// LDS, piece ^ column apart so that the columns' reads meet in no bank.
// Measured at 8 float32 tokens of the Qwen3-235B-A22B layer: 72 us, against 113
// with each lane loading its column; with two and four units of weights
// requested ahead 79 and 102, for their registers cost waves.  One-term tokens
// load by column: 6.0 us at one token of the Qwen3-30B-A3B layer, 6.7 through LDS.
// (Splitting x into its terms here instead of in a launch before saves one token
// that launch, about 1 us of 14, and costs eight 18 us of 72.)
template <int N>
__global__ __launch_bounds__(kThreads) void k_few_up(cfr_experts p, const uint16_t* __restrict__ x, int64_t xs,
                                                     int64_t term_stride, const int32_t* __restrict__ ids,
                                                     const float* __restrict__ gate_w, int slots) {
  constexpr int kWaves = kThreads / 64, NH = N < 2 ? 2 : N;
  constexpr int kCols = N == 1 ? 16 : N == 2 ? 8 : 4, kLoads = N == 1 ? 4 : kCols * N / 4;
  struct Request {
    Unit g, v;
    u32x4_t x[kLoads];
  };
  __shared__ u32x4_t spread[N == 1 ? 1 : kWaves][N == 1 ? 1 : kCols * N * 16];
  __shared__ f32x4_t part[kWaves][2][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), slot = blockIdx.y;
  const int id = lane < slots ? ids[lane] : -1;
  if (blockIdx.x == 0 && slot == 0 && wave == 0 && id >= p.cfg.n_experts) atomicOr(p.status, 1);
  const int e = __builtin_amdgcn_readlane(id, slot);
  if (e < 0 || e >= p.cfg.n_experts) return;
  const unsigned long long same = __ballot(id == e);
  if (same & ((1ull << slot) - 1ull)) return;  // an earlier slot has this expert
  const int all = __popcll(same);
  const int64_t tile = (int64_t)e * (p.ip / 32) + (blockIdx.x >> 1);
  const int r16 = (blockIdx.x & 1) * 16, units = (p.cfg.hidden + 127) / 128, q = lane >> 4;
  Request w;
  const auto request_weights = [&](Request& r, int u) {
    r.g.load(p.gate, p.gate_s, tile, p.sh, r16, u);
    r.v.load(p.up, p.up_s, tile, p.sh, r16, u);
  };
  if (wave < units) request_weights(w, wave);  // while the slots are sorted out
  // lane k < all: the k-th slot of this expert (the lanes trade places: its slots first, in order)
  const unsigned long long below = (1ull << lane) - 1ull;
  const int place = id == e ? __popcll(same & below) : all + __popcll(~same & below);
  const int mine = __builtin_amdgcn_ds_permute(place * 4, lane);
  for (int c0 = 0; c0 < all; c0 += kCols) {
    const int n = min(kCols, all - c0);
    const bool live = (lane & 15) < n;
    const int col = live ? lane & 15 : 0, at = __builtin_amdgcn_ds_bpermute((c0 + col) * 4, mine);
    const float gw = gate_w[at];  // requested here, used after the products
    // byte offsets of this lane's pieces: of its column's quarter q, or piece
    // lane & 15 of (slot, term) pair 4 i + q, and that one's place in LDS
    uint32_t from[kLoads], to[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      if constexpr (N == 1) {
        from[i] = (uint32_t)(at / p.cfg.top) * (uint32_t)(xs * 2) + q * 64 + i * 16;
      } else {
        const int ct = min(4 * i + q, n * N - 1), c = ct / N, t = ct % N;
        from[i] = (uint32_t)(__builtin_amdgcn_ds_bpermute((c0 + c) * 4, mine) / p.cfg.top) * (uint32_t)(xs * 2) +
                  t * (uint32_t)(term_stride * 2) + (lane & 15) * 16;
        to[i] = ct * 16 + ((lane & 15) ^ c);
      }
    }
    f32x4_t g = {0.f, 0.f, 0.f, 0.f}, v = {0.f, 0.f, 0.f, 0.f};
    const auto request_x = [&](Request& r, int u) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        if (N == 1 || 4 * i < n * N)
          r.x[i] = *reinterpret_cast<const u32x4_t*>(reinterpret_cast<const uint8_t*>(x) + u * 256 + from[i]);
    };
    // a unit is requested and multiplied; the other waves of the SIMD fill the wait
    for (int u = wave; u < units; u += kWaves) {
      if (c0 || u != wave) request_weights(w, u);
      request_x(w, u);
      if constexpr (N > 1) {  // the wave's LDS accesses are in order: these writes come after the last unit's reads
#pragma unroll
        for (int k = 0; k < kLoads; ++k)
          if (4 * k < n * N) spread[wave][to[k]] = w.x[k];
        __builtin_amdgcn_wave_barrier();
      }
      const float sg = w.g.scale(u), sv = w.v.scale(u);
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const Frag fg = weights8(w.g.c[m], sg), fv = weights8(w.v.c[m], sv);
#pragma unroll
        for (int t = 0; t < N; ++t) {
          Frag fx;
          if constexpr (N == 1)
            fx.w = w.x[m];
          else
            fx.w = spread[wave][(col * N + t) * 16 + ((4 * q + m) ^ col)];
          g = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fg.v, fx.v, g, 0, 0, 0);
          v = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fv.v, fx.v, v, 0, 0, 0);
        }
      }
      __builtin_amdgcn_wave_barrier();
    }
    part[wave][0][lane] = g;
    part[wave][1][lane] = v;
    lds_barrier();
    if (wave == 0 && live) {
#pragma unroll
      for (int k = 1; k < kWaves; ++k) g += part[k][0][lane], v += part[k][1][lane];
      const int ch = blockIdx.x * 16 + 4 * q;
      uint16_t t[4][NH];
#pragma unroll
      for (int j = 0; j < 4; ++j) split<NH>(ch + j < p.cfg.inter ? gw * (silu(g[j]) * v[j]) : 0.f, t[j]);
#pragma unroll
      for (int k = 0; k < NH; ++k)
        *reinterpret_cast<uint2*>(p.h + ((int64_t)k * slots + at) * p.ip + ch) =
            make_uint2(t[0][k] | (uint32_t)t[1][k] << 16, t[2][k] | (uint32_t)t[3][k] << 16);
    }
    lds_barrier();
  }
}

// Waves of k_few_down's workgroup and 128-column units of w h that it keeps in
// LDS at a time, four per wave.  Fewer workgroups than CUs: sixteen waves, so
// that one stage holds a token's slots (one token of the Qwen3-30B-A3B layer
// 5.2 us, 6.7 with eight waves); otherwise eight, whose LDS lets four share a
// CU (8 float32 tokens of the Qwen3-235B-A22B layer 52 us, 68 with sixteen).

// 16 rows of y of one token, all its slots.  The waves' weights are on their
// way, a stage of units ahead, while the workgroup brings the terms of w h
// into LDS; all 16 columns of the product are the token.  (Two row halves per
// workgroup, sharing what they read from LDS, took 62 us instead of 57 at 8
// float32 tokens of the Qwen3-235B-A22B layer.)
template <int DT, int W>
__global__ __launch_bounds__(W * 64) void k_few_down(cfr_experts p, const int32_t* __restrict__ ids, int slots,
                                                              void* __restrict__ y, int64_t ys) {
  constexpr int N = terms<DT>() < 2 ? 2 : terms<DT>(), kMine = 4, kUnits = kMine * W;
  __shared__ __align__(16) uint16_t wh[kUnits][N][128];
  __shared__ float part[W][16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), t = blockIdx.y;
  const int top = p.cfg.top;
  const int q = lane >> 4, units = p.si / 2, all = top * units, row0 = blockIdx.x * 16;
  ids += (int64_t)t * top;
  const uint16_t* h = p.h + (int64_t)t * top * p.ip;  // unit i of the token's slots is at 128 i
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  Unit ud[kMine];
  uint32_t live = 0;  // bit k: this wave's unit k of the stage has an expert
  const auto request = [&](int k, int i) {
    const int s = i / units, e = i < all ? ids[s] : -1;
    live &= ~(1u << k);
    if (e < 0 || e >= p.cfg.n_experts) return;
    live |= 1u << k;
    ud[k].load(p.down, p.down_s, (int64_t)e * (p.hp / 32) + (row0 >> 5), p.si, row0 & 16, i - s * units);
  };
#pragma unroll
  for (int k = 0; k < kMine; ++k) request(k, wave + k * W);
  for (int i0 = 0; i0 < all; i0 += kUnits) {
    if (i0) lds_barrier();  // the last stage is no longer read
    // what is not written at empty slots is not multiplied
    for (int c = threadIdx.x; c < min(kUnits, all - i0) * 16; c += W * 64)
#pragma unroll
      for (int k = 0; k < N; ++k)
        *reinterpret_cast<u32x4_t*>(&wh[c >> 4][k][(c & 15) * 8]) =
            *reinterpret_cast<const u32x4_t*>(h + (int64_t)k * slots * p.ip + (int64_t)i0 * 128 + c * 8);
    lds_barrier();
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      const int i = wave + k * W;
      if (live >> k & 1u) {
        const float sc = ud[k].scale((i0 + i) % units);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const Frag fd = weights8(ud[k].c[m], sc);
#pragma unroll
          for (int n = 0; n < N; ++n) {
            Frag fh;
            fh.w = *reinterpret_cast<const u32x4_t*>(&wh[i][n][q * 32 + 8 * m]);
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fd.v, fh.v, acc, 0, 0, 0);
          }
        }
      }
      if (i0 + kUnits < all) request(k, i0 + kUnits + i);
    }
  }
  if ((lane & 15) == 0) *reinterpret_cast<f32x4_t*>(&part[wave][4 * q]) = acc;
  lds_barrier();
  if (threadIdx.x < 16) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) v += part[k][threadIdx.x];
    const int row = row0 + threadIdx.x;
    if (row < p.cfg.hidden) store1(y, DT, t * ys + row, v);
  }
}

// ------------------------------------------------------------------ host ---

struct Call {
  const cfr_experts& p;
  const void* x;
  int64_t xs;
  const int32_t* ids;
  const float* gw;
  int tokens;
  int64_t slots;
  void* y;
  int64_t ys;
  bool x_aligned;  // x's rows can be read 16 aligned bytes at a time
  hipStream_t st;
};

// Whether x's rows are their own terms: bfloat16 that can be read 16 bytes at
// a time, whole units of `unit` columns, bytes counted in 32 bits (x's terms of
// 65536 tokens of 16384 values end at 2^31).
template <int DT>
bool in_place(const Call& c, int unit) {
  return DT == CFR_BF16 && c.x_aligned && c.p.cfg.hidden % unit == 0 && c.tokens * c.xs * 2 < (int64_t(1) << 32);
}

// The routing's counts and order for E experts, and x's terms if `copy`.
template <int DT>
void plan(const Call& c, int E, int tile, bool copy) {
  const cfr_experts& p = c.p;
  const int64_t pieces = (int64_t)c.tokens * (p.hp / 8);
  const unsigned g = E + (copy ? (unsigned)std::min<int64_t>((pieces + kPlanThreads - 1) / kPlanThreads, 512) : 0);
  hipLaunchKernelGGL((k_experts_plan<DT>), dim3(g), dim3(kPlanThreads), 0, c.st, c.ids, c.slots, E, tile, p.order, p.tiles,
                     p.status, c.x, c.xs, c.tokens, p.cfg.hidden, p.hp, p.xt);
}

template <int DT>
void few_slots(const Call& c) {
  const cfr_experts& p = c.p;
  const dim3 g1(p.ip / 16, (unsigned)c.slots);
  constexpr int N = terms<DT>();
  const bool own = in_place<DT>(c, 128);
  if (!own) plan<DT>(c, 0, 1, true);
  hipLaunchKernelGGL((k_few_up<N>), g1, dim3(kThreads), 0, c.st, p, own ? static_cast<const uint16_t*>(c.x) : p.xt,
                     own ? c.xs : (int64_t)p.hp, (int64_t)c.tokens * p.hp, c.ids,
                     c.gw, (int)c.slots);
  const dim3 g2((p.cfg.hidden + 15) / 16, c.tokens);
  if (g2.x * g2.y < 256)
    hipLaunchKernelGGL((k_few_down<DT, 16>), g2, dim3(1024), 0, c.st, p, c.ids, (int)c.slots, c.y, c.ys);
  else
    hipLaunchKernelGGL((k_few_down<DT, 8>), g2, dim3(512), 0, c.st, p, c.ids, (int)c.slots, c.y, c.ys);
}

template <int DT, int CF, int KU, int W>
void products(const Call& c) {
  constexpr int N = terms<DT>();
  const cfr_experts& p = c.p;
  const bool own = in_place<DT>(c, 256);
  plan<DT>(c, p.cfg.n_experts, 32 * CF, !own);
  // at most this many tiles: every expert with slots ends in one that is not full
  const int64_t tiles = c.slots / (32 * CF) + std::min<int64_t>(p.cfg.n_experts, c.slots);
  const auto grid = [&](int groups) { return dim3((unsigned)((tiles * groups + 7) / 8 * 8)); };
  hipLaunchKernelGGL((k_experts_up<N, CF, KU, W>), grid(p.ip / (32 * W)), dim3(W * 64), 0, c.st, p, c.slots,
                     own ? static_cast<const uint16_t*>(c.x) : p.xt, own ? c.xs : (int64_t)p.hp,
                     (int64_t)c.tokens * p.hp);
  hipLaunchKernelGGL((k_experts_down<N, CF, KU, W>), grid((p.hp + 64 * W - 1) / (64 * W)), dim3(W * 64), 0, c.st, p, c.slots, c.gw);
}

template <int DT>
void many_slots(const Call& c) {
  const cfr_experts& p = c.p;
  // Tokens per tile by the slots an expert has on average: short tiles let
  // more workgroups share a CU while the weights' bytes are the bound, long ones
  // convert each weight for more tokens once the products are.  Measured (us
  // per call with 32, 64 and 128-token tiles, bfloat16): Qwen3-30B-A3B layer, 64
  // slots per expert 129, 138, 168; 128: 208, 210, 231; 256: 372, 360, 363; 512:
  // -, 675, 663; Qwen3-235B-A22B layer, 64: 441, 436, 466; 128: 729, 692, 711;
  // 256: 1307, 1240, 1182.  Tokens of two and three terms gain nothing from
  // longer tiles (float16 at 128: 329 and 339; float32 at 256: 805 and 811).
  const int64_t per_expert = c.slots / p.cfg.n_experts;
  if constexpr (DT == CFR_BF16) {
    if (per_expert > 224)
      products<DT, 4, 2, 8>(c);
    else if (per_expert > 96)
      products<DT, 2, 2, 4>(c);
    else
      products<DT, 1, 2, 4>(c);
  } else {
    products<DT, 1, 2, 4>(c);
  }
  const int64_t out = (int64_t)c.tokens * ((p.cfg.hidden + 7) / 8);
  const dim3 g((unsigned)std::min<int64_t>((out + kThreads - 1) / kThreads, 256 * 16));
  hipLaunchKernelGGL((k_experts_combine<DT>), g, dim3(kThreads), 0, c.st, p, c.ids, c.tokens, c.y, c.ys);
}

int check_experts_config(const cfr_experts_config* c) {
  if (!c) return fail(CFR_EINVAL, "config is NULL");
  if (c->hidden < 1 || c->hidden > 16384) return fail(CFR_EINVAL, "hidden must be in 1..16384");
  if (c->n_experts < 1 || c->n_experts > 1024) return fail(CFR_EINVAL, "n_experts must be in 1..1024");
  if (c->inter < 1 || c->inter > 16384) return fail(CFR_EINVAL, "inter must be in 1..16384");
  if (c->top < 1 || c->top > 16) return fail(CFR_EINVAL, "top must be in 1..16");
  if (c->max_tokens < 1 || c->max_tokens > 65536) return fail(CFR_EINVAL, "max_tokens must be in 1..65536");
  return CFR_OK;
}

void free_experts(cfr_experts* h) {
  if (!h) return;
  if (h->mem) (void)hipFree(h->mem);
  delete h;
}

// Hands out 256-byte aligned pieces of one allocation; with base null it only adds up.
struct Carver {
  char* base;
  size_t at = 0;
  template <typename T>
  void take(T*& p, size_t bytes) {
    if (base) p = reinterpret_cast<T*>(base + at);
    at += (bytes + 255) / 256 * 256;
  }
};

size_t carve_experts(cfr_experts& h, char* base) {
  const cfr_experts_config& c = h.cfg;
  const size_t E = c.n_experts, slots = (size_t)c.max_tokens * c.top;
  const size_t wide = E * h.ip * (size_t)h.hp;  // weights of one matrix
  Carver k{base};
  k.take(h.gate, wide / 2), k.take(h.up, wide / 2), k.take(h.down, wide / 2);
  k.take(h.gate_s, wide / 32), k.take(h.up_s, wide / 32), k.take(h.down_s, wide / 32);
  k.take(h.order, slots * 4), k.take(h.tiles, (1 + slots / 32 + E) * sizeof(int4)), k.take(h.status, 4);
  k.take(h.xt, 3 * (size_t)c.max_tokens * h.hp * 2);
  k.take(h.h, 3 * slots * h.ip * 2);
  if (slots > kFewSlots) {
    k.take(h.yp, slots * h.hp * 4);
    k.take(h.ye, slots * (h.hp / 64));
  }
  return k.at;
}

}  // namespace
}  // namespace cfr

using namespace cfr;

extern "C" {

int cfr_build_experts(const cfr_experts_config* cfg, const uint8_t* gate_codes, const uint8_t* gate_scales,
                      const uint8_t* up_codes, const uint8_t* up_scales, const uint8_t* down_codes,
                      const uint8_t* down_scales, void* stream, cfr_experts** out) {
  clear_error();
  if (!out) return fail(CFR_EINVAL, "out is NULL");
  *out = nullptr;
  int rc = check_experts_config(cfg);
  if (rc) return rc;
  if (!gate_codes || !gate_scales || !up_codes || !up_scales || !down_codes || !down_scales)
    return fail(CFR_EINVAL, "codes and scales must be non-NULL");
  if ((rc = check_device(cfg->device))) return rc;
  DeviceGuard guard(cfg->device);
  if (!guard.ok) return fail(CFR_EHIP, "cannot select device");
  std::unique_ptr<cfr_experts, void (*)(cfr_experts*)> h(new (std::nothrow) cfr_experts(), free_experts);
  if (!h) return fail(CFR_ENOMEM, "host allocation");
  h->cfg = *cfg;
  h->hp = (cfg->hidden + 255) / 256 * 256, h->sh = h->hp / 64;
  h->ip = (cfg->inter + 255) / 256 * 256, h->si = h->ip / 64;
  hipError_t e = hipMalloc(&h->mem, carve_experts(*h, nullptr));
  if (e != hipSuccess) {
    h->mem = nullptr;
    (void)hipGetLastError();
    return fail(CFR_ENOMEM, std::string("device allocation: ") + hipGetErrorString(e));
  }
  carve_experts(*h, static_cast<char*>(h->mem));
  hipStream_t st = static_cast<hipStream_t>(stream);
  if ((e = hipMemsetAsync(h->status, 0, 4, st)) != hipSuccess) return hipf(e, "status clear");
  const auto lay = [&](const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, int64_t padded_rows,
                       int steps, uint8_t* to, uint32_t* to_s) {
    const int tiles = (int)(padded_rows / 32);
    const int64_t total = (int64_t)cfg->n_experts * tiles * steps * 64;
    const unsigned g = (unsigned)std::min<int64_t>((total + kThreads - 1) / kThreads, 1 << 20);
    hipLaunchKernelGGL(k_experts_layout, dim3(g), dim3(kThreads), 0, st, codes, scales, rows, cols, tiles, steps, total,
                       to, reinterpret_cast<uint8_t*>(to_s), h->status);
  };
  lay(gate_codes, gate_scales, cfg->inter, cfg->hidden, h->ip, h->sh, h->gate, h->gate_s);
  lay(up_codes, up_scales, cfg->inter, cfg->hidden, h->ip, h->sh, h->up, h->up_s);
  lay(down_codes, down_scales, cfg->hidden, cfg->inter, h->hp, h->si, h->down, h->down_s);
  if ((e = hipGetLastError()) != hipSuccess) return hipf(e, "layout launch");
  int32_t seen = 0;
  if ((e = hipMemcpyAsync(&seen, h->status, 4, hipMemcpyDeviceToHost, st)) != hipSuccess ||
      (e = hipStreamSynchronize(st)) != hipSuccess)
    return hipf(e, "layout");
  if (seen) return fail(CFR_EINVAL, "a weight block has a NaN scale (255)");
  *out = h.release();
  return CFR_OK;
}

int cfr_experts_forward(cfr_experts* h, const void* x, int32_t dtype, int64_t x_stride, const int32_t* expert_ids,
                        const float* gate_w, int32_t tokens, void* y, int64_t y_stride, void* stream) {
  clear_error();
  if (!h) return fail(CFR_EINVAL, "experts handle is NULL");
  const int bytes = dtype_bytes(dtype), H = h->cfg.hidden;
  if (!bytes) return fail(CFR_EINVAL, "dtype must be CFR_F32, CFR_BF16 or CFR_F16");
  if (tokens < 0 || tokens > h->cfg.max_tokens) return fail(CFR_EINVAL, "tokens must be in 0..max_tokens");
  if (tokens == 0) return CFR_OK;
  if (!x || !expert_ids || !gate_w || !y) return fail(CFR_EINVAL, "x, expert_ids, gate_w and y must be non-NULL");
  if (tokens > 1 && (x_stride < H || y_stride < H)) return fail(CFR_EINVAL, "row strides must be at least hidden");
  if (reinterpret_cast<uintptr_t>(x) % bytes || reinterpret_cast<uintptr_t>(y) % bytes)
    return fail(CFR_EINVAL, "x and y must be aligned to their type");
  if (reinterpret_cast<uintptr_t>(expert_ids) % 4 || reinterpret_cast<uintptr_t>(gate_w) % 4)
    return fail(CFR_EINVAL, "expert_ids and gate_w must be aligned to four bytes");
  const Span to = span(y, dtype, y_stride, tokens, H);
  const int64_t routed = (int64_t)tokens * h->cfg.top;  // int32 ids and fp32 weights, four bytes each
  if (overlap(span(x, dtype, x_stride, tokens, H), to) || overlap(span(expert_ids, CFR_F32, routed, 1, routed), to) ||
      overlap(span(gate_w, CFR_F32, routed, 1, routed), to))
    return fail(CFR_EINVAL, "y overlaps x, expert_ids or gate_w");
  DeviceGuard guard(h->cfg.device);
  if (!guard.ok) return fail(CFR_EHIP, "cannot select device");
  const Call c = {*h,
                  x,
                  x_stride,
                  expert_ids,
                  gate_w,
                  tokens,
                  routed,
                  y,
                  y_stride,
                  rows_aligned16(x, x_stride, tokens, bytes),
                  static_cast<hipStream_t>(stream)};
  if (c.slots <= kFewSlots) {
    if (dtype == CFR_F32)
      few_slots<CFR_F32>(c);
    else if (dtype == CFR_BF16)
      few_slots<CFR_BF16>(c);
    else
      few_slots<CFR_F16>(c);
  } else {
    if (dtype == CFR_F32)
      many_slots<CFR_F32>(c);
    else if (dtype == CFR_BF16)
      many_slots<CFR_BF16>(c);
    else
      many_slots<CFR_F16>(c);
  }
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? CFR_OK : hipf(e, "experts launch");
}

int cfr_experts_status(cfr_experts* h, int32_t* flags) {
  clear_error();
  if (!h || !flags) return fail(CFR_EINVAL, "handle and flags must be non-NULL");
  DeviceGuard guard(h->cfg.device);
  if (!guard.ok) return fail(CFR_EHIP, "cannot select device");
  hipError_t e;
  if ((e = hipDeviceSynchronize()) != hipSuccess) return hipf(e, "status sync");
  if ((e = hipMemcpy(flags, h->status, sizeof(int32_t), hipMemcpyDeviceToHost)) != hipSuccess)
    return hipf(e, "status read");
  // waited for: the next call may be on a stream that the null stream does not hold up
  if ((e = hipMemsetAsync(h->status, 0, sizeof(int32_t), nullptr)) != hipSuccess ||
      (e = hipStreamSynchronize(nullptr)) != hipSuccess)
    return hipf(e, "status clear");
  return CFR_OK;
}

void cfr_experts_free(cfr_experts* h) {
  if (!h) return;
  DeviceGuard guard(h->cfg.device);
  (void)hipDeviceSynchronize();
  free_experts(h);
}

}  // extern "C"
