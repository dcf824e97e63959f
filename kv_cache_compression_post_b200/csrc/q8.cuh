// The 8-bit block-scaled K/V cache: what its kernels share (views, E4M3 conversions,
// the split of (head, row tile, key tile) work over CTAs) and their launchers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <cuda_runtime.h>

#include "kvb.h"
#include "kvb_device.cuh"

namespace kvb {

constexpr int kQ8MaxHeads = 1024;
constexpr int kQ8MaxCapacity = 1 << 24;
constexpr int kQ8MaxRows = 1 << 30;
constexpr int kQ8MaxCtas = 160;  // grid cap of the kernels that split work (>= the SMs of a B200)

struct Q8View {
  int H, d, cap, block;
  int shift;  // block = 1 << shift
  const uint8_t* K;
  const uint8_t* V;
  const float* ks;
  const float* vs;
  const int* len;
  int* status;
};

__device__ __forceinline__ int q8_len(const int* len, int h, int cap) { return min(max(len[h], 0), cap); }

// four E4M3 codes -> four fp16 (exact).  In PTX, on the halves of the word: the two
// conversions take 5 clk of a warp's ALU; through the header's conversion of a 16-bit
// storage type, which goes by way of two 16-bit fields, they took 15.
struct F16x4 {
  uint32_t lo, hi;
};
__device__ __forceinline__ F16x4 e4m3x4_to_f16x4(uint32_t c) {
  F16x4 r;
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(r.lo), "=r"(r.hi)
      : "r"(c));
  return r;
}
__device__ __forceinline__ float2 f16x2_to_f32x2(uint32_t h) { return __half22float2(*reinterpret_cast<const __half2*>(&h)); }
__device__ __forceinline__ float4 e4m3x4_to_f32x4(uint32_t c) {
  const F16x4 h = e4m3x4_to_f16x4(c);
  const float2 a = f16x2_to_f32x2(h.lo), b = f16x2_to_f32x2(h.hi);
  return make_float4(a.x, a.y, b.x, b.y);
}
// four floats -> four E4M3 codes, to nearest even, saturating
__device__ __forceinline__ uint32_t f32x4_to_e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
      "mov.b32 %0, {l, h};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack_bf16x2(uint32_t w) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}
// 2^e as a float, e in [-126, 127]
__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }
// floor(log2 |x|) of a normal float; -126 or less for zero and subnormals
__device__ __forceinline__ int exponent_of(float x) { return static_cast<int>((__float_as_uint(x) >> 23) & 0xFFu) - 127; }

// The row sums add weights / V scale, which passes fp32's range where a head's scales are
// small (zeros have 2^-100; a million of them did).  They count in units of the power of two
// of the head's first scale: an exact factor, taken out of outputs and lse in the end.
__device__ __forceinline__ int sum_unit(const float* vs) { return min(max(exponent_of(__ldg(vs)), -126), 126); }
// what a row's sum divides its outputs by: a row that saw nothing, its every score -inf, is zeros
__device__ __forceinline__ float inverse_sum(float l) { return l == 0.f ? 0.f : 1.f / l; }

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ------------------------------------------------------------------ work split
// A unit is (head h, row tile r); it walks the T[h] key tiles its head holds.  The
// key tiles of every unit, in the order of (h, r), are one sequence of costs (w per
// tile, wlast in a head's last row tile); CTA c of G takes the tiles that start in
// [ceil(c total / G), ceil((c+1) total / G)).  Heads of very different length, one
// row or many, thus load every SM alike.  A unit cut between CTAs leaves one partial
// per piece: in a CTA's slot 0 for its first piece, slot 1 for its last one.
// Where there are at most half as many units as CTAs (chunk > 0) no CTA takes parts of
// two units: each unit is cut into ceil(T / chunk) equal pieces, chunk such that the CTAs
// suffice, and a CTA has one piece.  A CTA's second piece begins when its
// first is done, with every latency of a beginning once more: 4 of 25 us for 12 heads of
// 15600 tokens.
struct Q8Sched {
  long long C[kQ8MaxHeads + 1];  // cost before each head (chunk > 0: CTAs)
  int T[kQ8MaxHeads];
  long long total;
  int G;
  bool small;  // total * G < 2^32: 32-bit quotients do (a 64-bit one takes ~400 clk)
  int chunk;
};

struct Q8Split {
  const Q8Sched* s;
  int H, nrt;      // row tiles per head
  int w, wlast;    // cost of a key tile; in the last row tile
  __device__ int wt(int r) const { return r == nrt - 1 ? wlast : w; }
  __device__ long long start(int h, int r) const { return s->C[h] + static_cast<long long>(r) * w * s->T[h]; }
  __device__ int cta_of(long long x) const {
    if (s->small) return static_cast<int>((static_cast<uint32_t>(x) * static_cast<uint32_t>(s->G)) / static_cast<uint32_t>(s->total));
    return static_cast<int>((x * s->G) / s->total);
  }
  __device__ long long lo(int c) const {
    if (s->small)
      return (static_cast<uint32_t>(c) * static_cast<uint32_t>(s->total) + static_cast<uint32_t>(s->G - 1)) / static_cast<uint32_t>(s->G);
    return (static_cast<long long>(c) * s->total + s->G - 1) / s->G;
  }
};

// Filled by the whole CTA (blockDim.x a multiple of 32); `min_cost`: a CTA's share is
// at least this much.  Ends with a __syncthreads().
__device__ __forceinline__ void q8_build_sched(Q8Sched* s, const int* len, int cap, int H, int nrt, int tile, int w,
                                               int wlast, int grid, int min_cost, bool may_chunk = false) {
  for (int h = threadIdx.x; h < H; h += blockDim.x) s->T[h] = (q8_len(len, h, cap) + tile - 1) / tile;
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    long long per = static_cast<long long>(nrt - 1) * w + wlast;
    int chunk = 0;
    if (may_chunk && static_cast<long long>(H) * nrt * 2 <= grid) {
      int sum = 0;  // key tiles of all units: below 2^25 tokens x heads
      for (int h = lane; h < H; h += 32) sum += s->T[h] * nrt;
      sum = warp_sum_int(sum);
      // sum / chunk pieces, and at most one more per unit: no more than the CTAs
      const int spare = grid - H * nrt;
      chunk = max(min_cost, (sum + spare - 1) / spare);
    }
    long long carry = 0;
    for (int b = 0; b < H; b += 32) {
      long long n = b + lane < H ? per * s->T[b + lane] : 0;
      if (chunk > 0 && b + lane < H) n = static_cast<long long>((s->T[b + lane] + chunk - 1) / chunk) * nrt;
      long long x = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (b + lane < H) s->C[b + lane] = carry + x - n;
      carry += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) {
      s->C[H] = carry;
      s->total = carry;
      const long long g = carry / min_cost;
      s->G = static_cast<int>(g < 1 ? 1 : (g < grid ? g : grid));
      s->chunk = chunk;
      if (chunk > 0) s->G = static_cast<int>(carry < 1 ? 1 : carry);
      s->small = (carry + 1) * (s->G + 1) < (1ll << 32);
    }
  }
  __syncthreads();
}

struct Q8Piece {
  int h, r, j0, j1;
  int npieces;  // pieces the unit is cut into
  int which;    // this piece's slot
  int cfirst;   // CTA of the unit's first piece
  int wfirst;   // slot of it
};

__device__ __forceinline__ void q8_unit_pieces(const Q8Split& S, int h, int r, Q8Piece& pc) {
  const long long cu = S.start(h, r);
  const int w = S.wt(r);
  const int cf = S.cta_of(cu), cl = S.cta_of(cu + static_cast<long long>(w) * (S.s->T[h] - 1));
  pc.npieces = cl - cf + 1;
  pc.cfirst = cf;
  // the key tile before this unit, in the order of all units, starts wprev earlier
  const int wprev = r > 0 ? S.w : S.wlast;
  pc.wfirst = (cu == 0 || S.cta_of(cu - wprev) < cf) ? 0 : 1;
}

// The pieces of one CTA, in order; every role of a CTA walks the same sequence.
struct Q8Walk {
  int h = 0, r = 0, j = 0;
  long long hi = 0;
  bool first = true;

  __device__ void skip_done(const Q8Split& S) {
    while (h < S.H && (S.s->T[h] == 0 || j >= S.s->T[h])) {
      j = 0;
      if (S.s->T[h] != 0 && ++r < S.nrt) continue;
      ++h;
      r = 0;
    }
  }
  __device__ void init(const Q8Split& S, int cta) {
    first = true;
    h = S.H;
    if (S.s->total <= 0 || cta >= S.s->G) return;
    if (S.s->chunk > 0) {
      int a = 0, b = S.H;  // the last head with C[h] <= cta
      while (b - a > 1) {
        const int m = (a + b) / 2;
        if (S.s->C[m] <= cta) a = m;
        else b = m;
      }
      h = a;
      hi = cta;
      return;
    }
    const long long x = S.lo(cta);
    hi = S.lo(cta + 1);
    int a = 0, b = S.H;  // the last head with C[h] <= x
    while (b - a > 1) {
      const int m = (a + b) / 2;
      if (S.s->C[m] <= x) a = m;
      else b = m;
    }
    h = a;
    r = 0;
    j = 0;
    if (S.s->T[h] > 0) {
      const long long unit = static_cast<long long>(S.w) * S.s->T[h];
      r = S.s->small ? static_cast<int>(static_cast<uint32_t>(x - S.s->C[h]) / static_cast<uint32_t>(unit))
                     : static_cast<int>((x - S.s->C[h]) / unit);
      if (r > S.nrt - 1) r = S.nrt - 1;
      const int w = S.wt(r);
      const long long d = x - S.start(h, r) + w - 1;
      j = S.s->small ? static_cast<int>(static_cast<uint32_t>(d) / static_cast<uint32_t>(w)) : static_cast<int>(d / w);
    }
    skip_done(S);
  }
  // whole: with the unit's pieces (a caller in a hurry finds them later, q8_unit_pieces)
  __device__ bool next(const Q8Split& S, Q8Piece& pc, bool whole = true) {
    if (h >= S.H) return false;
    if (S.s->chunk > 0) {  // one piece
      const uint32_t T = S.s->T[h], np = (T + S.s->chunk - 1) / S.s->chunk;
      const uint32_t i = static_cast<uint32_t>(hi - S.s->C[h]), unit = i / np, k = i - unit * np;
      pc.h = h;
      pc.r = unit;
      pc.j0 = static_cast<int>(k * T / np);  // T <= 2^18, np <= 160
      pc.j1 = static_cast<int>((k + 1) * T / np);
      pc.npieces = np;
      pc.which = pc.wfirst = 0;
      pc.cfirst = static_cast<int>(hi - k);
      h = S.H;
      return true;
    }
    const long long cu = S.start(h, r);
    const int w = S.wt(r);
    if (cu + static_cast<long long>(w) * j >= hi) return false;
    const long long je = S.s->small ? static_cast<uint32_t>(hi - cu + w - 1) / static_cast<uint32_t>(w) : (hi - cu + w - 1) / w;
    const int T = S.s->T[h];
    pc.h = h;
    pc.r = r;
    pc.j0 = j;
    pc.j1 = je < T ? static_cast<int>(je) : T;
    if (whole) q8_unit_pieces(S, h, r, pc);
    pc.which = first ? 0 : 1;
    first = false;
    j = pc.j1;
    skip_done(S);
    return true;
  }
};

// The first r with (h * n + r) % G == blockIdx.x: this CTA's first turn at n things of
// head h that all CTAs share out.
__device__ __forceinline__ int q8_first_turn(int h, int n, int G) {
  const int at = static_cast<int>(static_cast<long long>(h) * n % G);
  const int r = static_cast<int>(blockIdx.x) - at;
  return r < 0 ? r + G : r;
}

// ------------------------------------------------------------------ launchers
struct Q8AttendArgs {
  Q8View c;
  int Nq;
  float scale;
  const void* Q;
  void* O;
  float* lse;
  float* part;  // partials: q8_part_floats(d) floats
  unsigned long long* flag;  // the row-tile kernels' piece flags: kQ8RowFlags
  unsigned long long tag;    // of this call, nonzero
};

struct Q8MassArgs {
  Q8View c;
  int Nq;
  float scale;
  const void* Q;
  const float* lse;
  float decay;
  const float* prev;
  float* mass;
};

cudaError_t launch_q8_attend_rows(const Q8AttendArgs& a, int n_sm, cudaStream_t st);  // bf16, 16-row tiles
cudaError_t launch_q8_attend_f32(const Q8AttendArgs& a, int n_sm, cudaStream_t st);   // f32, CUDA cores
cudaError_t launch_q8_mass_rows(const Q8MassArgs& a, int n_sm, cudaStream_t st);
cudaError_t launch_q8_mass_f32(const Q8MassArgs& a, int n_sm, cudaStream_t st);

constexpr int kQ8RowFlags = kQ8MaxCtas * 2;
// floats of partials the row-tile kernels need: two slots per CTA of 16 rows and
// their maxima and sums
inline size_t q8_part_floats(int d) { return static_cast<size_t>(kQ8MaxCtas) * 2 * (16 * d + 32); }

// Scratch of the tensor-core kernels for chunks of queries: the queries' E4M3 parts and
// row coefficients, and for attention the partials of cut units (two slots of two
// 128-row tiles per CTA) with their arrival counters.
struct Q8ChunkScratch {
  uint8_t* hi;           // [H][Nq][d]
  uint8_t* lo;
  float* coef;           // [H][Nq]
  float* part;           // q8_chunk_part_floats(d)
  unsigned int* cnt;     // [H][pairs of query tiles][2], or kQ8MassCounters
};
inline size_t q8_chunk_part_floats(int d) { return static_cast<size_t>(4) * kQ8MaxCtas * (128 * d + 256); }
// lse: of the rows, or null; rows of -inf, which weigh nothing whatever they hold, become zeros
cudaError_t launch_q8_split_q(const void* Q, const float* lse, long long rows, int d, float scale,
                              const Q8ChunkScratch& s, int ncnt, int n_sm, cudaStream_t st);
cudaError_t launch_q8_mass_chunk(const Q8MassArgs& a, const Q8ChunkScratch& s, int n_sm, cudaStream_t st);
constexpr int kQ8MassCounters = kQ8MaxCtas * 2 * 8;  // arrival counters of the weights' cut blocks
cudaError_t launch_q8_attend_chunk(const Q8AttendArgs& a, const Q8ChunkScratch& s, int n_sm, cudaStream_t st);

// Rows per head from which a bf16 call takes the tcgen05 kernel (128 or 256 rows at once,
// however few there are) instead of 16-row tiles, each of which reads the cache again.  One
// bound for attention and weights, by what the cache may hold (lengths are on the device):
// it lies near the crossing of the weights, and of the attention with eight heads and more.
// Few heads, whose long units a CTA alone merges in the tcgen05 kernel, cross later, at 112
// (4 x 65536) to 384 rows (1 x 131072), and short caches at hundreds: there the bound costs
// up to three times the tiles' time.  us of a captured call, 16-row tiles / tcgen05:
//   head_dim 128  heads x tokens   32 rows    48 rows    64 rows    80 rows    96 rows    128 rows   256 rows
//   attention     12 x 15616       36 / 61    45 / 61    53 / 61    69 / 60    70 / 60    93 / 61    164 / 72
//                 24 x 15616       54 / 71    71 / 71    96 / 71    113 / 71   128 / 71   167 / 72   308 / 84
//                 8 x 131072       113 / 151  159 / 151  227 / 150  294 / 150  296 / 150  429 / 150  790 / 175
//                 1 x 131072       36 / 168   40 / 168   46 / 168   50 / 170   56 / 170   68 / 170   111 / 203
//                 1 x 8192         15 / 40    15 / 41    15 / 40    16 / 41    16 / 41    16 / 41    20 / 43
//                 64 x 1024        30 / 46    37 / 46    42 / 47    48 / 47    53 / 47    64 / 47    107 / 37
//   weights       12 x 15616       20 / 29    25 / 29    30 / 29    35 / 29    40 / 29    50 / 29    91 / 30
//                 8 x 131072       74 / 113   96 / 113   119 / 113  141 / 113  164 / 113  210 / 113  465 / 114
//                 1 x 131072       14 / 22    17 / 23    20 / 23    24 / 23    27 / 23    34 / 23    61 / 25
//                 1 x 8192         4 / 10     5 / 10     6 / 10     7 / 10     8 / 10     10 / 10    17 / 11
//                 64 x 1024        9 / 18     10 / 18    12 / 18    14 / 18    16 / 18    20 / 18    34 / 19
//   head_dim 64
//   attention     12 x 15616       23 / 46    28 / 45    34 / 46    43 / 46    44 / 46    58 / 47    100 / 53
//                 8 x 131072       69 / 117   96 / 118   137 / 118  178 / 118  178 / 118  259 / 119  448 / 138
//   weights       12 x 15616       14 / 27    18 / 28    21 / 28    25 / 28    28 / 28    35 / 28    62 / 29
//                 8 x 131072       54 / 109   68 / 110   82 / 111   96 / 111   110 / 111  139 / 111  260 / 111
inline int q8_chunk_rows(long long heads, long long capacity) { return heads * capacity <= 131072 ? 81 : 49; }

struct Q8EvictArgs {
  Q8View src;
  const float* mass;
  uint8_t* K;
  uint8_t* V;
  float* ks;
  float* vs;
  int* len;
  float* to_mass;
  int cap;  // of the destination
  int budget, sink, recent;
  int* kept;  // [H][budget]
};
cudaError_t launch_q8_evict(const Q8EvictArgs& a, cudaStream_t st);

struct Q8AppendArgs {
  int H, d, cap, block;
  const void* X[2];  // K, V
  long long hs[2], ts[2];
  uint8_t* code[2];
  float* scale[2];
  int n;
  const int* start;
  int* len;
  float* mass;
  int* status;
};
cudaError_t launch_q8_append(const Q8AppendArgs& a, kvb_dtype dtype, cudaStream_t st);

}  // namespace kvb
