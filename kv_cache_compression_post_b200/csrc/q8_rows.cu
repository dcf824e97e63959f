// Attention and attention weights over the 8-bit cache for a few rows per head: the
// single-token form, and query heads that share a K/V head.
//
// Reading the cache once is the bound (2 bytes per token and channel), so the work is
// split over its tokens (Q8Split) and every warp streams 32 tokens at a time through a
// ring of its own in shared memory (cp.async, no barrier between warps) into the
// fragments of mma.sync.m16n8k16: 16 rows x 8 tokens, or with at most eight rows
// 16 tokens (or channels) x 8 rows, half the instructions.  What the layout relies on: a
// contraction may run over the channels, and over the tokens, in any order that both
// operands share.  Lane (g, t) = (lane / 4, lane % 4) takes 16 contiguous bytes of token
// g's K row and uses them as four MMA steps, so Q is fetched in that order of channels;
// it takes 16 contiguous bytes of V for the four tokens its P columns stand for, and
// row or column n of MMA j is channel 16 n + j.  Codes widen to fp16 exactly, four per
// word in two instructions, and Q enters as fp16 times a power of two per row (bf16 has
// 8 bits, fp16 11, so nothing is lost above 2^-14 of the row's largest).
// What bounds it (at most eight rows): memory.  8 rows over 8 heads, 819200 tokens in all,
// take 50 us, 49 with the arithmetic taken out; a long cache streams at 5.4 TB/s, and a
// call takes ~10 us besides (lengths, split and query 5.6, a merge of pieces 4), half
// of the 19 us of one row over 12 heads of 15600 tokens.  E4M3 operands of mma.sync do
// not help, they are widened all the same.
//
// Softmax in the log2 domain.  With ks, vs the scales of a token's block,
//     x = (q.k) ks scale log2 e,   P = 2^(x + log2 vs - m + kBias),
// m the running maximum of x + log2 vs: V's scale rides in the exponent at no cost,
// P stays below fp16's largest, and the row sum adds P / vs per block (in units of
// sum_unit).  Sums, maxima and partial outputs are fp32.  P is rounded to fp16: its 11 bits
// hold down to 2^-14, 2^-20 of the largest P or less, its smallest steps (2^-24) below that;
// bf16 would hold any, with 8 bits of each.
#include "host_util.h"
#include "q8.cuh"
#include "sm100.cuh"

namespace kvb {
using namespace sm100;

namespace {

constexpr int kThreads = 256;  // of the weights' kernels
constexpr int kWarps = kThreads / 32;
// of the attention's; ten or twelve warps, with their registers cut to fit, were slower
// (at most eight rows x 131072: 51 us with 256 threads, 53 with 320, 52 with 384, 54 with 192)
constexpr int kRowsThreads = 256, kFewThreads = 256;
constexpr int kRing = 2;  // stages of a warp's ring (three: 1 to 2 % slower)
constexpr int kTile = 64;    // tokens per key tile of the split
constexpr int kSub = 32;     // tokens a warp takes at a time
constexpr int kRows = 16;    // rows per row tile
constexpr int kMinTiles = 4;  // of a CTA of the f32 kernel

__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

// Query fragments: row g and, of a 16-row tile (I 2), g + 8 of this lane, channels
// 64 hb + 16 t .. + 15 in the order the K bytes come.  coef[i]: what turns a raw dot
// product of row g + 8 i into log2 units (but for the token's scale).
template <int D, int I>
struct QFrag {
  static constexpr int kI = I;
  uint32_t a[D / 16][2 * kI];  // [16-channel step][(half of the step) * kI + row]
  float coef[kI];
  uint4 raw[kI][D / 32];

  __device__ __forceinline__ void fetch(const __nv_bfloat16* Q, int rows, int g, int t) {
#pragma unroll
    for (int i = 0; i < kI; ++i) {
      const int row = g + 8 * i;
#pragma unroll
      for (int hb = 0; hb < D / 64; ++hb)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          raw[i][hb * 2 + k] = row < rows ? *(reinterpret_cast<const uint4*>(Q + static_cast<size_t>(row) * D + hb * 64 + t * 16) + k)
                                          : make_uint4(0u, 0u, 0u, 0u);
    }
  }
  __device__ __forceinline__ void widen(float scale) {
#pragma unroll
    for (int i = 0; i < kI; ++i) {
      const uint4(&w)[D / 32] = raw[i];
      float mx = 0.f;
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        const uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = unpack_bf16x2(u[e]);
          mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      }
      mx = quad_max(mx);
      const int e = min(max(exponent_of(mx), -100), 126);
      const float down = pow2f(-e);
      // an infinite element makes its row NaN, also where it would send every score to -inf
      coef[i] = mx == INFINITY ? NAN : pow2f(e) * scale * kLog2e;
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        // 8 channels: two MMA steps, (0,1) and (2,3) of each to their two halves
        const uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
        for (int e2 = 0; e2 < 4; ++e2) {
          const float2 f = unpack_bf16x2(u[e2]);
          a[k * 2 + (e2 >> 1)][i + kI * (e2 & 1)] = pack_f16x2(f.x * down, f.y * down);
        }
      }
    }
  }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Where the 16-byte unit c of row `row` lies in a stage: turned so that the fragments'
// reads below meet no bank twice (rows of 128 bytes).
template <int D>
__device__ __forceinline__ int k_unit(int row, int c) { return D == 128 ? c ^ ((row & 1) << 2) : c; }
template <int D>
__device__ __forceinline__ int v_unit(int row, int c) { return D == 128 ? c ^ (row & 6) : c ^ ((row >> 1) & 3); }

// Fetch K and V rows of 32 tokens from `kb` (token index in the head) into a stage;
// rows past the last held token repeat it (masked later).
template <int D>
__device__ __forceinline__ void fetch(uint32_t stage, const uint8_t* K, const uint8_t* V, int kb, int last, int lane) {
  constexpr int kU = D / 16;
#pragma unroll
  for (int i = 0; i < kU; ++i) {
    const int row = (lane + 32 * i) / kU, c = (lane + 32 * i) % kU;
    const size_t at = static_cast<size_t>(min(kb + row, last)) * D + c * 16;
    cp_async16(stage + row * D + k_unit<D>(row, c) * 16, K + at);
    cp_async16(stage + 32 * D + row * D + v_unit<D>(row, c) * 16, V + at);
  }
}

// K words of 32 tokens
template <int D>
struct KWords {
  uint4 w[4][D / 64];
  __device__ __forceinline__ void load(const uint8_t* stage, int g, int t) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int hb = 0; hb < D / 64; ++hb)
        w[j][hb] = *reinterpret_cast<const uint4*>(stage + (8 * j + g) * D + k_unit<D>(g, hb * 4 + t) * 16);
  }
  // straight from global memory, for the weights, which read K once and nothing else
  __device__ __forceinline__ void load_global(const uint8_t* K, int kb, int last, int g, int t) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int key = min(kb + 8 * j + g, last);
#pragma unroll
      for (int hb = 0; hb < D / 64; ++hb)
        w[j][hb] = __ldg(reinterpret_cast<const uint4*>(K + static_cast<size_t>(key) * D + hb * 64 + t * 16));
    }
  }
  // s[j]: raw dot products of rows g (0, 1) and g + 8 (2, 3) with tokens 8 j + 2 t, + 1
  __device__ __forceinline__ void dots(const QFrag<D, 2>& q, float (&s)[4][4]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int k = 0; k < 4; ++k) s[j][k] = 0.f;
#pragma unroll
      for (int hb = 0; hb < D / 64; ++hb) {
        const uint32_t u[4] = {w[j][hb].x, w[j][hb].y, w[j][hb].z, w[j][hb].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const F16x4 k4 = e4m3x4_to_f16x4(u[i]);
          mma_16816(s[j], q.a[hb * 4 + i], k4.lo, k4.hi);
        }
      }
    }
  }
  // at most eight rows: the tokens are the product's 16 rows and the queries its 8 columns,
  // half the instructions.  s[u]: tokens 16 u + g (0, 1) and 16 u + g + 8 (2, 3) with rows
  // 2 t, + 1.  Two chains of products each, so that they do not wait on one another.
  __device__ __forceinline__ void dots_few(const QFrag<D, 1>& q, float (&s)[2][4]) const {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float c[2][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) c[0][k] = c[1][k] = 0.f;
#pragma unroll
      for (int hb = 0; hb < D / 64; ++hb) {
        const uint4 &x = w[2 * u][hb], &y = w[2 * u + 1][hb];
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const F16x4 x4 = e4m3x4_to_f16x4(xs[i]), y4 = e4m3x4_to_f16x4(ys[i]);
          const uint32_t a[4] = {x4.lo, y4.lo, x4.hi, y4.hi};
          mma_16816(c[i & 1], a, q.a[hb * 4 + i][0], q.a[hb * 4 + i][1]);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) s[u][k] = c[0][k] + c[1][k];
    }
  }
};

template <int D>
struct VWords {
  static constexpr int kW = D / 32;  // 32-bit words per lane and token (8 lanes per row)
  uint32_t w[2][4][kW];
  __device__ __forceinline__ void load(const uint8_t* stage, int g, int t) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int row = 16 * u + 2 * t + (k & 1) + 8 * (k >> 1);
        const uint8_t* p = stage + row * D;
        if constexpr (D == 128) {
          const uint4 x = *reinterpret_cast<const uint4*>(p + v_unit<D>(row, g) * 16);
          w[u][k][0] = x.x, w[u][k][1] = x.y, w[u][k][2] = x.z, w[u][k][3] = x.w;
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(p + v_unit<D>(row, g >> 1) * 16 + (g & 1) * 8);
          w[u][k][0] = x.x, w[u][k][1] = x.y;
        }
      }
  }
  // o[j] += P[16 tokens of half u] V, channel (D / 8) n + j in column n
  __device__ __forceinline__ void accumulate(int u, const uint32_t (&p)[4], float (&o)[D / 8][4]) const {
#pragma unroll
    for (int q = 0; q < kW; ++q) {
      const uint32_t a0 = __byte_perm(w[u][0][q], w[u][1][q], 0x5140), a1 = __byte_perm(w[u][0][q], w[u][1][q], 0x7362);
      const uint32_t b0 = __byte_perm(w[u][2][q], w[u][3][q], 0x5140), b1 = __byte_perm(w[u][2][q], w[u][3][q], 0x7362);
      const F16x4 x0 = e4m3x4_to_f16x4(a0), y0 = e4m3x4_to_f16x4(b0), x1 = e4m3x4_to_f16x4(a1), y1 = e4m3x4_to_f16x4(b1);
      mma_16816(o[4 * q + 0], p, x0.lo, y0.lo);
      mma_16816(o[4 * q + 1], p, x0.hi, y0.hi);
      mma_16816(o[4 * q + 2], p, x1.lo, y1.lo);
      mma_16816(o[4 * q + 3], p, x1.hi, y1.hi);
    }
  }
  // at most eight rows: channels are the product's rows.  o[2 q + j]: channels (D / 8) g +
  // 4 q + 2 j (0, 1) and the next (2, 3) of rows 2 t, + 1; p: row g, tokens 2 t, + 1 and + 8
  __device__ __forceinline__ void accumulate_few(int u, uint32_t p0, uint32_t p1, float (&o)[D / 16][4]) const {
#pragma unroll
    for (int q = 0; q < kW; ++q) {
      const uint32_t a0 = __byte_perm(w[u][0][q], w[u][1][q], 0x5140), a1 = __byte_perm(w[u][0][q], w[u][1][q], 0x7362);
      const uint32_t b0 = __byte_perm(w[u][2][q], w[u][3][q], 0x5140), b1 = __byte_perm(w[u][2][q], w[u][3][q], 0x7362);
      const F16x4 x0 = e4m3x4_to_f16x4(a0), y0 = e4m3x4_to_f16x4(b0), x1 = e4m3x4_to_f16x4(a1), y1 = e4m3x4_to_f16x4(b1);
      const uint32_t f0[4] = {x0.lo, x0.hi, y0.lo, y0.hi}, f1[4] = {x1.lo, x1.hi, y1.lo, y1.hi};
      mma_16816(o[2 * q], f0, p0, p1);
      mma_16816(o[2 * q + 1], f1, p0, p1);
    }
  }
};

// 8 x 8 of 16 bits: lane (g, t) gives row g, columns 2 t, + 1 and receives those of the transpose
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

template <int D>
constexpr size_t slot_floats() { return static_cast<size_t>(kRows) * D + 2 * kRows; }

// what the warps of a CTA leave for their merge
template <int D, int WARPS, int ROWS>
struct RowsShared {
  float o[WARPS][ROWS][D + 4];
  float m[WARPS][ROWS], l[WARPS][ROWS];
};

// The scales of 32 tokens' two halves: K's, log2 and reciprocal (in the sums' units) of V's
struct StepScales {
  float kf[2], lv[2], iv[2];
};

// A warp's running softmax and outputs of up to 16 rows.
template <int D>
struct RowsAcc {
  static constexpr int kTileRows = 16, kThreads = kRowsThreads, kWarps = kThreads / 32;
  static constexpr float kBias = 8.f;
  using Shared = RowsShared<D, kWarps, kTileRows>;
  QFrag<D, 2> q;
  float o[D / 8][4];
  float m[2], l[2];  // rows g, g + 8

  __device__ __forceinline__ void begin(float scale, int) {
    q.widen(scale);
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[j][k] = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) m[i] = -INFINITY, l[i] = 0.f;
  }
  __device__ __forceinline__ void step(const KWords<D>& kw, const uint8_t* v_stage, const StepScales& sc, int kb, int end,
                                       int g, int t) {
    float s[4][4];
    kw.dots(q, s);
    float mt[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int key = kb + 8 * j + 2 * t + (k & 1);
        const float x = fmaf(s[j][k], q.coef[k >> 1] * sc.kf[j >> 1], sc.lv[j >> 1]);
        s[j][k] = key < end ? x : -INFINITY;
        mt[k >> 1] = fmaxf(mt[k >> 1], s[j][k]);
      }
    bool moved = false;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      mt[i] = quad_max(mt[i]);
      moved |= mt[i] > m[i];
    }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float mn = fmaxf(m[i], mt[i]);
        const float al = mn == -INFINITY ? 1.f : exp2f(m[i] - mn);
        m[i] = mn;
        l[i] *= al;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          o[j][2 * i] *= al;
          o[j][2 * i + 1] *= al;
        }
      }
    }
    VWords<D> vw;
    vw.load(v_stage, g, t);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint32_t p[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        // a row whose every score is -inf so far (NaN queries aside) keeps P = 0
        const float b = (m[i] == -INFINITY ? 0.f : -m[i]) + kBias;
        float r = 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float x = ex2_approx(s[2 * u + j][2 * i] + b), y = ex2_approx(s[2 * u + j][2 * i + 1] + b);
          r += x + y;
          p[2 * j + i] = pack_f16x2(x, y);
        }
        l[i] = fmaf(r, sc.iv[u], l[i]);
      }
      vw.accumulate(u, p, o);
    }
  }
  __device__ __forceinline__ void leave(Shared& sh, int warp, int rows, int g, int t) {
#pragma unroll
    for (int i = 0; i < 2; ++i) l[i] = quad_sum(l[i]);
    if (t == 0) {
#pragma unroll
      for (int i = 0; i < 2; ++i) sh.m[warp][g + 8 * i] = m[i], sh.l[warp][g + 8 * i] = l[i];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int row = g + 8 * (k >> 1);
      if (row >= rows) continue;
      float* to = &sh.o[warp][row][(2 * t + (k & 1)) * (D / 8)];
#pragma unroll
      for (int j = 0; j < D / 8; j += 4)
        *reinterpret_cast<float4*>(to + j) = make_float4(o[j][k], o[j + 1][k], o[j + 2][k], o[j + 3][k]);
    }
  }
};

// Of up to eight: rows 2 t, 2 t + 1 of this lane.  The maximum moves only when a score
// passes it by kLag, which a vote finds without reducing over the lanes.
template <int D>
struct FewAcc {
  static constexpr int kTileRows = 8, kThreads = kFewThreads, kWarps = kThreads / 32;
  static constexpr float kBias = 6.f, kLag = 8.f;  // P <= 2^(kBias + kLag) < 65504
  using Shared = RowsShared<D, kWarps, kTileRows>;
  QFrag<D, 1> q;
  float o[D / 16][4];
  float coef[2], m[2], l[2];

  __device__ __forceinline__ void begin(float scale, int t) {
    q.widen(scale);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      coef[r] = __shfl_sync(0xffffffffu, q.coef[0], 4 * (2 * t + r));
      m[r] = -INFINITY, l[r] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[j][k] = 0.f;
  }
  __device__ __forceinline__ void step(const KWords<D>& kw, const uint8_t* v_stage, const StepScales& sc, int kb, int end,
                                       int g, int t) {
    float s[2][4];
    kw.dots_few(q, s);
    float mt[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int key = kb + 16 * u + 8 * (k >> 1) + g;
        const float x = fmaf(s[u][k], coef[k & 1] * sc.kf[u], sc.lv[u]);
        s[u][k] = key < end ? x : -INFINITY;
        mt[k & 1] = fmaxf(mt[k & 1], s[u][k]);
      }
    if (__any_sync(0xffffffffu, mt[0] > m[0] + kLag || mt[1] > m[1] + kLag)) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) mt[r] = fmaxf(mt[r], __shfl_xor_sync(0xffffffffu, mt[r], k));
        const float mn = fmaxf(m[r], mt[r]);
        const float al = mn == -INFINITY ? 1.f : exp2f(m[r] - mn);
        m[r] = mn;
        l[r] *= al;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          o[j][r] *= al;
          o[j][2 + r] *= al;
        }
      }
    }
    VWords<D> vw;
    vw.load(v_stage, g, t);
    // a row whose every score is -inf so far (NaN queries aside) keeps P = 0
    const float b0 = (m[0] == -INFINITY ? 0.f : -m[0]) + kBias, b1 = (m[1] == -INFINITY ? 0.f : -m[1]) + kBias;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float x0 = ex2_approx(s[u][0] + b0), x1 = ex2_approx(s[u][1] + b1);
      const float y0 = ex2_approx(s[u][2] + b0), y1 = ex2_approx(s[u][3] + b1);
      l[0] = fmaf(x0 + y0, sc.iv[u], l[0]);
      l[1] = fmaf(x1 + y1, sc.iv[u], l[1]);
      vw.accumulate_few(u, transpose8(pack_f16x2(x0, x1)), transpose8(pack_f16x2(y0, y1)), o);
    }
  }
  __device__ __forceinline__ void leave(Shared& sh, int warp, int rows, int g, int t) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
      for (int k = 4; k < 32; k <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], k);
      const int row = 2 * t + r;
      if (g == 0) sh.m[warp][row] = m[r], sh.l[warp][row] = l[r];
      if (row >= rows) continue;
      float* to = &sh.o[warp][row][g * (D / 8)];
#pragma unroll
      for (int j = 0; j < D / 32; ++j)
        *reinterpret_cast<float4*>(to + 4 * j) = make_float4(o[2 * j][r], o[2 * j][2 + r], o[2 * j + 1][r], o[2 * j + 1][2 + r]);
    }
  }
};

// Whether every piece of a cut unit is there, this CTA's included, which it says first.
// Each piece has a flag of its own, set to the call's tag: no counter that pieces ending
// together queue up for (compare-and-swap on one took 8 us for 12 of them), nothing to
// initialise.  Every lane's fence lies between the setting and its looks at the others,
// and fences have one order: the piece whose fences come last sees all flags.  More than
// one may; they write the same values.  Whoever sees them all clears them, so that a
// replayed call finds none of its earlier run.  Called by one warp.
__device__ __forceinline__ bool all_there(unsigned long long* flag, unsigned long long tag, const Q8Piece& pc, int lane) {
  volatile unsigned long long* f = flag;
  if (lane == 0) f[blockIdx.x * 2 + pc.which] = tag;
  __syncwarp();
  __threadfence();
  bool all = true;
  for (int k = lane; k < pc.npieces; k += 32) all &= f[(pc.cfirst + k) * 2 + (k == 0 ? pc.wfirst : 0)] == tag;
  all = __all_sync(0xffffffffu, all);
  if (all)
    for (int k = lane; k < pc.npieces; k += 32) f[(pc.cfirst + k) * 2 + (k == 0 ? pc.wfirst : 0)] = 0ull;
  return all;
}

template <typename T, int D>
__device__ __forceinline__ void put_row4(void* O, size_t row, int c, float4 v) {
  T* p = static_cast<T*>(O) + row * D + c;
  if constexpr (sizeof(T) == 2) *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
  else *reinterpret_cast<float4*>(p) = v;
}

// A piece that finds all pieces of its unit there merges them, in their order: their maxima
// and sums, fetched at once, become one weight per (row, piece), and weigh the outputs,
// sixteen of which are on their way meanwhile.  (A second kernel for it cost 6 us.)  Called
// by the whole CTA after it has stored its own piece; unit: log2 of the sums' unit; s_w,
// s_l: shared memory, ROWS x kQ8MaxCtas each.
template <int D, typename T, int ROWS>
__device__ void finish_unit(const Q8AttendArgs& a, const Q8Piece& pc, size_t row0, int rows, float bias, int unit,
                            float* s_w, float* s_l, int* s_last) {
  const int tid = threadIdx.x, nthreads = blockDim.x, np = pc.npieces;
  __threadfence();
  __syncthreads();
  if (tid < 32) {
    const bool all = all_there(a.flag, a.tag, pc, tid);
    if (tid == 0) *s_last = all;
  }
  __syncthreads();
  if (!*s_last) return;
  __threadfence();
  const float* first = a.part + static_cast<size_t>(pc.cfirst * 2 + pc.wfirst) * slot_floats<D>();
  const float* rest = a.part + static_cast<size_t>(pc.cfirst) * 2 * slot_floats<D>();  // piece k > 0: slot 0 of CTA cfirst + k
  auto slot = [&](int k) { return k == 0 ? first : rest + static_cast<size_t>(k) * 2 * slot_floats<D>(); };
  // a thread's first outputs of the first sixteen pieces, in flight with the maxima and sums
  constexpr int kAhead = 16;
  float4 x[kAhead];
  auto outputs = [&](int row, int c, int k0) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (k0 + u < np) x[u] = __ldcg(reinterpret_cast<const float4*>(slot(k0 + u) + row * D + c));
  };
  if (tid < rows * (D / 4)) outputs(tid / (D / 4), (tid % (D / 4)) * 4, 0);
  for (int i = tid; i < rows * np; i += nthreads) {
    const int row = i / np, k = i - row * np;
    s_w[row * kQ8MaxCtas + k] = __ldcg(slot(k) + kRows * D + row);
    s_l[row * kQ8MaxCtas + k] = __ldcg(slot(k) + kRows * D + kRows + row);
  }
  __syncthreads();
  const int warp = tid >> 5, lane = tid & 31;
  for (int row = warp; row < rows; row += nthreads / 32) {
    float* w = s_w + row * kQ8MaxCtas;
    float* l = s_l + row * kQ8MaxCtas;
    float M = -INFINITY;
    for (int k = lane; k < np; k += 32) M = fmaxf(M, w[k]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float L = 0.f;
    for (int k = lane; k < np; k += 32) {
      const float f = M == -INFINITY ? 1.f : exp2f(w[k] - M);
      w[k] = f;
      L = fmaf(f, l[k], L);
    }
    L = warp_sum(L);
    __syncwarp();
    if (lane == 0) {
      l[0] = inverse_sum(L) * pow2f(unit);
      if (a.lse) a.lse[row0 + row] = (M - (bias + unit) + log2f(L)) * kLn2;
    }
  }
  __syncthreads();
  for (int i = tid; i < rows * (D / 4); i += nthreads) {
    const int row = i / (D / 4), c = (i % (D / 4)) * 4;
    const float* w = s_w + row * kQ8MaxCtas;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < np; k0 += kAhead) {
      if (i != tid || k0 != 0) outputs(row, c, k0);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (k0 + u >= np) continue;
        const float f = w[k0 + u];
        acc.x = fmaf(f, x[u].x, acc.x);
        acc.y = fmaf(f, x[u].y, acc.y);
        acc.z = fmaf(f, x[u].z, acc.z);
        acc.w = fmaf(f, x[u].w, acc.w);
      }
    }
    const float inv = s_l[row * kQ8MaxCtas];
    put_row4<T, D>(a.O, row0 + row, c, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
  }
}

// rows of heads without tokens: zeros (lse -inf), spread over the CTAs with work (or all
// left to CTA 0)
template <int D, typename T>
__device__ void empty_rows(const Q8AttendArgs& a, const Q8Sched& sch, int tile_rows, int nrt) {
  for (int h = 0; h < a.c.H; ++h) {
    if (sch.T[h] != 0) continue;
    for (int r = q8_first_turn(h, nrt, sch.G); r < nrt; r += sch.G) {
      const int rows = min(tile_rows, a.Nq - r * tile_rows);
      const size_t row0 = static_cast<size_t>(h) * a.Nq + r * tile_rows;
      for (int i = threadIdx.x; i < rows * (D / 4); i += blockDim.x)
        put_row4<T, D>(a.O, row0 + i / (D / 4), (i % (D / 4)) * 4, make_float4(0.f, 0.f, 0.f, 0.f));
      if (a.lse)
        for (int i = threadIdx.x; i < rows; i += blockDim.x) a.lse[row0 + i] = -INFINITY;
    }
  }
}

template <int D, typename Acc>
__global__ void __launch_bounds__(Acc::kThreads, 1) q8_attend_rows_kernel(const Q8AttendArgs a) {
  constexpr int kTileRows = Acc::kTileRows, kWarps = Acc::kWarps;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Q8Sched sch;
  __shared__ int s_last;
  typename Acc::Shared& sh = *reinterpret_cast<typename Acc::Shared*>(smem);  // over the rings, once they are done with
  pdl_wait();
  pdl_trigger();
  const int nrt = (a.Nq + kTileRows - 1) / kTileRows;
  // a CTA's share is at least one 32-token step for each warp
  q8_build_sched(&sch, a.c.len, a.c.cap, a.c.H, nrt, kTile, 1, 1, gridDim.x, kWarps * kSub / kTile, true);
  Q8Split S{&sch, a.c.H, nrt, 1, 1};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int blocks = a.c.cap >> a.c.shift;
  constexpr int kStage = 64 * D;  // K and V of 32 tokens
  uint8_t* ring = smem + static_cast<size_t>(warp) * kRing * kStage;
  const uint32_t ring32 = smem_u32(ring);
  Q8Walk walk;
  walk.init(S, blockIdx.x);
  Q8Piece pc;
  while (walk.next(S, pc, false)) {
    const int n = q8_len(a.c.len, pc.h, a.c.cap);
    const int end = min(pc.j1 * kTile, n);
    const int rows = min(kTileRows, a.Nq - pc.r * kTileRows);
    const size_t row0 = static_cast<size_t>(pc.h) * a.Nq + pc.r * kTileRows;
    const uint8_t* K = a.c.K + static_cast<size_t>(pc.h) * a.c.cap * D;
    const uint8_t* V = a.c.V + static_cast<size_t>(pc.h) * a.c.cap * D;
    const float* ks = a.c.ks + static_cast<size_t>(pc.h) * blocks;
    const float* vs = a.c.vs + static_cast<size_t>(pc.h) * blocks;
    Acc acc;
    acc.q.fetch(static_cast<const __nv_bfloat16*>(a.Q) + row0 * D, rows, g, t);
    constexpr int kHop = kWarps * kSub;
    const int first = pc.j0 * kTile + warp * kSub;
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i) {
      if (first + i * kHop < end) fetch<D>(ring32 + i * kStage, K, V, first + i * kHop, n - 1, lane);
      cp_async_commit();
    }
    // the scales of a step's two 16-token halves, a step ahead
    float nk[2], nv[2];
    auto scales = [&](int kb) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int b = min(kb + 16 * u, n - 1) >> a.c.shift;
        nk[u] = __ldg(ks + b);
        nv[u] = __ldg(vs + b);
      }
    };
    scales(first);
    const int unit = sum_unit(vs);
    if (sch.chunk == 0) q8_unit_pieces(S, pc.h, pc.r, pc);
    acc.begin(a.scale, t);
    int stage = 0;
    for (int kb = first; kb < end; kb += kHop) {
      __syncwarp();  // every lane is done with the stage that is fetched into next
      {
        const int ahead = kb + (kRing - 1) * kHop, st = stage == 0 ? kRing - 1 : stage - 1;
        if (ahead < end) fetch<D>(ring32 + st * kStage, K, V, ahead, n - 1, lane);
        cp_async_commit();
      }
      cp_async_wait<kRing - 1>();
      __syncwarp();
      KWords<D> kw;
      kw.load(ring + stage * kStage, g, t);
      StepScales sc;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        sc.kf[u] = nk[u];
        sc.lv[u] = log2f(nv[u]);
        sc.iv[u] = 1.f / (nv[u] * pow2f(-unit));
      }
      if (kb + kHop < end) scales(kb + kHop);
      acc.step(kw, ring + stage * kStage + 32 * D, sc, kb, end, g, t);
      stage = stage == kRing - 1 ? 0 : stage + 1;
    }
    // merge the warps: maxima first, then every output weighted by its warp
    cp_async_wait<0>();
    __syncthreads();  // every warp is done with its ring
    acc.leave(sh, warp, rows, g, t);
    __syncthreads();
    float* slot = a.part + static_cast<size_t>(blockIdx.x * 2 + pc.which) * slot_floats<D>();
    for (int i = threadIdx.x; i < rows * (D / 4); i += Acc::kThreads) {
      const int row = i / (D / 4), c = (i % (D / 4)) * 4;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sh.m[w][row]);
      float L = 0.f;
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = M == -INFINITY ? 1.f : exp2f(sh.m[w][row] - M);
        const float4 x = *reinterpret_cast<const float4*>(&sh.o[w][row][c]);
        L = fmaf(f, sh.l[w][row], L);
        sum.x = fmaf(f, x.x, sum.x);
        sum.y = fmaf(f, x.y, sum.y);
        sum.z = fmaf(f, x.z, sum.z);
        sum.w = fmaf(f, x.w, sum.w);
      }
      if (pc.npieces == 1) {
        const float inv = inverse_sum(L) * pow2f(unit);
        put_row4<__nv_bfloat16, D>(a.O, row0 + row, c, make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv));
        if (a.lse && c == 0) a.lse[row0 + row] = (M - (Acc::kBias + unit) + log2f(L)) * kLn2;
      } else {
        *reinterpret_cast<float4*>(slot + row * D + c) = sum;
        if (c == 0) {
          slot[kRows * D + row] = M;
          slot[kRows * D + kRows + row] = L;
        }
      }
    }
    if (pc.npieces > 1) {
      __syncthreads();  // the warps' outputs have been read
      float* s_w = reinterpret_cast<float*>(smem);
      finish_unit<D, __nv_bfloat16, kTileRows>(a, pc, row0, rows, Acc::kBias, unit, s_w, s_w + kTileRows * kQ8MaxCtas, &s_last);
    }
    __syncthreads();  // the merge is done with the shared memory
  }
  empty_rows<D, __nv_bfloat16>(a, sch, kTileRows, nrt);
}

// ------------------------------------------------------------------ f32 rows
// Queries and outputs of 32 bits keep 24-bit products: CUDA cores, kF32Rows rows at a
// time.  Eight lanes share a token (D / 8 channels each), so a warp works through four
// tokens side by side, each group of lanes with its own running maximum.
// Bound by latency: a step fetches its tokens and uses them at once, four warps an SM.  us
// for 1 / 4 / 16 / 256 rows over 12 x 15600 x 128 (bytes: 7.3 us): 91 / 91 / 317 / 3370;
// with two rows a tile 71 / 130 / 362 / 4230, with 64 threads 170 / 171 / 624 / 6660.
// kMinTiles counts where one short cache is cut (1 x 8192, a row: 20 us, 30 with 8, 16 with
// 2); elsewhere 2 to 8 are equal.
constexpr int kF32Rows = 4;
constexpr int kF32Threads = 128;
constexpr int kF32Groups = kF32Threads / 8;

template <int D>
__device__ __forceinline__ void load_codes(const uint8_t* p, float (&f)[D / 8]) {
  uint32_t w[D / 32];
  if constexpr (D == 128) {
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(p));
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
  } else {
    const uint2 x = __ldg(reinterpret_cast<const uint2*>(p));
    w[0] = x.x, w[1] = x.y;
  }
#pragma unroll
  for (int k = 0; k < D / 32; ++k) {
    const float4 x = e4m3x4_to_f32x4(w[k]);
    f[4 * k] = x.x, f[4 * k + 1] = x.y, f[4 * k + 2] = x.z, f[4 * k + 3] = x.w;
  }
}
template <int D>
__device__ __forceinline__ void load_q(const float* p, float mul, float (&f)[D / 8]) {
#pragma unroll
  for (int k = 0; k < D / 32; ++k) {
    const float4 x = *(reinterpret_cast<const float4*>(p) + k);
    f[4 * k] = x.x * mul, f[4 * k + 1] = x.y * mul, f[4 * k + 2] = x.z * mul, f[4 * k + 3] = x.w * mul;
  }
}
__device__ __forceinline__ float octet_sum(float v) {
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int D>
__global__ void __launch_bounds__(kF32Threads) q8_attend_f32_kernel(const Q8AttendArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int s_last;
  __shared__ Q8Sched sch;
  __shared__ float sm[kF32Groups][kF32Rows], sl[kF32Groups][kF32Rows];
  float* so = reinterpret_cast<float*>(smem);  // [group][row][D]
  pdl_wait();
  pdl_trigger();
  const int nrt = (a.Nq + kF32Rows - 1) / kF32Rows;
  q8_build_sched(&sch, a.c.len, a.c.cap, a.c.H, nrt, kTile, 1, 1, gridDim.x, kMinTiles, true);
  Q8Split S{&sch, a.c.H, nrt, 1, 1};
  const int grp = threadIdx.x >> 3, sub = threadIdx.x & 7;
  const int blocks = a.c.cap >> a.c.shift;
  Q8Walk walk;
  walk.init(S, blockIdx.x);
  Q8Piece pc;
  while (walk.next(S, pc)) {
    const int n = q8_len(a.c.len, pc.h, a.c.cap);
    const int end = min(pc.j1 * kTile, n);
    const int rows = min(kF32Rows, a.Nq - pc.r * kF32Rows);
    const size_t row0 = static_cast<size_t>(pc.h) * a.Nq + pc.r * kF32Rows;
    const size_t at = static_cast<size_t>(pc.h) * a.c.cap * D + sub * (D / 8);
    float q[kF32Rows][D / 8], acc[kF32Rows][D / 8], m[kF32Rows], l[kF32Rows];
#pragma unroll
    for (int r = 0; r < kF32Rows; ++r) {
      load_q<D>(static_cast<const float*>(a.Q) + (row0 + min(r, rows - 1)) * D + sub * (D / 8), a.scale * kLog2e, q[r]);
      // an infinite element makes its row NaN, also where it would send every score to -inf
#pragma unroll
      for (int k = 0; k < D / 8; ++k) q[r][k] = fabsf(q[r][k]) == INFINITY ? NAN : q[r][k];
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int k = 0; k < D / 8; ++k) acc[r][k] = 0.f;
    }
    // whole warps take the same number of steps, so that the sums can shuffle
    const int first = pc.j0 * kTile;
    const int steps = (end - first + kF32Groups - 1) / kF32Groups;
    for (int i = 0; i < steps; ++i) {
      const int key = first + i * kF32Groups + grp;
      const int kc = min(key, end - 1);
      float kf[D / 8], vf[D / 8];
      load_codes<D>(a.c.K + at + static_cast<size_t>(kc) * D, kf);
      load_codes<D>(a.c.V + at + static_cast<size_t>(kc) * D, vf);
      const float ks = __ldg(a.c.ks + static_cast<size_t>(pc.h) * blocks + (kc >> a.c.shift));
      const float vs = __ldg(a.c.vs + static_cast<size_t>(pc.h) * blocks + (kc >> a.c.shift));
#pragma unroll
      for (int r = 0; r < kF32Rows; ++r) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < D / 8; ++k) s = fmaf(q[r][k], kf[k], s);
        const float dot = octet_sum(s);
        const float x = key < end ? dot * ks : -INFINITY;
        if (x > m[r]) {
          const float al = exp2f(m[r] - x);
          m[r] = x;
          l[r] *= al;
#pragma unroll
          for (int k = 0; k < D / 8; ++k) acc[r][k] *= al;
        }
        const float p = x == -INFINITY ? 0.f : exp2f(x - m[r]);  // behind the end, or past fp32's range
        l[r] += p;
        const float pv = p * vs;
#pragma unroll
        for (int k = 0; k < D / 8; ++k) acc[r][k] = fmaf(pv, vf[k], acc[r][k]);
      }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kF32Rows; ++r) {
      if (sub == 0) sm[grp][r] = m[r], sl[grp][r] = l[r];
#pragma unroll
      for (int k = 0; k < D / 8; k += 4)
        *reinterpret_cast<float4*>(so + (static_cast<size_t>(grp) * kF32Rows + r) * D + sub * (D / 8) + k) =
            make_float4(acc[r][k], acc[r][k + 1], acc[r][k + 2], acc[r][k + 3]);
    }
    __syncthreads();
    float* slot = a.part + static_cast<size_t>(blockIdx.x * 2 + pc.which) * slot_floats<D>();
    for (int i = threadIdx.x; i < rows * D; i += kF32Threads) {
      const int row = i / D, c = i % D;
      float M = -INFINITY;
      for (int w = 0; w < kF32Groups; ++w) M = fmaxf(M, sm[w][row]);
      float L = 0.f, v = 0.f;
      for (int w = 0; w < kF32Groups; ++w) {
        const float f = M == -INFINITY ? 1.f : exp2f(sm[w][row] - M);
        L = fmaf(f, sl[w][row], L);
        v = fmaf(f, so[(static_cast<size_t>(w) * kF32Rows + row) * D + c], v);
      }
      if (pc.npieces == 1) {
        static_cast<float*>(a.O)[(row0 + row) * D + c] = L == 0.f ? 0.f : v / L;
        if (a.lse && c == 0) a.lse[row0 + row] = (M + log2f(L)) * kLn2;
      } else {
        slot[row * D + c] = v;
        if (c == 0) {
          slot[kRows * D + row] = M;
          slot[kRows * D + kRows + row] = L;
        }
      }
    }
    if (pc.npieces > 1) {
      __syncthreads();  // the groups' outputs have been read
      finish_unit<D, float, kF32Rows>(a, pc, row0, rows, 0.f, 0, so, so + kF32Rows * kQ8MaxCtas, &s_last);
    }
    __syncthreads();  // the merge is done with the shared memory
  }
  empty_rows<D, float>(a, sch, kF32Rows, nrt);
}

// ------------------------------------------------------------------ weights
// mass[k] = decay prev[k] + sum over rows of 2^(x - lse log2 e): a token's weight is
// whole within its warp, so there is nothing to split or merge, and the rows are added
// in one fixed order.  Up to sixteen rows (ONE) stay in registers for all of a warp's
// tokens; of more, each step fetches them again, 16 at a time.  FEW: at most eight.
template <int D, bool FEW>
struct WeightRows {
  static constexpr int kI = FEW ? 1 : 2;
  QFrag<D, kI> q;
  // of rows g, g + 8, or 2 t, 2 t + 1 of at most eight.  z: -lse log2 e; -inf: no such row,
  // or one that saw nothing, which weighs nothing
  float coef[2], z[2];
  __device__ __forceinline__ void load(const Q8MassArgs& a, int h, int r0, int g, int t) {
    const size_t row0 = static_cast<size_t>(h) * a.Nq + r0;
    const int rows = min(kRows, a.Nq - r0);
    q.fetch(static_cast<const __nv_bfloat16*>(a.Q) + row0 * D, rows, g, t);
    float zq[kI];  // of the fragments' rows
#pragma unroll
    for (int i = 0; i < kI; ++i) {
      const int row = g + 8 * i;
      const float v = row < rows ? a.lse[row0 + row] : -INFINITY;
      zq[i] = v == -INFINITY ? -INFINITY : -v * kLog2e;
      // whatever the queries of a row that weighs nothing hold, NaN say, stays out of the sums
#pragma unroll
      for (int k = 0; k < D / 32; ++k)
        if (v == -INFINITY) q.raw[i][k] = make_uint4(0u, 0u, 0u, 0u);
    }
    q.widen(a.scale);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      coef[i] = FEW ? __shfl_sync(0xffffffffu, q.coef[0], 4 * (2 * t + i)) : q.coef[i % kI];
      z[i] = FEW ? __shfl_sync(0xffffffffu, zq[0], 4 * (2 * t + i)) : zq[i % kI];
    }
  }
  // the weights of 32 tokens, summed over the rows; token mine(g, t) of them returned
  static __device__ __forceinline__ int mine(int g, int t) { return FEW ? 8 * t + g : 8 * (g >> 1) + 2 * t + (g & 1); }
  __device__ __forceinline__ void add(const KWords<D>& kw, const float (&kf)[2], float (&w)[4][2]) const {
    if constexpr (FEW) {
      float s[2][4];
      kw.dots_few(q, s);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int k = 0; k < 4; ++k) w[2 * u + (k >> 1)][0] += ex2_approx(fmaf(s[u][k], coef[k & 1] * kf[u], z[k & 1]));
    } else {
      float s[4][4];
      kw.dots(q, s);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) w[j][k & 1] += ex2_approx(fmaf(s[j][k], coef[k >> 1] * kf[j >> 1], z[k >> 1]));
    }
  }
  static __device__ __forceinline__ float total(const float (&w)[4][2], int g, int t) {
    float v = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (FEW) {
        const float x = quad_sum(w[j][0]);  // token 8 j + g
        if (t == j) v = x;
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float x = w[j][i];
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
          if (g == 2 * j + i) v = x;
        }
      }
    }
    return v;
  }
};

template <int D, bool FEW, bool ONE>
__global__ void __launch_bounds__(kThreads, FEW ? 2 : 1) q8_mass_rows_kernel(const Q8MassArgs a) {
  pdl_wait();
  pdl_trigger();
  const int h = blockIdx.y;
  const int n = q8_len(a.c.len, h, a.c.cap);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint8_t* K = a.c.K + static_cast<size_t>(h) * a.c.cap * D;
  const float* ks = a.c.ks + static_cast<size_t>(h) * (a.c.cap >> a.c.shift);
  const size_t m0 = static_cast<size_t>(h) * a.c.cap;
  const int hop = gridDim.x * kWarps * kSub;
  int kb = (blockIdx.x * kWarps + warp) * kSub;
  if (kb >= n) return;
  KWords<D> next;
  next.load_global(K, kb, n - 1, g, t);
  WeightRows<D, FEW> rows;
  if constexpr (ONE) rows.load(a, h, 0, g, t);
  // the token whose weight this lane stores, and fetches what it adds to
  const int mine = WeightRows<D, FEW>::mine(g, t);
  for (; kb < n; kb += hop) {
    const KWords<D> kw = next;
    float kf[2], w[4][2], before = 0.f;
#pragma unroll
    for (int u = 0; u < 2; ++u) kf[u] = __ldg(ks + (min(kb + 16 * u, n - 1) >> a.c.shift));
    if (a.prev && kb + mine < n) before = a.prev[m0 + kb + mine];
    if (kb + hop < n) next.load_global(K, kb + hop, n - 1, g, t);
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j][0] = w[j][1] = 0.f;
    for (int r0 = 0; r0 < (ONE ? 1 : a.Nq); r0 += kRows) {
      if constexpr (!ONE) rows.load(a, h, r0, g, t);
      rows.add(kw, kf, w);
    }
    const float v = WeightRows<D, FEW>::total(w, g, t);
    if (kb + mine < n) a.mass[m0 + kb + mine] = a.prev ? fmaf(a.decay, before, v) : v;
  }
}

// f32: eight lanes per token as in the attention, kF32Keys tokens per group of lanes at a
// time, so that a row's elements are fetched once for all of them; a single row (ONE) is
// held in registers for all tokens.  The loads of a round do not wait on one another.
constexpr int kF32Keys = 4;
template <int D, bool ONE>
__global__ void __launch_bounds__(kThreads, 2) q8_mass_f32_kernel(const Q8MassArgs a) {
  pdl_wait();
  pdl_trigger();
  const int h = blockIdx.y;
  const int n = q8_len(a.c.len, h, a.c.cap);
  const int grp = threadIdx.x >> 3, sub = threadIdx.x & 7;
  constexpr int kGroups = kThreads / 8;
  const float* Q = static_cast<const float*>(a.Q) + static_cast<size_t>(h) * a.Nq * D + sub * (D / 8);
  const float* lse = a.lse + static_cast<size_t>(h) * a.Nq;
  const uint8_t* K = a.c.K + static_cast<size_t>(h) * a.c.cap * D + sub * (D / 8);
  const float* ks = a.c.ks + static_cast<size_t>(h) * (a.c.cap >> a.c.shift);
  const size_t m0 = static_cast<size_t>(h) * a.c.cap;
  float q[D / 8], z = 0.f;
  if constexpr (ONE) {
    load_q<D>(Q, 1.f, q);
    z = lse[0];
  }
  for (int k0 = blockIdx.x * kGroups * kF32Keys; k0 < n; k0 += gridDim.x * kGroups * kF32Keys) {
    float kf[kF32Keys][D / 8], mul[kF32Keys], w[kF32Keys];
    // lane u of the group stores token u's weight, and fetches what it adds to
    const int mine = k0 + sub * kGroups + grp;
    float before = 0.f;
    if (sub < kF32Keys && mine < n && a.prev) before = a.prev[m0 + mine];
#pragma unroll
    for (int u = 0; u < kF32Keys; ++u) {
      const int kc = min(k0 + u * kGroups + grp, n - 1);
      load_codes<D>(K + static_cast<size_t>(kc) * D, kf[u]);
      mul[u] = __ldg(ks + (kc >> a.c.shift)) * a.scale;
      w[u] = 0.f;
    }
    for (int r = 0; r < (ONE ? 1 : a.Nq); ++r) {
      if constexpr (!ONE) {
        load_q<D>(Q + static_cast<size_t>(r) * D, 1.f, q);
        z = lse[r];
      }
#pragma unroll
      for (int u = 0; u < kF32Keys; ++u) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < D / 8; ++k) s = fmaf(q[k], kf[u][k], s);
        const float x = octet_sum(s);
        if (z != -INFINITY) w[u] += expf(fmaf(x, mul[u], -z));
      }
    }
    if (sub < kF32Keys && mine < n) {
      const float v = sub == 0 ? w[0] : (sub == 1 ? w[1] : (sub == 2 ? w[2] : w[3]));
      a.mass[m0 + mine] = a.prev ? fmaf(a.decay, before, v) : v;
    }
  }
}

int split_grid(int n_sm) { return n_sm < kQ8MaxCtas ? n_sm : kQ8MaxCtas; }

template <int D, typename Acc>
cudaError_t attend_rows(const Q8AttendArgs& a, int n_sm, cudaStream_t st) {
  const int grid = split_grid(n_sm);
  constexpr size_t ring = Acc::kWarps * kRing * 64 * D, shared = sizeof(typename Acc::Shared);
  constexpr size_t smem = ring > shared ? ring : shared;
  static_assert(smem >= 2 * Acc::kTileRows * kQ8MaxCtas * sizeof(float), "the merge's weights fit");
  const auto kernel = q8_attend_rows_kernel<D, Acc>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  LaunchTrace trace("q8_attend_rows_kernel", st);
  return launch_pdl(kernel, dim3(grid), dim3(Acc::kThreads), smem, st, a);
}

template <int D>
cudaError_t attend_f32(const Q8AttendArgs& a, int n_sm, cudaStream_t st) {
  constexpr size_t smem = static_cast<size_t>(kF32Groups) * kF32Rows * D * sizeof(float);
  static_assert(smem >= 2 * kF32Rows * kQ8MaxCtas * sizeof(float), "the merge's weights fit");
  LaunchTrace trace("q8_attend_f32_kernel", st);
  return launch_pdl(q8_attend_f32_kernel<D>, dim3(split_grid(n_sm)), dim3(kF32Threads), smem, st, a);
}

// CTAs per head so that the grid is about `waves` waves, no more than the tokens need
int mass_blocks(int cap, int per_cta, int H, int n_sm, int waves) {
  const int need = (cap + per_cta - 1) / per_cta;
  const int room = (n_sm * waves + H - 1) / H;
  return need < room ? need : (room < 1 ? 1 : room);
}

}  // namespace

cudaError_t launch_q8_attend_rows(const Q8AttendArgs& a, int n_sm, cudaStream_t st) {
  if (a.Nq <= 8) return a.c.d == 128 ? attend_rows<128, FewAcc<128>>(a, n_sm, st) : attend_rows<64, FewAcc<64>>(a, n_sm, st);
  return a.c.d == 128 ? attend_rows<128, RowsAcc<128>>(a, n_sm, st) : attend_rows<64, RowsAcc<64>>(a, n_sm, st);
}
cudaError_t launch_q8_attend_f32(const Q8AttendArgs& a, int n_sm, cudaStream_t st) {
  return a.c.d == 128 ? attend_f32<128>(a, n_sm, st) : attend_f32<64>(a, n_sm, st);
}
cudaError_t launch_q8_mass_rows(const Q8MassArgs& a, int n_sm, cudaStream_t st) {
  const dim3 grid(mass_blocks(a.c.cap, kWarps * kSub, a.c.H, n_sm, 2), a.c.H);
  LaunchTrace trace("q8_mass_rows_kernel", st);
  const bool wide = a.c.d == 128;
  if (a.Nq <= 8)
    return wide ? launch_pdl(q8_mass_rows_kernel<128, true, true>, grid, dim3(kThreads), 0, st, a)
                : launch_pdl(q8_mass_rows_kernel<64, true, true>, grid, dim3(kThreads), 0, st, a);
  if (a.Nq <= kRows)
    return wide ? launch_pdl(q8_mass_rows_kernel<128, false, true>, grid, dim3(kThreads), 0, st, a)
                : launch_pdl(q8_mass_rows_kernel<64, false, true>, grid, dim3(kThreads), 0, st, a);
  return wide ? launch_pdl(q8_mass_rows_kernel<128, false, false>, grid, dim3(kThreads), 0, st, a)
              : launch_pdl(q8_mass_rows_kernel<64, false, false>, grid, dim3(kThreads), 0, st, a);
}
cudaError_t launch_q8_mass_f32(const Q8MassArgs& a, int n_sm, cudaStream_t st) {
  const dim3 grid(mass_blocks(a.c.cap, kThreads / 8 * kF32Keys, a.c.H, n_sm, 4), a.c.H);
  LaunchTrace trace("q8_mass_f32_kernel", st);
  if (a.Nq == 1)
    return a.c.d == 128 ? launch_pdl(q8_mass_f32_kernel<128, true>, grid, dim3(kThreads), 0, st, a)
                        : launch_pdl(q8_mass_f32_kernel<64, true>, grid, dim3(kThreads), 0, st, a);
  return a.c.d == 128 ? launch_pdl(q8_mass_f32_kernel<128, false>, grid, dim3(kThreads), 0, st, a)
                      : launch_pdl(q8_mass_f32_kernel<64, false>, grid, dim3(kThreads), 0, st, a);
}

}  // namespace kvb
