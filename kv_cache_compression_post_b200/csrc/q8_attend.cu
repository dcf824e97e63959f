// Attention over the 8-bit cache for chunks of queries, on the 5th-generation tensor
// cores.
//
// The codes are multiplied as they lie.  A bf16 query element has 8 significant bits
// and E4M3 holds 4, so with the row scaled by a power of two to a largest element in
// [2^7, 2^8) an element is the exact sum of two E4M3 parts, q = hi + lo, down to 2^-9 of the
// power of two below the row's largest (its last bit is then E4M3's smallest step, 2^-9);
// smaller ones are off by half of that step, at most 2^-17 of the row's largest:
//     S = hi K^T + lo K^T        2 x kind::f8f6f4, K the cache's bytes from TMA
// which costs the tensor time of one bf16 product and never widens K.
// P V cannot be split so cheaply (every weight would be rounded twice, by the warps
// that are the scarce resource), so V is widened: a warpgroup of its own turns each V
// tile into fp16 (exact, two codes per instruction) in the layout the MMA reads, and
// clears rows behind the head's length, where anything may lie.  fp16 rather than bf16
// also makes P eight times more exact than a bf16 kernel's.
// Scales: K's block scale multiplies a 16-token chunk's scores inside the FFMA that
// feeds the exponential; V's rides in the exponent, P' = 2^(x + log2 vs - m + kPBias)
// with m the running maximum of x + log2 vs, and the row sum adds P' / vs per chunk (in units
// of sum_unit).
// Neither costs an instruction per score.
//
// Work: units of (head, pair of 128-query tiles A, B), split over a persistent grid at
// 128-token tiles (Q8Split); a unit cut between CTAs is finished by whichever of its
// pieces comes last, so no CTA waits for another.
// TMEM: S_A, S_B, O_A, O_B (128 columns each), P_t over S_t's first half.  Per key tile
// and query tile: S_t, softmax, P_t V, and S_t of the next tile behind it.
// What bounds it.  A 256 x 128 step has 2048 clk of tensor time and 2048 clk of
// exponentials per SM and takes ~4100 (at 1.8 GHz, the power cap active): softmax and
// products of one query tile follow one another, so the two tiles have to alternate.
// Kept for that, each measured on 12 heads x 4680 queries x 15600 tokens: one MMA warp
// per query tile, operands in uniform registers (627 -> 557 us with the scales' ring;
// issuing from one divergent lane cost ~110 clk an MMA), turns at the exponentials
// (552 -> 507 us; left alone the tiles fall into step and wait together), codes widened
// four at a time (502 -> 481 us).  Not kept: a
// part of the exponentials as polynomials on the FMA pipe (+6 % for one pair in eight:
// issue, not the exponential unit, is short in a turn); 64-token steps with two score
// buffers (542 us: N = 64 products read the query rows twice as often); two warpgroups
// per query tile, by steps (554 us) or by columns (584 us); the scores' scaling before
// the turn (+2 %), or nothing but exponentials in it (+6 %); handing the turn on before
// its last quarter or half (no gain); P V of the first tokens before the others' P is
// there (+4 %: the store has to be waited for twice).
// Warps: 0 loads, 1 and 3 MMAs of tile A and B, 2 TMEM and scales, 4-7 V widening,
// 8-11 softmax of tile A, 12-15 of tile B (one thread per row).
#include "host_util.h"
#include "q8.cuh"
#include "sm100.cuh"

namespace kvb {
using namespace sm100;

namespace {

constexpr int kThreads = 512;
constexpr int kTile = 128;  // queries per query tile, tokens per key tile
constexpr int kBarBytes = 512;
constexpr int kKStages = 3, kV8Stages = 2, kVStages = 2, kScStages = 4;
constexpr float kRescale = 8.f;   // the running maximum moves when it grows by more (log2)
constexpr float kPBias = 6.f;     // P' <= 2^(kRescale + kPBias) < 65504
// cost of a key tile to a pair of query tiles, to a lone one; least share of a CTA
constexpr int kW2 = 8, kW1 = 7, kMinCost = 8 * kW2;
// registers per thread of each warpgroup: loads and MMA, widening, softmax (x2).  Their
// sum must not pass the launch's (checked on the host against the compiled kernel).
constexpr int kRegsControl = 64, kRegsWiden = 80, kRegsSoftmax = 184;

struct alignas(8) Bars {
  uint64_t q_full, q_empty;
  uint64_t k_full[kKStages], k_empty[kKStages];
  uint64_t v8_full[kV8Stages], v8_empty[kV8Stages], v_full[kVStages], v_empty[kVStages];
  uint64_t s_full[2], p_full[2];
  uint64_t o_full[2];
  uint64_t sc_full[2][kScStages], sc_empty[kScStages];  // a tile's scales, per query tile that reads them
  uint64_t mma_done[2];
  uint64_t turn[2][4];  // the exponentials of a tile pair take turns: per query tile just done, lane quarter
  uint64_t grp[2];
  uint32_t tmem_base;
  int abort;
  int last[2];
};
static_assert(sizeof(Bars) <= kBarBytes, "barrier block overflows its reservation");

struct Maps {
  CUtensorMap hi, lo, k, v;
};

struct Args {
  Q8AttendArgs a;
  const float* coef;   // [H][Nq]: raw score -> log2 units (but for the token's scale)
  unsigned int* cnt;   // [H][npair][2] arrivals, zeroed by the split kernel
};

// --------------------------------------------------------------- query parts
// hi, lo codes and the coefficient of every row, 16 bytes of it a lane, eight or sixteen
// rows of a warp in flight (bound by memory: 12 x 4680 x 128 in 9 us; one row at a time
// took 12).  Also zeroes the arrival counters of the launch that follows.
constexpr int kSplitFlight = 4;
template <int D>
__global__ void __launch_bounds__(256) q8_split_q_kernel(const __nv_bfloat16* Q, const float* lse, long long rows,
                                                         float scale, uint8_t* hi, uint8_t* lo, float* coef,
                                                         unsigned int* cnt, int ncnt) {
  pdl_wait();
  pdl_trigger();
  const long long gt = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  const long long nt = static_cast<long long>(gridDim.x) * blockDim.x;
  for (long long i = gt; i < ncnt; i += nt) cnt[i] = 0u;
  constexpr int kLanes = D / 8, kPer = 32 / kLanes;  // lanes of a row, rows of a warp's load
  const int lane = threadIdx.x & 31, c = lane % kLanes;
  for (long long r0 = (gt >> 5) * (kPer * kSplitFlight); r0 < rows; r0 += (nt >> 5) * (kPer * kSplitFlight)) {
    uint4 w[kSplitFlight];
    float z[kSplitFlight];
#pragma unroll
    for (int u = 0; u < kSplitFlight; ++u) {
      const long long row = r0 + u * kPer + lane / kLanes;
      w[u] = row < rows ? __ldg(reinterpret_cast<const uint4*>(Q + row * D) + c) : make_uint4(0u, 0u, 0u, 0u);
      z[u] = lse && row < rows ? __ldg(lse + row) : 0.f;
    }
#pragma unroll
    for (int u = 0; u < kSplitFlight; ++u) {
      const long long row = r0 + u * kPer + lane / kLanes;
      if (z[u] == -INFINITY) w[u] = make_uint4(0u, 0u, 0u, 0u);
      const uint32_t v[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
      float f[8], mx = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 x = unpack_bf16x2(v[k]);
        f[2 * k] = x.x;
        f[2 * k + 1] = x.y;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (fabsf(f[k]) <= 3.4e38f) mx = fmaxf(mx, fabsf(f[k]));
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const int e = max(exponent_of(mx), -100) - 7;  // mx 2^-e in [2^7, 2^8)
      const float down = pow2f(-e);
      uint32_t h[2], l[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        // an infinite element becomes a NaN: its row is NaN, as its scores would be
        float x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = fabsf(f[4 * k + i]) <= 3.4e38f ? f[4 * k + i] * down : NAN;
        h[k] = f32x4_to_e4m3x4(x[0], x[1], x[2], x[3]);
        const float4 b = e4m3x4_to_f32x4(h[k]);
        l[k] = f32x4_to_e4m3x4(x[0] - b.x, x[1] - b.y, x[2] - b.z, x[3] - b.w);
      }
      if (row >= rows) continue;
      reinterpret_cast<uint2*>(hi + row * D)[c] = make_uint2(h[0], h[1]);
      reinterpret_cast<uint2*>(lo + row * D)[c] = make_uint2(l[0], l[1]);
      if (c == 0) coef[row] = pow2f(e) * scale * kLog2e;
    }
  }
}

// ----------------------------------------------------------------- attention
template <int D>
__global__ void __launch_bounds__(kThreads, 1) q8_attend_kernel(const __grid_constant__ Maps maps, const Args args) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Q8Sched sch;
  __shared__ Q8Walk s_it[8];
  __shared__ Q8Piece s_pc[8];
  // per ring slot: K scales, log2 of V's and their reciprocals (in the sums' units), of eight
  // 16-token chunks
  __shared__ alignas(16) float sScale[kScStages * 24];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const Q8AttendArgs& a = args.a;
  constexpr uint32_t kCodeTile = kTile * D, kHalfTile = kTile * D * 2;  // bytes of a code tile, of an fp16 one
  uint8_t* sQ = smem;                          // hi, lo of A; hi, lo of B
  uint8_t* sK = sQ + 4 * kCodeTile;
  uint8_t* sV8 = sK + kKStages * kCodeTile;
  uint8_t* sV = sV8 + kV8Stages * kCodeTile;
  Bars* bars = reinterpret_cast<Bars*>(sV + kVStages * kHalfTile);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int npair = (a.Nq + 2 * kTile - 1) / (2 * kTile);
  const bool single = ((a.Nq + kTile - 1) / kTile) & 1;  // the last pair is a lone tile

  if (tid == 0) {
    mbar_init(&bars->q_full, 1);
    mbar_init(&bars->q_empty, 2);  // the rings are handed back by both query tiles' MMA warps
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(&bars->k_full[i], 1);
      mbar_init(&bars->k_empty[i], 2);
    }
    for (int i = 0; i < kV8Stages; ++i) {
      mbar_init(&bars->v8_full[i], 1);
      mbar_init(&bars->v8_empty[i], 4);
    }
    for (int i = 0; i < kVStages; ++i) {
      mbar_init(&bars->v_full[i], 4);
      mbar_init(&bars->v_empty[i], 2);
    }
    for (int i = 0; i < kScStages; ++i) {
      mbar_init(&bars->sc_full[0][i], 1);
      mbar_init(&bars->sc_full[1][i], 1);
      mbar_init(&bars->sc_empty[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->p_full[i], 4);
      mbar_init(&bars->o_full[i], 1);
      mbar_init(&bars->grp[i], 4);
      for (int k = 0; k < 4; ++k) mbar_init(&bars->turn[i][k], 1);
      mbar_init(&bars->mma_done[i], 1);
    }
    bars->abort = 0;
    fence_barrier_init();
  }
  // lengths, query parts and coefficients come from earlier work on the stream
  pdl_wait();
  pdl_trigger();
  q8_build_sched(&sch, a.c.len, a.c.cap, a.c.H, npair, kTile, kW2, single ? kW1 : kW2, gridDim.x, kMinCost);
  if (static_cast<int>(blockIdx.x) >= sch.G) return;  // no share of the work
  if (warp == 2) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  volatile int* abort = &bars->abort;
  Q8Split S{&sch, a.c.H, npair, kW2, single ? kW1 : kW2};
  int* status = a.c.status;
  auto ntq = [&](int p) { return (single && p == npair - 1) ? 1 : 2; };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
    if (warp == 0 && lane == 0) {
      // ------------------------------------------------------------ loads
      prefetch_tmap(&maps.hi);
      prefetch_tmap(&maps.lo);
      prefetch_tmap(&maps.k);
      prefetch_tmap(&maps.v);
      bool ok = true;
      int g = 0, np = 0;
      Q8Walk it;
      it.init(S, blockIdx.x);
      Q8Piece pc;
      while (ok && it.next(S, pc)) {
        for (int j = pc.j0; j < pc.j1; ++j, ++g) {
          const int st = g % kKStages, s8 = g % kV8Stages;
          if (!(ok = mbar_wait_step(&bars->k_empty[st], ((g / kKStages) & 1) ^ 1, abort, status))) break;
          mbar_arrive_expect_tx(&bars->k_full[st], kCodeTile);
          tma_load_3d(sK + st * kCodeTile, &maps.k, &bars->k_full[st], 0, j * kTile, pc.h);
          if (j == pc.j0) {
            // this piece's queries, once the previous piece's S products are done
            if (np > 0 && !(ok = mbar_wait_step(&bars->q_empty, (np - 1) & 1, abort, status))) break;
            const int nt = ntq(pc.r);
            mbar_arrive_expect_tx(&bars->q_full, nt * 2 * kCodeTile);
            for (int t = 0; t < nt; ++t) {
              const int y = (pc.r * 2 + t) * kTile;
              tma_load_3d(sQ + (2 * t) * kCodeTile, &maps.hi, &bars->q_full, 0, y, pc.h);
              tma_load_3d(sQ + (2 * t + 1) * kCodeTile, &maps.lo, &bars->q_full, 0, y, pc.h);
            }
            ++np;
          }
          if (!(ok = mbar_wait_step(&bars->v8_empty[s8], ((g / kV8Stages) & 1) ^ 1, abort, status))) break;
          mbar_arrive_expect_tx(&bars->v8_full[s8], kCodeTile);
          tma_load_3d(sV8 + s8 * kCodeTile, &maps.v, &bars->v8_full[s8], 0, j * kTile, pc.h);
        }
      }
      if (!ok) {
        // let loads in flight land before the CTA exits (barriers a load was not issued on
        // complete their older phases at once, or run into the short limit)
        if (np > 0) mbar_wait_drain(&bars->q_full, (np - 1) & 1, 20000000ull);
        for (int i = max(0, g - kKStages); i <= g; ++i) {
          mbar_wait_drain(&bars->k_full[i % kKStages], (i / kKStages) & 1, 20000000ull);
          if (i > g - kV8Stages) mbar_wait_drain(&bars->v8_full[i % kV8Stages], (i / kV8Stages) & 1, 20000000ull);
        }
      }
    } else if (warp == 2) {
      // ------------------------------------------------------------ scales
      // lanes 0..15: K's, then V's scale of a tile's eight 16-token chunks, fetched a tile
      // ahead of the ring
      const int blocks = a.c.cap >> a.c.shift;
      bool ok = true;
      int g = 0, gb = 0;  // tiles so far; those that query tile B reads too
      Q8Walk it;
      it.init(S, blockIdx.x);
      Q8Piece pc;
      while (ok && it.next(S, pc)) {
        const int n = q8_len(a.c.len, pc.h, a.c.cap);
        const bool pair = ntq(pc.r) == 2;
        const float* sp = (lane < 8 ? a.c.ks : a.c.vs) + static_cast<size_t>(pc.h) * blocks;
        auto fetch = [&](int j) {
          return lane < 16 ? __ldg(sp + (min(j * kTile + (lane & 7) * 16, n - 1) >> a.c.shift)) : 1.f;
        };
        float next = fetch(pc.j0);
        const float per_unit = pow2f(-sum_unit(a.c.vs + static_cast<size_t>(pc.h) * blocks));
        for (int j = pc.j0; j < pc.j1; ++j, ++g) {
          const float s = next;
          if (j + 1 < pc.j1) next = fetch(j + 1);
          const int st = g % kScStages;
          ok = mbar_wait_step(&bars->sc_empty[st], ((g / kScStages) & 1) ^ 1, abort, status);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          float* to = sScale + st * 24 + (lane & 7);
          if (lane < 8) {
            to[0] = s;
          } else if (lane < 16) {
            to[8] = lg2_approx(s);
            to[16] = 1.f / (s * per_unit);
          }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&bars->sc_full[0][st]);
            if (pair) mbar_arrive(&bars->sc_full[1][gb % kScStages]);
          }
          if (pair) ++gb;
        }
      }
    } else if (warp == 1 || warp == 3) {
      // ------------------------------------------------------------ MMA
      // One warp per query tile: the issuing thread is held until the tensor core has taken
      // its MMAs, and then needs ~400 clk for the barriers of its next ones; with two, the
      // other tile's MMAs run meanwhile.  One elected lane issues.
      const int t = warp >> 1;
      const bool leader = elect_one();
      // f32 accumulator (bit 4), formats 0: E4M3 for kind::f8f6f4, fp16 for kind::f16
      constexpr uint32_t idS = (1u << 4) | (static_cast<uint32_t>(kTile >> 3) << 17) | (8u << 24);
      constexpr uint32_t idO = (1u << 4) | (1u << 16) | (static_cast<uint32_t>(D >> 3) << 17) | (8u << 24);
      constexpr uint32_t kLayout = D == 128 ? 2u : 4u;  // 128- or 64-byte swizzle: a row of codes
      const uint64_t qd = sdesc(smem_u32(sQ) + 2 * t * kCodeTile, 16, 8 * D, kLayout);
      const uint64_t kd = sdesc(smem_u32(sK), 16, 8 * D, kLayout);
      const uint64_t vd = sdesc_sw128(smem_u32(sV), 16384, 1024);
      const uint32_t dS = tmem + t * kTile, dO = tmem + 256 + t * kTile;
      bool ok = true, issued = false;
      int kst = 0, vst = 0, sst = 0, np = 0;  // ring positions of the next K, V, scale slot
      uint32_t kph = 0, vph = 0, pph = 0;     // phases of k_full, v_full, p_full[t]
      Q8Walk it;
      it.init(S, blockIdx.x);
      Q8Piece pc;
      auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait_step(bar, parity, abort, status));
      };
      for (;;) {
        if (!__all_sync(0xffffffffu, it.next(S, pc))) break;
        const int nj = __reduce_min_sync(0xffffffffu, pc.j1 - pc.j0);
        const bool mine = t < ntq(pc.r);  // else this tile has no rows: only hand the slots back
        if (!(ok = wait(&bars->q_full, np & 1))) break;
        for (int j = 0; j <= nj && ok; ++j) {
          // P V of tile j - 1, then the scores of tile j, over the P that has just been read
          if (j < nj && !(ok = wait(&bars->k_full[kst], kph))) break;
          if (j > 0 && !(ok = wait(&bars->v_full[vst], vph))) break;
          tc_fence_after();
          if (mine) {
            if (j > 0) {
              if (!(ok = wait(&bars->p_full[t], pph))) break;
              pph ^= 1u;
              tc_fence_after();
              if (leader) {
                const uint64_t vb = vd + static_cast<uint32_t>(vst) * (kHalfTile >> 4);
#pragma unroll
                for (int kk = 0; kk < kTile / 16; ++kk)
                  mma_f16_ts(dO, dS + kk * 8, vb + kk * 128, idO, (j > 1 || kk > 0) ? 1u : 0u);
                if (j == nj) mma_commit(&bars->o_full[t]);
              }
            }
            if (j < nj && leader) {
              const uint64_t kb = kd + static_cast<uint32_t>(kst) * (kCodeTile >> 4);
#pragma unroll
              for (int part = 0; part < 2; ++part)
#pragma unroll
                for (int kk = 0; kk < D / 32; ++kk)
                  mma_f8_ss(dS, qd + part * (kCodeTile >> 4) + kk * 2, kb + kk * 2, idS, (part > 0 || kk > 0) ? 1u : 0u);
              mma_commit(&bars->s_full[t]);
            }
            issued = true;
          }
          if (j > 0) {
            // P V done: V's slot is free, and so are the scales its softmax read
            if (leader) {
              mma_commit(&bars->v_empty[vst]);
              mma_commit(&bars->sc_empty[sst]);
            }
            sst = (sst + 1) % kScStages;
            if (++vst == kVStages) vst = 0, vph ^= 1u;
          }
          if (j < nj) {
            if (leader) {
              mma_commit(&bars->k_empty[kst]);
              if (j == nj - 1) mma_commit(&bars->q_empty);
            }
            if (++kst == kKStages) kst = 0, kph ^= 1u;
          }
        }
        if (!ok) break;
        ++np;
      }
      if (!ok && issued) {
        // no MMA may still write TMEM when it is freed
        if (leader) mma_commit(&bars->mma_done[t]);
        mbar_wait_drain(&bars->mma_done[t], 0, 200000000ull);
      }
    }
  } else if (warp < 8) {
    // -------------------------------------------------------------- V widening
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsWiden));
    const int wt = tid - 128;
    constexpr int kUnits = D / 8;                  // 8-code units per row; a thread keeps its own
    const int u = wt % kUnits, r0 = wt / kUnits;   // and takes every (128 / kUnits)-th row
    constexpr int kStep = 128 / kUnits;            // 8 or 16 rows: the swizzle (row & 7) stays
    const uint8_t* src0 = sV8 + wt * 8;
    uint8_t* dst0 = sV + (u >> 3) * 16384 + r0 * 128 + (((u & 7) ^ (r0 & 7)) << 4);
    bool ok = true;
    int g = 0;
    Q8Walk it;
    it.init(S, blockIdx.x);
    Q8Piece pc;
    while (ok && it.next(S, pc)) {
      const int n = q8_len(a.c.len, pc.h, a.c.cap);
      for (int j = pc.j0; j < pc.j1; ++j, ++g) {
        const int s8 = g % kV8Stages, st = g % kVStages;
        ok = mbar_wait_step(&bars->v_empty[st], ((g / kVStages) & 1) ^ 1, abort, status);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        ok = mbar_wait_step(&bars->v8_full[s8], (g / kV8Stages) & 1, abort, status);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        const int nv = n - j * kTile - r0;
        const uint8_t* src = src0 + s8 * kCodeTile;
        uint8_t* dst = dst0 + st * kHalfTile;
#pragma unroll
        for (int b = 0; b < kUnits; b += 8) {
          uint2 c[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) c[i] = *reinterpret_cast<const uint2*>(src + (b + i) * 1024);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if ((b + i) * kStep >= nv) c[i] = make_uint2(0u, 0u);
            const F16x4 x = e4m3x4_to_f16x4(c[i].x), y = e4m3x4_to_f16x4(c[i].y);
            *reinterpret_cast<uint4*>(dst + (b + i) * kStep * 128) = make_uint4(x.lo, x.hi, y.lo, y.hi);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bars->v_full[st]);
          mbar_arrive(&bars->v8_empty[s8]);
        }
      }
    }
  } else {
    // -------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int t = (warp - 8) >> 2;
    const int q = warp & 3;       // TMEM lane quarter
    const int r = q * 32 + lane;  // row of the query tile
    const uint32_t lane_off = static_cast<uint32_t>(q * 32) << 16;
    const uint32_t tS = tmem + t * kTile + lane_off;
    const uint32_t tO = tmem + 256 + t * kTile + lane_off;
    constexpr size_t kSlot = static_cast<size_t>(kTile) * D + 2 * kTile;
    constexpr size_t kMl = static_cast<size_t>(kTile) * D;  // m, then l, behind O in a slot
    bool ok = true;
    // tiles of the CTA's walk so far, and those of them that this query tile takes part in
    int ns = 0, npt = 0, ngs = 0, gt = 0, gm = 0, np2 = 0;
    auto wait_warp = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait_step(bar, parity, abort, status));
    };
    auto group_sync = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->grp[t]);
      return wait_warp(&bars->grp[t], (ngs++) & 1);
    };
    Q8Walk& it = s_it[warp - 8];
    Q8Piece& pc = s_pc[warp - 8];
    if (lane == 0) it.init(S, blockIdx.x);
    __syncwarp();
    for (;;) {
      int more = 0;
      __syncwarp();
      if (lane == 0) more = it.next(S, pc) ? 1 : 0;
      more = __shfl_sync(0xffffffffu, more, 0);
      __syncwarp();
      if (!more || !ok) break;
      if (t >= ntq(pc.r)) {
        gt += pc.j1 - pc.j0;
        continue;
      }
      const int n = q8_len(a.c.len, pc.h, a.c.cap);
      const int qrow = (pc.r * 2 + t) * kTile + r;
      const size_t row = static_cast<size_t>(pc.h) * a.Nq + qrow;
      const bool pair = ntq(pc.r) == 2;
      const float coef = qrow < a.Nq ? __ldg(args.coef + row) : 1.f;
      float m = -INFINITY, l = 0.f;
      for (int j = pc.j0; j < pc.j1; ++j, ++gt, ++gm) {
        const int nv = n - j * kTile;
        const float* sc = sScale + (gt % kScStages) * 24;
        if (!(ok = wait_warp(&bars->sc_full[t][gm % kScStages], (gm / kScStages) & 1))) break;
        if (!(ok = wait_warp(&bars->s_full[t], ns & 1))) break;
        ++ns;
        tc_fence_after();
        uint32_t v0[32], v1[32], v2[32], v3[32];
        tmem_ld32(tS + 0, v0);
        tmem_ld32(tS + 32, v1);
        tmem_ld32(tS + 64, v2);
        tmem_ld32(tS + 96, v3);
        tmem_wait_ld_reg(v0);
        tmem_wait_ld_reg(v1);
        tmem_wait_ld_reg(v2);
        tmem_wait_ld_reg(v3);
        auto X = [&](int k) -> uint32_t& {
          return k < 32 ? v0[k] : (k < 64 ? v1[k - 32] : (k < 96 ? v2[k - 64] : v3[k - 96]));
        };
        auto F = [&](int k) { return __uint_as_float(X(k)); };
        if (nv < kTile) {
#pragma unroll
          for (int k = 0; k < kTile; ++k)
            if (k >= nv) X(k) = __float_as_uint(-INFINITY);
        }
        // row maximum in log2 units: a 16-token chunk's raw maximum, scaled
        float av[8], lv[8], mc[8];
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          const float4 x = *reinterpret_cast<const float4*>(sc + i), y = *reinterpret_cast<const float4*>(sc + 8 + i);
          // at least the smallest normal float: -inf times it stays -inf
          av[i] = fmaxf(x.x * coef, 1.2e-38f), av[i + 1] = fmaxf(x.y * coef, 1.2e-38f);
          av[i + 2] = fmaxf(x.z * coef, 1.2e-38f), av[i + 3] = fmaxf(x.w * coef, 1.2e-38f);
          lv[i] = y.x, lv[i + 1] = y.y, lv[i + 2] = y.z, lv[i + 3] = y.w;
        }
#pragma unroll
        for (int ch = 0; ch < 8; ++ch) {
          const int k = ch * 16;
          const float c0 = fmax3(F(k), F(k + 1), F(k + 2)), c1 = fmax3(F(k + 3), F(k + 4), F(k + 5)),
                      c2 = fmax3(F(k + 6), F(k + 7), F(k + 8)), c3 = fmax3(F(k + 9), F(k + 10), F(k + 11)),
                      c4 = fmax3(F(k + 12), F(k + 13), F(k + 14));
          mc[ch] = fmaf(fmax3(fmax3(c0, c1, c2), fmax3(c3, c4, F(k + 15)), c0), av[ch], lv[ch]);
        }
        const float mt = fmax3(fmax3(mc[0], mc[1], mc[2]), fmax3(mc[3], mc[4], mc[5]), fmaxf(mc[6], mc[7]));
        float alpha = 1.f, rs = 0.f;
        bool moved = false;
        if (j == pc.j0) {
          m = fmaxf(mt, -3e38f);  // scores past fp32's range are -inf, and weigh 0 against any m
        } else if (mt > m + kRescale) {
          alpha = ex2_approx(m - mt);
          m = mt;
          moved = true;
        }
        // The two query tiles' warps of a scheduler take turns at the exponentials.  Left to
        // themselves they fall into step, and the exponential unit idles while both wait for
        // their products.
        if (pair && (t == 1 || np2 > 0) && !(ok = wait_warp(&bars->turn[t ^ 1][q], (t == 1 ? np2 : np2 - 1) & 1))) break;
        const float mb = kPBias - m;
#pragma unroll
        for (int ch = 0; ch < 8; ++ch) {
          const float2 a2 = make_float2(av[ch], av[ch]), b2 = make_float2(lv[ch] + mb, lv[ch] + mb);
          float2 sum = make_float2(0.f, 0.f);
          uint32_t pk[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int k = ch * 16 + 2 * e;
            const float2 x = __ffma2_rn(make_float2(F(k), F(k + 1)), a2, b2);
            const float2 p = make_float2(ex2_approx(x.x), ex2_approx(x.y));
            sum = __fadd2_rn(sum, p);
            pk[e] = pack_f16x2(p.x, p.y);
          }
          tmem_st8(tS + ch * 8, pk);
          rs = fmaf(sum.x + sum.y, sc[16 + ch], rs);
        }
        if (pair) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->turn[t][q]);
          ++np2;
        }
        // O_t is stable here (PV_t(j-1) completed before S_t(j) did), and PV_t(j) waits for
        // this tile's P
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t v[32];
            tmem_ld32(tO + c * 32, v);
            tmem_wait_ld_reg(v);
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * alpha);
            tmem_st32(tO + c * 32, v);
          }
        }
        l = fmaf(l, alpha, rs);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->p_full[t]);
      }
      if (!ok) break;
      const int unit = sum_unit(a.c.vs + static_cast<size_t>(pc.h) * (a.c.cap >> a.c.shift));
      if (!(ok = wait_warp(&bars->o_full[t], npt & 1))) break;
      ++npt;
      tc_fence_after();
      __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(a.O) + row * D;
      if (pc.npieces == 1) {
        const float inv = inverse_sum(l) * pow2f(unit);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t v[32];
          tmem_ld32(tO + c * 32, v);
          tmem_wait_ld_reg(v);
          if (qrow < a.Nq) {
#pragma unroll
            for (int k = 0; k < 32; k += 8) {
              uint4 o;
              o.x = pack_bf16x2(__uint_as_float(v[k + 0]) * inv, __uint_as_float(v[k + 1]) * inv);
              o.y = pack_bf16x2(__uint_as_float(v[k + 2]) * inv, __uint_as_float(v[k + 3]) * inv);
              o.z = pack_bf16x2(__uint_as_float(v[k + 4]) * inv, __uint_as_float(v[k + 5]) * inv);
              o.w = pack_bf16x2(__uint_as_float(v[k + 6]) * inv, __uint_as_float(v[k + 7]) * inv);
              *reinterpret_cast<uint4*>(orow + c * 32 + k) = o;
            }
          }
        }
        if (a.lse && qrow < a.Nq) a.lse[row] = (m - (kPBias + unit) + log2f(l)) * kLn2;
        continue;
      }
      // a piece of a cut unit: O as [D/4][128] float4, so that neighbouring rows are
      // neighbouring words, then m and l
      float* slot = a.part + static_cast<size_t>((blockIdx.x * 2 + pc.which) * 2 + t) * kSlot;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t v[32];
        tmem_ld32(tO + c * 32, v);
        tmem_wait_ld_reg(v);
#pragma unroll
        for (int k = 0; k < 32; k += 4)
          reinterpret_cast<float4*>(slot)[static_cast<size_t>(c * 8 + k / 4) * kTile + r] =
              make_float4(__uint_as_float(v[k]), __uint_as_float(v[k + 1]), __uint_as_float(v[k + 2]),
                          __uint_as_float(v[k + 3]));
      }
      slot[kMl + r] = m;
      slot[kMl + kTile + r] = l;
      __threadfence();
      if (!(ok = group_sync())) break;
      if (r == 0) {
        unsigned int* cp = args.cnt + (static_cast<size_t>(pc.h) * npair + pc.r) * 2 + t;
        bars->last[t] = atomicAdd(cp, 1u) + 1u == static_cast<unsigned int>(pc.npieces) ? 1 : 0;
      }
      if (!(ok = group_sync())) break;
      if (!bars->last[t]) continue;
      __threadfence();
      // the last piece merges them all, row by row, in their order
      auto slot_of = [&](int k) -> const float* {
        return a.part + static_cast<size_t>(((pc.cfirst + k) * 2 + (k == 0 ? pc.wfirst : 0)) * 2 + t) * kSlot;
      };
      // four pieces' loads in flight at a time: one after another they were 60 of the 100 us
      // of 64 queries over 12 heads of 15600 tokens
      constexpr int kAhead = 4;
      float M = -INFINITY;
      for (int k0 = 0; k0 < pc.npieces; k0 += 2 * kAhead) {
        float x[2 * kAhead];
#pragma unroll
        for (int u = 0; u < 2 * kAhead; ++u) x[u] = __ldcg(slot_of(min(k0 + u, pc.npieces - 1)) + kMl + r);
#pragma unroll
        for (int u = 0; u < 2 * kAhead; ++u) M = fmaxf(M, x[u]);
      }
      float L = 0.f;
      for (int k0 = 0; k0 < pc.npieces; k0 += kAhead) {
        float x[kAhead], y[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const float* s = slot_of(min(k0 + u, pc.npieces - 1)) + kMl + r;
          x[u] = __ldcg(s);
          y[u] = __ldcg(s + kTile);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
          if (k0 + u < pc.npieces) L = fmaf(y[u], ex2_approx(x[u] - M), L);
      }
      const float inv = inverse_sum(L) * pow2f(unit);
#pragma unroll 1
      for (int c4 = 0; c4 < D / 4; c4 += 4) {
        float4 acc[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int k0 = 0; k0 < pc.npieces; k0 += kAhead) {
          float4 x[kAhead][4];
          float w[kAhead];
#pragma unroll
          for (int u = 0; u < kAhead; ++u) {
            const float* s = slot_of(min(k0 + u, pc.npieces - 1));
            w[u] = __ldcg(s + kMl + r);
#pragma unroll
            for (int c = 0; c < 4; ++c)
              x[u][c] = __ldcg(reinterpret_cast<const float4*>(s) + static_cast<size_t>(c4 + c) * kTile + r);
          }
#pragma unroll
          for (int u = 0; u < kAhead; ++u) {
            if (k0 + u >= pc.npieces) continue;
            const float f = ex2_approx(w[u] - M) * inv;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              acc[c].x = fmaf(f, x[u][c].x, acc[c].x), acc[c].y = fmaf(f, x[u][c].y, acc[c].y);
              acc[c].z = fmaf(f, x[u][c].z, acc[c].z), acc[c].w = fmaf(f, x[u][c].w, acc[c].w);
            }
          }
        }
        if (qrow < a.Nq) {
#pragma unroll
          for (int c = 0; c < 4; c += 2)
            *reinterpret_cast<uint4*>(orow + (c4 + c) * 4) =
                make_uint4(pack_bf16x2(acc[c].x, acc[c].y), pack_bf16x2(acc[c].z, acc[c].w),
                           pack_bf16x2(acc[c + 1].x, acc[c + 1].y), pack_bf16x2(acc[c + 1].z, acc[c + 1].w));
        }
      }
      if (a.lse && qrow < a.Nq) a.lse[row] = (M - (kPBias + unit) + log2f(L)) * kLn2;
    }
    // rows of heads without tokens: zeros (lse -inf), spread over the CTAs
    if (ok) {
      for (int h = 0; h < a.c.H; ++h) {
        if (sch.T[h] != 0) continue;
        for (int p = q8_first_turn(h, npair, sch.G); p < npair; p += sch.G) {
          if (t >= ntq(p)) continue;
          const int qrow = (p * 2 + t) * kTile + r;
          if (qrow >= a.Nq) continue;
          const size_t row = static_cast<size_t>(h) * a.Nq + qrow;
          uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.O) + row * D);
          for (int c = 0; c < D / 8; ++c) o[c] = make_uint4(0u, 0u, 0u, 0u);
          if (a.lse) a.lse[row] = -INFINITY;
        }
      }
    }
  }

  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
size_t smem_bytes() {
  return 1024 + static_cast<size_t>(kTile) * D * (4 + kKStages + kV8Stages + 2 * kVStages) + kBarBytes;
}

template <int D>
cudaError_t launch(const Q8AttendArgs& a, const Q8ChunkScratch& s, int n_sm, cudaStream_t st) {
  const int npair = (a.Nq + 2 * kTile - 1) / (2 * kTile);
  const long long rows = static_cast<long long>(a.c.H) * a.Nq;
  Maps maps;
  if (!make_tmap_u8(&maps.hi, s.hi, D, a.Nq, a.c.H, kTile, true) ||
      !make_tmap_u8(&maps.lo, s.lo, D, a.Nq, a.c.H, kTile, true) ||
      !make_tmap_u8(&maps.k, a.c.K, D, a.c.cap, a.c.H, kTile, true) ||
      !make_tmap_u8(&maps.v, a.c.V, D, a.c.cap, a.c.H, kTile, false))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(q8_attend_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem_bytes<D>()));
  if (e != cudaSuccess) return e;
  // the warpgroups' register shares come out of what the launch is given: more would
  // wait for ever
  cudaFuncAttributes fa;
  e = cudaFuncGetAttributes(&fa, q8_attend_kernel<D>);
  if (e != cudaSuccess) return e;
  if (fa.numRegs * 4 < kRegsControl + kRegsWiden + 2 * kRegsSoftmax) return cudaErrorLaunchOutOfResources;
  e = launch_q8_split_q(a.Q, nullptr, rows, D, a.scale, s, a.c.H * npair * 2, n_sm, st);
  if (e != cudaSuccess) return e;
  Args args{a, s.coef, s.cnt};
  args.a.part = s.part;
  LaunchTrace trace("q8_attend_kernel", st);
  return launch_pdl(q8_attend_kernel<D>, dim3(n_sm < kQ8MaxCtas ? n_sm : kQ8MaxCtas), dim3(kThreads), smem_bytes<D>(),
                    st, maps, args);
}

}  // namespace

cudaError_t launch_q8_split_q(const void* Q, const float* lse, long long rows, int d, float scale,
                              const Q8ChunkScratch& s, int ncnt, int n_sm, cudaStream_t st) {
  const long long per = 8 * (256 / d) * kSplitFlight, need = (rows + per - 1) / per;  // rows of a CTA
  const int grid = static_cast<int>(need < 16LL * n_sm ? need : 16LL * n_sm);
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(Q);
  LaunchTrace trace("q8_split_q_kernel", st);
  return d == 128 ? launch_pdl(q8_split_q_kernel<128>, dim3(grid), dim3(256), 0, st, q, lse, rows, scale, s.hi, s.lo,
                               s.coef, s.cnt, ncnt)
                  : launch_pdl(q8_split_q_kernel<64>, dim3(grid), dim3(256), 0, st, q, lse, rows, scale, s.hi, s.lo,
                               s.coef, s.cnt, ncnt);
}

cudaError_t launch_q8_attend_chunk(const Q8AttendArgs& a, const Q8ChunkScratch& s, int n_sm, cudaStream_t st) {
  return a.c.d == 128 ? launch<128>(a, s, n_sm, st) : launch<64>(a, s, n_sm, st);
}

}  // namespace kvb
