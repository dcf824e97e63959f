// Attention weights of a chunk of queries over the 8-bit cache, on the 5th-generation
// tensor cores:  mass[k] = decay prev[k] + sum_q 2^(ks (q.k) coef_q - lse_q log2 e).
//
// Keys are the rows of the product and queries its columns, so a thread owns a key and a
// half of the columns and its sum stays in a register; nothing crosses threads but the
// two halves.  The product is the attention's, S = K hi^T + K lo^T in kind::f8f6f4 with
// the cache's bytes from TMA and the queries' two E4M3 parts (q8_split_q_kernel); the
// softmax is known (lse), so there is no maximum to track and V is not read.
// Work is the sequence of (256-key block, 256-query tile) steps over all heads, cut
// evenly over a persistent grid.  A CTA keeps its block's codes in shared memory and
// streams query tiles through a 2-stage ring; two 128 x 256 accumulators in TMEM
// ping-pong between the tensor core and eight epilogue warps each.  A block cut between
// CTAs is summed, in order, by whichever warp comes last to its 32 keys.
// What bounds it: exponentials.  A step is 65536 of them, 4096 clk at the unit's 16 per
// clock and SM, against 2048 clk of tensor time (12 heads x 4680 queries x 15600 tokens:
// 306 us; 16-row tiles on mma.sync took 2466).  One pair in eight as a polynomial on the FMA
// pipe took 1 to 2 % less, but its 2^n, put together from bits, is no infinity past 2^128,
// where a caller's lse far below the scores leads.
// Warps: 0 loads, 1 MMA, 2 TMEM, 3 column coefficients, 4-11 epilogue of row tile 0,
// 12-19 of row tile 1 (4 lane quarters x 2 column halves).
#include "host_util.h"
#include "q8.cuh"
#include "sm100.cuh"

namespace kvb {
using namespace sm100;

namespace {

constexpr int kThreads = 640;
constexpr int kRowTile = 128, kBlock = 256, kCols = 256;
constexpr int kStages = 2;
constexpr int kBarBytes = 256;

struct alignas(8) Bars {
  uint64_t a_full, a_empty;
  uint64_t full[kStages], empty[kStages];
  uint64_t c_full[kStages], c_empty[kStages];  // column coefficients
  uint64_t acc_full[2], acc_empty[2];
  uint64_t half[2][2][4];  // by parity of the finished block, row tile, lane quarter: the second column half's sums
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Bars) <= kBarBytes, "barrier block overflows its reservation");

struct Maps {
  CUtensorMap k, hi, lo;
};

struct Args {
  Q8MassArgs a;
  const float* coef;  // [H][Nq]
  float* part;        // [CTA][2][kBlock] sums of cut blocks
  unsigned int* cnt;  // [CTA][2][8] arrivals of a cut block's warps, at its first piece's slot; zeroed
};

// Key blocks of all heads in one sequence; column tiles are the same for every head.
struct Blocks {
  int C[kQ8MaxHeads + 1];  // blocks before each head
  long long total;         // steps
  int G, CT;
};

// One CTA's steps [L0, L1), block by block.
struct Walk {
  long long L, L1;
  int h = 0;
  __device__ void init(const Blocks& b, int cta) {
    L = cta < b.G ? b.total * cta / b.G : 0;
    L1 = cta < b.G ? b.total * (cta + 1) / b.G : 0;
  }
};
struct Piece {
  int h, rb, c0, c1;   // head, key block of the head, column tiles
  long long gb;        // key block of the sequence
};
__device__ __forceinline__ bool next_piece(const Blocks& b, int H, Walk& w, Piece& p) {
  if (w.L >= w.L1) return false;
  p.gb = w.L / b.CT;
  p.c0 = static_cast<int>(w.L - p.gb * b.CT);
  const long long left = w.L1 - w.L;
  p.c1 = p.c0 + static_cast<int>(left < b.CT - p.c0 ? left : b.CT - p.c0);
  int lo = w.h, hi = H;  // the last head with C[h] <= gb
  while (hi - lo > 1) {
    const int m = (lo + hi) / 2;
    if (b.C[m] <= p.gb) lo = m;
    else hi = m;
  }
  w.h = p.h = lo;
  p.rb = static_cast<int>(p.gb - b.C[lo]);
  w.L += p.c1 - p.c0;
  return true;
}
__device__ __forceinline__ int cta_of(const Blocks& b, long long L) {
  return static_cast<int>(((L + 1) * b.G - 1) / b.total);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) q8_mass_kernel(const __grid_constant__ Maps maps, const Args args) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Blocks blk;
  __shared__ alignas(16) float s_coef[kStages][kCols], s_nl[kStages][kCols];
  __shared__ float s_half[2][2][kRowTile];  // by parity of the finished block: sums of the second column half
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const Q8MassArgs& a = args.a;
  constexpr uint32_t kA = kRowTile * D, kB = kCols * D;  // bytes of a row tile, of one part of a column tile
  uint8_t* sA = smem;
  uint8_t* sB = sA + 2 * kA;  // kStages x (hi, lo)
  Bars* bars = reinterpret_cast<Bars*>(sB + kStages * 2 * kB);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    mbar_init(&bars->a_full, 1);
    mbar_init(&bars->a_empty, 1);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bars->full[i], 1);
      mbar_init(&bars->empty[i], 1);
      mbar_init(&bars->c_full[i], 1);
      mbar_init(&bars->c_empty[i], 16);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->acc_full[i], 1);
      mbar_init(&bars->acc_empty[i], 8);
      for (int k = 0; k < 4; ++k) {
        mbar_init(&bars->half[0][i][k], 1);
        mbar_init(&bars->half[1][i][k], 1);
      }
    }
    mbar_init(&bars->mma_done, 1);
    bars->abort = 0;
    fence_barrier_init();
  }
  if (warp == 2) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  // lengths, query parts and coefficients come from earlier work on the stream
  pdl_wait();
  pdl_trigger();
  if (warp == 3) {
    int carry = 0;
    for (int b = 0; b < a.c.H; b += 32) {
      const int h = b + lane;
      const int n = h < a.c.H ? (q8_len(a.c.len, h, a.c.cap) + kBlock - 1) / kBlock : 0;
      int x = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (h < a.c.H) blk.C[h] = carry + x - n;
      carry += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) {
      blk.C[a.c.H] = carry;
      blk.CT = (a.Nq + kCols - 1) / kCols;
      blk.total = static_cast<long long>(carry) * blk.CT;
      blk.G = static_cast<int>(blk.total < gridDim.x ? blk.total : gridDim.x);
    }
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  volatile int* abort = &bars->abort;
  int* status = a.c.status;
  auto row_tiles = [&](const Piece& p) {
    return q8_len(a.c.len, p.h, a.c.cap) - p.rb * kBlock > kRowTile ? 2 : 1;
  };
  Walk w;
  w.init(blk, blockIdx.x);
  Piece p;

  if (warp == 0) {
    // ------------------------------------------------------------ loads
    if (lane == 0) {
      prefetch_tmap(&maps.k);
      prefetch_tmap(&maps.hi);
      prefetch_tmap(&maps.lo);
      bool ok = true;
      int g = 0, na = 0;
      while (ok && next_piece(blk, a.c.H, w, p)) {
        if (na > 0 && !(ok = mbar_wait_step(&bars->a_empty, (na - 1) & 1, abort, status))) break;
        const int nt = row_tiles(p);
        mbar_arrive_expect_tx(&bars->a_full, nt * kA);
        for (int t = 0; t < nt; ++t) tma_load_3d(sA + t * kA, &maps.k, &bars->a_full, 0, p.rb * kBlock + t * kRowTile, p.h);
        ++na;
        for (int c = p.c0; c < p.c1; ++c, ++g) {
          const int st = g % kStages;
          if (!(ok = mbar_wait_step(&bars->empty[st], ((g / kStages) & 1) ^ 1, abort, status))) break;
          mbar_arrive_expect_tx(&bars->full[st], 2 * kB);
          tma_load_3d(sB + (2 * st) * kB, &maps.hi, &bars->full[st], 0, c * kCols, p.h);
          tma_load_3d(sB + (2 * st + 1) * kB, &maps.lo, &bars->full[st], 0, c * kCols, p.h);
        }
      }
      if (!ok) {
        // let loads in flight land before the CTA exits
        if (na > 0) mbar_wait_drain(&bars->a_full, (na - 1) & 1, 200000000ull);
        for (int i = max(0, g - kStages); i < g; ++i)
          mbar_wait_drain(&bars->full[i % kStages], (i / kStages) & 1, 200000000ull);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA
    const bool leader = elect_one();
    constexpr uint32_t id = (1u << 4) | (static_cast<uint32_t>(kCols >> 3) << 17) | (8u << 24);
    constexpr uint32_t kLayout = D == 128 ? 2u : 4u;
    const uint64_t ad = sdesc(smem_u32(sA), 16, 8 * D, kLayout), bd = sdesc(smem_u32(sB), 16, 8 * D, kLayout);
    bool ok = true, issued = false;
    int g = 0, na = 0;
    uint32_t eph = 0;  // acc_empty phases, bit t
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait_step(bar, parity, abort, status));
    };
    while (ok && __all_sync(0xffffffffu, next_piece(blk, a.c.H, w, p))) {
      const int nt = __reduce_min_sync(0xffffffffu, row_tiles(p));
      const int nc = __reduce_min_sync(0xffffffffu, p.c1 - p.c0);
      if (!(ok = wait(&bars->a_full, na & 1))) break;
      ++na;
      for (int c = 0; c < nc && ok; ++c, ++g) {
        const int st = g % kStages;
        if (!(ok = wait(&bars->full[st], (g / kStages) & 1))) break;
        for (int t = 0; t < nt; ++t) {
          if (!(ok = wait(&bars->acc_empty[t], ((eph >> t) & 1u) ^ 1u))) break;
          eph ^= 1u << t;
          tc_fence_after();
          if (leader) {
            const uint64_t aa = ad + static_cast<uint32_t>(t) * (kA >> 4);
            const uint64_t bb = bd + static_cast<uint32_t>(2 * st) * (kB >> 4);
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
              for (int kk = 0; kk < D / 32; ++kk)
                mma_f8_ss(tmem + t * kCols, aa + kk * 2, bb + part * (kB >> 4) + kk * 2, id, (part > 0 || kk > 0) ? 1u : 0u);
            mma_commit(&bars->acc_full[t]);
          }
          issued = true;
        }
        if (!ok) break;
        if (leader) {
          mma_commit(&bars->empty[st]);
          if (c == nc - 1) mma_commit(&bars->a_empty);
        }
      }
    }
    if (!ok && issued) {
      if (leader) mma_commit(&bars->mma_done);
      mbar_wait_drain(&bars->mma_done, 0, 200000000ull);
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------ column coefficients
    bool ok = true;
    int g = 0;
    while (ok && next_piece(blk, a.c.H, w, p)) {
      for (int c = p.c0; c < p.c1; ++c, ++g) {
        const int st = g % kStages;
        float cf[kCols / 32], nl[kCols / 32];
#pragma unroll
        for (int k = 0; k < kCols / 32; ++k) {
          const int q = c * kCols + k * 32 + lane;
          cf[k] = 0.f;
          nl[k] = -INFINITY;  // no such row, or one that saw nothing: weighs nothing
          if (q < a.Nq) {
            const size_t row = static_cast<size_t>(p.h) * a.Nq + q;
            cf[k] = __ldg(args.coef + row);
            const float z = __ldg(a.lse + row);
            if (z != -INFINITY) nl[k] = -z * kLog2e;
          }
        }
        ok = mbar_wait_step(&bars->c_empty[st], ((g / kStages) & 1) ^ 1, abort, status);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
#pragma unroll
        for (int k = 0; k < kCols / 32; ++k) {
          s_coef[st][k * 32 + lane] = cf[k];
          s_nl[st][k * 32 + lane] = nl[k];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->c_full[st]);
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    const int t = (warp - 4) >> 3, q = warp & 3, half = ((warp - 4) >> 2) & 1;
    const int r = q * 32 + lane;
    const uint32_t taddr = tmem + t * kCols + half * (kCols / 2) + (static_cast<uint32_t>(q * 32) << 16);
    bool ok = true;
    int g = 0, nacc = 0, nblk = 0;
    auto wait_warp = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait_step(bar, parity & 1u, abort, status));
    };
    while (ok && next_piece(blk, a.c.H, w, p)) {
      const int n = q8_len(a.c.len, p.h, a.c.cap);
      const int key = p.rb * kBlock + t * kRowTile + r;
      const bool mine = t < row_tiles(p);
      const float ks = __ldg(a.c.ks + static_cast<size_t>(p.h) * (a.c.cap >> a.c.shift) + (min(key, n - 1) >> a.c.shift));
      const float2 ks2 = make_float2(ks, ks);
      float2 sum = make_float2(0.f, 0.f);
      for (int c = p.c0; c < p.c1; ++c, ++g) {
        const int st = g % kStages;
        if (!(ok = wait_warp(&bars->c_full[st], g / kStages))) break;
        if (mine) {
          if (!(ok = wait_warp(&bars->acc_full[t], nacc++))) break;
          tc_fence_after();
          const float* cf = s_coef[st] + half * (kCols / 2);
          const float* nl = s_nl[st] + half * (kCols / 2);
          // four loads of 32 columns, the next in flight over this one's exponentials
          uint32_t va[32], vb[32];
          auto weigh = [&](const uint32_t (&v)[32], int k) {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float4 cc = *reinterpret_cast<const float4*>(cf + k + e), nn = *reinterpret_cast<const float4*>(nl + k + e);
              // the two scales first, as in the attention: a raw product times a key scale may pass fp32's range
              const float2 x = __ffma2_rn(make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])),
                                          __fmul2_rn(make_float2(cc.x, cc.y), ks2), make_float2(nn.x, nn.y));
              const float2 y = __ffma2_rn(make_float2(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3])),
                                          __fmul2_rn(make_float2(cc.z, cc.w), ks2), make_float2(nn.z, nn.w));
              sum = __fadd2_rn(sum, make_float2(ex2_approx(x.x), ex2_approx(x.y)));
              sum = __fadd2_rn(sum, make_float2(ex2_approx(y.x), ex2_approx(y.y)));
            }
          };
          tmem_ld32(taddr, va);
          tmem_wait_ld_reg(va);
          tmem_ld32(taddr + 32, vb);
          weigh(va, 0);
          tmem_wait_ld_reg(vb);
          tmem_ld32(taddr + 64, va);
          weigh(vb, 32);
          tmem_wait_ld_reg(va);
          tmem_ld32(taddr + 96, vb);
          weigh(va, 64);
          tmem_wait_ld_reg(vb);
          // the last columns are in registers: the accumulator is free
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->acc_empty[t]);
          weigh(vb, 96);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->c_empty[st]);
      }
      if (!ok) break;
      // the block is done (here): both column halves, then the pieces of other CTAs
      if (!mine) continue;
      const int par = nblk++ & 1;
      float s = sum.x + sum.y;
      if (half == 1) {
        s_half[par][t][r] = s;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->half[par][t][q]);
        continue;
      }
      if (!(ok = wait_warp(&bars->half[par][t][q], (nblk - 1) >> 1))) break;
      s += s_half[par][t][r];
      const long long b0 = p.gb * blk.CT;
      const int cf0 = cta_of(blk, b0), cl = cta_of(blk, b0 + blk.CT - 1);
      const size_t at = static_cast<size_t>(p.h) * a.c.cap + key;
      if (cf0 != cl) {
        // slot 1 of a CTA is the block its range ends in, slot 0 the one it begins in
        const int which = static_cast<int>(blockIdx.x) == cf0 ? 1 : 0;
        args.part[(static_cast<size_t>(blockIdx.x) * 2 + which) * kBlock + t * kRowTile + r] = s;
        __threadfence();
        __syncwarp();
        int last = 0;
        if (lane == 0)
          last = atomicAdd(args.cnt + (static_cast<size_t>(cf0) * 2 + 1) * 8 + t * 4 + q, 1u) == static_cast<unsigned int>(cl - cf0);
        if (!__shfl_sync(0xffffffffu, last, 0)) continue;
        __threadfence();
        s = 0.f;
        for (int k = cf0; k <= cl; ++k)
          s += __ldcg(args.part + (static_cast<size_t>(k) * 2 + (k == cf0 ? 1 : 0)) * kBlock + t * kRowTile + r);
      }
      if (key < n) a.mass[at] = a.prev ? fmaf(a.decay, a.prev[at], s) : s;
    }
  }

  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch(const Q8MassArgs& a, const Q8ChunkScratch& s, int n_sm, cudaStream_t st) {
  Maps maps;
  if (!make_tmap_u8(&maps.k, a.c.K, D, a.c.cap, a.c.H, kRowTile, true) ||
      !make_tmap_u8(&maps.hi, s.hi, D, a.Nq, a.c.H, kCols, true) ||
      !make_tmap_u8(&maps.lo, s.lo, D, a.Nq, a.c.H, kCols, true))
    return cudaErrorInvalidValue;
  constexpr size_t smem = 1024 + 2 * kRowTile * D + kStages * 2 * kCols * D + kBarBytes;
  cudaError_t e = cudaFuncSetAttribute(q8_mass_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  e = launch_q8_split_q(a.Q, a.lse, static_cast<long long>(a.c.H) * a.Nq, D, a.scale, s, kQ8MassCounters, n_sm, st);
  if (e != cudaSuccess) return e;
  const Args args{a, s.coef, s.part, s.cnt};
  LaunchTrace trace("q8_mass_kernel", st);
  return launch_pdl(q8_mass_kernel<D>, dim3(n_sm < kQ8MaxCtas ? n_sm : kQ8MaxCtas), dim3(kThreads), smem, st, maps, args);
}

}  // namespace

cudaError_t launch_q8_mass_chunk(const Q8MassArgs& a, const Q8ChunkScratch& s, int n_sm, cudaStream_t st) {
  return a.c.d == 128 ? launch<128>(a, s, n_sm, st) : launch<64>(a, s, n_sm, st);
}

}  // namespace kvb
