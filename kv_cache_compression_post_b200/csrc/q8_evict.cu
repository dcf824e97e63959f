// kvb_q8_evict: cut every head to a budget by accumulated attention weight.
//
// q8_select_kernel, a cluster of eight CTAs per head: the weight of the last token to
// stay is found digit by digit (8 bits of the order-preserving integer of a float, from
// the top: a radix select, up to four passes over keys held in shared memory, the CTAs'
// histograms exchanged over distributed shared memory; over once all keys of the digits
// found stay), then each warp counts and writes the
// positions of its own run of tokens, so the list comes out in order and of equal weights
// the lower positions stay.  Bound by latency: a head has one answer per pass to wait for
// (one CTA per head took 150 us for 8 heads of 131072 tokens).
// q8_gather_kernel, one CTA per 128 tokens of the result: reads and writes each kept row
// once, every word of its rows in flight at once.  The result's block takes the largest
// scale among its tokens; rows from blocks of smaller scale are rounded anew (exactly
// scaled where both are powers of two), others are copied bit for bit.
#include <cooperative_groups.h>

#include "host_util.h"
#include "q8.cuh"

namespace cg = cooperative_groups;

namespace kvb {
namespace {

constexpr int kSelCtas = 8;  // a head's cluster
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kCopies = 8;         // histograms, so that equal digits of a warp meet less often
constexpr int kSelKeys = 16384;    // keys of a CTA that stay in shared memory between the passes

__device__ __forceinline__ uint32_t weight_key(float w) {
  return w != w ? 0u : float_key(w + 0.f);  // NaN least; -0 as 0
}

struct SelShared {
  uint32_t key[kSelKeys];
  alignas(16) int in[2][kSelCtas][256];  // by parity of the pass: every CTA's digit counts, largest digit first
  int hist[kCopies][257];  // a bin's copies in different banks
  int above[kSelWarps], equal[kSelWarps];
  int cta[2][kSelCtas];  // every CTA's
  uint32_t prefix;
  int need;
  bool done;
};

__global__ void __cluster_dims__(kSelCtas, 1, 1) __launch_bounds__(kSelThreads) q8_select_kernel(const Q8EvictArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  SelShared& s = *reinterpret_cast<SelShared*>(smem);
  cg::cluster_group cluster = cg::this_cluster();
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  pdl_wait();
  pdl_trigger();
  const int rank = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = q8_len(a.src.len, h, a.src.cap);
  int* kept = a.kept + static_cast<size_t>(h) * a.budget;
  // every CTA of the cluster runs: its shared memory may be written to
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  if (n <= a.budget) {
    for (int i = rank * kSelThreads + tid; i < n; i += kSelCtas * kSelThreads) kept[i] = i;
    if (rank == 0 && tid == 0) a.len[h] = n;
    return;
  }
  const float* mass = a.mass + static_cast<size_t>(h) * a.src.cap;
  const int lo = a.sink, hi = n - a.recent;
  const int need = a.budget - a.sink - a.recent;
  // every warp of the cluster has one run of tokens, a multiple of 32 long
  const int run = ((n + kSelCtas * kSelWarps - 1) / (kSelCtas * kSelWarps) + 31) & ~31;
  const int c0 = min(rank * kSelWarps * run, n), c1 = min(c0 + kSelWarps * run, n);
  const bool held = c1 - c0 <= kSelKeys;
  auto key_at = [&](int i) { return held ? s.key[i - c0] : weight_key(__ldg(mass + i)); };
  if (held) {
    for (int i = c0 + tid; i < c1; i += kSelThreads) s.key[i - c0] = weight_key(__ldg(mass + i));
  }
  // the need-th largest key of [lo, hi): the digits found so far, and how many of the keys
  // that share them all stay
  uint32_t thr = 0xFFFFFFFFu;
  int quota = 0;
  if (need > 0) {
    if (tid == 0) {
      s.prefix = 0u;
      s.need = need;
      s.done = false;
    }
    for (int i = tid; i < kCopies * 257; i += kSelThreads) (&s.hist[0][0])[i] = 0;
    __syncthreads();
    const int p0 = max(c0, lo), p1 = min(c1, hi);
    for (int pass = 0; pass < 4; ++pass) {
      const int shift = 24 - 8 * pass;
      const uint32_t prefix = s.prefix;
      const int want = s.need;
      const uint32_t mask = pass == 0 ? 0u : 0xFFFFFFFFu << (shift + 8);
      for (int i = p0 + tid; i < p1; i += kSelThreads) {
        const uint32_t k = key_at(i);
        if ((k & mask) == prefix) atomicAdd(&s.hist[tid % kCopies][(k >> shift) & 255u], 1);
      }
      __syncthreads();
      // every CTA gives its counts to all, so that after the barrier they are read locally
      if (tid < 256) {
        int v = 0;
#pragma unroll
        for (int c = 0; c < kCopies; ++c) v += s.hist[c][tid];
#pragma unroll
        for (int c = 0; c < kSelCtas; ++c) cluster.map_shared_rank(&s.in[pass & 1][rank][0], c)[255 - tid] = v;
      }
      cluster.sync();
      if (warp == 0) {
        // keys of larger digits, eight digits a lane, from the top
        int v[8] = {0, 0, 0, 0, 0, 0, 0, 0}, mine = 0;
#pragma unroll
        for (int c = 0; c < kSelCtas; ++c) {
          const int4* x = reinterpret_cast<const int4*>(&s.in[pass & 1][c][lane * 8]);
          const int4 a4 = x[0], b4 = x[1];
          v[0] += a4.x, v[1] += a4.y, v[2] += a4.z, v[3] += a4.w;
          v[4] += b4.x, v[5] += b4.y, v[6] += b4.z, v[7] += b4.w;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) mine += v[k];
        int above = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, above, o);
          if (lane >= o) above += y;
        }
        above -= mine;
        if (above < want && above + mine >= want) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            if (above < want && above + v[k] >= want) {
              const uint32_t to = prefix | (static_cast<uint32_t>(255 - lane * 8 - k) << shift);
              s.prefix = to;
              s.need = want - above;
              // all keys with these digits stay: those above the largest key without them
              if (above + v[k] == want && to > 0) {
                s.done = true;
                s.prefix = to - 1;
                s.need = 0;
              }
            }
            above += v[k];
          }
        }
      }
      __syncthreads();
      if (s.done) break;
      // (between the barrier and the scan above, these stores cost 3 us in all)
      for (int i = tid; i < kCopies * 257; i += kSelThreads) (&s.hist[0][0])[i] = 0;
      __syncthreads();
    }
    thr = s.prefix;
    quota = s.need;
  } else {
    __syncthreads();  // the held keys
  }
  const int r0 = min(c0 + warp * run, n), r1 = min(r0 + run, n);
  auto state = [&](int i, bool& stays, bool& equal) {
    const bool in = i < r1;
    const bool forced = in && (i < lo || i >= hi);
    const uint32_t k = in && !forced ? key_at(i) : 0u;
    stays = forced || (in && k > thr);
    equal = in && !forced && need > 0 && k == thr;
  };
  int above = 0, equal_n = 0;
  for (int i = r0; i < r1; i += 32) {
    bool st, eq;
    state(i + lane, st, eq);
    above += __popc(__ballot_sync(0xffffffffu, st));
    equal_n += __popc(__ballot_sync(0xffffffffu, eq));
  }
  if (lane == 0) {
    s.above[warp] = above;
    s.equal[warp] = equal_n;
  }
  __syncthreads();
  if (warp < 2) {
    const int x = __reduce_add_sync(0xffffffffu, (warp ? s.equal : s.above)[lane]);
    if (lane < kSelCtas) *cluster.map_shared_rank(&s.cta[warp][rank], lane) = x;
  }
  // after which no CTA writes to another, so that each may leave when it is done
  cluster.sync();
  // what lies before this warp's run: in the CTAs before, in the warps before
  const int at_cta = lane < rank ? s.cta[0][lane] : 0, eq_cta = lane < rank ? s.cta[1][lane] : 0;
  int at = __reduce_add_sync(0xffffffffu, at_cta + (lane < warp ? s.above[lane] : 0));
  int eq_before = __reduce_add_sync(0xffffffffu, eq_cta + (lane < warp ? s.equal[lane] : 0));
  at += min(eq_before, quota);
  const uint32_t below = (1u << lane) - 1u;
  for (int i = r0; i < r1; i += 32) {
    bool st, eq;
    state(i + lane, st, eq);
    const uint32_t em = __ballot_sync(0xffffffffu, eq);
    const bool keep = st || (eq && eq_before + __popc(em & below) < quota);
    const uint32_t km = __ballot_sync(0xffffffffu, keep);
    if (keep) kept[at + __popc(km & below)] = i + lane;
    at += __popc(km);
    eq_before += __popc(em);
  }
  if (rank == 0 && tid == 0) a.len[h] = a.budget;
}

// 8 heads of 131072 to 32768, with the select: 256 threads 49.7 us, 512 48.5, 1024 55.5
constexpr int kGatherThreads = 512;
constexpr int kGatherTok = 128;  // tokens of the result per CTA: one to eight blocks

// four codes times r, rounded to E4M3
__device__ __forceinline__ uint32_t rescale4(uint32_t c, float r) {
  const float4 x = e4m3x4_to_f32x4(c);
  return f32x4_to_e4m3x4(x.x * r, x.y * r, x.z * r, x.w * r);
}

template <int D>
__global__ void __launch_bounds__(kGatherThreads) q8_gather_kernel(const Q8EvictArgs a) {
  __shared__ int s_src[kGatherTok];
  __shared__ float s_scale[2][kGatherTok], s_to[2][kGatherTok / 16];
  pdl_wait();
  pdl_trigger();
  const int t0 = blockIdx.x * kGatherTok, h = blockIdx.y, tid = threadIdx.x;
  const int shift = a.src.shift;
  const int left = min(q8_len(a.src.len, h, a.src.cap), a.budget);
  const int nt = min(kGatherTok, left - t0);
  if (nt <= 0) return;
  constexpr int kW = D / 16;                              // 16-byte words per row
  constexpr int kN = kGatherTok * kW * 2 / kGatherThreads;  // words per thread, K's and V's
  const size_t from = static_cast<size_t>(h) * a.src.cap;
  const size_t blocks = static_cast<size_t>(h) * (a.src.cap >> shift), to_blocks = static_cast<size_t>(h) * (a.cap >> shift);
  if (tid < nt) s_src[tid] = a.kept[static_cast<size_t>(h) * a.budget + t0 + tid];
  __syncthreads();
  // every row's words, in flight over the scales
  uint4 w[kN];
#pragma unroll
  for (int u = 0; u < kN; ++u) {
    const int i = (tid + u * kGatherThreads) % (kGatherTok * kW);
    const uint8_t* base = u < kN / 2 ? a.src.K : a.src.V;
    if (i / kW < nt) w[u] = __ldg(reinterpret_cast<const uint4*>(base + (from + s_src[i / kW]) * D) + i % kW);
  }
  const int tok = tid & (kGatherTok - 1), kv = tid / kGatherTok;  // the first 256: K's and V's scales
  if (kv < 2 && tok < nt) {
    const int src = s_src[tok];
    s_scale[kv][tok] = __ldg((kv ? a.src.vs : a.src.ks) + blocks + (src >> shift));
    if (kv == 0 && a.to_mass) a.to_mass[static_cast<size_t>(h) * a.cap + t0 + tok] = __ldg(a.mass + from + src);
  }
  __syncthreads();
  const int nb = (nt + (1 << shift) - 1) >> shift;
  if (kv < 2 && tok < nb) {
    float mx = 0.f;
    const int end = min((tok + 1) << shift, nt);
    for (int i = tok << shift; i < end; ++i) mx = fmaxf(mx, s_scale[kv][i]);
    s_to[kv][tok] = mx;
    (kv ? a.vs : a.ks)[to_blocks + (t0 >> shift) + tok] = mx;
  }
  __syncthreads();
  const size_t to = (static_cast<size_t>(h) * a.cap + t0) * D;
#pragma unroll
  for (int u = 0; u < kN; ++u) {
    const int i = (tid + u * kGatherThreads) % (kGatherTok * kW), row = i / kW;
    if (row >= nt) continue;
    const int half = u < kN / 2 ? 0 : 1;
    const float s = s_scale[half][row], big = s_to[half][row >> shift];
    if (s != big) {
      const float r = s / big;
      w[u] = make_uint4(rescale4(w[u].x, r), rescale4(w[u].y, r), rescale4(w[u].z, r), rescale4(w[u].w, r));
    }
    reinterpret_cast<uint4*>((half ? a.V : a.K) + to)[i] = w[u];
  }
}

}  // namespace

cudaError_t launch_q8_evict(const Q8EvictArgs& a, cudaStream_t st) {
  cudaError_t e;
  {
    LaunchTrace trace("q8_select_kernel", st);
    e = cudaFuncSetAttribute(q8_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(sizeof(SelShared)));
    if (e == cudaSuccess)
      e = launch_pdl(q8_select_kernel, dim3(kSelCtas, a.src.H), dim3(kSelThreads), sizeof(SelShared), st, a);
  }
  if (e != cudaSuccess) return e;
  LaunchTrace trace("q8_gather_kernel", st);
  const int most = a.budget < a.src.cap ? a.budget : a.src.cap;
  const dim3 grid((most + kGatherTok - 1) / kGatherTok, a.src.H);
  return a.src.d == 128 ? launch_pdl(q8_gather_kernel<128>, grid, dim3(kGatherThreads), 0, st, a)
                        : launch_pdl(q8_gather_kernel<64>, grid, dim3(kGatherThreads), 0, st, a);
}

}  // namespace kvb
