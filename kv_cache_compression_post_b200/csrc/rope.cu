// kvb_rope: rotary positions over three axes, forwards or backwards, with the
// change between token-major and head-major rows folded in.
//
// Pair j of axis a turns by pos[a] * base^(-j / n_a).  The angle depends on the token
// only, so a CTA forms the (cos, sin) of its kTok tokens once, in shared memory, and
// applies them to the rows of every head of its share.  Far positions lose their angle
// in fp32 (position 1e6 has steps of 0.06 rad), so angles are formed and reduced to
// [-pi, pi] in fp64; the remainder is split into two floats, sine and cosine taken of
// the first (in half turns) and corrected by the second: cos(h + l) = cos h - l sin h,
// error ~1 ulp.
// Bound by memory: one read and one write of every element.  A thread moves four
// pairs (16 bytes of bf16, interleaved), four such groups in flight.
#include <cuda_bf16.h>

#include <cmath>

#include "host_util.h"
#include "kvb_device.cuh"

namespace kvb {
namespace {

constexpr int kThreads = 128;
constexpr int kTok = 4;         // tokens per CTA
constexpr int kMaxPairs = 128;  // head_dim <= 256

struct RopeArgs {
  const void* X;
  void* out;
  const int* pos;
  int heads, n, d;
  int heads_per_cta;
  int np[3];
  double log2_base;
  int inverse;
  long long xh, xt, oh, ot;  // strides, elements
};

struct Group {
  float a[4], b[4];  // first and second element of four pairs
};

__device__ __forceinline__ float2 unpack2(uint32_t w) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// the raw words of one group: interleaved rows hold it in 8 consecutive elements,
// half-split rows in 4 consecutive elements of either half
template <typename T, bool HALVES>
struct Raw;
template <bool HALVES>
struct Raw<__nv_bfloat16, HALVES> {
  uint2 lo, hi;
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int half) {
    if constexpr (HALVES) {
      lo = *reinterpret_cast<const uint2*>(p);
      hi = *reinterpret_cast<const uint2*>(p + half);
    } else {
      const uint4 w = *reinterpret_cast<const uint4*>(p);
      lo = make_uint2(w.x, w.y);
      hi = make_uint2(w.z, w.w);
    }
  }
  __device__ __forceinline__ Group get() const {
    Group g;
    const float2 x = unpack2(lo.x), y = unpack2(lo.y), z = unpack2(hi.x), w = unpack2(hi.y);
    if constexpr (HALVES) {
      g = Group{{x.x, x.y, y.x, y.y}, {z.x, z.y, w.x, w.y}};
    } else {
      g = Group{{x.x, y.x, z.x, w.x}, {x.y, y.y, z.y, w.y}};
    }
    return g;
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, int half, const Group& g) {
    if constexpr (HALVES) {
      *reinterpret_cast<uint2*>(p) = make_uint2(pack2(g.a[0], g.a[1]), pack2(g.a[2], g.a[3]));
      *reinterpret_cast<uint2*>(p + half) = make_uint2(pack2(g.b[0], g.b[1]), pack2(g.b[2], g.b[3]));
    } else {
      *reinterpret_cast<uint4*>(p) = make_uint4(pack2(g.a[0], g.b[0]), pack2(g.a[1], g.b[1]), pack2(g.a[2], g.b[2]),
                                                pack2(g.a[3], g.b[3]));
    }
  }
};
template <bool HALVES>
struct Raw<float, HALVES> {
  float4 lo, hi;
  __device__ __forceinline__ void load(const float* p, int half) {
    lo = *reinterpret_cast<const float4*>(p);
    hi = *reinterpret_cast<const float4*>(p + (HALVES ? half : 4));
  }
  __device__ __forceinline__ Group get() const {
    if constexpr (HALVES) return Group{{lo.x, lo.y, lo.z, lo.w}, {hi.x, hi.y, hi.z, hi.w}};
    else return Group{{lo.x, lo.z, hi.x, hi.z}, {lo.y, lo.w, hi.y, hi.w}};
  }
  static __device__ __forceinline__ void store(float* p, int half, const Group& g) {
    if constexpr (HALVES) {
      *reinterpret_cast<float4*>(p) = make_float4(g.a[0], g.a[1], g.a[2], g.a[3]);
      *reinterpret_cast<float4*>(p + half) = make_float4(g.b[0], g.b[1], g.b[2], g.b[3]);
    } else {
      *reinterpret_cast<float4*>(p) = make_float4(g.a[0], g.b[0], g.a[1], g.b[1]);
      *reinterpret_cast<float4*>(p + 4) = make_float4(g.a[2], g.b[2], g.a[3], g.b[3]);
    }
  }
};

template <typename T, bool HALVES>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs a) {
  constexpr int kFlight = sizeof(T) == 2 ? 4 : 2;  // groups of four pairs in flight per thread: 64 bytes
  __shared__ double freq[kMaxPairs];
  __shared__ float2 cs[kTok][kMaxPairs];
  const int half = a.d / 2;
  const int tid = threadIdx.x;
  const int turned = a.np[0] + a.np[1] + a.np[2];
  if (tid < turned) {
    const int axis = tid < a.np[0] ? 0 : (tid < a.np[0] + a.np[1] ? 1 : 2);
    const int j = tid - (axis > 0 ? a.np[0] : 0) - (axis > 1 ? a.np[1] : 0);
    freq[tid] = exp2(-a.log2_base * j / a.np[axis]);
  }
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  const int t0 = blockIdx.x * kTok;
  const int nt = min(kTok, a.n - t0);
  const T* X = static_cast<const T*>(a.X);
  T* out = static_cast<T*>(a.out);
  const int h0 = blockIdx.y * a.heads_per_cta;
  const int nh = min(a.heads_per_cta, a.heads - h0);
  const int per = a.d / 8;  // groups per row
  const int total = nh * nt * per;
  Raw<T, HALVES> w[kFlight];
  int pair[kFlight], tok[kFlight];
  long long to[kFlight];
  auto load = [&](int base) {
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const int i = base + u * kThreads;
      pair[u] = -1;
      if (i >= total) continue;
      const int row = i / per, g = i - row * per;
      const int h = row / nt;
      tok[u] = row - h * nt;
      pair[u] = g * 4;
      const int e = HALVES ? g * 4 : g * 8;
      w[u].load(X + (h0 + h) * a.xh + (t0 + tok[u]) * a.xt + e, half);
      to[u] = (h0 + h) * a.oh + (t0 + tok[u]) * a.ot + e;
    }
  };
  load(tid);  // in flight over the angles
  for (int i = tid; i < nt * half; i += kThreads) {
    const int t = i / half, k = i % half;
    float2 v = make_float2(1.f, 0.f);
    if (k < turned) {
      const int axis = k < a.np[0] ? 0 : (k < a.np[0] + a.np[1] ? 1 : 2);
      const double x = static_cast<double>(a.pos[static_cast<size_t>(t0 + t) * 3 + axis]) * freq[k];
      // x - n 2 pi, 2 pi as two doubles
      const double n = rint(x * 0.15915494309189535);
      const double r = fma(-n, 2.4492935982947064e-16, fma(-n, 6.283185307179586, x));
      const double turn = r * 0.3183098861837907;  // in half turns, |turn| <= 1
      const float h = static_cast<float>(turn);
      const float l = static_cast<float>((turn - static_cast<double>(h)) * 3.141592653589793);
      float s, c;
      sincospif(h, &s, &c);
      v = make_float2(fmaf(-l, s, c), fmaf(l, c, s));
      if (a.inverse) v.y = -v.y;
    }
    cs[t][k] = v;
  }
  __syncthreads();
  for (int base = tid; base < total; base += kThreads * kFlight) {
    if (base != tid) load(base);
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      if (pair[u] < 0) continue;
      Group g = w[u].get();
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (pair[u] + k < turned) {  // a pair past the axes is copied, infinities included
          const float2 v = cs[tok[u]][pair[u] + k];
          const float x = g.a[k], y = g.b[k];
          g.a[k] = x * v.x - y * v.y;
          g.b[k] = x * v.y + y * v.x;
        }
      }
      Raw<T, HALVES>::store(out + to[u], half, g);
    }
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace
}  // namespace kvb

using namespace kvb;

extern "C" kvb_status kvb_rope(const void* X, const int32_t* pos, int32_t heads, int32_t n_tokens, int32_t head_dim,
                               kvb_dtype dtype, const int32_t* axis_pairs, float base, kvb_rope_pairing pairing,
                               int32_t inverse, int64_t x_head_stride, int64_t x_token_stride, void* out,
                               int64_t out_head_stride, int64_t out_token_stride, void* stream) {
  if (heads < 1 || heads > 65535 || n_tokens < 0 || head_dim < 8 || head_dim > 256 || head_dim % 8 != 0)
    return KVB_E_INVAL;
  if (dtype != KVB_BF16 && dtype != KVB_F32) return KVB_E_INVAL;
  if (pairing != KVB_ROPE_INTERLEAVED && pairing != KVB_ROPE_HALVES) return KVB_E_INVAL;
  // from 2^-21 on angles stay below 2^52, where their reduction knows its whole turns; past
  // that the remainder is no angle, and "sines" reached 10^11
  if (!axis_pairs || !(base >= 0x1p-21f) || !std::isfinite(base)) return KVB_E_INVAL;
  long long pairs = 0;
  for (int i = 0; i < 3; ++i) {
    if (axis_pairs[i] < 0) return KVB_E_INVAL;
    pairs += axis_pairs[i];
  }
  if (pairs > head_dim / 2) return KVB_E_INVAL;
  if (n_tokens == 0) return KVB_OK;
  if (!X || !pos || !out || !aligned16(X) || !aligned16(out) || (reinterpret_cast<uintptr_t>(pos) & 3))
    return KVB_E_INVAL;
  const int64_t unit = dtype == KVB_BF16 ? 8 : 4;  // elements of 16 bytes
  if (x_head_stride % unit || x_token_stride % unit || out_head_stride % unit || out_token_stride % unit)
    return KVB_E_INVAL;
  if ((heads > 1 && out_head_stride == 0) || (n_tokens > 1 && out_token_stride == 0)) return KVB_E_INVAL;
  if (X == out && (x_head_stride != out_head_stride || x_token_stride != out_token_stride)) return KVB_E_INVAL;
  DeviceInfo dev;
  if (!current_device(&dev)) return KVB_E_CUDA;
  RopeArgs a;
  a.X = X;
  a.out = out;
  a.pos = pos;
  a.heads = heads;
  a.n = n_tokens;
  a.d = head_dim;
  for (int i = 0; i < 3; ++i) a.np[i] = axis_pairs[i];
  a.log2_base = std::log2(static_cast<double>(base));
  a.inverse = inverse != 0;
  a.xh = x_head_stride;
  a.xt = x_token_stride;
  a.oh = out_head_stride;
  a.ot = out_token_stride;
  const int tiles = (n_tokens - 1) / kTok + 1;
  // all heads of a token share its angles; few tokens spread their heads over CTAs
  const int want = (4 * dev.n_sm - 1) / tiles + 1;
  const int split = want < heads ? (want < 1 ? 1 : want) : heads;
  a.heads_per_cta = (heads + split - 1) / split;
  const dim3 grid(tiles, (heads + a.heads_per_cta - 1) / a.heads_per_cta);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  LaunchTrace trace("rope_kernel", st);
  const bool hv = pairing == KVB_ROPE_HALVES;
  cudaError_t e;
  if (dtype == KVB_BF16)
    e = hv ? launch_pdl(rope_kernel<__nv_bfloat16, true>, grid, dim3(kThreads), 0, st, a)
           : launch_pdl(rope_kernel<__nv_bfloat16, false>, grid, dim3(kThreads), 0, st, a);
  else
    e = hv ? launch_pdl(rope_kernel<float, true>, grid, dim3(kThreads), 0, st, a)
           : launch_pdl(rope_kernel<float, false>, grid, dim3(kThreads), 0, st, a);
  return cuda_status(e);
}
