// kvb_q8_append: new K and V rows rounded to E4M3 under one power-of-two scale per
// (head, block of tokens).
//
// A CTA (or half of one) takes one block of one head of K or V: it holds the block's
// new elements in registers, finds their largest magnitude, and writes the codes, so
// every element is read once and written once; bound by memory.  The scale is the
// power of two 2^e with max|x| <= 448 * 2^e < 2 max|x|: multiplying by 2^-e is exact,
// so the E4M3 rounding is the only one, and a block whose scale has to grow for later
// tokens can round its older codes anew with nothing lost but what the coarser scale
// cannot hold.
#include "host_util.h"
#include "q8.cuh"

namespace kvb {
namespace {

constexpr int kHalf = 256;   // threads per (block, head, K or V)
constexpr int kMinExp = -100, kMaxExp = 119;

// exponent of the smallest power-of-two scale that holds amax (448 = 1.75 * 2^8)
__device__ __forceinline__ int scale_exp(float amax) {
  const uint32_t u = __float_as_uint(amax);
  if (amax == 0.f) return kMinExp;
  const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(e, kMinExp), kMaxExp);
}

// eight elements as loaded
template <typename T>
struct Words;
template <>
struct Words<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const float2 a = unpack_bf16x2(w.x), b = unpack_bf16x2(w.y), c = unpack_bf16x2(w.z), d = unpack_bf16x2(w.w);
    f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y, f[4] = c.x, f[5] = c.y, f[6] = d.x, f[7] = d.y;
  }
};
template <>
struct Words<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
};

__device__ __forceinline__ uint2 codes8(const float (&f)[8], float inv) {
  return make_uint2(f32x4_to_e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                    f32x4_to_e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
}

// One (block b, head h, kv) by kHalf threads; `bar`: their named barrier, `s_max`: 8
// floats of shared memory.  CH: 8-element chunks per thread (block * d / 8 / kHalf,
// at least 1).
template <typename T, int CH>
__device__ __forceinline__ void append_block(const Q8AppendArgs& a, int kv, int h, int b, int start, int tid, int bar,
                                             float* s_max) {
  const int per = a.d / 8;                       // chunks per row
  const int t0 = max(b * a.block, start);        // first new token of the block
  const int t1 = min((b + 1) * a.block, start + a.n);
  const int nch = (t1 - t0) * per;
  const T* X = static_cast<const T*>(a.X[kv]) + h * a.hs[kv];
  uint8_t* code = a.code[kv] + static_cast<size_t>(h) * a.cap * a.d;
  Words<T> w[CH];
#pragma unroll
  for (int u = 0; u < CH; ++u) {
    const int i = tid + u * kHalf;
    if (i < nch) w[u].load(X + static_cast<long long>(t0 - start + i / per) * a.ts[kv] + (i % per) * 8);
  }
  float mx = 0.f;
#pragma unroll
  for (int u = 0; u < CH; ++u) {
    if (tid + u * kHalf >= nch) continue;
    float f[8];
    w[u].get(f);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float v = fabsf(f[k]);
      if (v <= 3.402823466e38f) mx = fmaxf(mx, v);  // infinities and NaN take no part
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if ((tid & 31) == 0) s_max[tid >> 5] = mx;
  asm volatile("bar.sync %0, %1;" ::"r"(bar), "n"(kHalf) : "memory");
#pragma unroll
  for (int k = 0; k < kHalf / 32; ++k) mx = fmaxf(mx, s_max[k]);
  float scale = pow2f(scale_exp(mx));
  float* sp = a.scale[kv] + static_cast<size_t>(h) * (a.cap / a.block) + b;
  const int old = t0 - b * a.block;              // tokens the block held before
  float was = 0.f;
  if (old > 0) {
    was = *sp;
    scale = fmaxf(scale, was);
  }
  const float inv = 1.f / scale;                 // exact: a power of two
#pragma unroll
  for (int u = 0; u < CH; ++u) {
    const int i = tid + u * kHalf;
    if (i >= nch) continue;
    float f[8];
    w[u].get(f);
    *reinterpret_cast<uint2*>(code + (static_cast<size_t>(t0) * per + i) * 8) = codes8(f, inv);
  }
  if (old > 0 && scale > was) {
    const float shrink = was * inv;
    for (int i = tid; i < old * per; i += kHalf) {
      uint2* p = reinterpret_cast<uint2*>(code + (static_cast<size_t>(b) * a.block * per + i) * 8);
      const uint2 c = *p;
      const float4 x = e4m3x4_to_f32x4(c.x), y = e4m3x4_to_f32x4(c.y);
      const float f[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
      *p = codes8(f, shrink);
    }
  }
  if (kv == 0 && a.mass)
    for (int i = t0 + tid; i < t1; i += kHalf) a.mass[static_cast<size_t>(h) * a.cap + i] = 0.f;
  // every thread has read the old scale before it changes, and s_max is free again
  asm volatile("bar.sync %0, %1;" ::"r"(bar), "n"(kHalf) : "memory");
  if (tid == 0) *sp = scale;
}

__device__ __forceinline__ bool has_room(const Q8AppendArgs& a, int start) {
  return start >= 0 && static_cast<long long>(start) + a.n <= a.cap;
}

__device__ __forceinline__ void move_length(const Q8AppendArgs& a, int h, int start) {
  if (has_room(a, start)) a.len[h] = start + a.n;
  else latch_status(a.status, KVB_E_DEVICE_BOUNDS);
}

// grid (blocks touched at most, heads, 2).  APART: the starts are not len itself,
// so the lengths move here (480P chunk 18.8 -> 16.2 us); else other CTAs may not have
// read theirs yet.
template <typename T, int CH, bool APART>
__global__ void __launch_bounds__(kHalf) q8_append_kernel(const Q8AppendArgs a) {
  __shared__ float s_max[kHalf / 32];
  pdl_wait();
  pdl_trigger();
  const int h = blockIdx.y, kv = blockIdx.z;
  const int start = a.start[h];
  if (APART && blockIdx.x == 0 && kv == 0 && threadIdx.x == 0) move_length(a, h, start);
  if (!has_room(a, start)) return;
  const int b = start / a.block + blockIdx.x;
  if (b * a.block >= start + a.n) return;
  append_block<T, CH>(a, kv, h, b, start, threadIdx.x, 1, s_max);
}

// lengths after q8_append_kernel
__global__ void q8_len_kernel(const Q8AppendArgs a) {
  pdl_wait();
  pdl_trigger();
  const int h = blockIdx.x * blockDim.x + threadIdx.x;
  if (h < a.H) move_length(a, h, a.start[h]);
}

// At most `block` new tokens (one or two blocks): one CTA per head does all of it,
// K in its first half and V in its second, then moves the length itself, which saves
// the second launch where latency is all there is.
template <typename T, int CH>
__global__ void __launch_bounds__(2 * kHalf) q8_append_few_kernel(const Q8AppendArgs a) {
  __shared__ float s_max[2][kHalf / 32];
  pdl_wait();
  pdl_trigger();
  const int h = blockIdx.x;
  const int kv = threadIdx.x / kHalf, tid = threadIdx.x % kHalf;
  const int start = a.start[h];
  if (!has_room(a, start)) {
    if (threadIdx.x == 0) latch_status(a.status, KVB_E_DEVICE_BOUNDS);
    return;
  }
  // (an empty run touches no block, also where it starts inside one)
  for (int b = start / a.block; a.n > 0 && b * a.block < start + a.n; ++b)
    append_block<T, CH>(a, kv, h, b, start, tid, 1 + kv, s_max[kv]);
  __syncthreads();  // every thread has read start, which may be this word
  if (threadIdx.x == 0) a.len[h] = start + a.n;
}

template <typename T, int CH>
cudaError_t launch(const Q8AppendArgs& a, cudaStream_t st) {
  if (a.n <= a.block) {
    LaunchTrace trace("q8_append_few_kernel", st);
    return launch_pdl(q8_append_few_kernel<T, CH>, dim3(a.H), dim3(2 * kHalf), 0, st, a);
  }
  const dim3 grid((a.n + a.block - 1) / a.block + 1, a.H, 2);
  const bool apart = a.start != a.len;
  {
    LaunchTrace trace("q8_append_kernel", st);
    const cudaError_t e = apart ? launch_pdl(q8_append_kernel<T, CH, true>, grid, dim3(kHalf), 0, st, a)
                                : launch_pdl(q8_append_kernel<T, CH, false>, grid, dim3(kHalf), 0, st, a);
    if (apart || e != cudaSuccess) return e;
  }
  LaunchTrace trace("q8_len_kernel", st);
  return launch_pdl(q8_len_kernel, dim3((a.H + 127) / 128), dim3(128), 0, st, a);
}

template <typename T>
cudaError_t launch_t(const Q8AppendArgs& a, cudaStream_t st) {
  const int ch = (a.block * a.d / 8 + kHalf - 1) / kHalf;  // 1, 2, 4 or 8
  if (ch <= 1) return launch<T, 1>(a, st);
  if (ch <= 2) return launch<T, 2>(a, st);
  if (ch <= 4) return launch<T, 4>(a, st);
  return launch<T, 8>(a, st);
}

}  // namespace

cudaError_t launch_q8_append(const Q8AppendArgs& a, kvb_dtype dtype, cudaStream_t st) {
  return dtype == KVB_BF16 ? launch_t<__nv_bfloat16>(a, st) : launch_t<float>(a, st);
}

}  // namespace kvb
