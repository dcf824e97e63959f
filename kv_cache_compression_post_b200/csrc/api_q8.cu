// C entry points of the 8-bit block-scaled cache: argument checks, workspace layout
// and the choice of kernel.
#include <atomic>
#include <cmath>

#include "host_util.h"
#include "q8.cuh"

using namespace kvb;

namespace {

bool sizes_ok(const kvb_q8_cache* c) {
  if (!c || c->heads < 1 || c->heads > kQ8MaxHeads || c->capacity < 1 || c->capacity > kQ8MaxCapacity) return false;
  if (c->block != 16 && c->block != 32 && c->block != 64 && c->block != 128) return false;
  return c->capacity % c->block == 0;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

kvb_status check_cache(const kvb_q8_cache* c) {
  if (!sizes_ok(c)) return KVB_E_INVAL;
  if (c->head_dim != 64 && c->head_dim != 128) return KVB_E_UNSUPPORTED;
  if (!c->K || !c->V || !c->k_scale || !c->v_scale || !c->len) return KVB_E_INVAL;
  if (!aligned(c->K, 16) || !aligned(c->V, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) ||
      !aligned(c->len, 4) || !aligned(c->mass, 4) || !aligned(c->status, 4))
    return KVB_E_INVAL;
  return KVB_OK;
}

Q8View view(const kvb_q8_cache* c) {
  return Q8View{c->heads, c->head_dim, c->capacity, c->block, __builtin_ctz(c->block), c->K, c->V, c->k_scale, c->v_scale, c->len, c->status};
}

// rows per head of a call: sums of a row count and a tile stay below 2^31
bool rows_ok(int32_t n) { return n >= 1 && n <= kQ8MaxRows; }

bool dtype_ok(kvb_dtype t) { return t == KVB_BF16 || t == KVB_F32; }

// One scratch serves every call on a cache: the row-tile kernels' piece flags, which
// nothing else writes, then their partials, the positions an eviction keeps, or what a
// chunk of queries needs, each from there.
struct Scratch {
  unsigned long long* flag = nullptr;
  float* part = nullptr;
  int* kept = nullptr;
  Q8ChunkScratch chunk{};
  size_t bytes = 0;
};

bool chunk_kernel(const kvb_q8_cache* c, int32_t rows, kvb_dtype dtype) {
  return dtype == KVB_BF16 && rows >= q8_chunk_rows(c->heads, c->capacity);
}

Scratch scratch(const kvb_q8_cache* c, int32_t max_queries, kvb_dtype dtype, void* ws) {
  Scratch s;
  Carver a(ws);
  s.flag = a.take<unsigned long long>(kQ8RowFlags);
  Carver e = a, q = a;
  s.part = a.take<float>(q8_part_floats(c->head_dim));
  s.kept = e.take<int>(static_cast<size_t>(c->heads) * c->capacity);
  s.bytes = a.bytes() > e.bytes() ? a.bytes() : e.bytes();
  if (chunk_kernel(c, max_queries, dtype)) {
    const size_t rows = static_cast<size_t>(c->heads) * max_queries;
    s.chunk.hi = q.take<uint8_t>(rows * c->head_dim);
    s.chunk.lo = q.take<uint8_t>(rows * c->head_dim);
    s.chunk.coef = q.take<float>(rows);
    s.chunk.part = q.take<float>(q8_chunk_part_floats(c->head_dim));
    const size_t cut = static_cast<size_t>(c->heads) * ((max_queries + 255) / 256) * 2;
    s.chunk.cnt = q.take<unsigned int>(cut > kQ8MassCounters ? cut : kQ8MassCounters);
    if (q.bytes() > s.bytes) s.bytes = q.bytes();
  }
  return s;
}

// A tag that no other call of this process has, and that memory which was never written
// by one holds with probability 2^-64: the calls' count through SplitMix64, whose steps are
// bijective (Steele, Lea, Flood: Fast splittable pseudorandom number generators, 2014).
unsigned long long next_tag() {
  static std::atomic<unsigned long long> calls{0};
  unsigned long long z = 0;
  while (z == 0) {
    z = (calls.fetch_add(1, std::memory_order_relaxed) + 1) * 0x9E3779B97F4A7C15ull;
    z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
    z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
    z ^= z >> 31;
  }
  return z;
}

bool workspace_ok(const void* ws, size_t have, size_t want) { return ws && aligned(ws, 256) && have >= want; }

}  // namespace

extern "C" {

size_t kvb_q8_workspace_size(const kvb_q8_cache* c, int32_t max_queries, kvb_dtype dtype) {
  if (!sizes_ok(c) || (c->head_dim != 64 && c->head_dim != 128) || !rows_ok(max_queries) || !dtype_ok(dtype)) return 0;
  return scratch(c, max_queries, dtype, nullptr).bytes;
}

kvb_status kvb_q8_append(const kvb_q8_cache* c, const void* K, int64_t k_head_stride, int64_t k_token_stride,
                         const void* V, int64_t v_head_stride, int64_t v_token_stride, int32_t n, kvb_dtype dtype,
                         const int32_t* start, void* stream) {
  const kvb_status ok = check_cache(c);
  if (ok != KVB_OK) return ok;
  if (n < 0 || !dtype_ok(dtype) || !aligned(start, 4)) return KVB_E_INVAL;
  if (n > c->capacity) return KVB_E_INVAL;
  if (start && start != c->len) {
    // a length moved for one head must not be another's start
    const uintptr_t s = reinterpret_cast<uintptr_t>(start), l = reinterpret_cast<uintptr_t>(c->len), b = 4u * c->heads;
    if (s < l + b && l < s + b) return KVB_E_INVAL;
  }
  if (n == 0 && !start) return KVB_OK;
  if (n > 0 && (!K || !V)) return KVB_E_INVAL;
  const int64_t unit = dtype == KVB_BF16 ? 8 : 4;
  if (!aligned(K, 16) || !aligned(V, 16) || k_head_stride % unit || k_token_stride % unit || v_head_stride % unit ||
      v_token_stride % unit)
    return KVB_E_INVAL;
  Q8AppendArgs a;
  a.H = c->heads;
  a.d = c->head_dim;
  a.cap = c->capacity;
  a.block = c->block;
  a.X[0] = K;
  a.X[1] = V;
  a.hs[0] = k_head_stride;
  a.hs[1] = v_head_stride;
  a.ts[0] = k_token_stride;
  a.ts[1] = v_token_stride;
  a.code[0] = c->K;
  a.code[1] = c->V;
  a.scale[0] = c->k_scale;
  a.scale[1] = c->v_scale;
  a.n = n;
  a.start = start ? start : c->len;
  a.len = c->len;
  a.mass = c->mass;
  a.status = c->status;
  return cuda_status(launch_q8_append(a, dtype, static_cast<cudaStream_t>(stream)));
}

kvb_status kvb_q8_attend(const kvb_q8_cache* c, const void* Q, int32_t Nq, kvb_dtype dtype, float scale, void* O,
                         float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  const kvb_status ok = check_cache(c);
  if (ok != KVB_OK) return ok;
  if (!rows_ok(Nq) || !dtype_ok(dtype) || !(scale >= 0.f) || !std::isfinite(scale)) return KVB_E_INVAL;
  if (!Q || !O || !aligned(Q, 16) || !aligned(O, 16) || !aligned(lse, 4)) return KVB_E_INVAL;
  const Scratch s = scratch(c, Nq, dtype, workspace);
  if (!workspace_ok(workspace, workspace_bytes, s.bytes)) return KVB_E_WORKSPACE;
  DeviceInfo dev;
  if (!current_device(&dev)) return KVB_E_CUDA;
  Q8AttendArgs a;
  a.c = view(c);
  a.Nq = Nq;
  a.scale = scale > 0.f ? scale : 1.f / std::sqrt(static_cast<float>(c->head_dim));
  a.Q = Q;
  a.O = O;
  a.lse = lse;
  a.part = s.part;
  a.flag = s.flag;
  a.tag = next_tag();
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == KVB_F32) return cuda_status(launch_q8_attend_f32(a, dev.n_sm, st));
  if (chunk_kernel(c, Nq, dtype)) return cuda_status(launch_q8_attend_chunk(a, s.chunk, dev.n_sm, st));
  return cuda_status(launch_q8_attend_rows(a, dev.n_sm, st));
}

kvb_status kvb_q8_mass(const kvb_q8_cache* c, const void* Q, int32_t Nq, kvb_dtype dtype, float scale, const float* lse,
                       float decay, const float* prev, void* workspace, size_t workspace_bytes, void* stream) {
  const kvb_status ok = check_cache(c);
  if (ok != KVB_OK) return ok;
  if (!rows_ok(Nq) || !dtype_ok(dtype) || !(scale >= 0.f) || !std::isfinite(scale) || !std::isfinite(decay))
    return KVB_E_INVAL;
  if (!Q || !lse || !c->mass || !aligned(Q, 16) || !aligned(lse, 4) || !aligned(prev, 4)) return KVB_E_INVAL;
  const Scratch s = scratch(c, Nq, dtype, workspace);
  if (!workspace_ok(workspace, workspace_bytes, s.bytes)) return KVB_E_WORKSPACE;
  DeviceInfo dev;
  if (!current_device(&dev)) return KVB_E_CUDA;
  Q8MassArgs a;
  a.c = view(c);
  a.Nq = Nq;
  a.scale = scale > 0.f ? scale : 1.f / std::sqrt(static_cast<float>(c->head_dim));
  a.Q = Q;
  a.lse = lse;
  a.decay = decay;
  a.prev = prev;
  a.mass = c->mass;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == KVB_F32) return cuda_status(launch_q8_mass_f32(a, dev.n_sm, st));
  if (chunk_kernel(c, Nq, dtype)) return cuda_status(launch_q8_mass_chunk(a, s.chunk, dev.n_sm, st));
  return cuda_status(launch_q8_mass_rows(a, dev.n_sm, st));
}

kvb_status kvb_q8_evict(const kvb_q8_cache* src, const kvb_q8_cache* dst, int32_t budget, int32_t sink, int32_t recent,
                        int32_t* kept, void* workspace, size_t workspace_bytes, void* stream) {
  kvb_status ok = check_cache(src);
  if (ok == KVB_OK) ok = check_cache(dst);
  if (ok != KVB_OK) return ok;
  if (!src->mass || dst->heads != src->heads || dst->head_dim != src->head_dim || dst->block != src->block)
    return KVB_E_INVAL;
  if (budget < 1 || budget > dst->capacity || sink < 0 || recent < 0 || static_cast<int64_t>(sink) + recent > budget)
    return KVB_E_INVAL;
  if (dst->K == src->K || dst->V == src->V || dst->k_scale == src->k_scale || dst->v_scale == src->v_scale ||
      dst->len == src->len || dst->mass == src->mass || !aligned(kept, 4))
    return KVB_E_INVAL;
  const Scratch s = scratch(src, 1, KVB_BF16, workspace);
  if (!workspace_ok(workspace, workspace_bytes, s.bytes)) return KVB_E_WORKSPACE;
  Q8EvictArgs a;
  a.src = view(src);
  a.mass = src->mass;
  a.K = dst->K;
  a.V = dst->V;
  a.ks = dst->k_scale;
  a.vs = dst->v_scale;
  a.len = dst->len;
  a.to_mass = dst->mass;
  a.cap = dst->capacity;
  // the scratch list has a place per token of the source: a larger budget keeps them all
  // and needs no more
  a.budget = kept || budget < src->capacity ? budget : src->capacity;
  a.sink = sink;
  a.recent = recent;
  a.kept = kept ? kept : s.kept;
  return cuda_status(launch_q8_evict(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
