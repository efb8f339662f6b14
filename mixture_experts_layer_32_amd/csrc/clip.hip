// The norm over many tensors together, and their scaling: what a training step does with the weight gradients that
// the backward passes leave.
//
//   k_norm    each workgroup takes a contiguous run of the tensors' chunks and leaves one partial sum of squares.
//             Squares and sums in 64 bits: no range is lost, and the order (fixed by the sizes and addresses) hardly shows.
//             Bound by the reads, which go past the caches: 1.2 GB 183 us (6.6 TB/s; through them 231).
//   k_root    norm = sqrt(sum of the partial sums).
//   k_scale   out = c g, c = min(1, max_norm / (norm + 1e-6)); with the norm given, or from the partial sums, which
//             every workgroup then adds up for itself (one launch less). A copy at heart: 1.2 GB read and written in 405
//             us (6.0 TB/s), by kScaleBlocks workgroups whose chunks lie side by side, past the caches (plain stores 435;
//             256 or 512 workgroups 757 and 489; a contiguous run of chunks for each workgroup 470 to 504; from the last
//             chunk to the first, the norm's latest, no gain at any size and 12 MB 31 us a call where this takes 26).
//             Outputs that are another number of elements off a 16-byte boundary than their tensors go element by element:
//             600 M of bf16 1316 us for 414, 300 M of fp32 to bf16, both one element off, 674 for 338.
// The tensors' addresses and sizes travel in the launch's arguments, kTable (with outputs kPair) tensors a launch: 150 tensors
// of 400000 elements together 6 + 2 us.
#include <algorithm>
#include <type_traits>

#include "moe_device.h"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kChunk = 8192;    // elements
constexpr int kScaleBlocks = 1024;
constexpr int kTable = 184;     // 184 * 20 bytes: within the 4 KiB of a launch's arguments
constexpr int kPair = 128;

struct Table {                  // the norm's tensors, and those scaled in place
  static constexpr int MAX = kTable;
  const void* src[MAX];
  int64_t n[MAX];
  int first[MAX + 1];           // first chunk of each tensor, then their number
  unsigned f32[(MAX + 31) / 32];
  int count;
};
struct PairTable {              // tensors and outputs
  static constexpr int MAX = kPair;
  const void* src[MAX];
  void* dst[MAX];
  int64_t n[MAX];
  int first[MAX + 1];
  unsigned f32[(MAX + 31) / 32], d32[(MAX + 31) / 32];
  int count;
};
static_assert(sizeof(Table) <= 3900 && sizeof(PairTable) <= 3900, "launch arguments");

// the tensor that chunk c lies in
template <class T>
__device__ __forceinline__ int tensor_of(const T& a, int c) {
  int lo = 0, hi = a.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.first[mid] <= c) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}
__device__ __forceinline__ bool bit(const unsigned* w, int i) { return (w[i >> 5] >> (i & 31)) & 1; }

// elements ahead of the first 16-byte boundary
template <class T>
__device__ __forceinline__ int head16(const T* p, int m) {
  return min(m, (int)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / (int)sizeof(T));
}
template <class T>
__device__ __forceinline__ void add_sq(uint4 v, double& s) {
  const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
  for (int i = 0; i < 16 / (int)sizeof(T); ++i) {
    const double d = (double)(float)e[i];
    s = fma(d, d, s);
  }
}

// sum of squares of p[0 .. m), this thread's share
template <class T>
__device__ __forceinline__ void sq_chunk(const T* p, int m, double& s) {
  constexpr int V = 16 / sizeof(T);
  const int tid = threadIdx.x, h = head16(p, m), nv = (m - h) / V;
  if (tid < h) {
    const double d = (double)(float)p[tid];
    s = fma(d, d, s);
  }
  const uint4* v = reinterpret_cast<const uint4*>(p + h);
#pragma unroll 4
  for (int i = tid; i < nv; i += 256) add_sq<T>(ld16_nt(v + i), s);
  const int t = h + nv * V + tid;
  if (t < m) {
    const double d = (double)(float)p[t];
    s = fma(d, d, s);
  }
}

// the workgroup's sum, in every thread, in a fixed order
__device__ __forceinline__ double block_sum(double s, double* lds) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) s += __shfl_xor(s, off);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = s;
  __syncthreads();
  return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

__global__ __launch_bounds__(256) void k_norm(Table a, double* part) {
  __shared__ double lds[4];
  const int C = a.first[a.count];
  const int c0 = (int)((int64_t)C * blockIdx.x / gridDim.x), c1 = (int)((int64_t)C * (blockIdx.x + 1) / gridDim.x);
  double s = 0.0;
  int i = tensor_of(a, c0);
  for (int c = c0; c < c1; ++c) {
    while (c >= a.first[i + 1]) ++i;
    const int64_t at = (int64_t)(c - a.first[i]) * kChunk;
    const int m = (int)min((int64_t)kChunk, a.n[i] - at);
    if (bit(a.f32, i)) sq_chunk(static_cast<const float*>(a.src[i]) + at, m, s);
    else sq_chunk(static_cast<const bf16*>(a.src[i]) + at, m, s);
  }
  s = block_sum(s, lds);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// sqrt of the partial sums' sum in fp32, in every thread
__device__ __forceinline__ float root(const double* part, int64_t parts, double* lds) {
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < parts; i += 256) s += part[i];
  return (float)sqrt(block_sum(s, lds));
}

__global__ __launch_bounds__(256) void k_root(const double* part, int64_t parts, float* norm) {
  __shared__ double lds[4];
  const float r = root(part, parts, lds);
  if (threadIdx.x == 0) *norm = r;
}

template <class S, class D>
__device__ __forceinline__ void scale_chunk(const S* p, D* o, int m, float c) {
  constexpr int V = 16 / (sizeof(S) < sizeof(D) ? sizeof(S) : sizeof(D));   // whole 16-byte pieces of both
  const int tid = threadIdx.x;
  int h = head16(p, m);
  const bool vec = (reinterpret_cast<uintptr_t>(o + h) & 15) == 0;
  const int nv = vec ? (m - h) / V : 0;
  if (!vec) h = 0;
  if (tid < h) o[tid] = (D)(c * (float)p[tid]);
  constexpr int U = 4, LB = V * (int)sizeof(S) / 16, SB = V * (int)sizeof(D) / 16;
  for (int i0 = tid; i0 < nv; i0 += U * 256) {
    uint4 v[U][LB];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + 256 * u < nv)
#pragma unroll
        for (int b = 0; b < LB; ++b) v[u][b] = ld16_nt(reinterpret_cast<const uint4*>(p + h) + (i0 + 256 * u) * LB + b);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + 256 * u < nv) {
        uint4 w[SB];
#pragma unroll
        for (int e = 0; e < V; ++e) reinterpret_cast<D*>(w)[e] = (D)(c * (float)reinterpret_cast<const S*>(v[u])[e]);
#pragma unroll
        for (int b = 0; b < SB; ++b) st16_nt(reinterpret_cast<uint4*>(o + h) + (i0 + 256 * u) * SB + b, w[b]);
      }
  }
  for (int t = h + nv * V + tid; t < m; t += 256) o[t] = (D)(c * (float)p[t]);
}

template <class T>
__global__ __launch_bounds__(256) void k_scale(T a, float max_norm, const float* norm_in, const double* part, int64_t parts,
                                               float* norm_out) {
  constexpr bool PAIRS = std::is_same_v<T, PairTable>;
  __shared__ double lds[4];
  float norm;
  if (norm_in) {
    norm = *norm_in;
  } else {
    norm = root(part, parts, lds);
    if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = norm;
  }
  float c = max_norm / (norm + 1e-6f);
  c = c > 1.f ? 1.f : c;                       // NaN stays
  if (!PAIRS && c == 1.f) return;              // in place: nothing changes
  const int C = a.first[a.count];
  int i = tensor_of(a, (int)blockIdx.x);
  for (int b = (int)blockIdx.x; b < C; b += gridDim.x) {
    while (b >= a.first[i + 1]) ++i;
    const void* dst = a.src[i];
    bool f32 = bit(a.f32, i), d32 = f32;
    if constexpr (PAIRS) {
      dst = a.dst[i];
      d32 = bit(a.d32, i);
      if (c == 1.f && dst == a.src[i]) continue;
    }
    const int64_t at = (int64_t)(b - a.first[i]) * kChunk;
    const int m = (int)min((int64_t)kChunk, a.n[i] - at);
    const float* pf = static_cast<const float*>(a.src[i]) + at;
    const bf16* pb = static_cast<const bf16*>(a.src[i]) + at;
    float* of = static_cast<float*>(const_cast<void*>(dst)) + at;
    bf16* ob = static_cast<bf16*>(const_cast<void*>(dst)) + at;
    if (f32) {
      if (d32) scale_chunk(pf, of, m, c);
      else if constexpr (PAIRS) scale_chunk(pf, ob, m, c);
    } else {
      if (!d32) scale_chunk(pb, ob, m, c);
      else if constexpr (PAIRS) scale_chunk(pb, of, m, c);
    }
  }
}

int chunks(int64_t n) { return (int)((n + kChunk - 1) / kChunk); }
int parts_of(int C) { return std::min(C, kNormParts); }

// The next tensors from `from` on, at most MAX and as many as hold fewer than 2^31 chunks together; empty ones are
// passed over. Returns where to go on.
template <class T>
int fill(T& a, const moe_tensor* t, const moe_tensor* out, int count, int from) {
  a.count = 0;
  a.first[0] = 0;
  int i = from;
  for (; i < count && a.count < T::MAX; ++i) {
    if (t[i].n == 0) continue;
    const int k = a.count++;
    if (k % 32 == 0) a.f32[k / 32] = 0;
    a.src[k] = t[i].data;
    a.n[k] = t[i].n;
    a.first[k + 1] = a.first[k] + chunks(t[i].n);
    if (t[i].type == MOE_TYPE_FP32) a.f32[k / 32] |= 1u << (k % 32);
    if constexpr (std::is_same_v<T, PairTable>) {
      if (k % 32 == 0) a.d32[k / 32] = 0;
      a.dst[k] = out[i].data;
      if (out[i].type == MOE_TYPE_FP32) a.d32[k / 32] |= 1u << (k % 32);
    }
  }
  return i;
}

template <class T>
hipError_t scale_all(const moe_tensor* t, const moe_tensor* out, int count, float max_norm, const float* norm_in,
                     const double* part, int64_t parts, float* norm_out, hipStream_t s) {
  hipError_t err;
  T a;
  for (int i = 0; i < count;) {
    i = fill(a, t, out, count, i);
    const int grid = parts_of(a.first[a.count]);
    if (grid == 0) continue;
    prof_mark_begin("grad_clip", s);
    k_scale<T><<<std::min(grid, kScaleBlocks), 256, 0, s>>>(a, max_norm, norm_in, part, parts, norm_out);
    if ((err = hipGetLastError()) != hipSuccess) return err;
    prof_mark_end(s);
    norm_out = nullptr;
  }
  return hipSuccess;
}

}  // namespace

int64_t norm_parts(const moe_tensor* t, int count) {   // as launch_grad_norm cuts them
  int64_t parts = 0;
  for (int i = 0; i < count;) {
    int chunk = 0;
    for (int k = 0; i < count && k < Table::MAX; ++i) {
      chunk += chunks(t[i].n);
      k += t[i].n > 0;
    }
    parts += parts_of(chunk);
  }
  return parts;
}

hipError_t launch_grad_norm(const moe_tensor* t, int count, double* part, float* norm, hipStream_t s) {
  hipError_t err;
  int64_t parts = 0;
  Table a;
  for (int i = 0; i < count;) {
    i = fill(a, t, nullptr, count, i);
    const int grid = parts_of(a.first[a.count]);
    if (grid == 0) continue;
    prof_mark_begin("grad_norm", s);
    k_norm<<<grid, 256, 0, s>>>(a, part + parts);
    if ((err = hipGetLastError()) != hipSuccess) return err;
    prof_mark_end(s);
    parts += grid;
  }
  if (!norm) return hipSuccess;
  prof_mark_begin("grad_root", s);
  k_root<<<1, 256, 0, s>>>(part, parts, norm);
  if ((err = hipGetLastError()) == hipSuccess) prof_mark_end(s);
  return err;
}

hipError_t launch_grad_clip(const moe_tensor* t, const moe_tensor* out, int count, float max_norm, const float* norm_in,
                            const double* part, int64_t parts, float* norm_out, hipStream_t s) {
  return out ? scale_all<PairTable>(t, out, count, max_norm, norm_in, part, parts, norm_out, s)
             : scale_all<Table>(t, nullptr, count, max_norm, norm_in, part, parts, norm_out, s);
}

}  // namespace moe
