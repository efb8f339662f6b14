// The layer taken apart: (token, slot) pairs sorted by expert, tokens' rows brought into that order and back with
// the routing weights, and the gradients of both ("A Magia da Fusão" on "IA: MoE Kernel 3x Mais Rápido Chegou!"
// lists dispatch and combine among the layer's steps).
//
//   k_sort_small    up to kSortSmall pairs: one workgroup counts, scans and places them.
//   k_sort_count, k_sort_scan, k_sort_place   beyond: counts per block of kSortPairs pairs and expert, their
//                   exclusive sums over the blocks, positions.
//   k_dispatch      rows[pair_pos[t, j]] = x[t]: x is read once, each row written once.
//   k_pairs_combine y[t] = sum_j w_tj rows[pair_pos[t, j]]: each row read once.
//   k_pairs_combine_bwd  drows = w dy, dw = <dy, rows>, dlogits: each row read and written once.
#include <algorithm>

#include "moe_device.h"
#include "moe_internal.h"

namespace moe {
namespace {

// ------------------------------------------------------------------------------------------------ sort

// Lanes of the wave that hold the same e as this one (e < 1024), from ten ballots.
__device__ __forceinline__ unsigned long long same_lanes(int e, bool valid) {
  unsigned long long m = __ballot(valid);
#pragma unroll
  for (int b = 0; b < 10; ++b) {
    const unsigned long long s = __ballot((e >> b) & 1);
    m &= ((e >> b) & 1) ? s : ~s;
  }
  return m;
}
__device__ __forceinline__ int rank_below(unsigned long long m) {
  return __builtin_amdgcn_mbcnt_hi((unsigned)(m >> 32), __builtin_amdgcn_mbcnt_lo((unsigned)m, 0u));
}
__device__ __forceinline__ int local_expert(const SortParams& p, int64_t q) {
  const int64_t e = (int64_t)p.idx[q] - p.e0;
  return e >= 0 && e < p.El ? (int)e : p.El;   // El: no position
}

// Exclusive scan over bins[0 .. n) (n <= 1024, in LDS) by NT threads; every thread of the workgroup calls it.
template <int NT>
__device__ __forceinline__ void scan_bins(int* bins, int n, int* lds) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int carry = 0;
  for (int b0 = 0; b0 < n; b0 += NT) {
    const int b = b0 + tid, c = b < n ? bins[b] : 0;
    int v = c;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int u = __shfl_up(v, off);
      if (lane >= off) v += u;
    }
    if (lane == 63) lds[wave] = v;
    __syncthreads();
    int add = carry, tot = 0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) {
      add += w < wave ? lds[w] : 0;
      tot += lds[w];
    }
    if (b < n) bins[b] = add + v - c;
    carry += tot;
    __syncthreads();
  }
}

// Places the pairs [q0, q1) of this wave in order: base[e] is the position of the wave's next pair of expert e (LDS,
// this wave's own), and P the number of pairs with a position.
__device__ __forceinline__ void place(const SortParams& p, int64_t q0, int64_t q1, volatile int* base, int P) {
  const int lane = threadIdx.x & 63;
  for (int64_t qb = q0; qb < q1; qb += 64) {
    const int64_t q = qb + lane;
    const bool in = q < q1;
    const int e = in ? local_expert(p, q) : 0;
    const unsigned long long m = same_lanes(e, in);
    const int r = rank_below(m);
    int pos = 0;
    if (in) pos = base[e] + r;
    __builtin_amdgcn_wave_barrier();
    if (in && r == 0) base[e] = pos + __popcll(m);
    __builtin_amdgcn_wave_barrier();
    if (in) {
      p.perm[pos] = pos < P ? (int)q : -1;
      p.pair_pos[q] = pos < P ? pos : -1;
    }
  }
}

constexpr int kSW = 16;   // waves of k_sort_small
__global__ __launch_bounds__(kSW * 64) void k_sort_small(SortParams p) {
  __shared__ int cnt[kSW][kMaxExperts + 1];
  __shared__ int tot[kMaxExperts + 1];
  __shared__ int lds[kSW];
  const int tid = threadIdx.x, w = tid >> 6, nb = p.El + 1, n = (int)p.pairs;
  const int per = (n + kSW * 64 - 1) / (kSW * 64) * 64;   // pairs of a wave
  for (int i = tid; i < kSW * nb; i += kSW * 64) cnt[i / nb][i % nb] = 0;
  __syncthreads();
  for (int q = tid; q < n; q += kSW * 64) atomicAdd(&cnt[q / per][local_expert(p, q)], 1);
  __syncthreads();
  if (tid < nb) {
    int s = 0;
    for (int v = 0; v < kSW; ++v) {
      const int c = cnt[v][tid];
      cnt[v][tid] = s;
      s += c;
    }
    tot[tid] = s;
  }
  __syncthreads();
  scan_bins<kSW * 64>(tot, nb, lds);
  for (int i = tid; i < kSW * nb; i += kSW * 64) cnt[i / nb][i % nb] += tot[i % nb];
  if (tid < nb) p.offsets[tid] = tot[tid];
  __syncthreads();
  place(p, min(n, w * per), min(n, (w + 1) * per), cnt[w], tot[p.El]);
}

constexpr int kCW = 4;    // waves of a block of kSortPairs pairs
__global__ __launch_bounds__(kCW * 64) void k_sort_count(SortParams p) {
  __shared__ int cnt[kMaxExperts + 1];
  const int tid = threadIdx.x, nb = p.El + 1;
  for (int i = tid; i < nb; i += kCW * 64) cnt[i] = 0;
  __syncthreads();
  const int64_t q0 = (int64_t)blockIdx.x * kSortPairs, q1 = min(p.pairs, q0 + kSortPairs);
  for (int64_t q = q0 + tid; q < q1; q += kCW * 64) atomicAdd(&cnt[local_expert(p, q)], 1);
  __syncthreads();
  for (int i = tid; i < nb; i += kCW * 64) p.cnt[(size_t)blockIdx.x * nb + i] = cnt[i];
}

__global__ __launch_bounds__(256) void k_sort_scan(SortParams p) {
  __shared__ int lds[4];
  const int e = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, nb = p.El + 1;
  int carry = 0;
  for (int b0 = 0; b0 < p.nblk; b0 += 256) {
    const int b = b0 + tid, c = b < p.nblk ? p.cnt[(size_t)b * nb + e] : 0;
    int v = c;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int u = __shfl_up(v, off);
      if (lane >= off) v += u;
    }
    if (lane == 63) lds[wave] = v;
    __syncthreads();
    int add = carry, tot = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      add += w < wave ? lds[w] : 0;
      tot += lds[w];
    }
    if (b < p.nblk) p.prefix[(size_t)b * nb + e] = add + v - c;
    carry += tot;
    __syncthreads();
  }
  if (tid == 0) p.total[e] = carry;
}

__global__ __launch_bounds__(kCW * 64) void k_sort_place(SortParams p) {
  __shared__ int cnt[kCW][kMaxExperts + 1];
  __shared__ int tot[kMaxExperts + 1];
  __shared__ int lds[kCW];
  const int tid = threadIdx.x, w = tid >> 6, nb = p.El + 1;
  const int64_t q0 = (int64_t)blockIdx.x * kSortPairs, q1 = min(p.pairs, q0 + kSortPairs);
  constexpr int per = kSortPairs / kCW;
  for (int i = tid; i < kCW * nb; i += kCW * 64) cnt[i / nb][i % nb] = 0;
  for (int i = tid; i < nb; i += kCW * 64) tot[i] = p.total[i];
  __syncthreads();
  for (int64_t q = q0 + tid; q < q1; q += kCW * 64) atomicAdd(&cnt[(q - q0) / per][local_expert(p, q)], 1);
  scan_bins<kCW * 64>(tot, nb, lds);   // (its first barrier stands behind the counts too)
  __syncthreads();
  for (int i = tid; i < nb; i += kCW * 64) {
    int s = tot[i] + p.prefix[(size_t)blockIdx.x * nb + i];
    for (int v = 0; v < kCW; ++v) {
      const int c = cnt[v][i];
      cnt[v][i] = s;
      s += c;
    }
    if (blockIdx.x == 0) p.offsets[i] = tot[i];
  }
  __syncthreads();
  place(p, min(q1, q0 + w * per), min(q1, q0 + (w + 1) * per), cnt[w], tot[p.El]);
}

// ------------------------------------------------------------------------------------------------ rows

// VEC elements of T behind p, as floats; aligned to their size where that is 2, 4, 8 or 16 bytes.
template <class T, int VEC>
struct Raw {
  T v[VEC];
  __device__ __forceinline__ float operator[](int i) const { return (float)v[i]; }
};
template <class T, int VEC>
__device__ __forceinline__ Raw<T, VEC> ld_row(const T* p) {
  Raw<T, VEC> r;
  constexpr int B = VEC * sizeof(T);
  if constexpr (B % 16 == 0) {
    uint4* d = reinterpret_cast<uint4*>(&r);
#pragma unroll
    for (int i = 0; i < B / 16; ++i) d[i] = ld16(reinterpret_cast<const char*>(p) + 16 * i);
  } else if constexpr (B == 8) {
    *reinterpret_cast<uint2*>(&r) = *reinterpret_cast<const uint2*>(p);
  } else {
    static_assert(VEC == 1, "");
    r.v[0] = p[0];
  }
  return r;
}
template <class T, int VEC>
__device__ __forceinline__ void st_row(T* p, const float (&f)[VEC]) {
  alignas(16) T v[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) v[i] = (T)f[i];
  constexpr int B = VEC * sizeof(T);
  if constexpr (B % 16 == 0) {
    const uint4* s = reinterpret_cast<const uint4*>(v);
#pragma unroll
    for (int i = 0; i < B / 16; ++i) st16(reinterpret_cast<char*>(p) + 16 * i, s[i]);
  } else if constexpr (B == 8) {
    *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(v);
  } else {
    p[0] = v[0];
  }
}

// The position of slot `lane` of token t, -1 where there is none.
__device__ __forceinline__ int slot_pos(const PairsParams& p, int64_t t, int lane) {
  const int pos = lane < p.k ? p.pair_pos[t * p.k + lane] : -1;
  return pos >= 0 && pos < p.nrows ? pos : -1;
}
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), lane));
}
__device__ __forceinline__ float wave_sum(float v) {
  v = group_sum16(v);
  return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}

// One wavefront per token and part of its row (64 * kDispatch units of U); a unit is 16, 4, 2 or 1 bytes.
constexpr int kDispatch = 4;
template <class U>
__global__ __launch_bounds__(256) void k_dispatch(PairsParams p, int64_t units) {
  const int lane = threadIdx.x & 63;
  const int64_t nparts = (units + 64 * kDispatch - 1) / (64 * kDispatch);
  const U* x = static_cast<const U*>(p.x);
  U* rows = static_cast<U*>(p.out);
  for (int64_t u = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); u < p.T * nparts; u += (int64_t)gridDim.x * 4) {
    const int64_t t = u / nparts, c0 = (u - t * nparts) * 64 * kDispatch + lane;
    const int pos = slot_pos(p, t, lane);
    U v[kDispatch];
#pragma unroll
    for (int i = 0; i < kDispatch; ++i)
      if (c0 + 64 * i < units) v[i] = x[t * units + c0 + 64 * i];
    for (int j = 0; j < p.k; ++j) {
      const int r = __builtin_amdgcn_readlane(pos, j);
      if (r < 0) continue;
      U* to = rows + (int64_t)r * units + c0;
#pragma unroll
      for (int i = 0; i < kDispatch; ++i)
        if (c0 + 64 * i < units) to[64 * i] = v[i];
    }
  }
}

// One wavefront per token and part of its row (128 chunks of VEC elements).
template <class R, class D, int VEC>
__global__ __launch_bounds__(256) void k_pairs_combine(PairsParams p) {
  const int lane = threadIdx.x & 63;
  const int64_t nch = p.H / VEC, nparts = (nch + 127) / 128;
  const R* rows = static_cast<const R*>(p.x);
  D* y = static_cast<D*>(p.out);
  for (int64_t u = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); u < p.T * nparts; u += (int64_t)gridDim.x * 4) {
    const int64_t t = u / nparts, c0 = (u - t * nparts) * 128 + lane;
    const int pos = slot_pos(p, t, lane);
    const float wl = p.weight && lane < p.k ? p.weight[t * p.k + lane] : 1.f;
    float acc[2][VEC];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int v = 0; v < VEC; ++v) acc[h][v] = 0.f;
    for (int j0 = 0; j0 < p.k; j0 += 4) {
      Raw<R, VEC> raw[2][4];
      int ps[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        ps[j] = j0 + j < p.k ? __builtin_amdgcn_readlane(pos, j0 + j) : -1;
        if (ps[j] >= 0)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (c0 + 64 * h < nch) raw[h][j] = ld_row<R, VEC>(rows + (int64_t)ps[j] * p.H + (c0 + 64 * h) * VEC);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (ps[j] >= 0) {
          const float w = lane_value(wl, j0 + j);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int v = 0; v < VEC; ++v) acc[h][v] = fmaf(w, raw[h][j][v], acc[h][v]);
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (c0 + 64 * h < nch) st_row<D, VEC>(y + t * p.H + (c0 + 64 * h) * VEC, acc[h]);
  }
}

// One wavefront per token.
template <class R, class D, int VEC>
__global__ __launch_bounds__(256) void k_pairs_combine_bwd(PairsParams p) {
  const int lane = threadIdx.x & 63;
  const int64_t nch = p.H / VEC;
  for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < p.T; t += (int64_t)gridDim.x * 4) {
    const int pos = slot_pos(p, t, lane);
    const float wl = p.weight && lane < p.k ? p.weight[t * p.k + lane] : 1.f;
    const D* dy = static_cast<const D*>(p.x) + t * p.H;
    float dw = 0.f;
    for (int j = 0; j < p.k; ++j) {
      const int r = __builtin_amdgcn_readlane(pos, j);
      if (r < 0) continue;
      const float w = lane_value(wl, j);
      const R* row = static_cast<const R*>(p.rows) + (int64_t)r * p.H;
      R* drow = static_cast<R*>(p.out) + (int64_t)r * p.H;
      float dot = 0.f;
      for (int64_t c = lane; c < nch; c += 64) {
        const Raw<D, VEC> g = ld_row<D, VEC>(dy + c * VEC);
        const Raw<R, VEC> v = ld_row<R, VEC>(row + c * VEC);
        float o[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          dot = fmaf(g[i], v[i], dot);
          o[i] = w * g[i];
        }
        st_row<R, VEC>(drow + c * VEC, o);
      }
      dot = wave_sum(dot);
      if (lane == j) dw = dot;
    }
    if (lane < p.k) p.dweight[t * p.k + lane] = dw;
    if (!p.dlogits) continue;
    const int ex = lane < p.k ? p.idx[t * p.k + lane] : -1;
    const float prod = wl * dw;
    float mean = 0.f;
    for (int j = 0; j < p.k; ++j) mean += lane_value(prod, j);
    const float dl = wl * (dw - mean);
    for (int e0 = 0; e0 < p.E; e0 += 64) {
      float v = 0.f;
      for (int j = 0; j < p.k; ++j) {
        const float d = lane_value(dl, j);
        if (__builtin_amdgcn_readlane(ex, j) == e0 + lane) v += d;
      }
      if (e0 + lane < p.E) p.dlogits[t * p.E + e0 + lane] = v;
    }
  }
}

// Workgroups of 4 waves for `waves` of work, the rest in the kernels' loops (a dimension of a grid holds less than
// 2^32 threads).
unsigned grid4(int64_t waves) { return (unsigned)std::min<int64_t>((waves + 3) / 4, 1 << 22); }

bool multiple16(std::initializer_list<const void*> ps) {
  for (const void* q : ps)
    if (reinterpret_cast<uintptr_t>(q) % 16) return false;
  return true;
}

template <class U>
void dispatch_units(const PairsParams& p, int64_t bytes, hipStream_t s) {
  const int64_t units = bytes / (int64_t)sizeof(U), nparts = (units + 64 * kDispatch - 1) / (64 * kDispatch);
  k_dispatch<U><<<grid4(p.T * nparts), 256, 0, s>>>(p, units);
}

template <class R, class D>
void combine_types(const PairsParams& p, hipStream_t s) {
  constexpr int VEC = 16 / sizeof(R);
  if (p.H % VEC == 0 && p.H * sizeof(D) % 16 == 0 && multiple16({p.x, p.out}))
    k_pairs_combine<R, D, VEC><<<grid4(p.T * ((p.H / VEC + 127) / 128)), 256, 0, s>>>(p);
  else
    k_pairs_combine<R, D, 1><<<grid4(p.T * ((p.H + 127) / 128)), 256, 0, s>>>(p);
}

template <class R, class D>
void bwd_types(const PairsParams& p, hipStream_t s) {
  constexpr int VEC = 16 / sizeof(R);
  if (p.H % VEC == 0 && p.H * sizeof(D) % 16 == 0 && multiple16({p.x, p.rows, p.out}))
    k_pairs_combine_bwd<R, D, VEC><<<grid4(p.T), 256, 0, s>>>(p);
  else
    k_pairs_combine_bwd<R, D, 1><<<grid4(p.T), 256, 0, s>>>(p);
}

}  // namespace

hipError_t launch_sort_pairs(const SortParams& p, hipStream_t s) {
  hipError_t err;
  if (p.pairs <= kSortSmall) {
    prof_mark_begin("sort_pairs", s);
    k_sort_small<<<1, kSW * 64, 0, s>>>(p);
    if ((err = hipGetLastError()) == hipSuccess) prof_mark_end(s);
    return err;
  }
  prof_mark_begin("sort_count", s);
  k_sort_count<<<p.nblk, kCW * 64, 0, s>>>(p);
  if ((err = hipGetLastError()) != hipSuccess) return err;
  prof_mark_end(s);
  prof_mark_begin("sort_scan", s);
  k_sort_scan<<<p.El + 1, 256, 0, s>>>(p);
  if ((err = hipGetLastError()) != hipSuccess) return err;
  prof_mark_end(s);
  prof_mark_begin("sort_place", s);
  k_sort_place<<<p.nblk, kCW * 64, 0, s>>>(p);
  if ((err = hipGetLastError()) != hipSuccess) return err;
  prof_mark_end(s);
  return hipSuccess;
}

hipError_t launch_dispatch(const PairsParams& p, int elem, hipStream_t s) {
  const int64_t bytes = p.H * elem;
  prof_mark_begin("dispatch", s);
  const uintptr_t a = reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.out) | (uintptr_t)bytes;
  if (a % 16 == 0) dispatch_units<uint4>(p, bytes, s);
  else if (a % 4 == 0) dispatch_units<uint32_t>(p, bytes, s);
  else if (a % 2 == 0) dispatch_units<uint16_t>(p, bytes, s);
  else dispatch_units<uint8_t>(p, bytes, s);
  const hipError_t err = hipGetLastError();
  if (err == hipSuccess) prof_mark_end(s);
  return err;
}

hipError_t launch_pairs_combine(const PairsParams& p, hipStream_t s) {
  prof_mark_begin("pairs_combine", s);
  if (p.r32) p.x32 ? combine_types<float, float>(p, s) : combine_types<float, bf16>(p, s);
  else p.x32 ? combine_types<bf16, float>(p, s) : combine_types<bf16, bf16>(p, s);
  const hipError_t err = hipGetLastError();
  if (err == hipSuccess) prof_mark_end(s);
  return err;
}

hipError_t launch_pairs_combine_bwd(const PairsParams& p, hipStream_t s) {
  prof_mark_begin("pairs_combine_bwd", s);
  if (p.r32) p.x32 ? bwd_types<float, float>(p, s) : bwd_types<float, bf16>(p, s);
  else p.x32 ? bwd_types<bf16, float>(p, s) : bwd_types<bf16, bf16>(p, s);
  const hipError_t err = hipGetLastError();
  if (err == hipSuccess) prof_mark_end(s);
  return err;
}

}  // namespace moe
