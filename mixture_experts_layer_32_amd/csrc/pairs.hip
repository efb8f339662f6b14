// The layer taken apart: (token, slot) pairs sorted by expert, tokens' rows brought into that order and back with
// the routing weights, and the gradients of both ("A Magia da Fusão" on "IA: MoE Kernel 3x Mais Rápido Chegou!"
// lists dispatch and combine among the layer's steps).
//
//   k_sort_small    up to kSortSmall pairs: one workgroup counts, scans and places them (64 pairs of 128 experts 4 us).
//   k_sort_count, k_sort_place   beyond: counts per block of kSortPairs pairs and expert, positions. Up to kSortBlocks
//                   blocks every workgroup of the second adds up all blocks' counts by itself, a launch less (131072 pairs
//                   of 128 experts 5 + 7 us); for more, k_sort_scan makes their sums over the blocks (1048576 pairs 18 us).
//   k_dispatch      rows[pair_pos[t, j]] = x[t]: x is read once, each row written once. Bound by the writes: 131072 rows
//                   of 4 KB 98 to 106 us (5.7 to 6.2 TB/s; a plain write reaches 6.8 here).
//   k_pairs_combine y[t] = sum_j w_tj rows[pair_pos[t, j]]: each row read once. Bound by the reads: the same rows 106 to
//                   113 us (5.4 to 5.7 TB/s).
//   k_pairs_combine_bwd  drows = w dy, dw = <dy, rows>, dlogits: each row read and written once, a copy at heart: the same
//                   rows 219 to 230 us (5.0 to 5.2 TB/s; a copy reaches 4.9). Beyond 256 chunks a row, where dy is read again for
//                   each slot, 65536 rows of 8 KB 239 us (4.8 TB/s; by counter 0.99 GB read for 0.60) and of 14 KB 408 (4.9).
// Dispatch and combine have a form for short rows, several tokens to a wavefront (k_dispatch_short, k_pairs_combine_short);
// the gradients' rows keep a wavefront each, for their sums.
// A pair's place within its block comes from the lanes below it that hold the same expert (ballots over the expert's bits),
// so that the order is the pairs' own whatever the waves do; counts are LDS atomics of whole numbers, whose order is none.
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

// Places the wave's 64 pairs q, of experts e (-1: no pair): base[e] is the position of the wave's next pair of expert e (LDS,
// this wave's own), and P the number of pairs with a position. The wave's pairs come in order, 64 at a time.
__device__ __forceinline__ void place(const SortParams& p, int64_t q, int e, volatile int* base, int P) {
  const bool in = e >= 0;
  const unsigned long long m = same_lanes(in ? e : 0, in);
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

constexpr int kSW = 16;   // waves of k_sort_small
__global__ __launch_bounds__(kSW * 64) void k_sort_small(SortParams p) {
  __shared__ int cnt[kSW][kMaxExperts + 1];
  __shared__ int tot[kMaxExperts + 1];
  __shared__ int lds[kSW];
  const int tid = threadIdx.x, w = tid >> 6, nb = p.El + 1, n = (int)p.pairs;
  constexpr int NP = kSortSmall / (kSW * 64);            // pairs of a lane at most
  const int rounds = (n + kSW * 64 - 1) / (kSW * 64);    // 64 pairs of a wave, one wave's behind another's
  int e[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int q = (w * rounds + i) * 64 + (tid & 63);
    e[i] = i < rounds && q < n ? local_expert(p, q) : -1;
  }
  for (int i = tid; i < kSW * nb; i += kSW * 64) cnt[i / nb][i % nb] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NP; ++i)
    if (e[i] >= 0) atomicAdd(&cnt[w][e[i]], 1);
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
#pragma unroll
  for (int i = 0; i < NP; ++i)
    if (i < rounds) place(p, (w * rounds + i) * 64 + (tid & 63), e[i], cnt[w], tot[p.El]);
}

constexpr int kCW = 8;    // waves of a block of kSortPairs pairs
constexpr int kCP = kSortPairs / (64 * kCW);   // pairs of a lane: kCP w + i of 64 each, all loaded at once
__device__ __forceinline__ void load_experts(const SortParams& p, int64_t q0, int (&e)[kCP]) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
  for (int i = 0; i < kCP; ++i) {
    const int64_t q = q0 + (w * kCP + i) * 64 + lane;
    e[i] = q < p.pairs ? local_expert(p, q) : -1;
  }
}
__global__ __launch_bounds__(kCW * 64) void k_sort_count(SortParams p) {
  __shared__ int cnt[kMaxExperts + 1];
  const int tid = threadIdx.x, nb = p.El + 1;
  int e[kCP];
  load_experts(p, (int64_t)blockIdx.x * kSortPairs, e);
  for (int i = tid; i < nb; i += kCW * 64) cnt[i] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kCP; ++i)
    if (e[i] >= 0) atomicAdd(&cnt[e[i]], 1);
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
  __shared__ int tot[kMaxExperts + 1], pre[kMaxExperts + 1];
  __shared__ int2 part[kCW][64];
  __shared__ int lds[kCW];
  const int tid = threadIdx.x, w = tid >> 6, nb = p.El + 1;
  const int64_t q0 = (int64_t)blockIdx.x * kSortPairs;
  int e[kCP];
  load_experts(p, q0, e);
  if (p.prefix) {
    for (int i = tid; i < nb; i += kCW * 64) {
      tot[i] = p.total[i];
      pre[i] = p.prefix[(size_t)blockIdx.x * nb + i];
    }
  } else {
    // few blocks: their counts added up here, an eighth of the blocks by each wave
    for (int i0 = 0; i0 < nb; i0 += 64) {
      const int i = min(i0 + (tid & 63), nb - 1);
      int all = 0, before = 0;
#pragma unroll 8
      for (int b = w; b < p.nblk; b += kCW) {
        const int c = p.cnt[(size_t)b * nb + i];
        all += c;
        before += b < (int)blockIdx.x ? c : 0;
      }
      part[w][tid & 63] = make_int2(all, before);
      __syncthreads();
      if (tid < 64 && i0 + tid < nb) {
        int2 s = part[0][tid];
        for (int v = 1; v < kCW; ++v) {
          s.x += part[v][tid].x;
          s.y += part[v][tid].y;
        }
        tot[i0 + tid] = s.x;
        pre[i0 + tid] = s.y;
      }
      __syncthreads();
    }
  }
  for (int i = tid; i < kCW * nb; i += kCW * 64) cnt[i / nb][i % nb] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kCP; ++i)
    if (e[i] >= 0) atomicAdd(&cnt[w][e[i]], 1);
  scan_bins<kCW * 64>(tot, nb, lds);   // (its barriers stand behind the counts too)
  for (int i = tid; i < nb; i += kCW * 64) {
    int s = tot[i] + pre[i];
    for (int v = 0; v < kCW; ++v) {
      const int c = cnt[v][i];
      cnt[v][i] = s;
      s += c;
    }
    if (blockIdx.x == 0) p.offsets[i] = tot[i];
  }
  __syncthreads();
  const int P = tot[p.El];
#pragma unroll
  for (int i = 0; i < kCP; ++i) place(p, q0 + (w * kCP + i) * 64 + (tid & 63), e[i], cnt[w], P);
}

// ------------------------------------------------------------------------------------------------ rows
// Rows are worked on in chunks of VEC elements, 16 bytes of the rows' type (the other type's may be 8 or 32). Where every
// row begins at a multiple of 16 bytes and ends with a whole chunk (!ODD), rows that are read or written once go past the
// caches (non-temporal, whole lines: dispatch of 131072 rows of 4 KB 125 -> 105 us, combine 128 -> 108). Otherwise
// (ODD) chunks lie at any address of the elements, which the hardware loads and stores as well, and the last may be short.

template <class T, int VEC>
struct Raw {
  T v[VEC];
  __device__ __forceinline__ float operator[](int i) const { return (float)v[i]; }
};
template <int B> struct Bytes;   // B bytes at any address
typedef unsigned u32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned u32x2_t __attribute__((ext_vector_type(2)));
template <> struct Bytes<16> { typedef u32x4_t type __attribute__((aligned(1))); };
template <> struct Bytes<8> { typedef u32x2_t type __attribute__((aligned(1))); };

// Chunk at p, of which n elements are there (ODD; the others are 0). ONCE: read once.
template <class T, int VEC, bool ODD, bool ONCE>
__device__ __forceinline__ Raw<T, VEC> ld_row(const T* p, int n) {
  constexpr int B = VEC * sizeof(T), P = B < 16 ? B : 16;
  typedef typename Bytes<P>::type piece;
  Raw<T, VEC> r;
  if (!ODD || n >= VEC) {
#pragma unroll
    for (int i = 0; i < B / P; ++i) {
      const char* at = reinterpret_cast<const char*>(p) + P * i;
      if constexpr (ODD) reinterpret_cast<piece*>(&r)[i] = *reinterpret_cast<const piece*>(at);
      else if constexpr (P == 8) reinterpret_cast<uint2*>(&r)[i] = *reinterpret_cast<const uint2*>(at);
      else reinterpret_cast<uint4*>(&r)[i] = ONCE ? ld16_nt(at) : ld16(at);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) r.v[i] = i < n ? p[i] : (T)0.f;
  }
  return r;
}
template <class T, int VEC, bool ODD, bool ONCE>
__device__ __forceinline__ void st_row(T* p, const float (&f)[VEC], int n) {
  constexpr int B = VEC * sizeof(T), P = B < 16 ? B : 16;
  typedef typename Bytes<P>::type piece;
  alignas(16) T v[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) v[i] = (T)f[i];
  if (!ODD || n >= VEC) {
#pragma unroll
    for (int i = 0; i < B / P; ++i) {
      char* at = reinterpret_cast<char*>(p) + P * i;
      if constexpr (ODD) *reinterpret_cast<piece*>(at) = reinterpret_cast<const piece*>(v)[i];
      else if constexpr (P == 8) *reinterpret_cast<uint2*>(at) = reinterpret_cast<const uint2*>(v)[i];
      else if constexpr (ONCE && B == 16) st16_nt(at, reinterpret_cast<const uint4*>(v)[i]);
      else st16(at, reinterpret_cast<const uint4*>(v)[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (i < n) p[i] = v[i];
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

// A position of slot j of token t.
__device__ __forceinline__ int pos_of(const PairsParams& p, int64_t t, int j) {
  const int pos = p.pair_pos[t * p.k + j];
  return pos >= 0 && pos < p.nrows ? pos : -1;
}

// One wavefront per token and part of its row (64 kDispatch chunks of 16 bytes); E: the elements of a short last chunk.
constexpr int kDispatch = 4;
template <class E, bool ODD>
struct Copy16 {
  u32x4_t v;
  E e[ODD ? 16 / sizeof(E) : 1];
  __device__ __forceinline__ void load(const char* p, int bytes) {
    if (!ODD || bytes >= 16) v = *reinterpret_cast<const typename Bytes<16>::type*>(p);
    else
#pragma unroll
      for (int i = 0; i < 16 / (int)sizeof(E); ++i)
        if (i * (int)sizeof(E) < bytes) e[ODD ? i : 0] = reinterpret_cast<const E*>(p)[i];
  }
  __device__ __forceinline__ void store(char* p, int bytes) const {
    if (!ODD) st16_nt(p, make_uint4(v.x, v.y, v.z, v.w));
    else if (bytes >= 16) *reinterpret_cast<typename Bytes<16>::type*>(p) = v;
    else
#pragma unroll
      for (int i = 0; i < 16 / (int)sizeof(E); ++i)
        if (i * (int)sizeof(E) < bytes) reinterpret_cast<E*>(p)[i] = e[ODD ? i : 0];
  }
};
template <class E, bool ODD>
__global__ __launch_bounds__(256) void k_dispatch(PairsParams p, int64_t bytes) {
  const int lane = threadIdx.x & 63;
  const int64_t nch = (bytes + 15) / 16, nparts = (nch + 64 * kDispatch - 1) / (64 * kDispatch);
  const char* x = static_cast<const char*>(p.x);
  char* rows = static_cast<char*>(p.out);
  for (int64_t u = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); u < p.T * nparts; u += (int64_t)gridDim.x * 4) {
    const int64_t t = u / nparts, c0 = (u - t * nparts) * 64 * kDispatch + lane;
    const int pos = slot_pos(p, t, lane);
    Copy16<E, ODD> v[kDispatch];
#pragma unroll
    for (int i = 0; i < kDispatch; ++i)
      if (c0 + 64 * i < nch) v[i].load(x + t * bytes + (c0 + 64 * i) * 16, (int)min((int64_t)16, bytes - (c0 + 64 * i) * 16));
    for (int j = 0; j < p.k; ++j) {
      const int r = __builtin_amdgcn_readlane(pos, j);
      if (r < 0) continue;
#pragma unroll
      for (int i = 0; i < kDispatch; ++i)
        if (c0 + 64 * i < nch)
          v[i].store(rows + (int64_t)r * bytes + (c0 + 64 * i) * 16, (int)min((int64_t)16, bytes - (c0 + 64 * i) * 16));
    }
  }
}

// Short rows (at most 32 chunks): a thread takes one chunk of a token, a wavefront several tokens. L: the threads of a
// token, a power of two.
template <class E, bool ODD>
__global__ __launch_bounds__(256) void k_dispatch_short(PairsParams p, int bytes, int lg) {
  const int c = threadIdx.x & ((1 << lg) - 1), n = min(16, bytes - 16 * c);
  const char* x = static_cast<const char*>(p.x);
  char* rows = static_cast<char*>(p.out);
  for (int64_t t = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> lg; t < p.T; t += (int64_t)gridDim.x * 256 >> lg) {
    if (n <= 0) continue;
    Copy16<E, ODD> v;
    v.load(x + t * bytes + 16 * c, n);
    for (int j = 0; j < p.k; ++j) {
      const int r = pos_of(p, t, j);
      if (r >= 0) v.store(rows + (int64_t)r * bytes + 16 * c, n);
    }
  }
}

// One wavefront per token and part of its row (128 chunks), with the rows of four slots in flight (of eight: 131072 rows of 4
// KB 123 us where this takes 108; workgroups that take several tokens, 1024 of them, 118).
template <class R, class D, int VEC, bool ODD>
__global__ __launch_bounds__(256) void k_pairs_combine(PairsParams p) {
  const int lane = threadIdx.x & 63;
  const int64_t nch = (p.H + VEC - 1) / VEC, nparts = (nch + 127) / 128;
  const R* rows = static_cast<const R*>(p.x);
  D* y = static_cast<D*>(p.out);
  for (int64_t u = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); u < p.T * nparts; u += (int64_t)gridDim.x * 4) {
    const int64_t t = u / nparts, c0 = (u - t * nparts) * 128 + lane;
    const int pos = slot_pos(p, t, lane);
    const float wl = p.weight && lane < p.k ? p.weight[t * p.k + lane] : 1.f;
    int n[2];
    float acc[2][VEC];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      n[h] = (int)min((int64_t)VEC, p.H - (c0 + 64 * h) * VEC);
#pragma unroll
      for (int v = 0; v < VEC; ++v) acc[h][v] = 0.f;
    }
    for (int j0 = 0; j0 < p.k; j0 += 4) {
      Raw<R, VEC> raw[2][4];
      int ps[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        ps[j] = j0 + j < p.k ? __builtin_amdgcn_readlane(pos, j0 + j) : -1;
        if (ps[j] >= 0)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (c0 + 64 * h < nch)
              raw[h][j] = ld_row<R, VEC, ODD, true>(rows + (int64_t)ps[j] * p.H + (c0 + 64 * h) * VEC, n[h]);
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
      if (c0 + 64 * h < nch) st_row<D, VEC, ODD, false>(y + t * p.H + (c0 + 64 * h) * VEC, acc[h], n[h]);
  }
}

template <class R, class D, int VEC, bool ODD>
__global__ __launch_bounds__(256) void k_pairs_combine_short(PairsParams p, int lg) {
  const int c = threadIdx.x & ((1 << lg) - 1), n = min(VEC, (int)p.H - c * VEC);
  const R* rows = static_cast<const R*>(p.x);
  D* y = static_cast<D*>(p.out);
  for (int64_t t = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> lg; t < p.T; t += (int64_t)gridDim.x * 256 >> lg) {
    if (n <= 0) continue;
    float acc[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) acc[v] = 0.f;
    for (int j0 = 0; j0 < p.k; j0 += 4) {
      Raw<R, VEC> raw[4];
      int ps[4];
      float w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        ps[j] = j0 + j < p.k ? pos_of(p, t, j0 + j) : -1;
        w[j] = p.weight && j0 + j < p.k ? p.weight[t * p.k + j0 + j] : 1.f;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (ps[j] >= 0) raw[j] = ld_row<R, VEC, ODD, false>(rows + (int64_t)ps[j] * p.H + c * VEC, n);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (ps[j] >= 0)
#pragma unroll
          for (int v = 0; v < VEC; ++v) acc[v] = fmaf(w[j], raw[j][v], acc[v]);
    }
    st_row<D, VEC, ODD, false>(y + t * p.H + c * VEC, acc, n);
  }
}

// One wavefront per token. Its dy stays in registers where a row has at most 64 NV chunks, and a slot's row is loaded while
// the one before is worked on; longer rows (NV = 0) read dy again for each slot, from the caches.
template <class R, class D, int VEC, int NV, bool ODD>
__global__ __launch_bounds__(256) void k_pairs_combine_bwd(PairsParams p) {
  const int lane = threadIdx.x & 63;
  const int64_t nch = (p.H + VEC - 1) / VEC;
  auto there = [&](int64_t c) { return (int)min((int64_t)VEC, p.H - c * VEC); };
  for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < p.T; t += (int64_t)gridDim.x * 4) {
    const int pos = slot_pos(p, t, lane);
    const float wl = lane < p.k ? p.weight[t * p.k + lane] : 1.f;
    const D* dy = static_cast<const D*>(p.x) + t * p.H;
    const R* rows = static_cast<const R*>(p.rows);
    R* drows = static_cast<R*>(p.out);
    float dw = 0.f;
    auto chunk = [&](const Raw<D, VEC>& g, const Raw<R, VEC>& v, float w, float& dot, int r, int64_t c) {
      float o[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        dot = fmaf(g[i], v[i], dot);
        o[i] = w * g[i];
      }
      st_row<R, VEC, ODD, true>(drows + (int64_t)r * p.H + c * VEC, o, there(c));
    };
    if constexpr (NV > 0) {
      Raw<D, VEC> g[NV];
      Raw<R, VEC> v[NV], next[NV];
      auto load = [&](int r) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (lane + 64 * i < nch)
            next[i] = ld_row<R, VEC, ODD, true>(rows + (int64_t)r * p.H + (lane + 64 * i) * VEC, there(lane + 64 * i));
      };
      unsigned long long left = __ballot(pos >= 0);   // slots with a position
      if (left) {
        load(__builtin_amdgcn_readlane(pos, __ffsll((long long)left) - 1));
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (lane + 64 * i < nch) g[i] = ld_row<D, VEC, ODD, false>(dy + (lane + 64 * i) * VEC, there(lane + 64 * i));
      }
      while (left) {
        const int j = __ffsll((long long)left) - 1, r = __builtin_amdgcn_readlane(pos, j);
        left &= left - 1;
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = next[i];
        if (left) load(__builtin_amdgcn_readlane(pos, __ffsll((long long)left) - 1));
        const float w = lane_value(wl, j);
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (lane + 64 * i < nch) chunk(g[i], v[i], w, dot, r, lane + 64 * i);
        dot = wave_sum(dot);
        if (lane == j) dw = dot;
      }
    } else {
      for (int j = 0; j < p.k; ++j) {
        const int r = __builtin_amdgcn_readlane(pos, j);
        if (r < 0) continue;
        const float w = lane_value(wl, j);
        float dot = 0.f;
        for (int64_t c = lane; c < nch; c += 64)
          chunk(ld_row<D, VEC, ODD, false>(dy + c * VEC, there(c)),
                ld_row<R, VEC, ODD, true>(rows + (int64_t)r * p.H + c * VEC, there(c)), w, dot, r, c);
        dot = wave_sum(dot);
        if (lane == j) dw = dot;
      }
    }
    if (lane < p.k) p.dweight[t * p.k + lane] = dw;
    if (!p.dlogits) continue;
    const int ex = lane < p.k ? p.idx[t * p.k + lane] : -1;
    const float prod = pos >= 0 ? wl * dw : 0.f;   // (the weight of a slot without a position may be anything)
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

// A token's threads where it has at most 32 chunks: the next power of two's logarithm; -1 for longer rows.
int short_lg(int64_t nch) {
  if (nch > 32) return -1;
  int lg = 0;
  while ((1 << lg) < nch) ++lg;
  return lg;
}

template <class E, bool ODD>
void dispatch_rows(const PairsParams& p, int64_t bytes, hipStream_t s) {
  const int64_t nch = (bytes + 15) / 16;
  const int lg = short_lg(nch);
  if (lg >= 0) k_dispatch_short<E, ODD><<<grid4((p.T + (64 >> lg) - 1) >> (6 - lg)), 256, 0, s>>>(p, (int)bytes, lg);
  else k_dispatch<E, ODD><<<grid4(p.T * ((nch + 64 * kDispatch - 1) / (64 * kDispatch))), 256, 0, s>>>(p, bytes);
}

template <class R, class D, bool ODD>
void combine_rows(const PairsParams& p, hipStream_t s) {
  constexpr int VEC = 16 / sizeof(R);
  const int64_t nch = (p.H + VEC - 1) / VEC;
  const int lg = short_lg(nch);
  if (lg >= 0) k_pairs_combine_short<R, D, VEC, ODD><<<grid4((p.T + (64 >> lg) - 1) >> (6 - lg)), 256, 0, s>>>(p, lg);
  else k_pairs_combine<R, D, VEC, ODD><<<grid4(p.T * ((nch + 127) / 128)), 256, 0, s>>>(p);
}
template <class R, class D>
void combine_types(const PairsParams& p, hipStream_t s) {
  constexpr int VEC = 16 / sizeof(R);
  if (p.H % VEC == 0 && p.H * sizeof(D) % 16 == 0 && multiple16({p.x, p.out})) combine_rows<R, D, false>(p, s);
  else combine_rows<R, D, true>(p, s);
}

template <class R, class D, bool ODD>
void bwd_rows(const PairsParams& p, hipStream_t s) {
  constexpr int VEC = 16 / sizeof(R);
  const int64_t nch = (p.H + VEC - 1) / VEC;
  const unsigned grid = grid4(p.T);
  if (nch <= 64) k_pairs_combine_bwd<R, D, VEC, 1, ODD><<<grid, 256, 0, s>>>(p);
  else if (nch <= 128) k_pairs_combine_bwd<R, D, VEC, 2, ODD><<<grid, 256, 0, s>>>(p);
  else if (nch <= 256) k_pairs_combine_bwd<R, D, VEC, 4, ODD><<<grid, 256, 0, s>>>(p);
  else k_pairs_combine_bwd<R, D, VEC, 0, ODD><<<grid, 256, 0, s>>>(p);
}
template <class R, class D>
void bwd_types(const PairsParams& p, hipStream_t s) {
  constexpr int VEC = 16 / sizeof(R);
  if (p.H % VEC == 0 && p.H * sizeof(D) % 16 == 0 && multiple16({p.x, p.rows, p.out})) bwd_rows<R, D, false>(p, s);
  else bwd_rows<R, D, true>(p, s);
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
  if (p.prefix) {
    prof_mark_begin("sort_scan", s);
    k_sort_scan<<<p.El + 1, 256, 0, s>>>(p);
    if ((err = hipGetLastError()) != hipSuccess) return err;
    prof_mark_end(s);
  }
  prof_mark_begin("sort_place", s);
  k_sort_place<<<p.nblk, kCW * 64, 0, s>>>(p);
  if ((err = hipGetLastError()) != hipSuccess) return err;
  prof_mark_end(s);
  return hipSuccess;
}

hipError_t launch_dispatch(const PairsParams& p, int elem, hipStream_t s) {
  const int64_t bytes = p.H * elem;
  prof_mark_begin("dispatch", s);
  if (bytes % 16 == 0 && multiple16({p.x, p.out})) dispatch_rows<uint32_t, false>(p, bytes, s);
  else if (elem == 4) dispatch_rows<uint32_t, true>(p, bytes, s);
  else if (elem == 2) dispatch_rows<uint16_t, true>(p, bytes, s);
  else dispatch_rows<uint8_t, true>(p, bytes, s);
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
