// The whole layer for a few tokens (T <= 64), forward only, in bf16, fp32 or with 8-bit weights.
//
// At a few tokens the layer reads the weights of the experts that were chosen, once, and does little
// else: 6 H F flops against 3 H F elements per pair. These kernels are built around that read. One wave
// instruction takes 256 bytes of each of 4 weight rows (whole cache lines, non-temporal), and the
// arithmetic is v_mfma_*_4x4x4_16b: sixteen independent 4 x 4 products, here 4 rows by 4 tokens for
// sixteen 16-byte pieces of the rows, whose sums are added over the lanes at the end of a row. An expert's
// tokens are taken in sets of 4, up to 4 sets at a time, so that little of the matrix work is padding.
// Reads alone, 320 MB on 256 CUs: 4 rows x 256 B 6.5 TB/s (5.7 without the non-temporal hint), 16 rows x
// 64 B, the form a 16 x 16 MFMA would take, 5.2 TB/s either way.
//
//   k_few_prep    logits = x W_r^T (4 experts by 16 tokens per workgroup) and, with 8-bit weights, the quantised
//                 rows of x. Only launched where one of the two is asked for.
//   k_few_topk    the tokens' experts and weights; only launched for more than 16 tokens (with 8-bit weights and
//                 given logits k_few_prep does it).
//   k_few_gateup  every workgroup sorts the pairs for itself (and, up to 16 tokens, chooses them); then its
//                 waves take (expert, 4 or 8 rows of F) units, each on its own, and write h = w silu(a) b into
//                 the workspace. Bound by the read of the gate and up rows.
//   k_few_down    a workgroup owns 4 NQ rows of H for every expert: its waves share the (expert, F) axis,
//                 each keeping its own sum per token, and the sums are added in a fixed order, without
//                 atomics: repeated calls give the same bits. Bound by the read of the down rows.
// Experts of more than 8 tokens ("heavy") take 16 x 16 MFMA tiles with their tokens' rows in LDS, so that
// their weights too are read once: in k_few_gateup and, mostly, in k_few_heavy ahead of k_few_down (heavy_ahead), which
// leaves the heavy experts' products, [pairs, H] in fp32, in memory for k_few_down to add. The others' stay in LDS.
//
// Measured, one launch, median us (2048 x 768 and 4096 x 1536, 128 experts, top-8, bf16; read rate of the weights):
//                    1 token 2048     8 tokens 2048     64 skewed tokens 4096
//   k_few_gateup     15               61-65 (5.3 TB/s)  303 (6.0 TB/s)
//   k_few_heavy                                         61 (4.6 TB/s)
//   k_few_down       9                32 (5.4 TB/s)     117 (6.1 TB/s)
// About 5 us of the one-token k_few_gateup are its launch and the choice of experts, which it must wait for.
//
// h is kept as fp32, or in bf16 mode to 2^-18 of each value as the pair hi = bf16(h), lo = bf16(h - hi), whose two
// products cost matrix time that a read-bound kernel does not miss. y is off by 2.5e-6 of its rms for it, as much as fp32 sums
// of 4096 terms in a row are; with hi alone by 1.7e-3, as much as by y's own rounding.
#include <math.h>

#include <algorithm>

#include "engine.h"
#include "int8_device.h"
#include "moe_internal.h"
#include "route_device.h"

namespace moe {
namespace {

constexpr int kGW = 8;       // waves of k_few_gateup
constexpr int kDW = 16;      // waves of k_few_down
constexpr int kPW = 8;       // waves of k_few_prep
constexpr int kSeg = 256;    // bytes of one weight row per wave instruction
constexpr int kDown4 = 4096; // H from which a workgroup of k_few_down owns 16 rows
constexpr int kSets = 4;     // sets of 4 tokens taken at once

// Sixteen 4x4 products over 16 bytes of contraction. Lane l supplies row l & 3 of A and column l & 3 of
// B, piece l >> 2; accumulator element i of lane l is row i, column l & 3 of block l >> 2.
template <class T> struct Mma4;
template <> struct Mma4<bf16> {
  typedef f32x4 Acc;
  static __device__ __forceinline__ void go(Acc& c, const uint4& a, const uint4& b) {
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    c = __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(__builtin_bit_cast(s16x4, make_uint2(a.x, a.y)),
                                               __builtin_bit_cast(s16x4, make_uint2(b.x, b.y)), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(__builtin_bit_cast(s16x4, make_uint2(a.z, a.w)),
                                               __builtin_bit_cast(s16x4, make_uint2(b.z, b.w)), c, 0, 0, 0);
  }
};
template <> struct Mma4<float> {
  typedef f32x4 Acc;
  static __device__ __forceinline__ void go(Acc& c, const uint4& a, const uint4& b) {
    c = __builtin_amdgcn_mfma_f32_4x4x1f32(__uint_as_float(a.x), __uint_as_float(b.x), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_4x4x1f32(__uint_as_float(a.y), __uint_as_float(b.y), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_4x4x1f32(__uint_as_float(a.z), __uint_as_float(b.z), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_4x4x1f32(__uint_as_float(a.w), __uint_as_float(b.w), c, 0, 0, 0);
  }
};
template <> struct Mma4<int8_t> {
  typedef i32x4 Acc;
  static __device__ __forceinline__ void go(Acc& c, const uint4& a, const uint4& b) {
    c = __builtin_amdgcn_mfma_i32_4x4x4i8((int)a.x, (int)b.x, c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_i32_4x4x4i8((int)a.y, (int)b.y, c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_i32_4x4x4i8((int)a.z, (int)b.z, c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_i32_4x4x4i8((int)a.w, (int)b.w, c, 0, 0, 0);
  }
};

// One 16x16 product over 64 bytes of contraction: lane l supplies row (column) l & 15, 16-byte piece
// l >> 4; accumulator element i of lane l is row 4 (l >> 4) + i, column l & 15. For heavy experts.
__device__ __forceinline__ void mma16x16(f32x4& c, const uint4& a, const uint4& b, bf16) { mma16<bf16>(c, a, b); }
__device__ __forceinline__ void mma16x16(f32x4& c, const uint4& a, const uint4& b, float) { mma16<float>(c, a, b); }
__device__ __forceinline__ void mma16x16(i32x4& c, const uint4& a, const uint4& b, int8_t) {
  c = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}
constexpr int kStep = 64;    // bytes of a row per such step

// sum over the sixteen blocks (the lanes with equal l & 3), in every lane
__device__ __forceinline__ float block_sum(float v) {
  v += dpp_mov<0x124>(v);   // row_ror:4
  v += dpp_mov<0x128>(v);   // row_ror:8
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}
__device__ __forceinline__ int block_sum(int v) {
  v += (int)dpp_mov<0x124>((unsigned)v);
  v += (int)dpp_mov<0x128>((unsigned)v);
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// ------------------------------------------------------------------------------------------------
// routing of the few tokens inside a workgroup

// Experts with pairs, in classes by their number of tokens: more than 16, 9-16 (both "heavy"), 5-8, 3-4, 1-2.
constexpr int kClasses = 5;
constexpr int kClassBits = 12, kClassMask = (1 << kClassBits) - 1;   // of a count of experts by class, up to 512; five in 64 bits
__device__ __forceinline__ int few_class(int n) { return n > 16 ? 0 : n > 8 ? 1 : n > 4 ? 2 : n > 2 ? 3 : 4; }

// The routing of all T tokens in a workgroup's LDS, pairs sorted by (local expert, token).
struct FewRoute {
  unsigned long long* mask;   // [El] tokens that chose the expert
  int4* ent;                  // [El] active experts by class: expert, first pair, pairs
  int* cls;                   // [kClasses + 1] first entry of each class
  int* off;                   // [El + 1] first pair of each expert
  int* el;                    // [T k] local expert of pair t k + j, -1: not local
  float* wt;                  // [T k] its weight
  int* stok;                  // [T k] token of sorted pair p
  float* swt;                 // [T k] its weight
  static __host__ __device__ size_t bytes(int El, int n) {
    return (size_t)El * 24 + (kClasses + 1) * 4 + (size_t)(El + 1) * 4 + (size_t)n * 16 + 16;
  }
  __device__ __forceinline__ FewRoute(char* s, int El, int n) {
    ent = reinterpret_cast<int4*>(s);
    mask = reinterpret_cast<unsigned long long*>(ent + El);
    cls = reinterpret_cast<int*>(mask + El);
    off = cls + kClasses + 1;
    el = off + El + 1;
    wt = reinterpret_cast<float*>(el + n);
    stok = reinterpret_cast<int*>(wt + n);
    swt = reinterpret_cast<float*>(stok + n);
  }
};

// the k chosen experts of token t and their weights, by one wave: lane j < k returns slot j's
__device__ __forceinline__ void choose(const FewParams& p, int t, int lane, int& e, float& wt) {
  const float* row = p.logits + (size_t)t * p.E;
  float v = 0.f;
  e = 0;
  if (p.E <= 64) wave_topk<1>(row, p.E, p.k, lane, e, v);
  else if (p.E <= 128) wave_topk<2>(row, p.E, p.k, lane, e, v);
  else if (p.E <= 256) wave_topk<4>(row, p.E, p.k, lane, e, v);
  else wave_topk<8>(row, p.E, p.k, lane, e, v);
  const float top = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 0));
  const float z = lane < p.k ? expf(v - top) : 0.f;
  float s = 0.f;   // summed in slot order
  for (int j = 0; j < p.k; ++j) s += __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(z), j));
  wt = z / s;
}

// More than kRouteHere tokens: one wave a token, ahead of the kernels that use the choice, for 4.5 us. In every
// workgroup of k_few_gateup the choices of 9 tokens take 3 us, of 16 4, of 32 9 and of 64 20.
constexpr int kRouteHere = 16;
__device__ __forceinline__ void choose_store(const FewParams& p, int t, int lane) {
  int e;
  float wt;
  choose(p, t, lane, e, wt);
  if (lane < p.k) {
    p.r_idx[t * p.k + lane] = e;
    p.r_wt[t * p.k + lane] = wt;
  }
}
__global__ __launch_bounds__(64) void k_few_topk(FewParams p) { choose_store(p, blockIdx.x, threadIdx.x); }

template <int NW>
__device__ __forceinline__ void few_route(const FewRoute& R, const FewParams& p) {
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, n = p.T * p.k;
  for (int e = tid; e < p.El; e += NW * 64) R.mask[e] = 0ull;
  __syncthreads();
  auto put = [&](int i, int e, float wt) {   // pair i = t k + j
    const bool here = e >= 0 && e < p.El;
    R.el[i] = here ? e : -1;
    R.wt[i] = wt;
    if (here) atomicOr(&R.mask[e], 1ull << (i / p.k));
  };
  if (p.T > kRouteHere) {
    for (int i = tid; i < n; i += NW * 64) put(i, p.r_idx[i] - p.e0, p.r_wt[i]);
  } else {
    for (int t = w; t < p.T; t += NW) {
      int e;
      float wt;
      choose(p, t, lane, e, wt);
      if (lane < p.k) put(t * p.k + lane, e - p.e0, wt);
    }
  }
  __syncthreads();
  if (w == 0) {   // lane's experts: a contiguous run; counts of pairs, and of experts by class
    const int per = (p.El + 63) >> 6, e0 = lane * per;
    int c = 0;
    unsigned long long a = 0ull;
    for (int i = 0; i < per; ++i) {
      const int m = e0 + i < p.El ? __popcll(R.mask[e0 + i]) : 0;
      c += m;
      if (m > 0) a += 1ull << (kClassBits * few_class(m));
    }
    int ic = c;
    unsigned long long ia = a;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int nc = __shfl_up(ic, d);
      const unsigned long long na = __shfl_up(ia, d);
      if (lane >= d) {
        ic += nc;
        ia += na;
      }
    }
    const unsigned long long all = __shfl(ia, 63);
    unsigned long long at = ia - a;   // class q's next entry
#pragma unroll
    for (int q = 0; q < kClasses; ++q)
#pragma unroll
      for (int r = 0; r < q; ++r) at += ((all >> (kClassBits * r)) & kClassMask) << (kClassBits * q);
    int o = ic - c;
    for (int i = 0; i < per; ++i) {
      const int e = e0 + i;
      if (e >= p.El) break;
      const int m = __popcll(R.mask[e]);
      R.off[e] = o;
      if (m > 0) {
        const int q = kClassBits * few_class(m);
        R.ent[(at >> q) & kClassMask] = make_int4(e, o, m, 0);
        at += 1ull << q;
      }
      o += m;
    }
    if (lane == 63) R.off[p.El] = ic;
    if (lane == 0) {
      int first = 0;
#pragma unroll
      for (int q = 0; q < kClasses; ++q) {
        R.cls[q] = first;
        first += (int)((all >> (kClassBits * q)) & kClassMask);
      }
      R.cls[kClasses] = first;
    }
  }
  __syncthreads();
  for (int i = tid; i < n; i += NW * 64) {
    const int e = R.el[i], t = i / p.k;
    if (e >= 0) {
      const int pos = R.off[e] + __popcll(R.mask[e] & ((1ull << t) - 1ull));
      R.stok[pos] = t;
      R.swt[pos] = R.wt[i];
    }
  }
  __syncthreads();
}

__device__ __forceinline__ int4 uniform4(const int4& v) {
  return make_int4(__builtin_amdgcn_readfirstlane(v.x), __builtin_amdgcn_readfirstlane(v.y),
                   __builtin_amdgcn_readfirstlane(v.z), 0);
}

// ------------------------------------------------------------------------------------------------
// NQ times 4 weight rows times NS sets of 4 tokens, segments [s0, s1) of 256 bytes. Each lane's pointers
// are at its own 16-byte piece of the rows. Two buffers of U segments: the next one's loads are issued
// before the MFMAs of the current (past the run's end, the last segment again).
template <class T, int NQ, int NS, int U>
__device__ __forceinline__ void dot4(const char* const (&pw)[NQ], const char* const (&px)[NS], int s0, int s1,
                                     typename Mma4<T>::Acc (&acc)[NQ][NS]) {
  struct Buf {
    uint4 a[NQ][U], b[NS][U];
  };
  auto load = [&](Buf& v, int s) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int o = min(s + i, s1 - 1) * kSeg;
#pragma unroll
      for (int q = 0; q < NQ; ++q) v.a[q][i] = ld16_nt(pw[q] + o);
#pragma unroll
      for (int t = 0; t < NS; ++t) v.b[t][i] = ld16(px[t] + o);
    }
  };
  auto mul = [&](const Buf& v, int s) {
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (s + i < s1)
#pragma unroll
        for (int q = 0; q < NQ; ++q)
#pragma unroll
          for (int t = 0; t < NS; ++t) Mma4<T>::go(acc[q][t], v.a[q][i], v.b[t][i]);
  };
  if (s0 >= s1) return;
  Buf u, v;
  load(u, s0);
  for (int s = s0; s < s1; s += 2 * U) {
    if (s + U < s1) load(v, s + U);
    mul(u, s);
    if (s + 2 * U < s1) load(u, s + 2 * U);
    if (s + U < s1) mul(v, s + U);
  }
}

template <class A, int NQ, int NS>
__device__ __forceinline__ void clear(A (&acc)[NQ][NS]) {
#pragma unroll
  for (int q = 0; q < NQ; ++q)
#pragma unroll
    for (int t = 0; t < NS; ++t) acc[q][t] = A{0, 0, 0, 0};
}

__device__ __forceinline__ float4 ld4f(const float* p) { return make_float4(p[0], p[1], p[2], p[3]); }

// h of rows f0 .. f0+3 and pair pos (of token t, weight wt) from the products' sums; 8-bit weights: times
// the scales of the token's row and of the 4 gate and up rows
template <class T>
__device__ __forceinline__ void store_h(const FewParams& p, int pos, int t, float wt, int f0,
                                        const typename Mma4<T>::Acc& sa, const typename Mma4<T>::Acc& sb, const float4& sg,
                                        const float4& su) {
  const float g[4] = {sg.x, sg.y, sg.z, sg.w}, u[4] = {su.x, su.y, su.z, su.w};
  const float xs = sizeof(T) == 1 ? p.xs[t] : 1.f;
  float h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = (float)sa[i], b = (float)sb[i];
    if constexpr (sizeof(T) == 1) {
      a *= xs * g[i];
      b *= xs * u[i];
    }
    if constexpr (sizeof(T) == 1) h[i] = weighted_swiglu8(wt, a, b);
    else h[i] = wt * (a / (1.0f + expf(-a)) * b);
  }
  const size_t at = (size_t)pos * p.F + f0;
  if constexpr (sizeof(T) == 2) {
    // The high part is at most bf16's largest value: an h between that and fp32's would round to an infinity, and
    // the low part of an infinite h would be a NaN. An infinite h has an infinite low part instead, a NaN a NaN.
    constexpr float kTop = 0x1.fep127f;
    float hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      hi[i] = fminf(fmaxf(h[i], -kTop), kTop);
      lo[i] = h[i] - (float)(bf16)hi[i];
    }
    eng::st8(static_cast<bf16*>(p.h) + at, eng::pack4(hi[0], hi[1], hi[2], hi[3]));
    eng::st8(static_cast<bf16*>(p.hlo) + at, eng::pack4(lo[0], lo[1], lo[2], lo[3]));
  } else {
    *reinterpret_cast<float4*>(static_cast<float*>(p.h) + at) = make_float4(h[0], h[1], h[2], h[3]);
  }
  if (sizeof(T) == 1 && p.hmax)   // 4 rows' largest: k_few_down takes the pair's (one atomic maximum a pair
                                  // from every unit, on the same few cache lines, took 15 us for one token)
    p.hmax[(size_t)pos * (p.F / 4) + f0 / 4] =
        max(max(mag_bits(h[0]), mag_bits(h[1])), max(mag_bits(h[2]), mag_bits(h[3])));
}

// LDS of heavy_task's stages and gateup_unit's partial sums; more than 8 tokens can make an expert heavy
__host__ __device__ inline int few_red_bytes(int T) { return T > 16 ? 2 * 64 * kSeg : T > 8 ? 2 * 16 * kSeg : kGW * 32 * 16; }

// One unit of the gate/up products by a wave: rows f0 .. f0 + 4 QR - 1 of expert e, pairs base .. base+cnt-1
// (cnt <= 4 NS). QR = 2 with 3 to 8 tokens: their rows of x are read once for 8 rows of F (64 tokens of 128 experts,
// 4096 x 1536: 600 us with 4 rows, 534 with 8; with 1 or 2 tokens 8 rows are no better, 39 -> 42 us for 4 tokens of
// the 2048 x 768 layer). PART: only part kp of ks of H, whose sums go to red [token][QR][2] of the wave instead.
template <class T, int QR, int NS, bool PART>
__device__ __forceinline__ void gateup_unit(const FewParams& p, const FewRoute& R, typename Mma4<T>::Acc* red, int e,
                                            int base, int cnt, int f0, int ks, int kp) {
  typedef typename Mma4<T>::Acc Acc;
  constexpr int ES = sizeof(T);
  const int lane = threadIdx.x & 63, j = lane & 3, piece = 16 * (lane >> 2);
  const size_t rowb = (size_t)p.H * ES;
  const char* pw[2 * QR];
  float4 sg[QR] = {}, su[QR] = {};
#pragma unroll
  for (int q = 0; q < QR; ++q) {
    const size_t wo = ((size_t)e * p.F + f0 + 4 * q + j) * rowb + piece;
    pw[2 * q] = static_cast<const char*>(p.wg) + wo;
    pw[2 * q + 1] = static_cast<const char*>(p.wu) + wo;
    if constexpr (ES == 1 && !PART) {   // asked for before the products, used after them
      sg[q] = ld4f(p.sg + (size_t)e * p.F + f0 + 4 * q);
      su[q] = ld4f(p.su + (size_t)e * p.F + f0 + 4 * q);
    }
  }
  const char* px[NS];
#pragma unroll
  for (int t = 0; t < NS; ++t)
    px[t] = static_cast<const char*>(p.x) + R.stok[base + min(4 * t + j, cnt - 1)] * rowb + piece;
  Acc acc[2 * QR][NS];
  clear(acc);
  const int S = (int)(rowb / kSeg), s0 = PART ? kp * S / ks : 0, s1 = PART ? (kp + 1) * S / ks : S;
  dot4<T, 2 * QR, NS, (QR * NS > 2 ? 1 : QR > 1 || ES == 1 ? 2 : 4)>(pw, px, s0, s1, acc);
#pragma unroll
  for (int t = 0; t < NS; ++t)
#pragma unroll
    for (int q = 0; q < QR; ++q) {
      Acc a, b;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = block_sum(acc[2 * q][t][i]);
        b[i] = block_sum(acc[2 * q + 1][t][i]);
      }
      if constexpr (PART) {
        if (lane < 4) {
          red[2 * ((4 * t + j) * QR + q)] = a;
          red[2 * ((4 * t + j) * QR + q) + 1] = b;
        }
      } else if (lane < 4 && 4 * t + j < cnt) {
        const int pos = base + 4 * t + j;
        store_h<T>(p, pos, R.stok[pos], R.swt[pos], f0 + 4 * q, a, b, sg[q], su[q]);
      }
    }
}

// the parts' sums of a unit, added in order, and its h; red: the first part's wave's, 32 sums a wave
template <class T, int QR>
__device__ __forceinline__ void gateup_join(const FewParams& p, const FewRoute& R, const typename Mma4<T>::Acc* red, int e,
                                            int base, int cnt, int f0, int ks) {
  const int lane = threadIdx.x & 63;   // (token, quad)
  if (lane < cnt * QR) {
    const int f = f0 + 4 * (lane % QR), pos = base + lane / QR;
    float4 sg = {}, su = {};
    if constexpr (sizeof(T) == 1) {
      sg = ld4f(p.sg + (size_t)e * p.F + f);
      su = ld4f(p.su + (size_t)e * p.F + f);
    }
    typename Mma4<T>::Acc a = red[2 * lane], b = red[2 * lane + 1];
    for (int k = 1; k < ks; ++k) {
      a += red[32 * k + 2 * lane];
      b += red[32 * k + 2 * lane + 1];
    }
    store_h<T>(p, pos, R.stok[pos], R.swt[pos], f, a, b, sg, su);
  }
}

// ------------------------------------------------------------------------------------------------
// 128 weight rows of an expert with up to 16 NG tokens by a workgroup of 8 waves, on 16 x 16 tiles. The
// expert's rows of x (DOWN: of h) go through LDS 256 bytes of contraction at a time, so that each is read
// once per 128 weight rows; a wave takes 32 of those rows straight from memory, two chunks of 256 bytes ahead.
// Waves w and w + 4 take the same rows and each half of a chunk (16 rows a wave and whole chunks: twice the LDS
// reads, which then bound it, 70 us for 64 tokens on 8 experts of 4096 x 1536), and add their sums at the end.
// Not DOWN: gate and up rows r0 .. r0+63, a wave's 16 of each. DOWN: rows r0 .. r0+127 of W_down, and the
// products (8-bit: with their scales) go to oh [pairs, H].
// LDS: [2 stages][planes][16 NG rows][256 bytes], 16-byte piece c of row r at slot c ^ (r & 15); at the end
// [4 waves][2][NG][64] sums.
constexpr int heavy_lds(int ng, int planes) { return 2 * planes * 16 * ng * kSeg; }
template <class T, int NG, bool DOWN>
__device__ __forceinline__ void heavy_task(const FewParams& p, const int* stok, const float* swt, char* lds, int e, int base,
                                           int cnt, int r0) {
  typedef typename Mma4<T>::Acc Acc;
  constexpr int ES = sizeof(T), NP = DOWN && ES == 2 ? 2 : 1, BL = (NG + 1) / 2, PLANE = 16 * NG * kSeg;
  const int tid = threadIdx.x, lane = tid & 63, w = eng::wave_id(), rg = w & 3, kh = w >> 2;
  const int rowb = (DOWN ? p.F : p.H) * ES, nc = (rowb + kSeg - 1) / kSeg;
  // this thread's pieces of the staged rows (one column group: the first half of the threads)
  const bool puts = NG > 1 || tid < 256;
  const char* pb[NP][BL];
  int at[BL];
#pragma unroll
  for (int j = 0; j < BL; ++j) {
    const int i = (tid + 512 * j) % (256 * NG), r = i >> 4, c = i & 15, pos = base + min(r, cnt - 1);
    at[j] = r * kSeg + ((c ^ (r & 15)) << 4);
    if constexpr (DOWN) {
      pb[0][j] = (ES == 1 ? reinterpret_cast<const char*>(p.hq) : static_cast<const char*>(p.h)) + (size_t)pos * rowb + 16 * c;
      if constexpr (NP == 2) pb[1][j] = static_cast<const char*>(p.hlo) + (size_t)pos * rowb + 16 * c;
    } else {
      pb[0][j] = static_cast<const char*>(p.x) + (size_t)stok[pos] * rowb + 16 * c;
    }
  }
  // this lane's two weight rows, at its 16-byte piece of its half of a chunk
  const int wr = lane & 15, q4 = lane >> 4;
  const char* pa[2];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const size_t row = DOWN ? (size_t)e * p.H + r0 + 32 * rg + 16 * m + wr : (size_t)e * p.F + r0 + 16 * rg + wr;
    pa[m] = static_cast<const char*>(DOWN ? p.wd : m == 0 ? p.wg : p.wu) + row * rowb + 2 * kStep * kh + 16 * q4;
  }
  const uint4 zero = make_uint4(0, 0, 0, 0);
  struct Rows {
    uint4 a[2][2];
  };
  uint4 bb[NP][BL];
  // The chunks are taken from a place of the workgroup's own on: in step, the workgroups' rows, a power of two
  // apart, would meet on the same memory channels (8 % of the time).
  const int rot = (blockIdx.x * 7) % nc;
  auto at_chunk = [&](int c) { return (c + rot < nc ? c + rot : c + rot - nc) * kSeg; };
  // 8-bit rows of W_down may end in the middle of the last 256 bytes: the wave of the missing half takes the first
  // half again, against staged rows of zeros
  constexpr bool TAIL = DOWN && ES == 1;
  auto load_a = [&](Rows& v, int c) {
    int o = at_chunk(c);
    if (TAIL && o + 2 * kStep * kh >= rowb) o -= 2 * kStep * kh;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int s = 0; s < 2; ++s) v.a[m][s] = ld16(pa[m] + o + kStep * s);
  };
  auto load_b = [&](int c) {
    const int o = at_chunk(c);
#pragma unroll
    for (int j = 0; j < BL; ++j) {
      const bool in = !TAIL || o + 16 * (tid & 15) < rowb;
#pragma unroll
      for (int q = 0; q < NP; ++q) {
        bb[q][j] = ld16(pb[q][j] + (in ? o : 0));
        if (!in) bb[q][j] = zero;
      }
    }
  };
  auto put_b = [&](int c) {
#pragma unroll
    for (int j = 0; j < BL; ++j)
#pragma unroll
      for (int q = 0; q < NP; ++q)
        if (puts) st16(lds + ((c & 1) * NP + q) * PLANE + at[j], bb[q][j]);
    __syncthreads();
  };
  Acc acc[2][NG];
  clear(acc);
  // chunk c: the next one's staged rows and the weights of the one after it are asked for first
  auto step = [&](const Rows& cur, Rows& fill, int c) {
    if (c + 1 < nc) load_b(c + 1);
    if (c + 2 < nc) load_a(fill, c + 2);
    const char* st = lds + (c & 1) * NP * PLANE;
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const int r = 16 * g + wr, o = r * kSeg + (((4 * (2 * kh + s) + q4) ^ (r & 15)) << 4);
#pragma unroll
        for (int q = 0; q < NP; ++q) {
          const uint4 b = ld16(st + q * PLANE + o);
          mma16x16(acc[0][g], cur.a[0][s], b, T());
          mma16x16(acc[1][g], cur.a[1][s], b, T());
        }
      }
    if (c + 1 < nc) put_b(c + 1);
  };
  Rows a0, a1, a2;
  load_b(0);
  load_a(a0, 0);
  if (nc > 1) load_a(a1, 1);
  put_b(0);
  for (int c = 0; c < nc; c += 3) {
    step(a0, a2, c);
    if (c + 1 < nc) step(a1, a0, c + 1);
    if (c + 2 < nc) step(a2, a1, c + 2);
  }
  __syncthreads();   // the stages are free
  Acc* sums = reinterpret_cast<Acc*>(lds) + rg * 2 * NG * 64 + lane;
  static_assert(4 * 2 * NG * 64 * 16 <= heavy_lds(NG, 1), "the sums fit the stages");
  if (kh == 1) {
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int g = 0; g < NG; ++g) sums[(m * NG + g) * 64] = acc[m][g];
  }
  __syncthreads();
  if (kh == 0) {
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int g = 0; g < NG; ++g) acc[m][g] += sums[(m * NG + g) * 64];
    // rows 4 q4 .. + 3 of the tile, column wr
    if constexpr (DOWN) {
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const int h = r0 + 32 * rg + 16 * m + 4 * q4;
        float4 sd = make_float4(1.f, 1.f, 1.f, 1.f);
        if constexpr (ES == 1) sd = ld4f(p.sd + (size_t)e * p.H + h);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const int c = 16 * g + wr;
          if (c < cnt) {
            const float hs = ES == 1 ? p.hs[base + c] : 1.f;
            *reinterpret_cast<float4*>(p.oh + (size_t)(base + c) * p.H + h) =
                make_float4((float)acc[m][g][0] * (hs * sd.x), (float)acc[m][g][1] * (hs * sd.y),
                            (float)acc[m][g][2] * (hs * sd.z), (float)acc[m][g][3] * (hs * sd.w));
          }
        }
      }
    } else {
      const int f = r0 + 16 * rg + 4 * q4;
      float4 sg = {}, su = {};
      if constexpr (ES == 1) {
        sg = ld4f(p.sg + (size_t)e * p.F + f);
        su = ld4f(p.su + (size_t)e * p.F + f);
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const int c = 16 * g + wr;
        if (c < cnt) store_h<T>(p, base + c, stok[base + c], swt[base + c], f, acc[0][g], acc[1][g], sg, su);
      }
    }
  }
  __syncthreads();   // the next task's stages
}

template <class T>
__global__ __launch_bounds__(kGW * 64, 4) void k_few_gateup(FewParams p) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int tid = threadIdx.x, n = p.T * p.k;
  const FewRoute R(smem + few_red_bytes(p.T), p.El, n);
  few_route<kGW>(R, p);
  const int nact = R.cls[kClasses], heavy = R.cls[2];   // more than 8 tokens
  if (blockIdx.x == 0) {   // the routing for k_few_down
    if (tid <= kClasses) p.r_cls[tid] = R.cls[tid];
    if (tid == 0) p.r_cls[kClasses + 1] = R.off[p.El];
    for (int i = tid; i < nact; i += kGW * 64) p.r_ent[i] = R.ent[i];
    for (int i = tid; i < n; i += kGW * 64) p.r_tok[i] = i < R.off[p.El] ? R.stok[i] : 0;
  }
  static_assert(kGW == 8, "heavy_task");
  const int nh = p.F / 64, ntask = heavy * nh;
  for (int task = blockIdx.x; task < ntask; task += gridDim.x) {
    const int a = task / nh, f0 = (task - a * nh) * 64;
    const int4 x = uniform4(R.ent[a]);
    if (x.z <= 16) heavy_task<T, 1, false>(p, R.stok, R.swt, smem, x.x, x.y, x.z, f0);
    else if (x.z <= 32) heavy_task<T, 2, false>(p, R.stok, R.swt, smem, x.x, x.y, x.z, f0);
    else heavy_task<T, 4, false>(p, R.stok, R.swt, smem, x.x, x.y, x.z, f0);
  }
  // Consecutive units go to different workgroups: a few units still spread over all CUs. Where the waves
  // outnumber the units, two or four share a unit, so that more of its loads are in flight at once.
  typedef typename Mma4<T>::Acc Acc;
  // rows of a unit of an expert with 3 to 8 tokens; of 8 rows of 8-bit weights the scales and sums spill (68 -> 83 us
  // for 32 tokens of 128 experts of 2048 x 768)
  constexpr int WF = sizeof(T) == 1 ? 4 : 8, WQ = WF / 4;
  const int few = R.cls[4], wide_units = (few - heavy) * (p.F / WF), units = wide_units + (nact - few) * (p.F / 4);
  const int w = eng::wave_id(), waves = kGW * gridDim.x, ks = 4 * units <= waves ? 4 : 2 * units <= waves ? 2 : 1;
  // unit u: of an expert with 3 to 8 tokens, then of one with 1 or 2
  auto find = [&](int u, int& f0) {
    const bool wide = u < wide_units;
    const int v = wide ? u : u - wide_units, nf = p.F / (wide ? WF : 4), a = v / nf;
    f0 = (v - a * nf) * (wide ? WF : 4);
    return uniform4(R.ent[(wide ? heavy : few) + a]);
  };
  auto light = [&](int u) {
    int f0;
    const int4 x = find(u, f0);
    if (x.z > 4) gateup_unit<T, WQ, 2, false>(p, R, nullptr, x.x, x.y, x.z, f0, 1, 0);
    else if (WQ > 1 && x.z > 2) gateup_unit<T, WQ, 1, false>(p, R, nullptr, x.x, x.y, x.z, f0, 1, 0);
    else gateup_unit<T, 1, 1, false>(p, R, nullptr, x.x, x.y, x.z, f0, 1, 0);
  };
  if (ks == 1) {
    // A heavy task costs one to two rounds of units: the workgroups without one take a round ahead of the others, or
    // two where these hold all units. 48 skewed tokens of 64 experts, 4096 x 1536 (240 tasks, 2.9 rounds on 512
    // workgroups), none/one/two/three ahead: 200/197/206/220 us; 64 of 128, 2048 x 768 (192 tasks, one round)
    // 67/57/54/54 us.
    const int nb = gridDim.x, hb = ntask % nb, ahead = hb == 0 ? 0 : units > 2 * kGW * (nb - hb) ? 1 : 2;
    if ((int)blockIdx.x >= hb)
      for (int r = 0; r < ahead; ++r) {
        const int u = (r * kGW + w) * (nb - hb) + blockIdx.x - hb;
        if (u < units) light(u);
      }
    for (int u = ahead * kGW * (nb - hb) + w * nb + blockIdx.x; u < units; u += waves) light(u);
  } else {   // one round; a heavy task's last barrier is behind its reads of smem
    const int kp = w & (ks - 1), u = (w / ks) * gridDim.x + blockIdx.x;
    Acc* red = reinterpret_cast<Acc*>(smem) + 32 * w;
    int4 x = make_int4(0, 0, 0, 0);
    int f0 = 0;
    if (u < units) {
      x = find(u, f0);
      if (x.z > 4) gateup_unit<T, WQ, 2, true>(p, R, red, x.x, x.y, x.z, f0, ks, kp);
      else if (WQ > 1 && x.z > 2) gateup_unit<T, WQ, 1, true>(p, R, red, x.x, x.y, x.z, f0, ks, kp);
      else gateup_unit<T, 1, 1, true>(p, R, red, x.x, x.y, x.z, f0, ks, kp);
    }
    __syncthreads();
    if (u < units && kp == 0) {
      if (x.z > 2) gateup_join<T, WQ>(p, R, red, x.x, x.y, x.z, f0, ks);
      else gateup_join<T, 1>(p, R, red, x.x, x.y, x.z, f0, ks);
    }
  }
}

// ------------------------------------------------------------------------------------------------
// Rows h0 .. h0 + 4 NQ - 1 of W_down for the experts ent[0 .. na) of one class (up to 4 NS pairs each),
// segments [c, end) of their (expert, 256-byte segment) axis, S segments an expert; added to the wave's
// sums ya [T][4 NQ]. The stages of U segments run through expert boundaries: the next stage's loads, of
// weights and h, are in flight while the current one is multiplied (DB; without it the registers of the
// second stage would spill).
// FLY (8-bit weights): h is fp32 and quantised here, with the pairs' maxima hm.
template <class T, int NQ, int NS, int U, bool DB, bool FLY>
__device__ __forceinline__ void down_stream(const FewParams& p, const int4* ent, const int* stok, const unsigned* hm,
                                            float* ya, int h0, int S, int c, int end) {
  typedef typename Mma4<T>::Acc Acc;
  constexpr int ES = sizeof(T), NB = FLY ? 4 : ES == 2 ? 2 : 1;   // 16-byte pieces of h a lane loads
  static_assert(!FLY || (NS == 1 && ES == 1 && U == 1), "quantising on the fly");
  const int lane = threadIdx.x & 63, j = lane & 3, blk = lane >> 2, piece = 16 * blk;
  const int q4 = min(blk, NQ - 1);   // lane (blk, j) adds rows 4 q4 .. 4 q4 + 3 of token j
  const size_t rowb = (size_t)p.F * ES;
  if (c >= end) return;
  struct Stage {
    uint4 a[NQ][U], b[NS][U][NB];
    bool in;      // 8-bit: the row has this lane's piece of the last segment (else the row's first piece is in a and b)
    int4 x;       // its expert
    int n;        // segments in it
    bool last;    // the wave's last of this expert
  };
  int a = c / S, s = c - a * S;
  auto load = [&](Stage& v) {   // the stage at (a, s), and on to the next
    v.x = uniform4(ent[a]);
    v.n = min(min(U, S - s), end - c);
    const char* pw = static_cast<const char*>(p.wd) + ((size_t)v.x.x * p.H + h0 + j) * rowb + piece;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      int o = min(s + i, s + v.n - 1) * kSeg;
      v.in = ES > 1 || o + piece < (int)rowb;
      if (!v.in) o = -piece;
#pragma unroll
      for (int q = 0; q < NQ; ++q) v.a[q][i] = ld16_nt(pw + (ptrdiff_t)(4 * q) * (ptrdiff_t)rowb + o);
#pragma unroll
      for (int t = 0; t < NS; ++t) {
        const size_t pos = v.x.y + min(4 * t + j, v.x.z - 1);
        if constexpr (FLY) {
          const float* ph = static_cast<const float*>(p.h) + pos * p.F + (o + piece);
#pragma unroll
          for (int r = 0; r < 4; ++r) v.b[t][i][r] = ld16(ph + 4 * r);
        } else if constexpr (ES == 1) {
          v.b[t][i][0] = ld16(p.hq + pos * rowb + (o + piece));
        } else {
          v.b[t][i][0] = ld16(static_cast<const char*>(p.h) + pos * rowb + o + piece);
          if constexpr (ES == 2) v.b[t][i][1] = ld16(static_cast<const char*>(p.hlo) + pos * rowb + o + piece);
        }
      }
    }
    s += v.n;
    c += v.n;
    v.last = s == S || c == end;
    if (s == S) {
      s = 0;
      ++a;
    }
  };
  Acc acc[NQ][NS];
  clear(acc);
  auto use = [&](const Stage& v) {
    const int base = v.x.y, cnt = v.x.z;
    Q8Row qr;
    if constexpr (FLY) qr = Q8Row(hm[base + min(j, cnt - 1)]);
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (i < v.n)
#pragma unroll
        for (int t = 0; t < NS; ++t) {
          uint4 b = v.b[t][i][0];   // 8-bit: of a missing piece, zero (only the last segment can miss any)
          if constexpr (FLY) {
            float f[16];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              f[4 * r] = __uint_as_float(v.b[t][i][r].x);
              f[4 * r + 1] = __uint_as_float(v.b[t][i][r].y);
              f[4 * r + 2] = __uint_as_float(v.b[t][i][r].z);
              f[4 * r + 3] = __uint_as_float(v.b[t][i][r].w);
            }
            unsigned o[4];
            q8_pack<true>(f, qr, o);
            b = make_uint4(o[0], o[1], o[2], o[3]);
          }
          if constexpr (ES == 1)
            if (i == v.n - 1 && !v.in) b = make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            Mma4<T>::go(acc[q][t], v.a[q][i], b);
            if constexpr (ES == 2) Mma4<T>::go(acc[q][t], v.a[q][i], v.b[t][i][NB - 1]);
          }
        }
    if (!v.last) return;
    float4 sd = make_float4(1.f, 1.f, 1.f, 1.f);
    if constexpr (ES == 1) sd = ld4f(p.sd + (size_t)v.x.x * p.H + h0 + 4 * q4);
#pragma unroll
    for (int t = 0; t < NS; ++t) {
      float r[4] = {};
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float sum = (float)block_sum(acc[q][t][i]);
          r[i] = q == q4 ? sum : r[i];
        }
      if (blk < NQ && 4 * t + j < cnt) {
        if constexpr (ES == 1) {
          const float hs = FLY ? qr.scale : p.hs[base + 4 * t + j];
          r[0] *= hs * sd.x;
          r[1] *= hs * sd.y;
          r[2] *= hs * sd.z;
          r[3] *= hs * sd.w;
        }
        float4* y = reinterpret_cast<float4*>(ya + (stok[base + 4 * t + j] * NQ + blk) * 4);
        const float4 o = *y;
        *y = make_float4(o.x + r[0], o.y + r[1], o.z + r[2], o.w + r[3]);
      }
    }
    clear(acc);
  };
  Stage u;
  if constexpr (!DB) {
    while (c < end) {
      load(u);
      use(u);
    }
    return;
  }
  Stage v;
  load(u);
  for (;;) {
    const bool more = c < end;
    if (more) load(v);
    use(u);
    if (!more) break;
    const bool more2 = c < end;
    if (more2) load(u);
    use(v);
    if (!more2) break;
  }
}

// Whether k_few_heavy takes the down products of the experts of more than 8 tokens ahead of k_few_down: of 9 to 16
// tokens only where k_few_down's 16 rows a wave leave no registers for 16 tokens. 16 tokens on 8 experts of 4096 x
// 1536: 33 us in two kernels, 48 in one (on 16 x 16 tiles); 12 skewed tokens of 128 experts of 2048 x 768: 35 and 30.
__host__ __device__ inline bool heavy_ahead(const FewParams& p) { return p.T > 16 || (p.T > 8 && p.H >= kDown4); }

// FLY (8-bit weights, up to 4 tokens): h is quantised where it is read, with the maxima the gate/up kernel left;
// otherwise the quantiser has run between the two.
template <class T, int NQ, bool FLY>
__global__ __launch_bounds__(kDW * 64, 4) void k_few_down(FewParams p) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  constexpr int NR = 4 * NQ, ES = sizeof(T);
  const int tid = threadIdx.x, w = eng::wave_id(), h0 = blockIdx.x * NR, n = p.T * p.k;
  float* ya = reinterpret_cast<float*>(smem);   // [kDW][T][NR]
  int4* ent = reinterpret_cast<int4*>(ya + kDW * p.T * NR);
  int* stok = reinterpret_cast<int*>(ent + min(n, p.El));
  unsigned* hm = reinterpret_cast<unsigned*>(stok + n);
  int cls[kClasses + 1];
#pragma unroll
  for (int q = 0; q <= kClasses; ++q) cls[q] = __builtin_amdgcn_readfirstlane(p.r_cls[q]);
  for (int i = tid; i < kDW * p.T * NR; i += kDW * 64) ya[i] = 0.f;
  for (int i = tid; i < min(n, p.El); i += kDW * 64) ent[i] = p.r_ent[i];   // entries past the last are not used
  for (int i = tid; i < n; i += kDW * 64) stok[i] = p.r_tok[i];
  if constexpr (FLY) {   // each pair's largest |h|, a wave a pair
    const int lane = tid & 63, nf = p.F / 4;
    for (int i = w; i < p.r_cls[kClasses + 1]; i += kDW) {
      unsigned m = 0u;
      for (int f = lane; f < nf; f += 64) m = max(m, p.hmax[(size_t)i * nf + f]);
      m = wave_max_u32(m);
      if (lane == 0) hm[i] = m;
    }
  }
  __syncthreads();
  const int S = (p.F * ES + kSeg - 1) / kSeg;
  float* mine = ya + w * p.T * NR;
  // class by class, the waves sharing each class's (expert, segment) axis
  auto part = [&](int q, int q1, int& c, int& end) {
    const int64_t N = (int64_t)(cls[q1] - cls[q]) * S;
    c = (int)(w * N / kDW);
    end = (int)((w + 1) * N / kDW);
  };
  int c, end;
  if constexpr (!FLY) {
    // heavy experts: k_few_heavy's products, a wave an expert (whose pairs are of different tokens)
    const int done = heavy_ahead(p) ? cls[2] : 0;
    for (int a = w; a < done; a += kDW) {
      const int4 x = uniform4(ent[a]);
      for (int i = tid & 63; i < x.z * NQ; i += 64) {   // (pair, 4 rows)
        const int c = i / NQ, q = i % NQ;
        const float4 o = *reinterpret_cast<const float4*>(p.oh + (size_t)(x.y + c) * p.H + h0 + 4 * q);
        float4* y = reinterpret_cast<float4*>(mine + (stok[x.y + c] * NQ + q) * 4);
        const float4 v = *y;
        *y = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
      }
    }
    if constexpr (NQ < 4) {
      if (!done) {
        part(1, 2, c, end);
        down_stream<T, NQ, 4, 1, ES == 1 || NQ == 1, false>(p, ent + cls[1], stok, hm, mine, h0, S, c, end);
      }
    }
    part(2, 3, c, end);
    down_stream<T, NQ, 2, 1, ES != 2 || NQ < 4, false>(p, ent + cls[2], stok, hm, mine, h0, S, c, end);
  }
  part(3, 5, c, end);
  down_stream<T, NQ, 1, FLY || NQ == 4 ? 1 : ES == 1 ? 3 : 2, !FLY, FLY>(p, ent + cls[3], stok, hm, mine, h0, S, c, end);
  __syncthreads();
  for (int i = tid; i < p.T * NR; i += kDW * 64) {
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < kDW; ++v) s += ya[v * p.T * NR + i];
    const size_t at = (size_t)(i / NR) * p.H + h0 + i % NR;
    if constexpr (ES == 4) static_cast<float*>(p.y)[at] = s;
    else static_cast<bf16*>(p.y)[at] = (bf16)s;
  }
}

// the down products of the heavy experts, into oh: 64 tokens on 8 experts, 4096 x 1536, 36 us (101 MB of weights).
// Its 128 registers, for two workgroups a CU, leave 4 values of the bf16 form and one of the 8-bit form in scratch.
template <class T>
__global__ __launch_bounds__(512, 4) void k_few_heavy(FewParams p) {
  __shared__ __attribute__((aligned(16))) char smem[heavy_lds(4, sizeof(T) == 2 ? 2 : 1)];
  const int heavy = __builtin_amdgcn_readfirstlane(p.r_cls[2]), nh = p.H / 128;
  for (int task = blockIdx.x; task < heavy * nh; task += gridDim.x) {
    const int a = task / nh;
    const int4 x = uniform4(p.r_ent[a]);
    if (x.z <= 16) heavy_task<T, 1, true>(p, nullptr, nullptr, smem, x.x, x.y, x.z, (task - a * nh) * 128);
    else if (x.z <= 32) heavy_task<T, 2, true>(p, nullptr, nullptr, smem, x.x, x.y, x.z, (task - a * nh) * 128);
    else heavy_task<T, 4, true>(p, nullptr, nullptr, smem, x.x, x.y, x.z, (task - a * nh) * 128);
  }
}

// ------------------------------------------------------------------------------------------------
// router projection: experts e0 .. e0 + 3 for tokens t0 .. t0 + 4 NS - 1, the waves splitting H. Bound by its launch:
// 128 experts x 2048, 4 us for one token, 4.7 for 8.
template <class T, int NS>
__device__ __forceinline__ void router_tile(const FewParams& p, float* red, int e0, int t0) {
  const int tid = threadIdx.x, lane = tid & 63, w = eng::wave_id(), j = lane & 3;
  const size_t rowb = (size_t)p.H * sizeof(T), piece = 16 * (lane >> 2);
  const char* pw[1] = {static_cast<const char*>(p.wr) + min(e0 + j, p.E - 1) * rowb + piece};
  const char* px[NS];
#pragma unroll
  for (int t = 0; t < NS; ++t)
    px[t] = static_cast<const char*>(p.x0) + min(t0 + 4 * t + j, p.T - 1) * rowb + piece;
  const int S = (int)(rowb / kSeg);
  f32x4 acc[1][NS];
  clear(acc);
  dot4<T, 1, NS, NS == 4 ? 1 : 2>(pw, px, w * S / kPW, (w + 1) * S / kPW, acc);
#pragma unroll
  for (int t = 0; t < NS; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float s = block_sum(acc[0][t][i]);
      if (lane < 4) red[(w * NS * 4 + 4 * t + j) * 4 + i] = s;   // [wave][token][expert]
    }
  __syncthreads();
  if (tid < 16 * NS) {
    const int t = t0 + tid / 4, e = e0 + tid % 4;
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < kPW; ++v) s += red[v * NS * 16 + tid];
    if (t < p.T && e < p.E) p.logits[(size_t)t * p.E + e] = s;
  }
}

template <class T>
__global__ __launch_bounds__(kPW * 64, 4) void k_few_prep(FewParams p, int router_blocks) {
  __shared__ float smem[kPW * 16 * kSets];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  if ((int)blockIdx.x < router_blocks) {
    const int ne = (p.E + 3) / 4, e0 = 4 * (blockIdx.x % ne), t0 = 4 * kSets * (blockIdx.x / ne);
    if (p.T - t0 <= 4) router_tile<T, 1>(p, smem, e0, t0);
    else if (p.T - t0 <= 8) router_tile<T, 2>(p, smem, e0, t0);
    else router_tile<T, kSets>(p, smem, e0, t0);
    return;
  }
  if constexpr (sizeof(T) == 2) {   // with 8-bit weights: quantise row t of x
    const int t = blockIdx.x - router_blocks;
    if (t >= p.T) {   // a token's experts by each wave
      const int c = (t - p.T) * kPW + w;
      if (c < p.T) choose_store(p, c, lane);
      return;
    }
    unsigned* sm = reinterpret_cast<unsigned*>(smem);
    const bf16* row = static_cast<const bf16*>(p.x0) + (size_t)t * p.H;
    unsigned m = 0u;
    for (int c = tid; c < p.H / 8; c += kPW * 64) {
      float v[8];
      eng::unpack8(ld16(row + 8 * c), v);
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, mag_bits(v[i]));
    }
    m = wave_max_u32(m);
    if (lane == 0) sm[w] = m;
    __syncthreads();
    m = 0u;
#pragma unroll
    for (int v = 0; v < kPW; ++v) m = max(m, sm[v]);
    const Q8Row r(m);
    for (int c = tid; c < p.H / 8; c += kPW * 64) {
      float v[8];
      unsigned q[2];
      eng::unpack8(ld16(row + 8 * c), v);
      q8_pack<false>(v, r, q);
      *reinterpret_cast<uint2*>(p.xq + (size_t)t * p.H + 8 * c) = make_uint2(q[0], q[1]);
    }
    if (tid == 0) p.xs[t] = r.scale;
  }
}

bool topk_in_prep(const FewParams& p, bool quant) { return quant && !p.wr && p.T > kRouteHere; }

template <class T>
hipError_t launch_prep(const FewParams& p, hipStream_t s, bool quant) {
  const int nr = p.wr ? (p.E + 3) / 4 * ((p.T + 4 * kSets - 1) / (4 * kSets)) : 0;
  if (nr == 0 && !quant) return hipSuccess;
  // rows to quantise and, with given logits, the choice of experts: one launch for both (4.5 us of 114 at 32 tokens)
  const int nq = quant ? p.T + (topk_in_prep(p, quant) ? (p.T + kPW - 1) / kPW : 0) : 0;
  prof_mark_begin("few_prep", s);
  k_few_prep<T><<<nr + nq, kPW * 64, 0, s>>>(p, nr);
  const hipError_t err = hipGetLastError();
  if (err == hipSuccess) prof_mark_end(s);
  return err;
}

template <class T, int NQ, bool FLY>
hipError_t launch_down(const FewParams& p, hipStream_t s) {
  const size_t n = (size_t)p.T * p.k, lds = kDW * p.T * 16 * NQ + std::min<size_t>(n, p.El) * 16 + n * (FLY ? 8 : 4);
  hipError_t err;
  if (lds > 65536 && (err = hipFuncSetAttribute(reinterpret_cast<const void*>(k_few_down<T, NQ, FLY>),
                                                hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds)) != hipSuccess)
    return err;
  prof_mark_begin("few_down", s);
  k_few_down<T, NQ, FLY><<<p.H / (4 * NQ), kDW * 64, lds, s>>>(p);
  if ((err = hipGetLastError()) != hipSuccess) return err;
  prof_mark_end(s);
  return hipSuccess;
}

template <class T, bool FLY = false>
hipError_t launch_layer(const FewParams& p, hipStream_t s) {
  const int n = p.T * p.k, units = std::min(n, p.El) * (p.F / 4);
  const int grid = std::min(units, persistent_grid(2));
  hipError_t err;
  if (p.T > kRouteHere && !topk_in_prep(p, sizeof(T) == 1)) {
    prof_mark_begin("few_topk", s);
    k_few_topk<<<p.T, 64, 0, s>>>(p);
    if ((err = hipGetLastError()) != hipSuccess) return err;
    prof_mark_end(s);
  }
  const size_t lds = few_red_bytes(p.T) + FewRoute::bytes(p.El, n);
  if (lds > 65536 && (err = hipFuncSetAttribute(reinterpret_cast<const void*>(k_few_gateup<T>),
                                                hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds)) != hipSuccess)
    return err;
  prof_mark_begin("few_gateup", s);
  k_few_gateup<T><<<grid, kGW * 64, lds, s>>>(p);
  if ((err = hipGetLastError()) != hipSuccess) return err;
  prof_mark_end(s);
  if (sizeof(T) == 1 && !FLY &&
      (err = launch_int8_quant(p.h, true, n, p.F, p.r_cls + kClasses + 1, p.hq, p.hs, "int8_quant_h", s)) != hipSuccess)
    return err;
  if (!FLY && heavy_ahead(p)) {
    prof_mark_begin("few_heavy", s);
    k_few_heavy<T><<<std::min(std::max(1, n / 9) * (p.H / 128), persistent_grid(2)), 512, 0, s>>>(p);
    if ((err = hipGetLastError()) != hipSuccess) return err;
    prof_mark_end(s);
  }
  // as many rows per workgroup (each read of h serves them all) as leave each of 256 CUs one at H = 2048 and 4096, the
  // widths measured; between them the last round of workgroups is part empty. Half as many: 64 tokens of 128 experts,
  // 4096 x 1536 281 -> 370 us, 2048 x 768 102 -> 145; one token 23 -> 25 and 11.5 -> 15.
  if (p.H >= kDown4) return launch_down<T, 4, FLY>(p, s);
  return p.H >= 2048 ? launch_down<T, 2, FLY>(p, s) : launch_down<T, 1, FLY>(p, s);
}

}  // namespace

hipError_t launch_few(const FewParams& p, int type, hipStream_t s) {
  hipError_t err;
  if (type == 4) return (err = launch_prep<float>(p, s, false)) != hipSuccess ? err : launch_layer<float>(p, s);
  if (type == 2) return (err = launch_prep<bf16>(p, s, false)) != hipSuccess ? err : launch_layer<bf16>(p, s);
  if ((err = launch_prep<bf16>(p, s, true)) != hipSuccess) return err;
  return p.hmax ? launch_layer<int8_t, true>(p, s) : launch_layer<int8_t>(p, s);
}

}  // namespace moe
