// The whole layer for a few tokens (T <= 64), forward only, in bf16, fp32 or with 8-bit weights.
//
// At a few tokens the layer reads the weights of the experts that were chosen, once, and does little
// else: 6 H F flops against 3 H F elements per pair. These kernels are built to keep those reads in
// flight on every CU, with the arithmetic on MFMA tiles whose 16 columns are an expert's tokens.
//
//   k_few_prep    logits = x W_r^T (16 experts per workgroup) and, with 8-bit weights, the quantised rows
//                 of x. Only launched where one of the two is asked for.
//   k_few_gateup  every workgroup routes the tokens for itself (a few hundred cycles), then takes
//                 (expert, 16 rows of F) tasks: both weights' rows times the expert's tokens, split
//                 along H over the waves, h = w silu(a) b into the workspace.
//   k_few_down    a workgroup owns 16 rows of H for every expert: its waves share the (expert, F) axis,
//                 each keeping its own sum per token, and the sums are added in a fixed order. No
//                 partial sums in memory, no atomics on sums: repeated calls give the same bits.
//
// h is kept in fp32's accuracy: as fp32, or in bf16 mode as the pair hi = bf16(h), lo = bf16(h - hi),
// whose two products cost matrix time that a read-bound kernel does not miss.
#include <math.h>

#include <algorithm>

#include "engine.h"
#include "int8_device.h"
#include "moe_internal.h"
#include "route_device.h"

namespace moe {
namespace {

constexpr int kGW = 8;      // waves of k_few_gateup
constexpr int kDW = 16;     // waves of k_few_down and k_few_prep
constexpr int kStep = 64;   // bytes of one weight row per MFMA step

template <class T> struct Mma;   // one 16x16 MFMA step over 64 bytes of contraction
template <> struct Mma<bf16> {
  typedef f32x4 Acc;
  typedef float Sum;
  static __device__ __forceinline__ void go(Acc& c, const uint4& a, const uint4& b) { mma16<bf16>(c, a, b); }
};
template <> struct Mma<float> {
  typedef f32x4 Acc;
  typedef float Sum;
  static __device__ __forceinline__ void go(Acc& c, const uint4& a, const uint4& b) { mma16<float>(c, a, b); }
};
template <> struct Mma<int8_t> {
  typedef i32x4 Acc;
  typedef int Sum;
  static __device__ __forceinline__ void go(Acc& c, const uint4& a, const uint4& b) {
    c = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
  }
};

// ------------------------------------------------------------------------------------------------
// routing of the few tokens inside a workgroup

// the k best experts of a token by one wave: lane j < k ends with the j-th key
__device__ __forceinline__ unsigned long long wave_topk(const float* row, int E, int k, int lane) {
  unsigned long long key[kMaxExperts / 64], mine = 0ull;
  const int per = (E + 63) >> 6;
#pragma unroll
  for (int i = 0; i < kMaxExperts / 64; ++i) {
    const int e = lane + 64 * i;
    key[i] = i < per && e < E ? topk_key(row[e], e) : 0ull;
  }
  for (int j = 0; j < k; ++j) {
    unsigned long long b = key[0];
#pragma unroll
    for (int i = 1; i < kMaxExperts / 64; ++i)
      if (i < per) b = key[i] > b ? key[i] : b;
    auto step = [&](unsigned long long o) { b = o > b ? o : b; };
    step(((unsigned long long)dpp_mov<kDppXor1>((unsigned)(b >> 32)) << 32) | dpp_mov<kDppXor1>((unsigned)b));
    step(((unsigned long long)dpp_mov<kDppXor2>((unsigned)(b >> 32)) << 32) | dpp_mov<kDppXor2>((unsigned)b));
    step(((unsigned long long)dpp_mov<kDppHalfMirror>((unsigned)(b >> 32)) << 32) | dpp_mov<kDppHalfMirror>((unsigned)b));
    step(((unsigned long long)dpp_mov<kDppMirror>((unsigned)(b >> 32)) << 32) | dpp_mov<kDppMirror>((unsigned)b));
    unsigned long long best = 0ull;
#pragma unroll
    for (int q = 0; q < 4; ++q) {   // one lane of each 16-lane row
      const unsigned long long o = ((unsigned long long)(unsigned)__builtin_amdgcn_readlane((int)(b >> 32), 16 * q) << 32) |
                                   (unsigned)__builtin_amdgcn_readlane((int)b, 16 * q);
      best = o > best ? o : best;
    }
    if (lane == j) mine = best;
#pragma unroll
    for (int i = 0; i < kMaxExperts / 64; ++i) key[i] = key[i] == best ? 0ull : key[i];
  }
  return mine;
}

// The routing of all T tokens in a workgroup's LDS, pairs sorted by (local expert, token).
struct FewRoute {
  unsigned long long* mask;   // [El] tokens that chose the expert
  int* off;                   // [El + 1] first pair of each expert
  int* act;                   // [El] experts with pairs, ascending; nact of them
  int* nact;                  // [1]
  int* el;                    // [T k] local expert of pair t k + j, -1: not local
  float* wt;                  // [T k] its weight
  int* stok;                  // [T k] token of sorted pair p
  float* swt;                 // [T k] its weight
  static __host__ __device__ size_t bytes(int El, int n) {
    return (size_t)El * 8 + (size_t)(El + 1) * 4 + (size_t)El * 4 + 4 + (size_t)n * 16;
  }
  __device__ __forceinline__ FewRoute(char* s, int El, int n) {
    mask = reinterpret_cast<unsigned long long*>(s);
    off = reinterpret_cast<int*>(mask + El);
    act = off + El + 1;
    nact = act + El;
    el = nact + 1;
    wt = reinterpret_cast<float*>(el + n);
    stok = reinterpret_cast<int*>(wt + n);
    swt = reinterpret_cast<float*>(stok + n);
  }
};

template <int NW>
__device__ __forceinline__ void few_route(const FewRoute& R, const FewParams& p) {
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, n = p.T * p.k;
  for (int e = tid; e < p.El; e += NW * 64) R.mask[e] = 0ull;
  __syncthreads();
  for (int t = w; t < p.T; t += NW) {
    const unsigned long long key = wave_topk(p.logits + (size_t)t * p.E, p.E, p.k, lane);
    const float v = key_value(key);
    const float top = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 0));
    const float z = lane < p.k ? expf(v - top) : 0.f;
    float s = 0.f;   // summed in slot order
    for (int j = 0; j < p.k; ++j) s += __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(z), j));
    if (lane < p.k) {
      const int e = key_expert(key) - p.e0;
      const bool here = e >= 0 && e < p.El;
      R.el[t * p.k + lane] = here ? e : -1;
      R.wt[t * p.k + lane] = z / s;
      if (here) atomicOr(&R.mask[e], 1ull << t);
    }
  }
  __syncthreads();
  if (w == 0) {   // lane's experts: a contiguous run
    const int per = (p.El + 63) >> 6, e0 = lane * per;
    int c = 0, a = 0;
    for (int i = 0; i < per; ++i) {
      const int m = e0 + i < p.El ? __popcll(R.mask[e0 + i]) : 0;
      c += m;
      a += m > 0;
    }
    int ic = c, ia = a;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int nc = __shfl_up(ic, d), na = __shfl_up(ia, d);
      if (lane >= d) {
        ic += nc;
        ia += na;
      }
    }
    int o = ic - c, q = ia - a;
    for (int i = 0; i < per; ++i) {
      const int e = e0 + i;
      if (e >= p.El) break;
      const int m = __popcll(R.mask[e]);
      R.off[e] = o;
      if (m > 0) R.act[q++] = e;
      o += m;
    }
    if (lane == 63) {
      R.off[p.El] = ic;
      *R.nact = ia;
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

// ------------------------------------------------------------------------------------------------
// weight rows times tokens: NM weight matrices, NG groups of 16 columns, steps [s0, s1) of 64 bytes.
// U steps' loads are issued before their MFMAs (the last step's again where the run ends inside them).
template <class T, int NM, int NG, int U>
__device__ __forceinline__ void dot_rows(const char* const (&pw)[NM], const char* const (&px)[NG], int s0, int s1,
                                         typename Mma<T>::Acc (&acc)[NM][NG]) {
  for (int s = s0; s < s1; s += U) {
    uint4 a[NM][U], b[NG][U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const size_t o = (size_t)min(s + i, s1 - 1) * kStep;
#pragma unroll
      for (int m = 0; m < NM; ++m) a[m][i] = ld16(pw[m] + o);
#pragma unroll
      for (int g = 0; g < NG; ++g) b[g][i] = ld16(px[g] + o);
    }
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (s + i < s1)
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
          for (int g = 0; g < NG; ++g) Mma<T>::go(acc[m][g], a[m][i], b[g][i]);
  }
}

template <class A, int NM, int NG>
__device__ __forceinline__ void clear(A (&acc)[NM][NG]) {
#pragma unroll
  for (int m = 0; m < NM; ++m)
#pragma unroll
    for (int g = 0; g < NG; ++g) acc[m][g] = A{0, 0, 0, 0};
}

// one (expert e, rows f0 .. f0+15) task of the gate/up products; red: [kGW][2][64] accumulators
template <class T, int NG>
__device__ __forceinline__ void gateup_task(const FewParams& p, const FewRoute& R, char* red_, int e, int f0) {
  typedef typename Mma<T>::Acc Acc;
  constexpr int ES = sizeof(T);
  const int tid = threadIdx.x, lane = tid & 63, w = eng::wave_id();
  const int base = R.off[e], cnt = R.off[e + 1] - base;
  const size_t rowb = (size_t)p.H * ES;
  const size_t wo = ((size_t)e * p.F + f0 + (lane & 15)) * rowb + 16 * (lane >> 4);
  const char* pw[2] = {static_cast<const char*>(p.wg) + wo, static_cast<const char*>(p.wu) + wo};
  const char* px[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g)
    px[g] = static_cast<const char*>(p.x) + R.stok[base + min(16 * g + (lane & 15), cnt - 1)] * rowb + 16 * (lane >> 4);
  const int S = (int)(rowb / kStep);
  Acc acc[2][NG];
  clear(acc);
  dot_rows<T, 2, NG, NG == 4 ? 2 : 4>(pw, px, w * S / kGW, (w + 1) * S / kGW, acc);
  Acc* red = reinterpret_cast<Acc*>(red_);
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    if (16 * g >= cnt) break;
    red[(2 * w) * 64 + lane] = acc[0][g];
    red[(2 * w + 1) * 64 + lane] = acc[1][g];
    __syncthreads();
    // thread i of the first 256: row f0 + i % 16 of column i / 16
    if (tid < 256) {
      const int f = tid & 15, c = 16 * g + (tid >> 4), src = (f >> 2) * 16 + (tid >> 4);
      if (c < cnt) {
        typedef typename Mma<T>::Sum Sum;
        const Sum* rs = reinterpret_cast<const Sum*>(red) + src * 4 + (f & 3);
        Sum sa = rs[0], sb = rs[256];
#pragma unroll
        for (int v = 1; v < kGW; ++v) {
          sa += rs[2 * v * 256];
          sb += rs[(2 * v + 1) * 256];
        }
        const int pos = base + c;
        float a = (float)sa, b = (float)sb;
        if constexpr (ES == 1) {
          const float xs = p.xs[R.stok[pos]];
          a *= xs * p.sg[(size_t)e * p.F + f0 + f];
          b *= xs * p.su[(size_t)e * p.F + f0 + f];
        }
        const float h = R.swt[pos] * (a / (1.0f + expf(-a)) * b);
        const size_t at = (size_t)pos * p.F + f0 + f;
        if constexpr (ES == 2) {
          const bf16 hi = (bf16)h;
          static_cast<bf16*>(p.h)[at] = hi;
          static_cast<bf16*>(p.hlo)[at] = (bf16)(h - (float)hi);
        } else {
          static_cast<float*>(p.h)[at] = h;
        }
        if constexpr (ES == 1) {
          unsigned m = mag_bits(h);   // over the column's 16 rows: one 16-lane row
          m = max(m, dpp_mov<kDppXor1>(m));
          m = max(m, dpp_mov<kDppXor2>(m));
          m = max(m, dpp_mov<kDppHalfMirror>(m));
          m = max(m, dpp_mov<kDppMirror>(m));
          if (f == 0) atomicMax(p.hmax + pos, m);   // a maximum: any order gives the same bits
        }
      }
    }
    __syncthreads();
  }
}

template <class T>
__global__ __launch_bounds__(kGW * 64, 4) void k_few_gateup(FewParams p) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int tid = threadIdx.x, n = p.T * p.k;
  char* red = smem;
  const FewRoute R(smem + kGW * 2 * 64 * 16, p.El, n);
  few_route<kGW>(R, p);
  const int nact = *R.nact;
  if (blockIdx.x == 0) {   // the routing for k_few_down
    for (int i = tid; i <= p.El; i += kGW * 64) p.r_off[i] = R.off[i];
    for (int i = tid; i < nact; i += kGW * 64) p.r_act[i] = R.act[i];
    for (int i = tid; i < R.off[p.El]; i += kGW * 64) p.r_tok[i] = R.stok[i];
    if (tid == 0) *p.r_nact = nact;
  }
  const int nf = p.F / 16, ntask = nact * nf;
  for (int task = blockIdx.x; task < ntask; task += gridDim.x) {
    const int a = task / nf, e = __builtin_amdgcn_readfirstlane(R.act[a]), f0 = (task - a * nf) * 16;
    const int cnt = __builtin_amdgcn_readfirstlane(R.off[e + 1] - R.off[e]);
    if (cnt <= 16) gateup_task<T, 1>(p, R, red, e, f0);
    else if (cnt <= 32) gateup_task<T, 2>(p, R, red, e, f0);
    else gateup_task<T, 4>(p, R, red, e, f0);
  }
}

// ------------------------------------------------------------------------------------------------
// rows h0 .. h0+15 of W_down[e] times the h of pairs base .. base+cnt-1 (cnt <= 16 NG), steps [s0, s1) of 64 bytes of weight row, added to
// the wave's sums ya [T][16]
template <class T, int NG>
__device__ __forceinline__ void down_part(const FewParams& p, const int* stok, float* ya, int e, int base, int cnt,
                                          int h0, int s0, int s1) {
  typedef typename Mma<T>::Acc Acc;
  constexpr int ES = sizeof(T);
  const int lane = threadIdx.x & 63;
  const size_t rowb = (size_t)p.F * ES;
  const char* pw = static_cast<const char*>(p.wd) + ((size_t)e * p.H + h0 + (lane & 15)) * rowb + 16 * (lane >> 4);
  Acc acc[1][NG];
  clear(acc);
  float hs[NG];
  if constexpr (ES == 1) {
    static_assert(NG == 1, "a lane quantises one column's h");
    const int pos = base + min(lane & 15, cnt - 1);
    const Q8Row qr(p.hmax[pos]);
    hs[0] = qr.scale;
    const float* ph = static_cast<const float*>(p.h) + (size_t)pos * p.F + 16 * (lane >> 4);
    constexpr int U = 2;
    for (int s = s0; s < s1; s += U) {
      uint4 a[U];
      float b[U][16];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int si = min(s + i, s1 - 1);
        a[i] = ld16(pw + (size_t)si * kStep);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float4 f = *reinterpret_cast<const float4*>(ph + si * 64 + 4 * v);
          b[i][4 * v] = f.x; b[i][4 * v + 1] = f.y; b[i][4 * v + 2] = f.z; b[i][4 * v + 3] = f.w;
        }
      }
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (s + i < s1) {
          unsigned q[4];
          q8_pack<true>(b[i], qr, q);
          Mma<T>::go(acc[0][0], a[i], make_uint4(q[0], q[1], q[2], q[3]));
        }
    }
  } else {
    const char *ph[NG], *pl[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const size_t o = (size_t)(base + min(16 * g + (lane & 15), cnt - 1)) * rowb + 16 * (lane >> 4);
      ph[g] = static_cast<const char*>(p.h) + o;
      pl[g] = ES == 2 ? static_cast<const char*>(p.hlo) + o : nullptr;
    }
    constexpr int U = NG == 4 ? 2 : 4;
    for (int s = s0; s < s1; s += U) {
      uint4 a[U], b[U][NG], c[U][NG];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const size_t o = (size_t)min(s + i, s1 - 1) * kStep;
        a[i] = ld16(pw + o);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          b[i][g] = ld16(ph[g] + o);
          if constexpr (ES == 2) c[i][g] = ld16(pl[g] + o);
        }
      }
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (s + i < s1)
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            Mma<T>::go(acc[0][g], a[i], b[i][g]);
            if constexpr (ES == 2) Mma<T>::go(acc[0][g], a[i], c[i][g]);
          }
    }
  }
  float4 sd = make_float4(1.f, 1.f, 1.f, 1.f);
  if constexpr (ES == 1) {
    const float* q = p.sd + (size_t)e * p.H + h0 + 4 * (lane >> 4);
    sd = make_float4(q[0], q[1], q[2], q[3]);
  }
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const int c = 16 * g + (lane & 15);
    if (c < cnt) {
      float4* y = reinterpret_cast<float4*>(ya + stok[base + c] * 16 + 4 * (lane >> 4));
      float4 v = *y;
      if constexpr (ES == 1) {
        v.x += (float)acc[0][g][0] * (hs[g] * sd.x);
        v.y += (float)acc[0][g][1] * (hs[g] * sd.y);
        v.z += (float)acc[0][g][2] * (hs[g] * sd.z);
        v.w += (float)acc[0][g][3] * (hs[g] * sd.w);
      } else {
        v.x += acc[0][g][0];
        v.y += acc[0][g][1];
        v.z += acc[0][g][2];
        v.w += acc[0][g][3];
      }
      *y = v;
    }
  }
}

template <class T>
__global__ __launch_bounds__(kDW * 64, 4) void k_few_down(FewParams p) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int tid = threadIdx.x, w = eng::wave_id(), h0 = blockIdx.x * 16;
  float* ya = reinterpret_cast<float*>(smem);   // [kDW][T][16]
  int* off = reinterpret_cast<int*>(ya + kDW * p.T * 16);
  int* act = off + p.El + 1;
  int* stok = act + p.El;
  const int nact = *p.r_nact;
  for (int i = tid; i < kDW * p.T * 16; i += kDW * 64) ya[i] = 0.f;
  for (int i = tid; i <= p.El; i += kDW * 64) off[i] = p.r_off[i];
  for (int i = tid; i < nact; i += kDW * 64) act[i] = p.r_act[i];
  __syncthreads();
  for (int i = tid; i < off[p.El]; i += kDW * 64) stok[i] = p.r_tok[i];
  __syncthreads();
  constexpr int ES = sizeof(T);
  const int S = p.F * ES / kStep, N = nact * S;
  float* mine = ya + w * p.T * 16;
  for (int c = (int)((int64_t)w * N / kDW), end = (int)((int64_t)(w + 1) * N / kDW); c < end;) {
    const int a = c / S, s0 = c - a * S, s1 = min(S, s0 + end - c);
    const int e = __builtin_amdgcn_readfirstlane(act[a]);
    const int base = __builtin_amdgcn_readfirstlane(off[e]), cnt = __builtin_amdgcn_readfirstlane(off[e + 1]) - base;
    if constexpr (ES == 1) {   // more than 16 tokens: the weight rows again, from the caches
      for (int q = 0; q < cnt; q += 16) down_part<T, 1>(p, stok, mine, e, base + q, min(16, cnt - q), h0, s0, s1);
    } else {
      if (cnt <= 16) down_part<T, 1>(p, stok, mine, e, base, cnt, h0, s0, s1);
      else if (cnt <= 32) down_part<T, 2>(p, stok, mine, e, base, cnt, h0, s0, s1);
      else down_part<T, 4>(p, stok, mine, e, base, cnt, h0, s0, s1);
    }
    c += s1 - s0;
  }
  __syncthreads();
  for (int i = tid; i < p.T * 16; i += kDW * 64) {
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < kDW; ++v) s += ya[v * p.T * 16 + i];
    const size_t at = (size_t)(i >> 4) * p.H + h0 + (i & 15);
    if constexpr (ES == 4) static_cast<float*>(p.y)[at] = s;
    else static_cast<bf16*>(p.y)[at] = (bf16)s;
  }
}

// ------------------------------------------------------------------------------------------------
// router projection: experts 16 b .. 16 b + 15 for every token; red: [kDW][64] accumulators per group
template <class T, int NG>
__device__ __forceinline__ void router_tile(const FewParams& p, char* red_) {
  const int tid = threadIdx.x, lane = tid & 63, w = eng::wave_id(), e0 = blockIdx.x * 16;
  const size_t rowb = (size_t)p.H * sizeof(T);
  const char* pw[1] = {static_cast<const char*>(p.wr) + min(e0 + (lane & 15), p.E - 1) * rowb + 16 * (lane >> 4)};
  const char* px[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g)
    px[g] = static_cast<const char*>(p.x0) + min(16 * g + (lane & 15), p.T - 1) * rowb + 16 * (lane >> 4);
  const int S = (int)(rowb / kStep);
  f32x4 acc[1][NG];
  clear(acc);
  dot_rows<T, 1, NG, NG == 4 ? 2 : 4>(pw, px, w * S / kDW, (w + 1) * S / kDW, acc);
  f32x4* red = reinterpret_cast<f32x4*>(red_);
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    red[w * 64 + lane] = acc[0][g];
    __syncthreads();
    if (tid < 256) {
      const int f = tid & 15, t = 16 * g + (tid >> 4), src = (f >> 2) * 16 + (tid >> 4);
      const float* rs = reinterpret_cast<const float*>(red) + src * 4 + (f & 3);
      float s = 0.f;
#pragma unroll
      for (int v = 0; v < kDW; ++v) s += rs[v * 256];
      if (t < p.T && e0 + f < p.E) p.logits[(size_t)t * p.E + e0 + f] = s;
    }
    __syncthreads();
  }
}

template <class T>
__global__ __launch_bounds__(kDW * 64, 4) void k_few_prep(FewParams p, int router_blocks) {
  __shared__ __attribute__((aligned(16))) char smem[kDW * 64 * 16];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  if ((int)blockIdx.x < router_blocks) {
    if (p.T <= 16) router_tile<T, 1>(p, smem);
    else if (p.T <= 32) router_tile<T, 2>(p, smem);
    else router_tile<T, 4>(p, smem);
    return;
  }
  if constexpr (sizeof(T) == 2) {   // with 8-bit weights: quantise row t of x, clear its pairs' maxima
    const int t = blockIdx.x - router_blocks;
    unsigned* sm = reinterpret_cast<unsigned*>(smem);
    for (int j = tid; j < p.k; j += kDW * 64) p.hmax[t * p.k + j] = 0u;
    const bf16* row = static_cast<const bf16*>(p.x0) + (size_t)t * p.H;
    unsigned m = 0u;
    for (int c = tid; c < p.H / 8; c += kDW * 64) {
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
    for (int v = 0; v < kDW; ++v) m = max(m, sm[v]);
    const Q8Row r(m);
    for (int c = tid; c < p.H / 8; c += kDW * 64) {
      float v[8];
      unsigned q[2];
      eng::unpack8(ld16(row + 8 * c), v);
      q8_pack<false>(v, r, q);
      *reinterpret_cast<uint2*>(p.xq + (size_t)t * p.H + 8 * c) = make_uint2(q[0], q[1]);
    }
    if (tid == 0) p.xs[t] = r.scale;
  }
}

template <class T>
hipError_t launch_prep(const FewParams& p, hipStream_t s, bool quant) {
  const int nr = p.wr ? (p.E + 15) / 16 : 0;
  if (nr == 0 && !quant) return hipSuccess;
  prof_mark_begin("few_prep", s);
  k_few_prep<T><<<nr + (quant ? p.T : 0), kDW * 64, 0, s>>>(p, nr);
  const hipError_t err = hipGetLastError();
  if (err == hipSuccess) prof_mark_end(s);
  return err;
}

template <class T>
hipError_t launch_layer(const FewParams& p, hipStream_t s) {
  const int n = p.T * p.k, tasks = std::min(n, p.El) * (p.F / 16);
  const int grid = std::min(tasks, persistent_grid(2));
  const size_t lds_g = (size_t)kGW * 2 * 64 * 16 + FewRoute::bytes(p.El, n);
  const size_t lds_d = (size_t)kDW * p.T * 64 + ((size_t)2 * p.El + 1 + n) * 4;
  hipError_t err;
  if (lds_d > 65536 && (err = hipFuncSetAttribute(reinterpret_cast<const void*>(k_few_down<T>),
                                                  hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds_d)) != hipSuccess)
    return err;
  prof_mark_begin("few_gateup", s);
  k_few_gateup<T><<<grid, kGW * 64, lds_g, s>>>(p);
  if ((err = hipGetLastError()) != hipSuccess) return err;
  prof_mark_end(s);
  prof_mark_begin("few_down", s);
  k_few_down<T><<<p.H / 16, kDW * 64, lds_d, s>>>(p);
  if ((err = hipGetLastError()) != hipSuccess) return err;
  prof_mark_end(s);
  return hipSuccess;
}

}  // namespace

hipError_t launch_few(const FewParams& p, int type, hipStream_t s) {
  hipError_t err;
  if (type == 4) return (err = launch_prep<float>(p, s, false)) != hipSuccess ? err : launch_layer<float>(p, s);
  if (type == 2) return (err = launch_prep<bf16>(p, s, false)) != hipSuccess ? err : launch_layer<bf16>(p, s);
  return (err = launch_prep<bf16>(p, s, true)) != hipSuccess ? err : launch_layer<int8_t>(p, s);
}

}  // namespace moe
