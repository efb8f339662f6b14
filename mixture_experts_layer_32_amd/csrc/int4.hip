// Products with 4-bit weights and a scale for each group of inputs.
//
//   k_int4_pack   a weight's tiles, from fp32 or bf16 (quantised here) or from whole numbers and scales.
//   k_int4_rows   y = sum over groups of s (x q^T): a workgroup takes 16 output channels, its waves split K, and the
//                 weight is read once for up to 64 rows.
// A number q of a weight is held as u = q + 8 in four bits. Put into the upper bits of a bf16's significand they give
// 16 + u exactly with a shift and one and-or for two numbers, and x q = x (16 + u) - 24 x: the matrix instruction that
// multiplies with 16 + u starts from the sum that another one makes with the constant -24.
#include <algorithm>

#include "engine.h"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kTileN = 16, kTileK = 128, kTileBytes4 = 1024;

// Two numbers of each of the four words that a lane holds of a tile, 16 + u in bf16: element 2d in the low half,
// 2d + 1 in the high one.
__device__ __forceinline__ uint4 unpack16(unsigned w) {
  return make_uint4(((w << 3) & 0x00780078u) | 0x41804180u, ((w >> 1) & 0x00780078u) | 0x41804180u,
                    ((w >> 5) & 0x00780078u) | 0x41804180u, ((w >> 9) & 0x00780078u) | 0x41804180u);
}
constexpr unsigned kMinus24 = 0xC1C0C1C0u;   // bf16 -24 twice

__device__ __forceinline__ float bf16_bits(unsigned short b) { return __uint_as_float((unsigned)b << 16); }

// KIND 0: bf16, 1: fp32, 2: signed bytes with bf16 scales. One wavefront per tile; lane 16 h + c takes channel c and
// inputs 32 i + 8 h + j, i < 4, j < 8.
template <int KIND>
__global__ __launch_bounds__(256) void k_int4_pack(const void* __restrict__ in, const uint16_t* __restrict__ sin, int64_t tiles,
                                                   int N, int K, int group, uint8_t* __restrict__ q,
                                                   uint16_t* __restrict__ sout) {
  const int lane = threadIdx.x & 63, c = lane & 15, h = lane >> 4;
  const int Nt = (N + kTileN - 1) / kTileN, Kt = (K + kTileK - 1) / kTileK;
  const int per = group / 32, ng = 4 / per;     // steps of 32 inputs in a group, groups of a tile
  for (int64_t tile = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); tile < tiles; tile += (int64_t)gridDim.x * 4) {
    const int64_t nt = tile / Kt;               // over the weights
    const int kb = (int)(tile - nt * Kt);
    const int64_t g = nt / Nt;
    const int n = (int)(nt - g * Nt) * kTileN + c;
    const int64_t row = g * N + n;
    float v[4][8];
    unsigned m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = kb * kTileK + 32 * i + 8 * h;
      const bool ok = n < N && k < K;
      const size_t at = (size_t)row * K + k;
      m[i] = 0u;
      if constexpr (KIND == 0) {
        uint4 r = make_uint4(0u, 0u, 0u, 0u);
        if (ok) r = ld16(static_cast<const bf16*>(in) + at);
        eng::unpack8(r, v[i]);
      } else if constexpr (KIND == 1) {
        uint4 r[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
        if (ok) {
          r[0] = ld16(static_cast<const float*>(in) + at);
          r[1] = ld16(static_cast<const float*>(in) + at + 4);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = reinterpret_cast<const float*>(r)[j];
      } else {
        uint2 r = make_uint2(0u, 0u);
        if (ok) r = *reinterpret_cast<const uint2*>(static_cast<const int8_t*>(in) + at);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v[i][j] = (float)min(7, max(-8, (int)reinterpret_cast<const int8_t*>(&r)[j]));
      }
      if constexpr (KIND != 2) {
#pragma unroll
        for (int j = 0; j < 8; ++j) m[i] = max(m[i], __float_as_uint(v[i][j]) & 0x7fffffffu);
        m[i] = max(m[i], (unsigned)__shfl_xor((int)m[i], 16));
        m[i] = max(m[i], (unsigned)__shfl_xor((int)m[i], 32));
      }
    }
    unsigned w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int i0 = i / per * per;
      const bool ok = n < N && kb * kTileK + 32 * i0 < K;
      uint16_t sb = 0;
      if constexpr (KIND == 2) {
        if (ok) sb = sin[row * (K / group) + (kb * kTileK + 32 * i0) / group];
      } else {
        unsigned mg = 0u;
#pragma unroll
        for (int a = 0; a < 4; ++a) mg = a / per == i / per ? max(mg, m[a]) : mg;
        if (mg >= 0x7f800000u) {
          sb = 0x7fc0;
        } else {
          const bf16 s = (bf16)fmaxf(__uint_as_float(mg) / 7.0f, 0x1p-126f);
          sb = __builtin_bit_cast(uint16_t, s);
        }
        // the quotient in 64 bits, where no rounding can carry it onto or over a tie: numerator and denominator have 24
        // and 8 significant bits
        const double s = (double)bf16_bits(sb);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v[i][j] = mg >= 0x7f800000u ? 0.f : (float)fmin(7.0, fmax(-7.0, rint((double)v[i][j] / s)));
        if (!ok) sb = 0;
      }
      w[i] = 0u;
#pragma unroll
      for (int j = 0; j < 8; ++j) w[i] |= (unsigned)((int)v[i][j] + 8) << (16 * (j & 1) + 4 * (j >> 1));
      if (h == 0 && i == i0) sout[(tile * kTileN + c) * ng + i / per] = sb;
    }
    st16(q + tile * kTileBytes4 + 16 * lane, make_uint4(w[0], w[1], w[2], w[3]));
  }
}

// ------------------------------------------------------------------------------------------------
constexpr int kRW4 = 8;   // waves of k_int4_rows

// 16 channels from n0 of group g times its rows r0 .. r0 + cnt (up to 16 NG of them). PER: steps of 32 inputs a group.
template <int NG, int PER>
__device__ __forceinline__ void rows4_task(const I4Params& p, f32x4* red, int g, int nt, int64_t r0, int cnt) {
  constexpr int NS = 4 / PER;   // scales of a tile and channel
  const int tid = threadIdx.x, lane = tid & 63, w = eng::wave_id(), c = lane & 15, h = lane >> 4;
  const int Nt = (p.N + kTileN - 1) / kTileN, Kt = (p.K + kTileK - 1) / kTileK;
  const int64_t tile0 = ((int64_t)g * Nt + nt) * Kt;
  const uint8_t* pq = p.q + tile0 * kTileBytes4 + 16 * lane;
  const uint16_t* ps = static_cast<const uint16_t*>(p.s) + (tile0 * kTileN + c) * NS;
  const bf16* px[NG];
#pragma unroll
  for (int i = 0; i < NG; ++i) px[i] = static_cast<const bf16*>(p.x) + (r0 + min(16 * i + c, cnt - 1)) * p.K + 8 * h;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u), m24 = make_uint4(kMinus24, kMinus24, kMinus24, kMinus24);
  f32x4 acc[NG];
#pragma unroll
  for (int i = 0; i < NG; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int kb = w * Kt / kRW4; kb < (w + 1) * Kt / kRW4; ++kb) {
    const uint4 q = ld16(pq + (size_t)kb * kTileBytes4);
    const unsigned qw[4] = {q.x, q.y, q.z, q.w};
    uint16_t s[NS];
#pragma unroll
    for (int a = 0; a < NS; ++a) s[a] = ps[(size_t)kb * kTileN * NS + a];
#pragma unroll
    for (int a = 0; a < NS; ++a) {
      f32x4 part[NG];
#pragma unroll
      for (int i = 0; i < NG; ++i) part[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int b = 0; b < PER; ++b) {
        const int st = a * PER + b, k = kb * kTileK + 32 * st;
        const uint4 wv = unpack16(qw[st]);
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          const uint4 xv = k < p.K ? ld16(px[i] + k) : zero;
          mma16<bf16>(part[i], xv, m24);
          mma16<bf16>(part[i], xv, wv);
        }
      }
      const float sf = bf16_bits(s[a]);
#pragma unroll
      for (int i = 0; i < NG; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][e] = fmaf(sf, part[i][e], acc[i][e]);
    }
  }
#pragma unroll
  for (int i = 0; i < NG; ++i) {
    if (16 * i >= cnt) break;
    red[w * 64 + lane] = acc[i];
    __syncthreads();
    if (tid < 256) {
      const int f = tid & 15, r = tid >> 4, n = nt * kTileN + f;
      const float* rs = reinterpret_cast<const float*>(red) + ((r >> 2) * 16 + f) * 4 + (r & 3);
      float sum = 0.f;
#pragma unroll
      for (int v = 0; v < kRW4; ++v) sum += rs[v * 256];
      if (16 * i + r < cnt && n < p.N) {
        const size_t at = (size_t)(r0 + 16 * i + r) * p.N + n;
        if (p.f32) static_cast<float*>(p.y)[at] = sum;
        else static_cast<bf16*>(p.y)[at] = (bf16)sum;
      }
    }
    __syncthreads();
  }
}

template <int PER>
__global__ __launch_bounds__(kRW4 * 64) void k_int4_rows(I4Params p) {
  __shared__ f32x4 red[kRW4 * 64];
  const int g = blockIdx.y, nt = blockIdx.x;
  int64_t r0 = 0, r1 = p.M;
  if (p.offsets) {
    r0 = min(max((int64_t)p.offsets[g], (int64_t)0), p.M);
    r1 = min(max((int64_t)p.offsets[g + 1], r0), p.M);
  }
  for (int64_t r = r0 + 64 * (int64_t)blockIdx.z; r < r1; r += 64 * (int64_t)gridDim.z) {
    const int cnt = __builtin_amdgcn_readfirstlane((int)min((int64_t)64, r1 - r));
    if (cnt <= 16) rows4_task<1, PER>(p, red, g, nt, r, cnt);
    else if (cnt <= 32) rows4_task<2, PER>(p, red, g, nt, r, cnt);
    else rows4_task<4, PER>(p, red, g, nt, r, cnt);
  }
}

}  // namespace

hipError_t launch_int4_matmul(const I4Params& p, hipStream_t s) {
  prof_mark_begin("int4_rows", s);
  const dim3 grid((p.N + kTileN - 1) / kTileN, p.G, (unsigned)std::min<int64_t>((p.M + 63) / 64, 256));
  if (p.group == 32) k_int4_rows<1><<<grid, kRW4 * 64, 0, s>>>(p);
  else if (p.group == 64) k_int4_rows<2><<<grid, kRW4 * 64, 0, s>>>(p);
  else k_int4_rows<4><<<grid, kRW4 * 64, 0, s>>>(p);
  const hipError_t err = hipGetLastError();
  if (err == hipSuccess) prof_mark_end(s);
  return err;
}

hipError_t launch_int4_pack(const void* in, bool f32, const void* scales, int G, int N, int K, int group, uint8_t* q,
                            void* out_scales, hipStream_t s) {
  prof_mark_begin("int4_pack", s);
  const int64_t tiles = (int64_t)G * ((N + kTileN - 1) / kTileN) * ((K + kTileK - 1) / kTileK);
  const unsigned grid = (unsigned)std::min<int64_t>((tiles + 3) / 4, 1 << 22);
  const uint16_t* si = static_cast<const uint16_t*>(scales);
  uint16_t* so = static_cast<uint16_t*>(out_scales);
  if (scales) k_int4_pack<2><<<grid, 256, 0, s>>>(in, si, tiles, N, K, group, q, so);
  else if (f32) k_int4_pack<1><<<grid, 256, 0, s>>>(in, nullptr, tiles, N, K, group, q, so);
  else k_int4_pack<0><<<grid, 256, 0, s>>>(in, nullptr, tiles, N, K, group, q, so);
  const hipError_t err = hipGetLastError();
  if (err == hipSuccess) prof_mark_end(s);
  return err;
}

}  // namespace moe
