// Products with 4-bit weights and a scale for each group of inputs.
//
//   k_int4_pack   a weight's tiles, from fp32 or bf16 (quantised here) or from whole numbers and scales.
//   k_int4_rows   y = sum over groups of s (x q^T): a workgroup takes 16 output channels, its waves split K, and the
//                 weight is read once for up to 64 rows.
//   k_int4_tile   the same for many rows: tiles in LDS, the weight's numbers unpacked once for a workgroup.
// A number q of a weight is held in four bits, a sign and m = |q| (sign 1 and m = 0: -8). Two masks give four numbers
// each as bytes, a sign bit and the low three; such a byte is q 2^-9 in e4m3, and v_cvt_scalef32_pk_bf16_fp8 (two numbers
// an instruction, at the rate of a plain one) makes q in bf16 of it: 7 instructions for 8 numbers. -8, which a symmetric
// quantiser does not make, takes 12 more; 64 channels that hold none say so in a word of theirs. The matrix instruction's products x q
// are exact, and its fp32 sums of a group are multiplied with the scale.
#include <algorithm>
#include <type_traits>

#include "engine.h"
#include "group_tiles.h"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kTileN = 16, kTileK = 128, kTileBytes4 = 1024, kFlagBytes = 16;
// Four tiles share 64 channels: tile t's column c is channel 4 c + t of them, so that a wavefront that takes all four
// holds four neighbouring channels in a lane.
__host__ __device__ constexpr int rows64(int N) { return (N + 63) / 64; }
__device__ __forceinline__ int channel4(int nt, int c) { return nt / 4 * 64 + 4 * c + nt % 4; }
// 64 channels (row64 over all weights): their tiles, and behind them the word that says whether one holds a -8
__device__ __forceinline__ size_t row_bytes(int Kt) { return (size_t)4 * Kt * kTileBytes4 + kFlagBytes; }
__device__ __forceinline__ const uint8_t* tile_at(const uint8_t* q, int64_t row64, int t, int Kt) {
  return q + row64 * row_bytes(Kt) + (size_t)t * Kt * kTileBytes4;
}
__device__ __forceinline__ int holds_8(const uint8_t* q, int64_t row64, int Kt) {
  return eng::ld_uniform(reinterpret_cast<const int*>(q + row64 * row_bytes(Kt) + (size_t)4 * Kt * kTileBytes4), 0);
}
// the first scale of channel n of 64 in tile column kb, of ng each
__device__ __forceinline__ size_t scale_at(int64_t row64, int Kt, int kb, int n, int ng) {
  return ((size_t)(row64 * Kt + kb) * 64 + n) * ng;
}

// The numbers of a word as bytes: sign and magnitude.
struct Bytes8 { unsigned a, b; };   // numbers 0..3 and 4..7
__device__ __forceinline__ Bytes8 bytes8(unsigned w) {
  return {w & 0x87878787u, __builtin_amdgcn_alignbit(w, w, 4) & 0x87878787u};
}
__device__ __forceinline__ unsigned with_8(unsigned t) {   // sign 1 and magnitude 0 become -8
  const unsigned some = (t & 0x07070707u) + 0x07070707u;   // bit 3: a magnitude other than 0
  return t | ((t >> 4) & ~some & 0x08080808u);
}
// The numbers 2d and 2d + 1 in bf16, d = 0..3.
__device__ __forceinline__ uint4 numbers8(Bytes8 v) {
  const auto two = [](unsigned v, auto half) {
    return __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 512.f, decltype(half)::value));
  };
  return make_uint4(two(v.a, std::false_type{}), two(v.a, std::true_type{}), two(v.b, std::false_type{}),
                    two(v.b, std::true_type{}));
}
// A condition that the compiler does not know to be the same all the time: it would make two loops of one.
__device__ __forceinline__ bool here(int b) {
  int v = __builtin_amdgcn_readfirstlane(b);
  asm volatile("" : "+s"(v));
  return v != 0;
}
// The four words of a tile column that a lane holds, as fragments.
__device__ __forceinline__ void unpack4(uint4 q, int eights, uint4 (&f)[4]) {
  Bytes8 v[4] = {bytes8(q.x), bytes8(q.y), bytes8(q.z), bytes8(q.w)};
  if (here(eights))
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = {with_8(v[i].a), with_8(v[i].b)};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = numbers8(v[i]);
}
// the word's bits for its number j
__device__ __forceinline__ unsigned pack4(int q, int j) {
  const unsigned sign = q < 0, m = (unsigned)(q < 0 ? -q : q) & 7u;
  return j < 4 ? m << (8 * j) | sign << (8 * j + 7) : m << (8 * (j - 4) + 4) | sign << ((8 * (j - 4) + 11) & 31);
}

__device__ __forceinline__ float bf16_bits(unsigned short b) { return __uint_as_float((unsigned)b << 16); }

// N bf16 scales, two a word: taken apart where they are used, so that they do not fill a register each meanwhile.
template <int N>
struct alignas(N * 2 < 16 ? N * 2 : 16) Scales4 {
  unsigned w[N / 2];
  __device__ __forceinline__ float operator[](int i) const {
    return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
  }
};
template <>
struct Scales4<1> {
  uint16_t v;
  __device__ __forceinline__ float operator[](int) const { return bf16_bits(v); }
};

// KIND 0: bf16, 1: fp32, 2: signed bytes with bf16 scales. A workgroup takes 64 channels, a wave one of their tiles, every
// fourth column of it (in a grid of y workgroups to the channels: every 4 y-th); lane 16 h + c takes inputs 32 i + 8 h + j,
// i < 4, j < 8. KIND 2 takes y = 1, as the word that says whether there is a -8 is made of all columns.
constexpr int kPackWaves = 16;
template <int KIND>
__global__ __launch_bounds__(kPackWaves * 64) void k_int4_pack(const void* __restrict__ in, const uint16_t* __restrict__ sin, int64_t rows,
                                                   int N, int K, int group, uint8_t* __restrict__ q,
                                                   uint16_t* __restrict__ sout) {
  const int t = (threadIdx.x >> 6) & 3, lane = threadIdx.x & 63, c = lane & 15, h = lane >> 4;
  const int Kt = (K + kTileK - 1) / kTileK;
  const int per = group / 32, ng = 4 / per;     // steps of 32 inputs in a group, groups of a tile
  const int64_t row64 = blockIdx.x;             // over the weights
  const int64_t g = row64 / rows64(N);
  const int n = (int)(row64 - g * rows64(N)) * 64 + 4 * c + t;
  const int64_t row = g * N + n;
  unsigned* flag = reinterpret_cast<unsigned*>(q + row64 * row_bytes(Kt) + (size_t)4 * Kt * kTileBytes4);
  bool eights = false;
  for (int kb = blockIdx.y * (kPackWaves / 4) + (threadIdx.x >> 8); kb < Kt; kb += gridDim.y * (kPackWaves / 4)) {
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
        // v / s to the nearest whole number, ties to even. v and s have 24 and 8 significant bits, so that a quotient that is
        // no tie lies 2^-25 or more from one; v times 1 / s, each rounded to 64 bits, is off by 2^-49 at most, and rounded
        // to a multiple of 2^-32 (by adding a number with such a step) it is a tie where the quotient is one, and only there.
        const double r = 1.0 / (double)bf16_bits(sb), step = 0x1.8p20;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const double x = fma((double)v[i][j], r, step) - step;
          v[i][j] = mg >= 0x7f800000u ? 0.f : fminf(7.f, fmaxf(-7.f, (float)rint(x)));
        }
        if (!ok) sb = 0;
      }
      w[i] = 0u;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        w[i] |= pack4((int)v[i][j], j);
        if constexpr (KIND == 2) eights |= v[i][j] == -8.f;
      }
      if (h == 0 && i == i0) sout[scale_at(row64, Kt, kb, 4 * c + t, ng) + i / per] = sb;
    }
    st16(q + row64 * row_bytes(Kt) + ((size_t)t * Kt + kb) * kTileBytes4 + 16 * lane, make_uint4(w[0], w[1], w[2], w[3]));
  }
  const int any = __syncthreads_or(eights);
  if (blockIdx.y == 0 && threadIdx.x < kFlagBytes / 4) flag[threadIdx.x] = any != 0;
}

// ------------------------------------------------------------------------------------------------
// k_int4_rows: persistent workgroups take tasks round-robin, each up to 16 rows of a group. wk of the workgroup's waves
// share a task's channels and split K, and their sums meet in LDS. Behind a tile's products its numbers are replaced by the
// next ones needed, of this task or the next, so that some are in flight all the time; no load stands in a branch, where the
// compiler could not count those in flight.
//   tasks_more  a wave takes TL tiles of 16 channels, a tile column at a time, so that a row's fragments serve TL products.
//   tasks_few   up to 4 rows where there are few tasks (TL = 1), in units of kUnit columns, which are all in flight at
//               once. As the matrix instruction's 16 rows would be mostly empty, they are 4 rows of the unit's 4 columns, and
//               of a column's products the quarter of the lanes counts that holds its rows. One row of 1536 x 4096
//               5.1 us, 6.0 a column at a time; with TL = 4 the other form is as fast or faster (2 rows of 307200 x 4096
//               117 us, 142 here).
constexpr int kRows4 = 16, kFew4 = 4, kUnit = 4, kRowWaves = 4;

// A load of 2 to 32 bytes from a uniform address and a lane's offset. Made in the global address space: a flat load would
// wait for LDS as well, and for all loads before it.
template <class T>
__device__ __forceinline__ T ld_at(const void* base, unsigned off) {
  typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
  typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  const uint64_t u = (uint64_t)__builtin_amdgcn_readfirstlane((unsigned)(a >> 32)) << 32 |
                     (unsigned)__builtin_amdgcn_readfirstlane((unsigned)a);
  typedef const __attribute__((address_space(1))) char* global;
  const global at = (global)u + off;
#define MOE_LD(V) __builtin_bit_cast(T, *(const __attribute__((address_space(1))) V*)at)
  if constexpr (sizeof(T) == 2) return MOE_LD(uint16_t);
  else if constexpr (sizeof(T) == 4) return MOE_LD(unsigned);
  else if constexpr (sizeof(T) == 8) return MOE_LD(u32x2);
  else if constexpr (sizeof(T) == 16) return MOE_LD(u32x4);
  else {
    struct Two { u32x4 a, b; };
    const Two t = {*(const __attribute__((address_space(1))) u32x4*)at, *(const __attribute__((address_space(1))) u32x4*)(at + 16)};
    return __builtin_bit_cast(T, t);
  }
#undef MOE_LD
}

// find_tile with two LDS round trips instead of one for each halving
template <int BM>
__device__ __forceinline__ void find_tile64(const I4Params& p, const Groups& s, int mt, int lane, int& g, int& r0, int& end) {
  if (!p.offsets) return find_tile<BM>(p, s, mt, g, r0, end);
  const int per = (p.G + 63) / 64;
  const int a = __popcll(__ballot(s.tile0[min(lane * per, p.G)] <= mt && lane * per < p.G)) - 1;   // tile0[0] = 0
  const int b = a * per + min(lane, per - 1);
  const unsigned long long m = __ballot(lane < per && b < p.G && s.tile0[min(b, p.G)] <= mt);
  g = __builtin_amdgcn_readfirstlane(a * per + __popcll(m) - 1);
  r0 = __builtin_amdgcn_readfirstlane(s.row0[g] + (mt - s.tile0[g]) * BM);
  end = __builtin_amdgcn_readfirstlane(max(s.row0[g + 1], s.row0[g]));
}

// Where the waves of a task are: those of the workgroup, wk to a task.
struct Waves {
  int lane = threadIdx.x & 63, c = lane & 15, h = lane >> 4, wk, kw, tw, wt;
  __device__ __forceinline__ explicit Waves(int wk) : wk(wk) {
    const int w = eng::wave_id();
    kw = w % wk;
    tw = w / wk;
    wt = kRowWaves / wk;
  }
};

// The sums of the task's wk waves in LDS for each of TL tiles, as stored by lanes 16 h + c: rows 4 h .. 4 h + 3 of
// channel c (FEW: rows 0 .. 3, a quarter of the sum). They are added and stored to y from row r0 on, cnt rows, and channels
// of the tiles from nt on.
template <int TL, bool FEW>
__device__ __forceinline__ void store_sums(const I4Params& p, const f32x4* red, int wk, int64_t r0, int cnt, int nt, int ntiles) {
  constexpr int ROWS = FEW ? 4 : 16;
  for (int o = threadIdx.x; o < kRowWaves / wk * TL * 16 * ROWS; o += kRowWaves * 64) {
    const int f = o & 15, r = (o >> 4) % ROWS, t = o / (16 * ROWS), n = channel4(nt + t, f);
    if (r >= cnt || nt + t >= ntiles || n >= p.N) continue;
    // wave (t / TL) wk + v holds tile t % TL
    const float* rs = reinterpret_cast<const float*>(red + ((t / TL * wk) * TL + t % TL) * 64 + (r >> 2) * 16 + f) + (r & 3);
    float sum = 0.f;
    for (int v = 0; v < wk; ++v, rs += TL * 256) sum += FEW ? (rs[0] + rs[64]) + (rs[128] + rs[192]) : rs[0];
    const size_t at = (size_t)(r0 + r) * p.N + n;
    if (p.f32) static_cast<float*>(p.y)[at] = sum;
    else static_cast<bf16*>(p.y)[at] = (bf16)sum;
  }
}

template <int PER>
__device__ __forceinline__ void tasks_few(const I4Params& p, const Groups& groups, f32x4* red, int mtiles, int wk) {
  constexpr int NS = 4 / PER;   // scales of a tile and channel
  using Scales = Scales4<NS>;
  const Waves W(wk);
  const int lane = W.lane, c = W.c, h = W.h;
  const int Nt = 4 * rows64(p.N), Kt = (p.K + kTileK - 1) / kTileK, ntn = (Nt + W.wt - 1) / W.wt, tasks = mtiles * ntn;
  const int k0 = W.kw * Kt / wk, k1 = (W.kw + 1) * Kt / wk;   // the wave's tile columns
  // the unit that is loaded next: task `task`, from column kb on
  int task = (int)blockIdx.x - (int)gridDim.x, kb = k0, g = 0, r0 = 0, cnt = 0, nt = 0;
  auto find = [&] {
    do {
      task += gridDim.x;
      if (task >= tasks) return;
      const int mt = task / ntn;
      int end;
      find_tile64<kRows4>(p, groups, mt, lane, g, r0, end);
      cnt = min(end - r0, kRows4);
      nt = min((task - mt * ntn) * W.wt + W.tw, Nt - 1);      // (behind the last tile: that one again, not stored)
    } while (cnt > kFew4);
  };
  uint4 q[kUnit], x[4], xn[4];
  Scales sc[kUnit];
  const uint8_t* pq;
  const uint16_t* ps;
  int eights, eights_next;
  auto at = [&] {
    const int64_t row64 = (int64_t)g * (Nt / 4) + nt / 4;
    pq = tile_at(p.q, row64, nt % 4, Kt);
    ps = static_cast<const uint16_t*>(p.s) + scale_at(row64, Kt, 0, nt % 4, NS);
    eights_next = holds_8(p.q, row64, Kt);
  };
  auto load = [&](int b) {   // (behind the wave's last column: that one again, which is not added)
    const int k = max(min(kb + b, k1 - 1), 0);
    q[b] = ld_at<uint4>(pq + (size_t)k * kTileBytes4, 16 * lane);
    sc[b] = ld_at<Scales>(ps + (size_t)k * 64 * NS, 8 * c * NS);
  };
  auto load_x = [&] {   // inputs beyond K have zero weights: others of the row are read
    const unsigned off = min(c & 3, cnt - 1) * (unsigned)p.K * 2 + 16 * h;
    const int k = max(min(kb + (c >> 2), k1 - 1), 0) * kTileK;
#pragma unroll
    for (int st = 0; st < 4; ++st)
      xn[st] = ld_at<uint4>(static_cast<const bf16*>(p.x) + (size_t)r0 * p.K, off + 2 * min(k + 32 * st, p.K - 32));
  };
  find();
  if (task >= tasks) return;
  at();
  load_x();
#pragma unroll
  for (int b = 0; b < kUnit; ++b) load(b);
  int parity = 0;
  while (task < tasks) {
    const int mr0 = r0, mcnt = cnt, n0 = task % ntn * W.wt;
    eights = eights_next;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    for (int mkb = k0;;) {
      const int n = k1 - mkb;   // columns from this unit on
#pragma unroll
      for (int st = 0; st < 4; ++st) x[st] = xn[st];
      kb += kUnit;
      if (kb >= k1) {
        kb = k0;
        find();
        if (task < tasks) at();
      }
      load_x();
#pragma unroll
      for (int b = 0; b < kUnit; ++b) {
        uint4 f[4];
        unpack4(q[b], eights, f);
#pragma unroll
        for (int a = 0; a < NS; ++a) {
          f32x4 part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int st = a * PER; st < (a + 1) * PER; ++st) mma16<bf16>(part, x[st], f[st]);
          const float sf = sc[b][a];
          if (h == b && b < n)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] = fmaf(sf, part[e], acc[e]);
        }
        load(b);
        __builtin_amdgcn_sched_barrier(0);   // (columns worked on at the same time take more registers than there are)
      }
      mkb += kUnit;
      if (mkb >= k1) break;
    }
    f32x4* to = red + parity * kRowWaves * 64;
    parity ^= 1;
    to[threadIdx.x] = acc;
    __syncthreads();
    store_sums<1, true>(p, to, wk, mr0, mcnt, n0, Nt);
  }
}

template <int PER, int TL>
__device__ __forceinline__ void tasks_more(const I4Params& p, const Groups& groups, f32x4* red, int mtiles, int wk) {
  constexpr int NS = 4 / PER;
  using Scales = Scales4<TL * NS>;
  const Waves W(wk);
  const int lane = W.lane, c = W.c, h = W.h;
  const int Nt = 4 * rows64(p.N), Kt = (p.K + kTileK - 1) / kTileK, per = W.wt * TL, ntn = (Nt + per - 1) / per,
            tasks = mtiles * ntn;
  const int k0 = W.kw * Kt / wk, k1 = (W.kw + 1) * Kt / wk;
  int task = (int)blockIdx.x - (int)gridDim.x, kb = k0, g = 0, r0 = 0, cnt = 0, nt = 0;
  auto find = [&] {
    do {
      task += gridDim.x;
      if (task >= tasks) return;
      const int mt = task / ntn;
      int end;
      find_tile64<kRows4>(p, groups, mt, lane, g, r0, end);
      cnt = min(end - r0, kRows4);
      nt = min((task - mt * ntn) * per + W.tw * TL, Nt - TL);
    } while (TL == 1 && cnt <= kFew4);
  };
  uint4 q[TL], x[4], xn[4];
  Scales sc, sn;
  const uint8_t* pq;
  const uint16_t* ps;
  int eights, eights_next;
  auto at = [&] {
    const int64_t row64 = (int64_t)g * (Nt / 4) + nt / 4;
    pq = tile_at(p.q, row64, nt % 4, Kt);
    ps = static_cast<const uint16_t*>(p.s) + scale_at(row64, Kt, 0, nt % 4, NS);
    eights_next = holds_8(p.q, row64, Kt);
  };
  auto column = [&] { return max(min(kb, k1 - 1), 0); };
  auto load = [&](int t) { q[t] = ld_at<uint4>(pq + ((size_t)t * Kt + column()) * kTileBytes4, 16 * lane); };
  auto load_x = [&] {
    const bf16* row = static_cast<const bf16*>(p.x) + (size_t)r0 * p.K;
    const unsigned off = min(c, cnt - 1) * (unsigned)p.K * 2 + 16 * h;
#pragma unroll
    for (int st = 0; st < 4; ++st) xn[st] = ld_at<uint4>(row + min(column() * kTileK + 32 * st, p.K - 32), off);
    sn = ld_at<Scales>(ps + (size_t)column() * 64 * NS, 8 * c * NS);
  };
  find();
  if (task >= tasks) return;
  at();
  load_x();
#pragma unroll
  for (int t = 0; t < TL; ++t) load(t);
  while (task < tasks) {
    const int mr0 = r0, mcnt = cnt, n0 = task % ntn * per;
    eights = eights_next;
    f32x4 acc[TL];
#pragma unroll
    for (int t = 0; t < TL; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int mkb = k0;;) {
      const bool in = mkb < k1;   // (a wave without columns adds nothing)
#pragma unroll
      for (int st = 0; st < 4; ++st) x[st] = xn[st];
      sc = sn;
      if (++kb >= k1) {
        kb = k0;
        find();
        if (task < tasks) at();
      }
      load_x();
#pragma unroll
      for (int t = 0; t < TL; ++t) {
        uint4 f[4];
        unpack4(q[t], eights, f);
#pragma unroll
        for (int a = 0; a < NS; ++a) {
          f32x4 part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int st = a * PER; st < (a + 1) * PER; ++st) mma16<bf16>(part, x[st], f[st]);
          const float sf = in ? sc[t * NS + a] : 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[t][e] = fmaf(sf, part[e], acc[t][e]);
        }
        load(t);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (++mkb >= k1) break;
    }
    __syncthreads();   // the previous task's sums are read
#pragma unroll
    for (int t = 0; t < TL; ++t) red[(eng::wave_id() * TL + t) * 64 + lane] = acc[t];
    __syncthreads();
    store_sums<TL, false>(p, red, wk, mr0, mcnt, n0, Nt);
  }
}

// workgroups a CU: with four scales a tile column the registers serve three
constexpr int rows_wgs(int PER) { return PER == 1 ? 3 : 4; }
template <int PER, int TL>
__global__ __launch_bounds__(kRowWaves * 64, rows_wgs(PER)) void k_int4_rows(I4Params p, int wk) {
  __shared__ f32x4 red[(TL > 2 ? TL : 2) * kRowWaves * 64];
  __shared__ Groups groups;
  const int mtiles = group_tiles<kRows4>(p, groups);
  if constexpr (TL == 1) tasks_few<PER>(p, groups, red, mtiles, wk);
  tasks_more<PER, TL>(p, groups, red, mtiles, wk);
}

// ------------------------------------------------------------------------------------------------
// k_int4_tile: WM x WN waves of MI x NJ blocks of 16 x 16, K in stages of 64 inputs. x comes into LDS by direct loads,
// two stages of it in rows of 128 bytes; each wave unpacks its own channels' numbers into fragments, those of the next
// stage behind the last products of this one. A stage's sums (PER = 1: its halves') start from zero and are added to the
// accumulators times their scales, a row block later than they are made, so that the matrix cores have work meanwhile.
constexpr int kRowB = 128;   // bytes of a row in a stage

// The 16-byte chunk c of row r lies in slot c ^ swz_x(r): 16 consecutive rows at one chunk, which a fragment read
// takes, stand in distinct banks.
__device__ __forceinline__ int swz_x(int r) { return (r >> 1) & 7; }

// eng::gl2lds from a uniform address and a lane's offset
__device__ __forceinline__ void gl2lds_at(const void* base, unsigned off, char* lds) {
  const unsigned to = __builtin_amdgcn_readfirstlane((unsigned)(uintptr_t)lds);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(off), "s"(base) : "memory", "m0");
}

template <int MI, int NJ, int WM, int WN, int PER>
__global__ __launch_bounds__(64 * WM * WN, 2) void k_int4_tile(I4Params p) {
  constexpr int NW = WM * WN, BM = 16 * MI * WM, BN = 16 * NJ * WN, ST = BM * kRowB;
  constexpr int LA = BM / (8 * NW), NS = 4 / PER;
  __shared__ __attribute__((aligned(1024))) char smem[2 * ST];
  __shared__ Groups groups;
  const int lane = threadIdx.x & 63, w = eng::wave_id(), wm = w / WN, wn = w % WN, c = lane & 15, h = lane >> 4;
  const int R64 = rows64(p.N), Kt = (p.K + kTileK - 1) / kTileK, nst = (p.K + 63) / 64;
  const bool half = p.K % 64 != 0;             // the last stage has 32 inputs
  const int ntn = (p.N + BN - 1) / BN;
  const bool wide = p.N % NJ == 0 && reinterpret_cast<uintptr_t>(p.y) % (NJ * (p.f32 ? 4 : 2)) == 0;
  // the lane's fragment reads: chunk 4 s + h of row c of a block
  const char* ao[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) ao[s] = smem + (16 * MI * wm + c) * kRowB + ((4 * s + h) ^ swz_x(c)) * 16;
  const int mtiles = group_tiles<BM>(p, groups);
  const XcdRange xr = xcd_range(mtiles * ntn);
  for (int tile = xr.first; tile < xr.end; tile += xr.stride) {
    const int mt = tile / ntn, n0 = (tile - mt * ntn) * BN;
    int g, r0, end;
    find_tile<BM>(p, groups, mt, g, r0, end);
    const char* xb = reinterpret_cast<const char*>(static_cast<const bf16*>(p.x) + (size_t)r0 * p.K);
    // This lane moves chunk (lane % 8) ^ swz_x(r) of rows r = (w LA + j) 8 + lane / 8; of an even LA that is the same
    // chunk for all even j, and the one 4 further for the odd ones. (At most BM rows of 131072 inputs: 32 bits.)
    const unsigned K2 = 2u * (unsigned)p.K, x0 = K2 * (w * LA * 8 + lane / 8), xlast = K2 * min(end - 1 - r0, BM - 1);
    const unsigned ch = ((lane & 7) ^ swz_x(w * LA * 8 + lane / 8)) * 16;
    static_assert(LA % 2 == 0, "");
    // Inputs beyond K (half a stage, or a tile's second one) have zero weights; read for them are others of the same row.
    auto issue = [&](int st) {
      const int in = min(st, nst - 1);
      const char* at = xb + (size_t)in * kRowB;
      const unsigned in4 = half && in + 1 == nst ? 63u : 127u;
      char* to = smem + (st & 1) * ST + w * LA * 1024;
      unsigned x = x0, even = ch & in4, odd = (ch ^ 64u) & in4;
      asm volatile("" : "+v"(x), "+v"(even), "+v"(odd));   // the offsets are made here rather than kept in registers
#pragma unroll
      for (int j = 0; j < LA; ++j)
        gl2lds_at(at, min(x + 8 * j * K2, xlast) + (j & 1 ? odd : even), to + j * 1024);
    };
    const int nt = n0 / kTileN + NJ * wn, n1 = channel4(nt, c);   // the lane's channels: NJ from n1 on
    // (a wave whose channels lie behind the last works on others, for nothing)
    const int64_t row64 = (int64_t)g * R64 + min(nt / 4, R64 - 1);
    const uint8_t* qb = tile_at(p.q, row64, nt % 4, Kt);
    const uint16_t* ps = static_cast<const uint16_t*>(p.s) + scale_at(row64, Kt, 0, nt % 4, NS);
    const int eights = holds_8(p.q, row64, Kt);
    using Scales = Scales4<NJ * NS>;
    uint4 q[NJ], fb[2][NJ];
    Scales sc, sn;
    auto load = [&](int kb) {                  // (behind the last tile: read once more, and not used)
      const size_t k = min(kb, Kt - 1);
#pragma unroll
      for (int j = 0; j < NJ; ++j) q[j] = ld_at<uint4>(qb + ((size_t)j * Kt + k) * kTileBytes4, 16 * lane);
      sn = ld_at<Scales>(ps + k * 64 * NS, 4 * c * NS * 2);
    };
    f32x4 acc[MI][NJ];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    eng::block_sync();   // every wave is done reading the previous tile's stages
    issue(0);
    load(0);
    auto columns = [&](auto with8) {           // all of K, for weights with -8 among them or not
    auto word = [&](unsigned w) {
      const Bytes8 v = bytes8(w);
      if constexpr (decltype(with8)::value) return numbers8({with_8(v.a), with_8(v.b)});
      else return numbers8(v);
    };
    auto unpack = [&](bool odd) {              // the stage's words of q
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        fb[0][j] = word(odd ? q[j].z : q[j].x);
        fb[1][j] = word(odd ? q[j].w : q[j].y);
      }
    };
    unpack(false);
    auto stage = [&](int st, auto odd) {
      constexpr int O = decltype(odd)::value;
      eng::wait_vm<0>();
      if (O == 0) {
        // the scales have come too: said here, so that the compiler does not wait for them behind the loads below
#pragma unroll
        for (int b = 0; b < NJ * NS / 2; ++b) asm volatile("" : "+v"(sn.w[b]));
        sc = sn;
      }
      eng::block_sync();
      issue(st + 1);
      if (O == 1) load(st / 2 + 1);
      uint4 fa[2][2];
#pragma unroll
      for (int s = 0; s < 2; ++s) fa[0][s] = ld16(ao[s] + O * ST);
      constexpr int H = PER == 1 ? 2 : 1;      // sums of a stage and row block
      f32x4 part[2][NJ];
      auto add = [&](int u) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const float f = sc[j * NS + (PER == 1 ? 2 * O + u % H : PER == 2 ? O : 0)];
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[u / H][j][e] = fmaf(f, part[u & 1][j][e], acc[u / H][j][e]);
        }
      };
#pragma unroll
      for (int u = 0; u < MI * H; ++u) {
        const int i = u / H;
        if (u % H == 0 && i + 1 < MI)
#pragma unroll
          for (int s = 0; s < 2; ++s) fa[(i + 1) & 1][s] = ld16(ao[s] + O * ST + (i + 1) * 16 * kRowB);
#pragma unroll
        for (int s = u % H; s < 2; s += H)
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            f32x4& t = part[u & 1][j];
            if (s == u % H) t = f32x4{0.f, 0.f, 0.f, 0.f};
            mma16<bf16>(t, fa[i & 1][s], fb[s][j]);
          }
        if (u > 0) add(u - 1);
        __builtin_amdgcn_sched_barrier(0);
      }
      unpack(!O);
      add(MI * H - 1);
    };
    for (int kb = 0; kb < Kt; ++kb) {
      stage(2 * kb, std::integral_constant<int, 0>{});
      stage(2 * kb + 1, std::integral_constant<int, 1>{});
    }
    };
    if (eights) columns(std::true_type{});
    else columns(std::false_type{});
    eng::wait_vm<0>();
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = r0 + 16 * (MI * wm + i) + 4 * h + e;
        if (r >= end) continue;
        const size_t at = (size_t)r * p.N + n1;
        if (wide) {
          if (n1 >= p.N) continue;
          if (p.f32) {
            float* o = static_cast<float*>(p.y) + at;
            if constexpr (NJ == 4) *reinterpret_cast<f32x4*>(o) = f32x4{acc[i][0][e], acc[i][1][e], acc[i][2][e], acc[i][3][e]};
            else *reinterpret_cast<float2*>(o) = make_float2(acc[i][0][e], acc[i][1][e]);
          } else {
            alignas(8) bf16 v[NJ];
#pragma unroll
            for (int j = 0; j < NJ; ++j) v[j] = (bf16)acc[i][j][e];
            bf16* o = static_cast<bf16*>(p.y) + at;
            if constexpr (NJ == 4) *reinterpret_cast<uint2*>(o) = *reinterpret_cast<const uint2*>(v);
            else *reinterpret_cast<unsigned*>(o) = *reinterpret_cast<const unsigned*>(v);
          }
        } else {
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            if (n1 + j >= p.N) continue;
            if (p.f32) static_cast<float*>(p.y)[at + j] = acc[i][j][e];
            else static_cast<bf16*>(p.y)[at + j] = (bf16)acc[i][j][e];
          }
        }
      }
  }
}

// Tiles of bm rows by bn columns for the rows in as many groups as the product may have.
int64_t tiles4(const I4Params& p, int bm, int bn) {
  const int64_t m = p.M / bm + (p.offsets ? std::min<int64_t>(p.G, p.M) : 1);
  return std::min<int64_t>(m, p.M) * ((p.N + bn - 1) / bn);
}

// The kernel by the rows of a group that has any, as far as the host knows, and by how much work there is.
// Rows kernel, us, against the best tiles: 2048 rows in 64 groups of 1536 x 4096 76 and 104, 4096 rows 150 and 109; 128 rows of
// 4096 x 4096 16 and 21, 256 rows 28 and 30, 512 rows 50 and 35. TL = 4 against 1: one row of 4096 x 4096 9.3 and 5.0,
// of 32768 x 4096 14 and 17; 16 rows of 4096 x 4096 9.5 and 7.9, 32 rows 9.7 and 12.4.
// Tiles of 256 x 128, 128 x 128 and 64 x 64, us: 16384 rows of 2048 x 768 in 64 groups 63, 69, 138; 8192 rows of 1536 x 4096 in 64
// groups 224, 135, 285, 4096 rows 198, 111, 109; 1024 rows of 4096 x 4096 73, 49, 67, 512 rows 70, 44, 35.
template <int PER>
void launch4(const I4Params& p, int grid, hipStream_t s) {
  const int64_t groups = std::min<int64_t>(p.M, p.G);
  const int64_t mt = p.offsets ? p.M / kRows4 + groups : (p.M + kRows4 - 1) / kRows4;
  const int64_t work = mt * rows64(p.N);        // 16 rows by 64 channels
  const int Kt = (p.K + kTileK - 1) / kTileK;
  if (p.M <= 32 * groups || work <= 2 * grid) {
    auto go = [&](auto kernel, int TL) {
      // fewer waves a task where their columns would make less than a unit, as long as every CU keeps its workgroups
      const int64_t wgs = rows_wgs(PER) * grid;
      int wk = kRowWaves;
      while (wk > 1 && Kt < kUnit * wk && 4 * work * wk / kRowWaves >= 2 * wgs) wk /= 2;
      const int64_t tasks = (4 * work * wk / TL + kRowWaves - 1) / kRowWaves;
      kernel<<<(unsigned)std::min(tasks, wgs), kRowWaves * 64, 0, s>>>(p, wk);
    };
    if (work <= (p.M <= kFew4 * groups ? grid : 3 * grid / 8)) go(k_int4_rows<PER, 1>, 1);
    else go(k_int4_rows<PER, 4>, 4);
  } else if (p.M >= 192 * groups && 4 * tiles4(p, 256, 128) >= 6 * grid) {
    k_int4_tile<8, 4, 2, 2, PER><<<2 * grid, 256, 0, s>>>(p);
  } else if (p.M >= 72 * groups && 4 * tiles4(p, 128, 128) >= 3 * grid) {
    k_int4_tile<4, 4, 2, 2, PER><<<2 * grid, 256, 0, s>>>(p);
  } else {
    k_int4_tile<2, 2, 2, 2, PER><<<2 * grid, 256, 0, s>>>(p);
  }
}

}  // namespace

hipError_t launch_int4_matmul(const I4Params& p, hipStream_t s) {
  prof_mark_begin("int4_matmul", s);
  const int grid = persistent_grid(1);
  if (p.group == 32) launch4<1>(p, grid, s);
  else if (p.group == 64) launch4<2>(p, grid, s);
  else launch4<4>(p, grid, s);
  const hipError_t err = hipGetLastError();
  if (err == hipSuccess) prof_mark_end(s);
  return err;
}

hipError_t launch_int4_pack(const void* in, bool f32, const void* scales, int G, int N, int K, int group, uint8_t* q,
                            void* out_scales, hipStream_t s) {
  prof_mark_begin("int4_pack", s);
  const int64_t tiles = (int64_t)G * rows64(N);   // at most 2^23 workgroups
  const int columns = ((K + kTileK - 1) / kTileK + kPackWaves / 4 - 1) / (kPackWaves / 4), few = 2 * persistent_grid(1);
  const dim3 grid((unsigned)tiles, scales ? 1u : (unsigned)std::min<int64_t>(columns, std::max<int64_t>(few / tiles, 1)));
  const uint16_t* si = static_cast<const uint16_t*>(scales);
  uint16_t* so = static_cast<uint16_t*>(out_scales);
  if (scales) k_int4_pack<2><<<grid, kPackWaves * 64, 0, s>>>(in, si, tiles, N, K, group, q, so);
  else if (f32) k_int4_pack<1><<<grid, kPackWaves * 64, 0, s>>>(in, nullptr, tiles, N, K, group, q, so);
  else k_int4_pack<0><<<grid, kPackWaves * 64, 0, s>>>(in, nullptr, tiles, N, K, group, q, so);
  const hipError_t err = hipGetLastError();
  if (err == hipSuccess) prof_mark_end(s);
  return err;
}

}  // namespace moe
