// Products with 4-bit weights and a scale for each group of inputs.
//
//   k_int4_pack   a weight's tiles, from fp32 or bf16 (quantised here) or from whole numbers and scales.
//   k_int4_rows   y = sum over groups of s (x q^T) for few rows: 16 at a time, the weight straight from memory into
//                 registers, K split over a workgroup's waves. Bound by reading the weight (5.2 TB/s with 64 rows among 128
//                 experts of 1536 x 4096: 178 MB in 34 us), and with one weight by the launch (one row of 1536 x 4096 5.1 us).
//   k_int4_deep   64 x 64 and 64 x 128 tiles for products of few: all operands come straight into LDS.
//   k_int4_tile   256 x 128 and 128 x 128 tiles for products of many: x in LDS, the weight unpacked from registers.
//                 16384 x 4096 x 2048 270 to 300 us (920 to 1020 TFLOP/s, card to card); a bf16 product of this size by the
//                 library takes 243, and a loop of this many matrix instructions on such numbers, with nothing else, reached
//                 1120 to 1270 TFLOP/s (1415 on zeros): the clock falls with their load.
// launch4 says which takes what, with times. A number q of a weight is held in four bits, a sign and m = |q| (sign 1 and
// m = 0: -8). Two masks give four numbers each as bytes, a sign bit and the low three; such a byte is q 2^-9 in e4m3, and
// v_cvt_scalef32_pk_bf16_fp8 (two numbers an instruction, at the rate of a plain one) makes q in bf16 of it: 7 instructions
// for 8 numbers (13 from two's complement with masks and additions). -8, which a symmetric quantiser does not make, takes 12
// more; 64 channels that hold none say so in a word of theirs. The matrix instruction's products x q are exact, and its
// fp32 sums of a group are multiplied with the scale. Numbers in bytes 16 + q, with 16 times the sum of x taken off, would
// save the signs but lose bits where x's sum is large.
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
// 64 channels (row64 over all weights): their tiles, and behind them a word that says whether one holds a -8 and one
// that says K, of which the tiles themselves know no more than ceil(K / 128)
__device__ __forceinline__ size_t row_bytes(int Kt) { return (size_t)4 * Kt * kTileBytes4 + kFlagBytes; }
__device__ __forceinline__ const uint8_t* tile_at(const uint8_t* q, int64_t row64, int t, int Kt) {
  return q + row64 * row_bytes(Kt) + (size_t)t * Kt * kTileBytes4;
}
__device__ __forceinline__ int holds_8(const uint8_t* q, int64_t row64, int Kt) {
  return eng::ld_uniform(reinterpret_cast<const int*>(q + row64 * row_bytes(Kt) + (size_t)4 * Kt * kTileBytes4), 0);
}
constexpr unsigned kSaysK = 0x4b000000u;   // ahead of K in that word; without it K is not said
__device__ __forceinline__ unsigned says_K(const uint8_t* q, int64_t row64, int Kt) {
  return (unsigned)eng::ld_uniform(reinterpret_cast<const int*>(q + row64 * row_bytes(Kt) + (size_t)4 * Kt * kTileBytes4), 1);
}
// x has another number of inputs than the weight was laid out for: y is NaN then. (Compared behind the products, so that
// nothing waits for the word ahead of them.)
__device__ __forceinline__ bool other_K(unsigned says, int K) {
  return (says & 0xff000000u) == kSaysK && says != (kSaysK | (unsigned)K);
}
__device__ __forceinline__ f32x4 nan4() {
  const float v = __builtin_nanf("");
  return f32x4{v, v, v, v};
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

// Once for a weight: 128 x 1536 x 4096 from bf16 530 us (3.8 TB/s), 4096 x 4096 17 us, laid out from bytes 486 and 16.
// KIND 0: bf16, 1: fp32, 2: signed bytes with bf16 scales. A workgroup takes 64 channels, a wave one of their tiles, every
// fourth column of it; with few channels y workgroups share them, and each wave takes every 4 y-th column (values of
// 4096 x 4096 laid out in 16 us, by one workgroup to the channels in 42). Lane 16 h + c takes inputs 32 i + 8 h + j, i < 4, j < 8.
constexpr int kPackWaves = 16;
constexpr int kPackGrid = 1 << 21;   // workgroups along x at most, the rest along z

// The words behind the channels, that of -8 still 0, ahead of y > 1 workgroups that may find one.
__global__ __launch_bounds__(256) void k_int4_none(uint8_t* q, int64_t n, int K) {
  const int64_t r = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int Kt = (K + kTileK - 1) / kTileK;
  if (r < n) *reinterpret_cast<uint4*>(q + (r + 1) * row_bytes(Kt) - kFlagBytes) = make_uint4(0u, kSaysK | (unsigned)K, 0u, 0u);
}

template <int KIND>
__global__ __launch_bounds__(kPackWaves * 64) void k_int4_pack(const void* __restrict__ in, const uint16_t* __restrict__ sin, int64_t rows,
                                                   int N, int K, int group, uint8_t* __restrict__ q,
                                                   uint16_t* __restrict__ sout) {
  const int t = (threadIdx.x >> 6) & 3, lane = threadIdx.x & 63, c = lane & 15, h = lane >> 4;
  const int Kt = (K + kTileK - 1) / kTileK;
  const int per = group / 32, ng = 4 / per;     // steps of 32 inputs in a group, groups of a tile
  // over the weights (a dimension of a grid holds less than 2^32 threads; a loop here costs registers and a quarter of the time)
  const int64_t row64 = (int64_t)blockIdx.z * kPackGrid + blockIdx.x;
  if (row64 >= rows) return;
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
  if (KIND == 2 && gridDim.y > 1) {
    if (threadIdx.x == 0 && any) atomicOr(flag, 1u);
  } else if (blockIdx.y == 0 && threadIdx.x < kFlagBytes / 4) {
    flag[threadIdx.x] = threadIdx.x == 0 ? any != 0 : threadIdx.x == 1 ? kSaysK | (unsigned)K : 0u;
  }
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
  unsigned says, says_next;
  auto at = [&] {
    const int64_t row64 = (int64_t)g * (Nt / 4) + nt / 4;
    pq = tile_at(p.q, row64, nt % 4, Kt);
    ps = static_cast<const uint16_t*>(p.s) + scale_at(row64, Kt, 0, nt % 4, NS);
    eights_next = holds_8(p.q, row64, Kt);
    says_next = says_K(p.q, row64, Kt);
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
    says = says_next;
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
    if (other_K(says, p.K)) acc = nan4();
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
  unsigned says, says_next;
  auto at = [&] {
    const int64_t row64 = (int64_t)g * (Nt / 4) + nt / 4;
    pq = tile_at(p.q, row64, nt % 4, Kt);
    ps = static_cast<const uint16_t*>(p.s) + scale_at(row64, Kt, 0, nt % 4, NS);
    eights_next = holds_8(p.q, row64, Kt);
    says_next = says_K(p.q, row64, Kt);
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
    says = says_next;
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
    if (other_K(says, p.K))
#pragma unroll
      for (int t = 0; t < TL; ++t)
        acc[t] = nan4();
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
// k_int4_tile: WM x WN waves of MI x NJ blocks of 16 x 16, K in stages of 64 inputs, for products whose tiles hide what a
// stage waits for; a wave's tile as large as its registers allow, as each number is unpacked once for it. Unpacking into LDS,
// once for the workgroup, took 312 us (16384 x 4096 x 2048) where this took 299. x comes into LDS by direct loads, two stages
// of it in rows of 128 bytes; each wave unpacks its own channels' numbers into fragments, those of the next stage behind the
// last products of this one. A stage's sums (PER = 1: its halves') start from zero and are added to the accumulators times
// their scales, a row block later than they are made, so that the matrix cores have work meanwhile.
constexpr int kRowB = 128;   // bytes of a row in a stage

// The 16-byte chunk c of row r lies in slot c ^ swz_x(r): 16 consecutive rows at one chunk, which a fragment read
// takes, stand in distinct banks.
__device__ __forceinline__ int swz_x(int r) { return (r >> 1) & 7; }

// eng::gl2lds from a uniform address and a lane's offset
__device__ __forceinline__ void gl2lds_at(const void* base, unsigned off, char* lds) {
  const unsigned to = __builtin_amdgcn_readfirstlane((unsigned)(uintptr_t)lds);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(off), "s"(base) : "memory", "m0");
}

// 4 bytes a lane
__device__ __forceinline__ void gl2lds4_at(const void* base, unsigned off, char* lds) {
  const unsigned to = __builtin_amdgcn_readfirstlane((unsigned)(uintptr_t)lds);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(to), "v"(off), "s"(base) : "memory", "m0");
}

// NJ neighbouring channels of a row from n on, at element `at` of y; wide: all at once
template <int NJ, class F>
__device__ __forceinline__ void store_channels(const I4Params& p, size_t at, int n, bool wide, const F& v) {
  if (wide) {
    if (n >= p.N) return;
    if (p.f32) {
      float* o = static_cast<float*>(p.y) + at;
      if constexpr (NJ == 4) *reinterpret_cast<f32x4*>(o) = f32x4{v(0), v(1), v(2), v(3)};
      else *reinterpret_cast<float2*>(o) = make_float2(v(0), v(1));
    } else {
      alignas(8) bf16 b[NJ];
#pragma unroll
      for (int j = 0; j < NJ; ++j) b[j] = (bf16)v(j);
      bf16* o = static_cast<bf16*>(p.y) + at;
      if constexpr (NJ == 4) *reinterpret_cast<uint2*>(o) = *reinterpret_cast<const uint2*>(b);
      else *reinterpret_cast<unsigned*>(o) = *reinterpret_cast<const unsigned*>(b);
    }
  } else {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      if (n + j >= p.N) continue;
      if (p.f32) static_cast<float*>(p.y)[at + j] = v(j);
      else static_cast<bf16*>(p.y)[at + j] = (bf16)v(j);
    }
  }
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
    const unsigned says = says_K(p.q, row64, Kt);
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
    if (other_K(says, p.K))
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = nan4();
    eng::wait_vm<0>();
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = r0 + 16 * (MI * wm + i) + 4 * h + e;
        if (r >= end) continue;
        store_channels<NJ>(p, (size_t)r * p.N + n1, n1, wide, [&](int j) { return acc[i][j][e]; });
      }
  }
}

// ------------------------------------------------------------------------------------------------
// k_int4_deep: 64 rows by 64 channels, stages of 128 inputs. x, the words of q and the scales go straight into LDS, so
// that no load's latency stands between a stage's products; 4 waves of 2 x 2 blocks. KG = 2 groups of them share the inputs of
// a tile, where there is no more than a tile for a CU, and their sums meet in LDS; with more tiles three workgroups of KG = 1
// share a CU. WIDE: 64 rows by 128 channels, 4 waves of 4 x 2 blocks side by side, which unpack each number once instead of
// twice, two workgroups a CU, where there are so many. Bound by the unpacking and the matrix instructions together, 0.35 us
// a stage of 64 channels and CU (WIDE: 0.29). 256 rows of 4096 x 4096 17 us (KG = 1 21; in stages of 64 inputs with q and
// scales in registers 33), 4096 rows in 64 groups of 1536 x 4096 62 us with 64 rows
// each and 82 with about 64 (64 channels 99, in registers 157). Three stages in
// LDS, the next one's fragments in registers ahead of time, or 64 x 128 tiles of 2 x 4 blocks took as long or longer (256
// rows 17.5, 18.2 and 24 to 28 us).
template <int PER, int KG, bool WIDE>
__global__ __launch_bounds__(256 * KG, KG == 2 ? 1 : WIDE ? 2 : 3) void k_int4_deep(I4Params p) {
  constexpr int BM = 64, XB = BM * 2 * kTileK, NS = 4 / PER, R = WIDE ? 2 : 1, MI = 2 * R, NJ = 2,
                QB = 4 * R * kTileBytes4, SB = 1024, ST = XB + QB + SB;
  __shared__ __attribute__((aligned(1024))) char smem[KG * 2 * ST];
  __shared__ Groups groups;
  const int lane = threadIdx.x & 63, w = eng::wave_id() % 4, kg = eng::wave_id() / 4, wn = w % 2, c = lane & 15, h = lane >> 4;
  const int wm = WIDE ? 0 : w / 2, wr = WIDE ? w / 2 : 0;   // the wave's rows and 64 channels
  char* own = smem + kg * 2 * ST;   // the group's stages
  const int R64 = rows64(p.N), ntn = (R64 + R - 1) / R, Kt = (p.K + kTileK - 1) / kTileK;
  const bool wide = p.N % NJ == 0 && reinterpret_cast<uintptr_t>(p.y) % (NJ * (p.f32 ? 4 : 2)) == 0;
  const int mtiles = group_tiles<BM>(p, groups);
  const XcdRange xr = xcd_range(mtiles * ntn);
  for (int tile = xr.first; tile < xr.end; tile += xr.stride) {
    const int mt = tile / ntn, n64 = (tile - mt * ntn) * R;
    int g, r0, end;
    find_tile<BM>(p, groups, mt, g, r0, end);
    const char* xb = reinterpret_cast<const char*>(static_cast<const bf16*>(p.x) + (size_t)r0 * p.K);
    // A row's 16 chunks of a stage: chunk b of row r lies in slot b ^ (r % 16). This lane moves rows 16 w + 4 j + lane / 16.
    const unsigned K2 = 2u * (unsigned)p.K, x0 = K2 * (16 * w + (lane >> 4)), xlast = K2 * min(end - 1 - r0, BM - 1);
    const unsigned b0 = (lane & 15) ^ (lane >> 4);
    // 64 channels of the tile (behind the last of all: those again, for nothing)
    auto row64 = [&](int r) { return (int64_t)g * R64 + min(n64 + r, R64 - 1); };
    const uint16_t* ps = static_cast<const uint16_t*>(p.s) + scale_at(row64(wr), Kt, 0, 0, NS);
    // Inputs beyond K have zero weights; read for them is another chunk of the same row.
    auto issue = [&](int st, char* to) {
      const char* at = xb + (size_t)st * 2 * kTileK;
      const unsigned last = min(kTileK, p.K - st * kTileK) / 8 - 1;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        gl2lds_at(at, min(x0 + 4 * j * K2, xlast) + 16 * min(b0 ^ (4 * j), last), to + (4 * w + j) * 1024);
#pragma unroll
      for (int r = 0; r < R; ++r)
        gl2lds_at(tile_at(p.q, row64(r), w, Kt) + (size_t)st * kTileBytes4, 16 * lane, to + XB + (4 * r + w) * 1024);
      // 128 NS bytes, over and over
      gl2lds4_at(ps + (size_t)st * 64 * NS, (4 * lane + 256 * wn) & (128 * NS - 1), to + XB + QB + w * 256);
    };
    const int eights = holds_8(p.q, row64(wr), Kt);
    const unsigned says = says_K(p.q, row64(wr), Kt);
    using Scales = Scales4<NJ * NS>;
    f32x4 acc[MI][NJ];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    eng::block_sync();   // every wave is done reading the previous tile's stages
    // the group's stages are kg, kg + KG, .. of K, in two places in turn
    if (kg < Kt) issue(kg, own);
    auto columns = [&](auto with8) {
      int place = 0;
      for (int st = kg; st < Kt + kg; st += KG) {   // (as often in each group)
        eng::wait_vm<0>();
        eng::block_sync();
        const char* at = own + place;
        place ^= ST;
        if (st + KG < Kt) issue(st + KG, own + place);
        if (KG > 1 && st >= Kt) break;
        uint4 q[NJ], fa[MI][4];
#pragma unroll
        for (int j = 0; j < NJ; ++j) q[j] = ld16(at + XB + (4 * wr + 2 * wn + j) * 1024 + 16 * lane);
        const Scales sc = *reinterpret_cast<const Scales*>(at + XB + QB + 512 * wr + (4 * c + 2 * wn) * NS * 2);
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int s = 0; s < 4; ++s) fa[i][s] = ld16(at + (32 * wm + 16 * i + c) * 256 + 16 * ((4 * s + h) ^ c));
#pragma unroll
        for (int a = 0; a < NS; ++a) {
          f32x4 part[MI][NJ];
#pragma unroll
          for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j) part[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int s = a * PER; s < (a + 1) * PER; ++s)
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
              Bytes8 v = bytes8(s == 0 ? q[j].x : s == 1 ? q[j].y : s == 2 ? q[j].z : q[j].w);
              if constexpr (decltype(with8)::value) v = {with_8(v.a), with_8(v.b)};
              const uint4 f = numbers8(v);
#pragma unroll
              for (int i = 0; i < MI; ++i) mma16<bf16>(part[i][j], fa[i][s], f);
            }
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            const float sf = sc[j * NS + a];
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(sf, part[i][j][e], acc[i][j][e]);
          }
        }
      }
    };
    if (eights) columns(std::true_type{});
    else columns(std::false_type{});
    if (other_K(says, p.K))
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = nan4();
    // of KG = 2 groups, each stores a row block of its waves: the other's sums of it come through LDS
    static_assert(KG == 1 || (KG == 2 && !WIDE), "");
    if constexpr (KG == 2) {
      eng::block_sync();
      f32x4* red = reinterpret_cast<f32x4*>(smem) + (w * 2 * 64 + lane) * NJ;
#pragma unroll
      for (int j = 0; j < NJ; ++j) red[kg * 64 * NJ + j] = kg ? acc[0][j] : acc[1][j];
      eng::block_sync();
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const f32x4 o = red[(1 - kg) * 64 * NJ + j];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[0][j][e] = (kg ? acc[1][j][e] : acc[0][j][e]) + o[e];
      }
    }
    const int n1 = 64 * (n64 + wr) + 4 * c + 2 * wn;
#pragma unroll
    for (int i = 0; i < MI / KG; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = r0 + 32 * wm + 16 * (i + kg) + 4 * h + e;
        if (r >= end) continue;
        store_channels<NJ>(p, (size_t)r * p.N + n1, n1, wide, [&](int j) { return acc[i][j][e]; });
      }
  }
}

// Tiles of bm rows by bn columns; for groups, whose sizes the host does not know, as many as evenly spread ones have.
int64_t tiles4(const I4Params& p, int bm, int bn) {
  const int64_t groups = std::min<int64_t>(p.G, p.M);
  const int64_t m = p.offsets ? std::max(groups, p.M / bm + groups / 2) : (p.M + bm - 1) / bm;
  return m * ((p.N + bn - 1) / bn);
}

// The kernel by the rows of a group that has any, as far as the host knows, and by how much work there is. In us, R:
// rows with TL = 4 (1: with TL = 1), D, DD, DW: deep, with two groups of waves, WIDE, 128, 256: tiles of 128 x 128 and
// 256 x 128; W: the work in units of 16 rows by 64 channels, on 256 CUs.
//   rows of 4096 x 4096      16 (W 64): 1 8.4, R 10.2    64 (256): R 10.7, DD 15.3   128 (512): R 16.6, DD 15.7
//                            256: DD 17, D 21, 128 42    512: D 27, DD 30, DW 26     1024: D 49, DW 41, 128 46
//                            1536: DW 57, 128 67         2048: DW 79, 128 72, 256 79
//   rows of 1536 x 4096      64 (96): 1 12.8, R 10.1     192 (288): R 15.3, DD 15.8  384 (576): R 21, DD 16
//                            2048: D 37, DW 39, 128 45, 256 70
//   rows of 16384 x 2048     256: D 25, DW 23, 128 26    512: DW 43, 128 40, 256 42  768: DW 63, 128 57, 256 64
//                            1024: DW 81, 128 78, 256 69
//   64 groups, 1536 x 4096   of 8 rows: R 43, DW 60      16: R 60, DW 55   40: D 69, DW 57, 128 93   64: D 101, DW 82, 128 99
//                            80: DW 104, 128 107         100: DW 109, 128 115
//   128 groups, 768 x 2048   of 8 rows: R 30, DW 32      16: R 44, DW 32   40: D 39, DW 34, 128 50   64: D 56, DW 49, 128 51
//                            80: DW 61, 128 52           100: DW 63, 128 54
//   16 groups, 768 x 2048    of 4 rows (240): 1 9.4, R 8.1   128: D 16, 128 25
// One row of 32768 x 4096 (W 512): 1 17, R 14; 16384 rows of 2048 x 768 in 64 groups: 256 63, 128 69.
// These are with groups of 128 inputs and of evenly drawn rows. Groups of 64 and of 32 inputs take 1.1 and 1.25 times as long
// in all kernels alike (1024 rows of 4096 x 4096: DW 38, 42, 47), and the choice is within 10 % of the best kernel but for few
// rows each (208 in 16 groups of 768 x 2048: DD 11, R 9; 1500 in 128: R 34, DW 30). The host knows the mean of the groups' rows
// alone: where they differ much it chooses too large a tile. With groups drawn by odds 1 / e^1.1, of 1536 x 4096 in 64 groups
// 4608 rows: DW 99, 128 139, 12288: DW 191, 256 266; of 768 x 2048 in 128 groups 24576: DW 96, 256 140; by 1 / e^2, 1500: R 27,
// DW 22. Evenly drawn, 16384 rows of the first take DW 251, 256 273.
template <int PER>
void launch4(const I4Params& p, int grid, hipStream_t s) {
  const int64_t groups = std::min<int64_t>(p.M, p.G);
  const int64_t mt = p.offsets ? p.M / kRows4 + groups : (p.M + kRows4 - 1) / kRows4;
  const int64_t work = mt * rows64(p.N);        // 16 rows by 64 channels
  const int Kt = (p.K + kTileK - 1) / kTileK;
  if (p.M <= 12 * groups || 8 * work <= 9 * grid) {
    auto go = [&](auto kernel, int TL) {
      // fewer waves a task where their columns would make less than a unit, as long as every CU keeps its workgroups
      const int64_t wgs = rows_wgs(PER) * grid;
      int wk = kRowWaves;
      while (wk > 1 && Kt < kUnit * wk && 4 * work * wk / kRowWaves >= 2 * wgs) wk /= 2;
      const int64_t tasks = (4 * work * wk / TL + kRowWaves - 1) / kRowWaves;
      kernel<<<(unsigned)std::min(tasks, wgs), kRowWaves * 64, 0, s>>>(p, wk);
    };
    if (work <= (p.M <= kFew4 * groups ? 3 * grid / 4 : 5 * grid / 16)) go(k_int4_rows<PER, 1>, 1);
    else go(k_int4_rows<PER, 4>, 4);
  } else if (p.M >= 192 * groups && 4 * tiles4(p, 256, 128) >= 7 * grid) {
    k_int4_tile<8, 4, 2, 2, PER><<<2 * grid, 256, 0, s>>>(p);
  } else if (p.M >= 72 * groups && tiles4(p, 128, 128) >= 2 * grid) {
    k_int4_tile<4, 4, 2, 2, PER><<<2 * grid, 256, 0, s>>>(p);
  } else if (tiles4(p, 64, 128) >= 2 * grid) {
    k_int4_deep<PER, 1, true><<<2 * grid, 256, 0, s>>>(p);
  } else if (tiles4(p, 64, 64) <= grid) {
    k_int4_deep<PER, 2, false><<<grid, 512, 0, s>>>(p);
  } else {
    k_int4_deep<PER, 1, false><<<3 * grid, 256, 0, s>>>(p);
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
  const int64_t tiles = (int64_t)G * rows64(N);   // up to 2^23
  const int Kt = (K + kTileK - 1) / kTileK, columns = (Kt + kPackWaves / 4 - 1) / (kPackWaves / 4), few = 2 * persistent_grid(1);
  const dim3 grid((unsigned)std::min<int64_t>(tiles, kPackGrid),
                  (unsigned)std::min<int64_t>(columns, std::max<int64_t>(few / tiles, 1)),
                  (unsigned)((tiles + kPackGrid - 1) / kPackGrid));
  if (scales && grid.y > 1) k_int4_none<<<(unsigned)((tiles + 255) / 256), 256, 0, s>>>(q, tiles, K);
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
