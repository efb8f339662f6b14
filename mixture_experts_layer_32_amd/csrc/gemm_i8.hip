// 8-bit integer grouped GEMM on v_mfma_i32_32x32x32_i8 and the two expert products of the 8-bit layer.
//
// Products and sums are exact: |q p| <= 127^2, and K <= 131072 keeps the int32 sums below 2^31. The
// scales of a row and of a channel multiply the finished sum in fp32, once.
//
// Two engines, both on K-major operands in K-tiles of 128 elements (128 bytes a row: whole lines) that
// reach LDS by direct-to-LDS loads:
//
//  k_i8_256   a persistent workgroup of 8 waves computes 256 x 256 tiles. A wave owns 64 x 128 of one as
//             2 x 4 blocks of 32 x 32 (128 accumulators). A ring of two 64 KB stages; a K-tile is four
//             MFMA steps of 32 elements, each step's fragments (6 reads of 1 KB per wave) read while the
//             previous step's 8 MFMAs run. A tile of up to 128 rows runs half of them.
//             16384 x 4096 x 2048 in 128-146 us by card and run (149 and 154 in the median of two traces), 1.8-2.1 Pop/s,
//             the matrix cores busy half of the cycles at 1.95 GHz; the products of 65536 pairs with K = 768 in 172-187 us,
//             1.15 Pop/s. Bound by the main loop (2.4 Pop/s
//             alone) and the stores, which run at the write rate and which nothing overlaps: without them 114 and
//             138 us, without the loads 120 and 154. Tried against that: the next tile's first K-tiles ahead of the
//             stores (no gain); two workgroups of 4 waves a CU on 128 x 256 tiles (148 and 208 us: half as many
//             rows again to load); starting the CUs at different times (133 and 182 us).
//  k_i8_tile  64 x 64 or 128 x 128 tiles, one or two workgroups of 4 waves a CU, for products with too few tiles of
//             256 x 256 to fill the chip. Bound by latency: 10 us for 1117 x 777 x 1104.
//
// Epilogues store straight from the accumulators, in whole lines and without LDS: the B rows of a tile are
// placed in LDS so that the 4 column blocks of a lane are 4 neighbouring channels of one row (256 bytes of
// bf16 per row and instruction). Staging the rows in LDS instead took 68 us of the 239 us of the down product
// of 65536 pairs, the matrix cores idle.
//
// The contraction may end inside a K-tile (K is a multiple of 16): the missing 16-byte chunks of A are
// read from a page of zeros, those of B from the row's start (their products are zero).
#include <algorithm>
#include <type_traits>

#include "engine.h"
#include "group_tiles.h"
#include "int8_device.h"
#include "moe_internal.h"

namespace moe {
namespace {

using namespace eng;

typedef int i32x16 __attribute__((ext_vector_type(16)));

constexpr int KT8 = 128;                       // elements (bytes) of a row per K-tile
constexpr int OPB = 32768;                     // bytes per operand per stage (256 rows)
constexpr int STB = 2 * OPB;
constexpr int RING = 2 * STB;

// What a kernel computes: y = sums times scales as bf16 or fp32, or the gate/up half of the layer,
// h = w silu(a) b in fp32 (the row quantiser reads it next: its scale needs the whole row) from tiles of
// half as many gate rows and the same up rows of the weights, with gathered x rows.
enum Out { kBf16, kF32, kGateUp };

__device__ __attribute__((aligned(128))) unsigned g_zero16[4];   // never written

// lane i copies 4 bytes from g into lds + 4 i (lds wave-uniform); see gl2lds
__device__ __forceinline__ void gl2lds4(const void* g, char* lds) {
  const unsigned off = __builtin_amdgcn_readfirstlane((unsigned)(uintptr_t)lds);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(off), "v"(g) : "memory", "m0");
}

// 16-byte chunk c of row r of a staged K-tile (engine.h's layout for 128-byte rows)
__device__ __forceinline__ int swz8(int r) { return (r >> 1) & 7; }
__device__ __forceinline__ const char* at8(const char* tile, int r, int c) { return tile + r * KT8 + ((c ^ swz8(r)) << 4); }

// A K-major operand of ROWS rows loaded by NW waves: this lane moves chunk slot lane % 8 of rows
// (w LOADS + j) 8 + lane / 8.
template <int ROWS, int NW>
struct Op8 {
  static constexpr int LOADS = ROWS / (8 * NW);
  const char* p[LOADS];   // the lane's chunk of K-tile 0
  static __device__ __forceinline__ int row_of(int j) { return (wave_id() * LOADS + j) * 8 + (threadIdx.x & 63) / 8; }
  static __device__ __forceinline__ int chunk_of(int j) { return (threadIdx.x & 7) ^ swz8(row_of(j)); }
  // K-tile kt of nk; the last one holds `tail` bytes a row (0: whole), of whose missing chunks `past` is
  // read in place (null: the row's first chunk)
  __device__ __forceinline__ void issue(char* tile, int kt, int nk, int tail, const char* past) const {
    const int w = wave_id();
    if (tail == 0 || kt + 1 < nk) {
#pragma unroll
      for (int j = 0; j < LOADS; ++j) gl2lds(p[j] + (size_t)kt * KT8, tile + (w * LOADS + j) * 1024);
      return;
    }
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      const int c = 16 * chunk_of(j);
      gl2lds(c < tail ? p[j] + (size_t)kt * KT8 : past ? past : p[j] - c, tile + (w * LOADS + j) * 1024);
    }
  }
};

// Which channel of the tile the B row rho of LDS holds. A wave's NJ column blocks are rows 32 NJ wn + 32 j + l
// of LDS (l = lane % 32): channel 32 NJ wn + NJ l + j, so that a lane's blocks are neighbours. kGateUp: the
// first half of the blocks is gate rows and the second the same up rows (one block: lanes 16-31 are the up
// rows of lanes 0-15); `up` says which.
template <Out OUT, int NJ>
__device__ __forceinline__ int channel_of(int rho, bool& up) {
  const int wn = rho / (32 * NJ), j = rho % (32 * NJ) / 32, l = rho % 32;
  up = false;
  if constexpr (OUT != kGateUp) return 32 * NJ * wn + NJ * l + j;
  if constexpr (NJ == 1) {
    up = l >= 16;
    return 16 * wn + (l & 15);
  }
  constexpr int HJ = NJ > 1 ? NJ / 2 : 1;
  up = j >= HJ;
  return 32 * HJ * wn + HJ * l + j % HJ;
}

// The operand pointers of a tile of BM rows from r0 and BN weight rows from channel n0 (kGateUp: half of them
// gate, half up rows) of group g; NJ column blocks per wave.
template <Out OUT, int NJ, int BM, int BN, int NW>
__device__ __forceinline__ void tile_operands(const I8Params& p, int g, int r0, int end, int n0, Op8<BM, NW>& la,
                                              Op8<BN, NW>& lb) {
#pragma unroll
  for (int j = 0; j < Op8<BM, NW>::LOADS; ++j) {
    const int r = min(r0 + Op8<BM, NW>::row_of(j), end - 1);
    const size_t row = OUT == kGateUp ? (size_t)p.ptok[r] : (size_t)r;
    la.p[j] = reinterpret_cast<const char*>(p.x + row * p.K) + 16 * Op8<BM, NW>::chunk_of(j);
  }
#pragma unroll
  for (int j = 0; j < Op8<BN, NW>::LOADS; ++j) {
    bool up;
    const int n = min(n0 + channel_of<OUT, NJ>(Op8<BN, NW>::row_of(j), up), p.N - 1);
    const uint8_t* w = OUT == kGateUp && up ? p.wu : p.w;
    lb.p[j] = reinterpret_cast<const char*>(w + ((size_t)g * p.N + n) * p.K) + 16 * Op8<BN, NW>::chunk_of(j);
  }
}

// ------------------------------------------------------------------------------------------------
// Epilogue of a tile: rows r0 .. end-1 (block i of the wave: rows AST i + 32 wm of the tile, element 4 a + b of
// lane l its row 8 a + 4 (l / 32) + b), channels from n0. sx, wt: the tile rows' scales and routing weights,
// sw: the channels' scales (kGateUp: half of them gate, then as many up), all in LDS.
// Without WIDE the outputs are stored one by one, as any N and any address allow.
// WIDE (N a multiple of 8, y 16-byte aligned): vector stores through a buffer whose range ends behind the
// tile's last row, so that the hardware drops the rows past it, and channels past N at an offset outside. Every
// lane issues every store: no branch between them, and their number is known.
template <Out OUT, bool WIDE, int AST, int MI, int NJ>
__device__ __forceinline__ void epilogue(const I8Params& p, const i32x16 (&acc)[MI][NJ], int r0, int end, int n0,
                                         const float* sx, const float* sw, const float* wt, int wm, int wn, int lane) {
  constexpr int VW = OUT != kGateUp ? NJ : NJ == 4 ? 2 : 1;   // neighbouring channels a lane stores
  constexpr unsigned ES = OUT == kBf16 ? 2 : 4;
  typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
  typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
  const int l = lane & 31, h4 = 4 * (lane >> 5);
  const int c = OUT == kGateUp && NJ == 1 ? 16 * wn + (l & 15) : 32 * VW * wn + VW * l, n = n0 + c;
  float g[VW], u[VW];
#pragma unroll
  for (int v = 0; v < VW; ++v) {
    g[v] = sw[c + v];
    u[v] = OUT == kGateUp ? sw[32 * NJ + c + v] : 0.f;
  }
  const bool mine = n < p.N && (OUT != kGateUp || NJ > 1 || l < 16);
  char* base = static_cast<char*>(p.y) + ((size_t)r0 * p.N + n0) * ES;   // uniform; a tile spans less than 4 GB
  const unsigned ldb = (unsigned)p.N * ES, rows_in = (unsigned)min(end - r0, AST * MI);
  __amdgpu_buffer_rsrc_t rsrc;
  if constexpr (WIDE) rsrc = __builtin_amdgcn_make_buffer_rsrc(base, 0, rows_in * ldb, 0x00020000);
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int rl = AST * i + 32 * wm + h4, rows = end - r0 - rl;   // the lane's row 8 a + b is stored if below
    const unsigned off0 = (unsigned)rl * ldb + (unsigned)c * ES;
    unsigned off = WIDE && !mine ? 0xf0000000u : off0;
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      __builtin_amdgcn_sched_barrier(0);   // (the scales of every row read ahead would spill)
      const float4 s4 = *reinterpret_cast<const float4*>(sx + rl + 8 * a);
      const float s[4] = {s4.x, s4.y, s4.z, s4.w};
      float w[4] = {};
      if constexpr (OUT == kGateUp) {
        const float4 w4 = *reinterpret_cast<const float4*>(wt + rl + 8 * a);
        w[0] = w4.x; w[1] = w4.y; w[2] = w4.z; w[3] = w4.w;
      }
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int q = 4 * a + b;
        float o[VW];
#pragma unroll
        for (int v = 0; v < VW; ++v) {
          if constexpr (OUT != kGateUp) {
            o[v] = (float)acc[i][v][q] * (s[b] * g[v]);
          } else {
            const int us = NJ == 1 ? __shfl_xor(acc[i][0][q], 16) : acc[i][NJ == 1 ? 0 : NJ / 2 + v][q];
            const float ga = (float)acc[i][v][q] * (s[b] * g[v]), up = (float)us * (s[b] * u[v]);
            o[v] = weighted_swiglu8(w[b], ga, up);
          }
        }
        if constexpr (WIDE) {   // aux 2: non-temporal
          if constexpr (OUT == kBf16 && VW == 4) {
            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, pack4(o[0], o[1], o[2], o[3])), rsrc, off, 0, 2);
          } else if constexpr (VW == 4) {
            const u32x4 f = {__float_as_uint(o[0]), __float_as_uint(o[1]), __float_as_uint(o[2]), __float_as_uint(o[3])};
            __builtin_amdgcn_raw_buffer_store_b128(f, rsrc, off, 0, 2);
          } else {
            const u32x2 f = {__float_as_uint(o[0]), __float_as_uint(o[1])};
            __builtin_amdgcn_raw_buffer_store_b64(f, rsrc, off, 0, 2);
          }
          off += b < 3 ? ldb : 5 * ldb;   // rows 8 a + b, then 8 (a + 1)
        } else if (mine && 8 * a + b < rows) {
          char* y = base + off + (unsigned)(8 * a + b) * ldb;
#pragma unroll
          for (int v = 0; v < VW; ++v)
            if (n + v < p.N) {
              if constexpr (OUT == kBf16) reinterpret_cast<bf16*>(y)[v] = (bf16)o[v];
              else reinterpret_cast<float*>(y)[v] = o[v];
            }
        }
      }
    }
  }
}

// ------------------------------------------------------------------------------------------------
// k_i8_256
constexpr int NT256 = 512;                     // 8 waves: 64 x 128 of the tile each
typedef Op8<TILE, 8> Op256;
struct Frag8 {
  i32x4 a[2], b[4];
};

// step s (32 elements) of the K-tile staged at st; row blocks of the wave at am0 and am0 + 128, columns from bn0
template <int MI>
__device__ __forceinline__ void read_frags8(Frag8& f, const char* st, int s, int am0, int bn0, int lane) {
  const int c = 2 * s + (lane >> 5);
#pragma unroll
  for (int i = 0; i < MI; ++i) f.a[i] = *reinterpret_cast<const i32x4*>(at8(st, am0 + 128 * i + (lane & 31), c));
#pragma unroll
  for (int j = 0; j < 4; ++j) f.b[j] = *reinterpret_cast<const i32x4*>(at8(st + OPB, bn0 + 32 * j + (lane & 31), c));
}

// the step's 4 MI MFMAs, each of the first followed in issue order by one of the LDS reads around it
template <int MI>
__device__ __forceinline__ void mma8(i32x16 (&acc)[2][4], const Frag8& f) {
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.a[i], f.b[j], acc[i][j], 0, 0, 0);
#pragma unroll
  for (int q = 0; q < (MI == 2 ? 6 : 4); ++q) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
  }
  if (MI == 2) __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
}

// K-tiles 0 .. nk-1, of which 0 (landed, published) and 1 are issued. Per K-tile: the four steps, each after
// the reads of the next one's fragments; before the last step every wave waits for the next K-tile's
// loads and passes the barrier, and the stage just read is refilled with the K-tile two ahead.
template <int MI, class Issue>
__device__ __forceinline__ void ktiles8(i32x16 (&acc)[2][4], const char* smem, Issue issue, int nk, int am0, int bn0,
                                        int lane) {
  Frag8 f0, f1;
  read_frags8<MI>(f0, smem, 0, am0, bn0, lane);
  for (int kt = 0; kt < nk; ++kt) {
    const char* cur = smem + (kt & 1) * STB;
    read_frags8<MI>(f1, cur, 1, am0, bn0, lane);
    mma8<MI>(acc, f0);
    read_frags8<MI>(f0, cur, 2, am0, bn0, lane);
    mma8<MI>(acc, f1);
    read_frags8<MI>(f1, cur, 3, am0, bn0, lane);
    mma8<MI>(acc, f0);
    wait_vm<0>();
    block_sync();
    if (kt + 2 < nk) issue(kt + 2);
    read_frags8<MI>(f0, smem + ((kt + 1) & 1) * STB, 0, am0, bn0, lane);   // past the last K-tile: unused
    mma8<MI>(acc, f1);
  }
  block_sync();
}

template <Out OUT>
__global__ __launch_bounds__(NT256, 1) void k_i8_256(I8Params p) {
  __shared__ __attribute__((aligned(1024))) char smem[RING];
  __shared__ __attribute__((aligned(16))) float scales[3 * TILE];   // of rows and channels, and routing weights
  __shared__ Groups groups;
  constexpr int BN = OUT == kGateUp ? TILE / 2 : TILE;   // output columns of a tile
  const int tid = threadIdx.x, lane = tid & 63, w = wave_id(), wm = w >> 1, wn = w & 1;
  const int ntn = (p.N + BN - 1) / BN, nk = (p.K + KT8 - 1) / KT8, tail = p.K % KT8;
  const int mtiles = group_tiles<TILE>(p, groups);
  const XcdRange xr = xcd_range(mtiles * ntn);
  if (xr.first >= xr.end) return;
  Op256 la, lb;
  int r0 = 0, end = 0, n0 = 0;
  bool half = false;   // up to 128 rows: the second row blocks, and the loads of waves 4-7's A rows, are left out
  auto issue = [&](int kt) {
    char* st = smem + (kt & 1) * STB;
    if (!half || w < 4) la.issue(st, kt, nk, tail, reinterpret_cast<const char*>(g_zero16));
    lb.issue(st + OPB, kt, nk, tail, nullptr);
  };
  // tile `tile`: its operands, its scales into LDS and its first two K-tiles
  auto begin = [&](int tile) {
    const int mt = tile / ntn;
    int g;
    n0 = (tile - mt * ntn) * BN;
    find_tile<TILE>(p, groups, mt, g, r0, end);
    half = end - r0 <= 128;
    tile_operands<OUT, 4, TILE, TILE, 8>(p, g, r0, end, n0, la, lb);
    char* sc = reinterpret_cast<char*>(scales) + (w & 3) * 256;
    const int t = tid & 255;
    if (w < 4) {
      const int r = min(r0 + t, end - 1);
      if constexpr (OUT == kGateUp) gl2lds4(p.weight + p.perm[r], sc + 8 * TILE);
      gl2lds4(p.xs + (OUT == kGateUp ? p.ptok[r] : r), sc);
    } else {
      const bool up = OUT == kGateUp && t >= BN;
      gl2lds4((up ? p.wsu : p.ws) + (size_t)g * p.N + min(n0 + (up ? t - BN : t), p.N - 1), sc + 4 * TILE);
    }
    issue(0);
    if (nk > 1) issue(1);
  };
  for (int tile = xr.first; tile < xr.end; tile += xr.stride) {
    i32x16 acc[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][j][q] = 0;
    begin(tile);
    wait_vm<0>();
    block_sync();
    if (half) ktiles8<1>(acc, smem, issue, nk, 32 * wm, 128 * wn, lane);
    else ktiles8<2>(acc, smem, issue, nk, 32 * wm, 128 * wn, lane);
    const float* sc = scales;
    epilogue<OUT, true, 128>(p, acc, r0, end, n0, sc, sc + TILE, sc + 2 * TILE, wm, wn, lane);
    block_sync();   // every wave has read its scales
  }
}

// ------------------------------------------------------------------------------------------------
// k_i8_tile: persistent, MI x NJ blocks per wave, 2 x 2 waves, a ring of S stages with one barrier each: after it the
// stage read in the previous K-tile is refilled with the K-tile S - 1 ahead.
template <Out OUT, int MI, int NJ, int S>
__global__ __launch_bounds__(NTHR, 2) void k_i8_tile(I8Params p) {
  constexpr int BM = 64 * MI, BN = 64 * NJ, ST = (BM + BN) * KT8, NL = Op8<BM, 4>::LOADS + Op8<BN, 4>::LOADS;
  constexpr int BC = OUT == kGateUp ? BN / 2 : BN;   // output columns of a tile
  __shared__ __attribute__((aligned(1024))) char smem[S * ST];
  __shared__ __attribute__((aligned(16))) float sx[BM], sw[BN], wt[BM];
  __shared__ Groups groups;
  const int tid = threadIdx.x, lane = tid & 63, w = wave_id(), wm = w >> 1, wn = w & 1;
  const int ntn = (p.N + BC - 1) / BC, nk = (p.K + KT8 - 1) / KT8, tail = p.K % KT8;
  const int mtiles = group_tiles<BM>(p, groups);
  const XcdRange xr = xcd_range(mtiles * ntn);
  for (int tile = xr.first; tile < xr.end; tile += xr.stride) {
    const int mt = tile / ntn, n0 = (tile - mt * ntn) * BC;
    int g, r0, end;
    find_tile<BM>(p, groups, mt, g, r0, end);
    Op8<BM, 4> la;
    Op8<BN, 4> lb;
    tile_operands<OUT, NJ>(p, g, r0, end, n0, la, lb);
    auto issue = [&](int kt) {
      char* st = smem + (kt % S) * ST;
      la.issue(st, kt, nk, tail, reinterpret_cast<const char*>(g_zero16));
      lb.issue(st + BM * KT8, kt, nk, tail, nullptr);
    };
    block_sync();   // every wave is done with the previous tile's scales
    if (tid < BM) {
      const int r = min(r0 + tid, end - 1);
      sx[tid] = p.xs[OUT == kGateUp ? p.ptok[r] : r];
      if constexpr (OUT == kGateUp) wt[tid] = p.weight[p.perm[r]];
    }
    if (tid < BN) sw[tid] = (OUT == kGateUp && tid >= BC ? p.wsu : p.ws)[(size_t)g * p.N + min(n0 + tid % BC, p.N - 1)];
    wait_vm<0>();   // the compiler's own loads, and the previous tile's stores, do not count against the ring below
#pragma unroll
    for (int q = 0; q < S - 1; ++q)
      if (q < nk) issue(q);
    i32x16 acc[MI][NJ];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][j][q] = 0;
    for (int kt = 0; kt < nk; ++kt) {
      const int younger = min(S - 2, nk - 1 - kt);   // K-tiles issued after kt
      if (S > 3 && younger >= 2) wait_vm<2 * NL>();
      else if (S > 2 && younger == 1) wait_vm<NL>();
      else wait_vm<0>();
      block_sync();
      if (kt + S - 1 < nk) issue(kt + S - 1);
      const char* st = smem + (kt % S) * ST;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int c = 2 * s + (lane >> 5);
        i32x4 fa[MI], fb[NJ];
#pragma unroll
        for (int i = 0; i < MI; ++i) fa[i] = *reinterpret_cast<const i32x4*>(at8(st, 64 * i + 32 * wm + (lane & 31), c));
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          fb[j] = *reinterpret_cast<const i32x4*>(at8(st + BM * KT8, 32 * (NJ * wn + j) + (lane & 31), c));
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int j = 0; j < NJ; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa[i], fb[j], acc[i][j], 0, 0, 0);
      }
    }
    epilogue<OUT, false, 64>(p, acc, r0, end, n0, sx, sw, wt, wm, wn, lane);
    block_sync();   // every wave is done reading the ring
  }
}

// Tiles of bm rows by bn columns for `rows` rows in as many groups as the product may have.
int64_t tiles(const I8Params& p, int64_t rows, int bm, int bn) {
  const int64_t m = rows / bm + (p.offsets ? std::min<int64_t>(p.G, rows) : 1);
  return std::min<int64_t>(m, rows) * ((p.N + bn - 1) / bn);
}

// 256 x 256 tiles once the expected rows make enough to fill three quarters of the CUs, else 128 x 128 ones if
// they do, else 64 x 64. 1117 x 777 x 1104 in 9 groups: 55 us on 256 x 256, 10 us on 64 x 64. The products of
// 1333 tokens on 16 of 128 experts (2048 x 768): 28 and 14 us on 256 x 256, 18 and 12 us on 128 x 128.
// 256 x 256 tiles need the vector stores (`wide`); other N and addresses stay on the small tiles, which store any. 16384 x
// 2048 by 4104 and by 4100 channels, bf16: 156 and 236 us (4104 into an odd address 232), fp32 172 and 279; 65536 x 768 by 2048
// and by 2044: 123 and 249, fp32 154 and 294; 4096 rows of 2048 channels: 32 and 31 us.
template <Out OUT>
void launch_i8(const I8Params& p, int grid, hipStream_t s) {
  constexpr int half = OUT == kGateUp ? 2 : 1;
  const int64_t rows = std::max<int64_t>(1, p.expect);
  const bool wide = p.N % 8 == 0 && (reinterpret_cast<uintptr_t>(p.y) & 15) == 0;
  if (wide && 4 * tiles(p, rows, 256, 256 / half) >= 3 * grid) {
    k_i8_256<OUT><<<grid, NT256, 0, s>>>(p);
  } else if (4 * tiles(p, rows, 128, 128 / half) >= 3 * grid) {
    k_i8_tile<OUT, 2, 2, 3><<<grid, NTHR, 0, s>>>(p);
  } else {
    k_i8_tile<OUT, 1, 1, 4><<<2 * grid, NTHR, 0, s>>>(p);
  }
}

}  // namespace

hipError_t launch_int8_matmul(const I8Params& p, int grid, const char* name, hipStream_t s) {
  prof_mark_begin(name, s);
  if (p.wu) launch_i8<kGateUp>(p, grid, s);
  else if (p.f32) launch_i8<kF32>(p, grid, s);
  else launch_i8<kBf16>(p, grid, s);
  const hipError_t err = hipGetLastError();
  if (err == hipSuccess) prof_mark_end(s);
  return err;
}

}  // namespace moe
