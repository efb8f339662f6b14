// 8-bit integer grouped GEMM on v_mfma_i32_32x32x32_i8 and the two expert products of the 8-bit layer.
//
// Products and sums are exact: |q p| <= 127^2, and K <= 131072 keeps the int32 sums below 2^31. The
// scales of a row and of a channel multiply the finished sum in fp32, once.
//
// The engine is the K-major one of engine.h: a workgroup of 4 waves computes a 256 x 256 tile, a wave
// 128 x 128 of it as 4 x 4 blocks of 32 x 32 (256 accumulators). A K-tile is 128 elements, 128 bytes a
// row (whole lines), loaded straight into LDS through a ring of two 64 KB stages. It is four
// MFMA steps of 32 elements; each step's fragments (8 reads of 1 KB per wave) are read while the
// previous step's 16 MFMAs run. Four waves of 128 x 128 read 64 bytes of LDS per clock at the full MFMA
// rate, eight waves of 64 x 128 would read 96 beside the 32 the loads write, of 128 in all.
// The contraction may end inside a K-tile (K is a multiple of 16): the missing 16-byte chunks of A are
// read from a page of zeros, those of B from the row's start (their products are zero).
#include "engine.h"
#include "int8_device.h"
#include "moe_internal.h"

namespace moe {
namespace {

using namespace eng;

typedef int i32x16 __attribute__((ext_vector_type(16)));

constexpr int KT8 = 128;                       // elements (bytes) of a row per K-tile
typedef KRows<128> KOp;
constexpr int LOADS = KOp::LOADS;              // 8 loads per lane per operand per K-tile
constexpr int OPB = 32768;                     // bytes per operand per stage
constexpr int STB = 2 * OPB;
constexpr int SMEM_I8 = 2 * STB > 4 * SLAB * 4 ? 2 * STB : 4 * SLAB * 4;

__device__ __attribute__((aligned(128))) unsigned g_zero16[4];   // never written

// a K-major operand whose last K-tile holds `tail` bytes a row (0: whole)
struct Op8 {
  KOp k;
  const char* past;   // read in place of chunks past the row's end; null: the row's first chunk
  __device__ __forceinline__ void issue(char* tile, int kt, int nk, int tail) const {
    if (tail == 0 || kt + 1 < nk) {
      k.issue(tile, kt);
      return;
    }
    const int w = wave_id();
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      const int c = 16 * KOp::chunk_of(j);
      const char* p = c < tail ? k.p[j] + (size_t)kt * KT8 : past ? past : k.p[j] - c;
      gl2lds(p, tile + (w * LOADS + j) * 1024);
    }
  }
};

struct Frag8 {
  i32x4 a[4], b[4];
};

// step s (32 elements) of the K-tile staged at st
__device__ __forceinline__ void read_frags8(Frag8& f, const char* st, int s, int am0, const int (&bn)[4], int lane) {
  const int c = 2 * s + (lane >> 5);
#pragma unroll
  for (int i = 0; i < 4; ++i) f.a[i] = *reinterpret_cast<const i32x4*>(KOp::at(st, am0 + 32 * i + (lane & 31), c));
#pragma unroll
  for (int j = 0; j < 4; ++j) f.b[j] = *reinterpret_cast<const i32x4*>(KOp::at(st + OPB, bn[j] + (lane & 31), c));
}

// the step's 16 MFMAs (B fragment first: a block holds the transposed 32 x 32 product), each of the
// first eight followed in issue order by one of the LDS reads around it
__device__ __forceinline__ void mma8(i32x16 (&acc)[4][4], const Frag8& f) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.b[j], f.a[i], acc[i][j], 0, 0, 0);
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x008, 8, 0);
}

// nk K-tiles. Per K-tile: the four steps, each after the reads of the next one's fragments; before the
// last step every wave waits for the next K-tile's loads and passes the barrier, and the stage just
// read is refilled with the K-tile two ahead.
__device__ __forceinline__ void mainloop8(i32x16 (&acc)[4][4], char* smem, const Op8& la, const Op8& lb, int nk, int tail,
                                          int am0, const int (&bn)[4]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0;
  wait_vm<0>();   // the previous tile's epilogue stores do not count against the ring below
  block_sync();   // and every wave is done reading its staging slab
  auto issue = [&](int kt) {
    char* st = smem + (kt & 1) * STB;
    la.issue(st, kt, nk, tail);
    lb.issue(st + OPB, kt, nk, tail);
  };
  issue(0);
  if (nk > 1) issue(1);
  if (nk > 1) wait_vm<2 * LOADS>();
  else wait_vm<0>();
  block_sync();
  Frag8 f0, f1;
  read_frags8(f0, smem, 0, am0, bn, lane);
  for (int kt = 0; kt < nk; ++kt) {
    const char* cur = smem + (kt & 1) * STB;
    read_frags8(f1, cur, 1, am0, bn, lane);
    mma8(acc, f0);
    read_frags8(f0, cur, 2, am0, bn, lane);
    mma8(acc, f1);
    read_frags8(f1, cur, 3, am0, bn, lane);
    mma8(acc, f0);
    wait_vm<0>();
    block_sync();
    if (kt + 2 < nk) issue(kt + 2);
    read_frags8(f0, smem + ((kt + 1) & 1) * STB, 0, am0, bn, lane);   // past the last K-tile: unused
    mma8(acc, f1);
  }
  block_sync();
}

// rows 32 i .. 32 i + 31 of the wave's blocks into its slab, as integers
__device__ __forceinline__ void stage8(int* slab, const i32x16 (&acc)[4][4], int i, int lane) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int a = 0; a < 4; ++a)
      *reinterpret_cast<int4*>(slab + (lane & 31) * SLD + 32 * j + acc_n(a, lane)) =
          make_int4(acc[i][j][4 * a], acc[i][j][4 * a + 1], acc[i][j][4 * a + 2], acc[i][j][4 * a + 3]);
}

__device__ __forceinline__ void read8i(const int* slab, int row, int col, float (&v)[8]) {
  const int4 x = *reinterpret_cast<const int4*>(slab + row * SLD + col);
  const int4 y = *reinterpret_cast<const int4*>(slab + row * SLD + col + 4);
  v[0] = (float)x.x; v[1] = (float)x.y; v[2] = (float)x.z; v[3] = (float)x.w;
  v[4] = (float)y.x; v[5] = (float)y.y; v[6] = (float)y.z; v[7] = (float)y.w;
}

// ------------------------------------------------------------------------------------------------
// tiles of the groups: LDS prefix sums of the groups' 256-row tile counts
struct Groups {
  int* tile0;   // [G + 1]
  int* row0;    // [G + 1] clamped offsets
};

__device__ __forceinline__ int clamped_offset(const I8Params& p, int g) { return min(max(p.offsets[g], 0), (int)p.M); }

__device__ __forceinline__ void group_tiles(const I8Params& p, const Groups& s) {
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x, per = (p.G + 63) >> 6, g0 = lane * per;
    int t = 0;
    for (int i = 0; i < per; ++i)
      if (g0 + i < p.G) t += (max(clamped_offset(p, g0 + i + 1) - clamped_offset(p, g0 + i), 0) + TILE - 1) / TILE;
    int inc = t;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(inc, d);
      if (lane >= d) inc += o;
    }
    int at = inc - t;
    for (int i = 0; i < per; ++i) {
      const int g = g0 + i;
      if (g >= p.G) break;
      const int a = clamped_offset(p, g), b = max(clamped_offset(p, g + 1), a);
      s.tile0[g] = at;
      s.row0[g] = a;
      at += (b - a + TILE - 1) / TILE;
    }
    if (lane == 63) s.tile0[p.G] = inc;
  }
  __syncthreads();
}

template <bool F32>
__global__ __launch_bounds__(NTHR, 1) void k_int8_matmul(I8Params p) {
  __shared__ __attribute__((aligned(1024))) char smem[SMEM_I8];
  __shared__ int tile0[kMaxExperts + 1], row0[kMaxExperts + 1];
  const int lane = threadIdx.x & 63, w = wave_id(), wm = w >> 1, wn = w & 1;
  const int ntn = (p.N + TILE - 1) / TILE, nk = (p.K + KT8 - 1) / KT8, tail = p.K % KT8;
  int mtiles = (int)((p.M + TILE - 1) / TILE);
  if (p.offsets) {
    group_tiles(p, Groups{tile0, row0});
    mtiles = tile0[p.G];
  }
  const XcdRange xr = xcd_range(mtiles * ntn);
  const int bn[4] = {128 * wn, 128 * wn + 32, 128 * wn + 64, 128 * wn + 96};
  const bool wide = p.N % 8 == 0 && (reinterpret_cast<uintptr_t>(p.y) & 15) == 0;
  for (int tile = xr.first; tile < xr.end; tile += xr.stride) {
    const int mt = tile / ntn, n0 = (tile - mt * ntn) * TILE;
    int g = 0, r0 = mt * TILE, seg_end = (int)p.M;
    if (p.offsets) {   // the last group whose first tile is not past mt
      int lo = 0, hi = p.G;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tile0[mid] <= mt) lo = mid;
        else hi = mid;
      }
      g = __builtin_amdgcn_readfirstlane(lo);
      r0 = __builtin_amdgcn_readfirstlane(row0[g] + (mt - tile0[g]) * TILE);
      seg_end = __builtin_amdgcn_readfirstlane(max(clamped_offset(p, g + 1), row0[g]));
    }
    Op8 la, lb;
    la.past = reinterpret_cast<const char*>(g_zero16);
    lb.past = nullptr;
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      const int row = KOp::row_of(j), c = KOp::chunk_of(j);
      la.k.p[j] = reinterpret_cast<const char*>(p.x + (size_t)min(r0 + row, seg_end - 1) * p.K) + 16 * c;
      lb.k.p[j] = reinterpret_cast<const char*>(p.w + ((size_t)g * p.N + min(n0 + row, p.N - 1)) * p.K) + 16 * c;
    }
    i32x16 acc[4][4];
    mainloop8(acc, smem, la, lb, nk, tail, 128 * wm, bn);
    // epilogue: 32 rows at a time through the wave's slab, then 8 columns of a row per lane
    int* slab = reinterpret_cast<int*>(wave_slab(smem));
    const int c0 = (lane & 15) * 8, n = n0 + 128 * wn + c0;
    float sw[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) sw[e] = p.ws[(size_t)g * p.N + min(n + e, p.N - 1)];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      stage8(slab, acc, i, lane);
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const int rl = (lane >> 4) + 4 * s, r = r0 + 128 * wm + 32 * i + rl;
        if (r < seg_end && n < p.N) {
          float v[8];
          read8i(slab, rl, c0, v);
          const float sx = p.xs[r];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] *= sx * sw[e];
          const size_t at = (size_t)r * p.N + n;
          if constexpr (F32) {
            float* o = static_cast<float*>(p.y) + at;
            if (wide) {
              st16_nt(o, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])));
              st16_nt(o + 4, make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])));
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (n + e < p.N) o[e] = v[e];
            }
          } else {
            bf16* o = static_cast<bf16*>(p.y) + at;
            if (wide) {
              st16_nt(o, pack8(v));
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (n + e < p.N) o[e] = (bf16)v[e];
            }
          }
        }
      }
    }
  }
}

// ------------------------------------------------------------------------------------------------
// gate/up of the 8-bit layer: a tile is 256 pairs of an expert by 128 columns of F (128 gate rows and the
// same 128 up rows of the weights); x rows are gathered through the routing's token list. The epilogue
// writes h = w silu(a) b in fp32, which the row quantiser then reads: its scale needs the whole row.
__global__ __launch_bounds__(NTHR, 1) void k_gateup_i8(I8LayerParams p) {
  __shared__ __attribute__((aligned(1024))) char smem[SMEM_I8];
  const int lane = threadIdx.x & 63, w = wave_id(), wm = w >> 1, wn = w & 1;
  const int H = p.H, F = p.F, ntn = F / 128;
  const XcdRange xr = xcd_range(*p.num_mtiles2 * ntn);
  const int bn[4] = {64 * wn, 64 * wn + 32, 128 + 64 * wn, 128 + 64 * wn + 32};
  for (int tile = xr.first; tile < xr.end; tile += xr.stride) {
    const int mt = tile / ntn, nt = tile - mt * ntn;
    const int2 me = p.mtile2[mt];
    const int e = me.x, r0 = me.y, seg_end = p.offsets[e + 1];
    Op8 la, lb;
    la.past = lb.past = nullptr;
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      const int row = KOp::row_of(j), c = KOp::chunk_of(j);
      const int r = min(r0 + row, seg_end - 1);
      la.k.p[j] = reinterpret_cast<const char*>(p.xq + (size_t)p.ptok[r] * H) + 16 * c;
      const uint8_t* wrow = row < 128 ? p.wg + ((size_t)e * F + nt * 128 + row) * H
                                      : p.wu + ((size_t)e * F + nt * 128 + row - 128) * H;
      lb.k.p[j] = reinterpret_cast<const char*>(wrow) + 16 * c;
    }
    i32x16 acc[4][4];
    mainloop8(acc, smem, la, lb, H / KT8, 0, 128 * wm, bn);
    int* slab = reinterpret_cast<int*>(wave_slab(smem));
    const int c0 = (lane & 7) * 8, f = nt * 128 + 64 * wn + c0;
    float sg[8], su[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      sg[q] = p.sg[(size_t)e * F + f + q];
      su[q] = p.su[(size_t)e * F + f + q];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      stage8(slab, acc, i, lane);
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int rl = (lane >> 3) + 8 * s, r = r0 + 128 * wm + 32 * i + rl;
        if (r < seg_end) {
          float a[8], b[8], h[8];
          read8i(slab, rl, c0, a);
          read8i(slab, rl, 64 + c0, b);
          const float sx = p.xs[p.ptok[r]], wt = p.weight[p.perm[r]];
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            a[q] *= sx * sg[q];
            b[q] *= sx * su[q];
            h[q] = wt * (a[q] / (1.0f + expf(-a[q])) * b[q]);
          }
          float* o = p.h + (size_t)r * F + f;
          st16_nt(o, make_uint4(__float_as_uint(h[0]), __float_as_uint(h[1]), __float_as_uint(h[2]), __float_as_uint(h[3])));
          st16_nt(o + 4, make_uint4(__float_as_uint(h[4]), __float_as_uint(h[5]), __float_as_uint(h[6]), __float_as_uint(h[7])));
        }
      }
    }
  }
}

}  // namespace

hipError_t launch_int8_matmul(const I8Params& p, int grid, const char* name, hipStream_t s) {
  prof_mark_begin(name, s);
  if (p.f32) k_int8_matmul<true><<<grid, NTHR, 0, s>>>(p);
  else k_int8_matmul<false><<<grid, NTHR, 0, s>>>(p);
  const hipError_t err = hipGetLastError();
  if (err == hipSuccess) prof_mark_end(s);
  return err;
}

hipError_t launch_gateup_i8(const I8LayerParams& p, int grid, hipStream_t s) {
  prof_mark_begin("int8_gateup", s);
  k_gateup_i8<<<grid, NTHR, 0, s>>>(p);
  const hipError_t err = hipGetLastError();
  if (err == hipSuccess) prof_mark_end(s);
  return err;
}

}  // namespace moe
