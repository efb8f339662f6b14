// 8-bit integer rows: the quantiser, and the product for at most 64 rows.
//
// k_int8_quant       one wavefront per row. Rows of up to 4096 elements are held in registers between
//                    the maximum and the conversion, longer ones are read twice (the second time from
//                    L2). Bound by HBM: 2 (4) bytes read and 1 written per bf16 (fp32) element. 65536 x 512
//                    bf16 20.3 us (5.0 TB/s, a copy's rate), 131072 x 768 fp32 88 us (5.7 TB/s), 65536 x 768
//                    bf16 33 us (4.5 TB/s). Two or four short rows a wave: 26 us for 512 columns; several rows a
//                    wave in a loop and non-temporal loads: slower too.
// k_int8_rows        y = diag(s) (q p^T) diag(t) for M <= 64: a workgroup takes 16 output channels of one
//                    group, its waves split K, so that the weight is read once with every load of a
//                    workgroup in flight at the same time. Bound by reading the weight, and below some MB of it
//                    by the launch: 4.1 us for one row, 4096 channels and K = 2048; 6.7 us for 16 rows and K = 4096.
#include <algorithm>

#include "engine.h"
#include "int8_device.h"
#include "moe_internal.h"

namespace moe {
namespace {

template <class T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
  if constexpr (sizeof(T) == 2) {
    eng::unpack8(ld16(p), v);
  } else {
    const uint4 a = ld16(p), b = ld16(p + 4);
    v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y); v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
    v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y); v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
  }
}

template <class T, int EL>
__device__ __forceinline__ void load_el(const T* p, float (&v)[EL]) {
  if constexpr (EL == 8) {
    load8(p, v);
  } else if constexpr (sizeof(T) == 2) {
    const uint2 a = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(a.x << 16); v[1] = __uint_as_float(a.x & 0xffff0000u);
    v[2] = __uint_as_float(a.y << 16); v[3] = __uint_as_float(a.y & 0xffff0000u);
  } else {
    const uint4 a = ld16(p);
    v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y); v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
  }
}

// NV: pieces of a row, EL elements a lane, held in registers (0: rows of any length, read twice). nrows: the row
// count on the device, where the host does not know it (null: rows).
template <class T, int NV, int EL>
__global__ __launch_bounds__(256) void k_int8_quant(const T* __restrict__ x, int64_t rows, int cols,
                                                    const int* __restrict__ nrows, uint8_t* __restrict__ q,
                                                    float* __restrict__ scales) {
  constexpr bool F32 = sizeof(T) == 4;
  const int lane = threadIdx.x & 63;
  const int64_t r = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 4 + (threadIdx.x >> 6);
  const int64_t n = nrows ? min(rows, (int64_t)*nrows) : rows;
  if (r >= n) return;
  const T* row = x + (size_t)r * cols;
  uint8_t* out = q + (size_t)r * cols;
  unsigned m = 0u;
  if constexpr (NV > 0) {
    float v[NV][EL];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = EL * (64 * i + lane);
      if (c < cols) {
        load_el<T, EL>(row + c, v[i]);
      } else {
#pragma unroll
        for (int j = 0; j < EL; ++j) v[i][j] = 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < EL; ++j) m = max(m, mag_bits(v[i][j]));
    const Q8Row R(wave_max_u32(m));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = EL * (64 * i + lane);
      unsigned o[EL / 4];
      q8_pack<F32>(v[i], R, o);
      if (c < cols) {
        if constexpr (EL == 8) *reinterpret_cast<uint2*>(out + c) = make_uint2(o[0], o[1]);
        else *reinterpret_cast<unsigned*>(out + c) = o[0];
      }
    }
    if (lane == 0) scales[r] = R.scale;
  } else {
    for (int c = 8 * lane; c < cols; c += 512) {
      float v[8];
      load8(row + c, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, mag_bits(v[j]));
    }
    const Q8Row R(wave_max_u32(m));
    for (int c = 8 * lane; c < cols; c += 512) {
      float v[8];
      unsigned o[2];
      load8(row + c, v);
      q8_pack<F32>(v, R, o);
      *reinterpret_cast<uint2*>(out + c) = make_uint2(o[0], o[1]);
    }
    if (lane == 0) scales[r] = R.scale;
  }
}

template <class T>
void launch_quant_t(const void* x, int64_t rows, int cols, const int* nrows, uint8_t* q, float* scales, hipStream_t s) {
  const T* p = static_cast<const T*>(x);
  // a dimension of a grid holds less than 2^32 threads: 2^22 workgroups, then more rows of them
  const int64_t b = (rows + 3) / 4;
  const dim3 g((unsigned)std::min<int64_t>(b, 1 << 22), (unsigned)((b + (1 << 22) - 1) >> 22));
  // pieces of 256 or 512 elements, so that few of the lanes are idle: 65536 x 768 bf16 33 us, 36 in pieces of 512;
  // 262144 x 256 58 and 68; 32768 x 1536 31 in three pieces of 512, 34 in the registers of four
  if (cols <= 256) k_int8_quant<T, 1, 4><<<g, 256, 0, s>>>(p, rows, cols, nrows, q, scales);
  else if (cols <= 512) k_int8_quant<T, 1, 8><<<g, 256, 0, s>>>(p, rows, cols, nrows, q, scales);
  else if (cols <= 768) k_int8_quant<T, 3, 4><<<g, 256, 0, s>>>(p, rows, cols, nrows, q, scales);
  else if (cols <= 1024) k_int8_quant<T, 2, 8><<<g, 256, 0, s>>>(p, rows, cols, nrows, q, scales);
  else if (cols <= 1536) k_int8_quant<T, 3, 8><<<g, 256, 0, s>>>(p, rows, cols, nrows, q, scales);
  else if (cols <= 2048) k_int8_quant<T, 4, 8><<<g, 256, 0, s>>>(p, rows, cols, nrows, q, scales);
  else if (cols <= 4096) k_int8_quant<T, 8, 8><<<g, 256, 0, s>>>(p, rows, cols, nrows, q, scales);
  else k_int8_quant<T, 0, 8><<<g, 256, 0, s>>>(p, rows, cols, nrows, q, scales);
}

// ------------------------------------------------------------------------------------------------
constexpr int kRW = 8;   // waves of k_int8_rows

// 16 channels from n0 of group g times its NG x 16 rows from r0; steps of 64 elements, the last one
// possibly short (K is a multiple of 16: whole 16-element chunks)
template <int NG>
__device__ __forceinline__ void rows_task(const I8Params& p, char* red_, int g, int n0, int r0, int cnt) {
  const int tid = threadIdx.x, lane = tid & 63, w = eng::wave_id(), ch = lane >> 4;
  const size_t K = (size_t)p.K;
  const uint8_t* pw = p.w + ((size_t)g * p.N + min(n0 + (lane & 15), p.N - 1)) * K + 16 * ch;
  const uint8_t* px[NG];
#pragma unroll
  for (int i = 0; i < NG; ++i) px[i] = p.x + (size_t)(r0 + min(16 * i + (lane & 15), cnt - 1)) * K + 16 * ch;
  const int S = (p.K + 63) / 64, s0 = w * S / kRW, s1 = (w + 1) * S / kRW;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  i32x4 acc[NG];
#pragma unroll
  for (int i = 0; i < NG; ++i) acc[i] = i32x4{0, 0, 0, 0};
  constexpr int U = NG == 4 ? 2 : 4;
  for (int s = s0; s < s1; s += U) {
    uint4 a[U], b[NG][U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = min(s + u, s1 - 1) * 64;
      const bool in = k + 16 * ch < p.K;
      a[u] = in ? ld16(pw + k) : zero;
#pragma unroll
      for (int i = 0; i < NG; ++i) b[i][u] = in ? ld16(px[i] + k) : zero;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (s + u < s1)
#pragma unroll
        for (int i = 0; i < NG; ++i)
          acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a[u]),
                                                         __builtin_bit_cast(i32x4, b[i][u]), acc[i], 0, 0, 0);
  }
  i32x4* red = reinterpret_cast<i32x4*>(red_);
#pragma unroll
  for (int i = 0; i < NG; ++i) {
    if (16 * i >= cnt) break;
    red[w * 64 + lane] = acc[i];
    __syncthreads();
    if (tid < 256) {
      const int f = tid & 15, c = tid >> 4, r = 16 * i + c, n = n0 + f;
      const int* rs = reinterpret_cast<const int*>(red) + ((f >> 2) * 16 + c) * 4 + (f & 3);
      int sum = 0;
#pragma unroll
      for (int v = 0; v < kRW; ++v) sum += rs[v * 256];
      if (r < cnt && n < p.N) {
        const float y = (float)sum * (p.xs[r0 + r] * p.ws[(size_t)g * p.N + n]);
        const size_t at = (size_t)(r0 + r) * p.N + n;
        if (p.f32) static_cast<float*>(p.y)[at] = y;
        else static_cast<bf16*>(p.y)[at] = (bf16)y;
      }
    }
    __syncthreads();
  }
}

__global__ __launch_bounds__(kRW * 64, 4) void k_int8_rows(I8Params p) {
  __shared__ __attribute__((aligned(16))) char red[kRW * 64 * 16];
  const int g = blockIdx.y, n0 = blockIdx.x * 16;
  int r0 = 0, cnt = (int)p.M;
  if (p.offsets) {
    r0 = min(max(p.offsets[g], 0), (int)p.M);
    cnt = min(max(p.offsets[g + 1], r0), (int)p.M) - r0;
    r0 = __builtin_amdgcn_readfirstlane(r0);
    cnt = __builtin_amdgcn_readfirstlane(cnt);
  }
  if (cnt <= 0) return;
  if (cnt <= 16) rows_task<1>(p, red, g, n0, r0, cnt);
  else if (cnt <= 32) rows_task<2>(p, red, g, n0, r0, cnt);
  else rows_task<4>(p, red, g, n0, r0, cnt);
}

}  // namespace

hipError_t launch_int8_quant(const void* x, bool f32, int64_t rows, int cols, const int* nrows, uint8_t* q,
                             float* scales, const char* name, hipStream_t s) {
  prof_mark_begin(name, s);
  if (f32) launch_quant_t<float>(x, rows, cols, nrows, q, scales, s);
  else launch_quant_t<bf16>(x, rows, cols, nrows, q, scales, s);
  const hipError_t err = hipGetLastError();
  if (err == hipSuccess) prof_mark_end(s);
  return err;
}

// One weight is read through LDS tiles instead where many channels times many rows would read the rows of x too often:
// K = 4096, 64 rows of 4096 channels 13.1 us here, 13.5 on tiles; 16 and 32 rows of 8192 11.3 and 16.1, 14.0 and
// 14.4; 16 rows of 16384 22.2, 19.1. Groups are better off here at any size (64 rows in 2 to 16 groups: 6.5-8.7 us,
// 9.2-9.7 on tiles, mostly of rows that are not there).
bool int8_rows_fit(const I8Params& p) {
  return p.M <= kFewTokens && (p.offsets || p.N * ((p.M + 15) / 16) <= 12288);
}

hipError_t launch_int8_rows(const I8Params& p, hipStream_t s) {
  prof_mark_begin("int8_rows", s);
  k_int8_rows<<<dim3((p.N + 15) / 16, p.G), kRW * 64, 0, s>>>(p);
  const hipError_t err = hipGetLastError();
  if (err == hipSuccess) prof_mark_end(s);
  return err;
}

}  // namespace moe
