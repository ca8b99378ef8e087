// Rows of float values in 8 bits, one scale a row: with a = max |x|,
//     scale = a / 127,   q = round_half_even(127 x / a).
//
// One wave per row: the row is read once into registers (at most 16 chunks of
// 8 values a lane), its maximum found with lane shuffles, and the 8-byte
// groups of q written from the same registers, so a row costs its bytes once
// in and once out and no barrier (a 151936 x 4096 bf16 LM head: 288 to 299 us,
// 6.2 to 6.5 TB/s, among other calls, up to 343 us back to back; 339 us without
// non-temporal loads and stores where it took 287 with).  Few rows take four waves each,
// whose maxima meet in LDS: what a call of one block costs is the length of one
// wave's work (16 x 4096 on the device: 3.9 us against 6.2).
//
// Rounding: t = x * (127 / a) in float32 is off the exact quotient by less
// than 2^-16 (|t| <= 127, two roundings of 2^-24 each), so rint(t) is the
// rounded exact quotient unless t is within 2^-16 of a half.  Chunks with a t
// within 2e-5 of one decide it exactly instead: q > k + 1/2 exactly when
// 254 x > (2 k + 1) a, whose two sides are exact products in float64.
#include <math.h>

#include "common.h"
#include "rollout.h"

namespace domino {

constexpr int kQuantWaves = 4;  // waves per workgroup
constexpr int kFewRows = 2048;  // up to here four waves a row

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ u32x4 ldnt16(const unsigned char* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
}

template <class T>
struct Chunk8;  // 8 consecutive values of a row

template <>
struct Chunk8<Bf16> {
  u32x4 v;
  __device__ __forceinline__ void load(const unsigned char* row, int chunk) { v = ldnt16(row + (size_t)chunk * 16); }
  __device__ __forceinline__ void zero() { v = u32x4{0, 0, 0, 0}; }
  __device__ __forceinline__ float get(int e) const {
    const uint32_t u = v[e >> 1];
    return __uint_as_float(e & 1 ? u & 0xFFFF0000u : u << 16);
  }
};

template <>
struct Chunk8<F32> {
  u32x4 v[2];
  __device__ __forceinline__ void load(const unsigned char* row, int chunk) {
    v[0] = ldnt16(row + (size_t)chunk * 32);
    v[1] = ldnt16(row + (size_t)chunk * 32 + 16);
  }
  __device__ __forceinline__ void zero() { v[0] = v[1] = u32x4{0, 0, 0, 0}; }
  __device__ __forceinline__ float get(int e) const { return __uint_as_float(v[e >> 2][e & 3]); }
};

// The exact quotient 127 x / a rounded to the nearest integer, ties to even,
// from an approximation t of it that is off by less than 1/2.
__device__ __forceinline__ int round_quotient(float x, float a, float t) {
  const int k = (int)floorf(t);
  const double l = 254.0 * (double)x, h = (2.0 * k + 1.0) * (double)a;
  if (l > h) return k + 1;
  if (l < h) return k;
  return k + (k & 1);
}

template <class T, int NC, int WPR>
__global__ void __launch_bounds__(kQuantWaves * 64)
    quantize_rows_kernel(int rows, int cols, const typename T::elem* __restrict__ x, int8_t* __restrict__ q,
                         float* __restrict__ scale) {
  // lane of the row's WPR waves
  const int row = blockIdx.x * (kQuantWaves / WPR) + wave_id() / WPR, lane = threadIdx.x & (64 * WPR - 1);
  if (row >= rows) return;  // (with WPR = 4 a workgroup has one row)
  const int chunks = cols >> 3;
  const unsigned char* xr = reinterpret_cast<const unsigned char*>(x + (size_t)row * cols);
  Chunk8<T> c[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    if (i * 64 * WPR + lane < chunks)
      c[i].load(xr, i * 64 * WPR + lane);
    else
      c[i].zero();
  }
  // |x| by its bits: infinities and NaN compare above every finite value
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(c[i].get(e)) & 0x7FFFFFFFu);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
  if constexpr (WPR > 1) {
    __shared__ uint32_t tops[WPR];
    if ((threadIdx.x & 63) == 0) tops[wave_id()] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WPR; ++w) top = max(top, tops[w]);
  }
  const bool finite = top < 0x7F800000u;
  float a = __uint_as_float(top);
  if (lane == 0) scale[row] = finite ? a / 127.f : __uint_as_float(0x7FC00000u);
  // 127 / a would overflow below about 2^-121: such rows are scaled by 2^64
  // first (exact, and the quotient is the same)
  const float up = a < 8.673617379884035e-19f ? 18446744073709551616.f : 1.f;  // a < 2^-60
  a *= up;
  const float inv = finite && a > 0.f ? 127.f / a : 0.f;
  u32x2* qr = reinterpret_cast<u32x2*>(q + (size_t)row * cols);
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    float t[8];
    int k[8];
    bool near = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      t[e] = finite ? c[i].get(e) * up * inv : 0.f;
      const float r = rintf(t[e]);
      near |= fabsf(t[e] - r) > 0.49998f;
      k[e] = (int)r;
    }
    if (near) {
#pragma unroll
      for (int e = 0; e < 8; ++e) k[e] = round_quotient(c[i].get(e) * up, a, t[e]);
    }
    u32x2 w{0, 0};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      w[0] |= (uint32_t)(k[e] & 0xFF) << (8 * e);
      w[1] |= (uint32_t)(k[e + 4] & 0xFF) << (8 * e);
    }
    if (i * 64 * WPR + lane < chunks) __builtin_nontemporal_store(w, qr + i * 64 * WPR + lane);
  }
}

template <class T, int NC, int WPR>
static void quantize_launch(int rows, int cols, const void* x, int8_t* q, float* scale, hipStream_t s) {
  using E = typename T::elem;
  constexpr int kRows = kQuantWaves / WPR;
  hipLaunchKernelGGL((quantize_rows_kernel<T, NC, WPR>), dim3((unsigned)((rows + kRows - 1) / kRows)),
                     dim3(kQuantWaves * 64), 0, s, rows, cols, static_cast<const E*>(x), q, scale);
}

template <class T>
static hipError_t quantize_t(int rows, int cols, const void* x, int8_t* q, float* scale, hipStream_t s) {
  const int per_lane = (cols / 8 + 63) / 64;  // chunks, with one wave a row
  if (rows <= kFewRows && per_lane > 2) {
    if (per_lane <= 4)
      quantize_launch<T, 1, 4>(rows, cols, x, q, scale, s);
    else if (per_lane <= 8)
      quantize_launch<T, 2, 4>(rows, cols, x, q, scale, s);
    else
      quantize_launch<T, 4, 4>(rows, cols, x, q, scale, s);
  } else if (per_lane <= 1) {
    quantize_launch<T, 1, 1>(rows, cols, x, q, scale, s);
  } else if (per_lane <= 2) {
    quantize_launch<T, 2, 1>(rows, cols, x, q, scale, s);
  } else if (per_lane <= 4) {
    quantize_launch<T, 4, 1>(rows, cols, x, q, scale, s);
  } else if (per_lane <= 8) {
    quantize_launch<T, 8, 1>(rows, cols, x, q, scale, s);
  } else {
    quantize_launch<T, 16, 1>(rows, cols, x, q, scale, s);
  }
  return hipGetLastError();
}

hipError_t launch_quantize_rows(int rows, int cols, int dtype, const void* x, int8_t* q, float* scale, hipStream_t s) {
  if (rows <= 0) return hipSuccess;
  if (cols % 32 || cols > 8 * 64 * 16) return hipErrorNotSupported;
  return dtype == 1 ? quantize_t<Bf16>(rows, cols, x, q, scale, s) : quantize_t<F32>(rows, cols, x, q, scale, s);
}

}  // namespace domino
