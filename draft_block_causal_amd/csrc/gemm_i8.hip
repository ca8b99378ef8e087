// Product of 8-bit integers with scales for each row of A (token) and of W
// (channel): C[m][n] = a_scale[m] w_scale[n] sum_k A[m][k] W[n][k].
//
// The sums are exact in int32 (at most 8192 products of 128^2 or less).  Each
// is converted to float32 (one rounding), multiplied by the row's scale and
// then by the channel's (one each), which keeps the result within 3 2^-24 of
// the real value; scales are not multiplied together first, so that a channel
// of large scale meets the sum before an underflow can.
//
// Matrix-core tiles as in common.h with 8-bit elements: one
// v_mfma_i32_16x16x64_i8 multiplies 16 rows by 16 rows over 64 bytes of K, a
// lane holding 16 consecutive bytes of one row of each operand.  W is the
// first operand, so an accumulator lane holds 4 consecutive columns n of one
// row m of C, stored as 16 bytes.
#include <algorithm>

#include "common.h"
#include "kernels.h"

namespace domino {

typedef int i32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ i32x4 mma16_i8(i32x4 acc, u32x4 w, u32x4 a) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, w), __builtin_bit_cast(i32x4, a), acc, 0, 0, 0);
}

// ---------------------------------------------------------------------------
// Streaming kernel, at most 64 rows (G groups of 16): bound by the one read of
// W.  A workgroup of ceil(K / 512) waves takes a contiguous range of 16-row
// tiles of W; wave w holds its 512-byte K slice of A in registers (32 a group)
// and streams the same slice of W: 8 loads of 16 bytes a lane and tile, each
// two rows' runs of 512 contiguous bytes, non-temporal.  A tile goes through a
// private 8 KB of LDS into the operand layout (16-byte chunks of row r stored
// at chunk ^ r, so that both the row-wise writes and the column-wise reads
// touch 16 bank groups), while the next one is in flight in registers.  The
// waves' partial sums meet in LDS; finished tiles stay there until kHold of
// them make runs of 512 bytes a row of C.
// W is read through a descriptor sized to the tile's rows below N: the rest,
// and the prefetch past the range, read as zero without touching memory.
// Bytes past K within a slice belong to the next row and meet zeros of A.
// ---------------------------------------------------------------------------
constexpr int kSlice = 512;
constexpr int kSliceTile = 16 * kSlice;  // LDS bytes of one wave's tile
constexpr int kHold = 8;                 // finished 16-column tiles held in LDS

// LDS: the waves' tiles | red[R][nw][16 G][16] int32 | out[16 G][16 kHold] float.
// R = 2 (tiles take turns, one barrier a tile) up to 8 waves; 16 waves leave
// room for one (a second barrier a tile).
template <int G, int MAXW>
struct StreamLds {
  static constexpr int kRed = MAXW > 8 ? 1 : 2;
  __host__ __device__ static constexpr int red_bytes(int nw) { return nw * G * 1024; }
  __host__ __device__ static constexpr int out_at(int nw) { return nw * kSliceTile + kRed * red_bytes(nw); }
  __host__ __device__ static constexpr int total(int nw) { return out_at(nw) + G * kHold * 1024; }
  static_assert(total(MAXW) <= 160 * 1024, "LDS");
};

template <int G, int MAXW>
__global__ void __launch_bounds__(MAXW * 64)
    gemm_i8_stream_kernel(const int8_t* __restrict__ A, const float* __restrict__ as, int M,
                          const int8_t* __restrict__ W, const float* __restrict__ ws, int N, int K,
                          float* __restrict__ C) {
  using SL = StreamLds<G, MAXW>;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  const int nw = blockDim.x >> 6, wave = wave_id(), lane = threadIdx.x & 63;
  const int grp = lane >> 4, col = lane & 15;
  unsigned char* tile = smem + wave * kSliceTile;
  int* red = reinterpret_cast<int*>(smem + nw * kSliceTile);
  float* out = reinterpret_cast<float*>(smem + SL::out_at(nw));

  u32x4 af[G][8];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int m = g * 16 + col;
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const int k = wave * kSlice + s * 64 + grp * 16;
      af[g][s] = m < M && k < K ? ld16(A + (size_t)m * K + k) : u32x4{0, 0, 0, 0};
    }
  }

  const long ntiles = (N + 15) >> 4;
  const int t0 = (int)(ntiles * blockIdx.x / gridDim.x), t1 = (int)(ntiles * (blockIdx.x + 1) / gridDim.x);
  const int lrow = lane >> 5, lchunk = lane & 31;
  const int voff = lrow * K + wave * kSlice + lchunk * 16;
  auto load = [&](int t, u32x4 (&dst)[8]) {
    const int rows = t < t1 ? min(16, N - t * 16) : 0;
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<int8_t*>(W + (rows ? (size_t)t * 16 * K : 0)), (short)0, rows * K, kRsrcWord3);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      dst[j] = __builtin_amdgcn_raw_buffer_load_b128(r, voff + 2 * j * K, 0, kLoadNonTemporal);
  };
  // columns [16 ta, 16 tb) of C from the held tiles
  auto flush = [&](int ta, int tb) {
    const int n0 = ta * 16, cols = min(tb * 16, N) - n0;
    for (int e = threadIdx.x; e < G * 16 * (kHold * 16); e += blockDim.x) {
      const int m = e / (kHold * 16), c = e % (kHold * 16);
      if (m < M && c < cols) C[(size_t)m * N + n0 + c] = out[e];
    }
  };
  auto process = [&](int t, const u32x4 (&w)[8], int* rb) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int r = 2 * j + lrow;
      st16(tile + r * kSlice + ((lchunk ^ r) << 4), w[j]);
    }
    i32x4 acc[G];
#pragma unroll
    for (int g = 0; g < G; ++g) acc[g] = i32x4{0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const u32x4 b = ld16(tile + col * kSlice + (((s * 4 + grp) ^ col) << 4));
#pragma unroll
      for (int g = 0; g < G; ++g) acc[g] = mma16_i8(acc[g], b, af[g][s]);
    }
    // lane: C columns 4 grp .. + 3 of row 16 g + col
#pragma unroll
    for (int g = 0; g < G; ++g)
      *reinterpret_cast<i32x4*>(rb + ((wave * G + g) * 16 + col) * 16 + grp * 4) = acc[g];
    __syncthreads();
    const int held = (t - t0) % kHold;
    for (int e = threadIdx.x; e < G * 256; e += blockDim.x) {
      int sum = 0;
      for (int q = 0; q < nw; ++q) sum += rb[q * G * 256 + e];
      const int m = e >> 4, n = t * 16 + (e & 15);
      if (m < M && n < N) out[m * (kHold * 16) + held * 16 + (e & 15)] = (float)sum * as[m] * ws[n];
    }
    if (held == kHold - 1 || t == t1 - 1) {
      __syncthreads();
      flush(t - held, t + 1);
      // (the next write to `out` follows the next tile's barrier)
    } else if (SL::kRed == 1) {
      __syncthreads();  // the sums are read before the next tile's are written
    }
  };

  u32x4 w0[8], w1[8];
  int t = t0;
  load(t, w0);
  while (t < t1) {
    load(t + 1, w1);
    __builtin_amdgcn_sched_barrier(0);
    process(t, w0, red);
    if (++t >= t1) break;
    load(t + 1, w0);
    __builtin_amdgcn_sched_barrier(0);
    process(t, w1, red + (SL::kRed - 1) * nw * G * 256);
    ++t;
  }
}

template <int G, int MAXW>
static hipError_t launch_stream(const int8_t* A, const float* as, int M, const int8_t* W, const float* ws, int N, int K,
                                float* C, int num_cu, hipStream_t s) {
  const int nw = (K + kSlice - 1) / kSlice;
  auto kern = gemm_i8_stream_kernel<G, MAXW>;
  const int lds = StreamLds<G, MAXW>::total(nw);
  const hipError_t e =
      hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e != hipSuccess) return e;
  // about 8 waves a compute unit
  const int per_cu = std::max(1, 8 / nw);
  const int grid = std::min((N + 15) / 16, num_cu * per_cu);
  hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3((unsigned)nw * 64), lds, s, A, as, M, W, ws, N, K, C);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Tiled kernel: BM x BN outputs a workgroup of 8 waves (a 2 x 4 grid), operands
// from memory straight into LDS through a ring of 64-byte K steps, laid out
// and refilled as in gemm.hip (chunk c of a 64-byte row r in slot
// c ^ ((r >> 1) & 3)); two groups of waves, one per SIMD each, alternate
// between reading fragments and multiplying.
// ---------------------------------------------------------------------------
typedef __attribute__((address_space(1))) const void* gptr_t;
typedef __attribute__((address_space(3))) void* lptr_t;

__device__ const unsigned char kZeros[16] = {};  // what A reads past K

template <int BM, int BN>
struct TileI8 {
  static constexpr int kThreads = 512, kRow = 64;
  static constexpr int kStage = (BM + BN) * kRow;
  static constexpr int kStages = 160 * 1024 / kStage < 6 ? 160 * 1024 / kStage : 6;
  static constexpr int kRowsPerIssue = 128;  // 8 waves x 16 rows of 64 bytes
  static constexpr int kALoads = BM / kRowsPerIssue;
  static constexpr int kWLoads = (BN + kRowsPerIssue - 1) / kRowsPerIssue;
  static constexpr int kPerStage = kALoads + kWLoads;
  static constexpr int kFA = BM / 2 / 16, kFW = BN / 4 / 16;
  static_assert(BM % 128 == 0 && BN % 128 == 0, "whole DMA rounds");
  static_assert((kStages - 2) * kPerStage < 64, "vector-memory count field");
};

// vmcnt(n), lgkmcnt(0); expcnt at its maximum
#define DOMINO_I8_WAIT(n) __builtin_amdgcn_s_waitcnt(((n) & 15) | (((n) >> 4) << 14) | 0x0070)

// Until at most `ahead` younger stages of this wave's loads are in flight and
// its LDS reads have returned.
template <int PER, int MAXA>
__device__ __forceinline__ void wait_ahead(int ahead) {
  if constexpr (MAXA >= 4) {
    if (ahead >= 4) {
      DOMINO_I8_WAIT(4 * PER);
      return;
    }
  }
  if constexpr (MAXA >= 3) {
    if (ahead >= 3) {
      DOMINO_I8_WAIT(3 * PER);
      return;
    }
  }
  if (ahead >= 2) {
    DOMINO_I8_WAIT(2 * PER);
  } else if (ahead == 1) {
    DOMINO_I8_WAIT(PER);
  } else {
    DOMINO_I8_WAIT(0);
  }
}

template <int BM, int BN>
__global__ void __launch_bounds__(512, 1)
    gemm_i8_tiled_kernel(const int8_t* __restrict__ A, const float* __restrict__ as, int M,
                         const int8_t* __restrict__ W, const float* __restrict__ ws, int N, int K,
                         float* __restrict__ C, int num_m, int num_n) {
  using T = TileI8<BM, BN>;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  // one XCD takes every M tile of an N tile back to back (workgroups go
  // round-robin over 8 XCDs): W comes from memory once and from its L2 after
  const int xcd = blockIdx.x % 8, local = blockIdx.x / 8;
  const int nl = local / num_m, mt = local - nl * num_m, nt = nl * 8 + xcd;
  if (nt >= num_n) return;
  const int m0 = mt * BM, n0 = nt * BN;
  const int wave = wave_id(), lane = threadIdx.x & 63, grp = lane >> 4, col = lane & 15;
  const int wm = wave >> 2, wn = wave & 3;

  const int dchunk = (lane & 3) ^ ((lane >> 3) & 3);
  const int8_t *ag[T::kALoads], *wg[T::kWLoads];
#pragma unroll
  for (int i = 0; i < T::kALoads; ++i)
    ag[i] = A + (size_t)min(m0 + i * 128 + wave * 16 + (lane >> 2), M - 1) * K + dchunk * 16;
#pragma unroll
  for (int i = 0; i < T::kWLoads; ++i)
    wg[i] = W + (size_t)min(n0 + i * 128 + wave * 16 + (lane >> 2), N - 1) * K + dchunk * 16;
  const int nk = (K + 63) / 64;
  const bool past = K % 64 != 0 && dchunk >= 2;  // this lane's chunk of the last step lies past K
  auto issue = [&](int kt) {
    unsigned char* sA = smem + (kt % T::kStages) * T::kStage;
    unsigned char* sW = sA + BM * T::kRow;
    const bool skip = past && kt == nk - 1;
    const size_t k = (size_t)kt * 64;
#pragma unroll
    for (int i = 0; i < T::kALoads; ++i) {
      const void* p = ag[i] + k;
      if (skip) p = kZeros;
      __builtin_amdgcn_global_load_lds((gptr_t)p, (lptr_t)(sA + (i * 128 + wave * 16) * 64), 16, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < T::kWLoads; ++i) {
      const void* p = wg[i] + (skip ? k - 32 : k);  // (any bytes of the row: they meet zeros)
      __builtin_amdgcn_global_load_lds((gptr_t)p, (lptr_t)(sW + (i * 128 + wave * 16) * 64), 16, 0, 0);
    }
  };
  const int fslot = (grp ^ ((col >> 1) & 3)) * 16;

  i32x4 acc[T::kFA][T::kFW];
#pragma unroll
  for (int i = 0; i < T::kFA; ++i)
#pragma unroll
    for (int j = 0; j < T::kFW; ++j) acc[i][j] = i32x4{0, 0, 0, 0};

#pragma unroll
  for (int s = 0; s < T::kStages - 1; ++s)
    if (s < nk) issue(s);
  wait_ahead<T::kPerStage, T::kStages - 2>(min(T::kStages - 2, nk - 1));
  __builtin_amdgcn_s_barrier();
  if (wm == 1) __builtin_amdgcn_s_barrier();  // the second group starts one phase later
  for (int kt = 0; kt < nk; ++kt) {
    __builtin_amdgcn_sched_barrier(0);
    const unsigned char* sA = smem + (kt % T::kStages) * T::kStage;
    const unsigned char* sW = sA + BM * T::kRow;
    u32x4 af[T::kFA], wf[T::kFW];
#pragma unroll
    for (int i = 0; i < T::kFA; ++i) af[i] = ld16(sA + ((wm * T::kFA + i) * 16 + col) * 64 + fslot);
#pragma unroll
    for (int j = 0; j < T::kFW; ++j) wf[j] = ld16(sW + ((wn * T::kFW + j) * 16 + col) * 64 + fslot);
    if (kt + T::kStages - 1 < nk) issue(kt + T::kStages - 1);
    wait_ahead<T::kPerStage, T::kStages - 2>(max(0, min(T::kStages - 2, nk - 2 - kt)));
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < T::kFA; ++i)
#pragma unroll
      for (int j = 0; j < T::kFW; ++j) acc[i][j] = mma16_i8(acc[i][j], wf[j], af[i]);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
  }
  if (wm == 0) __builtin_amdgcn_s_barrier();  // equal barrier counts in both groups

  const bool vec = (N & 3) == 0;  // then every group of 4 columns is 16-byte aligned and whole
#pragma unroll
  for (int j = 0; j < T::kFW; ++j) {
    const int n = n0 + (wn * T::kFW + j) * 16 + grp * 4;
    if (n >= N) continue;
    float sn[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) sn[q] = ws[min(n + q, N - 1)];
#pragma unroll
    for (int i = 0; i < T::kFA; ++i) {
      const int m = m0 + (wm * T::kFA + i) * 16 + col;
      if (m >= M) continue;
      const float sm = as[m];
      float* c = C + (size_t)m * N + n;
      f32x4 v;
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = (float)acc[i][j][q] * sm * sn[q];
      if (vec) {
        *reinterpret_cast<f32x4*>(c) = v;
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (n + q < N) c[q] = v[q];
      }
    }
  }
}

template <int BM, int BN>
static hipError_t launch_tiled(const int8_t* A, const float* as, int M, const int8_t* W, const float* ws, int N, int K,
                               float* C, hipStream_t s) {
  using T = TileI8<BM, BN>;
  const int num_m = (M + BM - 1) / BM, num_n = (N + BN - 1) / BN;
  const unsigned blocks = (unsigned)((num_n + 7) / 8 * 8) * (unsigned)num_m;
  auto kern = gemm_i8_tiled_kernel<BM, BN>;
  const size_t lds = (size_t)T::kStages * T::kStage;
  const hipError_t e =
      hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3(blocks), dim3(T::kThreads), lds, s, A, as, M, W, ws, N, K, C, num_m, num_n);
  return hipGetLastError();
}

hipError_t launch_gemm_i8(const int8_t* A, const float* a_scale, int M, const int8_t* W, const float* w_scale, int N,
                          int K, float* C, int num_cu, hipStream_t s) {
  if (M <= 0 || N <= 0) return hipSuccess;
  if (K <= 0 || K % 32 || K > 8192) return hipErrorNotSupported;
  if (K <= 4096) {
    if (M <= 16) return launch_stream<1, 8>(A, a_scale, M, W, w_scale, N, K, C, num_cu, s);
    if (M <= 32) return launch_stream<2, 8>(A, a_scale, M, W, w_scale, N, K, C, num_cu, s);
    if (M <= 48) return launch_stream<3, 8>(A, a_scale, M, W, w_scale, N, K, C, num_cu, s);
    if (M <= 64) return launch_stream<4, 8>(A, a_scale, M, W, w_scale, N, K, C, num_cu, s);
  } else if (M <= 16) {
    return launch_stream<1, 16>(A, a_scale, M, W, w_scale, N, K, C, num_cu, s);
  }
  return M <= 128 ? launch_tiled<128, 256>(A, a_scale, M, W, w_scale, N, K, C, s)
                  : launch_tiled<256, 256>(A, a_scale, M, W, w_scale, N, K, C, s);
}

}  // namespace domino
