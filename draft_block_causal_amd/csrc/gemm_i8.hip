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
#include <atomic>

#include "common.h"
#include "rollout.h"

namespace domino {

typedef int i32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ i32x4 mma16_i8(i32x4 acc, u32x4 w, u32x4 a) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, w), __builtin_bit_cast(i32x4, a), acc, 0, 0,
                                               0);
}

// Allows a kernel its dynamic LDS, once a device (bit d of `done`).
static hipError_t allow_lds(const void* kern, int lds, std::atomic<uint64_t>& done) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return hipSuccess;
  e = hipFuncSetAttribute(kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e == hipSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// ---------------------------------------------------------------------------
// Streaming kernel: bound by the one read of W.  A workgroup of NW waves takes
// G groups of 16 rows of A and a contiguous range of 16-row tiles of W; wave w
// holds its slice of A (64 S bytes of K) in registers and streams the same
// slice of W: S loads of 16 bytes a lane and tile, contiguous runs of 64 S
// bytes a row.  A tile goes through private LDS into the operand layout while
// the next one is in flight in registers.  The waves' partial sums meet in LDS
// (two buffers in turn, so one barrier a tile); finished tiles stay there as
// long as they fit, all of a workgroup's where they do, since stores mixed into
// the stream of W cost it more than the same bytes behind it (one block of a
// Qwen3-8B head: 102 us with a store every 8 tiles, 95 with all at the end,
// 93 with none).
// W is read through a descriptor sized to the tile's rows below N: the rest,
// and the prefetch past the range, read as zero without touching memory.
// Bytes past K within a slice belong to the next row and meet zeros of A.
// The channel's scale is loaded with its tile: loads return in order, and one
// issued where it is used would wait for the tile in flight.
// ---------------------------------------------------------------------------
template <int S, int NW, int G>
struct Stream {
  static constexpr int kSlice = 64 * S, kChunks = 4 * S;
  // LDS row of a tile: 16-byte chunk c of row r.  8 lanes read one chunk of 8
  // rows at a time, which must fall into 8 groups of banks: chunks are swapped
  // by the row where their number is a power of two, else rows are padded by a
  // chunk (S = 5: 84 words, and 84 r mod 32 is different for 8 rows).
  static constexpr bool kSwap = (S & (S - 1)) == 0;
  static constexpr int kMask = kChunks < 16 ? kChunks - 1 : 15;
  static constexpr int kStride = kSlice + (kSwap ? 0 : 16);
  static constexpr int kTile = 16 * kStride;
  static constexpr int kRed = NW * G * 1024;  // bytes of one buffer of partial sums
  static constexpr int kOut = NW * kTile + 2 * kRed;
  static constexpr int kLds = kOut + G * 8 * 1024;  // with 8 finished tiles, the least
  static constexpr int kThreads = NW * 64;
  // workgroups a compute unit: LDS, and 16 waves (8 where the operands take
  // more than 128 registers)
  static constexpr int kWaves = G * S > 12 ? 8 : 16;
  // (as many finished tiles as fit: hold())
  static constexpr int kPerCu = 160 * 1024 / kLds < kWaves / NW ? 160 * 1024 / kLds : kWaves / NW;
  static_assert(kLds <= 160 * 1024 && kPerCu >= 1, "LDS");
  static int hold(int tiles) { return std::min(tiles, (160 * 1024 / kPerCu - kOut) / (G * 1024)); }
  __device__ static int at(int r, int c) { return r * kStride + ((kSwap ? c ^ (r & kMask) : c) << 4); }
};

template <int S, int NW, int G>
__global__ void __launch_bounds__(NW * 64)
    gemm_i8_stream_kernel(const int8_t* __restrict__ A, const float* __restrict__ as, int M,
                          const int8_t* __restrict__ W, const float* __restrict__ ws, int N, int K,
                          float* __restrict__ C, int hold) {
  using T = Stream<S, NW, G>;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  const int wave = wave_id(), lane = threadIdx.x & 63, grp = lane >> 4, col = lane & 15;
  unsigned char* tile = smem + wave * T::kTile;
  int* red = reinterpret_cast<int*>(smem + NW * T::kTile);
  float* out = reinterpret_cast<float*>(smem + T::kOut);

  u32x4 af[G][S];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int m = g * 16 + col;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int k = wave * T::kSlice + s * 64 + grp * 16;
      af[g][s] = m < M && k < K ? ld16(A + (size_t)m * K + k) : u32x4{0, 0, 0, 0};
    }
  }
  // partial sums of the outputs e = threadIdx.x, + kThreads, ...: row e / 16, column e % 16
  constexpr int kE = (G * 256 + T::kThreads - 1) / T::kThreads;
  float sm[kE];
#pragma unroll
  for (int i = 0; i < kE; ++i) sm[i] = as[min((int)(threadIdx.x + i * T::kThreads) / 16, M - 1)];

  const long ntiles = (N + 15) >> 4;
  const int t0 = (int)(ntiles * blockIdx.x / gridDim.x), t1 = (int)(ntiles * (blockIdx.x + 1) / gridDim.x);
  int vo[S], lo[S];  // load j: byte offset in the tile's rows of W, and in LDS
#pragma unroll
  for (int j = 0; j < S; ++j) {
    const int e = j * 64 + lane, r = e / T::kChunks, c = e % T::kChunks;
    vo[j] = r * K + wave * T::kSlice + c * 16;
    lo[j] = T::at(r, c);
  }
  const int rcol = threadIdx.x & 15;
  auto load = [&](int t, u32x4 (&dst)[S], float& scale) {
    const int rows = t < t1 ? min(16, N - t * 16) : 0;
    scale = ws[min(t * 16 + rcol, N - 1)];
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<int8_t*>(W + (rows ? (size_t)t * 16 * K : 0)), (short)0, rows * K, kRsrcWord3);
#pragma unroll
    for (int j = 0; j < S; ++j) dst[j] = __builtin_amdgcn_raw_buffer_load_b128(r, vo[j], 0, kLoadNonTemporal);
  };
  // columns [16 ta, 16 tb) of C from the held tiles
  auto flush = [&](int ta, int tb) {
    const int n0 = ta * 16, cols = min(tb * 16, N) - n0;
    const int stride = hold * 16;
    // a wave takes whole rows; 16 bytes a lane where rows of C start at multiples of 16 bytes
    for (int m = wave; m < M; m += NW) {
      float* c = C + (size_t)m * N + n0;
      const float* o = out + m * stride;
      if ((N & 3) == 0) {
        for (int e = lane * 4; e < cols; e += 256)
          __builtin_nontemporal_store(*reinterpret_cast<const f32x4*>(o + e), reinterpret_cast<f32x4*>(c + e));
      } else {
        for (int e = lane; e < cols; e += 64) c[e] = o[e];
      }
    }
  };
  int held = 0;
  auto process = [&](int t, const u32x4 (&w)[S], float scale, int* rb) {
#pragma unroll
    for (int j = 0; j < S; ++j) st16(tile + lo[j], w[j]);
    i32x4 acc[G];
#pragma unroll
    for (int g = 0; g < G; ++g) acc[g] = i32x4{0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const u32x4 b = ld16(tile + T::at(col, s * 4 + grp));
#pragma unroll
      for (int g = 0; g < G; ++g) acc[g] = mma16_i8(acc[g], b, af[g][s]);
    }
    // lane: C columns 4 grp .. + 3 of row 16 g + col
#pragma unroll
    for (int g = 0; g < G; ++g)
      *reinterpret_cast<i32x4*>(rb + ((wave * G + g) * 16 + col) * 16 + grp * 4) = acc[g];
    // taken by every wave here: a load that one side of a branch consumes makes
    // the compiler wait for the tile in flight later
    asm volatile("" : "+v"(scale));
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kE; ++i) {
      const int e = threadIdx.x + i * T::kThreads;
      if (kE * T::kThreads == G * 256 || e < G * 256) {
        int sum = 0;
#pragma unroll
        for (int q = 0; q < NW; ++q) sum += rb[q * G * 256 + e];
        out[(e >> 4) * (hold * 16) + held * 16 + rcol] = (float)sum * sm[i] * scale;
      }
    }
    if (++held == hold || t == t1 - 1) {
      __syncthreads();
      flush(t + 1 - held, t + 1);  // (the next write to `out` follows the next tile's barrier)
      held = 0;
    }
  };

  u32x4 w0[S], w1[S];
  float s0, s1;
  int t = t0;
  load(t, w0, s0);
  // The scheduling barriers keep each prefetch ahead of the LDS traffic of the
  // tile in hand.
  while (t < t1) {
    load(t + 1, w1, s1);
    __builtin_amdgcn_sched_barrier(0);
    process(t, w0, s0, red);
    if (++t >= t1) break;
    load(t + 1, w0, s0);
    __builtin_amdgcn_sched_barrier(0);
    process(t, w1, s1, red + T::kRed / 4);
    ++t;
  }
}

template <int S, int NW, int G>
static hipError_t launch_stream_g(const int8_t* A, const float* as, int M, const int8_t* W, const float* ws, int N,
                                  int K, float* C, int num_cu, hipStream_t s) {
  using T = Stream<S, NW, G>;
  auto kern = gemm_i8_stream_kernel<S, NW, G>;
  static std::atomic<uint64_t> done{0};
  const hipError_t e = allow_lds(reinterpret_cast<const void*>(kern), 160 * 1024, done);
  if (e != hipSuccess) return e;
  const int ntiles = (N + 15) / 16;
  const int grid = std::min(ntiles, num_cu * T::kPerCu);
  const int hold = T::hold((ntiles + grid - 1) / grid);
  hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(T::kThreads), T::kOut + G * hold * 1024, s, A, as, M, W, ws, N, K,
                     C, hold);
  return hipGetLastError();
}

// M <= 64
template <int S, int NW>
static hipError_t launch_stream(const int8_t* A, const float* as, int M, const int8_t* W, const float* ws, int N, int K,
                                float* C, int num_cu, hipStream_t s) {
  switch ((M + 15) / 16) {
    case 1: return launch_stream_g<S, NW, 1>(A, as, M, W, ws, N, K, C, num_cu, s);
    case 2: return launch_stream_g<S, NW, 2>(A, as, M, W, ws, N, K, C, num_cu, s);
    case 3: return launch_stream_g<S, NW, 3>(A, as, M, W, ws, N, K, C, num_cu, s);
    default: return launch_stream_g<S, NW, 4>(A, as, M, W, ws, N, K, C, num_cu, s);
  }
}

// ---------------------------------------------------------------------------
// Tiled kernel: BM x BN outputs a tile, 8 waves (a 2 x 4 grid), one workgroup
// a compute unit that walks its tiles without a break: the loads of the next
// tile are in flight while the last one's results are stored.
// Operands go from memory straight into LDS (16 bytes a lane), in steps of 128
// bytes of K: a load instruction covers whole 128-byte lines of 8 rows.  W and
// A have rings of WS and AS steps.  The
// first row of waves loads W and the second A: loads are counted back in the
// order of their issue, and a wave that loaded both would wait for W's later
// steps whenever it waits for A's next one.
// Chunk c of a 128-byte LDS row r sits in slot c ^ (r & 7): a 16-byte read is
// served 8 lanes at a time, and the 8 lanes of a fragment read (8 rows, one
// chunk) then touch 8 different groups of banks.
// W's loads are non-temporal, which leaves the L2 to A (128 rows of a Qwen3-8B
// head: 189 -> 172 us).  With one M tile, N tiles begin at different steps of K
// and wrap around (the sums are exact in any order): rows of W that lie a power
// of two apart are then not all read at the same offset, that is from the same
// memory channels, at a time (172 -> 149 us; with several M tiles, which share
// W in the L2, 353 -> 361 us at 512 rows: not done).
// With P = 2 a workgroup's tiles go in pairs: the first one's results are kept
// in registers and stored with the second's, since stores between two tiles
// hold up the second's loads (128 rows: vocabulary 151936, d = 2560 104 -> 100
// us, d = 1024 51 -> 48; 128000, d = 2560 81 -> 70; but d = 256 25.3 -> 25.9).  256 x
// 256 tiles have no registers left for it.
// The two rows of waves alternate, one phase apart: one reads the fragments of
// half a step (64 bytes of K) and issues loads while the other multiplies,
// with a barrier between phases.  Order: the loads into a slot are issued one
// step after its last reads (by both rows of waves, each of which waits for its
// reads before the barrier that ends them); a wave waits for its part of step
// D + 1 at the end of its reading in step D's second half, at least one barrier
// before the first wave reads it.
// ---------------------------------------------------------------------------
typedef __attribute__((address_space(1))) const void* gptr_t;
typedef __attribute__((address_space(3))) void* lptr_t;

__device__ const unsigned char kZeros[16] = {};  // what A reads past K

template <int BM, int BN, int WS, int AS, int P>
struct TileI8 {
  static constexpr int kThreads = 512, kBN = BN, kRow = 128;
  static constexpr int kABytes = BM * kRow, kWBytes = kBN * kRow;
  static constexpr int kRings = WS * kWBytes + AS * kABytes;
  // scales of a tile, in LDS where there is room (two tiles', or two pairs', in turn)
  static constexpr bool kScalesInLds = kRings + 2 * P * (BM + BN) * 4 <= 160 * 1024;
  static constexpr int kLds = kRings + (kScalesInLds ? 2 * P * (BM + BN) * 4 : 0);
  static constexpr int kAL = BM / 32, kWL = kBN / 32;  // loads of a step per loading wave
  static constexpr int kFA = BM / 2 / 16, kFW = kBN / 4 / 16;
  static_assert(BM % 128 == 0 && BN % 64 == 0 && WS >= 2 && AS >= 2 && (WS - 2) * kWL < 64 && (AS - 2) * kAL < 64,
                "rings");
  static_assert(kLds <= 160 * 1024, "LDS");
};

// vmcnt(n), lgkmcnt(0); expcnt at its maximum
#define DOMINO_I8_WAIT(n) __builtin_amdgcn_s_waitcnt(((n) & 15) | (((n) >> 4) << 14) | 0x0070)

template <int BM, int BN, int WS, int AS, int P>
__global__ void __launch_bounds__(512, 1)
    gemm_i8_tiled_kernel(const int8_t* __restrict__ A, const float* __restrict__ as, int M,
                         const int8_t* __restrict__ W, const float* __restrict__ ws, int N, int K,
                         float* __restrict__ C, int num_m, int num_n) {
  using T = TileI8<BM, BN, WS, AS, P>;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  const int wave = wave_id(), lane = threadIdx.x & 63, grp = lane >> 4, col = lane & 15;
  const int wm = wave >> 2, wn = wave & 3;
  // one XCD takes every M tile of an N tile back to back (workgroups go
  // round-robin over 8 XCDs): W comes from memory once and from its L2 after
  const int xcd = blockIdx.x & 7, per_xcd = gridDim.x >> 3;
  const int xcd_tiles = ((num_n + 7 - xcd) >> 3) * num_m;  // N tiles xcd, xcd + 8, ...
  const int first = blockIdx.x >> 3;
  if (first >= xcd_tiles) return;
  const int mine = (xcd_tiles - first + per_xcd - 1) / per_xcd;
  const int nd = (K + 127) >> 7;
  const int total = mine * nd;  // steps of all tiles
  auto tile_at = [&](int i, int& m0, int& n0) {
    const int l = first + i * per_xcd, nl = l / num_m;
    m0 = (l - nl * num_m) * BM;
    n0 = (nl * 8 + xcd) * T::kBN;
  };

  // loading: load i of wave w covers rows 32 i + 8 (w & 3) .. + 7 of the operand
  const bool loads_w = wm == 0;
  const int lrow = (wave & 3) * 8 + (lane >> 3), chunk = (lane & 7) ^ (lane >> 3);
  // this lane's bytes of a tile's last step lie past K: A reads zeros there, W
  // its row's first bytes of the step
  const bool past = (nd - 1) * 128 + chunk * 16 >= K;
  const int8_t* base = A;  // the tile's first row
  int last_row = 0;        // the operand's last row, counted from it
  int it = 0, id = 0, islot = 0;  // the next step to load: tile, step, ring slot
  int turn = 0;                   // the step of K that the tile begins with
  auto seek = [&]() {
    int m0, n0;
    tile_at(it, m0, n0);
    const int r0 = loads_w ? n0 : m0, rows = loads_w ? N : M;
    base = (loads_w ? W : A) + (size_t)r0 * K;
    last_row = rows - 1 - r0;
    turn = num_m == 1 ? (int)((unsigned)(n0 / T::kBN * 5) % (unsigned)nd) : 0;
  };
  auto issue = [&]() {
    const int kd = id + turn < nd ? id + turn : id + turn - nd;
    const bool skip = past && kd == nd - 1;
    const int8_t* p = base + kd * 128;
    const uint32_t c16 = chunk * 16;
    if (loads_w) {
      unsigned char* dst = smem + islot * T::kWBytes + (wave & 3) * 1024;
#pragma unroll
      for (int i = 0; i < T::kWL; ++i)
        __builtin_amdgcn_global_load_lds((gptr_t)(p + (uint32_t)(min(i * 32 + lrow, last_row) * K) + (skip ? 0 : c16)),
                                         (lptr_t)(dst + i * 4096), 16, 0, kLoadNonTemporal);
      if (++islot == WS) islot = 0;
    } else {
      unsigned char* dst = smem + WS * T::kWBytes + islot * T::kABytes + (wave & 3) * 1024;
#pragma unroll
      for (int i = 0; i < T::kAL; ++i) {
        const void* q = p + (uint32_t)(min(i * 32 + lrow, last_row) * K) + c16;
        if (skip) q = kZeros;
        __builtin_amdgcn_global_load_lds((gptr_t)q, (lptr_t)(dst + i * 4096), 16, 0, 0);
      }
      if (++islot == AS) islot = 0;
    }
    if (++id == nd) {
      id = 0;
      if (++it < mine) seek();
    }
  };

  i32x4 acc[T::kFA][T::kFW];
#pragma unroll
  for (int i = 0; i < T::kFA; ++i)
#pragma unroll
    for (int j = 0; j < T::kFW; ++j) acc[i][j] = i32x4{0, 0, 0, 0};

  // The tile's scales: loaded at its start, into LDS where there is room, else
  // into registers that are taken (the empty asm) behind a wait that the operands
  // need anyway.  Loaded where they are used, every store would wait for the loads
  // in flight.
  float sn[T::kFW][4], sm[T::kFA];
  int m0, n0;
  float* lds_scales = reinterpret_cast<float*>(smem + T::kRings);  // [2][BN of ws, BM of as]
  auto scales = [&](int parity) {
    if constexpr (T::kScalesInLds) {
      // 64 scales a load, dealt out to the waves that load the operand
      float* dst = lds_scales + parity * (BM + BN);
      const int w = wave & 3;
      if (loads_w) {
#pragma unroll
        for (int i = 0; i < BN / 64; ++i)
          if (i % 4 == w)
            __builtin_amdgcn_global_load_lds((gptr_t)(ws + min(n0 + i * 64 + lane, N - 1)), (lptr_t)(dst + i * 64), 4,
                                             0, 0);
      } else {
#pragma unroll
        for (int i = 0; i < BM / 64; ++i)
          if (i % 4 == w)
            __builtin_amdgcn_global_load_lds((gptr_t)(as + min(m0 + i * 64 + lane, M - 1)), (lptr_t)(dst + BN + i * 64),
                                             4, 0, 0);
      }
      return;
    }
#pragma unroll
    for (int j = 0; j < T::kFW; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) sn[j][q] = ws[min(n0 + (wn * T::kFW + j) * 16 + grp * 4 + q, N - 1)];
#pragma unroll
    for (int i = 0; i < T::kFA; ++i) sm[i] = as[min(m0 + (wm * T::kFA + i) * 16 + col, M - 1)];
  };
  auto take_scales = [&]() {
    if constexpr (T::kScalesInLds) return;
#pragma unroll
    for (int j = 0; j < T::kFW; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) asm volatile("" : "+v"(sn[j][q]));
#pragma unroll
    for (int i = 0; i < T::kFA; ++i) asm volatile("" : "+v"(sm[i]));
  };
  const bool vec = (N & 3) == 0;  // then every group of 4 columns is 16-byte aligned and whole
  // (writes the results and clears them)
  auto store = [&](int parity, i32x4 (&acc)[T::kFA][T::kFW], int m0, int n0) {
    if constexpr (T::kScalesInLds) {
      const float* src = lds_scales + parity * (BM + BN);
#pragma unroll
      for (int j = 0; j < T::kFW; ++j) {
        const f32x4 v = *reinterpret_cast<const f32x4*>(src + (wn * T::kFW + j) * 16 + grp * 4);
#pragma unroll
        for (int q = 0; q < 4; ++q) sn[j][q] = v[q];
      }
#pragma unroll
      for (int i = 0; i < T::kFA; ++i) sm[i] = src[BN + (wm * T::kFA + i) * 16 + col];
    }
    if (vec && m0 + BM <= M && n0 + T::kBN <= N) {  // a whole tile
      float* c = C + (size_t)(m0 + wm * T::kFA * 16 + col) * N + n0 + wn * T::kFW * 16 + grp * 4;
#pragma unroll
      for (int i = 0; i < T::kFA; ++i) {
#pragma unroll
        for (int j = 0; j < T::kFW; ++j) {
          f32x4 v;
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] = (float)acc[i][j][q] * sm[i] * sn[j][q];
          acc[i][j] = i32x4{0, 0, 0, 0};
          *reinterpret_cast<f32x4*>(c + j * 16) = v;
        }
        c += (size_t)16 * N;
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < T::kFA; ++i) {
      const int m = m0 + (wm * T::kFA + i) * 16 + col;
      float* c = C + (size_t)m * N;
#pragma unroll
      for (int j = 0; j < T::kFW; ++j) {
        const int n = n0 + (wn * T::kFW + j) * 16 + grp * 4;
        f32x4 v;
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = (float)acc[i][j][q] * sm[i] * sn[j][q];
        acc[i][j] = i32x4{0, 0, 0, 0};
        if (m < M) {
          if (vec) {
            if (n < N) *reinterpret_cast<f32x4*>(c + n) = v;
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (n + q < N) c[n + q] = v[q];
          }
        }
      }
    }
  };

  seek();
  const int ahead = loads_w ? WS - 1 : AS - 1;
  for (int q = 0; q < ahead; ++q)
    if (q < total) issue();
  DOMINO_I8_WAIT(0);
  __builtin_amdgcn_s_barrier();
  if (wm == 1) __builtin_amdgcn_s_barrier();  // the second row of waves starts one phase later

  int d = 0, tile = 0, sa_slot = 0, sw_slot = 0;
  tile_at(0, m0, n0);
  // the first tile of a pair, while the second is being multiplied
  i32x4 kept[P == 2 ? T::kFA : 1][P == 2 ? T::kFW : 1];
  bool have = false;
  int km = 0, kn = 0;
  for (int g = 0; g < total; ++g) {
    const unsigned char* sW = smem + sw_slot * T::kWBytes + wn * T::kFW * 2048 + col * 128;
    const unsigned char* sA = smem + WS * T::kWBytes + sa_slot * T::kABytes + wm * T::kFA * 2048 + col * 128;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      __builtin_amdgcn_sched_barrier(0);
      const int slot = ((h * 4 + grp) ^ (col & 7)) * 16;
      u32x4 af[T::kFA], wf[T::kFW];
#pragma unroll
      for (int j = 0; j < T::kFW; ++j) wf[j] = ld16(sW + j * 2048 + slot);
#pragma unroll
      for (int i = 0; i < T::kFA; ++i) af[i] = ld16(sA + i * 2048 + slot);
      if (h == 0) {
        if (d == 0) scales(tile & (2 * P - 1));
        if (g + ahead < total) issue();
        if (T::kScalesInLds && nd == 1) {
          // a tile of one step: the first row of waves stores while the second is
          // still reading, so the scales have to be there by now
          if (g + ahead >= total)
            DOMINO_I8_WAIT(0);
          else if (loads_w)
            DOMINO_I8_WAIT(T::kWL);
          else
            DOMINO_I8_WAIT(T::kAL);
        } else {
          __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
        }
      } else if (g + ahead >= total) {
        DOMINO_I8_WAIT(0);
      } else if (loads_w) {
        DOMINO_I8_WAIT((WS - 2) * T::kWL);
      } else {
        DOMINO_I8_WAIT((AS - 2) * T::kAL);
      }
      if (h == 1 && d == 0) take_scales();
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < T::kFA; ++i)
#pragma unroll
        for (int j = 0; j < T::kFW; ++j) acc[i][j] = mma16_i8(acc[i][j], wf[j], af[i]);
      __builtin_amdgcn_sched_barrier(0);
      if (h == 1 && d == nd - 1) {
        if (P == 2 && !have && tile + 1 < mine) {
#pragma unroll
          for (int i = 0; i < T::kFA; ++i)
#pragma unroll
            for (int j = 0; j < T::kFW; ++j) {
              if constexpr (P == 2) kept[i][j] = acc[i][j];
              acc[i][j] = i32x4{0, 0, 0, 0};
            }
          have = true;
          km = m0;
          kn = n0;
        } else {
          if constexpr (P == 2)
            if (have) store((tile - 1) & 3, kept, km, kn);
          store(tile & (2 * P - 1), acc, m0, n0);
          have = false;
        }
      }
      __builtin_amdgcn_s_barrier();
    }
    if (++sa_slot == AS) sa_slot = 0;
    if (++sw_slot == WS) sw_slot = 0;
    if (++d == nd) {
      d = 0;
      if (++tile < mine) tile_at(tile, m0, n0);
    }
  }
  if (wm == 0) __builtin_amdgcn_s_barrier();  // equal barrier counts in both rows of waves
}

template <int BM, int BN, int WS, int AS, int P>
static hipError_t launch_tiled(const int8_t* A, const float* as, int M, const int8_t* W, const float* ws, int N, int K,
                               float* C, int num_cu, hipStream_t s) {
  using T = TileI8<BM, BN, WS, AS, P>;
  const int num_m = (M + BM - 1) / BM, num_n = (N + T::kBN - 1) / T::kBN;
  // a multiple of 8 workgroups, at most one a compute unit
  const int want = (num_n + 7) / 8 * num_m, have = std::max(1, num_cu / 8);
  auto kern = gemm_i8_tiled_kernel<BM, BN, WS, AS, P>;
  static std::atomic<uint64_t> done{0};
  const hipError_t e = allow_lds(reinterpret_cast<const void*>(kern), T::kLds, done);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3((unsigned)(8 * std::min(want, have))), dim3(T::kThreads), T::kLds, s, A, as, M, W, ws,
                     N, K, C, num_m, num_n);
  return hipGetLastError();
}

hipError_t launch_gemm_i8(const int8_t* A, const float* a_scale, int M, const int8_t* W, const float* w_scale, int N,
                          int K, float* C, int num_cu, hipStream_t s) {
  if (M <= 0 || N <= 0) return hipSuccess;
  if (K <= 0 || K % 32 || K > 8192) return hipErrorNotSupported;
  // Up to 64 rows W is streamed past A in registers (Qwen3-8B head, 64 rows:
  // 118 us against 170 tiled, before its tiles went in pairs); above, two
  // workgroups would share each stream (128 rows: 160 us, against 135 tiled).
  if (M <= 64 && K <= 4096) {
    if (K <= 256) return launch_stream<4, 1>(A, a_scale, M, W, w_scale, N, K, C, num_cu, s);
    if (K <= 512) return launch_stream<4, 2>(A, a_scale, M, W, w_scale, N, K, C, num_cu, s);
    if (K <= 1024) return launch_stream<4, 4>(A, a_scale, M, W, w_scale, N, K, C, num_cu, s);
    if (K <= 2048) return launch_stream<4, 8>(A, a_scale, M, W, w_scale, N, K, C, num_cu, s);
    if (K <= 2560) return launch_stream<5, 8>(A, a_scale, M, W, w_scale, N, K, C, num_cu, s);
    return launch_stream<8, 8>(A, a_scale, M, W, w_scale, N, K, C, num_cu, s);
  }
  if (M <= 16) return launch_stream_g<16, 8, 1>(A, a_scale, M, W, w_scale, N, K, C, num_cu, s);
  if (M > 128) return launch_tiled<256, 256, 2, 3, 1>(A, a_scale, M, W, w_scale, N, K, C, num_cu, s);
  // One M tile: 256 or 320 columns a tile, whichever leaves a compute unit fewer
  // columns in all (vocabulary 151936 on 256 compute units: 3 rounds of 256 or 2 of
  // 320; 128 rows, d = 1024: 53 and 48 us, 2560: 101.5 and 99.7); but 256 for long
  // rows, unless 320 take a single round, as its deeper ring of A then counts for
  // more (d = 3200: 117 us both; 3584: 122 and 129, 4096: 135 and 150, 5120: 186 and
  // 181, 8192: 247 and 258; in one round, vocabulary 80000, d = 4096: 90 and 74).
  auto columns = [&](int bn) { return ((N + bn - 1) / bn + num_cu - 1) / num_cu * bn; };
  const int wide = columns(320);
  return wide < columns(256) && (K <= 3200 || wide == 320)
             ? launch_tiled<128, 320, 3, 2, 2>(A, a_scale, M, W, w_scale, N, K, C, num_cu, s)
             : launch_tiled<128, 256, 3, 3, 2>(A, a_scale, M, W, w_scale, N, K, C, num_cu, s);
}

}  // namespace domino
