// MXFP4 operands and their product on gfx950 (gift_mx_* of include/gift.h).
//
// An operand (rows x k) is cut into blocks of 64 rows x 128 k elements, 4352
// bytes each: four 1 KB fragments of 16 rows, then 256 bytes of scales.  A
// fragment is what one v_mfma_scale_f32_16x16x128_f8f6f4 takes from a wave:
// lane l holds row l % 16, k elements 32 (l / 16) .. +31, i.e. exactly one
// 32-element MX block (16 bytes of E2M1 codes) with one E8M0 scale.  The
// scale dword of lane l holds the bytes of the block's four fragments, which
// the instruction picks by its byte select, so neither codes nor scales need
// any rearranging between memory and the matrix cores.
#include <type_traits>

#include "device.hpp"
#include "mx.hpp"
#include "product.hpp"

namespace gift {

namespace {

typedef __attribute__((ext_vector_type(8))) int i32x8;
typedef __attribute__((ext_vector_type(4))) int i32x4;

constexpr int kFmtFp4 = 4;  // f8f6f4 operand format: E2M1

// acc += (fragment a) x (fragment b)^T with byte SA of a's and SB of b's scales
template <int SA, int SB>
__device__ __forceinline__ f32x4 mx_mfma(const i32x4& a, int sa, const i32x4& b, int sb, f32x4 acc) {
  const i32x8 va = {a[0], a[1], a[2], a[3], 0, 0, 0, 0};
  const i32x8 vb = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(va, vb, acc, kFmtFp4, kFmtFp4, SA, sa, SB, sb);
}

__device__ __forceinline__ float ld1(const float* p) { return *p; }
__device__ __forceinline__ float ld1(const __bf16* p) { return (float)*p; }

// ---------------------------------------------------------------------------
// quantize
// ---------------------------------------------------------------------------

// One MX block: 32 values -> 16 bytes of codes and the scale byte.
__device__ __forceinline__ uint4 mx_block(const float (&v)[32], uint32_t& code, uint32_t& flags) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const uint32_t b = abs_bits(v[i]);
    m = m > b ? m : b;
  }
  code = mx_scale_code(m, flags);
  const float s = mx_scale_operand(code);
  const bool nonfinite = code == kMxScaleNaN;
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = mx_encode4(make_float4(v[8 * i], v[8 * i + 1], v[8 * i + 2], v[8 * i + 3]), s, nonfinite) |
           mx_encode4(make_float4(v[8 * i + 4], v[8 * i + 5], v[8 * i + 6], v[8 * i + 7]), s, nonfinite) << 16;
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void unpack2(uint32_t w, float& a, float& b) {
  a = __uint_as_float(w << 16);
  b = __uint_as_float(w & 0xffff0000u);
}

// A quantize tile: a row panel and half a k step of either operand.
constexpr int kQRows = 64, kQCols = 64;
constexpr int kQBlocks = kQRows * kQCols / 32;  // of one operand, a thread each

// One tile of X through LDS, a block of 32 per thread; X is read once for
// both operands, whose blocks have threads of their own.  Bound by memory:
// 16384 x 4096 bf16 into both 36 to 39 us on inputs in turn, 205 MB at 5.3 to
// 5.7 TB/s (33 us on one input, then in part in the memory-side cache); a
// copy: 4.9.  Small matrices are bound by a launch
// and the chain of load, encode and store: with 128 rows a tile and a block of
// each operand in turn per thread 1000 x 1024 took 3.8 us, now 3.1, 2816 x 1024
// fp32 4.9 and 4.0, 16384 x 4096 fp32 61.7 and 60.6; with 128 columns a tile
// 16384 x 4096 bf16 took an eighth longer.  By rows: 32 consecutive columns
// of a row, threads in fragment order, so 32 lanes write 512 contiguous bytes
// of a fragment.  By columns: 32 rows of a column.  The LDS row stride is 4
// banks past a multiple of 32, so the 16 rows of a fragment fall in 16
// distinct groups of 4 banks.
template <class T, bool kByRow, bool kByCol>
__global__ __launch_bounds__((kByRow + kByCol) * kQBlocks) void k_mx_quant(
    const T* __restrict__ X, int64_t rows, int64_t cols, int64_t ld, uint8_t* R, uint8_t* C, int col_tiles,
    uint32_t* flags) {
  constexpr int kQThreads = (kByRow + kByCol) * kQBlocks;
  constexpr int kPer = 16 / sizeof(T);                  // elements of a 16-byte load
  constexpr int kStride = kQCols * sizeof(T) + 16;      // bytes of an LDS row
  constexpr int kChunks = kQCols / kPer;                // 16-byte chunks of a row
  constexpr int kLoads = kQRows * kChunks / kQThreads;  // chunks per thread
  __shared__ __attribute__((aligned(16))) char lds[kQRows * kStride];
  const int t = threadIdx.x;
  const int id = blockIdx.y * gridDim.x + blockIdx.x;
  const int tr = id / col_tiles, tc = id - tr * col_tiles;
  const int64_t r0 = (int64_t)tr * kQRows, c0 = (int64_t)tc * kQCols;
  // Loads go out together, from addresses clamped into X; what lies outside
  // becomes zero.
  if (cols >= kPer) {
    uint4 v[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int e = t + i * kQThreads;
      const int64_t r = min(r0 + e / kChunks, rows - 1), c = min(c0 + e % kChunks * kPer, cols - kPer);
      v[i] = ld16(X + r * ld + c);
    }
    // the chunk that the columns end in was loaded `over` elements early
    const int over = (int)(kPer - cols % kPer) % kPer;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int e = t + i * kQThreads, r = e / kChunks, c = e % kChunks;
      const int64_t left = cols - (c0 + c * kPer);
      if (r0 + r >= rows || left <= 0) {
        v[i] = make_uint4(0, 0, 0, 0);
      } else if (left < kPer) {
        T* to = reinterpret_cast<T*>(lds + r * kStride + c * 16);
        T x[kPer];
        __builtin_memcpy(x, &v[i], 16);
#pragma unroll
        for (int j = 0; j < kPer; ++j) to[(j - over + kPer) % kPer] = j < over ? (T)0.f : x[j];
        continue;
      }
      *reinterpret_cast<uint4*>(lds + r * kStride + c * 16) = v[i];
    }
  } else {
    for (int e = t; e < kQRows * kQCols; e += kQThreads) {
      const int r = e / kQCols, c = e % kQCols;
      T x = (T)0.f;
      if (r0 + r < rows && c0 + c < cols) x = X[(r0 + r) * ld + c0 + c];
      *reinterpret_cast<T*>(lds + r * kStride + c * sizeof(T)) = x;
    }
  }
  __syncthreads();
  uint32_t fl = 0;
  if (kByRow && t < kQBlocks) {
    // 4 fragments x 2 blocks x 16 rows; the panel's steps cover an even
    // number of tiles, the last of which may lie past the columns (zeros)
    const int f = t >> 5, bb = (t >> 4) & 1, r = f * 16 + (t & 15);
    if (r0 < rows) {
      float v[32];
      const char* src = lds + r * kStride + bb * 32 * sizeof(T);
#pragma unroll
      for (int j = 0; j < 32 / kPer; ++j) {
        const uint4 q = *reinterpret_cast<const uint4*>(src + 16 * j);
        if constexpr (sizeof(T) == 2) {
          unpack2(q.x, v[8 * j], v[8 * j + 1]);
          unpack2(q.y, v[8 * j + 2], v[8 * j + 3]);
          unpack2(q.z, v[8 * j + 4], v[8 * j + 5]);
          unpack2(q.w, v[8 * j + 6], v[8 * j + 7]);
        } else {
          v[4 * j] = __uint_as_float(q.x);
          v[4 * j + 1] = __uint_as_float(q.y);
          v[4 * j + 2] = __uint_as_float(q.z);
          v[4 * j + 3] = __uint_as_float(q.w);
        }
      }
      uint32_t code, bf = 0;
      const uint4 w = mx_block(v, code, bf);
      if (r0 + r < rows && c0 + bb * 32 < cols) fl |= bf;
      const int lane = ((tc & 1) * 2 + bb) * 16 + (t & 15);
      uint8_t* out = R + ((int64_t)tr * (col_tiles / 2) + (tc >> 1)) * kMxPanel;
      *reinterpret_cast<uint4*>(out + f * 1024 + lane * 16) = w;
      out[4096 + lane * 4 + f] = (uint8_t)code;
    }
  }
  if (kByCol && t >= kQThreads - kQBlocks) {
    // as above, an even number of tiles down the columns
    const int64_t steps = (rows + kMxStep - 1) / kMxStep;
    const int b = (t - (kQThreads - kQBlocks)) >> 6, c = t & 63;  // rows 32 b .. +31 of column c
    if (c0 < cols && (tr >> 1) < steps) {
      float v[32];
#pragma unroll
      for (int j = 0; j < 32; ++j)
        v[j] = ld1(reinterpret_cast<const T*>(lds + (b * 32 + j) * kStride + c * sizeof(T)));
      uint32_t code, bf = 0;
      const uint4 w = mx_block(v, code, bf);
      if (r0 + b * 32 < rows && c0 + c < cols) fl |= bf;
      uint8_t* out = C + (tc * steps + (tr >> 1)) * (int64_t)kMxPanel;
      const int f = c >> 4, lane = ((tr & 1) * 2 + b) * 16 + (c & 15);
      *reinterpret_cast<uint4*>(out + f * 1024 + lane * 16) = w;
      out[4096 + lane * 4 + f] = (uint8_t)code;
    }
  }
  if (flags && fl) atomicOr(flags, fl);
}

// A 64 x 128 block of the operand per workgroup: through LDS, then a thread
// decodes 16 bytes of a row.  Bound by its stores, which go around the caches
// where rows start aligned: 16384 x 4096 to bf16 38 -> 26 us, 170 MB at 6.5
// TB/s (and through them where not: 4095 columns 63 -> 36 us).
template <class T, bool kNt>
__global__ __launch_bounds__(256) void k_mx_dequant(const uint8_t* __restrict__ A, int64_t rows,
                                                    int64_t k, int steps, T* out, int64_t ld) {
  constexpr int kPer = 16 / sizeof(T), kPieces = kMxStep / kPer;  // a row of the block
  __shared__ __attribute__((aligned(16))) uint8_t lds[kMxPanel];
  const int t = threadIdx.x;
  const int64_t panel = blockIdx.x / steps;
  const int s = (int)(blockIdx.x - panel * steps);
  const uint8_t* src = A + (int64_t)blockIdx.x * kMxPanel;
  for (int i = t; i < kMxPanel / 16; i += 256)
    *reinterpret_cast<uint4*>(lds + 16 * i) = *reinterpret_cast<const uint4*>(src + 16 * i);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kMxRows * kPieces / 256; ++i) {
    const int e = t + 256 * i, r = e / kPieces, piece = e % kPieces, b = piece * kPer / 32;
    const int64_t row = panel * kMxRows + r, col = (int64_t)s * kMxStep + piece * kPer;
    if (row >= rows || col >= k) continue;
    const int lane = b * 16 + (r & 15), f = r >> 4;
    const uint8_t* codes = lds + f * 1024 + lane * 16 + piece * kPer % 32 / 2;
    const uint32_t sc = lds[4096 + lane * 4 + f];
    T o[kPer];
#pragma unroll
    for (int j = 0; j < kPer / 4; ++j) {
      const float4 v = mx_decode4(reinterpret_cast<const uint16_t*>(codes)[j], sc);
      o[4 * j] = (T)v.x;
      o[4 * j + 1] = (T)v.y;
      o[4 * j + 2] = (T)v.z;
      o[4 * j + 3] = (T)v.w;
    }
    T* dst = out + row * ld + col;
    uint4 w;
    __builtin_memcpy(&w, o, 16);
    if (col + kPer <= k) {
      if constexpr (kNt) st16_nt(dst, w);
      else st16(dst, w);
    } else {
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (col + j < k) dst[j] = o[j];
    }
  }
}

// ---------------------------------------------------------------------------
// product
// ---------------------------------------------------------------------------

struct MxGemm {
  const uint8_t* A;
  const uint8_t* B;
  void* C;
  const float* bias;
  float* part;     // split-k partials, [split][M][N] fp32
  int64_t ldc;
  int M, N;
  int steps;       // k steps of 128
  int per_split;   // k steps of a split
  int tm, tn;      // tiles
  int n_split;
  int mode;        // kOut*
};
enum { kOutBf16 = 0, kOutF32 = 1, kOutAcc = 2 };

// Four consecutive columns n .. n + 3 of row m.
__device__ __forceinline__ void mx_store4(const MxGemm& g, int m, int n, f32x4 v) {
  if (m >= g.M || n >= g.N) return;
  const bool whole = n + 4 <= g.N;
  if (g.bias)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < g.N) v[e] += g.bias[n + e];
  const int64_t at = (int64_t)m * g.ldc + n;
  if (g.mode == kOutBf16) {
    uint16_t* p = static_cast<uint16_t*>(g.C) + at;
    using any8 = unsigned __attribute__((ext_vector_type(2), aligned(2)));
    if (whole)
      *reinterpret_cast<any8*>(p) = any8{bf16_bits(v[0]) | bf16_bits(v[1]) << 16,
                                         bf16_bits(v[2]) | bf16_bits(v[3]) << 16};
    else
      for (int e = 0; e < 4 && n + e < g.N; ++e) p[e] = (uint16_t)bf16_bits(v[e]);
    return;
  }
  float* p = static_cast<float*>(g.C) + at;
  if (whole) {
    if (g.mode == kOutAcc) v += __builtin_bit_cast(f32x4, ld16(p));
    st16(p, __builtin_bit_cast(uint4, v));
  } else {
    for (int e = 0; e < 4 && n + e < g.N; ++e) p[e] = g.mode == kOutAcc ? p[e] + v[e] : v[e];
  }
}

// The product on tiles of (WR FA 16) x (WC FB 16): WR x WC waves, each with
// FA x FB accumulator tiles; a workgroup takes one tile and one range of k
// steps.  The operands' blocks of a step are copied as they lie into one of
// kStages LDS stages by the buffer unit; the fragments come out of LDS with
// one conflict-free 16-byte read per lane.  Per step i: wait until step
// i + 1's copies have landed, barrier, then run step i's MFMAs with, spread
// between them, the copies of step i + kStages into the stage that step i has
// left and the reads of step i + 1's fragments into the other register set.
// Two workgroups of 128 x 256 or three of 128 x 128 share a CU, so one's
// results leave under the other's MFMAs.  The loop holds no branch: the
// compiler would sink the MFMAs below it, away from the copies and reads they
// are spread among.
//
// Bound by power and by the loop's copies and LDS reads: on large products the
// matrix units are busy 65% of the cycles (SQ counters) at the 1.6 GHz that
// the clock falls to, 3.6 to 4.6 PFLOP/s; a loop of these MFMAs alone on the
// same random codes, with no loads, reaches 5.6 to 7.3 (9.7 on zeros), and of
// the time of a 256 x 256 loop 15% went without its copies or without its LDS
// reads, 25% without both.  With 12 k steps (16384 x 4096 x 1536, 62 to 70 us,
// 2.9 to 3.3 PFLOP/s) or one round of tiles (1999 x 4096 x 4096, 20 to 23 us)
// the three stages filled before a tile's first MFMA and the results stored
// after its last show: nothing of the same workgroup runs beside them.
// Accumulating reads C through the caches (11008 x 4096 x 16384 411 us, 336
// without; 4096 x 1536 x 16384 65 and 63).  LDS traffic decides among tiles: a
// wave of 128 x 64 reads 12 fragments for 32 MFMAs, one of 64 x 64 eight for 16.
// Measured against it, 16384 x 1536 x 4096 / 16384 x 4096 x 11008: 128 x 256
// tiles 52.7 / 338 us (waves of 64 x 128: 53.7 / 338), two waves of 128 x 128 a
// tile 65.7 / 348, 256 x 256 tiles, one to a CU, running on from tile to tile 64
// / 332, 128 x 128 tiles 55.9 / -.
template <int WR, int WC, int FA, int FB, int kStages, int kOut, bool kBias, bool kNt>
__global__ __launch_bounds__(64 * WR * WC, FA * FB > 16 ? 2 : 3) void k_mx_gemm(MxGemm g) {
  constexpr int kWaves = WR * WC;
  constexpr int kPA = WR * FA / 4, kPB = WC * FB / 4;  // panels of the tile
  static_assert(FA % 4 == 0 && FB % 4 == 0 && kPA * 4 % kWaves == 0 && kPB * 4 % kWaves == 0, "whole panels");
  constexpr int kStage = (kPA + kPB) * kMxPanel;
  // A wave's copies of a step: fragments of A and of B, then scales of a
  // panel or more of each (where waves outnumber panels, some copy the same)
  constexpr int kFA = kPA * 4 / kWaves, kFB = kPB * 4 / kWaves;
  constexpr int kSA = (kPA + kWaves - 1) / kWaves, kSB = (kPB + kWaves - 1) / kWaves;
  constexpr int kVm = kFA + kFB + kSA + kSB;
  constexpr int kRowData = FB * 32 > 256 ? 256 : FB * 32;  // bytes of a staged row of C
  constexpr int kRow = kRowData + 16;  // 4 banks past a power of two: 16 rows of one column, no conflict
  static_assert(kWaves * 16 * kRow <= kStages * kStage, "the results' staging fits in the stages");
  __shared__ __attribute__((aligned(1024))) char lds[kStages * kStage];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = w / WC, wc = w % WC;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds;

  const int tiles = g.tm * g.tn, split = (int)blockIdx.x / tiles;
  int ti, tj;
  tile_of((int)blockIdx.x - split * tiles, g.tm, g.tn, ti, tj);
  const int s0 = split * g.per_split, n_steps = min(g.steps, s0 + g.per_split) - s0;
  const int steps = (n_steps + 1) & ~1;

  // The tile's first panel of A and of B as raw buffers, and for every copy
  // of the wave its offset from there.  Panels past an operand's last repeat
  // it (their rows and columns of C are not written); steps past the last
  // lie outside both buffers and so become zeros.
  int c_step = 0, c_slot = 0;
  __amdgpu_buffer_rsrc_t rs[2];
  uint32_t vo[kVm];
  {
    const int fa = ti * kPA, fb = tj * kPB;  // first panels, and how many lie in the operand
    const int na = min(kPA, (g.M + kMxRows - 1) / kMxRows - fa), nb = min(kPB, (g.N + kMxRows - 1) / kMxRows - fb);
    const int64_t len = (int64_t)g.steps * kMxPanel;
    auto buffer = [&](const uint8_t* base, int first, int n) {
      return __builtin_amdgcn_make_buffer_rsrc(
          reinterpret_cast<void*>(uniform64(reinterpret_cast<uint64_t>(base) + first * len + (int64_t)s0 * kMxPanel)),
          (short)0, __builtin_amdgcn_readfirstlane((int)(uint32_t)(n * len - (int64_t)s0 * kMxPanel)),
          (int)kRawBufferWord3);
    };
    rs[0] = buffer(g.A, fa, na);
    rs[1] = buffer(g.B, fb, nb);
#pragma unroll
    for (int d = 0; d < kFA; ++d)
      vo[d] = (uint32_t)(min((w * kFA + d) / 4, na - 1) * len) + (w * kFA + d) % 4 * 1024 + lane * 16;
#pragma unroll
    for (int d = 0; d < kFB; ++d)
      vo[kFA + d] = (uint32_t)(min((w * kFB + d) / 4, nb - 1) * len) + (w * kFB + d) % 4 * 1024 + lane * 16;
#pragma unroll
    for (int d = 0; d < kSA; ++d)
      vo[kFA + kFB + d] = (uint32_t)(min((w + d * kWaves) % kPA, na - 1) * len) + 4096 + lane * 4;
#pragma unroll
    for (int d = 0; d < kSB; ++d)
      vo[kFA + kFB + kSA + d] = (uint32_t)(min((w + d * kWaves) % kPB, nb - 1) * len) + 4096 + lane * 4;
  }
  // copy `d` of the wave's kVm of a step
  auto copy = [&](auto D) {
    constexpr int d = decltype(D)::value;
    // The step goes into the vector offset, which the bounds check covers;
    // kOutside lies past four of the longest panels and does not carry.
    constexpr uint32_t kOutside = 0x89000000u, kLen = ((1u << 24) / kMxStep) * kMxPanel;
    static_assert(kOutside >= 4 * kLen && 3ull * kLen + kMxPanel + kOutside <= ~0u, "outside every buffer");
    const uint32_t to = lds0 + (uint32_t)c_slot * kStage;
    const uint32_t from = vo[d] + (c_step < n_steps ? (uint32_t)c_step * kMxPanel : kOutside);
    if constexpr (d < kFA)
      dma16(rs[0], to + (w * kFA + d) / 4 * kMxPanel + (w * kFA + d) % 4 * 1024, from);
    else if constexpr (d < kFA + kFB)
      dma16(rs[1], to + (kPA + (w * kFB + d - kFA) / 4) * kMxPanel + (w * kFB + d - kFA) % 4 * 1024, from);
    else if constexpr (d < kFA + kFB + kSA)
      dma4(rs[0], to + (w + (d - kFA - kFB) * kWaves) % kPA * kMxPanel + 4096, from);
    else
      dma4(rs[1], to + (kPA + (w + (d - kFA - kFB - kSA) * kWaves) % kPB) * kMxPanel + 4096, from);
  };
  auto copied = [&] {
    c_slot = c_slot + 1 == kStages ? 0 : c_slot + 1;
    ++c_step;
  };

  struct Frags {
    i32x4 f[FB + FA];  // B's, then A's
    int s[(FB + FA) / 4];
  };
  const char* rb = lds + (kPA + wc * (FB / 4)) * kMxPanel + lane * 16;
  const char* ra = lds + wr * (FA / 4) * kMxPanel + lane * 16;
  constexpr int kReads = (FA + FB) / 4 * 5;
  // read `d` of a step's kReads: per panel the scales, then four fragments
  auto read = [&](auto D, Frags& r, int o) {
    constexpr int d = decltype(D)::value, p = d / 5, e = d % 5;
    constexpr bool isb = p < FB / 4;
    const char* at = (isb ? rb + p * kMxPanel : ra + (p - FB / 4) * kMxPanel) + o;
    if constexpr (e == 0) r.s[p] = *reinterpret_cast<const int*>(at + 4096 - lane * 12);
    else r.f[p * 4 + e - 1] = *reinterpret_cast<const i32x4*>(at + (e - 1) * 1024);
  };

  f32x4 acc[FA][FB];
#pragma unroll
  for (int i = 0; i < FA; ++i)
#pragma unroll
    for (int j = 0; j < FB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

#pragma unroll
  for (int s = 0; s < kStages; ++s) {
    static_for<kVm>(copy);
    copied();
  }
  __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0((kStages - 1) * kVm));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  Frags fr[2];
  static_for<kReads>([&](auto D) { read(D, fr[0], 0); });
  int slot = 0;
  auto step = [&](auto P) {
    constexpr int p = decltype(P)::value;
    const int next = slot + 1 == kStages ? 0 : slot + 1;
    // step i's fragments are in registers, step i + 1's copies have landed
    __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0((kStages - 2) * kVm));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    const Frags& r = fr[p];
    constexpr int kGroups = FA * FB / 4, kSide = kReads + kVm;
    const int o = next * kStage;
    // reads and copies in their proportion
    static_for<kGroups>([&](auto G) {
      constexpr int gr = decltype(G)::value;
      constexpr int s0 = gr * kSide / kGroups, s1 = (gr + 1) * kSide / kGroups;
      static_for<s1 - s0>([&](auto S) {
        constexpr int k = s0 + decltype(S)::value;
        constexpr int c = k * kVm / kSide;  // copies before side op k
        if constexpr ((k + 1) * kVm / kSide > c) copy(std::integral_constant<int, c>{});
        else read(std::integral_constant<int, k - c>{}, fr[1 - p], o);
      });
      constexpr int i = gr / (FB / 4), j = gr % (FB / 4) * 4;
      auto one = [&](auto J) {
        constexpr int jj = decltype(J)::value;
        acc[i][j + jj] = mx_mfma<jj, i % 4>(r.f[j + jj], r.s[j / 4], r.f[FB + i], r.s[FB / 4 + i / 4], acc[i][j + jj]);
      };
      static_for<4>(one);
      __builtin_amdgcn_sched_barrier(0);
    });
    copied();
    slot = next;
  };
  for (int i = 0; i < steps; i += 2) {
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
  }
  // every copy has landed and every wave has read its last fragments: the
  // stages are free for the results
  __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0(0));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  // A lane holds four consecutive columns of a row (the MFMAs form C^T):
  // through a wave's own corner of LDS, 16 rows x kRowData bytes at a time, to
  // 16-byte stores of whole row segments.
  constexpr int kSize = kOut == kOutBf16 ? 2 : 4;
  constexpr int kCols = kRowData / kSize, kLanes = kRowData / 16, kE = 16 / kSize;
  using T = std::conditional_t<kOut == kOutBf16, uint16_t, float>;
  char* stage = lds + w * 16 * kRow;
  const int m0 = (ti * WR + wr) * FA * 16, n0 = (tj * WC + wc) * FB * 16;
  const int sr = lane / kLanes, sc = lane % kLanes;
  T* C = static_cast<T*>(g.C) + (g.n_split > 1 ? (int64_t)split * g.M * g.N : 0) +
         (int64_t)(m0 + sr) * g.ldc + n0 + sc * kE;
#pragma unroll
  for (int h = 0; h < FB * 16 / kCols; ++h) {
    f32x4 bias[kCols / 16];
    if constexpr (kBias)
#pragma unroll
      for (int j = 0; j < kCols / 16; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          bias[j][e] = g.bias[min(n0 + h * kCols + 16 * j + 4 * (lane >> 4) + e, g.N - 1)];
#pragma unroll
    for (int i = 0; i < FA; ++i) {
#pragma unroll
      for (int j = 0; j < kCols / 16; ++j) {
        f32x4 v = acc[i][h * (kCols / 16) + j];
        if constexpr (kBias) v += bias[j];
        char* to = stage + (lane & 15) * kRow + (16 * j + 4 * (lane >> 4)) * kSize;
        if constexpr (kOut == kOutBf16)
          *reinterpret_cast<uint2*>(to) = make_uint2(bf16_bits(v[0]) | bf16_bits(v[1]) << 16,
                                                     bf16_bits(v[2]) | bf16_bits(v[3]) << 16);
        else *reinterpret_cast<f32x4*>(to) = v;
      }
      asm volatile("" ::: "memory");
#pragma unroll
      for (int t = 0; t < kLanes / 4; ++t) {
        const int r = t * (64 / kLanes);
        const int m = m0 + 16 * i + r + sr, n = n0 + h * kCols + sc * kE;
        const uint4 q = *reinterpret_cast<const uint4*>(stage + (r + sr) * kRow + sc * 16);
        if (m >= g.M || n >= g.N) continue;
        T* p = C + (int64_t)(16 * i + r) * g.ldc + h * kCols;
        if (n + kE <= g.N) {
          // results around the caches where rows start aligned: 4096^3 36.1 ->
          // 34.5 us, 16384 x 11008 x 4096 448 -> 424 us
          if constexpr (kOut == kOutAcc)
            st16(p, __builtin_bit_cast(uint4, __builtin_bit_cast(f32x4, ld16(p)) + __builtin_bit_cast(f32x4, q)));
          else if constexpr (kNt) st16_nt(p, q);
          else st16(p, q);
        } else {
          T o[kE];
          __builtin_memcpy(o, &q, 16);
#pragma unroll
          for (int e = 0; e < kE; ++e)
            if (n + e < g.N) {
              if constexpr (kOut == kOutAcc) p[e] += o[e];
              else p[e] = o[e];
            }
        }
      }
      asm volatile("" ::: "memory");
    }
  }
}

// C = the splits' partials, added in split order (+ bias, or to C).
__global__ __launch_bounds__(256) void k_mx_reduce(MxGemm g) {
  const int64_t n4 = (g.N + 3) / 4, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n4 * g.M) return;
  const int m = (int)(i / n4), n = (int)(i - m * n4) * 4;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < g.n_split; ++s) {
    const float* p = g.part + ((int64_t)s * g.M + m) * g.N + n;
    if (n + 4 <= g.N) v += __builtin_bit_cast(f32x4, ld16(p));
    else
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < g.N) v[e] += p[e];
  }
  mx_store4(g, m, n, v);
}

// ---------------------------------------------------------------------------
// Small products: a workgroup owns FM x 16 rows of a row panel (blockIdx.y)
// and FN x 16 columns of a column panel of C.  Its 8 waves take the k steps
// in turn, straight from memory into the MFMA operands, with no LDS and no
// barrier in the loop, and their sums are added in wave order through LDS.
// kQuant: A is X itself (at most 16 rows), quantized into LDS first.
// Bound by a launch and chains of loads.  kQuant: one chain, B's loads before
// the rows are quantized (1 x 4096 -> 4096 4.0 us, an empty launch 2.3), or the
// weights' bytes (1 x 4096 -> 11008 24 MB in 6.3 us from memory, 4.8 from the
// caches); the last block of a ragged k is loaded element by element (1 x 4095
// -> 4096 6.1 us).  Else A's loads of a k step wait behind the branch that
// ends the sum, where the compiler puts them, for each step in turn: 11 steps a
// wave of 24 x 11008 -> 4096 take 11 us (9.4 with the weights in the caches),
// 64 rows 4096 -> 4096 7.2, 256 rows 10.3.  With many rows also by the operand
// bytes that every workgroup loads from the second-level caches (512 x 4096 x
// 4096 in 16 columns 20.6 us, 347 MB).
// ---------------------------------------------------------------------------
constexpr int kFewWaves = 8;

struct MxFew {
  MxGemm g;
  const void* X;
  int64_t ldx;
  int64_t k;
  uint32_t* flags;
};

template <int FM, int FN, class T, bool kQuant>
__global__ __launch_bounds__(64 * kFewWaves) void k_mx_few(MxFew q) {
  constexpr int kUnroll = FM + FN <= 5 ? 4 : 2;  // k steps of B (kQuant: of both) in flight per wave
  constexpr int kSub = 4 / FN;                   // workgroups of a column panel
  extern __shared__ __attribute__((aligned(16))) char dyn[];
  __shared__ float sums[kFewWaves][FN][256];
  const MxGemm& g = q.g;
  const int t = threadIdx.x, lane = t & 63;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6);
  // gridDim.x is a multiple of 8: a column panel stays on one XCD, with all
  // its workgroups and row panels; XCDs below `rem` hold one panel more
  const int panels = (g.N + kMxRows - 1) / kMxRows;
  const int id = blockIdx.x, x = id % kXcd, u0 = id / kXcd;
  const int pq = panels / kXcd, rem = panels % kXcd;
  if (u0 / kSub >= pq + (x < rem ? 1 : 0)) return;
  const int panel = x * pq + (x < rem ? x : rem) + u0 / kSub, frag = u0 % kSub * FN;
  if (panel * kMxRows + frag * 16 >= g.N) return;
  const uint8_t* Bp = g.B + (int64_t)panel * g.steps * kMxPanel + frag * 1024;
  i32x4 b[kUnroll][FN];
  int sb[kUnroll];
  auto load_b = [&](int s) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int st = min(s + u * kFewWaves, g.steps - 1);
      const uint8_t* p = Bp + (int64_t)st * kMxPanel;
#pragma unroll
      for (int f = 0; f < FN; ++f) b[u][f] = *reinterpret_cast<const i32x4*>(p + f * 1024 + lane * 16);
      const uint8_t* sc = p - frag * 1024 + 4096 + lane * 4;
      if constexpr (FN == 1) sb[u] = sc[frag];
      else if constexpr (FN == 2) sb[u] = *reinterpret_cast<const uint16_t*>(sc + frag);
      else sb[u] = *reinterpret_cast<const int*>(sc);
    }
  };
  load_b(w);
  if constexpr (kQuant) {
    const T* X = static_cast<const T*>(q.X);
    const int nb = g.steps * 4, M = g.M;
    uint8_t* sc = reinterpret_cast<uint8_t*>(dyn) + (int64_t)nb * M * 16;
    uint32_t fl = 0;
    for (int e = t; e < nb * M; e += 64 * kFewWaves) {
      const int m = e / nb, kb = e - m * nb;
      const int64_t k0 = (int64_t)kb * 32;
      const T* src = X + m * q.ldx + k0;
      float v[32];
      if (k0 + 32 <= q.k) {
        constexpr int kPer = 16 / sizeof(T);
#pragma unroll
        for (int j = 0; j < 32 / kPer; ++j) {
          const uint4 c = ld16(src + j * kPer);
          if constexpr (sizeof(T) == 2) {
            unpack2(c.x, v[8 * j], v[8 * j + 1]);
            unpack2(c.y, v[8 * j + 2], v[8 * j + 3]);
            unpack2(c.z, v[8 * j + 4], v[8 * j + 5]);
            unpack2(c.w, v[8 * j + 6], v[8 * j + 7]);
          } else {
            v[4 * j] = __uint_as_float(c.x);
            v[4 * j + 1] = __uint_as_float(c.y);
            v[4 * j + 2] = __uint_as_float(c.z);
            v[4 * j + 3] = __uint_as_float(c.w);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = k0 + j < q.k ? ld1(src + j) : 0.f;
      }
      uint32_t code, bf = 0;
      const uint4 c = mx_block(v, code, bf);
      if (k0 < q.k) fl |= bf;
      *reinterpret_cast<uint4*>(dyn + ((int64_t)kb * M + m) * 16) = c;
      sc[kb * M + m] = (uint8_t)code;
    }
    if (q.flags && fl && id == 0) atomicOr(q.flags, fl);
    __syncthreads();
  }
  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int s = w; s < g.steps; s += kFewWaves * kUnroll) {
    if (s != w) load_b(s);
    i32x4 a[kUnroll][FM];
    int sa[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int st = min(s + u * kFewWaves, g.steps - 1);
      if constexpr (kQuant) {
        const int r = lane & 15, at = (st * 4 + (lane >> 4)) * g.M + (r < g.M ? r : 0);
        a[u][0] = *reinterpret_cast<const i32x4*>(dyn + at * 16);
        sa[u] = reinterpret_cast<const uint8_t*>(dyn)[(int64_t)g.steps * 4 * g.M * 16 + at];
      } else {
        const uint8_t* p = g.A + ((int64_t)blockIdx.y * g.steps + st) * kMxPanel;
#pragma unroll
        for (int f = 0; f < FM; ++f) a[u][f] = *reinterpret_cast<const i32x4*>(p + f * 1024 + lane * 16);
        sa[u] = *reinterpret_cast<const int*>(p + 4096 + lane * 4);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (s + u * kFewWaves >= g.steps) break;  // wave-uniform
      static_for<FM * FN>([&](auto IJ) {
        constexpr int i = decltype(IJ)::value / FN, j = decltype(IJ)::value % FN;
        acc[i][j] = mx_mfma<j, i>(b[u][j], sb[u], a[u][i], sa[u], acc[i][j]);
      });
    }
  }
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    if (i) __syncthreads();
#pragma unroll
    for (int j = 0; j < FN; ++j) *reinterpret_cast<f32x4*>(&sums[w][j][lane * 4]) = acc[i][j];
    __syncthreads();
    if (t < FN * 64) {
      const int j = t >> 6, l = t & 63;
      f32x4 v = *reinterpret_cast<const f32x4*>(&sums[0][j][l * 4]);
#pragma unroll
      for (int k = 1; k < kFewWaves; ++k) v += *reinterpret_cast<const f32x4*>(&sums[k][j][l * 4]);
      mx_store4(g, blockIdx.y * kMxRows + i * 16 + (l & 15), (panel * 4 + frag + j) * 16 + (l >> 4) * 4, v);
    }
  }
}

hipError_t done() { return hipGetLastError(); }

// every row starts with a 128-byte line: whole lines can go around the caches
// (9000 columns of bf16, 16-byte aligned: dequantize 124 us around, 88 through)
bool rows_aligned(const void* p, int64_t ld, int dtype) {
  return (uintptr_t)p % 128 == 0 && ld * (dtype == GIFT_DTYPE_BF16 ? 2 : 4) % 128 == 0;
}

}  // namespace

hipError_t launch_mx_quantize(const void* X, int dtype, int64_t rows, int64_t cols, int64_t ld,
                              uint8_t* by_row, uint8_t* by_col, uint32_t* flags, hipStream_t s) {
  const int ct = (int)((cols + kMxStep - 1) / kMxStep) * (kMxStep / kQCols);
  // both halves of a step of the operand by columns, the second may lie past the rows
  const int64_t down = by_col ? (rows + kMxStep - 1) / kMxStep * (kMxStep / kQRows) : (rows + kQRows - 1) / kQRows;
  // a dimension of a grid holds fewer than 2^32 threads
  const dim3 grid = down * ct <= 1 << 23 ? dim3((uint32_t)(down * ct)) : dim3((uint32_t)((down * ct + 1) / 2), 2);
  auto go = [&](auto zero) {
    using T = decltype(zero);
    auto run = [&](auto kernel) {
      kernel<<<grid, dim3((by_row && by_col ? 2 : 1) * kQBlocks), 0, s>>>(
          static_cast<const T*>(X), rows, cols, ld, by_row, by_col, ct, flags);
    };
    if (by_row && by_col) run(k_mx_quant<T, true, true>);
    else if (by_row) run(k_mx_quant<T, true, false>);
    else run(k_mx_quant<T, false, true>);
  };
  if (dtype == GIFT_DTYPE_BF16) go((__bf16)0.f);
  else go(0.f);
  return done();
}

hipError_t launch_mx_dequantize(const uint8_t* A, int64_t rows, int64_t k, void* out, int dtype,
                                int64_t ld, hipStream_t s) {
  const int steps = (int)((k + kMxStep - 1) / kMxStep);
  const int64_t blocks = (rows + kMxRows - 1) / kMxRows * steps;
  auto run = [&](auto zero, auto NT) {
    using T = decltype(zero);
    k_mx_dequant<T, decltype(NT)::value><<<dim3((uint32_t)blocks), dim3(256), 0, s>>>(
        A, rows, k, steps, static_cast<T*>(out), ld);
  };
  auto typed = [&](auto zero) {
    if (rows_aligned(out, ld, dtype)) run(zero, std::true_type{});
    else run(zero, std::false_type{});
  };
  if (dtype == GIFT_DTYPE_BF16) typed((__bf16)0.f);
  else typed(0.f);
  return done();
}

// How a product is cut.  The time of every candidate is estimated from its
// sizes, in microseconds, with constants fitted to measurements on products
// of 1 .. 16384 rows, 256 .. 11008 columns and k 256 .. 16384; the estimates
// are within about 20% there.  Measured, the best and the next: 512 x 1024 x
// 1024 4.9 us in 32-column workgroups, 6.7 in 128 x 128 tiles; 1000 x 11008 x
// 4096 26.8 us in 128 x 128, 28.9 in 128 x 256; 16384 x 11008 x 4096 346.8 us
// in 128 x 256, 365.9 in 128 x 128; 256 x 1024 x 11008 11.1 us in 16 columns,
// 13.9 in 128 x 128 split four ways, 22.8 unsplit.
static int64_t up_div(int64_t x, int64_t m) { return (x + m - 1) / m; }

// k_mx_few with 16 fn columns a workgroup: a launch and a fixed latency, then
// the longer of a wave's chain of k steps and the operand bytes that all
// workgroups load, at the rate the second-level caches give.
static double few_us(int64_t M, int64_t N, int64_t steps, int fn) {
  const int i = fn == 1 ? 0 : fn == 2 ? 1 : 2;
  const int fm = M <= 16 ? 1 : M <= 32 ? 2 : 4;
  const double base[2][3] = {{3.6, 3.8, 3.9}, {4.3, 4.4, 4.7}}, chain[3] = {1.65, 2.1, 2.8};
  const double lat = (M <= 32 ? 0.65 : 1.0) * chain[i] * steps / 32, rate = i ? 17e6 : 22e6;
  const double bytes = (double)up_div(M, kMxRows) * up_div(N, 16 * fn) * steps * ((fm + fn) * 1024 + 512);
  // an XCD reads all of A and an eighth of B; past its 4 MB cache loads take
  // longer (x 700 x 16384: 256 rows 12.1 us, 512 rows 22.5)
  const double held = (double)((M + N / kXcd) * steps) * (kMxPanel / kMxRows);
  return base[fm > 2][i] + (lat > bytes / rate ? lat : bytes / rate) / (held > 4.5e6 ? 0.45 : 1.0);
}

static MxPlan plan_us(int64_t M, int64_t N, int64_t k, double& least) {
  const int64_t steps = up_div(k, kMxStep);
  MxPlan best{};
  least = 1e300;
  auto offer = [&](double us, int rows, int cols, int64_t per_split) {
    if (us >= least) return;
    least = us;
    best.rows = rows;
    best.cols = cols;
    best.per_split = (int)per_split;
    best.n_split = (int)up_div(steps, per_split);
  };
  if (up_div(M, kMxRows) <= 0xffff)  // grid.y
    for (int fn = 1; fn <= 4; fn *= 2) offer(few_us(M, N, steps, fn), 64, 16 * fn, steps);
  // k_mx_gemm: a k step's time by the workgroups per CU; split sums write and
  // read fp32 partials
  const int64_t tiles = up_div(M, 128) * up_div(N, 128);
  for (int64_t want = 1; want <= 16 && (want == 1 || want * 4 <= steps); want *= 2) {
    const int64_t per = up_div(steps, want), split = up_div(steps, per);
    const double x = tiles * split / 256.0, step = 0.25 * x > 0.21 ? 0.25 * x : 0.21;
    offer(5 + step * per + (split > 1 ? 2.5 + 0.35 * split + 1.6 * split * M * N * 4 / 4e6 : 0), 128, 128, per);
  }
  const double x = up_div(M, 128) * up_div(N, 256) / 256.0;
  offer(6.5 + (x <= 1 ? 0.42 : x <= 2 ? 0.25 + 0.33 * x : 0.47 * x) * steps, 128, 256, steps);
  return best;
}

MxPlan mx_plan(int64_t M, int64_t N, int64_t k) {
  double us;
  return plan_us(M, N, k, us);
}

size_t mx_matmul_ws(int64_t M, int64_t N, int64_t k) {
  const MxPlan p = mx_plan(M, N, k);
  return p.n_split > 1 ? (size_t)p.n_split * M * N * sizeof(float) : 0;
}

namespace {
MxGemm gemm_args(const uint8_t* A, const uint8_t* B, int64_t M, int64_t N, int64_t k, const float* bias,
                 void* C, int dtype, int64_t ldc, bool accumulate) {
  MxGemm g{};
  g.A = A;
  g.B = B;
  g.C = C;
  g.bias = bias;
  g.ldc = ldc;
  g.M = (int)M;
  g.N = (int)N;
  g.steps = (int)((k + kMxStep - 1) / kMxStep);
  g.mode = dtype == GIFT_DTYPE_BF16 ? kOutBf16 : accumulate ? kOutAcc : kOutF32;
  return g;
}

uint32_t few_blocks(const MxGemm& g, int fn) {
  // every XCD gets the grid of the one with the most panels
  const int panels = (g.N + kMxRows - 1) / kMxRows;
  return (uint32_t)((panels + kXcd - 1) / kXcd * kXcd * (4 / fn));
}
}  // namespace

hipError_t launch_mx_matmul(const uint8_t* A, const uint8_t* B, int64_t M, int64_t N, int64_t k,
                            const float* bias, void* C, int dtype, int64_t ldc, bool accumulate,
                            void* ws, hipStream_t s) {
  const MxPlan p = mx_plan(M, N, k);
  MxGemm g = gemm_args(A, B, M, N, k, bias, C, dtype, ldc, accumulate);
  if (p.rows == 64) {
    MxFew q{};
    q.g = g;
    auto run = [&](auto FM, auto FN) {
      constexpr int fm = decltype(FM)::value, fn = decltype(FN)::value;
      const dim3 grid(few_blocks(g, fn), (uint32_t)((M + kMxRows - 1) / kMxRows)), block(64 * kFewWaves);
      k_mx_few<fm, fn, float, false><<<grid, block, 0, s>>>(q);
    };
    const std::integral_constant<int, 1> i1;
    const std::integral_constant<int, 2> i2;
    const std::integral_constant<int, 4> i4;
    auto rows = [&](auto FN) {
      if (M <= 16) run(i1, FN);
      else if (M <= 32) run(i2, FN);
      else run(i4, FN);
    };
    if (p.cols == 16) rows(i1);
    else if (p.cols == 32) rows(i2);
    else rows(i4);
    return done();
  }
  g.tm = (int)up_div(M, p.rows);
  g.tn = (int)up_div(N, p.cols);
  g.per_split = p.per_split;
  g.n_split = p.n_split;
  MxGemm h = g;
  if (p.n_split > 1) {  // fp32 partials [split][M][N], summed by k_mx_reduce
    g.part = static_cast<float*>(ws);
    h.C = ws;
    h.ldc = N;
    h.mode = kOutF32;
    h.bias = nullptr;
  }
  const dim3 grid((uint32_t)((int64_t)g.tm * g.tn * p.n_split)), block(256);
  auto run = [&](auto OUT, auto BIAS, auto NT) {
    constexpr int kOut = decltype(OUT)::value;
    constexpr bool kBias = decltype(BIAS)::value, kNt = decltype(NT)::value;
    if (p.cols == 256) k_mx_gemm<1, 4, 8, 4, 3, kOut, kBias, kNt><<<grid, block, 0, s>>>(h);
    else k_mx_gemm<2, 2, 4, 4, 3, kOut, kBias, kNt><<<grid, block, 0, s>>>(h);
  };
  auto biased = [&](auto OUT, auto NT) {
    if (h.bias) run(OUT, std::true_type{}, NT);
    else run(OUT, std::false_type{}, NT);
  };
  auto typed = [&](auto OUT) {
    if (rows_aligned(h.C, h.ldc, h.mode == kOutBf16 ? GIFT_DTYPE_BF16 : GIFT_DTYPE_F32)) biased(OUT, std::true_type{});
    else biased(OUT, std::false_type{});
  };
  if (h.mode == kOutAcc) run(std::integral_constant<int, kOutAcc>{}, std::false_type{}, std::false_type{});
  else if (h.mode == kOutBf16) typed(std::integral_constant<int, kOutBf16>{});
  else typed(std::integral_constant<int, kOutF32>{});
  hipError_t e = done();
  if (e != hipSuccess || p.n_split == 1) return e;
  k_mx_reduce<<<dim3((uint32_t)((M * ((N + 3) / 4) + 255) / 256)), dim3(256), 0, s>>>(g);
  return done();
}

// Bytes of LDS that the rows' operand takes in the one-launch form.
static size_t few_lds(int64_t M, int64_t k) {
  return (size_t)((k + kMxStep - 1) / kMxStep * 4 * M * 17);
}

// Columns of a workgroup of the one-launch form, 0: quantize, then multiply.
// In one launch every workgroup quantizes all of X, 0.75 us for each 512
// blocks; a launch of its own takes 2.8 us (16 x 4096 -> 11008: 12.2, 10.0,
// 7.4 us with 16, 32, 64 columns; 16 x 11008 -> 4096: 13.5 us in one launch,
// 10.0 in two; 1 x 4096 -> 4096: 3.6 and 6.3).  The two launches' estimate is at
// most few_us + 2.8 with the same columns, so one launch is taken only where
// 0.75 M steps 4 / 512 < 2.8: M steps < 478, or 32.5 KB of LDS (few_lds).
int mx_linear_cols(int64_t M, int64_t N, int64_t k) {
  if (M > 16) return 0;
  const int64_t steps = up_div(k, kMxStep);
  double least;
  plan_us(M, N, k, least);
  least += 2.8;
  int cols = 0;
  for (int fn = 1; fn <= 4; fn *= 2) {
    const double load = up_div(N, 16 * fn) / 256.0;
    const double us = few_us(M, N, steps, fn) + 0.75 * (M * steps * 4 / 512.0) * (load > 1 ? load : 1);
    if (us < least) {
      least = us;
      cols = 16 * fn;
    }
  }
  return cols;
}

hipError_t launch_mx_linear_few(const void* X, int x_dtype, int64_t M, int64_t ldx, const uint8_t* W,
                                int64_t N, int64_t k, const float* bias, void* Y, int dtype, int64_t ldy,
                                uint32_t* flags, hipStream_t s) {
  MxFew q{};
  q.g = gemm_args(nullptr, W, M, N, k, bias, Y, dtype, ldy, false);
  q.X = X;
  q.ldx = ldx;
  q.k = k;
  q.flags = flags;
  const size_t lds = few_lds(M, k);
  auto run = [&](auto FN) {
    constexpr int fn = decltype(FN)::value;
    const dim3 grid(few_blocks(q.g, fn)), block(64 * kFewWaves);
    if (x_dtype == GIFT_DTYPE_BF16) k_mx_few<1, fn, __bf16, true><<<grid, block, lds, s>>>(q);
    else k_mx_few<1, fn, float, true><<<grid, block, lds, s>>>(q);
  };
  const int cols = mx_linear_cols(M, N, k);
  if (cols == 16) run(std::integral_constant<int, 1>{});
  else if (cols == 32) run(std::integral_constant<int, 2>{});
  else run(std::integral_constant<int, 4>{});
  return done();
}

}  // namespace gift
