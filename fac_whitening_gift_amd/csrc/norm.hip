// Layer norm and RMS norm, forward and backward (gift_norm_* of
// include/gift.h), one pass over the rows.
//
// A row belongs to kL lanes, which keep it in registers (kNV vectors each):
// the mean, the variance around it and the result come from one read.  Rows
// too wide for that (or shorter than a vector) are walked again from memory
// (k_norm_fwd_wide, k_norm_bwd_wide).  All sums are fp32, added in a fixed
// order.
//
// Bound by memory (16384 x 4096, inputs in turn): bf16 forward 49 to 57 us
// (268 MB, 4.7 to 5.5 TB/s), backward 80 us and 5 for the sum of its 512
// partial rows (with them layer norm 436 MB, 5.1 TB/s, RMS norm 419 MB, 4.9);
// fp32 forward 102 us (537 MB, 5.3 TB/s), backward 167 and 160 us and 5 (layer
// norm 839 MB, 4.9 TB/s, RMS norm 822, 5.0).  A copy of 4 GB runs at 4.9 TB/s.
#include <type_traits>

#include "rows.hpp"

namespace gift {

namespace {

struct NormFwd {
  const void* X;
  void* Y;
  const float* weight;
  const float* bias;
  float* mean;
  float* rstd;
  int64_t rows;
  int d;
  float eps;
};

// kTail: d is no multiple of the vector; the row's last vector is loaded to
// end with the row and moved into place.
template <class T, int kNV, int kL, bool kLayer, bool kTail>
__global__ __launch_bounds__(group_threads(kL)) void k_norm_fwd(NormFwd a) {
  constexpr int kVec = kVecOf<T>;
  constexpr int kGroups = group_threads(kL) / kL;
  __shared__ float buf[2][kGroups][waves_of(kL)];
  const int grp = threadIdx.x / kL, l = threadIdx.x % kL;
  const int64_t row = (int64_t)blockIdx.x * kGroups + grp;
  const bool live = row < a.rows;  // a dead group still meets the barriers
  const T* x = static_cast<const T*>(a.X) + row * a.d;
  float v[kNV][kVec];
#pragma unroll
  for (int i = 0; i < kNV; ++i) {
    const int at = (i * kL + l) * kVec;
    if (live && at < a.d) {
      const int from = kTail ? min(at, a.d - kVec) : at;
      unpack<T>(ld16(x + from), v[i]);
      if (kTail && at != from) shift(v[i], at - from, 0.f);
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j) v[i][j] = 0.f;
    }
  }
  float mu = 0.f;
  if constexpr (kLayer) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kNV; ++i)
#pragma unroll
      for (int j = 0; j < kVec; ++j) s += v[i][j];
    mu = group_sum<kL>(s, buf[0][grp]) / (float)a.d;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int at = (i * kL + l) * kVec;
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        if (at + (kTail ? j : 0) < a.d) v[i][j] -= mu;
    }
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < kNV; ++i)
#pragma unroll
    for (int j = 0; j < kVec; ++j) q = __builtin_fmaf(v[i][j], v[i][j], q);
  const float r = 1.0f / sqrtf(group_sum<kL>(q, buf[1][grp]) / (float)a.d + a.eps);
  if (!live) return;
  if (l == 0) {
    if (kLayer && a.mean) a.mean[row] = mu;
    if (a.rstd) a.rstd[row] = r;
  }
  T* y = static_cast<T*>(a.Y) + row * a.d;
#pragma unroll
  for (int i = 0; i < kNV; ++i) {
    const int at = (i * kL + l) * kVec;
    if (at >= a.d) continue;
    float w[kVec], b[kVec];
    ldw<kVec, kTail>(a.weight, at, a.d, 1.f, w);
    ldw<kVec, kTail>(a.bias, at, a.d, 0.f, b);
#pragma unroll
    for (int j = 0; j < kVec; ++j) v[i][j] = __builtin_fmaf(v[i][j] * r, w[j], b[j]);
    stv<T, false, kTail>(y, at, a.d, v[i]);
  }
}

// Threads of the wide kernels, one row per workgroup: rows of many vectors,
// and rows shorter than one, which may be 2^24 (a grid holds fewer than 2^32
// threads).
constexpr int kWide = 1024, kThin = 64;

template <class T, bool kLayer, int kThreads>
__global__ __launch_bounds__(kThreads) void k_norm_fwd_wide(NormFwd a) {
  constexpr int kVec = kVecOf<T>;
  __shared__ float buf[2][kThreads / 64];
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.X) + row * a.d;
  T* y = static_cast<T*>(a.Y) + row * a.d;
  auto each = [&](auto f) {
    for (int at = threadIdx.x * kVec; at < a.d; at += kThreads * kVec) {
      const int n = min(kVec, a.d - at);
      float v[kVec];
      ldn<T>(x + at, n, v);
      f(at, n, v);
    }
  };
  float mu = 0.f;
  if constexpr (kLayer) {
    float s = 0.f;
    each([&](int, int, const float (&v)[kVec]) {
#pragma unroll
      for (int j = 0; j < kVec; ++j) s += v[j];
    });
    mu = group_sum<kThreads>(s, buf[0]) / (float)a.d;
  }
  float q = 0.f;
  each([&](int, int n, const float (&v)[kVec]) {
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const float c = j < n ? v[j] - mu : 0.f;
      q = __builtin_fmaf(c, c, q);
    }
  });
  const float r = 1.0f / sqrtf(group_sum<kThreads>(q, buf[1]) / (float)a.d + a.eps);
  if (threadIdx.x == 0) {
    if (kLayer && a.mean) a.mean[row] = mu;
    if (a.rstd) a.rstd[row] = r;
  }
  each([&](int at, int n, float (&v)[kVec]) {
#pragma unroll
    for (int j = 0; j < kVec; ++j)
      if (j < n)
        v[j] = __builtin_fmaf((v[j] - mu) * r, a.weight ? a.weight[at + j] : 1.f, a.bias ? a.bias[at + j] : 0.f);
    stv<T, false, true>(y, at, a.d, v);
  });
}

struct NormBwd {
  const void* dY;
  const void* X;
  void* dX;
  const float* weight;
  const float* mean;
  const float* rstd;
  float* pw;        // partial weight gradients [parts][d], NULL: not wanted
  float* pb;        // partial bias gradients
  int64_t rows;
  int d;
  int parts;        // workgroups, each a run of rows
  int64_t per;      // rows of a workgroup
};

// A workgroup walks its run of rows; a group's lanes own the same columns in
// every row, so the weight's and the bias's gradients grow in registers and
// leave as one partial row per workgroup.
template <class T, int kNV, int kL, bool kLayer, bool kTail>
__global__ __launch_bounds__(group_threads(kL)) void k_norm_bwd(NormBwd a) {
  constexpr int kVec = kVecOf<T>;
  constexpr int kGroups = group_threads(kL) / kL;
  constexpr int kCols = kL * kVec * kNV;
  constexpr int kW = waves_of(kL);
  __shared__ float buf[2][2][kGroups][kW];
  const int grp = threadIdx.x / kL, l = threadIdx.x % kL;
  float gw[kNV][kVec], gb[kNV][kVec];
#pragma unroll
  for (int i = 0; i < kNV; ++i)
#pragma unroll
    for (int j = 0; j < kVec; ++j) gw[i][j] = gb[i][j] = 0.f;
  const int64_t begin = (int64_t)blockIdx.x * a.per, end = min(a.rows, begin + a.per);
  // Rows are fetched one ahead, from addresses clamped into the run and the
  // row; what lies outside counts as x = mean, dy = 0.
  uint4 nx[kNV], ng[kNV];
  float nr, nmu;
  auto fetch = [&](int64_t row) {
    row = min(row, end - 1);
    const T* x = static_cast<const T*>(a.X) + row * a.d;
    const T* dy = static_cast<const T*>(a.dY) + row * a.d;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int at = min((i * kL + l) * kVec, a.d - kVec);
      nx[i] = ld16(x + at);
      ng[i] = ld16(dy + at);
    }
    nr = a.rstd[row];
    nmu = kLayer ? a.mean[row] : 0.f;
  };
  fetch(begin + grp);
  int phase = 0;
  for (int64_t base = begin; base < end; base += kGroups, phase ^= 1) {
    const int64_t row = base + grp;
    const bool live = row < end;
    const float r = live ? nr : 0.f, mu = live ? nmu : 0.f;
    float h[kNV][kVec], g[kNV][kVec];
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int at = (i * kL + l) * kVec;
      const bool in = live && at < a.d;
      unpack<T>(nx[i], h[i]);
      unpack<T>(ng[i], g[i]);
      if (kTail && in && at > a.d - kVec) {
        shift(h[i], at - (a.d - kVec), mu);
        shift(g[i], at - (a.d - kVec), 0.f);
      }
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        h[i][j] = in ? h[i][j] : mu;
        g[i][j] = in ? g[i][j] : 0.f;
      }
    }
    if (base + kGroups < end) fetch(row + kGroups);
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int at = (i * kL + l) * kVec;
      float w[kVec];
      if (at < a.d) ldw<kVec, kTail>(a.weight, at, a.d, 1.f, w);
      else
#pragma unroll
        for (int j = 0; j < kVec; ++j) w[j] = 0.f;
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        h[i][j] = (h[i][j] - mu) * r;
        gw[i][j] = __builtin_fmaf(g[i][j], h[i][j], gw[i][j]);
        gb[i][j] += g[i][j];
        g[i][j] *= w[j];
        s2 = __builtin_fmaf(g[i][j], h[i][j], s2);
        if constexpr (kLayer) s1 += g[i][j];
      }
    }
    if (!a.dX) continue;
    // both sums in one exchange; the two phases' buffers let the next row
    // start without another barrier
    s2 = lane_sum<kL>(s2);
    if constexpr (kLayer) s1 = lane_sum<kL>(s1);
    if constexpr (kW > 1) {
      const int w = (threadIdx.x >> 6) % kW;
      if ((threadIdx.x & 63) == 0) {
        buf[phase][0][grp][w] = s1;
        buf[phase][1][grp][w] = s2;
      }
      __syncthreads();
      s1 = buf[phase][0][grp][0];
      s2 = buf[phase][1][grp][0];
#pragma unroll
      for (int i = 1; i < kW; ++i) {
        s1 += buf[phase][0][grp][i];
        s2 += buf[phase][1][grp][i];
      }
    }
    s1 /= (float)a.d;
    s2 /= (float)a.d;
    T* dx = static_cast<T*>(a.dX) + row * a.d;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int at = (i * kL + l) * kVec;
      if (!live || at >= a.d) continue;
#pragma unroll
      for (int j = 0; j < kVec; ++j) g[i][j] = r * (__builtin_fmaf(-h[i][j], s2, g[i][j]) - s1);
      stv<T, !kTail, kTail>(dx, at, a.d, g[i]);
    }
  }
  if (!a.pw && !a.pb) return;
  if constexpr (kGroups > 1) {  // the groups' sums, added in group order
    __shared__ float sums[kGroups][kCols];
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      float* p = which ? a.pb : a.pw;
      if (!p) continue;  // uniform
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kNV; ++i)
#pragma unroll
        for (int j = 0; j < kVec; ++j)
          sums[grp][(i * kL + l) * kVec + j] = which ? gb[i][j] : gw[i][j];
      __syncthreads();
      for (int c = threadIdx.x; c < a.d; c += group_threads(kL)) {
        float v = sums[0][c];
#pragma unroll
        for (int k = 1; k < kGroups; ++k) v += sums[k][c];
        p[(int64_t)blockIdx.x * a.d + c] = v;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int at = (i * kL + l) * kVec;
      if (at >= a.d) continue;
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        if (kTail && at + j >= a.d) continue;
        if (a.pw) a.pw[(int64_t)blockIdx.x * a.d + at + j] = gw[i][j];
        if (a.pb) a.pb[(int64_t)blockIdx.x * a.d + at + j] = gb[i][j];
      }
    }
  }
}

// Rows wider than the register form: dX only, a row per workgroup; the
// weight's and bias's gradients come from k_norm_cols.
template <class T, bool kLayer, int kThreads>
__global__ __launch_bounds__(kThreads) void k_norm_bwd_wide(NormBwd a) {
  constexpr int kVec = kVecOf<T>;
  __shared__ float buf[2][kThreads / 64];
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.X) + row * a.d;
  const T* dy = static_cast<const T*>(a.dY) + row * a.d;
  T* dx = static_cast<T*>(a.dX) + row * a.d;
  const float r = a.rstd[row], mu = kLayer ? a.mean[row] : 0.f;
  // g and h of a vector, zeros past the row
  auto each = [&](auto f) {
    for (int at = threadIdx.x * kVec; at < a.d; at += kThreads * kVec) {
      const int n = min(kVec, a.d - at);
      float h[kVec], g[kVec];
      ldn<T>(x + at, n, h);
      ldn<T>(dy + at, n, g);
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        h[j] = j < n ? (h[j] - mu) * r : 0.f;
        if (j < n && a.weight) g[j] *= a.weight[at + j];
      }
      f(at, g, h);
    }
  };
  float s1 = 0.f, s2 = 0.f;
  each([&](int, const float (&g)[kVec], const float (&h)[kVec]) {
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      s2 = __builtin_fmaf(g[j], h[j], s2);
      if constexpr (kLayer) s1 += g[j];
    }
  });
  s2 = group_sum<kThreads>(s2, buf[1]) / (float)a.d;
  if constexpr (kLayer) s1 = group_sum<kThreads>(s1, buf[0]) / (float)a.d;
  each([&](int at, float (&g)[kVec], const float (&h)[kVec]) {
#pragma unroll
    for (int j = 0; j < kVec; ++j) g[j] = r * (__builtin_fmaf(-h[j], s2, g[j]) - s1);
    stv<T, false, true>(dx, at, a.d, g);
  });
}

// Partial gradients of a run of rows, a column per thread.
template <class T, bool kLayer>
__global__ __launch_bounds__(256) void k_norm_cols(NormBwd a) {
  const int c = (int)blockIdx.x * 256 + threadIdx.x;
  if (c >= a.d) return;
  const int64_t begin = (int64_t)blockIdx.y * a.per, end = min(a.rows, begin + a.per);
  float gw = 0.f, gb = 0.f;
  for (int64_t row = begin; row < end; ++row) {
    const float g = (float)static_cast<const T*>(a.dY)[row * a.d + c];
    const float x = (float)static_cast<const T*>(a.X)[row * a.d + c];
    gw = __builtin_fmaf(g, (x - (kLayer ? a.mean[row] : 0.f)) * a.rstd[row], gw);
    gb += g;
  }
  if (a.pw) a.pw[(int64_t)blockIdx.y * a.d + c] = gw;
  if (a.pb) a.pb[(int64_t)blockIdx.y * a.d + c] = gb;
}

// The partial rows summed: 32 columns x 32 threads a column per workgroup,
// thread k of a column adds partials k, k + 32, ..., then the 32 in order.
// blockIdx.y: the weight's gradient, or the bias's.
__global__ __launch_bounds__(1024) void k_norm_sum(const float* pw, const float* pb, float* dw, float* db,
                                                   int parts, int d, bool accumulate) {
  __shared__ float s[32][33];
  const float* p = blockIdx.y ? pb : pw;
  float* o = blockIdx.y ? db : dw;
  if (!o) return;
  const int x = threadIdx.x & 31, k = threadIdx.x >> 5, c = (int)blockIdx.x * 32 + x;
  float v = 0.f;
  if (c < d) {
#pragma unroll 8
    for (int i = k; i < parts; i += 32) v += p[(int64_t)i * d + c];
  }
  s[k][x] = v;
  __syncthreads();
  if (k || c >= d) return;
#pragma unroll
  for (int i = 1; i < 32; ++i) v += s[i][x];
  o[c] = accumulate ? o[c] + v : v;
}

hipError_t done() { return hipGetLastError(); }

constexpr int kMaxCols = 512 * 32;  // widest row of the register form

// Launch the instance for a width: kL lanes a row and the elements of a lane.
// 128 lanes with 32 elements each serve 4096 columns best (16384 rows of bf16,
// forward / backward: 57.0 / 89.8 us; 64 with 64: 60.8; 256 with 16: 59.6 /
// 90.6; 512 with 8: 66.1 / 94.4).  fp32 takes the same lanes with twice the
// vectors: its backward instances of 32 elements need 297 to 324 registers, one
// wave a SIMD, which still keep the copy's rate (8192 columns 330 us, 1.6 GB),
// and above 12288 columns spill up to 332 bytes (8192 x 16384 481 us, 3.4 TB/s;
// bf16 of odd width there 76 to 92 bytes, 8192 x 16383 254 us, 208 for 16384).
template <int kVec, class F>
void by_width(int64_t d, F f) {
  auto go = [&](auto L, auto E) {
    const std::integral_constant<int, decltype(E)::value / kVec> nv;
    if (d % kVec) f(L, nv, std::true_type{});
    else f(L, nv, std::false_type{});
  };
  const std::integral_constant<int, 16> l16, e16;
  const std::integral_constant<int, 32> l32, e32;
  const std::integral_constant<int, 64> l64;
  const std::integral_constant<int, 128> l128;
  const std::integral_constant<int, 256> l256;
  const std::integral_constant<int, 512> l512;
  const std::integral_constant<int, 8> e8;
  const std::integral_constant<int, 24> e24;
  if (d <= 16 * 8) go(l16, e8);
  else if (d <= 32 * 8) go(l32, e8);
  else if (d <= 64 * 8) go(l64, e8);
  else if (d <= 64 * 16) go(l64, e16);
  else if (d <= 128 * 16) go(l128, e16);
  else if (d <= 128 * 32) go(l128, e32);
  else if (d <= 256 * 24) go(l256, e24);
  else if (d <= 256 * 32) go(l256, e32);
  else if (d <= 512 * 24) go(l512, e24);
  else go(l512, e32);
}

// Workgroups of the backward pass, each leaving one partial row of the
// weight's gradient: at least 4 rows each, and about as many as are resident in
// bf16 (of fp32 rows above 2048 columns fewer: there the runs take turns)
// (16384 rows of bf16, 256 / 512 / 1024 of them: 300 columns 28.0 / 19.9 /
// 18.0 us, 4096 columns 104.8 / 82.3 / 91.7, 9000 columns 236 / 251 / 282).
int norm_parts(int64_t rows, int64_t d) {
  const int64_t p = (rows + 3) / 4, most = d <= 512 ? 1024 : d <= 8192 ? 512 : 256;
  return (int)(p < most ? p : most);
}

}  // namespace

hipError_t launch_norm_forward(const void* X, int dtype, int64_t rows, int64_t d, int kind,
                               const float* weight, const float* bias, float eps, void* Y,
                               float* mean, float* rstd, hipStream_t s) {
  NormFwd a{X, Y, weight, bias, mean, rstd, rows, (int)d, eps};
  auto typed = [&](auto zero) {
    using T = decltype(zero);
    if (d > kMaxCols || d < kVecOf<T>) {
      auto run = [&](auto LAYER) {
        constexpr bool kLayer = decltype(LAYER)::value;
        const dim3 grid((uint32_t)rows);
        if (d > kMaxCols) k_norm_fwd_wide<T, kLayer, kWide><<<grid, dim3(kWide), 0, s>>>(a);
        else k_norm_fwd_wide<T, kLayer, kThin><<<grid, dim3(kThin), 0, s>>>(a);
      };
      if (kind == GIFT_NORM_LAYER) run(std::true_type{});
      else run(std::false_type{});
      return;
    }
    by_width<kVecOf<T>>(d, [&](auto L, auto NV, auto TAIL) {
      constexpr int kL = decltype(L)::value, kNV = decltype(NV)::value;
      constexpr bool kTail = decltype(TAIL)::value;
      constexpr int kGroups = group_threads(kL) / kL;
      const dim3 grid((uint32_t)((rows + kGroups - 1) / kGroups)), block(group_threads(kL));
      if (kind == GIFT_NORM_LAYER) k_norm_fwd<T, kNV, kL, true, kTail><<<grid, block, 0, s>>>(a);
      else k_norm_fwd<T, kNV, kL, false, kTail><<<grid, block, 0, s>>>(a);
    });
  };
  if (dtype == GIFT_DTYPE_BF16) typed((__bf16)0.f);
  else typed(0.f);
  return done();
}

size_t norm_backward_ws(int64_t rows, int64_t d) { return (size_t)norm_parts(rows, d) * d * 2 * sizeof(float); }

hipError_t launch_norm_backward(const void* dY, const void* X, int dtype, int64_t rows, int64_t d,
                                int kind, const float* weight, const float* mean, const float* rstd,
                                void* dX, float* dweight, float* dbias, bool accumulate, void* ws,
                                hipStream_t s) {
  NormBwd a{};
  a.dY = dY;
  a.X = X;
  a.dX = dX;
  a.weight = weight;
  a.mean = mean;
  a.rstd = rstd;
  a.rows = rows;
  a.d = (int)d;
  const int most = norm_parts(rows, d);
  a.per = (rows + most - 1) / most;
  a.parts = (int)((rows + a.per - 1) / a.per);
  const bool cols = dweight || dbias;
  if (dweight) a.pw = static_cast<float*>(ws);
  if (dbias) a.pb = static_cast<float*>(ws) + (size_t)most * d;
  auto typed = [&](auto zero) {
    using T = decltype(zero);
    if (d > kMaxCols || d < kVecOf<T>) {
      if (cols) {  // first: dX may overwrite dY
        const dim3 grid((uint32_t)((d + 255) / 256), (uint32_t)a.parts);
        if (kind == GIFT_NORM_LAYER) k_norm_cols<T, true><<<grid, dim3(256), 0, s>>>(a);
        else k_norm_cols<T, false><<<grid, dim3(256), 0, s>>>(a);
      }
      if (dX) {
        auto run = [&](auto LAYER) {
          constexpr bool kLayer = decltype(LAYER)::value;
          const dim3 grid((uint32_t)rows);
          if (d > kMaxCols) k_norm_bwd_wide<T, kLayer, kWide><<<grid, dim3(kWide), 0, s>>>(a);
          else k_norm_bwd_wide<T, kLayer, kThin><<<grid, dim3(kThin), 0, s>>>(a);
        };
        if (kind == GIFT_NORM_LAYER) run(std::true_type{});
        else run(std::false_type{});
      }
      return;
    }
    by_width<kVecOf<T>>(d, [&](auto L, auto NV, auto TAIL) {
      constexpr int kL = decltype(L)::value, kNV = decltype(NV)::value;
      constexpr bool kTail = decltype(TAIL)::value;
      const dim3 grid((uint32_t)a.parts), block(group_threads(kL));
      if (kind == GIFT_NORM_LAYER) k_norm_bwd<T, kNV, kL, true, kTail><<<grid, block, 0, s>>>(a);
      else k_norm_bwd<T, kNV, kL, false, kTail><<<grid, block, 0, s>>>(a);
    });
  };
  if (dtype == GIFT_DTYPE_BF16) typed((__bf16)0.f);
  else typed(0.f);
  hipError_t e = done();
  if (e != hipSuccess || !cols) return e;
  k_norm_sum<<<dim3((uint32_t)((d + 31) / 32), dbias ? 2 : 1), dim3(1024), 0, s>>>(a.pw, a.pb, dweight, dbias,
                                                                              a.parts, (int)d, accumulate);
  return done();
}

}  // namespace gift
