// Layer norm and RMS norm, forward and backward (gift_norm_* of
// include/gift.h), one pass over the rows.
//
// A row belongs to a group of kW waves, which keep it in registers (kNV
// vectors a lane): the mean, the variance around it and the result
// come from one read.  Rows too wide for that are walked again from memory
// (k_norm_fwd_wide, k_norm_bwd_wide).  All sums are fp32, added in a fixed
// order.
//
// Bound by memory: 16384 x 4096 bf16 forward 57 to 59 us (268 MB, 4.6 TB/s),
// backward 82 us and 5 us for the sum of its 1024 partial rows (437 MB, 5.0
// TB/s); a copy of 4 GB runs at 4.9 TB/s.  Eight-element lanes with 8 waves a
// row, and one row at a time without fetching the next, were slower or equal.
#include <type_traits>

#include "device.hpp"
#include "mx.hpp"

namespace gift {

namespace {

template <class T, int kVec>
struct Vec {
  T v[kVec];
};

template <class T, int kVec>
__device__ __forceinline__ void ldv(const T* p, float (&o)[kVec]) {
  if constexpr (kVec * sizeof(T) == 16) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    if constexpr (sizeof(T) == 2) {
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[2 * i] = __uint_as_float(w[i] << 16);
        o[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    } else {
      o[0] = __uint_as_float(q.x);
      o[1] = __uint_as_float(q.y);
      o[2] = __uint_as_float(q.z);
      o[3] = __uint_as_float(q.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i) o[i] = (float)p[i];
  }
}

// kNt: around the caches.  The backward pass gains by it (16384 x 4096 bf16:
// 89.8 -> 86.7 us), the forward pass loses (57.0 -> 59.7 us).
template <class T, int kVec, bool kNt>
__device__ __forceinline__ void stv(T* p, const float (&v)[kVec]) {
  Vec<T, kVec> o;
#pragma unroll
  for (int i = 0; i < kVec; ++i) o.v[i] = (T)v[i];
  if constexpr (kVec * sizeof(T) == 16) {
    if constexpr (kNt) __builtin_nontemporal_store(__builtin_bit_cast(nt_u4, o), reinterpret_cast<nt_u4*>(p));
    else *reinterpret_cast<uint4*>(p) = __builtin_bit_cast(uint4, o);
  } else
#pragma unroll
    for (int i = 0; i < kVec; ++i) p[i] = o.v[i];
}

template <class T, int kVec>
__device__ __forceinline__ Vec<T, kVec> ldraw(const T* p) {
  if constexpr (kVec * sizeof(T) == 16)
    return __builtin_bit_cast(Vec<T, kVec>, *reinterpret_cast<const uint4*>(p));
  Vec<T, kVec> o;
#pragma unroll
  for (int i = 0; i < kVec; ++i) o.v[i] = p[i];
  return o;
}

// kVec floats of a d-vector that may be NULL (then `none`)
template <int kVec>
__device__ __forceinline__ void ldw(const float* p, int at, float none, float (&o)[kVec]) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) o[i] = none;
    return;
  }
  if constexpr (kVec % 4 == 0) {
#pragma unroll
    for (int i = 0; i < kVec / 4; ++i) {
      const float4 q = *reinterpret_cast<const float4*>(p + at + 4 * i);
      o[4 * i] = q.x;
      o[4 * i + 1] = q.y;
      o[4 * i + 2] = q.z;
      o[4 * i + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i) o[i] = p[at + i];
  }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Sum of v over the kW waves of a row's group; buf: kW floats of the group.
template <int kW>
__device__ __forceinline__ float group_sum(float v, float* buf) {
  v = wave_sum(v);
  if constexpr (kW > 1) {
    const int w = (threadIdx.x >> 6) % kW;
    if ((threadIdx.x & 63) == 0) buf[w] = v;
    __syncthreads();
    v = buf[0];
#pragma unroll
    for (int i = 1; i < kW; ++i) v += buf[i];
  }
  return v;
}

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

constexpr int group_threads(int kW) { return kW < 4 ? 256 : 64 * kW; }

template <class T, int kVec, int kNV, int kW, bool kLayer>
__global__ __launch_bounds__(group_threads(kW)) void k_norm_fwd(NormFwd a) {
  constexpr int kGroups = group_threads(kW) / (64 * kW);
  __shared__ float buf[2][kGroups][kW];
  const int grp = threadIdx.x / (64 * kW), l = threadIdx.x % (64 * kW);
  const int64_t row = (int64_t)blockIdx.x * kGroups + grp;
  const bool live = row < a.rows;  // a dead group still meets the barriers
  const T* x = static_cast<const T*>(a.X) + row * a.d;
  float v[kNV][kVec];
#pragma unroll
  for (int i = 0; i < kNV; ++i) {
    const int at = (i * 64 * kW + l) * kVec;
    if (live && at < a.d) ldv<T, kVec>(x + at, v[i]);
    else
#pragma unroll
      for (int j = 0; j < kVec; ++j) v[i][j] = 0.f;
  }
  float mu = 0.f;
  if constexpr (kLayer) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kNV; ++i)
#pragma unroll
      for (int j = 0; j < kVec; ++j) s += v[i][j];
    mu = group_sum<kW>(s, buf[0][grp]) / (float)a.d;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      if ((i * 64 * kW + l) * kVec < a.d)
#pragma unroll
        for (int j = 0; j < kVec; ++j) v[i][j] -= mu;
    }
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < kNV; ++i)
#pragma unroll
    for (int j = 0; j < kVec; ++j) q = __builtin_fmaf(v[i][j], v[i][j], q);
  const float r = 1.0f / sqrtf(group_sum<kW>(q, buf[1][grp]) / (float)a.d + a.eps);
  if (!live) return;
  if (l == 0) {
    if (kLayer && a.mean) a.mean[row] = mu;
    if (a.rstd) a.rstd[row] = r;
  }
  T* y = static_cast<T*>(a.Y) + row * a.d;
#pragma unroll
  for (int i = 0; i < kNV; ++i) {
    const int at = (i * 64 * kW + l) * kVec;
    if (at >= a.d) continue;
    float w[kVec], b[kVec];
    ldw<kVec>(a.weight, at, 1.f, w);
    ldw<kVec>(a.bias, at, 0.f, b);
#pragma unroll
    for (int j = 0; j < kVec; ++j) v[i][j] = __builtin_fmaf(v[i][j] * r, w[j], b[j]);
    stv<T, kVec, false>(y + at, v[i]);
  }
}

constexpr int kWide = 1024;  // threads of the wide kernels, one row per workgroup

template <class T, bool kLayer>
__global__ __launch_bounds__(kWide) void k_norm_fwd_wide(NormFwd a) {
  __shared__ float buf[2][kWide / 64];
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.X) + row * a.d;
  T* y = static_cast<T*>(a.Y) + row * a.d;
  float mu = 0.f;
  if constexpr (kLayer) {
    float s = 0.f;
    for (int i = threadIdx.x; i < a.d; i += kWide) s += (float)x[i];
    mu = group_sum<kWide / 64>(s, buf[0]) / (float)a.d;
  }
  float q = 0.f;
  for (int i = threadIdx.x; i < a.d; i += kWide) {
    const float c = (float)x[i] - mu;
    q = __builtin_fmaf(c, c, q);
  }
  const float r = 1.0f / sqrtf(group_sum<kWide / 64>(q, buf[1]) / (float)a.d + a.eps);
  if (threadIdx.x == 0) {
    if (kLayer && a.mean) a.mean[row] = mu;
    if (a.rstd) a.rstd[row] = r;
  }
  for (int i = threadIdx.x; i < a.d; i += kWide)
    y[i] = (T)__builtin_fmaf(((float)x[i] - mu) * r, a.weight ? a.weight[i] : 1.f,
                             a.bias ? a.bias[i] : 0.f);
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
template <class T, int kVec, int kNV, int kW, bool kLayer>
__global__ __launch_bounds__(group_threads(kW)) void k_norm_bwd(NormBwd a) {
  constexpr int kGroups = group_threads(kW) / (64 * kW);
  constexpr int kCols = 64 * kW * kVec * kNV;
  __shared__ float buf[2][2][kGroups][kW];
  const int grp = threadIdx.x / (64 * kW), l = threadIdx.x % (64 * kW);
  float gw[kNV][kVec], gb[kNV][kVec];
#pragma unroll
  for (int i = 0; i < kNV; ++i)
#pragma unroll
    for (int j = 0; j < kVec; ++j) gw[i][j] = gb[i][j] = 0.f;
  const int64_t begin = (int64_t)blockIdx.x * a.per, end = min(a.rows, begin + a.per);
  // Rows are fetched one ahead (not by 16 waves, whose registers that would
  // overflow), from addresses clamped into the run and the
  // row; what lies outside counts as x = mean, dy = 0.
  Vec<T, kVec> nx[kNV], ng[kNV];
  float nr, nmu;
  auto fetch = [&](int64_t row) {
    row = min(row, end - 1);
    const T* x = static_cast<const T*>(a.X) + row * a.d;
    const T* dy = static_cast<const T*>(a.dY) + row * a.d;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int at = min((i * 64 * kW + l) * kVec, a.d - kVec);
      nx[i] = ldraw<T, kVec>(x + at);
      ng[i] = ldraw<T, kVec>(dy + at);
    }
    nr = a.rstd[row];
    nmu = kLayer ? a.mean[row] : 0.f;
  };
  constexpr bool kAhead = kW < 16;
  if (kAhead) fetch(begin + grp);
  int phase = 0;
  for (int64_t base = begin; base < end; base += kGroups, phase ^= 1) {
    const int64_t row = base + grp;
    const bool live = row < end;
    if (!kAhead) fetch(row);
    const float r = live ? nr : 0.f, mu = live ? nmu : 0.f;
    float h[kNV][kVec], g[kNV][kVec];
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const bool in = live && (i * 64 * kW + l) * kVec < a.d;
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        h[i][j] = in ? (float)nx[i].v[j] : mu;
        g[i][j] = in ? (float)ng[i].v[j] : 0.f;
      }
    }
    if (kAhead && base + kGroups < end) fetch(row + kGroups);
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int at = (i * 64 * kW + l) * kVec;
      float w[kVec];
      if (at < a.d) ldw<kVec>(a.weight, at, 1.f, w);
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
    s2 = wave_sum(s2);
    if constexpr (kLayer) s1 = wave_sum(s1);
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
      const int at = (i * 64 * kW + l) * kVec;
      if (!live || at >= a.d) continue;
#pragma unroll
      for (int j = 0; j < kVec; ++j) g[i][j] = r * (__builtin_fmaf(-h[i][j], s2, g[i][j]) - s1);
      stv<T, kVec, true>(dx + at, g[i]);
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
          sums[grp][(i * 64 * kW + l) * kVec + j] = which ? gb[i][j] : gw[i][j];
      __syncthreads();
      for (int c = threadIdx.x; c < a.d; c += group_threads(kW)) {
        float v = sums[0][c];
#pragma unroll
        for (int k = 1; k < kGroups; ++k) v += sums[k][c];
        p[(int64_t)blockIdx.x * a.d + c] = v;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int at = (i * 64 * kW + l) * kVec;
      if (at >= a.d) continue;
      if (a.pw)
#pragma unroll
        for (int j = 0; j < kVec; ++j) a.pw[(int64_t)blockIdx.x * a.d + at + j] = gw[i][j];
      if (a.pb)
#pragma unroll
        for (int j = 0; j < kVec; ++j) a.pb[(int64_t)blockIdx.x * a.d + at + j] = gb[i][j];
    }
  }
}

// Rows wider than the register form: dX only, a row per workgroup; the
// weight's and bias's gradients come from k_norm_cols.
template <class T, bool kLayer>
__global__ __launch_bounds__(kWide) void k_norm_bwd_wide(NormBwd a) {
  __shared__ float buf[2][kWide / 64];
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.X) + row * a.d;
  const T* dy = static_cast<const T*>(a.dY) + row * a.d;
  T* dx = static_cast<T*>(a.dX) + row * a.d;
  const float r = a.rstd[row], mu = kLayer ? a.mean[row] : 0.f;
  float s1 = 0.f, s2 = 0.f;
  for (int i = threadIdx.x; i < a.d; i += kWide) {
    const float g = (float)dy[i] * (a.weight ? a.weight[i] : 1.f);
    s2 = __builtin_fmaf(g, ((float)x[i] - mu) * r, s2);
    if constexpr (kLayer) s1 += g;
  }
  s2 = group_sum<kWide / 64>(s2, buf[1]) / (float)a.d;
  if constexpr (kLayer) s1 = group_sum<kWide / 64>(s1, buf[0]) / (float)a.d;
  for (int i = threadIdx.x; i < a.d; i += kWide) {
    const float g = (float)dy[i] * (a.weight ? a.weight[i] : 1.f);
    dx[i] = (T)(r * (__builtin_fmaf(-((float)x[i] - mu) * r, s2, g) - s1));
  }
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

// Widest row of the register form (single elements take more registers, for
// their addresses, than 16 waves have for 16 of them).
constexpr int max_cols(int kVec) { return 64 * 16 * (kVec > 1 ? 16 : 8); }

// Launch the instance for a width: kW waves a row and the elements of a lane.
// Two waves with 32 elements each serve 4096 columns best (16384 rows of bf16,
// forward / backward: 57.0 / 89.8 us; one wave with 64: 60.8; four with 16:
// 59.6 / 90.6; eight with 8: 66.1 / 94.4).
template <int kVec, class F>
void by_width(int64_t d, F f) {
  auto go = [&](auto W, auto E) { f(W, std::integral_constant<int, decltype(E)::value / kVec>{}); };
  const std::integral_constant<int, 1> w1;
  const std::integral_constant<int, 2> w2;
  const std::integral_constant<int, 8> w8, e8;
  const std::integral_constant<int, 16> w16, e16;
  const std::integral_constant<int, 32> e32;
  if (d <= 512) go(w1, e8);
  else if (d <= 1024) go(w1, e16);
  else if (d <= 2048) go(w2, e16);
  else if (d <= 4096) go(w2, e32);
  else if (d <= 8192) go(w8, e16);
  else go(w16, std::integral_constant<int, max_cols(kVec) / 1024>{});
}

constexpr int kNormParts = 1024;  // most partial rows of the weight's gradient

int norm_parts(int64_t rows) {
  // at least 4 rows a workgroup
  const int64_t p = (rows + 3) / 4;
  return (int)(p < kNormParts ? p : kNormParts);
}

}  // namespace

hipError_t launch_norm_forward(const void* X, int dtype, int64_t rows, int64_t d, int kind,
                               const float* weight, const float* bias, float eps, void* Y,
                               float* mean, float* rstd, hipStream_t s) {
  NormFwd a{X, Y, weight, bias, mean, rstd, rows, (int)d, eps};
  auto typed = [&](auto zero) {
    using T = decltype(zero);
    constexpr int kFull = 16 / sizeof(T);
    const bool vec = d % kFull == 0 && (((uintptr_t)X | (uintptr_t)Y | (uintptr_t)weight | (uintptr_t)bias) & 15) == 0;
    auto run = [&](auto VEC) {
      constexpr int kVec = decltype(VEC)::value;
      if (d > max_cols(kVec)) {
        if (kind == GIFT_NORM_LAYER) k_norm_fwd_wide<T, true><<<dim3((uint32_t)rows), dim3(kWide), 0, s>>>(a);
        else k_norm_fwd_wide<T, false><<<dim3((uint32_t)rows), dim3(kWide), 0, s>>>(a);
        return;
      }
      by_width<kVec>(d, [&](auto W, auto NV) {
        constexpr int kW = decltype(W)::value, kNV = decltype(NV)::value;
        constexpr int kGroups = group_threads(kW) / (64 * kW);
        const dim3 grid((uint32_t)((rows + kGroups - 1) / kGroups)), block(group_threads(kW));
        if (kind == GIFT_NORM_LAYER) k_norm_fwd<T, kVec, kNV, kW, true><<<grid, block, 0, s>>>(a);
        else k_norm_fwd<T, kVec, kNV, kW, false><<<grid, block, 0, s>>>(a);
      });
    };
    if (vec) run(std::integral_constant<int, kFull>{});
    else run(std::integral_constant<int, 1>{});
  };
  if (dtype == GIFT_DTYPE_BF16) typed((__bf16)0.f);
  else typed(0.f);
  return done();
}

size_t norm_backward_ws(int64_t rows, int64_t d) { return (size_t)norm_parts(rows) * d * 2 * sizeof(float); }

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
  const int most = norm_parts(rows);
  a.per = (rows + most - 1) / most;
  a.parts = (int)((rows + a.per - 1) / a.per);
  const bool cols = dweight || dbias;
  if (dweight) a.pw = static_cast<float*>(ws);
  if (dbias) a.pb = static_cast<float*>(ws) + (size_t)most * d;
  auto typed = [&](auto zero) {
    using T = decltype(zero);
    constexpr int kFull = 16 / sizeof(T);
    const bool vec = d % kFull == 0 && (((uintptr_t)X | (uintptr_t)dY | (uintptr_t)dX | (uintptr_t)weight) & 15) == 0;
    auto run = [&](auto VEC) {
      constexpr int kVec = decltype(VEC)::value;
      if (d > max_cols(kVec)) {
        if (cols) {  // first: dX may overwrite dY
          const dim3 grid((uint32_t)((d + 255) / 256), (uint32_t)a.parts);
          if (kind == GIFT_NORM_LAYER) k_norm_cols<T, true><<<grid, dim3(256), 0, s>>>(a);
          else k_norm_cols<T, false><<<grid, dim3(256), 0, s>>>(a);
        }
        if (dX) {
          if (kind == GIFT_NORM_LAYER) k_norm_bwd_wide<T, true><<<dim3((uint32_t)rows), dim3(kWide), 0, s>>>(a);
          else k_norm_bwd_wide<T, false><<<dim3((uint32_t)rows), dim3(kWide), 0, s>>>(a);
        }
        return;
      }
      by_width<kVec>(d, [&](auto W, auto NV) {
        constexpr int kW = decltype(W)::value, kNV = decltype(NV)::value;
        const dim3 grid((uint32_t)a.parts), block(group_threads(kW));
        if (kind == GIFT_NORM_LAYER) k_norm_bwd<T, kVec, kNV, kW, true><<<grid, block, 0, s>>>(a);
        else k_norm_bwd<T, kVec, kNV, kW, false><<<grid, block, 0, s>>>(a);
      });
    };
    if (vec) run(std::integral_constant<int, kFull>{});
    else run(std::integral_constant<int, 1>{});
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
