// The norm after a block, its gate and the residual scale, and the norm in front
// of the next block in one pass over the rows (gift_block_norm_* of
// include/gift.h):
//   n = norm(y), h' = scale h + gate n, x = norm(h')
// and backwards, with t the whole gradient of h',
//   t = dh' + dnorm(dx; h'), dh = scale t, dy = dnorm(gate t; y).
//
// A row belongs to kL lanes, which keep their columns of it in registers, so
// every tensor is read once and every result written once.  Four of the vector
// gradients are sums over rows of products with t: with A = sum t yhat and B =
// sum t over the rows that share a gate,
//   dgate = post_weight A + post_bias B,
//   dpost_weight = sum over gates of gate A, dpost_bias = sum of gate B,
// so A and B are all that a row adds to.  All sums are fp32, in a fixed order.
#include <type_traits>

#include "host.hpp"
#include "rows.hpp"
#include "step.hpp"

namespace gift {

namespace {

// 8 elements of T as they lie in memory
template <class T>
struct Raw {
  uint4 q[8 * sizeof(T) / 16];
};

// A lane's 8 columns at `at` of a row of d: the row's last vector is loaded to
// end with the row and moved into place (unpack8); columns past the row read its
// last ones.
template <class T, bool kTail>
__device__ __forceinline__ Raw<T> fetch8(const T* row, int at, int d) {
  Raw<T> r;
  if (kTail && d < 8) {
    T e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = row[min(j, d - 1)];
    __builtin_memcpy(&r, e, sizeof(r));
    return r;
  }
  const T* p = row + min(at, d - 8);
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.q[i] = ld16(p + i * kVecOf<T>);
  return r;
}

template <class T>
__device__ __forceinline__ void widen8(const Raw<T>& r, float (&o)[8]) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
    float v[kVecOf<T>];
    unpack<T>(r.q[i], v);
#pragma unroll
    for (int j = 0; j < kVecOf<T>; ++j) o[i * kVecOf<T> + j] = v[j];
  }
}

// -> the lane's values, `fill` past the row
template <class T, bool kTail>
__device__ __forceinline__ void unpack8(const Raw<T>& r, int at, int d, bool live, float fill, float (&o)[8]) {
  widen8(r, o);
  const bool in = live && at < d;
  if (kTail && in && at + 8 > d) {
    if (d >= 8) shift(o, at + 8 - d, fill);
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = at + j < d ? o[j] : fill;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = in ? o[j] : fill;
}

// the lane's values of a d-vector that may be NULL (then `none`), zeros past it
template <bool kTail>
__device__ __forceinline__ void vector8(const float* p, int at, int d, float none, float (&o)[8]) {
  if (p) {
    unpack8<float, kTail>(fetch8<float, kTail>(p, at, d), at, d, true, 0.f, o);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = at + j < d ? none : 0.f;
  }
}

template <class T, bool kTail>
__device__ __forceinline__ void store8(T* row, int at, int d, const float (&v)[8]) {
  if (at >= d) return;
  if (kTail && at + 8 > d) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (at + j < d) row[at + j] = (T)v[j];
    return;
  }
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
    float o[kVecOf<T>];
#pragma unroll
    for (int j = 0; j < kVecOf<T>; ++j) o[j] = v[i * kVecOf<T> + j];
    st16(row + at + i * kVecOf<T>, pack<T>(o));
  }
}

struct BlockFwd {
  gift_block_norm p;
  const void* Y;
  const void* H;
  void* H2;
  void* X;
  float* stats;   // [4][rows]
};

// mean and 1 / sqrt(mean square + eps) of a row held by its lanes, zeros past it;
// v becomes v - mean
template <int kL, int kNV, bool kTail>
__device__ __forceinline__ void row_stats(float (&v)[kNV][8], int l, int d, bool layer, float eps, float (*buf)[waves_of(kL)],
                                          float& mean, float& rstd) {
  mean = 0.f;
  if (layer) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kNV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) s += v[i][j];
    mean = group_sum<kL>(s, buf[0]) / (float)d;
#pragma unroll
    for (int i = 0; i < kNV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if ((i * kL + l) * 8 + (kTail ? j : 0) < d) v[i][j] -= mean;
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < kNV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) q = __builtin_fmaf(v[i][j], v[i][j], q);
  rstd = 1.0f / sqrtf(group_sum<kL>(q, buf[1]) / (float)d + eps);
}

template <class TY, class TH, int kL, int kNV, bool kTail>
__global__ __launch_bounds__(group_threads(kL)) void k_block_fwd(BlockFwd a) {
  constexpr int kGroups = group_threads(kL) / kL;
  __shared__ float buf[kGroups][4][waves_of(kL)];
  const int grp = threadIdx.x / kL, l = threadIdx.x % kL, d = (int)a.p.d;
  const int64_t row = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kGroups + grp, rows = a.p.rows;
  const bool live = row < rows;  // a dead group still meets the barriers
  const int64_t at_row = (live ? row : rows - 1) * d;
  const bool layer = a.p.kind == GIFT_NORM_LAYER;
  Raw<TY> ry[kNV];
  Raw<TH> rh[kNV];
#pragma unroll
  for (int i = 0; i < kNV; ++i) {
    ry[i] = fetch8<TY, kTail>(static_cast<const TY*>(a.Y) + at_row, (i * kL + l) * 8, d);
    rh[i] = fetch8<TH, kTail>(static_cast<const TH*>(a.H) + at_row, (i * kL + l) * 8, d);
  }
  float y[kNV][8], h[kNV][8];
#pragma unroll
  for (int i = 0; i < kNV; ++i) unpack8<TY, kTail>(ry[i], (i * kL + l) * 8, d, true, 0.f, y[i]);
  float pm = 0.f, pr = 1.f, m, r;
  if (a.p.post) row_stats<kL, kNV, kTail>(y, l, d, layer, a.p.eps, buf[grp], pm, pr);
  const float* gate = a.p.gate ? a.p.gate + (live ? row : rows - 1) / a.p.gate_rows * d : nullptr;
#pragma unroll
  for (int i = 0; i < kNV; ++i) {
    const int at = (i * kL + l) * 8;
    unpack8<TH, kTail>(rh[i], at, d, true, 0.f, h[i]);
    float w[8], b[8], g[8];
    vector8<kTail>(a.p.post_weight, at, d, 1.f, w);
    vector8<kTail>(a.p.post_bias, at, d, 0.f, b);
    vector8<kTail>(gate, at, d, 1.f, g);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float n = a.p.post ? __builtin_fmaf(y[i][j] * pr, w[j], b[j]) : y[i][j];
      y[i][j] = h[i][j] = __builtin_fmaf(g[j], n, a.p.scale * h[i][j]);
    }
  }
  row_stats<kL, kNV, kTail>(y, l, d, layer, a.p.eps, buf[grp] + 2, m, r);
  if (!live) return;
  if (l == 0) {
    a.stats[row] = pm;
    a.stats[rows + row] = pr;
    a.stats[2 * rows + row] = m;
    a.stats[3 * rows + row] = r;
  }
  // stored behind the sums' barriers: a row's last vector may have been read
  // from columns that another lane writes
  TH* h2 = static_cast<TH*>(a.H2) + at_row;
  TY* x = static_cast<TY*>(a.X) + at_row;
#pragma unroll
  for (int i = 0; i < kNV; ++i) {
    const int at = (i * kL + l) * 8;
    store8<TH, kTail>(h2, at, d, h[i]);
    float w[8], b[8];
    vector8<kTail>(a.p.weight, at, d, 1.f, w);
    vector8<kTail>(a.p.bias, at, d, 0.f, b);
#pragma unroll
    for (int j = 0; j < 8; ++j) y[i][j] = __builtin_fmaf(y[i][j] * r, w[j], b[j]);
    store8<TY, kTail>(x, at, d, y[i]);
  }
}

struct BlockBwd {
  gift_block_norm p;
  const void* dX;
  const void* dH2;
  const void* Y;
  const void* H2;
  const float* stats;
  void* dY;
  void* dH;
  float* sw;      // [runs][d]: sums of dx xhat, NULL: not wanted
  float* sb;      // [runs][d]: of dx
  float* sa;      // [runs + gates - 1][d]: of t yhat, a run's rows of one gate each
  float* st;      // of t
  int* gate_of;   // [runs + gates - 1]
  int64_t run;    // rows of a run
  int runs;
};

// A workgroup walks its run of rows, gate by gate; a group's lanes own the same
// columns in every row, so the sums grow in registers.  Those for the weight and
// the bias leave once a run, A and B once a gate: the rows of run r that gate g
// serves leave them in row r + g, which moves by one where a run or a gate ends;
// where both end at once a row between them holds zeros.
template <class TY, class TH, int kL, int kNV, bool kTail, bool kBias>
__global__ __launch_bounds__(group_threads(kL)) void k_block_bwd(BlockBwd a) {
  constexpr int kGroups = group_threads(kL) / kL, kW = waves_of(kL);
  constexpr int kCols = kL * kNV * 8;
  __shared__ float buf[2][2][2][kGroups][kW];
  __shared__ float sums[kGroups > 1 ? kGroups : 1][kGroups > 1 ? kCols : 1];
  const int grp = threadIdx.x / kL, l = threadIdx.x % kL, d = (int)a.p.d;
  const int64_t rows = a.p.rows, begin = (int64_t)blockIdx.x * a.run, end = min(rows, begin + a.run);
  const bool layer = a.p.kind == GIFT_NORM_LAYER, post = a.p.post;
  const float inv_d = 1.0f / (float)d;
  float gw[kNV][8], gb[kNV][8], ga[kNV][8], gt[kNV][8];
  auto clear = [&](float (&v)[kNV][8]) {
#pragma unroll
    for (int i = 0; i < kNV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
  };
  // the groups' sums, added in group order, to a row of `out`
  auto leave = [&](float* out, int64_t at_row, const float (&v)[kNV][8]) {
    float* o = out + at_row * d;
    if constexpr (kGroups > 1) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kNV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) sums[grp][(i * kL + l) * 8 + j] = v[i][j];
      __syncthreads();
      for (int c = threadIdx.x; c < d; c += group_threads(kL)) {
        float s = sums[0][c];
#pragma unroll
        for (int k = 1; k < kGroups; ++k) s += sums[k][c];
        o[c] = s;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kNV; ++i) store8<float, kTail>(o, (i * kL + l) * 8, d, v[i]);
    }
  };
  clear(gw);
  clear(gb);
  // rows are fetched one ahead, from addresses clamped into the run
  Raw<TY> nx[kNV], ny[kNV];
  Raw<TH> ng[kNV], nh[kNV];
  float npm, npr, nm, nr;
  auto fetch = [&](int64_t row) {
    row = min(row, end - 1);
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int at = (i * kL + l) * 8;
      nx[i] = fetch8<TY, kTail>(static_cast<const TY*>(a.dX) + row * d, at, d);
      nh[i] = fetch8<TH, kTail>(static_cast<const TH*>(a.H2) + row * d, at, d);
      ny[i] = fetch8<TY, kTail>(static_cast<const TY*>(a.Y) + row * d, at, d);
      if (a.dH2) ng[i] = fetch8<TH, kTail>(static_cast<const TH*>(a.dH2) + row * d, at, d);
    }
    npm = a.stats[row];
    npr = a.stats[rows + row];
    nm = a.stats[2 * rows + row];
    nr = a.stats[3 * rows + row];
  };
  // sums over a row's lanes of two values
  auto both = [&](float& s1, float& s2, float (&b)[2][kGroups][kW]) {
    s1 = layer ? lane_sum<kL>(s1) : 0.f;
    s2 = lane_sum<kL>(s2);
    if constexpr (kW > 1) {
      const int w = (threadIdx.x >> 6) % kW;
      if ((threadIdx.x & 63) == 0) {
        b[0][grp][w] = s1;
        b[1][grp][w] = s2;
      }
      __syncthreads();
      s1 = b[0][grp][0];
      s2 = b[1][grp][0];
#pragma unroll
      for (int i = 1; i < kW; ++i) {
        s1 += b[0][grp][i];
        s2 += b[1][grp][i];
      }
    }
    s1 *= inv_d;
    s2 *= inv_d;
  };
  fetch(begin + grp);
  int phase = 0;
  for (int64_t from = begin; from < end;) {
    const int64_t g = from / a.p.gate_rows, to = min(end, (g + 1) * a.p.gate_rows);
    const float* gate = a.p.gate ? a.p.gate + g * d : nullptr;
    clear(ga);
    clear(gt);
    for (int64_t base = from; base < to; base += kGroups, phase ^= 1) {
      const int64_t row = base + grp;
      const bool live = row < to;
      // a dead row adds nothing, whatever the row that was fetched for it holds
      const float m = live ? nm : 0.f, r = live ? nr : 0.f;
      const float pm = live && post ? npm : 0.f, pr = live && post ? npr : 0.f;
      float dx[kNV][8], u[kNV][8], t[kNV][8], v[kNV][8];
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        const int at = (i * kL + l) * 8;
        unpack8<TY, kTail>(nx[i], at, d, live, 0.f, dx[i]);
        unpack8<TH, kTail>(nh[i], at, d, live, m, u[i]);
        unpack8<TY, kTail>(ny[i], at, d, live, pm, v[i]);
        if (a.dH2) {
          unpack8<TH, kTail>(ng[i], at, d, live, 0.f, t[i]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) t[i][j] = 0.f;
        }
      }
      // the next row of the group: in this gate's rows, or the first of the next
      const int64_t next = base + kGroups < to ? row + kGroups : to + grp;
      if (base + kGroups < to || to < end) fetch(next);
      float s1 = 0.f, s2 = 0.f;
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        float w[8];
        vector8<kTail>(a.p.weight, (i * kL + l) * 8, d, 1.f, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          u[i][j] = (u[i][j] - m) * r;
          gw[i][j] = __builtin_fmaf(dx[i][j], u[i][j], gw[i][j]);
          if constexpr (kBias) gb[i][j] += dx[i][j];
          dx[i][j] *= w[j];
          s2 = __builtin_fmaf(dx[i][j], u[i][j], s2);
          s1 += dx[i][j];
        }
      }
      both(s1, s2, buf[0][phase]);
      float s3 = 0.f, s4 = 0.f;
      TH* dh = static_cast<TH*>(a.dH) + row * d;
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        const int at = (i * kL + l) * 8;
        float w[8], k[8];
        vector8<kTail>(gate, at, d, 1.f, k);
        vector8<kTail>(a.p.post_weight, at, d, 1.f, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (live && at + (kTail ? j : 0) < d) t[i][j] = __builtin_fmaf(r, __builtin_fmaf(-u[i][j], s2, dx[i][j]) - s1, t[i][j]);
          if (post) v[i][j] = (v[i][j] - pm) * pr;
          ga[i][j] = __builtin_fmaf(t[i][j], v[i][j], ga[i][j]);
          if constexpr (kBias) gt[i][j] += t[i][j];
          u[i][j] = a.p.scale * t[i][j];
          t[i][j] *= k[j] * (post ? w[j] : 1.f);
          s4 = __builtin_fmaf(t[i][j], v[i][j], s4);
          s3 += t[i][j];
        }
        if (live && a.dH) store8<TH, kTail>(dh, at, d, u[i]);
      }
      if (!a.dY) continue;
      TY* dy = static_cast<TY*>(a.dY) + row * d;
      if (post) both(s3, s4, buf[1][phase]);
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        if (post)
#pragma unroll
          for (int j = 0; j < 8; ++j) t[i][j] = pr * (__builtin_fmaf(-v[i][j], s4, t[i][j]) - s3);
        if (live) store8<TY, kTail>(dy, (i * kL + l) * 8, d, t[i]);
      }
    }
    const int64_t seg = blockIdx.x + g;
    if (a.sa) leave(a.sa, seg, ga);
    if (kBias && a.st) leave(a.st, seg, gt);
    if (a.gate_of && threadIdx.x == 0) a.gate_of[seg] = (int)g;
    if (from == begin && begin && begin == g * a.p.gate_rows) {
      // the row between two ends
      clear(ga);
      if (a.sa) leave(a.sa, seg - 1, ga);
      if (kBias && a.st) leave(a.st, seg - 1, ga);
      if (a.gate_of && threadIdx.x == 0) a.gate_of[seg - 1] = (int)g;
    }
    from = to;
  }
  if (a.sw) leave(a.sw, blockIdx.x, gw);
  if (kBias && a.sb) leave(a.sb, blockIdx.x, gb);
}

struct BlockSum {
  BlockBwd b;
  gift_block_norm_grads g;
  bool accumulate;
  int64_t gates;
};

// The vector gradients from the partial sums: 32 columns x 32 threads a column
// per workgroup, thread k of a column adds rows k, k + 32, ..., then the 32 in
// order.  blockIdx.y: 0 weight, 1 bias, 2 post_weight, 3 post_bias, then the
// gates.
__global__ __launch_bounds__(1024) void k_block_sum(BlockSum q) {
  __shared__ float s[2][32][33];
  const int x = threadIdx.x & 31, k = threadIdx.x >> 5, c = (int)blockIdx.x * 32 + x, d = (int)q.b.p.d;
  const int64_t segs = q.b.runs + q.gates - 1;
  auto sum = [&](int which, const float* p, int64_t from, int64_t to, bool gated) {
    float v = 0.f;
    if (c < d && p) {
#pragma unroll 8
      for (int64_t i = from + k; i < to; i += 32) {
        const float f = gated ? q.b.p.gate[(int64_t)q.b.gate_of[i] * d + c] : 1.f;
        v = __builtin_fmaf(f, p[i * d + c], v);
      }
    }
    s[which][k][x] = v;
  };
  auto total = [&](int which) {
    float v = s[which][0][x];
#pragma unroll
    for (int i = 1; i < 32; ++i) v += s[which][i][x];
    return v;
  };
  auto put = [&](float* o, float v) {
    if (k == 0 && c < d) o[c] = q.accumulate ? o[c] + v : v;
  };
  if (blockIdx.y < 4) {
    float* const out[4] = {q.g.dweight, q.g.dbias, q.g.dpost_weight, q.g.dpost_bias};
    const float* const in[4] = {q.b.sw, q.b.sb, q.b.sa, q.b.st};
    float* o = out[blockIdx.y];
    if (!o) return;
    sum(0, in[blockIdx.y], 0, blockIdx.y < 2 ? q.b.runs : segs, blockIdx.y >= 2 && q.b.p.gate);
    __syncthreads();
    put(o, total(0));
    return;
  }
  if (!q.g.dgate) return;
  for (int64_t g = blockIdx.y - 4; g < q.gates; g += gridDim.y - 4) {
    const int64_t first = g * q.b.p.gate_rows, last = min(first + q.b.p.gate_rows, q.b.p.rows) - 1;
    const int64_t from = first / q.b.run + g, to = last / q.b.run + g + 1;
    sum(0, q.b.sa, from, to, false);
    sum(1, q.b.st, from, to, false);
    __syncthreads();
    const float w = q.b.p.post && q.b.p.post_weight && c < d ? q.b.p.post_weight[c] : 1.f;
    const float b = q.b.p.post && q.b.p.post_bias && c < d ? q.b.p.post_bias[c] : 0.f;
    put(q.g.dgate + g * d, __builtin_fmaf(w, total(0), b * total(1)));
    __syncthreads();
  }
}

hipError_t done() { return hipGetLastError(); }

template <class F>
void by_width(int64_t d, F f) {
  auto go = [&](auto L, auto NV) {
    if (d % 8) f(L, NV, std::true_type{});
    else f(L, NV, std::false_type{});
  };
  const std::integral_constant<int, 1> v1;
  const std::integral_constant<int, 2> v2;
  const std::integral_constant<int, 16> l16;
  const std::integral_constant<int, 32> l32;
  const std::integral_constant<int, 64> l64;
  const std::integral_constant<int, 128> l128;
  const std::integral_constant<int, 256> l256;
  const std::integral_constant<int, 512> l512;
  const std::integral_constant<int, 1024> l1024;
  if (d <= 16 * 8) go(l16, v1);
  else if (d <= 32 * 8) go(l32, v1);
  else if (d <= 64 * 8) go(l64, v1);
  else if (d <= 64 * 16) go(l64, v2);
  else if (d <= 128 * 16) go(l128, v2);
  else if (d <= 256 * 16) go(l256, v2);
  else if (d <= 512 * 16) go(l512, v2);
  else go(l1024, v2);
}

template <class F>
void by_types(const gift_block_norm& p, F f) {
  if (p.y_dtype == GIFT_DTYPE_F32) f(0.f, 0.f);
  else if (p.h_dtype == GIFT_DTYPE_F32) f((__bf16)0.f, 0.f);
  else f((__bf16)0.f, (__bf16)0.f);
}

int64_t gates_of(const gift_block_norm& p) { return p.gate ? (p.rows + p.gate_rows - 1) / p.gate_rows : 1; }

// Workgroups of the backward pass: at least a row for each of their groups, and 4.
int64_t runs_of(int64_t rows, int64_t d) {
  const int64_t least = d <= 512 ? 16 : 4, p = (rows + least - 1) / least, most = d <= 512 ? 1024 : 512;
  return p < most ? p : most;
}

}  // namespace

hipError_t launch_block_norm_forward(const gift_block_norm& p, const void* Y, const void* H, void* H2, void* X,
                                     float* stats, hipStream_t s) {
  BlockFwd a{p, Y, H, H2, X, stats};
  if (!p.gate) a.p.gate_rows = p.rows;
  by_types(p, [&](auto y, auto h) {
    by_width(p.d, [&](auto L, auto NV, auto TAIL) {
      constexpr int kL = decltype(L)::value, kGroups = group_threads(kL) / kL;
      // a dimension of a grid holds fewer than 2^32 threads
      const int64_t n = (p.rows + kGroups - 1) / kGroups, most = 1 << 21;
      const dim3 grid((uint32_t)(n < most ? n : most), (uint32_t)((n + most - 1) / most));
      k_block_fwd<decltype(y), decltype(h), kL, decltype(NV)::value, decltype(TAIL)::value>
          <<<grid, dim3(group_threads(kL)), 0, s>>>(a);
    });
  });
  return done();
}

size_t block_norm_backward_ws(int64_t rows, int64_t d, int64_t gates) {
  const int64_t runs = runs_of(rows, d), segs = runs + gates - 1;
  return align_up((size_t)segs * 4) + 2 * align_up((size_t)runs * d * 4) + 2 * align_up((size_t)segs * d * 4);
}

hipError_t launch_block_norm_backward(const gift_block_norm& p, const void* dX, const void* dH2, const void* Y,
                                      const void* H2, const float* stats, void* dY, void* dH,
                                      const gift_block_norm_grads& g, bool accumulate, void* ws, hipStream_t s) {
  BlockSum q{};
  q.g = g;
  q.accumulate = accumulate;
  q.gates = gates_of(p);
  BlockBwd& a = q.b;
  a.p = p;
  if (!p.gate) a.p.gate_rows = p.rows;
  a.dX = dX;
  a.dH2 = dH2;
  a.Y = Y;
  a.H2 = H2;
  a.stats = stats;
  a.dY = dY;
  a.dH = dH;
  const int64_t most = runs_of(p.rows, p.d), segs = most + q.gates - 1;
  a.run = (p.rows + most - 1) / most;
  a.runs = (int)((p.rows + a.run - 1) / a.run);
  uint8_t* at = static_cast<uint8_t*>(ws);
  auto take = [&](bool want, size_t bytes) {
    float* r = want ? reinterpret_cast<float*>(at) : nullptr;
    at += align_up(bytes);
    return r;
  };
  const bool biased = p.post && p.post_bias;
  a.gate_of = reinterpret_cast<int*>(take(p.gate && (g.dpost_weight || g.dpost_bias), (size_t)segs * 4));
  a.sw = take(g.dweight, (size_t)most * p.d * 4);
  a.sb = take(g.dbias, (size_t)most * p.d * 4);
  a.sa = take(g.dpost_weight || g.dgate, (size_t)segs * p.d * 4);
  a.st = take(g.dpost_bias || (g.dgate && biased), (size_t)segs * p.d * 4);
  by_types(p, [&](auto y, auto h) {
    by_width(p.d, [&](auto L, auto NV, auto TAIL) {
      constexpr int kL = decltype(L)::value, kNV = decltype(NV)::value;
      constexpr bool kTail = decltype(TAIL)::value;
      const dim3 grid((uint32_t)a.runs), block(group_threads(kL));
      if (a.sb || a.st) k_block_bwd<decltype(y), decltype(h), kL, kNV, kTail, true><<<grid, block, 0, s>>>(a);
      else k_block_bwd<decltype(y), decltype(h), kL, kNV, kTail, false><<<grid, block, 0, s>>>(a);
    });
  });
  hipError_t e = done();
  if (e != hipSuccess || !(a.sw || a.sb || a.sa || a.st)) return e;
  const int64_t blocks = 4 + (g.dgate ? (q.gates < 60000 ? q.gates : 60000) : 0);
  k_block_sum<<<dim3((uint32_t)((p.d + 31) / 32), (uint32_t)blocks), dim3(1024), 0, s>>>(q);
  return done();
}

}  // namespace gift
