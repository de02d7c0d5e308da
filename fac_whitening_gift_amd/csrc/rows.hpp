// Rows of a matrix in the registers of a group of lanes: what norm.hip and
// block_norm.hip share.
#pragma once

#include "device.hpp"
#include "mx.hpp"

namespace gift {

template <class T>
constexpr int kVecOf = 16 / sizeof(T);  // elements of a 16-byte vector

// 16 bytes of T as floats
template <class T>
__device__ __forceinline__ void unpack(const uint4& q, float (&o)[kVecOf<T>]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2) {
      o[2 * i] = __uint_as_float(w[i] << 16);
      o[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
      o[i] = __uint_as_float(w[i]);
    }
  }
}

template <class T>
__device__ __forceinline__ uint4 pack(const float (&v)[kVecOf<T>]) {
  struct { T v[kVecOf<T>]; } o;
#pragma unroll
  for (int i = 0; i < kVecOf<T>; ++i) o.v[i] = (T)v[i];
  return __builtin_bit_cast(uint4, o);
}

// v moved down by `by` elements, `fill` behind: a row's last vector, loaded
// so as to end with the row
template <int kVec>
__device__ __forceinline__ void shift(float (&v)[kVec], int by, float fill) {
#pragma unroll
  for (int b = 1; b < kVec; b *= 2)
    if (by & b) {
#pragma unroll
      for (int j = 0; j < kVec; ++j) v[j] = j + b < kVec ? v[j + b < kVec ? j + b : 0] : fill;
    }
}

// kVec floats at `at` of a d-vector that may be NULL (then `none`)
template <int kVec, bool kTail>
__device__ __forceinline__ void ldw(const float* p, int at, int d, float none, float (&o)[kVec]) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) o[i] = none;
    return;
  }
  const int from = kTail ? min(at, d - kVec) : at;
#pragma unroll
  for (int i = 0; i < kVec / 4; ++i) {
    const uint4 q = ld16(p + from + 4 * i);
    o[4 * i] = __uint_as_float(q.x);
    o[4 * i + 1] = __uint_as_float(q.y);
    o[4 * i + 2] = __uint_as_float(q.z);
    o[4 * i + 3] = __uint_as_float(q.w);
  }
  if (kTail && at != from) shift(o, at - from, 0.f);
}

// A lane's vector at column `at` < d of a row of Y.  kNt: around the caches.
// The backward pass gains by it in whole vectors (16384 x 4096 bf16: 89.5 ->
// 81.5 us), the forward pass loses (57.0 -> 59.7 us).
template <class T, bool kNt, bool kTail>
__device__ __forceinline__ void stv(T* row, int at, int d, const float (&v)[kVecOf<T>]) {
  if (kTail && at + kVecOf<T> > d) {
#pragma unroll
    for (int i = 0; i < kVecOf<T>; ++i)
      if (at + i < d) row[at + i] = (T)v[i];
  } else if constexpr (kNt) {
    st16_nt(row + at, pack<T>(v));
  } else {
    st16(row + at, pack<T>(v));
  }
}

// n <= kVec elements (the wide kernels)
template <class T>
__device__ __forceinline__ void ldn(const T* p, int n, float (&o)[kVecOf<T>]) {
  if (n >= kVecOf<T>) {
    unpack<T>(ld16(p), o);
  } else {
#pragma unroll
    for (int i = 0; i < kVecOf<T>; ++i) o[i] = i < n ? (float)p[i] : 0.f;
  }
}

// Sum over the kL <= 64 lanes of a row (or over a wave).
template <int kL>
__device__ __forceinline__ float lane_sum(float v) {
#pragma unroll
  for (int o = (kL < 64 ? kL : 64) / 2; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

constexpr int waves_of(int kL) { return kL > 64 ? kL / 64 : 1; }

// Sum of v over the kL lanes of a row; buf: one float per wave of them.
template <int kL>
__device__ __forceinline__ float group_sum(float v, float* buf) {
  constexpr int kW = waves_of(kL);
  v = lane_sum<kL>(v);
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

constexpr int group_threads(int kL) { return kL < 256 ? 256 : kL; }

}  // namespace gift
