// Rotary positions shared by the rotation and cache-append kernels.
//
// Pair i of a rotated head turns by the angle p * w_i (w_i radians per token):
//
//   y_a = f (x_a cos - x_b sin),   y_b = f (x_a sin + x_b cos)
//
// with (a, b) = (2i, 2i + 1) in the interleaved layout and (i, i + rot / 2) in
// the half layout.  Only p * w_i modulo one turn matters.  w_i / 2 pi is held
// as a 64-bit fraction of a turn, so the product with the integer position
// wraps by itself: the angle of a far position is as exact as that of a near
// one (2^-62 of w_i and 2^-64 of a turn per token, 2^-34 of a turn in the
// reduction), without 64-bit floating point.
#pragma once
#include <cstdint>

namespace mla {

struct RopeArgs {
  const double* inv_freq;  // [rot / 2] radians per token, device
  int rot;                 // rotated dims, multiple of 16; 0: nothing is rotated
  int first;               // first rotated dim, multiple of 8
  int interleaved;         // pair layout
  float factor;            // on the rotated values
};

// Radians per token -> 2^64ths of a turn per token, modulo a turn: the product
// of w's 53 bits with those of 1 / 2 pi, in integers (64-bit floating point is
// 1/64 of the 32-bit rate here).
__device__ __forceinline__ unsigned long long turn_rate(double w) {
  const unsigned long long bits = (unsigned long long)__double_as_longlong(w);
  const int e = (int)((bits >> 52) & 0x7FFu) - 1024;        // w = 1.m 2^(e + 1)
  if (e < -1000) return 0;
  // w / 2 pi = hi 2^(e - 64) turns
  const unsigned long long hi =
      __umul64hi(((bits << 11) | (1ull << 63)), 0xa2f9836e4e441529ull);   // 2^66 / 2 pi
  unsigned long long r;
  if (e >= 0) r = e < 64 ? hi << e : 0;
  else r = e >= -64 ? ((hi >> (-e - 1)) + 1) >> 1 : 0;
  return (bits >> 63) ? 0 - r : r;
}

// (f cos, f sin) of position pos at `rate`.  The turn is split into the
// nearest quarter and a rest of at most an eighth, which is exact in integers;
// the rest's sine and cosine are their Taylor sums, which end below 2^-25 for
// |x| <= pi / 4.
__device__ __forceinline__ float2 turn_cs(unsigned long long rate, int pos, float f) {
  const unsigned long long u = rate * (unsigned long long)(long long)pos;
  const unsigned q = (unsigned)((u + (1ull << 61)) >> 62);
  const long long r = (long long)(u - ((unsigned long long)q << 62));
  const float x = (float)(int)(r >> 30) * 3.657295198e-10f;   // 2 pi 2^-34
  const float y = x * x;
  float s = fmaf(y, 1.0f / 362880.0f, -1.0f / 5040.0f);
  s = fmaf(y, s, 1.0f / 120.0f);
  s = fmaf(y, s, -1.0f / 6.0f);
  s = fmaf(x * y, s, x);
  float c = fmaf(y, 1.0f / 40320.0f, -1.0f / 720.0f);
  c = fmaf(y, c, 1.0f / 24.0f);
  c = fmaf(y, c, -0.5f);
  c = fmaf(y, c, 1.0f);
  if (q & 1) {
    const float t = c;
    c = -s;
    s = t;
  }
  if (q & 2) {
    c = -c;
    s = -s;
  }
  return make_float2(f * c, f * s);
}

__device__ __forceinline__ void turn_pair(float& a, float& b, float2 cs) {
  const float x = a;
  a = fmaf(x, cs.x, -b * cs.y);
  b = fmaf(x, cs.y, b * cs.x);
}

}  // namespace mla
