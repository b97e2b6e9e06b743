// One head row of a projection: root-mean-square norm and position rotation, shared by the kernels
// that prepare the attention's inputs (prep.cu) and that append to a paged cache (paged_append.cu).
//
// A row of D channels is held by D / 8 neighbouring lanes, eight consecutive channels each (16 bytes
// of bf16, 32 bytes of float32), so that a row is read and written in whole 32-byte sectors, the sum
// of squares takes log2(D / 8) shuffles, and the partner of a rotated channel is either in the same
// lane (neighbouring pairs) or in the same register of another lane of the row (halves).
#pragma once

#include "common.cuh"

namespace dma {

// Eight consecutive channels as stored, and as floats.
template <typename T> struct Raw8;
template <> struct Raw8<uint16_t> { uint4 a; };
template <> struct Raw8<float> { float4 a, b; };

DMA_DEVINL Raw8<uint16_t> load_raw8(const uint16_t* p) { return {*reinterpret_cast<const uint4*>(p)}; }
DMA_DEVINL Raw8<float> load_raw8(const float* p) {
  return {reinterpret_cast<const float4*>(p)[0], reinterpret_cast<const float4*>(p)[1]};
}
DMA_DEVINL void store_raw8(uint16_t* p, const Raw8<uint16_t>& v) { *reinterpret_cast<uint4*>(p) = v.a; }
DMA_DEVINL void store_raw8(float* p, const Raw8<float>& v) {
  reinterpret_cast<float4*>(p)[0] = v.a;
  reinterpret_cast<float4*>(p)[1] = v.b;
}
DMA_DEVINL void widen8(const Raw8<uint16_t>& r, float (&v)[8]) {
  const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
DMA_DEVINL void widen8(const Raw8<float>& r, float (&v)[8]) {
  v[0] = r.a.x; v[1] = r.a.y; v[2] = r.a.z; v[3] = r.a.w;
  v[4] = r.b.x; v[5] = r.b.y; v[6] = r.b.z; v[7] = r.b.w;
}
// The one rounding of a result (bf16: to nearest even).
DMA_DEVINL void store8(uint16_t* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                            pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
DMA_DEVINL void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// Sum over the L neighbouring lanes of a row.
template <int L> DMA_DEVINL float row_sum(float x) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// (cos, sin) of position x inv_freq.  The angle is formed and reduced in double precision, in turns:
// at position 2^24 float32 would leave it wrong by a radian.  The reduced angle is split into a float
// and its remainder, which the first-order term puts back, so that cos and sin are good to about one
// float32 rounding.
DMA_DEVINL float2 turn_of(int position, float inv_freq) {
  const double t = (double)position * ((double)inv_freq * 0.15915494309189533577);
  const double f = 2.0 * (t - rint(t));       // half turns in [-1, 1]
  const float hi = (float)f, lo = (float)(f - (double)hi) * 3.14159265f;
  float s, c;
  sincospif(hi, &s, &c);
  return make_float2(fmaf(-s, lo, c), fmaf(c, lo, s));
}

// The part of the rotation that one lane needs: its eight channels' (cos, sin), and where their
// partners are.  rot is a multiple of 16, so a lane's channels are all rotated or none, and (halves)
// all in the first or all in the second half.
struct LaneTurn {
  float c[8], s[8];   // halves: of channel i; neighbouring pairs: [2 i], [2 i + 1] alike
  int partner;        // lane (in the warp) that holds the partner channels; halves only
  bool on;            // this lane's channels are rotated
  bool upper;         // halves: the channels are second members of their pairs
};

// tab: (cos, sin) of the rot / 2 frequencies at this row's position.
template <int L> DMA_DEVINL void lane_turn(LaneTurn& t, const float2* tab, int rot, bool inter, int lane) {
  const int e = (lane % L) * 8, half = rot >> 1;
  t.on = e < rot;
  t.upper = !inter && e >= half;
  t.partner = inter || !t.on ? lane : lane + (t.upper ? -(half >> 3) : (half >> 3));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int k = inter ? (e + i) >> 1 : (t.upper ? e - half + i : e + i);
    const float2 v = t.on ? tab[k] : make_float2(1.f, 0.f);
    t.c[i] = v.x;
    t.s[i] = v.y;
  }
}

// y <- R y (BACK: R^T y): (a, b) -> (a cos - b sin, b cos + a sin).  Channels beyond rot stay as they
// are, bit for bit.
template <bool BACK> DMA_DEVINL void rotate8(float (&y)[8], const LaneTurn& t, bool inter) {
  if (inter) {
    if (t.on) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = y[2 * i], b = y[2 * i + 1], c = t.c[2 * i], s = BACK ? -t.s[2 * i] : t.s[2 * i];
        y[2 * i] = fmaf(a, c, -b * s);
        y[2 * i + 1] = fmaf(b, c, a * s);
      }
    }
  } else {
    const float sign = t.upper != BACK ? 1.f : -1.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float o = __shfl_sync(0xffffffffu, y[i], t.partner);
      if (t.on) y[i] = fmaf(y[i], t.c[i], sign * o * t.s[i]);
    }
  }
}

}  // namespace dma
