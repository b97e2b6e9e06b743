// Head rows of projections: root-mean-square norm, position rotation and their way from where a
// projection left them to where the attention reads them.  Shared by prep.cu (dense inputs) and
// paged_append.cu (slots of a paged cache).
//
// A row of D channels is held by D / 8 neighbouring lanes, eight consecutive channels each (16 bytes
// of bf16, 32 bytes of float32), so that a row is read and written in whole 32-byte sectors, the sum
// of squares takes log2(D / 8) shuffles, and the partner of a rotated channel is either in the same
// lane (neighbouring pairs) or in the same register of another lane of the row (halves).
// These kernels would be bound by the instructions they issue before they are by memory (a first form
// issued 210 for the two rows of a warp at 128 channels, where reading and writing them leaves time for 170;
// this one 122), so what belongs to a token or to its queries, keys or values is worked out once for all
// their heads, and addresses once for a chunk of rows.
#pragma once

#include "common.cuh"

namespace dma {

// ---------------------------------------------------------------- eight channels

// Eight consecutive channels as stored, and as floats.
template <typename T> struct Raw8;
template <> struct Raw8<uint16_t> { uint4 a; };
template <> struct Raw8<float> { float4 a, b; };
struct Chan8 { float v[8]; };

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
template <typename T> DMA_DEVINL Chan8 channels8(const Raw8<T>& r) {
  Chan8 p;
  widen8(r, p.v);
  return p;
}
// The one rounding of a result (bf16: to nearest even).
DMA_DEVINL void store8(uint16_t* p, const Chan8& y) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(y.v[0], y.v[1]), pack_bf16x2(y.v[2], y.v[3]),
                                            pack_bf16x2(y.v[4], y.v[5]), pack_bf16x2(y.v[6], y.v[7]));
}
DMA_DEVINL void store8(float* p, const Chan8& y) {
  reinterpret_cast<float4*>(p)[0] = make_float4(y.v[0], y.v[1], y.v[2], y.v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(y.v[4], y.v[5], y.v[6], y.v[7]);
}

// Sum over the L neighbouring lanes of a row.
template <int L> DMA_DEVINL float row_sum(float x) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
// Sum over a row of the products of two rows' channels.
template <int L> DMA_DEVINL float row_dot(const Chan8& a, const Chan8& b) {
  float s = a.v[0] * b.v[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) s = fmaf(a.v[i], b.v[i], s);
  return row_sum<L>(s);
}

// ---------------------------------------------------------------- rotation

// Turns a position advances a channel pair's angle by, as a 64-bit binary fraction: multiplied by an
// integer position it wraps around just as the angle does, so that the angle at any position is exact
// but for the fraction's own rounding (2^-53 of inv_freq / 2 pi a position; float32 would leave the angle
// at position 2^24 wrong by a radian).
DMA_DEVINL uint64_t turn_rate(float inv_freq) {
  double t = (double)inv_freq * 0.15915494309189533577;
  t -= floor(t);
  return __double2ull_rn(t * 18446744073709551616.0);
}
// (cos, sin) at a position.  The reduced angle's upper 24 bits go through sincospif, the 8 below them are
// put back to first order, so that both are good to about one float32 rounding.
DMA_DEVINL float2 turn_at(uint64_t rate, int position) {
  const uint32_t lo = (uint32_t)rate, hi = (uint32_t)(rate >> 32), n = (uint32_t)position;
  uint32_t f = __umulhi(lo, n) + hi * n;   // the product's bits 32 .. 63
  if (position < 0) f -= lo;
  const float half_turns = (float)(int)(f & 0xffffff00u) * 4.656612873077393e-10f;   // 2^-31
  const float rest = (float)(f & 0xffu) * (3.14159265f * 4.656612873077393e-10f);
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(fmaf(-s, rest, c), fmaf(c, rest, s));
}

// What a rotation does to a lane's eight channels: y = x c + o s, o being the partner channels (of the
// same row, in lane `partner`, or swapped within a pair).  rot is a multiple of 16, so a lane's channels
// are all rotated or none, and (halves) all in the first or all in the second half.
struct LaneTurn {
  Chan8 c, s;
  int partner;
  bool on;
};

constexpr int kTabPad = 8;   // entries (1, 0) behind a token's table: the turn of channels beyond rot

// What does not depend on the token: the partner, and where in the table this lane's entries begin.
template <int D> DMA_DEVINL int lane_start(LaneTurn& t, int rot, bool inter, int lane) {
  const int e = (lane % (D / 8)) * 8, half = rot >> 1;
  const bool upper = !inter && e >= half;
  t.on = e < rot;
  t.partner = inter || !t.on ? lane : lane + (upper ? -(half >> 3) : (half >> 3));
  return !t.on ? D / 2 : inter ? e >> 1 : upper ? e - half : e;
}

// The turn of a token: tab its (cos, sin).  The first member of a pair loses sin times the second, the
// second gains sin times the first; back: the other way round.
template <bool inter> DMA_DEVINL void lane_turn(LaneTurn& t, const float2* tab, int start, bool upper, bool back) {
  const float4* q = reinterpret_cast<const float4*>(tab + start);   // start is a multiple of 4
  if (inter) {
    const float plus = back ? -1.f : 1.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 v = q[i];
      t.c.v[4 * i] = t.c.v[4 * i + 1] = v.x;
      t.c.v[4 * i + 2] = t.c.v[4 * i + 3] = v.z;
      t.s.v[4 * i] = -plus * v.y;
      t.s.v[4 * i + 1] = plus * v.y;
      t.s.v[4 * i + 2] = -plus * v.w;
      t.s.v[4 * i + 3] = plus * v.w;
    }
  } else {
    const float sign = upper != back ? 1.f : -1.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = q[i];
      t.c.v[2 * i] = v.x;
      t.c.v[2 * i + 1] = v.z;
      t.s.v[2 * i] = sign * v.y;
      t.s.v[2 * i + 1] = sign * v.w;
    }
  }
}

// Channels beyond rot stay as they are, bit for bit.
template <bool inter> DMA_DEVINL Chan8 rotate8(const Chan8& x, const LaneTurn& t) {
  Chan8 y;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float o = inter ? x.v[i ^ 1] : __shfl_sync(0xffffffffu, x.v[i], t.partner);
    y.v[i] = x.v[i];
    if (t.on) y.v[i] = fmaf(o, t.s.v[i], x.v[i] * t.c.v[i]);
  }
  return y;
}

// ---------------------------------------------------------------- the walk over rows

constexpr int kRwThreads = 256;
constexpr int kRwWarps = kRwThreads / 32;

// The work of a warp: tokens tok, tok + step, .. and of each its chunks of queries, keys and values: chunk,
// chunk + wt, .., each U units of RPW = 32 / L neighbouring heads (wt = 1, 2, 4 or 8 warps share a token, many
// where there are few tokens).  The warp walks it twice, a ring's depth apart: once to send for the rows,
// once to work on them.
struct Walk {
  unsigned tok, tokens, step;
  unsigned b, n, N, step_b, step_n;   // the token as (batch row, position)
  int chunk, first, chunks, wt, cq, ck;
  // block of blocks share the tokens
  DMA_DEVINL Walk(const PrepArgs& a, int per_chunk, int wt_, unsigned block, unsigned blocks) : wt(wt_) {
    const int warp = threadIdx.x >> 5;
    N = (unsigned)a.N;
    tokens = (unsigned)a.B * N;
    step = blocks * (kRwWarps / wt);
    tok = block * (kRwWarps / wt) + warp / wt;
    b = tok / N;
    n = tok - b * N;
    step_b = step / N;
    step_n = step - step_b * N;
    cq = a.in[0] != nullptr || a.grad[0] != nullptr ? (a.H + per_chunk - 1) / per_chunk : 0;
    ck = (a.Hkv + per_chunk - 1) / per_chunk;
    chunks = cq + (a.out[2] != nullptr ? 2 : 1) * ck;
    first = chunk = warp % wt;
    if (first >= chunks) tok = tokens;
  }
  DMA_DEVINL bool more() const { return tok < tokens; }
  DMA_DEVINL void next() {
    chunk += wt;
    if (chunk >= chunks) {
      chunk = first;
      tok += step;
      b += step_b;
      n += step_n;
      if (n >= N) {
        n -= N;
        ++b;
      }
    }
  }
  // 0: queries, 1: keys, 2: values; and the number of the chunk among them
  DMA_DEVINL int part() const { return chunk < cq ? 0 : chunk < cq + ck ? 1 : 2; }
  DMA_DEVINL int within(int part) const { return part == 0 ? chunk : part == 1 ? chunk - cq : chunk - cq - ck; }
};

// Rows on their way: every lane copies its own channels of the chunks to come into its own places of a ring
// in shared memory (U rows of NP 16-byte pieces a chunk, DEPTH chunks) and reads back only those, so that no
// warp waits for another and the loads in flight cost no registers.
template <int NP, int U, int DEPTH> struct RowRing {
  static constexpr int kRow = NP * kRwThreads * 16, kBytes = DEPTH * U * kRow;
  template <typename T> static DMA_DEVINL void copy(unsigned char* row, int piece, const T* src, bool in) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i)
      cp_async_16(smem_u32(row) + (piece + i) * kRwThreads * 16, src + i * 4, in ? 16 : 0);
  }
  template <typename T> static DMA_DEVINL Raw8<T> read(const unsigned char* row, int piece) {
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i)
      reinterpret_cast<uint4*>(&r)[i] = *reinterpret_cast<const uint4*>(row + (piece + i) * kRwThreads * 16);
    return r;
  }
  // send(at, place) for every chunk of a walk, DEPTH - 1 chunks ahead of work(at, place); ready() (by every
  // warp of the block) once the first are on their way
  template <typename Send, typename Ready, typename Work>
  static DMA_DEVINL void run(Walk w, unsigned char* smem, Send send, Ready ready, Work work) {
    unsigned char* const ring = smem + threadIdx.x * 16;
    Walk s = w;
    int to = 0, from = 0;
    auto ahead = [&]() {
      if (s.more()) {
        send(s, ring + to * (U * kRow));
        s.next();
      }
      to = to + 1 == DEPTH ? 0 : to + 1;
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < DEPTH - 1; ++i) ahead();
    ready();
#pragma unroll 1
    while (w.more()) {
      ahead();
      cp_async_wait<DEPTH - 1>();
      work(w, ring + from * (U * kRow));
      from = from + 1 == DEPTH ? 0 : from + 1;
      w.next();
    }
  }
};

// Blocks of a walk, and the warps that share a token: as many as it takes to give every warp of a full GPU
// two shares (so that the last round weighs little), 8 at most.
inline int walk_blocks(long long tokens, int per_sm, int* wt) {
  const int sms = sm_count();
  *wt = 1;
  while (*wt < kRwWarps && tokens * *wt < 2LL * per_sm * sms * kRwWarps) *wt *= 2;
  const long long tpb = kRwWarps / *wt, need = (tokens + tpb - 1) / tpb;
  return (int)(need < (long long)per_sm * sms ? need : (long long)per_sm * sms);
}

// (cos, sin) of the angles at one position into the warp's own table.
DMA_DEVINL void token_table(const uint64_t* rate, int half, int position, float2* tab) {
  __syncwarp();
  for (int k = threadIdx.x & 31; k < half; k += 32) tab[k] = turn_at(rate[k], position);
  __syncwarp();
}

template <typename T> constexpr int fwd_rows() { return sizeof(T) == 2 ? 4 : 2; }
template <typename T, int DEPTH> using FwdRing = RowRing<sizeof(T) / 2, fwd_rows<T>(), DEPTH>;

// Queries and keys normed and rotated, values copied, from the projections (a.in, a.stride) to where Dest
// says: dest.enter(at, token) (every lane of the warp) is false if nothing of the token is written,
// else token.position is its position and dest.row(part, token) the address of its first head's row, heads
// dest.step(part) elements apart.  Dest::kDepth chunks are in flight.  By a block of kRwThreads, with
// FwdRing<T, Dest::kDepth>::kBytes of shared memory at ring_smem.
template <typename T, int D, bool INTER, typename Dest>
DMA_DEVINL void walk_rows(const PrepArgs& a, const Dest& dest, int wt, unsigned block, unsigned blocks,
                          unsigned char* ring_smem) {
  constexpr int L = D / 8, RPW = 32 / L, U = fwd_rows<T>();
  using Ring = FwdRing<T, Dest::kDepth>;
  __shared__ __align__(16) float2 tab[kRwWarps][D / 2 + kTabPad];
  __shared__ uint64_t rate[D / 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, grp = lane / L, e = (lane % L) * 8;
  const bool upper = e >= a.rot >> 1;
  auto ready = [&]() {
    for (int k = threadIdx.x; k < a.rot >> 1; k += kRwThreads) rate[k] = turn_rate(__ldg(a.inv_freq + k));
    if (lane < kTabPad) tab[warp][D / 2 + lane] = make_float2(1.f, 0.f);
    __syncthreads();
  };
  auto send = [&](const Walk& at, unsigned char* place) {
    const int part = at.part(), h = at.within(part) * (RPW * U) + grp, left = (part == 0 ? a.H : a.Hkv) - h;
    const long long sh = a.stride[part][2];
    const T* base = (const T*)a.in[part];
    const T* src = base + at.b * a.stride[part][0] + at.n * a.stride[part][1] + h * sh + e;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      Ring::copy(place + u * Ring::kRow, 0, u * RPW < left ? src : base, u * RPW < left);
      src += RPW * sh;
    }
  };
  typename Dest::Token token = {};
  LaneTurn turn;
  const int start = lane_start<D>(turn, a.rot, INTER, lane);
  unsigned have = 0xffffffffu;   // the token of the warp's table
  bool live = false;
  auto work = [&](const Walk& at, const unsigned char* place) {
    if (have != at.tok) {
      have = at.tok;
      live = dest.enter(at, token);
      if (live) {
        token_table(rate, a.rot >> 1, token.position, tab[warp]);
        lane_turn<INTER>(turn, tab[warp], start, upper, false);
      }
    }
    if (!live) return;
    const int part = at.part(), h = at.within(part) * (RPW * U) + grp, left = (part == 0 ? a.H : a.Hkv) - h;
    const size_t sh = dest.step(part);
    T* dst = (T*)dest.row(part, token) + h * sh + e;
    if (part == 2) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u * RPW < left) store_raw8(dst, Ring::template read<T>(place + u * Ring::kRow, 0));
        dst += RPW * sh;
      }
      return;
    }
    const T* wp = (const T*)a.weight[part];
    Chan8 g;
    if (wp != nullptr) g = channels8(load_raw8(wp + e));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      Chan8 x = channels8(Ring::template read<T>(place + u * Ring::kRow, 0));
      if (wp != nullptr) {
        const float r = rsqrtf(row_dot<L>(x, x) * (1.f / D) + a.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) x.v[i] *= r * g.v[i];
      }
      const Chan8 y = rotate8<INTER>(x, turn);
      if (u * RPW < left) store8(dst, y);
      dst += RPW * sh;
    }
  };
  Ring::run(Walk(a, RPW * U, wt, block, blocks), ring_smem, send, ready, work);
}

}  // namespace dma
