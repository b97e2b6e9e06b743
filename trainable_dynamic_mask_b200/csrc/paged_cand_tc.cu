// Candidates of a shared prefix against many sequences' queries, on tcgen05.
//
// CTA = (part of a head's candidates, head, 64 sequences).  S = Q K^T and O = P V are products of 128 rows: the
// 64 queries twice, so that all 128 TMEM lanes of a warpgroup have work on a tile of 128 candidates: row r
// holds sequence r mod 64, lanes 0 - 63 weigh the tile's first 64 keys, lanes 64 - 127 the others (their
// weights of the rest are stored as zeros).  The two warpgroups take tiles in turn, each with its own K and V
// buffers, S, P and O (512 TMEM columns: one CTA an SM), and meet at the end only.  K and V rows are gathered
// with 16-byte asynchronous copies into the swizzled operand layout; the next tile's K is sent for when S is
// done, its V when O is.
// A weight is split into two bf16 parts, both multiplied with V: one part alone would round every weight to 8
// bits, as much as the output's own rounding.  P's parts take the columns of the S they come from.
// A candidate that a sequence did not select has weight exactly 0 there; if a V row holds an infinity or NaN,
// 0 times that would still spoil the sum, so a tile with such a value is added up in plain arithmetic that
// leaves weights of 0 out.
//
// 2048 candidates of 32 heads, 64 sequences (33.5 MB of rows, 5.1 us at the copy rate): 19 us of a CTA's time, of
// which the first rows' way 4, the products and what waits for them 7 (the tensor pipe itself 3.3), weights 4,
// joining and writing the results 3.  A CTA passes through its code once or twice, so instructions that come
// from memory count: scores are read from TMEM twice, in loops of 16, which is a third faster than one pass
// over 64 registers.  Taken the other way round (S^T = K Q^T with the sequences as columns, half the tensor
// time, maxima by a reduction over lanes) it took 7 us more.
#include "rows.cuh"
#include "tc_ops.cuh"

namespace dma {
namespace {

enum : int { kErrTimeoutS = 0x400, kErrTimeoutPV = 0x1000 };

constexpr int kCtTile = 128, kCtThreads = 256, kCtMost = 512;   // candidates of a tile; threads; candidates of a CTA

template <int D> struct CtSmem {
  static constexpr int kTile = kCtTile * D * 2;               // K or V of a tile, or Q
  static constexpr int kQ = 4 * kTile;                        // [2 warpgroups][K, V], then Q
  static constexpr int kRow = (D + 4) * 4;                    // a row of results, in the tiles' place
  static constexpr int kUsed = 5 * kTile > 256 * kRow ? 5 * kTile : 256 * kRow;
  // above half of an SM's shared memory: a second CTA could not have its TMEM columns
  static constexpr int kBytes = (kUsed > 120 * 1024 ? kUsed : 120 * 1024) + 1024;
};

struct CtShared {
  uint64_t s_full[2], pv_done[2], drain[2];
  uint32_t tmem_base;
  int abort_flag;
  int odd[2];
};

DMA_DEVINL void wg_sync(int w) {
  if (w == 0) asm volatile("bar.sync 1, 128;\n" ::: "memory");
  else asm volatile("bar.sync 2, 128;\n" ::: "memory");
}

// Byte offset of 16-byte chunk c of row r in an operand tile of 128 rows.
DMA_DEVINL uint32_t ct_at(int r, int c) {
  return (uint32_t)((c >> 3) * (kCtTile * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

template <int KK, int NK> DMA_DEVINL void qk_steps(uint32_t d, uint64_t dq, uint64_t dk, uint32_t id) {
  if constexpr (KK < NK) {
    mma_ss_at<(KK >> 2) * (kCtTile * 128) + (KK & 3) * 32>(d, dq, dk, id, KK > 0 ? 1u : 0u);
    qk_steps<KK + 1, NK>(d, dq, dk, id);
  }
}
template <int KK, int NK>
DMA_DEVINL void pv_steps(uint32_t d, uint32_t a, uint64_t dv, uint32_t id, uint32_t accumulate) {
  if constexpr (KK < NK) {
    mma_ts_at<KK>(d, a, dv, id, KK > 0 ? 1u : accumulate);
    pv_steps<KK + 1, NK>(d, a, dv, id, accumulate);
  }
}

template <int D>
__global__ void __launch_bounds__(kCtThreads, 1)
paged_cand_tc_kernel(const uint16_t* Q, const uint16_t* K, const uint16_t* V, const int4* rows, const int32_t* crow,
                     const int2* cent, float* __restrict__ part, int32_t* __restrict__ status, int B, int H, int Hkv,
                     int page_shift, int n_slots, int cand_len, int cand_split, int n_part, float scale) {
  using S = CtSmem<D>;
  constexpr int CH = D / 8;
  extern __shared__ __align__(1024) unsigned char raw[];
  unsigned char* const sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  __shared__ __align__(16) uint32_t ckey[kCtMost];
  __shared__ __align__(16) float cdel[kCtMost];
  __shared__ int cslot[kCtMost];
  __shared__ float gm[4][64], gl[4][64];
  __shared__ CtShared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, w = warp >> 2, r = tid & 127;
  const int half = r >> 6, h = blockIdx.y, g = h / (H / Hkv), s0 = blockIdx.z * 64, s = s0 + (r & 63);
  const int c0 = blockIdx.x * cand_split;
  volatile int* abort_flag = &sh.abort_flag;
  pdl_trigger();
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sh.s_full[i], 1);
      tc::mbar_init(&sh.pv_done[i], 1);
      tc::mbar_init(&sh.drain[i], 1);
      sh.odd[i] = 0;
    }
    sh.abort_flag = 0;
    tc::fence_mbar_init();
  }
  if (warp == 0) {
    tc::tmem_alloc(&sh.tmem_base, 512);
    tc::tmem_relinquish();
  }
  pdl_wait();
  // the entries are read before it is known how many there are
  const int room = min(cand_len - c0, cand_split), known = crow[h];
  int2 ent[kCtMost / kCtThreads];
#pragma unroll
  for (int k = 0; k < kCtMost / kCtThreads; ++k) {
    ent[k] = make_int2(0, 0);
    if (tid + k * kCtThreads < room) ent[k] = cent[(size_t)h * cand_len + c0 + tid + k * kCtThreads];
  }
  const int nc = max(0, min(known - c0, room));
  const int nt = (nc + kCtTile - 1) / kCtTile;
#pragma unroll
  for (int k = 0; k < kCtMost / kCtThreads; ++k) {
    const int i = tid + k * kCtThreads;
    const int2 e = i < nc ? ent[k] : make_int2(0, 0);
    cslot[i] = (unsigned)e.x < (unsigned)n_slots ? e.x : 0;   // a workspace never written may hold anything
    cdel[i] = __int_as_float(e.y);
    ckey[i] = i < nc ? order_key(__int_as_float(e.y)) : 0u;
  }
#pragma unroll
  for (int i = 0; i < 64 * CH / kCtThreads; ++i) {
    const int u = tid + i * kCtThreads, q = u / CH, c = u % CH;
    const bool in = s0 + q < B;
    const uint16_t* src = Q + ((size_t)(in ? s0 + q : 0) * H + h) * D + c * 8;
    cp_async_16(smem_u32(sm) + S::kQ + ct_at(q, c), src, in ? 16 : 0);
    cp_async_16(smem_u32(sm) + S::kQ + ct_at(q + 64, c), src, in ? 16 : 0);
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = sh.tmem_base, lanes = (uint32_t)((warp & 3) * 32) << 16;
  const uint32_t tS = tmem + w * 128, tO = tmem + 256 + w * 128;   // of this warpgroup
  const uint32_t kbuf = smem_u32(sm) + w * 2 * S::kTile, vbuf = kbuf + S::kTile;
  const int mask = (1 << page_shift) - 1;
  auto load_tile = [&](const uint16_t* src, uint32_t to, int t) {   // by the warpgroup
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int u = r + i * 128, row = u / CH, c = u % CH, j = t * kCtTile + row, slot = cslot[j];
      const size_t at = ((((size_t)(slot >> page_shift) * Hkv + g) << page_shift) + (slot & mask)) * D + c * 8;
      cp_async_16(to + ct_at(row, c), src + at, j < nc ? 16 : 0);
    }
  };
  if (w < nt) load_tile(K, kbuf, w);
  cp_async_commit();
  if (w < nt) load_tile(V, vbuf, w);
  cp_async_commit();
  // this thread's sequence: keys above floor are selected, and where ties are only partly in (some), those equal
  // to edge among the first cut candidates
  uint32_t edge = 0xffffffffu, floor = 0xffffffffu;
  int cut = 0;
  bool some = false;
  if (s < B) {
    const int4 rec = rows[(size_t)s * H + h];
    edge = floor = (uint32_t)rec.y;
    cut = rec.z;
    if (cut == 0x7fffffff) floor = edge == 0u ? 0u : edge - 1u;
    else some = cut > 0;
  }
  some = __any_sync(0xffffffffu, some);
  cp_async_wait<1>();   // Q and the first K
  tc::fence_proxy_async_smem();
  __syncthreads();
  const uint64_t dq = tc::sdesc(smem_u32(sm) + S::kQ, 16, 1024), dk = tc::sdesc(kbuf, 16, 1024);
  const uint64_t dv = tc::sdesc(vbuf, kCtTile * 128, 1024);
  constexpr uint32_t idq = tc::idesc_bf16(128, kCtTile, false, false), idv = tc::idesc_bf16(128, D, false, true);
  float m = -INFINITY, l = 0.f;
  int n_pv = 0;   // products with V so far
  int i = 0;
  for (int t = w; t < nt; t += 2, ++i) {
    if (i > 0) {
      cp_async_wait<1>();   // this tile's K (its V may be on its way)
      tc::fence_proxy_async_smem();
      tc::fence_before();
      wg_sync(w);
    }
    if (r == 0) {
      tc::fence_after();
      qk_steps<0, D / 16>(tS, dq, dk, idq);
      tc::commit(&sh.s_full[w]);
    }
    __syncwarp();
    wait_all(&sh.s_full[w], i & 1, abort_flag, status, kErrTimeoutS);
    tc::fence_after();
    if (t + 2 < nt) load_tile(K, kbuf, t + 2);
    cp_async_commit();
    const int j0 = t * kCtTile + half * 64;
    const uint32_t own = tS + lanes + half * 64;   // this thread's 64 scores
    // scores of 16 keys from the k-th, of those not selected -inf
    auto scores = [&](int k, float (&z)[16]) {
      uint32_t x[16];
      tc::tmem_ld16(own + k, x);
      tc::tmem_wait_ld();
#pragma unroll
      for (int u = 0; u < 16; u += 4) {
        const uint4 key4 = *reinterpret_cast<const uint4*>(ckey + j0 + k + u);
        const float4 dl4 = *reinterpret_cast<const float4*>(cdel + j0 + k + u);
        const uint32_t key[4] = {key4.x, key4.y, key4.z, key4.w};
        const float dl[4] = {dl4.x, dl4.y, dl4.z, dl4.w};
#pragma unroll
        for (int v = 0; v < 4; ++v)
          z[u + v] = key[v] > floor ? fmaf(__uint_as_float(x[u + v]), scale, dl[v]) : -INFINITY;
        if (some)
#pragma unroll
          for (int v = 0; v < 4; ++v)
            if (key[v] == edge && key[v] != 0u && c0 + j0 + k + u + v < cut)
              z[u + v] = fmaf(__uint_as_float(x[u + v]), scale, dl[v]);
      }
    };
    float mx = m;
#pragma unroll 1
    for (int k = 0; k < 64; k += 16) {
      float z[16];
      scores(k, z);
#pragma unroll
      for (int u = 0; u < 16; u += 2) mx = fmaxf(mx, fmaxf(z[u], z[u + 1]));
    }
    // the weights' reference m moves only where a score is far above it: weights up to e^8 are as good
    float keep = 1.f;
    const bool far = mx > m + 8.f;
    if (far) {
      keep = exp_diff(m, mx);
      m = mx;
      l *= keep;
    }
    const float ref = m == -INFINITY ? 0.f : m;
    const bool rescale = i > 0 && __any_sync(0xffffffffu, far);
    // the weights over the scores, keys 2 k, 2 k + 1 of the tile in column k: the first parts in 64 columns, the
    // second behind them.  In an order that leaves scores not yet read alone: columns half * 32 + k / 2 and 64
    // behind that take what came from half * 64 + k.
#pragma unroll 1
    for (int n = 0; n < 64; n += 16) {
      const int k = half == 0 ? n : 48 - n;
      float z[16];
      scores(k, z);
      uint32_t hi[8], lo[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float p0 = exp_diff(z[2 * u], ref), p1 = exp_diff(z[2 * u + 1], ref);
        l += p0 + p1;
        hi[u] = pack_bf16x2(p0, p1);
        lo[u] = pack_bf16x2(p0 - __uint_as_float(hi[u] << 16), p1 - __uint_as_float(hi[u] & 0xffff0000u));
      }
      tc::tmem_st8(tS + lanes + half * 32 + (k >> 1), hi);
      tc::tmem_st8(tS + lanes + 64 + half * 32 + (k >> 1), lo);
    }
    {
      uint32_t zero[32];
#pragma unroll
      for (int u = 0; u < 32; ++u) zero[u] = 0u;
      tc::tmem_st32(tS + lanes + (half ^ 1) * 32, zero);
      tc::tmem_st32(tS + lanes + 64 + (half ^ 1) * 32, zero);
    }
    if (rescale) {   // O is complete: the last product has been waited for
#pragma unroll 1
      for (int c = 0; c < D; c += 16) {
        uint32_t o[16];
        tc::tmem_ld16(tO + lanes + c, o);
        tc::tmem_wait_ld();
#pragma unroll
        for (int u = 0; u < 16; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * keep);
        tc::tmem_st16(tO + lanes + c, o);
      }
    }
    tc::tmem_wait_st();
    cp_async_wait<1>();   // this tile's V (the next K may be on its way)
    {
      // an exponent of all ones in what this thread copied
      uint32_t bits = 0u;
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const int u = r + k * 128;
        const uint4 v = *reinterpret_cast<const uint4*>(sm + (vbuf - smem_u32(sm)) + ct_at(u / CH, u % CH));
        bits |= ((v.x & 0x7f807f80u) + 0x00800080u) | ((v.y & 0x7f807f80u) + 0x00800080u) |
                ((v.z & 0x7f807f80u) + 0x00800080u) | ((v.w & 0x7f807f80u) + 0x00800080u);
      }
      if ((bits & 0x80008000u) != 0u) sh.odd[w] = 1;
    }
    tc::fence_proxy_async_smem();
    tc::fence_before();
    wg_sync(w);
    if (*reinterpret_cast<volatile int*>(&sh.odd[w]) == 0) {
      if (r == 0) {
        tc::fence_after();
        pv_steps<0, kCtTile / 16>(tO, tS, dv, idv, i > 0 ? 1u : 0u);
        pv_steps<0, kCtTile / 16>(tO, tS + 64, dv, idv, 1u);
        tc::commit(&sh.pv_done[w]);
      }
      __syncwarp();
      wait_all(&sh.pv_done[w], n_pv & 1, abort_flag, status, kErrTimeoutPV);
      tc::fence_after();
      ++n_pv;
    } else {
      tc::fence_after();
      const unsigned char* vrow = sm + (vbuf - smem_u32(sm));
#pragma unroll 1
      for (int c = 0; c < D; c += 8) {
        uint32_t o[16];   // 8 columns used
#pragma unroll
        for (int u = 0; u < 8; ++u) o[u] = 0u;
        if (i > 0) {
          tc::tmem_ld16(tO + lanes + (c < D - 16 ? c : D - 16), o);
          tc::tmem_wait_ld();
          if (c == D - 8)
#pragma unroll
            for (int u = 0; u < 8; ++u) o[u] = o[u + 8];
        }
#pragma unroll 1
        for (int k0 = 0; k0 < 64; k0 += 32) {
          uint32_t hi[16], lo[16];
          tc::tmem_ld16(tS + lanes + half * 32 + (k0 >> 1), hi);
          tc::tmem_ld16(tS + lanes + 64 + half * 32 + (k0 >> 1), lo);
          tc::tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const uint32_t hw = (k & 1) ? hi[k >> 1] & 0xffff0000u : hi[k >> 1] << 16;
            const uint32_t lw = (k & 1) ? lo[k >> 1] & 0xffff0000u : lo[k >> 1] << 16;
            const float p = __uint_as_float(hw) + __uint_as_float(lw);
            const uint4 v = *reinterpret_cast<const uint4*>(vrow + ct_at(half * 64 + k0 + k, c / 8));
            const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
            if (p != 0.f) {
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const float v0 = __uint_as_float(vw[u] << 16), v1 = __uint_as_float(vw[u] & 0xffff0000u);
                o[2 * u] = __float_as_uint(fmaf(p, v0, __uint_as_float(o[2 * u])));
                o[2 * u + 1] = __float_as_uint(fmaf(p, v1, __uint_as_float(o[2 * u + 1])));
              }
            }
          }
        }
        uint32_t out8[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) out8[u] = o[u];
        tc::tmem_st8(tO + lanes + c, out8);
      }
      tc::tmem_wait_st();
      tc::fence_before();
      wg_sync(w);   // all have read the flag and the tile
      if (r == 0) sh.odd[w] = 0;
    }
    if (t + 2 < nt) load_tile(V, vbuf, t + 2);
    cp_async_commit();
  }
  cp_async_wait<0>();
  if (*abort_flag) {   // a wait has given up: no product may be under way when the columns are freed
    if (r == 0) {
      tc::commit(&sh.drain[w]);
      drain_wait(&sh.drain[w], 0);
    }
    __syncwarp();
  }
  // the four results of a sequence (two warpgroups, two halves of their tiles) side by side in the tiles' place
  gm[w * 2 + half][r & 63] = m;
  gl[w * 2 + half][r & 63] = l;
  __syncthreads();
  float M = -INFINITY;
#pragma unroll
  for (int q = 0; q < 4; ++q) M = fmaxf(M, gm[q][r & 63]);
  float* res = reinterpret_cast<float*>(sm);   // [4][64][D + 4]
  {
    float* mine = res + tid * (D + 4);
    // no tile of this warpgroup: nothing
    const float f = exp_diff(m, M == -INFINITY ? 0.f : M);
#pragma unroll 1
    for (int c = 0; c < D; c += 16) {
      uint32_t o[16];
      tc::tmem_ld16(tO + lanes + c, o);
      tc::tmem_wait_ld();
#pragma unroll
      for (int u = 0; u < 16; u += 4) {
        float v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = i > 0 ? __uint_as_float(o[u + q]) * f : 0.f;
        *reinterpret_cast<float4*>(mine + c + u) = make_float4(v[0], v[1], v[2], v[3]);
      }
    }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == 0) tc::tmem_dealloc(tmem, 512);
  float* out = part + ((size_t)s0 * H + h) * n_part * (D + 4) + (size_t)blockIdx.x * (D + 4);
  const size_t step = (size_t)H * n_part * (D + 4);   // from sequence to sequence
#pragma unroll 2
  for (int k = 0; k < 64 * (D / 4) / kCtThreads; ++k) {
    const int u = tid + k * kCtThreads, q = u / (D / 4), c = u % (D / 4) * 4;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const float4 v = *reinterpret_cast<const float4*>(res + (p * 64 + q) * (D + 4) + c);
      a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
    }
    if (s0 + q < B) *reinterpret_cast<float4*>(out + q * step + c) = a;
  }
  if (tid < 64 && s < B) {
    float sum = 0.f;
#pragma unroll
    for (int p = 0; p < 4; ++p) sum = fmaf(gl[p][tid], exp_diff(gm[p][tid], M == -INFINITY ? 0.f : M), sum);
    *reinterpret_cast<float2*>(out + tid * step + D) = make_float2(M, sum);
  }
}

template <int D> cudaError_t launch_d(const PagedPlan& P, const void* Q, void* ws, cudaStream_t s) {
  const cudaError_t e = ensure_smem_limit(paged_cand_tc_kernel<D>, CtSmem<D>::kBytes);
  if (e != cudaSuccess) return e;
  return launch_after(paged_cand_tc_kernel<D>, dim3(P.n_psplit, P.H, (P.B + 63) / 64), kCtThreads, CtSmem<D>::kBytes, s,
                      1, (const uint16_t*)Q, (const uint16_t*)P.K, (const uint16_t*)P.V, ws_ptr<int4>(ws, P.off_rows),
                      ws_ptr<int32_t>(ws, P.off_crow), ws_ptr<int2>(ws, P.off_cent), ws_ptr<float>(ws, P.off_part),
                      ws_ptr<int32_t>(ws, P.off_status), P.B, P.H, P.Hkv, P.page_shift, P.n_pages << P.page_shift,
                      P.cand_len, P.cand_split, P.n_psplit + P.n_split, P.scale);
}

}  // namespace

cudaError_t launch_paged_cand_tc(const PagedPlan& P, const void* Q, void* ws, cudaStream_t s) {
  return P.d == 128 ? launch_d<128>(P, Q, ws, s) : launch_d<64>(P, Q, ws, s);
}

}  // namespace dma
