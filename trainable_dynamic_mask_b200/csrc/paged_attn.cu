// Single-query attention over the keys that paged_topk.cu selected.
//
// s_j = q . k_j scale + delta_j for the selected j; o = softmax(s) V; LSE = ln sum_j exp(s_j).  Scores
// stay in natural units (exponents are taken of differences from the running maximum), so that values of
// delta near the end of float32's range neither overflow nor lose the LSE.
//
// paged_list_kernel takes a row's own list.  The rows it needs lie anywhere in the cache, so what bounds
// it is how many 256-byte reads are in flight: a group of d / 8 lanes handles one key at a time (K and V
// row, 16 bytes a lane), and the rows of the next keys are always on their way into a ring of shared
// memory.  Every lane reads back just what it copied itself, so nothing waits for another warp before the
// end.  Each group keeps its own running maximum and sum; they meet once per CTA.
// paged_cand_kernel (shared prefix) multiplies all sequences' queries of a head with the head's
// candidates, a sequence's selection being a comparison of the candidate's delta with the edge of its row.
// Few sequences or few candidates give the tensor cores little to do and CTAs of 128 rows little to share:
// 16 x 64 score tiles of warp-level products; the others go to paged_cand_tc.cu.
// The partial results (m, l, o) of a row are joined, in a fixed order, by the CTA of its list that
// finishes last.
#include <utility>

#include "rows.cuh"

namespace dma {
namespace {

// A slot of the cache; what the selection wrote always is one, a workspace it has not been run on may hold
// anything, which must not be followed.
DMA_DEVINL int inside(int slot, int n_slots) { return (unsigned)slot < (unsigned)n_slots ? slot : 0; }

// Writes the row's output from its sums: nothing kept: 0 and -inf; a NaN stays.
template <typename T> DMA_DEVINL void put_channel(T* O, float o, float l) {
  store_from_f32(O, l > 0.f ? o / l : (l == 0.f ? 0.f : l));
}
DMA_DEVINL void put_lse(float* LSE, float m, float l) {
  *LSE = l > 0.f ? m + logf(l) : (l == 0.f ? -INFINITY : l);
}

// Joins n partial results (o[D], m, l) with a row's running o (this thread's V channels from c), m and l.
template <int D, int V> DMA_DEVINL void join(const float* part, int n, int c, float& m, float& l, float (&o)[V]) {
  float big = m;
  for (int i = 0; i < n; ++i) big = fmaxf(big, __ldcg(part + (size_t)i * (D + 4) + D));
  const float ref = big == -INFINITY ? 0.f : big;
  const float w0 = exp_diff(m, ref);
  l *= w0;
#pragma unroll
  for (int u = 0; u < V; ++u) o[u] *= w0;
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float* p = part + (size_t)i * (D + 4);
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(p + D));
    float v[V];
    if constexpr (V == 4) {
      const float4 q = __ldcg(reinterpret_cast<const float4*>(p + c));
      v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
    } else if constexpr (V == 2) {
      const float2 q = __ldcg(reinterpret_cast<const float2*>(p + c));
      v[0] = q.x; v[1] = q.y;
    } else {
      v[0] = __ldcg(p + c);
    }
    const float w = exp_diff(ml.x, ref);
    l = fmaf(ml.y, w, l);
#pragma unroll
    for (int u = 0; u < V; ++u) o[u] = fmaf(v[u], w, o[u]);
  }
  m = big;
}

// Three stages on their way of 4 keys a group (K and V: 48 KB of a CTA of 128 threads, four of which share an
// SM).  2048 keys for each of 256 queries, 268 MB of 256-byte rows anywhere in 2 GB, take 50 us (5.3 TB/s, 81 % of the
// copy rate); with two stages or four 1 us more.
constexpr int kPlStages = 3;

template <typename T> constexpr int list_keys() { return sizeof(T) == 2 ? 4 : 2; }   // keys of a group and stage
// bytes of the ring: stages x keys x (K, V) x eight channels of every thread
template <typename T, int NT> constexpr int list_smem() { return kPlStages * list_keys<T>() * 2 * 8 * sizeof(T) * NT; }

// NT threads: 128, or one warp where the lists are short (behind a shared prefix), many of which then share
// an SM.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(NT, 512 / NT)
paged_list_kernel(const T* Q, const T* K, const T* V, const int4* rows, const int2* ent, float* part,
                  int32_t* counters, T* __restrict__ O, float* __restrict__ LSE, int H, int Hkv,
                  int page_shift, int n_slots, int sel_len, int n_split, int n_psplit, float scale) {
  constexpr int L = D / 8, RPW = 32 / L, NG = (NT / 32) * RPW;   // lanes of a row; groups of a warp, of the CTA
  constexpr int U = list_keys<T>(), NP = sizeof(T) / 2;         // 16-byte pieces of a lane's eight channels
  constexpr int E = kPagedSplit / NG / L;                       // entries of a lane
  static_assert(list_smem<T, NT>() >= NG * D * 4, "the ring's place takes the groups' results at the end");
  extern __shared__ __align__(128) unsigned char ring[];
  float* so = reinterpret_cast<float*>(ring);   // [NG][D], when the ring is done with
  __shared__ float sm[NG], sl[NG];
  __shared__ int last;
  const int row = blockIdx.y, h = row % H, g = h / (H / Hkv);
  const int tid = threadIdx.x, lane = tid & 31, grp = tid / L, e = (lane % L) * 8;
  pdl_trigger();
  pdl_wait();
  const int count = min(rows[row].x, sel_len);
  const int k0 = blockIdx.x * kPagedSplit, nk = min(count - k0, kPagedSplit);
  if (nk <= 0 && blockIdx.x > 0) return;   // the first CTA of a row works even if there is nothing
  // the group's keys: k0 + j NG + grp; lane i of it holds the entries of j = i, i + L, ..
  const int2* list = ent + (size_t)row * sel_len + k0;
  int2 en[E];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int k = (lane % L + i * L) * NG + grp;
    en[i] = make_int2(0, 0);
    if (k < nk) en[i] = list[k];
    en[i].x = inside(en[i].x, n_slots);
  }
  // the entry of the group's key j
  auto entry = [&](int j) {
    int2 v = en[0];
#pragma unroll
    for (int i = 1; i < E; ++i)
      if (j / L == i) v = en[i];
    return make_int2(__shfl_sync(0xffffffffu, v.x, j % L, L), __shfl_sync(0xffffffffu, v.y, j % L, L));
  };
  const int mask = (1 << page_shift) - 1;
  const uint32_t mine = smem_u32(ring) + tid * 16;
  auto issue = [&](int st) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = st * U + u, n = j * NG + grp < nk ? 16 : 0;
      const int slot = entry(j).x;
      const size_t at = (((((size_t)(slot >> page_shift) * Hkv + g) << page_shift) + (slot & mask)) * D) + e;
      const uint32_t to = mine + (((st % kPlStages) * U + u) * 2 * NP) * NT * 16;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        cp_async_16(to + i * NT * 16, K + at + i * 4, n);
        cp_async_16(to + (NP + i) * NT * 16, V + at + i * 4, n);
      }
    }
  };
  const int ns = nk > 0 ? ((nk + NG - 1) / NG + U - 1) / U : 0;
#pragma unroll
  for (int st = 0; st < kPlStages - 1; ++st) {
    if (st < ns) issue(st);
    cp_async_commit();
  }
  float q[8];
  widen8(load_raw8(Q + (size_t)row * D + e), q);
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] *= scale;
  float m = -INFINITY, l = 0.f, acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  for (int st = 0; st < ns; ++st) {
    if (st + kPlStages - 1 < ns) issue(st + kPlStages - 1);
    cp_async_commit();
    cp_async_wait<kPlStages - 1>();
    const unsigned char* from = ring + tid * 16 + ((st % kPlStages) * U * 2 * NP) * NT * 16;
    float x[U], mx = m;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      Raw8<T> raw;
#pragma unroll
      for (int i = 0; i < NP; ++i)
        reinterpret_cast<uint4*>(&raw)[i] =
            *reinterpret_cast<const uint4*>(from + (u * 2 * NP + i) * NT * 16);
      float k[8], s = 0.f;
      widen8(raw, k);
#pragma unroll
      for (int i = 0; i < 8; ++i) s = fmaf(k[i], q[i], s);
      s = row_sum<L>(s);
      const int j = st * U + u;
      const float dl = __int_as_float(entry(j).y);
      x[u] = j * NG + grp < nk ? s + dl : -INFINITY;
      mx = fmaxf(mx, x[u]);
    }
    const float ref = mx == -INFINITY ? 0.f : mx;
    const float keep = exp_diff(m, ref);
    m = mx;
    l *= keep;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] *= keep;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      Raw8<T> raw;
#pragma unroll
      for (int i = 0; i < NP; ++i)
        reinterpret_cast<uint4*>(&raw)[i] =
            *reinterpret_cast<const uint4*>(from + (u * 2 * NP + NP + i) * NT * 16);
      const float p = exp_diff(x[u], ref);
      float v[8];
      widen8(raw, v);
      l += p;
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = fmaf(p, v[i], acc[i]);
    }
  }
  __syncthreads();   // every lane is done with the ring
#pragma unroll
  for (int i = 0; i < 8; ++i) so[grp * D + e + i] = acc[i];
  if (lane % L == 0) {
    sm[grp] = m;
    sl[grp] = l;
  }
  __syncthreads();
  const int n_act = count > 0 ? (count + kPagedSplit - 1) / kPagedSplit : 1;
  constexpr int VC = D / NT > 1 ? D / NT : 1;   // channels of a thread
  const int c = tid * VC;
  float M = sm[0];
#pragma unroll
  for (int i = 1; i < NG; ++i) M = fmaxf(M, sm[i]);
  float lsum = 0.f, o[VC];
  {
    const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
    for (int u = 0; u < VC; ++u) o[u] = 0.f;
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      const float w = exp_diff(sm[i], ref);
      lsum = fmaf(sl[i], w, lsum);
      if (c < D)
#pragma unroll
        for (int u = 0; u < VC; ++u) o[u] = fmaf(so[i * D + c + u], w, o[u]);
    }
  }
  float* prow = part + (size_t)row * (n_psplit + n_split) * (D + 4);
  int others = n_psplit;   // partial results to join
  if (n_act > 1) {
    float* out = prow + (size_t)(n_psplit + blockIdx.x) * (D + 4);
    if (c < D)
#pragma unroll
      for (int u = 0; u < VC; ++u) out[c + u] = o[u];
    if (tid == 0) {
      out[D] = M;
      out[D + 1] = lsum;
    }
    __threadfence();
    __syncthreads();
    if (tid == 0) {
      last = atomicAdd(counters + row, 1) == n_act - 1;
      if (last) counters[row] = 0;   // as the next call expects it
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    // all of them in their order, this CTA's among them
    others = n_psplit + n_act;
    M = -INFINITY;
    lsum = 0.f;
#pragma unroll
    for (int u = 0; u < VC; ++u) o[u] = 0.f;
  }
  if (c >= D) return;
  if (others > 0) join<D, VC>(prow, others, c, M, lsum, o);
#pragma unroll
  for (int u = 0; u < VC; ++u) put_channel(O + (size_t)row * D + c + u, o[u], lsum);
  if (c == 0) put_lse(LSE + row, M == -INFINITY ? 0.f : M, lsum);
}

// ---------------------------------------------------------------- shared prefix

constexpr int kPcTile = 64;    // candidates of a pipeline stage
constexpr int kPcMost = 256;   // candidates of a CTA at most

template <int D> constexpr int cand_smem() { return (32 + 4 * kPcTile) * D * 2; }   // Q, 2 x (K, V)

// ldmatrix (and its transposing form) at a constant offset from a lane's address.
template <int OFF> DMA_DEVINL void ldm4(uint32_t at, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4 + %5];\n"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(at), "n"(OFF));
}
template <int OFF> DMA_DEVINL void ldm4t(uint32_t at, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4 + %5];\n"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(at), "n"(OFF));
}
// f(0) .. f(N - 1), each with its number as a constant
template <int... I, typename F> DMA_DEVINL void each_of(std::integer_sequence<int, I...>, F f) {
  (f(std::integral_constant<int, I>()), ...);
}
template <int N, typename F> DMA_DEVINL void each(F f) { each_of(std::make_integer_sequence<int, N>(), f); }

// CTA = (part of a head's candidates, head, 16 R sequences), R = 1 or 2.  Its 4 R warps are R groups of 16
// sequences times 4 groups of keys.  Tiles of 64 candidates' K and V rows are gathered with 16-byte asynchronous
// copies (swizzled by row, conflict-free for ldmatrix), one tile ahead.  A weight is split into two bf16 parts, both
// multiplied with V: one part alone would round every weight to 8 bits, as much as the output's own rounding.
// A candidate that a sequence did not select has weight exactly 0 there; if its V row holds an infinity or
// NaN, 0 times that would still spoil the sum, so a tile with such a value is added up in plain
// arithmetic that leaves weights of 0 out.
template <int R> constexpr int cand_threads() { return R == 1 ? 128 : 256; }

template <int D, int R>
__global__ void __launch_bounds__(cand_threads<R>(), 2)
paged_cand_kernel(const uint16_t* Q, const uint16_t* K, const uint16_t* V, const int4* rows, const int32_t* crow,
                  const int2* cent, float* __restrict__ part, int B, int H, int Hkv, int page_shift, int n_slots,
                  int cand_len, int cand_split, int n_part, float scale) {
  constexpr int kPcThreads = cand_threads<R>(), kPcWarps = kPcThreads / 32;
  constexpr int CH = D / 8, KG = kPcWarps / R, NT = 8 / KG, NO = D / 8;   // NT, NO: 8-wide tiles of keys, channels
  extern __shared__ __align__(128) unsigned char csm[];
  uint16_t* Qs = reinterpret_cast<uint16_t*>(csm);   // [16 R][D]
  uint16_t* Ks = Qs + 32 * D;                        // [2][64][D]
  uint16_t* Vs = Ks + 2 * kPcTile * D;               // [2][64][D]
  __shared__ __align__(8) uint32_t ckey[kPcMost];
  __shared__ __align__(8) float cdel[kPcMost];
  __shared__ int cslot[kPcMost];
  __shared__ float gm[kPcWarps][16], gl[kPcWarps][16];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.y, g = h / (H / Hkv), s0 = blockIdx.z * 16 * R;
  const int rg = warp / KG, kg = warp % KG;
  const int c0 = blockIdx.x * cand_split;
  pdl_trigger();
  pdl_wait();
  const int nc = max(0, min(crow[h], min(cand_len, c0 + cand_split)) - c0);
  const int nt = (nc + kPcTile - 1) / kPcTile;
  for (int i = tid; i < nt * kPcTile; i += kPcThreads) {
    int2 e = make_int2(0, 0);
    if (i < nc) e = cent[(size_t)h * cand_len + c0 + i];
    cslot[i] = inside(e.x, n_slots);
    cdel[i] = __int_as_float(e.y);
    ckey[i] = i < nc ? order_key(__int_as_float(e.y)) : 0u;
  }
  for (int u = tid; u < 16 * R * CH; u += kPcThreads) {
    const int r = u / CH, c = u % CH;
    const bool in = s0 + r < B;
    cp_async_16(smem_u32(Qs) + swz(r, c, CH), Q + ((size_t)(in ? s0 + r : 0) * H + h) * D + c * 8, in ? 16 : 0);
  }
  __syncthreads();
  const int mask = (1 << page_shift) - 1;
  auto load_tile = [&](int t) {
    const uint32_t kd = smem_u32(Ks + (t & 1) * kPcTile * D), vd = smem_u32(Vs + (t & 1) * kPcTile * D);
#pragma unroll
    for (int i = 0; i < kPcTile * CH / kPcThreads; ++i) {
      const int u = tid + i * kPcThreads, r = u / CH, c = u % CH, j = t * kPcTile + r, slot = cslot[j];
      const size_t at = ((((size_t)(slot >> page_shift) * Hkv + g) << page_shift) + (slot & mask)) * D + c * 8;
      const int n = j < nc ? 16 : 0;
      cp_async_16(kd + swz(r, c, CH), K + at, n);
      cp_async_16(vd + swz(r, c, CH), V + at, n);
    }
  };
  if (nt > 0) load_tile(0);
  cp_async_commit();
  // this lane's two sequences, s0 + 16 rg + lane / 4 and 8 behind it: keys above floor are selected, and where
  // ties are only partly in (some), those equal to edge among the first cut candidates
  uint32_t edge[2], floor[2];
  int cut[2];
  bool some = false;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int s = s0 + rg * 16 + (lane >> 2) + r * 8;
    edge[r] = floor[r] = 0xffffffffu;
    cut[r] = 0;
    if (s < B) {
      const int4 rec = rows[(size_t)s * H + h];
      edge[r] = floor[r] = (uint32_t)rec.y;
      cut[r] = rec.z;
      if (rec.z == 0x7fffffff) floor[r] = edge[r] == 0u ? 0u : edge[r] - 1u;
      else some = some || rec.z > 0;
    }
  }
  some = __any_sync(0xffffffffu, some);
  // addresses of ldmatrix: row and swizzle of a lane do not change from step to step, chunk 2 k of a row being
  // an exclusive or away from chunk 0
  const uint32_t qa = smem_u32(Qs) + (rg * 16 + (lane & 15)) * (CH * 16), qx = ((lane >> 4) ^ (lane & 7)) * 16;
  const int key0 = kg * (kPcTile / KG);   // this warp's keys of a tile
  const uint32_t ka = smem_u32(Ks) + (key0 + (lane & 7) + (lane >> 4) * 8) * (CH * 16);
  const uint32_t kx = (((lane >> 3) & 1) ^ (lane & 7)) * 16;
  const uint32_t va = smem_u32(Vs) + (key0 + (lane & 15)) * (CH * 16);
  float o[NO][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int n = 0; n < NO; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) o[n][i] = 0.f;
  for (int t = 0; t < nt; ++t) {
    if (t + 1 < nt) load_tile(t + 1);
    cp_async_commit();
    cp_async_wait<1>();
    __syncthreads();
    const uint32_t kb = ka + (t & 1) * kPcTile * D * 2, vb = va + (t & 1) * kPcTile * D * 2;
    // an exponent of all ones anywhere in the V tile
    uint32_t odd = 0u;
    {
      const uint4* vp = reinterpret_cast<const uint4*>(Vs + (t & 1) * kPcTile * D);
#pragma unroll
      for (int i = 0; i < kPcTile * CH / kPcThreads; ++i) {
        const uint4 w = vp[tid + i * kPcThreads];
        odd |= ((w.x & 0x7f807f80u) + 0x00800080u) | ((w.y & 0x7f807f80u) + 0x00800080u) |
               ((w.z & 0x7f807f80u) + 0x00800080u) | ((w.w & 0x7f807f80u) + 0x00800080u);
      }
    }
    const bool plain = __syncthreads_or((odd & 0x80008000u) != 0u);
    float x[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) x[n][i] = 0.f;
    each<D / 16>([&](auto k) {
      uint32_t qf[4];
      ldm4<0>(qa + (qx ^ (k * 32)), qf[0], qf[1], qf[2], qf[3]);
      each<NT / 2>([&](auto n) {
        uint32_t b0, b1, b2, b3;
        ldm4<n * 16 * CH * 16>(kb + (kx ^ (k * 32)), b0, b1, b2, b3);
        mma_bf16_16816(x[2 * n], qf, b0, b1);
        mma_bf16_16816(x[2 * n + 1], qf, b2, b3);
      });
    });
    float mx[2] = {m[0], m[1]};
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int j = t * kPcTile + key0 + n * 8 + 2 * (lane & 3);
      const uint2 key = *reinterpret_cast<const uint2*>(ckey + j);
      const float2 dl = *reinterpret_cast<const float2*>(cdel + j);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = i >> 1;
        const uint32_t k = (i & 1) ? key.y : key.x;
        bool take = k > floor[r];
        if (some) take = take || (k == edge[r] && k != 0u && c0 + j + (i & 1) < cut[r]);
        x[n][i] = take ? fmaf(x[n][i], scale, (i & 1) ? dl.y : dl.x) : -INFINITY;
        mx[r] = fmaxf(mx[r], x[n][i]);
      }
    }
    // the weights' reference m moves only where a score is far above it: weights up to e^8 are as good
    float ref[2];
    bool far = false;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
      mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
      far = far || mx[r] > m[r] + 8.f;
    }
    if (__any_sync(0xffffffffu, far)) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float keep = exp_diff(m[r], mx[r] == -INFINITY ? 0.f : mx[r]);
        m[r] = mx[r];
        l[r] *= keep;
#pragma unroll
        for (int n = 0; n < NO; ++n) {
          o[n][2 * r] *= keep;
          o[n][2 * r + 1] *= keep;
        }
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) ref[r] = m[r] == -INFINITY ? 0.f : m[r];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[n][i] = exp_diff(x[n][i], ref[i >> 1]);
        l[i >> 1] += x[n][i];
      }
    if (!plain) {
      each<NT / 2>([&](auto k) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p0 = x[2 * k + (i >> 1)][(i & 1) * 2], p1 = x[2 * k + (i >> 1)][(i & 1) * 2 + 1];
          hi[i] = pack_bf16x2(p0, p1);
          lo[i] = pack_bf16x2(p0 - __uint_as_float(hi[i] << 16), p1 - __uint_as_float(hi[i] & 0xffff0000u));
        }
        each<NO / 2>([&](auto n) {
          uint32_t b0, b1, b2, b3;
          ldm4t<k * 16 * CH * 16>(vb + (qx ^ (n * 32)), b0, b1, b2, b3);
          mma_bf16_16816(o[2 * n], hi, b0, b1);
          mma_bf16_16816(o[2 * n + 1], hi, b2, b3);
          mma_bf16_16816(o[2 * n], lo, b0, b1);
          mma_bf16_16816(o[2 * n + 1], lo, b2, b3);
        });
      });
    } else {
      const unsigned char* vrow = reinterpret_cast<const unsigned char*>(Vs + (t & 1) * kPcTile * D);
#pragma unroll
      for (int n8 = 0; n8 < NT; ++n8)
#pragma unroll 1
      for (int j8 = 0; j8 < 8; ++j8) {
        // weights of key j: in register j % 2 of lane (j % 8) / 2 of each quad
        const int j = n8 * 8 + j8, src = (lane & ~3) | (j8 >> 1);
        const float p0 = __shfl_sync(0xffffffffu, (j8 & 1) ? x[n8][1] : x[n8][0], src);
        const float p1 = __shfl_sync(0xffffffffu, (j8 & 1) ? x[n8][3] : x[n8][2], src);
#pragma unroll
        for (int n = 0; n < NO; ++n) {
          const uint32_t w = *reinterpret_cast<const uint32_t*>(vrow + swz(key0 + j, n, CH) + (lane & 3) * 4);
          const float v0 = __uint_as_float(w << 16), v1 = __uint_as_float(w & 0xffff0000u);
          if (p0 != 0.f) {
            o[n][0] = fmaf(p0, v0, o[n][0]);
            o[n][1] = fmaf(p0, v1, o[n][1]);
          }
          if (p1 != 0.f) {
            o[n][2] = fmaf(p1, v0, o[n][2]);
            o[n][3] = fmaf(p1, v1, o[n][3]);
          }
        }
      }
    }
    __syncthreads();   // the tile's buffers may be filled again
  }
  cp_async_wait<0>();
  __syncthreads();
  // the warps' results side by side in the tiles' place, the key groups of a sequence joined
  float* os = reinterpret_cast<float*>(Ks);   // [warps][16][D]
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    const int i = (lane >> 2) + r * 8;
    if ((lane & 3) == 0) {
      gm[warp][i] = m[r];
      gl[warp][i] = l[r];
    }
#pragma unroll
    for (int n = 0; n < NO; ++n)
      *reinterpret_cast<float2*>(os + (warp * 16 + i) * D + n * 8 + 2 * (lane & 3)) =
          make_float2(o[n][2 * r], o[n][2 * r + 1]);
  }
  __syncthreads();
  for (int u = tid; u < 16 * R * (D / 4); u += kPcThreads) {
    const int r = u / (D / 4), c = u % (D / 4) * 4, w0 = (r >> 4) * KG, i = r & 15;
    if (s0 + r >= B) continue;
    float M = -INFINITY;
#pragma unroll
    for (int q = 0; q < KG; ++q) M = fmaxf(M, gm[w0 + q][i]);
    const float ref = M == -INFINITY ? 0.f : M;
    float sum = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int q = 0; q < KG; ++q) {
      const float w = exp_diff(gm[w0 + q][i], ref);
      const float4 v = *reinterpret_cast<const float4*>(os + ((w0 + q) * 16 + i) * D + c);
      sum = fmaf(gl[w0 + q][i], w, sum);
      a.x = fmaf(v.x, w, a.x); a.y = fmaf(v.y, w, a.y); a.z = fmaf(v.z, w, a.z); a.w = fmaf(v.w, w, a.w);
    }
    float* out = part + (((size_t)(s0 + r) * H + h) * n_part + blockIdx.x) * (D + 4);
    if (c == 0) *reinterpret_cast<float2*>(out + D) = make_float2(M, sum);
    *reinterpret_cast<float4*>(out + c) = a;
  }
}

template <int D, int R>
cudaError_t launch_cand(const PagedPlan& P, const void* Q, void* ws, cudaStream_t s) {
  const cudaError_t e = ensure_smem_limit(paged_cand_kernel<D, R>, cand_smem<D>());
  if (e != cudaSuccess) return e;
  return launch_after(
      paged_cand_kernel<D, R>, dim3(P.n_psplit, P.H, (P.B + 16 * R - 1) / (16 * R)), cand_threads<R>(), cand_smem<D>(),
      s, 1, (const uint16_t*)Q, (const uint16_t*)P.K, (const uint16_t*)P.V, ws_ptr<int4>(ws, P.off_rows),
      ws_ptr<int32_t>(ws, P.off_crow), ws_ptr<int2>(ws, P.off_cent), ws_ptr<float>(ws, P.off_part), P.B, P.H, P.Hkv,
      P.page_shift, P.n_pages << P.page_shift, P.cand_len, P.cand_split, P.n_psplit + P.n_split, P.scale);
}

template <int D>
cudaError_t launch_cand_rows(const PagedPlan& P, const void* Q, void* ws, cudaStream_t s) {
  if (P.cand_tc) return launch_paged_cand_tc(P, Q, ws, s);
  return P.B <= 16 ? launch_cand<D, 1>(P, Q, ws, s) : launch_cand<D, 2>(P, Q, ws, s);
}

template <typename T, int D, int NT>
cudaError_t launch_list_t(const PagedPlan& P, const void* Q, void* ws, void* O, float* LSE, cudaStream_t s) {
  const cudaError_t e = ensure_smem_limit(paged_list_kernel<T, D, NT>, list_smem<T, NT>());
  if (e != cudaSuccess) return e;
  return launch_after(
      paged_list_kernel<T, D, NT>, dim3(P.n_split, P.B * P.H), NT, list_smem<T, NT>(), s, 1, (const T*)Q, (const T*)P.K,
      (const T*)P.V, ws_ptr<int4>(ws, P.off_rows), ws_ptr<int2>(ws, P.off_ent), ws_ptr<float>(ws, P.off_part),
      ws_ptr<int32_t>(ws, P.off_count), (T*)O, LSE, P.H, P.Hkv, P.page_shift, P.n_pages << P.page_shift, P.sel_len,
      P.n_split, P.n_psplit, P.scale);
}

template <typename T, int D>
cudaError_t launch_list(const PagedPlan& P, const void* Q, void* ws, void* O, float* LSE, cudaStream_t s) {
  // Behind a shared prefix a row lists about w (N - prefix) / N keys; one warp is enough for few of them, if there are
  // rows enough to fill the GPU with such CTAs.  The attention of 2048 rows, with one warp and with 128 threads, at
  // some 8 keys a row 21.7 us and 28.3, 14 33.6 and 38.6, 42 38.8 and 41.4, 48 34.6 and 34.0, 56 36.8 and 34.6, 64 47.1
  // and 44.7; of rows of 16 keys, 512 17.8 and 14.1, 1024 20.9 and 20.8, 1280 21.7 and 24.0.
  if (P.shared && P.B * P.H >= 8 * sm_count() && (int64_t)P.w * (P.N - P.prefix) <= (int64_t)48 * P.N)
    return launch_list_t<T, D, 32>(P, Q, ws, O, LSE, s);
  return launch_list_t<T, D, 128>(P, Q, ws, O, LSE, s);
}

}  // namespace

cudaError_t launch_paged_attn(const PagedPlan& P, const void* Q, void* ws, void* O, float* LSE, cudaStream_t s) {
  if (P.shared) {
    const cudaError_t e = P.d == 128 ? launch_cand_rows<128>(P, Q, ws, s) : launch_cand_rows<64>(P, Q, ws, s);
    if (e != cudaSuccess) return e;
  }
  if (P.bf16)
    return P.d == 128 ? launch_list<uint16_t, 128>(P, Q, ws, O, LSE, s)
                      : launch_list<uint16_t, 64>(P, Q, ws, O, LSE, s);
  return P.d == 128 ? launch_list<float, 128>(P, Q, ws, O, LSE, s) : launch_list<float, 64>(P, Q, ws, O, LSE, s);
}

}  // namespace dma
