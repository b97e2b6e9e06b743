// Top-w selection of every row (sequence, head) over the paged gate values.
//
// A row of n values is split over a cluster of C CTAs, each of which keeps its part in shared memory as
// order keys: the values are read once.  The edge (the key of the last place) is found by counting, from
// the row's smallest to its largest key, 2048 equal intervals at a time: the interval that holds the edge
// is split again, so that three rounds settle any 32-bit keys and values that lie close together (gate
// values do: exp of something near 0) still spread over all counters.  The counters of a cluster are
// summed through distributed shared memory.  Then each warp counts the selected keys of its own stretch,
// and writes them behind those of the stretches before it: the list comes out in ascending position, ties
// to the lower position, without sorting.
//
// With a shared prefix the same kernel first selects the prefix's best w for each head (the candidates),
// then takes each row's best w of (candidates, the row's own positions behind the prefix): the best of a
// union are among the best of its parts, and delta does not depend on the query.
#include <cooperative_groups.h>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace dma {
namespace {

constexpr int kPsThreads = 512;
constexpr int kPsWarps = kPsThreads / 32;
constexpr int kPsBins = 2048;
constexpr int kPsMaxCluster = 8;

enum SelMode { kRows, kCandidates, kRest };   // a whole row; the prefix, per head; candidates + the rest

// What the CTAs of a cluster tell each other.
struct PsShared {
  uint32_t kmin, kmax;
  int valid, bad;
  int4 count;   // keys above and at the edge among the candidates, above and at the edge behind them
};

template <SelMode M>
__global__ void __launch_bounds__(kPsThreads)
paged_select_kernel(PagedPlan P, int32_t* __restrict__ rows, int32_t* __restrict__ sel, int2* __restrict__ ent,
                    int32_t* __restrict__ crow, int32_t* __restrict__ cand, int2* __restrict__ cent,
                    int32_t* __restrict__ counters, int32_t* __restrict__ status, int cap) {
  extern __shared__ __align__(16) uint32_t keys[];   // [cap] this CTA's stretch, as far as it fits
  __shared__ __align__(16) int hist[2][kPsBins];
  __shared__ PsShared sh;
  __shared__ int wsum[kPsWarps][4];
  __shared__ int found_bin, found_above;
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int row = blockIdx.y, h = M == kCandidates ? row : row % P.H, b = M == kCandidates ? 0 : row / P.H;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int W = row_window(P.w_heads, h, P.H, P.w);
  const int page = 1 << P.page_shift;
  const int32_t* tab = P.table + (size_t)b * P.max_pages;

  // ---- the row: indices [0, n1) candidates, [n1, n1p) nothing, [n1p, n) positions base + (i - n1p)
  const int base = M == kRest ? P.prefix : 0;
  int n1 = 0, len = M == kCandidates ? P.prefix : __ldg(P.lens + b);
  bool bad = false;
  if (M == kRest) {
    n1 = crow[h];
    if (n1 < 0) { bad = true; n1 = 0; }
  }
  if (len > P.N || (len > 0 && len < (M == kCandidates ? 0 : P.prefix))) bad = true;
  const bool idle = len <= 0 || bad;
  const int n1p = (n1 + 3) & ~3;
  const int n = idle ? 0 : n1p + (len - base);
  const int seg = ((n + C - 1) / C + 3) & ~3;
  const int i0 = min(rank * seg, n), i1 = min(i0 + seg, n), ns = i1 - i0;
  const int2* ce = M == kRest ? cent + (size_t)h * P.cand_len : nullptr;

  // order keys of indices i .. i + 3 (i a multiple of 4); 0 where there is nothing
  auto load4 = [&](int i) -> uint4 {
    uint4 k = make_uint4(0u, 0u, 0u, 0u);
    uint32_t* kk = &k.x;
    if (M == kRest && i < n1p) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (i + u < n1) kk[u] = order_key(__int_as_float(ce[i + u].y));
      return k;
    }
    const int pos = base + i - n1p;
    const int pg = __ldg(tab + (pos >> P.page_shift));
    if (pg < 0 || pg >= P.n_pages) {
      bad = true;
      return k;
    }
    const float4 f = *reinterpret_cast<const float4*>(P.delta + (((size_t)pg * P.H + h) << P.page_shift) +
                                                      (pos & (page - 1)));
    k.x = order_key(f.x);
    if (i + 1 < n) k.y = order_key(f.y);
    if (i + 2 < n) k.z = order_key(f.z);
    if (i + 3 < n) k.w = order_key(f.w);
    return k;
  };
  const int res = min(ns, cap);   // resident part; what lies behind it is read again in every round
  auto key_at = [&](int i) -> uint32_t {
    if (i < res) return keys[i];
    const uint4 k = load4((i0 + i) & ~3);
    const int u = (i0 + i) & 3;
    return u == 0 ? k.x : u == 1 ? k.y : u == 2 ? k.z : k.w;
  };

  // ---- read the stretch once: keys, smallest, largest, how many
  if (tid == 0) {
    sh.kmin = 0xffffffffu;
    sh.kmax = 0u;
    sh.valid = 0;
    sh.bad = 0;
  }
  __syncthreads();
  uint32_t kmin = 0xffffffffu, kmax = 0u;
  int valid = 0;
  auto note = [&](uint32_t k) {
    if (k != 0u) {
      kmin = min(kmin, k);
      kmax = max(kmax, k);
      ++valid;
    }
  };
  {
    constexpr int kU = 4;   // 16-byte loads of a thread in flight
    for (int q0 = tid; q0 * 4 < ns; q0 += kPsThreads * kU) {
      uint4 k[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int i = (q0 + u * kPsThreads) * 4;
        k[u] = i < ns ? load4(i0 + i) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int i = (q0 + u * kPsThreads) * 4;
        if (i < cap) *reinterpret_cast<uint4*>(keys + i) = k[u];
        note(k[u].x); note(k[u].y); note(k[u].z); note(k[u].w);
      }
    }
  }
  kmin = __reduce_min_sync(0xffffffffu, kmin);
  kmax = __reduce_max_sync(0xffffffffu, kmax);
  valid = __reduce_add_sync(0xffffffffu, valid);
  const bool wbad = __any_sync(0xffffffffu, bad);
  if (lane == 0) {
    atomicMin(&sh.kmin, kmin);
    atomicMax(&sh.kmax, kmax);
    atomicAdd(&sh.valid, valid);
    if (wbad) sh.bad = 1;
  }
  for (int i = tid; i < 2 * kPsBins; i += kPsThreads) (&hist[0][0])[i] = 0;
  cl.sync();
  valid = 0;
  bad = false;
  for (int r = 0; r < C; ++r) {
    const PsShared* o = cl.map_shared_rank(&sh, r);
    kmin = r == 0 ? o->kmin : min(kmin, o->kmin);
    kmax = r == 0 ? o->kmax : max(kmax, o->kmax);
    valid += o->valid;
    bad = bad || o->bad != 0;
  }
  if (tid == 0 && rank == 0) {
    if (M != kCandidates) counters[row] = 0;
    if (bad) atomicOr(status, kPagedErr);
  }

  // ---- the edge T: keys above it are in, `need` of those equal to it, lowest positions first
  uint32_t T = 0u;
  int need = 0;
  if (!bad && valid > W) {
    uint32_t lo = kmin, span = 0xffffffffu;   // the edge lies in [lo, lo + span]
    int above = 0;                            // keys above that interval
    const uint32_t range = kmax - kmin;
    int shift = range == 0u ? 0 : max(0, 21 - __clz(range));
    if (range == 0u) T = kmin;
    for (int round = 0; range != 0u; ++round) {
      int* hs = hist[round & 1];
      if (round >= 2) {
        for (int i = tid; i < kPsBins; i += kPsThreads) hs[i] = 0;   // all have read it: they synced since
        __syncthreads();
      }
      for (int i = tid; i < ns; i += kPsThreads) {
        const uint32_t k = key_at(i);
        if (k >= lo && k - lo <= span) atomicAdd(&hs[(k - lo) >> shift], 1);
      }
      cl.sync();
      // thread t sums counters 4t' .. 4t'+3 over the cluster, from the top: t' = 511 - t
      const int b4 = (kPsThreads - 1 - tid) * 4;
      int4 c = make_int4(0, 0, 0, 0);
      for (int r = 0; r < C; ++r) {
        const int4 o = *reinterpret_cast<const int4*>(cl.map_shared_rank(hs + b4, r));
        c.x += o.x; c.y += o.y; c.z += o.z; c.w += o.w;
      }
      const int mine = c.x + c.y + c.z + c.w;
      int incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (lane == 31) wsum[warp][0] = incl;
      __syncthreads();
      int before = above;
      for (int w = 0; w < warp; ++w) before += wsum[w][0];
      const int excl = before + incl - mine;
      if (excl < W && excl + mine >= W) {   // one thread of the block
        int bin = b4 + 3, up = excl;
        const int cc[4] = {c.w, c.z, c.y, c.x};
#pragma unroll
        for (int u = 0; u < 3; ++u)
          if (bin == b4 + 3 - u && up + cc[u] < W) {
            up += cc[u];
            --bin;
          }
        found_bin = bin;
        found_above = up;
      }
      __syncthreads();
      above = found_above;
      lo += (uint32_t)found_bin << shift;
      if (shift == 0) {
        T = lo;
        break;
      }
      span = (1u << shift) - 1u;
      shift = max(0, shift - 11);
    }
    need = W - above;
  }
  if (bad || idle) T = 0xffffffffu;

  // ---- counts of this CTA's warps: contiguous stretches of whole 32s
  const int per = ((ns + kPsWarps - 1) / kPsWarps + 31) & ~31;
  const int j0 = min(warp * per, ns), j1 = min(j0 + per, ns);
  int cnt[4] = {0, 0, 0, 0};   // as PsShared::count
  if (!bad)
    for (int j = j0 + lane; j < j1; j += 32) {
      const uint32_t k = key_at(j);
      const int at = M == kRest && i0 + j < n1p ? 0 : 2;
      cnt[at] += k > T;
      cnt[at + 1] += k == T && k != 0u;
    }
#pragma unroll
  for (int u = 0; u < 4; ++u) cnt[u] = __reduce_add_sync(0xffffffffu, cnt[u]);
  if (lane == 0) {
#pragma unroll
    for (int u = 0; u < 4; ++u) wsum[warp][u] = cnt[u];
  }
  __syncthreads();
  if (tid < 4) {
    int s = 0;
    for (int w = 0; w < kPsWarps; ++w) s += wsum[w][tid];
    reinterpret_cast<int*>(&sh.count)[tid] = s;
  }
  cl.sync();
  int all[4] = {0, 0, 0, 0}, mine[4] = {0, 0, 0, 0};   // over the cluster; before this warp
  for (int r = 0; r < C; ++r) {
    const int4 o = cl.map_shared_rank(&sh, r)->count;
    const int oc[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      all[u] += oc[u];
      if (r < rank) mine[u] += oc[u];
    }
  }
  for (int w = 0; w < warp; ++w)
#pragma unroll
    for (int u = 0; u < 4; ++u) mine[u] += wsum[w][u];
  const int ties_c = min(need, all[1]);   // ties taken among the candidates
  int32_t* rec = M == kCandidates ? crow + h : rows + (size_t)row * 4;
  if (rank == 0 && tid == 0) {
    const int listed = all[2] + min(need, all[1] + all[3]) - ties_c;
    if (M == kCandidates) {
      rec[0] = bad ? -1 : listed;
    } else {
      rec[0] = bad ? 0 : listed;
      rec[1] = (int32_t)T;
      if (bad || idle) rec[2] = 0;
      else if (ties_c == all[1]) rec[2] = 0x7fffffff;   // else the warp that holds the last tie taken writes it
      rec[3] = bad ? 0 : all[0] + ties_c;
    }
  }

  // ---- the list
  if (!bad) {
    int eq = mine[1] + mine[3];                            // ties before this warp's keys
    int out = mine[2] + max(0, min(need, eq) - ties_c);    // listed keys before them
    int32_t* lp = M == kCandidates ? cand + (size_t)h * P.cand_len : sel + (size_t)row * P.sel_len;
    int2* le = M == kCandidates ? cent + (size_t)h * P.cand_len : ent + (size_t)row * P.sel_len;
    const unsigned lt = (1u << lane) - 1u;
    for (int j = j0; j < j1; j += 32) {
      const int i = i0 + j + lane;
      const uint32_t k = j + lane < j1 ? key_at(j + lane) : 0u;
      const bool is_eq = k == T && k != 0u;
      const unsigned em = __ballot_sync(0xffffffffu, is_eq);
      const int tie = eq + __popc(em & lt);
      const bool take = k > T || (is_eq && tie < need);
      if (M == kRest && is_eq && i < n1p && tie == need - 1 && ties_c < all[1]) rec[2] = i + 1;
      const bool list = take && !(M == kRest && i < n1p);
      const unsigned lm = __ballot_sync(0xffffffffu, list);
      if (list) {
        const int at = out + __popc(lm & lt), pos = base + i - n1p;
        const int slot = (__ldg(tab + (pos >> P.page_shift)) << P.page_shift) + (pos & (page - 1));
        lp[at] = pos;
        le[at] = make_int2(slot, (int)((k & 0x80000000u) ? k ^ 0x80000000u : ~k));
      }
      eq += __popc(em);
      out += __popc(lm);
    }
  }
  cl.sync();   // no CTA leaves while another may still read its shared memory
}

// Launches the selection of `n_rows` rows of at most n values.  Clusters: stretches of at most 16384
// values (64 KB, three CTAs an SM), and for few rows as many CTAs as give every SM one, down to stretches
// of 2048.
template <SelMode M>
cudaError_t launch_select(const PagedPlan& P, int n_rows, int n, void* ws, cudaStream_t s) {
  int C = 1;
  const int sms = sm_count();
  while (C < kPsMaxCluster && ((n + C - 1) / C > 16384 || (n_rows * C < sms && (n + C - 1) / C > 2048))) C *= 2;
  int cap = (((n + C - 1) / C + 3) & ~3) + 4;
  if (cap > 49152) cap = 49152;
  const size_t smem = (size_t)cap * 4;
  const cudaError_t e = ensure_smem_limit(paged_select_kernel<M>, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(C, n_rows);
  cfg.blockDim = dim3(kPsThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_select_kernel<M>, P, ws_ptr<int32_t>(ws, P.off_rows),
                            ws_ptr<int32_t>(ws, P.off_sel), ws_ptr<int2>(ws, P.off_ent),
                            ws_ptr<int32_t>(ws, P.off_crow), ws_ptr<int32_t>(ws, P.off_cand),
                            ws_ptr<int2>(ws, P.off_cent), ws_ptr<int32_t>(ws, P.off_count),
                            ws_ptr<int32_t>(ws, P.off_status), cap);
}

}  // namespace

cudaError_t launch_paged_topk(const PagedPlan& P, void* ws, cudaStream_t s) {
  if (!P.shared) return launch_select<kRows>(P, P.B * P.H, P.N, ws, s);
  const cudaError_t e = launch_select<kCandidates>(P, P.H, P.prefix, ws, s);
  if (e != cudaSuccess) return e;
  return launch_select<kRest>(P, P.B * P.H, ((P.cand_len + 3) & ~3) + P.N - P.prefix, ws, s);
}

}  // namespace dma
