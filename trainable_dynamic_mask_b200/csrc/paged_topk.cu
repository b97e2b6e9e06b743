// Top-w selection of every row (sequence, head) over the paged gate values.
//
// A row of n values is split over a cluster of C CTAs, each of which keeps its part in shared memory as
// order keys: the values are read once.  The edge (the key of the last place) is found by counting: the
// interval from the row's smallest to its largest key is cut into 4 counters a thread (gate values lie
// close together, so they spread over counters where fixed digits of the key would not), the counters of
// the cluster are summed through distributed shared memory, and the keys of the counter that holds the
// edge, a few dozen as a rule, are ranked against each other.  Where ties leave more of them than threads,
// that counter's interval is cut again; four rounds settle any keys.  Then each warp counts the selected
// keys of its own stretch, and writes them behind those of the stretches before it: the list comes out in
// ascending position, ties to the lower position, without sorting.
//
// Long rows in large numbers (SIEVE) are not kept: the first reading only keeps the maxima of groups of 8
// keys.  The w-th largest maximum is a lower bound of the edge, and with at least 2 w groups a close one:
// only the groups that reach it are read again (from L2 by then), and little more than w keys are left for
// the steps above.  All of that compares plain floats, and one key in 8 is counted: shared-memory atomics
// are what counting costs.
//
// With a shared prefix the same kernel first selects the prefix's best w for each head (the candidates),
// then takes each row's best w of (candidates, the row's own positions behind the prefix): the best of a
// union are among the best of its parts, and delta does not depend on the query.  Few of a row's own keys
// pass the last candidate, as a rule; they compete with as many of the last candidates, which are kept in
// order for that (rest_by_tail), and only where they are more is the row counted like any other.
//
// The bytes are one reading of the gate values; what bounds a row is the chain of its steps (page numbers,
// values, counters, the edge's interval, the list), each a wait of a microsecond, and the instructions of the
// rows that share an SM (58 % of the issue slots for 768 rows of up to 8192 values).  A CTA passes through
// most of its code once, so instructions that have to come from memory first are a part of that chain: loops
// over the resident keys are not unrolled and clusters of up to 4 have a kernel of their own, which takes 4 us
// off a selection of 20 (8 sequences behind a prefix of 2048).  Measured, the kernel alone: 8 sequences of 65536
// values, 32 heads, window 2048 (67 MB): 36 us, of which the first reading 13.5 (5 TB/s); without the sieve 95.  48
// sequences of up to 8192 values, 16 heads (12.6 MB): 24 us.  A prefix of 32768 values, 32 heads: candidates 16 us, 64
// sequences' own keys behind it 9 (25 more without rest_by_tail).  All of that with P.N the longest length: the
// variants below are chosen by P.N, since lengths are not known when a kernel is launched.
#include <cooperative_groups.h>

#include <type_traits>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace dma {
namespace {

constexpr int kPsMaxCluster = 8;
constexpr int kPsGroup = 8;           // sieve: keys of a maximum
constexpr int kPsMaxBatches = 512;    // 32 groups that a warp reads again together
// Rows are taken longest first where there are more CTAs than places (1024 threads an SM, whatever the CTA's size),
// so that no long one begins last.  Each CTA works the order out for itself, B lengths for each of B sequences.
// With 16 heads, in order and not: lengths up to 8192, 24 sequences 17.4 us and 18.1, 48 23.6 and 25.2, 80 34.0 and
// 33.3, 128 53.9 and 49.2; up to 4096, 64 17.6 and 18.5, 80 20.4 and 21.2, 96 25.4 and 24.8, 256 104 and 50.  Where all
// have a place at once (8 sequences) it gives nothing: 10.8 and 10.6.
constexpr int kPsMostOrdered = 80;

using Yes = std::integral_constant<bool, true>;
using No = std::integral_constant<bool, false>;

enum SelMode { kRows, kCandidates, kRest };   // a whole row; the prefix, per head; candidates + the rest

// What the CTAs of a cluster tell each other.
struct PsShared {
  uint32_t kmin, kmax;
  int valid, bad;
  int4 count;    // keys above and at the edge among the candidates, above and at the edge behind them
  int members;   // keys in the interval being ranked
};

// Sum of x over the warps before this one, and over all of them (NW <= 32 warps; x alike in a warp).
template <int NW> DMA_DEVINL int2 warps_before(int x, int* buf) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) buf[warp] = x;
  __syncthreads();
  int v = lane < NW ? buf[lane] : 0;
  const int own = v;
#pragma unroll
  for (int o = 1; o < NW; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  return make_int2(__shfl_sync(0xffffffffu, v - own, warp), __shfl_sync(0xffffffffu, v, NW - 1));
}

// Sorts the last in the order of selection (small key, then high position) first.
DMA_DEVINL uint64_t last_first(uint32_t key, uint32_t position) { return (uint64_t)key << 32 | (uint32_t)~position; }

// A row's selection where all w candidates would fill it and at most kPagedTail - 1 of its own keys pass the
// last of them: each of those m keys and of the last m candidates is in unless m of these 2 m come after it.
// keys, where: room for kPagedTail; false (for the whole block): not that simple, nothing written.
template <int NT>
DMA_DEVINL bool rest_by_tail(const PagedPlan& P, const int32_t* tab, int h, int len, int W, int n1, const int2* tail,
                             uint32_t* keys, int* where, int* buf, int4* rec, int32_t* lp, int2* le, bool& bad) {
  const int tid = threadIdx.x, lane = tid & 31, page = 1 << P.page_shift;
  const int known = tail[kPagedTail].x;
  if (n1 < W || known <= 0) return false;
  const uint32_t last = (uint32_t)tail[0].x;
  const float* head = P.delta + ((size_t)h << P.page_shift);
  int m = 0;   // keys that pass so far
  for (int p0 = P.prefix; p0 < len; p0 += NT * 4) {
    const int pos = p0 + tid * 4;
    uint32_t k[4] = {0u, 0u, 0u, 0u};
    bool wrong = false;
    if (pos < len) {
      const int pg = tab[pos >> P.page_shift];
      wrong = pg < 0 || pg >= P.n_pages;
      if (!wrong) {
        const float4 f = *reinterpret_cast<const float4*>(head + ((size_t)(unsigned)(pg * P.H) << P.page_shift) +
                                                          (pos & (page - 1)));
        k[0] = order_key(f.x);
        if (pos + 1 < len) k[1] = order_key(f.y);
        if (pos + 2 < len) k[2] = order_key(f.z);
        if (pos + 3 < len) k[3] = order_key(f.w);
      }
    }
    unsigned own = 0u;
#pragma unroll
    for (int u = 0; u < 4; ++u) own |= k[u] > last ? 1u << u : 0u;   // a tie goes to the candidate
    int incl = __popc(own);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const int2 w = warps_before<NT / 32>(__shfl_sync(0xffffffffu, incl, 31), buf);
    int at = m + w.x + incl - __popc(own);
    m += w.y;
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (own >> u & 1u) {
        if (at < kPagedTail) {
          keys[at] = k[u];
          where[at] = pos + u;
        }
        ++at;
      }
    if (__syncthreads_or(wrong)) {
      bad = true;
      return false;
    }
    if (m >= known) return false;
  }
  // survivors: threads 0 .. m - 1; the last m candidates: threads 64 .. 64 + m - 1
  int after = 0;
  if (tid < m) {
    const uint32_t k = keys[tid];
#pragma unroll 4
    for (int i = 0; i < m; ++i)
      after += (int)(last_first(keys[i], i) < last_first(k, tid)) + (int)((uint32_t)tail[i].x < k);
  } else if (tid >= 64 && tid < 64 + m) {
    const uint32_t k = (uint32_t)tail[tid - 64].x;
    after = tid - 64;
    for (int i = 0; i < m; ++i) after += keys[i] <= k;
  }
  const bool in = after >= m;
  const int out_c = __syncthreads_count(tid >= 64 && tid < 64 + m && !in);   // candidates that give way
  const unsigned mine = __ballot_sync(0xffffffffu, tid < m && in);
  if (lane == 0 && tid < 64) buf[tid >> 5] = __popc(mine);
  __syncthreads();
  if (tid < m && in) {
    const int at = (tid >= 32 ? buf[0] : 0) + __popc(mine & ((1u << lane) - 1u));
    const int pos = where[tid], pg = tab[pos >> P.page_shift];
    const uint32_t k = keys[tid];
    lp[at] = pos;
    le[at] = make_int2((pg << P.page_shift) + (pos & (page - 1)), (int)((k & 0x80000000u) ? k ^ 0x80000000u : ~k));
  }
  if (tid == 0) {
    // a cut only where the last to give way ties with the first that stays
    const int2 stays = tail[out_c];
    const bool tie = out_c > 0 && tail[max(out_c - 1, 0)].x == stays.x;
    *rec = make_int4(out_c, stays.x, tie ? stays.y + 1 : 0x7fffffff, W - out_c);
  }
  return true;
}

// MC: CTAs of a cluster at most.
template <SelMode M, int NT, bool SIEVE, int MC>
__global__ void __launch_bounds__(NT, NT == 512 ? 2 : NT == 256 ? 4 : 8)
paged_select_kernel(PagedPlan P, int32_t* __restrict__ rows, int32_t* __restrict__ sel, int2* __restrict__ ent,
                    int32_t* crow, int32_t* __restrict__ cand, int2* cent, int2* tail, int32_t* __restrict__ counters,
                    int32_t* __restrict__ status, int cap, int page_cap, int list_cap, bool longest_first) {
  constexpr int NW = NT / 32, BINS = 4 * NT, LB = NT == 512 ? 11 : NT == 256 ? 10 : 9;
  static_assert(BINS == 1 << LB, "four counters a thread");
  static_assert(!SIEVE || M == kRows, "candidates and their rest are short or few");
  extern __shared__ __align__(16) uint32_t keys[];   // [cap] this CTA's stretch, as far as it fits
  int* pages = reinterpret_cast<int*>(keys + cap);   // [page_cap] the stretch's pages
  __shared__ __align__(16) int hist[BINS];
  __shared__ uint32_t list[NT], every[NT];
  __shared__ __align__(16) int mhist[SIEVE ? BINS : 4];
  __shared__ PsShared sh, msh;
  __shared__ int2 batch[SIEVE ? kPsMaxBatches : 1];       // {first, number} in the list
  __shared__ int2 batch_in[SIEVE ? kPsMaxBatches : 1];    // keys above and at the edge, then those in front
  __shared__ int listed_total;
  __shared__ int wbuf[5][NW];
  __shared__ int found_bin, found_above, found_count, other_bin, other_above;
  __shared__ uint32_t found_key;
  cg::cluster_group cl = cg::this_cluster();
  constexpr int kMost = MC;
  constexpr bool CL = MC > 1;
  const int C = CL ? (int)cl.num_blocks() : 1, rank = CL ? (int)cl.block_rank() : 0;
  auto all_sync = [&]() {
    if (CL) cl.sync();
    else __syncthreads();
  };
  // p in the shared memory of CTA r of the cluster
  auto of = [&](auto* p, int r) { return CL ? cl.map_shared_rank(p, r) : p; };
  const int h = M == kCandidates ? blockIdx.y : blockIdx.y % P.H;
  int b = M == kCandidates ? 0 : blockIdx.y / P.H;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_trigger();
  pdl_wait();
  if (M == kRows && longest_first) {
    // this CTA's sequence: the one of that place in the order of lengths, the longest first
    __shared__ int place;
    const int want = b;
    if (tid == 0) place = want;
    __syncthreads();
    for (int t = tid; t < P.B; t += NT) {
      const int n = P.lens[t];
      int before = 0;
#pragma unroll 8
      for (int u = 0; u < P.B; ++u) {
        const int o = P.lens[u];
        before += o > n || (o == n && u < t);
      }
      if (before == want) place = t;
    }
    __syncthreads();
    b = place;
  }
  const int row = M == kCandidates ? h : b * P.H + h;
  const int W = row_window(P.w_heads, h, P.H, P.w);
  const int page = 1 << P.page_shift;
  const int32_t* tab = P.table + (size_t)b * P.max_pages;

  // ---- the row: indices [0, n1) candidates, [n1, n1p) nothing, [n1p, n) positions base + (i - n1p)
  const int base = M == kRest ? P.prefix : 0;
  int n1 = 0, len = M == kCandidates ? P.prefix : P.lens[b];
  bool bad = false;
  if (M == kRest) {
    n1 = crow[h];
    if (n1 < 0) { bad = true; n1 = 0; }
  }
  if (len > P.N || (len > 0 && len < (M == kCandidates ? 0 : P.prefix))) bad = true;
  const bool idle = len <= 0 || bad;
  if constexpr (M == kRest && !CL) {
    if (!idle && rest_by_tail<NT>(P, tab, h, len, W, n1, tail + (size_t)h * (kPagedTail + 1), list,
                                  reinterpret_cast<int*>(every), wbuf[0], reinterpret_cast<int4*>(rows) + row,
                                  sel + (size_t)row * P.sel_len, ent + (size_t)row * P.sel_len, bad)) {
      if (tid == 0) counters[row] = 0;
      return;
    }
    __syncthreads();
  }
  const int n1p = (n1 + 3) & ~3;
  const int n = idle ? 0 : n1p + (len - base);
  const int seg = CL ? ((n + C - 1) / C + 3) & ~3 : n;
  const int i0 = min(rank * seg, n), i1 = min(i0 + seg, n), ns = i1 - i0;
  const int2* ce = M == kRest ? cent + (size_t)h * P.cand_len : nullptr;
  // what the steps after the first reading work on: the stretch (the first `res` keys resident, what lies
  // behind them is read again in every round), or, sieved, a list of keys and their indices
  int items = ns, res = min(ns, cap);
  bool sieved = false;
  const int tab0 = (base + max(i0 - n1p, 0)) >> P.page_shift;
  const int np = i1 > n1p && i1 > i0 ? ((base + i1 - 1 - n1p) >> P.page_shift) - tab0 + 1 : 0;
  for (int i = tid; i < min(np, page_cap); i += NT) {
    int pg = tab[tab0 + i];
    if (pg < 0 || pg >= P.n_pages) {
      bad = true;
      pg = 0;
    }
    pages[i] = pg;
  }
  if (tid == 0) {
    sh.kmin = 0xffffffffu;
    sh.kmax = 0u;
    sh.valid = 0;
    sh.bad = 0;
    sh.members = 0;
    msh = sh;
    listed_total = 0;
    found_bin = found_above = found_count = other_bin = other_above = 0;
    found_key = 0u;
  }
  *reinterpret_cast<int4*>(hist + 4 * tid) = make_int4(0, 0, 0, 0);
  if (SIEVE) *reinterpret_cast<int4*>(mhist + 4 * tid) = make_int4(0, 0, 0, 0);
  __syncthreads();
  auto page_of = [&](int pos) -> int {
    const int i = (pos >> P.page_shift) - tab0;
    if (i < page_cap) return pages[i];
    int pg = tab[tab0 + i];
    if (pg < 0 || pg >= P.n_pages) {
      bad = true;
      pg = 0;
    }
    return pg;
  };
  auto slot_of = [&](int pos) -> int { return (page_of(pos) << P.page_shift) + (pos & (page - 1)); };
  // values of this head, of page pg
  const float* head = P.delta + ((size_t)h << P.page_shift);
  auto values_of = [&](int pg) { return head + ((size_t)(unsigned)(pg * P.H) << P.page_shift); };   // n_pages H < 2^31
  auto value4 = [&](int pos) -> float4 {
    return *reinterpret_cast<const float4*>(values_of(page_of(pos)) + (pos & (page - 1)));
  };
  // order keys of indices i .. i + 3 (i a multiple of 4); 0 where there is nothing
  auto load4 = [&](int i) -> uint4 {
    uint4 k = make_uint4(0u, 0u, 0u, 0u);
    if (M == kRest && i < n1p) {
      if (i < n1) k.x = order_key(__int_as_float(ce[i].y));
      if (i + 1 < n1) k.y = order_key(__int_as_float(ce[i + 1].y));
      if (i + 2 < n1) k.z = order_key(__int_as_float(ce[i + 2].y));
      if (i + 3 < n1) k.w = order_key(__int_as_float(ce[i + 3].y));
      return k;
    }
    const int pos = base + i - n1p;
    const float4 f = value4(pos);
    k.x = order_key(f.x);
    if (i + 1 < n) k.y = order_key(f.y);
    if (i + 2 < n) k.z = order_key(f.z);
    if (i + 3 < n) k.w = order_key(f.w);
    return k;
  };
  // fn(key) for every key of the stretch, in no particular order
  auto for_keys = [&](auto fn) {
#pragma unroll 1
    for (int i = tid * 4; i < res; i += NT * 4) {
      const uint4 k = *reinterpret_cast<const uint4*>(keys + i);
      fn(k.x); fn(k.y); fn(k.z); fn(k.w);
    }
    for (int i = cap + tid * 4; i < items; i += NT * 4) {
      const uint4 k = load4(i0 + i);
      fn(k.x); fn(k.y); fn(k.z); fn(k.w);
    }
  };

  // the counter (of 4 NT, summed over the cluster) that holds the want-th largest key, `above` keys lying
  // above all of them: found_bin, found_above, found_count; and (other > 0) the one that holds the other-th:
  // other_bin, other_above
  auto find_bin = [&](int* counts, int above, int want, int* buf, int other = 0) {
    // thread t sums counters 4 t' .. 4 t' + 3, t' = NT - 1 - t: from the top
    const int b4 = (NT - 1 - tid) * 4;
    int4 c = make_int4(0, 0, 0, 0);
    {
      int4 o[kMost];
#pragma unroll
      for (int r = 0; r < kMost; ++r)
        o[r] = r < C ? *reinterpret_cast<const int4*>(of(counts + b4, r)) : make_int4(0, 0, 0, 0);
#pragma unroll
      for (int r = 0; r < kMost; ++r) {
        c.x += o[r].x; c.y += o[r].y; c.z += o[r].z; c.w += o[r].w;
      }
    }
    const int mine = c.x + c.y + c.z + c.w;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const int excl = above + warps_before<NW>(__shfl_sync(0xffffffffu, incl, 31), buf).x + incl - mine;
    auto within = [&](int k, int& bin, int& up, int& here) {   // the counter of this thread that holds the k-th
      bin = b4 + 3;
      up = excl;
      here = c.w;
      const int cc[3] = {c.z, c.y, c.x};
#pragma unroll
      for (int u = 0; u < 3; ++u)
        if (up + here < k) {
          up += here;
          here = cc[u];
          --bin;
        }
    };
    int bin, up, here;
    if (excl < want && excl + mine >= want) {   // one thread of the block
      within(want, bin, up, here);
      found_bin = bin;
      found_above = up;
      found_count = here;
    }
    if (M == kCandidates && excl < other && excl + mine >= other) {
      within(other, bin, up, here);
      other_bin = bin;
      other_above = up;
    }
    __syncthreads();
  };
  // a thread's smallest key - 1 (0 wraps to the largest), largest and number -> the cluster's smallest,
  // largest and number; and whether any thread of it met a bad page
  auto publish = [&](PsShared& to, uint32_t& kmin, uint32_t& kmax, int& valid) {
    kmin = __reduce_min_sync(0xffffffffu, kmin);
    kmax = __reduce_max_sync(0xffffffffu, kmax);
    valid = __reduce_add_sync(0xffffffffu, valid);
    const bool wbad = __any_sync(0xffffffffu, bad);
    if (lane == 0) {
      atomicMin(&to.kmin, kmin);
      atomicMax(&to.kmax, kmax);
      atomicAdd(&to.valid, valid);
      if (wbad) to.bad = 1;
    }
    all_sync();
    PsShared o[kMost];
#pragma unroll
    for (int r = 0; r < kMost; ++r)
      if (r < C) {
        const PsShared* q = of(&to, r);
        o[r].kmin = q->kmin; o[r].kmax = q->kmax; o[r].valid = q->valid; o[r].bad = q->bad;
      }
    kmin = o[0].kmin; kmax = o[0].kmax; valid = o[0].valid; bad = o[0].bad != 0;
#pragma unroll
    for (int r = 1; r < kMost; ++r)
      if (r < C) {
        kmin = min(kmin, o[r].kmin);
        kmax = max(kmax, o[r].kmax);
        valid += o[r].valid;
        bad = bad || o[r].bad != 0;
      }
    ++kmin;
  };
  constexpr int kU = 8;   // 16-byte loads of a thread in flight
  uint32_t kmin = 0xffffffffu, kmax = 0u;
  int valid = 0;
  auto note = [&](uint32_t k) {
    kmin = min(kmin, k - 1u);
    kmax = max(kmax, k);
    valid += k != 0u;
  };

  // ---- sieve
  int* index = reinterpret_cast<int*>(keys + list_cap);                       // beside the list's keys
  uint16_t* again = reinterpret_cast<uint16_t*>(keys + 2 * list_cap);         // [list_cap] groups to read again
  int nb = 0;                                                                 // batches of the list, 512 at most
  if (SIEVE && n >= 2 * kPsGroup * W) {
    float* maxima = reinterpret_cast<float*>(keys);   // where the list will be
    const float nothing = __int_as_float(0x7fffffff);
    // values at i .. i + 3 of the stretch; a NaN where there is none (it passes no comparison)
    auto values4 = [&](int i) -> float4 {
      if (i >= ns) return make_float4(nothing, nothing, nothing, nothing);
      float4 f = value4(i0 + i);
      if (i + 1 >= ns) f.y = nothing;
      if (i + 2 >= ns) f.z = nothing;
      if (i + 3 >= ns) f.w = nothing;
      return f;
    };
    static_assert(kU * 128 == 1024, "a warp's chunk below: every maximum of it is written");
    float fmin = INFINITY, fmax = -INFINITY;
    for (int c0 = warp * 1024; c0 < ns; c0 += NW * 1024) {   // 1024 neighbouring keys of a warp
      float4 f[kU];
      const int i = c0 + lane * 4, pos = i0 + i;
      if (c0 + 1024 <= ns && (((i0 + c0 + 1023) >> P.page_shift) - tab0) < page_cap) {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int pu = pos + u * 128;
          f[u] = *reinterpret_cast<const float4*>(values_of(pages[(pu >> P.page_shift) - tab0]) + (pu & (page - 1)));
        }
      } else {
#pragma unroll
        for (int u = 0; u < kU; ++u) f[u] = values4(i + u * 128);
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        float m = fmaxf(fmaxf(f[u].x, f[u].y), fmaxf(f[u].z, f[u].w));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        if ((lane & 1) == 0) {
          maxima[(i + u * 128) >> 3] = m;
          valid += m == m;
        }
        fmin = fminf(fmin, m);
        fmax = fmaxf(fmax, m);
      }
    }
    if (fmin <= fmax) {
      kmin = order_key(fmin) - 1u;
      kmax = order_key(fmax);
    }
    publish(msh, kmin, kmax, valid);
    // more groups than keys wanted, or no bound
    if (!bad && valid >= W) {
      const uint32_t range = kmax - kmin;
      const int shift = range == 0u ? 0 : max(0, 32 - LB - __clz(range));
      const int ng = (ns + kPsGroup - 1) / kPsGroup;
      for (int i = tid; i < ng; i += NT) {
        const float m = maxima[i];
        if (m == m) atomicAdd(&mhist[(order_key(m) - kmin) >> shift], 1);
      }
      all_sync();
      find_bin(mhist, 0, W, wbuf[0]);
      // at least W keys are no smaller than this one
      const uint32_t lk = kmin + ((uint32_t)found_bin << shift);
      const float least = __uint_as_float((lk & 0x80000000u) ? lk ^ 0x80000000u : ~lk);
      // the groups that reach it, in order: a warp counts and writes those of its stretch
      const unsigned lt = (1u << lane) - 1u;
      const int gpw = ((ng + NW - 1) / NW + 31) & ~31, g0 = min(warp * gpw, ng), g1 = min(g0 + gpw, ng);
      int hits = 0;
#pragma unroll 4
      for (int i = g0; i < g1; i += 32)
        hits += __popc(__ballot_sync(0xffffffffu, i + lane < g1 && maxima[i + lane] >= least));
      const int2 wb = warps_before<NW>(hits, wbuf[1]);
      const int n_again = wb.y;
      const bool many = n_again > list_cap;   // many keys alike: the list would not hold them
      if (!many) {
        int at = wb.x;
#pragma unroll 4
        for (int i = g0; i < g1; i += 32) {
          const bool hit = i + lane < g1 && maxima[i + lane] >= least;
          const unsigned m = __ballot_sync(0xffffffffu, hit);
          if (hit) again[at + __popc(m & lt)] = (uint16_t)(i + lane);
          at += __popc(m);
        }
      }
      __syncthreads();
      // they are read again, 32 groups (one a lane) together: a place in the list for their keys, written there in
      // the order of positions (the places of different batches come in any order); a warp has the next batch on
      // the way while it works on one
      nb = many ? 0 : (n_again + 31) >> 5;
      auto fetch = [&](int bt, int& from, float4 (&f)[2]) {
        const int it = bt * 32 + lane;
        from = bt < nb && it < n_again ? again[it] * kPsGroup : ns;
        if (np <= page_cap) {   // as below
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int pos = i0 + min(from + u * 4, (ns - 1) & ~3);
            const float* at = values_of(pages[(pos >> P.page_shift) - tab0]);
            f[u] = *reinterpret_cast<const float4*>(at + (pos & (page - 1)));
          }
        } else {
#pragma unroll
          for (int u = 0; u < 2; ++u) f[u] = values4(from + u * 4);
        }
      };
      int from = ns, from_next;
      float4 f[2] = {}, f_next[2];
      if (nb > 0) fetch(warp, from, f);
      for (int bt = warp; bt < nb; bt += NW) {
        fetch(bt + NW, from_next, f_next);
        const int left = ns - from;   // of a whole group 8 or more
        unsigned own = (unsigned)(f[0].x >= least) | (unsigned)(f[0].y >= least) << 1 |
                       (unsigned)(f[0].z >= least) << 2 | (unsigned)(f[0].w >= least) << 3 |
                       (unsigned)(f[1].x >= least) << 4 | (unsigned)(f[1].y >= least) << 5 |
                       (unsigned)(f[1].z >= least) << 6 | (unsigned)(f[1].w >= least) << 7;
        if (left < kPsGroup) own &= left > 0 ? (1u << left) - 1u : 0u;
        const int c = __popc(own);
        int incl = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += v;
        }
        int first = 0;
        if (lane == 31) {
          first = atomicAdd(&listed_total, incl);
          batch[bt] = make_int2(first, incl);
        }
        first = __shfl_sync(0xffffffffu, first, 31);
        if (first + __shfl_sync(0xffffffffu, incl, 31) <= list_cap) {   // else many keys alike: they do not fit
          int at = first + incl - c;
          while (own != 0u) {   // nearly always one
            const int e = __ffs(own) - 1;
            const float4 q = e < 4 ? f[0] : f[1];
            const float v = (e & 3) == 0 ? q.x : (e & 3) == 1 ? q.y : (e & 3) == 2 ? q.z : q.w;
            keys[at] = order_key(v);
            index[at++] = i0 + from + e;
            own &= own - 1u;
          }
        }
        from = from_next;
        f[0] = f_next[0];
        f[1] = f_next[1];
      }
      __syncthreads();
      items = listed_total;
      if (tid == 0 && (many || items > list_cap)) sh.members = 1;
      if (items <= list_cap && tid < ((items + 3) & ~3) - items) keys[items + tid] = 0u;   // read four at a time
      // bounds of the list's keys and their number
      kmin = lk - 1u;
      valid = tid == 0 ? items : 0;
      publish(sh, kmin, kmax, valid);
      sieved = true;
      for (int r = 0; r < C; ++r) sieved = sieved && of(&sh, r)->members == 0;
    }
    if (!sieved) {
      all_sync();                          // all have seen it
      if (tid == 0) {
        sh.kmin = 0xffffffffu;
        sh.kmax = 0u;
        sh.valid = 0;
        sh.members = 0;
      }
      __syncthreads();
      items = ns;
      kmin = 0xffffffffu;
      kmax = 0u;
      valid = 0;
    } else {
      res = items;
    }
  }

  // ---- read the stretch: keys, smallest, largest, how many
  if (!SIEVE || !sieved) {
    auto keep = [&](int i, const uint4& k) {
      if (i < cap) *reinterpret_cast<uint4*>(keys + i) = k;
      note(k.x); note(k.y); note(k.z); note(k.w);
    };
    const int jc = M == kRest ? max(0, min(n1p - i0, ns)) : 0;   // candidates come first
    if (M == kRest)
      for (int i = tid * 4; i < jc; i += NT * 4) keep(i, load4(i0 + i));
    if (np <= page_cap) {
      // every page number at hand: addresses without branches, so that a thread's kU loads leave together
      for (int q0 = jc + tid * 4; q0 < ns; q0 += NT * 4 * kU) {
        float4 f[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int pos = base + i0 + min(q0 + u * NT * 4, (ns - 1) & ~3) - n1p;
          f[u] = *reinterpret_cast<const float4*>(values_of(pages[(pos >> P.page_shift) - tab0]) + (pos & (page - 1)));
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int i = q0 + u * NT * 4, left = ns - i;
          if (left > 0)
            keep(i, make_uint4(order_key(f[u].x), left > 1 ? order_key(f[u].y) : 0u, left > 2 ? order_key(f[u].z) : 0u,
                               left > 3 ? order_key(f[u].w) : 0u));
        }
      }
    } else {
      for (int i = jc + tid * 4; i < ns; i += NT * 4) keep(i, load4(i0 + i));
    }
    publish(sh, kmin, kmax, valid);
  }
  if (tid == 0 && rank == 0) {
    if (M != kCandidates) counters[row] = 0;
    if (bad) atomicOr(status, kPagedErr);
  }

  // ---- the edge T: keys above it are in, `need` of those equal to it, lowest positions first
  uint32_t T = 0u;
  int need = 0, tail_n = 0;
  uint64_t tail_end = 0u;   // candidates: the last ones' keys are below it, tail_n of them (0: not looked for)
  if (!bad && valid > W) {
    uint32_t lo = kmin, span = 0xffffffffu;   // the edge lies in [lo, lo + span]
    int above = 0;                            // keys above that interval
    const uint32_t range = kmax - kmin;
    int shift = range == 0u ? 0 : max(0, 32 - LB - __clz(range));
    T = kmin;
    while (range != 0u) {
      for_keys([&](uint32_t k) {
        if (k >= lo && k - lo <= span) atomicAdd(&hist[(k - lo) >> shift], 1);
      });
      all_sync();
      // (candidates) the first time, also the counter of the kPagedTail-th key from the edge: the last candidates
      // are those below its end
      const bool first = M == kCandidates && tail_end == 0u;
      find_bin(hist, above, W, wbuf[0], first ? max(1, W - kPagedTail + 1) : 0);
      if (first) {
        tail_n = W - other_above;
        tail_end = lo + (((uint64_t)other_bin + 1u) << shift);
      }
      above = found_above;
      lo += (uint32_t)found_bin << shift;
      T = lo;
      if (shift == 0) break;
      span = (1u << shift) - 1u;
      if (found_count <= NT) {
        // rank the interval's keys against each other
        for_keys([&](uint32_t k) {
          if (k >= lo && k - lo <= span) list[min(atomicAdd(&sh.members, 1), NT - 1)] = k;
        });
        all_sync();
        // each thread one of them: whose list it is in, and where
        int members[kMost], m = 0, from = -1, at = 0;
#pragma unroll
        for (int r = 0; r < kMost; ++r) members[r] = r < C ? of(&sh, r)->members : 0;
#pragma unroll
        for (int r = 0; r < kMost; ++r) {
          const int mr = min(members[r], NT - m);
          if (tid >= m && tid < m + mr) {
            from = r;
            at = tid - m;
          }
          m += mr;
        }
        if (from >= 0) every[tid] = *of(list + at, from);
        __syncthreads();
        if (tid < m) {
          const uint32_t k = every[tid];
          int gt = above, ge = above;
#pragma unroll 2
          for (int i = 0; i < m; ++i) {
            const uint32_t o = every[i];
            gt += o > k;
            ge += o >= k;
          }
          if (gt < W && ge >= W) {   // the edge's holders, all alike
            found_key = k;
            found_above = gt;
          }
        }
        __syncthreads();
        above = found_above;
        T = found_key;
        break;
      }
      shift = max(0, shift - LB);
      all_sync();   // every CTA has read the counters
      *reinterpret_cast<int4*>(hist + 4 * tid) = make_int4(0, 0, 0, 0);
      __syncthreads();
    }
    need = W - above;
  }
  if (bad || idle) T = 0xffffffffu;

  // ---- counts of this CTA's warps: contiguous stretches, four neighbouring keys a lane
  const int per = ((items + NW - 1) / NW + 127) & ~127;
  const int j0 = min(warp * per, items), j1 = min(j0 + per, items);
  int cnt[4] = {0, 0, 0, 0};   // as PsShared::count
  if (SIEVE && sieved) {
    // batches instead of stretches
    for (int bt = warp; bt < nb; bt += NW) {
      const int2 bb = batch[bt];
      int gt = 0, eq = 0;
      for (int j = lane; j < bb.y; j += 32) {
        const uint32_t k = keys[bb.x + j];
        gt += k > T;
        eq += k == T;
      }
      gt = __reduce_add_sync(0xffffffffu, gt);
      eq = __reduce_add_sync(0xffffffffu, eq);
      if (lane == 0) batch_in[bt] = make_int2(gt, eq);
    }
    __syncthreads();
    int2 own = make_int2(0, 0);
    if (tid < nb) own = batch_in[tid];
    int2 incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl.x, o), y = __shfl_up_sync(0xffffffffu, incl.y, o);
      if (lane >= o) {
        incl.x += x;
        incl.y += y;
      }
    }
    const int2 wx = warps_before<NW>(__shfl_sync(0xffffffffu, incl.x, 31), wbuf[1]);
    const int2 wy = warps_before<NW>(__shfl_sync(0xffffffffu, incl.y, 31), wbuf[2]);
    if (tid < nb) batch_in[tid] = make_int2(wx.x + incl.x - own.x, wy.x + incl.y - own.y);
    if (tid == 0) cnt[2] = wx.y, cnt[3] = wy.y;   // the CTA's, for the sums over the cluster
  } else if (!bad) {
    auto count = [&](auto resident) {
#pragma unroll 1
      for (int j = j0 + lane * 4; j < j1; j += 128) {
        const uint4 k4 = resident || j < cap ? *reinterpret_cast<const uint4*>(keys + j) : load4(i0 + j);
        const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
        const bool c = M == kRest && i0 + j < n1p;   // n1p and j are multiples of 4
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int gt = k[u] > T, eq = k[u] == T && T != 0u;
          if (M == kRest) {
            cnt[0] += c ? gt : 0;
            cnt[1] += c ? eq : 0;
          }
          cnt[2] += c ? 0 : gt;
          cnt[3] += c ? 0 : eq;
        }
      }
    };
    if (items <= cap) count(Yes());
    else count(No());
  }
  int2 cta_in = make_int2(0, 0);                // above and at the edge in the CTAs before this one
  int mine[4], tot[4], all[4] = {0, 0, 0, 0};   // before this warp; over the CTA; over the cluster
#pragma unroll
  for (int u = M == kRest ? 0 : 2; u < 4; ++u) {
    const int2 v = warps_before<NW>(__reduce_add_sync(0xffffffffu, cnt[u]), wbuf[1 + u]);
    mine[u] = v.x;
    tot[u] = v.y;
  }
  if (M != kRest) mine[0] = mine[1] = tot[0] = tot[1] = 0;
  if (CL) {
    if (tid == 0) sh.count = make_int4(tot[0], tot[1], tot[2], tot[3]);
    cl.sync();
    int4 o[kMost];
#pragma unroll
    for (int r = 0; r < kMost; ++r)
      o[r] = r < C ? of(&sh, r)->count : make_int4(0, 0, 0, 0);
#pragma unroll
    for (int r = 0; r < kMost; ++r) {
      const int oc[4] = {o[r].x, o[r].y, o[r].z, o[r].w};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        all[u] += oc[u];
        if (r < rank) mine[u] += oc[u];
      }
      if (r < rank) {
        cta_in.x += o[r].z;
        cta_in.y += o[r].w;
      }
    }
  } else {
#pragma unroll
    for (int u = 0; u < 4; ++u) all[u] = tot[u];
  }
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

  // ---- the list (room, like the limits above: values that change while they are read must not lead out of it)
  const int room = M == kCandidates ? P.cand_len : P.sel_len;
  if (SIEVE && sieved) {
    const int gt0 = cta_in.x, eq0 = cta_in.y;
    int32_t* lp = sel + (size_t)row * P.sel_len;
    int2* le = ent + (size_t)row * P.sel_len;
    const unsigned lt = (1u << lane) - 1u;
    for (int bt = warp; bt < nb; bt += NW) {
      const int2 bb = batch[bt], in = batch_in[bt];
      int eq = eq0 + in.y, out = gt0 + in.x + min(need, eq);
      for (int j = lane; j - lane < bb.y; j += 32) {
        const uint32_t k = j < bb.y ? keys[bb.x + j] : 0u;
        const unsigned em = __ballot_sync(0xffffffffu, k == T);   // T is a key of the row, not 0
        const bool take = k > T || (k == T && eq + __popc(em & lt) < need);
        const unsigned tm = __ballot_sync(0xffffffffu, take);
        const int at = out + __popc(tm & lt);
        if (take && at < room) {
          const int pos = index[bb.x + j];
          lp[at] = pos;
          le[at] = make_int2(slot_of(pos), (int)((k & 0x80000000u) ? k ^ 0x80000000u : ~k));
        }
        eq += __popc(em);
        out += __popc(tm);
      }
    }
  } else if (!bad) {
    int eq = mine[1] + mine[3];                            // ties before this warp's keys
    int out = mine[2] + max(0, min(need, eq) - ties_c);    // listed keys before them
    int32_t* lp = M == kCandidates ? cand + (size_t)h * P.cand_len : sel + (size_t)row * P.sel_len;
    int2* le = M == kCandidates ? cent + (size_t)h * P.cand_len : ent + (size_t)row * P.sel_len;
    const unsigned lt = (1u << lane) - 1u;
    auto emit = [&](auto resident) {
      for (int j = j0; j < j1; j += 128) {
        const int jl = j + lane * 4, i = i0 + jl;
        uint4 k4 = make_uint4(0u, 0u, 0u, 0u);
        if (jl < j1) k4 = resident || jl < cap ? *reinterpret_cast<const uint4*>(keys + jl) : load4(i0 + jl);
        const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
        const bool c = M == kRest && i < n1p;
        bool take[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) take[u] = k[u] > T && !c;
        const bool has = T != 0u && (k[0] == T || k[1] == T || k[2] == T || k[3] == T);
        if (__any_sync(0xffffffffu, has)) {   // ties, in the order of positions
          int before = eq, sum = 0;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const unsigned em = __ballot_sync(0xffffffffu, k[u] == T);
            before += __popc(em & lt);
            sum += __popc(em);
          }
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (k[u] == T) {
              if (!c) take[u] = before < need;
              else if (before == need - 1 && ties_c < all[1]) rec[2] = i + u + 1;
              ++before;
            }
          eq += sum;
        }
        unsigned tm[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) tm[u] = __ballot_sync(0xffffffffu, take[u]);
        if ((tm[0] | tm[1] | tm[2] | tm[3]) == 0u) continue;
        int at = out + __popc(tm[0] & lt) + __popc(tm[1] & lt) + __popc(tm[2] & lt) + __popc(tm[3] & lt);
        out += __popc(tm[0]) + __popc(tm[1]) + __popc(tm[2]) + __popc(tm[3]);
        if (take[0] || take[1] || take[2] || take[3]) {
          const int pos = base + i - n1p;   // all four on one page
          const int slot = slot_of(pos);
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (take[u] && at < room) {
              lp[at] = pos + u;
              le[at] = make_int2(slot + u, (int)((k[u] & 0x80000000u) ? k[u] ^ 0x80000000u : ~k[u]));
              if (M == kCandidates && tail_n <= NT && k[u] < tail_end) {
                const int o = atomicAdd(of(&listed_total, 0), 1);   // in any order: they are ranked below
                if (o < NT) {
                  of(list, 0)[o] = k[u];
                  of(every, 0)[o] = (uint32_t)at;
                }
              }
              ++at;
            }
        }
      }
    };
    if (items <= cap) emit(Yes());
    else emit(No());
  }
  if (CL) cl.sync();   // no CTA leaves while another may still read its shared memory
  if constexpr (M == kCandidates) {
    // the last candidates in order, for rest_by_tail
    if (!CL) __syncthreads();
    if (rank != 0) return;
    int2* out = tail + (size_t)h * (kPagedTail + 1);
    const int m = bad ? 0 : min(listed_total, NT), n_t = min(m, kPagedTail);
    if (tid < m) {
      const uint32_t k = list[tid], i = every[tid];
      const uint64_t mine_last = last_first(k, i);
      int after = 0;
#pragma unroll 8
      for (int o = 0; o < m; ++o) after += last_first(list[o], every[o]) < mine_last;
      if (after < n_t) out[after] = make_int2((int)k, (int)i);
    }
    if (tid == 0) out[kPagedTail] = make_int2(n_t, 0);
  }
}

// cap: words of shared memory for keys.
template <SelMode M, int NT, bool SIEVE, int MC>
cudaError_t launch_select_t(const PagedPlan& P, int n_rows, int n, int C, int cap, int list_cap, void* ws,
                            cudaStream_t s) {
  const int seg = ((n + C - 1) / C + 3) & ~3;
  int page_cap = (seg >> P.page_shift) + 2;
  if (page_cap > 4100) page_cap = 4100;   // 65536 positions in the smallest pages
  const size_t smem = (size_t)(cap + page_cap) * 4;
  const cudaError_t e = ensure_smem_limit(paged_select_kernel<M, NT, SIEVE, MC>, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_after(paged_select_kernel<M, NT, SIEVE, MC>, dim3(C, n_rows), NT, smem, s, MC > 1 ? C : 1, P,
                      ws_ptr<int32_t>(ws, P.off_rows), ws_ptr<int32_t>(ws, P.off_sel), ws_ptr<int2>(ws, P.off_ent),
                      ws_ptr<int32_t>(ws, P.off_crow), ws_ptr<int32_t>(ws, P.off_cand), ws_ptr<int2>(ws, P.off_cent),
                      ws_ptr<int2>(ws, P.off_tail), ws_ptr<int32_t>(ws, P.off_count),
                      ws_ptr<int32_t>(ws, P.off_status), cap, page_cap, list_cap,
                      M == kRows && P.B > 1 && P.B <= kPsMostOrdered && n_rows * NT > sm_count() * 1024);
}

// Launches the selection of `n_rows` rows of at most n values.
template <SelMode M>
cudaError_t launch_select(const PagedPlan& P, int n_rows, int n, void* ws, cudaStream_t s) {
  const int sms = sm_count();
  if constexpr (M == kRows) {
    // rows that would take the kernel below several waves of stretches (16384 values an SM at a time), and with
    // 16 values to a place in the window: 256 rows of 65536 values take 36 us, 95 by the kernel below
    if (n >= 16384 && n >= 2 * kPsGroup * (int64_t)P.w && (int64_t)n_rows * n > (int64_t)sms * 16384) {
      int C = 1;
      while (C < kPsMaxCluster && ((n + C - 1) / C > 65536 || n_rows * C < sms)) C *= 2;
      const int seg = ((n + C - 1) / C + 3) & ~3;
      // the list: twice the window, and room for the maxima (two words an entry) first
      int list_cap = 2 * P.w + 2048;
      if (list_cap < seg / (2 * kPsGroup) + 64) list_cap = seg / (2 * kPsGroup) + 64;
      list_cap = (list_cap + 7) & ~7;
      const int cap = 2 * list_cap + list_cap / 2;
      if (seg <= 65536 && list_cap <= 32 * kPsMaxBatches && cap <= 36864)
        return C > 1 ? launch_select_t<M, 512, true, kPsMaxCluster>(P, n_rows, n, C, cap, list_cap, ws, s)
                     : launch_select_t<M, 512, true, 1>(P, n_rows, n, C, cap, list_cap, ws, s);
    }
  }
  // clusters: stretches of at most 16384 values, and for few rows as many CTAs as there are SMs for (more
  // would wait: a cluster needs its SMs side by side), down to stretches of 2048 (32 rows of 32768 values in
  // four stretches rather than two: a sixth less time); short rows in large numbers go to small CTAs, more of
  // which share an SM: 768 rows of up to 8192 values with 256 threads 26 us, with 512 31 (with 128, or
  // five CTAs of 256 an SM, 28); 2048 rows of some 2300 with 128 threads 9 us, with 512 25
  int C = 1;
  while (C < kPsMaxCluster && ((n + C - 1) / C > 16384 || (2 * n_rows * C <= sms && (n + C - 1) / C > 2048))) C *= 2;
  const int seg = ((n + C - 1) / C + 3) & ~3, cap = seg + 4 < 40960 ? seg + 4 : 40960;
  if (C > 4) return launch_select_t<M, 512, false, kPsMaxCluster>(P, n_rows, n, C, cap, 0, ws, s);
  if (C > 1) return launch_select_t<M, 512, false, 4>(P, n_rows, n, C, cap, 0, ws, s);
  if (n_rows >= 4 * sms) {
    if (seg <= 4096) return launch_select_t<M, 128, false, 1>(P, n_rows, n, C, cap, 0, ws, s);
    if (seg <= 8192) return launch_select_t<M, 256, false, 1>(P, n_rows, n, C, cap, 0, ws, s);
  }
  return launch_select_t<M, 512, false, 1>(P, n_rows, n, C, cap, 0, ws, s);
}

}  // namespace

cudaError_t launch_paged_topk(const PagedPlan& P, void* ws, cudaStream_t s) {
  if (!P.shared) return launch_select<kRows>(P, P.B * P.H, P.N, ws, s);
  const cudaError_t e = launch_select<kCandidates>(P, P.H, P.prefix, ws, s);
  if (e != cudaSuccess) return e;
  return launch_select<kRest>(P, P.B * P.H, ((P.cand_len + 3) & ~3) + P.N - P.prefix, ws, s);
}

}  // namespace dma
