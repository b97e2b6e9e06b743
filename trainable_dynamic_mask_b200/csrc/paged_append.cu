// Appending tokens to the paged cache: keys normed and rotated into their slots, values copied, gate
// values delta = exp(A softplus(v Delta)) formed from the values on the way, queries of the same tokens
// normed and rotated.
//
// One kernel, two kinds of CTAs side by side: the first walk over the rows (rows.cuh, as in prep.cu), the
// others form the gate's product (the values of 16 tokens against Delta, tensor cores for bf16).  The walk's
// shares are fixed when it starts and it is the longer way, so it comes first, with three CTAs an SM (two for more
// than 32 heads in bf16) and two chunks of rows on their way; the gate's CTAs follow where those have ended.
//
// Bytes: each projection read once and each row written once, 16 KB a token at 16 + 8 + 8 heads of 128
// channels in bf16, Delta from L2.  5037 tokens of 5 prompts take 25.6 us among calls on other inputs (3.2 TB/s) and
// 34 in a graph from a cold L2, where a plain copy of as many bytes takes 37: a short call stays below a long
// one's rate.  Without the gate they would take 4 us less, the gate alone 9.  Two CTAs an SM with four chunks on
// their way took 28.6 us, three with four 27.5, four (64 registers) 29; the gate's CTAs first, or with four stages,
// the same.  float32, 32 + 8 + 8 heads: 126 us (floor 38); the gate's product on the FMA pipe reads Delta from L2
// for every 8 tokens.
// One token for each of 64 sequences takes 9 us in a graph, bound by latency: the lookup's reads, one wave of
// rows, the gate (3 us of it); in float32 34.
#include "rows.cuh"

namespace dma {
namespace {

DMA_DEVINL float softplus_of(float x) { return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))); }

// Where token t goes.
struct Place {
  int seq, pos;    // pos < 0: nothing of this token is written
  int page, slot;
};

// Sequence and slot of token t (a whole warp, each lane its own token; wanted: t < T).  What is read first
// depends on nothing, the page number on that: up to 31 sequences' starts and lengths are read at once, a
// sequence a lane, rather than searched for one after the other.
DMA_DEVINL Place place_of(const PagedPlan& P, const PagedAppendArgs& a, int t, bool wanted, int32_t* status) {
  constexpr unsigned kAll = 0xffffffffu;
  int seq = t, first = t, n = 1, len = 0;
  if (a.starts == nullptr) {
    if (wanted) len = __ldg(P.lens + seq);
  } else {
    // the sequence before the first that starts behind t; none: padding in front of them all, or behind
    int lo = 0, hi = P.B + 1;   // starts[i] <= t for i < lo, > t for i >= hi
    if (P.B < 32) {
      const int lane = threadIdx.x & 31;
      const int s = __ldg(a.starts + min(lane, P.B)), l = __ldg(P.lens + min(lane, P.B - 1));
#pragma unroll
      for (int i = 0; i < 6; ++i) {   // 33 answers at most
        const int mid = (lo + hi) >> 1, v = __shfl_sync(kAll, s, mid & 31);
        if (lo < hi) {
          if (v <= t) lo = mid + 1;
          else hi = mid;
        }
      }
      seq = lo - 1;
      first = __shfl_sync(kAll, s, seq & 31);
      n = __shfl_sync(kAll, s, (seq + 1) & 31) - first;
      len = __shfl_sync(kAll, l, seq & 31);
    } else if (wanted) {
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(a.starts + mid) <= t) lo = mid + 1;
        else hi = mid;
      }
      seq = lo - 1;
      if (seq >= 0 && seq < P.B) {
        first = __ldg(a.starts + seq);
        n = __ldg(a.starts + seq + 1) - first;
        len = __ldg(P.lens + seq);
      }
    }
    if (seq < 0 || seq >= P.B) return {0, -1, 0, 0};
  }
  if (!wanted || len <= 0) return {seq, -1, 0, 0};
  const int pos = len - n + (t - first);
  int page = -1;   // a length below the prefix would lead into the pages that the batch shares
  if (pos >= 0 && pos < len && len >= P.prefix && len <= P.N)
    page = __ldg(P.table + (size_t)seq * P.max_pages + (pos >> P.page_shift));
  if (page < 0 || page >= P.n_pages) {
    atomicOr(status, kPagedErr);
    return {seq, -1, 0, 0};
  }
  return {seq, pos, page, pos & ((1 << P.page_shift) - 1)};
}

// ---------------------------------------------------------------- rows

// Keys and values to their slots, queries to Q [T, H, D].  A warp looks up the places of its next 32 tokens
// together, a token a lane: the lookups' three or more dependent reads are then paid once.
struct SlotDest {
  static constexpr int kDepth = 2;
  struct Token {
    int position;
    unsigned tok;
    size_t slot;        // of head 0, in rows
    int looked_up = 0;  // tokens of the batch of 32 already entered
    int pos, page;      // this lane's token of the batch
  };
  PagedPlan P;
  PagedAppendArgs a;
  int32_t* status;
  int size;
  DMA_DEVINL bool enter(const Walk& at, Token& t) const {
    const int i = t.looked_up & 31;
    if (i == 0) {
      const unsigned mine = at.tok + (threadIdx.x & 31) * at.step;
      const Place pl = place_of(P, a, (int)mine, mine < at.tokens && mine >= at.tok, status);
      __syncwarp();
      t.pos = pl.pos;
      t.page = pl.page;
    }
    ++t.looked_up;
    t.tok = at.tok;
    t.position = __shfl_sync(0xffffffffu, t.pos, i);
    const int page = __shfl_sync(0xffffffffu, t.page, i);
    t.slot = ((size_t)page * P.Hkv << P.page_shift) + (t.position & ((1 << P.page_shift) - 1));
    return t.position >= 0;
  }
  DMA_DEVINL void* row(int part, const Token& t) const {
    if (part == 0) return (char*)a.Q + (size_t)t.tok * P.H * P.d * size;
    return (part == 1 ? P.K : P.V) + t.slot * P.d * size;
  }
  DMA_DEVINL size_t step(int part) const { return part == 0 ? (size_t)P.d : (size_t)P.d << P.page_shift; }
};

// ---------------------------------------------------------------- gate, tensor cores

constexpr int kAgTok = 16;        // tokens of a CTA: one m16 tile
constexpr int kAgThreads = kRwThreads;
constexpr int kAgWarps = kAgThreads / 32;

// Offset of (token's page, head 0, slot) in the delta pages of the CTA's tokens; -1: none.
DMA_DEVINL void gate_places(const PagedPlan& P, const PagedAppendArgs& a, int t0, int n, long long* where,
                            int32_t* status) {
  const int i = threadIdx.x;
  if (i < 32) {
    const Place pl = place_of(P, a, t0 + i, i < n && t0 + i < a.T, status);
    if (i < n) where[i] = pl.pos < 0 ? -1 : ((long long)pl.page * P.H << P.page_shift) + pl.slot;
  }
}

constexpr int kAgK = 256;         // channels of a stage, two stages

template <int HT> constexpr int gate_smem() {
  constexpr int stages = 2 * kAgK * (kAgTok + 8 * HT) * 2, sums = kAgWarps * kAgTok * 8 * HT * 4;
  return stages > sums ? stages : sums;
}

// x [16 tokens, H] = v [16, K] Delta [K, H], K = Hkv d, in stages of 256 channels: the warps split a stage in
// steps of 16 and their tiles are summed through shared memory (in a fixed order).  bf16 products are exact
// in float32, in which all is accumulated.  Two stages (32 to 80 KB) rather than all of K at once leave
// room for the rows' CTAs beside these.
template <int HT>   // column tiles of 8 heads
DMA_DEVINL void gate_mma(const PagedPlan& P, const PagedAppendArgs& a, int32_t* status, int block, unsigned char* sm) {
  __shared__ long long where[kAgTok];
  constexpr int KC = kAgK / 8, kStage = kAgK * (kAgTok + 8 * HT);   // elements
  uint16_t* const stage = reinterpret_cast<uint16_t*>(sm);   // [2]: v [16][256], chunk c of row r at c ^ (r & 7);
                                                             // Delta [256][8 HT]
  float* red = reinterpret_cast<float*>(sm);                 // [8 warps][16][8 HT], in the stages' place
  const int K = P.Hkv * P.d, dch = P.d / 8, n_st = (K + kAgK - 1) / kAgK;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int t0 = block * kAgTok;
  const uint16_t* v = static_cast<const uint16_t*>(a.v);
  const uint16_t* Delta = static_cast<const uint16_t*>(a.Delta);
  auto load = [&](int st) {
    uint16_t* Vs = stage + (st & 1) * kStage;
    uint16_t* Ds = Vs + kAgTok * kAgK;
#pragma unroll
    for (int u = tid; u < kAgTok * KC; u += kAgThreads) {
      const int r = u / KC, kc = u % KC, q = st * KC + kc, g = q / dch, c = q - g * dch;
      const bool in = t0 + r < a.T && q * 8 < K;
      const uint16_t* src = in ? v + (long long)(t0 + r) * a.st.v[1] + g * a.st.v[2] + c * 8 : v;
      cp_async_16(smem_u32(Vs + r * kAgK + ((kc ^ (r & 7)) * 8)), src, in ? 16 : 0);
    }
    if ((P.H & 7) == 0) {
      const int hc = P.H / 8;
#pragma unroll
      for (int u = tid; u < kAgK * HT; u += kAgThreads) {
        const int r = u / HT, c = u % HT, k = st * kAgK + r;
        const bool in = c < hc && k < K;
        cp_async_16(smem_u32(Ds + r * 8 * HT + c * 8), in ? Delta + (size_t)k * P.H + c * 8 : Delta, in ? 16 : 0);
      }
    } else {
      for (int u = tid; u < kAgK * 8 * HT; u += kAgThreads) {
        const int r = u / (8 * HT), h = u % (8 * HT), k = st * kAgK + r;
        Ds[u] = h < P.H && k < K ? Delta[(size_t)k * P.H + h] : (uint16_t)0;
      }
    }
    cp_async_commit();
  };
  load(0);
  gate_places(P, a, t0, kAgTok, where, status);
  float acc[HT][4];
#pragma unroll
  for (int n = 0; n < HT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
  const int arow = lane & 15, half = lane >> 4;
  for (int st = 0; st < n_st; ++st) {
    if (st + 1 < n_st) load(st + 1);
    else cp_async_commit();
    cp_async_wait<1>();
    __syncthreads();
    const uint32_t vs = smem_u32(stage + (st & 1) * kStage), ds = vs + kAgTok * kAgK * 2;
#pragma unroll
    for (int i = 0; i < kAgK / 16 / kAgWarps; ++i) {
      const int ks = warp + i * kAgWarps;
      uint32_t f[4];
      ldmatrix_x4(vs + (uint32_t)(arow * kAgK + (((ks * 2 + half) ^ (arow & 7)) * 8)) * 2, f[0], f[1], f[2], f[3]);
#pragma unroll
      for (int n = 0; n < HT; n += 2) {
        uint32_t b0, b1, b2, b3;
        ldmatrix_x4_trans(ds + (uint32_t)((ks * 16 + arow) * 8 * HT + (n + half) * 8) * 2, b0, b1, b2, b3);
        mma_bf16_16816(acc[n], f, b0, b1);
        mma_bf16_16816(acc[n + 1], f, b2, b3);
      }
    }
    __syncthreads();   // the stage may be filled again
  }
  const int g = lane >> 2, q = lane & 3;
#pragma unroll
  for (int n = 0; n < HT; ++n) {
    float* w = red + (size_t)warp * kAgTok * 8 * HT + n * 8 + 2 * q;
    *reinterpret_cast<float2*>(w + g * 8 * HT) = make_float2(acc[n][0], acc[n][1]);
    *reinterpret_cast<float2*>(w + (g + 8) * 8 * HT) = make_float2(acc[n][2], acc[n][3]);
  }
  __syncthreads();
  // consecutive threads take consecutive tokens of a head: neighbouring slots of one page
  for (int o = tid; o < kAgTok * P.H; o += kAgThreads) {
    const int t = o % kAgTok, h = o / kAgTok;
    const long long at = where[t];
    if (at < 0) continue;
    float x = 0.f;
#pragma unroll
    for (int w = 0; w < kAgWarps; ++w) x += red[((size_t)w * kAgTok + t) * 8 * HT + h];
    P.delta[at + ((long long)h << P.page_shift)] = expf(a.A[h] * softplus_of(x));
  }
}

// ---------------------------------------------------------------- gate, float32

constexpr int kAfTok = 8;      // tokens of a CTA
constexpr int kAfK = 512;      // channels staged at a time

// float32 storage: the same product on the FMA pipe, with the values' full precision.  Thread = one head and
// one of NS slices of the staged channels, for 8 tokens.
DMA_DEVINL void gate_fma(const PagedPlan& P, const PagedAppendArgs& a, int32_t* status, int block, float* fsm) {
  __shared__ long long where[kAfTok];
  float* Vs = fsm;                   // [kAfK][kAfTok]
  float* red = Vs + kAfK * kAfTok;   // [NS][kAfTok][HP]
  const int K = P.Hkv * P.d, HP = P.H <= 16 ? 16 : P.H <= 32 ? 32 : 64, NS = kAgThreads / HP;
  const int tid = threadIdx.x, h = tid % HP, sl = tid / HP;
  const int t0 = block * kAfTok;
  const float* v = static_cast<const float*>(a.v);
  const float* Delta = static_cast<const float*>(a.Delta);
  gate_places(P, a, t0, kAfTok, where, status);
  float acc[kAfTok];
#pragma unroll
  for (int i = 0; i < kAfTok; ++i) acc[i] = 0.f;
  for (int k0 = 0; k0 < K; k0 += kAfK) {
    const int kn = min(kAfK, K - k0);
    __syncthreads();
    for (int u = tid; u < kn * kAfTok; u += kAgThreads) {
      const int t = u / kn, kk = u % kn, g = (k0 + kk) / P.d, c = (k0 + kk) % P.d;
      Vs[kk * kAfTok + t] =
          t0 + t < a.T ? v[(long long)(t0 + t) * a.st.v[1] + g * a.st.v[2] + c] : 0.f;
    }
    __syncthreads();
    if (h < P.H && sl < NS) {
#pragma unroll 4
      for (int kk = sl; kk < kn; kk += NS) {
        const float dl = Delta[(size_t)(k0 + kk) * P.H + h];
        const float4 v0 = reinterpret_cast<const float4*>(Vs + kk * kAfTok)[0];
        const float4 v1 = reinterpret_cast<const float4*>(Vs + kk * kAfTok)[1];
        acc[0] = fmaf(v0.x, dl, acc[0]); acc[1] = fmaf(v0.y, dl, acc[1]);
        acc[2] = fmaf(v0.z, dl, acc[2]); acc[3] = fmaf(v0.w, dl, acc[3]);
        acc[4] = fmaf(v1.x, dl, acc[4]); acc[5] = fmaf(v1.y, dl, acc[5]);
        acc[6] = fmaf(v1.z, dl, acc[6]); acc[7] = fmaf(v1.w, dl, acc[7]);
      }
    }
  }
  if (h < P.H && sl < NS) {
#pragma unroll
    for (int i = 0; i < kAfTok; ++i) red[(sl * kAfTok + i) * HP + h] = acc[i];
  }
  __syncthreads();
  for (int o = tid; o < kAfTok * P.H; o += kAgThreads) {
    const int t = o % kAfTok, hh = o / kAfTok;
    const long long at = where[t];
    if (at < 0) continue;
    float x = 0.f;
    for (int s = 0; s < NS; ++s) x += red[(s * kAfTok + t) * HP + hh];
    P.delta[at + ((long long)hh << P.page_shift)] = expf(a.A[hh] * softplus_of(x));
  }
}

// ---------------------------------------------------------------- both

template <typename T, int HT> constexpr int append_smem() {
  constexpr int rows = FwdRing<T, SlotDest::kDepth>::kBytes;
  constexpr int gate = HT > 0 ? gate_smem<HT>() : (kAfK * kAfTok + kAgThreads * kAfTok) * 4;
  return rows > gate ? rows : gate;
}

// HT: column tiles of the gate's product (bf16), or 0 (float32).
template <typename T, int D, bool INTER, int HT>
__global__ void __launch_bounds__(kRwThreads, 3)
paged_append_kernel(const __grid_constant__ PrepArgs w, const __grid_constant__ SlotDest dest, int wt, int row_blocks) {
  extern __shared__ __align__(128) unsigned char smem[];
  const int block = (int)blockIdx.x - row_blocks;
  if (block < 0) {
    walk_rows<T, D, INTER>(w, dest, wt, blockIdx.x, row_blocks, smem);
  } else {
    if constexpr (HT > 0) gate_mma<HT>(dest.P, dest.a, dest.status, block, smem);
    else gate_fma(dest.P, dest.a, dest.status, block, reinterpret_cast<float*>(smem));
  }
}

template <typename T, int D, int HT>
cudaError_t launch_append(const PrepArgs& w, const SlotDest& d, cudaStream_t s) {
  // the gate's stages for more than 32 heads leave room for two CTAs an SM, so the rows' shares are made for two (5037
  // tokens of 64 heads: 80.8 us, in shares for three 88.3)
  int wt;
  constexpr int smem = append_smem<T, HT>(), per_sm = smem > 64 * 1024 ? 2 : 3;
  const int row_blocks = walk_blocks(d.a.T, per_sm, &wt), tok = HT > 0 ? kAgTok : kAfTok;
  auto kernel = w.inter ? paged_append_kernel<T, D, true, HT> : paged_append_kernel<T, D, false, HT>;
  const cudaError_t e = ensure_smem_limit(kernel, smem);
  if (e != cudaSuccess) return e;
  kernel<<<row_blocks + (d.a.T + tok - 1) / tok, kRwThreads, smem, s>>>(w, d, wt, row_blocks);
  return cudaGetLastError();
}

template <int D> cudaError_t launch_append_bf16(const PrepArgs& w, const SlotDest& d, cudaStream_t s) {
  if (d.P.H <= 16) return launch_append<uint16_t, D, 2>(w, d, s);
  if (d.P.H <= 32) return launch_append<uint16_t, D, 4>(w, d, s);
  return launch_append<uint16_t, D, 8>(w, d, s);
}

}  // namespace

cudaError_t launch_paged_append(const PagedPlan& P, const PagedAppendArgs& a, void* ws, cudaStream_t s) {
  PrepArgs w = {};
  w.inv_freq = a.r.inv_freq;
  w.weight[0] = a.r.q_weight;
  w.weight[1] = a.r.k_weight;
  w.in[0] = a.q; w.in[1] = a.k; w.in[2] = a.v;
  w.out[0] = a.Q; w.out[1] = P.K; w.out[2] = P.V;
  for (int i = 1; i < 3; ++i) {
    w.stride[0][i] = a.st.q[i];
    w.stride[1][i] = a.st.k[i];
    w.stride[2][i] = a.st.v[i];
  }
  w.eps = a.r.eps;
  w.B = 1; w.H = P.H; w.Hkv = P.Hkv; w.N = a.T; w.rot = a.r.rot;
  w.inter = a.r.interleaved != 0;
  SlotDest d = {};
  d.P = P;
  d.a = a;
  d.status = ws_ptr<int32_t>(ws, P.off_status);
  d.size = P.bf16 ? 2 : 4;
  if (P.bf16) return P.d == 128 ? launch_append_bf16<128>(w, d, s) : launch_append_bf16<64>(w, d, s);
  return P.d == 128 ? launch_append<float, 128, 0>(w, d, s) : launch_append<float, 64, 0>(w, d, s);
}

}  // namespace dma
