// Single-query attention over the keys that paged_topk.cu selected.
//
// s_j = q . k_j scale + delta_j for the selected j; o = softmax(s) V; LSE = ln sum_j exp(s_j).  Scores
// stay in natural units (exponents are taken of differences from the running maximum), so that values of
// delta near the end of float32's range neither overflow nor lose the LSE.
//
// paged_list_kernel takes a row's own list.  The rows it needs lie anywhere in the cache, so what bounds
// it is how many 256-byte reads are in flight: a group of d / 8 lanes handles one key at a time (K and V
// row, 16 bytes a lane), a warp has the rows of 8 keys for each of its groups on the way at once, all in
// registers, and nothing waits for another warp before the end.  Each group keeps its own running maximum
// and sum; they meet once per CTA.
// paged_cand_kernel (shared prefix) multiplies all sequences' queries of a head with the head's
// candidates: 16 x 64 score tiles on the tensor cores, a sequence's selection being a comparison of the
// candidate's delta with the edge of its row.
// The partial results (m, l, o) of a row are joined, in a fixed order, by the CTA of its list that
// finishes last.
#include "rows.cuh"

namespace dma {
namespace {

constexpr int kPlThreads = 128;
constexpr int kPlWarps = kPlThreads / 32;

DMA_DEVINL float exp_diff(float x, float m) { return fast_exp2((x - m) * kLog2e); }

// Joins n partial results (m, l, o[D]) and writes the row's output.
template <typename T, int D>
DMA_DEVINL void join_row(const float* part, int n, T* O, float* LSE) {
  for (int c = threadIdx.x; c < D; c += kPlThreads) {
    float m = -INFINITY;
    for (int i = 0; i < n; ++i) m = fmaxf(m, __ldcg(part + (size_t)i * (D + 2)));
    const float ref = m == -INFINITY ? 0.f : m;
    float l = 0.f, o = 0.f;
    for (int i = 0; i < n; ++i) {
      const float* p = part + (size_t)i * (D + 2);
      const float w = exp_diff(__ldcg(p), ref);
      l = fmaf(__ldcg(p + 1), w, l);
      o = fmaf(__ldcg(p + 2 + c), w, o);
    }
    store_from_f32(O + c, l > 0.f ? o / l : (l == 0.f ? 0.f : l));   // nothing kept: 0; NaN stays
    if (c == 0) *LSE = l > 0.f ? ref + logf(l) : (l == 0.f ? -INFINITY : l);
  }
}

template <typename T, int D, int U>
__global__ void __launch_bounds__(kPlThreads)
paged_list_kernel(const T* __restrict__ Q, const T* __restrict__ K, const T* __restrict__ V,
                  const int4* __restrict__ rows, const int2* __restrict__ ent, float* __restrict__ part,
                  int32_t* __restrict__ counters, T* __restrict__ O, float* __restrict__ LSE, int H, int Hkv,
                  int page_shift, int sel_len, int n_split, int n_psplit, float scale) {
  constexpr int L = D / 8, RPW = 32 / L, NG = kPlWarps * RPW;   // lanes of a row; groups of a warp, of the CTA
  __shared__ float so[NG][D];
  __shared__ float sm[NG], sl[NG];
  __shared__ int last;
  const int row = blockIdx.y, h = row % H, g = h / (H / Hkv);
  const int tid = threadIdx.x, lane = tid & 31, grp = tid / L, e = (lane % L) * 8;
  const int count = min(rows[row].x, sel_len);
  const int k0 = blockIdx.x * kPagedSplit, k1 = min(count, k0 + kPagedSplit);
  if (k0 >= count && blockIdx.x > 0) return;   // the first CTA of a row works even if there is nothing
  const int2* list = ent + (size_t)row * sel_len;
  float q[8];
  widen8(load_raw8(Q + (size_t)row * D + e), q);
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] *= scale;
  float m = -INFINITY, l = 0.f, acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  const int mask = (1 << page_shift) - 1;
  // group grp takes U keys at a time: k0 + (NG r + grp) U ..
  for (int kb = k0 + (tid / 32) * RPW * U; kb < k1; kb += NG * U) {
    const int mykey = kb + (lane / L) * U + (lane % L);   // lane i of the group fetches entry i
    int2 en = make_int2(0, 0);
    if (lane % L < U && mykey < k1) en = list[mykey];
    Raw8<T> kr[U], vr[U];
    float dl[U];
    bool on[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int slot = __shfl_sync(0xffffffffu, en.x, u, L);
      dl[u] = __int_as_float(__shfl_sync(0xffffffffu, en.y, u, L));
      on[u] = kb + (lane / L) * U + u < k1;
      const size_t at = (((((size_t)(slot >> page_shift) * Hkv + g) << page_shift) + (slot & mask)) * D) + e;
      if (on[u]) {
        kr[u] = load_raw8(K + at);
        vr[u] = load_raw8(V + at);
      } else {
        kr[u] = Raw8<T>{};
        vr[u] = Raw8<T>{};
      }
    }
    float x[U], mx = m;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float k[8], s = 0.f;
      widen8(kr[u], k);
#pragma unroll
      for (int i = 0; i < 8; ++i) s = fmaf(k[i], q[i], s);
      s = row_sum<L>(s);
      x[u] = on[u] ? s + dl[u] : -INFINITY;
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
      const float p = exp_diff(x[u], ref);
      float v[8];
      widen8(vr[u], v);
      l += p;
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = fmaf(p, v[i], acc[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) so[grp][e + i] = acc[i];
  if (lane % L == 0) {
    sm[grp] = m;
    sl[grp] = l;
  }
  __syncthreads();
  const int n_act = count > 0 ? (count + kPagedSplit - 1) / kPagedSplit : 1;
  float* prow = part + (size_t)row * (n_psplit + n_split) * (D + 2);
  float* out = prow + (size_t)(n_psplit + blockIdx.x) * (D + 2);
  {
    float M = sm[0];
#pragma unroll
    for (int i = 1; i < NG; ++i) M = fmaxf(M, sm[i]);
    const float ref = M == -INFINITY ? 0.f : M;
    float w[NG], lsum = 0.f;
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      w[i] = exp_diff(sm[i], ref);
      lsum = fmaf(sl[i], w[i], lsum);
    }
    for (int c = tid; c < D; c += kPlThreads) {
      float o = 0.f;
#pragma unroll
      for (int i = 0; i < NG; ++i) o = fmaf(so[i][c], w[i], o);
      if (n_act + n_psplit == 1) {
        store_from_f32(O + (size_t)row * D + c, lsum > 0.f ? o / lsum : (lsum == 0.f ? 0.f : lsum));
        if (c == 0) LSE[row] = lsum > 0.f ? ref + logf(lsum) : (lsum == 0.f ? -INFINITY : lsum);
      } else {
        out[2 + c] = o;
        if (c == 0) {
          out[0] = M;
          out[1] = lsum;
        }
      }
    }
  }
  if (n_act + n_psplit == 1) return;
  __threadfence();
  __syncthreads();
  if (tid == 0) {
    last = atomicAdd(counters + row, 1) == n_act - 1;
    if (last) counters[row] = 0;   // as the next call expects it
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  join_row<T, D>(prow, n_psplit + n_act, O + (size_t)row * D, LSE + row);
}

template <typename T, int D, int U>
cudaError_t launch_list(const PagedPlan& P, const void* Q, void* ws, void* O, float* LSE, cudaStream_t s) {
  paged_list_kernel<T, D, U><<<dim3(P.n_split, P.B * P.H), kPlThreads, 0, s>>>(
      (const T*)Q, (const T*)P.K, (const T*)P.V, ws_ptr<int4>(ws, P.off_rows), ws_ptr<int2>(ws, P.off_ent),
      ws_ptr<float>(ws, P.off_part), ws_ptr<int32_t>(ws, P.off_count), (T*)O, LSE, P.H, P.Hkv, P.page_shift, P.sel_len,
      P.n_split, P.n_psplit, P.scale);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_attn(const PagedPlan& P, const void* Q, void* ws, void* O, float* LSE, cudaStream_t s) {
  if (P.bf16)
    return P.d == 128 ? launch_list<uint16_t, 128, 8>(P, Q, ws, O, LSE, s)
                      : launch_list<uint16_t, 64, 8>(P, Q, ws, O, LSE, s);
  return P.d == 128 ? launch_list<float, 128, 4>(P, Q, ws, O, LSE, s) : launch_list<float, 64, 4>(P, Q, ws, O, LSE, s);
}

}  // namespace dma
