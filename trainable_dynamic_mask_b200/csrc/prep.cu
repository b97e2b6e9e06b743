// From the projections to the attention's inputs, and the gradients on their way back.
//
// Forward, per head row x of a query or key at position n (the norm where a weight g is given):
//   r = (mean(x^2) + eps)^(-1/2),  y = x r g,  out = R(n) y,
// R(n) the rotation of the first rot channels, pair i by the angle n f_i; value rows are copied.  Rows
// are read wherever the projection left them (strides) and written as [B, heads, N, d], so the
// transposition costs no pass of its own.
// Backward, with dy = R(n)^T dOut:  dx = r (g dy - x r^2 mean(x g dy)),  dg = sum over rows of dy x r,
// and dv = dV + dV_gate.  r is formed again from x, which the norm's gradient reads anyway.
#include <math.h>
#include <string.h>

#include "rows.cuh"

namespace dma {
namespace {

constexpr int kPrThreads = 256;
constexpr int kPrWarps = kPrThreads / 32;

// A warp works on one token at a time, its D / 8-lane groups on neighbouring heads; wt = 1, 2, 4 or 8
// warps of a block share a token's heads (many for few tokens, so that the heads of a single token
// spread over the block).  The angles of a block's tokens are computed once into shared memory and
// kept in registers over the token's heads.
template <typename T, int D, int U>
__global__ void __launch_bounds__(kPrThreads)
prep_fwd_kernel(PrepArgs a, int wt) {
  constexpr int L = D / 8, RPW = 32 / L;   // lanes of a row, rows of a warp
  __shared__ float2 tab[kPrWarps][D / 2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tpb = kPrWarps / wt;
  const long long t0 = (long long)blockIdx.x * tpb, nt = (long long)a.B * a.N;
  const int half = a.rot >> 1;
  for (int u = tid; u < tpb * half; u += kPrThreads) {
    const int tt = u / half, k = u - tt * half;
    const long long t = t0 + tt;
    if (t < nt) {
      const int pos = a.positions ? a.positions[t] : a.first + (int)(t % a.N);
      tab[tt][k] = turn_of(pos, __ldg(a.inv_freq + k));
    }
  }
  __syncthreads();
  const long long t = t0 + warp / wt;
  if (t >= nt) return;
  const int b = (int)(t / a.N), n = (int)(t - (long long)b * a.N);
  const int grp = lane / L, e = (lane % L) * 8;
  LaneTurn turn;
  lane_turn<L>(turn, tab[warp / wt], a.rot, a.inter, lane);
  const T* src[3];
  long long hs[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    src[i] = (const T*)a.in[i] + b * a.stride[i][0] + n * a.stride[i][1] + e;
    hs[i] = a.stride[i][2];
  }
  // queries, then keys, then values: U rows of loads in flight in each lane
#pragma unroll 1
  for (int part = 0; part < 3; ++part) {
    if (a.out[part] == nullptr) continue;
    const int heads = part == 0 ? a.H : a.Hkv;
    T* dst = (T*)a.out[part] + ((long long)b * heads * a.N + n) * D + e;
    const T* wp = part < 2 ? (const T*)a.weight[part] : nullptr;
    float g[8];
    if (wp) widen8(load_raw8(wp + e), g);
    const T* sp = src[part];
    const long long sh = hs[part], dh = (long long)a.N * D;
    for (int h0 = (warp % wt) * RPW * U; h0 < heads; h0 += wt * RPW * U) {
      Raw8<T> raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = min(h0 + u * RPW + grp, heads - 1);   // past the end: the last row again, not stored
        raw[u] = load_raw8(sp + h * sh);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * RPW + grp;
        if (part == 2) {
          if (h < heads) store_raw8(dst + h * dh, raw[u]);
          continue;
        }
        float y[8];
        widen8(raw[u], y);
        if (wp) {
          float ss = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(y[i], y[i], ss);
          const float r = rsqrtf(row_sum<L>(ss) * (1.f / D) + a.eps);
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] *= r * g[i];
        }
        rotate8<false>(y, turn, a.inter);
        if (h < heads) store8(dst + h * dh, y);
      }
    }
  }
}

// Blocks walk over the tokens in a fixed order, so the partial sums of the weights' gradients (float32
// within a lane, at most a few thousand rows each) do not depend on scheduling.
template <typename T, int D, int U>
__global__ void __launch_bounds__(kPrThreads)
prep_bwd_kernel(PrepArgs a, int wt) {
  constexpr int L = D / 8, RPW = 32 / L;
  __shared__ float2 tab[kPrWarps][D / 2];
  __shared__ float red[kPrWarps * RPW][D];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tpb = kPrWarps / wt;
  const long long nt = (long long)a.B * a.N;
  const int half = a.rot >> 1;
  const int grp = lane / L, e = (lane % L) * 8;
  float gw[2][8];   // this lane's share of the weights' gradients
#pragma unroll
  for (int i = 0; i < 8; ++i) gw[0][i] = gw[1][i] = 0.f;
  for (long long t0 = (long long)blockIdx.x * tpb; t0 < nt; t0 += (long long)gridDim.x * tpb) {
    __syncthreads();   // the angles of the last round are no longer read
    for (int u = tid; u < tpb * half; u += kPrThreads) {
      const int tt = u / half, k = u - tt * half;
      const long long t = t0 + tt;
      if (t < nt) {
        const int pos = a.positions ? a.positions[t] : a.first + (int)(t % a.N);
        tab[tt][k] = turn_of(pos, __ldg(a.inv_freq + k));
      }
    }
    __syncthreads();
    const long long t = t0 + warp / wt;
    if (t >= nt) continue;
    const int b = (int)(t / a.N), n = (int)(t - (long long)b * a.N);
    LaneTurn turn;
    lane_turn<L>(turn, tab[warp / wt], a.rot, a.inter, lane);
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      const int heads = part == 0 ? a.H : a.Hkv;
      const T* dy = (const T*)a.grad[part] + ((long long)b * heads * a.N + n) * D + e;
      const long long dh = (long long)a.N * D, sh = a.stride[part][2], gh = a.gstride[part][2];
      const T* xp = (const T*)a.in[part] + b * a.stride[part][0] + n * a.stride[part][1] + e;
      T* dx = (T*)a.out[part] + b * a.gstride[part][0] + n * a.gstride[part][1] + e;
      const T* wp = (const T*)a.weight[part];
      float g[8];
      if (wp) widen8(load_raw8(wp + e), g);
      for (int h0 = (warp % wt) * RPW * U; h0 < heads; h0 += wt * RPW * U) {
        Raw8<T> rg[U], rx[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int h = min(h0 + u * RPW + grp, heads - 1);
          rg[u] = load_raw8(dy + h * dh);
          if (wp) rx[u] = load_raw8(xp + h * sh);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int h = h0 + u * RPW + grp;
          float y[8];
          widen8(rg[u], y);
          rotate8<true>(y, turn, a.inter);
          if (wp) {
            float x[8], ss = 0.f, dot = 0.f;
            widen8(rx[u], x);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              ss = fmaf(x[i], x[i], ss);
              dot = fmaf(x[i] * g[i], y[i], dot);
            }
            const float r = rsqrtf(row_sum<L>(ss) * (1.f / D) + a.eps);
            const float k = row_sum<L>(dot) * (1.f / D) * r * r;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              if (h < heads) gw[part][i] = fmaf(y[i], x[i] * r, gw[part][i]);
              y[i] = r * fmaf(-x[i], k, g[i] * y[i]);
            }
          }
          if (h < heads) store8(dx + h * gh, y);
        }
      }
    }
    if (a.out[2]) {
      const T* dv = (const T*)a.grad[2] + ((long long)b * a.Hkv * a.N + n) * D + e;
      const float* dvg = a.dv_gate ? a.dv_gate + ((long long)b * a.Hkv * a.N + n) * D + e : nullptr;
      T* out = (T*)a.out[2] + b * a.gstride[2][0] + n * a.gstride[2][1] + e;
      for (int h0 = (warp % wt) * RPW * U; h0 < a.Hkv; h0 += wt * RPW * U) {
        Raw8<T> rv[U];
        Raw8<float> rg[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const long long h = min(h0 + u * RPW + grp, a.Hkv - 1);
          rv[u] = load_raw8(dv + h * a.N * D);
          if (dvg) rg[u] = load_raw8(dvg + h * a.N * D);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int h = h0 + u * RPW + grp;
          if (h >= a.Hkv) continue;
          if (dvg) {
            float v[8], w[8];
            widen8(rv[u], v);
            widen8(rg[u], w);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += w[i];
            store8(out + h * a.gstride[2][2], v);
          } else {
            store_raw8(out + h * a.gstride[2][2], rv[u]);
          }
        }
      }
    }
  }
  // the block's partial sums of dg, one row of the workspace each
#pragma unroll
  for (int part = 0; part < 2; ++part) {
    if (!a.weight[part]) continue;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) red[warp * RPW + grp][e + i] = gw[part][i];
    __syncthreads();
    for (int c = tid; c < D; c += kPrThreads) {
      float v = 0.f;
#pragma unroll
      for (int q = 0; q < kPrWarps * RPW; ++q) v += red[q][c];
      a.part[((size_t)part * gridDim.x + blockIdx.x) * D + c] = v;
    }
  }
}

// dg[c] = sum over blocks, in double precision: at most kPrepMaxBlocks terms per channel, 32 channels a block.
__global__ void __launch_bounds__(1024)
prep_reduce_kernel(const float* __restrict__ part, float* __restrict__ dq_weight, float* __restrict__ dk_weight,
                   int n_blocks, int D) {
  __shared__ double red[32][33];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
  float* out = blockIdx.y == 0 ? dq_weight : dk_weight;
  if (out == nullptr) return;
  const float* p = part + (size_t)blockIdx.y * n_blocks * D + c;
  double v = 0.0;
  for (int i = w; i < n_blocks; i += 32) v += (double)p[(size_t)i * D];
  red[w][threadIdx.x & 31] = v;
  __syncthreads();
  if (w == 0) {
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += red[i][threadIdx.x];
    out[c] = (float)s;
  }
}

// Warps that share a token: as many as it takes to give every SM a block, 8 at most.
int warps_per_token(long long tokens, int sms) {
  int wt = 1;
  while (wt < kPrWarps && tokens * wt < (long long)sms * kPrWarps) wt *= 2;
  return wt;
}

template <typename T, int D>
cudaError_t launch_fwd(const PrepArgs& a, cudaStream_t s) {
  const long long tokens = (long long)a.B * a.N;
  const int wt = warps_per_token(tokens, sm_count()), tpb = kPrWarps / wt;
  prep_fwd_kernel<T, D, 4><<<(unsigned)((tokens + tpb - 1) / tpb), kPrThreads, 0, s>>>(a, wt);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_bwd(const PrepArgs& a, float* dqw, float* dkw, cudaStream_t s) {
  const long long tokens = (long long)a.B * a.N;
  const int wt = warps_per_token(tokens, sm_count()), tpb = kPrWarps / wt;
  long long blocks = (tokens + tpb - 1) / tpb;
  if (blocks > kPrepMaxBlocks) blocks = kPrepMaxBlocks;
  prep_bwd_kernel<T, D, 2><<<(unsigned)blocks, kPrThreads, 0, s>>>(a, wt);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || (dqw == nullptr && dkw == nullptr)) return e;
  prep_reduce_kernel<<<dim3(D / 32, 2), 1024, 0, s>>>(a.part, dqw, dkw, (int)blocks, D);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prep_fwd(const PrepArgs& a, bool bf16, int d, cudaStream_t s) {
  if (bf16) return d == 128 ? launch_fwd<uint16_t, 128>(a, s) : launch_fwd<uint16_t, 64>(a, s);
  return d == 128 ? launch_fwd<float, 128>(a, s) : launch_fwd<float, 64>(a, s);
}

cudaError_t launch_prep_bwd(const PrepArgs& a, bool bf16, int d, float* dqw, float* dkw, cudaStream_t s) {
  if (bf16) return d == 128 ? launch_bwd<uint16_t, 128>(a, dqw, dkw, s) : launch_bwd<uint16_t, 64>(a, dqw, dkw, s);
  return d == 128 ? launch_bwd<float, 128>(a, dqw, dkw, s) : launch_bwd<float, 64>(a, dqw, dkw, s);
}

bool check_strides(const int64_t (&st)[3], bool bf16) {
  const int64_t unit = bf16 ? 8 : 4;
  for (int i = 0; i < 3; ++i)
    if (st[i] < 0 || st[i] % unit != 0 || st[i] > ((int64_t)1 << 40)) return false;
  return true;
}

dma_status_t check_prep(const dma_prep_t* r, int d) {
  if (r == nullptr || r->rot < 0 || r->rot > d) return DMA_ERR_INVALID_ARG;
  if (!(r->eps > 0.f) || isinf(r->eps)) return DMA_ERR_INVALID_ARG;
  if (r->interleaved != 0 && r->interleaved != 1) return DMA_ERR_INVALID_ARG;
  if ((r->rot > 0) != (r->inv_freq != nullptr)) return DMA_ERR_INVALID_ARG;
  auto bad = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15u) != 0; };
  if (bad(r->inv_freq) || bad(r->positions) || bad(r->q_weight) || bad(r->k_weight)) return DMA_ERR_INVALID_ARG;
  if (r->rot % 16 != 0) return DMA_ERR_UNSUPPORTED;
  return DMA_OK;
}

namespace {

bool ok_ptr(const void* q) { return q != nullptr && (reinterpret_cast<uintptr_t>(q) & 15u) == 0; }
bool null_or_ok(const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15u) == 0; }

// Checks and arguments that forward and backward have in common.
dma_status_t prep_args(const dma_params_t* p, const dma_prep_t* r, PrepArgs* a) {
  if (p == nullptr || p->B < 1 || p->H < 1 || p->Hkv < 1 || p->N < 1) return DMA_ERR_INVALID_ARG;
  if (p->Nq != p->N || p->H % p->Hkv != 0) return DMA_ERR_INVALID_ARG;
  if (p->dtype != DMA_BF16 && p->dtype != DMA_F32) return DMA_ERR_INVALID_ARG;
  if (p->d != 64 && p->d != 128) return DMA_ERR_UNSUPPORTED;
  if ((int64_t)p->B * p->H > 65535 || p->N > (1 << 24)) return DMA_ERR_UNSUPPORTED;
  dma_status_t st = check_prep(r, p->d);
  if (st != DMA_OK) return st;
  memset(a, 0, sizeof(*a));
  a->inv_freq = r->inv_freq;
  a->positions = r->positions;
  a->weight[0] = r->q_weight;
  a->weight[1] = r->k_weight;
  a->eps = r->eps;
  a->B = p->B; a->H = p->H; a->Hkv = p->Hkv; a->N = p->N; a->rot = r->rot; a->first = r->first;
  a->inter = r->interleaved != 0;
  return DMA_OK;
}

// Rows of d channels at the given strides do not overlap (a sufficient test: each dimension, from the
// closest to the widest, steps over all that lies below it).
bool rows_apart(const int64_t (&st)[3], int B, int N, int heads, int d) {
  int64_t step[3] = {st[0], st[1], st[2]}, size[3] = {B, N, heads};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (step[j] < step[i]) {
        const int64_t a = step[i], b = size[i];
        step[i] = step[j]; size[i] = size[j];
        step[j] = a; size[j] = b;
      }
  int64_t span = d;   // elements from the first to past the last of what lies below
  for (int i = 0; i < 3; ++i) {
    if (size[i] == 1) continue;
    if (step[i] < span) return false;
    span += step[i] * (size[i] - 1);
  }
  return true;
}

}  // namespace
}  // namespace dma

using namespace dma;

extern "C" {

dma_status_t dma_prep(const dma_params_t* p, const dma_prep_t* r, const dma_prep_strides_t* st, const void* q,
                      const void* k, const void* v, void* Q, void* K, void* V, void* stream) {
  PrepArgs a;
  dma_status_t e = prep_args(p, r, &a);
  if (e != DMA_OK) return e;
  const bool bf16 = p->dtype == DMA_BF16;
  if (st == nullptr || !ok_ptr(q) || !ok_ptr(k) || !ok_ptr(Q) || !ok_ptr(K)) return DMA_ERR_INVALID_ARG;
  if ((v == nullptr) != (V == nullptr) || !null_or_ok(v) || !null_or_ok(V)) return DMA_ERR_INVALID_ARG;
  if (!check_strides(st->q, bf16) || !check_strides(st->k, bf16) || (v != nullptr && !check_strides(st->v, bf16)))
    return DMA_ERR_INVALID_ARG;
  a.in[0] = q; a.in[1] = k; a.in[2] = v;
  a.out[0] = Q; a.out[1] = K; a.out[2] = V;
  for (int i = 0; i < 3; ++i) {
    a.stride[0][i] = st->q[i];
    a.stride[1][i] = st->k[i];
    a.stride[2][i] = v != nullptr ? st->v[i] : 0;
  }
  return launch_prep_fwd(a, bf16, p->d, (cudaStream_t)stream) == cudaSuccess ? DMA_OK : DMA_ERR_CUDA;
}

dma_status_t dma_prep_workspace_size(const dma_params_t* p, const dma_prep_t* r, size_t* bytes) {
  PrepArgs a;
  dma_status_t e = prep_args(p, r, &a);
  if (e != DMA_OK) return e;
  if (bytes == nullptr) return DMA_ERR_INVALID_ARG;
  *bytes = (size_t)2 * kPrepMaxBlocks * p->d * sizeof(float);
  return DMA_OK;
}

dma_status_t dma_prep_bwd(const dma_params_t* p, const dma_prep_t* r, const dma_prep_strides_t* st,
                          const dma_prep_strides_t* gst, const void* q, const void* k, const void* dQ,
                          const void* dK, const void* dV, const float* dV_gate, void* dq, void* dk, void* dv,
                          float* dq_weight, float* dk_weight, void* workspace, size_t workspace_bytes, void* stream) {
  PrepArgs a;
  dma_status_t e = prep_args(p, r, &a);
  if (e != DMA_OK) return e;
  const bool bf16 = p->dtype == DMA_BF16;
  if (st == nullptr || gst == nullptr || !ok_ptr(dQ) || !ok_ptr(dK) || !ok_ptr(dq) || !ok_ptr(dk)) return DMA_ERR_INVALID_ARG;
  if (r->q_weight != nullptr ? !ok_ptr(q) : !null_or_ok(q)) return DMA_ERR_INVALID_ARG;
  if (r->k_weight != nullptr ? !ok_ptr(k) : !null_or_ok(k)) return DMA_ERR_INVALID_ARG;
  if ((dv == nullptr) != (dV == nullptr) || (dv == nullptr && dV_gate != nullptr)) return DMA_ERR_INVALID_ARG;
  if (!null_or_ok(dv) || !null_or_ok(dV) || !null_or_ok(dV_gate)) return DMA_ERR_INVALID_ARG;
  if (!null_or_ok(dq_weight) || !null_or_ok(dk_weight)) return DMA_ERR_INVALID_ARG;
  if ((dq_weight != nullptr && r->q_weight == nullptr) || (dk_weight != nullptr && r->k_weight == nullptr))
    return DMA_ERR_INVALID_ARG;
  if ((q != nullptr && !check_strides(st->q, bf16)) || (k != nullptr && !check_strides(st->k, bf16)))
    return DMA_ERR_INVALID_ARG;
  if (!check_strides(gst->q, bf16) || !check_strides(gst->k, bf16) || (dv != nullptr && !check_strides(gst->v, bf16)))
    return DMA_ERR_INVALID_ARG;
  if (!rows_apart(gst->q, p->B, p->N, p->H, p->d) || !rows_apart(gst->k, p->B, p->N, p->Hkv, p->d) ||
      (dv != nullptr && !rows_apart(gst->v, p->B, p->N, p->Hkv, p->d)))
    return DMA_ERR_INVALID_ARG;
  if (!ok_ptr(workspace) || workspace_bytes < (size_t)2 * kPrepMaxBlocks * p->d * sizeof(float))
    return DMA_ERR_WORKSPACE;
  a.in[0] = q; a.in[1] = k;
  a.grad[0] = dQ; a.grad[1] = dK; a.grad[2] = dV;
  a.dv_gate = dV_gate;
  a.out[0] = dq; a.out[1] = dk; a.out[2] = dv;
  a.part = static_cast<float*>(workspace);
  for (int i = 0; i < 3; ++i) {
    a.stride[0][i] = st->q[i];
    a.stride[1][i] = st->k[i];
    a.gstride[0][i] = gst->q[i];
    a.gstride[1][i] = gst->k[i];
    a.gstride[2][i] = dv != nullptr ? gst->v[i] : 0;
  }
  return launch_prep_bwd(a, bf16, p->d, dq_weight, dk_weight, (cudaStream_t)stream) == cudaSuccess ? DMA_OK
                                                                                                   : DMA_ERR_CUDA;
}

}  // extern "C"
