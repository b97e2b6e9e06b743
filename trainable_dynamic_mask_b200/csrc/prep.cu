// From the projections to the attention's inputs, and the gradients on their way back.
//
// Forward, per head row x of a query or key at position n (the norm where a weight g is given):
//   r = (mean(x^2) + eps)^(-1/2),  y = x r g,  out = R(n) y,
// R(n) the rotation of the first rot channels, pair i by the angle n f_i; value rows are copied.  Rows
// are read wherever the projection left them (strides) and written as [B, heads, N, d], so the
// transposition costs no pass of its own.
// Backward, with dy = R(n)^T dOut:  dx = r (g dy - x r^2 mean(x g dy)),  dg = sum over rows of dy x r,
// and dv = dV + dV_gate.  r is formed again from x, which the norm's gradient reads anyway.
//
// Both are bound by memory where there are many rows: every row is read once and written once, and nothing
// else moves.  16384 tokens of 16 + 8 + 8 heads of 128 channels in bf16: forward 268 MB in 51 us (5.2 TB/s, 80 %
// of the copy rate of 6.56), backward 436 MB in 89 us (4.9 TB/s, 74 %); the rest is issue slots (71 % of them
// in the forward).  In a graph from a cold L2, forward with three CTAs an SM as here 60 us, with two 64, with four
// (64 registers) 67; backward with two as here 93, with one 122.
// Small calls are bound by the way through the binding and the launch: 8 tokens in 8.4 us, 5 in a
// graph (the backward has a second launch, of the weights' sums, that starts while the first ends).
#include <math.h>
#include <string.h>

#include "rows.cuh"

namespace dma {
namespace {

// Dense outputs [B, heads, N, D].
struct DenseDest {
  static constexpr int kDepth = 3;   // with two or four 0.2 and 1 us more at 16384 tokens
  struct Token {
    int position;
    unsigned b, n;
  };
  void* out[3];
  const int32_t* positions;
  unsigned N;
  int H, Hkv, D, size, first;
  DMA_DEVINL bool enter(const Walk& at, Token& t) const {
    t.b = at.b;
    t.n = at.n;
    t.position = positions ? __ldg(positions + at.tok) : first + (int)t.n;
    return true;
  }
  DMA_DEVINL void* row(int part, const Token& t) const {
    return (char*)out[part] + (((size_t)t.b * (part == 0 ? H : Hkv)) * N + t.n) * D * size;
  }
  DMA_DEVINL size_t step(int) const { return (size_t)N * D; }
};

template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kRwThreads, 3)
prep_fwd_kernel(const __grid_constant__ PrepArgs a, const __grid_constant__ DenseDest dest, int wt) {
  extern __shared__ __align__(128) unsigned char smem[];
  walk_rows<T, D, INTER>(a, dest, wt, blockIdx.x, gridDim.x, smem);
}

template <typename T> constexpr int bwd_rows() { return sizeof(T) == 2 ? 4 : 2; }
// a row's gradient, and its input or (values) the gate's share
template <typename T> using BwdRing = RowRing<sizeof(T) == 2 ? 3 : 4, bwd_rows<T>(), 2>;

// Warps walk over the tokens in a fixed order, so the partial sums of the weights' gradients do not depend on
// scheduling.  A lane adds up its own rows in float32, one in 4736 of all (148 SMs, 128 channels; one in 9472 of 64):
// 55 for 16384 tokens of 16 heads, some 50 000 for as many as 180 GB hold, each addition off by 2^-24 at most.
template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kRwThreads, 2)
prep_bwd_kernel(const __grid_constant__ PrepArgs a, int wt) {
  constexpr int L = D / 8, RPW = 32 / L, U = bwd_rows<T>(), SECOND = sizeof(T) / 2;
  using Ring = BwdRing<T>;
  extern __shared__ __align__(128) unsigned char ring_smem[];
  __shared__ __align__(16) float2 tab[kRwWarps][D / 2 + kTabPad];
  __shared__ uint64_t rate[D / 2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, grp = lane / L, e = (lane % L) * 8;
  const bool upper = e >= a.rot >> 1;
  pdl_trigger();
  auto ready = [&]() {
    for (int k = tid; k < a.rot >> 1; k += kRwThreads) rate[k] = turn_rate(__ldg(a.inv_freq + k));
    if (lane < kTabPad) tab[warp][D / 2 + lane] = make_float2(1.f, 0.f);
    __syncthreads();
  };
  auto send = [&](const Walk& at, unsigned char* place) {
    const int part = at.part(), h = at.within(part) * (RPW * U) + grp;
    const int heads = part == 0 ? a.H : a.Hkv, left = heads - h;
    const size_t dense = (((size_t)at.b * heads + h) * at.N + at.n) * D + e, step = (size_t)RPW * at.N * D;
    const T* base = (const T*)a.grad[part];
#pragma unroll
    for (int u = 0; u < U; ++u)
      Ring::copy(place + u * Ring::kRow, 0, u * RPW < left ? base + dense + u * step : base, u * RPW < left);
    if (part == 2) {
      if (a.dv_gate == nullptr) return;
#pragma unroll
      for (int u = 0; u < U; ++u)
        Ring::copy(place + u * Ring::kRow, SECOND, u * RPW < left ? a.dv_gate + dense + u * step : a.dv_gate,
                   u * RPW < left);
    } else if (a.weight[part] != nullptr) {
      const long long sh = a.stride[part][2];
      const T* x = (const T*)a.in[part];
      const T* src = x + at.b * a.stride[part][0] + at.n * a.stride[part][1] + h * sh + e;
#pragma unroll
      for (int u = 0; u < U; ++u)
        Ring::copy(place + u * Ring::kRow, SECOND, u * RPW < left ? src + u * RPW * sh : x, u * RPW < left);
    }
  };
  float gw[2][8];   // this lane's share of the weights' gradients
#pragma unroll
  for (int i = 0; i < 8; ++i) gw[0][i] = gw[1][i] = 0.f;
  LaneTurn turn;
  const int start = lane_start<D>(turn, a.rot, INTER, lane);
  unsigned have = 0xffffffffu;
  auto work = [&](const Walk& at, const unsigned char* place) {
    if (have != at.tok) {
      have = at.tok;
      token_table(rate, a.rot >> 1, a.positions ? __ldg(a.positions + at.tok) : a.first + (int)at.n, tab[warp]);
      lane_turn<INTER>(turn, tab[warp], start, upper, true);
    }
    const int part = at.part(), h = at.within(part) * (RPW * U) + grp, left = (part == 0 ? a.H : a.Hkv) - h;
    const long long sh = a.gstride[part][2];
    T* dst = (T*)a.out[part] + at.b * a.gstride[part][0] + at.n * a.gstride[part][1] + h * sh + e;
    if (part == 2) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u * RPW < left) {
          if (a.dv_gate != nullptr) {
            Chan8 v = channels8(Ring::template read<T>(place + u * Ring::kRow, 0));
            const Chan8 w = channels8(Ring::template read<float>(place + u * Ring::kRow, SECOND));
#pragma unroll
            for (int i = 0; i < 8; ++i) v.v[i] += w.v[i];
            store8(dst, v);
          } else {
            store_raw8(dst, Ring::template read<T>(place + u * Ring::kRow, 0));
          }
        }
        dst += RPW * sh;
      }
      return;
    }
    const T* wp = (const T*)a.weight[part];
    Chan8 g;
    if (wp != nullptr) g = channels8(load_raw8(wp + e));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      Chan8 y = rotate8<INTER>(channels8(Ring::template read<T>(place + u * Ring::kRow, 0)), turn);
      if (wp != nullptr) {
        const Chan8 x = channels8(Ring::template read<T>(place + u * Ring::kRow, SECOND));   // zeros past the last head
        float t[8], dot = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          t[i] = x.v[i] * y.v[i];
          dot = fmaf(t[i], g.v[i], dot);
        }
        const float rn = rsqrtf(row_dot<L>(x, x) * (1.f / D) + a.eps);
        const float k = row_sum<L>(dot) * (-1.f / D) * rn * rn * rn;
        if (part == 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i) gw[0][i] = fmaf(t[i], rn, gw[0][i]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) gw[1][i] = fmaf(t[i], rn, gw[1][i]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) y.v[i] = fmaf(x.v[i], k, y.v[i] * (g.v[i] * rn));
      }
      if (u * RPW < left) store8(dst, y);
      dst += RPW * sh;
    }
  };
  Ring::run(Walk(a, RPW * U, wt, blockIdx.x, gridDim.x), ring_smem, send, ready, work);
  // the block's partial sums of dg, one row of the workspace each, in the ring's place
  float* red = reinterpret_cast<float*>(ring_smem);   // [kRwWarps * RPW][D]
  static_assert(Ring::kBytes >= kRwWarps * RPW * D * 4, "the sums fit into the ring");
  cp_async_wait<0>();
#pragma unroll
  for (int part = 0; part < 2; ++part) {
    if (!a.weight[part]) continue;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) red[(warp * RPW + grp) * D + e + i] = gw[part][i];
    __syncthreads();
    for (int c = tid; c < D; c += kRwThreads) {
      float v = 0.f;
#pragma unroll
      for (int q = 0; q < kRwWarps * RPW; ++q) v += red[q * D + c];
      a.part[((size_t)part * gridDim.x + blockIdx.x) * D + c] = v;
    }
  }
}

// dg[c] = sum over blocks, in double precision: at most kPrepMaxBlocks terms per channel.  A block takes
// eight channels (a 32-byte sector of every partial row), so that a thread has only a few loads to wait for.
__global__ void __launch_bounds__(1024)
prep_reduce_kernel(const float* part, float* __restrict__ dq_weight, float* __restrict__ dk_weight, int n_blocks,
                   int D) {
  __shared__ double red[32][8];
  const int tid = threadIdx.x, c = blockIdx.x * 8 + (tid & 7), w = tid >> 3;
  float* out = blockIdx.y == 0 ? dq_weight : dk_weight;
  pdl_wait();
  if (out == nullptr) return;
  const float* p = part + (size_t)blockIdx.y * n_blocks * D + c;
  double v = 0.0;
#pragma unroll 5
  for (int i = w; i < n_blocks; i += 128) v += (double)p[(size_t)i * D];
  v += __shfl_xor_sync(0xffffffffu, v, 8);
  v += __shfl_xor_sync(0xffffffffu, v, 16);
  if ((tid & 31) < 8) red[tid >> 5][tid & 7] = v;
  __syncthreads();
  if (tid < 8) {
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += red[i][tid];
    out[c] = (float)s;
  }
}

template <typename T, int D>
cudaError_t launch_fwd(const PrepArgs& a, cudaStream_t s) {
  DenseDest d = {};
  for (int i = 0; i < 3; ++i) d.out[i] = a.out[i];
  d.positions = a.positions;
  d.N = (unsigned)a.N;
  d.H = a.H; d.Hkv = a.Hkv; d.D = D; d.size = (int)sizeof(T); d.first = a.first;
  int wt;
  const int blocks = walk_blocks((long long)a.B * a.N, 3, &wt);
  constexpr int smem = FwdRing<T, DenseDest::kDepth>::kBytes;
  auto kernel = a.inter ? prep_fwd_kernel<T, D, true> : prep_fwd_kernel<T, D, false>;
  const cudaError_t e = ensure_smem_limit(kernel, smem);
  if (e != cudaSuccess) return e;
  kernel<<<blocks, kRwThreads, smem, s>>>(a, d, wt);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_bwd(const PrepArgs& a, float* dqw, float* dkw, cudaStream_t s) {
  int wt;
  int blocks = walk_blocks((long long)a.B * a.N, 2, &wt);
  if (blocks > kPrepMaxBlocks) blocks = kPrepMaxBlocks;
  auto kernel = a.inter ? prep_bwd_kernel<T, D, true> : prep_bwd_kernel<T, D, false>;
  cudaError_t e = ensure_smem_limit(kernel, BwdRing<T>::kBytes);
  if (e != cudaSuccess) return e;
  kernel<<<blocks, kRwThreads, BwdRing<T>::kBytes, s>>>(a, wt);
  e = cudaGetLastError();
  if (e != cudaSuccess || (dqw == nullptr && dkw == nullptr)) return e;
  return launch_after(prep_reduce_kernel, dim3(D / 8, 2), 1024, 0, s, 1, (const float*)a.part, dqw, dkw, blocks, D);
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
  if ((int64_t)p->B * p->H > 65535 || p->N > (1 << 24) || (int64_t)p->B * p->N >= ((int64_t)1 << 31))
    return DMA_ERR_UNSUPPORTED;
  dma_status_t st = check_prep(r, p->d);
  if (st != DMA_OK) return st;
  if (r->positions == nullptr && (int64_t)r->first + p->N > ((int64_t)1 << 31)) return DMA_ERR_INVALID_ARG;
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
  return cuda_status(launch_prep_fwd(a, bf16, p->d, (cudaStream_t)stream));
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
  if (st == nullptr || gst == nullptr || !ok_ptr(dQ) || !ok_ptr(dK) || !ok_ptr(dq) || !ok_ptr(dk))
    return DMA_ERR_INVALID_ARG;
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
  return cuda_status(launch_prep_bwd(a, bf16, p->d, dq_weight, dk_weight, (cudaStream_t)stream));
}

}  // extern "C"
