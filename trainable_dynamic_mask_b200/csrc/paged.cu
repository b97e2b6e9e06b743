// Entry points of the paged cache: argument checks, workspace plan, dispatch.
#include <string.h>

#include "internal.h"

namespace dma {
namespace {

bool ok_ptr(const void* q) { return q != nullptr && (reinterpret_cast<uintptr_t>(q) & 15u) == 0; }

dma_status_t paged_plan(const dma_params_t* p, const dma_pages_t* c, PagedPlan* P) {
  Plan base;
  dma_status_t st = make_plan(p, &base);
  if (st != DMA_OK) return st;
  if (p->Nq != 1 || c == nullptr) return DMA_ERR_INVALID_ARG;
  if (!ok_ptr(c->K) || !ok_ptr(c->V) || !ok_ptr(c->delta) || !ok_ptr(c->table) || !ok_ptr(c->lens))
    return DMA_ERR_INVALID_ARG;
  if (c->n_pages < 1 || c->max_pages < 1 || c->page < 1 || c->prefix < 0) return DMA_ERR_INVALID_ARG;
  if ((p->w < p->N ? p->w : p->N) > kPagedMostKept * p->d) return DMA_ERR_UNSUPPORTED;
  if (c->page < 16 || c->page > 1024 || (c->page & (c->page - 1)) != 0) return DMA_ERR_UNSUPPORTED;
  if ((int64_t)c->n_pages * c->page >= ((int64_t)1 << 31) || (int64_t)c->n_pages * p->H >= ((int64_t)1 << 31))
    return DMA_ERR_UNSUPPORTED;
  if (p->N > (int64_t)c->max_pages * c->page || c->prefix % c->page != 0 || c->prefix > p->N)
    return DMA_ERR_INVALID_ARG;
  memset(P, 0, sizeof(*P));
  P->B = base.B; P->H = base.H; P->Hkv = base.Hkv; P->d = base.d; P->w = base.w; P->N = base.N; P->G = base.G;
  P->scale = base.scale;
  P->bf16 = base.bf16;
  P->w_heads = base.w_heads;
  P->K = static_cast<char*>(c->K);
  P->V = static_cast<char*>(c->V);
  P->delta = c->delta;
  P->table = c->table;
  P->lens = c->lens;
  P->n_pages = c->n_pages;
  P->max_pages = c->max_pages;
  P->prefix = c->prefix;
  while ((1 << P->page_shift) < c->page) ++P->page_shift;
  // the candidates are multiplied with all sequences' queries on the tensor cores, in bf16
  P->shared = c->prefix > 0 && P->bf16 && P->B > 1;
  const int rest = P->shared ? P->N - P->prefix : P->N;
  P->sel_len = P->w < rest ? P->w : rest;
  if (P->sel_len < 1) P->sel_len = 1;
  P->cand_len = P->shared ? (P->w < P->prefix ? P->w : P->prefix) : 0;
  P->n_split = (P->sel_len + kPagedSplit - 1) / kPagedSplit;
  // Candidates: the tcgen05 kernel (64 sequences a CTA, one CTA an SM) where every SM has 128 or more of them to
  // work on, else the smaller CTAs of paged_attn.cu.  Attention over 2048 candidates of 32 heads, 64 sequences:
  // 31.4 us against 42.3 (33.4 with 64 sequences a CTA there too); 1024 of 16 heads, 128 sequences: 26.3 against
  // 29.5; but 512 of 16 heads, 48 sequences: 19.1 against 16.4, 100 of 32 heads, 40 sequences: 17.4 against 15.6.
  // (a fixed count of 148 SMs keeps the workspace's plan independent of the device)
  const int64_t tiles = (int64_t)P->H * ((P->B + 63) / 64);
  P->cand_tc = P->shared && P->B > 32 && tiles * P->cand_len >= 148 * 128;
  if (P->cand_tc) {
    // 512 candidates a CTA, or 256 where that takes less than 4/3 as many rounds
    auto rounds = [&](int split) { return (tiles * ((P->cand_len + split - 1) / split) + 147) / 148; };
    P->cand_split = 3 * rounds(256) < 4 * rounds(512) ? 256 : 512;
  } else {
    // 256, or as few as 64 where that leaves SMs without one
    P->cand_split = 256;
    const int64_t small = (int64_t)P->H * ((P->B + 31) / 32);
    while (P->cand_split > 64 && small * ((P->cand_len + P->cand_split - 1) / P->cand_split) < 148) P->cand_split /= 2;
  }
  P->n_psplit = (P->cand_len + P->cand_split - 1) / P->cand_split;
  const size_t BH = (size_t)P->B * P->H;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  };
  P->off_status = take(256);
  P->off_rows = take(BH * 16);
  P->off_sel = take(BH * P->sel_len * 4);
  P->off_cand = take((size_t)P->H * P->cand_len * 4);
  P->off_ent = take(BH * P->sel_len * 8);
  P->off_crow = take((size_t)P->H * 4);
  P->off_cent = take((size_t)P->H * P->cand_len * 8);
  P->off_tail = take((size_t)P->H * (kPagedTail + 1) * 8);
  P->off_count = take(BH * 4);
  P->off_part = take(BH * (P->n_psplit + P->n_split) * (size_t)(P->d + 4) * 4);
  P->bytes = off;
  return DMA_OK;
}

dma_status_t check_ws(const PagedPlan& P, const void* ws, size_t bytes) {
  return ok_ptr(ws) && bytes >= P.bytes ? DMA_OK : DMA_ERR_WORKSPACE;
}

}  // namespace
}  // namespace dma

using namespace dma;

extern "C" {

dma_status_t dma_paged_layout(const dma_params_t* p, const dma_pages_t* c, dma_paged_layout_t* L) {
  PagedPlan P;
  dma_status_t st = paged_plan(p, c, &P);
  if (st != DMA_OK) return st;
  if (L == nullptr) return DMA_ERR_INVALID_ARG;
  L->bytes = P.bytes;
  L->off_status = P.off_status;
  L->off_rows = P.off_rows;
  L->off_sel = P.off_sel;
  L->off_cand = P.off_cand;
  L->sel_len = P.sel_len;
  L->cand_len = P.cand_len;
  return DMA_OK;
}

dma_status_t dma_paged_append(const dma_params_t* p, const dma_pages_t* c, const dma_prep_t* r,
                              const dma_prep_strides_t* strides, int32_t T, const int32_t* starts, const void* q,
                              const void* k, const void* v, const void* Delta, const float* A, void* Q,
                              void* workspace, size_t workspace_bytes, void* stream) {
  PagedPlan P;
  dma_status_t st = paged_plan(p, c, &P);
  if (st != DMA_OK) return st;
  if ((st = check_prep(r, P.d)) != DMA_OK) return st;
  if (r->positions != nullptr || strides == nullptr || T < 0) return DMA_ERR_INVALID_ARG;
  if (starts == nullptr ? T != P.B : !ok_ptr(starts)) return DMA_ERR_INVALID_ARG;
  if (P.H > kGateMaxH) return DMA_ERR_UNSUPPORTED;
  if ((st = check_ws(P, workspace, workspace_bytes)) != DMA_OK) return st;
  if (T == 0) return DMA_OK;   // no token, no tensors
  if ((q == nullptr) != (Q == nullptr) || (q != nullptr && (!ok_ptr(q) || !ok_ptr(Q)))) return DMA_ERR_INVALID_ARG;
  if (!ok_ptr(k) || !ok_ptr(v) || !ok_ptr(Delta) || !ok_ptr(A)) return DMA_ERR_INVALID_ARG;
  if ((q != nullptr && !check_strides(strides->q, P.bf16)) || !check_strides(strides->k, P.bf16) ||
      !check_strides(strides->v, P.bf16))
    return DMA_ERR_INVALID_ARG;
  PagedAppendArgs a;
  a.r = *r;
  a.st = *strides;
  a.T = T;
  a.starts = starts;
  a.q = q; a.k = k; a.v = v; a.Delta = Delta; a.A = A; a.Q = Q;
  return cuda_status(launch_paged_append(P, a, workspace, (cudaStream_t)stream));
}

dma_status_t dma_paged_topk(const dma_params_t* p, const dma_pages_t* c, void* workspace, size_t workspace_bytes,
                            void* stream) {
  PagedPlan P;
  dma_status_t st = paged_plan(p, c, &P);
  if (st != DMA_OK) return st;
  if ((st = check_ws(P, workspace, workspace_bytes)) != DMA_OK) return st;
  return cuda_status(launch_paged_topk(P, workspace, (cudaStream_t)stream));
}

dma_status_t dma_paged_attn(const dma_params_t* p, const dma_pages_t* c, const void* Q, void* workspace,
                            size_t workspace_bytes, void* O, float* LSE, void* stream) {
  PagedPlan P;
  dma_status_t st = paged_plan(p, c, &P);
  if (st != DMA_OK) return st;
  if (!ok_ptr(Q) || !ok_ptr(O) || !ok_ptr(LSE)) return DMA_ERR_INVALID_ARG;
  if ((st = check_ws(P, workspace, workspace_bytes)) != DMA_OK) return st;
  return cuda_status(launch_paged_attn(P, Q, workspace, O, LSE, (cudaStream_t)stream));
}

}  // extern "C"
