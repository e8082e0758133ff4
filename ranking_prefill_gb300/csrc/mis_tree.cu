// Attention of drafted token trees over a paged K/V cache, sm_103a.
//
// Row i of request b sees the cached rows [0, L_b) and, among the request's
// own new rows, its ancestors and itself:
//     o_i = sum_j p_ij v_j,  p_ij = exp(s_ij - lse_i),  s_ij = scale q_i k_j.
// One warp per (row, query head) walks the visible keys with a running
// maximum and sum; a lane owns D / 32 elements of the head.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "mis_internal.h"
#include "mis_ptx.cuh"

namespace mis {
namespace {

using namespace dev;

struct TreeParams {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  __nv_bfloat16* o;
  float* lse;
  int64_t qs, ks, vs, os;
  const __nv_bfloat16* kc;
  const __nv_bfloat16* vc;
  int64_t page_stride, row_stride, head_stride;
  int32_t n_pages, page_size, max_pages;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* cache_len;
  const int32_t* cu;
  const int32_t* parents;
  int32_t B, T, Hq, group, max_nodes;
  float scale;
  uint32_t* status;
};

template <int D>
__global__ void __launch_bounds__(128) mis_tree_attn_kernel(const TreeParams p) {
  griddep_wait();
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.y, h = blockIdx.x * 4 + warp;
  if (h >= p.Hq) return;
  const int i = blockIdx.z, r0 = p.cu[b], n = p.cu[b + 1] - r0, L = p.cache_len[b];
  if (r0 < 0 || n < 0 || n > p.max_nodes || r0 + n > p.T || L < 0 ||
      L > (int64_t)p.max_pages * p.page_size) {
    if (lane == 0) raise_status(p.status, kDevIndex, 0x40);
    return;
  }
  if (i >= n) return;
  const int kvh = h / p.group;
  float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(p.q[(int64_t)(r0 + i) * p.qs + h * D + lane * E + e]);
    o[e] = 0.f;
  }
  auto key = [&](const __nv_bfloat16* kr, const __nv_bfloat16* vr) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], __bfloat162float(kr[lane * E + e]), s);
#pragma unroll
    for (int w = 16; w; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    s *= p.scale;
    const float mn = fmaxf(m, s);
    if (mn == -INFINITY && s == s) return;
    const float a = m == -INFINITY ? 0.f : expf(m - mn), pr = expf(s - mn);
    m = mn;
    l = l * a + pr;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * a + pr * __bfloat162float(vr[lane * E + e]);
  };
  auto parent = [&](int j) { return p.parents ? p.parents[r0 + j] : j - 1; };
  if (parent(i) != MIS_TREE_UNUSED) {
    for (int j = 0; j < L; ++j) {
      const int page = p.table[b * p.table_stride + j / p.page_size];
      if (page < 0 || page >= p.n_pages) {
        if (lane == 0) raise_status(p.status, kDevIndex, 0x41);
        continue;
      }
      const int64_t at = page * p.page_stride + (j % p.page_size) * p.row_stride + kvh * p.head_stride;
      key(p.kc + at, p.vc + at);
    }
    for (int j = i; j >= 0;) {
      key(p.k + (int64_t)(r0 + j) * p.ks + kvh * D, p.v + (int64_t)(r0 + j) * p.vs + kvh * D);
      int up = parent(j);
      if (up >= j || up < MIS_TREE_UNUSED) {
        if (lane == 0) raise_status(p.status, kDevIndex, 0x42);
        up = MIS_TREE_ROOT;
      }
      j = up >= 0 && parent(up) != MIS_TREE_UNUSED ? up : -1;
    }
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;   // NaN stays
#pragma unroll
  for (int e = 0; e < E; ++e)
    p.o[(int64_t)(r0 + i) * p.os + h * D + lane * E + e] = __float2bfloat16(o[e] * inv);
  if (p.lse && lane == 0) p.lse[(int64_t)h * p.T + r0 + i] = l != 0.f ? m + logf(l) : -INFINITY;
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

mis_status_t check_desc(const mis_tree_desc* d, const mis_paged_cache* c) {
  if (!d) return MIS_ERR_INVALID_ARG;
  const mis_status_t cs = check_paged_cache(c);
  if (cs != MIS_OK) return cs;
  if (d->B < 1 || d->T < 0 || d->Hq < 1 || d->max_nodes < 1 || !std::isfinite(d->scale))
    return MIS_ERR_INVALID_ARG;
  if (d->max_nodes > MIS_TREE_MAX_NODES) return MIS_ERR_UNSUPPORTED;
  if (d->Hq % c->Hkv) return MIS_ERR_SHAPE;
  return MIS_OK;
}

}  // namespace
}  // namespace mis

using namespace mis;

extern "C" size_t mis_tree_attention_workspace_size(const mis_tree_desc* desc,
                                                    const mis_paged_cache* cache) {
  return check_desc(desc, cache) == MIS_OK ? kStatusBytes : 0;
}

extern "C" mis_status_t mis_tree_attention_fwd(
    const mis_tree_desc* desc, const mis_paged_cache* cache, const void* q, const void* k,
    const void* v, void* o, float* lse, int64_t q_row_stride, int64_t k_row_stride,
    int64_t v_row_stride, int64_t o_row_stride, const int32_t* block_table, int32_t max_pages,
    int64_t block_table_stride, const int32_t* cache_len, const int32_t* cu_nodes,
    const int32_t* parents, void* workspace, size_t ws_bytes, void* stream) {
  const mis_status_t ds = check_desc(desc, cache);
  if (ds != MIS_OK) return ds;
  if (max_pages < 1) return MIS_ERR_INVALID_ARG;
  if ((int64_t)max_pages * cache->page_size > 0x7fffffff || block_table_stride < max_pages)
    return MIS_ERR_SHAPE;
  if (!block_table || !cache_len || !cu_nodes || !aligned(block_table, 4) ||
      !aligned(cache_len, 4) || !aligned(cu_nodes, 4) || !aligned(parents, 4) || !aligned(lse, 4))
    return MIS_ERR_INVALID_ARG;
  const int D = cache->D;
  const int64_t wq = (int64_t)desc->Hq * D, wk = (int64_t)cache->Hkv * D;
  if (q_row_stride < wq || o_row_stride < wq || k_row_stride < wk || v_row_stride < wk)
    return MIS_ERR_SHAPE;
  if ((q_row_stride | k_row_stride | v_row_stride | o_row_stride) & 7) return MIS_ERR_SHAPE;
  if (desc->T > 0) {
    if (!q || !k || !v || !o) return MIS_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16))
      return MIS_ERR_INVALID_ARG;
  }
  if (!workspace || !aligned(workspace, 256) ||
      ws_bytes < mis_tree_attention_workspace_size(desc, cache))
    return MIS_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(workspace, 0, 8, st) != cudaSuccess) return MIS_ERR_CUDA;
  if (desc->T == 0) return MIS_OK;
  TreeParams p;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.qs = q_row_stride; p.ks = k_row_stride; p.vs = v_row_stride; p.os = o_row_stride;
  p.kc = static_cast<const __nv_bfloat16*>(cache->k);
  p.vc = static_cast<const __nv_bfloat16*>(cache->v);
  p.page_stride = cache->page_stride; p.row_stride = cache->row_stride;
  p.head_stride = cache->head_stride;
  p.n_pages = cache->n_pages; p.page_size = cache->page_size; p.max_pages = max_pages;
  p.table = block_table; p.table_stride = block_table_stride;
  p.cache_len = cache_len; p.cu = cu_nodes; p.parents = parents;
  p.B = desc->B; p.T = desc->T; p.Hq = desc->Hq; p.group = desc->Hq / cache->Hkv;
  p.max_nodes = desc->max_nodes;
  p.scale = desc->scale != 0.f ? desc->scale : 1.f / std::sqrt((float)D);
  p.status = static_cast<uint32_t*>(workspace);
  const dim3 grid((unsigned)(desc->Hq + 3) / 4, (unsigned)desc->B, (unsigned)desc->max_nodes);
  if (desc->B > 65535) return MIS_ERR_UNSUPPORTED;
  try {
    const cudaError_t e = D == 128 ? launch_pdl(mis_tree_attn_kernel<128>, grid, dim3(128), 0, st, p)
                                   : launch_pdl(mis_tree_attn_kernel<64>, grid, dim3(128), 0, st, p);
    return e == cudaSuccess ? MIS_OK : MIS_ERR_CUDA;
  } catch (...) {
    return MIS_ERR_CUDA;
  }
}
