// 8-bit paged K/V cache, sm_103a: rows quantised as they are stored (K normed
// and rotated on the way), and rows read back as bf16.
//
// A (row, kv head) is held as D e4m3 codes and one exponent e:
//   a = max |finite x|,  e = least integer in [-56, 120] with a <= 448 * 2^e,
//   code = e4m3(x * 2^-e) (nearest, ties to even), value = code * 2^e.
// The scale is a power of two because e4m3 is a float: a finer scale would not
// make its codes finer, while this one is a byte, x * 2^-e is exact, and the
// value is exact in bf16 (and the codes are what attention multiplies).
//
// Both kernels touch every byte once, so HBM bounds them: D / 16 lanes share a
// row of a head in the store (maximum and mean in 2 or 3 exchanges, as the
// rotation's pairs lie in a lane), and D / 16 lanes read one back. 128K rows of 8
// heads, 128 wide, are stored in 146 us and read back in 120 (5.5 and 6.7 TB/s of
// the 6.8 that a copy reaches); a few rows cost a launch, 2.3 to 2.5 us. Narrow rows
// are bound by one chain a thread (slot, row, exchange, store) at 512 threads an SM:
// 128K rows of 1 x 64 are stored in 25 us, 19 without norm and angles, and read in 13,
// where the bytes take 7.6 each way; of 4 x 128 by the look at the indices, 97 and 90
// (60).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "mis_internal.h"
#include "mis_ptx.cuh"
#include "mis_rows.cuh"

namespace mis {
namespace {

using namespace dev;

constexpr int kThreads = 256, kStoreThreads = 128;
// One block looks over every index beside the copy where that takes no longer
// than the copy. Else the status word is cleared by a node of its own and the
// rows' own threads raise it. Both ways, stored and read back: 32 rows of 8 x 128
// 4.5 and 11.0 us, 8,192 of 1 x 64 7.2 and 12.6; 131,072 of 1 x 64 99 and 40, of
// 2 x 128 133 and 101, of 4 x 128 159 and 158, of 8 x 128 264 and 272.
constexpr int kCheckRows = 8192, kCheckCells = 512;

struct Q8Cache {
  uint8_t* k;
  uint8_t* v;
  uint8_t* ke;                       // exponent bytes [page][head][row]
  uint8_t* ve;
  int64_t page_stride, row_stride, head_stride;
  int64_t n_slots;
  int32_t page_shift, Hkv;
};

__device__ __forceinline__ int64_t code_at(const Q8Cache& c, int s) {
  return (int64_t)(s >> c.page_shift) * c.page_stride +
         (int64_t)(s & ((1 << c.page_shift) - 1)) * c.row_stride;
}
__device__ __forceinline__ int64_t exp_at(const Q8Cache& c, int s, int h) {
  return (((int64_t)(s >> c.page_shift) * c.Hkv + h) << c.page_shift) + (s & ((1 << c.page_shift) - 1));
}

// One block looks over every index and writes the status word, 16 loads in
// flight a thread.
__device__ __forceinline__ void check_rows(const int32_t* slot, const int32_t* src, int n, int64_t n_slots,
                                           int T, uint32_t* status, uint32_t where) {
  constexpr int U = 16;
  uint32_t bad = 0;
  const int step = (int)blockDim.x;
  // unsigned: the last trip's indices pass 2^31 where n comes near it (in 64 bits 128K
  // rows of 8 x 128, stored and read back, take 269 us, so 263)
  for (uint32_t i0 = threadIdx.x; i0 < (uint32_t)n; i0 += U * step) {
    int s[U], r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t i = i0 + u * step;
      s[u] = i < (uint32_t)n ? slot[i] : -1;
      r[u] = src && i < (uint32_t)n ? src[i] : 0;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (s[u] >= 0 && (s[u] >= n_slots || r[u] < 0 || r[u] >= T)) bad = 1;
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) {
    status[0] = bad ? kDevIndex : 0u;
    status[1] = bad ? where : 0u;
  }
}

struct StoreParams {
  Q8Cache c;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  int64_t ks, vs;                    // source row strides, elements
  const int32_t* src;                // or null
  const int32_t* slot;
  const int32_t* pos;                // or null: no rotation
  const __nv_bfloat16* kw;           // or null: no norm
  float eps;
  int32_t n, T, hpt;                 // hpt: heads of a thread
  int32_t own_check;                 // block 0 looks over the indices
  uint32_t* status;
  uint64_t turn[64];
};

// Largest finite size of a lane's 8 + 8 elements; what is not finite becomes NaN
// (a maximum passes over NaN, so only infinities need a look at each).
__device__ __forceinline__ float lane_max(float* x, float* y) {
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = max3(m, fabsf(x[e]), fabsf(y[e]));
  if (m == INFINITY) {
    m = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (isfinite(x[e])) m = fmaxf(m, fabsf(x[e])); else x[e] = __int_as_float(0x7fffffff);
      if (isfinite(y[e])) m = fmaxf(m, fabsf(y[e])); else y[e] = __int_as_float(0x7fffffff);
    }
  }
  return m;
}

// Quantises a lane's 8 + 8 elements of a row with largest element m and stores them.
template <int D>
__device__ __forceinline__ void put_row(const float* x, const float* y, float m, uint8_t* code, uint8_t* exp,
                                        bool first) {
  const int ex = q8_exp_of(m);
  const float r = pow2(-ex);
  uint2 a, b;
  a.x = e4m3x4(x[0] * r, x[1] * r, x[2] * r, x[3] * r);
  a.y = e4m3x4(x[4] * r, x[5] * r, x[6] * r, x[7] * r);
  b.x = e4m3x4(y[0] * r, y[1] * r, y[2] * r, y[3] * r);
  b.y = e4m3x4(y[4] * r, y[5] * r, y[6] * r, y[7] * r);
  *reinterpret_cast<uint2*>(code) = a;
  *reinterpret_cast<uint2*>(code + D / 2) = b;
  if (first) *exp = (uint8_t)(ex + 127);
}

// U heads of a row at a time: nothing of one waits for another. Two where a thread
// has more than one, stored and read back: 128K rows of 8 x 128 264 us, one at a
// time 300; one where it has one: 32 rows 4.5 us, 5.1 by two, 128K rows of 1 x 64 40
// and 46. Blocks of 128: 264 us, of 256 269 (more of them stay resident).
template <int D, int U>
__global__ void __launch_bounds__(kStoreThreads, 4)
mis_paged_write_q8_kernel(const __grid_constant__ StoreParams p) {
  constexpr int HALF = D / 2, NC = D / 16;
  griddep_wait();
  if (p.own_check && blockIdx.x == 0) {
    check_rows(p.slot, p.src, p.n, p.c.n_slots, p.T, p.status, 0x40);
    return;
  }
  const int64_t gid = (int64_t)(blockIdx.x - p.own_check) * kStoreThreads + threadIdx.x;
  const int c = (int)(gid % NC);
  const int64_t cell = gid / NC;
  const int groups = (p.c.Hkv + p.hpt - 1) / p.hpt;
  const int grp = (int)(cell % groups);
  const int64_t i = cell / groups;
  if (i >= p.n) return;
  const int s = p.slot[i];
  if (s < 0) return;
  const int r = p.src ? p.src[i] : (int)i;
  if (s >= p.c.n_slots || r < 0 || r >= p.T) {
    if (!p.own_check) raise_status(p.status, kDevIndex, 0x40);
    return;
  }
  const uint32_t lanes = row_lanes<NC>();
  const int h0 = grp * p.hpt, h1 = min(h0 + p.hpt, p.c.Hkv);
  const __nv_bfloat16* ks = p.k + (int64_t)r * p.ks + c * 8;
  const __nv_bfloat16* vs = p.v + (int64_t)r * p.vs + c * 8;
  const int64_t at = code_at(p.c, s) + c * 8;
  uint4 ka[U], kb[U], va[U], vb[U];
  auto load = [&](int h) {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int64_t from = (int64_t)min(h + j, h1 - 1) * D;
      ka[j] = ld_row16(ks + from);
      kb[j] = ld_row16(ks + from + HALF);
      va[j] = ld_row16(vs + from);
      vb[j] = ld_row16(vs + from + HALF);
    }
  };
  // heads h and h + 1 of K and V come to L2, a lane a line of 128 bytes (128K rows
  // of 8 x 128 are stored in 146 us, without that in 158)
  auto ahead = [&](int h) {
    constexpr int LH = D / 64;
    const int x = h + c / (2 * LH);
    const __nv_bfloat16* at = ((c / LH) & 1 ? p.v + (int64_t)r * p.vs : p.k + (int64_t)r * p.ks) + (int64_t)x * D + (c % LH) * 64;
    if (x < h1) asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
  };
  if (U == 2) ahead(h0 + U);
  if (U == 1) load(h0);                          // in flight while the angles are taken
  float sn[8], cs[8], wx[8], wy[8];
  if (p.pos) {
    const int pos = p.pos[i];
#pragma unroll
    for (int e = 0; e < 8; ++e) sincos_quarters(pos, p.turn[c * 8 + e], sn[e], cs[e]);
  }
  if (p.kw) {
    bf16x8_to_float(*reinterpret_cast<const uint4*>(p.kw + c * 8), wx);
    bf16x8_to_float(*reinterpret_cast<const uint4*>(p.kw + HALF + c * 8), wy);
  }
#pragma unroll 1
  for (int hh = h0; hh < h1; hh += U) {
    if (U != 1 || hh != h0) load(hh);
    if (U == 2 && hh + 2 * U < h1) ahead(hh + 2 * U);
    float x[U][8], y[U][8], m[2 * U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      bf16x8_to_float(ka[i], x[i]);
      bf16x8_to_float(kb[i], y[i]);
    }
    if (p.kw) norm_rows<D, U>(x, y, wx, wy, p.eps, lanes);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (p.pos) rotate_row(x[i], y[i], sn, cs);
      m[i] = lane_max(x[i], y[i]);
    }
    float vx[U][8], vy[U][8];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      bf16x8_to_float(va[i], vx[i]);
      bf16x8_to_float(vb[i], vy[i]);
      m[U + i] = lane_max(vx[i], vy[i]);
    }
    row_maxima<NC, 2 * U>(m, lanes);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int h = hh + i;
      if (h >= h1) break;
      const int64_t to = at + (int64_t)h * p.c.head_stride, ex = exp_at(p.c, s, h);
      put_row<D>(x[i], y[i], m[i], p.c.k + to, p.c.ke + ex, c == 0);
      put_row<D>(vx[i], vy[i], m[U + i], p.c.v + to, p.c.ve + ex, c == 0);
    }
  }
}

struct ReadParams {
  Q8Cache c;
  __nv_bfloat16* k;
  __nv_bfloat16* v;
  int64_t ks, vs;
  const int32_t* slot;
  int32_t n, own_check;
  uint32_t* status;
};

// 8 codes times 2^e as bf16.
__device__ __forceinline__ void put_values(const uint2& codes, float scale, __nv_bfloat16* dst) {
  const uint32_t w[2] = {codes.x, codes.y};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t h = e4m3x2_to_half2((uint16_t)(w[i] >> (16 * j)));
      float lo, hi;
      half2_to_float(h, lo, hi);
      o[2 * i + j] = pack_bf16(lo * scale, hi * scale);
    }
  }
  *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
}

template <int D>
__global__ void __launch_bounds__(kThreads)
mis_paged_read_q8_kernel(const __grid_constant__ ReadParams p) {
  constexpr int NC = D / 16;
  griddep_wait();
  if (p.own_check && blockIdx.x == 0) {
    check_rows(p.slot, nullptr, p.n, p.c.n_slots, 0x7fffffff, p.status, 0x50);
    return;
  }
  const int64_t gid = (int64_t)(blockIdx.x - p.own_check) * kThreads + threadIdx.x;
  const int c = (int)(gid % NC);
  const int64_t cell = gid / NC;
  const int h = (int)(cell % p.c.Hkv);
  const int64_t i = cell / p.c.Hkv;
  if (i >= p.n) return;
  const int s = p.slot[i];
  if (s < 0) return;
  if (s >= p.c.n_slots) {
    if (!p.own_check) raise_status(p.status, kDevIndex, 0x50);
    return;
  }
  // a lane's 8 elements of each half of the head: its 16 bytes of a store lie beside
  // its neighbours' (16 elements a lane, every other 16 bytes a store: 135 us, not 120)
  const int64_t at = code_at(p.c, s) + (int64_t)h * p.c.head_stride + c * 8, ex = exp_at(p.c, s, h);
  const uint2 ka = *reinterpret_cast<const uint2*>(p.c.k + at), kb = *reinterpret_cast<const uint2*>(p.c.k + at + D / 2);
  const uint2 va = *reinterpret_cast<const uint2*>(p.c.v + at), vb = *reinterpret_cast<const uint2*>(p.c.v + at + D / 2);
  const float ke = pow2(q8_exp(p.c.ke[ex])), ve = pow2(q8_exp(p.c.ve[ex]));
  __nv_bfloat16* k = p.k + i * p.ks + (int64_t)h * D + c * 8;
  __nv_bfloat16* v = p.v + i * p.vs + (int64_t)h * D + c * 8;
  put_values(ka, ke, k);
  put_values(kb, ke, k + D / 2);
  put_values(va, ve, v);
  put_values(vb, ve, v + D / 2);
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

Q8Cache cache_of(const mis_paged_cache_q8* c) {
  Q8Cache d;
  d.k = static_cast<uint8_t*>(c->k);
  d.v = static_cast<uint8_t*>(c->v);
  d.ke = c->k_exp;
  d.ve = c->v_exp;
  d.page_stride = c->page_stride; d.row_stride = c->row_stride; d.head_stride = c->head_stride;
  d.n_slots = (int64_t)c->n_pages * c->page_size;
  d.page_shift = 31 - __builtin_clz((unsigned)c->page_size);
  d.Hkv = c->Hkv;
  return d;
}

}  // namespace

mis_status_t check_paged_cache_q8(const mis_paged_cache_q8* c) {
  if (!c || !c->k || !c->v || !c->k_exp || !c->v_exp) return MIS_ERR_INVALID_ARG;
  for (const void* x : {(const void*)c->k, (const void*)c->v, (const void*)c->k_exp, (const void*)c->v_exp})
    if (!aligned(x, 16)) return MIS_ERR_INVALID_ARG;
  if (c->n_pages < 1 || c->Hkv < 1) return MIS_ERR_INVALID_ARG;
  if (!page_size_ok(c->page_size) || (c->D != 64 && c->D != 128)) return MIS_ERR_UNSUPPORTED;
  if ((int64_t)c->n_pages * c->page_size > 0x7fffffff) return MIS_ERR_SHAPE;
  // the strides in use, smallest first, each past the extent of the ones below
  int64_t st[3] = {c->row_stride, c->page_stride, c->head_stride};
  int64_t ex[3] = {c->page_size, c->n_pages, c->Hkv};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (st[j] < st[i]) { std::swap(st[i], st[j]); std::swap(ex[i], ex[j]); }
  int64_t width = c->D;
  for (int i = 0; i < 3; ++i) {
    if (ex[i] == 1) continue;
    if (st[i] < width || (st[i] & 15) || st[i] >= (int64_t)1 << 38) return MIS_ERR_SHAPE;
    width = st[i] * (ex[i] - 1) + width;
  }
  return MIS_OK;
}

Span codes_span(const mis_paged_cache_q8* c, const void* base) {
  auto reach = [](int64_t extent, int64_t stride) { return extent > 1 ? (extent - 1) * stride : 0; };
  const int64_t heads = reach(c->Hkv, c->head_stride) + c->D;             // of one row
  const int64_t page = reach(c->page_size, c->row_stride) + heads;
  const int64_t all = reach(c->n_pages, c->page_stride) + page;
  // rows at one stride; else pages at one; else all as one piece
  const bool rows = c->n_pages == 1 || c->page_stride == c->page_size * c->row_stride;
  if (rows && heads <= c->row_stride) return {base, (int64_t)c->n_pages * c->page_size, c->row_stride, heads};
  if (c->n_pages > 1 && page <= c->page_stride) return {base, c->n_pages, c->page_stride, page};
  return {base, 1, all, all};
}

// Whether rows of K and rows of V (the same strides, `apart` bytes on) share
// bytes. The strides lie past each other's extents, so of each, largest first,
// only the two multiples around what is left can bring the rest near zero.
static bool rows_at(const int64_t* st, const int64_t* ex, int i, int64_t apart, int64_t D) {
  if (i < 0) return apart > -D && apart < D;
  if (ex[i] == 1) return rows_at(st, ex, i - 1, apart, D);
  int64_t d = apart / st[i] - (apart % st[i] < 0);
  for (int x = 0; x < 2; ++x, ++d)
    if (d > -ex[i] && d < ex[i] && rows_at(st, ex, i - 1, apart - d * st[i], D)) return true;
  return false;
}
static bool kv_rows_meet(const mis_paged_cache_q8* c) {
  int64_t st[3] = {c->row_stride, c->page_stride, c->head_stride};
  int64_t ex[3] = {c->page_size, c->n_pages, c->Hkv};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (ex[i] == 1 ? false : ex[j] == 1 || st[j] < st[i]) { std::swap(st[i], st[j]); std::swap(ex[i], ex[j]); }
  const int64_t apart = (int64_t)(reinterpret_cast<uintptr_t>(c->v) - reinterpret_cast<uintptr_t>(c->k));
  return rows_at(st, ex, 2, apart, c->D);
}

Span exps_span(const mis_paged_cache_q8* c, const void* base) {
  return {base, 1, 0, (int64_t)c->n_pages * c->page_size * c->Hkv};
}

}  // namespace mis

using namespace mis;

extern "C" mis_status_t mis_paged_write_kv_q8(const mis_paged_cache_q8* cache, const void* k, const void* v,
                                              int64_t k_row_stride, int64_t v_row_stride, int32_t T,
                                              const int32_t* src_rows, const int32_t* slot_map, int32_t n,
                                              const int32_t* position_ids, double rope_base,
                                              const void* k_weight, float eps, void* workspace,
                                              size_t ws_bytes, void* stream) {
  const mis_status_t cs = check_paged_cache_q8(cache);
  if (cs != MIS_OK) return cs;
  if (T < 0 || n < 0) return MIS_ERR_INVALID_ARG;
  if (position_ids && (!(rope_base > 1.0) || !std::isfinite(rope_base))) return MIS_ERR_INVALID_ARG;
  if (k_weight && !(eps >= 0.f && eps <= 1.f)) return MIS_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) || ws_bytes < mis_paged_write_workspace_size())
    return MIS_ERR_WORKSPACE;
  if (!src_rows && n > T) return MIS_ERR_SHAPE;
  const int64_t w = (int64_t)cache->Hkv * cache->D;
  if (k_row_stride < w || v_row_stride < w || ((k_row_stride | v_row_stride) & 7)) return MIS_ERR_SHAPE;
  if (n == 0) return MIS_OK;
  if (!slot_map || !aligned(slot_map, 4) || !aligned(src_rows, 4) || !aligned(position_ids, 4))
    return MIS_ERR_INVALID_ARG;
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16) || !aligned(k_weight, 16)) return MIS_ERR_INVALID_ARG;
  {
    const Span out[5] = {codes_span(cache, cache->k), codes_span(cache, cache->v),
                         exps_span(cache, cache->k_exp), exps_span(cache, cache->v_exp),
                         Span{workspace, 1, 0, (int64_t)kStatusBytes}};
    const Span in[6] = {{k, T, 2 * k_row_stride, 2 * w}, {v, T, 2 * v_row_stride, 2 * w},
                        {slot_map, 1, 0, 4 * (int64_t)n}, {src_rows, 1, 0, 4 * (int64_t)n},
                        {position_ids, 1, 0, 4 * (int64_t)n}, {k_weight, 1, 0, 2 * (int64_t)cache->D}};
    for (int i = 0; i < 5; ++i) {
      for (const Span& x : in)
        if (overlap(out[i], x)) return MIS_ERR_INVALID_ARG;
      for (int j = i < 2 ? i : 0; j < i; ++j)
        if (overlap(out[i], out[j])) return MIS_ERR_INVALID_ARG;
    }
    if (kv_rows_meet(cache)) return MIS_ERR_INVALID_ARG;
  }
  StoreParams p;
  p.c = cache_of(cache);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.ks = k_row_stride; p.vs = v_row_stride;
  p.src = src_rows; p.slot = slot_map; p.pos = position_ids;
  p.kw = static_cast<const __nv_bfloat16*>(k_weight);
  p.eps = eps;
  p.n = n; p.T = T;
  p.status = static_cast<uint32_t*>(workspace);
  p.own_check = n <= kCheckRows || cache->Hkv * cache->D >= kCheckCells;
  const int D = cache->D, Hkv = cache->Hkv;
  if (position_ids) fill_turns(rope_base, D, p.turn);
  // an angle serves all heads of a thread; a row's heads are split over
  // threads only while its lanes alone would leave SMs idle
  const int64_t cells = (int64_t)n * (D / 16), want = 512 * (int64_t)num_sms();
  const int64_t split = std::max<int64_t>(1, std::min<int64_t>(Hkv, want / cells));
  p.hpt = (int32_t)((Hkv + split - 1) / split);
  const int64_t threads = cells * ((Hkv + p.hpt - 1) / p.hpt);
  const int64_t blocks = p.own_check + (threads + kStoreThreads - 1) / kStoreThreads;
  if (blocks > 0x7fffffff) return MIS_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  try {
    if (!p.own_check && cudaMemsetAsync(workspace, 0, 8, st) != cudaSuccess) return MIS_ERR_CUDA;
    auto kern = D == 128 ? (p.hpt > 1 ? mis_paged_write_q8_kernel<128, 2> : mis_paged_write_q8_kernel<128, 1>)
                         : (p.hpt > 1 ? mis_paged_write_q8_kernel<64, 2> : mis_paged_write_q8_kernel<64, 1>);
    const cudaError_t e = launch_pdl(kern, dim3((unsigned)blocks), dim3(kStoreThreads), 0, st, p);
    return e == cudaSuccess ? MIS_OK : MIS_ERR_CUDA;
  } catch (...) {
    return MIS_ERR_CUDA;
  }
}

extern "C" mis_status_t mis_paged_read_kv_q8(const mis_paged_cache_q8* cache, const int32_t* slot_map,
                                             int32_t n, void* k_out, void* v_out, int64_t k_row_stride,
                                             int64_t v_row_stride, void* workspace, size_t ws_bytes,
                                             void* stream) {
  const mis_status_t cs = check_paged_cache_q8(cache);
  if (cs != MIS_OK) return cs;
  if (n < 0) return MIS_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) || ws_bytes < mis_paged_write_workspace_size())
    return MIS_ERR_WORKSPACE;
  const int64_t w = (int64_t)cache->Hkv * cache->D;
  if (k_row_stride < w || v_row_stride < w || ((k_row_stride | v_row_stride) & 7)) return MIS_ERR_SHAPE;
  if (n == 0) return MIS_OK;
  if (!slot_map || !aligned(slot_map, 4)) return MIS_ERR_INVALID_ARG;
  if (!k_out || !v_out || !aligned(k_out, 16) || !aligned(v_out, 16)) return MIS_ERR_INVALID_ARG;
  {
    const Span out[3] = {{k_out, n, 2 * k_row_stride, 2 * w}, {v_out, n, 2 * v_row_stride, 2 * w},
                         {workspace, 1, 0, (int64_t)kStatusBytes}};
    const Span in[5] = {codes_span(cache, cache->k), codes_span(cache, cache->v),
                        exps_span(cache, cache->k_exp), exps_span(cache, cache->v_exp),
                        Span{slot_map, 1, 0, 4 * (int64_t)n}};
    for (int i = 0; i < 3; ++i) {
      for (const Span& x : in)
        if (overlap(out[i], x)) return MIS_ERR_INVALID_ARG;
      for (int j = 0; j < i; ++j)
        if (overlap(out[i], out[j])) return MIS_ERR_INVALID_ARG;
    }
  }
  ReadParams p;
  p.c = cache_of(cache);
  p.k = static_cast<__nv_bfloat16*>(k_out);
  p.v = static_cast<__nv_bfloat16*>(v_out);
  p.ks = k_row_stride; p.vs = v_row_stride;
  p.slot = slot_map;
  p.n = n;
  p.own_check = n <= kCheckRows || cache->Hkv * cache->D >= kCheckCells;
  p.status = static_cast<uint32_t*>(workspace);
  const int64_t threads = (int64_t)n * (cache->D / 16) * cache->Hkv;
  const int64_t blocks = p.own_check + (threads + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffff) return MIS_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  try {
    if (!p.own_check && cudaMemsetAsync(workspace, 0, 8, st) != cudaSuccess) return MIS_ERR_CUDA;
    const cudaError_t e = cache->D == 128 ? launch_pdl(mis_paged_read_q8_kernel<128>, dim3((unsigned)blocks),
                                                       dim3(kThreads), 0, st, p)
                                          : launch_pdl(mis_paged_read_q8_kernel<64>, dim3((unsigned)blocks),
                                                       dim3(kThreads), 0, st, p);
    return e == cudaSuccess ? MIS_OK : MIS_ERR_CUDA;
  } catch (...) {
    return MIS_ERR_CUDA;
  }
}
