// Paged K/V cache for sm_103a: block tables and slot maps from request
// lengths, and K/V rows stored at slots (K rotated on the way).
//
// mis_paged_extend. need_b = ceil((L_b + n_b) / ps) - ceil(L_b / ps) pages of
// request b are the run of the free list that starts at the exclusive sum of
// need; its rows start at the exclusive sum of n. One block takes both sums
// over the batch and leaves a record per request; the rows' slots follow from
// the record of their request (found by bisection of cu_new) and one page id.
//
// What bounds it is latency: a chain of dependent loads and the block's scans,
// 4.3 us for 32 requests with a row each, 4.8 us for 16 with 187,165 rows, 7.3 us
// for 256 with 997,692 (8.5 MB, 1.2 TB/s).
//
// mis_paged_write_kv is a copy: every kept row is read and written once, so
// HBM bounds it: 131,072 rows of 8 heads, D = 128, rotated (1.07 GB), 164.6 us,
// 6.5 TB/s of 6.7 measured for a copy. A decoding step is the launch's 2 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "mis_internal.h"
#include "mis_ptx.cuh"

namespace mis {
namespace {

using namespace dev;

constexpr int kPlanThreads = 1024;
constexpr int kFillThreads = 256;
constexpr int kFillRows = 4;            // consecutive rows of a thread
constexpr int kCuShared = 2048;         // requests whose row starts a fill block keeps
// Rows up to which the planning block fills the maps itself: a second launch
// costs the host 3.2 us and the GPU about 2; eight rows a thread cost less
constexpr int kFillInPlan = 8 * kPlanThreads;

// What the rows of a request need to find their slots.
struct ExtendRec {
  int32_t len;    // rows cached before the call
  int32_t have;   // pages held before the call
  int32_t first;  // free-list index of its first fresh page
  int32_t pad;
};

struct ExtendParams {
  int32_t B, T, page_size, page_shift, n_pages, max_pages, n_free;
  const int32_t* new_len;
  const int32_t* cache_len;
  int32_t* cache_len_out;
  int32_t* table;
  int64_t table_stride;
  const int32_t* free_pages;
  const int32_t* free_head;
  int32_t* free_head_out;
  int32_t* cu_new;
  int32_t* slot_map;
  int32_t* position_ids;
  uint32_t* status;
  ExtendRec* rec;
  int32_t vec;       // slot_map and position_ids take 16-byte stores
};

// Inclusive sums of two values over the block's threads, and their totals.
struct Pair {
  int64_t x, y;
};
__device__ __forceinline__ Pair block_sum(Pair v, Pair* total, Pair* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, v.x, o), y = __shfl_up_sync(0xffffffffu, v.y, o);
    if (lane >= o) { v.x += x; v.y += y; }
  }
  __syncthreads();                       // the previous call's readers are done
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  // every warp adds up the warps' sums for itself
  Pair w = lane < warps ? warp_sums[lane] : Pair{0, 0};
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, w.x, o), y = __shfl_up_sync(0xffffffffu, w.y, o);
    if (lane >= o) { w.x += x; w.y += y; }
  }
  total->x = __shfl_sync(0xffffffffu, w.x, 31);
  total->y = __shfl_sync(0xffffffffu, w.y, 31);
  const int64_t bx = __shfl_sync(0xffffffffu, w.x, max(warp - 1, 0));
  const int64_t by = __shfl_sync(0xffffffffu, w.y, max(warp - 1, 0));
  return warp ? Pair{v.x + bx, v.y + by} : v;
}

// Slots and positions of rows t .. t + kFillRows - 1 (and the table entries of
// pages that start there). cu: cu_new, wherever it is read from.
__device__ __forceinline__ void fill_rows(const ExtendParams& p, const int32_t* cu, int t, int total) {
  int slot[kFillRows], pos[kFillRows];
  int b = 0;
  if (t < total) {
    int hi = p.B - 1;                    // first b with cu[b + 1] > t
    while (b < hi) {
      const int mid = (b + hi) >> 1;
      if (cu[mid + 1] > t) hi = mid; else b = mid + 1;
    }
  }
  ExtendRec r{0, 0, 0, 0};
  int start = 0, end = -1, col0 = -1, page = -1;
#pragma unroll
  for (int e = 0; e < kFillRows; ++e) {
    slot[e] = -1;
    pos[e] = 0;
    if (t + e >= total) continue;
    if (t + e >= end) {
      while (cu[b + 1] <= t + e) ++b;
      r = p.rec[b];
      start = cu[b];
      end = cu[b + 1];
      col0 = -1;
    }
    pos[e] = r.len + (t + e - start);
    const int col = pos[e] >> p.page_shift, off = pos[e] & ((1 << p.page_shift) - 1);
    if (col != col0) {
      int32_t* entry = p.table + (int64_t)b * p.table_stride + col;
      const bool fresh = col >= r.have;
      page = fresh ? p.free_pages[r.first + (col - r.have)] : *entry;
      if (page < 0 || page >= p.n_pages) {
        page = -1;
        raise_status(p.status, kDevIndex, 0x21);
      }
      if (fresh && off == 0) *entry = page;
      col0 = col;
    }
    if (page >= 0) slot[e] = (page << p.page_shift) + off;
  }
  if (p.vec && t + kFillRows <= p.T) {
    *reinterpret_cast<int4*>(p.slot_map + t) = make_int4(slot[0], slot[1], slot[2], slot[3]);
    if (p.position_ids)
      *reinterpret_cast<int4*>(p.position_ids + t) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    return;
  }
#pragma unroll
  for (int e = 0; e < kFillRows; ++e)
    if (t + e < p.T) {
      p.slot_map[t + e] = slot[e];
      if (p.position_ids) p.position_ids[t + e] = pos[e];
    }
}

__global__ void __launch_bounds__(kPlanThreads)
mis_paged_extend_kernel(const ExtendParams p) {
  __shared__ Pair warp_sums[32];
  __shared__ int s_head;
  __shared__ uint32_t s_bits, s_taken;
  griddep_launch_dependents();
  griddep_wait();
  if (threadIdx.x == 0) {
    s_head = *p.free_head;
    s_bits = s_taken = 0;
  }
  __syncthreads();
  const int head = s_head;
  const bool head_ok = head >= 0 && head <= p.n_free;
  const int64_t avail = head_ok ? p.n_free - head : 0;
  const int64_t cap = (int64_t)p.max_pages * p.page_size;
  uint32_t bits = head_ok ? 0u : kDevIndex;
  int64_t pages0 = 0, rows0 = 0, cu0 = 0, taken = 0;
  for (int b0 = 0; b0 < p.B; b0 += (int)blockDim.x) {
    const int b = b0 + threadIdx.x;
    int64_t len = 0, n = 0, need = 0;
    int have = 0;
    if (b < p.B) {
      len = p.cache_len[b];
      n = p.new_len[b];
      if (len < 0 || n < 0 || len + n > cap) {
        bits |= kDevIndex;
        n = 0;
      } else {
        have = (int)((len + p.page_size - 1) / p.page_size);
        need = (len + n + p.page_size - 1) / p.page_size - have;
      }
    }
    Pair sum;
    const Pair end = block_sum(Pair{need, n}, &sum, warp_sums);
    const int64_t pend = pages0 + end.x, rend = rows0 + end.y;
    bool ok = true;
    if (need > 0 && pend > avail) { bits |= kDevPages; ok = false; }
    if (n > 0 && rend > p.T) { bits |= kDevIndex; ok = false; }
    const int64_t g = ok ? n : 0;
    int64_t gend = cu0 + end.y, granted = sum.y;
    if (__syncthreads_or(!ok)) {           // rows of refused requests close up
      Pair gsum;
      gend = cu0 + block_sum(Pair{g, 0}, &gsum, warp_sums).x;
      granted = gsum.x;
    }
    if (ok && need > 0 && pend > taken) taken = pend;
    if (b < p.B) {
      ExtendRec r;
      r.len = (int32_t)len;
      r.have = have;
      r.first = (int32_t)(ok ? head + pend - need : 0);
      r.pad = 0;
      p.rec[b] = r;
      p.cu_new[b + 1] = (int32_t)gend;
      p.cache_len_out[b] = (int32_t)(len + g);
    }
    pages0 += sum.x;
    rows0 += sum.y;
    cu0 += granted;
  }
  // granted requests that took pages are a prefix of those that need any, so
  // the furthest end of a granted run is where the list continues
  if (bits) atomicOr(&s_bits, bits);
  if (taken) atomicMax(&s_taken, (uint32_t)taken);
  __syncthreads();
  if (threadIdx.x == 0) {
    p.cu_new[0] = 0;
    *p.free_head_out = head + (int)s_taken;
    p.status[0] = s_bits;
    p.status[1] = s_bits ? 0x20u : 0u;
  }
  if (p.T <= kFillInPlan) {
    __syncthreads();                     // cu_new, records and status are written
    for (int t = threadIdx.x * kFillRows; t < p.T; t += (int)blockDim.x * kFillRows)
      fill_rows(p, p.cu_new, t, (int)cu0);
  }
}

__global__ void __launch_bounds__(kFillThreads)
mis_paged_fill_kernel(const ExtendParams p) {
  griddep_wait();
  __shared__ int32_t s_cu[kCuShared + 1];
  const int32_t* cu = p.cu_new;
  if (p.B <= kCuShared) {
    for (int b = threadIdx.x; b <= p.B; b += blockDim.x) s_cu[b] = p.cu_new[b];
    __syncthreads();
    cu = s_cu;
  }
  const int64_t t = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * kFillRows;
  if (t < p.T) fill_rows(p, cu, (int)t, cu[p.B]);
}

// ------------------------------------------------------------------- write
struct WriteParams {
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  __nv_bfloat16* kc;
  __nv_bfloat16* vc;
  int64_t ks, vs;                    // source row strides, elements
  int64_t page_stride, row_stride, head_stride;
  const int32_t* src;                // or null
  const int32_t* slot;
  const int32_t* pos;                // or null: no rotation
  int32_t n, T, Hkv;
  int32_t hpt;                       // heads of a thread
  int32_t page_shift;
  int64_t n_slots;
  uint32_t* status;
  uint64_t turn[64];                 // base^(-2i/D) / (2 pi) as a 64-bit fraction of a turn
};

__device__ __forceinline__ void unpack8(const uint4& u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// sin and cos of position p times a frequency given as a 64-bit fraction of a
// turn: the product modulo 2^64 is the fraction of a turn left after whole
// turns. It is off by p times the frequency's error, which as a power in double
// is up to 2^-54 of a turn (2^-37 at position 131,072). Its top 32 bits, read as
// signed, are an angle in [-pi, pi), where the SFU approximations are good to 2^-21.
__device__ __forceinline__ void sincos_turn(int32_t p, uint64_t f, float& sn, float& cs) {
  const uint32_t lo = (uint32_t)f, hi = (uint32_t)(f >> 32), up = (uint32_t)p;
  uint32_t frac = __umulhi(up, lo) + up * hi;
  if (p < 0) frac -= lo;
  const float x = (float)(int32_t)frac * 1.46291807926715968e-9f;   // 2 pi / 2^32
  asm("sin.approx.f32 %0, %1;" : "=f"(sn) : "f"(x));
  asm("cos.approx.f32 %0, %1;" : "=f"(cs) : "f"(x));
}

// A source row's 16 bytes, read once.
__device__ __forceinline__ uint4 ld_once(const __nv_bfloat16* ptr) {
  uint4 u;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(ptr));
  return u;
}

template <int D>
__global__ void __launch_bounds__(256)
mis_paged_write_kernel(const WriteParams p) {
  constexpr int HALF = D / 2, NC = HALF / 8;
  griddep_wait();
  if (blockIdx.x == 0) {
    // one block looks over every index and writes the status word, 16 loads in
    // flight a thread (128K rows: 330 us when it took them one by one). It bounds
    // calls of many narrow rows: 128K rows of one head of 64 take 49 us (10 by
    // their bytes), of 2 heads 54 (20), of 8 97 (80)
    constexpr int U = 16;
    const int step = U * (int)blockDim.x;
    uint32_t bad = 0;
    for (int64_t i0 = threadIdx.x; i0 < p.n; i0 += step) {
      int s[U], r[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t i = i0 + u * (int)blockDim.x;
        s[u] = i < p.n ? p.slot[i] : -1;
        r[u] = p.src && i < p.n ? p.src[i] : 0;
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (s[u] >= 0 && (s[u] >= p.n_slots || r[u] < 0 || r[u] >= p.T)) bad = 1;
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) {
      p.status[0] = bad ? kDevIndex : 0u;
      p.status[1] = bad ? 0x30u : 0u;
    }
    return;
  }
  const int64_t gid = (int64_t)(blockIdx.x - 1) * blockDim.x + threadIdx.x;
  const int c = (int)(gid % NC);
  const int64_t cell = gid / NC;
  const int groups = (p.Hkv + p.hpt - 1) / p.hpt;
  const int grp = (int)(cell % groups);
  const int64_t i = cell / groups;
  if (i >= p.n) return;
  const int s = p.slot[i];
  const int r = p.src ? p.src[i] : (int)i;
  if (s < 0 || s >= p.n_slots || r < 0 || r >= p.T) return;
  const int h0 = grp * p.hpt, h1 = min(h0 + p.hpt, p.Hkv);
  const int64_t at = (int64_t)(s >> p.page_shift) * p.page_stride +
                     (int64_t)(s & ((1 << p.page_shift) - 1)) * p.row_stride + c * 8;
  const __nv_bfloat16* ks = p.k + (int64_t)r * p.ks + c * 8;
  const __nv_bfloat16* vs = p.v + (int64_t)r * p.vs + c * 8;
  float sn[8], cs[8];
  if (p.pos) {
    const int pos = p.pos[i];
#pragma unroll
    for (int e = 0; e < 8; ++e) sincos_turn(pos, p.turn[c * 8 + e], sn[e], cs[e]);
  }
#pragma unroll 2
  for (int h = h0; h < h1; ++h) {
    const int64_t from = (int64_t)h * D, to = at + (int64_t)h * p.head_stride;
    uint4 a = ld_once(ks + from), b = ld_once(ks + from + HALF);
    const uint4 va = ld_once(vs + from), vb = ld_once(vs + from + HALF);
    if (p.pos) {
      float x[8], y[8];
      unpack8(a, x);
      unpack8(b, y);
      uint32_t wa[4], wb[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x0 = x[2 * e], x1 = x[2 * e + 1], y0 = y[2 * e], y1 = y[2 * e + 1];
        const float s0 = sn[2 * e], s1 = sn[2 * e + 1], c0 = cs[2 * e], c1 = cs[2 * e + 1];
        wa[e] = pack_bf16(x0 * c0 - y0 * s0, x1 * c1 - y1 * s1);
        wb[e] = pack_bf16(y0 * c0 + x0 * s0, y1 * c1 + x1 * s1);
      }
      a = make_uint4(wa[0], wa[1], wa[2], wa[3]);
      b = make_uint4(wb[0], wb[1], wb[2], wb[3]);
    }
    *reinterpret_cast<uint4*>(p.kc + to) = a;
    *reinterpret_cast<uint4*>(p.kc + to + HALF) = b;
    *reinterpret_cast<uint4*>(p.vc + to) = va;
    *reinterpret_cast<uint4*>(p.vc + to + HALF) = vb;
  }
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

mis_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MIS_OK : MIS_ERR_CUDA; }

}  // namespace

bool page_size_ok(int32_t ps) {
  return ps == 16 || ps == 32 || ps == 64 || ps == 128 || ps == 256;
}

// The frequencies of a (base, D), kept from call to call: 64 powers cost the
// host 3 us.
void fill_turns(double base, int D, uint64_t* turn) {
  struct Kept {
    double base = 0;
    int D = 0;
    uint64_t turn[64];
  };
  static thread_local Kept kept;
  if (kept.base != base || kept.D != D) {
    for (int i = 0; i < 64; ++i)
      kept.turn[i] = i < D / 2 ? (uint64_t)(std::pow(base, -2.0 * i / D) / 6.283185307179586476925 *
                                            18446744073709551616.0)
                               : 0;
    kept.base = base;
    kept.D = D;
  }
  for (int i = 0; i < 64; ++i) turn[i] = kept.turn[i];
}

mis_status_t check_paged_cache(const mis_paged_cache* c) {
  if (!c || !c->k || !c->v) return MIS_ERR_INVALID_ARG;
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return MIS_ERR_INVALID_ARG;
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
    if (st[i] < width || (st[i] & 7) || st[i] >= (int64_t)1 << 38) return MIS_ERR_SHAPE;
    width = st[i] * (ex[i] - 1) + width;
  }
  return MIS_OK;
}

bool rows_meet(const Span& a, const Span& b) {
  if (a.rows > 1 && b.rows > 1 && a.stride != b.stride) return true;
  const int64_t stride = a.rows > 1 ? a.stride : b.stride;
  if ((a.rows == 1 && b.rows == 1) || stride < 1) return true;
  // where b's rows begin in a's
  const int64_t d = b.lo >= a.lo ? (int64_t)((b.lo - a.lo) % (uint64_t)stride)
                                 : (stride - (int64_t)((a.lo - b.lo) % (uint64_t)stride)) % stride;
  return d < a.width || d > stride - b.width;
}

Span cache_span(const mis_paged_cache* c, const void* base) {
  auto reach = [](int64_t extent, int64_t stride) { return extent > 1 ? (extent - 1) * stride : 0; };
  const int64_t heads = reach(c->Hkv, c->head_stride) + c->D;             // of one row
  const int64_t page = reach(c->page_size, c->row_stride) + heads;
  const int64_t all = reach(c->n_pages, c->page_stride) + page;
  // rows at one stride; else pages at one; else all as one piece
  const bool rows = c->n_pages == 1 || c->page_stride == c->page_size * c->row_stride;
  if (rows && heads <= c->row_stride)
    return {base, (int64_t)c->n_pages * c->page_size, c->row_stride * 2, heads * 2};
  if (c->n_pages > 1 && page <= c->page_stride) return {base, c->n_pages, c->page_stride * 2, page * 2};
  return {base, 1, all * 2, all * 2};
}

}  // namespace mis

using namespace mis;

extern "C" size_t mis_paged_extend_workspace_size(int32_t B) {
  return B < 1 ? 0 : kStatusBytes + (((size_t)B * sizeof(ExtendRec) + 255) & ~(size_t)255);
}

extern "C" mis_status_t mis_paged_extend(
    int32_t B, int32_t T, int32_t page_size, int32_t n_pages, const int32_t* new_len,
    const int32_t* cache_len, int32_t* cache_len_out, int32_t* block_table, int32_t max_pages,
    int64_t block_table_stride, const int32_t* free_pages, int32_t n_free,
    const int32_t* free_head, int32_t* free_head_out, int32_t* cu_new, int32_t* slot_map,
    int32_t* position_ids, void* workspace, size_t ws_bytes, void* stream) {
  if (B < 1 || T < 0 || n_pages < 1 || max_pages < 1 || n_free < 0) return MIS_ERR_INVALID_ARG;
  if (T > 0x7ffffff0) return MIS_ERR_SHAPE;
  if (!page_size_ok(page_size)) return MIS_ERR_UNSUPPORTED;
  if ((int64_t)n_pages * page_size > 0x7fffffff || (int64_t)max_pages * page_size > 0x7fffffff ||
      block_table_stride < max_pages)
    return MIS_ERR_SHAPE;
  if (!new_len || !cache_len || !cache_len_out || !block_table || !free_head || !free_head_out ||
      !cu_new || (T > 0 && !slot_map) || (n_free > 0 && !free_pages))
    return MIS_ERR_INVALID_ARG;
  for (const void* ptr : {(const void*)new_len, (const void*)cache_len, (const void*)cache_len_out,
                          (const void*)block_table, (const void*)free_pages,
                          (const void*)free_head, (const void*)free_head_out, (const void*)cu_new,
                          (const void*)slot_map, (const void*)position_ids})
    if (!aligned(ptr, 4)) return MIS_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) || ws_bytes < mis_paged_extend_workspace_size(B))
    return MIS_ERR_WORKSPACE;
  {
    auto ints = [](const int32_t* at, int64_t n) { return Span(at, 1, 0, 4 * n); };
    const Span in[4] = {ints(new_len, B), ints(cache_len, B), ints(free_pages, n_free), ints(free_head, 1)};
    const Span out[7] = {ints(cache_len_out, B), ints(free_head_out, 1), ints(cu_new, (int64_t)B + 1),
                         ints(slot_map, T), ints(position_ids, T),
                         Span{block_table, B, 4 * block_table_stride, 4 * (int64_t)max_pages},
                         Span{workspace, 1, 0, (int64_t)mis_paged_extend_workspace_size(B)}};
    for (int i = 0; i < 7; ++i) {
      for (int j = 0; j < 4; ++j)
        if (!(i == 0 && j == 1 && cache_len_out == cache_len) &&
            !(i == 1 && j == 3 && free_head_out == free_head) && overlap(out[i], in[j]))
          return MIS_ERR_INVALID_ARG;
      for (int j = 0; j < i; ++j)
        if (overlap(out[i], out[j])) return MIS_ERR_INVALID_ARG;
    }
  }
  ExtendParams p;
  p.page_shift = 31 - __builtin_clz((unsigned)page_size);
  p.vec = aligned(slot_map, 16) && aligned(position_ids, 16);
  p.B = B; p.T = T; p.page_size = page_size; p.n_pages = n_pages; p.max_pages = max_pages;
  p.n_free = n_free;
  p.new_len = new_len; p.cache_len = cache_len; p.cache_len_out = cache_len_out;
  p.table = block_table; p.table_stride = block_table_stride;
  p.free_pages = free_pages; p.free_head = free_head; p.free_head_out = free_head_out;
  p.cu_new = cu_new; p.slot_map = slot_map; p.position_ids = position_ids;
  p.status = static_cast<uint32_t*>(workspace);
  p.rec = reinterpret_cast<ExtendRec*>(static_cast<uint8_t*>(workspace) + kStatusBytes);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  try {
    mis_status_t r = cuda_status(
        launch_pdl(mis_paged_extend_kernel, dim3(1),
                   dim3(B <= 256 && (T <= 1024 || T > kFillInPlan) ? 256 : kPlanThreads), 0, st, p));
    if (r != MIS_OK || T <= kFillInPlan) return r;
    const int64_t blocks = ((int64_t)T + kFillThreads * kFillRows - 1) / (kFillThreads * kFillRows);
    return cuda_status(launch_pdl(mis_paged_fill_kernel, dim3((unsigned)blocks),
                                  dim3(kFillThreads), 0, st, p));
  } catch (...) {
    return MIS_ERR_CUDA;
  }
}

extern "C" size_t mis_paged_write_workspace_size(void) { return kStatusBytes; }

extern "C" mis_status_t mis_paged_write_kv(const mis_paged_cache* cache, const void* k,
                                           const void* v, int64_t k_row_stride,
                                           int64_t v_row_stride, int32_t T,
                                           const int32_t* src_rows, const int32_t* slot_map,
                                           int32_t n, const int32_t* position_ids,
                                           double rope_base, void* workspace, size_t ws_bytes,
                                           void* stream) {
  const mis_status_t cs = check_paged_cache(cache);
  if (cs != MIS_OK) return cs;
  if (T < 0 || n < 0) return MIS_ERR_INVALID_ARG;
  if (position_ids && (!(rope_base > 1.0) || !std::isfinite(rope_base))) return MIS_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) || ws_bytes < mis_paged_write_workspace_size())
    return MIS_ERR_WORKSPACE;
  if (!src_rows && n > T) return MIS_ERR_SHAPE;
  const int64_t w = (int64_t)cache->Hkv * cache->D;
  if (k_row_stride < w || v_row_stride < w || ((k_row_stride | v_row_stride) & 7))
    return MIS_ERR_SHAPE;
  if (n == 0) return MIS_OK;
  if (!slot_map || !aligned(slot_map, 4) || !aligned(src_rows, 4) || !aligned(position_ids, 4))
    return MIS_ERR_INVALID_ARG;
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16)) return MIS_ERR_INVALID_ARG;
  for (const Span& out : {cache_span(cache, cache->k), cache_span(cache, cache->v),
                          Span{workspace, 1, 0, (int64_t)kStatusBytes}})
    for (const Span& in : {Span{k, T, 2 * k_row_stride, 2 * w}, Span{v, T, 2 * v_row_stride, 2 * w},
                           Span{slot_map, 1, 0, 4 * (int64_t)n}, Span{src_rows, 1, 0, 4 * (int64_t)n},
                           Span{position_ids, 1, 0, 4 * (int64_t)n}})
      if (overlap(out, in)) return MIS_ERR_INVALID_ARG;
  WriteParams p;
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.kc = static_cast<__nv_bfloat16*>(cache->k);
  p.vc = static_cast<__nv_bfloat16*>(cache->v);
  p.ks = k_row_stride; p.vs = v_row_stride;
  p.page_stride = cache->page_stride; p.row_stride = cache->row_stride;
  p.head_stride = cache->head_stride;
  p.src = src_rows; p.slot = slot_map; p.pos = position_ids;
  p.n = n; p.T = T; p.Hkv = cache->Hkv;
  p.page_shift = 31 - __builtin_clz((unsigned)cache->page_size);
  p.n_slots = (int64_t)cache->n_pages * cache->page_size;
  p.status = static_cast<uint32_t*>(workspace);
  const int D = cache->D;
  if (position_ids) fill_turns(rope_base, D, p.turn);
  // an angle serves all heads of a thread; a row's heads are split over
  // threads only while its chunks alone would leave SMs idle
  const int64_t cells = (int64_t)n * (D / 16), want = 1024 * (int64_t)num_sms();
  const int64_t split = std::max<int64_t>(1, std::min<int64_t>(cache->Hkv, want / cells));
  p.hpt = (int32_t)((cache->Hkv + split - 1) / split);
  const int64_t threads = cells * ((cache->Hkv + p.hpt - 1) / p.hpt);
  const int64_t blocks = 1 + (threads + 255) / 256;
  if (blocks > 0x7fffffff) return MIS_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  try {
    return cuda_status(D == 128 ? launch_pdl(mis_paged_write_kernel<128>, dim3((unsigned)blocks),
                                             dim3(256), 0, st, p)
                                : launch_pdl(mis_paged_write_kernel<64>, dim3((unsigned)blocks),
                                             dim3(256), 0, st, p));
  } catch (...) {
    return MIS_ERR_CUDA;
  }
}
