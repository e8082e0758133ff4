// Attention of the newest rows of each request over an 8-bit paged K/V cache,
// sm_103a.
//
// Request b has len_b cached rows, the last n_b of them its new ones. New row i
// and query head q of kv head h see the keys j < len_b - n_b + i + 1:
//     s_j = scale * q k_j,   o = sum_j softmax(s)_j v_j,
// k_j and v_j being codes times 2^e of their row (mis_q8.cu). The R = n_b * G
// rows of a kv head share every key.
//
// What bounds it is the stream of codes: 2 D + 2 bytes a (key, kv head), read
// once. A warp takes 32 keys a step and 8 or 16 rows. Its lanes copy the codes
// that they need themselves (cp.async, 16 bytes each) into a ring of steps in
// shared memory, turn them into half floats in registers, where e4m3 is exact,
// and multiply with mma.sync: S^T = K Q^T with the keys on the 16-wide side,
// so that 8 rows fill a product, and O^T += V^T P^T. Neither side needs the
// codes in another order than memory's: both contractions may run over their
// index in any order that the two factors share. tcgen05 would want the codes
// as fp16 in shared memory first (its 8-bit products would round Q or P to
// 4 bits), twice their bytes written and read again, for rows that do not fill it.
//
// A row's key scale multiplies its score, its value scale its probability. The
// softmax keeps two things per row: a reference r below which weights are
// taken, and l = sum 2^(s - r). Products use P = 2^(s - r + e_v - 22): r is the
// largest s + e_v - 32 seen, moved only when one passes it by 2^5, so P lies
// below 2^15 and keeps fp16's 11 bits down to 2^-24 of the largest weighted
// value, whatever the spread of the value scales; 2^(s - r) stays within fp32
// for every e_v in [-56, 120].
//
// Work is cut evenly between blocks, not at requests: every block adds up the
// steps of all requests from the lengths on the device and walks its own
// share; pieces of a (request, kv head) that several blocks hold are joined by
// a second kernel in block order, so the same call gives the same bits.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "mis_internal.h"
#include "mis_ptx.cuh"
#include "mis_rows.cuh"

namespace mis {
namespace {

using namespace dev;

constexpr int kStep = 32;              // keys of a warp's step
constexpr int kJoinWarps = 8;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kNone = -3.0e38f;      // reference of a row that has seen nothing

struct AttnParams {
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;                          // or null
  int64_t qs, os;
  const uint8_t* k;
  const uint8_t* v;
  const uint8_t* ke;
  const uint8_t* ve;
  int64_t page_stride, row_stride, head_stride;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* cache_len;
  const int32_t* cu;
  int32_t n_pages, page_shift, max_pages;
  int32_t B, T, Hkv, G, max_rows, blocks;
  float scale_log2;
  // workspace
  uint32_t* status;
  uint32_t* flags;                     // [blocks]
  int64_t* first;                      // [B + 1]: steps before each request
  float2* rl;                          // [2 * blocks][slot rows]: (r, l) of a piece's rows
  float* part;                         // [2 * blocks][slot rows][D]
};

// A block's warps by their width (8 or 16 rows).
template <int NT>
struct Shape {
  static constexpr int kWarps = 8;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kStages = 3;
  static constexpr int kWarpRows = 8 * NT;
  static constexpr int kSlotRows = kWarps * kWarpRows;     // rows that a block holds at once
};

// A request's work. The n * G rows of a kv head are cut into tiles of a warp's
// rows; (kv head, tile) are its columns. A unit is cg columns, a warp each, over
// all keys, so that the heads of a cached row are read together (a row's 128
// bytes of one head alone are too short for HBM: 64 decoded tokens 97 us by
// single heads). Where cg leaves warps free, kWarps / cg groups of them split
// the keys. A step of 32 keys of a unit counts cg.
struct Job {
  int len, row0, n;                    // cached rows; first new row, new rows
  int steps, tiles, cols, cg, units;
  bool ok;
  __device__ __forceinline__ int64_t unit() const { return (int64_t)steps * cg; }
  __device__ __forceinline__ int64_t cost() const { return unit() * units; }
};

template <int NT>
__device__ __forceinline__ Job job_of(const AttnParams& p, int b) {
  constexpr int W = Shape<NT>::kWarps, WR = Shape<NT>::kWarpRows;
  Job j;
  j.len = p.cache_len[b];
  j.row0 = p.cu[b];
  const int end = p.cu[b + 1];
  j.ok = j.row0 >= 0 && end >= j.row0 && end <= p.T && end - j.row0 <= p.max_rows && j.len >= 0 &&
         j.len <= (int64_t)p.max_pages << p.page_shift && end - j.row0 <= j.len;
  j.n = j.ok ? end - j.row0 : 0;
  j.steps = j.n ? (j.len + kStep - 1) / kStep : 0;
  j.tiles = (j.n * p.G + WR - 1) / WR;
  j.cols = j.tiles * p.Hkv;
  j.units = (j.cols + W - 1) / W;
  j.cg = j.units > 1 ? (j.cols + j.units - 1) / j.units : j.cols;
  return j;
}

// Blocks that take part: none has less than 8 steps.
__device__ __forceinline__ int blocks_for(int64_t total, int blocks) {
  return (int)min((int64_t)blocks, max((int64_t)1, total / 8));
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 u;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(a));
  return u;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 u;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(u.x), "=r"(u.y) : "r"(a));
  return u;
}
__device__ __forceinline__ uint32_t lds_byte(uint32_t a) {
  uint32_t u;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(u) : "r"(a));
  return u;
}

__device__ __forceinline__ void mma16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Bytes of w that hold the NaN code, as 0x80 each.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

template <int D, int NT>
struct Cfg {
  static constexpr int kWarps = Shape<NT>::kWarps, STAGES = Shape<NT>::kStages;
  static constexpr int KC = D / 64;            // 64-wide chunks of a K row
  static constexpr int VB = D / 8;             // bytes of a V row that a lane takes
  static constexpr int MT = D / 16;            // 16-wide tiles of O^T
  static constexpr int kKBytes = kStep * D, kVBytes = kStep * D, kEBytes = 64;
  static constexpr int kStage = kKBytes + kVBytes + kEBytes;
  static constexpr int kRing = kWarps * STAGES * kStage;
  static constexpr int kSmem = kRing + kWarps * Shape<NT>::kWarpRows * 8;
  static_assert(Shape<NT>::kWarpRows * D * 4 <= kStage, "a warp's rows fit a step");
};

// Walks the pieces of units that a block's share holds.
template <int NT>
struct Walk {
  int64_t left;                        // of the share from this piece on, in costs
  int64_t off;                         // of the unit before this piece
  int b, u;                            // request, its unit
  int k0, k1;                          // key steps of the piece
  Job j;

  __device__ __forceinline__ void enter(const AttnParams& p, int b_, int64_t from) {
    b = b_;
    j = job_of<NT>(p, b);
    u = (int)(from / j.unit());
    off = from - u * j.unit();
    piece();
  }
  __device__ __forceinline__ void piece() {
    k0 = (int)(off / j.cg);
    k1 = ends() ? j.steps : (int)((off + left) / j.cg);
  }
  // whether the piece reaches the unit's end
  __device__ __forceinline__ bool ends() const { return off + left >= j.unit(); }
  // the next piece; false at the end of the share
  __device__ __forceinline__ bool next(const AttnParams& p) {
    left -= j.unit() - off;
    if (left <= 0) return false;
    off = 0;
    if (++u == j.units) {
      u = 0;
      do j = job_of<NT>(p, ++b);
      while (j.cost() == 0);
    }
    piece();
    return true;
  }
};

template <int D, int NT>
__global__ void __launch_bounds__(Shape<NT>::kThreads, 1)
mis_q8_attn_kernel(const __grid_constant__ AttnParams p) {
  using C = Cfg<D, NT>;
  constexpr int kWarps = Shape<NT>::kWarps, kThreads = Shape<NT>::kThreads, STAGES = Shape<NT>::kStages;
  constexpr int WR = Shape<NT>::kWarpRows, SR = Shape<NT>::kSlotRows;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t s_sum[kWarps];
  __shared__ int64_t s_from;
  __shared__ int s_req;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  griddep_launch_dependents();
  griddep_wait();

  // Every block adds up the steps of all requests, a run of them a thread, and
  // finds the request that its share starts in.
  const int run = (p.B + kThreads - 1) / kThreads;
  const int rb0 = min(p.B, tid * run), rb1 = min(p.B, rb0 + run);
  int64_t mine = 0;
  bool bad = false;
  for (int b = rb0; b < rb1; ++b) {
    const Job j = job_of<NT>(p, b);
    bad |= !j.ok;
    mine += j.cost();
  }
  int64_t upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) s_sum[warp] = upto;
  if (tid == 0) s_req = -1;
  bad = __syncthreads_or(bad);
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) upto += s_sum[w];
    total += s_sum[w];
  }
  const int blocks = blocks_for(total, p.blocks);
  Walk<NT> f;                          // of the copies, ahead of the products
  const int64_t share0 = total * min((int)blockIdx.x, blocks) / blocks;
  f.left = total * min((int)blockIdx.x + 1, blocks) / blocks - share0;
  {
    int64_t at = upto - mine;
    const bool here = share0 >= at && share0 < upto;
    if (here || blockIdx.x == 0)
      for (int b = rb0; b < rb1; ++b) {
        const int64_t next = at + job_of<NT>(p, b).cost();
        if (here && share0 >= at && share0 < next) { s_req = b; s_from = share0 - at; }
        if (blockIdx.x == 0) p.first[b] = at;
        at = next;
      }
    if (blockIdx.x == 0 && tid == 0) p.first[p.B] = total;
  }
  __syncthreads();
  if (f.left <= 0) {
    if (tid == 0) p.flags[blockIdx.x] = bad ? kDevIndex : 0u;
    return;
  }
  f.enter(p, s_req, s_from);
  Walk<NT> w = f;                      // of the products
  const int64_t share_left = f.left;

  const uint32_t ring = smem_u32(smem) + warp * (STAGES * C::kStage);
  float2* s_rl = reinterpret_cast<float2*>(smem + C::kRing);      // [warp][row]

  // ---- copies: the step at hand, whose page ids were asked for a step ago
  bool f_on = true;                    // a step is at hand
  int f_step = 0, f_h = 0, f_kgs = 1, f_head = 0, f_len = 0, id0 = 0, id1 = 0;
  uint32_t hidden = 0;                 // two bits a stage: strips without rows or page
  bool bad_page = false;
  auto first_step = [&] {              // none where the unit has no column for the warp
    const int kg = warp / f.j.cg, col = f.u * f.j.cg + warp - kg * f.j.cg;
    f_h = col / f.j.tiles;
    f_kgs = kWarps / f.j.cg;
    return kg < f_kgs && col < f.j.cols ? f.k0 + kg : f.k1;
  };
  auto find = [&](int step) {          // from this step on: the next one that the warp takes, and its ids
    for (;;) {
      if (step < f.k1) break;
      if (!f.next(p)) { f_on = false; return; }
      step = first_step();
    }
    f_step = step;
    const int32_t* row = p.table + (int64_t)f.b * p.table_stride;
    const int key = step * kStep;
    id0 = row[key >> p.page_shift];
    id1 = key + 16 < f.j.len ? row[(key + 16) >> p.page_shift] : id0;
    f_len = f.j.len;
    f_head = f_h;
  };
  auto copy = [&](int stage) {
    uint32_t hide = 0;
    if (f_on) {
      const uint32_t at = ring + stage * C::kStage;
      const int key = f_step * kStep;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int id = s ? id1 : id0;
        const bool off = id < 0 || id >= p.n_pages;
        if (key + 16 * s >= f_len) { hide |= 1u << s; continue; }
        if (off) { hide |= 1u << s; bad_page = true; continue; }
        const int in = (key + 16 * s) & ((1 << p.page_shift) - 1);
        const int64_t from = (int64_t)id * p.page_stride + (int64_t)in * p.row_stride + (int64_t)f_head * p.head_stride;
        const uint32_t dst = at + s * (16 * D) + lane * 16;
#pragma unroll
        for (int c = 0; c < C::KC; ++c) {
          cp16(dst + (2 * c) * 512, p.k + from + (int64_t)g * p.row_stride + 64 * c + 16 * t);
          cp16(dst + (2 * c + 1) * 512, p.k + from + (int64_t)(g + 8) * p.row_stride + 64 * c + 16 * t);
        }
        const uint32_t vdst = at + C::kKBytes + s * (16 * D) + lane * C::VB;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = 2 * t + (e & 1) + 8 * (e >> 1);
          const uint8_t* src = p.v + from + (int64_t)row * p.row_stride + C::VB * g;
          if constexpr (D == 128) cp16(vdst + e * (32 * C::VB), src);
          else cp8(vdst + e * (32 * C::VB), src);
        }
        if (lane < 2) {
          const int64_t ex = (((int64_t)id * p.Hkv + f_head) << p.page_shift) + in;
          cp16(at + C::kKBytes + C::kVBytes + 32 * s + 16 * lane, (lane ? p.ve : p.ke) + ex);
        }
      }
      find(f_step + f_kgs);
    }
    hidden = (hidden & ~(3u << (2 * stage))) | hide << (2 * stage);
    cp_commit();
  };
  find(first_step());
  int stage_in = 0, stage_out = 0;
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) copy(stage_in++);

  // ---- products, piece by piece
  for (;;) {
    const int cg = w.j.cg, kgs = kWarps / cg, kg = warp / cg, col = w.u * cg + warp - kg * cg;
    const int head = col / w.j.tiles;                     // kv head
    const int row_first = (col - head * w.j.tiles) * WR;  // of its n * G rows
    const int rows = kg < kgs && col < w.j.cols ? min(WR, w.j.n * p.G - row_first) : 0;
    const int len = w.j.len, n = w.j.n;
    // Q of the warp's rows as half floats, each row in units of its own power
    // of two (its largest element in [2^14, 2^15), so nothing that counts is lost)
    uint32_t qf[NT][4 * C::KC][2];
    float cq[NT][2];                   // of rows 2t, 2t + 1: that unit, the scale and log2(e)
    int lim[NT][2];                    // keys that they see
#pragma unroll
    for (int a = 0; a < NT; ++a) {
      const int row = 8 * a + g;
      uint4 x[2 * C::KC];
      const bool live = row < rows;
      float m = 0.f;
      if (live) {
        const int at = row_first + row, i = at / p.G;
        const __nv_bfloat16* src = p.q + (int64_t)(w.j.row0 + i) * p.qs + (int64_t)(head * p.G + at - i * p.G) * D + 16 * t;
#pragma unroll
        for (int c = 0; c < C::KC; ++c) {
          x[2 * c] = *reinterpret_cast<const uint4*>(src + 64 * c);
          x[2 * c + 1] = *reinterpret_cast<const uint4*>(src + 64 * c + 8);
        }
      } else {
#pragma unroll
        for (int c = 0; c < 2 * C::KC; ++c) x[c] = make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int c = 0; c < 2 * C::KC; ++c) {
        float f8[8];
        bf16x8_to_float(x[c], f8);
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(f8[e]));
      }
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      int ex = (__float_as_int(m) >> 23) - 127 - 14;      // m * 2^-ex in [2^14, 2^15)
      ex = m > 0.f && m <= 3.4e38f ? max(ex, -126) : 0;
      const float unit = pow2(-ex);
#pragma unroll
      for (int c = 0; c < C::KC; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4& y = x[2 * c + (i >> 1)];
          const uint32_t w0 = i & 1 ? y.z : y.x, w1 = i & 1 ? y.w : y.y;
          qf[a][4 * c + i][0] = half2_of(__uint_as_float(w0 << 16) * unit, __uint_as_float(w0 & 0xffff0000u) * unit);
          qf[a][4 * c + i][1] = half2_of(__uint_as_float(w1 << 16) * unit, __uint_as_float(w1 & 0xffff0000u) * unit);
        }
      const float mine_cq = pow2(ex) * p.scale_log2;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        cq[a][e] = __shfl_sync(0xffffffffu, mine_cq, (2 * t + e) * 4);
        const int r2 = 8 * a + 2 * t + e;
        lim[a][e] = r2 < rows ? len - n + (row_first + r2) / p.G + 1 : 0;
      }
    }
    const int all_see = rows > 0 ? len - n + row_first / p.G + 1 : 0;   // keys that every row sees

    float o[NT][C::MT][4], r[NT][2], l[NT][2];
#pragma unroll
    for (int a = 0; a < NT; ++a) {
      r[a][0] = r[a][1] = kNone;
      l[a][0] = l[a][1] = 0.f;
#pragma unroll
      for (int j = 0; j < C::MT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[a][j][e] = 0.f;
    }

    for (int step = rows > 0 ? w.k0 + kg : w.k1; step < w.k1; step += kgs) {
      __syncwarp();                    // every lane is done with the step before
      copy(stage_in);
      stage_in = stage_in + 1 == STAGES ? 0 : stage_in + 1;
      cp_wait<STAGES - 1>();
      __syncwarp();
      const uint32_t at = ring + stage_out * C::kStage;
      const uint32_t hide = (hidden >> (2 * stage_out)) & 3u;
      stage_out = stage_out + 1 == STAGES ? 0 : stage_out + 1;
      const int key0 = step * kStep;
      const bool masked = hide || key0 + kStep > all_see;

      // S^T of 2 x 16 keys
      float s[2][NT][4];
      float vs[2][2];                  // 2^(e_v - 22) of keys g, g + 8
      int ev[2][2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int a = 0; a < NT; ++a)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[k][a][e] = 0.f;
#pragma unroll
        for (int c = 0; c < C::KC; ++c) {
          const uint4 lo = lds16(at + k * (16 * D) + (2 * c) * 512 + lane * 16);
          const uint4 hi = lds16(at + k * (16 * D) + (2 * c + 1) * 512 + lane * 16);
          const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w}, wh[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t a0 = e4m3x2_to_half2((uint16_t)wl[i]), a2 = e4m3x2_to_half2((uint16_t)(wl[i] >> 16));
            const uint32_t a1 = e4m3x2_to_half2((uint16_t)wh[i]), a3 = e4m3x2_to_half2((uint16_t)(wh[i] >> 16));
#pragma unroll
            for (int a = 0; a < NT; ++a)
              mma16816(s[k][a], a0, a1, a2, a3, qf[a][4 * c + i][0], qf[a][4 * c + i][1]);
          }
        }
        const uint32_t ex = at + C::kKBytes + C::kVBytes + 32 * k + g;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float kf = pow2(q8_exp(lds_byte(ex + 8 * x)));
          ev[k][x] = q8_exp(lds_byte(ex + 16 + 8 * x));
          vs[k][x] = pow2(ev[k][x] - 22);
#pragma unroll
          for (int a = 0; a < NT; ++a)
#pragma unroll
            for (int e = 0; e < 2; ++e) s[k][a][2 * x + e] = s[k][a][2 * x + e] * kf * cq[a][e];
        }
      }
      if (masked) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int a = 0; a < NT; ++a)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = key0 + 16 * k + g + 8 * (e >> 1);
              if (((hide >> k) & 1) || key >= lim[a][e & 1]) s[k][a][e] = -INFINITY;
            }
      }
      // the references hold until a weighted value passes them by 2^5
      bool over = false;
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float most = 37.f - (float)ev[k][x];
#pragma unroll
          for (int a = 0; a < NT; ++a)
#pragma unroll
            for (int e = 0; e < 2; ++e) over |= s[k][a][2 * x + e] - r[a][e] > most;
        }
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int a = 0; a < NT; ++a)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float m = r[a][e];
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int x = 0; x < 2; ++x) m = fmaxf(m, s[k][a][2 * x + e] + (float)(ev[k][x] - 32));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
            const float f1 = m > r[a][e] ? ex2(r[a][e] - m) : 1.f;
            r[a][e] = m;
            l[a][e] *= f1;
#pragma unroll
            for (int j = 0; j < C::MT; ++j) {
              o[a][j][e] *= f1;
              o[a][j][e + 2] *= f1;
            }
          }
      }
      uint32_t pf[2][NT][2];           // P^T as the products' second factor
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int a = 0; a < NT; ++a) {
          float x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float y = ex2(s[k][a][e] - r[a][e & 1]);
            l[a][e & 1] += y;
            x[e] = y * vs[k][e >> 1];
          }
          pf[k][a][0] = transpose8x8(half2_of(x[0], x[1]));
          pf[k][a][1] = transpose8x8(half2_of(x[2], x[3]));
        }
      // O^T += V^T P^T
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        constexpr int W = C::VB / 4;
        uint32_t v[4][W];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t from = at + C::kKBytes + k * (16 * D) + e * (32 * C::VB) + lane * C::VB;
          if constexpr (D == 128) {
            const uint4 u = lds16(from);
            v[e][0] = u.x; v[e][1] = u.y; v[e][2] = u.z; v[e][3] = u.w;
          } else {
            const uint2 u = lds8(from);
            v[e][0] = u.x; v[e][1] = u.y;
          }
        }
        if (masked) {
          // rows that nobody sees hold anything; NaN that some rows see
          // reaches those alone (0 x NaN in the product would reach all)
          uint32_t any = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = key0 + 16 * k + 2 * t + (e & 1) + 8 * (e >> 1);
            const bool gone = ((hide >> k) & 1) || key >= len;
#pragma unroll
            for (int i = 0; i < W; ++i) {
              if (gone) v[e][i] = 0u;
              any |= nan_codes(v[e][i]);
            }
          }
          if (__any_sync(0xffffffffu, any)) {
            uint32_t see[NT][2];
#pragma unroll
            for (int a = 0; a < NT; ++a)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const int key = key0 + 16 * k + g + 8 * x;
                see[a][x] = transpose8x8((key < lim[a][0] ? 0x3c00u : 0u) | (key < lim[a][1] ? 0x3c000000u : 0u));
              }
#pragma unroll
            for (int i = 0; i < W; ++i) {
              uint32_t f1[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t nn = nan_codes(v[e][i]) >> 7;     // 1 in each byte
                v[e][i] &= ~(nn * 0xffu);
                f1[e] = nn * 0x38u;                              // the code of one
              }
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const uint32_t c01 = __byte_perm(f1[0], f1[1], y ? 0x7362 : 0x5140);
                const uint32_t c23 = __byte_perm(f1[2], f1[3], y ? 0x7362 : 0x5140);
#pragma unroll
                for (int a = 0; a < NT; ++a) {
                  float cnt[4] = {0.f, 0.f, 0.f, 0.f};
                  mma16816(cnt, e4m3x2_to_half2((uint16_t)c01), e4m3x2_to_half2((uint16_t)(c01 >> 16)),
                           e4m3x2_to_half2((uint16_t)c23), e4m3x2_to_half2((uint16_t)(c23 >> 16)), see[a][0], see[a][1]);
#pragma unroll
                  for (int e = 0; e < 4; ++e)
                    if (cnt[e] > 0.f) o[a][2 * i + y][e] = __int_as_float(0x7fffffff);
                }
              }
            }
          }
        }
#pragma unroll
        for (int i = 0; i < W; ++i)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t c01 = __byte_perm(v[0][i], v[1][i], y ? 0x7362 : 0x5140);
            const uint32_t c23 = __byte_perm(v[2][i], v[3][i], y ? 0x7362 : 0x5140);
            const uint32_t a0 = e4m3x2_to_half2((uint16_t)c01), a1 = e4m3x2_to_half2((uint16_t)(c01 >> 16));
            const uint32_t a2 = e4m3x2_to_half2((uint16_t)c23), a3 = e4m3x2_to_half2((uint16_t)(c23 >> 16));
#pragma unroll
            for (int a = 0; a < NT; ++a) mma16816(o[a][2 * i + y], a0, a1, a2, a3, pf[k][a][0], pf[k][a][1]);
          }
      }
    }

    // ---- the piece is done: the warps' sums meet in shared memory, each in
    // the ring's step that its next copy would fill
    __syncwarp();
    {
      float* dst = reinterpret_cast<float*>(smem + warp * (STAGES * C::kStage) + stage_in * C::kStage);
#pragma unroll
      for (int a = 0; a < NT; ++a)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = l[a][e];
          x += __shfl_xor_sync(0xffffffffu, x, 4);
          x += __shfl_xor_sync(0xffffffffu, x, 8);
          x += __shfl_xor_sync(0xffffffffu, x, 16);
          const int row = 8 * a + 2 * t + e;
          if (row >= rows) continue;
          if (g == 0) s_rl[warp * WR + row] = make_float2(r[a][e], x);
          float4* d4 = reinterpret_cast<float4*>(dst + row * D + g * (2 * C::MT));
#pragma unroll
          for (int j = 0; j < C::MT; j += 2)
            d4[j / 2] = make_float4(o[a][j][e], o[a][j][e + 2], o[a][j + 1][e], o[a][j + 1][e + 2]);
        }
      if (lane == 0) s_sum[warp] = stage_in;
    }
    __syncthreads();
    const bool first = w.left == share_left, whole = w.off == 0 && w.ends();
    const int slot = 2 * blockIdx.x + (first ? 0 : 1);
    const int height = min(WR, n * p.G);                  // of a column
    for (int x = tid; x < cg * height * (D / 4); x += kThreads) {
      const int c4 = x % (D / 4), y = x / (D / 4), wc = y / height, in = y - wc * height;
      const int ocol = w.u * cg + wc, ohead = ocol / w.j.tiles, row = (ocol - ohead * w.j.tiles) * WR + in;
      if (ocol >= w.j.cols || row >= n * p.G) continue;
      float m = kNone;
      for (int z = 0; z < kgs; ++z) m = fmaxf(m, s_rl[(z * cg + wc) * WR + in].x);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      float sum = 0.f;
      for (int z = 0; z < kgs; ++z) {
        const int from = z * cg + wc;
        const float2 rl = s_rl[from * WR + in];
        const float f1 = ex2(rl.x - m);
        const float4 v4 = *reinterpret_cast<const float4*>(smem + from * (STAGES * C::kStage) +
                                                           (int)s_sum[from] * C::kStage + (in * D + 4 * c4) * 4);
        sum += f1 * rl.y;
        acc.x += f1 * v4.x;
        acc.y += f1 * v4.y;
        acc.z += f1 * v4.z;
        acc.w += f1 * v4.w;
      }
      if (whole) {
        const int i = row / p.G, qh = ohead * p.G + row - i * p.G;
        // the products' weights carry 2^-22
        const float inv = sum != 0.f ? 4194304.f / sum : 0.f;
        *reinterpret_cast<uint2*>(p.o + (int64_t)(w.j.row0 + i) * p.os + (int64_t)qh * D + 4 * c4) =
            sum != 0.f ? make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv))
                       : make_uint2(0u, 0u);
        if (p.lse && c4 == 0)
          p.lse[(int64_t)qh * p.T + w.j.row0 + i] = sum != 0.f ? (m + log2f(sum)) * kLn2 : -INFINITY;
      } else {
        const int64_t at = (int64_t)slot * SR + wc * WR + in;
        *reinterpret_cast<float4*>(p.part + at * D + 4 * c4) = acc;
        if (c4 == 0) p.rl[at] = make_float2(m, sum);
      }
    }
    __syncthreads();
    if (!w.next(p)) break;
  }
  cp_wait<0>();
  bad_page = __syncthreads_or(bad_page);
  if (tid == 0) p.flags[blockIdx.x] = bad || bad_page ? kDevIndex : 0u;
}

// Joins the pieces of units that several blocks hold, in block order. Grid:
// (request, kv head) by groups of rows; `share` warps (a power of two) take a
// row's pieces in turn, so that a single long request's many pieces do not
// queue behind one warp (8192 rows of 8 heads: 63 us by one).
template <int D, int NT>
__global__ void __launch_bounds__(32 * kJoinWarps)
mis_q8_join_kernel(const __grid_constant__ AttnParams p, int share) {
  constexpr int SR = Shape<NT>::kSlotRows, WR = Shape<NT>::kWarpRows, E = D / 32;
  __shared__ float s_acc[kJoinWarps][D + 1];
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x == 0 && blockIdx.y == 0 && warp == 0) {
    uint32_t f = 0;
    for (int c = lane; c < p.blocks; c += 32) f |= p.flags[c];
    f = __reduce_or_sync(0xffffffffu, f);
    if (lane == 0) {
      p.status[0] = f;
      p.status[1] = f ? 0x60u : 0u;
    }
  }
  const int b = blockIdx.x / p.Hkv, h = blockIdx.x - b * p.Hkv;
  const int sub = warp & (share - 1), row = blockIdx.y * (kJoinWarps / share) + warp / share;
  const Job j = job_of<NT>(p, b);
  if ((int)blockIdx.y * (kJoinWarps / share) >= j.n * p.G) return;
  const int64_t total = p.first[p.B];
  const int blocks = blocks_for(total, p.blocks);
  // the blocks that hold the first and last step of the row's unit
  auto holder = [&](int64_t x) {
    int y = (int)(x * blocks / total);
    while (total * (y + 1) / blocks <= x) ++y;
    while (total * y / blocks > x) --y;
    return y;
  };
  const bool live = row < j.n * p.G;
  const int col = h * j.tiles + (live ? row : 0) / WR, u = col / j.cg;
  const int64_t u0 = p.first[b] + u * j.unit();
  const int c0 = holder(u0), c1 = holder(u0 + j.unit() - 1);
  const bool split = live && c0 != c1;
  const int64_t in = (col - u * j.cg) * WR + row % WR;
  // the first block's piece is its last one where its share starts before the unit
  const int64_t at0 = (2 * c0 + (total * c0 / blocks < u0 ? 1 : 0)) * (int64_t)SR + in;
  auto piece = [&](int y) { return y == c0 ? at0 : (int64_t)(2 * y) * SR + in; };
  float m = kNone, sum = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  if (split) {
    for (int y = c0 + lane; y <= c1; y += 32) m = fmaxf(m, p.rl[piece(y)].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll 4
    for (int y = c0 + sub; y <= c1; y += share) {
      const int64_t at = piece(y);
      const float2 rl = p.rl[at];
      const float f1 = ex2(rl.x - m);
      sum += f1 * rl.y;
      const float* z = p.part + at * D + lane * E;
      if constexpr (E == 4) {
        const float4 z4 = *reinterpret_cast<const float4*>(z);
        acc[0] += f1 * z4.x; acc[1] += f1 * z4.y; acc[2] += f1 * z4.z; acc[3] += f1 * z4.w;
      } else {
        const float2 z2 = *reinterpret_cast<const float2*>(z);
        acc[0] += f1 * z2.x; acc[1] += f1 * z2.y;
      }
    }
  }
  if (share > 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) s_acc[warp][e * 32 + lane] = acc[e];
    if (lane == 0) s_acc[warp][D] = sum;
    __syncthreads();
    if (sub) return;
    for (int y = 1; y < share; ++y) {
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += s_acc[warp + y][e * 32 + lane];
      sum += s_acc[warp + y][D];
    }
  }
  if (!split) return;
  const int i = row / p.G, head = h * p.G + row - i * p.G;
  const float inv = sum != 0.f ? 4194304.f / sum : 0.f;
  uint32_t out[E / 2];
#pragma unroll
  for (int e = 0; e < E / 2; ++e) out[e] = sum != 0.f ? pack_bf16(acc[2 * e] * inv, acc[2 * e + 1] * inv) : 0u;
  __nv_bfloat16* dst = p.o + (int64_t)(j.row0 + i) * p.os + (int64_t)head * D + lane * E;
  if constexpr (E == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
  else *reinterpret_cast<uint32_t*>(dst) = out[0];
  if (p.lse && lane == 0)
    p.lse[(int64_t)head * p.T + j.row0 + i] = sum != 0.f ? (m + log2f(sum)) * kLn2 : -INFINITY;
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

mis_status_t check_desc(const mis_paged_attn_desc* d, const mis_paged_cache_q8* c) {
  if (!d) return MIS_ERR_INVALID_ARG;
  const mis_status_t cs = check_paged_cache_q8(c);
  if (cs != MIS_OK) return cs;
  if (d->B < 1 || d->T < 0 || d->Hq < 1 || d->max_rows < 1) return MIS_ERR_INVALID_ARG;
  const float size = std::fabs(d->scale);
  if (!(size <= 1e20f) || (size != 0.f && size < 1e-20f)) return MIS_ERR_INVALID_ARG;
  if (d->max_rows > MIS_PAGED_MAX_ROWS) return MIS_ERR_UNSUPPORTED;
  if (d->Hq % c->Hkv) return MIS_ERR_SHAPE;
  if (d->Hq / c->Hkv > 128) return MIS_ERR_UNSUPPORTED;
  // columns, and the join's grid, are counted in 32 bits
  if ((int64_t)d->B * c->Hkv > 0x7fffffff || (int64_t)d->max_rows * d->Hq > 0x7fffffff) return MIS_ERR_UNSUPPORTED;
  return MIS_OK;
}

int head_rows(const mis_paged_attn_desc* d, const mis_paged_cache_q8* c) { return d->max_rows * (d->Hq / c->Hkv); }

struct AttnWs { size_t flags, first, rl, part, total; };

AttnWs workspace_of(const mis_paged_attn_desc* d, const mis_paged_cache_q8* c) {
  const size_t G = (size_t)num_sms(), SR = head_rows(d, c) <= 8 ? Shape<1>::kSlotRows : Shape<2>::kSlotRows;
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  AttnWs w;
  w.flags = kStatusBytes;
  w.first = w.flags + up(G * 4);
  w.rl = w.first + up(((size_t)d->B + 1) * 8);
  w.part = w.rl + up(2 * G * SR * sizeof(float2));
  w.total = w.part + 2 * G * SR * (size_t)c->D * sizeof(float);
  return w;
}

template <int D, int NT>
mis_status_t launch(const AttnParams& p, cudaStream_t st) {
  using C = Cfg<D, NT>;
  auto kern = mis_q8_attn_kernel<D, NT>;
  if (!kernel_attr_once(reinterpret_cast<const void*>(kern), C::kSmem)) return MIS_ERR_CUDA;
  if (launch_pdl(kern, dim3((unsigned)p.blocks), dim3(Shape<NT>::kThreads), C::kSmem, st, p) != cudaSuccess)
    return MIS_ERR_CUDA;
  // warps of a row: all of a block's while the rows are few
  const int64_t rows = (int64_t)p.max_rows * p.G, most = 4 * (int64_t)num_sms() / (p.B * (int64_t)p.Hkv * rows) + 1;
  const int share = most >= 8 ? 8 : most >= 4 ? 4 : most >= 2 ? 2 : 1, per = kJoinWarps / share;
  return launch_pdl(mis_q8_join_kernel<D, NT>, dim3((unsigned)(p.B * p.Hkv), (unsigned)((rows + per - 1) / per)),
                    dim3(32 * kJoinWarps), 0, st, p, share) == cudaSuccess
             ? MIS_OK
             : MIS_ERR_CUDA;
}

}  // namespace
}  // namespace mis

using namespace mis;

extern "C" size_t mis_paged_attention_q8_workspace_size(const mis_paged_attn_desc* desc,
                                                        const mis_paged_cache_q8* cache) {
  return check_desc(desc, cache) == MIS_OK ? workspace_of(desc, cache).total : 0;
}

extern "C" mis_status_t mis_paged_attention_q8_fwd(
    const mis_paged_attn_desc* desc, const mis_paged_cache_q8* cache, const void* q, void* o, float* lse,
    int64_t q_row_stride, int64_t o_row_stride, const int32_t* block_table, int32_t max_pages,
    int64_t block_table_stride, const int32_t* cache_len, const int32_t* cu_rows, void* workspace,
    size_t ws_bytes, void* stream) {
  const mis_status_t ds = check_desc(desc, cache);
  if (ds != MIS_OK) return ds;
  if (max_pages < 1) return MIS_ERR_INVALID_ARG;
  if ((int64_t)max_pages * cache->page_size > 0x7fffff00 || block_table_stride < max_pages) return MIS_ERR_SHAPE;
  if (!block_table || !cache_len || !cu_rows || !aligned(block_table, 4) || !aligned(cache_len, 4) ||
      !aligned(cu_rows, 4) || !aligned(lse, 4))
    return MIS_ERR_INVALID_ARG;
  const int D = cache->D;
  const int64_t wq = (int64_t)desc->Hq * D;
  if (q_row_stride < wq || o_row_stride < wq || ((q_row_stride | o_row_stride) & 7)) return MIS_ERR_SHAPE;
  if (desc->T > 0 && (!q || !o || !aligned(q, 16) || !aligned(o, 16))) return MIS_ERR_INVALID_ARG;
  const AttnWs ws = workspace_of(desc, cache);
  if (!workspace || !aligned(workspace, 256) || ws_bytes < ws.total) return MIS_ERR_WORKSPACE;
  if (desc->T > 0) {
    const int64_t T = desc->T, B = desc->B;
    const Span in[8] = {{q, T, 2 * q_row_stride, 2 * wq}, codes_span(cache, cache->k), codes_span(cache, cache->v),
                        exps_span(cache, cache->k_exp), exps_span(cache, cache->v_exp),
                        {block_table, B, 4 * block_table_stride, 4 * (int64_t)max_pages},
                        {cache_len, 1, 0, 4 * B}, {cu_rows, 1, 0, 4 * B + 4}};
    const Span out[3] = {{o, T, 2 * o_row_stride, 2 * wq}, {lse, 1, 0, 4 * T * desc->Hq},
                         {workspace, 1, 0, (int64_t)ws.total}};
    for (int i = 0; i < 3; ++i) {
      for (const Span& x : in)
        if (overlap(out[i], x)) return MIS_ERR_INVALID_ARG;
      for (int j = 0; j < i; ++j)
        if (overlap(out[i], out[j])) return MIS_ERR_INVALID_ARG;
    }
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (desc->T == 0) return cudaMemsetAsync(workspace, 0, 8, st) == cudaSuccess ? MIS_OK : MIS_ERR_CUDA;
  uint8_t* base = static_cast<uint8_t*>(workspace);
  AttnParams p;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.qs = q_row_stride; p.os = o_row_stride;
  p.k = static_cast<const uint8_t*>(cache->k);
  p.v = static_cast<const uint8_t*>(cache->v);
  p.ke = cache->k_exp; p.ve = cache->v_exp;
  // strides of extents of one are not used
  p.page_stride = cache->n_pages > 1 ? cache->page_stride : 0;
  p.row_stride = cache->row_stride;
  p.head_stride = cache->Hkv > 1 ? cache->head_stride : 0;
  p.table = block_table; p.table_stride = block_table_stride;
  p.cache_len = cache_len; p.cu = cu_rows;
  p.n_pages = cache->n_pages;
  p.page_shift = 31 - __builtin_clz((unsigned)cache->page_size);
  p.max_pages = max_pages;
  p.B = desc->B; p.T = desc->T; p.Hkv = cache->Hkv; p.G = desc->Hq / cache->Hkv;
  p.max_rows = desc->max_rows;
  p.blocks = num_sms();
  p.scale_log2 = (desc->scale != 0.f ? desc->scale : 1.f / std::sqrt((float)D)) * 1.4426950408889634f;
  p.status = reinterpret_cast<uint32_t*>(base);
  p.flags = reinterpret_cast<uint32_t*>(base + ws.flags);
  p.first = reinterpret_cast<int64_t*>(base + ws.first);
  p.rl = reinterpret_cast<float2*>(base + ws.rl);
  p.part = reinterpret_cast<float*>(base + ws.part);
  try {
    const bool narrow = head_rows(desc, cache) <= 8;
    if (D == 128) return narrow ? launch<128, 1>(p, st) : launch<128, 2>(p, st);
    return narrow ? launch<64, 1>(p, st) : launch<64, 2>(p, st);
  } catch (...) {
    return MIS_ERR_CUDA;
  }
}
