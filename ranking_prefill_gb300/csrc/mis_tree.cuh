// Parts of the two tree-attention kernels that are alike: parameters, requests
// and units, a block's share of the steps, the copies of Q, K and V, the
// cleaning of V rows.
#pragma once
#include <cuda_bf16.h>

#include "mis_internal.h"
#include "mis_ptx.cuh"

namespace mis {
namespace tree {

using namespace dev;

constexpr int kKeys = 128;                       // keys of a step
constexpr float kGrow = 8.0f;                    // log2 units a score may pass the reference by
constexpr float kEmpty = -3.402823466e38f;       // maximum of a row that has seen nothing: below any score
// Scores are taken times the scale's sign, maxima and references kept before
// its size. Scores this far from zero (log2 units) have their reference taken
// off first: scale * reference rounds by half its last bit, 2^-15 here
constexpr float kFar = 1024.0f;
constexpr float kLn2 = 0.69314718055994530942f;

struct TreeParams {
  const __nv_bfloat16* v;
  __nv_bfloat16* o;
  float* lse;
  int64_t vs, os;
  int32_t n_pages, page_shift, max_pages;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* cache_len;
  const int32_t* cu;
  const int32_t* parents;
  int32_t B, T, Hkv, G, max_nodes;
  int32_t npt;             // nodes of a row tile
  int32_t npu;             // nodes of a unit: of its row tile, or of its two
  int32_t lanes;           // units rt, rt + lanes, ... of all requests and kv heads form a lane, and the
                           // lanes lie end to end: units that share K and V are worked on at the same
                           // time, by blocks that start a lane's length apart, and meet in L2
  uint32_t g_magic;        // ceil(2^32 / G): n / G = umulhi(n, magic) for n < N, 1 < G <= 128
  float scale_log2;
  uint32_t* cta_status;    // [blocks][2]
  int4* meta;              // [blocks] the split unit that starts in the block: its first row of q,
                           // columns, kv head, pieces
  float2* ml;              // [2 * blocks][rows of a unit] (max before the scale, sum) of a piece
  float* part;             // [2 * blocks][rows of a unit][D]
  uint64_t wait_ns;
  uint32_t stall;
};

// A bounded wait in few instructions (it stands at some thirty places): a wait
// that runs out, or sees that another gave up, returns false. The site goes to
// shared memory and to the status word when the block ends.
struct Bound {
  volatile uint32_t* gave_up;
  uint64_t limit_ns;
};
__device__ __forceinline__ bool spin(uint32_t bar, uint32_t parity, const Bound& w, uint32_t where) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  do {
    if (mbar_try_wait(bar, parity)) return true;
    if (*w.gave_up) return false;
  } while (globaltimer() - t0 <= w.limit_ns);
  *w.gave_up = where;
  return false;
}

// One request, checked. Its steps are the 128-key tiles of its cached rows,
// then those of its new rows. When the new rows fit behind the last, partial
// cache tile (from the next multiple of 8 rows, a copy's granularity) they
// share its step: a decoded token costs no step of its own.
struct Req {
  int r0, n, L;
  int nkt;                 // steps in all
  int kt;                  // first step with new rows
  int a;                   // their first key row in that step (0 unless it is shared)
  int nrt;                 // units of a kv head
  bool bad;
};

__device__ __forceinline__ Req load_req(const TreeParams& p, int b) {
  const int64_t r0 = p.cu[b], r1 = p.cu[b + 1], L = p.cache_len[b];
  Req R;
  R.bad = r0 < 0 || r1 < r0 || r1 > p.T || r1 - r0 > p.max_nodes || L < 0 ||
          L > ((int64_t)p.max_pages << p.page_shift);
  R.r0 = (int)r0;
  R.n = R.bad ? 0 : (int)(r1 - r0);
  R.L = (int)L;
  const int nct = (int)((L + kKeys - 1) / kKeys);
  const int off = (int)L & (kKeys - 1), a = (off + 7) & ~7;
  const bool share = off > 0 && a + R.n <= kKeys;
  R.a = share ? a : 0;
  R.kt = share ? nct - 1 : nct;
  R.nkt = share ? nct : nct + (R.n + kKeys - 1) / kKeys;
  R.nrt = R.n <= p.npu ? 1 : (R.n + p.npu - 1) / p.npu;
  return R;
}

// Units of a request and kv head in lane z.
__device__ __forceinline__ int lane_tiles(const TreeParams& p, const Req& R, int z) {
  return R.n && R.nrt > z ? (R.nrt - z + p.lanes - 1) / p.lanes : 0;
}

// A unit of the block: nodes rt * npu onwards of request b for kv head h, steps
// [k0, k1);
// k1 = 0 ends the list.
struct Unit {
  Req R;
  int z, b, h, rt, k0, k1;
  // key rows of step k: the products run over them, the rest of the tile is void
  __device__ __forceinline__ int keys(int k) const {
    return k < R.kt ? min(kKeys, R.L - k * kKeys) : min(kKeys, R.a + R.n - (k - R.kt) * kKeys);
  }
};
constexpr int kUnits = 4;      // units the K producer may be ahead of the last reader

// The unit behind u; left: the block's share not yet in a unit.
template <int kCost>
__device__ __forceinline__ bool next_unit(const TreeParams& p, Unit& u, int& left) {
  if (left <= 0) return false;
  u.k0 = 0;
  u.rt += p.lanes;
  if (u.rt >= u.R.nrt) {
    u.rt = u.z;
    if (++u.h == p.Hkv) {
      u.h = 0;
      do {
        if (++u.b >= p.B) {
          u.b = 0;
          u.rt = ++u.z;
          if (u.z >= p.lanes) return false;
        }
        u.R = load_req(p, u.b);
      } while (u.R.n == 0 || u.R.nrt <= u.z);
    }
  }
  u.k1 = min(u.R.nkt, left);
  left -= u.R.nkt + kCost;
  return true;
}

// Node (in its tile) of row n of a tile.
__device__ __forceinline__ int over_g(const TreeParams& p, int n) {
  return p.G == 1 ? n : (int)__umulhi((uint32_t)n, p.g_magic);
}

// The units that the K producer lays out for the other warps: number lu is
// copied, and its place given back. False: the list has ended, or a wait ran out.
struct UnitRing {
  Unit* unit;                  // [kUnits]
  uint32_t full, empty;        // their barriers
};
__device__ __forceinline__ bool take(const UnitRing& ring, int lu, Unit& u, const Bound& w) {
  const int s = lu % kUnits;
  bool ok = spin(ring.full + 8 * s, (lu / kUnits) & 1, w, 0x900);
  ok = __all_sync(0xffffffffu, ok);
  if (!ok) return false;
  u = ring.unit[s];
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(ring.empty + 8 * s);
  return u.k1 > 0;
}

// The block's share: steps (with kCost steps for a unit's own cost) f0 to f0 +
// steps of all units laid end to end; blocks [0, rem) take quo + 1, the others
// quo. s_start: the unit it begins in. Called by all threads.
struct Share {
  int f0, steps, quo, rem;
  // blocks that hold a piece of the unit that starts in this one, as its last
  __device__ __forceinline__ int pieces(const Unit& w) const {
    const int last = f0 + steps - w.k1 + w.R.nkt - 1, cut = rem * (quo + 1);
    return (last < cut ? last / (quo + 1) : rem + (last - cut) / quo) - (int)blockIdx.x + 1;
  }
};
template <int LM, int TH, int kCost>
__device__ __forceinline__ Share find_share(const TreeParams& p, uint32_t* status, Unit* s_start,
                                            int (*s_sums)[TH / 32]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = (p.B + TH - 1) / TH;
  const int rb0 = min(p.B, (int)threadIdx.x * per), rb1 = min(p.B, rb0 + per);
  int mine[LM], incl[LM];                        // the host bounds the total below 2^31
#pragma unroll
  for (int z = 0; z < LM; ++z) mine[z] = 0;
  bool bad_req = false;
  Req R;
#pragma unroll 1
  for (int b = rb0; b < rb1; ++b) {
    R = load_req(p, b);
    bad_req |= R.bad;
#pragma unroll
    for (int z = 0; z < LM; ++z) mine[z] += p.Hkv * lane_tiles(p, R, z) * (R.nkt + kCost);
  }
#pragma unroll
  for (int z = 0; z < LM; ++z) {
    incl[z] = mine[z];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl[z], o);
      if (lane >= o) incl[z] += y;
    }
    if (lane == 31) s_sums[z][warp] = incl[z];
  }
  if (threadIdx.x == 0) {
    status[0] = 0;
    status[1] = 0;
    p.meta[blockIdx.x] = make_int4(0, 0, 0, 0);
  }
  tc_fence_before();
  const bool any_bad = __syncthreads_or(bad_req);
  tc_fence_after();
  int total = 0, before[LM];                     // before: steps ahead of this warp's, lane by lane
#pragma unroll
  for (int z = 0; z < LM; ++z)
#pragma unroll
    for (int w = 0; w < TH / 32; ++w) {
      if (w == warp) before[z] = total;
      total += s_sums[z][w];
    }
  if (any_bad && blockIdx.x == 0 && threadIdx.x == 0) raise_status(status, kDevIndex, 0x40);
  // blocks [0, rem) take quo + 1 steps, the others quo
  const int quo = total / (int)gridDim.x, rem = total - quo * (int)gridDim.x;
  const int blk = (int)blockIdx.x;
  const int f0 = blk * quo + min(blk, rem), steps = quo + (blk < rem ? 1 : 0);
#pragma unroll
  for (int z = 0; z < LM; ++z) {
    int at = before[z] + incl[z] - mine[z];
    if (steps > 0 && f0 >= at && f0 < at + mine[z]) {
#pragma unroll 1
      for (int b = rb0; b < rb1; ++b) {
        if (per > 1) R = load_req(p, b);
        const int nt = lane_tiles(p, R, z), cost = R.nkt + kCost, c = p.Hkv * nt * cost;
        if (f0 >= at + c) { at += c; continue; }
        const int off = f0 - at, u = off / cost;
        Unit v;
        v.R = R;
        v.z = z;
        v.b = b;
        v.k0 = off - u * cost;              // from nkt on: the unit's steps are all done
        v.k1 = min(R.nkt, v.k0 + steps);
        v.h = nt == 1 ? u : u / nt;
        v.rt = z + (u - v.h * nt) * p.lanes;
        *s_start = v;
        break;
      }
    }
  }
  __syncthreads();
  return Share{f0, steps, quo, rem};
}

// A producer warp: of K (y false; it also lays out the block's units), or of Q
// and V. Each follows its own ring, so a K tile never waits behind a V tile.
// QT row tiles of QR rows a unit, QS units of Q in flight.
struct Producer {
  const CUtensorMap *cmap, *c8map, *nmap, *qmap;
  uint32_t ring, sq;                        // shared memory: tiles of the ring, Q
  uint32_t full, empty, qf, qe;             // barriers
  int depth;
  UnitRing units;
  const Unit* start;
};
template <int NB, int QT, int QR, int QS, int kCost>
__device__ __forceinline__ void produce(const TreeParams& p, const Producer& io, bool y, int steps,
                                        uint32_t* status, const Bound& W) {
  constexpr int kTile = NB * kKeys * 128, kBox = kKeys * 128;
  const int lane = threadIdx.x & 31;
  const int box_shift = min(p.page_shift, 7);
  // K and V pass through L2 once, unless the units of several lanes share them
  const uint64_t policy = p.lanes > 1 ? policy_normal() : policy_once();
  // a lane's copy of a step: box x of key-row group g by lane g * NB + x.
  // Groups are whole boxes of a page, or 8 rows where new rows follow.
  // The page id is asked for a step ahead of its use
  const int g = lane / NB, x = lane % NB;
  struct Copy { int page, row, h, key; bool fresh, cached, want; };
  bool ok = true;
  Unit w;
  // the K producer also lays out the block's units for the other warps
  int k = 0, lu = 0, left = steps;
  int q_done = 0;
  bool q_due = false;
  bool begun = y || steps == 0;
  w.k1 = 0;
  auto advance = [&]() -> bool {
    if (y) {
      if (!take(io.units, lu, w, W)) return false;
      q_due = true;
    } else {
      bool more;
      if (!begun) {
        begun = true;
        w = *io.start;
        left -= w.R.nkt + kCost - w.k0;
        more = w.k1 > w.k0 || next_unit<kCost>(p, w, left);
      } else {
        more = steps > 0 && next_unit<kCost>(p, w, left);
      }
      const int sl = lu % kUnits;
      if (lu >= kUnits) {
        ok = spin(io.units.empty + 8 * sl, ((lu / kUnits) - 1) & 1, W, 0x910);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return false;
      }
      if (lane == 0) {
        if (more) io.units.unit[sl] = w;
        else io.units.unit[sl].k1 = 0;
        mbar_arrive(io.units.full + 8 * sl);
      }
      __syncwarp();
      if (!more) return false;
    }
    k = w.k0;
    ++lu;
    return true;
  };
  // Q too, the rows of a tile's nodes (nodes behind the request's are rows that
  // nobody reads). After the last V copy of the unit before: Q's place may be
  // free only once that unit's scores are done
  auto load_q = [&]() -> bool {
    q_due = false;
    const int u = lu - 1, sq = u % QS;
    if (u >= QS) ok = spin(io.qe + 8 * sq, ((u / QS) - 1) & 1, W, 0x600);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) return false;
    const int node = w.rt * p.npu, tiles = QT == 1 || w.R.n - node <= p.npt ? 1 : QT;
    if (lane == 0) {
      mbar_arrive_expect_tx(io.qf + 8 * sq, (uint32_t)(tiles * NB * p.npt * p.G * 128));
      for (int x = 0; x < tiles; ++x)
        for (int e = 0; e < NB; ++e)
          tma_load_3d(io.sq + (sq * QT + x) * (NB * QR * 128) + e * QR * 128, io.qmap, io.qf + 8 * sq,
                      e * 64, w.h * p.G, w.R.r0 + node + x * p.npt);
    }
    __syncwarp();
    q_done = lu;
    return true;
  };
  auto fetch = [&](Copy& c) -> bool {
    if (k >= w.k1 && !advance()) return false;
    c.fresh = k >= w.R.kt;
    c.h = w.h;
    c.key = g << (c.fresh ? 3 : box_shift);
    c.cached = !c.fresh || c.key < w.R.a;
    c.want = c.key < w.keys(k);
    c.page = 0;
    c.row = w.R.r0 + (k - w.R.kt) * kKeys + c.key - w.R.a;
    if (c.want && c.cached) {
      const int at = k * kKeys + c.key;
      c.page = p.table[(int64_t)w.b * p.table_stride + (at >> p.page_shift)];
      c.row = at & ((1 << p.page_shift) - 1);
    }
    ++k;
    return true;
  };
  // one copy is made while the next one's page id is on its way; the first
  // round only asks
  Copy cur, nxt;
  cur.h = -1;
  int t = 0, issued = 0;
  for (bool more = true; more;) {
    more = fetch(nxt);
    if (cur.h < 0) {
      cur = nxt;
      if (q_due && more && !load_q()) break;
      continue;
    }
    if (cur.cached && cur.want && (cur.page < 0 || cur.page >= p.n_pages)) {
      cur.want = false;
      raise_status(status, kDevIndex, 0x41);
    }
    const uint32_t each = 128u << (cur.fresh ? 3 : box_shift);
    const uint32_t bytes = each * __popc(__ballot_sync(0xffffffffu, cur.want));
    const int sl = t % io.depth;
    if (t >= io.depth) {
      ok = spin(io.empty + 8 * sl, ((t / io.depth) - 1) & 1, W, 0x100 + y);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
    }
    if (lane == 0) mbar_arrive_expect_tx(io.full + 8 * sl, bytes);
    __syncwarp();
    if (cur.want) {
      const uint32_t d = io.ring + sl * kTile + (uint32_t)(x * kBox + cur.key * 128);
      if (cur.cached)
        tma_load_4d(d, cur.fresh ? io.c8map : io.cmap, io.full + 8 * sl, x * 64, cur.h, cur.row, cur.page, policy);
      else tma_load_3d(d, io.nmap, io.full + 8 * sl, x * 64, cur.h, cur.row);
    }
    issued = ++t;
    cur = nxt;
    if (q_due && more && !load_q()) break;
  }
  __syncwarp();
  // drain: every copy has landed before the block exits
  for (int i = max(0, issued - io.depth); i < issued; ++i)
    wait_drain(io.full + 8 * (i % io.depth), (i / io.depth) & 1);
  if (y)
    for (int i = max(0, q_done - QS); i < q_done; ++i) wait_drain(io.qf + 8 * (i % QS), (i / QS) & 1);
}

// Key row r of a V tile (at address row) before its product: a new row (keep)
// loses its NaN and infinite elements, which marks it in nf_bits as row j (the
// epilogue adds them to the rows that see it); any other is zeroed. look: the
// row is read first, and mostly left as it is.
template <int NB>
__device__ __forceinline__ void clean_row(uint32_t row, int r, bool keep, bool look, uint32_t* nf_bits, int j) {
  // any order of the row's 16-byte chunks: lanes spread over the banks
  auto chunk = [&](int c) { return row + (c >> 3) * kKeys * 128 + (((c + r) & 7) << 4); };
  uint32_t top = 0x7f807f80u;                            // the largest exponents, by half
  if (look) {
    top = 0;
#pragma unroll
    for (int c = 0; c < 8 * NB; ++c) {
      uint32_t x[4];
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(chunk(c)) : "memory");
#pragma unroll
      for (int e = 0; e < 4; ++e) top = __vmaxu2(top, x[e] & 0x7f807f80u);
    }
  }
  if ((top & 0x7f80u) == 0x7f80u || (top >> 16) == 0x7f80u) {
    if (keep) atomicOr(nf_bits + (j >> 5), 1u << (j & 31));
#pragma unroll 1
    for (int c = 0; c < 8 * NB; ++c) {
      uint32_t x[4] = {0, 0, 0, 0};
      if (keep) {
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(chunk(c)) : "memory");
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if ((x[e] & 0x7f80u) == 0x7f80u) x[e] &= 0xffff0000u;
          if ((x[e] & 0x7f800000u) == 0x7f800000u) x[e] &= 0x0000ffffu;
        }
      }
      st_shared_v4(chunk(c), x[0], x[1], x[2], x[3]);
    }
  }
}

}  // namespace tree
}  // namespace mis
