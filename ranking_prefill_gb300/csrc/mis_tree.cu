// Attention of drafted token trees over a paged K/V cache, sm_103a.
//
// Row i of request b sees the cached rows [0, L_b) and, among the request's
// own new rows, its ancestors and itself:
//     o_i = sum_j p_ij v_j,  p_ij = exp(s_ij - lse_i),  s_ij = scale q_i k_j.
//
// The n_b * G rows of a request that share a kv head (G query heads each) are
// few, the keys many, so the tensor-core products are taken with the keys on
// the wide side:
//     S^T [128 keys x N rows] = K Q^T        (A = K tile, B = Q rows)
//     O^T [D x N rows]       += V^T P^T      (A = V tile, MN-major, B = P)
// with N = 16, 32 or 64 rows a tile: a decoded token costs N = 16 columns of
// softmax instead of 128 rows, and one pass over K and V serves every row of
// the tile. Requests with more rows go to mis_tree_wide.cu.
//
// A tile holds the G rows of N / G nodes (rounded down), so one TMA box loads
// its Q. Work is cut evenly: the (request, kv head) units are laid end to
// end in 128-key steps and every block takes the same number of consecutive
// steps, found on the device from the lengths (no host plan). A block that
// holds a whole unit writes O; the pieces of a unit that several blocks share
// leave (max, sum, unnormalised O) in the workspace and a second kernel adds
// them in block order, so the same call gives the same bits.
//
// Warp roles: 0 and 3 TMA producers of K and of Q and V (pages of the cache,
// 8-row groups of the new rows), 1 MMA issue, 2 the tree's masks, then one or
// two softmax warpgroups (a thread is a key, it owns N or N / 2 columns) and
// an epilogue warpgroup (a thread is an element of the head).
//
// Any reference serves a column's softmax as long as its scores stay within
// the exponent's reach of it. One reference for all columns of a warpgroup
// stays in a register: it is the largest maximum, taken when the columns'
// maxima so far lie within 2^40 of each other (else every column has its own,
// read from shared memory, at most 2^40 above its maximum). It is moved only
// when a score passes it by 2^8: one vote per step replaces the exchange of
// maxima, and O in tensor memory is rescaled only then. References are scores
// before the scale (times its sign). scale * score - scale * reference in one
// multiply-add is off by the rounding of scale * reference, so a reference that
// is far from zero is taken off first, exactly where the score equals it.
//
// What bounds it: the stream of K and V. 64 decoded tokens over 512 to 4096 rows
// (16 / 8 heads, D = 128, 562 MB): 94 to 96 us, 5.9 TB/s of 6.7 measured for a
// copy; 4 requests of 64K to 128K rows with 1 to 8 nodes x 4 heads (1.9 GB): 278
// to 286 us, 6.7 TB/s. Short ones are bound by the way there: launch and schedule 2 us,
// the first copies 3.5, the second kernel 2; 8 trees of 8 to 32 nodes over 512 to
// 4096 rows (79 MB): 26 us. K and V are marked to leave L2 first, which keeps
// the pieces, the tables and the code in it: 1 us of those 26 and 94.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "mis_internal.h"
#include "mis_ptx.cuh"
#include "mis_tree.cuh"

namespace mis {

CUtensorMap encode_tmap_bf16(const void* base, int rank, const uint64_t* dims,
                             const uint64_t* strides_bytes, const uint32_t* box, bool* ok);

namespace tree {
mis_status_t launch_wide(int D, const CUtensorMap* m, const TreeParams& p, int blocks, cudaStream_t st);
}

namespace {

using namespace dev;
using namespace tree;

constexpr float kSpread = 40.0f;                 // log2 units maxima may differ by under one reference

template <int D, int N>
struct TreeCfg {
  static constexpr int kNB = D / 64;             // 64-column boxes of a row
  static constexpr int kWG = N == 16 ? 1 : 2;    // softmax warpgroups
  static constexpr int kNC = N / kWG;            // columns of a softmax thread
  static constexpr int kThreads = 256 + 128 * kWG;
  // Register budgets of the warpgroups (N = 64): their sum is the launch's,
  // 512 threads x 128
  static constexpr int kRegCtl = 80, kRegEpi = 80, kRegSoft = 176;
  static_assert(N < 64 || 128 * (kRegCtl + kRegEpi + kWG * kRegSoft) <= kThreads * 128,
                "register split exceeds the launch allocation");
  static constexpr int kBox = kKeys * 128;       // 64 columns of a 128-key tile
  static constexpr int kTile = kNB * kBox;
  static constexpr int kQ = N * D * 2;
  static constexpr int kQBox = N * 128;
  static constexpr int kQS = 2;
  static constexpr int kP = kKeys * 128;
  static constexpr int kK = D == 128 ? 3 : 5;
  static constexpr int kV = D == 128 ? (N == 16 ? 3 : 2) : 5;
  static constexpr int kNW = N < 32 ? 1 : N / 32;       // mask words of a key: which columns see it
  static constexpr int kNodes = 64;              // N >= max_nodes * G
  static constexpr int kFew = D == 128 && N > 16 ? 8 : 16;     // new rows that the masks' warp reads itself
  // What a unit costs besides its steps (its first step, masks, epilogue), in
  // steps: blocks are given equal shares of both. N = 64, with 1, 2 and 3: 8 trees
  // of 17 to 32 nodes 24.7, 23.6, 24.9 us, 32 of them over 100 to 600 rows 34.6,
  // 33.0, 32.7. N = 16 and 32, with 0, 1 and 2: 4 decoded tokens 10.5, 11.0, 10.9;
  // 5 small trees 11.0, 11.4, 11.3; 64 decoded tokens 103.6, 102.8, 101.9. So none
  // for the small batches; 256 tokens over 100 to 600 rows (130, 118, 115) and 32
  // trees of 9 to 16 nodes over as many (33.5, 26.9, 25.4) would rather have 2
  static constexpr int kUnitCost = N == 64 ? 2 : 0;
  static constexpr int kTmem = N == 16 ? 64 : 4 * N;    // S_0 | S_1 | O_0 | O_1
  // floats / words behind the tiles
  static constexpr int oMask = 0;                       // [2][kNodes][kNW]
  static constexpr int oDead = oMask + 2 * kNodes * kNW;   // [2][kNW] unused rows of the tile
  static constexpr int kJW = kNodes / 32;               // words of a unit's new keys
  static constexpr int oNf = oDead + 2 * kNW;           // [2][kJW] those with a non-finite value
  static constexpr int oM = oNf + 2 * kJW;                  // [2][N] references, negated, for the epilogue
  static constexpr int oL = oM + 2 * N;                 // [2][4][N] sums of each softmax warp
  static constexpr int oMax = oL + 8 * N;               // [4][N] maxima of a step by warp
  static constexpr int oRef = oMax + 4 * N;             // [4][N] a warp's copy of the negated references
  static constexpr int oAl = oRef + 4 * N;              // [4][N] ... of the factors of a move
  static constexpr int oInv = oAl + 4 * N;              // [4][N] an epilogue warp's 1 / sum
  static constexpr int oPar = oInv + 4 * N;             // [kNodes] int16: parents
  static constexpr int kWords = oPar + kNodes / 2;
  static constexpr int kData = kQS * kQ + kP + (kK + kV) * kTile;
  static constexpr int kSmem = kData + 4 * kWords + 512 + 1024;
  static_assert(kSmem <= 232448, "shared memory");
};

__device__ __forceinline__ float warp_max(float x) {       // NaN only if all are
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float warp_min(float x) {
  float r;
  asm volatile("redux.sync.min.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// Sums (or maxima) over the warp of NV columns, of which every lane brings one
// value each, NV <= 32: halve the columns lane bit by lane bit, then fold the
// lanes that are left. Returns the column that ends up in v[0] of this lane.
// (One redux a column took three times as long.)
template <int NV, bool kMax>
__device__ __forceinline__ int fold_cols(float* v, int lane) {
  int cnt = NV, col = 0;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    if (cnt > 1) {
      const int hf = cnt / 2;
      const bool up = (lane & o) != 0;
#pragma unroll
      for (int n = 0; n < NV / 2; ++n) {
        if (n >= hf) break;
        const float give = up ? v[n] : v[n + hf], keep = up ? v[n + hf] : v[n];
        const float got = __shfl_xor_sync(0xffffffffu, give, o);
        v[n] = kMax ? fmaxf(keep, got) : keep + got;
      }
      col += up ? hf : 0;
      cnt = hf;
    } else {
      const float got = __shfl_xor_sync(0xffffffffu, v[0], o);
      v[0] = kMax ? fmaxf(v[0], got) : v[0] + got;
    }
  }
  return col;
}

template <int NC>
__device__ __forceinline__ void ld_cols(uint32_t taddr, uint32_t* r) {
  if constexpr (NC == 8) {
    tmem_ld8(taddr, r);
    tmem_ld_wait();
    reg_fence8(r);
  } else if constexpr (NC == 16) {
    tmem_ld16(taddr, r);
    tmem_ld_wait();
    reg_fence16(r);
  } else {
#pragma unroll
    for (int c = 0; c < NC; c += 32) tmem_ld32(taddr + c, r + c);
    tmem_ld_wait();
#pragma unroll
    for (int c = 0; c < NC; c += 32) reg_fence32(r + c);
  }
}

template <int D, int N>
__global__ void __launch_bounds__(TreeCfg<D, N>::kThreads, 1)
mis_tree_attn_kernel(const __grid_constant__ CUtensorMap qmap,
                     const __grid_constant__ CUtensorMap kcmap,
                     const __grid_constant__ CUtensorMap vcmap,
                     const __grid_constant__ CUtensorMap kc8map,
                     const __grid_constant__ CUtensorMap vc8map,
                     const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const TreeParams p) {
  using C = TreeCfg<D, N>;
  constexpr int NB = C::kNB, NC = C::kNC, WG = C::kWG, KS = C::kK, VS = C::kV, QS = C::kQS;
  constexpr int NW = C::kNW, JW = C::kJW;
  // barriers
  constexpr int bQF = 0, bQE = bQF + 2, bKF = bQE + 2, bKE = bKF + KS, bVF = bKE + KS,
                bVE = bVF + VS, bSF = bVE + VS, bPF = bSF + 2, bPV = bPF + 1, bOF = bPV + 1,
                bOE = bOF + 2, bST = bOE + 2, bSE = bST + 2, bMF = bSE + 2, bUF = bMF + 2,
                bUE = bUF + kUnits, bDR = bUE + kUnits, nBar = bDR + 1;
  static_assert(nBar * 8 + 64 <= 512, "barrier space");

  griddep_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* sQ = smem;
  uint8_t* sP = sQ + QS * C::kQ;
  uint8_t* sK = sP + C::kP;
  uint8_t* sV = sK + KS * C::kTile;
  uint32_t* words = reinterpret_cast<uint32_t*>(smem + C::kData);
  uint32_t* sMask = words + C::oMask;
  uint32_t* sDead = words + C::oDead;
  uint32_t* sNf = words + C::oNf;
  float* sM = reinterpret_cast<float*>(words + C::oM);
  float* sL = reinterpret_cast<float*>(words + C::oL);
  float* sMax = reinterpret_cast<float*>(words + C::oMax);
  float* sRef = reinterpret_cast<float*>(words + C::oRef);
  float* sAl = reinterpret_cast<float*>(words + C::oAl);
  float* sInv = reinterpret_cast<float*>(words + C::oInv);
  int16_t* sPar = reinterpret_cast<int16_t*>(words + C::oPar);
  uint64_t* bars = reinterpret_cast<uint64_t*>(words + C::kWords);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + nBar);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  __shared__ Unit s_start, s_unit[kUnits];
  __shared__ int s_sums[1][C::kThreads / 32];
  auto bar = [&](int i) { return smem_u32(bars + i); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(bQF + s), 1);
      mbar_init(bar(bQE + s), 1);
      mbar_init(bar(bSF + s), 1);
      mbar_init(bar(bOF + s), 1);
      mbar_init(bar(bOE + s), 4);
      mbar_init(bar(bST + s), 4 * WG);
      mbar_init(bar(bSE + s), 4);
      mbar_init(bar(bMF + s), 1);
    }
    for (int s = 0; s < KS; ++s) { mbar_init(bar(bKF + s), 1); mbar_init(bar(bKE + s), 1); }
    for (int s = 0; s < VS; ++s) { mbar_init(bar(bVF + s), 1); mbar_init(bar(bVE + s), 1); }
    mbar_init(bar(bPF), 4 * WG);
    mbar_init(bar(bPV), 1);
    mbar_init(bar(bDR), 1);
    for (int s = 0; s < kUnits; ++s) {
      mbar_init(bar(bUF + s), 1);
      mbar_init(bar(bUE + s), 7 + 4 * WG);               // every warp but the K producer
    }
    fence_mbar_init();
    fence_proxy_async();
    tma_prefetch_desc(&qmap); tma_prefetch_desc(&kcmap); tma_prefetch_desc(&vcmap);
    tma_prefetch_desc(&kc8map); tma_prefetch_desc(&vc8map);
    tma_prefetch_desc(&kmap); tma_prefetch_desc(&vmap);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), C::kTmem);
    tmem_relinquish();
  }
  griddep_wait();

  // ------------------------------------------------ this block's share of the steps
  uint32_t* status = p.cta_status + 2 * blockIdx.x;
  const Share share = find_share<1, C::kThreads, C::kUnitCost>(p, status, &s_start, s_sums);
  const uint32_t tmem = *tmem_slot;
  const Bound W{abort_flag, p.wait_ns};
  auto colS = [](int s) { return (uint32_t)(s * N); };
  auto colO = [](int s) { return (uint32_t)((2 + s) * N); };

  const UnitRing units_ring{s_unit, bar(bUF), bar(bUE)};
  auto take = [&](int lu, Unit& u) -> bool { return tree::take(units_ring, lu, u, W); };

  if (warp < 4) {
    if constexpr (N >= 64) regs_dec<C::kRegCtl>();
    if (warp == 0 || warp == 3) {
      const bool y = warp == 3;
      const Producer io{y ? &vcmap : &kcmap, y ? &vc8map : &kc8map, y ? &vmap : &kmap, &qmap,
                        smem_u32(y ? sV : sK), smem_u32(sQ), bar(y ? bVF : bKF), bar(y ? bVE : bKE),
                        bar(bQF), bar(bQE), y ? VS : KS, units_ring, &s_start};
      produce<NB, 1, N, QS, C::kUnitCost>(p, io, y, share.steps, status, W);
    } else if (warp == 1) {
      // --------------------------------------------------------------- MMA
      // the warp walks together and one elected lane issues, so loop state and
      // descriptors stay in uniform registers. This warp's own instructions are
      // the longest chain of a short step: slots and phases are counted along
      // instead of divided out, and no clock is read while it looks around
      constexpr uint32_t idS = idesc_bf16(128, N, false);
      constexpr uint32_t idO = idesc_bf16(128, N, true) | (1u << 15);   // A MN-major too
      bool ok = true;
      auto wait_all = [&](int b, uint32_t parity, uint32_t where) -> bool {
        const bool r = spin(bar(b), parity, W, where);
        return __all_sync(0xffffffffu, r);
      };
      if (p.stall) ok = wait_all(bDR, 0, 0x7ff);               // nothing arrives before the drain
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      // the next step with its S outstanding (nxt), the step whose S runs or
      // has run and whose P is awaited (cur), the one behind it (aft). One loop
      // looks for whatever can go next, each product at one place in the code
      struct Ring { int slot; uint32_t ph; };
      auto turn = [](Ring& r, int depth) { if (++r.slot == depth) { r.slot = 0; r.ph ^= 1; } };
      struct Step { int kv; bool first, last; } cur{0, false, false}, aft{0, false, false}, nxt;
      Ring rk{0, 0}, rv{0, 0}, rq{0, 0}, rs{0, 0}, ro{1, 1};
      Unit w;
      int k = 0, k1 = 0, lu = 0, running = 0;            // running: S products without their PV
      uint32_t pf = 0, units = 0, idle = 0;
      bool have = false, more = ok;
      uint64_t t0 = 0;
      while (true) {
        if (!have && more) {
          const bool first = k >= k1;
          if (first) {
            more = take(lu++, w);
            k = __shfl_sync(0xffffffffu, w.k0, 0);
            k1 = __shfl_sync(0xffffffffu, w.k1, 0);
          }
          if (more) {
            nxt.kv = __shfl_sync(0xffffffffu, w.keys(k), 0);
            nxt.first = first;
            nxt.last = ++k == k1;
            have = true;
          }
        }
        if (!have && running == 0) break;
        bool s_go = have && running < 2 && mbar_test_wait(bar(bKF + rk.slot), rk.ph) &&
                    (!nxt.first || mbar_test_wait(bar(bQF + rq.slot), rq.ph));
        bool p_go = running > 0 && mbar_test_wait(bar(bPF), pf) &&
                    mbar_test_wait(bar(bVF + rv.slot), rv.ph) &&
                    // O's buffer: the unit before the last must have been read out
                    (!cur.first || units < 2 || mbar_test_wait(bar(bOE + (ro.slot ^ 1)), ro.ph ^ (ro.slot ^ 1)));
        s_go = __all_sync(0xffffffffu, s_go);
        p_go = __all_sync(0xffffffffu, p_go);
        if (s_go) {
          // S of the next step, during the softmax of the one before
          tc_fence_after();
          const uint32_t d = tm + colS(rs.slot);
          const uint64_t a = sdesc_sw128(smem_u32(sK) + rk.slot * C::kTile, 16, 1024);
          const uint64_t b = sdesc_sw128(smem_u32(sQ) + rq.slot * C::kQ, 16, 1024);
          if (elect_uniform()) {
#pragma unroll
            for (int x = 0; x < NB; ++x)
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                mma_ss(d, a + ((x * C::kBox + ks * 32) >> 4), b + ((x * C::kQBox + ks * 32) >> 4), idS,
                       (x | ks) != 0);
            mma_commit(bar(bSF + rs.slot));
            mma_commit(bar(bKE + rk.slot));
            if (nxt.last) mma_commit(bar(bQE + rq.slot));
          }
          __syncwarp();
          turn(rk, KS);
          turn(rs, 2);
          if (nxt.last) turn(rq, QS);
          (running ? aft : cur) = nxt;
          ++running;
          have = false;
          idle = 0;
        } else if (p_go) {
          if (cur.first) {
            turn(ro, 2);
            ++units;
          }
          tc_fence_after();
          // V [key][d] and P [key][row], both MN-major: 8-key groups 1024 B
          // apart, 64-column boxes kBox apart. D = 64 repeats its one box
          // (stride 0): rows 64..127 of O^T equal rows 0..63.
          const uint32_t d = tm + colO(ro.slot), acc = cur.first ? 0u : 1u;
          const uint64_t a = sdesc_sw128(smem_u32(sV) + rv.slot * C::kTile, D == 128 ? C::kBox : 0, 1024);
          const uint64_t b = sdesc_sw128(smem_u32(sP), C::kBox, 1024);
          const int nks = (cur.kv + 15) >> 4;
          if (elect_uniform()) {
            mma_ss(d, a, b, idO, acc);
            if (nks == kKeys / 16) {
#pragma unroll
              for (int ks = 1; ks < kKeys / 16; ++ks) mma_ss(d, a + ks * 128, b + ks * 128, idO, 1u);
            } else {
#pragma unroll 1
              for (int ks = 1; ks < nks; ++ks) mma_ss(d, a + ks * 128, b + ks * 128, idO, 1u);
            }
            mma_commit(bar(bVE + rv.slot));
            mma_commit(bar(bPV));
            if (cur.last) mma_commit(bar(bOF + ro.slot));
          }
          __syncwarp();
          turn(rv, VS);
          pf ^= 1;
          cur = aft;
          --running;
          idle = 0;
        } else {
          // bounded: the clock is read every 64 fruitless rounds
          if ((++idle & 63) == 0) {
            const uint64_t now = globaltimer();
            if (idle == 64) t0 = now;
            if (__any_sync(0xffffffffu, *abort_flag != 0)) break;
            if (__any_sync(0xffffffffu, now - t0 > p.wait_ns && idle > 64)) {
              if (lane == 0) *abort_flag = 0x400;
              break;
            }
          }
        }
      }
      // drain: all tensor-core work of the elected lane completes before dealloc
      if (elect_uniform()) mma_commit(bar(bDR));
      __syncwarp();
      wait_drain(bar(bDR), 0);
    } else {
      // ------------------------------------------------------ the tree's masks
      int lu = 0;
      bool ok = true, bad = false;
      Unit w;
      while (ok && take(lu, w)) {
        const int node0 = w.rt * p.npt, rows = min(p.npt, w.R.n - node0) * p.G;
        const int sm = lu & 1;
        if (lu >= 2) ok = spin(bar(bSE + sm), ((lu >> 1) - 1) & 1, W, 0x610);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        // parents as the masks use them: the index, or -1 for roots, for
        // children of unused nodes, and for what is no index; unused nodes
        // themselves -2
        const bool tree = w.k1 > w.R.kt;
        int16_t* par = sPar;
        if (p.parents) {
          int raw[C::kNodes / 32];
#pragma unroll
          for (int x = 0; x < C::kNodes / 32; ++x) {
            const int j = x * 32 + lane;
            raw[x] = j < w.R.n ? p.parents[w.R.r0 + j] : MIS_TREE_ROOT;
          }
#pragma unroll
          for (int x = 0; x < C::kNodes / 32; ++x) {
            const int j = x * 32 + lane;
            if (raw[x] >= j || raw[x] < MIS_TREE_UNUSED) {
              bad |= j < w.R.n;
              raw[x] = MIS_TREE_ROOT;
            }
            par[j] = (int16_t)raw[x];
          }
          __syncwarp();
#pragma unroll
          for (int x = 0; x < C::kNodes / 32; ++x)
            if (raw[x] >= 0 && par[raw[x]] == MIS_TREE_UNUSED) par[x * 32 + lane] = MIS_TREE_ROOT;
          __syncwarp();
        }
        // columns of unused nodes
        if (lane < JW) sNf[sm * JW + lane] = 0;
#pragma unroll 1
        for (int c0 = 0; c0 < N; c0 += 32) {
          const int n = c0 + lane;
          const bool dead = n < rows && p.parents && par[node0 + over_g(p, n)] == MIS_TREE_UNUSED;
          const uint32_t dw = __ballot_sync(0xffffffffu, dead);
          if (lane == 0) sDead[sm * NW + (c0 >> 5)] = dw;
        }
        if (tree) {
          // who sees new key j: a bit a column
          uint32_t* m = sMask + sm * C::kNodes * NW;
          if (!p.parents) {
            for (int x = lane; x < w.R.n * NW; x += 32) {
              const int j = x / NW, c0 = x % NW * 32;
              m[x] = bit_range((j - node0) * p.G - c0, rows - c0);
            }
          } else {
            for (int x = lane; x < w.R.n * NW; x += 32) m[x] = 0;
            __syncwarp();
            for (int i = lane; i * p.G < rows; i += 32) {
              const int lo = i * p.G, hi = lo + p.G;
              if (par[node0 + i] == MIS_TREE_UNUSED) continue;
              for (int j = node0 + i; j >= 0; j = par[j])
                for (int x = lo >> 5; x <= (hi - 1) >> 5; ++x)
                  atomicOr(&m[j * NW + x], bit_range(lo - 32 * x, hi - 32 * x));
            }
          }
          // New rows whose V holds a NaN or an infinity (see the softmax): a few
          // are read from memory here, one trip that is over before their tile is
          // there (one decoded row from its tile: 0.8 us more); of more, the
          // softmax looks over the tile
          constexpr int LPR = D / 8, RPI = 32 / LPR;         // lanes a row, rows a load
          __syncwarp();
          if (w.R.n <= C::kFew) {
            const __nv_bfloat16* src = p.v + (int64_t)w.R.r0 * p.vs + w.h * D + lane % LPR * 8;
            uint4 u[C::kFew / RPI];
#pragma unroll
            for (int e = 0; e < C::kFew / RPI; ++e)
              u[e] = *reinterpret_cast<const uint4*>(src + (int64_t)min(e * RPI + lane / LPR, w.R.n - 1) * p.vs);
#pragma unroll
            for (int e = 0; e < C::kFew / RPI; ++e) {
              uint32_t top = __vmaxu2(__vmaxu2(u[e].x & 0x7f807f80u, u[e].y & 0x7f807f80u),
                                      __vmaxu2(u[e].z & 0x7f807f80u, u[e].w & 0x7f807f80u));
              if ((top & 0x7f80u) == 0x7f80u || (top >> 16) == 0x7f80u)
                atomicOr(&sNf[sm * JW], 1u << min(e * RPI + lane / LPR, w.R.n - 1));
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(bMF + sm));
        ++lu;
      }
      __syncwarp();
      if (bad) raise_status(status, kDevIndex, 0x42);
    }
  } else if (warp < 4 + 4 * WG) {
    // --------------------------------------------------------------- softmax
    if constexpr (N >= 64) regs_inc<C::kRegSoft>();
    const int wg = (warp - 4) >> 2, sw = warp & 3, r = sw * 32 + lane;
    const int c0 = wg * NC, id = 1 + wg;
    const uint32_t tl = tmem + ((uint32_t)(sw * 32) << 16);
    // scores are taken times the scale's sign, then scaled by its size: the
    // largest score is the largest product
    const float sa = fabsf(p.scale_log2), sign = p.scale_log2 < 0.f ? -1.f : 1.f;
    const uint64_t sax2 = f2_pack(__float_as_uint(sa), __float_as_uint(sa));
    // this thread's row of P: chunk c of its columns
    const uint32_t aP = smem_u32(sP) + r * 128;
    const int cP = c0 / 8;
    float* ref = sRef + sw * N + c0;                     // negated references, if not one for all
    float* al = sAl + sw * N + c0;
    Unit w;
    int t = 0, lu = 0;
    bool ok = true, gone = false;
    while (!gone) {
      // Every look at the list is followed by one vote of the warpgroup: here
      // by a warp that leaves, at the unit's first step by one that goes on
      if (!take(lu, w)) {
        bar_any128(id, *abort_flag != 0);
        break;
      }
      // live: columns of this warpgroup that are rows of the unit. The others hold
      // what Q's place held, other requests' rows mostly: nobody reads them, and
      // their scores, whatever they are, move no reference
      const int slot = lu & 1, rows = min(p.npt, w.R.n - w.rt * p.npt) * p.G, live = rows - c0;
      uint64_t l2[NC / 2];
#pragma unroll
      for (int n = 0; n < NC / 2; ++n) l2[n] = 0ull;
      bool one = true;                                   // one reference, -base / sa, for all columns
                                                         // (else their scores are shifted, base 0)
      float base = 0.f;
      // the largest score of column min(lane, NC - 1) in the steps that moved a
      // reference: how far that column lies below a reference all columns share
      float own = kEmpty;
      if (ok && lu >= 2) {
        ok = spin(bar(bSE + slot), ((lu >> 1) - 1) & 1, W, 0x700);
        ok = __all_sync(0xffffffffu, ok);
      }
      // the page under this thread's key row, asked for a step ahead (0 where
      // there is no cached row)
      const int32_t* row = p.table + (int64_t)w.b * p.table_stride;
      auto page_of = [&](int k) {
        const int at = k * kKeys + r;
        return k < w.k1 && at < w.R.L ? row[at >> p.page_shift] : 0;
      };
      int page = page_of(w.k0);
#pragma unroll 1
      for (int k = w.k0; k < w.k1; ++k, ++t) {
        const int kv = w.keys(k), kv16 = (kv + 15) & ~15;
        const bool first = k == w.k0, fresh = k >= w.R.kt;
        const bool active = sw * 32 < kv16;              // this warp holds keys of the product
        // what this thread's key row holds: a cached row, new row j, or nothing
        const int j = fresh ? (k - w.R.kt) * kKeys + r - w.R.a : -1;
        const bool node = fresh && j >= 0 && r < kv;
        const bool seen = node || (r < kv && k * kKeys + r < w.R.L && page >= 0 && page < p.n_pages);
        page = page_of(k + 1);
        if (ok) {
          ok = spin(bar(bSF + (t & 1)), (t >> 1) & 1, W, 0x710);
          if (ok && fresh) ok = spin(bar(bMF + slot), (lu >> 1) & 1, W, 0x720);
          ok = __all_sync(0xffffffffu, ok);
        }
        tc_fence_after();
        const uint32_t tS = tl + colS(t & 1) + c0;
        const uint32_t* mk = sMask + (slot * C::kNodes + (node ? j : 0)) * NW;
        const bool plain = __all_sync(0xffffffffu, seen && !node);
        // Steps that are not plain (new rows, a partial tile, a negative scale,
        // references by column) have their scores rewritten in tensor memory
        // first: hidden ones -inf, the others times the scale's sign; and under
        // references by column once more, less those, when they have been moved.
        // What is left is then the same short code for every step; unrolled for
        // each kind, the kernel waited for instruction fetches more than for
        // anything else.
        bool over = !ok || first;
        if (ok && active && !(plain && one && sign > 0.f)) {
#pragma unroll 1
          for (int q = 0; q < NC; q += 16) {
            const int c = c0 + q;
            const uint32_t bits = node ? mk[c >> 5] >> (c & 31) : seen ? bit_range(0, live - q) : 0u;
            __syncwarp();
            uint32_t x[16];
            ld_cols<16>(tS + q, x);
#pragma unroll
            for (int n = 0; n < 16; ++n)
              x[n] = (bits >> n) & 1u ? __float_as_uint(__uint_as_float(x[n]) * sign) : 0xff800000u;
            if (!one) {
              // passes, too, in a column that saw nothing so far (kEmpty)
#pragma unroll
              for (int n = 0; n < 16; ++n) over |= (__uint_as_float(x[n]) + ref[q + n]) * sa > kGrow;
            }
            tmem_st16(tS + q, x);
          }
          tmem_st_wait();
        }
        __syncwarp();
        uint32_t s[NC];
        if (ok && active) ld_cols<NC>(tS, s);
        bool move = first;
        if (!first) {
          if (ok && active && one) {
            float x0 = -INFINITY, x1 = -INFINITY;
            auto fold8 = [&](int c) {
#pragma unroll
              for (int n = c; n < c + 8; n += 4) {
                x0 = max3(x0, __uint_as_float(s[n]), __uint_as_float(s[n + 1]));
                x1 = max3(x1, __uint_as_float(s[n + 2]), __uint_as_float(s[n + 3]));
              }
            };
            if (live >= NC) {
#pragma unroll
              for (int c = 0; c < NC; c += 8) fold8(c);
            } else {
#pragma unroll
              for (int c = 0; c < NC; c += 8) {
                if (c + 8 <= live) {
                  fold8(c);
                } else if (c < live) {
#pragma unroll
                  for (int n = c; n < c + 8; ++n) x0 = fmaxf(x0, n < live ? __uint_as_float(s[n]) : -INFINITY);
                }
              }
            }
            over |= fmaf(fmaxf(x0, x1), sa, base) > kGrow;
          }
          move = bar_any128(id, over);
        }
        if (move) {
          // a unit begins or a score passed its reference (or a wait gave up:
          // then every warp of the warpgroup leaves here)
          if (bar_any128(id, !ok)) { gone = true; break; }
          // the step's maximum of every column over this warp's keys
          {
            float v[NC];
#pragma unroll
            for (int n = 0; n < NC; ++n) v[n] = active && n < live ? __uint_as_float(s[n]) : -INFINITY;
            const int n = fold_cols<NC, true>(v, lane);
            sMax[sw * N + c0 + n] = v[0];
          }
          bar_sync128(id);
          // every warp draws the same conclusion from the four warps' maxima,
          // a lane for a column
          const int n = min(lane, NC - 1);
          const float old = first ? kEmpty : -ref[n];
#pragma unroll
          for (int q = 0; q < 4; ++q) own = fmaxf(own, sMax[q * N + c0 + n]);
          const float hi = warp_max(own);
          const float lo = warp_min(n < live ? own : INFINITY);
          one = lo == INFINITY || (hi > kEmpty && (hi - lo) * sa <= kSpread && fabsf(hi) * sa <= kFar);
          base = one && hi > kEmpty ? -hi * sa : 0.f;
          // a column that leaves the shared reference keeps it until its own
          // scores pass it: references never go down
          const float to = one ? hi : fmaxf(old, own);
          __syncwarp();
          if (lane < NC) {
            ref[lane] = -to;
            al[lane] = ex2((old - to) * sa);
          }
          __syncwarp();
          if (!first) {
            ok = spin(bar(bPV), (t - 1) & 1, W, 0x730);    // O holds every step before
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
            if (ok) {
              const uint32_t tO = tl + colO(slot) + c0;
#pragma unroll 1
              for (int q = 0; q < NC; q += 16) {
                uint32_t ov[16];
                ld_cols<16>(tO + q, ov);
#pragma unroll
                for (int n = 0; n < 16; ++n) ov[n] = __float_as_uint(__uint_as_float(ov[n]) * al[q + n]);
                tmem_st16(tO + q, ov);
              }
              tmem_st_wait();
#pragma unroll
              for (int n = 0; n < NC; n += 2) {
                const float2 a = *reinterpret_cast<const float2*>(al + n);
                l2[n / 2] = f2_fma(l2[n / 2], f2_pack(__float_as_uint(a.x), __float_as_uint(a.y)), 0ull);
              }
            }
          }
        }
        if (!one && ok && active) {
#pragma unroll 1
          for (int q = 0; q < NC; q += 8) {
            uint32_t x[8];
            ld_cols<8>(tS + q, x);
#pragma unroll
            for (int n = 0; n < 8; ++n) x[n] = __float_as_uint(__uint_as_float(x[n]) + ref[q + n]);
            tmem_st8(tS + q, x);
          }
          tmem_st_wait();
          __syncwarp();
        }
        if ((move || !one) && ok && active) ld_cols<NC>(tS, s);
        if (ok && active) {
          const uint64_t basex2 = f2_pack(__float_as_uint(base), __float_as_uint(base));
          uint32_t pk[NC / 2];
#pragma unroll
          for (int n = 0; n < NC; n += 2) {
            float x0, x1;
            f2_unpack(f2_fma(f2_pack(s[n], s[n + 1]), sax2, basex2), x0, x1);
            const float p0 = ex2(x0), p1 = ex2(x1);
            l2[n / 2] = f2_add(l2[n / 2], f2_pack(__float_as_uint(p0), __float_as_uint(p1)));
            pk[n / 2] = pack_bf16(p0, p1);
          }
          if (t > 0) {                                   // P of the step before has been read
            ok = spin(bar(bPV), (t - 1) & 1, W, 0x740);
            ok = __all_sync(0xffffffffu, ok);
          }
          if (ok) {
#pragma unroll
            for (int c = 0; c < NC / 8; ++c)
              st_shared_v4(aP + (((cP + c) ^ (r & 7)) << 4), pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
          }
          // a V row that no row of the tile sees must not meet a zero
          // probability with a NaN or an infinity; one that some rows see
          // leaves its non-finite elements to the epilogue
          const bool look = N > 16 && node && w.R.n > C::kFew;
          if (ok && !plain && wg == 0 && r < kv16 &&
              (!seen || look || (node && ((sNf[slot * JW + (j >> 5)] >> (j & 31)) & 1u)))) {
            ok = spin(bar(bVF + t % VS), (t / VS) & 1, W, 0x750);
            if (ok) clean_row<NB>(smem_u32(sV + (t % VS) * C::kTile) + r * 128, r, seen, look, sNf + slot * JW, j);
          }
          ok = __all_sync(0xffffffffu, ok);
        } else if (ok && t > 0) {
          // a warp without keys still keeps step with the products
          ok = spin(bar(bPV), (t - 1) & 1, W, 0x741);
          ok = __all_sync(0xffffffffu, ok);
        }
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(bar(bPF));
      }
      if (gone) break;
      // the columns' sums over this warp's keys: halve the columns, fold the lanes
      float l[NC];
#pragma unroll
      for (int n = 0; n < NC / 2; ++n) f2_unpack(l2[n], l[2 * n], l[2 * n + 1]);
      const int col = fold_cols<NC, false>(l, lane);
      sL[(slot * 4 + sw) * N + c0 + col] = l[0];
      if (sw == 0)
        for (int n = lane; n < NC; n += 32) sM[slot * N + c0 + n] = ref[n];
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(bar(bST + slot));
      ++lu;
    }
  } else {
    // -------------------------------------------------------------- epilogue
    if constexpr (N >= 64) regs_dec<C::kRegEpi>();
    const int sw = warp & 3;
    const uint32_t tl = tmem + ((uint32_t)(sw * 32) << 16);
    // D = 128: a lane is element d, all columns. D = 64: the two copies of
    // O^T share the columns.
    const int d = (D == 128 ? sw * 32 : (sw & 1) * 32) + lane;
    constexpr int NE = D == 128 ? N : N / 2;            // columns of a warp
    constexpr int CH = NE < 16 ? 8 : 16;
    const int e0 = D == 128 ? 0 : (sw >> 1) * NE;
    Unit w;
    int lu = 0;
    bool ok = true;
    while (ok && take(lu, w)) {
      const int slot = lu & 1;
      const int node0 = w.rt * p.npt, rows = min(p.npt, w.R.n - node0) * p.G;
      const bool whole = w.k0 == 0 && w.k1 == w.R.nkt;
      ok = spin(bar(bST + slot), (lu >> 1) & 1, W, 0x800) &&
           spin(bar(bMF + slot), (lu >> 1) & 1, W, 0x801);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      // maximum and sum of columns lane, lane + 32, ...
      constexpr int NL = (N + 31) / 32;
      float mx[NL], sum[NL];
#pragma unroll
      for (int x = 0; x < NL; ++x) {
        const int n = x * 32 + lane;
        mx[x] = kEmpty;
        sum[x] = 0.f;
        if (n < N) {
          const float* l = sL + slot * 4 * N + n;
          const bool dead = (sDead[slot * NW + x] >> lane) & 1u;
          if (!dead) {
            mx[x] = -sM[slot * N + n];                   // as the references: before the scale
            sum[x] = (l[0] + l[N]) + (l[2 * N] + l[3 * N]);
          }
        }
      }
      const int piece = 2 * blockIdx.x + (w.k0 == 0 ? 1 : 0);
      if (sw == 0) {
#pragma unroll
        for (int x = 0; x < NL; ++x) {
          const int n = x * 32 + lane;
          if (n < rows) {
            if (!whole) {
              p.ml[(int64_t)piece * N + n] = make_float2(mx[x], sum[x]);
            } else if (p.lse) {
              const int i = over_g(p, n), g = n - i * p.G;
              p.lse[(int64_t)(w.h * p.G + g) * p.T + w.R.r0 + node0 + i] =
                  sum[x] != 0.f ? fmaf(mx[x], fabsf(p.scale_log2), log2f(sum[x])) * kLn2 : -INFINITY;
            }
          }
        }
        if (!whole && w.k0 == 0 && lane == 0)
          p.meta[blockIdx.x] = make_int4(w.R.r0 + node0, rows, w.h, share.pieces(w));
      }
      float* inv = sInv + sw * N;
#pragma unroll
      for (int x = 0; x < NL; ++x)
        if (x * 32 + lane < N) inv[x * 32 + lane] = sum[x] != 0.f ? 1.f / sum[x] : 0.f;   // NaN stays
      __syncwarp();
      ok = spin(bar(bOF + slot), (lu >> 1) & 1, W, 0x810);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      // non-finite values of the new rows, by key
      uint32_t nf = 0;
      if (w.k1 > w.R.kt)
        for (int x = 0; x < JW; ++x) nf |= sNf[slot * JW + x];
#pragma unroll 1
      for (int q = 0; q < NE; q += CH) {
        uint32_t ov[CH];
        ld_cols<CH>(tl + colO(slot) + e0 + q, ov);
        if (q + CH == NE) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(bOE + slot));
        }
        if (e0 + q >= rows) continue;
        if (nf) {
#pragma unroll 1
          for (int x = 0; x < JW; ++x)
            for (uint32_t bits = sNf[slot * JW + x]; bits; bits &= bits - 1) {
              const int j = x * 32 + __ffs(bits) - 1;
              const float val = __bfloat162float(p.v[(int64_t)(w.R.r0 + j) * p.vs + w.h * D + d]);
              if (isfinite(val)) continue;
              const uint32_t* m = sMask + (slot * C::kNodes + j) * NW;
#pragma unroll
              for (int n = 0; n < CH; ++n)
                if ((m[(e0 + q + n) >> 5] >> ((e0 + q + n) & 31)) & 1u)
                  ov[n] = __float_as_uint(__uint_as_float(ov[n]) + val);
            }
          __syncwarp();
        }
        if (!whole) {
          float* dst = p.part + ((int64_t)piece * N + e0 + q) * D + d;
#pragma unroll
          for (int n = 0; n < CH; ++n)
            if (e0 + q + n < rows) dst[n * D] = __uint_as_float(ov[n]);
          continue;
        }
        // neighbours exchange one of two rows: an even lane stores elements
        // d, d + 1 of row n, the odd one d - 1, d of row n + 1
        const bool odd = lane & 1;
#pragma unroll
        for (int n = 0; n < CH; n += 2) {
          // an empty row is zero, whatever its accumulator holds
          const float2 iv = *reinterpret_cast<const float2*>(inv + e0 + q + n);
          const float v2[2] = {iv.x != 0.f ? __uint_as_float(ov[n]) * iv.x : 0.f,
                               iv.y != 0.f ? __uint_as_float(ov[n + 1]) * iv.y : 0.f};
          const float other = __shfl_xor_sync(0xffffffffu, odd ? v2[0] : v2[1], 1);
          const int c = e0 + q + n + (odd ? 1 : 0);
          if (c < rows) {
            const int i = over_g(p, c), g = c - i * p.G;
            const uint32_t u = odd ? pack_bf16(other, v2[1]) : pack_bf16(v2[0], other);
            *reinterpret_cast<uint32_t*>(p.o + (int64_t)(w.R.r0 + node0 + i) * p.os +
                                         (int64_t)(w.h * p.G + g) * D + (d & ~1)) = u;
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bSE + slot));
      ++lu;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) raise_status(status, kDevTimeout, *abort_flag);
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
}

// Adds the pieces of split units in block order: blocks (x, c) take the unit
// whose first piece block c of the attention left, a warp four rows of it: the
// pieces come from L2, and what is done once a row (weights, sums) bounds the
// kernel, so 8 lanes a row do it for four rows at a time (a warp a row: 4 us
// longer for the 36 MB of pieces of 16 requests with 64 nodes x 4 heads). Block
// (0, 0) gathers the blocks' status words.
struct CombineParams {
  const uint32_t* cta_status;
  const int4* meta;
  const float2* ml;
  const float* part;
  uint32_t* status;
  __nv_bfloat16* o;
  float* lse;
  int64_t os;
  int32_t T, G, blocks;
  float scale_log2;        // its size
};

constexpr int kCombineWarps = 4;

template <int D, int N>
__global__ void __launch_bounds__(32 * kCombineWarps) mis_tree_combine_kernel(const CombineParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.y;
  const int4 u = p.meta[c];
  if (c == 0 && blockIdx.x == 0 && warp == 0) {
    uint32_t bits = 0, where = 0;
    for (int x = lane; x < p.blocks; x += 32) {
      const uint32_t s = p.cta_status[2 * x];
      if (s && !bits) where = p.cta_status[2 * x + 1];
      bits |= s;
    }
    const uint32_t any = __ballot_sync(0xffffffffu, bits != 0);
    where = __shfl_sync(0xffffffffu, where, any ? __ffs(any) - 1 : 0);
    bits = __reduce_or_sync(0xffffffffu, bits);
    if (lane == 0) {
      p.status[0] = bits;
      p.status[1] = where;
    }
  }
  const int n0 = (blockIdx.x * kCombineWarps + warp) * 4, pieces = u.w;
  if (pieces < 2 || n0 >= u.y) return;
  const int sub = lane & 7, n = min(n0 + (lane >> 3), u.y - 1);
  // piece s: the first lies in block c's second slot, the others in the first
  // slots of the blocks that follow. A row's lane s looks at piece s (of 8 at
  // a time), while the first pieces' elements are on their way
  auto at = [&](int s) { return (int64_t)(s == 0 ? 2 * c + 1 : 2 * (c + s)) * N + n; };
  constexpr int E = D / 32, A = 2;                     // float4s of a lane, pieces in flight
  auto load = [&](int s, float4* y) {
    const float4* src = reinterpret_cast<const float4*>(p.part + at(s) * D) + sub;
#pragma unroll
    for (int e = 0; e < E; ++e) y[e] = src[8 * e];
  };
  float4 y[A][E], acc[E];
#pragma unroll
  for (int s = 0; s < A; ++s) load(min(s, pieces - 1), y[s]);
  bool stuck = false;
  float m = kEmpty;
  for (int s = sub; s < pieces; s += 8) {
    m = fmaxf(m, p.ml[at(s)].x);
    stuck |= (p.cta_status[2 * (c + s)] & kDevTimeout) != 0;
  }
  if (__any_sync(0xffffffffu, stuck)) return;          // a piece is missing
#pragma unroll
  for (int o = 4; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
  for (int s0 = 0; s0 < pieces; s0 += 8) {
    float a = 0.f;
    if (s0 + sub < pieces) {
      const float2 x = p.ml[at(s0 + sub)];
      a = ex2((x.x - m) * p.scale_log2);
      l += a * x.y;
      // -0: a piece that saw something, but too far below the maximum to weigh
      if (a == 0.f && x.y != 0.f) a = -0.f;
    }
    __syncwarp();
    for (int s1 = 0; s1 < min(8, pieces - s0); s1 += A) {
      if (s0 + s1 > 0) {
#pragma unroll
        for (int s = 0; s < A; ++s) load(min(s0 + s1 + s, pieces - 1), y[s]);
      }
#pragma unroll
      for (int s = 0; s < A; ++s) {
        // a piece that saw nothing weighs nothing, whatever it holds; of one
        // that weighs too little, non-finite elements count, as where a block
        // has the whole unit
        const float b = __shfl_sync(0xffffffffu, a, (lane & 24) + s1 + s);
        if (b == 0.f && signbit(b)) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            acc[e].x += isfinite(y[s][e].x) ? 0.f : y[s][e].x;
            acc[e].y += isfinite(y[s][e].y) ? 0.f : y[s][e].y;
            acc[e].z += isfinite(y[s][e].z) ? 0.f : y[s][e].z;
            acc[e].w += isfinite(y[s][e].w) ? 0.f : y[s][e].w;
          }
        } else if (b != 0.f) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            acc[e].x = fmaf(b, y[s][e].x, acc[e].x);
            acc[e].y = fmaf(b, y[s][e].y, acc[e].y);
            acc[e].z = fmaf(b, y[s][e].z, acc[e].z);
            acc[e].w = fmaf(b, y[s][e].w, acc[e].w);
          }
        }
      }
    }
  }
#pragma unroll
  for (int o = 4; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (n0 + (lane >> 3) >= u.y) return;
  const int i = n / p.G, h = u.z * p.G + n - i * p.G;
  const float inv = l != 0.f ? 1.f / l : 0.f;
  uint2* dst = reinterpret_cast<uint2*>(p.o + (int64_t)(u.x + i) * p.os + (int64_t)h * D) + sub;
#pragma unroll
  for (int e = 0; e < E; ++e)
    dst[8 * e] = inv != 0.f ? make_uint2(pack_bf16(acc[e].x * inv, acc[e].y * inv),
                                         pack_bf16(acc[e].z * inv, acc[e].w * inv))
                            : make_uint2(0u, 0u);
  if (p.lse && sub == 0)
    p.lse[(int64_t)h * p.T + u.x + i] = l != 0.f ? fmaf(m, p.scale_log2, log2f(l)) * kLn2 : -INFINITY;
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

mis_status_t check_desc(const mis_tree_desc* d, const mis_paged_cache* c) {
  if (!d) return MIS_ERR_INVALID_ARG;
  const mis_status_t cs = check_paged_cache(c);
  if (cs != MIS_OK) return cs;
  if (d->B < 1 || d->T < 0 || d->Hq < 1 || d->max_nodes < 1) return MIS_ERR_INVALID_ARG;
  const float size = std::fabs(d->scale);
  if (!(size <= 1e20f) || (size != 0.f && size < 1e-20f)) return MIS_ERR_INVALID_ARG;
  if (d->max_nodes > MIS_TREE_MAX_NODES) return MIS_ERR_UNSUPPORTED;
  if (d->Hq % c->Hkv) return MIS_ERR_SHAPE;
  if (d->Hq / c->Hkv > 128) return MIS_ERR_UNSUPPORTED;
  return MIS_OK;
}

// Rows of a unit: the smallest tile that holds all rows of a request's kv
// head, and from 65 rows on the two tiles of 128 of mis_tree_wide.cu. 16
// requests of 2000 to 8000 cached rows (8 kv heads, D = 128): 32 nodes x 2 heads
// 63 us in a tile of 64, 68 us there, 64 x 1 65 and 68, at D = 64 56 and 55; over
// 100 to 600 rows 32 and 21, but lengths are not known here. 128 rows 70 us in a
// tile of 128 columns, 69 us there, and 26 and 21 us over 100 to 600 rows.
int unit_rows(const mis_tree_desc* d, const mis_paged_cache* c) {
  const int64_t rows = (int64_t)d->max_nodes * (d->Hq / c->Hkv);
  return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 256;
}

struct TreeWs { size_t status, meta, ml, part, total; };

TreeWs workspace_of(const mis_tree_desc* d, const mis_paged_cache* c) {
  const size_t G = (size_t)num_sms(), N = (size_t)unit_rows(d, c);
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  TreeWs w;
  w.status = kStatusBytes;
  w.meta = w.status + up(G * 8);
  w.ml = w.meta + up(G * sizeof(int4));
  w.part = w.ml + up(2 * G * N * sizeof(float2));
  w.total = w.part + 2 * G * N * (size_t)c->D * sizeof(float);
  return w;
}

template <int D, int N>
mis_status_t launch_tree(const CUtensorMap* m, const TreeParams& p, const CombineParams& c,
                         cudaStream_t st) {
  if constexpr (N <= 64) {
    using Cf = TreeCfg<D, N>;
    auto kern = mis_tree_attn_kernel<D, N>;
    if (!kernel_attr_once(reinterpret_cast<const void*>(kern), Cf::kSmem)) return MIS_ERR_CUDA;
    if (launch_pdl(kern, dim3((unsigned)c.blocks), dim3(Cf::kThreads), Cf::kSmem, st, m[0],
                   m[1], m[2], m[3], m[4], m[5], m[6], p) != cudaSuccess)
      return MIS_ERR_CUDA;
  } else {
    const mis_status_t r = launch_wide(D, m, p, c.blocks, st);
    if (r != MIS_OK) return r;
  }
  return launch_pdl(mis_tree_combine_kernel<D, N>, dim3(N / (4 * kCombineWarps), (unsigned)c.blocks),
                    dim3(32 * kCombineWarps), 0, st, c) == cudaSuccess
             ? MIS_OK
             : MIS_ERR_CUDA;
}

}  // namespace
}  // namespace mis

using namespace mis;

extern "C" size_t mis_tree_attention_workspace_size(const mis_tree_desc* desc,
                                                    const mis_paged_cache* cache) {
  return check_desc(desc, cache) == MIS_OK ? workspace_of(desc, cache).total : 0;
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
  if ((int64_t)max_pages * cache->page_size > 0x7fffff00 || block_table_stride < max_pages)
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
  const TreeWs ws = workspace_of(desc, cache);
  if (!workspace || !aligned(workspace, 256) || ws_bytes < ws.total) return MIS_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // steps (with a unit's own cost) are counted in 32 bits
  const int64_t tiles = ((int64_t)max_pages * cache->page_size + kKeys - 1) / kKeys + 16;
  const int64_t rows = (int64_t)desc->max_nodes * (desc->Hq / cache->Hkv);
  if ((double)tiles * desc->B * cache->Hkv * (rows > 64 ? 2.0 * ((rows + 127) / 128) : 1.0) >= 2147483648.0)
    return MIS_ERR_UNSUPPORTED;
  if (desc->T > 0) {                     // blocks still read what others write
    const int64_t T = desc->T, B = desc->B;
    const Span in[9] = {{q, T, 2 * q_row_stride, 2 * wq}, {k, T, 2 * k_row_stride, 2 * wk},
                        {v, T, 2 * v_row_stride, 2 * wk}, cache_span(cache, cache->k),
                        cache_span(cache, cache->v), {block_table, B, 4 * block_table_stride, 4 * (int64_t)max_pages},
                        {cache_len, 1, 0, 4 * B}, {cu_nodes, 1, 0, 4 * B + 4}, {parents, 1, 0, 4 * T}};
    const Span out[3] = {{o, T, 2 * o_row_stride, 2 * wq}, {lse, 1, 0, 4 * T * desc->Hq},
                         {workspace, 1, 0, (int64_t)ws.total}};
    for (int i = 0; i < 3; ++i) {
      for (const Span& x : in)
        if (overlap(out[i], x)) return MIS_ERR_INVALID_ARG;
      for (int j = 0; j < i; ++j)
        if (overlap(out[i], out[j])) return MIS_ERR_INVALID_ARG;
    }
  }
  if (desc->T == 0)
    return cudaMemsetAsync(workspace, 0, 8, st) == cudaSuccess ? MIS_OK : MIS_ERR_CUDA;
  try {
    // the cache as (element, head, row, page), boxes of 64 elements by the
    // rows of a page (128 at most), and by 8 rows for the step that new rows
    // share; the new rows in groups of 8, so that a short request copies
    // little more than its own rows. Strides of extents of one are never
    // used, but have to be valid.
    bool ok = true;
    const uint64_t cd[4] = {(uint64_t)D, (uint64_t)cache->Hkv, (uint64_t)cache->page_size,
                            (uint64_t)cache->n_pages};
    auto stride = [&](int64_t s, int64_t extent) { return (uint64_t)(extent > 1 ? s : D) * 2; };
    const uint64_t cs[3] = {stride(cache->head_stride, cache->Hkv),
                            stride(cache->row_stride, cache->page_size),
                            stride(cache->page_stride, cache->n_pages)};
    const uint32_t cb[4] = {64, 1, (uint32_t)std::min(cache->page_size, kKeys), 1};
    const uint32_t c8[4] = {64, 1, 8, 1};
    const uint64_t nd[3] = {(uint64_t)D, (uint64_t)cache->Hkv, (uint64_t)desc->T};
    const uint64_t nk[2] = {(uint64_t)D * 2, (uint64_t)k_row_stride * 2};
    const uint64_t nv[2] = {(uint64_t)D * 2, (uint64_t)v_row_stride * 2};
    const uint32_t nb[3] = {64, 1, 8};
    // Q by the rows of a tile's nodes
    const uint64_t qd[3] = {(uint64_t)D, (uint64_t)desc->Hq, (uint64_t)desc->T};
    const uint64_t qst[2] = {(uint64_t)D * 2, (uint64_t)q_row_stride * 2};
    const int N = unit_rows(desc, cache), G = desc->Hq / cache->Hkv, npt = (N == 256 ? 128 : N) / G;
    const uint32_t qb[3] = {64, (uint32_t)G, (uint32_t)npt};
    const CUtensorMap maps[7] = {
        encode_tmap_bf16(q, 3, qd, qst, qb, &ok),
        encode_tmap_bf16(cache->k, 4, cd, cs, cb, &ok), encode_tmap_bf16(cache->v, 4, cd, cs, cb, &ok),
        encode_tmap_bf16(cache->k, 4, cd, cs, c8, &ok), encode_tmap_bf16(cache->v, 4, cd, cs, c8, &ok),
        encode_tmap_bf16(k, 3, nd, nk, nb, &ok), encode_tmap_bf16(v, 3, nd, nv, nb, &ok)};
    if (!ok) return MIS_ERR_CUDA;
    uint8_t* base = static_cast<uint8_t*>(workspace);
    TreeParams p;
    p.v = static_cast<const __nv_bfloat16*>(v);
    p.o = static_cast<__nv_bfloat16*>(o);
    p.lse = lse;
    p.vs = v_row_stride; p.os = o_row_stride;
    p.n_pages = cache->n_pages;
    p.page_shift = 31 - __builtin_clz((unsigned)cache->page_size);
    p.max_pages = max_pages;
    p.table = block_table; p.table_stride = block_table_stride;
    p.cache_len = cache_len; p.cu = cu_nodes; p.parents = parents;
    p.B = desc->B; p.T = desc->T; p.Hkv = cache->Hkv;
    p.G = G; p.npt = npt; p.npu = N == 256 ? 2 * npt : npt;
    p.g_magic = (uint32_t)((0xffffffffull + (uint64_t)p.G) / (uint64_t)p.G);
    p.max_nodes = desc->max_nodes;
    p.lanes = std::min((desc->max_nodes + p.npu - 1) / p.npu, 2);
    p.scale_log2 = (desc->scale != 0.f ? desc->scale : 1.f / std::sqrt((float)D)) * 1.4426950408889634f;
    p.cta_status = reinterpret_cast<uint32_t*>(base + ws.status);
    p.meta = reinterpret_cast<int4*>(base + ws.meta);
    p.ml = reinterpret_cast<float2*>(base + ws.ml);
    p.part = reinterpret_cast<float*>(base + ws.part);
    p.wait_ns = wait_limit_ns();
    p.stall = inject_stall_mask() & 1u;
    CombineParams c;
    c.cta_status = p.cta_status; c.meta = p.meta; c.ml = p.ml; c.part = p.part;
    c.status = reinterpret_cast<uint32_t*>(base);
    c.o = p.o; c.lse = lse; c.os = o_row_stride;
    c.T = desc->T; c.G = G; c.blocks = num_sms(); c.scale_log2 = std::fabs(p.scale_log2);
    if (D == 128) {
      if (N == 16) return launch_tree<128, 16>(maps, p, c, st);
      if (N == 32) return launch_tree<128, 32>(maps, p, c, st);
      if (N == 64) return launch_tree<128, 64>(maps, p, c, st);
      return launch_tree<128, 256>(maps, p, c, st);
    }
    if (N == 16) return launch_tree<64, 16>(maps, p, c, st);
    if (N == 32) return launch_tree<64, 32>(maps, p, c, st);
    if (N == 64) return launch_tree<64, 64>(maps, p, c, st);
    return launch_tree<64, 256>(maps, p, c, st);
  } catch (...) {
    return MIS_ERR_CUDA;
  }
}
