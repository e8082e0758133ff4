// Tree attention for requests with many rows a kv head (more than 64), sm_103a:
// the products the usual way round,
//     S [128 rows x 128 keys] = Q K^T,     O [128 rows x D] += P V,
// for two row tiles that share every K and V tile. A thread owns a row: its
// maximum, sum and reference stay in registers (no exchange between threads),
// P goes to tensor memory, and one tile's softmax runs during the other's
// products. Everything else (units, shares, copies, pieces) is as in
// mis_tree.cu; a unit is a pair of row tiles, or one tile where the request has
// no more rows.
//
// What bounds it, at D = 128: a tile's round of a step is about 1060 cycles of PV
// and the next S, 320 until its scores are seen, 1130 of softmax and 450 until
// the products of its P go out: 2960, in which the other tile's 1060 fit. No pipe
// is full: the tensor pipe is active for 52% of the cycles, issue slots for 37%,
// exponentials for 27%, memory for 57%; a round is a chain of latencies, and
// tensor memory holds no third tile to fill it. Two warps a row's half took longer
// (81 us, one 77). K and V alone, all from L2, change little (2 us).
// 16 requests of 2000 to 8000 cached rows, 64 nodes x 4 heads, 8 kv heads: 77 to
// 78 us with the second kernel's 9, 4.5 TB/s and 1080 TFLOP/s. D = 64 is alike:
// 64 us where K and V take 26 (tensor pipe 30%, issue 41%, exponentials 30%,
// memory 41%).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "mis_internal.h"
#include "mis_ptx.cuh"
#include "mis_tree.cuh"

namespace mis {
namespace tree {
namespace {

template <int D>
struct WideCfg {
  static constexpr int kNB = D / 64;             // 64-column boxes of a row
  static constexpr int kThreads = 384;
  // Register budgets of the warpgroups: their sum is the launch's, 384 x 168
  static constexpr int kRegCtl = 88, kRegSoft = 208;
  static_assert(128 * (kRegCtl + 2 * kRegSoft) <= kThreads * 168, "register split exceeds the launch allocation");
  static constexpr int kBox = kKeys * 128;
  static constexpr int kTile = kNB * kBox;       // of K, V and Q alike
  static constexpr int kK = D == 128 ? 2 : 4, kV = D == 128 ? 2 : 4;
  // see TreeCfg; with 2, 3, 4 and 5: the pairs above 79.4, 78.0, 77.7, 78.2 us, over
  // other lengths 80.3, 79.4, 79.5, 79.5; 32 pairs over 100 to 600 rows 38.1, 40.1,
  // 39.5, 40.7; 16 single tiles 70.6, 70.5, 71.8, 71.9; pairs at D = 64 39.5, 39.8, 39.3, 40.1
  static constexpr int kUnitCost = 4;
  static constexpr int kW = MIS_TREE_MAX_NODES / 32;    // words of a node's mask
  static constexpr int oMask = 0;                       // [2][256][kW] new keys that a node sees
  static constexpr int oDead = oMask + 2 * MIS_TREE_MAX_NODES * kW;   // [2][kW] unused nodes
  static constexpr int oNf = oDead + 2 * kW;            // [2][kW] keys with a non-finite value
  static constexpr int oPar = oNf + 2 * kW;             // [256] int16: parents
  static constexpr int kWords = oPar + MIS_TREE_MAX_NODES / 2;
  static constexpr int kData = (2 + kK + kV) * kTile;
  static constexpr int kSmem = kData + 4 * kWords + 512 + 1024;
  static_assert(kSmem <= 232448, "shared memory");
};

// Four lanes exchange the four 16-byte pieces each holds of its row: piece e
// becomes piece lane % 4 of row e of the four. A store then covers 64 bytes of
// 8 rows (16 bytes of 32 rows took four times as long).
__device__ __forceinline__ void spread4(uint32_t* u, int lane) {
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (e & o) continue;
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const uint32_t give = up ? u[4 * e + y] : u[4 * (e | o) + y];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, give, o);
        if (up) u[4 * e + y] = got;
        else u[4 * (e | o) + y] = got;
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(WideCfg<D>::kThreads, 1)
mis_tree_wide_kernel(const __grid_constant__ CUtensorMap qmap,
                     const __grid_constant__ CUtensorMap kcmap,
                     const __grid_constant__ CUtensorMap vcmap,
                     const __grid_constant__ CUtensorMap kc8map,
                     const __grid_constant__ CUtensorMap vc8map,
                     const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const TreeParams p) {
  using C = WideCfg<D>;
  constexpr int NB = C::kNB, KS = C::kK, VS = C::kV, W8 = C::kW;
  // barriers
  constexpr int bQF = 0, bQE = bQF + 1, bKF = bQE + 1, bKE = bKF + KS, bVF = bKE + KS, bVE = bVF + VS,
                bSF = bVE + VS, bPF = bSF + 2, bOF = bPF + 2, bSE = bOF + 2, bMF = bSE + 2,
                bUF = bMF + 2, bUE = bUF + kUnits, bDR = bUE + kUnits, nBar = bDR + 1;
  static_assert(nBar * 8 + 64 <= 512, "barrier space");

  griddep_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + 2 * C::kTile;
  uint8_t* sV = sK + KS * C::kTile;
  uint32_t* words = reinterpret_cast<uint32_t*>(smem + C::kData);
  uint32_t* sMask = words + C::oMask;
  uint32_t* sDead = words + C::oDead;
  uint32_t* sNf = words + C::oNf;
  int16_t* sPar = reinterpret_cast<int16_t*>(words + C::oPar);
  uint64_t* bars = reinterpret_cast<uint64_t*>(words + C::kWords);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + nBar);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  __shared__ Unit s_start, s_unit[kUnits];
  __shared__ int s_sums[2][C::kThreads / 32];
  auto bar = [&](int i) { return smem_u32(bars + i); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    mbar_init(bar(bQF), 1);
    mbar_init(bar(bQE), 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(bSF + s), 1);
      mbar_init(bar(bPF + s), 4);
      mbar_init(bar(bOF + s), 1);
      mbar_init(bar(bSE + s), 8);
      mbar_init(bar(bMF + s), 1);
    }
    for (int s = 0; s < KS; ++s) { mbar_init(bar(bKF + s), 1); mbar_init(bar(bKE + s), 1); }
    for (int s = 0; s < VS; ++s) { mbar_init(bar(bVF + s), 1); mbar_init(bar(bVE + s), 1); }
    mbar_init(bar(bDR), 1);
    for (int s = 0; s < kUnits; ++s) {
      mbar_init(bar(bUF + s), 1);
      mbar_init(bar(bUE + s), 11);         // every warp but the K producer
    }
    fence_mbar_init();
    fence_proxy_async();
    tma_prefetch_desc(&qmap); tma_prefetch_desc(&kcmap); tma_prefetch_desc(&vcmap);
    tma_prefetch_desc(&kc8map); tma_prefetch_desc(&vc8map);
    tma_prefetch_desc(&kmap); tma_prefetch_desc(&vmap);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  griddep_wait();

  uint32_t* status = p.cta_status + 2 * blockIdx.x;
  const Share share = find_share<2, C::kThreads, C::kUnitCost>(p, status, &s_start, s_sums);
  const uint32_t tmem = *tmem_slot;
  const Bound W{abort_flag, p.wait_ns};
  // tensor memory: S_0 | S_1 | O_0 | O_1; P, as bf16 pairs, in the first half of S
  auto colS = [](int x) { return (uint32_t)(x * 128); };
  auto colO = [](int x) { return (uint32_t)(256 + x * D); };
  const UnitRing units_ring{s_unit, bar(bUF), bar(bUE)};
  auto take = [&](int lu, Unit& u) -> bool { return tree::take(units_ring, lu, u, W); };

  if (warp < 4) {
    regs_dec<C::kRegCtl>();
    if (warp == 0 || warp == 3) {
      const bool y = warp == 3;
      const Producer io{y ? &vcmap : &kcmap, y ? &vc8map : &kc8map, y ? &vmap : &kmap, &qmap,
                        smem_u32(y ? sV : sK), smem_u32(sQ), bar(y ? bVF : bKF), bar(y ? bVE : bKE),
                        bar(bQF), bar(bQE), y ? VS : KS, units_ring, &s_start};
      produce<NB, 2, 128, 1, C::kUnitCost>(p, io, y, share.steps, status, W);
    } else if (warp == 1) {
      // --------------------------------------------------------------- MMA
      // The warp walks together and one elected lane issues, so loop state and
      // descriptors stay in uniform registers. A tile's S of the next step
      // follows its PV at once; meanwhile the other tile's softmax goes on
      constexpr uint32_t idS = idesc_bf16(128, 128, false);
      constexpr uint32_t idO = idesc_bf16(128, D, true);
      auto wait_all = [&](int b, uint32_t parity, uint32_t where) -> bool {
        const bool r = spin(bar(b), parity, W, where);
        return __all_sync(0xffffffffu, r);
      };
      bool ok = true;
      if (p.stall) ok = wait_all(bDR, 0, 0x7ff);               // nothing arrives before the drain
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      struct Ring { int slot; uint32_t ph; };
      auto turn = [](Ring& r, int depth) { if (++r.slot == depth) { r.slot = 0; r.ph ^= 1; } };
      Ring rk{0, 0}, rv{0, 0};
      uint32_t pf0 = 0, pf1 = 0, qf = 0;                       // phases of P and Q
      // Once barrier wb (a lane's own; none below 0) has passed phase wp: PV of tile
      // x for the step whose P is there (nks > 0), then S of the step behind it
      // (more). V is MN-major: 8-key groups 1024 B apart, 64-column boxes kBox
      // apart. The last tile's products release K and V, and in the unit's last
      // step Q. Descriptors are made before the wait
      auto step = [&](int x, uint32_t acc, int nks, bool done, bool more, bool last, int wb, uint32_t wp) -> bool {
        const uint32_t dO = tm + colO(x), dS = tm + colS(x);
        uint64_t v = sdesc_sw128(smem_u32(sV) + rv.slot * C::kTile, C::kBox, 1024);
        uint64_t q = sdesc_sw128(smem_u32(sQ) + x * C::kTile, 16, 1024);
        uint64_t kd = sdesc_sw128(smem_u32(sK) + rk.slot * C::kTile, 16, 1024);
        asm volatile("" : "+l"(v), "+l"(q), "+l"(kd));
        if (wb >= 0 && !wait_all(wb, wp, 0x400 + 0x10 * x)) return false;
        tc_fence_after();
        if (elect_uniform()) {
          if (nks) {
            mma_ts(dO, dS, v, idO, acc);
            if (nks == kKeys / 16) {
#pragma unroll
              for (int ks = 1; ks < kKeys / 16; ++ks) mma_ts(dO, dS + ks * 8, v + ks * 128, idO, 1u);
            } else {
#pragma unroll 1
              for (int ks = 1; ks < nks; ++ks) mma_ts(dO, dS + ks * 8, v + ks * 128, idO, 1u);
            }
            if (done) mma_commit(bar(bVE + rv.slot));
            if (!more) mma_commit(bar(bOF + x));
          }
          if (more) {
#pragma unroll
            for (int e = 0; e < NB; ++e)
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                mma_ss(dS, q + ((e * C::kBox + ks * 32) >> 4), kd + ((e * C::kBox + ks * 32) >> 4), idS,
                       (e | ks) != 0);
            mma_commit(bar(bSF + x));
            if (done) mma_commit(bar(bKE + rk.slot));
            if (done && last) mma_commit(bar(bQE));
          }
        }
        __syncwarp();
        return true;
      };
      Unit w;
      for (int lu = 0; ok && take(lu, w); ++lu) {
        const int k0 = __shfl_sync(0xffffffffu, w.k0, 0), k1 = __shfl_sync(0xffffffffu, w.k1, 0);
        const int kt = __shfl_sync(0xffffffffu, w.R.kt, 0), L = __shfl_sync(0xffffffffu, w.R.L, 0);
        const int an = __shfl_sync(0xffffffffu, w.R.a + w.R.n, 0);
        const bool pair = __shfl_sync(0xffffffffu, w.R.n - w.rt * p.npu, 0) > p.npt;
        // before the first step: S alone. Lanes wait for a barrier each: one
        // trip for all that a product needs
        for (int k = k0 - 1; k < k1; ++k) {
          const bool begin = k < k0, more = k + 1 < k1, last = k + 2 == k1;
          const uint32_t acc = k > k0 ? 1u : 0u;
          const int kv = min(kKeys, k < kt ? L - k * kKeys : an - (k - kt) * kKeys);
          const int nks = begin ? 0 : (kv + 15) >> 4;
          const bool l1 = (lane & 1) != 0, l2 = more && (lane & 2);
          const int wb = l1 ? (begin ? bQF : bVF + rv.slot) : l2 || begin ? bKF + rk.slot : bPF;
          const uint32_t wp = l1 ? (begin ? qf : rv.ph) : l2 || begin ? rk.ph : pf0;
          if (!(ok = step(0, acc, nks, !pair, more, last, wb, wp))) break;
          if (pair && !(ok = step(1, acc, nks, true, more, last, begin ? -1 : bPF + 1, pf1))) break;
          if (begin) {
            qf ^= 1;
          } else {
            pf0 ^= 1;
            if (pair) pf1 ^= 1;
            turn(rv, VS);
          }
          if (more) turn(rk, KS);
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
        const int sm = lu & 1, n = w.R.n;
        if (lu >= 2) ok = spin(bar(bSE + sm), ((lu >> 1) - 1) & 1, W, 0x610);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const bool tree = w.k1 > w.R.kt;
        if (lane < W8) sNf[sm * W8 + lane] = 0;
        __syncwarp();
        // parents: the index, or -1 for roots, for children of unused nodes and
        // for what is no index; unused nodes themselves -2. A node's ancestors
        // among its batch of 32 are walked (they share a word), those before
        // are the ancestors of the first one before the batch
        uint32_t* m = sMask + sm * MIS_TREE_MAX_NODES * W8;
        if (p.parents) {
          int raw[W8];
#pragma unroll
          for (int q = 0; q < W8; ++q) raw[q] = q * 32 + lane < n ? p.parents[w.R.r0 + q * 32 + lane] : MIS_TREE_ROOT;
#pragma unroll
          for (int q = 0; q < W8; ++q) {
            if (raw[q] >= q * 32 + lane || raw[q] < MIS_TREE_UNUSED) {
              bad |= q * 32 + lane < n;
              raw[q] = MIS_TREE_ROOT;
            }
            sPar[q * 32 + lane] = (int16_t)raw[q];
          }
          __syncwarp();
        }
#pragma unroll 1
        for (int b0 = 0; b0 < MIS_TREE_MAX_NODES; b0 += 32) {
          const int i = b0 + lane, wi = b0 >> 5;
          int up = i - 1;
          if (p.parents) {
            up = sPar[i];
            if (up >= 0 && sPar[up] == MIS_TREE_UNUSED) {
              up = MIS_TREE_ROOT;
              sPar[i] = MIS_TREE_ROOT;
            }
          }
          const bool dead = i < n && up == MIS_TREE_UNUSED;
          const uint32_t dw = __ballot_sync(0xffffffffu, dead);
          if (lane == 0) sDead[sm * W8 + wi] = dw;
          if (!tree || b0 >= n) continue;
          __syncwarp();
          uint32_t own = 0;
          int j = -1;
          if (i < n && !dead) {
            if (p.parents) {
              for (j = i; j >= b0; j = sPar[j]) own |= 1u << (j & 31);
            } else {
              own = 0xffffffffu >> (31 - lane);
              j = b0 - 1;
            }
          }
          if (i < n) {
#pragma unroll 1
            for (int x = 0; x < W8; ++x) m[i * W8 + x] = x == wi ? own : x < wi && j >= 0 ? m[j * W8 + x] : 0u;
          }
          __syncwarp();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(bMF + sm));
        ++lu;
      }
      __syncwarp();
      if (bad) raise_status(status, kDevIndex, 0x42);
    }
  } else {
    // ------------------------------------------------- softmax and epilogue
    regs_inc<C::kRegSoft>();
    const int x = (warp - 4) >> 2, sw = warp & 3, r = sw * 32 + lane;
    const uint32_t tl = tmem + ((uint32_t)(sw * 32) << 16);
    const uint32_t tS = tl + colS(x), tO = tl + colO(x);
    // scores are taken times the scale's sign, then scaled by its size
    const float sa = fabsf(p.scale_log2), grow_by = kGrow / sa;
    const bool neg = p.scale_log2 < 0.f;
    const uint64_t sax2 = f2_pack(__float_as_uint(sa), __float_as_uint(sa));
    const int box_shift = min(p.page_shift, 7), boxes = kKeys >> box_shift;
    Unit w;
    uint32_t cs = 0, co = 0;                             // S tiles and units of this row tile so far
    int lu = 0, tk = 0;                                  // tk: steps of the block's units so far
    bool ok = true;
    while (ok && take(lu, w)) {
      const int slot = lu & 1, node0 = w.rt * p.npu + x * p.npt;
      const int rows = min(p.npt, w.R.n - node0) * p.G;
      if (rows <= 0) {
        // no such tile in this unit; its masks' place is given back all the same
        ok = spin(bar(bMF + slot), (lu >> 1) & 1, W, 0x701);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) mbar_arrive(bar(bSE + slot));
        tk += w.k1 - w.k0;
        ++lu;
        continue;
      }
      const int i = over_g(p, min(r, rows - 1));         // the row's node
      const uint32_t* mrow = sMask + (slot * MIS_TREE_MAX_NODES + node0 + i) * W8;
      float m = kEmpty, l = 0.f;                         // the row's reference and sum
      // the page under box `lane` of a step, asked for a step ahead (0 where
      // there is no cached row)
      const int32_t* trow = p.table + (int64_t)w.b * p.table_stride;
      auto page_of = [&](int k) {
        const int at = k * kKeys + (lane << box_shift);
        return k < w.k1 && lane < boxes && at < w.R.L ? trow[at >> p.page_shift] : 0;
      };
      int page = page_of(w.k0);
#pragma unroll 1
      for (int k = w.k0; k < w.k1; ++k, ++cs) {
        const int kv = w.keys(k);
        const bool fresh = k >= w.R.kt;
        const uint32_t pages = __ballot_sync(0xffffffffu, page >= 0 && page < p.n_pages);
        page = page_of(k + 1);
        const bool plain = !fresh && kv == kKeys && pages == 0xffffffffu;
        ok = spin(bar(bSF + x), cs & 1, W, 0x710);
        if (ok && fresh) ok = spin(bar(bMF + slot), (lu >> 1) & 1, W, 0x720);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        // the whole row of scores in registers
        uint32_t s[kKeys];
#pragma unroll
        for (int c = 0; c < kKeys; c += 32) tmem_ld32(tS + c, s + c);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < kKeys; c += 32) reg_fence32(s + c);
        if (neg) {
#pragma unroll
          for (int c = 0; c < kKeys; ++c) s[c] ^= 0x80000000u;
        }
        if (!plain) {
          // keys by words of 32: cached rows on pages of the cache, then new row
          // j0 + c for key c where the row's mask has it
          const int j0 = (k - w.R.kt) * kKeys - w.R.a;
          bool there = false;                            // key row r holds something
#pragma unroll
          for (int q = 0; q < kKeys / 32; ++q) {
            uint32_t vis = bit_range(-32 * q, w.R.L - k * kKeys - 32 * q);
            if (pages != 0xffffffffu) {
#pragma unroll 1
              for (int b = 0; b < boxes; ++b)
                if (!((pages >> b) & 1u)) vis &= ~bit_range((b << box_shift) - 32 * q, ((b + 1) << box_shift) - 32 * q);
            }
            if (q == sw) there = (vis >> lane) & 1u;
            if (fresh) {
              const int at = j0 + 32 * q, wd = at >> 5;
              const uint32_t lo = wd >= 0 && wd < W8 ? mrow[wd] : 0u;
              const uint32_t hi = wd + 1 >= 0 && wd + 1 < W8 ? mrow[wd + 1] : 0u;
              vis |= __funnelshift_r(lo, hi, at & 31);
            }
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!((vis >> c) & 1u)) s[32 * q + c] = 0xff800000u;
          }
          // a V row that nobody sees must not meet a zero probability with a NaN
          // or an infinity; a new one that some rows see leaves its non-finite
          // elements to the epilogue. The first tile's warps see to it, and the
          // second tile's product comes behind the first's
          const int j = j0 + r;
          const bool node = fresh && j >= 0 && j < w.R.n;
          if (x == 0 && r < ((kv + 15) & ~15) && !there) {
            const int t = tk + k - w.k0;
            ok = spin(bar(bVF + t % VS), (t / VS) & 1, W, 0x750);
            if (ok) {
              clean_row<NB>(smem_u32(sV + (t % VS) * C::kTile) + r * 128, r, node, node, sNf + slot * W8, j);
              fence_proxy_async();
            }
          }
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < kKeys; c += 2)
          mx[(c >> 1) & 3] = max3(mx[(c >> 1) & 3], __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
        const float top = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
        const bool grow = top > m + grow_by;
        const bool any_grow = __any_sync(0xffffffffu, grow);
        const float alpha = grow ? ex2((m - top) * sa) : 1.f;
        if (grow) { l *= alpha; m = top; }
        // the reference after the scale, negated; one far from zero is taken off
        // the scores instead (a row that saw nothing has no score to take it off)
        const float scaled = -m * sa;
        const bool far = fabsf(scaled) > kFar;
        const float off = far ? 0.f : scaled;
        if (far && m > kEmpty) {
#pragma unroll
          for (int c = 0; c < kKeys; ++c) s[c] = __float_as_uint(__uint_as_float(s[c]) - m);
        }
        const uint64_t offx2 = f2_pack(__float_as_uint(off), __float_as_uint(off));
        uint64_t sum[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t pk[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const int k2 = hf * 64 + 2 * c;
            float x0, x1;
            f2_unpack(f2_fma(f2_pack(s[k2], s[k2 + 1]), sax2, offx2), x0, x1);
            const float p0 = ex2(x0), p1 = ex2(x1);
            sum[c & 3] = f2_add(sum[c & 3], f2_pack(__float_as_uint(p0), __float_as_uint(p1)));
            pk[c] = pack_bf16(p0, p1);
          }
          tmem_st32(tS + hf * 32, pk);
        }
        {
          float a0, a1;
          f2_unpack(f2_add(f2_add(sum[0], sum[1]), f2_add(sum[2], sum[3])), a0, a1);
          l += a0 + a1;
        }
        if (any_grow && k > w.k0) {
          // S of this step was issued behind the products of the steps before,
          // so O holds them
#pragma unroll
          for (int c = 0; c < D; c += 32) {
            uint32_t ov[32];
            tmem_ld32(tO + c, ov);
            tmem_ld_wait();
            reg_fence32(ov);
#pragma unroll
            for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
            tmem_st32(tO + c, ov);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(bPF + x));
      }
      if (!ok) break;
      tk += w.k1 - w.k0;
      // ---------------------------------------------------------- epilogue
      ok = spin(bar(bMF + slot), (lu >> 1) & 1, W, 0x801);
      if (ok) ok = spin(bar(bOF + x), co & 1, W, 0x810);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      ++co;
      tc_fence_after();
      const bool whole = w.k0 == 0 && w.k1 == w.R.nkt, mine = r < rows;
      if ((sDead[slot * W8 + ((node0 + i) >> 5)] >> ((node0 + i) & 31)) & 1u) { m = kEmpty; l = 0.f; }
      const int g = r - i * p.G;
      const int64_t piece = 2 * (int64_t)blockIdx.x + (w.k0 == 0 ? 1 : 0);
      const int pr = x * p.npt * p.G + r;                          // a piece's rows lie end to end
      const int64_t orow = (int64_t)(w.R.r0 + node0 + i);
      if (!whole) {
        if (mine) p.ml[piece * 256 + pr] = make_float2(m, l);
        if (w.k0 == 0 && threadIdx.x == 128)
          p.meta[blockIdx.x] = make_int4(w.R.r0 + node0, min(p.npu, w.R.n - node0) * p.G, w.h, share.pieces(w));
      } else if (mine && p.lse) {
        p.lse[(int64_t)(w.h * p.G + g) * p.T + orow] = l != 0.f ? fmaf(m, sa, log2f(l)) * kLn2 : -INFINITY;
      }
      const float inv = l != 0.f ? 1.f / l : 0.f;                  // NaN stays
      const int64_t oat = mine ? orow * p.os + (int64_t)(w.h * p.G + g) * D : -1;
      uint32_t nf = 0;
      if (w.k1 > w.R.kt)
        for (int q = 0; q < W8; ++q) nf |= sNf[slot * W8 + q];
      if (nf) {
#pragma unroll 1
        for (int c = 0; c < D; c += 8) {
          uint32_t ov[8];
          tmem_ld8(tO + c, ov);
          tmem_ld_wait();
          reg_fence8(ov);
#pragma unroll 1
          for (int q = 0; q < W8; ++q)
#pragma unroll 1
            for (uint32_t bits = sNf[slot * W8 + q] & mrow[q]; bits; bits &= bits - 1) {
              const __nv_bfloat16* v = p.v + (int64_t)(w.R.r0 + q * 32 + __ffs(bits) - 1) * p.vs + w.h * D + c;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float val = __bfloat162float(v[e]);
                if (!isfinite(val)) ov[e] = __float_as_uint(__uint_as_float(ov[e]) + val);
              }
            }
          __syncwarp();
          tmem_st8(tO + c, ov);
        }
        tmem_st_wait();
      }
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t ov[32];
        tmem_ld32(tO + c, ov);
        tmem_ld_wait();
        reg_fence32(ov);
        if (!whole) {
          float* part = p.part + piece * 256 * D + c;
          spread4(ov, lane);
          spread4(ov + 16, lane);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int to = __shfl_sync(0xffffffffu, mine ? pr : -1, (lane & ~3) | e);
            uint4* dst = reinterpret_cast<uint4*>(part + (int64_t)to * D) + (lane & 3);
            if (to >= 0) dst[0] = make_uint4(ov[4 * e], ov[4 * e + 1], ov[4 * e + 2], ov[4 * e + 3]);
            if (to >= 0) dst[4] = make_uint4(ov[4 * e + 16], ov[4 * e + 17], ov[4 * e + 18], ov[4 * e + 19]);
          }
          continue;
        }
        uint32_t u[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          // an empty row is zero, whatever its accumulator holds
          const float v0 = __uint_as_float(ov[2 * e]), v1 = __uint_as_float(ov[2 * e + 1]);
          u[e] = inv != 0.f ? pack_bf16(v0 * inv, v1 * inv) : 0u;
        }
        spread4(u, lane);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int64_t to = __shfl_sync(0xffffffffu, oat, (lane & ~3) | e);
          if (to >= 0)
            *(reinterpret_cast<uint4*>(p.o + to + c) + (lane & 3)) =
                make_uint4(u[4 * e], u[4 * e + 1], u[4 * e + 2], u[4 * e + 3]);
        }
      }
      __syncwarp();
      tc_fence_before();
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
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
mis_status_t launch(const CUtensorMap* m, const TreeParams& p, int blocks, cudaStream_t st) {
  using C = WideCfg<D>;
  auto kern = mis_tree_wide_kernel<D>;
  if (!kernel_attr_once(reinterpret_cast<const void*>(kern), C::kSmem)) return MIS_ERR_CUDA;
  return launch_pdl(kern, dim3((unsigned)blocks), dim3(C::kThreads), C::kSmem, st, m[0], m[1], m[2], m[3],
                    m[4], m[5], m[6], p) == cudaSuccess
             ? MIS_OK
             : MIS_ERR_CUDA;
}

}  // namespace

mis_status_t launch_wide(int D, const CUtensorMap* m, const TreeParams& p, int blocks, cudaStream_t st) {
  return D == 128 ? launch<128>(m, p, blocks, st) : launch<64>(m, p, blocks, st);
}

}  // namespace tree
}  // namespace mis
