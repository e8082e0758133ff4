// Attention of the newest rows of each request over an 8-bit paged K/V cache,
// sm_103a.
//
// Request b has len_b cached rows, the last n_b of them its new ones. New row i
// and query head q of kv head h see the keys j < len_b - n_b + i + 1:
//     s_j = scale * q k_j,   o = sum_j softmax(s)_j v_j,
// k_j and v_j being codes times 2^e of their row (mis_q8.cu). The R = n_b * G
// rows of a kv head share every key; they are few, so the keys take the wide
// side of the products, as in mis_tree.cu:
//     S^T [128 keys x 2N] = K Q^T        (A = K tile, B = Q in two parts)
//     O^T [D x 3N]       += V^T P^T      (A = V tile, MN-major, B = P in three)
// with N = 16 or 32 rows a tile, all of it e4m3: K and V go from the cache to
// the tensor core as they lie there, and what the softmax computes anyway is
// what gets split. Q's parts are its leading 4 bits and 32 times the rest, in
// units of a power of two of each row: exact for bf16 elements down to 2^-14 of
// the row's largest, within 2^-22 of that below. P is rounded to fp16 (11 bits)
// and split into 4 bits, 16 times the next 4, 256 times the last 3: exact, but
// that weights below 2^-17 of the largest lose bits, to within 2^-25 of it. The
// parts' products stand in columns of their own and are added when they are read.
// (V converted to fp16 by a warpgroup of its own, P in one part: 64 decoded
// tokens 74 us. By mma.sync with K and V converted in registers: 73 us, and
// three times that for 64 rows a kv head.)
//
// A row's key scale multiplies its score, its value scale its probability. The
// softmax keeps two things per row: a reference r below which weights are
// taken, and l = sum 2^(s - r). Products use P = 2^(s - r + e_v - 26): r is the
// largest s + e_v - 32 seen, moved only when one passes it by 2^2.5, so P lies
// below e4m3's 448 and its largest above 2^6, whatever the spread of the value
// scales; 2^(s - r) stays within fp32 for every e_v in [-56, 120].
//
// Work is cut evenly between blocks, not at requests: every block adds up the
// 128-key steps of all units (request, kv head, row tile) from the lengths on
// the device and walks its own share; pieces of a unit that several blocks hold
// are joined by a second kernel in block order, so the same call gives the same
// bits. Warp roles: 0 and 3 TMA producers of K (with both tiles' exponents) and
// of V, 1 issues the products, 2 lays out Q, then the softmax (a thread is a key
// and owns 16 columns; with N = 16 in two streams that take the steps in turn,
// each with a reference and an accumulator of its own), and an epilogue that adds
// the streams (a thread is an element of the head). Every role walks the share by itself;
// waits are bounded.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "mis_internal.h"
#include "mis_ptx.cuh"
#include "mis_rows.cuh"

namespace mis {

CUtensorMap encode_tmap_u8(const void* base, int rank, const uint64_t* dims, const uint64_t* strides_bytes,
                           const uint32_t* box, bool* ok);

namespace {

using namespace dev;

constexpr int kKeys = 128;             // of a step
constexpr int kJoinWarps = 4;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kNone = -3.0e38f;      // reference of a row that has seen nothing
constexpr float kDead = 3.0e38f;       // ... of a column that is no row: its weights are zero

struct AttnParams {
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;                          // or null
  int64_t qs, os;
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
  uint64_t wait_ns;
  uint32_t stall;
  // workspace
  uint32_t* status;
  uint32_t* flags;                     // [blocks][2]: bits, site
  int4* meta;                          // [blocks][2]: the split unit that starts in the block
  float2* rl;                          // [2 * blocks][N]: (r, l) of a piece's rows
  float* part;                         // [2 * blocks][N][D]
};

// A request's work: units of N of a kv head's n * G rows, the tiles of a head
// side by side. A step of 128 keys of a unit counts one.
struct Job {
  int len, row0, n;                    // cached rows; first new row, new rows
  int steps, tiles, units;
  bool ok;
  __device__ __forceinline__ int64_t cost() const { return (int64_t)steps * units; }
};

// What a request brings, as read.
struct Given { int len, row0, end; };
__device__ __forceinline__ Given given(const AttnParams& p, int b) {
  return b < p.B ? Given{p.cache_len[b], p.cu[b], p.cu[b + 1]} : Given{0, 0, 0};
}
template <int N>
__device__ __forceinline__ Job job_of(const AttnParams& p, const Given& g) {
  Job j;
  j.len = g.len;
  j.row0 = g.row0;
  j.ok = j.row0 >= 0 && g.end >= j.row0 && g.end <= p.T && g.end - j.row0 <= p.max_rows && j.len >= 0 &&
         j.len <= (int64_t)p.max_pages << p.page_shift && g.end - j.row0 <= j.len;
  j.n = j.ok ? g.end - j.row0 : 0;
  j.steps = j.n ? (j.len + kKeys - 1) / kKeys : 0;
  j.tiles = (j.n * p.G + N - 1) / N;
  j.units = j.tiles * p.Hkv;
  return j;
}
template <int N>
__device__ __forceinline__ Job job_of(const AttnParams& p, int b) { return job_of<N>(p, given(p, b)); }

// Blocks that take part.
__device__ __forceinline__ int blocks_for(int64_t total, int blocks) {
  return (int)min((int64_t)blocks, max((int64_t)1, total));
}

// Walks the pieces of units that a block's share holds.
template <int N>
struct Walk {
  int64_t left;                        // steps of the share from this piece on
  int b, u;                            // request, its unit
  int k0, k1;                          // steps of the piece
  Job j;
  Given g;                             // of the request behind, asked for ahead of its turn

  __device__ __forceinline__ void enter(const AttnParams& p, int b_, int64_t from, int64_t share) {
    b = b_;
    left = share;
    j = job_of<N>(p, b);
    g = given(p, b + 1);
    u = (int)(from / j.steps);
    k0 = (int)(from - (int64_t)u * j.steps);
    k1 = (int)min((int64_t)j.steps, k0 + left);
  }
  // the next piece; false at the end of the share
  __device__ __forceinline__ bool next(const AttnParams& p) {
    left -= k1 - k0;
    if (left <= 0) return false;
    if (++u == j.units) {
      u = 0;
      do {
        j = job_of<N>(p, g);
        g = given(p, ++b + 1);
      } while (j.cost() == 0);
    }
    k0 = 0;
    k1 = (int)min((int64_t)j.steps, left);
    return true;
  }
  __device__ __forceinline__ int head() const { return j.tiles == 1 ? u : u / j.tiles; }
  __device__ __forceinline__ int row0(int h) const { return (u - h * j.tiles) * N; }   // of the kv head's rows
  // keys that every row of the unit sees
  __device__ __forceinline__ int all_see(const AttnParams& p, int first) const { return j.len - j.n + first / p.G + 1; }
};

// A bounded wait in few instructions: one that runs out, or sees that another
// gave up, returns false. The site goes to shared memory and to the block's
// flags when it ends.
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
__device__ __forceinline__ bool spin_all(uint32_t bar, uint32_t parity, const Bound& w, uint32_t where) {
  const bool ok = spin(bar, parity, w, where);
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 u;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(a) : "memory");
  return u;
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar) : "memory");
}
// Two half floats as e4m3 codes (the low 16 bits).
__device__ __forceinline__ uint16_t e4m3x2_of_half2(uint32_t h) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c) : "r"(h));
  return c;
}
// 16 (p - c), for the codes c of p: exact.
__device__ __forceinline__ uint32_t rest16(uint32_t p, uint16_t codes) {
  uint32_t d;
  asm("{.reg .b32 t; sub.rn.f16x2 t, %1, %2; mul.rn.f16x2 %0, t, %3;}"
      : "=r"(d) : "r"(p), "r"(e4m3x2_to_half2(codes)), "r"(0x4c004c00u));
  return d;
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

// kind::f8f6f4, e4m3 both, fp32 accumulate.
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Shared-memory descriptor of rows of W bytes (128 or 64) in the swizzle of that
// width, groups of 8 rows; lbo: between pieces of W elements of an MN-major operand.
template <int W>
__device__ __forceinline__ uint64_t rows_desc(uint32_t saddr, uint32_t lbo) {
  const uint64_t d = sdesc_sw128(saddr, lbo, 8 * W);
  return W == 128 ? d : (d & ~((uint64_t)7 << 61)) | (uint64_t)4 << 61;
}
// Byte of 16-byte chunk c of row r in that layout.
template <int W>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  return W == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// Sums (or maxima) over the warp of 16 columns, of which every lane brings one
// value each: halve the columns lane bit by lane bit, then fold the lanes that
// are left. Returns the column that ends up in v[0] of this lane.
template <bool kMax>
__device__ __forceinline__ int fold16(float* v, int lane) {
  int col = 0;
#pragma unroll
  for (int o = 16, hf = 8; o > 1; o >>= 1, hf >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int n = 0; n < hf; ++n) {
      const float give = up ? v[n] : v[n + hf], keep = up ? v[n + hf] : v[n];
      const float got = __shfl_xor_sync(0xffffffffu, give, o);
      v[n] = kMax ? fmaxf(keep, got) : keep + got;
    }
    col += up ? hf : 0;
  }
  const float got = __shfl_xor_sync(0xffffffffu, v[0], 1);
  v[0] = kMax ? fmaxf(v[0], got) : v[0] + got;
  return col;
}

template <int D, int N>
struct Cfg {
  static constexpr int kCG = N / 16;                   // softmax warpgroups of a stream
  static constexpr int kST = 3 - kCG;                  // streams
  static constexpr int kThreads = 512;
  static constexpr int kCodes = kKeys * D;             // a tile of codes
  static constexpr int kK = D == 128 ? 5 : 8, kV = D == 128 ? 6 : 8;     // stages
  static constexpr int kQS = N == 16 ? 4 : 2;          // units of Q
  static constexpr int kQ = 2 * N * D;                 // both parts of a unit's rows
  static constexpr int kPW = N == 16 ? 64 : 128;       // bytes of a key's row of P (3N used)
  static constexpr int kP = kKeys * kPW;
  static constexpr int kE = kK + 4;                    // exponents of a step: 128 of K, 128 of V, hidden boxes
  static constexpr int kEBytes = 272;
  static constexpr int kTmem = 512;                    // S of the streams (2N each), O by unit and stream (3N)
  static constexpr int oV = kK * kCodes, oP = oV + kV * kCodes, oQ = oP + kST * kP, oE = oQ + kQS * kQ,
                       oW = oE + kE * kEBytes;
  // words
  static constexpr int wCq = 0;                        // [kQS][N] scale of a column's scores
  static constexpr int wLim = wCq + kQS * N;           // [kQS][N] keys that it sees
  static constexpr int wAt = wLim + kQS * N;           // [kQS][N] new row << 8 | query head of the group
  static constexpr int wR = wAt + kQS * N;             // [2][2][N] references for the epilogue, by unit and stream
  static constexpr int wL = wR + 4 * N;                // [2][2][4][N] sums of each softmax warp
  static constexpr int wMax = wL + 16 * N;             // [2][4][N] maxima of a step by stream and warp
  static constexpr int wRef = wMax + 8 * N;            // [2][4][N] a warp's copy of the references
  static constexpr int wAl = wRef + 8 * N;             // [2][4][N] ... of the factors of a move
  static constexpr int wWt = wAl + 8 * N;              // [4][2][N] an epilogue warp's weights of the streams
  static constexpr int wNf = wWt + 8 * N;              // [2][2] NaN taken out of V tiles, by unit and stream
  static constexpr int kWords = wNf + 4;
  static constexpr int oBar = oW + 4 * kWords;
  static constexpr int kSmem = oBar + 512 + 1024;
  static_assert(kSmem <= 232448, "shared memory");
  static_assert(4 * N + 12 * N <= 512, "tensor memory");
};

template <int D, int N>
__global__ void __launch_bounds__(Cfg<D, N>::kThreads, 1)
mis_q8_attn_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                   const __grid_constant__ AttnParams p) {
  using C = Cfg<D, N>;
  constexpr int CG = C::kCG, ST = C::kST, KS = C::kK, VS = C::kV, QS = C::kQS;
  // barriers
  constexpr int bQF = 0, bKF = bQF + QS, bKE = bKF + KS, bVF = bKE + KS, bVE = bVF + VS, bSF = bVE + VS, bPF = bSF + 2,
                bPV = bPF + 2, bOF = bPV + 2, bOE = bOF + 2, bST = bOE + 2, bSE = bST + 2, bDR = bSE + QS, nBar = bDR + 1;
  static_assert(nBar * 8 + 16 <= 512, "barrier space");
  griddep_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t base = smem_u32(smem);
  float* words = reinterpret_cast<float*>(smem + C::oW);
  uint32_t* sNf = reinterpret_cast<uint32_t*>(words + C::wNf);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::oBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + nBar);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  __shared__ int64_t s_sum[C::kThreads / 32];
  __shared__ int64_t s_from;
  __shared__ int s_req;
  __shared__ uint32_t s_bad;
  auto bar = [&](int i) { return smem_u32(bars + i); };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    *abort_flag = 0;
    s_bad = 0;
    for (int s = 0; s < 4; ++s) sNf[s] = 0;
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(bSF + s), 1);
      mbar_init(bar(bPF + s), 4 * CG);
      mbar_init(bar(bPV + s), 1);
      mbar_init(bar(bOF + s), 1);
      mbar_init(bar(bOE + s), 4);
      mbar_init(bar(bST + s), 4 * CG * ST);
    }
    for (int s = 0; s < QS; ++s) { mbar_init(bar(bQF + s), 1); mbar_init(bar(bSE + s), 4); }
    for (int s = 0; s < KS; ++s) { mbar_init(bar(bKF + s), 1); mbar_init(bar(bKE + s), 1); }
    for (int s = 0; s < VS; ++s) { mbar_init(bar(bVF + s), 1); mbar_init(bar(bVE + s), 1); }
    mbar_init(bar(bDR), 1);
    fence_mbar_init();
    fence_proxy_async();
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), C::kTmem);
    tmem_relinquish();
  }
  griddep_wait();

  // Every block adds up the steps of all requests, a run of them a thread, and
  // finds the request that its share starts in.
  const int run = (p.B + C::kThreads - 1) / C::kThreads;
  const int rb0 = min(p.B, tid * run), rb1 = min(p.B, rb0 + run);
  int64_t mine = 0;
  bool bad = false;
  for (int b = rb0; b < rb1; ++b) {
    const Job j = job_of<N>(p, b);
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
  tc_fence_before();
  bad = __syncthreads_or(bad);
  tc_fence_after();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < C::kThreads / 32; ++w) {
    if (w < warp) upto += s_sum[w];
    total += s_sum[w];
  }
  const int blocks = blocks_for(total, p.blocks);
  const int64_t share0 = total * min((int)blockIdx.x, blocks) / blocks;
  const int64_t share = total * min((int)blockIdx.x + 1, blocks) / blocks - share0;
  if (tid == 0) p.meta[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
  {
    int64_t at = upto - mine;
    const bool here = share0 >= at && share0 < upto;
    if (here)
      for (int b = rb0; b < rb1; ++b) {
        const int64_t next = at + job_of<N>(p, b).cost();
        if (share0 >= at && share0 < next) { s_req = b; s_from = share0 - at; }
        at = next;
      }
  }
  __syncthreads();
  const uint32_t tmem = *tmem_slot;
  const Bound W{abort_flag, p.wait_ns};
  const int box_shift = min(p.page_shift, 7);
  auto colS = [](int s) { return (uint32_t)(s * 2 * N); };
  auto colO = [](int unit, int stream) { return (uint32_t)(4 * N + (ST * unit + stream) * 3 * N); };

  if (share > 0) {
    Walk<N> w;
    w.enter(p, s_req, s_from, share);
    if (warp == 0 || warp == 3) {
      // ------------------------------------------------- copies of K (V): a lane a box of a page
      const bool y = warp == 3;
      const int depth = y ? VS : KS, full = y ? bVF : bKF, empty = y ? bVE : bKE;
      const uint32_t ring = base + (y ? C::oV : 0);
      // tiles of several row tiles are read again soon
      const uint64_t policy = w.j.tiles > 1 ? policy_normal() : policy_once();
      // a lane's copy of a step: its page, the step's first key and keys, the
      // head. Page ids are asked for A steps ahead (a trip to L2 each would be
      // longer than a step), and what goes by the unit is kept: the few
      // instructions of a step are a chain that bounds short ones
      constexpr int A = 3;
      struct Copy { int page, key, keys, h; };
      const int off = lane << box_shift, mask = (1 << p.page_shift) - 1;
      const uint32_t rows = 1u << box_shift, each = rows * (y ? D : D + 2);
      const uint32_t dst = ring + lane * (rows * D), edst = base + C::oE + lane * rows;
      const CUtensorMap* map = y ? &vmap : &kmap;
      bool more = true, bad_page = false;
      int k = w.k0, t = 0, issued = 0, h = w.head(), sl = 0, se = 0;
      uint32_t ph = 1;
      const int32_t* trow = p.table + (int64_t)w.b * p.table_stride;
      Copy q[A];
      auto ahead = [&]() -> Copy {
        Copy c{0, k * kKeys, 0, h};
        if (!more) return c;
        c.keys = w.j.len - k * kKeys;
        if (off < min(kKeys, c.keys)) c.page = trow[(c.key + off) >> p.page_shift];
        if (++k == w.k1) {
          more = w.next(p);
          k = w.k0;
          h = w.head();
          trow = p.table + (int64_t)w.b * p.table_stride;
        }
        return c;
      };
#pragma unroll
      for (int i = 0; i < A; ++i) q[i] = ahead();
#pragma unroll 1
      while (q[0].keys > 0) {
        const Copy cur = q[0];
#pragma unroll
        for (int i = 0; i + 1 < A; ++i) q[i] = q[i + 1];
        q[A - 1] = ahead();
        if (t >= depth && !spin_all(bar(empty + sl), ph, W, 0x100 + y)) break;
        bool want = off < min(kKeys, cur.keys);
        const bool lost = want && (uint32_t)cur.page >= (uint32_t)p.n_pages;
        const uint32_t hide = __ballot_sync(0xffffffffu, lost);
        want &= !lost;
        bad_page |= lost;
        if (lane == 0) {
          const int n = (min(kKeys, cur.keys) + (int)rows - 1) >> box_shift;
          if (!y) *reinterpret_cast<uint32_t*>(smem + C::oE + se * C::kEBytes + 256) = hide;
          mbar_arrive_expect_tx(bar(full + sl), each * (uint32_t)(n - __popc(hide)));
        }
        __syncwarp();
        if (want) {
          const int row = (cur.key + off) & mask;
          tma_load_4d(dst + sl * C::kCodes, map, bar(full + sl), 0, cur.h, row, cur.page, policy);
          if (!y) {
            const int64_t ex = (((int64_t)cur.page * p.Hkv + cur.h) << p.page_shift) + row;
            bulk_load(edst + se * C::kEBytes, p.ke + ex, rows, bar(full + sl));
            bulk_load(edst + se * C::kEBytes + 128, p.ve + ex, rows, bar(full + sl));
          }
        }
        issued = ++t;
        if (++sl == depth) { sl = 0; ph ^= 1; }
        if (++se == C::kE) se = 0;
      }
      __syncwarp();
      if (__any_sync(0xffffffffu, bad_page) && lane == 0) atomicOr(&s_bad, kDevIndex);
      // drain: every copy has landed before the block exits
      for (int i = max(0, issued - depth); i < issued; ++i) wait_drain(bar(full + i % depth), (i / depth) & 1);
    } else if (warp == 1) {
      // --------------------------------------------------------------- products
      constexpr uint32_t idS = (1u << 4) | ((uint32_t)(2 * N >> 3) << 17) | (8u << 24);
      constexpr uint32_t idO = (1u << 4) | (1u << 15) | (1u << 16) | ((uint32_t)(3 * N >> 3) << 17) | (8u << 24);
      bool ok = true;
      if (p.stall) ok = spin_all(bar(bDR), 0, W, 0x7ff);       // nothing arrives before the drain
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      // S runs two steps ahead: O of step t and S of step t + 2, which takes the
      // place of S of t, go out together once P of t is there. One wait a step
      // (a lane a barrier): this warp's own instructions are a long chain of a
      // short step. What it counts has to be uniform over the warp for the
      // compiler too (shuffled where it comes from memory): the products'
      // operands are uniform registers
      int sk = 0, sv = 0, sq = 0, lu = 0;              // slots of K, V and Q; units
      uint32_t pk = 0, pv = 0, pq = 0, pp = 0;         // phases of K, V, Q and (a bit a stream) P
      int ts = 0, to = 0;                              // steps whose S (O) has gone out
      struct Step { int kv, unit; uint32_t first, open, last; } st[2] = {};     // those between, by parity
      int k = 0, k0 = 0, k1 = 0, len = 0;
      bool have = ok;
      uint64_t qd = 0;
      auto enter = [&] {
        k = k0 = __shfl_sync(0xffffffffu, w.k0, 0);
        k1 = __shfl_sync(0xffffffffu, w.k1, 0);
        len = __shfl_sync(0xffffffffu, w.j.len, 0);
      };
      enter();
      auto scores = [&] {                              // by the elected lane
        const uint32_t d = tm + colS(ts & 1);
        const uint64_t a = rows_desc<D>(base + sk * C::kCodes, 0);
#pragma unroll
        for (int x = 0; x < D / 32; ++x) mma_e4m3(d, a + 2 * x, qd + 2 * x, idS, x != 0);
        mma_commit(bar(bSF + (ts & 1)));
        mma_commit(bar(bKE + sk));
      };
      auto counted = [&] {                             // S of a step has gone out
        const Step x{min(kKeys, len - k * kKeys), lu, k < k0 + ST, k == k0, k + 1 == k1};
        if (ts & 1) st[1] = x; else st[0] = x;
        ++ts;
        if (++sk == KS) { sk = 0; pk ^= 1; }
        if (++k == k1) {
          if (++sq == QS) { sq = 0; pq ^= 1; }
          ++lu;
          have = __shfl_sync(0xffffffffu, w.next(p), 0);
          if (have) enter();
        }
      };
      auto next_scores = [&]() -> bool {
        if (k == k0) {
          if (!spin_all(bar(bQF + sq), pq, W, 0x400)) return false;
          qd = rows_desc<D>(base + C::oQ + sq * C::kQ, 0);
        }
        if (!spin_all(bar(bKF + sk), pk, W, 0x401)) return false;
        tc_fence_after();
        if (elect_uniform()) scores();
        __syncwarp();
        counted();
        return true;
      };
      if (have) ok = next_scores();
      if (ok && have) ok = next_scores();
#pragma unroll 1
      while (ok && to < ts) {
        const Step x = to & 1 ? st[1] : st[0];
        const int s0 = ST == 2 ? to & 1 : 0;
        // O's place: the unit before the last must have been read out
        if (x.open && x.unit >= 2) ok = spin_all(bar(bOE + (x.unit & 1)), ((x.unit >> 1) - 1) & 1, W, 0x410);
        ok = ok && spin_all(lane & 1 ? bar(bVF + sv) : bar(bPF + s0), lane & 1 ? pv : (pp >> s0) & 1, W, 0x411);
        if (!ok) break;
        const bool both = have && k != k0 && __all_sync(0xffffffffu, mbar_test_wait(bar(bKF + sk), pk));
        tc_fence_after();
        // V [key][d] and P [key][part, row], both MN-major, 32 keys a product.
        // D = 64 repeats its 64 columns (stride 0): rows 64..127 of O^T equal
        // rows 0..63.
        const uint32_t d = tm + colO(x.unit & 1, s0);
        const uint64_t a = rows_desc<D>(base + C::oV + sv * C::kCodes, 0);
        const uint64_t b = rows_desc<C::kPW>(base + C::oP + s0 * C::kP, 0);
        const int nks = (x.kv + 31) >> 5;
        if (elect_uniform()) {
          mma_e4m3(d, a, b, idO, x.first ^ 1u);
          if (nks == kKeys / 32) {
#pragma unroll
            for (int y = 1; y < kKeys / 32; ++y) mma_e4m3(d, a + y * (2 * D), b + y * (2 * C::kPW), idO, 1u);
          } else {
#pragma unroll 1
            for (int y = 1; y < nks; ++y) mma_e4m3(d, a + y * (2 * D), b + y * (2 * C::kPW), idO, 1u);
          }
          mma_commit(bar(bPV + s0));
          if (x.last) mma_commit(bar(bOF + (x.unit & 1)));
          if (both) scores();
          mma_commit(bar(bVE + sv));
        }
        __syncwarp();
        if (++sv == VS) { sv = 0; pv ^= 1; }
        pp ^= 1u << s0;
        ++to;
        if (both) counted();
        else if (have) ok = next_scores();
      }
      // drain: all tensor-core work of the elected lane completes before dealloc
      if (elect_uniform()) mma_commit(bar(bDR));
      __syncwarp();
      wait_drain(bar(bDR), 0);
    } else if (warp == 2) {
      // ------------------------------------------------- Q and what its columns are
      // A row by D / 16 lanes, 16 elements each. Rows that are none keep what
      // was there: nobody reads their columns. The next unit's first rows come
      // while this one's are turned
      constexpr int LR = D / 16, RI = 32 / LR;
      const int c = lane % LR, n0 = lane / LR;
      int lu = 0;
      bool more = true;
      struct Rows { int h, first, rows, row0, see; };
      auto of = [&] {
        const int h = w.head(), first = w.row0(h);
        return Rows{h, first, min(N, w.j.n * p.G - first), w.j.row0, w.j.len - w.j.n + 1};
      };
      auto load = [&](const Rows& a, int n, uint4& x, uint4& y, int& at) {
        x = y = make_uint4(0u, 0u, 0u, 0u);
        at = 0;
        if (n >= a.rows) return;
        const int i = (a.first + n) / p.G, g = a.first + n - i * p.G;
        at = i << 8 | g;
        const uint4* src = reinterpret_cast<const uint4*>(p.q + (int64_t)(a.row0 + i) * p.qs + (int64_t)(a.h * p.G + g) * D + 16 * c);
        x = src[0];
        y = src[1];
      };
      Rows cur = of();
      uint4 x, y;
      int at;
      load(cur, n0, x, y, at);
      while (true) {
        const Rows a = cur;
        uint4 xa = x, ya = y;
        int ata = at;
        more = w.next(p);
        if (more) {
          cur = of();
          load(cur, n0, x, y, at);
        }
        const int sl = lu % QS;
        // what the unit before left there has been read
        if (lu >= QS && !spin_all(bar(bSE + sl), ((lu / QS) - 1) & 1, W, 0x200)) break;
#pragma unroll 1
        for (int n = n0; n - n0 < a.rows; n += RI) {
          if (n >= RI) load(a, n, xa, ya, ata);
          float f[16];
          bf16x8_to_float(xa, f);
          bf16x8_to_float(ya, f + 8);
          float m = 0.f;
#pragma unroll
          for (int e = 0; e < 16; ++e) m = fmaxf(m, fabsf(f[e]));
          m = row_max<LR>(m, 0xffffffffu);
          // m * 2^-ex in [128, 256); a row with infinities is NaN
          const int ex = m > 0.f ? max((__float_as_int(m) >> 23) - 127 - 7, -126) : 0;
          const float unit = m <= 3.4e38f ? pow2(-ex) : __int_as_float(0x7fffffff);
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float z[4], b[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) z[e] = f[4 * q + e] * unit;
            hi[q] = e4m3x4(z[0], z[1], z[2], z[3]);
            half2_to_float(e4m3x2_to_half2((uint16_t)hi[q]), b[0], b[1]);
            half2_to_float(e4m3x2_to_half2((uint16_t)(hi[q] >> 16)), b[2], b[3]);
#pragma unroll
            for (int e = 0; e < 4; ++e) z[e] = (z[e] - b[e]) * 32.f;
            lo[q] = e4m3x4(z[0], z[1], z[2], z[3]);
          }
          const uint32_t q0 = base + C::oQ + sl * C::kQ;
          if (n < a.rows) {
            st_shared_v4(q0 + chunk_at<D>(n, c), hi[0], hi[1], hi[2], hi[3]);
            st_shared_v4(q0 + N * D + chunk_at<D>(n, c), lo[0], lo[1], lo[2], lo[3]);
            if (c == 0) {
              words[C::wCq + sl * N + n] = pow2(min(ex, 127)) * p.scale_log2;
              reinterpret_cast<int*>(words)[C::wLim + sl * N + n] = a.see + (ata >> 8);
              reinterpret_cast<int*>(words)[C::wAt + sl * N + n] = ata;
            }
          }
        }
        if (lane >= a.rows && lane < N) {
          words[C::wCq + sl * N + lane] = 0.f;
          reinterpret_cast<int*>(words)[C::wLim + sl * N + lane] = 0;
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(bQF + sl));
        ++lu;
        if (!more) break;
      }
    } else if (warp < 12) {
      // --------------------------------------------------------------- softmax
      const int wg = (warp - 4) >> 2, str = wg / CG, cg = wg % CG, sw = warp & 3, r = sw * 32 + lane;
      const int c0 = cg * 16, id = 1 + wg;
      const uint32_t tl = tmem + ((uint32_t)(sw * 32) << 16);
      const uint32_t aP = base + C::oP + str * C::kP;
      float* ref = words + C::wRef + (str * 4 + sw) * N + c0;
      float* al = words + C::wAl + (str * 4 + sw) * N + c0;
      float* mx = words + C::wMax + str * 4 * N + c0;
      int t = 0, lu = 0;                               // steps of both streams, units
      bool ok = true, more = true, gone = false;
      while (more) {
        const int slot = lu & 1, sq = lu % QS, first_row = w.row0(w.head()), rows = w.j.n * p.G - first_row;
        const int len = w.j.len, see = w.all_see(p, first_row);
        ok = spin(bar(bQF + sq), (lu / QS) & 1, W, 0x700) &&
             (lu < 2 || spin(bar(bSE + (lu - 2) % QS), ((lu - 2) / QS) & 1, W, 0x701));
        // one vote of the warpgroup: all go on, or all leave
        if (bar_any128(id, !ok)) break;
        const float* cq = words + C::wCq + sq * N + c0;
        const int* lim = reinterpret_cast<const int*>(words) + C::wLim + sq * N + c0;
        uint64_t l2[8];
#pragma unroll
        for (int n = 0; n < 8; ++n) l2[n] = 0ull;
        bool first = true, nan = false;
        // the stream's steps: every other one of the share
        int k = w.k0;
        if (ST == 2 && ((t ^ str) & 1)) { ++k; ++t; }
#pragma unroll 1
        for (; k < w.k1; k += ST, t += ST) {
          const uint32_t before = (uint32_t)(t / ST - 1) & 1u, tS = tl + colS(t & 1) + c0;      // phase of its last product
          ok = spin_all(bar(bSF + (t & 1)), (t >> 1) & 1, W, 0x710);
          tc_fence_after();
          uint32_t s[16], x[16];
          if (ok) {
            tmem_ld16(tS, s);
            tmem_ld16(tS + N, x);
          }
          const uint8_t* e = smem + C::oE + (t % C::kE) * C::kEBytes;
          const uint32_t hide = *reinterpret_cast<const uint32_t*>(e + 256);
          const float kf = pow2(q8_exp(e[r]));
          const int ev = q8_exp(e[128 + r]);
          const float vs = pow2(ev - 26), most = 34.5f - (float)ev;
          const int key = k * kKeys + r;
          if (ok) {
            tmem_ld_wait();
            reg_fence16(s);
            reg_fence16(x);
          }
          // scores before the key's scale
          const uint64_t part = f2_pack(0x3d000000u, 0x3d000000u);       // 1/32
#pragma unroll
          for (int n = 0; n < 16; n += 4) {
            const float4 c = *reinterpret_cast<const float4*>(cq + n);
            float y0, y1, y2, y3;
            f2_unpack(f2_mul(f2_fma(f2_pack(x[n], x[n + 1]), part, f2_pack(s[n], s[n + 1])),
                             f2_pack(__float_as_uint(c.x), __float_as_uint(c.y))), y0, y1);
            f2_unpack(f2_mul(f2_fma(f2_pack(x[n + 2], x[n + 3]), part, f2_pack(s[n + 2], s[n + 3])),
                             f2_pack(__float_as_uint(c.z), __float_as_uint(c.w))), y2, y3);
            s[n] = __float_as_uint(y0); s[n + 1] = __float_as_uint(y1);
            s[n + 2] = __float_as_uint(y2); s[n + 3] = __float_as_uint(y3);
          }
          const bool plain = k * kKeys + kKeys <= see && !hide;
          const bool gone_key = key >= len || ((hide >> (r >> box_shift)) & 1u);
          if (!plain) {
#pragma unroll
            for (int n = 0; n < 16; ++n)
              if (gone_key || key >= lim[n]) s[n] = 0xff800000u;
          }
          auto weigh = [&] {                           // x = s * kf - r
            const uint64_t k2 = f2_pack(__float_as_uint(kf), __float_as_uint(kf));
#pragma unroll
            for (int n = 0; n < 16; n += 4) {
              const float4 c = *reinterpret_cast<const float4*>(ref + n);
              float y0, y1, y2, y3;
              f2_unpack(f2_fma(f2_pack(s[n], s[n + 1]), k2, f2_pack(__float_as_uint(-c.x), __float_as_uint(-c.y))), y0, y1);
              f2_unpack(f2_fma(f2_pack(s[n + 2], s[n + 3]), k2, f2_pack(__float_as_uint(-c.z), __float_as_uint(-c.w))), y2, y3);
              x[n] = __float_as_uint(y0); x[n + 1] = __float_as_uint(y1);
              x[n + 2] = __float_as_uint(y2); x[n + 3] = __float_as_uint(y3);
            }
          };
          bool over = !ok;
          if (!first) {
            weigh();
            float z = -INFINITY;
#pragma unroll
            for (int n = 0; n < 16; n += 2) z = max3(z, __uint_as_float(x[n]), __uint_as_float(x[n + 1]));
            over |= z > most;
            over = bar_any128(id, over);
          }
          if (first || over) {
            // a unit begins or a weighted value passed its reference (or a wait
            // gave up: then every warp of the warpgroup leaves here)
            if (bar_any128(id, !ok)) { gone = true; break; }
            {
              float v[16];
#pragma unroll
              for (int n = 0; n < 16; ++n) v[n] = fmaf(__uint_as_float(s[n]), kf, (float)(ev - 32));
              const int n = fold16<true>(v, lane);
              mx[sw * N + n] = v[0];
            }
            bar_sync128(id);
            // every warp draws the same conclusion from the four warps' maxima
            if (lane < 16) {
              const float old = first ? kNone : ref[lane];
              float to = old;
#pragma unroll
              for (int q = 0; q < 4; ++q) to = fmaxf(to, mx[q * N + lane]);
              if (c0 + lane >= rows) to = kDead;
              al[lane] = to > old ? ex2(old - to) : 1.f;
              ref[lane] = to;
            }
            __syncwarp();
            if (!first) {
              ok = spin_all(bar(bPV + str), before, W, 0x730);    // O holds every step before
              tc_fence_after();
              if (ok) {
#pragma unroll 1
                for (int q = 0; q < 3; ++q) {
                  const uint32_t tO = tl + colO(slot, str) + q * N + c0;
                  tmem_ld16(tO, x);
                  tmem_ld_wait();
                  reg_fence16(x);
#pragma unroll
                  for (int n = 0; n < 16; ++n) x[n] = __float_as_uint(__uint_as_float(x[n]) * al[n]);
                  tmem_st16(tO, x);
                }
                tmem_st_wait();
#pragma unroll
                for (int n = 0; n < 8; ++n)
                  l2[n] = f2_mul(l2[n], f2_pack(__float_as_uint(al[2 * n]), __float_as_uint(al[2 * n + 1])));
              }
            }
            weigh();
          }
          first = false;
          uint32_t part3[3][4];
          const uint64_t v2 = f2_pack(__float_as_uint(vs), __float_as_uint(vs));
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            uint32_t lo[3], hi[3];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int i = 4 * n + 2 * y;
              const uint64_t w2 = f2_pack(__float_as_uint(ex2(__uint_as_float(x[i]))),
                                          __float_as_uint(ex2(__uint_as_float(x[i + 1]))));
              l2[i / 2] = f2_add(l2[i / 2], w2);
              float p0, p1;
              f2_unpack(f2_mul(w2, v2), p0, p1);
              const uint32_t h = half2_of(p0, p1);
              const uint16_t a = e4m3x2_of_half2(h);
              const uint32_t h1 = rest16(h, a);
              const uint16_t b = e4m3x2_of_half2(h1);
              const uint16_t c = e4m3x2_of_half2(rest16(h1, b));
              (y ? hi : lo)[0] = a;
              (y ? hi : lo)[1] = b;
              (y ? hi : lo)[2] = c;
            }
#pragma unroll
            for (int q = 0; q < 3; ++q) part3[q][n] = __byte_perm(lo[q], hi[q], 0x5410);
          }
          if (ok && t >= ST) ok = spin_all(bar(bPV + str), before, W, 0x740);   // its last P has been read
          if (ok) {
#pragma unroll
            for (int q = 0; q < 3; ++q)
              st_shared_v4(aP + chunk_at<C::kPW>(r, q * CG + cg), part3[q][0], part3[q][1], part3[q][2], part3[q][3]);
            // V rows that nobody sees hold anything; NaN that only some rows see
            // is left to the epilogue (0 x NaN would reach all)
            if (!plain && cg == 0 && r < ((len - k * kKeys + 31) & ~31) && (gone_key || key >= see)) {
              const int sv = t % VS;
              ok = spin(bar(bVF + sv), (t / VS) & 1, W, 0x750);
              const uint32_t row = base + C::oV + sv * C::kCodes;
#pragma unroll 1
              for (int c = 0; c < D / 16 && ok; ++c) {
                const uint32_t at = row + chunk_at<D>(r, c);
                uint4 u = lds16(at);
                uint32_t* y = reinterpret_cast<uint32_t*>(&u);
                uint32_t any = 0;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  const uint32_t nn = nan_codes(y[q]);
                  any |= nn;
                  y[q] = gone_key ? 0u : y[q] & ~((nn >> 7) * 0xffu);
                }
                if (gone_key || any) st_shared_v4(at, u.x, u.y, u.z, u.w);
                nan |= any && !gone_key;
              }
            }
            ok = __all_sync(0xffffffffu, ok);
          }
          fence_proxy_async();
          tc_fence_before();
          __syncwarp();
          if (ok && lane == 0) mbar_arrive(bar(bPF + str));
        }
        if (gone) break;
        t += w.k1 - k;                                 // the next unit's first step
        // the columns' sums over this warp's keys
        float l[16];
#pragma unroll
        for (int n = 0; n < 8; ++n) f2_unpack(l2[n], l[2 * n], l[2 * n + 1]);
        const int col = fold16<false>(l, lane);
        words[C::wL + ((slot * 2 + str) * 4 + sw) * N + c0 + col] = l[0];
        if (sw == 0 && lane < 16) words[C::wR + (slot * 2 + str) * N + c0 + lane] = first ? kNone : ref[lane];
        if (cg == 0 && __any_sync(0xffffffffu, nan) && lane == 0) sNf[slot * 2 + str] = 1u + (uint32_t)lu;
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(bar(bST + slot));
        ++lu;
        more = w.next(p);
      }
    } else {
      // -------------------------------------------------------------- epilogue
      const int sw = warp & 3;
      const uint32_t tl = tmem + ((uint32_t)(sw * 32) << 16);
      // D = 128: a lane is element d, all columns. D = 64: the two copies of
      // O^T share the columns.
      const int d = (D == 128 ? sw * 32 : (sw & 1) * 32) + lane;
      constexpr int NE = D == 128 ? N : N / 2, CH = 8;
      const int e0 = D == 128 ? 0 : (sw >> 1) * NE;
      int lu = 0, t = 0;
      bool ok = true, more = true;
      while (more) {
        const int slot = lu & 1, h = w.head(), first = w.row0(h), rows = min(N, w.j.n * p.G - first);
        const bool whole = w.k0 == 0 && w.k1 == w.j.steps;
        ok = spin_all(bar(bST + slot), (lu >> 1) & 1, W, 0x800);
        if (!ok) break;
        const int piece = 2 * blockIdx.x + (lu ? 1 : 0), sq = lu % QS;
        // weights of the two streams' accumulators (zero: the unit had no step there)
        float* wt = words + C::wWt + sw * 2 * N;
        float mx = kNone, sum = 0.f;
        if (lane < N) {
          const float* l0 = words + C::wL + slot * 8 * N + lane;
          const float* l1 = l0 + (ST - 1) * 4 * N;
          const float r0 = words[C::wR + slot * 2 * N + lane], r1 = ST == 2 ? words[C::wR + (slot * 2 + 1) * N + lane] : kNone;
          mx = fmaxf(r0, r1);
          const float a0 = ex2(r0 - mx), a1 = ex2(r1 - mx);
          sum = a0 * ((l0[0] + l0[N]) + (l0[2 * N] + l0[3 * N]));
          if (ST == 2) sum += a1 * ((l1[0] + l1[N]) + (l1[2 * N] + l1[3 * N]));
          // the products' weights carry 2^-26; NaN stays
          const float inv = whole ? (sum != 0.f ? 67108864.f / sum : 0.f) : 1.f;
          wt[lane] = a0 * inv;
          wt[N + lane] = a1 * inv;
        }
        if (sw == 0 && lane == 0 && !whole && w.k0 == 0) {
          // the block that holds its last step
          const int64_t last = share0 + share + w.j.steps - w.k1 - 1;
          int c = (int)(last * blocks / total);
          while (total * (c + 1) / blocks <= last) ++c;
          while (total * c / blocks > last) --c;
          p.meta[2 * blockIdx.x] = make_int4(c - (int)blockIdx.x + 1, rows, h, first);
          p.meta[2 * blockIdx.x + 1] = make_int4(w.j.row0, lu ? 1 : 0, 0, 0);
        }
        const int* at = reinterpret_cast<const int*>(words) + C::wAt + sq * N;
        const int* lim = reinterpret_cast<const int*>(words) + C::wLim + sq * N;
        if (sw == 0 && lane < rows) {
          if (!whole)
            p.rl[(int64_t)piece * N + lane] = make_float2(mx, sum);
          else if (p.lse)
            p.lse[(int64_t)(h * p.G + (at[lane] & 255)) * p.T + w.j.row0 + (at[lane] >> 8)] =
                sum != 0.f ? (mx + log2f(sum)) * kLn2 : -INFINITY;
        }
        __syncwarp();
        ok = spin_all(bar(bOF + slot), (lu >> 1) & 1, W, 0x810);
        if (!ok) break;
        tc_fence_after();
        const bool nf = sNf[slot * 2] == 1u + (uint32_t)lu || (ST == 2 && sNf[slot * 2 + 1] == 1u + (uint32_t)lu);
        // streams that had a step: both, or the one of a single step
        const bool use0 = ST == 1 || w.k1 - w.k0 > 1 || !(t & 1), use1 = ST == 2 && (w.k1 - w.k0 > 1 || (t & 1));
        t += w.k1 - w.k0;
        // the columns in use; what no row needs is given back unread
        const int used = min(NE, rows - e0);
        if (used <= 0) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(bOE + slot));
        }
#pragma unroll 1
        for (int q = 0; q < used; q += CH) {
          float ov[CH];
#pragma unroll
          for (int n = 0; n < CH; ++n) ov[n] = 0.f;
          uint32_t y[ST][3][CH];                       // the parts of the streams' accumulators
#pragma unroll
          for (int i = 0; i < 3 * ST; ++i) tmem_ld8(tl + colO(slot, i / 3) + (i % 3) * N + e0 + q, y[i / 3][i % 3]);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 3 * ST; ++i) reg_fence8(y[i / 3][i % 3]);
          auto add = [&](int stream) {
#pragma unroll
            for (int n = 0; n < CH; ++n) {
              const float x = fmaf(__uint_as_float(y[stream][2][n]), 0.00390625f,
                                   fmaf(__uint_as_float(y[stream][1][n]), 0.0625f, __uint_as_float(y[stream][0][n])));
              ov[n] = fmaf(wt[stream * N + e0 + q + n], x, ov[n]);
            }
          };
          if (use0) add(0);
          if constexpr (ST == 2) {
            if (use1) add(1);
          }
          if (q + CH >= used) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(bOE + slot));
          }
          if (nf) {
            // NaN of the newest rows' values, for the rows that see them
#pragma unroll 1
            for (int key = max(w.k0 * kKeys, w.all_see(p, first)); key < min(w.k1 * kKeys, w.j.len); ++key) {
              const int page = p.table[(int64_t)w.b * p.table_stride + (key >> p.page_shift)];
              if (page < 0 || page >= p.n_pages) continue;
              const uint8_t code = p.v[(int64_t)page * p.page_stride +
                                       (int64_t)(key & ((1 << p.page_shift) - 1)) * p.row_stride +
                                       (int64_t)h * p.head_stride + d];
              if ((code & 0x7f) != 0x7f) continue;
#pragma unroll
              for (int n = 0; n < CH; ++n)
                if (key < lim[e0 + q + n]) ov[n] = __int_as_float(0x7fffffff);
            }
            __syncwarp();
          }
          if (!whole) {
            float* dst = p.part + ((int64_t)piece * N + e0 + q) * D + d;
#pragma unroll
            for (int n = 0; n < CH; ++n)
              if (e0 + q + n < rows) dst[n * D] = ov[n];
            continue;
          }
          // neighbours exchange one of two rows: an even lane stores elements
          // d, d + 1 of row n, the odd one d - 1, d of row n + 1
          const bool odd = lane & 1;
#pragma unroll
          for (int n = 0; n < CH; n += 2) {
            // a row that saw nothing has no weight and no sum
            const float other = __shfl_xor_sync(0xffffffffu, odd ? ov[n] : ov[n + 1], 1);
            const int c = e0 + q + n + (odd ? 1 : 0);
            if (c < rows) {
              const uint32_t u = odd ? pack_bf16(other, ov[n + 1]) : pack_bf16(ov[n], other);
              *reinterpret_cast<uint32_t*>(p.o + (int64_t)(w.j.row0 + (at[c] >> 8)) * p.os +
                                           (int64_t)(h * p.G + (at[c] & 255)) * D + (d & ~1)) = u;
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(bSE + sq));
        ++lu;
        more = w.next(p);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0) {
    p.flags[2 * blockIdx.x] = s_bad | (bad ? kDevIndex : 0u) | (*abort_flag ? kDevTimeout : 0u);
    p.flags[2 * blockIdx.x + 1] = *abort_flag ? *abort_flag : 0x60u;
  }
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
}

// Joins the pieces of a unit that several blocks hold, in block order: a block of
// four warps a row of the unit that starts in block blockIdx.x, the warps taking
// the pieces in turn. What it needs lies in one place, since its time is that of
// the trips to L2 it makes one behind the other (found by bisection of the
// requests' steps: 10 us for 64 decoded tokens).
template <int D, int N>
__global__ void __launch_bounds__(32 * kJoinWarps)
mis_q8_join_kernel(const __grid_constant__ AttnParams p) {
  constexpr int E = D / 32;
  __shared__ float s_acc[kJoinWarps][D + 1];
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x, n = blockIdx.y;
  const int4 u = p.meta[2 * c], v = p.meta[2 * c + 1];
  if (c == 0 && n == 0 && warp == 0) {
    uint32_t f = 0, where = 0;
    for (int x = lane; x < p.blocks; x += 32) {
      const uint32_t y = p.flags[2 * x];
      if (y && !f) where = p.flags[2 * x + 1];
      f |= y;
    }
    const uint32_t any = __ballot_sync(0xffffffffu, f != 0);
    where = __shfl_sync(0xffffffffu, where, any ? __ffs(any) - 1 : 0);
    f = __reduce_or_sync(0xffffffffu, f);
    if (lane == 0) {
      p.status[0] = f;
      p.status[1] = where;
    }
  }
  const int pieces = u.x;
  if (pieces < 2 || n >= u.y) return;
  // the first piece lies in block c's first or second slot, the others in the
  // first slots of the blocks that follow
  auto at = [&](int y) { return (int64_t)(2 * (c + y) + (y == 0 ? v.y : 0)) * N + n; };
  float acc[E], sum = 0.f, m = kNone;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  bool stuck = false;
  for (int y = lane; y < pieces; y += 32) {
    m = fmaxf(m, p.rl[at(y)].x);
    stuck |= (p.flags[2 * (c + y)] & kDevTimeout) != 0;
  }
  if (__any_sync(0xffffffffu, stuck)) return;          // a piece is missing: every warp sees it
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll 4
  for (int y = warp; y < pieces; y += kJoinWarps) {
    const float2 rl = p.rl[at(y)];
    const float f1 = ex2(rl.x - m);
    sum += f1 * rl.y;
    const float* z = p.part + at(y) * D + lane * E;
    if constexpr (E == 4) {
      const float4 z4 = *reinterpret_cast<const float4*>(z);
      acc[0] += f1 * z4.x; acc[1] += f1 * z4.y; acc[2] += f1 * z4.z; acc[3] += f1 * z4.w;
    } else {
      const float2 z2 = *reinterpret_cast<const float2*>(z);
      acc[0] += f1 * z2.x; acc[1] += f1 * z2.y;
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) s_acc[warp][e * 32 + lane] = acc[e];
  if (lane == 0) s_acc[warp][D] = sum;
  __syncthreads();
  if (warp) return;
  for (int y = 1; y < min(kJoinWarps, pieces); ++y) {
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] += s_acc[y][e * 32 + lane];
    sum += s_acc[y][D];
  }
  const int i = (u.w + n) / p.G, head = u.z * p.G + u.w + n - i * p.G;
  // the products' weights carry 2^-26
  const float inv = sum != 0.f ? 67108864.f / sum : 0.f;
  uint32_t out[E / 2];
#pragma unroll
  for (int e = 0; e < E / 2; ++e) out[e] = sum != 0.f ? pack_bf16(acc[2 * e] * inv, acc[2 * e + 1] * inv) : 0u;
  __nv_bfloat16* dst = p.o + (int64_t)(v.x + i) * p.os + (int64_t)head * D + lane * E;
  if constexpr (E == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
  else *reinterpret_cast<uint32_t*>(dst) = out[0];
  if (p.lse && lane == 0)
    p.lse[(int64_t)head * p.T + v.x + i] = sum != 0.f ? (m + log2f(sum)) * kLn2 : -INFINITY;
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
  // a request's units are counted in 32 bits
  if ((int64_t)d->max_rows * d->Hq > 0x7fffffff) return MIS_ERR_UNSUPPORTED;
  return MIS_OK;
}

int head_rows(const mis_paged_attn_desc* d, const mis_paged_cache_q8* c) { return d->max_rows * (d->Hq / c->Hkv); }

// Rows of a unit. More than 32 rows of a kv head are several units over the same
// keys.
int unit_rows(const mis_paged_attn_desc* d, const mis_paged_cache_q8* c) { return head_rows(d, c) <= 16 ? 16 : 32; }

struct AttnWs { size_t flags, meta, rl, part, total; };

AttnWs workspace_of(const mis_paged_attn_desc* d, const mis_paged_cache_q8* c) {
  const size_t G = (size_t)num_sms(), N = unit_rows(d, c);
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  AttnWs w;
  w.flags = kStatusBytes;
  w.meta = w.flags + up(G * 8);
  w.rl = w.meta + up(G * 2 * sizeof(int4));
  w.part = w.rl + up(2 * G * N * sizeof(float2));
  w.total = w.part + 2 * G * N * (size_t)c->D * sizeof(float);
  return w;
}

template <int D, int N>
mis_status_t launch(const CUtensorMap& km, const CUtensorMap& vm, const AttnParams& p, cudaStream_t st) {
  using C = Cfg<D, N>;
  auto kern = mis_q8_attn_kernel<D, N>;
  if (!kernel_attr_once(reinterpret_cast<const void*>(kern), C::kSmem)) return MIS_ERR_CUDA;
  if (launch_pdl(kern, dim3((unsigned)p.blocks), dim3(C::kThreads), C::kSmem, st, km, vm, p) != cudaSuccess)
    return MIS_ERR_CUDA;
  return launch_pdl(mis_q8_join_kernel<D, N>, dim3((unsigned)p.blocks, N), dim3(32 * kJoinWarps), 0, st, p) == cudaSuccess
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
  p.wait_ns = wait_limit_ns();
  p.stall = inject_stall_mask() & 1u;
  p.scale_log2 = (desc->scale != 0.f ? desc->scale : 1.f / std::sqrt((float)D)) * 1.4426950408889634f;
  p.status = reinterpret_cast<uint32_t*>(base);
  p.flags = reinterpret_cast<uint32_t*>(base + ws.flags);
  p.meta = reinterpret_cast<int4*>(base + ws.meta);
  p.rl = reinterpret_cast<float2*>(base + ws.rl);
  p.part = reinterpret_cast<float*>(base + ws.part);
  try {
    // the cache as (code, head, row, page), boxes of the rows of a page (128 at
    // most). Strides of extents of one are never used, but have to be valid.
    bool ok = true;
    const uint64_t dims[4] = {(uint64_t)D, (uint64_t)cache->Hkv, (uint64_t)cache->page_size, (uint64_t)cache->n_pages};
    auto stride = [&](int64_t s, int64_t extent) { return (uint64_t)(extent > 1 ? s : D); };
    const uint64_t strides[3] = {stride(cache->head_stride, cache->Hkv), stride(cache->row_stride, cache->page_size),
                                 stride(cache->page_stride, cache->n_pages)};
    const uint32_t box[4] = {(uint32_t)D, 1, (uint32_t)std::min(cache->page_size, kKeys), 1};
    const CUtensorMap km = encode_tmap_u8(cache->k, 4, dims, strides, box, &ok);
    const CUtensorMap vm = encode_tmap_u8(cache->v, 4, dims, strides, box, &ok);
    if (!ok) return MIS_ERR_CUDA;
    const int N = unit_rows(desc, cache);
    if (D == 128) return N == 16 ? launch<128, 16>(km, vm, p, st) : launch<128, 32>(km, vm, p, st);
    return N == 16 ? launch<64, 16>(km, vm, p, st) : launch<64, 32>(km, vm, p, st);
  } catch (...) {
    return MIS_ERR_CUDA;
  }
}
