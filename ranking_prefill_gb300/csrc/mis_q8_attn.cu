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
// with N = 16 or 32 rows a tile, all of it in 8 bits: K and V go from the cache to
// the tensor core as they lie there, and what the softmax computes anyway is
// what gets split. Q's parts are its leading 4 bits and 32 times the rest, both
// e4m3, in units of a power of two of each row: exact for bf16 elements down to
// 2^-14 of the row's largest, within 2^-22 of that below. P is rounded to fp16 and
// split into its nearest e5m2, 16 times what is left, 16 times what that leaves:
// exact for every fp16 up to 2^15, subnormals too (a code has 3 bits, so its rest is
// a bit and more shorter than what is below them: 11, 7, 3 bits). The largest
// weight of a row lies in [2^11, 2^15], so one keeps 11 bits down to 2^-25 of it and
// is within 2^-36 of it below that (values above 2^118: weights below 2^-26 are
// zero, 2^(s - r) having left fp32). Three e4m3 parts, at the same times, lost bits
// from 2^-13 on and all below 2^-24, which the sum of the weights kept: 131,072 keys
// 2^-24.6 of one more left o 0.5% off. What stays is the tensor core's: products
// are added in fp32 and cut some 25 bits below the sum, so n weights that small
// beside one lose up to n 2^-25 of its value (1M of 2^-26 beside one of the same
// value in one block: o 1.1% off). The parts' products stand in columns of their
// own and are added when they are read.
// (V converted to fp16 by a warpgroup of its own and P in one part took 64 decoded
// tokens over 512 to 4096 rows 74 us and 4 requests of 117K rows 224; mma.sync with
// K and V converted in registers 73 and 270; this form took 57 and 178 before the
// steps noted below, 51 to 56 and 161 to 170 with them, by the GPU.)
//
// What bounds it: the K/V stream in long caches (4 single tokens over 65K to 131K
// rows 146 to 168 us, 5.7 to 6.6 TB/s where a copy reaches 6.7; 5.1 to 5.5 at 64 x
// 2.2K rows, which lose 6 us before the first product and 5 in the join); the
// softmax's chain of a step where a unit has more than 16 rows (1,700 cycles for the
// 32 KB of K and V that HBM brings in 1,440: 32 requests of 64 rows a kv head 86 us,
// their stream 21; of 128 155, of 256 288, every 32 rows walking the keys again); the
// same chain at D = 64, where a step brings half the bytes (64 tokens over 512 to 8192
// rows 75 us, their stream 40); what a unit takes to begin and end where it has a few
// steps (256 requests of 100 to 600 rows 68 us, their stream 27); the chain of one step
// and the second launch in small batches (4 requests of 100 to 300 rows 10.3 us).
//
// A row's key scale multiplies its score, its value scale its probability. The
// softmax keeps two things per row: a reference r below which weights are
// taken, and l = sum 2^(s - r). Products use P = 2^(s - r + e_v - 9): r is the
// largest s + e_v - 20 seen, moved only when one passes it by 2^4, so P stays below
// 2^15 (where 16 times the rests stay within e5m2) and its largest above 2^11,
// whatever the spread of the value scales. 2^(s - r) lies between 2^-100 and 2^80
// for the largest of every e_v in [-56, 120], with room in fp32 for sums and for
// what adds 24 bits below; s - r is about 20 - e_v, rounded at that size. r can move
// by more than fp32's exponents hold (a row of zeros, e_v = -56, and one of 2^80
// behind it): l of before, 2^76 a key, then still counts, so its factor is taken as
// a root that multiplies twice. What O held is 2^-126 of what comes and may go.
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
// Steps whose scores may be out, as many places of S (3 of them: units of 16 rows
// 36.3 us instead of 35.5, 4 long requests of 32 rows a kv head 191 instead of 187).
constexpr int kAhead = 4;
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
  int32_t n_pages, page_shift, most;       // most: rows that a table row can name
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

// What steps and units count in a block's share, so that shares take alike: a
// step in two streams kStep, one of more rows than that kWide; a unit what its
// beginning and end take besides. 4 long requests of 12 to 32 rows a kv head 180 us,
// with kWide = kStep 194 (requests of 64 rows alone, whose shares that leaves alike,
// 87 and 85.5). With kUnit and kUnitWide zero: requests of 64 rows 111 us instead of
// 87, units of 16 rows 36.6 and 35.5, 256 short requests 68.2 and 67.6. Where blocks
// have few steps each the longest share is what counts, and that is one step: there
// a step counts kStep and a unit nothing (5 small requests 11.6 us, otherwise 14.6).
constexpr int kStep = 4, kWide = 5, kUnit = 8, kUnitWide = 20;

// A request's work: units of N of a kv head's n * G rows, the tiles of a head
// side by side.
struct Job {
  int len, row0, n;                    // cached rows; first new row, new rows
  int steps, tiles, units;             // 128-key steps of a unit
  int step, own;                       // what one counts, and a unit besides
  bool ok;
  // what a unit counts, and all of them; the host bounds the sum
  __device__ __forceinline__ int unit() const { return steps * step + own; }
  __device__ __forceinline__ int cost() const { return unit() * units; }
};

// What a request brings, as read.
struct Given { int len, row0, end; };
__device__ __forceinline__ Given given(const AttnParams& p, int b) {
  return b < p.B ? Given{p.cache_len[b], p.cu[b], p.cu[b + 1]} : Given{0, 0, 0};
}
template <int N>
__device__ __forceinline__ Job job_of(const AttnParams& p, const Given& g, bool big) {
  Job j;
  j.len = g.len;
  j.row0 = g.row0;
  j.ok = j.row0 >= 0 && g.end >= j.row0 && g.end <= p.T && g.end - j.row0 <= p.max_rows && j.len >= 0 &&
         j.len <= p.most && g.end - j.row0 <= j.len;
  j.n = j.ok ? g.end - j.row0 : 0;
  j.steps = (uint32_t)(j.len + kKeys - 1) / kKeys;
  j.tiles = (uint32_t)(j.n * p.G + N - 1) / N;
  j.units = j.tiles * p.Hkv;
  const bool wide = N > 16 && j.n * p.G > 16;
  j.step = big && wide ? kWide : kStep;
  j.own = big ? (wide ? kUnitWide : kUnit) : 0;
  return j;
}

// A block's share: [from, from + size) of all units laid end to end; blocks
// [0, rem) take quo + 1, the others quo. So few take part that a share holds a
// unit's own cost and a step (`least`).
struct Share {
  int quo, rem, from, size;
  __device__ __forceinline__ Share(int total, int blocks, int b, int least) {
    if (total < blocks * least) blocks = max(1u, (uint32_t)total / (uint32_t)least);
    quo = (uint32_t)total / (uint32_t)blocks;
    rem = total - quo * blocks;
    from = b * quo + min(b, rem);
    size = b < blocks ? quo + (b < rem ? 1 : 0) : 0;
  }
  __device__ __forceinline__ int holder(int at) const {
    const int cut = rem * (quo + 1);
    return at < cut ? (uint32_t)at / (uint32_t)(quo + 1) : rem + (uint32_t)(at - cut) / (uint32_t)quo;
  }
};

// Walks the pieces of units that a block's share holds. A step is in the share
// that holds the last of what it counts.
template <int N>
struct Walk {
  int left, off;                       // of the share from this piece on; of the unit before it
  bool big;
  int b, u;                            // request, its unit
  int k0, k1;                          // steps of the piece
  Job j;
  Given g;                             // of the request behind, asked for ahead of its turn

  // the first piece; false where the share has none
  __device__ __forceinline__ bool enter(const AttnParams& p, int b_, int from, int share, bool big_) {
    b = b_;
    left = share;
    big = big_;
    j = job_of<N>(p, given(p, b), big);
    g = given(p, b + 1);
    u = (uint32_t)from / (uint32_t)j.unit();
    off = from - u * j.unit();
    k0 = (uint32_t)off / (uint32_t)j.step;
    if (k0 >= j.steps) return next(p);
    k1 = min(j.steps, (int)((uint32_t)(off + left) / (uint32_t)j.step));
    return k1 > k0;
  }
  // the next piece; false at the end of the share
  __device__ __forceinline__ bool next(const AttnParams& p) {
    left -= j.unit() - off;
    if (left < kStep) return false;
    off = 0;
    if (++u == j.units) {
      u = 0;
      do {
        j = job_of<N>(p, g, big);
        g = given(p, ++b + 1);
      } while (j.units == 0);
    }
    k0 = 0;
    k1 = min(j.steps, (int)((uint32_t)left / (uint32_t)j.step));
    return k1 > 0;
  }
  // the end of the unit's steps, counted from the piece on
  __device__ __forceinline__ int ahead() const { return j.steps * j.step - off; }
  __device__ __forceinline__ int head() const { return j.tiles == 1 ? u : (int)((uint32_t)u / (uint32_t)j.tiles); }
  __device__ __forceinline__ int row0(int h) const { return (u - h * j.tiles) * N; }   // of the kv head's rows
  // keys that every row of the unit sees
  __device__ __forceinline__ int all_see(const AttnParams& p, int first) const { return j.len - j.n + (first ? first / p.G : 0) + 1; }
};

// A bounded wait in few instructions: one that runs out, or sees that another
// gave up, returns false. The site goes to shared memory and to the block's
// flags when it ends.
struct Bound {
  volatile uint32_t* gave_up;
  uint64_t limit_ns;
};
static __device__ __noinline__ bool spin_on(uint32_t bar, uint32_t parity, volatile uint32_t* gave_up,
                                            uint64_t limit_ns, uint32_t where) {
  const uint64_t t0 = globaltimer();
  do {
    if (mbar_try_wait(bar, parity)) return true;
    if (*gave_up) return false;
  } while (globaltimer() - t0 <= limit_ns);
  *gave_up = where;
  return false;
}
__device__ __forceinline__ bool spin(uint32_t bar, uint32_t parity, const Bound& w, uint32_t where) {
  return mbar_try_wait(bar, parity) || spin_on(bar, parity, w.gave_up, w.limit_ns, where);
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
// Two half floats as e5m2 codes (the low 16 bits), to the nearest.
__device__ __forceinline__ uint16_t e5m2x2_of_half2(uint32_t h) {
  uint16_t c;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(c) : "r"(h));
  return c;
}
// 16 (p - c), for the codes c of p (a code is the upper byte of its half float): exact.
__device__ __forceinline__ uint32_t rest(uint32_t p, uint16_t codes) {
  uint32_t d;
  asm("{.reg .b32 t; sub.rn.f16x2 t, %1, %2; mul.rn.f16x2 %0, t, %3;}"
      : "=r"(d) : "r"(p), "r"(__byte_perm(codes, 0u, 0x1404)), "r"(0x4c004c00u));
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

// kind::f8f6f4, fp32 accumulate.
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
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

// ln(sum * 2^r), 2^20 taken out of the sum: near 1 the logarithm's bits are finest
__device__ __forceinline__ float lse_of(float r, float sum) {
  return ((r + 20.f) + log2f(sum * 9.5367431640625e-7f)) * kLn2;
}

template <int D, int N>
struct Cfg {
  static constexpr int kThreads = 512;
  static constexpr int kCodes = kKeys * D;             // a tile of codes
  // Stages, 64 KB of K and of V. More in flight than that and HBM reads slower: with
  // 80 and 96 KB 4 single tokens over 65K to 131K rows take 180 us instead of 166 (on
  // another GPU 160 and 146), with 48 and 48 148, with 32 and 48 166.
  static constexpr int kK = D == 128 ? 4 : 8, kV = kK;
  static constexpr int kQS = N == 16 ? 4 : 2;          // units of Q
  static constexpr int kQ = 2 * N * D;                 // both parts of a unit's rows
  static constexpr int kPW = N == 16 ? 64 : 128;       // bytes of a key's row of P (3N used)
  static constexpr int kP = kKeys * kPW;
  static constexpr int kE = kK + 4;                    // exponents of a step: 128 of K, 128 of V, hidden boxes
  static constexpr int kEBytes = 272;
  static constexpr int kTmem = 512;                    // S of kAhead steps (2N each), O by unit (96)
  static constexpr int oV = kK * kCodes, oP = oV + kV * kCodes, oQ = oP + 2 * kP, oE = oQ + kQS * kQ,
                       oW = oE + kE * kEBytes;
  // words
  static constexpr int wCq = 0;                        // [kQS][N] scale of a column's scores
  static constexpr int wLim = wCq + kQS * N;           // [kQS][N] keys that it sees
  static constexpr int wAt = wLim + kQS * N;           // [kQS][N] new row << 8 | query head of the group
  static constexpr int wR = wAt + kQS * N;             // [2][2][N] references for the epilogue, by unit and stream
  static constexpr int wL = wR + 4 * N;                // [2][2][4][N] sums of each softmax warp
  static constexpr int wMax = wL + 16 * N;             // [2][4][N] maxima of a step by stream and warp
  static constexpr int wRef = wMax + 8 * N;            // [2][4][N] a warp's copy of the references, negated
  static constexpr int wAl = wRef + 8 * N;             // [2][4][N] ... of the factors of a move
  static constexpr int wAh = wAl + 8 * N;              // [2][4][N] ... of their roots
  static constexpr int wWt = wAh + 8 * N;              // [4][2][N] an epilogue warp's weights of the streams
  static constexpr int wNf = wWt + 8 * N;              // [2][2] NaN taken out of V tiles, by unit and stream
  static constexpr int kWords = wNf + 4;
  static constexpr int oBar = oW + 4 * kWords;
  static constexpr int kSmem = oBar + 512 + 1024;
  static_assert(kSmem <= 232448, "shared memory");
  static_assert(2 * N * kAhead + 2 * 96 <= 512, "tensor memory");
};

template <int D, int N>
__global__ void __launch_bounds__(Cfg<D, N>::kThreads, 1)
mis_q8_attn_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                   const __grid_constant__ AttnParams p) {
  using C = Cfg<D, N>;
  constexpr int KS = C::kK, VS = C::kV, QS = C::kQS;
  // barriers
  constexpr int bQF = 0, bKF = bQF + QS, bKE = bKF + KS, bVF = bKE + KS, bVE = bVF + VS, bSF = bVE + VS, bPF = bSF + kAhead,
                bPV = bPF + 4, bOF = bPV + 2, bOE = bOF + 2, bST = bOE + 2, bSE = bST + 2, bDR = bSE + QS, nBar = bDR + 1;
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
  __shared__ int2 s_sum[C::kThreads / 32];
  __shared__ int s_from, s_req;
  __shared__ uint32_t s_bad;
  auto bar = [&](int i) { return smem_u32(bars + i); };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    *abort_flag = 0;
    s_bad = 0;
    for (int s = 0; s < 4; ++s) sNf[s] = 0;
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(bPF + s), 4);
      mbar_init(bar(bPF + 2 + s), 4);
      mbar_init(bar(bPV + s), 1);
      mbar_init(bar(bOF + s), 1);
      mbar_init(bar(bOE + s), 4);
      mbar_init(bar(bST + s), 8);
    }
    for (int s = 0; s < kAhead; ++s) mbar_init(bar(bSF + s), 1);
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
  int mine = 0, mineb = 0;             // what they count in a small batch and in a big one
  bool bad = false;
  for (int b = rb0; b < rb1; ++b) {
    const Given g = given(p, b);
    const Job j = job_of<N>(p, g, false);
    bad |= !j.ok;
    mine += j.cost();
    mineb += job_of<N>(p, g, true).cost();
  }
  int upto = mine, uptob = mineb;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, upto, o), y = __shfl_up_sync(0xffffffffu, uptob, o);
    if (lane >= o) { upto += x; uptob += y; }
  }
  if (lane == 31) s_sum[warp] = make_int2(upto, uptob);
  tc_fence_before();
  bad = __syncthreads_or(bad);
  tc_fence_after();
  int total = 0, totalb = 0;
#pragma unroll
  for (int w = 0; w < C::kThreads / 32; ++w) {
    if (w < warp) { upto += s_sum[w].x; uptob += s_sum[w].y; }
    total += s_sum[w].x;
    totalb += s_sum[w].y;
  }
  const bool big = total >= 8 * kStep * p.blocks;
  const Share share(big ? totalb : total, p.blocks, blockIdx.x, !big ? kStep : N == 16 ? kStep + kUnit : kWide + kUnitWide);
  if (tid == 0) p.meta[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
  if (big) { upto = uptob; mine = mineb; }
  if (share.size > 0 && share.from >= upto - mine && share.from < upto) {
    int at = upto - mine;
    for (int b = rb0; b < rb1; ++b) {
      const int next = at + job_of<N>(p, given(p, b), big).cost();
      if (share.from >= at && share.from < next) { s_req = b; s_from = share.from - at; }
      at = next;
    }
  }
  __syncthreads();
  const uint32_t tmem = *tmem_slot;
  const Bound W{abort_flag, p.wait_ns};
  const int box_shift = min(p.page_shift, 7);
  auto colS = [](int s) { return (uint32_t)(s * 2 * N); };
  // the streams of a unit lie side by side, three parts of 16 columns each; a
  // unit of more rows has three parts of 32
  auto colO = [](int unit, int stream) { return (uint32_t)(2 * N * kAhead + unit * 96 + stream * 48); };
  auto two_streams = [](int rows) { return N == 16 || rows <= 16; };

  Walk<N> w;
  if (share.size > 0 && w.enter(p, s_req, s_from, share.size, big)) {
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
      constexpr uint32_t idO = (1u << 4) | (1u << 10) | (1u << 15) | (1u << 16) | (8u << 24), idO48 = idO | (48u >> 3) << 17, idO96 = idO | (96u >> 3) << 17;
      bool ok = true;
      if (p.stall) ok = spin_all(bar(bDR), 0, W, 0x7ff);       // nothing arrives before the drain
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      // S of a step goes out as soon as its K is there, up to kAhead steps before
      // its O, so that the softmax finds its scores waiting; O once V and P are.
      // A lane a barrier looks for both at once: this warp's own instructions are
      // a long chain of a short step. What it counts has to be uniform over the
      // warp for the compiler too (shuffled where it comes from memory): the
      // products' operands are uniform registers
      int sk = 0, sv = 0, sq = 0, lu = 0;              // slots of K, V and Q; units
      uint32_t pk = 0, pv = 0, pq = 0;                 // their phases
      int ts = 0, to = 0;                              // steps whose S (O) has gone out
      // the steps between: unit << 7 | two streams << 6 | products of O << 3 |
      // last << 2 | opens its unit << 1 | first of its stream
      uint32_t wait[kAhead] = {};
      int k = 0, k0 = 0, k1 = 0, len = 0, two = 0;
      bool have = ok;
      uint32_t pp = 0;                                 // phases of P, by warpgroup and place
      auto enter = [&] {
        k = k0 = __shfl_sync(0xffffffffu, w.k0, 0);
        k1 = __shfl_sync(0xffffffffu, w.k1, 0);
        len = __shfl_sync(0xffffffffu, w.j.len, 0);
        two = __shfl_sync(0xffffffffu, two_streams(w.j.n * p.G - w.row0(w.head())) ? 1 : 0, 0);
      };
      enter();
      uint32_t idle = 0;
      uint64_t t0 = 0;
#pragma unroll 1
      while (ok && (have || to < ts)) {
        const uint32_t x = wait[0];
        const bool both = N > 16 && !(x & 64);         // both warpgroups have a part of P
        const int unit = x >> 7, pb = to & 1, s0 = both ? 0 : pb;         // place of P, stream
        // O's place: the unit before the last must have been read out
        const bool place = (x & 2) && unit >= 2;
        int b = bPF + 2 * s0 + pb;
        uint32_t ph = (pp >> (2 * s0 + pb)) & 1;
        if (lane == 1) { b = bVF + sv; ph = pv; }
        if (lane == 2) { b = bKF + sk; ph = pk; }
        if (lane == 3) { b = bQF + sq; ph = pq; }
        if (lane == 5) { b = bPF + 2 + pb; ph = (pp >> (2 + pb)) & 1; }
        if (lane == 4) { b = bOE + (unit & 1); ph = ((unit >> 1) - 1) & 1; }
        const uint32_t here = __ballot_sync(0xffffffffu, mbar_test_wait(bar(b), ph));
        const bool o_due = to < ts && (here & 3) == 3 && (!place || (here & 16)) && (!both || (here & 32));
        const bool s_due = have && ts - to < kAhead && (here & 4) && (k != k0 || (here & 8));
        if (!o_due && !s_due) {
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
          continue;
        }
        idle = 0;
        tc_fence_after();
        if (elect_uniform()) {
          if (o_due) {
            // V [key][d] and P [key][part, row], both MN-major, 32 keys a
            // product. D = 64 repeats its 64 columns (stride 0): rows 64..127 of
            // O^T equal rows 0..63.
            const uint32_t d = tm + colO(unit & 1, s0);
            const uint64_t a = rows_desc<D>(base + C::oV + sv * C::kCodes, 0);
            const uint64_t b2 = rows_desc<C::kPW>(base + C::oP + pb * C::kP, 0);
            const int nks = (x >> 3) & 7;
            const uint32_t id = both ? idO96 : idO48;
            mma_f8(d, a, b2, id, (x & 1) ^ 1u);
            if (nks == kKeys / 32) {
#pragma unroll
              for (int y = 1; y < kKeys / 32; ++y) mma_f8(d, a + y * (2 * D), b2 + y * (2 * C::kPW), id, 1u);
            } else {
#pragma unroll 1
              for (int y = 1; y < nks; ++y) mma_f8(d, a + y * (2 * D), b2 + y * (2 * C::kPW), id, 1u);
            }
            mma_commit(bar(bPV + pb));
            if (x & 4) mma_commit(bar(bOF + (unit & 1)));
          }
          if (s_due) {
            const uint32_t d = tm + colS(ts % kAhead);
            const uint64_t a = rows_desc<D>(base + sk * C::kCodes, 0), q = rows_desc<D>(base + C::oQ + sq * C::kQ, 0);
#pragma unroll
            for (int y = 0; y < D / 32; ++y) mma_f8(d, a + 2 * y, q + 2 * y, idS, y != 0);
            mma_commit(bar(bSF + ts % kAhead));
            mma_commit(bar(bKE + sk));
          }
          if (o_due) mma_commit(bar(bVE + sv));
        }
        __syncwarp();
        if (o_due) {
          if (++sv == VS) { sv = 0; pv ^= 1; }
          pp ^= both ? 5u << pb : 1u << (2 * s0 + pb);
          ++to;
#pragma unroll
          for (int i = 0; i + 1 < kAhead; ++i) wait[i] = wait[i + 1];
        }
        if (s_due) {
          const uint32_t y = (uint32_t)lu << 7 | (uint32_t)two << 6 | (uint32_t)((min(kKeys, len - k * kKeys) + 31) >> 5) << 3 |
                             (k + 1 == k1 ? 4u : 0u) | (k == k0 ? 2u : 0u) | (k < k0 + 1 + two ? 1u : 0u);
#pragma unroll
          for (int i = 0; i < kAhead; ++i)
            if (ts - to == i) wait[i] = y;
          ++ts;
          if (++sk == KS) { sk = 0; pk ^= 1; }
          if (++k == k1) {
            if (++sq == QS) { sq = 0; pq ^= 1; }
            ++lu;
            have = __shfl_sync(0xffffffffu, w.next(p), 0);
            if (have) enter();
          }
        }
      }
      // drain: all tensor-core work of the elected lane completes before dealloc
      if (elect_uniform()) mma_commit(bar(bDR));
      __syncwarp();
      wait_drain(bar(bDR), 0);
    } else if (warp == 2) {
      // ------------------------------------------------- Q and what its columns are
      // A row by D / 16 lanes, 16 elements each, RI rows at a time. Rows that are
      // none keep what was there: nobody reads their columns. The next rows come
      // while these are turned
      constexpr int LR = D / 16, RI = 32 / LR;
      const int c = lane % LR;
      int lu = 0, n = lane / LR;
      struct Rows { int h, first, rows, row0, see; } a, cur;
      bool more = true;
      uint4 x, y;
      int at;
      auto of = [&] {
        a.h = w.head();
        a.first = w.row0(a.h);
        a.rows = min(N, w.j.n * p.G - a.first);
        a.row0 = w.j.row0;
        a.see = w.j.len - w.j.n + 1;
      };
      auto load = [&] {                                // row n of unit a
        x = y = make_uint4(0u, 0u, 0u, 0u);
        at = 0;
        if (n >= a.rows) return;
        const int i = (a.first + n) / p.G, g = a.first + n - i * p.G;
        at = i << 8 | g;
        const uint4* src = reinterpret_cast<const uint4*>(p.q + (int64_t)(a.row0 + i) * p.qs + (int64_t)(a.h * p.G + g) * D + 16 * c);
        x = src[0];
        y = src[1];
      };
      of();
      load();
#pragma unroll 1
      while (true) {
        // these rows, and the next ones' loads
        const uint4 xa = x, ya = y;
        const int ata = at, na = n, sl = lu % QS, n0 = n - lane / LR;
        cur = a;
        const bool begins = n0 == 0, ends = n0 + RI >= a.rows;
        if (!ends) {
          n += RI;
        } else {
          n = lane / LR;
          more = w.next(p);
          of();
        }
        if (more) load();
        // what the unit before left there has been read
        if (begins && lu >= QS && !spin_all(bar(bSE + sl), ((lu / QS) - 1) & 1, W, 0x200)) break;
        float f[16];
        bf16x8_to_float(xa, f);
        bf16x8_to_float(ya, f + 8);
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < 16; e += 2) m = max3(m, fabsf(f[e]), fabsf(f[e + 1]));
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
        if (na < cur.rows) {
          st_shared_v4(q0 + chunk_at<D>(na, c), hi[0], hi[1], hi[2], hi[3]);
          st_shared_v4(q0 + N * D + chunk_at<D>(na, c), lo[0], lo[1], lo[2], lo[3]);
          if (c == 0) {
            words[C::wCq + sl * N + na] = pow2(min(ex, 127)) * p.scale_log2;
            reinterpret_cast<int*>(words)[C::wLim + sl * N + na] = cur.see + (ata >> 8);
            reinterpret_cast<int*>(words)[C::wAt + sl * N + na] = ata;
          }
        }
        if (!ends) continue;
        if (lane >= cur.rows && lane < N) {
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
      const int wg = (warp - 4) >> 2, sw = warp & 3, r = sw * 32 + lane, id = 1 + wg;
      const uint32_t tl = tmem + ((uint32_t)(sw * 32) << 16);
      int t = 0, lu = 0;                               // steps of both streams, units
      bool ok = true, more = true, gone = false;
      while (more) {
        const int slot = lu & 1, sq = lu % QS, first_row = w.row0(w.head()), rows = w.j.n * p.G - first_row;
        const int len = w.j.len, see = w.all_see(p, first_row);
        // every other step and all columns, or every step and its 16 of 32
        const bool two = two_streams(rows);
        const int str = two ? wg : 0, c0 = two ? 0 : 16 * wg, parts = two ? 16 : 32;
        float* ref = words + C::wRef + (str * 4 + sw) * N + c0;
        float* al = words + C::wAl + (str * 4 + sw) * N + c0;
        float* ah = words + C::wAh + (str * 4 + sw) * N + c0;
        float* mx = words + C::wMax + str * 4 * N + c0;
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
        int k = w.k0;
        const int stride = two ? 2 : 1;
        if (two && ((t ^ str) & 1)) { ++k; ++t; }
#pragma unroll 1
        for (; k < w.k1; k += stride, t += stride) {
          const int pb = t & 1;
          const uint32_t tS = tl + colS(t % kAhead) + c0;
          ok = spin_all(bar(bSF + t % kAhead), (t / kAhead) & 1, W, 0x710);
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
          const float vs = pow2(ev - 9), most = 24.f - (float)ev;
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
            const int seen = gone_key ? 0x7fffffff : key;
#pragma unroll
            for (int n = 0; n < 16; n += 4) {
              const int4 m = *reinterpret_cast<const int4*>(lim + n);
              if (seen >= m.x) s[n] = 0xff800000u;
              if (seen >= m.y) s[n + 1] = 0xff800000u;
              if (seen >= m.z) s[n + 2] = 0xff800000u;
              if (seen >= m.w) s[n + 3] = 0xff800000u;
            }
          }
          auto weigh = [&] {                           // x = s * kf - r
            const uint64_t k2 = f2_pack(__float_as_uint(kf), __float_as_uint(kf));
#pragma unroll
            for (int n = 0; n < 16; n += 4) {
              const float4 c = *reinterpret_cast<const float4*>(ref + n);
              float y0, y1, y2, y3;
              f2_unpack(f2_fma(f2_pack(s[n], s[n + 1]), k2, f2_pack(__float_as_uint(c.x), __float_as_uint(c.y))), y0, y1);
              f2_unpack(f2_fma(f2_pack(s[n + 2], s[n + 3]), k2, f2_pack(__float_as_uint(c.z), __float_as_uint(c.w))), y2, y3);
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
              for (int n = 0; n < 16; ++n) v[n] = fmaf(__uint_as_float(s[n]), kf, (float)(ev - 20));
              const int n = fold16<true>(v, lane);
              mx[sw * N + n] = v[0];
            }
            bar_sync128(id);
            // every warp draws the same conclusion from the four warps' maxima
            if (lane < 16) {
              const float old = first ? kNone : -ref[lane];
              float to = old;
#pragma unroll
              for (int q = 0; q < 4; ++q) to = fmaxf(to, mx[q * N + lane]);
              if (c0 + lane >= rows) to = kDead;
              const float root = to > old ? ex2(0.5f * (old - to)) : 1.f;
              al[lane] = root * root;
              ah[lane] = root;
              ref[lane] = -to;
            }
            __syncwarp();
            if (!first) {
              ok = spin_all(bar(bPV + ((t - stride) & 1)), ((t - stride) >> 1) & 1, W, 0x730);    // O holds every step before
              tc_fence_after();
              if (ok) {
#pragma unroll 1
                for (int q = 0; q < 3; ++q) {
                  const uint32_t tO = tl + colO(slot, str) + q * parts + c0;
                  tmem_ld16(tO, x);
                  tmem_ld_wait();
                  reg_fence16(x);
#pragma unroll
                  for (int n = 0; n < 16; ++n) x[n] = __float_as_uint(__uint_as_float(x[n]) * al[n]);
                  tmem_st16(tO, x);
                }
                tmem_st_wait();
#pragma unroll
                for (int n = 0; n < 8; ++n) {
                  const uint64_t root = f2_pack(__float_as_uint(ah[2 * n]), __float_as_uint(ah[2 * n + 1]));
                  l2[n] = f2_mul(f2_mul(l2[n], root), root);
                }
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
              const uint16_t a = e5m2x2_of_half2(h);
              const uint32_t h1 = rest(h, a);
              const uint16_t b = e5m2x2_of_half2(h1);
              const uint16_t c = e5m2x2_of_half2(rest(h1, b));
              (y ? hi : lo)[0] = a;
              (y ? hi : lo)[1] = b;
              (y ? hi : lo)[2] = c;
            }
#pragma unroll
            for (int q = 0; q < 3; ++q) part3[q][n] = __byte_perm(lo[q], hi[q], 0x5410);
          }
          if (ok && t >= 2) ok = spin_all(bar(bPV + pb), ((t - 2) >> 1) & 1, W, 0x740);   // what was there has been read
          if (ok) {
#pragma unroll
            for (int q = 0; q < 3; ++q)
              st_shared_v4(base + C::oP + pb * C::kP + chunk_at<C::kPW>(r, two ? q : 2 * q + wg), part3[q][0], part3[q][1], part3[q][2], part3[q][3]);
            // V rows that nobody sees hold anything; NaN that only some rows see
            // is left to the epilogue (0 x NaN would reach all)
            if (!plain && (two || wg == 0) && r < ((len - k * kKeys + 31) & ~31) && (gone_key || key >= see)) {
              const int sv = t % VS;
              ok = spin(bar(bVF + sv), (t / VS) & 1, W, 0x750);
              const uint32_t row = base + C::oV + sv * C::kCodes;
              if (gone_key) {
#pragma unroll
                for (int c = 0; c < D / 16; ++c)
                  if (ok) st_shared_v4(row + chunk_at<D>(r, c), 0u, 0u, 0u, 0u);
              } else {
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
                    y[q] &= ~((nn >> 7) * 0xffu);
                  }
                  if (any) st_shared_v4(at, u.x, u.y, u.z, u.w);
                  nan |= any != 0;
                }
              }
            }
            ok = __all_sync(0xffffffffu, ok);
          }
          fence_proxy_async();
          tc_fence_before();
          __syncwarp();
          if (ok && lane == 0) mbar_arrive(bar(bPF + 2 * wg + pb));
        }
        if (gone) break;
        t += w.k1 - k;                                 // the next unit's first step
        // the columns' sums over this warp's keys
        float l[16];
#pragma unroll
        for (int n = 0; n < 8; ++n) f2_unpack(l2[n], l[2 * n], l[2 * n + 1]);
        const int col = fold16<false>(l, lane);
        words[C::wL + ((slot * 2 + str) * 4 + sw) * N + c0 + col] = l[0];
        if (sw == 0 && lane < 16) words[C::wR + (slot * 2 + str) * N + c0 + lane] = first ? kNone : -ref[lane];
        if (__any_sync(0xffffffffu, nan) && lane == 0) sNf[slot * 2 + str] = 1u + (uint32_t)lu;
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
        const bool whole = w.k0 == 0 && w.k1 == w.j.steps, two = two_streams(rows);
        if (sw == 0 && lane == 0 && !whole && w.k0 == 0) {
          // the block that holds its last step; while there is nothing else to do
          const int c = share.holder(share.from + share.size - w.left + w.ahead() - 1);
          p.meta[2 * blockIdx.x] = make_int4(c - (int)blockIdx.x + 1, rows, h, first);
          p.meta[2 * blockIdx.x + 1] = make_int4(w.j.row0, lu ? 1 : 0, 0, 0);
        }
        ok = spin_all(bar(bST + slot), (lu >> 1) & 1, W, 0x800);
        if (!ok) break;
        const int piece = 2 * blockIdx.x + (lu ? 1 : 0), sq = lu % QS;
        // weights of the two streams' accumulators (zero: the unit had no step there)
        float* wt = words + C::wWt + sw * 2 * N;
        float mx = kNone, sum = 0.f;
        if (lane < N) {
          const float* l0 = words + C::wL + slot * 8 * N + lane;
          const float* l1 = l0 + 4 * N;
          const float r0 = words[C::wR + slot * 2 * N + lane], r1 = two ? words[C::wR + (slot * 2 + 1) * N + lane] : kNone;
          mx = fmaxf(r0, r1);
          const float h0 = ex2(0.5f * (r0 - mx)), h1 = ex2(0.5f * (r1 - mx)), a0 = h0 * h0, a1 = h1 * h1;
          sum = h0 * (h0 * ((l0[0] + l0[N]) + (l0[2 * N] + l0[3 * N])));
          if (two) sum += h1 * (h1 * ((l1[0] + l1[N]) + (l1[2 * N] + l1[3 * N])));
          // the products' weights carry 2^-9; NaN stays
          const float inv = whole ? (sum != 0.f ? __fdividef(512.f, sum) : 0.f) : 1.f;
          wt[lane] = a0 * inv;
          wt[N + lane] = a1 * inv;
        }
        const int* at = reinterpret_cast<const int*>(words) + C::wAt + sq * N;
        const int* lim = reinterpret_cast<const int*>(words) + C::wLim + sq * N;
        if (sw == 0 && lane < rows && !whole) p.rl[(int64_t)piece * N + lane] = make_float2(mx, sum);
        __syncwarp();
        ok = spin_all(bar(bOF + slot), (lu >> 1) & 1, W, 0x810);
        if (!ok) break;
        tc_fence_after();
        const bool nf = sNf[slot * 2] == 1u + (uint32_t)lu || (two && sNf[slot * 2 + 1] == 1u + (uint32_t)lu);
        // streams that had a step: both, or the one of a single step
        const bool use0 = !two || w.k1 - w.k0 > 1 || !(t & 1), use1 = two && (w.k1 - w.k0 > 1 || (t & 1));
        const int parts = two ? 16 : 32;
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
          uint32_t y[2][3][CH];                        // the parts of the streams' accumulators
#pragma unroll
          for (int i = 0; i < 3; ++i) tmem_ld8(tl + colO(slot, 0) + i * parts + e0 + q, y[0][i]);
          if (two) {
#pragma unroll
            for (int i = 0; i < 3; ++i) tmem_ld8(tl + colO(slot, 1) + i * parts + e0 + q, y[1][i]);
          }
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 6; ++i) reg_fence8(y[i / 3][i % 3]);
          auto add = [&](int stream) {
#pragma unroll
            for (int n = 0; n < CH; ++n) {
              const float x = fmaf(__uint_as_float(y[stream][2][n]), 0.00390625f,
                                   fmaf(__uint_as_float(y[stream][1][n]), 0.0625f, __uint_as_float(y[stream][0][n])));
              ov[n] = fmaf(wt[stream * N + e0 + q + n], x, ov[n]);
            }
          };
          if (use0) add(0);
          if (use1) add(1);
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
        // not before O was there: a sum whose waits ran out on the way is not written
        if (sw == 0 && lane < rows && whole && p.lse)
          p.lse[(int64_t)(h * p.G + (at[lane] & 255)) * p.T + w.j.row0 + (at[lane] >> 8)] =
              sum != 0.f ? lse_of(mx, sum) : -INFINITY;
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

// Joins the pieces of a unit that several blocks hold, in block order: block
// (c, y) takes rows of the unit that starts in block c, a row by `share` of its
// four warps, which take the pieces in turn (all four where rows are few: one
// request of 8192 rows, 2 a kv head, 13.5 us, by one warp 15.7; units of 16 rows 36.6
// and 35.5). What it needs lies in one place, since its time is that of the trips to
// L2 it makes one behind the other (units found by bisection of the requests' steps:
// 10 us for 64 decoded tokens), and that of its blocks' launch, which the attention's
// registers leave no room for before its own blocks end: no more of them than there
// can be rows.
template <int D, int N>
__global__ void __launch_bounds__(32 * kJoinWarps)
mis_q8_join_kernel(const __grid_constant__ AttnParams p, int share) {
  constexpr int E = D / 32;
  __shared__ float s_acc[kJoinWarps][D + 1];
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x;
  const int sub = warp & (share - 1), n = blockIdx.y * (kJoinWarps / share) + warp / share;
  const int4 u = p.meta[2 * c], v = p.meta[2 * c + 1];
  if (c == 0 && blockIdx.y == 0 && warp == 0) {
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
  if (pieces < 2) return;
  const bool live = n < u.y;
  // the first piece lies in block c's first or second slot, the others in the
  // first slots of the blocks that follow
  auto at = [&](int y) { return (int64_t)(2 * (c + y) + (y == 0 ? v.y : 0)) * N + (live ? n : 0); };
  float acc[E], sum = 0.f, m = kNone;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  auto load = [&](int y, float* z, float2& rl) {
    const float* from = p.part + at(y) * D + lane * E;
    rl = p.rl[at(y)];
    if constexpr (E == 4) {
      const float4 z4 = *reinterpret_cast<const float4*>(from);
      z[0] = z4.x; z[1] = z4.y; z[2] = z4.z; z[3] = z4.w;
    } else {
      const float2 z2 = *reinterpret_cast<const float2*>(from);
      z[0] = z2.x; z[1] = z2.y;
    }
  };
  // the first pieces come while the maximum is taken
  float z0[E], z1[E];
  float2 rl0, rl1;
  load(min(sub, pieces - 1), z0, rl0);
  load(min(sub + share, pieces - 1), z1, rl1);
  bool stuck = false;
  for (int y = lane; y < pieces; y += 32) {
    m = fmaxf(m, p.rl[at(y)].x);
    stuck |= (p.flags[2 * (c + y)] & kDevTimeout) != 0;
  }
  if (__any_sync(0xffffffffu, stuck)) return;          // a piece is missing: every warp sees it
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll 1
  for (int y = sub; y < pieces; y += 2 * share) {
    const float h0 = ex2(0.5f * (rl0.x - m)), h1 = y + share < pieces ? ex2(0.5f * (rl1.x - m)) : 0.f;
    const float f0 = h0 * h0, f1 = h1 * h1;
    sum += h0 * (h0 * rl0.y);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] += f0 * z0[e];
    if (y + share < pieces) {
      sum += h1 * (h1 * rl1.y);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += f1 * z1[e];
    }
    load(min(y + 2 * share, pieces - 1), z0, rl0);
    load(min(y + 3 * share, pieces - 1), z1, rl1);
  }
  if (share > 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) s_acc[warp][e * 32 + lane] = acc[e];
    if (lane == 0) s_acc[warp][D] = sum;
    __syncthreads();
    if (sub) return;
    for (int y = 1; y < min(share, pieces); ++y) {
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += s_acc[warp + y][e * 32 + lane];
      sum += s_acc[warp + y][D];
    }
  }
  if (!live) return;
  const int i = (u.w + n) / p.G, head = u.z * p.G + u.w + n - i * p.G;
  // the products' weights carry 2^-9
  const float inv = sum != 0.f ? __fdividef(512.f, sum) : 0.f;
  uint32_t out[E / 2];
#pragma unroll
  for (int e = 0; e < E / 2; ++e) out[e] = sum != 0.f ? pack_bf16(acc[2 * e] * inv, acc[2 * e + 1] * inv) : 0u;
  __nv_bfloat16* dst = p.o + (int64_t)(v.x + i) * p.os + (int64_t)head * D + lane * E;
  if constexpr (E == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
  else *reinterpret_cast<uint32_t*>(dst) = out[0];
  if (p.lse && lane == 0)
    p.lse[(int64_t)head * p.T + v.x + i] = sum != 0.f ? lse_of(m, sum) : -INFINITY;
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
// keys. Units of 16 and of 32: 64 requests of 16 rows 35.4 and 37.6 us, 256 short
// ones of 2 rows 67 and 79; 4 long ones of 32 rows 349 and 186, 32 of 64 rows 99 and
// 87 (4 long ones, of which one has 32 rows and the others fewer than 17, 169 and 176).
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
  const int rows = std::min(N, p.max_rows * p.G), share = rows <= 8 ? kJoinWarps : 1;
  return launch_pdl(mis_q8_join_kernel<D, N>, dim3((unsigned)p.blocks, (unsigned)(rows * share + kJoinWarps - 1) / kJoinWarps),
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
  // what steps and units count is counted in 32 bits
  const double tiles = (double)((head_rows(desc, cache) + 15) / 16) * cache->Hkv;
  if ((((double)max_pages * cache->page_size / kKeys + 1) * kWide + kUnitWide) * tiles * desc->B >= 2147483648.0) return MIS_ERR_UNSUPPORTED;
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
  p.most = max_pages << p.page_shift;
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
