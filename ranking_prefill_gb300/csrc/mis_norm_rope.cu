// Per-head root mean square norms of Q and K with the rotary embedding in the
// same pass, sm_103a (the Qwen3 family normalises each head's query and key
// before the rotation).
//
//   y = w * x / sqrt(mean(x^2) + eps) over the D elements of a (row, head),
//   the pair (y[i], y[i + D/2]) turns by p * base^(-2i/D), i < D/2.
//
// fp32 from the loaded bf16 values on, one rounding at the end. Every element is
// read and written once, so HBM bounds it. D / 16 lanes share a head: a lane
// holds 8 pairs, so the mean takes 2 or 3 exchanges and the rotation none. The
// angles of a lane's 8 pairs serve every head that its thread takes. 128K tokens
// of 24 heads, 128 wide, take 241 us (6.7 TB/s of the 6.8 that a copy reaches),
// without the next heads' way to L2 254, one head at a time 314; 4,099 of 16 heads,
// 64 wide, 7.5 us; 32 tokens 3.0, a launch.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "mis_internal.h"
#include "mis_ptx.cuh"
#include "mis_rows.cuh"

namespace mis {
namespace {

using namespace dev;

constexpr int kThreads = 256;

struct NormParams {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  __nv_bfloat16* qo;
  __nv_bfloat16* ko;
  int64_t qs, ks, qos, kos;        // row strides, elements
  const __nv_bfloat16* qw;         // or null: no norm
  const __nv_bfloat16* kw;
  const int32_t* pos;              // or null: no rotation
  float eps;
  int32_t T, Hq, Hkv, hpt;         // hpt: heads of a thread
  uint64_t turn[64];
};

template <int D, int U>
__global__ void __launch_bounds__(kThreads)
mis_qk_norm_rope_kernel(const __grid_constant__ NormParams p) {
  constexpr int HALF = D / 2, NC = D / 16;
  griddep_wait();
  const int H = p.Hq + p.Hkv, NG = (H + p.hpt - 1) / p.hpt;
  const int64_t gid = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int c = (int)(gid % NC);
  const int64_t cell = gid / NC;
  const int grp = (int)(cell % NG);
  const int64_t t = cell / NG;
  if (t >= p.T) return;                          // the lanes of a row leave together
  const uint32_t lanes = row_lanes<NC>();
  // U heads at a time, so that nothing of one waits for another. Where a thread
  // has few, the first ones' loads are in flight while the angles are taken (in
  // the other form that costs registers, and with them half the blocks)
  const int h0 = grp * p.hpt, h1 = min(h0 + p.hpt, H), last = h1 - 1;
  const __nv_bfloat16* qr = p.q + t * p.qs + c * 8;
  const __nv_bfloat16* kr = p.k + t * p.ks + c * 8 - (int64_t)p.Hq * D;
  uint4 a[U], b[U];
  auto load = [&](int h) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int x = min(h + i, last);
      const __nv_bfloat16* at = (x < p.Hq ? qr : kr) + (int64_t)x * D;
      a[i] = ld_row16(at);
      b[i] = ld_row16(at + HALF);
    }
  };
  // the U heads from h on come to L2, a lane a line of 128 bytes: loads of the
  // next ones in registers would cost half the blocks
  auto ahead = [&](int h) {
    constexpr int LH = D / 64;
    const int x = h + c / LH;
    const __nv_bfloat16* at = (x < p.Hq ? p.q + t * p.qs : p.k + t * p.ks - (int64_t)p.Hq * D) + (int64_t)x * D + (c % LH) * 64;
    if (x < h1 && c / LH < U) asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
  };
  if (U == 2) load(h0);
  float sn[8], cs[8];
  if (p.pos) {
    const int pos = p.pos[t];
#pragma unroll
    for (int e = 0; e < 8; ++e) sincos_quarters(pos, p.turn[c * 8 + e], sn[e], cs[e]);
  }
  // heads [g0, g1) of one tensor
  auto pass = [&](__nv_bfloat16* dst, const __nv_bfloat16* w, int g0, int g1) {
    float wx[8], wy[8];
    if (w) {
      bf16x8_to_float(*reinterpret_cast<const uint4*>(w + c * 8), wx);
      bf16x8_to_float(*reinterpret_cast<const uint4*>(w + HALF + c * 8), wy);
    }
#pragma unroll 1
    for (int h = g0; h < g1; h += U) {
      if (U != 2 || h != h0) load(h);
      if (h + U < h1) ahead(h + U);
      float x[U][8], y[U][8];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        bf16x8_to_float(a[i], x[i]);
        bf16x8_to_float(b[i], y[i]);
      }
      if (w) norm_rows<D, U>(x, y, wx, wy, p.eps, lanes);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (h + i >= g1) break;
        if (p.pos) rotate_row(x[i], y[i], sn, cs);
        uint32_t u[4], v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          u[e] = pack_bf16(x[i][2 * e], x[i][2 * e + 1]);
          v[e] = pack_bf16(y[i][2 * e], y[i][2 * e + 1]);
        }
        __nv_bfloat16* to = dst + (int64_t)(h + i) * D;
        *reinterpret_cast<uint4*>(to) = make_uint4(u[0], u[1], u[2], u[3]);
        *reinterpret_cast<uint4*>(to + HALF) = make_uint4(v[0], v[1], v[2], v[3]);
      }
    }
  };
  const int mid = min(max(h0, p.Hq), h1);
  pass(p.qo + t * p.qos + c * 8, p.qw, h0, mid);
  pass(p.ko + t * p.kos + c * 8 - (int64_t)p.Hq * D, p.kw, mid, h1);
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace
}  // namespace mis

using namespace mis;

extern "C" mis_status_t mis_qk_norm_rope(const void* q, const void* k, void* q_out, void* k_out,
                                         int64_t q_row_stride, int64_t k_row_stride,
                                         int64_t q_out_row_stride, int64_t k_out_row_stride, int32_t T,
                                         int32_t Hq, int32_t Hkv, int32_t D, const void* q_weight,
                                         const void* k_weight, float eps, const int32_t* position_ids,
                                         double rope_base, void* stream) {
  if (T < 0 || Hq < 0 || Hkv < 0 || Hq + (int64_t)Hkv < 1) return MIS_ERR_INVALID_ARG;
  // a tensor without heads: nothing of it is looked at
  if (Hq == 0) { q = q_out = nullptr; q_weight = nullptr; q_row_stride = q_out_row_stride = 0; }
  if (Hkv == 0) { k = k_out = nullptr; k_weight = nullptr; k_row_stride = k_out_row_stride = 0; }
  if (D != 64 && D != 128) return MIS_ERR_UNSUPPORTED;
  if ((int64_t)Hq + Hkv > 65536) return MIS_ERR_UNSUPPORTED;
  if ((q_weight || k_weight) && !(eps >= 0.f && eps <= 1.f)) return MIS_ERR_INVALID_ARG;
  if (position_ids && (!(rope_base > 1.0) || !std::isfinite(rope_base))) return MIS_ERR_INVALID_ARG;
  const int64_t wq = (int64_t)Hq * D, wk = (int64_t)Hkv * D;
  if (Hq > 0 && (q_row_stride < wq || q_out_row_stride < wq || ((q_row_stride | q_out_row_stride) & 7)))
    return MIS_ERR_SHAPE;
  if (Hkv > 0 && (k_row_stride < wk || k_out_row_stride < wk || ((k_row_stride | k_out_row_stride) & 7)))
    return MIS_ERR_SHAPE;
  if (T == 0) return MIS_OK;
  if ((Hq > 0 && (!q || !q_out)) || (Hkv > 0 && (!k || !k_out))) return MIS_ERR_INVALID_ARG;
  for (const void* x : {q, k, (const void*)q_out, (const void*)k_out, q_weight, k_weight})
    if (!aligned(x, 16)) return MIS_ERR_INVALID_ARG;
  if (!aligned(position_ids, 4)) return MIS_ERR_INVALID_ARG;
  {
    const Span in[5] = {{q, Hq ? T : 0, 2 * q_row_stride, 2 * wq}, {k, Hkv ? T : 0, 2 * k_row_stride, 2 * wk},
                        {q_weight, 1, 0, 2 * (int64_t)D}, {k_weight, 1, 0, 2 * (int64_t)D},
                        {position_ids, 1, 0, 4 * (int64_t)T}};
    const Span out[2] = {{q_out, Hq ? T : 0, 2 * q_out_row_stride, 2 * wq},
                         {k_out, Hkv ? T : 0, 2 * k_out_row_stride, 2 * wk}};
    // in place: the same rows, each element read and written by one thread
    const bool same[2] = {q_out == q && q_out_row_stride == q_row_stride,
                          k_out == k && k_out_row_stride == k_row_stride};
    for (int i = 0; i < 2; ++i)
      for (int j = 0; j < 5; ++j)
        if (!(i == j && same[i]) && overlap(out[i], in[j])) return MIS_ERR_INVALID_ARG;
    if (overlap(out[0], out[1])) return MIS_ERR_INVALID_ARG;
  }
  NormParams p;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.qo = static_cast<__nv_bfloat16*>(q_out);
  p.ko = static_cast<__nv_bfloat16*>(k_out);
  p.qs = q_row_stride; p.ks = k_row_stride; p.qos = q_out_row_stride; p.kos = k_out_row_stride;
  p.qw = static_cast<const __nv_bfloat16*>(q_weight);
  p.kw = static_cast<const __nv_bfloat16*>(k_weight);
  p.pos = position_ids;
  p.eps = eps;
  p.T = T; p.Hq = Hq; p.Hkv = Hkv;
  if (position_ids) fill_turns(rope_base, D, p.turn);
  const int H = Hq + Hkv;
  // an angle serves all heads of a thread; a row's heads are split over
  // threads only while its lanes alone would leave SMs idle (4,099 tokens of 16
  // heads, 64 wide: 512 threads an SM 7.5 us, 1,024 8.4)
  const int64_t cells = (int64_t)T * (D / 16), want = 512 * (int64_t)num_sms();
  const int64_t split = std::max<int64_t>(1, std::min<int64_t>(H, want / cells));
  p.hpt = (int32_t)((H + split - 1) / split);
  const int64_t threads = cells * ((H + p.hpt - 1) / p.hpt);
  const int64_t blocks = (threads + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffff) return MIS_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  try {
    // four heads at a time where a thread has eight or more: 128K tokens of 24 heads
    // 241 us, two at a time 256, of 8 heads 96 and 101, 16K of 24 36.6 and 38.2. Below,
    // the last four are mostly not full: 128K of 6 heads 88 and 81, 2,400 of 24, six a
    // thread, 11.3 and 10.3 (of 7 heads 92 and 96; 4,099 of 16, four a thread, 7.1 and
    // 7.6; 9 heads of 128K 115 either way)
    const bool many = p.hpt >= 8;
    auto kern = D == 128 ? (many ? mis_qk_norm_rope_kernel<128, 4> : mis_qk_norm_rope_kernel<128, 2>)
                         : (many ? mis_qk_norm_rope_kernel<64, 4> : mis_qk_norm_rope_kernel<64, 2>);
    const cudaError_t e = launch_pdl(kern, dim3((unsigned)blocks), dim3(kThreads), 0, st, p);
    return e == cudaSuccess ? MIS_OK : MIS_ERR_CUDA;
  } catch (...) {
    return MIS_ERR_CUDA;
  }
}
