// New keys and values into the paged cache: e4m3 codes with one scale for
// each page of tokens and head.
//   scale' = max(scale of the page if it holds older rows, max |x| / 448)
//   new codes = e4m3(x / scale'); where the scale grew, the older rows' codes
//   are rounded again: e4m3(code x (scale / scale'))
// fp32 divisions are correctly rounded, so the codes equal a plain evaluation
// of these expressions.  A NaN or infinity among a page's new rows makes its
// scale NaN or infinite, and with it the page's values for that head; the new
// codes are 0 then, so that no NaN code lies beside other rows' in a product.
//
// One CTA = one (sequence, page that the call changes) x key/value head, keys
// and values; the pages of a sequence are found on the device (slot_at), so
// the grid needs only the row count.  A thread keeps its pieces of the new rows
// (8 elements each) in registers between the maximum and the rounding: the
// rows are read once.  Bytes bound it: 2 or 4 read and 1 written per element,
// and the codes of the older rows where a scale grew.  Eight pieces a thread
// spread the set-up thin (43k rows of 8 heads of 128 in bf16, 265 MB: 53 us,
// 5.0 TB/s; with four 58 us).
#include <cuda_fp16.h>

#include "attn_view.cuh"
#include "layers.h"

namespace sf {
namespace {

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// four e4m3 codes of a .. d, saturating (NaN stays NaN); the instruction
// itself: cuda_fp8.h's function for two costs about four more
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t w;
  asm("{.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};}" : "=r"(w) : "f"(a), "f"(b), "f"(c), "f"(d));
  return w;
}
__device__ __forceinline__ float4 e4m3x4_to_f(uint32_t w) {
  uint32_t lo, hi;
  asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h;}" : "=r"(lo), "=r"(hi) : "r"(w));
  const float2 a = __half22float2(*reinterpret_cast<__half2*>(&lo)), b = __half22float2(*reinterpret_cast<__half2*>(&hi));
  return make_float4(a.x, a.y, b.x, b.y);
}

// x / by, correctly rounded: the rounded product with r = 1 / by, corrected by
// its exact residual (Markstein 1990); by, r and x far from the ends of the range
__device__ __forceinline__ float2 over2(float2 x, float2 nby, float2 r) {
  const float2 q = __fmul2_rn(x, r);
  return __ffma2_rn(__ffma2_rn(nby, q, x), r, q);
}

template <typename E> struct Piece;   // 8 consecutive elements
template <> struct Piece<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void get(float* x) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  // largest magnitude as fp32 bits: ordered as the values are, NaN above all
  __device__ __forceinline__ uint32_t top() const {
    return max(max(max(abs_bits(a.x), abs_bits(a.y)), max(abs_bits(a.z), abs_bits(a.w))),
               max(max(abs_bits(b.x), abs_bits(b.y)), max(abs_bits(b.z), abs_bits(b.w))));
  }
};
template <> struct Piece<bf16> {
  uint4 a;
  __device__ __forceinline__ void load(const bf16* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float* x) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[2 * k] = __uint_as_float(w[k] << 16);
      x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ uint32_t top() const {
    constexpr uint32_t A = 0x7fff7fffu;
    const uint32_t m = __vmaxu2(__vmaxu2(a.x & A, a.y & A), __vmaxu2(a.z & A, a.w & A));
    return max(m << 16, m & 0xffff0000u);
  }
};

}  // namespace

// NP pieces of the keys and of the values per thread: NP x blockDim.x = page x
// D / 8.
template <typename E, int NP>
__global__ void __launch_bounds__(256) kv_append_kernel(const E* __restrict__ kin, int64_t ldk, const E* __restrict__ vin,
                                                        int64_t ldv, KvCache c, KvSeqs q, int page_log2, int* err) {
  SF_PDL_ENTRY();
  __shared__ uint32_t red[2][16];
  int nth;
  int sb, se;
  const int s = slot_at(q.cu, q.n, q.T, blockIdx.x, 1, page_log2, 2, nth, sb, se);
  const int held = max(q.held[s], -1), n_new = se - sb;   // (differences stay in 32 bits)
  int first = held - n_new;                    // position of the first new row
  const bool bad = first < 0;
  if (bad) {                                   // rows before position 0 have no place
    sb -= first;
    first = 0;
  }
  if (threadIdx.x == 0) {
    if (bad) set_err(err, ERR_BOUNDS);
    if (blockIdx.y == 0) report_offsets(q.cu, blockIdx.x, q.n, q.T, err);
  }
  if (nth < 0 || n_new <= 0 || held <= first) return;
  const int pi = (first >> page_log2) + nth;
  if ((int64_t)pi * c.page >= held) return;
  const int p = pi < q.table_cols ? q.table[(int64_t)s * q.table_cols + pi] : -1;
  if (p < 0 || p >= c.n_pages) {
    if (threadIdx.x == 0) set_err(err, ERR_BOUNDS);
    return;
  }
  const int kvh = blockIdx.y;
  const int64_t ph = (int64_t)p * c.n_kv + kvh;
  const int t0 = pi * c.page;                  // position of the page's first row
  const int older = max(0, first - t0);        // rows of the page that were there before
  const int fill = min(c.page, held - t0);     // rows of the page with the new ones
  const int row_log2 = c.D == 64 ? 3 : 4;      // pieces of a row
  const float was[2] = {older > 0 ? c.kscale[ph] : 0.f, older > 0 ? c.vscale[ph] : 0.f};

  Piece<E> x[2][NP];
  uint32_t mx[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const int e = threadIdx.x + k * blockDim.x, r = e >> row_log2;
    if (r >= older && r < fill) {
      const int64_t row = sb + t0 + r - first;
      const int col = kvh * c.D + (e & ((1 << row_log2) - 1)) * 8;
      x[0][k].load(kin + row * ldk + col);
      x[1][k].load(vin + row * ldv + col);
    }
  }
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const int r = (threadIdx.x + k * blockDim.x) >> row_log2;
    if (r >= older && r < fill) {
      mx[0] = max(mx[0], x[0][k].top());
      mx[1] = max(mx[1], x[1][k].top());
    }
  }
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    mx[y] = __reduce_max_sync(0xffffffffu, mx[y]);
    if ((threadIdx.x & 31) == 0) red[y][threadIdx.x >> 5] = mx[y];
  }
  __shared__ float s_now[2], s_r[2], s_again[2];
  __syncthreads();
  if (threadIdx.x < 2) {   // the four divisions of a block once, not per thread (8 prompts: 61 -> 56 us)
    const int y = threadIdx.x;
    const float w = y ? was[1] : was[0];
    uint32_t top = 0;
    for (int k = 0; k < (int)blockDim.x / 32; ++k) top = max(top, red[y][k]);
    float now = __fdiv_rn(__uint_as_float(top), 448.f);
    if (w > now || w != w) now = w;
    const float by = now > 0.f || now != now ? now : 1.f;
    s_now[y] = now;
    s_r[y] = __fdiv_rn(1.f, by);
    s_again[y] = __fdiv_rn(w, by);
  }
  __syncthreads();
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    const float now = s_now[y];
    const float by = now > 0.f || now != now ? now : 1.f;
    const bool grew = now > was[y];
    const bool plain = !(by > 1e-30f && by < 1e30f);   // near the ends of the range: the division itself
    const bool lost = !isfinite(now);
    const float r1 = s_r[y], again = s_again[y];
    const float2 r2 = make_float2(r1, r1), nby = make_float2(-by, -by);
    uint8_t* codes = (y ? c.v : c.k) + ph * c.page * c.D;
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int e = threadIdx.x + k * blockDim.x, r = e >> row_log2;
      if (r >= fill) continue;
      uint2* dst = reinterpret_cast<uint2*>(codes + (int64_t)e * 8);
      if (r >= older) {
        float f[8];
        x[y][k].get(f);
        if (lost) {
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = 0.f;
        } else if (plain) {
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = __fdiv_rn(f[i], by);
        } else {
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const float2 d = over2(make_float2(f[i], f[i + 1]), nby, r2);
            f[i] = d.x;
            f[i + 1] = d.y;
          }
        }
        *dst = make_uint2(e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7]));
      } else if (grew) {
        const uint2 w = *dst;
        const float4 a = e4m3x4_to_f(w.x), b = e4m3x4_to_f(w.y);
        *dst = make_uint2(e4m3x4(a.x * again, a.y * again, a.z * again, a.w * again),
                          e4m3x4(b.x * again, b.y * again, b.z * again, b.w * again));
      }
    }
    if (threadIdx.x == 0 && (grew || older == 0 || now != now)) (y ? c.vscale : c.kscale)[ph] = now;
  }
}

template <typename E, int NP>
static cudaError_t launch_np(const E* k, int64_t ldk, const E* v, int64_t ldv, const KvCache& c, const KvSeqs& q,
                             int threads, int* err, cudaStream_t st) {
  int page_log2 = 4;
  while ((1 << page_log2) < c.page) ++page_log2;
  const dim3 grid((unsigned)(q.T / c.page + 2 * (int64_t)q.n), c.n_kv);
  CK_LAUNCH(launch_k(kv_append_kernel<E, NP>, grid, dim3(threads), 0, st, k, ldk, v, ldv, c, q, page_log2, err));
  return cudaGetLastError();
}

template <typename E>
cudaError_t launch_kv_append(const E* k, int64_t ldk, const E* v, int64_t ldv, const KvCache& c, const KvSeqs& q,
                             int* err, cudaStream_t st) {
  const int pieces = c.page * c.D / 8;   // 128 (16 x 64) .. 2048 (128 x 128)
  switch (pieces) {
    case 128: return launch_np<E, 1>(k, ldk, v, ldv, c, q, 128, err, st);
    case 256: return launch_np<E, 2>(k, ldk, v, ldv, c, q, 128, err, st);
    case 512: return launch_np<E, 4>(k, ldk, v, ldv, c, q, 128, err, st);
    case 1024: return launch_np<E, 8>(k, ldk, v, ldv, c, q, 128, err, st);
    default: return launch_np<E, 8>(k, ldk, v, ldv, c, q, 256, err, st);
  }
}
template cudaError_t launch_kv_append<float>(const float*, int64_t, const float*, int64_t, const KvCache&, const KvSeqs&,
                                             int*, cudaStream_t);
template cudaError_t launch_kv_append<bf16>(const bf16*, int64_t, const bf16*, int64_t, const KvCache&, const KvSeqs&,
                                            int*, cudaStream_t);

}  // namespace sf
