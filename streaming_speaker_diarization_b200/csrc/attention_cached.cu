// Attention of a sequence's newest rows over its cached keys and values (e4m3
// codes in pages, one scale per page and key/value head; attn_view.cuh has
// the score and mask).  Row r of the call's rows of a sequence with `held`
// cached rows stands at position held - n + r.
//
// The codes of a sequence are read once for up to 16 query rows of a key/value
// head (8 in fp32 at heads of 128): the G heads that share it times the new rows
// are packed as rows of 8- or 16-row tiles, each of which reads them (the 128-row
// tiles of the tcgen05 products would be nearly empty for the few rows of a
// step, whose work the bytes of the codes bound, not the products).
//
// Products are mma.sync m16n8k16 with fp16 operands and fp32 sums, keys (and
// then output dims) along M, query rows along N, so a tile of up to 8 rows
// wastes nothing.  e4m3 codes are exact in fp16 (the e4m3 form of the product
// was measured and is not faster here: 900 instructions per 32 keys of 128
// dims against 500).  A bf16 query is exact in fp16 once its row is scaled by
// a power of two (row maximum in [2^14, 2^15); what lies below 2^-39 of it is
// dropped); its softmax weights are rounded to 11 bits.  fp32 queries and
// weights are split into two fp16 parts, 22 bits.  The tensor cores cut their
// sums off instead of rounding them, which long chains of products turn into
// a bias: fp32 outputs are summed over 16 keys there and rounded onwards, the
// second parts' scores in a chain of their own (7 rows over 1740 keys,
// relative error 1.1e-6 -> 4.8e-7; the formula in fp32 operations 5.1e-7; 16
// requests of 3 rows over up to 6000 keys 23.7 -> 25.9 us).  (What is said of
// NaN codes and tiny scales below added about 2 % to 16 x 3 and 64 x 13 rows.)
// V's page scale goes into the exponent: with s' = s + log2(vscale), the
// weight 2^(s' - max s' + 14) lies in fp16's range whatever the scales are,
// and the sum of weights takes weight / vscale, so nothing else is rounded.
// Scales under 2^-60, 0 among them, count as 2^-60 there and take the rest in
// the outputs' weights.
//
// One warp takes 32 keys a step and copies their rows whole with cp.async into
// slots of its own, keys two steps ahead and values one.  A thread's fragment
// positions are a permutation of keys and dims chosen so that it reads 8 or 16
// consecutive bytes of a row at a time; the pieces of a row are stored in an
// order that keeps those reads free of bank conflicts (piece_at).  A row's
// reference maximum moves only when the new one exceeds it by 2^1.75 (weights
// stay in the operand's range), which makes the rescaling of the outputs rare.
// The keys of a (sequence, head, row tile) are split over the warps of a CTA
// and over the CTAs of a cluster; their (max, sum, output) parts meet in
// shared memory, then in distributed shared memory: one launch, no
// atomics, the same order of sums each time.  Few, long row tiles are split
// over several clusters, whose parts a second kernel joins.
#include <cuda_fp16.h>

#include <algorithm>

#include "attn_view.cuh"
#include "layers.h"
#include "tcgen05.cuh"

namespace sf {
namespace {

// log2 of the least V scale that an exponent carries.  The weights' sum undoes the scale (2^60 at most), and a rescaling or
// a weight of 2^-126 is the last one kept: scales 2^84 apart leave 2^-42 of the sum for a key, more than any count of keys
constexpr float VS_FLOOR = -60.f;

__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_new(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {   // c = a b
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
// two e4m3 codes -> fp16 pair, exact: the low and the high 16 bits of w (one
// instruction each: measured 1.7 per clock and SM, against 0.9 and a shift
// through cuda_fp8.h's 16-bit arguments)
__device__ __forceinline__ uint32_t cvt_lo(uint32_t w) {
  uint32_t r;
  asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, l;}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t cvt_hi(uint32_t w) {
  uint32_t r;
  asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, h;}" : "=r"(r) : "r"(w));
  return r;
}
// an fp16 pair and the pair of what it leaves over
__device__ __forceinline__ uint32_t half_pair(float x0, float x1, uint32_t& rest) {
  const __half2 h = __floats2half2_rn(x0, x1);
  const float2 b = __half22float2(h);
  rest = h2_bits(__floats2half2_rn(x0 - b.x, x1 - b.y));
  return h2_bits(h);
}
// zeros in the place of NaN codes; whether there was one
__device__ __forceinline__ uint32_t clear_nan(uint32_t& w) {
  const uint32_t is = __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu);
  w &= ~is;
  return is;
}
// transpose of an 8 x 8 matrix of 16-bit elements held as mma fragments
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// 16 consecutive elements
template <typename E> __device__ __forceinline__ void load16(const E* p, float* x);
template <> __device__ __forceinline__ void load16<float>(const float* p, float* x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = reinterpret_cast<const float4*>(p)[i];
    x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
  }
}
template <> __device__ __forceinline__ void load16<bf16>(const bf16* p, float* x) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 v = reinterpret_cast<const uint4*>(p)[i];
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[8 * i + 2 * k] = __uint_as_float(u[k] << 16);
      x[8 * i + 2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
    }
  }
}
// hardware 2^x (2^-inf = 0) and log2: relative / absolute error about 2^-22
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// tanh(y): the function itself for fp32 engines and wide caps; else 1 - 2 /
// (2^(2 y log2 e) + 1), absolute error 2.5e-7 (2e-5 of a weight at cap 64)
template <bool EXACT> __device__ __forceinline__ float tanh_of(float y, bool wide) {
  if (EXACT || wide) return tanhf(y);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(ex2(y * (2.f * LOG2E)) + 1.f));   // 1 / inf = 0
  return fmaf(-2.f, r, 1.f);
}

// A row tile of a call: R of the n_new G rows of sequence s (row r: new row r
// / G, head r % G of the key/value head).
struct RowTile {
  int s, sb, n_new, r0, rows;   // rows: 0 for an idle slot
};
template <int R> __device__ __forceinline__ RowTile row_tile(const KvSeqs& q, int64_t slot, int G) {
  RowTile r;
  int tile, se;
  r.s = slot_at(q.cu, q.n, q.T, slot, G, R == 8 ? 3 : 4, 1, tile, r.sb, se);
  r.n_new = se - r.sb;
  r.r0 = tile * R;
  r.rows = tile < 0 ? 0 : max(0, min(R, r.n_new * G - r.r0));
  return r;
}
// floats of one part in the workspace: output rows, then maxima, then sums
template <int D, int R> constexpr int part_floats() { return R * (D + 2); }
// weight of a part with maximum mk; a part without keys has sum and output 0
// (a NaN there, from a row without a finite score, has to stay)
__device__ __forceinline__ float part_weight(float mk, float mm) { return mk == -INFINITY ? 0.f : exp2f(mk - mm); }
__device__ __forceinline__ void add4(float4& a, float f, float4 v) {
  a.x = fmaf(f, v.x, a.x); a.y = fmaf(f, v.y, a.y); a.z = fmaf(f, v.z, a.z); a.w = fmaf(f, v.w, a.w);
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(bf16* p, float4 v) {
  __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
}
__device__ __forceinline__ float over(float v, float l) { return l == 0.f ? 0.f : v / l; }   // nothing in view: zeros

}  // namespace

// A warp's steps: keys of two in flight or in use, values of one.
template <int D> struct KeySlot {
  uint8_t k[32 * D];                  // 32 rows, 16-byte pieces at piece_at()
  float ks[2], vs[2];                 // page scales of the two 16-key halves
  int ok;                             // bit h: half h has a page of the cache
  int pad[3];
};
template <int D> struct WarpSlots {
  KeySlot<D> k[2];
  uint8_t v[32 * D];
};
// Byte place of 16-byte piece c of row r in a slot.  Copies are row after row
// (a warp's cp.async is 512 consecutive bytes: with each lane copying the
// pieces of its own fragments every sector of the values crossed from L2
// twice), the fragments' reads are 4 rows of 32 bytes (values) or 2 rows of 64
// (keys) at a time: the permutation sends both to all 32 banks.
template <int D> __device__ __forceinline__ int piece_at(int r, int c) {
  if (D == 64) return (r >> 1) * 128 + ((r ^ (r >> 2)) & 1) * 64 + ((c ^ (r & 2)) << 4);
  return r * 128 + ((c ^ (((r & 3) << 1) ^ (r & 4))) << 4);
}
constexpr int CW = 4;                 // warps per CTA
// CTAs of an SM, by the registers of the row tile (8 nq rows)
constexpr int cached_ctas(bool f32, int D, int nq) { return (f32 ? 2 : 1) * nq * D <= 128 ? 4 : 3; }
template <int D> constexpr int cached_smem() { return CW * (int)sizeof(WarpSlots<D>); }

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(su32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(su32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// P16: pages of 16 rows (a step's halves have pages of their own).  Each row
// tile's keys are split over ns clusters of nc CTAs; with ns > 1 the clusters
// leave their parts in the workspace and attn_cached_merge_kernel joins them.
// NQ: 8-row groups of a tile.
template <typename E, int D, int NQ, bool P16>
__global__ void __launch_bounds__(CW * 32, cached_ctas(sizeof(E) == 4, D, NQ))
    attn_cached_kernel(CachedArgs<E> a, KvCache c, KvSeqs q, AttnView w, int page_log2, int nc, int ns, int* err) {
  constexpr bool F32 = sizeof(E) == 4;
  constexpr int R = 8 * NQ;                // rows of a tile
  constexpr int NH = F32 ? 2 : 1;          // fp16 parts of a query or weight
  constexpr int NB = D / 64;               // 16-byte pieces of a key row per thread
  // log2 of the largest weight when the reference maximum is the row's, and how far it may fall behind
  constexpr float TOP = 14.f, LAZY = 1.75f;
  SF_PDL_ENTRY();
  extern __shared__ __align__(16) uint8_t ca_smem[];
  __shared__ float sM[CW][R], sL[CW][R];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  WarpSlots<D>& slot = reinterpret_cast<WarpSlots<D>*>(ca_smem)[warp];
  const int G = a.n_heads / c.n_kv, kvh = blockIdx.y;
  const int parts = nc * ns, part = blockIdx.x % parts, rank = blockIdx.x % nc;
  const RowTile rt = row_tile<R>(q, blockIdx.x / parts, G);
  const int s = rt.s, sb = rt.sb, n_new = rt.n_new, r0 = rt.r0, rows = rt.rows;
  const int most = q.table_cols << page_log2;
  int held = q.held[s];
  const bool bad = held < 0 || held > most;
  held = min(max(held, 0), most);
  if (threadIdx.x == 0 && part == 0) {
    if (bad) set_err(err, ERR_BOUNDS);
    if (kvh == 0) report_offsets(q.cu, blockIdx.x / parts, q.n, q.T, err);
  }
  if (rows == 0) return;    // the whole cluster agrees
  // row r of the tile: new row tok(r), head kvh G + head(r); quotients below 2^11 by a rounded reciprocal
  const int tok0 = r0 / G, head0 = r0 - tok0 * G;
  const float inv_G = 1.f / (float)G;
  auto tok_in = [&](int r) { return (int)(((float)(head0 + r) + 0.5f) * inv_G); };
  auto tok = [&](int r) { return tok0 + tok_in(r); };
  auto head = [&](int r) { return head0 + r - tok_in(r) * G; };
  const int pos0 = held - n_new + tok0, pos1 = held - n_new + tok(rows - 1);   // positions of the first and last row
  const int pre = w.prefix ? min(max(w.prefix[s], 0), held) : 0;
  // keys in view of some row: [0, pre) and [lo, hi)
  const int lo = w.left < 0 ? 0 : max(0, pos0 - w.left);
  const int hi = w.right < 0 ? held : max(0, min(held, pos1 + w.right + 1));
  const int np = pos1 < 0 ? 0 : (pre + 31) / 32;
  const int s_lo = max(lo / 32, np), s_hi = pos1 < 0 ? s_lo : max((hi + 31) / 32, s_lo);
  const int steps = np + s_hi - s_lo;
  // this CTA's steps [c0, c1), its warps take them in turn, the last (nearest) first: under a distance bias the
  // running maximum then settles at once
  const int share = (steps + parts - 1) / parts, c0 = min(steps, part * share), c1 = min(steps, c0 + share);

  const int* trow = q.table + (int64_t)s * q.table_cols;
  const int page_mask = (1 << page_log2) - 1;
  const uint32_t page_bytes = (uint32_t)c.n_kv << (page_log2 + (D == 64 ? 6 : 7));
  const uint8_t* kbase = c.k + ((int64_t)kvh << page_log2) * D + 16 * lane;
  const uint8_t* vbase = c.v + ((int64_t)kvh << page_log2) * D + 16 * lane;
  constexpr int RPC = 512 / D;   // rows of a warp's copy; this lane's piece of them:
  const int copy_row = lane / (D / 16), copy_piece = lane % (D / 16);
  auto key_of = [&](int st) { return (st < np ? st : s_lo + st - np) * 32; };
  // table entries of a step's halves (-2: behind the last key)
  auto pages_of = [&](int st, int* p) {
    if (st < c0) return;
    const int j0 = key_of(st);
    p[0] = j0 < held ? trow[j0 >> page_log2] : -2;
    if (P16) p[1] = j0 + 16 < held ? trow[(j0 + 16) >> 4] : -2;
  };
  // a half without a page of the cache reads page 0 and is masked
  auto issue_k = [&](int st, const int* p, KeySlot<D>& x) {
    if (st < c0) return;
    const uint32_t at = (uint32_t)(key_of(st) & page_mask) * D;
    int flags = 0;
#pragma unroll
    for (int hf = 0; hf < (P16 ? 2 : 1); ++hf) {
      const bool there = (unsigned)p[hf] < (unsigned)c.n_pages;
      const uint32_t pi = there ? p[hf] : 0;
      if (!there && p[hf] != -2 && lane == 0) set_err(err, ERR_BOUNDS);
      flags |= (there ? (P16 ? 1 << hf : 3) : 0);
      const uint8_t* src = kbase + (uint64_t)pi * page_bytes + (P16 ? 0 : at);
#pragma unroll
      for (int i = 0; i < (P16 ? 16 : 32) / RPC; ++i)
        cp_async16(x.k + piece_at<D>(16 * hf + RPC * i + copy_row, copy_piece), src + 512 * i);
      if (lane < 2) cp_async4((lane ? x.vs : x.ks) + hf, (lane ? c.vscale : c.kscale) + (int64_t)pi * c.n_kv + kvh);
    }
    if (lane == 0) x.ok = flags;
  };
  auto issue_v = [&](int st, const int* p) {
    if (st < c0) return;
    const uint32_t at = (uint32_t)(key_of(st) & page_mask) * D;
#pragma unroll
    for (int hf = 0; hf < (P16 ? 2 : 1); ++hf) {
      const uint32_t pi = (unsigned)p[hf] < (unsigned)c.n_pages ? p[hf] : 0;
      const uint8_t* src = vbase + (uint64_t)pi * page_bytes + (P16 ? 0 : at);
#pragma unroll
      for (int i = 0; i < (P16 ? 16 : 32) / RPC; ++i)
        cp_async16(slot.v + piece_at<D>(16 * hf + RPC * i + copy_row, copy_piece), src + 512 * i);
    }
  };

  // copies in flight, one group each: keys of the next two steps, values of the next
  const int first = c1 - 1 - warp;
  int pv[2] = {-2, -2}, pn[2] = {-2, -2};   // pages of the next values, of the next keys to be brought
  pages_of(first, pv);
  pages_of(first - CW, pn);
  issue_k(first, pv, slot.k[0]);
  cp_commit();
  issue_k(first - CW, pn, slot.k[1]);
  cp_commit();
  issue_v(first, pv);
  cp_commit();
  pv[0] = pn[0]; pv[1] = pn[1];
  pages_of(first - 2 * CW, pn);

  // ---- queries: B fragments; column g of group j is row 8 j + g of the tile.  The score of a pair stands with the
  // lanes t = row / 2 of its group, so each lane keeps what belongs to its two rows per group
  uint32_t qb[NQ][NH][D / 16][2];
  int pos[NQ][2];
  float slope[NQ][2], f_row[NQ][2];
  const float inv_cap = w.cap > 0.f ? 1.f / w.cap : 0.f, cap_l2 = w.cap * LOG2E;
  const bool wide = w.cap > 64.f;
#pragma unroll
  for (int j = 0; j < NQ; ++j) {
    const int r = 8 * j + g, rr = r < rows ? r : 0;
    const E* qr = a.q + (int64_t)(sb + tok(rr)) * a.ldq + (int64_t)(kvh * G + head(rr)) * D + 16 * t;
    float x[16 * NB];
    float mx = 0.f;
    bool odd = false;
#pragma unroll
    for (int b = 0; b < NB; ++b) load16<E>(qr + 64 * b, x + 16 * b);
#pragma unroll
    for (int i = 0; i < 16 * NB; ++i) {
      if (r >= rows) x[i] = 0.f;
      odd = odd || !isfinite(x[i]);
      mx = fmaxf(mx, fabsf(x[i]));
    }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    // power of two that brings the row's maximum into [2^14, 2^15)
    const int eb = min(253, 268 - (int)(__float_as_uint(mx) >> 23));
    const float up = __uint_as_float((uint32_t)eb << 23);
    // from products to scores over the cap, or to the log2 domain; NaN for a row that is not finite (fp16 may overflow)
    float fr = w.scale * (w.cap > 0.f ? inv_cap : LOG2E) * __uint_as_float((uint32_t)(254 - eb) << 23);
    if (__any_sync(0xffffffffu, odd)) {
      int f = odd;
      f |= __shfl_xor_sync(0xffffffffu, f, 1);
      f |= __shfl_xor_sync(0xffffffffu, f, 2);
      if (f) fr = NAN;
    }
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {   // word k of a key's pieces: 4 dims of this lane
      const float* y = x + 4 * k;
      uint32_t rest0, rest1;
      qb[j][0][k][0] = half_pair(y[0] * up, y[1] * up, rest0);
      qb[j][0][k][1] = half_pair(y[2] * up, y[3] * up, rest1);
      if (F32) {
        qb[j][NH - 1][k][0] = rest0;
        qb[j][NH - 1][k][1] = rest1;
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int mr = 8 * j + 2 * t + i;
      const bool there = mr < rows;
      f_row[j][i] = __shfl_sync(0xffffffffu, fr, 4 * (2 * t + i));
      pos[j][i] = there ? held - n_new + tok(mr) : -1;
      slope[j][i] = w.slopes ? w.slopes[kvh * G + head(there ? mr : 0)] * LOG2E : 0.f;
    }
  }

  auto seen = [&](int key, int at) {
    const int gap = key - at;
    return at >= 0 && (((w.left < 0 || -gap <= w.left) && (w.right < 0 || gap <= w.right)) || key < pre);
  };
  float m[NQ][2], l[NQ][2];   // reference maximum (log2 domain) and this lane's sum of weights
  float o[NQ][D / 16][4];     // dims (rows g, g + 8 of dim tile d: dims g D / 8 + 2 d, + 1) x rows 2 t, 2 t + 1
#pragma unroll
  for (int j = 0; j < NQ; ++j) {
    m[j][0] = m[j][1] = -INFINITY;
    l[j][0] = l[j][1] = 0.f;
#pragma unroll
    for (int d = 0; d < D / 16; ++d) o[j][d][0] = o[j][d][1] = o[j][d][2] = o[j][d][3] = 0.f;
  }

  int sl = 0;
  for (int st = first; st >= c0; st -= CW) {
    cp_wait<2>();   // this step's keys
    __syncwarp();   // scales and flags come from other lanes
    KeySlot<D>& in = slot.k[sl];
    const int j0 = key_of(st);
    // ---- scores: rows g and g + 8 of key tile h are keys j0 + 16 h + (0, 8) + 4 (g % 2) + g / 2
    float sc[NQ][2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float part[NB][NQ][4] = {};   // a chain of products per 64 dims
      float low[NQ][4] = {};        // fp32: of the queries' second parts
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint4 u = *reinterpret_cast<const uint4*>(in.k + piece_at<D>(16 * h + 4 * (g & 1) + (g >> 1), 4 * b + t));
        const uint4 v = *reinterpret_cast<const uint4*>(in.k + piece_at<D>(16 * h + 8 + 4 * (g & 1) + (g >> 1), 4 * b + t));
        const uint32_t kw[4] = {u.x, u.y, u.z, u.w}, kx[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t ka[4] = {cvt_lo(kw[k]), cvt_lo(kx[k]), cvt_hi(kw[k]), cvt_hi(kx[k])};
#pragma unroll
          for (int j = 0; j < NQ; ++j)
#pragma unroll
            for (int p = 0; p < NH; ++p) mma_f16(p ? low[j] : part[b][j], ka, qb[j][p][4 * b + k][0], qb[j][p][4 * b + k][1]);
        }
      }
#pragma unroll
      for (int j = 0; j < NQ; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float hi = NB == 1 ? part[0][j][v] : part[0][j][v] + part[NB - 1][j][v];
          sc[j][h][v] = F32 ? hi + low[j][v] : hi;
        }
    }
    // ---- weights
    const int ok = in.ok;
    // every row sees every key that is there; and all 32 are
    const int j1 = min(j0 + 32, held);
    const bool all_see = pos0 >= 0 && (((w.left < 0 || j0 >= pos1 - w.left) && (w.right < 0 || j1 - 1 <= pos0 + w.right)) || j1 <= pre);
    const bool full = all_see && ok == 3 && j0 + 32 <= held;
    float ks[2], lv[2], iv[2], faint[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h && !P16) {
        ks[1] = ks[0];
        lv[1] = lv[0];
        iv[1] = iv[0];
        faint[1] = faint[0];
        break;
      }
      ks[h] = in.ks[h];
      lv[h] = lg2(in.vs[h]);
      faint[h] = 1.f;
      if (lv[h] < VS_FLOOR) {   // the weights in the outputs alone are less by what the scale is under the floor
        faint[h] = ex2(lv[h] - VS_FLOOR);
        lv[h] = VS_FLOOR;
      }
      iv[h] = lv[h] == lv[h] ? ex2(-lv[h]) : 1.f;   // NaN: the weight has it already
    }
    __syncwarp();   // every lane has read the slot
    issue_k(st - 2 * CW, pn, slot.k[sl]);
    cp_commit();
    const int jl = j0 + 4 * (g & 1) + (g >> 1);   // key of row g of tile 0
    uint32_t pb[NQ][NH][4];                        // B fragments of the weights, 8 keys each
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
      // value (h, 2 e + i): key jl + 16 h + 8 e, row 2 t + i of group j
      float2 y[2][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float2 f = make_float2(f_row[j][0] * ks[h], f_row[j][1] * ks[h]);
#pragma unroll
        for (int e = 0; e < 2; ++e) y[h][e] = __fmul2_rn(make_float2(sc[j][h][2 * e], sc[j][h][2 * e + 1]), f);
      }
      if (w.cap > 0.f) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) y[h][e] = make_float2(cap_l2 * tanh_of<F32>(y[h][e].x, wide), cap_l2 * tanh_of<F32>(y[h][e].y, wide));
      }
      if (w.slopes) {
        const float at0 = (float)(jl - pos[j][0]), at1 = (float)(jl - pos[j][1]);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            y[h][e].x = fmaf(-slope[j][0], fabsf(at0 + (float)(16 * h + 8 * e)), y[h][e].x);
            y[h][e].y = fmaf(-slope[j][1], fabsf(at1 + (float)(16 * h + 8 * e)), y[h][e].y);
          }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e) y[h][e] = __fadd2_rn(y[h][e], make_float2(lv[h], lv[h]));
      if (!full) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int key = jl + 16 * h + 8 * e;
            const bool here = key < held && (ok >> h & 1);
            if (!here || !seen(key, pos[j][0])) y[h][e].x = -INFINITY;
            if (!here || !seen(key, pos[j][1])) y[h][e].y = -INFINITY;
          }
      }
      float mx[2];
      mx[0] = fmaxf(fmaxf(y[0][0].x, y[0][1].x), fmaxf(y[1][0].x, y[1][1].x));
      mx[1] = fmaxf(fmaxf(y[0][0].y, y[0][1].y), fmaxf(y[1][0].y, y[1][1].y));
#pragma unroll
      for (int k = 4; k < 32; k *= 2) {
        mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], k));
        mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], k));
      }
      if (__any_sync(0xffffffffu, mx[0] > m[j][0] + LAZY || mx[1] > m[j][1] + LAZY)) {
        float al[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float mn = fmaxf(m[j][i], mx[i]);
          al[i] = m[j][i] == -INFINITY ? 0.f : ex2(m[j][i] - mn);
          m[j][i] = mn;
          l[j][i] *= al[i];
        }
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
          o[j][d][0] *= al[0]; o[j][d][1] *= al[1];
          o[j][d][2] *= al[0]; o[j][d][3] *= al[1];
        }
      }
      const float2 base = make_float2(m[j][0] == -INFINITY ? 0.f : TOP - m[j][0], m[j][1] == -INFINITY ? 0.f : TOP - m[j][1]);
      float2 sum[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float2 p = __fadd2_rn(y[h][e], base);
          p = make_float2(ex2(p.x), ex2(p.y));
          sum[h] = e ? __fadd2_rn(sum[h], p) : p;
          if (faint[h] != 1.f) p = make_float2(p.x * faint[h], p.y * faint[h]);
          uint32_t rest;
          pb[j][0][2 * h + e] = transpose8(half_pair(p.x, p.y, rest));
          if (F32) pb[j][NH - 1][2 * h + e] = transpose8(rest);
        }
      }
      const float2 both = __ffma2_rn(sum[0], make_float2(iv[0], iv[0]), __fmul2_rn(sum[1], make_float2(iv[1], iv[1])));
      l[j][0] += both.x;
      l[j][1] += both.y;
    }
    cp_wait<1>();   // this step's values
    __syncwarp();
    if (!full) {   // places without a row hold whatever was there: no NaN code may meet a zero weight
      for (int r = copy_row; r < 32; r += RPC)
        if (j0 + r >= held || !(ok >> (r >> 4) & 1)) *reinterpret_cast<uint4*>(slot.v + piece_at<D>(r, copy_piece)) = make_uint4(0, 0, 0, 0);
      __syncwarp();
    }
    if (!all_see) {   // nor may one of a row that is there: the rows that see it get their NaN here
      uint32_t lost = 0;   // keys with a NaN among their values
      for (int r = copy_row; r < 32; r += RPC) {
        uint4* at = reinterpret_cast<uint4*>(slot.v + piece_at<D>(r, copy_piece));
        uint4 x = *at;
        if (clear_nan(x.x) | clear_nan(x.y) | clear_nan(x.z) | clear_nan(x.w)) {
          lost |= 1u << r;
          *at = x;
        }
      }
      for (lost = __reduce_or_sync(0xffffffffu, lost); lost; lost &= lost - 1) {
        const int key = j0 + __ffs(lost) - 1;
#pragma unroll
        for (int j = 0; j < NQ; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (seen(key, pos[j][i])) l[j][i] = NAN;
      }
      __syncwarp();
    }
    // ---- output: rows g, g + 8 of dim tile d are this lane's dims 2 d, 2 d + 1; slots 2 t, 2 t + 1 of 8 keys its rows
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t vr[4][2 * NB];   // this lane's dims of rows 16 h + 4 i + t
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint8_t* row = slot.v + piece_at<D>(16 * h + 4 * i + t, D == 64 ? g >> 1 : g);
        if (D == 64) {
          const uint2 u = *reinterpret_cast<const uint2*>(row + 8 * (g & 1));
          vr[i][0] = u.x;
          vr[i][1] = u.y;
        } else {
          const uint4 u = *reinterpret_cast<const uint4*>(row);
          vr[i][0] = u.x;
          vr[i][1] = u.y;
          vr[i][2 * NB - 2] = u.z;
          vr[i][2 * NB - 1] = u.w;
        }
      }
#pragma unroll
      for (int b = 0; b < 2 * NB; ++b) {   // 4 dims
        const uint32_t vw[4] = {vr[0][b], vr[1][b], vr[2][b], vr[3][b]};
        const uint32_t a01 = __byte_perm(vw[0], vw[1], 0x5140), a23 = __byte_perm(vw[0], vw[1], 0x7362);
        const uint32_t b01 = __byte_perm(vw[2], vw[3], 0x5140), b23 = __byte_perm(vw[2], vw[3], 0x7362);
        const uint32_t va[4] = {cvt_lo(a01), cvt_hi(a01), cvt_lo(b01), cvt_hi(b01)};
        const uint32_t vb[4] = {cvt_lo(a23), cvt_hi(a23), cvt_lo(b23), cvt_hi(b23)};
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
          if (F32) {   // 16 keys by themselves, the second parts first
            float y[2][4];
            mma_f16_new(y[0], va, pb[j][NH - 1][2 * h], pb[j][NH - 1][2 * h + 1]);
            mma_f16_new(y[1], vb, pb[j][NH - 1][2 * h], pb[j][NH - 1][2 * h + 1]);
            mma_f16(y[0], va, pb[j][0][2 * h], pb[j][0][2 * h + 1]);
            mma_f16(y[1], vb, pb[j][0][2 * h], pb[j][0][2 * h + 1]);
#pragma unroll
            for (int d = 0; d < 2; ++d)
#pragma unroll
              for (int v = 0; v < 4; ++v) o[j][2 * b + d][v] += y[d][v];
            continue;
          }
#pragma unroll
          for (int p = 0; p < NH; ++p) {
            mma_f16(o[j][2 * b], va, pb[j][p][2 * h], pb[j][p][2 * h + 1]);
            mma_f16(o[j][2 * b + 1], vb, pb[j][p][2 * h], pb[j][p][2 * h + 1]);
          }
        }
      }
    }
    __syncwarp();   // every lane has read the values
    issue_v(st - CW, pv);
    cp_commit();
    pv[0] = pn[0]; pv[1] = pn[1];
    pages_of(st - 3 * CW, pn);
    sl ^= 1;
  }
  cp_wait<0>();

  // ---- parts of the warps: (max, sum, output) per row
  // this warp's output rows take the place of its slots (all copies have landed)
  constexpr int WARP_FLOATS = (int)sizeof(WarpSlots<D>) / 4;
  float* sO = reinterpret_cast<float*>(ca_smem);   // warp k's rows at k WARP_FLOATS
  static_assert(WARP_FLOATS >= R * D, "output rows fit a warp's slots");
  __syncwarp();
#pragma unroll
  for (int j = 0; j < NQ; ++j)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int k = 4; k < 32; k *= 2) l[j][i] += __shfl_xor_sync(0xffffffffu, l[j][i], k);
      const int r = 8 * j + 2 * t + i;
      if (g == 0) {
        sM[warp][r] = m[j][i];
        sL[warp][r] = l[j][i];
      }
      float2* dst = reinterpret_cast<float2*>(sO + warp * WARP_FLOATS + r * D + g * (D / 8));
#pragma unroll
      for (int d = 0; d < D / 16; ++d) dst[d] = make_float2(o[j][d][i], o[j][d][2 + i]);
    }
  // parts in order, warps first: each row's weights of the parts once, then four outputs per thread
  __shared__ float fw[8][R], cM[R], cL[R], lastL[R];
  __syncthreads();
  if (threadIdx.x < rows) {
    const int r = threadIdx.x;
    float mm = -INFINITY, ll = 0.f;
#pragma unroll
    for (int k = 0; k < CW; ++k) mm = fmaxf(mm, sM[k][r]);
#pragma unroll
    for (int k = 0; k < CW; ++k) {
      fw[k][r] = part_weight(sM[k][r], mm);
      ll = fmaf(fw[k][r], sL[k][r], ll);
    }
    cM[r] = mm;
    cL[r] = ll;
  }
  __syncthreads();
  // four outputs e .. e + 3 of the tile, with their row's maximum and sum: to their place, or to this cluster's part
  float* mine = a.ws ? a.ws + ((int64_t)(blockIdx.x / nc) * c.n_kv + kvh) * part_floats<D, R>() : nullptr;
  auto store = [&](int e, float4 v, float mm, float ll) {
    const int r = e / D;
    if (ns > 1) {
      *reinterpret_cast<float4*>(mine + e) = v;
      if (e % D == 0) {
        mine[R * D + r] = mm;
        mine[R * D + R + r] = ll;
      }
    } else {
      const float inv = over(1.f, ll);
      store4(a.out + (int64_t)(sb + tok(r)) * a.ldo + (int64_t)(kvh * G + head(r)) * D + e % D,
             make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
    }
  };
  for (int e = 4 * threadIdx.x; e < rows * D; e += CW * 128) {
    const int r = e / D;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < CW; ++k) add4(acc, fw[k][r], *reinterpret_cast<const float4*>(sO + k * WARP_FLOATS + e));
    if (nc == 1) store(e, acc, cM[r], cL[r]);
    else *reinterpret_cast<float4*>(sO + e) = acc;   // read by this thread alone
  }
  if (nc == 1) return;
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  auto at_rank = [](const float* p, int r) -> uint32_t {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(su32(p)), "r"(r));
    return at;
  };
  auto peer = [&](const float* p, int r) -> float {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at_rank(p, r)) : "memory");
    return v;
  };
  // each CTA finishes its share of the outputs
  if (threadIdx.x < rows) {
    const int r = threadIdx.x;
    float mk[8], mm = -INFINITY, ll = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      mk[k] = k < nc ? peer(cM + r, k) : -INFINITY;
      mm = fmaxf(mm, mk[k]);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      fw[k][r] = part_weight(mk[k], mm);
      if (k < nc) ll = fmaf(fw[k][r], peer(cL + r, k), ll);
    }
    sM[0][r] = mm;
    lastL[r] = ll;
  }
  __syncthreads();
  for (int e = 4 * (rank * CW * 32 + threadIdx.x); e < rows * D; e += nc * CW * 128) {
    const int r = e / D;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < nc; ++k) {
      float4 v;
      asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                   : "r"(at_rank(sO + e, k))
                   : "memory");
      add4(acc, fw[k][r], v);
    }
    store(e, acc, sM[0][r], lastL[r]);
  }
  // no CTA leaves while another may still read its shared memory
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Joins the ns parts of each row tile in order.
template <typename E, int D, int R>
__global__ void __launch_bounds__(256) attn_cached_merge_kernel(CachedArgs<E> a, KvSeqs q, int n_kv, int ns) {
  SF_PDL_ENTRY();
  const int G = a.n_heads / n_kv, kvh = blockIdx.y;
  const RowTile rt = row_tile<R>(q, blockIdx.x, G);
  const int64_t stride = (int64_t)n_kv * part_floats<D, R>();
  const float* p = a.ws + ((int64_t)blockIdx.x * ns * n_kv + kvh) * part_floats<D, R>();
  for (int e = threadIdx.x; e < rt.rows * D; e += 256) {
    const int r = e / D, rr = rt.r0 + r;
    float mm = -INFINITY, ll = 0.f, acc = 0.f;
    for (int k = 0; k < ns; ++k) mm = fmaxf(mm, p[k * stride + R * D + r]);
    for (int k = 0; k < ns; ++k) {
      const float f = part_weight(p[k * stride + R * D + r], mm);
      ll = fmaf(f, p[k * stride + R * D + R + r], ll);
      acc = fmaf(f, p[k * stride + e], acc);
    }
    a.out[(int64_t)(rt.sb + rr / G) * a.ldo + (int64_t)(kvh * G + rr % G) * D + e % D] = from_f<E>(acc * over(1.f, ll));
  }
}

namespace {
int g_cached_sms = 148;
// clusters of 8 CTAs resident at once: fp32 or not, head dim 128 or not, tiles of 16 rows or not
int g_cached_clusters[2][2][2] = {{{48, 48}, {48, 48}}, {{48, 48}, {48, 48}}};

// Rows of a tile, and how a call's keys are split: over clusters of nc CTAs
// (joined on chip), and over ns clusters (joined by a second kernel) where
// the row tiles are so few that clusters alone leave SMs idle.
struct Plan {
  int R, nc, ns;
  int64_t tiles;   // row tiles, idle ones included
};
Plan cached_plan(bool f32, int64_t T, int n, int G, int n_kv, int D, int max_len, bool have_ws) {
  Plan p{};
  // more than 8 rows a sequence: tiles of 16 read the keys once for twice the rows (fp32, D = 128: too many registers)
  p.R = (!f32 || D == 64) && T * G > (int64_t)8 * n ? 16 : 8;
  p.tiles = T * G / p.R + n;
  // (row tile, head) units with work where the rows are spread evenly, and CTAs resident at once
  const int64_t live = std::max<int64_t>(1, std::min<int64_t>(n, T));
  const int64_t units = live * ((T * G + live * p.R - 1) / (live * p.R)) * n_kv;
  const int64_t slots = (int64_t)g_cached_sms * cached_ctas(f32, D, p.R / 8);
  p.nc = p.ns = 1;
  // idle SMs: as many CTAs as are resident, of 64 keys or more (undivided, in 2, 4, 8; us: 128 units of up to 1000 keys 11.6,
  // 10.3, 8.8, 14.1; 64 of 8000 80, 52, 36, 31; 8 of 376 6.4, 6.9, 6.1, 6.1; 512 of up to 1125 25.5, 30.6, 43, 72).  All SMs
  // busy: for a smaller last wave, where a CTA keeps 2048 keys (512 of up to 8190 147, 140, 138, 157; 1024 of up to 8000
  // 235, 221, 227, 270)
  while (p.nc < 8 && ((units * p.nc * 2 <= slots && max_len >= p.nc * 128) || (units * p.nc < 2 * slots && max_len >= (int64_t)p.nc * 4096)))
    p.nc *= 2;
  // more clusters than this kernel has resident at once would wait for a second round (180001 keys, 8 heads of 128: one row
  // 73 us with 6 clusters of 8 a head, 94 us with 9; 13 rows, 3 CTAs an SM, 93 us with 6 and 124 us with 8)
  if (have_ws && p.nc == 8) p.ns = (int)std::min<int64_t>(g_cached_clusters[f32][D == 128][p.R == 16] / units, max_len / (8 * 512));
  if (p.ns < 2) p.ns = 1;
  return p;
}

template <typename E, int D, int NQ, bool P16>
cudaError_t launch(const CachedArgs<E>& a, const KvCache& c, const KvSeqs& q, const AttnView& w, const Plan& p, int* err,
                   cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.tiles * p.nc * p.ns), c.n_kv);
  cfg.blockDim = dim3(CW * 32);
  cfg.dynamicSmemBytes = cached_smem<D>();
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  int na = 0;
  attr[na].id = cudaLaunchAttributeClusterDimension;
  attr[na].val.clusterDim.x = p.nc;
  attr[na].val.clusterDim.y = 1;
  attr[na].val.clusterDim.z = 1;
  ++na;
  if (g_launch_pdl) {
    attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[na].val.programmaticStreamSerializationAllowed = 1;
    ++na;
  }
  cfg.attrs = attr;
  cfg.numAttrs = na;
  int page_log2 = 4;
  while ((1 << page_log2) < c.page) ++page_log2;
  CK_LAUNCH(cudaLaunchKernelEx(&cfg, attn_cached_kernel<E, D, NQ, P16>, a, c, q, w, page_log2, p.nc, p.ns, err));
  if (p.ns > 1)
    CK_LAUNCH(launch_k(attn_cached_merge_kernel<E, D, 8 * NQ>, dim3((unsigned)p.tiles, c.n_kv), dim3(256), 0, st, a, q, c.n_kv,
                       p.ns));
  return cudaGetLastError();
}

template <typename E, int D>
cudaError_t launch_d(const CachedArgs<E>& a, const KvCache& c, const KvSeqs& q, const AttnView& w, int* err, cudaStream_t st) {
  constexpr int NQ = sizeof(E) == 4 && D == 128 ? 1 : 2;   // groups of the larger tile
  const Plan p = cached_plan(sizeof(E) == 4, q.T, q.n, a.n_heads / c.n_kv, c.n_kv, D, a.max_len, a.ws != nullptr);
  if (p.R == 16)
    return c.page == 16 ? launch<E, D, NQ, true>(a, c, q, w, p, err, st) : launch<E, D, NQ, false>(a, c, q, w, p, err, st);
  return c.page == 16 ? launch<E, D, 1, true>(a, c, q, w, p, err, st) : launch<E, D, 1, false>(a, c, q, w, p, err, st);
}

template <typename E, int D> cudaError_t allow_smem() {
  constexpr int NQ = sizeof(E) == 4 && D == 128 ? 1 : 2;
  const void* f[4] = {(const void*)attn_cached_kernel<E, D, 1, true>, (const void*)attn_cached_kernel<E, D, 1, false>,
                      (const void*)attn_cached_kernel<E, D, NQ, true>, (const void*)attn_cached_kernel<E, D, NQ, false>};
  for (const void* k : f) {
    const cudaError_t r = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, cached_smem<D>());
    if (r != cudaSuccess) return r;
  }
  return cudaSuccess;
}
// the lesser of both page forms
template <typename E, int D, int NQ> cudaError_t resident_clusters() {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(8);
  cfg.blockDim = dim3(CW * 32);
  cfg.dynamicSmemBytes = cached_smem<D>();
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 8;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0, n16 = 0;
  cudaError_t r = cudaOccupancyMaxActiveClusters(&n, attn_cached_kernel<E, D, NQ, false>, &cfg);
  if (r == cudaSuccess) r = cudaOccupancyMaxActiveClusters(&n16, attn_cached_kernel<E, D, NQ, true>, &cfg);
  if (r == cudaSuccess) g_cached_clusters[sizeof(E) == 4][D == 128][NQ == 2] = std::min(n, n16);
  return r;
}
}  // namespace

size_t attention_cached_ws_bytes(bool f32, int64_t T, int n, int n_heads, int n_kv, int D, int max_len) {
  const Plan p = cached_plan(f32, T, n, n_heads / n_kv, n_kv, D, max_len, true);
  return p.ns == 1 ? 0 : (size_t)(p.tiles * n_kv * p.ns * p.R * (D + 2)) * 4;
}

template <typename E>
cudaError_t launch_attention_cached(const CachedArgs<E>& a, const KvCache& c, const KvSeqs& q, const AttnView& w, int* err,
                                    cudaStream_t st) {
  return c.D == 64 ? launch_d<E, 64>(a, c, q, w, err, st) : launch_d<E, 128>(a, c, q, w, err, st);
}
template cudaError_t launch_attention_cached<float>(const CachedArgs<float>&, const KvCache&, const KvSeqs&, const AttnView&,
                                                    int*, cudaStream_t);
template cudaError_t launch_attention_cached<bf16>(const CachedArgs<bf16>&, const KvCache&, const KvSeqs&, const AttnView&,
                                                   int*, cudaStream_t);

cudaError_t attention_cached_init_attributes() {
  int dev = 0, n = 0;
  cudaError_t r = cudaGetDevice(&dev);
  if (r == cudaSuccess) r = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  if (r == cudaSuccess && n > 0) g_cached_sms = n;
  if (r == cudaSuccess) r = allow_smem<float, 64>();
  if (r == cudaSuccess) r = allow_smem<float, 128>();
  if (r == cudaSuccess) r = allow_smem<bf16, 64>();
  if (r == cudaSuccess) r = allow_smem<bf16, 128>();
  if (r == cudaSuccess) r = resident_clusters<bf16, 64, 1>();
  if (r == cudaSuccess) r = resident_clusters<bf16, 64, 2>();
  if (r == cudaSuccess) r = resident_clusters<bf16, 128, 1>();
  if (r == cudaSuccess) r = resident_clusters<bf16, 128, 2>();
  if (r == cudaSuccess) r = resident_clusters<float, 64, 1>();
  if (r == cudaSuccess) r = resident_clusters<float, 64, 2>();
  if (r == cudaSuccess) r = resident_clusters<float, 128, 1>();   // (its tiles have 8 rows at any size)
  return r;
}

}  // namespace sf
