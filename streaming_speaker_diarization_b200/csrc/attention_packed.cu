// Attention of packed sequences with capped scores, distance bias, window,
// prefix and document mask (attn_view.cuh has the formulas; each sequence is
// a document) for fp32 engines: fp32 products, softmax and sums.
//
// One CTA = 128 query rows of one sequence x one head, 256 threads as 16 x 16:
// thread (ty, tx) holds the scores of rows 8 ty .. + 7 and keys tx, tx + 16, ..
// of each 64-key tile and the outputs of its rows at D / 16 dims, as pairs of rows:
// an fp32 pair is one multiply-add, its other operand (a key's or a value's
// element) doubled.  Q and the weights lie transposed in shared memory, so all
// operands are 16-byte reads.  The next tile's keys come (cp.async) under this
// tile's weights and output product, its values under the next scores: two
// barriers per tile and one buffer each.  The running maximum and sum
// of a row are shared by the 16 threads of a row group with shuffles.  Only the
// key tiles that some row of the CTA sees are read: the prefix's, then the
// window's.
//
// Few query tiles of long sequences leave SMs idle, or busy with the longest
// tile alone: the key tiles are then split over a cluster of 2 or 4 CTAs whose
// (max, sum, output) parts are joined in distributed shared memory (4 clips of
// up to 1125 rows, 8 heads of 64, causal: 204 us undivided, 126 halved, 119 in
// four; eight were slower than four).
//
// Masked keys get weight 0 by selection, not by a product, except that
// 0 x V is added to rows that do not see a key of a tile: a row whose result
// is not finite although its sum is, and that sees no such value, is computed
// again from its own keys (attn_packed_row.cuh).
#include "attn_common.cuh"
#include "attn_packed_row.cuh"
#include "attn_view.cuh"
#include "layers.h"
#include "tcgen05.cuh"

namespace sf {
namespace {

constexpr int PR = 128;  // query rows per CTA (2^7)
constexpr int NR = PR / 16;   // rows of a thread
constexpr int PK = 64;   // keys per tile

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }

template <int D>
struct PackedSmem {
  static constexpr int QT = 0;                          // [D][PR + 4]
  static constexpr int K = QT + D * (PR + 4);           // [PK][D + 4]
  static constexpr int V = K + PK * (D + 4);            // [PK][D]
  static constexpr int P = V + PK * D;                  // [PK][PR + 4] weights
  static constexpr int BYTES = (P + PK * (PR + 4)) * 4;
};

}  // namespace

template <int D>
__global__ void __launch_bounds__(256, D == 64 ? 2 : 1) attn_packed_f32_kernel(const __grid_constant__ PackedArgs<float> a,
                                                               const __grid_constant__ AttnView w, int nc, int* err) {
  SF_PDL_ENTRY();
  extern __shared__ float ps_smem[];
  float* sQ = ps_smem + PackedSmem<D>::QT;
  float* sK = ps_smem + PackedSmem<D>::K;
  float* sV = ps_smem + PackedSmem<D>::V;
  float* sP = ps_smem + PackedSmem<D>::P;
  __shared__ int redo[PR];
  constexpr int LDT = PR + 4, LDK = D + 4, ND = D / 16;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int h = blockIdx.y, kvh = h / (a.n_heads / a.n_kv), rank = blockIdx.x % nc;
  int tile;
  int sb, se;
  const unsigned slot = (gridDim.x - 1 - blockIdx.x) / nc;
  const int s = slot_at(a.cu, a.n, a.T, slot, 1, 7, 1, tile, sb, se);
  if (tid == 0 && h == 0) report_offsets(a.cu, slot, a.n, a.T, err);
  const int S = se - sb, i0 = tile * PR;
  if (tile < 0 || i0 >= S) return;   // the whole cluster agrees
  const int rows = min(PR, S - i0);
  const int pre = w.prefix ? min(max(w.prefix[s], 0), S) : 0;
  // key tiles [0, np) hold the prefix, [t_lo, t_hi) the rows' windows
  const int np = (pre + PK - 1) / PK;
  const int lo = w.left < 0 ? 0 : max(0, i0 - w.left);
  const int hi = w.right < 0 ? S : (int)min((int64_t)S, (int64_t)i0 + rows + w.right);
  const int t_lo = max(lo / PK, np), t_hi = max((hi + PK - 1) / PK, t_lo);
  const int nt = np + t_hi - t_lo;
  const int share = (nt + nc - 1) / nc, tt0 = min(nt, rank * share), tt1 = min(nt, tt0 + share);   // this CTA's of the list
  const float slope = w.slopes ? w.slopes[h] * LOG2E : 0.f;

  // one row per thread of a warp: the transposed stores hit 32 banks, and the
  // 16-byte pieces of a row that consecutive steps read share L1 lines
  for (int c = tid; c < PR * D / 4; c += 256) {
    const int r = c % PR, d = (c / PR) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < rows) v = load4(a.q + (int64_t)(sb + i0 + r) * a.ldq + h * D + d);
    sQ[d * LDT + r] = v.x; sQ[(d + 1) * LDT + r] = v.y; sQ[(d + 2) * LDT + r] = v.z; sQ[(d + 3) * LDT + r] = v.w;
  }
  if (tid < PR) redo[tid] = 0;

  float2 o[NR / 2][ND];   // rows 8 ty + 2 r, + 1
  float m[NR], l[NR];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int d = 0; d < ND; ++d) o[r / 2][d] = make_float2(0.f, 0.f);
  }
  auto key_of = [&](int tt) { return (tt < np ? tt : t_lo + tt - np) * PK; };
  // rows of a tile of keys or values: 16-byte copies, zeros behind the sequence
  auto bring = [&](float* dst, int ld, const float* src, int64_t lds, int tt) {
    if (tt < tt1) {
      const int j0 = key_of(tt);
      for (int c = tid; c < PK * D / 4; c += 256) {
        const int r = c / (D / 4), d = (c % (D / 4)) * 4, there = j0 + r < S ? 16 : 0;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(su32(dst + r * ld + d)),
                     "l"(src + (int64_t)(sb + (there ? j0 + r : 0)) * lds + kvh * D + d), "r"(there)
                     : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto landed = [] { asm volatile("cp.async.wait_group 0;" ::: "memory"); };
  bring(sK, LDK, a.k, a.ldk, tt0);
  landed();
  __syncthreads();
  bring(sV, D, a.v, a.ldv, tt0);
  for (int tt = tt0; tt < tt1; ++tt) {
    const int j0 = key_of(tt);
    // the warp's rows are 16: it leaves out a tile that they do not see
    const int w0 = i0 + 16 * (tid >> 5), w1 = w0 + 15;
    const bool some = w0 < S && (j0 < pre || ((w.left < 0 || j0 + PK - 1 >= w0 - w.left) && (w.right < 0 || j0 <= w1 + w.right)));
    float2 sc[NR / 2][4] = {};
    if (some)
#pragma unroll 2
    for (int d = 0; d < D; d += 4) {
      float ka[4][4];   // keys tx + 16 c, dims d ..
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float4 k4 = *reinterpret_cast<const float4*>(sK + (tx + 16 * c) * LDK + d);
        ka[c][0] = k4.x; ka[c][1] = k4.y; ka[c][2] = k4.z; ka[c][3] = k4.w;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int r = 0; r < NR / 2; r += 2) {
          const float4 q4 = *reinterpret_cast<const float4*>(sQ + (d + e) * LDT + NR * ty + 2 * r);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            sc[r][c] = __ffma2_rn(make_float2(q4.x, q4.y), make_float2(ka[c][e], ka[c][e]), sc[r][c]);
            sc[r + 1][c] = __ffma2_rn(make_float2(q4.z, q4.w), make_float2(ka[c][e], ka[c][e]), sc[r + 1][c]);
          }
        }
    }
    landed();
    __syncthreads();   // the values are there, the keys are read
    bring(sK, LDK, a.k, a.ldk, tt + 1);
    if (some) {
    const bool whole = j0 + PK <= S && (((w.left < 0 || j0 >= w1 - w.left) && (w.right < 0 || j0 + PK - 1 <= w0 + w.right)) ||
                                        j0 + PK <= pre);
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const int i = i0 + NR * ty + r;
      float x[4], mx = -INFINITY;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int j = j0 + tx + 16 * c, gap = j - i;
        x[c] = capped_l2((r & 1 ? sc[r / 2][c].y : sc[r / 2][c].x) * w.scale, w.cap);
        if (slope != 0.f) x[c] -= slope * fabsf((float)gap);
        if (!whole) {
          const bool seen = j < S && (((w.left < 0 || -gap <= w.left) && (w.right < 0 || gap <= w.right)) || j < pre);
          x[c] = seen ? x[c] : -INFINITY;
        }
        mx = fmaxf(mx, x[c]);
      }
#pragma unroll
      for (int k = 8; k > 0; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
      const float mn = fmaxf(m[r], mx), base = mn == -INFINITY ? 0.f : mn;
      const float al = ex2_approx(m[r] - base);
      float sum = 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        x[c] = ex2_approx(x[c] - base);
        sum += x[c];
        if (r & 1) sc[r / 2][c].y = x[c]; else sc[r / 2][c].x = x[c];
      }
      l[r] = l[r] * al + sum;
      m[r] = mn;
#pragma unroll
      for (int d = 0; d < ND; ++d)
        if (r & 1) o[r / 2][d].y *= al; else o[r / 2][d].x *= al;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int r = 0; r < NR / 2; r += 2)
        *reinterpret_cast<float4*>(sP + (tx + 16 * c) * LDT + NR * ty + 2 * r) =
            make_float4(sc[r][c].x, sc[r][c].y, sc[r + 1][c].x, sc[r + 1][c].y);
    __syncwarp();   // a row group's 16 threads are one half of a warp
#pragma unroll 4
    for (int j = 0; j < PK; ++j) {
      float2 p[NR / 2];
#pragma unroll
      for (int r = 0; r < NR / 2; r += 2) {
        const float4 t = *reinterpret_cast<const float4*>(sP + j * LDT + NR * ty + 2 * r);
        p[r] = make_float2(t.x, t.y);
        p[r + 1] = make_float2(t.z, t.w);
      }
#pragma unroll
      for (int d4 = 0; d4 < ND; d4 += 4) {
        const float4 v4 = *reinterpret_cast<const float4*>(sV + j * D + d4 * 16 + 4 * tx);
        const float va[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
          for (int r = 0; r < NR / 2; ++r) o[r][d4 + d] = __ffma2_rn(p[r], make_float2(va[d], va[d]), o[r][d4 + d]);
      }
    }
    }
    landed();
    __syncthreads();   // the next keys are there, the values are read
    bring(sV, D, a.v, a.ldv, tt + 1);
  }
  landed();
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int k = 8; k > 0; k >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], k);
  // row `row` of the tile: four outputs at dim d, the row's sum
  auto store = [&](int row, int d, float4 v, float lt) {
    const float inv = lt > 0.f ? 1.f / lt : (lt == 0.f ? 0.f : lt);   // nothing in view: zeros; NaN stays NaN
    v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
    store4(a.out + (int64_t)(sb + i0 + row) * a.ldo + h * D + d, v);
    if (isfinite(lt) && !(isfinite(v.x) && isfinite(v.y) && isfinite(v.z) && isfinite(v.w))) redo[row] = 1;
  };
  auto part_of = [&](int r, int d4) {
    const float2 *y = o[r / 2] + d4;
    return r & 1 ? make_float4(y[0].y, y[1].y, y[2].y, y[3].y) : make_float4(y[0].x, y[1].x, y[2].x, y[3].x);
  };
  if (nc == 1) {
#pragma unroll
    for (int r = 0; r < NR; ++r)
      if (NR * ty + r < rows)
#pragma unroll
        for (int d4 = 0; d4 < ND; d4 += 4) store(NR * ty + r, d4 * 16 + 4 * tx, part_of(r, d4), l[r]);
  } else {
    __syncthreads();   // the operands are no longer read: their place takes this CTA's part
    float *pO = ps_smem, *pM = ps_smem + PR * D, *pL = pM + PR;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const int row = NR * ty + r;
#pragma unroll
      for (int d4 = 0; d4 < ND; d4 += 4) *reinterpret_cast<float4*>(pO + row * D + d4 * 16 + 4 * tx) = part_of(r, d4);
      if (tx == 0) {
        pM[row] = m[r];
        pL[row] = l[r];
      }
    }
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    auto at_rank = [](const float* p, int k) -> uint32_t {
      uint32_t at;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(su32(p)), "r"(k));
      return at;
    };
    // each CTA finishes its share of the rows, the parts in order; a part without a key has maximum -inf
    for (int e = tid; e < PR / nc * (D / 4); e += 256) {
      const int row = rank * (PR / nc) + e / (D / 4), d = e % (D / 4) * 4;
      if (row >= rows) break;
      float mk[4], mm = -INFINITY, lt = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        mk[k] = -INFINITY;
        if (k < nc) asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(mk[k]) : "r"(at_rank(pM + row, k)) : "memory");
        mm = fmaxf(mm, mk[k]);
      }
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (k >= nc) break;
        const float f = mk[k] == -INFINITY ? 0.f : ex2_approx(mk[k] - mm);
        float lk;
        float4 v;
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(lk) : "r"(at_rank(pL + row, k)) : "memory");
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                     : "r"(at_rank(pO + row * D + d, k))
                     : "memory");
        lt = fmaf(f, lk, lt);
        acc.x = fmaf(f, v.x, acc.x); acc.y = fmaf(f, v.y, acc.y); acc.z = fmaf(f, v.z, acc.z); acc.w = fmaf(f, v.w, acc.w);
      }
      store(row, d, acc, lt);
    }
    // no CTA leaves while another may still read its shared memory
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  __syncthreads();
  for (int row = tid >> 5; row < rows; row += 8)
    if (redo[row]) attn_packed_row<float, D>(a, w, h, kvh, sb, S, i0 + row, pre, slope);
}

namespace {
int g_simt_sms = 148;
}

template <int D>
static cudaError_t launch_simt(const PackedArgs<float>& a, const AttnView& w, int* err, cudaStream_t st) {
  const int64_t slots = a.T / PR + a.n, units = slots * a.n_heads;
  int nc = 1;
  while (nc < 4 && units * nc < 8 * g_simt_sms && a.T / a.n >= nc * 128) nc *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(slots * nc), a.n_heads);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = PackedSmem<D>::BYTES;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  int na = 0;
  attr[na].id = cudaLaunchAttributeClusterDimension;
  attr[na].val.clusterDim.x = nc;
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
  CK_LAUNCH(cudaLaunchKernelEx(&cfg, attn_packed_f32_kernel<D>, a, w, nc, err));
  return cudaGetLastError();
}

template <>
cudaError_t launch_attention_packed<float>(const PackedArgs<float>& a, int D, const AttnView& w, int* err, cudaStream_t st) {
  return D == 64 ? launch_simt<64>(a, w, err, st) : launch_simt<128>(a, w, err, st);
}

cudaError_t attention_packed_init_attributes() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) == cudaSuccess && cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && n > 0)
    g_simt_sms = n;
  cudaError_t r = cudaFuncSetAttribute(attn_packed_f32_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       PackedSmem<64>::BYTES);
  if (r != cudaSuccess) return r;
  return cudaFuncSetAttribute(attn_packed_f32_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              PackedSmem<128>::BYTES);
}

}  // namespace sf
