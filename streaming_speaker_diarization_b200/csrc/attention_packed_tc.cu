// Attention of packed sequences with capped scores, distance bias, window,
// prefix and document mask (attn_view.cuh has the formulas), bf16 operands on
// the Blackwell tensor cores.
//
// One CTA = 128 query rows of one sequence x one head.  Per 64-key tile t:
//   S_t = Q K^T      M 128, N 64, K D     TMEM columns 64 (t % NG) ..
//   O += P_t V       M 128, N D, K 64     TMEM columns 64 NG ..
// P_t (bf16) overwrites the first half of S_t's columns and is the A operand
// straight from TMEM; O stays in TMEM over all key tiles.  Warps: 0 loads Q,
// then K and V tiles into one ring with TMA; 1 issues the MMAs, the scores NG
// tiles ahead; 4 .. run the softmax, thread = query row = TMEM lane, NG groups of
// four warps that take the key tiles in turn, each with a score buffer of its
// own.  Two groups, two CTAs per SM: a group's next scores and last output
// product are made while the other group and the other CTA compute.  Heads of
// 64 with many query tiles run one group, four CTAs per SM.  (Measured, causal,
// heads of 64, one group against two: 16 x 1125 rows 60 and 61 us, 4 x 2000 x 32
// heads 122 and 140, 64 x 322 40 and 49; one sequence of 4000 79 and 51.  Two
// query tiles per CTA, one CTA per SM, took 1.1 .. 1.2 times as long in all but
// the longest.)
// Few query tiles leave SMs idle, or busy with the longest alone: the key tiles
// are then split over a cluster of 2 or 4 CTAs, whose (max, sum, output) parts
// are joined in distributed shared memory.
//
// The running maximum of a row is a reference that moves only when the new
// maximum exceeds it by 2^8: weights stay below 256 (bf16 rounds them alike at
// any size, the fp32 sums hold them), and O's rescaling, a TMEM round trip, is
// rare.  Weights are rounded to bf16 for P V, their sum is of the unrounded
// ones.  The groups hand the reference on from tile to tile.  Only key tiles
// that some row sees are visited, and only tiles that some row sees in part are
// masked.
//
// A capped score costs no special-function work while |s / cap| <= 3/4 holds
// for a warp's rows: tanh(y) / y as a polynomial of degree 4 in y^2 (our own
// fit at Chebyshev nodes, relative error 5.9e-7 on [0, 3/4]), with the score
// factor, the cap and log2 e in its coefficients, so that the exponent is one
// more multiply-add.  Other tiles, and caps whose coefficients leave fp32's
// range, have their scores rewritten in TMEM: by the polynomial in s / cap
// where that is in its range, else by 1 - 2 / (2^(2 y log2 e) + 1), whose
// absolute error of 2.5e-7 is small against a score of that size.
//
// 0 x V of rows that do not see a key of their tile would carry an infinity or
// NaN over: a row whose result is not finite although its sum is, and that sees
// no such value, is computed again from its own keys (attn_packed_row.cuh).
// Rows of the last value tile that lie behind the sequence are cleared by warp 3
// first.  Every wait is bounded: a wait that runs out raises ERR_TIMEOUT, the CTA
// drains its own copies and frees its TMEM.
#include "attn_common.cuh"
#include "attn_packed_row.cuh"
#include "attn_view.cuh"
#include "layers.h"
#include "tcgen05.cuh"

namespace sf {
namespace {

constexpr int TQ = 128;   // rows of a query tile
constexpr int TK = 64;    // keys of a tile
constexpr float LAZY = 8.f;   // log2 of the largest weight before the reference maximum moves
constexpr float FAR = 40.f;   // log2 of how far a magnitude may stand above a row's largest score as its reference

template <int NG, int D>
struct PTc {
  static constexpr int QTILE = 128 * D * 2;             // D / 64 atoms of 128 rows x 128 bytes
  static constexpr int TILE = TK * D * 2;               // K or V tile: D / 64 atoms of 64 rows x 128 bytes
  static constexpr int NS = NG == 1 || D == 128 ? 4 : 8;   // ring slots (K and V tiles in turn)
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_RING = QTILE;
  static constexpr int OFF_BAR = OFF_RING + NS * TILE;
  static constexpr int OFF_X = OFF_BAR + 512;           // [2 groups][128] references handed on, then sums
  static constexpr int SMEM = 1024 + OFF_X + (NG == 2 ? 2 * 128 * 8 : 0);
  static constexpr int THREADS = 128 + 128 * NG;
  static constexpr int PER_SM = NG == 2 ? 2 : 4;        // CTAs of an SM
  static constexpr int REGS = 65536 / (THREADS * PER_SM) / 8 * 8;   // a thread is launched with
  // registers: the service warps give theirs to the softmax warps, within what the block is launched with
  static constexpr int REG_LOW = NG == 2 ? 48 : 32, REG_HIGH = 96;
  static_assert(128 * REG_LOW + 128 * NG * REG_HIGH <= THREADS * REGS, "register split");
  static constexpr int TMEM = 512 / PER_SM;             // columns: 64 NG + D, a power of two
  static_assert(64 * NG + D <= TMEM && PER_SM * (SMEM + 1024) <= 233472, "TMEM and shared memory of an SM");
  // a cluster's part: output rows (padded: a thread writes a row), maxima, sums, flags, over Q and the ring
  static constexpr int LDO = D + 4;
  static_assert((128 * LDO + 3 * 128) * 4 <= OFF_BAR, "parts fit");
};

// One product step each, ACC: added to the accumulator.  Called by one elected
// lane from warp-uniform code: descriptors and addresses then come from uniform
// registers (the issuing warp shares its scheduler with the softmax warps, and
// moving them there per step made the issue of a step cost ~70 clocks).
template <bool ACC> __device__ __forceinline__ void mma_ss(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "n"(ACC ? 1 : 0)
      : "memory");
}
template <bool ACC> __device__ __forceinline__ void mma_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "l"(bdesc), "r"(idesc), "n"(ACC ? 1 : 0)
      : "memory");
}
// mbar_wait, with a look at the barrier before the clock is read: most waits of
// the product warp find their phase done
__device__ __forceinline__ bool wait_for(uint64_t* b, uint32_t parity, volatile int* abort_flag) {
  return mbar_try_wait(b, parity) || mbar_wait(b, parity, abort_flag);
}
// largest of three, of three magnitudes
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float r;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {"
      "%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {"
      "%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// MN-major B operand with D columns: 64-column atoms TK rows x 128 bytes apart
__device__ __forceinline__ uint64_t v_desc(uint32_t saddr) {
  const uint64_t d = sw128_desc_mn(saddr);
  return (d & ~((uint64_t)0x3fff << 16)) | ((uint64_t)(TK * 128 >> 4) << 16);
}

// tanh(y) / y = sum c_k y^2k on |y| <= TANH_Y
constexpr float TANH_Y = 0.75f;
constexpr float tanh_c(int k) {
  constexpr float c[5] = {9.99999463558197e-1f, -3.332834839820862e-1f, 1.3259831070899963e-1f, -5.008019134402275e-2f,
                          1.2950727716088295e-2f};
  return c[k];
}
// coefficients of the capped score in the log2 domain, s sum pc_k s^2k for |s / cap| <= TANH_Y; false where their powers of
// scale / cap leave fp32's range (caps far from the scores' size: at scale 1/8 below 1e-5 and above 1500) or there is no cap.
// Judged on the host: by each thread from its own registers it cost tiles without a cap too (64 windows 34.7 against 32.1 us)
__host__ __device__ __forceinline__ bool cap_coefficients(const AttnView& w, float* pc) {
  const float inv_cap = w.cap > 0.f ? w.scale / w.cap : 0.f;
  float y = w.cap * LOG2E * inv_cap;
#pragma unroll
  for (int k = 0; k < 5; ++k) {
    pc[k] = tanh_c(k) * y;
    y *= inv_cap * inv_cap;
  }
  return pc[4] > 1e-36f && pc[4] < 1e36f && pc[0] > 1e-36f && pc[0] < 1e36f;
}
// tanh at any argument: the exponential's form has an absolute error, which is too much for a small one
__device__ __forceinline__ float tanh_any(float y) {
  const float u = y * y;
  float p = tanh_c(4);
#pragma unroll
  for (int k = 3; k >= 0; --k) p = fmaf(p, u, tanh_c(k));
  return fabsf(y) <= TANH_Y ? p * y : 1.f - __fdividef(2.f, ex2_approx(y * (2.f * LOG2E)) + 1.f);
}

}  // namespace

template <int NG, int D>
__global__ void __launch_bounds__(PTc<NG, D>::THREADS, PTc<NG, D>::PER_SM)
    attn_packed_tc_kernel(const __grid_constant__ CUtensorMap t_q, const __grid_constant__ CUtensorMap t_k,
                          const __grid_constant__ CUtensorMap t_v, const __grid_constant__ PackedArgs<bf16> a,
                          const __grid_constant__ AttnView w, int poly, int G, unsigned slots, int nc_log2, int* err) {
  using L = PTc<NG, D>;
  extern __shared__ uint8_t pt_smem[];
  uint8_t* sm = pt_smem + ((1024 - (su32(pt_smem) & 1023)) & 1023);
  uint8_t* sQ = sm + L::OFF_Q;
  uint8_t* sRing = sm + L::OFF_RING;
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + L::OFF_BAR);   // [NS]
  uint64_t* empty = full + L::NS;                                   // [NS]
  uint64_t* q_full = empty + L::NS;
  uint64_t* s_full = q_full + 1;                                    // [NG] scores in TMEM
  uint64_t* p_full = s_full + NG;                                   // [NG] weights in TMEM, O rescaled
  uint64_t* pv_done = p_full + NG;                                  // P V added to O
  uint64_t* o_done = pv_done + 1;                                   // all products done
  uint64_t* handed = o_done + 1;                                    // [2][4] a warp's rows' references handed on
  uint64_t* v_tail = handed + 8;                                    // values that reach behind the sequence have landed
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(v_tail + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  // warp-uniform values, and known to be: the MMA warp computes with them in uniform registers
  auto uniform = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (warp == 2) {   // a lane each: one thread after the other they delayed every CTA
    constexpr int first_p = 2 * L::NS + 1 + NG, count = first_p + NG + 2 + 8 + 1;
    static_assert(count <= 32, "a lane per barrier");
    if (lane < count) mbar_init(&full[lane], lane >= first_p && lane < first_p + NG ? 4 : 1);
    if (lane == 0) *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  SF_PDL_ENTRY();

  // heads of one query tile side by side; the last tiles of a sequence (the
  // longest under a causal view) first
  const int nc = 1 << nc_log2, rank = blockIdx.x & (nc - 1);
  const unsigned unit = blockIdx.x >> nc_log2, behind = unit / (unsigned)a.n_heads;   // slots behind this one in the list
  const int h = unit - behind * a.n_heads;
  const int kvh = (unsigned)h / (unsigned)G;
  // one warp looks the tile up (64 windows, measured when added: 31.5 us, all eight 34.7) while another takes TMEM
  __shared__ int found[4];
  if (warp == 0) {
    int tile, sb, se;
    const int s = slot_at(a.cu, a.n, a.T, slots - 1 - behind, 1, 7, 1, tile, sb, se);
    if (lane == 0) {
      found[0] = tile;
      found[1] = sb;
      found[2] = se - sb;
      found[3] = w.prefix ? min(max(w.prefix[s], 0), se - sb) : 0;
    }
  } else if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(tmem_slot)),
                 "r"((uint32_t)L::TMEM)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else if (threadIdx.x == 96 && h == 0) {
    report_offsets(a.cu, slots - 1 - behind, a.n, a.T, err);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*tmem_slot);
  auto free_tmem = [&] {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"((uint32_t)L::TMEM) : "memory");
  };
  const int tile = uniform(found[0]), sb = uniform(found[1]), S = uniform(found[2]), pre = uniform(found[3]), r0 = tile * TQ;
  if (tile < 0 || r0 >= S) {   // the whole cluster, before any copy is in flight
    if (warp == 1) free_tmem();
    return;
  }
  // key tiles [0, np) hold the prefix, [t_lo, t_hi) the rows' windows; this CTA takes nt of the list from tb on
  const int np = (pre + TK - 1) / TK;
  const int k_lo = w.left < 0 ? 0 : max(0, r0 - w.left);
  const int k_hi = w.right < 0 ? S : min(S, min(r0 + TQ, S) + w.right);
  const int t_lo = max(k_lo / TK, np), t_hi = max((k_hi + TK - 1) / TK, t_lo);
  const int all = np + t_hi - t_lo, share = (all + nc - 1) >> nc_log2, tb = min(all, rank * share), nt = min(all, tb + share) - tb;
  auto tile_of = [&](int t) { return t + tb < np ? t + tb : t_lo + t + tb - np; };

  auto cluster_sync = [] {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  };

  if (warp < 4) {
    // the copy of the last values, where they reach behind the sequence (else none)
    const int v_rows = S - tile_of(nt - 1) * TK, tail = v_rows < TK ? 2 * nt - 1 : -1;
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::REG_LOW));
    if (warp == 0 && nt > 0) {
      // -------------------------------------------------------------- loads
      if (lane == 0) {
        mbar_expect_tx(q_full, L::QTILE);
        for (int x = 0; x < D / 64; ++x) tma_load_2d(sQ + x * 16384, &t_q, q_full, h * D + 64 * x, sb + r0);
        // copies in the order of use: K(0) (NG = 2: and K(1)), then V(t), K(t + NG) for t = 0, 1, .., the last values behind
        auto copy_tile = [&](int c, bool& is_v) -> int {
          if (NG == 1) {
            is_v = c & 1;
            return c >> 1;
          }
          is_v = c == 2 * nt - 1 || (c > 0 && !(c & 1));
          return c == 0 ? 0 : c == 2 * nt - 1 ? nt - 1 : c & 1 ? (c + 1) / 2 : c / 2 - 1;
        };
        int c = 0;
        for (; c < 2 * nt && !*abort_flag; ++c) {
          const int b = c % L::NS;
          if (!wait_for(&empty[b], ((c / L::NS) & 1) ^ 1, abort_flag)) {
            *abort_flag = 1;
            break;
          }
          bool is_v;
          const int t = copy_tile(c, is_v);
          uint64_t* bar = c == tail ? v_tail : &full[b];
          mbar_expect_tx(bar, L::TILE);
          for (int x = 0; x < D / 64; ++x)
            tma_load_2d(sRing + b * L::TILE + x * TK * 128, is_v ? &t_v : &t_k, bar, kvh * D + 64 * x, sb + tile_of(t) * TK);
        }
        if (*abort_flag) {   // let this CTA's own loads land before its shared memory is released
          auto drain = [&](uint64_t* bar, uint32_t parity) {
            const long long c0 = clock64();
            while (!mbar_try_wait(bar, parity) && clock64() - c0 < WAIT_CYCLES) {
            }
          };
          drain(q_full, 0);
          for (int k = c - L::NS > 0 ? c - L::NS : 0; k < c; ++k)
            drain(k == tail ? v_tail : &full[k % L::NS], k == tail ? 0 : (k / L::NS) & 1);
        }
      }
      __syncwarp();
    } else if (warp == 1 && nt > 0) {
      // --------------------------------------------------------------- MMAs
      constexpr uint32_t id_s = idesc_bf16_mn(TQ, TK, false);
      constexpr uint32_t id_pv = idesc_bf16_mn(TQ, D, true);
      const bool leader = elect_one();
      const uint64_t dq = sw128_desc(su32(sQ)), dk0 = sw128_desc(su32(sRing)), dv0 = v_desc(su32(sRing));
      const uint32_t to = tmem + 64 * NG;
      bool ok = wait_for(q_full, 0, abort_flag);
      // ring places of the next keys and values in the order of copies, and their parities
      int sk = 0, sv = NG == 1 || nt == 1 ? 1 : 2;
      uint32_t pk = 0, pv = 0;
      auto ahead = [&](int& place, uint32_t& parity, int by) {
        place += by;
        if (place >= L::NS) {
          place -= L::NS;
          parity ^= 1;
        }
      };
      // step t: P V of tile t - NG, then the scores of tile t
      for (int t = 0; ok && t < nt + NG; ++t) {
        const int g = NG == 2 ? t & 1 : 0;
        const uint32_t ts = tmem + 64 * g;
        if (t >= NG && t - NG < nt) {
          ok = wait_for(&p_full[g], (t - NG) / NG & 1, abort_flag) && wait_for(&full[sv], pv, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const uint64_t dv = dv0 + (uint64_t)(sv * (L::TILE >> 4));
          if (leader) {
            if (t > NG) mma_ts<true>(to, ts, dv, id_pv);
            else mma_ts<false>(to, ts, dv, id_pv);
#pragma unroll
            for (int k = 1; k < TK / 16; ++k) mma_ts<true>(to, ts + 8 * k, dv + (uint64_t)(128 * k), id_pv);
            umma_commit(pv_done);
            umma_commit(&empty[sv]);
          }
          ahead(sv, pv, NG == 2 && t == nt ? 1 : 2);   // V(nt - 2) and V(nt - 1) lie side by side
        }
        if (t < nt) {
          ok = wait_for(&full[sk], pk, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const uint64_t dk = dk0 + (uint64_t)(sk * (L::TILE >> 4));
          if (leader) {
            mma_ss<false>(ts, dq, dk, id_s);
#pragma unroll
            for (int k = 1; k < D / 16; ++k)
              mma_ss<true>(ts, dq + (uint64_t)((k >> 2) * (16384 >> 4) + (k & 3) * 2),
                           dk + (uint64_t)((k >> 2) * (TK * 128 >> 4) + (k & 3) * 2), id_s);
            umma_commit(&s_full[g]);
            umma_commit(&empty[sk]);
          }
          ahead(sk, pk, NG == 2 && t == 0 ? 1 : 2);    // so do K(0) and K(1)
        }
      }
      if (ok && leader) umma_commit(o_done);
      if (!ok) *abort_flag = 1;
      __syncwarp();
      pdl_trigger();
    } else if (warp == 3 && tail > 0) {
      // ------------------------------------------------ rows behind the sequence
      // The last values may reach behind it: those rows are made zeros before the products see them, since a NaN there would
      // have every row computed again (1125 rows: 6500 us against 25)
      if (__all_sync(0xffffffffu, mbar_wait(v_tail, 0, abort_flag))) {
        uint8_t* tile_v = sRing + tail % L::NS * L::TILE;
#pragma unroll 1
        for (int b = v_rows * 128 + 16 * lane; b < TK * 128; b += 512)
#pragma unroll
          for (int x = 0; x < D / 64; ++x) *reinterpret_cast<uint4*>(tile_v + x * TK * 128 + b) = make_uint4(0, 0, 0, 0);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[tail % L::NS]);
      }
    }
    if (nc > 1) {
      if (warp == 1) {
        asm volatile("bar.sync 2, %0;" ::"n"(32 + 128 * NG) : "memory");
        free_tmem();
      }
      cluster_sync();
      cluster_sync();
    }
  } else {
    // -------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(L::REG_HIGH));
    const int grp = NG == 2 ? (warp - 4) >> 2 & 1 : 0, quarter = warp & 3;
    const int row = 32 * quarter + lane, i = r0 + row;   // this thread's row in its sequence
    const uint32_t lane_base = (uint32_t)(32 * quarter) << 16;
    const uint32_t tm_s = tmem + lane_base + 64 * grp, tm_o = tmem + lane_base + 64 * NG;
    const bool row_ok = i < S;
    auto warp_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, wait_for(bar, parity, abort_flag));
    };
    // references handed on by either group's warp of these rows: its place and barrier
    float2* xch = reinterpret_cast<float2*>(sm + L::OFF_X) + row;
    uint64_t* hand = handed + quarter;
    const int lo = w.left < 0 ? 0 : max(0, i - w.left);
    const int hi = w.right < 0 ? S : min(S, i + w.right + 1);
    const float slope = w.slopes ? w.slopes[h] * LOG2E : 0.f;
    const float inv_cap = w.cap > 0.f ? w.scale / w.cap : 0.f;
    const float f = w.cap > 0.f ? w.cap * LOG2E : w.scale * LOG2E;   // from s (tanh of it) to the log2 domain
    const float2 f2 = make_float2(f, f);
    float pc[5];
    cap_coefficients(w, pc);
    auto capped = [&](float2 v, float2 add) {   // + add, for |s / cap| <= 3/4
      const float2 u = __fmul2_rn(v, v);
      float2 p = make_float2(pc[4], pc[4]);
      p = __ffma2_rn(p, u, make_float2(pc[3], pc[3]));
      p = __ffma2_rn(p, u, make_float2(pc[2], pc[2]));
      p = __ffma2_rn(p, u, make_float2(pc[1], pc[1]));
      p = __ffma2_rn(p, u, make_float2(pc[0], pc[0]));
      return __ffma2_rn(p, v, add);
    };
    // columns x .. x + cols of the scores as they enter the exponent, in place, for any cap and score; the largest of them
    // (rarely entered: a loop of its own, not unrolled)
    auto cap_in_place = [&](int x, int cols) {
      float top = -INFINITY;
#pragma unroll 1
      for (const int end = x + cols; x < end; x += 16) {
        uint32_t v[16];
        tmem_ld16(tm_s + x, v);
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float y = f * tanh_any(__uint_as_float(v[c]) * inv_cap);
          top = fmaxf(top, y);
          v[c] = __float_as_uint(y);
        }
        tmem_st16(tm_s + x, v);
      }
      tmem_st_wait();
      return top;
    };
    auto magnitude = [](const float* sc) {   // of 32
      float p0 = max3_abs(sc[0], sc[1], sc[2]), p1 = max3_abs(sc[3], sc[4], sc[5]);
#pragma unroll
      for (int c = 6; c < 30; c += 4) {
        p0 = max3_abs(p0, sc[c], sc[c + 1]);
        p1 = max3_abs(p1, sc[c + 2], sc[c + 3]);
      }
      return max3_abs(max3_abs(p0, sc[30], sc[31]), p1, 0.f);
    };
    // first keys of the tiles that every row of the query tile sees whole: [w_lo, w_hi] by the window, up to w_pre
    const int w_lo = w.left < 0 ? 0 : r0 + TQ - 1 - w.left;
    const int w_hi = min(S, w.right < 0 ? S : r0 + w.right + 1) - TK, w_pre = pre - TK;
    float m = -INFINITY;   // reference maximum (log2 domain) of this group's last tile
    float l = 0.f;         // sum of this group's weights, relative to m
    int mine = 0, got = 0; // this group's tiles so far, references taken over from the other group
    bool ok = true;
    for (int t = grp; t < nt; t += NG) {
      const int j0 = tile_of(t) * TK;
      ok = warp_wait(&s_full[grp], mine & 1);
      if (!ok) break;
      ++mine;
      tc_fence_after();
      const bool whole = (j0 >= w_lo && j0 <= w_hi) || j0 <= w_pre;
      // First pass: the row's largest score, 32 columns at a time.  Scores that are masked, biased or under a cap without
      // coefficients go back to TMEM as they enter the exponent; the others are taken as they are in the second pass.
      // Of capped scores the largest magnitude does: it bounds them and decides the polynomial's range.  As a reference it may
      // be far above the largest score, where all are negative; eight columns bound that, and the largest itself is looked for
      // where they are FAR or more below: the row's largest weight is 2^-FAR or more, so that neither lesser weights nor
      // products with small values leave fp32's range.
      const bool ready = !whole || slope != 0.f || (w.cap > 0.f && !poly);
      float mx = -INFINITY, mag = 0.f;   // under a cap: of the eight columns
#pragma unroll
      for (int x = 0; x < TK; x += 32) {
        uint32_t v[32];
        tmem_ld32(tm_s + x, v);
        float sc[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) sc[c] = __uint_as_float(v[c]);
        if (ready) {
          if (w.cap > 0.f) {
            if (poly && __all_sync(0xffffffffu, magnitude(sc) * inv_cap <= TANH_Y)) {
#pragma unroll
              for (int c = 0; c < 32; c += 2) {
                const float2 y = capped(make_float2(sc[c], sc[c + 1]), make_float2(0.f, 0.f));
                sc[c] = y.x;
                sc[c + 1] = y.y;
              }
            } else {
              cap_in_place(x, 32);
              tmem_ld32(tm_s + x, v);
#pragma unroll
              for (int c = 0; c < 32; ++c) sc[c] = __uint_as_float(v[c]);
            }
          } else {
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
              const float2 y = __fmul2_rn(make_float2(sc[c], sc[c + 1]), f2);
              sc[c] = y.x;
              sc[c + 1] = y.y;
            }
          }
          if (slope != 0.f) {
            const float at = (float)(j0 + x - i);   // distance of column 0 (exact below 2^24)
#pragma unroll
            for (int c = 0; c < 32; ++c) sc[c] = fmaf(-slope, fabsf(at + (float)c), sc[c]);
          }
          if (!whole) {
            // columns in view as bits: those of the row's window and below the prefix
            auto below = [&](int j) -> uint32_t {
              const int c = j - j0 - x;
              return c <= 0 ? 0u : c >= 32 ? 0xffffffffu : (1u << c) - 1u;
            };
            const uint32_t bits = (below(hi) & ~below(lo)) | below(pre);
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!(bits >> c & 1u)) sc[c] = -INFINITY;
          }
#pragma unroll
          for (int c = 0; c < 32; ++c) v[c] = __float_as_uint(sc[c]);
          tmem_st32(tm_s + x, v);
        }
        if (!ready && w.cap > 0.f) {
          mag = fmaxf(mag, magnitude(sc));
          mx = max3(max3(mx, sc[0], sc[8]), sc[16], sc[24]);
        } else {
          float p0 = max3(sc[0], sc[1], sc[2]), p1 = max3(sc[3], sc[4], sc[5]);
#pragma unroll
          for (int c = 6; c < 30; c += 4) {
            p0 = max3(p0, sc[c], sc[c + 1]);
            p1 = max3(p1, sc[c + 2], sc[c + 3]);
          }
          mx = max3(mx, max3(p0, sc[30], sc[31]), p1);
        }
      }
      bool placed = ready;   // the scores stand in TMEM as they enter the exponent
      if (!ready) {
        if (w.cap == 0.f) {
          mx *= f;
        } else {
          const float2 bound = capped(make_float2(mag, mx), make_float2(0.f, 0.f));
          placed = !__all_sync(0xffffffffu, mag * inv_cap <= TANH_Y && bound.x - bound.y <= FAR);
          mx = placed ? cap_in_place(0, TK) : bound.x;
        }
      }
      // the reference of the tile before: this group's own, or handed on by the other
      float ref = m;
      if (NG == 2 && t > 0) {
        ok = warp_wait(&hand[4 * (grp ^ 1)], got & 1);
        if (!ok) break;
        ++got;
        ref = xch[128 * (grp ^ 1)].x;
      }
      const float top = fmaxf(ref, mx);
      const bool moves = __any_sync(0xffffffffu, top > ref + LAZY);   // at the first tile, then rarely
      const float now = moves ? top : ref;
      if (moves && t > 0) {
        // O holds the products of the tiles before (scores of this tile imply that all but the last are done)
        ok = warp_wait(pv_done, (t - 1) & 1);
        if (!ok) break;
        tc_fence_after();
        const float al = ref == -INFINITY ? 0.f : ex2_approx(ref - now);
        const float2 al2 = make_float2(al, al);
#pragma unroll
        for (int x = 0; x < D; x += 16) {
          uint32_t v[16];
          tmem_ld16(tm_o + x, v);
#pragma unroll
          for (int k = 0; k < 16; k += 2) {
            const float2 y = __fmul2_rn(make_float2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), al2);
            v[k] = __float_as_uint(y.x);
            v[k + 1] = __float_as_uint(y.y);
          }
          tmem_st16(tm_o + x, v);
        }
      }
      if (now != m) l *= m == -INFINITY ? 0.f : ex2_approx(m - now);
      m = now;
      if (NG == 2 && t + 1 < nt) {   // hand the reference on to the next tile's group
        xch[128 * grp].x = m;
        __syncwarp();
        if (lane == 0) mbar_arrive(&hand[4 * grp]);
      }
      const float base = m == -INFINITY ? 0.f : m;
      const float2 b2 = make_float2(-base, -base);
      float2 ps[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      if (ready) tmem_st_wait();
      // Second pass: weights, packed over columns whose scores have been read
      auto weights = [&](auto exponent) {
#pragma unroll
        for (int x = 0; x < TK; x += 32) {
          uint32_t v[32], pw[16];
          tmem_ld32(tm_s + x, v);
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const float2 e = exponent(make_float2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])));
            const float2 p = make_float2(ex2_approx(e.x), ex2_approx(e.y));
            ps[(c >> 1) & 1] = __fadd2_rn(ps[(c >> 1) & 1], p);
            __nv_bfloat162 hp = __floats2bfloat162_rn(p.x, p.y);
            pw[c >> 1] = *reinterpret_cast<uint32_t*>(&hp);
          }
          tmem_st16(tm_s + x / 2, pw);
        }
      };
      if (placed) {
        weights([&](float2 v) { return __fadd2_rn(v, b2); });
      } else if (w.cap == 0.f) {
        weights([&](float2 v) { return __ffma2_rn(v, f2, b2); });
      } else {
        weights([&](float2 v) { return capped(v, b2); });
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[grp]);
      const float2 pt = __fadd2_rn(ps[0], ps[1]);
      l += pt.x + pt.y;
    }
    if (!ok) *abort_flag = 1;
    if (NG == 2) {   // the groups' sums meet (every warp comes here, also after a failed wait)
      xch[128 * grp] = make_float2(m, l);
      asm volatile("bar.sync 1, 256;" ::: "memory");
      const float2 theirs = xch[128 * (grp ^ 1)];
      const float fin = fmaxf(m, theirs.x);
      l = (m == -INFINITY ? l : l * ex2_approx(m - fin)) + (theirs.x == -INFINITY ? theirs.y : theirs.y * ex2_approx(theirs.x - fin));
      m = fin;
    }
    // each group has its share of the dims
    constexpr int DG = D / NG;
    if (nt > 0) {
      ok = ok && warp_wait(o_done, 0);
      tc_fence_after();
    }
    auto eight = [](const float* y, float inv, bool& fine) -> uint4 {
      uint32_t w4[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float y0 = y[2 * k] * inv, y1 = y[2 * k + 1] * inv;
        fine = fine && isfinite(y0) && isfinite(y1);
        __nv_bfloat162 ho = __floats2bfloat162_rn(y0, y1);
        w4[k] = *reinterpret_cast<uint32_t*>(&ho);
      }
      return make_uint4(w4[0], w4[1], w4[2], w4[3]);
    };
    auto over = [](float l) { return l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l); };   // nothing in view: zeros; NaN stays NaN
    if (nc == 1) {
      if (ok) {
        const float inv = over(l);
        bool fine = true;   // a sum that is not finite comes from the scores in view: the result says so as it is
        uint4* dst = reinterpret_cast<uint4*>(a.out + (int64_t)(sb + i) * a.ldo + (int64_t)h * D + DG * grp);
#pragma unroll
        for (int x = 0; x < DG; x += 32) {
          uint32_t v[32];
          tmem_ld32(tm_o + DG * grp + x, v);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint4 o8 = eight(reinterpret_cast<const float*>(v) + 8 * c, inv, fine);
            if (row_ok) dst[x / 8 + c] = o8;
          }
        }
        __syncwarp();   // the rows' stores are there for the whole warp
        // rows whose share is not finite: the same dims again, where the row sees no reason for it
        uint32_t redo = __ballot_sync(0xffffffffu, row_ok && !fine && isfinite(l));
        while (redo) {
          const int k = __ffs(redo) - 1;
          redo &= redo - 1;
          attn_packed_row<bf16, D>(a, w, h, kvh, sb, S, r0 + 32 * quarter + k, pre, slope, DG / 32 * grp, DG / 32 * (grp + 1));
        }
      }
    } else {
      // this CTA's part over its operands, which no product reads any more
      float *pO = reinterpret_cast<float*>(sm), *pM = pO + 128 * L::LDO, *pL = pM + 128;
      int* flag = reinterpret_cast<int*>(pL + 128);
      float4* mine4 = reinterpret_cast<float4*>(pO + row * L::LDO + DG * grp);
#pragma unroll
      for (int x = 0; x < DG; x += 32) {
        uint32_t v[32];
        tmem_ld32(tm_o + DG * grp + x, v);
#pragma unroll
        for (int c = 0; c < 8; ++c)   // without a key tile O was never written
          mine4[x / 4 + c] = nt == 0 ? make_float4(0.f, 0.f, 0.f, 0.f)
                                     : make_float4(__uint_as_float(v[4 * c]), __uint_as_float(v[4 * c + 1]),
                                                   __uint_as_float(v[4 * c + 2]), __uint_as_float(v[4 * c + 3]));
      }
      if (grp == 0) {
        pM[row] = m;
        pL[row] = l;
        flag[row] = 0;
      }
      // TMEM is free again before this CTA waits for its cluster: another kernel's cluster may wait for it
      tc_fence_before();
      asm volatile("bar.arrive 2, %0;" ::"n"(32 + 128 * NG) : "memory");
      cluster_sync();
      auto at_rank = [](const float* p, int k) -> uint32_t {
        uint32_t at;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(su32(p)), "r"(k));
        return at;
      };
      auto peer = [&](const float* p, int k) -> float {
        float v;
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at_rank(p, k)) : "memory");
        return v;
      };
      // each CTA finishes its share of the rows, eight dims a thread, the parts in order
      const int rows = 128 >> nc_log2, tid = threadIdx.x - 128;
      for (int e = tid; e < rows * (D / 8); e += 128 * NG) {
        const int rr = rank * rows + e / (D / 8), d = e % (D / 8) * 8;
        if (r0 + rr >= S) break;
        float mk[4], mm = -INFINITY, ll = 0.f, y[8] = {};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          mk[k] = k < nc ? peer(pM + rr, k) : -INFINITY;
          mm = fmaxf(mm, mk[k]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (k >= nc) break;
          const float f = mk[k] == -INFINITY ? 0.f : ex2_approx(mk[k] - mm);   // a part without a key: sum and output 0
          ll = fmaf(f, peer(pL + rr, k), ll);
#pragma unroll
          for (int q = 0; q < 8; q += 4) {
            float4 v;
            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                         : "r"(at_rank(pO + rr * L::LDO + d + q, k))
                         : "memory");
            y[q] = fmaf(f, v.x, y[q]); y[q + 1] = fmaf(f, v.y, y[q + 1]);
            y[q + 2] = fmaf(f, v.z, y[q + 2]); y[q + 3] = fmaf(f, v.w, y[q + 3]);
          }
        }
        bool fine = true;
        *reinterpret_cast<uint4*>(a.out + (int64_t)(sb + r0 + rr) * a.ldo + (int64_t)h * D + d) = eight(y, over(ll), fine);
        if (!fine && isfinite(ll)) flag[rr] = 1;
      }
      __syncwarp();
      cluster_sync();   // no CTA's part is read any more; the stores and flags are there
      for (int rr = rank * rows + (warp - 4); rr < (rank + 1) * rows; rr += 4 * NG)
        if (r0 + rr < S && flag[rr]) attn_packed_row<bf16, D>(a, w, h, kvh, sb, S, r0 + rr, pre, slope);
    }
    if (!ok) *abort_flag = 1;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1 && nc == 1) free_tmem();
  if (threadIdx.x == 0 && *abort_flag) set_err(err, ERR_TIMEOUT);
}

namespace {
int g_packed_sms = 148;

template <int NG, int D>
cudaError_t launch_tc(const PackedArgs<bf16>& a, const AttnView& w, int64_t units, int nc, int* err, cudaStream_t st) {
  CUtensorMap tq, tk, tv;
  CK_LAUNCH(make_bf16_map_sw128(&tq, a.q, a.T, a.n_heads * D, a.ldq, TQ));
  CK_LAUNCH(make_bf16_map_sw128(&tk, a.k, a.T, a.n_kv * D, a.ldk, TK));
  CK_LAUNCH(make_bf16_map_sw128(&tv, a.v, a.T, a.n_kv * D, a.ldv, TK));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * nc));
  cfg.blockDim = dim3(PTc<NG, D>::THREADS);
  cfg.dynamicSmemBytes = PTc<NG, D>::SMEM;
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
  float pc[5];
  CK_LAUNCH(cudaLaunchKernelEx(&cfg, attn_packed_tc_kernel<NG, D>, tq, tk, tv, a, w, (int)cap_coefficients(w, pc), a.n_heads / a.n_kv, (unsigned)(units / a.n_heads),
                               nc == 4 ? 2 : nc - 1, err));
  return cudaGetLastError();
}
}  // namespace

template <>
cudaError_t launch_attention_packed<bf16>(const PackedArgs<bf16>& a, int D, const AttnView& w, int* err, cudaStream_t st) {
  const int64_t units = ((int64_t)a.T / TQ + a.n) * a.n_heads;
  // split (heads of 64, causal, one sequence; undivided, halved, in four; us): 8 heads x 600 rows 11.0, 10.2, 12.4, x 1125
  // 16.5, 13.1, 19.2, x 4000 51.0, 41.9, 67.2; 2 heads x 4000 46.6, 27.7, 19.6.  In four only while all those clusters are
  // resident at once: they reach about seven eighths of the 2 CTAs per SM
  int nc = 1;
  if (units <= 2 * g_packed_sms && a.T / a.n >= 512) nc = 2;
  if (16 * units <= 7 * g_packed_sms && a.T / a.n >= 1024) nc = 4;
  if (D == 128) return launch_tc<2, 128>(a, w, units, nc, err, st);
  if (units >= 6 * g_packed_sms) return launch_tc<1, 64>(a, w, units, nc, err, st);
  return launch_tc<2, 64>(a, w, units, nc, err, st);
}

cudaError_t attention_packed_tc_init_attributes() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) == cudaSuccess && cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && n > 0)
    g_packed_sms = n;
  cudaError_t r = cudaFuncSetAttribute(attn_packed_tc_kernel<1, 64>, cudaFuncAttributeMaxDynamicSharedMemorySize, PTc<1, 64>::SMEM);
  if (r == cudaSuccess) r = cudaFuncSetAttribute(attn_packed_tc_kernel<2, 64>, cudaFuncAttributeMaxDynamicSharedMemorySize, PTc<2, 64>::SMEM);
  if (r == cudaSuccess) r = cudaFuncSetAttribute(attn_packed_tc_kernel<2, 128>, cudaFuncAttributeMaxDynamicSharedMemorySize, PTc<2, 128>::SMEM);
  return r;
}

}  // namespace sf
