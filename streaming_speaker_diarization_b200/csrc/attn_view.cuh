// The score and view shared by the packed and the cached attention:
//   s(i, j) = scale q_i . k_j, then cap tanh(s / cap) where cap > 0, then
//             s - slope_head |i - j|
//   seen(i, j) = (i - left <= j <= i + right) or j < prefix   (-1: no limit)
// and the bounds of the device-resident sequence offsets.  Scores are carried
// in the exp2 domain (times log2 e).
#pragma once
#include <math.h>

#include "common.cuh"

namespace sf {

constexpr float LOG2E = 1.4426950408889634f;

struct AttnView {
  float scale;          // score factor
  float cap;            // 0: none
  int left, right;      // positions seen before / after the query's own; -1: no limit
  const float* slopes;  // f32 [n_heads] distance bias, or null
  const int* prefix;    // i32 [n] leading keys that every row of a sequence sees, or null
};

// cap tanh(s / cap) log2 e, or s log2 e without a cap.  tanhf keeps the full
// fp32 accuracy (the capped score is an exponent, so its absolute error is the
// weight's relative error).
__device__ __forceinline__ float capped_l2(float s, float cap) {
  return cap > 0.f ? cap * tanhf(s / cap) * LOG2E : s * LOG2E;
}

// Rows [b, e) within [0, T) of a sequence with offsets rb and re: offsets are
// read from device memory that the host has not seen, so each is clamped, and
// bad says that an offset was out of order or out of range.
__host__ __device__ __forceinline__ void clamp_bounds(int rb, int re, int T, int& b, int& e, bool& bad) {
  b = rb < 0 ? 0 : rb > T ? T : rb;
  e = re < b ? b : re > T ? T : re;
  bad = rb != b || re != e;
}
// Whether sequence i (if there is one) has such offsets.  Slot i of a call,
// of which there are at least n, answers for sequence i: among offsets out of
// order a sequence may own no slot.
__host__ __device__ __forceinline__ bool bad_offsets(const int* __restrict__ cu, int64_t i, int n, int T) {
  if (i < 0 || i >= n) return false;
  int b, e;
  bool bad;
  clamp_bounds(cu[i], cu[i + 1], T, b, e, bad);
  return bad;
}
__device__ __forceinline__ void report_offsets(const int* __restrict__ cu, int64_t slot, int n, int T, int* err) {
  if (bad_offsets(cu, slot, n, T)) set_err(err, ERR_BOUNDS);
}

// Work slots over sequences whose lengths only the device knows: sequence i
// owns the slots [slot_base(i), slot_base(i + 1)), slot_base(i) =
// floor(cu[i] mul / 2^per) + i add: at least ceil(length mul / 2^per) of them with
// add = 1, so the grid needs no sizes from the host.
__host__ __device__ __forceinline__ int64_t slot_base(const int* __restrict__ cu, int i, int mul, int per, int add) {
  return ((int64_t)cu[i] * mul >> per) + (int64_t)i * add;
}
// slots of one sequence the kernels can index: 2^26 rows in tiles of 8 (x 128 rows, the largest tile or page, stays in 32 bits)
constexpr int64_t MAX_SLOT = 1 << 23;
// wild offsets must not wrap: -1 (idle) .. 2^23 (past every sequence's work)
__host__ __device__ __forceinline__ int slot_index(int64_t at) { return (int)(at < 0 ? -1 : at > MAX_SLOT ? MAX_SLOT : at); }
// The sequence of a slot (the last whose base is at or before it), the slot's
// index in it and its rows, by a whole warp: 32 bases are compared at once, one
// dependent load for up to 32 sequences, two for up to 1024 (128 bases at once,
// with the bounds, cost more in instructions than the loads: 64 windows 35.5
// against 34.8 us).  Slots past a sequence's work are idle.
__device__ __forceinline__ int slot_at(const int* __restrict__ cu, int n, int T, int64_t slot, int mul, int per, int add,
                                       int& idx, int& b, int& e) {
  const int lane = threadIdx.x & 31;
  int lo = 0, len = n;
  while (len > 1) {
    const int step = (len + 31) >> 5, i = lane * step;
    const uint32_t at = __ballot_sync(0xffffffffu, lane == 0 || (i < len && slot_base(cu, lo + i, mul, per, add) <= slot));
    const int k = 31 - __clz(at);
    lo += k * step;
    len = len - k * step < step ? len - k * step : step;
  }
  idx = slot_index(slot - slot_base(cu, lo, mul, per, add));
  bool bad;
  clamp_bounds(cu[lo], cu[lo + 1], T, b, e, bad);
  return lo;
}

}  // namespace sf
