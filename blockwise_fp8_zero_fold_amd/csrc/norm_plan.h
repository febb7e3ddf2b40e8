// How many workgroups the norm join's kernels are launched with, and of how many threads (host code
// without HIP, so that it can be tested by itself).
#pragma once

#include <cstdint>

namespace fp8z1 {

// compute units of the card, and the waves that one of them holds of these kernels by their registers
constexpr int64_t kNormUnits = 256, kNormUnitWaves = 16;

inline int norm_threads(int64_t C) {
  const int64_t per = C <= 8192 ? 8 : 16;  // elements a thread holds
  return static_cast<int>((C + 64 * per - 1) / (64 * per) * 64);
}

// Forward: a row per workgroup, as many on every compute unit, the workgroups walking over the rows side
// by side (each over rows of its own in a row: 20 % slower, a workgroup for every row 20 %).  A number that
// is no multiple of the compute units leaves some of them a workgroup more than others: 3584 / waves,
// even for rows of 14 waves only, took 170 us for 8192 rows of 6656 where this takes 111, 102 and 90
// of 5120, 299 and 240 of 10,240, 388 and 269 of 12,288.  (Twice as many waves: 13 % slower at 5120,
// half as many 11 % at 4096, both within 1 % at 7168.)
inline int64_t norm_fwd_groups(int64_t T, int64_t C) {
  const int64_t most = kNormUnits * (kNormUnitWaves / (norm_threads(C) / 64));
  return T < most ? T : most;
}

// Backward: up to 16 waves per workgroup, for several short rows at a time, since every workgroup also
// writes its column sums.  Rows for one turn of one workgroup go to one, which writes the gradients
// itself: no second launch (3 us on the host).  Not for more: a turn takes 4.3 us, the second launch and its kernel 4 (captured,
// 2 rows of 7168: one workgroup 13.2 us, two and the second launch 11.5; 32 rows of 1024: 20.9 and 8.2).
struct NormGroups {
  int64_t rows, count;  // rows at a time per workgroup, workgroups
};
inline NormGroups norm_bwd_groups(int64_t T, int64_t C) {
  const int64_t waves = norm_threads(C) / 64, all = C <= 8192 ? kNormUnitWaves / waves : 1;
  if (T <= all) return {T, 1};
  int64_t rows = (T + kNormUnits - 1) / kNormUnits;
  if (rows > all) rows = all;
  const int64_t most = kNormUnits * (kNormUnitWaves / (waves * rows)), want = (T + rows - 1) / rows;
  return {rows, want < most ? want : most};
}

}  // namespace fp8z1
