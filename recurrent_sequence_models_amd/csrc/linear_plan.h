// Which form a product of the projections takes, by its sizes: the rules of falcon_linear.hip, host side only (nothing of
// HIP, so that a test can ask them).
#pragma once
#include <stdint.h>

#include <algorithm>

namespace falcon {

constexpr int KB = 128;           // bytes of k that a step of the loop takes
constexpr int FEW_TOKENS = 64;    // at most, of the form without LDS tiles

// Forms of a product: `few` (16 rows of the left operand a workgroup), or tiles of 64 x 64, 128 x 128 (deep: four steps in
// LDS, one workgroup a compute unit) and 256 x 256.
enum class Form { few, small, deep, medium, large };
struct Plan { Form form; int splits; int64_t tiles; };

inline int64_t over(int64_t n, int64_t d) { return (n + d - 1) / d; }

// Workgroups that share a tile's k: as many as make `groups` of all, at 4 steps each and 16 at most.
inline int splits_of(int64_t tiles, int64_t groups, int64_t steps) {
  const int64_t s = std::min({groups / tiles, steps / 4, (int64_t)16});
  return s > 1 ? (int)s : 1;
}

// A compute unit holds one workgroup of 256 x 256 or two of 128 x 128; the larger tile reads less from LDS for a product
// (16384 x 2048 -> 4096 bf16: 287 us, 306 with the smaller; 16384 x 4096 -> 2048 e4m3 is level, 200 and 196), the smaller
// one leaves less of the last round empty (16384 x 768 -> 1536 bf16: 55 us, 62 with the larger; 2048 x 2048 -> 2048:
// 28, 53).  So rounds are counted, in tiles of 128 x 128 a compute unit.  fp32 takes too many registers for the larger.
// Where 128 x 128 tiles leave compute units idle, tiles are 64 x 64, and k is split where those do too: 512 x 2048 -> 2048
// bf16 15 us, 20 in four parts of 128 x 128; 100 x 2048 -> 4096 13.5, 16.  Not over more than 48 steps a
// workgroup: 512 x 8192 -> 2048 45 us, 32 in eight parts of 128 x 128; those for two workgroups a compute unit where
// each has 16 steps and more, which is level with one (768 x 16384 -> 1536, training: 161 to 170 us, 159 for one; 1000 x
// 16384 -> 512: 32.5 and 30.5; 100 x 8192 -> 4096: 22.4 and 22.9).  One workgroup of 128 x 128 a compute unit has LDS for
// four steps, three of them on their way, and 8 waves (2048 x 2048 -> 2048: 25 us, 28 with two steps, 34 as 64 x 64;
// training 2048 x 2048 -> 2048: 84 and 90).
inline Plan tiles_of(int64_t I, int64_t J, int64_t K, int e) {
  const int64_t large = over(I, 256) * over(J, 256), medium = over(I, 128) * over(J, 128), small = over(I, 64) * over(J, 64);
  if (e < 4 && large >= 256 && over(large, 256) * 4 * 20 <= over(medium, 512) * 2 * 21) return {Form::large, 1, large};
  const int64_t steps = over(K * e, KB);
  if (medium < 256) {
    const int s = splits_of(small, 256, steps);
    if (steps / s <= 48) return {Form::small, s, small};
  }
  const int s = medium < 256 ? splits_of(medium, steps * medium >= 16 * 512 ? 512 : 256, steps) : 1;
  return {medium * s <= 256 ? Form::deep : Form::medium, s, medium};
}

// The time of a plan's tiles, in rounds of the chip: 20 for tiles of 128 x 128 a compute unit.
inline int64_t rounds_of(const Plan &p) {
  return p.form == Form::large ? over(p.tiles, 256) * 4 * 20 : over(p.tiles * p.splits, 512) * 2 * 21;
}

// Few tokens take what a compute unit loads, at about 40 KB a us: 16 rows of W and the tokens (a multiple of 16) for each
// of its workgroups of `few`, or both operands of its tiles' steps (which fp32 products hold up by a quarter, by
// three halves in the larger tiles) and about 64 KB for the tile's beginning and the join.  16 x 2048 -> 4096 bf16: 7.5 us,
// 9.6 in tiles; 16 x 8192 -> 2048: 17.1 and 12.7; 64 x 4096 -> 8192: 38.5 and 18; 24 x 4096 -> 8192 fp32: 47 and 50.
inline Plan plan_of(int64_t I, int64_t J, int64_t K, int e) {
  const Plan p = tiles_of(I, J, K, e);
  if (J > FEW_TOKENS) return p;
  const int64_t rows = J <= 16 ? 32 : J <= 32 ? 48 : 80, groups = over(I, 16);
  const int64_t few = over(groups, 256) * rows * K * e, step = p.form == Form::small ? 2 * 64 * KB : 2 * 128 * KB;
  const int64_t tiles = over(p.tiles * p.splits, 256) * (over(K * e, KB) / p.splits) * step;
  const int64_t quarters = e < 4 ? 4 : p.form == Form::small ? 5 : 10;
  if (p.form == Form::large || few <= tiles * quarters / 4 + 65536) return {Form::few, 1, groups};
  return p;
}

// Tokens that a pass of their own takes: up to 64 behind the last whole tile of 256, where that saves the others a
// round (16387 x 4096 -> 2048 e4m3: 203 us, 257 as one pass).
inline int tokens_apart(int64_t I, int64_t J, int64_t K, int e) {
  const int rest = (int)(J % 256);
  if (!rest || rest > FEW_TOKENS || J < 512 || K < 512) return 0;
  const Plan with = plan_of(I, J, K, e), without = plan_of(I, J - rest, K, e);
  return with.form != Form::small && without.form != Form::small && rounds_of(without) < rounds_of(with) ? rest : 0;
}

}  // namespace falcon
