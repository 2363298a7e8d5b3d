// The sequences of a call, and how the convolution and the selective scan deal them out: the rules of falcon_conv.hip,
// falcon_ssm.hip and falcon_ssm_bwd.hip, host side only (a test can ask them).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace falcon {

// The sequences of a call: n of T tokens each, or (cu != null) packed on one axis of T tokens.
struct SeqMap {
  const int *cu;
  int n, T;
  __host__ __device__ int tokens() const { return cu ? T : n * T; }
  // token ranges, kept inside the arrays whatever the offsets hold
  __host__ __device__ int inside(int t) const { return t < 0 ? 0 : t > T ? T : t; }
  __host__ __device__ int begin(int i) const { return cu ? inside(cu[i]) : i * T; }
  __host__ __device__ int end(int i) const { return cu ? inside(cu[i + 1]) : (i + 1) * T; }
  // the largest i < n that begins at or before token t (0 if none)
  __host__ __device__ int of(int t) const {
    if (!cu) return t / T;
    int lo = 0, len = n;
    while (len > 1) {
      const int half = len >> 1;
      if (cu[lo + half] <= t) { lo += half; len -= half; } else { len = half; }
    }
    return lo;
  }
};

// ---- Short causal convolution ---------------------------------------------------------
// A pass's threads, its wave's lanes that lie side by side over channels, and the tokens of a run, which is those lanes'.
// With all 64 of a wave, where a run stands is the same in all of them (4 x 4096 x 1536 bf16: 24 us, 25 with runs of 16
// lanes, backward 33, 36 of 32; 13 packed sequences, 9001 x 2048: 22 and 29); but forward, where 16 hold all channels, the
// others would idle (16 x 4096 x 64 bf16: 13.3 us, 23.3 with 64 lanes; x 128: 13.2, 18.4; x 256 13.4 both; backward, 32
// lanes would save 2 of 23).  Long runs read fewer tokens twice, short ones make more workgroups (4 x 4096 x 1536 bf16, 24
// and 33 us: 30 and 36 with runs half as long, 24 and 41 twice).
constexpr int CONV_THR = 256, CONV_WIDE = 64, CONV_NARROW = 16;
struct ConvPlan {
  int lanes, run;
  int64_t blocks, wide;      // workgroups along time and channels
};
inline ConvPlan conv_plan(const SeqMap &seq, int D, bool bf16, bool back) {
  const int each = bf16 && !back ? 8 : 4;            // channels of a lane
  const int lanes = !back && D <= CONV_NARROW * each ? CONV_NARROW : CONV_WIDE, runs = CONV_THR / lanes;
  const int64_t wide = (D + lanes * each - 1) / (lanes * each), tokens = seq.tokens();
  const auto blocks = [&](int run) { return (tokens + run * runs - 1) / (run * runs); };
  int run = back ? 32 : 16;
  while (run > 4 && blocks(run) * wide < 512) run /= 2;
  return {lanes, run, blocks(run), wide};
}

// ---- Selective state-space scan ---------------------------------------------------------
inline int ssm_chunk(int N) { return 1024 / N; }   // steps between the states that the forward keeps
constexpr int SSM_ALIGN = 64;      // segments are a multiple of this long: whole chunks of every N

__host__ __device__ inline int segments_of(const SeqMap &q, int len) { return (q.T - 1) / len + 1; }   // T + len may pass 2^31
__host__ __device__ inline int slots_of(const SeqMap &q, int len) {
  return q.cu ? q.T / len + q.n : q.n * segments_of(q, len);
}

// Tokens of a segment, a whole number of chunks.  Whole sequences, where those make `enough` workgroups (of `channels`
// channels each) or have no more than `whole` tokens; else as many segments as make `want`, down to one tile each
// (1 x 1000 x 512 bf16, both directions: 56 us, 89 with 256 tokens and more; 1 x 16384 x 128: 125 and 122): forming their
// maps first costs half of a pass.
inline int ssm_segment(const SeqMap &q, int D, int channels, int enough, int want, int whole) {
  const int64_t groups = (D + channels - 1) / channels;
  int64_t len;
  if (q.T <= whole) return (q.T + SSM_ALIGN - 1) / SSM_ALIGN * SSM_ALIGN;
  if (q.cu) {
    if (groups >= enough) return (q.T + SSM_ALIGN - 1) / SSM_ALIGN * SSM_ALIGN;
    len = ((int64_t)q.T * groups + want - 1) / want;
  } else {
    const int64_t parts = q.n * groups >= enough ? 1 : want / (q.n * groups);
    if (parts < 2) return (q.T + SSM_ALIGN - 1) / SSM_ALIGN * SSM_ALIGN;
    len = (q.T + parts - 1) / parts;
  }
  return (int)((len + SSM_ALIGN - 1) / SSM_ALIGN * SSM_ALIGN);
}
// Whether any sequence has more than one segment (packed: may have).
inline bool ssm_segmented(const SeqMap &q, int seg) { return q.T > seg; }

constexpr int SSM_FWD_CH = 16;      // channels of a workgroup
// Below this many workgroups, 128 / N waves lie behind each other in time (of 8 steps each; N = 64: 16) instead of 64 / N
// of 16 steps: more waves for what there is, at twice the joins.  bf16, N = 16, 32, 64: 384 workgroups (4 x 2048 x 1536)
// 105, 209 and 341 us, 112, 225 and 359 with half the waves; 512 (4 x 2048 x 2048) 110, 221 and 349 us, 114, 226 and 378;
// 768 (8 x 2048 x 1536) 165, 358 and 552 us, 146, 270 and 450.
constexpr int SSM_FEW_GROUPS = 640;
inline bool ssm_few_fwd(const SeqMap &q, int seg, int D) {
  return (int64_t)((D + SSM_FWD_CH - 1) / SSM_FWD_CH) * slots_of(q, seg) < SSM_FEW_GROUPS;
}
// Sequences are cut where they make fewer than 256 workgroups, into 768 (1 x 16384 x 1536, 96 workgroups: 237 us with
// the maps' pass, 294 cut for 512, 386 for 256); with 384 they are not (4 x 4096 x 1536: 216 us, 218 cut).  Packed ones are
// where the total would be, as the host does not see the offsets: 100 sequences, 5000 x 1536: 128 us, 95 uncut; with the
// backward pass 517, of which its own cut is 42.
// Up to 4096 / N tokens they are left whole (1 x 192 x 512: 10.3 us, 12.8 cut; 320: 14.6 and 13.0; N = 64: 128 18.1 and 19.3,
// 192 25.3 and 19.4).
inline int ssm_segment_fwd(const SeqMap &q, int D, int N) { return ssm_segment(q, D, SSM_FWD_CH, 256, 768, 4096 / N); }

constexpr int SSM_BWD_CH = 32;      // channels of a workgroup
// Sequences are cut where they make fewer than 128 workgroups, into 256 (2 x 2048 x 768: 92 us with the maps' pass, 104 cut
// for 512; 1 x 16384 x 1536: 632 and 615).  Up to 2048 / N tokens they are left whole (with the forward, 1 x 128 x 512: 37
// us, 41 cut; 192: 48 and 42).  A compute unit holds one workgroup, so w of them, up to 4 rounds, leave the last round
// partly empty.  There sequences are cut once, into a long segment and the rest: a unit without a long one in the last round
// takes k rests one after the other, which are as long together.  That is worth r / (k + 1) of a sequence's tiles (2 at least)
// and costs the rests' maps (with the forward, 4 x 4096 x 1536, w = 192: 714 us, 791 whole; 4 x 2048 x 1024, w = 128: 282,
// 360; 3 x 500 x 1536, w = 144: 114, 118).
inline int ssm_segment_bwd(const SeqMap &q, int D, int N) {
  const int64_t w = (int64_t)q.n * ((D + SSM_BWD_CH - 1) / SSM_BWD_CH), rounds = (w + 255) / 256, idle = rounds * 256 - w;
  if (!q.cu && w >= 128 && rounds <= 4 && idle) {
    const int64_t k = (w + idle - 1) / idle;
    if ((int64_t)q.T * rounds >= 128 * (k + 1)) return (int)(((int64_t)q.T * k / (k + 1) + SSM_ALIGN) / SSM_ALIGN * SSM_ALIGN);
  }
  return ssm_segment(q, D, SSM_BWD_CH, 128, 256, 2048 / N);
}

}  // namespace falcon
