// Launch descriptors of the learner's inner step (gradient norm, AdamW), shared by
// the host orchestration and the gfx950 kernels.
//
// These calls work on learner rows only.  An element's arithmetic depends on its
// tensor through the tensor's group alone, so the host joins tensors of one group
// that follow each other without padding into one range, and a launch carries up
// to kMaxRanges ranges in its kernel arguments.  Within a launch each range owns a
// contiguous run of blocks (grid x); the present learners are grid y.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace dlc {

constexpr int kMaxRanges = 208;
constexpr int kRangeBuckets = 64;
constexpr int kMaxGroups = 16;
constexpr int kCodeBlock = 64;       // elements that share a scale byte
// AdamW with 32-bit moments: one wave takes 256 elements, four a thread, and is done.  The
// LDS that a block asks for and does not use keeps 11 of them on a CU: what the device then
// works on at a time is a shorter stretch of each of the arrays, and memory serves it
// faster.  1B set, bf16 gradients and working copy, on one machine: 11 blocks a CU 3.62 ms
// (6.6 TB/s), 9: 3.82, 14: 3.72, 20: 3.89, no bound: 4.02; with blocks of 128 threads and 14 waves a
// CU 3.76; runs of 8192 elements per block 4.55, a persistent grid 4.81 and more.
constexpr int kAdamWBlock = 64;
constexpr int kAdamWTile = 4 * kAdamWBlock;
constexpr int kAdamWLds = 14800;
// With coded moments: two waves, two quads a thread 256 elements apart.  Twice the
// arithmetic per byte and code loads of 4 bytes a lane: one quad a thread took 3.20 ms against 2.95
// on eight 135M learners; eight consecutive elements a thread, whose fp32 accesses are no
// longer whole kilobytes a wave, 3.48 against 2.86.  Its registers leave 20 waves a CU; fewer are
// slower.
constexpr int kCodedBlock = 128;
constexpr int kCodedQuads = 2;
constexpr int kCodedTile = 4 * kCodedBlock * kCodedQuads;
// Gradient norm: about kNormBlocks blocks a launch, each with its own run of whole steps of
// kNormBlock threads times kNormLoads 16-byte loads (half or twice the loads and 1024 to
// 16384 blocks are within 4%; steps dealt out in turn are 2% slower).
constexpr int kNormBlock = 256;
constexpr int kNormLoads = 4;
constexpr int kNormStep = kNormBlock * kNormLoads * 16;  // bytes
constexpr int kNormFinal = 1024;     // threads of the final sum

enum FloatType : int32_t { kF32 = 0, kBF16 = 1, kF16 = 2, kNone = -1 };

constexpr int kGroupShift = 28;  // blocks of a launch stay below 2^28

struct InnerRange {
  uint32_t lo64;         // first element of the row, in units of 64
  uint32_t count;        // elements
  uint32_t first_group;  // first block of this range within the launch, and its group << kGroupShift
  __host__ __device__ uint32_t block_first() const { return first_group & ((1u << kGroupShift) - 1); }
  __host__ __device__ uint32_t group() const { return first_group >> kGroupShift; }
};

struct InnerGeom {
  int32_t n_ranges;
  int32_t n_blocks;
  uint32_t per_block;    // elements per block
  int32_t slot_base;     // the launch's first slot of block partials
  int32_t bucket_shift;  // blocks [k << shift, (k + 1) << shift) lie in ranges first .. last of bucket k
  uint32_t bucket[kRangeBuckets];  // first | last << 16
  InnerRange r[kMaxRanges];
};

// Present position -> learner, four to a word: the kernels read words (a byte would be a
// vector load).
struct LearnerList {
  uint32_t word[16];
  __host__ __device__ int operator[](uint32_t k) const { return (int)(word[k >> 2] >> (8 * (k & 3)) & 0xFFu); }
};

struct InnerGroup {
  double lr, beta1, beta2, eps, weight_decay;
  double log_beta1, log_beta2;  // natural logarithms
};

struct AdamWArgs {
  float* theta;               // [n_learners][stride]
  const void* grads;          // [n_learners][stride]
  void* m;                    // fp32, or e4m3 codes
  void* v;                    // fp32, or e5m2 codes
  uint8_t* m_scale;           // [n_learners][stride / 64] (coded moments)
  uint8_t* v_scale;
  void* working;              // 16-bit copy of theta, or NULL
  int64_t* steps;             // [n_learners]
  const double* grad_scale;   // [n_learners], or NULL
  const double* lr_scale;     // [n_learners], or NULL
  int64_t stride;
  uint64_t seed;
  int32_t n_present;
  int32_t tickets;            // blocks per learner where the kernel counts the step itself, else 0
  LearnerList learner;
  InnerGroup group[kMaxGroups];
};

struct NormArgs {
  const void* grads;
  int64_t stride;
  double* part;               // [present][slot] sums of squares
  double* norm;               // [n_learners]
  double* grad_scale;         // [n_learners]
  double unscale, max_norm;
  int32_t n_present;
  int32_t n_slots;
  LearnerList learner;
};

// HIP passes at most 4 KB of kernel arguments.
static_assert(sizeof(AdamWArgs) + sizeof(InnerGeom) <= 4096 && sizeof(NormArgs) + sizeof(InnerGeom) <= 4096);

// Kernel launchers (dlc_inner.hip).  Each returns hipSuccess or the launch error.
hipError_t launch_norm_partial(const NormArgs& a, int32_t grad_type, const InnerGeom& g, hipStream_t s);
// one kernel: a block per learner over all of its ranges, and the final step
hipError_t launch_norm_small(const NormArgs& a, int32_t grad_type, const InnerGeom& g, hipStream_t s);
hipError_t launch_norm_final(const NormArgs& a, hipStream_t s);
hipError_t launch_adamw(const AdamWArgs& a, int32_t grad_type, int32_t working_type, bool coded, const InnerGeom& g,
                        hipStream_t s);
// steps[i] += 1 for every present learner whose step was not left out
hipError_t launch_adamw_advance(const AdamWArgs& a, hipStream_t s);

}  // namespace dlc
