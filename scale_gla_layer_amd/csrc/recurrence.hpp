// Launch parameters of the gated linear recurrence.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace msgla {

struct RecRows {
  void* p;
  int64_t sb, st;  // element strides of a sequence and of a position
};

// A wave takes REC_NT consecutive positions, a workgroup as many waves' as make
// its chunk; every REC_GROUP chunks the state itself passes between workgroups.
// The backward keeps four values of each position and channel in registers, so
// that smaller workgroups leave room for a second one to load while the first
// waits (of 4, 8 and 16 waves of 8 and 16 positions, measured; at B = 16, L =
// 4093, D = 1024: 177 us with 4 waves of 16, 190 with 8, 170 with 8 of 8, which
// take 72 us against 59 at B = 8, L = 2048).
constexpr int REC_NT = 16, REC_WAVES = 8, REC_BWAVES = 4, REC_GROUP = 16;
constexpr int REC_CHUNK = REC_NT * REC_WAVES, REC_BCHUNK = REC_NT * REC_BWAVES;

struct RecParams {
  RecRows x, z, y;    // y: the forward's output
  RecRows dy, dx, dz; // the backward's
  const float* bias;
  const uint8_t* mask;
  const float* h_in;
  float* h_out;
  const float* dh_out;
  float* dbias;
  float* dh_in;
  uint64_t *maps, *ends;    // [B][nch][D] chunk maps {A, H}, [B][groups][D] states {0, h}
  uint64_t *rmaps, *rends;  // the backward's, from the other end; the four lie one after the other
  int64_t words;            // of the four (forward: of the two)
  uint32_t* counters;       // [2][B slabs] chunks begun, forward and backward
  float* entry;             // [B][nchb][D] states that enter the backward's chunks
  float* dbp;               // [B nchb][D] dbias partials
  int B, L, D, slabs;
  int nch, groups, nchb, groupsb;  // chunks and their groups, forward and backward
  float inv_gamma;
};

hipError_t launch_recurrence_forward(const RecParams& P, int input, bool bf16_path, bool vec, hipStream_t st);
hipError_t launch_recurrence_backward(const RecParams& P, int input, bool bf16_path, bool vec, hipStream_t st);
hipError_t launch_recurrence_step(const RecParams& P, int input, bool bf16_path, bool vec, hipStream_t st);

}  // namespace msgla
