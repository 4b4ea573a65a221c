// Launch parameters of the gated linear recurrence.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace msgla {

struct RecRows {
  void* p;
  int64_t sb, st;  // element strides of a sequence and of a position
};

// A workgroup takes REC_CHUNK positions, its waves equal parts of them one after
// the other (fewer a wave backward, which keeps five values of each); every
// REC_GROUP chunks the state itself passes between workgroups.
constexpr int REC_CHUNK = 128, REC_FWD_WAVES = 8, REC_BWD_WAVES = 16, REC_GROUP = 16;

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
  uint64_t *rmaps, *rends;  // the same from the other end; the four lie one after the other
  int64_t words;            // of the four (forward: of the two)
  uint32_t* counters;       // [2][B slabs] chunks begun, forward and backward
  float* entry;             // [B][nch][D] states that enter the chunks, for the backward
  float* dbp;               // [B nch][D] dbias partials
  int B, L, D, nch, groups, slabs;
  float inv_gamma;
};

hipError_t launch_recurrence_forward(const RecParams& P, int input, bool bf16_path, bool vec, hipStream_t st);
hipError_t launch_recurrence_backward(const RecParams& P, int input, bool bf16_path, bool vec, hipStream_t st);
hipError_t launch_recurrence_step(const RecParams& P, int input, bool bf16_path, bool vec, hipStream_t st);

}  // namespace msgla
