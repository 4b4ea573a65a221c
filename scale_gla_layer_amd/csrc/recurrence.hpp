// Launch parameters of the gated linear recurrence.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace msgla {

struct RecRows {
  void* p;
  int64_t sb, st;  // element strides of a sequence and of a position
};

// A workgroup takes REC_CHUNK positions: REC_WAVES waves of REC_T positions
// each, all on the same channels.
constexpr int REC_T = 8, REC_WAVES = 8, REC_CHUNK = REC_T * REC_WAVES;

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
  float* agg;      // [B][nch][D][2]: a chunk's decay product and its state from zero, then its entry state
  float* rev;      // [B][nch][D]: a chunk's gradient carry from zero, then the carry that enters it
  float* dbp;      // [B * nch][D]: dbias partials
  int B, L, D, nch, slabs;
  float inv_gamma;
};

hipError_t launch_recurrence_forward(const RecParams& P, int input, bool bf16_path, bool vec, hipStream_t st);
hipError_t launch_recurrence_backward(const RecParams& P, int input, bool bf16_path, bool vec, hipStream_t st);
hipError_t launch_recurrence_step(const RecParams& P, int input, bool bf16_path, bool vec, hipStream_t st);

}  // namespace msgla
