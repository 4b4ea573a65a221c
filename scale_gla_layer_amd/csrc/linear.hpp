// Launch parameters of linear attention with a decay per head.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace msgla {

struct LinHeads {
  char* p;
  int64_t sb, st, sh;  // byte strides of a sequence, a position, a head
};

constexpr int LIN_CHUNK = 64;     // positions of a step of a walk
constexpr int LIN_SEGMENTS = 32;  // parts of a sequence that are walked side by side, at most

// One walk: out_t = scale q_t S_t, S_t = gamma S_{t-1} + k_t^T v_t, from the first
// token to the last or back.
struct LinJob {
  LinHeads q, k, v, o;
  const float* entry;  // [B][H][kw][vw] state before the first step, or NULL
  float* exit;         // the state after the last one, or NULL
  float* part;         // [B][H][segments][kw][vw] states before the segments; first what the one before each adds
  float entry_mul, exit_mul;
  int kw, vw;          // widths of q and k, and of v and o
  int turned;          // from the last token to the first; entry is then not decayed by the first step, exit is once more
  int flip_entry;      // entry is [vw][kw]
  int columns, slices; // of v: a workgroup's, and the workgroups they make
  int segments, seg_chunks;  // segments of so many chunks
};

struct LinParams {
  LinJob job[3];
  int jobs;
  const float* log_decay;
  const int32_t* lens;
  const uint8_t* mask;  // the step's
  int B, L, H;
  float scale;
};

// Columns of v that a workgroup takes.  128 share the work on the keys, where the state's
// two roundings leave LDS for them, at the price of half as many workgroups: they pay for
// keys of more than 64 (padded: kwp) once a launch has as many such walks as CUs, or more
// than two chunks of them a CU.  4 heads of 128 and 256, bf16, us with 128 and with 64
// columns: B = 8, L = 2048 (2048 chunks) 64 and 70, B = 6, L = 1024 (768) 41 and 45, B = 8, L = 512
// (512) 39 and 36, one sequence of 512 34 and 30; B = 32, L = 128 (256 walks) 16.6 and 18.0.  Keys
// of 64 (8 heads of 64 and 128): B = 1, L = 512 31 and 22, B = 4, L = 2048 40 and 35, 16 heads,
// B = 8, L = 2048 83 and 76.  es: bytes of an element.
inline int lin_columns(int es, int kwp, int vw, int64_t walks, int64_t chunks) {
  return es == 2 && kwp == 128 && vw > 64 && (walks >= 256 || chunks > 2 * 256) ? 128 : 64;
}
// Waves that keep the state: eight where one workgroup fills a CU (66 us at the size
// above, with four 98), four where two share one.
constexpr int lin_state_waves(int es, int kwp, int columns) { return es == 2 && kwp * columns >= 128 * 128 ? 8 : 4; }
inline int lin_kwp(int kw) { return kw <= 64 ? 64 : kw <= 128 ? 128 : 256; }

hipError_t launch_linear(const LinParams& P, bool bf16_path, hipStream_t st);
constexpr int LIN_STEP_COLUMNS = 32, LIN_STEP_THREADS = 256;
hipError_t launch_linear_step(const LinParams& P, bool bf16_path, hipStream_t st);

}  // namespace msgla
