// Internal interfaces of the operators around the recurrence (block_api.cu to
// conv.cu, scan_fwd.cu, scan_bwd.cu, group_norm.cu, norm_sequence.cu, norm_resident.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mlstm {

// A strided tensor, as mlstm_rows_t: element (b, t, g, j) at p[b sb + t st + g sh + j].
struct Rows {
  void* p = nullptr;
  long long sb = 0, st = 0, sh = 0;
};

enum { kActNone = 0, kActSilu = 1, kActSigmoid = 2 };

// MLSTM_OK, or MLSTM_ERR_CUDA with the error's text kept for mlstm_last_error.
int cuda_result(cudaError_t e, const char* where);

// dw[c, j] = sum over rows of partial[row, j, c] for j < W, dbias[c] = that of j = W; partial is
// [rows, W + 1, D].  Either output may be null.
cudaError_t launch_param_sums(const float* partial, int rows, int D, int W, float* dw, float* dbias,
                              cudaStream_t s);

// ---- causal convolution ----------------------------------------------------
struct ConvArgs {
  Rows x, y;                    // y: dy in the backward
  const float *w, *bias;        // [D, W], [D] or null
  const void* state_in;         // [B, W - 1, D] or null
  void* state_out;              // forward: or null
  Rows dx;                      // backward
  const void* dstate_out;       // backward: or null
  void* dstate_in;              // backward: or null
  float *dw, *dbias;            // backward; dbias or null
  float* partial;               // backward: [conv_bwd_rows, W + 1, D]
  int B, T, NH, d, W, act, dtype;
  bool wide;                    // 16-byte accesses are possible everywhere
  __host__ __device__ int D() const { return NH * d; }
};
int conv_bwd_rows(int B, int T, int D);  // rows of partial sums
cudaError_t launch_conv_fwd(const ConvArgs& a, cudaStream_t s);
cudaError_t launch_conv_step(const ConvArgs& a, cudaStream_t s);
cudaError_t launch_conv_bwd(const ConvArgs& a, cudaStream_t s);

// ---- selective scan ----------------------------------------------------------
struct ScanArgs {
  Rows x, dt, z, b, c;          // z.p null: no gate
  const float *A, *skip, *dt_bias;
  const float* state_in;
  Rows y;                       // forward output, or dy
  float* state_out;
  float* saved;                 // [B, ceil(T / 8), D, scan_pad(N)]; forward: or null
  // backward
  Rows dx, ddt, dz, db, dc;
  float *dA, *dskip, *ddt_bias, *dstate_in;
  const float* dstate_out;
  float *part_bc, *part_a, *part_d;
  // the sequence's segments (one: the whole of it).  At once: seg_state and seg_sum hold each
  // segment's own state and its sum of delta, [segs, B, D, scan_pad(N)] and [segs, B, D].  In turn:
  // seg_state is the state handed from a segment to the next, [B, D, scan_pad(N)], and `turn` the
  // launch's abort word, a counter of taken items and each channel tile's finished segments, zero at the
  // launch.
  float *seg_state, *seg_sum;
  unsigned int* turn;
  int seg_len, segs;
  bool in_turn;
  int B, T, D, G, N, softplus, dtype;
  bool wide, wide_bc;           // 16-byte accesses of the [B, T, D] tensors / of B and C
};
constexpr int kScanEvery = 8;  // tokens between two saved states
constexpr int kTurnAbort = 0, kTurnNext = 1, kTurnTiles = 2;  // words of ScanArgs::turn
// States per channel as the kernels hold them: four to a lane, 2, 4, 8 or 16 lanes to a channel.
inline int scan_pad(int N) { return N <= 8 ? 8 : N <= 16 ? 16 : N <= 32 ? 32 : 64; }
// How a pass cuts the sequence: into `count` segments of `len` tokens (a multiple of the kernels'
// tiles), worked on at once where whole sequences are too few to fill the GPU, or in turn, each
// segment's work taken up by whichever CTA is free, where they are so many that the last round of
// CTAs would leave SMs idle.
struct ScanSegments {
  int len, count;
  bool in_turn;
  int tiles;                    // CTAs of a segment (channel tiles of all batches)
};
ScanSegments scan_fwd_segments(int B, int T, int D, int G, int N);
ScanSegments scan_bwd_segments(int B, int T, int D, int G, int N);
// tile: tokens that segments are multiples of; ctas: those of an undivided scan; slots: CTAs that the GPU
// holds at once.
ScanSegments scan_cut(int T, int tile, long long ctas, int slots);
struct ScanBwdSizes {
  int tiles;                    // channel tiles of one group
  size_t part_bc, part_a, part_d;  // floats
};
ScanBwdSizes scan_bwd_sizes(int B, int T, int D, int G, int N);
cudaError_t launch_scan_fwd(const ScanArgs& a, cudaStream_t s);
cudaError_t launch_scan_step(const ScanArgs& a, cudaStream_t s);
cudaError_t launch_scan_reverse_segments(const ScanArgs& a, cudaStream_t s);
cudaError_t launch_scan_bwd(const ScanArgs& a, cudaStream_t s);
// Where a family counts its launches that gave up a wait (see LaunchAbort), and a launch that does: `words`
// are two, zero.
cudaError_t scan_fwd_flag(unsigned int** at);
cudaError_t scan_bwd_flag(unsigned int** at);
cudaError_t launch_scan_fwd_selftest(unsigned int* words, cudaStream_t s);
cudaError_t launch_scan_bwd_selftest(unsigned int* words, cudaStream_t s);

// ---- group norm --------------------------------------------------------------
struct NormArgs {
  Rows x, gate, y;              // y: dy in the backward
  Rows dx, dgate;
  const float *w, *bias;        // [NH d] or null
  float* stats;                 // (mean, rstd) pairs; forward: or null
  float *dw, *dbias;            // or null
  float* ws;
  int B, T, NH, d, scope, act, dtype;
  float eps;
  bool wide;
};
size_t norm_workspace(int B, int T, int NH, int d, int scope, int dtype, bool backward);  // bytes
cudaError_t launch_norm_fwd(const NormArgs& a, cudaStream_t s);
cudaError_t launch_norm_bwd(const NormArgs& a, cudaStream_t s);
// the sequence scope's part (norm_sequence.cu)
// items of its queue, which must stay below 2^31
long long norm_sequence_items(int B, int T, int NH, int d);
size_t norm_sequence_workspace(int B, int T, int NH, int d, int dtype, bool backward);
cudaError_t launch_norm_sequence(const NormArgs& a, bool backward, cudaStream_t s);
cudaError_t norm_flag(unsigned int** at);
cudaError_t launch_norm_selftest(unsigned int* words, cudaStream_t s);
// Groups that fit the shared memory of a cluster (norm_resident.cu); false: norm_sequence.cu takes them.
bool norm_resident_workspace(int B, int T, int NH, int d, int dtype, bool gated, bool backward, size_t* bytes);
bool launch_norm_resident(const NormArgs& a, bool backward, cudaStream_t s, cudaError_t* status);

}  // namespace mlstm
