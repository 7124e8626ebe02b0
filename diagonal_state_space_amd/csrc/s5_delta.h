// Internal launcher declarations of the gated delta rule and of the pass that
// prepares its queries and keys (validated arguments; include/s5.h has the
// contracts).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace s5 {

// Norm and rotation of query and key heads: rows of T tokens and Hq + Hk heads.
struct QkArgs {
  int64_t T, L;            // tokens; position of token t without `positions`: t % L
  int Hq, Hk, D, R;        // heads, features of a head, rotated features (even, <= D)
  int64_t ldq, ldk;        // elements between the tokens of q and of k
  bool bf16_io, interleaved, norm;
  float inv_m;             // 1/D (root mean square) or 1 (Euclidean)
  float eps, rope_scale;
  const void *q, *k;
  const float *wq, *wk;    // [D] or null
  const double* freqs;     // [R/2] radians per position
  const int32_t* positions;  // [T] or null
  void *q_out, *k_out;     // contiguous; backward: the gradients of q and k
  // backward only
  const void *dq_out, *dk_out;   // contiguous
  float *dwq, *dwk;              // [D] or null
  float* partials;               // qk_partial_blocks() * 2 * D floats, with dwq or dwk
};

// workgroups of the backward pass, each of which leaves one row of partial
// weight gradients
int qk_partial_blocks(const QkArgs& a);
hipError_t launch_qk(const QkArgs& a, bool backward, hipStream_t stream);
hipError_t launch_zero(float* p, int n, hipStream_t stream);

// Gated delta rule over B sequences of up to L tokens. Strides are at most
// kMostStride elements where a sequence has several tokens.
constexpr int64_t kMostStride = int64_t{1} << 22;
struct DeltaArgs {
  int B, L, Hk, Hv, Dk, Dv;
  int Nk, Nv;              // heads in a token's row of the contiguous arrays: Hk, Hv, or more in a slice of the heads
  int64_t ldq, ldk, ldv;   // elements between the tokens of q, k and v
  bool bf16_io;
  float scale;
  const void *q, *k, *v;
  const float *g, *beta;   // [B, L, Hv]
  const float* s0;         // [B, Hv, Dk, Dv] or null (zero)
  const int32_t* lengths;  // [B] or null (all L)
  void* y;                 // [B, L, Hv, Dv]
  float* s_last;           // [B, Hv, Dk, Dv] or null; may be s0 itself
  void* ws;
  unsigned char *frags, *recs;   // in ws: fragments of k and q by columns (backward), records of the chunks
  // backward only
  const void* dy;
  const float* ds_last;    // or null (zero)
  void *dq, *dk, *dv;
  float *dg, *dbeta;
  float* ds0;              // or null
};

// one token of each sequence, the state (s0 = s_last) in place
hipError_t launch_delta_step(const DeltaArgs& a, hipStream_t stream);

// What the chains leave for the gradients of a chunk (float32, columns padded
// with zeros to 16), one after the other for each of [B*Hv][chunks]: the state S
// at its start and the gradient D' of its end state [dkp][dvp], its writes U and
// their gradients dR [C][dvp]. Each is stored as the accumulators' tiles, those
// of 16 columns one after the other: four rows of a column in 16 bytes.
struct DeltaKeep {
  float* p;
  float* sums;   // gradients' workgroups' sums of dq and dk over the heads of a key (bf16, 64 features)
  int dkp, dvp;
  __host__ __device__ int at_d() const { return dkp * dvp; }
  __host__ __device__ int at_u() const { return 2 * dkp * dvp; }
  __host__ __device__ int at_r(int C) const { return (2 * dkp + C) * dvp; }
  __host__ __device__ int size(int C) const { return 2 * (dkp + C) * dvp; }
};

// Long sequences of few heads are cut into `count` segments of `chunks` chunks
// that run side by side: their states from a zero start, with the product of
// their transitions, are found first and joined in order. Of every [B*Hv]
// [segment]: [dkp][dvp + dkp] floats, the state from zero (after the join the
// state at the segment's end; of the last segment the sequence's start) and the
// transition; backward also [dkp][dvp], the
// gradient of the state at the segment's start.
struct DeltaSegs {
  float *p, *back;
  int count, chunks, dkp, dvp;
  __host__ __device__ int ld() const { return dvp + dkp; }
  __host__ __device__ int64_t at(int64_t bh, int seg) const { return (bh * count + seg) * dkp * ld(); }
  __host__ __device__ int64_t at_back(int64_t bh, int seg) const { return (bh * count + seg) * dkp * dvp; }
};

// Whether a chain's workgroups have 32 columns each instead of 64: where all of
// `chains` (heads, segments) with `columns` then run at once, one on a compute
// unit. Fewer waves share its LDS and memory paths: the chains of 64 heads of
// 2048 tokens at 128 x 128, bf16, took 90, 109 and 160 us instead of 94, 113, 168.
constexpr int64_t kUnits = 256;
inline bool narrow_groups(int64_t chains, int columns) { return chains * ((columns + 31) / 32) <= kUnits; }

// The chunked form: preparation of all chunks, then the chunks in order (with
// `keep` no outputs but S and U for the backward pass). delta_work finds the
// workspace's parts and gives the bytes of fragments, records and segments.
int64_t delta_work(DeltaArgs& a, DeltaSegs& segs, bool backward);
hipError_t launch_delta_prep(const DeltaArgs& a, bool backward, hipStream_t stream);
hipError_t launch_delta_scan(const DeltaArgs& a, const DeltaSegs& segs, const DeltaKeep* keep, hipStream_t stream);
// the gradients at the segments' starts from those of their sums
hipError_t launch_delta_join_back(const DeltaArgs& a, const DeltaSegs& segs, hipStream_t stream);

// whole sequences; bytes of workspace they need
int64_t delta_workspace(const DeltaArgs& a, bool backward);
hipError_t launch_delta(const DeltaArgs& a, hipStream_t stream);
hipError_t launch_delta_backward(const DeltaArgs& a, hipStream_t stream);

}  // namespace s5
