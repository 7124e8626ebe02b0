// One token of the gated delta rule for each sequence, the state in registers:
// read once, written once.
//
//   Sd = a S,  u = beta (v - Sd^T k),  S <- Sd + k u^T,  y = scale S^T q
// Both products with the old state come from one pass over it, since
//   S_new^T q = a S^T q + (k.q) u.
//
// The state's bytes bound it. A workgroup has 32 columns of one head's state, so
// that a row's piece is a cache line of 128 bytes; each thread has four columns
// of every 32nd row (four 16-byte loads, all under way before the first use),
// or, where rows are not of whole 16-byte groups, one column of every 8th.
// 128 sequences of 32 heads of 128 x 128 (537 MB): 104 us, 5.2 TB/s, as a copy.
#include "s5_common.h"
#include "s5_delta.h"

namespace s5 {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kCols = 32;        // columns of a workgroup: 128-byte row segments
constexpr int kMaxDk = 128;

template <bool BF16>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if constexpr (BF16) return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
  else return static_cast<const float*>(p)[i];
}

// V: columns of a thread, 4 with 16-byte rows of the state, else 1
template <bool BF16, int V>
__global__ void __launch_bounds__(kThreads) k_delta_step(DeltaArgs a) {
  constexpr int CL = kCols / V;              // column lanes
  constexpr int RG = kThreads / CL;          // rows side by side
  constexpr int NR = kMaxDk / RG;            // rows of a thread
  __shared__ float s_k[kMaxDk], s_q[kMaxDk];
  __shared__ float s_red[kWaves][2][kCols];
  const int tid = threadIdx.x, wave = tid >> 6;
  const int cl = tid % CL, rg = tid / CL;
  const int tiles = (a.Dv + kCols - 1) / kCols;
  const int ct = blockIdx.x % tiles;
  const int bh = blockIdx.x / tiles;
  const int b = bh / a.Hv, h = bh - b * a.Hv;
  const int hk = h / (a.Hv / a.Hk);
  const int col = ct * kCols + cl * V;
  const bool has = col < a.Dv;               // V = 4: Dv % 4 == 0, all or none

  const int64_t base = static_cast<int64_t>(bh) * a.Dk * a.Dv + col;
  float S[NR][V];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int row = i * RG + rg;
#pragma unroll
    for (int c = 0; c < V; ++c) S[i][c] = 0.0f;
    if (has && row < a.Dk) {
      const float* p = a.s0 + base + static_cast<int64_t>(row) * a.Dv;
      if constexpr (V == 4) {
        const float4 r = *reinterpret_cast<const float4*>(p);
        S[i][0] = r.x; S[i][1] = r.y; S[i][2] = r.z; S[i][3] = r.w;
      } else {
        S[i][0] = *p;
      }
    }
  }

  if (tid < kMaxDk) {
    s_k[tid] = tid < a.Dk ? load1<BF16>(a.k, b * a.ldk + static_cast<int64_t>(hk) * a.Dk + tid) : 0.0f;
  } else if (tid < 2 * kMaxDk) {
    const int j = tid - kMaxDk;
    s_q[j] = j < a.Dk ? load1<BF16>(a.q, b * a.ldq + static_cast<int64_t>(hk) * a.Dk + j) : 0.0f;
  }
  float v[V];
#pragma unroll
  for (int c = 0; c < V; ++c)
    v[c] = has ? load1<BF16>(a.v, b * a.ldv + static_cast<int64_t>(h) * a.Dv + col + c) : 0.0f;
  const float decay = expf(a.g[b * a.Hv + h]), beta = a.beta[b * a.Hv + h];
  __syncthreads();
  float kk[NR], pk[V], pq[V], kq = 0.0f;
#pragma unroll
  for (int c = 0; c < V; ++c) pk[c] = pq[c] = 0.0f;
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    kk[i] = s_k[i * RG + rg];
    const float qq = s_q[i * RG + rg];
#pragma unroll
    for (int c = 0; c < V; ++c) {
      pk[c] = fmaf(S[i][c], kk[i], pk[c]);
      pq[c] = fmaf(S[i][c], qq, pq[c]);
    }
  }
  for (int j = tid & 63; j < kMaxDk; j += 64) kq = fmaf(s_k[j], s_q[j], kq);
  for (int o = 1; o < 64; o <<= 1) kq += __shfl_xor(kq, o);
#pragma unroll
  for (int o = CL; o < 64; o <<= 1)
#pragma unroll
    for (int c = 0; c < V; ++c) {
      pk[c] += __shfl_xor(pk[c], o);
      pq[c] += __shfl_xor(pq[c], o);
    }
  if ((tid & 63) < CL) {
#pragma unroll
    for (int c = 0; c < V; ++c) {
      s_red[wave][0][cl * V + c] = pk[c];
      s_red[wave][1][cl * V + c] = pq[c];
    }
  }
  __syncthreads();
  float u[V], y[V];
#pragma unroll
  for (int c = 0; c < V; ++c) {
    float sk = 0.0f, sq = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      sk += s_red[w][0][cl * V + c];
      sq += s_red[w][1][cl * V + c];
    }
    u[c] = beta * (v[c] - decay * sk);
    y[c] = a.scale * fmaf(kq, u[c], decay * sq);
  }
#pragma unroll
  for (int i = 0; i < NR; ++i)
#pragma unroll
    for (int c = 0; c < V; ++c) S[i][c] = fmaf(kk[i], u[c], decay * S[i][c]);
  if (rg == 0 && has) {
    const int64_t o = static_cast<int64_t>(bh) * a.Dv + col;
#pragma unroll
    for (int c = 0; c < V; ++c) {
      if constexpr (BF16) static_cast<uint16_t*>(a.y)[o + c] = f32_to_bf16(y[c]);
      else static_cast<float*>(a.y)[o + c] = y[c];
    }
  }

  if (has) {
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int row = i * RG + rg;
      if (row < a.Dk) {
        float* p = a.s_last + base + static_cast<int64_t>(row) * a.Dv;
        if constexpr (V == 4) *reinterpret_cast<float4*>(p) = float4{S[i][0], S[i][1], S[i][2], S[i][3]};
        else *p = S[i][0];
      }
    }
  }
}

}  // namespace

hipError_t launch_delta_step(const DeltaArgs& a, hipStream_t stream) {
  const int64_t blocks = static_cast<int64_t>(a.B) * a.Hv * ((a.Dv + kCols - 1) / kCols);
  const bool vec = a.Dv % 4 == 0;   // the states are 16-byte aligned
  const dim3 grid(static_cast<unsigned>(blocks)), block(kThreads);
  if (a.bf16_io) {
    if (vec) k_delta_step<true, 4><<<grid, block, 0, stream>>>(a);
    else k_delta_step<true, 1><<<grid, block, 0, stream>>>(a);
  } else {
    if (vec) k_delta_step<false, 4><<<grid, block, 0, stream>>>(a);
    else k_delta_step<false, 1><<<grid, block, 0, stream>>>(a);
  }
  return hipGetLastError();
}

}  // namespace s5
