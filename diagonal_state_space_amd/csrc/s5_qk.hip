// Norm of each query and key head and rotation of its first R features by
// position * frequency, in one pass over q and k, and the gradients of that
// pass.
//
//   n = x r,  r = 1/sqrt(inv_m sum x^2 + eps)   (inv_m = 1/D or 1; r = 1 without a norm)
//   y = Rot(n w),  Rot: (a, b) -> s (a cos - b sin, b cos + a sin) on each pair
// backward, with d = Rot^T(dy):
//   dw = sum over rows of d n,   dx = r (d w - n inv_m (n . d w))
//
// A row (token, head) is held by G lanes, a lane holding U units of two chunks
// of V consecutive features, chosen so that both members of a pair are in one
// lane: in the half layout chunks u and u + R/2V, in the interleaved one chunks
// 2u and 2u + 1. So the rotation needs no exchange and only the sum of squares
// crosses lanes. With V features of 16 bytes a wave reads and writes whole
// lines; odd sizes, strides and bases take V = 1. The angles of a tile of
// tokens are computed once for all heads, into LDS: position * frequency in
// float64 turns (a float32 product loses the angle of far positions), whole
// turns dropped, then sine and cosine in float32.
// The pass is bound by the bytes of q and k in and out.
#include <algorithm>

#include "s5_common.h"
#include "s5_delta.h"

namespace s5 {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTile = 8;        // tokens whose angles a workgroup holds at once
constexpr int kBackwardBlocks = 1024;

template <bool BF16, int V>
__device__ __forceinline__ void load_chunk(const void* p, int64_t i, float (&x)[V]) {
  if constexpr (V == 1) {
    if constexpr (BF16) x[0] = bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
    else x[0] = static_cast<const float*>(p)[i];
  } else if constexpr (BF16) {
    const uint4 r = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = __uint_as_float(w[j] << 16);
      x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  } else {
    const float4 r = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    x[0] = r.x; x[1] = r.y; x[2] = r.z; x[3] = r.w;
  }
}

template <bool BF16, int V>
__device__ __forceinline__ void store_chunk(void* p, int64_t i, const float (&x)[V]) {
  if constexpr (V == 1) {
    if constexpr (BF16) static_cast<uint16_t*>(p)[i] = f32_to_bf16(x[0]);
    else static_cast<float*>(p)[i] = x[0];
  } else if constexpr (BF16) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = f32_to_bf16(x[2 * j]) | (static_cast<uint32_t>(f32_to_bf16(x[2 * j + 1])) << 16);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = uint4{w[0], w[1], w[2], w[3]};
  } else {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = float4{x[0], x[1], x[2], x[3]};
  }
}

template <bool BF16, int V, bool GRAD, bool INSIDE>
__global__ void __launch_bounds__(kThreads) k_qk(QkArgs a, int G, int tile) {
  constexpr int U = V == 1 ? 2 : 1;
  extern __shared__ __align__(16) float s_mem[];
  float2* s_cs = reinterpret_cast<float2*>(s_mem);      // [tile][R/2] cosine, sine
  const int tid = threadIdx.x;
  const int RP = a.R >> 1;                               // rotated pairs
  const int lane = tid & (G - 1);
  const int slot = tid / G, slots = kThreads / G;        // rows a pass of the workgroup handles
  const int heads = a.Hq + a.Hk;
  const int chunks = a.D / V;

  int c0[U], c1[U];      // the unit's chunks; chunks and beyond: none
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int u = lane + j * G;
    if (a.interleaved || u >= RP / V) {
      // interleaved: 2u; the rest of a half layout: from R on, two by two
      c0[j] = a.interleaved ? 2 * u : 2 * (RP / V) + 2 * (u - RP / V);
      c1[j] = c0[j] + 1;
    } else {
      c0[j] = u;
      c1[j] = u + RP / V;
    }
  }
  float w[2][U][2][V];   // weights of q and k at this lane's features
  float dw[2][U][2][V];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const float* p = m == 0 ? a.wq : a.wk;
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int c = h == 0 ? c0[j] : c1[j];
          w[m][j][h][i] = p != nullptr && c < chunks ? p[c * V + i] : 1.0f;
          dw[m][j][h][i] = 0.0f;
        }
  }

  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * tile; t0 < a.T; t0 += static_cast<int64_t>(gridDim.x) * tile) {
    const int nt = static_cast<int>(a.T - t0 < tile ? a.T - t0 : tile);
    __syncthreads();     // the previous tile's angles are read
    for (int i = tid; i < nt * RP; i += kThreads) {
      const int t = i / RP, p = i - t * RP;
      const int64_t pos = a.positions ? a.positions[t0 + t] : (t0 + t) % a.L;
      const double turns = static_cast<double>(pos) * (a.freqs[p] * 0.15915494309189533577);
      float sn, cs;
      sincospif(2.0f * static_cast<float>(turns - rint(turns)), &sn, &cs);
      s_cs[i] = float2{a.rope_scale * cs, a.rope_scale * sn};
    }
    __syncthreads();
    const int rows = nt * heads;
    for (int r0 = 0; r0 < rows; r0 += slots) {
      const int row = r0 + slot;
      const bool live = row < rows;
      const int t = live ? row / heads : 0, hh = live ? row - t * heads : 0;
      const int m = hh < a.Hq ? 0 : 1;
      const int64_t in = m == 0 ? (t0 + t) * a.ldq + static_cast<int64_t>(hh) * a.D
                                : (t0 + t) * a.ldk + static_cast<int64_t>(hh - a.Hq) * a.D;
      const int64_t out = m == 0 ? ((t0 + t) * a.Hq + hh) * a.D : ((t0 + t) * a.Hk + hh - a.Hq) * a.D;
      const void* src = m == 0 ? a.q : a.k;
      float x[U][2][V], d[U][2][V];
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < U; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c = h == 0 ? c0[j] : c1[j];
          if (live && c < chunks) {
            load_chunk<BF16, V>(src, in + c * V, x[j][h]);
            if constexpr (GRAD) load_chunk<BF16, V>(m == 0 ? a.dq_out : a.dk_out, out + c * V, d[j][h]);
          } else {
#pragma unroll
            for (int i = 0; i < V; ++i) x[j][h][i] = d[j][h][i] = 0.0f;
          }
#pragma unroll
          for (int i = 0; i < V; ++i) sum = fmaf(x[j][h][i], x[j][h][i], sum);
        }
      float r = 1.0f;
      if (a.norm) {
        for (int o = 1; o < G; o <<= 1) sum += __shfl_xor(sum, o);
        r = 1.0f / sqrtf(fmaf(sum, a.inv_m, a.eps));
      }
      // rotates the values of the unit (forward) or turns them back (gradient)
      auto rotate = [&](float (&v)[U][2][V]) {
#pragma unroll
        for (int j = 0; j < U; ++j) {
          const int u = lane + j * G;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const int p = u * V + i;
            if (p < RP) {
              float2 cs = s_cs[t * RP + p];
              if constexpr (GRAD) cs.y = -cs.y;
              float& e = v[j][INSIDE ? (2 * i) / V : 0][INSIDE ? (2 * i) % V : i];
              float& f = v[j][INSIDE ? (2 * i + 1) / V : 1][INSIDE ? (2 * i + 1) % V : i];
              const float e0 = e, f0 = f;
              e = e0 * cs.x - f0 * cs.y;
              f = f0 * cs.x + e0 * cs.y;
            }
          }
        }
      };
      if constexpr (!GRAD) {
#pragma unroll
        for (int j = 0; j < U; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < V; ++i) x[j][h][i] *= r * (m == 0 ? w[0][j][h][i] : w[1][j][h][i]);
        rotate(x);
      } else {
        rotate(d);
        float dot = 0.0f;
#pragma unroll
        for (int j = 0; j < U; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < V; ++i) {
              const float n = x[j][h][i] * r;
              const float dn = d[j][h][i] * n;
              if (m == 0) dw[0][j][h][i] += dn; else dw[1][j][h][i] += dn;
              const float e = d[j][h][i] * (m == 0 ? w[0][j][h][i] : w[1][j][h][i]);
              dot = fmaf(e, n, dot);
              d[j][h][i] = e;
              x[j][h][i] = n;
            }
        if (a.norm) {
          for (int o = 1; o < G; o <<= 1) dot += __shfl_xor(dot, o);
          dot *= a.inv_m;
        } else {
          dot = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < U; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < V; ++i) x[j][h][i] = r * (d[j][h][i] - x[j][h][i] * dot);
      }
      if (live) {
        void* dst = m == 0 ? a.q_out : a.k_out;
#pragma unroll
        for (int j = 0; j < U; ++j) {
          if (c0[j] < chunks) store_chunk<BF16, V>(dst, out + c0[j] * V, x[j][0]);
          if (c1[j] < chunks) store_chunk<BF16, V>(dst, out + c1[j] * V, x[j][1]);
        }
      }
    }
  }

  if constexpr (GRAD) {
    if (a.partials == nullptr) return;
    // sums over the workgroup's slots: one feature's sums sit in the lanes of
    // one place in the groups; slot by slot through LDS, in a fixed order
    float* s_dw = s_mem;   // [slots][2][D]
    __syncthreads();
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int j = 0; j < U; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c = h == 0 ? c0[j] : c1[j];
          if (c < chunks) {
#pragma unroll
            for (int i = 0; i < V; ++i) s_dw[(slot * 2 + m) * a.D + c * V + i] = dw[m][j][h][i];
          }
        }
    __syncthreads();
    for (int i = tid; i < 2 * a.D; i += kThreads) {
      float s = 0.0f;
      for (int b = 0; b < slots; ++b) s += s_dw[b * 2 * a.D + i];
      a.partials[static_cast<int64_t>(blockIdx.x) * 2 * a.D + i] = s;
    }
  }
}

// dw[i] = sum over the workgroups' partial rows, in float64 and a fixed order
__global__ void __launch_bounds__(kThreads) k_qk_weights(const float* partials, int blocks, int D, float* dwq, float* dwk) {
  __shared__ double s_sum[kThreads];
  const int i = blockIdx.x;          // feature of q (i < D) or of k
  double s = 0.0;
  for (int b = threadIdx.x; b < blocks; b += kThreads) s += partials[static_cast<int64_t>(b) * 2 * D + i];
  s_sum[threadIdx.x] = s;
  __syncthreads();
  for (int o = kThreads / 2; o > 0; o >>= 1) {
    if (static_cast<int>(threadIdx.x) < o) s_sum[threadIdx.x] += s_sum[threadIdx.x + o];
    __syncthreads();
  }
  float* dst = i < D ? dwq : dwk;
  if (threadIdx.x == 0 && dst != nullptr) dst[i < D ? i : i - D] = static_cast<float>(s_sum[0]);
}

__global__ void k_zero(float* p, int n) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) p[i] = 0.0f;
}

bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// whether whole 16-byte chunks of V features can be moved and hold pairs whole
bool vectored(const QkArgs& a, bool backward, int V) {
  return a.D % V == 0 && a.ldq % V == 0 && a.ldk % V == 0 && (a.interleaved || (a.R / 2) % V == 0) && aligned(a.q) &&
         aligned(a.k) && aligned(a.q_out) && aligned(a.k_out) &&
         (!backward || (aligned(a.dq_out) && aligned(a.dk_out)));
}

int lanes_of(const QkArgs& a, int V) {
  const int units = (a.D / V + 1) / 2;
  int G = 1;
  while (G < units && G < 64) G <<= 1;
  return G;
}

// tokens of a tile: up to eight share a workgroup's angles; fewer while that
// would leave compute units without a workgroup
int tile_of(const QkArgs& a) {
  int tile = kMaxTile;
  while (tile > 1 && a.T / tile < 1024) tile >>= 1;
  return tile;
}

// INSIDE: pairs sit inside a chunk, else across a unit's two chunks
template <bool BF16, int V, bool GRAD, bool INSIDE>
hipError_t run(const QkArgs& a, hipStream_t stream) {
  const int G = lanes_of(a, V), tile = tile_of(a);
  int64_t blocks = (a.T + tile - 1) / tile;
  blocks = std::min<int64_t>(blocks, GRAD ? kBackwardBlocks : 1 << 20);
  size_t lds = static_cast<size_t>(tile) * (a.R / 2) * sizeof(float2);
  if (GRAD) lds = std::max(lds, static_cast<size_t>(kThreads / G) * 2 * a.D * sizeof(float));
  k_qk<BF16, V, GRAD, INSIDE><<<dim3(static_cast<unsigned>(blocks)), dim3(kThreads), lds, stream>>>(a, G, tile);
  hipError_t e = hipGetLastError();
  if (GRAD && e == hipSuccess && a.partials != nullptr) {
    k_qk_weights<<<dim3(2 * a.D), dim3(kThreads), 0, stream>>>(a.partials, static_cast<int>(blocks), a.D, a.dwq, a.dwk);
    e = hipGetLastError();
  }
  return e;
}

template <bool BF16, int V, bool GRAD>
hipError_t dispatch(const QkArgs& a, hipStream_t stream) {
  if (!vectored(a, GRAD, V)) return run<BF16, 1, GRAD, false>(a, stream);
  return a.interleaved ? run<BF16, V, GRAD, true>(a, stream) : run<BF16, V, GRAD, false>(a, stream);
}

}  // namespace

int qk_partial_blocks(const QkArgs& a) {
  const int tile = tile_of(a);
  return static_cast<int>(std::min<int64_t>((a.T + tile - 1) / tile, kBackwardBlocks));
}

hipError_t launch_zero(float* p, int n, hipStream_t stream) {
  k_zero<<<dim3(1), dim3(kThreads), 0, stream>>>(p, n);
  return hipGetLastError();
}

hipError_t launch_qk(const QkArgs& a, bool backward, hipStream_t stream) {
  if (a.bf16_io) return backward ? dispatch<true, 8, true>(a, stream) : dispatch<true, 8, false>(a, stream);
  return backward ? dispatch<false, 4, true>(a, stream) : dispatch<false, 4, false>(a, stream);
}

}  // namespace s5
