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
// lines; odd sizes, strides and bases take V = 1. A half layout whose R/2 is not
// a multiple of V takes chunks 2u and 2u + 1 too and finds the other members of
// its pairs in a row of LDS (15 x 855 tokens of 7 + 6 heads of 96, 54 rotated, the
// gradients in bf16: 54 us, with V = 1 135). The angles of a tile of
// tokens are computed once for all heads, into LDS: position * frequency in
// float64 turns (a float32 product loses the angle of far positions), whole
// turns dropped, then sine and cosine in float32.
// The pass is bound by the bytes of q and k in and out.
#include <algorithm>
#include <type_traits>

#include "s5_common.h"
#include "s5_delta.h"

namespace s5 {

namespace {

constexpr int kThreads = 256;
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
constexpr int kMaxTile = 16;       // tokens whose angles a workgroup holds at once
constexpr int kBackwardBlocks = 1024;

template <bool BF16, int V>
__device__ __forceinline__ void store_chunk(void* p, int64_t i, const float (&x)[V]) {
  if constexpr (V == 1) {
    if constexpr (BF16) static_cast<uint16_t*>(p)[i] = f32_to_bf16(x[0]);
    else static_cast<float*>(p)[i] = x[0];
  } else if constexpr (BF16) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x[2 * j], x[2 * j + 1]}, bf16x2));
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = uint4{w[0], w[1], w[2], w[3]};
  } else {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = float4{x[0], x[1], x[2], x[3]};
  }
}

// a chunk's bits
template <bool BF16, int V>
struct Raw {
  uint32_t w[V == 1 ? 1 : 4];
};

template <bool BF16, int V>
__device__ __forceinline__ Raw<BF16, V> load_raw(const void* p, int64_t i) {
  Raw<BF16, V> r;
  if constexpr (V == 1) {
    if constexpr (BF16) r.w[0] = static_cast<const uint16_t*>(p)[i];
    else r.w[0] = static_cast<const uint32_t*>(p)[i];
  } else {
    const uint4 x = *reinterpret_cast<const uint4*>(static_cast<const char*>(p) + i * (BF16 ? 2 : 4));
    r.w[0] = x.x; r.w[1] = x.y; r.w[2] = x.z; r.w[3] = x.w;
  }
  return r;
}

template <bool BF16, int V>
__device__ __forceinline__ void values(const Raw<BF16, V>& r, float (&x)[V]) {
  if constexpr (V == 1) {
    x[0] = __uint_as_float(BF16 ? r.w[0] << 16 : r.w[0]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (BF16) {
        x[2 * j] = __uint_as_float(r.w[j] << 16);
        x[2 * j + 1] = __uint_as_float(r.w[j] & 0xffff0000u);
      } else {
        x[j] = __uint_as_float(r.w[j]);
      }
    }
  }
}

// where the members of a pair are: in a unit's two chunks, side by side, or in
// chunks of any lane of the row
enum Pairs { kAcross, kInside, kAnywhere };

template <bool BF16, int V, bool GRAD, Pairs PAIRS>
__global__ void __launch_bounds__(kThreads) k_qk(QkArgs a, int G, int tile) {
  constexpr int U = V == 1 ? 2 : 1;
  extern __shared__ __align__(16) float s_mem[];
  constexpr bool INSIDE = PAIRS == kInside;
  float2* s_cs = reinterpret_cast<float2*>(s_mem);      // [tile][R/2] cosine, sine
  const int tid = threadIdx.x;
  const int RP = a.R >> 1;                               // rotated pairs
  const int lane = tid & (G - 1);
  const int slot = tid / G, slots = kThreads / G;        // rows a pass of the workgroup handles
  const int chunks = a.D / V;

  int c0[U], c1[U];      // the unit's chunks; chunks and beyond: none
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int u = lane + j * G;
    if (PAIRS != kAcross || a.interleaved || u >= RP / V) {
      // 2u; the rest of a half layout: from R on, two by two
      c0[j] = PAIRS != kAcross || a.interleaved ? 2 * u : 2 * (RP / V) + 2 * (u - RP / V);
      c1[j] = c0[j] + 1;
    } else {
      c0[j] = u;
      c1[j] = u + RP / V;
    }
  }
  float* s_row = s_mem + ((2 * tile * RP + 3) & ~3) + slot * a.D;   // pairs anywhere: the row's values
  float dw[2][U][2][V];   // this lane's sums of the weights' gradients
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < V; ++i) dw[m][j][h][i] = 0.0f;

  struct Row {
    Raw<BF16, V> x[U][2], d[U][2];
  };
  // row i of q (m = 0) or k of the tile at t0: its token and head, and its bits
  auto place = [&](int m, int i, int& t, int& hh) {
    const int heads = m == 0 ? a.Hq : a.Hk;
    t = i / heads;
    hh = i - t * heads;
  };
  auto load = [&](int m, int64_t t0, int i, Row& row) {
    int t, hh;
    place(m, i, t, hh);
    const int heads = m == 0 ? a.Hq : a.Hk;
    const int64_t in = (t0 + t) * (m == 0 ? a.ldq : a.ldk) + static_cast<int64_t>(hh) * a.D;
    const int64_t out = ((t0 + t) * heads + hh) * a.D;
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = h == 0 ? c0[j] : c1[j];
        if (c < chunks) {
          row.x[j][h] = load_raw<BF16, V>(m == 0 ? a.q : a.k, in + c * V);
          if constexpr (GRAD) row.d[j][h] = load_raw<BF16, V>(m == 0 ? a.dq_out : a.dk_out, out + c * V);
        } else {
          row.x[j][h] = row.d[j][h] = Raw<BF16, V>{};
        }
      }
  };
  auto compute = [&](auto m_, int64_t t0, int i, bool live, const Row& row, const float (&w)[U][2][V]) {
    constexpr int m = decltype(m_)::value;
    int t, hh;
    place(m, i, t, hh);
    float x[U][2][V], d[U][2][V];
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        values<BF16, V>(row.x[j][h], x[j][h]);
        if constexpr (GRAD) values<BF16, V>(row.d[j][h], d[j][h]);
#pragma unroll
        for (int e = 0; e < V; ++e) sum = fmaf(x[j][h][e], x[j][h][e], sum);
      }
    float r = 1.0f;
    if (a.norm) {
      for (int o = 1; o < G; o <<= 1) sum += __shfl_xor(sum, o);
      r = 1.0f / sqrtf(fmaf(sum, a.inv_m, a.eps));
    }
    // rotates the values of the unit (forward) or turns them back (gradient)
    auto rotate = [&](float (&v)[U][2][V]) {
      if constexpr (PAIRS == kAnywhere) {
        // a row's lanes are of one wave, whose LDS accesses stay in order
        static_assert(U == 1);
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c = h == 0 ? c0[0] : c1[0];
          if (c < chunks) {
#pragma unroll
            for (int e = 0; e < V; e += 4) *reinterpret_cast<float4*>(s_row + c * V + e) = float4{v[0][h][e], v[0][h][e + 1], v[0][h][e + 2], v[0][h][e + 3]};
          }
        }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const int f = (h == 0 ? c0[0] : c1[0]) * V + e;
            if (f < 2 * RP) {
              const bool second = f >= RP;
              const int p = second ? f - RP : f;
              const float2 cs = s_cs[t * RP + p];
              const float sn = second != GRAD ? cs.y : -cs.y, other = s_row[second ? p : f + RP];
              v[0][h][e] = v[0][h][e] * cs.x + other * sn;
            }
          }
        return;
      }
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int u = lane + j * G;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const int p = u * V + e;
          if (p < RP) {
            float2 cs = s_cs[t * RP + p];
            if constexpr (GRAD) cs.y = -cs.y;
            float& f0 = v[j][INSIDE ? (2 * e) / V : 0][INSIDE ? (2 * e) % V : e];
            float& f1 = v[j][INSIDE ? (2 * e + 1) / V : 1][INSIDE ? (2 * e + 1) % V : e];
            const float v0 = f0, v1 = f1;
            f0 = v0 * cs.x - v1 * cs.y;
            f1 = v1 * cs.x + v0 * cs.y;
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
          for (int e = 0; e < V; ++e) x[j][h][e] *= r * w[j][h][e];
      rotate(x);
    } else {
      rotate(d);
      float dot = 0.0f;
#pragma unroll
      for (int j = 0; j < U; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float n = x[j][h][e] * r;
            if (live) dw[m][j][h][e] += d[j][h][e] * n;
            d[j][h][e] *= w[j][h][e];
            dot = fmaf(d[j][h][e], n, dot);
            x[j][h][e] = n;
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
          for (int e = 0; e < V; ++e) x[j][h][e] = r * (d[j][h][e] - x[j][h][e] * dot);
    }
    if (live) {
      void* dst = m == 0 ? a.q_out : a.k_out;
      const int64_t out = ((t0 + t) * (m == 0 ? a.Hq : a.Hk) + hh) * a.D;
#pragma unroll
      for (int j = 0; j < U; ++j) {
        if (c0[j] < chunks) store_chunk<BF16, V>(dst, out + c0[j] * V, x[j][0]);
        if (c1[j] < chunks) store_chunk<BF16, V>(dst, out + c1[j] * V, x[j][1]);
      }
    }
  };
  auto weights = [&](const float* p, float (&w)[U][2][V]) {
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int c = h == 0 ? c0[j] : c1[j];
          w[j][h][i] = p != nullptr && c < chunks ? p[c * V + i] : 1.0f;
        }
  };

  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * tile; t0 < a.T; t0 += static_cast<int64_t>(gridDim.x) * tile) {
    const int nt = static_cast<int>(a.T - t0 < tile ? a.T - t0 : tile);
    const int rq = nt * a.Hq, rk = nt * a.Hk;
    // every slot has a row in every pass (the last one again where there is none
    // left), so that the next row's loads need no condition; the first are on
    // their way while the angles are computed
    Row row;
    load(0, t0, min(slot, rq - 1), row);
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
    float w[U][2][V];
    weights(a.wq, w);
    for (int r0 = 0; r0 < rq; r0 += slots) {
      Row next;
      const int i = r0 + slot;
      if (r0 + slots < rq) load(0, t0, min(i + slots, rq - 1), next);
      else load(1, t0, min(slot, rk - 1), next);
      compute(std::integral_constant<int, 0>{}, t0, min(i, rq - 1), i < rq, row, w);
      row = next;
    }
    weights(a.wk, w);
    for (int r0 = 0; r0 < rk; r0 += slots) {
      Row next;
      const int i = r0 + slot;
      if (r0 + slots < rk) load(1, t0, min(i + slots, rk - 1), next);
      compute(std::integral_constant<int, 1>{}, t0, min(i, rk - 1), i < rk, row, w);
      row = next;
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

// whether whole 16-byte chunks of V features can be moved
bool vectored(const QkArgs& a, bool backward, int V) {
  return a.D % V == 0 && a.ldq % V == 0 && a.ldk % V == 0 && aligned(a.q) && aligned(a.k) && aligned(a.q_out) && aligned(a.k_out) &&
         (!backward || (aligned(a.dq_out) && aligned(a.dk_out)));
}

int lanes_of(const QkArgs& a, int V) {
  const int units = (a.D / V + 1) / 2;
  int G = 1;
  while (G < units && G < 64) G <<= 1;
  return G;
}

// tokens of a tile: as many as share a workgroup's angles, fewer while that would
// leave a compute unit with less than two workgroups. (40 heads of 128 over 16384
// tokens: tiles of 4, 8, 16 and 32 tokens take 79, 74, 71 and 97 us, the gradients
// of 32 heads over 8192 tokens 51, 46, 42 and 42.)
int tile_of(const QkArgs& a) {
  int tile = kMaxTile;
  while (tile > 1 && a.T / tile < 512) tile >>= 1;
  return tile;
}

template <bool BF16, int V, bool GRAD, Pairs PAIRS>
hipError_t run(const QkArgs& a, hipStream_t stream) {
  const int G = lanes_of(a, V), tile = tile_of(a);
  int64_t blocks = (a.T + tile - 1) / tile;
  blocks = std::min<int64_t>(blocks, GRAD ? kBackwardBlocks : 1 << 20);
  size_t lds = static_cast<size_t>(tile) * (a.R / 2) * sizeof(float2);
  if (PAIRS == kAnywhere) lds = (lds + 15) / 16 * 16 + static_cast<size_t>(kThreads / G) * a.D * sizeof(float);
  if (GRAD) lds = std::max(lds, static_cast<size_t>(kThreads / G) * 2 * a.D * sizeof(float));
  k_qk<BF16, V, GRAD, PAIRS><<<dim3(static_cast<unsigned>(blocks)), dim3(kThreads), lds, stream>>>(a, G, tile);
  hipError_t e = hipGetLastError();
  if (GRAD && e == hipSuccess && a.partials != nullptr) {
    k_qk_weights<<<dim3(2 * a.D), dim3(kThreads), 0, stream>>>(a.partials, static_cast<int>(blocks), a.D, a.dwq, a.dwk);
    e = hipGetLastError();
  }
  return e;
}

template <bool BF16, int V, bool GRAD>
hipError_t dispatch(const QkArgs& a, hipStream_t stream) {
  if (!vectored(a, GRAD, V)) return run<BF16, 1, GRAD, kAcross>(a, stream);
  if (a.interleaved) return run<BF16, V, GRAD, kInside>(a, stream);
  return (a.R / 2) % V == 0 ? run<BF16, V, GRAD, kAcross>(a, stream) : run<BF16, V, GRAD, kAnywhere>(a, stream);
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
