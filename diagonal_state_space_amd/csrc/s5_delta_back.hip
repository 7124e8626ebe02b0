// Backward pass of the chunked gated delta rule.
//
// Per chunk, with D' the gradient of its end state and the names of the
// forward kernels (from = e^G, to = e^{G_end - G}, M_ij = e^{G_i - G_j}):
//   dU = scale P^T dY + to K D',  dR = T^T dU,  dV = beta dR
//   D  = whole D' + scale (from Q)^T dY - (from K)^T dV       (start state)
// is a chain like the forward one, run from the last chunk to the first in
// columns of the state (k_delta_back_scan), after the forward chain has run
// again and left the states S at the chunks' starts and U. The rest has no
// chain (k_delta_grad, one workgroup per chunk and key head, over its value
// heads):
//   dQ    = scale (from dY S^T + (M o dY U^T) K)
//   Hrow  = -(from dR S^T + (M< o dR U^T) K),          dKrow = beta Hrow
//   dKcol = scale (M o dY U^T)^T Q + to U D'^T - (M< o beta dR U^T)^T K
//   dbeta = dR.V + k.Hrow
//   dG    = q.dQ + k.dKrow - k.dKcol,  + <D', S'> at the last token, S' the
//           end state: whole <D', S> + sum to k.(U D'^T);  dg = sums of dG from the end
// (M< is M without its diagonal; . are dot products of a token's rows.) Every
// term of dG is a row of a product that is there anyway.
#include "s5_delta_tile.h"

namespace s5 {

using namespace delta;

namespace {

// LDS of a chunk: fragments of k (by rows, by columns) and q (by columns) and
// the decays, two of them where they fit (one more wave copies them); the transposed T and P, which the
// next chunk's replace as soon as they are read.
template <bool BF16, int KP>
struct Back : Shape<BF16, KP> {
  using Z = Shape<BF16, KP>;
  static constexpr int kTri = tri_frags<Z::C>() * 3 * kFrag;
  static constexpr int kBuf = 3 * Z::kMat + kFrag;
  static constexpr bool kTwo = 2 * kBuf + 2 * kTri <= kMaxLds;
  static constexpr int oTri = (kTwo ? 2 : 1) * kBuf;
  static constexpr int kLds = oTri + 2 * kTri;
};

template <bool BF16, int KP, int NW>
__global__ void __launch_bounds__(64 * (NW + 1)) k_delta_back_scan(DeltaArgs a, int chunks, int groups, DeltaKeep keep) {
  using Z = Back<BF16, KP>;
  constexpr int C = Z::C, NI = Z::NI, KS = Z::KS, MT = Z::MT, CS = Z::CS, KT = Z::KT, es = Z::es;
  extern __shared__ __align__(16) unsigned char smem[];
  const int tid = threadIdx.x, l = tid & 63, g = l >> 4, m = l & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int die = blockIdx.x & 7, turn = blockIdx.x >> 3;
  const int bh = (turn / groups) * 8 + die, cg = turn % groups;
  if (bh >= a.B * a.Hv) return;
  const int b = bh / a.Hv, h = bh - b * a.Hv, hk = h / (a.Hv / a.Hk);
  const int col = (cg * NW + w) * 16 + m;
  const bool wave_live = (cg * NW + w) * 16 < a.Dv, live = col < a.Dv;
  const int len = length_of(a, b);
  const int nc = (len + C - 1) / C;

  if (w == NW) {   // the copying wave
    auto record = [&](int n) { return a.recs + (static_cast<int64_t>(bh) * chunks + n) * Record<C>::bytes(true, 3); };
    auto copy_tri = [&](int n) { lds_copy<1>(smem + Z::oTri, record(n) + Record<C>::P, 2 * Z::kTri, 0); };
    auto copy = [&](int n) {
      unsigned char* dst = smem + (Z::kTwo ? (n & 1) * Z::kBuf : 0);
      lds_copy<1>(dst, a.frags + (static_cast<int64_t>(b * a.Hk + hk) * chunks + n) * Z::frags(true), 3 * Z::kMat, 0);
      lds_copy<1>(dst + 3 * Z::kMat, record(n) + Record<C>::decays(true, 3), kFrag, 0);
    };
    if (nc > 0) {
      if (Z::kTwo) copy(nc - 1);
      copy_tri(nc - 1);
    }
    for (int n = nc - 1; n >= 0; --n) {
      if constexpr (!Z::kTwo) {
        barrier_copied();
        copy(n);
      }
      barrier_copied();
      if (Z::kTwo && n > 0) copy(n - 1);
      barrier_copied();
      if (n > 0) copy_tri(n - 1);
    }
    return;
  }

  f32x4 D[KT];
#pragma unroll
  for (int t = 0; t < KT; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * t + 4 * g + r;
      D[t][r] = a.ds_last != nullptr && live && row < a.Dk ? a.ds_last[(static_cast<int64_t>(bh) * a.Dk + row) * a.Dv + col] : 0.0f;
    }

  uint32_t ob[MT][4];
  const int ldy = a.Hv * a.Dv * es;
  const int yo = live ? 4 * g * ldy + col * es : kNowhere;
  const int ko = (4 * g * keep.dvp + col) * 4;   // rows behind the kept ones are outside their buffer
  const unsigned char* s_tt = smem + Z::oTri;
  const unsigned char* s_pt = s_tt + Z::kTri;
  auto fetch = [&](int n) {
    const int64_t tok = static_cast<int64_t>(b) * a.L + n * C;
    const Buf yr = rows_buf(static_cast<const char*>(a.dy) + (tok * a.Hv + h) * a.Dv * es, min(len - n * C, C), ldy, a.Dv * es);
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) ob[t][r] = load_raw<BF16>(yr, yo + (16 * t + r) * ldy);
  };

  if (nc > 0) fetch(nc - 1);
  for (int n = nc - 1; n >= 0; --n) {
    if constexpr (!Z::kTwo) barrier_read();   // the previous chunk is read
    barrier_read();                           // the chunk is there, the previous one read
    f32x4 dO[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) dO[t][r] = value<BF16>(ob[t][r]);
    if (n > 0) fetch(n - 1);

    const unsigned char* s_k = smem + (Z::kTwo ? (n & 1) * Z::kBuf : 0);
    const unsigned char *s_kt = s_k + Z::kMat, *s_qt = s_k + 2 * Z::kMat;
    const float* dec = reinterpret_cast<const float*>(s_k + 3 * Z::kMat);
    f32x4 dU[MT], P[MT], dR[MT];
    if (wave_live) {
      const Buf kd = rows_buf(keep.d + (static_cast<int64_t>(bh) * chunks + n) * keep.dkp * keep.dvp, keep.dkp, keep.dvp * 4, keep.dvp * 4);
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) store_el<false>(kd, ko + (16 * t + r) * keep.dvp * 4, D[t][r]);
#pragma unroll
      for (int t = 0; t < MT; ++t) dU[t] = P[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        Frag<NI> kf[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t) kf[t] = read_rows<NI, KS>(s_k, t, ks);
        mma(dU, kf, to_frag<3>(D[2 * ks], D[2 * ks + 1]));
      }
      tri_mma_t<C, 3, NI>(P, s_pt, dO);
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const float4 to = *reinterpret_cast<const float4*>(dec + C + 16 * t + 4 * g);
        const float tt[4] = {to.x, to.y, to.z, to.w};
#pragma unroll
        for (int r = 0; r < 4; ++r) dU[t][r] = fmaf(tt[r], dU[t][r], a.scale * P[t][r]);
      }
#pragma unroll
      for (int t = 0; t < MT; ++t) dR[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      tri_mma_t<C, 3, 3>(dR, s_tt, dU);
    }
    barrier_read();   // T and P are read
    if (!wave_live) continue;

    const int64_t tok = static_cast<int64_t>(b) * a.L + n * C;
    const Buf kr = rows_buf(keep.r + (static_cast<int64_t>(bh) * chunks + n) * C * keep.dvp, C, keep.dvp * 4, keep.dvp * 4);
    const Buf vr = rows_buf(static_cast<char*>(a.dv) + (tok * a.Hv + h) * a.Dv * es, min(len - n * C, C), ldy, a.Dv * es);
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const float4 f = *reinterpret_cast<const float4*>(dec + 16 * t + 4 * g);
      const float4 be = *reinterpret_cast<const float4*>(dec + 2 * C + 16 * t + 4 * g);
      const float ff[4] = {f.x, f.y, f.z, f.w}, bb[4] = {be.x, be.y, be.z, be.w};
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        store_el<false>(kr, ko + (16 * t + r) * keep.dvp * 4, dR[t][r]);
        dR[t][r] *= bb[r];
        store_el<BF16>(vr, yo + (16 * t + r) * ldy, dR[t][r]);
        dR[t][r] *= -ff[r];
        dO[t][r] *= a.scale * ff[r];
      }
    }
    const float whole = dec[3 * C];
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) D[t][r] *= whole;
#pragma unroll
    for (int ks = 0; ks < CS; ++ks) {
      cols_mma<NI, C>(D, s_kt, ks, to_frag<3>(dR[2 * ks], dR[2 * ks + 1]));
      cols_mma<NI, C>(D, s_qt, ks, to_frag<3>(dO[2 * ks], dO[2 * ks + 1]));
    }
  }

  if (a.ds0 != nullptr && live) {
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * t + 4 * g + r;
        if (row < a.Dk) a.ds0[(static_cast<int64_t>(bh) * a.Dk + row) * a.Dv + col] = D[t][r];
      }
  }
}

// ---- the gradients without a chain ------------------------------------------------
// Products on the float32 matrix instructions: wave w has the feature tiles
// w, w + 4 of all tokens. An operand block of 16 rows by 16 products is one
// float4 a lane (row m, products 4g..4g+3), four instructions.

__device__ __forceinline__ f32x4 mma16(float4 x, float4 y, f32x4 c) {
  c = __builtin_amdgcn_mfma_f32_16x16x4f32(x.x, y.x, c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_16x16x4f32(x.y, y.y, c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_16x16x4f32(x.z, y.z, c, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_16x16x4f32(x.w, y.w, c, 0, 0, 0);
}

template <bool BF16, int KP>
struct Grad {
  static constexpr int C = chunk_of<BF16>(), MT = C / 16, DT = KP / 64;
  static constexpr int LD = C + 4, LK = KP + (BF16 ? 8 : 4);
  static constexpr int es = BF16 ? 2 : 4;
  static constexpr int oQ = C * LK * es, oW1 = 2 * oQ, oW2 = oW1 + C * LD * 4;
  static constexpr int oG = oW2 + C * LD * 4;               // double sums of g
  static constexpr int oB = oG + C * 8;                     // beta, from, to
  static constexpr int oRed = oB + 3 * C * 4;               // [4 waves][3][C] row sums
  static constexpr int oSum = oRed + 12 * C * 4;            // [4 waves] sums
  static constexpr int oRV = oSum + 32;                     // [C] dR.V
  static constexpr int kLds = oRV + C * 4;
};

template <bool BF16, int KP>
__global__ void __launch_bounds__(256) k_delta_grad(DeltaArgs a, int chunks, DeltaKeep keep, bool vec_y) {
  using Z = Grad<BF16, KP>;
  constexpr int C = Z::C, MT = Z::MT, DT = Z::DT, LD = Z::LD, LK = Z::LK;
  extern __shared__ __align__(16) unsigned char smem[];
  unsigned char *s_k = smem, *s_q = smem + Z::oQ;
  float *s_w1 = reinterpret_cast<float*>(smem + Z::oW1), *s_w2 = reinterpret_cast<float*>(smem + Z::oW2);
  double* s_g = reinterpret_cast<double*>(smem + Z::oG);
  float *s_b = reinterpret_cast<float*>(smem + Z::oB), *s_from = s_b + C, *s_to = s_from + C;
  float *s_red = reinterpret_cast<float*>(smem + Z::oRed), *s_sum = reinterpret_cast<float*>(smem + Z::oSum);
  float* s_rv = reinterpret_cast<float*>(smem + Z::oRV);
  const int tid = threadIdx.x, l = tid & 63, g = l >> 4, m = l & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = blockIdx.x % chunks, bk = blockIdx.x / chunks;
  const int b = bk / a.Hk, hk = bk - b * a.Hk;
  const int left = length_of(a, b) - n * C;
  if (left <= 0) return;
  const int64_t tok = static_cast<int64_t>(b) * a.L + n * C;
  const int group = a.Hv / a.Hk;

  for (int i = tid; i < C * KP; i += 256) {
    const int t = i / KP, d = i % KP;
    const bool ok = t < left && d < a.Dk;
    const int64_t ki = (tok + t) * a.ldk + static_cast<int64_t>(hk) * a.Dk + d;
    const int64_t qi = (tok + t) * a.ldq + static_cast<int64_t>(hk) * a.Dk + d;
    if constexpr (BF16) {
      reinterpret_cast<uint16_t*>(s_k)[t * LK + d] = ok ? static_cast<const uint16_t*>(a.k)[ki] : uint16_t{0};
      reinterpret_cast<uint16_t*>(s_q)[t * LK + d] = ok ? static_cast<const uint16_t*>(a.q)[qi] : uint16_t{0};
    } else {
      reinterpret_cast<float*>(s_k)[t * LK + d] = ok ? static_cast<const float*>(a.k)[ki] : 0.0f;
      reinterpret_cast<float*>(s_q)[t * LK + d] = ok ? static_cast<const float*>(a.q)[qi] : 0.0f;
    }
  }

  f32x4 dQ[DT][MT], dK[DT][MT];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int t = 0; t < MT; ++t) dQ[d][t] = dK[d][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  for (int hh = 0; hh < group; ++hh) {
    const int h = hk * group + hh;
    const int64_t bh = static_cast<int64_t>(b) * a.Hv + h;
    __syncthreads();   // the previous head's sums are read
    float gi = 0.0f;
    if (w == 0) {
      const bool live = l < C && l < left;
      gi = live ? a.g[(tok + l) * a.Hv + h] : 0.0f;
      const double s = chunk_sums(gi);
      const double end = __shfl(s, C - 1);
      if (l < C) {
        s_g[l] = s;
        s_b[l] = live ? a.beta[(tok + l) * a.Hv + h] : 0.0f;
        s_from[l] = expf(static_cast<float>(s));
        s_to[l] = expf(static_cast<float>(end - s));
      }
    }

    // contraction over the value features
    const float* ks = keep.s + (bh * chunks + n) * keep.dkp * keep.dvp;
    const float* kd = keep.d + (bh * chunks + n) * keep.dkp * keep.dvp;
    const float* ku = keep.u + (bh * chunks + n) * C * keep.dvp;
    const float* kr = keep.r + (bh * chunks + n) * C * keep.dvp;
    f32x4 E[DT][MT], F[DT][MT], H[DT][MT], W1[MT], W2[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      W1[t] = W2[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int d = 0; d < DT; ++d) E[d][t] = F[d][t] = H[d][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    float sd = 0.0f;   // <D', S>
    const int64_t ldy = static_cast<int64_t>(a.Hv) * a.Dv;
    // rows of W1 and W2 of this wave: tiles w and MT - 1 - w (C = 32: the first two waves)
    const int r1 = w < MT ? w : 0, r2 = w < MT ? MT - 1 - w : 0;
    for (int v0 = 0; v0 < keep.dvp; v0 += 16) {
      const int v = v0 + 4 * g;
      auto load_dy = [&](int t) {
        const int i = 16 * t + m;
        float4 x = {0.0f, 0.0f, 0.0f, 0.0f};
        if (i < left) {
          const int64_t o = (tok + i) * ldy + static_cast<int64_t>(h) * a.Dv + v;
          if (vec_y && v + 4 <= a.Dv) {
            if constexpr (BF16) {
              const uint2 p = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.dy) + o);
              x = float4{__uint_as_float(p.x << 16), __uint_as_float(p.x & 0xffff0000u), __uint_as_float(p.y << 16),
                         __uint_as_float(p.y & 0xffff0000u)};
            } else {
              x = *reinterpret_cast<const float4*>(static_cast<const float*>(a.dy) + o);
            }
          } else {
            if (v < a.Dv) x.x = load_el<BF16>(a.dy, o);
            if (v + 1 < a.Dv) x.y = load_el<BF16>(a.dy, o + 1);
            if (v + 2 < a.Dv) x.z = load_el<BF16>(a.dy, o + 2);
            if (v + 3 < a.Dv) x.w = load_el<BF16>(a.dy, o + 3);
          }
        }
        return x;
      };
      auto load_row = [&](const float* p, int row) { return *reinterpret_cast<const float4*>(p + static_cast<int64_t>(row) * keep.dvp + v); };
      float4 y[MT], u[MT], r[MT];
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        y[t] = load_dy(t);
        u[t] = load_row(ku, 16 * t + m);
        r[t] = load_row(kr, 16 * t + m);
      }
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        const int row = 16 * (w + 4 * d);
        if (row < a.Dk) {
          const float4 s = load_row(ks, row + m), e = load_row(kd, row + m);
          sd += s.x * e.x + s.y * e.y + s.z * e.z + s.w * e.w;
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            E[d][t] = mma16(y[t], s, E[d][t]);
            F[d][t] = mma16(r[t], s, F[d][t]);
            H[d][t] = mma16(u[t], e, H[d][t]);
          }
        }
      }
      if (w < MT) {
        const float4 y1 = load_dy(r1), x2 = load_row(kr, 16 * r2 + m);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          if (t <= r1) W1[t] = mma16(y1, u[t], W1[t]);
          if (t <= r2) W2[t] = mma16(x2, u[t], W2[t]);
        }
      }
    }
    __syncthreads();   // s_g and the decays are there
    if (w < MT) {
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int j = 16 * t + m, i1 = 16 * r1 + 4 * g + r, i2 = 16 * r2 + 4 * g + r;
          if (t <= r1) s_w1[i1 * LD + j] = j <= i1 ? W1[t][r] * expf(static_cast<float>(s_g[i1] - s_g[j])) : 0.0f;
          if (t <= r2) s_w2[i2 * LD + j] = j < i2 ? W2[t][r] * expf(static_cast<float>(s_g[i2] - s_g[j])) : 0.0f;
        }
    }
    // dR.V of the tokens of this wave
    for (int i = w; i < C; i += 4) {
      float s = 0.0f;
      if (i < left)
        for (int v = l; v < a.Dv; v += 64)
          s = fmaf(kr[static_cast<int64_t>(i) * keep.dvp + v], load_el<BF16>(a.v, (tok + i) * a.ldv + static_cast<int64_t>(h) * a.Dv + v), s);
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) s += __shfl_xor(s, o);
      if (l == 0) s_rv[i] = s;
    }
    __syncthreads();

    float qa[MT][4], ka[MT][4], kc[MT][4];   // rows of q.dQ, k.Hrow, k.dKcol
    float kh = 0.0f;                         // sum of to k.(U D'^T)
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) qa[t][r] = ka[t][r] = kc[t][r] = 0.0f;
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      const int c = 16 * (w + 4 * d) + m;    // feature
      float4 kv[MT], qv[MT], kb[MT];         // k, q and beta k in accumulator order, the second operand's too
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        float x[4], y[4], z[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int i = 16 * t + 4 * g + r;
          x[r] = load_el<BF16>(s_k, i * LK + c);
          y[r] = load_el<BF16>(s_q, i * LK + c);
          z[r] = s_b[i] * x[r];
        }
        kv[t] = float4{x[0], x[1], x[2], x[3]};
        qv[t] = float4{y[0], y[1], y[2], y[3]};
        kb[t] = float4{z[0], z[1], z[2], z[3]};
      }
      auto rows = [&](const float* p, int it, int jt) { return *reinterpret_cast<const float4*>(p + (16 * it + m) * LD + 16 * jt + 4 * g); };
      auto cols = [&](const float* p, int it, int jt) {   // rows jt of the transposed
        const float* x = p + (16 * it + 4 * g) * LD + 16 * jt + m;
        return float4{x[0], x[LD], x[2 * LD], x[3 * LD]};
      };
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        f32x4 q1 = {0.0f, 0.0f, 0.0f, 0.0f}, k1 = q1, c1 = q1, c2 = q1;
#pragma unroll
        for (int s = 0; s < MT; ++s) {
          if (s <= t) {
            q1 = mma16(rows(s_w1, t, s), kv[s], q1);
            k1 = mma16(rows(s_w2, t, s), kv[s], k1);
          }
          if (s >= t) {
            c1 = mma16(cols(s_w1, s, t), qv[s], c1);
            c2 = mma16(cols(s_w2, s, t), kb[s], c2);
          }
        }
        const float ke[4] = {kv[t].x, kv[t].y, kv[t].z, kv[t].w}, qe[4] = {qv[t].x, qv[t].y, qv[t].z, qv[t].w};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int i = 16 * t + 4 * g + r;
          const float from = s_from[i], to = s_to[i];
          const float dq = a.scale * fmaf(from, E[d][t][r], q1[r]);
          const float hr = -fmaf(from, F[d][t][r], k1[r]);
          const float uh = to * H[d][t][r];
          const float dc = fmaf(a.scale, c1[r], uh) - c2[r];
          qa[t][r] = fmaf(qe[r], dq, qa[t][r]);
          ka[t][r] = fmaf(ke[r], hr, ka[t][r]);
          kc[t][r] = fmaf(ke[r], dc, kc[t][r]);
          kh = fmaf(ke[r], uh, kh);
          dQ[d][t][r] += dq;
          dK[d][t][r] += fmaf(s_b[i], hr, dc);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) {
          qa[t][r] += __shfl_xor(qa[t][r], o);
          ka[t][r] += __shfl_xor(ka[t][r], o);
          kc[t][r] += __shfl_xor(kc[t][r], o);
        }
        if (m == 0) {
          const int i = 16 * t + 4 * g + r;
          s_red[(w * 3 + 0) * C + i] = qa[t][r];
          s_red[(w * 3 + 1) * C + i] = ka[t][r];
          s_red[(w * 3 + 2) * C + i] = kc[t][r];
        }
      }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      sd += __shfl_xor(sd, o);
      kh += __shfl_xor(kh, o);
    }
    if (l == 0) {
      s_sum[w] = sd;
      s_sum[4 + w] = kh;
    }
    __syncthreads();
    if (w == 0) {
      float q1 = 0.0f, k1 = 0.0f, c1 = 0.0f, s1 = 0.0f, h1 = 0.0f;
      const int i = l < C ? l : 0;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        q1 += s_red[(x * 3 + 0) * C + i];
        k1 += s_red[(x * 3 + 1) * C + i];
        c1 += s_red[(x * 3 + 2) * C + i];
        s1 += s_sum[x];
        h1 += s_sum[4 + x];
      }
      const float whole = expf(static_cast<float>(s_g[C - 1]));
      double dg = l < C ? static_cast<double>(q1) + s_b[i] * k1 - c1 : 0.0;
      if (l == C - 1) dg += static_cast<double>(whole) * s1 + h1;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const double down = __shfl_down(dg, o);
        if (l + o < 64) dg += down;
      }
      if (l < C && l < left) {
        // a decay that clears the state hides what it multiplied
        a.dg[(tok + l) * a.Hv + h] = gi < kLeastDecay ? 0.0f : static_cast<float>(dg);
        a.dbeta[(tok + l) * a.Hv + h] = s_rv[l] + k1;
      }
    }
  }

#pragma unroll
  for (int d = 0; d < DT; ++d) {
    const int c = 16 * (w + 4 * d) + m;
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = 16 * t + 4 * g + r;
        if (i < left && c < a.Dk) {
          const int64_t o = ((tok + i) * a.Hk + hk) * a.Dk + c;
          store_el<BF16>(a.dq, o, dQ[d][t][r]);
          store_el<BF16>(a.dk, o, dK[d][t][r]);
        }
      }
  }
}

// finds the workspace's parts; bytes of all of them
int64_t keep_of(DeltaArgs& a, DeltaKeep& k) {
  const int C = a.bf16_io ? 64 : 32;
  const int64_t chunks = static_cast<int64_t>(a.B) * a.Hv * ((a.L + C - 1) / C);
  k.dkp = (a.Dk + 15) & ~15;
  k.dvp = (a.Dv + 15) & ~15;
  const int64_t head = delta_work(a, true), state = chunks * k.dkp * k.dvp * 4, rows = chunks * C * k.dvp * 4;
  unsigned char* p = static_cast<unsigned char*>(a.ws);
  k.s = reinterpret_cast<float*>(p + head);
  k.d = reinterpret_cast<float*>(p + head + state);
  k.u = reinterpret_cast<float*>(p + head + 2 * state);
  k.r = reinterpret_cast<float*>(p + head + 2 * state + rows);
  return head + 2 * state + 2 * rows;
}

template <bool BF16, int KP>
hipError_t run(DeltaArgs a, hipStream_t stream) {
  constexpr int NW = 4, C = chunk_of<BF16>();
  using Z = Back<BF16, KP>;
  using G = Grad<BF16, KP>;
  auto* scan = k_delta_back_scan<BF16, KP, NW>;
  auto* grad = k_delta_grad<BF16, KP>;
  static const hipError_t attr[2] = {
      hipFuncSetAttribute(reinterpret_cast<const void*>(scan), hipFuncAttributeMaxDynamicSharedMemorySize, Z::kLds),
      hipFuncSetAttribute(reinterpret_cast<const void*>(grad), hipFuncAttributeMaxDynamicSharedMemorySize, G::kLds)};
  for (hipError_t e : attr)
    if (e != hipSuccess) return e;
  const int chunks = (a.L + C - 1) / C;
  const int groups = (a.Dv + 16 * NW - 1) / (16 * NW);
  DeltaKeep keep{};
  keep_of(a, keep);
  if (a.L > 0) {
    hipError_t e = launch_delta_prep(a, true, stream);
    if (e == hipSuccess) e = launch_delta_scan(a, &keep, stream);
    if (e != hipSuccess) return e;
  }
  const int64_t blocks = (static_cast<int64_t>(a.B) * a.Hv + 7) / 8 * 8 * groups;
  scan<<<dim3(static_cast<unsigned>(blocks)), dim3(64 * (NW + 1)), Z::kLds, stream>>>(a, chunks, groups, keep);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.L == 0) return e;
  const bool vec_y = a.Dv % 4 == 0;   // dy is contiguous and 16-byte aligned
  grad<<<dim3(static_cast<unsigned>(static_cast<int64_t>(a.B) * a.Hk * chunks)), dim3(256), G::kLds, stream>>>(a, chunks, keep, vec_y);
  return hipGetLastError();
}

}  // namespace

int64_t delta_workspace(const DeltaArgs& args, bool backward) {
  DeltaArgs a = args;
  DeltaKeep k{};
  return backward ? keep_of(a, k) : delta_work(a, false);
}

hipError_t launch_delta_backward(const DeltaArgs& a, hipStream_t stream) {
  if (a.bf16_io) return a.Dk > 64 ? run<true, 128>(a, stream) : run<true, 64>(a, stream);
  return a.Dk > 64 ? run<false, 128>(a, stream) : run<false, 64>(a, stream);
}

}  // namespace s5
