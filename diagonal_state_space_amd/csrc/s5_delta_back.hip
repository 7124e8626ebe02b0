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
//
// What bounds them (128 x 128 bf16, 64 value heads of 2048 steps): the chain as the
// forward one, 158 us; the rest, 181 us, by its phases between barriers, one
// workgroup on a compute unit (of 47000 cycles for a head's chunk 6000 staging,
// 20500 products over the value features, of which matrix instructions 12400,
// 6500 finishing W1 and W2, 4200 the products over tokens, 5000 rows and results),
// next to the 540 MB of states, writes and their gradients that it reads.
#include <algorithm>

#include "s5_delta_tile.h"

namespace s5 {

using namespace delta;

namespace {

// LDS of a chunk: fragments of k (by rows, by columns) and q (by columns), the
// decays and (bf16) y's gradient, two of them where they fit; the transposed T
// and P, which the next chunk's replace as soon as they are read.
template <bool BF16, int KP, int NW>
struct Back : Shape<BF16, KP> {
  using Z = Shape<BF16, KP>;
  static constexpr int kTri = tri_frags<Z::C>() * 3 * kFrag;
  static constexpr int oV = 3 * Z::kMat + kFrag, kBuf = oV + (BF16 ? ValueStage<NW>::kBytes : 0);
  static constexpr bool kTwo = 2 * kBuf + 2 * kTri <= kMaxLds;
  static constexpr int oTri = (kTwo ? 2 : 1) * kBuf;
  static constexpr int kLds = oTri + 2 * kTri;
};

// SUM: only the gradients at the segments' starts, from zero ends (the last
// segment's from ds_last)
template <bool BF16, int KP, int NW, bool SUM>
__global__ void __launch_bounds__(64 * (NW + kCopy)) k_delta_back_scan(DeltaArgs a, int chunks, int groups, DeltaSegs segs, DeltaKeep keep) {
  using Z = Back<BF16, KP, NW>;
  constexpr int C = Z::C, NI = Z::NI, KS = Z::KS, MT = Z::MT, CS = Z::CS, KT = Z::KT, es = Z::es;
  extern __shared__ __align__(16) unsigned char smem[];
  const int tid = threadIdx.x, l = tid & 63, g = l >> 4, m = l & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int count = SUM ? segs.count - 1 : segs.count;   // sums: segments 1, 2, ...
  const int turn = blockIdx.x >> 3, cg = turn % groups, unit = turn / groups * 8 + (blockIdx.x & 7);
  const int bh = unit / count, seg = unit - bh * count + (SUM ? 1 : 0);
  if (bh >= a.B * a.Hv) return;
  const int b = bh / a.Hv, h = bh - b * a.Hv, hk = h / (a.Hv / a.Hk);
  const int wg = cg * NW + w, col = wg * 16 + m;
  const bool wave_live = wg * 16 < a.Dv, live = col < a.Dv;
  const int len = length_of(a, b);
  const int nc = (len + C - 1) / C;
  const int n0 = seg * segs.chunks, n1 = min(nc, n0 + segs.chunks);
  if (seg > 0 && n0 >= nc) return;
  const bool last = n0 + segs.chunks >= nc;

  if (w >= NW) {   // the copying waves
    const int id = tid - 64 * NW;
    const bool vec = vectored(a, BF16), vecy = a.Dv % 8 == 0;
    Stage<BF16, KP, 64 * kCopy> k, q;
    ValueStage<NW> y;
    auto record = [&](int n) { return a.recs + (static_cast<int64_t>(bh) * chunks + n) * Record<C>::bytes(true); };
    auto load = [&](int n) {
      const int64_t tok = static_cast<int64_t>(b) * a.L + n * C;
      if constexpr (BF16) {
        y.load(static_cast<const char*>(a.dy) + ((tok * a.Nv + h) * a.Dv + cg * 16 * NW) * es, a.Nv * a.Dv * es, min(len - n * C, C),
               a.Dv - cg * 16 * NW, id, vecy);
        k.load(a, a.k, a.ldk, tok, min(len - n * C, C), hk, id, vec);
        q.load(a, a.q, a.ldq, tok, min(len - n * C, C), hk, id, vec);
      }
    };
    auto copy_tri = [&](int n) { lds_copy<kCopy>(smem + Z::oTri, record(n) + Record<C>::P, 2 * Z::kTri, w - NW); };
    auto copy = [&](int n) {
      unsigned char* dst = smem + (Z::kTwo ? (n & 1) * Z::kBuf : 0);
      if constexpr (BF16) {
        y.store(dst + Z::oV, id);
        k.store(dst, dst + Z::kMat, id);
        q.store(nullptr, dst + 2 * Z::kMat, id);
      } else {
        const unsigned char* fr = a.frags + (static_cast<int64_t>(b * a.Hk + hk) * chunks + n) * Z::frags(true);
        lds_copy<kCopy>(dst, fr + Z::k_rows(true), Z::kMat, w - NW);
        lds_copy<kCopy>(dst + Z::kMat, fr, 2 * Z::kMat, w - NW);
      }
      lds_copy<kCopy>(dst + 3 * Z::kMat, record(n) + Record<C>::decays(true), kFrag, w - NW);
    };
    if (n0 < n1) {
      load(n1 - 1);
      if (Z::kTwo) {
        copy(n1 - 1);
        if (n1 - 1 > n0) load(n1 - 2);
      }
      copy_tri(n1 - 1);
    }
    for (int n = n1 - 1; n >= n0; --n) {
      if constexpr (Z::kTwo) {
        barrier_copied();
        if (n > n0) copy(n - 1);
        if (n - 1 > n0) load(n - 2);
        barrier_passed();   // T and P are read; the copies need not be there yet
        if (n > n0) copy_tri(n - 1);
      } else {
        barrier_copied();
        copy(n);
        barrier_copied();
        if (n > n0) load(n - 1);
        barrier_passed();
        if (n > n0) copy_tri(n - 1);
      }
    }
    return;
  }

  f32x4 D[KT];
  {
    // the end: the call's, or the start of the segment behind
    const int ld = (last ? a.Dv : segs.dvp) * 4;
    const Buf p = last ? rows_buf(a.ds_last + static_cast<int64_t>(bh) * a.Dk * a.Dv, a.ds_last != nullptr ? a.Dk : 0, ld, ld)
                       : rows_buf(segs.back + segs.at_back(bh, seg + 1), SUM ? 0 : segs.dkp, ld, ld);
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        D[t][r] = __uint_as_float(load_raw<false>(p, live ? (16 * t + 4 * g + r) * ld + col * 4 : kNowhere));
#pragma unroll
    for (int t = 0; t < KT; ++t) asm volatile("" : "+v"(D[t]));   // waited for here, not in every chunk
  }

  const int ldy = a.Nv * a.Dv * es;
  const int yo = live ? 4 * g * ldy + col * es : kNowhere;
  // whole 16-byte groups of bf16: lane l/2's row, its columns from 8 (l%2) on
  const bool vecy = BF16 && a.Dv % 8 == 0;
  const int vo = 16 * wg + 8 * (l & 1) < a.Dv ? (l >> 1) * ldy + (16 * wg + 8 * (l & 1)) * es : kNowhere;
  const unsigned char* s_tt = smem + Z::oTri;
  const unsigned char* s_pt = s_tt + Z::kTri;
  uint32_t ob[MT][4];   // float32: the next chunk's dO
  auto fetch = [&](int n) {
    const int64_t tok = static_cast<int64_t>(b) * a.L + n * C;
    const int o = here(yo);
    const Buf yr = rows_buf(static_cast<const char*>(a.dy) + (tok * a.Nv + h) * a.Dv * es, min(len - n * C, C), ldy, a.Dv * es);
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) ob[t][r] = load_raw<BF16>(yr, o + (16 * t + r) * ldy);
  };

  if (!BF16 && n0 < n1) fetch(n1 - 1);
  for (int n = n1 - 1; n >= n0; --n) {
    if constexpr (!Z::kTwo) barrier_read();   // the previous chunk is read
    barrier_read();                           // the chunk is there, the previous one read
    unsigned char* s_k = smem + (Z::kTwo ? (n & 1) * Z::kBuf : 0);
    const unsigned char *s_kt = s_k + Z::kMat, *s_qt = s_k + 2 * Z::kMat;
    const float* dec = reinterpret_cast<const float*>(s_k + 3 * Z::kMat);
    f32x4 dO[MT], dU[MT], dR[MT];
    Frag<NI> dy[CS];   // bf16: dO as it is
    Frag<NI> kx[2][MT];
    Frag<3> tf[2][MT];
    if constexpr (!BF16) {
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) dO[t][r] = value<BF16>(ob[t][r]);
      if (n > n0) fetch(n - 1);
    }
    if (wave_live) {
      if constexpr (!SUM) {
        const int o = here(16 * l);
        const Buf kd = rows_buf(keep.p + (static_cast<int64_t>(bh) * chunks + n) * keep.size(C) + keep.at_d() + 16 * wg * keep.dkp, 1, 0, keep.dkp * 64);
#pragma unroll
        for (int t = 0; t < KT; ++t) store16(kd, o + t * 1024, D[t]);
      }
      // dU = to K D' + P^T dO
#pragma unroll
      for (int t = 0; t < MT; ++t) dU[t] = dR[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      auto read_x = [&](int ks) {
#pragma unroll
        for (int t = 0; t < MT; ++t) kx[ks & 1][t] = read_rows<NI, KS>(s_k, t, ks);
      };
      read_x(0);
      stage_end();
      float4 to[MT];
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        if (ks + 1 < KS) {
          read_x(ks + 1);
        } else {
#pragma unroll
          for (int t = 0; t < MT; ++t) to[t] = *reinterpret_cast<const float4*>(dec + C + 16 * t + 4 * g);
          read_tri<true, C>(tf[0], s_pt, 0);
          if constexpr (BF16) {
#pragma unroll
            for (int s = 0; s < CS; ++s) dy[s] = read_cols<NI, C>(s_k + Z::oV, w, s);
          }
        }
        stage_end();
        mma(dU, kx[ks & 1], to_frag<3>(D[2 * ks], D[2 * ks + 1]));
        stage_end();
      }
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const float tt[4] = {to[t].x, to[t].y, to[t].z, to[t].w};
#pragma unroll
        for (int r = 0; r < 4; ++r) dU[t][r] *= tt[r];
      }
      // P^T and then T^T, from the first products to the last
#pragma unroll
      for (int i = 0; i < 2 * CS; ++i) {
        if (i + 1 < 2 * CS) read_tri<true, C>(tf[(i + 1) & 1], i + 1 < CS ? s_pt : s_tt, (i + 1) % CS);
        stage_end();
        const int ks = i % CS;
        if (i < CS) mma_tri<true, C>(dU, tf[i & 1], ks, BF16 ? dy[ks] : to_frag<NI>(dO[2 * ks], dO[2 * ks + 1]));
        else mma_tri<true, C>(dR, tf[i & 1], ks, to_frag<3>(dU[2 * ks], dU[2 * ks + 1]));
        stage_end();
      }
    }
    barrier_read();   // T and P are read
    if (!wave_live) continue;

    constexpr int kGroups = 2 * CS * KT / 4;   // k's fragments, then q's, four tiles at a time
    Frag<NI> cf[2][4];
    auto read_c = [&](int i) { read_cols4<NI, C>(cf[i & 1], i < kGroups / 2 ? s_kt : s_qt, 4 * (i % (KT / 4)), i % (kGroups / 2) / (KT / 4)); };
    read_c(0);
    const int64_t tok = static_cast<int64_t>(b) * a.L + n * C;
    const int o1 = here(16 * l);
    const Buf kr = rows_buf(keep.p + (static_cast<int64_t>(bh) * chunks + n) * keep.size(C) + keep.at_r(C) + 16 * wg * C, 1, 0, C * 64);
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const float4 be = *reinterpret_cast<const float4*>(dec + 2 * C + 16 * t + 4 * g);
      const float bb[4] = {be.x, be.y, be.z, be.w};
      if constexpr (!SUM) store16(kr, o1 + t * 1024, dR[t]);
#pragma unroll
      for (int r = 0; r < 4; ++r) dR[t][r] *= bb[r];
    }
    if constexpr (!SUM) {
      const Buf vr = rows_buf(static_cast<char*>(a.dv) + (tok * a.Nv + h) * a.Dv * es, min(len - n * C, C), ldy, a.Dv * es);
      if (vecy) {
        store_values(s_k + Z::oV + w * ValueStage<NW>::kWave, vr, here(vo), ldy, dR);
      } else {
        const int o2 = here(yo);
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int r = 0; r < 4; r += 2) store_el2<BF16>(vr, o2 + (16 * t + r) * ldy, ldy, dR[t][r], dR[t][r + 1]);
      }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const float4 f = *reinterpret_cast<const float4*>(dec + 16 * t + 4 * g);
      const float4 fs = *reinterpret_cast<const float4*>(dec + 3 * C + 16 * t + 4 * g);
      const float ff[4] = {f.x, f.y, f.z, f.w}, ss[4] = {fs.x, fs.y, fs.z, fs.w};
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        dR[t][r] *= -ff[r];
        dO[t][r] = ss[r] * (BF16 ? element(dy[t >> 1], t & 1, r) : dO[t][r]);
      }
    }
    const float whole = dec[C - 1];
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) D[t][r] *= whole;
    Frag<3> xf[2 * CS];
#pragma unroll
    for (int ks = 0; ks < CS; ++ks) {
      xf[ks] = to_frag<3>(dR[2 * ks], dR[2 * ks + 1]);
      xf[CS + ks] = to_frag<3>(dO[2 * ks], dO[2 * ks + 1]);
    }
    stage_end();
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      if (i + 1 < kGroups) read_c(i + 1);
      stage_end();
      mma_cols4(D, 4 * (i % (KT / 4)), cf[i & 1], xf[i / (KT / 4)]);
      stage_end();
    }
  }

  float* end = SUM ? segs.back + segs.at_back(bh, seg) : seg == 0 && a.ds0 != nullptr ? a.ds0 + static_cast<int64_t>(bh) * a.Dk * a.Dv : nullptr;
  if (end != nullptr && wave_live) {
    const int ld = (SUM ? segs.dvp : a.Dv) * 4;
    const Buf p = rows_buf(end, SUM ? segs.dkp : a.Dk, ld, ld);
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        store_el<false>(p, SUM || live ? (16 * t + 4 * g + r) * ld + col * 4 : kNowhere, D[t][r]);
  }
}

// ---- the gradients without a chain ------------------------------------------------
// A wave has 32 features of a key and half of the chunk's tokens (with 16
// features and all tokens it reads more of the LDS: 185 us instead of 181 for 64
// value heads of 2048 steps, 128 x 128 bf16).
// The products over the value features run in steps of 32: S, D', U, dR and dY
// are split into parts and put into row fragments in LDS once for the
// workgroup, the next step's loads on their way meanwhile; each wave has its
// part of E = dY S^T, F = dR S^T and H = U D'^T, and a share of the C x C
// products W1 = dY U^T and W2 = dR U^T. These are computed both ways round, since a product comes out
// with the rows of its first factor where an operand has its products: the
// result masked, decayed and split is an operand's fragment as it lies. Then
// the products over tokens go on in E, F and H.

template <bool BF16, int KP>
struct Grad : Shape<BF16, KP> {
  using Z = Shape<BF16, KP>;
  static constexpr int NW = KP / 16, kThreads = 64 * NW;
  static constexpr int kTri = tri_frags<Z::C>(), kJobs = (4 * kTri + NW - 1) / NW;
  static constexpr int kItems = 4 * Z::MT / NW;   // staged tiles of dR, U, dY and V of a wave
  // whether all waves' j-th jobs are of W2, or of W1
  static constexpr bool all_w2(int j) { return (j + 1) * NW <= 2 * kTri; }
  static constexpr bool all_w1(int j) { return j * NW >= 2 * kTri; }
  static constexpr int oR = 0, oU = oR + Z::MT * 3 * kFrag, oY = oU + Z::MT * 3 * kFrag, oV = oY + Z::MT * Z::NI * kFrag;
  static constexpr int oS = oV + Z::MT * Z::NI * kFrag, oD = oS + Z::KT * 3 * kFrag, kStage = oD + Z::KT * 3 * kFrag;
  static constexpr int kW = 4 * kTri * 3 * kFrag;           // over the stage when that is read
  static constexpr int oG = kStage > kW ? kStage : kW;      // double sums of g
  static constexpr int oB = oG + Z::C * 8;                  // beta, from, to
  static constexpr int TT = Z::MT / 2;                      // token tiles of a wave
  static constexpr int oRed = oB + 3 * Z::C * 4;            // [NW / 2][2][C] row sums
  static constexpr int oRV = oRed + NW * Z::C * 4;          // [C] dR.V
  static constexpr int oEnd = oRV + Z::C * 4;               // [NW] the waves' parts of the last token's dG
  static constexpr int oAcc = oEnd + NW * 4;                // [NW][2 MT][64] dq and dk, where heads share a key
  static constexpr int kAcc = NW * 2 * Z::MT * kFrag;
  // Up to 64 features two workgroups fit a compute unit; with these sums in the LDS
  // not of bf16, whose sums are in memory then (16 heads on 8 keys, 10 x 1481
  // tokens, 64 x 128: 210 us, in the LDS 285). Those of float32 fit too (16 heads on
  // 4 keys, 10 x 1481 tokens, 64 x 64, forward and gradients: 636 us, in memory 646).
  static constexpr bool kAccLds = KP > 64 || 2 * (oAcc + kAcc) <= kMaxLds;
  static constexpr int kLds = oAcc + (kAccLds ? kAcc : 0), kGroups = KP > 64 ? 256 : 512;
};

// Sums of N values each over the 16 lanes of a row: halves of the values and of
// the lanes are exchanged four times, after which lane m has N/16 of the sums,
// from index m N/16 on.
template <int CTRL>
__device__ __forceinline__ float from_lane(float x) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), CTRL, 0xf, 0xf, true));
}
template <int CTRL, int H, int N>
__device__ __forceinline__ void fold(float (&x)[N], bool upper) {
#pragma unroll
  for (int i = 0; i < H; ++i) {
    const float a = x[i], b = x[i + H];
    x[i] = (upper ? b : a) + from_lane<CTRL>(upper ? a : b);
  }
}
template <int N>
__device__ __forceinline__ void row_sums(float (&x)[N], int m) {
  fold<0x140, N / 2>(x, m & 8);    // row_mirror
  fold<0x141, N / 4>(x, m & 4);    // row_half_mirror
  fold<0x4e, N / 8>(x, m & 2);     // quad_perm 2, 3, 0, 1
  fold<0xb1, N / 16>(x, m & 1);    // quad_perm 1, 0, 3, 2
}

// Places of a lane's values in row fragments: of rows l/16 * 4.. of the columns
// 2 cp, 2 cp + 1 (cp = l%16) of a step, as they are kept, and of the columns
// 8 (l%4).. of row l/4. A wave has 16 rows of either.
__device__ __forceinline__ int kept_place(int l) {
  const int cp = l & 15, gc = (cp & 7) >> 1;
  return slot_of(gc, 4 * (l >> 4), gc) + 8 * (cp >> 3) + 4 * (cp & 1);
}
__device__ __forceinline__ int row_place(int l) { return slot_of(2 * (l & 1), l >> 2, 2 * (l & 1)) + 8 * ((l >> 1) & 1); }

__device__ __forceinline__ void store_kept(unsigned char* tile, int place, const uint4& lo, const uint4& hi) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float x = __uint_as_float(word(lo, j)), y = __uint_as_float(word(hi, j));
    unsigned char* p = tile + (place ^ 16 * j);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      *reinterpret_cast<uint32_t*>(p + i * kFrag) = upper(x, y);
      x -= cut(x);
      y -= cut(y);
    }
  }
}
// NI = 1: the bits of eight bf16, else two times four floats
template <int NI>
__device__ __forceinline__ void store_row8(unsigned char* tile, int place, const uint4& lo, const uint4& hi) {
  // the second four: the next slot group, whose rows are exchanged by one more
  unsigned char *p = tile + place, *q = tile + ((place + 256) ^ 16);
  if constexpr (NI == 1) {
    *reinterpret_cast<uint2*>(p) = uint2{lo.x, lo.y};
    *reinterpret_cast<uint2*>(q) = uint2{lo.z, lo.w};
  } else {
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = __uint_as_float(word(lo, i));
      x[4 + i] = __uint_as_float(word(hi, i));
    }
    const Frag<NI> f = to_frag<NI>(x);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const uint4 w = __builtin_bit_cast(uint4, f.p[i]);
      *reinterpret_cast<uint2*>(p + i * kFrag) = uint2{w.x, w.y};
      *reinterpret_cast<uint2*>(q + i * kFrag) = uint2{w.z, w.w};
    }
  }
}

// One of the C x C products' operand fragments: W1 = dY U^T (mat 0) and
// transposed (1), W2 = dR U^T (2, 3); the larger products first. Fragment f has
// the row tile rt and the products of 32 from tile 2 st on.
template <int C>
struct Job {
  static constexpr int kTri = tri_frags<C>();
  int q, mat, f, rt, st;
  __device__ __forceinline__ explicit Job(int n) : q(n), mat(n < 2 * kTri ? 2 + n / kTri : n / kTri - 2), f(n % kTri) {
    rt = C == 32 ? f : (mat & 1) ? (f < 4 ? f >> 1 : f - 2) : (f < 2 ? f : (f >> 1) + 1);
    st = C == 32 ? 0 : (mat & 1) ? (f < 4 ? f & 1 : 1) : (f < 2 ? 0 : f & 1);
  }
  __device__ __forceinline__ bool ours() const { return q < 4 * kTri; }
  __device__ __forceinline__ bool w2() const { return q < 2 * kTri; }
};

// VEC: whole 16-byte groups of dy and v are aligned
template <bool BF16, int KP, bool VEC>
__global__ void __launch_bounds__(4 * KP, 2) k_delta_grad(DeltaArgs a, int chunks, DeltaKeep keep) {
  using Z = Grad<BF16, KP>;
  constexpr int C = Z::C, MT = Z::MT, CS = Z::CS, NI = Z::NI, NW = Z::NW, TT = Z::TT, es = Z::es;
  extern __shared__ __align__(16) unsigned char smem[];
  double* s_g = reinterpret_cast<double*>(smem + Z::oG);
  float *s_b = reinterpret_cast<float*>(smem + Z::oB), *s_from = s_b + C, *s_to = s_from + C;
  float *s_red = reinterpret_cast<float*>(smem + Z::oRed), *s_rv = reinterpret_cast<float*>(smem + Z::oRV), *s_end = reinterpret_cast<float*>(smem + Z::oEnd);
  const int tid = threadIdx.x, l = tid & 63, g = l >> 4, m = l & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int f0 = w & ~1, th = w & 1, t0 = th * TT;   // feature tiles f0, f0 + 1, token tiles from t0 on
  const int group = a.Hv / a.Hk, items = a.B * a.Hk * chunks;

  auto value_of = [&](const Frag<NI>& f, int e) {
    float x = static_cast<float>(f.p[0][e]);
#pragma unroll
    for (int p = 1; p < NI; ++p) x += static_cast<float>(f.p[p][e]);
    return x;
  };

  // The workgroup's chunks it, it + gridDim, ... and their heads, one after the
  // other: the next one's first loads are under way while one is finished.
  struct Place {
    int it, hh, b, hk, n, left;
  };
  auto advance = [&](Place& p) {
    if (++p.hh < group) return true;
    p.hh = 0;
    for (p.it += gridDim.x; p.it < items; p.it += gridDim.x) {
      const int bk = p.it / chunks;
      p.n = p.it - bk * chunks;
      p.b = bk / a.Hk;
      p.hk = bk - p.b * a.Hk;
      p.left = length_of(a, p.b) - p.n * C;
      if (p.left > 0) return true;
    }
    return false;
  };

  // A step's values of a thread, eight of each: rows of S and D' (tile w); then
  // 16 rows of a wave at a time of dR, U, dY and V (tile w + j NW of all four)
  struct Eight {
    uint4 lo, hi;
  };
  constexpr int kFirstIo = 2 * MT;   // tile numbers of dY and V
  auto all_kept = [](int j) { return (j + 1) * NW <= kFirstIo; };
  auto all_io = [](int j) { return j * NW >= kFirstIo; };
  Eight kept_s, kept_d, et[Z::kItems];
  float gn = 0.0f, bn = 0.0f;    // the first two waves': g and beta
  const int lane_kept = g * 256 + (m & 7) * 32, lane_s = lane_kept + (m >> 3) * keep.dkp * 64, lane_r = lane_kept + (m >> 3) * C * 64;
  auto fetch = [&](const Place& p, int v0) {
    const int h = p.hk * group + p.hh;
    const int64_t tok = static_cast<int64_t>(p.b) * a.L + p.n * C;
    const float* kept = keep.p + ((static_cast<int64_t>(p.b) * a.Hv + h) * chunks + p.n) * keep.size(C);
    // four rows of two columns of the array at `at`, tile t of its `rows` rows:
    // what does not exist is outside the buffer
    auto load_kept = [&](int at, int rows, int t, int o) {
      const Buf b = rows_buf(kept + at + v0 * rows + t * 256, 16 * t < rows ? 1 : 0, 0, (v0 + 16 < keep.dvp ? rows * 64 : 0) + 1024);
      return Eight{load16(b, o), load16(b, o + 16)};
    };
    auto load_io = [&](bool second, int t) {
      const int64_t ld = second ? a.ldv : a.Nv * a.Dv;
      const char* src = static_cast<const char*>(second ? a.v : a.dy) + ((tok + 16 * t) * ld + static_cast<int64_t>(h) * a.Dv) * es;
      const int ldb = row_bytes(ld, es), v = v0 + 8 * (l & 3), o = (l >> 2) * ldb + v * es;
      const Buf r = rows_buf(src, min(p.left, C) - 16 * t, ldb, a.Dv * es);
      Eight x{};
      if constexpr (VEC) {
        x.lo = load16(r, v < a.Dv ? o : kNowhere);
        if constexpr (!BF16) x.hi = load16(r, v + 4 < a.Dv ? o + 16 : kNowhere);
      } else {
        uint32_t e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = load_raw<BF16>(r, v + i < a.Dv ? o + i * es : kNowhere);
        if constexpr (BF16) {
          x.lo = uint4{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16};
        } else {
          x.lo = uint4{e[0], e[1], e[2], e[3]};
          x.hi = uint4{e[4], e[5], e[6], e[7]};
        }
      }
      return x;
    };
    kept_s = load_kept(0, keep.dkp, w, lane_s);
    kept_d = load_kept(keep.at_d(), keep.dkp, w, lane_s);
#pragma unroll
    for (int j = 0; j < Z::kItems; ++j) {
      const int t = w + j * NW;
      if (all_kept(j) || (!all_io(j) && t < kFirstIo)) et[j] = load_kept(t < MT ? keep.at_r(C) : keep.at_u(), C, t % MT, lane_r);
      else et[j] = load_io(t >= kFirstIo + MT, t % MT);
    }
    if (v0 == 0 && w < 2) {
      const bool in = l < C && l < p.left;
      gn = in ? a.g[(tok + l) * a.Nv + h] : 0.0f;
      bn = in ? a.beta[(tok + l) * a.Nv + h] : 0.0f;
    }
  };
  const int kept_at = kept_place(l), row_at = row_place(l);

  Place at{static_cast<int>(blockIdx.x) - static_cast<int>(gridDim.x), group - 1, 0, 0, 0, 0};
  if (!advance(at)) return;
  // sums of g and the decays that come from them: the second wave's, while the
  // first one finishes the head before
  auto decays = [&] {
    const double s = chunk_sums(gn);
    const double end = __shfl(s, C - 1);
    if (l < C) {
      s_g[l] = s;
      s_b[l] = bn;
      s_from[l] = expf(static_cast<float>(s));
      s_to[l] = expf(static_cast<float>(end - s));
    }
  };
  fetch(at, 0);
  if (w == 1) decays();
  for (bool more = true; more;) {
    const int h = at.hk * group + at.hh, left = at.left, rows = min(left, C);
    const int64_t tok = static_cast<int64_t>(at.b) * a.L + at.n * C;
    const float gi = gn;

    f32x4 E[2][TT], F[2][TT], H[2][TT], W[Z::kJobs][2], RV = {0.0f, 0.0f, 0.0f, 0.0f}, SD = RV;
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int t = 0; t < TT; ++t) E[f][t] = F[f][t] = H[f][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < Z::kJobs; ++j) W[j][0] = W[j][1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    int v0 = 0;
#pragma clang loop unroll(disable)
    while (true) {
      {
        store_kept(smem + Z::oS + w * 3 * kFrag, here(kept_at), kept_s.lo, kept_s.hi);
        store_kept(smem + Z::oD + w * 3 * kFrag, here(kept_at), kept_d.lo, kept_d.hi);
#pragma unroll
        for (int j = 0; j < Z::kItems; ++j) {
          const int t = w + j * NW;
          if (all_kept(j) || (!all_io(j) && t < kFirstIo)) store_kept(smem + (t < MT ? Z::oR : Z::oU) + (t % MT) * 3 * kFrag, here(kept_at), et[j].lo, et[j].hi);
          else store_row8<NI>(smem + (t < kFirstIo + MT ? Z::oY : Z::oV) + (t % MT) * NI * kFrag, here(row_at), et[j].lo, et[j].hi);
        }
      }
      __syncthreads();
      v0 += 32;
      if (v0 < keep.dvp) fetch(at, v0);
      {
        const Frag<3> sf[2] = {read_frag<3>(smem + Z::oS, f0, g), read_frag<3>(smem + Z::oS, f0 + 1, g)};
        {
          Frag<NI> y[TT];
#pragma unroll
          for (int t = 0; t < TT; ++t) y[t] = read_frag<NI>(smem + Z::oY, t0 + t, g);
          mma(E[0], y, sf[0]);
          mma(E[1], y, sf[1]);
        }
        __builtin_amdgcn_sched_barrier(0);   // one product's fragments at a time: more would spill
        Frag<3> x[TT];
#pragma unroll
        for (int t = 0; t < TT; ++t) x[t] = read_frag<3>(smem + Z::oR, t0 + t, g);
        mma(F[0], x, sf[0]);
        mma(F[1], x, sf[1]);
        // dR.V is the diagonal of dR V^T: tile t0 + r of it by the r-th last wave of
        // this half (they have the fewest other products)
        const int r = (NW - 2 - f0) / 2;
#pragma unroll
        for (int t = 0; t < TT; ++t)
          if (t == r) RV = mma(x[t], read_frag<NI>(smem + Z::oV, t0 + t, g), RV);
        __builtin_amdgcn_sched_barrier(0);
        const Frag<3> df[2] = {read_frag<3>(smem + Z::oD, f0, g), read_frag<3>(smem + Z::oD, f0 + 1, g)};
        // <D', S> is the sum of the diagonal of D' S^T
        if (th == 0) SD = mma(df[0], sf[0], SD);
        else SD = mma(df[1], sf[1], SD);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int t = 0; t < TT; ++t) x[t] = read_frag<3>(smem + Z::oU, t0 + t, g);
        mma(H[0], x, df[0]);
        mma(H[1], x, df[1]);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int j = 0; j < Z::kJobs; ++j) {
        const Job<C> job(w + j * NW);
        if (job.ours()) {
          // tiles of the products (accumulator rows): 2 st, 2 st + 1; the row tile: columns
          if (Z::all_w2(j) || (!Z::all_w1(j) && job.w2())) {
            const unsigned char *s1 = smem + (job.mat == 2 ? Z::oU : Z::oR), *s2 = smem + (job.mat == 2 ? Z::oR : Z::oU);
            const Frag<3> c = read_frag<3>(s2, job.rt, g);
            Frag<3> p[2] = {read_frag<3>(s1, 2 * job.st, g), read_frag<3>(s1, 2 * job.st + 1, g)};
            mma(W[j], p, c);
          } else if (job.mat == 0) {
            const Frag<NI> c = read_frag<NI>(smem + Z::oY, job.rt, g);
            Frag<3> p[2] = {read_frag<3>(smem + Z::oU, 2 * job.st, g), read_frag<3>(smem + Z::oU, 2 * job.st + 1, g)};
            mma(W[j], p, c);
          } else {
            const Frag<3> c = read_frag<3>(smem + Z::oU, job.rt, g);
            Frag<NI> p[2] = {read_frag<NI>(smem + Z::oY, 2 * job.st, g), read_frag<NI>(smem + Z::oY, 2 * job.st + 1, g)};
            mma(W[j], p, c);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      __syncthreads();   // the step is read
      if (v0 >= keep.dvp) break;
    }
    // k and q of this wave's features, as operands over the tokens; their slots
    // are also the values at the accumulators' places
    Frag<NI> kf[2][CS], qf[2][CS];
    {
      const unsigned char* fr = a.frags + static_cast<int64_t>(at.it) * Z::frags(true);
#pragma unroll
      for (int s = 0; s < CS; ++s)
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          kf[f][s] = read_cols<NI, C>(fr, f0 + f, s);
          qf[f][s] = read_cols<NI, C>(fr + Z::kMat, f0 + f, s);
        }
    }
    __builtin_amdgcn_sched_barrier(0);   // under way while W1 and W2 are finished
#pragma unroll
    for (int j = 0; j < Z::kJobs; ++j) {
      const Job<C> job(w + j * NW);
      if (job.ours()) {
        // element e: product p of the fragment, row q; rows i and j of M are q and
        // p, or p and q in the transposed ones
        const bool up = job.mat & 1;
        const int gg = here(g), diff = up ? m - 4 * gg : 4 * gg - m, p0 = 32 * job.st, q0 = 16 * job.rt;
        const int most = (job.mat == 0 || job.mat == 1 ? 0 : -1);   // p - q (up: q - p) at most
        const double gq = s_g[q0 + m], sign = up ? -1.0 : 1.0;
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int o = p0 + 16 * (e >> 2) + (e & 3);
          const float f = decay_exp(sign * (gq - s_g[o + 4 * gg])) * W[j][e >> 2][e & 3];
          x[e] = diff <= (up ? most + o - q0 : most - o + q0) ? f : 0.0f;
        }
        if (job.w2()) {
          if (up) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= -s_b[p0 + 16 * (e >> 2) + 4 * gg + (e & 3)];
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] *= a.scale;
        }
        const Frag<3> fr = to_frag<3>(x);
        unsigned char* to = smem + (job.mat * Z::kTri + job.f) * 3 * kFrag + here(16 * l);
#pragma unroll
        for (int p = 0; p < 3; ++p) *reinterpret_cast<bf16x8*>(to + p * kFrag) = fr.p[p];
      }
    }
    const int gg = here(g), mm = here(m);
    if ((NW - 2 - f0) / 2 < TT) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (4 * gg + r == mm) s_rv[16 * (t0 + (NW - 2 - f0) / 2) + mm] = RV[r];
    }
    // <D', S> whole + sum of to k.(U D'^T): this lane's part
    float ends = 0.0f;
#pragma unroll
    for (int r = 0; r < 4; ++r) ends = 4 * gg + r == mm ? SD[r] : ends;
    ends *= s_from[C - 1];
    // this wave's tokens among the products of its fragments: one of two, or a half
    // of one
    auto own = [&](const Frag<NI> (&x)[CS]) {
      Frag<NI> y;
#pragma unroll
      for (int p = 0; p < NI; ++p) {
        const uint4 u = __builtin_bit_cast(uint4, x[0].p[p]), z = __builtin_bit_cast(uint4, x[CS - 1].p[p]);
        y.p[p] = __builtin_bit_cast(bf16x8, CS == 2 ? uint4{th == 0 ? u.x : z.x, th == 0 ? u.y : z.y, th == 0 ? u.z : z.z, th == 0 ? u.w : z.w}
                                                    : uint4{th == 0 ? u.x : u.z, th == 0 ? u.y : u.w, 0, 0});
      }
      return y;
    };
    const Frag<NI> kown[2] = {own(kf[0]), own(kf[1])};
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const float4 fr = *reinterpret_cast<const float4*>(s_from + 16 * (t0 + t) + 4 * gg);
      const float4 to = *reinterpret_cast<const float4*>(s_to + 16 * (t0 + t) + 4 * gg);
      const float ff[4] = {fr.x, fr.y, fr.z, fr.w}, tt[4] = {to.x, to.y, to.z, to.w};
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          E[f][t][r] *= a.scale * ff[r];
          F[f][t][r] *= ff[r];
          H[f][t][r] *= tt[r];
          ends = fmaf(value_of(kown[f], 4 * t + r), H[f][t][r], ends);
        }
    }
    __syncthreads();   // W1 and W2 are there
    Place next = at;
    more = advance(next);
    if (more) fetch(next, 0);
    // the wave's row tiles of a C x C matrix times k or q over all tokens
    auto triangle = [&](f32x4 (&c)[2][TT], int mat, const Frag<NI> (&x)[2][CS]) {
#pragma unroll
      for (int s = 0; s < CS; ++s) {
        if (CS == 2 && ((mat & 1) ? th > s : th < s)) continue;   // zeros
        Frag<3> f[TT];
#pragma unroll
        for (int t = 0; t < TT; ++t)
          f[t] = read_frag<3>(smem, mat * Z::kTri + ((mat & 1) ? tri_frag_t<C>(t0 + t, s) : tri_frag<C>(t0 + t, s)), 0);
#pragma unroll
        for (int i = 0; i < 3; ++i)
#pragma unroll
          for (int j = 0; j < NI && i + j < 3; ++j)
#pragma unroll
            for (int t = 0; t < TT; ++t) {
              c[0][t] = mfma(f[t].p[i], x[0][s].p[j], c[0][t]);
              c[1][t] = mfma(f[t].p[i], x[1][s].p[j], c[1][t]);
            }
      }
    };
    triangle(E, 0, kf);    // dQ
    __builtin_amdgcn_sched_barrier(0);
    triangle(F, 2, kf);    // -Hrow
    __builtin_amdgcn_sched_barrier(0);
    triangle(H, 1, qf);
    __builtin_amdgcn_sched_barrier(0);
    triangle(H, 3, kf);    // dKcol
    __builtin_amdgcn_sched_barrier(0);
    {
      // rows of dG and k.Hrow: this wave's features
      const Frag<NI> qown[2] = {own(qf[0]), own(qf[1])};
      float x[8 * TT];
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const float4 be = *reinterpret_cast<const float4*>(s_b + 16 * (t0 + t) + 4 * gg);
        const float bb[4] = {be.x, be.y, be.z, be.w};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float dg = 0.0f, hk = 0.0f;
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            const float kv = value_of(kown[f], 4 * t + r), qv = value_of(qown[f], 4 * t + r);
            const float row = bb[r] * F[f][t][r];
            dg += qv * E[f][t][r] - kv * (H[f][t][r] + row);
            hk -= kv * F[f][t][r];
            H[f][t][r] -= row;   // dK of the head
          }
          x[4 * t + r] = dg;
          x[4 * TT + 4 * t + r] = hk;
        }
      }
      float* to = s_red + f0 * C + 16 * t0 + 4 * gg;
      if constexpr (TT == 2) {
        row_sums(x, mm);   // lane m has sum m: of dG in the first eight lanes
        to[(mm >> 3) * C + 16 * ((mm >> 2) & 1) + (mm & 3)] = x[0];
      } else {
        float y[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          y[i] = x[i];
          y[8 + i] = 0.0f;
        }
        row_sums(y, mm);
        if (mm < 8) to[(mm >> 2) * C + (mm & 3)] = y[0];
      }
      ends += from_lane<0x128>(ends);   // row_ror 8, 4, 2, 1
      ends += from_lane<0x124>(ends);
      ends += from_lane<0x122>(ends);
      ends += from_lane<0x121>(ends);
      ends += __shfl_xor(ends, 16);
      ends += __shfl_xor(ends, 32);
      if (l == 0) s_end[w] = ends;
    }
    // dq and dk of the heads that share a key: in LDS until the last one
    f32x4* sum = (Z::kAccLds ? reinterpret_cast<f32x4*>(smem + Z::oAcc)
                             : reinterpret_cast<f32x4*>(keep.sums) + static_cast<int64_t>(blockIdx.x) * (Z::kAcc / 16)) +
                 w * 2 * MT * 64 + here(l);
    if (at.hh > 0) {
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          E[f][t] += sum[(f * TT + t) * 64];
          H[f][t] += sum[(MT + f * TT + t) * 64];
        }
    }
    if (at.hh + 1 < group) {
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          sum[(f * TT + t) * 64] = E[f][t];
          sum[(MT + f * TT + t) * 64] = H[f][t];
        }
    } else {
      const int ldo = here_s(a.Nk * a.Dk * es);
      const Buf qo = rows_buf(static_cast<char*>(a.dq) + (tok * a.Nk + at.hk) * a.Dk * es, rows, ldo, a.Dk * es);
      const Buf ko = rows_buf(static_cast<char*>(a.dk) + (tok * a.Nk + at.hk) * a.Dk * es, rows, ldo, a.Dk * es);
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const int c = 16 * (f0 + f) + m;
        const int oo = here(c < a.Dk ? (16 * t0 + 4 * g) * ldo + c * es : kNowhere);
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
          for (int r = 0; r < 4; r += 2) {
            store_el2<BF16>(qo, oo + (16 * t + r) * ldo, ldo, E[f][t][r], E[f][t][r + 1]);
            store_el2<BF16>(ko, oo + (16 * t + r) * ldo, ldo, H[f][t][r], H[f][t][r + 1]);
          }
      }
    }
    __syncthreads();   // the sums are there, the fragments and decays read
    if (w == 1 && more) decays();
    if (w == 0) {
      float g1 = 0.0f, k1 = 0.0f, last = 0.0f;
      const int i = l < C ? l : 0;
#pragma unroll
      for (int x = 0; x < NW / 2; ++x) {
        g1 += s_red[2 * x * C + i];
        k1 += s_red[(2 * x + 1) * C + i];
      }
#pragma unroll
      for (int x = 0; x < NW; ++x) last += s_end[x];
      g1 += l == C - 1 ? last : 0.0f;
      // sums from the end: the lanes the other way round
      const int r = C - 1 - l;
      const double sums = lane_sums(l < C ? __shfl(g1, r & 63) : 0.0f), dg = __shfl(sums, r & 63);
      if (l < C && l < left) {
        // a decay that clears the state hides what it multiplied
        a.dg[(tok + l) * a.Nv + h] = gi < kLeastDecay ? 0.0f : static_cast<float>(dg);
        a.dbeta[(tok + l) * a.Nv + h] = s_rv[l] + k1;
      }
    }
    at = next;
  }
}

// finds the workspace's parts (of a slice); bytes of all of them
int64_t keep_of(DeltaArgs& a, DeltaSegs& segs, DeltaKeep& k) {
  const int C = a.bf16_io ? 64 : 32;
  const int64_t chunks = static_cast<int64_t>(a.B) * a.Hv * ((a.L + C - 1) / C);
  k.dkp = (a.Dk + 15) & ~15;
  k.dvp = (a.Dv + 15) & ~15;
  const int64_t head = (delta_work(a, segs, true) + 15) & ~int64_t{15};
  k.p = reinterpret_cast<float*>(static_cast<unsigned char*>(a.ws) + head);
  k.sums = k.p + chunks * k.size(C);
  using G = Grad<true, 64>;
  static_assert(!G::kAccLds && Grad<false, 64>::kAccLds);
  const int64_t acc = a.bf16_io && a.Dk <= 64 && a.Hv > a.Hk ? G::kAcc * G::kGroups : 0;
  return head + chunks * k.size(C) * 4 + acc;
}

// the chain's passes, for all segments or for their sums
template <bool BF16, int KP, int NW, bool SUM>
hipError_t chain(const DeltaArgs& a, const DeltaSegs& segs, const DeltaKeep& keep, hipStream_t stream) {
  using Z = Back<BF16, KP, NW>;
  constexpr auto* kern = k_delta_back_scan<BF16, KP, NW, SUM>;
  if (const hipError_t e = allow_lds<kern>(Z::kLds); e != hipSuccess) return e;
  const int chunks = (a.L + Z::C - 1) / Z::C, groups = (a.Dv + 16 * NW - 1) / (16 * NW);
  const int64_t blocks = (static_cast<int64_t>(a.B) * a.Hv * (SUM ? segs.count - 1 : segs.count) + 7) / 8 * 8 * groups;
  kern<<<dim3(static_cast<unsigned>(blocks)), dim3(64 * (NW + kCopy)), Z::kLds, stream>>>(a, chunks, groups, segs, keep);
  return hipGetLastError();
}

template <bool BF16, int KP, bool VEC>
hipError_t grad(const DeltaArgs& a, const DeltaKeep& keep, hipStream_t stream) {
  using G = Grad<BF16, KP>;
  constexpr auto* kern = k_delta_grad<BF16, KP, VEC>;
  if (const hipError_t e = allow_lds<kern>(G::kLds); e != hipSuccess) return e;
  const int chunks = (a.L + G::C - 1) / G::C;
  const int64_t items = static_cast<int64_t>(a.B) * a.Hk * chunks;
  const int lds = G::kLds - (G::kAccLds && a.Hv == a.Hk ? G::kAcc : 0);
  kern<<<dim3(static_cast<unsigned>(items < G::kGroups ? items : G::kGroups)), dim3(G::kThreads), lds, stream>>>(a, chunks, keep);
  return hipGetLastError();
}

template <bool BF16, int KP>
hipError_t run(DeltaArgs a, hipStream_t stream) {   // a slice
  DeltaKeep keep{};
  DeltaSegs segs{};
  keep_of(a, segs, keep);
  const int64_t heads = static_cast<int64_t>(a.B) * a.Hv;
  hipError_t e = hipSuccess;
  if (a.L > 0) {
    e = launch_delta_prep(a, true, stream);
    if (e == hipSuccess) e = launch_delta_scan(a, segs, &keep, stream);
  }
  if (e == hipSuccess && segs.count > 1) {
    e = narrow_groups(heads * (segs.count - 1), a.Dv) ? chain<BF16, KP, 2, true>(a, segs, keep, stream) : chain<BF16, KP, 4, true>(a, segs, keep, stream);
    if (e == hipSuccess) e = launch_delta_join_back(a, segs, stream);
  }
  if (e == hipSuccess) e = narrow_groups(heads * segs.count, a.Dv) ? chain<BF16, KP, 2, false>(a, segs, keep, stream) : chain<BF16, KP, 4, false>(a, segs, keep, stream);
  if (e != hipSuccess || a.L == 0) return e;
  // dy is contiguous and 16-byte aligned
  constexpr int V = BF16 ? 8 : 4;
  const bool vec = a.Dv % V == 0 && a.ldv % V == 0 && (reinterpret_cast<uintptr_t>(a.v) & 15u) == 0;
  return vec ? grad<BF16, KP, true>(a, keep, stream) : grad<BF16, KP, false>(a, keep, stream);
}

// What the chains leave for the gradients is far more than the call's arrays (4.5
// KB for a token and head of 128 x 128 bf16, whose v, y and their gradients are 1
// KB), so a call that would leave more than kKeepMost is cut into slices that
// follow each other in one workspace: some sequences each, or some key heads (with
// their value heads) of one sequence. Slices of this size still fill the chip: forward
// and gradients of 9 x 8192 steps of 16 heads, 128 x 128 bf16, take 5.48 ms in one
// piece and 5.42 in two, of one sequence of 131072 steps 10.9 and 11.2.
constexpr int64_t kKeepMost = int64_t{4} << 30;

struct Slices {
  int seqs, heads;   // sequences and key heads of a slice
  int64_t bytes;     // of workspace
};

int64_t bytes_of(const DeltaArgs& a, int seqs, int heads) {
  DeltaArgs s = a;
  s.B = seqs;
  s.Hv = a.Hv / a.Hk * heads;
  s.Hk = heads;
  DeltaSegs segs{};
  DeltaKeep k{};
  return keep_of(s, segs, k);
}

// the fewest equal parts of n that need at most kKeepMost each (parts of one may need more)
template <class F>
int part_of(int n, F bytes) {
  const int64_t all = bytes(n);
  if (bytes(1) > kKeepMost) return 1;
  for (int64_t parts = (all + kKeepMost - 1) / kKeepMost; parts < n; ++parts) {
    const int part = static_cast<int>((n + parts - 1) / parts);
    if (bytes(part) <= kKeepMost) return part;
  }
  return 1;
}

Slices slices_of(const DeltaArgs& a) {
  Slices s{a.B, a.Hk, bytes_of(a, a.B, a.Hk)};
  if (s.bytes <= kKeepMost) return s;
  s.seqs = part_of(a.B, [&](int n) { return bytes_of(a, n, a.Hk); });
  if (s.seqs == 1) s.heads = part_of(a.Hk, [&](int n) { return bytes_of(a, 1, n); });
  // the last slice is smaller, but may have segments where the others have none
  s.bytes = bytes_of(a, s.seqs, s.heads);
  if (const int rest = a.B % s.seqs; rest > 0) s.bytes = std::max(s.bytes, bytes_of(a, rest, a.Hk));
  if (const int rest = a.Hk % s.heads; rest > 0) s.bytes = std::max(s.bytes, bytes_of(a, 1, rest));
  return s;
}

// sequences from b on and key heads from hk on (one sequence, if not all of them)
DeltaArgs slice(const DeltaArgs& a, const Slices& n, int b, int hk) {
  DeltaArgs s = a;
  const int group = a.Hv / a.Hk, h = hk * group;
  s.B = std::min(n.seqs, a.B - b);
  s.Hk = std::min(n.heads, a.Hk - hk);
  s.Hv = s.Hk * group;
  const int64_t tok = static_cast<int64_t>(b) * a.L, es = a.bf16_io ? 2 : 4;
  const int64_t vy = (tok * a.Nv + h) * a.Dv, qk = (tok * a.Nk + hk) * a.Dk, gb = tok * a.Nv + h;
  const int64_t state = (static_cast<int64_t>(b) * a.Hv + h) * a.Dk * a.Dv;
  auto at = [](auto* p, int64_t bytes) {
    using T = decltype(p);
    return p == nullptr ? p : reinterpret_cast<T>(reinterpret_cast<uintptr_t>(p) + bytes);
  };
  s.q = at(a.q, (tok * a.ldq + static_cast<int64_t>(hk) * a.Dk) * es);
  s.k = at(a.k, (tok * a.ldk + static_cast<int64_t>(hk) * a.Dk) * es);
  s.v = at(a.v, (tok * a.ldv + static_cast<int64_t>(h) * a.Dv) * es);
  s.g = at(a.g, gb * 4);
  s.beta = at(a.beta, gb * 4);
  s.s0 = at(a.s0, state * 4);
  s.lengths = at(a.lengths, b * 4);
  s.dy = at(a.dy, vy * es);
  s.ds_last = at(a.ds_last, state * 4);
  s.dq = at(a.dq, qk * es);
  s.dk = at(a.dk, qk * es);
  s.dv = at(a.dv, vy * es);
  s.dg = at(a.dg, gb * 4);
  s.dbeta = at(a.dbeta, gb * 4);
  s.ds0 = at(a.ds0, state * 4);
  return s;
}

hipError_t run(const DeltaArgs& a, hipStream_t stream) {
  if (a.bf16_io) return a.Dk > 64 ? run<true, 128>(a, stream) : run<true, 64>(a, stream);
  return a.Dk > 64 ? run<false, 128>(a, stream) : run<false, 64>(a, stream);
}

}  // namespace

int64_t delta_workspace(const DeltaArgs& args, bool backward) {
  DeltaArgs a = args;
  DeltaSegs segs{};
  return backward ? slices_of(a).bytes : delta_work(a, segs, false);
}

hipError_t launch_delta_backward(const DeltaArgs& a, hipStream_t stream) {
  const Slices n = slices_of(a);
  for (int b = 0; b < a.B; b += n.seqs)
    for (int hk = 0; hk < a.Hk; hk += n.heads) {
      const hipError_t e = run(slice(a, n, b, hk), stream);
      if (e != hipSuccess) return e;
    }
  return hipSuccess;
}

}  // namespace s5
