// Second kernel of the chunked gated delta rule: the chunks of a sequence one
// after the other, the state in registers.
//
// Columns of the state are independent, so each wave owns 16 columns of one
// head's state (as accumulator tiles) and needs nothing from the others: per
// chunk, with the fragments of T and P of the first kernel,
//   X = K S,  O = Q S,  R = beta (V - from X),  U = T R,
//   y = scale (from O + P U),  S <- whole S + K^T (to U).
// Every result is the next product's operand as it lies in the accumulators
// (the fragments' product order is that of two tiles), so the chain runs
// without an exchange or a barrier. What the waves share - k, its transpose,
// q, T and P of the chunk - is staged in LDS once for the workgroup, fetched
// into registers one chunk ahead.
// The state's chain is exact to float32 (three bf16 parts); what only reaches
// y of bf16 io takes two parts.
//
// A value that is not finite must not reach earlier steps through a zero of T
// or P: rows from the first such one on are taken out of R for this column and
// set to NaN in the results, the state's column too.
#include "s5_delta_tile.h"

namespace s5 {

using namespace delta;

namespace {

constexpr float kNaN = __builtin_nanf("");

// One more wave copies the chunks. LDS of a chunk: fragments of k (by rows, by columns) and q, T, P and the
// decays (KEEP: without q and P); two of them where they fit, the next chunk
// on its way while one is worked on.
template <bool BF16, int KP, bool KEEP>
struct Scan : Shape<BF16, KP> {
  using Z = Shape<BF16, KP>;
  static constexpr int kFrags = (KEEP ? 2 : 3) * Z::kMat;
  static constexpr int kRecT = tri_frags<Z::C>() * 3 * kFrag;
  static constexpr int kRec = KEEP ? kRecT + kFrag : Record<Z::C>::bytes(false, Z::NO);
  static constexpr int kBuf = kFrags + kRec;
  static constexpr bool kTwo = 2 * kBuf <= kMaxLds;
  static constexpr int kLds = (kTwo ? 2 : 1) * kBuf;
};

// KEEP: no outputs; the states at the chunks' starts and U are stored for the
// backward pass
template <bool BF16, int KP, int NW, bool KEEP>
__global__ void __launch_bounds__(64 * (NW + 1)) k_delta_scan(DeltaArgs a, int chunks, int groups, DeltaKeep keep) {
  using Z = Scan<BF16, KP, KEEP>;
  constexpr int C = Z::C, NI = Z::NI, NO = Z::NO, KS = Z::KS, MT = Z::MT, CS = Z::CS, KT = Z::KT, es = Z::es;
  extern __shared__ __align__(16) unsigned char smem[];
  const int tid = threadIdx.x, l = tid & 63, g = l >> 4, m = l & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  // workgroups go round the eight dies one by one: the column groups of a head
  // follow each other on one die, whose L2 then holds what they share
  const int die = blockIdx.x & 7, turn = blockIdx.x >> 3;
  const int bh = (turn / groups) * 8 + die, cg = turn % groups;
  if (bh >= a.B * a.Hv) return;
  const int b = bh / a.Hv, h = bh - b * a.Hv, hk = h / (a.Hv / a.Hk);
  const int col = (cg * NW + w) * 16 + m;
  const bool wave_live = (cg * NW + w) * 16 < a.Dv, live = col < a.Dv;
  const int len = length_of(a, b);
  const int nc = (len + C - 1) / C;

  if (w == NW) {   // the copying wave
    auto copy = [&](int n) {
      unsigned char* dst = smem + (Z::kTwo ? (n & 1) * Z::kBuf : 0);
      const unsigned char* rec = a.recs + (static_cast<int64_t>(bh) * chunks + n) * Record<C>::bytes(KEEP, NO);
      lds_copy<1>(dst, a.frags + (static_cast<int64_t>(b * a.Hk + hk) * chunks + n) * Z::frags(KEEP), Z::kFrags, 0);
      if constexpr (KEEP) {
        lds_copy<1>(dst + Z::kFrags, rec + Record<C>::T, Z::kRecT, 0);
        lds_copy<1>(dst + Z::kFrags + Z::kRecT, rec + Record<C>::decays(true, 3), kFrag, 0);
      } else {
        lds_copy<1>(dst + Z::kFrags, rec, Z::kRec, 0);
      }
    };
    if (Z::kTwo && nc > 0) copy(0);
    for (int n = 0; n < nc; ++n) {
      if constexpr (!Z::kTwo) {
        barrier_copied();
        copy(n);
      }
      barrier_copied();
      if (Z::kTwo && n + 1 < nc) copy(n + 1);
    }
    return;
  }

  f32x4 S[KT];
#pragma unroll
  for (int t = 0; t < KT; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * t + 4 * g + r;
      S[t][r] = a.s0 != nullptr && live && row < a.Dk ? a.s0[(static_cast<int64_t>(bh) * a.Dk + row) * a.Dv + col] : 0.0f;
    }

  uint32_t vb[MT][4];
  const int ldv = static_cast<int>(a.ldv) * es, ldy = a.Hv * a.Dv * es;
  const int vo = live ? 4 * g * ldv + col * es : kNowhere, yo = live ? 4 * g * ldy + col * es : kNowhere;
  const int ko = (4 * g * keep.dvp + col) * 4;   // rows behind the kept ones are outside their buffer
  auto fetch = [&](int n) {
    const int64_t tok = static_cast<int64_t>(b) * a.L + n * C;
    const Buf vr = rows_buf(static_cast<const char*>(a.v) + (tok * a.ldv + static_cast<int64_t>(h) * a.Dv) * es, min(len - n * C, C),
                            ldv, a.Dv * es);
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) vb[t][r] = load_raw<BF16>(vr, vo + (16 * t + r) * ldv);
  };

  if (nc > 0) fetch(0);
  for (int n = 0; n < nc; ++n) {
    if constexpr (!Z::kTwo) barrier_read();   // the previous chunk is read
    barrier_read();                           // the chunk is there, the previous one read
    if (!wave_live) continue;
    float V[MT][4];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) V[t][r] = value<BF16>(vb[t][r]);
    if (n + 1 < nc) fetch(n + 1);

    const unsigned char* s_k = smem + (Z::kTwo ? (n & 1) * Z::kBuf : 0);
    const unsigned char *s_kt = s_k + Z::kMat, *s_q = s_k + 2 * Z::kMat, *rec = s_k + Z::kFrags;
    const float* dec = reinterpret_cast<const float*>(rec + Z::kRec - kFrag);
    if constexpr (KEEP) {
      const Buf p = rows_buf(keep.p + (static_cast<int64_t>(bh) * chunks + n) * keep.size(C), keep.dkp, keep.dvp * 4, keep.dvp * 4);
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) store_el<false>(p, ko + (16 * t + r) * keep.dvp * 4, S[t][r]);
    }
    f32x4 X[MT], O[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) X[t] = O[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      Frag<NI> kf[MT];
#pragma unroll
      for (int t = 0; t < MT; ++t) kf[t] = read_rows<NI, KS>(s_k, t, ks);
      mma(X, kf, to_frag<3>(S[2 * ks], S[2 * ks + 1]));
      if constexpr (!KEEP) {
        Frag<NI> qf[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t) qf[t] = read_rows<NI, KS>(s_q, t, ks);
        mma(O, qf, to_frag<NO>(S[2 * ks], S[2 * ks + 1]));
      }
    }
    float from[MT][4];
    float odd = 0.0f;   // NaN if anything is not finite
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const float4 f = *reinterpret_cast<const float4*>(dec + 16 * t + 4 * g);
      const float4 be = *reinterpret_cast<const float4*>(dec + 2 * C + 16 * t + 4 * g);
      const float ff[4] = {f.x, f.y, f.z, f.w}, bb[4] = {be.x, be.y, be.z, be.w};
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        from[t][r] = ff[r];
        X[t][r] = bb[r] * (V[t][r] - ff[r] * X[t][r]);
        odd = fmaf(X[t][r], 0.0f, odd);
      }
    }
    int first = reinterpret_cast<const int*>(dec)[3 * C + 1];
    if (first < C || __any(odd != odd)) {
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (!(fabsf(X[t][r]) < INFINITY)) first = min(first, 16 * t + 4 * g + r);
      first = min(first, __shfl_xor(first, 16));
      first = min(first, __shfl_xor(first, 32));
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (16 * t + 4 * g + r >= first) X[t][r] = 0.0f;
    }
    // U = T R: 32 products at a time, of the row tiles they reach
    f32x4 U[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) U[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    tri_mma<C, 3>(U, rec + Record<C>::T, X);
    const int64_t tok = static_cast<int64_t>(b) * a.L + n * C;
    if constexpr (KEEP) {
      const Buf p = rows_buf(keep.p + (static_cast<int64_t>(bh) * chunks + n) * keep.size(C) + keep.at_u(), C, keep.dvp * 4, keep.dvp * 4);
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          store_el<false>(p, ko + (16 * t + r) * keep.dvp * 4, 16 * t + 4 * g + r < first ? U[t][r] : kNaN);
    } else {
      const Buf yr = rows_buf(static_cast<char*>(a.y) + (tok * a.Hv + h) * a.Dv * es, min(len - n * C, C), ldy, a.Dv * es);
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) O[t][r] *= from[t][r];
      tri_mma<C, NO>(O, rec + Record<C>::P, U);
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int i = 16 * t + 4 * g + r;
          store_el<BF16>(yr, yo + (16 * t + r) * ldy, i < first ? a.scale * O[t][r] : kNaN);
        }
    }
    const float whole = dec[3 * C];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const float4 to = *reinterpret_cast<const float4*>(dec + C + 16 * t + 4 * g);
      const float tt[4] = {to.x, to.y, to.z, to.w};
#pragma unroll
      for (int r = 0; r < 4; ++r) U[t][r] *= tt[r];
    }
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) S[t][r] *= whole;
#pragma unroll
    for (int ks = 0; ks < CS; ++ks) cols_mma<NI, C>(S, s_kt, ks, to_frag<3>(U[2 * ks], U[2 * ks + 1]));
    if (first < C) {
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[t][r] = kNaN;
    }
  }

  if (!KEEP && a.s_last != nullptr && live) {
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * t + 4 * g + r;
        if (row < a.Dk) a.s_last[(static_cast<int64_t>(bh) * a.Dk + row) * a.Dv + col] = S[t][r];
      }
  }
}

template <bool BF16, int KP, bool KEEP>
hipError_t run(const DeltaArgs& a, const DeltaKeep& keep, hipStream_t stream) {
  constexpr int NW = 4;
  using Z = Scan<BF16, KP, KEEP>;
  auto* kern = k_delta_scan<BF16, KP, NW, KEEP>;
  static const hipError_t attr =
      hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, Z::kLds);
  if (attr != hipSuccess) return attr;
  const int chunks = (a.L + Z::C - 1) / Z::C;
  const int groups = (a.Dv + 16 * NW - 1) / (16 * NW);
  const int64_t blocks = (static_cast<int64_t>(a.B) * a.Hv + 7) / 8 * 8 * groups;
  kern<<<dim3(static_cast<unsigned>(blocks)), dim3(64 * (NW + 1)), Z::kLds, stream>>>(a, chunks, groups, keep);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_scan(const DeltaArgs& a, const DeltaKeep* keep, hipStream_t stream) {
  const bool wide = a.Dk > 64;
  if (keep != nullptr) {
    if (a.bf16_io) return wide ? run<true, 128, true>(a, *keep, stream) : run<true, 64, true>(a, *keep, stream);
    return wide ? run<false, 128, true>(a, *keep, stream) : run<false, 64, true>(a, *keep, stream);
  }
  const DeltaKeep none{};
  if (a.bf16_io) return wide ? run<true, 128, false>(a, none, stream) : run<true, 64, false>(a, none, stream);
  return wide ? run<false, 128, false>(a, none, stream) : run<false, 64, false>(a, none, stream);
}

hipError_t launch_delta(const DeltaArgs& args, hipStream_t stream) {
  DeltaArgs a = args;
  delta_work(a, false);
  if (a.L > 0) {
    const hipError_t e = launch_delta_prep(a, false, stream);
    if (e != hipSuccess) return e;
  }
  return launch_delta_scan(a, nullptr, stream);
}

}  // namespace s5
