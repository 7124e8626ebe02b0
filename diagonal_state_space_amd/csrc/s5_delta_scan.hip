// Second kernel of the chunked gated delta rule: the chunks of a sequence one
// after the other, the state in registers.
//
// Columns of the state are independent, so each wave owns 16 columns of one
// head's state (as accumulator tiles) and needs nothing from the others: per
// chunk, with the fragments of T and P of the first kernel,
//   X = K S,  O = Q S,  R = beta (V - from X),  U = T R,
//   y = scale from O + P U,  S <- whole S + K^T (to U).
// Every result is the next product's operand as it lies in the accumulators
// (the fragments' product order is that of two tiles), so the chain runs
// without an exchange or a barrier. What the waves share - k, its transpose,
// q, T and P of the chunk - is staged in LDS once for the workgroup, by waves
// that do nothing else, a chunk ahead.
// All products are exact to float32 (three bf16 parts), those that lead to a y of
// bf16 io alone too: its terms scale from Q S and P U can be far larger than y
// (where a key is written over, y is what is left of them), and with two parts
// a y 4096 times smaller than its terms had two digits. The third part costs 7 %
// of 8 ragged sequences of 2048 steps, 16 heads of 128 x 128 (172 -> 183 us).
//
// What bounds it: the chain itself, with one wave on a SIMD (the LDS has room for
// one workgroup on a compute unit). Of 7900 cycles for a chunk of 64 steps (128 x
// 128 bf16, outputs) matrix instructions take 4000, and vector instructions, four
// cycles each and most of them splits into parts, 3000; neither can start
// before the other's results. 64 heads of 2048 steps: outputs 119 us, states and
// U for the gradients 91; 128 heads (ragged): 131.
//
// A value that is not finite must not reach earlier steps through a zero of T
// or P: rows from the first such one on are taken out of R for this column and
// set to NaN in the results, the state's column too.
#include "s5_delta_tile.h"

namespace s5 {

using namespace delta;

namespace {

constexpr float kNaN = __builtin_nanf("");

// What a pass of the chunks is for: y and the last state; the states at the
// chunks' starts and U for the backward pass; a segment's state from zero and
// its transition (run on the columns of the identity without values), in the
// workspace layout of the forward or the backward call.
enum Pass { kOut, kKeep, kSum, kSumBack };

// LDS of a chunk: fragments of k (by rows, by columns) and q, T, P and the
// decays (without y: no q and P); two of them where they fit, the next chunk on
// its way while one is worked on.
template <bool BF16, int KP, Pass PASS>
struct Scan : Shape<BF16, KP> {
  using Z = Shape<BF16, KP>;
  static constexpr bool kBack = PASS == kKeep || PASS == kSumBack, kY = PASS == kOut;
  static constexpr int kRecT = tri_frags<Z::C>() * 3 * kFrag;
  static constexpr int kRec = kY ? Record<Z::C>::bytes(false) : kRecT + kFrag;
  // q once where two of all do not fit (128 features): the next one replaces it
  // when it is read, in the middle of a chunk. With one buffer for all, 90 heads of
  // up to 4178 steps in float32 took 623 us instead of 443.
  static constexpr bool kOneQ = kY && 2 * (3 * Z::kMat + kRec) > kMaxLds;
  static constexpr int kFrags = (kY && !kOneQ ? 3 : 2) * Z::kMat;
  static constexpr int kBuf = kFrags + kRec, kOnce = kOneQ ? Z::kMat : 0;
  static constexpr bool kTwo = 2 * kBuf + kOnce <= kMaxLds;
  static constexpr int kLds = (kTwo ? 2 : 1) * kBuf + kOnce;
  static constexpr int oQ = kOneQ ? (kTwo ? 2 : 1) * kBuf : 2 * Z::kMat;   // in the buffer, if not once
};

template <bool BF16, int KP, int NW, Pass PASS>
__global__ void __launch_bounds__(64 * (NW + kCopy)) k_delta_scan(DeltaArgs a, int chunks, int groups, DeltaSegs segs, DeltaKeep keep) {
  using Z = Scan<BF16, KP, PASS>;
  constexpr int C = Z::C, NI = Z::NI, KS = Z::KS, MT = Z::MT, CS = Z::CS, KT = Z::KT, es = Z::es;
  constexpr bool SUM = PASS == kSum || PASS == kSumBack, KEEP = PASS == kKeep, Y = PASS == kOut;
  extern __shared__ __align__(16) unsigned char smem[];
  const int tid = threadIdx.x, l = tid & 63, g = l >> 4, m = l & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  // workgroups go round the eight dies one by one: the column groups of a
  // segment follow each other on one die, whose L2 then holds what they share
  const int count = SUM ? segs.count - 1 : segs.count;
  const int turn = blockIdx.x >> 3, cg = turn % groups, unit = turn / groups * 8 + (blockIdx.x & 7);
  const int bh = unit / count, seg = unit - bh * count;
  if (bh >= a.B * a.Hv) return;
  const int b = bh / a.Hv, h = bh - b * a.Hv, hk = h / (a.Hv / a.Hk);
  const int wg = cg * NW + w, col = wg * 16 + m;
  const bool wave_live = wg * 16 < (SUM ? segs.ld() : a.Dv), live = col < a.Dv;
  const int len = length_of(a, b);
  const int nc = (len + C - 1) / C;
  const int n0 = seg * segs.chunks, n1 = min(nc, n0 + segs.chunks);
  if (seg > 0 && n0 >= nc) return;
  if (SUM && n0 + segs.chunks >= nc) return;    // no segment follows

  if (w >= NW) {   // the copying waves
    const int id = tid - 64 * NW;
    const bool vec = vectored(a, BF16);
    Stage<BF16, KP, 64 * kCopy> k, q;
    auto load = [&](int n) {
      const int64_t tok = static_cast<int64_t>(b) * a.L + n * C;
      if constexpr (BF16) k.load(a, a.k, a.ldk, tok, min(len - n * C, C), hk, id, vec);
    };
    auto load_q = [&](int n) {
      const int64_t tok = static_cast<int64_t>(b) * a.L + n * C;
      if constexpr (BF16 && Y) q.load(a, a.q, a.ldq, tok, min(len - n * C, C), hk, id, vec);
    };
    auto copy = [&](int n) {
      unsigned char* dst = smem + (Z::kTwo ? (n & 1) * Z::kBuf : 0);
      const unsigned char* rec = a.recs + (static_cast<int64_t>(bh) * chunks + n) * Record<C>::bytes(Z::kBack);
      if constexpr (BF16) {
        k.store(dst, dst + Z::kMat, id);
      } else {
        const unsigned char* fr = a.frags + (static_cast<int64_t>(b * a.Hk + hk) * chunks + n) * Z::frags(Z::kBack);
        lds_copy<kCopy>(dst, fr + Z::k_rows(Z::kBack), Z::kMat, w - NW);
        lds_copy<kCopy>(dst + Z::kMat, fr, Z::kMat, w - NW);
      }
      if constexpr (Y) {
        lds_copy<kCopy>(dst + Z::kFrags, rec, Z::kRec, w - NW);
      } else {
        lds_copy<kCopy>(dst + Z::kFrags, rec + Record<C>::T, Z::kRecT, w - NW);
        lds_copy<kCopy>(dst + Z::kFrags + Z::kRecT, rec + Record<C>::decays(Z::kBack), kFrag, w - NW);
      }
    };
    auto copy_q = [&](int n) {
      unsigned char* dst = smem + (Z::kTwo && !Z::kOneQ ? (n & 1) * Z::kBuf : 0) + Z::oQ;
      if constexpr (BF16 && Y) {
        q.store(dst, nullptr, id);
      } else if constexpr (Y) {
        const unsigned char* fr = a.frags + (static_cast<int64_t>(b * a.Hk + hk) * chunks + n) * Z::frags(Z::kBack);
        lds_copy<kCopy>(dst, fr + Z::q_rows(Z::kBack), Z::kMat, w - NW);
      }
    };
    static_assert(!Z::kOneQ || Z::kTwo);
    if (n0 < n1) {
      load(n0);
      load_q(n0);
    }
    if (Z::kTwo && n0 < n1) {
      copy(n0);
      copy_q(n0);
      if (n0 + 1 < n1) {
        load(n0 + 1);
        load_q(n0 + 1);
      }
    }
    for (int n = n0; n < n1; ++n) {
      if constexpr (Z::kTwo) {
        barrier_copied();
        if (n + 1 < n1) copy(n + 1);
        if (!Z::kOneQ && n + 1 < n1) copy_q(n + 1);
        if (n + 2 < n1) load(n + 2);
        if constexpr (Z::kOneQ) {
          barrier_passed();   // q is read; the copies need not be there yet
          if (n + 1 < n1) copy_q(n + 1);
        }
        if (n + 2 < n1) load_q(n + 2);
      } else {
        barrier_copied();
        copy(n);
        copy_q(n);
        barrier_copied();
        if (n + 1 < n1) {
          load(n + 1);
          load_q(n + 1);
        }
      }
    }
    return;
  }

  f32x4 S[KT];
  {
    // the start: the call's, the end of the segment before, or (a segment's
    // sums) zero and the identity. Of several segments the first one's is the
    // join's copy behind the others: the last segment may have overwritten s0.
    const bool given = nc <= segs.chunks;
    const int ld = (given ? a.Dv : segs.ld()) * 4;
    const Buf p = given ? rows_buf(a.s0 + static_cast<int64_t>(bh) * a.Dk * a.Dv, a.s0 != nullptr ? a.Dk : 0, ld, ld)
                        : rows_buf(segs.p + segs.at(bh, seg > 0 ? seg - 1 : segs.count - 1), segs.dkp, ld, ld);
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * t + 4 * g + r;
        if constexpr (SUM) S[t][r] = row + segs.dvp == col ? 1.0f : 0.0f;
        else S[t][r] = __uint_as_float(load_raw<false>(p, live ? row * ld + col * 4 : kNowhere));
      }
#pragma unroll
    for (int t = 0; t < KT; ++t) asm volatile("" : "+v"(S[t]));   // waited for here, not in every chunk
  }

  uint32_t vb[MT][4];
  const int ldv = row_bytes(a.ldv, es), ldy = a.Nv * a.Dv * es;
  // byte of the first of this lane's elements in rows of `ld` bytes: bf16's y pass
  // has no register to keep it in, and one that is spilled is waited for with the
  // stores
  const int vo = live ? 4 * g * ldv + col * es : kNowhere, yo = live ? 4 * g * ldy + col * es : kNowhere;
  auto place = [&](int kept, int ld) {
    if constexpr (!BF16 || !Y) return here(kept);
    const int i = here(l), c = 16 * wg + (i & 15);
    return c < a.Dv ? 4 * (i >> 4) * ld + c * es : kNowhere;
  };
  auto fetch = [&](int n) {
    const int64_t tok = static_cast<int64_t>(b) * a.L + n * C;
    const int o = place(vo, ldv);
    const Buf vr = rows_buf(static_cast<const char*>(a.v) + (tok * a.ldv + static_cast<int64_t>(h) * a.Dv) * es, min(len - n * C, C),
                            ldv, a.Dv * es);
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) vb[t][r] = load_raw<BF16>(vr, o + (16 * t + r) * ldv);
  };

  if (n0 < n1) fetch(n0);
  if constexpr (Y && BF16) {
    // Stores of nothing, as many as a chunk's of y: the compiler then counts that
    // a chunk's v may be waited for without the stores of the chunk before, which
    // were issued after its loads.
    stage_end();
    const Buf none = rows_buf(a.y, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) store_el2<BF16>(none, here(kNowhere), 4, 0.0f, 0.0f);
    stage_end();
  }
  for (int n = n0; n < n1; ++n) {
    if constexpr (!Z::kTwo) barrier_read();   // the previous chunk is read
    barrier_read();                           // the chunk is there, the previous one read
    if (!wave_live) {
      if constexpr (Z::kOneQ) barrier_read();
      continue;
    }

    const unsigned char* s_k = smem + (Z::kTwo ? (n & 1) * Z::kBuf : 0);
    const unsigned char *s_kt = s_k + Z::kMat, *s_q = Z::kOneQ ? smem + Z::oQ : s_k + Z::oQ, *rec = s_k + Z::kFrags;
    const float* dec = reinterpret_cast<const float*>(rec + Z::kRec - kFrag);
    if constexpr (KEEP) {
      const int o = here(16 * l);
      const Buf p = rows_buf(keep.p + (static_cast<int64_t>(bh) * chunks + n) * keep.size(C) + 16 * wg * keep.dkp, 1, 0, keep.dkp * 64);
#pragma unroll
      for (int t = 0; t < KT; ++t) store16(p, o + t * 1024, S[t]);
    }
    // X = K S, R over it and U = T R are the chain; what is not (O = Q S) and the
    // splitting of the next operand go between, into the gaps of its stages
    f32x4 X[MT], O[MT], U[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) X[t] = O[t] = U[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    Frag<NI> kx[2][MT], qx[KS / 2][MT];
    Frag<3> tf[CS][MT], sf[2];
    Frag<3> so[KS / 2];
    auto read_k = [&](int ks) {
#pragma unroll
      for (int t = 0; t < MT; ++t) kx[ks & 1][t] = read_rows<NI, KS>(s_k, t, ks);
    };
    auto read_q = [&](int half) {
      if constexpr (Y) {
#pragma unroll
        for (int i = 0; i < KS / 2; ++i)
#pragma unroll
          for (int t = 0; t < MT; ++t) qx[i][t] = read_rows<NI, KS>(s_q, t, half * (KS / 2) + i);
      }
    };
    auto mma_q = [&](int half) {
      if constexpr (Y) {
#pragma unroll
        for (int i = 0; i < KS / 2; ++i) mma(O, qx[i], so[i]);
      }
    };
    read_k(0);
    sf[0] = to_frag<3>(S[0], S[1]);
    stage_end();
    float4 from[MT], beta[MT];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      if (ks + 1 < KS) {
        read_k(ks + 1);
      } else {
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          from[t] = *reinterpret_cast<const float4*>(dec + 16 * t + 4 * g);
          beta[t] = *reinterpret_cast<const float4*>(dec + 2 * C + 16 * t + 4 * g);
        }
        read_q(0);
      }
      stage_end();
      mma(X, kx[ks & 1], sf[ks & 1]);
      if (ks + 1 < KS) sf[(ks + 1) & 1] = to_frag<3>(S[2 * ks + 2], S[2 * ks + 3]);
      if (Y && ks < KS / 2) so[ks] = sf[ks & 1];
      stage_end();
    }
    read_tri<false, C>(tf[0], rec + Record<C>::T, 0);
    stage_end();
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const float ff[4] = {from[t].x, from[t].y, from[t].z, from[t].w}, bb[4] = {beta[t].x, beta[t].y, beta[t].z, beta[t].w};
#pragma unroll
      for (int r = 0; r < 4; ++r) X[t][r] = bb[r] * (value<BF16>(vb[t][r]) - ff[r] * X[t][r]);
    }
    mma_q(0);
    Frag<3> xf[CS];
    xf[0] = to_frag<3>(X[0], X[1]);
    stage_end();
    const float whole = dec[C - 1];
    float4 to[MT];
#pragma unroll
    for (int ks = 0; ks < CS; ++ks) {
      if (ks + 1 < CS) {
        read_tri<false, C>(tf[ks + 1], rec + Record<C>::T, ks + 1);
      } else {
        read_q(1);
#pragma unroll
        for (int t = 0; t < MT; ++t) to[t] = *reinterpret_cast<const float4*>(dec + C + 16 * t + 4 * g);
      }
      stage_end();
      mma_tri<false, C>(U, tf[ks], ks, xf[ks]);
      if (ks + 1 < CS) xf[ks + 1] = to_frag<3>(X[2 * ks + 2], X[2 * ks + 3]);
      if (Y && ks == 0) {
#pragma unroll
        for (int i = 0; i < KS / 2; ++i) so[i] = to_frag<3>(S[KS + 2 * i], S[KS + 2 * i + 1]);
      }
      if (ks == CS - 1) {
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) S[t][r] *= whole;
      }
      stage_end();
    }
    if (n + 1 < n1) fetch(n + 1);
    if constexpr (Z::kOneQ) barrier_read();   // q is read
    int first = C;   // first row that is not finite, of this lane's column
    // (the last tile's rows have all of R: a zero of T times NaN is NaN)
    if (__any(!(fabsf(U[MT - 1][0]) < INFINITY))) {
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (!(fabsf(X[t][r]) < INFINITY)) first = min(first, 16 * t + 4 * g + r);
      first = min(first, __shfl_xor(first, 16));
      first = min(first, __shfl_xor(first, 32));
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        U[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (16 * t + 4 * g + r >= first) X[t][r] = 0.0f;
      }
#pragma unroll
      for (int ks = 0; ks < CS; ++ks) {
        read_tri<false, C>(tf[ks], rec + Record<C>::T, ks);
        mma_tri<false, C>(U, tf[ks], ks, to_frag<3>(X[2 * ks], X[2 * ks + 1]));
      }
    }
    const int64_t tok = static_cast<int64_t>(b) * a.L + n * C;
    if constexpr (KEEP) {
      const int o = here(16 * l);
      const Buf p = rows_buf(keep.p + (static_cast<int64_t>(bh) * chunks + n) * keep.size(C) + keep.at_u() + 16 * wg * C, 1, 0, C * 64);
      if (first < C) {
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (16 * t + 4 * g + r >= first) U[t][r] = kNaN;
      }
#pragma unroll
      for (int t = 0; t < MT; ++t) store16(p, o + t * 1024, U[t]);
    }
    // S <- whole S + K^T (to U), and O <- scale from O + P U beside it
    constexpr int kGroups = CS * KT / 4;
    // the 32-steps of P: read in one of these groups (-1: before them), multiplied
    // in the next one (float32 with 64 features: the only one)
    auto read_at = [](int ks) { return CS == 1 ? 0 : kGroups >= 4 ? ks : ks - 1; };
    auto mma_at = [&](int ks) { return kGroups > 1 ? read_at(ks) + 1 : 0; };
    Frag<NI> cf[2][4];
    Frag<3> pf[CS][MT], ub[CS];
    auto read_p = [&](int i) {
      if constexpr (Y) {
#pragma unroll
        for (int ks = 0; ks < CS; ++ks)
          if (i == read_at(ks)) read_tri<false, C>(pf[ks], rec + Record<C>::P, ks);
      }
    };
    read_cols4<NI, C>(cf[0], s_kt, 0, 0);
    read_p(-1);
    stage_end();
    mma_q(1);
    Frag<3> uf[CS];
#pragma unroll
    for (int ks = 0; ks < CS; ++ks) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float4 f = to[2 * ks + (e >> 2)];
        x[e] = U[2 * ks + (e >> 2)][e & 3] * ((e & 3) == 0 ? f.x : (e & 3) == 1 ? f.y : (e & 3) == 2 ? f.z : f.w);
      }
      uf[ks] = to_frag<3>(x);
    }
    stage_end();
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      if (i + 1 < kGroups) read_cols4<NI, C>(cf[(i + 1) & 1], s_kt, 4 * ((i + 1) % (KT / 4)), (i + 1) / (KT / 4));
      read_p(i);
      if (Y && i == 0) {
#pragma unroll
        for (int t = 0; t < MT; ++t) from[t] = *reinterpret_cast<const float4*>(dec + 3 * C + 16 * t + 4 * g);
      }
      stage_end();
      mma_cols4(S, 4 * (i % (KT / 4)), cf[i & 1], uf[i / (KT / 4)]);
      if constexpr (Y) {
        if (i == 0) {
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            const float ff[4] = {from[t].x, from[t].y, from[t].z, from[t].w};
#pragma unroll
            for (int r = 0; r < 4; ++r) O[t][r] *= ff[r];
          }
#pragma unroll
          for (int ks = 0; ks < CS; ++ks) ub[ks] = to_frag<3>(U[2 * ks], U[2 * ks + 1]);
        }
#pragma unroll
        for (int ks = 0; ks < CS; ++ks)
          if (i == mma_at(ks)) mma_tri<false, C>(O, pf[ks], ks, ub[ks]);
        if (i == kGroups - 1) {
          if (first < C) {
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
              for (int r = 0; r < 4; ++r)
                if (16 * t + 4 * g + r >= first) O[t][r] = kNaN;
          }
          const int o = place(yo, ldy);
          const Buf yr = rows_buf(static_cast<char*>(a.y) + (tok * a.Nv + h) * a.Dv * es, min(len - n * C, C), ldy, a.Dv * es);
#pragma unroll
          for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int r = 0; r < 4; r += 2) store_el2<BF16>(yr, o + (16 * t + r) * ldy, ldy, O[t][r], O[t][r + 1]);
        }
      }
      stage_end();
    }
    if (first < C) {
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[t][r] = kNaN;
    }
  }

  if constexpr (SUM) {
    if (!wave_live) return;
    const Buf p = rows_buf(segs.p + segs.at(bh, seg), segs.dkp, segs.ld() * 4, segs.ld() * 4);
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) store_el<false>(p, ((16 * t + 4 * g + r) * segs.ld() + col) * 4, S[t][r]);
  } else if (Y && a.s_last != nullptr && n0 + segs.chunks >= nc) {
    const Buf p = rows_buf(a.s_last + static_cast<int64_t>(bh) * a.Dk * a.Dv, a.Dk, a.Dv * 4, a.Dv * 4);
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) store_el<false>(p, live ? ((16 * t + 4 * g + r) * a.Dv + col) * 4 : kNowhere, S[t][r]);
  }
}

// Joins the segments: with the states B and transitions M of their sums, the
// state at the end of segment s is M_s S + B_s (forward, written over B_s; the
// start is copied to the last segment's place, which has no sums), the
// gradient at its start M_s^T D + B_s (backward). A workgroup has 16 columns of
// a head, a wave the row tiles w, w + 4; the next segment's M and B are on
// their way while one is multiplied (float32 matrix instructions).
template <int KT, bool BACK>
__global__ void __launch_bounds__(256) k_delta_join(DeltaArgs a, DeltaSegs segs, int C) {
  constexpr int LD = 17, DT = KT / 4;
  __shared__ float s_x[16 * KT * LD];
  const int tid = threadIdx.x, l = tid & 63, g = l >> 4, m = l & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  // a head's workgroups on one die: they read the same transitions
  const int tiles = segs.dvp / 16, turn = blockIdx.x >> 3, bh = turn / tiles * 8 + (blockIdx.x & 7), col0 = turn % tiles * 16, col = col0 + m;
  if (bh >= a.B * a.Hv) return;
  const int nc = (length_of(a, bh / a.Hv) + C - 1) / C;
  const int last = nc > 0 ? (nc - 1) / segs.chunks : 0;   // the last segment there is
  const int ld = segs.ld() * 4, ldb = BACK ? segs.dvp * 4 : ld;
  // segments to join: forward 0 .. last - 1, backward last - 1 .. 1
  const int from = BACK ? last - 1 : 0, to = BACK ? 0 : last, step = BACK ? -1 : 1;
  if (BACK ? from <= to : from >= to) return;

  struct Segment {
    float4 A[DT][KT];
    float B[DT][4];
  };
  auto fetch = [&](Segment& x, int s) {
    const Buf mat = rows_buf(segs.p + segs.at(bh, s), segs.dkp, ld, ld);
    const Buf vec = BACK ? rows_buf(segs.back + segs.at_back(bh, s), segs.dkp, ldb, ldb) : mat;
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      const int t = w + 4 * d;
#pragma unroll
      for (int k = 0; k < KT; ++k) {
        const bool in = 16 * t < segs.dkp && 16 * k < segs.dkp;
        if constexpr (BACK) {
          const int o = (16 * k + 4 * g) * ld + (segs.dvp + 16 * t + m) * 4;
          x.A[d][k] = float4{__uint_as_float(load_raw<false>(mat, in ? o : kNowhere)), __uint_as_float(load_raw<false>(mat, in ? o + ld : kNowhere)),
                             __uint_as_float(load_raw<false>(mat, in ? o + 2 * ld : kNowhere)), __uint_as_float(load_raw<false>(mat, in ? o + 3 * ld : kNowhere))};
        } else {
          const uint4 v = load16(mat, in ? (16 * t + m) * ld + (segs.dvp + 16 * k + 4 * g) * 4 : kNowhere);
          x.A[d][k] = float4{__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w)};
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) x.B[d][r] = __uint_as_float(load_raw<false>(vec, (16 * t + 4 * g + r) * ldb + col * 4));
    }
  };

  Segment even, odd;
  fetch(even, from);
  if (from + step != to) fetch(odd, from + step);
  {
    // the first segment's start (backward: the gradient that its sums ended with)
    const int lds = BACK ? ldb : a.Dv * 4;
    const Buf p = BACK ? rows_buf(segs.back + segs.at_back(bh, last), segs.dkp, lds, lds)
                       : rows_buf(a.s0 + static_cast<int64_t>(bh) * a.Dk * a.Dv, a.s0 != nullptr ? a.Dk : 0, lds, lds);
    const Buf copy = rows_buf(segs.p + segs.at(bh, segs.count - 1), segs.dkp, ld, ld);
    const int c0 = col0 + (tid & 15);
    float x[KT];   // all under way before the first is waited for
#pragma unroll
    for (int i = 0; i < KT; ++i)
      x[i] = __uint_as_float(load_raw<false>(p, BACK || c0 < a.Dv ? (16 * i + (tid >> 4)) * lds + c0 * 4 : kNowhere));
#pragma unroll
    for (int i = 0; i < KT; ++i) {
      const int row = 16 * i + (tid >> 4);
      s_x[row * LD + (tid & 15)] = x[i];
      if constexpr (!BACK) store_el<false>(copy, row * ld + c0 * 4, x[i]);
    }
  }
  auto join = [&](Segment& x, int s) {
    __syncthreads();
    f32x4 acc[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[d][r] = x.B[d][r];
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      const float* v = s_x + (16 * k + 4 * g) * LD + m;
      const float vv[4] = {v[0], v[LD], v[2 * LD], v[3 * LD]};
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int d = 0; d < DT; ++d)
          acc[d] = __builtin_amdgcn_mfma_f32_16x16x4f32(r == 0 ? x.A[d][k].x : r == 1 ? x.A[d][k].y : r == 2 ? x.A[d][k].z : x.A[d][k].w, vv[r], acc[d], 0, 0, 0);
    }
    if ((to - s) * step > 2) fetch(x, s + 2 * step);
    __syncthreads();
    const Buf out = BACK ? rows_buf(segs.back + segs.at_back(bh, s), segs.dkp, ldb, ldb) : rows_buf(segs.p + segs.at(bh, s), segs.dkp, ld, ld);
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * (w + 4 * d) + 4 * g + r;
        s_x[row * LD + m] = acc[d][r];
        store_el<false>(out, row * ldb + col * 4, acc[d][r]);
      }
  };
  for (int s = from; s != to;) {
    join(even, s);
    s += step;
    if (s == to) break;
    join(odd, s);
    s += step;
  }
}

template <bool BF16, int KP, int NW, Pass PASS>
hipError_t run(const DeltaArgs& a, const DeltaSegs& segs, const DeltaKeep& keep, hipStream_t stream) {
  using Z = Scan<BF16, KP, PASS>;
  constexpr bool SUM = PASS == kSum || PASS == kSumBack;
  constexpr auto* kern = k_delta_scan<BF16, KP, NW, PASS>;
  if (const hipError_t e = allow_lds<kern>(Z::kLds); e != hipSuccess) return e;
  const int chunks = (a.L + Z::C - 1) / Z::C;
  const int groups = ((SUM ? segs.ld() : a.Dv) + 16 * NW - 1) / (16 * NW);
  const int64_t blocks = (static_cast<int64_t>(a.B) * a.Hv * (SUM ? segs.count - 1 : segs.count) + 7) / 8 * 8 * groups;
  kern<<<dim3(static_cast<unsigned>(blocks)), dim3(64 * (NW + kCopy)), Z::kLds, stream>>>(a, chunks, groups, segs, keep);
  return hipGetLastError();
}

template <Pass PASS>
hipError_t dispatch(const DeltaArgs& a, const DeltaSegs& segs, const DeltaKeep& keep, hipStream_t stream) {
  constexpr bool SUM = PASS == kSum || PASS == kSumBack;
  if (narrow_groups(static_cast<int64_t>(a.B) * a.Hv * (SUM ? segs.count - 1 : segs.count), SUM ? segs.ld() : segs.dvp)) {
    if (a.bf16_io) return a.Dk > 64 ? run<true, 128, 2, PASS>(a, segs, keep, stream) : run<true, 64, 2, PASS>(a, segs, keep, stream);
    return a.Dk > 64 ? run<false, 128, 2, PASS>(a, segs, keep, stream) : run<false, 64, 2, PASS>(a, segs, keep, stream);
  }
  if (a.bf16_io) return a.Dk > 64 ? run<true, 128, 4, PASS>(a, segs, keep, stream) : run<true, 64, 4, PASS>(a, segs, keep, stream);
  return a.Dk > 64 ? run<false, 128, 4, PASS>(a, segs, keep, stream) : run<false, 64, 4, PASS>(a, segs, keep, stream);
}

template <bool BACK>
hipError_t join(const DeltaArgs& a, const DeltaSegs& segs, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(a.B) * a.Hv + 7) / 8 * 8 * (segs.dvp / 16)));
  const int C = a.bf16_io ? chunk_of<true>() : chunk_of<false>();
  if (a.Dk > 64) k_delta_join<8, BACK><<<grid, dim3(256), 0, stream>>>(a, segs, C);
  else k_delta_join<4, BACK><<<grid, dim3(256), 0, stream>>>(a, segs, C);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_scan(const DeltaArgs& a, const DeltaSegs& segs, const DeltaKeep* keep, hipStream_t stream) {
  const DeltaKeep none{};
  if (segs.count > 1) {
    hipError_t e = keep != nullptr ? dispatch<kSumBack>(a, segs, none, stream) : dispatch<kSum>(a, segs, none, stream);
    if (e == hipSuccess) e = join<false>(a, segs, stream);
    if (e != hipSuccess) return e;
  }
  return keep != nullptr ? dispatch<kKeep>(a, segs, *keep, stream) : dispatch<kOut>(a, segs, none, stream);
}

hipError_t launch_delta_join_back(const DeltaArgs& a, const DeltaSegs& segs, hipStream_t stream) {
  return join<true>(a, segs, stream);
}

hipError_t launch_delta(const DeltaArgs& args, hipStream_t stream) {
  DeltaArgs a = args;
  DeltaSegs segs{};
  delta_work(a, segs, false);
  if (a.L > 0) {
    const hipError_t e = launch_delta_prep(a, false, stream);
    if (e != hipSuccess) return e;
  }
  return launch_delta_scan(a, segs, nullptr, stream);
}

}  // namespace s5
