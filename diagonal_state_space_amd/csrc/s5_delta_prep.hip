// First kernel of the chunked gated delta rule: what a chunk's steps need
// besides the state, for all chunks at once.
//
// With G_i the chunk's inclusive sums of g and M_ij = exp(G_i - G_j) (j <= i):
//   A_ij = beta_i M_ij k_i.k_j (j < i),  T = (I + A)^-1,  P_ij = scale M_ij q_i.k_j
// so that the chunk's writes are U = T beta (V - e^G K S) and its outputs
// scale e^G Q S + P U. One workgroup of four waves per chunk and value head.
//
// Both products run on the matrix cores from staged k and q; P comes out
// transposed, which is the order of its operand fragments, and is stored from
// the registers. float32 k and q are split into fragments by a kernel before
// this one. The inverse: the 16 x 16 diagonal blocks by substitution, a
// column a lane; then blocks of 32 and 64 from halves,
//   [X 0; B Y]^-1 = [X^-1 0; -Y^-1 B X^-1  Y^-1],
// by float32 matrix instructions, the second factor from the accumulators of
// the first. Substitution and halves keep the error of a triangular solve,
// which powers of A (they grow for equal keys) do not.
// The sums of g are float64: their differences stay exact to float32 however
// fast a head forgets.
//
// What bounds it: each workgroup's chain of loads, products, substitution and
// stores, of which four are on a compute unit; 128 x 128 bf16, 1 x 8192 steps of
// 16 heads: 27 us for 2048 chunks (37 KB of record each, 4.2 TB/s in and out),
// with the gradients' records (55 KB) and fragments 47 us (4 TB/s).
#include "s5_delta_tile.h"

namespace s5 {

using namespace delta;

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = 4;

__device__ __forceinline__ f32x4 mfma4(float a, float b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// float32 k and q of a chunk and key head as fragments
template <int KP, bool BACK>
__global__ void __launch_bounds__(kThreads) k_delta_frags(DeltaArgs a, int chunks) {
  using Z = Shape<false, KP>;
  constexpr int C = Z::C;
  extern __shared__ __align__(16) unsigned char smem[];
  const int tid = threadIdx.x;
  const int n = blockIdx.x % chunks, bk = blockIdx.x / chunks;
  const int b = bk / a.Hk, hk = bk - b * a.Hk;
  const int rows = min(length_of(a, b) - n * C, C);
  if (rows <= 0) return;
  const int64_t tok = static_cast<int64_t>(b) * a.L + n * C;
  const bool vec = vectored(a, false);
  Stage<false, KP, kThreads> x;
  x.load(a, a.k, a.ldk, tok, rows, hk, tid, vec);
  x.store(smem + Z::k_rows(BACK), smem, tid);
  x.load(a, a.q, a.ldq, tok, rows, hk, tid, vec);
  x.store(smem + Z::q_rows(BACK), BACK ? smem + Z::kMat : nullptr, tid);
  __syncthreads();
  uint4* dst = reinterpret_cast<uint4*>(a.frags + static_cast<int64_t>(blockIdx.x) * Z::frags(BACK));
  for (int i = tid; i < Z::frags(BACK) / 16; i += kThreads) dst[i] = reinterpret_cast<const uint4*>(smem)[i];
}

template <bool BF16, int KP, bool BACK>
__global__ void __launch_bounds__(kThreads, 4) k_delta_prep(DeltaArgs a, int chunks) {
  using Z = Shape<BF16, KP>;
  constexpr int C = Z::C, NI = Z::NI, KS = Z::KS, MT = Z::MT;
  constexpr int LD = C + 4;
  extern __shared__ __align__(16) unsigned char smem[];
  unsigned char* s_k = smem;
  unsigned char* s_q = s_k + Z::kMat;
  float *s_a = reinterpret_cast<float*>(smem), *s_t = s_a + C * LD;   // A and T, over k and q when they are read
  constexpr int kUsed = 2 * Z::kMat > 2 * C * LD * 4 ? 2 * Z::kMat : 2 * C * LD * 4;
  double* s_g = reinterpret_cast<double*>(smem + kUsed);              // sums of g
  float* s_b = reinterpret_cast<float*>(s_g + C);                     // beta
  int* s_bad = reinterpret_cast<int*>(s_b + C);

  const int tid = threadIdx.x, l = tid & 63, g = l >> 4, m = l & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = blockIdx.x % chunks, bh = blockIdx.x / chunks;
  const int b = bh / a.Hv, h = bh - b * a.Hv, hk = h / (a.Hv / a.Hk);
  const int left = length_of(a, b) - n * C;     // valid tokens from the chunk's start
  if (left <= 0) return;
  const int64_t tok = static_cast<int64_t>(b) * a.L + n * C;

  if constexpr (BF16) {
    const bool vec = vectored(a, true);
    Stage<BF16, KP, kThreads> k, q;
    k.load(a, a.k, a.ldk, tok, min(left, C), hk, tid, vec);
    q.load(a, a.q, a.ldq, tok, min(left, C), hk, tid, vec);
    // the first of the heads that share a key leaves k and q by columns for the
    // gradients
    unsigned char* cols = BACK && h == hk * (a.Hv / a.Hk)
                              ? a.frags + (static_cast<int64_t>(b * a.Hk + hk) * chunks + n) * Z::frags(BACK) : nullptr;
    k.store(s_k, cols, tid);
    q.store(s_q, cols != nullptr ? cols + Z::kMat : nullptr, tid);
  } else {
    const unsigned char* fr = a.frags + (static_cast<int64_t>(b * a.Hk + hk) * chunks + n) * Z::frags(BACK);
    lds_copy<kWaves>(s_k, fr + Z::k_rows(BACK), Z::kMat, w);
    lds_copy<kWaves>(s_q, fr + Z::q_rows(BACK), Z::kMat, w);
  }
  // sums of g (a wave's 64 lanes hold the chunk)
  if (w == 0) {
    const bool live = l < C && l < left;
    const float gi = live ? a.g[(tok + l) * a.Nv + h] : 0.0f;
    const float be = live ? a.beta[(tok + l) * a.Nv + h] : 0.0f;
    const double s = chunk_sums(gi);
    const bool bad = !(gi < INFINITY) || !(fabsf(be) < INFINITY);
    const uint64_t mask = __ballot(bad);
    if (l < C) {
      s_g[l] = s;
      s_b[l] = be;
    }
    if (l == 0) *s_bad = mask != 0 ? static_cast<int>(__ffsll(static_cast<unsigned long long>(mask))) - 1 : C;
  }
  if constexpr (!BF16) lds_copied();   // the other waves read what this one copied
  __syncthreads();

  unsigned char* rec = a.recs + static_cast<int64_t>(blockIdx.x) * Record<C>::bytes(BACK);
  // A: wave w the row tile w, in registers until k and q are read (in the same
  // LDS four workgroups fit a compute unit, not three: 62 -> 50 us for 8 ragged
  // sequences of 2048 steps, 16 heads)
  f32x4 A[MT];
  if (w < MT) {
    double gi[4];
    float bi[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      gi[r] = s_g[16 * w + 4 * g + r];
      bi[r] = s_b[16 * w + 4 * g + r];
    }
#pragma unroll
    for (int jt = 0; jt < MT; ++jt) {
      if (jt > w) continue;
      A[jt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
        A[jt] = mma(read_rows<NI, KS>(s_k, w, ks), read_rows<NI, KS>(s_k, jt, ks), A[jt]);
      const int j = 16 * jt + m;
      const double gj = s_g[j];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = 16 * w + 4 * g + r;
        // a key that is not finite, or whose length is not
        if (jt == w && i == j && !(A[jt][r] < INFINITY)) atomicMin(s_bad, i);
        const float x = bi[r] * decay_exp(gi[r] - gj) * A[jt][r];   // (formed for j >= i too, without a branch)
        A[jt][r] = j < i ? x : 0.0f;
      }
    }
  }
  // P transposed (forward: rows j in the accumulators, a lane's column is the
  // query) or as it is (backward), straight into fragments
  for (int f = w; f < tri_frags<C>(); f += kWaves) {
    // tile of the operand's rows and 32-step of its products
    int rt, ks;
    if constexpr (C == 32) { rt = f; ks = 0; }
    else if constexpr (BACK) { rt = f < 4 ? f >> 1 : f - 2; ks = f < 4 ? f & 1 : 1; }
    else { rt = f < 2 ? f : (f >> 1) + 1; ks = f < 2 ? 0 : f & 1; }
    float x[8];
    const double gq = s_g[16 * rt + m];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int pt = 2 * ks + half;   // tile of the products
      f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        if constexpr (BACK) acc = mma(read_rows<NI, KS>(s_q, pt, s), read_rows<NI, KS>(s_k, rt, s), acc);
        else acc = mma(read_rows<NI, KS>(s_k, pt, s), read_rows<NI, KS>(s_q, rt, s), acc);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int p = 16 * pt + 4 * g + r, q = 16 * rt + m;   // product and row
        const float v = a.scale * decay_exp(BACK ? s_g[p] - gq : gq - s_g[p]) * acc[r];
        x[4 * half + r] = (BACK ? q <= p : p <= q) ? v : 0.0f;
      }
    }
    const Frag<3> fr = to_frag<3>(x);
    unsigned char* dst = rec + (BACK ? Record<C>::PT : Record<C>::P) + f * 3 * kFrag + l * 16;
#pragma unroll
    for (int p = 0; p < 3; ++p) *reinterpret_cast<bf16x8*>(dst + p * kFrag) = fr.p[p];
  }
  __syncthreads();
  const int bad = *s_bad;   // rows from a token that is not finite on are those of I
  if (w < MT) {
#pragma unroll
    for (int jt = 0; jt < MT; ++jt) {
      if (jt > w) continue;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = 16 * w + 4 * g + r;
        s_a[i * LD + 16 * jt + m] = i < bad ? A[jt][r] : 0.0f;
      }
    }
  }
  __syncthreads();

  // diagonal blocks: column m of block w, rows one after the other
  for (int d = w; d < MT; d += kWaves) {
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s = i == m ? 1.0f : 0.0f;
      const float4* row = reinterpret_cast<const float4*>(s_a + (16 * d + i) * LD + 16 * d);
#pragma unroll
      for (int j = 0; j < i; j += 4) {
        const float4 v = row[j >> 2];
        s = fmaf(-v.x, x[j], s);
        if (j + 1 < i) s = fmaf(-v.y, x[j + 1], s);
        if (j + 2 < i) s = fmaf(-v.z, x[j + 2], s);
        if (j + 3 < i) s = fmaf(-v.w, x[j + 3], s);
      }
      x[i] = s;
    }
    if (g == 0) {
#pragma unroll
      for (int i = 0; i < 16; ++i) s_t[(16 * d + i) * LD + 16 * d + m] = x[i];
    } else if (g == 1 && (d & 1) == 0) {
      // the block above the next diagonal one, which its fragment holds too
#pragma unroll
      for (int i = 0; i < 16; ++i) s_t[(16 * d + i) * LD + 16 * (d + 1) + m] = 0.0f;
    }
  }
  __syncthreads();
  // one 16 x 16 block of -Y (B X): acc rows 4g + r are the products 4g + r of
  // the next factor, whose lane of row m holds 4g..4g+3
  auto quad = [&](const float* p, int it, int jt) {
    return *reinterpret_cast<const float4*>(p + (16 * it + m) * LD + 16 * jt + 4 * g);
  };
  auto column = [&](int kt, int jt, int r) { return s_t[(16 * kt + 4 * g + r) * LD + 16 * jt + m]; };
  auto put = [&](int it, int jt, f32x4 v) {
#pragma unroll
    for (int r = 0; r < 4; ++r) s_t[(16 * it + 4 * g + r) * LD + 16 * jt + m] = -v[r];
  };
  if (w < MT / 2) {
    const int it = 2 * w + 1, jt = 2 * w;
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f}, out = {0.0f, 0.0f, 0.0f, 0.0f};
    const float4 p = quad(s_a, it, jt);
    const float pa[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int r = 0; r < 4; ++r) acc = mfma4(pa[r], column(jt, jt, r), acc);
    const float4 q = quad(s_t, it, it);
    const float qa[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int r = 0; r < 4; ++r) out = mfma4(qa[r], acc[r], out);
    put(it, jt, out);
  }
  if constexpr (MT == 4) {
    __syncthreads();
    const int it = 2 + (w >> 1), jt = w & 1;
    f32x4 out = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int kt = 2; kt <= it; ++kt) {
      f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
      for (int lt = jt; lt < 2; ++lt) {
        const float4 p = quad(s_a, kt, lt);
        const float pa[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
        for (int r = 0; r < 4; ++r) acc = mfma4(pa[r], column(lt, jt, r), acc);
      }
      const float4 q = quad(s_t, it, kt);
      const float qa[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int r = 0; r < 4; ++r) out = mfma4(qa[r], acc[r], out);
    }
    put(it, jt, out);
  }
  __syncthreads();

  // T into fragments
  for (int f = w; f < tri_frags<C>(); f += kWaves) {
    const int it = C == 32 || f < 2 ? f : (f >> 1) + 1, ks = C == 32 || f < 2 ? 0 : f & 1;
    const float4 lo = quad(s_t, it, 2 * ks), hi = quad(s_t, it, 2 * ks + 1);
    const float x[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    const Frag<3> fr = to_frag<3>(x);
#pragma unroll
    for (int p = 0; p < 3; ++p)
      *reinterpret_cast<bf16x8*>(rec + Record<C>::T + (f * 3 + p) * kFrag + l * 16) = fr.p[p];
    if constexpr (BACK) {
      const int jt = C == 32 ? f : f < 4 ? f >> 1 : f - 2, kt = C == 32 ? 0 : f < 4 ? f & 1 : 1;
      float z[8];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        z[r] = column(2 * kt, jt, r);
        z[4 + r] = column(2 * kt + 1, jt, r);
      }
      const Frag<3> ft = to_frag<3>(z);
#pragma unroll
      for (int p = 0; p < 3; ++p)
        *reinterpret_cast<bf16x8*>(rec + Record<C>::P + (f * 3 + p) * kFrag + l * 16) = ft.p[p];
    }
  }
  if (tid < C) {
    float* dec = reinterpret_cast<float*>(rec + Record<C>::decays(BACK));
    const float from = expf(static_cast<float>(s_g[tid]));
    dec[tid] = from;
    dec[C + tid] = expf(static_cast<float>(s_g[C - 1] - s_g[tid]));
    dec[2 * C + tid] = tid < bad ? s_b[tid] : __builtin_nanf("");
    dec[3 * C + tid] = a.scale * from;
  }
}

template <bool BF16, int KP, bool BACK>
hipError_t run(const DeltaArgs& a, hipStream_t stream) {
  using Z = Shape<BF16, KP>;
  constexpr int C = Z::C;
  constexpr int square = C * (C + 4) * 4, stage = 2 * Z::kMat;
  constexpr int lds = (stage > 2 * square ? stage : 2 * square) + C * 8 + C * 4 + 16;
  constexpr auto* prep = k_delta_prep<BF16, KP, BACK>;
  if (const hipError_t e = allow_lds<prep>(lds); e != hipSuccess) return e;
  const int chunks = (a.L + C - 1) / C;
  if constexpr (!BF16) {
    constexpr auto* frags = k_delta_frags<KP, BACK>;
    if (const hipError_t e = allow_lds<frags>(Z::frags(BACK)); e != hipSuccess) return e;
    frags<<<dim3(static_cast<unsigned>(a.B * a.Hk * chunks)), dim3(kThreads), Z::frags(BACK), stream>>>(a, chunks);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  prep<<<dim3(static_cast<unsigned>(a.B * a.Hv * chunks)), dim3(kThreads), lds, stream>>>(a, chunks);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_prep(const DeltaArgs& a, bool backward, hipStream_t stream) {
  const bool wide = a.Dk > 64;
  if (a.bf16_io) {
    if (backward) return wide ? run<true, 128, true>(a, stream) : run<true, 64, true>(a, stream);
    return wide ? run<true, 128, false>(a, stream) : run<true, 64, false>(a, stream);
  }
  if (backward) return wide ? run<false, 128, true>(a, stream) : run<false, 64, true>(a, stream);
  return wide ? run<false, 128, false>(a, stream) : run<false, 64, false>(a, stream);
}

namespace {

// Segments of a call: none where the chain's workgroups (64 columns of a head
// each) fill half of the compute units or the sequence is short; otherwise as
// many as the estimate below favours, in microseconds fitted to calls (128 or 64
// features of a key): a chunk's pass for outputs and for a segment's sums with a
// workgroup on few units (with one on each they take 1.35 times as long), a
// segment's join. Over 148 calls (1 to 48 heads of 1024 to 8192 steps, 64 and 128
// features, both types, both directions) its choice took 0.7 % longer than the best
// of eleven numbers on average and 10 % at most; one head of 8192 steps, 128 x 128,
// bf16: 429 us in one piece, 108 in 16.
int segments_of(int64_t heads, int dvp, int dkp, int chunks, bool bf16) {
  const bool wide = dkp > 64;
  const double out = bf16 ? (wide ? 2.8 : 2.2) : (wide ? 2.1 : 1.5), sum = bf16 ? (wide ? 2.1 : 1.65) : (wide ? 1.6 : 1.1);
  const double join = wide ? 2.5 : 0.45;
  constexpr double kStart = 2.0;   // a workgroup's first loads
  if (heads * ((dvp + 63) / 64) >= kUnits / 2 || chunks < 16) return 1;
  auto rounds = [](int64_t chains, int columns) {
    const int64_t wgs = chains * (narrow_groups(chains, columns) ? (columns + 31) / 32 : (columns + 63) / 64);
    const int64_t whole = (wgs + kUnits - 1) / kUnits;
    return static_cast<double>(whole) * (1.0 + 0.35 * static_cast<double>(wgs < kUnits ? wgs : kUnits) / kUnits);
  };
  double best = chunks * out * rounds(heads, dvp);
  int count = 1;
  for (int n = 2; n <= 32 && n * 2 <= chunks; ++n) {
    const int each = (chunks + n - 1) / n;
    if ((chunks + each - 1) / each != n) continue;
    const double t = (each * sum + kStart) * rounds(heads * (n - 1), dvp + dkp) + (each * out + kStart) * rounds(heads * n, dvp) + n * join;
    if (t < (count == 1 ? 0.95 : 1.0) * best) {
      best = t;
      count = n;
    }
  }
  return count;
}

template <bool BF16, int KP>
int64_t work(DeltaArgs& a, DeltaSegs& segs, bool backward) {
  using Z = Shape<BF16, KP>;
  const int64_t heads = static_cast<int64_t>(a.B) * a.Hv;
  const int chunks = (a.L + Z::C - 1) / Z::C;
  const int64_t frags = static_cast<int64_t>(a.B) * a.Hk * chunks * Z::frags(backward);
  const int64_t recs = heads * chunks * Record<Z::C>::bytes(backward);
  a.frags = static_cast<unsigned char*>(a.ws);
  a.recs = a.frags + frags;
  segs.dkp = (a.Dk + 15) & ~15;
  segs.dvp = (a.Dv + 15) & ~15;
  segs.count = segments_of(heads, segs.dvp, segs.dkp, chunks, BF16);
  segs.chunks = segs.count > 1 ? (chunks + segs.count - 1) / segs.count : chunks;
  segs.p = reinterpret_cast<float*>(a.recs + recs);
  const int64_t states = segs.count > 1 ? segs.at(heads, 0) : 0;
  segs.back = segs.p + states;
  const int64_t backs = backward && segs.count > 1 ? segs.at_back(heads, 0) : 0;
  return frags + recs + (states + backs) * 4;
}

}  // namespace

int64_t delta_work(DeltaArgs& a, DeltaSegs& segs, bool backward) {
  if (a.bf16_io) return a.Dk > 64 ? work<true, 128>(a, segs, backward) : work<true, 64>(a, segs, backward);
  return a.Dk > 64 ? work<false, 128>(a, segs, backward) : work<false, 64>(a, segs, backward);
}

}  // namespace s5
