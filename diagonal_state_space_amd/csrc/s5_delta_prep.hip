// First kernel of the chunked gated delta rule: what a chunk's steps need
// besides the state, for all chunks at once.
//
// With G_i the chunk's inclusive sums of g and M_ij = exp(G_i - G_j) (j <= i):
//   A_ij = beta_i M_ij k_i.k_j (j < i),  T = (I + A)^-1,  P_ij = M_ij q_i.k_j
// so that the chunk's writes are U = T beta (V - e^G K S) and its outputs
// e^G Q S + P U. One workgroup of four waves per chunk and value head.
//
// Both products run on the matrix cores from staged k and q; P comes out
// transposed, which is the order of its operand fragments, and is stored from
// the registers. The inverse: the 16 x 16 diagonal blocks by substitution, a
// column a lane; then blocks of 32 and 64 from halves,
//   [X 0; B Y]^-1 = [X^-1 0; -Y^-1 B X^-1  Y^-1],
// by float32 matrix instructions, the second factor from the accumulators of
// the first. Substitution and halves keep the error of a triangular solve,
// which powers of A (they grow for equal keys) do not.
// The sums of g are float64: their differences stay exact to float32 however
// fast a head forgets.
#include "s5_delta_tile.h"

namespace s5 {

using namespace delta;

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = 4;

__device__ __forceinline__ f32x4 mfma4(float a, float b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

template <bool BF16, int C, int KP, bool BACK>
__global__ void __launch_bounds__(kThreads) k_delta_prep(DeltaArgs a, int chunks, bool vec) {
  constexpr int NI = BF16 ? 1 : 3;
  constexpr int NO = BF16 ? 2 : 3;
  constexpr int KS = KP / 32, MT = C / 16;
  constexpr int LD = C + 4;
  extern __shared__ __align__(16) unsigned char smem[];
  unsigned char* s_k = smem;
  unsigned char* s_q = s_k + MT * KS * NI * kFrag;
  constexpr int kStage = 2 * MT * KS * NI * kFrag;
  float* s_t = reinterpret_cast<float*>(smem);                        // T, over k and q when they are read
  float* s_a = reinterpret_cast<float*>(smem + (kStage > C * LD * 4 ? kStage : C * LD * 4));   // A
  double* s_g = reinterpret_cast<double*>(s_a + C * LD);              // sums of g
  float* s_b = reinterpret_cast<float*>(s_g + C);                     // beta
  int* s_bad = reinterpret_cast<int*>(s_b + C);

  const int tid = threadIdx.x, l = tid & 63, g = l >> 4, m = l & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = blockIdx.x % chunks, bh = blockIdx.x / chunks;
  const int b = bh / a.Hv, h = bh - b * a.Hv, hk = h / (a.Hv / a.Hk);
  const int left = length_of(a, b) - n * C;     // valid tokens from the chunk's start
  if (left <= 0) return;
  const int64_t tok = static_cast<int64_t>(b) * a.L + n * C;

  // stage k and q
  const int64_t es = BF16 ? 2 : 4;
  const Rows kr{static_cast<const char*>(a.k) + (tok * a.ldk + static_cast<int64_t>(hk) * a.Dk) * es, a.ldk, left, a.Dk, vec};
  const Rows qr{static_cast<const char*>(a.q) + (tok * a.ldq + static_cast<int64_t>(hk) * a.Dk) * es, a.ldq, left, a.Dk, vec};
  for (int i = tid; i < (C / 4) * (KP / 8); i += kThreads) {
    const int tg = i / (KP / 8), dg = i % (KP / 8);
    store_rows<BF16, KS>(s_k, Parts<BF16>(load_block<BF16>(kr, 4 * tg, 8 * dg)), tg, dg);
    store_rows<BF16, KS>(s_q, Parts<BF16>(load_block<BF16>(qr, 4 * tg, 8 * dg)), tg, dg);
  }
  // sums of g (a wave's 64 lanes hold the chunk)
  if (w == 0) {
    const bool live = l < C && l < left;
    const float gi = live ? a.g[(tok + l) * a.Hv + h] : 0.0f;
    const float be = live ? a.beta[(tok + l) * a.Hv + h] : 0.0f;
    const double s = chunk_sums(gi);
    const bool bad = !(gi < INFINITY) || !(fabsf(be) < INFINITY);
    const uint64_t mask = __ballot(bad);
    if (l < C) {
      s_g[l] = s;
      s_b[l] = be;
    }
    if (l == 0) *s_bad = mask != 0 ? static_cast<int>(__ffsll(static_cast<unsigned long long>(mask))) - 1 : C;
  }
  __syncthreads();

  unsigned char* rec = static_cast<unsigned char*>(a.ws) + static_cast<int64_t>(blockIdx.x) * Record<C>::bytes(BACK, NO);
  // A: wave w the row tiles w, w + 4 (C = 64: one each)
  for (int it = w; it < MT; it += kWaves) {
    for (int jt = 0; jt <= it; ++jt) {
      f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
        acc = mma(read_rows<NI, KS>(s_k, it, ks), read_rows<NI, KS>(s_k, jt, ks), acc);
      const int j = 16 * jt + m;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = 16 * it + 4 * g + r;
        float x = 0.0f;
        if (j < i) x = s_b[i] * expf(static_cast<float>(s_g[i] - s_g[j])) * acc[r];
        s_a[i * LD + j] = x;
        // a key that is not finite, or whose length is not
        if (i == j && !(acc[r] < INFINITY)) atomicMin(s_bad, i);
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
        const int i = BACK ? p : q, j = BACK ? q : p;
        x[4 * half + r] = j <= i ? expf(static_cast<float>(s_g[i] - s_g[j])) * acc[r] : 0.0f;
      }
    }
    constexpr int NPP = BACK ? 3 : NO;
    const Frag<NPP> fr = to_frag<NPP>(x);
    unsigned char* dst = rec + (BACK ? Record<C>::PT : Record<C>::P) + f * NPP * kFrag + l * 16;
#pragma unroll
    for (int p = 0; p < NPP; ++p) *reinterpret_cast<bf16x8*>(dst + p * kFrag) = fr.p[p];
  }
  __syncthreads();
  const int bad = *s_bad;

  // diagonal blocks: column m of block w, rows one after the other
  for (int d = w; d < MT; d += kWaves) {
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s = i == m ? 1.0f : 0.0f;
      const float* row = s_a + (16 * d + i) * LD + 16 * d;
      const bool ok = 16 * d + i < bad;    // rows from a bad token on stay those of I
#pragma unroll
      for (int j = 0; j < i; ++j) s = fmaf(ok ? -row[j] : 0.0f, x[j], s);
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
  auto a_block = [&](int it, int jt) {
    float4 v = quad(s_a, it, jt);
    if (16 * it + m >= bad) v = float4{0.0f, 0.0f, 0.0f, 0.0f};
    return v;
  };
  auto put = [&](int it, int jt, f32x4 v) {
#pragma unroll
    for (int r = 0; r < 4; ++r) s_t[(16 * it + 4 * g + r) * LD + 16 * jt + m] = -v[r];
  };
  if (w < MT / 2) {
    const int it = 2 * w + 1, jt = 2 * w;
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f}, out = {0.0f, 0.0f, 0.0f, 0.0f};
    const float4 p = a_block(it, jt);
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
        const float4 p = a_block(kt, lt);
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
    float* dec = reinterpret_cast<float*>(rec + Record<C>::decays(BACK, NO));
    dec[tid] = expf(static_cast<float>(s_g[tid]));
    dec[C + tid] = expf(static_cast<float>(s_g[C - 1] - s_g[tid]));
    dec[2 * C + tid] = s_b[tid];
    if (tid == 0) {
      dec[3 * C] = expf(static_cast<float>(s_g[C - 1]));
      reinterpret_cast<int*>(dec)[3 * C + 1] = bad;
    }
  }
}

template <bool BF16, int KP, bool BACK>
hipError_t run(const DeltaArgs& a, hipStream_t stream) {
  constexpr int C = chunk_of<BF16>(), NI = BF16 ? 1 : 3;
  const int chunks = (a.L + C - 1) / C;
  const int stage = 2 * (C / 16) * (KP / 32) * NI * kFrag, square = C * (C + 4) * 4;
  const size_t lds = (stage > square ? stage : square) + square + C * 8 + C * 4 + 16;
  const int64_t blocks = static_cast<int64_t>(a.B) * a.Hv * chunks;
  k_delta_prep<BF16, C, KP, BACK><<<dim3(static_cast<unsigned>(blocks)), dim3(kThreads), lds, stream>>>(
      a, chunks, delta_vectored(a));
  return hipGetLastError();
}

}  // namespace

bool delta_vectored(const DeltaArgs& a) {
  const int V = a.bf16_io ? 8 : 4;
  auto ok = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  return a.Dk % V == 0 && a.ldq % V == 0 && a.ldk % V == 0 && ok(a.q) && ok(a.k);
}

hipError_t launch_delta_prep(const DeltaArgs& a, bool backward, hipStream_t stream) {
  const bool wide = a.Dk > 64;
  if (a.bf16_io) {
    if (backward) return wide ? run<true, 128, true>(a, stream) : run<true, 64, true>(a, stream);
    return wide ? run<true, 128, false>(a, stream) : run<true, 64, false>(a, stream);
  }
  if (backward) return wide ? run<false, 128, true>(a, stream) : run<false, 64, true>(a, stream);
  return wide ? run<false, 128, false>(a, stream) : run<false, 64, false>(a, stream);
}

}  // namespace s5
