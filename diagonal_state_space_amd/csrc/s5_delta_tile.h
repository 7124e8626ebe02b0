// Tiles of the chunked gated delta rule: operand fragments in LDS, float32
// values as three bf16 parts, and the workspace records of a chunk.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "s5_common.h"
#include "s5_delta.h"

namespace s5 {
namespace delta {

// ---- float32 values as bf16 parts ----------------------------------------------
// A float32 is the sum of three bf16 values exactly (three times 8 of its 24
// bits, each cut off the rest), so products of float32 operands run on the
// bf16 matrix instructions: the six part products above 2^-24 of the result
// for two float32 operands, three for one with a bf16 operand. Measured
// alternatives: two parts leave 3e-6 in the float32 state, the float32 matrix
// instruction takes 8 x 32 cycles where six bf16 ones take 6 x 16.

__device__ __forceinline__ float cut(float x) { return __uint_as_float(__float_as_uint(x) & 0xffff0000u); }

// two floats rounded to a pair of bf16
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t round2(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

// upper halves of two floats as a pair of bf16
__device__ __forceinline__ uint32_t upper(float lo, float hi) {
  return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}

template <int NP>
struct Frag {
  bf16x8 p[NP];
};

// an operand fragment from eight float32 values (in the order of its slots);
// fewer than three parts round the last one (an error below 2^-16 with two)
template <int NP>
__device__ __forceinline__ Frag<NP> to_frag(const float (&x)[8]) {
  union {
    uint32_t w[4];
    bf16x8 v;
  } out[NP];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = x[2 * i], b = x[2 * i + 1];
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      out[p].w[i] = NP < 3 && p == NP - 1 ? round2(a, b) : upper(a, b);
      if (p + 1 < NP) {
        a -= cut(a);
        b -= cut(b);
      }
    }
  }
  Frag<NP> f;
#pragma unroll
  for (int p = 0; p < NP; ++p) f.p[p] = out[p].v;
  return f;
}

// two accumulator tiles (rows 4g + r of 32 rows) as the operand over these rows
template <int NP>
__device__ __forceinline__ Frag<NP> to_frag(f32x4 a, f32x4 b) {
  const float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  return to_frag<NP>(x);
}

// c += a b over 32 products, part products down to the parts' own rounding
template <int NA, int NB>
__device__ __forceinline__ f32x4 mma(const Frag<NA>& a, const Frag<NB>& b, f32x4 c) {
  constexpr int last = (NA > NB ? NA : NB) - 1;
#pragma unroll
  for (int i = 0; i < NA; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
      if (i + j <= last) c = mfma(a.p[i], b.p[j], c);
  return c;
}

// ---- fragments in LDS ----------------------------------------------------------
// A fragment holds 16 rows by 32 products; lane l has row l%16 and, with
// g = l/16, the products 4g..4g+3 and 16+4g..16+4g+3: the order in which two
// accumulator tiles hold their rows, so that results become operands without
// an exchange. It is stored as 64 slots of 16 bytes for each part; the row is
// exchanged (xor) with a number of the fragment and g, which spreads the
// writes of a staging wave over the banks.

constexpr int kFrag = 1024;   // bytes of one part of a fragment

__device__ __forceinline__ int slot_of(int g, int m, int mix) { return (g * 16 + (m ^ (mix & 15))) * 16; }

template <int NP>
__device__ __forceinline__ Frag<NP> read_frag(const unsigned char* base, int frag, int mix) {
  const int l = threadIdx.x & 63;
  const unsigned char* p = base + frag * NP * kFrag + slot_of(l >> 4, l & 15, mix);
  Frag<NP> f;
#pragma unroll
  for (int i = 0; i < NP; ++i) f.p[i] = *reinterpret_cast<const bf16x8*>(p + i * kFrag);
  return f;
}

// fragments of rows = tokens, products = features: index and exchange
template <int KS>
__device__ __forceinline__ int row_frag(int mt, int ks) { return mt * KS + ks; }
__device__ __forceinline__ int row_mix(int ks, int g) { return ks * 4 + g; }
template <int NP, int KS>
__device__ __forceinline__ Frag<NP> read_rows(const unsigned char* base, int mt, int ks) {
  return read_frag<NP>(base, row_frag<KS>(mt, ks), row_mix(ks, (threadIdx.x & 63) >> 4));
}
// fragments of rows = features, products = tokens
template <int NP, int C>
__device__ __forceinline__ Frag<NP> read_cols(const unsigned char* base, int mt, int ks) {
  return read_frag<NP>(base, mt * (C / 32) + ks, mt);
}

// ---- staging of token rows -----------------------------------------------------
// A block is four tokens by eight features of one head.
template <bool BF16>
struct Block {
  uint4 r[BF16 ? 4 : 8];
};

struct Rows {
  const void* p;      // element 0 of the chunk's first token and the head
  int64_t ld;         // elements between tokens
  int tokens, dims;   // valid ones; the rest is zero
  bool vec;           // whole 16-byte groups are aligned
};

template <bool BF16>
__device__ __forceinline__ Block<BF16> load_block(const Rows& x, int t0, int d0) {
  Block<BF16> b;
  const int nd = x.dims - d0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t i = (t0 + j) * x.ld + d0;
    const bool live = t0 + j < x.tokens;
    if constexpr (BF16) {
      const uint16_t* p = static_cast<const uint16_t*>(x.p) + i;
      if (live && nd >= 8 && x.vec) {
        b.r[j] = *reinterpret_cast<const uint4*>(p);
      } else {
        uint32_t w[4] = {0, 0, 0, 0};
        if (live) {
#pragma unroll
          for (int c = 0; c < 8; ++c)
            if (c < nd) w[c >> 1] |= static_cast<uint32_t>(p[c]) << (16 * (c & 1));
        }
        b.r[j] = uint4{w[0], w[1], w[2], w[3]};
      }
    } else {
      const uint32_t* p = static_cast<const uint32_t*>(x.p) + i;
      if (live && nd >= 8 && x.vec) {
        b.r[2 * j] = reinterpret_cast<const uint4*>(p)[0];
        b.r[2 * j + 1] = reinterpret_cast<const uint4*>(p)[1];
      } else {
        uint32_t w[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) w[c] = live && c < nd ? p[c] : 0u;
        b.r[2 * j] = uint4{w[0], w[1], w[2], w[3]};
        b.r[2 * j + 1] = uint4{w[4], w[5], w[6], w[7]};
      }
    }
  }
  return b;
}

__device__ __forceinline__ uint32_t word(const uint4& r, int i) { return i == 0 ? r.x : i == 1 ? r.y : i == 2 ? r.z : r.w; }

// the bf16 parts of a block as bits: part p of token j, feature c
template <bool BF16>
struct Parts {
  static constexpr int NP = BF16 ? 1 : 3;
  uint32_t pair[NP][4][4];   // [part][token][features 2i, 2i + 1]
  __device__ __forceinline__ explicit Parts(const Block<BF16>& b) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (BF16) {
          pair[0][j][i] = word(b.r[j], i);
        } else {
          float lo = __uint_as_float(word(b.r[2 * j + (i >> 1)], (2 * i) & 3));
          float hi = __uint_as_float(word(b.r[2 * j + (i >> 1)], (2 * i + 1) & 3));
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            pair[p][j][i] = upper(lo, hi);
            lo -= cut(lo);
            hi -= cut(hi);
          }
        }
      }
  }
};

// block (tokens 4 tg.., features 8 dg..) into row fragments
template <bool BF16, int KS>
__device__ __forceinline__ void store_rows(unsigned char* base, const Parts<BF16>& x, int tg, int dg) {
  constexpr int NP = Parts<BF16>::NP;
  const int ks = dg >> 2, h = (dg >> 1) & 1, g0 = 2 * (dg & 1);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int m = 4 * (tg & 3) + j, mt = tg >> 2;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      unsigned char* f = base + (row_frag<KS>(mt, ks) * NP + p) * kFrag + 8 * h;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        *reinterpret_cast<uint2*>(f + slot_of(g0 + i, m, row_mix(ks, g0 + i))) = uint2{x.pair[p][j][2 * i], x.pair[p][j][2 * i + 1]};
    }
  }
}

// the same block into fragments of rows = features
template <bool BF16, int C>
__device__ __forceinline__ void store_cols(unsigned char* base, const Parts<BF16>& x, int tg, int dg) {
  constexpr int NP = Parts<BF16>::NP;
  const int mt = dg >> 1, ks = tg >> 3, h = (tg >> 2) & 1, g = tg & 3;
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    unsigned char* f = base + ((mt * (C / 32) + ks) * NP + p) * kFrag + 8 * h;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const uint32_t sel = (c & 1) ? 0x07060302u : 0x05040100u;   // upper or lower halves of two words
      const uint32_t a = __builtin_amdgcn_perm(x.pair[p][1][c >> 1], x.pair[p][0][c >> 1], sel);
      const uint32_t b = __builtin_amdgcn_perm(x.pair[p][3][c >> 1], x.pair[p][2][c >> 1], sel);
      *reinterpret_cast<uint2*>(f + slot_of(g, 8 * (dg & 1) + c, mt)) = uint2{a, b};
    }
  }
}

// ---- elements of v, y and their gradients in accumulator order --------------------
template <bool BF16>
__device__ __forceinline__ float load_el(const void* p, int64_t i) {
  if constexpr (BF16) return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
  else return static_cast<const float*>(p)[i];
}

template <bool BF16>
__device__ __forceinline__ void store_el(void* p, int64_t i, float x) {
  if constexpr (BF16) static_cast<uint16_t*>(p)[i] = f32_to_bf16(x);
  else static_cast<float*>(p)[i] = x;
}

// ---- chunks and their workspace records -----------------------------------------
// Chunk length: 64 tokens for bf16 io; 32 for float32 io, whose three parts of
// q and k fill the LDS three times as fast.
template <bool BF16>
constexpr int chunk_of() { return BF16 ? 64 : 32; }

// fragments of the lower triangle of a C x C matrix (rows i, products j <= i),
// and of its transpose (rows j, products i >= j)
template <int C>
constexpr int tri_frags() { return C == 64 ? 6 : 2; }
template <int C>
__host__ __device__ constexpr int tri_frag(int it, int ks) { return it < 2 ? it : 2 * (it - 1) + ks; }
template <int C>
__host__ __device__ constexpr int tri_frag_t(int jt, int ks) { return C == 32 ? jt : jt < 2 ? 2 * jt + ks : 2 + jt; }

// The record of one head's chunk: the parts of T = (I + A)^-1 and of P = M o QK^T
// (backward: T, its transpose and that of P), then the decays
//   from[i] = e^{G_i}, to[i] = e^{G_end - G_i}, beta[i], whole = e^{G_end}, bad
// with bad the first token whose key, decay or strength is not finite (C if none).
template <int C>
struct Record {
  static constexpr int T = 0;
  static constexpr int P = tri_frags<C>() * 3 * kFrag;           // backward: T transposed
  static constexpr int PT = 2 * P;                               // backward only
  static constexpr int decays(bool backward, int np) { return backward ? 3 * P : P + tri_frags<C>() * np * kFrag; }
  static constexpr int bytes(bool backward, int np) { return decays(backward, np) + 4 * C * 4; }
};

// a log decay below this is 0 as a float32 factor: sums of g stay finite with
// it in the place of -inf, without -inf - (-inf)
constexpr float kLeastDecay = -110.0f;

// inclusive sums of g over a wave's lanes (one chunk), float64: their
// differences stay exact to float32 however fast a head forgets
__device__ __forceinline__ double chunk_sums(float g) {
  const int l = threadIdx.x & 63;
  double s = g < kLeastDecay ? kLeastDecay : g;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const double up = __shfl_up(s, o);
    if (l >= o) s += up;
  }
  return s;
}

__device__ __forceinline__ int length_of(const DeltaArgs& a, int b) {
  if (a.lengths == nullptr) return a.L;
  const int n = a.lengths[b];
  return n < 0 ? 0 : n > a.L ? a.L : n;
}

}  // namespace delta
}  // namespace s5
