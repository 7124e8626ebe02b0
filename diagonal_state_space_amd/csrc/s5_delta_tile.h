// Tiles of the chunked gated delta rule: operand fragments in LDS, float32
// values as three bf16 parts, and the workspace records of a chunk.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

#include "s5_common.h"
#include "s5_delta.h"

namespace s5 {
namespace delta {

// ---- float32 values as bf16 parts ----------------------------------------------
// A float32 is the sum of three bf16 values exactly (three times 8 of its 24
// bits, each cut off the rest), so products of float32 operands run on the
// bf16 matrix instructions: three part products for one with a bf16 operand
// (exact), six for two float32 operands. The two that would come next are left
// out, 2^-24.5 of a product on average (2^-21 at most): less than its rounding.
// Measured alternatives: two parts leave 3e-6 in the float32 state, the float32
// matrix instruction takes 8 x 32 cycles where six bf16 ones take 6 x 16.

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
  // a product that x is must not go into the differences below unrounded: the
  // parts are those of x wherever it is split
#pragma clang fp contract(off)
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

// the same for N tiles at once: neighbours in the order of issue do not wait for
// each other
template <int N, int NA, int NB>
__device__ __forceinline__ void mma(f32x4 (&c)[N], const Frag<NA> (&a)[N], const Frag<NB>& b) {
  constexpr int last = (NA > NB ? NA : NB) - 1;
#pragma unroll
  for (int i = 0; i < NA; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
      if (i + j <= last) {
#pragma unroll
        for (int t = 0; t < N; ++t) c[t] = mfma(a[t].p[i], b.p[j], c[t]);
      }
}

// ---- fragments in LDS ----------------------------------------------------------
// A fragment holds 16 rows by 32 products; lane l has row l%16 and, with
// g = l/16, the products 4g..4g+3 and 16+4g..16+4g+3: the order in which two
// accumulator tiles hold their rows, so that results become operands without
// an exchange. It is stored as 64 slots of 16 bytes for each part; the row is
// exchanged (xor) with a number of the fragment and g, which spreads the
// writes of a staging wave over the banks.

constexpr int kFrag = 1024;   // bytes of one part of a fragment
constexpr int kMaxLds = 160 * 1024;

// Asks once for each device (a kernel's attributes are those of one) that it may
// be launched with so much LDS.
template <auto* KERNEL>
hipError_t allow_lds(int bytes) {
  static std::atomic<uint64_t> allowed{0};
  int device = 0;
  hipError_t e = hipGetDevice(&device);
  if (e != hipSuccess) return e;
  const uint64_t bit = device < 64 ? uint64_t{1} << device : 0;
  if (allowed.load(std::memory_order_acquire) & bit) return hipSuccess;
  e = hipFuncSetAttribute(reinterpret_cast<const void*>(KERNEL), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess) allowed.fetch_or(bit, std::memory_order_release);
  return e;
}

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

// the same offset, of which the compiler makes no table for a loop: sums with it
// are formed where they are used instead of kept in registers throughout
__device__ __forceinline__ int here(int o) {
  asm volatile("" : "+v"(o));
  return o;
}

__device__ __forceinline__ int here_s(int o) {
  asm volatile("" : "+s"(o));
  return o;
}

// The chains' products run in stages whose fragments are read one stage ahead
// (left to itself the compiler reads a fragment right before its use, and the
// wave, alone on its SIMD, waits for the LDS each time). A stage ends here.
__device__ __forceinline__ void stage_end() { __builtin_amdgcn_sched_barrier(0); }

// four of the state's tiles by the fragments of 32 tokens. bf16's exchanged slots
// are formed where they are used: kept throughout they do not all find a register
// in its y pass, and what is spilled is waited for with v.
template <int NP, int C>
__device__ __forceinline__ void read_cols4(Frag<NP> (&f)[4], const unsigned char* a, int t0, int ks) {
  const int slot = 16 * (threadIdx.x & 63), l16 = NP == 1 ? here(slot) : slot;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const unsigned char* p = a + ((t0 + t) * (C / 32) + ks) * NP * kFrag + (l16 ^ 16 * (t0 + t));
#pragma unroll
    for (int i = 0; i < NP; ++i) f[t].p[i] = *reinterpret_cast<const bf16x8*>(p + i * kFrag);
  }
}
template <int NP, int KT>
__device__ __forceinline__ void mma_cols4(f32x4 (&s)[KT], int t0, const Frag<NP> (&f)[4], const Frag<3>& x) {
#pragma unroll
  for (int i = 0; i < NP; ++i)
#pragma unroll
    for (int j = 0; i + j < 3; ++j)
#pragma unroll
      for (int t = 0; t < 4; ++t) s[t0 + t] = mfma(f[t].p[i], x.p[j], s[t0 + t]);
}

// ---- staging of token rows -----------------------------------------------------
// A block is four tokens by eight features of one head.
template <bool BF16>
struct Block {
  uint4 r[BF16 ? 4 : 8];
};

// Rows of a chunk through a buffer descriptor that ends with the last valid
// one: what lies behind reads as zero and is not written, without a branch.
// Features that do not exist go to an offset behind every chunk.
typedef __amdgpu_buffer_rsrc_t Buf;
constexpr int kNowhere = 0x60000000;
constexpr int kBufferWord3 = 0x00020000;          // raw buffer, 32-bit data format

// `rows` rows of `width` bytes, `ld` bytes apart, from p
__device__ __forceinline__ Buf rows_buf(const void* p, int rows, int ld, int width) {
  const int bytes = rows > 0 ? (rows - 1) * ld + width : 0;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, kBufferWord3);
}

__device__ __forceinline__ uint4 load16(Buf r, int o) {
  return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, o, 0, 0));
}

__device__ __forceinline__ void store16(Buf r, int o, f32x4 x) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(__attribute__((ext_vector_type(4))) unsigned, x), r, o, 0, 0);
}

// bytes between a chunk's tokens. A longer stride than kMostStride is that of
// chunks of one token: only its row is in the buffer, whatever the distance.
__device__ __forceinline__ int row_bytes(int64_t stride, int es) {
  return static_cast<int>(stride < kMostStride ? stride : kMostStride) * es;
}

// four tokens `ld` bytes apart, the first at byte `o` (kNowhere: a block of
// features that do not exist); nd of the eight features exist
template <bool BF16>
__device__ __forceinline__ Block<BF16> load_block(Buf buf, int o, int ld, int nd, bool vec) {
  Block<BF16> b;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int at = o + j * ld;
    if (vec) {
      if constexpr (BF16) {
        b.r[j] = load16(buf, at);
      } else {
        b.r[2 * j] = load16(buf, at);
        b.r[2 * j + 1] = load16(buf, nd > 4 ? at + 16 : kNowhere);
      }
    } else if constexpr (BF16) {
      uint32_t w[8];
#pragma unroll
      for (int c = 0; c < 8; ++c)
        w[c] = static_cast<uint16_t>(__builtin_amdgcn_raw_buffer_load_b16(buf, c < nd ? at + 2 * c : kNowhere, 0, 0));
      b.r[j] = uint4{w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16};
    } else {
      uint32_t w[8];
#pragma unroll
      for (int c = 0; c < 8; ++c)
        w[c] = __builtin_amdgcn_raw_buffer_load_b32(buf, c < nd ? at + 4 * c : kNowhere, 0, 0);
      b.r[2 * j] = uint4{w[0], w[1], w[2], w[3]};
      b.r[2 * j + 1] = uint4{w[4], w[5], w[6], w[7]};
    }
  }
  return b;
}

// byte offset of the block (tg, dg) of rows `ld` bytes apart with `dims` features
template <bool BF16>
__device__ __forceinline__ int block_offset(int tg, int dg, int ld, int dims) {
  return 8 * dg < dims ? 4 * tg * ld + 8 * dg * (BF16 ? 2 : 4) : kNowhere;
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
// an element's bits, and its value (apart: a conversion at the load would wait for it)
template <bool BF16>
__device__ __forceinline__ uint32_t load_raw(Buf r, int o) {
  if constexpr (BF16) return static_cast<uint16_t>(__builtin_amdgcn_raw_buffer_load_b16(r, o, 0, 0));
  else return __builtin_amdgcn_raw_buffer_load_b32(r, o, 0, 0);
}
template <bool BF16>
__device__ __forceinline__ float value(uint32_t raw) {
  return __uint_as_float(BF16 ? raw << 16 : raw);
}

// two rows' elements, `ld` bytes apart (bf16: rounded in one instruction)
template <bool BF16>
__device__ __forceinline__ void store_el2(Buf r, int o, int ld, float x, float y) {
  if constexpr (BF16) {
    const uint32_t w = round2(x, y);
    __builtin_amdgcn_raw_buffer_store_b16(static_cast<short>(w), r, o, 0, 0);
    __builtin_amdgcn_raw_buffer_store_b16(static_cast<short>(w >> 16), r, o + ld, 0, 0);
  } else {
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_int(x), r, o, 0, 0);
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_int(y), r, o + ld, 0, 0);
  }
}

template <bool BF16>
__device__ __forceinline__ void store_el(Buf r, int o, float x) {
  if constexpr (BF16) __builtin_amdgcn_raw_buffer_store_b16(static_cast<short>(round2(x, x)), r, o, 0, 0);
  else __builtin_amdgcn_raw_buffer_store_b32(__float_as_int(x), r, o, 0, 0);
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

// the fragments of a lower triangular matrix for the products 32 ks.. (UP: of
// its transpose), the row tiles that have them, and c += a x with them
template <bool UP, int C>
__device__ __forceinline__ bool tri_has(int t, int ks) { return UP ? t <= 2 * ks + 1 : t >= 2 * ks; }
template <bool UP, int C, int NP>
__device__ __forceinline__ void read_tri(Frag<NP> (&f)[C / 16], const unsigned char* a, int ks) {
  // rows are not exchanged here: slot l; formed where it is used (bf16's y pass has
  // no register to keep it in)
  const unsigned char* p = a + here(16 * (threadIdx.x & 63));
#pragma unroll
  for (int t = 0; t < C / 16; ++t)
    if (tri_has<UP, C>(t, ks)) {
#pragma unroll
      for (int i = 0; i < NP; ++i)
        f[t].p[i] = *reinterpret_cast<const bf16x8*>(p + ((UP ? tri_frag_t<C>(t, ks) : tri_frag<C>(t, ks)) * NP + i) * kFrag);
    }
}
template <bool UP, int C, int NP, int NB>
__device__ __forceinline__ void mma_tri(f32x4 (&c)[C / 16], const Frag<NP> (&f)[C / 16], int ks, const Frag<NB>& b) {
#pragma unroll
  for (int i = 0; i < NP; ++i)
#pragma unroll
    for (int j = 0; j < NB && i + j < NP; ++j)
#pragma unroll
      for (int t = 0; t < C / 16; ++t)
        if (tri_has<UP, C>(t, ks)) c[t] = mfma(f[t].p[i], b.p[j], c[t]);
}

// The record of one head's chunk: the parts of T = (I + A)^-1 and of P = scale
// M o QK^T (backward: T, its transpose and that of P), then the decays
//   from[i] = e^{G_i}, to[i] = e^{G_end - G_i}, beta[i], scale from[i]
// (1 KB). From the first token on whose key, decay or strength is not finite
// beta is NaN and T the identity.
template <int C>
struct Record {
  static constexpr int T = 0;
  static constexpr int P = tri_frags<C>() * 3 * kFrag;           // backward: T transposed
  static constexpr int PT = 2 * P;                               // backward only
  static constexpr int decays(bool backward) { return (backward ? 3 : 2) * P; }
  static constexpr int bytes(bool backward) { return decays(backward) + kFrag; }
};

// What the kernels share for an io type and padded features of a key (KP = 64
// or 128): parts of k and q (NI), tiles of 16 and steps of 32 tokens (MT, CS) and
// features (KT, KS), bytes of the fragments of k or q of a chunk.
template <bool BF16, int KP>
struct Shape {
  static constexpr int C = chunk_of<BF16>();
  static constexpr int NI = BF16 ? 1 : 3;
  static constexpr int KS = KP / 32, KT = KP / 16, MT = C / 16, CS = C / 32;
  static constexpr int kMat = MT * KS * NI * kFrag;
  static constexpr int es = BF16 ? 2 : 4;
  // Fragments of a key head's chunk in the workspace: by columns k and (backward)
  // q, which the gradients read; float32 io also by rows k and q, made by a
  // kernel of their own. The copying waves of the chains take q and k of bf16 io
  // from the call's arrays (16 us less for 128 sequence heads of 2048 tokens than
  // through fragments), but splitting float32 would hold up the waves they share
  // a SIMD with (5 x 333 tokens of 4 heads: 42 us instead of 36).
  static constexpr int frags(bool back) { return ((back ? 2 : BF16 ? 0 : 1) + (BF16 ? 0 : 2)) * kMat; }
  static constexpr int k_rows(bool back) { return (back ? 2 : 1) * kMat; }
  static constexpr int q_rows(bool back) { return k_rows(back) + kMat; }
};

// Blocks of a chunk's k and q on their way from memory to fragments in LDS, one
// or more for each of N threads (`id`).
template <bool BF16, int KP, int N>
struct Stage {
  using Z = Shape<BF16, KP>;
  static constexpr int kBlocks = (Z::C / 4) * (KP / 8), kJobs = (kBlocks + N - 1) / N;
  Block<BF16> b[kJobs];

  // tokens [tok, tok + rows) of head `hk`
  __device__ __forceinline__ void load(const DeltaArgs& a, const void* p, int64_t stride, int64_t tok, int rows, int hk, int id, bool vec) {
    const int ld = row_bytes(stride, Z::es);
    const Buf buf = rows_buf(static_cast<const char*>(p) + (tok * stride + static_cast<int64_t>(hk) * a.Dk) * Z::es, rows, ld, a.Dk * Z::es);
#pragma unroll
    for (int j = 0; j < kJobs; ++j) {
      const int i = id + j * N, tg = i / (KP / 8), dg = i % (KP / 8);
      b[j] = load_block<BF16>(buf, block_offset<BF16>(tg, dg, ld, i < kBlocks ? a.Dk : 0), ld, a.Dk - 8 * dg, vec);
    }
  }
  // fragments by rows and by columns (null: without)
  __device__ __forceinline__ void store(unsigned char* rows, unsigned char* cols, int id) const {
#pragma unroll
    for (int j = 0; j < kJobs; ++j) {
      const int i = id + j * N, tg = i / (KP / 8), dg = i % (KP / 8);
      if (i < kBlocks) {
        const Parts<BF16> p(b[j]);
        if (rows != nullptr) store_rows<BF16, Z::KS>(rows, p, tg, dg);
        if (cols != nullptr) store_cols<BF16, Z::C>(cols, p, tg, dg);
      }
    }
  }
};

// The same for 16 NW columns of y's gradient in bf16, as fragments by columns: those
// are the accumulators' order, and operands as they are. Loaded element by
// element by the waves that need them, and v's gradient stored that way, the
// backward chain of 64 heads of 2048 tokens took 187 us instead of 169; float32
// in this way took longer (14 -> 21 us for 8 heads of 777 tokens): its chunks are
// shorter than the loads take.
template <int NW>
struct ValueStage {
  static constexpr int C = chunk_of<true>(), kWave = 32 * C, kBytes = NW * kWave, kBlocks = C / 4 * 2 * NW;
  Block<true> b;

  // rows [0, rows) of `ld` bytes from p, `dims` features from there on
  __device__ __forceinline__ void load(const void* p, int ld, int rows, int dims, int id, bool vec) {
    const int tg = id / (2 * NW), dg = id % (2 * NW);
    b = load_block<true>(rows_buf(p, rows, ld, dims * 2), block_offset<true>(tg, dg, ld, id < kBlocks ? dims : 0), ld, dims - 8 * dg, vec);
  }
  __device__ __forceinline__ void store(unsigned char* dst, int id) const {
    if (id < kBlocks) store_cols<true, C>(dst, Parts<true>(b), id / (2 * NW), id % (2 * NW));
  }
};

// element of row 4 (l/16) + r of tile t (0, 1) of such a fragment
template <int NP>
__device__ __forceinline__ float element(const Frag<NP>& f, int t, int r) {
  const uint32_t w = word(__builtin_bit_cast(uint4, f.p[0]), 2 * t + (r >> 1));
  return __uint_as_float((r & 1) ? w & 0xffff0000u : w << 16);
}

// A wave's 16 columns of v's gradient through its 2 KB of the LDS to rows of `ld`
// bytes in 16-byte groups (o: this lane's byte of row l/2).
template <int MT>
__device__ __forceinline__ void store_values(unsigned char* mine, Buf r, int o, int ld, const f32x4 (&x)[MT]) {
  const int l = threadIdx.x & 63, g = l >> 4, m = l & 15;
  unsigned char* p = mine + 4 * g * 32 + m * 2;
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      unsigned char* q = p + (16 * t + i) * 32;
      const uint32_t w = round2(x[t][i], x[t][i + 1]);
      *reinterpret_cast<uint16_t*>(q) = static_cast<uint16_t>(w);
      *reinterpret_cast<uint16_t*>(q + 32) = static_cast<uint16_t>(w >> 16);
    }
#pragma unroll
  for (int j = 0; j < MT / 2; ++j) store16(r, o + j * 32 * ld, *reinterpret_cast<const f32x4*>(mine + j * 1024 + l * 16));
}

// whether whole 16-byte groups of k and q are aligned
__device__ __forceinline__ bool vectored(const DeltaArgs& a, bool bf16) {
  const int V = bf16 ? 8 : 4;
  return a.Dk % V == 0 && a.ldq % V == 0 && a.ldk % V == 0 &&
         ((reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k)) & 15u) == 0;
}

// ---- 1 KB blocks from global memory straight into LDS ------------------------------
typedef __attribute__((address_space(3))) void lds_void;

// blocks w, w + NW, ... of `bytes` (a multiple of 1 KB) at src to dst
template <int NW>
__device__ __forceinline__ void lds_copy(unsigned char* dst, const unsigned char* src, int bytes, int w) {
  const Buf r = __builtin_amdgcn_make_buffer_rsrc(const_cast<unsigned char*>(src), 0, bytes, kBufferWord3);
  const int l = threadIdx.x & 63;
#pragma unroll 4
  for (int o = w * kFrag; o < bytes; o += NW * kFrag)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(dst + o), 16, o + l * 16, 0, 0, 0);
}

// this wave's copies are there (a barrier by itself does not wait for them)
__device__ __forceinline__ void lds_copied() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// Barriers of kernels whose last kCopy waves do nothing but copy the next chunk
// into LDS (the waves that compute then have no such copy in flight, for which
// the compiler would wait before each of their LDS reads): they arrive when
// their copies are there, the others when their reads are done.
constexpr int kCopy = 4;
__device__ __forceinline__ void barrier_copied() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}
__device__ __forceinline__ void barrier_passed() {   // the copying waves', with copies under way
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}
__device__ __forceinline__ void barrier_read() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// a log decay below this is 0 as a float32 factor: sums of g stay finite with
// it in the place of -inf, without -inf - (-inf)
constexpr float kLeastDecay = -110.0f;

// inclusive sums over a wave's lanes: within rows of 16, then the last lane of
// a row to the next one and of the first half to the second
template <int CTRL, int ROWS>
__device__ __forceinline__ double lane_before(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(u), CTRL, ROWS, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(u >> 32), CTRL, ROWS, 0xf, false);
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);   // 0 where there is none
}
__device__ __forceinline__ double lane_sums(double s) {
  s += lane_before<0x111, 0xf>(s);   // row_shr 1, 2, 4, 8
  s += lane_before<0x112, 0xf>(s);
  s += lane_before<0x114, 0xf>(s);
  s += lane_before<0x118, 0xf>(s);
  s += lane_before<0x142, 0xa>(s);   // row_bcast 15, 31
  s += lane_before<0x143, 0xc>(s);
  return s;
}

// inclusive sums of g over a wave's lanes (one chunk), float64: their
// differences stay exact to float32 however fast a head forgets
__device__ __forceinline__ double chunk_sums(float g) { return lane_sums(g < kLeastDecay ? kLeastDecay : g); }

// e^x for the factors M_ij <= 1 of products: the hardware's exponential of
// x log2(e), off by up to (1 + |x|) 2^-24 of e^x and so by less than 2^-23 of
// the factor of neighbours, which the small ones are added to
__device__ __forceinline__ float decay_exp(double x) { return __expf(static_cast<float>(x)); }

__device__ __forceinline__ int length_of(const DeltaArgs& a, int b) {
  if (a.lengths == nullptr) return a.L;
  const int n = __builtin_amdgcn_readfirstlane(a.lengths[b]);
  return n < 0 ? 0 : n > a.L ? a.L : n;
}

}  // namespace delta
}  // namespace s5
