// C ABI of the gated delta rule and of the query/key norm and rotation:
// host-side validation and dispatch. See include/s5.h for the contracts.
#include "s5.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "s5_delta.h"

namespace {

struct Range {
  uintptr_t lo = 0, hi = 0;  // [lo, hi); empty without an array
};

Range range_of(const void* p, int64_t bytes) {
  if (p == nullptr || bytes <= 0) return {};
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return {lo, lo + static_cast<uintptr_t>(bytes)};
}

bool overlaps(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// any output over an input or over another output
template <int NI, int NO>
bool any_overlap(const Range (&ins)[NI], const Range (&outs)[NO]) {
  for (int i = 0; i < NO; ++i) {
    for (const Range& r : ins)
      if (overlaps(outs[i], r)) return true;
    for (int j = i + 1; j < NO; ++j)
      if (overlaps(outs[i], outs[j])) return true;
  }
  return false;
}

// bytes from the first to the last element of `rows` rows of `width` elements
int64_t span(int64_t rows, int64_t stride, int64_t width, int64_t es) {
  return rows > 0 ? ((rows - 1) * stride + width) * es : 0;
}

// whether `rows` rows, `stride` elements apart, are farther apart than offsets reach
bool far(int64_t stride, int64_t rows) { return rows > 0 && stride > (int64_t{1} << 55) / rows; }

s5_status delta_sizes(int64_t B, int64_t L, int64_t Hk, int64_t Hv, int64_t Dk, int64_t Dv, s5_dtype io,
                      int64_t ldq, int64_t ldk, int64_t ldv, float scale) {
  if (B < 0 || L < 0 || Hk < 1 || Hv < 1 || Dk < 1 || Dv < 1) return S5_ERR_INVALID_ARGUMENT;
  if (Dk > S5_DELTA_MAX_DK || Dv > S5_DELTA_MAX_DV) return S5_ERR_UNSUPPORTED;
  if (io != S5_F32 && io != S5_BF16) return S5_ERR_UNSUPPORTED;
  if (Hv % Hk != 0 || !std::isfinite(scale)) return S5_ERR_INVALID_ARGUMENT;
  if (Hv > INT32_MAX / Dv || Hk > INT32_MAX / Dk) return S5_ERR_UNSUPPORTED;
  if (ldq < Hk * Dk || ldk < Hk * Dk || ldv < Hv * Dv) return S5_ERR_INVALID_ARGUMENT;
  constexpr int64_t kMost = s5::kMostStride;   // a chunk's rows stay below 2^30 bytes
  if (Hv * Dv > kMost || Hk * Dk > kMost) return S5_ERR_UNSUPPORTED;
  // the tokens of several steps; one step of each sequence is a row of its own, any
  // distance from the next one's
  if (L > 1 && (ldq > kMost || ldk > kMost || ldv > kMost)) return S5_ERR_UNSUPPORTED;
  if (B > 0 && (L > INT32_MAX / B || Hv * Dv > INT32_MAX / B)) return S5_ERR_UNSUPPORTED;
  if (far(ldq, B * L) || far(ldk, B * L) || far(ldv, B * L)) return S5_ERR_UNSUPPORTED;
  // A launch has fewer than 2^32 threads: 256 for each chunk of 32 or 64 steps and
  // head, and for each head up to 8 column groups of 512 (the chains) or 16 of 256
  // (the single step)
  constexpr int64_t kChunks = (int64_t{1} << 24) - 1, kHeads = (int64_t{1} << 19) - 1;
  if (B > 0 && (Hv > kHeads / B || (L + 31) / 32 > kChunks / (B * Hv))) return S5_ERR_UNSUPPORTED;
  return S5_OK;
}

s5::DeltaArgs delta_args(const s5_delta_desc& x) {
  s5::DeltaArgs a{};
  a.B = static_cast<int>(x.B);
  a.L = static_cast<int>(x.L);
  a.Hk = static_cast<int>(x.Hk);
  a.Hv = static_cast<int>(x.Hv);
  a.Nk = a.Hk;
  a.Nv = a.Hv;
  a.Dk = static_cast<int>(x.Dk);
  a.Dv = static_cast<int>(x.Dv);
  a.ldq = x.q_stride;
  a.ldk = x.k_stride;
  a.ldv = x.v_stride;
  a.bf16_io = x.io == S5_BF16;
  a.scale = x.scale;
  a.q = x.q;
  a.k = x.k;
  a.v = x.v;
  a.g = x.g;
  a.beta = x.beta;
  a.s0 = x.s0;
  a.lengths = x.lengths;
  a.y = x.y;
  a.s_last = x.s_last;
  a.ws = x.workspace;
  a.dy = x.dy;
  a.ds_last = x.ds_last;
  a.dq = x.dq;
  a.dk = x.dk;
  a.dv = x.dv;
  a.dg = x.dg;
  a.dbeta = x.dbeta;
  a.ds0 = x.ds0;
  return a;
}

s5_status delta_check(const s5_delta_desc* x) {
  if (x == nullptr || x->size != sizeof(s5_delta_desc)) return S5_ERR_INVALID_ARGUMENT;
  return delta_sizes(x->B, x->L, x->Hk, x->Hv, x->Dk, x->Dv, x->io, x->q_stride, x->k_stride, x->v_stride, x->scale);
}

int64_t delta_workspace(const s5_delta_desc& x, bool backward) {
  if (x.B == 0 || x.L == 0) return 0;
  return s5::delta_workspace(delta_args(x), backward);
}

s5_status run_delta(const s5_delta_desc* x, bool backward, hipStream_t stream) {
  s5_status st = delta_check(x);
  if (st != S5_OK) return st;
  const int64_t T = x->B * x->L;
  const int64_t es = x->io == S5_BF16 ? 2 : 4;
  const int64_t qk = T * x->Hk * x->Dk * es, vy = T * x->Hv * x->Dv * es, gb = T * x->Hv * 4;
  const int64_t state = x->B * x->Hv * x->Dk * x->Dv * 4;
  if (T > 0 && (!x->q || !x->k || !x->v || !x->g || !x->beta)) return S5_ERR_INVALID_ARGUMENT;
  if (T > 0 && !backward && !x->y) return S5_ERR_INVALID_ARGUMENT;
  if (T > 0 && backward && (!x->dy || !x->dq || !x->dk || !x->dv || !x->dg || !x->dbeta)) return S5_ERR_INVALID_ARGUMENT;
  const uintptr_t el = static_cast<uintptr_t>(es);
  if (!aligned(x->q, el) || !aligned(x->k, el) || !aligned(x->v, el) || !aligned(x->g, 4) || !aligned(x->beta, 4) ||
      !aligned(x->lengths, 4) || !aligned(x->s0, 16))
    return S5_ERR_UNSUPPORTED;
  if (backward) {
    const void* ptrs[] = {x->dy, x->ds_last, x->dq, x->dk, x->dv, x->dg, x->dbeta, x->ds0};
    for (const void* p : ptrs)
      if (!aligned(p, 16)) return S5_ERR_UNSUPPORTED;
  } else if (!aligned(x->y, 16) || !aligned(x->s_last, 16)) {
    return S5_ERR_UNSUPPORTED;
  }
  if (x->B == 0) return S5_OK;
  const int64_t need = delta_workspace(*x, backward);
  if (need > 0) {
    if (!x->workspace || x->workspace_bytes < need) return S5_ERR_INVALID_ARGUMENT;
    if (!aligned(x->workspace, 256)) return S5_ERR_UNSUPPORTED;
  }
  const Range ins[] = {range_of(x->q, span(T, x->q_stride, x->Hk * x->Dk, es)),
                       range_of(x->k, span(T, x->k_stride, x->Hk * x->Dk, es)),
                       range_of(x->v, span(T, x->v_stride, x->Hv * x->Dv, es)),
                       range_of(x->g, gb),
                       range_of(x->beta, gb),
                       range_of(!backward && x->s0 == x->s_last ? nullptr : x->s0, state),
                       range_of(x->lengths, x->B * 4),
                       range_of(backward ? x->dy : nullptr, vy),
                       range_of(backward ? x->ds_last : nullptr, state)};
  const Range ws = range_of(x->workspace, need);
  if (backward) {
    const Range outs[] = {range_of(x->dq, qk), range_of(x->dk, qk), range_of(x->dv, vy), range_of(x->dg, gb),
                          range_of(x->dbeta, gb), range_of(x->ds0, state), ws};
    if (any_overlap(ins, outs)) return S5_ERR_INVALID_ARGUMENT;
    return s5::launch_delta_backward(delta_args(*x), stream) == hipSuccess ? S5_OK : S5_ERR_HIP;
  }
  const Range outs[] = {range_of(x->y, vy), range_of(x->s_last, state), ws};
  if (any_overlap(ins, outs)) return S5_ERR_INVALID_ARGUMENT;
  return s5::launch_delta(delta_args(*x), stream) == hipSuccess ? S5_OK : S5_ERR_HIP;
}

s5_status qk_args(const s5_qk_desc* x, s5::QkArgs& a) {
  if (x == nullptr || x->size != sizeof(s5_qk_desc)) return S5_ERR_INVALID_ARGUMENT;
  const uint32_t norms = x->flags & (S5_QK_RMS | S5_QK_L2);
  if ((x->flags & ~static_cast<uint32_t>(S5_QK_RMS | S5_QK_L2 | S5_QK_INTERLEAVED)) != 0 ||
      norms == (S5_QK_RMS | S5_QK_L2))
    return S5_ERR_INVALID_ARGUMENT;
  if (x->T < 0 || x->L < 1 || x->Hq < 1 || x->Hk < 1 || x->D < 1) return S5_ERR_INVALID_ARGUMENT;
  if (x->R < 0 || x->R > x->D || x->R % 2 != 0) return S5_ERR_INVALID_ARGUMENT;
  if (x->D > S5_QK_MAX_D || (x->io != S5_F32 && x->io != S5_BF16)) return S5_ERR_UNSUPPORTED;
  if (x->Hq > INT32_MAX / 512 || x->Hk > INT32_MAX / 512 || x->T > INT32_MAX / (x->Hq + x->Hk)) return S5_ERR_UNSUPPORTED;
  if (x->q_stride < x->Hq * x->D || x->k_stride < x->Hk * x->D) return S5_ERR_INVALID_ARGUMENT;
  if (far(x->q_stride, x->T) || far(x->k_stride, x->T)) return S5_ERR_UNSUPPORTED;
  if (!std::isfinite(x->rope_scale)) return S5_ERR_INVALID_ARGUMENT;
  if (norms ? !(std::isfinite(x->eps) && x->eps > 0.0f) : (x->q_weight || x->k_weight)) return S5_ERR_INVALID_ARGUMENT;
  a = s5::QkArgs{};
  a.T = x->T;
  a.L = x->L;
  a.Hq = static_cast<int>(x->Hq);
  a.Hk = static_cast<int>(x->Hk);
  a.D = static_cast<int>(x->D);
  a.R = static_cast<int>(x->R);
  a.ldq = x->q_stride;
  a.ldk = x->k_stride;
  a.bf16_io = x->io == S5_BF16;
  a.interleaved = (x->flags & S5_QK_INTERLEAVED) != 0;
  a.norm = norms != 0;
  a.inv_m = norms == S5_QK_RMS ? 1.0f / static_cast<float>(x->D) : 1.0f;
  a.eps = x->eps;
  a.rope_scale = x->rope_scale;
  a.q = x->q;
  a.k = x->k;
  a.wq = x->q_weight;
  a.wk = x->k_weight;
  a.freqs = x->freqs;
  a.positions = x->positions;
  a.q_out = x->q_out;
  a.k_out = x->k_out;
  a.dq_out = x->dq_out;
  a.dk_out = x->dk_out;
  a.dwq = x->dq_weight;
  a.dwk = x->dk_weight;
  return S5_OK;
}

int64_t qk_workspace(const s5::QkArgs& a) {
  if (a.T == 0 || (!a.dwq && !a.dwk)) return 0;
  return static_cast<int64_t>(s5::qk_partial_blocks(a)) * 2 * a.D * 4;
}

s5_status run_qk(const s5_qk_desc* x, bool backward, hipStream_t stream) {
  s5::QkArgs a;
  s5_status st = qk_args(x, a);
  if (st != S5_OK) return st;
  if (backward && ((a.dwq && !a.wq) || (a.dwk && !a.wk))) return S5_ERR_INVALID_ARGUMENT;
  if (a.T > 0 && (!a.q || !a.k || !a.q_out || !a.k_out || (a.R > 0 && !a.freqs))) return S5_ERR_INVALID_ARGUMENT;
  if (a.T > 0 && backward && (!a.dq_out || !a.dk_out)) return S5_ERR_INVALID_ARGUMENT;
  const int64_t es = a.bf16_io ? 2 : 4;
  const uintptr_t el = static_cast<uintptr_t>(es);
  if (!aligned(a.q, el) || !aligned(a.k, el) || !aligned(a.wq, 16) || !aligned(a.wk, 16) || !aligned(a.freqs, 8) ||
      !aligned(a.positions, 4) || !aligned(a.q_out, 16) || !aligned(a.k_out, 16))
    return S5_ERR_UNSUPPORTED;
  if (backward && (!aligned(a.dq_out, 16) || !aligned(a.dk_out, 16) || !aligned(a.dwq, 16) || !aligned(a.dwk, 16)))
    return S5_ERR_UNSUPPORTED;
  const int64_t wq = static_cast<int64_t>(a.Hq) * a.D, wk = static_cast<int64_t>(a.Hk) * a.D;
  const int64_t need = backward ? qk_workspace(a) : 0;
  if (need > 0) {
    if (!x->workspace || x->workspace_bytes < need) return S5_ERR_INVALID_ARGUMENT;
    if (!aligned(x->workspace, 256)) return S5_ERR_UNSUPPORTED;
    a.partials = static_cast<float*>(x->workspace);
  }
  // a row is read whole before it is written, so a contiguous input may be its
  // own output, and a gradient of the results the place of the gradients
  const bool q_in_place = a.q == a.q_out && a.ldq == wq, k_in_place = a.k == a.k_out && a.ldk == wk;
  const Range ins[] = {range_of(q_in_place ? nullptr : a.q, span(a.T, a.ldq, wq, es)),
                       range_of(k_in_place ? nullptr : a.k, span(a.T, a.ldk, wk, es)),
                       range_of(a.wq, a.D * 4),
                       range_of(a.wk, a.D * 4),
                       range_of(a.R > 0 ? a.freqs : nullptr, a.R * 4),
                       range_of(a.positions, a.T * 4),
                       range_of(backward && a.dq_out != a.q_out ? a.dq_out : nullptr, a.T * wq * es),
                       range_of(backward && a.dk_out != a.k_out ? a.dk_out : nullptr, a.T * wk * es)};
  const Range outs[] = {range_of(a.q_out, a.T * wq * es), range_of(a.k_out, a.T * wk * es),
                        range_of(backward ? a.dwq : nullptr, a.D * 4), range_of(backward ? a.dwk : nullptr, a.D * 4),
                        range_of(need > 0 ? x->workspace : nullptr, need)};
  if (any_overlap(ins, outs)) return S5_ERR_INVALID_ARGUMENT;
  if (a.T == 0) {
    // no rows: the weights' gradients are empty sums
    if (!backward) return S5_OK;
    for (float* p : {a.dwq, a.dwk})
      if (p != nullptr && s5::launch_zero(p, a.D, stream) != hipSuccess) return S5_ERR_HIP;
    return S5_OK;
  }
  return s5::launch_qk(a, backward, stream) == hipSuccess ? S5_OK : S5_ERR_HIP;
}

}  // namespace

extern "C" {

s5_status s5_gated_delta_workspace(const s5_delta_desc* desc, int backward, int64_t* bytes) {
  const s5_status st = delta_check(desc);
  if (st != S5_OK) return st;
  if (bytes == nullptr) return S5_ERR_INVALID_ARGUMENT;
  *bytes = delta_workspace(*desc, backward != 0);
  return S5_OK;
}

s5_status s5_gated_delta(const s5_delta_desc* desc, hipStream_t stream) { return run_delta(desc, false, stream); }

s5_status s5_gated_delta_backward(const s5_delta_desc* desc, hipStream_t stream) { return run_delta(desc, true, stream); }

s5_status s5_gated_delta_step(int64_t B, int64_t Hk, int64_t Hv, int64_t Dk, int64_t Dv, s5_dtype io,
                              int64_t q_stride, int64_t k_stride, int64_t v_stride, float scale,
                              const void* q, const void* k, const void* v, const float* g,
                              const float* beta, float* s, void* y, hipStream_t stream) {
  const s5_status st = delta_sizes(B, 1, Hk, Hv, Dk, Dv, io, q_stride, k_stride, v_stride, scale);
  if (st != S5_OK) return st;
  if (B > 0 && (!q || !k || !v || !g || !beta || !s || !y)) return S5_ERR_INVALID_ARGUMENT;
  const int64_t es = io == S5_BF16 ? 2 : 4;
  const uintptr_t el = static_cast<uintptr_t>(es);
  if (!aligned(q, el) || !aligned(k, el) || !aligned(v, el) || !aligned(g, 4) || !aligned(beta, 4) || !aligned(s, 16) ||
      !aligned(y, 16))
    return S5_ERR_UNSUPPORTED;
  if (B == 0) return S5_OK;
  const Range ins[] = {range_of(q, span(B, q_stride, Hk * Dk, es)), range_of(k, span(B, k_stride, Hk * Dk, es)),
                       range_of(v, span(B, v_stride, Hv * Dv, es)), range_of(g, B * Hv * 4), range_of(beta, B * Hv * 4)};
  const Range outs[] = {range_of(s, B * Hv * Dk * Dv * 4), range_of(y, B * Hv * Dv * es)};
  if (any_overlap(ins, outs)) return S5_ERR_INVALID_ARGUMENT;
  s5::DeltaArgs a{};
  a.B = static_cast<int>(B);
  a.L = 1;
  a.Hk = static_cast<int>(Hk);
  a.Hv = static_cast<int>(Hv);
  a.Dk = static_cast<int>(Dk);
  a.Dv = static_cast<int>(Dv);
  a.ldq = q_stride;
  a.ldk = k_stride;
  a.ldv = v_stride;
  a.bf16_io = io == S5_BF16;
  a.scale = scale;
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.beta = beta;
  a.s0 = s;
  a.y = y;
  a.s_last = s;
  return s5::launch_delta_step(a, stream) == hipSuccess ? S5_OK : S5_ERR_HIP;
}

s5_status s5_qk_workspace(const s5_qk_desc* desc, int64_t* bytes) {
  s5::QkArgs a;
  const s5_status st = qk_args(desc, a);
  if (st != S5_OK) return st;
  if (bytes == nullptr) return S5_ERR_INVALID_ARGUMENT;
  *bytes = qk_workspace(a);
  return S5_OK;
}

s5_status s5_qk_norm_rope(const s5_qk_desc* desc, hipStream_t stream) { return run_qk(desc, false, stream); }

s5_status s5_qk_norm_rope_backward(const s5_qk_desc* desc, hipStream_t stream) { return run_qk(desc, true, stream); }

}  // extern "C"
