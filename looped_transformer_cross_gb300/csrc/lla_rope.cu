// lla_rope.cu — RoPE as operators of its own: tables built on the GPU, with the
// frequencies of long-context scalings, and the rotation of part of each head's
// vector (lla_rope_table_scaled, lla_rope_apply).
//
// The rotation of the LLA paper's §3 "RoPE and reconstruction" is the one that the
// decode kernels fuse; these calls serve what runs beside them: the exact attention of
// a prefill, the consumers of the window's keys, and the codec's training, whose
// gradient is the inverse rotation.
#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <utility>

#include "lla_kernels.h"

using namespace lla;

namespace {

// ----------------------------------------------------------------- table

constexpr int kMaxHalf = 128;         // frequencies of a row
constexpr int kTableThreads = 256;
constexpr int kTableRows = 16;        // rows of a thread at most

// Angular steps per position in turns, as 64-bit fixed-point fractions: position p
// sits at p * turn mod 2^64, an exact integer product, so a far position loses no more
// than p times the rounding of its frequency in fp64 (an fp32 angle would, and fp64 arithmetic is slow here).
struct TurnArgs {
  uint64_t turn[kMaxHalf];
  int half;
  int64_t pos0, n_pos;
  int rows;                           // rows of a thread
  float* cos_out;
  float* sin_out;
};

// cos and sin of phase / 2^64 turns.  The nearest quarter turn is taken off in integers,
// so what is left is at most an eighth of a turn u and its fp32 rounding is relative to
// it: values next to a zero of either function keep their digits.  u is put together from 23
// and 32 of its bits (a conversion of all 64 is slow).  The Taylor series of sin 2 pi u and
// cos 2 pi u to u^9 and u^10 are within 2^-28 of the functions there; in fp32, with 2 pi in two parts,
// both come out within 1.3 * 2^-24.  (131072 rows of 64: 16.4 us; with sincospif and a 64-bit
// conversion 26.6, bound by issuing instructions.)
__device__ __forceinline__ void cos_sin_turns(uint64_t phase, float& c, float& s) {
  const uint32_t top = static_cast<uint32_t>(phase >> 32), quarter = (top + 0x20000000u) >> 30;
  const uint32_t rest = top - (quarter << 30);   // its low word is the phase's
  const int high = static_cast<int>(rest) >> 7;  // |high| <= 2^22: 1.5 * 2^23 + high is its own fp32 encoding
  const uint32_t mid = __funnelshift_r(static_cast<uint32_t>(phase), rest, 7);
  const float u = fmaf(__int_as_float(0x4B400000 + high) - 12582912.f, 2.98023224e-8f,            // 2^-25
                       __uint2float_rn(mid) * 6.93889390e-18f);                                   // 2^-57
  const float v = u * u;
  float p = fmaf(42.058693f, v, -76.70586f);
  p = fmaf(p, v, 81.60525f);
  p = fmaf(p, v, -41.3417f);
  const float sr = fmaf(u, 6.2831855f, u * fmaf(p, v, -1.7484555e-7f));
  p = fmaf(-26.426256f, v, 60.24464f);
  p = fmaf(p, v, -85.45682f);
  p = fmaf(p, v, 64.93939f);
  const float cr = fmaf(fmaf(p, v, -19.739208f), v, 1.f);
  const bool odd = quarter & 1;
  c = __uint_as_float(__float_as_uint(odd ? sr : cr) ^ ((quarter + 1) & 2) << 30);
  s = __uint_as_float(__float_as_uint(odd ? cr : sr) ^ (quarter & 2) << 30);
}

// A thread takes VEC frequencies of every rows-per-block-th row of its block's stretch.
template <int VEC>
__global__ void __launch_bounds__(kTableThreads) rope_table_kernel(const __grid_constant__ TurnArgs a) {
  const int per_row = a.half / VEC;                       // threads of a row
  const int rows = kTableThreads / per_row;               // rows of the block at a time
  const int r = threadIdx.x / per_row, f = (threadIdx.x % per_row) * VEC;
  if (r >= rows) return;
  int64_t p = static_cast<int64_t>(blockIdx.x) * rows * a.rows + r;
  uint64_t phase[VEC], step[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    const uint64_t t = a.turn[f + e];
    phase[e] = static_cast<uint64_t>(a.pos0 + p) * t;
    step[e] = static_cast<uint64_t>(rows) * t;
  }
  for (int i = 0; i < a.rows && p < a.n_pos; ++i, p += rows) {
    float c[VEC], s[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      cos_sin_turns(phase[e], c[e], s[e]);
      phase[e] += step[e];
    }
    float* co = a.cos_out + p * a.half + f;
    float* so = a.sin_out + p * a.half + f;
    if constexpr (VEC == 4) {
      *reinterpret_cast<float4*>(co) = make_float4(c[0], c[1], c[2], c[3]);
      *reinterpret_cast<float4*>(so) = make_float4(s[0], s[1], s[2], s[3]);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) { co[e] = c[e]; so[e] = s[e]; }
    }
  }
}

// Frequencies of lla_rope_scaling in turns per position; false for values no scaling takes.
bool turns_of(const lla_dims* dims, const lla_rope_scaling* sc, TurnArgs* a) {
  const int d = dims->d_head, half = d / 2;
  double base = dims->rope_base;
  const int kind = sc ? sc->kind : LLA_ROPE_PLAIN;
  if (kind == LLA_ROPE_BASE) {
    if (d < 4) return false;
    base *= std::pow(sc->factor, static_cast<double>(d) / (d - 2));
  }
  const double two_pi = 6.283185307179586476925286766559;
  for (int f = 0; f < half; ++f) {
    double theta = std::pow(base, -2.0 * f / d);
    if (kind == LLA_ROPE_LINEAR) theta /= sc->factor;
    if (kind == LLA_ROPE_BY_PARTS) {
      double g = (static_cast<double>(sc->original_len) * theta / two_pi - sc->slow) / (sc->fast - sc->slow);
      g = g < 0 ? 0 : (g > 1 ? 1 : g);
      theta = (1 - g) * theta / sc->factor + g * theta;
    }
    const double t = theta / two_pi;
    if (!(t > 0) || !std::isfinite(t)) return false;   // a factor that drove theta out of range
    const double frac = t - std::floor(t);
    a->turn[f] = frac >= 1 ? 0 : static_cast<uint64_t>(std::ldexp(frac, 64));
  }
  return true;
}

// ----------------------------------------------------------------- rotation

constexpr int kApplyThreads = 128;
// Heads of a thread whose loads are in flight together (two 16-byte loads, 16 cosines and sines a head
// take the registers of two).
constexpr int kCopyHeads = 4;
__host__ __device__ constexpr int apply_heads(int vec, int style) { return style == 0 && vec == 8 ? 2 : 4; }

struct ApplyArgs {
  const void* x;
  void* out;
  int64_t x_tok, x_head, out_tok, out_head;   // strides in elements
  int offset, half;
  struct Deal {                               // a block's share: items of a token-head x strips x tokens
    FastDiv items, strips;                    // strips: threads that share a token's heads
    int toks;
  } deal[2];                                  // of rotated items, of copied ones
  int rot_items, n_items;                     // per token-head: rotated items, all
  unsigned rot_blocks;                        // blocks (x) of rotated items; copied ones follow
  int first;                                  // column of the first item (interleaved vectors)
  int heads;
  int64_t N;
  const int32_t* pos;
  const float* rope_cos;                      // [rope_len][half]
  const float* rope_sin;
  int64_t rope_len;
  float scale, sign;                          // sign -1: the inverse rotation
  uint32_t* status;
};

template <typename T, int N>
struct alignas(N * sizeof(T) < 16 ? N * sizeof(T) : 16) Vec {
  T v[N];
};

template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// One item = VEC rotation pairs of a token-head (two 16-byte loads and stores where
// VEC * sizeof(T) == 16), or VEC elements outside the rotated part, copied when the call
// is not in place.  Interleaved pairs lie within 16 bytes: there an item is one such vector, rotated or
// copied, in the order of the columns.  A thread keeps its item and token, and with them its
// position, cosines and sines, for two or four heads at a time, whose loads are all
// under way before the first is used.  (One item a thread, with its divisions and
// addresses, took 177 instructions per warp and was bound by issuing them; rotated and copied
// items in one warp take turns: 32768 x 16 vectors of 192, last 64 in half layout: 182 us, in blocks
// of their own and with 64 registers a thread 70.  An evict-first hint on the loads: 74.)  HBM-bound:
// each element is read and written once.  fp32 arithmetic, one rounding to the storage type.
template <typename T, int VEC, int kStyle>
__global__ void __launch_bounds__(kApplyThreads, 8) rope_apply_kernel(const __grid_constant__ ApplyArgs a) {
  constexpr bool kWhole = kStyle == 1 && VEC > 1;          // an item's pairs are one vector's
  constexpr int kHeads = apply_heads(VEC, kStyle);
  constexpr int kPairs = kWhole ? VEC / 2 : VEC;
  using V = Vec<T, VEC>;
  using F = Vec<float, kPairs>;
  // (rotated and copied items in blocks of their own: no warp has both)
  const bool copy = !kWhole && blockIdx.x >= a.rot_blocks;
  const ApplyArgs::Deal& D = a.deal[copy];
  const uint32_t slot = D.items.div(threadIdx.x), ts = D.strips.div(slot);
  const int item = (copy ? a.rot_items : 0) + static_cast<int>(blockIdx.y * D.items.d + threadIdx.x - slot * D.items.d);
  const int64_t n = static_cast<int64_t>(copy ? blockIdx.x - a.rot_blocks : blockIdx.x) * D.toks + ts;
  if (static_cast<int>(ts) >= D.toks || n >= a.N || item >= (kWhole || copy ? a.n_items : a.rot_items)) return;
  // the item's columns: i0, and of a split pair i1
  int i0, i1 = 0, f = -1;
  if constexpr (kWhole) {
    i0 = a.first + item * VEC;
    if (i0 >= a.offset && i0 < a.offset + 2 * a.half) f = (i0 - a.offset) / 2;
  } else if (!copy) {
    f = item * VEC;
    i0 = a.offset + (kStyle == 0 ? f : 2 * f);
    i1 = kStyle == 0 ? i0 + a.half : i0 + 1;
  } else {
    i0 = (item - a.rot_items) * VEC;
    if (i0 >= a.offset) i0 += 2 * a.half;
  }
  F c, s;
  if (f >= 0) {
    int p = __ldg(a.pos + n);
    if (p < 0 || p >= a.rope_len) {
      record_status(a.status, LLA_ERR_DEVICE_ARG);
      p = p < 0 ? 0 : static_cast<int>(a.rope_len - 1);
    }
    c = *reinterpret_cast<const F*>(a.rope_cos + static_cast<int64_t>(p) * a.half + f);
    s = *reinterpret_cast<const F*>(a.rope_sin + static_cast<int64_t>(p) * a.half + f);
#pragma unroll
    for (int e = 0; e < kPairs; ++e) s.v[e] *= a.sign;
  }
  int h = static_cast<int>(slot - ts * D.strips.d);
  const T* x = static_cast<const T*>(a.x) + n * a.x_tok + h * a.x_head + i0;
  T* out = static_cast<T*>(a.out) + n * a.out_tok + h * a.out_head + i0;
  const int strips = static_cast<int>(D.strips.d);
  const int64_t x_step = strips * a.x_head, out_step = strips * a.out_head;
  if (copy) {
    for (; h < a.heads; h += kCopyHeads * strips, x += kCopyHeads * x_step, out += kCopyHeads * out_step) {
      V u[kCopyHeads];
#pragma unroll
      for (int k = 0; k < kCopyHeads; ++k)
        if (h + k * strips < a.heads) u[k] = *reinterpret_cast<const V*>(x + k * x_step);
#pragma unroll
      for (int k = 0; k < kCopyHeads; ++k)
        if (h + k * strips < a.heads) *reinterpret_cast<V*>(out + k * out_step) = u[k];
    }
    return;
  }
  for (; h < a.heads; h += kHeads * strips) {
    V u[kHeads], w[kHeads];
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      if (h + k * strips >= a.heads) continue;
      u[k] = *reinterpret_cast<const V*>(x + k * x_step);
      if (!kWhole && f >= 0) w[k] = *reinterpret_cast<const V*>(x + k * x_step + (i1 - i0));
    }
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      if (h + k * strips >= a.heads) continue;
      if (f >= 0) {
#pragma unroll
        for (int e = 0; e < kPairs; ++e) {
          T& y0 = u[k].v[kWhole ? 2 * e : e];
          T& y1 = kWhole ? u[k].v[2 * e + 1] : w[k].v[e];
          const float x0 = to_f32<T>(y0), x1 = to_f32<T>(y1);
          y0 = from_f32<T>((x0 * c.v[e] - x1 * s.v[e]) * a.scale);
          y1 = from_f32<T>((x0 * s.v[e] + x1 * c.v[e]) * a.scale);
        }
        if (!kWhole) *reinterpret_cast<V*>(out + k * out_step + (i1 - i0)) = w[k];
      }
      *reinterpret_cast<V*>(out + k * out_step) = u[k];
    }
    x += kHeads * x_step;
    out += kHeads * out_step;
  }
}

template <typename T, int VEC>
cudaError_t launch_apply(ApplyArgs a, int style, cudaStream_t s) {
  const int copied = style != LLA_ROPE_HALF && VEC > 1 ? 0 : a.n_items - a.rot_items;
  auto blocks = [&](const ApplyArgs::Deal& d) { return static_cast<unsigned>((a.N + d.toks - 1) / d.toks); };
  a.rot_blocks = blocks(a.deal[0]);
  auto chunks = [](int n, const ApplyArgs::Deal& d) { return (n + d.items.d - 1) / d.items.d; };
  const int turned = a.n_items - copied;
  const dim3 grid(a.rot_blocks + (copied ? blocks(a.deal[1]) : 0),
                  std::max(chunks(turned, a.deal[0]), copied ? chunks(copied, a.deal[1]) : 0));
  if (style == LLA_ROPE_HALF) rope_apply_kernel<T, VEC, 0><<<grid, kApplyThreads, 0, s>>>(a);
  else rope_apply_kernel<T, VEC, 1><<<grid, kApplyThreads, 0, s>>>(a);
  return cudaGetLastError();
}

// Whether rows of d elements at i s + j t (i < n, j < m) keep clear of the same rows `gap` >= 0 elements on.  The
// rows of either set keep clear of each other (checked before), so with s <= t all rows of one j lie
// within t - d of its first, and only the two j around gap / t can come near; of these the two i.
bool rows_apart(int64_t gap, int64_t s, int64_t n, int64_t t, int64_t m, int64_t d) {
  if (n == 1) { s = t; n = m; m = 1; }
  if (m > 1 && s > t) { std::swap(s, t); std::swap(n, m); }
  const int64_t j0 = m > 1 ? std::min(gap / t, m - 1) : 0;
  for (int64_t j = j0; j < std::min(j0 + 2, m); ++j) {
    const int64_t r = std::abs(gap - (m > 1 ? j * t : 0)), i0 = n > 1 ? std::min(r / s, n - 1) : 0;
    for (int64_t i = i0; i < std::min(i0 + 2, n); ++i)
      if (std::abs(r - (n > 1 ? i * s : 0)) < d) return false;
  }
  return true;
}

}  // namespace

extern "C" {

lla_status lla_rope_table_scaled(const lla_dims* dims, const lla_rope_scaling* scaling, int64_t pos0, int64_t n_pos,
                                 float* rope_cos, float* rope_sin, void* stream) {
  if (!dims || dims->d_head < 2 || dims->d_head % 2 || !(dims->rope_base > 0.f) || !std::isfinite(dims->rope_base) ||
      n_pos < 0 || pos0 < 0)
    return LLA_ERR_INVALID_ARG;
  if (scaling) {
    if (scaling->kind < LLA_ROPE_PLAIN || scaling->kind > LLA_ROPE_BY_PARTS) return LLA_ERR_INVALID_ARG;
    if (scaling->kind != LLA_ROPE_PLAIN && !(scaling->factor > 0 && std::isfinite(scaling->factor)))
      return LLA_ERR_INVALID_ARG;
    if (scaling->kind == LLA_ROPE_BY_PARTS &&
        (scaling->original_len < 1 || !(scaling->slow >= 0) || !(scaling->fast > scaling->slow) ||
         !std::isfinite(scaling->fast)))
      return LLA_ERR_INVALID_ARG;
  }
  if (dims->d_head > 2 * kMaxHalf || n_pos > (int64_t(1) << 31) || pos0 > (int64_t(1) << 31)) return LLA_ERR_UNSUPPORTED;
  TurnArgs a{};
  if (!turns_of(dims, scaling, &a)) return LLA_ERR_INVALID_ARG;
  if (n_pos == 0) return LLA_OK;
  for (const void* p : {static_cast<const void*>(rope_cos), static_cast<const void*>(rope_sin)})
    if (!p || (reinterpret_cast<uintptr_t>(p) & 15u)) return LLA_ERR_INVALID_ARG;
  a.half = dims->d_head / 2;
  a.pos0 = pos0;
  a.n_pos = n_pos;
  a.cos_out = rope_cos;
  a.sin_out = rope_sin;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int vec = a.half % 4 == 0 ? 4 : 1;
  // a thread's frequencies are set up once for several rows, as long as every SM has four blocks
  const int64_t at_once = kTableThreads / (a.half / vec), sms = device_sm_count();
  if (sms <= 0) return LLA_ERR_CUDA;
  a.rows = static_cast<int>(std::min<int64_t>(kTableRows, std::max<int64_t>(1, n_pos / (at_once * 4 * sms))));
  const unsigned blocks = static_cast<unsigned>((n_pos + at_once * a.rows - 1) / (at_once * a.rows));
  if (vec == 4) rope_table_kernel<4><<<blocks, kTableThreads, 0, s>>>(a);
  else rope_table_kernel<1><<<blocks, kTableThreads, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? LLA_OK : LLA_ERR_CUDA;
}

lla_status lla_rope_apply(const lla_dims* dims, const void* x, int64_t x_tok_stride, int64_t x_head_stride, void* out,
                          int64_t out_tok_stride, int64_t out_head_stride, int N, int heads, int d_x, int offset,
                          int d_rope, const int32_t* pos, const float* rope_cos, const float* rope_sin,
                          int64_t rope_len, float scale, int inverse, void* workspace, size_t ws_bytes, void* stream) {
  if (!dims || (dims->dtype != LLA_BF16 && dims->dtype != LLA_F32) ||
      (dims->rope_style != LLA_ROPE_HALF && dims->rope_style != LLA_ROPE_INTERLEAVED))
    return LLA_ERR_INVALID_ARG;
  if (N < 0 || heads < 1 || d_x < 1 || offset < 0 || d_rope < 2 || d_rope % 2 || d_rope > d_x || offset > d_x - d_rope ||
      rope_len < 1)
    return LLA_ERR_INVALID_ARG;
  // rows of one token-head are contiguous; rows of different ones must not overlap
  // (their order of writing is not defined)
  if (x_tok_stride < 0 || x_head_stride < 0 || out_tok_stride < 0 || out_head_stride < 0) return LLA_ERR_INVALID_ARG;
  if (heads > 1 && out_head_stride < d_x) return LLA_ERR_INVALID_ARG;
  if (N > 1 && (out_tok_stride < d_x || (out_head_stride < out_tok_stride
                                             ? out_tok_stride < (heads - 1) * out_head_stride + d_x
                                             : heads > 1 && out_head_stride < (N - 1) * out_tok_stride + d_x)))
    return LLA_ERR_INVALID_ARG;
  if (heads > (1 << 20) || d_x > (1 << 16)) return LLA_ERR_UNSUPPORTED;
  if (N == 0) return LLA_OK;
  const size_t es = dims->dtype == LLA_BF16 ? 2 : 4;
  const uintptr_t xa = reinterpret_cast<uintptr_t>(x), oa = reinterpret_cast<uintptr_t>(out);
  if (!xa || !oa || xa % es || oa % es || ws_bytes < 256) return LLA_ERR_INVALID_ARG;
  const void* ptrs[] = {pos, rope_cos, rope_sin, workspace};
  for (const void* p : ptrs)
    if (!p || (reinterpret_cast<uintptr_t>(p) & 3u)) return LLA_ERR_INVALID_ARG;
  const bool in_place = x == out;
  if (in_place && ((N > 1 && x_tok_stride != out_tok_stride) || (heads > 1 && x_head_stride != out_head_stride)))
    return LLA_ERR_INVALID_ARG;
  if (!in_place) {
    // ranges that overlap without being the same tensor would be read after they are written
    const uintptr_t xe = xa + es * ((N - 1) * x_tok_stride + (heads - 1) * x_head_stride + d_x);
    const uintptr_t oe = oa + es * ((N - 1) * out_tok_stride + (heads - 1) * out_head_stride + d_x);
    // interleaved slices of one buffer (q and k of a fused projection) overlap as ranges but
    // not as rows: allowed when both have the same strides and no row meets another
    const bool same = (N == 1 || x_tok_stride == out_tok_stride) && (heads == 1 || x_head_stride == out_head_stride);
    const int64_t gap = static_cast<int64_t>((xa > oa ? xa - oa : oa - xa) / es);
    if (xa < oe && oa < xe && !(same && rows_apart(gap, out_tok_stride, N, out_head_stride, heads, d_x)))
      return LLA_ERR_INVALID_ARG;
  }
  ApplyArgs a{};
  a.x = x;
  a.out = out;
  a.x_tok = x_tok_stride;
  a.x_head = x_head_stride;
  a.out_tok = out_tok_stride;
  a.out_head = out_head_stride;
  a.offset = offset;
  a.half = d_rope / 2;
  a.pos = pos;
  a.rope_cos = rope_cos;
  a.rope_sin = rope_sin;
  a.rope_len = rope_len;
  a.scale = scale;
  a.sign = inverse ? -1.f : 1.f;
  a.status = static_cast<uint32_t*>(workspace);
  // 16-byte items where every address they touch allows it, else single elements
  const int wide = static_cast<int>(16 / es);
  const uintptr_t all = static_cast<uintptr_t>(offset | a.half | d_x) |
                        static_cast<uintptr_t>(N > 1 ? x_tok_stride | out_tok_stride : 0) |
                        static_cast<uintptr_t>(heads > 1 ? x_head_stride | out_head_stride : 0);
  const bool vec = ((xa | oa | reinterpret_cast<uintptr_t>(rope_cos) | reinterpret_cast<uintptr_t>(rope_sin)) & 15u) == 0 &&
                   all % wide == 0;
  const int V = vec ? wide : 1;
  a.rot_items = a.half / V;
  a.n_items = a.rot_items + (in_place ? 0 : (d_x - d_rope) / V);
  if (vec && dims->rope_style == LLA_ROPE_INTERLEAVED) {
    a.first = in_place ? offset : 0;
    a.n_items = (in_place ? d_rope : d_x) / V;
  }
  a.heads = heads;
  a.N = N;
  const bool whole = vec && dims->rope_style == LLA_ROPE_INTERLEAVED;
  auto deal = [&](int n, int per) {   // n items of a token-head, per heads of a thread at a time
    const int items = std::min(n, kApplyThreads), at_once = kApplyThreads / items;
    const int strips = std::min((heads + per - 1) / per, at_once);
    return ApplyArgs::Deal{FastDiv(items), FastDiv(strips), at_once / strips};
  };
  a.deal[0] = deal(whole ? a.n_items : a.rot_items, apply_heads(V, dims->rope_style == LLA_ROPE_HALF ? 0 : 1));
  a.deal[1] = deal(std::max(1, a.n_items - a.rot_items), kCopyHeads);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dims->dtype == LLA_BF16)
    e = vec ? launch_apply<__nv_bfloat16, 8>(a, dims->rope_style, s) : launch_apply<__nv_bfloat16, 1>(a, dims->rope_style, s);
  else
    e = vec ? launch_apply<float, 4>(a, dims->rope_style, s) : launch_apply<float, 1>(a, dims->rope_style, s);
  return e == cudaSuccess ? LLA_OK : LLA_ERR_CUDA;
}

}  // extern "C"
