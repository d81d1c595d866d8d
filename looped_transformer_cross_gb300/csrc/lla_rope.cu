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

#include "lla_kernels.h"

using namespace lla;

namespace {

// ----------------------------------------------------------------- table

constexpr int kMaxHalf = 128;         // frequencies of a row
constexpr int kTableThreads = 256;
constexpr int kTableRows = 16;        // rows of a thread at most

// Angular steps per position in turns, as 64-bit fixed-point fractions: position p
// sits at p * turn mod 2^64, an exact integer product, so a far position loses
// nothing to the size of its angle (an fp32 angle would, and fp64 arithmetic is slow here).
struct TurnArgs {
  uint64_t turn[kMaxHalf];
  int half;
  int64_t pos0, n_pos;
  int rows;                           // rows of a thread
  float* cos_out;
  float* sin_out;
};

// cos and sin of phase / 2^64 turns.  The nearest quarter turn is taken off in integers,
// so what is left is at most an eighth of a turn and its fp32 rounding is relative to
// it: values next to a zero of either function keep their digits.
__device__ __forceinline__ void cos_sin_turns(uint64_t phase, float& c, float& s) {
  const uint64_t shifted = phase + (1ull << 61);
  const uint32_t quarter = static_cast<uint32_t>(shifted >> 62);
  const int64_t rest = static_cast<int64_t>(phase - (static_cast<uint64_t>(quarter) << 62));
  float sr, cr;
  sincospif(__ll2float_rn(rest) * 1.0842021724855044e-19f, &sr, &cr);   // rest / 2^63: half turns
  c = quarter == 0 ? cr : quarter == 1 ? -sr : quarter == 2 ? -cr : sr;
  s = quarter == 0 ? sr : quarter == 1 ? cr : quarter == 2 ? -sr : -cr;
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

constexpr int kApplyThreads = 256;

struct ApplyArgs {
  const void* x;
  void* out;
  int64_t x_tok, x_head, out_tok, out_head;   // strides in elements
  int offset, half;
  int rot_items;                              // per token-head: rotated items, then copied ones
  FastDiv items, per_head;                    // items of a token-head; heads
  int64_t tok0;                               // first token of this launch
  uint32_t n_items;                           // items of this launch
  const int32_t* pos;
  const float* rope_cos;                      // [rope_len][half]
  const float* rope_sin;
  int64_t rope_len;
  float scale, sign;                          // sign -1: the inverse rotation
  uint32_t* status;
};

template <typename T, int N>
struct alignas(N * sizeof(T)) Vec {
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
// is not in place.  HBM-bound: each element is read and written once, and a token's
// cos / sin row comes from L1 or L2 for all of its heads but the first.  fp32
// arithmetic, one rounding to the storage type.
template <typename T, int VEC, int kStyle>
__global__ void __launch_bounds__(kApplyThreads) rope_apply_kernel(const __grid_constant__ ApplyArgs a) {
  const uint32_t i = blockIdx.x * kApplyThreads + threadIdx.x;
  if (i >= a.n_items) return;
  const uint32_t row = a.items.div(i), item = i - row * a.items.d;
  const uint32_t t = a.per_head.div(row), h = row - t * a.per_head.d;
  const int64_t n = a.tok0 + t;
  const T* x = static_cast<const T*>(a.x) + n * a.x_tok + h * a.x_head;
  T* out = static_cast<T*>(a.out) + n * a.out_tok + h * a.out_head;
  using V = Vec<T, VEC>;
  if (static_cast<int>(item) >= a.rot_items) {
    int c = (static_cast<int>(item) - a.rot_items) * VEC;
    if (c >= a.offset) c += 2 * a.half;
    *reinterpret_cast<V*>(out + c) = *reinterpret_cast<const V*>(x + c);
    return;
  }
  int p = __ldg(a.pos + n);
  if (p < 0 || p >= a.rope_len) {
    record_status(a.status, LLA_ERR_DEVICE_ARG);
    p = p < 0 ? 0 : static_cast<int>(a.rope_len - 1);
  }
  const int f = static_cast<int>(item) * VEC;
  const float* cr = a.rope_cos + static_cast<int64_t>(p) * a.half + f;
  const float* sr = a.rope_sin + static_cast<int64_t>(p) * a.half + f;
  float c[VEC], s[VEC];
  if constexpr (VEC % 4 == 0) {
#pragma unroll
    for (int e = 0; e < VEC; e += 4) {
      const float4 c4 = __ldg(reinterpret_cast<const float4*>(cr + e));
      const float4 s4 = __ldg(reinterpret_cast<const float4*>(sr + e));
      c[e] = c4.x; c[e + 1] = c4.y; c[e + 2] = c4.z; c[e + 3] = c4.w;
      s[e] = s4.x; s[e + 1] = s4.y; s[e + 2] = s4.z; s[e + 3] = s4.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) { c[e] = __ldg(cr + e); s[e] = __ldg(sr + e); }
  }
  // the pair (i0, i1) of frequency f: (f, f + half) or (2f, 2f + 1)
  const int i0 = a.offset + (kStyle == 0 ? f : 2 * f), i1 = kStyle == 0 ? i0 + a.half : i0 + VEC;
  const V u = *reinterpret_cast<const V*>(x + i0), w = *reinterpret_cast<const V*>(x + i1);
  V yu, yw;
  T* yp[2] = {yu.v, yw.v};
  const T* xp[2] = {u.v, w.v};
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    // members of pair e: half layout u[e], w[e]; interleaved layout elements 2e, 2e + 1 of (u, w)
    const int k0 = kStyle == 0 ? e : 2 * e, k1 = kStyle == 0 ? e + VEC : 2 * e + 1;
    const float x0 = to_f32<T>(xp[k0 / VEC][k0 % VEC]), x1 = to_f32<T>(xp[k1 / VEC][k1 % VEC]);
    const float sn = s[e] * a.sign;
    yp[k0 / VEC][k0 % VEC] = from_f32<T>((x0 * c[e] - x1 * sn) * a.scale);
    yp[k1 / VEC][k1 % VEC] = from_f32<T>((x0 * sn + x1 * c[e]) * a.scale);
  }
  *reinterpret_cast<V*>(out + i0) = yu;
  *reinterpret_cast<V*>(out + i1) = yw;
}

template <typename T, int VEC>
cudaError_t launch_apply(const ApplyArgs& a, int style, cudaStream_t s) {
  const unsigned blocks = (a.n_items + kApplyThreads - 1) / kApplyThreads;
  if (style == LLA_ROPE_HALF) rope_apply_kernel<T, VEC, 0><<<blocks, kApplyThreads, 0, s>>>(a);
  else rope_apply_kernel<T, VEC, 1><<<blocks, kApplyThreads, 0, s>>>(a);
  return cudaGetLastError();
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
    // not as rows: allowed when both have the same strides and the rows lie apart
    const bool same = x_tok_stride == out_tok_stride && x_head_stride == out_head_stride;
    const uintptr_t gap = (xa > oa ? xa - oa : oa - xa) / es;
    if (xa < oe && oa < xe && !(same && gap >= static_cast<uintptr_t>((heads - 1) * x_head_stride + d_x) &&
                                gap + (heads - 1) * x_head_stride + d_x <= static_cast<uintptr_t>(x_tok_stride)))
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
  a.items = FastDiv(a.rot_items + (in_place ? 0 : (d_x - d_rope) / V));
  a.per_head = FastDiv(heads);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // launches of at most 2^30 items keep the item arithmetic in 32 bits
  const int64_t per_tok = static_cast<int64_t>(heads) * a.items.d;
  if (per_tok > (int64_t(1) << 30)) return LLA_ERR_UNSUPPORTED;
  const int64_t chunk = (int64_t(1) << 30) / per_tok;
  for (int64_t t = 0; t < N; t += chunk) {
    const int64_t n = N - t < chunk ? N - t : chunk;
    a.tok0 = t;
    a.n_items = static_cast<uint32_t>(n * per_tok);
    cudaError_t e;
    if (dims->dtype == LLA_BF16)
      e = vec ? launch_apply<__nv_bfloat16, 8>(a, dims->rope_style, s) : launch_apply<__nv_bfloat16, 1>(a, dims->rope_style, s);
    else
      e = vec ? launch_apply<float, 4>(a, dims->rope_style, s) : launch_apply<float, 1>(a, dims->rope_style, s);
    if (e != cudaSuccess) return LLA_ERR_CUDA;
  }
  return LLA_OK;
}

}  // extern "C"
