// lla_q4.cu — the 4-bit paged latent cache: latents rounded into rows (lla_q4_store), rows
// read back (lla_q4_load), and the plain decode attention over them (fp32 storage).
//
// Latents are centred by construction (Eq. (2) subtracts mu), so codes are symmetric: per
// 32 columns s = bf16(max|c| / 7) and code = round(c / s), half to even, which both
// divide in fp32.  bf16 scales keep the whole exponent range of a bf16 latent; their
// 8-bit mantissa only moves the grid (a scale rounded down puts max|c| / s at no more
// than 7.03, which still rounds to 7).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "lla_q4.h"

namespace lla {

namespace {

constexpr int kQ4Threads = 32;       // copies: small blocks, a token's heads in few steps of one warp
constexpr float kQ4Normal = 1.17549435e-38f;   // 2^-126: scales below it have no finite reciprocal, or few bits

struct Q4CopyArgs {
  int H, r_k, r_v, row_bytes;
  FastDiv items, strips, page;       // halves of a row's scale groups, threads that share a token's heads, rows of a page
  int toks;                          // tokens of a block
  int64_t N, num_slots;              // num_pages * page_size
  const int64_t* slots;
  void* k;                           // [N][H][r_k] storage dtype
  void* v;
  uint8_t* rows;
  uint32_t* status;
};

// Two neighbouring threads hold one group of 32 columns, sixteen each (the last group of a
// rank may have 16: the second is idle), of one token and up to kQ4Heads of its heads at a
// time, whose loads go out together.  Both directions move 2 (r_k + r_v) bytes (bf16) and a
// row per token-head and should be bound by HBM, so the work per column is kept to a few
// instructions, and divisions and addresses to once per thread.  65536 tokens of 16 heads at
// (96, 160), store and load: 299 + 210 us with eight columns a thread, conversions by int
// and true divisions, 188 + 143 with sixteen columns of one head, 267 together as here (310 with
// four heads and 128 threads).
constexpr int kQ4Heads = 2;
struct Q4Item {
  int sub, col, r, code_at, scale_at;
  bool k_axis, active, last;
  int64_t n, row;                    // token; its row of head 0, -1: the thread has nothing to do
  int h;                             // first head
};
__device__ __forceinline__ Q4Item q4_item(const Q4CopyArgs& a) {
  Q4Item it;
  const uint32_t team = a.items.div(threadIdx.x), ts = a.strips.div(team);
  const int item = static_cast<int>(threadIdx.x - team * a.items.d), g = item >> 1, gk = q4_groups(a.r_k);
  it.sub = item & 1;
  it.n = static_cast<int64_t>(blockIdx.x) * a.toks + ts;
  it.h = static_cast<int>(team - ts * a.strips.d);
  it.k_axis = g < gk;
  it.r = it.k_axis ? a.r_k : a.r_v;
  it.col = (it.k_axis ? g : g - gk) * kQ4Group + 16 * it.sub;
  it.active = it.col < it.r;
  it.last = (item | 1) == static_cast<int>(a.items.d) - 1;
  it.code_at = (it.k_axis ? 0 : a.r_k / 2) + it.col / 2;
  it.scale_at = q4_scale_offset(a.r_k, a.r_v) + 2 * g;
  it.row = -1;
  if (static_cast<int>(ts) >= a.toks || it.n >= a.N) return it;
  const int64_t slot = __ldg(a.slots + it.n);
  if (slot < 0) return it;           // holds no token
  if (slot >= a.num_slots) {
    record_status(a.status, LLA_ERR_DEVICE_ARG);
    return it;
  }
  const int64_t P = a.page.d, page = slot < (int64_t(1) << 31) ? a.page.div(static_cast<uint32_t>(slot)) : slot / P;
  it.row = page * a.H * P + (slot - page * P);
  return it;
}

// Sixteen latents as they are stored, and the bits of the largest |c| among them
// (NaN sorts above infinity).
struct Half16 {
  uint4 x[2];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    x[0] = __ldg(reinterpret_cast<const uint4*>(p));
    x[1] = __ldg(reinterpret_cast<const uint4*>(p) + 1);
  }
  __device__ __forceinline__ uint32_t get(float (&v)[16]) const {
    const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      top = __vmaxu2(top, w[i] & 0x7FFF7FFFu);
    }
    return max(top << 16, top & 0xFFFF0000u);
  }
};
struct Full16 {
  float4 x[4];
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __ldg(reinterpret_cast<const float4*>(p) + i);
  }
  __device__ __forceinline__ uint32_t get(float (&v)[16]) const {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[4 * i] = x[i].x; v[4 * i + 1] = x[i].y; v[4 * i + 2] = x[i].z; v[4 * i + 3] = x[i].w;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
    return top;
  }
};

// Bit of column e of a code word.
__host__ __device__ constexpr int q4_bit(int e) { return 4 * (e >> 1) + 16 * (e & 1); }

// The sixteen columns' codes and scale, at their place in the row `dst`.
template <typename T>
__device__ __forceinline__ void q4_put(const Q4CopyArgs& a, const Q4Item& it, uint8_t* dst, uint32_t top, const float (&v)[16]) {
  const bool finite = top < 0x7f800000u;
  // a group with a value that is not finite stores a NaN scale: all of it reads as NaN
  const __nv_bfloat16 s16 =
      finite ? __float2bfloat16_rn(__fdiv_rn(__uint_as_float(top), 7.f)) : __ushort_as_bfloat16(0x7fc0);
  const float s = __bfloat162float(s16);
  uint32_t w[2];
  bool done = false;
  if (sizeof(T) == 2 && finite && s >= kQ4Normal) {
    // bf16 values: c / s has 8-bit numerator and denominator, so it is half an integer exactly or off
    // by 2^-10 at least (for |c / s| >= 1/4).  c * (1 / s), 2^-22 off at most, rounded to multiples of
    // 2^-11 is therefore on the same side or on the same tie, and rounds to the same code as
    // the quotient.  |c / s| <= 7.03: no clamp.  1.5 * 2^23 + 8 leaves code + 8 in the low bits;
    // a multiply-add per code packs the words, and the constant parts are taken off once.
    const float inv = __frcp_rn(s);
    constexpr uint32_t kBase = 0x4B400000u;   // bits of 1.5 * 2^23
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t sum = 0, base = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float t = __fadd_rn(__fmaf_rn(v[8 * j + e], inv, 6144.f), -6144.f);
        sum += __float_as_uint(__fadd_rn(t, 12582920.f)) * (1u << q4_bit(e));
        base += kBase * (1u << q4_bit(e));
      }
      w[j] = sum - base;
    }
    done = true;
  }
  if (sizeof(T) == 4 && finite && s >= kQ4Normal) {
    // fp32 values: c * (1 / s) is within 2^-23 of the quotient (8.4e-7 of up to 7.03), which fp32 division
    // moves by 2.4e-7 more: only next to a tie could either matter, and that group is divided.  (A
    // division for every value took four times as long as the bytes.)
    const float inv = __frcp_rn(s);
    constexpr uint32_t kBase = 0x4B400000u;
    float off = 0.f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t sum = 0, base = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float q = __fmul_rn(v[8 * j + e], inv), t = __fadd_rn(q, 12582920.f);
        off = fmaxf(off, fabsf(__fsub_rn(q, __fadd_rn(t, -12582920.f))));
        sum += __float_as_uint(t) * (1u << q4_bit(e));
        base += kBase * (1u << q4_bit(e));
      }
      w[j] = sum - base;
    }
    done = off < 0.5f - 2e-6f;
  }
  if (!done) {
    const bool some = finite && s > 0.f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      w[j] = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int code = some ? min(max(__float2int_rn(__fdiv_rn(v[8 * j + e], s)), -7), 7) : 0;
        w[j] |= static_cast<uint32_t>(code + 8) << q4_bit(e);
      }
    }
  }
  if (it.active) *reinterpret_cast<uint2*>(dst + it.code_at) = make_uint2(w[0], w[1]);
  if (it.sub == 0) *reinterpret_cast<__nv_bfloat16*>(dst + it.scale_at) = s16;
  // the row's padding, by the last group's threads: rows are fully defined
  if (it.last)
    for (int p = it.scale_at + 2 + 2 * it.sub; p < a.row_bytes; p += 4) *reinterpret_cast<uint16_t*>(dst + p) = 0;
}

template <typename T>
__global__ void __launch_bounds__(kQ4Threads) q4_store_kernel(const __grid_constant__ Q4CopyArgs a) {
  const Q4Item it = q4_item(a);
  if (it.row < 0) return;            // (both threads of a group, or neither)
  const uint32_t pair = 3u << (threadIdx.x & 30);
  const int strips = static_cast<int>(a.strips.d);
  const T* src = static_cast<const T*>(it.k_axis ? a.k : a.v) + (it.n * a.H + it.h) * it.r + it.col;
  const int64_t head = static_cast<int64_t>(a.page.d) * a.row_bytes;   // bytes between a token's heads
  uint8_t* dst = a.rows + it.row * a.row_bytes + it.h * head;
  for (int h = it.h; h < a.H; h += kQ4Heads * strips) {
    std::conditional_t<sizeof(T) == 2, Half16, Full16> c[kQ4Heads] = {};
#pragma unroll
    for (int i = 0; i < kQ4Heads; ++i)
      if (h + i * strips < a.H && it.active) c[i].load(src + i * strips * it.r);
#pragma unroll
    for (int i = 0; i < kQ4Heads; ++i) {
      if (h + i * strips >= a.H) break;
      float v[16];
      uint32_t top = c[i].get(v);
      top = max(top, __shfl_xor_sync(pair, top, 1));
      q4_put<T>(a, it, dst + i * strips * head, top, v);
    }
    src += kQ4Heads * strips * it.r;
    dst += kQ4Heads * strips * head;
  }
}

// Eight values of a code word: code * scale, rounded once to the storage type.
__device__ __forceinline__ void put8(__nv_bfloat16* p, uint32_t w, __nv_bfloat16 s) {
  // 128 + code + 8 has unit 1 in bf16; the difference is exact, the product rounds once
  const __nv_bfloat162 off = __bfloat162bfloat162(__ushort_as_bfloat16(0x4308)), s2 = __bfloat162bfloat162(s);   // 136
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t x = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
    const __nv_bfloat162 y = __hmul2(__hsub2(*reinterpret_cast<__nv_bfloat162*>(&x), off), s2);
    o[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(o[0], o[1], o[2], o[3]);
}
// Code of column e of a word: 2^23 + code + 8 has unit 1 in fp32.
__device__ __forceinline__ float q4_code(uint32_t w, int e) {
  return __uint_as_float(((w >> q4_bit(e)) & 15u) | 0x4B000000u) - 8388616.f;
}
__device__ __forceinline__ void put8(float* p, uint32_t w, __nv_bfloat16 s) {
  const float f = __bfloat162float(s);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    reinterpret_cast<float4*>(p)[i] = make_float4(q4_code(w, 4 * i) * f, q4_code(w, 4 * i + 1) * f, q4_code(w, 4 * i + 2) * f,
                                                  q4_code(w, 4 * i + 3) * f);
}

template <typename T>
__global__ void __launch_bounds__(kQ4Threads) q4_load_kernel(const __grid_constant__ Q4CopyArgs a) {
  const Q4Item it = q4_item(a);
  if (it.row < 0 || !it.active) return;
  const int strips = static_cast<int>(a.strips.d);
  const int64_t head = static_cast<int64_t>(a.page.d) * a.row_bytes;
  const uint8_t* src = a.rows + it.row * a.row_bytes + it.h * head;
  T* dst = static_cast<T*>(it.k_axis ? a.k : a.v) + (it.n * a.H + it.h) * it.r + it.col;
  for (int h = it.h; h < a.H; h += kQ4Heads * strips) {
    __nv_bfloat16 sc[kQ4Heads];
    uint2 w[kQ4Heads];
#pragma unroll
    for (int i = 0; i < kQ4Heads; ++i) {
      if (h + i * strips >= a.H) break;
      sc[i] = *reinterpret_cast<const __nv_bfloat16*>(src + i * strips * head + it.scale_at);
      w[i] = *reinterpret_cast<const uint2*>(src + i * strips * head + it.code_at);
    }
#pragma unroll
    for (int i = 0; i < kQ4Heads; ++i) {
      if (h + i * strips >= a.H) break;
      put8(dst + i * strips * it.r, w[i].x, sc[i]);
      put8(dst + i * strips * it.r + 8, w[i].y, sc[i]);
    }
    src += kQ4Heads * strips * head;
    dst += kQ4Heads * strips * it.r;
  }
}

// ----------------------------------------------------------------- fp32 decode

// Decode attention over 4-bit rows for fp32 storage, in fp32 arithmetic: one block
// per (sequence, head, split of whole 128-token tiles).  The score is Eq. (3) with RoPE
// after reconstruction, regrouped per frequency pair as in lla_paged_generic.cu, with the
// folded query in fp32.  A warp has eight of a tile's tokens, a thread four of them and eight of
// the 128 rotary coordinates (cosine and sine of four frequencies): two 16-byte reads of the
// folded query serve 32 multiply-adds.  (With 32 coordinates of one token a thread needed
// eight, and those reads bound the kernel: 34 us for 3 x 333 tokens of 2 heads, 24.5 as here.)  One online softmax over
// the split's tiles, the value path absorbed; a record per split, merged by the combine.
constexpr int kF32Threads = 512;
constexpr int kParts = 4;             // threads that fetch a token's row
constexpr float kQ4ScoreScale = 0.08838834764831845f * 1.4426950408889634f;   // log2(e) / sqrt(128)

// d += (a, a) * b: two fp32 multiply-adds in one instruction
__device__ __forceinline__ void fma2(float2& d, float a, float2 b) {
  uint64_t x, y, z;
  asm("mov.b64 %0, {%1, %1};" : "=l"(x) : "f"(a));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(z) : "f"(d.x), "f"(d.y));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(z) : "l"(x), "l"(y));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(z));
}

__device__ __forceinline__ int q4_len(const Q4DecodeArgs& a, int b) {
  const int L = __ldg(a.seq_lens + b);
  return L < 0 ? 0 : (L > a.L_max ? static_cast<int>(a.L_max) : L);
}

__global__ void __launch_bounds__(kF32Threads, 2) q4_f32_kernel(const __grid_constant__ Q4DecodeArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the combine waits for this grid
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(8) float bias[128];
  __shared__ float qr[kHeadDim], pw[kTile], red[kF32Threads / 32], sums[kF32Threads];
  const int rk = a.r_k, rv = a.r_v, rb = a.row_bytes;
  float* z = reinterpret_cast<float*>(smem);                         // [rk][128]: cosine, then sine coordinates
  uint8_t* tile = smem + static_cast<size_t>(rk) * 512;              // [128][rb + 16]
  const int ts = rb + 16;
  const int64_t id = blockIdx.x;
  const int64_t u = id / a.splits;
  const int sp = static_cast<int>(id - u * a.splits);
  const int b = static_cast<int>(u / a.H), h = static_cast<int>(u - static_cast<int64_t>(b) * a.H);
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int L0 = __ldg(a.seq_lens + b);
  if (sp == 0 && (L0 < 0 || L0 > a.L_max) && tid == 0) record_status(a.status, LLA_ERR_DEVICE_ARG);
  const int L = q4_len(a, b);
  int qp = __ldg(a.q_pos + b);
  if (qp < 0 || qp >= a.rope_len) {
    if (tid == 0) record_status(a.status, LLA_ERR_DEVICE_ARG);
    qp = qp < 0 ? 0 : static_cast<int>(a.rope_len - 1);
  }
  const int64_t j_lo = sp * a.chunk, j_hi = min(static_cast<int64_t>(L), j_lo + a.chunk);
  if (j_lo >= j_hi) return;
  auto pair_of = [&](int f, int& i0, int& i1) {
    i0 = a.rope_style == 0 ? f : 2 * f;
    i1 = a.rope_style == 0 ? f + 64 : 2 * f + 1;
  };
  // the split's first rows are requested before the folded query is formed
  auto fetch = [&](int64_t j0) {
    const int64_t j = j0 + tid / kParts;
    if (j >= j_hi) return;
    const int64_t row = latent_row(a.block_table, a.page_size, a.max_pages, a.num_pages, a.L_max, a.H, b, h, j, a.status);
    const uint4* src = reinterpret_cast<const uint4*>(a.rows + row * rb);
    uint4* dst = reinterpret_cast<uint4*>(tile + static_cast<size_t>(tid / kParts) * ts);
    for (int i = tid % kParts; i < rb / 16; i += kParts) dst[i] = __ldg(src + i);
  };
  fetch(j_lo);
  const float* q = static_cast<const float*>(a.q) + u * kHeadDim;
  const float* mk = a.mu_k + h * a.mu_hstride;
  if (tid < 64) {
    int i0, i1;
    pair_of(tid, i0, i1);
    const float c = __ldg(a.rope_cos + static_cast<int64_t>(qp) * 64 + tid);
    const float s = __ldg(a.rope_sin + static_cast<int64_t>(qp) * 64 + tid);
    const float x0 = __ldg(q + i0), x1 = __ldg(q + i1);
    const float q0 = (x0 * c - x1 * s) * kQ4ScoreScale, q1 = (x0 * s + x1 * c) * kQ4ScoreScale;
    qr[i0] = q0;
    qr[i1] = q1;
    bias[tid] = q0 * mk[i0] + q1 * mk[i1];
    bias[64 + tid] = q1 * mk[i0] - q0 * mk[i1];
  }
  __syncthreads();
  const float* W = static_cast<const float*>(a.w_up_k) + static_cast<int64_t>(h) * kHeadDim * rk;
  // four columns of one frequency per item: 16-byte loads, several in flight; 4 x 8 (columns,
  // frequencies) per warp
#pragma unroll 3
  for (int i = tid; i < 16 * rk; i += kF32Threads) {
    const int q4 = i & 3, f = (i >> 2) & 63, k = (i >> 8) * 16 + 4 * q4;   // rk is a multiple of 16
    int i0, i1;
    pair_of(f, i0, i1);
    const float4 w0 = __ldg(reinterpret_cast<const float4*>(W + static_cast<int64_t>(i0) * rk + k));
    const float4 w1 = __ldg(reinterpret_cast<const float4*>(W + static_cast<int64_t>(i1) * rk + k));
    const float q0 = qr[i0], q1 = qr[i1];
    const float u0[4] = {w0.x, w0.y, w0.z, w0.w}, u1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      z[(k + e) * 128 + f] = q0 * u0[e] + q1 * u1[e];
      z[(k + e) * 128 + 64 + f] = q1 * u0[e] - q0 * u1[e];
    }
  }
  // V: a thread's column, and which share of a tile's tokens it adds up
  const int shares = rv <= 128 ? 4 : 2, width = kF32Threads / shares, col = tid % width, share = tid / width;
  const int v_at = rk / 2 + 4 * (col / 8), v_bit = 4 * ((col & 7) >> 1) + 16 * (col & 1);
  const int v_scale = q4_scale_offset(rk, rv) + 2 * (q4_groups(rk) + col / kQ4Group);
  float acc = 0.f, m_run = -INFINITY, l_run = 0.f;
  __syncthreads();
  const int t0 = 8 * wid + 4 * (lane >> 4), f4 = 4 * (lane & 15);   // the thread's tokens and frequencies
  const bool owner = (lane & 12) == 0;                                // of one token's weight
  const int token = t0 + (lane & 3);
  for (int64_t j0 = j_lo; j0 < j_hi; j0 += kTile) {
    const bool valid = owner && j0 + token < j_hi;
    const int nt = static_cast<int>(min(static_cast<int64_t>(kTile), j_hi - j0));
    const uint8_t* mine = tile + static_cast<size_t>(t0) * ts;
    float s4[4];
    {
      float2 A[4][4];   // cosines, then sines of the four frequencies
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) A[i][e] = *reinterpret_cast<const float2*>(bias + 64 * (e >> 1) + f4 + 2 * (e & 1));
      const float* zp = z + f4;
#pragma unroll 1
      for (int k0 = 0; k0 < rk; k0 += 8) {
        float sc[4];
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // (a token behind the split's last may hold anything: its score is not used)
          sc[i] = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(
              mine + i * ts + q4_scale_offset(rk, rv) + 2 * (k0 / kQ4Group)));
          w[i] = *reinterpret_cast<const uint32_t*>(mine + i * ts + k0 / 2);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float4 zc = *reinterpret_cast<const float4*>(zp + (k0 + e) * 128);
          const float4 zs = *reinterpret_cast<const float4*>(zp + (k0 + e) * 128 + 64);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float c = q4_code(w[i], e) * sc[i];
            fma2(A[i][0], c, make_float2(zc.x, zc.y));
            fma2(A[i][1], c, make_float2(zc.z, zc.w));
            fma2(A[i][2], c, make_float2(zs.x, zs.y));
            fma2(A[i][3], c, make_float2(zs.z, zs.w));
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t j = min(j0 + t0 + i, j_hi - 1);
        const float4 c = __ldg(reinterpret_cast<const float4*>(a.rope_cos + j * 64 + f4));
        const float4 n = __ldg(reinterpret_cast<const float4*>(a.rope_sin + j * 64 + f4));
        float s = c.x * A[i][0].x;
        s = fmaf(c.y, A[i][0].y, fmaf(c.z, A[i][1].x, fmaf(c.w, A[i][1].y, s)));
        s4[i] = fmaf(n.x, A[i][2].x, fmaf(n.y, A[i][2].y, fmaf(n.z, A[i][3].x, fmaf(n.w, A[i][3].y, s))));
      }
    }
#pragma unroll
    for (int o = 1; o < 16; o <<= 1)
#pragma unroll
      for (int i = 0; i < 4; ++i) s4[i] += __shfl_xor_sync(0xffffffffu, s4[i], o);
    float s = -INFINITY;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (valid && (lane & 3) == i) s = s4[i];
    // ---- online softmax over the tile (log2 units)
    const float mw = warp_max(s);
    if (lane == 0) red[wid] = mw;
    __syncthreads();
    float m_new = m_run;
#pragma unroll
    for (int i = 0; i < kF32Threads / 32; ++i) m_new = fmaxf(m_new, red[i]);
    const float scale = m_new == -INFINITY ? 1.f : exp2f(m_run - m_new);   // the first tile: 0
    const float p = valid ? (m_new == -INFINITY ? s - s : exp2f(s - m_new)) : 0.f;   // all NaN: stays NaN
    if (owner) pw[token] = p;
    const float ps = warp_sum(p);
    __syncthreads();   // pw complete; red is read
    if (lane == 0) red[wid] = ps;
    if (col < rv) {
      float v = 0.f;
#pragma unroll 4
      for (int i = share; i < nt; i += shares) {
        const uint8_t* r = tile + static_cast<size_t>(i) * ts;
        const float c = static_cast<float>(static_cast<int>((*reinterpret_cast<const uint32_t*>(r + v_at) >> v_bit) & 15u) - 8);
        v = fmaf(pw[i], c * __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(r + v_scale)), v);
      }
      acc = fmaf(acc, scale, v);
    }
    __syncthreads();   // red holds the sums; the rows are free for the next tile
    if (j0 + kTile < j_hi) fetch(j0 + kTile);
    float ls = 0.f;
#pragma unroll
    for (int i = 0; i < kF32Threads / 32; ++i) ls += red[i];
    l_run = l_run * scale + ls;
    m_run = m_new;
    __syncthreads();   // the next rows are in place; everyone has read red
  }
  sums[tid] = acc;
  __syncthreads();
  float* rec = a.records + id * (rv + kRecordHead);
  if (tid == 0) {
    rec[0] = m_run;
    rec[1] = l_run;
  }
  if (tid < rv) {   // rv <= width
    float v = sums[tid];
    for (int i = 1; i < shares; ++i) v += sums[i * width + tid];
    rec[kRecordHead + tid] = v;
  }
}

// Merge a (sequence, head)'s split records by log-sum-exp, apply W_up,v once (Appendix J
// "Absorbed attention") and normalise.  Block = (head, sequence), two threads per output, their halves of
// its row requested before the wait for the decode grid.
constexpr int kF32CombineThreads = 256;
__global__ void __launch_bounds__(kF32CombineThreads) q4_f32_combine_kernel(const __grid_constant__ Q4DecodeArgs a) {
  constexpr int kRegs = kMaxRankPerHead / 8;   // 16-byte loads of half a row
  __shared__ float acc[kMaxRankPerHead];
  const int64_t u = blockIdx.x;
  const int b = static_cast<int>(u / a.H), h = static_cast<int>(u - static_cast<int64_t>(b) * a.H), tid = threadIdx.x;
  const int L = q4_len(a, b), rv = a.r_v, e = tid >> 1, half = tid & 1;
  const float4* W = reinterpret_cast<const float4*>(static_cast<const float*>(a.w_up_v) + (static_cast<int64_t>(h) * kHeadDim + e) * rv);
  float4 w[kRegs];
#pragma unroll
  for (int i = 0; i < kRegs; ++i) w[i] = 4 * (2 * i + half) < rv ? __ldg(W + 2 * i + half) : make_float4(0.f, 0.f, 0.f, 0.f);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float* out = static_cast<float*>(a.out) + u * kHeadDim;
  if (L == 0) {
    if (half == 0) out[e] = 0.f;
    if (tid == 0 && a.lse) a.lse[u] = -INFINITY;
    return;
  }
  const int n = static_cast<int>((L + a.chunk - 1) / a.chunk);
  const float* rec = a.records + u * a.splits * (rv + kRecordHead);
  float m = -INFINITY;
  for (int i = 0; i < n; ++i) m = fmaxf(m, rec[static_cast<int64_t>(i) * (rv + kRecordHead)]);
  float l = 0.f, v = 0.f;
  for (int i = 0; i < n; ++i) {
    const float* r = rec + static_cast<int64_t>(i) * (rv + kRecordHead);
    const float f = m == -INFINITY ? 1.f : exp2f(r[0] - m);   // no maximum: every score was NaN, and so is l
    l = fmaf(r[1], f, l);
    if (tid < rv) v = fmaf(r[kRecordHead + tid], f, v);
  }
  if (tid < rv) acc[tid] = v;
  __syncthreads();
  float o = 0.f;
#pragma unroll
  for (int i = 0; i < kRegs; ++i) {
    const int k = 4 * (2 * i + half);
    if (k < rv) o = fmaf(acc[k], w[i].x, fmaf(acc[k + 1], w[i].y, fmaf(acc[k + 2], w[i].z, fmaf(acc[k + 3], w[i].w, o))));
  }
  o += __shfl_xor_sync(0xffffffffu, o, 1);
  if (half == 0) out[e] = o / l + a.mu_v[h * a.mu_hstride + e];
  if (tid == 0 && a.lse) a.lse[u] = (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace

cudaError_t launch_q4_f32(const Q4DecodeArgs& a, cudaStream_t s) {
  auto bytes = [](int r_k, int row_bytes) { return static_cast<size_t>(r_k) * 512 + static_cast<size_t>(kTile) * (row_bytes + 16); };
  const size_t smem = bytes(a.r_k, a.row_bytes);
  cudaError_t e = allow_smem(q4_f32_kernel, bytes(kMaxRankPerHead, q4_row_bytes(kMaxRankPerHead, kMaxRankPerHead)));
  if (e != cudaSuccess) return e;
  const int64_t units = static_cast<int64_t>(a.B) * a.H;
  q4_f32_kernel<<<static_cast<unsigned>(units * a.splits), kF32Threads, smem, s>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_pdl(q4_f32_combine_kernel, dim3(static_cast<unsigned>(units)), dim3(kF32CombineThreads), 0, s, a);
}

int64_t q4_plain_chunk(int B, int H, int64_t L_max, int sms) {
  const int64_t tiles = (L_max + kTile - 1) / kTile, units = static_cast<int64_t>(B) * H;
  const int64_t want = std::max<int64_t>(1, (2 * static_cast<int64_t>(sms) + units - 1) / units);
  return (tiles + std::min(want, tiles) - 1) / std::min(want, tiles) * kTile;
}


}  // namespace lla

using namespace lla;

namespace {

// Host checks of a 4-bit pool description; LLA_OK also for B == 0.
lla_status q4_pool_checks(const lla_dims* dims, const lla_q4_cache* c) {
  if (!c || c->B < 0 || c->page_size < 1 || c->num_pages < 1) return LLA_ERR_INVALID_ARG;
  if (dims->variant != LLA_PER_HEAD) return LLA_ERR_UNSUPPORTED;
  if (c->num_pages >= (int64_t(1) << 31) || c->num_pages * static_cast<int64_t>(dims->H) >= (int64_t(1) << 31) ||
      c->num_pages * static_cast<int64_t>(c->page_size) >= (int64_t(1) << 40))
    return LLA_ERR_UNSUPPORTED;
  return LLA_OK;
}

bool at16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

lla_status q4_copy(const lla_dims* dims, void* k, void* v, int N, const int64_t* slots, const lla_q4_cache* cache,
                   void* workspace, size_t ws_bytes, void* stream, bool store) {
  lla_status st = checked_dims(dims);
  if (st != LLA_OK) return st;
  if ((st = q4_pool_checks(dims, cache)) != LLA_OK) return st;
  if (N < 0) return LLA_ERR_INVALID_ARG;
  if (N == 0) return LLA_OK;
  if (!at16(k) || !at16(v) || !at16(cache->rows) || !at16(workspace) || !slots ||
      (reinterpret_cast<uintptr_t>(slots) & 7u) || ws_bytes < 256)
    return LLA_ERR_INVALID_ARG;
  Q4CopyArgs a{};
  a.H = dims->H;
  a.r_k = dims->r_k;
  a.r_v = dims->r_v;
  a.row_bytes = q4_row_bytes(dims->r_k, dims->r_v);
  // a block: the halves of a row's groups x threads for kQ4Heads heads each x tokens
  const int items = 2 * (q4_groups(dims->r_k) + q4_groups(dims->r_v)), at_once = kQ4Threads / items;
  const int strips = std::min((dims->H + kQ4Heads - 1) / kQ4Heads, at_once);
  a.items = FastDiv(items);
  a.strips = FastDiv(strips);
  a.toks = at_once / strips;
  a.N = N;
  a.page = FastDiv(cache->page_size);
  a.num_slots = cache->num_pages * cache->page_size;
  a.slots = slots;
  a.k = k;
  a.v = v;
  a.rows = static_cast<uint8_t*>(cache->rows);
  a.status = static_cast<uint32_t*>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned blocks = static_cast<unsigned>((a.N + a.toks - 1) / a.toks);
  if (store) {
    if (dims->dtype == LLA_BF16) q4_store_kernel<__nv_bfloat16><<<blocks, kQ4Threads, 0, s>>>(a);
    else q4_store_kernel<float><<<blocks, kQ4Threads, 0, s>>>(a);
  } else {
    if (dims->dtype == LLA_BF16) q4_load_kernel<__nv_bfloat16><<<blocks, kQ4Threads, 0, s>>>(a);
    else q4_load_kernel<float><<<blocks, kQ4Threads, 0, s>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? LLA_OK : LLA_ERR_CUDA;
}

// Workspace of a decode call: status word; tensor-core kernel: the CTA range of every
// (sequence, head group), the units of every folded query, a record per head of every (unit, CTA) of a run (at most
// units + grid of them), the query operands of every (sequence, head group), the f16 rotary tiles of
// L_max positions; fp32 kernel: a record per split.
struct Q4Ws {
  size_t ranges, z_unit, records, zimg, row_tiles, total;
  int grid;
};
Q4Ws q4_ws(const lla_dims* d, int B, int64_t L_max, int sms) {
  Q4Ws w{};
  const int64_t tiles = std::max<int64_t>(1, (L_max + kTile - 1) / kTile);
  const size_t rec = static_cast<size_t>(d->r_v + kRecordHead) * 4;
  w.ranges = 256;
  if (d->dtype == LLA_BF16) {
    Q4Plan p;
    make_q4_plan(d->H, d->r_k, d->r_v, &p);
    const int64_t units = static_cast<int64_t>(B) * p.ngroups;
    w.grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(std::min(sms, kMaxGrid), units * tiles)));
    w.z_unit = 256 + static_cast<size_t>(units) * 8;
    w.records = (w.z_unit + static_cast<size_t>(B) * d->H * 8 + 255) / 256 * 256;
    w.zimg = (w.records + (static_cast<size_t>(units) + w.grid) * p.nh * q4_record_floats(p.nh, d->r_v) * 4 + 255) / 256 * 256;
    w.row_tiles = w.zimg + static_cast<size_t>(units) * 2 * p.z_chunk;
    w.total = w.row_tiles + static_cast<size_t>(tiles) * kTile * 256;
    return w;
  }
  const int64_t chunk = q4_plain_chunk(std::max(B, 1), d->H, std::max<int64_t>(L_max, 1), sms) / kTile;
  w.records = 256;
  w.total = 256 + static_cast<size_t>(B) * d->H * ((tiles + chunk - 1) / chunk) * rec;
  return w;
}

}  // namespace

extern "C" {

size_t lla_q4_row_bytes(const lla_dims* dims) {
  if (checked_dims(dims) != LLA_OK || dims->variant != LLA_PER_HEAD) return 0;
  return static_cast<size_t>(q4_row_bytes(dims->r_k, dims->r_v));
}

size_t lla_q4_workspace_size(const lla_dims* dims, int B, int64_t L_max) {
  if (checked_dims(dims) != LLA_OK || dims->variant != LLA_PER_HEAD || B < 0 || L_max < 0) return 0;
  return q4_ws(dims, B, L_max, device_sm_count()).total;
}

lla_status lla_q4_store(const lla_dims* dims, const void* c_k, const void* c_v, int N, const int64_t* slots,
                        const lla_q4_cache* cache, void* workspace, size_t ws_bytes, void* stream) {
  return q4_copy(dims, const_cast<void*>(c_k), const_cast<void*>(c_v), N, slots, cache, workspace, ws_bytes, stream, true);
}

lla_status lla_q4_load(const lla_dims* dims, const int64_t* slots, int N, const lla_q4_cache* cache, void* c_k,
                       void* c_v, void* workspace, size_t ws_bytes, void* stream) {
  return q4_copy(dims, c_k, c_v, N, slots, cache, workspace, ws_bytes, stream, false);
}

lla_status lla_decode_attn_q4(const lla_dims* dims, int loop_t, const void* q, const lla_q4_cache* cache,
                              const int32_t* seq_lens, const int32_t* q_pos, const void* w_up_k, const void* w_up_v,
                              const float* mu_k, const float* mu_v, const float* rope_cos, const float* rope_sin,
                              int64_t rope_len, void* out, float* lse, void* workspace, size_t ws_bytes,
                              void* stream) {
  lla_status st = checked_dims(dims);
  if (st != LLA_OK) return st;
  if ((st = q4_pool_checks(dims, cache)) != LLA_OK) return st;
  if (loop_t < 0 || loop_t >= dims->T || cache->max_pages < 1) return LLA_ERR_INVALID_ARG;
  const int64_t L_max = static_cast<int64_t>(cache->max_pages) * cache->page_size;
  if (L_max > (int64_t(1) << 30) || static_cast<int64_t>(cache->B) * cache->max_pages >= (int64_t(1) << 31) ||
      static_cast<int64_t>(cache->B) * dims->H > (int64_t(1) << 24) ||
      static_cast<int64_t>(cache->B) * ((L_max + kTile - 1) / kTile) >= (int64_t(1) << 31))
    return LLA_ERR_UNSUPPORTED;
  if (cache->B == 0) return LLA_OK;
  if (rope_len < L_max || rope_len < kTile) return LLA_ERR_INVALID_ARG;
  const void* ptrs[] = {q, cache->rows, seq_lens, q_pos, w_up_k, w_up_v, mu_k, mu_v, rope_cos, rope_sin, out, workspace};
  for (const void* p : ptrs)
    if (!at16(p)) return LLA_ERR_INVALID_ARG;
  if (!cache->block_table || (reinterpret_cast<uintptr_t>(cache->block_table) & 3u) ||
      (reinterpret_cast<uintptr_t>(lse) & 3u))
    return LLA_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  if (sms <= 0) return LLA_ERR_CUDA;
  const Q4Ws w = q4_ws(dims, cache->B, L_max, sms);
  if (ws_bytes < w.total) return LLA_ERR_INVALID_ARG;
  const size_t es = dims->dtype == LLA_BF16 ? 2 : 4;
  const size_t wk = static_cast<size_t>(dims->H) * kHeadDim * dims->r_k * es;
  const size_t wv = static_cast<size_t>(dims->H) * kHeadDim * dims->r_v * es;
  Q4DecodeArgs a{};
  a.B = cache->B;
  a.H = dims->H;
  a.r_k = dims->r_k;
  a.r_v = dims->r_v;
  a.rope_style = dims->rope_style;
  a.row_bytes = q4_row_bytes(dims->r_k, dims->r_v);
  a.L_max = L_max;
  a.rope_len = rope_len;
  a.mu_hstride = static_cast<int64_t>(dims->T) * kHeadDim;
  a.q = q;
  a.rows = static_cast<const uint8_t*>(cache->rows);
  a.block_table = cache->block_table;
  a.page_size = cache->page_size;
  a.max_pages = cache->max_pages;
  a.num_pages = cache->num_pages;
  a.seq_lens = seq_lens;
  a.q_pos = q_pos;
  a.w_up_k = static_cast<const uint8_t*>(w_up_k) + loop_t * wk;
  a.w_up_v = static_cast<const uint8_t*>(w_up_v) + loop_t * wv;
  a.mu_k = mu_k + static_cast<size_t>(loop_t) * kHeadDim;
  a.mu_v = mu_v + static_cast<size_t>(loop_t) * kHeadDim;
  a.rope_cos = rope_cos;
  a.rope_sin = rope_sin;
  a.out = out;
  a.lse = lse;
  a.status = static_cast<uint32_t*>(workspace);
  a.records = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + w.records);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dims->dtype == LLA_BF16) {
    if (!make_q4_plan(a.H, a.r_k, a.r_v, &a.plan)) return LLA_ERR_UNSUPPORTED;
    a.ranges = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + w.ranges);
    a.z_unit = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + w.z_unit);
    a.grid = w.grid;
    a.row_tiles = static_cast<uint8_t*>(workspace) + w.row_tiles;
    a.zimg = static_cast<uint8_t*>(workspace) + w.zimg;
    a.rec_stride = q4_record_floats(a.plan.nh, a.r_v);
    a.z_blocks = a.H * ((a.B + kQ4PrepSeqs - 1) / kQ4PrepSeqs);
    a.rows_grid = static_cast<int>(std::min<int64_t>((L_max + 15) / 16, 8 * sms));
    // sequences per combine block: W_up,v is read once for them while there are two blocks per SM (up to
    // four: 128 x 4096 at (16, 32) takes 150 us, with one 152, with seven 153; 64 x 1000 at (96, 160)
    // 70, with one 81)
    a.combine_units = static_cast<int>(std::min<int64_t>(kQ4CombineUnits, (static_cast<int64_t>(a.B) * a.H + 2 * sms - 1) / (2 * sms)));
    return launch_q4_tile(a, s) == cudaSuccess ? LLA_OK : LLA_ERR_CUDA;
  }
  a.chunk = q4_plain_chunk(a.B, a.H, L_max, sms);
  a.splits = static_cast<int>((L_max + a.chunk - 1) / a.chunk);
  return launch_q4_f32(a, s) == cudaSuccess ? LLA_OK : LLA_ERR_CUDA;
}

}  // extern "C"
