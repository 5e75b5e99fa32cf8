// kv4_store.cu -- rows of keys and values into the paged 4-bit cache and back.
//
// Append, per (token, head, group of channels): m = min x, s = bf16((max x -
// m) / 15), code = round((x - m) / s).  x and m are bf16, so m is exact and the
// codes can be too: where all of a group's values lie within 2^13 of each other
// in size (nearly always), D = x - m is exact in fp32 with at most 22
// significant bits, so that D / s is a midpoint between two codes or at least
// 2^-22 away from one, relative.  A quotient that is exact where the true one
// is representable, and off by 2^-24 else, then rounds to the right code; it
// comes from an approximate one by one correction with its exact remainder
// (Markstein's method).  The other groups, and those whose range leaves fp32's,
// take code_of, which compares D with the midpoint.
//
// Minimum and maximum of a group are taken on bf16 pairs (two values an
// instruction; a NaN stays) and cross the group's threads in one word.
//
// Append: a thread holds 16 channels (two loads each of K and V); what a group
// costs once -- range, scale, address -- is shared by twice the values it was
// with eight channels a thread (45 -> 38 us for 16381 tokens of 16 heads, d = 128).
// Bound: issue slots (70 % taken, about 115 instructions for eight values), then HBM.
// Gather: a thread holds eight channels of K and V of two tokens, four loads in
// flight.  Bound: HBM; 16384 tokens of 16 heads, d = 128 in 27 us.
#include <cuda_bf16.h>

#include "fa.h"
#include "kv4.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kRowThreads = 256;
constexpr int kTokens = 2;  // tokens a thread

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ float round_bf16(float x) {
  return __bfloat162float(__float2bfloat16_rn(x));
}

// The code of x given its group's minimum and scale > 0, inv ~ 1 / scale, for
// any finite values.
__device__ __forceinline__ uint32_t code_of(float x, float m, float s, float inv) {
  const float D = x - m;
  const float f = fminf(floorf(D * inv), 14.f);
  const float r = D - (f + 0.5f) * s;  // the midpoint has 13 bits; exact near 0
  bool up = r > 0.f;
  if (r == 0.f) {  // at the midpoint as far as fp32 sees
    const float bb = D - x;
    const float err = (x - (D - bb)) + (-m - bb);  // x - m - D, exactly
    up = err > 0.f || (err == 0.f && (static_cast<int>(f) & 1));
  }
  return static_cast<uint32_t>(static_cast<int>(f)) + (up ? 1u : 0u);
}

// Larger and smaller of bf16 pairs; NaN if either is.
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Quantises this thread's 16 channels; kLanes threads share a group.  Returns
// the words of codes, and the group's param in *param.
template <int kLanes>
__device__ __forceinline__ uint2 quantise16(const uint4 (&in)[2], uint32_t* param) {
  const uint32_t w[8] = {in[0].x, in[0].y, in[0].z, in[0].w, in[1].x, in[1].y, in[1].z, in[1].w};
  // Largest and smallest value, and the smallest size above zero (sizes moved by
  // 0x7fff: zero is then the top of the signed range, and no half carries into
  // the other).
  uint32_t top = w[0], bot = w[0], least = (w[0] & 0x7fff7fffu) + 0x7fff7fffu;
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    top = max_bf16x2(top, w[i]);
    bot = min_bf16x2(bot, w[i]);
    least = __vmins2(least, (w[i] & 0x7fff7fffu) + 0x7fff7fffu);
  }
  // (largest, smallest negated) of the halves, then of the group's threads
  uint32_t both = max_bf16x2(__byte_perm(top, bot, 0x5410) ^ 0x80000000u,
                             __byte_perm(top, bot, 0x7632) ^ 0x80000000u);
#pragma unroll
  for (int d = 1; d < kLanes; d <<= 1) both = max_bf16x2(both, __shfl_xor_sync(0xffffffffu, both, d));
  const float hi = bf16_lo(both), lo = -bf16_hi(both);
  const float big = fmaxf(fabsf(lo), fabsf(hi));
  // An infinity, or a NaN.
  if (!(big < INFINITY)) {
    *param = 0x7fc07fc0u;
    return make_uint2(0, 0);
  }
  const float span = hi - lo;
  // One below the smallest size, NaN if there is none.
  float small = __uint_as_float(min((least & 0xffffu) - 0x8000u, (least >> 16) - 0x8000u) << 16);
  if (lo != 0.f) small = fminf(small, fabsf(lo));
  const bool near = big < 0x1p125f && span > 0x1p-60f && !(small < 0x1p-13f * big);
  if (near) {
    // span / 15 as the quotients below: an approximate one and its exact remainder
    constexpr float k15th = 1.f / 15.f;
    const float q15 = span * k15th;
    *param = pack_bf16(fmaf(fmaf(-15.f, q15, span), k15th, q15), lo);
    const float s = bf16_lo(*param);
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
    const uint64_t m2 = f2_pack(lo, lo), s2 = f2_pack(-s, -s), i2 = f2_pack(inv, inv);
    constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: a sum's low bits are the integer
    const uint64_t magic = f2_pack(kMagic, kMagic);
    uint32_t t[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint64_t D = f2_sub(f2_pack(bf16_lo(w[i]), bf16_hi(w[i])), m2);
      const uint64_t q = f2_mul(D, i2);
      const uint64_t r = f2_fma(q, s2, D);
      float a, b;
      f2_unpack(f2_add(f2_fma(r, i2, q), magic), a, b);
      t[2 * i] = __float_as_uint(a);
      t[2 * i + 1] = __float_as_uint(b);
    }
    // Nibble p holds channel 2 p, nibble 4 + p channel 2 p + 1.  The integers
    // still carry the bits of kMagic: their sum is taken off at the end.
    uint32_t codes[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int p = 7; p >= 0; --p) codes[j] = codes[j] * 16u + t[8 * j + (p < 4 ? 2 * p : 2 * (p - 4) + 1)];
    return make_uint2(codes[0] - 0x4b400000u * 0x11111111u, codes[1] - 0x4b400000u * 0x11111111u);
  }
  // The difference of finite values can pass fp32's range, and a subnormal
  // scale has no reciprocal: such groups are scaled by a power of two first
  // (exact).
  float up = 1.f, down = 1.f;
  if (big >= 0x1p125f) {
    up = 0x1p-4f;
    down = 0x1p4f;
  } else if (span <= 0x1p-60f) {
    up = 0x1p64f;
    down = 0x1p-64f;
  }
  const float m = lo * up;
  const float s_true = round_bf16(__fdiv_rn(hi * up - m, 15.f) * down);
  *param = (__float_as_uint(s_true) >> 16) | (__float_as_uint(lo) & 0xffff0000u);
  if (!(s_true > 0.f)) return make_uint2(0, 0);
  const float s = s_true * up;
  const float inv = __frcp_rn(s);
  uint32_t codes[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    codes[i >> 2] |= code_of(bf16_lo(w[i]) * up, m, s, inv) << (4 * (i & 3));
    codes[i >> 2] |= code_of(bf16_hi(w[i]) * up, m, s, inv) << (4 * (i & 3) + 16);
  }
  return make_uint2(codes[0], codes[1]);
}

// grid (token blocks, heads); a block holds kRowThreads / (d / 16) tokens.
template <int kD, int kGroup>
__global__ void __launch_bounds__(kRowThreads) kv4_append_kernel(const Kv4RowsArgs a) {
  constexpr int tpr = kD / 16;  // threads a row: 4, 8 or 16, so a warp holds whole rows
  const int t = blockIdx.x * (kRowThreads / tpr) + threadIdx.x / tpr;
  const int part = threadIdx.x % tpr;
  const int h = blockIdx.y;
  int slot = -1;
  uint4 k[2], v[2];
  k[0] = k[1] = v[0] = v[1] = make_uint4(0, 0, 0, 0);
  if (t < a.T) {
    slot = a.slots[t];
    const uint4* ks = reinterpret_cast<const uint4*>(a.k_in + static_cast<long long>(t) * a.k_ts +
                                                     static_cast<long long>(h) * a.k_hs) + 2 * part;
    const uint4* vs = reinterpret_cast<const uint4*>(a.v_in + static_cast<long long>(t) * a.v_ts +
                                                     static_cast<long long>(h) * a.v_hs) + 2 * part;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      k[i] = __ldg(ks + i);
      v[i] = __ldg(vs + i);
    }
  }
  if (slot < -1 || slot >= a.num_slots) {
    atomicCAS(a.input_err, 0, FA_ERR_INVALID_ARG);
    slot = -1;
  }
  uint32_t kp, vp;
  const uint2 kc = quantise16<kGroup / 16>(k, &kp);
  const uint2 vc = quantise16<kGroup / 16>(v, &vp);
  if (slot < 0) return;
  const int off = slot & ((1 << a.lay.page_shift) - 1);
  uint8_t* rec =
      a.cache + (static_cast<long long>(slot >> a.lay.page_shift) * a.Hkv + h) * a.lay.record;
  uint8_t* codes = rec + off * a.lay.code_row + part * 8;
  *reinterpret_cast<uint2*>(codes) = kc;
  *reinterpret_cast<uint2*>(codes + a.lay.v_codes) = vc;
  if (part % (kGroup / 16) == 0) {
    uint8_t* params = rec + off * a.lay.param_row + part / (kGroup / 16) * 4;
    *reinterpret_cast<uint32_t*>(params + a.lay.k_params) = kp;
    *reinterpret_cast<uint32_t*>(params + a.lay.v_params) = vp;
  }
}

// The eight values of a word of codes: 0x4300 | c is 128 + c in bf16, c follows
// exactly, and one bf16 FMA rounds minimum + scale * c once.
__device__ __forceinline__ uint4 values8(uint32_t codes, uint32_t param) {
  const uint32_t s = __byte_perm(param, param, 0x1010), m = __byte_perm(param, param, 0x3232);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t c = ((codes >> (4 * i)) & 0x000f000fu) | 0x43004300u;
    asm("{\n\t.reg .b32 t;\n\t"
        "add.rn.bf16x2 t, %1, %2;\n\t"
        "fma.rn.bf16x2 %0, t, %3, %4;\n\t}"
        : "=r"(w[i])
        : "r"(c), "r"(0xc300c300u), "r"(s), "r"(m));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int kD, int kGroup>
__global__ void __launch_bounds__(kRowThreads) kv4_gather_kernel(const Kv4RowsArgs a) {
  constexpr int tpr = kD / 8, pass = kRowThreads / tpr;
  const int t0 = blockIdx.x * (kTokens * pass) + threadIdx.x / tpr;
  const int part = threadIdx.x % tpr;
  const int h = blockIdx.y;
  const int g = part / (kGroup / 8);
  int slot[kTokens];
  uint32_t kc[kTokens], vc[kTokens], kp[kTokens], vp[kTokens];
#pragma unroll
  for (int i = 0; i < kTokens; ++i) slot[i] = t0 + i * pass < a.T ? a.slots[t0 + i * pass] : -1;
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
    if (slot[i] < -1 || slot[i] >= a.num_slots) {
      atomicCAS(a.input_err, 0, FA_ERR_INVALID_ARG);
      slot[i] = -1;
    }
    if (slot[i] < 0) continue;
    const int off = slot[i] & ((1 << a.lay.page_shift) - 1);
    const uint8_t* rec =
        a.cache + (static_cast<long long>(slot[i] >> a.lay.page_shift) * a.Hkv + h) * a.lay.record;
    const uint8_t* c = rec + off * a.lay.code_row + part * 4;
    const uint8_t* p = rec + off * a.lay.param_row + g * 4;
    kc[i] = *reinterpret_cast<const uint32_t*>(c);
    vc[i] = *reinterpret_cast<const uint32_t*>(c + a.lay.v_codes);
    kp[i] = *reinterpret_cast<const uint32_t*>(p + a.lay.k_params);
    vp[i] = *reinterpret_cast<const uint32_t*>(p + a.lay.v_params);
  }
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
    if (slot[i] < 0) continue;
    const long long out = (static_cast<long long>(t0 + i * pass) * a.Hkv + h) * tpr + part;
    reinterpret_cast<uint4*>(a.k_out)[out] = values8(kc[i], kp[i]);
    reinterpret_cast<uint4*>(a.v_out)[out] = values8(vc[i], vp[i]);
  }
}

dim3 rows_grid(const Kv4RowsArgs& a) {
  const int per = kTokens * (kRowThreads / (a.d / 8));
  return dim3(static_cast<unsigned>((a.T + per - 1) / per), static_cast<unsigned>(a.Hkv));
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4RowsArgs& a, cudaStream_t stream) {
  const dim3 grid = rows_grid(a);
  const bool g32 = a.group == 32;
  switch (a.d) {
    case 64:
      if (g32) kv4_append_kernel<64, 32><<<grid, kRowThreads, 0, stream>>>(a);
      else kv4_append_kernel<64, 64><<<grid, kRowThreads, 0, stream>>>(a);
      break;
    case 128:
      if (g32) kv4_append_kernel<128, 32><<<grid, kRowThreads, 0, stream>>>(a);
      else kv4_append_kernel<128, 64><<<grid, kRowThreads, 0, stream>>>(a);
      break;
    case 256:
      if (g32) kv4_append_kernel<256, 32><<<grid, kRowThreads, 0, stream>>>(a);
      else kv4_append_kernel<256, 64><<<grid, kRowThreads, 0, stream>>>(a);
      break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

cudaError_t launch_kv4_gather(const Kv4RowsArgs& a, cudaStream_t stream) {
  const dim3 grid = rows_grid(a);
  const bool g32 = a.group == 32;
  switch (a.d) {
    case 64:
      if (g32) kv4_gather_kernel<64, 32><<<grid, kRowThreads, 0, stream>>>(a);
      else kv4_gather_kernel<64, 64><<<grid, kRowThreads, 0, stream>>>(a);
      break;
    case 128:
      if (g32) kv4_gather_kernel<128, 32><<<grid, kRowThreads, 0, stream>>>(a);
      else kv4_gather_kernel<128, 64><<<grid, kRowThreads, 0, stream>>>(a);
      break;
    case 256:
      if (g32) kv4_gather_kernel<256, 32><<<grid, kRowThreads, 0, stream>>>(a);
      else kv4_gather_kernel<256, 64><<<grid, kRowThreads, 0, stream>>>(a);
      break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace fa
