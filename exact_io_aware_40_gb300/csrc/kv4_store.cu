// kv4_store.cu -- rows of keys and values into the paged 4-bit cache and back.
//
// Append, per (token, head, group of channels): m = min x, s = bf16((max x -
// m) / 15), code = round((x - m) / s).  x and m are bf16, so m is exact and
// the code's decision can be exact too: with D = x - m in fp32 the quotient D *
// (1 / s) gives a candidate, and comparing D with the midpoint (f + 1/2) s,
// which is exact in fp32 (13 significant bits), decides between f and f + 1.
// Only where D equals the midpoint can D's own rounding error matter, and then
// its sign is the sign of that error (two-sum), or a tie.
//
// Both kernels move each byte once; a thread holds eight channels (16 bytes of
// bf16, one 32-bit word of codes) and a group's 4 or 8 threads reduce by shuffles.
#include <cuda_bf16.h>

#include <cfloat>

#include "fa.h"
#include "kv4.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kRowThreads = 256;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ float round_bf16(float x) {
  return __bfloat162float(__float2bfloat16_rn(x));
}

// The code of x given its group's minimum and scale > 0, inv ~ 1 / scale.
__device__ __forceinline__ uint32_t code_of(float x, float m, float s, float inv) {
  const float D = x - m;
  const float f = fminf(floorf(D * inv), 14.f);
  const float r = D - (f + 0.5f) * s;
  bool up = r > 0.f;
  if (r == 0.f) {  // at the midpoint as far as fp32 sees
    const float bb = D - x;
    const float err = (x - (D - bb)) + (-m - bb);  // x - m - D, exactly
    up = err > 0.f || (err == 0.f && (static_cast<int>(f) & 1));
  }
  return static_cast<uint32_t>(static_cast<int>(f)) + (up ? 1u : 0u);
}

// Quantises this thread's eight channels; `lanes` threads share a group.
// Returns the word of codes, and the group's param in *param.
template <int kLanes>
__device__ __forceinline__ uint32_t quantise8(const uint4 in, uint32_t* param) {
  const uint32_t w[4] = {in.x, in.y, in.z, in.w};
  float x[8];
  float lo = FLT_MAX, hi = -FLT_MAX;
  bool odd = false;  // NaN or infinity
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(w[i]);
    x[2 * i + 1] = bf16_hi(w[i]);
    odd = odd || (w[i] & 0x7f80u) == 0x7f80u || (w[i] & 0x7f800000u) == 0x7f800000u;
    lo = fminf(lo, fminf(x[2 * i], x[2 * i + 1]));
    hi = fmaxf(hi, fmaxf(x[2 * i], x[2 * i + 1]));
  }
#pragma unroll
  for (int d = 1; d < kLanes; d <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, d));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, d));
    odd = __shfl_xor_sync(0xffffffffu, odd ? 1 : 0, d) || odd;
  }
  if (odd) {
    *param = 0x7fc07fc0u;
    return 0;
  }
  // The difference of finite values can pass fp32's range, and a subnormal
  // scale has no reciprocal: such groups are scaled by a power of two first
  // (exact).
  const float big = fmaxf(fabsf(lo), fabsf(hi));
  float up = 1.f, down = 1.f;
  if (big > 0x1p125f) {
    up = 0x1p-4f;
    down = 0x1p4f;
  } else if (hi - lo < 0x1p-60f) {
    up = 0x1p64f;
    down = 0x1p-64f;
  }
  const float m = lo * up;
  const float s_true = round_bf16(__fdiv_rn(hi * up - m, 15.f) * down);
  *param = (__float_as_uint(s_true) >> 16) | (__float_as_uint(lo) & 0xffff0000u);
  if (!(s_true > 0.f)) return 0;
  const float s = s_true * up;
  const float inv = __frcp_rn(s);
  uint32_t codes = 0;
#pragma unroll
  for (int c = 0; c < 8; ++c)
    codes |= code_of(x[c] * up, m, s, inv) << (4 * ((c & 1) * 4 + c / 2));
  return codes;
}

// grid (token blocks, heads); a block holds kRowThreads / (d / 8) tokens.
template <int kGroup>
__global__ void __launch_bounds__(kRowThreads) kv4_append_kernel(const Kv4RowsArgs a) {
  const int tpr = a.d / 8;  // threads a row: 8, 16 or 32, so a warp holds whole rows
  const int t = blockIdx.x * (kRowThreads / tpr) + threadIdx.x / tpr;
  const int part = threadIdx.x % tpr;
  const int h = blockIdx.y;
  int slot = -1;
  if (t < a.T) slot = a.slots[t];
  if (slot < -1 || slot >= a.num_slots) {
    atomicCAS(a.input_err, 0, FA_ERR_INVALID_ARG);
    slot = -1;
  }
  uint4 k = make_uint4(0, 0, 0, 0), v = k;
  if (slot >= 0) {
    k = __ldg(reinterpret_cast<const uint4*>(a.k_in + static_cast<long long>(t) * a.k_ts +
                                             static_cast<long long>(h) * a.k_hs) + part);
    v = __ldg(reinterpret_cast<const uint4*>(a.v_in + static_cast<long long>(t) * a.v_ts +
                                             static_cast<long long>(h) * a.v_hs) + part);
  }
  uint32_t kp, vp;
  const uint32_t kc = quantise8<kGroup / 8>(k, &kp);
  const uint32_t vc = quantise8<kGroup / 8>(v, &vp);
  if (slot < 0) return;
  const int off = slot & ((1 << a.lay.page_shift) - 1);
  uint8_t* rec = a.cache + (static_cast<long long>(slot >> a.lay.page_shift) * a.Hkv + h) * a.lay.record;
  *reinterpret_cast<uint32_t*>(rec + off * a.lay.code_row + part * 4) = kc;
  *reinterpret_cast<uint32_t*>(rec + a.lay.v_codes + off * a.lay.code_row + part * 4) = vc;
  if (part % (kGroup / 8) == 0) {
    const int g = part / (kGroup / 8);
    *reinterpret_cast<uint32_t*>(rec + a.lay.k_params + off * a.lay.param_row + g * 4) = kp;
    *reinterpret_cast<uint32_t*>(rec + a.lay.v_params + off * a.lay.param_row + g * 4) = vp;
  }
}

__device__ __forceinline__ uint4 values8(uint32_t codes, uint32_t param) {
  const float s = bf16_lo(param), m = bf16_hi(param);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)  // s * code has at most 12 significant bits: one rounding in the fma
    w[i] = pack_bf16(fmaf(static_cast<float>((codes >> (4 * i)) & 15u), s, m),
                     fmaf(static_cast<float>((codes >> (4 * i + 16)) & 15u), s, m));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int kGroup>
__global__ void __launch_bounds__(kRowThreads) kv4_gather_kernel(const Kv4RowsArgs a) {
  const int tpr = a.d / 8;
  const int t = blockIdx.x * (kRowThreads / tpr) + threadIdx.x / tpr;
  const int part = threadIdx.x % tpr;
  const int h = blockIdx.y;
  if (t >= a.T) return;
  const int slot = a.slots[t];
  if (slot < 0 || slot >= a.num_slots) {
    if (slot != -1) atomicCAS(a.input_err, 0, FA_ERR_INVALID_ARG);
    return;
  }
  const int off = slot & ((1 << a.lay.page_shift) - 1);
  const int g = part / (kGroup / 8);
  const uint8_t* rec =
      a.cache + (static_cast<long long>(slot >> a.lay.page_shift) * a.Hkv + h) * a.lay.record;
  const uint32_t kc = *reinterpret_cast<const uint32_t*>(rec + off * a.lay.code_row + part * 4);
  const uint32_t vc =
      *reinterpret_cast<const uint32_t*>(rec + a.lay.v_codes + off * a.lay.code_row + part * 4);
  const uint32_t kp =
      *reinterpret_cast<const uint32_t*>(rec + a.lay.k_params + off * a.lay.param_row + g * 4);
  const uint32_t vp =
      *reinterpret_cast<const uint32_t*>(rec + a.lay.v_params + off * a.lay.param_row + g * 4);
  const long long out = (static_cast<long long>(t) * a.Hkv + h) * tpr + part;
  reinterpret_cast<uint4*>(a.k_out)[out] = values8(kc, kp);
  reinterpret_cast<uint4*>(a.v_out)[out] = values8(vc, vp);
}

dim3 rows_grid(const Kv4RowsArgs& a) {
  const int per = kRowThreads / (a.d / 8);
  return dim3(static_cast<unsigned>((a.T + per - 1) / per), static_cast<unsigned>(a.Hkv));
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4RowsArgs& a, cudaStream_t stream) {
  if (a.group == 32)
    kv4_append_kernel<32><<<rows_grid(a), kRowThreads, 0, stream>>>(a);
  else
    kv4_append_kernel<64><<<rows_grid(a), kRowThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv4_gather(const Kv4RowsArgs& a, cudaStream_t stream) {
  if (a.group == 32)
    kv4_gather_kernel<32><<<rows_grid(a), kRowThreads, 0, stream>>>(a);
  else
    kv4_gather_kernel<64><<<rows_grid(a), kRowThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace fa
