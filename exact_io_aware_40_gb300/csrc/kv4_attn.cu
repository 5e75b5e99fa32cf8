// kv4_attn.cu -- attention over the paged 4-bit cache for few query rows.
//
// Blocks of 8, 16 or 32 rows (queries x query heads of one K/V head) share each
// read of the cache; one read of the keys and values is all the memory traffic
// there is, so the kernel is built around it: a warp walks the cache on its own,
// 32 tokens at a time, with its copies (cp.async) several steps ahead and no
// barrier with any other warp until its item ends.  Per 16 tokens and a K/V head:
//
//   S^T = K Q^T   mma m16n8k16, A = 16 tokens x 16 channels of codes, B = Q^T
//   p   = 2^(S scale log2e - m), running maximum m and sums in fp32
//   O^T += V^T P^T   A = 16 channels x 16 tokens of values, B = P^T
//
// Tokens (then channels) are the 16 rows of the product and query rows its 8
// columns, so one to eight rows cost one product.
//
// Codes become numbers without a conversion.  K: 0x4300 | c is 128 + c in bf16,
// and per group of channels sum q (m + s c) = s sum q (128 + c) + (m - 128 s)
// sum q, two FMAs per score on exact products; 128 exceeds the codes by a factor
// of 8 to 128, which costs 7 of fp32's 24 bits at most.  V: 0x6400 | c is 1024 +
// c and 0x6400 | 16 c is 1024 + 16 c in fp16; one exact operation makes c - 8 of
// either, one FMA the value.  (An offset as K's is no choice here: the values
// average out over a long context and the offset would not.)  V and P are fp16
// in the product, which rounds them to 2^-12 where bf16 has 2^-9, so that the
// rounding of O to bf16 is what is left; the price is a scale.  V is taken in
// units of 2^vexp, a power of two that grows with the largest value met (as the
// running maximum does) and is 1 for values of ordinary size, P in units of
// 2^-kShift of the maximum's weight: weights below 2^-34 of it and values below
// 2^-20 of the largest one lose bits.
//
// Which token is which row of the product is free as long as both products
// agree; token_of and the swizzle of the staged 16-byte chunks (twist) are chosen
// so that a warp's reads of its staged codes meet no bank twice (K), or twice
// at most (V).
//
// Measured (d = 128, 16 requests of 8192 tokens, 8 K/V heads, 8 query heads each):
// 44 us for 168 MB of cache, of which 10 to 13 us are paid once a call (launch,
// shares, first copies, the exchange between warps, merge); in between 5.2 to 5.6
// TB/s.  Bound: issue slots (57 % taken, with 16 warps an SM and each warp's chain
// from codes to weights to hide), about 380 instructions for 16 tokens of a head.
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kernels.h"
#include "kv4.h"
#include "kv4_sched.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kWarps = 4;
constexpr int kAttnThreads = 32 * kWarps;
constexpr int kStepTokens = 32;
constexpr int kTile = kWarps * kStepTokens;  // one step of every warp
constexpr int kLead = 2;        // tiles that a change of items costs
constexpr float kGrow = 4.f;    // log2 units: m moves only when the maximum passes it by more
constexpr float kShift = 10.f;  // P is at most 2^(kGrow + kShift)
constexpr float kLn2f = 0.693147180559945309f;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// d = a b: a zero accumulator that takes no registers
__device__ __forceinline__ void mma_bf16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                               uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t add_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t keep, uint32_t set) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(x), "r"(keep), "r"(set));
  return r;
}
// Nibbles i and i + 4 of w as bf16 values 128 + code.
__device__ __forceinline__ uint32_t k_codes(uint32_t w, int i) {
  return and_or(w >> (4 * i), 0x000f000fu, 0x43004300u);
}
// Nibbles i and i + 4 of w as fp16 values code - 8.
__device__ __forceinline__ uint32_t v_codes(uint32_t w, int i) {
  const uint32_t x = i < 2 ? w : w >> 8;
  if ((i & 1) == 0) return add_f16x2(and_or(x, 0x000f000fu, 0x64006400u), 0xe408e408u);  // -1032
  return fma_f16x2(and_or(x, 0x00f000f0u, 0x64006400u), 0x2c002c00u, 0xd480d480u);  // / 16 - 72
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ bool odd_param(uint32_t p) {  // NaN or infinity in either half
  return (p & 0x7f80u) == 0x7f80u || (p & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ float param_scale(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float param_min(uint32_t p) { return __uint_as_float(p & 0xffff0000u); }

// Token (of 16) that is row r of the product.
__device__ __forceinline__ int token_of(int r) { return (r & 8) | ((r & 1) << 2) | ((r >> 1) & 3); }

// The 16-byte chunks of a staged row of codes are permuted by an XOR with this.
template <int HD>
__device__ __forceinline__ int twist(int tok) {
  if (HD == 64) return (tok >> 2) & 1;
  if (HD == 128) return (tok & 2) | ((tok >> 2) & 1);
  return ((tok << 1) | ((tok >> 2) & 1)) & 7;
}

template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (N == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    w[0] = x.x;
    w[1] = x.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 x = reinterpret_cast<const uint4*>(p)[i];
      w[4 * i] = x.x;
      w[4 * i + 1] = x.y;
      w[4 * i + 2] = x.z;
      w[4 * i + 3] = x.w;
    }
  }
}

template <int HD, int GROUP, int NT>
struct AttnCfg {
  static constexpr int kGroups = HD / GROUP;
  static constexpr int kCodeRow = HD / 2, kParamRow = 4 * kGroups;
  static constexpr int kCodes = kStepTokens * kCodeRow, kParams = kStepTokens * kParamRow;
  static constexpr int kStage = 2 * (kCodes + kParams);  // bytes: K codes, V codes, K, V params
  static_assert(kStage % 128 == 0, "the swizzle works on addresses");
  // As many as the resident CTAs leave room for.
  static constexpr int kStages = HD == 64 ? 4 : HD == 128 && (NT > 1 || GROUP == 64) ? 3 : 2;
  static constexpr int kStageBytes = kWarps * kStages * kStage;
  static constexpr int kMergeBytes = kWarps * 8 * HD * 4;  // 8 rows of every warp's O
  static constexpr int kSmem = kStageBytes > kMergeBytes ? kStageBytes : kMergeBytes;
  static constexpr int kRows = 8 * NT;
  // Resident CTAs per SM the registers are bounded for.  (Five or six at d = 64
  // are no faster: 16 requests of 8192 tokens 54 and 58 us, four 52.)
  static constexpr int kMinCtas = HD == 256 ? 2 : NT == 4 ? 2 : NT == 2 ? 3 : 4;
};

template <int HD, int GROUP, int NT>
__global__ void __launch_bounds__(kAttnThreads, AttnCfg<HD, GROUP, NT>::kMinCtas)
    kv4_attn_kernel(const Kv4AttnArgs a) {
  using C = AttnCfg<HD, GROUP, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long scratch[kWarps + 2];
  // The walk through the share: touched once an item, it would only take
  // registers.  Thread 0 moves it on between two barriers.
  __shared__ Kv4Walk<kTile> w;
  __shared__ int4 record;
  __shared__ float stat[2][kWarps][C::kRows];
  // The merge may be launched; it waits for this grid's end by itself.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = lane >> 2, q = lane & 3;  // row / column pair of the product's fragments

  const Kv4Share share = kv4_share<kTile, kAttnThreads, false>(a, C::kRows, a.whole_items ? 1 : kLead + 1, scratch);
  long long u = share.per * blockIdx.x;
  const long long u_end = min(share.total, u + share.per);
  if (tid == 0 && u >= share.total && !a.whole_items) a.split[blockIdx.x] = make_int4(0, 0, 0, 0);
  if (u >= share.total) return;
  bool first_item = true;
  if (tid == 0) {
    w.seek(a, share, u, C::kRows);
    record = make_int4(0, 0, 0, 0);
  }
  __syncthreads();
  const uint8_t* stage0 = smem + warp * C::kStages * C::kStage;
  const uint32_t stage0_u32 = smem_u32(stage0);

  const float inv_scale = 1.f / a.scale_log2;
  // Lane constants of the staged layout.
  const int t0 = token_of(r);  // K, P: rows r and r + 8 are tokens t0 and t0 + 8
  const int k_at = t0 * C::kCodeRow + twist<HD>(t0) * 16 + q * 4;
  const int kp_at = 2 * C::kCodes + t0 * C::kParamRow;
  int v_at[2], vp_at[2];       // V: tokens ta[e] and ta[e] + 8 of this lane's columns
  int ta[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    ta[e] = token_of(2 * q + e);
    const int byte = r * (HD / 16);
    v_at[e] = C::kCodes + ta[e] * C::kCodeRow + (((byte >> 4) ^ twist<HD>(ta[e])) << 4) + (byte & 15);
    vp_at[e] = 2 * C::kCodes + C::kParams + ta[e] * C::kParamRow + (r * (HD / 8)) / GROUP * 4;
  }
  // Copies: chunk `lane` of 16 tokens' codes.
  const long long page_bytes = static_cast<long long>(a.Hkv) * a.lay.record;
  const int in_page = (1 << a.lay.page_shift) - 1;
  const int cp_tok = (lane * 16) / C::kCodeRow;
  const uint32_t cp_dst =
      cp_tok * C::kCodeRow + ((((lane * 16) % C::kCodeRow >> 4) ^ twist<HD>(cp_tok & 7)) << 4);

  while (u < u_end) {
    int first_tile, last_tile;
    const long long u_next = kv4_part(a, w, u, u_end, &first_tile, &last_tile);
    if (first_tile >= last_tile) break;  // the share ends before the item's tiles
    const int tok0 = (w.blk.tile_lo + first_tile) * kTile + warp * kStepTokens;
    const int hi = w.blk.hi, all_hi = w.blk.all_hi, all_lo = w.blk.all_lo, kv = w.req.kv;
    const int* table = a.table + static_cast<long long>(w.b) * a.max_pages;
    // Steps of this warp that hold a key some row sees.
    const int steps =
        min(last_tile - first_tile, max(0, (hi - tok0 + kTile - 1) / kTile));

    // ------------------------------------------------ copies, kStages - 1 steps ahead
    int page = 0, page_next = 0;  // lane l: page of half l % 2 of step 16 k + l / 2
    auto fetch_page = [&](int i) -> int {
      const int tok = tok0 + (i + (lane >> 1)) * kTile + (lane & 1) * 16;
      if (i + (lane >> 1) >= steps || tok >= hi) return 0;
      int p;  // volatile: issued here, long before it is used
      asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(p) : "l"(table + (tok >> a.lay.page_shift)));
      return p;
    };
    auto valid_page = [&](int p) -> int {
      if (p >= 0 && p < a.num_pages) return p;
      atomicCAS(a.input_err, 0, 1);
      return 0;
    };
    page_next = fetch_page(0);
    const uint8_t* head_base = a.cache + static_cast<long long>(w.h) * a.lay.record;
    auto issue = [&](int i) {
      if (i < steps) {
        if ((i & 15) == 0) {
          page = valid_page(page_next);
          page_next = fetch_page(i + 16);
        }
        const uint32_t dst = stage0_u32 + (i % C::kStages) * C::kStage;
        const int tok = tok0 + i * kTile;
        // `n` tokens (16 or 32) from the step's token 16 hf on, in one page.
        auto copy = [&](int hf, auto tokens) {
          constexpr int n = decltype(tokens)::value;
          const int pg = __shfl_sync(0xffffffffu, page, 2 * (i & 15) + hf);
          const int off = (tok + hf * 16) & in_page;
          const uint8_t* rec = head_base + pg * page_bytes;
          const uint8_t* kc = rec + (off * C::kCodeRow + lane * 16);
          const uint8_t* vc = kc + a.lay.v_codes;
#pragma unroll
          for (int j = 0; j < n * C::kCodeRow / 512; ++j) {
            // 512 bytes are 16, 8 or 4 rows on; 4 rows change the twist's low bit
            const uint32_t at = dst + hf * 16 * C::kCodeRow + j * 512 +
                                (HD == 256 && (j & 1) ? cp_dst ^ 16u : cp_dst);
            cp_async16(at, kc + j * 512);
            cp_async16(at + C::kCodes, vc + j * 512);
          }
          // K's params, then V's: chunks of 16 bytes, side by side over the lanes
          constexpr int kChunks = n * C::kParamRow / 16;  // of either
          const uint32_t pat = dst + 2 * C::kCodes + hf * 16 * C::kParamRow;
          if constexpr (kChunks >= 32) {
            const uint8_t* kp = rec + (a.lay.k_params + off * C::kParamRow + lane * 16);
#pragma unroll
            for (int j = 0; j < kChunks / 32; ++j) {
              cp_async16(pat + lane * 16 + j * 512, kp + j * 512);
              cp_async16(pat + C::kParams + lane * 16 + j * 512,
                         kp + (a.lay.v_params - a.lay.k_params) + j * 512);
            }
          } else if (lane < 2 * kChunks) {
            const bool v = lane >= kChunks;
            const int l = (v ? lane - kChunks : lane) * 16;
            cp_async16(pat + (v ? C::kParams : 0) + l,
                       rec + ((v ? a.lay.v_params : a.lay.k_params) + off * C::kParamRow + l));
          }
        };
        if (in_page >= 31) {
          copy(0, std::integral_constant<int, 32>{});
        } else {
          copy(0, std::integral_constant<int, 16>{});
          // nothing there: left as it is, and masked
          if (tok + 16 < hi) copy(1, std::integral_constant<int, 16>{});
        }
      }
      cp_commit();
    };
    // This block's queries: loaded while the first pages are looked up.
    uint32_t qf[NT][HD / 32][4];       // B fragments of Q^T
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int row = 8 * n + r;
      const bool have = row < w.blk.rows;
      const int gr = w.blk.row0 + row;
      const int t = gr / a.per_kv, head = w.h * a.per_kv + gr - t * a.per_kv;
      const uint16_t* src = a.Q + static_cast<long long>(w.req.start + t) * a.q_ts +
                            static_cast<long long>(head) * a.q_hs + 8 * q;
#pragma unroll
      for (int c = 0; c < HD / 32; ++c) {
        qf[n][c][0] = qf[n][c][1] = qf[n][c][2] = qf[n][c][3] = 0;
        if (have)  // volatile: issued here
          asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(qf[n][c][0]), "=r"(qf[n][c][1]), "=r"(qf[n][c][2]), "=r"(qf[n][c][3])
                       : "l"(src + 32 * c));
      }
    }
#pragma unroll
    for (int i = 0; i < C::kStages - 1; ++i) issue(i);

    // ------------------------------------------------ sums over the queries' groups
    float qsum[NT][C::kGroups][2];     // rows 2 q, 2 q + 1
    int pos[NT][2];                    // position of rows 2 q, 2 q + 1 (-1: no such row)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float part[C::kGroups];
#pragma unroll
      for (int g = 0; g < C::kGroups; ++g) part[g] = 0.f;
#pragma unroll
      for (int c = 0; c < HD / 32; ++c) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          part[32 * c / GROUP] += __uint_as_float(qf[n][c][i] << 16) +
                                  __uint_as_float(qf[n][c][i] & 0xffff0000u);
      }
#pragma unroll
      for (int g = 0; g < C::kGroups; ++g) {
        part[g] += __shfl_xor_sync(0xffffffffu, part[g], 1);
        part[g] += __shfl_xor_sync(0xffffffffu, part[g], 2);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          qsum[n][g][e] = __shfl_sync(0xffffffffu, part[g], (2 * q + e) * 4);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int rr = 8 * n + 2 * q + e;
        pos[n][e] = rr < w.blk.rows ? w.blk.pos0 + (w.blk.row0 + rr) / a.per_kv : -1;
      }
    }

    float acc[NT][HD / 16][4];
    float m_run[NT][2], l_run[NT][2];
    float top_s[NT][2];  // scores above it move the maximum: (m_run + kGrow) / scale
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < HD / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][i][e] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m_run[n][e] = -INFINITY;
        top_s[n][e] = -INFINITY;
        l_run[n][e] = 0.f;
      }
    }
    // V's unit: |minimum| < 2^(vexp + 14) and |scale| < 2^(vexp + 10) keep every
    // value below 2^15; `limit` holds both bounds as a param does.
    int vexp = 0;
    float v_unit = 1.f;  // 2^-vexp
    uint32_t limit = 0;

    // ------------------------------------------------ the walk over the tokens
#pragma unroll 1
    for (int i = 0; i < steps; ++i) {
      cp_wait<C::kStages - 2>();
      __syncwarp();  // every lane's copies have landed; step i - 1 has been read
      issue(i + C::kStages - 1);
      const int tok = tok0 + i * kTile;
      const uint8_t* st = stage0 + (i % C::kStages) * C::kStage;
      const bool edge = tok + kStepTokens > all_hi || tok < all_lo;

      // S^T of both halves
      float s[2][NT][4];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        uint32_t p0[C::kGroups], p1[C::kGroups];
        load_words(st + kp_at + hf * 16 * C::kParamRow, p0);
        load_words(st + kp_at + (hf * 16 + 8) * C::kParamRow, p1);
        const uint32_t row = static_cast<uint32_t>(k_at + hf * 16 * C::kCodeRow);
#pragma unroll
        for (int g = 0; g < C::kGroups; ++g) {
          float d[NT][4];
#pragma unroll
          for (int cc = 0; cc < GROUP / 32; ++cc) {
            const int c = g * (GROUP / 32) + cc;
            const uint32_t at = row ^ static_cast<uint32_t>(c * 16);
            const uint32_t w0 = *reinterpret_cast<const uint32_t*>(st + at);
            const uint32_t w1 = *reinterpret_cast<const uint32_t*>(st + at + 8 * C::kCodeRow);
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
              const uint32_t af[4] = {k_codes(w0, 2 * ks), k_codes(w1, 2 * ks),
                                      k_codes(w0, 2 * ks + 1), k_codes(w1, 2 * ks + 1)};
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                if (cc == 0 && ks == 0)
                  mma_bf16_first(d[n], af, qf[n][c][0], qf[n][c][1]);
                else
                  mma_bf16(d[n], af, qf[n][c][2 * ks], qf[n][c][2 * ks + 1]);
              }
            }
          }
          const float s0 = param_scale(p0[g]), s1 = param_scale(p1[g]);
          const float b0 = fmaf(-128.f, s0, param_min(p0[g]));
          const float b1 = fmaf(-128.f, s1, param_min(p1[g]));
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float* z = s[hf][n];
            const float q0 = qsum[n][g][0], q1 = qsum[n][g][1];
            z[0] = fmaf(d[n][0], s0, g ? fmaf(b0, q0, z[0]) : b0 * q0);
            z[1] = fmaf(d[n][1], s0, g ? fmaf(b0, q1, z[1]) : b0 * q1);
            z[2] = fmaf(d[n][2], s1, g ? fmaf(b1, q0, z[2]) : b1 * q0);
            z[3] = fmaf(d[n][3], s1, g ? fmaf(b1, q1, z[3]) : b1 * q1);
          }
        }
      }
      const bool upto = a.causal || a.window >= 0;
      auto visible = [&](int token, int p) {
        bool v = token < kv;
        if (upto) v = v && token <= p;
        if (a.window >= 0) v = v && token >= p - a.window;
        return v;
      };
      if (edge) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int token = tok + hf * 16 + t0 + (e & 2) * 4;
              s[hf][n][e] = visible(token, pos[n][e & 1]) ? s[hf][n][e] : -INFINITY;
            }
      }

      // V's params of this lane's eight tokens
      uint32_t par[2][4];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          par[hf][e] = *reinterpret_cast<const uint32_t*>(
              st + vp_at[e & 1] + (hf * 16 + (e & 2) * 4) * C::kParamRow);
      if (edge) {
        // Rows behind the last visible token may hold anything, and a value
        // that is not a number must not reach rows that do not see it (see
        // below): their weights are 0, which counts only for finite values.
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int token = tok + hf * 16 + ta[e & 1] + (e & 2) * 4;
            if (token >= hi || odd_param(par[hf][e])) par[hf][e] = 0;
          }
      }

      // Running maximum and V's unit: moved only when they are passed (by
      // kGrow), which after the first steps of an item is rare.
      uint32_t top_par = 0;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int e = 0; e < 4; ++e) top_par = __vmaxu2(top_par, par[hf][e] & 0x7fff7fffu);
      bool grow = __vmaxu2(top_par, limit) != limit;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          grow = grow || max3(fmaxf(s[0][n][e], s[0][n][e + 2]), s[1][n][e], s[1][n][e + 2]) > top_s[n][e];
      if (__any_sync(0xffffffffu, grow)) {
        // Exponents of the largest minimum and scale of the step, numbers only.
        int em = 0, es = 0;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!odd_param(par[hf][e])) {
              em = max(em, static_cast<int>((par[hf][e] >> 23) & 255));
              es = max(es, static_cast<int>((par[hf][e] >> 7) & 255));
            }
        em = __reduce_max_sync(0xffffffffu, em);
        es = __reduce_max_sync(0xffffffffu, es);
        // 1 (vexp 0) as long as it does: no param too large, the largest not small.
        const int need = max(max(em - 127 + 1 - 14, es - 127 + 1 - 10), -110);
        const int want = need <= 0 && need >= -20 ? 0 : need;
        float shrink = 1.f;
        if (limit == 0 || want > vexp) {
          if (limit != 0) shrink = exp2f(static_cast<float>(max(vexp - want, -126)));
          vexp = want;
          v_unit = exp2f(static_cast<float>(-vexp));
          // the largest bf16 below 2^(vexp + 14), and below 2^(vexp + 10)
          limit = (static_cast<uint32_t>(min(vexp + 14 + 127, 255) * 128 - 1) << 16) |
                  static_cast<uint32_t>(vexp + 10 + 127) * 128 - 1;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float alpha[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = fmaxf(fmaxf(s[0][n][e], s[0][n][e + 2]), fmaxf(s[1][n][e], s[1][n][e + 2])) *
                        a.scale_log2;
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            const bool up = top > m_run[n][e] + kGrow;
            alpha[e] = up ? ex2(m_run[n][e] - top) : 1.f;
            m_run[n][e] = up ? top : m_run[n][e];
            top_s[n][e] = (m_run[n][e] + kGrow) * inv_scale;
            l_run[n][e] *= alpha[e];
          }
#pragma unroll
          for (int k = 0; k < HD / 16; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[n][k][e] *= alpha[e & 1] * shrink;
        }
      }

      // P^T as B fragments
      uint32_t pf[2][NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float m0 = m_run[n][0] == -INFINITY ? 0.f : m_run[n][0] - kShift;
        const float m1 = m_run[n][1] == -INFINITY ? 0.f : m_run[n][1] - kShift;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const float p0 = ex2(fmaf(s[hf][n][0], a.scale_log2, -m0));
          const float p1 = ex2(fmaf(s[hf][n][1], a.scale_log2, -m1));
          const float p2 = ex2(fmaf(s[hf][n][2], a.scale_log2, -m0));
          const float p3 = ex2(fmaf(s[hf][n][3], a.scale_log2, -m1));
          l_run[n][0] += p0 + p2;
          l_run[n][1] += p1 + p3;
          pf[hf][n][0] = transpose8x8(pack_f16(p0, p1));
          pf[hf][n][1] = transpose8x8(pack_f16(p2, p3));
        }
      }

      // O^T += V^T P^T: this lane's rows are the HD / 8 channels from r HD / 8 on,
      // its columns tokens ta[0], ta[1] (first half of k) and those + 8
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        uint32_t sc[2], mn[2];  // scale and minimum + 8 scale of two tokens
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float sa = param_scale(par[hf][2 * k]), sb = param_scale(par[hf][2 * k + 1]);
          sc[k] = pack_f16(sa, sb);
          mn[k] = pack_f16(fmaf(8.f, sa, param_min(par[hf][2 * k])),
                           fmaf(8.f, sb, param_min(par[hf][2 * k + 1])));
        }
        if (vexp != 0) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float sa = param_scale(par[hf][2 * k]) * v_unit, sb = param_scale(par[hf][2 * k + 1]) * v_unit;
            sc[k] = pack_f16(sa, sb);
            mn[k] = pack_f16(fmaf(8.f, sa, param_min(par[hf][2 * k]) * v_unit),
                             fmaf(8.f, sb, param_min(par[hf][2 * k + 1]) * v_unit));
          }
        }
        constexpr int kWords = HD / 64;  // words of codes a lane has per token
        uint32_t v[4][kWords];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          load_words(st + v_at[e & 1] + (hf * 16 + (e & 2) * 4) * C::kCodeRow, v[e]);
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
          // Even channels of two tokens, then odd ones, in one register each.
          const uint32_t e0 = __byte_perm(v[0][j], v[1][j], 0x5410), o0 = __byte_perm(v[0][j], v[1][j], 0x7632);
          const uint32_t e1 = __byte_perm(v[2][j], v[3][j], 0x5410), o1 = __byte_perm(v[2][j], v[3][j], 0x7632);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t af[4] = {fma_f16x2(v_codes(e0, k), sc[0], mn[0]),
                                    fma_f16x2(v_codes(o0, k), sc[0], mn[0]),
                                    fma_f16x2(v_codes(e1, k), sc[1], mn[1]),
                                    fma_f16x2(v_codes(o1, k), sc[1], mn[1])};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_f16(acc[n][4 * j + k], af, pf[hf][n][0], pf[hf][n][1]);
          }
        }
      }
      if (edge) {
        // A token whose values are not numbers, seen by some rows only: those
        // rows, and no others, take it.
#pragma unroll 1
        for (int t = 0; t < kStepTokens; ++t) {
          const uint32_t p = *reinterpret_cast<const uint32_t*>(
              st + 2 * C::kCodes + C::kParams + t * C::kParamRow + (r * (HD / 8)) / GROUP * 4);
          if (tok + t >= hi || !odd_param(p)) continue;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (visible(tok + t, pos[n][e]))
#pragma unroll
                for (int k = 0; k < HD / 16; ++k)
                  acc[n][k][e] = acc[n][k][e + 2] = __int_as_float(0x7fffffff);
        }
      }
    }
    cp_wait<0>();

    // ------------------------------------------------ the four warps' results
    const bool whole = first_tile == 0 && last_tile == w.blk.tiles;
    const long long part_no = 2ll * blockIdx.x + (first_item && first_tile > 0 ? 0 : 1);
    if (tid == 0 && first_tile == 0 && !whole) record = kv4_split_record(w, share);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l_run[n][e] += __shfl_xor_sync(0xffffffffu, l_run[n][e], d);
        if (r == 0) {
          stat[0][warp][8 * n + 2 * q + e] = m_run[n][e] - kShift;
          stat[1][warp][8 * n + 2 * q + e] = l_run[n][e];
        }
      }
    __syncthreads();  // and every warp's stages are free for the exchange below
    constexpr int kQuads = HD / 4;             // float4 of a row
    constexpr int kLaneQuads = HD / 32;        // float4 a lane holds of a row
    constexpr int kTwist = HD == 64 ? 2 : HD == 128 ? 1 : 0;
    float4* ex = reinterpret_cast<float4*>(smem);  // [warp][8 rows][kQuads]
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float f[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 8 * n + 2 * q + e;
        float top = stat[0][0][row];
#pragma unroll
        for (int v = 1; v < kWarps; ++v) top = fmaxf(top, stat[0][v][row]);
        f[e] = m_run[n][e] == -INFINITY ? 0.f : ex2(m_run[n][e] - kShift - top + static_cast<float>(vexp));
      }
      if (n) __syncthreads();  // the previous eight rows have been read
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int k = 0; k < kLaneQuads; ++k) {
          // channels 4 k .. 4 k + 3 of the lane's: products 2 k and 2 k + 1
          const float4 x = make_float4(acc[n][2 * k][e] * f[e], acc[n][2 * k][e + 2] * f[e],
                                       acc[n][2 * k + 1][e] * f[e], acc[n][2 * k + 1][e + 2] * f[e]);
          const int c = r * kLaneQuads + k;
          ex[(warp * 8 + 2 * q + e) * kQuads + (c ^ (r >> kTwist))] = x;
        }
      __syncthreads();
#pragma unroll
      for (int z = tid; z < 8 * kQuads; z += kAttnThreads) {
        const int row8 = z / kQuads, c = z % kQuads, row = 8 * n + row8;
        if (row >= w.blk.rows) continue;
        const int at = row8 * kQuads + (c ^ ((c / kLaneQuads) >> kTwist));
        float4 x = ex[at];
#pragma unroll
        for (int v = 1; v < kWarps; ++v) {
          const float4 y = ex[v * 8 * kQuads + at];
          x.x += y.x;
          x.y += y.y;
          x.z += y.z;
          x.w += y.w;
        }
        float top = stat[0][0][row];
#pragma unroll
        for (int v = 1; v < kWarps; ++v) top = fmaxf(top, stat[0][v][row]);
        float l = 0.f;
#pragma unroll
        for (int v = 0; v < kWarps; ++v) {
          const float g = stat[0][v][row] == -INFINITY ? 0.f : ex2(stat[0][v][row] - top);
          l = fmaf(stat[1][v][row], g, l);
        }
        if (whole) {
          const int gr = w.blk.row0 + row;
          const int t = gr / a.per_kv, head = w.h * a.per_kv + gr - t * a.per_kv;
          const long long o = static_cast<long long>(w.req.start + t) * a.Hq + head;
          const float inv = l == 0.f ? 0.f : 1.f / l;  // a NaN sum stays one
          reinterpret_cast<uint2*>(a.O)[o * kQuads + c] =
              make_uint2(pack_bf16(x.x * inv, x.y * inv), pack_bf16(x.z * inv, x.w * inv));
          if (c == 0) a.L[o] = l == 0.f ? -INFINITY : (top + log2f(l)) * kLn2f;
        } else {
          const long long o = part_no * C::kRows + row;
          reinterpret_cast<float4*>(a.part_o)[o * kQuads + c] = x;
          if (c == 0) a.part_stat[o] = make_float2(top, l);
        }
      }
    }
    first_item = false;
    u = u_next;
    __syncthreads();  // before the walk goes on, and before the next item's copies
    if (u < u_end) {
      if (tid == 0) w.next(a, C::kRows);
      __syncthreads();
    }
  }
  if (tid == 0 && !a.whole_items) a.split[blockIdx.x] = record;
}

// Joins the parts of the items that shares' ends cut: one warp per row.  The
// order of the sums is that of the parts, so the result does not depend on
// which CTA ran when.  Bound by latency: the record, then the parts' statistics
// (a lane each) and as many of their rows as registers hold, side by side.
constexpr int kMergeWarps = 4;
template <int HD, bool kMany>
__global__ void __launch_bounds__(32 * kMergeWarps)
    kv4_merge_kernel(const Kv4AttnArgs a, int block_rows) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 rec = a.split[blockIdx.x];
  const int rows = rec.z & 511, h = rec.z >> 9;
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.y * kMergeWarps + (threadIdx.x >> 5);
  if (row >= rows) return;
  const int first = blockIdx.x;
  const int parts = rec.w - first + 1;
  auto place = [&](int p) {  // part p: this CTA's last item, then its successors' first
    return (p == 0 ? 2ll * first + 1 : 2ll * (first + p)) * block_rows + row;
  };
  // A row is HD / 4 float4: at d = 64 the half-warps take every other part.
  constexpr int kSide = HD == 64 ? 2 : 1, kVec = HD == 256 ? 2 : 1;
  // Rows of parts in flight.  More registers keep blocks, most of which have
  // nothing to do, from starting.  With few rows an item may have dozens of parts:
  // 16 in flight 46.4 us (32 requests of up to 8K tokens) and 96.2 us (three of up
  // to 128K), 8 45.2 and 94.3, 4 45.5 and 96.4.  With many rows it has a few: 16
  // in flight 490 us where 4 take 472.
  constexpr int kFly = kMany || HD == 256 ? 4 : 8;
  const int side = HD == 64 ? lane >> 4 : 0, quad = HD == 64 ? lane & 15 : lane;
  float4 y[kFly][kVec];
  auto load = [&](int p) {  // volatile: issued here
#pragma unroll
    for (int i = 0; i < kFly; ++i) {
      const float4* src =
          reinterpret_cast<const float4*>(a.part_o + place(min(p + kSide * i + side, parts - 1)) * HD) + quad;
#pragma unroll
      for (int k = 0; k < kVec; ++k)
        if (p + kSide * i < parts)
          asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(y[i][k].x), "=f"(y[i][k].y), "=f"(y[i][k].z), "=f"(y[i][k].w)
                       : "l"(src + 32 * k));
        else
          y[i][k] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  float2 st = make_float2(-INFINITY, 0.f);  // of part `lane`
  if (lane < parts) st = a.part_stat[place(lane)];
  load(0);
  float top = st.x;
  for (int p = lane + 32; p < parts; p += 32) top = fmaxf(top, a.part_stat[place(p)].x);
#pragma unroll
  for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  float4 x[kVec];
#pragma unroll
  for (int k = 0; k < kVec; ++k) x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f, f = 0.f;
#pragma unroll 1
  for (int p = 0; p < parts; p += kFly * kSide) {
    if (p > 0) load(p);
    if ((p & 31) == 0) {
      if (p > 0) st = p + lane < parts ? a.part_stat[place(p + lane)] : make_float2(-INFINITY, 0.f);
      f = st.x == -INFINITY ? 0.f : ex2(st.x - top);
      l += st.y * f;
    }
#pragma unroll
    for (int i = 0; i < kFly; ++i) {
      const int q = p + kSide * i + side;
      const float g = __shfl_sync(0xffffffffu, f, q & 31);
#pragma unroll
      for (int k = 0; k < kVec; ++k)
        if (q < parts) {
          x[k].x = fmaf(y[i][k].x, g, x[k].x);
          x[k].y = fmaf(y[i][k].y, g, x[k].y);
          x[k].z = fmaf(y[i][k].z, g, x[k].z);
          x[k].w = fmaf(y[i][k].w, g, x[k].w);
        }
    }
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
  if (HD == 64) {
    x[0].x += __shfl_xor_sync(0xffffffffu, x[0].x, 16);
    x[0].y += __shfl_xor_sync(0xffffffffu, x[0].y, 16);
    x[0].z += __shfl_xor_sync(0xffffffffu, x[0].z, 16);
    x[0].w += __shfl_xor_sync(0xffffffffu, x[0].w, 16);
  }
  const int gr = rec.y + row;
  const int t = gr / a.per_kv, head = h * a.per_kv + gr - t * a.per_kv;
  const long long o = static_cast<long long>(rec.x + t) * a.Hq + head;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint2* dst = reinterpret_cast<uint2*>(a.O) + o * (HD / 4);
#pragma unroll
  for (int k = 0; k < kVec; ++k)
    if (side == 0)
      dst[quad + 32 * k] = make_uint2(pack_bf16(x[k].x * inv, x[k].y * inv), pack_bf16(x[k].z * inv, x[k].w * inv));
  if (lane == 0) a.L[o] = l == 0.f ? -INFINITY : (top + log2f(l)) * kLn2f;
}

template <int HD, bool kMany>
cudaError_t launch_merge(const Kv4AttnArgs& a, int ctas, int block_rows, cudaStream_t stream) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas),
                     static_cast<unsigned>((block_rows + kMergeWarps - 1) / kMergeWarps));
  cfg.blockDim = dim3(32 * kMergeWarps);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv4_merge_kernel<HD, kMany>, a, block_rows);
}

template <int HD, int GROUP, int NT>
cudaError_t launch_attn(const Kv4AttnArgs& a, cudaStream_t stream) {
  using C = AttnCfg<HD, GROUP, NT>;
  static std::atomic<int> resident[64] = {};  // CTAs per SM by device, once known
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int per_sm = dev < 64 ? resident[dev].load(std::memory_order_acquire) : 0;
  if (per_sm == 0) {
    e = cudaFuncSetAttribute(kv4_attn_kernel<HD, GROUP, NT>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kv4_attn_kernel<HD, GROUP, NT>,
                                                      kAttnThreads, C::kSmem);
    if (e != cudaSuccess) return e;
    if (per_sm < 1) return cudaErrorInvalidConfiguration;
    if (dev < 64) resident[dev].store(per_sm, std::memory_order_release);
  }
  const int sms = sm_count();
  if (sms < 1) return cudaErrorInvalidDevice;
  const int ctas = per_sm * sms < kKv4MaxCtas ? per_sm * sms : kKv4MaxCtas;
  Kv4AttnArgs ag = a;
  ag.lead = kLead;
  kv4_attn_kernel<HD, GROUP, NT><<<ctas, kAttnThreads, C::kSmem, stream>>>(ag);
  e = cudaGetLastError();
  if (e != cudaSuccess || a.whole_items) return e;
  return launch_merge<HD, false>(a, ctas, C::kRows, stream);
}

template <int HD, int GROUP>
cudaError_t launch_attn_rows(const Kv4AttnArgs& a, cudaStream_t stream) {
  const int block = kv4_attn_rows(HD, a.max_q * a.per_kv);
  if (block >= 128) {
    int ctas = 0;
    const cudaError_t e = launch_kv4_chunk(HD, GROUP, a, stream, &ctas);
    return e != cudaSuccess || a.whole_items ? e : launch_merge<HD, true>(a, ctas, block, stream);
  }
  if (block == 8) return launch_attn<HD, GROUP, 1>(a, stream);
  if constexpr (HD <= 128)
    if (block == 16) return launch_attn<HD, GROUP, 2>(a, stream);
  if constexpr (HD == 64)
    if (block == 32) return launch_attn<HD, GROUP, 4>(a, stream);
  return cudaErrorInvalidValue;
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

}  // namespace

// The block of rows that serves `rows` best.  More rows in a block cost a warp
// registers (32 at d = 128 and 16 at d = 256 spill, also with the queries in
// shared memory) and products, further blocks read the cache again; the kernel
// for many rows converts every tile once.
// Measured in us for blocks of 8, 16, 32, many, with 16 requests of 8192 tokens
// and with 64 of 768 (8 K/V heads at d = 128):
//   d = 64   32 rows 167 121 108 223 |  93  72  72 140     d = 128   16 rows  76  70 161 |  43  39 101
//            48      243 173 193 224 | 135 102 125 140               24      110 117 162 |  61  67 104
//            64      321 225 195 225 | 176 126 127 141               48      206 167 164 | 110  97 105
//            80      397 276 279 226 | 216 163 178 142               56      238 213 165 | 120 125 105
//   d = 256  32 rows 135 (8), 146 (many) | 78, 84              40 rows 166, 146 | 94, 85
int kv4_attn_rows(int d, int rows) {
  if (rows <= 8) return 8;
  if (d == 64) return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 48 ? 16 : rows <= 64 ? 32 : 256;
  if (d == 128) return rows <= 16 ? 16 : rows <= 24 ? 8 : rows <= 48 ? 16 : 256;
  return rows <= 32 ? 8 : 128;
}

namespace {
size_t part_rows(int d, int rows) {  // rows of all partial results
  const int block = kv4_attn_rows(d, rows);
  return 2 * static_cast<size_t>(block >= 128 ? kKv4MaxChunkCtas : kKv4MaxCtas) * block;
}
}  // namespace

size_t kv4_attn_workspace(int d, int rows) {
  const size_t parts = part_rows(d, rows);
  return align256(kKv4MaxCtas * sizeof(int4)) + align256(parts * sizeof(float2)) +
         align256(parts * d * sizeof(float));
}

// Cutting items of few keys saves less than it costs (the merge, and a second
// change of items): 512 tokens with few rows, and with many 1024, if there are not
// many more items than CTAs, over which uneven ones would not even out (8 K/V
// heads, d = 128: 512 queries 34 -> 25 us; but 64 times 512 414 -> 451 us).
bool kv4_attn_whole(int d, int max_q, int per_kv, int Hkv, int B, int total_q, long long table, int window) {
  const int block = kv4_attn_rows(d, max_q * per_kv);
  long long span = table;  // keys of an item, at most
  if (window >= 0) span = std::min(span, static_cast<long long>(window) + block / per_kv + 2);
  if (block < 128) return span <= 512;
  return span <= 1024 && (static_cast<long long>(total_q) * per_kv / block + B) * Hkv <= 2 * sm_count();
}

cudaError_t launch_kv4_attn(int d, int group, Kv4AttnArgs a, void* workspace, cudaStream_t stream) {
  const size_t parts = part_rows(d, a.max_q * a.per_kv);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.split = reinterpret_cast<int4*>(ws);
  ws += align256(kKv4MaxCtas * sizeof(int4));
  a.part_stat = reinterpret_cast<float2*>(ws);
  ws += align256(parts * sizeof(float2));
  a.part_o = reinterpret_cast<float*>(ws);
  a.whole_items = kv4_attn_whole(d, a.max_q, a.per_kv, a.Hkv, a.B, a.total_q,
                                 static_cast<long long>(a.max_pages) << a.lay.page_shift, a.window);
  const bool g32 = group == 32;
  switch (d) {
    case 64: return g32 ? launch_attn_rows<64, 32>(a, stream) : launch_attn_rows<64, 64>(a, stream);
    case 128: return g32 ? launch_attn_rows<128, 32>(a, stream) : launch_attn_rows<128, 64>(a, stream);
    case 256: return g32 ? launch_attn_rows<256, 32>(a, stream) : launch_attn_rows<256, 64>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fa
