// kv4_attn.cu -- attention over the paged 4-bit cache for few query rows.
//
// Up to 32 rows (queries x query heads of one K/V head) share each read of the
// cache; one read of the keys and values is all the memory traffic there is, so
// the kernel is built around it: a warp walks the cache on its own, 16 tokens at
// a time, with its copies (cp.async) several steps ahead and no barrier with any
// other warp until its item ends.  Per step of 16 tokens and a K/V head:
//
//   S^T = K Q^T   mma m16n8k16, A = 16 tokens x 16 channels of codes, B = Q^T
//   p   = 2^(S scale log2e - m), running maximum m and sums in fp32
//   O^T += V^T P^T   A = 16 channels x 16 tokens of values, B = P^T
//
// Tokens (then channels) are the 16 rows of the product and query rows its 8
// columns, so one to eight rows cost one product.
//
// Codes become bf16 without a conversion: 0x4300 | c is 128 + c.  For K that is
// all: per group of channels sum q (m + s c) = s sum q (128 + c) + (m - 128 s)
// sum q, two FMAs per score on exact products.  128 exceeds the codes by a
// factor of 8 to 128, which costs 7 of fp32's 24 bits at most.  For V, 128 is
// subtracted (exact) and one bf16 FMA gives the value rounded to bf16, as if V
// had been a bf16 tensor; P is rounded to bf16 as in the bf16 forward.  O is
// divided by the sum of the rounded weights, L uses the unrounded ones.
//
// Which token is which row of the product is free as long as both products
// agree; kTokenOf and the swizzle of the 16-byte chunks (chunk_of) are chosen so
// that a warp's reads of its staged codes touch every bank once.
#include <cuda_bf16.h>

#include <atomic>

#include "kernels.h"
#include "kv4.h"
#include "kv4_sched.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kWarps = 4;
constexpr int kAttnThreads = 32 * kWarps;
constexpr int kStepTokens = 16;
static_assert(kWarps * kStepTokens == kKv4Tile, "a tile is one step of every warp");
constexpr float kGrow = 8.f;  // log2 units: m moves only when the maximum passes it by more
constexpr float kLn2f = 0.693147180559945309f;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
// Nibbles i and i + 4 of w as bf16 values 128 + code.
__device__ __forceinline__ uint32_t codes2(uint32_t w, int i) {
  return ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
}

// Token (of a step's 16) that is row r of the product.
__device__ __forceinline__ int token_of(int r) { return (r & 8) | ((r & 1) << 2) | ((r >> 1) & 3); }

template <int HD>
__device__ __forceinline__ int chunk_of(int tok, int chunk) {  // 16-byte chunk of a staged row
  if (HD == 64) return chunk ^ ((tok >> 2) & 1);
  if (HD == 128) return chunk ^ ((tok & 2) | ((tok >> 2) & 1));
  return chunk ^ (((tok << 1) | ((tok >> 2) & 1)) & 7);
}

template <int HD, int GROUP, int NT>
struct AttnCfg {
  static constexpr int kGroups = HD / GROUP;
  static constexpr int kCodeRow = HD / 2, kParamRow = 4 * kGroups;
  static constexpr int kCodes = kStepTokens * kCodeRow, kParams = kStepTokens * kParamRow;
  static constexpr int kStage = 2 * (kCodes + kParams);  // bytes: K codes, V codes, K, V params
  static constexpr int kStages = HD == 64 ? 6 : 4;
  static constexpr int kStageBytes = kWarps * kStages * kStage;
  static constexpr int kMergeBytes = kWarps * 8 * HD * 4;  // 8 rows of every warp's O
  static constexpr int kSmem = kStageBytes > kMergeBytes ? kStageBytes : kMergeBytes;
  static constexpr int kRows = 8 * NT;
  // Resident CTAs per SM the registers are bounded for.
  static constexpr int kMinCtas = HD == 256 ? 2 : NT == 4 ? 2 : NT == 2 ? 3 : 4;
};

template <int HD, int GROUP, int NT>
__global__ void __launch_bounds__(kAttnThreads, AttnCfg<HD, GROUP, NT>::kMinCtas)
    kv4_attn_kernel(const Kv4AttnArgs a) {
  using C = AttnCfg<HD, GROUP, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long scratch[kWarps + 2];
  __shared__ float stat[3][kWarps][C::kRows];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = lane >> 2, q = lane & 3;  // row / column pair of the product's fragments

  const Kv4Share share = kv4_share<kAttnThreads>(a, C::kRows, 2, scratch);
  long long u = share.per * blockIdx.x;
  const long long u_end = min(share.total, u + share.per);
  if (tid == 0 && u >= share.total) a.split[blockIdx.x] = make_int4(0, 0, 0, 0);
  if (u >= share.total) return;
  bool first_item = true;
  Kv4Walk w;
  w.seek(a, share, u, C::kRows);
  const uint8_t* stage0 = smem + warp * C::kStages * C::kStage;
  const uint32_t stage0_u32 = smem_u32(stage0);
  int4 record = make_int4(0, 0, 0, 0);

  for (; u < u_end; w.next(a, C::kRows)) {
    const int ta = static_cast<int>(u - w.item);
    const int tb = static_cast<int>(min(static_cast<long long>(w.blk.tiles), u_end - w.item));
    const int steps = tb - ta;
    const int tok0 = (w.blk.tile_lo + ta) * kKv4Tile + warp * kStepTokens;

    // ------------------------------------------------ copies, S - 1 steps ahead
    int page = -1, page_next = -1;  // lane l: page of step 32 k + l
    uint32_t live = 0;              // bit i % 32: step i has something to do
    auto fetch_page = [&](int i) -> int {
      const int tok = tok0 + (i + lane) * kKv4Tile;
      if (i + lane >= steps || tok >= w.blk.hi) return -1;
      return __ldg(a.table + static_cast<long long>(w.b) * a.max_pages + (tok >> a.lay.page_shift));
    };
    page_next = fetch_page(0);
    auto issue = [&](int i) {
      if (i < steps) {
        if ((i & 31) == 0) {
          page = page_next;
          page_next = fetch_page(i + 32);
        }
        const int pg = __shfl_sync(0xffffffffu, page, i & 31);
        const int tok = tok0 + i * kKv4Tile;
        bool ok = tok < w.blk.hi;
        if (ok && (pg < 0 || pg >= a.num_pages)) {
          if (lane == 0) atomicCAS(a.input_err, 0, 1);
          ok = false;
        }
        live = (live & ~(1u << (i & 31))) | (ok ? 1u << (i & 31) : 0u);
        if (ok) {
          const int off = tok & ((1 << a.lay.page_shift) - 1);
          const uint8_t* rec =
              a.cache + (static_cast<long long>(pg) * a.Hkv + w.h) * a.lay.record;
          const uint8_t* kc = rec + off * C::kCodeRow;
          const uint8_t* vc = kc + a.lay.v_codes;
          const uint32_t dst = stage0_u32 + (i % C::kStages) * C::kStage;
          constexpr int kChunks = HD / 32;  // 16-byte chunks of a row of codes
#pragma unroll
          for (int k = lane; k < C::kCodes / 16; k += 32) {
            const int t = k / kChunks, c = k % kChunks;
            const uint32_t at = dst + (t * kChunks + chunk_of<HD>(t & 7, c)) * 16;
            cp_async16(at, kc + k * 16);
            cp_async16(at + C::kCodes, vc + k * 16);
          }
          constexpr int kP = C::kParams / 16;
          const uint8_t* kp = rec + a.lay.k_params + off * C::kParamRow;
          const uint8_t* vp = rec + a.lay.v_params + off * C::kParamRow;
#pragma unroll
          for (int k = lane; k < 2 * kP; k += 32)
            cp_async16(dst + 2 * C::kCodes + k * 16, (k < kP ? kp + k * 16 : vp + (k - kP) * 16));
        }
      }
      cp_commit();
    };
#pragma unroll
    for (int i = 0; i < C::kStages - 1; ++i) issue(i);

    // ------------------------------------------------ this block's queries
    uint32_t qf[NT][HD / 32][4];       // B fragments of Q^T
    float qsum[NT][C::kGroups][2];     // sums of Q over a group, rows 2 q, 2 q + 1
    int pos[NT][2];                    // position of rows 2 q, 2 q + 1 (-1: no such row)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int row = 8 * n + r;
      const bool have = row < w.blk.rows;
      const int gr = w.blk.row0 + row;
      const int t = gr / a.per_kv, head = w.h * a.per_kv + gr - t * a.per_kv;
      const uint16_t* src = a.Q + static_cast<long long>(w.req.start + t) * a.q_ts +
                            static_cast<long long>(head) * a.q_hs + 8 * q;
      float part[C::kGroups];
#pragma unroll
      for (int g = 0; g < C::kGroups; ++g) part[g] = 0.f;
#pragma unroll
      for (int c = 0; c < HD / 32; ++c) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (have) x = __ldg(reinterpret_cast<const uint4*>(src + 32 * c));
        qf[n][c][0] = x.x;
        qf[n][c][1] = x.y;
        qf[n][c][2] = x.z;
        qf[n][c][3] = x.w;
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
    float m_run[NT][2], l_run[NT][2], lh_run[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < HD / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][i][e] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m_run[n][e] = -INFINITY;
        l_run[n][e] = 0.f;
        lh_run[n][e] = 0.f;
      }
    }

    // ------------------------------------------------ the walk over the tokens
#pragma unroll 1
    for (int i = 0; i < steps; ++i) {
      cp_wait<C::kStages - 2>();
      __syncwarp();  // every lane's copies have landed; step i - 1 has been read
      issue(i + C::kStages - 1);
      if (!((live >> (i & 31)) & 1u)) continue;
      const int tok = tok0 + i * kKv4Tile;
      const uint8_t* st = stage0 + (i % C::kStages) * C::kStage;
      const bool edge = tok + kStepTokens > w.blk.all_hi || tok < w.blk.all_lo;

      // S^T: rows r and r + 8 are tokens t0 and t0 + 8
      const int t0 = token_of(r);
      float s[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
      {
        const uint32_t* p0 = reinterpret_cast<const uint32_t*>(st + 2 * C::kCodes) + t0 * C::kGroups;
        const uint32_t* p1 = p0 + 8 * C::kGroups;
#pragma unroll
        for (int g = 0; g < C::kGroups; ++g) {
          float d[NT][4];
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) d[n][e] = 0.f;
#pragma unroll
          for (int cc = 0; cc < GROUP / 32; ++cc) {
            const int c = g * (GROUP / 32) + cc;
            const int at = (t0 * (HD / 32) + chunk_of<HD>(t0, c)) * 16 + q * 4;
            const uint32_t w0 = *reinterpret_cast<const uint32_t*>(st + at);
            const uint32_t w1 = *reinterpret_cast<const uint32_t*>(st + at + 8 * C::kCodeRow);
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
              const uint32_t af[4] = {codes2(w0, 2 * ks), codes2(w1, 2 * ks),
                                      codes2(w0, 2 * ks + 1), codes2(w1, 2 * ks + 1)};
#pragma unroll
              for (int n = 0; n < NT; ++n) mma16816(d[n], af, qf[n][c][2 * ks], qf[n][c][2 * ks + 1]);
            }
          }
          const uint32_t k0 = p0[g], k1 = p1[g];
          const float s0 = __uint_as_float(k0 << 16), s1 = __uint_as_float(k1 << 16);
          const float b0 = fmaf(-128.f, s0, __uint_as_float(k0 & 0xffff0000u));
          const float b1 = fmaf(-128.f, s1, __uint_as_float(k1 & 0xffff0000u));
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            s[n][0] = fmaf(d[n][0], s0, fmaf(b0, qsum[n][g][0], s[n][0]));
            s[n][1] = fmaf(d[n][1], s0, fmaf(b0, qsum[n][g][1], s[n][1]));
            s[n][2] = fmaf(d[n][2], s1, fmaf(b1, qsum[n][g][0], s[n][2]));
            s[n][3] = fmaf(d[n][3], s1, fmaf(b1, qsum[n][g][1], s[n][3]));
          }
        }
      }
      const bool upto = a.causal || a.window >= 0;
      auto visible = [&](int token, int p) {
        bool v = token < w.req.kv;
        if (upto) v = v && token <= p;
        if (a.window >= 0) v = v && token >= p - a.window;
        return v;
      };
      if (edge) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int token = tok + t0 + (e & 2) * 4;
            s[n][e] = visible(token, pos[n][e & 1]) ? s[n][e] : -INFINITY;
          }
      }

      // running maximum: moved only when some score passes it by kGrow
      bool grow = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          grow = grow || fmaxf(s[n][e], s[n][e + 2]) * a.scale_log2 > m_run[n][e] + kGrow;
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float alpha[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = fmaxf(s[n][e], s[n][e + 2]) * a.scale_log2;
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            const bool up = top > m_run[n][e] + kGrow;
            alpha[e] = up ? ex2(m_run[n][e] - top) : 1.f;
            m_run[n][e] = up ? top : m_run[n][e];
            l_run[n][e] *= alpha[e];
            lh_run[n][e] *= alpha[e];
          }
#pragma unroll
          for (int k = 0; k < HD / 16; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[n][k][e] *= alpha[e & 1];
        }
      }

      // P^T as B fragments
      uint32_t pf[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float m0 = m_run[n][0] == -INFINITY ? 0.f : m_run[n][0];
        const float m1 = m_run[n][1] == -INFINITY ? 0.f : m_run[n][1];
        const float p0 = ex2(fmaf(s[n][0], a.scale_log2, -m0));
        const float p1 = ex2(fmaf(s[n][1], a.scale_log2, -m1));
        const float p2 = ex2(fmaf(s[n][2], a.scale_log2, -m0));
        const float p3 = ex2(fmaf(s[n][3], a.scale_log2, -m1));
        const uint32_t lo = pack_bf16(p0, p1), hi = pack_bf16(p2, p3);
        l_run[n][0] += p0 + p2;
        l_run[n][1] += p1 + p3;
        lh_run[n][0] += __uint_as_float(lo << 16) + __uint_as_float(hi << 16);
        lh_run[n][1] += __uint_as_float(lo & 0xffff0000u) + __uint_as_float(hi & 0xffff0000u);
        pf[n][0] = transpose8x8(lo);
        pf[n][1] = transpose8x8(hi);
      }

      // O^T += V^T P^T: this lane's rows are the HD / 8 channels from r HD / 8 on,
      // its columns tokens ta, tb (first half of k) and ta + 8, tb + 8
      {
        const int ta0 = token_of(2 * q), ta1 = token_of(2 * q + 1);
        const uint32_t* vp = reinterpret_cast<const uint32_t*>(st + 2 * C::kCodes + C::kParams) +
                             (r * (HD / 8)) / GROUP;
        uint32_t par[4] = {vp[ta0 * C::kGroups], vp[ta1 * C::kGroups], vp[(ta0 + 8) * C::kGroups],
                           vp[(ta1 + 8) * C::kGroups]};
        if (edge) {
          // Rows behind the request's last token may hold anything: their
          // weights are 0, and their values have to be finite for that to count.
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int token = tok + ((e & 1) ? ta1 : ta0) + (e & 2) * 4;
            const bool odd = (par[e] & 0x7f80u) == 0x7f80u || (par[e] & 0x7f800000u) == 0x7f800000u;
            if (token >= w.req.kv || odd) par[e] = 0;
          }
        }
        const uint32_t sc0 = __byte_perm(par[0], par[1], 0x5410), mn0 = __byte_perm(par[0], par[1], 0x7632);
        const uint32_t sc1 = __byte_perm(par[2], par[3], 0x5410), mn1 = __byte_perm(par[2], par[3], 0x7632);
        constexpr int kWords = HD / 64;  // words of codes a lane has per token
        uint32_t v[4][kWords];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = ((e & 1) ? ta1 : ta0) + (e & 2) * 4;
          const int byte = r * (HD / 16);
          const uint8_t* src = st + C::kCodes +
                               (t * (HD / 32) + chunk_of<HD>(t & 7, byte / 16)) * 16 + byte % 16;
          if constexpr (kWords == 1) {
            v[e][0] = *reinterpret_cast<const uint32_t*>(src);
          } else if constexpr (kWords == 2) {
            const uint2 x = *reinterpret_cast<const uint2*>(src);
            v[e][0] = x.x;
            v[e][1] = x.y;
          } else {
            const uint4 x = *reinterpret_cast<const uint4*>(src);
            v[e][0] = x.x;
            v[e][1] = x.y;
            v[e][2] = x.z;
            v[e][3] = x.w;
          }
        }
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
          // Even channels of two tokens, then odd ones, in one register each.
          const uint32_t e0 = __byte_perm(v[0][j], v[1][j], 0x5410), o0 = __byte_perm(v[0][j], v[1][j], 0x7632);
          const uint32_t e1 = __byte_perm(v[2][j], v[3][j], 0x5410), o1 = __byte_perm(v[2][j], v[3][j], 0x7632);
          constexpr uint32_t kMinus128 = 0xc300c300u;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t af[4] = {fma_bf16x2(add_bf16x2(codes2(e0, k), kMinus128), sc0, mn0),
                                    fma_bf16x2(add_bf16x2(codes2(o0, k), kMinus128), sc0, mn0),
                                    fma_bf16x2(add_bf16x2(codes2(e1, k), kMinus128), sc1, mn1),
                                    fma_bf16x2(add_bf16x2(codes2(o1, k), kMinus128), sc1, mn1)};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816(acc[n][4 * j + k], af, pf[n][0], pf[n][1]);
          }
        }
        if (edge) {
          // A token whose values are not numbers, seen by some rows only: those
          // rows, and no others, take it.
#pragma unroll 1
          for (int t = 0; t < kStepTokens; ++t) {
            const uint32_t p = vp[t * C::kGroups];
            const bool odd = (p & 0x7f80u) == 0x7f80u || (p & 0x7f800000u) == 0x7f800000u;
            if (!odd || tok + t >= w.req.kv) continue;
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
    }
    cp_wait<0>();

    // ------------------------------------------------ the four warps' results
    const bool whole = ta == 0 && tb == w.blk.tiles;
    const long long part_no = 2ll * blockIdx.x + (first_item && ta > 0 ? 0 : 1);
    if (ta == 0 && !whole) record = kv4_split_record(w, share);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
          l_run[n][e] += __shfl_xor_sync(0xffffffffu, l_run[n][e], d);
          lh_run[n][e] += __shfl_xor_sync(0xffffffffu, lh_run[n][e], d);
        }
        if (r == 0) {
          stat[0][warp][8 * n + 2 * q + e] = m_run[n][e];
          stat[1][warp][8 * n + 2 * q + e] = l_run[n][e];
          stat[2][warp][8 * n + 2 * q + e] = lh_run[n][e];
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
        f[e] = m_run[n][e] == -INFINITY ? 0.f : ex2(m_run[n][e] - top);
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
        float l = 0.f, lh = 0.f;
#pragma unroll
        for (int v = 0; v < kWarps; ++v) {
          const float g = stat[0][v][row] == -INFINITY ? 0.f : ex2(stat[0][v][row] - top);
          l = fmaf(stat[1][v][row], g, l);
          lh = fmaf(stat[2][v][row], g, lh);
        }
        if (whole) {
          const int gr = w.blk.row0 + row;
          const int t = gr / a.per_kv, head = w.h * a.per_kv + gr - t * a.per_kv;
          const long long o = static_cast<long long>(w.req.start + t) * a.Hq + head;
          const float inv = lh == 0.f ? 0.f : 1.f / lh;  // a NaN sum stays one
          reinterpret_cast<uint2*>(a.O)[o * kQuads + c] =
              make_uint2(pack_bf16(x.x * inv, x.y * inv), pack_bf16(x.z * inv, x.w * inv));
          if (c == 0) a.L[o] = l == 0.f ? -INFINITY : (top + log2f(l)) * kLn2f;
        } else {
          const long long o = part_no * C::kRows + row;
          reinterpret_cast<float4*>(a.part_o)[o * kQuads + c] = x;
          if (c == 0) a.part_stat[o] = make_float4(top, l, lh, 0.f);
        }
      }
    }
    __syncthreads();  // before the next item's copies
    first_item = false;
    u = w.item + tb;
  }
  if (tid == 0) a.split[blockIdx.x] = record;
}

// Joins the parts of the items that shares' ends cut: one warp per row.  The
// order of the sums is that of the parts, so the result does not depend on
// which CTA ran when.
constexpr int kMergeWarps = 4;
template <int HD>
__global__ void __launch_bounds__(32 * kMergeWarps)
    kv4_merge_kernel(const Kv4AttnArgs a, int block_rows) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 rec = a.split[blockIdx.x];
  const int rows = rec.z & 255, h = rec.z >> 8;
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.y * kMergeWarps + (threadIdx.x >> 5);
  if (row >= rows) return;
  const int first = blockIdx.x;
  const int parts = rec.w - first + 1;
  auto place = [&](int p) {  // part p: this CTA's last item, then its successors' first
    return (p == 0 ? 2ll * first + 1 : 2ll * (first + p)) * block_rows + row;
  };
  float top = -INFINITY;
  for (int p = lane; p < parts; p += 32) top = fmaxf(top, a.part_stat[place(p)].x);
#pragma unroll
  for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  constexpr int kVec = HD / 64;  // float2 a lane
  float2 x[kVec];
#pragma unroll
  for (int k = 0; k < kVec; ++k) x[k] = make_float2(0.f, 0.f);
  float l = 0.f, lh = 0.f;
#pragma unroll 4
  for (int p = 0; p < parts; ++p) {
    const float4 st = a.part_stat[place(p)];
    const float f = st.x == -INFINITY ? (st.y == st.y ? 0.f : st.y) : ex2(st.x - top);
    l = fmaf(st.y, f, l);
    lh = fmaf(st.z, f, lh);
    const float2* src = reinterpret_cast<const float2*>(a.part_o + place(p) * HD);
#pragma unroll
    for (int k = 0; k < kVec; ++k) {
      const float2 y = src[lane + 32 * k];
      x[k].x = fmaf(y.x, f, x[k].x);
      x[k].y = fmaf(y.y, f, x[k].y);
    }
  }
  const int gr = rec.y + row;
  const int t = gr / a.per_kv, head = h * a.per_kv + gr - t * a.per_kv;
  const long long o = static_cast<long long>(rec.x + t) * a.Hq + head;
  const float inv = lh == 0.f ? 0.f : 1.f / lh;
  uint32_t* dst = reinterpret_cast<uint32_t*>(a.O) + o * (HD / 2);
#pragma unroll
  for (int k = 0; k < kVec; ++k) dst[lane + 32 * k] = pack_bf16(x[k].x * inv, x[k].y * inv);
  if (lane == 0) a.L[o] = l == 0.f ? -INFINITY : (top + log2f(l)) * kLn2f;
}

template <int HD>
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
  return cudaLaunchKernelEx(&cfg, kv4_merge_kernel<HD>, a, block_rows);
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
  kv4_attn_kernel<HD, GROUP, NT><<<ctas, kAttnThreads, C::kSmem, stream>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_merge<HD>(a, ctas, C::kRows, stream);
}

template <int HD, int GROUP>
cudaError_t launch_attn_rows(const Kv4AttnArgs& a, cudaStream_t stream) {
  switch (kv4_attn_rows(HD, a.max_q * a.per_kv)) {
    case 8: return launch_attn<HD, GROUP, 1>(a, stream);
    case 16: return launch_attn<HD, GROUP, 2>(a, stream);
    default:
      if constexpr (HD == 256)
        return cudaErrorInvalidValue;
      else
        return launch_attn<HD, GROUP, 4>(a, stream);
  }
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

}  // namespace

int kv4_attn_rows(int d, int rows) {
  if (rows <= 8) return 8;
  if (rows <= 16 || d == 256) return 16;  // d = 256: 32 rows of O would not fit the registers
  return 32;
}

size_t kv4_attn_workspace(int d, int rows) {
  const size_t parts = 2 * static_cast<size_t>(kKv4MaxCtas) * kv4_attn_rows(d, rows);
  return align256(kKv4MaxCtas * sizeof(int4)) + align256(parts * sizeof(float4)) +
         align256(parts * d * sizeof(float));
}

cudaError_t launch_kv4_attn(int d, int group, Kv4AttnArgs a, void* workspace, cudaStream_t stream) {
  const size_t parts = 2 * static_cast<size_t>(kKv4MaxCtas) * kv4_attn_rows(d, a.max_q * a.per_kv);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.split = reinterpret_cast<int4*>(ws);
  ws += align256(kKv4MaxCtas * sizeof(int4));
  a.part_stat = reinterpret_cast<float4*>(ws);
  ws += align256(parts * sizeof(float4));
  a.part_o = reinterpret_cast<float*>(ws);
  const bool g32 = group == 32;
  switch (d) {
    case 64: return g32 ? launch_attn_rows<64, 32>(a, stream) : launch_attn_rows<64, 64>(a, stream);
    case 128: return g32 ? launch_attn_rows<128, 32>(a, stream) : launch_attn_rows<128, 64>(a, stream);
    case 256: return g32 ? launch_attn_rows<256, 32>(a, stream) : launch_attn_rows<256, 64>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fa
