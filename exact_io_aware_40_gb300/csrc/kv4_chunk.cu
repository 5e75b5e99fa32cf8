// kv4_chunk.cu -- attention over the paged 4-bit cache for many query rows: a
// chunk of a prompt, or drafted tokens of many query heads.
//
// One CTA per SM takes blocks of 256 query rows (128 at d = 256; queries x query
// heads of one K/V head) and walks its share of the tiles of 64 tokens
// (kv4_sched.cuh).  Both products run on the tensor cores out of tensor memory as
// in the bf16 forward (S double buffered, P over S as the A operand of P V, O
// resident); what differs is where K and V come from:
//   - two converters, four warps each for K and for V, copy a tile's codes and
//     params some tiles ahead (cp.async; a thread's own 16 bytes, so nobody waits
//     for anybody) and write them as fp16 tiles in the 128-byte-swizzled layout
//     the products take;
//   - a warpgroup for each 128 rows (thread = row = TMEM lane) loads Q, does the
//     softmax and writes O; the two share every converted tile;
//   - one warp for each 128 rows issues the products, by one elected lane.
// Two issuers and two converters because one of either was what a tile waited
// for: a thread's chain of dependent instructions, not the pipes (one of each:
// 3890 clocks a tile, of which the issuer worked 3040 and the converter 2480).
//
// K.  (code - 8) * scale has at most 8 + 3 significant bits and so is exact in
// fp16, as Q is (8 bits) after a scaling of each row by a power of two.  The
// rest of a key, minimum + 8 scale of each group, meets the sum of Q over the
// group; both are split into two fp16 (22 bits) and their three leading products
// are slots of one more k-step (two if there are eight groups): minima (h, l) by
// group, then h again, against sums (h, h), then l.  So scores have
// the accuracy of fp32 sums without a second pass over K.
// V.  minimum + scale * code rounded to fp16, P in fp16: see kv4_attn.cu.
// fp16's range: the K and V of a tile are taken in units of a power of two that
// fits the tile's largest param.  K's unit multiplies the tile's scores; V's goes
// into the exponent of P, whose reference then includes the largest unit so far.
//
// Measured (d = 128, 2 x 1024 queries of 32 heads over 8K to 16K keys): 472 us,
// 1026 TFLOP/s, 0.52 of the measured bf16 peak; a tile takes about 2300 clocks of
// which the products need 1100.  Bound: the rows' chain from S to P among the other
// roles' instructions (2270 of 2880 clocks a tile in a build that counted; about
// 17 instructions for eight codes, 3.5 for a score, 64 % of the issue slots).  A
// third stage of K or V is slower (526 to 549 us where two took 515), and so are
// weights taken before the maximum is known (545 for 515).  At d = 256 one block of
// 128 rows is all that shared and tensor memory hold, so a converted tile serves
// half the rows: 560 TFLOP/s.
#include <cuda_fp16.h>

#include <atomic>

#include "kernels.h"
#include "kv4.h"
#include "kv4_sched.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kRows = 128;  // rows of a warpgroup
constexpr int kTile = 64;
// Tiles that a change of items costs.  Measured with 2, 4, 6, 8, 10: 8192 queries
// without a past 812, 656, 584, 588, 592 us; 64 requests of 512 445, 427, 414,
// 416, 420 us (8 K/V heads, 32 query heads, d = 128).
constexpr int kLead = 6;
constexpr float kGrow = 4.f;
constexpr float kShift = 10.f;
constexpr float kLn2f = 0.693147180559945309f;
constexpr int kUnits = 8;  // ring of tile units: K's converter is at most five tiles ahead of the rows

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t add_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t keep, uint32_t set) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(x), "r"(keep), "r"(set));
  return r;
}
// Channels 2 i and 2 i + 1 of a word as fp16 values code - 8.
__device__ __forceinline__ uint32_t codes_m8(uint32_t w, int i) {
  const uint32_t x = i < 2 ? w : w >> 8;
  if ((i & 1) == 0) return add_f16x2(and_or(x, 0x000f000fu, 0x64006400u), 0xe408e408u);  // -1032
  return fma_f16x2(and_or(x, 0x00f000f0u, 0x64006400u), 0x2c002c00u, 0xd480d480u);  // / 16 - 72
}
__device__ __forceinline__ bool odd_param(uint32_t p) {
  return (p & 0x7f80u) == 0x7f80u || (p & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ float param_scale(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float param_min(uint32_t p) { return __uint_as_float(p & 0xffff0000u); }
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// 2^e, -126 <= e <= 127
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// Instruction descriptor of kind::f16 with fp16 A and B (format 0), fp32 D.
__host__ __device__ constexpr uint32_t idesc_f16(uint32_t M, uint32_t N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
// Shared-memory descriptor without swizzle, K-major: core matrices of 8 rows x
// 16 bytes, `lbo` bytes apart along K and `sbo` bytes apart along the rows.
__device__ __forceinline__ uint64_t sdesc_plain(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46);
}

// One lane of a converged warp, always the same one.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <int HD, int GROUP>
struct Cfg {
  static constexpr int kGroups = HD / GROUP;
  static constexpr int kCodeRow = HD / 2, kParamRow = 4 * kGroups;
  static constexpr int kAtoms = HD / 64;
  static constexpr int kBlocks = HD == 256 ? 1 : 2;      // warpgroups of rows
  static constexpr int kBlockRows = kBlocks * kRows;
  static constexpr int kThreads = 128 * (kBlocks + 3);   // + converters of K and V, products
  static constexpr int kQAtom = kRows * 128, kQTile = kAtoms * kQAtom;
  static constexpr int kAtom = kTile * 128, kTileBytes = kAtoms * kAtom;  // K or V tile
  static constexpr int kKSt = HD == 256 ? 1 : 2, kVSt = 2;
  // Extra slots: three for each group, in k-steps of 16.
  static constexpr int kExSteps = (3 * kGroups + 15) / 16;
  static constexpr int kExRow8 = kExSteps * 256;  // bytes of eight rows
  static constexpr int kQEx = kRows / 8 * kExRow8, kKEx = kTile / 8 * kExRow8;
  // Converter: threads a token's row of codes, tokens a pass, passes a tile;
  // tiles of codes in flight or in use, each thread's own 16 + 4 + 4 bytes a
  // pass (codes, params, K's converter: V's params too).
  static constexpr int kTpr = HD / 32, kPassTokens = 128 / kTpr, kPasses = kTile / kPassTokens;
  static constexpr int kRing = HD == 256 ? 2 : 4;
  static constexpr int kRingPass = 128 * 24, kRingTile = kPasses * kRingPass;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + kBlocks * kQTile;
  static constexpr int kOffV = kOffK + kKSt * kTileBytes;
  static constexpr int kOffQEx = kOffV + kVSt * kTileBytes;
  static constexpr int kOffKEx = kOffQEx + kBlocks * kQEx;
  static constexpr int kOffRing = kOffKEx + kKSt * kKEx;
  static constexpr int kOffBar = kOffRing + 2 * kRing * kRingTile;
  // k_full[2], k_empty[2], v_full[2], v_empty[2], then for each block of rows
  // q_full, s_full[2], p_full[2], o_done, drain
  static constexpr int kNumBar = 8 + 7 * kBlocks;
  static constexpr int kOffMisc = kOffBar + kNumBar * 8;
  static constexpr int kSmem = kOffMisc + 16 + 1024;
  static_assert(kSmem <= 230000, "shared memory budget");
  // TMEM: S buffers of a block side by side, then every block's O.
  static constexpr uint32_t kColO = 128 * kBlocks;
  static constexpr uint32_t kTmemCols = 512;
  static_assert(kColO + kBlocks * HD <= kTmemCols, "tensor memory budget");
  // Registers a thread of the warpgroups (rows, each converter, products) out
  // of the launch's.  Measured: d = 128, 2 x 1024 queries, 128 / 80 / 64 487 us,
  // 136 / 72 / 64 474, 136 / 80 / 48 473, 144 / 80 / 32 479, 152 / 64 / 48 486;
  // d = 256, 4096 queries, 208 / 104 / 96 1745 us, 232 / 112 / 56 1541,
  // 224 / 120 / 48 1475, 232 / 120 / 40 1552 (the issuing warp's code is the
  // better the less room it is given, down to 48).
  static constexpr int kLaunchRegs = kBlocks == 2 ? 96 : 128;
  static constexpr int kRowRegs = kBlocks == 2 ? 136 : 224;
  static constexpr int kConvRegs = kBlocks == 2 ? 80 : 120;
  static constexpr int kMmaRegs = 48;
  static_assert(kBlocks * kRowRegs + 2 * kConvRegs + kMmaRegs <= (kBlocks + 3) * kLaunchRegs, "register split");
};

__device__ __forceinline__ bool bar_and_128(int id, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(pred ? 1u : 0u), "r"(id)
      : "memory");
  return r != 0;
}

// The tiles of a CTA's share, item by item.
template <int kBlockRows>
struct Tiles {
  Kv4Walk<kTile> w;
  long long u, u_next, u_end;
  int first, last;  // the item's tiles in this share

  __device__ __forceinline__ void begin(const Kv4AttnArgs& a, const Kv4Share& s) {
    u = s.per * blockIdx.x;
    u_end = min(s.total, u + s.per);
    w.seek(a, s, u, kBlockRows);
    open(a);
  }
  __device__ __forceinline__ void open(const Kv4AttnArgs& a) {
    u_next = kv4_part(a, w, u, u_end, &first, &last);
  }
  // To the next item with tiles in this share; false if there is none.
  __device__ __forceinline__ bool next_item(const Kv4AttnArgs& a) {
    u = u_next;
    if (u >= u_end) return false;
    w.next(a, kBlockRows);
    open(a);
    return first < last;
  }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool have) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(have ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool have) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(have ? 4 : 0)
               : "memory");
}

// What K's converter leaves for the rows, by tile (a ring of kUnits); it comes
// to them with the scores.  (V's unit and marks are needed that early, too, so
// K's converter reads V's params for them; V's converter finds the same unit.)
// A unit is kept through an item as long as the params fit it.
struct Units {
  float k_unit[kUnits];          // 2^kexp
  int v_exp[kUnits];
  int any_odd[kUnits];
  uint8_t odd_v[kUnits][kTile];  // groups of a token's V that are not numbers
  uint32_t top_param[3][4];      // [K's, V's by K's converter, V's][warp]
  int meta[2][8];                // of a converter's tiles: bit 0 edge, bit 1 item's first
};

// The converter of K (kSide 0) or V (1): four warps.  `walk` is the warp's own,
// in shared memory: it is touched once an item and would only take registers.
template <int HD, int GROUP, int kSide>
__device__ __forceinline__ void convert(const Kv4AttnArgs& a, Tiles<Cfg<HD, GROUP>::kBlockRows>& walk,
                                        uint8_t* smem, uint32_t sb, uint32_t bar_full,
                                        uint32_t bar_empty, Units& un, const Abort& ab) {
  using C = Cfg<HD, GROUP>;
  constexpr int kSt = kSide ? C::kVSt : C::kKSt;
  constexpr int kBar = C::kBlocks + 1 + kSide;  // named barrier of these four warps
  const int ct = threadIdx.x & 127, cw = ct >> 5, lane = ct & 31;
  // Token of a pass and 32-channel block: eight lanes side by side write to
  // different chunks of the swizzled tile (eight tokens, at d = 256 four tokens
  // of two blocks).
  constexpr int kTok = HD == 256 ? 4 : 8;  // tokens of those lanes
  const int part = lane / kTok % C::kTpr;
  const int ptok = cw * (32 / C::kTpr) + lane / (kTok * C::kTpr) * kTok + lane % kTok;
  const int group = part * 32 / GROUP;
  __syncwarp();
  const long long page_bytes = static_cast<long long>(a.Hkv) * a.lay.record;
  const int shift = a.lay.page_shift, in_page = (1 << shift) - 1;
  // This thread's place in the ring: codes of pass p of tile n, then params.
  uint8_t* ring = smem + C::kOffRing + kSide * C::kRing * C::kRingTile;
  const uint32_t ring_u32 = sb + C::kOffRing + kSide * C::kRing * C::kRingTile;
  auto ring16 = [&](int n, int p) { return (n % C::kRing) * C::kRingTile + p * C::kRingPass + ct * 16; };
  auto ring4 = [&](int n, int p) { return (n % C::kRing) * C::kRingTile + p * C::kRingPass + 128 * 16 + ct * 4; };
  // Of the item the next tile to be copied belongs to:
  const int* table;           // its request's row of the block table
  const uint8_t *codes, *params;  // this thread's, of token 0 of page 0
  int key, key_end, hi, all_hi, all_lo;
  bool opening;               // that tile is its item's first
  auto open = [&]() {
    __syncwarp();
    const auto& w = walk;
    table = a.table + static_cast<long long>(w.w.b) * a.max_pages;
    const uint8_t* rec = a.cache + static_cast<long long>(w.w.h) * a.lay.record;
    codes = rec + (kSide ? a.lay.v_codes : 0) + part * 16;
    params = rec + (kSide ? a.lay.v_params : a.lay.k_params) + group * 4;
    key = (w.w.blk.tile_lo + w.first) * kTile;
    key_end = (w.w.blk.tile_lo + w.last) * kTile;
    hi = w.w.blk.hi;
    all_hi = w.w.blk.all_hi;
    all_lo = w.w.blk.all_lo;
    opening = true;
    __syncwarp();
  };
  int pages[C::kPasses];      // of that tile
  auto locate = [&]() {
#pragma unroll
    for (int p = 0; p < C::kPasses; ++p) {
      const int tok = key + p * C::kPassTokens + ptok;
      pages[p] = 0;
      // volatile: issued here, an iteration before it is used
      if (tok < hi) asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(pages[p]) : "l"(table + (tok >> shift)));
    }
  };
  int n = 0;         // tiles copied
  bool more = true;  // is there another one?
  auto copy = [&]() {
    if (more) {
      if (ct == 0)
        un.meta[kSide][n & 7] = (key + kTile > all_hi || key < all_lo ? 1 : 0) | (opening ? 2 : 0);
#pragma unroll
      for (int p = 0; p < C::kPasses; ++p) {
        const int tok = key + p * C::kPassTokens + ptok;
        int pg = pages[p];
        if (static_cast<unsigned>(pg) >= static_cast<unsigned>(a.num_pages)) {
          atomicCAS(a.input_err, 0, 1);
          pg = 0;
        }
        const int off = tok & in_page;
        const long long at = pg * page_bytes;
        cp_async16(ring_u32 + ring16(n, p), codes + at + off * C::kCodeRow, tok < hi);
        const uint8_t* par = params + at + off * C::kParamRow;
        cp_async4(ring_u32 + ring4(n, p), par, tok < hi);
        if (kSide == 0) cp_async4(ring_u32 + ring4(n, p) + 128 * 4, par + (a.lay.v_params - a.lay.k_params), tok < hi);
      }
      opening = false;
      key += kTile;
      ++n;
      if (key >= key_end) {
        __syncwarp();
        int on = 0;
        if (lane == 0) on = walk.next_item(a);
        more = __shfl_sync(0xffffffffu, on, 0) != 0;
        if (more) open();
      }
      if (more) locate();
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // Byte of the tile where word 0 of pass 0 goes (128-byte swizzle); word i is
  // chunk i, and a pass later the swizzle is the same.
  static_assert(C::kPassTokens % 8 == 0, "a pass later the swizzle is the same");
  const int place = (part >> 1) * C::kAtom + ptok * 128 + ((((part & 1) * 4) ^ (ptok & 7)) << 4);

  // Units: |minimum| < 2^(e + 14), scale < 2^(e + 10).  `limit` holds both bounds
  // as a param does; params within it need no new unit.
  auto unit_of = [&](const uint32_t* top) -> int {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __vmaxu2(m, top[i]);
    const int em = static_cast<int>(m >> 23), es = static_cast<int>((m >> 7) & 255);
    return max(max(em - 127 + 1 - 14, es - 127 + 1 - 10), -110);
  };
  auto limit_of = [&](int e) -> uint32_t {
    return (static_cast<uint32_t>(min(e + 14 + 127, 255) * 128 - 1) << 16) |
           (static_cast<uint32_t>(e + 10 + 127) * 128 - 1);
  };
  auto post = [&](uint32_t top, int which) {
    const uint32_t m = __reduce_max_sync(0xffffffffu, top >> 16), sc = __reduce_max_sync(0xffffffffu, top & 0xffffu);
    if (lane == 0) un.top_param[which][cw] = (m << 16) | sc;
  };
  int e_mine = 0, e_v = 0;                // this side's unit; K's converter: V's
  uint32_t lim_mine = 0, lim_v = 0;
  bool ok = true;
  open();
  locate();
  for (int i = 0; i < C::kRing - 1; ++i) copy();
  for (int it = 0; it < n; ++it) {
    const int st = it % kSt, slot = it & (kUnits - 1);
    copy();
    asm volatile("cp.async.wait_group %0;" ::"n"(C::kRing - 1) : "memory");
    uint32_t par[C::kPasses], par_v[C::kPasses];
    uint32_t top = 0, top_v = 0;
#pragma unroll
    for (int p = 0; p < C::kPasses; ++p) {
      par[p] = *reinterpret_cast<const uint32_t*>(ring + ring4(it, p));
      if (!odd_param(par[p])) top = __vmaxu2(top, par[p] & 0x7fff7fffu);
      if (kSide == 0) {
        par_v[p] = *reinterpret_cast<const uint32_t*>(ring + ring4(it, p) + 128 * 4);
        if (!odd_param(par_v[p])) top_v = __vmaxu2(top_v, par_v[p] & 0x7fff7fffu);
      }
    }
    // Do all params fit the units?  Every warp passes here once a tile, so that
    // one that gave up on a wait takes the others along (a wait is given up
    // only with the flag set); the flags of the tile are there behind it, too.
    const bool fits = __vmaxu2(top, lim_mine) == lim_mine && (kSide || __vmaxu2(top_v, lim_v) == lim_v);
    const bool keep = bar_and_128(kBar, fits && ok);
    const int flags = un.meta[kSide][it & 7];
    if (!keep || (flags & 2)) {
      ok = bar_and_128(kBar, ok && *ab.flag == 0);
      if (!ok) break;
      post(top, 2 * kSide);
      if (kSide == 0) post(top_v, 1);
      asm volatile("bar.sync %0, 128;" ::"n"(kBar) : "memory");
      const int e = unit_of(un.top_param[2 * kSide]);
      e_mine = (flags & 2) ? e : max(e_mine, e);
      lim_mine = limit_of(e_mine);
      if (kSide == 0) {
        const int v = unit_of(un.top_param[1]);
        e_v = (flags & 2) ? v : max(e_v, v);
        lim_v = limit_of(e_v);
      }
    }
    const float unit = pow2i(-e_mine);
    if (kSide == 0 && ct == 0) {
      un.k_unit[slot] = pow2i(e_mine);
      un.v_exp[slot] = e_v;
      un.any_odd[slot] = 0;
    }
    if (flags & 1) {
      // Values that are not numbers, where some row does not see them: left out
      // of the product; the rows that see them add them by themselves.
      if (kSide == 0) asm volatile("bar.sync %0, 128;" ::"n"(kBar) : "memory");  // any_odd is 0
#pragma unroll
      for (int p = 0; p < C::kPasses; ++p) {
        if (kSide == 1) {
          if (odd_param(par[p])) par[p] = 0;
        } else {
          uint32_t bits = odd_param(par_v[p]) ? 1u << group : 0u;
#pragma unroll
          for (int d = kTok; d < kTok * C::kTpr; d <<= 1) bits |= __shfl_xor_sync(0xffffffffu, bits, d);
          if (part == 0) un.odd_v[slot][p * C::kPassTokens + ptok] = static_cast<uint8_t>(bits);
          if (bits) un.any_odd[slot] = 1;
        }
      }
    }
    if (it >= kSt && !__all_sync(0xffffffffu, mbar_wait(bar_empty + 8u * st, ((it / kSt) & 1) ^ 1, ab))) {
      ok = false;
      continue;
    }
    uint8_t* tile = smem + (kSide ? C::kOffV : C::kOffK) + st * C::kTileBytes;
#pragma unroll
    for (int p = 0; p < C::kPasses; ++p) {
      const uint4 x = *reinterpret_cast<const uint4*>(ring + ring16(it, p));
      const float s = param_scale(par[p]) * unit;
      const float m = fmaf(8.f, s, param_min(par[p]) * unit);
      const uint32_t s2 = pack_f16(s, s), m2 = pack_f16(m, m);
      const uint32_t ww[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t c = codes_m8(ww[i], e);
          o[e] = kSide ? fma_f16x2(c, s2, m2) : mul_f16x2(c, s2);
        }
        *reinterpret_cast<uint4*>(tile + (place ^ (i << 4)) + p * C::kPassTokens * 128) =
            make_uint4(o[0], o[1], o[2], o[3]);
      }
      if (kSide == 0 && (GROUP == 32 || (part & 1) == 0)) {
        const int tok = p * C::kPassTokens + ptok;
        const __half h = __float2half_rn(m);
        uint8_t* ex = smem + C::kOffKEx + st * C::kKEx + (tok >> 3) * C::kExRow8 + (tok & 7) * 16;
        const int k0 = 2 * group, k1 = 2 * C::kGroups + group;
        *reinterpret_cast<uint32_t*>(ex + (k0 >> 3) * 128 + (k0 & 7) * 2) =
            pack_f16(m, m - __half2float(h));
        *reinterpret_cast<__half*>(ex + (k1 >> 3) * 128 + (k1 & 7) * 2) = h;
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_full + 8u * st);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <int HD, int GROUP>
__global__ void __launch_bounds__(Cfg<HD, GROUP>::kThreads, 1) kv4_chunk_kernel(const Kv4AttnArgs a) {
  using C = Cfg<HD, GROUP>;
  constexpr int kThreads = C::kThreads;
  constexpr int kConvK = 4 * C::kBlocks, kConvV = kConvK + 4, kMma = kConvV + 4;  // first warps
  extern __shared__ uint8_t smem_raw[];
  __shared__ long long scratch[kThreads / 32 + 2];
  __shared__ Units un;
  // Every warp's walk through the share: touched once an item, it would only
  // take registers.
  __shared__ Tiles<C::kBlockRows> walks[kThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t raw_u32 = smem_u32(smem_raw);
  const uint32_t pad = ((raw_u32 + 1023u) & ~1023u) - raw_u32;
  uint8_t* smem = smem_raw + pad;
  const uint32_t sb = raw_u32 + pad;
  const uint32_t bar0 = sb + C::kOffBar;
  const uint32_t bar_kfull = bar0, bar_kempty = bar0 + 16, bar_vfull = bar0 + 32,
                 bar_vempty = bar0 + 48;
  auto bar_q = [&](int g) { return bar0 + 64u + 56u * g; };
  auto bar_sfull = [&](int g, int b) { return bar0 + 72u + 56u * g + 8u * b; };
  auto bar_pfull = [&](int g, int b) { return bar0 + 88u + 56u * g + 8u * b; };
  auto bar_odone = [&](int g) { return bar0 + 104u + 56u * g; };
  auto bar_drain = [&](int g) { return bar0 + 112u + 56u * g; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  const Kv4Share share = kv4_share<kTile, kThreads, true>(a, C::kBlockRows, a.whole_items ? 1 : kLead + 2, scratch);
  if (share.per * blockIdx.x >= share.total) {
    if (tid == 0 && !a.whole_items) a.split[blockIdx.x] = make_int4(0, 0, 0, 0);
    return;
  }

  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar_kfull + 8 * s, 4);
      mbar_init(bar_kempty + 8 * s, C::kBlocks);
      mbar_init(bar_vfull + 8 * s, 4);
      mbar_init(bar_vempty + 8 * s, C::kBlocks);
    }
    for (int g = 0; g < C::kBlocks; ++g) {
      mbar_init(bar_q(g), 4);
      for (int b = 0; b < 2; ++b) {
        mbar_init(bar_sfull(g, b), 1);
        mbar_init(bar_pfull(g, b), 4);
      }
      mbar_init(bar_odone(g), 1);
      mbar_init(bar_drain(g), 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  // Slots of the extra k-steps that no group uses stay zero.
  for (int i = tid; i < (C::kBlocks * C::kQEx + C::kKSt * C::kKEx) / 16; i += kThreads)
    reinterpret_cast<uint4*>(smem + C::kOffQEx)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  if (warp == kMma) {
    tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Abort ab{a.wait_err, abort_flag};
  Tiles<C::kBlockRows>& w = walks[warp];
  if (lane == 0) w.begin(a, share);
  __syncwarp();
  auto next_item = [&]() -> bool {
    __syncwarp();
    int more = 0;
    if (lane == 0) more = w.next_item(a);
    return __shfl_sync(0xffffffffu, more, 0) != 0;  // (and the walk is the warp's again)
  };

  if (warp < kConvK) {
    // ---------------------------------------------------------- rows
    regs_inc<C::kRowRegs>();
    const int g = warp >> 2;                 // block of 128 rows
    const int row = (warp & 3) * 32 + lane;  // of the block
    const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + 128u * g;  // S
    const uint32_t to = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + C::kColO + HD * g;
    uint8_t* sq = smem + C::kOffQ + g * C::kQTile;
    const uint32_t sq_u32 = sb + C::kOffQ + g * C::kQTile;
    constexpr int kChunks = HD / 8;  // 16 bytes each of a row of bf16 or fp16
    auto row_chunk = [](int r, int c) {  // where chunk c of row r is (128-byte swizzle)
      return (c >> 3) * C::kQAtom + r * 128 + (((c & 7) ^ (r & 7)) << 4);
    };
    uint8_t* sqx = smem + C::kOffQEx + g * C::kQEx;
    int4 record = make_int4(0, 0, 0, 0);
    bool ok = true, first_item = true;
    int tile = 0;  // of the share
    int it = 0;    // of this block of rows: the tiles of the items that reach it
    do {
      const auto& k = w.w;
      const int first_tile = w.first, last_tile = w.last;
      const bool whole = first_tile == 0 && last_tile == k.blk.tiles;
      if (first_tile == 0 && !whole) record = kv4_split_record(k, share);
      if (k.blk.rows <= kRows * g) {  // nothing for these rows
        tile += last_tile - first_tile;
        first_item = false;
        continue;
      }
      const int key_first = (k.blk.tile_lo + first_tile) * kTile;
      const int key_end = (k.blk.tile_lo + last_tile) * kTile;
      const int all_hi = k.blk.all_hi, all_lo = k.blk.all_lo;
      const bool have = kRows * g + row < k.blk.rows;
      const int gr = k.blk.row0 + (have ? kRows * g + row : 0);
      const int t = gr / a.per_kv, head = k.h * a.per_kv + gr - t * a.per_kv;
      int row_lo = 0, row_hi = have ? k.req.kv : 0;
      if (have && (a.causal || a.window >= 0)) row_hi = max(min(row_hi, k.blk.pos0 + t + 1), 0);
      if (a.window >= 0) row_lo = max(k.blk.pos0 + t - min(a.window, 0x3fffffff), 0);
      const uint32_t seen = static_cast<uint32_t>(max(row_hi - row_lo, 0));

      // Q: the row scaled by a power of two into [2^7, 2^8), in fp16, and the
      // slots of its sums over the groups.  The products of the item before
      // have all completed (its O was read), so the tile is free.  The warp copies
      // its rows whole rows at a time (a thread's own row would be a line for each
      // lane), then each thread works on its own.
      float row_scale;
      {
        const long long q_at = have ? static_cast<long long>(k.req.start + t) * a.q_ts +
                                          static_cast<long long>(head) * a.q_hs
                                    : -1;
#pragma unroll 4
        for (int i = 0; i < kChunks; ++i) {
          const int r = i * (32 / kChunks) + lane / kChunks, c = lane % kChunks;
          const long long at = __shfl_sync(0xffffffffu, q_at, r);
          cp_async16(sq_u32 + row_chunk((warp & 3) * 32 + r, c), a.Q + max(at, 0ll) + 8 * c, at >= 0);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncwarp();
        uint32_t top = 0;
#pragma unroll 8
        for (int c = 0; c < kChunks; ++c) {
          const uint4 x = *reinterpret_cast<const uint4*>(sq + row_chunk(row, c));
          top = __vmaxu2(top, __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                                       __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu)));
        }
        // (A row below 2^-119 is left below 2^7: fp16's step, 2^-24, still is
        // 2^-17 of the smallest bf16.)
        const int et = static_cast<int>(max(top & 0xffffu, top >> 16) >> 7) - 127;  // -127: zero
        const int up = min(7 - et, 126);
        const float unit = pow2i(up);
        row_scale = a.scale_log2 * pow2i(-up);
        const uint64_t unit2 = f2_pack(unit, unit);
        uint64_t sum2 = 0;
#pragma unroll 4
        for (int c = 0; c < kChunks; ++c) {
          uint4* place = reinterpret_cast<uint4*>(sq + row_chunk(row, c));
          const uint4 x = *place;
          const uint32_t in[4] = {x.x, x.y, x.z, x.w};
          uint32_t out[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint64_t y =
                f2_mul(f2_pack(__uint_as_float(in[i] << 16), __uint_as_float(in[i] & 0xffff0000u)), unit2);
            sum2 = f2_add(sum2, y);
            float lo, hi;
            f2_unpack(y, lo, hi);
            out[i] = pack_f16(lo, hi);
          }
          *place = make_uint4(out[0], out[1], out[2], out[3]);
          if ((c + 1) % (GROUP / 8) == 0) {
            const int grp = c / (GROUP / 8);
            float s0, s1;
            f2_unpack(sum2, s0, s1);
            const float sum = s0 + s1;
            const __half h = __float2half_rn(sum), l = __float2half_rn(sum - __half2float(h));
            const __half slot[3] = {h, h, l};
#pragma unroll
            for (int e = 0; e < 3; ++e) {
              const int kk = e < 2 ? 2 * grp + e : 2 * C::kGroups + grp;
              *reinterpret_cast<__half*>(sqx + (row >> 3) * C::kExRow8 + (kk >> 3) * 128 +
                                         (row & 7) * 16 + (kk & 7) * 2) = slot[e];
            }
            sum2 = 0;
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_q(g));

      float m_run = -INFINITY, l_run = 0.f;
      int v_ref = 0;
      uint32_t nan_groups = 0;
      for (int key0 = key_first; key0 < key_end; key0 += kTile, ++it, ++tile) {
        const int bb = it & 1, slot = tile & (kUnits - 1);
        const uint32_t scol = tl + (bb ? 64u : 0u);
        if (!__all_sync(0xffffffffu, mbar_wait(bar_sfull(g, bb), (it >> 1) & 1, ab))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const float mult = row_scale * un.k_unit[slot];
        const bool start = key0 == key_first;
        const bool edge = key0 + kTile > all_hi || key0 < all_lo;
        float alpha = 1.f;
        bool rescale = false;
        {
          uint32_t sr[2][32];
          tmem_ld32(scol, sr[0]);
          tmem_ld32(scol + 32, sr[1]);
          tmem_wait_ld();
          if (edge) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                sr[c][e] = static_cast<uint32_t>(key0 + 32 * c + e - row_lo) < seen
                               ? sr[c][e]
                               : __float_as_uint(-INFINITY);
          }
          float mxp[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int e = 0; e < 32; e += 2)
              mxp[(e >> 1) & 3] = max3(mxp[(e >> 1) & 3], __uint_as_float(sr[c][e]), __uint_as_float(sr[c][e + 1]));
          const float cand = fmaxf(fmaxf(mxp[0], mxp[1]), fmaxf(mxp[2], mxp[3])) * mult;
          const bool up = cand > m_run + kGrow;
          const float m_new = up ? cand : m_run;
          alpha = up ? ex2(m_run - m_new) : 1.f;
          rescale = up;
          const float base = m_new == -INFINITY ? 0.f : kShift - m_new;
          const uint64_t mult2 = f2_pack(mult, mult), base2 = f2_pack(base, base);
          uint64_t sum2[2] = {0ull, 0ull};
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float x0, x1;
              f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[c][2 * e]), __uint_as_float(sr[c][2 * e + 1])),
                               mult2, base2),
                        x0, x1);
              const float p0 = ex2(x0), p1 = ex2(x1);
              pk[e] = pack_f16(p0, p1);
              sum2[e & 1] = f2_add(sum2[e & 1], f2_pack(p0, p1));
            }
            tmem_st16(scol + 16 * c, pk);
          }
          float z0, z1;
          f2_unpack(f2_add(sum2[0], sum2[1]), z0, z1);
          l_run = l_run * alpha + (z0 + z1);
          m_run = m_new;
        }
        if (edge && un.any_odd[slot])
          for (int e = 0; e < kTile; ++e)
            if (static_cast<uint32_t>(key0 + e - row_lo) < seen) nan_groups |= un.odd_v[slot][e];
        const int ve = un.v_exp[slot];
        if (!start && ve != v_ref) {  // grown
          alpha *= ex2(static_cast<float>(v_ref - ve));
          rescale = true;
        }
        v_ref = ve;
        if (!start) {
          // The product of the tile before has to be complete: O may be rescaled
          // then, and the phase waited for is the only one that can be open
          // (the next product needs this tile's P).
          if (!__all_sync(0xffffffffu, mbar_wait(bar_odone(g), (it - 1) & 1, ab))) {
            ok = false;
            break;
          }
          if (__any_sync(0xffffffffu, rescale)) {
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < HD / 16; ++c) {
              uint32_t o[16];
              tmem_ld16(to + 16 * c, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st16(to + 16 * c, o);
            }
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_pfull(g, bb));
      }
      if (ok) {
        ok = __all_sync(0xffffffffu, mbar_wait(bar_odone(g), (it - 1) & 1, ab));
        tc_fence_after();
      }
      ok = bar_and_128(1 + g, ok && *abort_flag == 0);
      if (!ok) break;

      const float v_up = ex2(static_cast<float>(v_ref));
      const float top = m_run - kShift;
      const float f = whole ? (l_run == 0.f ? 0.f : v_up / l_run) : v_up;
      const long long o_row = static_cast<long long>(k.req.start + t) * a.Hq + head;
      const long long p_row =
          (2ll * blockIdx.x + (first_item && first_tile > 0 ? 0 : 1)) * C::kBlockRows + kRows * g + row;
      // Out by way of the item's Q tile, which has served: a thread puts its row
      // there, as bf16 or one half after the other as fp32, and the warp writes
      // whole rows.
      const long long out_at = !have ? -1 : whole ? o_row * (HD * 2) : p_row * (HD * 4);  // bytes
#pragma unroll 1
      for (int part = 0; part < (whole ? 1 : 2); ++part) {
        __syncwarp();
#pragma unroll 1
        for (int c = 0; c < (whole ? HD / 16 : HD / 32); ++c) {
          const int col = 16 * c + part * (HD / 2);
          uint32_t o[16];
          tmem_ld16(to + col, o);
          tmem_wait_ld();
          const bool odd = (nan_groups >> (col / GROUP)) & 1;
          float x[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = odd ? __int_as_float(0x7fffffff) : __uint_as_float(o[e]) * f;
          if (whole) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
              *reinterpret_cast<uint4*>(sq + row_chunk(row, 2 * c + e)) =
                  make_uint4(pack_bf16(x[8 * e], x[8 * e + 1]), pack_bf16(x[8 * e + 2], x[8 * e + 3]),
                             pack_bf16(x[8 * e + 4], x[8 * e + 5]), pack_bf16(x[8 * e + 6], x[8 * e + 7]));
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              *reinterpret_cast<float4*>(sq + row_chunk(row, 4 * c + e)) =
                  make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
          }
        }
        __syncwarp();
        uint8_t* dst = whole ? reinterpret_cast<uint8_t*>(a.O)
                             : reinterpret_cast<uint8_t*>(a.part_o) + part * (HD * 2);
#pragma unroll 4
        for (int i = 0; i < kChunks; ++i) {
          const int r = i * (32 / kChunks) + lane / kChunks, c = lane % kChunks;
          const long long at = __shfl_sync(0xffffffffu, out_at, r);
          const uint4 x = *reinterpret_cast<const uint4*>(sq + row_chunk((warp & 3) * 32 + r, c));
          if (at >= 0) *reinterpret_cast<uint4*>(dst + at + 16 * c) = x;
        }
      }
      if (have) {
        if (whole)
          a.L[o_row] = l_run == 0.f ? -INFINITY : (top + log2f(l_run)) * kLn2f;
        else
          a.part_stat[p_row] = make_float2(top, l_run);
      }
      // O has been read before the next item's products may overwrite it: they
      // wait for p_full, which this warp signals after this point.
      tc_fence_before();
      __syncwarp();  // and the tile before the next item's Q
      first_item = false;
    } while (next_item());
    if (tid == 0 && !a.whole_items) a.split[blockIdx.x] = record;
  } else if (warp < kConvV) {
    regs_dec<C::kConvRegs>();
    convert<HD, GROUP, 0>(a, w, smem, sb, bar_kfull, bar_kempty, un, ab);
  } else if (warp < kMma) {
    regs_dec<C::kConvRegs>();
    convert<HD, GROUP, 1>(a, w, smem, sb, bar_vfull, bar_vempty, un, ab);
  } else {
    regs_dec<C::kMmaRegs>();
  }
  if (warp >= kMma && warp < kMma + C::kBlocks) {
    // ---------------------------------------------------------- products
    // The whole warp walks along and one elected lane issues: what the warp
    // computes is the same in every lane, so the descriptors live in uniform
    // registers, where the products take them from.
    constexpr uint32_t idS = idesc_f16(kRows, kTile, false);
    constexpr uint32_t idO = idesc_f16(kRows, HD, true);
    constexpr int kD = HD / 16, kC = kTile / 16;
    const int g = __shfl_sync(0xffffffffu, warp - kMma, 0);  // block of rows
    const bool leader = elect_one();
    auto wait = [&](uint32_t bar, int parity) {
      return __all_sync(0xffffffffu, mbar_wait(bar, static_cast<uint32_t>(parity), ab)) != 0;
    };
    bool ok = true;
    int tile = 0;                 // of the share
    int it = 0, item = 0;         // tiles and items of this block of rows
    bool prev_first = false;      // was its last tile its item's first?
    const uint64_t q0 = sdesc_sw128(sb + C::kOffQ + g * C::kQTile, 16, 1024);
    const uint64_t qx = sdesc_plain(sb + C::kOffQEx + g * C::kQEx, 128, C::kExRow8);
    const uint64_t k0 = sdesc_sw128(sb + C::kOffK, 16, 1024);
    const uint64_t kx = sdesc_plain(sb + C::kOffKEx, 128, C::kExRow8);
    const uint64_t v0 = sdesc_sw128(sb + C::kOffV, C::kAtom, 1024);
    const uint32_t tbase = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t ts = tbase + 128u * g, to = tbase + C::kColO + HD * g;
    // P V of tile `tile - 1`, this block's `it - 1`.
    auto issue_pv = [&]() -> bool {
      const int vs = (tile - 1) % C::kVSt, bb = (it - 1) & 1;
      if (!wait(bar_vfull + 8u * vs, ((tile - 1) / C::kVSt) & 1)) return false;
      if (!wait(bar_pfull(g, bb), ((it - 1) >> 1) & 1)) return false;
      tc_fence_after();
      if (leader) {
        uint64_t b[kC];
        uint32_t p[kC];
#pragma unroll
        for (int k = 0; k < kC; ++k) {
          b[k] = sdesc_add(v0, vs * C::kTileBytes + k * 2048);
          p[k] = ts + (bb ? 64u : 0u) + 8u * k;
        }
        mma_ts_k(to, p, b, idO, prev_first ? 0u : 1u);
        mma_commit(bar_odone(g));
        mma_commit(bar_vempty + 8u * vs);
      }
      __syncwarp();
      return true;
    };
    bool pending = false;         // is P V of the tile before still to be issued?
    do {
      const int tiles = w.last - w.first;
      const bool none = w.w.blk.rows <= kRows * g;
      // The rows put an item's Q in place once they have read the O before, for
      // which the last product has to be issued first.
      if (pending && !issue_pv()) {
        ok = false;
        break;
      }
      pending = false;
      if (none) {  // nothing for these rows: the tiles are let go
        for (int i = 0; ok && i < tiles; ++i, ++tile) {
          const int ks = tile % C::kKSt, vs = tile % C::kVSt;
          ok = wait(bar_kfull + 8u * ks, (tile / C::kKSt) & 1);
          if (ok && leader) mbar_arrive(bar_kempty + 8u * ks);
          ok = ok && wait(bar_vfull + 8u * vs, (tile / C::kVSt) & 1);
          if (ok && leader) mbar_arrive(bar_vempty + 8u * vs);
        }
        continue;
      }
      if (!wait(bar_q(g), item & 1)) {
        ok = false;
        break;
      }
      ++item;
      for (int i = 0; i < tiles; ++i) {
        const int ks = tile % C::kKSt, bb = it & 1;
        // S over P of two tiles before: its product has to be complete.  (At an
        // item's first tile the wait for Q has shown more than that, and the
        // phase waited for here may be over already.)
        if (it >= 2 && pending && !wait(bar_odone(g), (it - 2) & 1)) { ok = false; break; }
        if (!wait(bar_kfull + 8u * ks, (tile / C::kKSt) & 1)) { ok = false; break; }
        tc_fence_after();
        if (leader) {
          const uint32_t dst = ts + (bb ? 64u : 0u);
          uint64_t q[kD], b[kD];
#pragma unroll
          for (int k = 0; k < kD; ++k) {
            q[k] = sdesc_add(q0, (k >> 2) * C::kQAtom + (k & 3) * 32);
            b[k] = sdesc_add(k0, ks * C::kTileBytes + (k >> 2) * C::kAtom + (k & 3) * 32);
          }
          mma_ss_k(dst, q, b, idS, 0u);
#pragma unroll
          for (int k = 0; k < C::kExSteps; ++k)
            mma_ss(dst, sdesc_add(qx, k * 256), sdesc_add(kx, ks * C::kKEx + k * 256), idS, 1u);
          mma_commit(bar_sfull(g, bb));
          mma_commit(bar_kempty + 8u * ks);
        }
        __syncwarp();
        if (pending && !issue_pv()) { ok = false; break; }
        ++it;
        ++tile;
        prev_first = i == 0;
        pending = true;
      }
    } while (ok && next_item());
    if (ok && pending && *abort_flag == 0) issue_pv();
    if (leader) {
      mma_commit(bar_drain(g));
      mbar_wait_drain(bar_drain(g), 0);
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMma) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int HD, int GROUP>
cudaError_t launch_chunk(const Kv4AttnArgs& a, cudaStream_t stream, int* ctas) {
  using C = Cfg<HD, GROUP>;
  static std::atomic<bool> ready[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !ready[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kv4_chunk_kernel<HD, GROUP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready[dev].store(true, std::memory_order_release);
  }
  const int sms = sm_count();
  if (sms < 1) return cudaErrorInvalidDevice;
  *ctas = sms < kKv4MaxChunkCtas ? sms : kKv4MaxChunkCtas;
  Kv4AttnArgs ag = a;
  ag.lead = kLead;
  kv4_chunk_kernel<HD, GROUP><<<*ctas, C::kThreads, C::kSmem, stream>>>(ag);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_chunk(int d, int group, const Kv4AttnArgs& a, cudaStream_t stream, int* ctas) {
  const bool g32 = group == 32;
  switch (d) {
    case 64: return g32 ? launch_chunk<64, 32>(a, stream, ctas) : launch_chunk<64, 64>(a, stream, ctas);
    case 128: return g32 ? launch_chunk<128, 32>(a, stream, ctas) : launch_chunk<128, 64>(a, stream, ctas);
    case 256: return g32 ? launch_chunk<256, 32>(a, stream, ctas) : launch_chunk<256, 64>(a, stream, ctas);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fa
