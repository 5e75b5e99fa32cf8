// kv4_sched.cuh -- how attention over the paged cache is dealt out to CTAs.
//
// The work is a list of items: request b, block rb of its query rows, K/V head
// h.  A request's rows are its n queries times the per_kv query heads that
// share a K/V head (row = query * per_kv + head in the group), so that a tile of
// the cache that was read once serves all of them.  An item is a run of
// kTile-token tiles, those that hold a key visible to one of its rows (at least
// one, so that a block that sees nothing still writes its zeros).  All tiles of
// all items form one list which is cut into equal shares, one per CTA: lengths
// may differ by any factor and the shares do not.  Changing from one item to the
// next costs a CTA about as much as some tiles (its results, the first copies),
// so an item's tiles are led in the list by `lead` places that stand for that.  An item that a share's end
// cuts is finished from partial results by a second kernel.  Where no item is
// long (whole_items) a place in the list is an item instead, and that kernel is
// not launched.
#pragma once
#include "kv4.h"

namespace fa {

struct Kv4Req {
  int start, n, kv;  // first row of Q, queries, keys
};

__device__ __forceinline__ Kv4Req kv4_request(const Kv4AttnArgs& a, int b, bool* bad) {
  const int start = a.cu_q[b], end = a.cu_q[b + 1];
  Kv4Req r;
  r.start = start;
  r.n = end - start;
  if (start < 0 || end < start || end > a.total_q || r.n > a.max_q) {
    r.n = 0;
    *bad = true;
  }
  const long long room = static_cast<long long>(a.max_pages) << a.lay.page_shift;
  r.kv = static_cast<int>(min(static_cast<long long>(max(a.kv_len[b], 0)), room));
  return r;
}

struct Kv4Block {
  int row0, rows;         // rows of the block
  int pos0;               // position of the request's first query
  int lo, hi;             // keys that some row sees
  int all_lo, all_hi;     // keys that every row sees
  int tile_lo, tiles;
  int units;              // places in the list: a.lead + tiles, or 1 if items are not cut
};

template <int kTile>
__device__ __forceinline__ Kv4Block kv4_block(const Kv4AttnArgs& a, const Kv4Req& r, int rb,
                                              int block_rows) {
  Kv4Block k;
  k.row0 = rb * block_rows;
  k.rows = min(r.n * a.per_kv - k.row0, block_rows);
  k.pos0 = r.kv - r.n;
  int first = 0, last = r.n - 1;
  if (rb > 0 || k.rows < r.n * a.per_kv) {  // (one block holds all: no divisions)
    first = k.row0 / a.per_kv;
    last = (k.row0 + k.rows - 1) / a.per_kv;
  }
  k.lo = 0;
  k.hi = r.kv;
  k.all_lo = 0;
  k.all_hi = r.kv;
  if (a.causal || a.window >= 0) {
    k.hi = max(min(r.kv, k.pos0 + last + 1), 0);
    k.all_hi = max(k.pos0 + first + 1, 0);
  }
  if (a.window >= 0) {
    // p - w, without passing the range of int for a large window
    k.lo = max(k.pos0 + first - min(a.window, 0x3fffffff), 0);
    k.all_lo = max(k.pos0 + last - min(a.window, 0x3fffffff), 0);
  }
  k.tile_lo = k.lo / kTile;
  k.tiles = max((k.hi + kTile - 1) / kTile - k.tile_lo, 1);
  k.units = a.whole_items ? 1 : a.lead + k.tiles;
  return k;
}

// A request of more blocks of rows than this is looked through by a whole warp
// (65536 queries with a window: 145 -> 54 us).  The kernel for few rows has no
// such requests (kMany false), and the choice would cost it half a microsecond.
constexpr int kKv4OwnBlocks = 4;

// Places of request b (none: -1) in the list.  Every lane of a warp calls it, each
// with a request of its own.
template <int kTile, bool kMany>
__device__ __forceinline__ long long kv4_units(const Kv4AttnArgs& a, int b, int block_rows,
                                               bool* bad) {
  Kv4Req r{0, 0, 0};
  if (b >= 0) r = kv4_request(a, b, bad);
  const int blocks = (r.n * a.per_kv + block_rows - 1) / block_rows;
  long long n = 0;
  if (!kMany || blocks <= kKv4OwnBlocks)
    for (int rb = 0; rb < blocks; ++rb) n += kv4_block<kTile>(a, r, rb, block_rows).units;
  if (!kMany) return n * a.Hkv;
  uint32_t many = __ballot_sync(0xffffffffu, blocks > kKv4OwnBlocks);
  for (; many; many &= many - 1) {
    const int lane = threadIdx.x & 31, whose = __ffs(many) - 1;
    const Kv4Req o{0, __shfl_sync(0xffffffffu, r.n, whose), __shfl_sync(0xffffffffu, r.kv, whose)};
    const int o_blocks = __shfl_sync(0xffffffffu, blocks, whose);
    long long sum = 0;
    for (int rb = lane; rb < o_blocks; rb += 32) sum += kv4_block<kTile>(a, o, rb, block_rows).units;
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == whose) n = sum;
  }
  return n * a.Hkv;
}

// n / d for 0 <= n, 0 < d, in 32 bits where that is enough.
__device__ __forceinline__ long long kv4_div(long long n, long long d) {
  if (((n | d) >> 32) == 0)
    return static_cast<long long>(static_cast<uint32_t>(n) / static_cast<uint32_t>(d));
  return n / d;
}

struct Kv4Share {
  long long total, per;  // places in the list, and in a share
  long long begin;       // first place that belongs to blocks of rows from rb on of request b
  int b, rb;             // (of few blocks: rb is 0 and the walk looks for its own)
};

// Finds the block of rows of request s.b that holds place u0, if there are many.
// Every lane of a warp calls it.
template <int kTile>
__device__ __forceinline__ void kv4_find_block(const Kv4AttnArgs& a, int block_rows, long long u0, Kv4Share* s) {
  bool bad = false;
  const int lane = threadIdx.x & 31;
  const Kv4Req r = kv4_request(a, s->b, &bad);
  const int blocks = (r.n * a.per_kv + block_rows - 1) / block_rows;
  if (blocks <= kKv4OwnBlocks) return;
  for (int base = 0; base < blocks; base += 32) {
    const int rb = base + lane;
    const long long mine =
        rb < blocks ? static_cast<long long>(kv4_block<kTile>(a, r, rb, block_rows).units) * a.Hkv : 0;
    long long incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    const uint32_t who = __ballot_sync(0xffffffffu, u0 < s->begin + incl);
    if (who) {
      s->rb = base + __ffs(who) - 1;
      s->begin += __shfl_sync(0xffffffffu, incl - mine, __ffs(who) - 1);
      return;
    }
    s->begin += __shfl_sync(0xffffffffu, incl, 31);
  }
}

// Every thread of the block finds the block's share; `scratch` holds
// kThreads / 32 + 2 long longs.  Shares are at least min_tiles long.  begin/b are
// set when the share is not empty (blockIdx.x * per < total).  Up to 128 requests
// every warp adds up all of them by itself, which spares the barriers.
template <int kTile, int kThreads, bool kMany>
__device__ __forceinline__ Kv4Share kv4_share(const Kv4AttnArgs& a, int block_rows, int min_tiles,
                                              long long* scratch) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  bool bad = false;
  Kv4Share s;
  s.b = s.rb = 0;
  s.begin = 0;
  if (a.B <= 128) {
    long long mine[4], at[4];  // request 32 i + lane: its tiles, those before it
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int b = 32 * i + lane;
      if (32 * i < a.B) mine[i] = kv4_units<kTile, kMany>(a, b < a.B ? b : -1, block_rows, &bad);
    }
    if (bad && blockIdx.x == 0) atomicCAS(a.input_err, 0, 1);
    s.total = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (32 * i >= a.B) break;
      long long incl = mine[i];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
      }
      at[i] = s.total + incl - mine[i];
      s.total += __shfl_sync(0xffffffffu, incl, 31);
    }
    s.per = max(kv4_div(s.total + gridDim.x - 1, gridDim.x), static_cast<long long>(min_tiles));
    const long long u0 = s.per * blockIdx.x;
    if (u0 >= s.total) return s;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (32 * i >= a.B) break;
      const uint32_t who = __ballot_sync(0xffffffffu, u0 >= at[i] && u0 < at[i] + mine[i]);
      if (who) {
        s.b = 32 * i + __ffs(who) - 1;
        s.begin = __shfl_sync(0xffffffffu, at[i], __ffs(who) - 1);
      }
    }
    if (kMany) kv4_find_block<kTile>(a, block_rows, u0, &s);
    return s;
  }
  const long long first = kv4_units<kTile, kMany>(a, tid < a.B ? tid : -1, block_rows, &bad);
  long long sum = first;
  for (int base = kThreads; base < a.B; base += kThreads)
    sum += kv4_units<kTile, kMany>(a, base + tid < a.B ? base + tid : -1, block_rows, &bad);
  if (bad && blockIdx.x == 0) atomicCAS(a.input_err, 0, 1);
#pragma unroll
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if (lane == 0) scratch[warp] = sum;
  __syncthreads();
  s.total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) s.total += scratch[w];
  s.per = max(kv4_div(s.total + gridDim.x - 1, gridDim.x), static_cast<long long>(min_tiles));
  const long long u0 = s.per * blockIdx.x;
  if (u0 >= s.total) return s;
  long long run = 0;
  for (int base = 0; base < a.B; base += kThreads) {
    const int b = base + tid;
    long long v = first;
    if (base) v = kv4_units<kTile, kMany>(a, b < a.B ? b : -1, block_rows, &bad);
    long long incl = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    __syncthreads();  // the last reads of scratch are done
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    long long before = run;
    for (int w = 0; w < warp; ++w) before += scratch[w];
    for (int w = 0; w < kThreads / 32; ++w) run += scratch[w];
    if (u0 >= before + incl - v && u0 < before + incl) {
      scratch[kThreads / 32] = before + incl - v;
      scratch[kThreads / 32 + 1] = b;
    }
    if (run > u0) break;
  }
  __syncthreads();
  s.begin = scratch[kThreads / 32];
  s.b = static_cast<int>(scratch[kThreads / 32 + 1]);
  if (kMany) kv4_find_block<kTile>(a, block_rows, u0, &s);
  return s;
}

// A CTA's walk through its share, item by item.
template <int kTile>
struct Kv4Walk {
  Kv4Req req;
  Kv4Block blk;
  int b, rb, h, blocks;
  long long item;  // the item's first place in the list

  __device__ __forceinline__ void open(const Kv4AttnArgs& a, int block_rows) {
    bool bad = false;
    req = kv4_request(a, b, &bad);
    blocks = (req.n * a.per_kv + block_rows - 1) / block_rows;
    rb = 0;
    h = 0;
    if (blocks) blk = kv4_block<kTile>(a, req, 0, block_rows);
  }
  // To the item that holds place u of the list, from the request that holds it.
  __device__ __forceinline__ void seek(const Kv4AttnArgs& a, const Kv4Share& s, long long u,
                                       int block_rows) {
    b = s.b;
    item = s.begin;
    open(a, block_rows);
    if (s.rb > 0) {
      rb = s.rb;
      blk = kv4_block<kTile>(a, req, rb, block_rows);
    }
    while (rb + 1 < blocks && u >= item + static_cast<long long>(blk.units) * a.Hkv) {
      item += static_cast<long long>(blk.units) * a.Hkv;
      ++rb;
      blk = kv4_block<kTile>(a, req, rb, block_rows);
    }
    h = static_cast<int>(kv4_div(u - item, blk.units));
    item += static_cast<long long>(h) * blk.units;
  }
  __device__ __forceinline__ void next(const Kv4AttnArgs& a, int block_rows) {
    item += blk.units;
    if (++h < a.Hkv) return;
    h = 0;
    if (++rb < blocks) {
      blk = kv4_block<kTile>(a, req, rb, block_rows);
      return;
    }
    while (++b < a.B) {
      open(a, block_rows);
      if (blocks) return;
    }
  }
};

// The tiles [first, last) of the walk's item that places [u, u_end) of the list
// stand for, none if the share ends within its lead; returns the place behind
// them.
template <int kTile>
__device__ __forceinline__ long long kv4_part(const Kv4AttnArgs& a, const Kv4Walk<kTile>& w, long long u,
                                              long long u_end, int* first, int* last) {
  if (a.whole_items) {
    *first = 0;
    *last = w.blk.tiles;
    return w.item + 1;
  }
  const int end = static_cast<int>(min(static_cast<long long>(w.blk.units), u_end - w.item));
  *first = max(static_cast<int>(u - w.item) - a.lead, 0);
  *last = max(end - a.lead, 0);
  return w.item + end;
}

// The record a CTA leaves for the merge: the item, cut by this share's end,
// that begins in it (x: first query of its request, y: first row of its block,
// z: rows + 512 * K/V head, 0: there is none, w: the last CTA with a part of
// it).  Partial results of CTA i are number 2 i (of its first item, begun
// before) and 2 i + 1 (of its last, begun here).
template <int kTile>
__device__ __forceinline__ int4 kv4_split_record(const Kv4Walk<kTile>& w, const Kv4Share& s) {
  return make_int4(w.req.start, w.blk.row0, w.blk.rows + 512 * w.h,
                   static_cast<int>(kv4_div(w.item + w.blk.units - 1, s.per)));
}

}  // namespace fa
