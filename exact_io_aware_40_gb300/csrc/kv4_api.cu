// kv4_api.cu -- the C ABI declared in include/fa_kv4.h: argument validation and
// launches.  Nothing here touches the device before the arguments are valid.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "fa_kv4.h"
#include "kv4.h"

namespace {

constexpr float kLog2e = 1.4426950408889634f;

constexpr int kMaxTokens = 1 << 30;  // token numbers stay within int

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

bool page_ok(int page_size) {
  return page_size == 16 || page_size == 32 || page_size == 64 || page_size == 128;
}

// Geometry of a cache: pages, page size, channels, group, heads.
fa_status check_cache(int num_pages, int page_size, int d, int group, int Hkv) {
  if (num_pages < 1 || Hkv < 1) return FA_ERR_INVALID_ARG;
  if (fa_kv4_page_bytes(d, page_size, group) == 0) return FA_ERR_UNSUPPORTED;
  if (Hkv > 65535) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(num_pages) * page_size > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

bool strides_ok(int token, int head) {
  return token >= 0 && head >= 0 && token % 8 == 0 && head % 8 == 0;
}

fa_status launched(cudaError_t e) { return e == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

}  // namespace

extern "C" {

size_t fa_kv4_page_bytes(int d, int page_size, int group) {
  if (d != 64 && d != 128 && d != 256) return 0;
  if (!page_ok(page_size) || (group != 32 && group != 64)) return 0;
  return static_cast<size_t>(fa::kv4_layout(d, page_size, group).record);
}

fa_status fa_kv4_plan(const int32_t* past_len, const int32_t* new_len, int B, int page_size,
                      int num_pages, int32_t* block_table, int max_pages, int32_t* free_list,
                      const int32_t* free_state, int max_tokens, int32_t* kv_len, int32_t* cu_q,
                      int32_t* slots, int32_t* state_out, fa_stream_t stream) {
  if (!past_len || !new_len || !block_table || !free_list || !free_state || !kv_len || !cu_q ||
      !slots || !state_out)
    return FA_ERR_INVALID_ARG;
  if (B < 1 || num_pages < 1 || max_pages < 1 || max_tokens < 1) return FA_ERR_INVALID_ARG;
  if (!page_ok(page_size) || B > FA_KV4_MAX_BATCH) return FA_ERR_UNSUPPORTED;
  // Slots, ring positions and token counts stay within int.
  if (static_cast<long long>(num_pages) * page_size > 0x7fffffffLL || num_pages > (1 << 30) ||
      static_cast<long long>(max_pages) * page_size > 0x7fffffffLL || max_tokens > kMaxTokens)
    return FA_ERR_UNSUPPORTED;
  const void* words[] = {past_len, new_len, block_table, free_list, free_state,
                         kv_len,   cu_q,    slots,       state_out};
  for (const void* p : words)
    if (!aligned(p, 4)) return FA_ERR_INVALID_ARG;
  fa::ErrorWords err;
  const int st = fa::error_words(&err);
  if (st != FA_OK) return static_cast<fa_status>(st);
  fa::Kv4PlanArgs a{};
  a.past = past_len;
  a.fresh = new_len;
  a.B = B;
  a.page_shift = fa::kv4_layout(64, page_size, 32).page_shift;
  a.num_pages = num_pages;
  a.table = block_table;
  a.max_pages = max_pages;
  a.ring = free_list;
  a.ring_state = free_state;
  a.max_tokens = max_tokens;
  a.kv_len = kv_len;
  a.cu_q = cu_q;
  a.slots = slots;
  a.state_out = state_out;
  a.input_err = err.input;
  return launched(fa::launch_kv4_plan(a, stream));
}

fa_status fa_kv4_append(const void* K, const void* V, int T, int Hkv, int d, int k_token_stride,
                        int k_head_stride, int v_token_stride, int v_head_stride,
                        const int32_t* slots, void* cache, int num_pages, int page_size,
                        int group, fa_stream_t stream) {
  if (!K || !V || !slots || !cache || T < 1) return FA_ERR_INVALID_ARG;
  fa_status st = check_cache(num_pages, page_size, d, group, Hkv);
  if (st != FA_OK) return st;
  if (T > kMaxTokens) return FA_ERR_UNSUPPORTED;
  if (!strides_ok(k_token_stride, k_head_stride) || !strides_ok(v_token_stride, v_head_stride) ||
      !aligned(K, 16) || !aligned(V, 16) || !aligned(cache, 16) || !aligned(slots, 4))
    return FA_ERR_INVALID_ARG;
  fa::ErrorWords err;
  const int es = fa::error_words(&err);
  if (es != FA_OK) return static_cast<fa_status>(es);
  fa::Kv4RowsArgs a{};
  a.k_in = static_cast<const uint16_t*>(K);
  a.v_in = static_cast<const uint16_t*>(V);
  a.k_ts = k_token_stride;
  a.k_hs = k_head_stride;
  a.v_ts = v_token_stride;
  a.v_hs = v_head_stride;
  a.slots = slots;
  a.cache = static_cast<uint8_t*>(cache);
  a.lay = fa::kv4_layout(d, page_size, group);
  a.T = T;
  a.Hkv = Hkv;
  a.d = d;
  a.group = group;
  a.num_slots = num_pages * page_size;
  a.input_err = err.input;
  return launched(fa::launch_kv4_append(a, stream));
}

fa_status fa_kv4_gather(const int32_t* slots, const void* cache, int num_pages, int page_size,
                        int group, int T, int Hkv, int d, void* K, void* V, fa_stream_t stream) {
  if (!K || !V || !slots || !cache || T < 1) return FA_ERR_INVALID_ARG;
  fa_status st = check_cache(num_pages, page_size, d, group, Hkv);
  if (st != FA_OK) return st;
  if (T > kMaxTokens) return FA_ERR_UNSUPPORTED;
  if (!aligned(K, 16) || !aligned(V, 16) || !aligned(cache, 16) || !aligned(slots, 4))
    return FA_ERR_INVALID_ARG;
  fa::ErrorWords err;
  const int es = fa::error_words(&err);
  if (es != FA_OK) return static_cast<fa_status>(es);
  fa::Kv4RowsArgs a{};
  a.k_out = static_cast<uint16_t*>(K);
  a.v_out = static_cast<uint16_t*>(V);
  a.slots = slots;
  a.cache = static_cast<uint8_t*>(const_cast<void*>(cache));
  a.lay = fa::kv4_layout(d, page_size, group);
  a.T = T;
  a.Hkv = Hkv;
  a.d = d;
  a.group = group;
  a.num_slots = num_pages * page_size;
  a.input_err = err.input;
  return launched(fa::launch_kv4_gather(a, stream));
}

size_t fa_kv4_attn_workspace_bytes(int Hq, int Hkv, int d, int max_q) {
  if (Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || max_q < 1) return 0;
  if (d != 64 && d != 128 && d != 256) return 0;
  const long long rows = static_cast<long long>(max_q) * (Hq / Hkv);
  return fa::kv4_attn_workspace(d, rows > (1 << 30) ? (1 << 30) : static_cast<int>(rows));
}

size_t fa_kv4_attn_call_workspace_bytes(int B, int total_q, int max_q, int Hq, int Hkv, int d,
                                        int max_pages, int page_size, int window) {
  const size_t most = fa_kv4_attn_workspace_bytes(Hq, Hkv, d, max_q);
  if (most == 0 || B < 1 || total_q < 1 || max_pages < 1 || !page_ok(page_size) || window < -1 ||
      static_cast<long long>(max_q) * (Hq / Hkv) > 0x3fffffffLL)
    return most;  // (the call says what is wrong)
  return fa::kv4_attn_whole(d, max_q, Hq / Hkv, Hkv, B, total_q,
                            static_cast<long long>(max_pages) * page_size, window)
             ? 0
             : most;
}

fa_status fa_kv4_attn(const void* Q, const void* cache, const int32_t* block_table,
                      const int32_t* cu_q, const int32_t* kv_len, void* O, float* L, int B,
                      int total_q, int max_q, int Hq, int Hkv, int d, int q_token_stride,
                      int q_head_stride, int num_pages, int max_pages, int page_size, int group,
                      float scale, int causal, int window, void* workspace,
                      size_t workspace_bytes, fa_stream_t stream) {
  if (!Q || !cache || !block_table || !cu_q || !kv_len || !O || !L) return FA_ERR_INVALID_ARG;
  if (!workspace && workspace_bytes) return FA_ERR_INVALID_ARG;
  if (B < 1 || total_q < 1 || max_q < 1 || Hq < 1 || max_pages < 1) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(scale * kLog2e) || !(scale > 0.f) || window < -1) return FA_ERR_INVALID_ARG;
  fa_status st = check_cache(num_pages, page_size, d, group, Hkv);
  if (st != FA_OK) return st;
  if (Hq % Hkv != 0) return FA_ERR_INVALID_ARG;
  // Positions and row numbers stay within int.
  if (static_cast<long long>(max_pages) * page_size > 0x3fffffffLL || total_q > kMaxTokens ||
      static_cast<long long>(max_q) * (Hq / Hkv) > 0x3fffffffLL)
    return FA_ERR_UNSUPPORTED;
  if (!strides_ok(q_token_stride, q_head_stride) || !aligned(Q, 16) || !aligned(O, 16) ||
      !aligned(cache, 16) || !aligned(L, 4) || !aligned(block_table, 4) || !aligned(cu_q, 4) ||
      !aligned(kv_len, 4) || !aligned(workspace, 256) ||
      workspace_bytes <
          (workspace ? fa_kv4_attn_workspace_bytes(Hq, Hkv, d, max_q)
                     : fa_kv4_attn_call_workspace_bytes(B, total_q, max_q, Hq, Hkv, d, max_pages,
                                                        page_size, window)))
    return FA_ERR_INVALID_ARG;
  fa::ErrorWords err;
  const int es = fa::error_words(&err);
  if (es != FA_OK) return static_cast<fa_status>(es);
  fa::Kv4AttnArgs a{};
  a.Q = static_cast<const uint16_t*>(Q);
  a.cache = static_cast<const uint8_t*>(cache);
  a.table = block_table;
  a.cu_q = cu_q;
  a.kv_len = kv_len;
  a.O = static_cast<uint16_t*>(O);
  a.L = L;
  a.B = B;
  a.total_q = total_q;
  a.max_q = max_q;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.per_kv = Hq / Hkv;
  a.q_ts = q_token_stride;
  a.q_hs = q_head_stride;
  a.num_pages = num_pages;
  a.max_pages = max_pages;
  a.lay = fa::kv4_layout(d, page_size, group);
  a.scale_log2 = scale * kLog2e;
  a.causal = causal != 0;
  a.window = window;
  a.wait_err = err.wait;
  a.input_err = err.input;
  return launched(fa::launch_kv4_attn(d, group, a, workspace, stream));
}

}  // extern "C"
