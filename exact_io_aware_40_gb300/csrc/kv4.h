// kv4.h -- internal interface between the C-ABI layer of the paged 4-bit
// key/value cache (kv4_api.cu) and its kernels.  Not part of the public ABI.
#pragma once
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

namespace fa {

// Device addresses of the current device's error words: `wait` takes
// FA_ERR_TIMEOUT from kernels that gave up on a stalled pipeline (it also ends
// other kernels' waits), `input` FA_ERR_INVALID_ARG from kernels that met data
// outside its range (it ends nothing).  fa_check_error reads both.
struct ErrorWords {
  int* wait;
  int* input;
};
int error_words(ErrorWords* out);  // an fa_status

// Where the parts of a page's record are: K codes, K params, V codes, V params.
struct Kv4Layout {
  int page_shift;    // log2(page_size)
  int code_row;      // bytes of a token's codes: d / 2
  int param_row;     // bytes of a token's params: 4 * d / group
  int k_params;      // byte offsets inside the record
  int v_codes;
  int v_params;
  int record;        // bytes of a record
};
inline Kv4Layout kv4_layout(int d, int page_size, int group) {
  Kv4Layout l{};
  while ((1 << l.page_shift) < page_size) ++l.page_shift;
  l.code_row = d / 2;
  l.param_row = 4 * (d / group);
  l.k_params = page_size * l.code_row;
  l.v_codes = l.k_params + page_size * l.param_row;
  l.v_params = l.v_codes + page_size * l.code_row;
  l.record = l.v_params + page_size * l.param_row;
  return l;
}

struct Kv4PlanArgs {
  const int *past, *fresh;  // past_len, new_len
  int B, page_shift, num_pages;
  int* table;
  int max_pages;
  int* ring;
  const int* ring_state;
  int max_tokens;
  int *kv_len, *cu_q, *slots, *state_out;
  int* input_err;
};
cudaError_t launch_kv4_plan(const Kv4PlanArgs& a, cudaStream_t stream);

struct Kv4RowsArgs {
  const uint16_t *k_in, *v_in;   // append: bf16 rows
  int k_ts, k_hs, v_ts, v_hs;    // their strides, elements
  uint16_t *k_out, *v_out;       // gather: bf16 [T, Hkv, d]
  const int* slots;
  uint8_t* cache;
  Kv4Layout lay;
  int T, Hkv, d, group;
  int num_slots;                 // num_pages * page_size
  int* input_err;
};
cudaError_t launch_kv4_append(const Kv4RowsArgs& a, cudaStream_t stream);
cudaError_t launch_kv4_gather(const Kv4RowsArgs& a, cudaStream_t stream);

struct Kv4AttnArgs {
  const uint16_t* Q;
  const uint8_t* cache;
  const int *table, *cu_q, *kv_len;
  uint16_t* O;
  float* L;
  int B, total_q, max_q, Hq, Hkv, per_kv;  // per_kv = Hq / Hkv
  int q_ts, q_hs;
  int num_pages, max_pages;
  Kv4Layout lay;
  float scale_log2;  // scale * log2(e)
  int causal, window;
  int whole_items;   // items are not cut (kv4_sched.cuh)
  int lead;          // places an item takes in the list beside its tiles' (set by the launcher)
  int *wait_err, *input_err;
  // workspace: one Kv4Split per CTA, then per CTA two partial results of
  // `rows` query rows: statistics (m, l) and fp32 O
  int4* split;
  float2* part_stat;
  float* part_o;
};

// CTAs of a launch never exceed these, so that the workspace's size does not
// depend on the device.
constexpr int kKv4MaxCtas = 640;       // few query rows (kv4_attn.cu)
constexpr int kKv4MaxChunkCtas = 160;  // many (kv4_chunk.cu)
// Query rows of one CTA's block, given the most rows (queries x heads per K/V
// head) a request may have; 128 and more select the kernel for many.
int kv4_attn_rows(int d, int rows);
size_t kv4_attn_workspace(int d, int rows);
// Are a call's items left whole, so that nothing is merged?  `table` is the tokens
// a row of the block table can hold.
bool kv4_attn_whole(int d, int max_q, int per_kv, int Hkv, int B, int total_q, long long table, int window);
cudaError_t launch_kv4_attn(int d, int group, Kv4AttnArgs a, void* workspace, cudaStream_t stream);
// The kernel for many rows; *ctas: CTAs launched, for the merge that follows.
cudaError_t launch_kv4_chunk(int d, int group, const Kv4AttnArgs& a, cudaStream_t stream, int* ctas);

}  // namespace fa
