// Host-side declarations shared by the C-ABI layer (api.cu) and the kernel
// translation units.  Not part of the public interface.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "device_common.cuh"

struct dustin_kv;

namespace dustin {

// Everything the kernels need of dustin_kv4 (strides in bytes).
struct Kv4View {
  const uint8_t* data;
  long long sb, sh, sn;
  const int* page_table;
  int page_size, pages_per_seq, num_pages;
  int k_exp, v_exp;
};

// ---- scoring
constexpr int kMaxPairs = 64;

struct ScorePair {
  KvView kv;
  int kv_head;
};

struct ScoreArgs {
  const __nv_bfloat16* q;  // [n_pairs][b][rows][d]
  float* s_out;            // [b][n]
  float* logits;           // workspace [n_pairs][rows][b][n], log2 units
  float2* stats;           // workspace [n_pairs][rows][b][nchunks]
  int b, n, n_pairs, rows;
  int chunk, nchunks;
  float scale_log2;
  int keys_shared;         // two pairs read the same keys (same cache, kv head)
  ScorePair pairs[kMaxPairs];
};

int score_chunk();
int check_score_args(int b, int n, int d, int n_pairs, int rows, const void* q,
                     const ::dustin_kv* kv, const int32_t* kv_head, float scale,
                     const float* s_out, const char* what, bool* paged, bool* empty);
cudaError_t launch_score(const ScoreArgs& a, int d, bool paged, cudaStream_t st);
cudaError_t take_score_flags(unsigned* flags);

// ---- Quest page scoring (baseline selector)
struct QuestArgs {
  KvView kv;                     // keys (stats pass)
  __nv_bfloat16* stats;          // [b][hkv][P][2][d] out (stats pass)
  const __nv_bfloat16* stats_in; // the same, in (score pass)
  const __nv_bfloat16* q;        // [b][hq][d] (score pass)
  float* scores;                 // [b][hq][P] (score pass)
  int b, hq, hkv, n, page, n_pages;
};
cudaError_t launch_quest_stats(const QuestArgs& a, int d, bool paged, cudaStream_t st);
cudaError_t launch_quest_scores(const QuestArgs& a, int d, cudaStream_t st);
cudaError_t take_quest_flags(unsigned* flags);

// ---- selection
struct SelectArgs {
  const float* sd;
  const float* st;
  int32_t* idx;
  double alpha;
  int b, n, k, n_sink, n_recent, m, norm;
};
constexpr int kSelectMaxN = 1 << 20;
cudaError_t launch_select(const SelectArgs& a, cudaStream_t st);

// ---- verification attention (AttnArgs in attn.cuh, AttnSkArgs in
// attn_streamk.cuh)
struct AttnArgs;
struct AttnSkArgs;
cudaError_t launch_attn_sparse(const AttnArgs& a, int d, int mt, bool paged,
                               cudaStream_t st);
cudaError_t launch_attn_dense(const AttnSkArgs& a, int d, int mt, bool paged,
                              cudaStream_t st);
struct AttnMlArgs;
cudaError_t launch_attn_ml(const AttnMlArgs& a, int d, int mt, bool paged, int grid,
                           cudaStream_t st);
cudaError_t take_attn_ml_flags(unsigned* flags);
int occupancy_attn_sparse(int d, int mt);
int occupancy_attn_dense(int d, int mt);
cudaError_t take_attn_sparse_flags(unsigned* flags);
cudaError_t take_attn_dense_flags(unsigned* flags);

// ---- attention of a batch that shares prefixes
struct PrefixArgs {
  const __nv_bfloat16* q;   // [b][h_q][w][d]
  __nv_bfloat16* o;
  float* lse;
  KvView prefix, own, win;
  const int* prefix_len;    // [groups] or null
  const int* own_len;       // [b] or null
  int b, groups, hq, hkv, d, w, n_prefix, n_own, has_win;
  float scale_log2;
};
size_t prefix_workspace(const PrefixArgs& p, int sms);
cudaError_t launch_attn_prefix(const PrefixArgs& p, int sms, void* ws, cudaStream_t st);
cudaError_t take_prefix_flags(unsigned* flags);

// ---- verification of drafted tokens
struct TokenArgs {
  const void* p;                 // target rows, fp32 or bf16
  const void* q;                 // draft rows of the same type (may be null)
  long long stride_tb, stride_tw, stride_db, stride_dw;
  const int* draft;              // [b][w - 1]
  const int* n_draft;            // [b] or null
  const float* u_accept;         // [b][w - 1]
  const float* u_sample;         // [b]
  int* tokens;                   // [b][w]
  int* n_accepted;               // [b]
  int b, w, vocab;
};
cudaError_t launch_tokens(const TokenArgs& a, bool bf16, int sms, cudaStream_t st);
cudaError_t take_tokens_flags(unsigned* flags);

// ---- cache compaction and shared pages
constexpr int kCompactMaxLayers = 128;   // per launch (kernel parameter space)
struct CompactArgs {
  const int* idx;      // [b][k]
  const int* k_len;    // [b] or null
  int layers, b, hkv, n, k, in_place, splits;
  struct { KvView src, dst; } layer[kCompactMaxLayers];
};
struct ForkArgs {
  const int* parent;   // [n_forks]
  const int* child;
  int* page_table;     // [n_seqs][pages_per_seq]
  int* seq_len;        // [n_seqs]
  int* refcount;       // [num_pages]
  int n_seqs, pages_per_seq, page_size, num_pages, n_forks;
};
constexpr int kResizeMaxList = 1024;
constexpr int kResizeMaxPages = 1 << 22;
struct ResizeArgs {
  const int* seqs;     // [n_list]
  const int* new_len;  // [n_list] or null (zeros)
  int* page_table;
  int* seq_len;
  int* refcount;
  int* copies;         // [n_list][2]
  int n_seqs, pages_per_seq, page_size, num_pages, n_list;
};
struct CopyArgs {
  const int* copies;
  int layers, hkv;
  KvView kv[kCompactMaxLayers];
};
cudaError_t launch_compact(const CompactArgs& a, int d, int sms, cudaStream_t st);
cudaError_t launch_fork(const ForkArgs& a, cudaStream_t st);
cudaError_t launch_resize(const ResizeArgs& a, cudaStream_t st);
cudaError_t launch_copy_pages(const CopyArgs& a, int n_list, int d, cudaStream_t st);
cudaError_t take_pages_flags(unsigned* flags);

// ---- a cache held in 4 bits
constexpr int kKv4MaxLayers = 128;       // per launch (kernel parameter space)
struct Kv4Args {
  const int* start;    // [b] or null: position of row 0 (writing)
  const int* idx;      // [b][rows] or null: position of each row (reading)
  const int* lens;     // [b] or null: rows of each sequence
  int layers, hkv, n, rows;
  unsigned count;      // records per layer: b * hkv * rows
  struct { KvView rows; Kv4View cache; } layer[kKv4MaxLayers];
};
cudaError_t launch_kv4_write(const Kv4Args& a, int d, cudaStream_t st);
cudaError_t launch_kv4_read(const Kv4Args& a, int d, cudaStream_t st);
cudaError_t take_kv4_flags(unsigned* flags);

// ---- attention over a 4-bit cache
struct Kv4AttnArgs {
  const __nv_bfloat16* q;   // [b][h_q][w][d]
  __nv_bfloat16* o;
  float* lse;
  Kv4View kv;
  KvView win;
  const int* idx;           // [b][k] or null
  const int* k_len;         // [b] or null
  int b, hq, hkv, d, w, n, k, has_win;
  float scale;
};
size_t attn_kv4_workspace(const Kv4AttnArgs& a, int sms);
cudaError_t launch_attn_kv4(const Kv4AttnArgs& a, int sms, void* ws, cudaStream_t st);
cudaError_t take_attn_kv4_flags(unsigned* flags);

// ---- log probabilities
constexpr int kLogprobsMaxTop = 64;
constexpr int kLogprobsMaxTokens = 512;
struct LogprobArgs {
  const void* x;       // [b][w][vocab], fp32 or bf16
  long long stride_b, stride_w;
  const int* n_rows;   // [b] or null
  const int* tokens;   // [b][w][m]
  float* logprobs;     // [b][w][m]
  float* entropy;      // [b][w] or null
  float* lse;          // [b][w] or null
  int* top_ids;        // [b][w][top]
  float* top_logprobs;
  int b, w, vocab, m, top;
  float scale;
};
cudaError_t launch_logprobs(const LogprobArgs& a, bool bf16, int sms, cudaStream_t st);
cudaError_t take_logprobs_flags(unsigned* flags);

// ---- bookkeeping (api.cu)
void note_launches(int count);
int record_error(int status, const char* message);  // sets dustin_last_error()

}  // namespace dustin
