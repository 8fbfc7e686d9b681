// attn.cuh -- parameters and launchers of the GQE attention kernels.
#pragma once

#include "sm100.cuh"

namespace gqe {

typedef uint16_t gqe_bf16_t;

// Bits i of a 32-position word at position pos with pos + i < x.
__device__ __forceinline__ uint32_t bits_below(int x, int pos) {
  const int n = min(max(x - pos, 0), 32);
  return n == 32 ? 0xFFFFFFFFu : (1u << n) - 1u;
}

struct AttnParams {
  gqe_bf16_t* o_routed;   // [B, G, T, k, d]
  gqe_bf16_t* o_sh;       // [B, T, d]
  float* lse;             // optional
  int B, T, G, k, n_shared, sg;
  float scale_log2;       // scale * log2(e)
  unsigned* err;          // device error word
  int window, sinks;      // windowed launches only: 1 <= window <= T, 0 <= sinks <= T
};

// diag.cu: a bounded wait that runs out (failure-path test)
cudaError_t launch_debug_wait(unsigned* err, cudaStream_t stream);
cudaError_t launch_debug_wait_short(unsigned* err, cudaStream_t stream);

cudaError_t launch_attn_prefill(const CUtensorMap& mQ, const CUtensorMap& mQs, const CUtensorMap& mK,
                                const CUtensorMap& mV, const AttnParams& p, int d,
                                cudaStream_t stream);
// The same attention under a sliding window with sinks (p.window, p.sinks);
// the K and V maps' boxes hold kWindowKeyTile rows.
constexpr int kWindowKeyTile = 64;
cudaError_t launch_attn_prefill_window(const CUtensorMap& mQ, const CUtensorMap& mQs, const CUtensorMap& mK,
                                       const CUtensorMap& mV, const AttnParams& p, int d, cudaStream_t stream);

struct DecodeParams {
  const gqe_bf16_t* q_routed;   // [B, G, k, d]
  const gqe_bf16_t* q_sh;       // [B, d]
  const gqe_bf16_t* Kc;         // [B, G, L_max, d]
  const gqe_bf16_t* Vc;
  const int* cache_len;         // [B]
  gqe_bf16_t* o_routed;         // [B, G, k, d]
  gqe_bf16_t* o_sh;             // [B, d]
  float* part;                  // [B, G, n_chunks, nq_max, d + 2]
  int B, G, k, d, n_shared, sg, L_max;
  int chunk;                    // keys per split
  int n_chunks;
  int nq_max;                   // k + n_shared
  float scale_log2;
  unsigned* err;                // device error word
};

// Backward of the prefill attention.  Query rows live in a padded row space:
// routed sequence s (= b*G + g) owns rows [s*rows_pad, (s+1)*rows_pad), the
// shared head of sequence b owns B*G*rows_pad + [b*rows_pad_sh, ...); rows
// past a sequence's T*k (or T) are padding.
struct AttnBwdParams {
  const float* lse;                 // forward LSE (natural log), routed rows then shared rows
  const gqe_bf16_t* o_routed;       // [B, G, T, k, d]
  const gqe_bf16_t* o_sh;           // [B, T, d]
  const gqe_bf16_t* do_routed;
  const gqe_bf16_t* do_sh;
  float* lse2;                      // [n_rows_pad] LSE * log2(e), +inf on padding (windowed: negated)
  float* delta;                     // [n_rows_pad] sum_c dO * O (windowed: negated)
  float* dq_acc;                    // [n_rows_pad, d] fp32
  gqe_bf16_t* dq_routed;            // [B, G, T, k, d]
  gqe_bf16_t* dq_sh;                // [B, T, d]
  gqe_bf16_t* dK;                   // [B, G, T, d]
  gqe_bf16_t* dV;
  int B, T, G, k, n_shared, sg, d;
  int rows_pad, rows_pad_sh;
  long long n_rows_pad;
  float scale, scale_log2;
  unsigned* err;
  // windowed launches only: 1 <= window <= T, 0 <= sinks <= T
  int window, sinks;
  const gqe_bf16_t* q_routed;       // the forward's inputs (rows that see few keys)
  const gqe_bf16_t* q_sh;
  const gqe_bf16_t* K;
  const gqe_bf16_t* V;
  float* part;                      // cut walks' sums: [2 * stretches, 2 (dK, dV), 128, d] fp32
};

struct AttnBwdLayout {
  int rows_pad, rows_pad_sh;
  long long n_rows_pad;
  size_t off_lse2, off_delta, off_dq, bytes;
};


// Windowed backward (attn_bwd_window.cu): the list of (sequence, key tile, query
// tile of its walk) cut into n_rounds * n_ctas equal stretches; CTA c runs
// stretches c, n_ctas + c, 2 n_ctas + c, ...
constexpr int kBwdWindowCtas = 148, kBwdWindowRounds = 4;
struct AttnBwdSchedule {
  int n_ctas, n_rounds;
  int seq[kBwdWindowCtas * kBwdWindowRounds];      // where each stretch starts
  int jt[kBwdWindowCtas * kBwdWindowRounds];
  int off[kBwdWindowCtas * kBwdWindowRounds];
  int count[kBwdWindowCtas * kBwdWindowRounds];    // its query tiles
};
// The schedule, the bytes of scratch (attn_bwd_layout's, then the cut walks'
// sums) and where the sums lie.
void attn_bwd_window_plan(int B, int T, int G, int k, int n_shared, int sg, int d, int window, int sinks,
                          AttnBwdSchedule* S, size_t* off_part, size_t* bytes);
cudaError_t launch_attn_bwd_window(const CUtensorMap& mQ, const CUtensorMap& mQs, const CUtensorMap& mdO,
                                   const CUtensorMap& mdOs, const CUtensorMap& mK, const CUtensorMap& mV,
                                   const CUtensorMap& mdQ, const AttnBwdParams& p, const AttnBwdSchedule& S,
                                   cudaStream_t stream);

void attn_bwd_layout(int B, int T, int G, int k, int n_shared, int d, AttnBwdLayout* L);
cudaError_t launch_attn_bwd(const CUtensorMap& mQ, const CUtensorMap& mQs, const CUtensorMap& mdO,
                            const CUtensorMap& mdOs, const CUtensorMap& mK, const CUtensorMap& mV,
                            const CUtensorMap& mdQ, const AttnBwdParams& p, cudaStream_t stream);

// Attention of a few tokens per sequence against a dense cache (attn_cache.cu):
// a tree of drafted tokens, or one new token under a window.
constexpr int kMaxTree = 128;     // drafted tokens per sequence at most

struct CacheAttnParams {
  const gqe_bf16_t* q_routed;   // [B, G, T, k, d]
  const gqe_bf16_t* q_sh;       // [B, T, d]
  gqe_bf16_t* o_routed;
  gqe_bf16_t* o_sh;
  const int* cache_len;         // [B] cache rows of each sequence
  const int* parent;            // [B, T] (tree)
  const int* tree_len;          // [B] drafted tokens of each sequence, or null: T (tree)
  int B, T, G, k, n_shared, sg, L_max;
  int tree;                     // 1: T drafted tokens behind the cache; 0: the cache's last row is the token itself
  int window, sinks;            // window 0: unlimited
  int n_qt, n_split;            // query tiles per (b, g); shares (CTAs of a cluster) per query tile
  float scale_log2;
  unsigned* err;
};

struct CacheAttnPlan {
  int n_qt, n_split;
  long long items;              // CTAs: B * G * n_qt * n_split
};

void cache_attn_plan(int B, int T, int G, int k, int n_shared, int d, int L_max, bool tree, int window, int sinks,
                     CacheAttnPlan* P);
// Key rows per box of the K and V maps.
constexpr int cache_attn_key_tile(int d) { return d == 64 ? 128 : 64; }
cudaError_t launch_attn_cache(const CUtensorMap& mK, const CUtensorMap& mV, const CUtensorMap& mKt,
                              const CUtensorMap& mVt, const CacheAttnParams& p, int d, long long items,
                              cudaStream_t stream);

struct CommitParams {
  const gqe_bf16_t* Kt;         // [B, G, T, d]
  const gqe_bf16_t* Vt;
  const int* path;              // [B, T]
  const int* n_accept;          // [B]
  gqe_bf16_t* Kc;               // [B, G, L_max, d]
  gqe_bf16_t* Vc;
  const int* cache_len;         // [B]
  int* new_len;                 // [B], may be cache_len
  int B, T, G, d, L_max;
  unsigned* err;
};
cudaError_t launch_cache_commit(const CommitParams& p, cudaStream_t stream);

size_t decode_workspace_bytes(int B, int G, int k, int d, int n_shared, int L_max);
cudaError_t launch_attn_decode_maps(const CUtensorMap& mK, const CUtensorMap& mV, const DecodeParams& p,
                                   cudaStream_t stream);
void decode_split_plan(int L_max, int* chunk, int* n_chunks);

}  // namespace gqe
