// What the host side of the training operators (muon_ops.cpp) shares with their
// kernels and with muon_api.cpp.  Each launcher returns hipError_t as int; its
// arguments have been checked.
#pragma once
#include <stddef.h>
#include <stdint.h>

#include "muon.h"

namespace muon {

// Host helpers of muon_api.cpp: keep the HIP error text for
// muon_status_string (returns MUON_EHIP); whether MUON_DEBUG is set; whether
// `stream` (a hipStream_t) can belong to device `dev`.
int host_hip_fail(int hip_error, const char* what);
bool host_debug();
bool host_stream_on_device(void* stream, int dev);

// muon_act8.hip
int launch_act8_pack(const void* x, int64_t ld_x, int32_t dtype, int64_t rows, int64_t cols,
                     const muon_act8_t& out, void* stream);
int launch_act8_unpack(const muon_act8_t& in, int64_t rows, int64_t cols, void* out, int64_t ld_out,
                       int32_t dtype, void* stream);
int launch_swiglu(const muon_swiglu_t& op, void* stream);
int launch_swiglu_grad(const muon_swiglu_grad_t& op, void* stream);

// muon_norm.hip
int launch_rmsnorm(const muon_rmsnorm_t& op, void* stream);
// blocks of the backward pass, each with its own partial dgain (one: none needed)
int64_t rmsnorm_grad_blocks(int64_t rows, int64_t cols);
int launch_rmsnorm_grad(const muon_rmsnorm_grad_t& op, float* partial, void* stream);
int launch_rmsnorm_dgain(const float* partial, int64_t blocks, int64_t cols, float* dgain, void* stream);

// muon_wgrad.hip
// Workspace: the token ranges' partial outputs where there are several, and
// aligned copies of a dy or x8 that the kernel's loads cannot take as they are.
struct WgradPlan {
  int tn, tk;                 // output tile: 256 x 256, 256 x 128 or 128 x 128
  int64_t tiles_n, tiles_k;   // output tiles
  int64_t whole;              // tiles (the first ones) that one block makes from all tokens
  int64_t splits, split_rows; // token ranges of the others, of split_rows (the last may be shorter)
  bool copy_dy, copy_x;
  size_t partial_off, dy_off, x_off, s_off;
  size_t bytes;
};
WgradPlan wgrad_plan(const muon_act8_wgrad_t& op);
int launch_wgrad_copy(muon_act8_wgrad_t& op, const WgradPlan& p, char* ws, void* stream);   // op: now the copies
int launch_wgrad(const muon_act8_wgrad_t& op, const WgradPlan& p, char* ws, void* stream);
int launch_wgrad_join(const muon_act8_wgrad_t& op, const WgradPlan& p, const char* ws, void* stream);

// muon_embed.hip
// Workspace of the gradient (nothing for few tokens, which are not sorted):
// keys and tokens before and after a pass, each block's digit counts, each
// row's first place, the sums of the long runs' pieces.
struct EmbedSortPlan {
  int passes;                 // digits of the keys 0 .. vocab (0: not sorted)
  int log_buckets;            // sorted in one launch, by the low bits of the ids (0: digit by digit)
  uint32_t highs;             // values of the other bits
  int64_t blocks;             // blocks of a pass, block_tokens tokens each
  int64_t block_tokens;
  int64_t chunks;             // pieces of long runs lie in one chunk
  size_t keys_off[2], toks_off[2], count_off, start_off, pieces_off;
  size_t bytes;
  // after the last pass
  uint32_t* keys(char* ws) const { return reinterpret_cast<uint32_t*>(ws + keys_off[(passes - 1) & 1]); }
  uint32_t* toks(char* ws) const { return reinterpret_cast<uint32_t*>(ws + toks_off[(passes - 1) & 1]); }
  uint32_t* starts(char* ws) const { return reinterpret_cast<uint32_t*>(ws + start_off); }
  float* pieces(char* ws) const { return reinterpret_cast<float*>(ws + pieces_off); }
};
EmbedSortPlan embed_sort_plan(int64_t tokens, int64_t vocab, int64_t cols);
int launch_embed(const muon_embed_t& op, void* stream);
int launch_embed_buckets(const muon_embed_grad_t& op, const EmbedSortPlan& p, char* ws, void* stream);
int launch_embed_count(const muon_embed_grad_t& op, const EmbedSortPlan& p, int pass, char* ws, void* stream);
int launch_embed_scatter(const muon_embed_grad_t& op, const EmbedSortPlan& p, int pass, char* ws, void* stream);
int launch_embed_starts(const muon_embed_grad_t& op, const EmbedSortPlan& p, char* ws, void* stream);
int launch_embed_sums(const muon_embed_grad_t& op, const EmbedSortPlan& p, char* ws, void* stream);
int launch_embed_join(const muon_embed_grad_t& op, const EmbedSortPlan& p, char* ws, void* stream);

}  // namespace muon
