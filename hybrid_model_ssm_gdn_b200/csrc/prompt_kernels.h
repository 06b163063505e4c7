// prompt_kernels.h -- launches of the kernels around the decode step: prompts, short convolution, draft verification.
#pragma once

#include "kernels.h"
#include "prompts.cuh"

namespace rssm {

// Mamba-2 scan over packed prompts
constexpr int kScanChunk = 128;      // tokens of a chunk on the tensor cores
struct ScanArgs {
  int H, P, G;
  int piece_len;                    // tokens of a piece (total + 1: every prompt is one piece)
  const void *x, *Bin, *C, *dt;     // [total][H][P], [total][G][128] x2, [total][H]
  const float *A, *D;
  float *S;                         // [nslots][H][P][128]
  float *y;                         // [total][H][P]
  void *work;                       // piece states, where prompts are cut (piece_len <= total)
  int *err;                         // error word, may be null
  long long wait_cycles;            // bound of the tensor-core kernel's waits
  int withhold;                     // test hook: no block loads X of this chunk (-1: off)
};
// short prompts: bf16 inputs, prompts not cut
cudaError_t launch_scan_mma(const ScanArgs &a, const Prompts &pr, cudaStream_t stream);
// long prompts: bf16 inputs, total > 0
cudaError_t launch_scan_tc(const ScanArgs &a, const Prompts &pr, cudaStream_t stream);
size_t scan_tc_workspace(int H, int P, int pieces, size_t *seg_dt);
// fp32 inputs, prompts not cut
cudaError_t launch_scan(const ScanArgs &a, const Prompts &pr, int num_sms, cudaStream_t stream);
// NaN in the output rows of refused prompts
cudaError_t launch_refuse(const Prompts &pr, float *y, int row, int num_sms, cudaStream_t stream);
cudaError_t launch_prefill_meta(const Prompts &pr, const int4 *meta_in, int4 *meta_out, unsigned char *skip, int H,
                                int *err, cudaStream_t stream);

// Gated delta rule over packed prompts
constexpr int kGdnChunk = 64;        // tokens of a chunk on the tensor cores
struct GdnScanArgs {
  int H, Hk, R;                     // heads of v; of q and k (Hk divides H); rows of a head's state (d_v)
  int by_prompt;                    // S is indexed by prompt instead of by slot
  float q_scale;
  const void *q, *k, *v;            // [total][Hk][128] x2, [total][H][R]
  const float *alpha, *beta;        // [total][H]
  float *S;                         // [nslots or nseq][H][R][128]
  float *y;                         // [total][H][R]
  int *err;                         // error word, may be null
  long long wait_cycles;            // bound of the tensor-core kernel's waits
  int withhold;                     // test hook: no block loads v of this chunk (-1: off)
};
// token by token: fp32 inputs, prompts of a few tokens
cudaError_t launch_gdn_scan(const GdnScanArgs &a, const Prompts &pr, int esz, int num_sms, cudaStream_t stream);
// chunks on the tensor cores: bf16 inputs, total > 0
cudaError_t launch_gdn_tc(const GdnScanArgs &a, const Prompts &pr, int num_sms, cudaStream_t stream);
// states of packed prompts [nseq][H][rows][128] from and to a GDN context's stored formats
struct PromptStateArgs {
  int H, rows, hp_mode, read_mode;
  float *states;
  void *hp;
  float *hs;
  unsigned char *rq, *rs;
  float *rg;
  unsigned char *rc;
  unsigned long long seed;
};
cudaError_t launch_prompt_states(const PromptStateArgs &a, const Prompts &pr, bool store, cudaStream_t stream);

// short causal convolution
struct ShortConvArgs {
  int batch, channels, width, ring, silu;
  int split[3];
  const void *weight, *bias;        // [channels][width], [channels] or null
  void *hist;                       // [batch][ring][channels]
  const int *cur;                   // [batch]
  int *cur_out;                     // the same array where a call advances it
  const void *in;
  long long in_stride;
  void *out[3];
};
cudaError_t launch_shortconv_prompt(const ShortConvArgs &a, const Prompts &pr, int esz, int num_sms,
                                    cudaStream_t stream);
cudaError_t launch_shortconv_tokens(const ShortConvArgs &a, int T, int advance, int esz, int num_sms,
                                    cudaStream_t stream);
cudaError_t launch_shortconv_commit(int *cur, const int *accepted, int batch, int ring, int most, cudaStream_t stream);

// draft verification
constexpr int kMaxAccept = 16;
struct AcceptArgs {
  int batch, T, vocab;
  const float *target, *draft;      // rows (b, j) at (b (T+1) + j) ld_target, (b T + j) ld_draft; draft may be null
  long long ld_target, ld_draft;
  const int *tokens, *count;        // [batch][T]; [batch] or null
  const float *u;                   // [batch][T+1]
  int *accepted, *committed, *next; // [batch]; committed may be null
};
cudaError_t launch_accept(const AcceptArgs &a, int num_sms, cudaStream_t stream);

}  // namespace rssm
