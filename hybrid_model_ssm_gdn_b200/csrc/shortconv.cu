// shortconv.cu -- the short causal convolution in front of a layer's inputs, for prompts and for decoding.
//
//   out[t][c] = act(bias[c] + sum_k w[c][k] in[t - (K-1) + k][c]),  K = 2..4
//
// A few multiply-adds per value against one read and one write of it: the bound is memory.  A thread owns 8
// consecutive channels (16 bytes of bf16), keeps their K taps and the last K-1 inputs in registers as fp32 and walks
// along the tokens, so every input is loaded once (plus K-1 rows where a prompt is cut into tiles).
#include "kernels.h"

namespace rssm {

namespace {

constexpr int kTile = 32;         // tokens of a prompt tile: K-1 = 3 rows read twice in 32 is 9%, served by L2
constexpr int kPromptThreads = 128;

template <typename TI>
__device__ __forceinline__ void store8(TI *p, const float (&v)[8]);
template <>
__device__ __forceinline__ void store8<float>(float *p, const float (&v)[8]) {
  *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16 *p, const float (&v)[8]) {
  uint4 u;
  uint32_t *w = reinterpret_cast<uint32_t *>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  *reinterpret_cast<uint4 *>(p) = u;
}

// the taps and bias of 8 channels from c
template <typename TI, int K>
struct Filter {
  float w[K][8], b[8];
  bool silu;
  __device__ __forceinline__ void load(const ShortConvArgs &a, int c) {
    const TI *wp = reinterpret_cast<const TI *>(a.weight) + (size_t)c * K;
    float flat[8 * K];
#pragma unroll
    for (int i = 0; i < K; ++i) {
      float v[8];
      load8(wp + 8 * i, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) flat[8 * i + j] = v[j];
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) w[k][j] = flat[j * K + k];
#pragma unroll
    for (int j = 0; j < 8; ++j) b[j] = 0.f;
    if (a.bias) load8(reinterpret_cast<const TI *>(a.bias) + c, b);
    silu = a.silu;
  }
  // v / (1 + exp(-v)); where exp overflows the quotient is -0
  __device__ __forceinline__ float act(float v) const { return silu ? v / (1.f + expf(-v)) : v; }
  __device__ __forceinline__ void apply(const float (&win)[K - 1][8], const float (&x)[8], float (&o)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float v = b[j];
#pragma unroll
      for (int k = 0; k < K - 1; ++k) v = fmaf(w[k][j], win[k][j], v);
      o[j] = act(fmaf(w[K - 1][j], x[j], v));
    }
  }
};

template <int K>
__device__ __forceinline__ void push(float (&win)[K - 1][8], const float (&x)[8]) {
#pragma unroll
  for (int k = 0; k + 2 < K; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) win[k][j] = win[k + 1][j];
#pragma unroll
  for (int j = 0; j < 8; ++j) win[K - 2][j] = x[j];
}

__device__ __forceinline__ int wrap(int v, int ring) {
  v %= ring;
  return v < 0 ? v + ring : v;
}

// where the channels from c go: the output that holds them, its row length and the offset in a row
template <typename TI>
__device__ __forceinline__ TI *split_out(const ShortConvArgs &a, int c, int &row) {
  int s = 0, c0 = 0;
  if (c >= a.split[0]) { c0 = a.split[0]; s = 1; }
  if (s == 1 && c >= c0 + a.split[1]) { c0 += a.split[1]; s = 2; }
  row = a.split[s];
  return reinterpret_cast<TI *>(a.out[s]) + (c - c0);
}

// Prompts.  blockIdx.x: tile of a prompt; blockIdx.y: block of channels.  The block of a prompt's first tile alone
// reads and rewrites the sequence's history, each thread its own channels, so the rewrite is safe in place.
template <typename TI, int K>
__global__ void __launch_bounds__(kPromptThreads) prompt_kernel(ShortConvArgs a, Prompts pr) {
  __shared__ int found;
  Piece pc;
  if (!find_piece(pr, blockIdx.x, kTile, pc, &found)) return;
  const int c = (blockIdx.y * kPromptThreads + threadIdx.x) * 8;
  const int len = pc.end - pc.begin;
  if (c >= a.channels || (pc.first >= len && pc.index > 0)) return;
  Filter<TI, K> f;
  f.load(a, c);
  const TI *in = reinterpret_cast<const TI *>(a.in) + (size_t)pc.begin * a.in_stride + c;
  float win[K - 1][8];
  TI *hist = reinterpret_cast<TI *>(a.hist) + (size_t)pc.slot * a.ring * a.channels + c;
  if (pc.index == 0) {
    const int cur = wrap(a.cur[pc.slot], a.ring);
    float held[K - 1][8];
#pragma unroll
    for (int k = 0; k < K - 1; ++k) {
#pragma unroll
      for (int j = 0; j < 8; ++j) held[k][j] = 0.f;
      if (pc.resume) load8(hist + (size_t)wrap(cur - (K - 1) + k, a.ring) * a.channels, held[k]);
    }
    if (len > 0 || !pc.resume) {
#pragma unroll
      for (int k = 0; k < K - 1; ++k) {  // newest K-1 of (held, prompt)
        const int t = len - (K - 1) + k;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.f;
        if (t >= 0) {
          load8(in + (size_t)t * a.in_stride, v);
        } else {
#pragma unroll
          for (int m = 0; m < K - 1; ++m)
            if (m == K - 1 + t)
#pragma unroll
              for (int j = 0; j < 8; ++j) v[j] = held[m][j];
        }
        store8<TI>(hist + (size_t)wrap(cur - (K - 1) + k, a.ring) * a.channels, v);
      }
    }
#pragma unroll
    for (int k = 0; k < K - 1; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) win[k][j] = held[k][j];
  } else {
#pragma unroll
    for (int k = 0; k < K - 1; ++k) load8(in + (size_t)(pc.first - (K - 1) + k) * a.in_stride, win[k]);
  }
  int row;
  TI *out = split_out<TI>(a, c, row) + (size_t)(pc.begin + pc.first) * row;
  const int n = min(kTile, len - pc.first);
  in += (size_t)pc.first * a.in_stride;
  for (int t = 0; t < n; ++t) {
    float x[8], o[8];
    load8(in + (size_t)t * a.in_stride, x);
    f.apply(win, x, o);
    push<K>(win, x);
    store8<TI>(out + (size_t)t * row, o);
  }
}

// T tokens a sequence on top of its history.  One block a sequence, so that the cursor can advance in place once
// every thread has read it (`advance`: one token that stands; otherwise the rows stay tentative).
template <typename TI, int K>
__global__ void __launch_bounds__(1024) token_kernel(ShortConvArgs a, int T, int advance) {
  const int b = blockIdx.x;
  const int cur = wrap(a.cur[b], a.ring);
  for (int c = threadIdx.x * 8; c < a.channels; c += blockDim.x * 8) {
    Filter<TI, K> f;
    f.load(a, c);
    TI *hist = reinterpret_cast<TI *>(a.hist) + (size_t)b * a.ring * a.channels + c;
    const TI *in = reinterpret_cast<const TI *>(a.in) + (size_t)b * T * a.in_stride + c;
    float win[K - 1][8];
#pragma unroll
    for (int k = 0; k < K - 1; ++k) load8(hist + (size_t)wrap(cur - (K - 1) + k, a.ring) * a.channels, win[k]);
    int row;
    TI *out = split_out<TI>(a, c, row) + (size_t)b * T * row;
    for (int t = 0; t < T; ++t) {
      float x[8], o[8];
      load8(in + (size_t)t * a.in_stride, x);
      f.apply(win, x, o);
      push<K>(win, x);
      store8<TI>(hist + (size_t)wrap(cur + t, a.ring) * a.channels, x);
      store8<TI>(out + (size_t)t * row, o);
    }
  }
  if (advance) {
    __syncthreads();
    if (threadIdx.x == 0) a.cur_out[b] = wrap(cur + 1, a.ring);
  }
}

__global__ void commit_kernel(int *cur, const int *accepted, int batch, int ring, int most) {
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= batch) return;
  const int acc = max(0, min(most, accepted[b]));
  cur[b] = wrap(wrap(cur[b], ring) + acc, ring);
}

template <typename TI>
cudaError_t launch_prompt(const ShortConvArgs &a, const Prompts &pr, cudaStream_t stream) {
  const dim3 grid(prompt_pieces(pr.total, pr.nseq, kTile), (a.channels / 8 + kPromptThreads - 1) / kPromptThreads);
  if (a.width == 2) prompt_kernel<TI, 2><<<grid, kPromptThreads, 0, stream>>>(a, pr);
  else if (a.width == 3) prompt_kernel<TI, 3><<<grid, kPromptThreads, 0, stream>>>(a, pr);
  else prompt_kernel<TI, 4><<<grid, kPromptThreads, 0, stream>>>(a, pr);
  return cudaGetLastError();
}

template <typename TI>
cudaError_t launch_tokens(const ShortConvArgs &a, int T, int advance, cudaStream_t stream) {
  int threads = (a.channels / 8 + 31) / 32 * 32;
  threads = threads > 256 ? 256 : threads;
  if (a.width == 2) token_kernel<TI, 2><<<a.batch, threads, 0, stream>>>(a, T, advance);
  else if (a.width == 3) token_kernel<TI, 3><<<a.batch, threads, 0, stream>>>(a, T, advance);
  else token_kernel<TI, 4><<<a.batch, threads, 0, stream>>>(a, T, advance);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_shortconv_prompt(const ShortConvArgs &a, const Prompts &pr, int esz, cudaStream_t stream) {
  return esz == 2 ? launch_prompt<__nv_bfloat16>(a, pr, stream) : launch_prompt<float>(a, pr, stream);
}

cudaError_t launch_shortconv_tokens(const ShortConvArgs &a, int T, int advance, int esz, cudaStream_t stream) {
  return esz == 2 ? launch_tokens<__nv_bfloat16>(a, T, advance, stream) : launch_tokens<float>(a, T, advance, stream);
}

cudaError_t launch_shortconv_commit(int *cur, const int *accepted, int batch, int ring, int most, cudaStream_t stream) {
  commit_kernel<<<(batch + 255) / 256, 256, 0, stream>>>(cur, accepted, batch, ring, most);
  return cudaGetLastError();
}

}  // namespace rssm
