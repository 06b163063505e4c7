// shortconv.cu -- the short causal convolution in front of a layer's inputs, for prompts and for decoding.
//
//   out[t][c] = act(bias[c] + sum_k w[c][k] in[t - (K-1) + k][c]),  K = 2..4
//
// A few multiply-adds per value against one read and one write of it: the bound is memory.  A thread owns V
// consecutive channels, keeps their K taps and the last K-1 inputs in registers as fp32 and walks along the tokens, so
// every input is loaded once (plus K-1 rows where a prompt is cut into tiles), a group of tokens ahead of its use.  SiLU
// is one exponential and one reciprocal of the special-function unit, which alone would take three quarters of the
// memory's time; the exact division and expf took twice that.
#include <cooperative_groups.h>

#include "kernels.h"

namespace cg = cooperative_groups;

namespace rssm {

namespace {

constexpr int kPromptThreads = 128, kTokenThreads = 256;
// Channels a thread and tokens loaded together: 16 bytes of bf16 and four tokens ahead for prompts (143 us for 16384 tokens
// of 10240 channels, 4 channels: 150 us); decoding has registers for two ahead (8 drafts of 512 sequences 80 us; 4
// channels with twice the threads: 92 us).
constexpr int kPromptV = 8, kPromptGroup = 4;
constexpr int kTokenV = 8, kTokenGroup = 2, kTokenBlocks = 2;

// V values as they lie in memory
template <typename TI, int V>
struct Raw {
  static constexpr int kWords = V * (int)sizeof(TI) / 4;  // 2, 4 or 8
  uint32_t u[kWords];
  __device__ __forceinline__ void load(const TI *p) {
    if constexpr (kWords == 2) {
      const uint2 v = *reinterpret_cast<const uint2 *>(p);
      u[0] = v.x; u[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const uint4 v = reinterpret_cast<const uint4 *>(p)[i];
        u[4 * i] = v.x; u[4 * i + 1] = v.y; u[4 * i + 2] = v.z; u[4 * i + 3] = v.w;
      }
    }
  }
  __device__ __forceinline__ void store(TI *p) const {
    if constexpr (kWords == 2) {
      *reinterpret_cast<uint2 *>(p) = make_uint2(u[0], u[1]);
    } else {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i)
        reinterpret_cast<uint4 *>(p)[i] = make_uint4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) u[i] = 0;
  }
  __device__ __forceinline__ void widen(float (&o)[V]) const {
    if constexpr (sizeof(TI) == 4) {
#pragma unroll
      for (int j = 0; j < V; ++j) o[j] = __uint_as_float(u[j]);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) o[j] = __uint_as_float(j & 1 ? u[j / 2] & 0xffff0000u : u[j / 2] << 16);
    }
  }
  __device__ __forceinline__ void round(const float (&o)[V]) {
    if constexpr (sizeof(TI) == 4) {
#pragma unroll
      for (int j = 0; j < V; ++j) u[j] = __float_as_uint(o[j]);
    } else {
#pragma unroll
      for (int j = 0; j < kWords; ++j) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(o[2 * j], o[2 * j + 1]);
        u[j] = *reinterpret_cast<const uint32_t *>(&h);
      }
    }
  }
};

// the taps and bias of V channels from c
template <typename TI, int K, int V>
struct Filter {
  float w[K][V], b[V];
  bool silu;
  __device__ __forceinline__ void load(const ShortConvArgs &a, int c) {
    const TI *wp = reinterpret_cast<const TI *>(a.weight) + (size_t)c * K;
    float flat[K][V];
    Raw<TI, V> r;
#pragma unroll
    for (int i = 0; i < K; ++i) {
      r.load(wp + V * i);
      r.widen(flat[i]);
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < V; ++j) w[k][j] = flat[(j * K + k) / V][(j * K + k) % V];
    r.clear();
    if (a.bias) r.load(reinterpret_cast<const TI *>(a.bias) + c);
    r.widen(b);
    silu = a.silu;
  }
  // v / (1 + exp(-v)), to about 2^-21 of it; where exp overflows the quotient is -0
  __device__ __forceinline__ float act(float v) const {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return silu ? v * r : v;
  }
  __device__ __forceinline__ void apply(const float (&win)[K - 1][V], const float (&x)[V], float (&o)[V]) const {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float v = b[j];
#pragma unroll
      for (int k = 0; k < K - 1; ++k) v = fmaf(w[k][j], win[k][j], v);
      o[j] = act(fmaf(w[K - 1][j], x[j], v));
    }
  }
};

template <int K, int V>
__device__ __forceinline__ void push(float (&win)[K - 1][V], const float (&x)[V]) {
#pragma unroll
  for (int k = 0; k + 2 < K; ++k)
#pragma unroll
    for (int j = 0; j < V; ++j) win[k][j] = win[k + 1][j];
#pragma unroll
  for (int j = 0; j < V; ++j) win[K - 2][j] = x[j];
}

__device__ __forceinline__ int wrap(int v, int ring) {
  v %= ring;
  return v < 0 ? v + ring : v;
}

// where the channels from c go: the output that holds them (at its first row) and its row length
template <typename TI>
__device__ __forceinline__ TI *split_out(const ShortConvArgs &a, int c, int &row) {
  const int c1 = a.split[0], c2 = c1 + a.split[1];
  row = c < c1 ? a.split[0] : c < c2 ? a.split[1] : a.split[2];
  void *const p = c < c1 ? a.out[0] : c < c2 ? a.out[1] : a.out[2];
  return reinterpret_cast<TI *>(p) + (c < c1 ? c : c < c2 ? c - c1 : c - c2);
}

// n tokens from `in` through the filter, loaded a group ahead; `keep(raw)` sees every input in turn
template <typename TI, int K, int V, int kGroup, typename Keep>
__device__ __forceinline__ void walk(const Filter<TI, K, V> &f, float (&win)[K - 1][V], const TI *in, size_t in_stride,
                                     TI *out, int row, int n, Keep keep) {
  Raw<TI, V> now[kGroup], next[kGroup];
#pragma unroll
  for (int i = 0; i < kGroup; ++i)
    if (i < n) now[i].load(in + i * in_stride);
  for (int t = 0; t < n; t += kGroup) {
#pragma unroll
    for (int i = 0; i < kGroup; ++i)
      if (t + kGroup + i < n) next[i].load(in + (t + kGroup + i) * in_stride);
#pragma unroll
    for (int i = 0; i < kGroup; ++i) {
      if (t + i < n) {
        float x[V], o[V];
        now[i].widen(x);
        f.apply(win, x, o);
        push<K, V>(win, x);
        Raw<TI, V> r;
        r.round(o);
        r.store(out + (size_t)(t + i) * row);
        keep(now[i]);
      }
      now[i] = next[i];
    }
  }
}

// Prompts.  blockIdx.x: tile of a prompt; blockIdx.y: block of channels.  The block of a prompt's first tile alone
// reads and rewrites the sequence's history, each thread its own channels, so the rewrite is safe in place.
template <typename TI, int K>
__global__ void __launch_bounds__(kPromptThreads) prompt_kernel(ShortConvArgs a, Prompts pr, int tile) {
  constexpr int V = kPromptV;
  __shared__ PieceWord found;
  Piece pc;
  if (!find_piece(pr, blockIdx.x, tile, pc, &found)) return;
  const int c = (blockIdx.y * kPromptThreads + threadIdx.x) * V;
  const int len = pc.end - pc.begin;
  if (c >= a.channels || (pc.first >= len && pc.index > 0)) return;
  Filter<TI, K, V> f;
  f.load(a, c);
  const TI *in = reinterpret_cast<const TI *>(a.in) + (size_t)pc.begin * a.in_stride + c;
  float win[K - 1][V];
  if (pc.index == 0) {
    TI *hist = reinterpret_cast<TI *>(a.hist) + (size_t)pc.slot * a.ring * a.channels + c;
    const int cur = wrap(a.cur[pc.slot], a.ring);
    Raw<TI, V> held[K - 1];
#pragma unroll
    for (int k = 0; k < K - 1; ++k) {
      held[k].clear();
      if (pc.resume) held[k].load(hist + (size_t)wrap(cur - (K - 1) + k, a.ring) * a.channels);
      held[k].widen(win[k]);
    }
    if (len > 0 || !pc.resume) {
#pragma unroll
      for (int k = 0; k < K - 1; ++k) {  // newest K-1 of (held, prompt)
        const int t = len - (K - 1) + k;
        Raw<TI, V> r;
        r.clear();
        if (t >= 0) {
          r.load(in + (size_t)t * a.in_stride);
        } else {
#pragma unroll
          for (int m = 0; m < K - 1; ++m)
            if (m == K - 1 + t) r = held[m];
        }
        r.store(hist + (size_t)wrap(cur - (K - 1) + k, a.ring) * a.channels);
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < K - 1; ++k) {
      Raw<TI, V> r;
      r.load(in + (size_t)(pc.first - (K - 1) + k) * a.in_stride);
      r.widen(win[k]);
    }
  }
  int row;
  TI *out = split_out<TI>(a, c, row);
  out += (size_t)(pc.begin + pc.first) * row;
  walk<TI, K, V, kPromptGroup>(f, win, in + (size_t)pc.first * a.in_stride, a.in_stride, out, row,
                               min(tile, len - pc.first), [](const Raw<TI, V> &) {});
}

// T tokens a sequence on top of its history.  A thread keeps the taps of its channels and takes the sequences of its
// cluster one after the other, with one token (kOne) the next sequence's rows on their way.  The blocks of a cluster
// share out the channels, so that the cursors can advance in place once all of them have read them (`advance`: one token
// that stands; otherwise the rows stay tentative).
template <typename TI, int K, bool kOne>
__global__ void __launch_bounds__(kTokenThreads, kTokenBlocks) token_kernel(ShortConvArgs a, int T, int advance) {
  constexpr int V = kTokenV;
  cg::cluster_group cluster = cg::this_cluster();
  const int blocks = cluster.num_blocks(), rank = cluster.block_rank();
  const int first = blockIdx.x / blocks, stride = gridDim.x / blocks;
  const size_t row_hist = a.channels;
  for (int c = (rank * blockDim.x + threadIdx.x) * V; c < a.channels; c += blocks * blockDim.x * V) {
    TI *hist0 = reinterpret_cast<TI *>(a.hist) + c;
    const TI *in0 = reinterpret_cast<const TI *>(a.in) + c;
    int row;
    TI *out0 = split_out<TI>(a, c, row);
    if (kOne) {
      Raw<TI, V> now[K], next[K];  // K-1 rows of history, then the token
      auto load = [&](int b, int cur, Raw<TI, V>(&r)[K]) {
#pragma unroll
        for (int k = 0; k < K - 1; ++k)
          r[k].load(hist0 + ((size_t)b * a.ring + wrap(cur - (K - 1) + k, a.ring)) * row_hist);
        r[K - 1].load(in0 + (size_t)b * a.in_stride);
      };
      int cur = wrap(a.cur[first], a.ring);
      load(first, cur, now);
      Filter<TI, K, V> f;
      f.load(a, c);
      int cur_next = first + stride < a.batch ? wrap(a.cur[first + stride], a.ring) : 0;
      for (int b = first; b < a.batch; b += stride) {
        const int after = b + 2 * stride < a.batch ? a.cur[b + 2 * stride] : 0;
        if (b + stride < a.batch) load(b + stride, cur_next, next);
        float win[K - 1][V], x[V], o[V];
#pragma unroll
        for (int k = 0; k < K - 1; ++k) now[k].widen(win[k]);
        now[K - 1].widen(x);
        f.apply(win, x, o);
        now[K - 1].store(hist0 + ((size_t)b * a.ring + cur) * row_hist);
        Raw<TI, V> r;
        r.round(o);
        r.store(out0 + (size_t)b * row);
        cur = cur_next;
        cur_next = wrap(after, a.ring);
#pragma unroll
        for (int k = 0; k < K; ++k) now[k] = next[k];
      }
    } else {
      Filter<TI, K, V> f;
      f.load(a, c);
      for (int b = first; b < a.batch; b += stride) {
        int slot = wrap(a.cur[b], a.ring);
        TI *hist = hist0 + (size_t)b * a.ring * row_hist;
        float win[K - 1][V];
#pragma unroll
        for (int k = 0; k < K - 1; ++k) {
          Raw<TI, V> r;
          r.load(hist + (size_t)wrap(slot - (K - 1) + k, a.ring) * row_hist);
          r.widen(win[k]);
        }
        walk<TI, K, V, kTokenGroup>(f, win, in0 + (size_t)b * T * a.in_stride, a.in_stride, out0 + (size_t)b * T * row,
                                    row, T, [&](const Raw<TI, V> &r) {
                                      r.store(hist + (size_t)slot * row_hist);
                                      slot = slot + 1 == a.ring ? 0 : slot + 1;
                                    });
      }
    }
  }
  if (advance) {
    cluster.sync();
    if (rank == 0)
      for (int b = first + threadIdx.x * stride; b < a.batch; b += blockDim.x * stride) {
        const int cur = wrap(a.cur[b], a.ring);
        a.cur_out[b] = cur + 1 == a.ring ? 0 : cur + 1;
      }
  }
}

__global__ void commit_kernel(int *cur, const int *accepted, int batch, int ring, int most) {
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= batch) return;
  const int acc = max(0, min(most, accepted[b]));
  cur[b] = wrap(wrap(cur[b], ring) + acc, ring);
}

template <typename TI>
cudaError_t launch_prompt(const ShortConvArgs &a, const Prompts &pr, int num_sms, cudaStream_t stream) {
  // Tiles as long as they still give two blocks an SM: K-1 rows are read twice a tile (from L2) and the taps once, and a
  // short tile is soon done, which is what counts when there are few.
  const int columns = (a.channels / kPromptV + kPromptThreads - 1) / kPromptThreads;
  int tile = 8;
  while (tile < 64 && (long long)(pr.total / (2 * tile) + 1) * columns >= 2LL * num_sms) tile *= 2;
  const dim3 grid(prompt_pieces(pr.total, pr.nseq, tile), columns);
  if (a.width == 2) prompt_kernel<TI, 2><<<grid, kPromptThreads, 0, stream>>>(a, pr, tile);
  else if (a.width == 3) prompt_kernel<TI, 3><<<grid, kPromptThreads, 0, stream>>>(a, pr, tile);
  else prompt_kernel<TI, 4><<<grid, kPromptThreads, 0, stream>>>(a, pr, tile);
  return cudaGetLastError();
}

template <typename TI, int K>
cudaError_t launch_tokens(const ShortConvArgs &a, int T, int advance, int num_sms, cudaStream_t stream) {
  const int vectors = a.channels / kTokenV;
  int threads = (vectors + 31) / 32 * 32;
  threads = threads > kTokenThreads ? kTokenThreads : threads;
  int blocks = (vectors + threads - 1) / threads;
  blocks = blocks > 8 ? 8 : blocks;  // the portable cluster
  // as many clusters as fit the SMs at once: the taps are read once a cluster
  int clusters = kTokenBlocks * num_sms / blocks;
  clusters = a.batch < clusters ? a.batch : clusters;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)clusters * blocks);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = blocks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return T == 1 ? cudaLaunchKernelEx(&cfg, token_kernel<TI, K, true>, a, T, advance)
                : cudaLaunchKernelEx(&cfg, token_kernel<TI, K, false>, a, T, advance);
}

template <typename TI>
cudaError_t launch_tokens(const ShortConvArgs &a, int T, int advance, int num_sms, cudaStream_t stream) {
  if (a.width == 2) return launch_tokens<TI, 2>(a, T, advance, num_sms, stream);
  if (a.width == 3) return launch_tokens<TI, 3>(a, T, advance, num_sms, stream);
  return launch_tokens<TI, 4>(a, T, advance, num_sms, stream);
}

}  // namespace

cudaError_t launch_shortconv_prompt(const ShortConvArgs &a, const Prompts &pr, int esz, int num_sms,
                                    cudaStream_t stream) {
  return esz == 2 ? launch_prompt<__nv_bfloat16>(a, pr, num_sms, stream) : launch_prompt<float>(a, pr, num_sms, stream);
}

cudaError_t launch_shortconv_tokens(const ShortConvArgs &a, int T, int advance, int esz, int num_sms,
                                    cudaStream_t stream) {
  return esz == 2 ? launch_tokens<__nv_bfloat16>(a, T, advance, num_sms, stream)
                  : launch_tokens<float>(a, T, advance, num_sms, stream);
}

cudaError_t launch_shortconv_commit(int *cur, const int *accepted, int batch, int ring, int most, cudaStream_t stream) {
  commit_kernel<<<(batch + 255) / 256, 256, 0, stream>>>(cur, accepted, batch, ring, most);
  return cudaGetLastError();
}

}  // namespace rssm
