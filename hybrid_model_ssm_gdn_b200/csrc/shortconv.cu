// shortconv.cu -- the short causal convolution in front of a layer's inputs, for prompts and for decoding.
//
//   out[t][c] = act(bias[c] + sum_k w[c][k] in[t - (K-1) + k][c]),  K = 2..4
//
// A few multiply-adds per value against one read and one write of it: the bound is memory, closely followed by the
// instructions (prompts: DRAM 62 %, issue 79 % busy).  A thread owns V
// consecutive channels, keeps their K taps and the last K-1 inputs in registers as fp32 and walks along the tokens, so
// every input is loaded once (plus K-1 rows where a prompt is cut into tiles).  Its next rows are on their way to shared
// memory: as many bytes in flight as the bandwidth times the latency ask for do not fit the registers beside the taps.
// SiLU is one exponential and one reciprocal of the special-function unit, which alone would take three quarters of the
// memory's time; the exact division and expf took twice that.
//
// Measured (bf16, 10240 channels, K 4): 16384 tokens in 8 prompts 127 us, 5.3 TB/s (four tokens ahead in registers 145 us);
// 8 drafts of 512 sequences with their commit 57 us, 4.9 TB/s (two tokens ahead in registers 81 us).
#include <cooperative_groups.h>

#include "prompt_kernels.h"

namespace cg = cooperative_groups;

namespace rssm {

namespace {

constexpr int kPromptThreads = 128, kTokenThreads = 256;
// Channels a thread: 16 bytes of bf16 (half as many with rows ahead in registers: prompts 150 us for 143, drafts 92 for 80).
constexpr int kPromptV = 8, kTokenV = 8, kTokenBlocks = 2;

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
  // v / (1 + exp(-v)).  For bf16 outputs with the rounding of v log2(e), which costs |v| 2^-24 of the exponential, far below
  // their own rounding of 2^-9; where exp(-v) passes 2^126 (v < -87.3) the quotient, below 2^-119, is -0 (a form that
  // kept those, too, cost prompts 20 % more time).  For fp32 outputs to within 2^-20 of the value down to its last bits: the
  // rounding is given back to first order, and for v < 0 the quotient is v h h / (1 + h h) with h = exp(v / 2), which stays
  // in the normal range as long as the result has bits.
  __device__ __forceinline__ float act(float v) const {
    constexpr float kL = 1.4426950408889634f, kRest = (float)(1.4426950408889634 - (double)kL), kLn2 = 0.69314718f;
    float e, r;
    if constexpr (sizeof(TI) == 2) {
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v * -kL));
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
      return silu ? v * r : v;
    } else {
      const float a = fminf(fabsf(v), 1e6f), t = a * (-0.5f * kL);
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
      const float h = fmaf(e * kLn2, fmaf(a, -0.5f * kRest, fmaf(a, -0.5f * kL, -t)), e);
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaf(h, h, 1.f)));
      const float q = v * r;
      return silu ? v < 0.f ? q * h * h : q : v;
    }
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

// A thread's own rows on their way, in shared memory: kAheadBytes of them, the oldest taken while a new one is asked for.
// Only the thread itself writes and reads its slots, so there is nothing to wait for but its own copies.
constexpr int kAheadBytes = 128;
template <typename TI, int V, int kThreads>
struct Ahead {
  static constexpr int kWords = V * (int)sizeof(TI) / 16, kRows = kAheadBytes / (16 * kWords);
  uint4 (*slots)[kThreads];  // [kRows * kWords]
  int put, get;
  __device__ __forceinline__ void ask(const TI *p, bool live) {
    if (live) {
#pragma unroll
      for (int i = 0; i < kWords; ++i)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(&slots[put * kWords + i][threadIdx.x])),
                     "l"(p + 16 / sizeof(TI) * i)
                     : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    put = (put + 1) % kRows;
  }
  __device__ __forceinline__ void take(Raw<TI, V> &r) {  // after kRows rows were asked for beyond the last one taken
    asm volatile("cp.async.wait_group %0;" ::"n"(kRows - 1) : "memory");
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      uint4 v;
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                   : "r"(smem_u32(&slots[get * kWords + i][threadIdx.x]))
                   : "memory");
      r.u[4 * i] = v.x; r.u[4 * i + 1] = v.y; r.u[4 * i + 2] = v.z; r.u[4 * i + 3] = v.w;
    }
    get = (get + 1) % kRows;
  }
};

// Prompts.  blockIdx.x: tile of a prompt; blockIdx.y: block of channels.  The block of a prompt's first tile alone
// reads and rewrites the sequence's history, each thread its own channels, so the rewrite is safe in place.
template <typename TI, int K>
__global__ void __launch_bounds__(kPromptThreads) prompt_kernel(ShortConvArgs a, Prompts pr, int tile) {
  constexpr int V = kPromptV;
  using Rows = Ahead<TI, V, kPromptThreads>;
  __shared__ uint4 slots[kAheadBytes / 16][kPromptThreads];
  __shared__ PieceWord found;
  Piece pc;
  const PieceStatus status = find_piece(pr, blockIdx.x, tile, pc, &found);
  if (status != kPieceRun) {
    if (pr.refused_nan)
      for (int s = 0; s < 3; ++s)
        refuse(pr, status, pc, tile, reinterpret_cast<TI *>(a.out[s]), a.split[s], blockIdx.y, gridDim.y);
    return;
  }
  const int c = (blockIdx.y * kPromptThreads + threadIdx.x) * V;
  const int len = pc.end - pc.begin;
  if (c >= a.channels || (pc.first >= len && pc.index > 0)) return;
  const TI *in = reinterpret_cast<const TI *>(a.in) + (size_t)pc.begin * a.in_stride + c;
  const int n = min(tile, len - pc.first);
  Rows rows{slots, 0, 0};
  const TI *next = in + (size_t)pc.first * a.in_stride;
#pragma unroll
  for (int i = 0; i < Rows::kRows; ++i, next += a.in_stride) rows.ask(next, i < n);
  Filter<TI, K, V> f;
  f.load(a, c);
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
  for (int t = 0; t < n; ++t) {
    Raw<TI, V> r;
    rows.take(r);
    rows.ask(next, t + Rows::kRows < n);
    next += a.in_stride;
    float x[V], o[V];
    r.widen(x);
    f.apply(win, x, o);
    push<K, V>(win, x);
    r.round(o);
    r.store(out);
    out += row;
  }
}

// One token a sequence on top of its history.  A thread keeps the taps of its channels and takes the sequences of its
// cluster one after the other, the next sequence's rows on their way.  The blocks of a cluster share out the channels, so
// that the cursors can advance in place once all of them have read them (`advance`: the token stands; otherwise it is a
// tentative row).
template <typename TI, int K>
__global__ void __launch_bounds__(kTokenThreads, kTokenBlocks) token_kernel(ShortConvArgs a, int advance) {
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

// T drafts a sequence on top of its history: tentative rows, the cursors stay.  blockIdx.x: which sequences, blockIdx.y:
// block of channels.  A thread sees one stream of rows, K-1 of history and T of input for each of its sequences in turn, and
// asks for them several ahead, across sequences.
template <typename TI, int K>
__global__ void __launch_bounds__(kTokenThreads, kTokenBlocks) draft_kernel(ShortConvArgs a, int T) {
  constexpr int V = kTokenV;
  using Rows = Ahead<TI, V, kTokenThreads>;
  __shared__ uint4 slots[kAheadBytes / 16][kTokenThreads];
  const int c = (blockIdx.y * kTokenThreads + threadIdx.x) * V, stride = gridDim.x;
  if (c >= a.channels) return;
  TI *hist0 = reinterpret_cast<TI *>(a.hist) + c;
  const TI *in0 = reinterpret_cast<const TI *>(a.in) + c;
  auto cursor = [&](int b) { return b < a.batch ? wrap(a.cur[b], a.ring) : 0; };
  int row;
  TI *out0 = split_out<TI>(a, c, row);

  Rows rows{slots, 0, 0};
  int ab = blockIdx.x, at = 1 - K;  // the row to ask for: history below 0, else a draft
  int acur = cursor(ab), acur_next = cursor(ab + stride);
  auto ask = [&] {
    const TI *p = at < 0 ? hist0 + ((size_t)ab * a.ring + wrap(acur + at, a.ring)) * a.channels
                         : in0 + ((size_t)ab * T + at) * a.in_stride;
    rows.ask(p, ab < a.batch);
    if (++at == T) {
      at = 1 - K;
      ab += stride;
      acur = acur_next;
      acur_next = cursor(ab + stride);
    }
  };
#pragma unroll
  for (int i = 0; i < Rows::kRows; ++i) ask();
  Filter<TI, K, V> f;
  f.load(a, c);
  int slot_next = cursor(blockIdx.x);
  for (int b = blockIdx.x; b < a.batch; b += stride) {
    int slot = slot_next;
    slot_next = cursor(b + stride);
    TI *hist = hist0 + (size_t)b * a.ring * a.channels;
    TI *out = out0 + (size_t)b * T * row;
    float win[K - 1][V];
#pragma unroll
    for (int k = 0; k < K - 1; ++k) {
      Raw<TI, V> r;
      rows.take(r);
      ask();
      r.widen(win[k]);
    }
    for (int t = 0; t < T; ++t) {
      Raw<TI, V> r;
      rows.take(r);
      ask();
      r.store(hist + (size_t)slot * a.channels);
      slot = slot + 1 == a.ring ? 0 : slot + 1;
      float x[V], o[V];
      r.widen(x);
      f.apply(win, x, o);
      push<K, V>(win, x);
      r.round(o);
      r.store(out);
      out += row;
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
  if (T > 1) {  // as many blocks as fit the SMs at once: the taps are read once a block
    const int columns = (vectors + kTokenThreads - 1) / kTokenThreads;
    const int groups = max(1, min(a.batch, kTokenBlocks * num_sms / columns));
    draft_kernel<TI, K><<<dim3(groups, columns), kTokenThreads, 0, stream>>>(a, T);
    return cudaGetLastError();
  }
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
  return cudaLaunchKernelEx(&cfg, token_kernel<TI, K>, a, advance);
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
