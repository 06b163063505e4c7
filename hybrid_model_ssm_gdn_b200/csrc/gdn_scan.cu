// gdn_scan.cu -- the gated delta rule over whole prompts, token by token on CUDA cores, and a context's stored states.
//
//   p = S_{t-1} k_t,  u = beta_t (v_t - alpha_t p),  S_t = alpha_t S_{t-1} + u k_t^T,
//   y_t = q_scale S_t q_t = q_scale (alpha_t S_{t-1} q_t + u (k_t . q_t))
//
// Both products of a token are taken from the state before it, so that one round of sums over a row's columns is all that
// stands between two tokens.  A row of 128 fp32 lies in 4 or 16 lanes (two or four shuffles a sum); k, q, v come from shared
// memory, 16 tokens at a time with the next ones on their way.  fp32 throughout: inputs of 24 bits would need six bf16 products
// for each one of the chunk form.
// Bound by the sums' way through the lanes where rows are few (0.19 us a token, 2 prompts of 8 heads), by the instructions of
// 4 x 128 x R multiply-adds a token where they are many (25 TFLOP/s, 32 prompts of 32 heads).
#include "prompt_kernels.h"
#include "packed.cuh"

namespace rssm {

namespace {

constexpr int kTok = 16;  // tokens staged at a time

// 16 bytes to shared memory, zeros where `live` is not set
__device__ __forceinline__ void copy16(void *dst, const void *src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(live ? 16 : 0) : "memory");
}

template <typename T, int R>
struct Stage {
  T k[kTok][kCols], q[kTok][kCols];
  T v[kTok][R];
  float4 g[kTok];  // alpha, beta, k . q
};

// this lane's 128 / L columns of a row of T in shared memory: runs of 16 bytes, L lanes side by side
template <typename T>
struct Columns;
template <>
struct Columns<float> {
  static constexpr int kRun = 4;
  template <int L>
  static __device__ __forceinline__ void load(const float *row, int lane, f2 (&o)[64 / L]) {
#pragma unroll
    for (int i = 0; i < 32 / L; ++i) {
      const float4 v = *reinterpret_cast<const float4 *>(row + 4 * (lane + L * i));
      o[2 * i] = pack2(v.x, v.y);
      o[2 * i + 1] = pack2(v.z, v.w);
    }
  }
  static __device__ __forceinline__ void quad(const float *row, int i, f2 (&o)[2]) {  // columns 4 i .. 4 i + 3
    const float4 v = *reinterpret_cast<const float4 *>(row + 4 * i);
    o[0] = pack2(v.x, v.y);
    o[1] = pack2(v.z, v.w);
  }
};
template <>
struct Columns<__nv_bfloat16> {
  static constexpr int kRun = 8;
  template <int L>
  static __device__ __forceinline__ void load(const __nv_bfloat16 *row, int lane, f2 (&o)[64 / L]) {
#pragma unroll
    for (int i = 0; i < 16 / L; ++i) {
      const uint4 v = *reinterpret_cast<const uint4 *>(row + 8 * (lane + L * i));
      o[4 * i] = pack2(v.x << 16, v.x & 0xffff0000u);
      o[4 * i + 1] = pack2(v.y << 16, v.y & 0xffff0000u);
      o[4 * i + 2] = pack2(v.z << 16, v.z & 0xffff0000u);
      o[4 * i + 3] = pack2(v.w << 16, v.w & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void quad(const __nv_bfloat16 *row, int i, f2 (&o)[2]) {
    const uint2 v = *reinterpret_cast<const uint2 *>(row + 4 * i);
    o[0] = pack2(v.x << 16, v.x & 0xffff0000u);
    o[1] = pack2(v.y << 16, v.y & 0xffff0000u);
  }
};

template <int N>
__device__ __forceinline__ float sum_of(const f2 (&v)[4]) {  // of the first N pairs
  const f2 one = pack2(1.f, 1.f);
  float lo, hi;
  unpack2(N == 2 ? fma2(one, v[0], v[1]) : fma2(one, fma2(one, v[0], v[1]), fma2(one, v[2], v[3])), lo, hi);
  return lo + hi;
}

template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int off = 1; off < L; off <<= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// the first column of this lane's `i`-th four (of 32 / L)
template <typename T, int L>
__device__ __forceinline__ int four_at(int lane, int i) {
  return Columns<T>::kRun == 4 ? 4 * (lane + L * i) : 8 * (lane + L * (i >> 1)) + 4 * (i & 1);
}

// R rows of head blockIdx.y from row blockIdx.z * R on, L lanes a row
template <typename T, int R, int L>
__global__ void __launch_bounds__(L * R) gdn_scan_kernel(GdnScanArgs a, Prompts pr) {
  __shared__ __align__(16) Stage<T, R> st[2];
  __shared__ PieceWord found;
  constexpr int kThreads = L * R, kWarps = kThreads / 32, kPairs = 64 / L;
  Piece pc;
  const int h = blockIdx.y, row0 = blockIdx.z * R;
  allow_next();
  if (find_piece(pr, blockIdx.x, pr.total + 1, pc, &found) != kPieceRun) return;
  const int len = pc.end - pc.begin;
  if (len == 0 && pc.resume) return;
  const int tid = threadIdx.x, lane = tid & 31, l = lane & (L - 1);
  const int mine = tid / L;  // this lane's row within the block
  const bool have = row0 + mine < a.R;
  const int hk = h / (a.H / a.Hk);
  const T *kg = static_cast<const T *>(a.k) + ((size_t)pc.begin * a.Hk + hk) * kCols;
  const T *qg = static_cast<const T *>(a.q) + ((size_t)pc.begin * a.Hk + hk) * kCols;
  const T *vg = static_cast<const T *>(a.v) + ((size_t)pc.begin * a.H + h) * a.R + row0;
  const float *ag = a.alpha + (size_t)pc.begin * a.H + h, *bg = a.beta + (size_t)pc.begin * a.H + h;

  float alpha_next = 0.f, beta_next = 0.f;
  auto fetch = [&](int t0, Stage<T, R> &s) {
    constexpr int run = 16 / sizeof(T);
    for (int e = tid; e < kTok * (kCols / run); e += kThreads) {
      const int t = e / (kCols / run), n = run * (e % (kCols / run));
      const bool live = t0 + t < len;
      const size_t at = live ? (size_t)(t0 + t) * a.Hk * kCols + n : 0;
      copy16(&s.k[t][n], kg + at, live);
      copy16(&s.q[t][n], qg + at, live);
    }
    for (int e = tid; e < kTok * (R / run); e += kThreads) {
      const int t = e / (R / run), r = run * (e % (R / run));
      const bool live = t0 + t < len && row0 + r < a.R;  // a.R is a multiple of 8
      copy16(&s.v[t][r], vg + (live ? (size_t)(t0 + t) * a.H * a.R + r : 0), live);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (tid < kTok && t0 + tid < len) {
      alpha_next = ag[(size_t)(t0 + tid) * a.H];
      beta_next = bg[(size_t)(t0 + tid) * a.H];
    }
  };
  if (len > 0) fetch(0, st[0]);

  f2 s[kPairs];
  float *Sg = a.S + (((size_t)(a.by_prompt ? pc.seq : pc.slot) * a.H + h) * a.R + row0 + mine) * kCols;
#pragma unroll
  for (int i = 0; i < kPairs / 2; ++i) {
    float4 v = f4zero();
    if (pc.resume && have) v = *reinterpret_cast<const float4 *>(Sg + four_at<T, L>(l, i));
    s[2 * i] = pack2(v.x, v.y);
    s[2 * i + 1] = pack2(v.z, v.w);
  }
  float *yg = a.y + ((size_t)pc.begin * a.H + h) * a.R + row0 + mine;

  for (int t0 = 0, b = 0; t0 < len; t0 += kTok, b ^= 1) {
    Stage<T, R> &m = st[b];
    const float alpha_now = alpha_next, beta_now = beta_next;
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    if (t0 + kTok < len) fetch(t0 + kTok, st[b ^ 1]);  // read last before the barrier above
    // k . q of each token, a warp at a time
#pragma unroll
    for (int j = 0; j < kTok; j += kWarps) {
      const int t = j + (tid >> 5);
      f2 k[2], q[2];
      Columns<T>::quad(m.k[t], lane, k);
      Columns<T>::quad(m.q[t], lane, q);
      float lo, hi;
      unpack2(fma2(k[0], q[0], mul2(k[1], q[1])), lo, hi);
      lo = lanes_sum<32>(lo + hi);
      if (lane == 0) m.g[t].z = lo;
    }
    if (tid < kTok) {
      m.g[tid].x = alpha_now;
      m.g[tid].y = beta_now;
    }
    __syncthreads();
    const int n = min(kTok, len - t0);
    f2 k[kPairs], q[kPairs];
    constexpr bool kAhead = L > 4;  // registers for two tokens' k and q
    if (kAhead) {
      Columns<T>::template load<L>(m.k[0], l, k);
      Columns<T>::template load<L>(m.q[0], l, q);
    }
    float4 g = m.g[0];
    float v = to_f32(m.v[0][mine]);
#pragma unroll 1
    for (int t = 0; t < n; ++t) {
      // the next token's inputs set out before this one's sums (the last of a stage reads itself again)
      const int next = min(t + 1, kTok - 1);
      f2 k2[kPairs], q2[kPairs], p[4], w[4];
      if (kAhead) {
        Columns<T>::template load<L>(m.k[next], l, k2);
        Columns<T>::template load<L>(m.q[next], l, q2);
      } else {
        Columns<T>::template load<L>(m.k[t], l, k);
        Columns<T>::template load<L>(m.q[t], l, q);
      }
      const float4 g2 = m.g[next];
      const float v2 = to_f32(m.v[next][mine]);
      constexpr int kSums = kPairs < 8 ? 2 : 4;
#pragma unroll
      for (int i = 0; i < kSums; ++i) {
        p[i] = mul2(s[i], k[i]);
        w[i] = mul2(s[i], q[i]);
      }
#pragma unroll
      for (int i = kSums; i < kPairs; ++i) {
        p[i & (kSums - 1)] = fma2(s[i], k[i], p[i & (kSums - 1)]);
        w[i & (kSums - 1)] = fma2(s[i], q[i], w[i & (kSums - 1)]);
      }
      const float sk = lanes_sum<L>(sum_of<kSums>(p)), sq = lanes_sum<L>(sum_of<kSums>(w));
      const float u = g.y * fmaf(-g.x, sk, v);
      const f2 uu = pack2(u, u), aa = pack2(g.x, g.x);
#pragma unroll
      for (int i = 0; i < kPairs; ++i) s[i] = fma2(uu, k[i], mul2(aa, s[i]));
      if (l == 0 && have) yg[(size_t)(t0 + t) * a.H * a.R] = a.q_scale * fmaf(u, g.z, g.x * sq);
      if (kAhead) {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          k[i] = k2[i];
          q[i] = q2[i];
        }
      }
      g = g2;
      v = v2;
    }
    __syncthreads();  // g and the stage are read no more
  }
  if (have) {
#pragma unroll
    for (int i = 0; i < kPairs / 2; ++i) {
      float4 v;
      unpack2(s[2 * i], v.x, v.y);
      unpack2(s[2 * i + 1], v.z, v.w);
      *reinterpret_cast<float4 *>(Sg + four_at<T, L>(l, i)) = v;
    }
  }
}

template <typename T, int R, int L>
cudaError_t launch_rows(const GdnScanArgs &a, const Prompts &pr, cudaStream_t stream) {
  gdn_scan_kernel<T, R, L><<<dim3(pr.nseq, a.H, (a.R + R - 1) / R), L * R, 0, stream>>>(a, pr);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_type(const GdnScanArgs &a, const Prompts &pr, int num_sms, cudaStream_t stream) {
  // All rows of a block share one staging of k and q, so many heads are best off with 64 rows a block, and 4 lanes a row need
  // the fewest shuffles.  Few heads wait for each token's sums alone: 8 rows over 16 lanes put a warp on each quarter of an SM
  // (fp32, us, 8 / 16 / 64 rows a block: 2 prompts of 150 tokens, 8 heads of 64 rows 39 / 53 / 79; 8 prompts 60 / 57 / 79;
  // 8 of 32 heads of 128 rows 340 / 239 / 235; 32 of them 1287 / 858 / 789).
  const long long heads = (long long)pr.nseq * a.H;
  if (heads * ((a.R + 7) / 8) <= 2LL * num_sms) return launch_rows<T, 8, 16>(a, pr, stream);
  if (heads < 2LL * num_sms) return launch_rows<T, 16, 4>(a, pr, stream);
  return launch_rows<T, 64, 4>(a, pr, stream);
}

}  // namespace

cudaError_t launch_gdn_scan(const GdnScanArgs &a, const Prompts &pr, int esz, int num_sms, cudaStream_t stream) {
  return esz == 2 ? launch_type<__nv_bfloat16>(a, pr, num_sms, stream) : launch_type<float>(a, pr, num_sms, stream);
}

}  // namespace rssm
