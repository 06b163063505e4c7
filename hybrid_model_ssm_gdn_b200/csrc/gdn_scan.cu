// gdn_scan.cu -- the gated delta rule over whole prompts, token by token on CUDA cores, and a context's stored states.
//
//   p = S_{t-1} k_t,  u = beta_t (v_t - alpha_t p),  S_t = alpha_t S_{t-1} + u k_t^T,
//   y_t = q_scale S_t q_t = q_scale (alpha_t S_{t-1} q_t + u (k_t . q_t))
//
// Both products of a token are taken from the state before it, so that one round of sums over a row's columns is all that
// stands between two tokens.  A row of 128 fp32 lies in four lanes (two shuffles a sum), a warp carries 8 rows; k, q, v
// come from shared memory, 16 tokens at a time with the next ones on their way.  fp32 throughout: inputs of 24 bits would
// need six bf16 products for each one of the chunk form.
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

// this lane's 32 columns of a row of T in shared memory: runs of 16 bytes, 4 lanes side by side
template <typename T>
struct Columns;
template <>
struct Columns<float> {
  static constexpr int kRun = 4;
  static __device__ __forceinline__ void load(const float *row, int l4, f2 (&o)[16]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 v = *reinterpret_cast<const float4 *>(row + 4 * (l4 + 4 * i));
      o[2 * i] = pack2(v.x, v.y);
      o[2 * i + 1] = pack2(v.z, v.w);
    }
  }
};
template <>
struct Columns<__nv_bfloat16> {
  static constexpr int kRun = 8;
  static __device__ __forceinline__ void load(const __nv_bfloat16 *row, int l4, f2 (&o)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 v = *reinterpret_cast<const uint4 *>(row + 8 * (l4 + 4 * i));
      o[4 * i] = pack2(v.x << 16, v.x & 0xffff0000u);
      o[4 * i + 1] = pack2(v.y << 16, v.y & 0xffff0000u);
      o[4 * i + 2] = pack2(v.z << 16, v.z & 0xffff0000u);
      o[4 * i + 3] = pack2(v.w << 16, v.w & 0xffff0000u);
    }
  }
};

__device__ __forceinline__ float sum4(f2 a, f2 b, f2 c, f2 d) {  // over the registers and a row's four lanes
  const f2 one = pack2(1.f, 1.f);
  float lo, hi;
  unpack2(fma2(one, fma2(one, a, b), fma2(one, c, d)), lo, hi);
  float v = lo + hi;
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

// R rows of head blockIdx.y from row blockIdx.z * R on
template <typename T, int R>
__global__ void __launch_bounds__(4 * R) gdn_scan_kernel(GdnScanArgs a, Prompts pr) {
  __shared__ __align__(16) Stage<T, R> st[2];
  __shared__ PieceWord found;
  constexpr int kThreads = 4 * R, kRun = Columns<T>::kRun, kShare = kThreads / kTok;
  Piece pc;
  const int h = blockIdx.y, row0 = blockIdx.z * R;
  allow_next();
  if (find_piece(pr, blockIdx.x, pr.total + 1, pc, &found) != kPieceRun) return;
  const int len = pc.end - pc.begin;
  if (len == 0 && pc.resume) return;
  const int tid = threadIdx.x, lane = tid & 31, l4 = lane & 3;
  const int mine = tid >> 2;  // this lane's row within the block
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

  f2 s[16];
  float *Sg = a.S + (((size_t)(a.by_prompt ? pc.seq : pc.slot) * a.H + h) * a.R + row0 + mine) * kCols;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float4 v = f4zero();
    const int col = kRun == 4 ? 4 * (l4 + 4 * i) : 8 * (l4 + 4 * (i >> 1)) + 4 * (i & 1);
    if (pc.resume && have) v = *reinterpret_cast<const float4 *>(Sg + col);
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
    {  // k . q of each token, by kShare neighbouring threads
      const int t = tid / kShare, part = tid % kShare;
      float v = 0.f;
#pragma unroll
      for (int n = part; n < kCols; n += kShare) v = fmaf(to_f32(m.k[t][n]), to_f32(m.q[t][n]), v);
#pragma unroll
      for (int off = kShare / 2; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
      if (part == 0) m.g[t].z = v;
      if (tid < kTok) {
        m.g[tid].x = alpha_now;
        m.g[tid].y = beta_now;
      }
    }
    __syncthreads();
    const int n = min(kTok, len - t0);
#pragma unroll 2
    for (int t = 0; t < n; ++t) {
      const float4 g = m.g[t];
      f2 k[16], q[16];
      Columns<T>::load(m.k[t], l4, k);
      Columns<T>::load(m.q[t], l4, q);
      f2 p[4], w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[i] = mul2(s[i], k[i]);
        w[i] = mul2(s[i], q[i]);
      }
#pragma unroll
      for (int i = 4; i < 16; ++i) {
        p[i & 3] = fma2(s[i], k[i], p[i & 3]);
        w[i & 3] = fma2(s[i], q[i], w[i & 3]);
      }
      const float sk = sum4(p[0], p[1], p[2], p[3]), sq = sum4(w[0], w[1], w[2], w[3]);
      const float u = g.y * fmaf(-g.x, sk, to_f32(m.v[t][mine]));
      const f2 uu = pack2(u, u), aa = pack2(g.x, g.x);
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = fma2(uu, k[i], mul2(aa, s[i]));
      if (l4 == 0 && have) yg[(size_t)(t0 + t) * a.H * a.R] = a.q_scale * fmaf(u, g.z, g.x * sq);
    }
    __syncthreads();  // g and the stage are read no more
  }
  if (have) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int col = kRun == 4 ? 4 * (l4 + 4 * i) : 8 * (l4 + 4 * (i >> 1)) + 4 * (i & 1);
      float4 v;
      unpack2(s[2 * i], v.x, v.y);
      unpack2(s[2 * i + 1], v.z, v.w);
      *reinterpret_cast<float4 *>(Sg + col) = v;
    }
  }
}

template <typename T, int R>
cudaError_t launch_rows(const GdnScanArgs &a, const Prompts &pr, cudaStream_t stream) {
  gdn_scan_kernel<T, R><<<dim3(pr.nseq, a.H, (a.R + R - 1) / R), 4 * R, 0, stream>>>(a, pr);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_type(const GdnScanArgs &a, const Prompts &pr, int num_sms, cudaStream_t stream) {
  // All rows a block share one staging of k and q; 8 rows, one warp, spread few heads and prompts over the SMs.
  const long long heads = (long long)pr.nseq * a.H;
  if (heads >= 2LL * num_sms) return launch_rows<T, 64>(a, pr, stream);
  if (heads * 4 >= num_sms) return launch_rows<T, 16>(a, pr, stream);
  return launch_rows<T, 8>(a, pr, stream);
}

}  // namespace

cudaError_t launch_gdn_scan(const GdnScanArgs &a, const Prompts &pr, int esz, int num_sms, cudaStream_t stream) {
  return esz == 2 ? launch_type<__nv_bfloat16>(a, pr, num_sms, stream) : launch_type<float>(a, pr, num_sms, stream);
}

}  // namespace rssm
