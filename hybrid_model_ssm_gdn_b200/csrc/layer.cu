// layer.cu -- what stands between a layer's projections: the inputs of the gated delta rule, the norm in front of a layer
// with the residual's addition, and the gated norm behind it, each with an optional 8-bit output.
//
// All of it is bound by memory: every value is read once into registers, and sums and maxima go over lanes.
#include <cuda_fp8.h>

#include "layer_kernels.h"

namespace rssm {

namespace {

// ------------------------------------------------------------------------------------------ inputs of the gated delta rule

constexpr int kItems = 4;  // heads' vectors that 16 lanes have on their way at a time

// 8 values as T, 16-byte aligned (32 for fp32)
__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
  *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8]) {
  *reinterpret_cast<uint4 *>(p) =
      make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7]));
}

// Vectors: 16 lanes a head of 128, q / sqrt(sum q^2 + eps).  The blocks behind them: one thread a gate,
//   alpha = exp(-exp(A_log) softplus(a + bias)),  beta = 1 / (1 + exp(-b)).
template <typename T>
__global__ void __launch_bounds__(256) gdn_inputs_kernel(GdnInputsArgs a, int vector_blocks) {
  if ((int)blockIdx.x >= vector_blocks) {
    const long long n = (long long)a.rows * a.H;
    const long long i = (long long)(blockIdx.x - vector_blocks) * 256 + threadIdx.x;
    if (i >= n) return;
    const int row = (int)(i / a.H), h = (int)(i % a.H);
    const float z = to_f32(static_cast<const T *>(a.a)[row * a.stride_a + h]) + a.bias[h];
    const float b = to_f32(static_cast<const T *>(a.b)[row * a.stride_b + h]);
    const float softplus = fmaxf(z, 0.f) + log1pf(expf(-fabsf(z)));
    // a NaN in z would be lost in the maximum
    a.alpha[i] = expf(-expf(a.A_log[h]) * (z == z ? softplus : z));
    a.beta[i] = 1.f / (1.f + expf(-b));
    return;
  }
  const int l16 = threadIdx.x & 15, rep = a.out_heads / a.Hk;
  const long long items = 2LL * a.rows * a.Hk, step = (long long)vector_blocks * 16;
  for (long long first = (long long)blockIdx.x * 16 + (threadIdx.x >> 4); first - (threadIdx.x >> 4) < items; first += kItems * step) {
    float v[kItems][8];
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
      const long long e = first + j * step;
      if (e < items) {
        const long long rh = e >> 1;
        const int row = (int)(rh / a.Hk), h = (int)(rh % a.Hk);
        const T *src = static_cast<const T *>(e & 1 ? a.k : a.q) + row * (e & 1 ? a.stride_k : a.stride_q) + h * kCols;
        load8(src + 8 * l16, v[j]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] = 0.f;
      }
    }
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(v[j][i], v[j][i], sum);
#pragma unroll
      for (int off = 8; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      const float r = 1.f / sqrtf(sum + a.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] *= r;
      const long long e = first + j * step;
      if (e < items) {
        const long long rh = e >> 1;
        const int row = (int)(rh / a.Hk), h = (int)(rh % a.Hk);
        T *dst = static_cast<T *>(e & 1 ? a.k_out : a.q_out) + ((size_t)row * a.out_heads + (size_t)h * rep) * kCols + 8 * l16;
        for (int i = 0; i < rep; ++i) store8(dst + i * kCols, v[j]);
      }
    }
  }
}

// ------------------------------------------------------------------------------------------ norms

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

constexpr int kMaxWarps = 32;

struct NormShared {
  float warp[kMaxWarps];
  float max[kMaxWarps];
};

// A team of threads takes one row, 8 columns a thread in each of NV rounds: a warp (kWarp; eight teams a block), or the
// whole block.
template <bool kWarp>
__device__ __forceinline__ float team_sum(float v, float *words) {
  v = warp_sum(v);
  if (kWarp) return v;
  const int warps = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) words[threadIdx.x >> 5] = v;
  __syncthreads();
  v = (int)(threadIdx.x & 31) < warps ? words[threadIdx.x & 31] : 0.f;
  return warp_sum(v);
}

__device__ __forceinline__ float lanes_max(float v, int lanes) {
  for (int off = lanes >> 1; off >= 1; off >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}

template <bool kWarp>
__device__ __forceinline__ float team_max(float v, float *words) {
  v = lanes_max(v, 32);
  if (kWarp) return v;
  const int warps = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) words[threadIdx.x >> 5] = v;
  __syncthreads();
  v = (int)(threadIdx.x & 31) < warps ? words[threadIdx.x & 31] : 0.f;
  return lanes_max(v, 32);
}

__device__ __forceinline__ void load_any(const void *p, size_t at, int dtype, float (&v)[8]) {
  if (dtype == RSSM_BF16) load8(static_cast<const __nv_bfloat16 *>(p) + at, v);
  else load8(static_cast<const float *>(p) + at, v);
}
__device__ __forceinline__ void store_any(void *p, size_t at, int dtype, const float (&v)[8]) {
  if (dtype == RSSM_BF16) store8(static_cast<__nv_bfloat16 *>(p) + at, v);
  else store8(static_cast<float *>(p) + at, v);
}

// Two bytes a code pair; values beyond 448 become 448, NaN stays
__device__ __forceinline__ uint2 e4m3_codes(const float (&v)[8], float by) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i] * by, v[4 * i + 1] * by), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2] * by, v[4 * i + 3] * by), __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | (hi << 16);
  }
  return make_uint2(w[0], w[1]);
}

// the scale that maps `most` to 448 (a NaN stays one; not below the normal numbers, so that its inverse is finite)
__device__ __forceinline__ float scale_of(float most) { return max_nan(most / 448.f, 1.17549435e-38f); }

template <bool kGated, bool kWarp, int NV>
__global__ void __launch_bounds__(kWarp ? 256 : 1024) norm_kernel(NormArgs a) {
  __shared__ NormShared sh;
  extern __shared__ float parts[];  // groups that are neither the row nor within a warp: sums of 8 columns, sums of groups
  const int team = kWarp ? 32 : blockDim.x, t = kWarp ? threadIdx.x & 31 : threadIdx.x;
  const long long row = kWarp ? (long long)blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x;
  if (kWarp && row >= a.rows) return;
  const int vecs = a.columns >> 3;
  float h[NV][8], z[kGated ? NV : 1][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = i * team + t;
#pragma unroll
    for (int j = 0; j < 8; ++j) h[i][j] = 0.f;
    if (c < vecs) load_any(a.x, (size_t)row * a.stride_x + 8 * c, a.x_dtype, h[i]);
  }
  if (kGated) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * team + t;
#pragma unroll
      for (int j = 0; j < 8; ++j) z[i][j] = 0.f;
      if (c < vecs) load_any(a.gate, (size_t)row * a.stride_gate + 8 * c, a.gate_dtype, z[i]);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        z[i][j] = z[i][j] / (1.f + expf(-z[i][j]));
        if (!a.norm_first) h[i][j] *= z[i][j];
      }
  } else if (a.residual) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * team + t;
      if (c < vecs) {
        float r[8];
        load_any(a.residual, (size_t)row * a.stride_residual + 8 * c, a.x_dtype, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] += r[j];
        // rounded once for the next addition; the norm below takes the sum itself
        store_any(a.residual, (size_t)row * a.stride_residual + 8 * c, a.x_dtype, h[i]);
      }
    }
  }
  float sq[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    sq[i] = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) sq[i] = fmaf(h[i][j], h[i][j], sq[i]);
  }
  const float inv_n = 1.f / (float)a.group;
  if (a.group == a.columns) {
    float sum = sq[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) sum += sq[i];
    sum = team_sum<kWarp>(sum, sh.warp);
    const float r = 1.f / sqrtf(sum * inv_n + a.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) sq[i] = r;
  } else if (a.group <= 256 && (a.group & (a.group - 1)) == 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      for (int off = a.group >> 4; off >= 1; off >>= 1) sq[i] += __shfl_xor_sync(0xffffffffu, sq[i], off);
      sq[i] = 1.f / sqrtf(sq[i] * inv_n + a.eps);
    }
  } else {
    float *part = kWarp ? parts + (threadIdx.x >> 5) * 2 * vecs : parts, *group = part + vecs;
    const int per = a.group >> 3, groups = a.columns / a.group;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (i * team + t < vecs) part[i * team + t] = sq[i];
    if (kWarp) __syncwarp(); else __syncthreads();
    for (int g = t >> 5; g < groups; g += team >> 5) {
      float sum = 0.f;
      for (int c = t & 31; c < per; c += 32) sum += part[g * per + c];
      sum = warp_sum(sum);
      if ((t & 31) == 0) group[g] = 1.f / sqrtf(sum * inv_n + a.eps);
    }
    if (kWarp) __syncwarp(); else __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) sq[i] = i * team + t < vecs ? group[(i * team + t) / per] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = i * team + t;
    if (c < vecs) {
      float w[8];
      load_any(a.weight, a.weight_columns == a.columns ? 8 * c : 8 * c % a.weight_columns, a.weight_dtype, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        h[i][j] = h[i][j] * sq[i] * (a.offset + w[j]);
        if (kGated && a.norm_first) h[i][j] *= z[i][j];
      }
    }
  }
  if (a.scale == RSSM_SCALE_NONE) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (i * team + t < vecs) store_any(a.out, (size_t)row * a.columns + 8 * (i * team + t), a.out_dtype, h[i]);
    return;
  }
  float most[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    most[i] = 0.f;
    if (i * team + t < vecs)
#pragma unroll
      for (int j = 0; j < 8; ++j) most[i] = max_nan(most[i], fabsf(h[i][j]));
  }
  float scale[NV];
  if (a.scale == RSSM_SCALE_ROW) {
    float m = most[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) m = max_nan(m, most[i]);
    m = scale_of(team_max<kWarp>(m, sh.max));
    if (t == 0) a.scales[row] = m;
#pragma unroll
    for (int i = 0; i < NV; ++i) scale[i] = m;
  } else {
    const int blocks = (vecs + 15) >> 4;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      scale[i] = scale_of(lanes_max(most[i], 16));
      const int c = i * team + t;
      if ((c & 15) == 0 && c < vecs) a.scales[row * blocks + (c >> 4)] = scale[i];
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = i * team + t;
    if (c < vecs)
      *reinterpret_cast<uint2 *>(static_cast<unsigned char *>(a.out) + (size_t)row * a.columns + 8 * c) =
          e4m3_codes(h[i], 1.f / scale[i]);
  }
}

template <bool kGated, bool kWarp, int NV>
cudaError_t launch_norm_as(const NormArgs &a, int threads, cudaStream_t stream) {
  const bool general = a.group != a.columns && (a.group > 256 || (a.group & (a.group - 1)));
  const size_t smem = general ? (size_t)(kWarp ? 8 : 1) * 2 * (a.columns >> 3) * 4 : 0;
  const unsigned grid = kWarp ? (unsigned)((a.rows + 7) / 8) : (unsigned)a.rows;
  norm_kernel<kGated, kWarp, NV><<<grid, kWarp ? 256 : threads, smem, stream>>>(a);
  return cudaGetLastError();
}

template <bool kGated>
cudaError_t launch_norm_type(const NormArgs &a, cudaStream_t stream) {
  const int vecs = a.columns >> 3;
  if (vecs <= 32) return launch_norm_as<kGated, true, 1>(a, 0, stream);
  if (vecs <= 64) return launch_norm_as<kGated, true, 2>(a, 0, stream);
  if (vecs <= 128) return launch_norm_as<kGated, true, 4>(a, 0, stream);
  auto threads = [&](int nv) { return ((vecs + nv - 1) / nv + 31) / 32 * 32; };
  if (vecs <= 2048) return launch_norm_as<kGated, false, 2>(a, threads(2), stream);
  return launch_norm_as<kGated, false, 4>(a, threads(4), stream);
}

}  // namespace

cudaError_t launch_gdn_inputs(const GdnInputsArgs &a, int esz, int num_sms, cudaStream_t stream) {
  const long long vectors = (2LL * a.rows * a.Hk + 15) / 16, gates = ((long long)a.rows * a.H + 255) / 256;
  const long long full = (vectors + kItems - 1) / kItems;
  const long long vb = vectors <= 8LL * num_sms ? vectors : full < 8LL * num_sms ? 8LL * num_sms : full;
  if (esz == 2) gdn_inputs_kernel<__nv_bfloat16><<<(unsigned)(vb + gates), 256, 0, stream>>>(a, (int)vb);
  else gdn_inputs_kernel<float><<<(unsigned)(vb + gates), 256, 0, stream>>>(a, (int)vb);
  return cudaGetLastError();
}

cudaError_t launch_norm(const NormArgs &a, bool gated, cudaStream_t stream) {
  return gated ? launch_norm_type<true>(a, stream) : launch_norm_type<false>(a, stream);
}

}  // namespace rssm
