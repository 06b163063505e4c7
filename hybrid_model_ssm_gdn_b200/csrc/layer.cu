// layer.cu -- what stands between a layer's projections: the inputs of the gated delta rule, the norm in front of a layer
// with the residual's addition, and the gated norm behind it, each with an optional 8-bit output.
//
// All of it is bound by memory: every value is read once into registers, and sums and maxima go over lanes.  A thread issues
// all of its loads before it widens the first (16384 rows, us: inputs of 16 heads 107 -> 48, 87 % of the measured copy bandwidth;
// norm of 4096 columns with residual to E4M3 112 -> 76, 95 %; gated 141 -> 90, 80 % beside 31 instructions a value).
#include <cuda_fp8.h>

#include "layer_kernels.h"
#include "lowprec.cuh"

namespace rssm {

namespace {

// ------------------------------------------------------------------------------------------ inputs of the gated delta rule

constexpr int kItems = kInputItems;

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// Eight values as they lie in memory: loads of several are issued before the first is widened.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { a = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void wide(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float *p) {
    a = *reinterpret_cast<const float4 *>(p);
    b = *reinterpret_cast<const float4 *>(p + 4);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void wide(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};

// 8 values as T, 16-byte aligned
__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
  *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8]) {
  *reinterpret_cast<uint4 *>(p) =
      make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7]));
}

// Vectors: 16 lanes a head of 128, q / sqrt(sum q^2 + eps); a block takes a.vector_rows rows of q or of k.  The blocks behind
// them take a.gate_rows rows, one thread a gate:
//   alpha = exp(-exp(A_log) softplus(a + bias)),  beta = 1 / (1 + exp(-b)).
template <typename T>
__global__ void __launch_bounds__(256) gdn_inputs_kernel(GdnInputsArgs a, unsigned vector_blocks) {
  if (blockIdx.x >= 2 * vector_blocks) {
    const int row0 = (int)(blockIdx.x - 2 * vector_blocks) * a.gate_rows;
    const int n = min(a.gate_rows, a.rows - row0) * a.H;
    for (int i = threadIdx.x; i < n; i += 256) {
      const int dr = (unsigned)i / (unsigned)a.H, h = i - dr * a.H;
      const long long row = row0 + dr;
      const float z = to_f32(static_cast<const T *>(a.a)[row * a.stride_a + h]) + a.bias[h];
      const float b = to_f32(static_cast<const T *>(a.b)[row * a.stride_b + h]);
      const float softplus = fmaxf(z, 0.f) + log1pf(expf(-fabsf(z)));
      // a NaN in z would be lost in the maximum
      a.alpha[row * a.H + h] = expf(-expf(a.A_log[h]) * (z == z ? softplus : z));
      a.beta[row * a.H + h] = 1.f / (1.f + expf(-b));
    }
    return;
  }
  const bool key = blockIdx.x >= vector_blocks;
  const int row0 = (int)(key ? blockIdx.x - vector_blocks : blockIdx.x) * a.vector_rows;
  const int n = min(a.vector_rows, a.rows - row0) * a.Hk;
  const int l16 = threadIdx.x & 15, rep = a.out_heads / a.Hk;
  const T *in = static_cast<const T *>(key ? a.k : a.q) + 8 * l16;
  T *out = static_cast<T *>(key ? a.k_out : a.q_out) + 8 * l16;
  const long long stride = key ? a.stride_k : a.stride_q;
  for (int first = 0; first < n; first += 16 * kItems) {
    Raw8<T> raw[kItems];
    int dr[kItems], h[kItems];
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
      const int e = first + 16 * j + (threadIdx.x >> 4);
      dr[j] = (unsigned)e / (unsigned)a.Hk;
      h[j] = e - dr[j] * a.Hk;
      raw[j].zero();
      if (e < n) raw[j].load(in + (row0 + dr[j]) * stride + h[j] * kCols);
    }
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
      float v[8], sum = 0.f;
      raw[j].wide(v);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(v[i], v[i], sum);
#pragma unroll
      for (int off = 8; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      const float r = rsqrtf(sum + a.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= r;
      if (first + 16 * j + (int)(threadIdx.x >> 4) < n) {
        T *dst = out + ((size_t)(row0 + dr[j]) * a.out_heads + (size_t)h[j] * rep) * kCols;
        for (int i = 0; i < rep; ++i) store8(dst + i * kCols, v);
      }
    }
  }
}

// ------------------------------------------------------------------------------------------ norms

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

template <int kLanes>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int off = kLanes >> 1; off >= 1; off >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}

template <bool kWarp>
__device__ __forceinline__ float team_max(float v, float *words) {
  v = lanes_max<32>(v);
  if (kWarp) return v;
  const int warps = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) words[threadIdx.x >> 5] = v;
  __syncthreads();
  v = (int)(threadIdx.x & 31) < warps ? words[threadIdx.x & 31] : 0.f;
  return lanes_max<32>(v);
}

// Eight values of a type known at run time: the loads do not wait for their widening
struct RawAny {
  uint4 a, b;
  __device__ __forceinline__ void load(const void *p, size_t at, int dtype) {
    const uint4 *from = reinterpret_cast<const uint4 *>(static_cast<const char *>(p) + at * (dtype == RSSM_BF16 ? 2 : 4));
    a = from[0];
    if (dtype != RSSM_BF16) b = from[1];
  }
  __device__ __forceinline__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void wide(int dtype, float (&v)[8]) const {
    if (dtype == RSSM_BF16) {
      Raw8<__nv_bfloat16> r;
      r.a = a;
      r.wide(v);
    } else {
      const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
    }
  }
};
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
__device__ __forceinline__ float scale_of(float most) { return max_nan(most * (1.f / 448.f), 1.17549435e-38f); }

// h silu(gate) = h z / (1 + e^-z).  For bf16 gates and outputs of 16 or 8 bits e^-z = 2^(-z log2 e) takes the argument's rounding
// along, up to |z| 2^-23 of itself (1e-6 at z = -8, where silu is -3e-3; it fades for positive z); 2^x and the reciprocal add
// 2 units in the last place.  The library's expf and __fdividef take 8 instructions a value more, of which the kernel has 30 in
// all: 100 us against 87 at 16384 x 4096.  Past e^-z = 2^126 (z < -87.3) the reciprocal is 0, where silu is below 2^-119.
// Otherwise (kFine) to within 2^-20 of the value down to its last bits: with h = 2^(-|z| log2 e / 2), whose argument's rounding is
// given back to first order, silu is z / (1 + h^2) for z > 0 and z h^2 / (1 + h^2) for z < 0, which stays in the normal range as
// long as the result has bits.
template <bool kFine, typename T>
__device__ __forceinline__ void times_silu(const Raw8<T> &gate, float (&h)[8]) {
  constexpr float kL = 1.4426950408889634f, kRest = (float)(1.4426950408889634 - (double)kL), kLn2 = 0.69314718f;
  float z[8];
  gate.wide(z);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float e, r;
    if constexpr (kFine) {
      const float a = fminf(fabsf(z[j]), 1e6f), t = a * (-0.5f * kL);
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
      e = fmaf(e * kLn2, fmaf(a, -0.5f * kRest, fmaf(a, -0.5f * kL, -t)), e);
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaf(e, e, 1.f)));
      const float q = z[j] * r;
      h[j] *= z[j] < 0.f ? q * e * e : q;
    } else {
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z[j] * -kL));
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
      h[j] *= z[j] * r;
    }
  }
}

template <typename T, typename TG, bool kGated, bool kFine, bool kWarp, int NV>
__global__ void __launch_bounds__(kWarp ? 256 : 512) norm_kernel(NormArgs a) {
  __shared__ NormShared sh;
  extern __shared__ float parts[];  // groups that are neither the row nor within a warp: sums of 8 columns, sums of groups
  const int team = kWarp ? 32 : blockDim.x, t = kWarp ? threadIdx.x & 31 : threadIdx.x;
  const long long row = kWarp ? (long long)blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x;
  if (kWarp && row >= a.rows) return;
  const int vecs = a.columns >> 3;
  const T *x = static_cast<const T *>(a.x) + row * a.stride_x;
  // 8 columns of this thread in round i; threads past the row's end read its last 8 once more and add nothing
  auto at = [&](int i) { return 8 * min(i * team + t, vecs - 1); };
  auto inside = [&](int i) { return i * team + t < vecs; };
  float h[NV][8];
  Raw8<T> in[NV];
  Raw8<TG> gate[kGated ? NV : 1];
#pragma unroll
  for (int i = 0; i < NV; ++i) in[i].load(x + at(i));
  if (kGated) {
    const TG *g = static_cast<const TG *>(a.gate) + row * a.stride_gate;
#pragma unroll
    for (int i = 0; i < NV; ++i) gate[i].load(g + at(i));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      in[i].wide(h[i]);
      if (!a.norm_first) times_silu<kFine>(gate[i], h[i]);
    }
  } else if (a.residual) {
    T *residual = static_cast<T *>(a.residual) + row * a.stride_residual;
    Raw8<T> add[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) add[i].load(residual + at(i));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float r[8];
      in[i].wide(h[i]);
      add[i].wide(r);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] += r[j];
      // rounded once for the next addition; the norm below takes the sum itself
      if (inside(i)) store8(residual + at(i), h[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) in[i].wide(h[i]);
  }
  RawAny weight[NV];
  auto load_weight = [&]() {
    const unsigned wc = a.weight_columns;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const unsigned c = at(i);
      weight[i].load(a.weight, wc == (unsigned)a.columns ? c : (wc & (wc - 1)) == 0 ? c & (wc - 1) : c % wc, a.weight_dtype);
    }
  };
  if (kWarp) load_weight();  // on its way during the sums; a whole block's registers are better spent on another row
  float sq[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    sq[i] = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) sq[i] = fmaf(h[i][j], h[i][j], sq[i]);
    if (!inside(i)) sq[i] = 0.f;
  }
  const float inv_n = 1.f / (float)a.group;
  if (a.group == a.columns) {
    float sum = sq[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) sum += sq[i];
    sum = team_sum<kWarp>(sum, sh.warp);
    const float r = rsqrtf(sum * inv_n + a.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) sq[i] = r;
  } else if (a.group <= 256 && (a.group & (a.group - 1)) == 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      for (int off = a.group >> 4; off >= 1; off >>= 1) sq[i] += __shfl_xor_sync(0xffffffffu, sq[i], off);
      sq[i] = rsqrtf(sq[i] * inv_n + a.eps);
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
      if ((t & 31) == 0) group[g] = rsqrtf(sum * inv_n + a.eps);
    }
    if (kWarp) __syncwarp(); else __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) sq[i] = i * team + t < vecs ? group[(i * team + t) / per] : 0.f;
  }
  if (!kWarp) load_weight();
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float w[8];
    weight[i].wide(a.weight_dtype, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) h[i][j] = h[i][j] * sq[i] * (a.offset + w[j]);
    if (kGated && a.norm_first) times_silu<kFine>(gate[i], h[i]);
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
#pragma unroll
    for (int j = 0; j < 8; ++j) most[i] = max_nan(most[i], fabsf(h[i][j]));
    if (!inside(i)) most[i] = 0.f;
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
      scale[i] = scale_of(lanes_max<16>(most[i]));
      const int c = i * team + t;
      if ((c & 15) == 0 && c < vecs) a.scales[row * blocks + (c >> 4)] = scale[i];
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = i * team + t;
    if (c < vecs)
      *reinterpret_cast<uint2 *>(static_cast<unsigned char *>(a.out) + (size_t)row * a.columns + 8 * c) =
          e4m3_codes(h[i], __fdividef(1.f, scale[i]));
  }
}

template <typename T, typename TG, bool kGated, bool kFine, bool kWarp, int NV>
cudaError_t launch_norm_as(const NormArgs &a, cudaStream_t stream) {
  const int vecs = a.columns >> 3, threads = kWarp ? 256 : ((vecs + NV - 1) / NV + 31) / 32 * 32;
  const bool general = a.group != a.columns && (a.group > 256 || (a.group & (a.group - 1)));
  const size_t smem = general ? (size_t)(kWarp ? 8 : 1) * 2 * vecs * 4 : 0;
  const unsigned grid = kWarp ? (unsigned)((a.rows + 7) / 8) : (unsigned)a.rows;
  norm_kernel<T, TG, kGated, kFine, kWarp, NV><<<grid, threads, smem, stream>>>(a);
  return cudaGetLastError();
}

template <typename T, typename TG, bool kGated, bool kFine>
cudaError_t launch_norm_type(const NormArgs &a, cudaStream_t stream) {
  const int vecs = a.columns >> 3;
  // Rows of up to 256 columns: a warp each (bf16 with a residual / gated, us: 131072 x 128 37 / 45, as blocks 74 / 74; 65536 x 256
  // 27 / 29 against 39 / 39).  From there on a block a row, 8 columns a thread up to 1024 (65536 x 1024 84 / 78; a warp with 32
  // columns a lane 84 / 96), then 32, gated 16, so that sums and scales, which cost the same for any number of columns, are spread
  // over more (16384 x 4096 to E4M3, 8 / 16 / 32 columns a thread: 88 / 81 / 76; gated 119 / 107 / 117, where 32 leave too few
  // registers for other rows; 4096 x 16384 gated, 32 / 64: 123 / 156).
  if (vecs <= 32) return launch_norm_as<T, TG, kGated, kFine, true, 1>(a, stream);
  if (vecs <= 128) return launch_norm_as<T, TG, kGated, kFine, false, 1>(a, stream);
  constexpr int kFew = kGated ? 2 : 4;
  if (vecs <= 512 * kFew) return launch_norm_as<T, TG, kGated, kFine, false, kFew>(a, stream);
  if (vecs <= 512 * 4) return launch_norm_as<T, TG, kGated, kFine, false, 4>(a, stream);
  return launch_norm_as<T, TG, kGated, kFine, false, 8>(a, stream);
}

}  // namespace

cudaError_t launch_gdn_inputs(const GdnInputsArgs &args, int esz, int num_sms, cudaStream_t stream) {
  GdnInputsArgs a = args;
  const InputsCut cut = cut_inputs(a.rows, a.H, a.Hk, a.rows <= 4 * num_sms);
  a.vector_rows = cut.vectors;
  a.gate_rows = cut.gates;
  const unsigned vb = (unsigned)(((long long)a.rows + a.vector_rows - 1) / a.vector_rows), grid = (unsigned)cut.blocks;
  if (esz == 2) gdn_inputs_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(a, vb);
  else gdn_inputs_kernel<float><<<grid, 256, 0, stream>>>(a, vb);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_norm_in(const NormArgs &a, bool gated, cudaStream_t stream) {
  using bf16 = __nv_bfloat16;
  if (!gated) return launch_norm_type<T, T, false, false>(a, stream);
  if (a.gate_dtype != RSSM_BF16) return launch_norm_type<T, float, true, true>(a, stream);
  if (a.scale == RSSM_SCALE_NONE && a.out_dtype != RSSM_BF16) return launch_norm_type<T, bf16, true, true>(a, stream);
  return launch_norm_type<T, bf16, true, false>(a, stream);
}

cudaError_t launch_norm(const NormArgs &a, bool gated, cudaStream_t stream) {
  return a.x_dtype == RSSM_BF16 ? launch_norm_in<__nv_bfloat16>(a, gated, stream) : launch_norm_in<float>(a, gated, stream);
}

}  // namespace rssm
