// scan.cu -- the Mamba-2 recurrence over whole prompts, on CUDA cores.
//
//   S_t = exp(dt_t A_h) S_{t-1} + dt_t x_t B_t^T,   y_t = S_t C_t + D_h x_t
//
// A block carries R rows of one head's state along one prompt: four threads a row, each with 32 of its 128 columns in
// registers as packed fp32 pairs, so a token costs a thread 48 packed multiply-adds and the columns' sum two shuffles.
// Tokens are staged in shared memory 16 at a time.
#include "kernels.h"
#include "packed.cuh"

namespace rssm {

namespace {

constexpr int kTok = 16;   // tokens staged at a time

template <int R>
struct Stage {
  float b[kTok][kCols], c[kTok][kCols];
  float x[kTok][R];
  float dt[kTok], decay[kTok];
};

template <typename TI, int R>
__global__ void __launch_bounds__(4 * R) scan_kernel(ScanArgs a, Prompts pr) {
  __shared__ __align__(16) Stage<R> st;
  __shared__ int found;
  Piece pc;
  const int h = blockIdx.y, row0 = blockIdx.z * R;
  if (!find_piece(pr, blockIdx.x, a.piece_len, pc, &found)) return;
  const int len = pc.end - pc.begin;
  if (pc.first >= len && pc.index > 0) return;
  const int tid = threadIdx.x, q = tid & 3, row = row0 + (tid >> 2);
  const bool live = row < a.P;
  const int g = h / (a.H / a.G);
  const float A = a.A[h], D = a.D[h];

  // column 4 (q + 4 i) + j of the row sits in s[2 i + j / 2]
  f2 s[16];
  float *Sg = a.S + (((size_t)pc.slot * a.H + h) * a.P + row) * kCols;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float4 v = f4zero();
    if (pc.resume && live) v = *reinterpret_cast<const float4 *>(Sg + 4 * (q + 4 * i));
    s[2 * i] = pack2(v.x, v.y);
    s[2 * i + 1] = pack2(v.z, v.w);
  }
  const TI *xg = reinterpret_cast<const TI *>(a.x), *Bg = reinterpret_cast<const TI *>(a.Bin);
  const TI *Cg = reinterpret_cast<const TI *>(a.C), *dg = reinterpret_cast<const TI *>(a.dt);

  for (int t0 = 0; t0 < len; t0 += kTok) {
    const int m = min(kTok, len - t0);
    __syncthreads();
    for (int e = tid; e < m * (kCols / 4); e += 4 * R) {
      const int t = e / (kCols / 4), n = 4 * (e % (kCols / 4));
      const size_t tok = (size_t)(pc.begin + t0 + t) * a.G + g;
      *reinterpret_cast<float4 *>(&st.b[t][n]) = load4(Bg + tok * kCols + n);
      *reinterpret_cast<float4 *>(&st.c[t][n]) = load4(Cg + tok * kCols + n);
    }
    for (int e = tid; e < m * R; e += 4 * R) {
      const int t = e / R, r = e % R;
      st.x[t][r] = row0 + r < a.P ? to_f32(xg[((size_t)(pc.begin + t0 + t) * a.H + h) * a.P + row0 + r]) : 0.f;
    }
    if (tid < m) {
      const float dt = to_f32(dg[(size_t)(pc.begin + t0 + tid) * a.H + h]);
      st.dt[tid] = dt;
      st.decay[tid] = expf(dt * A);
    }
    __syncthreads();
    for (int t = 0; t < m; ++t) {
      const float x = st.x[t][tid >> 2], w = st.dt[t] * x, da = st.decay[t];
      const f2 w2 = pack2(w, w), d2 = pack2(da, da);
      f2 acc0 = pack2(0.f, 0.f), acc1 = acc0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 b = *reinterpret_cast<const float4 *>(&st.b[t][4 * (q + 4 * i)]);
        const float4 c = *reinterpret_cast<const float4 *>(&st.c[t][4 * (q + 4 * i)]);
        s[2 * i] = fma2(w2, pack2(b.x, b.y), mul2(d2, s[2 * i]));
        s[2 * i + 1] = fma2(w2, pack2(b.z, b.w), mul2(d2, s[2 * i + 1]));
        acc0 = fma2(s[2 * i], pack2(c.x, c.y), acc0);
        acc1 = fma2(s[2 * i + 1], pack2(c.z, c.w), acc1);
      }
      float y0, y1, y2, y3;
      unpack2(acc0, y0, y1);
      unpack2(acc1, y2, y3);
      float y = (y0 + y1) + (y2 + y3);
      y += __shfl_xor_sync(0xffffffffu, y, 1);
      y += __shfl_xor_sync(0xffffffffu, y, 2);
      if (q == 0 && live) a.y[((size_t)(pc.begin + t0 + t) * a.H + h) * a.P + row] = fmaf(D, x, y);
    }
  }
  if (live && (len > 0 || !pc.resume)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float4 v;
      unpack2(s[2 * i], v.x, v.y);
      unpack2(s[2 * i + 1], v.z, v.w);
      *reinterpret_cast<float4 *>(Sg + 4 * (q + 4 * i)) = v;
    }
  }
}

// The bookkeeping of a context after a prefill: one thread a sequence looks for the prompt that names it.
__global__ void prefill_meta_kernel(Prompts pr, const int4 *meta_in, int4 *meta_out, unsigned char *skip, int H, int *err) {
  bool bad = false;
  for (int i = threadIdx.x; i < pr.nseq; i += blockDim.x) {
    if (prompt_bad(pr, i)) {
      record_error(err, i, RSSM_DEV_PROMPT);
      bad = true;
    }
  }
  bad = __syncthreads_or(bad);
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= pr.nslots) return;
  const int4 m = meta_in[b];
  int4 o = m;
  int which = -1, times = 0;
  if (!pr.slots) {
    if (b < pr.nseq) {
      which = b;
      times = 1;
    }
  } else {
    for (int i = 0; i < pr.nseq; ++i) {
      if (pr.slots[i] == b) {
        which = i;
        ++times;
      }
    }
  }
  if (!bad && times > 1) record_error(err, which, RSSM_DEV_PROMPT);
  if (!bad && times == 1) {
    const bool resume = pr.resume && pr.resume[which];
    if (resume && m.z != 0) {
      record_error(err, b, RSSM_DEV_PENDING);
    } else if (resume && m.x != 0) {
      record_error(err, b, RSSM_DEV_BUFFERED);
    } else if (!resume || pr.off[which + 1] > pr.off[which]) {
      o = make_int4(0, m.y + 1, 0, 0);
      if (skip)
        for (int h = 0; h < H; ++h) skip[(size_t)b * H + h] = 0;
    }
  }
  meta_out[b] = o;
}

template <typename TI>
cudaError_t launch_scan_t(const ScanArgs &a, const Prompts &pr, int num_sms, cudaStream_t stream) {
  const int pieces = prompt_pieces(pr.total, pr.nseq, a.piece_len);
  // 64 rows a block share one staging of B and C; 16 rows give four times the blocks when heads and prompts are few
  if ((long long)pieces * a.H >= num_sms || a.P <= 16) {
    scan_kernel<TI, 64><<<dim3(pieces, a.H, (a.P + 63) / 64), 256, 0, stream>>>(a, pr);
  } else {
    scan_kernel<TI, 16><<<dim3(pieces, a.H, (a.P + 15) / 16), 64, 0, stream>>>(a, pr);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_scan(const ScanArgs &a, const Prompts &pr, int num_sms, cudaStream_t stream) {
  return launch_scan_t<float>(a, pr, num_sms, stream);
}

cudaError_t launch_prefill_meta(const Prompts &pr, const int4 *meta_in, int4 *meta_out, unsigned char *skip, int H,
                                int *err, cudaStream_t stream) {
  prefill_meta_kernel<<<(pr.nslots + 127) / 128, 128, 0, stream>>>(pr, meta_in, meta_out, skip, H, err);
  return cudaGetLastError();
}

}  // namespace rssm
