// scan.cu -- the Mamba-2 recurrence over whole prompts on CUDA cores (fp32 inputs), and a context's bookkeeping after it.
//
//   S_t = exp(dt_t A_h) S_{t-1} + dt_t x_t B_t^T,   y_t = S_t C_t + D_h x_t
//
// Token by token in fp32: inputs of 24 bits would need six bf16 products for each one of the chunk form.  A warp carries
// 8 rows of one head's state: 16 lanes take 8 columns each (two runs of 4, so that B and C come from shared memory
// without bank conflicts) of 4 rows, 32 fp32 values a lane as packed pairs; a token costs 48 packed operations, five
// 16-byte reads and four shuffles that sum the four rows' columns.  Tokens are staged 16 at a time, the next ones on
// their way.  The chain of tokens sets the time of few prompts, so blocks are as small as it takes to use the SMs.
// Measured: two prompts of 301 tokens in all, 8 heads, 44 to 55 us by the box's clock, 0.2 us a token of the longer one.
#include "prompt_kernels.h"
#include "packed.cuh"

namespace rssm {

namespace {

constexpr int kTok = 16;   // tokens staged at a time

// 16 bytes to shared memory, zeros where `live` is not set
__device__ __forceinline__ void copy16(void *dst, const void *src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(live ? 16 : 0) : "memory");
}

template <int R>
struct Stage {
  float b[kTok][kCols], c[kTok][kCols];
  float x[kTok][R];
  float2 dt[kTok];  // dt, exp(dt A)
};

// R rows of head blockIdx.y from row blockIdx.z * R on
template <int R>
__global__ void __launch_bounds__(4 * R) scan_kernel(ScanArgs a, Prompts pr) {
  __shared__ __align__(16) Stage<R> st[2];
  __shared__ PieceWord found;
  Piece pc;
  const int h = blockIdx.y, row0 = blockIdx.z * R;
  allow_next();
  if (find_piece(pr, blockIdx.x, a.piece_len, pc, &found) != kPieceRun) return;
  const int len = pc.end - pc.begin;
  if (len == 0 && pc.resume) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, l16 = lane & 15;
  const int mine = 8 * warp + 4 * (lane >> 4);  // this lane's four rows within the block
  const int g = h / (a.H / a.G);
  const float A = a.A[h], D = a.D[h];
  const float *xg = static_cast<const float *>(a.x) + ((size_t)pc.begin * a.H + h) * a.P + row0;
  const float *Bg = static_cast<const float *>(a.Bin) + ((size_t)pc.begin * a.G + g) * kCols;
  const float *Cg = static_cast<const float *>(a.C) + ((size_t)pc.begin * a.G + g) * kCols;
  const float *dg = static_cast<const float *>(a.dt) + (size_t)pc.begin * a.H + h;

  float dt_next = 0.f;
  auto fetch = [&](int t0, Stage<R> &s) {
    for (int e = tid; e < kTok * (kCols / 4); e += 4 * R) {
      const int t = e / (kCols / 4), n = 4 * (e % (kCols / 4));
      const bool live = t0 + t < len;
      const size_t at = live ? (size_t)(t0 + t) * a.G * kCols + n : 0;
      copy16(&s.b[t][n], Bg + at, live);
      copy16(&s.c[t][n], Cg + at, live);
    }
    for (int e = tid; e < kTok * (R / 4); e += 4 * R) {
      const int t = e / (R / 4), r = 4 * (e % (R / 4));
      const bool live = t0 + t < len && row0 + r < a.P;  // P is a multiple of 8
      copy16(&s.x[t][r], xg + (live ? (size_t)(t0 + t) * a.H * a.P + r : 0), live);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (tid < kTok) dt_next = t0 + tid < len ? dg[(size_t)(t0 + tid) * a.H] : 0.f;
  };
  if (len > 0) fetch(0, st[0]);

  // columns 4 l16 + 64 i + 2 j .. of row mine + r in s[r][2 i + j]
  f2 s[4][4];
  float *Sg = a.S + (((size_t)pc.slot * a.H + h) * a.P + row0 + mine) * kCols + 4 * l16;
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float4 v = f4zero();
      if (pc.resume && row0 + mine + r < a.P) v = *reinterpret_cast<const float4 *>(Sg + r * kCols + 64 * i);
      s[r][2 * i] = pack2(v.x, v.y);
      s[r][2 * i + 1] = pack2(v.z, v.w);
    }
  // after the sums below, this lane holds row `out` of the block
  const int out = mine + 2 * ((lane >> 3) & 1) + ((lane >> 2) & 1);
  const bool write = (lane & 3) == 0 && row0 + out < a.P;
  float *yg = a.y + ((size_t)pc.begin * a.H + h) * a.P + row0 + out;

  for (int t0 = 0, k = 0; t0 < len; t0 += kTok, k ^= 1) {
    if (tid < kTok) st[k].dt[tid] = make_float2(dt_next, expf(dt_next * A));
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    if (t0 + kTok < len) fetch(t0 + kTok, st[k ^ 1]);  // read last before the barrier above
    const Stage<R> &m = st[k];
    const int n = min(kTok, len - t0);
#pragma unroll 4
    for (int t = 0; t < n; ++t) {
      const float2 d = m.dt[t];
      const float4 x = *reinterpret_cast<const float4 *>(&m.x[t][mine]);
      const float4 b0 = *reinterpret_cast<const float4 *>(&m.b[t][4 * l16]);
      const float4 b1 = *reinterpret_cast<const float4 *>(&m.b[t][4 * l16 + 64]);
      const float4 c0 = *reinterpret_cast<const float4 *>(&m.c[t][4 * l16]);
      const float4 c1 = *reinterpret_cast<const float4 *>(&m.c[t][4 * l16 + 64]);
      const f2 bb[4] = {pack2(b0.x, b0.y), pack2(b0.z, b0.w), pack2(b1.x, b1.y), pack2(b1.z, b1.w)};
      const f2 cc[4] = {pack2(c0.x, c0.y), pack2(c0.z, c0.w), pack2(c1.x, c1.y), pack2(c1.z, c1.w)};
      const float xs[4] = {x.x, x.y, x.z, x.w};
      const f2 da = pack2(d.y, d.y);
      float v[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float w = d.x * xs[r];
        const f2 ww = pack2(w, w);
        f2 acc = pack2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[r][i] = fma2(ww, bb[i], mul2(da, s[r][i]));
          acc = fma2(s[r][i], cc[i], acc);
        }
        float lo, hi;
        unpack2(acc, lo, hi);
        v[r] = lo + hi;
      }
      // the 16 lanes' sums: two rows are handed over, then one
      const bool up = lane & 8;
      const float a0 = (up ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, up ? v[0] : v[2], 8);
      const float a1 = (up ? v[3] : v[1]) + __shfl_xor_sync(0xffffffffu, up ? v[1] : v[3], 8);
      const bool up2 = lane & 4;
      float y = (up2 ? a1 : a0) + __shfl_xor_sync(0xffffffffu, up2 ? a0 : a1, 4);
      y += __shfl_xor_sync(0xffffffffu, y, 2);
      y += __shfl_xor_sync(0xffffffffu, y, 1);
      if (write) yg[(size_t)(t0 + t) * a.H * a.P] = fmaf(D, m.x[t][out], y);
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (row0 + mine + r < a.P)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float4 v;
        unpack2(s[r][2 * i], v.x, v.y);
        unpack2(s[r][2 * i + 1], v.z, v.w);
        *reinterpret_cast<float4 *>(Sg + r * kCols + 64 * i) = v;
      }
}

// NaN in the rows of y [total][row] whose prompts a scan refuses; blockIdx.x: the prompt.  A launch of its own, where the
// call asks for it: as a branch at the start of the scan kernels it changed their loops' code, and two prompts of 301
// tokens in all (fp32) took 16 % longer, 48 resumed ones of 31 tokens each 4.5 %.
__global__ void __launch_bounds__(256) refuse_kernel(Prompts pr, float *y, int row) {
  __shared__ PieceWord found;
  Piece pc;
  const PieceStatus status = find_piece(pr, blockIdx.x, pr.total + 1, pc, &found);
  if (status != kPieceRun) refuse(pr, status, pc, pr.total, y, row, blockIdx.y, gridDim.y);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // what comes after this launch comes after the scan
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

template <int R>
cudaError_t launch_rows(const ScanArgs &a, const Prompts &pr, int pieces, cudaStream_t stream) {
  scan_kernel<R><<<dim3(pieces, a.H, (a.P + R - 1) / R), 4 * R, 0, stream>>>(a, pr);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_scan(const ScanArgs &a, const Prompts &pr, int num_sms, cudaStream_t stream) {
  const int pieces = prompt_pieces(pr.total, pr.nseq, a.piece_len);
  // All 64 rows a block share one staging of B and C; 8 rows, one warp, spread few heads and prompts over the SMs.
  const long long heads = (long long)pieces * a.H;
  if (heads >= 2LL * num_sms) return launch_rows<64>(a, pr, pieces, stream);
  if (heads * 2 >= num_sms) return launch_rows<16>(a, pr, pieces, stream);
  return launch_rows<8>(a, pr, pieces, stream);
}

cudaError_t launch_refuse(const Prompts &pr, float *y, int row, int num_sms, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(pr.nseq, max(1, 2 * num_sms / pr.nseq));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];  // it runs beside the scan's last blocks (1 us a call, 4 us after them): the rows are others
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, refuse_kernel, pr, y, row);
}

cudaError_t launch_prefill_meta(const Prompts &pr, const int4 *meta_in, int4 *meta_out, unsigned char *skip, int H,
                                int *err, cudaStream_t stream) {
  prefill_meta_kernel<<<(pr.nslots + 127) / 128, 128, 0, stream>>>(pr, meta_in, meta_out, skip, H, err);
  return cudaGetLastError();
}

}  // namespace rssm
