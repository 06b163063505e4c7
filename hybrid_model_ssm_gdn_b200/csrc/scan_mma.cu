// scan_mma.cu -- the Mamba-2 scan over short prompts (bf16 inputs).
//
// The chunk form of scan_tc.cu with chunks of 16 tokens and everything in registers: a block of four warps carries one
// head, each warp 16 rows of its state as fp32 accumulators of m16n8k16 (64 registers), which are at the same time, cut
// into two bf16 pieces, the right operand of C S^T.  M's accumulators are the left operand of M X the same way, and X,
// loaded transposed once, is both the right operand of M X and, weighted, the left one of the state's update.
//
// A prompt of a few tokens is a read and a write of its state (64 KB a head) around little work.  Here four blocks share
// an SM, so one block's state is on its way while the others compute; a block of the 128-token kernel has an SM to
// itself and pays its start, its loads and its whole chunk of products one after the other: 48 resumed prompts of 31
// tokens on average (128 heads; 483 MB) take 160 us here and 342 us there.  Per token this kernel costs more (every 16
// tokens the state is cut anew, and mma.sync runs at a quarter of tcgen05's rate), so longer prompts go there.  What
// bounds it: the LSU data path (59 % busy) and a block's latency; DRAM 33 %, tensor pipe 25 %.
#include "prompt_kernels.h"
#include "packed.cuh"

namespace rssm {

namespace {

constexpr int kTok = 16;
constexpr int kPitchX = 144, kPitchN = 272;  // bytes of a row: ldmatrix reads eight rows without bank conflicts
constexpr float kLog2e = 1.4426950408889634f;

struct __align__(16) MmaStage {
  unsigned char x[kTok * kPitchX], b[kTok * kPitchN], c[kTok * kPitchN];
};

__device__ __forceinline__ float exp2_ftz(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// 16 bytes to shared memory, zeros where `live` is not set
__device__ __forceinline__ void copy16(void *dst, const void *src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(live ? 16 : 0) : "memory");
}

// whether one of 8 bf16 values is an infinity or no number: times 0 those give no number, all others 0
__device__ __forceinline__ bool not_finite(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
  __nv_bfloat162 s = zero;
  for (const uint32_t v : {a, b, c, d}) s = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&v), zero, s);
  return *reinterpret_cast<const uint32_t *>(&s) & 0x7fff7fffu;
}

// Fragments of X, 16 tokens by 16 values, with values that are not finite as 0, and of Y with NaN from the first of them on.
struct Cleared {
  float y[8];
  uint32_t x[4];
};
__device__ __noinline__ Cleared clear_not_finite(float y0, float y1, float y2, float y3, float y4, float y5, float y6, float y7,
                                                 uint32_t x0, uint32_t x1, uint32_t x2, uint32_t x3) {
  Cleared f{{y0, y1, y2, y3, y4, y5, y6, y7}, {x0, x1, x2, x3}};
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int from = kTok;  // first such token of column 8 i + g
#pragma unroll
    for (int k = 3; k >= 0; --k) {
      uint32_t &w = f.x[2 * i + (k >> 1)];
      const uint32_t mask = k & 1 ? 0x7f800000u : 0x7f80u;
      if ((w & mask) == mask) {
        from = 2 * t + (k & 1) + 8 * (k >> 1);
        w &= k & 1 ? 0xffffu : 0xffff0000u;
      }
    }
    from = min(from, __shfl_xor_sync(0xffffffffu, from, 1));
    from = min(from, __shfl_xor_sync(0xffffffffu, from, 2));
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int col = __shfl_sync(0xffffffffu, from, 4 * (2 * t + e));
      if (g >= col) f.y[4 * i + e] = __int_as_float(0x7fffffff);
      if (g + 8 >= col) f.y[4 * i + 2 + e] = __int_as_float(0x7fffffff);
    }
  }
  return f;
}

__global__ void __launch_bounds__(128, 4) scan_mma_kernel(ScanArgs a, Prompts pr) {
  __shared__ MmaStage st[2];
  __shared__ PieceWord found;
  Piece pc;
  allow_next();
  if (find_piece(pr, blockIdx.x, a.piece_len, pc, &found) != kPieceRun) return;
  const int h = blockIdx.y, len = pc.end - pc.begin;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int group = h / (a.H / a.G), p0 = 16 * warp;
  float *Sg = a.S + ((size_t)pc.slot * a.H + h) * a.P * kCols;
  if (len == 0 && pc.resume) return;

  // rows of P < 64 are shorter than the tile: the rest of X stays zero
  for (int i = tid; i < 2 * kTok * kPitchX / 16; i += 128) {
    MmaStage &s = st[i / (kTok * kPitchX / 16)];
    *reinterpret_cast<uint4 *>(s.x + i % (kTok * kPitchX / 16) * 16) = make_uint4(0, 0, 0, 0);
  }
  __syncthreads();

  const __nv_bfloat16 *xg = static_cast<const __nv_bfloat16 *>(a.x) + ((size_t)pc.begin * a.H + h) * a.P;
  const __nv_bfloat16 *bg = static_cast<const __nv_bfloat16 *>(a.Bin) + ((size_t)pc.begin * a.G + group) * kCols;
  const __nv_bfloat16 *cg = static_cast<const __nv_bfloat16 *>(a.C) + ((size_t)pc.begin * a.G + group) * kCols;
  const __nv_bfloat16 *dg = static_cast<const __nv_bfloat16 *>(a.dt) + (size_t)pc.begin * a.H + h;
  auto fetch = [&](int t0, MmaStage &s) {
    {
      const int row = tid >> 3, col = tid & 7;
      const bool live = t0 + row < len;
      if (8 * col < a.P)
        copy16(s.x + row * kPitchX + 16 * col, xg + (live ? (size_t)(t0 + row) * a.H * a.P + 8 * col : 0), live);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = (tid >> 4) + 8 * i, col = tid & 15;
      const bool live = t0 + row < len;
      const size_t at = live ? (size_t)(t0 + row) * a.G * kCols + 8 * col : 0;
      copy16(s.b + row * kPitchN + 16 * col, bg + at, live);
      copy16(s.c + row * kPitchN + 16 * col, cg + at, live);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto fetch_dt = [&](int t0) {
    const int at = t0 + (lane & 15);
    return at < len ? __bfloat162float(dg[(size_t)at * a.H]) : 0.f;
  };
  float dt = 0.f;
  if (len > 0) {
    fetch(0, st[0]);
    dt = fetch_dt(0);
  }
  const float lA = a.A[h] * kLog2e, D = a.D[h];

  // S[p0 + g (+ 8)][8 j + 2 t ..] in s[j][0..1] ([2..3])
  float s[16][4];
  const bool top = p0 + g < a.P, bottom = p0 + g + 8 < a.P;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    float2 u = make_float2(0.f, 0.f), v = u;
    if (pc.resume && top) u = *reinterpret_cast<const float2 *>(Sg + (size_t)(p0 + g) * kCols + 8 * j + 2 * t);
    if (pc.resume && bottom) v = *reinterpret_cast<const float2 *>(Sg + (size_t)(p0 + g + 8) * kCols + 8 * j + 2 * t);
    s[j][0] = u.x; s[j][1] = u.y; s[j][2] = v.x; s[j][3] = v.y;
  }
  bool carried = pc.resume;
  float *yg = a.y + ((size_t)pc.begin * a.H + h) * a.P + p0;

  for (int t0 = 0, k0 = 0; t0 < len; t0 += kTok, k0 ^= 1) {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    // sums of dt (lanes 0-15: tokens, 16-31 the same again) and this thread's rows and columns of the decays
    float c = dt;
#pragma unroll
    for (int off = 1; off < 16; off <<= 1) {
      const float v = __shfl_up_sync(0xffffffffu, c, off, 16);
      if ((lane & 15) >= off) c += v;
    }
    const float total = __shfl_sync(0xffffffffu, c, 15);
    const float weight = exp2_ftz(lA * (total - c)) * dt;
    float cj[2], ci[4], di[4], wi[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) cj[i] = __shfl_sync(0xffffffffu, c, g + 8 * i);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int from = 2 * t + (i & 1) + 8 * (i >> 1);
      ci[i] = __shfl_sync(0xffffffffu, c, from);
      di[i] = __shfl_sync(0xffffffffu, dt, from);
      wi[i] = __shfl_sync(0xffffffffu, weight, from);
    }
    const MmaStage &m = st[k0];
    if (t0 + kTok < len) {  // the other stage was read before the barrier above
      fetch(t0 + kTok, st[k0 ^ 1]);
      dt = fetch_dt(t0 + kTok);
    }
    if (p0 < a.P) {
      // G = C B^T and C S^T, 16 columns n at a time
      float G[2][4] = {}, y[2][4] = {};
      const int r8 = lane & 7, q = lane >> 3;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        uint32_t c0, c1, c2, c3, b0, b1, b2, b3;
        ldmatrix_x4(m.c + ((q & 1) * 8 + r8) * kPitchN + 32 * k + (q >> 1) * 16, c0, c1, c2, c3);
        ldmatrix_x4(m.b + ((q >> 1) * 8 + r8) * kPitchN + 32 * k + (q & 1) * 16, b0, b1, b2, b3);
        mma_16816(G[0], c0, c1, c2, c3, b0, b1);
        mma_16816(G[1], c0, c1, c2, c3, b2, b3);
        if (carried) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {  // rows p0 + g, p0 + g + 8 of the state
            uint32_t h0, l0, h1, l1;
            cut2(pack2(s[2 * k][2 * i], s[2 * k][2 * i + 1]), h0, l0);
            cut2(pack2(s[2 * k + 1][2 * i], s[2 * k + 1][2 * i + 1]), h1, l1);
            mma_16816(y[i], c0, c1, c2, c3, h0, h1);
            mma_16816(y[i], c0, c1, c2, c3, l0, l1);
          }
        }
      }
      // M in two pieces; rows j = g, g + 8, columns i as in ci
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float rise = exp2_ftz(lA * cj[r]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // D x in fp32: on M's diagonal it would be cut like M
          const uint32_t x = *reinterpret_cast<const uint32_t *>(m.x + (g + 8 * r) * kPitchX + 2 * (p0 + 8 * i + 2 * t));
          y[i][2 * r] = fmaf(D, __uint_as_float(x << 16), y[i][2 * r] * rise);
          y[i][2 * r + 1] = fmaf(D, __uint_as_float(x & 0xffff0000u), y[i][2 * r + 1] * rise);
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float v[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int i = 2 * half + e, col = 2 * t + e + 8 * half, row = g + 8 * r;
            const float w = G[half][2 * r + e] * (exp2_ftz(lA * (cj[r] - ci[i])) * di[i]);
            v[e] = col <= row ? w : 0.f;
          }
          cut2(pack2(v[0], v[1]), hi[r + 2 * half], lo[r + 2 * half]);
        }
      }
      uint32_t x0, x1, x2, x3;  // tokens 0-7, 8-15 of rows p0.., of rows p0 + 8..
      const unsigned char *xt = m.x + ((q & 1) * 8 + r8) * kPitchX + 2 * p0 + (q >> 1) * 16;
      ldmatrix_x4_trans(xt, x0, x1, x2, x3);
      // M's zeros above the diagonal would carry values that are not finite to earlier tokens: they enter as 0, and the
      // outputs from the first of them on become NaN here
      const bool odd = __any_sync(0xffffffffu, not_finite(x0, x1, x2, x3));
      if (odd) {
        const Cleared f = clear_not_finite(y[0][0], y[0][1], y[0][2], y[0][3], y[1][0], y[1][1], y[1][2], y[1][3], x0, x1, x2, x3);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i >> 2][i & 3] = f.y[i];
        x0 = f.x[0]; x1 = f.x[1]; x2 = f.x[2]; x3 = f.x[3];
      }
      mma_16816(y[0], hi[0], hi[1], hi[2], hi[3], x0, x1);
      mma_16816(y[0], lo[0], lo[1], lo[2], lo[3], x0, x1);
      mma_16816(y[1], hi[0], hi[1], hi[2], hi[3], x2, x3);
      mma_16816(y[1], lo[0], lo[1], lo[2], lo[3], x2, x3);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int at = t0 + g + 8 * r;
        if (at < len) {
          float *yp = yg + (size_t)at * a.H * a.P + 2 * t;
          if (p0 + 2 * t < a.P) __stcs(reinterpret_cast<float2 *>(yp), make_float2(y[0][2 * r], y[0][2 * r + 1]));
          if (p0 + 8 + 2 * t < a.P) __stcs(reinterpret_cast<float2 *>(yp + 8), make_float2(y[1][2 * r], y[1][2 * r + 1]));
        }
      }
      // S <- decay S + (weighted X)^T B
      if (odd) ldmatrix_x4_trans(xt, x0, x1, x2, x3);
      uint32_t xh[4], xl[4];
      const uint32_t xs[4] = {x0, x2, x1, x3};  // as a left operand: rows g, g + 8 of tokens 0-7, then of 8-15
#pragma unroll
      for (int i = 0; i < 4; ++i)
        cut2(mul2(pack2(xs[i] << 16, xs[i] & 0xffff0000u), pack2(wi[i & 2], wi[(i & 2) + 1])), xh[i], xl[i]);
      const float decay = exp2_ftz(lA * total);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        uint32_t b0, b1, b2, b3;
        ldmatrix_x4_trans(m.b + ((q & 1) * 8 + r8) * kPitchN + 32 * k + (q >> 1) * 16, b0, b1, b2, b3);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[2 * k][i] *= decay;
          s[2 * k + 1][i] *= decay;
        }
        mma_16816(s[2 * k], xh[0], xh[1], xh[2], xh[3], b0, b1);
        mma_16816(s[2 * k], xl[0], xl[1], xl[2], xl[3], b0, b1);
        mma_16816(s[2 * k + 1], xh[0], xh[1], xh[2], xh[3], b2, b3);
        mma_16816(s[2 * k + 1], xl[0], xl[1], xl[2], xl[3], b2, b3);
      }
      carried = true;
    }
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    if (top) *reinterpret_cast<float2 *>(Sg + (size_t)(p0 + g) * kCols + 8 * j + 2 * t) = make_float2(s[j][0], s[j][1]);
    if (bottom)
      *reinterpret_cast<float2 *>(Sg + (size_t)(p0 + g + 8) * kCols + 8 * j + 2 * t) = make_float2(s[j][2], s[j][3]);
  }
}

}  // namespace

cudaError_t launch_scan_mma(const ScanArgs &a, const Prompts &pr, cudaStream_t stream) {
  scan_mma_kernel<<<dim3(prompt_pieces(pr.total, pr.nseq, a.piece_len), a.H), 128, 0, stream>>>(a, pr);
  return cudaGetLastError();
}

}  // namespace rssm
