// gdn_tc.cu -- the gated delta rule over packed prompts on the tensor cores (bf16 inputs).
//
// Chunks of Q = 64 tokens.  With D_ji the product of alpha over i < l <= j within the chunk, g_j = D over its first j + 1
// tokens, and S the state before it, u_j = beta_j (v_j - alpha_j S_{j-1} k_j) solves a triangular system:
//   A_ji = [i < j] beta_j D_ji (k_j . k_i),   T = (I + A)^-1,   M_ji = [i <= j] D_ji (q_j . k_i)
//   R = diag(beta) (V - diag(g) K S^T)         U = T R
//   Y = q_scale (diag(g) Q S^T + M U)          S <- g_Q S + (diag(g_Q / g) U)^T K
// A block carries one head along one prompt; lanes of tensor memory are rows of the state (d_v), so R, U and Y are held
// transposed, and S stays on the chip.
#include "prompt_kernels.h"
#include "packed.cuh"
#include "tcgen05.cuh"
#include "tensor_map.h"

namespace rssm {

namespace {

constexpr int Q = kGdnChunk;
constexpr int kHalf = Q * 128;  // bytes of a tile: 64 rows of 64 bf16
constexpr int kStages = 3;      // of q and k: one chunk in the chain of the state, one in front of it, one on its way
constexpr uint32_t kColR = 0, kColU = 64, kColY = 128, kColG = 192, kColD = 256, kColS = 384;
constexpr int kChain = 16;                                    // warps: lanes' quarter w % 4, columns' quarter w / 4
constexpr int kWarpPrep = 16, kWarpLoad = 20, kWarpState = 21, kWarpGram = 22;
constexpr int kGdnThreads = 23 * 32;
constexpr int kByLength = 64;

struct __align__(16) Table {
  float rise[Q], fall[Q], beta[Q];  // g_j, g_Q / g_j
  float carry;                      // g_Q
  int tokens;                       // of the chunk, or up to the first whose k, alpha or beta is not finite
};

struct GdnShared {
  unsigned char in[kStages][4][kHalf];  // k, q of columns 0..63, k, q of columns 64..127
  unsigned char V[2][2][kHalf];
  unsigned char T[2][2][kHalf], M[2][2][kHalf];  // hi, lo; row = token j
  unsigned char A[2][kHalf];
  float diag[4][16][20];
  Table tab[2];
  float alpha[Q], prefix[Q], tot[4];
  int first[128];  // per row of the state, the first token of the prompt whose v is not finite
  uint64_t full_kq[kStages], free_kq[kStages], full_v[2], free_v[2], full_t[2], free_t[2];
  uint64_t ks_done, qs_done, u_done, d_done, y_done, g_done, g_free, drained[2];
  uint64_t s_ready, r_ready, u_ready, y_free;
  uint32_t tmem;
  int abort, not_finite, bad;
  PieceWord found;
};
constexpr int kGdnSmem = (int)sizeof(GdnShared);
static_assert(kGdnSmem <= 227 * 1024, "shared memory of a block");

struct GdnTcArgs {
  int H, Hk, R, by_prompt;
  int by_length;            // hand out the prompts by length (at most kByLength of them)
  float q_scale;
  const float *alpha, *beta;  // [total][H]
  float *S;                 // [nslots or nseq][H][R][128]
  float *y;                 // [total][H][R]
  int *err;                 // may be null
  long long wait_cycles;
  int withhold;             // test hook: no block loads k and q of this chunk (-1: off)
};

struct Waiter {
  GdnShared *sh;
  int *err;
  int slot;
  WaitSpec ws;
  __device__ __forceinline__ void gave_up() const {
    *(volatile int *)&sh->abort = 1;
    if (err) record_error(err, slot, RSSM_DEV_TIMEOUT);
  }
  __device__ __forceinline__ void operator()(uint64_t &bar, int phase) const {
    if (!mbar_wait_or_abort(&bar, phase & 1, &sh->abort, ws)) gave_up();
  }
  // by a whole warp, whose lanes stay together
  __device__ __forceinline__ void warp(uint64_t &bar, int phase) const {
    if (__all_sync(0xffffffffu, mbar_try_wait(&bar, phase & 1, ws.hint_ns))) return;
    const long long t0 = clock64();
    while (!__all_sync(0xffffffffu, mbar_try_wait(&bar, phase & 1, ws.hint_ns))) {
      const bool late = clock64() - t0 > ws.limit;
      if (late) gave_up();
      if (__any_sync(0xffffffffu, late || *(volatile int *)&sh->abort)) return;
    }
  }
};

// after a warp's writes to tensor memory, or its reads of what is to be overwritten
__device__ __forceinline__ void warp_arrive(uint64_t &bar, int lane) {
  tm_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(&bar);
}

__device__ __forceinline__ void prep_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool prep_sync_or(bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v)
      : "memory");
  return r != 0;
}

// 16 bytes of columns col .. col + 7 of a tile's row
__device__ __forceinline__ unsigned char *at_tile(unsigned char *tile, int row, int col) {
  return tile + row * 128 + (((col >> 3) ^ (row & 7)) << 4);
}

// operands of m16n8k16 from a block of 16 x 16 of a tile at (row, col): as the left operand, as the left one transposed, and
// as the right one of two tiles of 8 columns whose columns are the block's rows
__device__ __forceinline__ void load_left(unsigned char *tile, int row, int col, int lane, uint32_t (&f)[4]) {
  ldmatrix_x4(at_tile(tile, row + (lane & 15), col + 8 * (lane >> 4)), f[0], f[1], f[2], f[3]);
}
__device__ __forceinline__ void load_left_t(unsigned char *tile, int row, int col, int lane, uint32_t (&f)[4]) {
  ldmatrix_x4_trans(at_tile(tile, row + (lane & 7) + 8 * (lane >> 4), col + (lane & 8)), f[0], f[1], f[2], f[3]);
}
__device__ __forceinline__ void load_right(unsigned char *tile, int row, int col, int lane, uint32_t (&f)[4]) {
  ldmatrix_x4(at_tile(tile, row + (lane & 7) + 8 * (lane >> 4), col + (lane & 8)), f[0], f[1], f[2], f[3]);
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  mma_16816(d, a[0], a[1], a[2], a[3], b0, b1);
}

// X^T (+)= Z^T B^T for blocks of 16 x 16, Z at (zr, zc) of T and B at (br, bc) of A, in two pieces each; x[n]: columns 8 n ..
__device__ __forceinline__ void block_x(unsigned char (*T)[kHalf], int zr, int zc, unsigned char (*A)[kHalf], int br, int bc,
                                        int lane, float (&x)[2][4]) {
  uint32_t zh[4], zl[4], bh[4], bl[4];
  load_left_t(T[0], zr, zc, lane, zh);
  load_left_t(T[1], zr, zc, lane, zl);
  load_right(A[0], br, bc, lane, bh);
  load_right(A[1], br, bc, lane, bl);
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    mma(x[n], zh, bl[2 * n], bl[2 * n + 1]);
    mma(x[n], zl, bh[2 * n], bh[2 * n + 1]);
    mma(x[n], zh, bh[2 * n], bh[2 * n + 1]);
  }
}
// T block (+)= W X for W at (wr, wc) of T and X from block_x
__device__ __forceinline__ void block_t(unsigned char (*T)[kHalf], int wr, int wc, int lane, const float (&x)[2][4],
                                        float (&t)[2][4]) {
  uint32_t wh[4], wl[4], h[2][2], l[2][2];
  load_left(T[0], wr, wc, lane, wh);
  load_left(T[1], wr, wc, lane, wl);
#pragma unroll
  for (int n = 0; n < 2; ++n)  // the accumulators of X^T are the right operand of W X
#pragma unroll
    for (int k = 0; k < 2; ++k) split_bf16x2(x[k][2 * n], x[k][2 * n + 1], h[n][k], l[n][k]);
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    mma(t[n], wh, l[n][0], l[n][1]);
    mma(t[n], wl, h[n][0], h[n][1]);
    mma(t[n], wh, h[n][0], h[n][1]);
  }
}
__device__ __forceinline__ void store_block(unsigned char (*T)[kHalf], int row, int col, int lane, const float (&t)[2][4]) {
  const int g = lane >> 2, p = 2 * (lane & 3);
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t h, l;
      split_bf16x2(-t[n][2 * i], -t[n][2 * i + 1], h, l);
      *reinterpret_cast<uint32_t *>(at_tile(T[0], row + g + 8 * i, col + 8 * n) + 2 * p) = h;
      *reinterpret_cast<uint32_t *>(at_tile(T[1], row + g + 8 * i, col + 8 * n) + 2 * p) = l;
    }
}

// A wait gave up: nothing that looks like a result stays.
__device__ __noinline__ void overwrite(const GdnTcArgs &a, GdnShared &sh, int h, float *S) {
  __syncthreads();
  const volatile PieceWord &w = sh.found;
  const float nan = __int_as_float(0x7fffffff);
  for (int i = threadIdx.x; i < a.R * kCols; i += kGdnThreads) S[i] = nan;
  for (int t = w.begin + threadIdx.x / 32; t < w.end; t += kGdnThreads / 32)
    for (int r = threadIdx.x % 32; r < a.R; r += 32) a.y[((size_t)t * a.H + h) * a.R + r] = nan;
}

__global__ void __launch_bounds__(kGdnThreads, 1)
    gdn_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v, const __grid_constant__ GdnTcArgs a, Prompts pr) {
  extern __shared__ __align__(1024) unsigned char raw[];
  GdnShared &sh = *reinterpret_cast<GdnShared *>(raw);
  if (smem_u32(raw) & 1023u) {
    if (threadIdx.x == 0 && a.err) record_error(a.err, 0, RSSM_DEV_TIMEOUT);
    return;
  }
  allow_next();
  int number = blockIdx.x / a.H;
  const int h = blockIdx.x % a.H;
  if (a.by_length) {  // the longest first: the last blocks to finish are short ones
    int *lens = reinterpret_cast<int *>(sh.diag);
    if (threadIdx.x < pr.nseq) lens[threadIdx.x] = pr.off[threadIdx.x + 1] - pr.off[threadIdx.x];
    __syncthreads();
    if (threadIdx.x < pr.nseq) {
      const int mine = lens[threadIdx.x];
      int rank = 0;
      for (int j = 0; j < pr.nseq; ++j) rank += lens[j] > mine || (lens[j] == mine && j < (int)threadIdx.x);
      if (rank == number) sh.found.seq = threadIdx.x;
    }
    __syncthreads();
    number = sh.found.seq;
    __syncthreads();
  }
  Piece pc;
  if (find_piece(pr, number, pr.total + 1, pc, &sh.found) != kPieceRun) return;
  const int ntok = pc.end - pc.begin, t0 = pc.begin, chunks = (ntok + Q - 1) / Q;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  float *S = a.S + ((size_t)(a.by_prompt ? pc.seq : pc.slot) * a.H + h) * a.R * kCols;
  if (ntok == 0) {
    if (!pc.resume)
      for (int i = tid; i < a.R * kCols / 4; i += kGdnThreads) reinterpret_cast<float4 *>(S)[i] = f4zero();
    return;
  }
  if (tid == 0) {
    uint64_t *one[] = {&sh.full_kq[0], &sh.full_kq[1], &sh.full_kq[2], &sh.free_kq[0], &sh.free_kq[1], &sh.free_kq[2],
                       &sh.full_v[0], &sh.full_v[1], &sh.free_t[0], &sh.free_t[1], &sh.ks_done, &sh.qs_done, &sh.u_done,
                       &sh.d_done, &sh.y_done, &sh.g_done, &sh.drained[0], &sh.drained[1]};
    for (uint64_t *b : one) mbar_init(b, 1);
    uint64_t *prep[] = {&sh.full_t[0], &sh.full_t[1], &sh.g_free};
    for (uint64_t *b : prep) mbar_init(b, 4);
    uint64_t *team[] = {&sh.free_v[0], &sh.free_v[1], &sh.s_ready, &sh.r_ready, &sh.u_ready, &sh.y_free};
    for (uint64_t *b : team) mbar_init(b, kChain);
    sh.abort = sh.not_finite = 0;
    fence_barrier_init();
  }
  if (tid < 128) sh.first[tid] = 0x7fffffff;
  if (warp == kWarpLoad) tm_alloc(&sh.tmem, 512);
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  const uint32_t tm = sh.tmem;
  const Waiter wait{&sh, a.err, pc.slot, {a.wait_cycles, 0}};

  if (warp == kWarpLoad) {
    if (lane == 0) {
      const int hk = h / (a.H / a.Hk), halves = a.R > 64 ? 2 : 1;
      auto stopped = [&] { return *(volatile int *)&sh.abort != 0; };
      int asked_kq = 0, asked_v = 0;  // chunks whose loads are on their way or done
      for (int c = 0; c < chunks; ++c) {
        const int s = c % kStages, t = t0 + c * Q;
        if (c >= kStages) wait(sh.free_kq[s], c / kStages - 1);
        if (stopped() || c == a.withhold) break;
        mbar_arrive_expect_tx(&sh.full_kq[s], 4 * kHalf);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          tma_load_2d(sh.in[s][2 * half], &map_k, hk * kCols + 64 * half, t, &sh.full_kq[s]);
          tma_load_2d(sh.in[s][2 * half + 1], &map_q, hk * kCols + 64 * half, t, &sh.full_kq[s]);
        }
        asked_kq = c + 1;
        if (c >= 2) wait(sh.free_v[c & 1], (c >> 1) - 1);
        if (stopped()) break;
        mbar_arrive_expect_tx(&sh.full_v[c & 1], halves * kHalf);
        for (int half = 0; half < halves; ++half)
          tma_load_3d(sh.V[c & 1][half], &map_v, 64 * half, h, t, &sh.full_v[c & 1]);
        asked_v = c + 1;
      }
      // No copy outlives the block: the last phase of each barrier that was asked for.
      for (int c = max(0, asked_kq - kStages); c < asked_kq; ++c) mbar_wait(&sh.full_kq[c % kStages], (c / kStages) & 1, wait.ws);
      for (int c = max(0, asked_v - 2); c < asked_v; ++c) mbar_wait(&sh.full_v[c & 1], (c >> 1) & 1, wait.ws);
    }
    __syncwarp();
  } else if (warp == kWarpState || warp == kWarpGram) {
    // The products: the whole warp goes through the steps, on values the compiler knows to be the same in every lane.
    const uint32_t leader = lane == 0, td = __shfl_sync(0xffffffffu, tm, 0);
    const int n = __shfl_sync(0xffffffffu, chunks, 0);
    constexpr uint32_t shape = mma_shape(128, 64, false, false), shape_d = mma_shape(128, 128, false, true);
    constexpr uint32_t kStep = (2 * kHalf) >> 4, kStage = (4 * kHalf) >> 4;  // descriptor units between column halves, stages
    const uint32_t dk = tile_desc(sh.in[0][0], 16);
    int s = 0, turn = 0;  // c % kStages, c / kStages
    if (warp == kWarpGram) {
      for (int c = 0; c < n; ++c) {
        wait.warp(sh.full_kq[s], turn);
        if (c > 0) wait.warp(sh.g_free, c - 1);
        tm_fence_after();
        const uint32_t k0 = dk + s * kStage;
#pragma unroll
        for (int k = 0; k < 8; ++k) {  // rows of k, then of q
          const int at = (k >> 2) * kStep + 2 * (k & 3);
          mma_ss(td + kColG, k0 + at, k0 + at, shape, k > 0, leader);
        }
        mma_commit(&sh.g_done, leader);
        if (++s == kStages) s = 0, ++turn;
      }
      mma_commit(&sh.drained[1], leader);
      mbar_wait(&sh.drained[1], 0, wait.ws);
    } else {
      const uint32_t dkn = tile_desc(sh.in[0][0], 2 * kHalf);  // MN-major, two tiles
      const uint32_t dT = tile_desc(sh.T[0][0], 16), dM = tile_desc(sh.M[0][0], 16);
      constexpr uint32_t kPiece = kHalf >> 4, kBuffer = (2 * kHalf) >> 4;
      for (int c = 0; c < n; ++c) {
        const int b = c & 1;
        const uint32_t k0 = dk + s * kStage, q0 = k0 + (kHalf >> 4);
        wait.warp(sh.full_kq[s], turn);
        wait.warp(sh.s_ready, c);
        tm_fence_after();
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int p = 0; p < 2; ++p)
            mma_ts(td + kColR, td + kColS + 16 * k + 8 * p, k0 + (k >> 2) * kStep + 2 * (k & 3), shape, k > 0 || p > 0, leader);
        mma_commit(&sh.ks_done, leader);
        if (c > 0) wait.warp(sh.y_free, c - 1);
        tm_fence_after();
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int p = 0; p < 2; ++p)
            mma_ts(td + kColY, td + kColS + 16 * k + 8 * p, q0 + (k >> 2) * kStep + 2 * (k & 3), shape, k > 0 || p > 0, leader);
        mma_commit(&sh.qs_done, leader);
        wait.warp(sh.full_t[b], c >> 1);
        wait.warp(sh.r_ready, c);
        tm_fence_after();
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // pieces (hi, lo), (lo, hi), (hi, hi)
          const uint32_t r = td + kColR + 16 * k, t = dT + b * kBuffer + 2 * k;
          mma_ts(td + kColU, r, t + kPiece, shape, k > 0, leader);
          mma_ts(td + kColU, r + 8, t, shape, 1, leader);
          mma_ts(td + kColU, r, t, shape, 1, leader);
        }
        mma_commit(&sh.u_done, leader);
        wait.warp(sh.u_ready, c);
        tm_fence_after();
#pragma unroll
        for (int k = 0; k < 4; ++k)  // 16 token rows are 2048 bytes
#pragma unroll
          for (int p = 0; p < 2; ++p)
            mma_ts(td + kColD, td + kColR + 16 * k + 8 * p, dkn + s * kStage + 128 * k, shape_d, k > 0 || p > 0, leader);
        mma_commit(&sh.d_done, leader);
        mma_commit(&sh.free_kq[s], leader);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t u = td + kColU + 16 * k, m = dM + b * kBuffer + 2 * k;
          mma_ts(td + kColY, u, m + kPiece, shape, k > 0, leader);
          mma_ts(td + kColY, u + 8, m, shape, 1, leader);
          mma_ts(td + kColY, u, m, shape, 1, leader);
        }
        mma_commit(&sh.y_done, leader);
        mma_commit(&sh.free_t[b], leader);
        if (++s == kStages) s = 0, ++turn;
      }
      mma_commit(&sh.drained[0], leader);
      mbar_wait(&sh.drained[0], 0, wait.ws);
    }
    __syncwarp();
  } else if (warp >= kWarpPrep) {
    // A, T and M of a chunk, a chunk ahead of the state: lanes 0..63 of the Gram matrix are k_j . k_i, the others q_j . k_i
    const int pw = warp - kWarpPrep, p = tid - 32 * kWarpPrep, j = p & 63, bj = j >> 4, jj = j & 15;
    const bool of_k = p < 64;
    const uint32_t lanes = (uint32_t)(32 * pw) << 16;
    for (int i = p; i < 2 * 2 * 2 * kHalf / 16; i += 128)  // blocks above the diagonal stay zero
      reinterpret_cast<uint4 *>(sh.T[0][0])[i] = make_uint4(0, 0, 0, 0);
    const float *ag = a.alpha + (size_t)t0 * a.H + h, *bg = a.beta + (size_t)t0 * a.H + h;
    float alpha_next = 1.f, beta_next = 0.f;
    auto fetch = [&](int c) {
      const int t = c * Q + j;
      alpha_next = 1.f;
      beta_next = 0.f;  // a token behind the end changes nothing
      if (of_k && t < ntok) {
        alpha_next = ag[(size_t)t * a.H];
        beta_next = bg[(size_t)t * a.H];
      }
    };
    fetch(0);
    for (int c = 0; c < chunks; ++c) {
      const int b = c & 1, valid = min(Q, ntok - c * Q);
      const float al = alpha_next, be = beta_next;
      if (c + 1 < chunks) fetch(c + 1);
      float up = al, down = al;  // products within the block of 16: up to this token, and behind it
      if (of_k) {
#pragma unroll
        for (int off = 1; off < 16; off <<= 1) {
          const float u = __shfl_up_sync(0xffffffffu, up, off, 16), d = __shfl_down_sync(0xffffffffu, down, off, 16);
          if (jj >= off) up *= u;
          if (jj + off < 16) down *= d;
        }
        down = __shfl_down_sync(0xffffffffu, down, 1, 16);
        if (jj == 15) {
          down = 1.f;
          sh.tot[bj] = up;
        }
        sh.alpha[j] = al;
        sh.prefix[j] = up;
      }
      if (valid < Q) {  // rows of k that belong to other prompts must not reach the state, whatever they hold
        wait(sh.full_kq[c % kStages], c / kStages);
        for (int i = p + valid * 8; i < Q * 8; i += 128) {
          *reinterpret_cast<uint4 *>(sh.in[c % kStages][0] + 16 * i) = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4 *>(sh.in[c % kStages][2] + 16 * i) = make_uint4(0, 0, 0, 0);
        }
      }
      prep_sync();
      if (c > 1) wait(sh.free_t[b], (c >> 1) - 1);
      const float tot[4] = {sh.tot[0], sh.tot[1], sh.tot[2], sh.tot[3]};
      Table &tab = sh.tab[b];
      if (of_k) {
        float rise = up, fall = down;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (i < bj) rise *= tot[i];
          if (i > bj) fall *= tot[i];
        }
        tab.rise[j] = rise;
        tab.fall[j] = fall;
        tab.beta[j] = be;
        if (j == 0) {
          tab.carry = (tot[0] * tot[1]) * (tot[2] * tot[3]);
          tab.tokens = valid;
        }
      }
      float f[4];  // product of alpha from the end of a block to this token
      f[3] = 0.f;
      {
        float run = sh.prefix[j];
#pragma unroll
        for (int i = 2; i >= 0; --i) {
          f[i] = i < bj ? run : 0.f;
          if (i < bj) run *= tot[i];
        }
      }
      const float by = of_k ? be : 1.f;
      float seen = fmaf(al, 0.f, be * 0.f);  // stays 0 while what goes into this row is finite
      unsigned char(*const out)[kHalf] = of_k ? sh.A : sh.M[b];
      wait(sh.g_done, c);
      tm_fence_after();
#pragma unroll
      for (int blk = 0; blk < 4; ++blk) {
        if (blk > 2 * (pw & 1) + 1) break;
        uint32_t G[16];
        tm_ld16(tm + lanes + kColG + 16 * blk, G);
        const int own = blk == bj ? jj : -1;                  // column of the diagonal in this block
        // columns of this row; a token behind the end has none (its beta is 0, but its k may hold anything)
        const int most = of_k && j >= valid ? 0 : blk < bj ? 16 : own + (of_k ? 0 : 1);
        float al16[16], v[16];
#pragma unroll
        for (int i = 0; i < 16; i += 4) *reinterpret_cast<float4 *>(al16 + i) = *reinterpret_cast<const float4 *>(&sh.alpha[16 * blk + i]);
        float d = f[blk];
        tm_wait_ld();
#pragma unroll
        for (int i = 15; i >= 0; --i) {
          if (i == own) d = 1.f;
          v[i] = i < most ? by * d * __uint_as_float(G[i]) : 0.f;
          if (i == own) seen = fmaf(__uint_as_float(G[i]), 0.f, seen);
          seen = fmaf(v[i], 0.f, seen);
          d *= al16[i];
        }
        if (of_k && blk == bj) {
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<float4 *>(&sh.diag[bj][jj][i]) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint4 hi, lo;
          cut2(pack2(v[8 * i], v[8 * i + 1]), hi.x, lo.x);
          cut2(pack2(v[8 * i + 2], v[8 * i + 3]), hi.y, lo.y);
          cut2(pack2(v[8 * i + 4], v[8 * i + 5]), hi.z, lo.z);
          cut2(pack2(v[8 * i + 6], v[8 * i + 7]), hi.w, lo.w);
          *reinterpret_cast<uint4 *>(at_tile(out[0], j, 16 * blk + 8 * i)) = hi;
          *reinterpret_cast<uint4 *>(at_tile(out[1], j, 16 * blk + 8 * i)) = lo;
        }
      }
      warp_arrive(sh.g_free, lane);
      if (prep_sync_or(of_k && j < valid && !(seen == 0.f))) {
        // From the first token on whose k, alpha or beta is not finite, the chunk's tokens change nothing; the state warps
        // write NaN for them.  Rows before it have used none of them.
        if (p == 0) sh.bad = Q;
        prep_sync();
        if (of_k && j < valid && !(seen == 0.f)) atomicMin(&sh.bad, j);
        prep_sync();
        const int bad = sh.bad;
        if (of_k && j >= bad) {
          for (int i = 0; i < 16; ++i) sh.diag[bj][jj][i] = 0.f;
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4 *>(at_tile(sh.A[0], j, 8 * i)) = *reinterpret_cast<uint4 *>(at_tile(sh.A[1], j, 8 * i)) =
                make_uint4(0, 0, 0, 0);
        }
        if (p == 0) tab.tokens = bad;
        prep_sync();
      }
      unsigned char(*const T)[kHalf] = sh.T[b];
      {  // blocks on the diagonal by substitution, one a warp, lane = column
        const int col = lane & 15;
        float t[16];
        t[0] = col == 0 ? 1.f : 0.f;
#pragma unroll
        for (int i = 1; i < 16; ++i) {
          float s0 = col == i ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
          for (int l = 0; l < i; l += 4) {
            const float4 r = *reinterpret_cast<const float4 *>(&sh.diag[pw][i][l]);
            s0 = fmaf(-r.x, t[l], s0);
            if (l + 1 < i) s1 = fmaf(-r.y, t[l + 1], s1);
            if (l + 2 < i) s0 = fmaf(-r.z, t[l + 2], s0);
            if (l + 3 < i) s1 = fmaf(-r.w, t[l + 3], s1);
          }
          t[i] = s0 + s1;
        }
        const int lo = lane >> 4;  // lanes 0..15 write the first pieces, the others the second
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const __nv_bfloat16 hi = __float2bfloat16_rn(t[i]);
          const __nv_bfloat16 v = lo ? __float2bfloat16_rn(t[i] - __bfloat162float(hi)) : hi;
          *reinterpret_cast<__nv_bfloat16 *>(at_tile(T[lo], 16 * pw + i, 16 * pw + (col & 8)) + 2 * (col & 7)) = v;
        }
      }
      prep_sync();
      if (!(pw & 1)) {  // T10 = -T11 A10 T00 in both blocks of 32
        const int r0 = 16 * pw;
        float x[2][4] = {}, t[2][4] = {};
        block_x(T, r0, r0, sh.A, r0 + 16, r0, lane, x);
        block_t(T, r0 + 16, r0 + 16, lane, x, t);
        store_block(T, r0 + 16, r0, lane, t);
      }
      prep_sync();
      {  // the same of the whole: block (32 + 16 to, 16 from)
        const int to = pw >> 1, from = pw & 1;
        float t[2][4] = {};
        for (int l = 0; l <= to; ++l) {
          float x[2][4] = {};
          for (int m = from; m < 2; ++m) block_x(T, 16 * m, 16 * from, sh.A, 32 + 16 * l, 16 * m, lane, x);
          block_t(T, 32 + 16 * to, 32 + 16 * l, lane, x, t);
        }
        store_block(T, 32 + 16 * to, 16 * from, lane, t);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.full_t[b]);
    }
  } else {
    // rows of the state: R, U, S, Y
    const int w = warp >> 2, q4 = warp & 3, row = 32 * q4 + lane;
    const uint32_t here = tm + ((uint32_t)(32 * q4) << 16);
    const bool have = row < a.R;
    const float nan = __int_as_float(0x7fffffff);
    float *const Sg = S + (size_t)row * kCols + 32 * w;
    f2 s[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float4 v = f4zero();
      if (pc.resume && have) v = *reinterpret_cast<const float4 *>(Sg + 4 * i);
      s[2 * i] = pack2(v.x, v.y);
      s[2 * i + 1] = pack2(v.z, v.w);
    }
    // pieces of 16 columns of the state: 8 columns of pairs hi, 8 lo
    auto put_state = [&](int half) {
      uint32_t o[16];
#pragma unroll
      for (int i = 0; i < 8; ++i) cut2(s[8 * half + i], o[i], o[8 + i]);
      tm_st16(here + kColS + 32 * w + 16 * half, o);
    };
    put_state(0);
    put_state(1);
    tm_wait_st();
    warp_arrive(sh.s_ready, lane);
    const unsigned char *const vrow = sh.V[0][row >> 6] + 2 * (row & 7);
    const int vchunk = (row & 63) >> 3;
    float *yg = a.y + ((size_t)t0 * a.H + h) * a.R + row;
    for (int c = 0; c < chunks; ++c) {
      const int b = c & 1, valid = min(Q, ntok - c * Q);
      const Table &tab = sh.tab[b];
      wait(sh.full_t[b], c >> 1);
      wait(sh.full_v[b], c >> 1);
      const int tokens = tab.tokens;
      {  // R = beta (v - rise K S^T)
        uint32_t x[16];
        wait(sh.ks_done, c);
        tm_fence_after();
        tm_ld16(here + kColR + 16 * w, x);
        tm_wait_ld();
        f2 r[8];
        f2 seen = pack2(0.f, 0.f);
        const f2 zero = pack2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float4 g = *reinterpret_cast<const float4 *>(&tab.rise[16 * w + i]);
          const float4 be = *reinterpret_cast<const float4 *>(&tab.beta[16 * w + i]);
          float v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int t = 16 * w + i + k;
            const unsigned short bits =
                *reinterpret_cast<const unsigned short *>(vrow + 2 * kHalf * b + t * 128 + ((vchunk ^ (t & 7)) << 4));
            v[k] = have ? __uint_as_float((uint32_t)bits << 16) : 0.f;
          }
          r[i / 2] = mul2(pack2(be.x, be.y), fma2(pack2(-g.x, -g.y), pack2(x[i], x[i + 1]), pack2(v[0], v[1])));
          r[i / 2 + 1] = mul2(pack2(be.z, be.w), fma2(pack2(-g.z, -g.w), pack2(x[i + 2], x[i + 3]), pack2(v[2], v[3])));
          seen = fma2(r[i / 2], zero, fma2(r[i / 2 + 1], zero, seen));
        }
        float lo, hi;
        unpack2(seen, lo, hi);
        if (tokens < 16 * w + 16 || !(lo + hi == 0.f)) {  // not all tokens count, or v holds values that are not finite
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float e[2];
            unpack2(r[i], e[0], e[1]);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int t = 16 * w + 2 * i + k;
              if (t >= tokens) e[k] = 0.f;
              else if (!(fabsf(e[k]) < __int_as_float(0x7f800000))) {
                atomicMin(&sh.first[row], c * Q + t);
                *(volatile int *)&sh.not_finite = 1;
                e[k] = 0.f;
              }
            }
            r[i] = pack2(e[0], e[1]);
          }
        }
        if (tokens < valid && w == 0) {
          atomicMin(&sh.first[row], c * Q + tokens);
          *(volatile int *)&sh.not_finite = 1;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) cut2(r[i], x[i], x[8 + i]);
        tm_st16(here + kColR + 16 * w, x);
        tm_wait_st();
        warp_arrive(sh.r_ready, lane);
        if (lane == 0) mbar_arrive(&sh.free_v[b]);
      }
      f2 y[8];
      {  // rise Q S^T, while U is on its way
        uint32_t x[16];
        wait(sh.qs_done, c);
        tm_fence_after();
        tm_ld16(here + kColY + 16 * w, x);
        tm_wait_ld();
        const f2 scale = pack2(a.q_scale, a.q_scale);
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float4 g = *reinterpret_cast<const float4 *>(&tab.rise[16 * w + i]);
          y[i / 2] = mul2(mul2(scale, pack2(g.x, g.y)), pack2(x[i], x[i + 1]));
          y[i / 2 + 1] = mul2(mul2(scale, pack2(g.z, g.w)), pack2(x[i + 2], x[i + 3]));
        }
      }
      float carry = tab.carry;
      {  // U, and U as it counts at the chunk's end
        uint32_t x[16], o[16];
        wait(sh.u_done, c);
        tm_fence_after();
        tm_ld16(here + kColU + 16 * w, x);
        tm_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float4 g = *reinterpret_cast<const float4 *>(&tab.fall[16 * w + i]);
          cut2(mul2(pack2(g.x, g.y), pack2(x[i], x[i + 1])), o[i / 2], o[8 + i / 2]);
          cut2(mul2(pack2(g.z, g.w), pack2(x[i + 2], x[i + 3])), o[i / 2 + 1], o[8 + i / 2 + 1]);
        }
        tm_st16(here + kColR + 16 * w, o);
#pragma unroll
        for (int i = 0; i < 8; ++i) cut2(pack2(x[2 * i], x[2 * i + 1]), o[i], o[8 + i]);
        tm_st16(here + kColU + 16 * w, o);
        tm_wait_st();
        warp_arrive(sh.u_ready, lane);
      }
      int first = 0x7fffffff;  // of this chunk's tokens, from where on the row is NaN
      if (*(volatile int *)&sh.not_finite) {
        first = *(volatile int *)&sh.first[row] - c * Q;
        if (first < valid) carry = nan;
      }
      {
        const f2 cc = pack2(carry, carry);
        wait(sh.d_done, c);
        tm_fence_after();
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t x[16];
          tm_ld16(here + kColD + 32 * w + 16 * half, x);
          tm_wait_ld();
#pragma unroll
          for (int i = 0; i < 8; ++i) s[8 * half + i] = fma2(cc, s[8 * half + i], pack2(x[2 * i], x[2 * i + 1]));
          if (c + 1 < chunks) put_state(half);
        }
        if (c + 1 < chunks) {
          tm_wait_st();
          warp_arrive(sh.s_ready, lane);
        }
      }
      {
        uint32_t x[16];
        wait(sh.y_done, c);
        tm_fence_after();
        tm_ld16(here + kColY + 16 * w, x);
        tm_wait_ld();
        warp_arrive(sh.y_free, lane);
        const f2 scale = pack2(a.q_scale, a.q_scale);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float e[2];
          unpack2(fma2(scale, pack2(x[2 * i], x[2 * i + 1]), y[i]), e[0], e[1]);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int t = 16 * w + 2 * i + k;
            if (t >= first) e[k] = nan;
            if (have && t < valid) yg[(size_t)(c * Q + t) * a.H * a.R] = e[k];
          }
        }
      }
    }
    if (have) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float4 v;
        unpack2(s[2 * i], v.x, v.y);
        unpack2(s[2 * i + 1], v.z, v.w);
        *reinterpret_cast<float4 *>(Sg + 4 * i) = v;
      }
    }
    tm_fence_before();
  }
  __syncthreads();
  if (warp == kWarpLoad) {
    tm_fence_after();
    tm_free(tm, 512);
  }
  if (*(volatile int *)&sh.abort) overwrite(a, sh, h, S);
}

}  // namespace

cudaError_t launch_gdn_tc(const GdnScanArgs &s, const Prompts &pr, cudaStream_t stream) {
  GdnTcArgs a{};
  a.H = s.H; a.Hk = s.Hk; a.R = s.R; a.by_prompt = s.by_prompt; a.q_scale = s.q_scale;
  a.alpha = s.alpha; a.beta = s.beta; a.S = s.S; a.y = s.y;
  a.err = s.err; a.wait_cycles = s.wait_cycles; a.withhold = s.withhold;
  a.by_length = pr.nseq > 1 && pr.nseq <= kByLength && pr.total / pr.nseq >= 4 * Q;
  EncodeTiled fn;
  cudaError_t e = map_encoder(&fn);
  if (e != cudaSuccess) return e;
  CUtensorMap mq, mk, mv;
  const CUtensorMapDataType bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const cuuint64_t sk[2] = {(cuuint64_t)s.Hk * kCols, (cuuint64_t)pr.total};
  const cuuint64_t tk[1] = {(cuuint64_t)s.Hk * kCols * 2};
  const cuuint32_t bk[2] = {64, Q};
  e = make_map(fn, &mq, bf16, s.q, 2, sk, tk, bk);
  if (e == cudaSuccess) e = make_map(fn, &mk, bf16, s.k, 2, sk, tk, bk);
  const cuuint64_t sv[3] = {(cuuint64_t)s.R, (cuuint64_t)s.H, (cuuint64_t)pr.total};
  const cuuint64_t tv[2] = {(cuuint64_t)s.R * 2, (cuuint64_t)s.H * s.R * 2};
  const cuuint32_t bv[3] = {64, 1, Q};
  if (e == cudaSuccess) e = make_map(fn, &mv, bf16, s.v, 3, sv, tv, bv);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(gdn_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kGdnSmem);
  if (e != cudaSuccess) return e;
  gdn_tc_kernel<<<(unsigned)pr.nseq * s.H, kGdnThreads, kGdnSmem, stream>>>(mq, mk, mv, a, pr);
  return cudaGetLastError();
}

}  // namespace rssm
