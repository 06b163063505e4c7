// gdn_tc.cu -- the gated delta rule over packed prompts on the tensor cores (bf16 inputs).
//
// Chunks of Q = 64 tokens.  With D_ji the product of alpha over i < l <= j within the chunk, g_j = D over its first j + 1
// tokens, and S the state before it, u_j = beta_j (v_j - alpha_j S_{j-1} k_j) solves a triangular system:
//   A_ji = [i < j] beta_j D_ji (k_j . k_i),   T = (I + A)^-1,   M_ji = [i <= j] D_ji (q_j . k_i)
//   R = diag(beta) (V - diag(g) K S^T)         U = T R
//   Y = q_scale (diag(g) Q S^T + M U)          S <- g_Q S + (diag(g_Q / g) U)^T K
// A block carries one head along one prompt; lanes of tensor memory are rows of the state (d_v), so R, U and Y are held
// transposed, and S stays on the chip.
//
// Two forms.  Where no product of alpha from an end of a block of 16 on passes 1 and the chunk's is 2^-24 or more ("mild"), they leave
// the matrices: with f_j = g_Q / g_j,  A_ji = [i < j] beta_j (k_j . k_i),  M_ji = [i <= j] (q_j . k_i),  R = diag(beta)
// (diag(f) V - g_Q K S^T) = diag(f) of the R above,  Y = q_scale diag(1 / f) (g_Q Q S^T + M U),  S <- g_Q S + U^T K: one cut
// of U serves both products.  f lies in 2^-24 .. 1, so nothing overflows that would not without it, and values down to 2^-85
// keep their 24 bits in the pieces of f U (the last one's resolution is 2^-133).  Otherwise ("strong") D is formed from products
// within and between blocks of 16, never as a quotient, so that decays to nothing stay what they are; such chunks take 9 % more
// (8191 tokens of 32 heads 667 -> 730 us).
//
// Precision.  q, k, v are bf16; S, R, U, M and T go into the products as three bf16 pieces each (24 bits), accumulated in
// fp32.  (I + A)^-1 is formed in fp32 on the diagonal blocks of 16 and from there by products of blocks in three pieces with
// mma.sync.  512 tokens are 2e-7 (decays of 2^-60 a chunk) to 5.5e-7 (2^-1) of a norm off, whether keys are independent or alike
// (mean cosines of 0 to 0.95, beta 0.5 to 1).  With T and the blocks' products in two pieces it was 1.3e-6 for independent
// keys and 1.3e-5 for keys alike, for 3 to 5 % less time in one long prompt.
//
// What bounds it: two chains of a chunk that are about as long, some 5.2 us (5.7 with strong decays) for few blocks. The state's:
// S -> K S^T -> R -> U -> S, each step a product of 0.4 to 1 us and a pass of its results through registers into pieces. Beside it
// the next chunk's preparation: the rows of A and M, the inverse's blocks one after another, 120 mma.sync of three pieces; the state
// waits for it 0.3 to 0.7 us of a chunk. 8191 tokens of 32 heads take 0.75 ms, on 32 SMs; 16384 tokens of 8 prompts 0.44 to 0.62 ms by
// their lengths. The tensor cores are busy a quarter of that. Rows of the state split over more blocks, and more warps for the
// preparation and for Y, took as long or longer: the steps wait for one another, and instructions for their way to the SM, so
// that the preparation's loops stay rolled (unrolled, 405 -> 475 us for 8 prompts of 2048).
#include "prompt_kernels.h"
#include "packed.cuh"
#include "tcgen05.cuh"
#include "tensor_map.h"

namespace rssm {

namespace {

constexpr int Q = kGdnChunk;
constexpr int kHalf = Q * 128;  // bytes of a tile: 64 rows of 64 bf16
constexpr int kStepA = 52;      // floats from row to row of A: eight rows' 16-byte stores meet 32 different banks
constexpr int kStages = 3;      // of q and k: one chunk in the chain of the state, one in front of it, one on its way
// Tensor memory.  K S^T, U and the increment of S are cut where they lie: a warp's 16 (32) columns of results become 24 (48)
// of pieces in a range of its own, so results stand in the middle of the two ranges that they share.
constexpr uint32_t kColR = 0, kColU = 96, kColS = 192, kColY = 384, kColG = 448;
constexpr int kChain = 16;                                    // warps: lanes' quarter w % 4, columns' quarter w / 4
constexpr int kWarpPrep = 16, kWarpLoad = 20, kWarpState = 21, kWarpGram = 22, kWarpLoadV = 23;
constexpr int kGdnThreads = 24 * 32;
constexpr int kUnits = 4;                                     // that the loading warp is ahead at most
constexpr int kUnitReaders = 23;                              // all warps but the one that hands them out
constexpr int kByLength = 64;
constexpr int kMostInTurn = 4096;
constexpr float kMild = 1.f / 16777216.f;

// Factors of a chunk's tokens in either form.
struct __align__(16) Table {
  float v[Q], k[Q];   // R = v V + k K S^T
  float q[Q], u[Q];   // Y = q Q S^T + u M U
  float fall[Q];      // g_Q / g_j
  float carry;        // g_Q
  int tokens;         // of the chunk, or up to the first whose k, alpha or beta is not finite
  int mild;           // the form without decays within the chunk
};

// What a block works on next: a head along a prompt.
struct Unit {
  int seq, slot, head, begin, tokens;  // no tokens: nothing more
  int resume;
};

struct GdnShared {
  unsigned char in[kStages][4][kHalf];  // k, q of columns 0..63, k, q of columns 64..127; then Y on its way out
  __nv_bfloat16 V[Q][kCols];
  unsigned char T[2][3][kHalf], M[2][3][kHalf];  // pieces; row = token j
  float A[32 * kStepA];           // blocks of A below the diagonal, see store_a
  __align__(16) float diag[4][16 * 20 + 16];  // blocks of A on the diagonal, [column][row]; then X, see block_x
  Table tab[2];
  float alpha[2][Q], prefix[2][Q], fall[2][Q], tot[2][4];  // products within a token's block of 16: up to it, and behind it
  int first[2][128];  // per row of the state, the first token of the unit (odd ones, even ones) whose v is not finite
  Unit unit[kUnits];
  int order[kByLength];  // prompts by length
  uint64_t full_kq[kStages], free_kq[kStages], full_v, free_v, full_t[2], free_t[2];
  uint64_t ks_done[2], qs_done, u_done[2], d_done[2], y_done, g_done, g_free, drained[2];
  uint64_t s_ready[2], r_ready[2], u_ready[2], y_taken, y_free, full_unit[kUnits], free_unit[kUnits];
  uint32_t tmem;
  int abort, not_finite, bad;
  int slot;  // of the unit whose state is on the chip: what a wait that runs out reports, for units end in turn
};
constexpr int kGdnSmem = (int)sizeof(GdnShared);
static_assert(kGdnSmem <= 227 * 1024, "shared memory of a block");

struct GdnTcArgs {
  int H, Hk, R, by_prompt;
  int units;                // heads x prompts
  int by_length;            // hand out the prompts by length (at most kByLength of them)
  float q_scale;
  const float *alpha, *beta;  // [total][H]
  float *S;                 // [nslots or nseq][H][R][128]
  float *y;                 // [total][H][R]
  int *err;                 // may be null
  long long wait_cycles;
  int withhold;             // test hook: no block loads v of this chunk of a prompt (-1: off)
};

struct Waiter {
  GdnShared *sh;
  int *err;
  WaitSpec ws;
  __device__ __forceinline__ void gave_up() const {
    *(volatile int *)&sh->abort = 1;
    if (err) record_error(err, *(volatile int *)&sh->slot, RSSM_DEV_TIMEOUT);
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

// operands of m16n8k16: a block of 16 x 16 of a tile at (row, col) as the left operand, and as the left one transposed, in three
// pieces
__device__ __forceinline__ void load_left(unsigned char (*T)[kHalf], int row, int col, int lane, uint32_t (&f)[3][4]) {
#pragma unroll
  for (int p = 0; p < 3; ++p)
    ldmatrix_x4(at_tile(T[p], row + (lane & 15), col + 8 * (lane >> 4)), f[p][0], f[p][1], f[p][2], f[p][3]);
}
__device__ __forceinline__ void load_left_t(unsigned char (*T)[kHalf], int row, int col, int lane, uint32_t (&f)[3][4]) {
#pragma unroll
  for (int p = 0; p < 3; ++p)
    ldmatrix_x4_trans(at_tile(T[p], row + (lane & 7) + 8 * (lane >> 4), col + (lane & 8)), f[p][0], f[p][1], f[p][2], f[p][3]);
}
// d += a b for 16 columns, the right operand words of fp32 values that are cut here: the products above 2^-24 of the result, as
// four sums of three that do not wait for one another
__device__ __forceinline__ void mma3(float (&d)[2][4], const uint32_t (&a)[3][4], const f2 (&b)[2][2]) {
  uint32_t p[2][3][2];
  float small[2][4] = {};
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int k = 0; k < 2; ++k) cut3(b[n][k], p[n][0][k], p[n][1][k], p[n][2][k]);
  auto both = [&](float (&to)[2][4], int i, int k) {
#pragma unroll
    for (int n = 0; n < 2; ++n) mma_16816(to[n], a[i][0], a[i][1], a[i][2], a[i][3], p[n][k][0], p[n][k][1]);
  };
  both(small, 2, 0);
  both(d, 1, 0);
  both(small, 0, 2);
  both(d, 0, 1);
  both(small, 1, 1);
  both(d, 0, 0);
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) d[n][i] += small[n][i];
}

// X^T (+)= Z^T B^T for blocks of 16 x 16, Z at (zr, zc) of T and B at (br, bc) of A; x[n]: columns 8 n ..
__device__ __forceinline__ void block_x(unsigned char (*T)[kHalf], int zr, int zc, const float *A, int br, int bc, int lane,
                                        float (&x)[2][4]) {
  uint32_t z[3][4];
  f2 b[2][2];
  load_left_t(T, zr, zc, lane, z);
#pragma unroll
  for (int n = 0; n < 2; ++n)  // columns of B^T are rows of B
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float2 v = *reinterpret_cast<const float2 *>(A + (br + 8 * n + (lane >> 2)) * kStepA + bc + 8 * k + 2 * (lane & 3));
      b[n][k] = pack2(v.x, v.y);
    }
  mma3(x, z, b);
}
// the accumulators of X^T as the right operand of a product with X
__device__ __forceinline__ void turn_x(const float (&x)[2][4], f2 (&b)[2][2]) {
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int k = 0; k < 2; ++k) b[n][k] = pack2(x[k][2 * n], x[k][2 * n + 1]);
}
// T block (+)= W X for W at (wr, wc) of T
__device__ __forceinline__ void block_t(unsigned char (*T)[kHalf], int wr, int wc, int lane, const f2 (&x)[2][2],
                                        float (&t)[2][4]) {
  uint32_t w[3][4];
  load_left(T, wr, wc, lane, w);
  mma3(t, w, x);
}
__device__ __forceinline__ void store_block(unsigned char (*T)[kHalf], int row, int col, int lane, const float (&t)[2][4]) {
  const int g = lane >> 2, p = 2 * (lane & 3);
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t c[3];
      cut3(pack2(-t[n][2 * i], -t[n][2 * i + 1]), c[0], c[1], c[2]);
#pragma unroll
      for (int k = 0; k < 3; ++k) *reinterpret_cast<uint32_t *>(at_tile(T[k], row + g + 8 * i, col + 8 * n) + 2 * p) = c[k];
    }
}

// The i-th unit of this block, heads of a prompt side by side: prompts from the longest to the shortest, dealt out forwards and
// backwards in turn, so that no block has all of the long ones.  (prompt, head), or false behind the last.
__device__ __forceinline__ bool nth_unit(const GdnTcArgs &a, const GdnShared &sh, int i, int &seq, int &head) {
  const long long at = (long long)i * gridDim.x + (i & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
  if (at >= a.units) return false;
  seq = (int)at / a.H;
  head = (int)at - seq * a.H;
  if (a.by_length) seq = sh.order[seq];
  return true;
}
__device__ __forceinline__ float *state_of(const GdnTcArgs &a, int seq, int slot, int head) {
  return a.S + ((size_t)(a.by_prompt ? seq : slot) * a.H + head) * a.R * kCols;
}
// whether a prompt is one to work on, asked by `team` threads: a resumed sequence needs an empty buffer, and no slot two prompts
__device__ __forceinline__ bool refused(const Prompts &pr, int seq, int slot, int resume, int thread, int team) {
  bool no = resume && pr.meta && (pr.meta[slot].x != 0 || pr.meta[slot].z != 0);
  if (pr.slots)
    for (int j = thread; j < pr.nseq; j += team) no |= j != seq && pr.slots[j] == slot;
  return no;
}

// A wait gave up: nothing of this block that looks like a result stays.
__device__ __noinline__ void overwrite(const GdnTcArgs &a, const Prompts &pr, const GdnShared &sh) {
  if (threadIdx.x % 32 == 0) bulk_wait_all();  // this warp's own stores of Y
  __syncthreads();
  const float nan = __int_as_float(0x7fffffff);
  int seq, head;
  for (int n = 0; nth_unit(a, sh, n, seq, head); ++n) {
    const int slot = pr.slots ? pr.slots[seq] : seq, begin = pr.off[seq], end = pr.off[seq + 1];
    if (__syncthreads_or(refused(pr, seq, slot, pr.resume ? pr.resume[seq] : 0, threadIdx.x, kGdnThreads)) || begin == end)
      continue;
    float *S = state_of(a, seq, slot, head);
    for (int i = threadIdx.x; i < a.R * kCols; i += kGdnThreads) S[i] = nan;
    for (int t = begin + threadIdx.x / 32; t < end; t += kGdnThreads / 32)
      for (int r = threadIdx.x % 32; r < a.R; r += 32) a.y[((size_t)t * a.H + head) * a.R + r] = nan;
  }
}

// Rows of A (threads 0..63 of the preparing warps) and M (the others) of a chunk, from the Gram matrix in tensor memory.
struct PrepRow {
  int j, bj, jj;     // token, its block of 16 and place there
  bool of_k;
  int upper;         // rows of tokens 32..63
  uint32_t gram;     // this warp's lanes of the Gram matrix
  float by;          // beta, or 1
  float f[4];        // product of alpha from the end of an earlier block to this token
};

// Where A is held, in 32 rows: the block of 32 x 32 below the diagonal at columns 0..31, and the two of 16 x 16 within the
// diagonal blocks of 32 at columns 32..47.
__device__ __forceinline__ void store_a(GdnShared &sh, const PrepRow &r, int blk, const f2 (&v)[8]) {
  const int row = blk < 2 * r.upper ? r.j - 32 : 16 * r.upper + r.jj, col = blk < 2 * r.upper ? 16 * blk : 32;
  if (blk >= r.bj) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float4 e;
    unpack2(v[2 * i], e.x, e.y);
    unpack2(v[2 * i + 1], e.z, e.w);
    *reinterpret_cast<float4 *>(&sh.A[row * kStepA + col + 4 * i]) = e;
  }
}
__device__ __forceinline__ void store_m(unsigned char (*M)[kHalf], const PrepRow &r, int blk, const f2 (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint4 p0, p1, p2;
    cut3(v[4 * i], p0.x, p1.x, p2.x);
    cut3(v[4 * i + 1], p0.y, p1.y, p2.y);
    cut3(v[4 * i + 2], p0.z, p1.z, p2.z);
    cut3(v[4 * i + 3], p0.w, p1.w, p2.w);
    if (blk <= r.bj) {
      *reinterpret_cast<uint4 *>(at_tile(M[0], r.j, 16 * blk + 8 * i)) = p0;
      *reinterpret_cast<uint4 *>(at_tile(M[1], r.j, 16 * blk + 8 * i)) = p1;
      *reinterpret_cast<uint4 *>(at_tile(M[2], r.j, 16 * blk + 8 * i)) = p2;
    }
  }
}

// The factors of a row of the Gram matrix and a block of columns: by_j, with decays by_j D_ji up to the diagonal.
__device__ __forceinline__ void row_factors(const GdnShared &sh, const PrepRow &r, bool strong, int b, int blk, f2 (&e)[8]) {
  if (!strong) {
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = pack2(r.by, r.by);
    return;
  }
  const float f = r.by * (blk == 0 ? r.f[0] : blk == 1 ? r.f[1] : r.f[2]);
  if (blk < 2 * r.upper) {  // before the blocks of all of this warp's rows
    const f2 ff = pack2(f, f);
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const float4 a4 = *reinterpret_cast<const float4 *>(&sh.fall[b][16 * blk + i]);
      e[i / 2] = mul2(ff, pack2(a4.x, a4.y));
      e[i / 2 + 1] = mul2(ff, pack2(a4.z, a4.w));
    }
    return;
  }
  const int last = blk == r.bj ? r.jj : 15;  // factors behind the row's token do not count
  float d = blk < r.bj ? f : r.by;
#pragma unroll
  for (int i = 12; i >= 0; i -= 4) {
    const float4 a4 = *reinterpret_cast<const float4 *>(&sh.alpha[b][16 * blk + i]);
    const float d3 = d, d2 = d3 * (i + 3 <= last ? a4.w : 1.f), d1 = d2 * (i + 2 <= last ? a4.z : 1.f),
                d0 = d1 * (i + 1 <= last ? a4.y : 1.f);
    e[i / 2 + 1] = pack2(d2, d3);
    e[i / 2] = pack2(d0, d1);
    d = d0 * (i <= last ? a4.x : 1.f);
  }
}

// Rows of A = beta_j D G, or of M = D G up to the diagonal; D is left out in the form without decays.  Returns a sum that is not 0
// where a value of k or beta that this row of A uses, or that lies in its block, is not finite.  What rows before it take is
// finite: they take nothing behind them, and M is selected up to the diagonal.
__device__ __forceinline__ f2 prep_rows(GdnShared &sh, const PrepRow &r, bool strong, unsigned char (*M)[kHalf], int b) {
  f2 seen = pack2(0.f, 0.f);
  const f2 zero = seen;
#pragma unroll 1
  for (int blk = 0; blk < 2 * r.upper + 2; ++blk) {
    uint32_t G[16];
    f2 v[8];
    tm_ld16(r.gram + 16 * blk, G);
    row_factors(sh, r, strong, b, blk, v);
    tm_wait_ld();
    if (r.of_k) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = mul2(v[i], pack2(G[2 * i], G[2 * i + 1]));
        seen = fma2(v[i], zero, seen);
      }
      if (blk == r.bj) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float e0, e1;
          unpack2(v[i], e0, e1);
          sh.diag[r.bj][40 * i + r.jj] = e0;
          sh.diag[r.bj][40 * i + 20 + r.jj] = e1;
        }
      }
      store_a(sh, r, blk, v);
    } else {
      if (blk >= 2 * r.upper) {
        const int most = blk < r.bj ? 15 : r.jj;  // last column of this row (rows above the block are not stored)
#pragma unroll
        for (int i = 0; i < 16; ++i) G[i] = i <= most ? G[i] : 0u;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = mul2(v[i], pack2(G[2 * i], G[2 * i + 1]));
      store_m(M, r, blk, v);
    }
  }
  return seen;
}
__device__ __forceinline__ bool not_zero(f2 v) {
  float a, b;
  unpack2(v, a, b);
  return !(a + b == 0.f);
}
// Some value of the chunk is not finite.  From the first token on whose k, alpha or beta is not (k_j . k_j is not, if k_j is
// not), or whose products of alpha pass fp32's range, the tokens change nothing; the state warps write NaN for them.  Rows
// before it have used none of them.  Returns that token, or the number of tokens.
__device__ __noinline__ int prep_careful(GdnShared &sh, PrepRow r, bool odd, bool strong, int b, int valid) {
  float own = r.by;
#pragma unroll 1
  for (int blk = 0; blk < 2 * r.upper + 2; ++blk) {
    uint32_t G[16];
    f2 e[8];
    tm_ld16(r.gram + 16 * blk, G);
    row_factors(sh, r, strong, b, blk, e);
    tm_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float e0, e1;
      unpack2(e[i / 2], e0, e1);
      if (blk == r.bj && i == r.jj) own = fmaf(__uint_as_float(G[i]), 0.f, own);
      else if (strong && (blk < r.bj || (blk == r.bj && i < r.jj)))
        own = fmaf((i & 1 ? e1 : e0) * __uint_as_float(G[i]), 0.f, own);
    }
  }
  if (threadIdx.x == 32 * kWarpPrep) sh.bad = valid;
  prep_sync();
  if (r.of_k && r.j < valid && (odd || !(own * 0.f == 0.f))) atomicMin(&sh.bad, r.j);
  prep_sync();
  const int bad = sh.bad;
  if (r.of_k && r.j >= bad) {
    for (int i = 0; i < 16; ++i) sh.diag[r.bj][20 * i + r.jj] = 0.f;
    const f2 zero[8] = {};
    for (int blk = 0; blk < r.bj; ++blk) store_a(sh, r, blk, zero);
  }
  return bad;
}

// Of 16 tokens of U from `first` on (of the unit's from `at` on), what grew past fp32's range becomes 0 and its row ends there: it
// must not meet the zeros that M has for earlier tokens.  A whole warp.
__device__ __noinline__ void clear_u(GdnShared &sh, uint32_t taddr, int first, int tokens, int at, int *bad_from) {
  uint32_t x[16];
  tm_ld16(taddr, x);
  tm_wait_ld();
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (!(fabsf(__uint_as_float(x[i])) < __int_as_float(0x7f800000))) {
      if (first + i < tokens) {
        atomicMin(bad_from, at + first + i);
        *(volatile int *)&sh.not_finite = 1;
      }
      x[i] = 0;
    }
  __syncwarp();
  tm_st16(taddr, x);
  tm_wait_st();
}

// kMany: the block takes units in turn, otherwise one.
template <bool kMany>
__global__ void __launch_bounds__(kGdnThreads, 1)
    gdn_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_y,
                  const __grid_constant__ GdnTcArgs a, Prompts pr) {
  extern __shared__ __align__(1024) unsigned char raw[];
  GdnShared &sh = *reinterpret_cast<GdnShared *>(raw);
  if (smem_u32(raw) & 1023u) {
    if (threadIdx.x == 0 && a.err) record_error(a.err, 0, RSSM_DEV_TIMEOUT);
    return;
  }
  allow_next();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  {
    bool bad = false;
    for (int i = tid; i < pr.nseq; i += kGdnThreads) bad |= prompt_bad(pr, i);
    if (__syncthreads_or(bad)) return;
  }
  if (a.by_length) {
    int *lens = reinterpret_cast<int *>(sh.diag);
    const int mine = tid < pr.nseq ? pr.off[tid + 1] - pr.off[tid] : 0;
    if (tid < pr.nseq) lens[tid] = mine;
    __syncthreads();
    if (tid < pr.nseq) {
      int rank = 0;
      for (int j = 0; j < pr.nseq; ++j) rank += lens[j] > mine || (lens[j] == mine && j < tid);
      sh.order[rank] = tid;
    }
  }
  if (tid == 0) {
    uint64_t *one[] = {&sh.full_kq[0], &sh.full_kq[1], &sh.full_kq[2], &sh.full_v, &sh.ks_done[0], &sh.ks_done[1],
                       &sh.qs_done, &sh.u_done[0], &sh.u_done[1], &sh.d_done[0], &sh.d_done[1], &sh.y_done, &sh.g_done,
                       &sh.drained[0], &sh.drained[1]};
    for (uint64_t *b : one) mbar_init(b, 1);
    uint64_t *prep[] = {&sh.full_t[0], &sh.full_t[1], &sh.g_free};
    for (uint64_t *b : prep) mbar_init(b, 4);
    uint64_t *half[] = {&sh.s_ready[0], &sh.s_ready[1], &sh.r_ready[0], &sh.r_ready[1], &sh.u_ready[0], &sh.u_ready[1]};
    for (uint64_t *b : half) mbar_init(b, kChain / 2);
    uint64_t *team[] = {&sh.free_kq[0], &sh.free_kq[1], &sh.free_kq[2], &sh.free_v, &sh.y_taken, &sh.y_free};
    for (uint64_t *b : team) mbar_init(b, kChain);
    for (uint64_t &b : sh.free_t) mbar_init(&b, kChain + 1);
    for (uint64_t &b : sh.full_unit) mbar_init(&b, 1);
    for (uint64_t &b : sh.free_unit) mbar_init(&b, kUnitReaders);
    sh.abort = sh.not_finite = sh.slot = 0;
    fence_barrier_init();
  }
  if (tid < 256) sh.first[tid >> 7][tid & 127] = 0x7fffffff;
  if (warp == kWarpLoad) tm_alloc(&sh.tmem, 512);
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  const uint32_t tm = sh.tmem;
  const Waiter wait{&sh, a.err, {a.wait_cycles, 0}};
  // the n-th unit, for a whole warp, which lets go of it again; false: there is none, or the block gives up
  auto has_unit = [&](int n) {
    if (!kMany && n > 0) return false;
    wait.warp(sh.full_unit[n % kUnits], n / kUnits);
    return !__any_sync(0xffffffffu, *(volatile int *)&sh.abort) && sh.unit[n % kUnits].tokens > 0;
  };
  auto leave_unit = [&](int n) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.free_unit[n % kUnits]);
  };
  auto next_unit = [&](int n, Unit &u) {
    if (!has_unit(n)) return false;
    u = sh.unit[n % kUnits];
    leave_unit(n);
    return true;
  };
  if (warp == kWarpLoad) {
    // Hands out the units, and reads k and q ahead of the others.
    int asked = 0, s = 0, turn = 0;  // chunks whose loads are on their way or done; asked % kStages, asked / kStages
    bool more = true;
    for (int i = 0, n = 0; more && (kMany || i == 0); ++i) {
      Unit u{};
      more = nth_unit(a, sh, i, u.seq, u.head);
      if (more) {
        u.begin = pr.off[u.seq];
        u.tokens = pr.off[u.seq + 1] - u.begin;
        u.slot = pr.slots ? pr.slots[u.seq] : u.seq;
        if (lane == 0 && n == 0) *(volatile int *)&sh.slot = u.slot;  // the first to come
        u.resume = pr.resume ? pr.resume[u.seq] : 0;
        bool skip = __any_sync(0xffffffffu, refused(pr, u.seq, u.slot, u.resume, lane, 32));
        if (!skip && u.tokens == 0) {
          float4 *const S = reinterpret_cast<float4 *>(state_of(a, u.seq, u.slot, u.head));
          if (!u.resume)
            for (int e = lane; e < a.R * kCols / 4; e += 32) S[e] = f4zero();
          skip = true;
        }
        if (skip && kMany) continue;
        more = !skip;
      }
      if (!more) u.tokens = 0;
      if (kMany && n >= kUnits) wait.warp(sh.free_unit[n % kUnits], n / kUnits - 1);
      if (__any_sync(0xffffffffu, *(volatile int *)&sh.abort)) break;
      if (lane == 0) {
        sh.unit[n % kUnits] = u;
        mbar_arrive(&sh.full_unit[n % kUnits]);
        if (kMany && u.resume)  // on its way to the L2 before the rows of the state ask for it
          asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(state_of(a, u.seq, u.slot, u.head)), "r"(a.R * kCols * 4)
                       : "memory");
        const int hk = u.head / (a.H / a.Hk), chunks = (u.tokens + Q - 1) / Q;
        for (int c = 0; c < chunks; ++c) {
          const int t = u.begin + c * Q;
          if (asked >= kStages) wait(sh.free_kq[s], turn - 1);
          if (*(volatile int *)&sh.abort) {
            more = false;
            break;
          }
          mbar_arrive_expect_tx(&sh.full_kq[s], 4 * kHalf);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            tma_load_2d(sh.in[s][2 * half], &map_k, hk * kCols + 64 * half, t, &sh.full_kq[s]);
            tma_load_2d(sh.in[s][2 * half + 1], &map_q, hk * kCols + 64 * half, t, &sh.full_kq[s]);
          }
          ++asked;
          if (++s == kStages) s = 0, ++turn;
        }
      }
      ++n;
      more = __all_sync(0xffffffffu, more);
    }
    // No copy outlives the block: the last phase of each barrier that was asked for.
    if (lane == 0)
      for (int c = max(0, asked - kStages); c < asked; ++c) mbar_wait(&sh.full_kq[c % kStages], (c / kStages) & 1, wait.ws);
    __syncwarp();
  } else if (warp == kWarpLoadV) {
    Unit u;
    int asked = 0;
    bool more = true;
    for (int i = 0; more && next_unit(i, u); ++i) {
      if (lane == 0) {
        for (int t = 0; t < u.tokens; t += Q) {
          if (asked > 0) wait(sh.free_v, asked - 1);
          if (*(volatile int *)&sh.abort || t / Q == a.withhold) {
            more = false;
            break;
          }
          mbar_arrive_expect_tx(&sh.full_v, 2 * kHalf);
          tma_load_3d(sh.V, &map_v, 0, u.head, u.begin + t, &sh.full_v);
          ++asked;
        }
      }
      more = __all_sync(0xffffffffu, more);
    }
    if (lane == 0 && asked) mbar_wait(&sh.full_v, (asked - 1) & 1, wait.ws);
    __syncwarp();
  } else if (warp == kWarpState || warp == kWarpGram) {
    // The products: the whole warp waits, one thread issues.
    const uint32_t td = __shfl_sync(0xffffffffu, tm, 0);
    constexpr uint32_t kStep = (2 * kHalf) >> 4, kStage = (4 * kHalf) >> 4;  // descriptor units between column halves, stages
    const uint32_t dk = tile_desc(sh.in[0][0], 16);
    int s = 0, turn = 0, c = 0;  // chunk % kStages, chunk / kStages, chunk of all units
    Unit unit;
    if (warp == kWarpGram) {
      constexpr uint32_t shape = mma_shape(128, 64, false, false);
      for (int i = 0; next_unit(i, unit); ++i)
        for (int left = __shfl_sync(0xffffffffu, unit.tokens, 0); left > 0; left -= Q, ++c) {
          wait.warp(sh.full_kq[s], turn);
          if (c > 0) wait.warp(sh.g_free, c - 1);
          tm_fence_after();
          const uint64_t k0 = wide_desc(dk + s * kStage);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {  // rows of k, then of q
              const int at = (k >> 2) * kStep + 2 * (k & 3);
              one_ss(td + kColG, k0 + at, k0 + at, shape, k > 0);
            }
            one_commit(&sh.g_done);
          }
          __syncwarp();
          if (++s == kStages) s = 0, ++turn;
        }
      if (elect_one()) one_commit(&sh.drained[1]);
      mbar_wait(&sh.drained[1], 0, wait.ws);
    } else {
      constexpr uint32_t half_q = mma_shape(128, 32, false, false), all_q = mma_shape(128, 64, false, false);
      constexpr uint32_t half_d = mma_shape(128, 64, false, true);
      constexpr uint32_t kRows = (32 * 128) >> 4;  // 32 token rows
      const uint32_t dkn = tile_desc(sh.in[0][0], 2 * kHalf);  // MN-major, two tiles
      const uint32_t dT = tile_desc(sh.T[0][0], 16), dM = tile_desc(sh.M[0][0], 16);
      constexpr uint32_t kPiece = kHalf >> 4;
      for (int i = 0; next_unit(i, unit); ++i)
        for (int left = __shfl_sync(0xffffffffu, unit.tokens, 0); left > 0; left -= Q, ++c) {
          const int b = c & 1;
          const uint64_t k0 = wide_desc(dk + s * kStage), q0 = k0 + (kHalf >> 4), kn = wide_desc(dkn + s * kStage);
          const uint64_t T = wide_desc(dT + b * 3 * kPiece), M = wide_desc(dM + b * 3 * kPiece);
          wait.warp(sh.full_kq[s], turn);
#pragma unroll
          for (int part = 0; part < 2; ++part) {  // K S^T: halves of S as they come, the last ones by halves of the tokens
            wait.warp(sh.s_ready[part], c);
            tm_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int half = 0; half < 2; ++half) {
#pragma unroll
                for (int k = 4 * part; k < 4 * part + 4; ++k)
#pragma unroll
                  for (int p = 2; p >= 0; --p)
                    one_ts(td + kColR + 48 * half + 8, td + kColS + 24 * k + 8 * p,
                           k0 + (k >> 2) * kStep + 2 * (k & 3) + half * kRows, half_q, k > 0 || p < 2);
                if (part == 1) one_commit(&sh.ks_done[half]);
              }
            }
            __syncwarp();
          }
          if (c > 0) wait.warp(sh.y_free, c - 1);
          tm_fence_after();
          auto qs = [&](int part) {  // Q S^T over half of S
#pragma unroll
            for (int k = 4 * part; k < 4 * part + 4; ++k)
#pragma unroll
              for (int p = 2; p >= 0; --p)
                one_ts(td + kColY, td + kColS + 24 * k + 8 * p, q0 + (k >> 2) * kStep + 2 * (k & 3), all_q, k > 0 || p < 2);
          };
          if (elect_one()) qs(0);  // while R is formed
          __syncwarp();
          wait.warp(sh.full_t[b], c >> 1);
          const uint32_t kColE = sh.tab[b].mild ? kColU : kColR;  // U as it counts at the chunk's end
#pragma unroll
          for (int half = 0; half < 2; ++half) {  // U of 32 tokens from R up to them
            wait.warp(sh.r_ready[half], c);
            tm_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < 2 * half + 2; ++k) {  // pieces of R by pieces of T; the others are below 2^-24
                const uint32_t r = td + kColR + 24 * k, u = td + kColU + 48 * half + 8;
                const uint64_t t = T + half * kRows + 2 * k;
                one_ts(u, r, t + 2 * kPiece, half_q, k > 0);
                one_ts(u, r + 8, t + kPiece, half_q, true);
                one_ts(u, r + 16, t, half_q, true);
                one_ts(u, r, t + kPiece, half_q, true);
                one_ts(u, r + 8, t, half_q, true);
                one_ts(u, r, t, half_q, true);
              }
              one_commit(&sh.u_done[half]);
            }
            __syncwarp();
          }
          if (elect_one()) {  // while U is cut
            qs(1);
            one_commit(&sh.qs_done);
          }
          __syncwarp();
          wait.warp(sh.u_ready[0], c);
          wait.warp(sh.u_ready[1], c);
          tm_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int part = 0; part < 2; ++part) {  // 64 columns of the state
#pragma unroll
              for (int k = 0; k < 4; ++k)  // 16 token rows are 2048 bytes
#pragma unroll
                for (int p = 2; p >= 0; --p)
                  one_ts(td + kColS + 96 * part + 16, td + kColE + 24 * k + 8 * p, kn + part * kStep + 128 * k, half_d,
                         k > 0 || p < 2);
              one_commit(&sh.d_done[part]);
            }
          }
          __syncwarp();
          wait.warp(sh.y_taken, c);
          tm_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
              for (int k = 0; k < 2 * half + 2; ++k) {
                const uint32_t u = td + kColU + 24 * k, y = td + kColY + 32 * half;
                const uint64_t m = M + half * kRows + 2 * k;
                one_ts(y, u, m + 2 * kPiece, half_q, k > 0);
                one_ts(y, u + 8, m + kPiece, half_q, true);
                one_ts(y, u + 16, m, half_q, true);
                one_ts(y, u, m + kPiece, half_q, true);
                one_ts(y, u + 8, m, half_q, true);
                one_ts(y, u, m, half_q, true);
              }
            one_commit(&sh.y_done);
            one_commit(&sh.free_t[b]);
          }
          __syncwarp();
          if (++s == kStages) s = 0, ++turn;
        }
      if (elect_one()) one_commit(&sh.drained[0]);
      mbar_wait(&sh.drained[0], 0, wait.ws);
    }
    __syncwarp();
  } else if (warp >= kWarpPrep) {
    // A, T and M of a chunk, a chunk ahead of the state: lanes 0..63 of the Gram matrix are k_j . k_i, the others q_j . k_i
    const int pw = warp - kWarpPrep, p = tid - 32 * kWarpPrep;
    PrepRow r;
    r.upper = pw & 1;
    r.j = p & 63; r.bj = r.j >> 4; r.jj = r.j & 15;
    r.of_k = p < 64;
    r.gram = tm + ((uint32_t)(32 * pw) << 16) + kColG;
    const int j = r.j, bj = r.bj, jj = r.jj;
    const bool of_k = r.of_k;
    for (int i = p; i < 2 * 3 * kHalf / 16; i += 128)  // blocks above the diagonal stay zero
      reinterpret_cast<uint4 *>(sh.T[0][0])[i] = make_uint4(0, 0, 0, 0);
    for (int i = p; i < 2 * 3 * kHalf / 16; i += 128) reinterpret_cast<uint4 *>(sh.M[0][0])[i] = make_uint4(0, 0, 0, 0);
    float alpha_next = 1.f, beta_next = 0.f;
    Unit unit;
    int c = 0;  // chunk of all units
    // The four warps go on or stop together: they meet at barriers of their own, and a block may be given up between their looks.
    for (int i = 0; !prep_sync_or(!next_unit(i, unit)); ++i) {
      const int ntok = unit.tokens;
      size_t next = ((size_t)unit.begin + j) * a.H + unit.head;  // this thread's token of the next chunk
      auto fetch = [&](int first) {
        alpha_next = 1.f;
        beta_next = 0.f;  // a token behind the end changes nothing
        if (of_k && first + j < ntok) {
          alpha_next = a.alpha[next];
          beta_next = a.beta[next];
        }
        next += (size_t)Q * a.H;
      };
      fetch(0);
      // What follows from alpha alone is worked out a chunk ahead, by two warps while the others form the first blocks of T.
      float up = 1.f, down = 1.f, be = 0.f;  // products within the block of 16: up to this token, and behind it; beta
      bool odd = false;                      // alpha is not finite (the chunk ends before it)
      for (int at = -Q; at < ntok; at += Q) {
        const int b = c & 1;
        unsigned char(*const T)[kHalf] = sh.T[b];
        if (at >= 0) {
          const int valid = min(Q, ntok - at);
          if (valid < Q) {  // rows of k that belong to other prompts must not reach the state, whatever they hold
            wait(sh.full_kq[c % kStages], c / kStages);
            for (int i = p + valid * 8; i < Q * 8; i += 128) {
              *reinterpret_cast<uint4 *>(sh.in[c % kStages][0] + 16 * i) = make_uint4(0, 0, 0, 0);
              *reinterpret_cast<uint4 *>(sh.in[c % kStages][2] + 16 * i) = make_uint4(0, 0, 0, 0);
            }
          }
          const bool grows = prep_sync_or(!(fabsf(up) <= 1.f && fabsf(down) <= 1.f));
          if (c > 1) wait(sh.free_t[b], (c >> 1) - 1);
          const float tot[4] = {sh.tot[b][0], sh.tot[b][1], sh.tot[b][2], sh.tot[b][3]};
          const float carry = (tot[0] * tot[1]) * (tot[2] * tot[3]);
          const bool strong = grows || !(fabsf(carry) >= kMild);  // otherwise f_j = carry / (product up to j) >= carry
          Table &tab = sh.tab[b];
          r.by = of_k ? be : 1.f;
          r.f[3] = 0.f;
          {
            float run = sh.prefix[b][j];
#pragma unroll
            for (int i = 2; i >= 0; --i) {
              r.f[i] = i < bj ? run : 0.f;
              if (i < bj) run *= tot[i];
            }
          }
          if (of_k) {
            float rise = up, fall = down;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (i < bj) rise *= tot[i];
              if (i > bj) fall *= tot[i];
            }
            tab.v[j] = strong ? be : be * fall;
            tab.k[j] = strong ? -be * rise : -be * carry;
            tab.q[j] = a.q_scale * rise;
            tab.u[j] = strong ? a.q_scale : a.q_scale / fall;
            tab.fall[j] = fall;
            if (j == 0) {
              tab.carry = carry;
              tab.mild = !strong;
            }
          }
          int tokens = valid;
          wait(sh.g_done, c);
          tm_fence_after();
          const f2 seen = prep_rows(sh, r, strong, sh.M[b], b);
          if (prep_sync_or(of_k && (odd || not_zero(seen)))) {
            tokens = prep_careful(sh, r, odd, strong, b, valid);
            prep_sync();
          }
          if (of_k && j == 0) tab.tokens = tokens;
          warp_arrive(sh.g_free, lane);
          {  // blocks on the diagonal by substitution, one a warp, lane = column
            const int col = lane & 15;
            float t[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) t[i] = col == i ? 1.f : 0.f;
#pragma unroll
            for (int i = 0; i < 15; ++i) {  // t_i is known: off it goes from the rows below
#pragma unroll
              for (int l = (i + 1) & ~3; l < 16; l += 4) {
                const float4 v = *reinterpret_cast<const float4 *>(&sh.diag[pw][20 * i + l]);
                if (l > i) t[l] = fmaf(-v.x, t[i], t[l]);
                if (l + 1 > i) t[l + 1] = fmaf(-v.y, t[i], t[l + 1]);
                if (l + 2 > i) t[l + 2] = fmaf(-v.z, t[i], t[l + 2]);
                if (l + 3 > i) t[l + 3] = fmaf(-v.w, t[i], t[l + 3]);
              }
            }
            const int lo = lane >> 4;  // lanes 0..15 write the first pieces, the others the second; each the third of 8 rows
            auto put_t = [&](int piece, int i, __nv_bfloat16 v) {
              *reinterpret_cast<__nv_bfloat16 *>(at_tile(T[piece], 16 * pw + i, 16 * pw + (col & 8)) + 2 * (col & 7)) = v;
            };
            auto left_of = [](float v) { return v - __bfloat162float(__float2bfloat16_rn(v)); };
#pragma unroll
            for (int i = 0; i < 16; ++i) put_t(lo, i, __float2bfloat16_rn(lo ? left_of(t[i]) : t[i]));
#pragma unroll
            for (int i = 0; i < 8; ++i) put_t(2, 8 * lo + i, __float2bfloat16_rn(left_of(left_of(lo ? t[8 + i] : t[i]))));
          }
          prep_sync();
        }
        if (of_k) {
          if (at + Q < ntok) {
            const int to = at < 0 ? b : b ^ 1;
            odd = !(fabsf(alpha_next) < __int_as_float(0x7f800000));
            const float al = odd ? 1.f : alpha_next;
            be = beta_next;
            fetch(at + 2 * Q);
            up = down = al;
#pragma unroll
            for (int off = 1; off < 16; off <<= 1) {
              const float u = __shfl_up_sync(0xffffffffu, up, off, 16), d = __shfl_down_sync(0xffffffffu, down, off, 16);
              if (jj >= off) up *= u;
              if (jj + off < 16) down *= d;
            }
            down = __shfl_down_sync(0xffffffffu, down, 1, 16);
            if (jj == 15) {
              down = 1.f;
              sh.tot[to][bj] = up;
            }
            sh.alpha[to][j] = al;
            sh.prefix[to][j] = up;
            sh.fall[to][j] = down;
          }
        } else if (at >= 0) {  // T10 = -T11 A10 T00 in both blocks of 32
          const int r0 = 32 * (pw & 1);
          float x[2][4] = {}, t[2][4] = {};
          f2 right[2][2];
          block_x(T, r0, r0, sh.A, r0 >> 1, 32, lane, x);
          turn_x(x, right);
          block_t(T, r0 + 16, r0 + 16, lane, right, t);
          store_block(T, r0 + 16, r0, lane, t);
        }
        if (at < 0) continue;
        prep_sync();
        {  // the same of the whole: rows 16 l of X = A T00 at columns 16 from, one a warp, and block (32 + 16 to, 16 from) of T
          const int to = pw >> 1, from = pw & 1;
          float t[2][4] = {}, x[2][4] = {};
          f2 right[2][2];
          if (from == 0) block_x(T, 0, 0, sh.A, 16 * to, 0, lane, x);
          block_x(T, 16, 16 * from, sh.A, 16 * to, 16, lane, x);
          turn_x(x, right);
          ulonglong2 *const held = reinterpret_cast<ulonglong2 *>(sh.diag[0]);  // the blocks on the diagonal are done with
#pragma unroll
          for (int n = 0; n < 2; ++n) held[(2 * pw + n) * 32 + lane] = make_ulonglong2(right[n][0].v, right[n][1].v);
          prep_sync();
#pragma unroll
          for (int l = 0; l < 2; ++l)
            if (l <= to) {
#pragma unroll
              for (int n = 0; n < 2; ++n) {
                const ulonglong2 v = held[(2 * (2 * l + from) + n) * 32 + lane];
                right[n][0].v = v.x;
                right[n][1].v = v.y;
              }
              block_t(T, 32 + 16 * to, 32 + 16 * l, lane, right, t);
            }
          store_block(T, 32 + 16 * to, 16 * from, lane, t);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.full_t[b]);
        ++c;
      }
    }
  } else {
    // rows of the state: R, U, S, Y
    const int w = warp >> 2, q4 = warp & 3, row = 32 * q4 + lane, part = w >> 1, ww = w & 1;
    const uint32_t here = tm + ((uint32_t)(32 * q4) << 16);
    const bool have = row < a.R;
    const float nan = __int_as_float(0x7fffffff);
    // A warp's 32 columns of the state in two halves of 16, in the order in which they are cut: the pieces of the first may
    // lie over increments that have been read, not over the other half's.
    const int at0 = 16 * ww, at1 = 16 - at0;
    f2 s[2][8];
    // This warp's 32 x 32 of a unit's state.  A load takes 4 rows of 128 bytes, lane 8 a + k the k-th 16 bytes of row 8 a + i;
    // exchanges between lanes' bits of k and i leave each lane with a row.
    auto state_at = [&](int n) {
      const Unit &u = sh.unit[n % kUnits];
      return state_of(a, u.seq, u.slot, u.head) + (size_t)(32 * q4 + (lane & 24)) * kCols + 32 * w + 4 * (lane & 7);
    };
    auto turn_state = [&](f2 (&v)[16]) {
#pragma unroll
      for (int bit = 1; bit < 8; bit <<= 1) {
        const bool up = lane & bit;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (!(i & bit)) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              f2 &x = v[2 * i + k], &y = v[2 * (i | bit) + k];
              const unsigned long long got = __shfl_xor_sync(0xffffffffu, up ? x.v : y.v, bit);
              (up ? x.v : y.v) = got;
            }
          }
      }
    };
    auto load_state = [&](int n) {
      f2 v[16];
      if (sh.unit[n % kUnits].resume) {
        const float *const from = state_at(n);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float4 x = f4zero();
          if (32 * q4 + (lane & 24) + i < a.R) x = *reinterpret_cast<const float4 *>(from + i * kCols);
          v[2 * i] = pack2(x.x, x.y);
          v[2 * i + 1] = pack2(x.z, x.w);
        }
        turn_state(v);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = pack2(0.f, 0.f);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s[0][i] = ww ? v[8 + i] : v[i];
        s[1][i] = ww ? v[i] : v[8 + i];
      }
    };
    auto store_state = [&](int n) {
      f2 v[16];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = ww ? s[1][i] : s[0][i];
        v[8 + i] = ww ? s[0][i] : s[1][i];
      }
      turn_state(v);
      float *const to = state_at(n);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float4 x;
        unpack2(v[2 * i], x.x, x.y);
        unpack2(v[2 * i + 1], x.z, x.w);
        if (32 * q4 + (lane & 24) + i < a.R) *reinterpret_cast<float4 *>(to + i * kCols) = x;
      }
    };
    // 16 columns as three pieces of 8 columns of pairs
    auto put = [&](uint32_t at, const f2 *v) {
      uint32_t o[16], lo[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) cut3(v[i], o[i], o[8 + i], lo[i]);
      tm_st16(here + at, o);
      tm_st8(here + at + 16, lo);
    };
    const uint32_t piece0 = kColS + 48 * w + 24 * ww, piece1 = kColS + 48 * w + 24 - 24 * ww;
    const unsigned short *const vrow = reinterpret_cast<const unsigned short *>(sh.V[16 * w]) + row;
    const size_t ystep = (size_t)a.H * a.R;
    int stage = 0, c = 0;  // c: chunk of all units
    bool more = has_unit(0);
    if (more) load_state(0);
    for (int number = 0; more; ++number) {
      put(piece0, s[0]);
      put(piece1, s[1]);
      tm_wait_st();
      warp_arrive(sh.s_ready[part], lane);
      const Unit &unit = sh.unit[number % kUnits];
      if (tid == 0) *(volatile int *)&sh.slot = unit.slot;
      const int ntok = unit.tokens;
      int *const bad_from = &sh.first[number & 1][row];
      float *yg = a.y + ((size_t)(unit.begin + 16 * w) * a.H + unit.head) * a.R + row;
      for (int at = 0; at < ntok; at += Q, ++c, yg += Q * ystep) {
        const int b = c & 1, valid = min(Q, ntok - at);
        const bool last = at + Q >= ntok;
        const Table &tab = sh.tab[b];
        wait(sh.full_t[b], c >> 1);
        wait(sh.full_v, c);
        const int tokens = tab.tokens;
        {  // R
          f2 r[8];
          f2 seen = pack2(0.f, 0.f);
          const f2 zero = seen;
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(&tab.v[16 * w + i]);
            uint32_t v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = (uint32_t)vrow[(i + k) * kCols] << 16;
            r[i / 2] = mul2(pack2(f.x, f.y), pack2(v[0], v[1]));
            r[i / 2 + 1] = mul2(pack2(f.z, f.w), pack2(v[2], v[3]));
          }
          uint32_t x[16];
          wait(sh.ks_done[part], c);
          tm_fence_after();
          tm_ld16(here + kColR + 48 * part + 8 + 16 * ww, x);
          tm_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(&tab.k[16 * w + i]);
            r[i / 2] = fma2(pack2(f.x, f.y), pack2(x[i], x[i + 1]), r[i / 2]);
            r[i / 2 + 1] = fma2(pack2(f.z, f.w), pack2(x[i + 2], x[i + 3]), r[i / 2 + 1]);
            seen = fma2(r[i / 2], zero, fma2(r[i / 2 + 1], zero, seen));
          }
          if (tokens < 16 * w + 16 || not_zero(seen)) {  // not all tokens count, or v holds values that are not finite
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float e[2];
              unpack2(r[i], e[0], e[1]);
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int t = 16 * w + 2 * i + k;
                if (t >= tokens) e[k] = 0.f;
                else if (!(fabsf(e[k]) < __int_as_float(0x7f800000))) {
                  atomicMin(bad_from, at + t);
                  *(volatile int *)&sh.not_finite = 1;
                  e[k] = 0.f;
                }
              }
              r[i] = pack2(e[0], e[1]);
            }
          }
          if (tokens < valid && w == 0) {
            atomicMin(bad_from, at + tokens);
            *(volatile int *)&sh.not_finite = 1;
          }
          __syncwarp();
          put(kColR + 24 * w, r);
          tm_wait_st();
          warp_arrive(sh.r_ready[part], lane);
          if (lane == 0) {
            mbar_arrive(&sh.free_v);
            if (c > 0) {  // Y of the last chunk has left its stage
              bulk_wait_read();
              mbar_arrive(&sh.free_kq[stage == 0 ? kStages - 1 : stage - 1]);
            }
          }
        }
        float carry = tab.carry;
        {  // U, and where it differs U as it counts at the chunk's end
          uint32_t x[16];
          f2 u[8];
          wait(sh.u_done[part], c);
          // every warp has brought this unit's state, so none reads the last unit's list any more: it is the next one's
          if (at == 0 && w == 0) *(volatile int *)&sh.first[(number & 1) ^ 1][row] = 0x7fffffff;
          tm_fence_after();
          tm_ld16(here + kColU + 48 * part + 8 + 16 * ww, x);
          tm_wait_ld();
          f2 seen[2] = {};
          const f2 zero = seen[0];
#pragma unroll
          for (int i = 0; i < 8; ++i) seen[i & 1] = fma2(pack2(x[2 * i], x[2 * i + 1]), zero, seen[i & 1]);
          if (__any_sync(0xffffffffu, not_zero(fma2(seen[0], zero, seen[1])))) {
            clear_u(sh, here + kColU + 48 * part + 8 + 16 * ww, 16 * w, tokens, at, bad_from);
            tm_ld16(here + kColU + 48 * part + 8 + 16 * ww, x);
            tm_wait_ld();
          }
          if (!tab.mild) {
            if (part == 0) wait(sh.u_done[1], c);  // R of these tokens goes into U of the others
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              const float4 f = *reinterpret_cast<const float4 *>(&tab.fall[16 * w + i]);
              u[i / 2] = mul2(pack2(f.x, f.y), pack2(x[i], x[i + 1]));
              u[i / 2 + 1] = mul2(pack2(f.z, f.w), pack2(x[i + 2], x[i + 3]));
            }
            put(kColR + 24 * w, u);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) u[i] = pack2(x[2 * i], x[2 * i + 1]);
          put(kColU + 24 * w, u);
          tm_wait_st();
          warp_arrive(sh.u_ready[part], lane);
        }
        f2 y[8];
        {  // g Q S^T
          uint32_t x[16];
          wait(sh.qs_done, c);
          tm_fence_after();
          tm_ld16(here + kColY + 16 * w, x);
          tm_wait_ld();
          warp_arrive(sh.y_taken, lane);
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(&tab.q[16 * w + i]);
            y[i / 2] = mul2(pack2(f.x, f.y), pack2(x[i], x[i + 1]));
            y[i / 2 + 1] = mul2(pack2(f.z, f.w), pack2(x[i + 2], x[i + 3]));
          }
        }
        int first = 0x7fffffff;  // of this chunk's tokens, from where on the row is NaN
        {
          wait(sh.d_done[part], c);  // all of the row's R and U have been looked at
          if (*(volatile int *)&sh.not_finite) {
            first = *(volatile int *)bad_from - at;
            if (first < valid) carry = nan;
          }
          const f2 cc = pack2(carry, carry);
          tm_fence_after();
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t x[16];
            tm_ld16(here + kColS + 96 * part + 16 + 32 * ww + (half ? at1 : at0), x);
            tm_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i) s[half][i] = fma2(cc, s[half][i], pack2(x[2 * i], x[2 * i + 1]));
            if (!last) put(half ? piece1 : piece0, s[half]);
          }
          if (!last) {
            tm_wait_st();
            warp_arrive(sh.s_ready[part], lane);
          }
        }
        {
          uint32_t x[16];
          wait(sh.y_done, c);
          tm_fence_after();
          tm_ld16(here + kColY + 16 * w, x);
          tm_wait_ld();
          warp_arrive(sh.y_free, lane);
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(&tab.u[16 * w + i]);
            y[i / 2] = fma2(pack2(f.x, f.y), pack2(x[i], x[i + 1]), y[i / 2]);
            y[i / 2 + 1] = fma2(pack2(f.z, f.w), pack2(x[i + 2], x[i + 3]), y[i / 2 + 1]);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.free_t[b]);
          if (valid >= 16 * w + 16 && __all_sync(0xffffffffu, first >= Q)) {
            if (32 * q4 < a.R) {  // through the chunk's stage of k and q, which nobody reads any more
              unsigned char *const out = sh.in[stage][0] + 2048 * warp;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                float e[2];
                unpack2(y[i], e[0], e[1]);
                *reinterpret_cast<float *>(out + 256 * i + 4 * lane) = e[0];
                *reinterpret_cast<float *>(out + 256 * i + 128 + 4 * lane) = e[1];
              }
              fence_async_smem();
              __syncwarp();
              if (lane == 0) {
                tma_store_3d(&map_y, out, 32 * q4, unit.head, unit.begin + at + 16 * w);
                bulk_commit();
              }
            }
          } else if (have) {
            float *at = yg;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float e[2];
              unpack2(y[i], e[0], e[1]);
#pragma unroll
              for (int k = 0; k < 2; ++k, at += ystep) {
                const int t = 16 * w + 2 * i + k;
                if (t < valid) *at = t >= first ? nan : e[k];
              }
            }
          }
          if (++stage == kStages) stage = 0;
        }
      }
      store_state(number);
      more = has_unit(number + 1);
      if (more) load_state(number + 1);
      leave_unit(number);
    }
    if (lane == 0) bulk_wait_read();
    tm_fence_before();
  }
  __syncthreads();
  if (warp == kWarpLoad) {
    tm_fence_after();
    tm_free(tm, 512);
  }
  if (*(volatile int *)&sh.abort) overwrite(a, pr, sh);
}

}  // namespace

cudaError_t launch_gdn_tc(const GdnScanArgs &s, const Prompts &pr, int num_sms, cudaStream_t stream) {
  GdnTcArgs a{};
  a.H = s.H; a.Hk = s.Hk; a.R = s.R; a.by_prompt = s.by_prompt; a.q_scale = s.q_scale;
  a.alpha = s.alpha; a.beta = s.beta; a.S = s.S; a.y = s.y;
  a.err = s.err; a.wait_cycles = s.wait_cycles; a.withhold = s.withhold;
  a.by_length = pr.nseq > 1 && pr.nseq <= kByLength;
  a.units = pr.nseq * s.H;
  EncodeTiled fn;
  cudaError_t e = map_encoder(&fn);
  if (e != cudaSuccess) return e;
  CUtensorMap mq, mk, mv, my;
  const CUtensorMapDataType bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const cuuint64_t sk[2] = {(cuuint64_t)s.Hk * kCols, (cuuint64_t)pr.total};
  const cuuint64_t tk[1] = {(cuuint64_t)s.Hk * kCols * 2};
  const cuuint32_t bk[2] = {64, Q};
  e = make_map(fn, &mq, bf16, s.q, 2, sk, tk, bk);
  if (e == cudaSuccess) e = make_map(fn, &mk, bf16, s.k, 2, sk, tk, bk);
  const cuuint64_t sv[3] = {(cuuint64_t)s.R, (cuuint64_t)s.H, (cuuint64_t)pr.total};
  const cuuint64_t tv[2] = {(cuuint64_t)s.R * 2, (cuuint64_t)s.H * s.R * 2};
  const cuuint32_t bv[3] = {kCols, 1, Q};
  if (e == cudaSuccess) e = make_map(fn, &mv, bf16, s.v, 3, sv, tv, bv, CU_TENSOR_MAP_SWIZZLE_NONE);
  const cuuint64_t ty[2] = {(cuuint64_t)s.R * 4, (cuuint64_t)s.H * s.R * 4};
  const cuuint32_t by[3] = {32, 1, 16};
  if (e == cudaSuccess) e = make_map(fn, &my, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, s.y, 3, sv, ty, by, CU_TENSOR_MAP_SWIZZLE_NONE);
  if (e != cudaSuccess) return e;
  auto run = [&](auto kernel, int blocks) {
    const cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kGdnSmem);
    if (r != cudaSuccess) return r;
    kernel<<<(unsigned)blocks, kGdnThreads, kGdnSmem, stream>>>(mq, mk, mv, my, a, pr);
    return cudaGetLastError();
  };
  // Units in turn save a block's start and its end and bring the next state closer; one a block is what the hardware hands out
  // as blocks finish, and 7 % faster in a long prompt (32 heads of 128 rows, us, in turn / one a block: 48 prompts of 64 tokens
  // 137 / 178, of 256 331 / 373, of 512 602 / 633; 16 of 256 142 / 146, of 1024 479 / 447; 4 of 64, fewer units than SMs, 28 / 24).
  // Not with many thousands of prompts: one warp looks through all slots for each unit, and the others' waits for it are bounded.
  if (a.units > num_sms && pr.total <= 256LL * pr.nseq && pr.nseq <= kMostInTurn) return run(gdn_tc_kernel<true>, num_sms);
  return run(gdn_tc_kernel<false>, a.units);
}

}  // namespace rssm
