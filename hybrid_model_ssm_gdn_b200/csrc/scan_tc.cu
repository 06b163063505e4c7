// scan_tc.cu -- the Mamba-2 scan over packed prompts on the tensor cores (bf16 inputs).
//
// Chunks of Q = 128 tokens turn the recurrence into matrix products.  With c_j the sum of dt over the chunk's tokens up
// to j (included), per head:
//   G   = C B^T                                          tokens x tokens, one for all heads of a group
//   M   = [j >= i] G_ji exp(A (c_j - c_i)) dt_i
//   Y   = M X + diag(exp(A c)) C S^T + D X                tokens x P
//   S  <- exp(A c_Q) S + (diag(exp(A (c_Q - c)) dt) X)^T B   P x 128
// A block carries two heads of one group (2 x 64 rows of state fill the 128 lanes of tensor memory) along one piece of a
// prompt, chunk after chunk, so the state never leaves the chip.
//
// Precision: C, B and X are bf16 and enter exactly; sums are fp32.  The three fp32 operands M, S and the weighted X are
// cut into two bf16 pieces (hi = RN(v), lo = RN(v - hi): what is lost is below 2^-17 of v) and multiplied twice.  Outputs
// and states are 3e-7 to 6e-7 off in all, where fp32 arithmetic throughout is 4e-8 to 7e-8 off: coarser than the decode
// kernels' folds, whose three pieces are exact, for which shared memory has no room here; one piece would leave 2^-9.
// Differences of sums of dt within a block of 32 tokens carry the rounding of those sums.  Two pieces double three of the
// four products: 14.7 M multiply-adds for a chunk of two heads, 3500 cycles of the tensor core as measured, against the
// 2.3 us that its bytes take at the measured bandwidth (x, y and the group's share of B and C): both limits lie close
// together, and tcgen05 is needed for either (mma.sync measured a quarter of its rate).
//
// Measured: 16384 tokens in 8 prompts of 128 heads, P 64, 8 groups, 0.41 ms (910 MB, 0.14 ms at the copy bandwidth), some
// 13000 cycles a chunk of two heads; one prompt of 8191 tokens 0.29 ms.  What bounds a chunk is the loop below with its
// conversions, not the tensor core (27 % busy) and not memory (25 %).  Two of the waits in it come from buffers that are
// shared, not from the recurrence: the weighted X waits until C S^T has used the pieces of S, and M of the second head
// until M X of the first is done.
//
// Tensor memory (512 columns): S 128 (row = head and p, column = n), Y 128 (row = token, column = head and p), G 128, and
// M as hi | lo pairs 128, for one head after the other; M is the left operand straight from tensor memory.  Shared
// memory: C, three buffers for B and X, a stage for Y, and one 64 KB buffer that holds the pieces of S until C S^T is done
// and then the pieces of the weighted X; all of an SM's, so one block each.
//
// Decays never divide and never exceed what they stand for: a token's weight is a product of exp of sums of dt over
// tokens between, by blocks of 32: within the row's block exp(A (c_j - c_i)), else exp(A (c_j - end)) exp(A (end - c_i))
// with `end` the end of i's block, both at most 1, so only 32 exponentials a row and head are left.
//
// Twenty warps: 0-7 make M from G, scale C S^T and write Y; 8-15 weigh X and cut S; then one for the loads, one for the
// products along the state (C S^T, S), one for those along the tokens (G, M X), one for the decay tables.  The loop that
// bounds a chunk is  cut S -> C S^T -> weigh X -> S product -> cut S; all else runs beside it.
// Every wait is bounded; after one runs out the others stop waiting and the block goes through its remaining steps, so
// all barriers and the release of tensor memory are still reached, and then writes NaN over its outputs and its state:
// a context reports it, a call on the caller's own states has nothing else to show it.
#include <cuda.h>

#include "prompt_kernels.h"
#include "packed.cuh"
#include "tcgen05.cuh"

namespace rssm {

namespace {

constexpr int Q = kScanChunk;
constexpr int kTile = Q * 128;  // bytes of a tile: 128 rows of 64 bf16
constexpr uint32_t kColS = 0, kColY = 128, kColG = 256, kColM = 384;
constexpr int kWarpLoad = 16, kWarpState = 17, kWarpToken = 18, kWarpTable = 19;
constexpr int kTcThreads = 640;
constexpr int kByLength = 64;

// 227 KB to the last few bytes, and tiles start on 1024-byte boundaries: there is no static shared memory in this
// file's kernels, so the block's dynamic part starts aligned (checked).
struct TcShared {
  unsigned char in[4][2][kTile];    // 0: C (halves of n); the others B (halves of n) and X (token rows, per head)
  unsigned char U[4][kTile];        // S pieces: hi, lo x halves of n; weighted X pieces: hi, lo x heads
  unsigned char Y[8][4096];         // Y on its way out: 32 tokens by 32 columns a warp
  float cl[2][Q];                   // sum of dt within the token's block of 32, included  (head, token)
  float e[2][Q];                    // exp(A (end of block - c_i)) dt_i
  __nv_bfloat16 dt[2][Q];
  float tot[2][2][4];               // sums of the blocks of 32 (chunk parity, head, block)
  uint64_t full_C, full_X[2], full_B[2], tab_full, tab_free, tot_full;
  uint64_t g_done, y1_done, y20_done, y2_done[2], y_free, s_done[2], sp_ready[2], m_ready[2], xs_ready[2], drained[2];
  uint32_t tmem;
  int abort, number;
  int not_finite;                   // X held values that are not finite (see overwrite)
  PieceWord found;
};
constexpr int kTcSmem = (int)sizeof(TcShared);
static_assert(kTcSmem <= 227 * 1024, "shared memory of a block");

// The buffers of a chunk's B and X: B(0), X(0), B(1), X(1), ... take three in turn, so that X of a chunk follows B of the
// chunk before, free when that chunk's state is done, and B follows X of two chunks before.  Without outputs there is no C:
// its buffer is a fourth, and both have two of their own.
template <bool kState>
__device__ __forceinline__ int buffer_B(int c) { return kState ? 1 + (c & 1) : 1 + 2 * c % 3; }
template <bool kState>
__device__ __forceinline__ int buffer_X(int c) { return kState ? 3 * (c & 1) : 1 + (2 * c + 1) % 3; }

struct TcArgs {
  int H, P, G, pairs;       // pairs of heads in a group
  int piece_len;
  int by_length;            // hand out the prompts by length (at most kByLength of them, not cut)
  const float *A, *D;
  const __nv_bfloat16 *x;   // [total][H][P]
  const __nv_bfloat16 *dt;  // [total][H]
  float *S;                 // [nslots][H][P][128]
  float *y;                 // [total][H][P]
  float *seg;               // piece states [pieces][H][P][128], or null: prompts are not cut
  float *seg_dt;            // their sums of dt [pieces][H]
  int *err;                 // may be null
  long long wait_cycles;
  int withhold;             // test hook: no block loads X of this chunk (-1: off)
};

__device__ __forceinline__ void scale2(uint32_t &a, uint32_t &b, f2 by) {
  float x, y;
  unpack2(mul2(pack2(a, b), by), x, y);
  a = __float_as_uint(x);
  b = __float_as_uint(y);
}

constexpr float kLog2e = 1.4426950408889634f;

struct Waiter {
  TcShared *sh;
  int *err;
  int slot;
  WaitSpec ws;
  __device__ __forceinline__ void operator()(uint64_t &bar, int phase) const {
    if (!mbar_wait_or_abort(&bar, phase & 1, &sh->abort, ws)) {
      *(volatile int *)&sh->abort = 1;
      if (err) record_error(err, slot, RSSM_DEV_TIMEOUT);
    }
  }
  // by a whole warp, whose lanes stay together
  __device__ __forceinline__ void warp(uint64_t &bar, int phase) const {
    if (__all_sync(0xffffffffu, mbar_try_wait(&bar, phase & 1, ws.hint_ns))) return;
    const long long t0 = clock64();
    while (!__all_sync(0xffffffffu, mbar_try_wait(&bar, phase & 1, ws.hint_ns))) {
      const bool late = clock64() - t0 > ws.limit;
      if (late) {
        *(volatile int *)&sh->abort = 1;
        if (err) record_error(err, slot, RSSM_DEV_TIMEOUT);
      }
      if (__any_sync(0xffffffffu, late || *(volatile int *)&sh->abort)) return;
    }
  }
};

// after a warp's writes to shared or tensor memory, or its reads of what is to be overwritten
__device__ __forceinline__ void warp_arrive(uint64_t &bar, int lane) {
  tm_fence_before();
  fence_async_smem();
  __syncwarp();
  if (lane == 0) mbar_arrive(&bar);
}

// the values of a row of X, 64 bf16, that are not finite become 0
__device__ __noinline__ void clear_not_finite(unsigned char *row) {
  for (int i = 0; i < 64; ++i) {
    unsigned short *v = reinterpret_cast<unsigned short *>(row) + i;
    if ((*v & 0x7f80) == 0x7f80) *v = 0;
  }
  fence_async_smem();
}

// A wait gave up: nothing that looks like a result stays.  Or x holds values that are not finite: M X saw zeros in their
// place, so that its own zeros above the diagonal do not carry them to earlier tokens, and from the first of them on
// the row's outputs and its state become NaN here.  What to overwrite is worked out anew, from shared memory and x: kept
// in registers all along it made the whole kernel 3 % slower, and within the kernel's own code 1.5 %.
template <bool kState>
__device__ __noinline__ void overwrite(const TcArgs &a, TcShared &sh) {
  const bool gave_up = *(volatile int *)&sh.abort;
  if (!kState && threadIdx.x % 32 == 0) bulk_wait_all();  // this warp's own stores of Y
  __syncthreads();
  const volatile PieceWord &w = sh.found;
  const int per = a.G * a.pairs, r = a.H / a.G, u = blockIdx.x % per;
  const int ha = u / a.pairs * r + 2 * (u % a.pairs), hb = min(ha + 2, (u / a.pairs + 1) * r);
  const int first = (*(volatile int *)&sh.number - (w.begin / a.piece_len + w.seq)) * a.piece_len;
  const int len = w.end - w.begin, n = min(a.piece_len, len - first);
  float *S = nullptr;
  if (kState) S = a.seg + (size_t)sh.number * a.H * a.P * kCols;
  else if (first + n >= len) S = a.S + (size_t)w.slot * a.H * a.P * kCols;
  const float nan = __int_as_float(0x7fffffff);
  int *from = reinterpret_cast<int *>(sh.cl);  // per value of a row, the first token of the piece to overwrite
  for (int h = ha; h < hb; ++h) {
    for (int p = threadIdx.x; p < a.P; p += kTcThreads) from[p] = gave_up ? 0 : n;
    __syncthreads();
    if (!gave_up) {
      for (int i = threadIdx.x / 32; i < n; i += kTcThreads / 32)
        for (int p = threadIdx.x % 32; p < a.P; p += 32) {
          const float v = __bfloat162float(a.x[((size_t)(w.begin + first + i) * a.H + h) * a.P + p]);
          if (!(fabsf(v) < __int_as_float(0x7f800000))) atomicMin(&from[p], i);
        }
      __syncthreads();
    }
    if (S)
      for (int i = threadIdx.x; i < a.P * kCols; i += kTcThreads)
        if (from[i / kCols] < n) S[(size_t)h * a.P * kCols + i] = nan;
    if (!kState)
      for (int i = threadIdx.x / 32; i < n; i += kTcThreads / 32)
        for (int p = threadIdx.x % 32; p < a.P; p += 32)
          if (i >= from[p]) a.y[((size_t)(w.begin + first + i) * a.H + h) * a.P + p] = nan;
    __syncthreads();
  }
}

// kState: only the state at the piece's end, from zero (first pass of prompts that are cut into pieces)
template <bool kState>
__global__ void __launch_bounds__(kTcThreads, 1)
    scan_tc_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_B,
                   const __grid_constant__ CUtensorMap map_C, const __grid_constant__ CUtensorMap map_y,
                   const __grid_constant__ TcArgs a, Prompts pr) {
  extern __shared__ __align__(1024) unsigned char raw[];
  TcShared &sh = *reinterpret_cast<TcShared *>(raw);
  if (smem_u32(raw) & 1023u) {
    if (threadIdx.x == 0 && a.err) record_error(a.err, 0, RSSM_DEV_TIMEOUT);
    return;
  }
  if (!kState) allow_next();
  const int units = a.G * a.pairs;
  int number = blockIdx.x / units;
  const int unit = blockIdx.x % units;
  if (a.by_length) {  // prompts that are not cut, the longest first: the last blocks to finish are short ones
    int *lens = reinterpret_cast<int *>(sh.cl);
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
  if (find_piece(pr, number, a.piece_len, pc, &sh.found) != kPieceRun) return;
  const int r = a.H / a.G, group = unit / a.pairs;
  const int h0 = group * r + 2 * (unit % a.pairs);
  const bool two = h0 + 1 < (group + 1) * r;  // without a second head the first is computed twice and stored once
  const int h1 = two ? h0 + 1 : h0;
  const int len = pc.end - pc.begin, ntok = min(a.piece_len, len - pc.first);
  const bool cut_up = len > a.piece_len, last_piece = pc.first + ntok >= len;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const size_t head_elems = (size_t)a.P * kCols;

  if (ntok <= 0 || (kState && last_piece)) {
    if (!kState && pc.index == 0 && !pc.resume) {  // an empty prompt from zero
      float *S0 = a.S + ((size_t)pc.slot * a.H + h0) * head_elems;
      for (size_t i = tid; i < head_elems * (two ? 2 : 1) / 4; i += kTcThreads) reinterpret_cast<float4 *>(S0)[i] = f4zero();
    }
    return;
  }
  const float *init = nullptr;  // state at the piece's start: [H][P][128] from its first head
  if (!kState) {
    if (cut_up) init = a.seg + (size_t)number * a.H * head_elems;
    else if (pc.resume) init = a.S + (size_t)pc.slot * a.H * head_elems;
  }
  float *final = nullptr;
  if (kState) final = a.seg + (size_t)number * a.H * head_elems;
  else if (last_piece) final = a.S + (size_t)pc.slot * a.H * head_elems;
  const int chunks = (ntok + Q - 1) / Q;
  const int t0 = pc.begin + pc.first;

  if (tid == 0) {
    uint64_t *one[] = {&sh.full_C, &sh.full_X[0], &sh.full_X[1], &sh.full_B[0], &sh.full_B[1], &sh.tab_full, &sh.tot_full, &sh.g_done, &sh.y1_done,
                       &sh.y20_done, &sh.y2_done[0], &sh.y2_done[1], &sh.s_done[0], &sh.s_done[1], &sh.drained[0],
                       &sh.drained[1]};
    for (uint64_t *b : one) mbar_init(b, 1);
    uint64_t *team[] = {&sh.y_free, &sh.sp_ready[0], &sh.sp_ready[1], &sh.m_ready[0],
                        &sh.m_ready[1], &sh.xs_ready[0], &sh.xs_ready[1]};
    for (uint64_t *b : team) mbar_init(b, 8);
    mbar_init(&sh.tab_free, kState ? 8 : 16);
    sh.abort = sh.not_finite = 0;
    sh.number = number;
    fence_barrier_init();
  }
  if (warp == kWarpLoad) tm_alloc(&sh.tmem, 512);
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  const uint32_t tm = sh.tmem;
  const Waiter wait{&sh, a.err, pc.slot, {a.wait_cycles, 0}};  // errors name the sequence, not the prompt's place

  if (warp == kWarpLoad) {
    if (lane == 0) {
      // After a wait of the block has given up nothing more is asked for than the chunk's own loads.  A barrier is armed again
      // only with its last phase over, and the products of the chunk that it was for show that as long as nobody gave up:
      // s_done of chunk c - 2 for B and X, y1_done of chunk c - 1 for C.
      auto stopped = [&] { return *(volatile int *)&sh.abort != 0; };
      int asked_B = 0, asked_C = 0, asked_X = 0;  // chunks whose loads are on their way or done
      for (int c = 0; c < chunks; ++c) {
        const int t = t0 + c * Q, s = c & 1;
        unsigned char *b = sh.in[buffer_B<kState>(c)][0], *x = sh.in[buffer_X<kState>(c)][0];
        if (kState && c > 1) wait(sh.s_done[s], (c - 2) >> 1);  // with outputs, it was waited for with the last X
        if (stopped()) break;
        if (!kState && c > 1) wait(sh.y2_done[s], (c - 2) >> 1);
        mbar_arrive_expect_tx(&sh.full_B[s], 2 * kTile);
        tma_load_2d(b, &map_B, group * kCols, t, &sh.full_B[s]);
        tma_load_2d(b + kTile, &map_B, group * kCols + 64, t, &sh.full_B[s]);
        asked_B = c + 1;
        if (!kState) {
          if (c > 0) {
            wait(sh.y1_done, c - 1);
            wait(sh.g_done, c - 1);
            if (stopped()) break;
          }
          mbar_arrive_expect_tx(&sh.full_C, 2 * kTile);
          tma_load_2d(sh.in[0][0], &map_C, group * kCols, t, &sh.full_C);
          tma_load_2d(sh.in[0][1], &map_C, group * kCols + 64, t, &sh.full_C);
          asked_C = c + 1;
        }
        if (!kState && c > 0) wait(sh.s_done[1 - s], (c - 1) >> 1);
        if (c == a.withhold) break;  // test hook: this chunk's X never comes
        mbar_arrive_expect_tx(&sh.full_X[s], 2 * kTile);
        tma_load_3d(x, &map_x, 0, h0, t, &sh.full_X[s]);
        tma_load_3d(x + kTile, &map_x, 0, h1, t, &sh.full_X[s]);
        asked_X = c + 1;
      }
      // No copy outlives the block: the last phase of each barrier that was asked for.
      if (asked_C) mbar_wait(&sh.full_C, (asked_C - 1) & 1, wait.ws);
      for (int c = max(0, asked_B - 2); c < asked_B; ++c) mbar_wait(&sh.full_B[c & 1], (c >> 1) & 1, wait.ws);
      for (int c = max(0, asked_X - 2); c < asked_X; ++c) mbar_wait(&sh.full_X[c & 1], (c >> 1) & 1, wait.ws);
    }
    __syncwarp();
  } else if (warp == kWarpState || warp == kWarpToken) {
    // The products: the whole warp goes through the steps, on values the compiler knows to be the same in every lane.
    const uint32_t leader = lane == 0, td = __shfl_sync(0xffffffffu, tm, 0);
    const int n = __shfl_sync(0xffffffffu, chunks, 0), rest = __shfl_sync(0xffffffffu, ntok, 0) - (n - 1) * Q;
    const uint32_t started = __shfl_sync(0xffffffffu, init != nullptr, 0), ends = __shfl_sync(0xffffffffu, final != nullptr, 0);
    const uint32_t dC = tile_desc(sh.in[0][0], 16);
    constexpr int step = kTile >> 4;
    if (warp == kWarpState) {
      constexpr uint32_t shape_y = mma_shape(128, 128, false, false), shape_s = mma_shape(128, 128, true, true);
      const uint32_t dSp = tile_desc(sh.U[0], 16);                                        // K-major
      const uint32_t dXs = tile_desc(sh.U[0], kTile), dB = tile_desc(sh.in[0][0], kTile);  // MN-major, two tiles
      for (int c = 0; c < n; ++c) {
        const int s = c & 1;
        const uint32_t carried = c > 0 || started;
        if (!kState) {
          wait.warp(sh.full_C, c);
          if (c > 0) wait.warp(sh.y_free, c - 1);
#pragma unroll
          for (int part = 0; part < 2; ++part) {  // columns n of S as their pieces arrive: 32 of each half
            wait.warp(sh.sp_ready[part], c);
            tm_fence_after();
            if (carried) {
#pragma unroll
              for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const int at = (k >> 1) * step + 2 * (k & 1) + 4 * part;
                  mma_ss(td + kColY, dC + at, dSp + 2 * p * step + at, shape_y, part > 0 || p > 0 || k > 0, leader);
                }
            }
          }
          mma_commit(&sh.y1_done, leader);
        } else {
          wait.warp(sh.sp_ready[0], c);
          wait.warp(sh.sp_ready[1], c);
        }
        wait.warp(sh.full_B[s], c >> 1);
#pragma unroll
        for (int part = 0; part < 2; ++part) {  // tokens as their weighted X arrives
          wait.warp(sh.xs_ready[part], c);
          tm_fence_after();
          if (c + 1 < n || ends) {
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
              for (int k = 0; k < 4; ++k) {  // 16 token rows are 2048 bytes
                const int at = 128 * (4 * part + k);
                mma_ss(td + kColS, dXs + 2 * p * step + at, dB + 2 * buffer_B<kState>(c) * step + at, shape_s,
                       part > 0 || p > 0 || k > 0 ? 1u : carried, leader);
              }
          }
        }
        mma_commit(&sh.s_done[s], leader);
      }
      mma_commit(&sh.drained[0], leader);
      mbar_wait(&sh.drained[0], 0, wait.ws);
    } else if (!kState) {
      constexpr uint32_t shape_g = mma_shape(128, 128, false, false), shape_y = mma_shape(128, 64, false, true);
      const uint32_t dB = tile_desc(sh.in[0][0], 16);
      for (int c = 0; c < n; ++c) {
        wait.warp(sh.full_B[c & 1], c >> 1);
        wait.warp(sh.full_C, c);
        tm_fence_after();
        const uint32_t b = dB + 2 * buffer_B<kState>(c) * step, x = dB + 2 * buffer_X<kState>(c) * step;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int at = (k >> 2) * step + 2 * (k & 3);
          mma_ss(td + kColG, dC + at, b + at, shape_g, k > 0, leader);
        }
        mma_commit(&sh.g_done, leader);
        wait.warp(sh.full_X[c & 1], c >> 1);
        if (c + 1 == n && rest < Q) wait.warp(sh.xs_ready[0], c);  // the rows behind the prompt's end have been cleared
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          wait.warp(sh.m_ready[h], c);
          tm_fence_after();
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int k = 0; k < 8; ++k)
              mma_ts(td + kColY + 64 * h, td + kColM + 64 * p + 8 * k, x + h * step + 128 * k, shape_y, 1, leader);
          mma_commit(h ? &sh.y2_done[c & 1] : &sh.y20_done, leader);
        }
      }
      mma_commit(&sh.drained[1], leader);
      mbar_wait(&sh.drained[1], 0, wait.ws);
    }
    __syncwarp();
  } else if (warp == kWarpTable) {
    // decay tables, a chunk ahead: lane = token of a block of 32, four blocks a head
    const __nv_bfloat16 *dtp[2] = {a.dt + (size_t)t0 * a.H + h0, a.dt + (size_t)t0 * a.H + h1};
    const float lA[2] = {a.A[h0] * kLog2e, a.A[h1] * kLog2e};
    float total_dt[2] = {0.f, 0.f};
    __nv_bfloat16 next[2][4];
    auto fetch = [&](int c) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = c * Q + 32 * i + lane;
          next[h][i] = t < ntok ? dtp[h][(size_t)t * a.H] : __ushort_as_bfloat16(0);
        }
    };
    fetch(0);
    for (int c = 0; c < chunks; ++c) {
      const int b = c & 1;
      float d[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) d[h][i] = __bfloat162float(next[h][i]);
      if (c + 1 < chunks) fetch(c + 1);
      // the state warps have read the sums of chunk c - 1 (and so waited for them), all warps those of chunk c - 2
      if (c > 0) wait(sh.sp_ready[1], c - 1);
      float cl[2][4], e[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float s = d[h][i];
#pragma unroll
          for (int off = 1; off < 32; off <<= 1) {
            const float t = __shfl_up_sync(0xffffffffu, s, off);
            if (lane >= off) s += t;
          }
          const float tot = __shfl_sync(0xffffffffu, s, 31);
          cl[h][i] = s;
          e[h][i] = exp2_approx(lA[h] * (tot - s)) * d[h][i];
          if (lane == 0) sh.tot[b][h][i] = tot;
          total_dt[h] += tot;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.tot_full);
      if (c > 0) wait(sh.tab_free, c - 1);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sh.cl[h][32 * i + lane] = cl[h][i];
          sh.e[h][32 * i + lane] = e[h][i];
          sh.dt[h][32 * i + lane] = __float2bfloat16(d[h][i]);
        }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.tab_full);
    }
    if (kState && lane == 0) {
      a.seg_dt[(size_t)number * a.H + h0] = total_dt[0];
      if (two) a.seg_dt[(size_t)number * a.H + h1] = total_dt[1];
    }
  } else if (warp < 8) {
    // token rows: M from G, Y
    if (!kState) {
      const int g = warp >> 2, q = warp & 3, row = 32 * q + lane;
      const uint32_t lanes = (uint32_t)(32 * q) << 16;
      const int hg = g ? h1 : h0;
      const float lA0 = a.A[h0] * kLog2e, lA1 = a.A[h1] * kLog2e, D0 = a.D[h0], D1 = a.D[h1];
      const bool store = g == 0 || two;
      unsigned char *stage = sh.Y[warp];
      {  // blocks above the diagonal stay zero
        const uint32_t zero[8] = {};
        for (int i = q + 1; i < 4; ++i) {
          tm_st8(tm + lanes + kColM + 16 * i + 8 * g, zero);
          tm_st8(tm + lanes + kColM + 64 + 16 * i + 8 * g, zero);
        }
      }
      // 32 columns of Y of chunk c to global memory: whole quarters through the stage, others row by row
      auto put_y = [&](const uint32_t (&v)[32], int part, int c) {
        if (!store || 32 * part >= a.P) return;
        if (lane == 0) bulk_wait_read();  // the stage's last store has left it
        __syncwarp();
        const int t = t0 + c * Q + 32 * q, valid = ntok - c * Q;
        if (32 * q + 32 <= valid) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4 *>(stage + lane * 128 + (i ^ (lane & 7)) * 16) =
                make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(&map_y, stage, 32 * part, hg, t);
            bulk_commit();
          }
        } else if (row < valid) {
          float *yp = a.y + ((size_t)(t + lane) * a.H + hg) * a.P + 32 * part;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (32 * part + 4 * i < a.P)
              *reinterpret_cast<uint4 *>(yp + 4 * i) = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
      };
      for (int c = 0; c < chunks; ++c) {
        const int b = c & 1;
        wait(sh.tab_full, c);
        wait(sh.g_done, c);
        tm_fence_after();
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          // both warps of a quarter take its rows, each 16 of a block's 32 columns
          const float lA = h ? lA1 : lA0;
          const float cl = sh.cl[h][row];
          if (h == 1) {  // M of the first head has been used
            wait(sh.y20_done, c);
            tm_fence_after();
          }
          float since = cl;  // sum of dt from the end of block i to this token
#pragma unroll 1
          for (int i = q; i >= 0; --i) {
            uint32_t G[16], hi[8], lo[8];
            tm_ld16(tm + lanes + kColG + 32 * i + 16 * g, G);
            tm_wait_ld();
            if (i < q) {
              const float f = exp2_approx(lA * since);
              const f2 ff = pack2(f, f);
              since += sh.tot[b][h][i];
#pragma unroll
              for (int k = 0; k < 16; k += 4) {
                const float4 e = *reinterpret_cast<const float4 *>(&sh.e[h][32 * i + 16 * g + k]);
                cut2(mul2(pack2(G[k], G[k + 1]), mul2(ff, pack2(e.x, e.y))), hi[k / 2], lo[k / 2]);
                cut2(mul2(pack2(G[k + 2], G[k + 3]), mul2(ff, pack2(e.z, e.w))), hi[k / 2 + 1], lo[k / 2 + 1]);
              }
            } else {
              // the block on the diagonal: its columns' tokens are this warp's rows
#pragma unroll
              for (int k = 0; k < 16; k += 4) {
                const float4 ci = *reinterpret_cast<const float4 *>(&sh.cl[h][32 * i + 16 * g + k]);
                const float4 di = load4(&sh.dt[h][32 * i + 16 * g + k]);
                const float cs[4] = {ci.x, ci.y, ci.z, ci.w}, ds[4] = {di.x, di.y, di.z, di.w};
                float m[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const int col = 16 * g + k + j;
                  const float v = __uint_as_float(G[k + j]) * (exp2_approx(lA * (cl - cs[j])) * ds[j]);
                  m[j] = col <= lane ? v : 0.f;
                }
                cut2(pack2(m[0], m[1]), hi[k / 2], lo[k / 2]);
                cut2(pack2(m[2], m[3]), hi[k / 2 + 1], lo[k / 2 + 1]);
              }
            }
            tm_st8(tm + lanes + kColM + 16 * i + 8 * g, hi);
            tm_st8(tm + lanes + kColM + 64 + 16 * i + 8 * g, lo);
          }
          if (h == 0) {
            // diag(exp(A c)) C S^T + D X in place, before M X is added; this warp's half of the columns is head g.
            // D X stays fp32: on M's diagonal, D would be cut like M and lose 2^-17 of what is often most of y.
            float sum = sh.cl[g][row];
#pragma unroll
            for (int i = 0; i < 3; ++i) sum += i < q ? sh.tot[b][g][i] : 0.f;
            const float rise = exp2_approx((g ? lA1 : lA0) * sum);
            const f2 rise2 = pack2(rise, rise), D2 = g ? pack2(D1, D1) : pack2(D0, D0);
            wait(sh.full_X[b], c >> 1);
            wait(sh.y1_done, c);
            tm_fence_after();
            uint32_t seen = 0;  // stays 0 (or -0) while the row's values are finite: the others times 0 give NaN
#pragma unroll 1
            for (int part = 0; part < 2; ++part) {
              uint32_t v[32] = {};
              if (c > 0 || init != nullptr) {
                tm_ld32(tm + lanes + kColY + 64 * g + 32 * part, v);
                tm_wait_ld();
              }
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint4 x = *reinterpret_cast<const uint4 *>(sh.in[buffer_X<kState>(c)][g] + row * 128 + ((4 * part + i) ^ (row & 7)) * 16);
                const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  uint32_t &lo = v[8 * i + 2 * j], &hi = v[8 * i + 2 * j + 1];
                  float y0, y1;
                  asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(seen) : "r"(xs[j]), "r"(0));
                  unpack2(fma2(pack2(xs[j] << 16, xs[j] & 0xffff0000u), D2, mul2(pack2(lo, hi), rise2)), y0, y1);
                  lo = __float_as_uint(y0);
                  hi = __float_as_uint(y1);
                }
              }
              tm_st32(tm + lanes + kColY + 64 * g + 32 * part, v);
            }
            if ((seen & 0x7fff7fffu) && row < ntok - c * Q) {
              clear_not_finite(sh.in[buffer_X<kState>(c)][g] + row * 128);
              *(volatile int *)&sh.not_finite = 1;
            }
          }
          tm_wait_st();
          tm_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.m_ready[h]);
        }
        if (lane == 0) mbar_arrive(&sh.tab_free);
        wait(sh.y2_done[b], c >> 1);
        tm_fence_after();
        uint32_t Y[2][32];
        tm_ld32(tm + lanes + kColY + 64 * g, Y[0]);
        tm_ld32(tm + lanes + kColY + 64 * g + 32, Y[1]);
        tm_wait_ld();
        tm_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.y_free);
        put_y(Y[0], 0, c);
        put_y(Y[1], 1, c);
      }
      if (lane == 0) bulk_wait_read();
    }
  } else {
    // state rows: weighted X, S
    const int g = (warp >> 2) & 1, q = warp & 3, t128 = tid & 127, row = t128;
    const uint32_t lanes = (uint32_t)(32 * q) << 16;
    const int hs = q >> 1;  // head of this thread's state row
    const float lAs = a.A[hs ? h1 : h0] * kLog2e, lAg = a.A[g ? h1 : h0] * kLog2e;
    const int sp = row & 63;  // its p
    // decay of this thread's state row over chunk c
    auto row_decay = [&](int c) {
      const float *t = sh.tot[c & 1][hs];
      return exp2_approx(lAs * ((t[0] + t[1]) + (t[2] + t[3])));
    };
    // 32 columns of the state row from 64 g + 32 part: pieces to U, the decayed row to tensor memory
    auto put_state = [&](uint32_t (&v)[32], int part, float decay) {
      if (!kState) {
        unsigned char *hi = sh.U[g] + row * 128, *lo = sh.U[2 + g] + row * 128;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint4 h, l;
          cut2(pack2(v[8 * i], v[8 * i + 1]), h.x, l.x);
          cut2(pack2(v[8 * i + 2], v[8 * i + 3]), h.y, l.y);
          cut2(pack2(v[8 * i + 4], v[8 * i + 5]), h.z, l.z);
          cut2(pack2(v[8 * i + 6], v[8 * i + 7]), h.w, l.w);
          const int off = ((4 * part + i) ^ (row & 7)) * 16;
          *reinterpret_cast<uint4 *>(hi + off) = h;
          *reinterpret_cast<uint4 *>(lo + off) = l;
        }
      }
#pragma unroll
      for (int i = 0; i < 32; i += 2) scale2(v[i], v[i + 1], pack2(decay, decay));
      tm_st32(tm + lanes + kColS + 64 * g + 32 * part, v);
    };

    if (init) {
      wait(sh.tot_full, 0);
      const float decay = row_decay(0);
      const float *src = init + (size_t)(hs ? h1 : h0) * head_elems + (size_t)sp * kCols + 64 * g;
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        uint32_t v[32];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 f = sp < a.P ? *reinterpret_cast<const float4 *>(src + 32 * part + 4 * i) : f4zero();
          v[4 * i] = __float_as_uint(f.x);
          v[4 * i + 1] = __float_as_uint(f.y);
          v[4 * i + 2] = __float_as_uint(f.z);
          v[4 * i + 3] = __float_as_uint(f.w);
        }
        put_state(v, part, decay);
      }
      tm_wait_st();
    }
    warp_arrive(sh.sp_ready[0], lane);
    if (lane == 0) mbar_arrive(&sh.sp_ready[1]);

    for (int c = 0; c < chunks; ++c) {
      const int b = c & 1, valid = min(Q, ntok - c * Q);
      wait(sh.tab_full, c);
      wait(sh.full_X[b], c >> 1);
      unsigned char *const X = sh.in[buffer_X<kState>(c)][g];
      if (valid < Q) {  // rows of the chunk that belong to other prompts must not reach a sum, whatever they hold
        wait(sh.full_B[b], c >> 1);
        for (int i = t128 + valid * 8; i < Q * 8; i += 128) {
          *reinterpret_cast<uint4 *>(X + 16 * i) = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4 *>(sh.in[buffer_B<kState>(c)][g] + 16 * i) = make_uint4(0, 0, 0, 0);
        }
      }
      if (!kState) wait(sh.y1_done, c);  // the pieces of S have been used
      // weighted X in two pieces, element by element in the layout of X
      float after[4];  // decay from the end of a block of 32 to the chunk's end
      {
        const float *tt = sh.tot[b][g];
        after[3] = 1.f;
        after[2] = exp2_approx(lAg * tt[3]);
        after[1] = exp2_approx(lAg * (tt[3] + tt[2]));
        after[0] = exp2_approx(lAg * (tt[3] + tt[2] + tt[1]));
      }
#pragma unroll 1
      for (int part = 0; part < 2; ++part) {
      const float w0 = part ? after[2] : after[0], w1 = part ? after[3] : after[1];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int rr = 64 * part + 16 * i + (t128 >> 3), off = rr * 128 + (t128 & 7) * 16;
        const uint4 x = *reinterpret_cast<const uint4 *>(X + off);
        const float w = sh.e[g][rr] * (i < 2 ? w0 : w1);
        uint4 h = make_uint4(0, 0, 0, 0), l = h;
        if (rr < valid) {
          const f2 ww = pack2(w, w);
          cut2(mul2(pack2(x.x << 16, x.x & 0xffff0000u), ww), h.x, l.x);
          cut2(mul2(pack2(x.y << 16, x.y & 0xffff0000u), ww), h.y, l.y);
          cut2(mul2(pack2(x.z << 16, x.z & 0xffff0000u), ww), h.z, l.z);
          cut2(mul2(pack2(x.w << 16, x.w & 0xffff0000u), ww), h.w, l.w);
        }
        *reinterpret_cast<uint4 *>(sh.U[g] + off) = h;
        *reinterpret_cast<uint4 *>(sh.U[2 + g] + off) = l;
      }
      warp_arrive(sh.xs_ready[part], lane);
      }
      if (lane == 0) mbar_arrive(&sh.tab_free);
      // the state: next chunk's operand, or the piece's result
      if (c + 1 < chunks) {
        wait(sh.s_done[b], c >> 1);
        wait(sh.tot_full, c + 1);
        const float decay = row_decay(c + 1);
        tm_fence_after();
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          uint32_t v[32];
          tm_ld32(tm + lanes + kColS + 64 * g + 32 * part, v);
          tm_wait_ld();
          put_state(v, part, decay);
          tm_wait_st();
          warp_arrive(sh.sp_ready[part], lane);
        }
      } else if (final) {
        wait(sh.s_done[b], c >> 1);
        tm_fence_after();
        float *dst = final + (size_t)(hs ? h1 : h0) * head_elems + (size_t)sp * kCols + 64 * g;
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          uint32_t v[32];
          tm_ld32(tm + lanes + kColS + 64 * g + 32 * part, v);
          tm_wait_ld();
          if (sp < a.P && (hs == 0 || two)) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<uint4 *>(dst + 32 * part + 4 * i) =
                  make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          }
        }
      }
    }
    tm_fence_before();
  }
  __syncthreads();
  if (warp == kWarpLoad) {
    tm_fence_after();
    tm_free(tm, 512);
  }
  if (*(volatile int *)&sh.abort || *(volatile int *)&sh.not_finite) overwrite<kState>(a, sh);
}

// States at the starts of the pieces of prompts that are cut: seg[s] <- state before piece s, from the pieces' own end
// states and decays, one thread four elements.  Small against the pieces' tokens, and its loads mostly hit L2.
__global__ void __launch_bounds__(256) join_kernel(TcArgs a, Prompts pr) {
  __shared__ PieceWord found;
  Piece pc;
  if (find_piece(pr, pr.off[blockIdx.x] / a.piece_len + (int)blockIdx.x, a.piece_len, pc, &found) != kPieceRun) return;
  const int len = pc.end - pc.begin, h = blockIdx.y;
  if (len <= a.piece_len) return;
  const int elem = 4 * (blockIdx.z * 256 + threadIdx.x);
  const size_t head_elems = (size_t)a.P * kCols;
  if (elem >= (int)head_elems) return;
  const int pieces = (len + a.piece_len - 1) / a.piece_len;
  const int number = pc.begin / a.piece_len + pc.seq;
  float4 carry = f4zero();
  if (pc.resume) carry = *reinterpret_cast<const float4 *>(a.S + ((size_t)pc.slot * a.H + h) * head_elems + elem);
  for (int s = 0; s < pieces; ++s) {
    const size_t at = (size_t)(number + s) * a.H + h;
    float4 *p = reinterpret_cast<float4 *>(a.seg + at * head_elems + elem);
    const float4 prev = carry;
    if (s + 1 < pieces) {
      const float4 v = *p;
      const float d = expf(a.A[h] * a.seg_dt[at]);
      carry = make_float4(fmaf(d, carry.x, v.x), fmaf(d, carry.y, v.y), fmaf(d, carry.z, v.z), fmaf(d, carry.w, v.w));
    }
    *p = prev;
  }
}

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled from the driver that is loaded (the library links the runtime alone)
cudaError_t encoder(EncodeTiled *fn) {
  void *p = nullptr;
  cudaDriverEntryPointQueryResult found;
  const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found);
  if (e != cudaSuccess) return e;
  if (found != cudaDriverEntryPointSuccess || !p) return cudaErrorNotSupported;
  *fn = reinterpret_cast<EncodeTiled>(p);
  return cudaSuccess;
}

// rows of 128 bytes with the 128-byte swizzle; what lies outside the tensor reads as zero and is not written
cudaError_t make_map(EncodeTiled fn, CUtensorMap *map, CUtensorMapDataType type, const void *p, int dims,
                     const cuuint64_t *size, const cuuint64_t *stride, const cuuint32_t *box) {
  const cuuint32_t one[3] = {1, 1, 1};
  const CUresult r = fn(map, type, dims, const_cast<void *>(p), size, stride, box, one,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

size_t scan_tc_workspace(int H, int P, int pieces, size_t *seg_dt) {
  const size_t states = align_up((size_t)pieces * H * P * kCols * 4, 256);
  if (seg_dt) *seg_dt = states;
  return states + align_up((size_t)pieces * H * 4, 256);
}

cudaError_t launch_scan_tc(const ScanArgs &s, const Prompts &pr, cudaStream_t stream) {
  TcArgs a{};
  a.H = s.H; a.P = s.P; a.G = s.G;
  a.pairs = (s.H / s.G + 1) / 2;
  a.piece_len = s.piece_len;
  a.A = s.A; a.D = s.D; a.dt = static_cast<const __nv_bfloat16 *>(s.dt); a.S = s.S; a.y = s.y;
  a.x = static_cast<const __nv_bfloat16 *>(s.x);
  a.err = s.err; a.wait_cycles = s.wait_cycles; a.withhold = s.withhold;
  const int pieces = prompt_pieces(pr.total, pr.nseq, s.piece_len);
  const bool cut_up = s.piece_len <= pr.total;
  if (cut_up) {
    size_t off;
    scan_tc_workspace(s.H, s.P, pieces, &off);
    a.seg = static_cast<float *>(s.work);
    a.seg_dt = reinterpret_cast<float *>(static_cast<unsigned char *>(s.work) + off);
  }
  // finding the order costs each block some 500 cycles, worth it where a prompt has a few chunks
  a.by_length = !cut_up && pr.nseq > 1 && pr.nseq <= kByLength && pr.total / pr.nseq >= 4 * Q;
  EncodeTiled fn;
  cudaError_t e = encoder(&fn);
  if (e != cudaSuccess) return e;
  CUtensorMap mx, mB, mC, my;
  const CUtensorMapDataType bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const cuuint64_t sx[3] = {(cuuint64_t)s.P, (cuuint64_t)s.H, (cuuint64_t)pr.total};
  const cuuint64_t tx[2] = {(cuuint64_t)s.P * 2, (cuuint64_t)s.H * s.P * 2};
  const cuuint32_t bx[3] = {64, 1, Q};
  e = make_map(fn, &mx, bf16, s.x, 3, sx, tx, bx);
  const cuuint64_t sB[2] = {(cuuint64_t)s.G * kCols, (cuuint64_t)pr.total};
  const cuuint64_t tB[1] = {(cuuint64_t)s.G * kCols * 2};
  const cuuint32_t bB[2] = {64, Q};
  if (e == cudaSuccess) e = make_map(fn, &mB, bf16, s.Bin, 2, sB, tB, bB);
  if (e == cudaSuccess) e = make_map(fn, &mC, bf16, s.C, 2, sB, tB, bB);
  const cuuint64_t ty[2] = {(cuuint64_t)s.P * 4, (cuuint64_t)s.H * s.P * 4};
  const cuuint32_t by[3] = {32, 1, 32};
  if (e == cudaSuccess) e = make_map(fn, &my, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, s.y, 3, sx, ty, by);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(scan_tc_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kTcSmem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(scan_tc_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kTcSmem);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)pieces * a.G * a.pairs;
  if (cut_up) {
    scan_tc_kernel<true><<<grid, kTcThreads, kTcSmem, stream>>>(mx, mB, mC, my, a, pr);
    join_kernel<<<dim3(pr.nseq, s.H, (s.P * kCols / 4 + 255) / 256), 256, 0, stream>>>(a, pr);
  }
  scan_tc_kernel<false><<<grid, kTcThreads, kTcSmem, stream>>>(mx, mB, mC, my, a, pr);
  return cudaGetLastError();
}

}  // namespace rssm
