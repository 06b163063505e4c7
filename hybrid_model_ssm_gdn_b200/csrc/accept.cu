// accept.cu -- verification of drafted tokens: the accepted prefix and the next token.
//
// The drafts' test reads two values a draft.  What costs is the draw: one row of the target's probabilities and, after
// a rejection, one of the draft's, vocab fp32 each, with a sum over all of it and the place where the running sum
// passes u times that.  The bound is memory: one pass forms the sums of contiguous chunks (one a warp), and only the
// chunk in which the sum passes the goal is read again, from L2.
//
// The drawn token is a whole number next to a border of the sums, so masses (p - q is exact in fp64) and sums are
// fp64: fp32 sums of a vocabulary's values would move the border by more than many tokens' mass.  Conversions to fp64
// run at an eighth of the fp32 rate, so the long pass makes one an element instead of two: the fp32 difference goes to the
// fp64 sum, and its rounding error, which fp32 arithmetic gives exactly, to an fp32 sum of its own (errors are below 2^-24
// of their values and lose 2^-24 of that in turn).  Infinities are not looked for: they show in the sum.
//
// A cluster of blocks shares a sequence (when there are few, so that one row is read by several SMs); the blocks'
// totals are exchanged through distributed shared memory.
//
// Measured: 256 sequences, vocabulary 131072, with draft rows, 54 us (226 MB, 35 us at the copy bandwidth), 64 us
// with five blocks an SM instead of eight and lines left in L1.  What is left besides the stream are a
// sequence's dependent steps: drafts, their probabilities, sums, totals, search.
#include <cooperative_groups.h>

#include "prompt_kernels.h"

namespace cg = cooperative_groups;

namespace rssm {

namespace {

constexpr int kWarps = 8;
constexpr int kUnroll = 8;
constexpr int kBlocksSm = 8;  // 32 registers a thread: more loads in flight count for more than longer rounds
constexpr int kFine = 256;  // longest run that one warp searches by itself: 8 consecutive elements a lane

struct Row {
  const float *p, *q;  // q null: no draft row
  int hot;             // element without mass (a rejected draft that was looked up), or -1
  __device__ __forceinline__ double mass(int v) const {
    const float pv = p[v];
    double m = (double)pv;
    if (q) m -= (double)q[v];
    return (m > 0.0 && m < __longlong_as_double(0x7ff0000000000000LL) && v != hot) ? m : 0.0;
  }
};

// A load that keeps its place in the source, so that all of a round are on their way before the first is used, and leaves
// no line in L1, which the stream would only fill (256 rows of 131072: 64 us with the L2 cold; with lines in L1 72 us).
__device__ __forceinline__ float load_now(const float *p) {
  float v;
  asm volatile("ld.global.L1::no_allocate.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}

__device__ __forceinline__ double warp_sum_f64(double v) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// sum of the masses of [lo, hi), the whole warp
template <bool kDraft>
__device__ __forceinline__ double warp_mass(const Row &r, int lo, int hi, int lane) {
  double s = 0.0;
  float lost = 0.f;
  auto add = [&](float p, float q, int v) {
    if (kDraft) {
      const float d = p - q, back = d - p;
      const float err = (p - (d - back)) - (q + back);  // p - q = d + err, unless d overflows: then err is no number
      s += (double)(d > 0.f ? d : 0.f);
      lost += d > 0.f ? err : 0.f;
    } else {
      s += (double)(p > 0.f && v != r.hot ? p : 0.f);
    }
  };
  int v = lo + lane;
  for (; v + (kUnroll - 1) * 32 < hi; v += kUnroll * 32) {
    float p[kUnroll], q[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      p[i] = load_now(r.p + v + 32 * i);
      q[i] = kDraft ? load_now(r.q + v + 32 * i) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) add(p[i], q[i], v + 32 * i);
  }
  for (; v < hi; v += 32) add(r.p[v], kDraft ? r.q[v] : 0.f, v);
  s = warp_sum_f64(s + (double)lost);
  if (!(s < __longlong_as_double(0x7ff0000000000000LL))) {  // an infinity, or a difference beyond fp32's range: once more
    s = 0.0;
    for (v = lo + lane; v < hi; v += 32) s += r.mass(v);
    s = warp_sum_f64(s);
  }
  return s;
}
__device__ __forceinline__ double warp_mass(const Row &r, int lo, int hi, int lane) {
  return r.q ? warp_mass<true>(r, lo, hi, lane) : warp_mass<false>(r, lo, hi, lane);
}

// lowest v of [lo, hi), at most kFine long, where base + the inclusive sum passes goal; else the last one with mass;
// else -1.  Whole warp.
__device__ __forceinline__ int warp_find(const Row &r, int lo, int hi, double base, double goal, int lane) {
  double m[8], own = 0.0;
  const int v0 = lo + 8 * lane;
#pragma unroll
  for (int i = 0; i < 8; ++i) m[i] = v0 + i < hi ? r.mass(v0 + i) : 0.0;
#pragma unroll
  for (int i = 0; i < 8; ++i) own += m[i];
  double s = own;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const double t = __shfl_up_sync(0xffffffffu, s, off);
    if (lane >= off) s += t;
  }
  const unsigned pass = __ballot_sync(0xffffffffu, own > 0.0 && base + s > goal);
  const unsigned any = __ballot_sync(0xffffffffu, own > 0.0);
  if (!any) return -1;
  const int who = pass ? __ffs(pass) - 1 : 31 - __clz(any);
  const double before = __shfl_up_sync(0xffffffffu, s, 1);
  double run = base + (lane > 0 ? before : 0.0);
  int v = -1;
  bool found = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    run += m[i];
    if (m[i] > 0.0 && !found) {
      v = v0 + i;
      found = run > goal;
    }
  }
  return __shfl_sync(0xffffffffu, v, who);
}

struct Shared {
  double sum[kWarps];   // masses of the warps' chunks
  double total;         // of the block's slice
  int n, count;
};

__global__ void __launch_bounds__(kWarps * 32, kBlocksSm) accept_kernel(AcceptArgs a) {
  __shared__ Shared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = cluster.block_rank(), blocks = cluster.num_blocks();
  const int b = blockIdx.x / blocks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int T = a.T;

  if (warp == 0) {  // every block of the cluster tests the drafts for itself
    // a draft past the sequence's own number is read all the same, so that its number and its token come together
    const int count = a.count ? max(0, min(T, a.count[b])) : T;
    bool stands = false;
    if (lane < T) {
      const int d = a.tokens[(size_t)b * T + lane];
      const double u = a.u[(size_t)b * (T + 1) + lane];
      if (lane < count && d >= 0 && d < a.vocab) {
        const double p = a.target[((size_t)b * (T + 1) + lane) * a.ld_target + d];
        const double q = a.draft ? (double)a.draft[((size_t)b * T + lane) * a.ld_draft + d] : 1.0;
        stands = p > 0.0 && p < __longlong_as_double(0x7ff0000000000000LL) && u * q < p;  // 24 x 24 bits: exact
      }
    }
    const unsigned fell = ~__ballot_sync(0xffffffffu, stands);
    if (lane == 0) {
      sh.n = __ffs(fell) - 1;  // T <= 16 lanes take part, so some lane always falls
      sh.count = count;
    }
  }
  __syncthreads();
  const int n = sh.n;
  const bool rejected = n < sh.count;
  const double u = a.u[(size_t)b * (T + 1) + T];

  Row r;
  r.p = a.target + ((size_t)b * (T + 1) + n) * a.ld_target;
  r.q = rejected && a.draft ? a.draft + ((size_t)b * T + n) * a.ld_draft : nullptr;
  r.hot = rejected && !a.draft ? a.tokens[(size_t)b * T + n] : -1;

  // block `rank` owns [lo, hi), warp w the chunk [w0, w1) of it
  const int slice = (a.vocab + blocks - 1) / blocks;
  const int lo = min(a.vocab, rank * slice), hi = min(a.vocab, lo + slice);
  const int chunk = ((slice + kWarps - 1) / kWarps + 31) / 32 * 32;
  const int w0 = min(hi, lo + warp * chunk), w1 = min(hi, w0 + chunk);

  double total = 0.0, before = 0.0;
  bool mine = false;
  for (int attempt = 0; attempt < 2; ++attempt) {
    const double s = warp_mass(r, w0, w1, lane);
    if (lane == 0) sh.sum[warp] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
      double t = 0.0;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) t += sh.sum[i];
      sh.total = t;
    }
    cluster.sync();
    total = before = 0.0;
    int owner = -1;
    const double slices = lane < blocks ? *cluster.map_shared_rank(&sh.total, lane) : 0.0;
    for (int i = 0; i < blocks; ++i) total += __shfl_sync(0xffffffffu, slices, i);
    const double goal = u * total;
    double run = 0.0;
    for (int i = 0; i < blocks; ++i) {  // the first slice whose end passes the goal, else the last with mass
      const double t = __shfl_sync(0xffffffffu, slices, i);
      if (t > 0.0) {
        owner = i;
        before = run;
        run += t;
        if (run > goal) break;
      }
    }
    mine = owner == rank;
    cluster.sync();  // the totals have been read
    if (total > 0.0 || (r.q == nullptr && r.hot < 0)) break;
    r.q = nullptr;  // nothing is left of max(p - q, 0): draw from p
    r.hot = -1;
  }

  if (rank == 0 && threadIdx.x == 0) {
    a.accepted[b] = n;
    if (a.committed) a.committed[b] = n + 1;
    if (!(total > 0.0)) a.next[b] = -1;
  }
  if (!mine) return;
  const double goal = u * total;
  int pick = 0;  // the chunk in the slice, by the same rule
  double base = before, run = before;
  for (int i = 0; i < kWarps; ++i) {
    if (sh.sum[i] > 0.0) {
      pick = i;
      base = run;
      run += sh.sum[i];
      if (run > goal) break;
    }
  }
  int f0 = min(hi, lo + pick * chunk), f1 = min(hi, f0 + chunk);
  while (f1 - f0 > kFine) {  // a long chunk: a part a warp, then one of them
    const int part = ((f1 - f0 + kWarps - 1) / kWarps + 31) / 32 * 32;
    const int p0 = min(f1, f0 + warp * part), p1 = min(f1, p0 + part);
    const double s = warp_mass(r, p0, p1, lane);
    __syncthreads();  // the last sums have been read
    if (lane == 0) sh.sum[warp] = s;
    __syncthreads();
    double at = base;
    run = base;
    pick = 0;
    for (int i = 0; i < kWarps; ++i) {
      if (sh.sum[i] > 0.0) {
        pick = i;
        at = run;
        run += sh.sum[i];
        if (run > goal) break;
      }
    }
    base = at;
    f0 = min(f1, f0 + pick * part);
    f1 = min(f1, f0 + part);
  }
  if (warp == 0) {
    const int v = warp_find(r, f0, f1, base, goal, lane);
    if (lane == 0) a.next[b] = v;
  }
}

}  // namespace

cudaError_t launch_accept(const AcceptArgs &a, int num_sms, cudaStream_t stream) {
  // Blocks a sequence: up to the portable cluster of 8 as long as all of them fit the SMs at once (eight an SM; 1024 rows
  // of 8000: 25 us, and 29 us with twice the blocks), none with less than 2048 elements, one round of loads of a block.
  int blocks = 1;
  while (blocks < 8 && (long long)a.batch * blocks * 2 <= (long long)kBlocksSm * num_sms && a.vocab / (blocks * 2) >= 2048) blocks *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)a.batch * blocks);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = blocks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, accept_kernel, a);
}

}  // namespace rssm
