// accept.cu -- verification of drafted tokens: the accepted prefix and the next token.
//
// The drafts' test reads two values a draft.  What costs is the draw: one row of the target's probabilities and, after
// a rejection, one of the draft's, vocab fp32 each, with a sum over all of it and the place where the running sum
// passes u times that.  The bound is memory: one pass forms the sums of contiguous chunks (one a warp), and only the
// chunk in which the sum passes the goal is read again, from L2.
//
// The drawn token is a whole number next to a border of the sums, so masses (p - q is exact in fp64) and sums are
// fp64: fp32 sums of a vocabulary's values would move the border by more than many tokens' mass.
//
// A cluster of blocks shares a sequence (when there are few, so that one row is read by several SMs); the blocks'
// totals are exchanged through distributed shared memory.
#include <cooperative_groups.h>

#include "kernels.h"

namespace cg = cooperative_groups;

namespace rssm {

namespace {

constexpr int kWarps = 16;
constexpr int kFine = 1024;  // longest run that one warp scans element by element

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

__device__ __forceinline__ double warp_sum_f64(double v) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// sum of the masses of [lo, hi), the whole warp
__device__ __forceinline__ double warp_mass(const Row &r, int lo, int hi, int lane) {
  double s0 = 0.0, s1 = 0.0;
  int v = lo + lane;
  for (; v + 7 * 32 < hi; v += 8 * 32) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      s0 += r.mass(v + i * 32);
      s1 += r.mass(v + (i + 1) * 32);
    }
  }
  for (; v < hi; v += 32) s0 += r.mass(v);
  return warp_sum_f64(s0 + s1);
}

// lowest v of [lo, hi) where base + the inclusive sum passes goal; else the last one with mass; else -1.  Whole warp.
__device__ __forceinline__ int warp_find(const Row &r, int lo, int hi, double base, double goal, int lane) {
  int last = -1;
  for (int v0 = lo; v0 < hi; v0 += 32) {
    const int v = v0 + lane;
    const double m = v < hi ? r.mass(v) : 0.0;
    double s = m;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const double t = __shfl_up_sync(0xffffffffu, s, off);
      if (lane >= off) s += t;
    }
    const unsigned pass = __ballot_sync(0xffffffffu, m > 0.0 && base + s > goal);
    if (pass) return v0 + __ffs(pass) - 1;
    const unsigned any = __ballot_sync(0xffffffffu, m > 0.0);
    if (any) last = v0 + 31 - __clz(any);
    base += __shfl_sync(0xffffffffu, s, 31);
  }
  return last;
}

struct Shared {
  double sum[kWarps];   // masses of the warps' chunks
  double total;         // of the block's slice
  int n, count;
  int pick;
  double base;
};

__global__ void __launch_bounds__(kWarps * 32) accept_kernel(AcceptArgs a) {
  __shared__ Shared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = cluster.block_rank(), blocks = cluster.num_blocks();
  const int b = blockIdx.x / blocks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int T = a.T;

  if (warp == 0) {  // every block of the cluster tests the drafts for itself
    const int count = a.count ? max(0, min(T, a.count[b])) : T;
    bool stands = false;
    if (lane < count) {
      const int d = a.tokens[(size_t)b * T + lane];
      if (d >= 0 && d < a.vocab) {
        const double p = a.target[((size_t)b * (T + 1) + lane) * a.ld_target + d];
        const double q = a.draft ? (double)a.draft[((size_t)b * T + lane) * a.ld_draft + d] : 1.0;
        stands = (double)a.u[(size_t)b * (T + 1) + lane] * q < p;  // 24 x 24 bits: exact
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
    double mass = 0.0;
    int owner = -1;
    double goal = 0.0;
    for (int i = 0; i < blocks; ++i) total += *cluster.map_shared_rank(&sh.total, i);
    goal = u * total;
    double run = 0.0;
    for (int i = 0; i < blocks; ++i) {  // the first slice whose end passes the goal, else the last with mass
      const double t = *cluster.map_shared_rank(&sh.total, i);
      if (t > 0.0) {
        owner = i;
        before = run;
        mass = run + t;
        run += t;
        if (mass > goal) break;
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
  if (threadIdx.x == 0) {  // the chunk in the slice, by the same rule
    double run = before;
    int pick = 0;
    double base = before;
    for (int i = 0; i < kWarps; ++i) {
      if (sh.sum[i] > 0.0) {
        pick = i;
        base = run;
        run += sh.sum[i];
        if (run > goal) break;
      }
    }
    sh.pick = pick;
    sh.base = base;
  }
  __syncthreads();
  int f0 = min(hi, lo + sh.pick * chunk), f1 = min(hi, f0 + chunk);
  double base = sh.base;
  while (f1 - f0 > kFine) {  // a long chunk: its 16 parts, then one of them
    const int part = ((f1 - f0 + kWarps - 1) / kWarps + 31) / 32 * 32;
    const int p0 = min(f1, f0 + warp * part), p1 = min(f1, p0 + part);
    const double s = warp_mass(r, p0, p1, lane);
    __syncthreads();
    if (lane == 0) sh.sum[warp] = s;
    __syncthreads();
    double run = base;
    int pick = 0;
    double at = base;
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
  // Blocks a sequence: as many as fill the SMs once (two blocks fit an SM), up to the portable cluster of 8, and
  // none with less than 4096 elements, below which the exchange costs more than the reading it spreads.
  int blocks = 1;
  while (blocks < 8 && (long long)a.batch * blocks * 2 <= 2LL * num_sms && a.vocab / (blocks * 2) >= 4096) blocks *= 2;
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
