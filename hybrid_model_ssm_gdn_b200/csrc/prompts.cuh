// prompts.cuh -- packed prompts: which piece of which prompt a block works on.
//
// Prompt i holds tokens off[i] .. off[i+1]-1.  Work is handed out in pieces of `len` tokens that start at the
// prompt's own first token.  The host knows the total and the number of prompts but not the offsets, so a piece
// number maps to a prompt on the device: prompt i owns the numbers off[i]/len + i .. off[i+1]/len + i, which are
// disjoint, at least one for every prompt (empty ones too) and at least ceil(length/len).  total/len + nseq numbers
// cover them all.  One coalesced pass of the block over the offsets finds the owner and checks every offset and slot
// on the way; for a few hundred prompts that is one load a thread.
#pragma once

#include "common.cuh"

namespace rssm {

struct Prompts {
  int total, nseq, nslots;
  const int *off;
  const int *slots;             // may be null
  const unsigned char *resume;  // may be null
  const int4 *meta;             // bookkeeping of a context (a resumed sequence needs an empty buffer), or null
  int refused_nan;              // whether output rows of refused prompts become NaN
};

struct Piece {
  int seq, slot;
  int begin, end;  // the prompt's tokens
  int first;       // first token of this piece, relative to begin (may lie at or past the end)
  int index;       // number of this piece within the prompt
  bool resume;
};

__host__ __device__ inline int prompt_pieces(int total, int nseq, int len) { return total / len + nseq; }

__device__ __forceinline__ bool prompt_bad(const Prompts &p, int i) {
  const int o0 = p.off[i], o1 = p.off[i + 1];
  const int s = p.slots ? p.slots[i] : i;
  return o0 < 0 || o1 < o0 || o1 > p.total || s < 0 || s >= p.nslots;
}

// what the owner of a piece leaves for its block, in shared memory
struct PieceWord {
  int seq, begin, end, slot, resume;
};

// what find_piece found: a number without owner, a piece to work on, one of a refused prompt (slot named twice, buffered
// records), or an offset or slot out of range somewhere in the call
enum PieceStatus { kPieceNone, kPieceRun, kPieceRefused, kPieceBad };

// Collective over the block.
// A block can do nothing before it knows its piece, so the loads are one round trip: a thread reads all of its prompt at
// once, before the first barrier, and the owner hands it on.
__device__ __forceinline__ PieceStatus find_piece(const Prompts &p, int number, int len, Piece &out, PieceWord *word) {
  int o0 = 0, o1 = 0, s0 = 0, r0 = 0;
  auto load = [&](int i, int &s, int &r) {
    o0 = p.off[i];
    o1 = p.off[i + 1];
    s = p.slots ? p.slots[i] : i;
    r = p.resume ? p.resume[i] : 0;
  };
  if ((int)threadIdx.x < p.nseq) load(threadIdx.x, s0, r0);
  if (threadIdx.x == 0) word->seq = -1;
  __syncthreads();
  bool bad = false;
  int s = s0, r = r0;
  for (int i = threadIdx.x; i < p.nseq; i += blockDim.x) {
    if (i >= (int)blockDim.x) load(i, s, r);
    bad |= o0 < 0 || o1 < o0 || o1 > p.total || s < 0 || s >= p.nslots;
    if (!bad && o0 / len + i <= number && number <= o1 / len + i) *word = PieceWord{i, o0, o1, s, r};
  }
  bad = __syncthreads_or(bad);
  if (bad) return kPieceBad;
  if (word->seq < 0) return kPieceNone;
  out.seq = word->seq;
  out.begin = word->begin;
  out.end = word->end;
  out.slot = word->slot;
  out.index = number - (out.begin / len + out.seq);
  out.first = out.index * len;
  out.resume = word->resume != 0;
  if (out.resume && p.meta && (p.meta[out.slot].x != 0 || p.meta[out.slot].z != 0)) return kPieceRefused;
  if (p.slots) {  // a slot named twice
    bool twice = false;
    for (int j = threadIdx.x; j < p.nseq; j += blockDim.x)
      twice |= j != out.seq && (j < (int)blockDim.x ? s0 : p.slots[j]) == out.slot;
    if (__syncthreads_or(twice)) return kPieceRefused;
  }
  return kPieceRun;
}

// lets refuse_kernel start once all blocks have come here
__device__ __forceinline__ void allow_next() { asm volatile("griddepcontrol.launch_dependents;"); }

template <typename T>
__device__ __forceinline__ void fill_nan(T *p, size_t elems, size_t part, size_t parts) {
  for (size_t i = part * blockDim.x + threadIdx.x; i < elems; i += parts * blockDim.x) p[i] = (T)__int_as_float(0x7fffffff);
}

// A block that found a piece of `len` tokens refused, or a bad offset or slot anywhere: its share of the rows of y
// [total][row] that become NaN.  `part` of `parts` blocks have the same piece.
template <typename T>
__device__ __forceinline__ void refuse(const Prompts &p, PieceStatus found, const Piece &pc, int len, T *y, size_t row,
                                       int part, int parts) {
  if (found == kPieceBad)
    fill_nan(y, p.total * row, blockIdx.y * gridDim.x + blockIdx.x, gridDim.x * gridDim.y);
  else if (found == kPieceRefused && pc.first < pc.end - pc.begin)
    fill_nan(y + (size_t)(pc.begin + pc.first) * row, min(len, pc.end - pc.begin - pc.first) * row, part, parts);
}

}  // namespace rssm
