// How paged attention cuts its work.  The query rows of one sequence that
// share a key head (chunk tokens x g query heads, token-major: row r is token
// r / g, head r % g of the group) are cut into tiles of R rows; a unit is one
// (sequence, key head, tile) and costs the key blocks that its last row can
// see.  All units' blocks, laid end to end in (sequence, key head, tile)
// order, are cut into one equal range per CTA, so that a few long sequences
// fill the GPU as well as many short ones, with nothing decided on the host
// (the lengths are device memory).  A unit that a range boundary cuts is
// computed in pieces: each piece leaves its unnormalised output, row maxima
// and row sums in the CTA's slot, and the piece that finishes last (a counter
// per unit) joins them in range order, so the result does not depend on who
// was last.
#pragma once

#include "common.cuh"

namespace medusa {
namespace paged {

constexpr int kCounters = 2;   // per unit: row groups that are joined on their own

struct Work {
  PagedDev kv;
  TreeDev t;               // T = 0: causal chunks
  int N, H, g;             // g = H / Hkv
  int R;                   // query rows per tile
  const int32_t* starts;
  unsigned* counters;      // kCounters per unit, zero between calls
  float* slots;            // 2 per CTA
  int* status;
};

struct Plan {
  int L[MEDUSA_MAX_B], n[MEDUSA_MAX_B], first[MEDUSA_MAX_B];
  int tile0[MEDUSA_MAX_B + 1];                  // tiles of the sequences before
  unsigned long long before[MEDUSA_MAX_B + 1];  // key blocks of the sequences before, all heads
  unsigned long long scan[12];
  int tile, block;                              // where this CTA starts
};

// A run of key blocks of one unit.
struct Piece {
  int b, h, tile;
  int kb0, kb1, blocks;        // [kb0, kb1) of the unit's blocks
  unsigned long long start;    // offset of the unit in the whole list
};

template <int BK>
struct Cut {
  static __device__ __forceinline__ int tiles(const Work& w, int n) {
    return static_cast<int>((static_cast<long long>(n) * w.g + w.R - 1) / w.R);
  }
  // Rows of the cache that the tile's last row can see.
  static __device__ __forceinline__ long long keys(const Work& w, const Plan& p, int b, int tile) {
    const int n = p.n[b];
    if (w.t.T > 0) return static_cast<long long>(p.L[b]) + n;
    const int last = static_cast<int>((static_cast<long long>(tile + 1) * w.R - 1) / w.g) + 1;
    return static_cast<long long>(p.L[b]) + (last < n ? last : n);
  }
  static __device__ __forceinline__ int blocks(const Work& w, const Plan& p, int b, int tile) {
    return static_cast<int>((keys(w, p, b, tile) + BK - 1) / BK);
  }

  // Every thread of the CTA; returns this CTA's range [begin, end) of the list
  // and sets p.tile / p.block and *b, *h to its start.
  template <int kThreads>
  static __device__ void plan(const Work& w, Plan& p, unsigned long long* begin, unsigned long long* end, int* b_out,
                              int* h_out) {
    const int tid = threadIdx.x, lane = tid & 31, B = w.kv.B;
    if (tid < MEDUSA_MAX_B) {
      int L = 0, n = 0, first = 0;
      if (tid < B) {
        L = w.kv.lens[tid];
        if (w.starts) {
          first = w.starts[tid];
          n = w.starts[tid + 1] - first;
        } else {
          n = w.N / B;
          first = n * tid;
        }
        const long long cap = static_cast<long long>(w.kv.max_pages) << w.kv.page_shift;
        const bool ok = n == 0 || (n > 0 && first >= 0 && first <= w.N - n && L >= 0 && static_cast<long long>(L) + n <= cap &&
                                   static_cast<long long>(L) + n < 0x7fffff00ll);
        if (!ok) {
          n = 0;
          if (blockIdx.x == 0) set_device_status(w.status, MEDUSA_ERR_DEVICE_CHECK, kDetailPagedChunk);
        }
      }
      p.L[tid] = L;
      p.n[tid] = n;
      p.first[tid] = first;
      p.before[tid + 1] = 0ull;              // first: key blocks of one head of the sequence
    }
    __syncthreads();
    if (tid < 32) {
      const int x = tiles(w, p.n[2 * lane]), y = tiles(w, p.n[2 * lane + 1]);
      int s = x + y;
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += v;
      }
      p.tile0[2 * lane + 1] = s - y;
      p.tile0[2 * lane + 2] = s;
      if (lane == 0) p.tile0[0] = 0;
    }
    __syncthreads();
    const int total_tiles = p.tile0[B];
    for (int t = tid; t < total_tiles; t += kThreads) {
      int lo = 0, hi = B;                    // largest b with tile0[b] <= t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.tile0[mid] <= t) lo = mid; else hi = mid;
      }
      atomicAdd(&p.before[lo + 1], static_cast<unsigned long long>(blocks(w, p, lo, t - p.tile0[lo])));
    }
    __syncthreads();
    if (tid < 32) {
      const unsigned long long hk = w.kv.Hkv;
      const unsigned long long x = p.before[2 * lane + 1] * hk, y = p.before[2 * lane + 2] * hk;
      unsigned long long s = x + y;
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long v = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += v;
      }
      p.before[2 * lane + 1] = s - y;
      p.before[2 * lane + 2] = s;
      if (lane == 0) p.before[0] = 0ull;
    }
    __syncthreads();
    // No more ranges than blocks, so that none is empty.
    const unsigned long long W = p.before[B], C = ranges(W), c = blockIdx.x;
    *begin = *end = 0ull;
    if (c >= C) return;
    *begin = W * c / C;
    *end = W * (c + 1) / C;
    int lo = 0, hi = B;                      // largest b with before[b] <= begin (empty sequences in between skip ahead)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.before[mid] <= *begin) lo = mid; else hi = mid;
    }
    unsigned long long rem = *begin - p.before[lo];
    const unsigned long long per_head = (p.before[lo + 1] - p.before[lo]) / w.kv.Hkv;
    *b_out = lo;
    *h_out = static_cast<int>(rem / per_head);
    rem -= *h_out * per_head;
    const int nt = p.tile0[lo + 1] - p.tile0[lo];
    if (nt == 1) {
      if (tid == 0) {
        p.tile = 0;
        p.block = static_cast<int>(rem);
      }
      __syncthreads();
      return;
    }
    // The tile of that head whose blocks hold offset rem.
    unsigned long long acc = 0ull;
    for (int t0 = 0; t0 < nt; t0 += kThreads) {
      const int t = t0 + tid;
      const unsigned long long mine = t < nt ? blocks(w, p, lo, t) : 0;
      unsigned long long s = mine;
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long v = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += v;
      }
      if (lane == 31) p.scan[tid >> 5] = s;
      __syncthreads();
      unsigned long long off = acc, all = acc;
      for (int k = 0; k < kThreads / 32; ++k) {
        if (k < (tid >> 5)) off += p.scan[k];
        all += p.scan[k];
      }
      s += off;
      if (mine > 0 && rem >= s - mine && rem < s) {
        p.tile = t;
        p.block = static_cast<int>(rem - (s - mine));
      }
      __syncthreads();
      acc = all;
      if (acc > rem) break;
    }
    __syncthreads();
  }

  // The first piece of a CTA's range, and the one after `x`; `left` counts the
  // range's blocks that no piece has taken yet (0: there is none).
  static __device__ __forceinline__ Piece first_piece(const Work& w, const Plan& p, unsigned long long begin, int b, int h,
                                                      unsigned long long& left) {
    Piece x;
    x.b = b;
    x.h = h;
    x.tile = p.tile;
    x.kb0 = p.block;
    x.start = begin - p.block;
    x.blocks = blocks(w, p, b, x.tile);
    take(x, left);
    return x;
  }
  static __device__ __forceinline__ void next_piece(const Work& w, const Plan& p, Piece& x, unsigned long long& left) {
    x.start += x.blocks;
    x.kb0 = 0;
    if (++x.tile == p.tile0[x.b + 1] - p.tile0[x.b]) {
      x.tile = 0;
      if (++x.h == w.kv.Hkv) {
        x.h = 0;
        do ++x.b; while (p.n[x.b] == 0);     // left > 0, so there is one
      }
    }
    x.blocks = blocks(w, p, x.b, x.tile);
    take(x, left);
  }
  static __device__ __forceinline__ void take(Piece& x, unsigned long long& left) {
    const unsigned long long room = static_cast<unsigned long long>(x.blocks - x.kb0);
    const int m = static_cast<int>(room < left ? room : left);
    x.kb1 = x.kb0 + m;
    left -= m;
  }
  static __device__ __forceinline__ bool whole(const Piece& x) { return x.kb0 == 0 && x.kb1 == x.blocks; }

  static __device__ __forceinline__ unsigned long long ranges(unsigned long long W) {
    return W < gridDim.x ? W : gridDim.x;
  }
  // The CTA whose range holds an offset of the list.
  static __device__ __forceinline__ int owner(unsigned long long off, unsigned long long W) {
    return static_cast<int>(((off + 1) * ranges(W) - 1) / W);
  }
  static __device__ __forceinline__ unsigned* counter(const Work& w, const Plan& p, const Piece& x) {
    return w.counters + (static_cast<size_t>(p.tile0[x.b] + x.tile) * w.kv.Hkv + x.h) * kCounters;
  }
  // Which of CTA c's two slots holds its piece of the unit starting at `start`.
  static __device__ __forceinline__ int slot(int c, unsigned long long start, unsigned long long W) {
    return 2 * c + (start < W * static_cast<unsigned long long>(c) / ranges(W) ? 0 : 1);
  }
};

// Bytes of the counters (for the largest possible number of units) and floats
// of a slot (R rows of hd outputs, a maximum and a sum).
inline size_t counter_bytes(int N, int H, int Hkv, int B, int R) {
  const long long tiles = (static_cast<long long>(N) * (H / Hkv) + R - 1) / R + B;
  return align_up(static_cast<size_t>(tiles) * Hkv * kCounters * sizeof(unsigned), 256);
}
constexpr size_t slot_floats(int R, int hd) { return static_cast<size_t>(R) * (hd + 2); }

}  // namespace paged
}  // namespace medusa
