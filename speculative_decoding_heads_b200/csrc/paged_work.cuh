// How paged attention cuts its work.  The query rows of one sequence that
// share a key head (chunk tokens x g query heads, token-major: row r is token
// r / g, head r % g of the group) are cut into tiles of R rows; a unit is one
// (sequence, key head, tile) and costs the key blocks that its last row can
// see.  All units' blocks, laid end to end in (sequence, key head, tile)
// order, are cut into one equal range per CTA, so that a few long sequences
// fill the GPU as well as many short ones, with nothing decided on the host
// (the lengths are device memory).  Behind every unit come a few blocks that
// nobody computes: its set-up and output cost as much, and a CTA with many
// short units gets fewer blocks.  A unit that a range boundary cuts is
// computed in pieces: each piece leaves its unnormalised output, row maxima
// and row sums in the CTA's slot, and the piece that finishes last (a counter
// per unit and row group) joins them in range order, so the result does not
// depend on who was last.
//
// Where a sequence's units all cost the same (one tile, or a tree's) and there
// are fewer units than CTAs (a few requests decoding), a cut at unit boundaries
// is better: every unit gets a whole number of CTAs, at most `each` blocks to
// each, and no CTA pays for two pieces.  It is taken when it costs a CTA at
// most two blocks more than the equal cut (the set-up and output of a second
// piece take about as long): one token of 32 heads over 1024 rows 10.9 us, cut
// equally 13.0.
//
// One warp lays the plan, two sequences to a lane: the blocks of a sequence's
// first t tiles, sum_{i=1..t} ceil((g L + i R) / (g BK)), have a closed form
// (the floor sum of an arithmetic progression, by the Euclidean descent of
// its slope), so neither the total nor a CTA's start needs a walk over tiles.
#pragma once

#include <climits>

#include "common.cuh"

namespace medusa {
namespace paged {

constexpr int kCounters = 2;   // per unit: row groups that are joined on their own
constexpr int kNoPage = INT_MIN;   // in place of a table entry: nothing to look up

// x / d for 0 <= x < 2^31 and 1 <= d <= 2^15 as one product: with 2^k >= d and
// m = ceil(2^(31+k) / d), x m / 2^(31+k) exceeds x / d by less than 2^-k <= 1/d.
// (The chain of divisions between two units took the products' warp 2000 clocks.)
struct Divisor {
  unsigned m;
  int shift;
  Divisor() = default;
  explicit Divisor(unsigned d) {
    shift = 31;
    while ((1u << (shift - 31)) < d) ++shift;
    m = static_cast<unsigned>(((1ull << shift) + d - 1) / d);
  }
};
__device__ __forceinline__ int operator/(int x, const Divisor& d) {
  return static_cast<int>((static_cast<unsigned long long>(static_cast<unsigned>(x)) * d.m) >> d.shift);
}

struct Work {
  PagedDev kv;
  TreeDev t;               // T = 0: causal chunks
  int N, H, g;             // g = H / Hkv
  int R;                   // query rows per tile
  Divisor by_g, by_R, by_hk;
  float join;              // joining one piece of a unit, in units of computing one block
  unsigned extra;          // blocks that a unit's set-up and output cost besides its own
  const int32_t* starts;
  float* slots;            // 2 per CTA, at the start of the workspace
  unsigned* counters;      // kCounters per unit, zero between calls
  int* status;
  uint64_t wait_limit;     // ns after which a wait gives up
  unsigned wait_extra;     // test hook: arrivals that one barrier expects and never gets
};

struct Plan {
  int L[MEDUSA_MAX_B], n[MEDUSA_MAX_B], first[MEDUSA_MAX_B];
  unsigned each;                       // cut at unit boundaries: blocks per CTA; 0: equal ranges
  unsigned extra;                      // equal ranges: Work::extra, otherwise 0
  unsigned per, more;                  // equal ranges: blocks of a CTA, and how many of the first hold one more
  unsigned begin, end;                 // this CTA's range
  int b, h, tile, block;               // where it starts
  int lo, hi;                          // cut at unit boundaries: the CTAs of its unit
};

// A run of key blocks of one unit.
struct Piece {
  int b, h, tile;
  int kb0, kb1, blocks;        // [kb0, kb1) of the unit's blocks
  unsigned start;              // offset of the unit in the whole list
};

// sum_{i=0}^{n-1} floor((a i + b) / m); a n + b below 2^32.
__device__ __forceinline__ unsigned long long floor_sum(unsigned n, unsigned m, unsigned a, unsigned b) {
  unsigned long long s = 0;
  while (n > 0) {
    if (a >= m) {
      s += static_cast<unsigned long long>(n) * (n - 1) / 2 * (a / m);
      a %= m;
    }
    if (b >= m) {
      s += static_cast<unsigned long long>(n) * (b / m);
      b %= m;
    }
    const unsigned y = a * n + b;             // the line's height: count its lattice points from the other axis
    if (y < m) break;
    n = y / m;
    b = y % m;
    const unsigned t = m;
    m = a;
    a = t;
  }
  return s;
}

template <int BK>
struct Cut {
  // Rows of the cache that the tile's last row can see.
  static __device__ __forceinline__ int keys(const Work& w, const Plan& p, int b, int tile) {
    const int n = p.n[b];
    if (w.t.T > 0) return p.L[b] + n;
    const int last = ((tile + 1) * w.R - 1) / w.by_g + 1;
    return p.L[b] + (last < n ? last : n);
  }
  static __device__ __forceinline__ int blocks(const Work& w, const Plan& p, int b, int tile) {
    return (keys(w, p, b, tile) + BK - 1) / BK;
  }
  // Blocks of the first t tiles of one head.
  static __device__ __forceinline__ unsigned long long before_tile(const Work& w, int L, int n, int tiles, int t) {
    const unsigned long long all = (static_cast<unsigned>(L) + n + BK - 1) / BK;
    if (t == 0) return 0ull;
    if (w.t.T > 0) return all * t;
    // With L = BK q + r the quotients are q + ceil((g r + i R) / (g BK)): 32 bits suffice (t R < 2^31).
    const unsigned m = w.g * BK, q = static_cast<unsigned>(L) / BK, r = static_cast<unsigned>(L) % BK;
    const int k = t < tiles ? t : tiles - 1;     // the last tile ends with the chunk
    const unsigned long long s =
        k == 0 ? 0ull : static_cast<unsigned long long>(k) * q + floor_sum(k, m, w.R, w.g * r + w.R + m - 1);
    return t < tiles ? s : s + all;
  }
  static __device__ __forceinline__ int tiles_of(const Work& w, int n) { return (n * w.g + w.R - 1) / w.by_R; }

  static_assert(MEDUSA_MAX_B <= 64, "two sequences to a lane of the plan's warp");
  // One whole warp; the other threads see the plan after the next __syncthreads.
  static __device__ void plan(const Work& w, Plan& p) {
    const int lane = threadIdx.x & 31, B = w.kv.B;
    const unsigned hk = w.kv.Hkv;
    int L[2], n[2], tiles[2];
    unsigned long long work[2];
    const long long cap = static_cast<long long>(w.kv.max_pages) << w.kv.page_shift;
    bool bad = false, descends = false;
    int first[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int b = 2 * lane + i;
      first[i] = 0;
      L[i] = n[i] = 0;
      if (b < B) {
        L[i] = w.kv.lens[b];
        if (w.starts) {
          first[i] = w.starts[b];
          n[i] = w.starts[b + 1] - first[i];
          descends |= n[i] < 0;
        } else {
          n[i] = w.N / B;
          first[i] = n[i] * b;
        }
        const bool ok = n[i] == 0 || (n[i] > 0 && first[i] >= 0 && first[i] <= w.N - n[i] && L[i] >= 0 &&
                                      static_cast<long long>(L[i]) + n[i] <= cap &&
                                      static_cast<long long>(L[i]) + n[i] <= kMaxPagedRows);
        if (!ok) {
          n[i] = 0;
          bad = true;
        }
      }
    }
    const bool none = __any_sync(0xffffffffu, descends);   // overlapping chunks: nothing is computed
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int b = 2 * lane + i;
      if (none) n[i] = 0;
      p.L[b] = L[i];
      p.n[b] = n[i];
      p.first[b] = first[i];
      tiles[i] = tiles_of(w, n[i]);
      work[i] = n[i] > 0 ? before_tile(w, L[i], n[i], tiles[i], tiles[i]) * hk : 0ull;
      if (work[i] > 1ull << 31) work[i] = 1ull << 31;      // too many on its own: refused below
    }
    // Tiles (N g / R + B: below 2^25) and blocks (at most 2^37), summed over the lanes before in one word.
    unsigned long long both = (work[0] + work[1]) << 26 | static_cast<unsigned>(tiles[0] + tiles[1]);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long v = __shfl_up_sync(0xffffffffu, both, o);
      if (lane >= o) both += v;
    }
    const unsigned long long ws = both >> 26;
    const unsigned upto = static_cast<unsigned>(both & 0x3ffffffu);   // tiles, this lane's included
    both = __shfl_sync(0xffffffffu, both, 31);
    unsigned long long W = both >> 26;
    if (W > 0x3fffffffull) {     // 2^30 blocks of keys in one call: refused like any other impossible chunk
      W = 0;
      bad = true;
    }
    if (bad && blockIdx.x == 0) set_device_status(w.status, MEDUSA_ERR_DEVICE_CHECK, kDetailPagedChunk);
    const unsigned c = blockIdx.x, C = gridDim.x, units = static_cast<unsigned>(both & 0x3ffffffu) * hk;
    // A unit of n blocks in pieces of k takes about k + join n / k: below k =
    // sqrt(join n) a finer cut costs more than it gains (a 64-node tree of 8
    // heads on one key head over 2000 rows 21.4 us, without this bound 36;
    // 500 tokens of two such heads after 3000 rows 28, 53; the same tree of
    // four heads over 8000 rows 23, 34).
    const unsigned least = W > 0 ? max(1, __float2int_rn(sqrtf(w.join * static_cast<float>(W) / static_cast<float>(units)))) : 1u;
    if (W > 0 && units < C && (w.t.T > 0 || __all_sync(0xffffffffu, tiles[0] <= 1 && tiles[1] <= 1))) {
      // sum_u ceil(blocks_u / each) <= W / each + units <= C
      const unsigned total = static_cast<unsigned>(W);
      unsigned each = (total + C - units - 1) / (C - units);
      if (each <= 2 || static_cast<unsigned long long>(each - 2) * C <= total) {
        each = max(each, least);
        if (lane == 0) {
          p.each = each;
          p.extra = 0u;
          p.begin = p.end = 0;
        }
        __syncwarp();
        unsigned cnt[2], blk[2], all[2];                  // a unit's CTAs and blocks, a sequence's CTAs
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          blk[i] = static_cast<int>(work[i]) / w.by_hk;
          if (tiles[i] > 1) blk[i] /= tiles[i];           // all of a tree's tiles see the same keys
          cnt[i] = (blk[i] + each - 1) / each;
          all[i] = cnt[i] * hk * tiles[i];
        }
        unsigned at = all[0] + all[1];                    // CTAs before the next lane's sequences
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned v = __shfl_up_sync(0xffffffffu, at, o);
          if (lane >= o) at += v;
        }
        at -= all[0] + all[1];
        const int i = c >= at + all[0] ? 1 : 0;
        if (i) at += all[0];
        const unsigned k = i ? cnt[1] : cnt[0], nb = i ? blk[1] : blk[0], nt = i ? tiles[1] : tiles[0];
        if (c >= at && c < at + (i ? all[1] : all[0])) {
          const unsigned u = (c - at) / k, part = c - at - u * k, h = nt > 1 ? u / nt : u;
          p.b = 2 * lane + i;
          p.h = static_cast<int>(h);
          p.tile = static_cast<int>(u - h * nt);
          // Inside 32 bits: the condition above holds only for W <= 2 C (C - units) / units, so nb k <= 2 C^3 < 2^30.
          p.block = static_cast<int>(nb * part / k);
          p.end = nb * (part + 1) / k - p.block;
          p.lo = static_cast<int>(at + u * k);
          p.hi = static_cast<int>(at + u * k + k - 1);
        }
        return;
      }
    }
    // No more ranges than blocks, so that none is empty.
    const unsigned fit = max(1u, static_cast<unsigned>(W) / least), r = W == 0 ? 0u : min(fit, C);
    // Every unit is followed by its extra blocks, which nobody computes.
    const unsigned all = static_cast<unsigned>(W) + (W == 0 ? 0u : w.extra * units), per = r > 0 ? all / r : 0u;
    const unsigned more = all - per * r;
    const unsigned begin = c < r ? range_begin(c, per, more) : 0u;
    const unsigned end = c < r ? range_begin(c + 1, per, more) : 0u;
    if (lane == 0) {
      p.per = per;
      p.more = more;
      p.each = 0u;
      p.extra = w.extra;
      p.begin = begin;
      p.end = end;
    }
    if (begin >= end) return;
    // The lane whose sequences hold offset begin, and where in them it lies.
    work[0] += w.extra * hk * tiles[0];
    work[1] += w.extra * hk * tiles[1];
    const unsigned long long to = ws + w.extra * hk * upto, from = to - work[0] - work[1];
    unsigned long long off = from;                        // blocks before this lane's sequences
    const int src = __ffs(__ballot_sync(0xffffffffu, begin >= from && begin < to)) - 1;
    const int i = begin >= off + work[0] ? 1 : 0;
    if (i) off += work[0];
    const unsigned rem = begin - static_cast<unsigned>(off), per_head = static_cast<int>(i ? work[1] : work[0]) / w.by_hk;
    const unsigned head = per_head > 0 ? rem / per_head : 0u;
    const unsigned at = __shfl_sync(0xffffffffu, rem - head * per_head, src);
    const int Li = __shfl_sync(0xffffffffu, i ? L[1] : L[0], src), ni = __shfl_sync(0xffffffffu, i ? n[1] : n[0], src);
    const int nt = __shfl_sync(0xffffffffu, i ? tiles[1] : tiles[0], src);
    // The largest tile with before_tile(tile) <= at: all lanes probe, 32 tiles apart by powers of 32.
    int lo = 0;
    unsigned at_lo = 0u;
    int step = 1;
    while (step * 32 < nt) step *= 32;
    for (; nt > 1 && step > 0; step /= 32) {
      const long long t = lo + static_cast<long long>(lane) * step;
      const unsigned long long s = t < nt ? before_tile(w, Li, ni, nt, static_cast<int>(t)) + w.extra * static_cast<unsigned>(t) : ~0ull;
      const int k = 31 - __clz(__ballot_sync(0xffffffffu, s <= at));   // lane 0's always is
      lo += k * step;
      at_lo = __shfl_sync(0xffffffffu, static_cast<unsigned>(s), k);
    }
    __syncwarp();              // the lengths of all sequences, and lane 0's begin and end
    if (lane == src) {
      Piece x;
      x.b = 2 * lane + i;
      x.h = static_cast<int>(head);
      x.tile = lo;
      int block = static_cast<int>(at - at_lo);
      const int own = blocks(w, p, x.b, lo);
      if (block >= own) {      // behind a unit's own blocks: the next unit's, if the range reaches it
        const unsigned skip = own + w.extra - block;
        p.begin = end - begin > skip ? begin + skip : end;
        block = 0;
        if (end - begin > skip) next_unit(w, p, x);
      }
      p.b = x.b;
      p.h = x.h;
      p.tile = x.tile;
      p.block = block;
    }
  }

  static __device__ __forceinline__ unsigned range_begin(unsigned c, unsigned per, unsigned more) {
    return per * c + (c < more ? c : more);
  }
  // The CTAs that hold a piece's unit.
  static __device__ __forceinline__ void owners(const Plan& p, const Piece& x, int& lo, int& hi) {
    lo = p.each ? p.lo : owner(p, x.start);
    hi = p.each ? p.hi : owner(p, x.start + x.blocks - 1);
  }
  static __device__ __forceinline__ int owner(const Plan& p, unsigned off) {
    const unsigned longer = p.more * (p.per + 1);
    return off < longer ? off / (p.per + 1) : p.more + (off - longer) / p.per;
  }

  // The first piece of a CTA's range, and the one after `x`; `left` counts the
  // range's blocks that no piece has taken yet (0: there is none).
  static __device__ __forceinline__ Piece first_piece(const Work& w, const Plan& p, unsigned& left) {
    Piece x;
    left = p.end - p.begin;
    x.b = p.b;
    x.h = p.h;
    x.tile = p.tile;
    x.kb0 = p.block;
    x.start = p.begin - p.block;
    x.blocks = blocks(w, p, x.b, x.tile);
    take(p, x, left);
    return x;
  }
  static __device__ __forceinline__ void next_piece(const Work& w, const Plan& p, Piece& x, unsigned& left) {
    x.start += x.blocks + p.extra;
    x.kb0 = 0;
    next_unit(w, p, x);
    x.blocks = blocks(w, p, x.b, x.tile);
    take(p, x, left);
  }
  static __device__ __forceinline__ void next_unit(const Work& w, const Plan& p, Piece& x) {
    if (++x.tile == tiles_of(w, p.n[x.b])) {
      x.tile = 0;
      if (++x.h == w.kv.Hkv) {
        x.h = 0;
        do ++x.b; while (p.n[x.b] == 0);     // blocks are left, so there is one
      }
    }
  }
  static __device__ __forceinline__ void take(const Plan& p, Piece& x, unsigned& left) {
    const unsigned room = static_cast<unsigned>(x.blocks - x.kb0);
    const unsigned m = room < left ? room : left, used = m == room ? room + p.extra : m;
    x.kb1 = x.kb0 + static_cast<int>(m);
    left = left > used ? left - used : 0u;
  }
  static __device__ __forceinline__ bool whole(const Piece& x) { return x.kb0 == 0 && x.kb1 == x.blocks; }

  // Chunks do not overlap, so floor(first g / R) + b starts a sequence's tiles clear of the one before.
  static __device__ __forceinline__ unsigned* counter(const Work& w, const Plan& p, const Piece& x) {
    const int tile0 = p.first[x.b] * w.g / w.by_R + x.b;
    return w.counters + (static_cast<size_t>(tile0 + x.tile) * w.kv.Hkv + x.h) * kCounters;
  }
  // Which of CTA c's two slots holds its piece of the unit starting at
  // `start`: the first if the unit began before the CTA's range.
  static __device__ __forceinline__ int slot(const Plan& p, int c, unsigned start) {
    return 2 * c + (p.each || start < range_begin(c, p.per, p.more) ? 0 : 1);
  }
};

// Floats of a slot (R rows of hd outputs, a maximum and a sum) and bytes of the
// counters (for the largest possible number of units).  The slots come first
// and take the same room whatever the call, so that calls of any shapes can
// use one workspace in turn: none leaves its slots where another counts.
constexpr size_t slot_floats(int R, int hd) { return static_cast<size_t>(R) * (hd + 2); }
constexpr size_t kSlotFloatsPerSm = 2 * slot_floats(256, 128);   // the largest: each kernel asserts that its own fit
inline size_t slots_bytes() { return align_up(sm_count() * kSlotFloatsPerSm * sizeof(float), 256); }
inline unsigned* counters_of(void* ws) {
  return reinterpret_cast<unsigned*>(static_cast<unsigned char*>(ws) + slots_bytes());
}
inline size_t counter_bytes(int N, int H, int Hkv, int B, int R) {
  const long long tiles = static_cast<long long>(N) * (H / Hkv) / R + B + 1;
  return align_up(static_cast<size_t>(tiles) * Hkv * kCounters * sizeof(unsigned), 256);
}

}  // namespace paged
}  // namespace medusa
