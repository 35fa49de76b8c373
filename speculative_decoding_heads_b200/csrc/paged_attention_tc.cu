// Attention of new tokens over a paged cache on the tensor cores: bf16 heads
// of 64 or 128, any group of up to 128 query heads.
//
// A unit (paged_work.cuh) is up to two groups of 128 query rows of one
// sequence and key head; the cache streams past it in tiles of 128 keys:
//   S = Q K^T (tcgen05, M 128 x N 128), P = 2^(scale S - m) in registers,
//   O += P V (P read back from tensor memory), l += sum P, m the running
// maximum.  Two softmax warpgroups keep the tensor cores busy in turn.  A
// unit of more than 128 rows gives each warpgroup its own 128 rows and every
// key tile to both, so a tile's 64 KB from L2 serve 256 rows (prompts: bound
// by the tensor cores and the exponentials).  A unit of fewer rows gives the
// key tiles to the warpgroups alternately, each with its own O, m and l
// (tokens and trees: bound by the cache's bytes); the two are joined with
// factors 2^(m_w - m) when they are written, by the first warpgroup while the
// second takes the next unit's first tile.
//
// The maximum is moved (and O rescaled) only when a tile's exceeds it by more
// than 2^8: any reference that keeps the exponents finite gives the same
// quotient.  P is rounded to bf16 for the second product, which costs at most
// half a bf16 step of each probability, as much as rounding the output costs
// it: the error against 64 bits is 0.0023 of the outputs' root mean square,
// 0.0017 of which is the output's rounding.  A pair (high part and remainder,
// as the dense tree attention with its fp32 output needs) takes that away and
// half as many products again: prompts 690 us in place of 520, four 65-node
// trees 160-190 in place of 150, 29 sequences of 16 rows 165 in place of 114;
// with a bf16 output it is not worth that.  Sums, maxima and O are fp32.
//
// Tensor memory (512 columns): S_w at 128 w, its P (two keys per column) over
// the first half of it, O_w at 256 + 128 w.  P V of a step is issued before
// the next Q K^T that overwrites P, and tensor-core operations of one thread
// run in order.
//
// Warp 0 loads (TMA, one box per page; the table's entries of a tile are
// fetched by as many lanes one tile ahead), warp 1 issues the products, warps
// 4-11 are the two softmax warpgroups, a row per thread.  K and V tiles go
// through one ring in the order in which they are used.  Every wait is bounded.
//
// Measured: chunks of 3001 and 4096 tokens of 32 heads (8 key heads) after
// 2048..4095 rows 473 us in short bursts at 1.965 GHz, 1160 TFLOP/s, and 551 us
// in calls without end, which the power cap holds at 1.67 GHz (as many clocks).
// A tile is 1024 clocks of products and about 2300 of softmax latency, so two
// groups leave the tensor cores a third of the time; the exponentials alone are
// not it (without them 2048 tokens after 2048 rows take 109 us, 111 with).
// Four 65-node trees of 52 heads over 8192 rows 150 us in bursts, 5.8 TB/s, and
// 165-176 at the cap's 1.25 GHz.  Halves of 64 keys with double-buffered scores
// (620 us where this took 518), two threads per row (1055) and polynomials for
// a share of the exponentials (526-575) were slower.
#include <cudaTypedefs.h>

#include "paged_work.cuh"
#include "tcgen05.cuh"

namespace medusa {
namespace {

using namespace paged;

constexpr int kBK = 128;                 // keys per tile
constexpr int kGroup = 128;              // rows per softmax warpgroup
constexpr int kThreads = 384;
constexpr uint32_t kTmemCols = 512;
constexpr float kRescaleLog2 = 8.0f;
constexpr float kLog2e = 1.4426950408889634f;

template <int HD>
struct Shape {
  static constexpr int kHalves = HD / 64;
  static constexpr int kHalf = kBK * 128;                 // 128 rows x 64 elements
  static constexpr int kTile = kHalves * kHalf;           // a K, V or Q tile
  static constexpr int kStages = HD == 128 ? 5 : 8;
  static constexpr int kOffRing = 2 * kTile;              // after two Q tiles
  static constexpr int kOffBars = kOffRing + kStages * kTile;
};

struct Bars {
  uint64_t full[8], empty[8];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2], p_half[2], p_full[2], pv_done[2], o_free[2];
  uint64_t drain;
  uint64_t stat_full, stat_free, group[2];   // statistics handed over; the warps of one warpgroup
  uint32_t tmem_base;
  int abort, last[2];
  float m1[kGroup], l1[kGroup];          // alternating units: the second warpgroup's statistics
  Plan plan;
};

template <int HD>
constexpr int smem_bytes() { return Shape<HD>::kOffBars + static_cast<int>(sizeof(Bars)); }
static_assert(smem_bytes<128>() <= 232448, "shared memory budget");
static_assert(smem_bytes<64>() <= 232448, "shared memory budget");
static_assert(2 * slot_floats(2 * kGroup, 128) <= kSlotFloatsPerSm, "two slots per CTA");

struct Params {
  Work w;
  int rows;                // query rows per group: 128 cut to whole tokens
  int q_tokens;            // tokens per Q box
  int box;                 // page rows per TMA box
  float scale_log2;
  uint16_t* out;
};

// A whole warp waits and agrees on the outcome (a wait that runs out in one
// lane ends the role for all of them).
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, Bars* b, const Work& w) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const bool ok = *reinterpret_cast<volatile int*>(&b->abort) == 0 && mbar_wait(bar, parity, w.wait_limit);
  if (__all_sync(0xffffffffu, ok)) return true;
  set_device_status(w.status, MEDUSA_ERR_TIMEOUT, kDetailPagedWait);
  *reinterpret_cast<volatile int*>(&b->abort) = 1;
  return false;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two fp32 operations in one instruction.
typedef unsigned long long F2;
__device__ __forceinline__ F2 pair(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(F2 v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// What every role knows of a piece.
struct Seg {
  int n;             // key tiles of this piece
  int rows;          // query rows of the unit
  bool two;          // both groups have rows: each takes every tile
};

__device__ __forceinline__ Seg segment(const Params& p, const Plan& pl, const Piece& x) {
  Seg s;
  s.n = x.kb1 - x.kb0;
  s.rows = min(p.w.R, pl.n[x.b] * p.w.g - x.tile * p.w.R);
  s.two = s.rows > p.rows;
  return s;
}

using C = Cut<kBK>;

// Groups of 32 keys that a tile with that many keys left has.
__device__ __forceinline__ int tile_chunks(int keys) { return keys >= kBK ? kBK / 32 : (keys + 31) >> 5; }

// ---- loads (warp 0) --------------------------------------------------------

template <int HD>
__device__ void run_loads(const CUtensorMap* q_map, const CUtensorMap* k_map, const CUtensorMap* v_map, const Params& p,
                          unsigned char* smem, Bars* bar, Piece x, unsigned left) {
  using S = Shape<HD>;
  const int lane = threadIdx.x & 31;
  const Plan& pl = bar->plan;
  const int sub = kBK / p.box;                         // boxes per half tile
  const int shift = p.w.kv.page_shift, mask = (1 << shift) - 1;
  const int none = p.w.kv.n_pages * p.w.kv.Hkv;        // past the last page block: reads as zeros
  int e = 0, nq[2] = {0, 0};
  // Table entry of this lane's box of key tile kb.
  auto lookup = [&](int b, int kb, int keys) {
    const int j = kb * kBK + lane * p.box;
    return lane < sub && j < keys ? p.w.kv.table[static_cast<long long>(b) * p.w.kv.max_pages + (j >> shift)] : kNoPage;
  };
  // The block (page, head) of a table entry, when its copy is issued: until then the entry is on its way.
  auto block_of = [&](int page, int h) {
    if (page >= 0 && page < p.w.kv.n_pages) return page * p.w.kv.Hkv + h;
    if (page != kNoPage) set_device_status(p.w.status, MEDUSA_ERR_DEVICE_CHECK, kDetailPagedPage);
    return none;
  };
  auto entry = [&](const CUtensorMap* map, int kb, int block) {
    const int st = e % S::kStages;
    if (e >= S::kStages && !wait(&bar->empty[st], (e / S::kStages - 1) & 1, bar, p.w)) return false;
    unsigned char* d = smem + S::kOffRing + st * S::kTile;
    if (lane == 0) mbar_arrive_expect_tx(&bar->full[st], S::kTile);
    __syncwarp();
    if (lane < sub) {
      const int row = (kb * kBK + lane * p.box) & mask;
#pragma unroll
      for (int hf = 0; hf < S::kHalves; ++hf)
        tc::tma_load_4d(d + hf * S::kHalf + lane * p.box * 128, map, 0, row, hf, block, &bar->full[st]);
    }
    ++e;
    return true;
  };
  auto query = [&](int w, int b, int h, int row0) {
    if (nq[w] > 0 && !wait(&bar->q_empty[w], (nq[w] - 1) & 1, bar, p.w)) return false;
    if (lane == 0) {
      mbar_arrive_expect_tx(&bar->q_full[w], S::kHalves * p.w.g * p.q_tokens * 128);
      for (int hf = 0; hf < S::kHalves; ++hf)
        tc::tma_load_4d(smem + w * S::kTile + hf * S::kHalf, q_map, 0, h * p.w.g, pl.first[b] + row0 / p.w.by_g, hf, &bar->q_full[w]);
    }
    ++nq[w];
    return true;
  };
  for (bool ok = true; ok;) {
    const Seg s = segment(p, pl, x);
    const int keys = C::keys(p.w, pl, x.b, x.tile);
    int cur = lookup(x.b, x.kb0, keys), next = s.n > 1 ? lookup(x.b, x.kb0 + 1, keys) : kNoPage;
    ok = query(0, x.b, x.h, x.tile * p.w.R) && (!s.two || query(1, x.b, x.h, x.tile * p.w.R + p.rows));
    ok = ok && entry(k_map, x.kb0, block_of(cur, x.h));
    if (!s.two && s.n > 1) ok = ok && entry(k_map, x.kb0 + 1, block_of(next, x.h));
    for (int i = 0; ok && i < s.n; ++i) {
      const int after = i + 2 < s.n ? lookup(x.b, x.kb0 + i + 2, keys) : kNoPage;
      ok = entry(v_map, x.kb0 + i, block_of(cur, x.h));
      if (s.two) {
        if (ok && i + 1 < s.n) ok = entry(k_map, x.kb0 + i + 1, block_of(next, x.h));
      } else if (ok && i + 2 < s.n) {
        ok = entry(k_map, x.kb0 + i + 2, block_of(after, x.h));
      }
      cur = next;
      next = after;
    }
    if (!ok || left == 0) break;
    C::next_piece(p.w, pl, x, left);
  }
  // Every copy issued lands before the CTA exits (bounded).
  for (int st = 0; st < S::kStages; ++st)
    if (e > st) mbar_wait(&bar->full[st], ((e - 1 - st) / S::kStages) & 1, p.w.wait_limit);
  for (int w = 0; w < 2; ++w)
    if (nq[w] > 0) mbar_wait(&bar->q_full[w], (nq[w] - 1) & 1, p.w.wait_limit);
}

// ---- products (warp 1) -------------------------------------------------------
// The whole warp waits, so that addresses stay in uniform registers, and the
// elected lane (always the same one) issues: a thread that computed every
// descriptor on its own path took as long to issue a product as to run it.

__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
  return ok != 0;
}

template <int HD>
__device__ void run_products(const Params& p, uint32_t sbase, uint32_t tmem, Bars* bar, Piece x, unsigned left) {
  using S = Shape<HD>;
  constexpr uint32_t idS = tc::idesc_bf16_f32(kGroup, kBK, 0);
  constexpr uint32_t idO = tc::idesc_bf16_f32(kGroup, HD, 1);
  const Plan& pl = bar->plan;
  int st = 0, ph = 0;                        // the next ring entry's stage and parity
  int nq[2] = {0, 0}, np[2] = {0, 0}, piece = 0;
  const uint32_t ring = sbase + S::kOffRing;
  // Descriptors of a tile's first 16 columns (Q, K) or keys (V); the others add to the address field.
  const uint64_t q0 = tc::smem_desc_sw128(sbase, 16, 1024), k0 = tc::smem_desc_sw128(ring, 16, 1024),
                 v0 = tc::smem_desc_sw128(ring, S::kHalf, 1024);
  auto next = [&] {
    if (++st == S::kStages) {
      st = 0;
      ph ^= 1;
    }
  };
  auto landed = [&] { return wait(&bar->full[st], ph, bar, p.w); };
  auto scores = [&](int w, int q, bool release, bool last) {          // S_w = Q_q K^T
    const uint64_t qd = q0 + q * (S::kTile >> 4), kd = k0 + static_cast<uint64_t>(st) * (S::kTile >> 4);
    tc::fence_after_sync();
    if (elect_one()) {
#pragma unroll
      for (int c = 0; c < HD / 16; ++c) {
        const uint32_t off = ((c >> 2) * S::kHalf + (c & 3) * 32) >> 4;
        tc::mma_ss(tmem + 128 * w, qd + off, kd + off, idS, c > 0);
      }
      tc::mma_commit(&bar->s_full[w]);
      if (release) tc::mma_commit(&bar->empty[st]);
      if (last) tc::mma_commit(&bar->q_empty[q]);
    }
    __syncwarp();
  };
  // O_w += P_w V over the tile's first `chunks` groups of 32 keys; the second half of P follows on its own.
  auto values = [&](int w, bool first, int chunks, bool release) {
    const uint64_t vd = v0 + static_cast<uint64_t>(st) * (S::kTile >> 4);
    const uint32_t o = tmem + 256 + 128 * w, ps = tmem + 128 * w;
    if (!landed()) return false;
    if (first && piece > 0 && !wait(&bar->o_free[w], (piece - 1) & 1, bar, p.w)) return false;
    if (!wait(&bar->p_half[w], np[w] & 1, bar, p.w)) return false;
    tc::fence_after_sync();
    if (elect_one()) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c < 2 * chunks) tc::mma_ts(o, ps + c * 8, vd + c * (16 * 128 >> 4), idO, (!first || c > 0) ? 1u : 0u);
    }
    __syncwarp();
    if (!wait(&bar->p_full[w], np[w] & 1, bar, p.w)) return false;
    ++np[w];
    tc::fence_after_sync();
    if (elect_one()) {
#pragma unroll
      for (int c = 4; c < 8; ++c)
        if (c < 2 * chunks) tc::mma_ts(o, ps + c * 8, vd + c * (16 * 128 >> 4), idO, 1u);
      tc::mma_commit(&bar->pv_done[w]);
      if (release) tc::mma_commit(&bar->empty[st]);
    }
    __syncwarp();
    return true;
  };
  for (;;) {
    const Seg s = segment(p, pl, x);
    const int keys = C::keys(p.w, pl, x.b, x.tile);
    if (!wait(&bar->q_full[0], nq[0] & 1, bar, p.w)) return;
    ++nq[0];
    if (s.two) {
      if (!landed()) return;
      scores(0, 0, false, s.n == 1);
      if (!wait(&bar->q_full[1], nq[1] & 1, bar, p.w)) return;
      ++nq[1];
      scores(1, 1, true, s.n == 1);
      next();
      for (int i = 0; i < s.n; ++i) {
        // V_i serves both groups, K_{i+1} behind it in the ring too.
        const bool more = i + 1 < s.n;
        const int vst = st, vph = ph;
        if (!values(0, i == 0, kBK / 32, false)) return;
        if (more) {
          next();
          if (!landed()) return;
          scores(0, 0, false, i + 2 == s.n);
          st = vst;
          ph = vph;
        }
        if (!values(1, i == 0, kBK / 32, true)) return;
        next();
        if (more) {
          scores(1, 1, true, i + 2 == s.n);
          next();
        }
      }
    } else {
      for (int i = 0; i < 2 && i < s.n; ++i) {
        if (!landed()) return;
        scores(1 - i, 0, true, i + 1 == s.n);
        next();
      }
      // No phase of a barrier goes by unseen, where the first warpgroup has no tile either.
      if (s.n == 1 && piece > 0 && !wait(&bar->o_free[0], (piece - 1) & 1, bar, p.w)) return;
      for (int i = 0; i < s.n; ++i) {
        if (!values(1 - (i & 1), i < 2, tile_chunks(keys - (x.kb0 + i) * kBK), true)) return;
        next();
        if (i + 2 < s.n) {
          if (!landed()) return;
          scores(1 - (i & 1), 0, true, i + 3 == s.n);
          next();
        }
      }
    }
    ++piece;
    if (left == 0) return;
    C::next_piece(p.w, pl, x, left);
  }
}

// ---- softmax and output (warps 4-11) ----------------------------------------

// Bits o .. o + 63 (o >= 0) of an ancestor-mask row of four words.
__device__ __forceinline__ uint64_t anc_window(const uint64_t (&a)[4], int o) {
  if (o >= 256) return 0ull;
  const int wi = o >> 6, sh = o & 63;
  const uint64_t w0 = wi == 0 ? a[0] : wi == 1 ? a[1] : wi == 2 ? a[2] : a[3];
  const uint64_t w1 = wi == 0 ? a[1] : wi == 1 ? a[2] : wi == 2 ? a[3] : 0ull;
  return sh == 0 ? w0 : (w0 >> sh) | (w1 << (64 - sh));
}
// Bits of 64 keys starting at key d rows before (d > 0) or after (d <= 0) the
// prefix's end: the prefix, then the row's ancestors and itself.
__device__ __forceinline__ uint64_t tree_bits(const uint64_t (&a)[4], int d) {
  if (d >= 64) return ~0ull;
  return d > 0 ? ((1ull << d) - 1ull) | (a[0] << d) : anc_window(a, -d);
}

// A slot: 256 maxima, 256 sums, then O as [row / 8][column / 4][row % 8] of
// four columns each, which a warp writes (a row per lane) and reads (eight
// lanes per group of columns) in whole 128-byte lines.
template <int HD>
__device__ __forceinline__ float4* slot_out(float* slot, int row, int col4) {
  return reinterpret_cast<float4*>(slot + 4 * kGroup) + ((row >> 3) * (HD / 4) + col4) * 8 + (row & 7);
}

// Joins the pieces that CTAs lo..hi left of a unit's row group (128 threads):
// out = sum_y 2^(m_y - m) O_y / sum_y 2^(m_y - m) l_y.  A thread owns row
// thread % 8 of kRB blocks of eight rows and every 16th group of columns; the
// loads of kPB pieces (from L2) are in flight together.
template <int HD, int kRB, int kPB, typename Put>
__device__ __forceinline__ void join_rows(const Work& w, const Plan& pl, unsigned start, int lo, int hi, int row0, int thread,
                                          int rows, Put put) {
  constexpr int kCols = HD / 64;             // column groups per thread and row
  const int r8 = thread & 7, c4 = thread >> 3;
  for (int rb = 0; rb < rows; rb += 8 * kRB) {
    float m[kRB], l[kRB];
    float4 o[kRB][kCols];
#pragma unroll
    for (int i = 0; i < kRB; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int k = 0; k < kCols; ++k) o[i][k] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll 1
    for (int y0 = lo; y0 <= hi; y0 += kPB) {
      float ms[kRB][kPB], ls[kRB][kPB];
      float4 os[kRB][kPB][kCols];
#pragma unroll
      for (int y = 0; y < kPB; ++y) {
        float* slot = w.slots + static_cast<size_t>(C::slot(pl, y0 + y <= hi ? y0 + y : hi, start)) * slot_floats(2 * kGroup, HD);
#pragma unroll
        for (int i = 0; i < kRB; ++i) {
          const int r = rb + 8 * i + r8, row = row0 + r;
          ms[i][y] = -INFINITY;
          ls[i][y] = 0.f;
#pragma unroll
          for (int k = 0; k < kCols; ++k) os[i][y][k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (y0 + y <= hi && r < rows) {
            ms[i][y] = __ldcg(slot + row);
            ls[i][y] = __ldcg(slot + 2 * kGroup + row);
#pragma unroll
            for (int k = 0; k < kCols; ++k) os[i][y][k] = __ldcg(slot_out<HD>(slot, row, c4 + 16 * k));
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kRB; ++i) {
        float mn = m[i];
#pragma unroll
        for (int y = 0; y < kPB; ++y) mn = fmaxf(mn, ms[i][y]);
        const float ref = mn == -INFINITY ? 0.f : mn, keep = tc::ex2_ftz(m[i] - ref);
        m[i] = mn;
        l[i] *= keep;
#pragma unroll
        for (int k = 0; k < kCols; ++k)
          o[i][k] = make_float4(o[i][k].x * keep, o[i][k].y * keep, o[i][k].z * keep, o[i][k].w * keep);
#pragma unroll
        for (int y = 0; y < kPB; ++y) {
          const float f = tc::ex2_ftz(ms[i][y] - ref);
          l[i] = fmaf(f, ls[i][y], l[i]);
#pragma unroll
          for (int k = 0; k < kCols; ++k) {
            o[i][k].x = fmaf(f, os[i][y][k].x, o[i][k].x);
            o[i][k].y = fmaf(f, os[i][y][k].y, o[i][k].y);
            o[i][k].z = fmaf(f, os[i][y][k].z, o[i][k].z);
            o[i][k].w = fmaf(f, os[i][y][k].w, o[i][k].w);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kRB; ++i) {
      const int r = rb + 8 * i + r8;
      const float inv = 1.f / l[i];
      if (r < rows)
#pragma unroll
        for (int k = 0; k < kCols; ++k)
          put(r, 4 * (c4 + 16 * k), make_uint2(pack2(o[i][k].x * inv, o[i][k].y * inv), pack2(o[i][k].z * inv, o[i][k].w * inv)));
    }
  }
}

template <int HD>
__device__ void run_softmax(const Params& p, unsigned char* smem, uint32_t tmem, Bars* bar, Piece x, unsigned left) {
  using S = Shape<HD>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int w = (warp - 4) >> 2;             // softmax warpgroup
  const int quarter = warp & 3;              // tensor-memory lanes of this warp
  const int row = 32 * quarter + lane;       // row of the group
  const uint32_t lanes = static_cast<uint32_t>(32 * quarter) << 16;
  const uint32_t tS = tmem + lanes + 128 * w;
  const Plan& pl = bar->plan;
  int steps = 0;                             // tiles this warpgroup has taken
  int pv[2] = {0, 0};                        // P V products of both warpgroups before this piece
  int entries = 0;                           // ring entries before this piece
  int syncs = 0;                             // uses of this warpgroup's barrier
  int singles = 0;                           // alternating pieces before this one
  for (;;) {
    const Seg s = segment(p, pl, x);
    const int b = x.b, L = pl.L[b], n = pl.n[b];
    const int grp_row = x.tile * p.w.R + (s.two ? w * p.rows : 0);   // this group's first row
    const int rows = s.two ? (w == 0 ? p.rows : s.rows - p.rows) : s.rows;
    const bool active = 32 * quarter < rows; // a warp without rows only keeps the barriers going
    const int tok = (grp_row + row) / p.w.by_g;
    const int keys = C::keys(p.w, pl, b, x.tile);
    const bool tree = p.w.t.T > 0;
    // Keys below this row's limit are visible (chunks); a tile below every row's limit needs no mask.
    const int limit = L + min(tok, n - 1) + 1;
    const int clear = tree ? L : L + grp_row / p.w.by_g + 1;
    float m = -INFINITY, l = 0.f;
    // One arrival per warp: those of 128 threads on one barrier took 1000 clocks.
    auto arrive = [&](uint64_t* to) {
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(to);
    };
    auto hand_over = [&](uint64_t* to) {
      tc::fence_before_sync();
      arrive(to);
    };
    for (int i = s.two ? 0 : 1 - w; i < s.n; i += s.two ? 1 : 2, ++steps) {
      const int j0 = (x.kb0 + i) * kBK;
      // The keys that this row sees, looked up while S is on its way.
      uint32_t bits[4] = {0u, 0u, 0u, 0u};
      if (j0 + kBK > clear) {
        if (!tree) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int lim = limit - j0 - 32 * c;
            bits[c] = lim >= 32 ? ~0u : lim <= 0 ? 0u : (1u << lim) - 1u;
          }
        } else if (row < rows) {
          uint64_t anc[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) anc[k] = k < p.w.t.W ? p.w.t.anc[tok * p.w.t.W + k] : 0ull;
#pragma unroll
          for (int c = 0; c < 4; ++c) bits[c] = static_cast<uint32_t>(tree_bits(anc, L - j0 - 32 * c));
        }
      }
      if (!wait(&bar->s_full[w], steps & 1, bar, p.w)) return;
      tc::fence_after_sync();
      const bool zero = (w == 0 || !s.two) && x.kb0 + i == x.blocks - 1 && (keys & (p.box - 1)) != 0;
      if (active) {
        float sv[kBK];
#pragma unroll
        for (int c = 0; c < kBK; c += 32) tc::tmem_ld32(tS + c, sv + c);
        tc::tmem_wait_ld();
        if (j0 + kBK > clear) {
#pragma unroll
          for (int k = 0; k < kBK; ++k) sv[k] = (bits[k >> 5] >> (k & 31)) & 1u ? sv[k] : -INFINITY;
        }
        float mx[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
        for (int k = 4; k < kBK; k += 8)
#pragma unroll
          for (int u = 0; u < 4; ++u) mx[u] = fmaxf(mx[u], k + 4 < kBK ? fmaxf(sv[k + u], sv[k + 4 + u]) : sv[k + u]);
        const float tm = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
        float factor = 1.f;
        if (tm > m + kRescaleLog2 || (m == -INFINITY && tm > -INFINITY)) {
          factor = m == -INFINITY ? 0.f : tc::ex2_ftz(m - tm);
          m = tm;
        }
        const float ref = m == -INFINITY ? 0.f : -m;
        // O is rescaled before P is handed over; P V of the step before is done (S was issued after it).
        if (i >= (s.two ? 1 : 2) && __any_sync(0xffffffffu, factor != 1.f)) {
#pragma unroll 1
          for (int c = 0; c < HD; c += 32) {
            float o[32];
            tc::tmem_ld32(tmem + lanes + 256 + 128 * w + c, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] *= factor;
            tc::tmem_st32(tmem + lanes + 256 + 128 * w + c, o);
          }
        }
        const F2 sc = pair(p.scale_log2, p.scale_log2), rf = pair(ref, ref);
        F2 sum[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < kBK / 32; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float a, d;
            unpair(fma2(pair(sv[32 * c + 2 * k], sv[32 * c + 2 * k + 1]), sc, rf), a, d);
            a = tc::ex2_ftz(a);
            d = tc::ex2_ftz(d);
            sum[k & 1] = add2(sum[k & 1], pair(a, d));
            pk[k] = pack2(a, d);
          }
          tc::tmem_st16(tS + 16 * c, pk);
          if (c == 1 && !zero) {             // the first half of P V can start
            tc::tmem_wait_st();
            hand_over(&bar->p_half[w]);
          }
        }
        float s0, s1;
        unpair(add2(sum[0], sum[1]), s0, s1);
        l = l * factor + (s0 + s1);
        tc::tmem_wait_st();
      }
      if (zero) {
        // Rows of the last page past the sequence may hold anything: zero
        // their values, so that 0 * (stale value) stays 0.
        const int v = entries + 2 * s.n - 1;            // a piece's last ring entry
        if (!wait(&bar->full[v % S::kStages], (v / S::kStages) & 1, bar, p.w)) return;
        const int r0 = keys - j0, r1 = (r0 + p.box - 1) & ~(p.box - 1);
        unsigned char* d = smem + S::kOffRing + (v % S::kStages) * S::kTile + r0 * 128;
        for (int c = row; c < (r1 - r0) * 8; c += kGroup)
#pragma unroll
          for (int hf = 0; hf < S::kHalves; ++hf) *reinterpret_cast<uint4*>(d + hf * S::kHalf + c * 16) = make_uint4(0, 0, 0, 0);
        tc::fence_proxy_async_smem();
      }
      if (zero || !active) hand_over(&bar->p_half[w]);
      hand_over(&bar->p_full[w]);
    }

    // Output, a row per thread.  Where the tiles alternated, the second
    // warpgroup hands over its statistics and the first joins and writes both.
    const int n0 = s.two ? s.n : s.n / 2, n1 = s.two ? s.n : (s.n + 1) / 2;
    entries += 2 * s.n;
    bool second = false;                       // both O_0 and O_1 belong to this thread's row
    float f0 = 1.f, f1 = 0.f;
    if (!s.two) {
      if (w == 1) {
        // the first warpgroup has read the last hand-over
        if (singles > 0 && !wait(&bar->stat_free, (singles - 1) & 1, bar, p.w)) return;
        bar->m1[row] = m;
        bar->l1[row] = l;
        arrive(&bar->stat_full);
      } else {
        if (!wait(&bar->stat_full, singles & 1, bar, p.w)) return;
        const float m1 = bar->m1[row], l1 = bar->l1[row], mm = fmaxf(m, m1);
        arrive(&bar->stat_free);
        f0 = m == -INFINITY ? 0.f : tc::ex2_ftz(m - mm);
        f1 = m1 == -INFINITY ? 0.f : tc::ex2_ftz(m1 - mm);
        m = mm;
        l = f0 * l + f1 * l1;
        second = n0 > 0;
      }
      ++singles;
    }
    if (s.two || w == 0) {
      const int own = s.two ? w : 1;           // the first tile of an alternating unit is the second warpgroup's
      if (second && !wait(&bar->pv_done[0], (pv[0] + n0 - 1) & 1, bar, p.w)) return;
      if (!wait(&bar->pv_done[own], (pv[own] + (own == 0 ? n0 : n1) - 1) & 1, bar, p.w)) return;
      tc::fence_after_sync();
      const bool whole = C::whole(x);
      const int slot_row = (s.two ? w * kGroup : 0) + row;           // rows of a slot: 2 * kGroup
      float* slot = p.w.slots + C::slot(pl, blockIdx.x, x.start) * slot_floats(2 * kGroup, HD);
      uint16_t* dst = p.out + (static_cast<size_t>(pl.first[b] + tok) * p.w.H + x.h * p.w.g + (grp_row + row - tok * p.w.g)) * HD;
      const float inv = 1.f / l;
      // Columns c .. c + 3 of row r of the group.
      auto put = [&](int r, int c, uint2 v) {
        const int t = (grp_row + r) / p.w.by_g;
        *reinterpret_cast<uint2*>(p.out + (static_cast<size_t>(pl.first[b] + t) * p.w.H + x.h * p.w.g + (grp_row + r - t * p.w.g)) * HD + c) = v;
      };
      if (active) {
#pragma unroll 1
        for (int c = 0; c < HD; c += 32) {
          float o[32];
          tc::tmem_ld32(tmem + lanes + 256 + 128 * own + c, o);
          if (second) {
            float o0[32];
            tc::tmem_ld32(tmem + lanes + 256 + c, o0);
            tc::tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = fmaf(o0[k], f0, o[k] * f1);
          } else {
            tc::tmem_wait_ld();
          }
          if (whole) {
            if (row < rows)
#pragma unroll
              for (int k = 0; k < 32; k += 8)
                *reinterpret_cast<uint4*>(dst + c + k) =
                    make_uint4(pack2(o[k] * inv, o[k + 1] * inv), pack2(o[k + 2] * inv, o[k + 3] * inv),
                               pack2(o[k + 4] * inv, o[k + 5] * inv), pack2(o[k + 6] * inv, o[k + 7] * inv));
          } else {
            float4* d = slot_out<HD>(slot, slot_row, c / 4);
#pragma unroll
            for (int k = 0; k < 8; ++k) __stcg(d + 8 * k, make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]));
          }
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(&bar->o_free[w]);
        if (!s.two) tc::mbar_arrive(&bar->o_free[1]);
      }
      if (!whole) {
        if (active) {
          __stcg(slot + slot_row, m);
          __stcg(slot + 2 * kGroup + slot_row, l);
        }
        arrive(&bar->group[w]);                // then one thread's release covers all of them
        if (!wait(&bar->group[w], syncs++ & 1, bar, p.w)) return;
        int lo, hi;
        C::owners(pl, x, lo, hi);
        if (row == 0) {
          unsigned* ctr = C::counter(p.w, pl, x) + w;
          bar->last[w] = atom_add_acq_rel_gpu(ctr, 1u) == static_cast<unsigned>(hi - lo);
          if (bar->last[w]) *ctr = 0u;
        }
        arrive(&bar->group[w]);
        if (!wait(&bar->group[w], syncs++ & 1, bar, p.w)) return;
        if (bar->last[w]) {
          const int row0 = s.two ? w * kGroup : 0;
          // Few rows or many pieces: more pieces at a time; else more rows (100 tokens of 16 heads after 9000 rows
          // 33.0 us, always more rows 35.2; 500 of 8 heads on one after 3000 28.7, always more pieces 30.3).
          if (rows <= 16 || hi - lo >= 6) join_rows<HD, 2, 4>(p.w, pl, x.start, lo, hi, row0, row, rows, put);
          else join_rows<HD, 4, 2>(p.w, pl, x.start, lo, hi, row0, row, rows, put);
        }
      }
    }
    pv[0] += n0;
    pv[1] += n1;
    if (left == 0) return;
    C::next_piece(p.w, pl, x, left);
  }
}

template <int HD>
__global__ void __launch_bounds__(kThreads, 1)
    paged_attn_tc(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                  const __grid_constant__ CUtensorMap v_map, const Params p) {
  using S = Shape<HD>;
  extern __shared__ __align__(1024) unsigned char smem[];
  if ((smem_u32(smem) & 1023u) != 0u) {      // the swizzle pattern needs it; no static shared memory precedes it
    if (threadIdx.x == 0) set_device_status(p.w.status, MEDUSA_ERR_DEVICE_CHECK, kDetailPagedShared);
    return;
  }
  Bars* bar = reinterpret_cast<Bars*>(smem + S::kOffBars);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // Registers: launched with 168 a thread; the softmax warpgroups take what the others give up
  // (128 * 104 + 256 * 200 = 384 * 168).  A warpgroup's threads all execute the same setmaxnreg, which
  // the instruction demands: the branch that holds it is a warpgroup's, and roles part behind it.
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == 0) {
      if (lane == 0) {
        for (int st = 0; st < S::kStages; ++st) {
          mbar_init(&bar->full[st], 1);
          mbar_init(&bar->empty[st], 1);
        }
        for (int w = 0; w < 2; ++w) {
          mbar_init(&bar->q_full[w], 1);
          mbar_init(&bar->q_empty[w], 1);
          mbar_init(&bar->s_full[w], 1);
          mbar_init(&bar->p_half[w], 4 + p.w.wait_extra);
          mbar_init(&bar->p_full[w], 4);
          mbar_init(&bar->pv_done[w], 1);
          mbar_init(&bar->o_free[w], 4);
          mbar_init(&bar->group[w], 4);
        }
        mbar_init(&bar->drain, 1);
        mbar_init(&bar->stat_full, 4);
        mbar_init(&bar->stat_free, 4);
        bar->abort = 0;
        fence_barrier_init();
      }
      __syncwarp();
      C::plan(p.w, bar->plan);
      __syncwarp();
      // The loads need nothing of the other warps: they start here.
      __threadfence_block();
      asm volatile("barrier.cta.arrive 1, 384;" ::: "memory");
      if (bar->plan.begin < bar->plan.end) {
        unsigned left;
        const Piece x = C::first_piece(p.w, bar->plan, left);
        run_loads<HD>(&q_map, &k_map, &v_map, p, smem, bar, x, left);
      }
    } else {
      if (warp == 1) {
        tc::tmem_alloc(&bar->tmem_base, kTmemCols);
        tc::tmem_relinquish();
      } else if (tid == 64) {
        tc::prefetch_tensormap(&q_map);
        tc::prefetch_tensormap(&k_map);
        tc::prefetch_tensormap(&v_map);
      }
      tc::fence_before_sync();
      asm volatile("barrier.cta.sync 1, 384;" ::: "memory");
      tc::fence_after_sync();
      if (warp == 1 && bar->plan.begin < bar->plan.end) {
        unsigned left;
        const Piece x = C::first_piece(p.w, bar->plan, left);
        run_products<HD>(p, smem_u32(smem), bar->tmem_base, bar, x, left);
        // However it ended: products in flight end before their operands and tensor memory go (bounded).
        if (elect_one()) tc::mma_commit(&bar->drain);
        __syncwarp();
        mbar_wait(&bar->drain, 0, p.w.wait_limit);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    asm volatile("barrier.cta.sync 1, 384;" ::: "memory");
    tc::fence_after_sync();
    if (bar->plan.begin < bar->plan.end) {
      unsigned left;
      const Piece x = C::first_piece(p.w, bar->plan, left);
      run_softmax<HD>(p, smem, bar->tmem_base, bar, x, left);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(bar->tmem_base, kTmemCols);
  }
}

// Two groups to a unit read the keys once for both, but where that leaves fewer
// units than SMs every unit is cut into pieces, and the SM that joins them
// reads them all (32 bytes a clock): with one group there are twice as many
// joins of half the size.  One group against two: two 64-node trees of 32 heads
// over 2000 rows 23.8 us, 31.9; 100 tokens of 16 heads after 9000 rows 42.4,
// 57.6; 256 and 1024 of 32 heads after 4000 rows 37.6 and 84, 45.2 and 86.
int rows_per_unit(int N, int H, int rows) {
  return static_cast<long long>(N) * H < 2ll * rows * sm_count() ? rows : 2 * rows;
}

template <int HD>
medusa_status_t launch(const PagedDev& kv, int N, int H, const void* q, float scale, const TreeDev* tree,
                       const int32_t* starts, void* out, void* ws, cudaStream_t stream) {
  using S = Shape<HD>;
  auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
  if (!enc) return fail(MEDUSA_ERR_UNSUPPORTED, "medusa_paged_attention: cuTensorMapEncodeTiled unavailable");
  Params p{};
  p.w.kv = kv;
  if (tree) p.w.t = *tree;
  p.w.N = N;
  p.w.H = H;
  p.w.g = H / kv.Hkv;
  p.w.starts = starts;
  p.w.status = device_status_ptr();
  p.w.wait_limit = paged_wait().limit_ns;
  p.w.wait_extra = paged_wait().extra;
  const int tokens = kGroup / p.w.g;
  p.rows = tokens * p.w.g;
  p.w.R = rows_per_unit(N, H, p.rows);
  p.w.by_g = Divisor(p.w.g);
  p.w.by_R = Divisor(p.w.R);
  p.w.by_hk = Divisor(kv.Hkv);
  p.w.join = 1.5f;         // a 64-node tree of 8 heads on one over 2000 rows 22.0 us (0: 40, 6: 23.0), 500 such tokens after 3000 28.7 (28.9, 34.5)
  p.w.extra = 3u;          // 6000 clocks between units, 1900 a block: 26 prompts of 75..865 tokens 83 us (0: 90, 6: 89)
  const int most = starts ? N : N / kv.B;                // tokens of one sequence
  p.q_tokens = tokens < most ? tokens : most;
  const int page = 1 << kv.page_shift;
  p.box = page < kBK ? page : kBK;
  p.scale_log2 = scale * kLog2e;
  p.out = static_cast<uint16_t*>(out);
  p.w.slots = static_cast<float*>(ws);
  p.w.counters = counters_of(ws);
  const cuuint32_t es[4] = {1, 1, 1, 1};
  CUtensorMap qm, km, vm;
  {
    const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(N), S::kHalves};
    const cuuint64_t strides[3] = {HD * 2, static_cast<cuuint64_t>(H) * HD * 2, 128};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(p.w.g), static_cast<cuuint32_t>(p.q_tokens), 1};
    if (enc(&qm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(q), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return fail(MEDUSA_ERR_UNSUPPORTED, "medusa_paged_attention: q tensor map rejected");
  }
  for (int which = 0; which < 2; ++which) {
    const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(page), S::kHalves, static_cast<cuuint64_t>(kv.n_pages) * kv.Hkv};
    const cuuint64_t strides[3] = {HD * 2, 128, static_cast<cuuint64_t>(page) * HD * 2};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(p.box), 1, 1};
    if (enc(which ? &vm : &km, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, which ? kv.v : kv.k, dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return fail(MEDUSA_ERR_UNSUPPORTED, "medusa_paged_attention: page tensor map rejected");
  }
  cudaError_t e = cudaFuncSetAttribute(paged_attn_tc<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<HD>());
  if (e == cudaSuccess)
    e = launch_kernel(paged_attn_tc<HD>, dim3(sm_count()), dim3(kThreads), smem_bytes<HD>(), stream, false, qm, km, vm, p);
  return e == cudaSuccess ? MEDUSA_OK : cuda_fail("medusa_paged_attention: tcgen05 launch", e);
}

}  // namespace

bool paged_attention_tc_supported(const PagedDev& kv, medusa_dtype_t dtype, int H) {
  return dtype == MEDUSA_BF16 && (kv.hd == 64 || kv.hd == 128) && H / kv.Hkv <= kGroup &&
         static_cast<long long>(kv.n_pages) * kv.Hkv < 0x7fffffffll;
}

size_t paged_attention_tc_workspace_bytes(const PagedDev& kv, int N, int H) {
  const int g = H / kv.Hkv;
  return slots_bytes() + counter_bytes(N, H, kv.Hkv, kv.B, rows_per_unit(N, H, kGroup / g * g));
}

medusa_status_t launch_paged_attention_tc(const PagedDev& kv, int N, int H, const void* q, float scale, const TreeDev* tree,
                                          const int32_t* starts, void* out, void* ws, cudaStream_t stream) {
  return kv.hd == 128 ? launch<128>(kv, N, H, q, scale, tree, starts, out, ws, stream)
                      : launch<64>(kv, N, H, q, scale, tree, starts, out, ws, stream);
}

}  // namespace medusa
