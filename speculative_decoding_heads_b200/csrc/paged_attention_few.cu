// Attention over a paged cache for few query rows per key head (at most 16:
// single tokens, small trees), bf16 heads of 64 or 128.
//
// Bound by the cache's bytes: 128 keys and values of a head are 64 KB, which
// an SM's share of HBM takes 2800 clocks to deliver, and a 128-row tensor
// product would leave three of its four softmax warps without a row.
// Here eight warps take 16 keys each of every tile, with their own maximum, sum
// and output (mma.sync m16n8k16, operands by ldmatrix), so the softmax is
// spread over all of them whatever the number of rows, and no warp waits for
// another before the end of a piece.  Then the eight are joined through shared
// memory, and the pieces of a unit (paged_work.cuh) through the slots.
//
// P enters the second product as a bf16 pair (high part and remainder), whose
// second multiplication is free here: the output is rounded once, to bf16.
// The maximum is moved only when it grows by more than 2^8, as in
// paged_attention_tc.cu.
//
// Measured: 13 tokens of 40 heads in groups of 5 over 4099..60001 rows 255 us,
// 6.7 TB/s; one token of 32 heads over 1024 rows in pages of 16 10.9 us, all
// of it latency (plan, page ids, three tiles of eight copies each, join).
#include <cudaTypedefs.h>

#include "paged_work.cuh"
#include "tcgen05.cuh"

namespace medusa {
namespace {

using namespace paged;

constexpr int kBK = 128;                 // keys per tile
constexpr int kWarps = 8;                // computing warps, 16 keys of a tile each
constexpr int kThreads = 32 * (kWarps + 1);   // and a loading warp
constexpr float kRescaleLog2 = 8.0f;
constexpr float kLog2e = 1.4426950408889634f;

using C = Cut<kBK>;

template <int HD>
struct Shape {
  static constexpr int kRows = 16;
  static constexpr int kHalves = HD / 64;
  static constexpr int kHalf = kBK * 128;                 // 128 keys x 64 elements
  static constexpr int kTile = kHalves * kHalf;           // a K or V tile
  static constexpr int kStages = 5 * (128 / HD);
  static constexpr int kPitch = HD + 8;                   // floats per joined row: conflict-free pairs
  static constexpr int kOffJoin = kStages * kTile;        // four warps' outputs
  static constexpr int kOffBars = kOffJoin + 4 * kRows * kPitch * 4;
};

struct Bars {
  uint64_t full[10], empty[10], group;
  int abort, last;
  float m[kWarps][16], l[kWarps][16];
  Plan plan;
};

template <int HD>
constexpr int smem_bytes() { return Shape<HD>::kOffBars + static_cast<int>(sizeof(Bars)); }
static_assert(smem_bytes<128>() <= 232448 && smem_bytes<64>() <= 232448, "shared memory budget");
static_assert(2 * slot_floats(16, 128) <= kSlotFloatsPerSm, "two slots per CTA");

struct Params {
  Work w;
  int box;                 // page rows per TMA box
  const uint16_t* q;
  float scale_log2;
  uint16_t* out;
};

// A whole warp waits and agrees on the outcome.
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
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// ---- loads (the last warp) ---------------------------------------------------

template <int HD>
__device__ void run_loads(const CUtensorMap* k_map, const CUtensorMap* v_map, const Params& p, unsigned char* smem, Bars* bar,
                          Piece x, unsigned left) {
  using S = Shape<HD>;
  const int lane = threadIdx.x & 31;
  const Plan& pl = bar->plan;
  const int sub = kBK / p.box;                         // boxes per half tile
  const int shift = p.w.kv.page_shift, mask = (1 << shift) - 1;
  const int none = p.w.kv.n_pages * p.w.kv.Hkv;        // past the last page block: reads as zeros
  int e = 0;
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
    unsigned char* d = smem + st * S::kTile;
    if (lane == 0) mbar_arrive_expect_tx(&bar->full[st], S::kTile);
    __syncwarp();
    if (lane < sub) {
      const int row = (kb * kBK + lane * p.box) & mask;
      tc::tma_load_4d(d + lane * p.box * 128 * S::kHalves, map, 0, row, 0, block, &bar->full[st]);
    }
    ++e;
    return true;
  };
  for (bool ok = true; ok;) {
    const int keys = C::keys(p.w, pl, x.b, x.tile);
    int cur = lookup(x.b, x.kb0, keys);
    for (int kb = x.kb0; ok && kb < x.kb1; ++kb) {
      const int next = kb + 1 < x.kb1 ? lookup(x.b, kb + 1, keys) : kNoPage;
      const int block = block_of(cur, x.h);
      ok = entry(k_map, kb, block) && entry(v_map, kb, block);
      cur = next;
    }
    if (!ok || left == 0) break;
    C::next_piece(p.w, pl, x, left);
  }
  // Every copy issued lands before the CTA exits (bounded).
  for (int st = 0; st < S::kStages; ++st)
    if (e > st) mbar_wait(&bar->full[st], ((e - 1 - st) / S::kStages) & 1, p.w.wait_limit);
}

// ---- the eight computing warps ------------------------------------------------

// A slot: kRows maxima, kRows sums, kRows outputs.
template <int HD>
__device__ void run_rows(const Params& p, unsigned char* smem, Bars* bar, Piece x, unsigned left) {
  using S = Shape<HD>;
  constexpr int kN = HD / 8, kC4 = HD / 4;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gr = lane >> 2, qc = lane & 3;
  const Plan& pl = bar->plan;
  const int g = p.w.g;
  const uint32_t ring = smem_u32(smem);
  float* join = reinterpret_cast<float*>(smem + S::kOffJoin);
  int st = 0, ph = 0, syncs = 0;
  auto next = [&] {
    if (++st == S::kStages) {
      st = 0;
      ph ^= 1;
    }
  };
  auto all = [&] {                                     // the computing warps
    __syncwarp();
    if (lane == 0) mbar_arrive_cta(&bar->group);
    return wait(&bar->group, syncs++ & 1, bar, p.w);
  };
  // ldmatrix rows: K (keys x dimensions) and V (transposed) of this warp's 16 keys.
  const int k_key = 16 * warp + (lane >> 4) * 8 + (lane & 7), k_ch = (lane >> 3) & 1;
  const int v_key = 16 * warp + ((lane >> 3) & 1) * 8 + (lane & 7), v_ch = lane >> 4;
  // A tile is its boxes one after the other, each [halves][rows][64] in the 128-byte swizzle.
  const int box = p.box;
  auto key_at = [&](int key) { return (key & ~(box - 1)) * 128 * S::kHalves + (key & (box - 1)) * 128; };
  const int k_at = key_at(k_key), v_at = key_at(v_key);
  auto at = [&](uint32_t tile, int off, int key, int chunk) {   // 16-byte chunk of a row
    return tile + (chunk >> 3) * box * 128 + off + (((chunk & 7) ^ (key & 7)) << 4);
  };
  for (;;) {
    const int b = x.b, L = pl.L[b], n = pl.n[b], first = pl.first[b];
    const int row0 = x.tile * S::kRows, rows = min(S::kRows, n * g - row0);
    const int keys = C::keys(p.w, pl, b, x.tile);
    const bool tree = p.w.t.T > 0;
    const int clear = tree ? L : L + row0 / p.w.by_g + 1;     // below every row's limit
    int tok[2];                                    // tokens of this thread's rows
    uint32_t sees[2];                              // and the tree's nodes that they see (T <= 16 here)
    uint32_t qa[HD / 16][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 8 * i + gr, rr = row0 + r;
      tok[i] = rr / p.w.by_g;
      sees[i] = tree && r < rows ? static_cast<uint32_t>(p.w.t.anc[tok[i]]) : 0u;
      const uint16_t* src = p.q + (static_cast<size_t>(first + tok[i]) * p.w.H + x.h * g + rr - tok[i] * g) * HD + 2 * qc;
#pragma unroll
      for (int c = 0; c < HD / 16; ++c) {
        qa[c][i] = r < rows ? *reinterpret_cast<const uint32_t*>(src + 16 * c) : 0u;
        qa[c][2 + i] = r < rows ? *reinterpret_cast<const uint32_t*>(src + 16 * c + 8) : 0u;
      }
    }
    float m[2], l[2], o[kN][4];
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int c = 0; c < kN; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[c][e] = 0.f;
    for (int kb = x.kb0; kb < x.kb1; ++kb) {
      const int j0 = kb * kBK, mine = keys - j0 - 16 * warp;    // keys of this warp's 16
      if (!wait(&bar->full[st], ph, bar, p.w)) return;
      const uint32_t kt = ring + st * S::kTile;
      float s[2][4];
      if (mine > 0) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[u][e] = 0.f;
#pragma unroll
        for (int c = 0; c < HD / 16; ++c) {
          uint32_t kf[4];
          ldmatrix4(kf, at(kt, k_at, k_key, 2 * c + k_ch));
          mma(s[0], qa[c], kf[0], kf[1]);
          mma(s[1], qa[c], kf[2], kf[3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive_cta(&bar->empty[st]);
      next();
      uint32_t ph_[4], pl_[4];                         // P and its remainder as the second product's operand
      if (mine > 0) {
        const bool masked = j0 + kBK > clear;
        float f[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (masked) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int j = j0 + 16 * warp + 8 * u + 2 * qc + e, rel = j - L, tk = tok[i];
                bool see;
                if (tree)
                  see = rel < 0 || (rel < n && (sees[i] >> rel & 1u));
                else
                  see = rel <= tk && rel < n;
                if (!see) s[u][2 * i + e] = -INFINITY;
              }
          }
          float mx = fmaxf(fmaxf(s[0][2 * i], s[0][2 * i + 1]), fmaxf(s[1][2 * i], s[1][2 * i + 1]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) * p.scale_log2;
          f[i] = 1.f;
          if (mx > m[i] + kRescaleLog2 || (m[i] == -INFINITY && mx > -INFINITY)) {
            f[i] = m[i] == -INFINITY ? 0.f : tc::ex2_ftz(m[i] - mx);
            m[i] = mx;
          }
          const float ref = m[i] == -INFINITY ? 0.f : -m[i];
          float sum = 0.f;
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float v = tc::ex2_ftz(fmaf(s[u][2 * i + e], p.scale_log2, ref));
              s[u][2 * i + e] = v;
              sum += v;
            }
          l[i] = l[i] * f[i] + sum;            // this thread's keys; the row's four threads are summed at the end
        }
        if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f))
#pragma unroll
          for (int c = 0; c < kN; ++c) {
            o[c][0] *= f[0];
            o[c][1] *= f[0];
            o[c][2] *= f[1];
            o[c][3] *= f[1];
          }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float a = s[u][2 * i], d = s[u][2 * i + 1];
            const uint32_t h = pack2(a, d);
            ph_[2 * u + i] = h;
            pl_[2 * u + i] = pack2(a - bf16lo(h), d - bf16hi(h));
          }
      }
      if (!wait(&bar->full[st], ph, bar, p.w)) return;
      const uint32_t vt = ring + st * S::kTile;
      if (mine > 0) {
        const bool stale = mine < 16;                  // rows past the sequence may hold anything: 0 * value must stay 0
        if (stale) {
          for (int i = lane; i < (16 - mine) * 8 * S::kHalves; i += 32) {
            const int r = i / (8 * S::kHalves), c = i - r * 8 * S::kHalves;
            *reinterpret_cast<uint4*>(smem + st * S::kTile + key_at(16 * warp + mine + r) + (c >> 3) * box * 128 + (c & 7) * 16) =
                make_uint4(0, 0, 0, 0);
          }
          __syncwarp();
        }
#pragma unroll
        for (int c = 0; c < kN / 2; ++c) {
          uint32_t vf[4];
          ldmatrix4t(vf, at(vt, v_at, v_key, 2 * c + v_ch));
          mma(o[2 * c], ph_, vf[0], vf[1]);
          mma(o[2 * c + 1], ph_, vf[2], vf[3]);
          mma(o[2 * c], pl_, vf[0], vf[1]);
          mma(o[2 * c + 1], pl_, vf[2], vf[3]);
        }
        if (stale) tc::fence_proxy_async_smem();       // before the next copy into this stage
      }
      __syncwarp();
      if (lane == 0) mbar_arrive_cta(&bar->empty[st]);
      next();
    }

    // Joins the eight warps: statistics, then the outputs scaled to the common
    // maximum, first warps 4-7 into 0-3, then those four.
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      if (qc == 0) {
        bar->m[warp][8 * i + gr] = m[i];
        bar->l[warp][8 * i + gr] = l[i];
      }
    }
    if (!all()) return;
    float f[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float mm = -INFINITY;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) mm = fmaxf(mm, bar->m[k][8 * i + gr]);
      f[i] = m[i] == -INFINITY ? 0.f : tc::ex2_ftz(m[i] - mm);
    }
    float* own = join + (warp & 3) * S::kRows * S::kPitch + 2 * qc;
    auto put = [&] {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 8 * i + gr;
        if (r < rows)
#pragma unroll
          for (int c = 0; c < kN; ++c)
            *reinterpret_cast<float2*>(own + r * S::kPitch + 8 * c) = make_float2(o[c][2 * i], o[c][2 * i + 1]);
      }
    };
#pragma unroll
    for (int c = 0; c < kN; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[c][e] *= f[e >> 1];
    if (warp >= 4) put();
    if (!all()) return;
    if (warp < 4) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 8 * i + gr;
        if (r < rows)
#pragma unroll
          for (int c = 0; c < kN; ++c) {
            const float2 v = *reinterpret_cast<const float2*>(own + r * S::kPitch + 8 * c);
            o[c][2 * i] += v.x;
            o[c][2 * i + 1] += v.y;
          }
      }
      put();                                           // the same addresses, by the thread that read them
    }
    if (!all()) return;
    const bool whole = C::whole(x);
    float* slot = p.w.slots + C::slot(pl, blockIdx.x, x.start) * slot_floats(S::kRows, HD);
    auto place = [&](int r) {
      const int t = (row0 + r) / p.w.by_g;
      return p.out + (static_cast<size_t>(first + t) * p.w.H + x.h * g + row0 + r - t * g) * HD;
    };
    for (int i = tid; i < rows * kC4; i += 32 * kWarps) {
      const int r = i / kC4, c = 4 * (i - r * kC4);
      float mm = -INFINITY, ll = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) mm = fmaxf(mm, bar->m[k][r]);
      const float ref = mm == -INFINITY ? 0.f : mm;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) ll = fmaf(tc::ex2_ftz(bar->m[k][r] - ref), bar->l[k][r], ll);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 w = *reinterpret_cast<const float4*>(join + (k * S::kRows + r) * S::kPitch + c);
        v.x += w.x;
        v.y += w.y;
        v.z += w.z;
        v.w += w.w;
      }
      if (whole) {
        const float inv = 1.f / ll;
        *reinterpret_cast<uint2*>(place(r) + c) = make_uint2(pack2(v.x * inv, v.y * inv), pack2(v.z * inv, v.w * inv));
      } else {
        __stcg(reinterpret_cast<float4*>(slot + 2 * S::kRows + r * HD + c), v);
        if (c == 0) {
          __stcg(slot + r, mm);
          __stcg(slot + S::kRows + r, ll);
        }
      }
    }
    if (!whole) {
      if (!all()) return;                              // then one thread's release covers all of them
      int lo, hi;
      C::owners(pl, x, lo, hi);
      if (tid == 0) {
        unsigned* ctr = C::counter(p.w, pl, x);
        bar->last = atom_add_acq_rel_gpu(ctr, 1u) == static_cast<unsigned>(hi - lo);
        if (bar->last) *ctr = 0u;
      }
      if (!all()) return;
      if (bar->last) {
        // The last piece joins them all in range order: `teams` of threads (one
        // for up to four pieces) take every teams-th piece each, four at a
        // time, and are joined in order.
        const int items = rows * kC4, most = items >= 256 ? 1 : 256 / items, want = (hi - lo + 4) / 4;
        const int teams = want < most ? want : most;
        for (int i0 = 0; i0 < items; i0 += 256) {
          const int team = teams > 1 ? tid / items : 0, i = i0 + (teams > 1 ? tid - team * items : tid);
          const int r = i / kC4, c = 4 * (i - r * kC4);
          float mm = -INFINITY, ll = 0.f;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          auto add = [&](float m1, float l1, float4 o1) {
            const float mn = fmaxf(mm, m1), ref = mn == -INFINITY ? 0.f : mn;
            const float a = tc::ex2_ftz(mm - ref), d = tc::ex2_ftz(m1 - ref);
            mm = mn;
            ll = a * ll + d * l1;
            v = make_float4(a * v.x + d * o1.x, a * v.y + d * o1.y, a * v.z + d * o1.z, a * v.w + d * o1.w);
          };
          const bool busy = team < teams && i < items;
          if (busy)
            for (int y = lo + team; y <= hi; y += 4 * teams) {
              float m4[4], l4[4];
              float4 o4[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                m4[k] = -INFINITY;
                l4[k] = 0.f;
                o4[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (y + k * teams <= hi) {
                  const float* sl = p.w.slots + C::slot(pl, y + k * teams, x.start) * slot_floats(S::kRows, HD);
                  m4[k] = __ldcg(sl + r);
                  l4[k] = __ldcg(sl + S::kRows + r);
                  o4[k] = __ldcg(reinterpret_cast<const float4*>(sl + 2 * S::kRows + r * HD + c));
                }
              }
#pragma unroll
              for (int k = 0; k < 4; ++k) add(m4[k], l4[k], o4[k]);
            }
          if (teams > 1) {
            float* mine = join + tid * 8;              // m, l, four outputs
            if (busy) {
              mine[0] = mm;
              mine[1] = ll;
              *reinterpret_cast<float4*>(mine + 4) = v;
            }
            if (!all()) return;
            if (team == 0 && busy)
              for (int k = 1; k < teams; ++k) {
                const float* other = join + (k * items + i) * 8;
                add(other[0], other[1], *reinterpret_cast<const float4*>(other + 4));
              }
          }
          if (team == 0 && busy) {
            const float inv = 1.f / ll;
            *reinterpret_cast<uint2*>(place(r) + c) = make_uint2(pack2(v.x * inv, v.y * inv), pack2(v.z * inv, v.w * inv));
          }
        }
      }
    }
    if (left == 0) return;
    C::next_piece(p.w, pl, x, left);
    if (!all()) return;                                // the join buffer and the statistics have been read
  }
}

template <int HD>
__global__ void __launch_bounds__(kThreads, 1)
    paged_attn_few(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map, const Params p) {
  using S = Shape<HD>;
  extern __shared__ __align__(1024) unsigned char smem[];
  if ((smem_u32(smem) & 1023u) != 0u) {      // the swizzle pattern needs it; no static shared memory precedes it
    if (threadIdx.x == 0) set_device_status(p.w.status, MEDUSA_ERR_DEVICE_CHECK, kDetailPagedShared);
    return;
  }
  Bars* bar = reinterpret_cast<Bars*>(smem + S::kOffBars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == kWarps) {
    if (lane == 0) {
      for (int st = 0; st < S::kStages; ++st) {
        mbar_init(&bar->full[st], 1);
        mbar_init(&bar->empty[st], kWarps);
      }
      mbar_init(&bar->group, kWarps + p.w.wait_extra);
      bar->abort = 0;
      fence_barrier_init();
    }
    __syncwarp();
    C::plan(p.w, bar->plan);
    __syncwarp();
    __threadfence_block();
    asm volatile("barrier.cta.arrive 1, 288;" ::: "memory");   // the loads need nothing of the other warps
    if (bar->plan.begin < bar->plan.end) {
      unsigned left;
      const Piece x = C::first_piece(p.w, bar->plan, left);
      run_loads<HD>(&k_map, &v_map, p, smem, bar, x, left);
    }
  } else {
    if (threadIdx.x == 0) {
      tc::prefetch_tensormap(&k_map);
      tc::prefetch_tensormap(&v_map);
    }
    asm volatile("barrier.cta.sync 1, 288;" ::: "memory");
    if (bar->plan.begin < bar->plan.end) {
      unsigned left;
      const Piece x = C::first_piece(p.w, bar->plan, left);
      run_rows<HD>(p, smem, bar, x, left);
    }
  }
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
  p.w.R = S::kRows;
  p.w.by_g = Divisor(p.w.g);
  p.w.by_R = Divisor(p.w.R);
  p.w.by_hk = Divisor(kv.Hkv);
  p.w.join = 0.15f;        // one token of 32 heads on 8 over 5000 rows 12.6 us (0: 12.9, 0.75: 13.9), 8 on one over 500 9.1 (9.4, 10.2)
  p.w.extra = 4u;          // 11 ragged tokens of 32 heads up to 12308 rows 32.5 us (0: 39), 29 of 40 heads 105 (0: 117, 6: 113)
  p.w.starts = starts;
  p.w.status = device_status_ptr();
  p.w.wait_limit = paged_wait().limit_ns;
  p.w.wait_extra = paged_wait().extra;
  const int page = 1 << kv.page_shift;
  p.box = page < kBK ? page : kBK;
  p.q = static_cast<const uint16_t*>(q);
  p.scale_log2 = scale * kLog2e;
  p.out = static_cast<uint16_t*>(out);
  p.w.slots = static_cast<float*>(ws);
  p.w.counters = counters_of(ws);
  const cuuint32_t es[4] = {1, 1, 1, 1};
  CUtensorMap km, vm;
  for (int which = 0; which < 2; ++which) {
    const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(page), S::kHalves, static_cast<cuuint64_t>(kv.n_pages) * kv.Hkv};
    const cuuint64_t strides[3] = {HD * 2, 128, static_cast<cuuint64_t>(page) * HD * 2};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(p.box), S::kHalves, 1};
    if (enc(which ? &vm : &km, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, which ? kv.v : kv.k, dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return fail(MEDUSA_ERR_UNSUPPORTED, "medusa_paged_attention: page tensor map rejected");
  }
  cudaError_t e = cudaFuncSetAttribute(paged_attn_few<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<HD>());
  if (e == cudaSuccess)
    e = launch_kernel(paged_attn_few<HD>, dim3(sm_count()), dim3(kThreads), smem_bytes<HD>(), stream, false, km, vm, p);
  return e == cudaSuccess ? MEDUSA_OK : cuda_fail("medusa_paged_attention: launch (few rows)", e);
}

// Rows of one key head in the largest chunk that the host can vouch for.
long long most_rows(const PagedDev& kv, int N, int H, const int32_t* starts) {
  return static_cast<long long>(starts ? N : N / kv.B) * (H / kv.Hkv);
}

}  // namespace

// Up to 16 rows.  Against 128-row products, with 1, 8 and 16 rows: one sequence
// of 32 heads over 1024 rows 11.1, 11.3 and 12.6 us (13.2, 13.3, 13.5), 8 of 32
// over 4000 85.9, 87.2 (4 rows) and 90.5 (89.1, 90.0, 90.2), 29 of 40 heads of
// 64 over 467..1515 87.7, 92.7 and 99.9 (113, 108, 104).  Many short units of
// heads of 128 pay for every row in the join of the eight warps: 29 sequences
// of 40 heads take 118.5, 121.5, 125, 126.5 and 143.5 us with 2, 4, 6, 8 and 16
// rows (119.5, 121, 122, 115, 114), so those with more than four rows go to
// the other kernel.  17 rows would double the products here: 395 us.
bool paged_attention_few_supported(const PagedDev& kv, medusa_dtype_t dtype, int N, int H, const int32_t* starts) {
  const long long rows = most_rows(kv, N, H, starts);
  const bool many_units = kv.B * kv.Hkv > 4 * sm_count();
  return dtype == MEDUSA_BF16 && (kv.hd == 64 || kv.hd == 128) && rows <= (many_units && kv.hd == 128 ? 4 : 16) &&
         static_cast<long long>(kv.n_pages) * kv.Hkv < 0x7fffffffll;
}

size_t paged_attention_few_workspace_bytes(const PagedDev& kv, int N, int H) {
  return slots_bytes() + counter_bytes(N, H, kv.Hkv, kv.B, 16);
}

medusa_status_t launch_paged_attention_few(const PagedDev& kv, int N, int H, const void* q, float scale, const TreeDev* tree,
                                           const int32_t* starts, void* out, void* ws, cudaStream_t stream) {
  return kv.hd == 128 ? launch<128>(kv, N, H, q, scale, tree, starts, out, ws, stream)
                      : launch<64>(kv, N, H, q, scale, tree, starts, out, ws, stream);
}

}  // namespace medusa
