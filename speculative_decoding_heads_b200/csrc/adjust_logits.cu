// Penalties for repeated tokens, biases and grammar masks on the base logits
// of every tree node, in one pass over [B, T, V].
//
// A block owns kChunk tokens of one sequence's vocabulary.  It counts the
// history's tokens of its chunk in shared memory (one word per token: bit 31
// the token is in the prompt, the low bits its generated occurrences), sums
// the biases, lists the path tokens of its nodes, and turns the counts into
// one addend per token (bias less penalties) and one bit (it occurred), so
// that a logit costs z -> z m + addend with m one of 1, 1/repetition and
// repetition.  Then it streams the chunk of every node of its group, a warp
// per piece of a node's row.  The tokens on
// a node's own path (at most 17) differ from node to node: a lane per path
// token recomputes that token from the logit as it was before the warp wrote
// the piece, and overwrites it.
//
// Trees are bound by HBM, 8 bytes per logit (49 nodes of 16 sequences of 32003
// tokens 42 us, 4.8 TB/s; a plain copy of as many bytes takes 35), in what is
// left after a block's set-up.  Single tokens are bound by that set-up, the
// history's scan above all, which a block's next chunks find in L1 (64 tokens
// of 128001 after 900 tokens each 20 us, with a block for each chunk 22; after
// 257 to 8191 of them 32 us either way).
#include <type_traits>

#include "common.cuh"

namespace medusa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = 2048;                  // tokens per block
constexpr int kPath = MEDUSA_MAX_K + 1;       // nodes on a path
constexpr uint32_t kPrompt = 0x80000000u;

struct LogitArgs {
  TreeDev t;
  int V, words, groups, chunks;
  const float* logits;
  const int32_t* tokens;
  medusa_logit_rules_t r;
  float* out;
  int* status;
};

// 1/repetition is rounded once per block: a division per logit cost more than
// the logit's traffic (86 us for 49 nodes of 16 sequences of 32003, without it 44).
struct Penalty {
  float rep, inv, pres, freq;
};

// What is added to a token's logit apart from the repetition penalty.
__device__ __forceinline__ float addend(uint32_t count, float bias, const Penalty& p) {
  const uint32_t made = count & ~kPrompt;
  return made != 0u ? bias - fmaf(p.freq, static_cast<float>(made), p.pres) : bias;
}
__device__ __forceinline__ float adjust(float z, bool occurred, float add, const Penalty& p) {
  const float m = occurred ? (z > 0.f ? p.inv : p.rep) : 1.f;
  return fmaf(z, m, add);
}

// Node of the l-th set bit of an ancestor-mask row, -1 past the last.
__device__ __forceinline__ int nth_ancestor(const uint64_t* anc, int words, int l) {
  for (int w = 0; w < words; ++w) {
    uint64_t x = anc[w];
    const int c = __popcll(x);
    if (l < c) {
      for (; l > 0; --l) x &= x - 1;
      return 64 * w + __ffsll(static_cast<long long>(x)) - 1;
    }
    l -= c;
  }
  return -1;
}

// kOne: one node per block (T = 1), whose logits use a chunk's counts once: no addends are laid out.
template <bool kOne>
struct Shape {
  static constexpr int kPiece = kOne ? 256 : 512;   // tokens a warp streams at a time, all their loads in flight
  static constexpr int kPerSm = kOne ? 6 : 4;       // blocks that an SM holds
};

template <bool kOne, bool kVec, bool kBias, bool kMask>
__global__ void __launch_bounds__(kThreads, Shape<kOne>::kPerSm) adjust_logits_kernel(const LogitArgs a) {
  __shared__ __align__(16) uint32_t count[kChunk];
  __shared__ __align__(16) float add[kOne ? 1 : kChunk];
  __shared__ uint32_t occurred[kOne ? 1 : kChunk / 32];
  __shared__ __align__(16) float bias[kBias ? kChunk : 1];
  __shared__ int32_t bias_ids[kBias ? MEDUSA_MAX_BIAS : 1];
  constexpr int kPiece = Shape<kOne>::kPiece;
  extern __shared__ int32_t paths[];          // [nodes of the group][kPath] tokens, -1 past a path's end
  const int b = blockIdx.z, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int c0 = blockIdx.x * kChunk, c1 = min(c0 + kChunk, a.V);
  const int T = a.t.T;
  const bool penalties = a.r.repetition || a.r.presence || a.r.frequency;
  const int node0 = static_cast<int>(static_cast<long long>(T) * blockIdx.y / a.groups);
  const int node1 = static_cast<int>(static_cast<long long>(T) * (blockIdx.y + 1) / a.groups);

  int pieces = (c1 - c0 + kPiece - 1) / kPiece, total = (node1 - node0) * pieces;
  float x[kPiece / 32];
  // Tokens v0 .. v1 - 1 of the row z.  A whole piece, the usual one, tests no
  // bounds, and its addresses differ by constants.  Single tokens stream past
  // L1, which keeps the history.
  auto load = [&](const float* z, int v0, int v1) {
    if constexpr (kVec) {
      const float4* p = reinterpret_cast<const float4*>(z + v0) + lane;
#pragma unroll
      for (int k = 0; k < kPiece / 128; ++k)
        if (v1 - v0 == kPiece || v0 + k * 128 + 4 * lane < v1) *reinterpret_cast<float4*>(x + 4 * k) = kOne ? __ldcs(p + 32 * k) : p[32 * k];
    } else {
      const float* p = z + v0 + lane;
      if (v1 - v0 == kPiece) {
#pragma unroll
        for (int k = 0; k < kPiece / 32; ++k) x[k] = kOne ? __ldcs(p + 32 * k) : p[32 * k];
      } else {
#pragma unroll
        for (int k = 0; k < kPiece / 32; ++k)
          if (v0 + k * 32 + lane < v1) x[k] = kOne ? __ldcs(p + 32 * k) : p[32 * k];
      }
    }
  };
  // Piece u of the group: node n of it, tokens [v0, v1).
  auto piece = [&](int u, int& n, int& v0, int& v1) {
    n = u / pieces;
    v0 = c0 + (u - n * pieces) * kPiece;
    v1 = min(v0 + kPiece, c1);
  };
  // A chunk's first piece is loaded while the block sets the chunk up.
  int n, v0, v1;
  auto load_first = [&] {
    if (warp < total) {
      piece(warp, n, v0, v1);
      load(a.logits + (static_cast<size_t>(b) * T + node0 + n) * a.V, v0, v1);
    }
  };
  load_first();

  int hist = 0, prompt = 0;
  if (a.r.history) {
    hist = a.r.history_lens[b];
    if (a.r.prompt_lens) prompt = a.r.prompt_lens[b];
    if (hist < 0 || hist > a.r.history_cap || prompt < 0) {
      if (tid == 0) set_device_status(a.status, MEDUSA_ERR_DEVICE_CHECK, kDetailLogitHistory);
      return;
    }
  }
  const int n_bias = kBias ? a.r.n_bias : 0;
  if constexpr (kBias)
    for (int i = tid; i < n_bias; i += kThreads) bias_ids[i] = a.r.bias_ids[static_cast<size_t>(b) * n_bias + i];
  Penalty pen{1.f, 1.f, 0.f, 0.f};
  if (penalties) {
    if (a.r.repetition) pen.rep = a.r.repetition[b];
    pen.inv = 1.f / pen.rep;
    if (a.r.presence) pen.pres = a.r.presence[b];
    if (a.r.frequency) pen.freq = a.r.frequency[b];
    for (int i = tid; i < (node1 - node0) * kPath; i += kThreads) {
      const int k = i / kPath, l = i - k * kPath;
      const int node = nth_ancestor(a.t.anc + static_cast<size_t>(node0 + k) * a.t.W, a.t.W, l);
      paths[i] = node < 0 ? -1 : a.tokens[static_cast<size_t>(b) * T + node];
    }
  }
  for (int chunk = blockIdx.x;;) {
    for (int i = tid; i < kChunk; i += kThreads) {
      count[i] = 0u;
      if constexpr (kBias) bias[i] = 0.f;
    }
    __syncthreads();
    if (penalties && hist > 0) {
      const int32_t* h = a.r.history + static_cast<size_t>(b) * a.r.history_cap;
      auto note = [&](int v, int i) {
        if (v >= c0 && v < c1) {
          if (i < prompt) atomicOr(&count[v - c0], kPrompt);
          else atomicAdd(&count[v - c0], 1u);
        }
      };
      // 16-byte loads between the first and the last aligned entry.
      const int head = min(hist, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(h) & 15u)) & 15u) / 4);
      const int quads = (hist - head) / 4;
      if (tid < head) note(h[tid], tid);
      const int tail = head + 4 * quads + tid;
      if (tail < hist) note(h[tail], tail);
      const int4* h4 = reinterpret_cast<const int4*>(h + head);
#pragma unroll 4
      for (int i = tid; i < quads; i += kThreads) {
        const int4 v = h4[i];
        note(v.x, head + 4 * i);
        note(v.y, head + 4 * i + 1);
        note(v.z, head + 4 * i + 2);
        note(v.w, head + 4 * i + 3);
      }
    }
    if constexpr (kBias) {
      // A repeated id's values are added in list order by its first entry.
      const float* val = a.r.bias + static_cast<size_t>(b) * n_bias;
      for (int i = tid; i < n_bias; i += kThreads) {
        const int v = bias_ids[i];
        if (v < c0 || v >= c1) continue;
        bool first = true;
        for (int k = 0; k < i && first; ++k) first = bias_ids[k] != v;
        if (!first) continue;
        float s = val[i];
        for (int k = i + 1; k < n_bias; ++k)
          if (bias_ids[k] == v) s += val[k];
        bias[v - c0] = s;
      }
    }
    __syncthreads();
    if constexpr (!kOne) {
      for (int i = tid; i < kChunk; i += kThreads) {
        add[i] = addend(count[i], kBias ? bias[i] : 0.f, pen);
        const uint32_t bits = __ballot_sync(0xffffffffu, count[i] != 0u);
        if (lane == 0) occurred[i >> 5] = bits;
      }
      __syncthreads();
    }

    for (int u = warp; u < total; u += kWarps) {
      piece(u, n, v0, v1);
      const size_t row = static_cast<size_t>(b) * T + node0 + n;
      const float* z = a.logits + row * a.V;
      float* o = a.out + row * a.V;
      const uint32_t* allowed = kMask ? a.r.allowed + row * a.words : nullptr;
      if (u != warp) load(z, v0, v1);
      // Lane l's path token, if it lies in this piece, with its count on the path.
      int mine = -1;
      float fixed = 0.f;
      if (penalties) {
        if (lane < kPath) mine = paths[n * kPath + lane];
        if (mine < v0 || mine >= v1) mine = -1;
        const uint32_t same = __match_any_sync(0xffffffffu, mine);
        if (mine >= 0) {
          fixed = adjust(z[mine], true, addend(count[mine - c0] + __popc(same), kBias ? bias[mine - c0] : 0.f, pen), pen);
          if constexpr (kMask) {
            if (!((allowed[mine >> 5] >> (mine & 31)) & 1u)) fixed = -INFINITY;
          }
        }
        __syncwarp();            // the reads above before the writes below (out may be logits)
      }
      // c0 and v0 are multiples of 32: a word of bits belongs to 32 neighbours of the warp.
      const int at = v0 - c0;
      const uint32_t ok = kMask && lane < kPiece / 32 && v0 + 32 * lane < v1 ? allowed[(v0 >> 5) + lane] : 0u;
      auto finish = [&](bool whole) {
        if constexpr (kVec) {
          float4* p = reinterpret_cast<float4*>(o + v0) + lane;
#pragma unroll
          for (int k = 0; k < kPiece / 128; ++k) {
            float4 y = *reinterpret_cast<float4*>(x + 4 * k);
            float4 w;
            uint32_t c;
            if constexpr (kOne) {
              const uint4 n4 = reinterpret_cast<const uint4*>(count + at)[32 * k + lane];
              w = kBias ? reinterpret_cast<const float4*>(bias + at)[32 * k + lane] : make_float4(0.f, 0.f, 0.f, 0.f);
              w = make_float4(addend(n4.x, w.x, pen), addend(n4.y, w.y, pen), addend(n4.z, w.z, pen), addend(n4.w, w.w, pen));
              c = (n4.x != 0u) | (n4.y != 0u) << 1 | (n4.z != 0u) << 2 | (n4.w != 0u) << 3;
            } else {
              w = reinterpret_cast<const float4*>(add + at)[32 * k + lane];
              c = occurred[(at >> 5) + 4 * k + (lane >> 3)] >> (4 * (lane & 7));
            }
            y.x = adjust(y.x, c & 1u, w.x, pen);
            y.y = adjust(y.y, c & 2u, w.y, pen);
            y.z = adjust(y.z, c & 4u, w.z, pen);
            y.w = adjust(y.w, c & 8u, w.w, pen);
            if constexpr (kMask) {
              const uint32_t m = __shfl_sync(0xffffffffu, ok, 4 * k + (lane >> 3)) >> (4 * (lane & 7));
              if (!(m & 1u)) y.x = -INFINITY;
              if (!(m & 2u)) y.y = -INFINITY;
              if (!(m & 4u)) y.z = -INFINITY;
              if (!(m & 8u)) y.w = -INFINITY;
            }
            if (whole || v0 + k * 128 + 4 * lane < v1) p[32 * k] = y;
          }
        } else {
          float* p = o + v0 + lane;
          const uint32_t bit = 1u << lane;
#pragma unroll
          for (int k = 0; k < kPiece / 32; ++k) {
            float y;
            if constexpr (kOne) {
              const uint32_t c = count[at + 32 * k + lane];
              y = adjust(x[k], c != 0u, addend(c, kBias ? bias[at + 32 * k + lane] : 0.f, pen), pen);
            } else {
              y = adjust(x[k], (occurred[(at >> 5) + k] & bit) != 0u, add[at + 32 * k + lane], pen);
            }
            if constexpr (kMask) {
              if (!(__shfl_sync(0xffffffffu, ok, k) & bit)) y = -INFINITY;
            }
            if (whole || v0 + k * 32 + lane < v1) p[32 * k] = y;
          }
        }
      };
      if (v1 - v0 == kPiece) finish(true);
      else finish(false);
      if (penalties) {
        __syncwarp();
        if (mine >= 0) o[mine] = fixed;   // lanes with the same token write the same value
      }
    }
    chunk += gridDim.x;
    if (chunk >= a.chunks) return;
    c0 = chunk * kChunk;
    c1 = min(c0 + kChunk, a.V);
    pieces = (c1 - c0 + kPiece - 1) / kPiece;
    total = (node1 - node0) * pieces;
    load_first();
    __syncthreads();           // the chunk before is done with shared memory
  }
}

}  // namespace

medusa_status_t launch_adjust_logits(const TreeDev& t, int B, int V, const float* logits, const int32_t* tree_tokens,
                                     const medusa_logit_rules_t& rules, float* out, cudaStream_t stream) {
  LogitArgs a{};
  a.t = t;
  a.V = V;
  a.words = (V + 31) / 32;
  a.logits = logits;
  a.tokens = tree_tokens;
  a.r = rules;
  a.out = out;
  a.status = device_status_ptr();
  a.chunks = (V + kChunk - 1) / kChunk;
  // One wave of the blocks that the SMs hold: node groups where there are too
  // few chunks (a block's set-up scans the whole history), each with a piece
  // for every warp, or several chunks to a block, which finds the history in
  // L1 again.
  const bool one = t.T == 1;
  const int slots = (one ? Shape<true>::kPerSm : Shape<false>::kPerSm) * sm_count();
  const long long base = static_cast<long long>(a.chunks) * B;
  const long long want = slots / base < 1 ? 1 : slots / base;
  const int per_warp = t.T * (kChunk / Shape<false>::kPiece) / kWarps, most = one || per_warp < 1 ? 1 : per_warp;
  a.groups = want > most ? most : static_cast<int>(want);
  const int rounds = static_cast<int>((base + slots - 1) / slots);
  const dim3 grid((a.chunks + rounds - 1) / rounds, a.groups, B);
  const size_t smem = static_cast<size_t>((t.T + a.groups - 1) / a.groups) * kPath * sizeof(int32_t);   // at most 17 KB
  const bool vec = V % 4 == 0 && ((reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
  const bool bias = rules.bias != nullptr, mask = rules.allowed != nullptr;
  auto go = [&](auto kernel) { kernel<<<grid, kThreads, smem, stream>>>(a); };
  auto pick = [&](auto size) {
    constexpr bool P = decltype(size)::value;
    if (vec) {
      if (bias) mask ? go(adjust_logits_kernel<P, true, true, true>) : go(adjust_logits_kernel<P, true, true, false>);
      else mask ? go(adjust_logits_kernel<P, true, false, true>) : go(adjust_logits_kernel<P, true, false, false>);
    } else {
      if (bias) mask ? go(adjust_logits_kernel<P, false, true, true>) : go(adjust_logits_kernel<P, false, true, false>);
      else mask ? go(adjust_logits_kernel<P, false, false, true>) : go(adjust_logits_kernel<P, false, false, false>);
    }
  };
  if (one) pick(std::true_type{});
  else pick(std::false_type{});
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? MEDUSA_OK : cuda_fail("medusa_adjust_logits", e);
}

}  // namespace medusa
