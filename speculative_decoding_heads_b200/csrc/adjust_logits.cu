// Penalties for repeated tokens, biases and grammar masks on the base logits
// of every tree node, in one pass over [B, T, V].
//
// A block owns kChunk tokens of one sequence's vocabulary.  It counts the
// history's tokens of its chunk in shared memory (one word per token: bit 31
// the token is in the prompt, the low bits its generated occurrences), sums
// the biases, and then streams the chunk of every node of its group, a warp
// per piece of a node's row.  The tokens on a node's own path (at most 17)
// differ from node to node: a lane per path token recomputes that token from
// the logit it read before the warp wrote the piece, and overwrites it.
//
// Bound by HBM: 8 bytes per logit; the history is read once per block, from L2.
#include "common.cuh"

namespace medusa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = 2048;                  // tokens per block
constexpr int kPiece = 512;                   // tokens a warp streams at a time: 16 per lane
constexpr uint32_t kPrompt = 0x80000000u;

struct LogitArgs {
  TreeDev t;
  int V, words, groups;
  const float* logits;
  const int32_t* tokens;
  medusa_logit_rules_t r;
  float* out;
  int* status;
};

struct Penalty {
  float rep, pres, freq;
};

__device__ __forceinline__ float penalise(float z, uint32_t count, const Penalty& p) {
  if (count != 0u) z = z > 0.f ? z / p.rep : z * p.rep;
  const uint32_t made = count & ~kPrompt;
  if (made != 0u) z -= p.freq * static_cast<float>(made) + p.pres;
  return z;
}

// Tokens [v, v + 4) of a piece, aligned (kVec) or one token.
template <bool kVec, bool kBias, bool kMask>
__device__ __forceinline__ void stream_piece(const float* z, float* o, const uint32_t* allowed, const uint32_t* count,
                                             const float* bias, int v0, int v1, int lane, const Penalty& pen) {
  if constexpr (kVec) {
    float4 x[kPiece / 128];
#pragma unroll
    for (int u = 0; u < kPiece / 128; ++u) {
      const int v = v0 + u * 128 + 4 * lane;
      if (v < v1) x[u] = *reinterpret_cast<const float4*>(z + v);
    }
#pragma unroll
    for (int u = 0; u < kPiece / 128; ++u) {
      const int v = v0 + u * 128 + 4 * lane;
      if (v >= v1) continue;
      const uint4 c = *reinterpret_cast<const uint4*>(count + (v & (kChunk - 1)));
      if ((c.x | c.y | c.z | c.w) != 0u) {
        x[u].x = penalise(x[u].x, c.x, pen);
        x[u].y = penalise(x[u].y, c.y, pen);
        x[u].z = penalise(x[u].z, c.z, pen);
        x[u].w = penalise(x[u].w, c.w, pen);
      }
      if constexpr (kBias) {
        const float4 w = *reinterpret_cast<const float4*>(bias + (v & (kChunk - 1)));
        x[u].x += w.x;
        x[u].y += w.y;
        x[u].z += w.z;
        x[u].w += w.w;
      }
      if constexpr (kMask) {
        const uint32_t m = allowed[v >> 5] >> (v & 31);
        if (!(m & 1u)) x[u].x = -INFINITY;
        if (!(m & 2u)) x[u].y = -INFINITY;
        if (!(m & 4u)) x[u].z = -INFINITY;
        if (!(m & 8u)) x[u].w = -INFINITY;
      }
      *reinterpret_cast<float4*>(o + v) = x[u];
    }
  } else {
    float x[kPiece / 32];
#pragma unroll
    for (int u = 0; u < kPiece / 32; ++u) {
      const int v = v0 + u * 32 + lane;
      if (v < v1) x[u] = z[v];
    }
#pragma unroll
    for (int u = 0; u < kPiece / 32; ++u) {
      const int v = v0 + u * 32 + lane;
      if (v >= v1) continue;
      x[u] = penalise(x[u], count[v & (kChunk - 1)], pen);
      if constexpr (kBias) x[u] += bias[v & (kChunk - 1)];
      if constexpr (kMask) {
        if (!((allowed[v >> 5] >> (v & 31)) & 1u)) x[u] = -INFINITY;
      }
      o[v] = x[u];
    }
  }
}

template <bool kVec, bool kBias, bool kMask>
__global__ void __launch_bounds__(kThreads) adjust_logits_kernel(const LogitArgs a) {
  __shared__ __align__(16) uint32_t count[kChunk];
  __shared__ __align__(16) float bias[kBias ? kChunk : 4];
  const int b = blockIdx.z, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c0 = blockIdx.x * kChunk, c1 = min(c0 + kChunk, a.V);
  const int T = a.t.T;
  const bool penalties = a.r.repetition || a.r.presence || a.r.frequency;

  int hist = 0, prompt = 0;
  if (a.r.history) {
    hist = a.r.history_lens[b];
    if (a.r.prompt_lens) prompt = a.r.prompt_lens[b];
    if (hist < 0 || hist > a.r.history_cap || prompt < 0) {
      if (tid == 0) set_device_status(a.status, MEDUSA_ERR_DEVICE_CHECK, kDetailLogitHistory);
      return;
    }
  }
  for (int i = tid; i < kChunk; i += kThreads) {
    count[i] = 0u;
    if constexpr (kBias) bias[i] = 0.f;
  }
  __syncthreads();
  Penalty pen{1.f, 0.f, 0.f};
  if (penalties) {
    if (a.r.repetition) pen.rep = a.r.repetition[b];
    if (a.r.presence) pen.pres = a.r.presence[b];
    if (a.r.frequency) pen.freq = a.r.frequency[b];
    if (a.r.history) {
      const int32_t* h = a.r.history + static_cast<size_t>(b) * a.r.history_cap;
#pragma unroll 8
      for (int i = tid; i < hist; i += kThreads) {
        const int v = h[i];
        if (v >= c0 && v < c1) {
          if (i < prompt) atomicOr(&count[v - c0], kPrompt);
          else atomicAdd(&count[v - c0], 1u);
        }
      }
    }
  }
  if constexpr (kBias) {
    // A repeated id's values are added in list order by its first entry.
    const int32_t* ids = a.r.bias_ids + static_cast<size_t>(b) * a.r.n_bias;
    const float* val = a.r.bias + static_cast<size_t>(b) * a.r.n_bias;
    for (int i = tid; i < a.r.n_bias; i += kThreads) {
      const int v = ids[i];
      if (v < c0 || v >= c1) continue;
      bool first = true;
      for (int k = 0; k < i && first; ++k) first = ids[k] != v;
      if (!first) continue;
      float s = val[i];
      for (int k = i + 1; k < a.r.n_bias; ++k)
        if (ids[k] == v) s += val[k];
      bias[v - c0] = s;
    }
  }
  __syncthreads();

  const int pieces = (c1 - c0 + kPiece - 1) / kPiece;
  const int node0 = static_cast<int>(static_cast<long long>(T) * blockIdx.y / a.groups);
  const int node1 = static_cast<int>(static_cast<long long>(T) * (blockIdx.y + 1) / a.groups);
  for (int u = warp; u < (node1 - node0) * pieces; u += kWarps) {
    const int i = node0 + u / pieces, v0 = c0 + (u % pieces) * kPiece, v1 = min(v0 + kPiece, c1);
    const size_t row = (static_cast<size_t>(b) * T + i);
    const float* z = a.logits + row * a.V;
    float* o = a.out + row * a.V;
    const uint32_t* allowed = kMask ? a.r.allowed + row * a.words : nullptr;
    // Lane l holds the path's node l steps above i, if any.
    int mine = -1;
    float fixed = 0.f;
    if (penalties) {
      int node = i;
      const int up = a.t.depth[i];
      for (int l = 0; l <= up; ++l) {
        if (l == lane) mine = a.tokens[static_cast<size_t>(b) * T + node];
        node = a.t.parent[node];
      }
      const bool here = mine >= v0 && mine < v1;
      if (!here) mine = -1;
      if (__any_sync(0xffffffffu, here)) {
        uint32_t more = 0u;
        for (int l = 0; l <= up; ++l) more += __shfl_sync(0xffffffffu, mine, l) == mine;
        if (here) {
          fixed = penalise(z[mine], count[mine - c0] + more, pen);
          if constexpr (kBias) fixed += bias[mine - c0];
          if constexpr (kMask) {
            if (!((allowed[mine >> 5] >> (mine & 31)) & 1u)) fixed = -INFINITY;
          }
        }
      }
      __syncwarp();            // the reads above before the writes below (out may be logits)
    }
    stream_piece<kVec, kBias, kMask>(z, o, allowed, count, bias, v0, v1, lane, pen);
    if (penalties) {
      __syncwarp();
      if (mine >= 0) o[mine] = fixed;   // lanes with the same token write the same value
    }
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
  const int chunks = (V + kChunk - 1) / kChunk;
  // Node groups until the launch has about four blocks per SM, each with at
  // least eight nodes (a block's set-up scans the whole history).
  const long long base = static_cast<long long>(chunks) * B;
  const int want = static_cast<int>((4ll * sm_count() + base - 1) / base);
  const int most = t.T / 8 < 1 ? 1 : t.T / 8;
  a.groups = want < 1 ? 1 : want > most ? most : want;
  const dim3 grid(chunks, a.groups, B);
  const bool vec = V % 4 == 0 && ((reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
  const bool bias = rules.bias != nullptr, mask = rules.allowed != nullptr;
  auto go = [&](auto kernel) { kernel<<<grid, kThreads, 0, stream>>>(a); };
  if (vec) {
    if (bias) mask ? go(adjust_logits_kernel<true, true, true>) : go(adjust_logits_kernel<true, true, false>);
    else mask ? go(adjust_logits_kernel<true, false, true>) : go(adjust_logits_kernel<true, false, false>);
  } else {
    if (bias) mask ? go(adjust_logits_kernel<false, true, true>) : go(adjust_logits_kernel<false, true, false>);
    else mask ? go(adjust_logits_kernel<false, false, true>) : go(adjust_logits_kernel<false, false, false>);
  }
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? MEDUSA_OK : cuda_fail("medusa_adjust_logits", e);
}

}  // namespace medusa
