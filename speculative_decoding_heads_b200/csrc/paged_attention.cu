// Attention of new tokens over a paged cache, fp32 arithmetic on the CUDA
// cores: every dtype, head size and group size.  Bf16 heads of 64 and 128
// come here only with a scale of at most 0, or in groups of more than 128 query
// heads; otherwise paged_attention_few.cu takes them where a sequence's rows of
// a key head are few, paged_attention_tc.cu the rest.
//
// One pass over the keys with a running maximum and sum per query row: with
// m' = max(m, max_j s_j), O <- O 2^(m - m') + sum_j 2^(s_j - m') V_j and the
// same for the sum l, the output is O / l whatever the order of the blocks.
// A CTA holds R query rows and takes 32 or 64 keys at a time through shared
// memory as fp32; a thread owns R / 16 or R / 8 rows x 2 or 4 keys of the
// scores and the same rows x HD / 16 dimensions of O, so one 16-byte
// shared-memory read feeds 4 products of the scores and 5 to 7 of the outputs
// (R = 16), or 8 and 8 to 13 (R = 64).  The probabilities take the place of the
// keys, which leaves room for more CTAs per SM: some compute while the others'
// loads are in flight.
//
// R = 16 where a sequence's rows fit (decoding and small trees): bound by the
// latency of a block's loads, products and barriers, hence blocks of 32 keys,
// four or five CTAs per SM, and warps without a row that only load (4 tokens
// of 32 fp32 heads over 2721 rows 103 us, 3.5 TB/s; blocks of 64 keys, two
// CTAs and every warp computing took 263).  R = 64 otherwise, bound by fp32
// arithmetic and its shared-memory reads (4 x 257 tokens of the same heads
// 1.78 ms, 27 TFLOP/s).
#include "paged_work.cuh"

namespace medusa {
namespace {

using namespace paged;

constexpr float kLog2e = 1.4426950408889634f;

template <typename T>
__device__ __forceinline__ float4 load4(const T* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) { return *reinterpret_cast<const float4*>(p); }
template <>
__device__ __forceinline__ float4 load4<uint16_t>(const uint16_t* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return make_float4(bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y));
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(uint16_t* p, float4 v) {
  *reinterpret_cast<uint2*>(p) =
      make_uint2(static_cast<uint32_t>(f32_to_bf16_rne(v.x)) | (static_cast<uint32_t>(f32_to_bf16_rne(v.y)) << 16),
                 static_cast<uint32_t>(f32_to_bf16_rne(v.z)) | (static_cast<uint32_t>(f32_to_bf16_rne(v.w)) << 16));
}

template <int HD, int R>
struct Shape {
  static constexpr int kBK = R == 16 ? 32 : 64;       // keys per block
  static constexpr int kRows = R == 16 ? 2 : 4;       // query rows per thread
  static constexpr int kThreads = R / kRows * 16;     // 16 threads side by side per row group
  static constexpr int kPitch = HD + 4;               // floats per row: conflict-free 16-byte reads down a column
  static constexpr int kPPitch = kBK + 4;
  static_assert(R * kPPitch <= kBK * kPitch, "the probabilities take the place of the keys");
  static constexpr size_t kSmem = static_cast<size_t>(R + 2 * kBK) * kPitch * sizeof(float);
  static constexpr int kPerSm = kSmem > 112 * 1024 ? 1 : kSmem > 74 * 1024 || R == 64 ? 2 : HD == 128 ? 4 : 5;
  static constexpr int kLoads = kBK * (HD / 4) / kThreads;   // four-element loads of K, and of V, per thread and block
  static constexpr int kBatch = kLoads < 8 ? kLoads : 8;     // in flight together
  static_assert(2 * kPerSm * slot_floats(R, HD) <= kSlotFloatsPerSm, "two slots per CTA");
  static_assert(kLoads % kBatch == 0 && kBK * (HD / 4) % kThreads == 0, "whole batches");
};

template <typename T, int HD, int R>
__global__ void __launch_bounds__(Shape<HD, R>::kThreads, Shape<HD, R>::kPerSm) paged_attn_kernel(const Work w, const T* q, float scale_log2, T* out) {
  using S = Shape<HD, R>;
  constexpr int kBK = S::kBK, KC = kBK / 16;       // KC keys per thread
  using C = Cut<kBK>;
  constexpr int NT = S::kThreads, RR = S::kRows, DV = HD / 64;   // DV groups of 4 dimensions per thread
  extern __shared__ __align__(16) float sh[];
  float* qs = sh;
  float* ks = qs + R * S::kPitch;
  float* vs = ks + kBK * S::kPitch;
  float* ps = ks;
  __shared__ Plan plan;
  __shared__ int s_last;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int hd = w.kv.hd, g = w.g, hd4 = hd / 4;
  if (tid < 32) C::plan(w, plan);
  __syncthreads();
  if (plan.begin >= plan.end) return;
  unsigned left;
  Piece x = C::first_piece(w, plan, left);
  const int shift = w.kv.page_shift, mask = (1 << shift) - 1;
  for (;;) {
    const int b = x.b, L = plan.L[b], n = plan.n[b], first = plan.first[b];
    const int rows = min(R, n * g - x.tile * R);
    const bool mine = R > 16 || (ty & ~1) * RR < rows;     // this warp has rows
    const int keys = C::keys(w, plan, b, x.tile);
    __syncthreads();                       // the piece before is done with shared memory
    for (int i = tid; i < R * (HD / 4); i += NT) {
      const int r = i / (HD / 4), d = i - r * (HD / 4);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows && d < hd4) {
        const int rr = x.tile * R + r, tok = rr / w.by_g, head = x.h * g + rr - tok * g;
        v = load4<T>(q + (static_cast<size_t>(first + tok) * w.H + head) * hd + 4 * d);
      }
      *reinterpret_cast<float4*>(qs + r * S::kPitch + 4 * d) = v;
    }
    float m[RR], l[RR], o[RR][DV][4];
#pragma unroll
    for (int r = 0; r < RR; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int d = 0; d < DV; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[r][d][e] = 0.f;
    }
    for (int kb = x.kb0; kb < x.kb1; ++kb) {
      const int j0 = kb * kBK;
      __syncthreads();
      // A batch's places first, then its loads together: one after the other
      // they took as long as the products.
#pragma unroll 1
      for (int base = 0; base < S::kLoads; base += S::kBatch) {
        long long off[S::kBatch];
        float4 tk[S::kBatch], tv[S::kBatch];
#pragma unroll
        for (int u = 0; u < S::kBatch; ++u) {
          const int i = tid + (base + u) * NT, r = i / (HD / 4), d = i - r * (HD / 4);
          off[u] = -1;
          if (j0 + r < keys && d < hd4) {    // rows past the sequence are not read
            const int page = w.kv.table[static_cast<long long>(b) * w.kv.max_pages + ((j0 + r) >> shift)];
            if (page >= 0 && page < w.kv.n_pages)
              off[u] = (((static_cast<long long>(page) * w.kv.Hkv + x.h) << shift) + ((j0 + r) & mask)) * hd + 4 * d;
            else
              set_device_status(w.status, MEDUSA_ERR_DEVICE_CHECK, kDetailPagedPage);
          }
        }
        auto fetch = [&](const void* from, float4 (&t)[S::kBatch]) {
#pragma unroll
          for (int u = 0; u < S::kBatch; ++u) t[u] = off[u] >= 0 ? load4<T>(static_cast<const T*>(from) + off[u]) : make_float4(0.f, 0.f, 0.f, 0.f);
        };
        auto put = [&](const float4 (&t)[S::kBatch], float* to) {
#pragma unroll
          for (int u = 0; u < S::kBatch; ++u) {
            const int i = tid + (base + u) * NT, r = i / (HD / 4), d = i - r * (HD / 4);
            *reinterpret_cast<float4*>(to + r * S::kPitch + 4 * d) = t[u];
          }
        };
        fetch(w.kv.k, tk);
        fetch(w.kv.v, tv);
        put(tk, ks);
        put(tv, vs);
      }
      __syncthreads();
      float s[RR][KC];
      if (mine) {
#pragma unroll
        for (int r = 0; r < RR; ++r)
#pragma unroll
          for (int c = 0; c < KC; ++c) s[r][c] = 0.f;
#pragma unroll 4
        for (int d = 0; d < HD / 4; ++d) {
          float4 a[RR], k4[KC];
#pragma unroll
          for (int r = 0; r < RR; ++r) a[r] = *reinterpret_cast<const float4*>(qs + (ty * RR + r) * S::kPitch + 4 * d);
#pragma unroll
          for (int c = 0; c < KC; ++c) k4[c] = *reinterpret_cast<const float4*>(ks + (tx + 16 * c) * S::kPitch + 4 * d);
#pragma unroll
          for (int r = 0; r < RR; ++r)
#pragma unroll
            for (int c = 0; c < KC; ++c)
              s[r][c] = fmaf(a[r].x, k4[c].x, fmaf(a[r].y, k4[c].y, fmaf(a[r].z, k4[c].z, fmaf(a[r].w, k4[c].w, s[r][c]))));
        }
      }
      __syncthreads();                     // P goes where K was
      if (!mine) continue;
#pragma unroll
      for (int r = 0; r < RR; ++r) {
        const int rr = x.tile * R + ty * RR + r, tok = rr / w.by_g;
        float mx = -INFINITY;
        // Nodes j0 - L .. of the tree that this row sees, one bit per key of the block.
        uint64_t sees = 0ull;
        if (w.t.T > 0 && j0 + kBK > L && tok < n) {
          const int o = j0 - L, wi = o >= 0 ? o >> 6 : 0, sh = o >= 0 ? o & 63 : -o;
          const uint64_t* a = w.t.anc + tok * w.t.W;
          const uint64_t w0 = wi < w.t.W ? a[wi] : 0ull, w1 = wi + 1 < w.t.W ? a[wi + 1] : 0ull;
          sees = o < 0 ? w0 << sh | ((1ull << sh) - 1ull) : sh == 0 ? w0 : (w0 >> sh) | (w1 << (64 - sh));
        }
#pragma unroll
        for (int c = 0; c < KC; ++c) {
          const int j = j0 + tx + 16 * c, rel = j - L;
          bool see;
          if (w.t.T > 0)
            see = rel < 0 || (rel < n && (sees >> (tx + 16 * c) & 1ull));
          else
            see = rel <= tok && rel < n;
          s[r][c] = see ? s[r][c] * scale_log2 : -INFINITY;
          mx = fmaxf(mx, s[r][c]);
        }
        for (int off = 8; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const float mn = fmaxf(m[r], mx), ref = mn == -INFINITY ? 0.f : mn;
        const float f = exp2f(m[r] - ref);
        float sum = 0.f;
#pragma unroll
        for (int c = 0; c < KC; ++c) {
          const float p = exp2f(s[r][c] - ref);
          ps[(ty * RR + r) * S::kPPitch + tx + 16 * c] = p;
          sum += p;
        }
        for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        m[r] = mn;
        l[r] = l[r] * f + sum;
#pragma unroll
        for (int d = 0; d < DV; ++d)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[r][d][e] *= f;
      }
      __syncwarp();                        // a row's probabilities are written and read by one half-warp
#pragma unroll 4
      for (int j = 0; j < kBK; j += 4) {
        float4 pr[RR];
#pragma unroll
        for (int r = 0; r < RR; ++r) pr[r] = *reinterpret_cast<const float4*>(ps + (ty * RR + r) * S::kPPitch + j);
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int d = 0; d < DV; ++d) {
            const float4 v4 = *reinterpret_cast<const float4*>(vs + (j + u) * S::kPitch + 64 * d + 4 * tx);
#pragma unroll
            for (int r = 0; r < RR; ++r) {
              const float p = u == 0 ? pr[r].x : u == 1 ? pr[r].y : u == 2 ? pr[r].z : pr[r].w;
              o[r][d][0] = fmaf(p, v4.x, o[r][d][0]);
              o[r][d][1] = fmaf(p, v4.y, o[r][d][1]);
              o[r][d][2] = fmaf(p, v4.z, o[r][d][2]);
              o[r][d][3] = fmaf(p, v4.w, o[r][d][3]);
            }
          }
      }
    }
    bool write = C::whole(x);
    if (!write) {
      // Leave the piece in this CTA's slot; the last piece of the unit joins them.
      float* slot = w.slots + C::slot(plan, blockIdx.x, x.start) * slot_floats(R, HD);
#pragma unroll
      for (int r = 0; r < RR; ++r) {
        const int row = ty * RR + r;
        if (tx == 0) {
          __stcg(slot + row, m[r]);
          __stcg(slot + R + row, l[r]);
        }
#pragma unroll
        for (int d = 0; d < DV; ++d)
          __stcg(reinterpret_cast<float4*>(slot + 2 * R + row * HD + 64 * d + 4 * tx),
                 make_float4(o[r][d][0], o[r][d][1], o[r][d][2], o[r][d][3]));
      }
      __syncthreads();                     // then one thread's release covers all of them
      int c_lo, c_hi;
      C::owners(plan, x, c_lo, c_hi);
      if (tid == 0) {
        unsigned* ctr = C::counter(w, plan, x);
        s_last = atom_add_acq_rel_gpu(ctr, 1u) == static_cast<unsigned>(c_hi - c_lo);
        if (s_last) *ctr = 0u;
      }
      __syncthreads();
      write = s_last != 0;
      if (write) {
        // kPB pieces' loads (from L2) in flight together: one after the other they took as long as a block.
        constexpr int kPB = RR * DV <= 4 ? 4 : RR * DV <= 8 ? 2 : 1;
#pragma unroll
        for (int r = 0; r < RR; ++r) {
          m[r] = -INFINITY;
          l[r] = 0.f;
#pragma unroll
          for (int d = 0; d < DV; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[r][d][e] = 0.f;
        }
#pragma unroll 1
        for (int c0 = c_lo; c0 <= c_hi; c0 += kPB) {
          float ms[RR][kPB], ls[RR][kPB];
          float4 v[RR][kPB][DV];
#pragma unroll
          for (int c = 0; c < kPB; ++c) {
            const float* sl = w.slots + C::slot(plan, min(c0 + c, c_hi), x.start) * slot_floats(R, HD);
#pragma unroll
            for (int r = 0; r < RR; ++r) {
              const int row = ty * RR + r;
              const bool have = c0 + c <= c_hi;
              ms[r][c] = have ? __ldcg(sl + row) : -INFINITY;
              ls[r][c] = have ? __ldcg(sl + R + row) : 0.f;
#pragma unroll
              for (int d = 0; d < DV; ++d)
                v[r][c][d] = have ? __ldcg(reinterpret_cast<const float4*>(sl + 2 * R + row * HD + 64 * d + 4 * tx))
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
            }
          }
#pragma unroll
          for (int r = 0; r < RR; ++r) {
            float mn = m[r];
#pragma unroll
            for (int c = 0; c < kPB; ++c) mn = fmaxf(mn, ms[r][c]);
            const float ref = mn == -INFINITY ? 0.f : mn, keep = exp2f(m[r] - ref);
            m[r] = mn;
            l[r] *= keep;
#pragma unroll
            for (int d = 0; d < DV; ++d)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[r][d][e] *= keep;
#pragma unroll
            for (int c = 0; c < kPB; ++c) {
              const float f = exp2f(ms[r][c] - ref);
              l[r] = fmaf(f, ls[r][c], l[r]);
#pragma unroll
              for (int d = 0; d < DV; ++d) {
                o[r][d][0] = fmaf(f, v[r][c][d].x, o[r][d][0]);
                o[r][d][1] = fmaf(f, v[r][c][d].y, o[r][d][1]);
                o[r][d][2] = fmaf(f, v[r][c][d].z, o[r][d][2]);
                o[r][d][3] = fmaf(f, v[r][c][d].w, o[r][d][3]);
              }
            }
          }
        }
      }
    }
    if (write) {
#pragma unroll
      for (int r = 0; r < RR; ++r) {
        const int row = ty * RR + r;
        if (row >= rows) continue;
        const int rr = x.tile * R + row, tok = rr / w.by_g, head = x.h * g + rr - tok * g;
        const float inv = 1.f / l[r];
        T* dst = out + (static_cast<size_t>(first + tok) * w.H + head) * hd;
#pragma unroll
        for (int d = 0; d < DV; ++d)
          if (64 * d + 4 * tx < hd)
            store4(dst + 64 * d + 4 * tx, make_float4(o[r][d][0] * inv, o[r][d][1] * inv, o[r][d][2] * inv, o[r][d][3] * inv));
      }
    }
    if (left == 0) break;
    C::next_piece(w, plan, x, left);
  }
}

struct Choice {
  int R, HD, per_sm;
};

// R = 16 while a sequence's rows of one key head fit in 16 on average.
Choice choose(const PagedDev& kv, int N, int H) {
  Choice c;
  c.HD = kv.hd <= 64 ? 64 : kv.hd <= 128 ? 128 : 256;
  c.R = static_cast<long long>(N) * (H / kv.Hkv) <= 16ll * kv.B ? 16 : 64;
  auto per = [&](auto hd) {
    constexpr int kHD = decltype(hd)::value;
    return c.R == 16 ? Shape<kHD, 16>::kPerSm : Shape<kHD, 64>::kPerSm;
  };
  c.per_sm = c.HD == 64 ? per(std::integral_constant<int, 64>{})
             : c.HD == 128 ? per(std::integral_constant<int, 128>{})
                           : per(std::integral_constant<int, 256>{});
  return c;
}

template <typename T, int HD, int R>
cudaError_t run(const Work& w, int grid, const void* q, float scale_log2, void* out, cudaStream_t stream) {
  auto fn = paged_attn_kernel<T, HD, R>;
  constexpr size_t smem = Shape<HD, R>::kSmem;
  const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  fn<<<grid, Shape<HD, R>::kThreads, smem, stream>>>(w, static_cast<const T*>(q), scale_log2, static_cast<T*>(out));
  return cudaGetLastError();
}

template <typename T>
cudaError_t run_for(const Choice& c, const Work& w, int grid, const void* q, float s, void* out, cudaStream_t st) {
  if (c.R == 16) {
    if (c.HD == 64) return run<T, 64, 16>(w, grid, q, s, out, st);
    if (c.HD == 128) return run<T, 128, 16>(w, grid, q, s, out, st);
    return run<T, 256, 16>(w, grid, q, s, out, st);
  }
  if (c.HD == 64) return run<T, 64, 64>(w, grid, q, s, out, st);
  if (c.HD == 128) return run<T, 128, 64>(w, grid, q, s, out, st);
  return run<T, 256, 64>(w, grid, q, s, out, st);
}

}  // namespace

size_t paged_attention_workspace_bytes(const PagedDev& kv, medusa_dtype_t dtype, int N, int H) {
  const Choice c = choose(kv, N, H);
  size_t tc = paged_attention_tc_supported(kv, dtype, H) ? paged_attention_tc_workspace_bytes(kv, N, H) : 0;
  if (paged_attention_few_supported(kv, dtype, N, H, nullptr)) {
    const size_t few = paged_attention_few_workspace_bytes(kv, N, H);
    tc = few > tc ? few : tc;
  }
  const size_t any = slots_bytes() + counter_bytes(N, H, kv.Hkv, kv.B, c.R);
  return tc > any ? tc : any;      // the scale and the chunks, known only at the call, decide between them
}

medusa_status_t launch_paged_attention(const PagedDev& kv, medusa_dtype_t dtype, int N, int H, const void* q,
                                       float scale, const TreeDev* tree, const int32_t* starts, void* out, void* ws,
                                       cudaStream_t stream) {
  // These two take the maximum of the unscaled scores.
  if (scale > 0.f && paged_attention_few_supported(kv, dtype, N, H, starts))
    return launch_paged_attention_few(kv, N, H, q, scale, tree, starts, out, ws, stream);
  if (scale > 0.f && paged_attention_tc_supported(kv, dtype, H))
    return launch_paged_attention_tc(kv, N, H, q, scale, tree, starts, out, ws, stream);
  Work w{};
  w.kv = kv;
  if (tree) w.t = *tree;
  w.N = N;
  w.H = H;
  w.g = H / kv.Hkv;
  w.starts = starts;
  w.status = device_status_ptr();
  const Choice c = choose(kv, N, H);
  w.R = c.R;
  w.by_g = Divisor(w.g);
  w.by_R = Divisor(w.R);
  w.by_hk = Divisor(kv.Hkv);
  // Both measured: a 15-node fp32 tree of 4 heads over 4000 rows 23.5 us (no bound on the cut: 36.1, 0.15: 23.7), 64
  // tokens of 4 heads on one after 1500 rows 30.9 (31.1, with 0.1 36.8).  Extra blocks behind a unit only cost: 29
  // ragged fp32 tokens of 40 heads on 8 over 50..700 rows 42.0 us (one: 43.9, two: 45.7), 257 tokens of 64 heads 63.1
  // (one: 68.0).
  w.join = c.R == 16 ? 0.03f : 0.02f;
  w.extra = 0u;
  w.slots = static_cast<float*>(ws);
  w.counters = counters_of(ws);
  const int grid = sm_count() * c.per_sm;
  const float s = scale * kLog2e;
  const cudaError_t e = dtype == MEDUSA_BF16 ? run_for<uint16_t>(c, w, grid, q, s, out, stream)
                                             : run_for<float>(c, w, grid, q, s, out, stream);
  return e == cudaSuccess ? MEDUSA_OK : cuda_fail("medusa_paged_attention", e);
}

}  // namespace medusa
