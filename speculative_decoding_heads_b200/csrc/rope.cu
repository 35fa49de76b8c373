// Rotary positions of new tokens and their place in a paged cache: queries
// and keys are rotated, keys and values written to their pages, in one pass.
//
// Pair i of a head turns by position * f_i.  At position 10^6 the product has
// an absolute error of 0.06 rad in fp32, so the frequency is kept as a 64-bit
// fraction of a turn: position * turns modulo 2^64 is the angle by integer
// wrap-around, exact for any position; its top 32 bits give the angle to
// 2^-32 turns.  A block computes cos and sin once per (token, pair) into
// shared memory for all H + Hkv heads.
//
// Bound by HBM: every element is read once and written once (8445 tokens of
// 32 + 2 x 8 heads of 128 46 us, 4.5 TB/s; a plain copy of as many bytes takes
// 35).  One wave of blocks, so that each sets up once: two to eight waves took
// as long, a block per token 51 us.
#include "common.cuh"

namespace medusa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTok = 32;     // tokens per block

struct RopeArgs {
  PagedDev kv;
  int N, H, rot, half, tok;     // half: MEDUSA_ROPE_HALF
  const void* q;
  const void* k;
  const void* v;
  int64_t qs, ks, vs;
  void* q_out;
  const uint64_t* turns;
  float amplitude;
  const int32_t* positions;
  const int32_t* starts;
  int* status;
};

// Where a token of the packed list goes: `base` is its element offset inside
// its page block (head 0), or -1 when it is to be left alone.
struct Place {
  long long base;
  int pos;
};

__device__ Place place_token(const RopeArgs& a, int n, const int32_t* starts /* shared, or null */) {
  Place pl{-1, 0};
  const int B = a.kv.B;
  int b, first, last;
  if (starts == nullptr) {
    const int each = a.N / B;
    b = n / each;
    first = b * each;
    last = first + each;
  } else {
    int lo = 0, hi = B;          // largest b with starts[b] <= n
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (starts[mid] <= n) lo = mid; else hi = mid;
    }
    b = lo;
    first = starts[b];
    last = starts[b + 1];
    if (first < 0 || n < first || n >= last || last > a.N) return pl;   // behind the last sequence, or no chunk
  }
  const int L = a.kv.lens[b];
  const long long cap = min(static_cast<long long>(a.kv.max_pages) << a.kv.page_shift, kMaxPagedRows);
  if (L < 0 || static_cast<long long>(L) + (last - first) > cap) {
    set_device_status(a.status, MEDUSA_ERR_DEVICE_CHECK, kDetailPagedChunk);
    return pl;
  }
  const long long row = static_cast<long long>(L) + (n - first);
  const int page = a.kv.table[static_cast<long long>(b) * a.kv.max_pages + (row >> a.kv.page_shift)];
  if (page < 0 || page >= a.kv.n_pages) {
    set_device_status(a.status, MEDUSA_ERR_DEVICE_CHECK, kDetailPagedPage);
    return pl;
  }
  pl.base = ((static_cast<long long>(page) * a.kv.Hkv << a.kv.page_shift) + (row & ((1 << a.kv.page_shift) - 1))) * a.kv.hd;
  pl.pos = a.positions ? a.positions[n] : static_cast<int>(row);
  return pl;
}

template <typename T>
struct Vec16;
template <>
struct Vec16<float> {
  static constexpr int kE = 4;
  static __device__ __forceinline__ void unpack(const uint4& w, float* f) {
    f[0] = __uint_as_float(w.x);
    f[1] = __uint_as_float(w.y);
    f[2] = __uint_as_float(w.z);
    f[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};
template <>
struct Vec16<uint16_t> {
  static constexpr int kE = 8;
  static __device__ __forceinline__ void unpack(const uint4& w, float* f) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16lo(u[i]);
      f[2 * i + 1] = bf16hi(u[i]);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
};

template <typename T>
__device__ __forceinline__ float load1(const T* p);
template <>
__device__ __forceinline__ float load1<float>(const float* p) { return *p; }
template <>
__device__ __forceinline__ float load1<uint16_t>(const uint16_t* p) { return __uint_as_float(static_cast<uint32_t>(*p) << 16); }
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }
__device__ __forceinline__ void store1(uint16_t* p, float x) { *p = f32_to_bf16_rne(x); }

// Shared per block: the tokens' places and their cos / sin (times amplitude).
template <typename T>
__device__ int prepare_tokens(const RopeArgs& a, int n0, Place* place, float2* cs) {
  __shared__ int32_t starts[MEDUSA_MAX_B + 1];
  const int tid = threadIdx.x, B = a.kv.B;
  bool none = false;
  if (a.starts) {
    for (int i = tid; i <= B; i += kThreads) starts[i] = a.starts[i];
    __syncthreads();
    if (blockIdx.x == 0 && tid < B && (starts[tid] < 0 || starts[tid + 1] < starts[tid] || starts[tid + 1] > a.N))
      set_device_status(a.status, MEDUSA_ERR_DEVICE_CHECK, kDetailPagedChunk);
    // Chunks that overlap have no one owner of a row: nothing is written, as attention then computes nothing.
    none = __syncthreads_or(tid < B && starts[tid + 1] < starts[tid]) != 0;
  }
  const int count = min(a.tok, a.N - n0);
  if (tid < count) place[tid] = none ? Place{-1, 0} : place_token(a, n0 + tid, a.starts ? starts : nullptr);
  __syncthreads();
  const int pairs = a.rot >> 1;
  for (int x = tid; x < count * pairs; x += kThreads) {
    const int t = x / pairs, i = x - t * pairs;
    const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(place[t].pos)) * a.turns[i];
    float s, c;
    sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f /* 2^-31: half turns */, &s, &c);
    cs[x] = make_float2(c * a.amplitude, s * a.amplitude);
  }
  __syncthreads();
  return count;
}

// 16-byte path: a thread owns vector j of one head (in the half layout also
// its partner rot/2 further on) and walks the block's tokens; the next step's
// loads are in flight while a step is turned and stored (two steps' registers
// take turns; under the six blocks' 40 registers the compiler spills 52 bytes
// of them in bf16).  Narrow models put several tokens side by side, wide ones
// sweep over their heads (one sweep per blockIdx.y when there are few tokens).
template <typename T>
__global__ void __launch_bounds__(kThreads, 6) rope_append_vec(const RopeArgs a) {
  constexpr int E = Vec16<T>::kE;
  extern __shared__ __align__(16) float2 cs[];
  __shared__ Place place[kMaxTok];
  const int n0 = blockIdx.x * a.tok, count = min(a.tok, a.N - n0);
  const int hd = a.kv.hd, H = a.H, Hkv = a.kv.Hkv, pairs = a.rot >> 1;
  const int turned = a.half ? pairs / E : a.rot / E;          // units that rotate
  const int units = turned + (hd - a.rot) / E;
  const int per = kThreads / units, heads = H + 2 * Hkv;      // heads per sweep
  const int i0 = threadIdx.x / units, j = threadIdx.x - i0 * units;
  const int side = per > heads ? per / heads : 1;             // tokens side by side
  const int t0 = side > 1 ? i0 / heads : 0;
  const bool idle = i0 >= per || t0 >= side;
  const bool two = a.half && j < turned;
  const int va = j < turned ? j * E : a.rot + (j - turned) * E;   // element offset of the (first) vector
  struct Step {                                               // a token of one head
    int h, t, kind, hk;                                       // q, k or v, and the head in it
    uint4 x, y;
  };
  auto load = [&](Step& s) {
    s.kind = s.h < H ? 0 : s.h < H + Hkv ? 1 : 2;
    s.hk = s.kind == 0 ? s.h : s.kind == 1 ? s.h - H : s.h - H - Hkv;
    const long long step = s.kind == 0 ? a.qs : s.kind == 1 ? a.ks : a.vs;
    const T* src = static_cast<const T*>(s.kind == 0 ? a.q : s.kind == 1 ? a.k : a.v) + (n0 + s.t) * step + s.hk * hd + va;
    s.x = *reinterpret_cast<const uint4*>(src);
    if (two) s.y = *reinterpret_cast<const uint4*>(src + pairs);
  };
  auto follow = [&](const Step& s, Step& next) {              // false: s was the last
    next.h = s.h;
    next.t = s.t + side;
    if (next.t >= count) {
      next.t = t0;
      next.h += gridDim.y * per;
    }
    return next.h < heads;
  };
  auto finish = [&](Step& s) {
    T* dst = s.kind == 0 ? static_cast<T*>(a.q_out) + (static_cast<long long>(n0) * H + s.hk) * hd + va
                         : static_cast<T*>(s.kind == 1 ? a.kv.k : a.kv.v) + (static_cast<long long>(s.hk) * hd << a.kv.page_shift) + va;
    if (place[s.t].base < 0) return;
    if (j < turned && s.kind < 2) {
      const float2* w = cs + s.t * pairs + (a.half ? va : va >> 1);
      float f[E];
      Vec16<T>::unpack(s.x, f);
      if (two) {
        float g[E];
        Vec16<T>::unpack(s.y, g);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float p = f[e] * w[e].x - g[e] * w[e].y, r = g[e] * w[e].x + f[e] * w[e].y;
          f[e] = p;
          g[e] = r;
        }
        s.y = Vec16<T>::pack(g);
      } else {
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
          const float p = f[2 * e] * w[e].x - f[2 * e + 1] * w[e].y, r = f[2 * e + 1] * w[e].x + f[2 * e] * w[e].y;
          f[2 * e] = p;
          f[2 * e + 1] = r;
        }
      }
      s.x = Vec16<T>::pack(f);
    }
    T* to = dst + (s.kind == 0 ? static_cast<long long>(s.t) * H * hd : place[s.t].base);
    *reinterpret_cast<uint4*>(to) = s.x;
    if (two) *reinterpret_cast<uint4*>(to + pairs) = s.y;
  };
  // The first loads wait for nothing: they run while the places and angles are
  // worked out; later ones run while the step before is turned and stored
  // (every vector is read before it is written, also when q_out is q).
  Step s0, s1;
  s0.h = i0 - t0 * heads + blockIdx.y * per;
  s0.t = t0;
  const bool some = !idle && s0.h < heads && s0.t < count;
  if (some) load(s0);
  prepare_tokens<T>(a, n0, place, cs);
  if (!some) return;
  for (;;) {
    const bool more = follow(s0, s1);
    if (more) load(s1);
    finish(s0);
    if (!more) return;
    const bool again = follow(s1, s0);
    if (again) load(s0);
    finish(s1);
    if (!again) return;
  }
}

// Element path, for rotated parts that 16-byte vectors do not divide.
template <typename T>
__global__ void __launch_bounds__(kThreads) rope_append_any(const RopeArgs a) {
  extern __shared__ float2 cs[];
  __shared__ Place place[kMaxTok];
  const int n0 = blockIdx.x * a.tok;
  const int count = prepare_tokens<T>(a, n0, place, cs);
  const int hd = a.kv.hd, H = a.H, Hkv = a.kv.Hkv, pairs = a.rot >> 1;
  const int units = pairs + hd - a.rot;                        // pairs, then single elements
  const long long page_head = static_cast<long long>(hd) << a.kv.page_shift;
  for (int t = 0; t < count; ++t) {
    const long long base = place[t].base;
    if (base < 0) continue;
    const long long n = n0 + t;
    for (int x = threadIdx.x; x < (H + 2 * Hkv) * units; x += kThreads) {
      const int h = x / units, j = x - h * units;
      const T* src = h < H ? static_cast<const T*>(a.q) + n * a.qs + static_cast<long long>(h) * hd
                     : h < H + Hkv ? static_cast<const T*>(a.k) + n * a.ks + static_cast<long long>(h - H) * hd
                                   : static_cast<const T*>(a.v) + n * a.vs + static_cast<long long>(h - H - Hkv) * hd;
      T* dst = h < H ? static_cast<T*>(a.q_out) + (n * H + h) * hd
               : h < H + Hkv ? static_cast<T*>(a.kv.k) + base + (h - H) * page_head
                             : static_cast<T*>(a.kv.v) + base + (h - H - Hkv) * page_head;
      if (j >= pairs) {
        dst[a.rot + j - pairs] = src[a.rot + j - pairs];
        continue;
      }
      const int ia = a.half ? j : 2 * j, ib = a.half ? j + pairs : 2 * j + 1;
      if (h >= H + Hkv) {
        dst[ia] = src[ia];
        dst[ib] = src[ib];
        continue;
      }
      const float f = load1<T>(src + ia), g = load1<T>(src + ib);
      const float2 w = cs[t * pairs + j];
      store1(dst + ia, f * w.x - g * w.y);
      store1(dst + ib, g * w.x + f * w.y);
    }
  }
}

}  // namespace

medusa_status_t launch_rope_append(const PagedDev& kv, medusa_dtype_t dtype, int N, int H, const void* q,
                                   int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                                   void* q_out, const medusa_rotary_t& rotary, const int32_t* positions,
                                   const int32_t* starts, cudaStream_t stream) {
  RopeArgs a{};
  a.kv = kv;
  a.N = N;
  a.H = H;
  a.rot = rotary.rot;
  a.half = rotary.layout == MEDUSA_ROPE_HALF;
  a.q = q;
  a.k = k;
  a.v = v;
  a.qs = q_stride;
  a.ks = k_stride;
  a.vs = v_stride;
  a.q_out = q_out;
  a.turns = rotary.turns;
  a.amplitude = rotary.amplitude;
  a.positions = positions;
  a.starts = starts;
  a.status = device_status_ptr();
  // Tokens per block: as many as give every SM its six blocks once (a second
  // wave that is not full left a quarter of the SMs' time unused), up to 32.
  const int es = dtype == MEDUSA_BF16 ? 2 : 4, slots = 6 * sm_count();
  a.tok = (N + slots - 1) / slots < kMaxTok ? (N + slots - 1) / slots : kMaxTok;
  const int grid = (N + a.tok - 1) / a.tok;
  const size_t smem = static_cast<size_t>(a.tok) * (a.rot / 2) * sizeof(float2);   // at most 32 KB
  const int E = 16 / es;
  const bool vec = (a.half ? a.rot / 2 : a.rot) % E == 0;
  const int turned = a.half ? a.rot / 2 / E : a.rot / E, per = vec ? kThreads / (turned + (kv.hd - a.rot) / E) : 1;
  // Up to two tokens per SM: a block of its own for every sweep over the heads (one token of 64 + 2 x 8 heads
  // 3.6 us, one block 4.9; 64 of 32 + 2 x 32 4.0, 5.1).  With more, every block would set up its tokens again for
  // each (400 of 32 + 2 x 32 6.7 us, with them 7.1).
  const int sweeps = N <= 2 * sm_count() ? (H + 2 * kv.Hkv + per - 1) / per : 1;
  if (dtype == MEDUSA_BF16) {
    if (vec) rope_append_vec<uint16_t><<<dim3(grid, sweeps), kThreads, smem, stream>>>(a);
    else rope_append_any<uint16_t><<<grid, kThreads, smem, stream>>>(a);
  } else {
    if (vec) rope_append_vec<float><<<dim3(grid, sweeps), kThreads, smem, stream>>>(a);
    else rope_append_any<float><<<grid, kThreads, smem, stream>>>(a);
  }
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? MEDUSA_OK : cuda_fail("medusa_rope_append", e);
}

}  // namespace medusa
