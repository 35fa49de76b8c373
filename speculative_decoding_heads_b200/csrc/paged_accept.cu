// The accepted path's rows moved to the end of the cached prefix inside the
// pages: row L + j <- row L + n_j for j = 0..a, every layer and head, K and V.
// A source can be the destination of a later j, so each thread owns one
// 16-byte column of one head's K or V rows and loads all its sources before it
// writes any (row 0 is the root and stays).  A block first looks up the path's
// page offsets once, with one thread per accepted row.
//
// Bound by the latency of these dependent reads, so by how many threads are in
// flight: the registers are those of the tree's own depth (4, 8 or 16 rows).
// 8 sequences of 40 layers of 40 heads of 128 take 7.1 us, 4.6 TB/s (16 rows
// for every tree 15.0), one of 32 layers 2.6 us.
//
// new_lens may be the lengths that the blocks read: then the last block to
// finish (a ticket in the workspace) writes it.
#include "common.cuh"

namespace medusa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxRows = MEDUSA_MAX_K + 1;   // a <= D <= K

struct AcceptArgs {
  TreeDev t;
  PagedDev kv;
  int chunks;                  // 16-byte columns per row
  long long layer_stride;      // columns per layer
  const int32_t* best_path;
  const int32_t* accept_len;
  int32_t* new_lens;
  unsigned* ticket;            // null: new_lens is not read here
  int* status;
};

// a, or -1 when sequence b's path or lengths are not usable.
__device__ __forceinline__ int accepted(const AcceptArgs& a, int b, int* L, int* best) {
  *L = a.kv.lens[b];
  *best = a.best_path[b];
  const int n = a.accept_len[b];
  const long long cap = min(static_cast<long long>(a.kv.max_pages) << a.kv.page_shift, kMaxPagedRows);
  if (*L < 0 || n < 0 || n > a.t.D || *best < 0 || *best >= a.t.P || static_cast<long long>(*L) + a.t.T > cap) return -1;
  return a.t.retrieve[*best * (a.t.D + 1) + n] < 0 ? -1 : n;
}

// kRows: accepted rows below the root that a thread can hold.
template <int kRows>
__global__ void __launch_bounds__(kThreads) paged_accept_kernel(const AcceptArgs a) {
  __shared__ long long from[kMaxRows], to[kMaxRows];   // column offset of head 0, from < 0: nothing to move
  __shared__ int s_n;
  const int b = blockIdx.y, layer = blockIdx.z, tid = threadIdx.x;
  if (tid < 32) {
    int L, best;
    int n = accepted(a, b, &L, &best);
    int bad = 0;
    if (n >= 0 && tid <= n) {
      const int node = a.t.retrieve[best * (a.t.D + 1) + tid];
      const int32_t* table = a.kv.table + static_cast<long long>(b) * a.kv.max_pages;
      const int shift = a.kv.page_shift, mask = (1 << shift) - 1;
      const long long src = static_cast<long long>(L) + node, dst = static_cast<long long>(L) + tid;
      const int ps = table[src >> shift], pd = table[dst >> shift];
      bad = ps < 0 || ps >= a.kv.n_pages || pd < 0 || pd >= a.kv.n_pages;
      from[tid] = node == tid ? -1 : ((static_cast<long long>(ps) * a.kv.Hkv << shift) + (src & mask)) * a.chunks;
      to[tid] = ((static_cast<long long>(pd) * a.kv.Hkv << shift) + (dst & mask)) * a.chunks;
    }
    bad = __any_sync(0xffffffffu, bad);
    if (tid == 0) {
      if (n < 0) set_device_status(a.status, MEDUSA_ERR_DEVICE_CHECK, kDetailPagedAccept);
      if (bad) set_device_status(a.status, MEDUSA_ERR_DEVICE_CHECK, kDetailPagedPage);
      s_n = bad ? -1 : n;
      if (!a.ticket && blockIdx.x == 0 && layer == 0 && s_n >= 0) a.new_lens[b] = L + n + 1;
    }
  }
  __syncthreads();
  const int n = s_n;
  const int col = blockIdx.x * kThreads + tid;
  const int per = a.kv.Hkv * a.chunks;
  if (n >= 0 && col < 2 * per) {
    const int which = col >= per, rem = col - which * per;
    const int h = rem / a.chunks, c = rem - h * a.chunks;
    uint4* base = static_cast<uint4*>(which ? a.kv.v : a.kv.k) + layer * a.layer_stride +
                  (static_cast<long long>(h) << a.kv.page_shift) * a.chunks + c;
    uint4 r[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j)
      if (j < n && from[j + 1] >= 0) r[j] = base[from[j + 1]];
#pragma unroll
    for (int j = 0; j < kRows; ++j)
      if (j < n && from[j + 1] >= 0) base[to[j + 1]] = r[j];
  }
  if (a.ticket) {
    __shared__ unsigned s_last;
    __syncthreads();          // this block has read the lengths
    if (tid == 0) s_last = atom_add_acq_rel_gpu(a.ticket, 1u) == gridDim.x * gridDim.y * gridDim.z - 1u;
    __syncthreads();
    if (s_last) {
      // The same checks again: a sequence whose rows stayed keeps its length.
      for (int s = tid; s < a.kv.B; s += kThreads) {
        int L, best;
        const int m = accepted(a, s, &L, &best);
        bool ok = m >= 0;
        for (int j = 0; ok && j <= m; ++j) {
          const int32_t* table = a.kv.table + static_cast<long long>(s) * a.kv.max_pages;
          const int ps = table[(static_cast<long long>(L) + a.t.retrieve[best * (a.t.D + 1) + j]) >> a.kv.page_shift];
          const int pd = table[(static_cast<long long>(L) + j) >> a.kv.page_shift];
          ok = ps >= 0 && ps < a.kv.n_pages && pd >= 0 && pd < a.kv.n_pages;
        }
        if (ok) a.new_lens[s] = L + m + 1;
      }
      if (tid == 0) *a.ticket = 0u;
    }
  }
}

}  // namespace

medusa_status_t launch_paged_accept(const TreeDev& t, const PagedDev& kv, int layers, medusa_dtype_t dtype,
                                    const int32_t* best_path, const int32_t* accept_len, int32_t* new_lens, void* ws,
                                    cudaStream_t stream) {
  AcceptArgs a{};
  a.t = t;
  a.kv = kv;
  a.chunks = kv.hd * (dtype == MEDUSA_BF16 ? 2 : 4) / 16;
  a.layer_stride = (static_cast<long long>(kv.n_pages) * kv.Hkv << kv.page_shift) * a.chunks;
  a.best_path = best_path;
  a.accept_len = accept_len;
  a.new_lens = new_lens;
  a.ticket = new_lens == kv.lens ? static_cast<unsigned*>(ws) : nullptr;
  a.status = device_status_ptr();
  const dim3 grid((2 * kv.Hkv * a.chunks + kThreads - 1) / kThreads, kv.B, layers);
  if (t.D <= 4) paged_accept_kernel<4><<<grid, kThreads, 0, stream>>>(a);
  else if (t.D <= 8) paged_accept_kernel<8><<<grid, kThreads, 0, stream>>>(a);
  else paged_accept_kernel<16><<<grid, kThreads, 0, stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? MEDUSA_OK : cuda_fail("medusa_paged_accept_kv", e);
}

}  // namespace medusa
