// The C ABI of the paged-cache calls and of the logit adjustment: argument
// checks on the host before any launch, and the table of rotary frequencies.
#include <atomic>
#include <cmath>
#include <string>

#include "common.cuh"

namespace medusa {
namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int kMaxTokens = 1 << 22;   // packed rows of a call: row * heads stays inside 32 bits
constexpr int kMaxHeads = 256;
constexpr float kMaxScale = 18446744073709551616.f;   // 2^64: scale * log2(e) stays finite
constexpr int kMaxVocab = 1 << 30;    // a chunk's end stays inside 31 bits

medusa_status_t check_kv(const medusa_paged_kv_t* kv, const char* fn) {
  const std::string f(fn);
  if (!kv) return fail(MEDUSA_ERR_INVALID_ARG, f + ": kv is null");
  if (!kv->k_pages || !kv->v_pages || !kv->page_table || !kv->seq_lens)
    return fail(MEDUSA_ERR_INVALID_ARG, f + ": null cache pointer");
  if (kv->dtype != MEDUSA_BF16 && kv->dtype != MEDUSA_F32) return fail(MEDUSA_ERR_UNSUPPORTED, f + ": dtype");
  if (kv->layers < 1 || kv->n_pages < 1 || kv->Hkv < 1 || kv->Hkv > kMaxHeads || kv->max_pages < 1 || kv->B < 1 ||
      kv->B > MEDUSA_MAX_B)
    return fail(MEDUSA_ERR_INVALID_ARG, f + ": layers, n_pages, Hkv, max_pages or B out of range");
  if (kv->page < 8 || kv->page > 256 || (kv->page & (kv->page - 1)) != 0)
    return fail(MEDUSA_ERR_UNSUPPORTED, f + ": page must be a power of two in [8, 256]");
  if (kv->hd < 8 || kv->hd > 256 || kv->hd % 8 != 0)
    return fail(MEDUSA_ERR_UNSUPPORTED, f + ": hd must be a multiple of 8 in [8, 256]");
  if (!aligned(kv->k_pages, 16) || !aligned(kv->v_pages, 16) || !aligned(kv->page_table, 4) ||
      !aligned(kv->seq_lens, 4))
    return fail(MEDUSA_ERR_INVALID_ARG, f + ": misaligned cache pointer");
  return MEDUSA_OK;
}

int element_bytes(medusa_dtype_t t) { return t == MEDUSA_BF16 ? 2 : 4; }

// Sequences hold at most kMaxPagedRows rows; a longer table's tail is never used.
PagedDev device_view(const medusa_paged_kv_t* kv, int layer) {
  PagedDev d{};
  d.n_pages = kv->n_pages;
  d.Hkv = kv->Hkv;
  while ((1 << d.page_shift) < kv->page) ++d.page_shift;
  d.hd = kv->hd;
  d.B = kv->B;
  d.max_pages = kv->max_pages;
  d.table = kv->page_table;
  d.lens = kv->seq_lens;
  const size_t off = static_cast<size_t>(layer) * kv->n_pages * kv->Hkv * kv->page * kv->hd * element_bytes(kv->dtype);
  d.k = static_cast<unsigned char*>(kv->k_pages) + off;
  d.v = static_cast<unsigned char*>(kv->v_pages) + off;
  return d;
}

medusa_status_t check_tokens(const medusa_paged_kv_t* kv, int layer, int N, int H, const int32_t* starts,
                             const char* fn) {
  const std::string f(fn);
  if (layer < 0 || layer >= kv->layers) return fail(MEDUSA_ERR_INVALID_ARG, f + ": layer out of range");
  if (N < 1 || N > kMaxTokens) return fail(MEDUSA_ERR_INVALID_ARG, f + ": N out of range");
  if (H < 1 || H > kMaxHeads) return fail(MEDUSA_ERR_INVALID_ARG, f + ": H out of range");
  if (!starts && N % kv->B != 0)
    return fail(MEDUSA_ERR_INVALID_ARG, f + ": without chunk_starts N must be a multiple of B");
  if (!aligned(starts, 4)) return fail(MEDUSA_ERR_INVALID_ARG, f + ": misaligned chunk_starts");
  return MEDUSA_OK;
}

bool overlap(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + bn && y < x + an;
}

// Whether [a, a + an) holds a byte of the cache's pages.
bool in_pages(const medusa_paged_kv_t* kv, const void* a, size_t an) {
  const size_t bytes = static_cast<size_t>(kv->layers) * kv->n_pages * kv->Hkv * kv->page * kv->hd * element_bytes(kv->dtype);
  return overlap(a, an, kv->k_pages, bytes) || overlap(a, an, kv->v_pages, bytes);
}

std::atomic<unsigned> g_test_extra{0};
std::atomic<unsigned long long> g_test_limit_ns{0};

}  // namespace

PagedWait paged_wait() {
  const unsigned long long lim = g_test_limit_ns.load();
  return {g_test_extra.load(), lim ? lim : kSpinLimitNs};
}

}  // namespace medusa

using namespace medusa;

extern "C" medusa_status_t medusa_test_paged_wait(int extra_arrivals, long long limit_ns) {
  if (extra_arrivals < 0 || extra_arrivals > 1024 || limit_ns < 0)
    return fail(MEDUSA_ERR_INVALID_ARG, "medusa_test_paged_wait: extra_arrivals in [0, 1024], limit_ns >= 0");
  g_test_extra.store(static_cast<unsigned>(extra_arrivals));
  g_test_limit_ns.store(static_cast<unsigned long long>(limit_ns));
  return MEDUSA_OK;
}

extern "C" medusa_status_t medusa_rotary_turns(int rot, double base, medusa_rope_scaling_t scaling, double factor,
                                               int original_length, double beta_fast, double beta_slow,
                                               uint64_t* turns, float* amplitude) {
  const std::string f("medusa_rotary_turns");
  if (!turns || !amplitude) return fail(MEDUSA_ERR_INVALID_ARG, f + ": null pointer");
  if (rot < 2 || rot > 256 || rot % 2 != 0) return fail(MEDUSA_ERR_INVALID_ARG, f + ": rot must be even, in [2, 256]");
  if (!(base > 1.0) || !std::isfinite(base)) return fail(MEDUSA_ERR_INVALID_ARG, f + ": base must exceed 1");
  if (scaling != MEDUSA_ROPE_NONE && scaling != MEDUSA_ROPE_LINEAR && scaling != MEDUSA_ROPE_NTK &&
      scaling != MEDUSA_ROPE_YARN)
    return fail(MEDUSA_ERR_INVALID_ARG, f + ": scaling");
  if (!(factor >= 1.0) || !std::isfinite(factor)) return fail(MEDUSA_ERR_INVALID_ARG, f + ": factor must be at least 1");
  if (scaling == MEDUSA_ROPE_NTK && rot < 4) return fail(MEDUSA_ERR_INVALID_ARG, f + ": NTK scaling needs rot >= 4");
  if (scaling == MEDUSA_ROPE_YARN && (original_length < 1 || !(beta_slow > 0.0) || !(beta_fast > beta_slow) ||
                                      !std::isfinite(beta_fast)))
    return fail(MEDUSA_ERR_INVALID_ARG, f + ": YARN needs original_length >= 1 and beta_fast > beta_slow > 0");
  const double two_pi = 6.283185307179586476925286766559;
  double b = base, amp = 1.0, lo = 0.0, hi = 0.0;
  if (scaling == MEDUSA_ROPE_NTK) b = base * std::pow(factor, static_cast<double>(rot) / (rot - 2));
  if (scaling == MEDUSA_ROPE_YARN) {
    // The pair index at which a pair makes `beta` turns over the original
    // length: original_length * base^(-2 i / rot) = 2 pi beta.
    const auto at = [&](double beta) { return rot * std::log(original_length / (beta * two_pi)) / (2.0 * std::log(base)); };
    lo = std::fmax(std::floor(at(beta_fast)), 0.0);
    hi = std::fmin(std::ceil(at(beta_slow)), rot - 1.0);
    amp = 0.1 * std::log(factor) + 1.0;
  }
  for (int i = 0; i < rot / 2; ++i) {
    double w = std::pow(b, -2.0 * i / rot);
    if (scaling == MEDUSA_ROPE_LINEAR) w /= factor;
    if (scaling == MEDUSA_ROPE_YARN) {
      const double ramp = std::fmin(std::fmax((i - lo) / std::fmax(hi - lo, 0.001), 0.0), 1.0);
      w = w / factor * ramp + w * (1.0 - ramp);
    }
    turns[i] = static_cast<uint64_t>(std::ldexp(w / two_pi, 64));   // w <= 1, so below 2^62
  }
  *amplitude = static_cast<float>(amp);
  return MEDUSA_OK;
}

extern "C" medusa_status_t medusa_rope_append(const medusa_paged_kv_t* kv, int layer, int N, int H, const void* q,
                                              int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                              int64_t v_stride, void* q_out, const medusa_rotary_t* rotary,
                                              const int32_t* positions, const int32_t* chunk_starts,
                                              cudaStream_t stream) {
  const char* fn = "medusa_rope_append";
  const std::string f(fn);
  medusa_status_t st = check_kv(kv, fn);
  if (st == MEDUSA_OK) st = check_tokens(kv, layer, N, H, chunk_starts, fn);
  if (st != MEDUSA_OK) return st;
  if (!q || !k || !v || !q_out || !rotary || !rotary->turns) return fail(MEDUSA_ERR_INVALID_ARG, f + ": null pointer");
  if (rotary->layout != MEDUSA_ROPE_HALF && rotary->layout != MEDUSA_ROPE_INTERLEAVED)
    return fail(MEDUSA_ERR_INVALID_ARG, f + ": layout");
  if (rotary->rot < 2 || rotary->rot > kv->hd || rotary->rot % 2 != 0)
    return fail(MEDUSA_ERR_INVALID_ARG, f + ": rot must be even, in [2, hd]");
  if (!std::isfinite(rotary->amplitude)) return fail(MEDUSA_ERR_INVALID_ARG, f + ": amplitude must be finite");
  const int es = element_bytes(kv->dtype);
  const int64_t qw = static_cast<int64_t>(H) * kv->hd, kw = static_cast<int64_t>(kv->Hkv) * kv->hd;
  const int64_t most = int64_t(1) << 31;
  if (q_stride < qw || k_stride < kw || v_stride < kw || q_stride > most || k_stride > most || v_stride > most)
    return fail(MEDUSA_ERR_INVALID_ARG, f + ": a token stride is smaller than the token's heads, or too large");
  if (q_stride * es % 16 || k_stride * es % 16 || v_stride * es % 16)
    return fail(MEDUSA_ERR_UNSUPPORTED, f + ": token strides must be multiples of 16 bytes");
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) || !aligned(rotary->turns, 8) ||
      !aligned(positions, 4))
    return fail(MEDUSA_ERR_INVALID_ARG, f + ": misaligned pointer");
  const size_t span_q = (static_cast<size_t>(N - 1) * q_stride + qw) * es, out_bytes = static_cast<size_t>(N) * qw * es;
  const size_t span_k = (static_cast<size_t>(N - 1) * k_stride + kw) * es, span_v = (static_cast<size_t>(N - 1) * v_stride + kw) * es;
  if (q_out == q ? q_stride != qw : overlap(q, span_q, q_out, out_bytes))
    return fail(MEDUSA_ERR_INVALID_ARG, f + ": q_out may be q itself when q is contiguous, and must not overlap it otherwise");
  if (overlap(k, span_k, q_out, out_bytes) || overlap(v, span_v, q_out, out_bytes))
    return fail(MEDUSA_ERR_INVALID_ARG, f + ": q_out overlaps k or v");
  if (in_pages(kv, q_out, out_bytes) || in_pages(kv, q, span_q) || in_pages(kv, k, span_k) || in_pages(kv, v, span_v))
    return fail(MEDUSA_ERR_INVALID_ARG, f + ": q, k, v or q_out overlaps the pages");
  if (sm_count() <= 0) return fail(MEDUSA_ERR_CUDA, f + ": no usable CUDA device");
  return launch_rope_append(device_view(kv, layer), kv->dtype, N, H, q, q_stride, k, k_stride, v, v_stride, q_out,
                            *rotary, positions, chunk_starts, stream);
}

extern "C" size_t medusa_paged_attention_workspace_size(const medusa_paged_kv_t* kv, int N, int H) {
  if (check_kv(kv, "medusa_paged_attention_workspace_size") != MEDUSA_OK || N < 1 || N > kMaxTokens || H < 1 ||
      H > kMaxHeads || H % kv->Hkv != 0 || sm_count() <= 0)
    return 0;
  return paged_attention_workspace_bytes(device_view(kv, 0), kv->dtype, N, H);
}

extern "C" medusa_status_t medusa_paged_attention(const medusa_paged_kv_t* kv, int layer, int N, int H, const void* q,
                                                  float scale, const medusa_tree_t* tree, const int32_t* chunk_starts,
                                                  void* out, void* workspace, size_t workspace_bytes,
                                                  cudaStream_t stream) {
  const char* fn = "medusa_paged_attention";
  const std::string f(fn);
  medusa_status_t st = check_kv(kv, fn);
  if (st == MEDUSA_OK) st = check_tokens(kv, layer, N, H, chunk_starts, fn);
  if (st != MEDUSA_OK) return st;
  if (!q || !out || !workspace) return fail(MEDUSA_ERR_INVALID_ARG, f + ": null pointer");
  if (H % kv->Hkv != 0) return fail(MEDUSA_ERR_INVALID_ARG, f + ": H must be a multiple of Hkv");
  if (!(std::fabs(scale) <= kMaxScale)) return fail(MEDUSA_ERR_INVALID_ARG, f + ": |scale| must be at most 2^64");
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 256))
    return fail(MEDUSA_ERR_INVALID_ARG, f + ": misaligned pointer");
  const size_t bytes = static_cast<size_t>(N) * H * kv->hd * element_bytes(kv->dtype);
  if (overlap(q, bytes, out, bytes)) return fail(MEDUSA_ERR_INVALID_ARG, f + ": out overlaps q");
  if (in_pages(kv, out, bytes)) return fail(MEDUSA_ERR_INVALID_ARG, f + ": out overlaps the pages");
  if (tree) {
    st = check_tree(tree, fn);
    if (st != MEDUSA_OK) return st;
    if (chunk_starts || N != kv->B * tree->T)
      return fail(MEDUSA_ERR_INVALID_ARG, f + ": with a tree N must be B * T and chunk_starts NULL");
  }
  if (sm_count() <= 0) return fail(MEDUSA_ERR_CUDA, f + ": no usable CUDA device");
  const PagedDev d = device_view(kv, layer);
  if (workspace_bytes < paged_attention_workspace_bytes(d, kv->dtype, N, H))
    return fail(MEDUSA_ERR_INVALID_ARG, f + ": workspace too small");
  return launch_paged_attention(d, kv->dtype, N, H, q, scale, tree ? &tree->dev : nullptr, chunk_starts, out,
                                workspace, stream);
}

extern "C" size_t medusa_paged_accept_workspace_size(const medusa_paged_kv_t* kv) {
  return check_kv(kv, "medusa_paged_accept_workspace_size") == MEDUSA_OK ? 256 : 0;
}

extern "C" medusa_status_t medusa_paged_accept_kv(const medusa_tree_t* tree, const medusa_paged_kv_t* kv,
                                                  const int32_t* best_path, const int32_t* accept_len,
                                                  int32_t* new_lens, void* workspace, size_t workspace_bytes,
                                                  cudaStream_t stream) {
  const char* fn = "medusa_paged_accept_kv";
  const std::string f(fn);
  medusa_status_t st = check_kv(kv, fn);
  if (st != MEDUSA_OK) return st;
  if (!best_path || !accept_len || !new_lens || !workspace)
    return fail(MEDUSA_ERR_INVALID_ARG, f + ": null pointer");
  if (!aligned(best_path, 4) || !aligned(accept_len, 4) || !aligned(new_lens, 4) || !aligned(workspace, 256))
    return fail(MEDUSA_ERR_INVALID_ARG, f + ": misaligned pointer");
  const size_t n = static_cast<size_t>(kv->B) * sizeof(int32_t);
  if ((new_lens != kv->seq_lens && overlap(new_lens, n, kv->seq_lens, n)) || overlap(new_lens, n, best_path, n) ||
      overlap(new_lens, n, accept_len, n))
    return fail(MEDUSA_ERR_INVALID_ARG, f + ": new_lens overlaps an input other than seq_lens as a whole");
  if (workspace_bytes < medusa_paged_accept_workspace_size(kv))
    return fail(MEDUSA_ERR_INVALID_ARG, f + ": workspace too small");
  if (kv->layers > 65535) return fail(MEDUSA_ERR_UNSUPPORTED, f + ": more than 65535 layers");
  st = check_tree(tree, fn);
  if (st != MEDUSA_OK) return st;
  return launch_paged_accept(tree->dev, device_view(kv, 0), kv->layers, kv->dtype, best_path, accept_len, new_lens,
                             workspace, stream);
}

extern "C" medusa_status_t medusa_adjust_logits(const medusa_tree_t* tree, int B, int V, const float* logits,
                                                const int32_t* tree_tokens, const medusa_logit_rules_t* rules,
                                                float* out, cudaStream_t stream) {
  const char* fn = "medusa_adjust_logits";
  const std::string f(fn);
  if (!logits || !out || !rules) return fail(MEDUSA_ERR_INVALID_ARG, f + ": null pointer");
  if (B < 1 || B > MEDUSA_MAX_B || V < 1 || V > kMaxVocab) return fail(MEDUSA_ERR_INVALID_ARG, f + ": B or V");
  const medusa_logit_rules_t& r = *rules;
  if ((r.history != nullptr) != (r.history_lens != nullptr) || (r.history && r.history_cap < 1) ||
      (r.prompt_lens && !r.history))
    return fail(MEDUSA_ERR_INVALID_ARG, f + ": history needs history_lens and history_cap >= 1, and prompt_lens a history");
  if ((r.bias_ids != nullptr) != (r.bias != nullptr) || (r.bias && (r.n_bias < 1 || r.n_bias > MEDUSA_MAX_BIAS)))
    return fail(MEDUSA_ERR_INVALID_ARG, f + ": bias_ids and bias go together, with 1 <= n_bias <= MEDUSA_MAX_BIAS");
  if ((r.repetition || r.presence || r.frequency) && !tree_tokens)
    return fail(MEDUSA_ERR_INVALID_ARG, f + ": the penalties need tree_tokens");
  if (!aligned(logits, 4) || !aligned(out, 4) || !aligned(tree_tokens, 4) || !aligned(r.history, 4) ||
      !aligned(r.history_lens, 4) || !aligned(r.prompt_lens, 4) || !aligned(r.repetition, 4) ||
      !aligned(r.presence, 4) || !aligned(r.frequency, 4) || !aligned(r.bias_ids, 4) || !aligned(r.bias, 4) ||
      !aligned(r.allowed, 4))
    return fail(MEDUSA_ERR_INVALID_ARG, f + ": misaligned pointer");
  const medusa_status_t st = check_tree(tree, fn);
  if (st != MEDUSA_OK) return st;
  const size_t n = static_cast<size_t>(B) * tree->T * V * sizeof(float);
  if (out != logits && overlap(out, n, logits, n))
    return fail(MEDUSA_ERR_INVALID_ARG, f + ": out may be logits itself, and must not overlap it otherwise");
  return launch_adjust_logits(tree->dev, B, V, logits, tree_tokens, r, out, stream);
}
