// C ABI of the calls ahead of a step's attention: block tables and slots from the requests'
// lengths, and the norm of queries and keys with their rotation.  See include/csattn.h for the
// contract of every entry point.
#include <cmath>
#include <cstring>

#include "csattn.h"
#include "internal.h"
#include "places.h"

namespace csattn {
namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

struct Span {
  uintptr_t begin, end;
  Span(const void* p, size_t bytes)
      : begin(reinterpret_cast<uintptr_t>(p)), end(reinterpret_cast<uintptr_t>(p) + bytes) {}
  bool meets(const Span& o) const { return begin < o.end && o.begin < end; }
};

// theta_p * 2 / pi, theta_p = base^(-2p/d), as float hi + lo; a thread keeps its last table.
void turns_of(float base, int d, RopeTable* out) {
  static thread_local struct {
    int d = 0;
    float base = 0.f;
    RopeTable table;
  } last;
  if (last.d != d || last.base != base) {
    std::memset(&last.table, 0, sizeof(last.table));
    for (int p = 0; p < d / 2; ++p) {
      const double th = std::pow(static_cast<double>(base), -2.0 * p / d) * 0.63661977236758134308;
      last.table.hi[p] = static_cast<float>(th);
      last.table.lo[p] = static_cast<float>(th - static_cast<double>(last.table.hi[p]));
    }
    last.d = d;
    last.base = base;
  }
  *out = last.table;
}

int check_stride(const char* fn, long long s, int extent, int size) {
  if (extent > 1 && (s < 0 || s * size % 16 != 0 || s >= (1LL << 40)))
    return api_fail(CSATTN_ERR_INVALID_ARG,
                    "%s: a stride of %lld elements is not a multiple of 16 bytes", fn, s);
  return CSATTN_OK;
}

// strides: of the batch, the heads and the tokens (null: [B, H, T, d] dense)
int set_strides(const char* fn, const int64_t* strides, int B, int H, int T, int d, int size,
                long long* batch, long long* head, long long* token) {
  *batch = strides != nullptr ? strides[0] : static_cast<long long>(H) * T * d;
  *head = strides != nullptr ? strides[1] : static_cast<long long>(T) * d;
  *token = strides != nullptr ? strides[2] : d;
  int rc = check_stride(fn, *batch, B, size);
  if (rc == CSATTN_OK) rc = check_stride(fn, *head, H, size);
  if (rc == CSATTN_OK) rc = check_stride(fn, *token, T, size);
  return rc;
}

// Nothing that a call writes may lie on what it reads or writes besides.
int check_apart(const char* fn, const Places* written, int nw, const Places* read, int nr) {
  for (int i = 0; i < nw; ++i) {
    for (int j = 0; j < nr; ++j)
      if (share_a_place(written[i], read[j]))
        return api_fail(CSATTN_ERR_INVALID_ARG, "%s: an output overlaps an input", fn);
    for (int j = 0; j < i; ++j)
      if (share_a_place(written[i], written[j]))
        return api_fail(CSATTN_ERR_INVALID_ARG, "%s: two outputs overlap", fn);
  }
  return CSATTN_OK;
}

// What both directions of the norm are given; *a receives it.
int norm_args(const char* fn, QkNormArgs* a, const void* q, const void* k, const void* q_weight,
              const void* k_weight, const int32_t* positions, const void* q_out, const void* k_out,
              int B, int Hq, int Hkv, int T, int d, int dtype, const int64_t* strides, int pos0,
              int norm, float eps, float rope_base, int rope_layout) {
  if (q == nullptr || k == nullptr || q_out == nullptr || k_out == nullptr)
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: null pointer argument", fn);
  for (const void* p : {q, k, q_weight, k_weight, q_out, k_out})
    if (!aligned(p, 16)) return api_fail(CSATTN_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
  if (!aligned(positions, 4))
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
  if (B < 1 || Hq < 1 || Hkv < 1 || T < 1)
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: B=%d Hq=%d Hkv=%d T=%d must be >= 1", fn, B, Hq,
                    Hkv, T);
  if (dtype != CSATTN_BF16 && dtype != CSATTN_F32)
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: dtype %d is not bf16 or fp32", fn, dtype);
  const bool wide = d == 64 || d == 128;
  if (!wide && !(dtype == CSATTN_F32 && (d == 16 || d == 32)))
    return api_fail(CSATTN_ERR_UNSUPPORTED, "%s: d=%d not in {64,128} (fp32: {16,32,64,128})", fn,
                    d);
  for (const long long h : {static_cast<long long>(Hq), static_cast<long long>(Hkv)})
    if (B > (1 << 24) || T >= (1 << 24) || h > (1 << 20) ||
        static_cast<double>(B) * h * T * d >= 8589934592.0)  // 2^33
      return api_fail(CSATTN_ERR_UNSUPPORTED, "%s: B * heads * T * d too large", fn);
  if (norm != 0 && norm != 1)
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: norm=%d is not 0 or 1", fn, norm);
  if (norm == 0 && (q_weight != nullptr || k_weight != nullptr))
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: gains without the norm", fn);
  if (!(eps >= 0.f) || !std::isfinite(eps))
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: eps must be finite and not negative", fn);
  if (rope_layout != CSATTN_ROPE_SPLIT_HALF && rope_layout != CSATTN_ROPE_ADJACENT)
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: unknown rope_layout %d", fn, rope_layout);
  if (!std::isfinite(rope_base))
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: rope_base must be finite", fn);
  if (rope_base > 0.f && rope_base < 1.f)
    return api_fail(CSATTN_ERR_UNSUPPORTED, "%s: rope_base=%g below 1", fn, rope_base);
  if (pos0 < 0 || (rope_base > 0.f && pos0 > (1 << 24) - T))
    return api_fail(pos0 < 0 ? CSATTN_ERR_INVALID_ARG : CSATTN_ERR_UNSUPPORTED,
                    "%s: positions %d.. not in [0, 2^24)", fn, pos0);
  const int size = dtype == CSATTN_BF16 ? 2 : 4;
  int rc = set_strides(fn, strides, B, Hq, T, d, size, &a->q.batch, &a->q.head, &a->q.token);
  if (rc != CSATTN_OK) return rc;
  rc = set_strides(fn, strides != nullptr ? strides + 3 : nullptr, B, Hkv, T, d, size, &a->k.batch,
                   &a->k.head, &a->k.token);
  if (rc != CSATTN_OK) return rc;
  a->q.x = q;
  a->k.x = k;
  a->q.w = q_weight;
  a->k.w = k_weight;
  a->q.H = Hq;
  a->k.H = Hkv;
  a->positions = positions;
  a->B = B;
  a->T = T;
  a->d = d;
  a->pos0 = pos0;
  a->norm = norm;
  a->eps = eps;
  a->rope = 0;
  if (rope_base > 0.f) {
    a->rope = rope_layout == CSATTN_ROPE_SPLIT_HALF ? 1 : 2;
    turns_of(rope_base, d, &a->turns);
  }
  return CSATTN_OK;
}

}  // namespace
}  // namespace csattn

using namespace csattn;

extern "C" {

int csattn_page_tables(const int32_t* cache_lens, const int32_t* new_lens, int32_t* block_table,
                       const int32_t* free_pages, const int32_t* num_free, int32_t* seq_lens,
                       int32_t* starts, int64_t* slots, int32_t* positions, int32_t* free_left,
                       int B, int N, int page_size, int num_pages, int max_pages, int free_size,
                       void* stream) {
  const char* fn = "page_tables";
  for (const void* p : {static_cast<const void*>(cache_lens), static_cast<const void*>(new_lens),
                        static_cast<const void*>(block_table), static_cast<const void*>(num_free),
                        static_cast<const void*>(seq_lens), static_cast<const void*>(starts),
                        static_cast<const void*>(slots), static_cast<const void*>(positions),
                        static_cast<const void*>(free_left)}) {
    if (p == nullptr) return api_fail(CSATTN_ERR_INVALID_ARG, "%s: null pointer argument", fn);
    if (!aligned(p, 4)) return api_fail(CSATTN_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
  }
  if (free_size < 0 || (free_size > 0 && free_pages == nullptr))
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: %d free pages without a list", fn, free_size);
  if (!aligned(free_pages, 4) || !aligned(slots, 8))
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
  if (B < 1 || N < 1)
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: B=%d and N=%d must be >= 1", fn, B, N);
  if (!api_valid_page_size(page_size))
    return api_fail(CSATTN_ERR_INVALID_ARG,
                    "%s: page_size=%d must be 16, 32 or a multiple of 64 in [64, 65536]", fn,
                    page_size);
  if (num_pages < 1 || max_pages < 1)
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: num_pages=%d and max_pages=%d must be >= 1", fn,
                    num_pages, max_pages);
  if (B > 65535) return api_fail(CSATTN_ERR_UNSUPPORTED, "%s: B=%d too large", fn, B);
  if (N > (1 << 30)) return api_fail(CSATTN_ERR_UNSUPPORTED, "%s: N=%d too large", fn, N);
  if (static_cast<long long>(max_pages) * page_size >= (1 << 30))
    return api_fail(CSATTN_ERR_UNSUPPORTED, "%s: max_pages * page_size too large", fn);
  // CTAs read the inputs while others write
  const Span in[] = {{cache_lens, 4ull * B}, {new_lens, 4ull * B}, {num_free, 4},
                     {free_pages, 4ull * free_size},
                     {block_table, 4ull * B * static_cast<size_t>(max_pages)}};
  const Span out[] = {{seq_lens, 4ull * B}, {starts, 4ull * B + 4}, {slots, 8ull * N},
                      {positions, 4ull * N}, {free_left, 4}};
  for (const Span& o : out)
    for (const Span& i : in)
      if (o.meets(i)) return api_fail(CSATTN_ERR_INVALID_ARG, "%s: an output overlaps an input", fn);
  for (int i = 0; i < 5; ++i)
    for (int j = 0; j < i; ++j)
      if (out[i].meets(out[j]))
        return api_fail(CSATTN_ERR_INVALID_ARG, "%s: two outputs overlap", fn);
  for (int i = 0; i < 4; ++i)
    if (in[4].meets(in[i]))
      return api_fail(CSATTN_ERR_INVALID_ARG, "%s: block_table overlaps an input", fn);
  PageTablesArgs a{};
  a.held = cache_lens;
  a.fresh = new_lens;
  a.block_table = block_table;
  a.free_pages = free_pages;
  a.num_free = num_free;
  a.seq_lens = seq_lens;
  a.starts = starts;
  a.slots = slots;
  a.positions = positions;
  a.free_left = free_left;
  a.B = B;
  a.N = N;
  a.page_size = page_size;
  a.num_pages = num_pages;
  a.max_pages = max_pages;
  a.free_size = free_size;
  int sms = 0;
  const int rc = api_device_info(&a.status, &sms);
  if (rc != CSATTN_OK) return rc;
  const cudaError_t e = launch_page_tables(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CSATTN_OK : api_fail_cuda(e, "page_tables: kernel launch");
}

int csattn_qk_norm_rope(const void* q, const void* k, const void* q_weight, const void* k_weight,
                        const int32_t* positions, void* q_out, void* k_out, int B, int Hq, int Hkv,
                        int T, int d, int dtype, const int64_t* strides, int pos0, int norm,
                        float eps, float rope_base, int rope_layout, void* stream) {
  QkNormArgs a{};
  int rc = norm_args("qk_norm_rope", &a, q, k, q_weight, k_weight, positions, q_out, k_out, B, Hq,
                     Hkv, T, d, dtype, strides, pos0, norm, eps, rope_base, rope_layout);
  if (rc != CSATTN_OK) return rc;
  a.q.y = q_out;
  a.k.y = k_out;
  for (QkNormSide* s : {&a.q, &a.k}) {
    s->y_token = d;
    s->y_head = static_cast<long long>(T) * d;
    s->y_batch = s->H * s->y_head;
  }
  const int size = dtype == CSATTN_BF16 ? 2 : 4;
  const long long each = 1LL * T * d * size * B;
  const Places written[] = {{q_out, each * Hq}, {k_out, each * Hkv}};
  const Places read[] = {{q, B, Hq, T, d, size, a.q.batch, a.q.head, a.q.token},
                         {k, B, Hkv, T, d, size, a.k.batch, a.k.head, a.k.token},
                         {q_weight, 1LL * d * size}, {k_weight, 1LL * d * size},
                         {positions, 4LL * B * T}};
  if ((rc = check_apart("qk_norm_rope", written, 2, read, 5)) != CSATTN_OK) return rc;
  int sms = 0;
  if ((rc = api_device_info(&a.status, &sms)) != CSATTN_OK) return rc;
  const cudaError_t e =
      launch_qk_norm(a, dtype == CSATTN_BF16, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CSATTN_OK : api_fail_cuda(e, "qk_norm_rope: kernel launch");
}

size_t csattn_qk_norm_rope_bwd_workspace_size(int d) {
  return d > 0 && d <= 128 ? (qk_norm_bwd_blocks() + 2) * static_cast<size_t>(d) * 4 : 0;
}

int csattn_qk_norm_rope_bwd(const void* dq_out, const void* dk_out, const void* q, const void* k,
                            const void* q_weight, const void* k_weight, const int32_t* positions,
                            void* dq, void* dk, float* dq_weight, float* dk_weight, int B, int Hq,
                            int Hkv, int T, int d, int dtype, const int64_t* strides, int pos0,
                            int norm, float eps, float rope_base, int rope_layout, void* workspace,
                            size_t workspace_bytes, void* stream) {
  const char* fn = "qk_norm_rope_bwd";
  QkNormArgs a{};
  int rc = norm_args(fn, &a, q, k, q_weight, k_weight, positions, dq_out, dk_out, B, Hq, Hkv, T, d,
                     dtype, strides, pos0, norm, eps, rope_base, rope_layout);
  if (rc != CSATTN_OK) return rc;
  if (dq == nullptr || dk == nullptr)
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: null pointer argument", fn);
  if (!aligned(dq, 16) || !aligned(dk, 16) || !aligned(dq_weight, 4) || !aligned(dk_weight, 4))
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
  if ((dq_weight == nullptr) != (q_weight == nullptr) ||
      (dk_weight == nullptr) != (k_weight == nullptr))
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: a gain and its gradient go together", fn);
  const int size = dtype == CSATTN_BF16 ? 2 : 4;
  rc = set_strides(fn, strides != nullptr ? strides + 6 : nullptr, B, Hq, T, d, size,
                   &a.q.y_batch, &a.q.y_head, &a.q.y_token);
  if (rc != CSATTN_OK) return rc;
  rc = set_strides(fn, strides != nullptr ? strides + 9 : nullptr, B, Hkv, T, d, size,
                   &a.k.y_batch, &a.k.y_head, &a.k.y_token);
  if (rc != CSATTN_OK) return rc;
  a.q.dy = dq_out;
  a.k.dy = dk_out;
  a.q.y = dq;
  a.k.y = dk;
  if (dq_weight != nullptr || dk_weight != nullptr) {
    const size_t need = csattn_qk_norm_rope_bwd_workspace_size(d);
    if (workspace == nullptr || workspace_bytes < need || !aligned(workspace, 16))
      return api_fail(CSATTN_ERR_WORKSPACE,
                      "%s: needs a 16-byte aligned workspace of %zu bytes (got %zu)", fn, need,
                      workspace_bytes);
    a.partial = static_cast<float*>(workspace);
  }
  const long long each = 1LL * T * d * size * B;
  const Places written[] = {
      {dq, B, Hq, T, d, size, a.q.y_batch, a.q.y_head, a.q.y_token},
      {dk, B, Hkv, T, d, size, a.k.y_batch, a.k.y_head, a.k.y_token},
      {dq_weight, 4LL * d}, {dk_weight, 4LL * d},
      {a.partial, static_cast<long long>(csattn_qk_norm_rope_bwd_workspace_size(d))}};
  const Places read[] = {{q, B, Hq, T, d, size, a.q.batch, a.q.head, a.q.token},
                         {k, B, Hkv, T, d, size, a.k.batch, a.k.head, a.k.token},
                         {dq_out, each * Hq}, {dk_out, each * Hkv},
                         {q_weight, 1LL * d * size}, {k_weight, 1LL * d * size},
                         {positions, 4LL * B * T}};
  if ((rc = check_apart(fn, written, 5, read, 7)) != CSATTN_OK) return rc;
  int sms = 0;
  if ((rc = api_device_info(&a.status, &sms)) != CSATTN_OK) return rc;
  const cudaError_t e = launch_qk_norm_bwd(a, dtype == CSATTN_BF16, dq_weight, dk_weight,
                                           static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CSATTN_OK : api_fail_cuda(e, "qk_norm_rope_bwd: kernel launch");
}

}  // extern "C"
