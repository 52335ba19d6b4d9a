// C ABI of the 8-bit KV cache and of the token-tree calls: argument checks, split sizes,
// workspace layout and dispatch.  See include/csattn.h for the contract of every entry point.
#include <algorithm>
#include <cmath>

#include "csattn.h"
#include "internal.h"

namespace csattn {
namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

constexpr int kMaxTree = 256;  // drafts of a tree
constexpr int kMaxHeads = 1 << 20;

// The paged arguments; *lmax receives the rows a sequence has room for.
int check_pages(const char* fn, const int32_t* block_table, int Hkv, int page_size, int num_pages,
                int max_pages, int* lmax) {
  if (block_table == nullptr)
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: block_table must be non-null", fn);
  if (!aligned(block_table, 4))
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: block_table must be 4-byte aligned", fn);
  if (!api_valid_page_size(page_size))
    return api_fail(CSATTN_ERR_INVALID_ARG,
                    "%s: page_size=%d must be 16, 32 or a multiple of 64 in [64, 65536]", fn,
                    page_size);
  if (num_pages < 1 || max_pages < 1)
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: num_pages=%d and max_pages=%d must be >= 1", fn,
                    num_pages, max_pages);
  if (Hkv >= 1 && static_cast<long long>(num_pages) * Hkv > (1LL << 31) - 1)
    return api_fail(CSATTN_ERR_UNSUPPORTED, "%s: num_pages * Hkv too large", fn);
  const long long rows = static_cast<long long>(max_pages) * page_size;
  if (rows >= (1 << 30))
    return api_fail(CSATTN_ERR_UNSUPPORTED, "%s: max_pages * page_size too large", fn);
  *lmax = static_cast<int>(rows);
  return CSATTN_OK;
}

// The cache itself (its pointers, sizes and head width); `scales`: 1 wanted, 0 must be null.
int check_cache(const char* fn, const KvCache& c, bool scales, const int32_t* lens, int B, int Hkv,
                int d) {
  if (c.k == nullptr || c.v == nullptr || lens == nullptr ||
      (scales && (c.k_scale == nullptr || c.v_scale == nullptr)))
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: null pointer argument", fn);
  if (!scales && (c.k_scale != nullptr || c.v_scale != nullptr))
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: a bf16 cache has no scales", fn);
  if (B < 1 || Hkv < 1 || c.Lmax < 1)
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: B=%d Hkv=%d Lmax=%d must be >= 1", fn, B, Hkv,
                    c.Lmax);
  if (d != 64 && d != 128)
    return api_fail(CSATTN_ERR_UNSUPPORTED, "%s: d=%d not in {64,128}", fn, d);
  if (c.Lmax >= (1 << 30))
    return api_fail(CSATTN_ERR_UNSUPPORTED, "%s: %d cache rows too many", fn, c.Lmax);
  if (B > 65535 || Hkv > 65535 || static_cast<long long>(B) * Hkv > (1LL << 31) - 1)
    return api_fail(CSATTN_ERR_UNSUPPORTED, "%s: B=%d or Hkv=%d too large", fn, B, Hkv);
  if (!aligned(c.k, 16) || !aligned(c.v, 16) || !aligned(lens, 4))
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
  return CSATTN_OK;
}

int check_dtype(const char* fn, int dtype) {
  if (dtype == CSATTN_BF16) return CSATTN_OK;
  return api_fail(dtype == CSATTN_F32 ? CSATTN_ERR_UNSUPPORTED : CSATTN_ERR_INVALID_ARG,
                  "%s: only bf16 is implemented (dtype %d)", fn, dtype);
}

// positions: how many the call may rotate at.  (With a base below 1 the last frequency is the
// largest, and the angles' reduction bounds its angle like that of theta_0 = 1.)
int check_rope(const char* fn, float rope_base, int rope_layout, int positions, int d) {
  if (rope_layout != CSATTN_ROPE_SPLIT_HALF && rope_layout != CSATTN_ROPE_ADJACENT)
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: unknown rope_layout %d", fn, rope_layout);
  if (!std::isfinite(rope_base))
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: rope_base must be finite", fn);
  if (rope_base > 0.f && positions > kMaxRopePositions)
    return api_fail(CSATTN_ERR_UNSUPPORTED, "%s: RoPE supports positions < %d, got %d", fn,
                    kMaxRopePositions, positions);
  if (rope_base > 0.f && rope_base < 1.f &&
      positions * std::pow(static_cast<double>(rope_base), -(d - 2.0) / d) > kMaxRopePositions)
    return api_fail(CSATTN_ERR_UNSUPPORTED, "%s: RoPE angles past %d (rope_base=%g, %d positions)",
                    fn, kMaxRopePositions, rope_base, positions);
  return CSATTN_OK;
}

// The frequencies depend on nothing but (d, base) and take d/2 powers to compute, as long as a
// launch; a thread keeps its last ones.
int rope_of(float rope_base, int rope_layout, int d, RopeTable* th) {
  if (!(rope_base > 0.f)) return 0;
  static thread_local struct {
    int d = 0;
    float base = 0.f;
    RopeTable table;
  } last;
  if (last.d != d || last.base != rope_base) {
    api_rope_table(&last.table, d, static_cast<double>(rope_base));
    last.d = d;
    last.base = rope_base;
  }
  *th = last.table;
  return rope_layout == CSATTN_ROPE_SPLIT_HALF ? 1 : 2;
}

int check_heads(const char* fn, int B, int Hq, int Hkv, int T, float scale, int max_seq_len,
                int lmax, int num_splits) {
  if (Hq < 1 || Hq % Hkv != 0)
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: Hq=%d is not a multiple of Hkv=%d", fn, Hq, Hkv);
  if (max_seq_len < T || max_seq_len > lmax)
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: max_seq_len=%d not in [%d, Lmax=%d]", fn,
                    max_seq_len, T, lmax);
  if (num_splits < 0) return api_fail(CSATTN_ERR_INVALID_ARG, "%s: num_splits < 0", fn);
  if (!std::isfinite(scale))
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: scale not finite", fn);
  if (Hq > kMaxHeads || static_cast<long long>(B) * Hq * T > (1LL << 31) - 1)
    return api_fail(CSATTN_ERR_UNSUPPORTED, "%s: Hq=%d or B * Hq * queries too large", fn, Hq);
  return CSATTN_OK;
}

// The kernel for `rows` query rows per KV head, and how its work is shared out: a wave of CTAs,
// or, with an explicit number of splits, as many CTAs as parts of that many equal ones of the
// longest sequence can fill.
// Trees with more query rows per KV head than this go to launch_group_tc (128 channels, 8
// sequences of 8000 rows: 16 rows 50.4 us bf16, 41.7 e4m3 here; 20 rows 52.5 and 55.5 there; the
// other way round, when this was chosen, 16 rows took 58 and 58, and 20 rows 91 and 69, the cache
// being read once per 16 rows here).
constexpr int kTcRows = 16;

GroupPlan plan_for(int B, int Hkv, int rows, int d, bool tc, bool f8, int max_seq_len,
                   int num_splits) {
  GroupPlan p{};
  p.tc = tc;
  p.unit = tc ? 128 : 64;
  p.block_rows = tc ? (rows > 128 ? 256 : 128) : (rows > 8 ? 16 : 8);
  p.rblocks = (rows + p.block_rows - 1) / p.block_rows;
  p.part_rows = std::min(rows, p.block_rows);
  p.subs = tc ? 1 : 4;  // launch_group_attn: one for each of its four warps
  if (num_splits > 0) {
    const long long tiles = (max_seq_len + p.unit - 1) / p.unit;
    p.tiles_per_cta = static_cast<int>((tiles + num_splits - 1) / num_splits);
    const long long parts = (tiles + p.tiles_per_cta - 1) / p.tiles_per_cta;
    // (a shorter bound may cut finer: as many parts as asked for, or a tile each)
    p.most_grid = static_cast<int>(std::min<long long>(
        0x7fffffff, std::min<long long>(num_splits, tiles) * B * Hkv * p.rblocks));
    p.grid = static_cast<int>(std::min<long long>(0x7fffffff, parts * B * Hkv * p.rblocks));
  } else {
    // Resident CTAs (launch bounds and shared memory of the kernels), or as many as the longest
    // sequences could occupy.  The small kernel's CTAs take two tiles at least: with one, a
    // short cache ends in as many partial results as tiles (one sequence of 1000 rows, 8 KV
    // heads: 9.8 us against 8.6).
    p.least_tiles = tc ? 1 : 2;
    const long long tiles = (max_seq_len + p.unit - 1) / p.unit;
    const long long line = tiles * B * Hkv * p.rblocks;
    const int resident = kSms * (tc ? 1 : group_attn_ctas(d, f8, p.block_rows));
    p.most_grid = p.grid = static_cast<int>(
        std::min<long long>(resident, (line + p.least_tiles - 1) / p.least_tiles));
  }
  return p;
}

// Bytes of the partial results: [grid + segments, subs, part_rows] rows of d + 2 floats, with
// room for any smaller max_seq_len.
size_t partial_floats(const GroupPlan& p, int B, int Hkv) {
  return (static_cast<size_t>(p.most_grid) + static_cast<size_t>(B) * Hkv * p.rblocks) * p.subs *
         p.part_rows;
}
size_t partial_bytes(const GroupPlan& p, int B, int Hkv, int d) {
  return partial_floats(p, B, Hkv) * (static_cast<size_t>(d) + 2) * 4;
}
// What the kernel leaves the merge of each segment (GroupLine::seg) follows the partials.
size_t seg_bytes(const GroupPlan& p, int B, int Hkv) {
  return align256(static_cast<size_t>(B) * Hkv * p.rblocks * 8);
}

// (GroupLine counts tiles in 31 bits)
int check_line(const char* fn, const GroupPlan& p, int B, int Hkv, int max_seq_len) {
  if (static_cast<long long>(B) * Hkv * p.rblocks > ((1LL << 31) - 1) / (max_seq_len / p.unit + 1))
    return api_fail(CSATTN_ERR_UNSUPPORTED, "%s: B * Hkv * max_seq_len too large", fn);
  return CSATTN_OK;
}

// (as check_cache and check_heads, for the workspace sizes)
bool sizes_ok(int B, int Hq, int Hkv, int T, int Lmax, int d, int num_splits) {
  return B >= 1 && B <= 65535 && Hq >= 1 && Hq <= kMaxHeads && Hkv >= 1 && Hkv <= 65535 &&
         Hq % Hkv == 0 && static_cast<long long>(B) * Hq * T <= (1LL << 31) - 1 && Lmax >= 1 &&
         Lmax < (1 << 30) && (d == 64 || d == 128) && num_splits >= 0;
}

// csattn_selftest_lost_arrival: the thread's next call
thread_local int g_lost = 0;
int take_lost() {
  const int lost = g_lost;
  g_lost = 0;
  return lost;
}

int check_workspace(const char* fn, const void* workspace, size_t bytes, size_t need) {
  if (workspace == nullptr || bytes < need || !aligned(workspace, 16))
    return api_fail(CSATTN_ERR_WORKSPACE,
                    "%s: needs a 16-byte aligned workspace of %zu bytes (got %zu)", fn, need,
                    bytes);
  return CSATTN_OK;
}

int encoder_ready(const char* fn) {
  if (tensor_map_encoder() == nullptr)
    return api_fail(CSATTN_ERR_CUDA, "%s: cuTensorMapEncodeTiled is unavailable", fn);
  return CSATTN_OK;
}

int append_fp8(const char* fn, const void* k_new, const void* v_new, const KvCache& c,
               const int32_t* cache_lens, int B, int Hkv, int Tn, int d, int dtype,
               float rope_base, int rope_layout, void* stream) {
  int rc = check_cache(fn, c, true, cache_lens, B, Hkv, d);
  if (rc != CSATTN_OK) return rc;
  if (k_new == nullptr || v_new == nullptr)
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: null pointer argument", fn);
  if (!aligned(k_new, 16) || !aligned(v_new, 16))
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
  if ((rc = check_dtype(fn, dtype)) != CSATTN_OK) return rc;
  if (Tn < 1 || Tn > c.Lmax)
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: Tn=%d not in [1, cache rows %d]", fn, Tn, c.Lmax);
  if (static_cast<long long>(B) * Hkv * Tn * d >= (1LL << 33))
    return api_fail(CSATTN_ERR_UNSUPPORTED, "%s: Tn=%d too large", fn, Tn);
  if ((rc = check_rope(fn, rope_base, rope_layout, c.Lmax, d)) != CSATTN_OK) return rc;
  RopeTable th{};
  const int rope = rope_of(rope_base, rope_layout, d, &th);
  uint32_t* status = nullptr;
  int sms = 0;
  if ((rc = api_device_info(&status, &sms)) != CSATTN_OK) return rc;
  const cudaError_t e = launch_cache_append_fp8(k_new, v_new, c, cache_lens, B, Hkv, Tn, d, rope,
                                                th, status, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CSATTN_OK : api_fail_cuda(e, "cache_append_fp8: kernel launch");
}

int read_fp8(const char* fn, const KvCache& c, const int32_t* seq_lens, void* k_out, void* v_out,
             int B, int Hkv, int Lout, int d, int dtype, void* stream) {
  int rc = check_cache(fn, c, true, seq_lens, B, Hkv, d);
  if (rc != CSATTN_OK) return rc;
  if (k_out == nullptr || v_out == nullptr)
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: null pointer argument", fn);
  if (!aligned(k_out, 16) || !aligned(v_out, 16))
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
  if ((rc = check_dtype(fn, dtype)) != CSATTN_OK) return rc;
  if (Lout < 1) return api_fail(CSATTN_ERR_INVALID_ARG, "%s: Lout=%d must be >= 1", fn, Lout);
  if (Lout >= (1 << 24) || static_cast<long long>(B) * Hkv * Lout >= (1LL << 33))
    return api_fail(CSATTN_ERR_UNSUPPORTED, "%s: Lout=%d too large", fn, Lout);
  if (static_cast<long long>(B) * Hkv >= (1LL << 30))
    return api_fail(CSATTN_ERR_UNSUPPORTED, "%s: B=%d * Hkv=%d too large", fn, B, Hkv);
  uint32_t* status = nullptr;
  int sms = 0;
  if ((rc = api_device_info(&status, &sms)) != CSATTN_OK) return rc;
  const cudaError_t e = launch_cache_read_fp8(c, seq_lens, k_out, v_out, B, Hkv, Lout, d, status,
                                              static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CSATTN_OK : api_fail_cuda(e, "cache_read_fp8: kernel launch");
}

int decode_fp8(const char* fn, const void* q, const KvCache& c, const int32_t* seq_lens, void* out,
               int B, int Hq, int Hkv, int d, int dtype, float rope_base, int rope_layout,
               float scale, int max_seq_len, int num_splits, void* workspace,
               size_t workspace_bytes, void* stream) {
  int rc = check_cache(fn, c, true, seq_lens, B, Hkv, d);
  if (rc != CSATTN_OK) return rc;
  if (q == nullptr || out == nullptr)
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: null pointer argument", fn);
  if (!aligned(q, 16) || !aligned(out, 16))
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
  if ((rc = check_dtype(fn, dtype)) != CSATTN_OK) return rc;
  if ((rc = check_heads(fn, B, Hq, Hkv, 1, scale, max_seq_len, c.Lmax, num_splits)) != CSATTN_OK)
    return rc;
  if ((rc = check_rope(fn, rope_base, rope_layout, max_seq_len, d)) != CSATTN_OK) return rc;
  GroupArgs a{};
  a.plan = plan_for(B, Hkv, Hq / Hkv, d, false, true, max_seq_len, num_splits);
  if ((rc = check_line(fn, a.plan, B, Hkv, max_seq_len)) != CSATTN_OK) return rc;
  const size_t partials = partial_bytes(a.plan, B, Hkv, d);
  if ((rc = check_workspace(fn, workspace, workspace_bytes,
                            align256(partials) + seg_bytes(a.plan, B, Hkv))) != CSATTN_OK)
    return rc;
  a.cache = c;
  a.q = q;
  a.lens = seq_lens;
  a.rope = rope_of(rope_base, rope_layout, d, &a.theta);
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.T = 1;
  a.d = d;
  a.scale = scale > 0.f ? scale : static_cast<float>(1.0 / std::sqrt(static_cast<double>(d)));
  a.max_seq_len = max_seq_len;
  a.min_len = 1;
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = a.part_o + partial_floats(a.plan, B, Hkv) * d;
  a.seg = reinterpret_cast<int2*>(static_cast<uint8_t*>(workspace) + align256(partials));
  int sms = 0;
  if ((rc = api_device_info(&a.status, &sms)) != CSATTN_OK) return rc;
  if ((rc = encoder_ready(fn)) != CSATTN_OK) return rc;
  a.lost = take_lost();
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_group_attn(a, st);
  if (e != cudaSuccess) return api_fail_cuda(e, "attn_decode_fp8: kernel launch");
  e = launch_group_merge(a, nullptr, nullptr, out, nullptr, st);
  return e == cudaSuccess ? CSATTN_OK : api_fail_cuda(e, "attn_decode_fp8: merge launch");
}

// Workspace of a tree step: partials, then rotated queries, masks, lengths and value flags.
struct TreeSpace {
  size_t seg, q_rot, q_factor, anc, lens, vflag, total;
  TreeSpace(const GroupPlan& p, int B, int Hq, int Hkv, int Tn, int d) {
    const size_t words = (Tn + 31) / 32;
    seg = align256(partial_bytes(p, B, Hkv, d));
    q_rot = seg + seg_bytes(p, B, Hkv);
    q_factor = q_rot + align256(static_cast<size_t>(B) * Hq * Tn * d * 2);
    anc = q_factor + align256(static_cast<size_t>(B) * Hq * Tn * 4);
    lens = anc + align256(static_cast<size_t>(B) * Tn * words * 4);
    vflag = lens + align256(static_cast<size_t>(B) * 4);
    total = vflag + align256(static_cast<size_t>(B) * Hkv * Tn);
  }
};

GroupPlan tree_plan(int B, int Hq, int Hkv, int Tn, int d, bool f8, int max_seq_len,
                    int num_splits) {
  const int rows = Tn * (Hq / Hkv);
  return plan_for(B, Hkv, rows, d, rows > kTcRows, f8, max_seq_len, num_splits);
}

int tree_step(const char* fn, const void* q_new, const void* k_new, const void* v_new,
              const KvCache& c, const int32_t* cache_lens, const int32_t* parents, void* out,
              float* lse, int B, int Hq, int Hkv, int Tn, int d, int cache_dtype, float rope_base,
              int rope_layout, float scale, int max_seq_len, int num_splits, void* workspace,
              size_t workspace_bytes, void* stream) {
  if (cache_dtype != CSATTN_BF16 && cache_dtype != CSATTN_E4M3)
    return api_fail(cache_dtype == CSATTN_F32 ? CSATTN_ERR_UNSUPPORTED : CSATTN_ERR_INVALID_ARG,
                    "%s: the cache is bf16 or e4m3 (cache_dtype %d)", fn, cache_dtype);
  int rc = check_cache(fn, c, cache_dtype == CSATTN_E4M3, cache_lens, B, Hkv, d);
  if (rc != CSATTN_OK) return rc;
  if (q_new == nullptr || k_new == nullptr || v_new == nullptr || parents == nullptr ||
      out == nullptr)
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: null pointer argument", fn);
  if (!aligned(q_new, 16) || !aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(out, 16) ||
      !aligned(parents, 4) || !aligned(lse, 4))
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
  if (Tn < 1) return api_fail(CSATTN_ERR_INVALID_ARG, "%s: Tn=%d must be >= 1", fn, Tn);
  if (Tn > kMaxTree)
    return api_fail(CSATTN_ERR_UNSUPPORTED, "%s: Tn=%d exceeds %d drafts", fn, Tn, kMaxTree);
  if ((rc = check_heads(fn, B, Hq, Hkv, Tn, scale, max_seq_len, c.Lmax, num_splits)) != CSATTN_OK)
    return rc;
  if ((rc = check_rope(fn, rope_base, rope_layout, max_seq_len, d)) != CSATTN_OK) return rc;
  GroupArgs a{};
  a.plan = tree_plan(B, Hq, Hkv, Tn, d, cache_dtype == CSATTN_E4M3, max_seq_len, num_splits);
  if ((rc = check_line(fn, a.plan, B, Hkv, max_seq_len)) != CSATTN_OK) return rc;
  const TreeSpace at(a.plan, B, Hq, Hkv, Tn, d);
  if ((rc = check_workspace(fn, workspace, workspace_bytes, at.total)) != CSATTN_OK) return rc;
  uint8_t* ws = static_cast<uint8_t*>(workspace);

  TreePrepArgs p{};
  p.q_new = q_new;
  p.k_new = k_new;
  p.v_new = v_new;
  p.cache = c;
  p.cache_lens = cache_lens;
  p.parents = parents;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.Tn = Tn;
  p.d = d;
  p.max_seq_len = max_seq_len;
  p.rope = rope_of(rope_base, rope_layout, d, &p.theta);
  p.q_rot = ws + at.q_rot;
  p.q_factor = reinterpret_cast<float*>(ws + at.q_factor);
  p.anc = reinterpret_cast<uint32_t*>(ws + at.anc);
  p.lens = reinterpret_cast<int32_t*>(ws + at.lens);
  p.vflag = ws + at.vflag;
  p.words = (Tn + 31) / 32;
  int sms = 0;
  if ((rc = api_device_info(&p.status, &sms)) != CSATTN_OK) return rc;
  if ((rc = encoder_ready(fn)) != CSATTN_OK) return rc;

  a.cache = c;
  a.q = p.q_rot;
  a.q_factor = cache_dtype == CSATTN_E4M3 ? p.q_factor : nullptr;
  a.lens = p.lens;
  a.anc = p.anc;
  a.drafts = Tn;
  a.words = p.words;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.T = Tn;
  a.d = d;
  a.scale = scale > 0.f ? scale : static_cast<float>(1.0 / std::sqrt(static_cast<double>(d)));
  a.max_seq_len = max_seq_len;
  a.min_len = 0;
  a.part_o = reinterpret_cast<float*>(ws);
  a.part_ml = a.part_o + partial_floats(a.plan, B, Hkv) * d;
  a.seg = reinterpret_cast<int2*>(ws + at.seg);
  a.status = p.status;
  a.lost = take_lost();
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_tree_prep(p, st);
  if (e != cudaSuccess) return api_fail_cuda(e, "attn_tree_step: append launch");
  e = a.plan.tc ? launch_group_tc(a, st) : launch_group_attn(a, st);
  if (e != cudaSuccess) return api_fail_cuda(e, "attn_tree_step: kernel launch");
  e = a.plan.tc ? launch_group_tc_merge(a, p.vflag, v_new, out, lse, st)
                : launch_group_merge(a, p.vflag, v_new, out, lse, st);
  return e == cudaSuccess ? CSATTN_OK : api_fail_cuda(e, "attn_tree_step: merge launch");
}

int tree_commit(const char* fn, const KvCache& c, const int32_t* cache_lens,
                const int32_t* parents, const int32_t* accepted, int32_t* new_lens, int B, int Hkv,
                int Tn, int d, int cache_dtype, void* stream) {
  if (cache_dtype != CSATTN_BF16 && cache_dtype != CSATTN_E4M3)
    return api_fail(cache_dtype == CSATTN_F32 ? CSATTN_ERR_UNSUPPORTED : CSATTN_ERR_INVALID_ARG,
                    "%s: the cache is bf16 or e4m3 (cache_dtype %d)", fn, cache_dtype);
  int rc = check_cache(fn, c, cache_dtype == CSATTN_E4M3, cache_lens, B, Hkv, d);
  if (rc != CSATTN_OK) return rc;
  if (parents == nullptr || accepted == nullptr || new_lens == nullptr)
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: null pointer argument", fn);
  if (!aligned(parents, 4) || !aligned(accepted, 4) || !aligned(new_lens, 4))
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
  if (Tn < 1 || Tn > c.Lmax)
    return api_fail(CSATTN_ERR_INVALID_ARG, "%s: Tn=%d not in [1, cache rows %d]", fn, Tn, c.Lmax);
  if (Tn > kMaxTree)
    return api_fail(CSATTN_ERR_UNSUPPORTED, "%s: Tn=%d exceeds %d drafts", fn, Tn, kMaxTree);
  // every KV head's CTA reads the lengths while one writes the new ones
  const uintptr_t n0 = reinterpret_cast<uintptr_t>(new_lens), n1 = n0 + 4ull * B;
  for (const void* in : {static_cast<const void*>(cache_lens), static_cast<const void*>(accepted),
                         static_cast<const void*>(parents)}) {
    const uintptr_t i0 = reinterpret_cast<uintptr_t>(in);
    const uintptr_t i1 = i0 + 4ull * B * (in == parents ? Tn : 1);
    if (n0 < i1 && i0 < n1)
      return api_fail(CSATTN_ERR_INVALID_ARG, "%s: new_lens overlaps an input", fn);
  }
  uint32_t* status = nullptr;
  int sms = 0;
  if ((rc = api_device_info(&status, &sms)) != CSATTN_OK) return rc;
  const cudaError_t e = launch_tree_commit(c, cache_lens, parents, accepted, new_lens, B, Hkv, Tn,
                                           d, status, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CSATTN_OK : api_fail_cuda(e, "tree_commit: kernel launch");
}

KvCache contiguous(const void* k, const void* v, const void* ks, const void* vs, int Lmax) {
  KvCache c{};
  c.k = const_cast<void*>(k);
  c.v = const_cast<void*>(v);
  c.k_scale = const_cast<void*>(ks);
  c.v_scale = const_cast<void*>(vs);
  c.Lmax = Lmax;
  return c;
}
KvCache paged(const void* k, const void* v, const void* ks, const void* vs,
              const int32_t* block_table, int lmax, int page_size, int num_pages, int max_pages) {
  KvCache c = contiguous(k, v, ks, vs, lmax);
  c.block_table = block_table;
  c.page_size = page_size;
  c.num_pages = num_pages;
  c.max_pages = max_pages;
  return c;
}

}  // namespace
}  // namespace csattn

using namespace csattn;

extern "C" {

int csattn_cache_append_fp8(const void* k_new, const void* v_new, void* k_cache, void* v_cache,
                            void* k_scale, void* v_scale, const int32_t* cache_lens, int B,
                            int Hkv, int Tn, int Lmax, int d, int dtype, float rope_base,
                            int rope_layout, void* stream) {
  return append_fp8("cache_append_fp8", k_new, v_new,
                    contiguous(k_cache, v_cache, k_scale, v_scale, Lmax), cache_lens, B, Hkv, Tn,
                    d, dtype, rope_base, rope_layout, stream);
}

int csattn_cache_append_fp8_paged(const void* k_new, const void* v_new, void* k_pages,
                                  void* v_pages, void* k_scale, void* v_scale,
                                  const int32_t* block_table, const int32_t* cache_lens, int B,
                                  int Hkv, int Tn, int page_size, int num_pages, int max_pages,
                                  int d, int dtype, float rope_base, int rope_layout,
                                  void* stream) {
  const char* fn = "cache_append_fp8_paged";
  int lmax = 0;
  const int rc = check_pages(fn, block_table, Hkv, page_size, num_pages, max_pages, &lmax);
  if (rc != CSATTN_OK) return rc;
  return append_fp8(fn, k_new, v_new,
                    paged(k_pages, v_pages, k_scale, v_scale, block_table, lmax, page_size,
                          num_pages, max_pages),
                    cache_lens, B, Hkv, Tn, d, dtype, rope_base, rope_layout, stream);
}

int csattn_cache_read_fp8(const void* k_cache, const void* v_cache, const void* k_scale,
                          const void* v_scale, const int32_t* seq_lens, void* k_out, void* v_out,
                          int B, int Hkv, int Lmax, int Lout, int d, int dtype, void* stream) {
  return read_fp8("cache_read_fp8", contiguous(k_cache, v_cache, k_scale, v_scale, Lmax), seq_lens,
                  k_out, v_out, B, Hkv, Lout, d, dtype, stream);
}

int csattn_cache_read_fp8_paged(const void* k_pages, const void* v_pages, const void* k_scale,
                                const void* v_scale, const int32_t* block_table,
                                const int32_t* seq_lens, void* k_out, void* v_out, int B, int Hkv,
                                int page_size, int num_pages, int max_pages, int Lout, int d,
                                int dtype, void* stream) {
  const char* fn = "cache_read_fp8_paged";
  int lmax = 0;
  const int rc = check_pages(fn, block_table, Hkv, page_size, num_pages, max_pages, &lmax);
  if (rc != CSATTN_OK) return rc;
  return read_fp8(fn,
                  paged(k_pages, v_pages, k_scale, v_scale, block_table, lmax, page_size,
                        num_pages, max_pages),
                  seq_lens, k_out, v_out, B, Hkv, Lout, d, dtype, stream);
}

size_t csattn_decode_fp8_workspace_size(int B, int Hq, int Hkv, int Lmax, int d, int num_splits) {
  if (!sizes_ok(B, Hq, Hkv, 1, Lmax, d, num_splits)) return 0;
  const GroupPlan p = plan_for(B, Hkv, Hq / Hkv, d, false, true, Lmax, num_splits);
  return align256(partial_bytes(p, B, Hkv, d)) + seg_bytes(p, B, Hkv);
}

int csattn_attn_decode_fp8(const void* q, const void* k_cache, const void* v_cache,
                           const void* k_scale, const void* v_scale, const int32_t* seq_lens,
                           void* out, int B, int Hq, int Hkv, int Lmax, int d, int dtype,
                           float rope_base, int rope_layout, float scale, int max_seq_len,
                           int num_splits, void* workspace, size_t workspace_bytes,
                           void* stream) {
  return decode_fp8("attn_decode_fp8", q, contiguous(k_cache, v_cache, k_scale, v_scale, Lmax),
                    seq_lens, out, B, Hq, Hkv, d, dtype, rope_base, rope_layout, scale,
                    max_seq_len, num_splits, workspace, workspace_bytes, stream);
}

int csattn_attn_decode_fp8_paged(const void* q, const void* k_pages, const void* v_pages,
                                 const void* k_scale, const void* v_scale,
                                 const int32_t* block_table, const int32_t* seq_lens, void* out,
                                 int B, int Hq, int Hkv, int page_size, int num_pages,
                                 int max_pages, int d, int dtype, float rope_base, int rope_layout,
                                 float scale, int max_seq_len, int num_splits, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  const char* fn = "attn_decode_fp8_paged";
  int lmax = 0;
  const int rc = check_pages(fn, block_table, Hkv, page_size, num_pages, max_pages, &lmax);
  if (rc != CSATTN_OK) return rc;
  return decode_fp8(fn, q,
                    paged(k_pages, v_pages, k_scale, v_scale, block_table, lmax, page_size,
                          num_pages, max_pages),
                    seq_lens, out, B, Hq, Hkv, d, dtype, rope_base, rope_layout, scale,
                    max_seq_len, num_splits, workspace, workspace_bytes, stream);
}

size_t csattn_tree_workspace_size(int B, int Hq, int Hkv, int Tn, int Lmax, int d,
                                  int num_splits) {
  if (Tn < 1 || Tn > kMaxTree || !sizes_ok(B, Hq, Hkv, Tn, Lmax, d, num_splits)) return 0;
  // (an 8-bit cache's plan takes no less room)
  const GroupPlan p = tree_plan(B, Hq, Hkv, Tn, d, true, Lmax, num_splits);
  return TreeSpace(p, B, Hq, Hkv, Tn, d).total;
}

int csattn_attn_tree_step(const void* q_new, const void* k_new, const void* v_new, void* k_cache,
                          void* v_cache, void* k_scale, void* v_scale, const int32_t* cache_lens,
                          const int32_t* parents, void* out, float* lse, int B, int Hq, int Hkv,
                          int Tn, int Lmax, int d, int cache_dtype, float rope_base,
                          int rope_layout, float scale, int max_seq_len, int num_splits,
                          void* workspace, size_t workspace_bytes, void* stream) {
  return tree_step("attn_tree_step", q_new, k_new, v_new,
                   contiguous(k_cache, v_cache, k_scale, v_scale, Lmax), cache_lens, parents, out,
                   lse, B, Hq, Hkv, Tn, d, cache_dtype, rope_base, rope_layout, scale, max_seq_len,
                   num_splits, workspace, workspace_bytes, stream);
}

int csattn_attn_tree_step_paged(const void* q_new, const void* k_new, const void* v_new,
                                void* k_pages, void* v_pages, void* k_scale, void* v_scale,
                                const int32_t* block_table, const int32_t* cache_lens,
                                const int32_t* parents, void* out, float* lse, int B, int Hq,
                                int Hkv, int Tn, int page_size, int num_pages, int max_pages,
                                int d, int cache_dtype, float rope_base, int rope_layout,
                                float scale, int max_seq_len, int num_splits, void* workspace,
                                size_t workspace_bytes, void* stream) {
  const char* fn = "attn_tree_step_paged";
  int lmax = 0;
  const int rc = check_pages(fn, block_table, Hkv, page_size, num_pages, max_pages, &lmax);
  if (rc != CSATTN_OK) return rc;
  return tree_step(fn, q_new, k_new, v_new,
                   paged(k_pages, v_pages, k_scale, v_scale, block_table, lmax, page_size,
                         num_pages, max_pages),
                   cache_lens, parents, out, lse, B, Hq, Hkv, Tn, d, cache_dtype, rope_base,
                   rope_layout, scale, max_seq_len, num_splits, workspace, workspace_bytes,
                   stream);
}

int csattn_tree_commit(void* k_cache, void* v_cache, void* k_scale, void* v_scale,
                       const int32_t* cache_lens, const int32_t* parents, const int32_t* accepted,
                       int32_t* new_lens, int B, int Hkv, int Tn, int Lmax, int d, int cache_dtype,
                       void* stream) {
  return tree_commit("tree_commit", contiguous(k_cache, v_cache, k_scale, v_scale, Lmax),
                     cache_lens, parents, accepted, new_lens, B, Hkv, Tn, d, cache_dtype, stream);
}

int csattn_tree_commit_paged(void* k_pages, void* v_pages, void* k_scale, void* v_scale,
                             const int32_t* block_table, const int32_t* cache_lens,
                             const int32_t* parents, const int32_t* accepted, int32_t* new_lens,
                             int B, int Hkv, int Tn, int page_size, int num_pages, int max_pages,
                             int d, int cache_dtype, void* stream) {
  const char* fn = "tree_commit_paged";
  int lmax = 0;
  const int rc = check_pages(fn, block_table, Hkv, page_size, num_pages, max_pages, &lmax);
  if (rc != CSATTN_OK) return rc;
  return tree_commit(fn,
                     paged(k_pages, v_pages, k_scale, v_scale, block_table, lmax, page_size,
                           num_pages, max_pages),
                     cache_lens, parents, accepted, new_lens, B, Hkv, Tn, d, cache_dtype, stream);
}

int csattn_selftest_lost_arrival(void) {
  g_lost = 1;
  return CSATTN_OK;
}

}  // extern "C"
