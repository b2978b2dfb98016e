// paged_plan.cpp -- argument checks of the paged serving operators, and the C entry points of the two that
// need no workspace (ala_paged_step, ala_paged_write).  Nothing here reads device memory, so every refusal is
// testable on a machine without a GPU.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "../../include/ala.h"
#include "internal.h"
#include "paged.h"

namespace ala {
void set_last_error(const char* msg);
}

using namespace ala;

namespace {

constexpr int64_t kMaxKeys = (int64_t)1 << 30;  // keys of one request and rows of a cache: positions stay in int32
constexpr int64_t kMaxElems = (int64_t)1 << 40;  // of a dim, a row or a stride: bytes, and sums of a few, stay in int64

struct Err {
  char* buf;
  size_t len;
  int operator()(int status, const char* fmt, ...) const {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, len, fmt, ap);
    va_end(ap);
    return status;
  }
};

bool header_ok(const ala_tensor* t) {
  if (t->ndim < 1 || t->ndim > 4) return false;
  for (int i = 0; i < t->ndim; ++i)
    if (t->dims[i] < 0 || t->dims[i] >= kMaxElems) return false;
  return true;
}

bool is_vector(const ala_tensor* t, int64_t n) { return t->ndim == 1 && t->dims[0] == n; }

int elem_bytes(int32_t dtype) {
  return dtype == ALA_F32 || dtype == ALA_I32 ? 4 : dtype == ALA_F16 || dtype == ALA_BF16 ? 2 : dtype == ALA_I8 ? 1 : 0;
}

// A run of memory: `rows` rows of `row` bytes, `stride` apart (what is past 2^62 bytes, which no memory holds, is left out).
// Two of them share some where neither is empty and each starts before the other ends.
struct Span {
  uint64_t at, end;
  Span(const void* p, int64_t rows, int64_t stride, int64_t row) : at(reinterpret_cast<uintptr_t>(p)), end(at) {
    if (rows > 0 && row > 0) end += (uint64_t)std::min((__int128)(rows - 1) * stride + row, (__int128)1 << 62);
  }
  Span(const void* p, int64_t bytes) : Span(p, 1, 0, bytes) {}
  bool shares(const Span& o) const { return at < end && o.at < o.end && at < o.end && o.at < end; }
};

bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Elements of a row, whose dims are t's from `first` on (one, or heads and headSize); -1 for more than can be counted.
int64_t row_elems(const ala_tensor* t, int first) {
  if (t->ndim == first + 1) return t->dims[first];
  const int64_t heads = t->dims[first], d = t->dims[first + 1];
  return heads > 0 && d > (kMaxElems - 1) / heads ? -1 : heads * d;
}

// [numBlocks, blockSize, row] or [numBlocks, blockSize, heads, headSize]
bool cache_dims(const ala_tensor* t, int64_t* blocks, int64_t* block_size, int64_t* row) {
  if (t->ndim != 3 && t->ndim != 4) return false;
  *blocks = t->dims[0];
  *block_size = t->dims[1];
  *row = row_elems(t, 2);
  return *row >= 0 && *block_size > 0 && *blocks < kMaxKeys && *block_size < kMaxKeys && *blocks * *block_size <= kMaxKeys;
}

}  // namespace

int ala::paged_plan(PagedPlan* plan, const PagedAttnArgs& a, char* errbuf, size_t errlen) {
  const Err fail{errbuf, errlen};
  const int maps = a.diff ? 2 : 1;
  for (const ala_tensor* t : {a.query, a.key, a.value, a.block_tables, a.seq_len, a.kv_seq_len, a.out})
    if (!t) return fail(ALA_NULL_REQUIRED, "query, key, value, blockTables, seqLen, kvSeqLen and attnOut are required");
  if (a.diff && !a.lambda) return fail(ALA_NULL_REQUIRED, "lambda is required");
  for (const ala_tensor* t : {a.query, a.key, a.value, a.block_tables, a.seq_len, a.kv_seq_len, a.out, a.slopes, a.lambda,
                              a.norm_weight, a.lse})
    if (t && !header_ok(t)) return fail(ALA_INVALID_SHAPE, "tensor with bad ndim or dims");
  if (a.heads <= 0) return fail(ALA_INVALID_PARAM, "headNum must be > 0 (got %d)", a.heads);
  if (a.kv_heads <= 0 || a.heads % a.kv_heads)
    return fail(ALA_INVALID_PARAM, "kvHeadNum must be > 0 and divide headNum (%d, %d)", a.heads, a.kv_heads);
  if (a.heads > 65536) return fail(ALA_UNSUPPORTED, "headNum %d is above 65536", a.heads);
  const bool alibi = a.mask_type == 3 || a.mask_type == 4 || a.mask_type == 5;
  if (a.diff ? !(a.mask_type == 0 || a.mask_type == 9) : !(a.mask_type == 0 || alibi || a.mask_type == 9))
    return fail(ALA_INVALID_PARAM, a.diff ? "maskType %d not in {0,9}" : "maskType %d not in {0,3,4,5,9}", a.mask_type);
  if (!std::isfinite(a.qk_scale)) return fail(ALA_INVALID_PARAM, "qkScale must be finite");
  if (!std::isfinite(a.out_scale)) return fail(ALA_INVALID_PARAM, "outScale must be finite");
  if (!(std::isfinite(a.norm_eps) && a.norm_eps >= 0.f)) return fail(ALA_INVALID_PARAM, "normEps must be finite and >= 0");

  // query [nTokens, heads * d] or [nTokens, heads, d], heads counting both maps
  const int64_t heads = (int64_t)a.heads * maps, kv_heads = a.kv_heads;
  const int32_t dt = a.query->dtype;
  if (dt != ALA_F16 && dt != ALA_BF16) return fail(ALA_INVALID_DTYPE, "query dtype must be f16 or bf16");
  if (a.key->dtype != dt || a.value->dtype != dt || a.out->dtype != dt)
    return fail(ALA_INVALID_DTYPE, "key, value and attnOut must have the query's dtype");
  if (a.query->ndim != 2 && a.query->ndim != 3) return fail(ALA_INVALID_SHAPE, "query must be 2-D or 3-D");
  if (a.query->ndim == 2 ? a.query->dims[1] % heads != 0 : a.query->dims[1] != heads)
    return fail(ALA_INVALID_SHAPE, "query must hold %lld heads", (long long)heads);
  const int64_t n_tokens = a.query->dims[0], d = a.query->ndim == 2 ? a.query->dims[1] / heads : a.query->dims[2];
  const int64_t row = d * maps;
  if (n_tokens > kMaxKeys) return fail(ALA_UNSUPPORTED, "more than 2^30 tokens");
  if (d < 8 || d % 8 || paged_kernel_d(row) == 0)
    return fail(ALA_UNSUPPORTED, "headSize %lld is not built (a multiple of 8 up to %d)", (long long)d, 256 / maps);
  if (alibi && d > 128) return fail(ALA_INVALID_PARAM, "headSize must be <= 128 with ALiBi masks (got %lld)", (long long)d);
  const int64_t group = heads / kv_heads;
  if (group > 128) return fail(ALA_UNSUPPORTED, "more than %d query heads per kv head", 128 / maps);
  const int64_t stride = a.query_stride ? a.query_stride : heads * d;
  if (stride < heads * d || stride % 8 || stride >= kMaxElems)
    return fail(ALA_INVALID_PARAM, "queryStride must be 0, or a multiple of 8 that holds a token's heads (got %lld)",
                (long long)stride);
  // attnOut [nTokens, headNum * row] or [nTokens, headNum, row]
  const int64_t out_heads = a.heads;
  if (!(a.out->dims[0] == n_tokens && ((a.out->ndim == 2 && a.out->dims[1] == out_heads * row) ||
                                       (a.out->ndim == 3 && a.out->dims[1] == out_heads && a.out->dims[2] == row))))
    return fail(ALA_INVALID_SHAPE, "attnOut must be [%lld, %lld, %lld]", (long long)n_tokens, (long long)out_heads,
                (long long)row);
  // caches
  int64_t nb = 0, bs = 0, r = 0, vnb = 0, vbs = 0, vr = 0;
  if (!cache_dims(a.key, &nb, &bs, &r) || !cache_dims(a.value, &vnb, &vbs, &vr))
    return fail(ALA_INVALID_SHAPE, "key and value must be [numBlocks, blockSize, ...] with at most 2^30 rows");
  if (r != kv_heads * row || vr != kv_heads * row || (a.key->ndim == 4 && a.key->dims[3] != d) ||
      (a.value->ndim == 4 && a.value->dims[3] != row))
    return fail(ALA_INVALID_SHAPE, "key rows must hold %lld heads of %lld, value rows %lld of %lld", (long long)(kv_heads * maps),
                (long long)d, (long long)kv_heads, (long long)row);
  if (nb != vnb || bs != vbs) return fail(ALA_INVALID_SHAPE, "key and value caches differ in shape");
  if (bs % 16) return fail(ALA_UNSUPPORTED, "blockSize %lld must be a multiple of 16", (long long)bs);
  // device metadata
  if (a.block_tables->dtype != ALA_I32 || a.seq_len->dtype != ALA_I32 || a.kv_seq_len->dtype != ALA_I32)
    return fail(ALA_INVALID_DTYPE, "blockTables, seqLen and kvSeqLen must be int32 (device)");
  if (a.block_tables->ndim != 2) return fail(ALA_INVALID_SHAPE, "blockTables must be [batch, maxBlockNum]");
  const int64_t batch = a.block_tables->dims[0], max_blocks = a.block_tables->dims[1];
  if (!is_vector(a.seq_len, batch) || !is_vector(a.kv_seq_len, batch))
    return fail(ALA_INVALID_SHAPE, "seqLen and kvSeqLen must be [batch]");
  if (batch > (1 << 20)) return fail(ALA_UNSUPPORTED, "more than 2^20 sequences");
  if (max_blocks > kMaxKeys / bs) return fail(ALA_UNSUPPORTED, "maxBlockNum * blockSize is above 2^30");
  if (alibi && !a.slopes) return fail(ALA_NULL_REQUIRED, "slopes are required for maskType %d", a.mask_type);
  if (!alibi && a.slopes) return fail(ALA_INVALID_PARAM, "slopes must be NULL for maskType %d", a.mask_type);
  for (const ala_tensor* t : {a.slopes, a.lambda, a.norm_weight, a.lse})
    if (t && t->dtype != ALA_F32) return fail(ALA_INVALID_DTYPE, "slopes, lambda, normWeight and lse must be fp32");
  if (a.slopes && !is_vector(a.slopes, a.heads)) return fail(ALA_INVALID_SHAPE, "slopes must be [headNum]");
  if (a.lambda && !is_vector(a.lambda, a.heads)) return fail(ALA_INVALID_SHAPE, "lambda must be [headNum]");
  if (a.norm_weight && !is_vector(a.norm_weight, row)) return fail(ALA_INVALID_SHAPE, "normWeight must be [2 * headSize]");
  if (a.lse) {
    const bool shape = a.lse->ndim >= 2 && a.lse->dims[0] == n_tokens && a.lse->dims[1] == a.heads &&
                       (a.lse->ndim == 2 || (a.lse->ndim == 3 && a.lse->dims[2] == 1));
    if (!shape) return fail(ALA_INVALID_SHAPE, "lse must be [nTokens, headNum]");
  }
  // a tensor with no elements may come without an address; one with elements may not
  const bool empty = n_tokens == 0 || batch == 0;
  if (!empty) {
    for (const ala_tensor* t : {a.query, a.seq_len, a.kv_seq_len, a.out, a.slopes, a.lambda, a.norm_weight, a.lse})
      if (t && !t->data) return fail(ALA_NULL_REQUIRED, "a tensor has a NULL data pointer");
    if ((nb > 0 && (!a.key->data || !a.value->data)) || (max_blocks > 0 && !a.block_tables->data))
      return fail(ALA_NULL_REQUIRED, "a tensor has a NULL data pointer");
    if (nb == 0) return fail(ALA_INVALID_SHAPE, "the cache has no blocks");
    if (!aligned(a.query->data, 16) || !aligned(a.key->data, 16) || !aligned(a.value->data, 16))
      return fail(ALA_INVALID_PARAM, "query, key and value must be 16-byte aligned");
    for (const ala_tensor* t : {a.block_tables, a.seq_len, a.kv_seq_len, a.slopes, a.lambda, a.norm_weight, a.lse})
      if (t && !aligned(t->data, 4)) return fail(ALA_INVALID_PARAM, "a tensor is not aligned to its elements");
    if (!aligned(a.out->data, 32)) return fail(ALA_INVALID_PARAM, "attnOut must be 32-byte aligned");
    // Outputs share no memory with anything, but for attnOut over a dense query: a row of it lies where its own query
    // rows are, which its CTA, or all that hold a part of it, has read by then.
    const Span out(a.out->data, n_tokens * heads * d * 2), lse(a.lse ? a.lse->data : nullptr, a.lse ? n_tokens * a.heads * 4 : 0);
    const Span query(a.query->data, n_tokens, stride * 2, heads * d * 2), cache_k(a.key->data, nb * bs, r * 2, r * 2);
    const Span ins[] = {cache_k, Span(a.value->data, nb * bs, vr * 2, vr * 2), Span(a.block_tables->data, batch * max_blocks * 4),
                        Span(a.seq_len->data, batch * 4), Span(a.kv_seq_len->data, batch * 4)};
    bool shared = out.shares(lse) || lse.shares(query) || (out.shares(query) && !(a.out->data == a.query->data && (stride == heads * d || n_tokens == 1)));
    for (const Span& x : ins) shared = shared || out.shares(x) || lse.shares(x);
    for (const ala_tensor* t : {a.slopes, a.lambda, a.norm_weight})
      if (t) shared = shared || out.shares(Span(t->data, t->dims[0] * 4)) || lse.shares(Span(t->data, t->dims[0] * 4));
    if (shared) return fail(ALA_INVALID_PARAM, "attnOut or lse overlaps another tensor (only attnOut may lie on a dense query)");
  }
  auto f32 = [](const ala_tensor* t) { return t ? static_cast<const float*>(t->data) : nullptr; };
  plan->dtype = dt;
  plan->maps = maps;
  plan->heads = (int32_t)heads;
  plan->kv_heads = a.kv_heads;
  plan->d = (int32_t)d;
  plan->row = (int32_t)row;
  plan->batch = (int32_t)batch;
  plan->max_blocks = (int32_t)max_blocks;
  plan->block_size = (int32_t)bs;
  plan->num_blocks = (int32_t)nb;
  plan->mask_type = a.mask_type;
  plan->n_tokens = n_tokens;
  plan->q_stride = stride;
  plan->qk_scale = a.qk_scale;
  plan->norm_eps = a.norm_eps;
  plan->out_scale = a.out_scale;
  plan->q = a.query->data;
  plan->k = a.key->data;
  plan->v = a.value->data;
  plan->out = a.out->data;
  plan->block_tables = static_cast<const int32_t*>(a.block_tables->data);
  plan->seq_len = static_cast<const int32_t*>(a.seq_len->data);
  plan->kv_seq_len = static_cast<const int32_t*>(a.kv_seq_len->data);
  plan->slopes = f32(a.slopes);
  plan->lambda = f32(a.lambda);
  plan->norm_weight = f32(a.norm_weight);
  plan->lse = a.lse ? static_cast<float*>(a.lse->data) : nullptr;
  paged_layout(plan);
  return ALA_OK;
}

namespace {

// Reports through ala_last_error under the entry point's name.
struct Report {
  const char* fn;
  int operator()(int status, const char* fmt, ...) const {
    char text[384], buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(text, sizeof text, fmt, ap);
    va_end(ap);
    snprintf(buf, sizeof buf, "%s: %s", fn, text);
    set_last_error(buf);
    return status;
  }
};

}  // namespace

extern "C" int ala_paged_step(const ala_tensor* seqLen, const ala_tensor* contextLens, const ala_tensor* finished,
                              ala_tensor* blockTables, ala_tensor* freeBlocks, const ala_tensor* freeCount,
                              int32_t blockSize, ala_tensor* kvSeqLen, ala_tensor* freeCountOut, ala_tensor* cuSeqLen,
                              ala_tensor* slotMapping, ala_tensor* positions, ala_tensor* status, ala_stream_t stream) {
  NvtxRange nvtx_range("ala_paged_step");
  const Report fail{"ala_paged_step"};
  const ala_tensor* all[] = {seqLen,   contextLens, blockTables, freeBlocks, freeCount, kvSeqLen, freeCountOut,
                             cuSeqLen, slotMapping, positions,   status,     finished};
  for (const ala_tensor* t : all) {
    if (!t) {
      if (t == finished) continue;
      return fail(ALA_NULL_REQUIRED, "every tensor but finished is required");
    }
    if (!header_ok(t)) return fail(ALA_INVALID_SHAPE, "tensor with bad ndim or dims");
    if (t->dtype != ALA_I32) return fail(ALA_INVALID_DTYPE, "every tensor must be int32");
    int64_t n = 1;
    for (int i = 0; i < t->ndim; ++i) n *= t->dims[i] > kMaxKeys ? kMaxKeys : t->dims[i];
    if (n > 0 && !t->data) return fail(ALA_NULL_REQUIRED, "a tensor has a NULL data pointer");
    if (!aligned(t->data, 4)) return fail(ALA_INVALID_PARAM, "a tensor is not aligned to its elements");
  }
  if (blockSize <= 0) return fail(ALA_INVALID_PARAM, "blockSize must be > 0 (got %d)", blockSize);
  if (blockTables->ndim != 2) return fail(ALA_INVALID_SHAPE, "blockTables must be [batch, maxBlockNum]");
  const int64_t batch = blockTables->dims[0], max_blocks = blockTables->dims[1];
  if (!is_vector(seqLen, batch) || !is_vector(contextLens, batch) || !is_vector(kvSeqLen, batch) ||
      (finished && !is_vector(finished, batch)))
    return fail(ALA_INVALID_SHAPE, "seqLen, contextLens, finished and kvSeqLen must be [batch]");
  if (!is_vector(cuSeqLen, batch + 1)) return fail(ALA_INVALID_SHAPE, "cuSeqLen must be [batch + 1]");
  if (!is_vector(freeCount, 1) || !is_vector(freeCountOut, 1) || !is_vector(status, 1))
    return fail(ALA_INVALID_SHAPE, "freeCount, freeCountOut and status must be [1]");
  if (freeBlocks->ndim != 1) return fail(ALA_INVALID_SHAPE, "freeBlocks must be [numBlocks]");
  if (slotMapping->ndim != 1 || !is_vector(positions, slotMapping->dims[0]))
    return fail(ALA_INVALID_SHAPE, "slotMapping and positions must both be [nTokens]");
  if (batch > kPagedStepMaxBatch) return fail(ALA_UNSUPPORTED, "more than %d requests", kPagedStepMaxBatch);
  if (slotMapping->dims[0] > kMaxKeys) return fail(ALA_UNSUPPORTED, "more than 2^30 tokens");
  if (max_blocks > kMaxKeys / blockSize || freeBlocks->dims[0] > kMaxKeys / blockSize)
    return fail(ALA_UNSUPPORTED, "maxBlockNum * blockSize and numBlocks * blockSize must be at most 2^30");
  // kvSeqLen may be contextLens and freeCountOut freeCount (updated in place); every other output stands alone
  const ala_tensor* outs[] = {kvSeqLen, freeCountOut, cuSeqLen, slotMapping, positions, status, blockTables, freeBlocks};
  const ala_tensor* rest[] = {seqLen, contextLens, finished, freeCount};
  auto span = [](const ala_tensor* t) {
    int64_t n = 4;
    for (int i = 0; i < t->ndim; ++i) n *= t->dims[i];
    return Span(t->data, n);
  };
  auto overlap = [&](const ala_tensor* x, const ala_tensor* y) { return span(x).shares(span(y)); };
  for (size_t i = 0; i < sizeof outs / sizeof *outs; ++i) {
    for (size_t j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return fail(ALA_INVALID_PARAM, "two outputs overlap");
    for (const ala_tensor* t : rest) {
      if (!t || !overlap(outs[i], t)) continue;
      const bool in_place = outs[i]->data == t->data && ((outs[i] == kvSeqLen && t == contextLens) ||
                                                         (outs[i] == freeCountOut && t == freeCount));
      if (!in_place) return fail(ALA_INVALID_PARAM, "an output overlaps an input (only kvSeqLen = contextLens and "
                                                    "freeCountOut = freeCount may be the same memory)");
    }
  }
  auto in = [](const ala_tensor* t) { return t ? static_cast<const int32_t*>(t->data) : nullptr; };
  auto io = [](ala_tensor* t) { return static_cast<int32_t*>(t->data); };
  PagedStepArgs a{};
  a.seq_len = in(seqLen);
  a.finished = in(finished);
  a.context_len = in(contextLens);
  a.block_tables = io(blockTables);
  a.free_blocks = io(freeBlocks);
  a.free_count = in(freeCount);
  a.kv_seq_len = io(kvSeqLen);
  a.free_count_out = io(freeCountOut);
  a.cu_seq_len = io(cuSeqLen);
  a.slot_mapping = io(slotMapping);
  a.positions = io(positions);
  a.status = io(status);
  a.batch = (int32_t)batch;
  a.max_blocks = (int32_t)max_blocks;
  a.block_size = blockSize;
  a.capacity = (int32_t)freeBlocks->dims[0];
  a.n_tokens = (int32_t)slotMapping->dims[0];
  const cudaError_t e = launch_paged_step(a, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(ALA_CUDA_ERROR, "%s", cudaGetErrorString(e));
  set_last_error("");
  return ALA_OK;
}

extern "C" int ala_paged_write(const ala_tensor* key, int64_t keyStride, const ala_tensor* value, int64_t valueStride,
                               const ala_tensor* slotMapping, ala_tensor* keyCache, ala_tensor* valueCache,
                               ala_stream_t stream) {
  NvtxRange nvtx_range("ala_paged_write");
  const Report fail{"ala_paged_write"};
  if (!key || !slotMapping || !keyCache) return fail(ALA_NULL_REQUIRED, "key, slotMapping and keyCache are required");
  if (!value != !valueCache) return fail(ALA_NULL_REQUIRED, "value and valueCache come together");
  for (const ala_tensor* t : {key, value, slotMapping, (const ala_tensor*)keyCache, (const ala_tensor*)valueCache})
    if (t && !header_ok(t)) return fail(ALA_INVALID_SHAPE, "tensor with bad ndim or dims");
  if (slotMapping->dtype != ALA_I32) return fail(ALA_INVALID_DTYPE, "slotMapping must be int32");
  if (slotMapping->ndim != 1) return fail(ALA_INVALID_SHAPE, "slotMapping must be [nTokens]");
  const int64_t n = slotMapping->dims[0];
  if (n > kMaxKeys) return fail(ALA_UNSUPPORTED, "more than 2^30 tokens");
  PagedWriteArgs a{};
  int64_t blocks[2] = {0, 0}, block_size[2] = {0, 0};
  const ala_tensor *rows[2] = {key, value}, *caches[2] = {keyCache, valueCache};
  const int64_t strides[2] = {keyStride, valueStride};
  int64_t stride_bytes[2] = {0, 0}, row_bytes[2] = {0, 0};
  for (int i = 0; i < 2 && rows[i]; ++i) {
    const char* what = i ? "value" : "key";
    const int es = elem_bytes(rows[i]->dtype);
    if (es == 0) return fail(ALA_INVALID_DTYPE, "%s has an unknown dtype", what);
    if (caches[i]->dtype != rows[i]->dtype) return fail(ALA_INVALID_DTYPE, "%s and its cache differ in dtype", what);
    int64_t row = 0;
    if (!cache_dims(caches[i], blocks + i, block_size + i, &row))
      return fail(ALA_INVALID_SHAPE, "the %s cache must be [numBlocks, blockSize, ...] with at most 2^30 rows", what);
    if ((rows[i]->ndim != 2 && rows[i]->ndim != 3) || rows[i]->dims[0] != n || row_elems(rows[i], 1) != row)
      return fail(ALA_INVALID_SHAPE, "%s must be [nTokens, ...] with the cache's rows of %lld elements", what, (long long)row);
    const int64_t stride = strides[i] ? strides[i] : row;
    if (stride < row || stride >= kMaxElems)
      return fail(ALA_INVALID_PARAM, "the %s stride must be 0 or at least a row (%lld elements, got %lld)", what,
                  (long long)row, (long long)stride);
    stride_bytes[i] = stride * es;
    row_bytes[i] = row * es;
    if ((n > 0 && row > 0 && !rows[i]->data) || (blocks[i] > 0 && row > 0 && !caches[i]->data))
      return fail(ALA_NULL_REQUIRED, "%s or its cache has a NULL data pointer", what);
    if (!aligned(rows[i]->data, es) || !aligned(caches[i]->data, es))
      return fail(ALA_INVALID_PARAM, "%s or its cache is not aligned to its elements", what);
  }
  if (value && (blocks[0] != blocks[1] || block_size[0] != block_size[1]))
    return fail(ALA_INVALID_SHAPE, "the key and value caches differ in blocks");
  if (n > 0 && !slotMapping->data) return fail(ALA_NULL_REQUIRED, "slotMapping has a NULL data pointer");
  if (!aligned(slotMapping->data, 4)) return fail(ALA_INVALID_PARAM, "slotMapping is not aligned to its elements");
  const int64_t n_slots = blocks[0] * block_size[0];
  for (int i = 0; i < 2 && rows[i]; ++i) {
    const Span cache(caches[i]->data, n_slots, row_bytes[i], row_bytes[i]);
    bool shared = cache.shares(Span(slotMapping->data, 4 * n));
    for (int j = 0; j < 2 && rows[j]; ++j) {
      shared = shared || cache.shares(Span(rows[j]->data, n, stride_bytes[j], row_bytes[j]));
      shared = shared || (j < i && cache.shares(Span(caches[j]->data, n_slots, row_bytes[j], row_bytes[j])));
    }
    if (shared) return fail(ALA_INVALID_PARAM, "the %s cache overlaps another tensor", i ? "value" : "key");
  }
  a.key = static_cast<const uint8_t*>(key->data);
  a.value = value ? static_cast<const uint8_t*>(value->data) : nullptr;
  a.key_cache = static_cast<uint8_t*>(keyCache->data);
  a.value_cache = value ? static_cast<uint8_t*>(valueCache->data) : nullptr;
  a.slots = static_cast<const int32_t*>(slotMapping->data);
  a.key_stride = stride_bytes[0];
  a.value_stride = stride_bytes[1];
  a.key_row = row_bytes[0];
  a.value_row = row_bytes[1];
  a.n_tokens = n;
  a.n_slots = n_slots;
  const cudaError_t e = launch_paged_write(a, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(ALA_CUDA_ERROR, "%s", cudaGetErrorString(e));
  set_last_error("");
  return ALA_OK;
}
