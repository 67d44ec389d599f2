// The C ABI of the paged 4-bit cache (declared in include/raattn.h): argument validation and dispatch.  Nothing
// here allocates device memory.
#include <climits>
#include <cmath>

#include "paged.cuh"

namespace raattn {
namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool dtype_ok(ra_dtype_t t) { return t == RA_F32 || t == RA_BF16; }
bool fits(int64_t a, int64_t b) { return a * b <= INT_MAX; }

// The most tokens of a sequence: loops over its blocks step by less than 16384 tokens in 32 bits.
constexpr int kMostTokens = INT_MAX - 16384;

int shift_of(int page) {
  for (int s = 4; s <= 8; ++s)
    if (page == 1 << s) return s;
  return -1;
}

// A pool's description, of keys and values with (D > 0) a known layout.
ra_status_t pool_of(PagePool* p, const void* pool, int64_t page_stride, int pages, int page, int Hkv, int D, int M) {
  if (!pool || !aligned(pool, 16) || page_stride % 16 || pages < 1 || page < 1 || Hkv < 1 || D < 1 || M < 1) return RA_ERR_ARG;
  if (shift_of(page) < 0 || (D != 64 && D != 128)) return RA_ERR_UNSUPPORTED;
  const int part = page * paged::row_bytes(D);
  if (Hkv > INT_MAX / (2 * part) || (pages > 1 && page_stride < static_cast<int64_t>(2) * Hkv * part)) return RA_ERR_ARG;
  if (static_cast<int64_t>(M) * page > kMostTokens || page_stride > INT_MAX) return RA_ERR_ARG;
  *p = PagePool{static_cast<uint8_t*>(const_cast<void*>(pool)), static_cast<int>(pages > 1 ? page_stride : 0), part, pages, Hkv, D,
                page, shift_of(page)};
  return RA_OK;
}

ra_status_t rows_of(PageRows* a, const void* pool, int64_t page_stride, const int32_t* table, const int32_t* start,
                    const int32_t* limit, int B, int N, int Hkv, int D, int pages, int page, int M, ra_dtype_t dtype) {
  if (!table || !aligned(table, 4) || !aligned(start, 4) || !aligned(limit, 4) || !dtype_ok(dtype)) return RA_ERR_ARG;
  if (B < 1 || N < 1) return RA_ERR_ARG;
  const ra_status_t s = pool_of(&a->pool, pool, page_stride, pages, page, Hkv, D, M);
  if (s != RA_OK) return s;
  if (!fits(B, M) || !fits(B, Hkv) || !fits(static_cast<int64_t>(B) * Hkv, N) ||
      !fits(static_cast<int64_t>(B) * Hkv * N, 2 * (D / paged::kGroup)))
    return RA_ERR_ARG;
  a->table = table;
  a->M = M;
  a->start = start;
  a->limit = limit;
  a->B = B;
  a->N = N;
  return RA_OK;
}

ra_status_t decode_of(PagedDecodeArgs* p, int B, int Hq, int Hkv, int M, int page, int D) {
  if (B < 1 || Hq < 1 || Hkv < 1 || M < 1 || page < 1 || D < 1 || Hq % Hkv) return RA_ERR_ARG;
  if (!fits(B, Hq) || !fits(B, M) || static_cast<int64_t>(M) * page > kMostTokens) return RA_ERR_ARG;
  if (shift_of(page) < 0 || (D != 64 && D != 128) || B > kDecodeMaxBatch || Hq / Hkv > 1024) return RA_ERR_UNSUPPORTED;
  p->a = DecodeArgs{};
  p->a.B = B;
  p->a.Hq = Hq;
  p->a.Hkv = Hkv;
  p->a.C = M * page;
  p->a.D = D;
  p->M = M;
  return RA_OK;
}

int per_row_of(int tokens, int page) { return (tokens + page - 2) / page + 1; }
size_t padded(int64_t ints) { return (static_cast<size_t>(ints) * 4 + 255) & ~static_cast<size_t>(255); }

}  // namespace
}  // namespace raattn

using namespace raattn;

extern "C" {

ra_status_t ra_page_write(const void* k, const void* v, const int64_t* k_strides, const int64_t* v_strides, void* pool,
                          int64_t page_stride, const int32_t* table, const int32_t* start, const int32_t* count,
                          void* k_held, void* v_held, int B, int N, int H_KV, int D, int pages, int page, int M,
                          ra_dtype_t dtype, void* stream) {
  PageRows a{};
  if (!k || !v || !k_strides || !v_strides || !k_held != !v_held) return RA_ERR_ARG;
  const void* const data[4] = {k, v, k_held, v_held};
  for (const void* p : data)
    if (!aligned(p, 16)) return RA_ERR_ARG;
  const ra_status_t s = rows_of(&a, pool, page_stride, table, start, count, B, N, H_KV, D, pages, page, M, dtype);
  if (s != RA_OK) return s;
  const int vec = dtype == RA_BF16 ? 8 : 4;
  for (int i = 0; i < 3; ++i) {
    if (k_strides[i] % vec || v_strides[i] % vec) return RA_ERR_ARG;
    a.k_stride[i] = k_strides[i];
    a.v_stride[i] = v_strides[i];
  }
  a.k = k;
  a.v = v;
  a.k_out = k_held;
  a.v_out = v_held;
  return launch_page_write(a, dtype == RA_BF16, static_cast<cudaStream_t>(stream)) == cudaSuccess ? RA_OK : RA_ERR_LAUNCH;
}

ra_status_t ra_page_read(const void* pool, int64_t page_stride, const int32_t* table, const int32_t* start,
                         const int32_t* length, void* k, void* v, int B, int N, int H_KV, int D, int pages, int page,
                         int M, ra_dtype_t dtype, void* stream) {
  PageRows a{};
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16)) return RA_ERR_ARG;
  const ra_status_t s = rows_of(&a, pool, page_stride, table, start, length, B, N, H_KV, D, pages, page, M, dtype);
  if (s != RA_OK) return s;
  a.k_out = k;
  a.v_out = v;
  return launch_page_read(a, dtype == RA_BF16, static_cast<cudaStream_t>(stream)) == cudaSuccess ? RA_OK : RA_ERR_LAUNCH;
}

size_t ra_attention_decode_paged_workspace_size(int B, int H_Q, int H_KV, int M, int page, int D) {
  PagedDecodeArgs p{};
  if (decode_of(&p, B, H_Q, H_KV, M, page, D) != RA_OK) return 0;
  const size_t wide = plan_decode_paged(&p, false, nullptr), narrow = plan_decode_paged(&p, true, nullptr);   // of either dtype
  return wide > narrow ? wide : narrow;
}

ra_status_t ra_attention_decode_paged(const void* q, const void* pool, int64_t page_stride, const int32_t* table,
                                      const int32_t* length, void* o, void* workspace, int B, int H_Q, int H_KV, int D,
                                      int pages, int page, int M, float scale, ra_dtype_t dtype, void* stream) {
  if (!q || !table || !length || !o || !workspace || !dtype_ok(dtype)) return RA_ERR_ARG;
  const void* const data[3] = {q, o, workspace};
  for (const void* p : data)
    if (!aligned(p, 16)) return RA_ERR_ARG;
  if (!aligned(table, 4) || !aligned(length, 4)) return RA_ERR_ARG;
  PagedDecodeArgs p{};
  ra_status_t s = decode_of(&p, B, H_Q, H_KV, M, page, D);
  if (s == RA_ERR_ARG) return s;
  const ra_status_t sp = pool_of(&p.pool, pool, page_stride, pages, page, H_KV, D, M);
  if (sp != RA_OK) return sp;
  if (!std::isfinite(scale)) return RA_ERR_ARG;   // NaN is no default
  if (scale <= 0.0f) scale = 1.0f / std::sqrt(static_cast<float>(D));
  if (s != RA_OK) return s;
  p.table = table;
  p.a.q = q;
  p.a.o = o;
  p.a.length = length;
  p.a.scale = scale;
  if (plan_decode_paged(&p, dtype == RA_BF16, static_cast<char*>(workspace)) == 0) return RA_ERR_UNSUPPORTED;
  return launch_decode_paged(p, dtype == RA_BF16, static_cast<cudaStream_t>(stream)) == cudaSuccess ? RA_OK : RA_ERR_LAUNCH;
}

ra_status_t ra_page_fork(int32_t* table, int32_t* length, int32_t* uses, const int32_t* parent, int B, int M, int pages,
                         void* stream) {
  if (!table || !length || !uses || !parent || B < 1 || M < 1 || pages < 1 || !fits(B, M)) return RA_ERR_ARG;
  const int32_t* const data[4] = {table, length, uses, parent};
  for (const int32_t* p : data)
    if (!aligned(p, 4)) return RA_ERR_ARG;
  if (B > kMostForkRows) return RA_ERR_UNSUPPORTED;
  const PageFork a{table, length, uses, parent, B, M, pages};
  return launch_page_fork(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? RA_OK : RA_ERR_LAUNCH;
}

size_t ra_page_reserve_workspace_size(int B, int tokens, int page) {
  if (B < 1 || tokens < 1 || shift_of(page) < 0 || tokens > kMostTokens || !fits(B, per_row_of(tokens, page))) return 0;
  return 2 * padded(static_cast<int64_t>(B) * per_row_of(tokens, page)) + padded(2ll * B);
}

ra_status_t ra_page_reserve(void* pool, int64_t page_stride, int64_t page_bytes, int32_t* table, const int32_t* length,
                            int32_t* uses, const int32_t* count, int32_t* granted, void* workspace, int B, int M,
                            int tokens, int pages, int page, void* stream) {
  if (!pool || !table || !length || !uses || !granted || !workspace) return RA_ERR_ARG;
  const int32_t* const data[5] = {table, length, uses, count, granted};
  for (const int32_t* p : data)
    if (!aligned(p, 4)) return RA_ERR_ARG;
  if (!aligned(pool, 16) || !aligned(workspace, 16) || page_stride % 16 || page_bytes % 16 || page_bytes < 16) return RA_ERR_ARG;
  if (B < 1 || M < 1 || tokens < 1 || pages < 1 || page < 1 || (pages > 1 && page_stride < page_bytes)) return RA_ERR_ARG;
  if (!fits(B, M) || static_cast<int64_t>(M) * page > kMostTokens || tokens > kMostTokens) return RA_ERR_ARG;
  if (page_stride > INT_MAX) return RA_ERR_ARG;
  if (shift_of(page) < 0) return RA_ERR_UNSUPPORTED;
  const int per_row = per_row_of(tokens, page);
  if (!fits(B, per_row)) return RA_ERR_ARG;
  PageReserve a{};
  a.pool = PagePool{static_cast<uint8_t*>(pool), static_cast<int>(page_stride), 0, pages, 0, 0, page, shift_of(page)};
  a.table = table;
  a.uses = uses;
  a.granted = granted;
  a.length = length;
  a.count = count;
  a.B = B;
  a.M = M;
  a.tokens = tokens;
  a.per_row = per_row;
  a.page_bytes = page_bytes;
  char* w = static_cast<char*>(workspace);
  a.place = reinterpret_cast<int32_t*>(w);
  a.freed = reinterpret_cast<int32_t*>(w + padded(static_cast<int64_t>(B) * per_row));
  a.copy = reinterpret_cast<int32_t*>(w + 2 * padded(static_cast<int64_t>(B) * per_row));
  return launch_page_reserve(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? RA_OK : RA_ERR_LAUNCH;
}

size_t ra_page_compact_workspace_size(int pages) { return pages < 1 ? 0 : 2 * padded(pages); }

ra_status_t ra_page_compact(const void* pool, int64_t page_stride, const int32_t* table, const int32_t* uses,
                            void* pool_out, int64_t page_stride_out, int32_t* table_out, int32_t* uses_out,
                            int32_t* live, void* workspace, int64_t page_bytes, int B, int M, int pages, int pages_out,
                            void* stream) {
  if (!pool || !table || !uses || !pool_out || !table_out || !uses_out || !live || !workspace) return RA_ERR_ARG;
  const int32_t* const data[5] = {table, uses, table_out, uses_out, live};
  for (const int32_t* p : data)
    if (!aligned(p, 4)) return RA_ERR_ARG;
  const void* const wide[3] = {pool, pool_out, workspace};
  for (const void* p : wide)
    if (!aligned(p, 16)) return RA_ERR_ARG;
  if (page_stride % 16 || page_stride_out % 16 || page_bytes % 16 || page_bytes < 16) return RA_ERR_ARG;
  if (B < 1 || M < 1 || pages < 1 || pages_out < 1 || !fits(B, M)) return RA_ERR_ARG;
  if ((pages > 1 && page_stride < page_bytes) || (pages_out > 1 && page_stride_out < page_bytes)) return RA_ERR_ARG;
  if (pool == pool_out || table == table_out || uses == uses_out) return RA_ERR_ARG;
  char* w = static_cast<char*>(workspace);
  const PageCompact a{static_cast<const uint8_t*>(pool), static_cast<uint8_t*>(pool_out), page_stride, page_stride_out,
                      page_bytes, table, uses, table_out, uses_out, live, B, M, pages, pages_out,
                      reinterpret_cast<int32_t*>(w), reinterpret_cast<int32_t*>(w + padded(pages))};
  return launch_page_compact(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? RA_OK : RA_ERR_LAUNCH;
}

}  // extern "C"
