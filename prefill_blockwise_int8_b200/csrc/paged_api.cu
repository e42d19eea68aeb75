// C entry points of the rotary and paged-cache calls (include/tilemix.h):
// argument checks, tensor maps, dispatch.  Host code only; allocates nothing.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "api_common.h"
#include "paged.h"
#include "tilemix.h"

using tilemix::aligned;
using tilemix::check_device;
using tilemix::encode_fn;
using tilemix::fail;
using tilemix::ok;

namespace {

bool power_of_two(int x) { return x > 0 && (x & (x - 1)) == 0; }

int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

// A strided tensor argument: 16-byte base, strides multiples of `unit`
// elements (16 bytes).
bool rows_ok(const void* p, int64_t st, int64_t sh, int unit) {
  return aligned(p, 16) && st % unit == 0 && sh % unit == 0 && st >= 0 && sh >= 0;
}

// The rows of a page or an output may not overlap: one axis steps over all that
// the other spans (strides of axes of one are not used).
bool apart(int64_t st, int64_t sh, int tokens, int heads, int d) {
  if (tokens <= 1) return heads <= 1 || sh >= d;
  if (heads <= 1) return st >= d;
  // (in double: a stride may be anything)
  const double span_t = d + static_cast<double>(st) * (tokens - 1);
  const double span_h = d + static_cast<double>(sh) * (heads - 1);
  return st < sh ? st >= d && sh >= span_t : sh >= d && st >= span_h;
}

// Shared checks of the cache arguments.
tilemix_status check_cache(const char* where, int kv_format, const void* k_pages,
                           const void* v_pages, int64_t page_stride,
                           int64_t token_stride, int64_t head_stride,
                           const float* k_scale, const float* v_scale,
                           const int32_t* page_table, int64_t table_stride,
                           const int32_t* cu_seqlens, const int32_t* kv_lens,
                           int batch, int total_tokens, int num_pages,
                           int page_size, int max_pages, int hkv, int head_dim,
                           const int32_t* status) {
  if (kv_format != TILEMIX_KV_FP16 && kv_format != TILEMIX_KV_INT8)
    return fail(TILEMIX_ERR_INVALID_ARG, "%s: bad kv_format %d", where, kv_format);
  const bool int8 = kv_format == TILEMIX_KV_INT8;
  if (batch < 0 || total_tokens < 0 || num_pages < 0 || max_pages < 0 || hkv <= 0)
    return fail(TILEMIX_ERR_INVALID_ARG, "%s: bad size", where);
  if (head_dim != 64 && head_dim != 128)
    return fail(TILEMIX_ERR_UNSUPPORTED, "%s: head_dim %d not in {64, 128}",
                where, head_dim);
  if (!power_of_two(page_size) || page_size < 16 || page_size > 256)
    return fail(TILEMIX_ERR_UNSUPPORTED,
                "%s: page_size %d not a power of two in [16, 256]", where,
                page_size);
  // positions are int32 and the kernels look up to 1023 keys past the last one
  if (static_cast<long long>(max_pages) * page_size > (1ll << 31) - 1024)
    return fail(TILEMIX_ERR_UNSUPPORTED,
                "%s: max_pages * page_size above 2^31 - 1024", where);
  if (batch == 0 || total_tokens == 0) return ok();
  if (!k_pages || !v_pages || !page_table || !cu_seqlens || !kv_lens ||
      (int8 && (!k_scale || !v_scale)))
    return fail(TILEMIX_ERR_INVALID_ARG, "%s: null pointer", where);
  if (num_pages == 0 || max_pages == 0)
    return fail(TILEMIX_ERR_INVALID_ARG, "%s: num_pages and max_pages must be positive",
                where);
  const int unit = int8 ? 16 : 8;
  if (!rows_ok(k_pages, token_stride, head_stride, unit) ||
      !rows_ok(v_pages, page_stride, 0, unit))
    return fail(TILEMIX_ERR_INVALID_ARG,
                "%s: pages must be 16-byte aligned with strides of whole 16 bytes",
                where);
  if (token_stride < head_dim || (hkv > 1 && head_stride < head_dim) ||
      (num_pages > 1 && page_stride < head_dim))
    return fail(TILEMIX_ERR_INVALID_ARG, "%s: page strides below head_dim", where);
  if (table_stride < max_pages)
    return fail(TILEMIX_ERR_INVALID_ARG, "%s: table_stride below max_pages", where);
  if (!aligned(page_table, 4) || !aligned(cu_seqlens, 4) || !aligned(kv_lens, 4) ||
      (k_scale && !aligned(k_scale, 16)) || (v_scale && !aligned(v_scale, 16)) ||
      (status && !aligned(status, 4)))
    return fail(TILEMIX_ERR_INVALID_ARG, "%s: misaligned pointer", where);
  return ok();
}

tilemix_status check_heads(const char* where, int hq, int hkv) {
  if (hq <= 0 || hkv <= 0 || hq % hkv != 0)
    return fail(TILEMIX_ERR_INVALID_ARG, "%s: hq %d not a multiple of hkv %d",
                where, hq, hkv);
  if (hq / hkv > 128)
    return fail(TILEMIX_ERR_UNSUPPORTED,
                "%s: more than 128 query heads per KV head", where);
  return ok();
}

// Packed rows of a sequence are counted in int32.
bool too_many_rows(int max_q_len, int group) {
  return static_cast<long long>(max_q_len) * group > (1ll << 30);
}

// Which attention kernel: the step kernel reads the cache once per 16 packed
// rows, the chunk kernel once per 256 but with more to begin and end.  Step
// against chunk, us in a graph, 8 KV heads, at 16 / 24 rows (INT8, whose chunk
// kernel converts tiles first: at 16 / 32):
//                          d 64                    d 128
//   16 x 6000 keys   49 : 62 / 67 : 62       77 : 75 / 125 : 76
//   1 x 32000        23 : 30 / 27 : 30       37 : 38 / 54 : 38
//   64 x 1000        41 : 56 / 61 : 56       60 : 66 / 99 : 67
//   4 x 500          13 : 13 / 13 : 13       13 : 14 / 16 : 14
//   INT8 16 x 6000   39 : 109 / 61 : 110     58 : 128 / 93 : 129
//   INT8 1 x 32000   26 : 47 / 31 : 47       32 : 50 / 42 : 51
//   INT8 64 x 1000   35 : 106 / 55 : 106     54 : 131 / 84 : 132
//   INT8 4 x 500     13 : 17 / 14 : 17       16 : 18 / 17 : 19
bool use_step(int max_q_len, int group, bool int8) {
  return static_cast<long long>(max_q_len) * group <= (int8 ? 32 : 16);
}

// {d, page_size, hkv, num_pages} map over a page array.
bool make_pages_map(CUtensorMap* m, const void* base, bool int8, bool bf16,
                    int d, int page_size, int hkv, int num_pages,
                    int64_t page_stride, int64_t token_stride,
                    int64_t head_stride, int box_tokens,
                    CUtensorMapSwizzle sw) {
  auto enc = encode_fn();
  if (!enc) return false;
  const int e = int8 ? 1 : 2;
  // the stride of an axis of one is never used, but has to be valid
  if (hkv == 1) head_stride = token_stride;
  if (num_pages == 1) page_stride = token_stride;
  const cuuint64_t dims[4] = {
      static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(page_size),
      static_cast<cuuint64_t>(hkv), static_cast<cuuint64_t>(num_pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(token_stride) * e,
                                 static_cast<cuuint64_t>(head_stride) * e,
                                 static_cast<cuuint64_t>(page_stride) * e};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(int8 ? d : 64),
                             static_cast<cuuint32_t>(box_tokens), 1u, 1u};
  const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
  return enc(m,
             int8   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
             : bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                    : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
             4, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
             CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

extern "C" {

tilemix_status tilemix_rope_frequencies(int scaling, int rot_dim, double base,
                                        double factor, double low_freq_factor,
                                        double high_freq_factor,
                                        int original_max_position,
                                        double* freqs, float* attn_factor) {
  if (!freqs)
    return fail(TILEMIX_ERR_INVALID_ARG, "rope_frequencies: null freqs");
  if (scaling < TILEMIX_ROPE_SCALE_NONE || scaling > TILEMIX_ROPE_SCALE_YARN)
    return fail(TILEMIX_ERR_INVALID_ARG, "rope_frequencies: bad scaling %d", scaling);
  if (rot_dim <= 0 || rot_dim % 2 != 0 ||
      (scaling == TILEMIX_ROPE_SCALE_NTK && rot_dim <= 2))
    return fail(TILEMIX_ERR_INVALID_ARG, "rope_frequencies: bad rot_dim %d", rot_dim);
  if (!(base > 1.0) || !(factor > 0.0) || std::isinf(base) || std::isinf(factor))
    return fail(TILEMIX_ERR_INVALID_ARG,
                "rope_frequencies: base must exceed 1 and factor 0");
  const bool banded = scaling == TILEMIX_ROPE_SCALE_WAVELENGTH ||
                      scaling == TILEMIX_ROPE_SCALE_YARN;
  if (banded && (original_max_position <= 0 || !(low_freq_factor > 0.0) ||
                 !(high_freq_factor > low_freq_factor)))
    return fail(TILEMIX_ERR_INVALID_ARG,
                "rope_frequencies: original_max_position and 0 < "
                "low_freq_factor < high_freq_factor are required");
  const double pi = 3.14159265358979323846;
  const double n = original_max_position;
  if (scaling == TILEMIX_ROPE_SCALE_NTK)
    base *= std::pow(factor, double(rot_dim) / (rot_dim - 2));
  auto turn_dim = [&](double rotations) {
    return rot_dim * std::log(n / (rotations * 2.0 * pi)) / (2.0 * std::log(base));
  };
  double lo = 0.0, hi = 0.0;
  if (scaling == TILEMIX_ROPE_SCALE_YARN) {
    lo = std::fmax(std::floor(turn_dim(high_freq_factor)), 0.0);
    hi = std::fmin(std::ceil(turn_dim(low_freq_factor)), rot_dim - 1.0);
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / rot_dim);
    double r = f;
    if (scaling == TILEMIX_ROPE_SCALE_LINEAR) {
      r = f / factor;
    } else if (scaling == TILEMIX_ROPE_SCALE_WAVELENGTH) {
      const double t =
          std::fmin(std::fmax((n * f / (2.0 * pi) - low_freq_factor) /
                                  (high_freq_factor - low_freq_factor),
                              0.0),
                    1.0);
      r = (1.0 - t) * f / factor + t * f;
    } else if (scaling == TILEMIX_ROPE_SCALE_YARN) {
      const double t = std::fmin(
          std::fmax((i - lo) / std::fmax(hi - lo, 0.001), 0.0), 1.0);
      r = t * f / factor + (1.0 - t) * f;
    }
    freqs[i] = r;
  }
  if (attn_factor)
    *attn_factor = scaling == TILEMIX_ROPE_SCALE_YARN && factor > 1.0
                       ? static_cast<float>(0.1 * std::log(factor) + 1.0)
                       : 1.0f;
  return ok();
}

tilemix_status tilemix_rope(const tilemix_rope_params* a, tilemix_stream_t stream) {
  if (!a) return fail(TILEMIX_ERR_INVALID_ARG, "rope: params is NULL");
  if (a->struct_size != sizeof(tilemix_rope_params))
    return fail(TILEMIX_ERR_INVALID_ARG,
                "rope: struct_size %u != sizeof(tilemix_rope_params) %zu",
                a->struct_size, sizeof(tilemix_rope_params));
  if ((a->dtype != TILEMIX_FP16 && a->dtype != TILEMIX_BF16) ||
      (a->layout != TILEMIX_ROPE_HALF && a->layout != TILEMIX_ROPE_INTERLEAVED) ||
      (a->inverse != 0 && a->inverse != 1))
    return fail(TILEMIX_ERR_INVALID_ARG, "rope: bad dtype, layout or inverse");
  if (a->total_tokens < 0 || a->hq <= 0 || (a->k && a->hkv <= 0) ||
      static_cast<long long>(a->hq) + (a->k ? a->hkv : 0) > 65535)
    return fail(TILEMIX_ERR_INVALID_ARG, "rope: bad size");
  if (a->head_dim <= 0 || a->head_dim > 256 || a->head_dim % 16 != 0)
    return fail(TILEMIX_ERR_UNSUPPORTED,
                "rope: head_dim %d must be a multiple of 16 in [16, 256]",
                a->head_dim);
  if (a->rot_dim <= 0 || a->rot_dim > a->head_dim || a->rot_dim % 16 != 0)
    return fail(TILEMIX_ERR_UNSUPPORTED,
                "rope: rot_dim %d must be a multiple of 16 in [16, head_dim]",
                a->rot_dim);
  if (!(std::isfinite(a->attn_factor) && a->attn_factor >= 0.0f))
    return fail(TILEMIX_ERR_INVALID_ARG, "rope: bad attn_factor");
  if (a->total_tokens == 0) return ok();
  if (!a->q || !a->q_out || !a->positions || !a->freqs || (a->k && !a->k_out))
    return fail(TILEMIX_ERR_INVALID_ARG, "rope: null pointer");
  if (!rows_ok(a->q, a->q_stride_t, a->q_stride_h, 8) ||
      !rows_ok(a->q_out, a->q_out_stride_t, a->q_out_stride_h, 8) ||
      (a->k && (!rows_ok(a->k, a->k_stride_t, a->k_stride_h, 8) ||
                !rows_ok(a->k_out, a->k_out_stride_t, a->k_out_stride_h, 8))) ||
      !aligned(a->positions, 4) || !aligned(a->freqs, 8))
    return fail(TILEMIX_ERR_INVALID_ARG,
                "rope: misaligned pointer or a stride that is not a multiple "
                "of 8 elements");
  if (!apart(a->q_out_stride_t, a->q_out_stride_h, a->total_tokens, a->hq, a->head_dim) ||
      (a->k && !apart(a->k_out_stride_t, a->k_out_stride_h, a->total_tokens,
                      a->hkv, a->head_dim)))
    return fail(TILEMIX_ERR_INVALID_ARG, "rope: output rows overlap");
  tilemix_status d = check_device();
  if (d != TILEMIX_OK) return d;
  tilemix::RopeArgs r;
  memset(&r, 0, sizeof(r));
  auto rows = [](const void* p, int64_t st, int64_t sh) {
    return tilemix::RowTensor{static_cast<uint16_t*>(const_cast<void*>(p)), st, sh};
  };
  r.q = rows(a->q, a->q_stride_t, a->q_stride_h);
  r.q_out = rows(a->q_out, a->q_out_stride_t, a->q_out_stride_h);
  r.k = rows(a->k, a->k_stride_t, a->k_stride_h);
  r.k_out = rows(a->k_out, a->k_out_stride_t, a->k_out_stride_h);
  r.positions = a->positions;
  r.freqs = a->freqs;
  r.attn_factor = a->attn_factor > 0.0f ? a->attn_factor : 1.0f;
  r.sign = a->inverse ? -1.0f : 1.0f;
  r.total_tokens = a->total_tokens;
  r.hq = a->hq;
  r.hk = a->k ? a->hkv : 0;
  r.head_dim = a->head_dim;
  r.rot_dim = a->rot_dim;
  r.interleaved = a->layout == TILEMIX_ROPE_INTERLEAVED;
  const cudaError_t e = tilemix::launch_rope(r, a->dtype == TILEMIX_BF16, 0, stream);
  if (e != cudaSuccess)
    return fail(TILEMIX_ERR_CUDA, "rope launch: %s", cudaGetErrorString(e));
  return ok();
}

tilemix_status tilemix_paged_append(const tilemix_append_params* a,
                                    tilemix_stream_t stream) {
  const char* where = "paged_append";
  if (!a) return fail(TILEMIX_ERR_INVALID_ARG, "%s: params is NULL", where);
  if (a->struct_size != sizeof(tilemix_append_params))
    return fail(TILEMIX_ERR_INVALID_ARG,
                "%s: struct_size %u != sizeof(tilemix_append_params) %zu", where,
                a->struct_size, sizeof(tilemix_append_params));
  if ((a->dtype != TILEMIX_FP16 && a->dtype != TILEMIX_BF16) ||
      (a->layout != TILEMIX_ROPE_HALF && a->layout != TILEMIX_ROPE_INTERLEAVED))
    return fail(TILEMIX_ERR_INVALID_ARG, "%s: bad dtype or layout", where);
  tilemix_status st = check_cache(
      where, a->kv_format, a->k_pages, a->v_pages, a->page_stride,
      a->token_stride, a->head_stride, a->k_scale, a->v_scale, a->page_table,
      a->table_stride, a->cu_seqlens, a->kv_lens, a->batch, a->total_tokens,
      a->num_pages, a->page_size, a->max_pages, a->hkv, a->head_dim, a->status);
  if (st != TILEMIX_OK) return st;
  if ((a->q && a->hq <= 0) ||
      2ll * a->hkv + (a->q ? a->hq : 0) > 65535)
    return fail(TILEMIX_ERR_INVALID_ARG, "%s: bad head count", where);
  if (a->freqs && (a->rot_dim <= 0 || a->rot_dim > a->head_dim || a->rot_dim % 16))
    return fail(TILEMIX_ERR_UNSUPPORTED,
                "%s: rot_dim %d must be a multiple of 16 in [16, head_dim]",
                where, a->rot_dim);
  if (a->q && (!a->freqs || !a->q_out))
    return fail(TILEMIX_ERR_INVALID_ARG, "%s: q needs freqs and q_out", where);
  if (!(std::isfinite(a->attn_factor) && a->attn_factor >= 0.0f))
    return fail(TILEMIX_ERR_INVALID_ARG, "%s: bad attn_factor", where);
  if (a->batch == 0 || a->total_tokens == 0) return ok();
  if (!a->k || !a->v)
    return fail(TILEMIX_ERR_INVALID_ARG, "%s: null pointer", where);
  if (!rows_ok(a->k, a->k_stride_t, a->k_stride_h, 8) ||
      !rows_ok(a->v, a->v_stride_t, a->v_stride_h, 8) ||
      (a->q && (!rows_ok(a->q, a->q_stride_t, a->q_stride_h, 8) ||
                !rows_ok(a->q_out, a->q_out_stride_t, a->q_out_stride_h, 8))) ||
      (a->positions && !aligned(a->positions, 4)) ||
      (a->freqs && !aligned(a->freqs, 8)))
    return fail(TILEMIX_ERR_INVALID_ARG,
                "%s: misaligned pointer or a stride that is not a multiple of 8 "
                "elements", where);
  if (a->q && !apart(a->q_out_stride_t, a->q_out_stride_h, a->total_tokens, a->hq,
                     a->head_dim))
    return fail(TILEMIX_ERR_INVALID_ARG, "%s: rows of q_out overlap", where);
  if (!apart(a->token_stride, a->head_stride, a->page_size, a->hkv, a->head_dim))
    return fail(TILEMIX_ERR_INVALID_ARG, "%s: rows of a page overlap", where);
  tilemix_status d = check_device();
  if (d != TILEMIX_OK) return d;
  tilemix::RopeArgs r;
  memset(&r, 0, sizeof(r));
  auto rows = [](const void* p, int64_t t, int64_t h) {
    return tilemix::RowTensor{static_cast<uint16_t*>(const_cast<void*>(p)), t, h};
  };
  r.k = rows(a->k, a->k_stride_t, a->k_stride_h);
  r.v = rows(a->v, a->v_stride_t, a->v_stride_h);
  r.q = rows(a->q, a->q_stride_t, a->q_stride_h);
  r.q_out = rows(a->q_out, a->q_out_stride_t, a->q_out_stride_h);
  r.positions = a->positions;
  r.freqs = a->freqs;
  r.attn_factor = a->attn_factor > 0.0f ? a->attn_factor : 1.0f;
  r.sign = 1.0f;
  r.total_tokens = a->total_tokens;
  r.hq = a->q ? a->hq : 0;
  r.hk = r.hv = a->hkv;
  r.head_dim = a->head_dim;
  r.rot_dim = a->freqs ? a->rot_dim : 0;
  r.interleaved = a->layout == TILEMIX_ROPE_INTERLEAVED;
  r.k_pages = a->k_pages;
  r.v_pages = a->v_pages;
  r.page_stride = a->page_stride;
  r.token_stride = a->token_stride;
  r.head_stride = a->head_stride;
  r.k_scale = a->k_scale;
  r.v_scale = a->v_scale;
  r.page_table = a->page_table;
  r.table_stride = a->table_stride;
  r.cu_seqlens = a->cu_seqlens;
  r.kv_lens = a->kv_lens;
  r.batch = a->batch;
  r.num_pages = a->num_pages;
  r.page_shift = log2_of(a->page_size);
  r.max_pages = a->max_pages;
  r.status = a->status;
  const cudaError_t e =
      tilemix::launch_rope(r, a->dtype == TILEMIX_BF16,
                           a->kv_format == TILEMIX_KV_INT8 ? 2 : 1, stream);
  if (e != cudaSuccess)
    return fail(TILEMIX_ERR_CUDA, "%s launch: %s", where, cudaGetErrorString(e));
  return ok();
}

size_t tilemix_attn_paged_workspace_bytes(int max_q_len, int hq, int hkv,
                                          int head_dim) {
  if (max_q_len < 0 || hq <= 0 || hkv <= 0 || hq % hkv != 0 || hq / hkv > 128 ||
      (head_dim != 64 && head_dim != 128) || too_many_rows(max_q_len, hq / hkv))
    return 0;
  // (of 17 to 32 rows either kernel may come: the chunk kernel needs more)
  return use_step(max_q_len, hq / hkv, false)
             ? tilemix::paged_step_workspace_bytes(head_dim)
             : tilemix::paged_chunk_workspace_bytes(head_dim);
}

tilemix_status tilemix_attn_paged(const tilemix_attn_paged_params* a,
                                  tilemix_stream_t stream) {
  const char* where = "attn_paged";
  if (!a) return fail(TILEMIX_ERR_INVALID_ARG, "%s: params is NULL", where);
  if (a->struct_size != sizeof(tilemix_attn_paged_params))
    return fail(TILEMIX_ERR_INVALID_ARG,
                "%s: struct_size %u != sizeof(tilemix_attn_paged_params) %zu",
                where, a->struct_size, sizeof(tilemix_attn_paged_params));
  if ((a->dtype != TILEMIX_FP16 && a->dtype != TILEMIX_BF16) ||
      (a->causal != 0 && a->causal != 1))
    return fail(TILEMIX_ERR_INVALID_ARG, "%s: bad dtype or causal", where);
  if (a->flags & ~TILEMIX_FLAG_TEST_EXPIRE_WAIT)
    return fail(TILEMIX_ERR_INVALID_ARG, "%s: bad flags 0x%x", where, a->flags);
  tilemix_status st = check_cache(
      where, a->kv_format, a->k_pages, a->v_pages, a->page_stride,
      a->token_stride, a->head_stride, a->k_scale, a->v_scale, a->page_table,
      a->table_stride, a->cu_seqlens, a->kv_lens, a->batch, a->total_tokens,
      a->num_pages, a->page_size, a->max_pages, a->hkv, a->head_dim, a->status);
  if (st != TILEMIX_OK) return st;
  st = check_heads(where, a->hq, a->hkv);
  if (st != TILEMIX_OK) return st;
  if (a->max_q_len < 0 || a->max_kv_len < 0)
    return fail(TILEMIX_ERR_INVALID_ARG, "%s: bad size", where);
  if (std::isnan(a->softmax_scale) || std::isinf(a->softmax_scale))
    return fail(TILEMIX_ERR_INVALID_ARG, "%s: bad softmax_scale", where);
  if (too_many_rows(a->max_q_len, a->hq / a->hkv))
    return fail(TILEMIX_ERR_UNSUPPORTED, "%s: too many packed query rows", where);
  if (a->batch == 0 || a->total_tokens == 0 || a->max_q_len == 0) return ok();
  if (!a->q || !a->out)
    return fail(TILEMIX_ERR_INVALID_ARG, "%s: null pointer", where);
  if (!rows_ok(a->q, a->q_stride_t, a->q_stride_h, 8) || !aligned(a->out, 16) ||
      (a->lse && !aligned(a->lse, 4)))
    return fail(TILEMIX_ERR_INVALID_ARG,
                "%s: misaligned pointer or a stride that is not a multiple of 8 "
                "elements", where);
  const size_t need = tilemix_attn_paged_workspace_bytes(a->max_q_len, a->hq,
                                                         a->hkv, a->head_dim);
  if (!a->workspace || !aligned(a->workspace, 16) || a->workspace_bytes < need)
    return fail(TILEMIX_ERR_INVALID_ARG,
                "%s: workspace of %zu bytes (16-byte aligned) needed, %zu given",
                where, need, a->workspace ? a->workspace_bytes : size_t(0));
  tilemix_status dv = check_device();
  if (dv != TILEMIX_OK) return dv;
  if (!encode_fn())
    return fail(TILEMIX_ERR_CUDA, "%s: cuTensorMapEncodeTiled unavailable", where);

  const int d = a->head_dim;
  const bool int8 = a->kv_format == TILEMIX_KV_INT8;
  const bool bf16 = a->dtype == TILEMIX_BF16;
  tilemix::PagedArgs p;
  memset(&p, 0, sizeof(p));
  const CUtensorMapSwizzle sw = int8 && d == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                : CU_TENSOR_MAP_SWIZZLE_128B;
  const bool step = use_step(a->max_q_len, a->hq / a->hkv, int8);
  const int most = step ? tilemix::paged_step_group(d, int8) : 128;
  const int box = a->page_size < most ? a->page_size : most;
  if (!make_pages_map(&p.tm_k, a->k_pages, int8, bf16, d, a->page_size, a->hkv,
                      a->num_pages, a->page_stride, a->token_stride,
                      a->head_stride, box, sw) ||
      !make_pages_map(&p.tm_v, a->v_pages, int8, bf16, d, a->page_size, a->hkv,
                      a->num_pages, a->page_stride, a->token_stride,
                      a->head_stride, box, sw))
    return fail(TILEMIX_ERR_CUDA, "%s: tensor map encoding failed", where);
  p.q = static_cast<const uint16_t*>(a->q);
  p.q_st = a->q_stride_t;
  p.q_sh = a->q_stride_h;
  p.k_scale = a->k_scale;
  p.v_scale = a->v_scale;
  p.page_table = a->page_table;
  p.table_stride = a->table_stride;
  p.cu_seqlens = a->cu_seqlens;
  p.kv_lens = a->kv_lens;
  p.batch = a->batch;
  p.total_tokens = a->total_tokens;
  p.max_q_len = a->max_q_len;
  p.max_kv_len = a->max_kv_len;
  p.hq = a->hq;
  p.hkv = a->hkv;
  p.group = a->hq / a->hkv;
  p.num_pages = a->num_pages;
  p.page_shift = log2_of(a->page_size);
  p.max_pages = a->max_pages;
  p.causal = a->causal;
  const float scale =
      a->softmax_scale > 0.0f ? a->softmax_scale : 1.0f / std::sqrt(float(d));
  p.scale_log2 = scale * 1.4426950408889634f;
  p.test_expire_wait = (a->flags & TILEMIX_FLAG_TEST_EXPIRE_WAIT) ? 1 : 0;
  p.out = static_cast<uint16_t*>(a->out);
  p.lse = a->lse;
  p.status = a->status;
  const tilemix::PagedShape shape{d, bf16, int8};
  const cudaError_t e =
      step ? tilemix::launch_paged_step(p, shape, a->workspace, stream)
           : tilemix::launch_paged_chunk(p, shape, a->workspace, stream);
  if (e != cudaSuccess)
    return fail(TILEMIX_ERR_CUDA, "%s launch: %s", where, cudaGetErrorString(e));
  return ok();
}

}  // extern "C"
