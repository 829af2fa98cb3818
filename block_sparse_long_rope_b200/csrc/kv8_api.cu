// C entry points of the operators that serve a ragged batch from an 8-bit
// paged cache (declared in include/star.h): argument checks, workspace layout
// and launches on the caller's stream. Nothing here allocates or waits.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include "kv8_kernels.cuh"
#include "star.h"
#include "star_common.cuh"
#include "star_kernels.cuh"

namespace {

star_status fail(star_status s, const char* fmt, ...) {
  char buf[320];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  star::set_last_error(buf);
  return s;
}

star_status ok() {
  star::set_last_error("");
  return STAR_OK;
}

star_status check_ptr(const void* p, const char* name, uintptr_t align = 16) {
  if (!p) return fail(STAR_ERR_INVALID_ARG, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) & (align - 1))
    return fail(STAR_ERR_INVALID_ARG, "%s is not %d-byte aligned", name, (int)align);
  return STAR_OK;
}

star_status check_workspace(const void* ws, size_t bytes, size_t need) {
  star_status s = check_ptr(ws, "workspace", 256);
  if (s != STAR_OK) return s;
  if (bytes < need) return fail(STAR_ERR_INVALID_ARG, "workspace too small: %zu < %zu bytes", bytes, need);
  return STAR_OK;
}

// log2 of a supported page length, or -1
int page_shift_of(int page_len) {
  for (int s = 4; s <= 7; ++s)
    if (page_len == 1 << s) return s;
  return -1;
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// Checks that the cache arguments share; *shift receives log2(page_len).
star_status check_cache(const void* k_pages, const void* v_pages, const float* k_scale,
                        const float* v_scale, int num_pages, int page_len, int kv_type, int Hkv,
                        int D, int* shift) {
  if (D != 64 && D != 128) return fail(STAR_ERR_UNSUPPORTED, "head_dim %d not supported (64 or 128)", D);
  if (Hkv < 1 || Hkv > star::kMaxHeads)
    return fail(STAR_ERR_INVALID_ARG, "Hkv (%d) must lie in [1, %d]", Hkv, star::kMaxHeads);
  *shift = page_shift_of(page_len);
  if (*shift < 0) return fail(STAR_ERR_UNSUPPORTED, "page_len %d not supported (16, 32, 64 or 128)", page_len);
  if (kv_type != STAR_KV8_E4M3 && kv_type != STAR_KV8_INT8)
    return fail(STAR_ERR_INVALID_ARG, "kv_type %d is neither e4m3 (0) nor int8 (1)", kv_type);
  if (num_pages < 1 || ((long long)num_pages << *shift) > INT32_MAX)
    return fail(STAR_ERR_INVALID_ARG, "num_pages (%d) must be >= 1 and num_pages * page_len fit int32", num_pages);
  star_status s;
  if ((s = check_ptr(k_pages, "k_pages")) || (s = check_ptr(v_pages, "v_pages")) ||
      (s = check_ptr(k_scale, "k_scale", 4)) || (s = check_ptr(v_scale, "v_scale", 4)))
    return s;
  return STAR_OK;
}

star_status check_requests(int B) {
  if (B < 1 || B > star::kMaxRequests)
    return fail(STAR_ERR_INVALID_ARG, "B (%d) must lie in [1, %d]", B, star::kMaxRequests);
  return STAR_OK;
}

star_status check_strides(const int64_t* s, int n, const char* name) {
  if (!s) return fail(STAR_ERR_INVALID_ARG, "%s is NULL", name);
  for (int i = 0; i < n; ++i)
    if (s[i] % 8 != 0) return fail(STAR_ERR_INVALID_ARG, "%s must be multiples of 8 elements", name);
  return STAR_OK;
}

star_status launched(cudaError_t e, const char* what) {
  if (e != cudaSuccess) return fail(STAR_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  return ok();
}

bool positive(double x) { return isfinite(x) && x > 0.0; }

// Workspace of star_kv8_attend: status word, then the finished-part counters
// (the same place for every call, since they have to be zero between calls),
// the parts' statistics and their outputs.
struct AttendLayout {
  int rows;
  size_t part_ml, part_o, total;
};
constexpr size_t kAttendHeader = star::kStatusBytes + star::kKv8MaxCtas * sizeof(unsigned);
AttendLayout attend_layout(int rows, int D) {
  AttendLayout l;
  l.rows = rows;
  const size_t ctas = l.rows == star::kKv8ChunkRows ? star::kKv8ChunkMaxCtas : star::kKv8MaxCtas;
  const size_t parts = 2 * ctas * l.rows;
  l.part_ml = kAttendHeader;
  l.part_o = l.part_ml + align256(parts * 2 * sizeof(float));
  l.total = l.part_o + align256(parts * D * sizeof(float));
  return l;
}

}  // namespace

extern "C" {

star_status star_rope_frequencies(int rot_dim, double theta, int scaling, double factor,
                                  double orig_len, double a, double b, double* inv_freq,
                                  double* mscale) {
  if (!inv_freq || !mscale) return fail(STAR_ERR_INVALID_ARG, "inv_freq or mscale is NULL");
  if (rot_dim < 2 || rot_dim > 128 || rot_dim % 2)
    return fail(STAR_ERR_INVALID_ARG, "rot_dim (%d) must be even and lie in [2, 128]", rot_dim);
  if (!isfinite(theta) || !(theta > 1.0)) return fail(STAR_ERR_INVALID_ARG, "theta must be > 1");
  if (scaling < STAR_ROPE_NONE || scaling > STAR_ROPE_LLAMA3)
    return fail(STAR_ERR_INVALID_ARG, "unknown scaling %d", scaling);
  if (scaling != STAR_ROPE_NONE && !(isfinite(factor) && factor >= 1.0))
    return fail(STAR_ERR_INVALID_ARG, "factor must be >= 1");
  if (scaling == STAR_ROPE_YARN || scaling == STAR_ROPE_LLAMA3) {
    if (!positive(orig_len) || !positive(a) || !positive(b))
      return fail(STAR_ERR_INVALID_ARG, "orig_len and the two turn counts must be finite and > 0");
    if (scaling == STAR_ROPE_YARN ? a < b : a >= b)
      return fail(STAR_ERR_INVALID_ARG, "the turn counts are in the wrong order");
  }
  if (scaling == STAR_ROPE_NTK && rot_dim == 2)
    return fail(STAR_ERR_INVALID_ARG, "NTK scaling needs more than one pair");
  const double two_pi = 6.283185307179586;
  const double base = scaling == STAR_ROPE_NTK ? theta * pow(factor, rot_dim / (rot_dim - 2.0)) : theta;
  double lo = 0.0, span = 1.0;
  if (scaling == STAR_ROPE_YARN) {
    const double per = rot_dim / (2.0 * log(theta));
    lo = fmax(floor(per * log(orig_len / (a * two_pi))), 0.0);
    const double hi = fmin(ceil(per * log(orig_len / (b * two_pi))), rot_dim - 1.0);
    span = hi != lo ? hi - lo : 0.001;
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = pow(base, -2.0 * i / rot_dim);
    if (scaling == STAR_ROPE_LINEAR) {
      f /= factor;
    } else if (scaling == STAR_ROPE_YARN) {
      const double r = fmin(1.0, fmax(0.0, (i - lo) / span));
      f = f / factor * r + f * (1.0 - r);
    } else if (scaling == STAR_ROPE_LLAMA3) {
      const double u = fmin(1.0, fmax(0.0, (orig_len * f / two_pi - a) / (b - a)));
      f = (1.0 - u) * f / factor + u * f;
    }
    inv_freq[i] = f;
  }
  *mscale = scaling == STAR_ROPE_YARN ? 0.1 * log(factor) + 1.0 : 1.0;
  return ok();
}

star_status star_rope_scaled(const void* x, const int64_t x_stride[3], void* y,
                             const int64_t y_stride[3], const int32_t* pos, int64_t pos_stride_b,
                             int64_t pos0, int B, int S, int H, int D, int rot_dim,
                             const double* inv_freq, double mscale, int interleaved,
                             int transpose, void* cuda_stream) {
  star_status s;
  if ((s = check_strides(x_stride, 3, "x_stride")) || (s = check_strides(y_stride, 3, "y_stride"))) return s;
  if (B < 0 || B > 65535 || S < 0 || H < 1 || H > star::kMaxHeads)
    return fail(STAR_ERR_INVALID_ARG, "bad shape B=%d S=%d H=%d (B <= 65535, H <= %d)", B, S, H,
                star::kMaxHeads);
  if (D != 64 && D != 128) return fail(STAR_ERR_UNSUPPORTED, "head_dim %d not supported (64 or 128)", D);
  if (rot_dim < 16 || rot_dim > D || rot_dim % 16)
    return fail(STAR_ERR_INVALID_ARG, "rot_dim (%d) must be a multiple of 16 in [16, %d]", rot_dim, D);
  if (interleaved < 0 || interleaved > 1 || transpose < 0 || transpose > 1)
    return fail(STAR_ERR_INVALID_ARG, "interleaved and transpose must be 0 or 1");
  if (!inv_freq) return fail(STAR_ERR_INVALID_ARG, "inv_freq is NULL");
  for (int i = 0; i < rot_dim / 2; ++i)
    if (!isfinite(inv_freq[i])) return fail(STAR_ERR_INVALID_ARG, "inv_freq[%d] is not finite", i);
  if (!isfinite(mscale) || fabs(mscale) > 1e30) return fail(STAR_ERR_INVALID_ARG, "mscale must be finite (at most 1e30)");
  const bool empty = B == 0 || S == 0;  // an empty tensor has no address
  if (!empty && ((s = check_ptr(x, "x")) || (s = check_ptr(y, "y")))) return s;
  if (pos && (s = check_ptr(pos, "pos", 4))) return s;
  if (x == y && !empty)
    for (int i = 0; i < 3; ++i)
      if (x_stride[i] != y_stride[i])
        return fail(STAR_ERR_INVALID_ARG, "in place, x and y must have the same strides");
  if (star::device_sms() <= 0) return STAR_ERR_UNSUPPORTED;  // message set by the device check
  if (empty) return ok();
  star::RopeScaledParams p{};
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.y = static_cast<__nv_bfloat16*>(y);
  for (int i = 0; i < 3; ++i) {
    p.xs[i] = x_stride[i];
    p.ys[i] = y_stride[i];
  }
  p.pos = pos;
  p.pos_stride_b = pos_stride_b;
  p.pos0 = pos0;
  p.B = B;
  p.S = S;
  p.H = H;
  p.D = D;
  p.rot = rot_dim;
  p.copy_rest = x != y;
  p.mscale = mscale;
  p.mscale_abs = (float)fabs(mscale);
  p.sign = transpose ? -1.0 : 1.0;
  memcpy(p.inv_freq, inv_freq, sizeof(double) * (rot_dim / 2));
  return launched(star::launch_rope_scaled(p, interleaved != 0, static_cast<cudaStream_t>(cuda_stream)),
                  "scaled rope launch");
}

int star_batch_plan_runs(int n_tokens, int B, int page_len) {
  if (n_tokens < 0 || B < 1 || page_len < 1) return 0;
  const long long r = (long long)n_tokens / page_len + 2ll * B;
  return (int)(r < n_tokens ? r : n_tokens);
}

size_t star_batch_plan_workspace_bytes(int B) {
  (void)B;
  return star::kStatusBytes;
}

star_status star_batch_plan(const int32_t* ctx_len, const int32_t* new_len, int B,
                            const int32_t* free_pages, int num_free, const int32_t* free_begin,
                            int page_len, int32_t* block_table, int max_pages, int32_t* cu_new,
                            int32_t* pos, int32_t* slot, int n_cap, int32_t* run_start,
                            int run_cap, int32_t* kv_len, int32_t* free_next, void* workspace,
                            size_t workspace_bytes, void* cuda_stream) {
  star_status s;
  if ((s = check_requests(B))) return s;
  const int shift = page_shift_of(page_len);
  if (shift < 0) return fail(STAR_ERR_UNSUPPORTED, "page_len %d not supported (16, 32, 64 or 128)", page_len);
  if (max_pages < 1 || ((long long)max_pages << shift) > INT32_MAX)
    return fail(STAR_ERR_INVALID_ARG, "max_pages (%d) must be >= 1 and max_pages * page_len fit int32", max_pages);
  if (num_free < 0 || n_cap < 0 || run_cap < 0)
    return fail(STAR_ERR_INVALID_ARG, "num_free, n_cap and run_cap must be >= 0");
  if (n_cap > (1 << 30)) return fail(STAR_ERR_INVALID_ARG, "n_cap (%d) must be at most 2^30", n_cap);
  if (run_cap < star_batch_plan_runs(n_cap, B, page_len))
    return fail(STAR_ERR_INVALID_ARG, "run_cap (%d) < star_batch_plan_runs (%d)", run_cap,
                star_batch_plan_runs(n_cap, B, page_len));
  if (run_cap > (1 << 30)) return fail(STAR_ERR_INVALID_ARG, "run_cap (%d) must be at most 2^30", run_cap);
  if ((s = check_ptr(ctx_len, "ctx_len", 4)) || (s = check_ptr(new_len, "new_len", 4)) ||
      (s = check_ptr(free_begin, "free_begin", 4)) || (s = check_ptr(block_table, "block_table", 4)) ||
      (s = check_ptr(cu_new, "cu_new", 4)) || (s = check_ptr(run_start, "run_start", 4)) ||
      (s = check_ptr(kv_len, "kv_len", 4)) || (s = check_ptr(free_next, "free_next", 4)))
    return s;
  if (num_free > 0 && (s = check_ptr(free_pages, "free_pages", 4))) return s;
  if (n_cap > 0 && ((s = check_ptr(pos, "pos", 4)) || (s = check_ptr(slot, "slot", 4)))) return s;
  if ((s = check_workspace(workspace, workspace_bytes, star_batch_plan_workspace_bytes(B)))) return s;
  if (star::device_sms() <= 0) return STAR_ERR_UNSUPPORTED;
  star::BatchPlanParams p{};
  p.ctx_len = ctx_len;
  p.new_len = new_len;
  p.free_pages = free_pages;
  p.free_begin = free_begin;
  p.table = block_table;
  p.cu_new = cu_new;
  p.pos = pos;
  p.slot = slot;
  p.run_start = run_start;
  p.kv_len = kv_len;
  p.free_next = free_next;
  p.B = B;
  p.num_free = num_free;
  p.page_shift = shift;
  p.max_pages = max_pages;
  p.n_cap = n_cap;
  p.run_cap = run_cap;
  p.status = static_cast<int*>(workspace);
  p.ticket = static_cast<unsigned*>(workspace) + 2;  // words 0 and 1: star_device_status
  return launched(star::launch_batch_plan(p, static_cast<cudaStream_t>(cuda_stream)), "batch plan launch");
}

star_status star_kv8_append(const void* k, const int64_t k_stride[2], const void* v,
                            const int64_t v_stride[2], int n_tokens, int Hkv, int D,
                            const int32_t* slot, const int32_t* run_start, int run_cap,
                            void* k_pages, void* v_pages, float* k_scale, float* v_scale,
                            int num_pages, int page_len, int kv_type, void* workspace,
                            size_t workspace_bytes, void* cuda_stream) {
  star_status s;
  int shift = 0;
  if ((s = check_cache(k_pages, v_pages, k_scale, v_scale, num_pages, page_len, kv_type, Hkv, D, &shift)))
    return s;
  if (n_tokens < 0 || run_cap < 0) return fail(STAR_ERR_INVALID_ARG, "n_tokens and run_cap must be >= 0");
  if ((s = check_strides(k_stride, 2, "k_stride")) || (s = check_strides(v_stride, 2, "v_stride"))) return s;
  if ((s = check_workspace(workspace, workspace_bytes, star::kStatusBytes))) return s;
  if (n_tokens > 0 && run_cap > 0 &&
      ((s = check_ptr(k, "k")) || (s = check_ptr(v, "v")) || (s = check_ptr(slot, "slot", 4)) ||
       (s = check_ptr(run_start, "run_start", 4))))
    return s;
  if (star::device_sms() <= 0) return STAR_ERR_UNSUPPORTED;
  if (n_tokens == 0 || run_cap == 0) return ok();
  star::Kv8AppendParams p{};
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  for (int i = 0; i < 2; ++i) {
    p.ks[i] = k_stride[i];
    p.vs[i] = v_stride[i];
  }
  p.slot = slot;
  p.run_start = run_start;
  p.k_pages = static_cast<uint8_t*>(k_pages);
  p.v_pages = static_cast<uint8_t*>(v_pages);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.n_tokens = n_tokens;
  p.Hkv = Hkv;
  p.run_cap = run_cap;
  p.num_pages = num_pages;
  p.page_shift = shift;
  p.status = static_cast<int*>(workspace);
  return launched(star::launch_kv8_append(p, D, kv_type, static_cast<cudaStream_t>(cuda_stream)),
                  "8-bit append launch");
}

size_t star_kv8_attend_workspace_bytes(int B, int n_tokens, int Hq, int Hkv, int D, int max_new) {
  (void)n_tokens;
  if (B < 1 || Hq < 1 || Hkv < 1 || D < 1 || max_new < 1 || Hq % Hkv) return star::kStatusBytes;
  return attend_layout(star::kv8_rows(max_new, Hq / Hkv), D).total;
}

star_status star_kv8_attend(const void* q, const int64_t q_stride[2], int n_tokens,
                            const int32_t* cu_new, const int32_t* kv_len, int B,
                            const int32_t* block_table, int max_pages, const void* k_pages,
                            const void* v_pages, const float* k_scale, const float* v_scale,
                            int num_pages, int page_len, int kv_type, int Hq, int Hkv, int D,
                            int max_new, int max_kv, void* o, float* lse, void* workspace,
                            size_t workspace_bytes, void* cuda_stream) {
  star_status s;
  int shift = 0;
  if ((s = check_cache(k_pages, v_pages, k_scale, v_scale, num_pages, page_len, kv_type, Hkv, D, &shift)))
    return s;
  if ((s = check_requests(B))) return s;
  if (Hq < 1 || Hq > star::kMaxHeads || Hq % Hkv)
    return fail(STAR_ERR_INVALID_ARG, "Hq (%d) must be a multiple of Hkv (%d), at most %d", Hq, Hkv,
                star::kMaxHeads);
  if (max_pages < 1 || ((long long)max_pages << shift) > INT32_MAX)
    return fail(STAR_ERR_INVALID_ARG, "max_pages (%d) must be >= 1 and max_pages * page_len fit int32", max_pages);
  if (n_tokens < 0) return fail(STAR_ERR_INVALID_ARG, "n_tokens must be >= 0");
  if (max_new < 1) return fail(STAR_ERR_INVALID_ARG, "max_new must be >= 1");
  // (keys and the ends of their tiles are counted in int32)
  if (max_kv < 1 || max_kv > ((long long)max_pages << shift) || max_kv > INT32_MAX - 2 * star::kKv8Tile)
    return fail(STAR_ERR_INVALID_ARG, "max_kv (%d) must lie in [1, max_pages * page_len], at most 2^31 - 257", max_kv);
  if ((s = check_strides(q_stride, 2, "q_stride"))) return s;
  if ((s = check_ptr(cu_new, "cu_new", 4)) || (s = check_ptr(kv_len, "kv_len", 4)) ||
      (s = check_ptr(block_table, "block_table", 4)))
    return s;
  if (n_tokens > 0 && ((s = check_ptr(q, "q")) || (s = check_ptr(o, "o")))) return s;
  if (lse && (s = check_ptr(lse, "lse", 4))) return s;
  const int g = Hq / Hkv;
  // what the kernels count in 32 bits: rows of a request, tiles of a call
  if ((long long)max_new * g > (1 << 24))
    return fail(STAR_ERR_INVALID_ARG, "max_new * Hq / Hkv (%lld) must be at most 2^24", (long long)max_new * g);
  // tiles of a call with row tiles of this many rows, were every request as long as
  // the bounds allow
  auto tiles_with = [&](int rows) {
    return (double)B * Hkv * ((max_new * g + rows - 1) / rows) * ((max_kv - 1) / star::kKv8Tile + 1);
  };
  // the most that n_tokens tokens can make of them
  auto most_tiles = [&](int rows) {
    return fmin(tiles_with(rows), Hkv * ((double)n_tokens * g / rows + B) * ((max_kv - 1) / star::kKv8Tile + 1));
  };
  const size_t need = attend_layout(star::kv8_rows(max_new, g), D).total;
  const int rows = star::kv8_rows(max_new, g) == star::kKv8ChunkRows && tiles_with(16) <= star::kKv8FewTiles
                       ? 16 : star::kv8_rows(max_new, g);
  const AttendLayout lay = attend_layout(rows, D);
  const double tiles = most_tiles(rows);
  if (tiles >= 2147483647.0)
    return fail(STAR_ERR_INVALID_ARG, "problem too large: %.0f tiles of %d rows by %d keys", tiles,
                lay.rows, star::kKv8Tile);
  if ((s = check_workspace(workspace, workspace_bytes, need))) return s;
  const int sms = star::device_sms();
  if (sms <= 0) return STAR_ERR_UNSUPPORTED;
  if (n_tokens == 0) return ok();
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  star::Kv8AttendParams p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.qs[0] = q_stride[0];
  p.qs[1] = q_stride[1];
  p.cu_new = cu_new;
  p.kv_len = kv_len;
  p.table = block_table;
  p.k_pages = static_cast<const uint8_t*>(k_pages);
  p.v_pages = static_cast<const uint8_t*>(v_pages);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.n_tokens = n_tokens;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.g = g;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  p.page_shift = shift;
  p.max_new = max_new;
  p.max_kv = max_kv;
  p.scale_log2 = (float)(1.4426950408889634 / sqrt((double)D));
  p.status = reinterpret_cast<int*>(ws);
  p.header_bytes = (int)kAttendHeader;
  p.counters = reinterpret_cast<unsigned*>(ws + star::kStatusBytes);
  p.part_ml = reinterpret_cast<float*>(ws + lay.part_ml);
  p.part_o = reinterpret_cast<float*>(ws + lay.part_o);
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  return launched(lay.rows == star::kKv8ChunkRows ? star::launch_kv8_chunk(p, D, kv_type, sms, st)
                                                  : star::launch_kv8_decode(p, D, kv_type, lay.rows, sms, st),
                  "8-bit attention launch");
}

}  // extern "C"
