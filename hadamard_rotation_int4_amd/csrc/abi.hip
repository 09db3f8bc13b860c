// extern "C" entry points of libhr.so (declared in include/hr.h): host-side
// argument validation, then a launch on the caller's stream.  A call that
// fails validation makes no HIP call at all.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include <algorithm>
#include <string>

#include "hr.h"
#include "hr_internal.h"
#include "kv4.h"
#include "mx4.h"

namespace {

thread_local std::string g_last_error;

int32_t fail(int32_t status, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return status;
}

int32_t ok() { return HR_OK; }

int32_t from_hip(hipError_t e, const char* what) {
  if (e == hipSuccess) return ok();
  return fail(HR_EDEVICE, "%s: launch failed: %s", what, hipGetErrorString(e));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool pow2(int64_t v) { return v > 0 && (v & (v - 1)) == 0; }
int ilog2(int64_t v) {
  int l = 0;
  while ((int64_t(1) << l) < v) ++l;
  return l;
}
bool valid_group(int32_t g) { return g == 32 || g == 64 || g == 128 || g == 256; }

// Shared checks of hr_rotate and hr_rotate_quant_int4; fills p.
int32_t check_rotation(const char* fn, const void* x, int32_t x_dtype, int64_t rows, int32_t n,
                       int32_t m, const int8_t* signs, const float* block, int* p_out) {
  if (rows < 0) return fail(HR_EINVAL, "%s: rows < 0", fn);
  if (!x && rows > 0) return fail(HR_EINVAL, "%s: x is NULL", fn);
  if (x_dtype != HR_BF16 && x_dtype != HR_F32)
    return fail(HR_EINVAL, "%s: x_dtype must be HR_BF16 or HR_F32", fn);
  if (!aligned16(x) || (signs && !aligned16(signs)))
    return fail(HR_EINVAL, "%s: x and signs must be 16-byte aligned", fn);
  if (m < 1 || m > 16) return fail(HR_EUNSUPPORTED, "%s: m=%d outside [1, 16]", fn, m);
  if (n <= 0 || n % m) return fail(HR_EUNSUPPORTED, "%s: n=%d is not a multiple of m=%d", fn, n, m);
  const int p = n / m;
  if (!pow2(p) || p < 64 || p > 16384)
    return fail(HR_EUNSUPPORTED, "%s: n/m=%d is not a power of two in [64, 16384]", fn, p);
  if (n > 16384) return fail(HR_EUNSUPPORTED, "%s: n=%d > 16384", fn, n);
  if (m == 1 && block) return fail(HR_EINVAL, "%s: block must be NULL when m == 1", fn);
  if (m > 1 && !block) return fail(HR_EINVAL, "%s: block is NULL with m=%d", fn, m);
  if (block && (reinterpret_cast<uintptr_t>(block) & 3u))
    return fail(HR_EINVAL, "%s: block must be 4-byte aligned", fn);
  *p_out = p;
  return HR_OK;
}

}  // namespace

extern "C" {

int32_t hr_abi_version(void) { return HR_ABI_VERSION; }

// HR_SOURCE_HASH is defined by the build: a hash of the library's sources, so
// a binding can tell a library built from other sources.
#ifndef HR_SOURCE_HASH
#define HR_SOURCE_HASH "unknown"
#endif
const char* hr_build_id(void) { return HR_SOURCE_HASH; }

const char* hr_status_string(int32_t status) {
  switch (status) {
    case HR_OK: return "HR_OK: success";
    case HR_EINVAL: return "HR_EINVAL: invalid argument";
    case HR_EUNSUPPORTED: return "HR_EUNSUPPORTED: size or mode not supported";
    case HR_EDEVICE: return "HR_EDEVICE: kernel launch failed";
    default: return "unknown hr_status";
  }
}

const char* hr_last_error(void) { return g_last_error.c_str(); }

int32_t hr_rotate(const void* x, int32_t x_dtype, float* y, int64_t rows, int32_t n, int32_t m,
                  const int8_t* signs, const float* block, void* stream) {
  int p = 0;
  const int32_t st = check_rotation("hr_rotate", x, x_dtype, rows, n, m, signs, block, &p);
  if (st) return st;
  if (!y && rows > 0) return fail(HR_EINVAL, "hr_rotate: y is NULL");
  if (!aligned16(y)) return fail(HR_EINVAL, "hr_rotate: y must be 16-byte aligned");
  if (rows == 0) return ok();
  hr::RhtArgs a{};
  a.x = x;
  a.x_bf16 = x_dtype == HR_BF16;
  a.rows = rows;
  a.n = n;
  a.m = m;
  a.p = p;
  a.signs = signs;
  a.block = block;
  a.y = y;
  return from_hip(hr::launch_rht(a, static_cast<hipStream_t>(stream)), "hr_rotate");
}

// Shared body of hr_rotate_quant_int4 and hr_rotate_quant_int8.
static int32_t rotate_quant(const char* fn, int bits, const void* x, int32_t x_dtype, int64_t rows,
                            int32_t n, int32_t m, const int8_t* signs, const float* block,
                            int32_t group, uint8_t* codes, void* scales, int32_t scale_dtype,
                            void* stream) {
  int p = 0;
  const int32_t st = check_rotation(fn, x, x_dtype, rows, n, m, signs, block, &p);
  if (st) return st;
  if ((!codes || !scales) && rows > 0)
    return fail(HR_EINVAL, "%s: codes and scales are required", fn);
  if (!aligned16(codes) || !aligned16(scales))
    return fail(HR_EINVAL, "%s: codes and scales must be 16-byte aligned", fn);
  if (scale_dtype != HR_F16 && scale_dtype != HR_F32)
    return fail(HR_EINVAL, "%s: scale_dtype must be HR_F16 or HR_F32", fn);
  if (!valid_group(group)) return fail(HR_EUNSUPPORTED, "%s: group=%d not in {32,64,128,256}", fn, group);
  if (p % group) return fail(HR_EUNSUPPORTED, "%s: group=%d does not divide p=%d", fn, group, p);
  if (rows == 0) return ok();
  hr::RhtArgs a{};
  a.x = x;
  a.x_bf16 = x_dtype == HR_BF16;
  a.rows = rows;
  a.n = n;
  a.m = m;
  a.p = p;
  a.signs = signs;
  a.block = block;
  a.group = group;
  a.codes = codes;
  a.bits = bits;
  a.scales = scales;
  a.scale_f16 = scale_dtype == HR_F16;
  return from_hip(hr::launch_rht(a, static_cast<hipStream_t>(stream)), fn);
}

int32_t hr_rotate_quant_int4(const void* x, int32_t x_dtype, int64_t rows, int32_t n, int32_t m,
                             const int8_t* signs, const float* block, int32_t group,
                             uint8_t* codes, void* scales, int32_t scale_dtype, void* stream) {
  return rotate_quant("hr_rotate_quant_int4", 4, x, x_dtype, rows, n, m, signs, block, group, codes,
                      scales, scale_dtype, stream);
}

int32_t hr_rotate_quant_int8(const void* x, int32_t x_dtype, int64_t rows, int32_t n, int32_t m,
                             const int8_t* signs, const float* block, int32_t group,
                             int8_t* codes, void* scales, int32_t scale_dtype, void* stream) {
  return rotate_quant("hr_rotate_quant_int8", 8, x, x_dtype, rows, n, m, signs, block, group,
                      reinterpret_cast<uint8_t*>(codes), scales, scale_dtype, stream);
}

// Shared body of hr_quant_int4 and hr_quant_int8.
static int32_t quant_plain(const char* fn, int bits, const void* x, int32_t x_dtype, int64_t rows,
                           int32_t n, int32_t group, uint8_t* codes, void* scales, int32_t scale_dtype,
                           void* stream) {
  if (rows < 0) return fail(HR_EINVAL, "%s: rows < 0", fn);
  if ((!x || !codes || !scales) && rows > 0)
    return fail(HR_EINVAL, "%s: x, codes and scales are required", fn);
  if (x_dtype != HR_BF16 && x_dtype != HR_F32)
    return fail(HR_EINVAL, "%s: x_dtype must be HR_BF16 or HR_F32", fn);
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scales))
    return fail(HR_EINVAL, "%s: x, codes and scales must be 16-byte aligned", fn);
  if (scale_dtype != HR_F16 && scale_dtype != HR_F32)
    return fail(HR_EINVAL, "%s: scale_dtype must be HR_F16 or HR_F32", fn);
  if (!valid_group(group)) return fail(HR_EUNSUPPORTED, "%s: group=%d not in {32,64,128,256}", fn, group);
  if (n <= 0 || n % group || n > (1 << 30))
    return fail(HR_EUNSUPPORTED, "%s: n=%d must be a positive multiple of group=%d", fn, n, group);
  if (rows == 0) return ok();
  hr::QuantArgs a{};
  a.x = x;
  a.x_bf16 = x_dtype == HR_BF16;
  a.rows = rows;
  a.n = n;
  a.group = group;
  a.bits = bits;
  a.codes = codes;
  a.scales = scales;
  a.scale_f16 = scale_dtype == HR_F16;
  return from_hip(hr::launch_quant(a, static_cast<hipStream_t>(stream)), fn);
}

int32_t hr_quant_int4(const void* x, int32_t x_dtype, int64_t rows, int32_t n, int32_t group,
                      uint8_t* codes, void* scales, int32_t scale_dtype, void* stream) {
  return quant_plain("hr_quant_int4", 4, x, x_dtype, rows, n, group, codes, scales, scale_dtype, stream);
}

int32_t hr_quant_int8(const void* x, int32_t x_dtype, int64_t rows, int32_t n, int32_t group,
                      int8_t* codes, void* scales, int32_t scale_dtype, void* stream) {
  return quant_plain("hr_quant_int8", 8, x, x_dtype, rows, n, group, reinterpret_cast<uint8_t*>(codes),
                     scales, scale_dtype, stream);
}

int32_t hr_butterfly_coeffs(const float* angles, int32_t n, int32_t precondition, float* coeffs,
                            void* stream) {
  const char* fn = "hr_butterfly_coeffs";
  if (!angles || !coeffs) return fail(HR_EINVAL, "%s: angles and coeffs are required", fn);
  if (!aligned16(angles) || !aligned16(coeffs))
    return fail(HR_EINVAL, "%s: angles and coeffs must be 16-byte aligned", fn);
  if (precondition != 0 && precondition != 1) return fail(HR_EINVAL, "%s: precondition must be 0 or 1", fn);
  if (!pow2(n) || n < 64 || n > 8192)
    return fail(HR_EUNSUPPORTED, "%s: n=%d is not a power of two in [64, 8192]", fn, n);
  return from_hip(hr::launch_butterfly_coeffs(angles, n, ilog2(n), precondition, coeffs,
                                              static_cast<hipStream_t>(stream)), fn);
}

int32_t hr_butterfly_apply(const float* x, float* y, int64_t rows, int32_t n, const float* coeffs,
                           int32_t precondition, const int32_t* perm, int32_t inverse,
                           int32_t group, uint8_t* codes, void* scales, int32_t scale_dtype,
                           void* stream) {
  const char* fn = "hr_butterfly_apply";
  if (rows < 0) return fail(HR_EINVAL, "%s: rows < 0", fn);
  if (!coeffs) return fail(HR_EINVAL, "%s: coeffs is required", fn);
  if (!x && rows > 0) return fail(HR_EINVAL, "%s: x is NULL", fn);
  if (!y && !codes && rows > 0) return fail(HR_EINVAL, "%s: y and codes are both NULL", fn);
  if (!codes && scales) return fail(HR_EINVAL, "%s: scales given without codes", fn);
  if (codes && !scales) return fail(HR_EINVAL, "%s: codes given without scales", fn);
  if (!aligned16(x) || (y && !aligned16(y)) || !aligned16(coeffs) || (perm && !aligned16(perm)) ||
      (codes && !aligned16(codes)) || (scales && !aligned16(scales)))
    return fail(HR_EINVAL, "%s: pointers must be 16-byte aligned", fn);
  if (precondition != 0 && precondition != 1) return fail(HR_EINVAL, "%s: precondition must be 0 or 1", fn);
  if (inverse != 0 && inverse != 1) return fail(HR_EINVAL, "%s: inverse must be 0 or 1", fn);
  if (!pow2(n) || n < 64 || n > 8192)
    return fail(HR_EUNSUPPORTED, "%s: n=%d is not a power of two in [64, 8192]", fn, n);
  if (codes) {
    if (inverse) return fail(HR_EUNSUPPORTED, "%s: quantization needs inverse == 0", fn);
    if (scale_dtype != HR_F16 && scale_dtype != HR_F32)
      return fail(HR_EINVAL, "%s: scale_dtype must be HR_F16 or HR_F32", fn);
    if (!valid_group(group) || n % group)
      return fail(HR_EUNSUPPORTED, "%s: group=%d invalid for n=%d", fn, group, n);
  }
  if (rows == 0) return ok();
  hr::ButterflyArgs a{};
  a.x = x;
  a.y = y;
  a.rows = rows;
  a.n = n;
  a.log2n = ilog2(n);
  a.coeffs = coeffs;
  a.precondition = precondition;
  a.perm = perm;
  a.inverse = inverse;
  a.group = group;
  a.codes = codes;
  a.scales = scales;
  a.scale_f16 = scale_dtype == HR_F16;
  return from_hip(hr::launch_butterfly(a, static_cast<hipStream_t>(stream)), fn);
}

// Checks a HARP schedule given on the host and fills the per-stage offsets.
static int32_t harp_schedule(const char* fn, const int32_t* radices, int32_t nstages, int32_t* d_out,
                             hr::HarpSchedule* sc) {
  if (!radices) return fail(HR_EINVAL, "%s: radices is NULL", fn);
  if (nstages < 1 || nstages > hr::kHarpMaxStages)
    return fail(HR_EUNSUPPORTED, "%s: nstages=%d outside [1, %d]", fn, nstages, hr::kHarpMaxStages);
  int64_t d = 1;
  for (int t = 0; t < nstages; ++t) {
    if (radices[t] < 2 || radices[t] > hr::kHarpMaxRadix)
      return fail(HR_EUNSUPPORTED, "%s: radix %d of stage %d outside [2, %d]", fn, radices[t], t,
                  hr::kHarpMaxRadix);
    d *= radices[t];
    if (d > 16384) return fail(HR_EUNSUPPORTED, "%s: the radices multiply past 16384", fn);
  }
  if (d % 4) return fail(HR_EUNSUPPORTED, "%s: d=%lld is not a multiple of 4", fn, (long long)d);
  *sc = hr::HarpSchedule{};
  sc->nstages = nstages;
  int64_t stride = 1, nblk = 0, th = 0, fb = 0, bo = 0;
  for (int t = 0; t < nstages; ++t) {
    const int b = radices[t];
    sc->radix[t] = b;
    sc->stride[t] = (int)stride;
    sc->block_begin[t] = nblk;
    sc->theta_off[t] = th;
    sc->fallback_off[t] = fb;
    sc->blocks_off[t] = bo;
    stride *= b;
    nblk += d / b;
    th += (d / b) * (b == 2 ? 1 : b * (b - 1) / 2);
    if (!pow2(b)) fb += (int64_t)b * b;
    bo += (int64_t)4 * ((b * b + 3) / 4) * (d / b);   // quads of coefficients, the last one padded
  }
  sc->block_begin[nstages] = nblk;
  *d_out = (int32_t)d;
  return HR_OK;
}

int32_t hr_harp_blocks(const int32_t* radices, int32_t nstages, const float* theta,
                       const float* fallbacks, float* blocks, void* stream) {
  const char* fn = "hr_harp_blocks";
  hr::HarpSchedule sc;
  int32_t d = 0;
  const int32_t st = harp_schedule(fn, radices, nstages, &d, &sc);
  if (st) return st;
  bool need_fb = false;
  for (int t = 0; t < nstages; ++t) need_fb |= !pow2(radices[t]);
  if (!theta || !blocks) return fail(HR_EINVAL, "%s: theta and blocks are required", fn);
  if (need_fb && !fallbacks)
    return fail(HR_EINVAL, "%s: a radix is not a power of two but fallbacks is NULL", fn);
  if (!aligned16(theta) || !aligned16(blocks) || (fallbacks && !aligned16(fallbacks)))
    return fail(HR_EINVAL, "%s: pointers must be 16-byte aligned", fn);
  return from_hip(hr::launch_harp_blocks(sc, theta, fallbacks, blocks, static_cast<hipStream_t>(stream)),
                  fn);
}

int32_t hr_harp_apply(const float* x, float* y, int64_t rows, const int32_t* radices, int32_t nstages,
                      const float* blocks, int32_t inverse, int32_t group, uint8_t* codes,
                      void* scales, int32_t scale_dtype, void* stream) {
  const char* fn = "hr_harp_apply";
  hr::HarpSchedule sc;
  int32_t d = 0;
  const int32_t st = harp_schedule(fn, radices, nstages, &d, &sc);
  if (st) return st;
  if (rows < 0) return fail(HR_EINVAL, "%s: rows < 0", fn);
  if (!blocks) return fail(HR_EINVAL, "%s: blocks is required", fn);
  if (!x && rows > 0) return fail(HR_EINVAL, "%s: x is NULL", fn);
  if (!y && !codes && rows > 0) return fail(HR_EINVAL, "%s: y and codes are both NULL", fn);
  if (!codes && scales) return fail(HR_EINVAL, "%s: scales given without codes", fn);
  if (codes && !scales) return fail(HR_EINVAL, "%s: codes given without scales", fn);
  if (!aligned16(x) || (y && !aligned16(y)) || !aligned16(blocks) || (codes && !aligned16(codes)) ||
      (scales && !aligned16(scales)))
    return fail(HR_EINVAL, "%s: pointers must be 16-byte aligned", fn);
  if (inverse != 0 && inverse != 1) return fail(HR_EINVAL, "%s: inverse must be 0 or 1", fn);
  if (codes) {
    if (scale_dtype != HR_F16 && scale_dtype != HR_F32)
      return fail(HR_EINVAL, "%s: scale_dtype must be HR_F16 or HR_F32", fn);
    if (!valid_group(group) || d % group)
      return fail(HR_EUNSUPPORTED, "%s: group=%d invalid for d=%d", fn, group, d);
  }
  if (rows == 0) return ok();
  hr::HarpArgs a{};
  a.x = x;
  a.y = y;
  a.rows = rows;
  a.d = d;
  a.sc = sc;
  a.blocks = blocks;
  a.inverse = inverse;
  a.group = group;
  a.codes = codes;
  a.scales = scales;
  a.scale_f16 = scale_dtype == HR_F16;
  return from_hip(hr::launch_harp_apply(a, static_cast<hipStream_t>(stream)), fn);
}

int32_t hr_dequant_int4(const uint8_t* codes, const void* scales, int32_t scale_dtype, int64_t rows,
                        int32_t n, int32_t group, float* out, void* stream) {
  const char* fn = "hr_dequant_int4";
  if (rows < 0) return fail(HR_EINVAL, "%s: rows < 0", fn);
  if ((!codes || !scales || !out) && rows > 0)
    return fail(HR_EINVAL, "%s: codes, scales and out are required", fn);
  if (!aligned16(codes) || !aligned16(scales) || !aligned16(out))
    return fail(HR_EINVAL, "%s: pointers must be 16-byte aligned", fn);
  if (scale_dtype != HR_F16 && scale_dtype != HR_F32)
    return fail(HR_EINVAL, "%s: scale_dtype must be HR_F16 or HR_F32", fn);
  if (!valid_group(group)) return fail(HR_EUNSUPPORTED, "%s: group=%d not in {32,64,128,256}", fn, group);
  if (n <= 0 || n % group || n > (1 << 30))
    return fail(HR_EUNSUPPORTED, "%s: n=%d must be a positive multiple of group=%d", fn, n, group);
  if (rows == 0) return ok();
  return from_hip(hr::launch_dequant(codes, scales, scale_dtype == HR_F16, rows, n, group, out,
                                     static_cast<hipStream_t>(stream)), fn);
}

// Shared body of hr_w4a4_gemm, hr_w4a8_gemm and hr_w8a8_gemm.
static int32_t gemm(const char* fn, int a_int8, int w_int8, const uint8_t* a_codes, const void* a_scales,
                    const uint8_t* w_codes, const void* w_scales, int32_t scale_dtype, int64_t M,
                    int64_t N, int64_t K, int32_t group, float* c, int32_t* group_acc,
                    void* stream) {
  if (M < 0 || N < 0 || K < 0) return fail(HR_EINVAL, "%s: negative size", fn);
  if (M > 0 && N > 0 && (!a_codes || !a_scales || !w_codes || !w_scales || !c))
    return fail(HR_EINVAL, "%s: a_codes, a_scales, w_codes, w_scales and c are required", fn);
  if (!aligned16(a_codes) || !aligned16(a_scales) || !aligned16(w_codes) || !aligned16(w_scales) ||
      !aligned16(c) || (group_acc && !aligned16(group_acc)))
    return fail(HR_EINVAL, "%s: pointers must be 16-byte aligned", fn);
  if (scale_dtype != HR_F16 && scale_dtype != HR_F32)
    return fail(HR_EINVAL, "%s: scale_dtype must be HR_F16 or HR_F32", fn);
  if (!valid_group(group)) return fail(HR_EUNSUPPORTED, "%s: group=%d not in {32,64,128,256}", fn, group);
  if (N % 64) return fail(HR_EUNSUPPORTED, "%s: N=%lld is not a multiple of 64", fn, (long long)N);
  if (K == 0 || K % 256 || K % group || K > 65536)
    return fail(HR_EUNSUPPORTED, "%s: K=%lld must be a multiple of 256 and of group, <= 65536", fn,
                (long long)K);
  if (M == 0 || N == 0) return ok();
  hr::GemmArgs a{};
  a.a = a_codes;
  a.a_int8 = a_int8;
  a.w_int8 = w_int8;
  a.sa = a_scales;
  a.w = w_codes;
  a.sw = w_scales;
  a.scale_f16 = scale_dtype == HR_F16;
  a.M = M;
  a.N = N;
  a.K = K;
  a.group = group;
  a.c = c;
  a.group_acc = group_acc;
  return from_hip(hr::launch_gemm(a, static_cast<hipStream_t>(stream)), fn);
}

int32_t hr_w4a4_gemm(const uint8_t* a_codes, const void* a_scales, const uint8_t* w_codes,
                     const void* w_scales, int32_t scale_dtype, int64_t M, int64_t N, int64_t K,
                     int32_t group, float* c, int32_t* group_acc, void* stream) {
  return gemm("hr_w4a4_gemm", 0, 0, a_codes, a_scales, w_codes, w_scales, scale_dtype, M, N, K, group,
              c, group_acc, stream);
}

int32_t hr_w4a8_gemm(const int8_t* a_codes, const void* a_scales, const uint8_t* w_codes,
                     const void* w_scales, int32_t scale_dtype, int64_t M, int64_t N, int64_t K,
                     int32_t group, float* c, int32_t* group_acc, void* stream) {
  return gemm("hr_w4a8_gemm", 1, 0, reinterpret_cast<const uint8_t*>(a_codes), a_scales, w_codes,
              w_scales, scale_dtype, M, N, K, group, c, group_acc, stream);
}

int32_t hr_w8a8_gemm(const int8_t* a_codes, const void* a_scales, const int8_t* w_codes,
                     const void* w_scales, int32_t scale_dtype, int64_t M, int64_t N, int64_t K,
                     int32_t group, float* c, int32_t* group_acc, void* stream) {
  return gemm("hr_w8a8_gemm", 1, 1, reinterpret_cast<const uint8_t*>(a_codes), a_scales,
              reinterpret_cast<const uint8_t*>(w_codes), w_scales, scale_dtype, M, N, K, group, c,
              group_acc, stream);
}

int32_t hr_rotate_quant_w4a4_gemm(const void* x, int32_t x_dtype, const int8_t* signs, int32_t group,
                                  const uint8_t* w_codes, const void* w_scales, int32_t scale_dtype,
                                  int64_t M, int64_t N, int64_t K, float* c, uint8_t* a_codes,
                                  void* a_scales, void* stream) {
  const char* fn = "hr_rotate_quant_w4a4_gemm";
  if (M < 0 || N < 0 || K < 0) return fail(HR_EINVAL, "%s: negative size", fn);
  if (M > 0 && N > 0 && (!x || !w_codes || !w_scales || !c))
    return fail(HR_EINVAL, "%s: x, w_codes, w_scales and c are required", fn);
  if ((a_codes == nullptr) != (a_scales == nullptr))
    return fail(HR_EINVAL, "%s: a_codes and a_scales are given together or not at all", fn);
  if (!aligned16(x) || (signs && !aligned16(signs)) || !aligned16(w_codes) || !aligned16(w_scales) ||
      !aligned16(c) || (a_codes && !aligned16(a_codes)) || (a_scales && !aligned16(a_scales)))
    return fail(HR_EINVAL, "%s: pointers must be 16-byte aligned", fn);
  if (x_dtype != HR_BF16) return fail(HR_EUNSUPPORTED, "%s: x_dtype must be HR_BF16", fn);
  if (scale_dtype != HR_F16 && scale_dtype != HR_F32)
    return fail(HR_EINVAL, "%s: scale_dtype must be HR_F16 or HR_F32", fn);
  if (!valid_group(group)) return fail(HR_EUNSUPPORTED, "%s: group=%d not in {32,64,128,256}", fn, group);
  if (M > 16) return fail(HR_EUNSUPPORTED, "%s: M=%lld > 16 (decode shapes only)", fn, (long long)M);
  if (K != 2048 && K != 4096) return fail(HR_EUNSUPPORTED, "%s: K=%lld not 2048 or 4096", fn, (long long)K);
  if (N % 64) return fail(HR_EUNSUPPORTED, "%s: N=%lld is not a multiple of 64", fn, (long long)N);
  if (M == 0 || N == 0) return ok();
  hr::FusedDecodeArgs a{};
  a.x = static_cast<const uint16_t*>(x);
  a.signs = signs;
  a.norm = (float)(1.0 / sqrt((double)K));
  a.w = w_codes;
  a.sw = w_scales;
  a.scale_f16 = scale_dtype == HR_F16;
  a.M = M;
  a.N = N;
  a.K = K;
  a.group = group;
  a.c = c;
  a.a_codes = a_codes;
  a.a_scales = a_scales;
  return from_hip(hr::launch_rotate_quant_gemm_decode(a, static_cast<hipStream_t>(stream)), fn);
}

int32_t hr_w4a4_to_fp6(const uint8_t* codes, const void* scales, int32_t scale_dtype, int64_t rows, int64_t K,
                       int32_t group, uint8_t* out, void* out_scales, void* stream) {
  const char* fn = "hr_w4a4_to_fp6";
  if (rows < 0 || K < 0) return fail(HR_EINVAL, "%s: negative size", fn);
  if (rows > 0 && K > 0 && (!codes || !out)) return fail(HR_EINVAL, "%s: codes and out are required", fn);
  if (!scales != !out_scales) return fail(HR_EINVAL, "%s: scales and out_scales go together", fn);
  if (!aligned16(codes) || !aligned16(out) || !aligned16(scales) || !aligned16(out_scales))
    return fail(HR_EINVAL, "%s: pointers must be 16-byte aligned", fn);
  if (K % 128 || K > (int64_t(1) << 30))
    return fail(HR_EUNSUPPORTED, "%s: K=%lld must be a multiple of 128", fn, (long long)K);
  if (rows > int64_t(128) * 65535)
    return fail(HR_EUNSUPPORTED, "%s: rows=%lld above 128 * 65535", fn, (long long)rows);
  if (scales) {
    if (scale_dtype != HR_F16 && scale_dtype != HR_F32)
      return fail(HR_EINVAL, "%s: scale_dtype must be HR_F16 or HR_F32", fn);
    if ((group != 128 && group != 256) || K % group)
      return fail(HR_EUNSUPPORTED, "%s: group=%d must be 128 or 256 and divide K", fn, group);
  }
  if (rows == 0 || K == 0) return ok();
  return from_hip(hr::launch_int4_to_fp6(codes, scales, scale_dtype == HR_F16, rows, K, group, out, out_scales,
                                         static_cast<hipStream_t>(stream)),
                  fn);
}

int32_t hr_rotate_quant_fp6(const void* x, int32_t x_dtype, const int8_t* signs, int64_t rows, int32_t n,
                            int32_t group, int32_t scale_dtype, uint8_t* tiles, void* scales, void* stream) {
  const char* fn = "hr_rotate_quant_fp6";
  if (rows < 0) return fail(HR_EINVAL, "%s: rows < 0", fn);
  if (rows > 0 && (!x || !tiles || !scales)) return fail(HR_EINVAL, "%s: x, tiles and scales are required", fn);
  if (x_dtype != HR_BF16) return fail(HR_EUNSUPPORTED, "%s: x_dtype must be HR_BF16", fn);
  if (!aligned16(x) || !aligned16(tiles) || !aligned16(scales))
    return fail(HR_EINVAL, "%s: x, tiles and scales must be 16-byte aligned", fn);
  if (scale_dtype != HR_F16 && scale_dtype != HR_F32)
    return fail(HR_EINVAL, "%s: scale_dtype must be HR_F16 or HR_F32", fn);
  if (n != 2048 && n != 4096) return fail(HR_EUNSUPPORTED, "%s: n=%d not 2048 or 4096", fn, n);
  if (group != 128 && group != 256) return fail(HR_EUNSUPPORTED, "%s: group=%d not in {128,256}", fn, group);
  if (rows == 0) return ok();
  hr::RhtArgs a{};
  a.x = x;
  a.x_bf16 = 1;
  a.rows = rows;
  a.n = n;
  a.m = 1;
  a.p = n;
  a.signs = signs;
  a.block = nullptr;
  a.y = nullptr;
  a.group = group;
  a.codes = tiles;
  a.bits = 6;
  a.scales = scales;
  a.scale_f16 = scale_dtype == HR_F16;
  if (!hr::launch_rotate_quant_fp6(a, static_cast<hipStream_t>(stream)))
    return fail(HR_EUNSUPPORTED, "%s: unsupported case", fn);
  return from_hip(hipGetLastError(), fn);
}

int32_t hr_w4a4_gemm_fp6(const uint8_t* a_f6, const void* a_scales, const uint8_t* w_f6, const void* w_scales,
                         int32_t scale_dtype, int64_t M, int64_t N, int64_t K, int32_t group, float* c,
                         int32_t* group_acc, void* stream) {
  const char* fn = "hr_w4a4_gemm_fp6";
  if (M < 0 || N < 0 || K < 0) return fail(HR_EINVAL, "%s: negative size", fn);
  if (M > 0 && N > 0 && (!a_f6 || !a_scales || !w_f6 || !w_scales || !c))
    return fail(HR_EINVAL, "%s: a_f6, a_scales, w_f6, w_scales and c are required", fn);
  if (!aligned16(a_f6) || !aligned16(a_scales) || !aligned16(w_f6) || !aligned16(w_scales) || !aligned16(c) ||
      (group_acc && !aligned16(group_acc)))
    return fail(HR_EINVAL, "%s: pointers must be 16-byte aligned", fn);
  if (scale_dtype != HR_F16 && scale_dtype != HR_F32)
    return fail(HR_EINVAL, "%s: scale_dtype must be HR_F16 or HR_F32", fn);
  if (group != 128 && group != 256)
    return fail(HR_EUNSUPPORTED, "%s: group=%d not in {128,256}", fn, group);
  if (N % 128) return fail(HR_EUNSUPPORTED, "%s: N=%lld is not a multiple of 128", fn, (long long)N);
  if (K == 0 || K % group || K > 65536)
    return fail(HR_EUNSUPPORTED, "%s: K=%lld must be a multiple of group, <= 65536", fn, (long long)K);
  if (M == 0 || N == 0) return ok();
  hr::GemmArgs a{};
  a.a = a_f6;
  a.sa = a_scales;
  a.w = w_f6;
  a.sw = w_scales;
  a.scale_f16 = scale_dtype == HR_F16;
  a.M = M;
  a.N = N;
  a.K = K;
  a.group = group;
  a.c = c;
  a.group_acc = group_acc;
  return from_hip(hr::launch_gemm_fp6(a, static_cast<hipStream_t>(stream)), fn);
}

// Vectors of one call: a launch holds fewer than 2^32 threads.
constexpr int64_t kKv4MaxVectors = int64_t(1) << 26;
constexpr int32_t kKv4MaxHeads = 65535, kKv4MaxBatch = 65535;
constexpr int32_t kKv4MaxQHeads = 1 << 22;   // times 256 dims: a row's elements are counted in 32 bits

// Checks a cache description and fills the internal one.  The arrays may be
// NULL only when no token is touched (`need` false).
static int32_t kv4_cache(const char* fn, const hr_kv4_cache* c, bool need, hr::Kv4Cache* out) {
  if (!c) return fail(HR_EINVAL, "%s: cache is NULL", fn);
  if (c->pages < 0) return fail(HR_EINVAL, "%s: pages < 0", fn);
  if (c->rotate != 0 && c->rotate != 1) return fail(HR_EINVAL, "%s: rotate must be 0 or 1", fn);
  if (need && c->pages > 0 && (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales))
    return fail(HR_EINVAL, "%s: the cache's codes and scales are required", fn);
  if (!aligned16(c->k_codes) || !aligned16(c->k_scales) || !aligned16(c->v_codes) || !aligned16(c->v_scales) ||
      !aligned16(c->signs))
    return fail(HR_EINVAL, "%s: the cache's pointers must be 16-byte aligned", fn);
  if (c->dim != 64 && c->dim != 128 && c->dim != 256)
    return fail(HR_EUNSUPPORTED, "%s: dim=%d not in {64,128,256}", fn, c->dim);
  if (!valid_group(c->group) || c->dim % c->group)
    return fail(HR_EUNSUPPORTED, "%s: group=%d invalid for dim=%d", fn, c->group, c->dim);
  if (!pow2(c->page) || c->page < 16 || c->page > (1 << 20))
    return fail(HR_EUNSUPPORTED, "%s: page=%d is not a power of two in [16, 2^20]", fn, c->page);
  if (c->heads < 1 || c->heads > kKv4MaxHeads)
    return fail(HR_EUNSUPPORTED, "%s: heads=%d outside [1, 65535]", fn, c->heads);
  if (c->pages > INT32_MAX) return fail(HR_EUNSUPPORTED, "%s: more than 2^31 - 1 pages", fn);
  *out = hr::Kv4Cache{};
  out->codes[0] = c->k_codes;
  out->codes[1] = c->v_codes;
  out->scales[0] = static_cast<_Float16*>(c->k_scales);
  out->scales[1] = static_cast<_Float16*>(c->v_scales);
  out->signs = c->rotate ? c->signs : nullptr;
  out->pages = c->pages;
  out->heads = c->heads;
  out->dim = c->dim;
  out->group = c->group;
  out->page_log2 = ilog2(c->page);
  out->rotate = c->rotate;
  return HR_OK;
}

static bool kv4_dtype(int32_t dt) { return dt == HR_F32 || dt == HR_BF16 || dt == HR_F16; }

// Rows `stride` elements apart: long enough and 16-byte aligned.
static bool kv4_stride(int64_t stride, int64_t row, int32_t dtype) {
  return stride >= row && stride % (dtype == HR_F32 ? 4 : 8) == 0;
}

int32_t hr_kv4_append(const hr_kv4_cache* cache, const void* k, const void* v, int32_t dtype, int64_t k_stride,
                      int64_t v_stride, const int64_t* slots, int64_t tokens, void* stream) {
  const char* fn = "hr_kv4_append";
  if (tokens < 0) return fail(HR_EINVAL, "%s: tokens < 0", fn);
  if (!kv4_dtype(dtype)) return fail(HR_EINVAL, "%s: dtype must be HR_F32, HR_BF16 or HR_F16", fn);
  hr::Kv4AppendArgs a{};
  const int32_t st = kv4_cache(fn, cache, tokens > 0, &a.c);
  if (st) return st;
  if (tokens > 0 && (!k || !v || !slots)) return fail(HR_EINVAL, "%s: k, v and slots are required", fn);
  if (!aligned16(k) || !aligned16(v)) return fail(HR_EINVAL, "%s: k and v must be 16-byte aligned", fn);
  if (reinterpret_cast<uintptr_t>(slots) & 7u) return fail(HR_EINVAL, "%s: slots must be 8-byte aligned", fn);
  const int64_t row = (int64_t)cache->heads * cache->dim;
  if (!kv4_stride(k_stride, row, dtype) || !kv4_stride(v_stride, row, dtype))
    return fail(HR_EINVAL, "%s: k_stride and v_stride must be at least heads * dim and multiples of 16 bytes", fn);
  if (tokens > kKv4MaxVectors / cache->heads)
    return fail(HR_EUNSUPPORTED, "%s: tokens * heads above 2^26", fn);
  if (tokens == 0 || cache->pages == 0) return ok();
  a.x[0] = k;
  a.x[1] = v;
  a.stride[0] = k_stride;
  a.stride[1] = v_stride;
  a.dtype = dtype;
  a.slots = slots;
  a.tokens = tokens;
  return from_hip(hr::launch_kv4_append(a, static_cast<hipStream_t>(stream)), fn);
}

int32_t hr_kv4_read(const hr_kv4_cache* cache, const int64_t* slots, int64_t tokens, int32_t dtype, void* k,
                    void* v, void* stream) {
  const char* fn = "hr_kv4_read";
  if (tokens < 0) return fail(HR_EINVAL, "%s: tokens < 0", fn);
  if (!kv4_dtype(dtype)) return fail(HR_EINVAL, "%s: dtype must be HR_F32, HR_BF16 or HR_F16", fn);
  hr::Kv4ReadArgs a{};
  const int32_t st = kv4_cache(fn, cache, tokens > 0, &a.c);
  if (st) return st;
  if (tokens > 0 && (!k || !v || !slots)) return fail(HR_EINVAL, "%s: k, v and slots are required", fn);
  if (!aligned16(k) || !aligned16(v)) return fail(HR_EINVAL, "%s: k and v must be 16-byte aligned", fn);
  if (reinterpret_cast<uintptr_t>(slots) & 7u) return fail(HR_EINVAL, "%s: slots must be 8-byte aligned", fn);
  if (tokens > kKv4MaxVectors / cache->heads)
    return fail(HR_EUNSUPPORTED, "%s: tokens * heads above 2^26", fn);
  if (tokens == 0) return ok();
  a.y[0] = k;
  a.y[1] = v;
  a.dtype = dtype;
  a.slots = slots;
  a.tokens = tokens;
  return from_hip(hr::launch_kv4_read(a, static_cast<hipStream_t>(stream)), fn);
}

// A window past every cached length hides nothing.  Without it the kernels' 32-bit positions cannot wrap: a first
// visible token that did would lead to page ids read far outside the table.
static int32_t kv4_window(int32_t window) { return window < hr::kKv4MaxLen ? window : 0; }

// Workspace of a planned call: partial sums, then (max, sum) pairs.
static int64_t kv4_workspace(const hr::Kv4AttnArgs& a) {
  return a.nsplit > 1 ? a.total * a.q_heads * a.nsplit * (4 * (int64_t)a.c.dim + 8) : 0;
}

int64_t hr_kv4_attention_workspace(int32_t heads, int32_t dim, int32_t dtype, int64_t total, int32_t batch,
                                   int32_t q_heads, int32_t max_new, int64_t max_len, int32_t window) {
  // nothing that the call itself refuses: the plan's products then stay in 64 bits
  if (heads < 1 || heads > kKv4MaxHeads || (dim != 64 && dim != 128 && dim != 256) || !kv4_dtype(dtype) || q_heads < 1 ||
      q_heads > kKv4MaxQHeads || q_heads % heads || total < 1 || total > kKv4MaxVectors / q_heads || batch < 1 || batch > kKv4MaxBatch || max_new < 1 ||
      max_new > kKv4MaxVectors / q_heads || max_len < 0 || max_len > hr::kKv4MaxLen || window < 0)
    return 0;
  hr::Kv4AttnArgs a{};
  a.c.heads = heads;
  a.c.dim = dim;
  a.dtype = dtype;
  a.total = total;
  a.batch = batch;
  a.q_heads = q_heads;
  a.rep = q_heads / heads;
  a.max_new = max_new;
  a.max_len = max_len;
  a.window = kv4_window(window);
  // the plan also looks at whether a head has several scale groups: enough for either
  int64_t need = 0;
  for (int group : {dim, dim / 2}) {
    a.c.group = group;
    hr::kv4_attention_plan(&a);
    need = std::max(need, kv4_workspace(a));
  }
  return need;
}

int32_t hr_kv4_attention(const hr_kv4_cache* cache, const void* q, int32_t dtype, int64_t q_stride, int64_t total,
                         const int32_t* starts, const int32_t* table, int64_t width, const int32_t* lens,
                         int32_t batch, int32_t q_heads, int32_t max_new, int64_t max_len, float scale,
                         int32_t causal, int32_t window, void* out, void* workspace, int64_t workspace_bytes,
                         void* stream) {
  const char* fn = "hr_kv4_attention";
  if (total < 0 || batch < 0 || width < 0 || max_new < 0 || max_len < 0 || window < 0 || workspace_bytes < 0)
    return fail(HR_EINVAL, "%s: negative size", fn);
  if (!kv4_dtype(dtype)) return fail(HR_EINVAL, "%s: dtype must be HR_F32, HR_BF16 or HR_F16", fn);
  if (causal != 0 && causal != 1) return fail(HR_EINVAL, "%s: causal must be 0 or 1", fn);
  if (!(scale > 0.0f) || !(scale <= 3.4028235e38f)) return fail(HR_EINVAL, "%s: scale must be positive and finite", fn);
  hr::Kv4AttnArgs a{};
  const bool some = total > 0 && batch > 0;
  const int32_t st = kv4_cache(fn, cache, some, &a.c);
  if (st) return st;
  if (some && (!q || !lens || !out || (!table && width > 0)))
    return fail(HR_EINVAL, "%s: q, table, lens and out are required", fn);
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace))
    return fail(HR_EINVAL, "%s: q, out and workspace must be 16-byte aligned", fn);
  if ((reinterpret_cast<uintptr_t>(starts) | reinterpret_cast<uintptr_t>(table) | reinterpret_cast<uintptr_t>(lens)) & 3u)
    return fail(HR_EINVAL, "%s: starts, table and lens must be 4-byte aligned", fn);
  if (q_heads < 1 || q_heads % cache->heads)
    return fail(HR_EUNSUPPORTED, "%s: q_heads=%d is not a multiple of heads=%d", fn, q_heads, cache->heads);
  if (q_heads > kKv4MaxQHeads) return fail(HR_EUNSUPPORTED, "%s: q_heads=%d above 2^22", fn, q_heads);
  if (!kv4_stride(q_stride, (int64_t)q_heads * cache->dim, dtype))
    return fail(HR_EINVAL, "%s: q_stride must be at least q_heads * dim and a multiple of 16 bytes", fn);
  if (!starts && (int64_t)batch * max_new != total)
    return fail(HR_EINVAL, "%s: without starts, total must be batch * max_new", fn);
  if (total > kKv4MaxVectors / q_heads || max_new > kKv4MaxVectors / q_heads)
    return fail(HR_EUNSUPPORTED, "%s: rows * q_heads above 2^26", fn);
  if (batch > kKv4MaxBatch) return fail(HR_EUNSUPPORTED, "%s: batch=%d above %d", fn, batch, kKv4MaxBatch);
  if (width > INT32_MAX) return fail(HR_EUNSUPPORTED, "%s: width above 2^31 - 1", fn);
  if (max_len > hr::kKv4MaxLen) return fail(HR_EUNSUPPORTED, "%s: max_len above 2^30", fn);
  if (!some || max_new == 0) return ok();
  a.q = q;
  a.q_stride = q_stride;
  a.dtype = dtype;
  a.total = total;
  a.starts = starts;
  a.table = table;
  a.width = cache->pages > 0 ? width : 0;
  a.lens = lens;
  a.batch = batch;
  a.q_heads = q_heads;
  a.rep = q_heads / cache->heads;
  a.max_new = max_new;
  a.max_len = max_len;
  a.scale = scale;
  a.causal = causal;
  a.window = kv4_window(window);
  a.out = out;
  hr::kv4_attention_plan(&a);
  if (a.groups > (1 << 22))
    return fail(HR_EUNSUPPORTED, "%s: too many rows for one launch", fn);
  const int64_t need = kv4_workspace(a);
  if (need > 0) {
    if (!workspace || workspace_bytes < need)
      return fail(HR_EINVAL, "%s: workspace of %lld bytes needed", fn, (long long)need);
    a.part_o = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + total * q_heads * a.nsplit * cache->dim);
  }
  return from_hip(hr::launch_kv4_attention(a, static_cast<hipStream_t>(stream)), fn);
}

// ---------------------------------------------------------------- MXFP4

static bool mx_order(int32_t order) { return order == 32 || order == 64 || order == 128 || order == 256; }

// What quantizing rows and reading them back have in common.
static int32_t mx_rows(const char* fn, int64_t rows, int32_t n, int32_t order, const int8_t* signs) {
  if (rows < 0) return fail(HR_EINVAL, "%s: rows < 0", fn);
  if (!aligned16(signs)) return fail(HR_EINVAL, "%s: signs must be 16-byte aligned", fn);
  if (n <= 0 || n % hr::kMxBlock || n > hr::kMxMaxN)
    return fail(HR_EUNSUPPORTED, "%s: n=%d is not a multiple of 32 in [32, 2^18]", fn, n);
  if (order != 0 && (!mx_order(order) || n % order))
    return fail(HR_EUNSUPPORTED, "%s: order=%d not in {32,64,128,256} or not dividing n=%d", fn, order, n);
  if (rows > (int64_t(1) << 34) / n) return fail(HR_EUNSUPPORTED, "%s: rows * n above 2^34", fn);
  return HR_OK;
}

static int32_t mx_quant(const char* fn, const void* x, int32_t x_dtype, int64_t x_stride, int64_t rows, int32_t n,
                        int32_t order, const int8_t* signs, int32_t rule, uint8_t* codes, uint8_t* scales,
                        void* stream) {
  const int32_t st = mx_rows(fn, rows, n, order, signs);
  if (st) return st;
  if (!kv4_dtype(x_dtype)) return fail(HR_EINVAL, "%s: x_dtype must be HR_F32, HR_BF16 or HR_F16", fn);
  if (rule != HR_MX_FLOOR && rule != HR_MX_CEIL)
    return fail(HR_EINVAL, "%s: rule must be HR_MX_FLOOR or HR_MX_CEIL", fn);
  if (rows > 0 && (!x || !codes || !scales)) return fail(HR_EINVAL, "%s: x, codes and scales are required", fn);
  if (!aligned16(x) || !aligned16(codes))
    return fail(HR_EINVAL, "%s: x and codes must be 16-byte aligned", fn);
  if (!kv4_stride(x_stride, n, x_dtype))
    return fail(HR_EINVAL, "%s: x_stride must be at least n and a multiple of 16 bytes", fn);
  if (rows == 0) return ok();
  hr::Mx4QuantArgs a{};
  a.x = x;
  a.dtype = x_dtype;
  a.x_stride = x_stride;
  a.rows = rows;
  a.n = n;
  a.order = order;
  a.signs = signs;
  a.ceil = rule == HR_MX_CEIL;
  a.codes = codes;
  a.scales = scales;
  return from_hip(hr::launch_mx4_quant(a, static_cast<hipStream_t>(stream)), fn);
}

int32_t hr_quant_mxfp4(const void* x, int32_t x_dtype, int64_t x_stride, int64_t rows, int32_t n, int32_t rule,
                       uint8_t* codes, uint8_t* scales, void* stream) {
  return mx_quant("hr_quant_mxfp4", x, x_dtype, x_stride, rows, n, 0, nullptr, rule, codes, scales, stream);
}

int32_t hr_rotate_quant_mxfp4(const void* x, int32_t x_dtype, int64_t x_stride, int64_t rows, int32_t n,
                              int32_t order, const int8_t* signs, int32_t rule, uint8_t* codes, uint8_t* scales,
                              void* stream) {
  if (!mx_order(order))
    return fail(HR_EUNSUPPORTED, "hr_rotate_quant_mxfp4: order=%d not in {32,64,128,256}", order);
  return mx_quant("hr_rotate_quant_mxfp4", x, x_dtype, x_stride, rows, n, order, signs, rule, codes, scales, stream);
}

int32_t hr_dequant_mxfp4(const uint8_t* codes, const uint8_t* scales, int64_t rows, int32_t n, int32_t order,
                         const int8_t* signs, int32_t dtype, void* out, void* stream) {
  const char* fn = "hr_dequant_mxfp4";
  const int32_t st = mx_rows(fn, rows, n, order, signs);
  if (st) return st;
  if (!kv4_dtype(dtype)) return fail(HR_EINVAL, "%s: dtype must be HR_F32, HR_BF16 or HR_F16", fn);
  if (order == 0 && signs) return fail(HR_EINVAL, "%s: signs go with an order", fn);
  if (rows > 0 && (!codes || !scales || !out)) return fail(HR_EINVAL, "%s: codes, scales and out are required", fn);
  if (!aligned16(codes) || !aligned16(out))
    return fail(HR_EINVAL, "%s: codes and out must be 16-byte aligned", fn);
  if (rows == 0) return ok();
  hr::Mx4DequantArgs a{};
  a.codes = codes;
  a.scales = scales;
  a.rows = rows;
  a.n = n;
  a.order = order;
  a.signs = signs;
  a.dtype = dtype;
  a.y = out;
  return from_hip(hr::launch_mx4_dequant(a, static_cast<hipStream_t>(stream)), fn);
}

int32_t hr_mxfp4_gemm(const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* w_codes,
                      const uint8_t* w_scales, int64_t M, int64_t N, int64_t K, int32_t dtype, void* c, void* stream) {
  const char* fn = "hr_mxfp4_gemm";
  if (M < 0 || N < 0) return fail(HR_EINVAL, "%s: negative size", fn);
  if (!kv4_dtype(dtype)) return fail(HR_EINVAL, "%s: dtype must be HR_F32, HR_BF16 or HR_F16", fn);
  if (K <= 0 || K % hr::kMxBlock || K > hr::kMxMaxN)
    return fail(HR_EUNSUPPORTED, "%s: K=%lld is not a multiple of 32 in [32, 2^18]", fn, (long long)K);
  // what one launch holds: 2^20 tiles of 256 x 256 (K below 128: 2^22 of 128 x 128)
  if (M > (1 << 21) || N > (1 << 21) || M * N > int64_t(1) << 36)
    return fail(HR_EUNSUPPORTED, "%s: M=%lld, N=%lld too large", fn, (long long)M, (long long)N);
  const bool some = M > 0 && N > 0;
  if (some && (!a_codes || !a_scales || !w_codes || !w_scales || !c))
    return fail(HR_EINVAL, "%s: codes, scales and c are required", fn);
  if (!aligned16(a_codes) || !aligned16(w_codes) || !aligned16(c))
    return fail(HR_EINVAL, "%s: codes and c must be 16-byte aligned", fn);
  if (!some) return ok();
  hr::Mx4GemmArgs a{};
  a.a = a_codes;
  a.sa = a_scales;
  a.w = w_codes;
  a.sw = w_scales;
  a.M = M;
  a.N = N;
  a.K = (int)K;
  a.dtype = dtype;
  a.c = c;
  return from_hip(hr::launch_mx4_gemm(a, static_cast<hipStream_t>(stream)), fn);
}

// ---------------------------------------------------------------- norms

// Checks of hr_norm_residual and its quantizing form; fills the internal arguments.
static int32_t norm_args(const char* fn, const hr_norm* p, void* residual, int64_t residual_stride, hr::NormArgs* out) {
  if (!p) return fail(HR_EINVAL, "%s: the description is NULL", fn);
  if (p->rows < 0) return fail(HR_EINVAL, "%s: rows < 0", fn);
  if (!kv4_dtype(p->x_dtype) || !kv4_dtype(p->dtype))
    return fail(HR_EINVAL, "%s: x_dtype and dtype must be HR_F32, HR_BF16 or HR_F16", fn);
  if (p->x_dtype != HR_F32 && p->x_dtype != p->dtype)
    return fail(HR_EUNSUPPORTED, "%s: dtype must be x_dtype unless that is HR_F32", fn);
  if (p->post_norm != 0 && p->post_norm != 1) return fail(HR_EINVAL, "%s: post_norm must be 0 or 1", fn);
  if (!(p->eps >= 0.0f) || !(p->eps <= 3.4028235e38f) || !(fabsf(p->scale) <= 3.4028235e38f))
    return fail(HR_EINVAL, "%s: eps must be finite and not negative, scale finite", fn);
  if (p->n < 1 || p->n > hr::kNormMaxN) return fail(HR_EUNSUPPORTED, "%s: n=%d outside [1, %d]", fn, p->n, hr::kNormMaxN);
  if (p->rows > (1 << 24)) return fail(HR_EUNSUPPORTED, "%s: more than 2^24 rows", fn);
  if (p->rows > 0 && !p->x) return fail(HR_EINVAL, "%s: x is NULL", fn);
  if (p->block_out) {
    if (!residual) return fail(HR_EINVAL, "%s: residual is NULL", fn);
    if (p->block_stride < p->n || residual_stride < p->n)
      return fail(HR_EINVAL, "%s: block_stride and residual_stride must be at least n", fn);
    if (p->gate && (p->gates < 1 || p->rows % p->gates))
      return fail(HR_EINVAL, "%s: gates=%lld does not divide rows", fn, (long long)p->gates);
    if (p->post_weight && !p->post_norm) return fail(HR_EINVAL, "%s: post_weight goes with post_norm", fn);
  } else if (p->rows > 0 && (residual || p->gate || p->post_norm || p->post_weight)) {
    return fail(HR_EINVAL, "%s: residual, gate and post_norm go with block_out", fn);
  }
  if (p->x_stride < p->n) return fail(HR_EINVAL, "%s: x_stride must be at least n", fn);
  const uintptr_t xs = p->x_dtype == HR_F32 ? 3u : 1u, ds = p->dtype == HR_F32 ? 3u : 1u;
  if (((reinterpret_cast<uintptr_t>(p->x) | reinterpret_cast<uintptr_t>(residual)) & xs) ||
      ((reinterpret_cast<uintptr_t>(p->block_out) | reinterpret_cast<uintptr_t>(p->gate)) & ds) ||
      ((reinterpret_cast<uintptr_t>(p->weight) | reinterpret_cast<uintptr_t>(p->post_weight)) & 3u))
    return fail(HR_EINVAL, "%s: every array must be aligned to its elements", fn);
  *out = hr::NormArgs{};
  out->x = p->x;
  out->block = p->block_out;
  out->post_weight = p->post_weight;
  out->gate = p->gate;
  out->weight = p->weight;
  out->x_stride = p->x_stride;
  out->block_stride = p->block_stride;
  out->residual_stride = residual_stride;
  out->rows = p->rows;
  out->gate_rows = p->gate && p->gates > 0 && p->rows > 0 ? p->rows / p->gates : 1;
  out->n = p->n;
  out->x_dtype = p->x_dtype;
  out->dtype = p->dtype;
  out->post_norm = p->post_norm;
  out->scale = p->scale;
  out->eps = p->eps;
  out->residual = residual;
  return HR_OK;
}

int32_t hr_norm_residual(const hr_norm* p, void* residual, int64_t residual_stride, void* h, void* stream) {
  const char* fn = "hr_norm_residual";
  hr::NormArgs a{};
  const int32_t st = norm_args(fn, p, residual, residual_stride, &a);
  if (st) return st;
  if (reinterpret_cast<uintptr_t>(h) & (p->dtype == HR_F32 ? 3u : 1u))
    return fail(HR_EINVAL, "%s: h must be aligned to its elements", fn);
  if (p->rows > 0 && !h && !p->block_out) return fail(HR_EINVAL, "%s: neither block_out nor h", fn);
  if (p->rows == 0) return ok();
  a.h = h;
  return from_hip(hr::launch_norm(a, static_cast<hipStream_t>(stream)), fn);
}

int32_t hr_norm_residual_quant_mxfp4(const hr_norm* p, void* residual, int64_t residual_stride, int32_t order,
                                     const int8_t* signs, int32_t rule, uint8_t* codes, uint8_t* scales,
                                     void* stream) {
  const char* fn = "hr_norm_residual_quant_mxfp4";
  hr::NormArgs a{};
  int32_t st = norm_args(fn, p, residual, residual_stride, &a);
  if (st) return st;
  st = mx_rows(fn, p->rows, p->n, order, signs);
  if (st) return st;
  if (rule != HR_MX_FLOOR && rule != HR_MX_CEIL)
    return fail(HR_EINVAL, "%s: rule must be HR_MX_FLOOR or HR_MX_CEIL", fn);
  if (order == 0 && signs) return fail(HR_EINVAL, "%s: signs go with an order", fn);
  if (p->rows > 0 && (!codes || !scales)) return fail(HR_EINVAL, "%s: codes and scales are required", fn);
  if (!aligned16(codes)) return fail(HR_EINVAL, "%s: codes must be 16-byte aligned", fn);
  if (p->rows == 0) return ok();
  a.order = order;
  a.signs = signs;
  a.ceil = rule == HR_MX_CEIL;
  a.codes = codes;
  a.scales = scales;
  return from_hip(hr::launch_norm(a, static_cast<hipStream_t>(stream)), fn);
}

}  // extern "C"
