// Host side of the matrix-vector products with group scales (include/mmq_q4g.h): argument checks and
// launches. As in api.cpp nothing touches the device before every argument has been checked.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "api_util.h"
#include "mmq.h"
#include "mmq_layer.h"
#include "mmq_q4g.h"
#include "q4g_internal.h"

namespace {

using mmq::check_pointers;
using mmq::fail;
using mmq::hip_status;
using mmq::Q4GShape;

static_assert(MMQ_F32 == mmq::kTypeF32 && MMQ_F16 == mmq::kTypeF16 && MMQ_BF16 == mmq::kTypeBF16,
              "types");
static_assert(MMQ_Q4G_MAX_TOKENS == mmq::kG4MaxTokens, "limits");

int check_weights(int64_t N, int64_t K, const mmq_q4G_format* f, Q4GShape* out) {
  if (!f) return fail(MMQ_E_ARG, "format is NULL");
  if (f->reserved != 0) return fail(MMQ_E_ARG, "mmq_q4G_format.reserved must be 0");
  if (f->zeros != 0 && f->zeros != 1) return fail(MMQ_E_ARG, "mmq_q4G_format.zeros must be 0 or 1");
  if (f->scale_type != MMQ_F16 && f->scale_type != MMQ_BF16)
    return fail(MMQ_E_ARG, "scale type %d is neither MMQ_F16 nor MMQ_BF16", f->scale_type);
  if (f->group <= 0) return fail(MMQ_E_ARG, "group %d must be positive", f->group);
  if (N <= 0 || K <= 0)
    return fail(MMQ_E_ARG, "N and K must be positive (%lld, %lld)", (long long)N, (long long)K);
  if (K % 32) return fail(MMQ_E_SHAPE, "K = %lld is not a multiple of 32", (long long)K);
  if (f->group % 32 && f->group < K)
    return fail(MMQ_E_SHAPE, "group %d is neither a multiple of 32 nor K or more", f->group);
  // a grid holds fewer than 2^32 work-items: up to 1024 per 16 rows of the product, 256 per record of
  // the repack
  if (N > ((int64_t)1 << 25) || K > ((int64_t)1 << 24))
    return fail(MMQ_E_SHAPE, "N = %lld or K = %lld too large", (long long)N, (long long)K);
  *out = Q4GShape{N, K, f->group < K ? f->group : K, f->zeros != 0};
  if (out->tiles() * out->records() >= ((int64_t)1 << 24))
    return fail(MMQ_E_SHAPE, "N = %lld, K = %lld: 2^24 records of 16 x 128 values or more",
                (long long)N, (long long)K);
  return MMQ_OK;
}

bool is_type(int32_t t) { return t >= MMQ_F32 && t <= MMQ_BF16; }

}  // namespace

extern "C" {

int mmq_q4G_repacked_bytes(int64_t N, int64_t K, const mmq_q4G_format* format, size_t* bytes) {
  if (!bytes) return fail(MMQ_E_ARG, "bytes is NULL");
  Q4GShape g;
  const int st = check_weights(N, K, format, &g);
  if (st) return st;
  *bytes = (size_t)g.bytes();
  return mmq::api_ok();
}

int repack_q4_G(const void* w, const void* scales, const void* zeros, int64_t N, int64_t K,
                const mmq_q4G_format* format, void* w_rep, void* stream) {
  Q4GShape g;
  int st = check_weights(N, K, format, &g);
  if (!st && g.zeros != (zeros != nullptr))
    st = fail(MMQ_E_ARG, "zeros must be given where the format has them, and only there");
  if (!st) st = check_pointers({w, scales, w_rep}, zeros);
  if (!st) st = mmq::api_current_device();
  if (st) return st;
  return hip_status("repack_q4_G", mmq::launch_repack_q4g(w, scales, zeros, g, w_rep,
                                                          static_cast<hipStream_t>(stream)));
}

int mmq_q4G(int64_t M, int64_t N, int64_t K, int32_t x_type, const void* x, const void* w_rep,
            const mmq_q4G_format* format, int32_t y_type, void* y, const mmq_q4G_epilogue* epi,
            void* stream) {
  Q4GShape g;
  int st = check_weights(N, K, format, &g);
  if (!st && M <= 0) st = fail(MMQ_E_ARG, "M must be positive (%lld)", (long long)M);
  if (!st && M > MMQ_Q4G_MAX_TOKENS)
    st = fail(MMQ_E_SHAPE, "M = %lld is above %d tokens", (long long)M, MMQ_Q4G_MAX_TOKENS);
  if (!st && (!is_type(x_type) || !is_type(y_type)))
    st = fail(MMQ_E_ARG, "x or y type (%d, %d) is not an mmq_type", x_type, y_type);
  mmq::Q4GEpilogue e{nullptr, nullptr, MMQ_ACT_NONE};
  if (!st && epi) {
    if (epi->reserved != 0) st = fail(MMQ_E_ARG, "mmq_q4G_epilogue.reserved must be 0");
    else if (epi->act < MMQ_ACT_NONE || epi->act > MMQ_ACT_GELU_TANH)
      st = fail(MMQ_E_ARG, "act %d is not an mmq_act", epi->act);
    e = mmq::Q4GEpilogue{epi->bias, epi->residual, epi->act};
  }
  if (!st) st = check_pointers({x, w_rep, y}, e.bias);
  if (!st) st = check_pointers({}, e.residual);
  int64_t budget = 0, cus = 0;
  if (!st) st = mmq::api_current_device(&budget, &cus);
  if (st) return st;
  const int64_t need = mmq::q4g_lds_bytes(x_type, M, g, cus);
  if (need > budget)
    return fail(MMQ_E_LDS, "the product needs %lld bytes of LDS, the device allows %lld",
                (long long)need, (long long)budget);
  return hip_status("mmq_q4G", mmq::launch_q4g(x, x_type, w_rep, format->scale_type, y, y_type, M, g,
                                               e, cus, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
