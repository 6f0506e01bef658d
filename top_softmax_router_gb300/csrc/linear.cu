// Products grouped by expert (include/moe_linear.h): checks, the workspace and the launches of linear_gemm.cuh.
#include <algorithm>

#include "../../include/moe_blocks8.h"
#include "../../include/moe_linear.h"
#include "linear_gemm.cuh"

namespace moe {
namespace {

inline int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

int linear_validate(const moe_linear_config* c) {
  if (!c || c->N < 0 || c->K < 1 || c->O < 1 || c->E < 1 || (c->blocks8 != 0 && c->blocks8 != 1)) return MOE_ERR_INVALID_ARG;
  constexpr int most = 1 << 20;
  if (c->E > MOE_LINEAR_MAX_E || c->K % 16 || c->O % 16 || c->K > most || c->O > most) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (c->N > MOE_LINEAR_MAX_N) return MOE_ERR_UNSUPPORTED_SHAPE;   // a row and the kernels' steps past it are counted in 32 bits,
  if (c->blocks8 && c->N * up(std::max(c->K, c->O), MOE_BLOCK8) > INT32_MAX) return MOE_ERR_UNSUPPORTED_SHAPE;   // and so are blocks
  // and tiles
  const int64_t rows = c->N / 256 + c->E, wide = up(std::max(c->K, c->O), 256);
  if (rows * wide > INT32_MAX / 4 || c->E * up(c->K, 256) * up(c->O, 256) > INT32_MAX / 4) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

struct LinearLayout {
  size_t done, part, fwd_total, dy_codes, dy_scales, x_values, bwd_total;
};
LinearLayout linear_layout(const moe_linear_config& c) {
  LinearLayout L;
  size_t at = sizeof(WsHeader);
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align256(bytes);
    return here;
  };
  L.done = take((size_t)kLinClusters / 2 * 16 * 4);
  L.part = take((size_t)kLinClusters * 256 * 256 * 4);
  L.fwd_total = at;
  L.dy_codes = L.dy_scales = L.x_values = at;
  if (c.blocks8) {
    L.dy_codes = take((size_t)c.N * c.O);
    L.dy_scales = take((size_t)c.N * up(c.O, MOE_BLOCK8));
    L.x_values = take((size_t)c.N * c.K * 2);
  }
  L.bwd_total = at;
  return L;
}

LinGemm linear_params(const moe_linear_config& c, const LinearLayout& L, const int32_t* offsets, uint8_t* w) {
  LinGemm p = {};
  p.n = c.N;
  p.E = c.E;
  p.offsets = offsets;
  p.status = reinterpret_cast<int*>(w);
  p.limit_ns = wait_limit_ns();
  p.part = reinterpret_cast<float*>(w + L.part);
  p.done = reinterpret_cast<unsigned*>(w + L.done);
  return p;
}

bool ok16(const void* p) { return p && aligned_to(p, 16); }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_linear_workspace_bytes(const moe_linear_config* cfg, size_t* fwd_bytes, size_t* bwd_bytes) {
  const int v = linear_validate(cfg);
  if (v != MOE_OK) return v;
  const LinearLayout L = linear_layout(*cfg);
  if (fwd_bytes) *fwd_bytes = L.fwd_total;
  if (bwd_bytes) *bwd_bytes = L.bwd_total;
  return MOE_OK;
}

int moe_linear_forward(const moe_linear_config* cfg, const void* x, int64_t ldx, const uint8_t* x_scales, const void* w,
                       const uint8_t* w_scales, const int32_t* offsets, uint16_t* y, void* ws, size_t ws_bytes,
                       void* stream) {
  const int v = linear_validate(cfg);
  if (v != MOE_OK) return v;
  const moe_linear_config& c = *cfg;
  const bool mx = x_scales != nullptr;
  if (mx != (w_scales != nullptr) || ldx < c.K || ldx % (mx ? 16 : 8) || (!offsets && c.E != 1)) return MOE_ERR_INVALID_ARG;
  if (!aligned_to(offsets, 4) || !ok16(ws)) return MOE_ERR_INVALID_ARG;
  const LinearLayout L = linear_layout(c);
  if (ws_bytes < L.fwd_total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (c.N == 0) return MOE_OK;
  if (!ok16(x) || !ok16(w) || !ok16(y)) return MOE_ERR_INVALID_ARG;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  LinMaps m = {};
  const bool made = mx ? make_map_2d_u8(&m.a, x, c.K, c.N, ldx, 128, 128) && make_map_2d_u8(&m.few, x, c.K, c.N, ldx, 128, kFewRows) && make_map_3d_u8(&m.b, w, c.K, c.O, c.E, 128, 128)
                       : make_map_2d_strided(&m.a, x, c.K, c.N, ldx, 64, 128) && make_map_2d_strided(&m.few, x, c.K, c.N, ldx, 64, kFewRows) && make_map_3d(&m.b, w, c.K, c.O, c.E, 64, 128);
  if (!made) return record_cuda_error(cudaErrorInvalidValue, "linear tensor maps");
  LinGemm p = linear_params(c, L, offsets, static_cast<uint8_t*>(ws));
  p.cols = c.O;
  p.nk = (int)up(c.K, mx ? 128 : 64);
  p.tiles_n = (int)up(c.O, 256);
  p.a_scale = x_scales;
  p.lda_s = (int)up(c.K, MOE_BLOCK8);
  p.b_scale = w_scales;
  p.b_col = p.lda_s;
  p.b_k = 1;
  p.b_expert = up(c.O, MOE_BLOCK8) * p.lda_s;
  p.out = y;
  return timed_launch(MOE_K_LINEAR_Y, "linear y", s, [&] {
    return mx ? launch_linear_gemm<LIN_Y, true>(m, p, device_sm_count(), s)
              : launch_linear_gemm<LIN_Y, false>(m, p, device_sm_count(), s);
  });
}

int moe_linear_backward(const moe_linear_config* cfg, const void* x, int64_t ldx, const uint8_t* x_scales, const void* w,
                        const uint8_t* w_scales, const int32_t* offsets, const uint16_t* dy, uint16_t* dx, void* dw,
                        int32_t dw_type, void* ws, size_t ws_bytes, void* stream) {
  int v = linear_validate(cfg);
  if (v != MOE_OK) return v;
  const moe_linear_config& c = *cfg;
  const bool x8 = x_scales != nullptr, w8 = w_scales != nullptr;
  if ((!offsets && c.E != 1) || !aligned_to(offsets, 4) || !ok16(ws)) return MOE_ERR_INVALID_ARG;
  if (dw && (!ok16(dw) || (dw_type != MOE_TYPE_F32 && dw_type != MOE_TYPE_BF16) || ldx < c.K || ldx % (x8 ? 16 : 8)))
    return MOE_ERR_INVALID_ARG;
  if (x8 && dw && ldx != c.K) return MOE_ERR_INVALID_ARG;   // a checkpoint's codes are dense
  if (((x8 && dw) || (w8 && dx)) && !c.blocks8) return MOE_ERR_INVALID_ARG;
  const LinearLayout L = linear_layout(c);
  if (ws_bytes < L.bwd_total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (c.N == 0) {
    if (!dw) return MOE_OK;
    const cudaError_t e = cudaMemsetAsync(dw, 0, (size_t)c.E * c.O * c.K * type_size(dw_type), s);
    return e == cudaSuccess ? MOE_OK : record_cuda_error(e, "clear dW");
  }
  if (!ok16(dy) || (dx && (!ok16(w) || !ok16(dx))) || (dw && !ok16(x))) return MOE_ERR_INVALID_ARG;
  uint8_t* b = static_cast<uint8_t*>(ws);
  const int sms = device_sm_count();
  const int ob = (int)up(c.O, MOE_BLOCK8), kb = (int)up(c.K, MOE_BLOCK8);
  if (dx) {
    LinMaps m = {};
    const bool made = w8 ? make_map_2d_u8(&m.a, b + L.dy_codes, c.O, c.N, c.O, 128, 128) && make_map_2d_u8(&m.few, b + L.dy_codes, c.O, c.N, c.O, 128, kFewRows) && make_map_3d_u8(&m.b, w, c.K, c.O, c.E, 128, 128)
                         : make_map_2d(&m.a, dy, c.O, c.N, 64, 128) && make_map_2d(&m.few, dy, c.O, c.N, 64, kFewRows) && make_map_3d(&m.b, w, c.K, c.O, c.E, 64, 64);
    if (!made) return record_cuda_error(cudaErrorInvalidValue, "linear tensor maps");
    if (w8 && (v = timed_launch(MOE_K_BLOCKS8, "pack dy", s, [&] {
                 return launch_pack_rows(dy, c.O, MOE_TYPE_BF16, c.N, c.O, b + L.dy_codes, b + L.dy_scales, s);
               })) != MOE_OK)
      return v;
    LinGemm p = linear_params(c, L, offsets, b);
    p.cols = c.K;
    p.nk = (int)up(c.O, w8 ? 128 : 64);
    p.tiles_n = (int)up(c.K, 256);
    p.a_scale = b + L.dy_scales;
    p.lda_s = ob;
    p.b_scale = w_scales;
    p.b_col = 1;
    p.b_k = kb;
    p.b_expert = (int64_t)ob * kb;
    p.out = dx;
    if ((v = timed_launch(MOE_K_LINEAR_DX, "linear dx", s, [&] {
           return w8 ? launch_linear_gemm<LIN_DX, true>(m, p, sms, s) : launch_linear_gemm<LIN_DX, false>(m, p, sms, s);
         })) != MOE_OK)
      return v;
  }
  if (!dw) return MOE_OK;
  const void* xv = x8 ? b + L.x_values : x;
  LinDwMaps m = {};
  for (int i = 0; i < 7; ++i)
    if (!make_map_2d(&m.a[i], dy, c.O, c.N, 64, 64 >> i) || !make_map_2d_strided(&m.b[i], xv, c.K, c.N, ldx, 64, 64 >> i))
      return record_cuda_error(cudaErrorInvalidValue, "linear tensor maps");
  if (x8 && (v = timed_launch(MOE_K_BLOCKS8, "unpack x", s, [&] {
               return launch_unpack_rows(static_cast<const uint8_t*>(x), x_scales, c.N, c.K, b + L.x_values, MOE_TYPE_BF16, s);
             })) != MOE_OK)
    return v;
  LinGemm p = linear_params(c, L, offsets, b);
  p.cols = c.K;
  p.rows_out = c.O;
  p.tiles_n = (int)up(c.K, 256);
  p.tiles_m = (int)up(c.O, 256);
  p.out = dw;
  p.out32 = dw_type == MOE_TYPE_F32;
  return timed_launch(MOE_K_LINEAR_DW, "linear dW", s, [&] { return launch_linear_gemm<LIN_DW, false>(m, p, sms, s); });
}

}  // extern "C"
