// ep_expert_api.cpp -- the experts' products' part of the C ABI (include/ep.h):
// argument checks, scratch sizes and launches, all on the host.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include "ep.h"
#include "ep_expert.h"

namespace {

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

uint64_t up256(uint64_t v) { return (v + 255) / 256 * 256; }

int wide(const ep_expert_config_t *c) {
    return c->activation == EP_ACTIVATION_SWIGLU ? 2 * c->out_features : c->out_features;
}

int check_config(const ep_expert_config_t *c) {
    if (!c) return EP_ERR_INVALID_ARG;
    if (c->num_experts < 1 || c->num_rows < 0 || c->in_features < 1 || c->out_features < 1 ||
        c->reserved != 0)
        return EP_ERR_INVALID_ARG;
    if (c->x_dtype != EP_DTYPE_BF16 && c->x_dtype != EP_DTYPE_FP8_E4M3FN) return EP_ERR_INVALID_ARG;
    if (c->activation < EP_ACTIVATION_NONE || c->activation > EP_ACTIVATION_SWIGLU) return EP_ERR_INVALID_ARG;
    if (c->num_experts > EP_MAX_EXPERTS || c->in_features > EP_MAX_HIDDEN || c->out_features > EP_MAX_HIDDEN ||
        c->num_rows > EP_MAX_EXPERT_ROWS)
        return EP_ERR_UNSUPPORTED;
    const int step = c->x_dtype == EP_DTYPE_FP8_E4M3FN ? 128 : 8;
    if (c->in_features % step || c->out_features % 8) return EP_ERR_UNSUPPORTED;
    return EP_OK;
}

uint64_t grad_bytes(const ep_expert_config_t *c) {
    if (c->activation == EP_ACTIVATION_NONE) return 0;
    return up256((uint64_t)c->num_rows * wide(c) * 2);
}

void set_shape(const ep_expert_config_t *c, ep::ExpertArgs *out) {
    ep::ExpertArgs &a = *out;
    memset(&a, 0, sizeof(a));
    a.E = c->num_experts;
    a.I = c->in_features;
    a.N = c->out_features;
    a.Nw = wide(c);
    a.act = c->activation;
    a.fp8 = c->x_dtype == EP_DTYPE_FP8_E4M3FN;
    a.rows = c->num_rows;
}

int make_args(const ep_expert_config_t *c, const int32_t *base, const void *x, const void *w, ep::ExpertArgs *out) {
    const int rc = check_config(c);
    if (rc != EP_OK) return rc;
    if (!base || !aligned(base, 4) || !w || !aligned(w, 16) || !aligned(x, 16)) return EP_ERR_INVALID_ARG;
    set_shape(c, out);
    out->base = base;
    out->x = x;
    out->w = w;
    return EP_OK;
}

}  // namespace

extern "C" {

int ep_query_expert_sizes(const ep_expert_config_t *cfg, ep_expert_sizes_t *sz) {
    const int rc = check_config(cfg);
    if (rc != EP_OK) return rc;
    if (!sz) return EP_ERR_INVALID_ARG;
    memset(sz, 0, sizeof(*sz));
    const uint64_t rows = cfg->num_rows, E = cfg->num_experts, Nw = wide(cfg), I = cfg->in_features;
    const bool fp8 = cfg->x_dtype == EP_DTYPE_FP8_E4M3FN;
    const uint64_t el = fp8 ? 1 : 2;
    sz->x = rows * I * el;
    sz->x_sf = fp8 ? rows * (I / 128) * 4 : 0;
    sz->w = E * Nw * I * el;
    sz->w_sf = fp8 ? E * ((Nw + 127) / 128) * (I / 128) * 4 : 0;
    sz->bias = E * Nw * 4;
    sz->out = rows * cfg->out_features * 2;
    sz->pre = rows * Nw * 2;
    if (!fp8) sz->backward_scratch = grad_bytes(cfg) + ep::expert_row_tiles(rows, (int)E, ep::kActRows) * Nw * 4;
    return EP_OK;
}

int ep_query_expert_tiles(const ep_expert_config_t *cfg, ep_expert_tiles_t *tiles) {
    const int rc = check_config(cfg);
    if (rc != EP_OK) return rc;
    if (!tiles) return EP_ERR_INVALID_ARG;
    memset(tiles, 0, sizeof(*tiles));
    if (cfg->num_rows == 0) return EP_OK;
    ep::ExpertArgs a;
    set_shape(cfg, &a);
    ep::expert_tiles(a, &tiles->forward, &tiles->d_x, &tiles->d_w);
    return EP_OK;
}

int ep_expert_mm(const ep_expert_config_t *cfg, const int32_t *expert_base_dev, const void *x_dev,
                 const float *x_sf_dev, const void *w_dev, const float *w_sf_dev, const float *bias_dev,
                 const void *residual_dev, void *out_dev, void *pre_dev, void *stream) {
    ep::ExpertArgs a;
    const int rc = make_args(cfg, expert_base_dev, x_dev, w_dev, &a);
    if (rc != EP_OK) return rc;
    if (a.rows == 0) return EP_OK;
    if (!x_dev || !out_dev || !aligned(out_dev, 16) || !aligned(bias_dev, 16) || !aligned(residual_dev, 16) ||
        !aligned(pre_dev, 16))
        return EP_ERR_INVALID_ARG;
    if (a.fp8 ? (!x_sf_dev || !w_sf_dev || !aligned(x_sf_dev, 4) || !aligned(w_sf_dev, 4)) : (x_sf_dev || w_sf_dev))
        return EP_ERR_INVALID_ARG;
    a.x_sf = x_sf_dev;
    a.w_sf = w_sf_dev;
    a.bias = bias_dev;
    a.residual = static_cast<const uint16_t *>(residual_dev);
    a.out = static_cast<uint16_t *>(out_dev);
    a.pre = static_cast<uint16_t *>(pre_dev);
    return ep::launch_expert(a, (hipStream_t)stream) == hipSuccess ? EP_OK : EP_ERR_HIP;
}

int ep_expert_mm_backward(const ep_expert_config_t *cfg, const int32_t *expert_base_dev, const void *x_dev,
                          const void *w_dev, const void *pre_dev, const void *d_out_dev, void *d_x_dev, void *d_w_dev,
                          float *d_bias_dev, void *scratch_dev, void *stream) {
    ep::ExpertArgs a;
    const int rc = make_args(cfg, expert_base_dev, x_dev, w_dev, &a);
    if (rc != EP_OK) return rc;
    if (a.fp8) return EP_ERR_UNSUPPORTED;
    // Without rows a caller's d_x is empty and may have no address.
    if ((a.rows > 0 && !d_x_dev && !d_w_dev && !d_bias_dev) || !aligned(d_x_dev, 16) || !aligned(d_w_dev, 16) ||
        !aligned(d_bias_dev, 4) || !aligned(pre_dev, 16) || !aligned(d_out_dev, 16) || !scratch_dev ||
        !aligned(scratch_dev, 16))
        return EP_ERR_INVALID_ARG;
    if (a.rows > 0 && (!d_out_dev || (d_w_dev && !x_dev) || (a.act != EP_ACTIVATION_NONE && !pre_dev)))
        return EP_ERR_INVALID_ARG;
    a.pre = static_cast<uint16_t *>(const_cast<void *>(pre_dev));
    a.d_out = static_cast<const uint16_t *>(d_out_dev);
    a.d = static_cast<uint16_t *>(scratch_dev);
    a.part = reinterpret_cast<float *>(static_cast<char *>(scratch_dev) + grad_bytes(cfg));
    a.part_tiles = ep::expert_row_tiles(a.rows, a.E, ep::kActRows);
    a.d_x = static_cast<uint16_t *>(d_x_dev);
    a.d_w = static_cast<uint16_t *>(d_w_dev);
    a.d_bias = d_bias_dev;
    return ep::launch_expert_backward(a, (hipStream_t)stream) == hipSuccess ? EP_OK : EP_ERR_HIP;
}

}  // extern "C"
