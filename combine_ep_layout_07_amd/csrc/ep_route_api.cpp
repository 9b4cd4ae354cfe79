// ep_route_api.cpp -- the router's part of the C ABI (include/ep.h): argument
// checks, scratch sizes and launches, all on the host.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "ep.h"
#include "ep_kernels.h"

namespace {

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

int check_config(const ep_route_config_t *c) {
    if (!c) return EP_ERR_INVALID_ARG;
    if (c->num_src_ranks < 1 || c->num_tokens < 0 || c->num_experts < 1 || c->num_topk < 1 ||
        c->num_topk > c->num_experts || !isfinite(c->scale))
        return EP_ERR_INVALID_ARG;
    if (c->logits_dtype != EP_DTYPE_FP32 && c->logits_dtype != EP_DTYPE_BF16) return EP_ERR_INVALID_ARG;
    if (c->scoring != EP_SCORING_SOFTMAX && c->scoring != EP_SCORING_SIGMOID) return EP_ERR_INVALID_ARG;
    if (c->num_experts > EP_MAX_EXPERTS || c->num_topk > EP_MAX_TOPK || c->num_src_ranks > 65535 ||
        c->num_tokens > EP_MAX_TOKENS)
        return EP_ERR_UNSUPPORTED;
    if ((int64_t)c->num_src_ranks * c->num_tokens > 2147483647ll / c->num_topk) return EP_ERR_UNSUPPORTED;
    return EP_OK;
}

uint64_t units(const ep_route_config_t *c) {
    return (uint64_t)c->num_src_ranks * ep::route_blocks(c->num_src_ranks, c->num_tokens, c->num_experts, c->num_topk);
}

int pitch(const ep_route_config_t *c) { return (c->num_experts + 3) / 4 * 4; }

// Bytes of the scratch before the partial sums: shares of the loss, counters.
uint64_t head_bytes(const ep_route_config_t *c) {
    const uint64_t S = c->num_src_ranks;
    return (S * ep::route_sum_blocks(c->num_experts) * 8 + S * 4 + 15) / 16 * 16;
}

// Shape and tables common to both directions.
int make_args(const ep_route_config_t *c, const void *logits_dev, const uint8_t *token_mask_dev,
              const ep_route_t *r, ep::RouteArgs *out) {
    const int rc = check_config(c);
    if (rc != EP_OK) return rc;
    if (!r) return EP_ERR_INVALID_ARG;
    const bool tok = c->num_tokens > 0;
    const uintptr_t el = c->logits_dtype == EP_DTYPE_BF16 ? 2 : 4;
    if (tok && (!logits_dev || !aligned(logits_dev, el) || !r->topk_idx_dev || !aligned(r->topk_idx_dev, 8)))
        return EP_ERR_INVALID_ARG;
    if (!aligned(r->topk_weights_dev, 4) || !aligned(r->tokens_per_expert_dev, 4) || !aligned(r->tokens_valid_dev, 4) ||
        !aligned(r->balance_loss_dev, 4) || !aligned(r->scratch_dev, 16))
        return EP_ERR_INVALID_ARG;
    ep::RouteArgs &a = *out;
    memset(&a, 0, sizeof(a));
    a.S = c->num_src_ranks;
    a.T = c->num_tokens;
    a.E = c->num_experts;
    a.K = c->num_topk;
    a.pitch = pitch(c);
    a.logits_bf16 = c->logits_dtype == EP_DTYPE_BF16;
    a.sigmoid = c->scoring == EP_SCORING_SIGMOID;
    a.scale = c->scale;
    a.logits = logits_dev;
    a.token_mask = token_mask_dev;
    a.topk_idx = r->topk_idx_dev;
    a.topk_weights = r->topk_weights_dev;
    a.tokens_per_expert = r->tokens_per_expert_dev;
    a.tokens_valid = r->tokens_valid_dev;
    a.balance_loss = r->balance_loss_dev;
    return EP_OK;
}

}  // namespace

extern "C" {

int ep_query_route_sizes(const ep_route_config_t *cfg, ep_route_sizes_t *sz) {
    const int rc = check_config(cfg);
    if (rc != EP_OK) return rc;
    if (!sz) return EP_ERR_INVALID_ARG;
    memset(sz, 0, sizeof(*sz));
    const uint64_t S = cfg->num_src_ranks, E = cfg->num_experts;
    const uint64_t lanes = S * (uint64_t)cfg->num_tokens * cfg->num_topk;
    sz->topk_idx = lanes * sizeof(int64_t);
    sz->topk_weights = lanes * sizeof(float);
    sz->tokens_per_expert = S * E * sizeof(int32_t);
    sz->tokens_valid = S * sizeof(int32_t);
    sz->balance_loss = S * sizeof(float);
    sz->scratch = head_bytes(cfg) + units(cfg) * (2 * pitch(cfg) + 1) * 4;
    return EP_OK;
}

int ep_route(const ep_route_config_t *cfg, const void *logits_dev, const float *bias_dev,
             const uint8_t *token_mask_dev, const ep_route_t *route, void *stream) {
    ep::RouteArgs a;
    const int rc = make_args(cfg, logits_dev, token_mask_dev, route, &a);
    if (rc != EP_OK) return rc;
    if (!aligned(bias_dev, 4) || (a.T > 0 && !a.topk_weights)) return EP_ERR_INVALID_ARG;
    const int given = !!a.tokens_per_expert + !!a.tokens_valid + !!a.balance_loss + !!route->scratch_dev;
    if (given != 0 && given != 4) return EP_ERR_INVALID_ARG;
    a.bias = bias_dev;
    if (given) {
        const uint64_t words = units(cfg) * (uint64_t)a.pitch;
        a.part_loss = static_cast<double *>(route->scratch_dev);
        a.part_done = reinterpret_cast<int32_t *>(a.part_loss + (uint64_t)a.S * ep::route_sum_blocks(a.E));
        a.part_p = reinterpret_cast<float *>(static_cast<char *>(route->scratch_dev) + head_bytes(cfg));
        a.part_cnt = reinterpret_cast<int32_t *>(a.part_p + words);
        a.part_seen = a.part_cnt + words;
    }
    return ep::launch_route(a, (hipStream_t)stream) == hipSuccess ? EP_OK : EP_ERR_HIP;
}

int ep_route_backward(const ep_route_config_t *cfg, const void *logits_dev, const uint8_t *token_mask_dev,
                      const ep_route_t *route, const float *d_topk_weights_dev, const float *d_balance_loss_dev,
                      void *d_logits_dev, void *stream) {
    ep::RouteArgs a;
    const int rc = make_args(cfg, logits_dev, token_mask_dev, route, &a);
    if (rc != EP_OK) return rc;
    if (a.T == 0) return EP_OK;
    const uintptr_t el = a.logits_bf16 ? 2 : 4;
    if (!d_logits_dev || !aligned(d_logits_dev, el) || (!d_topk_weights_dev && !d_balance_loss_dev) ||
        !aligned(d_topk_weights_dev, 4) || !aligned(d_balance_loss_dev, 4))
        return EP_ERR_INVALID_ARG;
    if (d_balance_loss_dev && (!a.tokens_per_expert || !a.tokens_valid)) return EP_ERR_INVALID_ARG;
    a.d_weights = d_topk_weights_dev;
    a.d_loss = d_balance_loss_dev;
    a.d_logits = d_logits_dev;
    return ep::launch_route_backward(a, (hipStream_t)stream) == hipSuccess ? EP_OK : EP_ERR_HIP;
}

}  // extern "C"
