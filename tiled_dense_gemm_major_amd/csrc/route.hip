// libtgemm: routing of tokens to experts, its plan and the combination of the experts'
// rows (C ABI): argument checks and launches.  Declarations and conventions are in
// include/tgemm.h.
#include "tgemm.h"

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "route.hpp"

namespace {

using tgemm::u16;

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t span(int64_t rows, int64_t cols, int64_t ld) {
    return rows > 0 && cols > 0 ? (rows - 1) * ld + cols : 0;
}
bool al16(const void* p) { return (uintptr_t)p % 16 == 0; }
bool overlaps(const void* p, int64_t pb, const void* q, int64_t qb) {
    const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
    return p && q && pb > 0 && qb > 0 && a < b + (uintptr_t)qb && b < a + (uintptr_t)pb;
}
int status(hipError_t e) { return e == hipSuccess ? TGEMM_OK : TGEMM_ERR_LAUNCH; }

int logit_bytes(int dtype) { return dtype == TGEMM_F32 ? 4 : 2; }

// The checks that the routing and its backward pass share.
int check_route(int dtype, int64_t tokens, int64_t experts, int64_t k, int64_t ldx, int scoring, int renormalize,
                float scale) {
    if (dtype != TGEMM_F16 && dtype != TGEMM_BF16 && dtype != TGEMM_F32)
        return TGEMM_ERR_INVALID_VALUE;
    if (tokens < 0 || experts < 1 || k < 1 || k > experts || ldx < experts)
        return TGEMM_ERR_INVALID_VALUE;
    if ((scoring != TGEMM_SCORE_SOFTMAX && scoring != TGEMM_SCORE_SIGMOID) ||
        (renormalize != 0 && renormalize != 1) || !isfinite(scale))
        return TGEMM_ERR_INVALID_VALUE;
    if (tokens > kMaxDim || experts > tgemm::kMaxExperts || k > tgemm::kMaxChoices || ldx > kMaxDim ||
        tokens * k > kMaxDim)
        return TGEMM_ERR_UNSUPPORTED;
    return TGEMM_OK;
}

}  // namespace

extern "C" {

int moe_route(int logits_dtype, int64_t tokens, int64_t experts, int64_t k, const void* logits, int64_t ldx,
              const float* bias, int scoring, int64_t groups, int64_t topk_groups, int group_score,
              int renormalize, float scale, int32_t* ids, float* weights, void* stream) {
    int rc = check_route(logits_dtype, tokens, experts, k, ldx, scoring, renormalize, scale);
    if (rc != TGEMM_OK)
        return rc;
    if (groups < 1 || groups > experts || experts % groups != 0 || topk_groups < 1 || topk_groups > groups ||
        (group_score != TGEMM_GROUP_MAX && group_score != TGEMM_GROUP_TOP2))
        return TGEMM_ERR_INVALID_VALUE;
    if (groups > tgemm::kMaxExpertGroups)
        return TGEMM_ERR_UNSUPPORTED;
    if (tokens == 0)
        return TGEMM_OK;
    if (!logits || !ids || !weights)
        return TGEMM_ERR_NULL_POINTER;
    const int size = logit_bytes(logits_dtype);
    if ((uintptr_t)logits % size || (uintptr_t)bias % 4 || (uintptr_t)ids % 4 || (uintptr_t)weights % 4)
        return TGEMM_ERR_ALIGNMENT;
    const int64_t xb = size * span(tokens, experts, ldx), ob = 4 * tokens * k;
    if (overlaps(ids, ob, logits, xb) || overlaps(weights, ob, logits, xb) || overlaps(ids, ob, weights, ob) ||
        overlaps(ids, ob, bias, 4 * experts) || overlaps(weights, ob, bias, 4 * experts))
        return TGEMM_ERR_ALIASING;
    const tgemm::RouteArgs p{logits,       bias,        ids,         weights,
                             ldx,          (int)tokens, (int)experts, (int)k,
                             scoring,      (int)groups, (int)topk_groups, group_score,
                             renormalize,  scale};
    // all groups kept: no choice among them
    const bool scored = bias || (groups > 1 && topk_groups < groups);
    const dim3 grid((unsigned)cdiv(tokens, 4));
    const hipStream_t s = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();
#define ROUTE_V(DT, V)                                                                     \
    if (scored)                                                                            \
        hipLaunchKernelGGL((tgemm::route_tokens<DT, V, true>), grid, dim3(256), 0, s, p);  \
    else                                                                                   \
        hipLaunchKernelGGL((tgemm::route_tokens<DT, V, false>), grid, dim3(256), 0, s, p)
#define ROUTE(DT)                                                                          \
    if (experts <= 64) {                                                                   \
        ROUTE_V(DT, 1);                                                                    \
    } else if (experts <= 128) {                                                           \
        ROUTE_V(DT, 2);                                                                    \
    } else if (experts <= 256) {                                                           \
        ROUTE_V(DT, 4);                                                                    \
    } else if (experts <= 512) {                                                           \
        ROUTE_V(DT, 8);                                                                    \
    } else {                                                                               \
        ROUTE_V(DT, 16);                                                                   \
    }
    if (logits_dtype == TGEMM_F16) {
        ROUTE(0)
    } else if (logits_dtype == TGEMM_BF16) {
        ROUTE(1)
    } else {
        ROUTE(2)
    }
#undef ROUTE
#undef ROUTE_V
    return status(hipGetLastError());
}

int moe_route_backward(int logits_dtype, int64_t tokens, int64_t experts, int64_t k, const void* logits,
                       int64_t ldx, const int32_t* ids, const float* dweights, int scoring, int renormalize,
                       float scale, void* dlogits, int64_t lddx, void* stream) {
    int rc = check_route(logits_dtype, tokens, experts, k, ldx, scoring, renormalize, scale);
    if (rc != TGEMM_OK)
        return rc;
    if (lddx < experts)
        return TGEMM_ERR_INVALID_VALUE;
    if (lddx > kMaxDim)
        return TGEMM_ERR_UNSUPPORTED;
    if (tokens == 0)
        return TGEMM_OK;
    if (!logits || !ids || !dweights || !dlogits)
        return TGEMM_ERR_NULL_POINTER;
    const int size = logit_bytes(logits_dtype);
    if ((uintptr_t)logits % size || (uintptr_t)dlogits % size || (uintptr_t)ids % 4 || (uintptr_t)dweights % 4)
        return TGEMM_ERR_ALIGNMENT;
    const int64_t db = size * span(tokens, experts, lddx), ib = 4 * tokens * k;
    if (overlaps(dlogits, db, logits, size * span(tokens, experts, ldx)) || overlaps(dlogits, db, ids, ib) ||
        overlaps(dlogits, db, dweights, ib))
        return TGEMM_ERR_ALIASING;
    const tgemm::RouteGradArgs p{logits, ids,         dweights,     dlogits, ldx,     lddx,
                                 (int)tokens, (int)experts, (int)k, scoring, renormalize, scale};
    const dim3 grid((unsigned)cdiv(tokens, 4));
    const hipStream_t s = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();
#define GRAD_V(DT, V) hipLaunchKernelGGL((tgemm::route_grad<DT, V>), grid, dim3(256), 0, s, p)
#define GRAD(DT)                                                                           \
    if (experts <= 64)                                                                     \
        GRAD_V(DT, 1);                                                                     \
    else if (experts <= 128)                                                               \
        GRAD_V(DT, 2);                                                                     \
    else if (experts <= 256)                                                               \
        GRAD_V(DT, 4);                                                                     \
    else if (experts <= 512)                                                               \
        GRAD_V(DT, 8);                                                                     \
    else                                                                                   \
        GRAD_V(DT, 16);
    if (logits_dtype == TGEMM_F16) {
        GRAD(0)
    } else if (logits_dtype == TGEMM_BF16) {
        GRAD(1)
    } else {
        GRAD(2)
    }
#undef GRAD
#undef GRAD_V
    return status(hipGetLastError());
}

int moe_plan_workspace_size(int64_t choices, int64_t experts, int64_t* bytes) {
    if (!bytes)
        return TGEMM_ERR_NULL_POINTER;
    if (choices < 0 || experts < 1)
        return TGEMM_ERR_INVALID_VALUE;
    if (choices > kMaxDim || experts > tgemm::kMaxExperts)
        return TGEMM_ERR_UNSUPPORTED;
    const int64_t chunks = cdiv(choices, tgemm::kPlanChunk);
    *bytes = chunks > 1 ? 4 * chunks * experts : 0;
    return TGEMM_OK;
}

int moe_plan(int64_t choices, int64_t experts, const int32_t* ids, int32_t* offsets, int32_t* order,
             int32_t* slots, void* workspace, int64_t workspace_bytes, void* stream) {
    int64_t need = 0;
    const int rc = moe_plan_workspace_size(choices, experts, &need);
    if (rc != TGEMM_OK)
        return rc;
    if (workspace_bytes < 0)
        return TGEMM_ERR_INVALID_VALUE;
    if (!offsets || (choices > 0 && (!ids || !order || !slots)))
        return TGEMM_ERR_NULL_POINTER;
    if (need > 0 && (!workspace || workspace_bytes < need))
        return TGEMM_ERR_WORKSPACE;
    if (((uintptr_t)ids | (uintptr_t)offsets | (uintptr_t)order | (uintptr_t)slots |
         (uintptr_t)(need > 0 ? workspace : nullptr)) % 4)
        return TGEMM_ERR_ALIGNMENT;
    const void* t[] = {ids, offsets, order, slots, need > 0 ? workspace : nullptr};
    const int64_t b[] = {4 * choices, 4 * (experts + 1), 4 * choices, 4 * choices, need};
    for (int i = 1; i < 5; ++i)
        for (int j = 0; j < i; ++j)
            if (overlaps(t[i], b[i], t[j], b[j]))
                return TGEMM_ERR_ALIASING;
    const int64_t chunks = choices > 0 ? cdiv(choices, tgemm::kPlanChunk) : 1;
    const tgemm::PlanArgs p{ids, offsets, order, slots, static_cast<int32_t*>(workspace), choices,
                            (int)experts, (int)chunks};
    const hipStream_t s = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    if (chunks > 1) {
        hipLaunchKernelGGL(tgemm::plan_count, dim3((unsigned)chunks), dim3(1024), 0, s, p);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return status(e);
    }
    const dim3 grid((unsigned)chunks), block(tgemm::kPlanWaves * 64);
    if (experts <= 64)
        hipLaunchKernelGGL((tgemm::plan_place<64>), grid, block, 0, s, p);
    else if (experts <= 256)
        hipLaunchKernelGGL((tgemm::plan_place<256>), grid, block, 0, s, p);
    else
        hipLaunchKernelGGL((tgemm::plan_place<tgemm::kMaxExperts>), grid, block, 0, s, p);
    return status(hipGetLastError());
}

int moe_combine(int dtype, int64_t tokens, int64_t k, int64_t width, const void* O, int64_t rows, int64_t ldo,
                const int32_t* slots, const float* weights, const void* residual, int64_t ldr, void* Y,
                int64_t ldy, void* stream) {
    if (dtype != TGEMM_F16 && dtype != TGEMM_BF16)
        return TGEMM_ERR_INVALID_VALUE;
    if (tokens < 0 || k < 1 || width < 0 || rows < 0 || ldo < 1 || ldo < width || ldy < 1 || ldy < width ||
        (residual && (ldr < 1 || ldr < width)))
        return TGEMM_ERR_INVALID_VALUE;
    if (tokens > kMaxDim || k > kMaxDim || width > kMaxDim - 8 || rows > kMaxDim || ldo > kMaxDim ||
        ldy > kMaxDim || (residual && ldr > kMaxDim) || (tokens > 0 && k > kMaxDim / tokens))
        return TGEMM_ERR_UNSUPPORTED;
    if (tokens == 0 || width == 0)
        return TGEMM_OK;
    if (!slots || !Y || (rows > 0 && !O))
        return TGEMM_ERR_NULL_POINTER;
    if (((uintptr_t)O | (uintptr_t)residual | (uintptr_t)Y) & 1 || (uintptr_t)slots % 4 || (uintptr_t)weights % 4)
        return TGEMM_ERR_ALIGNMENT;
    const int64_t yb = 2 * span(tokens, width, ldy);
    const bool in_place = residual == Y && ldr == ldy;
    if (overlaps(Y, yb, O, 2 * span(rows, width, ldo)) || overlaps(Y, yb, slots, 4 * tokens * k) ||
        overlaps(Y, yb, weights, 4 * tokens * k) ||
        (!in_place && overlaps(Y, yb, residual, 2 * span(tokens, width, ldr))))
        return TGEMM_ERR_ALIASING;
    const int64_t grid = cdiv(tokens * cdiv(width, 8), 256);
    if (grid > kMaxDim)
        return TGEMM_ERR_UNSUPPORTED;
    const int vec = al16(O) && al16(Y) && ldo % 8 == 0 && ldy % 8 == 0 &&
                    (!residual || (al16(residual) && ldr % 8 == 0));
    const tgemm::CombineArgs p{static_cast<const u16*>(O), slots, weights, static_cast<const u16*>(residual),
                               static_cast<u16*>(Y), (int)tokens, (int)k, (int)width, (int)rows, (int)ldo,
                               (int)ldr, (int)ldy, vec};
    const hipStream_t s = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    if (dtype == TGEMM_F16)
        hipLaunchKernelGGL((tgemm::combine_rows<0>), dim3((unsigned)grid), dim3(256), 0, s, p);
    else
        hipLaunchKernelGGL((tgemm::combine_rows<1>), dim3((unsigned)grid), dim3(256), 0, s, p);
    return status(hipGetLastError());
}

int moe_combine_backward(int dtype, int64_t tokens, int64_t k, int64_t width, const void* dY, int64_t lddy,
                         const void* O, int64_t rows, int64_t ldo, const int32_t* slots, const float* weights,
                         void* dO, int64_t lddo, float* dweights, void* stream) {
    if (dtype != TGEMM_F16 && dtype != TGEMM_BF16)
        return TGEMM_ERR_INVALID_VALUE;
    if (tokens < 0 || k < 1 || width < 0 || rows < 0 || lddy < 1 || lddy < width ||
        (dweights && (ldo < 1 || ldo < width)) || (dO && (lddo < 1 || lddo < width)))
        return TGEMM_ERR_INVALID_VALUE;
    if (tokens > kMaxDim || k > kMaxDim || width > kMaxDim - 512 || rows > kMaxDim || lddy > kMaxDim ||
        (dweights && ldo > kMaxDim) || (dO && lddo > kMaxDim) || (tokens > 0 && k > kMaxDim / tokens))
        return TGEMM_ERR_UNSUPPORTED;
    if (tokens == 0 || (!dO && !dweights))
        return TGEMM_OK;
    if (!slots || (width > 0 && (!dY || (dweights && rows > 0 && !O))))
        return TGEMM_ERR_NULL_POINTER;
    if (((uintptr_t)dY | (uintptr_t)O | (uintptr_t)dO) & 1 || (uintptr_t)slots % 4 || (uintptr_t)weights % 4 ||
        (uintptr_t)dweights % 4)
        return TGEMM_ERR_ALIGNMENT;
    const int64_t choices = tokens * k;
    const void* in[] = {dY, dweights ? O : nullptr, slots, weights};
    const int64_t ib[] = {2 * span(tokens, width, lddy), 2 * span(rows, width, ldo), 4 * choices, 4 * choices};
    const int64_t ob = 2 * span(rows, width, lddo);
    for (int i = 0; i < 4; ++i)
        if (overlaps(dO, ob, in[i], ib[i]) || overlaps(dweights, 4 * choices, in[i], ib[i]))
            return TGEMM_ERR_ALIASING;
    if (overlaps(dO, ob, dweights, 4 * choices))
        return TGEMM_ERR_ALIASING;
    const int vec = al16(dY) && lddy % 8 == 0 && (!dweights || (al16(O) && ldo % 8 == 0)) &&
                    (!dO || (al16(dO) && lddo % 8 == 0));
    const tgemm::CombineGradArgs p{static_cast<const u16*>(dY), static_cast<const u16*>(O), slots, weights,
                                   static_cast<u16*>(dO), dweights, choices, (int)k, (int)width, (int)rows,
                                   (int)lddy, (int)ldo, (int)lddo, vec};
    const dim3 grid((unsigned)cdiv(choices, 4));
    const hipStream_t s = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    if (dtype == TGEMM_F16)
        hipLaunchKernelGGL((tgemm::combine_grad<0>), grid, dim3(256), 0, s, p);
    else
        hipLaunchKernelGGL((tgemm::combine_grad<1>), grid, dim3(256), 0, s, p);
    return status(hipGetLastError());
}

}  // extern "C"
