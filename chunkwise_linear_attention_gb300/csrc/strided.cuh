// strided.cuh -- element strides of the tensors that an entry point takes as
// views: a {batch, head, token} triple each, the last dimension dense.
#pragma once

#include "cla_internal.cuh"

namespace cla {
namespace {

struct Triple {
    long long b, h, t;
};

// The triples of a call's tensors, dense [B, heads, T, d] where `strides` is NULL.  heads[i], d[i]: of tensor i;
// step: what every stride has to be a multiple of (16-byte pieces need 8 or 4, single elements 1).
int view_strides(const char *fn, const int64_t *strides, const char *const *names, const int64_t *heads, const int64_t *d, int n,
                 int64_t B, int64_t T, int64_t step, Triple *out) {
    for (int i = 0; i < n; ++i) {
        if (strides == nullptr) {
            out[i] = Triple{heads[i] * T * d[i], T * d[i], d[i]};
            continue;
        }
        const int64_t *s = strides + 3 * i, size[3] = {B, heads[i], T};
        for (int j = 0; j < 3; ++j)
            if (size[j] > 1 && (s[j] <= 0 || s[j] % step != 0 || s[j] >= (int64_t)1 << 39))
                return fail(CLA_ERR_INVALID_ARG, "%s: stride %lld of %s: a positive multiple of %lld below 2^39 elements is needed", fn,
                            (long long)s[j], names[i], (long long)step);
        out[i] = Triple{B > 1 ? s[0] : 0, heads[i] > 1 ? s[1] : 0, T > 1 ? s[2] : 0};
    }
    return CLA_OK;
}

}  // namespace
}  // namespace cla
