// Host checks that the entry points of rotary positions, the 4-bit cache and
// packed rows share.  Each sets qa_last_error().
#pragma once

#include <cuda_runtime.h>
#include <math.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "qa.h"
#include "qa_internal.h"

#define QA_API extern "C" __attribute__((visibility("default")))

namespace qa {
namespace checks {

constexpr int kMaxAxes = 4;

inline qa_status reject(qa_status st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
inline qa_status reject(qa_status st, const char *fmt, ...) {
    char msg[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof msg, fmt, ap);
    va_end(ap);
    set_last_error(msg);
    return st;
}

inline qa_status invalid(const char *fn, const char *what) { return reject(QA_STATUS_INVALID_PARAMS, "%s: %s", fn, what); }

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline qa_status launched(cudaError_t e, const char *fn) {
    if (e != cudaSuccess) return reject(QA_STATUS_LAUNCH_FAILED, "%s: CUDA error %s", fn, cudaGetErrorString(e));
    return QA_STATUS_OK;
}

// A row stride: 0 (packed) or a multiple of 8 elements that holds the row.
inline qa_status check_stride(const char *fn, const char *name, long long ld, long long width) {
    if (ld != 0 && (ld < width || ld % 8 || ld > (1LL << 31)))
        return reject(QA_STATUS_INVALID_PARAMS, "%s: %s %lld must be 0 or a multiple of 8 of at least %lld", fn, name, ld,
                      width);
    return QA_STATUS_OK;
}

inline qa_status check_rope(const char *fn, const qa_rope *r, int head_dim, bool gains, bool positions) {
    if (!r) return invalid(fn, "rope is NULL");
    // below 1 a pair would turn by more than a radian a position, which sincos_turns's reduction is not exact for
    if (!(r->theta >= 1.f) || !isfinite(r->theta)) return invalid(fn, "rope theta must be finite and >= 1");
    if (!r->q_gain != !r->k_gain) return invalid(fn, "q_gain and k_gain must both be given or both be NULL");
    if (gains && !r->q_gain) return invalid(fn, "NULL gain");
    if (r->q_gain && (!(r->rms_eps > 0.f) || !isfinite(r->rms_eps))) return invalid(fn, "rms_eps must be finite and > 0");
    if (!aligned(r->q_gain, 16) || !aligned(r->k_gain, 16) || !aligned(r->positions, 4))
        return invalid(fn, "gains must be 16-byte aligned (positions 4-byte)");
    if (r->n_axes < 1 || r->n_axes > kMaxAxes)
        return reject(QA_STATUS_INVALID_PARAMS, "%s: n_axes %d outside [1, %d]", fn, r->n_axes, kMaxAxes);
    if (!r->positions && (positions || r->n_axes != 1)) return invalid(fn, "positions is NULL");
    if (r->pair_axis)
        for (int i = 0; i < head_dim / 2; ++i)
            if (r->pair_axis[i] >= r->n_axes)
                return reject(QA_STATUS_INVALID_PARAMS, "%s: pair_axis[%d] = %d outside [0, n_axes)", fn, i,
                              (int)r->pair_axis[i]);
    return QA_STATUS_OK;
}

}  // namespace checks
}  // namespace qa
