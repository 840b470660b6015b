// Code decisions of the q8_0 and q5_1 formats, shared by the appends.
#pragma once

#include <cuda_runtime.h>

namespace kvq {

// round-half-away-from-zero of an fp64 value, exact
__device__ __forceinline__ double rha64(double t) {
    double a = fabs(t);
    double f = floor(a);
    double n = f + ((a - f) >= 0.5 ? 1.0 : 0.0);
    return t < 0.0 ? -n : n;
}

__device__ __forceinline__ bool near_boundary(float a) {
    // a = |t| + 0.5 (or t + 0.5): a code boundary is an integer value of a
    float fr = a - floorf(a);
    return fr < 1e-3f || fr > 0.999f || fabsf(a) >= 4194304.0f;
}

// q8_0 code of x for stored scale d (d > 0), inv = 1/d
__device__ __forceinline__ int q8_code(float x, float d, float inv) {
    float t = x * inv;
    float a = fabsf(t) + 0.5f;
    if (near_boundary(a)) {
        double n = rha64((double)x / (double)d);
        n = fmin(fmax(n, -127.0), 127.0);
        return (int)n;
    }
    int n = min((int)floorf(a), 127);
    return t < 0.f ? -n : n;
}

// q5_1 code of x for stored min m and scale d (d > 0), inv = 1/d
__device__ __forceinline__ int q5_code(float x, float m, float d, float inv) {
    float t = (x - m) * inv;
    float a = t + 0.5f;
    if (near_boundary(a)) {
        double n = rha64(((double)x - (double)m) / (double)d);
        n = fmin(fmax(n, 0.0), 31.0);
        return (int)n;
    }
    float f = floorf(a);
    f = fminf(fmaxf(f, 0.f), 31.f);
    return (int)f;
}

}  // namespace kvq
