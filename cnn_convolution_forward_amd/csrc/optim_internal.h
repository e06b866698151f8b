// optim_internal.h -- the optimiser's table entries, shared by its entry
// points and its kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace convfwd {

struct AdamwHyper {
    float b1, ob1, b2, ob2;         // beta1, 1 - beta1, beta2, 1 - beta2
    float lr_c1, inv_sqrt_c2, eps;  // lr / (1 - beta1^step), 1 / sqrt(1 - beta2^step)
    float pad;
    const float *grad_scale;        // device scalar or NULL
};

struct AdamwTensor {
    float *p;
    const void *g;
    void *m, *v;
    float *m_scale, *v_scale;
    uint16_t *copy;
    int64_t n;                      // >= 1
    float keep;                     // 1 - lr * weight_decay
    uint32_t key;                   // of the random bits
    uint32_t first;                 // first block of this tensor in its launch
    uint32_t pad;
};

constexpr int kMaxTensors = 50;     // tensors per launch: their table fits the kernel's 4 KB of arguments

enum { kAdamw32 = 0, kAdamw8 = 1, kAdamwValues = 2 };

// Steps (or decodes) tensors t[0..count) with as many launches as they need.
// A launch counts its blocks in 32 bits: n < 2^31 per tensor, 50 tensors.
hipError_t launch_adamw(const AdamwHyper &h, const AdamwTensor *t, int count, int mode, bool grad_bf16, hipStream_t st);

}  // namespace convfwd
