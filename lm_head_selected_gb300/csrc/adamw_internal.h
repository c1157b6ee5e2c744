// Internal declarations of the AdamW step's kernels (adamw.cu).
#pragma once

#include "llp_internal.h"

namespace llp {

constexpr int kAdamBlock = 256;   // values of an 8-bit state that share a scale
constexpr int kAdamChunk = 4096;         // elements that a CTA takes at a time, states in 32 bits
constexpr int kAdamPackedChunk = 16384;  // and in 8

// One tensor, as the kernel's parameters hold it.
struct AdamTensor {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  float* master;
  long long n;
  float decay;        // of the parameters
  int first_chunk;    // in the launch
  short head;         // elements before the first 16-byte boundary of all arrays; -1: there is none
  unsigned char param_dtype, grad_dtype;
};

struct AdamScalars {
  double beta1, beta2;  // for the corrections, where the step is on the device
  float b1, c1, b2, c2;  // beta and 1 - beta
  float eps, rate;
  float rate_m, root_v;  // rate / (1 - beta1^t) and 1 / sqrt(1 - beta2^t), of a step on the host
  long long step;
  const long long* device_step;
  const float* device_lr;
  const float* grad_scale;
};

constexpr int kAdamFew = 40, kAdamMany = 320;  // tensors of a launch: 3.3 KB or 25.7 KB of parameters

template <int MOST>
struct AdamTable {
  AdamScalars k;
  int count, chunks;
  AdamTensor t[MOST];
};
static_assert(sizeof(AdamTable<kAdamMany>) <= 32764, "what a kernel's parameters may take");

cudaError_t adamw_setup();
template <int MOST>
cudaError_t launch_adamw(const AdamTable<MOST>& table, int bits, int num_sms, cudaStream_t s);

}  // namespace llp
