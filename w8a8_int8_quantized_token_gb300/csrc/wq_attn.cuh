// Pieces shared by the attention kernels: the key ranges of a work item, the
// page lookup and the writes of a row's result.
#pragma once

#include <type_traits>

#include "wq_serve.cuh"

namespace wq {
namespace attn {

// The query tokens and keys of one source: the prefix (seq = -1), seen whole
// by every token of the call, or the suffix of one sequence.
struct Source {
  int t0, n;             // first query token, count
  int len;               // keys
  const int32_t *pages;  // its pages
  int slot0;             // first partial-result slot
  bool causal;
};

__device__ __forceinline__ Source source_of(const AttnArgs &a, int seq) {
  if (seq < 0) return {0, a.T, a.P, a.prefix_pages, 0, false};
  int t0, n;
  if (a.cu_q) {
    const int c0 = a.cu_q[seq], c1 = a.cu_q[seq + 1];
    t0 = min(max(c0, 0), a.T);
    n = min(max(c1 - t0, 0), min(a.max_q, a.T - t0));
    if (t0 != c0 || t0 + n != c1) set_status(a.status, WQ_ERR_INDEX);
  } else {
    n = a.T / a.B;
    t0 = seq * n;
  }
  const int l = a.max_suffix > 0 ? a.suffix_len[seq] : 0, len = min(max(l, 0), a.max_suffix);
  if (len != l) set_status(a.status, WQ_ERR_INDEX);
  return {t0, n, len, a.page_table + seq * a.ld_table, a.sp, true};
}

// Weights are taken 2^7 times their size in fp16 (at most 2^15 with 2^8 for a
// maximum that is behind), where they would be subnormal below 2^-14 and vanish
// below 2^-25: now below 2^-21 and 2^-32 of the largest.  The sums carry the
// same factor, the log-sum-exp takes it off.
template <class DT>
constexpr float kWeightUp = std::is_same<DT, F16>::value ? 7.0f : 0.0f;
template <class DT>
__device__ __forceinline__ float lse_of(float max, float scale_log2, float sum) {
  return sum == 0.0f ? -INFINITY : (max * scale_log2 + (log2f(sum) - kWeightUp<DT>)) * 0.6931471805599453f;
}

// Keys that query token j of the source sees
__device__ __forceinline__ int visible(const Source &s, int j) {
  return s.causal ? s.len - s.n + j + 1 : s.len;
}

// The kernels of one call follow each other closely: each lets the next one's
// blocks take the room that its own leave (start_next_kernel, in every block),
// and none ends before the one before it has (its last block waits in
// wait_last_kernel; were all to wait, those that are done would keep others
// from starting), so that the join may read what all of them wrote.  The first is launched in plain
// stream order, after everything that came before the call.
__device__ __forceinline__ void start_next_kernel() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_last_kernel() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <class... Args>
int launch_chained(void (*k)(Args...), unsigned grid, int threads, int smem, bool chained,
                   cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = chained ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, k, args...) != cudaSuccess) return WQ_ERR_LAUNCH;
  return launched(1);
}

}  // namespace attn
}  // namespace wq
