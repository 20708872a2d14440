// kda_ssm.cuh -- what the selective state space operator's kernels share:
// parameters, the runs of a row, the convolution at one token.  Internal.
#pragma once

#include "kda_internal.cuh"

namespace kda {

constexpr int kSsmTaps = 4;

// Where a row's sequences lie (written by ssm_rows_kernel): the first run is
// [first, first_end), the last token that counts is `last` (-1: none).  A
// run that starts later resets the state.
struct SsmRow {
  int first, first_end, last, pad;
};

struct SsmParams {
  int B, T, H, P, N, G, channels;
  const void *xbc, *z, *dt;
  long long xbc_sb, xbc_st, z_sb, z_st, dt_sb, dt_st;
  const float *w, *bias, *A, *D, *dt_bias;
  const float *initial_state;
  const void *conv_state;
  const int32_t *segment_ids;
  void *y, *conv_out;
  float *final_state;
  SsmRow *rows;           // [B] in the workspace
  unsigned char *ws;      // the tensor-core path's buffers
};

// Token t of a row: whether it counts, whether its run resets the state, and
// how many tokens of its run precede it (at most 3).
struct SsmToken {
  bool live, reset, first;
  int place;
};

__device__ __forceinline__ int ssm_id(const int32_t *ids, int t, int T) {
  if (t < 0 || t >= T) return 0;
  return ids ? ids[t] : 1;
}

__device__ __forceinline__ SsmToken ssm_token(const int32_t *ids, int t, int T,
                                              const SsmRow &row) {
  SsmToken k;
  const int id = ssm_id(ids, t, T);
  k.live = id != 0;
  k.first = t >= row.first && t < row.first_end;
  k.place = 0;
  if (k.live) {
#pragma unroll
    for (int i = 1; i < kSsmTaps; ++i)
      if (k.place == i - 1 && ssm_id(ids, t - i, T) == id) k.place = i;
  }
  k.reset = k.live && k.place == 0 && t > row.first;
  return k;
}

// The input `age` tokens before token t of channel c: in t's run, from the
// cache where that lies before the row's first run, else 0.
template <typename T>
__device__ __forceinline__ float ssm_tap(const T *x, long long st, const T *past, int channels,
                                         int c, int t, int age, const SsmToken &k) {
  if (age <= k.place) return to_f32(x[(long long)(t - age) * st + c]);
  if (k.first && past) return to_f32(past[(size_t)(kSsmTaps - 1 + k.place - age) * channels + c]);
  return 0.f;
}

// Entry i (oldest first) of the convolution's cache after a row that ends with
// token `last`, k its place; a row without a token keeps the cache it had.
template <typename T>
__device__ __forceinline__ T ssm_cached(const T *x, long long st, const T *past, int channels,
                                        int c, int i, int last, const SsmToken &k) {
  float v = past ? to_f32(past[(size_t)i * channels + c]) : 0.f;
  if (k.live) v = ssm_tap(x, st, past, channels, c, last, kSsmTaps - 2 - i, k);
  return from_f32<T>(v);
}

__device__ __forceinline__ float ssm_softplus(float x) {
  return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x)));
}

kda_status check_ssm_shape(const kda_ssm_shape *s);

// Tensor-core path (kda_ssm_tc.cu): its workspace after the row table,
// and its launches (with segment ids the row table must be there).
size_t ssm_tc_bytes(const SsmParams &p, bool f32);
cudaError_t launch_ssm_tc(const SsmParams &p, bool f32, uint32_t *status, cudaStream_t cs);

}  // namespace kda
