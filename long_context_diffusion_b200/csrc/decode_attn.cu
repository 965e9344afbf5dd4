// (c2) Attention of one new token per sequence over its cached tokens.
//
//   a_t = scale q.k_t,  lse = ln sum_t e^{a_t},  o = sum_t e^{a_t - lse} v_t
//   mass_t <- decay mass_t + sum_h e^{a_t - lse_h}
//
// One CTA per (sequence, query head); its warps take the keys in turn, a lane
// holding D/32 columns, with the running maximum and sum of an online softmax
// per warp; the warps' states are joined in shared memory.  Logits go to the
// workspace when masses are kept, and a second kernel adds the weights.
#include "common.cuh"
#include "internal.h"
#include "launch.cuh"

namespace dl {

namespace {

constexpr int kDecWarps = 8;

struct DecodeWs {
  float* logit;  // [batch][H][Lp], natural units
  float* lse;    // [batch][H]
};
int padded_ctx(const Shape& s) { return (s.L_ctx + 63) / 64 * 64; }

DecodeWs decode_ws(void* ws, const Shape& s) {
  DecodeWs w;
  w.logit = reinterpret_cast<float*>(ws);
  w.lse = reinterpret_cast<float*>(reinterpret_cast<char*>(ws) +
                                   round256((size_t)s.batch * s.H * padded_ctx(s) * sizeof(float)));
  return w;
}

__device__ __forceinline__ int seq_len(const DecodeArgs& a, int b, bool report) {
  const int n = a.ctx_len[b];
  if (n >= 0 && n <= a.s.L_ctx) return n;
  if (report) flag_error(a.err, ERR_BAD_INDEX);
  return 0;
}

template <typename T, int D>
__global__ void __launch_bounds__(kDecWarps * 32)
decode_kernel(DecodeArgs a, float* logit, float* lse_ws, int Lp) {
  pdl_trigger();
  pdl_wait();
  constexpr int C = D / 32;
  __shared__ float s_o[kDecWarps][D], s_m[kDecWarps], s_l[kDecWarps];
  const Shape& s = a.s;
  const int h = blockIdx.x, b = blockIdx.y, g = h / s.G;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = seq_len(a, b, threadIdx.x == 0 && h == 0);
  const T* q = reinterpret_cast<const T*>(a.Q) + ((size_t)b * s.H + h) * D;
  float qv[C], o[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    qv[c] = to_f32(q[lane + 32 * c]) * (float)s.scale;
    o[c] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  for (int t = warp; t < n; t += kDecWarps) {
    const int slot = a.page_table[(size_t)b * s.n_pages + t / 64];
    if (slot < 0 || slot >= s.n_slots) {
      if (lane == 0) flag_error(a.err, ERR_BAD_INDEX);
      if (lane == 0 && logit) logit[((size_t)b * s.H + h) * Lp + t] = -INFINITY;
      continue;
    }
    const size_t row = (((size_t)slot * s.H_kv + g) * 64 + t % 64) * D;
    const T* k = reinterpret_cast<const T*>(a.Kp) + row;
    const T* v = reinterpret_cast<const T*>(a.Vp) + row;
    float x = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) x = fmaf(qv[c], to_f32(k[lane + 32 * c]), x);
    x = warp_sum(x);
    if (lane == 0 && logit) logit[((size_t)b * s.H + h) * Lp + t] = x;
    const float m2 = fmaxf(m, x);
    const float keep = m == -INFINITY ? 0.0f : expf(m - m2), p = expf(x - m2);
    l = l * keep + p;
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] = o[c] * keep + p * to_f32(v[lane + 32 * c]);
    m = m2;
  }
#pragma unroll
  for (int c = 0; c < C; ++c) s_o[warp][lane + 32 * c] = o[c];
  if (lane == 0) { s_m[warp] = m; s_l[warp] = l; }
  __syncthreads();
  if (threadIdx.x < D) {
    float M = -INFINITY, L = 0.0f, acc = 0.0f;
    for (int w = 0; w < kDecWarps; ++w) M = fmaxf(M, s_m[w]);
    for (int w = 0; w < kDecWarps; ++w) {
      if (s_m[w] == -INFINITY) continue;
      const float f = expf(s_m[w] - M);
      L += s_l[w] * f;
      acc += s_o[w][threadIdx.x] * f;
    }
    reinterpret_cast<T*>(a.O)[((size_t)b * s.H + h) * D + threadIdx.x] =
        from_f32<T>(L > 0.0f ? acc / L : 0.0f);
    if (threadIdx.x == 0) {
      const float lse = L > 0.0f ? M + logf(L) : -INFINITY;
      if (a.lse) a.lse[(size_t)b * s.H + h] = lse;
      lse_ws[(size_t)b * s.H + h] = lse;
    }
  }
}

__global__ void decode_mass_kernel(DecodeArgs a, const float* logit, const float* lse_ws, int Lp) {
  pdl_trigger();
  pdl_wait();
  const Shape& s = a.s;
  const int b = blockIdx.y / a.n_mass, m = blockIdx.y % a.n_mass;
  const int n = seq_len(a, b, false), rows = s.H / a.n_mass;
  for (int t = blockIdx.x * blockDim.x + threadIdx.x; t < n; t += gridDim.x * blockDim.x) {
    float sum = 0.0f;
    for (int r = 0; r < rows; ++r) {
      const size_t row = (size_t)b * s.H + m * rows + r;
      const float lse = lse_ws[row];
      if (lse != -INFINITY) sum += expf(logit[row * Lp + t] - lse);
    }
    float* dst = a.tok_mass + ((size_t)b * a.n_mass + m) * s.L_ctx + t;
    *dst = a.decay == 0.0f ? sum : fmaf(a.decay, *dst, sum);
  }
}

}  // namespace

size_t decode_workspace(const Shape& s) {
  return round256((size_t)s.batch * s.H * padded_ctx(s) * sizeof(float)) +
         round256((size_t)s.batch * s.H * sizeof(float));
}

cudaError_t launch_decode_attn(const DecodeArgs& a, cudaStream_t st) {
  const Shape& s = a.s;
  const DecodeWs w = decode_ws(a.ws, s);
  const int Lp = padded_ctx(s);
  float* logit = a.tok_mass ? w.logit : nullptr;
#define DL_DEC(T, D_) \
  DL_LAUNCH((decode_kernel<T, D_>), dim3(s.H, s.batch), kDecWarps * 32, 0, st, a, logit, w.lse, Lp)
  if (s.dtype == DL_BF16) {
    if (s.d == 128) DL_DEC(__nv_bfloat16, 128); else DL_DEC(__nv_bfloat16, 64);
  } else {
    if (s.d == 128) DL_DEC(float, 128); else DL_DEC(float, 64);
  }
#undef DL_DEC
  if (a.tok_mass && s.L_ctx > 0) {
    const int chunks = min((s.L_ctx + 255) / 256, 64);
    DL_LAUNCH(decode_mass_kernel, dim3(chunks, s.batch * a.n_mass), 256, 0, st, a, (const float*)logit,
              (const float*)w.lse, Lp);
  }
  return cudaGetLastError();
}

}  // namespace dl
