// (c1) Per-head norm of queries and keys, position rotation, head split and
// cache append, in one pass over the projection's output.
//
//   y = x w / sqrt(mean(x^2) + eps)          (query and key heads)
//   (y_u, y_v) <- (y_u cos a - y_v sin a, y_v cos a + y_u sin a),  a = p f_j
//
// Bound: HBM (every row is read once and written once, 8 flops per value).
// A CTA takes one token and a run of its head rows.  D/8 threads hold a row,
// two vectors of four values each, placed so that a rotated pair is always in
// one thread: for the split pairing the vectors at 4c and rot/2 + 4c (values
// past rot_dim likewise, as two halves), for the interleaved one 8c and 8c+4.
// The row's mean square is a butterfly over its D/8 lanes.  Cosine and sine
// are taken once per token and shared by its heads: the angle in turns,
// p f / (2 pi), is reduced to [-1/2, 1/2] in fp64 (in fp32 the phase of far
// positions would be lost: at position 32768 an fp32 angle is off by 2e-3),
// then sincospi in fp32.
#include "common.cuh"
#include "internal.h"
#include "launch.cuh"

namespace dl {

namespace {

constexpr int kRopeThreads = 256;

template <typename T> struct Vec4;
template <> struct Vec4<float> {
  using Raw = float4;
  __device__ __forceinline__ static void unpack(const Raw& r, float* v) {
    v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w;
  }
  __device__ __forceinline__ static Raw pack(const float* v) {
    return make_float4(v[0], v[1], v[2], v[3]);
  }
};
template <> struct Vec4<__nv_bfloat16> {
  using Raw = uint2;
  __device__ __forceinline__ static void unpack(const Raw& r, float* v) {
    const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&r.x));
    const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&r.y));
    v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
  }
  __device__ __forceinline__ static Raw pack(const float* v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]);
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2], v[3]);
    Raw r;
    r.x = *reinterpret_cast<const uint32_t*>(&a);
    r.y = *reinterpret_cast<const uint32_t*>(&b);
    return r;
  }
};

template <typename T, int D>
__global__ void __launch_bounds__(kRopeThreads)
qk_norm_rope_kernel(RopeArgs a, int rows_per_cta) {
  using V = Vec4<T>;
  using Raw = typename V::Raw;
  constexpr int TPR = D / 8;                 // threads per row
  constexpr int RPP = kRopeThreads / TPR;    // rows per pass
  pdl_trigger();
  pdl_wait();
  __shared__ float s_cos[D / 2], s_sin[D / 2];
  const Shape& s = a.s;
  const int tok = blockIdx.x, b = tok / a.n_tok, i = tok - b * a.n_tok;
  const int tid = threadIdx.x, c = tid % TPR;
  const int half = a.rot_dim / 2;
  if (tid < half) {
    const double turns = (double)a.pos[tok] * (double)a.inv_freq[tid] * 0.15915494309189533577;
    sincospif(2.0f * (float)(turns - rint(turns)), &s_sin[tid], &s_cos[tid]);
  }
  // the token's place in the cache
  T* krow = nullptr;  // KV head 0's row in the pools; a head is 64 * D further
  T* vrow = nullptr;
  if (a.start) {
    const int st = a.start[b];
    const bool fits = st >= 0 && (long long)st + a.n_tok <= s.L_ctx;
    if (blockIdx.y == 0 && i == 0 && tid == 0) {
      if (!fits) flag_error(a.err, ERR_BAD_INDEX);
      if (a.end) a.end[b] = fits ? st + a.n_tok : st;
    }
    if (fits) {
      const int t = st + i;
      const int slot = a.page_table[(size_t)b * s.n_pages + t / 64];
      if (slot < 0 || slot >= s.n_slots) {
        if (blockIdx.y == 0 && tid == 0) flag_error(a.err, ERR_BAD_INDEX);
      } else {
        const size_t row = ((size_t)slot * s.H_kv * 64 + (t % 64)) * D;
        krow = reinterpret_cast<T*>(a.K_pool) + row;
        vrow = reinterpret_cast<T*>(a.V_pool) + row;
        if (blockIdx.y == 0) {
          for (int m = tid; m < a.n_mass; m += kRopeThreads) {
            const size_t e = ((size_t)b * a.n_mass + m) * s.L_ctx + t;
            if (a.tok_pos) a.tok_pos[e] = a.pos[tok];
            if (a.tok_mass) a.tok_mass[e] = 0.0f;
          }
        }
      }
    }
  }
  __syncthreads();

  // this thread's two vectors of four
  int off0, off1;
  bool rotated;
  if (a.interleaved) {
    off0 = 8 * c;
    off1 = off0 + 4;
    rotated = off0 < a.rot_dim;
  } else if (4 * c < half) {
    off0 = 4 * c;
    off1 = half + off0;
    rotated = true;
  } else {
    off0 = a.rot_dim + 4 * c - half;
    off1 = off0 + (D - a.rot_dim) / 2;
    rotated = false;
  }
  float cs[4], sn[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    cs[e] = rotated ? s_cos[4 * c + e] : 1.0f;
    sn[e] = rotated ? s_sin[4 * c + e] : 0.0f;
  }
  const int n_rows = s.H + 2 * s.H_kv;
  const int r0 = blockIdx.y * rows_per_cta, r1 = min(n_rows, r0 + rows_per_cta);
  const T* src = reinterpret_cast<const T*>(a.qkv) + (size_t)tok * a.qkv_stride;
#pragma unroll 2
  for (int rr = r0; rr < r1; rr += RPP) {  // uniform over the CTA: the butterfly needs every lane
    const int r = rr + tid / TPR;
    const bool live = r < r1;
    Raw raw0{}, raw1{};
    if (live) {
      raw0 = *reinterpret_cast<const Raw*>(src + (size_t)r * D + off0);
      raw1 = *reinterpret_cast<const Raw*>(src + (size_t)r * D + off1);
    }
    const bool is_q = r < s.H, is_v = r >= s.H + s.H_kv;
    const T* w = reinterpret_cast<const T*>(is_q ? a.q_weight : a.k_weight);
    float x[8];
    V::unpack(raw0, x);
    V::unpack(raw1, x + 4);
    float sq = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) sq = fmaf(x[e], x[e], sq);
#pragma unroll
    for (int o = TPR / 2; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
    if (live && !is_v) {
      if (w) {
        const float inv = __frsqrt_rn(sq * (1.0f / D) + a.eps);
        float g[8];
        V::unpack(*reinterpret_cast<const Raw*>(w + off0), g);
        V::unpack(*reinterpret_cast<const Raw*>(w + off1), g + 4);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * inv * g[e];
      }
      if (rotated) {
        if (a.interleaved) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float u = x[2 * e], v = x[2 * e + 1];
            x[2 * e] = u * cs[e] - v * sn[e];
            x[2 * e + 1] = v * cs[e] + u * sn[e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float u = x[e], v = x[4 + e];
            x[e] = u * cs[e] - v * sn[e];
            x[4 + e] = v * cs[e] + u * sn[e];
          }
        }
      }
      raw0 = V::pack(x);
      raw1 = V::pack(x + 4);
    }
    if (!live) continue;
    auto put = [&](T* row) {
      *reinterpret_cast<Raw*>(row + off0) = raw0;
      *reinterpret_cast<Raw*>(row + off1) = raw1;
    };
    if (is_q) {
      put(reinterpret_cast<T*>(a.Q_out) + (((size_t)b * s.H + r) * a.n_tok + i) * D);
    } else {
      const int g = is_v ? r - s.H - s.H_kv : r - s.H;
      T* out = reinterpret_cast<T*>(is_v ? a.V_out : a.K_out);
      if (out) put(out + (((size_t)b * s.H_kv + g) * a.n_tok + i) * D);
      T* row = is_v ? vrow : krow;
      if (row) put(row + (size_t)g * 64 * D);
    }
  }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeArgs& a, cudaStream_t st) {
  const Shape& s = a.s;
  const int n_rows = s.H + 2 * s.H_kv;
  dim3 grid(s.batch * a.n_tok, 1);
#define DL_ROPE(T, D_) DL_LAUNCH((qk_norm_rope_kernel<T, D_>), grid, kRopeThreads, 0, st, a, n_rows)
  if (s.dtype == DL_BF16) {
    if (s.d == 128) DL_ROPE(__nv_bfloat16, 128); else DL_ROPE(__nv_bfloat16, 64);
  } else {
    if (s.d == 128) DL_ROPE(float, 128); else DL_ROPE(float, 64);
  }
#undef DL_ROPE
  return cudaGetLastError();
}

}  // namespace dl
