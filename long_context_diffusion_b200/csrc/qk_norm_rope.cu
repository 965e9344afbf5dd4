// (c1) Per-head norm of queries and keys, position rotation, head split and
// cache append, in one pass over the projection's output.
//
//   y = x w / sqrt(mean(x^2) + eps)          (query and key heads)
//   (y_u, y_v) <- (y_u cos a - y_v sin a, y_v cos a + y_u sin a),  a = p f_j
//
// Bound: HBM (every row is read once and written once, 8 flops per value; a
// prompt of 8192 tokens with 96 head rows moves 405 MB).  A CTA takes TT
// neighbouring tokens of a sequence and a run of their head rows, so that it
// reads whole stretches of the projection and writes TT rows of a head side by
// side.  D/8 threads hold a row, two vectors of four values each, placed so
// that a rotated pair is always in one thread: for the split pairing the
// vectors at 4c and rot/2 + 4c (values past rot_dim likewise, as two halves),
// for the interleaved one 8c and 8c+4.  The row's mean square is a butterfly
// over its D/8 lanes.  U rows a thread are loaded ahead; the first are under
// way while the rotation is computed.
// Cosine and sine are taken once per token and shared by its rows of the CTA:
// the angle in turns, p f / (2 pi), is reduced to [-1/2, 1/2] in fp64 (in fp32
// the phase of far positions would be lost: at position 32768 an fp32 angle
// is off by 2e-3), then sincospi in fp32.
#include "common.cuh"
#include "internal.h"
#include "launch.cuh"
#include "tc_common.cuh"

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

template <typename T, int D, int TT, int U>
__global__ void __launch_bounds__(kRopeThreads)
qk_norm_rope_kernel(const __grid_constant__ RopeArgs a, int tiles, int rows_per_cta) {
  using V = Vec4<T>;
  using Raw = typename V::Raw;
  constexpr int TPR = D / 8;                 // threads per row
  constexpr int RPP = kRopeThreads / TPR;    // rows per pass
  __shared__ float4 s_cos[TT][D / 8], s_sin[TT][D / 8];
  __shared__ long long s_row[TT];            // the token's row of KV head 0 in the pools, or -1
  const Shape& s = a.s;
  const int tid = threadIdx.x, c = tid % TPR, grp = tid / TPR;
  const int b = blockIdx.x / tiles, i0 = (blockIdx.x - b * tiles) * TT;
  const int n_tok = min(TT, a.n_tok - i0), half = a.rot_dim / 2;
  const size_t tok0 = (size_t)b * a.n_tok + i0;

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
  const int n_rows = s.H + 2 * s.H_kv;
  const int r0 = blockIdx.y * rows_per_cta, r1 = min(n_rows, r0 + rows_per_cta);
  const int items = (r1 - r0) * TT;          // (row, token), tokens side by side
  const T* src = reinterpret_cast<const T*>(a.qkv) + tok0 * a.qkv_stride + (size_t)r0 * D;
  pdl_trigger();
  pdl_wait();
#pragma unroll 1
  for (int it0 = 0; it0 < items; it0 += U * RPP) {  // uniform over the CTA: the butterfly needs every lane
    Raw raw0[U], raw1[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int it = it0 + u * RPP + grp, t = it % TT;
      const bool live = it < items && t < n_tok;
      const T* x = src + (live ? (size_t)t * a.qkv_stride + (size_t)(it / TT) * D : 0);
      raw0[u] = *reinterpret_cast<const Raw*>(x + off0);
      raw1[u] = *reinterpret_cast<const Raw*>(x + off1);
    }
    if (it0 == 0) {
      for (int e = tid; e < n_tok * half; e += kRopeThreads) {
        const int t = e / half, j = e - t * half;
        const double turns = (double)a.pos[tok0 + t] * (double)a.inv_freq[j] * 0.15915494309189533577;
        sincospif(2.0f * (float)(turns - rint(turns)), reinterpret_cast<float*>(s_sin[t]) + j,
                  reinterpret_cast<float*>(s_cos[t]) + j);
      }
      if (tid < n_tok) {                     // the token's place in the cache
        long long row = -1;
        if (a.start) {
          const int st = a.start[b];
          const bool fits = st >= 0 && (long long)st + a.n_tok <= s.L_ctx;
          if (blockIdx.y == 0 && i0 == 0 && tid == 0) {
            if (!fits) flag_error(a.err, ERR_BAD_INDEX);
            if (a.end) a.end[b] = fits ? st + a.n_tok : st;
          }
          if (fits) {
            const int t = st + i0 + tid;
            const int slot = a.page_table[(size_t)b * s.n_pages + t / 64];
            if (slot < 0 || slot >= s.n_slots) {
              if (blockIdx.y == 0) flag_error(a.err, ERR_BAD_INDEX);
            } else {
              row = (long long)slot * s.H_kv * 64 + (t % 64);
              if (blockIdx.y == 0) {
                for (int m = 0; m < a.n_mass; ++m) {
                  const size_t e = ((size_t)b * a.n_mass + m) * s.L_ctx + t;
                  if (a.tok_pos) a.tok_pos[e] = a.pos[tok0 + tid];
                  if (a.tok_mass) a.tok_mass[e] = 0.0f;
                }
              }
            }
          }
        }
        s_row[tid] = row;
      }
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int it = it0 + u * RPP + grp, t = it % TT, r = r0 + it / TT;
      const bool live = it < items && t < n_tok;
      const bool is_q = r < s.H, is_v = r >= s.H + s.H_kv;
      float x[8];
      V::unpack(raw0[u], x);
      V::unpack(raw1[u], x + 4);
      const T* w = reinterpret_cast<const T*>(is_q ? a.q_weight : a.k_weight);
      float sq = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sq = fmaf(x[e], x[e], sq);
#pragma unroll
      for (int o = TPR / 2; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
      if (!live) continue;
      if (!is_v) {
        if (w) {
          const float inv = __frsqrt_rn(sq * (1.0f / D) + a.eps);
          float g[8];
          V::unpack(*reinterpret_cast<const Raw*>(w + off0), g);
          V::unpack(*reinterpret_cast<const Raw*>(w + off1), g + 4);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = x[e] * inv * g[e];
        }
        if (rotated) {
          const float4 c4 = s_cos[t][c], s4 = s_sin[t][c];
          const float cs[4] = {c4.x, c4.y, c4.z, c4.w}, sn[4] = {s4.x, s4.y, s4.z, s4.w};
          if (a.interleaved) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float p = x[2 * e], q = x[2 * e + 1];
              x[2 * e] = p * cs[e] - q * sn[e];
              x[2 * e + 1] = q * cs[e] + p * sn[e];
            }
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float p = x[e], q = x[4 + e];
              x[e] = p * cs[e] - q * sn[e];
              x[4 + e] = q * cs[e] + p * sn[e];
            }
          }
        }
        raw0[u] = V::pack(x);
        raw1[u] = V::pack(x + 4);
      }
      auto put = [&](T* row) {
        *reinterpret_cast<Raw*>(row + off0) = raw0[u];
        *reinterpret_cast<Raw*>(row + off1) = raw1[u];
      };
      if (is_q) {
        put(reinterpret_cast<T*>(a.Q_out) + (((size_t)b * s.H + r) * a.n_tok + i0 + t) * D);
      } else {
        const int g = is_v ? r - s.H - s.H_kv : r - s.H;
        T* out = reinterpret_cast<T*>(is_v ? a.V_out : a.K_out);
        if (out) put(out + (((size_t)b * s.H_kv + g) * a.n_tok + i0 + t) * D);
        const long long row = s_row[t];
        if (row >= 0) put(reinterpret_cast<T*>(is_v ? a.V_pool : a.K_pool) + (row + (long long)g * 64) * D);
      }
    }
  }
}

template <typename T, int D>
cudaError_t run_rope(const RopeArgs& a, cudaStream_t st) {
  const Shape& s = a.s;
  constexpr int RPP = kRopeThreads / (D / 8);
  const int n_rows = s.H + 2 * s.H_kv;
  // Eight tokens a CTA when a sequence has them.  Rows are split over CTAs down
  // to one pass each while that is needed to fill the GPU six CTAs deep.
  const int tt = a.n_tok >= 8 ? 8 : 1;
  const int tiles = (a.n_tok + tt - 1) / tt;
  const long long all = (long long)s.batch * tiles, want = 6ll * tc_sm_count();
  const int most = (n_rows * tt + RPP - 1) / RPP;
  long long split = all < want ? (want + all - 1) / all : 1;
  split = split < most ? split : most;
  const int per = (n_rows + (int)split - 1) / (int)split;
  const dim3 grid((unsigned)all, (n_rows + per - 1) / per);
  if (tt == 1) {
    DL_LAUNCH((qk_norm_rope_kernel<T, D, 1, 1>), grid, kRopeThreads, 0, st, a, tiles, per);
  } else if (per * tt <= RPP) {
    DL_LAUNCH((qk_norm_rope_kernel<T, D, 8, 1>), grid, kRopeThreads, 0, st, a, tiles, per);
  } else {
    DL_LAUNCH((qk_norm_rope_kernel<T, D, 8, 4>), grid, kRopeThreads, 0, st, a, tiles, per);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeArgs& a, cudaStream_t st) {
  if (a.s.dtype == DL_BF16)
    return a.s.d == 128 ? run_rope<__nv_bfloat16, 128>(a, st) : run_rope<__nv_bfloat16, 64>(a, st);
  return a.s.d == 128 ? run_rope<float, 128>(a, st) : run_rope<float, 64>(a, st);
}

}  // namespace dl
