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
#include "sm100.cuh"
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

// Row of KV head 0 of token i of sequence b in the pools, or -1 (no cache, or
// the token is not appended).  The CTA that reports also writes the token's
// bookkeeping and, for the first token, the sequence's new end.
__device__ __forceinline__ long long cache_row(const RopeArgs& a, int b, int i, bool report) {
  if (!a.start) return -1;
  const Shape& s = a.s;
  const int st = a.start[b];
  const bool fits = st >= 0 && (long long)st + a.n_tok <= s.L_ctx;
  if (report && i == 0) {
    if (!fits) flag_error(a.err, ERR_BAD_INDEX);
    if (a.end) a.end[b] = fits ? st + a.n_tok : st;
  }
  if (!fits) return -1;
  const int t = st + i, slot = a.page_table[(size_t)b * s.n_pages + t / 64];
  if (slot < 0 || slot >= s.n_slots) {
    if (report) flag_error(a.err, ERR_BAD_INDEX);
    return -1;
  }
  if (report) {
    for (int m = 0; m < a.n_mass; ++m) {
      const size_t e = ((size_t)b * a.n_mass + m) * s.L_ctx + t;
      if (a.tok_pos) a.tok_pos[e] = a.pos[(size_t)b * a.n_tok + i];
      if (a.tok_mass) a.tok_mass[e] = 0.0f;
    }
  }
  return (long long)slot * s.H_kv * 64 + (t % 64);
}

// Sine and cosine of a position's turn at frequency j.
__device__ __forceinline__ void turn(const RopeArgs& a, size_t tok, int j, float* sn, float* cs) {
  const double turns = (double)a.pos[tok] * (double)a.inv_freq[j] * 0.15915494309189533577;
  sincospif(2.0f * (float)(turns - rint(turns)), sn, cs);
}

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
        turn(a, tok0 + t, j, reinterpret_cast<float*>(s_sin[t]) + j, reinterpret_cast<float*>(s_cos[t]) + j);
      }
      if (tid < n_tok) s_row[tid] = cache_row(a, b, i0 + tid, blockIdx.y == 0);
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

// ---- long prompts: eight tokens a CTA and all their rows, a thread keeping to
// its token and columns.
//
// With the kernel above the instructions, not HBM, set the time of a prompt
// (176 for two rows of a warp, 62 of 91 us).  Here a thread holds two runs of
// eight columns (off0.. and off1..) of one token and walks the heads, so that
// the row's coefficients stay in registers with the norm's weights multiplied in,
//   y_u' = inv (x_u (w_u cos) - x_v (w_v sin)),
//   y_v' = inv (x_v (w_v cos) + x_u (w_u sin)),
// and pairs of columns share an instruction (f32x2).  Rows under way stand in a
// ring of shared memory: asynchronous copies of 16 bytes into slots of the thread
// that reads them, so that no thread waits for another, across the kinds of heads.
// 8192 tokens of 96 rows (405 MB): 70 us, 5.8 TB/s; 65536: 506 us, 6.4 TB/s.
// With rows loaded ahead into registers 74.5 and 542; two, six and eight rows
// under way 75.1, 69.9 and 70.2; five CTAs per SM 73.9.
__device__ __forceinline__ unsigned long long pack2(float x, float y) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpack2(unsigned long long v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b,
                                                   unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

constexpr int kWideTokens = 8, kWideThreads = 128;

// 16 bytes into shared memory.  Of fp32 rows a thread's pieces are halves of a
// sector, so they pass L1 (133 us at 8192 tokens of 96 rows, 199 beside it).
template <typename T>
__device__ __forceinline__ void copy16(uint32_t dst, const T* src) {
  if (sizeof(T) == 4) asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Eight consecutive values as loaded.  take(): from a thread's slots of the ring.
template <typename T> struct Oct;
template <> struct Oct<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void take(uint32_t slot) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(slot) : "memory");
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = v; }
  __device__ __forceinline__ void get(unsigned long long (&x)[4]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  }
  __device__ __forceinline__ void set(const unsigned long long (&x)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2(x[i]);
      w[i] = pack_bf16x2(f.x, f.y);
    }
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <> struct Oct<float> {
  float4 v[2];
  __device__ __forceinline__ void load(const float* p) {
    v[0] = *reinterpret_cast<const float4*>(p);
    v[1] = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void take(uint32_t slot) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(v[i].x), "=f"(v[i].y), "=f"(v[i].z), "=f"(v[i].w)
                   : "r"(slot + i * kWideThreads * 16) : "memory");
  }
  __device__ __forceinline__ void store(float* p) const {
    *reinterpret_cast<float4*>(p) = v[0];
    *reinterpret_cast<float4*>(p + 4) = v[1];
  }
  __device__ __forceinline__ void get(unsigned long long (&x)[4]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x[2 * i] = pack2(v[i].x, v[i].y);
      x[2 * i + 1] = pack2(v[i].z, v[i].w);
    }
  }
  __device__ __forceinline__ void set(const unsigned long long (&x)[4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 p = unpack2(x[2 * i]), q = unpack2(x[2 * i + 1]);
      v[i] = make_float4(p.x, p.y, q.x, q.y);
    }
  }
};

template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kWideThreads, 4)
qk_norm_rope_wide_kernel(const __grid_constant__ RopeArgs a, int tiles) {
  constexpr int TT = kWideTokens, TPR = D / 16;       // threads per row
  constexpr int GR = kWideThreads / (TT * TPR);       // heads taken at a time
  constexpr int V = (int)sizeof(T);                   // 16-byte pieces of a thread's columns of a row
  constexpr int S = 8 / (int)sizeof(T);               // rows under way
  __shared__ __align__(16) char s_ring[S * V * kWideThreads * 16];
  __shared__ float s_cos[TT][D / 2], s_sin[TT][D / 2];
  __shared__ long long s_row[TT];
  const Shape& s = a.s;
  const int tid = threadIdx.x, c = tid % TPR, t = (tid / TPR) % TT, grp = tid / (TPR * TT);
  const int b = blockIdx.x / tiles, i0 = (blockIdx.x - b * tiles) * TT;
  const int n_tok = min(TT, a.n_tok - i0), half = a.rot_dim / 2;
  const size_t tok0 = (size_t)b * a.n_tok + i0;
  const bool live = t < n_tok;
  // columns: off0 .. + 7 and off1 .. + 7.  Split pairing: a run and its partners, or
  // two runs left alone; interleaved: whole pairs, side by side over the lanes
  int off0, off1;
  bool rot0, rot1;
  if (INTER) {
    off0 = 8 * c;
    off1 = D / 2 + off0;
    rot0 = off0 < a.rot_dim;
    rot1 = off1 < a.rot_dim;
  } else if (8 * c < half) {
    off0 = 8 * c;
    off1 = half + off0;
    rot0 = rot1 = true;
  } else {
    off0 = a.rot_dim + 8 * c - half;
    off1 = off0 + (D - a.rot_dim) / 2;
    rot0 = rot1 = false;
  }
  pdl_trigger();
  pdl_wait();
  // a token past the last reads the last one's rows and writes nothing
  const T* src = reinterpret_cast<const T*>(a.qkv) + (tok0 + min(t, n_tok - 1)) * a.qkv_stride;
  const int rows = s.H + 2 * s.H_kv;                  // query, key, value heads, side by side
  const uint32_t slot0 = sm100::smem_u32(s_ring) + tid * 16;
  auto fetch = [&](int slot, int r) {
    if (r < rows) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        copy16<T>(slot0 + (slot * V + i) * kWideThreads * 16,
                  src + (size_t)r * D + (i < V / 2 ? off0 : off1) + i % (V / 2) * (16 / (int)sizeof(T)));
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll 1
  for (int u = 0; u < S; ++u) fetch(u, grp + u * GR);
  for (int e = tid; e < n_tok * half; e += kWideThreads) {
    const int tt = e / half, j = e - tt * half;
    turn(a, tok0 + tt, j, &s_sin[tt][j], &s_cos[tt][j]);
  }
  if (tid < n_tok) s_row[tid] = cache_row(a, b, i0 + tid, true);
  __syncthreads();
  const long long row = live ? s_row[t] : -1;
  int kind = 0, last = 0, slot = 0;
  T *out = nullptr, *pool = nullptr;
  bool scaled = false;
  unsigned long long A[4], B[4], C[4], E[4];
#pragma unroll 1
  for (int r = grp; r < rows; r += GR) {  // uniform over a warp
    if (r >= last) {                                  // the first row of a kind
      kind = r < s.H ? 0 : r < s.H + s.H_kv ? 1 : 2;
      const int n = kind == 0 ? s.H : s.H_kv;
      const int h0 = kind == 0 ? 0 : kind == 1 ? s.H : s.H + s.H_kv;
      last = h0 + n;
      out = reinterpret_cast<T*>(kind == 0 ? a.Q_out : kind == 1 ? a.K_out : a.V_out);
      if (out) out += ((size_t)b * n * a.n_tok + i0 + t + (long long)(r - h0) * a.n_tok) * D;
      pool = nullptr;
      if (kind > 0 && row >= 0)
        pool = reinterpret_cast<T*>(kind == 1 ? a.K_pool : a.V_pool) + (row + (long long)(r - h0) * 64) * D;
      const T* w = reinterpret_cast<const T*>(kind == 0 ? a.q_weight : kind == 1 ? a.k_weight : nullptr);
      scaled = w != nullptr;
      if (kind < 2) {
        unsigned long long w0[4], w1[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w0[i] = w1[i] = pack2(1.0f, 1.0f);
        if (w) {
          Oct<T> o;
          o.load(w + off0);
          o.get(w0);
          o.load(w + off1);
          o.get(w1);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 p = unpack2(w0[i]), q = unpack2(w1[i]);
          float c0 = 1.0f, c1 = 1.0f, c2 = 1.0f, c3 = 1.0f, s0 = 0.0f, s1 = 0.0f, s2 = 0.0f, s3 = 0.0f;
          if (INTER) {                                // pair i of each run
            if (rot0 && live) { c0 = c1 = s_cos[t][4 * c + i]; s0 = s1 = s_sin[t][4 * c + i]; }
            if (rot1 && live) { c2 = c3 = s_cos[t][D / 4 + 4 * c + i]; s2 = s3 = s_sin[t][D / 4 + 4 * c + i]; }
          } else if (rot0 && live) {
            c0 = c2 = s_cos[t][8 * c + 2 * i]; s0 = s2 = s_sin[t][8 * c + 2 * i];
            c1 = c3 = s_cos[t][8 * c + 2 * i + 1]; s1 = s3 = s_sin[t][8 * c + 2 * i + 1];
          }
          A[i] = pack2(p.x * c0, p.y * c1);
          C[i] = pack2(q.x * c2, q.y * c3);
          // what the partner adds: its own weight, minus for the first of a pair
          B[i] = INTER ? pack2(-p.y * s0, p.x * s1) : pack2(-q.x * s0, -q.y * s1);
          E[i] = INTER ? pack2(-q.y * s2, q.x * s3) : pack2(p.x * s2, p.y * s3);
        }
      }
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
    Oct<T> v0, v1;
    v0.take(slot0 + slot * V * kWideThreads * 16);
    v1.take(slot0 + (slot * V + V / 2) * kWideThreads * 16);
    fetch(slot, r + S * GR);
    slot = slot + 1 < S ? slot + 1 : 0;
    if (kind < 2) {
      unsigned long long x[4], y[4];
      v0.get(x);
      v1.get(y);
      unsigned long long inv = pack2(1.0f, 1.0f);
      if (scaled) {
        unsigned long long sq = mul2(x[0], x[0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) sq = fma2(x[i], x[i], sq);
#pragma unroll
        for (int i = 0; i < 4; ++i) sq = fma2(y[i], y[i], sq);
        const float2 f = unpack2(sq);
        float q = f.x + f.y;
#pragma unroll
        for (int o = TPR / 2; o > 0; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
        const float z = __frsqrt_rn(q * (1.0f / D) + a.eps);
        inv = pack2(z, z);
      }
      unsigned long long p[4], q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[i] = mul2(x[i], A[i]);
        q[i] = mul2(y[i], C[i]);
      }
      // where nothing is rotated the partner's values must not reach a column
      if (INTER) {
        if (rot0) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = unpack2(x[i]);
            p[i] = fma2(pack2(f.y, f.x), B[i], p[i]);
          }
        }
        if (rot1) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 g = unpack2(y[i]);
            q[i] = fma2(pack2(g.y, g.x), E[i], q[i]);
          }
        }
      } else if (rot0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p[i] = fma2(y[i], B[i], p[i]);
          q[i] = fma2(x[i], E[i], q[i]);
        }
      }
      if (scaled) {
#pragma unroll
        for (int i = 0; i < 4; ++i) { p[i] = mul2(p[i], inv); q[i] = mul2(q[i], inv); }
      }
      v0.set(p);
      v1.set(q);
    }
    if (live && out) {
      v0.store(out + off0);
      v1.store(out + off1);
    }
    if (pool) {
      v0.store(pool + off0);
      v1.store(pool + off1);
      pool += (size_t)GR * 64 * D;
    }
    if (out) out += (size_t)GR * a.n_tok * D;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <typename T, int D>
cudaError_t run_rope(const RopeArgs& a, cudaStream_t st) {
  const Shape& s = a.s;
  constexpr int RPP = kRopeThreads / (D / 8);
  const int n_rows = s.H + 2 * s.H_kv;
  // Tokens a CTA: eight when a sequence has them; 32 where a token has few rows
  // and there are enough (3 rows of 64, 138 K tokens: 66.6 us at 8, 43.0 at 32;
  // 3000 tokens: 5.5 at 8, 8.5 at 32).  Rows are split over CTAs down to one pass
  // each while that is needed to fill the GPU six CTAs deep.
  const int sms = tc_sm_count();
  const bool few = n_rows * D < 1280;
  const int tt = few && (long long)s.batch * (a.n_tok / 32) >= 4ll * sms ? 32 : a.n_tok >= 8 ? 8 : 1;
  const int tiles = (a.n_tok + tt - 1) / tt;
  const long long all = (long long)s.batch * tiles, want = 6ll * sms;
  // The long-prompt kernel, where
  // - the tokens fill the GPU without splitting their rows (96 rows of bf16: 1800
  //   tokens 29.8 against 25.0 us, 2400: 30.6 against 31.6, 8192: 69 against 90;
  //   fp32: 2400 tokens 61.4 against 50.6, 3600: 73.5 against 74.8, 8192: 135
  //   against 159);
  // - a token has the rows to share the coefficients (60000 tokens: 8 rows 76.0
  //   against 70.0 us, 10: 82.9 against 83.5, 16: 103 against 120; fp32 99.8 against
  //   100, 115 against 122, 169 against 190; of 64 columns, 16 rows 73.7 against 63.7,
  //   20: 80.7 against 76.5, 24: 88.0 against 89.3, 32: 102 against 116; fp32 94.1
  //   against 83.5, 109 against 103, 126 against 123, 166 against 164);
  // - runs of eight columns are rotated or left alone as a whole.
  if (tt == 8 && !few && all >= (sizeof(T) == 2 ? 2ll : 3ll) * sms && a.rot_dim % 16 == 0) {
    if (a.interleaved)
      DL_LAUNCH_DEPENDENT((qk_norm_rope_wide_kernel<T, D, true>), (unsigned)all, kWideThreads, 0, st, a, tiles);
    else
      DL_LAUNCH_DEPENDENT((qk_norm_rope_wide_kernel<T, D, false>), (unsigned)all, kWideThreads, 0, st, a, tiles);
    return cudaGetLastError();
  }
  const int most = (n_rows * tt + RPP - 1) / RPP;
  long long split = all < want ? (want + all - 1) / all : 1;
  split = split < most ? split : most;
  const int per = (n_rows + (int)split - 1) / (int)split;
  const dim3 grid((unsigned)all, (n_rows + per - 1) / per);
  if (tt == 32) {
    DL_LAUNCH_DEPENDENT((qk_norm_rope_kernel<T, D, 32, 4>), grid, kRopeThreads, 0, st, a, tiles, per);
  } else if (tt == 1) {
    DL_LAUNCH_DEPENDENT((qk_norm_rope_kernel<T, D, 1, 1>), grid, kRopeThreads, 0, st, a, tiles, per);
  } else if (per * tt <= RPP) {
    DL_LAUNCH_DEPENDENT((qk_norm_rope_kernel<T, D, 8, 1>), grid, kRopeThreads, 0, st, a, tiles, per);
  } else {
    DL_LAUNCH_DEPENDENT((qk_norm_rope_kernel<T, D, 8, 4>), grid, kRopeThreads, 0, st, a, tiles, per);
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
