// (c2) Attention of one new token per sequence over its cached tokens.
//
//   a_t = scale q.k_t,  lse = ln sum_t e^{a_t},  o = sum_t e^{a_t - lse} v_t
//   mass_t <- decay mass_t + sum_h e^{a_t - lse_h}
//
// Bound: HBM.  A key or value row is read once for every block of RB query heads of
// its KV group: once for groups of up to 16 heads (fp32: 8), ceil(G / RB) times for
// larger ones, whose blocks are items with copies of their own (4 x 32K, 32/2 heads
// 31.6 us, 64/2 heads 49.9); a group of G heads does 4 G d flops per 4 d bytes (bf16).
//
// Work split.  An item is (sequence, KV head, block of RB query heads); its
// keys are tiles of KT.  The tiles of all items, in order, are cut into one
// equal run per CTA, whatever the lengths are: the lengths are read on the
// device, so a batch of very different sequences stays balanced and a single
// long one spreads over the whole GPU.  An item counts as kItemCost tiles more
// than it has, for what its start and end take.  A run is walked item by item
// (segments).  An item inside one run is finished there; otherwise each of
// its runs leaves a partial (maximum, sum, unnormalised output) in the
// workspace, and the join kernel adds them in run order.
//
// Small problems (few tiles for every CTA, all CTAs resident at once) take the
// items whole instead: a cluster of up to 8 CTAs shares an item's tiles, joins
// through its shared memory and adds the masses itself, so the join kernel,
// half of such a call's time, is not needed.
//
// Roles.  Warp 4 copies pages into a ring of shared-memory stages by TMA
// (128-byte swizzle) through the page table, running ahead across segments.
// Warps 0-3 take a quarter of each tile's keys each, with a running maximum
// and sum of their own, so that nothing but the ring synchronises them until
// the segment ends; then their states are added in warp order.
//
// bf16: S = Q K^T and O += P V on m16n8k16 tensor core instructions, fp32
// accumulation, query heads on the M side.  Weights are fed as bf16 high and
// low parts, p = hi + lo + O(2^-17 p), so O keeps the precision of fp32
// weights; with at most 8 heads the two parts share one instruction (rows 0-7
// high, 8-15 low), with 9-16 they take two.  The instruction is used because
// a tile has at most 16 useful rows and the operands' conversion and traffic,
// not the products, are what fills an SM here.
// fp32: the same walk on the CUDA cores: lane = (two or four keys, eighth of d) for
// S, lane = four columns for O.  The dot products are summed in fp64 and stay so
// until the reference is subtracted: beside a sink's logit of 35 one fp32 rounding
// of a logit is 1e-6 of its weight, as large as all other errors together.  Groups
// of up to four heads reach HBM (2 x 32K, 32/8 heads of 128: 87 to 99 us from card to
// card, 5.4 to 6.2 TB/s); with eight (8 x 32K, 32/4 heads) it takes 270 us against 164:
// issue slots are 54 % busy, the fp64 pipe 24 %, and the eight computing warps (of ten,
// 168 registers) per SM do not hide the rest (fp32 sums took 215).  Several keys a lane
// share a read of Q: with one, and quarters of d, 300 us; with Q in registers, every
// lane four columns and the sums dealt out over 32 lanes, 338.
//
// Weights.  With c = scale log2 e and a maximum m of the dot products x, the
// reference is M = m c rounded once, and p = 2^(x c - M) in one fused
// operation: its argument is rounded at its own size, not at that of x c (a
// sink's logit of 35 would cost 1e-6 of every weight beside it).  Everything
// that is joined is relative to these M.
//
// Masses.  The main kernel leaves the dot products in the workspace; the join
// kernel's other CTAs turn them into weights with the joined maxima and sums
// and add them over the heads, in head order.
#include <atomic>

#include "cluster.cuh"
#include "common.cuh"
#include "internal.h"
#include "launch.cuh"
#include "sm100.cuh"
#include "tc_common.cuh"

namespace dl {

using namespace sm100;

namespace {

constexpr int kWarps = 4;                       // computing warps
constexpr int kThreads = (kWarps + 1) * 32;     // + the copying warp
constexpr int kCtasPerSm = 2;
constexpr int kMaxCtas = 148 * kCtasPerSm;      // partial slots are sized for this many
constexpr int kJoinThreads = 256;
constexpr int kMaxCluster = 8;
// Most tiles of a cluster CTA: 4, or 16 when clusters fill three quarters of the
// GPU and equal runs would be as long (bf16, d 128, clusters against runs: 8
// items of 4 tiles a CTA 10.3 to 12.3 us, of 8 tiles 14.4 to 12.3; 32 items of 8
// tiles 18.3 to 21.4, of 16 tiles 28.1 to 31.2).  The same borders serve 64 columns
// and fp32, back to back in a graph: bf16 of 64, 8 items of 4 tiles 6.8 to 8.3, of 8
// tiles 9.5 to 8.5; 30 items of 16 tiles 22.0 to 22.3; fp32 of 64, 8 items of 4 tiles
// 9.1 to 10.1, of 8 tiles 13.8 to 11.0; 30 items of 16 tiles 34.2 to 33.1; fp32 of 128,
// 8.9 to 9.7, 13.0 to 10.8, 32.4 to 32.0.  Two items of 4 fp32 tiles lose by it (four
// heads 8.7 to 8.3, eight 11.9 to 10.3), sixty and more win at any size.
constexpr int kClusterTiles = 4, kClusterTilesFull = 16;
constexpr float kLn2 = 0.69314718055994531f;
constexpr double kLog2e = 1.4426950408889634;

// Query heads per item block: 8; 16 for bf16 groups of more than 8; 4 or 2 for fp32
// groups of at most as many (on the CUDA cores empty rows cost as much as others:
// four heads in a block of eight 170 us, of four 88).
__host__ __device__ inline int rows_per_block(const Shape& s) {
  if (s.dtype == DL_BF16) return s.G > 8 ? 16 : 8;
  return s.G > 4 ? 8 : s.G > 2 ? 4 : 2;
}
__host__ __device__ inline int items_per_seq(const Shape& s) {
  const int rb = rows_per_block(s);
  return s.H_kv * ((s.G + rb - 1) / rb);
}

// Extra count of an item: at full load a tile takes 1.5 us of a CTA, an item's
// query load, state join and output 3 to 4 us (ragged 32 x 8K, 32/8 heads of 128, bf16:
// 0 -> 64.5 us, 1 -> 60.9, 3 -> 60.4, 6 -> 60.5; of 64: 47.0, 42.6, 40.8, 41.7).  fp32
// tiles hold as many bytes and take as long or longer, so it serves them too (32/8
// heads of 64: 80.4, 69.3, 63.5, 66.1; 64/8 of 128: 186, 169, 164, 170; 32 x 2000, 16/8
// heads of 128: 43.3, 35.6, 30.7, 31.8).
constexpr int kItemCost = 3;

struct DecodeWs {
  int* runs;         // [batch][items][2]: first and last run of each item
  float* po;         // [2 kMaxCtas][RB][d] unnormalised partial outputs
  float2* pml;       // [2 kMaxCtas][RB] (reference, sum)
  float2* norm;      // [batch][H] (reference, 1 / sum) of the items finished in one run
  void* logit;       // [batch][H][Lp] dot products (with masses): fp32, fp64 of fp32 keys
  int Lp;
};

size_t carve(const Shape& s, bool mass, void* ws, DecodeWs* w) {
  const int rb = rows_per_block(s);
  char* p = reinterpret_cast<char*>(ws);
  size_t at = 0;
  auto take = [&](size_t n) { char* q = p + at; at += round256(n); return q; };
  DecodeWs d;
  d.Lp = (s.L_ctx + 63) / 64 * 64;
  d.runs = reinterpret_cast<int*>(take((size_t)s.batch * items_per_seq(s) * 8));
  d.po = reinterpret_cast<float*>(take((size_t)2 * kMaxCtas * rb * s.d * 4));
  d.pml = reinterpret_cast<float2*>(take((size_t)2 * kMaxCtas * rb * 8));
  d.norm = reinterpret_cast<float2*>(take((size_t)s.batch * s.H * 8));
  d.logit = take(mass ? (size_t)s.batch * s.H * d.Lp * (s.dtype == DL_BF16 ? 4 : 8) : 0);
  if (w) *w = d;
  return at;
}

// Dot products in the workspace, and the exponent of a weight from one.
template <typename T> struct Logit;
template <> struct Logit<__nv_bfloat16> {
  using Type = float;
  __device__ __forceinline__ static float exponent(float x, float c2, double, float M) { return fmaf(x, c2, -M); }
};
template <> struct Logit<float> {
  using Type = double;
  __device__ __forceinline__ static float exponent(double x, float, double c2d, float M) {
    return (float)fma(x, c2d, -(double)M);
  }
};

// Cached tokens of sequence b; a length out of range counts as 0.
__device__ __forceinline__ int seq_len(const DecodeArgs& a, int b) {
  const int n = a.ctx_len[b];
  return n >= 0 && n <= a.s.L_ctx ? n : 0;
}

// a b / c and the like on tile counts: 32 bits where they suffice (a 64-bit
// division is a long chain at the head of every CTA).
__device__ __forceinline__ long long div_tiles(long long x, long long y) {
  if (((x | y) >> 32) == 0) return (unsigned)x / (unsigned)y;
  return x / y;
}

// One run's part of an item.
struct Segment {
  int b, item, t0, t1, nt, len;
};

// Tiles that a sequence of `len` tokens counts as.
__device__ __forceinline__ long long seq_cost(int len, int kt, int ips) {
  return len == 0 ? 0 : (long long)((len + kt - 1) / kt + kItemCost) * ips;
}

// Walks the segments of a run; every role of a CTA walks the same ones.
struct Walk {
  const DecodeArgs& a;
  long long left;  // of the run, in counted tiles
  int ips, kt, b, item, v, nt, len;
  // The run of n counted tiles starts `off` of them into sequence b_ of len_ tokens.
  __device__ Walk(const DecodeArgs& a_, int ips_, int kt_, int b_, int len_, long long off, long long n)
      : a(a_), left(n), ips(ips_), kt(kt_), b(b_), len(len_) {
    nt = (len + kt - 1) / kt;
    item = (int)div_tiles(off, nt + kItemCost);
    v = (int)(off - (long long)item * (nt + kItemCost));
  }
  __device__ bool next(Segment* s) {
    while (left > 0) {
      const int n = (int)min((long long)(nt + kItemCost - v), left);
      *s = Segment{b, item, max(0, v - kItemCost), max(0, v + n - kItemCost), nt, len};
      left -= n;
      v = 0;
      if (left > 0 && ++item == ips) {
        item = 0;
        do len = seq_len(a, ++b); while (len == 0);
        nt = (len + kt - 1) / kt;
      }
      if (s->t1 > s->t0) return true;  // else the run ends inside the item's extra count
    }
    return false;
  }
};

// A cluster CTA's only segment (possibly without tiles).
struct Single {
  Segment seg;
  bool done;
  __device__ bool next(Segment* s) {
    if (done) return false;
    done = true;
    *s = seg;
    return true;
  }
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The larger of two, NaN if either is: a NaN dot product has to reach its row's
// maximum, or a warp that holds nothing else would pass for one without keys.
__device__ __forceinline__ float max_nan(float x, float y) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float warp_max_nan(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
// Two fp32 values as bf16 high parts and bf16 remainders.
__device__ __forceinline__ void split_bf16(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  const float2 f = __bfloat1622float2(h);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = pack_bf16x2(x - f.x, y - f.y);
}
// Two bf16 values, infinities and NaN as the largest finite ones: what the low parts
// of the weights multiply.  A low part may be 0 or negative, and would turn the
// infinity that the high part gives into NaN.  (8 x 32K, 128/8 heads of 64: 94.0 us,
// without it 94.5, by a minimum and a maximum 99.4.)
__device__ __forceinline__ uint32_t finite_bf16x2(uint32_t v) {
  asm("min.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(v) : "r"(0x7F7F7F7Fu));  // v's sign, the smaller magnitude
  return v;
}

template <typename T, int D_, int RB_>
struct Cfg {
  static constexpr int D = D_, RB = RB_;
  static constexpr bool BF16 = sizeof(T) == 2;
  // Keys per tile, 32 KB of K and V; half of that for blocks of eight fp32 rows of
  // 64, which 16 keys a warp would spill (32K keys: 357 us against 413; of four
  // rows, 8 x 32K, 32/8 heads, 64 keys 184, 32 keys 245).
  static constexpr int KT = BF16 || (D == 64 && RB < 8) ? 64 : 32;
  static constexpr int BOX = KT * 128;                 // bytes of one 128-byte-wide box
  static constexpr int BOXES = D * (int)sizeof(T) / 128;
  static constexpr int HALF = BOX * BOXES;             // K (or V) of a stage
  static constexpr int STAGE = 2 * HALF;
  static constexpr int ST = 96 * 1024 / STAGE;         // stages: 96 KB of copies in flight per CTA
  // states of the other warps at a segment's end: all three at once, or one by one
  static constexpr int COPIES = BF16 && RB == 8 ? 3 : 1;
  static constexpr int O_OFF = ST * STAGE;
  static constexpr int Q_OFF = O_OFF + COPIES * RB * D * 4;        // fp32 keys: rows of Q in fp64
  static constexpr int P_OFF = Q_OFF + (BF16 ? 0 : RB * D * 8);    // fp32 keys: weights [warp][RB][KT / 4]
  static constexpr int ML_OFF = P_OFF + (BF16 ? 0 : RB * KT * 4);
  static constexpr int BAR_OFF = ML_OFF + kWarps * RB * 8;
  static constexpr int MISC_OFF = BAR_OFF + 2 * ST * 8;            // info [ST], abort
  static constexpr int SMEM = MISC_OFF + (ST + 4) * 4 + 1024;      // + alignment slack
  static_assert(2 * (SMEM + 1024) <= 228 * 1024, "two CTAs per SM");
};

// Running state of one warp's keys of a segment, bf16.
template <int D, int RB>
struct StateTc {
  static constexpr int NR = RB / 8;  // fragment rows per thread: lane/4 (and + 8)
  float o[D / 8][4];
  float m[NR], l[NR];
  uint32_t q[D / 16][2 * NR];
  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
#pragma unroll
    for (int r = 0; r < NR; ++r) { m[r] = -INFINITY; l[r] = 0.0f; }
  }
  __device__ __forceinline__ void load_q(const __nv_bfloat16* Q, int n_rows, int lane) {
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const int row = lane / 4 + 8 * r;
      const uint32_t* p = reinterpret_cast<const uint32_t*>(Q + (size_t)row * D) + (lane & 3);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        q[k][r] = row < n_rows ? p[8 * k] : 0u;
        q[k][NR + r] = row < n_rows ? p[8 * k + 4] : 0u;
      }
    }
  }
  // 16 keys of the stage; `valid` of the tile's 64 hold tokens.
  __device__ __forceinline__ void tile(uint32_t ks, uint32_t vs, int warp, int lane, int valid,
                                       float c2, float* logit, int Lp, int n_rows) {
    float s[2][4] = {};
    {
      const int key = warp * 16 + (lane & 7) + ((lane >> 4) << 3), hi = (lane >> 3) & 1;
      const uint32_t row = ks + key * 128;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const int c = 2 * k + hi;
        uint32_t kf[4];
        ldsm4(row + (c >> 3) * (64 * 128) + (((c & 7) ^ (key & 7)) << 4), kf);
        uint32_t af[4];
        if constexpr (NR == 1) {
          af[0] = q[k][0]; af[1] = 0u; af[2] = q[k][1]; af[3] = 0u;
        } else {
          af[0] = q[k][0]; af[1] = q[k][1]; af[2] = q[k][2]; af[3] = q[k][3];
        }
        mma16816(s[0], af, kf[0], kf[1]);
        mma16816(s[1], af, kf[2], kf[3]);
      }
    }
    const int k0 = warp * 16 + 2 * (lane & 3);  // this thread's keys: k0, k0+1, k0+8, k0+9
    const bool part = valid < 64;
    bool ok[2][2];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) ok[n][e] = k0 + 8 * n + e < valid;
    float x[NR][4];
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[r][j] = !part || ok[j >> 1][j & 1] ? s[j >> 1][2 * r + (j & 1)] : -INFINITY;
      }
    if (logit) {
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const int row = lane / 4 + 8 * r;
        if (row < n_rows) {
          float* p = logit + (size_t)row * Lp + k0;
          *reinterpret_cast<float2*>(p) = make_float2(x[r][0], x[r][1]);
          *reinterpret_cast<float2*>(p + 8) = make_float2(x[r][2], x[r][3]);
        }
      }
    }
    bool raise = false;
    float top[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      float t = max_nan(max_nan(x[r][0], x[r][1]), max_nan(x[r][2], x[r][3]));
      t = max_nan(t, __shfl_xor_sync(0xffffffffu, t, 1));
      t = max_nan(t, __shfl_xor_sync(0xffffffffu, t, 2));
      top[r] = max_nan(m[r], t);
      raise |= !(top[r] <= m[r]);
    }
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float f = top[r] == -INFINITY ? 1.0f : ex2_approx(__fmul_rn(m[r], c2) - __fmul_rn(top[r], c2));
        m[r] = top[r];
        l[r] *= f;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          o[i][2 * r] *= f; o[i][2 * r + 1] *= f;
          if (NR == 1) { o[i][2] *= f; o[i][3] *= f; }  // the low parts' sums
        }
      }
    }
    uint32_t hi[NR][2], lo[NR][2];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const float M = m[r] == -INFINITY ? 0.0f : __fmul_rn(m[r], c2);
      float p[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) p[j] = ex2_approx(fmaf(x[r][j], c2, -M));
      l[r] += (p[0] + p[1]) + (p[2] + p[3]);
      split_bf16(p[0], p[1], hi[r][0], lo[r][0]);
      split_bf16(p[2], p[3], hi[r][1], lo[r][1]);
    }
    // rows behind the last token hold anything: their values are cleared
    const uint32_t keep0 = (ok[0][0] ? 0xFFFFu : 0u) | (ok[0][1] ? 0xFFFF0000u : 0u);
    const uint32_t keep1 = (ok[1][0] ? 0xFFFFu : 0u) | (ok[1][1] ? 0xFFFF0000u : 0u);
    const int key = warp * 16 + (lane & 7) + (((lane >> 3) & 1) << 3);
    const uint32_t row = vs + key * 128;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      const int c = 2 * i + (lane >> 4);
      uint32_t vf[4];
      ldsm4_t(row + (c >> 3) * (64 * 128) + (((c & 7) ^ (key & 7)) << 4), vf);
      if (part) { vf[0] &= keep0; vf[1] &= keep1; vf[2] &= keep0; vf[3] &= keep1; }
      if constexpr (NR == 1) {
        const uint32_t af[4] = {hi[0][0], lo[0][0], hi[0][1], lo[0][1]};
        mma16816(o[2 * i], af, vf[0], vf[1]);
        mma16816(o[2 * i + 1], af, vf[2], vf[3]);
      } else {
        const uint32_t ah[4] = {hi[0][0], hi[1][0], hi[0][1], hi[1][1]};
        const uint32_t al[4] = {lo[0][0], lo[1][0], lo[0][1], lo[1][1]};
        mma16816(o[2 * i], ah, vf[0], vf[1]);
        mma16816(o[2 * i + 1], ah, vf[2], vf[3]);
#pragma unroll
        for (int e = 0; e < 4; ++e) vf[e] = finite_bf16x2(vf[e]);
        mma16816(o[2 * i], al, vf[0], vf[1]);
        mma16816(o[2 * i + 1], al, vf[2], vf[3]);
      }
    }
  }
  // ---- segment end
  __device__ __forceinline__ void finish(int) {
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    }
    if constexpr (NR == 1) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {  // beside an infinite value the low sums are NaN: 0 or less times it
        if (isfinite(o[i][0])) o[i][0] += o[i][2];
        if (isfinite(o[i][1])) o[i][1] += o[i][3];
      }
    }
  }
  __device__ __forceinline__ void put_ml(float2* ml, int lane, float c2) const {
    if ((lane & 3) == 0) {
#pragma unroll
      for (int r = 0; r < NR; ++r) ml[lane / 4 + 8 * r] = make_float2(__fmul_rn(m[r], c2), l[r]);
    }
  }
  __device__ __forceinline__ void scale(const float* f, int lane) {  // f: per row, shared memory
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const float w = f[lane / 4 + 8 * r];
#pragma unroll
      for (int i = 0; i < D / 8; ++i) { o[i][2 * r] *= w; o[i][2 * r + 1] *= w; }
    }
  }
  __device__ __forceinline__ void put(float* dst, int lane) const {
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int r = 0; r < NR; ++r)
        reinterpret_cast<float2*>(dst)[(i * NR + r) * 32 + lane] = make_float2(o[i][2 * r], o[i][2 * r + 1]);
  }
  __device__ __forceinline__ void add(const float* src, int lane) {
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float2 v = reinterpret_cast<const float2*>(src)[(i * NR + r) * 32 + lane];
        o[i][2 * r] += v.x; o[i][2 * r + 1] += v.y;
      }
  }
  template <typename F>
  __device__ __forceinline__ void each(int lane, F f) const {  // f(row, column, two values)
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        f(lane / 4 + 8 * r, 8 * i + 2 * (lane & 3), make_float2(o[i][2 * r], o[i][2 * r + 1]));
  }
};

// Running state of one warp's keys of a segment, fp32: o holds columns
// 4 (lane % (D/4)) .. + 3, of every second key when D is 64.
template <int D, int RB, int KT>
struct StateF32 {
  static constexpr int CH = D / 4;          // 16-byte columns of a row
  static constexpr int KS = 32 / CH;        // keys taken at a time by the P V lanes
  static constexpr int NKW = KT / kWarps;   // this warp's keys of a tile: 8 or 16
  static constexpr int NK = NKW / 4;        // of them under one lane while S is taken
  static constexpr int DUP = 32 / NKW;      // lanes with the same key afterwards
  float o[RB][4];
  float m[RB], l[RB];                       // l: of this lane's key
  const double* sq;                         // Q rows in shared memory, see q_at
  float* sp;                                // this warp's weights [RB][NKW]
  // Column e of row r: pairs of a 16-byte column of K apart, so that the lanes of
  // eight columns read 128 bytes side by side.
  __device__ __forceinline__ static int q_at(int r, int e) {
    return r * D + (e >> 1 & 1) * (D / 2) + (e >> 2) * 2 + (e & 1);
  }
  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      o[r][0] = o[r][1] = o[r][2] = o[r][3] = 0.0f;
      m[r] = -INFINITY; l[r] = 0.0f;
    }
  }
  __device__ __forceinline__ static uint32_t chunk_at(int key, int c) {
    return (c >> 3) * (KT * 128) + key * 128 + (((c & 7) ^ (key & 7)) << 4);
  }
  __device__ __forceinline__ void tile(const char* ks, const char* vs, int warp, int lane, int valid,
                                       float c2, double c2d, double* logit, int Lp, int n_rows) {
    if (warp * NKW >= valid) return;        // none of this warp's keys
    // S: lane = (NK keys 4 apart, eighth of the columns); lane bit 2 is the eighth's
    // top bit, so that eight neighbouring lanes hit all banks
    const int kk = lane & 3, dq = (lane & 4) | lane >> 3;
    double y[NK][RB];
#pragma unroll
    for (int n = 0; n < NK; ++n)
#pragma unroll
      for (int r = 0; r < RB; ++r) y[n][r] = 0.0;
#pragma unroll
    for (int j = 0; j < CH / 8; ++j) {
      const int c = 8 * j + dq;
      double k[NK][4];
#pragma unroll
      for (int n = 0; n < NK; ++n) {
        const float4 f = *reinterpret_cast<const float4*>(ks + chunk_at(warp * NKW + 4 * n + kk, c));
        k[n][0] = f.x; k[n][1] = f.y; k[n][2] = f.z; k[n][3] = f.w;
      }
#pragma unroll
      for (int r = 0; r < RB; ++r) {
        const double2 p = *reinterpret_cast<const double2*>(sq + q_at(r, 4 * c));
        const double2 q = *reinterpret_cast<const double2*>(sq + q_at(r, 4 * c + 2));
#pragma unroll
        for (int n = 0; n < NK; ++n)
          y[n][r] = fma(p.x, k[n][0], fma(p.y, k[n][1], fma(q.x, k[n][2], fma(q.y, k[n][3], y[n][r]))));
      }
    }
    // the eighths' sums; a lane gives away keys while it has several
    const int kl = 4 * (lane >> (NK == 2 ? 4 : 3)) + kk, key = warp * NKW + kl, dup = (lane >> 2) % DUP;
    const bool ok = key < valid;
    bool raise = false;
    double x[RB];
    float top[RB];
#pragma unroll
    for (int r = 0; r < RB; ++r) {
#pragma unroll
      for (int w = 16, n = NK; w >= 4; w >>= 1) {
        if (n > 1) {
          n /= 2;
#pragma unroll
          for (int i = 0; i < n; ++i) {
            const double keep = lane & w ? y[n + i][r] : y[i][r], give = lane & w ? y[i][r] : y[n + i][r];
            y[i][r] = keep + __shfl_xor_sync(0xffffffffu, give, w);
          }
        } else {
          y[0][r] += __shfl_xor_sync(0xffffffffu, y[0][r], w);
        }
      }
      x[r] = ok ? y[0][r] : -INFINITY;
      if (logit && dup == 0 && r < n_rows) logit[(size_t)r * Lp + key] = x[r];
      float t = (float)x[r];
      t = max_nan(t, __shfl_xor_sync(0xffffffffu, t, 1));
      t = max_nan(t, __shfl_xor_sync(0xffffffffu, t, 2));
      t = max_nan(t, __shfl_xor_sync(0xffffffffu, t, 16));
      if (NK == 4) t = max_nan(t, __shfl_xor_sync(0xffffffffu, t, 8));
      top[r] = max_nan(m[r], t);
      raise |= !(top[r] <= m[r]);
    }
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int r = 0; r < RB; ++r) {
        const float f = top[r] == -INFINITY ? 1.0f : ex2_approx(__fmul_rn(m[r], c2) - __fmul_rn(top[r], c2));
        m[r] = top[r];
        l[r] *= f;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[r][e] *= f;
      }
    }
    __syncwarp();
    // weights, those of one P V lane side by side
    const int at = kl % KS * (NKW / KS) + kl / KS;
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      const float M = m[r] == -INFINITY ? 0.0f : __fmul_rn(m[r], c2);
      const float p = ex2_approx((float)fma(x[r], c2d, -(double)M));
      l[r] += p;
      if (dup == r % DUP) sp[r * NKW + at] = p;
    }
    __syncwarp();
    const int c = lane % CH, ks0 = lane / CH;
#pragma unroll
    for (int k0 = 0; k0 < NKW / KS; k0 += 4) {
      float4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = warp * NKW + (k0 + i) * KS + ks0;
        v[i] = *reinterpret_cast<const float4*>(vs + chunk_at(t, c));
        if (t >= valid) v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);  // behind the last token
      }
#pragma unroll
      for (int r = 0; r < RB; ++r) {
        const float4 q = *reinterpret_cast<const float4*>(sp + r * NKW + ks0 * (NKW / KS) + k0);
        const float p[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          o[r][0] = fmaf(p[i], v[i].x, o[r][0]);
          o[r][1] = fmaf(p[i], v[i].y, o[r][1]);
          o[r][2] = fmaf(p[i], v[i].z, o[r][2]);
          o[r][3] = fmaf(p[i], v[i].w, o[r][3]);
        }
      }
    }
  }
  __device__ __forceinline__ void finish(int) {
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 16);
      if (NK == 4) l[r] += __shfl_xor_sync(0xffffffffu, l[r], 8);
      if constexpr (KS == 2) {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[r][e] += __shfl_xor_sync(0xffffffffu, o[r][e], 16);
      }
    }
  }
  __device__ __forceinline__ void put_ml(float2* ml, int lane, float c2) const {
    if (lane == 0) {
#pragma unroll
      for (int r = 0; r < RB; ++r) ml[r] = make_float2(__fmul_rn(m[r], c2), l[r]);
    }
  }
  __device__ __forceinline__ void scale(const float* f, int) {
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      const float w = f[r];
#pragma unroll
      for (int e = 0; e < 4; ++e) o[r][e] *= w;
    }
  }
  __device__ __forceinline__ void put(float* dst, int lane) const {
    if (lane >= CH) return;
#pragma unroll
    for (int r = 0; r < RB; ++r)
      reinterpret_cast<float4*>(dst)[r * CH + lane] = make_float4(o[r][0], o[r][1], o[r][2], o[r][3]);
  }
  __device__ __forceinline__ void add(const float* src, int lane) {
    if (lane >= CH) return;
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      const float4 v = reinterpret_cast<const float4*>(src)[r * CH + lane];
      o[r][0] += v.x; o[r][1] += v.y; o[r][2] += v.z; o[r][3] += v.w;
    }
  }
  template <typename F>
  __device__ __forceinline__ void each(int lane, F f) const {
    if (lane >= CH) return;
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      f(r, 4 * lane, make_float2(o[r][0], o[r][1]));
      f(r, 4 * lane + 2, make_float2(o[r][2], o[r][3]));
    }
  }
};

// Natural log-sum of a row with reference M and sum L (L = 0: no key; a dot product
// of +infinity makes M that and L NaN).
__device__ __forceinline__ float lse_of(float M, float L) {
  if (M == INFINITY) return M;
  return L > 0.0f ? (M + log2f(L)) * kLn2 : (L != L ? L : -INFINITY);
}

__device__ __forceinline__ void store2(float* p, float2 v) { *reinterpret_cast<float2*>(p) = v; }
__device__ __forceinline__ void store2(__nv_bfloat16* p, float2 v) {
  *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(v.x, v.y);
}

// The end of a cluster CTA, by all its threads: the cluster's states are joined
// (each CTA some of the columns), then each CTA adds its own tokens' masses if
// no other item adds to them (`own_mass`); else the join kernel does, with the
// norms left here.
template <typename T, int D, int RB>
__device__ __forceinline__ void cluster_finish(const DecodeArgs& a, const DecodeWs& ws, char* sm, const Segment& seg,
                                               int cs, bool own_mass) {
  using C = Cfg<T, D, RB>;
  __shared__ float2 s_norm[RB];          // joined (reference, 1 / sum) of each row
  const Shape& s = a.s;
  const float2* s_ml = reinterpret_cast<const float2*>(sm + C::ML_OFF);
  const float2* s_o = reinterpret_cast<const float2*>(sm + C::O_OFF);
  const int tid = threadIdx.x, rank = cs > 1 ? cluster_rank() : 0;
  const int nrb = (s.G + RB - 1) / RB, g = seg.item / nrb, r0 = (seg.item % nrb) * RB, n_rows = min(RB, s.G - r0);
  const size_t row0 = (size_t)seg.b * s.H + g * s.G + r0;
  if (cs > 1) cluster_sync(); else __syncthreads();
  auto state = [&](const float2* p, int k) { return cs > 1 ? peer_float2(p, k) : *p; };
  const int cols = D / 2 / cs;           // pairs of columns of this CTA
  for (int e = tid; e < n_rows * cols; e += kThreads) {
    const int r = e / cols, col = rank * cols + e % cols;
    float2 ml[kMaxCluster], v[kMaxCluster];
#pragma unroll
    for (int k = 0; k < kMaxCluster; ++k) {
      ml[k] = k < cs ? state(s_ml + r, k) : make_float2(-INFINITY, 0.0f);
      v[k] = k < cs ? state(s_o + r * (D / 2) + col, k) : make_float2(0.0f, 0.0f);
    }
    float M = -INFINITY, L = 0.0f;
    float2 o = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < kMaxCluster; ++k) M = max_nan(M, ml[k].x);
#pragma unroll
    for (int k = 0; k < kMaxCluster; ++k) {
      const float f = ml[k].x == -INFINITY ? 0.0f : ex2_approx(ml[k].x - M);
      L = fmaf(ml[k].y, f, L);
      o.x = fmaf(v[k].x, f, o.x);
      o.y = fmaf(v[k].y, f, o.y);
    }
    float inv = L > 0.0f ? 1.0f / L : 0.0f;
    if (L != L) inv = L;
    store2(reinterpret_cast<T*>(a.O) + (row0 + r) * D + 2 * col, make_float2(o.x * inv, o.y * inv));
    if (col == rank * cols) {
      s_norm[r] = make_float2(L == 0.0f ? INFINITY : M, inv);  // no key: weights 2^-inf
      if (rank == 0) {
        if (a.lse) a.lse[row0 + r] = lse_of(M, L);
        if (!own_mass) {
          ws.norm[row0 + r] = s_norm[r];
          if (r == 0) reinterpret_cast<int2*>(ws.runs)[(size_t)seg.b * s.H_kv * nrb + seg.item] = make_int2(0, 0);
        }
      }
    }
  }
  if (cs > 1) cluster_sync(); else __syncthreads();  // no CTA leaves while its state is read
  if (!a.tok_mass || !own_mass) return;
  const float c2 = (float)(s.scale * kLog2e);
  float* mass = a.tok_mass + ((size_t)seg.b * s.H_kv + g) * s.L_ctx;
  using X = typename Logit<T>::Type;
  const X* x = static_cast<const X*>(ws.logit) + row0 * ws.Lp;
  const double c2d = s.scale * kLog2e;
  for (int t = seg.t0 * C::KT + tid; t < min(seg.len, seg.t1 * C::KT); t += kThreads) {
    const float old = a.decay != 0.0f ? mass[t] : 0.0f;
    float sum = 0.0f;
#pragma unroll 4
    for (int r = 0; r < n_rows; ++r)
      sum = fmaf(ex2_approx(Logit<T>::exponent(x[(size_t)r * ws.Lp + t], c2, c2d, s_norm[r].x)), s_norm[r].y, sum);
    mass[t] = a.decay == 0.0f ? sum : fmaf(a.decay, old, sum);
  }
}

// The run of CTA c of `grid`: its part of the counted tiles of all sequences.
// Every warp finds it for itself: a lane counts `per` sequences; the one whose
// count passes the run's first tile has the place.
__device__ __forceinline__ Walk find_run(const DecodeArgs& a, int c, int grid, int ips, int kt, bool report) {
  const Shape& s = a.s;
  const int lane = threadIdx.x & 31;
  const int per = (s.batch + 31) / 32, b0 = min(s.batch, lane * per), b1 = min(s.batch, b0 + per);
  long long mine = 0;
  int n0 = 0;                            // length of sequence b0
#pragma unroll 4
  for (int b = b0; b < b1; ++b) {
    const int n = a.ctx_len[b];
    const bool ok = n >= 0 && n <= s.L_ctx;
    if (!ok && report) flag_error(a.err, ERR_BAD_INDEX);
    const int len = ok ? n : 0;
    if (b == b0) n0 = len;
    mine += seq_cost(len, kt, ips);
  }
  long long before = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += v;
  }
  const long long total = __shfl_sync(0xffffffffu, before, 31);
  before -= mine;
  const int P = (int)min((long long)grid, total);  // runs that hold a tile
  if (c >= P) return Walk(a, ips, kt, 0, 0, 0, 0);
  const long long lo = div_tiles(total * c, P), hi = div_tiles(total * (c + 1), P);
  int wb = b0, wlen = n0;
  long long woff = lo - before;
  const bool here = lo >= before && lo < before + mine;
  if (here && per > 1) {
    for (long long at = before; wb < b1; ++wb) {
      wlen = seq_len(a, wb);
      const long long w = seq_cost(wlen, kt, ips);
      woff = lo - at;
      if (woff < w) break;
      at += w;
    }
  }
  const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
  wb = __shfl_sync(0xffffffffu, wb, src);
  wlen = __shfl_sync(0xffffffffu, wlen, src);
  woff = __shfl_sync(0xffffffffu, woff, src);
  return Walk(a, ips, kt, wb, wlen, woff, hi - lo);
}

// The segment of a cluster CTA: its share of item blockIdx.x / cs.
__device__ __forceinline__ Single find_share(const DecodeArgs& a, int cs, int ips, int kt, bool report) {
  const int id = blockIdx.x / cs, rank = blockIdx.x % cs, b = id / ips, item = id % ips;
  const int n = a.ctx_len[b];
  const bool ok = n >= 0 && n <= a.s.L_ctx;
  if (!ok && report && rank == 0 && item == 0 && (threadIdx.x & 31) == 0) flag_error(a.err, ERR_BAD_INDEX);
  const int len = ok ? n : 0, nt = (len + kt - 1) / kt;
  return Single{Segment{b, item, nt * rank / cs, nt * (rank + 1) / cs, nt, len}, false};
}

// CL: clusters of cs CTAs take one item each; else equal runs.
template <typename T, int D, int RB, bool CL>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
decode_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
              const __grid_constant__ DecodeArgs a, const __grid_constant__ DecodeWs ws, int cs,
              bool own_mass) {
  using C = Cfg<T, D, RB>;
  extern __shared__ char smem_raw[];
  char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + C::BAR_OFF);
  uint64_t* empty = full + C::ST;
  volatile int* info = reinterpret_cast<volatile int*>(sm + C::MISC_OFF);
  volatile int* abort_flag = info + C::ST;
  __shared__ float s_f[kWarps][RB];
  const Shape& s = a.s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nrb = (s.G + RB - 1) / RB, ips = s.H_kv * nrb;
  if (tid == 0) {
    for (int i = 0; i < C::ST; ++i) { mbar_init(full + i, 1); mbar_init(empty + i, kWarps); }
    fence_mbar_init();
    *abort_flag = 0;
  }
  if (warp == kWarps && lane == 0) { prefetch_tmap(&mk); prefetch_tmap(&mv); }
  pdl_wait();
  pdl_trigger();

  auto walk = [&] {
    if constexpr (CL) return find_share(a, cs, ips, C::KT, warp == 0);
    else return find_run(a, blockIdx.x, gridDim.x, ips, C::KT, blockIdx.x == 0 && warp == 0);
  }();
  const int c = blockIdx.x;
  if constexpr (!CL) {
    if (walk.left <= 0) return;          // the whole CTA: fewer tiles than CTAs
  }
  __syncthreads();                       // the barriers are set up
  Segment seg;

  if (warp == kWarps) {
    // ---- copies
    int k = 0, have_b = -1, have_t = 0, slots = 0;
    bool dead = false;
    while (walk.next(&seg)) {
      const int g = seg.item / nrb;
      for (int base = seg.t0; base < seg.t1; base += 32) {
        // 32 tiles' pages at a time; the next KV head of a short sequence reuses them
        if (seg.b != have_b || base < have_t || min(base + 32, seg.t1) > have_t + 32) {
          const int t = base + lane;
          slots = t < seg.nt ? a.page_table[(size_t)seg.b * s.n_pages + (t * C::KT) / 64] : -1;
          have_b = seg.b;
          have_t = base;
        }
        const int n = min(32, seg.t1 - base);
        for (int j = 0; j < n; ++j, ++k) {
          const int slot = __shfl_sync(0xffffffffu, slots, base - have_t + j);
          if (lane != 0) continue;
          const int st = k % C::ST;
          if (!dead && k >= C::ST) dead = !mbar_wait(empty + st, (k / C::ST - 1) & 1, abort_flag);
          if (dead) continue;
          const int tile = base + j;
          if (slot < 0 || slot >= s.n_slots) {
            flag_error(a.err, ERR_BAD_INDEX);
            info[st] = 0;
            mbar_arrive(full + st);
            continue;
          }
          info[st] = min(C::KT, seg.len - tile * C::KT);
          mbar_arrive_expect_tx(full + st, C::STAGE);
          const int y = (slot * s.H_kv + g) * 64 + (tile * C::KT) % 64;
          char* dst = sm + st * C::STAGE;
#pragma unroll
          for (int x = 0; x < C::BOXES; ++x) {
            tma_load_2d(dst + x * C::BOX, &mk, x * (128 / (int)sizeof(T)), y, full + st);
            tma_load_2d(dst + C::HALF + x * C::BOX, &mv, x * (128 / (int)sizeof(T)), y, full + st);
          }
        }
      }
    }
    if (lane == 0 && *abort_flag) {  // gave up: wait (bounded) for the copies in flight
      flag_error(a.err, ERR_TIMEOUT);
      for (int i = max(0, k - C::ST); i < k; ++i)
        for (uint32_t n = 0; n < 4096 && !mbar_try_wait(full + i % C::ST, (i / C::ST) & 1); ++n) {}
    }
    __syncwarp();
    if constexpr (!CL) return;
  }

  // ---- computing warps
  using State = typename std::conditional<C::BF16, StateTc<D, RB>, StateF32<D, RB, C::KT>>::type;
  State st8;
  float* s_o = reinterpret_cast<float*>(sm + C::O_OFF);
  float2* s_ml = reinterpret_cast<float2*>(sm + C::ML_OFF);
  const float c2 = (float)(s.scale * kLog2e);
  int k = 0;
  bool dead = false;
  while ((!CL || warp < kWarps) && walk.next(&seg)) {
    const int g = seg.item / nrb, r0 = (seg.item % nrb) * RB, n_rows = min(RB, s.G - r0);
    const size_t row0 = (size_t)seg.b * s.H + g * s.G + r0;  // the block's first (b, h)
    const T* q = reinterpret_cast<const T*>(a.Q) + row0 * D;
    if constexpr (C::BF16) {
      st8.load_q(q, n_rows, lane);
    } else {
      double* sq = reinterpret_cast<double*>(sm + C::Q_OFF);
      named_bar_sync(1, kWarps * 32);  // the last segment's rows are no longer read
      for (int e = tid; e < RB * D; e += kWarps * 32)
        sq[State::q_at(e / D, e % D)] = e < n_rows * D ? (double)q[e] : 0.0;
      named_bar_sync(1, kWarps * 32);
      st8.sq = sq;
      st8.sp = reinterpret_cast<float*>(sm + C::P_OFF) + warp * RB * State::NKW;
    }
    st8.reset();
    for (int t = seg.t0; t < seg.t1; ++t, ++k) {
      const int st = k % C::ST;
      if (!dead) dead = !mbar_wait(full + st, (k / C::ST) & 1, abort_flag);
      if (__any_sync(0xffffffffu, dead)) { dead = true; continue; }
      const int valid = info[st];
      using X = typename Logit<T>::Type;
      X* logit = a.tok_mass ? static_cast<X*>(ws.logit) + row0 * ws.Lp + (size_t)t * C::KT : nullptr;
      if constexpr (C::BF16) {
        const uint32_t ks = smem_u32(sm + st * C::STAGE);
        st8.tile(ks, ks + C::HALF, warp, lane, valid, c2, logit, ws.Lp, n_rows);
      } else {
        const char* ks = sm + st * C::STAGE;
        st8.tile(ks, ks + C::HALF, warp, lane, valid, c2, s.scale * kLog2e, logit, ws.Lp, n_rows);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + st);
    }
    // segment end: the four warps' states, added in warp order
    st8.finish(lane);
    st8.put_ml(s_ml + warp * RB, lane, c2);
    named_bar_sync(1, kWarps * 32);
    if (lane < RB) {
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = max_nan(M, s_ml[w * RB + lane].x);
      const float own = s_ml[warp * RB + lane].x;
      s_f[warp][lane] = own == -INFINITY ? 0.0f : ex2_approx(own - M);
    }
    __syncwarp();
    st8.scale(s_f[warp], lane);
    float M = -INFINITY, L = 0.0f;  // row `lane`, on warp 0
    if (warp == 0 && lane < RB) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = max_nan(M, s_ml[w * RB + lane].x);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 v = s_ml[w * RB + lane];
        if (v.x != -INFINITY) L = fmaf(v.y, ex2_approx(v.x - M), L);
      }
    }
#pragma unroll
    for (int w0 = 1; w0 < kWarps; w0 += C::COPIES) {
      if (warp >= w0 && warp < w0 + C::COPIES) st8.put(s_o + (warp - w0) * RB * D, lane);
      named_bar_sync(1, kWarps * 32);
      if (warp == 0) {
#pragma unroll
        for (int w = 0; w < C::COPIES; ++w) st8.add(s_o + w * RB * D, lane);
      }
      if (w0 + C::COPIES < kWarps) named_bar_sync(1, kWarps * 32);
    }
    if constexpr (CL) {                  // this CTA's state, for the cluster
      if (warp == 0) {
        if (lane < RB) s_ml[lane] = make_float2(M, L);
        __syncwarp();
        st8.each(lane, [&](int r, int col, float2 v) { store2(s_o + r * D + col, v); });
      }
      continue;
    }
    if (warp != 0) continue;
    if (lane == 0) {                     // for the join kernel
      int* runs = ws.runs + ((size_t)seg.b * ips + seg.item) * 2;
      if (seg.t0 == 0) runs[0] = c;
      if (seg.t1 == seg.nt) runs[1] = c;
    }
    if (seg.t0 == 0 && seg.t1 == seg.nt) {
      float inv = L > 0.0f ? 1.0f / L : 0.0f;
      if (L != L) inv = L;
      if (lane < n_rows) {
        ws.norm[row0 + lane] = make_float2(L == 0.0f ? INFINITY : M, inv);  // no key: weights 2^-inf
        if (a.lse) a.lse[row0 + lane] = lse_of(M, L);
      }
      T* O = reinterpret_cast<T*>(a.O) + row0 * D;
      __syncwarp();
      if (lane < RB) s_f[0][lane] = inv;
      __syncwarp();
      st8.each(lane, [&](int r, int col, float2 v) {
        const float f = s_f[0][r];
        if (r < n_rows) store2(O + (size_t)r * D + col, make_float2(v.x * f, v.y * f));
      });
    } else {
      const int slot = 2 * c + (seg.t0 == 0 ? 1 : 0);
      if (lane < n_rows) ws.pml[(size_t)slot * RB + lane] = make_float2(M, L);
      float* po = ws.po + (size_t)slot * RB * D;
      st8.each(lane, [&](int r, int col, float2 v) {
        if (r < n_rows) store2(po + (size_t)r * D + col, v);
      });
    }
  }
  if constexpr (CL) cluster_finish<T, D, RB>(a, ws, sm, walk.seg, cs, own_mass);
}

// The partials of one item: runs c0..c0 + n - 1 and their slots.
struct Parts {
  int c0, n, r;  // first run, number of runs, row in the block
  __device__ __forceinline__ int slot(int i) const { return 2 * (c0 + i) + (i == 0 ? 1 : 0); }
};
__device__ __forceinline__ Parts parts_of(const DecodeArgs& a, const DecodeWs& ws, int b, int h, int rb) {
  const Shape& s = a.s;
  const int g = h / s.G, nrb = (s.G + rb - 1) / rb, r = h % s.G;
  const int2 runs = reinterpret_cast<const int2*>(ws.runs)[(size_t)b * s.H_kv * nrb + g * nrb + r / rb];
  return Parts{runs.x, runs.y - runs.x + 1, r % rb};
}

// Reference and inverse sum of one query row over its runs, by one warp.  A
// row finished by its run has them in the workspace.
__device__ __forceinline__ float2 row_norm(const DecodeArgs& a, const DecodeWs& ws, const Parts& p, size_t row,
                                           int rb, int lane) {
  if (p.n == 1) return ws.norm[row];
  float M = -INFINITY, L = 0.0f;
#pragma unroll 3
  for (int i = lane; i < p.n; i += 32) {
    const float2 v = ws.pml[(size_t)p.slot(i) * rb + p.r];
    const float m = max_nan(M, v.x);
    if (m != -INFINITY) {
      L = L * ex2_approx(M - m) + v.y * ex2_approx(v.x - m);
      M = m;
    }
  }
  const float top = warp_max_nan(M);
  L = warp_sum(top == -INFINITY ? L : L * ex2_approx(M - top));
  return L == 0.0f ? make_float2(INFINITY, 0.0f) : make_float2(top, 1.0f / L);
}

// CTA `id` of the masses: one of `chunks` of a decision row.  A thread has
// eight logits in flight, of 8 / QR tokens and QR rows.
template <typename T, int QR>
__device__ __forceinline__ void add_masses(const DecodeArgs& a, const DecodeWs& ws, int rb, int id,
                                           int chunks) {
  using X = typename Logit<T>::Type;
  constexpr int NW = kJoinThreads / 32, TJ = 8 / QR;
  __shared__ float2 s_norm[64];          // 64 rows at a time
  const Shape& s = a.s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bm = id / chunks, b = bm / a.n_mass, m = bm % a.n_mass;
  const int rows = s.H / a.n_mass, h0 = m * rows;
  const int first = (id % chunks) * TJ * kJoinThreads, step = chunks * TJ * kJoinThreads;
  float* mass = a.tok_mass + ((size_t)b * a.n_mass + m) * s.L_ctx;
  const double c2d = s.scale * kLog2e;
  const float c2 = (float)c2d;
  pdl_wait();
  const int n = seq_len(a, b);
  if (first >= n) return;
#pragma unroll 1
  for (int r0 = 0; r0 < rows; r0 += 64) {
    const int nr = min(64, rows - r0);
    const float decay = r0 == 0 ? a.decay : 1.0f;
    const X* x = static_cast<const X*>(ws.logit) + ((size_t)b * s.H + h0 + r0) * ws.Lp;
    bool sums = false;
#pragma unroll 1
    for (int t0 = first; t0 < n; t0 += step) {
      float old[TJ], sum[TJ];
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        old[j] = decay != 0.0f ? mass[min(t0 + tid + j * kJoinThreads, n - 1)] : 0.0f;
        sum[j] = 0.0f;
      }
#pragma unroll 1
      for (int q0 = 0; q0 < nr; q0 += QR) {
        X v[QR][TJ];
#pragma unroll
        for (int q = 0; q < QR; ++q)
#pragma unroll
          for (int j = 0; j < TJ; ++j)
            v[q][j] = x[(size_t)min(q0 + q, nr - 1) * ws.Lp + min(t0 + tid + j * kJoinThreads, n - 1)];
        if (!sums) {
          sums = true;
          __syncthreads();
          for (int r = warp; r < nr; r += NW) {
            const float2 norm = row_norm(a, ws, parts_of(a, ws, b, h0 + r0 + r, rb),
                                         (size_t)b * s.H + h0 + r0 + r, rb, lane);
            if (lane == 0) s_norm[r] = norm;
          }
          __syncthreads();
        }
#pragma unroll
        for (int q = 0; q < QR; ++q) {
          if (q0 + q >= nr) continue;
          const float2 norm = s_norm[q0 + q];
#pragma unroll
          for (int j = 0; j < TJ; ++j) sum[j] = fmaf(ex2_approx(Logit<T>::exponent(v[q][j], c2, c2d, norm.x)), norm.y, sum[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        const int t = t0 + tid + j * kJoinThreads;
        if (t < n) mass[t] = decay == 0.0f ? sum[j] : fmaf(decay, old[j], sum[j]);
      }
    }
  }
}

// The last CTAs: join the partials of query rows (or write an empty sequence's
// rows), rpc rows each.  Those before them, which take longer: masses, `chunks`
// CTAs a decision row.
// Bound by latency: chains of dependent loads, and the first fetch of the
// code, so loops are short rather than unrolled.  Nothing is read before the wait,
// the lengths least of all: an append two kernels ahead may have written them, and
// only the wait orders that write before this grid's reads.  Each chain's bulk loads
// (partial outputs, logits) are issued ahead of the weights they wait for.
template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads, 4)
decode_join_kernel(const __grid_constant__ DecodeArgs a, const __grid_constant__ DecodeWs ws, int rb,
                   int chunks, int rpc) {
  const Shape& s = a.s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int NW = kJoinThreads / 32;
  pdl_trigger();
  const int mass_ctas = s.batch * a.n_mass * chunks;
  if ((int)blockIdx.x >= mass_ctas) {
    __shared__ float s_m[NW], s_l[NW], s_w[kMaxCtas];
    __shared__ float4 s_o[kJoinThreads];
    constexpr int CH = D / 4, GR = kJoinThreads / CH, U = 5;
    const int col = tid % CH, grp = tid / CH;  // thread = (run group, four columns)
    // a warp looks up a row each
    __shared__ Parts s_parts[NW];
    const int row0 = (blockIdx.x - mass_ctas) * rpc, rows = min(rpc, s.batch * s.H - row0);
    pdl_wait();
    if (warp < rows && lane == 0) {
      const int b = (row0 + warp) / s.H;
      const Parts p = parts_of(a, ws, b, (row0 + warp) % s.H, rb);  // of an empty sequence: anything
      s_parts[warp] = seq_len(a, b) > 0 ? p : Parts{0, 0, 0};
    }
    __syncthreads();
#pragma unroll 1
    for (int w = 0; w < rows; ++w) {
      const int row = row0 + w;
      const Parts p = s_parts[w];
      if (p.n == 1) continue;  // finished by its run
      const float4* po = reinterpret_cast<const float4*>(ws.po) + (size_t)p.r * CH + col;
      float4 v[U], o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float M = -INFINITY, L = 0.0f;
#pragma unroll 1
      for (int i0 = grp; i0 - grp < p.n; i0 += U * GR) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = min(i0 + u * GR, p.n - 1);  // the last run again, with no weight
          v[u] = po[(size_t)p.slot(i) * rb * CH];
        }
        if (i0 == grp) {  // the runs' weights 2^(m - M)
          constexpr int N = (kMaxCtas + kJoinThreads - 1) / kJoinThreads;
          float2 ml[N];
#pragma unroll
          for (int q = 0; q < N; ++q) {
            const int i = tid + q * kJoinThreads;
            ml[q] = i < p.n ? ws.pml[(size_t)p.slot(i) * rb + p.r] : make_float2(-INFINITY, 0.0f);
            M = max_nan(M, ml[q].x);
          }
          M = warp_max_nan(M);
          if (lane == 0) s_m[warp] = M;
          __syncthreads();
          M = warp_max_nan(s_m[lane % NW]);
#pragma unroll
          for (int q = 0; q < N; ++q) {
            const int i = tid + q * kJoinThreads;
            const float f = ml[q].x == -INFINITY ? 0.0f : ex2_approx(ml[q].x - M);
            if (i < p.n) s_w[i] = f;
            L = fmaf(ml[q].y, f, L);
          }
          L = warp_sum(L);
          if (lane == 0) s_l[warp] = L;
          __syncthreads();
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float f = i0 + u * GR < p.n ? s_w[i0 + u * GR] : 0.0f;
          if (i0 + u * GR >= p.n) continue;
          o.x = fmaf(f, v[u].x, o.x); o.y = fmaf(f, v[u].y, o.y);
          o.z = fmaf(f, v[u].z, o.z); o.w = fmaf(f, v[u].w, o.w);
        }
      }
      s_o[tid] = o;
      __syncthreads();
      if (tid < CH) {
        L = 0.0f;
        if (p.n > 0) {
#pragma unroll 1
          for (int i = 0; i < NW; ++i) L += s_l[i];
#pragma unroll 1
          for (int i = 1; i < GR; ++i) {
            const float4 x = s_o[i * CH + tid];
            o.x += x.x; o.y += x.y; o.z += x.z; o.w += x.w;
          }
        }
        float inv = L > 0.0f ? 1.0f / L : 0.0f;
        if (L != L) inv = L;
        T* dst = reinterpret_cast<T*>(a.O) + (size_t)row * D + 4 * tid;
        store2(dst, make_float2(o.x * inv, o.y * inv));
        store2(dst + 2, make_float2(o.z * inv, o.w * inv));
        if (tid == 0 && a.lse) a.lse[row] = lse_of(M, L);
      }
      __syncthreads();                   // the next row writes what this one reads
    }
    return;
  }
  // ---- masses
  const int id = blockIdx.x, rows = s.H / a.n_mass;
  if (rows > 4) add_masses<T, 8>(a, ws, rb, id, chunks);
  else if (rows > 2) add_masses<T, 4>(a, ws, rb, id, chunks);
  else if (rows > 1) add_masses<T, 2>(a, ws, rb, id, chunks);
  else add_masses<T, 1>(a, ws, rb, id, chunks);
}

template <typename T, int D, int RB>
cudaError_t run_decode(const DecodeArgs& a, cudaStream_t st) {
  using C = Cfg<T, D, RB>;
  const Shape& s = a.s;
  DecodeWs w;
  carve(s, a.tok_mass != nullptr, a.ws, &w);
  const uint64_t rows = (uint64_t)s.n_slots * s.H_kv * 64;
  CUtensorMap mk, mv;
  const bool ok = C::BF16 ? tc_map_2d(&mk, a.Kp, D, rows, C::KT) && tc_map_2d(&mv, a.Vp, D, rows, C::KT)
                          : tc_map_f32_2d(&mk, a.Kp, D, rows, C::KT) &&
                                tc_map_f32_2d(&mv, a.Vp, D, rows, C::KT);
  if (!ok) return cudaErrorInvalidValue;
  const int tiles = (s.L_ctx + C::KT - 1) / C::KT, fit = kCtasPerSm * tc_sm_count();
  const long long items = (long long)s.batch * items_per_seq(s);
  // Small enough for clusters, all resident at once?  (8 heads on one, 2400 tokens,
  // 71 clusters of four fit: 71 items 28.5 us, as runs 32.0; 72 items 36.2 and 30.0.)
  int cs = 1;
  auto all_fit = [&](int n) {
    return items * n <= fit && items <= resident_clusters<decode_kernel<T, D, RB, true>>(n, kThreads, C::SMEM);
  };
  while (cs < kMaxCluster && cs < tiles && all_fit(2 * cs)) cs *= 2;
  const bool clusters = items * cs <= fit &&
                        tiles <= cs * (4 * items * cs >= 3 * fit ? kClusterTilesFull : kClusterTiles);
  const bool own_mass = !a.tok_mass || (a.n_mass == s.H_kv && s.G <= RB);
  if (clusters) {
    cudaError_t e = allow_smem<decode_kernel<T, D, RB, true>>(C::SMEM);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(items * cs));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0] = cluster_of(cs);
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, decode_kernel<T, D, RB, true>, mk, mv, a, w, cs, own_mass);
    if (e != cudaSuccess || own_mass) return e;
  } else {
    cudaError_t e = allow_smem<decode_kernel<T, D, RB, false>>(C::SMEM);
    if (e != cudaSuccess) return e;
    const long long most = items * tiles;
    int P = fit < kMaxCtas ? fit : kMaxCtas;
    P = (int)(most < P ? (most > 0 ? most : 1) : P);
    auto kern = decode_kernel<T, D, RB, false>;
    DL_LAUNCH_DEPENDENT(kern, P, kThreads, C::SMEM, st, mk, mv, a, w, 0, false);
  }
  // masses: three batches of loads a thread, which share the join's first 3 us
  // (32 x 8K ragged, 1 / 2 / 3 batches: 63.1 / 60.9 / 60.3 us), fewer while that
  // leaves SMs idle
  int chunks = 0;
  if (a.tok_mass && s.L_ctx > 0) {
    const int rows = s.H / a.n_mass, tj = rows > 4 ? 1 : rows > 2 ? 2 : rows > 1 ? 4 : 8;
    const int dec = s.batch * a.n_mass, idle = (4 * tc_sm_count() + dec - 1) / dec;
    const int most = (s.L_ctx + kJoinThreads * tj - 1) / (kJoinThreads * tj);
    const int few = (s.L_ctx + 3 * kJoinThreads * tj - 1) / (3 * kJoinThreads * tj);
    chunks = idle > few ? idle : few;
    chunks = chunks < most ? chunks : most;
    chunks = chunks < 4096 ? chunks : 4096;
  }
  auto join = decode_join_kernel<T, D>;
  // a row a CTA up to two waves, then up to eight: of many rows most are
  // finished by their runs (32 sequences x 512 heads, lengths up to 64: the call
  // takes 43.4 us with a row a CTA, 25.4 with eight)
  const int all_rows = s.batch * s.H, once = 8 * tc_sm_count();
  const int rpc = (all_rows + once - 1) / once < 8 ? (all_rows + once - 1) / once : 8;  // 8: a warp each
  DL_LAUNCH_DEPENDENT(join, (all_rows + rpc - 1) / rpc + s.batch * a.n_mass * chunks, kJoinThreads, 0, st, a, w, RB,
                      chunks, rpc);
  return cudaGetLastError();
}

}  // namespace

size_t decode_workspace(const Shape& s, bool mass) { return carve(s, mass, nullptr, nullptr); }

namespace {

template <int D>
cudaError_t run_decode_f32(const DecodeArgs& a, cudaStream_t st) {
  const int rb = rows_per_block(a.s);
  if (rb == 8) return run_decode<float, D, 8>(a, st);
  return rb == 4 ? run_decode<float, D, 4>(a, st) : run_decode<float, D, 2>(a, st);
}

}  // namespace

cudaError_t launch_decode_attn(const DecodeArgs& a, cudaStream_t st) {
  const Shape& s = a.s;
  if (s.dtype == DL_BF16) {
    if (s.d == 128)
      return s.G > 8 ? run_decode<__nv_bfloat16, 128, 16>(a, st) : run_decode<__nv_bfloat16, 128, 8>(a, st);
    return s.G > 8 ? run_decode<__nv_bfloat16, 64, 16>(a, st) : run_decode<__nv_bfloat16, 64, 8>(a, st);
  }
  return s.d == 128 ? run_decode_f32<128>(a, st) : run_decode_f32<64>(a, st);
}

}  // namespace dl
