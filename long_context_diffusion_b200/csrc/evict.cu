// (c3) The eviction plan of a cache with a budget, and (c4) its moves.
//
// Plan: the `budget` tokens of largest key stay, key = the accumulated mass
// in the order of its bits (held tokens at +infinity, NaN at -infinity),
// equal keys by the lower index.
//
// Bound: latency (a row of n tokens is 8 n bytes; 128 rows of 32K, 38 MB, are
// 6 us of HBM).  A decision row is taken by a cluster of 1 to 8 CTAs that
// splits its n tokens evenly in index order and keeps their keys in shared
// memory, so that masses and positions are read once; a warp owns 32 it
// consecutive tokens, lane l of iteration j having token 32 j + l.
//  - The budget-th key by radix select: a histogram of the top 12 bits (sign,
//    exponent, three bits of mantissa), then of the next 10 and the last 10
//    among the keys that share the digits found.  Each CTA counts its own
//    tokens and sums its bins by groups of 32; every CTA then adds the groups'
//    sums over the cluster, finds the group, and adds that group's 32 bins
//    alone (adding all bins over the cluster took four times as long).  The
//    search ends at the first digit whose whole bin stays.
//  - One vote per iteration gives the 32 tokens' keep bits as a word, lane j
//    holding iteration j's; holes and fills are then counted and listed by
//    words, with prefix sums over lanes, warps and CTAs.
// Rows too long for the cluster's shared memory (KEEP false) recompute their
// keys from memory in every pass.
//
// Moves: bound by HBM (each moved row is read and written once).  A warp
// resolves 32 moves at a time, one per lane, then all lanes copy their rows in
// 16-byte pieces, eight loads ahead of the stores.
#include "common.cuh"
#include "internal.h"
#include "launch.cuh"
#include "tc_common.cuh"

namespace dl {

namespace {

constexpr int kEvThreads = 1024;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kKeepTokens = 48;          // most tokens of a thread kept in shared memory (192 KB)
constexpr unsigned kHeldKey = 0xFF800000u;  // the key of +infinity

// Order-preserving bits of a mass: a < b as numbers <=> key(a) < key(b);
// -0 like +0, NaN like -infinity.  No key is 0, which marks "no token".
__device__ __forceinline__ unsigned mass_key(float x) {
  if (x != x) x = -INFINITY;
  const unsigned u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Value at the same shared-memory place of CTA `rank` of the cluster.
__device__ __forceinline__ int peer_int(const int* p, unsigned rank) {
  const unsigned here = static_cast<unsigned>(__cvta_generic_to_shared(p));
  unsigned there;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(here), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(there) : "memory");
  return v;
}
__device__ __forceinline__ int warp_inclusive(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// KEEP: keys in shared memory; else recomputed from memory.
template <bool KEEP>
__global__ void __launch_bounds__(kEvThreads, 1)
evict_select_kernel(const __grid_constant__ EvictArgs a, int cs) {
  extern __shared__ unsigned s_key[];
  __shared__ __align__(16) int s_hist[4096 + 2 * 1024];
  __shared__ int s_group[3][128];        // this CTA's counts of 32 bins
  __shared__ int s_gsum[128], s_bsum[32];  // the cluster's
  __shared__ int s_wt[3][kEvWarps];      // per warp: ties, holes, fills
  __shared__ int s_ct[4];                // this CTA's: largest position, ties, holes, fills
  __shared__ int s_max[kEvWarps];
  const Shape& s = a.s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = cs > 1 ? (int)cluster_rank() : 0;
  const int row = blockIdx.x / cs, b = row / a.n_mass;
  pdl_trigger();
  pdl_wait();
  const int n = a.ctx_len[b];
  for (int i = tid; i < 4096 + 2 * 1024; i += kEvThreads) s_hist[i] = 0;
  const bool bad = n < 0 || n > s.L_ctx;
  if (tid == 0 && rank == 0 && row % a.n_mass == 0) {
    if (bad) flag_error(a.err, ERR_BAD_INDEX);
    a.new_len[b] = bad ? n : min(n, a.budget);
  }
  int32_t* hole = a.hole_idx + (size_t)row * a.max_move;
  int32_t* fill = a.fill_idx + (size_t)row * a.max_move;
  int moves = 0;
  if (!bad && n > a.budget) {            // the same for the whole cluster
    const float* mass = a.tok_mass + (size_t)row * s.L_ctx;
    const int32_t* pos = a.tok_pos ? a.tok_pos + (size_t)row * s.L_ctx : nullptr;
    // this warp's tokens [w0, w0 + 32 it) (those below n exist); 64-bit: the
    // last warps' may lie past 2^31
    const int it = (int)(((long long)n + cs * kEvThreads - 1) / (cs * kEvThreads));
    const long long w0 = ((long long)rank * kEvWarps + warp) * 32 * it;
    const int live = (int)max(0ll, min((long long)it, ((long long)n - w0 + 31) / 32));  // iterations
    unsigned* keys = s_key + warp * 32 * it + lane;
    // Loads are unconditional (indices clamped to the row), so that a thread's
    // are all in flight together; the first masses do not wait for the largest
    // position.
    constexpr int U = 8;
    auto index = [&](int j) { return (int)min(w0 + 32 * j + lane, (long long)n - 1); };
    float m0[U];
#pragma unroll
    for (int u = 0; u < U; ++u) m0[u] = mass[index(u)];
    int last = INT32_MIN;
    for (int j0 = 0; j0 < live; j0 += U) {
      int p[U];
#pragma unroll
      for (int u = 0; u < U; ++u) p[u] = pos ? pos[index(j0 + u)] : index(j0 + u);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        last = max(last, p[u]);          // a clamped index repeats a token of the row
        if (KEEP && j0 + u < live) keys[32 * (j0 + u)] = (unsigned)p[u];
      }
    }
    last = __reduce_max_sync(0xffffffffu, last);
    if (lane == 0) s_max[warp] = last;
    __syncthreads();
    last = __reduce_max_sync(0xffffffffu, s_max[lane]);
    if (cs > 1) {
      if (tid == 0) s_ct[0] = last;
      cluster_sync();
      last = __reduce_max_sync(0xffffffffu, lane < cs ? peer_int(&s_ct[0], lane) : INT32_MIN);
    }
    const long long recent = (long long)last - a.n_recent;
    auto key_of = [&](long long t, int p, float m) {
      return t >= n ? 0u : (p < a.n_first || p > recent) ? kHeldKey : mass_key(m);
    };
    if (KEEP) {
#pragma unroll 1
      for (int j0 = 0; j0 < live; j0 += U) {
        if (j0 > 0) {
#pragma unroll
          for (int u = 0; u < U; ++u) m0[u] = mass[index(j0 + u)];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int j = j0 + u;
          if (j < live) keys[32 * j] = key_of(w0 + 32 * j + lane, (int)keys[32 * j], m0[u]);
        }
      }
    }
    // key of iteration j (0: no token)
    auto get = [&](int j) -> unsigned {
      if (KEEP) return keys[32 * j];
      const int t = index(j);
      return key_of(w0 + 32 * j + lane, pos ? pos[t] : t, mass[t]);
    };

    // ---- the budget-th key
    unsigned thr = 0;
    int want = a.budget;
    bool whole = false;                  // every key of the last bin stays
#pragma unroll 1
    for (int pass = 0; pass < 3 && !whole; ++pass) {
      const int sh = pass == 0 ? 20 : pass == 1 ? 10 : 0, groups = pass == 0 ? 128 : 32;
      int* hist = s_hist + (pass == 0 ? 0 : 4096 + (pass - 1) * 1024);
      if (pass == 0) {
#pragma unroll 4
        for (int j = 0; j < live; ++j) {
          const unsigned u = get(j), bin = u >> 20;
          // many equal masses (zeros): one count for the warp
          const unsigned first = __shfl_sync(0xffffffffu, bin, 0);
          if (__all_sync(0xffffffffu, bin == first && u != 0u)) {
            if (lane == 0) atomicAdd(&hist[bin], 32);
          } else if (u != 0u) {
            atomicAdd(&hist[bin], 1);
          }
        }
      } else {
        const unsigned above = thr >> (sh + 10);
#pragma unroll 4
        for (int j = 0; j < live; ++j) {
          const unsigned u = get(j);
          if (u != 0u && (u >> (sh + 10)) == above) atomicAdd(&hist[(u >> sh) & 1023u], 1);
        }
      }
      __syncthreads();
      if (tid < groups * 8) {            // eight lanes a group
        const int4 v = reinterpret_cast<const int4*>(hist)[tid];
        int c = (v.x + v.y) + (v.z + v.w);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
        if ((lane & 7) == 0) s_group[pass][tid >> 3] = c;
      }
      if (cs > 1) cluster_sync(); else __syncthreads();
      if (cs > 1) {
        if (tid < groups * 8) {          // lane & 7 = rank
          int c = (lane & 7) < cs ? peer_int(&s_group[pass][tid >> 3], lane & 7) : 0;
#pragma unroll
          for (int o = 4; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
          if ((lane & 7) == 0) s_gsum[tid >> 3] = c;
        }
        __syncthreads();
      }
      // every warp for itself: the group, counted from the top
      const int* gs = cs > 1 ? s_gsum : s_group[pass];
      int c[4] = {0, 0, 0, 0}, group = 0, before = 0;
      const int per = groups / 32, top = groups - 1 - per * lane;  // this lane's first group
      for (int q = 0; q < per; ++q) c[q] = gs[top - q];
      const int mine = (c[0] + c[1]) + (c[2] + c[3]), upto = warp_inclusive(mine, lane);
      {
        const unsigned hit = __ballot_sync(0xffffffffu, upto >= want);  // not empty: want of them exist
        const int l = __ffs(hit) - 1;
        int q = 0, at = upto - mine;
        while (q < per - 1 && at + c[q] < want) at += c[q++];
        group = __shfl_sync(0xffffffffu, top - q, l);
        before = __shfl_sync(0xffffffffu, at, l);
      }
      // its 32 bins
      if (cs > 1) {
        if (tid < 256) {
          int v = (lane & 7) < cs ? peer_int(&hist[group * 32 + (tid >> 3)], lane & 7) : 0;
#pragma unroll
          for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
          if ((lane & 7) == 0) s_bsum[tid >> 3] = v;
        }
        __syncthreads();
      }
      const int v = cs > 1 ? s_bsum[31 - lane] : hist[group * 32 + 31 - lane];
      const int sum = before + warp_inclusive(v, lane);
      const int l = __ffs(__ballot_sync(0xffffffffu, sum >= want)) - 1;
      thr |= (unsigned)(group * 32 + 31 - l) << sh;
      const int upper = __shfl_sync(0xffffffffu, sum, l);
      want -= upper - __shfl_sync(0xffffffffu, v, l);
      whole = want == __shfl_sync(0xffffffffu, v, l);
    }

    // ---- keep words; equal keys beyond `want` leave from the highest index down
    int tie_left = 0;                    // equal keys that may stay, from this warp on
    if (!whole) {
      int ties = 0;
      for (int j = 0; j < live; ++j) ties += __popc(__ballot_sync(0xffffffffu, get(j) == thr));
      if (lane == 0) s_wt[0][warp] = ties;
      __syncthreads();
      const int t = s_wt[0][lane];
      int before = __reduce_add_sync(0xffffffffu, lane < warp ? t : 0);
      if (cs > 1) {
        const int all = __reduce_add_sync(0xffffffffu, t);
        if (tid == 0) s_ct[1] = all;
        cluster_sync();
        before += __reduce_add_sync(0xffffffffu, lane < rank ? peer_int(&s_ct[1], lane) : 0);
      }
      tie_left = max(0, want - before);
    }
    // this lane's word of iterations j0 .. j0 + 31: bit i = token w0 + 32 (j0 + lane) + i
    int tie_run = tie_left;
    auto keep_word = [&](int j0) {
      const int nj = min(32, live - j0);
      unsigned w = 0u, tw = 0u;
#pragma unroll 4
      for (int j = 0; j < nj; ++j) {
        const unsigned u = get(j0 + j);
        const unsigned kw = __ballot_sync(0xffffffffu, whole ? u >= thr : u > thr);
        if (lane == j) w = kw;
        if (!whole) {
          const unsigned e = __ballot_sync(0xffffffffu, u == thr);
          if (lane == j) tw = e;
        }
      }
      if (!whole) {
        const int c = __popc(tw), upto = warp_inclusive(c, lane);
        const int stay = min(c, max(0, tie_run - (upto - c)));
        tie_run = max(0, tie_run - __shfl_sync(0xffffffffu, upto, 31));
        for (int drop = c - stay; drop > 0; --drop) tw &= ~(0x80000000u >> __clz(tw));
        w |= tw;
      }
      return w;
    };
    // this lane's tokens before the budget, as a mask
    auto front_word = [&](int j0) {
      const long long m = j0 + lane < live ? a.budget - (w0 + 32 * (j0 + lane)) : 0;
      return m <= 0 ? 0u : m >= 32 ? 0xffffffffu : (1u << (int)m) - 1u;
    };
    unsigned word = 0u;
    int holes = 0, fills = 0;
    for (int j0 = 0; j0 < live; j0 += 32) {
      word = keep_word(j0);
      const unsigned front = front_word(j0);
      holes += __popc(~word & front);    // budget < n: every token before it exists
      fills += __popc(word & ~front);
    }
    holes = __reduce_add_sync(0xffffffffu, holes);
    fills = __reduce_add_sync(0xffffffffu, fills);
    if (lane == 0) { s_wt[1][warp] = holes; s_wt[2][warp] = fills; }
    __syncthreads();
    const int th = s_wt[1][lane], tf = s_wt[2][lane];
    int hole_at = __reduce_add_sync(0xffffffffu, lane < warp ? th : 0);
    int fill_at = __reduce_add_sync(0xffffffffu, lane < warp ? tf : 0);
    moves = __reduce_add_sync(0xffffffffu, tf);
    if (cs > 1) {
      const int all_h = __reduce_add_sync(0xffffffffu, th);
      if (tid == 0) { s_ct[2] = all_h; s_ct[3] = moves; }
      cluster_sync();
      const int f = lane < cs ? peer_int(&s_ct[3], lane) : 0;
      const int h = lane < rank ? peer_int(&s_ct[2], lane) : 0;
      moves = __reduce_add_sync(0xffffffffu, f);
      hole_at += __reduce_add_sync(0xffffffffu, h);
      fill_at += __reduce_add_sync(0xffffffffu, lane < rank ? f : 0);
    }
    tie_run = tie_left;
    // Lists the set bits of the lanes' words in order, from list[at] on: word
    // by word, so that neighbours are written together, or each lane its own
    // when no word is crowded.
    auto list = [&](unsigned w, int32_t* out, int at, int j0) {
      const int c = __popc(w), upto = warp_inclusive(c, lane);
      if (__reduce_max_sync(0xffffffffu, c) <= 12) {
        int32_t* o = out + at + upto - c;
        const int t0 = (int)(w0 + 32 * (j0 + lane));
        for (; w; w &= w - 1) *o++ = t0 + __ffs(w) - 1;
      } else {
        const unsigned bit = 1u << lane;
        for (unsigned some = __ballot_sync(0xffffffffu, w != 0u); some; some &= some - 1) {
          const int j = __ffs(some) - 1;
          const unsigned v = __shfl_sync(0xffffffffu, w, j);
          const int o = at + __shfl_sync(0xffffffffu, upto - c, j);
          if (v & bit) out[o + __popc(v & (bit - 1))] = (int)(w0 + 32 * (j0 + j)) + lane;
        }
      }
      return at + __shfl_sync(0xffffffffu, upto, 31);
    };
    for (int j0 = 0; j0 < live; j0 += 32) {
      if (live > 32) word = keep_word(j0);
      const unsigned front = front_word(j0);
      hole_at = list(~word & front, hole, hole_at, j0);
      fill_at = list(word & ~front, fill, fill_at, j0);
    }
    if (cs > 1) cluster_sync();          // no CTA leaves while its counts are read
  }
  for (int i = moves + rank * kEvThreads + tid; i < a.max_move; i += cs * kEvThreads)
    hole[i] = fill[i] = -1;
  if (tid == 0 && rank == 0) a.move_cnt[row] = moves;
}

// A warp task is 32 moves of one (decision row, KV head).  CH: 16-byte pieces
// of a row.
template <int CH>
__global__ void __launch_bounds__(256)
cache_compact_kernel(const __grid_constant__ CompactArgs a, int groups, long long tasks) {
  constexpr int PER = 2 * CH;            // pieces of a move, K then V
  constexpr int U = 8;                   // loads in flight per lane
  pdl_trigger();
  pdl_wait();
  const Shape& s = a.s;
  const int lane = threadIdx.x & 31;
  const int heads = a.n_mass == 1 ? s.H_kv : 1;
  uint4* Kp = reinterpret_cast<uint4*>(a.Kp);
  uint4* Vp = reinterpret_cast<uint4*>(a.Vp);
  for (long long task = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); task < tasks;
       task += (long long)gridDim.x * 8) {
    const int grp = (int)(task % groups);
    const long long rh = task / groups;
    const int row = (int)(rh / heads), hd = (int)(rh % heads);
    const int b = row / a.n_mass, g = a.n_mass == 1 ? hd : row % a.n_mass;
    int cnt = a.move_cnt[row];
    if (cnt < 0 || cnt > a.max_move) {
      if (grp == 0 && hd == 0 && lane == 0) flag_error(a.err, ERR_BAD_INDEX);
      cnt = cnt < 0 ? 0 : a.max_move;
    }
    const int left = cnt - grp * 32;
    if (left <= 0) continue;
    // lane = move
    long long src = -1, dst = -1;        // 16-byte pieces from the pools' start; -1: no move
    if (lane < left) {
      const size_t at = (size_t)row * a.max_move + grp * 32 + lane;
      const int to = a.hole_idx[at], from = a.fill_idx[at];
      bool ok = to >= 0 && to < s.L_ctx && from >= 0 && from < s.L_ctx;
      if (ok) {
        const int32_t* table = a.page_table + (size_t)b * s.n_pages;
        const int st = table[to / 64], sf = table[from / 64];
        ok = st >= 0 && st < s.n_slots && sf >= 0 && sf < s.n_slots;
        if (ok) {
          dst = (((long long)st * s.H_kv + g) * 64 + to % 64) * CH;
          src = (((long long)sf * s.H_kv + g) * 64 + from % 64) * CH;
          if (hd == 0) {
            const size_t o = (size_t)row * s.L_ctx;
            if (a.tok_pos) a.tok_pos[o + to] = a.tok_pos[o + from];
            if (a.tok_mass) a.tok_mass[o + to] = a.tok_mass[o + from];
          }
        }
      }
      if (!ok && hd == 0) flag_error(a.err, ERR_BAD_INDEX);
    }
    const int n = min(32, left);
#pragma unroll 1
    for (int p0 = 0; p0 < n * PER; p0 += 32 * U) {
      uint4 v[U];
      long long to[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int p = p0 + 32 * u + lane, mv = p / PER, c = p % CH;
        const long long f = __shfl_sync(0xffffffffu, src, mv & 31);
        const long long t = __shfl_sync(0xffffffffu, dst, mv & 31);
        to[u] = mv < n && t >= 0 ? t + c : -1;
        if (to[u] >= 0) v[u] = (p / CH) % 2 ? Vp[f + c] : Kp[f + c];
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int p = p0 + 32 * u + lane;
        if (to[u] >= 0) ((p / CH) % 2 ? Vp : Kp)[to[u]] = v[u];
      }
    }
  }
}

template <bool KEEP>
cudaError_t run_evict(const EvictArgs& a, int cs, size_t smem, cudaStream_t st) {
  auto kern = evict_select_kernel<KEEP>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kKeepTokens * kEvThreads * 4);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.s.batch * a.n_mass) * cs);
  cfg.blockDim = dim3(kEvThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cs;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, a, cs);
}

}  // namespace

cudaError_t launch_evict_select(const EvictArgs& a, cudaStream_t st) {
  // As many CTAs a row as keep one per SM, at least 1024 tokens each; longer
  // rows take more, up to the cluster's eight.
  const long long rows = (long long)a.s.batch * a.n_mass, L = a.s.L_ctx;
  const int sms = tc_sm_count();
  int cs = 1;
  while (cs < kMaxCluster && ((rows * cs * 2 <= sms && L > (long long)cs * kEvThreads) ||
                              L > (long long)cs * kKeepTokens * kEvThreads))
    cs *= 2;
  const long long it = (L + (long long)cs * kEvThreads - 1) / ((long long)cs * kEvThreads);
  if (it <= kKeepTokens) return run_evict<true>(a, cs, (size_t)it * kEvThreads * 4, st);
  return run_evict<false>(a, cs, 0, st);
}

cudaError_t launch_cache_compact(const CompactArgs& a, cudaStream_t st) {
  if (a.max_move == 0) return cudaSuccess;
  const Shape& s = a.s;
  const int groups = (a.max_move + 31) / 32, heads = a.n_mass == 1 ? s.H_kv : 1;
  const long long tasks = (long long)s.batch * a.n_mass * heads * groups;
  const long long want = (tasks + 7) / 8, most = (long long)tc_sm_count() * 8;
  const int grid = (int)(want < most ? want : most);
  const int pieces = s.d * (s.dtype == DL_BF16 ? 2 : 4) / 16;
  if (pieces == 8) {
    DL_LAUNCH(cache_compact_kernel<8>, grid, 256, 0, st, a, groups, tasks);
  } else if (pieces == 16) {
    DL_LAUNCH(cache_compact_kernel<16>, grid, 256, 0, st, a, groups, tasks);
  } else {
    DL_LAUNCH(cache_compact_kernel<32>, grid, 256, 0, st, a, groups, tasks);
  }
  return cudaGetLastError();
}

}  // namespace dl
