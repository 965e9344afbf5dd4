// (c3) The eviction plan of a cache with a budget, and (c4) its moves.
//
// Plan: the `budget` tokens of largest key stay, key = the accumulated mass
// in the order of its bits (held tokens at +infinity, NaN at -infinity),
// equal keys by the lower index.
//
// Bound: latency (a row of n tokens is 8 n bytes; 128 rows of 32K, 38 MB, are
// 6 us of HBM).  A decision row is taken by a cluster of 1 to 8 CTAs that
// splits it in index order and keeps its keys in registers, so that masses and
// positions are read once; a warp owns 32 E consecutive tokens and reads them
// coalesced, lane l of iteration j holding token 32 j + l.
//  - The budget-th key by radix select: a histogram of the top 12 bits (sign,
//    exponent, three bits of mantissa), then of the next 10 and the last 10
//    among the keys that share the digits found.  The CTAs' counts are added
//    through the cluster's shared memory by every CTA for itself.  The search
//    ends at the first digit whose whole bin stays.
//  - One vote per iteration gives the 32 tokens' keep bits as a word, lane j
//    holding iteration j's; holes and fills are then counted and listed by
//    words, with prefix sums over lanes, warps and CTAs.
// Rows too long for the registers (E = 0) recompute their keys from memory in
// every pass.
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
constexpr int kRegTokens = 32;           // most tokens of a thread kept in registers
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
__device__ __forceinline__ int4 peer_int4(const int* p, unsigned rank) {
  const unsigned here = static_cast<unsigned>(__cvta_generic_to_shared(p));
  unsigned there;
  int4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(here), "r"(rank));
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(there)
               : "memory");
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

// E: tokens per thread in registers; 0: keys recomputed from memory, NB blocks
// of 1024 tokens per warp.
template <int E>
__global__ void __launch_bounds__(kEvThreads, 1)
evict_select_kernel(const __grid_constant__ EvictArgs a, int cs, int blocks) {
  constexpr int ITERS = E ? E : 32;      // iterations of one block of a warp
  __shared__ __align__(16) int s_h0[4096];
  __shared__ int s_h1[1024], s_h2[1024];
  __shared__ int s_wt[3][kEvWarps];      // per warp: ties, holes, fills
  __shared__ int s_ct[4];                // this CTA's: largest position, ties, holes, fills
  __shared__ int s_scan[kEvWarps], s_pick[3], s_max[kEvWarps];
  const Shape& s = a.s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const unsigned rank = cs > 1 ? cluster_rank() : 0u;
  const int row = blockIdx.x / cs, b = row / a.n_mass;
  pdl_trigger();
  for (int i = tid; i < 4096; i += kEvThreads) s_h0[i] = 0;
  s_h1[tid] = s_h2[tid] = 0;
  pdl_wait();
  const int n = a.ctx_len[b];
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
    // first token of this warp's block k
    auto block_at = [&](int k) {
      return (((long long)rank * kEvWarps + warp) * blocks + k) * (32 * ITERS);
    };
    unsigned key[E ? E : 1];
    // largest position
    int last = INT32_MIN;
    for (int k = 0; k < blocks; ++k) {
      const long long t0 = block_at(k) + lane;
#pragma unroll
      for (int j = 0; j < ITERS; ++j) {
        const long long t = t0 + 32 * j;
        const int p = t < n ? (pos ? pos[t] : (int)t) : INT32_MIN;
        last = max(last, p);
        if constexpr (E > 0) key[j] = (unsigned)p;
      }
    }
    last = __reduce_max_sync(0xffffffffu, last);
    if (lane == 0) s_max[warp] = last;
    __syncthreads();
    last = __reduce_max_sync(0xffffffffu, s_max[lane]);
    if (cs > 1) {
      if (tid == 0) s_ct[0] = last;
      cluster_sync();
      for (int r = 0; r < cs; ++r) last = max(last, peer_int(&s_ct[0], r));
    }
    const long long recent = (long long)last - a.n_recent;
    auto key_of = [&](long long t, int p) {
      return (p < a.n_first || p > recent) ? kHeldKey : mass_key(mass[t]);
    };
    if constexpr (E > 0) {
      const long long t0 = block_at(0) + lane;
#pragma unroll
      for (int j = 0; j < ITERS; ++j) {
        const long long t = t0 + 32 * j;
        // the mass is read whether or not it counts, so that no load waits on a position
        const float m = t < n ? mass[t] : 0.0f;
        const int p = (int)key[j];
        key[j] = t < n ? ((p < a.n_first || p > recent) ? kHeldKey : mass_key(m)) : 0u;
      }
    }
    // key of iteration j of block k (0: no token)
    auto get = [&](int k, int j) -> unsigned {
      if constexpr (E > 0) {
        return key[j];
      } else {
        const long long t = block_at(k) + 32 * j + lane;
        return t < n ? key_of(t, pos ? pos[t] : (int)t) : 0u;
      }
    };

    // ---- the budget-th key
    unsigned thr = 0;
    int want = a.budget;
    bool whole = false;                  // every key equal to thr (or above, in its bin) stays
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      if (whole) break;
      const int sh = pass == 0 ? 20 : pass == 1 ? 10 : 0;
      int* hist = pass == 0 ? s_h0 : pass == 1 ? s_h1 : s_h2;
      const unsigned above = pass == 0 ? 0u : thr >> (sh + 10);
      for (int k = 0; k < blocks; ++k) {
#pragma unroll
        for (int j = 0; j < ITERS; ++j) {
          const unsigned u = get(k, j);
          if (pass == 0) {
            const unsigned bin = u >> 20;
            // many equal masses (zeros): one count for the warp
            if (__all_sync(0xffffffffu, bin == __shfl_sync(0xffffffffu, bin, 0) && u != 0u)) {
              if (lane == 0) atomicAdd(&hist[bin], 32);
            } else if (u != 0u) {
              atomicAdd(&hist[bin], 1);
            }
          } else if (u != 0u && (u >> (sh + 10)) == above) {
            atomicAdd(&hist[(u >> sh) & 1023u], 1);
          }
        }
      }
      if (cs > 1) cluster_sync(); else __syncthreads();
      // counts from the top: thread t has bins 4 (1023 - t) .. + 3, or bin 1023 - t
      int c[4] = {0, 0, 0, 0};
      if (pass == 0) {
        const int at = 4 * (kEvThreads - 1 - tid);
        for (int r = 0; r < cs; ++r) {
          const int4 v = cs > 1 ? peer_int4(&hist[at], r) : *reinterpret_cast<const int4*>(&hist[at]);
          c[0] += v.w; c[1] += v.z; c[2] += v.y; c[3] += v.x;
        }
      } else {
        const int at = kEvThreads - 1 - tid;
        for (int r = 0; r < cs; ++r) c[0] += cs > 1 ? peer_int(&hist[at], r) : hist[at];
      }
      const int mine = c[0] + c[1] + c[2] + c[3];
      int upto = warp_inclusive(mine, lane);
      if (lane == 31) s_scan[warp] = upto;
      __syncthreads();
      upto += __reduce_add_sync(0xffffffffu, lane < warp ? s_scan[lane] : 0);
      int before = upto - mine;
      if (before < want && want <= upto) {  // one thread
        int q = 0;
        while (before + c[q] < want) before += c[q++];
        s_pick[0] = pass == 0 ? 4 * (kEvThreads - 1 - tid) + 3 - q : kEvThreads - 1 - tid;
        s_pick[1] = want - before;
        s_pick[2] = c[q];
      }
      __syncthreads();
      thr |= (unsigned)s_pick[0] << sh;
      want = s_pick[1];
      whole = want == s_pick[2];
    }

    // ---- keep words; equal keys beyond `want` leave from the highest index down
    int tie_left = 0;                    // equal keys that may stay, from this warp on
    if (!whole) {
      int ties = 0;
      for (int k = 0; k < blocks; ++k) {
#pragma unroll
        for (int j = 0; j < ITERS; ++j) ties += __popc(__ballot_sync(0xffffffffu, get(k, j) == thr));
      }
      if (lane == 0) s_wt[0][warp] = ties;
      __syncthreads();
      const int t = s_wt[0][lane];
      int before = __reduce_add_sync(0xffffffffu, lane < warp ? t : 0);
      if (cs > 1) {
        const int all = __reduce_add_sync(0xffffffffu, t);
        if (tid == 0) s_ct[1] = all;
        cluster_sync();
        for (unsigned r = 0; r < rank; ++r) before += peer_int(&s_ct[1], r);
      }
      tie_left = max(0, want - before);
    }
    // this lane's word of block k: bit i = token block_at(k) + 32 lane + i
    int tie_run = tie_left;
    auto keep_word = [&](int k) {
      unsigned w = 0u, tw = 0u;
#pragma unroll
      for (int j = 0; j < ITERS; ++j) {
        const unsigned u = get(k, j);
        const unsigned kw = __ballot_sync(0xffffffffu, whole ? u >= thr : u > thr);
        if (lane == j) w = kw;
        if (!whole) {
          const unsigned e = __ballot_sync(0xffffffffu, u == thr);
          if (lane == j) tw = e;
        }
      }
      if (!whole) {
        const int c = __popc(tw), upto = warp_inclusive(c, lane);
        int stay = min(c, max(0, tie_run - (upto - c)));
        tie_run = max(0, tie_run - __shfl_sync(0xffffffffu, upto, 31));
        unsigned t = tw;
        for (int drop = c - stay; drop > 0; --drop) t &= ~(0x80000000u >> __clz(t));
        w |= t;
      }
      return w;
    };
    // tokens of the word before `limit`, as a mask
    auto below = [&](long long t0, long long limit) {
      const long long m = limit - t0;
      return m <= 0 ? 0u : m >= 32 ? 0xffffffffu : (1u << (int)m) - 1u;
    };
    unsigned word = 0u;
    int holes = 0, fills = 0;
    for (int k = 0; k < blocks; ++k) {
      word = keep_word(k);
      const long long t0 = block_at(k) + 32 * lane;
      const unsigned front = lane < ITERS ? below(t0, a.budget) : 0u;
      holes += __popc(~word & front);    // budget < n: every token before it exists
      fills += __popc(lane < ITERS ? word & ~front : 0u);
    }
    const int lane_holes = holes, lane_fills = fills;
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
      moves = 0;
      for (int r = 0; r < cs; ++r) {
        const int f = peer_int(&s_ct[3], r);
        moves += f;
        if (r < (int)rank) { hole_at += peer_int(&s_ct[2], r); fill_at += f; }
      }
    }
    tie_run = tie_left;
    for (int k = 0; k < blocks; ++k) {
      if (blocks > 1) word = keep_word(k);
      const long long t0 = block_at(k) + 32 * lane;
      const unsigned front = lane < ITERS ? below(t0, a.budget) : 0u;
      unsigned hw = ~word & front, fw = lane < ITERS ? word & ~front : 0u;
      const int ch = blocks > 1 ? __popc(hw) : lane_holes, cf = blocks > 1 ? __popc(fw) : lane_fills;
      const int uh = warp_inclusive(ch, lane), uf = warp_inclusive(cf, lane);
      int32_t* h = hole + hole_at + uh - ch;
      for (; hw; hw &= hw - 1) *h++ = (int32_t)(t0 + __ffs(hw) - 1);
      int32_t* f = fill + fill_at + uf - cf;
      for (; fw; fw &= fw - 1) *f++ = (int32_t)(t0 + __ffs(fw) - 1);
      hole_at += __shfl_sync(0xffffffffu, uh, 31);
      fill_at += __shfl_sync(0xffffffffu, uf, 31);
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

template <int E>
cudaError_t run_evict(const EvictArgs& a, int cs, int blocks, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.s.batch * a.n_mass) * cs);
  cfg.blockDim = dim3(kEvThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cs;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel<E>, a, cs, blocks);
}

}  // namespace

cudaError_t launch_evict_select(const EvictArgs& a, cudaStream_t st) {
  // As many CTAs a row as keep one per SM, at least 1024 tokens each; longer
  // rows take more, up to the cluster's eight.
  const long long rows = (long long)a.s.batch * a.n_mass, L = a.s.L_ctx;
  const int sms = tc_sm_count();
  int cs = 1;
  while (cs < kMaxCluster && ((rows * cs * 2 <= sms && L > (long long)cs * 1024) ||
                              L > (long long)cs * kRegTokens * kEvThreads))
    cs *= 2;
  const long long per = (L + (long long)cs * kEvThreads - 1) / ((long long)cs * kEvThreads);
  if (per <= 2) return run_evict<2>(a, cs, 1, st);
  if (per <= 4) return run_evict<4>(a, cs, 1, st);
  if (per <= 8) return run_evict<8>(a, cs, 1, st);
  if (per <= 16) return run_evict<16>(a, cs, 1, st);
  if (per <= kRegTokens) return run_evict<32>(a, cs, 1, st);
  return run_evict<0>(a, cs, (int)((per + 31) / 32), st);
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
