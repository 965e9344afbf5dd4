// (c3) The eviction plan of a cache with a budget, and (c4) its moves.
//
// Plan: the `budget` tokens of largest key stay, key = the accumulated mass
// in the order of its bits (held tokens at +infinity, NaN at -infinity),
// equal keys by the lower index.
//
// Bound: latency and instruction issue (a row of n tokens is 8 n bytes; 128
// rows of 32K, 38 MB, are 6 us of HBM; every instruction a token takes is 1 us
// there, so tokens are handled four at a time where they can be).  A decision
// row is taken by a cluster of 1 to 8 CTAs that splits its n tokens evenly in
// index order.  A warp reads its tokens coalesced, 16 bytes a lane, and turns
// them through shared memory so that each lane ends with `it` consecutive
// tokens; their keys stay there, masses and positions are read once.
//  - The budget-th key by radix select: a histogram of the top 12 bits (sign,
//    exponent, three bits of mantissa), then of the next 10 and the last 10
//    among the keys that share the digits found.  Each CTA counts its own
//    tokens and sums its bins by groups of 32; every CTA then adds the groups'
//    sums over the cluster, finds the group, and adds that group's 32 bins
//    alone (adding all bins over the cluster took four times as long).  The
//    search ends at the first digit whose whole bin stays.
//  - A lane's keep bits are one word; holes and fills are counted and listed
//    by words, with prefix sums over lanes, warps and CTAs.
// Rows too long for the cluster's shared memory go through it in tiles, read
// again for every pass.
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
constexpr int kMaxIt = 44;               // most tokens of a thread: 11 16-byte chunks, 176 KB a CTA
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

// Lists the set bits of the lanes' words, in order, from out[at] on; bit i of
// lane l is token t0 + i of that lane.  Word by word, so that neighbours are
// written together, or each lane its own when no word is crowded.
__device__ __forceinline__ int list_bits(unsigned long long w, int32_t* out, int at, long long t0,
                                         int it, int lane) {
  const int c = __popcll(w), upto = warp_inclusive(c, lane);
  if (__reduce_max_sync(0xffffffffu, c) <= 12) {
    int32_t* o = out + at + upto - c;
    for (; w; w &= w - 1) *o++ = (int32_t)(t0 + __ffsll(w) - 1);
  } else {
    for (unsigned some = __ballot_sync(0xffffffffu, w != 0ull); some; some &= some - 1) {
      const int j = __ffs(some) - 1;
      const unsigned long long v = __shfl_sync(0xffffffffu, w, j);
      const int o = at + __shfl_sync(0xffffffffu, upto - c, j);
      const long long t = __shfl_sync(0xffffffffu, t0, j);
      for (int i = lane; i < it; i += 32)
        if ((v >> i) & 1) out[o + __popcll(v & ((1ull << i) - 1))] = (int32_t)(t + i);
    }
  }
  return at + __shfl_sync(0xffffffffu, upto, 31);
}

// VEC: masses and positions may be read 16 bytes at a time.
template <bool VEC>
__global__ void __launch_bounds__(kEvThreads, 1)
evict_select_kernel(const __grid_constant__ EvictArgs a, int cs, int max_it) {
  extern __shared__ uint4 s_key[];       // [thread][it / 4 | 1]
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
    // Tokens per thread of a tile, a multiple of 4; tiles; the tile's first
    // token of this warp.  64 bits: the last ones may lie past 2^31.
    const int span = cs * kEvThreads;
    int it = (int)(((long long)n + 4 * span - 1) / (4 * span)) * 4, tiles = 1;
    if (it > max_it) {
      tiles = (it + max_it - 1) / max_it;
      it = max_it;
    }
    const int cpl = it / 4, pitch = cpl | 1;  // chunks of a lane; an odd pitch spreads the banks
    uint4* warp_keys = s_key + warp * 32 * pitch;
    uint4* my_keys = warp_keys + lane * pitch;
    auto warp_at = [&](int k) {
      return (((long long)rank * tiles + k) * kEvWarps + warp) * 32 * it;
    };
    // chunk q (16 bytes) of a warp's tile belongs to lane q / cpl
    const int step_l = 32 / cpl, step_c = 32 % cpl;
    struct Spot { int l, c; };
    auto first_spot = [&]() { return Spot{lane / cpl, lane % cpl}; };
    auto next_spot = [&](Spot& p) {
      p.l += step_l;
      p.c += step_c;
      if (p.c >= cpl) { p.c -= cpl; ++p.l; }
    };
    // four values at token t (a chunk behind the row's end repeats its last)
    auto load4 = [&](const int* x, long long t) -> int4 {
      if (VEC) return *reinterpret_cast<const int4*>(x + min(t, (long long)((n - 1) & ~3)));
      int4 v;
      v.x = x[min(t, (long long)n - 1)];
      v.y = x[min(t + 1, (long long)n - 1)];
      v.z = x[min(t + 2, (long long)n - 1)];
      v.w = x[min(t + 3, (long long)n - 1)];
      return v;
    };
    auto load_pos = [&](long long t) -> int4 {
      return pos ? load4(pos, t) : make_int4((int)t, (int)t + 1, (int)t + 2, (int)t + 3);
    };
    const int* massi = reinterpret_cast<const int*>(mass);
    constexpr int U = 4;                 // 16-byte loads ahead
    int4 m0[U];                          // the first masses do not wait for the largest position
    if (tiles == 1) {
#pragma unroll
      for (int u = 0; u < U; ++u) m0[u] = load4(massi, warp_at(0) + 4 * (32 * u + lane));
    }
    int last = INT32_MIN;
    for (int k = 0; k < tiles; ++k) {
      const long long t0 = warp_at(k) + 4 * lane;
      Spot sp = first_spot();
      for (int i0 = 0; i0 < cpl; i0 += U) {
        if (warp_at(k) + 128 * i0 >= n) break;
        int4 p[U];
#pragma unroll
        for (int u = 0; u < U; ++u) p[u] = load_pos(t0 + 128 * (i0 + u));
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const long long t = t0 + 128 * (i0 + u);
          if (t + 3 < n) {
            last = max(max(max(last, p[u].x), max(p[u].y, p[u].z)), p[u].w);
          } else {
            if (t < n) last = max(last, p[u].x);
            if (t + 1 < n) last = max(last, p[u].y);
            if (t + 2 < n) last = max(last, p[u].z);
          }
          if (tiles == 1 && i0 + u < cpl) {
            warp_keys[sp.l * pitch + sp.c] = make_uint4(p[u].x, p[u].y, p[u].z, p[u].w);
            next_spot(sp);
          }
        }
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
    // not held: n_first <= pos <= last - n_recent, as one unsigned comparison
    const long long room = (long long)last - a.n_recent - a.n_first + 1;
    const unsigned loose = room > 0 ? (unsigned)min(room, 0xffffffffll) : 0u;
    auto key_of = [&](int p, int m) {
      return (unsigned)p - (unsigned)a.n_first < loose ? mass_key(__int_as_float(m)) : kHeldKey;
    };
    // Keys of tile k, each lane's own chunks in order (0: no token).
    auto load_tile = [&](int k) {
      const long long t0 = warp_at(k) + 4 * lane;
      Spot sp = first_spot();
      __syncwarp();
#pragma unroll 1
      for (int i0 = 0; i0 < cpl; i0 += U) {
        const bool none = warp_at(k) + 128 * i0 >= n;  // nothing here for the warp
        if (!none && (i0 > 0 || tiles > 1)) {
#pragma unroll
          for (int u = 0; u < U; ++u) m0[u] = load4(massi, t0 + 128 * (i0 + u));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (i0 + u >= cpl) break;
          const long long t = t0 + 128 * (i0 + u);
          uint4* at = warp_keys + sp.l * pitch + sp.c;
          uint4 q = make_uint4(0u, 0u, 0u, 0u);
          if (t < n) {
            int4 p;
            if (tiles == 1) {
              const uint4 v = *at;
              p = make_int4(v.x, v.y, v.z, v.w);
            } else {
              p = load_pos(t);
            }
            q.x = key_of(p.x, m0[u].x);
            if (t + 1 < n) q.y = key_of(p.y, m0[u].y);
            if (t + 2 < n) q.z = key_of(p.z, m0[u].z);
            if (t + 3 < n) q.w = key_of(p.w, m0[u].w);
          }
          *at = q;
          next_spot(sp);
        }
      }
      __syncwarp();
    };
    if (tiles == 1) load_tile(0);

    // ---- the budget-th key
    unsigned thr = 0;
    int want = a.budget;
    bool whole = false;                  // every key of the last bin stays
#pragma unroll 1
    for (int pass = 0; pass < 3 && !whole; ++pass) {
      const int sh = pass == 0 ? 20 : pass == 1 ? 10 : 0, groups = pass == 0 ? 128 : 32;
      int* hist = s_hist + (pass == 0 ? 0 : 4096 + (pass - 1) * 1024);
      for (int k = 0; k < tiles; ++k) {
        if (tiles > 1) load_tile(k);
        if (warp_at(k) >= n) break;
        if (pass == 0) {
          for (int c = 0; c < cpl; ++c) {
            const uint4 q = my_keys[c];
            const unsigned first = __shfl_sync(0xffffffffu, q.x, 0) >> 20;
            // many equal masses (zeros): one count for the warp
            if (__all_sync(0xffffffffu, q.w != 0u && (q.x >> 20) == first && (q.y >> 20) == first &&
                                            (q.z >> 20) == first && (q.w >> 20) == first)) {
              if (lane == 0) atomicAdd(&hist[first], 128);
            } else {
              if (q.x) atomicAdd(&hist[q.x >> 20], 1);
              if (q.y) atomicAdd(&hist[q.y >> 20], 1);
              if (q.z) atomicAdd(&hist[q.z >> 20], 1);
              if (q.w) atomicAdd(&hist[q.w >> 20], 1);
            }
          }
        } else {
          // no key is 0 above the digits: bit patterns of "no token" never match
          const unsigned above = thr >> (sh + 10);
          for (int c = 0; c < cpl; ++c) {
            const uint4 q = my_keys[c];
            if ((q.x >> (sh + 10)) == above) atomicAdd(&hist[(q.x >> sh) & 1023u], 1);
            if ((q.y >> (sh + 10)) == above) atomicAdd(&hist[(q.y >> sh) & 1023u], 1);
            if ((q.z >> (sh + 10)) == above) atomicAdd(&hist[(q.z >> sh) & 1023u], 1);
            if ((q.w >> (sh + 10)) == above) atomicAdd(&hist[(q.w >> sh) & 1023u], 1);
          }
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
#pragma unroll
      for (int q = 0; q < 4; ++q) c[q] = q < per ? gs[top - q] : 0;
      const int mine = (c[0] + c[1]) + (c[2] + c[3]), upto = warp_inclusive(mine, lane);
      {
        const unsigned hit = __ballot_sync(0xffffffffu, upto >= want);  // not empty: want of them exist
        const int l = __ffs(hit) - 1;
        int q = 0, at = upto - mine;
#pragma unroll
        for (int e = 0; e < 3; ++e)
          if (q == e && e < per - 1 && at + c[e] < want) { at += c[e]; ++q; }
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
      const int in_bin = __shfl_sync(0xffffffffu, v, l);
      thr |= (unsigned)(group * 32 + 31 - l) << sh;
      want -= __shfl_sync(0xffffffffu, sum, l) - in_bin;
      whole = want == in_bin;
    }

    // ---- keep words; equal keys beyond `want` leave from the highest index down
    auto word_of = [&](auto in) {        // bit i: in(key of this lane's token i)
      unsigned long long w = 0ull;
      for (int c = 0; c < cpl; ++c) {
        const uint4 q = my_keys[c];
        const unsigned f = (in(q.x) ? 1u : 0u) | (in(q.y) ? 2u : 0u) | (in(q.z) ? 4u : 0u) | (in(q.w) ? 8u : 0u);
        w |= (unsigned long long)f << (4 * c);
      }
      return w;
    };
    const unsigned thr_c = thr;
    int tie_first = 0;                   // equal keys of the CTAs before this one
    if (!whole && cs > 1) {
      int ties = 0;
      for (int k = 0; k < tiles; ++k) {
        if (tiles > 1) load_tile(k);
        ties += __popcll(word_of([&](unsigned u) { return u == thr_c; }));
      }
      ties = __reduce_add_sync(0xffffffffu, ties);
      if (lane == 0) s_wt[0][warp] = ties;
      __syncthreads();
      const int all = __reduce_add_sync(0xffffffffu, s_wt[0][lane]);
      if (tid == 0) s_ct[1] = all;
      cluster_sync();
      tie_first = __reduce_add_sync(0xffffffffu, lane < rank ? peer_int(&s_ct[1], lane) : 0);
    }
    // this lane's keep bits of tile k; `seen`: equal keys of the tiles before
    auto keep_word = [&](int k, int& seen) {
      if (tiles > 1) load_tile(k);
      if (whole) return word_of([&](unsigned u) { return u >= thr_c; });
      unsigned long long tw = word_of([&](unsigned u) { return u == thr_c; });
      const int c = __popcll(tw), upto = warp_inclusive(c, lane);
      __syncthreads();                   // the last counts are no longer read
      if (lane == 31) s_wt[0][warp] = upto;
      __syncthreads();
      const int t = s_wt[0][lane];
      const int before = seen + __reduce_add_sync(0xffffffffu, lane < warp ? t : 0) + upto - c;
      seen += __reduce_add_sync(0xffffffffu, t);
      const int stay = min(c, max(0, want - before));
      for (int drop = c - stay; drop > 0; --drop) tw &= ~(0x8000000000000000ull >> __clzll(tw));
      return tw | word_of([&](unsigned u) { return u > thr_c; });
    };
    auto lane_at = [&](int k) { return warp_at(k) + (long long)lane * it; };
    // this lane's tokens before the budget (they exist: budget < n), as a mask
    auto front_word = [&](int k) {
      const long long m = a.budget - lane_at(k);
      return m <= 0 ? 0ull : (1ull << (int)min(m, (long long)it)) - 1ull;  // it <= 44
    };
    unsigned long long word = 0ull;
    int holes = 0, fills = 0, seen = tie_first;
    for (int k = 0; k < tiles; ++k) {
      word = keep_word(k, seen);
      const unsigned long long front = front_word(k);
      holes += __popcll(~word & front);
      fills += __popcll(word & ~front);
    }
    holes = __reduce_add_sync(0xffffffffu, holes);
    fills = __reduce_add_sync(0xffffffffu, fills);
    if (lane == 0) { s_wt[1][warp] = holes; s_wt[2][warp] = fills; }
    __syncthreads();
    const int th = s_wt[1][lane], tf = s_wt[2][lane];
    int hole_first = 0, fill_first = 0;  // of the CTAs before this one
    moves = __reduce_add_sync(0xffffffffu, tf);
    if (cs > 1) {
      const int all_h = __reduce_add_sync(0xffffffffu, th);
      if (tid == 0) { s_ct[2] = all_h; s_ct[3] = moves; }
      cluster_sync();
      const int f = lane < cs ? peer_int(&s_ct[3], lane) : 0;
      const int h = lane < rank ? peer_int(&s_ct[2], lane) : 0;
      moves = __reduce_add_sync(0xffffffffu, f);
      hole_first = __reduce_add_sync(0xffffffffu, h);
      fill_first = __reduce_add_sync(0xffffffffu, lane < rank ? f : 0);
    }
    if (tiles == 1) {
      const unsigned long long front = front_word(0);
      list_bits(~word & front, hole, hole_first + __reduce_add_sync(0xffffffffu, lane < warp ? th : 0),
                lane_at(0), it, lane);
      list_bits(word & ~front, fill, fill_first + __reduce_add_sync(0xffffffffu, lane < warp ? tf : 0),
                lane_at(0), it, lane);
    } else {
      seen = tie_first;
      for (int k = 0; k < tiles; ++k) {
        word = keep_word(k, seen);
        const unsigned long long front = front_word(k);
        const int h = __reduce_add_sync(0xffffffffu, __popcll(~word & front));
        const int f = __reduce_add_sync(0xffffffffu, __popcll(word & ~front));
        __syncthreads();
        if (lane == 0) { s_wt[1][warp] = h; s_wt[2][warp] = f; }
        __syncthreads();
        const int uh = s_wt[1][lane], uf = s_wt[2][lane];
        list_bits(~word & front, hole, hole_first + __reduce_add_sync(0xffffffffu, lane < warp ? uh : 0),
                  lane_at(k), it, lane);
        list_bits(word & ~front, fill, fill_first + __reduce_add_sync(0xffffffffu, lane < warp ? uf : 0),
                  lane_at(k), it, lane);
        hole_first += __reduce_add_sync(0xffffffffu, uh);
        fill_first += __reduce_add_sync(0xffffffffu, uf);
      }
    }
    if (cs > 1) cluster_sync();          // no CTA leaves while its counts are read
  }
  for (int i = moves + rank * kEvThreads + tid; i < a.max_move; i += cs * kEvThreads)
    hole[i] = fill[i] = -1;
  if (tid == 0 && rank == 0) a.move_cnt[row] = moves;
}

// A warp task is M moves of one (decision row, KV head).  CH: 16-byte pieces
// of a row.
template <int CH, int M>
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
    // the moves do not wait for their number (their lists are max_move long)
    const int i = grp * M + lane;
    const bool in = lane < M && i < a.max_move;
    const size_t at = (size_t)row * a.max_move + (in ? i : 0);
    const int to = a.hole_idx[at], from = a.fill_idx[at];
    int cnt = a.move_cnt[row];
    if (cnt < 0 || cnt > a.max_move) {
      if (grp == 0 && hd == 0 && lane == 0) flag_error(a.err, ERR_BAD_INDEX);
      cnt = cnt < 0 ? 0 : a.max_move;
    }
    const int n = min(M, cnt - grp * M);
    if (n <= 0) continue;
    // lane = move; rows of the pools, -1: no move
    int src = -1, dst = -1;
    if (lane < n) {
      bool ok = to >= 0 && to < s.L_ctx && from >= 0 && from < s.L_ctx;
      if (ok) {
        const int32_t* table = a.page_table + (size_t)b * s.n_pages;
        const int st = table[to / 64], sf = table[from / 64];
        ok = st >= 0 && st < s.n_slots && sf >= 0 && sf < s.n_slots;
        if (ok) {
          dst = (st * s.H_kv + g) * 64 + to % 64;
          src = (sf * s.H_kv + g) * 64 + from % 64;
          if (hd == 0) {
            const size_t o = (size_t)row * s.L_ctx;
            if (a.tok_pos) a.tok_pos[o + to] = a.tok_pos[o + from];
            if (a.tok_mass) a.tok_mass[o + to] = a.tok_mass[o + from];
          }
        }
      }
      if (!ok && hd == 0) flag_error(a.err, ERR_BAD_INDEX);
    }
#pragma unroll 1
    for (int p0 = 0; p0 < n * PER; p0 += 32 * U) {
      uint4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int p = p0 + 32 * u + lane, f = __shfl_sync(0xffffffffu, src, (p / PER) & 31);
        if (p < n * PER && f >= 0) v[u] = ((p / CH) % 2 ? Vp : Kp)[(size_t)f * CH + p % CH];
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int p = p0 + 32 * u + lane, t = __shfl_sync(0xffffffffu, dst, (p / PER) & 31);
        if (p < n * PER && t >= 0) ((p / CH) % 2 ? Vp : Kp)[(size_t)t * CH + p % CH] = v[u];
      }
    }
  }
}

template <bool VEC>
cudaError_t run_evict(const EvictArgs& a, int cs, int it, cudaStream_t st) {
  cudaError_t e = allow_smem<evict_select_kernel<VEC>>((kMaxIt / 4 | 1) * 16 * kEvThreads);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.s.batch * a.n_mass) * cs);
  cfg.blockDim = dim3(kEvThreads);
  cfg.dynamicSmemBytes = (size_t)(it / 4 | 1) * 16 * kEvThreads;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cs;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel<VEC>, a, cs, it);
}

}  // namespace

cudaError_t launch_evict_select(const EvictArgs& a, cudaStream_t st) {
  // As many CTAs a row as keep one per SM, at least 1024 tokens each; longer
  // rows take more, up to the cluster's eight.
  const long long rows = (long long)a.s.batch * a.n_mass, L = a.s.L_ctx;
  const int sms = tc_sm_count();
  int cs = 1;
  while (cs < kMaxCluster && ((rows * cs * 2 <= sms && L > (long long)cs * kEvThreads) ||
                              L > (long long)cs * kMaxIt * kEvThreads))
    cs *= 2;
  const long long per = (L + 4ll * cs * kEvThreads - 1) / (4ll * cs * kEvThreads) * 4;
  const int it = (int)(per < kMaxIt ? (per > 0 ? per : 4) : kMaxIt);
  const bool vec = L % 4 == 0 && (reinterpret_cast<uintptr_t>(a.tok_mass) & 15) == 0 &&
                   (reinterpret_cast<uintptr_t>(a.tok_pos) & 15) == 0;
  return vec ? run_evict<true>(a, cs, it, st) : run_evict<false>(a, cs, it, st);
}

cudaError_t launch_cache_compact(const CompactArgs& a, cudaStream_t st) {
  if (a.max_move == 0) return cudaSuccess;
  const Shape& s = a.s;
  const long long rows = (long long)s.batch * a.n_mass * (a.n_mass == 1 ? s.H_kv : 1);
  // Eight moves a warp (one round of loads) while that leaves SMs idle, else 32.
  const int sms = tc_sm_count(), few = (a.max_move + 31) / 32;
  const bool wide = rows * few >= 20ll * sms;
  const int groups = wide ? few : (a.max_move + 7) / 8;
  const long long tasks = rows * groups, want = (tasks + 7) / 8, most = (long long)sms * 8;
  const int grid = (int)(want < most ? want : most);
#define DL_COMPACT(CH_)                                                                           \
  do {                                                                                            \
    if (wide) DL_LAUNCH((cache_compact_kernel<CH_, 32>), grid, 256, 0, st, a, groups, tasks);     \
    else DL_LAUNCH((cache_compact_kernel<CH_, 8>), grid, 256, 0, st, a, groups, tasks);           \
  } while (0)
  const int pieces = s.d * (s.dtype == DL_BF16 ? 2 : 4) / 16;
  if (pieces == 8) DL_COMPACT(8);
  else if (pieces == 16) DL_COMPACT(16);
  else DL_COMPACT(32);
#undef DL_COMPACT
  return cudaGetLastError();
}

}  // namespace dl
