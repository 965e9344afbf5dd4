// (c3) The eviction plan of a cache with a budget, and (c4) its moves.
//
// Plan: the `budget` tokens of largest key stay, key = the accumulated mass
// in the order of its bits (held tokens at +infinity, NaN at -infinity),
// equal keys by the lower index.
//
// Bound: latency and instruction issue (a row of n tokens is 8 n bytes; 128
// rows of 32K, 38 MB, are 6 us of HBM; every instruction a token takes is 1 us
// there, so tokens are handled four at a time where they can be).  A decision
// row is taken by a cluster of 1 to 8 CTAs that splits the row's capacity
// evenly in index order, 4 CPL tokens a thread.  A warp reads its tokens
// coalesced, 16 bytes a lane, and turns them through shared memory so that
// each lane ends with consecutive tokens; their keys stay there, masses and
// positions are read once.
//  - The budget-th key by radix select: a histogram of the top 12 bits (sign,
//    exponent, three bits of mantissa), then of the next 10 and the last 10
//    among the keys that share the digits found.  Each CTA counts its own
//    tokens and sums its bins by groups of 32; every CTA then adds the groups'
//    sums over the cluster, finds the group, and adds that group's 32 bins
//    alone (adding all bins over the cluster took four times as long).  The
//    search ends at the first digit whose whole bin stays.
//  - A lane's keep bits are one word; holes and fills are counted by words,
//    with prefix sums over lanes, warps and CTAs, listed in shared memory and
//    copied out side by side.
// Rows too long for the cluster's shared memory go through it in tiles, read
// again for every pass.
//
// Moves: bound by HBM (each moved row is read and written once) with rows of 128
// to 512 bytes at random places: 206 MB of them at 4.95 TB/s.  A warp resolves 32
// moves at a time, one per lane, then all lanes copy their rows in 16-byte
// pieces, eight loads ahead of the stores.  (Bulk copies through shared memory,
// with 2.5 times as much in flight, took as long: 42.8 against 41.9 us.)
#include "cluster.cuh"
#include "common.cuh"
#include "internal.h"
#include "launch.cuh"
#include "tc_common.cuh"

namespace dl {

namespace {

constexpr int kMaxCluster = 8;
constexpr int kMaxChunks = 8;            // 16-byte chunks of a thread
constexpr unsigned kHeldKey = 0xFF800000u;  // the key of +infinity

// Order-preserving bits of a mass: a < b as numbers <=> key(a) < key(b);
// -0 like +0, NaN like -infinity.  No key is 0, which marks "no token".
__device__ __forceinline__ unsigned mass_key(float x) {
  if (x != x) x = -INFINITY;
  const unsigned u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ int warp_inclusive(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// NT: threads, 512 or 1024.  CPL: 16-byte chunks (four tokens) of a thread.  VEC:
// masses and positions may be read 16 bytes at a time.
template <int NT, int CPL, bool VEC>
__global__ void __launch_bounds__(NT, 1024 / NT)
evict_select_kernel(const __grid_constant__ EvictArgs a, int cs, int tiles) {
  constexpr int NW = NT / 32;            // warps
  constexpr int IT = 4 * CPL;            // tokens of a thread
  constexpr int PITCH = CPL | 1;         // chunks from lane to lane: odd, to spread the banks
  extern __shared__ uint4 s_key[];       // [thread][PITCH], later the lists
  __shared__ __align__(16) int s_hist[4096 + 2 * 1024];
  __shared__ int s_group[3][128];        // this CTA's counts of 32 bins
  __shared__ int s_gsum[128], s_bsum[32];  // the cluster's
  __shared__ int s_wt[3][NW];      // per warp: ties, holes, fills
  __shared__ int s_ct[4];                // this CTA's: largest position, ties, holes, fills
  __shared__ int s_max[NW];
  const Shape& s = a.s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = cs > 1 ? cluster_rank() : 0;
  const int row = blockIdx.x / cs, b = row / a.n_mass;
  pdl_trigger();
  pdl_wait();
  const int n = a.ctx_len[b];
  for (int i = tid; i < 4096 + 2 * 1024; i += NT) s_hist[i] = 0;
  const bool bad = n < 0 || n > s.L_ctx;
  if (tid == 0 && rank == 0 && row % a.n_mass == 0) {
    if (bad) flag_error(a.err, ERR_BAD_INDEX);
    a.new_len[b] = bad ? n : min(n, a.budget);
  }
  int32_t* hole = a.hole_idx + (size_t)row * a.max_move;
  int32_t* fill = a.fill_idx + (size_t)row * a.max_move;
  int moves = 0;
  if (!bad && n > a.budget) {            // the same for the whole cluster
    const int* mass = reinterpret_cast<const int*>(a.tok_mass + (size_t)row * s.L_ctx);
    const int* pos = a.tok_pos ? a.tok_pos + (size_t)row * s.L_ctx : nullptr;
    const unsigned len = (unsigned)n;
    // this warp's first token of tile k (unsigned: the last may lie past 2^31)
    auto warp_at = [&](int k) { return (unsigned)((rank * tiles + k) * NW + warp) * (32u * IT); };
    // four values from token t on; behind the row's end, its last ones
    auto load4 = [&](const int* x, unsigned t) -> int4 {
      if (VEC) return *reinterpret_cast<const int4*>(x + min(t, (len - 1u) & ~3u));
      int4 v;
      v.x = x[min(t, len - 1u)];
      v.y = x[min(t + 1u, len - 1u)];
      v.z = x[min(t + 2u, len - 1u)];
      v.w = x[min(t + 3u, len - 1u)];
      return v;
    };
    auto load_pos = [&](unsigned t) -> int4 {
      return pos ? load4(pos, t) : make_int4((int)t, (int)t + 1, (int)t + 2, (int)t + 3);
    };
    // chunk 32 i + lane of a warp's tile belongs to lane (32 i + lane) / CPL
    uint4* warp_keys = s_key + warp * 32 * PITCH;
    uint4* my_keys = warp_keys + lane * PITCH;
    uint4* put_at = warp_keys + (lane / CPL) * PITCH + lane % CPL;
    constexpr int PUT = (32 / CPL) * PITCH;  // from chunk to chunk of the loading order

    // ---- largest position
    int last = INT32_MIN;
#pragma unroll 1
    for (int k = 0; k < tiles; ++k) {
      const unsigned t0 = warp_at(k) + 4u * lane;
      if (warp_at(k) >= len) break;
      int4 p[CPL];
#pragma unroll
      for (int i = 0; i < CPL; ++i) p[i] = load_pos(t0 + 128u * i);
#pragma unroll
      for (int i = 0; i < CPL; ++i) {
        const unsigned t = t0 + 128u * i;
        if (t < len) last = max(last, p[i].x);
        if (t + 1u < len) last = max(last, p[i].y);
        if (t + 2u < len) last = max(last, p[i].z);
        if (t + 3u < len) last = max(last, p[i].w);
        if (tiles == 1) put_at[i * PUT] = make_uint4(p[i].x, p[i].y, p[i].z, p[i].w);
      }
    }
    constexpr int U = CPL < 4 ? CPL : 4;   // masses loaded ahead
    const bool here = warp_at(0) < len;
    int4 m0[U];                          // the first do not wait for the largest position
    if (tiles == 1 && here) {
#pragma unroll
      for (int u = 0; u < U; ++u) m0[u] = load4(mass, warp_at(0) + 4u * lane + 128u * u);
    }
    last = __reduce_max_sync(0xffffffffu, last);
    if (lane == 0) s_max[warp] = last;
    __syncthreads();
    last = __reduce_max_sync(0xffffffffu, s_max[lane % NW]);
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
    // Keys of tile k, each lane's own chunks in order (0: no token).  False:
    // the warp has none.
    auto load_tile = [&](int k) {
      const unsigned w0 = warp_at(k), t0 = w0 + 4u * lane;
      if (w0 >= len) return false;
      __syncwarp();
#pragma unroll 1
      for (int i0 = 0; i0 < CPL; i0 += U) {
        if (i0 > 0 || tiles > 1) {
#pragma unroll
          for (int u = 0; u < U; ++u) m0[u] = load4(mass, t0 + 128u * (i0 + u));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const unsigned t = t0 + 128u * (i0 + u);
          uint4* at = put_at + (i0 + u) * PUT;
          int4 p;
          if (tiles == 1) {
            const uint4 v = *at;
            p = make_int4(v.x, v.y, v.z, v.w);
          } else {
            p = load_pos(t);
          }
          uint4 q;
          q.x = t < len ? key_of(p.x, m0[u].x) : 0u;
          q.y = t + 1u < len ? key_of(p.y, m0[u].y) : 0u;
          q.z = t + 2u < len ? key_of(p.z, m0[u].z) : 0u;
          q.w = t + 3u < len ? key_of(p.w, m0[u].w) : 0u;
          *at = q;
        }
      }
      __syncwarp();
      return true;
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
      // no key is 0 in the digits above: "no token" never matches them
      const unsigned above = pass == 0 ? 0u : thr >> (sh + 10), mask = pass == 0 ? 4095u : 1023u;
#pragma unroll 1
      for (int k = 0; k < tiles; ++k) {
        if (tiles > 1 ? !load_tile(k) : !here) break;
#pragma unroll 2
        for (int c = 0; c < CPL; ++c) {
          const uint4 q = my_keys[c];
          auto count = [&](unsigned u) {
            if (pass == 0 ? u != 0u : (u >> (sh + 10)) == above) atomicAdd(&hist[(u >> sh) & mask], 1);
          };
          // many equal masses (zeros): one count for the warp
          const unsigned first = __shfl_sync(0xffffffffu, q.x, 0);
          if (pass == 0 &&
              __all_sync(0xffffffffu, ((q.x ^ first) | (q.y ^ first) | (q.z ^ first) | (q.w ^ first)) == 0u)) {
            if (lane == 0 && first) atomicAdd(&hist[first >> 20], 128);
          } else {
            count(q.x); count(q.y); count(q.z); count(q.w);
          }
        }
      }
      __syncthreads();
      for (int e = tid; e < groups * 8; e += NT) {  // eight lanes a group
        const int4 v = reinterpret_cast<const int4*>(hist)[e];
        int c = (v.x + v.y) + (v.z + v.w);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
        if ((lane & 7) == 0) s_group[pass][e >> 3] = c;
      }
      if (cs > 1) cluster_sync(); else __syncthreads();
      if (cs > 1) {
        for (int e = tid; e < groups * 8; e += NT) {  // lane & 7 = rank
          int c = (lane & 7) < cs ? peer_int(&s_group[pass][e >> 3], lane & 7) : 0;
#pragma unroll
          for (int o = 4; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
          if ((lane & 7) == 0) s_gsum[e >> 3] = c;
        }
        __syncthreads();
      }
      // every warp for itself: the group, counted from the top
      const int* gs = cs > 1 ? s_gsum : s_group[pass];
      int group = 0, before = 0;
      {
        // lane's groups: top, top - 1 .. (four in the first pass, else one)
        const int per = groups / 32, top = groups - 1 - per * lane;
        int c[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) c[q] = q < per ? gs[top - q] : 0;
        const int mine = (c[0] + c[1]) + (c[2] + c[3]), upto = warp_inclusive(mine, lane);
        const int l = __ffs(__ballot_sync(0xffffffffu, upto >= want)) - 1;  // want of them exist
        int q = 0, at = upto - mine;
#pragma unroll
        for (int e = 0; e < 3; ++e)
          if (q == e && at + c[e] < want) { at += c[e]; ++q; }
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
    // bit i: this lane's token i has a key above (or at least) x
    auto word_of = [&](unsigned x, bool equal) {
      unsigned w = 0u;
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        const uint4 q = my_keys[c];
        const unsigned f = equal ? (q.x == x ? 1u : 0u) | (q.y == x ? 2u : 0u) | (q.z == x ? 4u : 0u) | (q.w == x ? 8u : 0u)
                                 : (q.x >= x ? 1u : 0u) | (q.y >= x ? 2u : 0u) | (q.z >= x ? 4u : 0u) | (q.w >= x ? 8u : 0u);
        w |= f << (4 * c);
      }
      return w;
    };
    int tie_first = 0;                   // equal keys of the CTAs before this one
    if (!whole && cs > 1) {
      int ties = 0;
#pragma unroll 1
      for (int k = 0; k < tiles; ++k) {
        if (tiles > 1 ? !load_tile(k) : !here) break;
        ties += __popc(word_of(thr, true));
      }
      ties = __reduce_add_sync(0xffffffffu, ties);
      if (lane == 0) s_wt[0][warp] = ties;
      __syncthreads();
      const int all = __reduce_add_sync(0xffffffffu, lane < NW ? s_wt[0][lane] : 0);
      if (tid == 0) s_ct[1] = all;
      cluster_sync();
      tie_first = __reduce_add_sync(0xffffffffu, lane < rank ? peer_int(&s_ct[1], lane) : 0);
    }
    // this lane's keep bits of tile k; `seen`: equal keys of the tiles before
    auto keep_word = [&](int k, int& seen) {
      const bool any = tiles > 1 ? load_tile(k) : here;
      unsigned w = any ? word_of(thr, false) : 0u;
      if (whole) return w;
      unsigned tw = any ? word_of(thr, true) : 0u;
      w &= ~tw;
      const int c = __popc(tw), upto = warp_inclusive(c, lane);
      __syncthreads();                   // the last counts are no longer read
      if (lane == 31) s_wt[0][warp] = upto;
      __syncthreads();
      const int t = lane < NW ? s_wt[0][lane] : 0;
      const int before = seen + __reduce_add_sync(0xffffffffu, lane < warp ? t : 0) + upto - c;
      seen += __reduce_add_sync(0xffffffffu, t);
      const int stay = min(c, max(0, want - before));
      for (int drop = c - stay; drop > 0; --drop) tw &= ~(0x80000000u >> __clz(tw));
      return w | tw;
    };
    auto lane_at = [&](int k) { return warp_at(k) + (unsigned)(lane * IT); };
    // this lane's tokens before the budget (they exist: budget < n), as a mask
    auto front_word = [&](int k) {
      const unsigned t = lane_at(k), m = (unsigned)a.budget > t ? (unsigned)a.budget - t : 0u;
      return m >= (unsigned)IT ? 0xffffffffu >> (32 - IT) : (1u << m) - 1u;
    };
    unsigned word = 0u;
    int holes = 0, fills = 0, seen = tie_first;
#pragma unroll 1
    for (int k = 0; k < tiles; ++k) {
      word = keep_word(k, seen);
      const unsigned front = front_word(k);
      holes += __popc(~word & front);
      fills += __popc(word & ~front);
    }
    // ---- lists: holes and fills of this tile in shared memory, then out
    int hole_first = 0, fill_first = 0;  // of the CTAs (and tiles) before
    if (cs > 1) {
      const int h = __reduce_add_sync(0xffffffffu, holes), f = __reduce_add_sync(0xffffffffu, fills);
      if (lane == 0) { s_wt[1][warp] = h; s_wt[2][warp] = f; }
      __syncthreads();
      const int all_h = __reduce_add_sync(0xffffffffu, lane < NW ? s_wt[1][lane] : 0);
      const int all_f = __reduce_add_sync(0xffffffffu, lane < NW ? s_wt[2][lane] : 0);
      if (tid == 0) { s_ct[2] = all_h; s_ct[3] = all_f; }
      cluster_sync();
      const int pf = lane < cs ? peer_int(&s_ct[3], lane) : 0;
      const int ph = lane < rank ? peer_int(&s_ct[2], lane) : 0;
      moves = __reduce_add_sync(0xffffffffu, pf);
      hole_first = __reduce_add_sync(0xffffffffu, ph);
      fill_first = __reduce_add_sync(0xffffffffu, lane < rank ? pf : 0);
    }
    seen = tie_first;
    int* list = reinterpret_cast<int*>(s_key);
#pragma unroll 1
    for (int k = 0; k < tiles; ++k) {
      if (tiles > 1) word = keep_word(k, seen);
      const unsigned front = front_word(k);
      unsigned hw = ~word & front, fw = word & ~front;
      const int both = __popc(hw) | __popc(fw) << 16, upto = warp_inclusive(both, lane);
      __syncthreads();                   // keys and the last counts are no longer read
      if (lane == 31) s_wt[1][warp] = upto;
      __syncthreads();
      const int t = lane < NW ? s_wt[1][lane] : 0;  // at most 2^15 of each: no carry
      const unsigned before = (unsigned)(__reduce_add_sync(0xffffffffu, lane < warp ? (unsigned)t : 0u) + upto - both);
      const unsigned all = __reduce_add_sync(0xffffffffu, (unsigned)t);
      const int nh = all & 0xffffu, nf = all >> 16;
      const int t0 = (int)lane_at(k);
      for (int at = before & 0xffffu; hw; hw &= hw - 1) list[at++] = t0 + __ffs(hw) - 1;
      for (int at = nh + (before >> 16); fw; fw &= fw - 1) list[at++] = t0 + __ffs(fw) - 1;
      __syncthreads();
      for (int i = tid; i < nh; i += NT) hole[hole_first + i] = list[i];
      for (int i = tid; i < nf; i += NT) fill[fill_first + i] = list[nh + i];
      hole_first += nh;
      fill_first += nf;
      if (tiles > 1) __syncthreads();
    }
    if (cs == 1) moves = fill_first;
    if (cs > 1) cluster_sync();          // no CTA leaves while its counts are read
  }
  for (int i = moves + rank * NT + tid; i < a.max_move; i += cs * NT)
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

template <int NT, int CPL>
constexpr int evict_smem() { return (CPL | 1) * 16 * NT; }

template <int NT, int CPL, bool VEC>
cudaError_t run_evict(const EvictArgs& a, int cs, int tiles, cudaStream_t st) {
  constexpr int kSmem = evict_smem<NT, CPL>();
  cudaError_t e = allow_smem<evict_select_kernel<NT, CPL, VEC>>(kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.s.batch * a.n_mass) * cs);
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0] = cluster_of(cs);
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel<NT, CPL, VEC>, a, cs, tiles);
}

template <int NT, bool VEC>
cudaError_t run_evict(const EvictArgs& a, cudaStream_t st) {
  // As many CTAs a row as keep one per SM, at least one chunk a thread; longer
  // rows take more, up to the cluster's eight.  All clusters have to be resident at
  // once (16 rows of 17548 tokens, 15 clusters of eight fit: 22.9 us by eights, 14.0
  // by fours; 34 rows of 30000, 33 of four fit: 23.7 by fours, 17.2 by twos).
  const long long rows = (long long)a.s.batch * a.n_mass, L = a.s.L_ctx;
  auto fit = [&](int n) {
    return rows * n <= tc_sm_count() &&
           rows <= resident_clusters<evict_select_kernel<NT, kMaxChunks, VEC>>(n, NT, evict_smem<NT, kMaxChunks>());
  };
  int cs = 1;
  while (cs < kMaxCluster && ((fit(cs * 2) && L > 4ll * cs * NT) ||
                              L > 4ll * cs * kMaxChunks * NT))
    cs *= 2;
  const long long chunks = (L + 4ll * cs * NT - 1) / (4ll * cs * NT);
  if (chunks <= 1) return run_evict<NT, 1, VEC>(a, cs, 1, st);
  if (chunks <= 2) return run_evict<NT, 2, VEC>(a, cs, 1, st);
  if (chunks <= 4) return run_evict<NT, 4, VEC>(a, cs, 1, st);
  return run_evict<NT, kMaxChunks, VEC>(a, cs, (int)((chunks + kMaxChunks - 1) / kMaxChunks), st);
}

}  // namespace

cudaError_t launch_evict_select(const EvictArgs& a, cudaStream_t st) {
  const bool vec = a.s.L_ctx % 4 == 0 && (reinterpret_cast<uintptr_t>(a.tok_mass) & 15) == 0 &&
                   (reinterpret_cast<uintptr_t>(a.tok_pos) & 15) == 0;
  // 1024 threads a row, one CTA per SM.  Rows in more than one wave of those take
  // 512, two per SM, while one CTA holds a row (512 rows of 2112 tokens 24.3 ->
  // 14.2 us, of 8192 36.1 -> 25.6, of 16384 49.0 -> 40.4; of 32768, in clusters of
  // two, 72.3 -> 86.6; 128 rows of 2112 6.7 -> 7.6).
  if ((long long)a.s.batch * a.n_mass > tc_sm_count() && a.s.L_ctx <= 4 * kMaxChunks * 512)
    return vec ? run_evict<512, true>(a, st) : run_evict<512, false>(a, st);
  return vec ? run_evict<1024, true>(a, st) : run_evict<1024, false>(a, st);
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
    if (wide) DL_LAUNCH_DEPENDENT((cache_compact_kernel<CH_, 32>), grid, 256, 0, st, a, groups, tasks);     \
    else DL_LAUNCH_DEPENDENT((cache_compact_kernel<CH_, 8>), grid, 256, 0, st, a, groups, tasks);           \
  } while (0)
  const int pieces = s.d * (s.dtype == DL_BF16 ? 2 : 4) / 16;
  if (pieces == 8) DL_COMPACT(8);
  else if (pieces == 16) DL_COMPACT(16);
  else DL_COMPACT(32);
#undef DL_COMPACT
  return cudaGetLastError();
}

}  // namespace dl
