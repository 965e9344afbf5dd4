// (c3) The eviction plan of a cache with a budget, and (c4) its moves.
//
// Plan: the `budget` tokens of largest key stay, key = the accumulated mass
// in the order of its bits (held tokens at +infinity, NaN at -infinity),
// equal keys by the lower index.  One CTA per decision row: radix select of
// the budget-th key (four 8-bit digits from the top), then one ordered walk
// that lists the holes before the budget and the kept tokens behind it.
// Moves: a thread per 16 bytes.
#include "common.cuh"
#include "internal.h"
#include "launch.cuh"

namespace dl {

namespace {

constexpr int kEvThreads = 512;
constexpr unsigned kHeldKey = 0xFF800000u;  // the key of +infinity

// Order-preserving bits of a mass: a < b as numbers <=> key(a) < key(b);
// -0 like +0, NaN like -infinity.
__device__ __forceinline__ unsigned mass_key(float x) {
  if (x != x) x = -INFINITY;
  const unsigned u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kEvThreads) evict_select_kernel(EvictArgs a) {
  pdl_trigger();
  pdl_wait();
  __shared__ int s_hist[256], s_warp[33], s_pick[2], s_max[kEvThreads / 32];
  const Shape& s = a.s;
  const int row = blockIdx.x, b = row / a.n_mass, tid = threadIdx.x;
  const int n = a.ctx_len[b];
  const bool bad = n < 0 || n > s.L_ctx;
  if (tid == 0 && row % a.n_mass == 0) {
    if (bad) flag_error(a.err, ERR_BAD_INDEX);
    a.new_len[b] = bad ? n : min(n, a.budget);
  }
  int32_t* hole = a.hole_idx + (size_t)row * a.max_move;
  int32_t* fill = a.fill_idx + (size_t)row * a.max_move;
  int moves = 0;
  if (!bad && n > a.budget) {
    const float* mass = a.tok_mass + (size_t)row * s.L_ctx;
    const int32_t* pos = a.tok_pos ? a.tok_pos + (size_t)row * s.L_ctx : nullptr;
    int last = INT32_MIN;
    if (pos) {
      for (int t = tid; t < n; t += kEvThreads) last = max(last, pos[t]);
      last = __reduce_max_sync(0xffffffffu, last);
      if ((tid & 31) == 0) s_max[tid >> 5] = last;
      __syncthreads();
      for (int w = 0; w < kEvThreads / 32; ++w) last = max(last, s_max[w]);
    } else {
      last = n - 1;
    }
    const long long recent = (long long)last - a.n_recent;
    auto key = [&](int t) {
      const int p = pos ? pos[t] : t;
      return (p < a.n_first || p > recent) ? kHeldKey : mass_key(mass[t]);
    };
    unsigned prefix = 0, mask = 0;
    int want = a.budget;
    for (int sh = 24; sh >= 0; sh -= 8) {
      __syncthreads();
      if (tid < 256) s_hist[tid] = 0;
      __syncthreads();
      for (int t = tid; t < n; t += kEvThreads) {
        const unsigned k = key(t);
        if ((k & mask) == prefix) atomicAdd(&s_hist[(k >> sh) & 255], 1);
      }
      __syncthreads();
      if (tid == 0) {
        int d = 255;
        while (s_hist[d] < want) want -= s_hist[d--];
        s_pick[0] = d;
        s_pick[1] = want;
      }
      __syncthreads();
      prefix |= (unsigned)s_pick[0] << sh;
      mask |= 255u << sh;
      want = s_pick[1];
    }
    // keys above `prefix` stay, and the first `want` equal ones
    int ties = 0, holes = 0;
    for (int t0 = 0; t0 < n; t0 += kEvThreads) {
      const int t = t0 + tid;
      const unsigned k = t < n ? key(t) : 0u;
      int total;
      const bool tie = t < n && k == prefix;
      const int before = block_exclusive_count(tie, s_warp, &total);
      const bool keep = t < n && (k > prefix || (tie && ties + before < want));
      ties += total;
      const bool h = t < n && t < a.budget && !keep;
      const int hi = block_exclusive_count(h, s_warp, &total);
      if (h) hole[holes + hi] = t;
      holes += total;
      const bool f = keep && t >= a.budget;
      const int fi = block_exclusive_count(f, s_warp, &total);
      if (f) fill[moves + fi] = t;
      moves += total;
    }
  }
  for (int i = moves + tid; i < a.max_move; i += kEvThreads) hole[i] = fill[i] = -1;
  if (tid == 0) a.move_cnt[row] = moves;
}

// grid (move blocks, decision rows); thread = 16 bytes of a row pair
__global__ void __launch_bounds__(256) cache_compact_kernel(CompactArgs a, int row_bytes) {
  pdl_trigger();
  pdl_wait();
  const Shape& s = a.s;
  const int row = blockIdx.y, b = row / a.n_mass, m = row % a.n_mass;
  int cnt = a.move_cnt[row];
  if (cnt < 0 || cnt > a.max_move) {
    if (blockIdx.x == 0 && threadIdx.x == 0) flag_error(a.err, ERR_BAD_INDEX);
    cnt = cnt < 0 ? 0 : a.max_move;
  }
  const int chunks = row_bytes / 16;            // per row
  const int heads = a.n_mass == 1 ? s.H_kv : 1;
  const long long per = (long long)heads * chunks;
  const long long n = (long long)cnt * per;
  const int32_t* table = a.page_table + (size_t)b * s.n_pages;
  for (long long e = (long long)blockIdx.x * blockDim.x + threadIdx.x; e < n;
       e += (long long)gridDim.x * blockDim.x) {
    const int i = (int)(e / per), rest = (int)(e % per);
    const int g = a.n_mass == 1 ? rest / chunks : m, c = rest % chunks;
    const int to = a.hole_idx[(size_t)row * a.max_move + i];
    const int from = a.fill_idx[(size_t)row * a.max_move + i];
    bool ok = to >= 0 && to < s.L_ctx && from >= 0 && from < s.L_ctx;
    int st = 0, sf = 0;
    if (ok) {
      st = table[to / 64];
      sf = table[from / 64];
      ok = st >= 0 && st < s.n_slots && sf >= 0 && sf < s.n_slots;
    }
    if (!ok) {
      if (rest == 0) flag_error(a.err, ERR_BAD_INDEX);
      continue;
    }
    const size_t dst = (((size_t)st * s.H_kv + g) * 64 + to % 64) * chunks + c;
    const size_t src = (((size_t)sf * s.H_kv + g) * 64 + from % 64) * chunks + c;
    reinterpret_cast<uint4*>(a.Kp)[dst] = reinterpret_cast<const uint4*>(a.Kp)[src];
    reinterpret_cast<uint4*>(a.Vp)[dst] = reinterpret_cast<const uint4*>(a.Vp)[src];
    if (rest == 0) {
      const size_t o = (size_t)row * s.L_ctx;
      if (a.tok_pos) a.tok_pos[o + to] = a.tok_pos[o + from];
      if (a.tok_mass) a.tok_mass[o + to] = a.tok_mass[o + from];
    }
  }
}

}  // namespace

cudaError_t launch_evict_select(const EvictArgs& a, cudaStream_t st) {
  DL_LAUNCH(evict_select_kernel, a.s.batch * a.n_mass, kEvThreads, 0, st, a);
  return cudaGetLastError();
}

cudaError_t launch_cache_compact(const CompactArgs& a, cudaStream_t st) {
  if (a.max_move == 0) return cudaSuccess;
  const int row_bytes = a.s.d * (a.s.dtype == DL_BF16 ? 2 : 4);
  DL_LAUNCH(cache_compact_kernel, dim3(min((a.max_move + 7) / 8, 64), a.s.batch * a.n_mass), 256, 0,
            st, a, row_bytes);
  return cudaGetLastError();
}

}  // namespace dl
