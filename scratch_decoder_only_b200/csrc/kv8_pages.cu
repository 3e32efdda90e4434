// The pages of the 8-bit key/value cache: growing rows, forking, freeing and
// compacting them, all decided on the device (include/gpt.h).
//
// Free pages are the zeros of ref[n_pages]; a request takes the k-th lowest
// one.  One cluster of eight blocks reads ref once to count the zeros of every
// 1024 pages, the blocks in turn (the lowest pages are wanted, so slices would
// leave the first block with all the work); the counts meet through distributed
// shared memory, and the pages whose ranks are wanted are looked at again: page
// number k goes to the request of that rank, found by bisection in the requests'
// running sums.  Every launch reads the whole of ref (4 bytes a page; a pool of
// 100,000 pages is 0.4 MB in L2) and nothing depends on an earlier call, so any
// table that a host writes is as good as one that these kernels made.  What
// bounds them is latency: the launch, the barriers between the phases and the
// trips to memory, not the bytes.
#include <cooperative_groups.h>
#include <algorithm>
#include <string>
#include "kv8.cuh"

namespace cg = cooperative_groups;

#define KVP_CTAS 8
#define KVP_THREADS 1024
#define KVP_MAX 16384        // requests a call
#define KVP_PAGES (1 << 24)   // pages of a pool

struct Kv8PoolP {
  int *table, *lens, *ref;
  int n_rows, max_pages, ld_table, n_pages, lp;
  unsigned* err;
};

// Exclusive sum over the block in thread order; total: of the whole block.  Where
// sums may pass 32 bits, v <= cap <= 2^25 and what matters of a sum is only whether
// it reaches cap: a warp's sum (below 2^30) counts as cap at most, so the results
// are below 2^31, right where the true sum is below cap and at least cap elsewhere.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int& total, int cap = 0x7fffffff) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, k);
    if (lane >= k) inc += y;
  }
  __syncthreads();   // the sums of an earlier call have been read
  if (lane == 31) warp_sums[warp] = min(inc, cap);
  __syncthreads();
  int w = warp_sums[lane];
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, w, k);
    if (lane >= k) w += y;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const int before = __shfl_sync(0xffffffffu, w, warp ? warp - 1 : 0);
  return (warp ? before : 0) + inc - v;
}

// This block's slice of the pages, and four pages of it: bit i of the result
// is set where page i0 + i is in the slice and (live) in use or (!live) free.
struct Slice {
  int a, b;
};
__device__ __forceinline__ Slice kvp_slice(int n, int rank) {
  const int per = ((n + KVP_CTAS - 1) / KVP_CTAS + 3) & ~3;
  return {min(n, rank * per), min(n, (rank + 1) * per)};
}
__device__ __forceinline__ unsigned kvp_mask(const int* ref, int i0, int end, bool live) {
  unsigned m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i0 + i < end && (ref[i0 + i] > 0) == live) m |= 1u << i;
  return m;
}

// Each block's value v, as the sum over the blocks before this one and over all.
__device__ __forceinline__ int cluster_sum(cg::cluster_group& cl, int* slot, int v, int& total) {
  if (threadIdx.x == 0) *slot = v;
  cl.sync();
  int before = 0, all = 0;
  for (int r = 0; r < KVP_CTAS; ++r) {
    const int x = *cl.map_shared_rank(slot, r);
    before += r < (int)cl.block_rank() ? x : 0;
    all += x;
  }
  total = all;
  return before;
}

// FORK = false: request i grows row i by add[i].  FORK = true: request i makes
// row dst[i] a copy of row src[i].  Both need pages; fork's copies of them
// follow in kvp_fork_copy_kernel.
//
// Forks to the same row: the claims are negative numbers put into lens[dst]
// (0 while empty) with a minimum, so the first pair wins whatever the order of
// the threads; the row's length replaces the claim at the end.
template <bool FORK>
__global__ void __cluster_dims__(KVP_CTAS, 1, 1) __launch_bounds__(KVP_THREADS)
    kvp_grow_kernel(Kv8PoolP p, const int* __restrict__ add, const int* __restrict__ src, const int* __restrict__ dst,
                    int n, int* __restrict__ done) {
  griddep_wait();
  griddep_release();
  // [n + 1] running sum of the pages needed, [n] the place in the row of a request's first page, [chunks] free
  // pages of each 1024, then those before it
  extern __shared__ int first[];
  __shared__ int wsum[32], sflag;
  cg::cluster_group cl = cg::this_cluster();
  const int rank = cl.block_rank(), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int P1 = (1 << p.lp) - 1, claim0 = -0x7fffffff, chunks = (p.n_pages + KVP_THREADS - 1) / KVP_THREADS;
  int *place = first + n + 1, *chunk = place + n;
  if (FORK && rank == 0) {
    for (int i = tid; i < n; i += KVP_THREADS) {
      const int a = src[i], z = dst[i];
      first[i] = (unsigned)a < (unsigned)p.n_rows && (unsigned)z < (unsigned)p.n_rows && p.lens[z] == 0;
    }
    __syncthreads();
    for (int i = tid; i < n; i += KVP_THREADS)
      if (first[i]) atomicMin(&p.lens[dst[i]], claim0 + i);
    __threadfence();
  }
  if (FORK) cl.sync();   // the claims are there
  // ---- pages that each request needs (an invalid one: none); all sums end at one more page than there are, for
  // rows may ask for 2^27 each
  const int cap = p.n_pages + 1;
  int carry = 0;
  bool bad_pos = false;
  for (int i0 = 0; i0 < n; i0 += KVP_THREADS) {
    const int i = i0 + tid;
    int need = 0, at = 0;
    if (i < n) {
      if (FORK) {
        const int z = dst[i], a = src[i];
        if ((unsigned)z < (unsigned)p.n_rows && (unsigned)a < (unsigned)p.n_rows && p.lens[z] == claim0 + i) {
          const int len = p.lens[a];
          at = max(len, 0) >> p.lp;
          need = len > 0 && (len & P1) && at < p.max_pages;
        }
      } else {
        const int len = p.lens[i], ad = add[i];
        const long want = (long)len + ad;
        if (ad < 0 || len < 0 || want > ((long)p.max_pages << p.lp)) {
          bad_pos = true;
        } else {
          at = (len + P1) >> p.lp;
          need = min((int)((want + P1) >> p.lp) - at, cap);
        }
      }
    }
    int tot;
    const int ex = block_scan(need, wsum, tot, cap);
    if (i < n) {
      first[i] = min(carry + ex, cap);
      place[i] = at;
    }
    carry = min(carry + tot, cap);
  }
  if (tid == 0) first[n] = carry;
  if (bad_pos && rank == 0) set_dev_err(p.err, GPT_DEVERR_POS);
  __syncthreads();
  const int total = carry;

  int avail = 0x7fffffff;
  if (total > 0) {   // (as in 15 of 16 decode steps it is not)
    // ---- free pages of this block's chunks, then of all of them
    for (int c = rank + tid * KVP_CTAS; c < chunks; c += KVP_CTAS * KVP_THREADS) chunk[c] = 0;
    __syncthreads();
    for (int c0 = rank; c0 < chunks; c0 += 8 * KVP_CTAS) {
      int r[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int id = (c0 + i * KVP_CTAS) * KVP_THREADS + tid;
        r[i] = id < p.n_pages ? p.ref[id] : 1;   // (n_pages <= 2^24: no overflow)
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const unsigned m = __ballot_sync(0xffffffffu, r[i] <= 0);
        if (lane == 0 && m) atomicAdd(&chunk[c0 + i * KVP_CTAS], __popc(m));
      }
    }
    cl.sync();   // the counts are there
    for (int c = tid; c < chunks; c += KVP_THREADS)
      if (c % KVP_CTAS != rank) chunk[c] = *cl.map_shared_rank(chunk + c, c % KVP_CTAS);
    cl.sync();   // the blocks have each other's: they may be overwritten
    // ---- free pages before each chunk, and in all
    avail = 0;
    for (int c0 = 0; c0 < chunks; c0 += KVP_THREADS) {
      const int c = c0 + tid;
      int tot;
      const int ex = block_scan(c < chunks ? chunk[c] : 0, wsum, tot);
      if (c < chunks) chunk[c] = avail + ex;
      avail += tot;
    }
    __syncthreads();
    // ---- page number k of the pool goes to the request that holds rank k
    for (int c = rank; c < chunks && chunk[c] < total; c += KVP_CTAS) {
      const int id = c * KVP_THREADS + tid;
      const bool free = id < p.n_pages && p.ref[id] <= 0;
      const unsigned m = __ballot_sync(0xffffffffu, free);
      __syncthreads();
      if (lane == 0) wsum[warp] = __popc(m);
      __syncthreads();
      int k = chunk[c] + __popc(m & ((1u << lane) - 1));
      // the warps before this one
      const int w = lane < warp ? wsum[lane] : 0;
      k += __reduce_add_sync(0xffffffffu, w);
      if (!free || k >= total) continue;
      int lo = 0, hi = n - 1;   // the last request with first <= k
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= k) lo = mid;
        else hi = mid - 1;
      }
      if (first[lo + 1] > avail) continue;   // not served
      const int r = FORK ? dst[lo] : lo;
      p.table[(long)r * p.ld_table + place[lo] + k - first[lo]] = id;
      p.ref[id] = 1;
    }
  }
  // ---- whole pages of the forks: shared
  if (FORK) {
    const int warps = KVP_CTAS * (KVP_THREADS / 32), w = rank * (KVP_THREADS / 32) + warp;
    for (int i = w; i < n; i += warps) {
      const int a = src[i], z = dst[i];
      if ((unsigned)a >= (unsigned)p.n_rows || (unsigned)z >= (unsigned)p.n_rows || p.lens[z] != claim0 + i) continue;
      if (first[i + 1] > first[i] && first[i + 1] > avail) continue;
      const int full = min(place[i], p.max_pages);
      for (int j = lane; j < full; j += 32) {
        const int id = p.table[(long)a * p.ld_table + j];
        p.table[(long)z * p.ld_table + j] = id;
        if ((unsigned)id < (unsigned)p.n_pages) atomicAdd(&p.ref[id], 1);
        else set_dev_err(p.err, GPT_DEVERR_PAGE);
      }
    }
  }
  cl.sync();   // every block has read the lengths
  if (rank) return;
  // ---- the new lengths
  if (tid == 0) sflag = 0;
  __syncthreads();
  if (FORK) {
    // every fork's length first (a source that is another fork's target counts
    // as empty: its claim is negative), then the claims are replaced
    for (int i = tid; i < n; i += KVP_THREADS) {
      const int a = src[i], z = dst[i];
      int len = -1;
      if ((unsigned)a < (unsigned)p.n_rows && (unsigned)z < (unsigned)p.n_rows && p.lens[z] == claim0 + i) {
        len = max(p.lens[a], 0);
        if (first[i + 1] > first[i] && first[i + 1] > avail) len = -2;   // no page for it: the row is empty again
      }
      if (len < 0) sflag = 1;
      done[i] = len;
    }
    __syncthreads();
    for (int i = tid; i < n; i += KVP_THREADS) {
      const int len = done[i];
      if (len >= 0) p.lens[dst[i]] = len;
      else if (len == -2) p.lens[dst[i]] = 0;
      done[i] = len >= 0;
    }
  } else {
    for (int i = tid; i < n; i += KVP_THREADS) {
      const int ad = add[i], len = p.lens[i];
      const long want = (long)len + ad;
      if (ad < 0 || len < 0 || want > ((long)p.max_pages << p.lp)) continue;
      // (whether it needs pages the capped sums do not tell)
      if ((want + P1) >> p.lp > (len + P1) >> p.lp && first[i + 1] > avail) sflag = 1;
      else p.lens[i] = len + ad;
    }
    __syncthreads();
  }
  if (tid == 0 && sflag) set_dev_err(p.err, GPT_DEVERR_PAGE);
}

// ---- copies of whole pages, all layers
struct Kv8CopyP {
  uint8_t *k, *v;
  float *ks, *vs;
  long layer_pages;    // n_pages
  int layers, Hkv;
  int bytes;           // of one page in one layer (all heads), a multiple of 256
};
#define KVP_CHUNK 16384   // bytes a block copies: 256 threads x 4 vectors of 16

// A copy of up to KVP_CHUNK bytes by 256 threads, in two halves, so that the next
// one's loads are under way while this one's stores are issued.
struct KvpChunk {
  uint4 r[4];
  uint4* to;
  int n;   // vectors
};
// Chunk `sub` = (layer * 2 + is_v) * chunks + chunk of page a, to go to page z; the
// first chunk takes the scales along.
__device__ __forceinline__ void kvp_load(KvpChunk& k, const Kv8CopyP& c, int a, int z, int sub, int chunks) {
  const int chunk = sub % chunks, lv = sub / chunks, layer = lv >> 1;
  const bool is_v = lv & 1;
  const long pa = (long)layer * c.layer_pages + a, pz = (long)layer * c.layer_pages + z;
  uint8_t* x = is_v ? c.v : c.k;
  const uint4* from = reinterpret_cast<const uint4*>(x + pa * c.bytes + (long)chunk * KVP_CHUNK) + threadIdx.x;
  k.to = reinterpret_cast<uint4*>(x + pz * c.bytes + (long)chunk * KVP_CHUNK) + threadIdx.x;
  k.n = (min(c.bytes - chunk * KVP_CHUNK, KVP_CHUNK) / 16 - (int)threadIdx.x + 255) / 256;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < k.n) k.r[j] = from[256 * j];
  if (chunk == 0) {
    float* s = is_v ? c.vs : c.ks;
    for (int h = threadIdx.x; h < c.Hkv; h += 256) s[pz * c.Hkv + h] = s[pa * c.Hkv + h];
  }
}
__device__ __forceinline__ void kvp_store(const KvpChunk& k) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < k.n) k.to[256 * j] = k.r[j];
}

// The part-filled last pages of the forks: gridDim.x blocks per pair share its
// layers, keys and values.
__global__ void __launch_bounds__(256) kvp_fork_copy_kernel(Kv8PoolP p, Kv8CopyP c, const int* __restrict__ src,
                                                            const int* __restrict__ dst, const int* __restrict__ done,
                                                            int chunks) {
  griddep_wait();
  griddep_release();
  const int i = blockIdx.y;
  if (!done[i]) return;
  const int len = p.lens[dst[i]], last = len >> p.lp;
  if (!(len & ((1 << p.lp) - 1)) || last >= p.max_pages) return;
  const int a = p.table[(long)src[i] * p.ld_table + last], z = p.table[(long)dst[i] * p.ld_table + last];
  if ((unsigned)a >= (unsigned)p.n_pages || (unsigned)z >= (unsigned)p.n_pages) {
    if (threadIdx.x == 0) set_dev_err(p.err, GPT_DEVERR_PAGE);
    return;
  }
  const int subs = 2 * c.layers * chunks;
  KvpChunk now, next;
  if (blockIdx.x < subs) kvp_load(now, c, a, z, blockIdx.x, chunks);
  for (int sub = blockIdx.x; sub < subs; sub += gridDim.x) {
    if (sub + gridDim.x < subs) kvp_load(next, c, a, z, sub + gridDim.x, chunks);
    kvp_store(now);
    now = next;
  }
}

// ---- free: one block per listed row.  The exchange of the length gives the
// row to one of the blocks that list it.
__global__ void __launch_bounds__(128) kvp_free_kernel(Kv8PoolP p, const int* __restrict__ rows) {
  griddep_wait();
  griddep_release();
  __shared__ int slen;
  const int r = rows[blockIdx.x];
  if ((unsigned)r >= (unsigned)p.n_rows) {
    if (threadIdx.x == 0) set_dev_err(p.err, GPT_DEVERR_PAGE);
    return;
  }
  if (threadIdx.x == 0) slen = atomicExch(&p.lens[r], 0);
  __syncthreads();
  const int n = min((max(slen, 0) + (1 << p.lp) - 1) >> p.lp, p.max_pages);
  int* row = p.table + (long)r * p.ld_table;
  for (int j = threadIdx.x; j < n; j += 128) {
    const int id = row[j];
    row[j] = -1;
    if ((unsigned)id >= (unsigned)p.n_pages) set_dev_err(p.err, GPT_DEVERR_PAGE);
    else if (atomicSub(&p.ref[id], 1) <= 0) {
      atomicAdd(&p.ref[id], 1);   // nobody held it
      set_dev_err(p.err, GPT_DEVERR_PAGE);
    }
  }
}

// ---- compaction.  work: n_live, the number of moves, then (from entry 8 on)
// from[k], the k-th used page from n_live on, and to[k], the k-th hole below it,
// n_pages / 2 entries each (there are no more moves than that), then the move
// of each page.
__global__ void __cluster_dims__(KVP_CTAS, 1, 1) __launch_bounds__(KVP_THREADS)
    kvp_plan_kernel(Kv8PoolP p, int64_t* __restrict__ n_live, int* __restrict__ work) {
  griddep_wait();
  griddep_release();
  __shared__ int wsum[32], slot[2];
  cg::cluster_group cl = cg::this_cluster();
  const int rank = cl.block_rank(), tid = threadIdx.x, n = p.n_pages, half = n / 2;
  int *from = work + 8, *to = from + half, *move = to + half;
  const Slice sl = kvp_slice(n, rank);
  int cnt = 0, mine, live;
  for (int i = sl.a + 4 * tid; i < sl.b; i += 4 * KVP_THREADS) cnt += __popc(kvp_mask(p.ref, i, sl.b, true));
  block_scan(cnt, wsum, mine);
  const int before = cluster_sum(cl, &slot[0], mine, live);
  // Ranks follow from the used pages before a place: hole i is number
  // i - used(i) of the holes, mover i number used(i) - used(live) of the movers.
  int below = 0;   // used(live)
  cnt = 0;
  for (int i = sl.a + 4 * tid; i < min(sl.b, live); i += 4 * KVP_THREADS)
    cnt += __popc(kvp_mask(p.ref, i, min(sl.b, live), true));
  block_scan(cnt, wsum, mine);
  cluster_sum(cl, &slot[1], mine, below);
  const int moves = live - below;
  if (rank == 0 && tid == 0) {
    work[0] = live;
    work[1] = moves;
    if (n_live) *n_live = live;
  }
  int base = before;
  for (int i0 = sl.a; i0 < sl.b; i0 += 4 * KVP_THREADS) {
    const int i = i0 + 4 * tid;
    const unsigned m = i < sl.b ? kvp_mask(p.ref, i, sl.b, true) : 0u;
    int tot;
    int used = base + block_scan(__popc(m), wsum, tot);
    for (int e = 0; e < 4 && i + e < sl.b; ++e) {
      const int id = i + e;
      const bool on = m >> e & 1;
      if (id < live && !on) to[id - used] = id;
      if (id >= live && on) {
        from[used - below] = id;
        move[id] = used - below;
      }
      used += on;
    }
    base += tot;
  }
  cl.sync();   // no block leaves while another reads its shared memory
}

// The moves: blocks first follow them in the rows' tables, then copy pages.
__global__ void __launch_bounds__(256) kvp_move_kernel(Kv8PoolP p, Kv8CopyP c, const int* __restrict__ work,
                                                       int chunks) {
  griddep_wait();
  griddep_release();
  const int live = work[0], moves = work[1], half = p.n_pages / 2;
  const int *from = work + 8, *to = from + half, *move = to + half;
  for (int r = blockIdx.x; r < p.n_rows; r += gridDim.x) {
    const int n = min((max(p.lens[r], 0) + (1 << p.lp) - 1) >> p.lp, p.max_pages);
    int* row = p.table + (long)r * p.ld_table;
    for (int j = threadIdx.x; j < n; j += 256) {
      const int id = row[j];
      if (id >= 0 && id < live) continue;
      const int k = (unsigned)id < (unsigned)p.n_pages ? move[id] : -1;
      if ((unsigned)k < (unsigned)moves && from[k] == id) row[j] = to[k];
      else set_dev_err(p.err, GPT_DEVERR_PAGE);   // a page that nobody is said to hold
    }
  }
  const int per = 2 * c.layers * chunks;
  const long jobs = (long)moves * per;
  KvpChunk now, next;
  auto load = [&](KvpChunk& k, long i) {
    const int m = (int)(i / per), sub = (int)(i % per), a = from[m], z = to[m];
    if (sub == 0 && threadIdx.x == 0) {
      p.ref[z] = p.ref[a];
      p.ref[a] = 0;
    }
    kvp_load(k, c, a, z, sub, chunks);
  };
  if (blockIdx.x < jobs) load(now, blockIdx.x);
  for (long i = blockIdx.x; i < jobs; i += gridDim.x) {
    if (i + gridDim.x < jobs) load(next, i + gridDim.x);
    kvp_store(now);
    now = next;
  }
}

// ---------------------------------------------------------------------------
// Entry points
// ---------------------------------------------------------------------------
static int kvp_refuse(const char* what, const char* why) {
  set_global_error((std::string(what) + ": " + why).c_str());
  return GPT_ERR_ARG;
}
static int kvp_done(const char* what, cudaError_t e) {
  if (e == cudaSuccess) return GPT_OK;
  set_global_error((std::string(what) + ": " + cudaGetErrorString(e)).c_str());
  return GPT_ERR_CUDA;
}

static const char* kvp_check(const gpt_kv8_pool* p) {
  if (!p) return "pool is NULL";
  if (!p->table || !p->lens || !p->ref) return "table, lens and ref must be non-NULL";
  if (p->page != 16 && p->page != 32 && p->page != 64 && p->page != 128) return "page must be 16, 32, 64 or 128";
  if (p->n_rows < 1 || p->n_rows > KVP_MAX) return "n_rows out of range [1, 16384]";
  if (p->n_pages < 1 || p->n_pages > KVP_PAGES) return "n_pages out of range [1, 2^24]";
  if (p->max_pages < 1 || p->ld_table < p->max_pages || (long)p->max_pages * p->page > 0x7fffff00L)
    return "need 1 <= max_pages <= ld_table and max_pages * page < 2^31";
  return "";
}
static const char* kvp_check_cache(const gpt_kv8_pool* p, const gpt_kv8_cache* c) {
  const char* why = kv8_check_cache(c);
  if (*why) return why;
  if (c->n_pages != p->n_pages || c->page != p->page) return "cache and pool differ in n_pages or page";
  return "";
}
static Kv8PoolP kvp_pool(const gpt_kv8_pool& p, uint32_t* err) {
  return {p.table, p.lens, p.ref, p.n_rows, p.max_pages, p.ld_table, p.n_pages, ilog2(p.page), err};
}
static Kv8CopyP kvp_copy(const gpt_kv8_cache& c) {
  return {(uint8_t*)c.k, (uint8_t*)c.v, c.k_scale, c.v_scale, c.n_pages, c.n_layers, c.n_kv_heads,
          c.n_kv_heads * c.page * c.head_dim};
}

template <bool FORK>
static cudaError_t kvp_grow(const Kv8PoolP& p, const int* add, const int* src, const int* dst, int n, int* done,
                            cudaStream_t s) {
  const size_t smem = (2 * (size_t)n + 1 + (p.n_pages + KVP_THREADS - 1) / KVP_THREADS) * sizeof(int);
  if (smem > 40000) {
    const cudaError_t e = cudaFuncSetAttribute(kvp_grow_kernel<FORK>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (2 * KVP_MAX + 1 + KVP_PAGES / KVP_THREADS) * (int)sizeof(int));
    if (e != cudaSuccess) return e;
  }
  ++g_kernel_launches;
  return launch_k(kvp_grow_kernel<FORK>, dim3(KVP_CTAS), dim3(KVP_THREADS), smem, s, p, add, src, dst, n, done);
}

extern "C" {

int gpt_kv8_extend(const gpt_kv8_pool* p, const int32_t* add, uint32_t* err, void* stream) {
  const char* why = kvp_check(p);
  if (!*why && !add) why = "add is NULL";
  if (*why) return kvp_refuse("gpt_kv8_extend", why);
  return kvp_done("gpt_kv8_extend", kvp_grow<false>(kvp_pool(*p, err), add, nullptr, nullptr, p->n_rows, nullptr,
                                                    (cudaStream_t)stream));
}

int gpt_kv8_fork(const gpt_kv8_pool* p, const gpt_kv8_cache* c, const int32_t* src, const int32_t* dst, int n,
                 int32_t* done, uint32_t* err, void* stream) {
  const char* why = kvp_check(p);
  if (!*why) why = kvp_check_cache(p, c);
  if (!*why && (n < 0 || n > KVP_MAX)) why = "n out of range [0, 16384]";
  if (!*why && n && (!src || !dst || !done)) why = "src, dst and done must be non-NULL";
  if (*why) return kvp_refuse("gpt_kv8_fork", why);
  if (n == 0) return GPT_OK;
  const Kv8PoolP P = kvp_pool(*p, err);
  const Kv8CopyP C = kvp_copy(*c);
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = kvp_grow<true>(P, nullptr, src, dst, n, done, s);
  if (e != cudaSuccess) return kvp_done("gpt_kv8_fork", e);
  const int chunks = (C.bytes + KVP_CHUNK - 1) / KVP_CHUNK, subs = 2 * C.layers * chunks;
  // two waves of eight blocks an SM: a block looks its pages up once for all that it copies
  const int share = std::max(1, std::min(subs, kv8_sms() * 16 / n));
  ++g_kernel_launches;
  return kvp_done("gpt_kv8_fork", launch_k(kvp_fork_copy_kernel, dim3((unsigned)share, n), dim3(256), 0, s, P, C, src,
                                           dst, (const int*)done, chunks));
}

int gpt_kv8_free(const gpt_kv8_pool* p, const int32_t* rows, int n, uint32_t* err, void* stream) {
  const char* why = kvp_check(p);
  if (!*why && (n < 0 || (n && !rows))) why = "need n >= 0 and rows non-NULL";
  if (*why) return kvp_refuse("gpt_kv8_free", why);
  if (n == 0) return GPT_OK;
  ++g_kernel_launches;
  return kvp_done("gpt_kv8_free",
                  launch_k(kvp_free_kernel, dim3(n), dim3(128), 0, (cudaStream_t)stream, kvp_pool(*p, err), rows));
}

int gpt_kv8_compact(const gpt_kv8_pool* p, const gpt_kv8_cache* c, int64_t* n_live, int32_t* work, uint32_t* err,
                    void* stream) {
  const char* why = kvp_check(p);
  if (!*why) why = kvp_check_cache(p, c);
  if (!*why && !work) why = "work is NULL";
  if (!*why && ((uintptr_t)n_live & 7)) why = "n_live must be 8-byte aligned";
  if (*why) return kvp_refuse("gpt_kv8_compact", why);
  const Kv8PoolP P = kvp_pool(*p, err);
  const Kv8CopyP C = kvp_copy(*c);
  cudaStream_t s = (cudaStream_t)stream;
  ++g_kernel_launches;
  cudaError_t e = launch_k(kvp_plan_kernel, dim3(KVP_CTAS), dim3(KVP_THREADS), 0, s, P, n_live, work);
  if (e != cudaSuccess) return kvp_done("gpt_kv8_compact", e);
  const int chunks = (C.bytes + KVP_CHUNK - 1) / KVP_CHUNK;
  ++g_kernel_launches;
  return kvp_done("gpt_kv8_compact",
                  launch_k(kvp_move_kernel, dim3(kv8_sms() * 6), dim3(256), 0, s, P, C, (const int*)work, chunks));
}

}  // extern "C"
