// The 8-bit paged key/value cache: quantising new tokens into it, reading
// tokens back, and attention over it (include/gpt.h has the definitions).
#include <float.h>
#include <math.h>
#include <algorithm>
#include <string>
#include <type_traits>
#include "kv8.cuh"

// The part of a sequence that an append or read job covers: unit `unit` of
// 1 << lu tokens (a page, or 16 tokens), slots [lo, hi) of it, the row of the
// call's matrices that holds slot lo.  All threads of the block call this.
struct Kv8Unit {
  int b, unit, lo, hi, row;
};
__device__ __forceinline__ bool kv8_unit(const Kv8Seqs& q, int job, int lu, int cap, Kv8Unit& u, unsigned* err) {
  Kv8Seq s;
  int off = 0;
  if (q.start) {
    // a sequence of n tokens touches at most floor(n / 2^lu) + 2 units
    if (!kv8_find(q, job, [lu](int b, int s0) { return (s0 >> lu) + 2 * b; }, s, off, err) || s.n == 0) return false;
  } else {
    s.b = job; s.s0 = job; s.n = 1; s.len = q.lens[job];
  }
  if (off == 0 && threadIdx.x == 0 && (s.len < s.n || s.len > cap)) set_dev_err(err, GPT_DEVERR_POS);
  const int p0 = max(s.len - s.n, 0), p1 = min(s.len, cap);
  u.b = s.b;
  u.unit = (p0 >> lu) + off;
  const int base = u.unit << lu;
  u.lo = max(p0 - base, 0);
  u.hi = min(p1 - base, 1 << lu);
  u.row = s.s0 + s.n - s.len + base + u.lo;
  return u.lo < u.hi;
}
static int kv8_jobs(const gpt_kv8_batch& b, int lu) { return b.start ? (b.rows >> lu) + 2 * b.B : b.B; }

__device__ __forceinline__ int kv8_page(const Kv8Seqs& q, const Kv8Layer& L, int b, int page, unsigned* err) {
  const int id = q.table[(long)b * q.ld_table + page];
  if ((unsigned)id < (unsigned)L.n_pages) return id;
  set_dev_err(err, GPT_DEVERR_PAGE);
  return -1;
}

// ---------------------------------------------------------------------------
// Append.  One block of 128 threads per (page touched, head, keys | values).
// The page's new rows stay in registers (VPT 16-byte vectors a thread) between
// their largest magnitude (an unsigned 16-bit maximum over the bit patterns
// without the sign, in which infinities and NaNs are the largest) and their
// codes, so every input byte is read once.  Value codes are turned over through
// shared memory: 16 tokens of a channel leave in one 16-byte store.  The work
// is a copy with a maximum; bytes bound it, for single tokens the launch does.
// ---------------------------------------------------------------------------
struct Kv8AppendP {
  Kv8Layer L;
  Kv8Seqs q;
  const uint16_t *k, *v;
  long ldk, ldv;
  unsigned* err;
};

#define KV8_PAD 8   // bytes behind each token's codes in the turning buffer

template <typename T>
__device__ __forceinline__ float bits16_f(unsigned b) {
  const unsigned short u = (unsigned short)b;
  return to_f(*reinterpret_cast<const T*>(&u));
}

// one 16-byte vector of values times inv, as eight codes
template <typename T, int KIND>
__device__ __forceinline__ uint2 kv8_code8(const uint4& x, float inv) {
  float f[8];
  Vec<T>::load(reinterpret_cast<const T*>(&x), f);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] *= inv;
  return make_uint2(kv8_code4<KIND>(f[0], f[1], f[2], f[3]), kv8_code4<KIND>(f[4], f[5], f[6], f[7]));
}
// four codes times ratio (at most 1), rounded anew
template <int KIND>
__device__ __forceinline__ uint32_t kv8_recode4(uint32_t w, float ratio) {
  uint32_t lo, hi;
  kv8_widen<KIND>(w, lo, hi);
  const float2 a = f16x2_float(lo), b = f16x2_float(hi);
  return kv8_code4<KIND>(a.x * ratio, a.y * ratio, b.x * ratio, b.y * ratio);
}

template <typename T, int KIND, int VPT>
__global__ void __launch_bounds__(128) kv8_append_kernel(Kv8AppendP p) {
  griddep_wait();
  griddep_release();
  extern __shared__ __align__(16) uint8_t turn[];   // value codes [P][D + KV8_PAD]
  __shared__ unsigned wmax[4];
  const Kv8Layer& L = p.L;
  const int tid = threadIdx.x, h = blockIdx.y, lp = L.lp, ld = L.ld, D = 1 << ld;
  const bool is_v = blockIdx.z != 0;
  Kv8Unit u;
  if (!kv8_unit(p.q, blockIdx.x, lp, p.q.max_pages << lp, u, p.err)) return;
  const int id = kv8_page(p.q, L, u.b, u.unit, p.err);
  if (id < 0) return;
  const long ldx = is_v ? p.ldv : p.ldk;
  const uint16_t* x = (is_v ? p.v : p.k) + (long)u.row * ldx + (h << ld);
  const int nv = (u.hi - u.lo) << (ld - 3);
  uint4 r[VPT];
  unsigned mx = 0;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int i = tid + j * 128;
    r[j] = i < nv ? *reinterpret_cast<const uint4*>(x + (long)(i >> (ld - 3)) * ldx + ((i & ((D >> 3) - 1)) << 3))
                  : make_uint4(0, 0, 0, 0);
  }
  const size_t ph = (size_t)id * L.Hkv + h;
  float* sp = (is_v ? L.vs : L.ks) + ph;
  const float s_old = u.lo > 0 ? *sp : 0.f;   // read by all before the barrier, written behind it
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const unsigned a = __vmaxu2(__vmaxu2(r[j].x & 0x7fff7fffu, r[j].y & 0x7fff7fffu),
                                __vmaxu2(r[j].z & 0x7fff7fffu, r[j].w & 0x7fff7fffu));
    mx = max(mx, max(a & 0xffffu, a >> 16));
  }
  mx = __reduce_max_sync(0xffffffffu, mx);
  if ((tid & 31) == 0) wmax[tid >> 5] = mx;
  __syncthreads();
  mx = max(max(wmax[0], wmax[1]), max(wmax[2], wmax[3]));
  constexpr float TOP = KIND == GPT_KV8_INT8 ? 127.f : 448.f;
  const float a = bits16_f<T>(mx);
  float s = a / TOP;
  if (s < FLT_MIN) s = 0.f;             // 1 / s would overflow
  if (s_old > s) s = s_old;
  if (!(a <= FLT_MAX) || s_old != s_old) s = NAN;
  const bool live = s > 0.f;            // false for 0 and NaN: every code of the page is 0
  const float inv = live ? 1.f / s : 0.f;
  const bool recode = u.lo > 0 && s != s_old;
  const float ratio = live ? s_old / s : 0.f;
  if (tid == 0) *sp = s;
  uint8_t* page = (is_v ? L.v : L.k) + (ph << (lp + ld));
  if (!is_v) {
    if (recode) {
      uint32_t* o = reinterpret_cast<uint32_t*>(page);
      for (int i = tid; i < (u.lo << (ld - 2)); i += 128) o[i] = live ? kv8_recode4<KIND>(o[i], ratio) : 0u;
    }
    uint2* o = reinterpret_cast<uint2*>(page + (u.lo << ld));
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int i = tid + j * 128;
      if (i < nv) o[i] = live ? kv8_code8<T, KIND>(r[j], inv) : make_uint2(0, 0);
    }
    return;
  }
  const int row = D + KV8_PAD;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int i = tid + j * 128;
    if (i < nv)
      *reinterpret_cast<uint2*>(turn + (u.lo + (i >> (ld - 3))) * row + ((i & ((D >> 3) - 1)) << 3)) =
          live ? kv8_code8<T, KIND>(r[j], inv) : make_uint2(0, 0);
  }
  __syncthreads();
  // 16-token groups that change: those with new tokens, all earlier ones too when the scale grew
  const int g0 = recode ? 0 : u.lo >> 4, g1 = (u.hi + 15) >> 4;
  uint4* o = reinterpret_cast<uint4*>(page);
  for (int i = (g0 << ld) + tid; i < (g1 << ld); i += 128) {
    const int t0 = (i >> ld) << 4, d = i & (D - 1);
    uint32_t w[4] = {0, 0, 0, 0};
    if (t0 < u.lo) {
      const uint4 old = o[i];
      w[0] = old.x; w[1] = old.y; w[2] = old.z; w[3] = old.w;
      if (recode) {
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = live ? kv8_recode4<KIND>(w[q], ratio) : 0u;
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t n = 0, keep = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = t0 + 4 * q + e;
        if (t < u.lo) keep |= 0xffu << (8 * e);
        else if (t < u.hi) n |= (uint32_t)turn[t * row + d] << (8 * e);
      }
      w[q] = (w[q] & keep) | n;
    }
    o[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// ---------------------------------------------------------------------------
// Read back.  One block of 128 threads per (16 tokens, 128 channels of the
// concatenated heads, keys | values), one 16-byte load of codes a thread:
// 16 channels of a token (keys), or 16 tokens of a channel, turned over through
// shared memory (values).
// ---------------------------------------------------------------------------
struct Kv8ReadP {
  Kv8Layer L;
  Kv8Seqs q;
  uint16_t *k, *v;
  long ldk, ldv;
  unsigned* err;
};

template <typename T, int KIND>
__global__ void __launch_bounds__(128) kv8_read_kernel(Kv8ReadP p) {
  griddep_wait();
  griddep_release();
  __shared__ __align__(16) uint16_t tile[16][128 + 8];
  const Kv8Layer& L = p.L;
  const int tid = threadIdx.x, lp = L.lp, ld = L.ld, D = 1 << ld, C = L.Hkv << ld, c0 = blockIdx.y * 128;
  const bool is_v = blockIdx.z != 0;
  Kv8Unit u;
  if (!kv8_unit(p.q, blockIdx.x, 4, p.q.max_pages << lp, u, p.err)) return;
  const int id = kv8_page(p.q, L, u.b, u.unit >> (lp - 4), p.err);
  if (id < 0) return;
  const int slot0 = (u.unit << 4) & ((1 << lp) - 1);
  // this thread's 16 codes: channels c .. c + 15 of token t, or tokens 0 .. 15 of channel c
  const int t = tid >> 3, c = c0 + (is_v ? tid : (tid & 7) << 4), h = c >> ld, d = c & (D - 1);
  uint16_t y[16];
  if (c < C) {
    const size_t ph = (size_t)id * L.Hkv + h;
    const uint8_t* page = (is_v ? L.v : L.k) + (ph << (lp + ld)) + ((size_t)slot0 << ld);
    const uint4 w = *reinterpret_cast<const uint4*>(page + (is_v ? d << 4 : (t << ld) + d));
    const float s = (is_v ? L.vs : L.ks)[ph];
    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t lo, hi;
      kv8_widen<KIND>(ww[i], lo, hi);
      const float2 a = f16x2_float(lo), b = f16x2_float(hi);
      const float f[4] = {a.x * s, a.y * s, b.x * s, b.y * s};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const T r = from_f<T>(f[e]);
        y[4 * i + e] = *reinterpret_cast<const uint16_t*>(&r);
      }
    }
  }
  const int cv = c0 + ((tid & 7) << 4);
  if (is_v) {
#pragma unroll
    for (int i = 0; i < 16; ++i) tile[i][tid] = c < C ? y[i] : (uint16_t)0;
    __syncthreads();
  }
  if (cv >= C || t < u.lo || t >= u.hi) return;
  uint4* o = reinterpret_cast<uint4*>((is_v ? p.v : p.k) + (long)(u.row + t - u.lo) * (is_v ? p.ldv : p.ldk) + cv);
  if (is_v) {
    o[0] = *reinterpret_cast<const uint4*>(&tile[t][(tid & 7) << 4]);
    o[1] = *reinterpret_cast<const uint4*>(&tile[t][((tid & 7) << 4) + 8]);
  } else {
    uint32_t z[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = (uint32_t)y[2 * i] | (uint32_t)y[2 * i + 1] << 16;
    o[0] = make_uint4(z[0], z[1], z[2], z[3]);
    o[1] = make_uint4(z[4], z[5], z[6], z[7]);
  }
}

// ---------------------------------------------------------------------------
// Attention.  In x_t = scale * q . k_t (per key/value head, its G query heads
// and the sequence's n newest tokens are nG queries of one key row) a tile is
// 64 tokens by NQ = 8 NT queries.  One pass over the tokens with a running
// maximum m and sum l per query (base-2 exponents).
//
// Bound: one byte per key and value channel from HBM, about 23 bytes a cycle
// and SM, each of which has to be widened.  So the product with the fewest
// instructions per byte is taken: mma m16n8k16 on f16 with the TOKENS as its
// 16 rows (scores^T = K Q^T, out^T = V^T W^T), so that eight queries fill the
// instruction and a single query wastes no exponentials on empty token rows.
// Codes go from global memory to the operand registers without shared memory:
// which k index of the instruction stands for which channel (or token) is free
// as long as both operands agree, so lane (c, t) = (lane / 4, lane % 4) takes
// quarter t of a key's channels, and for values the 16 tokens of 16-token
// group t of the tile, one 16-byte load each (the layout of v is made for
// it).  Score row c of an instruction is then a token of group c / 2, all of
// one page: its two scales are one register each.  The weights reach the
// layout of the second product's B operand by an 8x8 transpose (movmatrix).
//
// Rounding: q is taken to f16 with a power of two of its own per query, which
// keeps all of bf16's and f16's bits down to 2^-28 of the query's largest
// element (2^-24 of the largest for fp16, where the power is 1); codes are
// exact in f16; scores, m, l and the output sum are fp32.  Only the weights
// lose bits: w * (page's value scale) / (largest value scale so far) is at
// most 1 and rounded to f16 (2^-12 relative, below the output's own 2^-9 or
// 2^-12), and the output accumulates in units of that largest scale.
//
// Split: (64-query job, head) pairs may be few and a context long, so its
// tiles are cut into up to S pieces, one block of four warps each (the warps
// take tiles in turn, and merge their m, l and sums in shared memory in a fixed
// order); with more than one piece, fp32 partials go to scratch and a second
// kernel merges them, again in a fixed order.  S comes from the host's bound on
// the lengths, the pieces in use from the device's lengths: at least MINT tiles each.
// ---------------------------------------------------------------------------
#define KV8_NW 4
#define KV8_MINT 4

struct Kv8AttnP {
  Kv8Layer L;
  Kv8Seqs q;
  const uint16_t* x;   // queries
  uint16_t* out;
  float* lse;
  long ldq, ldo;
  int H, G, S;
  float scale;
  float *part, *part_ml;   // [job][Hkv][S][NQ][D] sums, [..][NQ][2] (m, l)
  unsigned* err;
};

__device__ __forceinline__ float kv8_ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ void kv8_mma(float* c, const uint32_t* a, const uint32_t* b) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
__device__ __forceinline__ uint32_t kv8_transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// A job: NQ queries of one sequence and key/value head, numbered (row of the
// sequence) * G + (query head of the group).
struct Kv8Job {
  int b, s0, n, len, q0, nq;   // first query, valid queries (nq < 1: no such job)
  int maxlim;                  // tokens that its last query sees, within the row's pages
  int chunk, pieces;           // tiles a piece, pieces in use
};
template <int NQ>
__device__ __forceinline__ bool kv8_job(const Kv8AttnP& p, int job, Kv8Job& J, unsigned* err) {
  Kv8Seq s;
  int off;
  if (p.q.start) {
    const int G = p.G;
    if (!kv8_find(p.q, job, [G](int b, int s0) { return (int)((long)s0 * G / NQ) + b; }, s, off, err)) return false;
  } else {
    const int per = (p.G + NQ - 1) / NQ;
    s.b = s.s0 = job / per; s.n = 1; s.len = p.q.lens[s.b];
    off = job % per;
  }
  J.b = s.b; J.s0 = s.s0; J.n = s.n; J.len = s.len;
  J.q0 = off * NQ;
  J.nq = min(NQ, s.n * p.G - J.q0);
  if (J.nq < 1) return false;
  const int cap = p.q.max_pages << p.L.lp;
  if (off == 0 && threadIdx.x == 0 && (s.len < s.n || s.len > cap)) set_dev_err(err, GPT_DEVERR_POS);
  const int last = (J.q0 + J.nq - 1) / p.G;
  J.maxlim = min(max(s.len - s.n + last + 1, 0), cap);
  const int tiles = (J.maxlim + 63) >> 6;
  const int want = max(1, min(p.S, (tiles + KV8_MINT - 1) / KV8_MINT));
  J.chunk = max(1, (tiles + want - 1) / want);
  J.pieces = max(1, (tiles + J.chunk - 1) / J.chunk);
  return true;
}

// keep the low n bytes (0..16) of 16
__device__ __forceinline__ uint32_t kv8_low_bytes(uint32_t w, int n) {
  return n >= 4 ? w : n <= 0 ? 0u : w & ((1u << (8 * n)) - 1u);
}

template <typename T, int D, int NT, int KIND>
__global__ void __launch_bounds__(32 * KV8_NW) kv8_attn_kernel(Kv8AttnP p) {
  constexpr int NQ = 8 * NT, KW = D / 16, ROW = D + 4;
  griddep_wait();
  griddep_release();
  __shared__ __align__(16) float so[KV8_NW][NQ][ROW];
  __shared__ float sm[KV8_NW][NQ], sl[KV8_NW][NQ];
  const Kv8Layer& L = p.L;
  const int job = blockIdx.x / p.S, piece = blockIdx.x % p.S, h = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane >> 2, t = lane & 3;
  Kv8Job J;
  if (!kv8_job<NQ>(p, job, J, h == 0 && piece == 0 ? p.err : nullptr) || piece >= J.pieces) return;
  const int G = p.G, lp = L.lp;
  const long pd = (long)D << lp;

  // ---- queries: operand registers, score factors of this lane's two columns, tokens they see
  uint32_t qf[NT][KW][2];
  float cq[NT][2];
  int lim[NT][2], minlim = 0x7fffffff;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int qi = J.q0 + j * 8 + c;
    const bool ok = j * 8 + c < J.nq;
    float f[D / 4], mx = 0.f;
    if (ok) {
      const int i = qi / G;
      const uint16_t* x = p.x + (long)(J.s0 + i) * p.ldq + (h * G + qi - i * G) * D + t * (D / 4);
#pragma unroll
      for (int e = 0; e < D / 4; e += 4) {
        const uint2 w = *reinterpret_cast<const uint2*>(x + e);
        f[e] = bits16_f<T>(w.x & 0xffffu); f[e + 1] = bits16_f<T>(w.x >> 16);
        f[e + 2] = bits16_f<T>(w.y & 0xffffu); f[e + 3] = bits16_f<T>(w.y >> 16);
      }
    } else {
#pragma unroll
      for (int e = 0; e < D / 4; ++e) f[e] = 0.f;
    }
    bool bad = false;
#pragma unroll
    for (int e = 0; e < D / 4; ++e) {
      bad |= !(fabsf(f[e]) <= FLT_MAX);
      mx = fmaxf(mx, fabsf(f[e]));
    }
    float up = 1.f;
    if constexpr (sizeof(T) == 2 && !std::is_same<T, f16>::value) {
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      // the power of two that brings the largest element to [16, 32)
      const int ex = (__float_as_int(mx) >> 23) & 255;
      up = __int_as_float(max(1, min(254, 258 - max(ex, 1))) << 23);
    }
    bad = (__ballot_sync(0xffffffffu, bad) >> (lane & 28) & 15u) != 0;   // of the query's four lanes
    const float fac = bad ? NAN : p.scale * 1.4426950408889634f * (1.f / up);
#pragma unroll
    for (int w = 0; w < KW; ++w) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const __half2 v = __floats2half2_rn(bad ? 0.f : f[4 * w + 2 * e] * up, bad ? 0.f : f[4 * w + 2 * e + 1] * up);
        qf[j][w][e] = *reinterpret_cast<const uint32_t*>(&v);
      }
    }
    // columns 2t, 2t + 1 of the accumulators are the queries held by lanes 8t and 8t + 4
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      cq[j][e] = __shfl_sync(0xffffffffu, fac, 8 * t + 4 * e);
      const int n = j * 8 + 2 * t + e;
      lim[j][e] = n < J.nq ? min(max(J.len - J.n + (J.q0 + n) / G + 1, 0), J.maxlim) : J.maxlim;
      minlim = min(minlim, lim[j][e]);
    }
  }
  minlim = min(minlim, __shfl_xor_sync(0xffffffffu, minlim, 1));
  minlim = min(minlim, __shfl_xor_sync(0xffffffffu, minlim, 2));

  float o[NT][KW][4], m[NT][2], l[NT][2], vref = 0.f;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
#pragma unroll
    for (int i = 0; i < KW; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][i][e] = 0.f;
    m[j][0] = m[j][1] = -INFINITY;
    l[j][0] = l[j][1] = 0.f;
  }

  const int t1 = min((J.maxlim + 63) >> 6, (piece + 1) * J.chunk);
  const int* row = p.q.table + (long)J.b * p.q.ld_table;
  for (int tile = piece * J.chunk + warp; tile < t1; tile += KV8_NW) {
    const int tb = tile << 6, gv = tb + 16 * t, gk = tb + 16 * (c >> 1);
    // pages of the tile's four 16-token groups: group t in lane t
    int id = -1;
    if (gv < J.maxlim) {
      id = row[gv >> lp];
      if ((unsigned)id >= (unsigned)L.n_pages) {
        set_dev_err(p.err, GPT_DEVERR_PAGE);
        id = -1;
      }
    }
    const int idk = __shfl_sync(0xffffffffu, id, c >> 1);
    // ---- loads: 8 keys' quarters, 2 KW channels' 16 tokens
    uint32_t kr[8][KW], vr[2 * KW][4];
    float ks = 0.f, vs = 0.f;
    if (idk >= 0) {
      const size_t ph = (size_t)idk * L.Hkv + h;
      const uint8_t* kp = L.k + ph * pd + ((gk & ((1 << lp) - 1)) + (c & 1)) * D + t * (D / 4);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint8_t* a = kp + 2 * i * D;
        if constexpr (KW == 1) kr[i][0] = *reinterpret_cast<const uint32_t*>(a);
        else if constexpr (KW == 2) {
          const uint2 w = *reinterpret_cast<const uint2*>(a);
          kr[i][0] = w.x; kr[i][1] = w.y;
        } else {
#pragma unroll
          for (int w4 = 0; w4 < KW; w4 += 4) {
            const uint4 w = *reinterpret_cast<const uint4*>(a + 4 * w4);
            kr[i][w4] = w.x; kr[i][w4 + 1] = w.y; kr[i][w4 + 2] = w.z; kr[i][w4 + 3] = w.w;
          }
        }
      }
      ks = L.ks[ph];
      vs = L.vs[ph];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int w = 0; w < KW; ++w) kr[i][w] = 0;
    }
    if (id >= 0) {
      const uint8_t* vp = L.v + ((size_t)id * L.Hkv + h) * pd + (gv & ((1 << lp) - 1)) * D + c * 16;
#pragma unroll
      for (int i = 0; i < 2 * KW; ++i) {
        const uint4 w = *reinterpret_cast<const uint4*>(vp + i * 128);
        vr[i][0] = w.x; vr[i][1] = w.y; vr[i][2] = w.z; vr[i][3] = w.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2 * KW; ++i) vr[i][0] = vr[i][1] = vr[i][2] = vr[i][3] = 0;
    }
    const bool whole = tb + 64 <= minlim && !__any_sync(0xffffffffu, id < 0);
    if (!whole) {
      // unwritten slots may hold any byte, also e4m3's NaN: 0 * NaN must not reach the sums
#pragma unroll
      for (int i = 0; i < 2 * KW; ++i)
#pragma unroll
        for (int w = 0; w < 4; ++w) vr[i][w] = kv8_low_bytes(vr[i][w], J.maxlim - gv - 4 * w);
    }
    // ---- scores^T: s[i][j][e + 2 r] is token gk + (c & 1) + 4 i + 2 r with query 8 j + 2 t + e
    float s[4][NT][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int j = 0; j < NT; ++j) s[i][j][0] = s[i][j][1] = s[i][j][2] = s[i][j][3] = 0.f;
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        uint32_t a[4];
        kv8_widen<KIND>(kr[2 * i][w], a[0], a[2]);
        kv8_widen<KIND>(kr[2 * i + 1][w], a[1], a[3]);
#pragma unroll
        for (int j = 0; j < NT; ++j) kv8_mma(s[i][j], a, qf[j][w]);
      }
    }
    float tv = fmaxf(vs, __shfl_xor_sync(0xffffffffu, vs, 8));
    tv = fmaxf(tv, __shfl_xor_sync(0xffffffffu, tv, 16));
    const float vnew = fmaxf(vref, tv), vinv = vnew > 0.f ? 1.f / vnew : 0.f;
    const float vfac = vnew > 0.f ? vs * vinv : vs, vold = vnew > 0.f ? vref * vinv : 1.f;
    vref = vnew;
    uint32_t wf[4][NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float fac = cq[j][e] * ks;
        float x[8], mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] = s[i >> 1][j][e + 2 * (i & 1)] * fac;
          if (!whole && (gk + (c & 1) + 2 * i >= lim[j][e] || idk < 0)) x[i] = -INFINITY;
          mx = fmaxf(mx, x[i]);
        }
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
        const float mn = fmaxf(m[j][e], mx), mu = mn == -INFINITY ? 0.f : mn;
        const float al = kv8_ex2(m[j][e] - mu);
        m[j][e] = mn;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float w = kv8_ex2(x[i] - mu);
          sum += w;
          s[i >> 1][j][e + 2 * (i & 1)] = x[i] == -INFINITY ? 0.f : w * vfac;
        }
        l[j][e] = l[j][e] * al + sum;
#pragma unroll
        for (int i = 0; i < KW; ++i) {
          o[j][i][e] *= al * vold;
          o[j][i][e + 2] *= al * vold;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const __half2 w = __floats2half2_rn(s[i][j][2 * e], s[i][j][2 * e + 1]);
          wf[i][j][e] = kv8_transpose8(*reinterpret_cast<const uint32_t*>(&w));
        }
    }
    // ---- out^T += V^T W^T
#pragma unroll
    for (int k = 0; k < KW; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t a[4];
        kv8_widen<KIND>(vr[2 * k][i], a[0], a[2]);
        kv8_widen<KIND>(vr[2 * k + 1][i], a[1], a[3]);
#pragma unroll
        for (int j = 0; j < NT; ++j) kv8_mma(o[j][k], a, wf[i][j]);
      }
  }

  // ---- merge the warps
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int n = j * 8 + 2 * t + e;
#pragma unroll
      for (int k = 4; k < 32; k <<= 1) l[j][e] += __shfl_xor_sync(0xffffffffu, l[j][e], k);
#pragma unroll
      for (int i = 0; i < KW; ++i) {
        so[warp][n][i * 16 + c] = o[j][i][e] * vref;
        so[warp][n][i * 16 + c + 8] = o[j][i][e + 2] * vref;
      }
      if (c == 0) {
        sm[warp][n] = m[j][e];
        sl[warp][n] = l[j][e];
      }
    }
  __syncthreads();
  const long slot = ((long)job * L.Hkv + h) * p.S + piece;
  for (int i = threadIdx.x; i < J.nq * (D / 4); i += 32 * KV8_NW) {
    const int n = i / (D / 4), d = (i % (D / 4)) * 4;
    float M = sm[0][n];
#pragma unroll
    for (int w = 1; w < KV8_NW; ++w) M = fmaxf(M, sm[w][n]);
    const float mu = M == -INFINITY ? 0.f : M;
    float lt = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < KV8_NW; ++w) {
      const float f = kv8_ex2(sm[w][n] - mu);
      const float4 v = *reinterpret_cast<const float4*>(&so[w][n][d]);
      lt += sl[w][n] * f;
      y[0] += v.x * f; y[1] += v.y * f; y[2] += v.z * f; y[3] += v.w * f;
    }
    if (J.pieces > 1) {
      *reinterpret_cast<float4*>(p.part + (slot * NQ + n) * D + d) = make_float4(y[0], y[1], y[2], y[3]);
      if (d == 0) *reinterpret_cast<float2*>(p.part_ml + (slot * NQ + n) * 2) = make_float2(M, lt);
      continue;
    }
    const int qi = J.q0 + n, r = J.s0 + qi / G, hq = h * G + qi % G;
    const float inv = lt == 0.f ? 0.f : 1.f / lt;
    union { T v[4]; uint2 u; } z;
#pragma unroll
    for (int e = 0; e < 4; ++e) z.v[e] = from_f<T>(y[e] * inv);
    *reinterpret_cast<uint2*>(p.out + (long)r * p.ldo + hq * D + d) = z.u;
    if (d == 0 && p.lse) p.lse[(long)r * p.H + hq] = lt == 0.f ? -INFINITY : (M + log2f(lt)) * 0.6931471805599453f;
  }
}

// Merges the pieces of a (job, head): one block, NQ D / 4 columns of four
// channels, the pieces spread over the threads that are left; sums in a fixed order.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(128) kv8_attn_merge_kernel(Kv8AttnP p) {
  constexpr int NQ = 8 * NT, C4 = D / 4;
  griddep_wait();
  griddep_release();
  extern __shared__ float sw[];            // [S][NQ] weights of the pieces
  __shared__ float4 red[128];
  __shared__ float linv[NQ];
  const int job = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
  Kv8Job J;
  if (!kv8_job<NQ>(p, job, J, nullptr) || J.pieces == 1) return;
  const long slot = ((long)job * p.L.Hkv + h) * p.S;
  // a warp per query: its total and the weight of each piece
  for (int n = tid >> 5; n < J.nq; n += 4) {
    const int lane = tid & 31;
    float M = -INFINITY, lt = 0.f;
    for (int s = lane; s < J.pieces; s += 32) M = fmaxf(M, p.part_ml[((slot + s) * NQ + n) * 2]);
    M = warp_max(M);
    const float mu = M == -INFINITY ? 0.f : M;
    for (int s = lane; s < J.pieces; s += 32) {
      const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + ((slot + s) * NQ + n) * 2);
      const float f = kv8_ex2(ml.x - mu);
      sw[s * NQ + n] = f;
      lt += ml.y * f;
    }
    lt = warp_sum(lt);
    if (lane == 0) {
      linv[n] = lt == 0.f ? 0.f : 1.f / lt;
      const int qi = J.q0 + n, r = J.s0 + qi / p.G, hq = h * p.G + qi % p.G;
      if (p.lse) p.lse[(long)r * p.H + hq] = lt == 0.f ? -INFINITY : (M + log2f(lt)) * 0.6931471805599453f;
    }
  }
  __syncthreads();
  const int cols = J.nq * C4, groups = max(1, 128 / cols), per = min(cols, 128);
  for (int c0 = 0; c0 < cols; c0 += 128) {
    const int g = tid / per, col = c0 + tid % per;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    const bool on = g < groups && col < cols;
    const int n = col / C4, d = (col % C4) * 4;
    if (on)
      for (int s = g; s < J.pieces; s += groups) {
        const float4 v = *reinterpret_cast<const float4*>(p.part + ((slot + s) * NQ + n) * D + d);
        const float f = sw[s * NQ + n];
        y.x += v.x * f; y.y += v.y * f; y.z += v.z * f; y.w += v.w * f;
      }
    if (groups > 1) {
      red[tid] = y;
      __syncthreads();
      if (g == 0)
        for (int k = 1; k < groups; ++k) {
          const float4 v = red[k * per + tid];
          y.x += v.x; y.y += v.y; y.z += v.z; y.w += v.w;
        }
    }
    if (on && g == 0) {
      const int qi = J.q0 + n, r = J.s0 + qi / p.G, hq = h * p.G + qi % p.G;
      const float inv = linv[n];
      union { T v[4]; uint2 u; } z;
      z.v[0] = from_f<T>(y.x * inv); z.v[1] = from_f<T>(y.y * inv);
      z.v[2] = from_f<T>(y.z * inv); z.v[3] = from_f<T>(y.w * inv);
      *reinterpret_cast<uint2*>(p.out + (long)r * p.ldo + hq * D + d) = z.u;
    }
  }
}

// ---------------------------------------------------------------------------
// Entry points
// ---------------------------------------------------------------------------
const char* kv8_check_cache(const gpt_kv8_cache* c) {
  if (!c) return "cache is NULL";
  if (c->kind != GPT_KV8_INT8 && c->kind != GPT_KV8_E4M3) return "unknown cache kind";
  if (c->n_layers < 1 || c->n_pages < 1 || c->n_kv_heads < 1 || c->n_kv_heads > 1024)
    return "n_layers, n_pages and n_kv_heads must be >= 1 (n_kv_heads <= 1024)";
  if (c->head_dim != 16 && c->head_dim != 32 && c->head_dim != 64 && c->head_dim != 128)
    return "head_dim must be 16, 32, 64 or 128";
  if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) return "page must be 16, 32, 64 or 128";
  if (!c->k || !c->v || !c->k_scale || !c->v_scale) return "cache buffers must be non-NULL";
  if (((uintptr_t)c->k | (uintptr_t)c->v) & 15) return "k and v of the cache must be 16-byte aligned";
  if (((uintptr_t)c->k_scale | (uintptr_t)c->v_scale) & 3) return "scales must be 4-byte aligned";
  return "";
}

static const char* kv8_check_call(const gpt_kv8_cache* c, int layer, const gpt_kv8_batch* b, int dtype, const void* x,
                                  long ldx, const void* y, long ldy, long width_x, long width_y) {
  const char* why = kv8_check_cache(c);
  if (*why) return why;
  if (layer < 0 || layer >= c->n_layers) return "layer out of range [0, n_layers)";
  if (!b) return "batch is NULL";
  if (b->B < 0 || b->rows < 0 || b->max_pages < 1 || b->ld_table < b->max_pages)
    return "need B >= 0, rows >= 0 and 1 <= max_pages <= ld_table";
  if ((long)b->max_pages * c->page > 0x7fffff00L || b->rows > (1 << 28) || b->B > (1 << 24))
    return "max_pages * page, rows or B too large";
  if (b->B && (!b->lens || !b->table)) return "lens and table must be non-NULL";
  if (!b->start && b->rows != b->B) return "rows must equal B without start";
  if (dtype != GPT_PRECISION_BF16 && dtype != GPT_PRECISION_FP16) return "dtype must be bf16 or fp16";
  if (b->B == 0 || b->rows == 0) return "";
  if (!x || !y) return "matrices must be non-NULL";
  if (((uintptr_t)x | (uintptr_t)y) & 15) return "matrices must be 16-byte aligned";
  if (ldx % 8 || ldy % 8 || ldx < width_x || ldy < width_y)
    return "row strides must be multiples of 8 and cover all heads";
  return "";
}

static int kv8_refuse(const char* what, const char* why) {
  set_global_error((std::string(what) + ": " + why).c_str());
  return GPT_ERR_ARG;
}
static int kv8_done(const char* what, cudaError_t e) {
  if (e == cudaSuccess) return GPT_OK;
  set_global_error((std::string(what) + ": " + cudaGetErrorString(e)).c_str());
  return GPT_ERR_CUDA;
}

static Kv8Seqs kv8_seqs(const gpt_kv8_batch& b) {
  return {b.start, b.lens, b.table, b.B, b.max_pages, b.ld_table, b.rows};
}

template <typename T, int KIND>
static cudaError_t append_t(const Kv8AppendP& p, const gpt_kv8_cache& c, dim3 grid, cudaStream_t s) {
  const size_t smem = (size_t)c.page * (c.head_dim + KV8_PAD);
  switch (c.page * c.head_dim / 1024) {
    case 0:
    case 1: return launch_k(kv8_append_kernel<T, KIND, 1>, grid, dim3(128), smem, s, p);
    case 2: return launch_k(kv8_append_kernel<T, KIND, 2>, grid, dim3(128), smem, s, p);
    case 4: return launch_k(kv8_append_kernel<T, KIND, 4>, grid, dim3(128), smem, s, p);
    case 8: return launch_k(kv8_append_kernel<T, KIND, 8>, grid, dim3(128), smem, s, p);
    default: return launch_k(kv8_append_kernel<T, KIND, 16>, grid, dim3(128), smem, s, p);
  }
}

struct Kv8Plan {
  int nt, jobs, S;
  size_t part, ml;   // floats
};
// Queries a tile: 8, 16 or 32 (16 at most for 128 channels, whose sums fill
// the registers), by the mean number of queries a sequence; more of them read
// the cache fewer times, fewer waste less of the products.  Pieces: as many
// as give every SM three blocks or so of a quarter of a wave each, no more than
// the longest row has tiles for.
static Kv8Plan kv8_plan(const gpt_kv8_cache& c, const gpt_kv8_batch& b, int H) {
  static int sms = 0;
  if (!sms) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1) {
      cudaGetLastError();
      sms = 148;
    }
  }
  Kv8Plan P;
  const int G = H / c.n_kv_heads;
  const long per = b.B ? ((long)b.rows + b.B - 1) / b.B * G : G;
  P.nt = per <= 8 ? 1 : per <= 16 || c.head_dim == 128 ? 2 : 4;
  const int nq = 8 * P.nt;
  P.jobs = b.start ? (int)((long)b.rows * G / nq) + b.B : b.B * ((G + nq - 1) / nq);
  const long base = (long)P.jobs * c.n_kv_heads, tiles = ((long)b.max_pages * c.page + 63) / 64;
  const long want = base ? (12L * sms + base - 1) / base : 1;
  P.S = (int)std::max(1L, std::min(std::min(want, 128L), (tiles + KV8_MINT - 1) / KV8_MINT));
  const size_t n = P.S > 1 ? (size_t)base * P.S * nq : 0;
  P.part = n * c.head_dim;
  P.ml = n * 2;
  return P;
}

template <typename T, int D, int NT, int KIND>
static cudaError_t attn_nt(const Kv8AttnP& p, const Kv8Plan& P, int Hkv, cudaStream_t s) {
  cudaError_t e = launch_k(kv8_attn_kernel<T, D, NT, KIND>, dim3((unsigned)P.jobs * P.S, Hkv), dim3(32 * KV8_NW), 0, s, p);
  ++g_kernel_launches;
  if (e != cudaSuccess || P.S == 1) return e;
  ++g_kernel_launches;
  return launch_k(kv8_attn_merge_kernel<T, D, NT>, dim3(P.jobs, Hkv), dim3(128), (size_t)P.S * 8 * NT * 4, s, p);
}
template <typename T, int D, int KIND>
static cudaError_t attn_d(const Kv8AttnP& p, const Kv8Plan& P, int Hkv, cudaStream_t s) {
  if (P.nt == 1) return attn_nt<T, D, 1, KIND>(p, P, Hkv, s);
  if constexpr (D < 128) {
    if (P.nt == 4) return attn_nt<T, D, 4, KIND>(p, P, Hkv, s);
  }
  return attn_nt<T, D, 2, KIND>(p, P, Hkv, s);
}
template <typename T, int KIND>
static cudaError_t attn_t(const Kv8AttnP& p, const Kv8Plan& P, const gpt_kv8_cache& c, cudaStream_t s) {
  switch (c.head_dim) {
    case 16: return attn_d<T, 16, KIND>(p, P, c.n_kv_heads, s);
    case 32: return attn_d<T, 32, KIND>(p, P, c.n_kv_heads, s);
    case 64: return attn_d<T, 64, KIND>(p, P, c.n_kv_heads, s);
    default: return attn_d<T, 128, KIND>(p, P, c.n_kv_heads, s);
  }
}

extern "C" {

int gpt_kv8_append(const gpt_kv8_cache* c, int layer, const gpt_kv8_batch* b, const void* k, long ldk, const void* v,
                   long ldv, int dtype, uint32_t* err, void* stream) {
  const long w = c ? (long)c->n_kv_heads * c->head_dim : 0;
  const char* why = kv8_check_call(c, layer, b, dtype, k, ldk, v, ldv, w, w);
  if (*why) return kv8_refuse("gpt_kv8_append", why);
  if (b->B == 0 || b->rows == 0) return GPT_OK;
  Kv8AppendP p = {kv8_layer(*c, layer), kv8_seqs(*b), (const uint16_t*)k, (const uint16_t*)v, ldk, ldv, err};
  const dim3 grid(kv8_jobs(*b, p.L.lp), c->n_kv_heads, 2);
  cudaStream_t s = (cudaStream_t)stream;
  const bool i8 = c->kind == GPT_KV8_INT8;
  ++g_kernel_launches;
  return kv8_done("gpt_kv8_append",
                  dtype == GPT_PRECISION_BF16
                      ? (i8 ? append_t<bf16, GPT_KV8_INT8>(p, *c, grid, s) : append_t<bf16, GPT_KV8_E4M3>(p, *c, grid, s))
                      : (i8 ? append_t<f16, GPT_KV8_INT8>(p, *c, grid, s) : append_t<f16, GPT_KV8_E4M3>(p, *c, grid, s)));
}

int gpt_kv8_read(const gpt_kv8_cache* c, int layer, const gpt_kv8_batch* b, void* k, long ldk, void* v, long ldv,
                 int dtype, uint32_t* err, void* stream) {
  const long w = c ? (long)c->n_kv_heads * c->head_dim : 0;
  const char* why = kv8_check_call(c, layer, b, dtype, k, ldk, v, ldv, w, w);
  if (*why) return kv8_refuse("gpt_kv8_read", why);
  if (b->B == 0 || b->rows == 0) return GPT_OK;
  Kv8ReadP p = {kv8_layer(*c, layer), kv8_seqs(*b), (uint16_t*)k, (uint16_t*)v, ldk, ldv, err};
  const dim3 grid(kv8_jobs(*b, 4), (unsigned)((w + 127) / 128), 2);
  cudaStream_t s = (cudaStream_t)stream;
  const bool i8 = c->kind == GPT_KV8_INT8;
  ++g_kernel_launches;
  return kv8_done("gpt_kv8_read",
                  dtype == GPT_PRECISION_BF16
                      ? (i8 ? launch_k(kv8_read_kernel<bf16, GPT_KV8_INT8>, grid, dim3(128), 0, s, p)
                            : launch_k(kv8_read_kernel<bf16, GPT_KV8_E4M3>, grid, dim3(128), 0, s, p))
                      : (i8 ? launch_k(kv8_read_kernel<f16, GPT_KV8_INT8>, grid, dim3(128), 0, s, p)
                            : launch_k(kv8_read_kernel<f16, GPT_KV8_E4M3>, grid, dim3(128), 0, s, p)));
}

static const char* kv8_check_heads(const gpt_kv8_cache* c, const gpt_kv8_batch* b, int H) {
  const char* why = kv8_check_cache(c);
  if (*why) return why;
  if (H < 1 || H % c->n_kv_heads) return "n_heads must be a positive multiple of n_kv_heads";
  if (!b || b->B < 0 || b->rows < 0 || b->max_pages < 1) return "need a batch with B >= 0, rows >= 0, max_pages >= 1";
  if ((long)b->rows * (H / c->n_kv_heads) > (1L << 28) || (long)b->B * H > (1L << 28)) return "too many queries";
  return "";
}

int gpt_kv8_attention_work(const gpt_kv8_cache* c, const gpt_kv8_batch* b, int n_heads, size_t* bytes) {
  const char* why = kv8_check_heads(c, b, n_heads);
  if (!*why && !bytes) why = "bytes is NULL";
  if (*why) return kv8_refuse("gpt_kv8_attention_work", why);
  const Kv8Plan P = kv8_plan(*c, *b, n_heads);
  *bytes = (P.part + P.ml) * sizeof(float);
  return GPT_OK;
}

int gpt_kv8_attention(const gpt_kv8_cache* c, int layer, const gpt_kv8_batch* b, const void* q, long ldq, int n_heads,
                      int dtype, float scale, void* out, long ldo, float* lse, void* work, size_t work_bytes,
                      uint32_t* err, void* stream) {
  const char* why = kv8_check_heads(c, b, n_heads);
  const long w = c ? (long)n_heads * c->head_dim : 0;
  if (!*why) why = kv8_check_call(c, layer, b, dtype, q, ldq, out, ldo, w, w);
  if (!*why && !(fabsf(scale) <= FLT_MAX)) why = "scale must be finite";
  if (!*why && ((uintptr_t)lse & 3)) why = "lse must be 4-byte aligned";
  if (*why) return kv8_refuse("gpt_kv8_attention", why);
  if (b->B == 0 || b->rows == 0) return GPT_OK;
  const Kv8Plan P = kv8_plan(*c, *b, n_heads);
  if ((long)P.jobs * P.S > 0x7fffffffL) return kv8_refuse("gpt_kv8_attention", "too many queries");
  if (P.S > 1 && (!work || work_bytes < (P.part + P.ml) * sizeof(float) || ((uintptr_t)work & 15)))
    return kv8_refuse("gpt_kv8_attention", "work must be 16-byte aligned and hold gpt_kv8_attention_work bytes");
  Kv8AttnP p = {kv8_layer(*c, layer), kv8_seqs(*b), (const uint16_t*)q, (uint16_t*)out, lse, ldq, ldo,
                n_heads, n_heads / c->n_kv_heads, P.S, scale, (float*)work, (float*)work + P.part, err};
  cudaStream_t s = (cudaStream_t)stream;
  const bool i8 = c->kind == GPT_KV8_INT8;
  return kv8_done("gpt_kv8_attention",
                  dtype == GPT_PRECISION_BF16
                      ? (i8 ? attn_t<bf16, GPT_KV8_INT8>(p, P, *c, s) : attn_t<bf16, GPT_KV8_E4M3>(p, P, *c, s))
                      : (i8 ? attn_t<f16, GPT_KV8_INT8>(p, P, *c, s) : attn_t<f16, GPT_KV8_E4M3>(p, P, *c, s)));
}

}  // extern "C"
