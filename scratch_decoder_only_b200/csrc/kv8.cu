// The 8-bit paged key/value cache: quantising new tokens into it, reading
// tokens back, and attention over it (include/gpt.h has the definitions).
#include <float.h>
#include <math.h>
#include <algorithm>
#include <string>
#include <type_traits>
#include "kv8.cuh"

__device__ __forceinline__ void kv8_copy16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void kv8_lds(uint32_t* r, uint32_t src) {
  if constexpr (N == 4) asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r[0]) : "r"(src) : "memory");
  else if constexpr (N == 8) asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(src) : "memory");
  else
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(src) : "memory");
}

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
  // (a negative length, INT_MIN too, is no token: it must not wrap below)
  const int p0 = max(max(s.len, 0) - s.n, 0), p1 = min(s.len, cap);
  if (p1 <= 0) return false;
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
// Append.  A block of 128 threads takes a page of a sequence and a run of heads,
// keys or values, one head after the other, or four at a time, a warp each (fewer warps
// for fewer heads), where a page has at most 2048 elements of a head (TPH threads a head).  The next head's
// rows travel by asynchronous copies into shared memory, each thread's to places
// of its own, while a head's stay in registers (VPT 16-byte vectors a thread)
// between their largest magnitude (an unsigned 16-bit maximum over the bit
// patterns without the sign, in which infinities and NaNs are the largest) and
// their codes, so every input byte is read once.  Value codes are turned over
// through shared memory, four tokens by four channels at a time, and leave as 16
// tokens of a channel.  Instruction issue bounds it, not far above the bytes: 29181
// tokens of 64 ragged prompts, 8 heads of 128, pages of 64: 39 us (27 at the copy
// rate); 16 x 1024 tokens, 12 heads of 64, pages of 16: 25 us (11.5; 40 with a
// block per head instead of a warp).
// ---------------------------------------------------------------------------
struct Kv8AppendP {
  Kv8Layer L;
  Kv8Seqs q;
  const uint16_t *k, *v;
  long ldk, ldv;
  int heads;   // a block's
  unsigned* err;
};

#define KV8_PAD 8   // bytes behind each token's codes in the turning buffer

template <typename T>
__device__ __forceinline__ float bits16_f(unsigned b) {
  const unsigned short u = (unsigned short)b;
  return to_f(*reinterpret_cast<const T*>(&u));
}

template <typename T>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  if constexpr (std::is_same<T, f16>::value) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
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

// Bytes 0 .. n - 1 of four.
__device__ __forceinline__ uint32_t kv8_bytes(int n) { return n >= 4 ? ~0u : n <= 0 ? 0u : (1u << (8 * n)) - 1u; }
// w[i] = channels of token i  ->  w[i] = tokens of channel i
__device__ __forceinline__ void kv8_turn4(uint32_t* w) {
  const uint32_t a = __byte_perm(w[0], w[1], 0x5140), b = __byte_perm(w[2], w[3], 0x5140);
  const uint32_t c = __byte_perm(w[0], w[1], 0x7362), d = __byte_perm(w[2], w[3], 0x7362);
  w[0] = __byte_perm(a, b, 0x5410);
  w[1] = __byte_perm(a, b, 0x7632);
  w[2] = __byte_perm(c, d, 0x5410);
  w[3] = __byte_perm(c, d, 0x7632);
}

// (the second bound: 96 registers a thread up to 8 vectors, so that enough blocks are resident to cover a block's chain
// of dependent loads)
template <typename T, int KIND, int VPT, int TPH>
__global__ void __launch_bounds__(128, VPT <= 8 ? 5 : 3) kv8_append_kernel(Kv8AppendP p) {
  griddep_wait();
  griddep_release();
  // the next head's rows, [VPT][threads] vectors, each thread's own; value codes [P][D + KV8_PAD]
  extern __shared__ __align__(16) uint8_t ahead[];
  __shared__ unsigned wmax[2][4];
  const int THREADS = TPH == 128 ? 128 : blockDim.x, HEADS = THREADS / TPH;   // heads at a time
  const Kv8Layer& L = p.L;
  const int tid = threadIdx.x % TPH, mate = threadIdx.x / TPH, lp = L.lp, ld = L.ld, D = 1 << ld, row = D + KV8_PAD;
  uint8_t* turn = ahead + VPT * THREADS * 16 + mate * (row << lp);
  auto meet = [] {
    if constexpr (TPH == 128) __syncthreads();
    else __syncwarp();
  };
  const int h0 = blockIdx.y * p.heads, h1 = min(h0 + p.heads, L.Hkv);
  const bool is_v = blockIdx.z != 0;
  Kv8Unit u;
  if (!kv8_unit(p.q, blockIdx.x, lp, p.q.max_pages << lp, u, p.err)) return;
  const int id = kv8_page(p.q, L, u.b, u.unit, p.err);
  if (id < 0) return;
  const long ldx = is_v ? p.ldv : p.ldk;
  const uint16_t* x = (is_v ? p.v : p.k) + (long)u.row * ldx;
  float* scales = (is_v ? L.vs : L.ks) + (size_t)id * L.Hkv;
  const int nv = (u.hi - u.lo) << (ld - 3);
  // vector tid + TPH j of a head: this thread's first one, and TPH vectors further
  const int mine = (nv - tid + TPH - 1) / TPH;   // vectors of this thread
  const long step = (long)(TPH >> (ld - 3)) * ldx;
  x += (long)(tid >> (ld - 3)) * ldx + ((tid & ((D >> 3) - 1)) << 3);
  const uint32_t slot = (uint32_t)__cvta_generic_to_shared(ahead) + threadIdx.x * 16;
  float s_next = 0.f;
  auto load = [&](int h) {
    const uint16_t* y = x + (h << ld);
#pragma unroll
    for (int j = 0; j < VPT; ++j, y += step)
      if (j < mine) kv8_copy16(slot + j * THREADS * 16, reinterpret_cast<const uint8_t*>(y));
    asm volatile("cp.async.commit_group;" ::: "memory");
    s_next = u.lo > 0 ? scales[h] : 0.f;   // read by all before the barrier, written behind it
  };
  if (h0 + mate < h1) load(h0 + mate);
  for (int h = h0 + mate, par = 0; h < h1; h += HEADS, par ^= 1) {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    uint4 r[VPT];
    unsigned pair = 0;   // the largest magnitudes of even and odd elements
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      uint32_t w[4] = {0, 0, 0, 0};
      if (j < mine) kv8_lds<16>(w, slot + j * THREADS * 16);
      r[j] = make_uint4(w[0], w[1], w[2], w[3]);
#pragma unroll
      for (int e = 0; e < 4; ++e) pair = __vmaxu2(pair, w[e] & 0x7fff7fffu);
    }
    const float s_old = s_next;
    if (h + HEADS < h1) load(h + HEADS);
    unsigned mx = max(pair & 0xffffu, pair >> 16);
    mx = __reduce_max_sync(0xffffffffu, mx);
    if (TPH == 128 && (tid & 31) == 0) wmax[par][tid >> 5] = mx;
    meet();   // (also: the turning buffer's codes of the head before have been read)
    if (TPH == 128) mx = max(max(wmax[par][0], wmax[par][1]), max(wmax[par][2], wmax[par][3]));
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
    if (tid == 0) scales[h] = s;
    uint8_t* page = (is_v ? L.v : L.k) + (((size_t)id * L.Hkv + h) << (lp + ld));
    if (!is_v) {
      if (recode) {
        uint32_t* o = reinterpret_cast<uint32_t*>(page);
        for (int i = tid; i < (u.lo << (ld - 2)); i += TPH) o[i] = live ? kv8_recode4<KIND>(o[i], ratio) : 0u;
      }
      uint2* o = reinterpret_cast<uint2*>(page + (u.lo << ld)) + tid;
#pragma unroll
      for (int j = 0; j < VPT; ++j)
        if (j < mine) o[TPH * j] = live ? kv8_code8<T, KIND>(r[j], inv) : make_uint2(0, 0);
    } else {
      uint8_t* o = turn + (u.lo + (tid >> (ld - 3))) * row + ((tid & ((D >> 3) - 1)) << 3);
#pragma unroll
      for (int j = 0; j < VPT; ++j)
        if (j < mine)
          *reinterpret_cast<uint2*>(o + j * (TPH >> (ld - 3)) * row) =
              live ? kv8_code8<T, KIND>(r[j], inv) : make_uint2(0, 0);
    }
    if (!is_v) continue;
    meet();
    // 16-token groups that change: those with new tokens, all earlier ones too when the scale grew; a thread
    // takes four channels of one
    const int g0 = recode ? 0 : u.lo >> 4, g1 = (u.hi + 15) >> 4;
    for (int i = (g0 << (ld - 2)) + tid; i < (g1 << (ld - 2)); i += TPH) {
      const int t0 = (i >> (ld - 2)) << 4, d = (i << 2) & (D - 1);
      uint32_t w[4][4];   // [four tokens][channel]
#pragma unroll
      for (int q = 0; q < 4; ++q) {
#pragma unroll
        for (int e = 0; e < 4; ++e) w[q][e] = *reinterpret_cast<const uint32_t*>(turn + (t0 + 4 * q + e) * row + d);
        kv8_turn4(w[q]);
      }
      uint4* o = reinterpret_cast<uint4*>(page + ((size_t)t0 << ld) + (d << 4));
      if (t0 >= u.lo && t0 + 16 <= u.hi) {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = make_uint4(w[0][e], w[1][e], w[2][e], w[3][e]);
        continue;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint4 old = o[e];
        const uint32_t was[4] = {old.x, old.y, old.z, old.w};
        uint32_t z[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t keep = kv8_bytes(u.lo - t0 - 4 * q), upto = kv8_bytes(u.hi - t0 - 4 * q);
          const uint32_t held = recode ? (live ? kv8_recode4<KIND>(was[q], ratio) : 0u) : was[q];
          z[q] = (held & keep) | (w[q][e] & upto & ~keep);
        }
        o[e] = make_uint4(z[0], z[1], z[2], z[3]);
      }
    }
  }
}

// One new token per sequence (no starts), as every decode step has: a warp per
// (sequence, head, keys | values), lanes over channels, no barrier.  Three
// dependent loads (length, page, then the token, its page's scale and the values'
// 16-token group together) are all there is: 3.1 us where the block form above
// takes 4.7 (32 sequences, 12 heads of 64).
template <typename T, int KIND, int D>
__global__ void __launch_bounds__(128) kv8_append_one_kernel(Kv8AppendP p) {
  griddep_wait();
  griddep_release();
  constexpr int E = D < 32 ? 1 : D / 32;   // channels a lane
  const Kv8Layer& L = p.L;
  const int lane = threadIdx.x & 31, lp = L.lp;
  const long job = (long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int b = (int)(job / (2 * L.Hkv)), h = (int)(job % (2 * L.Hkv)) >> 1, c = lane * E;
  const bool is_v = job & 1, on = D >= 32 || lane < D;
  if (b >= p.q.B) return;
  const int len = p.q.lens[b], slot = (len - 1) & ((1 << lp) - 1);
  if (len < 1 || len > p.q.max_pages << lp) {
    if (lane == 0 && h == 0) set_dev_err(p.err, GPT_DEVERR_POS);
    return;
  }
  const int id = kv8_page(p.q, L, b, (len - 1) >> lp, p.err);
  if (id < 0) return;
  const size_t ph = (size_t)id * L.Hkv + h;
  uint8_t* page = (is_v ? L.v : L.k) + (ph << lp) * D;
  float* sp = (is_v ? L.vs : L.ks) + ph;
  const uint16_t* x = (is_v ? p.v : p.k) + (long)b * (is_v ? p.ldv : p.ldk) + h * D + c;
  uint4* group = reinterpret_cast<uint4*>(page + (slot & ~15) * D) + c;   // this lane's channels, 16 tokens each
  unsigned raw[E], mx = 0;
  uint4 old[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    raw[e] = on ? x[e] : 0;
    old[e] = make_uint4(0, 0, 0, 0);
    if (is_v && on && (slot & 15)) old[e] = group[e];
    mx = max(mx, raw[e] & 0x7fffu);
  }
  const float s_old = slot > 0 ? *sp : 0.f;
  mx = __reduce_max_sync(0xffffffffu, mx);   // (all lanes have read the scale)
  constexpr float TOP = KIND == GPT_KV8_INT8 ? 127.f : 448.f;
  const float a = bits16_f<T>(mx);
  float s = a / TOP;
  if (s < FLT_MIN) s = 0.f;             // 1 / s would overflow
  if (s_old > s) s = s_old;
  if (!(a <= FLT_MAX) || s_old != s_old) s = NAN;
  const bool live = s > 0.f, recode = slot > 0 && s != s_old;
  const float inv = live ? 1.f / s : 0.f, ratio = live ? s_old / s : 0.f;
  if (lane == 0) *sp = s;
  if (!is_v) {
    if (recode) {
      uint32_t* o = reinterpret_cast<uint32_t*>(page);
      for (int i = lane; i < slot * (D / 4); i += 32) o[i] = live ? kv8_recode4<KIND>(o[i], ratio) : 0u;
    }
  } else if (recode) {
    uint4* o = reinterpret_cast<uint4*>(page);
    for (int i = lane; i < (slot >> 4) * D; i += 32) {
      uint4 w = o[i];
      w.x = live ? kv8_recode4<KIND>(w.x, ratio) : 0u;
      w.y = live ? kv8_recode4<KIND>(w.y, ratio) : 0u;
      w.z = live ? kv8_recode4<KIND>(w.z, ratio) : 0u;
      w.w = live ? kv8_recode4<KIND>(w.w, ratio) : 0u;
      o[i] = w;
    }
  }
  if (!on) return;
  float f[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int e = 0; e < E; ++e) f[e] = bits16_f<T>(raw[e]) * inv;
  const uint32_t code = live ? kv8_code4<KIND>(f[0], f[1], f[2], f[3]) : 0u;
  if (!is_v) {
    uint8_t* o = page + slot * D + c;
    if constexpr (E == 4) *reinterpret_cast<uint32_t*>(o) = code;
    else if constexpr (E == 2) *reinterpret_cast<uint16_t*>(o) = (uint16_t)code;
    else *o = (uint8_t)code;
    return;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const uint32_t was[4] = {old[e].x, old[e].y, old[e].z, old[e].w};
    uint32_t z[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int at = (slot & 15) - 4 * q;   // of the new byte in this word
      const uint32_t held = recode ? (live ? kv8_recode4<KIND>(was[q], ratio) : 0u) : was[q];
      z[q] = (held & kv8_bytes(at)) | (at >= 0 && at < 4 ? (code >> (8 * e) & 0xffu) << (8 * at) : 0u);
    }
    group[e] = make_uint4(z[0], z[1], z[2], z[3]);
  }
}

// ---------------------------------------------------------------------------
// Read back.  A block of 128 threads takes 16 tokens, keys or values, and a run of
// 128-channel columns of the concatenated heads, one 16-byte load of codes a
// thread and column, the next two ahead: 16 channels of a token (keys), or 16
// tokens of a channel, turned over through shared memory (values).
// ---------------------------------------------------------------------------
struct Kv8ReadP {
  Kv8Layer L;
  Kv8Seqs q;
  uint16_t *k, *v;
  long ldk, ldv;
  int cols;   // a block's columns
  unsigned* err;
};

template <typename T, int KIND>
__global__ void __launch_bounds__(128) kv8_read_kernel(Kv8ReadP p) {
  griddep_wait();
  griddep_release();
  __shared__ __align__(16) uint16_t tile[2][16][128 + 8];
  const Kv8Layer& L = p.L;
  const int tid = threadIdx.x, lp = L.lp, ld = L.ld, D = 1 << ld, C = L.Hkv << ld;
  const int b0 = blockIdx.y * p.cols * 128, b1 = min(b0 + p.cols * 128, C);
  const bool is_v = blockIdx.z != 0;
  Kv8Unit u;
  if (!kv8_unit(p.q, blockIdx.x, 4, p.q.max_pages << lp, u, p.err)) return;
  const int id = kv8_page(p.q, L, u.b, u.unit >> (lp - 4), p.err);
  if (id < 0) return;
  const int slot0 = (u.unit << 4) & ((1 << lp) - 1);
  // this thread's 16 codes: channels c .. c + 15 of token t, or tokens 0 .. 15 of channel c
  const int t = tid >> 3, cv = (tid & 7) << 4;
  const uint8_t* codes = (is_v ? L.v : L.k) + (((size_t)id * L.Hkv) << (lp + ld)) + ((size_t)slot0 << ld);
  const float* scales = (is_v ? L.vs : L.ks) + (size_t)id * L.Hkv;
  uint4 next[2] = {};
  float s_next[2] = {};
  auto load = [&](int c0, int at) {
    const int c = c0 + (is_v ? tid : cv), h = c >> ld, d = c & (D - 1);
    if (c0 >= b1 || c >= C) return;
    next[at] = *reinterpret_cast<const uint4*>(codes + ((size_t)h << (lp + ld)) + (is_v ? d << 4 : (t << ld) + d));
    s_next[at] = scales[h];
  };
  uint16_t* out = (is_v ? p.v : p.k) + (long)(u.row + t - u.lo) * (is_v ? p.ldv : p.ldk) + cv;
  const bool mine = t >= u.lo && t < u.hi;
  load(b0, 0);
  load(b0 + 128, 1);
  for (int c0 = b0, par = 0; c0 < b1; c0 += 128, par ^= 1) {
    const uint32_t w[4] = {next[0].x, next[0].y, next[0].z, next[0].w};
    const float s = s_next[0];
    next[0] = next[1];
    s_next[0] = s_next[1];
    load(c0 + 256, 1);
    uint32_t y[8];   // pairs of 16-bit values
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t lo, hi;
      kv8_widen<KIND>(w[i], lo, hi);
      const float2 a = f16x2_float(lo), b = f16x2_float(hi);
      y[2 * i] = pack16<T>(a.x * s, a.y * s);
      y[2 * i + 1] = pack16<T>(b.x * s, b.y * s);
    }
    if (is_v) {
      // (two tiles in turn: one barrier keeps a tile's readers ahead of its next writers)
#pragma unroll
      for (int i = 0; i < 16; ++i) tile[par][i][tid] = (uint16_t)(y[i >> 1] >> (16 * (i & 1)));
      __syncthreads();
    }
    if (!mine || c0 + cv >= C) continue;
    uint4* o = reinterpret_cast<uint4*>(out + c0);
    if (is_v) {
      o[0] = *reinterpret_cast<const uint4*>(&tile[par][t][cv]);
      o[1] = *reinterpret_cast<const uint4*>(&tile[par][t][cv + 8]);
    } else {
      o[0] = make_uint4(y[0], y[1], y[2], y[3]);
      o[1] = make_uint4(y[4], y[5], y[6], y[7]);
    }
  }
}

// ---------------------------------------------------------------------------
// Attention.  Per key/value head, its G query heads and the sequence's n newest
// tokens are nG queries of one row of keys; a job is NQ = 8 NT of them, and its
// work is tiles of TILE tokens, in one pass with a running maximum m and sum l
// per query (base-2 exponents).
//
// Bound: one byte per key and value channel from HBM, about 23 bytes a cycle
// and SM, each of which has to be widened.  So the product with the fewest
// instructions per byte is taken: mma m16n8k16 on f16 with the TOKENS as its
// 16 rows (scores^T = K Q^T, out^T = V^T W^T), so that eight queries fill the
// instruction and a single query wastes no exponentials on empty rows.  Which
// k index of the instruction stands for which channel (or token) is free as
// long as both operands agree, so lane (c, t) = (lane / 4, lane % 4) takes
// quarter t of a key's channels, and for values the t-th quarter of the tile's
// tokens, 16 bytes a load either way (the layout of v is made for it).  Score
// row c of an instruction is then a token of quarter c / 2, all in one page:
// its two scales are one register each.  The weights reach the layout of the
// second product's B operand by an 8x8 transpose (movmatrix).  The maximum is
// brought up to date only when a score passes it by 2^8 (w <= 256 in f16), so
// most tiles need no reduction over lanes and no rescaling.
//
// Latency: a tile's values travel by asynchronous copies into shared memory
// while the warp works on its keys, the next tile's keys while it works on the
// weights and values; the page ids of the tile after that are being loaded.  One
// buffer of 4 KB each (8 KB for 128 channels) is enough for that, so registers,
// not shared memory, set the number of warps (16 an SM with eight queries, 12 for
// 128 channels), and a warp meets no barrier while it runs.  (A second buffer for
// the values, copied a whole tile ahead: 58 us instead of 55 for 64 x 4096 tokens.)  Lanes copy whole 128-byte lines (an asynchronous copy
// whose eight lanes lie in different lines is taken apart lane by lane) to places
// permuted so that the reads above have no bank conflicts.
//
// Rounding: q is taken to f16 with a power of two of its own per query, which
// keeps all of bf16's bits down to 2^-28 of the query's largest element (fp16
// queries are f16); codes are exact in f16; scores, m, l and the output sum are
// fp32.  Only the weights lose bits: w * (page's value scale) / (largest value
// scale so far) is rounded to f16 (a lone token's 1 stays exact).  Each query's
// products of a tile are brought by a power of two of their own to a
// largest of [2^14, 2^15) first, and the tile's sums taken back as they join the
// output's, which are in units of that scale.  So the rounding is 2^-11 relative down to 2^-28 of the tile's largest
// product, and 2^-39 of that largest below, whatever the row's other tiles hold:
// one key far above a long row of small weights, its own value near zero, costs the
// rest no bits, nor does a page of large values that hardly weighs.  (One unit for
// the whole row lost both: 17 nats below the row's largest a weight had one bit.)
// Scales that differ by more than 2^126 leave fp32 on the way.
//
// Split: lengths are known on the device only, and a batch may mix a few tokens
// with a hundred thousand.  So the tiles of all (sequence, NQ queries, head)
// jobs are numbered, KV8_OVER units ahead of each job's first for what a job
// costs besides its tiles, and each warp of the grid's resident blocks takes an
// equal run of units.  A job that a run cuts leaves fp32 partials in scratch,
// two at most per run, and a second kernel merges them in a fixed order, its
// columns spread over the runs that have a piece.  Where the host knows that rows are short
// (KV8_WHOLE tokens at most), a block takes a whole job, its four or eight warps
// the tiles in turn, and merges it in shared memory.
//
// Measured (one B200, L2 too small for the caches): 64 sequences of 4096 tokens, 8
// heads of 64, int8: 56 us = 4.8 TB/s of codes (73 % of the copy rate), the merge 7
// of them; one sequence of 131071 tokens, 8 heads
// of 128, 32 query heads, e4m3: 57 us (72 %); 64 sequences of 0 to 16384 tokens
// with 1 to 5 rows, 32 query heads of 64: 48.5 us, bound by the 1.8 passes over each
// key that 4 to 20 queries take in jobs of 8.  Short rows are bound by the chain
// length, page, codes, weights, merge: 32 sequences of up to 512 tokens, 12 heads of
// 64: 10.7 us, one: 5.8.  The weights' own powers of two take 0 to 1 us of these, 2.3
// of the 48.5 (and 4 of 72 for 64 x 4096 tokens with 16 queries each); skipping them by a
// vote where all of a tile's weights are large took 48 and 72, a power kept from
// tile to tile until a maximum leaves a window 48 and 78.
// ---------------------------------------------------------------------------
#define KV8_NW 4       // warps of a block that takes runs, or a whole job
#define KV8_WIDE 8     // of one that takes a whole job where jobs are few
#define KV8_WHOLE 1024 // tokens
#define KV8_OVER 4      // units (1: mixed batches 25 % slower; 2: 5 %; uniform ones 1 % faster)

struct Kv8AttnP {
  Kv8Layer L;
  Kv8Seqs q;
  const uint16_t* x;   // queries
  uint16_t* out;
  float* lse;
  long ldq, ldo;
  int H, G, cap;
  float scale;
  float *part, *part_ml;   // [run][2][NQ][D] sums, [run][2][NQ][2] (m, l)
  struct Kv8Piece* piece;  // [run][2]
  unsigned* err;
};

// A partial result of a run: its job is cut into `pieces` (0: there is none), the
// first of them from run w0; the job's first row, query, queries, head.
struct __align__(16) Kv8Piece {
  int pieces, w0, s0, q0, nq, h, pad[2];
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
// keep the low n bytes of four
__device__ __forceinline__ uint32_t kv8_low_bytes(uint32_t w, int n) {
  return n >= 4 ? w : n <= 0 ? 0u : w & ((1u << (8 * n)) - 1u);
}

// A sequence's share of the work: jobs = ceil(n G / NQ) * heads, tiles a job
// (an empty sequence has one, for its rows' zeros).
struct Kv8Share {
  int s0, n, len, jobs, tiles;
};
template <int NQ, int TILE>
__device__ __forceinline__ Kv8Share kv8_share(const Kv8AttnP& p, int b) {
  Kv8Share s;
  if (p.q.start) {
    s.s0 = min(max(p.q.start[b], 0), p.q.rows);
    s.n = min(max(p.q.start[b + 1], s.s0), p.q.rows) - s.s0;
  } else {
    s.s0 = b;
    s.n = 1;
  }
  s.len = p.q.lens[b];
  s.jobs = (int)(((long)s.n * p.G + NQ - 1) / NQ) * p.L.Hkv;
  s.tiles = max(1, (min(max(s.len, 0), p.cap) + TILE - 1) / TILE);
  return s;
}

// Where this warp's run begins (WHOLE: where the block's job is): the sequence,
// its job, the unit in the job.  Run number run0 + warp of `runs` covers units
// [run * quota, (run + 1) * quota) of total.  All threads of the block call
// this; false: no such run.
struct Kv8Run {
  int b, job, x, u, quota, total;
};
template <int NQ, int TILE, bool WHOLE>
__device__ __forceinline__ bool kv8_locate(const Kv8AttnP& p, int runs, int run0, Kv8Run& r) {
  __shared__ int wsum[KV8_WIDE], sh_rem[KV8_NW], sh_at[KV8_NW];
  constexpr int PER = WHOLE ? 1 : KV8_NW;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = p.q.B, nth = blockDim.x, nw = nth >> 5;
  if (WHOLE && !p.q.start) {
    // the same jobs for each sequence
    const int per = (p.G + NQ - 1) / NQ * p.L.Hkv;
    r.b = run0 / per;
    r.job = run0 % per;
    r.x = KV8_OVER;
    return r.b < B;
  }
  auto units = [&](int b) -> int {
    if (b >= B) return 0;
    const Kv8Share s = kv8_share<NQ, TILE>(p, b);
    return WHOLE ? s.jobs : s.jobs * (s.tiles + KV8_OVER);
  };
  // a thread adds up its share of the sequences, one scan over the threads finds the
  // share and one over a warp's lanes the sequence in it (8192 sequences of up to 64
  // tokens: 83 us; 102 where the block scanned 128 sequences at a time)
  const int share = B <= nth ? 1 : (int)((unsigned)(B + nth - 1) / (unsigned)nth);
  long sum = units(tid * share);
  for (int i = 1; i < share; ++i) sum += units(tid * share + i);
  const int mine = (int)sum;
  r.total = 0;
  r.quota = 1;
  int u0 = run0;
  if (!WHOLE) {
    // the host has made sure that 32 bits hold the units of `rows` rows; starts that
    // decrease can make the same rows count many times over, and then nothing is done
    __shared__ long total[KV8_NW];
#pragma unroll
    for (int k = 16; k; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
    if (lane == 0) total[warp] = sum;
    __syncthreads();
    sum = 0;
    for (int w = 0; w < nw; ++w) sum += total[w];
    if (sum > 0x7fffffffL) return false;
    r.total = (int)sum;
    r.quota = max(KV8_OVER + 1, (r.total - 1) / runs + 1);
    if (run0 >= (r.total - 1) / r.quota + 1) return false;
    u0 = run0 * r.quota;
    if (tid < PER) sh_at[tid] = -1;
  }
  const int ask = PER == 1 ? 0 : warp;
  const int left = r.total - 1 - u0;   // units behind u0, not to pass 2^31
  r.u = PER == 1 ? u0 : ask * r.quota <= left ? u0 + ask * r.quota : r.total;
  auto scan = [&](int v) {   // over the warp, this lane's included
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, v, k);
      if (lane >= k) v += y;
    }
    return v;
  };
  const int inc = scan(mine);
  if (lane == 31) wsum[warp] = inc;
  __syncthreads();
  int first = inc - mine, all = 0;
  for (int w = 0; w < nw; ++w) {
    if (w < warp) first += wsum[w];
    all += wsum[w];
  }
  for (int w = 0; w < PER; ++w) {
    const int u = u0 + w * r.quota;
    if ((WHOLE || w * r.quota <= left) && u >= first && u - first < mine) {
      sh_at[w] = tid;
      sh_rem[w] = u - first;
    }
  }
  if (WHOLE && all <= u0) return false;
  __syncthreads();
  int rem = sh_rem[ask];
  r.b = sh_at[ask];
  if (share > 1 && r.b >= 0) {
    const int b0 = r.b * share;
    r.b = -1;
    for (int i = 0; i < share; i += 32) {
      const int v = i + lane < share ? units(b0 + i + lane) : 0, upto = scan(v);
      const unsigned past = __ballot_sync(0xffffffffu, upto > rem);
      const int at = past ? __ffs(past) - 1 : 31, before = __shfl_sync(0xffffffffu, past ? upto - v : upto, at);
      rem -= before;
      if (past) {
        r.b = b0 + i + at;
        break;
      }
    }
  }
  if (WHOLE) {
    r.job = rem;
    r.x = KV8_OVER;
    return r.b >= 0;
  }
  if (r.b >= 0) {
    const int w = kv8_share<NQ, TILE>(p, r.b).tiles + KV8_OVER;
    r.job = rem / w;
    r.x = rem % w;
  }
  return true;
}

// 64 tokens; 32 where 128 channels of 16 queries fill the registers, and for 128
// channels where a block takes a whole job: more warps for few tokens.  NW: warps
// of blocks that take whole jobs (0: blocks of KV8_NW warps take runs).
__host__ __device__ constexpr int kv8_tile(int D, int nt, bool whole) { return D == 128 && (nt == 2 || whole) ? 32 : 64; }
template <int D, int NT, bool WHOLE>
struct Kv8Tile {
  static constexpr int TILE = kv8_tile(D, NT, WHOLE);
  static constexpr int HALF = TILE * D;   // bytes of a tile's keys, and of its values
};
template <int D, int NT, int NW>
constexpr size_t kv8_attn_smem() {
  return (size_t)(NW ? NW : KV8_NW) * 2 * Kv8Tile<D, NT, NW != 0>::HALF + (size_t)NW * 8 * NT * (D + 4) * 4;
}
// Blocks an SM holds by their registers: of four warps 128, 168 or 255 a thread, of
// eight 128 (255 where 16 queries of 128 channels need them).
__host__ __device__ constexpr int kv8_resident(int D, int nt, int nw) {
  return nw == KV8_WIDE ? (nt == 2 && D == 128 ? 1 : 2)
                        : nt == 1 && (D < 128 || nw) ? 4 : nt == 1 || D < 128 ? 3 : 2;
}

// Two partial results of a query, four channels.
struct Kv8Sum {
  float M, l;
  float4 y;
};
__device__ __forceinline__ void kv8_join(Kv8Sum& a, float M, float l, float4 y) {
  const float Mn = fmaxf(a.M, M), mu = Mn == -INFINITY ? 0.f : Mn, f = kv8_ex2(a.M - mu), g = kv8_ex2(M - mu);
  a.M = Mn;
  a.l = a.l * f + l * g;
  a.y.x = a.y.x * f + y.x * g; a.y.y = a.y.y * f + y.y * g;
  a.y.z = a.y.z * f + y.z * g; a.y.w = a.y.w * f + y.w * g;
}

// The result of query q0 + n of a job, four channels from d on.
template <typename T>
__device__ __forceinline__ void kv8_out(const Kv8AttnP& p, int s0, int h, int qi, int d, int D, float4 y, float M,
                                        float lt) {
  const int row = s0 + qi / p.G, hq = h * p.G + qi % p.G;
  const float inv = lt == 0.f ? 0.f : 1.f / lt;
  *reinterpret_cast<uint2*>(p.out + (long)row * p.ldo + hq * D + d) =
      make_uint2(pack16<T>(y.x * inv, y.y * inv), pack16<T>(y.z * inv, y.w * inv));
  if (d == 0 && p.lse) p.lse[(long)row * p.H + hq] = lt == 0.f ? -INFINITY : (M + log2f(lt)) * 0.6931471805599453f;
}

template <typename T, int D, int NT, int KIND, int NW>
__global__ void __launch_bounds__(32 * (NW ? NW : KV8_NW), kv8_resident(D, NT, NW))
    kv8_attn_kernel(Kv8AttnP p) {
  constexpr bool WHOLE = NW != 0;
  constexpr int WARPS = WHOLE ? NW : KV8_NW;
  constexpr int NQ = 8 * NT, KW = D / 16, TILE = Kv8Tile<D, NT, WHOLE>::TILE, HALF = Kv8Tile<D, NT, WHOLE>::HALF;
  constexpr int TQ = TILE / 4;                         // tokens of a quarter
  constexpr int KP = D / 4 < 16 ? D / 4 : 16, KT = D / 4 / KP;   // bytes of a key read, reads of a quarter key
  constexpr int STEP = WHOLE ? WARPS : 1;
  griddep_wait();
  griddep_release();
  extern __shared__ __align__(128) uint8_t ring[];
  const Kv8Layer& L = p.L;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane >> 2, t = lane & 3;
  const int G = p.G, lp = L.lp, pmask = (1 << lp) - 1, Hkv = L.Hkv;
  if (blockIdx.x == 0) {
    for (int b = threadIdx.x; b < p.q.B; b += 32 * WARPS) {
      if (p.q.start && (p.q.start[b] < 0 || p.q.start[b + 1] < p.q.start[b] || p.q.start[b + 1] > p.q.rows))
        set_dev_err(p.err, GPT_DEVERR_START);
      const Kv8Share s = kv8_share<NQ, TILE>(p, b);
      if (s.n && (s.len < s.n || s.len > p.cap)) set_dev_err(p.err, GPT_DEVERR_POS);
    }
  }
  Kv8Run r;
  const int run = blockIdx.x * WARPS + warp;
  if (!WHOLE && lane < 2) p.piece[2 * run + lane].pieces = 0;
  if (!kv8_locate<NQ, TILE, WHOLE>(p, gridDim.x * KV8_NW, blockIdx.x * (WHOLE ? 1 : KV8_NW), r)) return;
  if (!WHOLE && (r.u >= r.total || r.b < 0)) return;   // no barrier follows
  // a whole job's first page ids do not wait for its length
  const uint32_t id0 = WHOLE ? p.q.table[(long)r.b * p.q.ld_table + min((warp * TILE + TQ * t) >> lp, p.q.max_pages - 1)] : 0;
  Kv8Share sh = kv8_share<NQ, TILE>(p, r.b);
  // units of this run, counted from its begin; a job's first KV8_OVER have no tile
  const int R = WHOLE ? sh.tiles : min(r.quota, r.total - r.u);

  // ---- the warp's next tile: sequence nb, head nh, tile nt of nm, the job's number nj of njobs; nu: the unit; the
  // page-and-head number of this lane's quarter (none: KV8_NONE)
  constexpr uint32_t KV8_NONE = 0xffffffffu;
  int nb = r.b, nj = r.job, nh = r.job % Hkv, nt = r.x - KV8_OVER, nm = sh.tiles, njobs = sh.jobs;
  int nlen = min(max(sh.len, 0), p.cap), nu = 0;
  uint32_t nph = KV8_NONE;
  if (nt < 0) {
    nu = -nt;
    nt = 0;
  }
  auto page = [&](bool first) {
    const int tok = nt * TILE + TQ * t;
    nph = KV8_NONE;
    if (nu < R && tok < nlen) {
      const uint32_t id = first ? id0 : p.q.table[(long)nb * p.q.ld_table + (tok >> lp)];
      if (id < (uint32_t)L.n_pages) nph = id * Hkv + nh;
      else set_dev_err(p.err, GPT_DEVERR_PAGE);
    }
  };
  auto advance = [&]() {
    nu += STEP;
    nt += STEP;
    if (!WHOLE && nt >= nm) {
      nu += KV8_OVER;
      nt = 0;
      if (++nh == Hkv) nh = 0;
      if (++nj == njobs && nu < R) {
        Kv8Share s;
        do {
          if (++nb >= p.q.B) {   // only where lens changed meanwhile
            nu = R;
            break;
          }
          s = kv8_share<NQ, TILE>(p, nb);
        } while (s.jobs == 0);
        if (nu < R) {
          nj = 0;
          nm = s.tiles;
          njobs = s.jobs;
          nlen = min(max(s.len, 0), p.cap);
        }
      }
    }
    page(false);
  };
  const uint32_t kbuf = (uint32_t)__cvta_generic_to_shared(ring) + warp * 2 * HALF, vbuf = kbuf + HALF;
  float ks_next = 0.f, vs_next = 0.f;
  bool kon_next = false, von_next = false;   // the key's quarter, the value's has a page
  unsigned has = 0;                          // bit t: quarter t has one
  uint32_t place = 0;
  // Keys lie in their buffer token by token, values by group of 16 tokens and
  // channel, 16 bytes a piece.  Bits 4 to 6 of the address are exchanged by
  // exclusive or within a 128-byte line so that the eight lanes of a 16-byte
  // read (16 of an 8-byte, 32 of a 4-byte one) meet different bank groups.
  // Both have the same place in k and in v, here in units of 16 bytes, which
  // 32 bits hold for 64 GB a layer.
  auto copy = [&](uint32_t buf, const uint8_t* from, bool keys) {
#pragma unroll
    for (int g = 0; g < TILE / 16; ++g) {
      const uint32_t at = __shfl_sync(0xffffffffu, place, g * (16 / TQ));
      constexpr int N = D / 32 ? D / 32 : 1;   // copies of 32 lanes a group
      const uint32_t kx = D == 128 ? (lane >> 3 & 1) << 6 : D == 64 ? 0 : (g & (64 / D - 1)) * 2 * D;
      const uint32_t vx = TQ == 16 ? (g & 3) << 5 : (g & 1) << 6;
      if (has >> g * (16 / TQ) & 1 && (D >= 32 || lane < 16)) {
        const uint8_t* a = from + (size_t)at * 16;
#pragma unroll
        for (int i = 0; i < N; ++i) kv8_copy16(buf + g * 16 * D + i * 512 + (lane * 16 ^ (keys ? kx : vx)), a + i * 512);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto fetch_keys = [&]() {
    // of this lane's quarter: its 16-token group (the token's slot rounded down)
    place = nph * (uint32_t)(D / 16 << lp) + ((nt * TILE + TQ * t) & pmask & ~15) * (D / 16);
    has = __ballot_sync(0xffffffffu, nph != KV8_NONE) & 15u;
    copy(kbuf, L.k + lane * 16, true);
    const uint32_t ph = __shfl_sync(0xffffffffu, nph, c >> 1);
    kon_next = ph != KV8_NONE;
    von_next = nph != KV8_NONE;
    ks_next = kon_next ? L.ks[ph] : 0.f;
    vs_next = kon_next ? L.vs[ph] : 0.f;
  };
  if (WHOLE) {
    nu += warp;
    nt += warp;
  }
  page(WHOLE);
  fetch_keys();
  advance();

  // ---- this lane's read offsets in a stage
  // keys: token TQ (c / 2) + (c & 1) + 2 i, bytes t D / 4 .. (128 channels: 16 t .. and 64 + 16 t ..); the bits of
  // 2 i D are 0 in koff's place of them before the exchange, so they join by exclusive or where both meet (D < 64)
  uint32_t koff, voff;
  {
    const int tk = TQ * (c >> 1) + (c & 1);
    if constexpr (D == 128) koff = tk * D + (t * 16 ^ (tk & 1) << 6);
    else koff = tk * D + t * (D / 4);
    if constexpr (D < 64) koff ^= (tk >> 4 & (64 / D - 1)) * 2 * D;
    const int g = t * TQ >> 4;
    voff = g * 16 * D + (c * 16 ^ (TQ == 16 ? g << 5 : g << 6)) + (t * TQ & 15);
  }
  int cu = WHOLE ? warp : max(0, KV8_OVER - r.x);
  int b = r.b, job = r.job, x = r.x;
  for (int su = 0; su < R;) {
    // ---- one job of the run: units [su, su + span), tiles [tile0, tile0 + cnt)
    const int tile0 = max(0, x - KV8_OVER), skip = max(0, KV8_OVER - x);
    const int span = WHOLE ? R : min(sh.tiles + KV8_OVER - x, R - su), cnt = span - skip;
    if (!WHOLE && cnt <= 0) break;   // the run ends ahead of the job's tiles
    const int h = job % Hkv, q0 = job / Hkv * NQ, nq = min(NQ, sh.n * G - q0), slen = min(max(sh.len, 0), p.cap);
    // queries: operand registers, score factors of this lane's two columns, tokens they see
    uint32_t qf[NT][KW][2];
    float cq[NT][2];
    int lim[NT][2], minlim = 0x7fffffff;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int qi = q0 + j * 8 + c;
      const bool ok = j * 8 + c < nq;
      float f[D / 4], mx = 0.f;
      if (ok) {
        const int i = qi / G;
        const uint16_t* y = p.x + (long)(sh.s0 + i) * p.ldq + (h * G + qi - i * G) * D + t * (D == 128 ? 16 : D / 4);
#pragma unroll
        for (int e = 0; e < D / 4; e += 4) {
          const uint2 w = *reinterpret_cast<const uint2*>(y + e + (D == 128 && e >= 16 ? 48 : 0));
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
      if constexpr (!std::is_same<T, f16>::value) {
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // the power of two that brings the largest element to [16, 32)
        const int ex = (__float_as_int(mx) >> 23) & 255;
        up = __int_as_float(max(1, min(254, 258 - max(ex, 1))) << 23);
      }
      bad = (__ballot_sync(0xffffffffu, bad) >> (lane & 28) & 15u) != 0;   // of the query's four lanes
      const float fac = bad ? NAN : fabsf(p.scale) * 1.4426950408889634f * (1.f / up);
      if (p.scale < 0.f) up = -up;   // the factors are not negative
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
        lim[j][e] = n < nq ? min(max(sh.len - sh.n + (q0 + n) / G + 1, 0), slen) : slen;
        minlim = min(minlim, lim[j][e]);
      }
    }
    minlim = min(minlim, __shfl_xor_sync(0xffffffffu, minlim, 1));
    minlim = min(minlim, __shfl_xor_sync(0xffffffffu, minlim, 2));

    float o[NT][KW][4], m[NT][2], l[NT][2], vref = 0.f, vinv = 1.f;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int i = 0; i < KW; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][i][e] = 0.f;
      m[j][0] = m[j][1] = -INFINITY;
      l[j][0] = l[j][1] = 0.f;
    }

    for (; cu < su + span; cu += STEP) {
      const float ks = ks_next, vs = vs_next;
      const bool kon = kon_next, von = von_next, on = has == 15u;
      __syncwarp();   // the values of the tile before have been read by all lanes
      copy(vbuf, L.v + lane * 16, false);
      asm volatile("cp.async.wait_group 1;" ::: "memory");   // the keys
      __syncwarp();
      const int tb = (tile0 + cu - su - skip) * TILE, gv = tb + TQ * t, gk = tb + TQ * (c >> 1);
      const bool full = on && tb + TILE <= minlim;
      // ---- scores^T: s[i][j][e + 2 r] is token gk + (c & 1) + 4 i + 2 r with query 8 j + 2 t + e
      float s[TQ / 4][NT][4];
#pragma unroll
      for (int i = 0; i < TQ / 4; ++i) {
        uint32_t kr[2][KW];
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int w = 0; w < KT; ++w) {
            const uint32_t at = w ? koff ^ 64 : koff, more = (4 * i + 2 * e) * D;
            kv8_lds<KP>(&kr[e][w * 4], kbuf + (D < 64 ? at ^ more : at + more));
          }
#pragma unroll
        for (int j = 0; j < NT; ++j) s[i][j][0] = s[i][j][1] = s[i][j][2] = s[i][j][3] = 0.f;
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          uint32_t a[4];
          kv8_widen<KIND>(kr[0][w], a[0], a[2]);
          kv8_widen<KIND>(kr[1][w], a[1], a[3]);
#pragma unroll
          for (int j = 0; j < NT; ++j) kv8_mma(s[i][j], a, qf[j][w]);
        }
      }
      __syncwarp();   // all lanes have read the keys
      fetch_keys();
      advance();
      // ---- weights; a tile that some query sees in part takes the form with comparisons
      float fac[NT][2], down[NT][2];
      uint32_t wf[TQ / 4][NT][2];
      auto weigh = [&](auto part) {
        constexpr bool PART = decltype(part)::value;
        auto seen = [&](int i, int j, int e) { return !PART || (gk + (c & 1) + 2 * i < lim[j][e] && kon); };
        bool stale = vs > vref && vs <= FLT_MAX;
        float top[NT][2];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = -INFINITY;
#pragma unroll
            for (int i = 0; i < TQ / 2; ++i)
              if (seen(i, j, e)) mx = fmaxf(mx, s[i >> 1][j][e + 2 * (i & 1)]);
            top[j][e] = fmaxf(-INFINITY, mx * fac[j][e]);   // (-inf * 0 and a NaN scale: NaN, which no maximum takes)
            stale |= top[j][e] > m[j][e] + 8.f;
          }
        if (__any_sync(0xffffffffu, stale)) {
          const float vwas = vref;
          float tv = vs <= FLT_MAX ? fmaxf(vs, FLT_MIN) : FLT_MIN;   // (an infinite scale makes its own rows infinite, no others)
          tv = fmaxf(tv, __shfl_xor_sync(0xffffffffu, tv, 8));
          vref = fmaxf(vref, fmaxf(tv, __shfl_xor_sync(0xffffffffu, tv, 16)));
          vinv = 1.f / vref;
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float mx = top[j][e];
#pragma unroll
              for (int k = 4; k < 32; k <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
              const float mn = fmaxf(m[j][e], mx), al = kv8_ex2(m[j][e] - (mn == -INFINITY ? 0.f : mn));
              m[j][e] = mn;
              l[j][e] *= al;
#pragma unroll
              for (int i = 0; i < KW; ++i) {
                o[j][i][e] *= al * (vwas * vinv);
                o[j][i][e + 2] *= al * (vwas * vinv);
              }
            }
        }
        const float vr = vs * vinv;   // at most 1, or infinite or NaN as the scale is
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          // the largest product of each column, to a power of two: the upper halves of two fp32 numbers that
          // are not negative compare as integers (a scale of NaN or nothing seen: 0)
          uint32_t most[2];
#pragma unroll
          for (int e = 0; e < 2; ++e)
            most[e] = __float_as_uint(fmaxf(0.f, kv8_ex2(top[j][e] - (m[j][e] == -INFINITY ? 0.f : m[j][e])) * vr));
          uint32_t both = __vmaxu2(__byte_perm(most[0], most[1], 0x7632), 0x07800780u);   // (2^-112 at least)
#pragma unroll
          for (int k = 4; k < 32; k <<= 1) both = __vmaxu2(both, __shfl_xor_sync(0xffffffffu, both, k));
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float mu = m[j][e] == -INFINITY ? 0.f : m[j][e];
            const uint32_t p2 = (e ? both : both << 16) & 0x7f800000u;
            const float vfac = vr * __uint_as_float((268u << 23) - p2);   // 2^14 / p2
            down[j][e] = __uint_as_float(p2 - (14u << 23));
#pragma unroll
            for (int i = 0; i < TQ / 2; ++i) {
              float& y = s[i >> 1][j][e + 2 * (i & 1)];
              const float w = kv8_ex2(fmaf(y, fac[j][e], -mu));
              // a token that is not seen weighs 0 even where its page's scale is NaN
              l[j][e] += seen(i, j, e) ? w : 0.f;
              y = seen(i, j, e) ? w * vfac : 0.f;
            }
          }
#pragma unroll
          for (int i = 0; i < TQ / 4; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const __half2 w = __floats2half2_rn(s[i][j][2 * e], s[i][j][2 * e + 1]);
              wf[i][j][e] = kv8_transpose8(*reinterpret_cast<const uint32_t*>(&w));
            }
        }
      };
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        fac[j][0] = cq[j][0] * ks;
        fac[j][1] = cq[j][1] * ks;
      }
      if (full) weigh(std::false_type{});
      else weigh(std::true_type{});
      // ---- out^T += V^T W^T
      asm volatile("cp.async.wait_group 1;" ::: "memory");   // the values
      __syncwarp();
#pragma unroll
      for (int k = 0; k < KW; ++k) {
        uint32_t vr[2][TQ / 4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          kv8_lds<TQ>(vr[e], vbuf + voff + (2 * k + e) * 128);
          if (!full) {
            // unwritten slots may hold any byte, also e4m3's NaN: 0 * NaN must not reach the sums
#pragma unroll
            for (int w = 0; w < TQ / 4; ++w) vr[e][w] = von ? kv8_low_bytes(vr[e][w], slen - gv - 4 * w) : 0u;
          }
        }
        float sum[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j) sum[j][0] = sum[j][1] = sum[j][2] = sum[j][3] = 0.f;
#pragma unroll
        for (int i = 0; i < TQ / 4; ++i) {
          uint32_t a[4];
          kv8_widen<KIND>(vr[0][i], a[0], a[2]);
          kv8_widen<KIND>(vr[1][i], a[1], a[3]);
#pragma unroll
          for (int j = 0; j < NT; ++j) kv8_mma(sum[j], a, wf[i][j]);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[j][k][e] = fmaf(sum[j][e], down[j][e & 1], o[j][k][e]);
      }
    }

#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) l[j][e] += __shfl_xor_sync(0xffffffffu, l[j][e], k);
#pragma unroll
        for (int i = 0; i < KW; ++i) {
          o[j][i][e] *= vref;
          o[j][i][e + 2] *= vref;
        }
      }
    if constexpr (WHOLE) {
      // ---- merge the warps' queries, each warp's in a buffer of its own
      constexpr int ROW = D + 4;
      float* so = reinterpret_cast<float*>(ring + WARPS * 2 * HALF);   // [WARPS][NQ][ROW]
      __shared__ float sm[WARPS][NQ], sl[WARPS][NQ];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int n = j * 8 + 2 * t + e;
          if (n >= nq) continue;
#pragma unroll
          for (int i = 0; i < KW; ++i) {
            so[(warp * NQ + n) * ROW + i * 16 + c] = o[j][i][e];
            so[(warp * NQ + n) * ROW + i * 16 + c + 8] = o[j][i][e + 2];
          }
          if (c == 0) {
            sm[warp][n] = m[j][e];
            sl[warp][n] = l[j][e];
          }
        }
      __syncthreads();
      const int used = min(WARPS, sh.tiles);   // warps that had a tile
      for (int i = threadIdx.x; i < nq * (D / 4); i += 32 * WARPS) {
        const int n = i / (D / 4), d = (i % (D / 4)) * 4;
        Kv8Sum a = {sm[0][n], sl[0][n], *reinterpret_cast<const float4*>(so + n * ROW + d)};
        for (int w = 1; w < used; ++w)
          kv8_join(a, sm[w][n], sl[w][n], *reinterpret_cast<const float4*>(so + (w * NQ + n) * ROW + d));
        kv8_out<T>(p, sh.s0, h, q0 + n, d, D, a.y, a.M, a.l);
      }
      return;
    } else {
      // ---- out, or to scratch, eight queries at a time through the values' buffer
      constexpr int ROW = D == 128 ? D : D + 4;
      const bool all = cnt == sh.tiles;
      const int slot = 2 * run + (tile0 == 0);
      __syncwarp();
      if (!all && lane == (tile0 == 0)) {   // the lane that cleared it
        const int t0 = r.u + su - x + KV8_OVER, w0 = t0 / r.quota;
        p.piece[slot] = {(t0 + sh.tiles - 1) / r.quota - w0 + 1, w0, sh.s0, q0, nq, h, {0, 0}};
      }
      float* so = reinterpret_cast<float*>(ring + (warp * 2 + 1) * HALF);   // [8][ROW]
      static_assert(8 * ROW * 4 <= HALF, "");
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int i = 0; i < KW; ++i) {
            so[(2 * t + e) * ROW + i * 16 + c] = o[j][i][e];
            so[(2 * t + e) * ROW + i * 16 + c + 8] = o[j][i][e + 2];
          }
        __syncwarp();
        for (int i = lane; i < 8 * (D / 4); i += 32) {
          const int n = i / (D / 4), d = (i % (D / 4)) * 4, from = n >> 1;
          const float4 y = *reinterpret_cast<const float4*>(so + n * ROW + d);
          const float ma = __shfl_sync(0xffffffffu, m[j][0], from), mb = __shfl_sync(0xffffffffu, m[j][1], from);
          const float la = __shfl_sync(0xffffffffu, l[j][0], from), lb = __shfl_sync(0xffffffffu, l[j][1], from);
          const float M = n & 1 ? mb : ma, lt = n & 1 ? lb : la;
          if (j * 8 + n >= nq) continue;
          if (all) {
            kv8_out<T>(p, sh.s0, h, q0 + j * 8 + n, d, D, y, M, lt);
          } else {
            const long at = (long)slot * NQ + j * 8 + n;
            *reinterpret_cast<float4*>(p.part + at * D + d) = y;
            if (d == 0) *reinterpret_cast<float2*>(p.part_ml + at * 2) = make_float2(M, lt);
          }
        }
      }
      __syncwarp();
      // ---- the next job
      su += span;
      x = 0;
      cu = su + KV8_OVER;
      if (su < R && ++job == sh.jobs) {
        job = 0;
        do {
          if (++b >= p.q.B) return;   // only where lens changed meanwhile
          sh = kv8_share<NQ, TILE>(p, b);
        } while (sh.jobs == 0);
      }
    }
  }
}

// Merges the jobs that runs cut.  Block w looks at the one or two pieces that run
// w left, and takes its share of each one's job's columns (four channels of a
// query) over all pieces: threads over columns, and over pieces where the share
// has fewer columns than threads.  Latency bounds it: a look at what the run left,
// then loads that do not depend on one another.
// A column of job J over the pieces first, first + step, ...
template <int NQ, int D>
__device__ __forceinline__ Kv8Sum kv8_gather(const Kv8AttnP& p, const Kv8Piece& J, int col, int first, int step) {
  constexpr int BATCH = 8;   // pieces whose loads are in flight together
  const int n = col / (D / 4), d = (col % (D / 4)) * 4;
  Kv8Sum a = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  for (int s0 = first; s0 < J.pieces; s0 += BATCH * step) {
    float2 ml[BATCH];
    float4 y[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int s = min(s0 + i * step, J.pieces - 1);
      const long at = (2 * (long)(J.w0 + s) + (s == 0)) * NQ + n;
      ml[i] = *reinterpret_cast<const float2*>(p.part_ml + at * 2);
      y[i] = *reinterpret_cast<const float4*>(p.part + at * D + d);
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i)
      if (s0 + i * step < J.pieces) kv8_join(a, ml[i].x, ml[i].y, y[i]);
  }
  return a;
}
#define KV8_MERGE 64   // threads
template <typename T, int D, int NT>
__global__ void __launch_bounds__(KV8_MERGE) kv8_attn_merge_kernel(Kv8AttnP p) {
  constexpr int NQ = 8 * NT, C4 = D / 4;
  __shared__ Kv8Sum part[32];
  griddep_wait();
  griddep_release();
  const int tid = threadIdx.x, lane = tid & 31, run = blockIdx.x;
  const Kv8Piece left[2] = {p.piece[2 * run], p.piece[2 * run + 1]};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const Kv8Piece& J = left[k];
    if (J.pieces == 0) continue;
    const int i = run - J.w0, cols = J.nq * C4;
    const int c0 = (int)((long)i * cols / J.pieces), c1 = (int)((long)(i + 1) * cols / J.pieces);
    auto out = [&](const Kv8Sum& a, int col) {
      kv8_out<T>(p, J.s0, J.h, J.q0 + col / C4, (col % C4) * 4, D, a.y, a.M, a.l);
    };
    if (c1 - c0 > 32) {
      for (int col = c0 + tid; col < c1; col += KV8_MERGE) out(kv8_gather<NQ, D>(p, J, col, 0, 1), col);
    } else if (c0 < c1) {
      int wide = 1;
      while (wide < c1 - c0) wide <<= 1;
      const int col = min(c0 + (lane & (wide - 1)), c1 - 1);
      Kv8Sum a = kv8_gather<NQ, D>(p, J, col, tid / wide, KV8_MERGE / wide);
      for (int o = wide; o < 32; o <<= 1) {
        const float M = __shfl_xor_sync(0xffffffffu, a.M, o), l = __shfl_xor_sync(0xffffffffu, a.l, o);
        float4 y;
        y.x = __shfl_xor_sync(0xffffffffu, a.y.x, o); y.y = __shfl_xor_sync(0xffffffffu, a.y.y, o);
        y.z = __shfl_xor_sync(0xffffffffu, a.y.z, o); y.w = __shfl_xor_sync(0xffffffffu, a.y.w, o);
        kv8_join(a, M, l, y);
      }
      if (J.pieces > 32 / wide) {   // the second warp has some
        __syncthreads();
        if (tid >= 32) part[lane] = a;
        __syncthreads();
        if (tid < 32) kv8_join(a, part[lane].M, part[lane].l, part[lane].y);
      }
      if (tid < wide && c0 + tid < c1) out(a, c0 + tid);
    }
  }
}

// ---------------------------------------------------------------------------
// Entry points
// ---------------------------------------------------------------------------
static const char* kv8_check_shape(const gpt_kv8_cache* c) {
  if (!c) return "cache is NULL";
  if (c->kind != GPT_KV8_INT8 && c->kind != GPT_KV8_E4M3) return "unknown cache kind";
  if (c->n_layers < 1 || c->n_pages < 1 || c->n_kv_heads < 1 || c->n_kv_heads > 1024)
    return "n_layers, n_pages and n_kv_heads must be >= 1 (n_kv_heads <= 1024)";
  if ((long)c->n_pages * c->n_kv_heads * (c->page * c->head_dim / 16) >= 0xffffffffL)
    return "one layer's keys must be below 64 GB";
  if (c->head_dim != 16 && c->head_dim != 32 && c->head_dim != 64 && c->head_dim != 128)
    return "head_dim must be 16, 32, 64 or 128";
  if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) return "page must be 16, 32, 64 or 128";
  return "";
}
const char* kv8_check_cache(const gpt_kv8_cache* c) {
  const char* why = kv8_check_shape(c);
  if (*why) return why;
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

int kv8_sms() {
  static PerDevice known;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return 148;
  }
  const int n = per_device(known, dev, [](int d) {
    int x = 0;
    if (cudaDeviceGetAttribute(&x, cudaDevAttrMultiProcessorCount, d) == cudaSuccess) return x;
    cudaGetLastError();
    return 0;
  });
  return n > 0 ? n : 148;
}

// Heads (columns of heads) that a block of append or read takes: all of them when
// there are blocks enough for every SM to hold eight of them even so, fewer for
// small calls, down to one.
static int kv8_per_block(int jobs, int n) {
  const int groups = std::min(n, (kv8_sms() * 8 * 2 + 2 * jobs - 1) / (2 * jobs));
  return (n + groups - 1) / groups;
}

template <typename T, int KIND, int VPT, int TPH>
static cudaError_t append_v(Kv8AppendP p, const gpt_kv8_cache& c, int jobs, cudaStream_t s) {
  // (a warp per head: no more of them than heads; 84653 tokens of one head of 128, pages of 16: 21 us with one warp a
  // block, 47 with four)
  const int threads = TPH == 128 ? 128 : 32 * std::min(4, c.n_kv_heads), heads = threads / TPH;
  const size_t smem = (size_t)VPT * threads * 16 + (size_t)heads * c.page * (c.head_dim + KV8_PAD);
  if (VPT == 16) {   // 50 KB
    const cudaError_t e = cudaFuncSetAttribute(kv8_append_kernel<T, KIND, VPT, TPH>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, 56 * 1024);
    if (e != cudaSuccess) return e;
  }
  p.heads = kv8_per_block(jobs, (c.n_kv_heads + heads - 1) / heads) * heads;
  const dim3 grid(jobs, (c.n_kv_heads + p.heads - 1) / p.heads, 2);
  return launch_k(kv8_append_kernel<T, KIND, VPT, TPH>, grid, dim3(threads), smem, s, p);
}

template <typename T, int KIND>
static cudaError_t append_t(const Kv8AppendP& p, const gpt_kv8_cache& c, int jobs, cudaStream_t s) {
  if (!p.q.start) {
    const dim3 one((unsigned)(((long)p.q.B * c.n_kv_heads * 2 + 3) / 4));
    switch (c.head_dim) {
      case 16: return launch_k(kv8_append_one_kernel<T, KIND, 16>, one, dim3(128), 0, s, p);
      case 32: return launch_k(kv8_append_one_kernel<T, KIND, 32>, one, dim3(128), 0, s, p);
      case 64: return launch_k(kv8_append_one_kernel<T, KIND, 64>, one, dim3(128), 0, s, p);
      default: return launch_k(kv8_append_one_kernel<T, KIND, 128>, one, dim3(128), 0, s, p);
    }
  }
  switch (c.page * c.head_dim) {
    case 256: return append_v<T, KIND, 1, 32>(p, c, jobs, s);
    case 512: return append_v<T, KIND, 2, 32>(p, c, jobs, s);
    case 1024: return append_v<T, KIND, 4, 32>(p, c, jobs, s);
    case 2048: return append_v<T, KIND, 8, 32>(p, c, jobs, s);
    case 4096: return append_v<T, KIND, 4, 128>(p, c, jobs, s);
    case 8192: return append_v<T, KIND, 8, 128>(p, c, jobs, s);
    default: return append_v<T, KIND, 16, 128>(p, c, jobs, s);
  }
}

struct Kv8Plan {
  int nt, blocks, warps;   // warps of blocks that take whole jobs, or 0
  bool fits;
  size_t part, ml, piece;  // floats (piece: in floats too)
};
// Queries a job: 16 where that saves enough passes over the cache (12 warps an SM
// instead of 16, and more instructions a pass).  64 x 4096 tokens, 8 heads of 64, us
// with 8 and with 16: 8 queries a sequence 58 and 73, 9 to 16 92 and 73, 17 to 24 128
// and 128, 25 to 32 178 and 129, so 9 to 16 and 25 to 32 take 16.  Where the
// sequences' rows differ, only their mean is known here, and half a job is lost
// a sequence on average: 64 x 3000 tokens, means of 8, 12, 14, 16, 18, 22, 34: 55, 70,
// 76, 80, 93, 99, 132 with 8 and 63, 74, 81, 81, 87, 95, 124 with 16, so 16 from 19 on.
// Jobs of 32 queries were no faster than two of 16.
//
// Blocks: as many as are resident at once, or one per job where no row has room
// for more than KV8_WHOLE tokens and the jobs are not many times the blocks that fit.
// Heads of 64, us whole and in runs: 300 jobs of 64, 256, 1024 tokens 5.5, 6.9, 16 and
// 8.6, 16, 22; 1200 jobs 13, 18, 39 and 11, 23, 46; 1700 jobs 14, 21, 46 and 12, 23, 56;
// 3000 jobs 25, 34, 79 and 18, 35, 82, with lengths spread below those 32, 33, 45 and
// 22, 26, 38.  (Rows of up to 64 tokens would be better in runs from about 900 jobs on;
// the bound is the longer rows'.)  Whole jobs have twice the warps where two blocks an
// SM are enough (one sequence of 512 tokens and 12 heads: 5.9 us, 6.6 with four warps).
static Kv8Plan kv8_plan(const gpt_kv8_cache& c, const gpt_kv8_batch& b, int H) {
  Kv8Plan P = {};
  const int G = H / c.n_kv_heads, nsm = kv8_sms();
  const long mean = b.B ? ((long)b.rows * G + b.B - 1) / b.B : G;
  P.nt = (b.start && b.rows != b.B ? mean > 18 : 10 * ((G + 7) / 8) > 17 * ((G + 15) / 16)) ? 2 : 1;
  const int nq = 8 * P.nt;
  const long jobs = (b.start ? (long)b.rows * G / nq + b.B : (long)b.B * ((G + nq - 1) / nq)) * c.n_kv_heads;
  const bool whole = (long)b.max_pages * c.page <= KV8_WHOLE && jobs <= 12L * nsm;
  const int tile = kv8_tile(c.head_dim, P.nt, whole);
  const long tiles = ((long)b.max_pages * c.page + tile - 1) / tile;
  P.fits = jobs * (tiles + KV8_OVER) <= 0x7fffffffL;   // units are counted in 32 bits
  if (whole) {
    P.blocks = (int)jobs;
    P.warps = jobs <= 2 * nsm ? KV8_WIDE : KV8_NW;
    return P;
  }
  P.blocks = (int)std::min((long)kv8_resident(c.head_dim, P.nt, 0) * nsm, (jobs * tiles + KV8_NW - 1) / KV8_NW);
  const size_t slots = (size_t)P.blocks * KV8_NW * 2;
  P.part = slots * nq * c.head_dim;
  P.ml = slots * nq * 2;
  P.piece = slots * (sizeof(Kv8Piece) / sizeof(float));
  return P;
}

template <typename T, int D, int NT, int KIND, int NW>
static cudaError_t attn_launch(const Kv8AttnP& p, const Kv8Plan& P, cudaStream_t s) {
  constexpr size_t smem = kv8_attn_smem<D, NT, NW>();
  if (smem > 40000) {
    static PerDevice ready;   // 1: the attribute is set
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    per_device(ready, dev, [&](int) {
      e = cudaFuncSetAttribute(kv8_attn_kernel<T, D, NT, KIND, NW>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)smem);
      return e == cudaSuccess ? 1 : 0;
    });
    if (e != cudaSuccess) return e;
  }
  ++g_kernel_launches;
  return launch_k(kv8_attn_kernel<T, D, NT, KIND, NW>, dim3(P.blocks), dim3(32 * (NW ? NW : KV8_NW)), smem, s, p);
}
template <typename T, int D, int NT, int KIND>
static cudaError_t attn_nt(const Kv8AttnP& p, const Kv8Plan& P, cudaStream_t s) {
  if (P.warps == KV8_WIDE) return attn_launch<T, D, NT, KIND, KV8_WIDE>(p, P, s);
  if (P.warps == KV8_NW) return attn_launch<T, D, NT, KIND, KV8_NW>(p, P, s);
  const cudaError_t e = attn_launch<T, D, NT, KIND, 0>(p, P, s);
  if (e != cudaSuccess) return e;
  ++g_kernel_launches;
  return launch_k(kv8_attn_merge_kernel<T, D, NT>, dim3(P.blocks * KV8_NW), dim3(KV8_MERGE), 0, s, p);
}
template <typename T, int D, int KIND>
static cudaError_t attn_d(const Kv8AttnP& p, const Kv8Plan& P, cudaStream_t s) {
  return P.nt == 1 ? attn_nt<T, D, 1, KIND>(p, P, s) : attn_nt<T, D, 2, KIND>(p, P, s);
}
template <typename T, int KIND>
static cudaError_t attn_t(const Kv8AttnP& p, const Kv8Plan& P, int D, cudaStream_t s) {
  switch (D) {
    case 16: return attn_d<T, 16, KIND>(p, P, s);
    case 32: return attn_d<T, 32, KIND>(p, P, s);
    case 64: return attn_d<T, 64, KIND>(p, P, s);
    default: return attn_d<T, 128, KIND>(p, P, s);
  }
}

extern "C" {

int gpt_kv8_append(const gpt_kv8_cache* c, int layer, const gpt_kv8_batch* b, const void* k, long ldk, const void* v,
                   long ldv, int dtype, uint32_t* err, void* stream) {
  const long w = c ? (long)c->n_kv_heads * c->head_dim : 0;
  const char* why = kv8_check_call(c, layer, b, dtype, k, ldk, v, ldv, w, w);
  if (*why) return kv8_refuse("gpt_kv8_append", why);
  if (b->B == 0 || b->rows == 0) return GPT_OK;
  Kv8AppendP p = {kv8_layer(*c, layer), kv8_seqs(*b), (const uint16_t*)k, (const uint16_t*)v, ldk, ldv, 0, err};
  const int jobs = kv8_jobs(*b, p.L.lp);
  cudaStream_t s = (cudaStream_t)stream;
  const bool i8 = c->kind == GPT_KV8_INT8;
  ++g_kernel_launches;
  return kv8_done("gpt_kv8_append",
                  dtype == GPT_PRECISION_BF16
                      ? (i8 ? append_t<bf16, GPT_KV8_INT8>(p, *c, jobs, s) : append_t<bf16, GPT_KV8_E4M3>(p, *c, jobs, s))
                      : (i8 ? append_t<f16, GPT_KV8_INT8>(p, *c, jobs, s) : append_t<f16, GPT_KV8_E4M3>(p, *c, jobs, s)));
}

int gpt_kv8_read(const gpt_kv8_cache* c, int layer, const gpt_kv8_batch* b, void* k, long ldk, void* v, long ldv,
                 int dtype, uint32_t* err, void* stream) {
  const long w = c ? (long)c->n_kv_heads * c->head_dim : 0;
  const char* why = kv8_check_call(c, layer, b, dtype, k, ldk, v, ldv, w, w);
  if (*why) return kv8_refuse("gpt_kv8_read", why);
  if (b->B == 0 || b->rows == 0) return GPT_OK;
  Kv8ReadP p = {kv8_layer(*c, layer), kv8_seqs(*b), (uint16_t*)k, (uint16_t*)v, ldk, ldv, 0, err};
  const int jobs = kv8_jobs(*b, 4), cols = (int)((w + 127) / 128);
  p.cols = kv8_per_block(jobs, cols);
  const dim3 grid(jobs, (cols + p.cols - 1) / p.cols, 2);
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
  const char* why = kv8_check_shape(c);
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
  *bytes = (P.part + P.ml + P.piece) * sizeof(float);
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
  if (!P.fits) return kv8_refuse("gpt_kv8_attention", "too many queries and tokens");
  if (!P.warps && (!work || work_bytes < (P.part + P.ml + P.piece) * sizeof(float) || ((uintptr_t)work & 15)))
    return kv8_refuse("gpt_kv8_attention", "work must be 16-byte aligned and hold gpt_kv8_attention_work bytes");
  Kv8AttnP p = {kv8_layer(*c, layer), kv8_seqs(*b), (const uint16_t*)q, (uint16_t*)out, lse, ldq, ldo,
                n_heads, n_heads / c->n_kv_heads, b->max_pages * c->page, scale, (float*)work, (float*)work + P.part,
                (Kv8Piece*)((float*)work + P.part + P.ml), err};
  cudaStream_t s = (cudaStream_t)stream;
  const bool i8 = c->kind == GPT_KV8_INT8;
  const int D = c->head_dim;
  return kv8_done("gpt_kv8_attention",
                  dtype == GPT_PRECISION_BF16
                      ? (i8 ? attn_t<bf16, GPT_KV8_INT8>(p, P, D, s) : attn_t<bf16, GPT_KV8_E4M3>(p, P, D, s))
                      : (i8 ? attn_t<f16, GPT_KV8_INT8>(p, P, D, s) : attn_t<f16, GPT_KV8_E4M3>(p, P, D, s)));
}

}  // extern "C"
