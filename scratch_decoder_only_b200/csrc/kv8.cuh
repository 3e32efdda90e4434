// Shared by the kernels of the 8-bit paged key/value cache (kv8.cu: append,
// read, attention; kv8_pages.cu: the pages' bookkeeping).
#pragma once
#include "gpt.h"
#include "launch.h"
#include "per_device.h"

// One layer of a cache: codes k [n_pages][Hkv][P][D], v [n_pages][Hkv][P/16][D][16]
// and one scale per (page, head).
struct Kv8Layer {
  uint8_t *k, *v;
  float *ks, *vs;
  int n_pages, Hkv, lp, ld;   // lp = log2(P), ld = log2(D)
};

struct Kv8Seqs {
  const int *start, *lens, *table;
  int B, max_pages, ld_table, rows;
};

static inline int ilog2(int x) {
  int r = 0;
  while ((1 << r) < x) ++r;
  return r;
}

// "" or why the description of a cache cannot be used
const char* kv8_check_cache(const gpt_kv8_cache* c);
// SMs of the current device (148, a B200's, where there is none to ask)
int kv8_sms();

static inline Kv8Layer kv8_layer(const gpt_kv8_cache& c, int layer) {
  Kv8Layer L;
  const size_t pages = (size_t)layer * c.n_pages * c.n_kv_heads, bytes = (size_t)c.page * c.head_dim;
  L.k = (uint8_t*)c.k + pages * bytes;
  L.v = (uint8_t*)c.v + pages * bytes;
  L.ks = c.k_scale + pages;
  L.vs = c.v_scale + pages;
  L.n_pages = c.n_pages;
  L.Hkv = c.n_kv_heads;
  L.lp = ilog2(c.page);
  L.ld = ilog2(c.head_dim);
  return L;
}

// Rows [s0, s0 + n) of a batch belong to sequence b, whose newest token is
// row s0 + n - 1 at position len - 1.
struct Kv8Seq {
  int b, s0, n, len;
};

// Ragged batches cut every sequence's work into jobs on the device, without
// the host knowing its rows: base(b), non-decreasing in b, is a bound on the
// jobs of the sequences before b, and job j belongs to the last b with
// base(b) <= j.  All threads of the block call this; false: no such sequence.
// It is found among as many places as the block has threads at a time: two rounds
// for 128 x 128 sequences (8192 of 4 tokens, 2 heads of 64: 67 us an append; 425 with a
// look at every start and blocks of four warps). Where starts decrease any b may come out, and the caller's
// bounds hold all the same.
template <class Base>
__device__ __forceinline__ bool kv8_find(const Kv8Seqs& q, int job, Base base, Kv8Seq& s, int& first, unsigned* err) {
  const int nth = blockDim.x;
  if (job == 0) {
    bool bad = false;
    for (int i = threadIdx.x; i < q.B; i += nth)
      bad |= q.start[i] < 0 || q.start[i + 1] < q.start[i] || q.start[i + 1] > q.rows;
    if (bad) set_dev_err(err, GPT_DEVERR_START);
  }
  int b = 0;
  for (int n = q.B;;) {   // one of n from b on
    const int step = n <= nth ? 1 : (int)((unsigned)(n + nth - 1) / (unsigned)nth), i = b + (int)threadIdx.x * step;
    const bool le = i < b + n && base(i, min(max(q.start[i], 0), q.rows)) <= job;
    const int cnt = __syncthreads_count(le);
    if (cnt == 0) return false;
    b += (cnt - 1) * step;
    if (step == 1) break;
    n = min(step, n - (cnt - 1) * step);
  }
  s.b = b;
  s.s0 = min(max(q.start[s.b], 0), q.rows);
  s.n = min(max(q.start[s.b + 1], s.s0), q.rows) - s.s0;
  s.len = q.lens[s.b];
  first = job - base(s.b, s.s0);
  return true;
}

// ---- 8-bit codes
__device__ __forceinline__ uint32_t f16x2_sub(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Four codes widened to two f16 pairs, exactly: int8 by setting the biased
// byte into the low mantissa bits of 1024 and subtracting 1152; every e4m3
// value is an f16 value.
template <int KIND>
__device__ __forceinline__ void kv8_widen(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (KIND == GPT_KV8_INT8) {
    const uint32_t x = w ^ 0x80808080u;
    lo = f16x2_sub(__byte_perm(x, 0x64646464u, 0x4140), 0x64806480u);
    hi = f16x2_sub(__byte_perm(x, 0x64646464u, 0x4342), 0x64806480u);
  } else {
    asm("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
  }
}
__device__ __forceinline__ float2 f16x2_float(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// Four scaled values (magnitude at most the code type's largest) to codes,
// rounded half to even.
template <int KIND>
__device__ __forceinline__ uint32_t kv8_code4(float a, float b, float c, float d) {
  if constexpr (KIND == GPT_KV8_INT8) {
    const int ia = min(max(__float2int_rn(a), -127), 127), ib = min(max(__float2int_rn(b), -127), 127);
    const int ic = min(max(__float2int_rn(c), -127), 127), id = min(max(__float2int_rn(d), -127), 127);
    return __byte_perm(__byte_perm(ia, ib, 0x0040), __byte_perm(ic, id, 0x0040), 0x5410);
  } else {
    uint32_t r;
    asm("{.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
        "mov.b32 %0, {l, h};\n\t}" : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
  }
}
