// Single-token attention over a paged cache held in 4 bits or in bf16.
//
// out[b][h] = sum_j softmax_j(<m R(L-1) q[b][h], K_j> / sqrt(128)) V_j over the rows j that head h's KV
// head attends: every row, or sinks and window, or sinks, window and a selected list.
//
// Work layout.  The attended rows of all (sequence, KV head) slices are cut into units of 16
// rows: whole 16-token blocks of the pages (edges masked), or 16 listed rows; U consecutive units of a
// slice are an item.  Every CTA (one an SM) takes an equal contiguous share of the items, and its
// warps take them in turn, each through a ring of its own in shared memory.  A warp looks up 32 units at a
// time, a lane each (slice, page, byte offset, row mask), so the search, the division and the block
// table cost 1/32 a unit, and those lanes start the copies: a block is one bulk copy (2304 bytes in 4
// bits: K, V and scales together).  Listed units are gathered by 16-byte asynchronous copies, their
// positions loaded two items ahead, their pages one.
// (Two producer warps for the whole CTA took 737 us for 1M rows where this took 411: one lane's waits and copies in turn.)
// Where the slices fit the CTAs well, every CTA's share lies in one slice: a share that straddles two
// pays for their queries and their merge twice.
// Warps keep their own running maximum and sum, merged in a fixed order at the end of a slice's piece;
// the last CTA to finish a slice (a ticket) merges the CTAs' states in order, so the result does
// not depend on timing.
//
// Matrix mapping (mma.sync m16n8k16, float32 sums).  The 16 rows of the operand hold the group's heads more
// than once, as a high part and residuals, so that no bits of queries and probabilities are lost:
//   4 bits: float16 high parts (rows 0-7) and residuals (rows 8-15), 22 bits.  Queries are brought to a maximum of
//     2^14 a head; a scale group whose own maximum is 2^-13 of that still keeps 22 bits.  Probabilities are 2^14 times
//     their value at most, and value scales below 2 by the largest scale the warp has met (a power of two, moved like the
//     running maximum); the products that count keep 22 bits while the scales met lie within 2^16 of each other.  Where queries
//     or scales lie farther apart, the CTA takes its piece of the slice once more at the end, in float32 (attend_wide).
//     A code word (8 nibbles) becomes four float16 pairs, (nibble j, nibble j + 4).
//     Scores: word w of a lane's 16 bytes is scale group w of its 32 dims, so the products of a group
//     are summed by themselves (starting at -8 times the sum of the queries, which centres
//     the codes) and scaled once a (row, group), not once an element.
//     Values: the halves of two rows' words are merged by one byte permute into (row, row + 1)
//     pairs and centred by a multiply-add (their sums run over the whole context: no cancellation is
//     put into them); column tile t holds dims 16 n + t, all of scale group t / 4, whose
//     scales go into the probabilities (four sets of them, in packed float16 with exact residuals).
//   bf16: three bf16 parts (24 bits).  Up to 4 heads they share one operand (high rows 0-3, middle rows 4-7, low
//     rows 8-11; lanes 16 apart add up), more heads take a second product for the low part.
//     Rows come by matrix loads from the swizzled block.
//
// Masked rows: their score is -infinity and their value scale (bf16: their value) 0, whatever the page holds there.
#include <cfloat>
#include <climits>

#include <cuda_fp16.h>

#include "spa_paged.cuh"

namespace spa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kNoMax = -FLT_MAX;     // running maximum before the first row: no score is below it

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void mbar_init(uint32_t bar, unsigned n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar, unsigned n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar, uint64_t pol) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar), "l"(pol)
      : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, unsigned parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0u;
}
__device__ __forceinline__ unsigned long long now_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}
// Waits for a phase to end, for two seconds at most; for 100 us once a wait of the CTA has run out (*late): the phases
// behind a missing copy do not match any more, and two seconds an item would not end.
// Out of line where it really waits: inlined, the loop's registers cost 1M rows 356 us in place of 347.
__device__ __noinline__ bool mbar_wait_on(uint32_t bar, unsigned parity, volatile int* late) {
  const unsigned long long t0 = now_ns();
  while (!mbar_try(bar, parity)) {
    if (now_ns() - t0 > (*late ? 100000ull : 2000000000ull)) {
      *late = 1;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool mbar_wait(uint32_t bar, unsigned parity, volatile int* late) {
  return mbar_try(bar, parity) || mbar_wait_on(bar, parity, late);
}
__device__ __forceinline__ uint64_t l2_evict_first() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;\n" : "=l"(p));
  return p;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// d = A B + c, c.x in the upper rows and c.y in the lower ones.
template <bool F16>
__device__ __forceinline__ void mma16816_from(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float2 c) {
  if (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%10,%11,%11};\n"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c.x), "f"(c.y));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%10,%11,%11};\n"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c.x), "f"(c.y));
}
__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
// A read that stays where it is: 32 registers of query operands would not fit beside the sums.
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
  return r;
}
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Nibbles (0, 4), (1, 5), (2, 6), (3, 7) of w as float16 pairs of n 2^-22, the second and fourth 16 times that: a
// mask each, since small integers under a zero exponent are subnormals.  The tensor cores align a product by its
// operands' exponent fields, so a subnormal's leading zeros are lost from the sum: as high up as two
// pairs of a shift can go they cost 2^-22 of the sum (at the bottom, 2^-20).
__device__ __forceinline__ void code_pairs(uint32_t w, uint32_t (&r)[4]) {
  const uint32_t u = w << 2, v = w >> 6;
  r[0] = u & 0x003c003cu;
  r[1] = u & 0x03c003c0u;
  r[2] = v & 0x003c003cu;
  r[3] = v & 0x03c003c0u;
}
constexpr float kKeyUnit = 4194304.f;   // 2^22: what a key's code of 1 stands for, inverted
// The same nibbles as (n - 8) 2^-10, normal numbers and exact.
__device__ __forceinline__ void centred_pairs(uint32_t w, uint32_t (&r)[4]) {
  const uint32_t v = w >> 8;
  const uint32_t up = 0x74007400u, up16 = 0x64006400u, centre = 0xa000a000u;   // 2^14, 2^10, -8 2^-10
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r[0]) : "r"(w & 0x000f000fu), "r"(up), "r"(centre));
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r[1]) : "r"(w & 0x00f000f0u), "r"(up16), "r"(centre));
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r[2]) : "r"(v & 0x000f000fu), "r"(up), "r"(centre));
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r[3]) : "r"(v & 0x00f000f0u), "r"(up16), "r"(centre));
}
constexpr float kValueUnit = 1024.f;   // 2^10: what a value's code of 1 stands for, inverted
__device__ __forceinline__ uint32_t bits(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
__device__ __forceinline__ __half2 half2_of(uint32_t u) { return *reinterpret_cast<const __half2*>(&u); }
// Float16 high parts and residuals of a pair.
__device__ __forceinline__ void split_f16(float x, float y, __half2& hi, __half2& lo) {
  hi = __floats2half2_rn(x, y);
  const float2 f = __half22float2(hi);
  lo = __floats2half2_rn(x - f.x, y - f.y);
}
// The three bf16 parts of a pair.
__device__ __forceinline__ void split_bf16(float x, float y, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  hi = pack2(x, y);
  x -= bf16_lo(hi);
  y -= bf16_hi(hi);
  mid = pack2(x, y);
  lo = pack2(x - bf16_lo(mid), y - bf16_hi(mid));
}
// 4 bits: probabilities are 2^14 times their value (less where scores' steps are coarser), value scales in float16 below 2.  A
// probability in two float16 parts is off by 2^-25 at most where its leading bits run out, against 2^14 of the row with the
// largest: a row whose scale is 2^16 above that row's puts 2^-23 of the sum into it, and a scale that far down is exact.
constexpr float kProbExp = 14.f;
// In bf16 bits: the least and the largest bound of the value scales (2^-100, 2^80: 2^14 times the sum of 2^24 rows stays
// in float32; what has larger ones is taken in float32, too), and 2^8 and 2^16: scales from the bound down to 2^-8 of it need no look.
constexpr unsigned kScaleLow = 0x0d80u, kScaleHigh = 0x6780u, kScaleNear = 0x400u, kScaleSpan = 0x800u;

// Rows of one slice: blocks [0, nb0) (sinks), blocks [b1, b1 + nb1) (window, or every block), then cnt listed rows.
struct Slice {
  int L, n_s, w_lo;
  int nb0, b1, nb1, cnt;
};
__device__ __forceinline__ int units_of(const Slice& S) { return S.nb0 + S.nb1 + (S.cnt + 15) / 16; }
__device__ __forceinline__ Slice make_slice(const PagedAttendArgs& A, int g, int L, int cnt) {
  Slice S;
  S.L = L;
  S.cnt = cnt;
  const int nbk = (L + kBlockTok - 1) / kBlockTok;
  if (A.all_rows[g]) {
    S.n_s = S.w_lo = S.nb0 = S.b1 = 0;
    S.nb1 = nbk;
    return S;
  }
  const SinkWindow sw(L, A.n_sink, A.window);
  S.n_s = sw.n_s;
  S.w_lo = sw.w_lo;
  S.nb0 = (sw.n_s + kBlockTok - 1) / kBlockTok;
  S.b1 = max(S.nb0, sw.w_lo / kBlockTok);
  S.nb1 = sw.w_lo < L ? max(nbk - S.b1, 0) : 0;
  return S;
}

// A unit, held by the lane that looked it up.
struct Unit {
  long long off;   // block: byte offset in the pool; list: index of its first entry
  unsigned info;   // attended rows (16 bits), kList
  int s;           // slice
  int bg;          // its sequence (<< 8) and head
};
// Listed rows on their way.
struct Rows {
  int pos, id;      // lane l: position of row l of the item (-1: not attended or not listed) and its page
  int s, bg;        // the slice, its sequence (<< 8) and head
};
constexpr unsigned kList = 0x10000u;

// Rotated queries in shared memory: the dims 32 apart of 8 heads fall into 32 banks.
constexpr int kQRow = 161;
__device__ __forceinline__ int q_at(int d) { return d + 8 * (d >> 5); }

// Queries of slice s: warp h takes head h of the group, a lane the pairs lane and lane + 32 (of dims that do not turn: neighbours).
__device__ __forceinline__ void pair_at(const RopeTab128& tab, int j, int& d0, int& d1) {
  const int half = tab.rot / 2;
  d0 = j >= half ? tab.rot + 2 * (j - half) : tab.interleaved ? 2 * j : j;
  d1 = j >= half || tab.interleaved ? d0 + 1 : d0 + half;
}
__device__ __forceinline__ float4 load_queries(const PagedAttendArgs& A, const RopeTab128& tab, int s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, Hkv = A.pool.Hkv;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  if (warp < A.G) {
    const size_t at = ((size_t)(s / Hkv) * A.Hq + (size_t)(s % Hkv) * A.G + warp) * kHeadDim;
    int a0, a1, b0, b1;
    pair_at(tab, lane, a0, a1);
    pair_at(tab, lane + 32, b0, b1);
    if (A.q_f32) {
      const float* q = static_cast<const float*>(A.q) + at;
      x = make_float4(q[a0], q[a1], q[b0], q[b1]);
    } else {
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(A.q) + at;
      x = make_float4(__bfloat162float(q[a0]), __bfloat162float(q[a1]), __bfloat162float(q[b0]), __bfloat162float(q[b1]));
    }
  }
  return x;
}
// To qs, rotated at position L - 1, times scale / ln 2.
__device__ __forceinline__ void turn_queries(const PagedAttendArgs& A, const RopeTab128& tab, float4 x, float* qs, int L) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (warp >= A.G) return;
  float* const q = qs + warp * kQRow;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int j = lane + 32 * i;
    int d0, d1;
    pair_at(tab, j, d0, d1);
    const float q0 = i ? x.z : x.x, q1 = i ? x.w : x.y;
    float c = 1.f, sn = 0.f;
    if (j < tab.rot / 2) rope_cs(tab.f_pi[j], (double)(L - 1), (float)tab.mag, c, sn);
    q[q_at(d0)] = (q0 * c - q1 * sn) * A.scale_log2;
    q[q_at(d1)] = (q0 * sn + q1 * c) * A.scale_log2;
  }
}

// The warps' states in mbuf to the output, or to the CTA's state and, from the last of the slice's CTAs c0 .. c1, to the output.
template <int W, bool kF16>
__device__ __forceinline__ void finish(const PagedAttendArgs& A, const float* mbuf, int* s_merge, int s, int c0, int c1) {
  constexpr int kBoxes = (W + 1) / 2;
  const int tid = threadIdx.x, G = A.G;
  const int b = s / A.pool.Hkv;
  const size_t h0 = (size_t)b * A.Hq + (size_t)(s - b * A.pool.Hkv) * G;
  const int xl = tid & 31, xh = xl >> 2;   // thread x: lane xl's sums of column tiles 2 (x / 32) and the next; its head
  const bool takes = tid < 256 && xh < G;
  float4* const part = reinterpret_cast<float4*>(A.part);
  constexpr int kState = kMergeWords / 4;
  // normalised sums of 4, to the output
  auto put = [&](float4 v, float M, float Ls) {
    const float inv = Ls == 0.f ? 0.f : 1.f / Ls;   // no weight at all: zeros
    const int k2 = 2 * (tid >> 5);                  // column tile
    float* const to = A.out + (h0 + xh) * kHeadDim;
    // (tile nt, e) is dim 32 t4 + 16 e + nt in 4 bits, 8 nt + 2 t4 + e in bf16
    if (kF16) {
      float2* const at = reinterpret_cast<float2*>(to + 32 * (xl & 3) + k2);
      at[0] = make_float2(v.x * inv, v.z * inv);
      at[8] = make_float2(v.y * inv, v.w * inv);
    } else {
      float2* const at = reinterpret_cast<float2*>(to + 8 * k2 + 2 * (xl & 3));
      at[0] = make_float2(v.x * inv, v.y * inv);
      at[4] = make_float2(v.z * inv, v.w * inv);
    }
    if (A.lse && tid < 32 && (xl & 3) == 0) A.lse[h0 + xh] = Ls == 0.f ? -INFINITY : M + log2f(Ls);
  };
  if (takes) {
    float M = kNoMax, Ls = 0.f;
    float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
    float2 ml[kBoxes];
#pragma unroll
    for (int i = 0; i < kBoxes; ++i) {
      ml[i] = *reinterpret_cast<const float2*>(mbuf + (size_t)i * kMergeWords + 1024 + 4 * xl);
      M = fmaxf(M, ml[i].x);
    }
#pragma unroll
    for (int i = 0; i < kBoxes; ++i) {
      const float w = exp2f(ml[i].x - M);
      const float4 v = *reinterpret_cast<const float4*>(mbuf + (size_t)i * kMergeWords + 4 * tid);
      Ls += ml[i].y * w;
      num.x += v.x * w;
      num.y += v.y * w;
      num.z += v.z * w;
      num.w += v.w * w;
    }
    if (c0 == c1) {
      put(num, M, Ls);
    } else {
      float4* const to = part + (size_t)(blockIdx.x + s) * kState;
      to[tid] = num;
      if (tid < 32) to[256 + xl] = make_float4(M, Ls, 0.f, 0.f);
      __threadfence();
    }
  }
  if (c0 == c1) return;
  // ---- the last CTA of the slice merges the CTAs' states in order
  __syncthreads();
  if (tid == 0) *s_merge = atomicAdd(&A.ticket[s], 1u) == (unsigned)(c1 - c0);
  __syncthreads();
  if (!*s_merge) return;
  __threadfence();
  if (takes) {
    float M = kNoMax, Ls = 0.f;
    float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kB = 8;
    for (int c = c0; c <= c1; c += kB) {
      float4 v[kB], ml[kB];
#pragma unroll
      for (int i = 0; i < kB; ++i) {
        const float4* from = part + (size_t)(min(c + i, c1) + s) * kState;
        v[i] = __ldcg(from + tid);
        ml[i] = __ldcg(from + 256 + xl);
      }
#pragma unroll
      for (int i = 0; i < kB; ++i) {
        if (c + i > c1) break;
        const float mn = fmaxf(M, ml[i].x), sa = exp2f(M - mn), sb = exp2f(ml[i].x - mn);
        Ls = Ls * sa + ml[i].y * sb;
        num.x = num.x * sa + v[i].x * sb;
        num.y = num.y * sa + v[i].y * sb;
        num.z = num.z * sa + v[i].z * sb;
        num.w = num.w * sa + v[i].w * sb;
        M = mn;
      }
    }
    put(num, M, Ls);
  }
  if (tid == 0) A.ticket[s] = 0u;   // ready for the next call
}

// 4-bit word to 8 values n - 8 (exact small integers).
__device__ __forceinline__ void centred(unsigned w, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(0x4b000000u | (w >> (4 * i) & 15u)) - 8388616.f;
}
// A CTA's piece of a slice of 4-bit pages in float32 throughout, for value scales, or scale groups of a query, that are too far
// apart for float16 products.  The queries are in qs; `unit` is the piece's first unit of the slice, `items` the number of its
// items, which the warps take in turn.  A lane scores one row of an item for every head, then sums 4 dims over the rows.
// Leaves the states in mbuf as the kernel's own hand-over does.  One such row among 1M, 8 KV heads of 8 queries: 2.2 ms in
// place of 0.37 (one CTA takes 57000 rows again); among 64K, 170 us in place of 50.  Loads of queries and shuffles bound it.
template <int W, int U>
__device__ __forceinline__ void attend_wide(const PagedAttendArgs& A, const Slice& S, const float* qs, float* mbuf, int s, int unit, int items) {
  static_assert(U == 2, "a lane a row of an item");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = A.G;
  const int b = s / A.pool.Hkv, g = s - b * A.pool.Hkv;
  // queries as [8][128], for 16-byte loads; zeros for heads that the group does not have
  for (int i = threadIdx.x; i < kMaxGroup * kHeadDim; i += W * 32)
    mbuf[i] = i / kHeadDim < G ? qs[i / kHeadDim * kQRow + q_at(i % kHeadDim)] : 0.f;
  __syncthreads();
  const float4* const q4 = reinterpret_cast<const float4*>(mbuf);
  float m[kMaxGroup], l[kMaxGroup], acc[kMaxGroup][4];
#pragma unroll
  for (int h = 0; h < kMaxGroup; ++h) {
    m[h] = kNoMax;
    l[h] = 0.f;
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[h][c] = 0.f;
  }
#pragma unroll 1
  for (int k = warp; k < items; k += W) {
    // ---- the lane's row: byte offset of its block, plus its place; -1: not attended
    const int u = unit + k * U + lane / 16, r16 = lane & 15;
    int pos = -1;
    if (u < S.nb0 + S.nb1) {
      const int at = (u < S.nb0 ? u : S.b1 + (u - S.nb0)) * kBlockTok + r16;
      if (at < S.L && (at < S.n_s || at >= S.w_lo)) pos = at;
    } else if ((u - S.nb0 - S.nb1) * 16 + r16 < S.cnt) {
      pos = __ldg(A.list + (long long)s * A.list_stride + (u - S.nb0 - S.nb1) * 16 + r16);
      if (pos >= S.L) pos = -1;
    }
    long long row = -1;
    if (pos >= 0) {
      const unsigned blk = (unsigned)pos / kBlockTok, pg = blk / (unsigned)A.pool.page_blocks;
      const int id = __ldg(A.pool.table + (size_t)b * A.pool.max_pages + pg);
      if ((unsigned)id < (unsigned)A.pool.n_pages)
        row = ((long long)id * A.pool.Hkv + g) * A.pool.head_bytes + (long long)(blk - pg * A.pool.page_blocks) * kBlockBytes4 +
              pos % kBlockTok;
    }
    // ---- its scores
    float p[kMaxGroup];
#pragma unroll
    for (int h = 0; h < kMaxGroup; ++h) p[h] = row >= 0 ? 0.f : -INFINITY;
    if (row >= 0) {
      const int r = (int)(row & 15);
      const unsigned char* const blk = A.pool.pages + (row - r);
      const uint2 sc = __ldg(reinterpret_cast<const uint2*>(blk + 2 * kBlockTok * kRow4 + r * 16));
      const float ks[4] = {bf16_lo(sc.x), bf16_hi(sc.x), bf16_lo(sc.y), bf16_hi(sc.y)};
#pragma unroll 1
      for (int w4 = 0; w4 < 4; ++w4) {
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(blk + r * kRow4) + w4);
        const uint32_t code[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int gr = 0; gr < 4; ++gr) {
          float f[8];
          centred(code[gr], f);
#pragma unroll
          for (int h = 0; h < kMaxGroup; ++h) {
            const float4 x = q4[32 * h + 8 * w4 + 2 * gr], y = q4[32 * h + 8 * w4 + 2 * gr + 1];
            float d = x.x * f[0];
            d = fmaf(x.y, f[1], d);
            d = fmaf(x.z, f[2], d);
            d = fmaf(x.w, f[3], d);
            d = fmaf(y.x, f[4], d);
            d = fmaf(y.y, f[5], d);
            d = fmaf(y.z, f[6], d);
            d = fmaf(y.w, f[7], d);
            p[h] = fmaf(ks[gr], d, p[h]);
          }
        }
      }
    }
    // ---- probabilities
#pragma unroll
    for (int h = 0; h < kMaxGroup; ++h) {
      float mx = p[h];
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
      const float mn = fmaxf(m[h], mx), alpha = exp2f(m[h] - mn);
      m[h] = mn;
      p[h] = exp2f(p[h] - mn);
      l[h] = fmaf(l[h], alpha, p[h]);
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[h][c] *= alpha;
    }
    // ---- sums of dims 4 lane .. 4 lane + 3, of value scale group lane % 4; 8 rows' loads under way together
    constexpr int kRows = 8;
#pragma unroll 1
    for (int j0 = 0; j0 < 32; j0 += kRows) {
      unsigned w[kRows];
      float y[kRows];
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        const long long at = __shfl_sync(kFull, row, j0 + j);
        const int r = at < 0 ? 0 : (int)(at & 15);
        const unsigned char* const blk = A.pool.pages + (at < 0 ? 0 : at - r);
        w[j] = __ldg(reinterpret_cast<const unsigned short*>(blk + kBlockTok * kRow4 + r * kRow4) + lane);
        const unsigned vs = __ldg(reinterpret_cast<const unsigned short*>(blk + 2 * kBlockTok * kRow4 + r * 16 + 8) + (lane & 3));
        y[j] = at < 0 ? 0.f : __uint_as_float(vs << 16);
      }
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        float v[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = y[j] * (__uint_as_float(0x4b000000u | (w[j] >> (4 * c) & 15u)) - 8388616.f);
#pragma unroll
        for (int h = 0; h < kMaxGroup; ++h) {
          const float x = __shfl_sync(kFull, p[h], j0 + j);
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[h][c] = fmaf(x, v[c], acc[h][c]);
        }
      }
    }
  }
  // ---- the upper half of the warps first, the lower adds its own: dim d = 32 t + 16 e + n of head h at [n / 2][4 h + t][2 (n % 2) + e]
  constexpr int kBoxes = (W + 1) / 2;
  float* const box = mbuf + (size_t)(warp % kBoxes) * kMergeWords;
#pragma unroll 1
  for (int half = 1; half >= 0; --half) {
    __syncthreads();
    if (warp / kBoxes == half) {
      const bool other = half == 0 && warp + kBoxes < W;
#pragma unroll
      for (int h = 0; h < kMaxGroup; ++h) {
        float ls = l[h];
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) ls += __shfl_xor_sync(kFull, ls, o);
        float* const ml = box + 1024 + 16 * h;
        const float m2 = other ? ml[0] : kNoMax, l2 = other ? ml[1] : 0.f;
        const float mn = fmaxf(m[h], m2), sa = exp2f(m[h] - mn), sb = exp2f(m2 - mn);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int d = 4 * lane + c, n = d & 15;
          float* const x = box + 4 * (32 * (n >> 1) + 4 * h + (d >> 5)) + 2 * (n & 1) + (d >> 4 & 1);
          *x = acc[h][c] * sa + (other ? *x * sb : 0.f);
        }
        __syncwarp();
        if (lane < 4) {
          ml[4 * lane] = mn;
          ml[4 * lane + 1] = ls * sa + l2 * sb;
        }
      }
    }
  }
  __syncthreads();
}

// The CTAs that share a slice whose items are [lo, hi).  split: see s_split.
__device__ __forceinline__ void owners(const int4& split, int nb, long long T, long long lo, long long hi, int& c0, int& c1) {
  const bool aligned = split.z >= 0;
  c0 = aligned ? split.y : (int)(((lo + 1) * nb - 1) / T);
  c1 = aligned ? split.y + split.z - 1 : (int)((hi * nb - 1) / T);
}
// The pieces marked in redo, once more in float32.  Finds everything out again from shared memory: handed over, the
// CTA's share alone cost 1M rows 18 us.
template <int W, int U, int S>
__device__ __noinline__ void redo_wide(const PagedAttendArgs& A, const RopeTab128& tab, const unsigned* redo, const int4* s_split, int* s_merge) {
  extern __shared__ __align__(128) unsigned char smem[];
  float* const mbuf = reinterpret_cast<float*>(smem + (size_t)W * S * U * kBlockBytes4);
  float* const qs = mbuf + (W + 1) / 2 * kMergeWords;
  const long long* const rpre = reinterpret_cast<const long long*>(qs + kMaxGroup * kQRow);
  const int2* const sinfo = reinterpret_cast<const int2*>(rpre + A.n_slices + 1);
  const int NS = A.n_slices;
  bool big = NS > (int)gridDim.x;
  for (int s = threadIdx.x; s < NS; s += W * 32) big = big || rpre[s + 1] - rpre[s] > 2 * W;
  const bool small = !__syncthreads_or(big);
  const int4 split = small ? make_int4(blockIdx.x, blockIdx.x, 1, 0) : *s_split;
  const long long T = rpre[NS];
  const int nb = (long long)gridDim.x < T ? (int)gridDim.x : (int)T;
  for (int s = 0; s < NS; ++s) {
    if (!(redo[s >> 5] >> (s & 31) & 1u)) continue;
    __syncthreads();
    turn_queries(A, tab, load_queries(A, tab, s), qs, sinfo[s].x);
    __syncthreads();
    long long lo = rpre[s], hi = rpre[s + 1];
    if (split.z >= 0) {
      const long long n = hi - lo;
      hi = lo + (blockIdx.x - split.y + 1) * n / split.z;
      lo = lo + (blockIdx.x - split.y) * n / split.z;
    } else {
      lo = max(lo, (long long)blockIdx.x * T / nb);
      hi = min(hi, (long long)(blockIdx.x + 1) * T / nb);
    }
    attend_wide<W, U>(A, make_slice(A, s % A.pool.Hkv, sinfo[s].x, sinfo[s].y), qs, mbuf, s, (int)(lo - rpre[s]) * U, (int)(hi - lo));
    int c0, c1;
    owners(split, nb, T, rpre[s], rpre[s + 1], c0, c1);
    finish<W, true>(A, mbuf, s_merge, s, c0, c1);
  }
}

// W warps, items of U units (4 bits 2, bf16 1), S ring slots a warp; WIDE: more than 4 heads a group (bf16 only, see the matrix mapping); LISTED: a
// selection is given.
template <int FMT, int W, int U, int S, bool WIDE, bool LISTED>
__global__ void __launch_bounds__(W * 32, 1) k_attend_paged(const __grid_constant__ PagedAttendArgs A, const __grid_constant__ RopeTab128 tab) {
  constexpr bool kF16 = FMT == kPageInt4;
  constexpr int kBlk = FMT == kPageInt4 ? kBlockBytes4 : kBlockBytes16;
  constexpr int kItems = 32 / U;   // items that 32 lanes look up
  static_assert(U == (kF16 ? 2 : 1), "items of each format");
  extern __shared__ __align__(128) unsigned char smem[];
  unsigned char* const ring = smem;                                              // [W][S][U][kBlk]
  float* const mbuf = reinterpret_cast<float*>(smem + (size_t)W * S * U * kBlk);     // [(W + 1) / 2][kMergeWords]
  float* const qs = mbuf + (W + 1) / 2 * kMergeWords;                            // [8][kQRow]
  long long* const rpre = reinterpret_cast<long long*>(qs + kMaxGroup * kQRow);  // [n_slices + 1]
  int2* const sinfo = reinterpret_cast<int2*>(rpre + A.n_slices + 1);            // [n_slices] (L, listed rows)
  __shared__ __align__(8) unsigned long long full[W * S];
  __shared__ unsigned vmask[W * S * U];   // attended rows of a slot's units; bit 16: gathered
  __shared__ long long shl[W];
  __shared__ int s_merge;
  __shared__ int s_late;                       // a wait has run out
  __shared__ float qun[kMaxGroup];             // 4 bits: what a head's scores are multiplied by
  __shared__ int4 s_split;                     // aligned shares: slice, its first CTA, its CTAs, -1: equal shares
  __shared__ uint4 qf[kF16 ? 8 * 32 : 1];      // 4 bits: query operands, a lane's 16 bytes of each k-step
  __shared__ float2 q8[kF16 ? 4 * 8 : 1];      // 4 bits: -8 times a scale group's sum of queries (high, residual), each head
  __shared__ __align__(16) float kscale[kF16 ? 4 * W * 32 : 4];   // 4 bits, of the item in hand: scales of K, by group and row
  __shared__ int s_wide, any_redo;             // 4 bits: the piece in hand has to be taken again; some piece has
  __shared__ unsigned redo[kF16 ? kMaxPagedSlices / 32 : 1];   // 4 bits: a bit for each slice of such a piece
  __shared__ uint4 vscale[kF16 ? W * 16 : 1];  // and of V in float16, (row, row + 1) pairs of each group

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gid = lane >> 2, t4 = lane & 3;
  const int NS = A.n_slices, Hkv = A.pool.Hkv, G = A.G;

  if (tid < W * S) mbar_init(smem_u32(&full[tid]), U);
  if (tid == 0) s_late = 0;
  if (kF16) {   // heads that the group does not have
    if (tid < 256) qf[kF16 ? tid : 0] = make_uint4(0u, 0u, 0u, 0u);
    if (tid < 32) q8[kF16 ? tid : 0] = make_float2(0.f, 0.f);
    if (tid < kMaxPagedSlices / 32) redo[kF16 ? tid : 0] = 0u;
    if (tid == 0) s_wide = any_redo = 0;
  }
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");

  // ---- item prefix over slices
  bool small;   // no slice has more than two items a warp
  {
    long long carry = 0;
    bool big = false;
    for (int base = 0; base < NS; base += W * 32) {
      const int s = base + tid;
      int n = 0;
      if (s < NS) {
        const int b = Hkv == 1 ? s : (int)__umulhi((unsigned)s, A.by_heads), g = s - b * Hkv;
        int64_t L = A.seq_lens[b];
        if (L < 0 || L > A.cap) {
          atomicOr(A.pool.err, kErrSeqLen);
          L = L < 0 ? 0 : A.cap;
        }
        int cnt = 0;
        if (A.has_list[g]) {
          cnt = A.list_count[s];
          if (cnt < 0 || cnt > A.list_stride) {
            atomicOr(A.pool.err, kErrList);
            cnt = 0;
          }
        }
        sinfo[s] = make_int2((int)L, cnt);
        n = (units_of(make_slice(A, g, (int)L, cnt)) + U - 1) / U;
        big = big || n > 2 * W;
      }
      int v = n;   // 32 slices of 2^21 units at most
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, v, o);
        if (lane >= o) v += y;
      }
      if (lane == 31) shl[warp] = v;
      __syncthreads();
      long long before = carry, total = 0;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const long long x = shl[w];
        if (w < warp) before += x;
        total += x;
      }
      if (s < NS) rpre[s] = before + v - n;
      carry += total;
      __syncthreads();
    }
    if (tid == 0) rpre[NS] = carry;
    small = !__syncthreads_or(big) && NS <= (int)gridDim.x;
  }
  const long long T = rpre[NS];
  // slices without a row: zeros
  for (int s = blockIdx.x; s < NS; s += gridDim.x) {
    if (rpre[s + 1] != rpre[s]) continue;
    const size_t h0 = (size_t)(s / Hkv) * A.Hq + (size_t)(s % Hkv) * G;
    for (int i = tid; i < G * kHeadDim; i += W * 32) A.out[h0 * kHeadDim + i] = 0.f;
    if (A.lse && tid < G) A.lse[h0 + tid] = -INFINITY;
  }
  // ---- shares: a CTA a slice where the slices are small and few; else aligned to slices or equal.
  // Aligned: a slice of n items takes ceil(n / most) CTAs, with `most` the least (but an item a warp) for which the CTAs suffice.
  // A CTA then has one slice's queries and merge, at the price of a largest share above the equal one.  Taken where that
  // price is no more than the slices that an equal share passes through: kPieceItems for a second, as much again where some
  // slice is shorter than a share (a CTA then meets three).  Over bf16 pages, where memory bounds the call and
  // a few idle CTAs cost little, kUneven of a share is accepted too.
  // Equal: down to one item a CTA.
  // us, equal against aligned: one sequence of 4096 rows 19.4 / 14.1, 16 of them 37.4 / 32.7, 4 x 128K with lists 55.2 / 51.6,
  // 3 x 128K with half of the heads streaming 80.7 / 75.8; but 1M rows of 8 heads 344 / 348, and 16 x 64K of bf16, a
  // quarter of the heads seeing every row, 134 / 429.
  // us, bf16 of 64K with kUneven at 0, 0.3, 0.6: 5 sequences, a quarter of the heads seeing every row, 64.7 / 60.4 / 60.4;
  // 7 of them - / 82.5 / 76.4; 8 - / 86.6 / 84.8; 10, half of the heads, - / 171.4 / 179.
  constexpr int kLaneSlices = 5, kPieceItems = 24;
  constexpr float kUneven = 0.3f;
  if (!small) {
    if (NS > 32 * kLaneSlices || NS > (int)gridDim.x) {
      if (tid == 0) s_split = make_int4(0, 0, -1, 0);
    } else if (warp == 0) {
      float n[kLaneSlices];
      float top = 0.f, low = FLT_MAX;
#pragma unroll
      for (int i = 0; i < kLaneSlices; ++i) {
        const int s = lane * kLaneSlices + i;
        // listed items weigh more: their gathering is worth 0.3 of an item (4 x 128K with lists: 55.0 us without, 51.6 with)
        n[i] = s < NS ? (float)(rpre[s + 1] - rpre[s]) : 0.f;
        if (LISTED && s < NS) n[i] += 0.3f / (16 * U) * sinfo[s].y;
        top = fmaxf(top, n[i]);
        if (n[i] > 0.f) low = fminf(low, n[i]);
      }
      top = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(top)));
      low = __uint_as_float(__reduce_min_sync(kFull, __float_as_uint(low)));
      float all = 0.f;
#pragma unroll
      for (int i = 0; i < kLaneSlices; ++i) all += n[i];
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) all += __shfl_xor_sync(kFull, all, o);
      const float equal = __fdividef(all, (float)gridDim.x);
      float most = fmaxf(equal, (float)W);
      int k[kLaneSlices], sum = 0;
#pragma unroll 1
      for (int t = 0; t < 9; ++t) {
        const float inv = __fdividef(0.999999f, most);
        int mine = 0;
#pragma unroll
        for (int i = 0; i < kLaneSlices; ++i) {
          k[i] = (int)ceilf(n[i] * inv);
          mine += k[i];
        }
        sum = __reduce_add_sync(kFull, mine);
        if (sum <= (int)gridDim.x) break;
        most = t == 7 ? top * 1.0001f : fminf(fmaxf(most * __fdividef((float)sum, (float)gridDim.x), most * 1.01f), top * 1.0001f);
      }
      float share = 0.f;
      int mine = 0;
#pragma unroll
      for (int i = 0; i < kLaneSlices; ++i) {
        if (k[i] > 0) share = fmaxf(share, __fdividef(n[i], (float)k[i]));
        mine += k[i];
      }
      share = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(share)));
      int before = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, before, o);
        if (lane >= o) before += y;
      }
      before -= mine;
      const float more = low < equal ? 2.f * kPieceItems : (float)kPieceItems;
      const bool fits = sum <= (int)gridDim.x && share <= equal + (kF16 ? more : fmaxf(more, kUneven * equal));
      if (lane == 0) s_split = make_int4(0, 0, fits ? 0 : -1, 0);
      __syncwarp();
      if (fits) {
#pragma unroll
        for (int i = 0; i < kLaneSlices; ++i) {
          if ((int)blockIdx.x >= before && (int)blockIdx.x < before + k[i]) s_split = make_int4(lane * kLaneSlices + i, before, k[i], 0);
          before += k[i];
        }
      }
    }
    __syncthreads();
  }
  const int4 split = small ? make_int4(blockIdx.x, blockIdx.x, (int)blockIdx.x < NS ? 1 : 0, 0) : s_split;
  const bool aligned = split.z >= 0;
  const int nb = (long long)gridDim.x < T ? (int)gridDim.x : (int)T;
  long long r_lo, r_hi;
  if (aligned) {
    if (split.z == 0) return;
    const long long n = rpre[split.x + 1] - rpre[split.x];
    r_lo = rpre[split.x] + (blockIdx.x - split.y) * n / split.z;
    r_hi = rpre[split.x] + (blockIdx.x - split.y + 1) * n / split.z;
    if (r_lo == r_hi) return;
  } else {
    if ((int)blockIdx.x >= nb) return;
    r_lo = (long long)blockIdx.x * T / nb;
    r_hi = (long long)(blockIdx.x + 1) * T / nb;
  }
  auto slice_of = [&](long long r) {
    int lo = 0, hi = NS - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (rpre[mid] <= r) lo = mid;
      else hi = mid - 1;
    }
    return lo;
  };
  const int s_first = aligned ? split.x : slice_of(r_lo), s_last = aligned ? split.x : slice_of(r_hi - 1);

  auto load_q = [&](int s) { return load_queries(A, tab, s); };
  float4 q_next = load_q(s_first);
  const uint32_t ring_a = smem_u32(ring) + warp * S * U * kBlk, bar_a = smem_u32(&full[warp * S]);
  const uint64_t pol = l2_evict_first();

  // ---- the warp's items r_lo + warp + W k, k < nk: lane i looks up unit i % U of item kItems j + i / U
  const int nk = r_lo + warp < r_hi ? (int)((r_hi - r_lo - warp + W - 1) / W) : 0;
  auto page_of = [&](unsigned blk) { return A.pool.page_blocks == 1 ? blk : __umulhi(blk, A.by_blocks); };
  auto find = [&](int k) {
    Unit X;
    X.s = X.bg = 0;
    X.off = 0;
    X.info = 0u;
    k += lane / U;
    if (k >= nk) return X;
    const long long r = r_lo + warp + (long long)W * k;
    const int s = slice_of(r);
    const int b = Hkv == 1 ? s : (int)__umulhi((unsigned)s, A.by_heads), g = s - b * Hkv;
    const Slice sl = make_slice(A, g, sinfo[s].x, sinfo[s].y);
    const int u = (int)(r - rpre[s]) * U + lane % U;
    X.s = s;
    X.bg = b << 8 | g;
    if (u >= units_of(sl)) return X;
    if (LISTED && u >= sl.nb0 + sl.nb1) {
      const int i = (u - sl.nb0 - sl.nb1) * 16;
      X.off = (long long)s * A.list_stride + i;
      X.info = kList | (0xffffu >> (16 - min(16, sl.cnt - i)));
      return X;
    }
    const int blk = u < sl.nb0 ? u : sl.b1 + (u - sl.nb0);
    const int p0 = blk * kBlockTok;
    // rows [0, L), below n_s or at least w_lo
    auto below = [&](int q) { return q <= p0 ? 0u : 0xffffu >> (16 - min(16, q - p0)); };
    const unsigned rows = below(sl.L) & (below(sl.n_s) | ~below(sl.w_lo));
    const unsigned pg = page_of((unsigned)blk), in = (unsigned)blk - pg * (unsigned)A.pool.page_blocks;
    const int id = __ldg(A.pool.table + (size_t)b * A.pool.max_pages + pg);
    if ((unsigned)id < (unsigned)A.pool.n_pages) {
      X.off = ((long long)id * Hkv + g) * A.pool.head_bytes + (long long)in * kBlk;
      X.info = rows;
    } else {
      atomicOr(A.pool.err, kErrPage);
    }
    return X;
  };
  // `cur` holds the item to be issued; `nxt`, where it differs, the item two or three ahead of it (lists)
  Unit cur = find(0), nxt = cur;
  int ki = 0;   // the next item to issue
  auto list_rows = [&](int k) {   // starts the loads of item k's positions
    Rows R;
    R.pos = R.id = -1;
    R.s = R.bg = 0;
    if (k >= nk) return R;
    const Unit& B = k / kItems == ki / kItems ? cur : nxt;
    const int from = k % kItems * U + (U == 2 ? lane >> 4 : 0);
    const unsigned info = __shfl_sync(kFull, B.info, from);
    if (!__any_sync(kFull, info & kList)) return R;
    const long long off = __shfl_sync(kFull, B.off, from);
    R.s = __shfl_sync(kFull, B.s, from);
    R.bg = __shfl_sync(kFull, B.bg, from);
    if (lane < 16 * U && (info & kList) && (info >> (lane & 15) & 1u)) {
      R.pos = __ldg(A.list + off + (lane & 15));
      if (R.pos < 0) R.pos = INT_MAX;   // refused with the positions past the end
    }
    return R;
  };
  auto list_pages = [&](Rows& R) {   // checks the positions, starts the loads of their pages
    if (R.pos < 0) return;
    if (R.pos >= sinfo[R.s].x) {
      atomicOr(A.pool.err, kErrList);
      R.pos = -1;
      return;
    }
    R.id = __ldg(A.pool.table + (size_t)(R.bg >> 8) * A.pool.max_pages + page_of((unsigned)R.pos / kBlockTok));
  };
  Rows r0, r1, r2;   // of items ki, ki + 1 (their pages loaded, too) and ki + 2
  if (LISTED) {
    r0 = list_rows(0);
    r1 = list_rows(1);
    r2 = list_rows(2);
    list_pages(r0);
    list_pages(r1);
  }
  int islot = 0;           // ring slot of item ki
  unsigned was_list = 0u;  // slots last written by gathers
  // Every unit arrives once at its slot's barrier: with its copy, or plainly.
  auto issue = [&]() {
    if (ki < nk) {
      const uint32_t dst = ring_a + islot * U * kBlk, bar = bar_a + 8 * islot;
      const bool mine = lane / U == ki % kItems;
      const bool gather = LISTED && mine && (cur.info & kList);
      if (mine && !gather) {
        vmask[(warp * S + islot) * U + lane % U] = cur.info;
        if (cur.info) {
          if (LISTED && (was_list >> islot & 1u)) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          bulk_load(dst + lane % U * kBlk, A.pool.pages + cur.off, kBlk, bar, pol);
        } else {
          mbar_arrive(bar, 1);
        }
      }
      if (LISTED) was_list &= ~(1u << islot);
      if (LISTED && __any_sync(kFull, gather)) {
        was_list |= 1u << islot;
        const bool page_ok = (unsigned)r0.id < (unsigned)A.pool.n_pages;
        if (r0.pos >= 0 && !page_ok) atomicOr(A.pool.err, kErrPage);
        const unsigned m = __ballot_sync(kFull, r0.pos >= 0 && page_ok);
        // row of the pool, in rows of a head: memory holds fewer than 2^32
        const unsigned blkno = (unsigned)r0.pos / kBlockTok, in = blkno - page_of(blkno) * (unsigned)A.pool.page_blocks;
        const unsigned from = (((unsigned)r0.id * Hkv + (r0.bg & 255)) * A.pool.page_blocks + in) * kBlockTok + (r0.pos & (kBlockTok - 1));
        if (FMT == kPageInt4) {
#pragma unroll
          for (int i = 0; i < 2 * U; ++i) {
            const int r = i * 8 + gid;   // row of the item
            const unsigned a = __shfl_sync(kFull, from, r);
            if (m >> r & 1u) {
              const unsigned char* src = A.pool.pages + (size_t)(a / kBlockTok) * kBlk + (a % kBlockTok) * kRow4 + t4 * 16;
              const uint32_t d = dst + i / 2 * kBlk + (r & 15) * kRow4 + t4 * 16;
              cp_async16(d, src);
              cp_async16(d + kBlockTok * kRow4, src + kBlockTok * kRow4);
            }
          }
          if (m >> lane & 1u) {
            cp_async16(dst + lane / 16 * kBlk + 2 * kBlockTok * kRow4 + (lane & 15) * 16,
                       A.pool.pages + (size_t)(from / kBlockTok) * kBlk + 2 * kBlockTok * kRow4 + (from % kBlockTok) * 16);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = i * 2 + (lane >> 4), c = lane & 15;
            const unsigned a = __shfl_sync(kFull, from, r), rin = a % kBlockTok;
            if (m >> r & 1u) {
              const unsigned char* src = A.pool.pages + (size_t)(a / kBlockTok) * kBlk + rin * 256 + ((c ^ (rin & 7)) << 4);
              const uint32_t d = dst + r * 256 + ((c ^ (r & 7)) << 4);
              cp_async16(d, src);
              cp_async16(d + kBlockTok * 256, src + kBlockTok * 256);
            }
          }
        }
        if (gather) {
          vmask[(warp * S + islot) * U + lane % U] = (m >> lane % U * 16 & 0xffffu) | kList;
          mbar_arrive(bar, 1);
        }
      }
      islot = islot + 1 == S ? 0 : islot + 1;
    }
    if (LISTED) asm volatile("cp.async.commit_group;\n" ::: "memory");
    ++ki;
    if (LISTED) {   // the items behind: found three early, for the lists' pipeline
      if ((ki + 3) % kItems == 0) nxt = find(ki + 3);
      if (ki % kItems == 0) cur = nxt;
      r0 = r1;
      r1 = r2;
      list_pages(r1);
      r2 = list_rows(ki + 2);
    } else if (ki % kItems == 0) {
      cur = find(ki);
    }
  };
#pragma unroll 1
  for (int i = 0; i < S - 1; ++i) issue();

  const uint32_t qf_a = smem_u32(qf) + lane * 16;
  int slot = 0;         // ring slot to consume
  unsigned phase = 0u;  // of its barrier
  int i = warp;         // its item, from r_lo

  for (int s = s_first; s <= s_last; ++s) {
    if (rpre[s + 1] == rpre[s]) continue;
    const int i_end = (int)(min(r_hi, rpre[s + 1]) - r_lo);
    // ---- the group's queries, rotated at position L - 1, times scale / ln 2
    turn_queries(A, tab, q_next, qs, sinfo[s].x);
    if (warp < G) {
      float* const q = qs + warp * kQRow;
      if (kF16) {
        __syncwarp();
        // dim lane + 32 t of scale group lane / 8: k-step 2 (lane / 8) + i holds dims 32 t + 8 (lane / 8) + 2 i + {0, 4, 1, 5}
        float x[4], top = 0.f;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          x[t] = q[q_at(lane + 32 * t)];
          top = fmaxf(top, fabsf(x[t]));
        }
        float part = top;   // of the scale group
#pragma unroll
        for (int o = 1; o <= 4; o <<= 1) part = fmaxf(part, __shfl_xor_sync(kFull, part, o));
        top = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(top)));
        const int e = min(max((int)(__float_as_uint(top) >> 23) - 127, -112), 112);
        if (part > 0.f && part < top * 0x1p-13f) s_wide = 1;
        const bool odd = lane & 1;   // the operand's second half, whose codes count 16 times
        const float f = __uint_as_float((unsigned)(127 + 14 - e) << 23) * (odd ? 0.0625f : 1.f);
        if (lane == 0) qun[warp] = __uint_as_float((unsigned)(127 - 14 + e) << 23) * kKeyUnit;
        const int kk = 2 * (lane >> 3) + ((lane & 3) >> 1);
        float sh = 0.f, sl = 0.f;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const __half hi = __float2half_rn(x[t] * f), lo = __float2half_rn(x[t] * f - __half2float(hi));
          __half* const to = reinterpret_cast<__half*>(qf + 32 * kk + 4 * warp + t) + (odd ? 4 : 0) + ((lane >> 2) & 1);
          to[0] = hi;
          to[2] = lo;
          sh += __half2float(hi);
          sl += __half2float(lo);
        }
        if (odd) {
          sh *= 16.f;
          sl *= 16.f;
        }
#pragma unroll
        for (int o = 1; o <= 4; o <<= 1) {
          sh += __shfl_xor_sync(kFull, sh, o);
          sl += __shfl_xor_sync(kFull, sl, o);
        }
        if ((lane & 7) == 0) q8[8 * (lane >> 3) + warp] = make_float2(sh * (-8.f / kKeyUnit), sl * (-8.f / kKeyUnit));
      }
    }
    __syncthreads();
    // A operand: 4 bits in shared memory, bf16 in registers and in natural order
    uint32_t qa[kF16 ? 1 : 8][4];
    uint32_t qb[WIDE ? 8 : 1][2];   // the low part's rows where they need a product of their own
    const float unscale = kF16 ? qun[gid < G ? gid : 0] : 1.f;
    if (!kF16) {
      const int h = WIDE ? gid : gid & 3;
      const bool in = h < G;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        const float* x = qs + (in ? h : 0) * kQRow + q_at(16 * kk) + 2 * t4;
        uint32_t hi[2], mid[2], lo[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) split_bf16(in ? x[8 * i] : 0.f, in ? x[8 * i + 1] : 0.f, hi[i], mid[i], lo[i]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          qa[kF16 ? 0 : kk][2 * i] = WIDE || gid < 4 ? hi[i] : mid[i];
          qa[kF16 ? 0 : kk][2 * i + 1] = WIDE ? mid[i] : gid < 4 ? lo[i] : 0u;
          if (WIDE) qb[WIDE ? kk : 0][i] = lo[i];
        }
      }
    }
    float m = kNoMax, l = 0.f;
    // 4 bits: bound of the value scales met, a power of two in bf16 bits, with the number of binades below it that they reach (zeros
    // aside) in its low bits; and the inverse of the bound.  (A variable of its own for the binades cost 1M rows 10 us.)
    unsigned vlim = 0u;
    float vmul = __uint_as_float((254u << 23) - (kScaleLow << 16));
    // Sums over the rows, of column tile nt.  An item's products are summed apart and added by rounded additions: the
    // tensor cores truncate what they add to, and over the hundreds of items of a long context that
    // pulls sums towards zero (4e-6 at 1M rows).  High and residual rows meet here, so it is half the registers.
    float acc[16][2];
#pragma unroll
    for (int nt = 0; nt < 16; ++nt) acc[nt][0] = acc[nt][1] = 0.f;

#pragma unroll 1
    for (; i < i_end; i += W) {
      __syncwarp();
      issue();   // refills the slot consumed last time
      const unsigned char* const st = ring + (warp * S + slot) * U * kBlk;
      if (!mbar_wait(bar_a + 8 * slot, phase, &s_late) && lane == 0) atomicOr(A.pool.err, kErrTimeout);
      unsigned vm[U], any = 0u, all = 0xffffu;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        vm[u] = vmask[(warp * S + slot) * U + u];
        any |= vm[u];
        all &= vm[u];
      }
      if (++slot == S) {
        slot = 0;
        phase ^= 1u;
      }
      if (LISTED && (any & kList)) {
        asm volatile("cp.async.wait_group %0;\n" ::"n"(S - 1) : "memory");
        __syncwarp();
      }
      if (!(any & 0xffffu)) continue;
      const bool part = (all & 0xffffu) != 0xffffu;
      // ---- 4 bits: lane l widens the scales of row l of the item, those of V times vmul to float16
      if (kF16) {
        uint4 w = *reinterpret_cast<const uint4*>(st + lane / 16 * kBlk + 2 * kBlockTok * kRow4 + (lane & 15) * 16);
        if (part && !((lane < 16 ? vm[0] : vm[U - 1]) >> (lane & 15) & 1u)) w = make_uint4(0u, 0u, 0u, 0u);
        // any of the four outside (vlim - kScaleNear, vlim] (a borrow comes from one outside)
        if (__any_sync(kFull, max_u16x2(vlim * 0x10001u - w.z, vlim * 0x10001u - w.w) & (0x10000u - kScaleNear) * 0x10001u)) {
          auto finite = [](uint32_t x) { return x < 0x7f80u ? x : 0u; };           // NaN: the finite ones decide,
          auto some = [](uint32_t x) { return x - 1u < 0x7f7fu ? x : 0x7f80u; };   // and those that are not 0
          unsigned vtop = max(max(finite(w.z & 0xffffu), finite(w.z >> 16)), max(finite(w.w & 0xffffu), finite(w.w >> 16)));
          unsigned vmin = min(min(some(w.z & 0xffffu), some(w.z >> 16)), min(some(w.w & 0xffffu), some(w.w >> 16)));
          vtop = __reduce_max_sync(kFull, vtop);
          vmin = __reduce_min_sync(kFull, vmin) & 0x7f80u;
          unsigned lim = vlim & 0x7f80u, low = vlim ? min(vmin, lim - (vlim & 0x7fu) * 0x80u) : vmin;
          if (vtop > lim) {   // the power of two at or above it
            lim = min(max((vtop + 0x7fu) & 0x7f80u, kScaleLow), kScaleHigh);
            const float now = __uint_as_float((254u << 23) - (lim << 16)), by = now / vmul;
            vmul = now;
#pragma unroll
            for (int nt = 0; nt < 16; ++nt) {
              acc[nt][0] *= by;
              acc[nt][1] *= by;
            }
            low = min(low, lim - kScaleNear);   // rows that are not looked at
          }
          const unsigned span = min(lim - min(low, lim), kScaleSpan + 0x80u) >> 7;
          if (span > kScaleSpan >> 7 || vtop > kScaleHigh) s_wide = 1;
          vlim = lim | span;
        }
        kscale[128 * warp + lane] = bf16_lo(w.x);
        kscale[128 * warp + 32 + lane] = bf16_hi(w.x);
        kscale[128 * warp + 64 + lane] = bf16_lo(w.y);
        kscale[128 * warp + 96 + lane] = bf16_hi(w.y);
        const uint32_t a01 = bits(__floats2half2_rn(bf16_lo(w.z) * vmul, bf16_hi(w.z) * vmul));
        const uint32_t a23 = bits(__floats2half2_rn(bf16_lo(w.w) * vmul, bf16_hi(w.w) * vmul));
        const uint32_t b01 = __shfl_down_sync(kFull, a01, 1), b23 = __shfl_down_sync(kFull, a23, 1);
        if (!(lane & 1))
          vscale[16 * warp + lane / 2] = make_uint4(__byte_perm(a01, b01, 0x5410), __byte_perm(a01, b01, 0x7632),
                                                    __byte_perm(a23, b23, 0x5410), __byte_perm(a23, b23, 0x7632));
        __syncwarp();
      }
      // ---- scores of head gid for rows 8 j + 2 t4 + e of unit u (4 bits: still to be multiplied by unscale)
      float p[U][2][2];
      if (kF16) {
        uint4 kw[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            kw[u][j] = *reinterpret_cast<const uint4*>(st + u * kBlk + (8 * j + gid) * kRow4 + t4 * 16);
#pragma unroll
        for (int g4 = 0; g4 < 4; ++g4) {
          const uint4 a0 = lds128(qf_a + 1024 * g4), a1 = lds128(qf_a + 1024 * g4 + 512);
          const uint32_t a0r[4] = {a0.x, a0.y, a0.z, a0.w}, a1r[4] = {a1.x, a1.y, a1.z, a1.w};
          const float2 centre = q8[8 * g4 + gid];
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t w = g4 == 0 ? kw[u][j].x : g4 == 1 ? kw[u][j].y : g4 == 2 ? kw[u][j].z : kw[u][j].w;
              uint32_t c[4];
              float d[4];
              code_pairs(w, c);
              mma16816_from<true>(d, a0r, c[0], c[1], centre);
              mma16816<true>(d, a1r, c[2], c[3]);
              const float2 k = *reinterpret_cast<const float2*>(kscale + 128 * warp + 32 * g4 + 16 * u + 8 * j + 2 * t4);
              p[u][j][0] = g4 == 0 ? k.x * (d[0] + d[2]) : fmaf(k.x, d[0] + d[2], p[u][j][0]);
              p[u][j][1] = g4 == 0 ? k.y * (d[1] + d[3]) : fmaf(k.y, d[1] + d[3], p[u][j][1]);
            }
        }
      } else {
        float d[2][2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) d[j][e][0] = d[j][e][1] = d[j][e][2] = d[j][e][3] = 0.f;
        const int mi = lane >> 3, rr = lane & 7;
        const uint32_t row = smem_u32(st) + (8 * (mi >> 1) + rr) * 256;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          uint32_t bk[4];
          ldsm_x4(bk, row + (((2 * kk + (mi & 1)) ^ rr) << 4));
          mma16816<false>(d[0][kk & 1], qa[kF16 ? 0 : kk], bk[0], bk[1]);
          mma16816<false>(d[1][kk & 1], qa[kF16 ? 0 : kk], bk[2], bk[3]);
          if (WIDE) {
            const uint32_t low[4] = {qb[WIDE ? kk : 0][0], 0u, qb[WIDE ? kk : 0][1], 0u};
            mma16816<false>(d[0][kk & 1], low, bk[0], bk[1]);
            mma16816<false>(d[1][kk & 1], low, bk[2], bk[3]);
          }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            p[0][j][e] = (d[j][0][e] + d[j][1][e]) + (d[j][0][2 + e] + d[j][1][2 + e]);
            if (!WIDE) p[0][j][e] += __shfl_xor_sync(kFull, p[0][j][e], 16);
          }
      }
      if (part) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (!(vm[u] >> (8 * j + 2 * t4 + e) & 1u)) p[u][j][e] = -INFINITY;
      }
      // ---- running maximum and sum; scores become probabilities
      float mx = -INFINITY;
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < 2; ++j) mx = fmaxf(mx, fmaxf(p[u][j][0], p[u][j][1]));
      mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
      // rounded up: where 14 is less than a step of the score, a rounding down would let the top probability past 2^14
      const float mn = fmaxf(m, __fmaf_ru(mx, unscale, kF16 ? -kProbExp : 0.f));
      if (__any_sync(kFull, mn != m)) {
        const float alpha = ex2(m - mn);
        l *= alpha;
        m = mn;
#pragma unroll
        for (int nt = 0; nt < 16; ++nt) {
          acc[nt][0] *= alpha;
          acc[nt][1] *= alpha;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            p[u][j][e] = ex2(fmaf(p[u][j][e], unscale, -m));
            l += p[u][j][e];
          }
      // ---- acc += P V
      if (kF16) {
        uint2 vw[U][2][2];
        __half2 ph[U][2], pl[U][2];
        uint4 sv[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const unsigned char* vb = st + u * kBlk + kBlockTok * kRow4 + gid * 8;
#pragma unroll
            for (int e = 0; e < 2; ++e) {   // a word here, the other as late as it may be (one load of both: 1M rows 357 us in place of 345)
              vw[u][j][e].x = *reinterpret_cast<const volatile uint32_t*>(vb + (8 * j + 2 * t4 + e) * kRow4);
              vw[u][j][e].y = *reinterpret_cast<const uint32_t*>(vb + (8 * j + 2 * t4 + e) * kRow4 + 4);
            }
            split_f16(p[u][j][0], p[u][j][1], ph[u][j], pl[u][j]);
            sv[u][j] = lds128(smem_u32(&vscale[16 * warp + 8 * u + 4 * j + t4]));   // in place: 1M rows 356 us otherwise
          }
#pragma unroll
        for (int g4 = 0; g4 < 4; ++g4) {
          float x[4][4];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            uint32_t pa[4], w[2], c0[4], c1[4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              // high part of the product; its exact rounding error and the low part make the residual
              const __half2 sg = half2_of(g4 == 0 ? sv[u][j].x : g4 == 1 ? sv[u][j].y : g4 == 2 ? sv[u][j].z : sv[u][j].w);
              const __half2 hi = __hmul2(ph[u][j], sg);
              pa[2 * j] = bits(hi);
              pa[2 * j + 1] = bits(__hfma2(pl[u][j], sg, __hfma2(ph[u][j], sg, __hneg2(hi))));
              w[j] = g4 < 2 ? __byte_perm(vw[u][j][0].x, vw[u][j][1].x, (g4 & 1) ? 0x7632 : 0x5410)
                            : __byte_perm(vw[u][j][0].y, vw[u][j][1].y, (g4 & 1) ? 0x7632 : 0x5410);
            }
            centred_pairs(w[0], c0);
            centred_pairs(w[1], c1);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              if (u == 0) mma16816_from<true>(x[t], pa, c0[t], c1[t], make_float2(0.f, 0.f));
              else mma16816<true>(x[t], pa, c0[t], c1[t]);
            }
          }
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            acc[4 * g4 + t][0] += x[t][0] + x[t][2];
            acc[4 * g4 + t][1] += x[t][1] + x[t][3];
          }
        }
      } else {
        uint32_t pa[4], pb[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t hi, mid, lo;
          split_bf16(p[0][j][0], p[0][j][1], hi, mid, lo);
          pa[2 * j] = WIDE || gid < 4 ? hi : mid;
          pa[2 * j + 1] = WIDE ? mid : gid < 4 ? lo : 0u;
          pb[2 * j] = lo;
          pb[2 * j + 1] = 0u;
        }
        const int mi = lane >> 3, rr = lane & 7;
        const uint32_t row = smem_u32(st) + kBlockTok * 256 + (8 * (mi & 1) + rr) * 256;
        // rows 2 t4 + {0, 1} and + 8 as bit masks of the operand's halves
        uint32_t live0 = kFull, live1 = kFull;
        if (part) {
          const unsigned v0 = vm[0] >> (2 * t4), v1 = vm[0] >> (8 + 2 * t4);
          live0 = ((v0 & 1u) ? 0xffffu : 0u) | ((v0 & 2u) ? 0xffff0000u : 0u);
          live1 = ((v1 & 1u) ? 0xffffu : 0u) | ((v1 & 2u) ? 0xffff0000u : 0u);
        }
#pragma unroll
        for (int nt = 0; nt < 16; nt += 2) {
          uint32_t bv[4];
          ldsm_x4_t(bv, row + (((nt + (mi >> 1)) ^ rr) << 4));
          if (part) {
            bv[0] &= live0;
            bv[1] &= live1;
            bv[2] &= live0;
            bv[3] &= live1;
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float x[4];
            mma16816_from<false>(x, pa, bv[2 * i], bv[2 * i + 1], make_float2(0.f, 0.f));
            if (WIDE) mma16816<false>(x, pb, bv[2 * i], bv[2 * i + 1]);
            acc[nt + i][0] += x[0] + x[2];
            acc[nt + i][1] += x[1] + x[3];
          }
        }
      }
    }

    // ---- warp state: a head's sum over its 4 lanes, high and residual rows together
    l += __shfl_xor_sync(kFull, l, 1);
    l += __shfl_xor_sync(kFull, l, 2);
    float o[16][2];
#pragma unroll
    for (int nt = 0; nt < 16; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        o[nt][e] = acc[nt][e];
        if (kF16) o[nt][e] *= kValueUnit / vmul;
        else if (!WIDE) o[nt][e] += __shfl_xor_sync(kFull, o[nt][e], 16);
      }
    }
    // ---- the warps' states as their lanes hold them: the upper half of the warps hands over to the lower, then thread x
    // takes 4 of the 32 sums of one lane over what is left
    constexpr int kBoxes = (W + 1) / 2;
    float4* const box = reinterpret_cast<float4*>(mbuf + (size_t)(warp % kBoxes) * kMergeWords) + lane;
    auto hand_over = [&]() {
#pragma unroll
      for (int k = 0; k < 8; ++k) box[32 * k] = make_float4(o[2 * k][0], o[2 * k][1], o[2 * k + 1][0], o[2 * k + 1][1]);
      box[256] = make_float4(m, l, 0.f, 0.f);
    };
    if (warp >= kBoxes) hand_over();
    int s_after = s + 1;
    while (s_after <= s_last && rpre[s_after + 1] == rpre[s_after]) ++s_after;
    if (s_after <= s_last) q_next = load_q(s_after);
    __syncthreads();
    if (warp < kBoxes) {
      if (warp + kBoxes < W) {
        const float4 ml = box[256];
        const float mn = fmaxf(m, ml.x), sa = exp2f(m - mn), sb = exp2f(ml.x - mn);
        l = l * sa + ml.y * sb;
        m = mn;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float4 v = box[32 * k];
          o[2 * k][0] = o[2 * k][0] * sa + v.x * sb;
          o[2 * k][1] = o[2 * k][1] * sa + v.y * sb;
          o[2 * k + 1][0] = o[2 * k + 1][0] * sa + v.z * sb;
          o[2 * k + 1][1] = o[2 * k + 1][1] * sa + v.w * sb;
        }
      }
      hand_over();
    }
    const bool wide = kF16 && s_wide;   // its result is left for redo_wide
    __syncthreads();
    if (wide) {
      if (tid == 0) {
        s_wide = 0;
        any_redo = 1;
        redo[kF16 ? s >> 5 : 0] |= 1u << (s & 31);
      }
      __syncthreads();
      continue;
    }
    int c0, c1;
    owners(split, nb, T, rpre[s], rpre[s + 1], c0, c1);
    finish<W, kF16>(A, mbuf, &s_merge, s, c0, c1);
  }
  if constexpr (kF16) {   // any_redo is set before a barrier
    if (any_redo) redo_wide<W, U, S>(A, tab, redo, &s_split, &s_merge);
  }
}

template <int FMT, int W, int U, int S>
constexpr size_t smem_bytes(int n_slices) {
  const size_t blk = FMT == kPageInt4 ? kBlockBytes4 : kBlockBytes16;
  return W * U * S * blk + (size_t)(W + 1) / 2 * kMergeWords * 4 + kMaxGroup * kQRow * 4 +
         (size_t)(n_slices + 1) * 8 + (size_t)n_slices * 8;
}
constexpr size_t smem_most(int format) { return (format == kPageInt4 ? 212 : 226) * 1024; }   // 227 KB less the static arrays
// Warps and units an item.  Ring slots: 2, and 3 for 4-bit calls without lists where the slices' prefix leaves room.
// us with 2 slots against 3: 1M rows of 4 bits 359 / 344; 4 x 128K with lists 50.1 / 51.6; 16 x 64K of bf16 127 / 134.
constexpr int kW4 = 12, kU4 = 2;
constexpr int kW16 = 8, kU16 = 1;
constexpr int kSlots = 2, kDeep4 = 3;

template <int FMT, int W, int U, int S, bool WIDE, bool LISTED>
bool setup_one() {
  return cudaFuncSetAttribute(k_attend_paged<FMT, W, U, S, WIDE, LISTED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)smem_most(FMT)) == cudaSuccess;
}
template <int FMT, int W, int U, bool WIDE>
bool setup() {
  static_assert(smem_bytes<FMT, W, U, kSlots>(kMaxPagedSlices) <= smem_most(FMT), "two slots fit every call");
  return setup_one<FMT, W, U, kSlots, WIDE, false>() && setup_one<FMT, W, U, kSlots, WIDE, true>();
}
template <int FMT, int W, int U, int S, bool WIDE, bool LISTED>
cudaError_t launch(const PagedAttendArgs& a, int grid, const RopeTab128& tab, cudaStream_t st) {
  k_attend_paged<FMT, W, U, S, WIDE, LISTED><<<grid, W * 32, smem_bytes<FMT, W, U, S>(a.n_slices), st>>>(a, tab);
  return cudaGetLastError();
}
template <int FMT, int W, int U, bool WIDE>
cudaError_t go(const PagedAttendArgs& a, int grid, const RopeTab128& tab, cudaStream_t st) {
  return a.list ? launch<FMT, W, U, kSlots, WIDE, true>(a, grid, tab, st)
                : launch<FMT, W, U, kSlots, WIDE, false>(a, grid, tab, st);
}

}  // namespace

int page_attend_setup(int format) {
  if (format == kPageInt4) return setup<kPageInt4, kW4, kU4, false>() && setup_one<kPageInt4, kW4, kU4, kDeep4, false, false>();
  return setup<kPageBf16, kW16, kU16, false>() && setup<kPageBf16, kW16, kU16, true>();
}

cudaError_t launch_page_attend(const PagedAttendArgs& a, int format, int grid, const RopeTab128& tab, cudaStream_t st) {
  if (format == kPageInt4) {
    if (!a.list && smem_bytes<kPageInt4, kW4, kU4, kDeep4>(a.n_slices) <= smem_most(kPageInt4))
      return launch<kPageInt4, kW4, kU4, kDeep4, false, false>(a, grid, tab, st);
    return go<kPageInt4, kW4, kU4, false>(a, grid, tab, st);
  }
  return a.G <= 4 ? go<kPageBf16, kW16, kU16, false>(a, grid, tab, st) : go<kPageBf16, kW16, kU16, true>(a, grid, tab, st);
}

}  // namespace spa
