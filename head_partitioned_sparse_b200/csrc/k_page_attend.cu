// Single-token attention over a paged cache held in 4 bits or in bf16.
//
// out[b][h] = sum_j softmax_j(<m R(L-1) q[b][h], K_j> / sqrt(128)) V_j over the rows j that head h's KV
// head attends: every row, or sinks and window, or sinks, window and a selected list.
//
// Work layout.  The attended rows of all (sequence, KV head) slices are cut into units of 16
// rows: whole 16-token blocks of the pages (edges masked), or 16 listed rows.  Every CTA (one an
// SM) takes an equal contiguous share of the units, one piece per slice it touches, and its warps the units
// of a piece in turn.  Each warp streams its units through its own ring in shared memory: a
// block is one bulk copy (2304 bytes in 4 bits, K, V and scales together), a listed unit is
// gathered by 16-byte asynchronous copies.  The list position of the unit after next and the block table
// entry of the next one are loaded ahead, so no copy waits for an index.  Warps keep their own
// running maximum and sum, merged by a tree at the end of a piece; the last CTA to finish a
// slice (a ticket) merges the CTAs' states in order, so the result does not depend on timing.
//
// Matrix mapping (mma.sync m16n8k16, M = 8 heads as bf16 high parts over 8 rows of bf16 residuals, so scores and
// sums keep about 17 bits):
//   4 bits: a code word (8 nibbles) becomes four bf16 pairs of 128 + n, (nibble j, nibble j + 4), less 136.
//     Scores: word w of a lane's 16 bytes is scale group w of its 32 dims, so the products of a group
//     are summed by themselves and scaled once a (row, group), not once an element.
//     Values: the halves of two rows' words are merged by one byte permute into (row, row + 1)
//     pairs; column tile t holds dims 16 n + t, all of scale group t / 4, whose scales go into the
//     probabilities (four sets of them).
//   bf16: matrix loads from the swizzled rows.
//
// Masked rows: their score is -infinity and their value scale (bf16: their value) 0, whatever the page holds there.
#include "spa_paged.cuh"

namespace spa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 8;
constexpr float kNoMax = -1e30f;        // running maximum before the first row
constexpr unsigned kWaitTries = 1u << 22;

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void mbar_init(uint32_t bar, unsigned n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar, uint64_t pol) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar), "l"(pol)
      : "memory");
}
__device__ __forceinline__ bool mbar_wait(uint32_t bar, unsigned parity) {
  for (unsigned i = 0; i < kWaitTries; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
  }
  return false;
}
__device__ __forceinline__ uint64_t l2_evict_first() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;\n" : "=l"(p));
  return p;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// (nibble j, nibble j + 4) of w as a bf16 pair of n - 8: 128 + n by its bits, less 136 (exact).
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int j) {
  uint32_t u = ((w >> (4 * j)) & 0x000f000fu) | 0x43004300u;
  __nv_bfloat162 v = *reinterpret_cast<__nv_bfloat162*>(&u);
  v = __hsub2(v, __nv_bfloat162(__float2bfloat16_rn(136.f), __float2bfloat16_rn(136.f)));
  return *reinterpret_cast<uint32_t*>(&v);
}
// The bf16 high parts and residuals of a pair.
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack2(x, y);
  lo = pack2(x - bf16_lo(hi), y - bf16_hi(hi));
}

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

// A unit on its way to the ring: what has been loaded of it so far.
struct Unit {
  int s;        // slice, -1: none
  int list;     // listed rows (else one block)
  int pos;      // lane l < 16: position of row l (block: of row 0)
  bool ok;      // lane l < 16: row l is attended
  int id;       // page of pos
};

template <int FMT, int S>
__global__ void __launch_bounds__(kWarps * 32, 1) k_attend_paged(const PagedAttendArgs A, const __grid_constant__ RopeTab128 tab) {
  constexpr int kBlk = FMT == kPageInt4 ? kBlockBytes4 : kBlockBytes16;
  extern __shared__ __align__(128) unsigned char smem[];
  unsigned char* const ring = smem;                                              // [8][S][kBlk]
  float* const mbuf = reinterpret_cast<float*>(smem + (size_t)kWarps * S * kBlk);   // [4][8][kPartStride]
  float* const cbuf = mbuf + 4 * kMaxGroup * kPartStride;                        // [8][kPartStride]
  float* const qs = cbuf + kWarps * kPartStride;                                 // [8][128]
  long long* const rpre = reinterpret_cast<long long*>(qs + kMaxGroup * kHeadDim);  // [n_slices + 1]
  int2* const sinfo = reinterpret_cast<int2*>(rpre + A.n_slices + 1);            // [n_slices] (L, listed rows)
  __shared__ __align__(8) unsigned long long bars[kWarps * S];
  __shared__ unsigned vmask[kWarps * S];   // attended rows of a ring slot; bit 16: gathered
  __shared__ long long shl[kWarps];
  __shared__ int s_merge;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gid = lane >> 2, t4 = lane & 3;
  const int NS = A.n_slices, Hkv = A.pool.Hkv, G = A.G;

  if (tid < kWarps * S) mbar_init(smem_u32(&bars[tid]), 1);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");

  // ---- unit prefix over slices
  {
    long long carry = 0;
    for (int base = 0; base < NS; base += kWarps * 32) {
      const int s = base + tid;
      long long n = 0;
      if (s < NS) {
        const int b = s / Hkv, g = s - b * Hkv;
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
        n = units_of(make_slice(A, g, (int)L, cnt));
      }
      long long v = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(kFull, v, o);
        if (lane >= o) v += y;
      }
      if (lane == 31) shl[warp] = v;
      __syncthreads();
      long long before = carry, total = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const long long x = shl[w];
        if (w < warp) before += x;
        total += x;
      }
      if (s < NS) rpre[s] = before + v - n;
      carry += total;
      __syncthreads();
    }
    if (tid == 0) rpre[NS] = carry;
    __syncthreads();
  }
  const long long T = rpre[NS];
  // slices without a row: zeros
  for (int s = blockIdx.x; s < NS; s += gridDim.x) {
    if (rpre[s + 1] != rpre[s]) continue;
    const size_t h0 = (size_t)(s / Hkv) * A.Hq + (size_t)(s % Hkv) * G;
    for (int i = tid; i < G * kHeadDim; i += kWarps * 32) A.out[h0 * kHeadDim + i] = 0.f;
    if (A.lse && tid < G) A.lse[h0 + tid] = -INFINITY;
  }
  // every active CTA has at least one unit a warp
  const long long want = (T + kWarps - 1) / kWarps;
  const int nb = (long long)gridDim.x < want ? (int)gridDim.x : (int)want;
  if ((int)blockIdx.x >= nb) return;
  const long long r_lo = (long long)blockIdx.x * T / nb, r_hi = (long long)(blockIdx.x + 1) * T / nb;
  auto owner = [&](long long r) { return (int)(((r + 1) * nb - 1) / T); };
  auto slice_of = [&](long long r) {
    int lo = 0, hi = NS - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (rpre[mid] <= r) lo = mid;
      else hi = mid - 1;
    }
    return lo;
  };
  const int s_first = slice_of(r_lo), s_last = slice_of(r_hi - 1);
  // units of slice s in this CTA's share
  auto piece = [&](int s, int& u0, int& n) {
    const long long a = max(r_lo, rpre[s]), e = min(r_hi, rpre[s + 1]);
    u0 = (int)(a - rpre[s]);
    n = e > a ? (int)(e - a) : 0;
  };

  unsigned char* const myring = ring + (size_t)warp * S * kBlk;
  const uint32_t ring_a = smem_u32(myring), bar_a = smem_u32(&bars[warp * S]);
  const uint64_t pol = l2_evict_first();

  // ---- the warp's unit cursor and the two units whose indices are being loaded
  int cs = s_first, cu = warp, c_u0, c_n;
  piece(cs, c_u0, c_n);
  Slice cS = make_slice(A, cs % Hkv, sinfo[cs].x, sinfo[cs].y);
  auto next_unit = [&]() {   // the cursor's unit with its position loads started; moves the cursor
    Unit U;
    U.s = -1;
    U.list = 0;
    U.pos = 0;
    U.ok = false;
    U.id = -1;
    while (cu >= c_n) {
      if (cs >= s_last) return U;
      ++cs;
      cu = warp;
      piece(cs, c_u0, c_n);
      cS = make_slice(A, cs % Hkv, sinfo[cs].x, sinfo[cs].y);
    }
    const int u = c_u0 + cu;
    cu += kWarps;
    U.s = cs;
    if (u < cS.nb0 + cS.nb1) {
      const int blk = u < cS.nb0 ? u : cS.b1 + (u - cS.nb0);
      U.pos = blk * kBlockTok;
      const int p = U.pos + lane;
      U.ok = lane < kBlockTok && p < cS.L && (p < cS.n_s || p >= cS.w_lo);
    } else {
      U.list = 1;
      const int i = (u - cS.nb0 - cS.nb1) * 16 + lane;
      U.ok = lane < 16 && i < cS.cnt;
      if (U.ok) U.pos = __ldg(A.list + (size_t)cs * A.list_stride + i);
    }
    return U;
  };
  auto load_page = [&](Unit& U) {
    if (U.s < 0) return;
    if (U.list && U.ok && (U.pos < 0 || U.pos >= sinfo[U.s].x)) {
      atomicOr(A.pool.err, kErrList);
      U.ok = false;
      U.pos = 0;
    }
    const int b = U.s / Hkv;
    const unsigned pg = ((unsigned)U.pos / kBlockTok) / (unsigned)A.pool.page_blocks;
    if (!U.list || U.ok) U.id = __ldg(A.pool.table + (size_t)b * A.pool.max_pages + pg);
  };
  int issued = 0;          // ring slot of the next issue
  unsigned was_list = 0u;  // slots last written by gathers
  auto issue = [&](const Unit& U) {
    if (U.s >= 0) {
      const bool page_ok = (unsigned)U.id < (unsigned)A.pool.n_pages;
      if (!page_ok && (U.ok || (!U.list && lane == 0))) atomicOr(A.pool.err, kErrPage);
      const unsigned m = __ballot_sync(kFull, U.ok && page_ok) & 0xffffu;
      const int g = U.s % Hkv;
      const unsigned blkno = (unsigned)U.pos / kBlockTok;
      const unsigned in = blkno % (unsigned)A.pool.page_blocks;
      const long long off = page_ok ? ((long long)U.id * Hkv + g) * A.pool.head_bytes + (long long)in * kBlk : 0;
      const uint32_t dst = ring_a + issued * kBlk;
      if (!U.list) {
        if (m && lane == 0) {
          if (was_list >> issued & 1u) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          bulk_load(dst, A.pool.pages + off, kBlk, bar_a + 8 * issued, pol);
        }
        was_list &= ~(1u << issued);
      } else {
        was_list |= 1u << issued;
        const long long at = off + (U.pos & (kBlockTok - 1));   // block offset (a multiple of 256) and row
        if (FMT == kPageInt4) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = i * 8 + gid;
            const long long a = __shfl_sync(kFull, at, r);
            if (m >> r & 1u) {
              const int rin = (int)(a & 15);
              const unsigned char* src = A.pool.pages + (a - rin) + rin * kRow4 + t4 * 16;
              cp_async16(dst + r * kRow4 + t4 * 16, src);
              cp_async16(dst + kBlockTok * kRow4 + r * kRow4 + t4 * 16, src + kBlockTok * kRow4);
            }
          }
          if (lane < 16 && (m >> lane & 1u)) {
            const int rin = (int)(at & 15);
            cp_async16(dst + 2 * kBlockTok * kRow4 + lane * 16, A.pool.pages + (at - rin) + 2 * kBlockTok * kRow4 + rin * 16);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = i * 2 + (lane >> 4), c = lane & 15;
            const long long a = __shfl_sync(kFull, at, r);
            if (m >> r & 1u) {
              const int rin = (int)(a & 15);
              const unsigned char* src = A.pool.pages + (a - rin) + rin * 256 + ((c ^ (rin & 7)) << 4);
              const uint32_t d = dst + r * 256 + ((c ^ (r & 7)) << 4);
              cp_async16(d, src);
              cp_async16(d + kBlockTok * 256, src + kBlockTok * 256);
            }
          }
        }
      }
      if (lane == 0) vmask[warp * S + issued] = m | (U.list ? 0x10000u : 0u);
      issued = issued + 1 == S ? 0 : issued + 1;
    }
    asm volatile("cp.async.commit_group;\n" ::: "memory");
  };
  Unit ub = next_unit();
  load_page(ub);
  Unit ua = next_unit();
  auto step = [&]() {
    issue(ub);
    ub = ua;
    load_page(ub);
    ua = next_unit();
  };
#pragma unroll 1
  for (int i = 0; i < S - 1; ++i) step();

  int slot = 0;           // ring slot to consume
  unsigned parity = 0u;   // phase of each slot's barrier

  for (int s = s_first; s <= s_last; ++s) {
    int u0, n_u;
    piece(s, u0, n_u);
    if (n_u == 0) continue;
    const int b = s / Hkv, g = s - b * Hkv;
    const size_t h0 = (size_t)b * A.Hq + (size_t)g * G;
    // ---- the group's queries, rotated at position L - 1, times scale / ln 2
    {
      const int pos = sinfo[s].x - 1, half = tab.rot / 2;
      for (int i = tid; i < G * (kHeadDim / 2); i += kWarps * 32) {
        const int h = i >> 6, j = i & 63;
        const int d0 = j >= half ? tab.rot + 2 * (j - half) : tab.interleaved ? 2 * j : j;
        const int d1 = j >= half || tab.interleaved ? d0 + 1 : d0 + half;
        float x, y;
        if (A.q_f32) {
          const float* q = static_cast<const float*>(A.q) + (h0 + h) * kHeadDim;
          x = q[d0];
          y = q[d1];
        } else {
          const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(A.q) + (h0 + h) * kHeadDim;
          x = __bfloat162float(q[d0]);
          y = __bfloat162float(q[d1]);
        }
        float c = 1.f, sn = 0.f;
        if (j < half) rope_cs(tab.f_pi[j], (double)pos, (float)tab.mag, c, sn);
        qs[h * kHeadDim + d0] = (x * c - y * sn) * A.scale_log2;
        qs[h * kHeadDim + d1] = (x * sn + y * c) * A.scale_log2;
      }
      __syncthreads();
    }
    // A operand: 4 bits: k-step 2w + i of word w holds dims 32 t4 + 8 w + 2 i + {0, 4, 1, 5}; bf16: natural order
    uint32_t qa[8][4];
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      const float* q = qs + (gid < G ? gid : 0) * kHeadDim;
      float x[4];
      if (FMT == kPageInt4) {
        const int d = 32 * t4 + 8 * (kk >> 1) + 2 * (kk & 1);
        x[0] = q[d];
        x[1] = q[d + 4];
        x[2] = q[d + 1];
        x[3] = q[d + 5];
      } else {
        const int d = 16 * kk + 2 * t4;
        x[0] = q[d];
        x[1] = q[d + 1];
        x[2] = q[d + 8];
        x[3] = q[d + 9];
      }
      if (gid >= G) x[0] = x[1] = x[2] = x[3] = 0.f;
      split2(x[0], x[1], qa[kk][0], qa[kk][1]);
      split2(x[2], x[3], qa[kk][2], qa[kk][3]);
    }
    float m = kNoMax, l = 0.f;
    float acc[16][4];
#pragma unroll
    for (int nt = 0; nt < 16; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;

#pragma unroll 1
    for (int u = warp; u < n_u; u += kWarps) {
      __syncwarp();
      step();   // refills the slot consumed last time
      const unsigned vm = vmask[warp * S + slot];
      const unsigned char* st = myring + slot * kBlk;
      const int my_slot = slot;
      slot = slot + 1 == S ? 0 : slot + 1;
      const unsigned rows = vm & 0xffffu;
      if (vm & 0x10000u) {
        asm volatile("cp.async.wait_group %0;\n" ::"n"(S - 1) : "memory");
        __syncwarp();
      } else if (rows) {
        if (!mbar_wait(bar_a + 8 * my_slot, parity >> my_slot & 1u)) {
          if (lane == 0) atomicOr(A.pool.err, kErrTimeout);
        }
        parity ^= 1u << my_slot;
      }
      if (!rows) continue;

      // ---- scores of head gid for rows 8 j + 2 t4 + e
      float sc[2][2];
      uint4 rs[2][2];   // 4 bits: the rows' scales
      if (FMT == kPageInt4) {
        uint4 kw[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          kw[j] = *reinterpret_cast<const uint4*>(st + (8 * j + gid) * kRow4 + t4 * 16);
#pragma unroll
          for (int e = 0; e < 2; ++e)
            rs[j][e] = *reinterpret_cast<const uint4*>(st + 2 * kBlockTok * kRow4 + (8 * j + 2 * t4 + e) * 16);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t w[4] = {kw[j].x, kw[j].y, kw[j].z, kw[j].w};
          float d[4][4];
#pragma unroll
          for (int g4 = 0; g4 < 4; ++g4) {
            d[g4][0] = d[g4][1] = d[g4][2] = d[g4][3] = 0.f;
            mma16816(d[g4], qa[2 * g4], code_pair(w[g4], 0), code_pair(w[g4], 1));
            mma16816(d[g4], qa[2 * g4 + 1], code_pair(w[g4], 2), code_pair(w[g4], 3));
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float a0 = bf16_lo(rs[j][e].x) * (d[0][e] + d[0][2 + e]);
            const float a1 = bf16_hi(rs[j][e].x) * (d[1][e] + d[1][2 + e]);
            sc[j][e] = fmaf(bf16_lo(rs[j][e].y), d[2][e] + d[2][2 + e], a0) +
                       fmaf(bf16_hi(rs[j][e].y), d[3][e] + d[3][2 + e], a1);
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
          mma16816(d[0][kk & 1], qa[kk], bk[0], bk[1]);
          mma16816(d[1][kk & 1], qa[kk], bk[2], bk[3]);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) sc[j][e] = (d[j][0][e] + d[j][1][e]) + (d[j][0][2 + e] + d[j][1][2 + e]);
      }
      const bool part = rows != 0xffffu;
      if (part) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (!(rows >> (8 * j + 2 * t4 + e) & 1u)) {
              sc[j][e] = -INFINITY;
              rs[j][e].z = rs[j][e].w = 0u;
            }
      }
      // ---- running maximum and sum
      float mx = fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[1][0], sc[1][1]));
      mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
      const float mn = fmaxf(m, mx);
      if (__any_sync(kFull, mn != m)) {
        const float alpha = ex2(m - mn);
#pragma unroll
        for (int nt = 0; nt < 16; ++nt) {
          acc[nt][0] *= alpha;
          acc[nt][1] *= alpha;
          acc[nt][2] *= alpha;
          acc[nt][3] *= alpha;
        }
        l *= alpha;
        m = mn;
      }
      float p[2][2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          p[j][e] = ex2(sc[j][e] - mn);
          l += p[j][e];
        }
      // ---- values
      if (FMT == kPageInt4) {
        const unsigned char* vb = st + kBlockTok * kRow4 + gid * 8;
        uint2 vw[2][2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) vw[j][e] = *reinterpret_cast<const uint2*>(vb + (8 * j + 2 * t4 + e) * kRow4);
#pragma unroll
        for (int g4 = 0; g4 < 4; ++g4) {
          float pv[2][2];
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t w = g4 < 2 ? rs[j][e].z : rs[j][e].w;
              pv[j][e] = p[j][e] * ((g4 & 1) ? bf16_hi(w) : bf16_lo(w));
            }
          uint32_t pa[4];
          split2(pv[0][0], pv[0][1], pa[0], pa[1]);
          split2(pv[1][0], pv[1][1], pa[2], pa[3]);
          uint32_t w[2];
#pragma unroll
          for (int j = 0; j < 2; ++j)
            w[j] = g4 < 2 ? __byte_perm(vw[j][0].x, vw[j][1].x, (g4 & 1) ? 0x7632 : 0x5410)
                          : __byte_perm(vw[j][0].y, vw[j][1].y, (g4 & 1) ? 0x7632 : 0x5410);
#pragma unroll
          for (int t = 0; t < 4; ++t) mma16816(acc[4 * g4 + t], pa, code_pair(w[0], t), code_pair(w[1], t));
        }
      } else {
        uint32_t pa[4];
        split2(p[0][0], p[0][1], pa[0], pa[1]);
        split2(p[1][0], p[1][1], pa[2], pa[3]);
        const int mi = lane >> 3, rr = lane & 7;
        const uint32_t row = smem_u32(st) + kBlockTok * 256 + (8 * (mi & 1) + rr) * 256;
        // rows 2 t4 + {0, 1} and + 8 as bit masks of the operand's halves
        uint32_t live0 = kFull, live1 = kFull;
        if (part) {
          const unsigned r0 = rows >> (2 * t4), r1 = rows >> (8 + 2 * t4);
          live0 = ((r0 & 1u) ? 0xffffu : 0u) | ((r0 & 2u) ? 0xffff0000u : 0u);
          live1 = ((r1 & 1u) ? 0xffffu : 0u) | ((r1 & 2u) ? 0xffff0000u : 0u);
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
          mma16816(acc[nt], pa, bv[0], bv[1]);
          mma16816(acc[nt + 1], pa, bv[2], bv[3]);
        }
      }
    }

    // ---- warp state: a head's sum over its 4 lanes, high and residual rows together
    l += __shfl_xor_sync(kFull, l, 1);
    l += __shfl_xor_sync(kFull, l, 2);
    float o[16][2];
#pragma unroll
    for (int nt = 0; nt < 16; ++nt) {
      o[nt][0] = acc[nt][0] + acc[nt][2];
      o[nt][1] = acc[nt][1] + acc[nt][3];
    }
    // dims of (column tile nt, e): 4 bits 32 t4 + 16 e + nt, bf16 8 nt + 2 t4 + e
    auto put = [&](float* dst) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int nt = 0; nt < 16; nt += 4)
          if (FMT == kPageInt4)
            *reinterpret_cast<float4*>(dst + 32 * t4 + 16 * e + nt) = make_float4(o[nt][e], o[nt + 1][e], o[nt + 2][e], o[nt + 3][e]);
          else if (e == 0)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              *reinterpret_cast<float2*>(dst + 8 * (nt + k) + 2 * t4) = make_float2(o[nt + k][0], o[nt + k][1]);
    };
    auto add = [&](const float* src, float sa, float sb) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int nt = 0; nt < 16; ++nt) {
          const float v = src[FMT == kPageInt4 ? 32 * t4 + 16 * e + nt : 8 * nt + 2 * t4 + e];
          o[nt][e] = o[nt][e] * sa + v * sb;
        }
    };
#pragma unroll 1
    for (int half = kWarps / 2; half >= 1; half >>= 1) {
      if (warp >= half && warp < 2 * half && gid < G) {
        float* dst = mbuf + ((size_t)(warp - half) * kMaxGroup + gid) * kPartStride;
        put(dst);
        if (t4 == 0) {
          dst[kHeadDim] = m;
          dst[kHeadDim + 1] = l;
        }
      }
      __syncthreads();
      if (warp < half && gid < G) {
        const float* src = mbuf + ((size_t)warp * kMaxGroup + gid) * kPartStride;
        const float m2 = src[kHeadDim], l2 = src[kHeadDim + 1];
        const float mn = fmaxf(m, m2);
        const float sa = exp2f(m - mn), sb = exp2f(m2 - mn);
        l = l * sa + l2 * sb;
        add(src, sa, sb);
        m = mn;
      }
      __syncthreads();
    }
    // ---- alone on the slice: the output; else its state, and the last CTA merges them
    const int c0 = owner(rpre[s]), c1 = owner(rpre[s + 1] - 1);
    if (warp == 0 && gid < G) {
      float* dst;
      if (c0 == c1) {
        const float inv = l == 0.f ? 0.f : 1.f / l;   // no weight at all: zeros
#pragma unroll
        for (int nt = 0; nt < 16; ++nt) {
          o[nt][0] *= inv;
          o[nt][1] *= inv;
        }
        dst = A.out + (h0 + gid) * kHeadDim;
        if (A.lse && t4 == 0) A.lse[h0 + gid] = l == 0.f ? -INFINITY : m + log2f(l);
      } else {
        dst = A.part + ((size_t)(blockIdx.x + s) * G + gid) * kPartStride;
        if (t4 == 0) {
          dst[kHeadDim] = m;
          dst[kHeadDim + 1] = l;
        }
      }
      put(dst);
      __threadfence();
    }
    if (c0 == c1) continue;
    __syncthreads();
    if (tid == 0) s_merge = atomicAdd(&A.ticket[s], 1u) == (unsigned)(c1 - c0);
    __syncthreads();
    if (!s_merge) continue;
    __threadfence();
    // warp w: head w % G, states c0 + w / G, c0 + w / G + per, ...; then the warps of a head in order
    {
      const int per = max(1, kWarps / G);
      const int h = warp % G, sub = warp / G;
      float M = kNoMax, Ls = 0.f;
      float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
      if (sub < per) {
        constexpr int kB = 8;
        for (int c = c0 + sub; c <= c1; c += per * kB) {
          float4 v[kB];
          float mi[kB], li[kB];
#pragma unroll
          for (int i = 0; i < kB; ++i) {
            const int cc = c + i * per;
            mi[i] = kNoMax;
            li[i] = 0.f;
            v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (cc <= c1) {
              const float* src = A.part + ((size_t)(cc + s) * G + h) * kPartStride;
              v[i] = __ldcg(reinterpret_cast<const float4*>(src) + lane);
              mi[i] = __ldcg(src + kHeadDim);
              li[i] = __ldcg(src + kHeadDim + 1);
            }
          }
#pragma unroll
          for (int i = 0; i < kB; ++i) {
            const float mn = fmaxf(M, mi[i]);
            const float sa = exp2f(M - mn), sb = exp2f(mi[i] - mn);
            Ls = Ls * sa + li[i] * sb;
            num.x = num.x * sa + v[i].x * sb;
            num.y = num.y * sa + v[i].y * sb;
            num.z = num.z * sa + v[i].z * sb;
            num.w = num.w * sa + v[i].w * sb;
            M = mn;
          }
        }
      }
      float* mine = cbuf + (size_t)warp * kPartStride;
      *reinterpret_cast<float4*>(mine + 4 * lane) = num;
      if (lane == 0) {
        mine[kHeadDim] = M;
        mine[kHeadDim + 1] = Ls;
      }
      __syncthreads();
      if (warp < G) {
        M = kNoMax;
        Ls = 0.f;
        num = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < per; ++k) {
          const float* src = cbuf + (size_t)(warp + G * k) * kPartStride;
          const float m2 = src[kHeadDim], l2 = src[kHeadDim + 1];
          const float mn = fmaxf(M, m2);
          const float sa = exp2f(M - mn), sb = exp2f(m2 - mn);
          const float4 v = *reinterpret_cast<const float4*>(src + 4 * lane);
          Ls = Ls * sa + l2 * sb;
          num.x = num.x * sa + v.x * sb;
          num.y = num.y * sa + v.y * sb;
          num.z = num.z * sa + v.z * sb;
          num.w = num.w * sa + v.w * sb;
          M = mn;
        }
        const float inv = Ls == 0.f ? 0.f : 1.f / Ls;
        reinterpret_cast<float4*>(A.out + (h0 + warp) * kHeadDim)[lane] = make_float4(num.x * inv, num.y * inv, num.z * inv, num.w * inv);
        if (A.lse && lane == 0) A.lse[h0 + warp] = Ls == 0.f ? -INFINITY : M + log2f(Ls);
      }
      if (tid == 0) A.ticket[s] = 0u;   // ready for the next call
      __syncthreads();
    }
  }
  asm volatile("cp.async.wait_all;\n" ::: "memory");
}

size_t smem_bytes(int format, int stages, int n_slices) {
  const size_t blk = format == kPageInt4 ? kBlockBytes4 : kBlockBytes16;
  return kWarps * stages * blk + (size_t)(4 * kMaxGroup + kWarps) * kPartStride * 4 + kMaxGroup * kHeadDim * 4 +
         (size_t)(n_slices + 1) * 8 + (size_t)n_slices * 8;
}
constexpr size_t kSmemMost = 226 * 1024;   // of 227 KB, less the static arrays
constexpr int kStages4 = 6, kStages16 = 3, kStages16Many = 2;
// bf16 blocks: three ring slots a warp where the slices' prefix leaves room for them, else two.
int stages_for(int format, int n_slices) {
  if (format == kPageInt4) return kStages4;
  return smem_bytes(format, kStages16, n_slices) <= kSmemMost ? kStages16 : kStages16Many;
}

template <int FMT, int S>
int setup_one() {
  return cudaFuncSetAttribute(k_attend_paged<FMT, S>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMost) == cudaSuccess;
}
template <int FMT, int S>
cudaError_t go(const PagedAttendArgs& a, int grid, const RopeTab128& tab, cudaStream_t st) {
  k_attend_paged<FMT, S><<<grid, kWarps * 32, smem_bytes(FMT, S, a.n_slices), st>>>(a, tab);
  return cudaGetLastError();
}

}  // namespace

int page_attend_setup(int format) {
  if (format == kPageInt4) return setup_one<kPageInt4, kStages4>();
  return setup_one<kPageBf16, kStages16>() && setup_one<kPageBf16, kStages16Many>();
}

cudaError_t launch_page_attend(const PagedAttendArgs& a, int format, int grid, const RopeTab128& tab, cudaStream_t st) {
  if (format == kPageInt4) return go<kPageInt4, kStages4>(a, grid, tab, st);
  return stages_for(format, a.n_slices) == kStages16 ? go<kPageBf16, kStages16>(a, grid, tab, st)
                                                      : go<kPageBf16, kStages16Many>(a, grid, tab, st);
}

}  // namespace spa
