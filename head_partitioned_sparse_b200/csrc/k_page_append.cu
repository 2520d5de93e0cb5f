// Appending key and value rows to a paged cache, the rotation of the keys applied on the way,
// and reading pages back into contiguous rows.
//
// Block of 16 tokens of one KV head (pages are made of them):
//   4 bits (2304 bytes): K codes [16][64], V codes [16][64], bf16 scales [16][8];
//     dim d of a row is nibble d, low nibble first; its value is scale * (nibble - 8).
//     K dim d is in scale group (d / 8) % 4, V dim d in group (d / 4) % 4: 32 dims a group.  The
//     groups are strided so that one 8-code word of the attention's K operand, and one column
//     tile of its V operand, belong to a single group.
//   bf16 (8192 bytes): K [16][128], V [16][128]; 16-byte piece c of row r at piece c ^ (r % 8),
//     which makes the attention's matrix loads conflict-free after a straight bulk copy.
//
// Rounding to 4 bits: scale = bf16(amax / 7), code = clamp(round_even(x / scale), -7, 7) + 8.
// Sixteen levels lose one to the symmetric range, and need no offset beside the scale: 144 bytes a
// row pair instead of 160.  Every decision is the one exact arithmetic takes: a float32
// quotient within its error of a border is decided again by an exact product (rows that are
// stored as given), or the whole row is computed again in 64 bits (rotated keys; about 1 row in 500).
//
// Bound by memory: a row pair moves 512 + 144 bytes at bf16.  16 lanes own the K and V rows of one
// (token, head), 8 dims each: 16-byte loads, one 32-bit code word a lane, group maxima in 2-3 shuffles.
// A lane's cosines and sines serve all the heads it takes of its token.
#include "spa_paged.cuh"

namespace spa {
namespace {

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&f)[8]) {
  const uint4 w = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(u[i]);
    f[2 * i + 1] = bf16_hi(u[i]);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&f)[8]) { *reinterpret_cast<uint4*>(p) = pack8(f); }
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

// bf16(x / 7) rounded to nearest even, x >= 0 finite.  The bf16 below is found by division; the
// border above it has 9 significant bits, so 7 times it is exact in float32 and decides.
template <typename F>
__device__ __forceinline__ float seventh(F x) {
  const unsigned u = __float_as_uint((float)x / 7.f) & 0xffff0000u;
  const float border = __uint_as_float(u | 0x8000u);
  const F b7 = (F)border * (F)7;
  const bool up = x > b7 || (x == b7 && (u & 0x10000u));
  return __uint_as_float(up ? u + 0x10000u : u);
}
// Groups this small (2^-110: the reciprocal of their scale would overflow) are stored as zeros.
constexpr float kTiny = 7.7037198e-34f;
__device__ __forceinline__ float group_scale(float amax) {
  if (!(amax <= 3.4028235e38f)) return __uint_as_float(0x7fc00000u);   // infinity or NaN in the group
  return amax < kTiny ? 0.f : seventh(amax);
}

// Code 1..15 of x under scale s (inv = 1 / s), decided exactly.
__device__ __forceinline__ unsigned code_exact(float x, float s, float inv) {
  const float q = x * inv;
  float n = rintf(q);
  if (fabsf(fabsf(q - n) - 0.5f) < 1e-5f) {
    const float k = floorf(fabsf(q)), border = (k + 0.5f) * s;   // 4 bits times 8 bits: exact
    const float ax = fabsf(x);
    const float m = ax > border ? k + 1.f : ax < border ? k : 2.f * rintf(0.5f * (k + 0.5f));   // a tie goes to the even one
    n = copysignf(m, x);
  }
  return (unsigned)((int)fminf(fmaxf(n, -7.f), 7.f) + 8);
}

template <typename F>
__device__ __forceinline__ F shfl_max(unsigned mask, F v, int o) {
  const F w = __shfl_xor_sync(mask, v, o);
  return w > v ? w : v;
}

// Page base of (sequence b, position pos, head 0), or null.
__device__ __forceinline__ unsigned char* page_of(const PagePool& P, int b, int64_t pos, int& blk, int& r) {
  if (pos < 0 || pos >= (int64_t)P.max_pages * P.page_size) {
    atomicOr(P.err, kErrStartPos);
    return nullptr;
  }
  const unsigned p = (unsigned)pos;
  const unsigned pg = p / (unsigned)P.page_size, in = p - pg * (unsigned)P.page_size;
  const int id = P.table[(size_t)b * P.max_pages + pg];
  if (id < 0 || id >= P.n_pages) {
    atomicOr(P.err, kErrPage);
    return nullptr;
  }
  blk = (int)(in / kBlockTok);
  r = (int)(in % kBlockTok);
  return P.pages + (size_t)id * P.Hkv * P.head_bytes;
}

// Rows of sequence b that a call covers.
__device__ __forceinline__ int row_count(const int64_t* n, int b, int T, unsigned* err) {
  if (!n) return T;
  const int64_t v = n[b];
  if (v < 0 || v > T) {
    atomicOr(err, kErrSeqLen);
    return v < 0 ? 0 : T;
  }
  return (int)v;
}

// PAIR: how a lane gets the partners of its 8 dims.
constexpr int kNone = 0;      // no rotation
constexpr int kInLane = 1;    // interleaved pairs
constexpr int kShuffle = 2;   // halves, rot / 2 a multiple of 8: the partners are one lane's 8 dims
constexpr int kReload = 3;    // halves, any rot: single loads

template <typename T, int FMT, int PAIR>
__global__ void __launch_bounds__(256) k_page_append(const PagePool P, const AppendArgs a, const __grid_constant__ RopeTab128 tab) {
  const int lane = threadIdx.x & 31, e = lane & 15;
  const unsigned mask = 0xffffu << (lane & 16);
  const int64_t item = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 4;
  const int64_t tok = item / a.head_groups;
  if (tok >= (int64_t)a.B * a.T) return;
  const int hg = (int)(item - tok * a.head_groups);
  const int b = (int)(tok / a.T), t = (int)(tok - (int64_t)b * a.T);
  if (t >= row_count(a.n_new, b, a.T, P.err)) return;
  const int64_t pos = a.start[b] + t;
  int blk, r;
  unsigned char* const page = page_of(P, b, pos, blk, r);
  if (!page) return;
  const int half = tab.rot / 2;
  const bool turned = PAIR != kNone && 8 * e < tab.rot;

  // element i of the lane (dim 8 e + i) becomes x c[i] + partner sn[i]
  float c[8], sn[8];
  const float mag = (float)tab.mag;
  if (PAIR == kInLane) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      c[i] = c[i + 1] = 1.f;
      sn[i] = sn[i + 1] = 0.f;
      if (8 * e + i < tab.rot) {
        rope_cs(tab.f_pi[4 * e + i / 2], (double)pos, mag, c[i], sn[i + 1]);
        c[i + 1] = c[i];
        sn[i] = -sn[i + 1];
      }
    }
  } else if (PAIR != kNone) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int d = 8 * e + i;
      c[i] = 1.f;
      sn[i] = 0.f;
      if (d < tab.rot) {
        rope_cs(tab.f_pi[d < half ? d : d - half], (double)pos, mag, c[i], sn[i]);
        if (d < half) sn[i] = -sn[i];
      }
    }
  }
  const T* krow = static_cast<const T*>(a.k) + b * a.ks.b + t * a.ks.t;
  const T* vrow = static_cast<const T*>(a.v) + b * a.vs.b + t * a.vs.t;

  for (int g = hg; g < P.Hkv; g += a.head_groups) {
    float x[8], p[8], y[8], v[8];
    const T* kh = krow + g * a.ks.h;
    load8(kh + 8 * e, x);
    load8(vrow + g * a.vs.h + 8 * e, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = 0.f;
    if (PAIR == kInLane) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (8 * e + i < tab.rot) p[i] = x[i ^ 1];
    } else if (PAIR == kShuffle) {
      const int n8 = half / 8, src = e < n8 ? e + n8 : e - n8;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float w = __shfl_sync(mask, x[i], (lane & 16) + (src & 15));
        if (turned) p[i] = w;
      }
    } else if (PAIR == kReload) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int d = 8 * e + i;
        if (d < tab.rot) p[i] = Elem<T>::get(kh, d < half ? d + half : d - half);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = PAIR == kNone ? x[i] : fmaf(x[i], c[i], p[i] * sn[i]);

    unsigned char* const blkp = page + (size_t)g * P.head_bytes + (size_t)blk * (FMT == kPageInt4 ? kBlockBytes4 : kBlockBytes16);
    if (FMT == kPageBf16) {
      // the cache keeps 16 bits: one rounding of the float32 rotation
      *reinterpret_cast<uint4*>(blkp + r * 256 + ((e ^ (r & 7)) << 4)) = pack8(y);
      *reinterpret_cast<uint4*>(blkp + kBlockTok * 256 + r * 256 + ((e ^ (r & 7)) << 4)) = pack8(v);
      continue;
    }
    // ---- group maxima of |K| (as bit patterns, so that NaN is above infinity) and |V|
    unsigned kb = 0u, v0 = 0u, v1 = 0u;
    float off = 0.f;   // bound of the float32 rotation's error over the group
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      kb = max(kb, __float_as_uint(y[i]) & 0x7fffffffu);
      const unsigned w = __float_as_uint(v[i]) & 0x7fffffffu;
      if (i < 4) v0 = max(v0, w);
      else v1 = max(v1, w);
      // cos and sin are off by at most 1.6e-7 (argument and function) and 6e-8 (magnitude), the
      // products and the sum by 6e-8 each
      if (PAIR != kNone) off = fmaxf(off, (fabsf(x[i]) + fabsf(p[i])));
    }
#pragma unroll
    for (int o = 4; o <= 8; o <<= 1) {
      kb = shfl_max(mask, kb, o);
      if (PAIR != kNone) off = shfl_max(mask, off, o);
    }
#pragma unroll
    for (int o = 2; o <= 8; o <<= 1) {
      v0 = shfl_max(mask, v0, o);
      v1 = shfl_max(mask, v1, o);
    }
    off *= 5e-7f * fmaxf(mag, 1.f);
    const float amax = __uint_as_float(kb);
    float ks = group_scale(amax);
    const float vs0 = group_scale(__uint_as_float(v0)), vs1 = group_scale(__uint_as_float(v1));
    unsigned kw = 0u, vw = 0u;
    bool plain = ks > 0.f;   // a scale of 0 or NaN goes with code 8 everywhere
    const float ki = plain ? 1.f / ks : 0.f;
    if (PAIR == kNone) {
#pragma unroll
      for (int i = 0; i < 8; ++i) kw |= (plain ? code_exact(y[i], ks, ki) : 8u) << (4 * i);
    } else {
      // near: a border of the scale's or of a code's rounding lies within the error
      bool near = plain && (group_scale(amax + off) != ks || group_scale(fmaxf(amax - off, 0.f)) != ks);
      const float lim = off * ki + 2e-6f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float q = y[i] * ki, n = rintf(q);
        near |= plain && 0.5f - fabsf(q - n) < lim;
        kw |= (plain ? (unsigned)((int)fminf(fmaxf(n, -7.f), 7.f) + 8) : 8u) << (4 * i);
      }
      if (__any_sync(mask, near)) {   // the row again in 64 bits
        double z[8], am = 0.0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int d = 8 * e + i;
          z[i] = (double)x[i];
          if (d < tab.rot) {
            const int j = PAIR == kInLane ? d >> 1 : d < half ? d : d - half;
            double s64, c64;
            sincospi(angle_pi(tab.f_pi[j], (double)pos), &s64, &c64);
            if (PAIR == kInLane ? !(i & 1) : d < half) s64 = -s64;
            z[i] = (double)x[i] * (c64 * tab.mag) + (double)p[i] * (s64 * tab.mag);
          }
          am = fmax(am, fabs(z[i]));
        }
        am = shfl_max(mask, am, 4);
        am = shfl_max(mask, am, 8);
        if (plain) {
          ks = seventh(am);
          kw = 0u;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            kw |= (unsigned)((int)fmin(fmax(rint(z[i] / (double)ks), -7.0), 7.0) + 8) << (4 * i);
        }
      }
    }
    const float vi0 = vs0 > 0.f ? 1.f / vs0 : 0.f, vi1 = vs1 > 0.f ? 1.f / vs1 : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = i < 4 ? vs0 : vs1, inv = i < 4 ? vi0 : vi1;
      vw |= (s > 0.f ? code_exact(v[i], s, inv) : 8u) << (4 * i);
    }
    reinterpret_cast<unsigned*>(blkp + r * kRow4)[e] = kw;
    reinterpret_cast<unsigned*>(blkp + kBlockTok * kRow4 + r * kRow4)[e] = vw;
    // scales: K group g in lane g; V groups 0, 1 in lane 0 and 2, 3 in lane 1
    unsigned char* const sc = blkp + 2 * kBlockTok * kRow4 + r * 16;
    if (e < 4) reinterpret_cast<unsigned short*>(sc)[e] = (unsigned short)(__float_as_uint(ks) >> 16);
    if (e < 2) reinterpret_cast<unsigned*>(sc + 8)[e] = (__float_as_uint(vs0) >> 16) | (__float_as_uint(vs1) & 0xffff0000u);
  }
}

// 4-bit word to 8 values n - 8 (exact small integers).
__device__ __forceinline__ void nibbles(unsigned w, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(0x4b000000u | ((w >> (4 * i)) & 15u)) - 8388616.f;
}

// A warp takes 16 consecutive rows of one (sequence, head); a half-warp reads and writes whole
// rows, all 8 row pairs in flight together.
template <typename T, int FMT>
__global__ void __launch_bounds__(256) k_page_read(const PagePool P, const ReadArgs a) {
  const int lane = threadIdx.x & 31, e = lane & 15;
  const int64_t unit = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 5;
  const int per_seq = (a.T + 15) / 16;
  const int64_t slice = unit / per_seq;
  if (slice >= (int64_t)a.B * P.Hkv) return;
  const int b = (int)(slice / P.Hkv), g = (int)(slice - (int64_t)b * P.Hkv);
  const int i0 = (int)(unit - slice * per_seq) * 16;
  const int n = row_count(a.n_rows, b, a.T, P.err);
  if (i0 >= n) return;
  // lane l < 16: where row i0 + l lies (-1: nowhere)
  long long at = -1;
  if (lane < 16 && i0 + lane < n) {
    int blk, r;
    unsigned char* const page = page_of(P, b, a.start[b] + i0 + lane, blk, r);
    if (page)
      at = (page - P.pages) + (long long)g * P.head_bytes + (long long)blk * (FMT == kPageInt4 ? kBlockBytes4 : kBlockBytes16) + r;
  }
  T* const kd = static_cast<T*>(a.k) + b * a.ks.b + g * a.ks.h;
  T* const vd = static_cast<T*>(a.v) + b * a.vs.b + g * a.vs.h;
  unsigned kw[8], vw[8];
  uint4 kq[8], vq[8], sc[8];
  long long base[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int row = 2 * u + (lane >> 4);
    base[u] = __shfl_sync(0xffffffffu, at, row);
    if (base[u] < 0) continue;
    // at packs the block's offset (a multiple of 256) and the row within the block
    const int r = (int)(base[u] & 15);
    const unsigned char* blkp = P.pages + (base[u] - r);
    if (FMT == kPageInt4) {
      kw[u] = __ldg(reinterpret_cast<const unsigned*>(blkp + r * kRow4) + e);
      vw[u] = __ldg(reinterpret_cast<const unsigned*>(blkp + kBlockTok * kRow4 + r * kRow4) + e);
      sc[u] = __ldg(reinterpret_cast<const uint4*>(blkp + 2 * kBlockTok * kRow4) + r);
    } else {
      const int o = r * 256 + ((e ^ (r & 7)) << 4);
      kq[u] = __ldg(reinterpret_cast<const uint4*>(blkp + o));
      vq[u] = __ldg(reinterpret_cast<const uint4*>(blkp + kBlockTok * 256 + o));
    }
  }
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    if (base[u] < 0) continue;
    const int i = i0 + 2 * u + (lane >> 4);
    float k[8], v[8];
    if (FMT == kPageInt4) {
      nibbles(kw[u], k);
      nibbles(vw[u], v);
      const unsigned kg = (e & 2) ? sc[u].y : sc[u].x, vg = (e & 1) ? sc[u].w : sc[u].z;
      const float s = (e & 1) ? bf16_hi(kg) : bf16_lo(kg), v0 = bf16_lo(vg), v1 = bf16_hi(vg);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        k[j] *= s;
        v[j] *= j < 4 ? v0 : v1;
      }
    } else {
      const uint32_t uk[4] = {kq[u].x, kq[u].y, kq[u].z, kq[u].w}, uv[4] = {vq[u].x, vq[u].y, vq[u].z, vq[u].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        k[2 * j] = bf16_lo(uk[j]);
        k[2 * j + 1] = bf16_hi(uk[j]);
        v[2 * j] = bf16_lo(uv[j]);
        v[2 * j + 1] = bf16_hi(uv[j]);
      }
    }
    store8(kd + i * a.ks.t + 8 * e, k);
    store8(vd + i * a.vs.t + 8 * e, v);
  }
}

template <typename T, int FMT>
cudaError_t append_go(const PagePool& pool, const AppendArgs& a, const RopeTab128& tab, unsigned blocks, cudaStream_t st) {
  if (tab.rot == 0) k_page_append<T, FMT, kNone><<<blocks, 256, 0, st>>>(pool, a, tab);
  else if (tab.interleaved) k_page_append<T, FMT, kInLane><<<blocks, 256, 0, st>>>(pool, a, tab);
  else if (tab.rot % 16 == 0) k_page_append<T, FMT, kShuffle><<<blocks, 256, 0, st>>>(pool, a, tab);
  else k_page_append<T, FMT, kReload><<<blocks, 256, 0, st>>>(pool, a, tab);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_page_append(const PagePool& pool, AppendArgs a, int dtype, int format, const RopeTab128& tab,
                               int num_sms, cudaStream_t st) {
  // A thread takes up to 8 heads of its token, fewer while the GPU would not be full.
  const int64_t toks = (int64_t)a.B * a.T;
  a.head_groups = (pool.Hkv + 7) / 8;
  while (a.head_groups < pool.Hkv && toks * a.head_groups * 16 < (int64_t)num_sms * 1024) a.head_groups *= 2;
  if (a.head_groups > pool.Hkv) a.head_groups = pool.Hkv;
  const int64_t blocks = (toks * a.head_groups * 16 + 255) / 256;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  if (dtype == 0)
    return format == kPageInt4 ? append_go<__nv_bfloat16, kPageInt4>(pool, a, tab, (unsigned)blocks, st)
                               : append_go<__nv_bfloat16, kPageBf16>(pool, a, tab, (unsigned)blocks, st);
  return format == kPageInt4 ? append_go<float, kPageInt4>(pool, a, tab, (unsigned)blocks, st)
                             : append_go<float, kPageBf16>(pool, a, tab, (unsigned)blocks, st);
}

cudaError_t launch_page_read(const PagePool& pool, const ReadArgs& a, int dtype, int format, cudaStream_t st) {
  const int64_t units = (int64_t)a.B * pool.Hkv * ((a.T + 15) / 16);
  const int64_t blocks = (units * 32 + 255) / 256;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  const unsigned nb = (unsigned)blocks;
  if (dtype == 0) {
    if (format == kPageInt4) k_page_read<__nv_bfloat16, kPageInt4><<<nb, 256, 0, st>>>(pool, a);
    else k_page_read<__nv_bfloat16, kPageBf16><<<nb, 256, 0, st>>>(pool, a);
  } else {
    if (format == kPageInt4) k_page_read<float, kPageInt4><<<nb, 256, 0, st>>>(pool, a);
    else k_page_read<float, kPageBf16><<<nb, 256, 0, st>>>(pool, a);
  }
  return cudaGetLastError();
}

}  // namespace spa
