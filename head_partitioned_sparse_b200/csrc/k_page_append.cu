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
// row pair instead of 160.  Every decision is the one exact arithmetic takes.  bf16 rows stored as
// given have 8 bits, so their scales and quotients are far from a border or exactly on it, and float32 decides both;
// a rotated key within the rotation's error of a border (about 1 row in 500 by the bounds used), a float32 row near one and a group
// that is tiny or not finite take a second, exact way: products of few bits, and 64 bits for the rotation.
//
// A row pair moves 512 + 144 bytes at bf16, so memory would bound it; the exact rounding does, by its instructions and the waits
// between them: 32K tokens of 8 heads take 51 us (3.4 TB/s) where a copy of the bytes takes 26 and the 247 instructions
// of two row pairs 28 at full issue (67 % of the slots are filled, by 16 warps an SM of 124 registers).  In float32 rows the append and the
// read of them take 138 us for 93 of bytes.  Into bf16
// pages, without them, that append and the read of its rows run at 0.9 of the copy rate (91 us, 537 MB).  8 lanes own the K and V rows of one (token, head),
// lane e the dims 8 e .. 8 e + 7 and 64 further of both: the pairs of a whole-head rotation meet in one lane, its 16
// dims are of one scale group of K and of two of V (group maxima in 1 and 2 shuffles), and every
// load and code word is 16 and 4 bytes.  A lane's cosines and sines serve all the heads it takes of its token.
#include "spa_paged.cuh"

namespace spa {
namespace {

// 8 dims of a row as loaded.  top(): float bits of the largest magnitude, NaN above infinity.
template <typename T>
struct Dims;
template <>
struct Dims<__nv_bfloat16> {
  uint32_t w[4];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_lo(w[i]);
      f[2 * i + 1] = bf16_hi(w[i]);
    }
  }
  // largest magnitudes of the even and the odd dims of words i and i + 1, 16 bits each
  __device__ __forceinline__ uint32_t top2(int i) const { return max_u16x2(w[i] & 0x7fff7fffu, w[i + 1] & 0x7fff7fffu); }
  __device__ __forceinline__ unsigned top() const {
    const uint32_t m = max_u16x2(top2(0), top2(2));
    return max(m << 16, m & 0xffff0000u);
  }
};
template <>
struct Dims<float> {
  float f[8];
  __device__ __forceinline__ void load(const float* p) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  __device__ __forceinline__ void get(float (&g)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = f[i];
  }
  __device__ __forceinline__ unsigned top4(int i) const {
    unsigned m = 0u;
#pragma unroll
    for (int j = 0; j < 4; ++j) m = max(m, __float_as_uint(f[i + j]) & 0x7fffffffu);
    return m;
  }
  __device__ __forceinline__ unsigned top() const { return max(top4(0), top4(4)); }
};
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

constexpr float kSeventh = 0.142857149f;
// Groups this small (2^-110: the reciprocal of their scale would overflow) are stored as zeros.
constexpr unsigned kTinyBits = 0x08800000u;
constexpr unsigned kInfBits = 0x7f800000u;
__device__ __forceinline__ bool odd_group(unsigned top) { return top - kTinyBits >= kInfBits - kTinyBits; }
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float bf16_of(float x) { return __bfloat162float(__float2bfloat16_rn(x)); }

// Rounding by the sum with 1.5 * 2^23 + 8: the float's bits are kMagicBits + n + 8.  |x / s| stays below 7.04 (the
// scale is off by 2^-8 at most), so n needs no clamp.
constexpr float kMagic = 12582920.f;
constexpr unsigned kMagicBits = 0x4b400000u;
// Word of 8 codes out of such bits: their sum times 16^i, less the constants' (modulo 2^32).
__device__ __forceinline__ unsigned pack_codes(const float (&t)[8]) {
  unsigned w = __float_as_uint(t[7]);
#pragma unroll
  for (int i = 6; i >= 0; --i) w = w * 16u + __float_as_uint(t[i]);
  return w - kMagicBits * 0x11111111u;
}
// The codes of 4 bf16 values under s: the quotient with one correction is exact where it is a tie (8 bits by 8
// bits: other quotients are 2^-17 away from one), so the sum rounds as the definition does.
__device__ __forceinline__ void round4(const float* x, float s, float inv, float* t) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float q = x[i] * inv;
    t[i] = fmaf(fmaf(-q, s, x[i]), inv, q) + kMagic;
  }
}

// ---- the exact way
// Scale of a group with largest magnitude x (float or double, >= 0; NaN above infinity): bf16(x / 7), ties to even.  The
// bf16 at or next below is found by a product; the border above that has 9 significant bits, so 7
// times it is exact and decides.
template <typename F>
__device__ float exact_scale(F x) {
  if (!(x <= (F)3.4028235e38f)) return __uint_as_float(0x7fc00000u);
  if (x < (F)__uint_as_float(kTinyBits)) return 0.f;
  const unsigned u = __float_as_uint((float)x * kSeventh) & 0xffff0000u;
  const F border7 = (F)__uint_as_float(u | 0x8000u) * (F)7;
  const bool up = x > border7 || (x == border7 && (u & 0x10000u));
  return __uint_as_float(up ? u + 0x10000u : u);
}
template <typename F>
__device__ __forceinline__ F shfl_max(unsigned mask, F v, int o) {
  const F w = __shfl_xor_sync(mask, v, o);
  return max(w, v);
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

// PAIR: where the partner of a dim is.
constexpr int kNone = 0;      // no rotation
constexpr int kInLane = 1;    // interleaved pairs: beside it
constexpr int kWhole = 2;     // halves of the whole head: in the lane's other 8 dims
constexpr int kFetch = 3;     // halves of a part of the head: loaded again

struct RowPair {
  const void* k;        // the head's key row and value row
  const void* v;
  unsigned char* block;
  int r;                // row in the block
  int e;                // the lane's place, 0..7
  unsigned mask;        // the row's lanes
  double pos;
};

__device__ __forceinline__ void store_scales(const RowPair& R, float ks, float vs0, float vs1) {
  // K group g in lane g; V groups 0, 1 in lane 0 and 2, 3 in lane 1
  unsigned char* const sc = R.block + 2 * kBlockTok * kRow4 + R.r * 16;
  if (R.e < 4) reinterpret_cast<unsigned short*>(sc)[R.e] = (unsigned short)(__float_as_uint(ks) >> 16);
  if (R.e < 2) reinterpret_cast<unsigned*>(sc + 8)[R.e] = (__float_as_uint(vs0) >> 16) | (__float_as_uint(vs1) & 0xffff0000u);
}

// Codes of 8 values under s: the quotient in 64 bits, corrected once, is an exact tie where there is one and far enough
// from one elsewhere (24 bits by 8), or known to 64 bits (rotated values).  8 everywhere where s is 0 or NaN.
__device__ __forceinline__ unsigned exact_codes(const double* z, float s0, float s1) {
  unsigned w = 0u;
  const double i0 = 1.0 / (double)s0, i1 = 1.0 / (double)s1;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const double s = (double)(i < 4 ? s0 : s1), inv = i < 4 ? i0 : i1, q = z[i] * inv;
    const int n = s > 0.0 ? (int)rint(fma(fma(-q, s, z[i]), inv, q)) : 0;
    w |= (unsigned)(n + 8) << (4 * i);
  }
  return w;
}
// Rounds and stores a row pair by exact decisions.  Rarely called, and out of line: its registers are not the others'.
template <typename T, int PAIR>
__device__ __noinline__ void store_exact(const RowPair R, const RopeTab128& tab) {
  const T* k = static_cast<const T*>(R.k) + 8 * R.e;
  const T* v = static_cast<const T*>(R.v) + 8 * R.e;
  const int half = tab.rot / 2;
  const double inf = __longlong_as_double(0x7ff0000000000000ll);
  double z[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = (double)Elem<T>::get(k, (i & 7) + 64 * (i >> 3));
  if (PAIR == kWhole || PAIR == kInLane) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int i0 = PAIR == kWhole ? i : 2 * i, i1 = PAIR == kWhole ? i + 8 : 2 * i + 1;
      const int j = PAIR == kWhole ? 8 * R.e + i : 4 * R.e + (i & 3) + 32 * (i >> 2);
      if (j < half) {
        double s64, c64;
        sincospi(angle_pi(tab.f_pi[j], R.pos), &s64, &c64);
        c64 *= tab.mag;
        s64 *= tab.mag;
        const double x = (double)Elem<T>::get(k, (i0 & 7) + 64 * (i0 >> 3)), p = (double)Elem<T>::get(k, (i1 & 7) + 64 * (i1 >> 3));
        z[i0] = x * c64 - p * s64;
        z[i1] = x * s64 + p * c64;
      }
    }
  } else if (PAIR == kFetch) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int d = 8 * R.e + (i & 7) + 64 * (i >> 3);
      if (d < tab.rot) {
        double s64, c64;
        sincospi(angle_pi(tab.f_pi[d < half ? d : d - half], R.pos), &s64, &c64);
        const double p = (double)Elem<T>::get(static_cast<const T*>(R.k), d < half ? d + half : d - half);
        z[i] = z[i] * (c64 * tab.mag) + p * ((d < half ? -s64 : s64) * tab.mag);
      }
    }
  }
  double km = 0.0;
#pragma unroll
  for (int i = 0; i < 16; ++i) km = fabs(z[i]) <= 3.4028235e38 ? fmax(km, fabs(z[i])) : inf;   // once infinite, it stays
  km = shfl_max(R.mask, km, 4);
  const float ks = exact_scale(km);
#pragma unroll
  for (int h = 0; h < 2; ++h) reinterpret_cast<unsigned*>(R.block + R.r * kRow4)[R.e + 8 * h] = exact_codes(z + 8 * h, ks, ks);
  float m0 = 0.f, m1 = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    z[i] = (double)Elem<T>::get(v, (i & 7) + 64 * (i >> 3));
    float& m = (i & 4) ? m1 : m0;
    m = fabs(z[i]) <= 3.4028235e38 ? fmaxf(m, (float)fabs(z[i])) : INFINITY;
  }
#pragma unroll
  for (int o = 2; o <= 4; o <<= 1) {
    m0 = shfl_max(R.mask, m0, o);
    m1 = shfl_max(R.mask, m1, o);
  }
  const float vs0 = exact_scale(m0), vs1 = exact_scale(m1);
#pragma unroll
  for (int h = 0; h < 2; ++h)
    reinterpret_cast<unsigned*>(R.block + kBlockTok * kRow4 + R.r * kRow4)[R.e + 8 * h] = exact_codes(z + 8 * h, vs0, vs1);
  store_scales(R, ks, vs0, vs1);
}

// Whether the bf16 scale s of u = amax / 7 (float32) may be another for an amax that is off by err.
__device__ __forceinline__ bool scale_unsure(float u, float s, float err) {
  const float half_step = __uint_as_float((__float_as_uint(u) & 0x7f800000u) - (8u << 23));
  return !(fabsf(fabsf(u - s) - half_step) > fmaf(err, kSeventh, 2.5e-7f * u));
}
// Code bits of 8 values, and how far the quotients are from integers.
__device__ __forceinline__ void round8(const float (&y)[8], float i0, float i1, float (&t)[8], float& far) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float inv = i < 4 ? i0 : i1;
    t[i] = fmaf(y[i], inv, kMagic);
    far = fmaxf(far, fabsf(fmaf(y[i], inv, kMagic - t[i])));
  }
}

template <typename T, int FMT, int PAIR>
__global__ void __launch_bounds__(128, 4) k_page_append(const PagePool P, const AppendArgs a, const __grid_constant__ RopeTab128 tab) {
  const int lane = threadIdx.x & 31;
  RowPair R;
  R.e = lane & 7;
  R.mask = 0xffu << (lane & 24);
  const int64_t item = ((int64_t)blockIdx.x * 128 + threadIdx.x) >> 3;
  int hg, b, t;
  if (item >= (int64_t)a.B * a.T * a.head_groups) return;
  if (a.small) {   // 32-bit divisions where they suffice
    const unsigned tok = (unsigned)item / (unsigned)a.head_groups;
    hg = (int)((unsigned)item - tok * a.head_groups);
    b = (int)(tok / (unsigned)a.T);
    t = (int)(tok - (unsigned)b * a.T);
  } else {
    const int64_t tok = item / a.head_groups;
    hg = (int)(item - tok * a.head_groups);
    b = (int)(tok / a.T);
    t = (int)(tok - (int64_t)b * a.T);
  }
  if (t >= row_count(a.n_new, b, a.T, P.err)) return;
  const int64_t pos = a.start[b] + t;
  int blk;
  unsigned char* const page = page_of(P, b, pos, blk, R.r);
  if (!page) return;
  R.pos = (double)pos;
  const int half = tab.rot / 2;
  const float mag = (float)tab.mag;

  // cosines and sines: kInLane pairs 4 e + i of the first 8 dims and 32 further; kWhole pairs 8 e + i; kFetch each dim's
  constexpr int kAngles = PAIR == kNone ? 1 : PAIR == kFetch ? 16 : 8;
  float c[kAngles], sn[kAngles];
  if (PAIR != kNone) {
#pragma unroll
    for (int i = 0; i < kAngles; ++i) {
      const int j = PAIR == kInLane ? 4 * R.e + (i & 3) + 32 * (i >> 2) : PAIR == kWhole ? 8 * R.e + i : 8 * R.e + (i & 7) + 64 * (i >> 3);
      c[i] = 1.f;
      sn[i] = 0.f;
      if (PAIR == kFetch) {
        if (j < tab.rot) {
          rope_cs(tab.f_pi[j < half ? j : j - half], R.pos, mag, c[i], sn[i]);
          if (j < half) sn[i] = -sn[i];
        }
      } else if (PAIR == kWhole || j < half) {
        rope_cs(tab.f_pi[j], R.pos, mag, c[i], sn[i]);
      }
    }
  }
  const T* krow = static_cast<const T*>(a.k) + b * a.ks.b + t * a.ks.t;
  const T* vrow = static_cast<const T*>(a.v) + b * a.vs.b + t * a.vs.t;

  Dims<T> kn[2], vn[2];   // the next head's rows, under way while this one's are rounded
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    kn[h].load(krow + hg * a.ks.h + 8 * R.e + 64 * h);
    vn[h].load(vrow + hg * a.vs.h + 8 * R.e + 64 * h);
  }
  for (int g = hg; g < P.Hkv; g += a.head_groups) {
    const T* kh = krow + g * a.ks.h;
    const T* vh = vrow + g * a.vs.h;
    Dims<T> kd[2], vd[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      kd[h] = kn[h];
      vd[h] = vn[h];
      if (g + a.head_groups < P.Hkv) {
        kn[h].load(kh + a.head_groups * a.ks.h + 8 * R.e + 64 * h);
        vn[h].load(vh + a.head_groups * a.vs.h + 8 * R.e + 64 * h);
      }
    }
    float y[2][8];
    unsigned xtop = 0u;   // float bits of the largest |x| + |partner|
    {
      float x[2][8];
      kd[0].get(x[0]);
      kd[1].get(x[1]);
      const float top0 = __uint_as_float(FMT == kPageInt4 && PAIR != kNone ? kd[0].top() : 0u);
      const float top1 = __uint_as_float(FMT == kPageInt4 && PAIR != kNone ? kd[1].top() : 0u);
      if (PAIR == kNone) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          y[0][i] = x[0][i];
          y[1][i] = x[1][i];
        }
      } else if (PAIR == kWhole) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int j = i % kAngles;
          turn(x[0][i], x[1][i], c[j], sn[j], y[0][i], y[1][i]);
        }
        xtop = __float_as_uint(top0 + top1);
      } else if (PAIR == kInLane) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = (4 * h + i) % kAngles;
            // dims that do not turn stay out of it: their neighbours may be infinite
            const bool turns = 8 * R.e + 64 * h + 2 * i < tab.rot;
            const float u = x[h][2 * i], w = x[h][2 * i + 1];
            y[h][2 * i] = u;
            y[h][2 * i + 1] = w;
            if (turns) turn(u, w, c[j], sn[j], y[h][2 * i], y[h][2 * i + 1]);
          }
        xtop = max(__float_as_uint(top0 + top0), __float_as_uint(top1 + top1));
      } else {
        float most = 0.f;
        bool nan = false;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int d = 8 * R.e + i + 64 * h, j = (8 * h + i) % kAngles;
            y[h][i] = x[h][i];
            float sum = fabsf(x[h][i]);
            if (d < tab.rot) {
              const float p = Elem<T>::get(kh, d < half ? d + half : d - half);
              y[h][i] = fmaf(x[h][i], c[j], p * sn[j]);
              sum += fabsf(p);
            }
            nan = nan || !(sum <= 3.4028235e38f);
            most = fmaxf(most, sum);
          }
        xtop = nan ? 0x7fc00000u : __float_as_uint(most);
      }
    }
    R.block = page + (size_t)g * P.head_bytes + (size_t)blk * (FMT == kPageInt4 ? kBlockBytes4 : kBlockBytes16);
    float v[2][8];
    vd[0].get(v[0]);
    vd[1].get(v[1]);
    if (FMT == kPageBf16) {
      // the cache keeps 16 bits: one rounding of the float32 rotation
      unsigned char* const to = R.block + R.r * 256 + ((R.e ^ (R.r & 7)) << 4);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        *reinterpret_cast<uint4*>(to + 128 * h) = pack8(y[h]);
        *reinterpret_cast<uint4*>(to + kBlockTok * 256 + 128 * h) = pack8(v[h]);
      }
      continue;
    }
    // ---- K: the lane's 16 dims are of scale group e % 4, shared with lane e ^ 4.
    // V: dims 4 further are of the next group than 2 (e % 2), both shared with the lanes of e's parity.
    unsigned ktop, v0, v1;   // float bits of the groups' largest magnitudes
    if (PAIR == kNone) {
      ktop = max(kd[0].top(), kd[1].top());
    } else {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, fmaxf(fabsf(y[0][i]), fabsf(y[1][i])));
      ktop = __float_as_uint(m);
      xtop = shfl_max(R.mask, xtop, 4);
    }
    ktop = shfl_max(R.mask, ktop, 4);
    if constexpr (sizeof(T) == 2) {
      const uint32_t m0 = max_u16x2(vd[0].top2(0), vd[1].top2(0)), m1 = max_u16x2(vd[0].top2(2), vd[1].top2(2));
      uint32_t m = max_u16x2(__byte_perm(m0, m1, 0x5410), __byte_perm(m0, m1, 0x7632));   // group low, group high
#pragma unroll
      for (int o = 2; o <= 4; o <<= 1) m = max_u16x2(m, __shfl_xor_sync(R.mask, m, o));
      v0 = m << 16;
      v1 = m & 0xffff0000u;
    } else {
      v0 = max(vd[0].top4(0), vd[1].top4(0));
      v1 = max(vd[0].top4(4), vd[1].top4(4));
#pragma unroll
      for (int o = 2; o <= 4; o <<= 1) {
        v0 = shfl_max(R.mask, v0, o);
        v1 = shfl_max(R.mask, v1, o);
      }
    }
    bool unsure = odd_group(ktop) || odd_group(v0) || odd_group(v1);
    const float ku = __uint_as_float(ktop) * kSeventh, vu0 = __uint_as_float(v0) * kSeventh, vu1 = __uint_as_float(v1) * kSeventh;
    const float ks = bf16_of(ku), vs0 = bf16_of(vu0), vs1 = bf16_of(vu1);
    const float ki = rcp(ks), vi0 = rcp(vs0), vi1 = rcp(vs1);
    unsigned kw[2], vw[2];
    // bf16 rows as given: exact by round4 (and the scale of 8 bits likewise)
    if (sizeof(T) == 2 && PAIR == kNone) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float q[8];
        round4(y[h], ks, ki, q);
        round4(y[h] + 4, ks, ki, q + 4);
        kw[h] = pack_codes(q);
      }
    } else {
      // A rotated value is off by at most 3.5e-7 m (|x| + |partner|): cos and sin by 1.6e-7 (argument and function)
      // and 6e-8 (magnitude), the products and the sum by 6e-8 each.  NaN and infinity show here, too.
      const float err = PAIR == kNone ? 0.f : __uint_as_float(xtop) * (3.5e-7f * fmaxf(mag, 1.f));
      float far = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float q[8];
        round8(y[h], ki, ki, q, far);
        kw[h] = pack_codes(q);
      }
      // a border of a code's rounding, or of the scale's, within the error of the value and of the quotient
      unsure = unsure || !(0.5f - far > fmaf(err, ki, 2e-6f)) || scale_unsure(ku, ks, err);
    }
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float q[8];
        round4(v[h], vs0, vi0, q);
        round4(v[h] + 4, vs1, vi1, q + 4);
        vw[h] = pack_codes(q);
      }
    } else {
      float far = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float q[8];
        round8(v[h], vi0, vi1, q, far);
        vw[h] = pack_codes(q);
      }
      unsure = unsure || !(0.5f - far > 2e-6f) || scale_unsure(vu0, vs0, 0.f) || scale_unsure(vu1, vs1, 0.f);
    }
    if (__any_sync(R.mask, unsure)) {
      R.k = kh;
      R.v = vh;
      store_exact<T, PAIR>(R, tab);
      continue;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      reinterpret_cast<unsigned*>(R.block + R.r * kRow4)[R.e + 8 * h] = kw[h];
      reinterpret_cast<unsigned*>(R.block + kBlockTok * kRow4 + R.r * kRow4)[R.e + 8 * h] = vw[h];
    }
    store_scales(R, ks, vs0, vs1);
  }
}

// 4-bit word to 8 values n - 8 (exact small integers).
__device__ __forceinline__ void nibbles(unsigned w, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(0x4b000000u | ((w >> (4 * i)) & 15u)) - 8388616.f;
}

// 8 codes as bf16: 128 + n by its bits, less 136, times the scale (dims 0-3, dims 4-7): one rounding, of the exact product.
__device__ __forceinline__ uint4 expand_bf16(unsigned w, uint32_t s0, uint32_t s1) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {   // nibbles i and i + 4
    r[i] = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
    asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(r[i]) : "r"(0xc308c308u));   // -136
  }
  uint32_t o[4] = {__byte_perm(r[0], r[1], 0x5410), __byte_perm(r[2], r[3], 0x5410), __byte_perm(r[0], r[1], 0x7632),
                   __byte_perm(r[2], r[3], 0x7632)};
#pragma unroll
  for (int i = 0; i < 4; ++i) asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(o[i]) : "r"(i < 2 ? s0 : s1));
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// A warp takes 16 consecutive rows of one (sequence, head); a half-warp reads and writes whole
// rows, all 8 row pairs in flight together.  Bound by memory, the writes above all: 32K tokens of 8 heads, 4 bits to bf16,
// 172 MB in 30.4 us (5.7 TB/s, 0.86 of a copy; 33.7 us with the codes expanded in float32); 120K rows of 4 heads from
// bf16 pages, 307 MB in 50.5 us (0.93).
template <typename T, int FMT>
__global__ void __launch_bounds__(128) k_page_read(const PagePool P, const ReadArgs a) {
  const int lane = threadIdx.x & 31, e = lane & 15;
  const int64_t unit = ((int64_t)blockIdx.x * 128 + threadIdx.x) >> 5;
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
    if constexpr (FMT == kPageInt4 && sizeof(T) == 2) {
      const unsigned kg = (e & 2) ? sc[u].y : sc[u].x, vg = (e & 1) ? sc[u].w : sc[u].z;
      const uint32_t s = __byte_perm(kg, kg, (e & 1) ? 0x3232 : 0x1010);
      *reinterpret_cast<uint4*>(kd + i * a.ks.t + 8 * e) = expand_bf16(kw[u], s, s);
      *reinterpret_cast<uint4*>(vd + i * a.vs.t + 8 * e) =
          expand_bf16(vw[u], __byte_perm(vg, vg, 0x1010), __byte_perm(vg, vg, 0x3232));
      continue;
    }
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

__global__ void k_clear_bits(unsigned* word, unsigned bits) { atomicAnd(word, ~bits); }

template <typename T, int FMT>
cudaError_t append_go(const PagePool& pool, const AppendArgs& a, const RopeTab128& tab, unsigned blocks, cudaStream_t st) {
  if (tab.rot == 0) k_page_append<T, FMT, kNone><<<blocks, 128, 0, st>>>(pool, a, tab);
  else if (tab.interleaved) k_page_append<T, FMT, kInLane><<<blocks, 128, 0, st>>>(pool, a, tab);
  else if (tab.rot == kHeadDim) k_page_append<T, FMT, kWhole><<<blocks, 128, 0, st>>>(pool, a, tab);
  else k_page_append<T, FMT, kFetch><<<blocks, 128, 0, st>>>(pool, a, tab);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_page_append(const PagePool& pool, AppendArgs a, int dtype, int format, const RopeTab128& tab,
                               int num_sms, cudaStream_t st) {
  // A thread takes up to 8 heads of its token, fewer while the GPU would not be full.  us of 8 heads' append and read
  // with 8 heads a thread against one: 32K tokens 81 / 125, 4096 tokens 22.6 / 23.2 (this rule 20.5), 512
  // tokens 15.4 / 10.6, 16 tokens 10.1 / 6.3.  Equal shares of (4 tokens, head) units for 4 blocks an SM, in place of
  // this grid's last partial wave: 85 at 32K tokens, 33.2 against 34.4 at 10007.
  const int64_t toks = (int64_t)a.B * a.T;
  a.head_groups = (pool.Hkv + 7) / 8;
  while (a.head_groups < pool.Hkv && toks * a.head_groups * 8 < (int64_t)num_sms * 512) a.head_groups *= 2;
  if (a.head_groups > pool.Hkv) a.head_groups = pool.Hkv;
  const int64_t blocks = (toks * a.head_groups * 8 + 127) / 128;
  a.small = toks * a.head_groups < INT32_MAX;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  if (dtype == 0)
    return format == kPageInt4 ? append_go<__nv_bfloat16, kPageInt4>(pool, a, tab, (unsigned)blocks, st)
                               : append_go<__nv_bfloat16, kPageBf16>(pool, a, tab, (unsigned)blocks, st);
  return format == kPageInt4 ? append_go<float, kPageInt4>(pool, a, tab, (unsigned)blocks, st)
                             : append_go<float, kPageBf16>(pool, a, tab, (unsigned)blocks, st);
}

cudaError_t launch_clear_bits(unsigned* word, unsigned bits, cudaStream_t st) {
  k_clear_bits<<<1, 1, 0, st>>>(word, bits);
  return cudaGetLastError();
}

cudaError_t launch_page_read(const PagePool& pool, const ReadArgs& a, int dtype, int format, cudaStream_t st) {
  const int64_t units = (int64_t)a.B * pool.Hkv * ((a.T + 15) / 16);
  const int64_t blocks = (units * 32 + 127) / 128;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  const unsigned nb = (unsigned)blocks;
  if (dtype == 0) {
    if (format == kPageInt4) k_page_read<__nv_bfloat16, kPageInt4><<<nb, 128, 0, st>>>(pool, a);
    else k_page_read<__nv_bfloat16, kPageBf16><<<nb, 128, 0, st>>>(pool, a);
  } else {
    if (format == kPageInt4) k_page_read<float, kPageInt4><<<nb, 128, 0, st>>>(pool, a);
    else k_page_read<float, kPageBf16><<<nb, 128, 0, st>>>(pool, a);
  }
  return cudaGetLastError();
}

}  // namespace spa
