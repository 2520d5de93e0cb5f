// Rotary positions: y = m R(pos) x on the first rot dims of every head, the others copied.
//
// R turns the pair (u, v) by the angle a = pos * f_i:  (u cos a - v sin a, u sin a + v cos a).  The
// gradient of x is the transposed map m R(pos)^T dy: the same kernel with sin a negated.
//
// Bound by memory: 2 elements moved for 3 flops (32K tokens of 40 heads in bf16: 671 MB in 102 us, 6.6 TB/s, the rate of
// a plain copy; 36 of 80 dims in float32, where one chunk width serves the whole row and 18 pairs allow 8 bytes: 47 MB
// in 12.7 us, 3.7 TB/s).  A thread owns one chunk of pairs of one
// token (16 bytes of each half, or 16 bytes of interleaved pairs), takes the cosines and
// sines of its pairs once and applies them to several heads, so the 64-bit angle and the
// sincos are paid once for up to kHeads rows.  The table travels with the launch, so it belongs to no
// device; its 256 pairs cost a small call no more than 128 or 64 would (5.3 to 5.7 us of the host and 2.74 of the GPU with each).
#include "spa_paged.cuh"

namespace spa {
namespace {

constexpr int kHeads = 8;   // heads a thread of a large call takes
constexpr int64_t kThreads = 16384;

template <typename T, int V>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16, 8> {
  uint4 w;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = w; }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_lo(u[i]);
      f[2 * i + 1] = bf16_hi(u[i]);
    }
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    w = make_uint4(u[0], u[1], u[2], u[3]);
  }
};
template <>
struct Chunk<__nv_bfloat16, 2> {
  uint32_t w;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = *reinterpret_cast<const uint32_t*>(p); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint32_t*>(p) = w; }
  __device__ __forceinline__ void get(float (&f)[2]) const {
    f[0] = bf16_lo(w);
    f[1] = bf16_hi(w);
  }
  __device__ __forceinline__ void set(const float (&f)[2]) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(f[0], f[1]);
    w = *reinterpret_cast<const uint32_t*>(&b);
  }
};
template <>
struct Chunk<__nv_bfloat16, 1> {
  __nv_bfloat16 w;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = *p; }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *p = w; }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = __bfloat162float(w); }
  __device__ __forceinline__ void set(const float (&f)[1]) { w = __float2bfloat16_rn(f[0]); }
};
template <>
struct Chunk<float, 4> {
  float4 w;
  __device__ __forceinline__ void load(const float* p) { w = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<float4*>(p) = w; }
  __device__ __forceinline__ void get(float (&f)[4]) const { f[0] = w.x; f[1] = w.y; f[2] = w.z; f[3] = w.w; }
  __device__ __forceinline__ void set(const float (&f)[4]) { w = make_float4(f[0], f[1], f[2], f[3]); }
};
template <>
struct Chunk<float, 2> {
  float2 w;
  __device__ __forceinline__ void load(const float* p) { w = *reinterpret_cast<const float2*>(p); }
  __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<float2*>(p) = w; }
  __device__ __forceinline__ void get(float (&f)[2]) const { f[0] = w.x; f[1] = w.y; }
  __device__ __forceinline__ void set(const float (&f)[2]) { w = make_float2(f[0], f[1]); }
};
template <>
struct Chunk<float, 1> {
  float w;
  __device__ __forceinline__ void load(const float* p) { w = *p; }
  __device__ __forceinline__ void store(float* p) const { *p = w; }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = w; }
  __device__ __forceinline__ void set(const float (&f)[1]) { w = f[0]; }
};

struct RopeArgs {
  const void* x;
  void* y;
  Strides3 xs, ys;
  const int64_t* start;       // [B], or
  const int64_t* positions;   // [B][T]
  int64_t items;              // B * T * head_groups * chunks of a row
  int T, H, d;
  int head_groups;
  int n_rot, n_copy;          // threads of a row whose chunks turn, and are copied
  float sign;                 // -1: transposed
};

// One item = (token, head group, chunk).  V elements of each half (half layout) or V
// consecutive elements = V / 2 pairs (interleaved); V = 1 serves pairs of any alignment
// (an interleaved pair is then two single loads).
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(256) k_rope(const RopeArgs a, const __grid_constant__ RopeTabAny tab) {
  constexpr int kPairs = INTER ? (V + 1) / 2 : V;   // pairs of a chunk
  const int64_t item = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (item >= a.items) return;
  const int per_row = a.n_rot + a.n_copy;
  int64_t q = item;
  int j, hg, t, b;
  if (a.items <= INT32_MAX) {   // 32-bit divisions where they suffice
    const unsigned u = (unsigned)item;
    const unsigned r = u / (unsigned)per_row;
    j = (int)(u - r * per_row);
    const unsigned r2 = r / (unsigned)a.head_groups;
    hg = (int)(r - r2 * a.head_groups);
    b = (int)(r2 / (unsigned)a.T);
    t = (int)(r2 - (unsigned)b * a.T);
  } else {
    j = (int)(q % per_row);
    q /= per_row;
    hg = (int)(q % a.head_groups);
    q /= a.head_groups;
    t = (int)(q % a.T);
    b = (int)(q / a.T);
  }
  const T* x = static_cast<const T*>(a.x) + b * a.xs.b + t * a.xs.t;
  T* y = static_cast<T*>(a.y) + b * a.ys.b + t * a.ys.t;

  // A chunk past the rotated dims goes the same way (a warp holds both kinds), its bits as they are.
  const bool turns = j < a.n_rot;
  float c[kPairs], s[kPairs];
#pragma unroll
  for (int i = 0; i < kPairs; ++i) c[i] = s[i] = 0.f;
  if (turns) {
    const double pos = (double)(a.positions ? a.positions[(int64_t)b * a.T + t] : a.start[b] + t);
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      rope_cs(tab.f_pi[j * kPairs + i], pos, (float)tab.mag, c[i], s[i]);
      s[i] *= a.sign;
    }
  }
  // offsets of the chunk's first and second load
  constexpr bool kTwo = !INTER || V == 1;
  int d0 = INTER ? (V == 1 ? 2 * j : j * V) : j * V;
  int d1 = INTER ? 2 * j + 1 : tab.rot / 2 + j * V;
  bool two = kTwo;
  if (!turns) {
    d0 = tab.rot + (j - a.n_rot) * (kTwo ? 2 * V : V);
    d1 = d0 + V;
    two = kTwo && d1 < a.d;
  }
  constexpr int U = 4;   // heads in flight
  const int64_t xstep = a.head_groups * a.xs.h, ystep = a.head_groups * a.ys.h;
  x += hg * a.xs.h;
  y += hg * a.ys.h;
  for (int h0 = hg; h0 < a.H; h0 += U * a.head_groups) {
    Chunk<T, V> p0[U], p1[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (h0 + u * a.head_groups < a.H) {
        p0[u].load(x + u * xstep + d0);
        if (two) p1[u].load(x + u * xstep + d1);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (h0 + u * a.head_groups < a.H) {
        if (turns) {
          float f0[V], f1[V];
          p0[u].get(f0);
          if (kTwo) {
            p1[u].get(f1);
#pragma unroll
            for (int i = 0; i < V; ++i) {
              const float u0 = f0[i], v0 = f1[i];
              turn(u0, v0, c[i], s[i], f0[i], f1[i]);
            }
            p1[u].set(f1);
          } else {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
              const float u0 = f0[2 * i], v0 = f0[2 * i + 1];
              turn(u0, v0, c[i], s[i], f0[2 * i], f0[2 * i + 1]);
            }
          }
          p0[u].set(f0);
        }
        p0[u].store(y + u * ystep + d0);
        if (two) p1[u].store(y + u * ystep + d1);
      }
    }
    x += U * xstep;
    y += U * ystep;
  }
}

template <typename T, int V>
cudaError_t go(RopeArgs a, int B, const RopeTabAny& tab, cudaStream_t st) {
  const bool inter = tab.interleaved != 0;
  a.n_rot = inter ? tab.rot / (V == 1 ? 2 : V) : tab.rot / 2 / V;
  const int two = inter && V > 1 ? 1 : 2;   // chunks a thread copies
  a.n_copy = ((a.d - tab.rot) / V + two - 1) / two;
  // Up to kHeads heads a thread, fewer while the threads are below kThreads.  us with one head a thread against
  // kHeads: 40 heads of bf16, 32K tokens 436 / 102, 1024 tokens 15.7 / 5.9; 16 tokens of 32 heads 3.1 / 4.6.
  // kThreads of 16K against 64K: 6.2 / 6.5 at 1024 tokens, 3.9 / 5.6 at 256.
  const int64_t per_group = (int64_t)B * a.T * (a.n_rot + a.n_copy);
  a.head_groups = (a.H + kHeads - 1) / kHeads;
  while (a.head_groups < a.H && per_group * a.head_groups < kThreads) a.head_groups *= 2;
  if (a.head_groups > a.H) a.head_groups = a.H;
  a.items = (int64_t)B * a.T * a.head_groups * (a.n_rot + a.n_copy);
  const int64_t blocks = (a.items + 255) / 256;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  if (tab.interleaved) k_rope<T, V, true><<<(unsigned)blocks, 256, 0, st>>>(a, tab);
  else k_rope<T, V, false><<<(unsigned)blocks, 256, 0, st>>>(a, tab);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const void* x, void* y, Strides3 xs, Strides3 ys, const int64_t* start, const int64_t* positions,
                        int B, int T, int H, int d, int dtype, int transpose, const RopeTabAny& tab, cudaStream_t st) {
  RopeArgs a{};
  a.x = x;
  a.y = y;
  a.xs = xs;
  a.ys = ys;
  a.start = start;
  a.positions = positions;
  a.T = T;
  a.H = H;
  a.d = d;
  a.sign = transpose ? -1.f : 1.f;
  // Widest chunk that every load and store of the call can take aligned.
  auto fits = [&](int v) {
    const int es = dtype == 0 ? 2 : 4;
    const uintptr_t bytes = (uintptr_t)v * es;
    const int part = tab.interleaved ? tab.rot : tab.rot / 2;
    if (part % v || d % v || (d - tab.rot) % v) return false;
    if ((uintptr_t)x % bytes || (uintptr_t)y % bytes) return false;
    for (int64_t s : {xs.b, xs.t, xs.h, ys.b, ys.t, ys.h})
      if (s % v) return false;
    return true;
  };
  if (dtype == 0) {
    if (fits(8)) return go<__nv_bfloat16, 8>(a, B, tab, st);
    if (fits(2)) return go<__nv_bfloat16, 2>(a, B, tab, st);
    return go<__nv_bfloat16, 1>(a, B, tab, st);
  }
  if (fits(4)) return go<float, 4>(a, B, tab, st);
  if (fits(2)) return go<float, 2>(a, B, tab, st);
  return go<float, 1>(a, B, tab, st);
}

}  // namespace spa
