// Shared definitions of the rotary and paged-cache operators (not part of the public ABI).
#pragma once

#include "spa_internal.cuh"

namespace spa {

constexpr int kPageInt4 = 0;
constexpr int kPageBf16 = 1;
constexpr int kBlockTok = 16;                       // tokens of a block, the unit every page is made of
constexpr int kRow4 = 64;                           // bytes of a row's 4-bit codes (K or V)
constexpr int kBlockBytes4 = 2 * kBlockTok * kRow4 + kBlockTok * 16;   // codes K, codes V, 8 bf16 scales a token
constexpr int kBlockBytes16 = 2 * kBlockTok * kHeadDim * 2;
constexpr int kMaxPagedSlices = 4096;               // max_batch * n_kv_heads (row prefix of the attention in shared memory)
constexpr int kMaxRopePairs = 256;
constexpr int kMergeWords = 9 * 32 * 4;             // a warp's or CTA's attention state as lanes hold it: 32 sums, maximum and sum

// Device status bits of a paged cache (kErrSeqLen, kErrStartPos and kErrTimeout as for spa_handle).
constexpr unsigned kErrPage = 16u;    // block_table entry outside [0, n_pages)
constexpr unsigned kErrList = 32u;    // selected count or position out of range

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Rotation of a head's first rot dims.  f_pi: effective inverse frequencies / pi.  Passed to
// kernels by value, so that a table belongs to no device and a captured graph keeps its own.
template <int N>
struct RopeTab {
  int rot;            // 0: no rotation
  int interleaved;    // pairs (2i, 2i+1), else (i, i + rot / 2)
  double mag;         // multiplier of the rotated dims
  double f_pi[N];
};
using RopeTab128 = RopeTab<kHeadDim / 2>;
using RopeTabAny = RopeTab<kMaxRopePairs>;

// Angle pos * f reduced to units of pi in [-1, 1], in 64 bits: a float32 product would be off
// by a whole radian at position 2^24.  rint by the 1.5 * 2^52 constant (|t| < 2^51).
__device__ __forceinline__ double angle_pi(double f_pi, double pos) {
  const double t = __dmul_rn(pos, f_pi);
  const double big = 6755399441055744.0;
  const double k = __dadd_rn(__dadd_rn(__dmul_rn(t, 0.5), big), -big);
  return __fma_rn(-2.0, k, t);
}
__device__ __forceinline__ void rope_cs(double f_pi, double pos, float mag, float& c, float& s) {
  float sn, cs;
  sincospif((float)angle_pi(f_pi, pos), &sn, &cs);
  c = cs * mag;
  s = sn * mag;
}

// A pair turned: the same roundings wherever rows are rotated.
__device__ __forceinline__ void turn(float u, float v, float c, float s, float& a, float& b) {
  a = fmaf(u, c, -(v * s));
  b = fmaf(v, c, u * s);
}

// Strides of a [batch][token][head][128] tensor, in elements.
struct Strides3 {
  int64_t b, t, h;
};

// A paged pool: [n_pages][Hkv][blocks of a page][block bytes].
struct PagePool {
  unsigned char* pages;
  const int* table;        // [B][max_pages]
  int Hkv, n_pages, max_pages;
  int page_blocks;         // blocks of a page
  int page_size;           // tokens of a page
  int64_t head_bytes;      // page_blocks * block bytes
  unsigned* err;
};

struct AppendArgs {
  const void* k;
  const void* v;
  Strides3 ks, vs;
  const int64_t* start;
  const int64_t* n_new;    // optional
  int B, T;
  int head_groups;         // a thread takes the heads h, h + head_groups, ...
  int small;               // B * T * head_groups fits 31 bits
};

struct ReadArgs {
  void* k;
  void* v;
  Strides3 ks, vs;
  const int64_t* start;
  const int64_t* n_rows;   // optional
  int B, T;
};

struct PagedAttendArgs {
  PagePool pool;
  const void* q;           // [B][Hq][128]
  const int64_t* seq_lens;
  const int* list;         // optional [B * Hkv][list_stride]
  const int* list_count;   // with list
  int64_t list_stride;
  float* out;              // [B][Hq][128]
  float* lse;              // optional [B][Hq]
  float* part;             // [grid + n_slices][kMergeWords]
  unsigned* ticket;        // [n_slices], zero between calls
  int B, Hq, G, n_slices;
  int64_t cap;             // largest accepted length
  int q_f32;
  int n_sink, window;
  float scale_log2;
  unsigned by_heads;       // ceil(2^32 / Hkv), ceil(2^32 / page_blocks): the high word of a product divides
  unsigned by_blocks;      // slices (below 2^12) and blocks (below 2^20) exactly; unused for a divisor of 1
  unsigned char all_rows[kMaxKvHeads];   // the head attends every row
  unsigned char has_list[kMaxKvHeads];   // the head attends its list too
};

cudaError_t launch_rope(const void* x, void* y, Strides3 xs, Strides3 ys, const int64_t* start, const int64_t* positions,
                        int B, int T, int H, int d, int dtype, int transpose, const RopeTabAny& tab, cudaStream_t st);
cudaError_t launch_page_append(const PagePool& pool, AppendArgs a, int dtype, int format, const RopeTab128& tab,
                               int num_sms, cudaStream_t st);
cudaError_t launch_page_read(const PagePool& pool, const ReadArgs& a, int dtype, int format, cudaStream_t st);
cudaError_t launch_clear_bits(unsigned* word, unsigned bits, cudaStream_t st);
int page_attend_setup(int format);   // 0: the kernel cannot be resident
cudaError_t launch_page_attend(const PagedAttendArgs& a, int format, int grid, const RopeTab128& tab, cudaStream_t st);

}  // namespace spa
