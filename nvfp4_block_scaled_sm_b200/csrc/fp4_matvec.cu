// fp4_matvec.cu -- products of a few rows with weights held in 4 bits
// (MXFP4 and NVFP4): y[m, n] = sum_k x[m, k] w[n, k], for one weight and for
// the experts of a stack.
//
// Mathematics. An E2M1 code is exact in fp16, and so is its product with an
// E4M3 block scale (2 + 4 significant bits, 2^-10 .. 2688). A row x is brought
// to fp16 as well, 256 elements under one power of two: with E the exponent of
// their largest finite magnitude, the piece of a bf16 row is x 2^(15 - E), so
// every element of at least 2^-32 of that magnitude keeps all its eight bits;
// fp32 rows take three pieces (11 + 11 + 2 bits, the first x 2^(14 - E)). What
// the pieces leave is computed exactly (x minus the pieces); if any of it is not
// zero, another pass over the weights adds it, with a power of two for each 32
// elements, and so on: the products that are summed are those of x itself
// whatever its range. Sums of 16 to 256 products are formed by m16n8k16 MMAs
// (fp16 products exact, fp32 sums); the scales (MXFP4's E8M0, NVFP4's global
// one, the power of two of the piece) multiply them in fp32 as they are added
// to the row's fp32 accumulator.
//
// Tiling. A warp holds 16 weight rows; a CTA 128 rows (8 warps, two CTAs a
// multiprocessor, for up to 8 columns) or 256 (16 warps, for 16 or 32: the x
// pieces are made by each CTA, and more rows share them) of a share of K; up to
// 8 CTAs of a cluster take the shares of the same rows and send their sums to
// the CTA that puts a row out, which adds them up in rank order (the same bits
// every run). Codes arrive by 16-byte asynchronous copies in a ring of three
// stages a warp (256 codes of each of its rows a stage), each warp waiting for
// its own; the x pieces of the CTA's share are made in the order in which a lane
// feeds them to the MMA, while the first codes are on their way.
//
// What bounds it: instructions issued, then memory. With the MMAs and scales
// left out, 64 tokens' 512 rows against 64 experts' 2048 x 7168 (MXFP4, 500 MB)
// take 108 us, without x's pieces too 87 us (5.8 TB/s); all of it takes 198 us.
// One row against 100003 x 4096 takes 56 us (3.9 TB/s), against 4096 x 4096
// 6.9 us, of which 3.5 us are the start, the pieces of x and the exchange of sums.
// A row that spans too much for one pass costs the CTAs that meet it their share
// of the weight once more, and all their sums by groups: 8 rows against 7168 x 7168
// take 38.5 us for 14.3, one row 17 for 10.7.
// Tried and slower: 32 rows a warp with half the warps (the experts 228 us for
// 198), three CTAs of 80 registers (5 to 9 %). x's pieces made once by a kernel
// before, in a first version of this one: faster for the experts (64 tokens 210 us
// for 227), slower for single weights (8 rows against 7168 x 7168 21 us for 18);
// not taken up again since.
#include <type_traits>

#include "common.cuh"

namespace mxq {
namespace {

constexpr int kStageK = 256;              // codes of a row in one stage
constexpr int kStageGroups = 8;           // groups of 32 in one stage
constexpr int kRowPitch = 144;            // bytes of a row of codes in shared memory: 128 + 16
constexpr int kWarpTile = 16 * kRowPitch; // 16 rows; the pad keeps 8 rows x 4 words off each other's banks
constexpr int kMaxPasses = 32;            // each pass takes at least 11 bits of a range of 277

constexpr uint32_t kNarrow = 4;           // columns (rows of x times pieces) that stage_narrow takes

enum Fmt { kMx = 0, kNv = 1 };

struct MatvecArgs {
  const void* x;
  const uint8_t* w;
  const uint8_t* s;
  const float* g;           // NVFP4: global scales
  void* y;
  const int64_t* off;       // NULL: one weight, else E + 1 row offsets
  const int32_t* order;     // NULL, or the source of each row: order[r] / top_k
  int64_t ld_x;
  int64_t N, K;             // rows and columns of a weight
  int64_t M;                // rows of the product (all experts)
  int64_t x_rows;           // rows of x
  int64_t w_pitch, s_pitch; // bytes of a weight row's codes and scales
  int64_t w_expert, s_expert;
  uint32_t E;
  int32_t top_k;
  uint32_t stages;          // of K
  uint32_t split;           // CTAs that share K (the cluster)
  uint32_t share, longer;   // stages of a CTA's share; the first `longer` CTAs have one more
  uint32_t chunk;           // stages of x pieces in shared memory
  int64_t tiles;            // of weight rows
  uint32_t colw;            // columns held for one n-tile
  uint32_t red_at;          // the sums, behind the pieces
  uint32_t g_per;           // global scales of an expert: 1, or 2 (one per half)
  int swiglu;
  int out_bf16;
  uint32_t scale_align;     // scale rows start on boundaries of 16, 4 or 1 bytes
};

__device__ __forceinline__ uint32_t smem_ptr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// Asynchronous copies to shared memory; where `bytes` is given, that many of
// the source are read and the rest of the destination is zero. The 16-byte
// form asks L2 for 256 bytes around it: a warp reads 128 bytes of a row in one
// stage and the next 128 in the following one.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 r;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
  return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
  return r;
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

// Four fp16 pairs of the eight E2M1 codes of a word, lowest byte first. The
// bytes are named within one asm statement: the conversion picks its byte of
// the register, where shifting them down first costs an instruction each.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{ .reg .b8 b0, b1, b2, b3; mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0; cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2; cvt.rn.f16x2.e2m1x2 %3, b3; }"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// c += A B for a 16 x 16 tile A (rows of weights) and a 16 x 8 tile B.
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// c = A B.
__device__ __forceinline__ void mma16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// NVFP4's global scale g = in(g) out(g), out a power of two: 1, or what keeps
// the products with in(g) inside fp32's range where g lies near its ends. The
// sums c of products that meet it are multiples of 2^-34 (2^-24 of a piece of x,
// 2^-10 of a code and block scale) below 2^36, so |g| in [2^-92, 2^92) leaves c g
// a finite normal number. Beyond, in(g) is in [2^56, 2^92), where a term of the
// result is 2^-103 at least, or in [2^-92, 2^-35), where the sum of 2^23 terms
// stays below 2^128; out(g) multiplies the finished sums.
__device__ __forceinline__ float global_out(float g) {
  const float m = fabsf(g);
  if (m >= 0x1p92f) return 0x1p36f;
  return m < 0x1p-92f && m > 0.f ? 0x1p-57f : 1.f;
}
__device__ __forceinline__ float global_in(float g) {
  const float out = global_out(g);
  return out == 1.f ? g : g * (out > 1.f ? 0x1p-36f : 0x1p57f);
}

__device__ __forceinline__ uint32_t cvt_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <typename XT>
struct Pieces;
template <>
struct Pieces<uint16_t> { static constexpr int n = 1, top = 15; };
template <>
struct Pieces<float> { static constexpr int n = 3, top = 14; };

// One fp16 piece of elements held 8 a lane, of a group of 32 (four
// neighbouring lanes) or, with COMMON, of the warp's 256: h = fp16(v m) with
// m = 2^(TOP - E), E the exponent of their largest finite magnitude; v becomes
// what the piece leaves (exact: h / m is a rounding of v to fewer bits). TOP
// is 15 for bf16 values (at most 65280 then) and 14 for fp32 ones, which 15
// could round up to 2^16, fp16's infinity. Infinities and NaNs go into the
// piece as they are and leave nothing. Returns 1 / m.
template <int TOP, bool COMMON>
__device__ __forceinline__ float take_piece(float (&v)[8], uint32_t (&h)[4]) {
  constexpr uint32_t kInf = 0x7f800000u;
  uint32_t top = 0;                               // bits of magnitudes order as they do
  bool odd = false;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const uint32_t b = __float_as_uint(v[i]) & 0x7fffffffu;
    odd |= b >= kInf;
    top = max(top, b);
  }
  if (odd) {
    top = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const uint32_t b = __float_as_uint(v[i]) & 0x7fffffffu;
      top = max(top, b < kInf ? b : 0u);
    }
  }
  if constexpr (COMMON) {
    top = __reduce_max_sync(kFull, top);
  } else {
    top = max(top, __shfl_xor_sync(kFull, top, 1));
    top = max(top, __shfl_xor_sync(kFull, top, 2));
  }
  const uint32_t mb = min(254u + TOP - (top >> 23), 254u);          // biased exponent of m
  const float m = __uint_as_float(mb << 23);
  const float inv = __uint_as_float(mb == 254 ? 0x00400000u : (254u - mb) << 23);
#pragma unroll
  for (int k = 0; k < 4; k++) {
    h[k] = cvt_f16x2(v[2 * k] * m, v[2 * k + 1] * m);
    const float2 f = f16x2_to_f32x2(h[k]);
    v[2 * k] = __fmaf_rn(-f.x, inv, v[2 * k]);
    v[2 * k + 1] = __fmaf_rn(-f.y, inv, v[2 * k + 1]);
  }
  if (odd) {                                      // inf - inf
#pragma unroll
    for (int i = 0; i < 8; i++)
      if ((__float_as_uint(v[i]) & kInf) == kInf) v[i] = 0.f;
  }
  return inv;
}

// The piece of a warp's 256 bf16 values (pairs, 8 a lane) under one scale,
// taken on the packed values: the largest and the smallest non-zero magnitude
// tell whether it holds all of them (an element of biased exponent e has its
// last bit at 2^(e - 134), the piece's last bit is 2^-24 / m with
// m = 2^(142 - E)). False if it does not; `odd` (and no piece) if there is an
// infinity.
__device__ __forceinline__ bool whole_piece(const uint32_t (&w)[4], uint32_t (&h)[4], float& inv, bool& odd) {
  const uint32_t am = absmax_bf16x2(absmax_bf16x2(w[0], w[1]), absmax_bf16x2(w[2], w[3])) & 0x7fff7fffu;
  const uint32_t top = __reduce_max_sync(kFull, max(am >> 16, am & 0xffffu));
  uint32_t low = 0xffffffffu;                     // smallest magnitude less one, zeros as 65535
#pragma unroll
  for (int k = 0; k < 4; k++) {
    uint32_t b = w[k] & 0x7fff7fffu;
    asm("{ .reg .b32 t; add.u16x2 t, %1, %2; min.u16x2 %0, %0, t; }" : "+r"(low) : "r"(b), "r"(0xffffffffu));
  }
  low = __reduce_min_sync(kFull, min(low >> 16, low & 0xffffu));
  const uint32_t E = top >> 7;
  const uint32_t mb = min(269u - E, 254u);        // biased exponent of m
  const float m = __uint_as_float(mb << 23);
  inv = __uint_as_float(mb == 254 ? 0x00400000u : (254u - mb) << 23);
#pragma unroll
  for (int k = 0; k < 4; k++) {
    const float2 f = mul_bf16x2_pow2(w[k], m);
    h[k] = cvt_f16x2(f.x, f.y);
  }
  odd = top >= 0x7f80u;
  return !odd && int(low) + 1 >= (int(E) - 32) * 128;
}

// The pieces of a warp's 256 elements under one scale each, as the first pass
// takes them; true (for all lanes) if they leave something.
template <typename XT>
__device__ __forceinline__ bool common_pieces(const In8<XT>& in, uint32_t (&h)[Pieces<XT>::n][4],
                                              float (&inv)[Pieces<XT>::n]) {
  bool odd = false;
  if constexpr (Pieces<XT>::n == 1) {
    if (whole_piece(in.w, h[0], inv[0], odd)) return false;
    if (!odd) return true;
  }
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; i++) v[i] = in[i];
#pragma unroll
  for (int p = 0; p < Pieces<XT>::n; p++) inv[p] = take_piece<Pieces<XT>::top, true>(v, h[p]);
  bool rest = false;
#pragma unroll
  for (int i = 0; i < 8; i++) rest |= v[i] != 0.f;
  return __any_sync(kFull, rest);
}

// The (expert, rows) pair number `slot` of the pairs that the row offsets
// make, TT rows at most in each: expert in *e, first row and row count; false
// if there are fewer. Offsets are clamped to [0, M], so no row outside the
// product is touched whatever they hold. One thread looks after one expert.
template <int W>
__device__ __forceinline__ bool find_slot(const MatvecArgs& a, uint32_t slot, uint32_t TT, int32_t* sh,
                                          uint32_t* e, int64_t* r0, uint32_t* m) {
  // sh: [0] result expert, [1] first row, [2] rows, [3 ..] warp totals (M and
  // every count of tiles are below 2^31)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) sh[2] = 0;
  uint32_t before = 0;
  for (uint32_t base = 0; base < a.E; base += W * 32) {
    const uint32_t i = base + tid;
    int32_t b = 0, n = 0;
    if (i < a.E) {
      b = int32_t(min(max(a.off[i], int64_t(0)), a.M));
      n = max(int32_t(min(max(a.off[i + 1], int64_t(0)), a.M)) - b, 0);
    }
    const uint32_t tiles = (uint32_t(n) + TT - 1) / TT;
    uint32_t incl = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += up;
    }
    if (base > 0) __syncthreads();                // the last totals are read
    if (lane == 31) sh[3 + warp] = int32_t(incl);
    __syncthreads();
    uint32_t first = before + incl - tiles;
#pragma unroll
    for (int w = 0; w < W; w++) {
      const uint32_t n_w = uint32_t(sh[3 + w]);
      first += w < warp ? n_w : 0;
      before += n_w;
    }
    if (slot >= first && slot < first + tiles) {
      const int32_t skip = int32_t((slot - first) * TT);
      sh[0] = int32_t(i);
      sh[1] = b + skip;
      sh[2] = min(n - skip, int32_t(TT));
    }
    if (before > slot) break;                     // the same for every thread
  }
  __syncthreads();
  *e = uint32_t(sh[0]);
  *r0 = sh[1];
  *m = uint32_t(sh[2]);
  return sh[2] > 0;
}

__device__ __forceinline__ void cluster_arrive_wait() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_map(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

// Scales are copied for two stages at a time (16 bytes of a row or more): two
// blocks of 16 rows a warp. A block is overwritten when the second one after it
// is begun, which is kRingStages - 1 stages ahead of the reader.
constexpr int kRingStages = 3;
template <int FMT>
struct ScaleBlock {
  static constexpr int stages = 2;
  static_assert(kRingStages - 1 <= stages, "two blocks do not cover the stages in flight");
  static constexpr int stage = FMT == kMx ? 8 : 16;              // bytes of a row in one stage
  static constexpr int row = stages * stage;
  static constexpr int bytes = 16 * row;
};

// One stage of a warp: 16 rows x 256 codes against the first NC of NT tiles of
// 8 columns. codes / scales: the stage's buffers of this warp; xf: the pieces
// of the stage's first group at this lane's place; sx: their scales at this
// lane's columns, sx_group bytes from group to group; even: all eight groups of
// a column have the same one (the first pass).
template <int FMT, int NC, int NA>
__device__ __forceinline__ void stage_math(float (&acc)[NA][4], uint32_t codes, uint32_t scales, uint32_t xf,
                                           uint32_t xf_group, uint32_t sx, uint32_t sx_group, bool even,
                                           const float (&global)[2], int lane) {
  constexpr int kRow = ScaleBlock<FMT>::row;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t rowA = codes + g * kRowPitch + t * 4, rowB = rowA + 8 * kRowPitch;
  float c[NC][4];
  if constexpr (FMT == kMx) {
    const uint2 sA = lds64(scales + g * kRow), sB = lds64(scales + (g + 8) * kRow);
    // every scale byte in [64, 191]: the fp32 products c 2^(s - 127) can
    // neither overflow nor leave the normal range, and the byte is the fp32
    // exponent field as it stands
    const uint32_t v = lds32(scales + (lane >> 1) * kRow + (lane & 1) * 4);
    const bool plain = ((v ^ (v << 1)) & 0x80808080u) == 0x80808080u;
    if (__all_sync(kFull, plain && even)) {
      float part[NC][4];
#pragma unroll
      for (int j = 0; j < kStageGroups; j++) {
        uint32_t hA[4], hB[4];
        codes_f16(lds32(rowA + j * 16), hA);
        codes_f16(lds32(rowB + j * 16), hB);
        const uint32_t wa = j < 4 ? sA.x : sA.y, wb = j < 4 ? sB.x : sB.y;
        const int sh = 23 - 8 * (j & 3);
        const float fA = __uint_as_float((sh >= 0 ? wa << (sh & 31) : wa >> 1) & 0x7f800000u);
        const float fB = __uint_as_float((sh >= 0 ? wb << (sh & 31) : wb >> 1) & 0x7f800000u);
#pragma unroll
        for (int n = 0; n < NC; n++) {
          const uint4 b = lds128(xf + j * xf_group + n * 512);
          mma16816_first(c[n], hA[0], hB[0], hA[1], hB[1], b.x, b.y);
          mma16816(c[n], hA[2], hB[2], hA[3], hB[3], b.z, b.w);
#pragma unroll
          for (int i = 0; i < 4; i++)
            part[n][i] = j == 0 ? c[n][i] * (i < 2 ? fA : fB) : __fmaf_rn(c[n][i], i < 2 ? fA : fB, part[n][i]);
        }
      }
#pragma unroll
      for (int n = 0; n < NC; n++) {
        const uint2 u = lds64(sx + n * 32);
#pragma unroll
        for (int i = 0; i < 4; i++)
          acc[n][i] = __fmaf_rn(part[n][i], __uint_as_float(i & 1 ? u.y : u.x), acc[n][i]);
      }
    } else {
      // pieces with a scale for each group, scales near the ends of the range,
      // and the NaN byte 255: the scaled sum is formed in fp64, where neither
      // factor order can overflow or underflow, and rounded once to fp32
#pragma unroll 1
      for (int j = 0; j < kStageGroups; j++) {
        uint32_t hA[4], hB[4];
        codes_f16(lds32(rowA + j * 16), hA);
        codes_f16(lds32(rowB + j * 16), hB);
        const uint32_t ba = ((j < 4 ? sA.x : sA.y) >> (8 * (j & 3))) & 255u;
        const uint32_t bb = ((j < 4 ? sB.x : sB.y) >> (8 * (j & 3))) & 255u;
        const double fA = double(pow2_dequant(ba)), fB = double(pow2_dequant(bb));
#pragma unroll
        for (int n = 0; n < NC; n++) {
          const uint4 b = lds128(xf + j * xf_group + n * 512);
          const uint2 u = lds64(sx + j * sx_group + n * 32);
          mma16816_first(c[n], hA[0], hB[0], hA[1], hB[1], b.x, b.y);
          mma16816(c[n], hA[2], hB[2], hA[3], hB[3], b.z, b.w);
#pragma unroll
          for (int i = 0; i < 4; i++)
            acc[n][i] += float(double(c[n][i]) * (i < 2 ? fA : fB) * double(__uint_as_float(i & 1 ? u.y : u.x)));
        }
      }
    }
  } else {
    // 16 block scales of each row; this lane's codes of group j lie in block
    // 2j + t / 2, whose byte is doubled into an fp16 pair
    const uint4 sA = lds128(scales + g * kRow), sB = lds128(scales + (g + 8) * kRow);
    const uint32_t pick = (t >> 1) * 0x11u;
    auto weights = [&](int j, uint32_t (&hA)[4], uint32_t (&hB)[4]) {
      codes_f16(lds32(rowA + j * 16), hA);
      codes_f16(lds32(rowB + j * 16), hB);
      const uint32_t wa = j < 2 ? sA.x : j < 4 ? sA.y : j < 6 ? sA.z : sA.w;
      const uint32_t wb = j < 2 ? sB.x : j < 4 ? sB.y : j < 6 ? sB.z : sB.w;
      const uint32_t sel = pick + ((j & 1) ? 0x22u : 0u);
      const uint32_t fA = cvt_f16x2_from_e4m3x2(__byte_perm(wa, 0, sel));
      const uint32_t fB = cvt_f16x2_from_e4m3x2(__byte_perm(wb, 0, sel));
#pragma unroll
      for (int k = 0; k < 4; k++) {
        hA[k] = mul_f16x2(hA[k], fA);
        hB[k] = mul_f16x2(hB[k], fB);
      }
    };
    auto add = [&](int j) {
#pragma unroll
      for (int n = 0; n < NC; n++) {
        const uint2 u = lds64(sx + j * sx_group + n * 32);
#pragma unroll
        for (int i = 0; i < 4; i++)
          acc[n][i] = __fmaf_rn(c[n][i] * global[i >> 1], __uint_as_float(i & 1 ? u.y : u.x), acc[n][i]);
      }
    };
    if (even) {                                   // the stage's 256 products are one sum
#pragma unroll
      for (int j = 0; j < kStageGroups; j++) {
        uint32_t hA[4], hB[4];
        weights(j, hA, hB);
#pragma unroll
        for (int n = 0; n < NC; n++) {
          const uint4 b = lds128(xf + j * xf_group + n * 512);
          if (j == 0) mma16816_first(c[n], hA[0], hB[0], hA[1], hB[1], b.x, b.y);
          else mma16816(c[n], hA[0], hB[0], hA[1], hB[1], b.x, b.y);
          mma16816(c[n], hA[2], hB[2], hA[3], hB[3], b.z, b.w);
        }
      }
      add(0);
    } else {
#pragma unroll 1
      for (int j = 0; j < kStageGroups; j++) {
        uint32_t hA[4], hB[4];
        weights(j, hA, hB);
#pragma unroll
        for (int n = 0; n < NC; n++) {
          const uint4 b = lds128(xf + j * xf_group + n * 512);
          mma16816_first(c[n], hA[0], hB[0], hA[1], hB[1], b.x, b.y);
          mma16816(c[n], hA[2], hB[2], hA[3], hB[3], b.z, b.w);
        }
        add(j);
      }
    }
  }
}

// Products of one MMA chain with its scales: acc += c f s, f the blocks' scales
// of rows g (0, 1) and g + 8 (2, 3), s the pieces'.
__device__ __forceinline__ void add_scaled(float (&acc)[4], const float (&c)[4], const float (&f)[4], float s0,
                                           float s1) {
#pragma unroll
  for (int i = 0; i < 4; i++) acc[i] = __fmaf_rn(c[i] * f[i], i & 1 ? s1 : s0, acc[i]);
}

// The same for a few columns (rows of x times pieces), where the MMA's eight
// columns keep apart what the scales keep apart: lane t of four takes a whole
// block of codes (32 with one MXFP4 scale, 16 with one NVFP4 scale) into its
// places of K, and a column of B holds x at the places of one lane only; all
// its other elements are zeros (lanes read them from shared memory as well).
// The sum of four blocks is then one chain of MMAs, and each lane scales four
// sums of blocks, where stage_math scales four sums of every group: about half
// the instructions, for MMAs that are mostly zeros.
//   COLS == 1: column n of B is block n of eight.
//   else     : column n of B is block n % 4 of four, for x's column n / 4; NC
//              tiles of B for x's columns 2n and 2n + 1.
// acc[n][i]: row g (i < 2) or g + 8. x0: x's pieces of this stage's first
// group; zero: a place of zeros.
template <int FMT, int COLS, int NA>
__device__ __forceinline__ void stage_narrow(float (&acc)[NA][4], uint32_t codes, uint32_t scales, uint32_t x0,
                                             uint32_t x_group, uint32_t zero, uint32_t sx, uint32_t sx_group,
                                             const float (&global)[2], int lane) {
  constexpr int kRow = ScaleBlock<FMT>::row;
  constexpr int NC = COLS <= 2 ? 1 : 2;
  const int g = lane >> 2, t = lane & 3;
  const bool diagonal = (g & 3) == t;
  const uint32_t xcol = COLS == 1 ? 0 : (g >> 2) * 64;
  float c[NC][4];
  if constexpr (FMT == kMx) {
    const uint2 sA = lds64(scales + g * kRow), sB = lds64(scales + (g + 8) * kRow);
    const uint32_t v = lds32(scales + (lane >> 1) * kRow + (lane & 1) * 4);
    const bool plain = __all_sync(kFull, ((v ^ (v << 1)) & 0x80808080u) == 0x80808080u);
    const int shift = 16 * (t & 1);
    // one or two sums of blocks: this lane's are group gi and gi + 1 of the stage
    auto scale = [&](uint32_t wa, uint32_t wb, int gi) {
      const uint32_t a2 = wa >> shift, b2 = wb >> shift;
      if (plain) {
        const float f[4] = {__uint_as_float((a2 << 23) & 0x7f800000u), __uint_as_float((a2 << 15) & 0x7f800000u),
                            __uint_as_float((b2 << 23) & 0x7f800000u), __uint_as_float((b2 << 15) & 0x7f800000u)};
#pragma unroll
        for (int n = 0; n < NC; n++) {
          const uint32_t at = sx + gi * sx_group + (COLS == 1 ? 0 : n * 8 + (t >> 1) * 4);
          add_scaled(acc[n], c[n], f, __uint_as_float(lds32(at)), __uint_as_float(lds32(at + sx_group)));
        }
      } else {                                    // as in stage_math
        const double f[4] = {double(pow2_dequant(a2 & 255u)), double(pow2_dequant((a2 >> 8) & 255u)),
                             double(pow2_dequant(b2 & 255u)), double(pow2_dequant((b2 >> 8) & 255u))};
#pragma unroll
        for (int n = 0; n < NC; n++) {
          const uint32_t at = sx + gi * sx_group + (COLS == 1 ? 0 : n * 8 + (t >> 1) * 4);
          const double s0 = double(__uint_as_float(lds32(at))), s1 = double(__uint_as_float(lds32(at + sx_group)));
#pragma unroll
          for (int i = 0; i < 4; i++) acc[n][i] += float(double(c[n][i]) * f[i] * (i & 1 ? s1 : s0));
        }
      }
    };
#pragma unroll
    for (int b = 0; b < 2; b++) {
      // rows of 128 bytes; odd rows have their halves exchanged, so that two
      // rows' 64 bytes fall on all banks
      const uint32_t row = codes + g * 128 + ((b ^ (g & 1)) * 64) + t * 16;
      const uint4 wA = lds128(row), wB = lds128(row + 8 * 128);
      const bool on = diagonal && (COLS > 1 || (g >> 2) == b);
      const uint32_t xb = on ? x0 + (4 * b + t) * x_group + xcol : zero;
#pragma unroll
      for (int r = 0; r < 4; r++) {
        uint32_t hA[4], hB[4];
        codes_f16(r == 0 ? wA.x : r == 1 ? wA.y : r == 2 ? wA.z : wA.w, hA);
        codes_f16(r == 0 ? wB.x : r == 1 ? wB.y : r == 2 ? wB.z : wB.w, hB);
#pragma unroll
        for (int n = 0; n < NC; n++) {
          const uint4 x = lds128(xb + n * 128 + r * 16);
          if (r == 0 && (COLS > 1 || b == 0)) mma16816_first(c[n], hA[0], hB[0], hA[1], hB[1], x.x, x.y);
          else mma16816(c[n], hA[0], hB[0], hA[1], hB[1], x.x, x.y);
          mma16816(c[n], hA[2], hB[2], hA[3], hB[3], x.z, x.w);
        }
      }
      if constexpr (COLS > 1) scale(b ? sA.y : sA.x, b ? sB.y : sB.x, 4 * b + 2 * (t & 1));
    }
    if constexpr (COLS == 1) scale(t < 2 ? sA.x : sA.y, t < 2 ? sB.x : sB.y, 2 * t);
  } else {
    const uint4 sA = lds128(scales + g * kRow), sB = lds128(scales + (g + 8) * kRow);
    const int shift = 16 * (t & 1);
    // this lane's two blocks are those of one group, gi of the stage
    auto scale = [&](uint32_t wa, uint32_t wb, int gi) {
      const float2 fA = f16x2_to_f32x2(cvt_f16x2_from_e4m3x2(wa >> shift));
      const float2 fB = f16x2_to_f32x2(cvt_f16x2_from_e4m3x2(wb >> shift));
      const float f[4] = {fA.x * global[0], fA.y * global[0], fB.x * global[1], fB.y * global[1]};
#pragma unroll
      for (int n = 0; n < NC; n++) {
        const float s = __uint_as_float(lds32(sx + gi * sx_group + (COLS == 1 ? 0 : n * 8 + (t >> 1) * 4)));
        add_scaled(acc[n], c[n], f, s, s);
      }
    };
#pragma unroll
    for (int q = 0; q < 4; q++) {
      // 32 bytes of four rows on all banks
      const uint32_t row = codes + g * 128 + ((q ^ (g & 3)) * 32) + t * 8;
      const uint2 wA = lds64(row), wB = lds64(row + 8 * 128);
      const bool on = diagonal && (COLS > 1 || (g >> 2) == (q & 1));
      const uint32_t xb = on ? x0 + (2 * q + (t >> 1)) * x_group + (t & 1) * 32 + xcol : zero;
#pragma unroll
      for (int r = 0; r < 2; r++) {
        uint32_t hA[4], hB[4];
        codes_f16(r == 0 ? wA.x : wA.y, hA);
        codes_f16(r == 0 ? wB.x : wB.y, hB);
#pragma unroll
        for (int n = 0; n < NC; n++) {
          const uint4 x = lds128(xb + n * 128 + r * 16);
          if (r == 0 && (COLS > 1 || q % 2 == 0)) mma16816_first(c[n], hA[0], hB[0], hA[1], hB[1], x.x, x.y);
          else mma16816(c[n], hA[0], hB[0], hA[1], hB[1], x.x, x.y);
          mma16816(c[n], hA[2], hB[2], hA[3], hB[3], x.z, x.w);
        }
      }
      if constexpr (COLS > 1) {
        scale(q == 0 ? sA.x : q == 1 ? sA.y : q == 2 ? sA.z : sA.w,
              q == 0 ? sB.x : q == 1 ? sB.y : q == 2 ? sB.z : sB.w, 2 * q + (t & 1));
      } else if (q % 2 == 1) {
        scale(q == 1 ? (t < 2 ? sA.x : sA.y) : (t < 2 ? sA.z : sA.w),
              q == 1 ? (t < 2 ? sB.x : sB.y) : (t < 2 ? sB.z : sB.w), 2 * (q - 1) + t);
      }
    }
  }
}

// Bytes of the warps' rings of stages of codes and two blocks of scales.
template <int FMT, int W>
struct Ring {
  static constexpr int warp = kRingStages * kWarpTile + 2 * ScaleBlock<FMT>::bytes;
  static constexpr int bytes = W * warp;
};

// The copies of a stage whose rows or columns are not all there, kept out of
// the loop's code: `bytes` of each row that exists, zeros for the rest.
template <bool A16, int COPIES>
__device__ __noinline__ void copy_codes_edge(uint32_t dst, uint32_t step, uint32_t second, const uint8_t* pa,
                                             const uint8_t* pb, int64_t row_step, int rows_a, int rows_b,
                                             uint32_t bytes, const uint8_t* any) {
#pragma unroll 1
  for (int i = 0; i < COPIES; i++) {
    const uint32_t na = i < rows_a ? bytes : 0u, nb = i < rows_b ? bytes : 0u;
    if constexpr (A16) {
      cp_async16(dst, na ? pa : any, na);
      cp_async16(dst + second, nb ? pb : any, nb);
    } else {
      cp_async8(dst, na ? pa : any, na);
      cp_async8(dst + second, nb ? pb : any, nb);
    }
    dst += step;
    pa += row_step;
    pb += row_step;
  }
}

// 16 bytes of scales of which n exist (none if n <= 0), at a source on a
// boundary of `align` bytes; the rest is `none`.
__device__ __noinline__ void copy_scales_edge(uint32_t dst, const uint8_t* p, int n, uint32_t align, uint32_t none) {
#pragma unroll 1
  for (int w = 0; w < 4; w++) {
    if (n >= 4 * w + 4 && align >= 4) {
      cp_async4(dst + 4 * w, p + 4 * w);
    } else {
      uint32_t v = none;
      for (int b = 0; b < 4; b++)
        if (4 * w + b < n) v = (v & ~(255u << (8 * b))) | (uint32_t(p[4 * w + b]) << (8 * b));
      sts32(dst + 4 * w, v);
    }
  }
}

// silu(gate) up for gates far below zero: silu is a normal fp32 number down to
// about -90, where e^90 is none, and up may be large enough to bring back what
// lies far below. Kept out of the kernel's code: such gates are rare.
__device__ __noinline__ float swiglu_far(float gate, float up) {
  return float(double(gate) / (1.0 + exp(-double(gate))) * double(up));
}

template <int FMT, typename XT, int NT, bool A16, int W>
__global__ void __launch_bounds__(32 * W, W == 8 ? 2 : 1) fp4_matvec_kernel(const MatvecArgs a) {
  constexpr int kTileRows = 16 * W;
  constexpr int ST = kRingStages;
  constexpr int P = Pieces<XT>::n;
  constexpr uint32_t TT = 8 * NT / P;                  // rows of x in a tile
  using Scales = ScaleBlock<FMT>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int32_t found[3 + W];
  __shared__ const XT* source[TT];
  __shared__ __align__(128) uint32_t zeros[64];
  pdl_enter();

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // grid: x the shares of K (a cluster) of each (expert, rows) pair, y and z
  // the tiles of weight rows
  uint32_t rank, slot;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm("mov.u32 %0, %%clusterid.x;" : "=r"(slot));
  const int64_t tile = int64_t(blockIdx.z) * gridDim.y + blockIdx.y;
  if (tile >= a.tiles) return;                         // the same for the whole cluster
  uint32_t e = 0, m = 0;
  int64_t r0 = 0;
  if (a.off) {
    if (!find_slot<W>(a, slot, TT, found, &e, &r0, &m)) return;   // the same for the whole cluster
  } else {
    r0 = int64_t(slot) * TT;
    m = uint32_t(min(int64_t(TT), a.M - r0));
  }

  // every CTA of the cluster has to be there before its memory is written:
  // arrive now, wait before the sums are sent
  if (a.split > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  // the same for the whole cluster; rows on 8-byte boundaries are rare, and
  // left to the general form
  const bool narrow = A16 && m * P <= kNarrow;
  if (tid < 64) zeros[tid] = 0;                        // read after the barriers of the first chunk

  // ---- this warp's 16 weight rows: consecutive, or 8 of the gate half and
  // the 8 of the up half that meet them (rows 0-7 and 8-15 of the MMA tile, so
  // one lane ends up with both)
  const int64_t half = a.N / 2;
  const int64_t outs = a.swiglu ? half : a.N;
  const int64_t o0 = tile * (a.swiglu ? kTileRows / 2 : kTileRows);
  const uint8_t* const we = a.w + int64_t(e) * a.w_expert;
  const uint8_t* const se = a.s + int64_t(e) * a.s_expert;
  // sources by 32-bit distances from the first row of the CTA (K <= 2^23 keeps
  // them below 2^32): row r < 8 of the warp from baseA, row r + 8 from baseB
  const int64_t second = a.swiglu ? half : 8;
  const uint8_t* const baseA = we + o0 * a.w_pitch;
  const uint8_t* const baseB = baseA + second * a.w_pitch;
  const uint8_t* const scaleA = se + o0 * a.s_pitch;
  const uint8_t* const scaleB = scaleA + second * a.s_pitch;
  const uint32_t wrow = warp * (a.swiglu ? 8 : 16);
  const int64_t last = outs - (o0 + wrow);                          // outputs from the warp's first on
  const int64_t lastB = a.swiglu ? last : last - 8;                 // rows of the second eight

  const uint32_t ring = smem_ptr(smem) + warp * Ring<FMT, W>::warp;
  const uint32_t scale_ring = ring + ST * kWarpTile;
  const uint32_t s_begin = rank * a.share + min(rank, a.longer);
  const uint32_t s_end = s_begin + a.share + (rank < a.longer ? 1 : 0);

  // copies: 16 bytes a lane, 4 rows of 128 bytes an instruction (8 bytes and 2
  // rows where rows start on 8-byte boundaries only), rows 0-7 and 8-15 apart.
  // Rows in shared memory are 144 bytes apart for stage_math; for stage_narrow
  // 128 apart with their 64 or 32 bytes exchanged.
  constexpr int kLanes = A16 ? 8 : 16, kBytes = A16 ? 16 : 8, kStep = 32 / kLanes, kCopies = 8 / kStep;
  const int cr = lane / kLanes, cc = (lane % kLanes) * kBytes;
  const int flip = !narrow ? 0 : FMT == kMx ? (cr & 1) * 64 : (cr & 3) * 32;
  const uint32_t pitch = narrow ? 128 : kRowPitch;
  const uint32_t code_dst = ring + cr * pitch + (cc ^ flip);
  // stages and blocks of scales that need no check: all 16 rows there, whole
  const bool all_rows = last >= (a.swiglu ? 8 : 16);
  const uint32_t whole = all_rows ? uint32_t(a.w_pitch / (kStageK / 2)) : 0;
  const uint32_t whole_scales = all_rows && a.scale_align == 16 ? uint32_t(a.s_pitch / Scales::row) : 0;
  uint32_t from[kCopies];                                           // of the next stage to copy
  auto copy_codes = [&](uint32_t stage, uint32_t slot_at) {
    if (stage < whole) {
#pragma unroll
      for (int i = 0; i < kCopies; i++) {
        const uint32_t dst = code_dst + slot_at + i * kStep * pitch;
        if constexpr (A16) {
          cp_async16(dst, baseA + from[i]);
          cp_async16(dst + 8 * pitch, baseB + from[i]);
        } else {
          cp_async8(dst, baseA + from[i]);
          cp_async8(dst + 8 * pitch, baseB + from[i]);
        }
      }
    } else {
      const int64_t left = a.w_pitch - int64_t(stage) * (kStageK / 2) - cc;
      const int rows_a = last <= cr ? 0 : int(min((last - cr + kStep - 1) / kStep, int64_t(kCopies)));
      const int rows_b = lastB <= cr ? 0 : int(min((lastB - cr + kStep - 1) / kStep, int64_t(kCopies)));
      copy_codes_edge<A16, kCopies>(code_dst + slot_at, kStep * pitch, 8 * pitch, baseA + from[0],
                                    baseB + from[0], kStep * a.w_pitch, rows_a, rows_b,
                                    left >= kBytes ? kBytes : left > 0 ? uint32_t(left) : 0u, a.w);
    }
#pragma unroll
    for (int i = 0; i < kCopies; i++) from[i] += kStageK / 2;
  };

  // the scales of a block of stages, 16 bytes a lane
  constexpr int kSLanes = Scales::row / 16;                         // lanes of a row
  constexpr int kSCopies = (16 * kSLanes + 31) / 32;
  uint32_t sfrom[kSCopies];                                         // of the next block to copy
  auto copy_scales = [&](uint32_t block) {
#pragma unroll
    for (int i = 0; i < kSCopies; i++) {
      const int idx = lane + 32 * i, r = idx / kSLanes;
      if (16 * kSLanes >= 32 || lane < 16) {
        const uint32_t dst = scale_ring + (block & 1) * Scales::bytes + idx * 16;
        const uint8_t* const p = (r < 8 ? scaleA : scaleB) + sfrom[i];
        if (block < whole_scales) {
          cp_async16(dst, p);
        } else {
          const bool there = (r & 7) < (r < 8 ? last : lastB);
          const int64_t n = there ? a.s_pitch - (int64_t(block) * Scales::row + (idx % kSLanes) * 16) : 0;
          copy_scales_edge(dst, p, int(min(max(n, int64_t(0)), int64_t(16))), a.scale_align,
                           FMT == kMx ? 0x7f7f7f7fu : 0u);          // scale 1, or block scale 0
        }
      }
      sfrom[i] += Scales::row;
    }
  };
  auto rewind = [&](uint32_t stage) {
#pragma unroll
    for (int i = 0; i < kCopies; i++)
      from[i] = (wrow + cr + kStep * i) * uint32_t(a.w_pitch) + cc + stage * (kStageK / 2);
#pragma unroll
    for (int i = 0; i < kSCopies; i++) {
      const int idx = lane + 32 * i;
      sfrom[i] = (wrow + (idx / kSLanes & 7)) * uint32_t(a.s_pitch) + idx % kSLanes * 16 +
                 stage / Scales::stages * Scales::row;
    }
  };

  // ---- x pieces of a chunk of stages, in shared memory: [group][column][32]
  // fp16 and [group][8] scales of each n-tile
  const uint32_t xbase = smem_ptr(smem) + Ring<FMT, W>::bytes;
  const uint32_t gstride = NT == 1 ? a.colw * 64 : NT * 512;        // bytes of one group's pieces
  const uint32_t sbase = xbase + a.chunk * kStageGroups * gstride;
  const uint32_t sstride = NT == 1 ? a.colw * 4 : NT * 32;          // bytes of one group's scales
  if (uint32_t(tid) < m) {                                          // read after the barriers of the first chunk
    int64_t row = r0 + tid;
    if (a.order) {
      const int32_t pair = a.order[row];
      row = pair >= 0 && pair / a.top_k < a.x_rows ? pair / a.top_k : -1;
    }
    source[tid] = row < 0 ? nullptr : static_cast<const XT*>(a.x) + row * a.ld_x;
  }

  // Makes the pieces of n stages. A warp takes one stage of one row, 8 elements
  // a lane. The first pass takes pieces under one scale each; a further one
  // takes, with a scale for each group of 32, what those and the passes since
  // have left. Returns whether anything is left.
  const uint32_t piece_dst = xbase + (lane >> 2) * gstride + (lane & 3) * 16;
  const uint32_t scale_dst = sbase + (lane >> 2) * sstride;
  auto put = [&](uint32_t st, uint32_t col, const uint32_t (&h)[4], float inv) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(piece_dst + st * (kStageGroups * gstride) + col * 64),
                 "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]) : "memory");
    if ((lane & 3) == 0) sts32(scale_dst + st * (kStageGroups * sstride) + col * 4, __float_as_uint(inv));
  };
  auto stage_x = [&](uint32_t first, uint32_t n, int pass) -> bool {
    bool left = false;
    // units whose loads are in flight together: two of bf16 where other CTAs are
    // resident to hide them (the shorter code is worth 5 to 9 % there), else four
    constexpr int kAhead = (NT == 1 ? 2 : 4) / (P == 1 ? 1 : 2);
    const uint32_t k_end = uint32_t(a.K);
    uint32_t mi = 0, st = warp;                                     // row and stage; the next unit is W stages on
    while (st >= n) {
      st -= n;
      mi++;
    }
    while (mi < m) {
      In8<XT> in[kAhead];
      uint32_t mis[kAhead], sts[kAhead];
#pragma unroll
      for (int q = 0; q < kAhead; q++) {
        mis[q] = mi;
        sts[q] = st;
        if (mi < m) {
          const uint32_t k = (first + st) * kStageK + lane * 8;
          const XT* const row = source[mi];
          if (k < k_end && row) in[q].load(row + k); else in[q].zero();
        }
        st += W;
        while (st >= n) {
          st -= n;
          mi++;
        }
      }
      if (pass == 0) {
#pragma unroll
        for (int q = 0; q < kAhead; q++) {
          if (mis[q] >= m) break;
          uint32_t h[P][4];
          float inv[P];
          left |= common_pieces(in[q], h, inv);
#pragma unroll
          for (int p = 0; p < P; p++) put(sts[q], mis[q] * P + p, h[p], inv[p]);
        }
      } else {
#pragma unroll
        for (int q = 0; q < kAhead; q++) {
          if (mis[q] >= m) break;
          float v[8];
          uint32_t h[4];
#pragma unroll
          for (int i = 0; i < 8; i++) v[i] = in[q][i];
#pragma unroll 1
          for (int i = 0; i < P; i++) (void)take_piece<Pieces<XT>::top, true>(v, h);
#pragma unroll 1
          for (int i = 0; i < pass * P; i++) {
            const float inv = take_piece<Pieces<XT>::top, false>(v, h);
            if (i >= (pass - 1) * P) put(sts[q], mis[q] * P + i - (pass - 1) * P, h, inv);
          }
#pragma unroll
          for (int i = 0; i < 8; i++) left |= v[i] != 0.f;
        }
      }
    }
    return left;
  };

  const int g = lane >> 2, t = lane & 3;
  const uint32_t lane_x = (NT == 1 ? (min(uint32_t(g), a.colw - 1) * 4 + t) : uint32_t(lane)) * 16;
  const uint32_t zero = smem_ptr(zeros) + 32;                       // 32 past a multiple of 64: not x's banks

  // NVFP4's global scales of rows g and g + 8. They multiply the sums of a stage
  // (a group, in further passes) as these are added up: the products of x and
  // the block-scaled codes alone may lie up to 2688 * 448 times higher than the
  // result, out of fp32's range.
  auto global_scale = [&](int i) {
    const bool upper = a.swiglu ? i == 1 : o0 + wrow + g + 8 * i >= half;
    return a.g[int64_t(e) * a.g_per + (a.g_per == 2 && upper ? 1 : 0)];
  };
  float global[2] = {1.f, 1.f};
  bool far = false;                                                 // a scale near the ends of fp32's range
  if constexpr (FMT == kNv) {
#pragma unroll
    for (int i = 0; i < 2; i++) global[i] = global_scale(i);
  }

  constexpr int NA = NT < 2 ? 2 : NT;
  float acc[NA][4];
#pragma unroll
  for (int n = 0; n < NA; n++)
#pragma unroll
    for (int i = 0; i < 4; i++) acc[n][i] = 0.f;

  // The CTA's share of K: one way of taking a stage, chosen once. FORM < 0:
  // stage_narrow for -FORM columns; else stage_math for FORM n-tiles.
  auto sweep = [&](auto form_of) {
    constexpr int FORM = decltype(form_of)::value;
    for (int pass = 0; pass < kMaxPasses; pass++) {
      bool more = false;
      rewind(s_begin);
#pragma unroll
      for (int i = 0; i < ST - 1; i++) {
        if (s_begin + i < s_end) {
          if (i == 0 || (s_begin + i) % Scales::stages == 0) copy_scales((s_begin + i) / Scales::stages);
          copy_codes(s_begin + i, i * kWarpTile);
        }
        cp_commit();
      }
      uint32_t read = 0, fill = (ST - 1) * kWarpTile;               // slots of the ring
      for (uint32_t c_begin = s_begin; c_begin < s_end; c_begin += a.chunk) {
        const uint32_t n = min(a.chunk, s_end - c_begin);
        __syncthreads();                                            // the last chunk has been read
        const bool left = stage_x(c_begin, n, pass);
        more |= __syncthreads_or(left) != 0;
        if (FMT == kNv && pass == 0 && c_begin == s_begin) {        // (the scales' loads have come by now)
#pragma unroll
          for (int i = 0; i < 2; i++) {
            far |= global_out(global[i]) != 1.f;
            global[i] = global_in(global[i]);
          }
        }
        uint32_t xg = xbase, sg = sbase;
#pragma unroll 1
        for (uint32_t s = c_begin; s < c_begin + n; s++) {
          cp_wait<ST - 2>();
          __syncwarp();                                             // the stage is in; the one before is read
          const uint32_t ahead = s + ST - 1;
          if (ahead < s_end) {
            if (ahead % Scales::stages == 0) copy_scales(ahead / Scales::stages);
            copy_codes(ahead, fill);
          }
          cp_commit();
          const uint32_t codes = ring + read;
          const uint32_t scales =
              scale_ring + (s / Scales::stages & 1) * Scales::bytes + s % Scales::stages * Scales::stage;
          if constexpr (FORM < 0)
            stage_narrow<FMT, -FORM, NA>(acc, codes, scales, xg, gstride, zero, sg, sstride, global,
                                              lane);
          else
            stage_math<FMT, FORM, NA>(acc, codes, scales, xg + lane_x, gstride, sg + t * 8, sstride, pass == 0,
                                          global, lane);
          xg += kStageGroups * gstride;
          sg += kStageGroups * sstride;
          read = read == (ST - 1) * kWarpTile ? 0 : read + kWarpTile;
          fill = fill == (ST - 1) * kWarpTile ? 0 : fill + kWarpTile;
        }
      }
      if (!more) break;
      __syncthreads();
    }
  };
  const uint32_t cols = m * P, used = (cols + 7) / 8;               // n-tiles with columns
  if (narrow) {
    if (cols == 1) sweep(std::integral_constant<int, -1>{});
    else if (cols == 2) sweep(std::integral_constant<int, -2>{});
    else sweep(std::integral_constant<int, -4>{});
  } else if (NT == 1 || used == 1) {
    sweep(std::integral_constant<int, 1>{});
  } else if (NT == 2 || used == 2) {
    sweep(std::integral_constant<int, NT < 2 ? 1 : 2>{});
  } else {
    sweep(std::integral_constant<int, NT>{});
  }

  if (FMT == kNv && far) {
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const float out = global_out(global_scale(i));
#pragma unroll
      for (int n = 0; n < NA; n++) {
        acc[n][2 * i] *= out;
        acc[n][2 * i + 1] *= out;
      }
    }
  }

  // ---- sums of the cluster's shares: each CTA writes its sums of an output
  // row to the CTA that puts that row out, which adds up what came in rank order
  // once all have arrived (no CTA reads another's memory, so each is done then).
  // [rank][column][row of the slice], in memory that the rings do not use: other
  // CTAs may still be at work.
  const uint32_t per = a.swiglu ? kTileRows / 2 : kTileRows;        // outputs
  if (a.split > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  const uint32_t slice = (per + a.split - 1) / a.split;             // of a CTA
  const uint32_t rows_slice = a.swiglu ? 2 * slice : slice;         // weight rows of them
  const uint32_t red = xbase + a.red_at;
  auto send = [&](uint32_t col, uint32_t row, float v) {
    // rows 0-7 of each 16 are gate and 8-15 up rows with swiglu
    const uint32_t o = a.swiglu ? (row >> 4) * 8 + (row & 7) : row;
    const uint32_t to = o / slice, at = (o - to * slice) + (a.swiglu && (row & 8) ? slice : 0);
    uint32_t addr = red + ((rank * (8 * NT) + col) * rows_slice + at) * 4;
    if (a.split > 1) addr = cluster_map(addr, to);
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
  };
  if (narrow) {
#pragma unroll
    for (int n = 0; n < 2; n++) {
      float lo = acc[n][0] + acc[n][1], hi = acc[n][2] + acc[n][3];   // rows g and g + 8
      lo += __shfl_xor_sync(kFull, lo, 1);
      hi += __shfl_xor_sync(kFull, hi, 1);
      if (cols == 1) {
        lo += __shfl_xor_sync(kFull, lo, 2);
        hi += __shfl_xor_sync(kFull, hi, 2);
      }
      const uint32_t col = 2 * n + (t >> 1);
      if ((t & 1) == 0 && col < cols) {
        send(col, warp * 16 + g, lo);
        send(col, warp * 16 + g + 8, hi);
      }
    }
  } else {
#pragma unroll
    for (int n = 0; n < NT; n++) {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const uint32_t col = n * 8 + 2 * t + (i & 1);
        if (col < cols) send(col, warp * 16 + g + (i < 2 ? 0 : 8), acc[n][i]);
      }
    }
  }
  if (a.split > 1) cluster_arrive_wait(); else __syncthreads();

  const uint32_t lo = rank * slice, len = min(slice, per - min(per, lo));
  auto total = [&](uint32_t col, uint32_t at) -> float {
    float v = 0.f;
#pragma unroll
    for (int p = 0; p < P; p++)
      for (uint32_t q = 0; q < a.split; q++)
        v += __uint_as_float(lds32(red + ((q * (8 * NT) + col * P + p) * rows_slice + at) * 4));
    return v;
  };
  for (uint32_t i = tid; i < m * len; i += 32 * W) {
    const uint32_t mi = i / len, o = i % len;
    const int64_t out = o0 + lo + o;
    if (out >= outs) continue;
    float v;
    if (a.swiglu) {
      const float gate = total(mi, o), up = total(mi, slice + o);
      // silu(z) = z / (1 + e^-z); where e^-z nears fp32's largest value, in fp64
      v = gate < -80.f ? swiglu_far(gate, up) : gate / (1.f + expf(-gate)) * up;
    } else {
      v = total(mi, o);
    }
    const int64_t at = (r0 + mi) * outs + out;
    if (a.out_bf16)
      static_cast<uint16_t*>(a.y)[at] = uint16_t(cvt_bf16x2(v, 0.f));
    else
      static_cast<float*>(a.y)[at] = v;
  }
}

// y[t, n] = sum_j weights[t, j] rows[positions[t, j], n]: a token's rows added
// up in fp32 in the order of its choices (the same bits every run); a position
// outside [0, R) adds nothing. One thread holds VEC neighbouring outputs.
template <int VEC>
__global__ void __launch_bounds__(kThreads) moe_combine_kernel(const float* __restrict__ rows,
                                                               const int32_t* __restrict__ positions,
                                                               const float* __restrict__ weights, void* y,
                                                               int64_t R, int64_t T, int64_t N, int32_t top_k,
                                                               uint32_t col_blocks, int out_bf16) {
  pdl_enter();
  const int64_t t = blockIdx.x / col_blocks;
  const int64_t n = (int64_t(blockIdx.x % col_blocks) * kThreads + threadIdx.x) * VEC;
  if (n >= N) return;
  float v[VEC];
#pragma unroll
  for (int i = 0; i < VEC; i++) v[i] = 0.f;
  for (int32_t j = 0; j < top_k; j++) {
    const int64_t at = positions[t * top_k + j];
    if (at < 0 || at >= R) continue;
    const float w = weights[t * top_k + j];
    const float* p = rows + at * N + n;
    if constexpr (VEC == 4) {
      const uint4 q = ld_nc_v4(p);
      v[0] = __fmaf_rn(w, __uint_as_float(q.x), v[0]);
      v[1] = __fmaf_rn(w, __uint_as_float(q.y), v[1]);
      v[2] = __fmaf_rn(w, __uint_as_float(q.z), v[2]);
      v[3] = __fmaf_rn(w, __uint_as_float(q.w), v[3]);
    } else {
      v[0] = __fmaf_rn(w, *p, v[0]);
    }
  }
  const int64_t at = t * N + n;
  if constexpr (VEC == 4) {
    if (out_bf16)
      st_v2(static_cast<uint16_t*>(y) + at, make_uint2(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3])));
    else
      st_v4(static_cast<float*>(y) + at, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]),
                                                    __float_as_uint(v[2]), __float_as_uint(v[3])));
  } else if (out_bf16) {
    static_cast<uint16_t*>(y)[at] = uint16_t(cvt_bf16x2(v[0], 0.f));
  } else {
    static_cast<float*>(y)[at] = v[0];
  }
}

// ------------------------------------------------------------------ host


constexpr uint32_t kMostSplit = 8;        // the largest portable cluster

// Clusters of `split` CTAs of Kernel (with `threads` threads and `smem` bytes)
// that can be resident at once on the current device: fewer than the CTAs alone
// would allow, since a cluster stays within one GPC. Asked for once per device.
template <auto Kernel>
uint64_t resident_clusters(uint32_t split, uint32_t threads, uint32_t smem, uint64_t ctas) {
  static std::atomic<int> known[64][kMostSplit + 1];
  int dev = 0;
  const bool slot = cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < 64;
  int n = slot ? known[dev][split].load(std::memory_order_relaxed) : 0;
  if (n > 0) return uint64_t(n);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(split);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, Kernel, &cfg) != cudaSuccess || n <= 0) {
    (void)cudaGetLastError();
    return std::max<uint64_t>(1, ctas / split);
  }
  if (slot) known[dev][split].store(n, std::memory_order_relaxed);
  return uint64_t(n);
}

// How K is shared out: the split that takes least time by this estimate, in
// tenths of a stage of one CTA alone on its multiprocessor (1 us). Two CTAs
// beside one another take 1.2 times as long for a stage (measured on 8 experts'
// 2048 x 7168). A round of resident clusters has fixed work (x's pieces, the
// exchange of the sums) of about five stages, and up to four more where its CTAs
// go from one and a half a multiprocessor to two: 1 row against 7168 x 7168 takes
// 10.3 us with 224 CTAs and 12.1 with 280. Rounds are counted by clusters: 16
// rows against 5120 x 5120 take 12.4 us with shares of five CTAs and 20.8 with
// seven, of which fewer fit a GPC.
template <auto Kernel>
uint32_t choose_split(uint64_t units, uint32_t stages, uint32_t resident, uint32_t threads, uint32_t smem) {
  const uint64_t sms = uint64_t(sm_count());
  constexpr uint64_t kTogether[3] = {0, 10, 12};
  uint32_t best = 1;
  uint64_t best_cost = ~0ull;
  for (uint32_t c = 1; c <= kMostSplit && (c == 1 || c <= stages); c++) {
    const uint64_t share = (stages + c - 1) / c;
    const uint64_t most = c == 1 ? sms * resident : resident_clusters<Kernel>(c, threads, smem, sms * resident);
    const auto round = [&](uint64_t clusters) {
      const uint64_t ctas = clusters * c, beside = std::min<uint64_t>(resident, (ctas + sms - 1) / sms);
      const uint64_t crowded = 2 * ctas > 3 * sms ? (2 * ctas - 3 * sms) * 40 / sms : 0;
      return clusters ? share * kTogether[beside] + 50 + crowded : 0;
    };
    const uint64_t cost = units / most * round(most) + round(units % most);
    if (cost < best_cost) {
      best_cost = cost;
      best = c;
    }
  }
  return best;
}

template <int FMT, typename XT, int NT, bool A16>
mxq_status launch_matvec(MatvecArgs a, cudaStream_t stream) {
  // one n-tile: two CTAs of 8 warps a multiprocessor, 128 registers a thread
  // (three of 80 registers took 5 to 9 % more instructions and time); more: one
  // of 16 warps, whose 256 rows share the x pieces
  constexpr int W = NT == 1 ? 8 : 16;
  // the sums: a slice is rounded up, by one output (two weight rows) a CTA at
  // most
  constexpr uint32_t kSums = 8 * NT * (16 * W + 8 * 2) * 4;
  constexpr uint32_t P = Pieces<XT>::n;
  constexpr uint32_t TT = 8 * NT / P;
  const uint64_t tile_rows = a.swiglu ? 8 * W : 16 * W;
  const uint64_t tiles = (uint64_t(a.swiglu ? a.N / 2 : a.N) + tile_rows - 1) / tile_rows;
  uint64_t slots, likely;
  if (a.off) {
    // non-empty experts, and the tiles beyond their first
    const uint64_t n = std::min<uint64_t>(a.E, uint64_t(a.M));
    slots = n + (uint64_t(a.M) - n) / TT;
    likely = n;
  } else {
    slots = likely = (uint64_t(a.M) + TT - 1) / TT;
  }
  // columns in shared memory: those that the widest form reads, which are one,
  // two or four in stage_narrow and all eight of an n-tile in stage_math
  const uint64_t most = std::min<uint64_t>(TT, uint64_t(a.M)) * P;
  a.colw = NT == 1 && most <= kNarrow && A16 ? (most <= 2 ? uint32_t(most) : 4) : 8;
  constexpr uint32_t kMostSmem = NT == 1 ? 111u << 10 : 225u << 10;
  constexpr uint32_t kPieces = kMostSmem - Ring<FMT, W>::bytes - kSums;
  constexpr auto kernel = fp4_matvec_kernel<FMT, XT, NT, A16, W>;
  const cudaError_t attr_err = ensure_smem_limit<kernel>(int(kMostSmem));
  if (attr_err != cudaSuccess) {
    record_cuda_error(attr_err);
    return MXQ_ERR_CUDA;
  }
  a.split = choose_split<kernel>(likely * tiles, a.stages, NT == 1 ? 2 : 1, 32 * W, kMostSmem);
  if (slots * a.split > 0x7fffffffull) return MXQ_ERR_SHAPE;
  a.tiles = int64_t(tiles);
  a.share = a.stages / a.split;
  a.longer = a.stages % a.split;
  const uint32_t per_stage = kStageGroups * NT * a.colw * (64 + 4);
  const uint32_t share = a.share + (a.longer ? 1 : 0);
  a.chunk = std::max(1u, std::min(share, kPieces / per_stage));
  a.red_at = (a.chunk * per_stage + 15) / 16 * 16;
  const size_t smem = size_t(Ring<FMT, W>::bytes) + a.red_at + kSums;

  static_assert(kStageGroups * NT * 8 * (64 + 4) + 16 + kSums + Ring<FMT, W>::bytes <= kMostSmem,
                "a stage of pieces has to fit");
  cudaLaunchConfig_t cfg = {};
  const uint64_t ny = std::min<uint64_t>(tiles, 65535), nz = (tiles + ny - 1) / ny;
  if (nz > 65535) return MXQ_ERR_SHAPE;
  cfg.gridDim = dim3(uint32_t(slots) * a.split, uint32_t(ny), uint32_t(nz));
  cfg.blockDim = dim3(32 * W);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.split > 1 ? 2 : 1;
  return launched(cudaLaunchKernelEx(&cfg, kernel, a));
}

template <int FMT, typename XT, bool A16>
mxq_status launch_columns(const MatvecArgs& a, cudaStream_t stream) {
  // columns of the MMA that a tile of rows takes; an expert's rows vary, so
  // twice the average has to fit
  const uint64_t rows = a.off ? (2 * uint64_t(a.M) + a.E - 1) / a.E : uint64_t(a.M);
  const uint64_t cols = rows * Pieces<XT>::n;
  if (cols <= 8) return launch_matvec<FMT, XT, 1, A16>(a, stream);
  if (cols <= 16) return launch_matvec<FMT, XT, 2, A16>(a, stream);
  return launch_matvec<FMT, XT, 4, A16>(a, stream);
}

template <int FMT>
mxq_status launch_fp4(const MatvecArgs& a, int dt, cudaStream_t stream) {
  if constexpr (FMT == kNv) {
    if (a.w_pitch % 16 != 0)
      return dt == MXQ_BF16 ? launch_columns<FMT, uint16_t, false>(a, stream)
                            : launch_columns<FMT, float, false>(a, stream);
  }
  return dt == MXQ_BF16 ? launch_columns<FMT, uint16_t, true>(a, stream)
                        : launch_columns<FMT, float, true>(a, stream);
}

struct Call {
  const void* x;
  int dt;
  int64_t x_rows, K, ld_x;
  const uint8_t* packed;
  const uint8_t* scale;
  const float* g;
  int64_t N;
  void* y;
  int out_dt;
};

constexpr int64_t kMostRows = 0x7fffffff, kMostK = 1 << 23;

// The checks that one weight and the experts' weights share; MXQ_OK with
// *done set when there is nothing to do.
template <int FMT>
mxq_status check_call(const Call& c, int64_t M, bool* done) {
  constexpr int kBlock = FMT == kMx ? 32 : 16;
  *done = false;
  if (!valid_dtype(c.dt) || !valid_dtype(c.out_dt)) return MXQ_ERR_DTYPE;
  if (M < 0 || c.x_rows < 0 || c.N < 0 || c.K < 0 || c.K % kBlock != 0 || c.ld_x < c.K) return MXQ_ERR_SHAPE;
  if (M > kMostRows || c.x_rows > kMostRows || c.N > kMostRows || c.K > kMostK) return MXQ_ERR_SHAPE;
  if (M == 0 || c.N == 0) {
    *done = true;
    return MXQ_OK;
  }
  // (the kernel reads the global scale for every K)
  if (!c.y || (FMT == kNv && !c.g)) return MXQ_ERR_NULL;
  if (c.K > 0 && (!c.x || !c.packed || !c.scale)) return MXQ_ERR_NULL;
  if (!aligned16(c.y)) return MXQ_ERR_ALIGN;
  if (c.K > 0 && (!aligned16(c.x) || !aligned16(c.packed) || (c.ld_x * elem_size(c.dt)) % 16 != 0))
    return MXQ_ERR_ALIGN;                         // (without columns neither is read)
  if (FMT == kNv && (reinterpret_cast<uintptr_t>(c.g) & 3u)) return MXQ_ERR_ALIGN;
  return MXQ_OK;
}

template <int FMT>
MatvecArgs make_args(const Call& c, int64_t M) {
  constexpr int kBlock = FMT == kMx ? 32 : 16;
  MatvecArgs a{};
  a.x = c.x;
  a.w = c.packed;
  a.s = c.scale;
  a.g = c.g;
  a.y = c.y;
  a.ld_x = c.ld_x;
  a.N = c.N;
  a.K = c.K;
  a.M = M;
  a.x_rows = c.x_rows;
  a.w_pitch = c.K / 2;
  a.s_pitch = c.K / kBlock;
  a.w_expert = c.N * a.w_pitch;
  a.s_expert = c.N * a.s_pitch;
  a.top_k = 1;
  a.g_per = 1;
  a.stages = uint32_t((c.K + kStageK - 1) / kStageK);
  a.out_bf16 = c.out_dt == MXQ_BF16;
  const uintptr_t low = uintptr_t(a.s_pitch) | reinterpret_cast<uintptr_t>(c.scale);
  a.scale_align = low % 16 == 0 ? 16 : low % 4 == 0 ? 4 : 1;
  return a;
}

template <int FMT>
mxq_status matvec_entry(const Call& c, mxq_stream_t stream) {
  bool done;
  const mxq_status st = check_call<FMT>(c, c.x_rows, &done);
  if (st != MXQ_OK || done) return st;
  return launch_fp4<FMT>(make_args<FMT>(c, c.x_rows), c.dt, reinterpret_cast<cudaStream_t>(stream));
}

template <int FMT>
mxq_status grouped_entry(const Call& c, int32_t E, int32_t scales_per_expert, const int64_t* row_offsets,
                         int64_t R, const int32_t* order, int32_t top_k, int32_t swiglu,
                         mxq_stream_t stream) {
  if (E < 1 || E > MXQ_GROUPED_MAX_EXPERTS) return MXQ_ERR_SHAPE;
  if (swiglu != 0 && swiglu != 1) return MXQ_ERR_ARG;
  if (scales_per_expert != 1 && scales_per_expert != 2) return MXQ_ERR_ARG;
  if ((swiglu || scales_per_expert == 2) && c.N % 2 != 0) return MXQ_ERR_SHAPE;
  // an order of no rows may be NULL: an empty array need not have an address
  if (order ? top_k < 1 : R != 0 && (top_k != 1 || c.x_rows != R)) return MXQ_ERR_ARG;
  bool done;
  const mxq_status st = check_call<FMT>(c, R, &done);
  if (st != MXQ_OK || done) return st;
  if (!row_offsets) return MXQ_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(row_offsets) & 7u) || (reinterpret_cast<uintptr_t>(order) & 3u))
    return MXQ_ERR_ALIGN;
  MatvecArgs a = make_args<FMT>(c, R);
  a.off = row_offsets;
  a.order = order;
  a.top_k = top_k;
  a.E = uint32_t(E);
  a.g_per = uint32_t(scales_per_expert);
  a.swiglu = swiglu;
  return launch_fp4<FMT>(a, c.dt, reinterpret_cast<cudaStream_t>(stream));
}

}  // namespace
}  // namespace mxq

extern "C" {

mxq_status mxfp4_matvec(const void* x, int dt, int64_t M, int64_t K, int64_t ld_x, const uint8_t* packed,
                        const uint8_t* scale, int64_t N, void* y, int out_dt, mxq_stream_t stream) {
  return mxq::matvec_entry<mxq::kMx>({x, dt, M, K, ld_x, packed, scale, nullptr, N, y, out_dt}, stream);
}

mxq_status nvfp4_matvec(const void* x, int dt, int64_t M, int64_t K, int64_t ld_x, const uint8_t* packed,
                        const uint8_t* block_scale, const float* global_scale, int64_t N, void* y, int out_dt,
                        mxq_stream_t stream) {
  return mxq::matvec_entry<mxq::kNv>({x, dt, M, K, ld_x, packed, block_scale, global_scale, N, y, out_dt},
                                     stream);
}

mxq_status mxfp4_matvec_grouped(const void* x, int dt, int64_t x_rows, int64_t K, int64_t ld_x,
                                const uint8_t* packed, const uint8_t* scale, int32_t E, int64_t N,
                                const int64_t* row_offsets, int64_t R, const int32_t* order, int32_t top_k,
                                int32_t swiglu, void* y, int out_dt, mxq_stream_t stream) {
  return mxq::grouped_entry<mxq::kMx>({x, dt, x_rows, K, ld_x, packed, scale, nullptr, N, y, out_dt}, E, 1,
                                      row_offsets, R, order, top_k, swiglu, stream);
}

mxq_status nvfp4_matvec_grouped(const void* x, int dt, int64_t x_rows, int64_t K, int64_t ld_x,
                                const uint8_t* packed, const uint8_t* block_scale, const float* global_scales,
                                int32_t scales_per_expert, int32_t E, int64_t N, const int64_t* row_offsets,
                                int64_t R, const int32_t* order, int32_t top_k, int32_t swiglu, void* y,
                                int out_dt, mxq_stream_t stream) {
  return mxq::grouped_entry<mxq::kNv>({x, dt, x_rows, K, ld_x, packed, block_scale, global_scales, N, y, out_dt},
                                      E, scales_per_expert, row_offsets, R, order, top_k, swiglu, stream);
}

mxq_status moe_combine(const float* rows, int64_t R, int64_t N, const int32_t* positions, const float* weights,
                       int64_t T, int32_t top_k, void* y, int out_dt, mxq_stream_t stream) {
  using namespace mxq;
  if (!valid_dtype(out_dt)) return MXQ_ERR_DTYPE;
  if (R < 0 || N < 0 || T < 0 || top_k < 0 || R > kMostRows || N > kMostRows || T > kMostRows)
    return MXQ_ERR_SHAPE;
  if (T == 0 || N == 0) return MXQ_OK;
  if (!y || (top_k > 0 && (!positions || !weights)) || (R > 0 && !rows)) return MXQ_ERR_NULL;
  if (!aligned16(rows) || !aligned16(y) || (reinterpret_cast<uintptr_t>(positions) & 3u) ||
      (reinterpret_cast<uintptr_t>(weights) & 3u))
    return MXQ_ERR_ALIGN;
  const bool wide = N % 4 == 0;
  const int64_t per = int64_t(kThreads) * (wide ? 4 : 1);
  const int64_t blocks = (N + per - 1) / per;
  if (blocks * T > 0x7fffffffll) return MXQ_ERR_SHAPE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int bf16 = out_dt == MXQ_BF16;
  return launched(wide ? launch_pdl(moe_combine_kernel<4>, uint32_t(blocks * T), s, rows, positions, weights, y, R,
                                    T, N, top_k, uint32_t(blocks), bf16)
                       : launch_pdl(moe_combine_kernel<1>, uint32_t(blocks * T), s, rows, positions, weights, y, R,
                                    T, N, top_k, uint32_t(blocks), bf16));
}

}  // extern "C"
