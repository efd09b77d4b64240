// mxfp8_gemm_grouped.cu -- the experts' MXFP8 products on the tensor cores
// (tcgen05 kind::mxf8f6f4.block_scale): rows sorted by expert times their
// expert's weight, and the weights' gradients, for sm_100a.
//
//   rows:   D[r, n]    = sum_k A[r, k] B[e(r), n, k]      r in expert e's range of rows
//   wgrad:  D[e, a, b] = sum_{r in e} A[r, a] B[r, b]     a sum over expert e's rows
//
// with A and B the values that E4M3 codes and E8M0 scales stand for; products
// exact, sums in fp32. The ranges come from row offsets on the device, so no
// size of an expert is known to the host: the grid is as many CTAs (or pairs)
// as can be resident, and each walks the output tiles t = its index, + grid,
// ... of the list that the offsets define. Every warp that needs a tile's
// place finds it by itself (ExpertCursor): 32 experts' offsets at a time in
// the lanes, a scan for the tiles before each, a ballot for the expert. That
// takes no shared memory, which the operand ring needs.
//
// Where operands lie. rows: A [M, K] with each expert's scales in 128x4 tiles
// of its own, expert after expert (mxfp8_quantize_grouped_swizzled); B [E, N,
// K] likewise. An output tile's rows start anywhere in A: a TMA box may start
// at any row. wgrad: A [Na, P] and B [Nb, P] hold the experts' rows as
// columns, each expert padded with zeros to a multiple of 128
// (mxfp8_quantize_columnwise_grouped), so that an expert's sum is over whole
// K blocks of 128 and whole scale tiles. What a box or a scale tile reads
// beyond an expert's rows only reaches output rows or columns that are not
// stored: rows and columns of a product do not mix.
//
// Waits are bounded as in mxfp8_gemm.cu.
#include "common.cuh"
#include "mxf8_mma.cuh"

namespace mxq {
namespace {

constexpr int kEpiWarps = 8;
constexpr int kGroupThreads = 32 * (4 + kEpiWarps);   // warps: 0, 10, 11 load, 1 issues the MMAs, 2-9 are the epilogue
// staging of a warp's stores: 16 rows x 128 bytes, pitch 144
constexpr uint32_t kSlicePitch = 144;
constexpr uint32_t kSliceBytes = 16 * kSlicePitch;
constexpr uint32_t kBarrierBytes = 256;
constexpr uint32_t kScTileW = kSfTile >> 4;      // descriptors count 16 bytes
constexpr int64_t kMostSum = int64_t(1) << 26;  // terms of a sum: a tile takes less than the waits' limit

// Tiles of the weights' gradients.
template <bool PAIR>
struct TileCfg {
  static constexpr int BN = PAIR ? 256 : 128;
  static constexpr uint32_t kRows = PAIR ? 256 : 128;                  // output rows of a tile
  static constexpr int kStages = 6;
  static constexpr uint32_t kTileA = 128 * kBK;                        // and as much of B
  static constexpr uint32_t kOperands = 2 * kTileA;                    // a multiple of 1 KiB
  static constexpr uint32_t kSfbTiles = BN / 128;
  static constexpr uint32_t kScales = kSfTile * (1 + kSfbTiles);
  static constexpr uint32_t kStageTx = kOperands + kScales;            // bytes that one CTA loads a stage
  static constexpr uint32_t kSfCols = 4 * (1 + kSfbTiles);
  static constexpr uint32_t kTmemCols = BN + kStages * kSfCols <= 256 ? 256 : 512;
  static constexpr uint32_t kSmem =
      kStages * (kOperands + kScales) + kBarrierBytes + kEpiWarps * kSliceBytes + 1024;
  static_assert(BN + kStages * kSfCols <= 512, "tensor memory");
  static_assert(kSmem <= 232448, "shared memory");
};

struct GroupArgs {
  const int64_t* offsets;   // [E + 1]; the first is taken as 0
  void* d;
  int32_t* err;
  uint32_t E;
  uint32_t rows;            // rows: M (offsets are clamped to it); wgrad: P
  uint32_t rows_a;          // wgrad: Na
  uint32_t n;               // columns of D (rows: of SWIGLU, N / 2; wgrad: Nb)
  uint32_t b_rows;          // rows: N, the rows of an expert's B
  uint32_t nk;              // rows: K blocks
  uint32_t kp4;             // scale tiles along K of a 128-row block
  uint32_t nb128;           // rows: 128-row blocks of an expert's B scales
  uint32_t tiles_m;         // wgrad: output tiles along Na
  uint32_t tiles_n;         // output tiles along the columns
  const uint8_t* sfw;       // rows, SWIGLU: the weights' scales
};

// Walks the experts in order, 32 at a time in the lanes of a converged warp.
// Offsets are clamped into a rising sequence from 0 to `limit`.
struct ExpertCursor {
  const int64_t* offsets;
  uint32_t E, limit, unit;     // unit: rows of a tile
  uint32_t first;              // expert of lane 0
  uint32_t off0, off1;         // this lane's expert: its rows
  uint32_t tiles, blocks;      // row tiles / 128-row blocks up to and with this lane's expert
  uint32_t tiles0, blocks0;    // of the experts before lane 0

  __device__ __forceinline__ void load(uint32_t lane, uint32_t carry) {
    const uint32_t e = first + lane;
    uint32_t v = 0;
    if (e < E) {
      const int64_t o = offsets[e + 1];
      v = o <= 0 ? 0u : (o >= int64_t(limit) ? limit : uint32_t(o));
    }
    v = max(v, carry);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t t = __shfl_up_sync(kFull, v, o);
      if (lane >= o) v = max(v, t);
    }
    off1 = v;
    off0 = __shfl_up_sync(kFull, v, 1);
    if (lane == 0) off0 = carry;
    const uint32_t n = off1 - off0;
    uint32_t t = (n + unit - 1) / unit, b = (n + 127) / 128;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t ut = __shfl_up_sync(kFull, t, o), ub = __shfl_up_sync(kFull, b, o);
      if (lane >= o) {
        t += ut;
        b += ub;
      }
    }
    tiles = tiles0 + t;
    blocks = blocks0 + b;
  }
  __device__ __forceinline__ void start(const int64_t* o, uint32_t experts, uint32_t lim, uint32_t u,
                                        uint32_t lane) {
    offsets = o;
    E = experts;
    limit = lim;
    unit = u;
    first = tiles0 = blocks0 = 0;
    load(lane, 0);
  }
  __device__ __forceinline__ void advance(uint32_t lane) {
    first += 32;
    tiles0 = __shfl_sync(kFull, tiles, 31);
    blocks0 = __shfl_sync(kFull, blocks, 31);
    load(lane, __shfl_sync(kFull, off1, 31));
  }
};

constexpr uint32_t kBand = 8;  // row tiles of a band

// An output tile's place: all lanes of a warp hold the same.
struct Place {
  uint32_t expert;
  uint32_t row, block;         // rows: its first row, and that row's 128-row scale block
  uint32_t left;               // rows: rows of the expert from there on
  uint32_t n_blk;              // tile along the columns
  uint32_t m_blk;              // wgrad: tile along Na
  uint32_t kb0, nk;            // wgrad: K blocks
};

// rows: the tile t of the list (rising from call to call); false behind the last.
__device__ __forceinline__ bool find_rows(const GroupArgs& a, ExpertCursor& c, uint32_t t, uint32_t lane,
                                          Place& p) {
  for (;;) {
    const uint32_t hit = __ballot_sync(kFull, uint64_t(c.tiles) * a.tiles_n > t);
    if (hit) {
      const int j = __ffs(hit) - 1;
      const uint32_t incl = __shfl_sync(kFull, c.tiles, j), off0 = __shfl_sync(kFull, c.off0, j),
                     off1 = __shfl_sync(kFull, c.off1, j), blocks = __shfl_sync(kFull, c.blocks, j);
      const uint32_t n = off1 - off0, tm = (n + c.unit - 1) / c.unit;
      const uint32_t local = t - (incl - tm) * a.tiles_n;
      // bands of kBand row tiles, row tiles first in a band: neighbouring pairs
      // read the same rows of B, and what the pairs read at one time stays in L2
      const uint32_t band = local / (kBand * a.tiles_n), in_band = local - band * kBand * a.tiles_n;
      const uint32_t rows = min(kBand, tm - band * kBand);
      p.n_blk = in_band / rows;
      const uint32_t m0 = (band * kBand + in_band - p.n_blk * rows) * c.unit;
      p.expert = c.first + j;
      p.row = off0 + m0;
      p.block = blocks - (n + 127) / 128 + m0 / 128;
      p.left = n - m0;
      return true;
    }
    if (c.first + 32 >= c.E) return false;
    c.advance(lane);
  }
}

// wgrad: every expert has the same tiles; what differs is where its columns lie.
__device__ __forceinline__ bool find_wgrad(const GroupArgs& a, ExpertCursor& c, uint32_t t, uint32_t lane,
                                           Place& p) {
  const uint32_t per = a.tiles_m * a.tiles_n;
  const uint32_t e = t / per, rest = t - e * per;
  if (e >= a.E) return false;
  while (e >= c.first + 32) c.advance(lane);
  const int j = int(e - c.first);
  const uint32_t blocks = __shfl_sync(kFull, c.blocks, j), off0 = __shfl_sync(kFull, c.off0, j),
                 off1 = __shfl_sync(kFull, c.off1, j);
  const uint32_t nk = (off1 - off0 + 127) / 128, total = a.rows / 128;
  p.n_blk = rest / a.tiles_m;
  p.m_blk = rest - p.n_blk * a.tiles_m;
  p.expert = e;
  p.kb0 = min(blocks - nk, total);
  p.nk = min(nk, total - p.kb0);
  return true;
}

// silu(g) u = g u / (1 + e^-g) of two outputs. For g < 0 as (g t) (u t) / (1 +
// t^2) with t = e^(g/2): e^-g has no fp32 value from -88.8 on where silu still
// has one, and a large u brings back what lies below. t = 2^p (1 + r ln 2), with
// p = -|g| log2(e) / 2 rounded and r what the rounding and the constant's last
// bits took from it, so that the error of p (2^-24 of it) stays out of t.
// From g = -128 on t carries a factor 2^64, which the product gives back: down
// to g = -198 the largest u makes a number of silu's value. The divisor is in
// [1, 2], where the approximate reciprocal is off by at most an ulp (and 1 where
// t carries the factor).
//
// Ends of the range: t is NaN for infinite g, which the divisor's minimum (it
// drops NaN) keeps away from silu(inf) = inf, while silu(-inf) is the formula's
// NaN. Where t leaves the range the least fp32 number stands for it: a finite u
// still gives zero, an infinite one an infinity.
//
// As the epilogue is what bounds small K, its instructions count: 32768 rows of
// 64 experts, N = 4096, K = 512 162 us; one output at a time 170, and 199 before
// with the factors chosen after silu. With expf and a division 65 % more time,
// with expf alone 11 %, and 8 % at K = 2048.
__device__ __forceinline__ void swiglu2(float2 g, float2 u, uint32_t& y0, uint32_t& y1) {
  constexpr float kHi = 0.72134752f, kLo = 9.6298152e-9f;   // log2(e) / 2
  const float2 n = make_float2(-fabsf(g.x), -fabsf(g.y)), p = mul2v(n, twice(kHi));
  const float2 rest = fma2v(n, twice(kLo), fma2v(n, twice(kHi), mul2v(n, twice(-kHi))));
  const bool far[2] = {g.x <= -128.f, g.y <= -128.f};
  float2 t, m, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t.x) : "f"(far[0] ? p.x + 64.f : p.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t.y) : "f"(far[1] ? p.y + 64.f : p.y));
  t = fma2v(t, mul2v(rest, twice(0.69314718f)), t);
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m.x) : "f"(g.x < 0.f ? t.x : 1.f), "f"(0x1p-149f));
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m.y) : "f"(g.y < 0.f ? t.y : 1.f), "f"(0x1p-149f));
  const float2 d = fma2v(t, t, twice(1.f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(fminf(d.x, 2.f)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(fminf(d.y, 2.f)));
  const float2 v = mul2v(mul2v(mul2v(g, m), r), mul2v(u, m));
  y0 = __float_as_uint(far[0] ? v.x * 0x1p-128f : v.x);
  y1 = __float_as_uint(far[1] ? v.y * 0x1p-128f : v.y);
}

// ---------------------------------------------------------- rows
//
// The product is formed transposed: a pair of CTAs (tcgen05 cta_group::2)
// holds 256 rows of the weight as the MMA's M side, and up to 256 of the
// expert's rows as its N side, in steps of 32. The ragged side is so the one
// whose size an MMA may choose: a tile of 20 rows costs an eighth of one of
// 256, where rows on the M side fill 128 or 256 whatever they are. Measured
// against that form (256 x 256 over pairs, 128 x 256 in single CTAs for few
// rows), with 64 weights of 4096 x 7168 and rows spread over them like e^(0.7
// normal): 16384 rows 475 us against 658, 8192 rows 352 against 411, 8 rows
// 46 against 56.
//
// Per K block of 128 each CTA loads its 128 rows of the weight (16 KiB), its
// half of the tile's rows (up to 16 KiB, in at most three boxes of 128, 64, 32
// and 16 rows), and the scale tiles of both; six stages. The accumulator has a
// weight row per lane and a row of the experts' per column.
//
// Warps: 0, 10 and 11 load, 1 (of the even CTA) issues the MMAs, 2-9 are the
// epilogue. The issue of TMA loads is what bound the first version: a lone lane
// took 165 cycles a load, five or more a K block of 512 MMA cycles (32768
// rows, 1156 us). Converged warps whose elected lane issues take about 105, and
// three of them side by side (weight and its scales, rows, their scales) leave
// the MMA issue as the longest (835 us). Prefetches into L2, by TMA or by
// loads of another warp, made it slower: they take from the same queues.
//
// The epilogue has two warps a quarter of the lanes, each with half of the
// columns. Each takes its columns into registers in one go (at most 128 fp32),
// hands the accumulator back, and does everything else while the next tile's
// MMAs run: tensor memory has no room for a second accumulator beside the
// scales. A column of 32 lanes is 32 neighbouring outputs of a row, stored as
// 64 (bf16, lanes exchanging halves of column pairs) or 128 bytes.
//
// SWIGLU: each CTA holds 64 rows of the gate and the same 64 of the up half, so
// that the factors of an output are in one CTA, 64 accumulator lanes apart, and
// two warps exchange them through shared memory; the halves of the product are
// never written to memory. (With the gate in one CTA and the up half in the
// other, sends to the peer's shared memory took 25000 cycles a tile and bound
// the kernel below K = 4096.) The scale tile of those 128 rows is no tile of
// memory: its quarters 0 and 1 come from a half of the gate's tile, 2 and 3
// from a half of the up half's, and a TMA copy cannot put eight of 16 bytes
// beside eight others; warp 11 joins them. 32768 rows of 64 experts, N = 4096,
// K = 2048: 265 us in short runs, 313 under load (505 with the sends; without
// SWIGLU 250 and 297); from K = 4096 on within 3 % of the product's own time. At K
// = 512 silu itself is what bounds it, 4.7 us a tile: 161 us (without SWIGLU 94 in
// short runs, 113 under load).
//
// What bounds it: with few rows a weight, HBM (512 rows 297 us for weights of
// 1.9 GB; 6.4 TB/s). With many, the clock that the power limit leaves and the
// ragged tails: 32768 rows of one expert take 671 us, as the single product does
// (2.87 PFLOP/s). Spread over 64 experts they are about 159 row tiles instead of
// 128, and a tail takes as long as a whole tile (its stages are part empty, so
// that the bytes in flight do not cover the latency of the weight's): 750 to 835
// us, and 960 to 1000 once the clock has settled at 1.1 to 1.2 GHz under load.

constexpr uint32_t kWeightTile = 128 * kBK;                 // a CTA's rows of the weight
constexpr uint32_t kSendBytes = 32 * 8 * 4;                 // eight columns of a warp
constexpr uint32_t kJoin = 8;                               // K blocks of a group of joined scale tiles
constexpr uint32_t kJoinRing = 2;                           // groups
constexpr uint32_t kRowBars = 256;

// FEW: calls of at most 64 rows, whose tiles leave the shared memory to more
// stages: a pair's loads are bound by the bytes in flight where few pairs have
// tiles, and by the issue of the loads (8 rows of eight experts, 4096 x 7168,
// 42.9 us with six stages, 40.2 with ten; one expert 17.0 and 12.6).
template <bool SWIGLU, bool FEW>
struct RowCfg {
  static constexpr uint32_t kTile = FEW ? 64 : 256;                      // most rows of a tile
  static constexpr int kStages = FEW ? (SWIGLU ? 9 : 10) : 6;
  static constexpr uint32_t kStage = kWeightTile + kTile / 2 * kBK;      // and its half of the rows
  static constexpr uint32_t kXTiles = FEW ? 1 : 2;                       // scale tiles of the rows
  static constexpr uint32_t kXSf = SWIGLU ? 0 : kSfTile;                 // behind the weight's, which SWIGLU joins
  static constexpr uint32_t kScales = kXSf + kXTiles * kSfTile;
  static constexpr uint32_t kSfCols = 4 * (1 + kXTiles);
  // shared memory behind the stages' tiles; SWIGLU: joined scale tiles [group][K
  // block], columns for the other warp [warp][2]
  static constexpr uint32_t kScalesAt = kStages * kStage;
  static constexpr uint32_t kJoinedAt = kScalesAt + kStages * kScales;
  static constexpr uint32_t kSlotsAt = kJoinedAt + (SWIGLU ? kJoinRing * kJoin * kSfTile : 0);
  static constexpr uint32_t kBarsAt = kSlotsAt + (SWIGLU ? 2 * kEpiWarps * kSendBytes : 0);
  static constexpr uint32_t kSmem = kBarsAt + kRowBars + 1024;           // (the start is rounded up to 1 KiB)
  static_assert(256 + kStages * kSfCols <= 512, "tensor memory");
  static_assert(kSmem <= 232448, "shared memory");
  static_assert(8 * (2 * kStages + 2 + 2 * kJoinRing + kJoinRing) + 4 <= kRowBars, "barriers");
};

// The rows in boxes of 128, 64, 32 and 16.
struct RowMaps {
  CUtensorMap box[4];
};

// Instruction descriptor as instr_desc_pair for N columns (a multiple of 32), k = 0.
__device__ __forceinline__ uint32_t instr_desc_n(uint32_t n) {
  return ((n >> 3) << 17) | (1u << 23) | (uint32_t(256 >> 4) << 24);
}

// Two warps (64 threads) at barrier `id`; true where `ok` was true in all of them.
__device__ __forceinline__ bool meet(uint32_t id, bool ok) {
  uint32_t r;
  asm volatile(
      "{ .reg .pred p, q; setp.ne.u32 p, %2, 0; barrier.cta.red.and.pred q, %1, 64, p; selp.u32 %0, 1, 0, q; }"
      : "=r"(r)
      : "r"(id), "r"(uint32_t(ok))
      : "memory");
  return r != 0;
}

__device__ __forceinline__ uint2 ldg64(const void* p) {
  uint2 v;
  asm volatile("ld.global.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

// COLS columns v of this lane's weight row, the tile's rows t .. (COLS even): p is
// this lane's output of row t (fp32), or of row t, t + 1 for an even, odd lane
// the pair of outputs that its pair of lanes has (bf16). Rows from `left` on
// are not written; left is 0 for lanes without outputs.
template <int COLS, typename OutT>
__device__ __forceinline__ void store_columns(OutT* p, uint32_t ld, const uint32_t* v, int32_t left) {
  if constexpr (sizeof(OutT) == 2) {
    const uint32_t odd = threadIdx.x & 1;
#pragma unroll
    for (int c = 0; c < COLS; c += 2) {
      const uint32_t x = __shfl_xor_sync(kFull, odd ? v[c] : v[c + 1], 1);
      const uint32_t w = odd ? cvt_bf16x2(__uint_as_float(x), __uint_as_float(v[c + 1]))
                             : cvt_bf16x2(__uint_as_float(v[c]), __uint_as_float(x));
      if (c + int32_t(odd) < left) st_u32(p + uint64_t(uint32_t(c)) * ld, w);
    }
  } else {
#pragma unroll
    for (int c = 0; c < COLS; c++)
      if (c < left) st_u32(p + uint64_t(uint32_t(c)) * ld, v[c]);
  }
}

template <bool SWIGLU, bool FEW, typename OutT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGroupThreads, 1)
mxfp8_rows_kernel(const __grid_constant__ CUtensorMap tma_w, const __grid_constant__ RowMaps rows,
                  const __grid_constant__ CUtensorMap tma_sfw,
                  const __grid_constant__ CUtensorMap tma_sfx, const __grid_constant__ GroupArgs a) {
  using R = RowCfg<SWIGLU, FEW>;
  constexpr int kStages = R::kStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;           // operand tiles: 128-byte swizzle atoms of 1 KiB
  uint8_t* smem = smem_raw + (base - raw);
  const uint32_t scales = base + R::kScalesAt, joined = base + R::kJoinedAt, slots = base + R::kSlotsAt;
  const uint32_t bars = base + R::kBarsAt;
  auto full_bar = [&](uint32_t s) { return bars + 8u * s; };
  auto empty_bar = [&](uint32_t s) { return bars + 8u * (kStages + s); };
  const uint32_t acc_full = bars + 8u * (2 * kStages);
  const uint32_t acc_empty = acc_full + 8u;
  auto join_full = [&](uint32_t g) { return acc_empty + 8u * (1 + g); };
  auto join_empty = [&](uint32_t g) { return acc_empty + 8u * (1 + kJoinRing + g); };
  auto join_odd = [&](uint32_t g) { return acc_empty + 8u * (1 + 2 * kJoinRing + g); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + (join_odd(kJoinRing) - base));

  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();                // 0: issues the MMAs
  const uint32_t step = gridDim.x >> 1;
  uint32_t tile = blockIdx.x >> 1;

  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                 ::"r"(smem_u32(tmem_slot)), "r"(512u) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  if (threadIdx.x == 32) {
    for (int s = 0; s < kStages; s++) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (uint32_t g = 0; g < kJoinRing; g++) {
      mbar_init(join_full(g), 2);  // this CTA's warp 11 and the odd CTA's warp 1
      mbar_init(join_empty(g), 1);
      mbar_init(join_odd(g), 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, 2 * kEpiWarps);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the peer's barriers are initialised before any remote arrival
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_enter();  // (all of the above overlaps the end of the grid before)

  ExpertCursor cursor;
  cursor.start(a.offsets, a.E, a.rows, R::kTile, lane);
  Place p{};
  // columns of a tile's accumulator: its rows, a multiple of 32
  auto columns = [&]() { return min(R::kTile, (p.left + 31u) & ~31u); };

  // first row of the weight of this CTA in a tile (SWIGLU: of the gate's), and its scale block
  auto w_row_of = [&](const Place& q) {
    return q.expert * a.b_rows + (SWIGLU ? q.n_blk * 128 + rank * 64 : q.n_blk * 256 + rank * 128);
  };
  auto w_blk_of = [&](const Place& q) { return q.expert * a.nb128 + (SWIGLU ? q.n_blk : q.n_blk * 2 + rank); };

  if (warp == 0 || warp == 2 + kEpiWarps || (!SWIGLU && warp == 3 + kEpiWarps)) {
    // --------------------------------------------------------- producers
    // The issue of a TMA load holds a warp for 100 cycles and more. Warp 0 loads
    // the weight and its scales, warp 10 the rows, warp 11 their scales; SWIGLU:
    // warp 0 the two halves of the weight and the rows' scales. FEW without
    // SWIGLU: the three take the K blocks in turn, each all loads of its own, as
    // no MMAs hide the longest share (one expert of 4096 x 7168 15.5 us, in turn
    // 12.6). Else a stage would only be loaded later (32768 rows of 64 970 us, in
    // turn 1050; SWIGLU, two warps, 8 rows 42.6 and 44.2).
    constexpr bool kTurns = FEW && !SWIGLU;
    constexpr uint32_t kStep = kTurns ? 3 : 1;
    const bool weights = warp == 0, rows_warp = warp == 2 + kEpiWarps;
    const uint32_t first = !kTurns || warp == 0 ? 0 : warp - (1 + kEpiWarps);
    const uint32_t bar0 = cluster_addr(full_bar(0), 0);
    uint32_t s = first, phase = 1, kb = first;
    bool ok = true;
    for (; ok && find_rows(a, cursor, tile, lane, p); tile += step) {
      const uint32_t n = columns(), mine = n / 2;         // this CTA's share of the rows, a multiple of 16
      const uint32_t x_row = p.row + rank * mine;
      const uint32_t w_row = w_row_of(p), w_sf = 4 * w_blk_of(p) * a.kp4;
      const uint32_t x_sf = 4 * p.block * a.kp4;
      const uint32_t tx = 2 * (kWeightTile + mine * kBK + kSfTile * ((n > 128 ? 2 : 1) + (SWIGLU ? 0 : 1)));
      for (; kb < a.nk; kb += kStep) {
        if (!__all_sync(kFull, mbar_wait(empty_bar(s), phase, kWaitNs))) {
          if (lane == 0) record_error(a.err, kErrEmptyWait);
          ok = false;
          break;
        }
        const uint32_t bar = bar0 + 8u * s, x = kb * kBK;
        const uint32_t st = base + s * R::kStage, sf = scales + s * R::kScales;
        auto load_weight = [&]() {
          if (rank == 0) mbar_elect_expect_tx(full_bar(s), tx);
          tma_elect_2d_pair(st, &tma_w, bar, int32_t(x), int32_t(w_row));
          if constexpr (SWIGLU)
            tma_elect_2d_pair(st + kWeightTile / 2, &tma_w, bar, int32_t(x), int32_t(w_row + a.n));
          else
            tma_elect_2d_pair(sf, &tma_sfw, bar, 0, int32_t(w_sf + 4 * kb));
        };
        auto load_rows = [&]() {
          uint32_t r = 0;
#pragma unroll
          for (int b = FEW ? 2 : 0; b < 4; b++)
            if (mine & (128u >> b)) {
              tma_elect_2d_pair(st + kWeightTile + r * kBK, &rows.box[b], bar, int32_t(x), int32_t(x_row + r));
              r += 128u >> b;
            }
        };
        auto load_row_scales = [&]() {
          tma_elect_2d_pair(sf + R::kXSf, &tma_sfx, bar, 0, int32_t(x_sf + 4 * kb));
          if (!FEW && n > 128)
            tma_elect_2d_pair(sf + R::kXSf + kSfTile, &tma_sfx, bar, 0, int32_t(x_sf + 4 * a.kp4 + 4 * kb));
        };
        if constexpr (kTurns) {
          load_weight();
          load_rows();
          load_row_scales();
        } else if (weights) {
          load_weight();
          if constexpr (SWIGLU) load_row_scales();
        } else if (rows_warp) {
          load_rows();
        } else {
          load_row_scales();
        }
        s += kStep;
        if (s >= kStages) {
          s -= kStages;
          phase ^= 1u;
        }
      }
      kb -= a.nk;                                         // of the next tile
    }
  } else if (SWIGLU && warp == 3 + kEpiWarps) {
    // ------------------------------------- joined scale tiles of the weight
    // Quarters 0 and 1 of a joined tile are the gate's 64 rows, 2 and 3 the up
    // half's: a lane's line of it is eight bytes of the gate's tile and eight of
    // the up half's. They go in groups of kJoin K blocks: a release that the
    // other CTA may rely on takes 1000 to 3000 cycles (one per K block: 610 us
    // for K = 2048), and is left to the odd CTA's warp 1, which has no MMAs to
    // issue (released by this warp: 310 us for 512 rows, 288 so).
    uint32_t g = 0, phase = 1;
    uint2 gate[kJoin], up[kJoin];
    const uint64_t up_sf = uint64_t(a.n / 128) * a.kp4 * kSfTile;
    auto load = [&](uint32_t kb) {
      const uint8_t* src = a.sfw + (uint64_t(w_blk_of(p)) * a.kp4 + kb) * kSfTile + lane * 16 + rank * 8;
#pragma unroll
      for (uint32_t i = 0; i < kJoin; i++)
        if (kb + i < a.nk) {
          gate[i] = ldg64(src + uint64_t(i) * kSfTile);
          up[i] = ldg64(src + up_sf + uint64_t(i) * kSfTile);
        }
    };
    bool have = a.nk > 0 && find_rows(a, cursor, tile, lane, p);
    if (have) load(0);
    for (uint32_t kb = 0; have;) {
      if (!__all_sync(kFull, mbar_wait(join_empty(g), phase, kWaitNs))) {
        if (lane == 0) record_error(a.err, kErrEmptyWait);
        break;
      }
#pragma unroll
      for (uint32_t i = 0; i < kJoin; i++)
        sts128_u32(joined + (g * kJoin + i) * kSfTile + lane * 16, make_uint4(gate[i].x, gate[i].y, up[i].x, up[i].y));
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if ((kb += kJoin) >= a.nk) {
        kb = 0;
        have = find_rows(a, cursor, tile += step, lane, p);
      }
      if (lane == 0) mbar_arrive(rank == 0 ? join_full(g) : join_odd(g));
      if (have) load(kb);
      if (++g == kJoinRing) {
        g = 0;
        phase ^= 1u;
      }
    }
  } else if (SWIGLU && warp == 1 && rank == 1) {
    // hands the odd CTA's joined scale tiles over to the MMA issuer
    if (a.nk > 0) {
      uint32_t g = 0, phase = 0;
      bool ok = true;
      for (; ok && find_rows(a, cursor, tile, lane, p); tile += step)
        for (uint32_t kb = 0; kb < a.nk; kb += kJoin) {
          if (!__all_sync(kFull, mbar_wait(join_odd(g), phase, kWaitNs))) {
            if (lane == 0) record_error(a.err, kErrFullWait);
            ok = false;
            break;
          }
          if (lane == 0) mbar_release_remote(cluster_addr(join_full(g), 0));
          if (++g == kJoinRing) {
            g = 0;
            phase ^= 1u;
          }
        }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------- MMA issuer
    // a converged warp with descriptors as 32-bit words plus offsets, as in
    // mxfp8_gemm.cu
    if (rank == 0 && a.nk > 0) {
      const uint64_t op0 = operand_desc(base), sc0 = scale_desc(scales);
      const uint32_t op_lo = uint32_t(op0), op_hi = uint32_t(op0 >> 32);
      const uint32_t sc_lo = uint32_t(sc0), sc_hi = uint32_t(sc0 >> 32);
      constexpr uint32_t kStageW = R::kStage >> 4, kTileW = kWeightTile >> 4;
      constexpr uint32_t kScaleW = R::kScales >> 4;
      const uint32_t join_lo = uint32_t(scale_desc(joined));
      uint32_t s = 0, phase = 0, done = 0, g = 0, join_phase = 0;
      for (; find_rows(a, cursor, tile, lane, p); tile += step, done++) {
        const uint32_t n = columns(), idesc = instr_desc_n(n);
        // the epilogue must have read the previous tile's accumulator
        if (done > 0 && !__all_sync(kFull, mbar_wait(acc_empty, (done - 1) & 1u, kWaitNs))) {
          if (lane == 0) record_error(a.err, kErrAccumWait);
          break;
        }
        tc_fence_after();
        bool ok = true;
        for (uint32_t kb = 0; kb < a.nk; kb++) {
          const bool first = SWIGLU && kb % kJoin == 0, last = SWIGLU && (kb % kJoin == kJoin - 1 || kb + 1 == a.nk);
          if (!__all_sync(kFull, (!first || mbar_wait<true>(join_full(g), join_phase, kWaitNs)) &&
                                     mbar_wait(full_bar(s), phase, kWaitNs))) {
            if (lane == 0) record_error(a.err, kErrFullWait);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t so = s * kStageW, sc = sc_lo + s * kScaleW;
          const uint32_t sfw_t = tmem + 256 + R::kSfCols * s, sfx_t = sfw_t + 4u;
          mma_block_pair(tmem, op_lo + so, op_lo + so + kTileW, op_hi, idesc, sfw_t, sfx_t,
                         SWIGLU ? join_lo + (g * kJoin + kb % kJoin) * kScTileW : sc, sc + (R::kXSf >> 4), sc_hi, !FEW && n > 128, kb,
                         empty_bar(s));
          if (last) {
            mma_commit_pair(join_empty(g));
            if (++g == kJoinRing) {
              g = 0;
              join_phase ^= 1u;
            }
          }
          if (++s == kStages) {
            s = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        mma_commit_pair(acc_full);
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    // warp w reads accumulator lanes (weight rows) 32 (w % 4) .. + 31; the
    // second four warps take the second half of the columns
    const uint32_t quarter = warp & 3, half = (warp - 2) >> 2;
    const uint32_t lead_acc_empty = cluster_addr(acc_empty, 0);
    // SWIGLU: quarters 0 and 1 hold the gate, 2 and 3 the up half of the same
    // outputs; the two warps that share outputs meet at a barrier of their own
    const bool upper = quarter >= 2;
    const uint32_t pair_id = 1 + 2 * half + (quarter & 1);
    const uint32_t my_slots = slots + (4 * half + quarter) * 2 * kSendBytes;
    const uint32_t its_slots = slots + (4 * half + (quarter ^ 2)) * 2 * kSendBytes;
    uint32_t done = 0;
    for (; find_rows(a, cursor, tile, lane, p); tile += step, done++) {
      const uint32_t cols = columns() / 2;                // of this warp, a multiple of 16
      const uint32_t taddr = tmem + ((quarter * 32) << 16) + half * cols;
      constexpr int kCols = R::kTile / 2;                 // most columns of a warp
      uint32_t v[kCols];
      // the phase completes once for everyone: a lane that saw it lets the warp go
      bool ok = a.nk == 0 || __any_sync(kFull, mbar_wait(acc_full, done & 1u, kWaitNs));
      if constexpr (SWIGLU) ok = meet(pair_id, ok);       // (both warps go on, or neither; the slots are read)
      if (!ok) {
        if (lane == 0) record_error(a.err, kErrAccumWait);
        break;
      }
      if (a.nk > 0) {
        tc_fence_after();
        // (columns that the tile does not have are read and not used)
#pragma unroll
        for (int c = 0; c < kCols; c += 32) tmem_ld32_start(taddr + c, *reinterpret_cast<uint32_t(*)[32]>(&v[c]));
#pragma unroll
        for (int c = 0; c < kCols; c += 32) tmem_ld_wait(*reinterpret_cast<uint32_t(*)[32]>(&v[c]));
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(lead_acc_empty);
      } else {
#pragma unroll
        for (int c = 0; c < kCols; c++) v[c] = 0;
      }
      const uint32_t f = (SWIGLU ? p.n_blk * 128 + rank * 64 + (quarter & 1) * 32 : p.n_blk * 256 + rank * 128 + quarter * 32) + lane;
      const uint32_t t0 = half * cols + (SWIGLU && upper ? 8 : 0);
      int32_t left = f < a.n ? int32_t(min(p.left, R::kTile)) - int32_t(t0) : 0;
      OutT* d = static_cast<OutT*>(a.d) + uint64_t(p.row + t0) * a.n + f;
      if constexpr (sizeof(OutT) == 2) d += int64_t(lane & 1) * (int64_t(a.n) - 1);
#pragma unroll
      for (int c = 0; c < kCols; c += 16) {
        if (uint32_t(c) >= cols) break;
        if constexpr (!SWIGLU) {
          store_columns<16>(d, a.n, &v[c], left);
        } else {
          // of 16 columns the gate's warp finishes the first eight and the up
          // half's the last: each gives the other's eight away. Two slots: what
          // is written two chunks on was read before the barrier between.
          const uint32_t off = (c & 16 ? kSendBytes : 0) + lane * 16;
#pragma unroll
          for (int i = 0; i < 8; i += 4)
            sts128_u32(my_slots + off + 128 * i,
                       upper ? make_uint4(v[c + i], v[c + i + 1], v[c + i + 2], v[c + i + 3])
                             : make_uint4(v[c + 8 + i], v[c + 9 + i], v[c + 10 + i], v[c + 11 + i]));
          meet(pair_id, true);
          const uint4 q0 = lds128_u32(its_slots + off), q1 = lds128_u32(its_slots + off + 512);
          uint32_t y[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const float2 mine = make_float2(__uint_as_float(upper ? v[c + 8 + i] : v[c + i]),
                                            __uint_as_float(upper ? v[c + 9 + i] : v[c + 1 + i]));
            const float2 other = make_float2(__uint_as_float(y[i]), __uint_as_float(y[i + 1]));
            swiglu2(upper ? other : mine, upper ? mine : other, y[i], y[i + 1]);
          }
          store_columns<8>(d, a.n, y, left);
        }
        d += 16 * uint64_t(a.n);
        left -= 16;
      }
    }
  }

  // neither CTA leaves while the other may still reach its shared memory or
  // tensor memory (barrier arrivals, MMA operand reads, scale copies)
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

// --------------------------------------------------------- wgrad
//
// Output tiles of 256 x 256 over a pair of CTAs (cta_group::2, six stages of 32
// KiB of operands in each CTA), or 128 x 128 in one CTA where a side has at
// most 128: every expert has the same tiles, with as many K blocks as its rows
// come to, and none for an expert without rows (zeros are written). Warps as
// above; the accumulator has a row of D per lane, a warp's columns go through
// staging rows of its own.

template <bool PAIR, typename OutT>
__global__ void __launch_bounds__(kGroupThreads, 1)
mxfp8_wgrad_kernel(const __grid_constant__ CUtensorMap tma_a, const __grid_constant__ CUtensorMap tma_b,
                   const __grid_constant__ CUtensorMap tma_sfa,
                   const __grid_constant__ CUtensorMap tma_sfb, const __grid_constant__ GroupArgs a) {
  using C = TileCfg<PAIR>;
  constexpr int BN = C::BN;
  constexpr int kStages = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;           // operand tiles: 128-byte swizzle atoms of 1 KiB
  uint8_t* smem = smem_raw + (base - raw);
  const uint32_t scales = base + kStages * C::kOperands;
  const uint32_t bars = scales + kStages * C::kScales;
  auto full_bar = [&](uint32_t s) { return bars + 8u * s; };
  auto empty_bar = [&](uint32_t s) { return bars + 8u * (kStages + s); };
  const uint32_t acc_full = bars + 8u * (2 * kStages);
  const uint32_t acc_empty = acc_full + 8u;
  uint32_t* tmem_slot =
      reinterpret_cast<uint32_t*>(smem + (bars - base) + 8 * (2 * kStages + 2));

  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0;     // 0: issues the MMAs
  const uint32_t step = PAIR ? gridDim.x >> 1 : gridDim.x;
  uint32_t tile = PAIR ? blockIdx.x >> 1 : blockIdx.x;

  if (warp == 0) {
    if constexpr (PAIR) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                   ::"r"(smem_u32(tmem_slot)), "r"(C::kTmemCols) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                   ::"r"(smem_u32(tmem_slot)), "r"(C::kTmemCols) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
  }
  if (threadIdx.x == 32) {
    for (int s = 0; s < kStages; s++) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, (PAIR ? 2 : 1) * kEpiWarps);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // the peer's barriers are initialised before any remote arrival
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_enter();  // (all of the above overlaps the end of the grid before)

  ExpertCursor cursor;
  // (rows are clamped by K blocks, in find_wgrad)
  cursor.start(a.offsets, a.E, 0x7fffff00u, 128, lane);
  Place p;

  if (warp == 0 || warp >= 2 + kEpiWarps) {
    // --------------------------------------------------------- producers
    // (A and its scales, B, B's scales)
    const uint32_t bar0 = PAIR ? cluster_addr(full_bar(0), 0) : full_bar(0);
    auto load = [&](uint32_t dst, const CUtensorMap* map, uint32_t bar, uint32_t x, uint32_t y) {
      if constexpr (PAIR)
        tma_elect_2d_pair(dst, map, bar, int32_t(x), int32_t(y));
      else
        tma_elect_2d(dst, map, bar, int32_t(x), int32_t(y));
    };
    uint32_t s = 0, phase = 1;
    bool ok = true;
    for (; ok && find_wgrad(a, cursor, tile, lane, p); tile += step) {
      const uint32_t a_row = p.m_blk * C::kRows + 128 * rank, a_blk = p.m_blk * (C::kRows / 128) + rank;
      const uint32_t b_row = p.n_blk * BN + 128 * rank, b_blk = p.n_blk * C::kSfbTiles;
      for (uint32_t i = 0; i < p.nk; i++) {
        if (!__all_sync(kFull, mbar_wait(empty_bar(s), phase, kWaitNs))) {
          if (lane == 0) record_error(a.err, kErrEmptyWait);
          ok = false;
          break;
        }
        const uint32_t kb = p.kb0 + i, bar = bar0 + 8u * s;
        const uint32_t st = base + s * C::kOperands, sf = scales + s * C::kScales;
        if (warp == 0) {
          if (rank == 0) mbar_elect_expect_tx(full_bar(s), (PAIR ? 2 : 1) * C::kStageTx);
          load(st, &tma_a, bar, kb * kBK, a_row);
          load(sf, &tma_sfa, bar, 0, 4 * (a_blk * a.kp4 + kb));
        } else if (warp == 2 + kEpiWarps) {
          load(st + C::kTileA, &tma_b, bar, kb * kBK, b_row);
        } else {
          load(sf + kSfTile, &tma_sfb, bar, 0, 4 * (b_blk * a.kp4 + kb));
          if constexpr (C::kSfbTiles == 2) load(sf + 2 * kSfTile, &tma_sfb, bar, 0, 4 * ((b_blk + 1) * a.kp4 + kb));
        }
        if (++s == kStages) {
          s = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------- MMA issuer
    // a converged warp with descriptors as 32-bit words plus offsets, as in
    // mxfp8_gemm.cu
    if (rank == 0) {
      const uint64_t op0 = operand_desc(base), sc0 = scale_desc(scales);
      const uint32_t op_lo = uint32_t(op0), op_hi = uint32_t(op0 >> 32);
      const uint32_t sc_lo = uint32_t(sc0), sc_hi = uint32_t(sc0 >> 32);
      constexpr uint32_t kStageW = C::kOperands >> 4, kTileAW = C::kTileA >> 4;
      constexpr uint32_t kScaleW = C::kScales >> 4, kSfW = kSfTile >> 4;
      uint32_t s = 0, phase = 0, done = 0;
      for (; find_wgrad(a, cursor, tile, lane, p); tile += step) {
        if (p.nk == 0) continue;
        // the epilogue must have read the previous tile's accumulator
        if (done > 0 && !__all_sync(kFull, mbar_wait(acc_empty, (done - 1) & 1u, kWaitNs))) {
          if (lane == 0) record_error(a.err, kErrAccumWait);
          break;
        }
        tc_fence_after();
        bool ok = true;
        for (uint32_t i = 0; i < p.nk; i++) {
          if (!__all_sync(kFull, mbar_wait(full_bar(s), phase, kWaitNs))) {
            if (lane == 0) record_error(a.err, kErrFullWait);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t so = s * kStageW, sc = sc_lo + s * kScaleW;
          const uint32_t sfa_t = tmem + BN + C::kSfCols * s, sfb_t = sfa_t + 4u;
          if constexpr (PAIR) {
            mma_block_pair(tmem, op_lo + so, op_lo + so + kTileAW, op_hi, instr_desc_n(BN), sfa_t, sfb_t, sc, sc + kScTileW, sc_hi, 1u, i,
                           empty_bar(s));
          } else {
            tmem_copy_scales(sfb_t, sc + kSfW, sc_hi);
            tmem_copy_scales(sfa_t, sc, sc_hi);
#pragma unroll
            for (uint32_t k = 0; k < 4; k++)
              mma_mxf8(tmem, op_lo + so + 2 * k, op_lo + so + kTileAW + 2 * k, op_hi, instr_desc<BN>(k),
                       sfa_t | (k << 30), sfb_t | (k << 30), (i | k) != 0u);
            mma_commit(empty_bar(s));
          }
          if (++s == kStages) {
            s = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if constexpr (PAIR)
          mma_commit_pair(acc_full);
        else
          mma_commit(acc_full);
        done++;
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    // warp w reads accumulator lanes (rows) 32 (w % 4) .. + 31; the warps of
    // the second four take the second half of the columns
    constexpr int kCols = BN / 2;                                     // columns of a warp
    const uint32_t quarter = warp & 3, half = (warp - 2) >> 2;
    const uint32_t taddr = tmem + ((quarter * 32) << 16);
    const uint32_t slice = bars + kBarrierBytes + kSliceBytes * (warp - 2);
    const uint32_t lead_acc_empty = PAIR ? cluster_addr(acc_empty, 0) : acc_empty;
    uint32_t done = 0;
    for (; find_wgrad(a, cursor, tile, lane, p); tile += step) {
      uint32_t v[kCols];
      if (p.nk > 0) {
        // the phase completes once for everyone: a lane that saw it lets the warp go
        if (!__any_sync(kFull, mbar_wait(acc_full, done & 1u, kWaitNs))) {
          if (lane == 0) record_error(a.err, kErrAccumWait);
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < kCols; c += 32)
          tmem_ld32_start(taddr + kCols * half + c, *reinterpret_cast<uint32_t(*)[32]>(&v[c]));
#pragma unroll
        for (int c = 0; c < kCols; c += 32) tmem_ld_wait(*reinterpret_cast<uint32_t(*)[32]>(&v[c]));
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (PAIR)
            mbar_arrive_remote(lead_acc_empty);
          else
            mbar_arrive(acc_empty);
        }
        done++;
      } else {
#pragma unroll
        for (int c = 0; c < kCols; c++) v[c] = 0;
      }
      const uint32_t r0 = 128 * rank + 32 * quarter;                  // the warp's first row of the tile
      const uint32_t row0 = p.m_blk * C::kRows + r0;
      if (row0 >= a.rows_a) continue;
      const uint32_t rows = min(32u, a.rows_a - row0);
      const uint32_t col0 = p.n_blk * BN + kCols * half;
      if (col0 >= a.n) continue;
      const uint32_t cols = min(uint32_t(kCols), a.n - col0);         // a multiple of 16
      OutT* d = static_cast<OutT*>(a.d) + (uint64_t(p.expert) * a.rows_a + row0) * a.n + col0;
      // slices of 128 bytes a row (64 bf16 columns or 32 fp32), 16 rows at a
      // time, through the warp's staging rows, so that a store instruction
      // writes whole 128-byte lines (with lines in halves the writes took 1.3
      // times as long)
      constexpr uint32_t kSlice = 128 / sizeof(OutT);
      const uint32_t rsub = lane >> 3, ch = lane & 7;
#pragma unroll
      for (uint32_t c0 = 0; c0 < uint32_t(kCols); c0 += kSlice) {
        if (c0 >= cols) break;
        const uint32_t col = c0 + kSlice / 8 * ch;
#pragma unroll
        for (uint32_t h = 0; h < 2; h++) {
          if (lane >> 4 == h) {
#pragma unroll
            for (uint32_t q = 0; q < 8; q++) {
              uint32_t w[4];
#pragma unroll
              for (uint32_t i = 0; i < 4; i++) {
                if constexpr (sizeof(OutT) == 2)
                  w[i] = cvt_bf16x2(__uint_as_float(v[c0 + 8 * q + 2 * i]), __uint_as_float(v[c0 + 8 * q + 2 * i + 1]));
                else
                  w[i] = v[c0 + 4 * q + i];
              }
              sts128_u32(slice + (lane & 15) * kSlicePitch + 16 * q, make_uint4(w[0], w[1], w[2], w[3]));
            }
          }
          __syncwarp();
#pragma unroll
          for (uint32_t j = 0; j < 4; j++) {
            const uint32_t rr = 4 * j + rsub;
            const uint4 x = lds128_u32(slice + rr * kSlicePitch + 16 * ch);
            if (16 * h + rr < rows && col < cols) st_v4(d + uint64_t(16 * h + rr) * a.n + col, x);
          }
          __syncwarp();
        }
      }
    }
  }

  // neither CTA of a pair leaves while the other may still reach its shared
  // memory or tensor memory (barrier arrivals, MMA operand reads, scale copies)
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();
  if (warp == 0) {
    tc_fence_after();
    if constexpr (PAIR)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTmemCols)
                   : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTmemCols)
                   : "memory");
  }
}

// ------------------------------------------------------------------ host

struct GroupMaps {
  CUtensorMap a, b, sfa, sfb;
  RowMaps rows;                // rows: A
};

template <auto Kernel>
uint32_t max_group_clusters(size_t smem) {
  static std::atomic<int> cached[256];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 256) dev = 0;
  int n = cached[dev].load(std::memory_order_relaxed);
  if (n > 0) return uint32_t(n);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * 256);
  cfg.blockDim = dim3(kGroupThreads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, Kernel, &cfg) != cudaSuccess || n <= 0) {
    (void)cudaGetLastError();
    n = sm_count() / 2;
  }
  cached[dev].store(n, std::memory_order_relaxed);
  return uint32_t(n);
}

// Launches a persistent kernel of pairs (or of single CTAs) for at most `most` output tiles.
template <auto Kernel, bool PAIR, typename... Args>
mxq_status launch_group(uint32_t smem, uint64_t most, cudaStream_t s, const Args&... args) {
  const cudaError_t attr_err = ensure_smem_limit<Kernel>(int(smem));
  if (attr_err != cudaSuccess) {
    record_cuda_error(attr_err);
    return MXQ_ERR_CUDA;
  }
  const uint64_t resident = PAIR ? max_group_clusters<Kernel>(smem) : uint64_t(sm_count());
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(uint32_t(std::min(most, resident)) * (PAIR ? 2 : 1));
  cfg.blockDim = dim3(kGroupThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = PAIR ? 2 : 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return launched(cudaLaunchKernelEx(&cfg, Kernel, args...));
}

template <bool SWIGLU, bool FEW, typename OutT>
mxq_status launch_rows(const GroupMaps& m, const GroupArgs& args, uint64_t most, cudaStream_t s) {
  return launch_group<mxfp8_rows_kernel<SWIGLU, FEW, OutT>, true>(RowCfg<SWIGLU, FEW>::kSmem, most, s, m.b, m.rows,
                                                                   m.sfb, m.sfa, args);
}

template <typename OutT>
mxq_status launch_rows(const GroupMaps& m, const GroupArgs& args, bool swiglu, uint64_t active, cudaStream_t s) {
  const bool few = args.rows <= RowCfg<false, true>::kTile;
  // tiles that the experts with rows can have
  const uint64_t most = (few ? active : args.rows / RowCfg<false, false>::kTile + active) * args.tiles_n;
  if (few) return swiglu ? launch_rows<true, true, OutT>(m, args, most, s) : launch_rows<false, true, OutT>(m, args, most, s);
  return swiglu ? launch_rows<true, false, OutT>(m, args, most, s) : launch_rows<false, false, OutT>(m, args, most, s);
}

template <bool PAIR, typename OutT>
mxq_status launch_wgrad(const GroupMaps& m, const GroupArgs& args, uint64_t most, cudaStream_t s) {
  return launch_group<mxfp8_wgrad_kernel<PAIR, OutT>, PAIR>(TileCfg<PAIR>::kSmem, most, s, m.a, m.b, m.sfa, m.sfb, args);
}

}  // namespace
}  // namespace mxq

extern "C" {

int64_t mxq_grouped_padded_rows(int32_t E, int64_t M_total) {
  if (E < 0 || M_total < 0) return -1;
  return (M_total + 127 * int64_t(E)) / 128 * 128;
}

mxq_status mxfp8_gemm_grouped(const uint8_t* qa, const uint8_t* sa_swz, int64_t sa_bytes, const uint8_t* qb,
                              const uint8_t* sb_swz, int32_t E, const int64_t* row_offsets, int64_t M,
                              int64_t N, int64_t K, int swiglu, void* d, int out_dt, int32_t* error_flag,
                              mxq_stream_t stream) {
  using namespace mxq;
  if (!valid_dtype(out_dt)) return MXQ_ERR_DTYPE;
  if (swiglu != 0 && swiglu != 1) return MXQ_ERR_ARG;
  if (E < 1 || E > MXQ_GROUPED_MAX_EXPERTS) return MXQ_ERR_SHAPE;
  if (M < 0 || N < 0 || K < 0 || sa_bytes < 0 || K % 32 != 0 || N % (swiglu ? 256 : 16) != 0)
    return MXQ_ERR_SHAPE;
  // coordinates of the loads and the list of tiles are counted in 32 bits
  constexpr int64_t kMost = 0x7fffff00ll;
  if (M > kMost || N > kMost || K > kMostSum || N * E > kMost) return MXQ_ERR_SHAPE;
  const int64_t kp4 = (K + 127) / 128, nb128 = (N + 127) / 128;
  if ((M / 128 + E + 1) * kp4 > kMost / 4 || nb128 * E * kp4 > kMost / 4) return MXQ_ERR_SHAPE;
  if ((M / 128 + E) * ((N + 127) / 128) > kMost) return MXQ_ERR_SHAPE;
  if (M == 0 || N == 0) return MXQ_OK;
  if (!d || !row_offsets) return MXQ_ERR_NULL;
  if (!aligned16(d) || (reinterpret_cast<uintptr_t>(row_offsets) & 7u)) return MXQ_ERR_ALIGN;
  GroupArgs args{};
  GroupMaps maps;
  std::memset(&maps, 0, sizeof(maps));
  args.offsets = row_offsets;
  args.d = d;
  args.err = error_flag;
  args.E = uint32_t(E);
  args.rows = uint32_t(M);
  args.n = uint32_t(swiglu ? N / 2 : N);
  args.b_rows = uint32_t(N);
  args.nk = args.kp4 = uint32_t(kp4);
  args.nb128 = uint32_t(nb128);
  args.sfw = sb_swz;
  // experts that can have rows, and the tiles that they can have
  const uint64_t active = uint64_t(std::min<int64_t>(E, M));
  if (K > 0) {
    if (!qa || !qb || !sa_swz || !sb_swz) return MXQ_ERR_NULL;
    if (!aligned16(qa) || !aligned16(qb) || !aligned16(sa_swz) || !aligned16(sb_swz)) return MXQ_ERR_ALIGN;
    // the blocks of no more than M rows, whatever the experts' padding
    if (sa_bytes < (M + 127) / 128 * kp4 * int64_t(kSfTile) || sa_bytes % int64_t(kSfTile) != 0) return MXQ_ERR_SHAPE;
    for (int b = 0; b < 4; b++)
      if (!make_operand_map(&maps.rows.box[b], qa, uint64_t(M), uint64_t(K), 128u >> b)) return MXQ_ERR_CUDA;
    if (!make_operand_map(&maps.b, qb, uint64_t(N) * E, uint64_t(K), swiglu ? 64 : 128) ||
        !make_scale_map(&maps.sfa, sa_swz, uint64_t(sa_bytes)) ||
        !make_scale_map(&maps.sfb, sb_swz, uint64_t(nb128) * E * kp4 * kSfTile))
      return MXQ_ERR_CUDA;
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  args.tiles_n = uint32_t((N + 255) / 256);               // swiglu: 128 rows of each half
  return out_dt == MXQ_BF16 ? launch_rows<uint16_t>(maps, args, swiglu != 0, active, s)
                            : launch_rows<float>(maps, args, swiglu != 0, active, s);
}

mxq_status mxfp8_gemm_grouped_wgrad(const uint8_t* qa_t, const uint8_t* sa_swz, const uint8_t* qb_t,
                                    const uint8_t* sb_swz, int32_t E, const int64_t* row_offsets, int64_t P,
                                    int64_t Na, int64_t Nb, void* d, int out_dt, int32_t* error_flag,
                                    mxq_stream_t stream) {
  using namespace mxq;
  if (!valid_dtype(out_dt)) return MXQ_ERR_DTYPE;
  if (E < 1 || E > MXQ_GROUPED_MAX_EXPERTS) return MXQ_ERR_SHAPE;
  if (P < 0 || Na < 0 || Nb < 0 || P % 128 != 0 || Nb % 16 != 0) return MXQ_ERR_SHAPE;
  constexpr int64_t kMost = 0x7fffff00ll;
  if (P > kMostSum || Na > kMost || Nb > kMost) return MXQ_ERR_SHAPE;
  const int64_t kp4 = P / 128;
  if ((Na + 127) / 128 * kp4 > kMost / 4 || (Nb + 127) / 128 * kp4 > kMost / 4) return MXQ_ERR_SHAPE;
  const bool pair = Na > 128 && Nb > 128;
  const int64_t rows = pair ? 256 : 128, bn = pair ? 256 : 128;
  const int64_t tiles_m = (Na + rows - 1) / rows, tiles_n = (Nb + bn - 1) / bn;
  if (tiles_m * tiles_n > kMost / E) return MXQ_ERR_SHAPE;
  if (Na == 0 || Nb == 0) return MXQ_OK;
  if (!d || !row_offsets) return MXQ_ERR_NULL;
  if (!aligned16(d) || (reinterpret_cast<uintptr_t>(row_offsets) & 7u)) return MXQ_ERR_ALIGN;
  GroupArgs args{};
  GroupMaps maps;
  std::memset(&maps, 0, sizeof(maps));
  if (P > 0) {
    if (!qa_t || !qb_t || !sa_swz || !sb_swz) return MXQ_ERR_NULL;
    if (!aligned16(qa_t) || !aligned16(qb_t) || !aligned16(sa_swz) || !aligned16(sb_swz)) return MXQ_ERR_ALIGN;
    if (!make_operand_map(&maps.a, qa_t, uint64_t(Na), uint64_t(P), 128) ||
        !make_operand_map(&maps.b, qb_t, uint64_t(Nb), uint64_t(P), 128) ||
        !make_scale_map(&maps.sfa, sa_swz, uint64_t((Na + 127) / 128 * kp4) * kSfTile) ||
        !make_scale_map(&maps.sfb, sb_swz, uint64_t((Nb + 127) / 128 * kp4) * kSfTile))
      return MXQ_ERR_CUDA;
  }
  args.offsets = row_offsets;
  args.d = d;
  args.err = error_flag;
  args.E = uint32_t(E);
  args.rows = uint32_t(P);
  args.rows_a = uint32_t(Na);
  args.n = uint32_t(Nb);
  args.kp4 = uint32_t(kp4);
  args.tiles_m = uint32_t(tiles_m);
  args.tiles_n = uint32_t(tiles_n);
  const uint64_t most = uint64_t(tiles_m) * uint64_t(tiles_n) * uint64_t(E);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (out_dt == MXQ_BF16)
    return pair ? launch_wgrad<true, uint16_t>(maps, args, most, s) : launch_wgrad<false, uint16_t>(maps, args, most, s);
  return pair ? launch_wgrad<true, float>(maps, args, most, s) : launch_wgrad<false, float>(maps, args, most, s);
}

}  // extern "C"
