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
// One kernel, three shapes of tile:
//  - PAIR: 256 x 256 over a cluster of two CTAs (tcgen05 cta_group::2), six
//    stages of 32 KiB and 1.5 KiB of scales in each CTA;
//  - 128 x 256 and 128 x 128 in one CTA, four and six stages.
// Warps: 0 loads (TMA), 1 issues the MMAs, 2-9 are the epilogue: two warps a
// quarter of the accumulator's lanes, each with half of its columns. Each
// takes its columns into registers in one go (at most 128 fp32), hands the
// accumulator back, and does everything else (SwiGLU, rounding, stores)
// while the next tile's MMAs run: tensor memory has no room for a second
// accumulator beside the scales.
//  - SWIGLU: the B tile is 128 rows of the gate and the 128 rows of the up
//    half with the same places (the pair's CTAs load one each), so a thread
//    holds both factors of its outputs: D[r, h] = silu(gate) up is written
//    and the halves never are.
//
// Waits are bounded as in mxfp8_gemm.cu.
#include "common.cuh"
#include "mxf8_mma.cuh"

namespace mxq {
namespace {

constexpr int kEpiWarps = 8;
constexpr int kGroupThreads = 32 * (2 + kEpiWarps);
// staging of a warp's bf16 stores: 32 rows x 32 columns (64 bytes), pitch 80
constexpr uint32_t kSlicePitch = 80;
constexpr uint32_t kSliceBytes = 32 * kSlicePitch;
constexpr uint32_t kBarrierBytes = 256;

template <bool PAIR, int BN>
struct TileCfg {
  static constexpr uint32_t kRows = PAIR ? 256 : 128;                  // output rows of a tile
  static constexpr uint32_t kBRows = PAIR ? 128 : BN;                  // rows of B that a CTA loads
  static constexpr int kStages = PAIR || BN == 128 ? 6 : 4;
  static constexpr uint32_t kTileA = 128 * kBK, kTileB = kBRows * kBK;
  static constexpr uint32_t kOperands = kTileA + kTileB;               // a multiple of 1 KiB
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

// An output tile's place: all lanes of a warp hold the same.
struct Place {
  uint32_t expert;
  uint32_t a_row, a_block;     // first row of A (rows) or of the tile along Na (wgrad), its 128-row scale block
  uint32_t n_blk;
  uint32_t kb0, nk;            // K blocks
  uint32_t left;               // rows of D from the tile's first one on
  uint64_t d_row;              // D's row of the tile's first one
};

// rows: the tile t of the list (rising from call to call); false behind the last.
template <uint32_t ROWS>
__device__ __forceinline__ bool find_rows(const GroupArgs& a, ExpertCursor& c, uint32_t t, uint32_t lane,
                                          Place& p) {
  for (;;) {
    const uint32_t hit = __ballot_sync(kFull, uint64_t(c.tiles) * a.tiles_n > t);
    if (hit) {
      const int j = __ffs(hit) - 1;
      const uint32_t incl = __shfl_sync(kFull, c.tiles, j), off0 = __shfl_sync(kFull, c.off0, j),
                     off1 = __shfl_sync(kFull, c.off1, j), blocks = __shfl_sync(kFull, c.blocks, j);
      const uint32_t n = off1 - off0, tm = (n + ROWS - 1) / ROWS;
      const uint32_t local = t - (incl - tm) * a.tiles_n;
      // row tiles first: neighbouring CTAs read the same rows of B
      const uint32_t m = local % tm;
      p.n_blk = local / tm;
      p.expert = c.first + j;
      p.a_row = off0 + m * ROWS;
      p.a_block = blocks - (n + 127) / 128 + m * (ROWS / 128);
      p.kb0 = 0;
      p.nk = a.nk;
      p.left = n - m * ROWS;
      p.d_row = p.a_row;
      return true;
    }
    if (c.first + 32 >= c.E) return false;
    c.advance(lane);
  }
}

// wgrad: every expert has the same tiles; what differs is where its columns lie.
template <uint32_t ROWS>
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
  const uint32_t m = rest % a.tiles_m;
  p.n_blk = rest / a.tiles_m;
  p.expert = e;
  p.a_row = m * ROWS;
  p.a_block = m * (ROWS / 128);
  p.kb0 = min(blocks - nk, total);
  p.nk = min(nk, total - p.kb0);
  p.left = a.rows_a - m * ROWS;
  p.d_row = uint64_t(e) * a.rows_a + m * ROWS;
  return true;
}

// silu(g) u = g u / (1 + e^-g). For g < 0 as (g t) (u t) / (1 + t^2) with t =
// e^(g/2): e^-g has no fp32 value from -88.8 on where silu still has one, and a
// large u brings back what lies below. The divisor is in [1, 2], where the
// approximate division is off by at most 2 ulps.
__device__ __forceinline__ float swiglu(float g, float u) {
  const float t = expf(-0.5f * fabsf(g));
  if (g < 0.f) {
    g *= t;
    u *= t;
  }
  return __fdividef(g, 1.f + t * t) * u;
}

template <bool PAIR, int BN, bool WGRAD, bool SWIGLU, typename OutT>
__global__ void __launch_bounds__(kGroupThreads, 1)
mxfp8_group_kernel(const __grid_constant__ CUtensorMap tma_a, const __grid_constant__ CUtensorMap tma_b,
                   const __grid_constant__ CUtensorMap tma_sfa,
                   const __grid_constant__ CUtensorMap tma_sfb, const __grid_constant__ GroupArgs a) {
  using C = TileCfg<PAIR, BN>;
  static_assert(!SWIGLU || BN == 256, "halves of 128 columns");
  constexpr int kStages = C::kStages;
  constexpr uint32_t kOutCols = SWIGLU ? BN / 2 : BN;     // columns of D in a tile
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

  ExpertCursor cursor;
  cursor.start(a.offsets, a.E, WGRAD ? 0x7fffff00u : a.rows, C::kRows, lane);
  auto find = [&](Place& p) {
    if constexpr (WGRAD)
      return find_wgrad<C::kRows>(a, cursor, tile, lane, p);
    else
      return find_rows<C::kRows>(a, cursor, tile, lane, p);
  };
  Place p;

  if (warp == 0) {
    // ---------------------------------------------------------- producer
    const uint32_t bar0 = PAIR ? cluster_addr(full_bar(0), 0) : full_bar(0);
    auto load = [&](uint32_t dst, const CUtensorMap* map, uint32_t bar, uint32_t x, uint32_t y) {
      if constexpr (PAIR)
        tma_load_2d_pair(dst, map, bar, int32_t(x), int32_t(y));
      else
        tma_load_2d(dst, map, bar, int32_t(x), int32_t(y));
    };
    uint32_t s = 0, phase = 1;
    for (; find(p); tile += step) {
      bool ok = true;
      if (lane == 0) {
        // rows of B of this CTA's box(es) and the 128-row blocks of its scale tiles
        uint32_t b_row, b_row1 = 0, b_blk, b_blk1;
        if constexpr (WGRAD) {
          b_row = p.n_blk * BN + (PAIR ? 128 * rank : 0);
          b_blk = p.n_blk * C::kSfbTiles;
          b_blk1 = b_blk + 1;
        } else if constexpr (SWIGLU) {
          const uint32_t gate = p.expert * a.b_rows + p.n_blk * 128, up = gate + a.n;
          b_row = rank == 0 ? gate : up;
          b_row1 = up;
          b_blk = p.expert * a.nb128 + p.n_blk;
          b_blk1 = b_blk + a.n / 128;
        } else {
          b_row = p.expert * a.b_rows + p.n_blk * BN + (PAIR ? 128 * rank : 0);
          b_blk = p.expert * a.nb128 + p.n_blk * C::kSfbTiles;
          b_blk1 = b_blk + 1;
        }
        const uint32_t a_row = p.a_row + 128 * rank, a_blk = p.a_block + rank;
        for (uint32_t i = 0; i < p.nk; i++) {
          if (!mbar_wait(empty_bar(s), phase, kWaitNs)) {
            record_error(a.err, kErrEmptyWait);
            ok = false;
            break;
          }
          if (rank == 0) mbar_expect_tx(full_bar(s), (PAIR ? 2 : 1) * C::kStageTx);
          const uint32_t kb = p.kb0 + i, bar = bar0 + 8u * s;
          const uint32_t st = base + s * C::kOperands, sf = scales + s * C::kScales;
          load(st, &tma_a, bar, kb * kBK, a_row);
          load(st + C::kTileA, &tma_b, bar, kb * kBK, b_row);
          if constexpr (SWIGLU && !PAIR) load(st + C::kTileA + 128 * kBK, &tma_b, bar, kb * kBK, b_row1);
          load(sf, &tma_sfa, bar, 0, 4 * (a_blk * a.kp4 + kb));
          load(sf + kSfTile, &tma_sfb, bar, 0, 4 * (b_blk * a.kp4 + kb));
          if constexpr (C::kSfbTiles == 2)
            load(sf + 2 * kSfTile, &tma_sfb, bar, 0, 4 * (b_blk1 * a.kp4 + kb));
          if (++s == kStages) {
            s = 0;
            phase ^= 1u;
          }
        }
      }
      if (!__shfl_sync(kFull, int(ok), 0)) break;
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
      for (; find(p); tile += step) {
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
#pragma unroll
          for (uint32_t j = 0; j <= C::kSfbTiles; j++) {   // B's tiles first, then A's
            const uint32_t w = j == C::kSfbTiles ? 0 : j + 1;
            if constexpr (PAIR)
              tmem_copy_scales_pair(sfa_t + 4u * w, sc + kSfW * w, sc_hi);
            else
              tmem_copy_scales(sfa_t + 4u * w, sc + kSfW * w, sc_hi);
          }
#pragma unroll
          for (uint32_t k = 0; k < 4; k++) {
            if constexpr (PAIR)
              mma_mxf8_pair(tmem, op_lo + so + 2 * k, op_lo + so + kTileAW + 2 * k, op_hi, instr_desc_pair(k),
                            sfa_t | (k << 30), sfb_t | (k << 30), (i | k) != 0u);
            else
              mma_mxf8(tmem, op_lo + so + 2 * k, op_lo + so + kTileAW + 2 * k, op_hi, instr_desc<BN>(k),
                       sfa_t | (k << 30), sfb_t | (k << 30), (i | k) != 0u);
          }
          if constexpr (PAIR)
            mma_commit_pair(empty_bar(s));
          else
            mma_commit(empty_bar(s));
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
    // the second four take the second half of the columns (SWIGLU: of each
    // half's columns)
    constexpr int kCols = BN / 2;                                     // accumulator columns of a warp
    constexpr uint32_t kOut = kOutCols / 2;                           // columns of D of a warp
    const uint32_t quarter = warp & 3, half = (warp - 2) >> 2;
    const uint32_t taddr = tmem + ((quarter * 32) << 16);
    const uint32_t slice = bars + kBarrierBytes + kSliceBytes * (warp - 2);
    const uint32_t lead_acc_empty = PAIR ? cluster_addr(acc_empty, 0) : acc_empty;
    uint32_t done = 0;
    for (; find(p); tile += step) {
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
          tmem_ld32_start(taddr + (SWIGLU ? (c < 64 ? 64 * half + c : 128 + 64 * half + c - 64) : kCols * half + c),
                          *reinterpret_cast<uint32_t(*)[32]>(&v[c]));
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
      if constexpr (SWIGLU) {
#pragma unroll
        for (int c = 0; c < 64; c++)
          v[c] = __float_as_uint(swiglu(__uint_as_float(v[c]), __uint_as_float(v[c + 64])));
      }
      const uint32_t r0 = 128 * rank + 32 * quarter;                  // the warp's first row of the tile
      if (r0 >= p.left) continue;
      const uint32_t rows = min(32u, p.left - r0);
      const uint32_t col0 = p.n_blk * kOutCols + kOut * half;
      if (col0 >= a.n) continue;
      const uint32_t cols = min(kOut, a.n - col0);                    // a multiple of 16
      OutT* d = static_cast<OutT*>(a.d) + (p.d_row + r0) * a.n + col0;
      if constexpr (sizeof(OutT) == 2) {
        // 32-column slices through the warp's staging rows, so that a store
        // instruction writes 64 bytes of each of eight rows
        const uint32_t rsub = lane >> 2, ch = lane & 3;
#pragma unroll
        for (uint32_t c0 = 0; c0 < kOut; c0 += 32) {
#pragma unroll
          for (int q = 0; q < 4; q++) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; i++)
              w[i] = cvt_bf16x2(__uint_as_float(v[c0 + 8 * q + 2 * i]), __uint_as_float(v[c0 + 8 * q + 2 * i + 1]));
            sts128_u32(slice + lane * kSlicePitch + 16 * q, make_uint4(w[0], w[1], w[2], w[3]));
          }
          __syncwarp();
          const uint32_t col = c0 + 8 * ch;
#pragma unroll
          for (uint32_t j = 0; j < 4; j++) {
            const uint32_t rr = 8 * j + rsub;
            const uint4 x = lds128_u32(slice + rr * kSlicePitch + 16 * ch);
            if (rr < rows && col < cols) st_v4(d + uint64_t(rr) * a.n + col, x);
          }
          __syncwarp();
        }
      } else {
        if (lane < rows) {
          OutT* drow = d + uint64_t(lane) * a.n;
#pragma unroll
          for (uint32_t c = 0; c < kOut; c += 4)
            if (c < cols) st_v4(drow + c, make_uint4(v[c], v[c + 1], v[c + 2], v[c + 3]));
        }
        __syncwarp();
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

// `most`: an upper bound of the output tiles.
template <bool PAIR, int BN, bool WGRAD, bool SWIGLU, typename OutT>
mxq_status launch_group(const GroupMaps& m, const GroupArgs& args, uint64_t most, cudaStream_t s) {
  constexpr auto kernel = mxfp8_group_kernel<PAIR, BN, WGRAD, SWIGLU, OutT>;
  constexpr uint32_t smem = TileCfg<PAIR, BN>::kSmem;
  const cudaError_t attr_err = ensure_smem_limit<kernel>(int(smem));
  if (attr_err != cudaSuccess) {
    record_cuda_error(attr_err);
    return MXQ_ERR_CUDA;
  }
  const uint64_t resident = PAIR ? max_group_clusters<kernel>(smem) : uint64_t(sm_count());
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(uint32_t(std::min(most, resident)) * (PAIR ? 2 : 1));
  cfg.blockDim = dim3(kGroupThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = PAIR ? 2 : 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return launched(cudaLaunchKernelEx(&cfg, kernel, m.a, m.b, m.sfa, m.sfb, args));
}

template <bool PAIR, int BN, bool WGRAD, bool SWIGLU>
mxq_status launch_group(const GroupMaps& m, const GroupArgs& args, uint64_t most, int out_dt, cudaStream_t s) {
  return out_dt == MXQ_BF16 ? launch_group<PAIR, BN, WGRAD, SWIGLU, uint16_t>(m, args, most, s)
                            : launch_group<PAIR, BN, WGRAD, SWIGLU, float>(m, args, most, s);
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
  if (M > kMost || N > kMost || K > kMost || N * E > kMost) return MXQ_ERR_SHAPE;
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
  // experts that can have rows, and the tiles that they can have
  const uint64_t active = uint64_t(std::min<int64_t>(E, M));
  const bool pair = M > 128 * int64_t(E);
  const uint32_t sms = uint32_t(sm_count());
  const bool narrow = !pair && !swiglu && active * ((uint64_t(N) + 255) / 256) < sms;
  const uint32_t bn = narrow ? 128 : 256;
  if (K > 0) {
    if (!qa || !qb || !sa_swz || !sb_swz) return MXQ_ERR_NULL;
    if (!aligned16(qa) || !aligned16(qb) || !aligned16(sa_swz) || !aligned16(sb_swz)) return MXQ_ERR_ALIGN;
    // the blocks of no more than M rows, whatever the experts' padding
    if (sa_bytes < (M + 127) / 128 * kp4 * int64_t(kSfTile) || sa_bytes % int64_t(kSfTile) != 0) return MXQ_ERR_SHAPE;
    if (!make_operand_map(&maps.a, qa, uint64_t(M), uint64_t(K), 128) ||
        !make_operand_map(&maps.b, qb, uint64_t(N) * E, uint64_t(K), pair || swiglu ? 128u : bn) ||
        !make_scale_map(&maps.sfa, sa_swz, uint64_t(sa_bytes)) ||
        !make_scale_map(&maps.sfb, sb_swz, uint64_t(nb128) * E * kp4 * kSfTile))
      return MXQ_ERR_CUDA;
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  args.tiles_n = swiglu ? uint32_t(N / 256) : uint32_t((N + bn - 1) / bn);
  const uint64_t rows = pair ? 256 : 128;
  const uint64_t most = (uint64_t(M) / rows + active) * args.tiles_n;
  if (pair)
    return swiglu ? launch_group<true, 256, false, true>(maps, args, most, out_dt, s)
                  : launch_group<true, 256, false, false>(maps, args, most, out_dt, s);
  if (swiglu) return launch_group<false, 256, false, true>(maps, args, most, out_dt, s);
  return narrow ? launch_group<false, 128, false, false>(maps, args, most, out_dt, s)
                : launch_group<false, 256, false, false>(maps, args, most, out_dt, s);
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
  if (P > kMost || Na > kMost || Nb > kMost) return MXQ_ERR_SHAPE;
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
  return pair ? launch_group<true, 256, true, false>(maps, args, most, out_dt, s)
              : launch_group<false, 128, true, false>(maps, args, most, out_dt, s);
}

}  // extern "C"
