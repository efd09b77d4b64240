// norm.cu -- root-mean-square norm of rows with the residual's addition, its
// output quantized to MXFP8 in the same pass, and the norm's gradient, for
// sm_100a.
//
//   h = x (+ residual, rounded to x's type), rstd = fp32(1 / sqrt(mean(h^2) + eps))
//   y = fp32(fp32(h rstd) weight), codes and scales of y by mx_rowwise.cu's rule
//
// The squares are added up in fp64 (the square of a bf16 or fp32 value leaves
// fp32's range long before the value does), and the root's reciprocal is one of
// fp64 (an ulp or two), so that rstd is the correctly rounded fp32 number but
// where fp64 leaves it on a border, and every step after it is one IEEE
// operation: codes and scales are functions of the inputs' bits whatever the
// order of the sum.
//
// Gradient: dx = grad_hidden + rstd (g w - xh mean(g w xh)) with xh = h rstd,
// dweight = sum over the rows of g xh.
#include "common.cuh"

namespace mxq {
namespace {

// ------------------------------------------------------------- forward
//
// HBM-bound: per bf16 element 2 bytes read (4 with a residual), 1 + 1/32
// written (3 + 1/32). A row lies in the registers of its warps: a lane owns 16
// consecutive elements (a 256-bit load of bf16), two lanes a group of 32, C
// such pieces a lane; the warps of a row exchange their sums through shared
// memory once. Small rows share a CTA. Rows of more than 32 * 1024 elements are
// read twice instead (LOOP), the second time from L2.
// 16384 x 7168 bf16 with a residual 125 us (127 at the copy rate); without one
// 87-91 (54), where a row's chain of load, sum, barrier and codes bounds it, at
// the four rows a multiprocessor that 64 registers a thread allow (the bound of
// 1024 threads that every form is compiled for). 4096 x 65536 bf16 with a residual
// in rows read twice 318 us (207).

struct NormArgs {
  const void* x;
  const void* residual;
  const void* weight;
  void* hidden;
  uint8_t* q;
  uint8_t* scale;
  uint8_t* swz;
  void* normed;
  float* rstd;
  int64_t ld_x, ld_res;
  int64_t M;
  uint32_t N;
  uint32_t S4;            // ceil(N / 128)
  uint32_t row_threads;   // threads of a row, a multiple of 32
  uint32_t row_ctas;      // CTAs with rows
  double eps, inv_n;      // inv_n = 1 / N
  int weight_bf16;
  bool weight_v8;         // the weights lie on a 32-byte boundary
  bool v8;                // x, residual, hidden and normed: rows on 32-byte boundaries
  bool scale_words;       // compact scales can be written as words
};

// As In16::load, by plain loads: hidden may be x or residual itself, and LOOP
// reads what this thread has written.
template <typename T>
__device__ __forceinline__ void load16(In16<T>& v, const T* p, bool v8) {
  constexpr int kWords = sizeof(v.w) / 4;
  if (v8) {
#pragma unroll
    for (int i = 0; i < kWords; i += 8)
      asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(v.w[i]), "=r"(v.w[i + 1]), "=r"(v.w[i + 2]), "=r"(v.w[i + 3]), "=r"(v.w[i + 4]),
                     "=r"(v.w[i + 5]), "=r"(v.w[i + 6]), "=r"(v.w[i + 7])
                   : "l"(reinterpret_cast<const uint32_t*>(p) + i));
  } else {
#pragma unroll
    for (int i = 0; i < kWords; i += 4)
      asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(v.w[i]), "=r"(v.w[i + 1]), "=r"(v.w[i + 2]), "=r"(v.w[i + 3])
                   : "l"(reinterpret_cast<const uint32_t*>(p) + i));
  }
}

template <typename T>
__device__ __forceinline__ void store16(T* p, const In16<T>& v, bool v8) {
  constexpr int kWords = sizeof(v.w) / 4;
  uint32_t* o = reinterpret_cast<uint32_t*>(p);
#pragma unroll
  for (int i = 0; i < kWords; i += 8) {
    if (v8) {
      const uint32_t w[8] = {v.w[i], v.w[i + 1], v.w[i + 2], v.w[i + 3], v.w[i + 4], v.w[i + 5], v.w[i + 6], v.w[i + 7]};
      st_v8(o + i, w);
    } else {
      st_v4(o + i, make_uint4(v.w[i], v.w[i + 1], v.w[i + 2], v.w[i + 3]));
      st_v4(o + i + 4, make_uint4(v.w[i + 4], v.w[i + 5], v.w[i + 6], v.w[i + 7]));
    }
  }
}

__device__ __forceinline__ void set_pair(In16<uint16_t>& v, int k, float lo, float hi) { v.w[k] = cvt_bf16x2(lo, hi); }
__device__ __forceinline__ void set_pair(In16<float>& v, int k, float lo, float hi) {
  v.w[2 * k] = __float_as_uint(lo);
  v.w[2 * k + 1] = __float_as_uint(hi);
}

// Rounded to T and back in registers: h = x + residual.
template <typename T>
__device__ __forceinline__ void add16(In16<T>& v, const In16<T>& r) {
#pragma unroll
  for (int k = 0; k < 8; k++) set_pair(v, k, v.lo(k) + r.lo(k), v.hi(k) + r.hi(k));
}

template <typename T>
__device__ __forceinline__ double squares(const In16<T>& v) {
  double s = 0.0;
#pragma unroll
  for (int k = 0; k < 8; k++) {
    const double a = double(v.lo(k)), b = double(v.hi(k));
    s = fma(a, a, s);
    s = fma(b, b, s);
  }
  return s;
}

// 16 weights, as they lie in memory. fp32 ones by 32 bytes a load where they
// lie on such boundaries: a warp's load by 16 touches as many lines for half of
// them (16384 x 7168 bf16 115 us, so 100). bf16 ones are not faster so.
template <bool WB>
struct Weights16 {
  static constexpr int kWords = WB ? 8 : 16;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const NormArgs& a, uint32_t c) {
    const uint32_t* p = static_cast<const uint32_t*>(a.weight) + uint64_t(c >> 4) * kWords;
    if (!WB && a.weight_v8) {
#pragma unroll
      for (int i = 0; i < kWords; i += 8)
        asm("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
            : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3]), "=r"(w[i + 4]), "=r"(w[i + 5]),
              "=r"(w[i + 6]), "=r"(w[i + 7])
            : "l"(p + i));
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 q = __ldg(reinterpret_cast<const uint4*>(p + i));
        w[i] = q.x; w[i + 1] = q.y; w[i + 2] = q.z; w[i + 3] = q.w;
      }
    }
  }
  __device__ __forceinline__ float2 pair(int k) const {
    return WB ? make_float2(bf16_lo(w[k]), bf16_hi(w[k]))
              : make_float2(__uint_as_float(w[2 * k % kWords]), __uint_as_float(w[(2 * k + 1) % kWords]));
  }
};

// y of 16 elements of a row, their codes, the group's scale (two lanes a
// group, both or neither of them active; the lanes of a warp call together) and, where asked for, y itself.
template <typename T, bool WB>
__device__ __forceinline__ void finish16(const NormArgs& a, const In16<T>& h, const Weights16<WB>& w, int64_t row,
                                         uint32_t c, float rstd, bool active) {
  const uint32_t lane = threadIdx.x & 31;
  float2 y[8];
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < 8; k++) {
    y[k] = mul2v(mul2(h.lo(k), h.hi(k), rstd), w.pair(k));
    amax = fmaxf(amax, fmaxf(fabsf(y[k].x), fabsf(y[k].y)));   // NaN raises no maximum
  }
  amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
  const uint32_t b = mx_scale_byte<8>(amax);
  const float mul = pow2_quant(b);
  uint32_t code[8];
#pragma unroll
  for (int k = 0; k < 8; k++) {
    const float2 u = mul2(y[k].x, y[k].y, mul);
    code[k] = cvt_e4m3x2(u.x, u.y);
  }
  // a word of the row's next four groups in every eighth lane; groups past N are zeros
  uint32_t word = active ? b : 0;
  word |= __shfl_down_sync(kFull, word, 2) << 8;
  word |= __shfl_down_sync(kFull, word, 4) << 16;
  if (!active) return;
  st_v4(a.q + row * a.N + c,
        make_uint4(__byte_perm(code[0], code[1], 0x5410), __byte_perm(code[2], code[3], 0x5410),
                   __byte_perm(code[4], code[5], 0x5410), __byte_perm(code[6], code[7], 0x5410)));
  const uint32_t g = c >> 5;
  uint8_t* s = a.scale + row * (a.N >> 5) + g;
  if (a.scale_words) {
    if ((lane & 7) == 0) st_u32(s, word);
  } else if ((lane & 1) == 0) {
    st_u8(s, b);
  }
  if (a.swz && (lane & 7) == 0)
    st_u32(a.swz + (((uint64_t(row) >> 7) * a.S4 + (g >> 2)) << 9) + ((row & 31) << 4) + (((row >> 5) & 3) << 2), word);
  if (a.normed) {
    In16<T> o;
#pragma unroll
    for (int k = 0; k < 8; k++) set_pair(o, k, y[k].x, y[k].y);
    store16(static_cast<T*>(a.normed) + row * a.N + c, o, a.v8);
  }
}

// The scale tiles' rows past M are zeros: a warp a row, of CTAs behind those of the rows.
__device__ __forceinline__ void pad_tiles(const NormArgs& a, uint32_t cta) {
  const int64_t r = a.M + int64_t(cta) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (r >= ((a.M + 127) & ~int64_t(127))) return;
  uint8_t* p = a.swz + ((uint64_t(r) >> 7) * a.S4 << 9) + ((r & 31) << 4) + (((r >> 5) & 3) << 2);
  for (uint32_t j = threadIdx.x & 31; j < a.S4; j += 32) st_u32(p + (uint64_t(j) << 9), 0);
}

template <typename T, bool RES, bool WB, int C, bool LOOP>
__global__ void __launch_bounds__(1024) mxfp8_rmsnorm_kernel(const __grid_constant__ NormArgs a) {
  pdl_enter();
  if (blockIdx.x >= a.row_ctas) return pad_tiles(a, blockIdx.x - a.row_ctas);
  __shared__ double sums[32];
  __shared__ float rstds[32];
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t row_warps = a.row_threads >> 5, sub = warp / row_warps;
  const uint32_t rows = (blockDim.x >> 5) / row_warps;                 // rows of a CTA
  const uint32_t t = threadIdx.x - sub * a.row_threads;
  const int64_t row = int64_t(blockIdx.x) * rows + sub;
  const bool have = row < a.M;
  const T* x = static_cast<const T*>(a.x) + row * a.ld_x;
  const T* res = static_cast<const T*>(a.residual) + (RES ? row * a.ld_res : 0);
  T* hidden = static_cast<T*>(a.hidden) + (RES ? row * int64_t(a.N) : 0);

  // the first piece's weights are asked for before the row's sum is known where
  // the registers have room for them (16384 x 7168 98 us, so 90) and a row has
  // work to hide the rest (32768 x 2048, one piece, 57 and 59)
  constexpr bool kEarly = sizeof(T) == 2 && WB && C == 2;
  In16<T> v[C];
  Weights16<WB> w;
  double ss = 0.0;
  if constexpr (LOOP) {
    for (uint32_t c = t * 16; have && c < a.N; c += a.row_threads * 16) {
      load16(v[0], x + c, a.v8);
      if constexpr (RES) {
        In16<T> r;
        load16(r, res + c, a.v8);
        add16(v[0], r);
        store16(hidden + c, v[0], a.v8);
      }
      ss += squares(v[0]);
    }
  } else {
    In16<T> r[C];
#pragma unroll
    for (int i = 0; i < C; i++) {
      const uint32_t c = (i * a.row_threads + t) * 16;
      if (have && c < a.N) {
        load16(v[i], x + c, a.v8);
        if constexpr (RES) load16(r[i], res + c, a.v8);
      } else {
        v[i].zero();
        if constexpr (RES) r[i].zero();
      }
    }
    if (kEarly && t * 16 < a.N) w.load(a, t * 16);
#pragma unroll
    for (int i = 0; i < C; i++) {
      const uint32_t c = (i * a.row_threads + t) * 16;
      if constexpr (RES) {
        add16(v[i], r[i]);
        if (have && c < a.N) store16(hidden + c, v[i], a.v8);
      }
      ss += squares(v[i]);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
  if (lane == 0) sums[warp] = ss;
  __syncthreads();
  // one thread a row: the other warps' fp64 pipes stay free; no division, no
  // square root and its reciprocal (32768 x 2048 57 us with them, so 51)
  if (t == 0) {
    double s = 0.0;
    for (uint32_t i = 0; i < row_warps; i++) s += sums[warp + i];
    const float r = float(rsqrt(fma(s, a.inv_n, a.eps)));
    rstds[sub] = r;
    if (have) a.rstd[row] = r;
  }
  __syncthreads();
  const float rstd = rstds[sub];
  if constexpr (LOOP) {
    const T* h = RES ? hidden : x;
    for (uint32_t c0 = (t & ~31u) * 16; c0 < a.N; c0 += a.row_threads * 16) {   // warps stay together
      const uint32_t c = c0 + lane * 16;
      const bool active = have && c < a.N;
      if (active) {
        load16(v[0], h + c, a.v8);
        w.load(a, c);
      } else {
        v[0].zero();
      }
      finish16(a, v[0], w, row, c, rstd, active);
    }
  } else {
#pragma unroll
    for (int i = 0; i < C; i++) {
      const uint32_t c = (i * a.row_threads + t) * 16;
      const bool active = have && c < a.N;
      if ((!kEarly || i > 0) && active) w.load(a, c);
      finish16(a, v[i], w, row, c, rstd, active);
    }
  }
}

template <typename T, bool RES, bool WB, int C, bool LOOP>
mxq_status launch_norm(NormArgs& a, uint32_t rows, cudaStream_t s) {
  const uint32_t threads = a.row_threads * rows;
  a.row_ctas = uint32_t((uint64_t(a.M) + rows - 1) / rows);
  const uint32_t pad = a.swz ? uint32_t(-a.M & 127) : 0;
  const uint64_t grid = uint64_t(a.row_ctas) + (pad + threads / 32 - 1) / (threads / 32);
  if (grid > 0x7fffffffull) return MXQ_ERR_SHAPE;
  return launched(launch_pdl_ex(mxfp8_rmsnorm_kernel<T, RES, WB, C, LOOP>, uint32_t(grid), threads, 0, s, a));
}

template <typename T, bool RES, bool WB>
mxq_status norm_dispatch(NormArgs& a, cudaStream_t s) {
  const uint32_t pieces = a.N / 16;
  if (pieces > 2048) {
    a.row_threads = 1024;
    return launch_norm<T, RES, WB, 1, true>(a, 1, s);
  }
  // one piece a lane for short rows; also for fp32 with a residual, whose two
  // pieces a lane leave the registers (16384 x 4096 fp32 146 us, so 132; at 14336
  // columns 142 against 146)
  const int C = pieces <= (sizeof(T) == 4 && RES ? 512 : 128) ? 1 : 2;
  a.row_threads = ((pieces + C - 1) / C + 31) / 32 * 32;
  const uint32_t rows = std::max(1u, 128 / a.row_threads);
  return C == 1 ? launch_norm<T, RES, WB, 1, false>(a, rows, s) : launch_norm<T, RES, WB, 2, false>(a, rows, s);
}

template <typename T, bool RES>
mxq_status norm_weight(NormArgs& a, cudaStream_t s) {
  return a.weight_bf16 ? norm_dispatch<T, RES, true>(a, s) : norm_dispatch<T, RES, false>(a, s);
}

// ------------------------------------------------------------ gradient
//
// HBM-bound: per bf16 element 4 bytes read (6 with grad_hidden), 2 written.
// Persistent CTAs take rows blockIdx.x, + grid, ...: a thread owns the same C
// 16-byte units of every row, so that the weight's gradient stays in its
// registers until the end. Rows are copied into a ring of DEPTH rows in shared
// memory with cp.async, each thread its own units: no thread waits for
// another's copies, and the only barrier of a row is that of the sum
// mean(g w xh). The CTAs' sums of dweight go to the workspace [grid, N] and a
// second kernel adds them up in a fixed order; for few rows the CTAs are a
// cluster and add them up in its shared memory. Rows of more than 16384
// elements take a kernel that reads them twice, and dweight one of its own (4096
// x 32768 bf16 310 us for 123 at the copy rate).

struct GradArgs {
  const void *g, *h, *gh, *weight;
  const float* rstd;
  void* dx;
  float* part;            // [grid, N], or NULL
  void* dweight;          // of a cluster, or NULL
  int64_t ld_g, ld_h, ld_gh;
  int64_t M;
  uint32_t N;
  int weight_bf16;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// (plain: dx may be grad_hidden itself)
__device__ __forceinline__ uint4 load_plain(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// The values of T in 16 bytes, in pairs.
template <typename T>
struct Unit {
  static constexpr int kPairs = 8 / sizeof(T);
  float2 f[kPairs];
  __device__ __forceinline__ void load(const uint4& a) {
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int k = 0; k < kPairs; k++)
      f[k] = sizeof(T) == 2 ? make_float2(bf16_lo(u[k]), bf16_hi(u[k]))
                            : make_float2(__uint_as_float(u[2 * k % 4]), __uint_as_float(u[(2 * k + 1) % 4]));
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (sizeof(T) == 2)
      st_v4(p, make_uint4(cvt_bf16x2(f[0].x, f[0].y), cvt_bf16x2(f[1].x, f[1].y), cvt_bf16x2(f[2].x, f[2].y),
                          cvt_bf16x2(f[3].x, f[3].y)));
    else
      st_v4(p, make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x),
                          __float_as_uint(f[1].y)));
  }
};

__device__ __forceinline__ void sync_cluster() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The float at this CTA's shared address `at`, in CTA `rank` of the cluster.
__device__ __forceinline__ float load_cluster(uint32_t at, uint32_t rank) {
  float v;
  asm volatile("{ .reg .b32 a; mapa.shared::cluster.u32 a, %1, %2; ld.shared::cluster.f32 %0, [a]; }"
               : "=f"(v)
               : "r"(at), "r"(rank)
               : "memory");
  return v;
}

__device__ __forceinline__ void store_weight(void* dweight, int bf16, uint32_t c, float s) {
  if (bf16)
    static_cast<uint16_t*>(dweight)[c] = uint16_t(cvt_bf16x2(s, 0.f));
  else
    static_cast<float*>(dweight)[c] = s;
}

constexpr uint32_t kCluster = 16;        // most CTAs of a cluster (more than the portable eight)

// The weights of P pairs of columns from c on (a multiple of 2 P).
template <int P>
__device__ __forceinline__ void weights_at(float2 (&w)[P], const GradArgs& a, uint32_t c) {
  if (a.weight_bf16) {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.weight) + c);
#pragma unroll
    for (int k = 0; k < P; k += 2) {
      const uint2 q = __ldg(reinterpret_cast<const uint2*>(p + k));
      w[k] = make_float2(bf16_lo(q.x), bf16_hi(q.x));
      w[k + 1] = make_float2(bf16_lo(q.y), bf16_hi(q.y));
    }
  } else {
    const float* p = static_cast<const float*>(a.weight) + c;
#pragma unroll
    for (int k = 0; k < P; k += 2) {
      const float4 q = __ldg(reinterpret_cast<const float4*>(p + 2 * k));
      w[k] = make_float2(q.x, q.y);
      w[k + 1] = make_float2(q.z, q.w);
    }
  }
}

// Sums over the CTA of s[0 .. ROWS); `red` is 32 ROWS floats that the next call does not use.
template <int ROWS>
__device__ __forceinline__ void block_sums(float (&s)[ROWS], float* red) {
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int r = 0; r < ROWS; r++) s[r] += __shfl_xor_sync(kFull, s[r], o);
  if (lane == 0)
#pragma unroll
    for (int r = 0; r < ROWS; r++) red[32 * r + warp] = s[r];
  __syncthreads();
#pragma unroll
  for (int r = 0; r < ROWS; r++) s[r] = lane < warps ? red[32 * r + lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int r = 0; r < ROWS; r++) s[r] += __shfl_xor_sync(kFull, s[r], o);
}

template <typename T, bool GH, int C, int ROWS, int DEPTH>
__global__ void __launch_bounds__(512, 1) rmsnorm_grad_kernel(const __grid_constant__ GradArgs a) {
  pdl_enter();
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float red[2][32 * ROWS];
  constexpr uint32_t kVec = 16 / sizeof(T);                        // columns of a unit
  constexpr int kPairs = Unit<T>::kPairs;
  constexpr bool kGhRing = GH && sizeof(T) == 2;                   // else grad_hidden goes through registers
  constexpr uint32_t kTensors = kGhRing ? 3 : 2;
  const uint32_t t = threadIdx.x, T0 = blockDim.x;
  const uint32_t plane = T0 * 16;                                  // a unit of all threads
  const uint32_t stage = plane * C * kTensors * ROWS;
  const uint32_t ring0 = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  auto column = [&](int i) { return (uint32_t(i) * T0 + t) * kVec; };
  // unit i of tensor k of row r in a stage
  auto place = [&](uint32_t s, int r, uint32_t k, int i) {
    return s * stage + ((uint32_t(r) * kTensors + k) * C + uint32_t(i)) * plane + t * 16;
  };
  auto fetch = [&](int64_t row0, uint32_t s) {
#pragma unroll
    for (int r = 0; r < ROWS; r++) {
      const int64_t row = row0 + r;
      if (row < a.M) {
        const T* g = static_cast<const T*>(a.g) + row * a.ld_g;
        const T* h = static_cast<const T*>(a.h) + row * a.ld_h;
        const T* gh = static_cast<const T*>(a.gh) + (kGhRing ? row * a.ld_gh : 0);
#pragma unroll
        for (int i = 0; i < C; i++) {
          const uint32_t c = column(i);
          if (c < a.N) {
            copy16(ring0 + place(s, r, 0, i), g + c);
            copy16(ring0 + place(s, r, 1, i), h + c);
            if constexpr (kGhRing) copy16(ring0 + place(s, r, 2, i), gh + c);
          }
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto read = [&](Unit<T>& v, uint32_t s, int r, uint32_t k, int i) {
    v.load(*reinterpret_cast<const uint4*>(ring + place(s, r, k, i)));
  };
  const int64_t stride = int64_t(gridDim.x) * ROWS;
#pragma unroll
  for (int s = 0; s < DEPTH - 1; s++) fetch(int64_t(blockIdx.x) * ROWS + s * stride, s);

  float2 w[C][kPairs], dw[C][kPairs];
#pragma unroll
  for (int i = 0; i < C; i++) {
    if (column(i) < a.N) weights_at(w[i], a, column(i));
#pragma unroll
    for (int k = 0; k < kPairs; k++) dw[i][k] = twice(0.f);
  }
  const float inv_n = 1.f / float(a.N);
  uint32_t s = 0, par = 0;
  float next[ROWS];                                                // 1 / rms of the rows to come
  auto ask = [&](int64_t row) {
#pragma unroll
    for (int r = 0; r < ROWS; r++) next[r] = row + r < a.M ? __ldg(a.rstd + row + r) : 0.f;
  };
  ask(int64_t(blockIdx.x) * ROWS);
  for (int64_t row = int64_t(blockIdx.x) * ROWS; row < a.M; row += stride, par ^= 1) {
    // the stage that was read last is filled again (each thread's own units)
    fetch(row + (DEPTH - 1) * stride, s == 0 ? DEPTH - 1 : s - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
    float rstd[ROWS], mean[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; r++) rstd[r] = next[r];
    ask(row + stride);
    uint4 gh[GH && !kGhRing ? ROWS * C : 1];
    if constexpr (GH && !kGhRing) {
#pragma unroll
      for (int r = 0; r < ROWS; r++)
#pragma unroll
        for (int i = 0; i < C; i++)
          if (column(i) < a.N && (ROWS == 1 || row + r < a.M))
            gh[r * C + i] = load_plain(static_cast<const T*>(a.gh) + (row + r) * a.ld_gh + column(i));
    }
#pragma unroll
    for (int r = 0; r < ROWS; r++) {
      mean[r] = 0.f;
      if (ROWS > 1 && row + r >= a.M) continue;
      float2 sum = twice(0.f);
#pragma unroll
      for (int i = 0; i < C; i++) {
        if (column(i) < a.N) {
          Unit<T> g, h;
          read(g, s, r, 0, i);
          read(h, s, r, 1, i);
#pragma unroll
          for (int k = 0; k < kPairs; k++) {
            const float2 xh = mul2v(h.f[k], twice(rstd[r]));
            dw[i][k] = fma2v(g.f[k], xh, dw[i][k]);
            sum = fma2v(mul2v(g.f[k], w[i][k]), xh, sum);
          }
        }
      }
      mean[r] = sum.x + sum.y;
    }
    block_sums<ROWS>(mean, red[par]);
#pragma unroll
    for (int r = 0; r < ROWS; r++) {
      if (ROWS > 1 && row + r >= a.M) continue;
      mean[r] *= inv_n;
      T* dx = static_cast<T*>(a.dx) + (row + r) * int64_t(a.N);
#pragma unroll
      for (int i = 0; i < C; i++) {
        if (column(i) < a.N) {
          Unit<T> g, h, o;
          read(g, s, r, 0, i);
          read(h, s, r, 1, i);
          if constexpr (kGhRing) read(o, s, r, 2, i);
          if constexpr (GH && !kGhRing) o.load(gh[r * C + i]);
#pragma unroll
          for (int k = 0; k < kPairs; k++) {
            const float2 d = fma2v(mul2v(h.f[k], twice(rstd[r])), twice(-mean[r]), mul2v(g.f[k], w[i][k]));
            o.f[k] = GH ? fma2v(d, twice(rstd[r]), o.f[k]) : mul2v(d, twice(rstd[r]));
          }
          o.store(dx + column(i));
        }
      }
    }
    if (++s == DEPTH) s = 0;
  }
  if (a.part) {
#pragma unroll
    for (int i = 0; i < C; i++) {
      if (column(i) < a.N) {
        float* p = a.part + uint64_t(blockIdx.x) * a.N + column(i);
#pragma unroll
        for (int k = 0; k < kPairs; k += 2)
          st_v4(p + 2 * k, make_uint4(__float_as_uint(dw[i][k].x), __float_as_uint(dw[i][k].y),
                                      __float_as_uint(dw[i][k + 1].x), __float_as_uint(dw[i][k + 1].y)));
      }
    }
  }
  if (a.dweight) {
    // the ring, which holds at least 8 N bytes, takes the sums
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
#pragma unroll
    for (int i = 0; i < C; i++)
      if (column(i) < a.N)
#pragma unroll
        for (int k = 0; k < kPairs; k++) *reinterpret_cast<float2*>(ring + 4 * column(i) + 8 * k) = dw[i][k];
    sync_cluster();
    for (uint32_t c = blockIdx.x * T0 + t; c < a.N; c += gridDim.x * T0) {
      float v[kCluster], sum = 0.f;
#pragma unroll
      for (uint32_t r = 0; r < kCluster; r++) v[r] = r < gridDim.x ? load_cluster(ring0 + 4 * c, r) : 0.f;
#pragma unroll
      for (uint32_t r = 0; r < kCluster; r++) sum += v[r];
      store_weight(a.dweight, a.weight_bf16, c, sum);
    }
    sync_cluster();      // no CTA leaves while another reads its sums
  }
}

// dx of long rows, one row a CTA at a time, read twice.
template <typename T, bool GH>
__global__ void __launch_bounds__(1024) rmsnorm_grad_long_kernel(const __grid_constant__ GradArgs a) {
  pdl_enter();
  __shared__ float red[2][32];
  const float inv_n = 1.f / float(a.N);
  uint32_t par = 0;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, par ^= 1) {
    const float rstd = __ldg(a.rstd + row);
    const T* g = static_cast<const T*>(a.g) + row * a.ld_g;
    const T* h = static_cast<const T*>(a.h) + row * a.ld_h;
    constexpr uint32_t kVec = 16 / sizeof(T);
    float2 two = twice(0.f), w[Unit<T>::kPairs];
    Unit<T> g8, h8;
    for (uint32_t c = threadIdx.x * kVec; c < a.N; c += blockDim.x * kVec) {
      g8.load(load_plain(g + c));
      h8.load(load_plain(h + c));
      weights_at(w, a, c);
#pragma unroll
      for (int k = 0; k < Unit<T>::kPairs; k++) two = fma2v(mul2v(g8.f[k], w[k]), mul2v(h8.f[k], twice(rstd)), two);
    }
    float sum[1] = {two.x + two.y};
    block_sums<1>(sum, red[par]);
    const float mean = sum[0] * inv_n;
    for (uint32_t c = threadIdx.x * kVec; c < a.N; c += blockDim.x * kVec) {
      g8.load(load_plain(g + c));
      h8.load(load_plain(h + c));
      weights_at(w, a, c);
      Unit<T> o;
      if constexpr (GH) o.load(load_plain(static_cast<const T*>(a.gh) + row * a.ld_gh + c));
#pragma unroll
      for (int k = 0; k < Unit<T>::kPairs; k++) {
        const float2 d = fma2v(mul2v(h8.f[k], twice(rstd)), twice(-mean), mul2v(g8.f[k], w[k]));
        o.f[k] = GH ? fma2v(d, twice(rstd), o.f[k]) : mul2v(d, twice(rstd));
      }
      o.store(static_cast<T*>(a.dx) + row * int64_t(a.N) + c);
    }
  }
}

// dweight's partial sums of long rows, before dx may overwrite an input: CTA
// (column block, share of the rows).
template <typename T>
__global__ void __launch_bounds__(kThreads) rmsnorm_dweight_kernel(const __grid_constant__ GradArgs a) {
  pdl_enter();
  const uint32_t c = (blockIdx.x * kThreads + threadIdx.x) * (16 / sizeof(T));
  if (c >= a.N) return;
  float2 dw[Unit<T>::kPairs] = {};
  for (int64_t row = blockIdx.y; row < a.M; row += gridDim.y) {
    const float rstd = __ldg(a.rstd + row);
    Unit<T> g, h;
    g.load(load_plain(static_cast<const T*>(a.g) + row * a.ld_g + c));
    h.load(load_plain(static_cast<const T*>(a.h) + row * a.ld_h + c));
#pragma unroll
    for (int k = 0; k < Unit<T>::kPairs; k++) dw[k] = fma2v(g.f[k], mul2v(h.f[k], twice(rstd)), dw[k]);
  }
  float* p = a.part + uint64_t(blockIdx.y) * a.N + c;
#pragma unroll
  for (int k = 0; k < Unit<T>::kPairs; k++) {
    p[2 * k] = dw[k].x;
    p[2 * k + 1] = dw[k].y;
  }
}

// dweight[c] = the sum of `parts` partial sums, 32 columns a CTA, eight shares
// of the parts joined in a fixed order.
__global__ void __launch_bounds__(kThreads) rmsnorm_join_kernel(const float* __restrict__ part, uint32_t parts,
                                                                uint32_t N, void* dweight, int bf16) {
  pdl_enter();
  __shared__ float red[8][33];
  const uint32_t lane = threadIdx.x & 31, share = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < N) {
    uint32_t p = share;
    for (; p + 56 < parts; p += 64) {                  // eight loads in flight
      float v[8];
#pragma unroll
      for (uint32_t i = 0; i < 8; i++) v[i] = part[uint64_t(p + 8 * i) * N + c];
#pragma unroll
      for (uint32_t i = 0; i < 8; i++) s += v[i];
    }
    for (; p < parts; p += 8) s += part[uint64_t(p) * N + c];
  }
  red[share][lane] = s;
  __syncthreads();
  if (share != 0 || c >= N) return;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; i++) s += red[i][lane];
  store_weight(dweight, bf16, c, s);
}

constexpr uint32_t kLongRow = 16384;     // elements
constexpr uint32_t kSms = 148;
constexpr uint32_t kRingBytes = 225 * 1024;

// CTAs of the gradient: short rows need more of them on a multiprocessor for as
// many bytes in flight (65536 x 1024 bf16: 75 us with four, 93 with eight;
// 16384 x 4096: 68 with two of 256 threads, 82 with two of 512).
uint32_t grad_ctas(int64_t M, int64_t row_bytes) {
  const uint32_t per = row_bytes > 8192 ? 1 : row_bytes > 4096 ? 2 : 4;
  return uint32_t(std::min<int64_t>(M, int64_t(kSms) * per));
}

// Few rows: one cluster, no workspace and no second kernel. From the host 12.9 us
// for 17.0; on the device 61 x 1056 fp32 4.4 for 4.5, 32 x 7168 bf16 6.2 for 5.7,
// and 64 x 7168, which the rule leaves to the two kernels, 8.1 for 5.8. (Eight
// CTAs: 6.6, 7.6, 11.4; as many as there are pairs of rows, one 1 x 16384 16.0 for
// 7.5, two 4 x 7168 7.5 for 5.8.)
bool grad_cluster(int64_t M, int64_t N) { return M <= 64 && N <= kLongRow && M * N <= 262144; }

// The largest cluster of CTAs of Kernel, 16, 8, 4, 2 or 1, that the current device
// can hold: clusters of more than eight have to be allowed, and need as many
// multiprocessors within one's reach. Asked for once per device, for CTAs of the
// most shared memory.
template <auto Kernel>
uint32_t largest_cluster() {
  static std::atomic<uint32_t> known[256];
  int dev = 0;
  const bool slot = cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < 256;
  uint32_t n = slot ? known[dev].load(std::memory_order_acquire) : 0;
  if (n > 0) return n;
  const bool large = cudaFuncSetAttribute(Kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
  for (n = large ? kCluster : 8; n > 1; n /= 2) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(n);
    cfg.blockDim = dim3(512);
    cfg.dynamicSmemBytes = kRingBytes;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = n;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int resident = 0;
    if (cudaOccupancyMaxActiveClusters(&resident, Kernel, &cfg) == cudaSuccess && resident > 0) break;
  }
  (void)cudaGetLastError();
  if (slot && n > 1) known[dev].store(n, std::memory_order_release);
  return n;
}

template <typename T, bool GH, int C, int ROWS, int DEPTH>
mxq_status launch_grad(const GradArgs& a, uint32_t grid, uint32_t threads, cudaStream_t s) {
  const uint32_t smem = ROWS * DEPTH * threads * C * 16 * (GH && sizeof(T) == 2 ? 3 : 2);
  const cudaError_t e = ensure_smem_limit<rmsnorm_grad_kernel<T, GH, C, ROWS, DEPTH>>(int(kRingBytes));
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return MXQ_ERR_CUDA;
  }
  if (a.dweight) {
    const uint32_t ctas = largest_cluster<rmsnorm_grad_kernel<T, GH, C, ROWS, DEPTH>>();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return launched(cudaLaunchKernelEx(&cfg, rmsnorm_grad_kernel<T, GH, C, ROWS, DEPTH>, a));
  }
  return launched(launch_pdl_ex(rmsnorm_grad_kernel<T, GH, C, ROWS, DEPTH>, grid, threads, smem, s, a));
}

// Two rows at a time, and one barrier for both, where two stages of them fit
// (16384 x 7168 bf16: 109 us, one row at a time in four stages 131); rows of up
// to two units a thread always do, with the CTAs that share a multiprocessor.
template <typename T, bool GH, int C>
mxq_status grad_depth(const GradArgs& a, uint32_t grid, uint32_t threads, cudaStream_t s) {
  const uint32_t row = threads * C * 16 * (GH && sizeof(T) == 2 ? 3 : 2);
  if constexpr (C <= 2)
    return launch_grad<T, GH, C, 2, 2>(a, grid, threads, s);
  else if constexpr (C == 4)
    return row * 4 <= kRingBytes ? launch_grad<T, GH, C, 2, 2>(a, grid, threads, s)
                                 : launch_grad<T, GH, C, 1, 2>(a, grid, threads, s);
  else
    return row * 2 <= kRingBytes ? launch_grad<T, GH, C, 1, 2>(a, grid, threads, s)
                                 : launch_grad<T, GH, C, 1, 1>(a, grid, threads, s);
}

template <typename T, bool GH>
mxq_status grad_dispatch(const GradArgs& a, uint32_t grid, cudaStream_t s) {
  constexpr uint32_t kVec = 16 / sizeof(T);
  const uint32_t units = (a.N + kVec - 1) / kVec;
  if (a.N > kLongRow) {
    if (a.part) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3((units + kThreads - 1) / kThreads, grid);
      cfg.blockDim = dim3(kThreads);
      cfg.stream = s;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      attr[0].val.programmaticStreamSerializationAllowed = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      const mxq_status st = launched(cudaLaunchKernelEx(&cfg, rmsnorm_dweight_kernel<T>, a));
      if (st != MXQ_OK) return st;
    }
    return launched(launch_pdl_ex(rmsnorm_grad_long_kernel<T, GH>, grid, 1024, 0, s, a));
  }
  // units of a thread: one for short rows, two up to 512 threads, and as many
  // as it takes beyond
  auto threads = [&](uint32_t c) { return ((units + c - 1) / c + 31) / 32 * 32; };
  if (units <= 128) return grad_depth<T, GH, 1>(a, grid, threads(1), s);
  if (units <= 1024) return grad_depth<T, GH, 2>(a, grid, threads(2), s);
  if (sizeof(T) == 2 || units <= 2048) return grad_depth<T, GH, 4>(a, grid, threads(4), s);
  return grad_depth<T, GH, sizeof(T) == 2 ? 4 : 8>(a, grid, threads(8), s);
}

bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

}  // namespace
}  // namespace mxq

extern "C" {

mxq_status mxfp8_rmsnorm(const void* x, int dt, int64_t M, int64_t N, int64_t ld_x, const void* residual,
                         int64_t ld_res, const void* weight, int weight_dt, double eps, void* hidden,
                         uint8_t* qweight, uint8_t* scale, uint8_t* scale_swz, void* normed, float* rstd,
                         mxq_stream_t stream) {
  using namespace mxq;
  if (!valid_dtype(dt) || !valid_dtype(weight_dt)) return MXQ_ERR_DTYPE;
  if (M < 0 || N < 0 || N % 32 != 0 || ld_x < N || (residual && ld_res < N)) return MXQ_ERR_SHAPE;
  // a row's elements are counted in 32 bits; rows on the grid's first axis
  if (N > 0x3fffffe0ll || M > 0x7fffffffll || ld_x > (int64_t(1) << 40) || ld_res > (int64_t(1) << 40))
    return MXQ_ERR_SHAPE;
  if (!(eps >= 0.0)) return MXQ_ERR_ARG;
  if ((residual == nullptr) != (hidden == nullptr)) return MXQ_ERR_ARG;
  if (M == 0 || N == 0) return MXQ_OK;
  if (!x || !weight || !qweight || !scale || !rstd) return MXQ_ERR_NULL;
  const int es = elem_size(dt);
  if (!aligned16(x) || (uint64_t(ld_x) * es) % 16 != 0 || !aligned16(weight) || !aligned16(qweight) ||
      !aligned16(hidden) || !aligned16(normed) || !aligned16(residual) || !aligned16(scale_swz) ||
      (residual && (uint64_t(ld_res) * es) % 16 != 0) || (reinterpret_cast<uintptr_t>(rstd) & 3u))
    return MXQ_ERR_ALIGN;
  NormArgs a{};
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.hidden = hidden;
  a.q = qweight;
  a.scale = scale;
  a.swz = scale_swz;
  a.normed = normed;
  a.rstd = rstd;
  a.ld_x = ld_x;
  a.ld_res = ld_res;
  a.M = M;
  a.N = uint32_t(N);
  a.S4 = uint32_t((N + 127) / 128);
  a.eps = eps;
  a.inv_n = 1.0 / double(N);
  a.weight_bf16 = weight_dt == MXQ_BF16;
  a.weight_v8 = aligned32(weight);
  a.v8 = aligned32(x) && (uint64_t(ld_x) * es) % 32 == 0 && aligned32(hidden) && aligned32(normed) &&
         aligned32(residual) && (!residual || (uint64_t(ld_res) * es) % 32 == 0);
  a.scale_words = (reinterpret_cast<uintptr_t>(scale) & 3u) == 0 && (N / 32) % 4 == 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dt == MXQ_BF16) return residual ? norm_weight<uint16_t, true>(a, s) : norm_weight<uint16_t, false>(a, s);
  return residual ? norm_weight<float, true>(a, s) : norm_weight<float, false>(a, s);
}

size_t mxq_rmsnorm_backward_workspace_bytes(int64_t M, int64_t N) {
  if (M <= 0 || N <= 0 || mxq::grad_cluster(M, N)) return 0;
  return size_t(mxq::grad_ctas(M, 2 * N)) * size_t(N) * sizeof(float);   // (fp32 rows take no more)
}

mxq_status mxq_rmsnorm_backward(const void* grad, int dt, int64_t M, int64_t N, int64_t ld_g, const void* hidden,
                                int64_t ld_h, const void* weight, int weight_dt, const float* rstd,
                                const void* grad_hidden, int64_t ld_gh, void* dx, void* dweight, void* workspace,
                                size_t workspace_bytes, mxq_stream_t stream) {
  using namespace mxq;
  if (!valid_dtype(dt) || !valid_dtype(weight_dt)) return MXQ_ERR_DTYPE;
  if (M < 0 || N < 0 || N % 8 != 0 || ld_g < N || ld_h < N || (grad_hidden && ld_gh < N)) return MXQ_ERR_SHAPE;
  if (N > 0x3fffffe0ll || M > 0x7fffffffll || ld_g > (int64_t(1) << 40) || ld_h > (int64_t(1) << 40) ||
      ld_gh > (int64_t(1) << 40))
    return MXQ_ERR_SHAPE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (N == 0) return MXQ_OK;
  const int es = elem_size(dt);
  if (M == 0) {                                       // a sum of no rows
    if (!dweight) return MXQ_OK;
    const cudaError_t e = cudaMemsetAsync(dweight, 0, size_t(N) * elem_size(weight_dt), s);
    if (e != cudaSuccess) {
      record_cuda_error(e);
      return MXQ_ERR_CUDA;
    }
    return MXQ_OK;
  }
  if (!grad || !hidden || !weight || !rstd || !dx) return MXQ_ERR_NULL;
  if (!aligned16(grad) || !aligned16(hidden) || !aligned16(weight) || !aligned16(grad_hidden) || !aligned16(dx) ||
      (uint64_t(ld_g) * es) % 16 != 0 || (uint64_t(ld_h) * es) % 16 != 0 ||
      (grad_hidden && (uint64_t(ld_gh) * es) % 16 != 0) || (reinterpret_cast<uintptr_t>(rstd) & 3u) ||
      (reinterpret_cast<uintptr_t>(dweight) & (weight_dt == MXQ_BF16 ? 1u : 3u)) || (dweight && !aligned16(workspace)))
    return MXQ_ERR_ALIGN;
  const bool cluster = dweight && grad_cluster(M, N);
  if (dweight && !cluster && (!workspace || workspace_bytes < mxq_rmsnorm_backward_workspace_bytes(M, N)))
    return MXQ_ERR_WORKSPACE;
  GradArgs a{};
  a.g = grad;
  a.h = hidden;
  a.gh = grad_hidden;
  a.weight = weight;
  a.rstd = rstd;
  a.dx = dx;
  a.part = dweight && !cluster ? static_cast<float*>(workspace) : nullptr;
  a.dweight = cluster ? dweight : nullptr;
  a.ld_g = ld_g;
  a.ld_h = ld_h;
  a.ld_gh = ld_gh;
  a.M = M;
  a.N = uint32_t(N);
  a.weight_bf16 = weight_dt == MXQ_BF16;
  const uint32_t parts = grad_ctas(M, N * es);
  mxq_status st;
  if (dt == MXQ_BF16)
    st = grad_hidden ? grad_dispatch<uint16_t, true>(a, parts, s) : grad_dispatch<uint16_t, false>(a, parts, s);
  else
    st = grad_hidden ? grad_dispatch<float, true>(a, parts, s) : grad_dispatch<float, false>(a, parts, s);
  if (st != MXQ_OK || !a.part) return st;
  return launched(launch_pdl_ex(rmsnorm_join_kernel, (a.N + 31) / 32, kThreads, 0, s,
                                static_cast<const float*>(workspace), parts, a.N, dweight, a.weight_bf16));
}

}  // extern "C"
