// LC-VQ backward from an 8-bit checkpoint of X, for layers of few tiles.
//
// The products of gemm_kernels.hip take 256 x 256 tiles: a layer of a few hundred rows and
// columns leaves most CUs idle, and each of its workgroups runs a long epilogue. Here the
// tiles are 64 x 64, or 64 x 128 (NB = 2) with X or the codes decoded once for both halves, and
// one launch runs all of dW's and dX's, with no prologue. 1000 x 1024 x 4096 (d = 4, bf16)
// takes 39 us, 434 TFLOP/s (the sums 4.6 more); the CUs' VALU (decoding), LDS and L2 (15 TB/s)
// are each about half busy there, and layers of a few dozen tiles wait for one stage's loads
// after the other.
//   dW tile (k0, n0): G^T = X^T dY over the tokens. X's codes are decoded to bf16 (exact) on
//     their way into LDS; dWp = mask (I kron A^T) G, and the tile's sums for dA = G z^T and
//     dB = G 1, are formed from G in LDS in float32.
//   dX tile (m0, k0): C' = dY V over the outputs n, with V = 2 + z / 2, whose bf16 is a code
//     moved to bits 5 and 6 of 2.0; C = 2 C' - 4 r and dX = C (I kron A^T) + r B, with r = dY 1
//     summed from the same values, in float32.
// A second launch adds the tiles' dA and dB sums in a fixed order. The contraction runs in
// stages of 64, double-buffered in LDS; operands whose contraction runs along LDS rows are
// read with the transposing 64-bit reads. float32 dY is carried as bf16 hi + lo.
#include "mx_device.h"
#include "lcvq_internal.h"

namespace lcvq {

namespace {

constexpr int ST = 64;                         // tile edge and contraction per stage
constexpr int TB = ST * ST * 2;                // one bf16 tile, 8 KiB
constexpr int GS = ST + 4;                     // row of a float32 tile in LDS

typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));

// Tile [row][64 columns], 128 bytes per row. Read along rows (contraction = columns): the
// 8-chunk swizzle spreads 32 consecutive rows at one chunk. Read transposed (contraction =
// rows): 8 rows x 4 chunks per read, spread by the second.
__device__ __forceinline__ int off_rows(int r, int c) { return r * 128 + ((c ^ ((r ^ (r >> 3)) & 7)) << 4); }
__device__ __forceinline__ int off_cols(int r, int c) { return r * 128 + ((c ^ ((r & 2) << 1)) << 4); }

// Columns col0 .. col0 + 31 (lane % 32), 8 consecutive rows 16 s + 8 (lane / 32) .. + 7.
__device__ __forceinline__ bf16x8 frag_cols(const uint8_t* t, int col0, int s, int lane) {
  const int g = lane >> 4, l = lane & 15;
  const int col = col0 + 16 * (g & 1) + 4 * (l & 3);
  const int r = 16 * s + 8 * (g >> 1) + (l >> 2);
  const LCVQ_LDS uint8_t* b = (const LCVQ_LDS uint8_t*)t;
  const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (LCVQ_LDS v4s*)(b + off_cols(r, col >> 3) + ((col & 4) << 1)));
  const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (LCVQ_LDS v4s*)(b + off_cols(r + 4, col >> 3) + ((col & 4) << 1)));
  return __builtin_bit_cast(bf16x8, v8s{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
}
// Rows row0 .. row0 + 31 (lane % 32), 8 consecutive columns 16 s + 8 (lane / 32) .. + 7.
__device__ __forceinline__ bf16x8 frag_rows(const uint8_t* t, int row0, int s, int lane) {
  return *reinterpret_cast<const bf16x8*>(t + off_rows(row0 + (lane & 31), 2 * s + (lane >> 5)));
}

// 16 values of one row: thread t holds row t / 4, columns 16 (t % 4) .. + 15 of a tile.
struct Row16 {
  u32x4 a, b;                                  // bf16
};
__device__ __forceinline__ Row16 pack16(const float (&v)[16]) {
  Row16 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.a[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    r.b[i] = pack_bf16x2(v[8 + 2 * i], v[9 + 2 * i]);
  }
  return r;
}
template <bool COLS>
__device__ __forceinline__ void put16(uint8_t* t, int tid, const Row16& r) {
  const int row = tid >> 2, c = (tid & 3) * 2;
  *reinterpret_cast<u32x4*>(t + (COLS ? off_cols(row, c) : off_rows(row, c))) = r.a;
  *reinterpret_cast<u32x4*>(t + (COLS ? off_cols(row, c + 1) : off_rows(row, c + 1))) = r.b;
}

// Eight codes as the bf16 values 2 + z / 2.
__device__ __forceinline__ u32x4 code_pairs(uint32_t w) {
  const uint32_t u = w | w << 14;                            // pair j at bits 4 j and 4 j + 16
  u32x4 v;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    v[j] = ((j < 2 ? u << (5 - 4 * j) : u >> (4 * j - 5)) & 0x00600060u) | 0x40004000u;
  return v;
}

// dY's 16 values of a row in registers, as loaded.
template <typename T> struct DyRaw;
template <> struct DyRaw<uint16_t> {
  Row16 r;
  __device__ __forceinline__ void load(const uint16_t* p) {
    r.a = reinterpret_cast<const u32x4*>(p)[0];
    r.b = reinterpret_cast<const u32x4*>(p)[1];
  }
  template <bool COLS>
  __device__ __forceinline__ void put(uint8_t* hi, uint8_t*, int tid, bool in) const {
    const u32x4 o = {0, 0, 0, 0};
    put16<COLS>(hi, tid, Row16{in ? r.a : o, in ? r.b : o});
  }
  __device__ __forceinline__ float sum() const {
    const bf16x2 one = {(__bf16)1.f, (__bf16)1.f};
    float s = 0.f, t = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = r.a[i], b = r.b[i];       // (a bit cast of r.a[i] itself takes r.a[0])
      s = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, a), one, s, false);
      t = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, b), one, t, false);
    }
    return s + t;
  }
};
template <> struct DyRaw<float> {
  f32x4 v[4];
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = reinterpret_cast<const f32x4*>(p)[i];
  }
  template <bool COLS>
  __device__ __forceinline__ void put(uint8_t* hi, uint8_t* lo, int tid, bool in) const {
    float h[16], l[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float x = in ? v[i >> 2][i & 3] : 0.f;
      h[i] = (float)(__bf16)x;
      l[i] = x - h[i];
    }
    put16<COLS>(hi, tid, pack16(h));
    put16<COLS>(lo, tid, pack16(l));
  }
  // Of hi + lo, the values that the products take: in 2 C' - 4 r the 2 of each code's 2 + z / 2
  // cancels only if both see the same dY (what the pair leaves of it, up to 2^-18, would weigh
  // 4 + z). 1000 x 1024 x 4096, d = 4: 92 us, 89 with the plain sum.
  __device__ __forceinline__ float sum() const {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float x = v[i >> 2][i & 3], h = (float)(__bf16)x;
      s += h + (float)(__bf16)(x - h);
    }
    return s;
  }
};

// Stage: the 64 x 64 tile of X or of codes, then NB tiles of dY (float32: hi, lo).
template <typename T, int NB> constexpr int stage_bytes() { return (1 + NB * (int)sizeof(T) / 2) * TB; }
// Stage buffers, or the epilogue's G (or C) and z as float32 tiles; then A and B.
template <typename T, int D, int NB> constexpr int lds_bytes() {
  return (2 * stage_bytes<T, NB>() > 2 * ST * GS * 4 ? 2 * stage_bytes<T, NB>() : 2 * ST * GS * 4) +
         (D * D + D) * 4;
}

__device__ __forceinline__ void store16(uint16_t* p, const float (&v)[16]) {
  const Row16 r = pack16(v);
  reinterpret_cast<u32x4*>(p)[0] = r.a;
  reinterpret_cast<u32x4*>(p)[1] = r.b;
}
__device__ __forceinline__ void store16(float* p, const float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    reinterpret_cast<f32x4*>(p)[i] = f32x4{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
}

// Accumulator block (column l % 32, rows 8 (r / 4) + 4 (l / 32) + r % 4) to a float32 tile.
// TR: as [column][row] (quads of consecutive rows), else as [row][column].
template <bool TR>
__device__ __forceinline__ void put_block(float* g, const f32x16& c, int row0, int col0, int lane) {
  const int col = col0 + (lane & 31), h = lane >> 5;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int row = row0 + 8 * q + 4 * h;
    if constexpr (TR) {
      *reinterpret_cast<f32x4*>(g + col * GS + row) =
          f32x4{c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3]};
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) g[(row + e) * GS + col] = c[4 * q + e];
    }
  }
}

// The contraction over `len`, in stages of ST: a stage's values go from registers into one of
// two LDS buffers, the next stage's loads are issued, and after the barrier come the
// products. The barrier is not __syncthreads(), which would wait for the loads as well (both
// measured: 64 x 4096 x 4096, d = 8, 84 -> 69 us). Loads two, four and six stages ahead took
// 73, 76 and 92 us: their registers leave a CU fewer waves.
template <typename L, typename P, typename C>
__device__ __forceinline__ void stages(int64_t len, L&& load, P&& put, C&& products, uint8_t* smem,
                                       int sb) {
  load(0);
  int cur = 0;
  for (int64_t x = 0; x < len; x += ST) {
    put(smem + cur, x);
    load(x + ST);
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    products(smem + cur);
    cur = sb - cur;
  }
}

}  // namespace

struct Bwd8Args {
  const void* dY;
  const int8_t* Xc;
  const uint8_t* Xs;
  int64_t M, N, K;
  const uint8_t* packed;
  const uint8_t* mask;
  const float* A;
  const float* B;
  void* dX;
  float* dWp;
  float* partials;             // [dW tiles][d*d + d]
  int dw_tiles;
};

template <typename T, int D, int NB>
__global__ __launch_bounds__(256) void k_bwd8_small(Bwd8Args a) {
  constexpr int SB = stage_bytes<T, NB>(), YB = (int)sizeof(T) / 2 * TB;
  constexpr bool F32 = sizeof(T) == 4;
  __shared__ __attribute__((aligned(128))) uint8_t smem[lds_bytes<T, D, NB>()];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int p0 = (wave >> 1) * 32, q0 = (wave & 1) * 32;     // this wave's block
  const int row = tid >> 2, c16 = (tid & 3) * 16;            // this thread's 16 values
  float* As = reinterpret_cast<float*>(smem + lds_bytes<T, D, NB>() - (D * D + D) * 4);
  for (int i = tid; i < D * D + D; i += 256) As[i] = i < D * D ? a.A[i] : a.B[i - D * D];
  float* g = reinterpret_cast<float*>(smem);                 // epilogue tiles
  float* z = g + ST * GS;
  const T* dY = static_cast<const T*>(a.dY);
  // float32: dY's low halves in sums of their own. Added to the large ones each product would be
  // rounded against them, toward one side (dB of 1000 tokens, 2048 x 2496: 8e-6, so 3e-7).
  constexpr int NA = F32 ? 2 * NB : NB;
  f32x16 acc[NA];
#pragma unroll
  for (int b = 0; b < NA; ++b)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[b][r] = 0.f;

  if ((int)blockIdx.x < a.dw_tiles) {
    const int tk = (int)(a.K / ST);
    const int64_t k0 = (int64_t)(blockIdx.x % tk) * ST, n0 = (int64_t)(blockIdx.x / tk) * (ST * NB);
    u32x4 xc;
    uint32_t xs;
    DyRaw<T> dy[NB];
    auto load = [&](int64_t m0) __attribute__((always_inline)) {
      const int64_t m = m0 + row;
      const bool in = m < a.M;
      const int64_t mm = in ? m : a.M - 1;
      xc = *reinterpret_cast<const u32x4*>(a.Xc + mm * a.K + k0 + c16);
      xs = a.Xs[mm * (a.K / 32) + (k0 + c16) / 32];
#pragma unroll
      for (int b = 0; b < NB; ++b)      // (a block past N: loaded again, not used)
        dy[b].load(dY + mm * a.N + min(n0 + b * ST, a.N - ST) + c16);
    };
    auto put = [&](uint8_t* buf, int64_t m0) __attribute__((always_inline)) {
      const bool in = m0 + row < a.M;   // rows past M: zeros in dY, against the last row's X
      float lo[8], hi[8], v[16];
      mx_decode_int8(make_uint2(xc[0], xc[1]), xs, lo);
      mx_decode_int8(make_uint2(xc[2], xc[3]), xs, hi);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = lo[i];
        v[8 + i] = hi[i];
      }
      put16<true>(buf, tid, pack16(v));
#pragma unroll
      for (int b = 0; b < NB; ++b)
        dy[b].template put<true>(buf + TB + b * YB, buf + 2 * TB + b * YB, tid, in);
    };
    stages(a.M, load, put, [&](const uint8_t* t) __attribute__((always_inline)) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const bf16x8 x = frag_cols(t, p0, s, lane);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const uint8_t* y = t + TB + b * YB;
          acc[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, frag_cols(y, q0, s, lane), acc[b], 0, 0, 0);
          if constexpr (F32)
            acc[NB + b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, frag_cols(y + TB, q0, s, lane), acc[NB + b], 0, 0, 0);
        }
      }
    }, smem, SB);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if (n0 + b * ST >= a.N) break;
      __syncthreads();
      // G as [n][k] and the codes as float32
      if constexpr (F32) acc[b] += acc[NB + b];
      put_block<true>(g, acc[b], p0, q0, lane);
      const int64_t n = n0 + b * ST + row;
      const uint32_t code = *reinterpret_cast<const uint32_t*>(a.packed + n * (a.K / 4) + (k0 + c16) / 4);
#pragma unroll
      for (int i = 0; i < 16; ++i) z[row * GS + c16 + i] = (float)((code >> (2 * i)) & 3u);
      const uint32_t mk = *reinterpret_cast<const uint16_t*>(a.mask + n * (a.K / 8) + (k0 + c16) / 8);
      __syncthreads();
      float v[16], o[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = g[row * GS + c16 + i];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < D; ++i) s = __builtin_fmaf(As[i * D + j % D], v[j / D * D + i], s);
        o[j] = (mk >> j) & 1u ? s : 0.f;
      }
      store16(a.dWp + n * a.K + k0 + c16, o);
      // dA[i][j .. j + 3] and dB[i]: d^2 / 4 threads per group, the tile's vectors shared among
      // the groups, whose sums are added in two steps
      constexpr int TPG = D * D / 4, NG = 256 / TPG, VECS = ST * ST / D, PER = VECS / NG, GPR = ST / D;
      const int in_g = tid % TPG, i = in_g / (D / 4), j = in_g % (D / 4) * 4, grp = tid / TPG;
      f32x4 sa = {0.f, 0.f, 0.f, 0.f};
      float sb = 0.f;
#pragma unroll 8
      for (int w = 0; w < PER; ++w) {
        const int at = (grp * PER + w) / GPR * GS + (grp * PER + w) % GPR * D;
        const float x = g[at + i];
        const f32x4 zz = *reinterpret_cast<const f32x4*>(z + at + j);
#pragma unroll
        for (int e = 0; e < 4; ++e) sa[e] = __builtin_fmaf(x, zz[e], sa[e]);
        sb += x;
      }
      __syncthreads();
      constexpr int NO = D * D + D, RS = NO + 1;               // a group's sums, padded
      float* red = g;                                          // [NG][RS]
#pragma unroll
      for (int e = 0; e < 4; ++e) red[grp * RS + i * D + j + e] = sa[e];
      if (j == 0) red[grp * RS + D * D + i] = sb;
      __syncthreads();
      float* out = a.partials + ((n0 / ST + b) * tk + k0 / ST) * NO;
      for (int o = tid; o < NO; o += 256) {
        float s = 0.f;
#pragma unroll 8
        for (int w = 0; w < NG; ++w) s += red[w * RS + o];
        out[o] = s;
      }
    }
  } else {
    const int tk = (int)(a.K / ST), t = (int)blockIdx.x - a.dw_tiles;
    const int64_t k0 = (int64_t)(t % tk) * ST, m0 = (int64_t)(t / tk) * (ST * NB);
    uint32_t code;
    DyRaw<T> dy[NB];
    float rsum[NB] = {};
    auto load = [&](int64_t n0) __attribute__((always_inline)) {
      const int64_t nn = min(n0, a.N - ST);                  // (a stage past the end: not used)
#pragma unroll
      for (int b = 0; b < NB; ++b) dy[b].load(dY + min(m0 + b * ST + row, a.M - 1) * a.N + nn + c16);
      code = *reinterpret_cast<const uint32_t*>(a.packed + (nn + row) * (a.K / 4) + (k0 + c16) / 4);
    };
    auto put = [&](uint8_t* buf, int64_t) __attribute__((always_inline)) {
      put16<true>(buf, tid, Row16{code_pairs(code & 0xffffu), code_pairs(code >> 16)});
#pragma unroll
      for (int b = 0; b < NB; ++b) {                         // (rows past M: not stored)
        dy[b].template put<false>(buf + TB + b * YB, buf + 2 * TB + b * YB, tid, true);
        rsum[b] += dy[b].sum();
      }
    };
    stages(a.N, load, put, [&](const uint8_t* t) __attribute__((always_inline)) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const bf16x8 zf = frag_cols(t, q0, s, lane);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const uint8_t* y = t + TB + b * YB;
          acc[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(frag_rows(y, p0, s, lane), zf, acc[b], 0, 0, 0);
          if constexpr (F32)
            acc[NB + b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(frag_rows(y + TB, p0, s, lane), zf, acc[NB + b], 0, 0, 0);
        }
      }
    }, smem, SB);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      __syncthreads();
      // the row's four threads hold its sum in parts
      float r = rsum[b];
      r += __shfl_xor(r, 1);
      r += __shfl_xor(r, 2);
      if constexpr (F32) acc[b] += acc[NB + b];
      put_block<false>(g, acc[b], p0, q0, lane);                  // C as [m][k]
      __syncthreads();
      float v[16], o[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = 2.f * g[row * GS + c16 + i] - 4.f * r;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float s = r * As[D * D + i % D];
#pragma unroll
        for (int j = 0; j < D; ++j) s = __builtin_fmaf(As[i % D * D + j], v[i / D * D + j], s);
        o[i] = s;
      }
      const int64_t m = m0 + b * ST + row;
      if (m < a.M) store16(static_cast<T*>(a.dX) + m * a.K + k0 + c16, o);
    }
  }
}

// Tiles of 64 x 64 (also dW's rows of partial sums).
int64_t bwd8_small_tiles(int64_t M, int64_t N, int64_t K, bool dx) {
  return (K / ST) * (N / ST) + (dx ? (K / ST) * ((M + ST - 1) / ST) : 0);
}

template <typename T, int NB>
static hipError_t launch_t(Bwd8Args a, int d, hipStream_t s) {
  const int64_t kt = a.K / ST, e = ST * NB;
  a.dw_tiles = (int)(kt * ((a.N + e - 1) / e));
  const unsigned blocks = (unsigned)(a.dw_tiles + (a.dX ? kt * ((a.M + e - 1) / e) : 0));
  switch (d) {
    case 4: LCVQ_LAUNCH(PROF_DW, (k_bwd8_small<T, 4, NB>), dim3(blocks), dim3(256), 0, s, a); break;
    case 8: LCVQ_LAUNCH(PROF_DW, (k_bwd8_small<T, 8, NB>), dim3(blocks), dim3(256), 0, s, a); break;
    default: LCVQ_LAUNCH(PROF_DW, (k_bwd8_small<T, 16, NB>), dim3(blocks), dim3(256), 0, s, a); break;
  }
  return hipGetLastError();
}

hipError_t launch_bwd8_small(const void* dY, const int8_t* Xc, const uint8_t* Xs, bool f32,
                             int64_t M, int64_t N, int64_t K, int d, const uint8_t* packed,
                             const uint8_t* mask, const float* A, const float* B, void* dX,
                             float* dWp, float* dA, float* dB, float* partials, hipStream_t s) {
  const Bwd8Args a{dY, Xc, Xs, M, N, K, packed, mask, A, B, dX, dWp, partials, 0};
  // Two tiles of dY per workgroup, which halve the decoding, where dW's and dX's products have
  // 1024 tiles of 64 x 64 each (1000 x 1024 x 4096, d = 4: 40.8 us against 47.1; 2048^3: 78 and
  // 91; fewer tiles leave CUs idle: 1024^3, 256 each, 19.7 and 16.9; 64 x 4096 x 4096, dX with
  // 64, 79 and 70). float32 dY would need half a CU's LDS and more.
  const int64_t dw = bwd8_small_tiles(M, N, K, false);
  const bool wide = dw >= 1024 && (!dX || bwd8_small_tiles(M, N, K, true) - dw >= 1024);
  const hipError_t e = f32    ? launch_t<float, 1>(a, d, s)
                       : wide ? launch_t<uint16_t, 2>(a, d, s)
                              : launch_t<uint16_t, 1>(a, d, s);
  if (e != hipSuccess) return e;
  return launch_reduce_partials(partials, (int)dw, d, dA, dB, s);
}

}  // namespace lcvq
