// MXFP4 products on gfx950's block-scaled matrix instructions.
#include <algorithm>

#include "mx_device.h"
#include "lcvq_internal.h"

namespace lcvq {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// One scaled product step: 32 x 32 += 32 x 64 . (32 x 64)^T. Lane l holds row l % 32,
// values 32 (l / 32) .. + 31 of each operand (16 bytes, one block) and that block's scale
// byte in byte SA / SB of its scale word.
template <int SA, int SB>
__device__ __forceinline__ f32x16 mfma_fp4(u32x4 a, u32x4 b, f32x16 c, uint32_t sa, uint32_t sb) {
  const i32x8 A = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 B = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(A, B, c, 4, 4, SA, (int)sa, SB, (int)sb);
}

__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = (uint16_t)pack_bf16x2(v, 0.f); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store4(uint16_t* p, f32x4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}
__device__ __forceinline__ void store4(float* p, f32x4 v) { *reinterpret_cast<f32x4*>(p) = v; }

// 16 scale bytes of a row. Rows of 4 n blocks start at a multiple of 4 and take one load
// (AL). Others start anywhere, and a 16-byte load off its 4-byte boundary is slow (515 x 4096
// x 4128, tiles of 128: 20.6 us): they take the aligned words that hold the bytes, four in
// one load and the last (17.0 us; four and three single bytes 19.5). An aligned word that holds
// a byte of the array may hold up to three bytes beyond its ends, in the same page.
template <bool AL> struct MxScale16;
template <> struct MxScale16<true> {
  u32x4 d;
  __device__ __forceinline__ void load(const uint8_t* p) { __builtin_memcpy(&d, __builtin_assume_aligned(p, 4), 16); }
  __device__ __forceinline__ u32x4 get() const { return d; }
};
template <> struct MxScale16<false> {
  u32x4 d;
  uint32_t last, sh;
  __device__ __forceinline__ void load(const uint8_t* p) {
    sh = (uint32_t)reinterpret_cast<uintptr_t>(p) & 3u;
    __builtin_memcpy(&d, __builtin_assume_aligned(p - sh, 4), 16);
    last = *reinterpret_cast<const uint32_t*>(p - sh + (sh ? 16 : 12));
  }
  __device__ __forceinline__ u32x4 get() const {
    return u32x4{__builtin_amdgcn_alignbyte(d[1], d[0], sh), __builtin_amdgcn_alignbyte(d[2], d[1], sh),
                 __builtin_amdgcn_alignbyte(d[3], d[2], sh), __builtin_amdgcn_alignbyte(last, d[3], sh)};
  }
};

// The n < 16 scale bytes of a row's partial last chunk at p, and 1 (2^0) for the rest: the
// aligned words that hold them (words past the last valid byte repeat its word). One load
// per word: byte by byte they took 0.8 us more of a 515 x 4096 x 4224 product (15.0).
template <bool AL> struct MxScaleTail {
  static constexpr int W = AL ? 3 : 5;
  uint32_t d[W], sh;
  __device__ __forceinline__ void load(const uint8_t* p, int n) {
    sh = AL ? 0u : (uint32_t)reinterpret_cast<uintptr_t>(p) & 3u;
    const int end = ((int)sh + n - 1) & ~3;            // offset of the last byte's word
#pragma unroll
    for (int i = 0; i < W; ++i) d[i] = *reinterpret_cast<const uint32_t*>(p - sh + min(4 * i, end));
  }
  __device__ __forceinline__ u32x4 get(int n) const {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w = 0x7f7f7f7fu;
      if constexpr (AL) {
        if (i < W) w = d[i < W ? i : 0];
      } else {
        w = __builtin_amdgcn_alignbyte(d[i + 1], d[i], sh);
      }
      const int in = min(max(n - 4 * i, 0), 4);        // bytes of this word that are valid
      const uint32_t m = in == 4 ? 0xffffffffu : (1u << (8 * in)) - 1u;
      v[i] = (w & m) | (0x7f7f7f7fu & ~m);
    }
    return v;
  }
};

// ---- Y = X W^T --------------------------------------------------------------------------
// C[n, m] = sum_k W[n, k] X[m, k] in tiles of BN rows of W by BM rows of X: W is the first
// operand, so that a lane's accumulator quads are 4 consecutive n of one row of Y. The
// contraction runs in stages of 128 values (64 bytes, 4 blocks of a row). Stages go from
// HBM straight into a ring of LDS slots, all but one in flight while one is consumed.
// A lane's fragment is one block (16 bytes, ds_read_b128); chunk c of tile row r sits at
// position c ^ ((r / 4) mod 4) of its 64 bytes, so that 16 consecutive rows read at one c
// cover the 64 banks once. Scale bytes come 16 per row and 512 values through registers
// into a double-buffered LDS area; a wave reads the 4 bytes of a stage as one word and
// moves the byte of its half (blocks 2s + h, h = lane / 32) to bytes 0 and 2.
// Large products are bound by the matrix units' power: 8192 x 14336 x 4096 259 us, 3.7 PFLOP/s
// (8192^3: 268 us on random values, 203 us on zeros). At one tile of 128 x 128 per CU or
// fewer a stage takes 0.3 us, 256 cycles of products and 384 of LDS that nothing overlaps,
// and filling and emptying the pipeline 4 us (1024 x 4096 x 4096: 13.1 us).
constexpr int MXK = 128;                       // values per stage
constexpr int MXROWB = MXK / 2;                // bytes per row and stage

struct MxGemmArgs {
  const uint8_t* Xc;
  const uint8_t* Xs;
  const uint8_t* Wc;
  const uint8_t* Ws;
  int64_t M, N, nb;                            // nb: blocks per row
  void* Y;
  int tilesN, tilesM, ntiles;
};

template <int WI, int WJ, int NWN, int NWM, int RING> struct MxTile {
  static constexpr int BN = 32 * WI * NWN, BM = 32 * WJ * NWM, NW = NWN * NWM;
  static constexpr int ROWS = BN + BM, SLOTB = ROWS * MXROWB, SCB = ROWS * 16;
  static constexpr int RW = BN / NW, RX = BM / NW;    // rows of W and X that a wave loads
  static constexpr int LOADS = (RW + RX) / 16;        // 16-byte loads per lane and stage
  static constexpr int RPT = (ROWS + NW * 64 - 1) / (NW * 64);   // scale rows per thread
  // Waves per SIMD that the registers leave room for (128 x 128 per wave: one).
  static constexpr int EU = WI * WJ >= 16 ? 1 : (WI * WJ >= 2 ? 2 : 4) * 4 / RING;
  static_assert(RW % 16 == 0 && RX % 16 == 0, "a load takes 16 rows");
};

// s_waitcnt immediate: at most n vector-memory operations outstanding.
constexpr int mx_vmcnt(int n) { return (n & 15) | ((n >> 4) << 14) | 0x0F70; }

// All loads but the N youngest have landed.
template <int N>
__device__ __forceinline__ void mx_landed() {
  __builtin_amdgcn_s_waitcnt(mx_vmcnt(N));
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

template <int WI, int WJ>
struct MxFrags {
  u32x4 a[WI], b[WJ];
};
template <int WI, int WJ>
struct MxScales {
  uint32_t a[WI], b[WJ];
};

__device__ __forceinline__ void mx_wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Four consecutive outputs n .. n + 3 of one staged row (see the epilogue).
__device__ __forceinline__ void mx_stage_quad(uint16_t* row, int cpr, int m, int n, float a,
                                              float b, float c, float d) {
  uint2* p = reinterpret_cast<uint2*>(row + (((n >> 3) ^ (m % cpr)) << 3) + (n & 4));
  *p = make_uint2(pack_bf16x2(a, b), pack_bf16x2(c, d));
}
__device__ __forceinline__ void mx_stage_quad(float* row, int cpr, int m, int n, float a, float b,
                                              float c, float d) {
  *reinterpret_cast<f32x4*>(row + (((n >> 2) ^ (m % cpr)) << 2)) = f32x4{a, b, c, d};
}

// Scheduling of one sub-step: R LDS reads and V direct loads spread over its P products.
template <int P, int R, int V>
__device__ __forceinline__ void mx_interleave() {
#pragma unroll
  for (int i = 0; i < P; ++i) {
    if ((i + 1) * R / P > i * R / P) __builtin_amdgcn_sched_group_barrier(0x100, (R + P - 1) / P, 0);
    if ((i + 1) * V / P > i * V / P) __builtin_amdgcn_sched_group_barrier(0x020, (V + P - 1) / P, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
  }
}

template <typename T, int WI, int WJ, int NWN, int NWM, int RING, bool AL>
__global__ __launch_bounds__(NWN * NWM * 64)
__attribute__((amdgpu_waves_per_eu(MxTile<WI, WJ, NWN, NWM, RING>::EU,
                                   MxTile<WI, WJ, NWN, NWM, RING>::EU)))
void k_mxfp4_tile(MxGemmArgs g) {
  using C = MxTile<WI, WJ, NWN, NWM, RING>;
  static_assert(RING == 4 || RING == 8, "the loop is unrolled over the ring");
  // The slots are arrays of their own, so that the compiler can tell a read of one from a
  // direct load into another and makes no read wait for all loads.
  __shared__ __attribute__((aligned(1024))) uint8_t s0[C::SLOTB], s1[C::SLOTB], s2[C::SLOTB],
      s3[C::SLOTB], s4[RING == 8 ? C::SLOTB : 16], s5[RING == 8 ? C::SLOTB : 16],
      s6[RING == 8 ? C::SLOTB : 16], s7[RING == 8 ? C::SLOTB : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t sc[3 * C::SCB];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave / NWM, wm = wave % NWM;
  // Consecutive workgroups go to the 8 XCDs in turn; each XCD takes a run of tiles, in
  // groups of 4 tile-rows, so that its L2 holds the panels they share.
  int tn, tm;
  {
    const int per = (g.ntiles + 7) >> 3;
    const int t = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
    if (t >= g.ntiles) return;
    constexpr int GR = 4;
    const int group = t / (GR * g.tilesM), within = t - group * GR * g.tilesM;
    const int rows = min(g.tilesN - group * GR, GR);
    tn = group * GR + within % rows;
    tm = within / rows;
  }
  const int64_t n0 = (int64_t)tn * C::BN, m0 = (int64_t)tm * C::BM;
  const int64_t nb = g.nb, rowb = nb * 16;

  // The loads of this wave are buffer loads, whose range check gives zeros for rows past the
  // matrix; a chunk past the row (the last stages) gets an offset outside every buffer. The
  // check takes a stage's offset, added to all lanes, off the buffer's size, so a buffer is
  // never shorter than a row: a wave past the matrix takes the last row, whose products are
  // not stored.
  const int64_t roww = min(n0 + wave * C::RW, g.N - 1), rowx = min(m0 + wave * C::RX, g.M - 1);
  const int leftw = (int)min(g.N - roww, (int64_t)C::RW);
  const int leftx = (int)min(g.M - rowx, (int64_t)C::RX);
  const auto wsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(g.Wc + roww * rowb), 0,
                                                      (int)(leftw * rowb), 0x00020000);
  const auto xsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(g.Xc + rowx * rowb), 0,
                                                      (int)(leftx * rowb), 0x00020000);
  const int rl = lane >> 2;
  const int chunk = (lane & 3) ^ ((rl >> 2) & 3);     // rows advance by 16 per load
  const uint32_t voff0 = (uint32_t)(rl * rowb + chunk * 16);
  const uint32_t vstep = (uint32_t)(16 * rowb);
  auto issue = [&](uint8_t* slot, int kt) __attribute__((always_inline)) {
    const bool in = kt * 4 + chunk < (int)nb;
#pragma unroll
    for (int i = 0; i < C::RW / 16; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          wsrc, (LCVQ_LDS void*)(slot + (wave * C::RW + i * 16) * MXROWB), 16,
          (int)(in ? voff0 + i * vstep : 0xffffffffu), kt * MXROWB, 0, 0);
#pragma unroll
    for (int i = 0; i < C::RX / 16; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          xsrc, (LCVQ_LDS void*)(slot + (C::BN + wave * C::RX + i * 16) * MXROWB), 16,
          (int)(in ? voff0 + i * vstep : 0xffffffffu), kt * MXROWB, 0, 0);
  };
  // Scales: thread t fetches 16 bytes (blocks 16 c .. + 15) of tile rows t, t + 64 NW, ...
  // ahead of their use, for each full chunk c of 512 values; those of a last partial chunk
  // go into an area of their own before the loop (blocks past the row: scale 1).
  constexpr int NT = C::NW * 64;
  const bool sown = C::ROWS % NT == 0 || tid < C::ROWS;
  const uint8_t* ssrc[C::RPT];
#pragma unroll
  for (int p = 0; p < C::RPT; ++p) {
    const int t = p * NT + tid;
    ssrc[p] = t < C::BN ? g.Ws + min(n0 + t, g.N - 1) * nb
                        : g.Xs + min(m0 + (t - C::BN), g.M - 1) * nb;
  }
  uint8_t* const sdst = sc + tid * 16;
  const int nfull = (int)(nb >> 4), ntail = (int)((nb & 15) + 3) >> 2;   // chunks, stages
  MxScale16<AL> sv[C::RPT];
  auto scale_load = [&](int c) __attribute__((always_inline)) {
#pragma unroll
    for (int p = 0; p < C::RPT; ++p) sv[p].load(ssrc[p] + (int64_t)min(c, nfull - 1) * 16);
  };
  auto scale_put = [&](int area) __attribute__((always_inline)) {
#pragma unroll
    for (int p = 0; p < C::RPT; ++p)
      if (sown) *reinterpret_cast<u32x4*>(sdst + area * C::SCB + p * NT * 16) = sv[p].get();
  };

  f32x16 acc[WI][WJ];
#pragma unroll
  for (int i = 0; i < WI; ++i)
#pragma unroll
    for (int j = 0; j < WJ; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  // Fragment offsets (sub-step 0; sub-step 1 is chunk ^ 2) and scale offsets.
  const int fr = lane & 31, h = lane >> 5;
  int fo = fr * MXROWB + ((h ^ ((fr >> 2) & 3)) << 4);
  int so = fr * 16;
  asm volatile("" : "+v"(fo));
  asm volatile("" : "+v"(so));
  const int an = wn * 32 * WI, bm = C::BN + wm * 32 * WJ;
  auto read = [&](const uint8_t* slot, int s, MxFrags<WI, WJ>& f) __attribute__((always_inline)) {
    const int o = fo ^ (s << 5);
#pragma unroll
    for (int i = 0; i < WI; ++i)
      f.a[i] = *reinterpret_cast<const u32x4*>(slot + (an + 32 * i) * MXROWB + o);
#pragma unroll
    for (int j = 0; j < WJ; ++j)
      f.b[j] = *reinterpret_cast<const u32x4*>(slot + (bm + 32 * j) * MXROWB + o);
  };
  auto read_scales = [&](const uint8_t* area, int ph, MxScales<WI, WJ>& q)
      __attribute__((always_inline)) {
    const uint8_t* base = area + ph * 4 + so;
#pragma unroll
    for (int i = 0; i < WI; ++i)
      q.a[i] = *reinterpret_cast<const uint32_t*>(base + (an + 32 * i) * 16);
#pragma unroll
    for (int j = 0; j < WJ; ++j)
      q.b[j] = *reinterpret_cast<const uint32_t*>(base + (bm + 32 * j) * 16);
  };
  auto shift_scales = [&](MxScales<WI, WJ>& q) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < WI; ++i) q.a[i] >>= 8 * h;
#pragma unroll
    for (int j = 0; j < WJ; ++j) q.b[j] >>= 8 * h;
  };

  // Scale loads go out before the stages' (the counter is in order, so what is waited for
  // first is loaded first).
  if (nfull) scale_load(0);
  MxScaleTail<AL> tb[C::RPT];
  if (ntail) {
#pragma unroll
    for (int p = 0; p < C::RPT; ++p) tb[p].load(ssrc[p] + (int64_t)nfull * 16, (int)(nb & 15));
  }
  issue(s0, 0);
  issue(s1, 1);
  issue(s2, 2);
  if constexpr (RING == 8) {
    issue(s3, 3);
    issue(s4, 4);
    issue(s5, 5);
    issue(s6, 6);
  }
  if (nfull) {
    scale_put(0);
    scale_load(1);
  }
  if (ntail) {
#pragma unroll
    for (int p = 0; p < C::RPT; ++p)
      if (sown)
        *reinterpret_cast<u32x4*>(sdst + 2 * C::SCB + p * NT * 16) = tb[p].get((int)(nb & 15));
  }
  __builtin_amdgcn_s_waitcnt(mx_vmcnt((RING - 2) * C::LOADS));       // stage 0 has landed
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  MxFrags<WI, WJ> f0, f1;
  MxScales<WI, WJ> q, qn;
  read(s0, 0, f0);
  read_scales(sc, 0, q);
  shift_scales(q);

  // One stage. Its barrier sits before its second sub-step, under whose products the next
  // stage's first fragments are read. Loads and reads past the last stage bring zeros: the
  // loop has no branch, which keeps the products in the order written.
  auto stage = [&](uint8_t* cur, uint8_t* nxt, uint8_t* far, int kt, int ph,
                   const uint8_t* area, int other)
      __attribute__((always_inline)) {
    read(cur, 1, f1);
#pragma unroll
    for (int i = 0; i < WI; ++i)
#pragma unroll
      for (int j = 0; j < WJ; ++j) acc[i][j] = mfma_fp4<0, 0>(f0.a[i], f0.b[j], acc[i][j], q.a[i], q.b[j]);
    mx_interleave<WI * WJ, WI + WJ, 0>();
    __builtin_amdgcn_sched_barrier(0);
    if (ph == 3) {
      // the next 512 values' scales: fetched four stages ago, read from the next stage on
      const int c = (kt >> 2) + 1;
      scale_put(c & 1);
      scale_load(c + 1);
    }
    // stage kt + 1 has landed; the RING - 3 after it may still be in flight
    __builtin_amdgcn_s_waitcnt(mx_vmcnt((RING - 3) * C::LOADS));
    if (ph == 3) asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    else asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    issue(far, kt + RING - 1);
    read(nxt, 0, f0);
    read_scales(area + (ph == 3 ? other : 0), (ph + 1) & 3, qn);
#pragma unroll
    for (int i = 0; i < WI; ++i)
#pragma unroll
      for (int j = 0; j < WJ; ++j) acc[i][j] = mfma_fp4<2, 2>(f1.a[i], f1.b[j], acc[i][j], q.a[i], q.b[j]);
    mx_interleave<WI * WJ, WI + WJ + 4, C::LOADS>();
    __builtin_amdgcn_sched_barrier(0);
    q = qn;
    shift_scales(q);
  };
  auto areas = [&](int c, const uint8_t*& area, int& other) __attribute__((always_inline)) {
    area = sc + (c & 1) * C::SCB;
    other = (c & 1) ? -C::SCB : C::SCB;                // from this chunk's area to the next's
  };
  int c = 0;                                           // chunks done
  if constexpr (RING == 4) {
    for (; c < nfull; ++c) {
      const uint8_t* area;
      int other;
      areas(c, area, other);
      stage(s0, s1, s3, 4 * c, 0, area, other);
      stage(s1, s2, s0, 4 * c + 1, 1, area, other);
      stage(s2, s3, s1, 4 * c + 2, 2, area, other);
      stage(s3, s0, s2, 4 * c + 3, 3, area, other);
    }
  } else {
    for (; c + 1 < nfull; c += 2) {
      const uint8_t* area;
      int other;
      areas(c, area, other);
      stage(s0, s1, s7, 4 * c, 0, area, other);
      stage(s1, s2, s0, 4 * c + 1, 1, area, other);
      stage(s2, s3, s1, 4 * c + 2, 2, area, other);
      stage(s3, s4, s2, 4 * c + 3, 3, area, other);
      areas(c + 1, area, other);
      stage(s4, s5, s3, 4 * c + 4, 0, area, other);
      stage(s5, s6, s4, 4 * c + 5, 1, area, other);
      stage(s6, s7, s5, 4 * c + 6, 2, area, other);
      stage(s7, s0, s6, 4 * c + 7, 3, area, other);
    }
    if (c < nfull) {                                   // an odd chunk
      const uint8_t* area;
      int other;
      areas(c, area, other);
      stage(s0, s1, s7, 4 * c, 0, area, other);
      stage(s1, s2, s0, 4 * c + 1, 1, area, other);
      stage(s2, s3, s1, 4 * c + 2, 2, area, other);
      stage(s3, s4, s2, 4 * c + 3, 3, area, other);
    }
  }
  // the partial last chunk; with 8 slots it starts at slot 0 or 4
  auto tail = [&](uint8_t* t0, uint8_t* t1, uint8_t* t2, uint8_t* t3, uint8_t* t4, uint8_t* far)
      __attribute__((always_inline)) {
    const uint8_t* area = sc + 2 * C::SCB;
    read_scales(area, 0, q);
    shift_scales(q);
    stage(t0, t1, far, 4 * nfull, 0, area, 0);
    if (ntail > 1) stage(t1, t2, t0, 4 * nfull + 1, 1, area, 0);
    if (ntail > 2) stage(t2, t3, t1, 4 * nfull + 2, 2, area, 0);
    if (ntail > 3) stage(t3, t4, t2, 4 * nfull + 3, 4, area, 0);
  };
  if (ntail) {
    if constexpr (RING == 4) {
      tail(s0, s1, s2, s3, s0, s3);
    } else if (nfull & 1) {
      tail(s4, s5, s6, s7, s0, s3);
    } else {
      tail(s0, s1, s2, s3, s4, s7);
    }
  }
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();

  // Epilogue. A lane holds column m = lane % 32 and, in register r, row n = 8 (r / 4) +
  // 4 h + r % 4 of each 32 x 32 block, i.e. quads of consecutive n. Each wave passes 32 rows
  // of Y at a time through its part of the ring (free by now) and writes whole runs of
  // 32 WI columns; 16-byte chunk c of row m sits at c ^ (m mod chunks per row).
  constexpr int RB = 32 * WI * (int)sizeof(T), CPR = RB / 16, SB = 32 * RB;
  constexpr int WPS = C::SLOTB / SB;                   // waves per slot
  static_assert(C::NW <= 4 * WPS, "staging in the ring");
  uint8_t* S = (wave / WPS == 0 ? s0 : wave / WPS == 1 ? s1 : wave / WPS == 2 ? s2 : s3) +
               (wave % WPS) * SB;
  T* Y = static_cast<T*>(g.Y);
  const int64_t nw = n0 + an;                          // first column of this wave
  const int cols = (int)max((int64_t)0, min((int64_t)32 * WI, g.N - nw));
  const bool whole = (g.N * (int64_t)sizeof(T)) % 16 == 0;
#pragma unroll
  for (int j = 0; j < WJ; ++j) {
    const int64_t mb = m0 + wm * 32 * WJ + 32 * j;
    mx_wave_sync();
#pragma unroll
    for (int i = 0; i < WI; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        mx_stage_quad(reinterpret_cast<T*>(S + fr * RB), CPR, fr, 32 * i + 8 * q + 4 * h,
                      acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                      acc[i][j][4 * q + 3]);
    mx_wave_sync();
    if (whole) {
      constexpr int RPI = 64 / CPR;                    // rows per store instruction
      const int c = lane % CPR;
#pragma unroll
      for (int it = 0; it < 32 / RPI; ++it) {
        const int r = it * RPI + lane / CPR;
        const u32x4 v = *reinterpret_cast<const u32x4*>(S + r * RB + ((c ^ (r % CPR)) << 4));
        if (mb + r < g.M && c * (16 / (int)sizeof(T)) < cols)
          __builtin_nontemporal_store(
              v, reinterpret_cast<u32x4*>(Y + (mb + r) * g.N + nw + c * (16 / sizeof(T))));
      }
    } else {
      // Rows start at any element: words from each row's first 4-byte boundary on, then, in
      // bf16, all rows' single first and last elements together. Everything that does not
      // change from row to row is formed once: the stores were bound by their addresses
      // (515 x 4001 x 4096 bf16: one element per store 16.5 us, so 14.8; N = 4096 13.1).
      constexpr int EPW = 4 / (int)sizeof(T), EPC = 4 * EPW;      // elements per word, chunk
      constexpr int WPR = 32 * WI / EPW;                          // words per row
      constexpr int RPI = WPR < 64 ? 64 / WPR : 1, KW = WPR > 64 ? WPR / 64 : 1;
      const int r0 = WPR < 64 ? lane / WPR : 0;
      T* y = Y + (mb + r0) * g.N + nw;
      const int rows_left = (int)min(g.M - mb - r0, (int64_t)32);
      auto odd = [](const T* q) __attribute__((always_inline)) {
        return EPW == 2 ? (int)(reinterpret_cast<uintptr_t>(q) >> 1) & 1 : 0;
      };
      auto place = [&](int r, int e) __attribute__((always_inline)) {
        return r * RB + (((e / EPC) ^ (r % CPR)) << 4) + e % EPC * (int)sizeof(T);
      };
      // per parity of the row's start: the word's first element and the places of its elements
      int e[2][KW], pl[2][KW], ph[2][KW];
      const int o0 = odd(y), o1 = o0 ^ (RPI == 1 ? (int)(g.N & 1) : 0);
#pragma unroll
      for (int k = 0; k < KW; ++k)
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          e[v][k] = EPW * (64 * k + lane % WPR) + (EPW == 2 ? (v ? o1 : o0) : 0);
          pl[v][k] = place(r0, e[v][k]);
          ph[v][k] = place(r0, min(e[v][k] + EPW - 1, 32 * WI - 1));
        }
#pragma unroll
      for (int it = 0; it < 32 / RPI; ++it) {
        constexpr int MASK = CPR - 1;
        const int x = ((RPI * it) & MASK) << 4, o = RPI * it * RB, v = RPI == 1 ? it & 1 : 0;
#pragma unroll
        for (int k = 0; k < KW; ++k) {
          uint32_t w;
          if constexpr (EPW == 2)
            w = *reinterpret_cast<const uint16_t*>(S + (pl[v][k] ^ x) + o) |
                (uint32_t)*reinterpret_cast<const uint16_t*>(S + (ph[v][k] ^ x) + o) << 16;
          else
            w = *reinterpret_cast<const uint32_t*>(S + (pl[v][k] ^ x) + o);
          if (RPI * it < rows_left && e[v][k] + EPW - 1 < cols)
            *reinterpret_cast<uint32_t*>(y + e[v][k]) = w;
        }
        y += RPI * g.N;
      }
      if constexpr (EPW == 2) {
        const int r = lane & 31;
        T* q = Y + (mb + r) * g.N + nw;
        const bool last = lane >= 32;                  // lanes 0 .. 31: first elements
        if (mb + r < g.M && cols > 0 && (last ? (cols - odd(q)) & 1 : odd(q))) {
          const int f = last ? cols - 1 : 0;
          q[f] = *reinterpret_cast<const T*>(S + place(r, f));
        }
      }
    }
  }
}

// ---- few rows of X ------------------------------------------------------------------------
// Y = X W^T for up to 16 MB rows of X, in MXFP4 (one scaled 16x16x128 product per step of 128
// values) or bfloat16 (four 16x16x32 products on W's values, which are exact in bfloat16). A
// workgroup takes 16 RG rows of W and its waves split the contraction by 512 values; their
// sums are added in wave order through LDS.
// Fragments want row l % 16 in lane l, and a load in which neighbouring lanes read different
// rows costs an address unit 64 lookups instead of 16 (16 rows of bf16 X, 4096 x 14336: the
// units were 80% busy and the product took 18.3 us). So each wave passes its operands through
// a ring of four steps of its own in LDS: direct loads of 16 rows x 64 bytes, 4 lanes to a
// row, chunk c of row r at c ^ ((r / 4) mod 4), and a step's slot is loaded anew as soon as
// it has been read (10.7 us). Waves never wait for each other before the sums. Bound by HBM
// for one row (14336 x 8192: 13.4 us, 4.7 TB/s of weight), with more rows by X, which every
// workgroup reads from L2 (16 rows: 16.1 us); small weights by the launch and one trip to
// memory (4096 x 4096, one row: 3.5 us).
// Step, MXFP4: lane l holds the block q = l / 16 of row l % 16, one scaled operand. bf16 X:
// the four lanes of a row of W first exchange words (a 4 x 4 transpose of rows of 16 lanes),
// after which lane q's word v is word q of block v: product v covers k = 32 v + 8 q .. + 7,
// piece q of the v-th 64 bytes of X, and its scale byte is the same in every lane.
struct MxSkinnyArgs {
  const void* X;               // bf16 [M][K] or MXFP4 codes
  const uint8_t* Xs;
  const uint8_t* Wc;
  const uint8_t* Ws;
  int M;
  int64_t N, nb;
  void* Y;
};

// Eight bfloat16 values of the codes in one word. The conversion takes the scale as a
// float32 exponent: the scale byte in bits 30..23, 0 standing for 2^-127 and 255 for NaN.
__device__ __forceinline__ bf16x8 mx_fp4_bf16(uint32_t w, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Word v of the row-of-16 q <-> word q of the row-of-16 v.
__device__ __forceinline__ u32x4 mx_transpose4(u32x4 w) {
  const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return u32x4{c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ f32x4 mfma16_fp4(u32x4 a, u32x4 b, f32x4 c, uint32_t sa, uint32_t sb) {
  const i32x8 A = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 B = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, c, 4, 4, 0, (int)sa, 0, (int)sb);
}

// Waves per workgroup: four, and eight where a step is short (16 rows of W, up to 4 of bf16 X:
// 1 x 4096 x 14336 8.5 us with four, 7.1 with eight; 1 x 14336 x 8192, 64 rows: 13.4, 14.1).
constexpr int mx_skinny_waves(int xr, int rg) { return xr == 4 && rg == 1 ? 8 : 4; }

// XR: bf16 X of at most XR rows, or 0 for MXFP4 X of up to 16 MB rows. Four rows of bf16 take a
// quarter of the loads and the ring that sixteen do (one row, 4096 x 4096: 4.0 -> 3.5 us).
template <int XR, typename T, int MB, int RG, bool AL>
__global__ __launch_bounds__(mx_skinny_waves(XR, RG) * 64) void k_mxfp4_skinny(MxSkinnyArgs g) {
  constexpr bool XBF = XR > 0;
  static_assert(!XBF || MB == 1, "bf16 rows: one block of 16");
  constexpr int NW = mx_skinny_waves(XR, RG);
  constexpr int XV = XR == 16 ? 4 : 1;               // loads of X per step and block of rows
  constexpr int LOADS = RG + MB * XV, STEPB = LOADS * 1024;
  __shared__ __attribute__((aligned(1024))) uint8_t s0[NW * STEPB], s1[NW * STEPB],
      s2[NW * STEPB], s3[NW * STEPB];
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * (16 * RG), nb = g.nb, rowb = nb * 16;
  const int nch = (int)((nb + 15) >> 4);             // chunks of four steps (512 values)
  const int nfull = (int)(nb >> 4), nt = (int)(nb & 15);

  // direct loads: rows past the matrix are out of the buffer's range and give zeros, and so
  // do pieces past the row, which get an offset outside every buffer
  const int rl = lane >> 2, pc = (lane & 3) ^ ((rl >> 2) & 3);
  const auto wsrc = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(g.Wc + n0 * rowb), 0,
      (int)(min(g.N - n0, (int64_t)(16 * RG)) * rowb), 0x00020000);
  const auto xsrc = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<void*>(g.X), 0, (int)(min(g.M, 16 * MB) * rowb * (XBF ? 4 : 1)), 0x00020000);
  const uint32_t wv = (uint32_t)(rl * rowb + pc * 16);
  // (four rows of bf16: all 256 bytes of a step's row in 16 lanes, piece p of row r at p ^ 4 r)
  const int xr = XR == 4 ? lane >> 4 : rl, xp = XR == 4 ? (lane & 15) ^ (xr << 2) : pc;
  const uint32_t xv = (uint32_t)(xr * rowb * (XBF ? 4 : 1) + xp * 16);
  const uint32_t vstep = (uint32_t)(16 * rowb);
  const int fo = wave * STEPB;
  auto issue = [&](uint8_t* slot, int step) __attribute__((always_inline)) {
    uint8_t* to = slot + fo;
    const bool in = 4 * step + pc < (int)nb;
#pragma unroll
    for (int i = 0; i < RG; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(wsrc, (LCVQ_LDS void*)(to + i * 1024), 16,
                                               (int)(in ? wv + i * vstep : 0xffffffffu), step * 64,
                                               0, 0);
#pragma unroll
    for (int j = 0; j < MB * XV; ++j) {
      const bool xin = XR == 16 ? 4 * step + j < (int)nb
                     : XR == 4  ? 4 * step + (xp >> 2) < (int)nb : in;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          xsrc, (LCVQ_LDS void*)(to + (RG + j) * 1024), 16,
          (int)(xin ? xv + (XBF ? 64 * j : j * vstep) : 0xffffffffu), step * (XBF ? 256 : 64), 0, 0);
    }
  };
  // scales: 16 bytes per row and chunk; of the partial last chunk before everything else
  const uint8_t* sp[RG];
  const uint8_t* xsp[MB];
#pragma unroll
  for (int i = 0; i < RG; ++i) sp[i] = g.Ws + min(n0 + 16 * i + r, g.N - 1) * nb;
#pragma unroll
  for (int j = 0; j < MB; ++j) xsp[j] = XBF ? nullptr : g.Xs + (int64_t)min(16 * j + r, g.M - 1) * nb;
  MxScale16<AL> wsr[RG], xsr[MB];
  u32x4 wtail[RG], xtail[MB];
  auto scale_load = [&](int c) __attribute__((always_inline)) {
    const int64_t b0 = (int64_t)min(c, nfull - 1) * 16;
#pragma unroll
    for (int i = 0; i < RG; ++i) wsr[i].load(sp[i] + b0);
    if constexpr (!XBF) {
#pragma unroll
      for (int j = 0; j < MB; ++j) xsr[j].load(xsp[j] + b0);
    }
  };

  f32x4 acc[RG][MB];
#pragma unroll
  for (int i = 0; i < RG; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // this lane's piece in a slot
  const int ro = fo + r * 64 + ((q ^ ((r >> 2) & 3)) << 4);
  const int xo = fo + RG * 1024 + (r & 3) * 320 + q * 16;    // of X's row r mod 4, v = 0
  auto step = [&](uint8_t* slot, int t, const u32x4 (&ws)[RG], const u32x4 (&xs)[MB], bool more, int next)
      __attribute__((always_inline)) {
    u32x4 w[RG], x[XBF ? 4 : MB];
#pragma unroll
    for (int i = 0; i < RG; ++i) w[i] = *reinterpret_cast<const u32x4*>(slot + ro + i * 1024);
#pragma unroll
    for (int j = 0; j < (XBF ? 4 : MB); ++j)
      x[j] = *reinterpret_cast<const u32x4*>(slot + (XR == 4 ? xo ^ (j << 6) : ro + (RG + j) * 1024));
    if (more) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");     // read, so it may be overwritten
      issue(slot, next);
    }
#pragma unroll
    for (int i = 0; i < RG; ++i) {
      if constexpr (XBF) {
        const u32x4 a = mx_transpose4(w[i]);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float sc = __uint_as_float((ws[i][t] >> (8 * v) & 255u) << 23);
          acc[i][0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              mx_fp4_bf16(a[v], sc), __builtin_bit_cast(bf16x8, x[v]), acc[i][0], 0, 0, 0);
        }
      } else {
#pragma unroll
        for (int j = 0; j < MB; ++j)
          acc[i][j] = mfma16_fp4(w[i], x[j], acc[i][j], ws[i][t] >> (8 * q), xs[j][t] >> (8 * q));
      }
    }
  };
  int c = wave;
  if (c < nch) {
    if (nt) {
#pragma unroll
      for (int i = 0; i < RG; ++i) {
        MxScaleTail<AL> tl;
        tl.load(sp[i] + (int64_t)nfull * 16, nt);
        wtail[i] = tl.get(nt);
      }
      if constexpr (!XBF) {
#pragma unroll
        for (int j = 0; j < MB; ++j) {
          MxScaleTail<AL> tl;
          tl.load(xsp[j] + (int64_t)nfull * 16, nt);
          xtail[j] = tl.get(nt);
        }
      }
    }
    if (nfull) scale_load(c);
    issue(s0, 4 * c);
    issue(s1, 4 * c + 1);
    issue(s2, 4 * c + 2);
    issue(s3, 4 * c + 3);
    u32x4 ws[RG], xs[MB];
    auto scales = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < RG; ++i) ws[i] = c < nfull ? wsr[i].get() : wtail[i];
      if constexpr (!XBF) {
#pragma unroll
        for (int j = 0; j < MB; ++j) xs[j] = c < nfull ? xsr[j].get() : xtail[j];
      }
    };
    for (; c + NW < nch; c += NW) {
      scales();
      if (nfull) scale_load(c + NW);
      // (the scale loads may be among the youngest: then a little more is waited for)
      const int f = 4 * (c + NW);
      mx_landed<3 * LOADS>();
      step(s0, 0, ws, xs, true, f);
      mx_landed<3 * LOADS>();
      step(s1, 1, ws, xs, true, f + 1);
      mx_landed<3 * LOADS>();
      step(s2, 2, ws, xs, true, f + 2);
      mx_landed<3 * LOADS>();
      step(s3, 3, ws, xs, true, f + 3);
    }
    scales();
    mx_landed<3 * LOADS>();
    step(s0, 0, ws, xs, false, 0);
    mx_landed<2 * LOADS>();
    step(s1, 1, ws, xs, false, 0);
    mx_landed<LOADS>();
    step(s2, 2, ws, xs, false, 0);
    mx_landed<0>();
    step(s3, 3, ws, xs, false, 0);
  }

  // the sums: block ij of a wave takes 1 KiB of its part of the ring (which only it reads)
  constexpr int F = STEPB / 1024;
  static_assert(RG * MB <= 2 * F, "sums in the ring");
  auto red = [&](int w, int ij) __attribute__((always_inline)) {
    return reinterpret_cast<f32x4*>((ij < F ? s0 : s1) + w * STEPB + (ij % F) * 1024);
  };
#pragma unroll
  for (int i = 0; i < RG; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j) red(wave, i * MB + j)[lane] = acc[i][j];
  __syncthreads();
  T* Y = static_cast<T*>(g.Y);
  const bool quad = (g.N & 3) == 0;
  for (int e = threadIdx.x; e < RG * MB * 64; e += NW * 64) {
    const int ij = e >> 6, l = e & 63;
    f32x4 v = red(0, ij)[l];
#pragma unroll
    for (int w = 1; w < NW; ++w) v += red(w, ij)[l];
    const int m = 16 * (ij % MB) + (l & 15);
    const int64_t n = n0 + 16 * (ij / MB) + 4 * (l >> 4);
    if (m >= g.M || n >= g.N) continue;
    T* y = Y + (int64_t)m * g.N + n;
    if (quad) {
      store4(y, v);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (n + k < g.N) store1(y + k, v[k]);
    }
  }
}

template <typename T, int WI, int WJ, int NWN, int NWM, int RING>
static hipError_t launch_tile(MxGemmArgs g, hipStream_t s) {
  using C = MxTile<WI, WJ, NWN, NWM, RING>;
  g.tilesN = (int)((g.N + C::BN - 1) / C::BN);
  g.tilesM = (int)((g.M + C::BM - 1) / C::BM);
  g.ntiles = g.tilesN * g.tilesM;
  const dim3 grid((unsigned)((g.ntiles + 7) / 8 * 8)), block(C::NW * 64);
  constexpr int id = C::BN == 256   ? PROF_MX_256
                     : C::BN == 128 ? PROF_MX_128
                     : C::BM == 128 ? PROF_MX_64_128 : PROF_MX_64;
  if (g.nb % 4 == 0)
    LCVQ_LAUNCH(id, (k_mxfp4_tile<T, WI, WJ, NWN, NWM, RING, true>), grid, block, 0, s, g);
  else
    LCVQ_LAUNCH(id, (k_mxfp4_tile<T, WI, WJ, NWN, NWM, RING, false>), grid, block, 0, s, g);
  return hipGetLastError();
}

template <int XR, typename T, int MB, int RG>
static hipError_t launch_skinny(const MxSkinnyArgs& g, hipStream_t s) {
  const dim3 grid((unsigned)((g.N + 16 * RG - 1) / (16 * RG))), block(mx_skinny_waves(XR, RG) * 64);
  constexpr int id = XR ? PROF_MX_GEMV : PROF_MX_FEW;
  if (g.nb % 4 == 0)
    LCVQ_LAUNCH(id, (k_mxfp4_skinny<XR, T, MB, RG, true>), grid, block, 0, s, g);
  else
    LCVQ_LAUNCH(id, (k_mxfp4_skinny<XR, T, MB, RG, false>), grid, block, 0, s, g);
  return hipGetLastError();
}

// Rows of W per workgroup: the more, the fewer times X is read (from L2), the fewer, the more
// workgroups share the weight: the fewest of 16, 32 and 64 that give a CU at most one.
// (bf16 X, 16 rows, 16 / 32 / 64: 4096 x 4096 4.2 us, 5.6, 7.7; 8192 x 4096 7.7, 6.7, 8.6;
// 14336 x 4096 11.7, 11.2, 10.2; MXFP4 X: 3.0, 4.0, 5.6; 5.4, 4.9, 6.3; 8.2, 7.4, 7.6.)
template <int XR, typename T, int MB>
static hipError_t skinny_rows(const MxSkinnyArgs& g, hipStream_t s) {
  if (g.N <= 16 * 256) return launch_skinny<XR, T, MB, 1>(g, s);
  if (g.N <= 32 * 256) return launch_skinny<XR, T, MB, 2>(g, s);
  return launch_skinny<XR, T, MB, 4>(g, s);
}

template <int WI, int WJ, int RING>
static hipError_t tile_typed(const MxGemmArgs& g, bool y_f32, hipStream_t s) {
  return y_f32 ? launch_tile<float, WI, WJ, 2, 2, RING>(g, s)
               : launch_tile<uint16_t, WI, WJ, 2, 2, RING>(g, s);
}

hipError_t launch_mxfp4_gemm(const uint8_t* Xc, const uint8_t* Xs, int64_t M, int64_t N,
                             int64_t K, const uint8_t* Wc, const uint8_t* Ws, void* Y, bool y_f32,
                             hipStream_t s) {
  const MxSkinnyArgs k{Xc, Xs, Wc, Ws, (int)std::min<int64_t>(M, 64), N, K / MXB, Y};
  if (M <= 16) return y_f32 ? skinny_rows<0, float, 1>(k, s) : skinny_rows<0, uint16_t, 1>(k, s);
  if (M <= 32) return y_f32 ? skinny_rows<0, float, 2>(k, s) : skinny_rows<0, uint16_t, 2>(k, s);
  MxGemmArgs g = {};
  g.Xc = Xc; g.Xs = Xs; g.Wc = Wc; g.Ws = Ws;
  g.M = M; g.N = N; g.nb = K / MXB;
  g.Y = Y;
  // Tiles: 256 x 256 where more than half of the 256 CUs get one; else the largest of which
  // a smaller one would give a CU more than one: 64 x 64, 64 rows of W by 128 of X, 128 x 128.
  // (K = 4096, with 256 / 128 / 64 x 128 / 64: 2048 x 4096 28.4 us, 26.8; 1024 x 4096 24.4,
  // 13.1, 18.7; 512 x 4096 23.9, 10.7, 10.4, 12.9; 128 x 14336 with 128 on: 11.4, 10.7, 12.4;
  // 256 x 4096 9.8, 9.3, 7.9.) One small tile per CU needs eight slots for its loads to be on
  // time (64 x 4096 x 14336: 24.7 us with four, 17.6); for the larger the longer fill costs
  // as much as it gives (515 x 4001 x 4128, 128: 16.0 us with four, 16.9).
  auto tiles = [&](int64_t n, int64_t m) { return ((M + m - 1) / m) * ((N + n - 1) / n); };
  if (tiles(256, 256) > 128) return tile_typed<4, 4, 4>(g, y_f32, s);
  if (tiles(64, 64) <= 256) return tile_typed<1, 1, 8>(g, y_f32, s);
  if (tiles(64, 128) <= 256) return tile_typed<1, 2, 4>(g, y_f32, s);
  return tile_typed<2, 2, 4>(g, y_f32, s);
}

hipError_t launch_mxfp4_gemv(const uint16_t* X, int M, int64_t N, int64_t K, const uint8_t* Wc,
                             const uint8_t* Ws, uint16_t* Y, hipStream_t s) {
  const MxSkinnyArgs k{X, nullptr, Wc, Ws, M, N, K / MXB, Y};
  return M <= 4 ? skinny_rows<4, uint16_t, 1>(k, s) : skinny_rows<16, uint16_t, 1>(k, s);
}

}  // namespace lcvq
