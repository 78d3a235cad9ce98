// Products with 16-bit weights: out[p, q] = act(sum_r a(p, r) b(q, r) + bias[q]) + res[p, q], each
// operand's inner index r along its rows or down its columns.
#include <algorithm>

#include "swq_dense.h"
#include "swq_dense_device.h"

namespace swq {
namespace {

// A buffer offset past every buffer's end: the load returns zeros and touches no memory.
constexpr uint32_t kNowhere = 0xFFFFFFF0u;

typedef short i16x4 __attribute__((ext_vector_type(4)));

template <int N, int I = 0, class F>
__device__ __forceinline__ void each(F f) {
  if constexpr (I < N) {
    f.template operator()<I>();
    each<N, I + 1>(f);
  }
}

template <int TYPE>
__device__ __forceinline__ f32x4 mfma_16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (TYPE == kTypeF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                   0);
}
// XCD-aware order of the tiles: the hardware deals consecutive blocks to the eight XCDs in turn, so block b
// takes tile b / 8 of a contiguous eighth of the order, and an XCD's L2 sees neighbours.  In the
// order, bands of eight row tiles run along their columns (bands of 4 the same, of 2 and 16 3 % slower, of 1 and 32 5 to 15).
__device__ __forceinline__ bool tile_at(int b, int ntp, int ntq, int& tp, int& tq) {
  constexpr int high = 8;
  const int total = ntp * ntq, per = (total + 7) / 8;
  const int t = (b & 7) * per + (b >> 3);
  if ((b >> 3) >= per || t >= total) return false;
  const int band = t / (high * ntq), in = t - band * high * ntq, rows = min(high, ntp - high * band);
  tp = high * band + in % rows;
  tq = in / rows;
  return true;
}

// ------------------------------------------------------------------ epilogue ----

// Eight neighbouring 16-bit values, n of them (0 .. 8) there.
__device__ __forceinline__ u32x4 load8(const uint16_t* f, int n) {
  if (n == 8) return *(const u32x4_any*)f;
  u32x4 w = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < n) w[j >> 1] |= (uint32_t)f[j] << (16 * (j & 1));
  return w;
}
template <int TYPE>
__device__ __forceinline__ void add8(float (&v)[8], u32x4 w) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] += from_16((uint16_t)(w[j >> 1] >> (16 * (j & 1))), TYPE);
}
// The bias of columns q .., and the residual of (p, q ..); zeros where there is none.
__device__ __forceinline__ u32x4 bias_at(const DenseGemm& g, int64_t q, int n) {
  return g.bias ? load8(g.bias + q, n) : (u32x4){0, 0, 0, 0};
}
__device__ __forceinline__ u32x4 residual_at(const DenseGemm& g, int64_t p, int64_t q, int n) {
  return g.res && p < g.P ? load8(g.res + p * g.Q + q, n) : (u32x4){0, 0, 0, 0};
}

// STREAM: stores marked as not to be kept, for the tiles.  256 tiles of 256 x 256 leave 33 MB at once, as much as
// the L2s hold, which would drive the operands out: 2 to 9 % of the time (8192 x 2560 x 4096 with GELU and a checkpoint 151
// against 166 us, 2048 x 2048 x 5632 53 against 56).
template <bool STREAM, class T>
__device__ __forceinline__ void put(T* o, T w) {
  if constexpr (STREAM) __builtin_nontemporal_store(w, o);
  else *o = w;
}
template <int TYPE, bool STREAM>
__device__ __forceinline__ void store8(uint16_t* o, const float (&v)[8], int n) {
  if (n == 8) {
    put<STREAM>((u32x4_any*)o, (u32x4_any){pack16<TYPE>(v[0], v[1]), pack16<TYPE>(v[2], v[3]), pack16<TYPE>(v[4], v[5]),
                                           pack16<TYPE>(v[6], v[7])});
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) o[j] = to_16(v[j], TYPE);
  }
}

// The largest of four neighbouring lanes.
__device__ __forceinline__ uint32_t max_of_four(uint32_t m) {
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, true));
  return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, true));
}

// Eight neighbouring sums of row p from column q on, n of them (0 .. 8) in the matrix; four neighbouring lanes
// have a block of 32 columns, and all four call it.  STREAM: as above.
template <int TYPE, bool STREAM>
__device__ __forceinline__ void finish8(const DenseGemm& g, float (&v)[8], int64_t p, int64_t q, int n, u32x4 bias,
                                        u32x4 residual) {
  const int64_t at = p * g.Q + q;
  if (g.bias) add8<TYPE>(v, bias);
  if (g.z) {
    if (g.z_scales) {
      if (n < 8) {                     // (what is behind the last column counts for nothing)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < n ? v[j] : 0.0f;
      }
      const Mx8Step s = mx8_step(max_of_four(mx8_amax(v)));
      const u32x2 w = mx8_codes(v, s);
      uint8_t* z = (uint8_t*)g.z + at;
      if (n == 8) {
        put<STREAM>((u32x2_any*)z, (u32x2_any)w);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < n) z[j] = (uint8_t)(w[j >> 2] >> (8 * (j & 3)));
      }
      if ((q & 31) == 0 && n > 0) g.z_scales[p * ((g.Q + 31) / 32) + q / 32] = (uint8_t)s.byte;
    } else {
      store8<TYPE, STREAM>((uint16_t*)g.z + at, v, n);
    }
  }
  const auto through = [&](int act) SWQ_INLINE {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = activate(v[j], act);
  };
  switch (g.act) {                     // one branch for eight values
    case kActRelu: through(kActRelu); break;
    case kActSilu: through(kActSilu); break;
    case kActGelu: through(kActGelu); break;
    case kActGeluTanh: through(kActGeluTanh); break;
  }
  if (g.res) add8<TYPE>(v, residual);
  if (g.out_type == kTypeF32) {
    float* o = (float*)g.out + at;
    if (n == 8) {
      put<STREAM>((u32x4_any*)o, __builtin_bit_cast(u32x4_any, (f32x4){v[0], v[1], v[2], v[3]}));
      put<STREAM>((u32x4_any*)(o + 4), __builtin_bit_cast(u32x4_any, (f32x4){v[4], v[5], v[6], v[7]}));
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) o[j] = v[j];
    }
  } else {
    store8<TYPE, STREAM>((uint16_t*)g.out + at, v, n);
  }
}

// -------------------------------------------------------------------- tiles ----
//
// WP x WQ waves, each AF by BF accumulators of 16 x 16 (rows by columns).  A stage is 64 inner indexes of both operands in
// LDS, S stages, filled by loads that write LDS.  A step of 32 takes its products row by row; a row's operand is read for
// the next step as soon as its products are issued, the columns' operands are read ahead into a second set.  In the
// last step of a stage the waves meet after the first rows, when every read of the stage has long been
// answered: then the next stage is there, and the one that was read makes room for the loads of the one S ahead.
//
// Along: a row's 64 elements are 128 bytes, 16-byte unit u at u ^ (row / 2 & 7), and a lane's operand (eight
// neighbours of a row) is one read.  Down: an inner index's BP elements are a row of LDS, unit u at
// u ^ (4 (r & 3) + 2 (r / 8 & 1)) (BP = 64: 4 (r / 2 & 1) for the first), and an operand is two transposing reads of
// four inner indexes by 16 columns each.  Either way the rows that a read touches lie in different banks.
//
// The second operand of the products is a, so that lane 16 h + r has row r's columns 4 h .. 4 h + 3; the sums leave
// through the wave's own stretch of LDS, 32 rows at a time, as whole lines.
//
// What bounds it: matrix units 71 % of the cycles busy at the 1.9 GHz that the card's power leaves (8192 x 8192 x 8192
// in 784 to 838 us, 1.31 to 1.40 PFLOP/s).  Without its loads the same loop takes 624, with all of them from L2 726: the
// misses' latency, a stage's loads having one stage's time to come, and the loads' share of power and LDS.  Products of
// 32 x 32 x 16 took a tenth longer.  8192 x 4096 x 4096 takes 202 to 215, 2048 x 4096 x 14336 203 to 217 (448 tiles fill
// seven eighths of two rounds of 256 CUs); of that 8 to 14 a round are the stores of 256 tiles at once, as
// nothing else runs on a CU meanwhile.  An epilogue of GELU, bias and residual adds 18 us there, of SiLU, residual and checkpoint 24.
template <int AF_, int BF_, int WP_, int WQ_, int S_, int OCC_>
struct DenseShape {
  static constexpr int AF = AF_, BF = BF_, WP = WP_, WQ = WQ_, S = S_, OCC = OCC_, KS = 64;
  static constexpr int W = WP * WQ, BP = 16 * AF * WP, BQ = 16 * BF * WQ;
  static constexpr int LOADS_A = BP * KS / (512 * W), LOADS = (BP + BQ) * KS / (512 * W);     // per wave and stage
  static constexpr int STAGE_A = LOADS_A * W * 1024, STAGE = LOADS * W * 1024;
  static constexpr int PITCH = 16 * BF + 4, FLUSH = 32 * PITCH * 4;             // floats; bytes of a wave's stretch
  static constexpr int LDS = S * STAGE > W * FLUSH ? S * STAGE : W * FLUSH;
  static_assert(BP * KS % (512 * W) == 0 && BQ * KS % (512 * W) == 0 && W % 2 == 0 && AF % 2 == 0 && BF % 2 == 0);
};

// A load of 16 bytes per lane to LDS at lds + FROM, `soff` bytes further than the lane's offset (which alone counts for
// the range check; the wait state is what a load that writes LDS needs behind a write of m0).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
template <int FROM>
__device__ __forceinline__ void dma16_at(i32x4 rs, uint32_t lds, uint32_t voff, uint32_t soff) {
  asm volatile("s_add_u32 m0, %0, %4\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               ::"s"(lds), "v"(voff), "s"(rs), "s"(soff), "n"(FROM) : "memory", "m0", "scc");
}
#pragma clang diagnostic pop

// One operand: its loads and its place in LDS.  Load i of a wave takes the 64 units (W i + wave) 64 + lane of a stage.
// Along: the descriptor has the tile's rows, a stage's offset is added behind the range check, so there are no
// bytes at all behind the last stage, whose lanes past R read nothing.  Down: the descriptor moves with the stage
// and ends at R.
template <int WAY, int BP, int W>
struct Operand {
  static constexpr int KS = 64;
  static constexpr int UNITS = WAY == kAlong ? KS / 8 : BP / 8, LOADS = BP * KS / (512 * W);  // 16-byte units of a row of LDS
  static constexpr int along_swap(int row) { return row >> 1 & 7; }
  i32x4 rs;
  uint64_t at;              // Down: the stage's address
  int64_t left;             // Down: bytes from there to the end
  int64_t ld;
  uint32_t off[LOADS];      // the lane's offsets
  int k, tail;              // Along: the lane's first inner index of a stage; indexes of the last stage

  // Down: rows of LDS of 256 bytes and more begin in the same bank, of 128 every second; a read takes four neighbouring
  // rows twice, eight rows apart
  static constexpr int swap(int r) { return (BP >= 128 ? (r & 3) << 2 : (r >> 1 & 1) << 2) ^ (r >> 3 & 1) << 1; }

  __device__ __forceinline__ void aim(const uint16_t* x, int64_t ld_, int64_t first, int64_t n, int64_t r0, int64_t r1,
                                      int wave, int lane) {
    ld = ld_;
    if constexpr (WAY == kAlong) {
      const int64_t rows = min(n - first, (int64_t)BP);
      rs = make_srsrc(x + first * ld + r0, (uint32_t)((rows * ld - r0) * 2));
      const int unit = lane % UNITS ^ along_swap(64 / UNITS * wave + lane / UNITS);     // (W even: the same in every load)
#pragma unroll
      for (int i = 0; i < LOADS; ++i)
        off[i] = (uint32_t)((64 / UNITS * (W * i + wave) + lane / UNITS) * ld * 2) + unit * 16;
      k = unit * 8;
      tail = (int)((r1 - r0 - 1) & (KS - 1)) + 1;
    } else {
      at = (uint64_t)(x + r0 * ld + first);
      left = ((r1 - r0) * ld - first) * 2;
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int u = (W * i + wave) * 64 + lane, row = u / UNITS;
        off[i] = (uint32_t)(row * ld * 2) + (u % UNITS ^ swap(row)) * 16;
      }
    }
  }
  // before the loads of stage t; the stages come in order
  __device__ __forceinline__ void begin(int t, int stages) {
    if constexpr (WAY == kDown) {
      const int64_t n = left < 0 ? 0 : left < (int64_t)kNowhere ? left : (int64_t)kNowhere;
      rs = make_srsrc((const void*)at, (uint32_t)n);
    } else {
      if (t == stages - 1) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) off[i] = k < tail ? off[i] : kNowhere;
      }
      if (t >= stages) rs[2] = 0;
    }
  }
  template <int i, int FROM>
  __device__ __forceinline__ void load(int t, uint32_t lds) const {
    dma16_at<FROM + W * i * 1024>(rs, lds, off[i], WAY == kAlong ? (uint32_t)t * (2u * KS) : 0u);
  }
  __device__ __forceinline__ void end() {
    if constexpr (WAY == kDown) {
      at += (uint64_t)(ld * (2 * KS));
      left -= ld * (2 * KS);
    }
  }
  // the lane's operand of step s, tile `tile` (of 16) of the block's
  static __device__ __forceinline__ u32x4 read(const char* lds, int s, int tile, int lane) {
    const int h = lane >> 4, r = lane & 15;
    if constexpr (WAY == kAlong) {
      return *(const u32x4*)(lds + (16 * tile + r) * (2 * KS) + (((4 * s + h) ^ along_swap(r)) * 16));
    } else {
      const int row = 8 * h + (r >> 2);
      const char* a = lds + (32 * s + row) * (BP * 2) + (((2 * tile + (r >> 1 & 1)) ^ swap(row)) * 16) + (r & 1) * 8;
      typedef __attribute__((address_space(3))) i16x4* lds4;
      const i16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(lds_ptr_t)a);
      const i16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(lds_ptr_t)(a + 4 * BP * 2));
      const u32x2 u = __builtin_bit_cast(u32x2, x), v = __builtin_bit_cast(u32x2, y);
      return (u32x4){u[0], u[1], v[0], v[1]};
    }
  }
};

// A tile of g by the block: split `part` of the tile that `block` stands for (none: nothing is done).  PLAIN: nothing but the
// sums, rounded.
template <int TYPE, int WAY_A, int WAY_B, bool PLAIN, class Sh>
__device__ __forceinline__ void dense_tile(const DenseGemm& g, int block, int part, char* lds) {
  constexpr int AF = Sh::AF, BF = Sh::BF, WQ = Sh::WQ, S = Sh::S, W = Sh::W, BP = Sh::BP, BQ = Sh::BQ;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wp = wave / WQ, wq = wave % WQ;
  int tp, tq;
  if (!tile_at(block, (int)((g.P + BP - 1) / BP), (int)((g.Q + BQ - 1) / BQ), tp, tq)) return;
  const int64_t p0 = (int64_t)tp * BP, q0 = (int64_t)tq * BQ;
  const int64_t r0 = (int64_t)part * g.split_len, r1 = min(r0 + g.split_len, g.R);
  constexpr int KS = Sh::KS;
  const int stages = (int)((r1 - r0 + KS - 1) / KS);

  Operand<WAY_A, BP, W> oa;
  Operand<WAY_B, BQ, W> ob;
  oa.aim(g.a, g.lda, p0, g.P, r0, r1, wave, lane);
  ob.aim(g.b, g.ldb, q0, g.Q, r0, r1, wave, lane);
  // load i of a stage; the stages are asked for in order
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(lds) + wave * 1024);
  const auto load = [&]<int i>(int t, int slot) SWQ_INLINE {
    if constexpr (i == 0) oa.begin(t, stages), ob.begin(t, stages);
    const uint32_t base = lds0 + slot * Sh::STAGE;
    if constexpr (i < Sh::LOADS_A) oa.template load<i, 0>(t, base);
    else ob.template load<i - Sh::LOADS_A, Sh::STAGE_A>(t, base);
    if constexpr (i == Sh::LOADS - 1) oa.end(), ob.end();
  };

  f32x4 acc[AF][BF];
  u32x4 a[AF], b[2][BF];
  const auto read_a = [&]<int i>(int s, int slot) SWQ_INLINE {
    a[i] = oa.read(lds + slot * Sh::STAGE, s, wp * AF + i, lane);
  };
  const auto read_b = [&]<int set, int j>(int slot) SWQ_INLINE {
    b[set][j] = ob.read(lds + slot * Sh::STAGE + Sh::STAGE_A, set, wq * BF + j, lane);
  };
  const auto meet = [&]() SWQ_INLINE {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  // The products of rows FROM .. TO - 1 of a step; before(n) is issued in front of the n-th, after(i) behind a row's.
  const auto products = [&]<int SET, int FROM, int TO>(auto before, auto after) SWQ_INLINE {
    each<(TO - FROM) * BF>([&]<int n>() SWQ_INLINE {
      constexpr int i = FROM + n / BF, j = n % BF;
      before.template operator()<n>();
      acc[i][j] = mfma_16<TYPE>(b[SET][j], a[i], acc[i][j]);
      if constexpr (j == BF - 1) after.template operator()<i>();
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  each<S>([&]<int t>() SWQ_INLINE { each<Sh::LOADS>([&]<int i>() SWQ_INLINE { load.template operator()<i>(t, t); }); });
#pragma unroll
  for (int i = 0; i < AF; ++i)
#pragma unroll
    for (int j = 0; j < BF; ++j) acc[i][j] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
  wait_vmcnt<(S - 1) * Sh::LOADS>();
  meet();
  int slot = 0;
  each<BF>([&]<int j>() SWQ_INLINE { read_b.template operator()<0, j>(0); });
  each<AF>([&]<int i>() SWQ_INLINE { read_a.template operator()<i>(0, 0); });
  // Loads are issued past the last stage too (they read nothing), so the counts hold to the end.
  constexpr int EARLY = AF >= 4 ? AF / 4 : 1, LEFT = (AF - EARLY) * BF;
  constexpr int FREE = BF + EARLY + Sh::LOADS, PER = (FREE + LEFT - 1) / LEFT;
  for (int t = 0; t < stages; ++t) {
    products.template operator()<0, 0, AF>(
        [&]<int n>() SWQ_INLINE {
          if constexpr (n < BF) read_b.template operator()<1, n>(slot);
        },
        [&]<int i>() SWQ_INLINE { read_a.template operator()<i>(1, slot); });
    products.template operator()<1, 0, EARLY>([&]<int n>() SWQ_INLINE {}, [&]<int i>() SWQ_INLINE {});
    wait_vmcnt<(S - 2) * Sh::LOADS>();           // stage t + 1 is there
    meet();
    const int was = slot;
    slot = slot + 1 == S ? 0 : slot + 1;
    products.template operator()<1, EARLY, AF>(
        [&]<int n>() SWQ_INLINE {
          each<PER>([&]<int e>() SWQ_INLINE {
            constexpr int k = n * PER + e;
            if constexpr (k < BF) read_b.template operator()<0, k>(slot);
            else if constexpr (k < BF + EARLY) read_a.template operator()<k - BF>(0, slot);
            else if constexpr (k < FREE) load.template operator()<k - BF - EARLY>(t + S, was);
          });
        },
        [&]<int i>() SWQ_INLINE { read_a.template operator()<i>(0, slot); });
  }
  wait_vmcnt<0>();           // no load past the end may still write LDS
  meet();

  float* buf = (float*)(lds + wave * Sh::FLUSH);
  constexpr int LANES = 2 * BF, ROWS = 64 / LANES;                     // of a row; rows at a time
  const int r = lane & 15, h = lane >> 4, col = lane % LANES * 8;
  const int64_t q = q0 + wq * 16 * BF + col;
  const int n = q + 8 <= g.Q ? 8 : q < g.Q ? (int)(g.Q - q) : 0;
  // The residual comes a round of 32 rows ahead.
  constexpr int PASSES = (32 + ROWS - 1) / ROWS;
  const int64_t pw = p0 + wp * 16 * AF + lane / LANES;
  const bool idle = lane >= ROWS * LANES;      // (of rows that do not fill the wave)
  const bool whole = g.splits <= 1, ahead_too = !PLAIN && whole && g.res;
  const u32x4 bias = PLAIN || !whole ? (u32x4){0, 0, 0, 0} : bias_at(g, q, n);
  u32x4 ahead[PASSES] = {};
  if (ahead_too) {
#pragma unroll
    for (int k = 0; k < PASSES; ++k) ahead[k] = residual_at(g, pw + k * ROWS, q, idle ? 0 : n);
  }
  each<AF / 2>([&]<int i>() SWQ_INLINE {
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int j = 0; j < BF; ++j) *(f32x4*)(buf + (16 * e + r) * Sh::PITCH + 16 * j + 4 * h) = acc[2 * i + e][j];
#pragma unroll(64 % LANES ? 1 : 2)
    for (int k = 0; k < 32; k += ROWS) {             // (two at once: 1 to 4 % faster, of rows of twelve lanes 4 % slower)
      const int row = min(k + lane / LANES, 31);
      const int64_t p = pw + i * 32 + k;
      const f32x4 x = *(const f32x4*)(buf + row * Sh::PITCH + col), y = *(const f32x4*)(buf + row * Sh::PITCH + col + 4);
      float v[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
      const u32x4 residual = ahead[0];
      if (ahead_too) {
#pragma unroll
        for (int e = 0; e + 1 < PASSES; ++e) ahead[e] = ahead[e + 1];
        if constexpr (2 * i + 2 < AF) ahead[PASSES - 1] = residual_at(g, p + 32, q, idle ? 0 : n);
      }
      if (p >= g.P || idle || k + lane / LANES >= 32) continue;
      if (!whole) {
        if (n > 0) {
          float* o = g.parts + ((int64_t)part * g.P + p) * g.part_ld + q;
          *(f32x4*)o = x;
          *(f32x4*)(o + 4) = y;
        }
      } else if constexpr (PLAIN) {
        store8<TYPE, true>((uint16_t*)g.out + p * g.Q + q, v, n);
      } else {
        finish8<TYPE, true>(g, v, p, q, n, bias, residual);
      }
    }
  });
}

template <int TYPE, class Sh>
__global__ __launch_bounds__(64 * Sh::W, Sh::OCC * Sh::W / 4) void dense_kernel(DenseGemm g) {
  __shared__ __attribute__((aligned(1024))) char lds[Sh::LDS];
#ifdef SWQ_LDS_POISON
  lds_poison(lds, sizeof(lds), kPoisonFloat);
  __syncthreads();
#endif
  dense_tile<TYPE, kAlong, kAlong, false, Sh>(g, blockIdx.x, blockIdx.y, lds);
}

// The gradients by x and by W in one launch, the longer tiles first, so that each fills the CUs that the other leaves
// idle; behind them the bias's gradient, the sums of the stretches' sums, 64 columns a block.  2048 x 4096 x 14336 takes 385
// to 415 us (1.16 to 1.25 PFLOP/s, matrix units 54 % of the cycles busy, 1.3 GB past the L2s), one launch each 210 + 220.
template <int TYPE, class Sh>
__global__ __launch_bounds__(64 * Sh::W, Sh::OCC * Sh::W / 4) void dense_pair_kernel(DensePair d) {
  __shared__ __attribute__((aligned(1024))) char lds[Sh::LDS];
#ifdef SWQ_LDS_POISON
  lds_poison(lds, sizeof(lds), kPoisonFloat);
  __syncthreads();
#endif
  int block = blockIdx.x;
  const int first = d.w_first ? d.w_blocks : d.x_blocks, both = d.x_blocks + d.w_blocks;
  if (block < both) {
    const bool of_w = (block < first) == (d.w_first != 0);
    if (block >= first) block -= first;
    if (of_w) {
      const int each = d.w_blocks / d.w.splits;
      dense_tile<TYPE, kDown, kDown, true, Sh>(d.w, block % each, block / each, lds);
    } else {
      const int each = d.x_blocks / d.x.splits;
      dense_tile<TYPE, kAlong, kDown, true, Sh>(d.x, block % each, block / each, lds);
    }
    return;
  }
  const int c = threadIdx.x & 63, team = threadIdx.x >> 6;
  const int64_t n = (int64_t)(block - both) * 64 + c;
  float sum = 0.0f;
  if (n < d.N) {
#pragma unroll 8
    for (int i = team; i < d.n_sums; i += Sh::W) sum += d.sums[(int64_t)i * d.N + n];
  }
  float* meet = (float*)lds;
  meet[threadIdx.x] = sum;
  __syncthreads();
  if (team == 0 && n < d.N) {
    for (int i = 1; i < Sh::W; ++i) sum += meet[64 * i + c];
    d.dbias[n] = to_16(sum, TYPE);
  }
}

// The sums of a split, added in its order.
template <int TYPE>
__global__ __launch_bounds__(256) void dense_join_kernel(DenseGemm g, uint32_t per_row) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t p = over(i, per_row), q = 8 * (i - p * per_row);
  if (p >= g.P) return;                        // four neighbouring lanes leave together
  const int n = q + 8 <= g.Q ? 8 : q < g.Q ? (int)(g.Q - q) : 0;
  float v[8] = {};
  if (n > 0) {
#pragma unroll 4
    for (int s = 0; s < g.splits; ++s) {
      const float* f = g.parts + ((int64_t)s * g.P + p) * g.part_ld + q;
      const f32x4 x = *(const f32x4*)f, y = *(const f32x4*)(f + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += x[j], v[4 + j] += y[j];
    }
  }
  finish8<TYPE, false>(g, v, p, q, n, bias_at(g, q, n), residual_at(g, p, q, n));
}

// ----------------------------------------------------------------- few rows ----
//
// Up to 16 RT rows by 16 CT columns per block, both operands along their rows and straight to registers, at any
// address and of any length.  The waves take chunks of 256 inner indexes in turn, all loads of a chunk in flight, and
// their sums meet in LDS, added in wave order.  The weights' bytes count here: every weight is read once per block
// of rows.  1 x 2048 x 5632 from memory 7.1 us (3.2 TB/s, latency: the launch, one round of loads, the join), 1 x 4096 x
// 14336 23.7 (5.0 TB/s).  Sixteen waves with chunks of 128 took 8.8 and 36, four waves 8.9 and 26.  ODD: the rows begin at
// odd elements (32 x 1003 x 2049 7.0 us; by 16-byte loads at any address 8.6; 32 x 1024 x 2048 5.3).
constexpr int kFewWaves = 8;
// Eight neighbours at any address: as aligned words, which load several times faster than 16 bytes at an odd
// element.  (A word holds one of the eight at least, so none lies outside the tensor's pages.)
template <bool ODD>
__device__ __forceinline__ u32x4 load8_odd(const uint16_t* f) {
  typedef __attribute__((ext_vector_type(4), aligned(4))) uint32_t u32x4_words;
  if constexpr (!ODD) return *(const u32x4_words*)f;
  const uint32_t shift = (uint32_t)(uintptr_t)f & 2u;
  const uint32_t* w = (const uint32_t*)((uintptr_t)f - shift);
  const u32x4 v = *(const u32x4_words*)w;
  const uint32_t next = w[3 + (shift >> 1)];
  return (u32x4){__builtin_amdgcn_alignbyte(v[1], v[0], shift), __builtin_amdgcn_alignbyte(v[2], v[1], shift),
                 __builtin_amdgcn_alignbyte(v[3], v[2], shift), __builtin_amdgcn_alignbyte(next, v[3], shift)};
}

template <int TYPE, int RT, int CT, bool ODD>
__global__ __launch_bounds__(64 * kFewWaves) void dense_few_kernel(DenseGemm g) {
  constexpr int PITCH = 16 * CT + 4, W = kFewWaves, U = ODD && RT > 1 ? 4 : 8;
  __shared__ __attribute__((aligned(16))) float sums[W * 16 * RT * PITCH];
#ifdef SWQ_LDS_POISON
  lds_poison(sums, sizeof(sums), kPoisonFloat);
  __syncthreads();
#endif
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, h = lane >> 4;
  const int64_t q0 = (int64_t)blockIdx.x * (16 * CT), p0 = (int64_t)blockIdx.y * (16 * RT);
  const uint16_t* x[RT];
  const uint16_t* w[CT];
#pragma unroll
  for (int i = 0; i < RT; ++i) x[i] = g.a + min(p0 + 16 * i + r, g.P - 1) * g.lda + 8 * h;
#pragma unroll
  for (int j = 0; j < CT; ++j) w[j] = g.b + min(q0 + 16 * j + r, g.Q - 1) * g.ldb + 8 * h;
  f32x4 acc[RT][CT] = {};
  const int R = (int)g.R, full = R / (32 * U);
  for (int c = wave; c < full; c += W) {
    u32x4 a[RT][U], b[CT][U];
#pragma unroll
    for (int s = 0; s < U; ++s)
#pragma unroll
      for (int j = 0; j < CT; ++j) b[j][s] = load8_odd<ODD>(w[j] + 32 * (U * c + s));
#pragma unroll
    for (int s = 0; s < U; ++s)
#pragma unroll
      for (int i = 0; i < RT; ++i) a[i][s] = load8_odd<ODD>(x[i] + 32 * (U * c + s));
    __builtin_amdgcn_sched_barrier(0);         // (all of them on their way first)
#pragma unroll
    for (int s = 0; s < U; ++s)
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < CT; ++j) acc[i][j] = mfma_16<TYPE>(b[j][s], a[i][s], acc[i][j]);
  }
  // the rest, a step per wave, element by element at its end
#pragma unroll 1
  for (int k = 32 * (U * full + wave); k < R; k += 32 * W) {
    u32x4 a[RT], b[CT];
    const int n = min(max(R - k - 8 * h, 0), 8);
#pragma unroll
    for (int j = 0; j < CT; ++j) b[j] = load8(w[j] + k, n);
#pragma unroll
    for (int i = 0; i < RT; ++i) a[i] = load8(x[i] + k, n);
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < CT; ++j) acc[i][j] = mfma_16<TYPE>(b[j], a[i], acc[i][j]);
  }
  // lane 16 h + r has columns 4 h .. 4 h + 3 of row r
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < CT; ++j)
      *(f32x4*)(sums + ((wave * RT + i) * 16 + r) * PITCH + 16 * j + 4 * h) = acc[i][j];
  __syncthreads();
  for (int t = threadIdx.x; t < 32 * RT * CT; t += 64 * W) {
    const int row = t / (2 * CT), col = t % (2 * CT) * 8;
    const int64_t p = p0 + row, q = q0 + col;
    if (p >= g.P) continue;
    f32x4 s0 = {0.0f, 0.0f, 0.0f, 0.0f}, s1 = s0;
#pragma unroll 4
    for (int u = 0; u < W; ++u) {
      const float* f = sums + (u * RT * 16 + row) * PITCH + col;
      s0 += *(const f32x4*)f;
      s1 += *(const f32x4*)(f + 4);
    }
    float v[8] = {s0[0], s0[1], s0[2], s0[3], s1[0], s1[1], s1[2], s1[3]};
    const int n = q + 8 <= g.Q ? 8 : q < g.Q ? (int)(g.Q - q) : 0;
    finish8<TYPE, false>(g, v, p, q, n, bias_at(g, q, n), residual_at(g, p, q, n));
  }
}

template <int TYPE, int RT>
void launch_few_rows(const DenseGemm& g, hipStream_t st) {
  // 32 columns a block where a checkpoint's blocks need them, and where 16 would give some CUs two blocks and others
  // one (1 x 2048 x 5632 7.1 us against 9.0; 1 x 4096 x 14336 29.8 against 24.4)
  const int64_t blocks = (g.Q + 15) / 16, cus = device_cus();
  const int ct = g.z_scales || (blocks > cus && blocks <= 2 * cus) ? 2 : 1;
  const dim3 grid((unsigned)((g.Q + 16 * ct - 1) / (16 * ct)), (unsigned)((g.P + 16 * RT - 1) / (16 * RT)));
  const auto go = [&]<bool ODD>() {
    if (ct == 2) dense_few_kernel<TYPE, RT, 2, ODD><<<grid, 64 * kFewWaves, 0, st>>>(g);
    else dense_few_kernel<TYPE, RT, 1, ODD><<<grid, 64 * kFewWaves, 0, st>>>(g);
  };
  if (g.R & 1) go.template operator()<true>();
  else go.template operator()<false>();
}

template <int TYPE>
void launch_few(const DenseGemm& g, hipStream_t st) {
  if (g.P <= 16) launch_few_rows<TYPE, 1>(g, st);
  else if (g.P <= 32) launch_few_rows<TYPE, 2>(g, st);
  else launch_few_rows<TYPE, 4>(g, st);
}

// -------------------------------------------------------------------- choice ----

enum : int { kFewRows = 0, kTiles64 = 1, kTiles128 = 2, kTiles256 = 3, kTiles192 = 4 };
constexpr int kRows[] = {0, 64, 128, 256, 256}, kColumns[] = {0, 64, 128, 256, 192};

using Shape256 = DenseShape<8, 4, 2, 4, 2, 1>;
using Shape192 = DenseShape<4, 6, 4, 2, 2, 1>;
using Shape128 = DenseShape<4, 4, 2, 2, 2, 2>;
using Shape64 = DenseShape<2, 2, 2, 2, 4, 2>;

int64_t tiles_of(const DenseGemm& g, int kind) {
  return (g.P + kRows[kind] - 1) / kRows[kind] * ((g.Q + kColumns[kind] - 1) / kColumns[kind]);
}
int64_t blocks_of(const DenseGemm& g) { return (tiles_of(g, g.kind) + 7) / 8 * 8; }     // (eight XCDs)

template <int TYPE>
void launch_forward(const DenseGemm& g, hipStream_t st) {
  const dim3 grid((unsigned)blocks_of(g), (unsigned)g.splits);
  if (g.kind == kTiles256) dense_kernel<TYPE, Shape256><<<grid, 64 * Shape256::W, 0, st>>>(g);
  else if (g.kind == kTiles192) dense_kernel<TYPE, Shape192><<<grid, 64 * Shape192::W, 0, st>>>(g);
  else if (g.kind == kTiles128) dense_kernel<TYPE, Shape128><<<grid, 64 * Shape128::W, 0, st>>>(g);
  else dense_kernel<TYPE, Shape64><<<grid, 256, 0, st>>>(g);
}

template <int TYPE>
void launch_pair(const DensePair& d, int kind, unsigned blocks, hipStream_t st) {
  if (kind == kTiles256) dense_pair_kernel<TYPE, Shape256><<<blocks, 64 * Shape256::W, 0, st>>>(d);
  else if (kind == kTiles128) dense_pair_kernel<TYPE, Shape128><<<blocks, 64 * Shape128::W, 0, st>>>(d);
  else dense_pair_kernel<TYPE, Shape64><<<blocks, 256, 0, st>>>(d);
}

void launch_join(const DenseGemm& g, hipStream_t st) {
  const uint32_t per_row = (uint32_t)((g.Q + 31) / 32 * 4);
  const unsigned blocks = (unsigned)((g.P * per_row + 255) / 256);
  if (g.type == kTypeF16) dense_join_kernel<kTypeF16><<<blocks, 256, 0, st>>>(g, per_row);
  else dense_join_kernel<kTypeBf16><<<blocks, 256, 0, st>>>(g, per_row);
}

// One launch holds fewer than 2^32 threads (of more the rest is left out, with no error).  Splits (four blocks a CU at most)
// and the sums of the bias's gradient (2^14 blocks at most) are counted as 2^15 blocks.  So products from about 2^39 outputs on,
// more than the card's memory holds, are refused.
bool launch_holds(const DenseGemm* x, const DenseGemm* w, int kind) {
  const int64_t blocks = tiles_of(*x, kind) + (w ? tiles_of(*w, kind) : 0) + (int64_t(1) << 15);
  return blocks * (kind >= kTiles256 ? 512 : 256) < (int64_t(1) << 32);
}

void split_into(DenseGemm& g, int64_t splits) {
  const int64_t stages = (g.R + 63) / 64, len = (stages + splits - 1) / splits;
  g.splits = (int)((stages + len - 1) / len);
  g.split_len = len * 64;
  g.part_ld = ceil8(g.Q);
}

}  // namespace

// The few-row kernel: up to 16 rows, and of small products up to 32, or 128 where a row's length is no multiple of 8,
// which the tiles would have copied first.  Rows x K x N, few rows / tiles, us: 8 x 2048 x 5632 7.3 / 10.2,
// 16 x 4096 x 4096 9.6 / 10.5, 24 x 2048 x 2048 7.0 / 8.8, 32 x 4096 x 4096 13.2 / 11.3, 37 x 1003 x 2049 8.7 / 18,
// 128 x 517 x 1001 7.7 / 10.2, 128 x 1003 x 2049 22 / 14.  The rule
// is made for these and does badly by large weights: with 14336 outputs 16 rows of 4096 take 35 (17 rows, by tiles, 26), and where K is
// no multiple of 8 the copy of W makes a step from 16 to 17 rows: K = 4095 58 to 75, K = 8190 69 to 165 (K = 8192 69 to 48).
constexpr int64_t kFewRowsMost = 16, kFewRowsSmall = 32, kFewRowsOdd = 128, kFewSmall = int64_t(1) << 27;
bool takes_few_rows(const DenseGemm& g) {
  return g.P <= kFewRowsMost || (g.P <= (g.R % 8 ? kFewRowsOdd : kFewRowsSmall) && g.P * g.Q * g.R <= kFewSmall);
}

// The tile shape, one for both of a pair, and the splits of the inner indexes, by the time in us at which the CUs are done.
// Measured: a CU takes 0.2 us per stage of a 64 x 64 tile, 0.46 of a 128 x 128 one (alone on its CU
// 0.47, 0.72 where all CUs are busy) and 1.1 of a 256 x 256 one, 1.45 where all CUs are busy and the card's power limits
// them; a split writes and reads its float32 sums at 5.5 TB/s and takes another launch.  A product alone goes
// in rounds of tiles, where tiles of 256 x 192 may fill a last round better; of a pair the longer tiles begin and the
// shorter ones fill the gaps.  Tiles of 256 / 256 x 192 / 128 / 64, us (rows x K x N):
//   forward  2048 x 4096 x 14336 203 / 240 / 238 / 359    2048 x 2048 x 5632 52 / 48 / 61 / 76
//            512 x 2048 x 5632 33 / 40 / 28 / 23          128 x 2048 x 5632 22 / 21 / 18 / 9.5
//   both gradients (256 / 128 / 64)  2048 x 4096 x 14336 429 / 492 / 900   2048 x 2048 x 5632 120 / 105 / 158
//            128 x 2048 x 5632 30 / 23 / 30               1000 x 1000 x 1000 30 / 15 / 13
// (Tiles of 256 x 224, which 14336 columns fill in two rounds of 256 CUs, gained 1 %: idle CUs leave the others
// their power.)
bool plan_tiles(DenseGemm* x, DenseGemm* w, bool gradients) {
  const int cus = device_cus();
  static constexpr int kSplits[] = {1, 2, 3, 4, 6, 8, 12, 16};
  DenseGemm* const g[2] = {x ? x : w, x && w ? w : nullptr};
  double best = 1e300;
  int kind = kTiles64;
  int64_t splits[2] = {1, 1};
  for (int k = kTiles64; k <= (gradients ? kTiles256 : kTiles192); ++k) {
    if (!launch_holds(g[0], g[1], k)) continue;
    const auto block_us = [&](int64_t stages, double load, bool alone) {
      return k >= kTiles256 ? 2.2 + stages * (1.1 + 0.35 * load) * (kColumns[k] + 8) / 264
             : k == kTiles128 ? 0.7 + stages * (alone ? 0.47 + 0.25 * load : 0.46) : 0.3 + stages * (alone ? 0.23 : 0.2);
    };
    struct Cost {
      int64_t blocks, len;
      double join;
    } c[2][8];
    int n[2] = {0, 0};
    for (int i = 0; i < 2 && g[i]; ++i) {
      const int64_t stages = (g[i]->R + 63) / 64, tiles = tiles_of(*g[i], k);
      for (int s : kSplits) {
        if (s > 1 && (s > stages || tiles * s > 4 * cus)) break;
        c[i][n[i]++] = {tiles * s, (stages + s - 1) / s, s > 1 ? 4.0 + (8.0 * s + 2.0) * g[i]->P * g[i]->Q / 5.5e6 : 0.0};
      }
    }
    for (int i = 0; i < n[0]; ++i) {
      for (int j = 0; j < (g[1] ? n[1] : 1); ++j) {
        const int64_t blocks = c[0][i].blocks + (g[1] ? c[1][j].blocks : 0);
        const double load = blocks < cus ? (double)blocks / cus : 1.0;
        double us;
        if (!g[1]) {
          const int64_t rounds = (blocks + cus - 1) / cus;
          us = rounds * block_us(c[0][i].len, load, rounds == 1) + c[0][i].join;
        } else {
          const double a = block_us(c[0][i].len, load, false), b = block_us(c[1][j].len, load, false);
          const double longest = block_us(std::max(c[0][i].len, c[1][j].len), load, true);
          us = (c[0][i].blocks * a + c[1][j].blocks * b) / cus + 0.5 * std::min(a, b);
          us = std::max(us, longest) + c[0][i].join + c[1][j].join;
        }
        if (us < best) {
          best = us, kind = k;
          splits[0] = c[0][i].blocks / tiles_of(*g[0], k);
          splits[1] = g[1] ? c[1][j].blocks / tiles_of(*g[1], k) : 1;
        }
      }
    }
  }
  for (int i = 0; i < 2 && g[i]; ++i) {
    g[i]->kind = kind;
    split_into(*g[i], splits[i]);
  }
  return best < 1e300;
}

bool plan_dense_gemm(DenseGemm& g) {
  if (!takes_few_rows(g)) return plan_tiles(&g, nullptr, false);
  g.kind = kFewRows;
  split_into(g, 1);
  return true;
}

bool plan_dense_pair(DensePair& d, bool with_x, bool with_w) {
  if ((with_x || with_w) && !plan_tiles(with_x ? &d.x : nullptr, with_w ? &d.w : nullptr, true)) return false;
  d.x_blocks = with_x ? (int)(blocks_of(d.x) * d.x.splits) : 0;
  d.w_blocks = with_w ? (int)(blocks_of(d.w) * d.w.splits) : 0;
  d.w_first = with_w && d.w.split_len > d.x.split_len;
  return true;
}

int64_t dense_parts_bytes(const DenseGemm& g) { return g.splits > 1 ? g.splits * g.P * g.part_ld * 4 : 0; }

hipError_t launch_dense_gemm(const DenseGemm& g, hipStream_t st) {
  if (g.kind == kFewRows) {
    if (g.type == kTypeF16) launch_few<kTypeF16>(g, st);
    else launch_few<kTypeBf16>(g, st);
    return hipGetLastError();
  }
  if (g.type == kTypeF16) launch_forward<kTypeF16>(g, st);
  else launch_forward<kTypeBf16>(g, st);
  if (g.splits > 1) launch_join(g, st);
  return hipGetLastError();
}

hipError_t launch_dense_pair(const DensePair& d, int type, hipStream_t st) {
  const int kind = d.x_blocks ? d.x.kind : d.w_blocks ? d.w.kind : kTiles64;
  const unsigned blocks = (unsigned)(d.x_blocks + d.w_blocks + (d.n_sums ? (d.N + 63) / 64 : 0));
  if (type == kTypeF16) launch_pair<kTypeF16>(d, kind, blocks, st);
  else launch_pair<kTypeBf16>(d, kind, blocks, st);
  if (d.x_blocks && d.x.splits > 1) launch_join(d.x, st);
  if (d.w_blocks && d.w.splits > 1) launch_join(d.w, st);
  return hipGetLastError();
}

}  // namespace swq
