// The dense product with its epilogue, and the pass that a backward of it
// starts with (the slope of the activation, and the bias gradient).
//
//   y = act(x W^T + b) + residual
//   dz = dy * act'(z);  dx = dz W;  dW = dz^T x;  db = column sums of dz
#include <algorithm>

#include "topk_ops_device.hpp"

namespace tk {

namespace {

// ---------------------------------------------------------------- epilogue
struct Epi {
  const void* bias;
  const void* residual;
  void* c;
  void* pre;
  int64_t ldr, ldc, ldp;
  uint32_t m, n;
  int act;
  int stream;    // store y past the caches
};

// The activation of V values; the switch is the same for every lane.
template <class T, int V>
__device__ __forceinline__ void act_any(float* v, int act) {
  if (act == ACT_RELU) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = act_of<ACT_RELU, T>(v[i]);
  } else if (act == ACT_GELU) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = act_of<ACT_GELU, T>(v[i]);
  } else if (act == ACT_SILU) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = act_of<ACT_SILU, T>(v[i]);
  }
}

// V sums of row r from column c on, in order: bias (given), pre-activation,
// activation, residual, one rounding, one store.  V is the 16-byte width or 1.
template <class T, int V>
__device__ __forceinline__ void finish(float* v, const float* bias, uint32_t r, uint32_t c, const Epi& e) {
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] += bias[i];
  if (e.pre) store_vec<T, V>(static_cast<T*>(e.pre) + (int64_t)r * e.ldp + c, v);
  act_any<T, V>(v, e.act);
  if (e.residual) {
    float q[V];
    load_vec<T, V>(static_cast<const T*>(e.residual) + (int64_t)r * e.ldr + c, q);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] += q[i];
  }
  T* y = static_cast<T*>(e.c) + (int64_t)r * e.ldc + c;
  if (V > 1 && e.stream) {
    // (the empty statements keep the compiler from merging the two stores into a plain one)
    asm volatile("");
    stream_vec<T>(y, v);
    asm volatile("");
  } else {
    store_vec<T, V>(y, v);
  }
}

// The same for a row's last columns, `have` < V of them, element by element:
// all loads first, so that they wait together.
template <class T, int V>
__device__ __forceinline__ void finish_some(float* v, const float* bias, uint32_t r, uint32_t c, uint32_t have,
                                            const Epi& e) {
  float q[V];
  if (e.residual) {
    const T* p = static_cast<const T*>(e.residual) + (int64_t)r * e.ldr + c;
#pragma unroll
    for (int i = 0; i < V; ++i) q[i] = (uint32_t)i < have ? to_f32(p[i]) : 0.f;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] += bias[i];
  if (e.pre) {
    T* p = static_cast<T*>(e.pre) + (int64_t)r * e.ldp + c;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if ((uint32_t)i < have) p[i] = from_f32<T>(v[i]);
  }
  act_any<T, V>(v, e.act);
  if (e.residual) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] += q[i];
  }
  T* y = static_cast<T*>(e.c) + (int64_t)r * e.ldc + c;
#pragma unroll
  for (int i = 0; i < V; ++i)
    if ((uint32_t)i < have) y[i] = from_f32<T>(v[i]);
}

// The bias of V columns, 0 where there is none.
template <class T, int V>
__device__ __forceinline__ void bias_of(float* b, uint32_t c, const Epi& e) {
#pragma unroll
  for (int i = 0; i < V; ++i) b[i] = 0.f;
  if (e.bias) load_vec<T, V>(static_cast<const T*>(e.bias) + c, b);
}
template <class T, int V>
__device__ __forceinline__ void bias_some(float* b, uint32_t c, uint32_t have, const Epi& e) {
#pragma unroll
  for (int i = 0; i < V; ++i) b[i] = e.bias && (uint32_t)i < have ? to_f32(static_cast<const T*>(e.bias)[c + i]) : 0.f;
}

// ---------------------------------------------------------------- product
// Tiles of 128 bytes along the summed axis (64 bf16 or 32 f32) go from memory
// straight to LDS (buffer loads with an LDS destination, 16 bytes a lane), two
// stages deep; reads beyond a tensor's end return 0 there.  A wave's matrix
// instructions take 16-byte fragments: 8 bf16 of one row (16x16x32), or 4 f32
// used by four 32x32x2 instructions in turn; the summed axis is permuted the
// same way in both operands.
//
// LDS layouts.  An operand whose summed axis is contiguous is kept as rows of
// 128 bytes, the 16-byte chunk c of row r at place c ^ (r & 7), so that the
// eight rows read in one clock use all banks once.  An operand stored the
// other way round ("trans") is kept as it lies in memory, one line per summed
// index; f32 fragments are then read element by element, bf16 ones with the
// transposing LDS read, for which the 16-row units of a line are rotated by
// the summed index so that the lines read together lie in different banks.
//
// W's rows are the first operand of the matrix instruction and x's the second,
// so a lane ends with four neighbouring columns of one output row.
typedef __attribute__((address_space(3))) char lds_char;
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

struct KOperand {
  const void* p;
  int64_t ld;        // elements
  uint32_t rows;     // valid rows
  uint32_t red;      // valid extent of the summed axis
};

struct KGemm {
  KOperand a, b;     // x and W
  Epi e;
  float* part;       // sums of split tiles: [split][rest][TM][TN]
  uint32_t tiles_m, tiles_n;
  uint32_t whole, rest, split;   // the first `whole` tiles run the epilogue, the others are split
  uint32_t pieces;               // whole + rest * split: the workgroups
  uint32_t steps, all_steps;     // steps along the summed axis of a piece, and of a whole tile
};

// FR: rows of a fragment; SUB: fragments along a step.  32-bit fragments are
// 32 rows high: 32x32x2 runs at 140 to 154 TFLOP/s with one to four waves on a
// SIMD, 16x16x4 at 114 to 138.
typedef float f32x16 __attribute__((ext_vector_type(16)));
template <class T> struct Elem;
template <> struct Elem<bf16_t> {
  static constexpr int ES = 2, BK = 64, FR = 16, SUB = 2;
  typedef f32x4 Acc;
};
template <> struct Elem<float> {
  static constexpr int ES = 4, BK = 32, FR = 32, SUB = 4;
  typedef f32x16 Acc;
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* p, int64_t bytes) {
  const int n = bytes > 0x7FFFFFFF ? 0x7FFFFFFF : (bytes < 0 ? 0 : (int)bytes);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, n, 0x00020000);
}

// Loads one operand's tile of R rows: R / 8 instructions of 1 KB, shared by W waves.
template <class T, int R, bool TR, int W>
struct Loader {
  static constexpr int N = R / 8 / W;
  uint32_t off[N];
  uint32_t chunk;    // the lane's place on the summed axis within a step (not TR)
  const char* base;
  int64_t bytes;     // from base to the end of the valid data
  int64_t step;      // bytes from one step to the next
  uint32_t red;

  __device__ void init(const KOperand& o, uint32_t r0, uint32_t wave, uint32_t lane) {
    constexpr int ES = Elem<T>::ES;
    const uint32_t rows = o.rows - r0 < R ? o.rows - r0 : R;
    red = o.red;
    if constexpr (!TR) {
      base = static_cast<const char*>(o.p) + (int64_t)r0 * o.ld * ES;
      bytes = ((int64_t)(rows - 1) * o.ld + o.red) * ES;
      step = 128;
      const uint32_t c = (lane % 8) ^ (lane / 8);
      chunk = c * (16 / ES);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const uint32_t row = (wave * N + j) * 8 + lane / 8;
        off[j] = row * (uint32_t)o.ld * ES + c * 16;
      }
    } else {
      constexpr uint32_t RB = R * ES, US = 32;
      base = static_cast<const char*>(o.p) + (int64_t)r0 * ES;
      // rounded up to whole words: a range check that ends inside a word would drop its first half
      bytes = ((((int64_t)o.red - 1) * o.ld + rows) * ES + 3) & ~(int64_t)3;
      step = (int64_t)Elem<T>::BK * o.ld * ES;
      chunk = 0;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const uint32_t at = (wave * N + j) * 1024 + lane * 16;
        const uint32_t k = at / RB, in = at % RB;
        const uint32_t turn = ES == 2 ? (k & 3) : 0;
        off[j] = k * (uint32_t)o.ld * ES + (((in / US) ^ turn) * US) + in % US;
      }
    }
  }

  __device__ void issue(lds_char* dst, uint32_t kt, uint32_t wave) {
    const int64_t at = (int64_t)kt * step;
    const __amdgpu_buffer_rsrc_t r = rsrc_of(base + at, bytes - at);
    bool in = true;
    if constexpr (!TR) in = kt * Elem<T>::BK + chunk < red;
#pragma unroll
    for (int j = 0; j < N; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          r, reinterpret_cast<__attribute__((address_space(3))) void*>(dst + (wave * N + j) * 1024), 16,
          in ? off[j] : 0x7FFFFFF0u, 0, 0, 0);
  }
};

// Waits for this wave's loads to LDS: a barrier alone does not, and the
// other waves read what they bring.
__device__ __forceinline__ void wait_loads() {
  __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0)
}

// A lane's 16 bytes of fragment f (FR rows), sub-step s of a tile.
template <class T, int R, bool TR>
__device__ __forceinline__ u32x4 fragment(lds_char* t, uint32_t f, uint32_t s, uint32_t lane) {
  constexpr uint32_t FR = Elem<T>::FR, G = 64 / FR;    // G lanes share a row
  const uint32_t i = lane % FR, g = lane / FR;
  if constexpr (!TR) {
    const uint32_t at = (f * FR + i) * 128 + (((s * G + g) ^ (i & 7)) * 16);
    return *reinterpret_cast<__attribute__((address_space(3))) u32x4*>(t + at);
  } else if constexpr (Elem<T>::ES == 2) {
    constexpr uint32_t RB = R * 2;
    const uint32_t k = s * 32 + g * 8 + i / 4;
    lds_char* at = t + k * RB + ((f ^ (i / 4)) * 32) + (i % 4) * 8;
    union {
      s16x4 h[2];
      u32x4 v;
    } q;
    q.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        reinterpret_cast<__attribute__((address_space(3))) s16x4*>(at));
    q.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        reinterpret_cast<__attribute__((address_space(3))) s16x4*>(at + 4 * RB));
    return q.v;
  } else {
    constexpr uint32_t RB = R * 4;
    lds_char* at = t + (s * 8 + g * 4) * RB + (f * 32 + i) * 4;   // 32 lanes use all banks once
    u32x4 v;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = *reinterpret_cast<__attribute__((address_space(3))) uint32_t*>(at + j * RB);
    return v;
  }
}

// acc[i][j] += w[i] x[j].  The four f32 instructions of a fragment pair go
// round all pairs in turn: one that waited for its own last result would
// leave the matrix core idle.
template <class T, int FM, int FN, class Acc>
__device__ __forceinline__ void mma_all(const u32x4* w, const u32x4* x, Acc (&acc)[FN][FM]) {
  if constexpr (Elem<T>::ES == 2) {
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int j = 0; j < FM; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            __builtin_bit_cast(bf16x8, w[i]), __builtin_bit_cast(bf16x8, x[j]), acc[i][j], 0, 0, 0);
  } else {
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j) {
          const float a = __uint_as_float(w[i][u]), b = __uint_as_float(x[j][u]);
          if constexpr (sizeof(Acc) == 64) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(a, b, acc[i][j], 0, 0, 0);
          else acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, acc[i][j], 0, 0, 0);
        }
  }
}

// Consecutive workgroups go to the eight dies in turn, so each die gets a
// contiguous range of a launch's tiles.
__device__ __forceinline__ uint32_t die_order(uint32_t id, uint32_t total) {
  const uint32_t q = total / 8, r = total % 8, x = id % 8;
  return x * q + (x < r ? x : r) + id / 8;
}

// A range of tiles walks the product in bands of 1024 rows: W's tile and the
// band's rows of x then stay in the die's L2 (4096 x 512 x 65536 bf16 in
// 256-tiles, in the form that they had when this was chosen: 360 us in bands of
// 4 tiles, 380 to 451 in bands of 1, 8, 16 or 32).  Each band begins 37 tiles further right: dies that work on different
// bands would else store the same columns at the same time, and where the row
// stride is a power of two those lie in the same memory channels (338 us with
// the shift, 322 for rows of 65600, both then; the present form 313 and 322).
__device__ __forceinline__ void place_of(uint32_t id, uint32_t tm, uint32_t tn, uint32_t tile, uint32_t* im,
                                         uint32_t* in) {
  const uint32_t band_rows = 1024 / tile;
  const uint32_t band = id / (band_rows * tn);
  const uint32_t rows = tm - band * band_rows < band_rows ? tm - band * band_rows : band_rows;
  const uint32_t at = id - band * band_rows * tn;
  *im = band * band_rows + at % rows;
  *in = (at / rows + band * 37) % tn;
}

// One step: the tiles of step kt are in `cur`; the loads of step kt + 1 go to
// `next` while this step's fragments are read and multiplied.  The two stages
// are separate LDS variables, so that the compiler knows that the loads in
// flight do not write what the fragment reads read.
template <class T, int TM, int TN, int FM, int FN, bool TA, bool TB, class LA, class LB, class Acc>
__device__ __forceinline__ void gemm_step(lds_char* cur, lds_char* next, LA& la, LB& lb, uint32_t kt,
                                          bool more, uint32_t wave, uint32_t lane, uint32_t wm,
                                          uint32_t wn, Acc (&acc)[FN][FM]) {
  constexpr int SUB = Elem<T>::SUB;
  wait_loads();
  __syncthreads();   // this step's tiles have arrived; the other stage is free
  auto ahead = [&]() {
    if (more) {
      la.issue(next, kt + 1, wave);
      lb.issue(next + TM * 128, kt + 1, wave);
    }
    // the loads leave now: the scheduler would let them sink to the end of the step
    __builtin_amdgcn_sched_barrier(0);
  };
  if constexpr (FM * FN <= 16) {
    // all fragments first: the later ones' reads are covered by the first ones' products
    u32x4 fa[SUB][FM], fb[SUB][FN];
#pragma unroll
    for (int s = 0; s < SUB; ++s) {
#pragma unroll
      for (int i = 0; i < FN; ++i) fb[s][i] = fragment<T, TN, TB>(cur + TM * 128, wn + i, s, lane);
#pragma unroll
      for (int j = 0; j < FM; ++j) fa[s][j] = fragment<T, TM, TA>(cur, wm + j, s, lane);
    }
    ahead();
#pragma unroll
    for (int s = 0; s < SUB; ++s) mma_all<T, FM, FN>(fb[s], fa[s], acc);
  } else {   // the registers hold one sub-step's
    ahead();
#pragma unroll
    for (int s = 0; s < SUB; ++s) {
      u32x4 fa[FM], fb[FN];
#pragma unroll
      for (int i = 0; i < FN; ++i) fb[i] = fragment<T, TN, TB>(cur + TM * 128, wn + i, s, lane);
#pragma unroll
      for (int j = 0; j < FM; ++j) fa[j] = fragment<T, TM, TA>(cur, wm + j, s, lane);
      mma_all<T, FM, FN>(fb, fa, acc);
    }
  }
}

// Workgroup `id` of a product: a tile, or a piece of one.
template <class T, int TM, int TN, int NWM, int NWN, bool TA, bool TB>
__device__ __forceinline__ void gemm_tile(const KGemm& p, uint32_t id, lds_char* s0, lds_char* s1, char* stage0) {
  constexpr int FR = Elem<T>::FR, W = NWM * NWN, FM = TM / FR / NWM, FN = TN / FR / NWN;
  typedef typename Elem<T>::Acc Acc;
  const uint32_t lane = threadIdx.x % 64;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  uint32_t tile, piece = 0, k0 = 0, k1 = p.all_steps;
  const bool split = id >= p.whole;
  if (!split) {
    tile = die_order(id, p.whole);
  } else {
    const uint32_t sp = (id - p.whole) / p.rest, at = die_order(id - p.whole - sp * p.rest, p.rest);
    tile = p.whole + at;
    piece = sp * p.rest + at;
    k0 = sp * p.steps;
    if (k1 - k0 > p.steps) k1 = k0 + p.steps;
  }
  uint32_t im, in;
  place_of(tile, p.tiles_m, p.tiles_n, TM, &im, &in);
  const uint32_t m0 = im * TM, n0 = in * TN;
  Loader<T, TM, TA, W> la;
  Loader<T, TN, TB, W> lb;
  la.init(p.a, m0, wave, lane);
  lb.init(p.b, n0, wave, lane);
  const uint32_t wm = (wave / NWN) * FM, wn = (wave % NWN) * FN;   // the wave's first fragments
  Acc acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j)
#pragma unroll
      for (int u = 0; u < FR * FR / 64; ++u) acc[i][j][u] = 0.f;
  if (k0 < k1) {
    la.issue(s0, k0, wave);
    lb.issue(s0 + TM * 128, k0, wave);
  }
  uint32_t kt = k0;
  for (; kt + 1 < k1; kt += 2) {
    gemm_step<T, TM, TN, FM, FN, TA, TB>(s0, s1, la, lb, kt, true, wave, lane, wm, wn, acc);
    gemm_step<T, TM, TN, FM, FN, TA, TB>(s1, s0, la, lb, kt + 1, kt + 2 < k1, wave, lane, wm, wn, acc);
  }
  if (kt < k1) gemm_step<T, TM, TN, FM, FN, TA, TB>(s0, s1, la, lb, kt, false, wave, lane, wm, wn, acc);
  __syncthreads();
  // 32 output rows at a time through a part of LDS that is the wave's own: in
  // as four columns a lane, out as 16-byte pieces of rows.  The four-column
  // chunk u of row r lies at place u ^ (r mod chunks).  A lane keeps its
  // columns, and so their bias, for all rows.
  constexpr uint32_t C = TN / NWN, CH = C / 4;
  constexpr int V = Vec<T>::N;
  constexpr uint32_t LANES = C / V, ROWS = 64 / LANES;
  static_assert(W * 32 * C * 4 <= (TM + TN) * 128, "the rows fit one stage");
  float* mine = reinterpret_cast<float*>(stage0) + wave * 32 * C;
  uint32_t cc = (lane % LANES) * V, c = n0 + wn * FR + cc;
  // A row's last vector begins earlier, so that it ends with the row, and two
  // lanes store the same values to the columns between (3067 x 4686 bf16 15.6
  // us; 30.7 with those columns one by one, which the last tiles' waves did
  // after all others).  Not where y is its own residual: the one could read
  // what the other has stored.
  const bool slid = !split && c < p.e.n && c + V > p.e.n && p.e.n >= n0 + wn * FR + V && p.e.residual != p.e.c;
  if (slid) {
    cc -= c + V - p.e.n;
    c = p.e.n - V;
  }
  const bool whole = c + V <= p.e.n;   // the lane's columns are one vector of every row
  float bias[V] = {};
  const uint32_t have = c < p.e.n ? p.e.n - c : 0u;
  if (whole && !split) bias_of<T, V>(bias, c, p.e);
  else if (TM < 256 && !split) bias_some<T, V>(bias, c, have, p.e);
  constexpr int HIGH = 32 / FR;        // fragments that 32 rows take
#pragma unroll
  for (int j = 0; j < FM; j += HIGH) {
#pragma unroll
    for (int h = 0; h < HIGH; ++h)
#pragma unroll
      for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int q = 0; q < FR * FR / 256; ++q) {   // four columns each, 8 apart in a fragment of 32
          const uint32_t r = h * FR + lane % FR, u = i * (FR / 4) + q * 2 + lane / FR;
          const Acc& v = acc[i][j + h];
          *reinterpret_cast<f32x4*>(mine + r * C + (u ^ (r % CH)) * 4) =
              f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
        }
    const uint32_t r0 = m0 + (wm + j) * FR;
#pragma unroll 2
    for (uint32_t rr = lane / LANES; rr < 32; rr += ROWS) {
      if (r0 + rr >= p.e.m) break;
      float v[V];
      if (slid) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = mine[rr * C + (((cc + i) / 4) ^ (rr % CH)) * 4 + (cc + i) % 4];
      } else {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
          const f32x4 q = *reinterpret_cast<const f32x4*>(mine + rr * C + ((cc / 4 + i / 4) ^ (rr % CH)) * 4);
#pragma unroll
          for (int u = 0; u < 4; ++u) v[i + u] = q[u];
        }
      }
      if (split) {
        float* o = p.part + ((size_t)piece * TM + (wm + j) * FR + rr) * TN + wn * FR + cc;
#pragma unroll
        for (int i = 0; i < V; i += 4) Vec<float>::store(o + i, v + i);
      } else if (whole) {
        finish<T, V>(v, bias, r0 + rr, c, p.e);
      } else if constexpr (TM < 256) {   // the last columns
        if (have) finish_some<T, V>(v, bias, r0 + rr, c, have, p.e);
      } else {   // (one by one: the registers are full)
#pragma unroll 1
        for (uint32_t i = 0; i < have; ++i) {
          float z = mine[rr * C + ((cc / 4 + i / 4) ^ (rr % CH)) * 4 + i % 4], b1;
          bias_of<T, 1>(&b1, c + i, p.e);
          finish<T, 1>(&z, &b1, r0 + rr, c + i, p.e);
        }
      }
    }
  }
}

// Measured beside the vendor library's plain product of the same operands
// (normal random numbers, both on one card; the rates follow the clock, which
// follows the data and differs by a tenth from card to card): bf16 8192^3 796 us
// against 708, 4096^3 101 against 97; 4096 x 512 x 65536, which the store of 537
// MB bounds as much as the products, 313 against 308 (with bias and relu and an
// autoencoder's weights 324; 320 to 334 on two other cards, the library's plain
// product 342 on one of them); f32 4096^3 1026 against 922.
template <class T, int TM, int TN, int NWM, int NWN, bool TA, bool TB>
__global__ __launch_bounds__(NWM * NWN * 64, 2) void k_gemm(KGemm p) {
#ifdef __HIP_DEVICE_COMPILE__   // buffer resources exist in the device pass only
  __shared__ __align__(1024) char stage0[(TM + TN) * 128];
  __shared__ __align__(1024) char stage1[(TM + TN) * 128];
  const uint32_t id = block_id();
  if (id >= p.pieces) return;
  gemm_tile<T, TM, TN, NWM, NWN, TA, TB>(p, id, (lds_char*)stage0, (lds_char*)stage1, stage0);
#endif
}

// Both products of a gradient, dx = dz W and dW = dz^T x, side by side: the
// workgroups of one fill the compute units that the other's last ones leave
// (the whole call, 4096 x 512 x 12288 bf16 208 us in two launches, 201 in one;
// 2048 x 1024 x 4096 f32 311, 292).  The one with the longer pieces goes first
// (`b_first`).
template <class T, int TM, int TN, int NWM, int NWN>
__global__ __launch_bounds__(NWM * NWN * 64, 2) void k_gemm_pair(KGemm a, KGemm b, int b_first) {
#ifdef __HIP_DEVICE_COMPILE__
  __shared__ __align__(1024) char stage0[(TM + TN) * 128];
  __shared__ __align__(1024) char stage1[(TM + TN) * 128];
  const uint32_t id = block_id(), first = b_first ? b.pieces : a.pieces;
  if (id >= a.pieces + b.pieces) return;
  if ((id < first) == (b_first != 0))
    gemm_tile<T, TM, TN, NWM, NWN, true, true>(b, id < first ? id : id - first, (lds_char*)stage0, (lds_char*)stage1, stage0);
  else
    gemm_tile<T, TM, TN, NWM, NWN, false, true>(a, id < first ? id : id - first, (lds_char*)stage0, (lds_char*)stage1, stage0);
#endif
}

// Adds partial sums in a fixed order, then the epilogue: the split tiles of up
// to two products, and the column sums' blocks (a product of one row), in one
// launch.  A thread takes 16 bytes of y; where there are many parts several
// threads share them, and add theirs in LDS: 64 parts read one after another
// would take longer than the tiles (33 x 12288 x 512 bf16: 33 us against 15).
// Four parts of 4096 x 512 bf16 and 64 of 12288 column sums: 9.8 us, 3.8 TB/s.
struct KJoin {
  const float* part;     // [split][m][ldpart], or, for split tiles, [split][rest][tile][tile]
  uint32_t split, ldpart;
  uint32_t whole, rest, tile, tiles_m, tiles_n;   // rest 0: rows
  uint32_t ways, blocks;
  Epi e;
};
struct KJoins {
  KJoin j[3];
};

template <class T>
__global__ __launch_bounds__(256) void k_join(KJoins js) {
  constexpr int V = Vec<T>::N;
  __shared__ __align__(16) float sums[256 * V];
  uint32_t b = blockIdx.x, which = 0;
  while (b >= js.j[which].blocks) b -= js.j[which++].blocks;
  const KJoin& p = js.j[which];
  const uint32_t each = 256 / p.ways, group = threadIdx.x / each;
  const uint64_t i = (uint64_t)b * each + threadIdx.x % each;
  uint32_t r, c, limit = ~0u;
  const float* q;
  size_t next;
  bool in;
  if (p.rest) {
    const uint32_t per_row = p.tile / V, t = (uint32_t)(i / (p.tile * per_row)), at = (uint32_t)(i % (p.tile * per_row));
    uint32_t im = 0, jn = 0;
    if (t < p.rest) place_of(p.whole + t, p.tiles_m, p.tiles_n, p.tile, &im, &jn);
    r = im * p.tile + at / per_row;
    c = jn * p.tile + at % per_row * V;
    in = t < p.rest && r < p.e.m && c < p.e.n;
    q = p.part + i * V;
    next = (size_t)p.rest * p.tile * p.tile;
  } else {
    const uint32_t per_row = (p.e.n + V - 1) / V;
    r = (uint32_t)(i / per_row);
    c = (uint32_t)(i % per_row) * V;
    in = i < (uint64_t)per_row * p.e.m;
    q = p.part + (size_t)r * p.ldpart + c;
    next = (size_t)p.e.m * p.ldpart;
    limit = p.ldpart;      // a multiple of 4
  }
  float v[V] = {};
  if (in) {
    q += group * next;
#pragma unroll 8
    for (uint32_t s = group; s < p.split; s += p.ways) {
#pragma unroll
      for (int j = 0; j < V; j += 4) {
        if (c + j >= limit) continue;
        const f32x4 t = *reinterpret_cast<const f32x4*>(q + j);
#pragma unroll
        for (int u = 0; u < 4; ++u) v[j + u] += t[u];
      }
      q += p.ways * next;
    }
  }
  if (p.ways > 1) {
#pragma unroll
    for (int j = 0; j < V; ++j) sums[threadIdx.x * V + j] = v[j];
    __syncthreads();
    if (group) return;
    for (uint32_t g = 1; g < p.ways; ++g) {
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] += sums[(g * each + threadIdx.x) * V + j];
    }
  }
  if (!in) return;
  if (c + V <= p.e.n) {
    float bias[V];
    bias_of<T, V>(bias, c, p.e);
    finish<T, V>(v, bias, r, c, p.e);
  } else {
    float bias[V];
    bias_some<T, V>(bias, c, p.e.n - c, p.e);
    finish_some<T, V>(v, bias, r, c, p.e.n - c, p.e);
  }
}

template <class T>
hipError_t run_joins(const KJoin* js, int n, hipStream_t s) {
  KJoins k{};
  uint32_t blocks = 0;
  for (int i = 0; i < n; ++i) {
    KJoin& j = k.j[i];
    j = js[i];
    j.ways = j.split <= 8 ? 1 : j.split <= 32 ? 4 : 16;   // a thread's loads fit one round trip
    const int64_t vecs = j.rest ? (int64_t)j.rest * j.tile * j.tile / Vec<T>::N
                                : ceil_div(j.e.n, Vec<T>::N) * (int64_t)j.e.m;
    j.blocks = (uint32_t)ceil_div(vecs, 256 / j.ways);
    blocks += j.blocks;
  }
  if (!blocks) return hipSuccess;
  hipLaunchKernelGGL((k_join<T>), dim3(blocks), dim3(256), 0, s, k);
  return hipGetLastError();
}

// Copies lines of `red` elements to lines of `ldo`, zeros behind their end;
// both operands of a product in one launch (`vecs` 0: not this one).  Rows of
// 515 f32 of 1001 x 515 and 4099 x 515: 6.7 us, 3.1 TB/s.
struct KPack {
  const void* src;
  void* dst;
  int64_t ld;
  uint32_t red, ldo;
  uint64_t vecs;       // 16-byte vectors written
};

template <class T>
__device__ __forceinline__ void pack_vec(const KPack& a, const KPack& b, uint64_t i) {
  constexpr int V = Vec<T>::N;
  const bool second = i >= a.vecs;
  if (second) i -= a.vecs;
  const KPack p = second ? b : a;
  if (i >= p.vecs) return;
  const uint32_t per = p.ldo / V;
  const uint64_t r = i / per;
  const uint32_t c = (uint32_t)(i - r * per) * V;
  const T* src = static_cast<const T*>(p.src) + (int64_t)r * p.ld + c;
  u32x4 q;
  if (c + V <= p.red) {
    q = read16(src);
  } else {
    T v[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      v[j] = T{};
      if (c + j < p.red) v[j] = src[j];
    }
    q = __builtin_bit_cast(u32x4, v);
  }
  *reinterpret_cast<u32x4*>(static_cast<T*>(p.dst) + r * p.ldo + c) = q;
}

template <class T>
__global__ __launch_bounds__(256) void k_pack(KPack a, KPack b) {
  pack_vec<T>(a, b, (uint64_t)block_id() * 256 + threadIdx.x);
}

// Few rows of x: the call is bound by reading W once.  A workgroup takes 16
// rows of W (columns of y), 16 or 32 rows of x and the whole summed axis; its
// W waves take turns of 256 bytes per row of it, straight from memory into the
// matrix instructions' operands, with all loads of a turn issued before the
// first is used, and join their sums in LDS in wave order.  One row through 12288 x 512
// bf16 (12.6 MB): 4.4 us, 2.9 TB/s; its launch takes longer than that.
template <class T>
__device__ __forceinline__ u32x4 row_piece(const T* p, bool in, uint32_t k, uint32_t red) {
  constexpr uint32_t V = Vec<T>::N;
  u32x4 q = {0u, 0u, 0u, 0u};
  if (in && k + V <= red) {
    q = read16(p + k);
  } else if (in && k < red) {
    T v[V];
#pragma unroll
    for (uint32_t i = 0; i < V; ++i) {
      v[i] = T{};
      if (k + i < red) v[i] = p[k + i];
    }
    q = __builtin_bit_cast(u32x4, v);
  }
  return q;
}

// Blocks of rows along the grid's second dimension, which takes 65536 at most;
// the third goes on.  (One dimension and a division: 4.28 us against 4.08.)
constexpr uint32_t FEW_Y = 32768;

template <class T, int MF, int W>
__global__ __launch_bounds__(W * 64) void k_few_rows(KGemm p) {
  constexpr uint32_t V = Vec<T>::N, PIECE = 4 * V, TURN = 4;   // summed elements per instruction, pieces per turn
  __shared__ float join[W][MF][16][17];
  const uint32_t lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const uint32_t i = lane % 16, g = lane / 16;
  const uint32_t n0 = blockIdx.x * 16, m0 = (blockIdx.z * FEW_Y + blockIdx.y) * 16 * MF, red = p.a.red;
  const bool win = n0 + i < p.b.rows;
  const T* w = static_cast<const T*>(p.b.p) + (int64_t)(win ? n0 + i : 0) * p.b.ld;
  const T* x[MF];
  bool xin[MF];
#pragma unroll
  for (int f = 0; f < MF; ++f) {
    const uint32_t row = m0 + f * 16 + i;
    xin[f] = row < p.a.rows;
    x[f] = static_cast<const T*>(p.a.p) + (int64_t)(xin[f] ? row : 0) * p.a.ld;
  }
  f32x4 acc[1][MF];
#pragma unroll
  for (int f = 0; f < MF; ++f) acc[0][f] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (uint32_t k0 = wave * TURN * PIECE; k0 < red; k0 += W * TURN * PIECE) {
    u32x4 wf[TURN][1], xf[TURN][MF];
#pragma unroll
    for (uint32_t t = 0; t < TURN; ++t) {
      wf[t][0] = row_piece<T>(w, win, k0 + t * PIECE + g * V, red);
#pragma unroll
      for (int f = 0; f < MF; ++f) xf[t][f] = row_piece<T>(x[f], xin[f], k0 + t * PIECE + g * V, red);
    }
#pragma unroll
    for (uint32_t t = 0; t < TURN; ++t) mma_all<T, MF, 1>(wf[t], xf[t], acc);
  }
#pragma unroll
  for (int f = 0; f < MF; ++f)
#pragma unroll
    for (int j = 0; j < 4; ++j) join[wave][f][i][g * 4 + j] = acc[0][f][j];
  __syncthreads();
  const uint32_t c = n0 + threadIdx.x % 16;
  if (threadIdx.x >= 256 || c >= p.e.n) return;
  float bias;
  bias_of<T, 1>(&bias, c, p.e);
#pragma unroll
  for (int f = 0; f < MF; ++f) {
    const uint32_t r = threadIdx.x / 16, at = threadIdx.x % 16, row = m0 + f * 16 + r;
    if (row >= p.e.m) continue;
    float z = 0.f;
#pragma unroll
    for (int q = 0; q < W; ++q) z += join[q][f][r][at];
    finish<T, 1>(&z, &bias, row, c, p.e);
  }
}

// How a product runs.
struct Plan2 {
  bool few = false;                  // k_few_rows
  uint32_t tile = 128;
  uint32_t tiles_m = 0, tiles_n = 0, whole = 0, rest = 0, split = 1, steps = 0, all_steps = 0;
  bool pack_a = false, pack_b = false;
  uint32_t lda = 0, ldb = 0;         // packed strides
  size_t off_b = 0, off_part = 0, total = 0;
};

// Direct loads need 16-byte aligned lines, lines whose summed extent fills
// 16-byte chunks (rows beyond it would be summed otherwise), and strides
// that keep the offsets within a tile in range.
bool needs_pack(const Operand& o, int64_t rows, int64_t red, int64_t es) {
  if (!rows || !red) return false;
  const int64_t line = o.trans ? rows : red, lines = o.trans ? red : rows;
  const int64_t ld = lines > 1 ? o.ld : line;
  return reinterpret_cast<uintptr_t>(o.p) % 16 || (lines > 1 && (ld * es) % 16) ||
         (!o.trans && !o.padded && (red * es) % 16) || ld >= WIDTH_MAX;
}

// Microseconds of one step of a tile on a compute unit that shares its time
// among the tiles it holds, and with one alone; of a tile's start and end;
// and the tiles a compute unit holds at once.  Measured, each tile forced, in the
// form that the tiles had then: bf16 8192^3 in 64-, 128- and 256-tiles 1768, 991
// and 811 us, 4096 x 512 x 65536 626, 375 and 358; f32 4096^3 in 64- and
// 128-tiles 1027 and 996 us.
struct TileCost {
  uint32_t tile, holds;
  double shared, alone, ends;
};
constexpr TileCost COST_BF16[] = {{64, 4, 0.2, 0.7, 4}, {128, 2, 0.49, 0.8, 6}, {256, 1, 1.55, 1.55, 12}};
constexpr TileCost COST_F32[] = {{64, 4, 0.45, 0.95, 4}, {128, 2, 1.75, 2.0, 6}};

// Ways to split a summed axis that are looked at.
constexpr int64_t SPLITS[] = {1, 2, 3, 4, 5, 6, 7, 8, 10, 12, 14, 16, 20, 24, 28, 32, 40, 48, 56, 64};

// The tile, and the tiles whose summed axis is split, that are estimated
// cheapest (returned, in microseconds): none, all, or those behind the last full round of the compute
// units (1001 x 515 x 4099 f32 in 64-tiles is 1040 of them on 256 units of
// four: whole, the last 16 cost as much again as a quarter of the others).
double choose_tile(const GemmArgs& g, Plan2* p) {
  const bool half = g.dtype == DT_BF16;
  const int64_t steps = std::max<int64_t>(p->all_steps, 1);
  double best = 1e300;
  for (int i = 0; i < (half ? 3 : 2); ++i) {
    const TileCost& t = half ? COST_BF16[i] : COST_F32[i];
    // the 256-tile with both operands transposed does not fit the registers
    if (t.tile == 256 && g.a.trans && g.b.trans) continue;
    const int64_t tm = ceil_div(g.m, t.tile), tn = ceil_div(g.n, t.tile), tiles = tm * tn;
    const int64_t slots = (int64_t)g.cus * t.holds;
    // so many pieces of so many steps side by side on a compute unit
    auto round = [&](int64_t together, int64_t per) {
      return together ? (double)per * std::max(t.alone, (double)together * t.shared) + t.ends : 0.0;
    };
    const int64_t wholes[] = {0, tiles / g.cus * g.cus, tiles / slots * slots};
    for (int w = 0; w < 3; ++w) {
      const int64_t whole = wholes[w], rest = tiles - whole;
      if (!rest || (w && whole == wholes[w - 1])) continue;
      for (const int64_t split : SPLITS) {
        if (split > 1 && (steps / split < 2 || rest * split > 2 * slots)) break;
        const int64_t per = ceil_div(steps, split), parts = ceil_div(steps, per);
        const int64_t a = whole / g.cus, b = ceil_div(rest * parts, g.cus);   // of the busiest compute unit
        const int64_t left = a % t.holds;
        double us = (double)(a / t.holds) * round(t.holds, steps);
        if (!left) us += (double)(b / t.holds) * round(t.holds, per) + round(b % t.holds, per);
        else
          us += std::max((double)steps * t.alone, (double)(left * steps + b * per) * t.shared) +
                t.ends * (double)ceil_div(left + b, t.holds);
        // joining the parts: a launch (4 us on the device, 5 of the host), and their way through memory
        if (parts > 1) us += 6 + (double)g.m * (double)g.n * (double)rest / (double)tiles * (double)parts * 2e-6;
        if (us < best) {
          best = us;
          p->tile = t.tile;
          p->tiles_m = (uint32_t)tm;
          p->tiles_n = (uint32_t)tn;
          p->steps = (uint32_t)per;
          p->split = (uint32_t)parts;
          p->whole = (uint32_t)(parts > 1 ? whole : tiles);
          p->rest = (uint32_t)(parts > 1 ? rest : 0);
        }
      }
    }
  }
  return best;
}

Plan2 plan_gemm(const GemmArgs& g) {
  Plan2 p;
  const int64_t es = g.dtype == DT_BF16 ? 2 : 4, v = 16 / es, bk = 128 / es;
  // Few rows and a summed axis that one workgroup soon reads: one launch.
  // bf16, 16 rows, against split tiles: 64 x 4096 (n x k) 9.4 us to 15.4,
  // 16384 x 4096 30 to 28, 512 x 12288 23 to 15; f32 4096 x 4096 19 to 29.
  // Beyond 16 rows x is read twice as often as by the tiles: 32 rows of bf16,
  // 4096 x 4096 14 us to 16, 16384 x 4096 46 to 28.
  const int64_t line = g.k * es;
  if (!g.a.trans && !g.b.trans && ((g.m <= 16 && line <= 16384) ||
                                   (g.m <= 32 && line <= 8192 && g.n * g.k <= (int64_t(1) << 24)))) {
    p.few = true;
    return p;
  }
  p.pack_a = needs_pack(g.a, g.m, g.k, es);
  p.pack_b = needs_pack(g.b, g.n, g.k, es);
  auto packed = [&](const Operand& o, int64_t rows, size_t* bytes) {
    const int64_t line = o.trans ? rows : g.k, lines = o.trans ? g.k : rows;
    const int64_t ld = ceil_div(line, v) * v;
    *bytes = align256((size_t)ld * (size_t)lines * (size_t)es);
    return (uint32_t)ld;
  };
  size_t ba = 0, bb = 0;
  if (p.pack_a) p.lda = packed(g.a, g.m, &ba);
  if (p.pack_b) p.ldb = packed(g.b, g.n, &bb);
  p.off_b = ba;
  p.off_part = ba + bb;
  p.total = p.off_part;
  p.all_steps = (uint32_t)ceil_div(g.k, bk);
  const double us = choose_tile(g, &p);
  // More rows of a small product whose operands would have to be copied first
  // go the same way, 32 at a time, where the rows read again, out of the
  // caches, cost less than the copies and their launch (x of m rows, n x k; bf16
  // 206 x 1810 x 157 9.9 us to 13.8, 1000 x 1000 x 131 13.0 to 13.9, 500 x 2000 x 259
  // 17.5 to 14.1, 837 x 4439 x 31 22.7 to 14.0; f32 300 x 1000 x 515 11.9 to 19.4,
  // 100 x 5000 x 515 19.8 to 25.9, 500 x 2000 x 259 18.0 to 15.1).
  if ((ba || bb) && !g.a.trans && !g.b.trans && line <= 8192) {
    const double blocks = (double)ceil_div(g.m, 32) * (double)ceil_div(g.n, 16);
    const double few = blocks * (1.5e-3 + (double)(48 * g.k) / (es == 2 ? 2.5e6 : 2.0e6));
    if (few + 4 < us + 6 + (double)(ba + bb) / 1.5e6) {
      p = Plan2();
      p.few = true;
      return p;
    }
  }
  p.total += (size_t)p.split * p.rest * p.tile * p.tile * 4;
  return p;
}

template <class T, int R, int NWM, int NWN>
void go(const KGemm& k, bool ta, bool tb, dim3 grid, hipStream_t s) {
  const dim3 block(NWM * NWN * 64);
  if (ta && tb) {   // (no 256-tile: see choose_tile)
    if constexpr (R < 256) hipLaunchKernelGGL((k_gemm<T, R, R, NWM, NWN, true, true>), grid, block, 0, s, k);
  } else if (ta) hipLaunchKernelGGL((k_gemm<T, R, R, NWM, NWN, true, false>), grid, block, 0, s, k);
  else if (tb) hipLaunchKernelGGL((k_gemm<T, R, R, NWM, NWN, false, true>), grid, block, 0, s, k);
  else hipLaunchKernelGGL((k_gemm<T, R, R, NWM, NWN, false, false>), grid, block, 0, s, k);
}

// A product in steps: copies of the operands that need one, the tiles, the
// join of split sums (which several products share).
template <class T>
struct Product {
  static constexpr int64_t ES = sizeof(T), V = 16 / ES;
  GemmArgs g;
  Plan2 p;
  char* ws;

  Product(const GemmArgs& args, char* scratch) : g(args), p(plan_gemm(args)), ws(scratch) {}

  KPack pack_of(const Operand& o, int64_t rows, uint32_t ldo, void* dst) const {
    const int64_t line = o.trans ? rows : g.k, lines = o.trans ? g.k : rows;
    return KPack{o.p, dst, o.ld, (uint32_t)line, ldo, (uint64_t)(ldo / V) * (uint64_t)lines};
  }
  int packs(KPack* out) const {
    int n = 0;
    if (p.pack_a) out[n++] = pack_of(g.a, g.m, p.lda, ws);
    if (p.pack_b) out[n++] = pack_of(g.b, g.n, p.ldb, ws + p.off_b);
    return n;
  }
  KOperand operand(const Operand& o, int64_t rows, bool pack, uint32_t ldp, const char* at) const {
    KOperand k;
    const int64_t line = o.trans ? rows : g.k, lines = o.trans ? g.k : rows;
    k.p = pack ? at : o.p;
    k.ld = pack ? ldp : (lines > 1 ? o.ld : line);
    k.rows = (uint32_t)rows;
    // for the tiles a line that ends in zeros counts as whole chunks; the few
    // rows' kernel masks the last chunk itself, of both operands alike, and the
    // other one's lines may go on with anything
    k.red = (uint32_t)((pack || o.padded) && !o.trans && !p.few ? ceil_div(g.k, V) * V : g.k);
    return k;
  }
  // Rows that begin inside a line are stored in pieces that the caches have to
  // put together (2000 x 65537 bf16 169 us past them, 91 through them; where a
  // residual comes through the caches too, 180 and 201).
  static bool aligned(const void* p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * ES % 16 == 0; }
  Epi epilogue() const {
    return Epi{g.bias, g.residual, g.c, g.pre, g.ldr, g.ldc, g.ldp, (uint32_t)g.m, (uint32_t)g.n, g.act,
               g.m * g.n * ES >= STREAM_BYTES && (g.residual || aligned(g.c, g.ldc))};
  }
  KGemm args() const {
    KGemm k{};
    k.a = operand(g.a, g.m, p.pack_a, p.lda, ws);
    k.b = operand(g.b, g.n, p.pack_b, p.ldb, ws + p.off_b);
    k.e = epilogue();
    k.part = reinterpret_cast<float*>(ws + p.off_part);
    k.tiles_m = p.tiles_m;
    k.tiles_n = p.tiles_n;
    k.whole = p.whole;
    k.rest = p.rest;
    k.split = p.split;
    k.pieces = p.whole + p.rest * p.split;
    k.steps = p.steps;
    k.all_steps = p.all_steps;
    return k;
  }
  hipError_t tiles(hipStream_t s) const {
    const KGemm k = args();
    if (p.few) {
      const uint32_t rows = (uint32_t)ceil_div(g.m, g.m <= 16 ? 16 : 32);
      const dim3 grid((uint32_t)ceil_div(g.n, 16), std::min(rows, FEW_Y), (uint32_t)ceil_div(rows, FEW_Y));
      // 16 waves where each has a turn, unless the workgroups alone fill the card
      // (4096 x 4096 f32 16.8 us against 21.4; 16384 x 4096 56 against 54.7)
      const bool deep = g.k * ES >= 4096 && g.n < 16384;
      if (g.m <= 16 && deep) hipLaunchKernelGGL((k_few_rows<T, 1, 16>), grid, dim3(1024), 0, s, k);
      else if (g.m <= 16) hipLaunchKernelGGL((k_few_rows<T, 1, 4>), grid, dim3(256), 0, s, k);
      else if (deep) hipLaunchKernelGGL((k_few_rows<T, 2, 16>), grid, dim3(1024), 0, s, k);
      else hipLaunchKernelGGL((k_few_rows<T, 2, 4>), grid, dim3(256), 0, s, k);
      return hipGetLastError();
    }
    const dim3 grid = wide_grid(k.pieces);
    if constexpr (ES == 2) {
      if (p.tile == 256) {
        go<T, 256, 2, 4>(k, g.a.trans, g.b.trans, grid, s);
        return hipGetLastError();
      }
    }
    if (p.tile == 128) go<T, 128, 2, 2>(k, g.a.trans, g.b.trans, grid, s);
    else go<T, 64, 2, 2>(k, g.a.trans, g.b.trans, grid, s);
    return hipGetLastError();
  }
  int joins(KJoin* out) const {
    if (!p.rest) return 0;
    KJoin& j = out[0] = KJoin{};
    j.part = reinterpret_cast<const float*>(ws + p.off_part);
    j.split = p.split;
    j.whole = p.whole;
    j.rest = p.rest;
    j.tile = p.tile;
    j.tiles_m = p.tiles_m;
    j.tiles_n = p.tiles_n;
    j.e = epilogue();
    return 1;
  }
};

template <class T>
hipError_t run_packs(KPack* packs, int n, hipStream_t s) {
  if (!n) return hipSuccess;
  if (n == 1) packs[1] = KPack{};
  hipLaunchKernelGGL((k_pack<T>), wide_grid((packs[0].vecs + packs[1].vecs + 255) / 256), dim3(256), 0, s, packs[0],
                     packs[1]);
  return hipGetLastError();
}

template <class T>
hipError_t run_gemm(const GemmArgs& g, char* ws, hipStream_t s) {
  const Product<T> q(g, ws);
  KPack packs[2];
  KJoin join;
  hipError_t e = run_packs<T>(packs, q.packs(packs), s);
  if (e == hipSuccess) e = q.tiles(s);
  if (e == hipSuccess) e = run_joins<T>(&join, q.joins(&join), s);
  return e;
}

// ---------------------------------------------------------------- slope pass
// dz = dy * act'(z), and the column sums of dz in 32 bits.  Bound by memory:
// 4096 x 12288 bf16 with relu reads 201 MB and writes 101, 55 us, 5.5 TB/s.  A
// workgroup of four waves takes 64 VEC columns and a block of rows; each lane
// sums its VEC columns down the block's rows, the four waves join in LDS, and
// one partial row per block goes to the workspace, to be joined in block
// order; a single block writes the sums themselves.  The workgroups behind
// copy the products' other operands where they need it: small calls take as
// long as their launches.
template <class T>
struct KSlope {
  const T* dy;
  const T* pre;
  T* dz;             // null: not wanted
  float* part;       // null: no column sums, or `db` takes them
  T* db;
  int64_t ldd, ldp, ldz;
  uint32_t m, n, rows_per, ldpart;
  uint32_t columns, blocks;   // workgroups side by side, and in all
};

constexpr uint32_t SLOPE_AHEAD = 8;

// A lane's elements of a row as they were read: 16 bytes, or one element.
template <class T, int VEC>
__device__ __forceinline__ u32x4 raw_vec(const T* p) {
  if constexpr (VEC == 1) return u32x4{__float_as_uint(to_f32(p[0])), 0u, 0u, 0u};
  else return read16(p);
}
template <class T, int VEC>
__device__ __forceinline__ void unpack_vec(u32x4 q, float* v) {
  if constexpr (VEC == 1) v[0] = __uint_as_float(q[0]);
  else Vec<T>::unpack(q, v);
}

template <class T, int ACT, int VEC>
__global__ __launch_bounds__(256) void k_slope(KSlope<T> p, KPack pack_a, KPack pack_b) {
  const uint32_t id = block_id();
  if (id >= p.blocks) {
    pack_vec<T>(pack_a, pack_b, (uint64_t)(id - p.blocks) * 256 + threadIdx.x);
    return;
  }
  const T* __restrict__ dy = p.dy;
  const T* __restrict__ pre = p.pre;
  T* __restrict__ dz = p.dz;
  const uint32_t bx = id % p.columns, by = id / p.columns, n = p.n;
  const uint32_t wave = threadIdx.x / 64, lane = threadIdx.x % 64;
  const uint32_t c0 = (bx * 64 + lane) * VEC;
  const uint32_t c = c0 < n ? column_of<VEC>(c0, n) : 0u;
  const uint32_t r0 = by * p.rows_per;
  const uint32_t r1 = p.m - r0 < p.rows_per ? p.m : r0 + p.rows_per;
  // behind the last column: zeros up to whole 16 bytes
  constexpr uint32_t CHUNK = Vec<T>::N;
  const uint32_t fill = c0 < n && c0 + VEC >= n ? (n + CHUNK - 1) / CHUNK * CHUNK : n;
  float sum[VEC] = {};
  // all loads of SLOPE_AHEAD rows leave before the first is used
  for (uint32_t rr = r0 + wave; rr < r1 && c0 < n; rr += 4 * SLOPE_AHEAD) {
    u32x4 qd[SLOPE_AHEAD], qz[SLOPE_AHEAD];
#pragma unroll
    for (uint32_t u = 0; u < SLOPE_AHEAD; ++u) {
      const uint32_t r = rr + 4 * u < r1 ? rr + 4 * u : rr;
      qd[u] = raw_vec<T, VEC>(dy + (int64_t)r * p.ldd + c);
      if constexpr (ACT != ACT_NONE) qz[u] = raw_vec<T, VEC>(pre + (int64_t)r * p.ldp + c);
    }
#pragma unroll
    for (uint32_t u = 0; u < SLOPE_AHEAD; ++u) {
      const uint32_t r = rr + 4 * u;
      if (r >= r1) break;
      float v[VEC];
      unpack_vec<T, VEC>(qd[u], v);
      if constexpr (ACT != ACT_NONE) {
        float z[VEC];
        unpack_vec<T, VEC>(qz[u], z);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          if constexpr (ACT == ACT_RELU) v[i] = z[i] <= 0.f ? 0.f : v[i];
          else v[i] *= slope_of<ACT, T>(z[i]);
        }
      }
      if (dz) {
        T* o = dz + (int64_t)r * p.ldz;
        store_vec<T, VEC>(o + c, v);
        for (uint32_t i = n; i < fill; ++i) o[i] = T{};
      }
#pragma unroll
      for (int i = 0; i < VEC; ++i) sum[i] += v[i];
    }
  }
  if (!p.part && !p.db) return;
  __shared__ float join[4][64 * VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) join[wave][lane * VEC + i] = sum[i];
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < 64 * VEC; i += 256) {
    const uint32_t cc = (bx * 64 + i / VEC) * VEC;
    if (cc >= n) continue;
    // (columns that two lanes hold get the same sum from both)
    const uint32_t at = column_of<VEC>(cc, n) + i % VEC;
    const float v = (join[0][i] + join[1][i]) + (join[2][i] + join[3][i]);
    if (p.part) p.part[(size_t)by * p.ldpart + at] = v;
    else p.db[at] = from_f32<T>(v);
  }
}

// Workgroups side by side.
uint32_t slope_columns(const SlopeArgs& a) {
  const int64_t v = a.dtype == DT_BF16 ? 8 : 4;
  return (uint32_t)ceil_div(a.n, 64 * (a.n >= v ? v : 1));
}
// Rows of a block: 64, fewer while there is less than a workgroup for each of
// 256 compute units (a row of gelu or silu takes a wave alone 1.6 us: 225 x 35
// bf16 30 us in blocks of 64), more beyond 65535 blocks.  A few rows are one
// block, which spares the join's launch.
uint32_t slope_rows(const SlopeArgs& a) {
  if (a.m <= (a.act > ACT_RELU ? 16 : 64)) return 64;
  const int64_t share = ceil_div(a.m * slope_columns(a), 256 * 4) * 4;
  return (uint32_t)std::max(std::min<int64_t>(64, share), ceil_div(a.m, 65535));
}
uint32_t slope_blocks(const SlopeArgs& a) { return (uint32_t)ceil_div(a.m, slope_rows(a)); }
uint32_t slope_ld(int64_t n) { return (uint32_t)(ceil_div(n, 4) * 4); }

template <class T, int ACT>
hipError_t run_slope(const SlopeArgs& a, float* part, const KPack* packs, hipStream_t s) {
  constexpr int V = Vec<T>::N;
  const bool wide = a.n >= V, one = slope_blocks(a) == 1;
  KSlope<T> k;
  k.dy = static_cast<const T*>(a.dy);
  k.pre = static_cast<const T*>(a.pre);
  k.dz = static_cast<T*>(a.dz);
  k.part = a.db && !one ? part : nullptr;
  k.db = one ? static_cast<T*>(a.db) : nullptr;
  k.ldd = a.ldd;
  k.ldp = a.ldp;
  k.ldz = a.ldz;
  k.m = (uint32_t)a.m;
  k.n = (uint32_t)a.n;
  k.rows_per = slope_rows(a);
  k.ldpart = slope_ld(a.n);
  k.columns = slope_columns(a);
  k.blocks = k.columns * slope_blocks(a);
  const dim3 grid = wide_grid(k.blocks + (packs[0].vecs + packs[1].vecs + 255) / 256);
  if (wide) hipLaunchKernelGGL((k_slope<T, ACT, V>), grid, dim3(256), 0, s, k, packs[0], packs[1]);
  else hipLaunchKernelGGL((k_slope<T, ACT, 1>), grid, dim3(256), 0, s, k, packs[0], packs[1]);
  return hipGetLastError();
}

bool slope_wanted(const SlopeArgs& a) { return a.m && a.n && (a.dz || a.db); }

template <class T>
hipError_t run_slope_act(const SlopeArgs& a, float* part, const KPack* packs, hipStream_t s) {
  if (!slope_wanted(a)) return hipSuccess;
  switch (a.act) {
    case ACT_RELU: return run_slope<T, ACT_RELU>(a, part, packs, s);
    case ACT_GELU: return run_slope<T, ACT_GELU>(a, part, packs, s);
    case ACT_SILU: return run_slope<T, ACT_SILU>(a, part, packs, s);
    default: return run_slope<T, ACT_NONE>(a, part, packs, s);
  }
}

// The column sums' join, as a product of one row whose parts are the blocks
// (none for no rows: zeros).  One block has written them.
int slope_join(const SlopeArgs& a, const float* part, KJoin* out) {
  if (!a.db || !a.n || slope_blocks(a) == 1) return 0;
  KJoin& j = out[0] = KJoin{};
  j.part = part;
  j.split = slope_blocks(a);
  j.ldpart = slope_ld(a.n);
  j.e.c = a.db;
  j.e.m = 1;
  j.e.n = (uint32_t)a.n;
  return 1;
}

// ---------------------------------------------------------------- gradients
// Scratch: dz, then the column sums' parts, then each product's.
struct GradPlan {
  SlopeArgs slope;
  GemmArgs dx, dw;
  size_t off_sums = 0, off_dx = 0, off_dw = 0, total = 0;
};

GradPlan plan_grad(const GradArgs& a) {
  GradPlan p;
  const int64_t es = a.slope.dtype == DT_BF16 ? 2 : 4;
  const int64_t m = a.slope.m, n = a.slope.n;
  p.slope = a.slope;
  const bool products = (a.dx || a.dw) && m && n;
  // dz of its own where there is a slope to take, or where dy would have to be
  // copied for the products anyway
  const Operand dy{a.slope.dy, a.slope.ldd, false};
  const bool own = products && (a.slope.act != ACT_NONE || needs_pack(dy, m, n, es));
  Operand dz = dy;
  if (own) {
    p.slope.ldz = ceil_div(n, 64) * 64;
    p.off_sums = align256((size_t)m * (size_t)p.slope.ldz * (size_t)es);
    dz = Operand{nullptr, p.slope.ldz, false, true};
  }
  p.off_dx = p.off_sums + slope_workspace(a.slope);
  auto product = [&](const Operand& x, const Operand& y, int64_t rows, int64_t cols, int64_t red, void* c, int64_t ldc) {
    GemmArgs g;
    g.a = x;
    g.b = y;
    g.m = rows;
    g.n = cols;
    g.k = red;
    g.dtype = a.slope.dtype;
    g.c = c;
    g.ldc = ldc;
    g.cus = a.cus;
    return g;
  };
  Operand dzt = dz, wt = a.w, xt = a.x;
  dzt.trans = true;
  wt.trans = !wt.trans;   // the second operands' summed axes are n and m
  xt.trans = !xt.trans;
  p.dx = product(dz, wt, m, a.k, n, a.dx, a.lddx);
  p.dw = product(dzt, xt, n, a.k, m, a.dw, a.lddw);
  p.off_dw = p.off_dx + (a.dx ? gemm_workspace(p.dx) : 0);
  p.total = p.off_dw + (a.dw ? gemm_workspace(p.dw) : 0);
  return p;
}

// Whether one launch can take both products: the same tile, dz and the
// others as they lie when x and W are stored by rows, no product of few rows.
template <class T>
bool pairs(const Product<T>& x, const Product<T>& w) {
  return !x.p.few && !w.p.few && x.p.tile == w.p.tile && x.p.tile < 256 && !x.g.a.trans && x.g.b.trans &&
         w.g.a.trans && w.g.b.trans;
}

template <class T>
hipError_t run_pair(const Product<T>& x, const Product<T>& w, hipStream_t s) {
  const KGemm a = x.args(), b = w.args();
  const uint32_t la = a.whole ? a.all_steps : a.steps, lb = b.whole ? b.all_steps : b.steps;
  const dim3 grid = wide_grid((uint64_t)a.pieces + b.pieces);
  if (x.p.tile == 128) hipLaunchKernelGGL((k_gemm_pair<T, 128, 128, 2, 2>), grid, dim3(256), 0, s, a, b, lb > la);
  else hipLaunchKernelGGL((k_gemm_pair<T, 64, 64, 2, 2>), grid, dim3(256), 0, s, a, b, lb > la);
  return hipGetLastError();
}

template <class T>
hipError_t run_grad(const GradArgs& a, char* ws, hipStream_t s) {
  GradPlan p = plan_grad(a);
  if (p.slope.ldz) {
    p.slope.dz = ws;
    p.dx.a.p = p.dw.a.p = ws;
  }
  float* sums = reinterpret_cast<float*>(ws + p.off_sums);
  const bool dx = a.dx && p.dx.m && p.dx.n, dw = a.dw && p.dw.m && p.dw.n;
  const Product<T> qx(p.dx, ws + p.off_dx), qw(p.dw, ws + p.off_dw);
  KPack packs[6] = {};
  KJoin joins[3];
  int np = 0, nj = 0;
  if (dx) np += qx.packs(packs + np);
  if (dw) np += qw.packs(packs + np);
  // the copies ride in the pass over dy, unless one is of its result
  const KPack none[2] = {};
  const bool ride = slope_wanted(p.slope) && np <= 2 && !(dx && qx.p.pack_a) && !(dw && qw.p.pack_a);
  hipError_t e = run_slope_act<T>(p.slope, sums, ride ? packs : none, s);
  for (int i = 0; i < np && !ride && e == hipSuccess; i += 2) e = run_packs<T>(packs + i, std::min(2, np - i), s);
  if (e == hipSuccess && dx && dw && pairs(qx, qw)) {
    e = run_pair(qx, qw, s);
  } else {
    if (e == hipSuccess && dx) e = qx.tiles(s);
    if (e == hipSuccess && dw) e = qw.tiles(s);
  }
  if (dx) nj += qx.joins(joins + nj);
  if (dw) nj += qw.joins(joins + nj);
  nj += slope_join(p.slope, sums, joins + nj);
  if (e == hipSuccess) e = run_joins<T>(joins, nj, s);
  return e;
}

}  // namespace

size_t gemm_workspace(const GemmArgs& g) {
  return g.m && g.n ? plan_gemm(g).total : 0;
}

hipError_t launch_gemm(const GemmArgs& g, void* ws, hipStream_t s) {
  if (g.m == 0 || g.n == 0) return hipSuccess;
  return g.dtype == DT_BF16 ? run_gemm<bf16_t>(g, static_cast<char*>(ws), s)
                            : run_gemm<float>(g, static_cast<char*>(ws), s);
}

size_t slope_workspace(const SlopeArgs& a) {
  return a.db ? align256((size_t)slope_blocks(a) * slope_ld(a.n) * 4) : 0;
}

hipError_t launch_slope(const SlopeArgs& a, void* ws, hipStream_t s) {
  float* part = static_cast<float*>(ws);
  KJoin join;
  const int n = slope_join(a, part, &join);
  const KPack none[2] = {};
  hipError_t e = a.dtype == DT_BF16 ? run_slope_act<bf16_t>(a, part, none, s) : run_slope_act<float>(a, part, none, s);
  if (e != hipSuccess) return e;
  return a.dtype == DT_BF16 ? run_joins<bf16_t>(&join, n, s) : run_joins<float>(&join, n, s);
}

hipError_t launch_join(const JoinArgs& a, hipStream_t s) {
  KJoin join{};
  join.part = a.part;
  join.split = a.split;
  join.ldpart = a.ldpart;
  join.e.bias = a.bias;
  join.e.c = a.out;
  join.e.ldc = a.ldo;
  join.e.m = (uint32_t)a.m;
  join.e.n = (uint32_t)a.n;
  return a.dtype == DT_BF16 ? run_joins<bf16_t>(&join, 1, s) : run_joins<float>(&join, 1, s);
}

size_t grad_workspace(const GradArgs& a) { return plan_grad(a).total; }

hipError_t launch_grad(const GradArgs& a, void* ws, hipStream_t s) {
  return a.slope.dtype == DT_BF16 ? run_grad<bf16_t>(a, static_cast<char*>(ws), s)
                                  : run_grad<float>(a, static_cast<char*>(ws), s);
}

}  // namespace tk
