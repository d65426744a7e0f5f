// A cache of keys and values that keeps what attention looked at.
//
//   attend   s_ij = scale <q_i, k_j>,  p_i = softmax(s_i),  out_i = sum_j p_ij v_j,
//            scores_j += sum of p_ij over the heads i that share the keys
//   evict    the entries with the largest scores, and the newest, in their old order
//
// Both are bound by the cache that they read.  16 sequences of 8192, 32 heads on
// 8, 128 wide bf16 (537 MB) take 85 us without the scores, 6.3 TB/s, and 109
// with them: the logits go through memory once, for a probability is known only
// when the whole row is (17 MB written and read).  Lengths spread evenly up to
// 8192 take 60 to 72, with the lengths drawn: 45 to 60 the first launch, 7.5 the
// second.  One sequence of 4099, 12 heads on 4, 80 wide f32: 8.3 + 6 us, latency.
// Eviction of 16 x 8 heads of 16384 down to 4096, 128 wide bf16 (549 MB): 18 us
// to choose, 93 to copy, 5.9 TB/s.
#include <algorithm>

#include "topk_model.hpp"
#include "topk_ops_device.hpp"

namespace tk {

namespace {

constexpr float LOG2E = 1.4426950408889634f;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ uint32_t length_of(const int64_t* lengths, uint64_t b, uint32_t n) {
  if (!lengths) return n;
  const int64_t v = lengths[b];
  return v < 0 ? 0u : v > (int64_t)n ? n : (uint32_t)v;
}

// ---------------------------------------------------------------- attend
// One key-value head serves `group` query heads, taken 16 at a time as one side
// of the matrix instructions; the keys are the other.  A wave takes STEP keys
// at a time:
//
//   S[key, head] = K Q^T: a lane's registers of K are one vector of a key's row
//     as it lies in memory, and S lands with a head to a lane and four keys to
//     a register quad;
//   O[head, column] += P V: the order of the summed keys is free, so P is used
//     where S left it, and V is loaded by whole vectors of the rows that match
//     (bf16: pairs of rows are interleaved by v_perm; f32: as they are).
//
// So neither operand goes through LDS.  The running maximum is raised only when
// some logit exceeds it, which a ballot tells: the exchange between lanes that
// this takes is rare.
constexpr uint32_t ATT_WAVES = 4;
constexpr uint32_t ATT_THREADS = 64 * ATT_WAVES;
constexpr uint32_t HEADS = 16;          // query heads of a workgroup
constexpr uint32_t JOIN_THREADS = 256;
constexpr uint32_t JOIN_KEYS = 4 * JOIN_THREADS;

struct AttArgs {
  const void* q;
  const void* k;
  const void* v;
  const int64_t* lengths;
  float* scores;      // null: not wanted
  void* out;
  float* logits;      // [batch * heads][n], in units of log 2; null: not wanted
  float* part;        // [pieces][min(group, HEADS)][d]
  float* ml;          // [pieces][HEADS][2]: maximum and sum
  uint32_t* ends;     // [rows][2]: the first and the last workgroup of a row's pieces
  int64_t sqb, sqh, skb, skh, skn, svb, svh, svn, ssb, ssh, sob, soh;
  uint64_t work;      // workgroups of the launch
  uint32_t batch, kv_heads, group, blocks16, n, d;
  uint32_t share;     // workgroups that share the keys; 0: each has a row to itself
  float scale2;
};

// Word i of a vector without the vector's first `seen` elements.
template <class T>
__device__ __forceinline__ uint32_t unseen(uint32_t word, uint32_t i, uint32_t seen) {
  if constexpr (sizeof(T) == 4) return i < seen ? 0u : word;
  return 2 * i >= seen ? word : 2 * i + 1 == seen ? word & 0xFFFF0000u : 0u;
}

template <class T> struct Att;
template <> struct Att<bf16_t> {
  static constexpr uint32_t STEP = 32, KVEC = 8, KCHUNK = 32;
  typedef bf16x8 Frag;
};
template <> struct Att<float> {
  static constexpr uint32_t STEP = 16, KVEC = 4, KCHUNK = 16;
  typedef f32x4 Frag;
};

// One vector of a row, at its column c (c + N <= d, or d < N: what the row has, then zeros).
template <class T, uint32_t N, bool NARROW, bool ONCE>
__device__ __forceinline__ void load_cols(const T* at, uint32_t c, uint32_t d, T* v) {
  if constexpr (NARROW) {
#pragma unroll
    for (uint32_t i = 0; i < N; ++i) {
      v[i] = T{};
      if (c + i < d) v[i] = at[i];
    }
  } else {
    if constexpr (ONCE && N * sizeof(T) == 16) {
      const u32x4 q = read16_once(at);
      __builtin_memcpy(v, &q, 16);
    } else {
      __builtin_memcpy(v, at, N * sizeof(T));
    }
  }
}

// An element at a byte offset below 2^32 from an address that all lanes share:
// the form that a load takes from a scalar register and one vector register.
template <class T>
__device__ __forceinline__ const T* at_offset(const T* base, uint32_t bytes) {
  return reinterpret_cast<const T*>(reinterpret_cast<const char*>(base) + bytes);
}

// The keys are shared out evenly, whatever the sequences' lengths: a sequence
// is `rows` rows (a key-value head and up to 16 of its query heads) of units of
// ATT_WAVES steps, all units of all sequences are numbered in that order, and
// workgroup w of `share` (at most one a unit) has those from w * all / share on.
// What it does of one row is a piece; row r of all and workgroup w make piece
// r + w, for no two pieces have the same sum, and those of a row are
// consecutive.
struct Place {
  uint64_t all;       // units of all sequences
  uint64_t from, to;  // the workgroup's
  uint64_t before;    // those before sequence b, in which `from` lies
  uint32_t b, units;  // units: of one of b's rows
};

// a / b; a 64-bit division takes hundreds of instructions, and is seldom one.
__device__ __forceinline__ uint64_t quotient(uint64_t a, uint64_t b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

template <uint32_t UNIT>
__device__ __forceinline__ uint32_t units_of(const AttArgs& a, uint32_t b) {
  return (length_of(a.lengths, b, a.n) + UNIT - 1) / UNIT;
}

// Where workgroup w begins; false if nothing is left for it.  Every wave for
// itself: a lane adds up a 64th of the sequences, then the 64th that holds the
// unit looked for is divided in the same way.
template <uint32_t UNIT>
__device__ __forceinline__ bool place_of(const AttArgs& a, uint64_t w, Place* p) {
  const uint32_t lane = threadIdx.x % 64, rows = a.kv_heads * a.blocks16;
  auto share_out = [&](uint64_t all) {
    p->all = all;
    const uint64_t share = min((uint64_t)a.share, all);
    if (w >= share) return false;
    p->from = quotient(w * all, share);
    p->to = quotient((w + 1) * all, share);
    return true;
  };
  if (!a.lengths) {
    p->units = (a.n + UNIT - 1) / UNIT;
    const uint64_t each = (uint64_t)p->units * rows;
    if (!share_out(each * a.batch)) return false;
    p->b = (uint32_t)quotient(p->from, each);
    p->before = p->b * each;
    return true;
  }
  uint32_t lo = 0, count = a.batch;
  p->before = 0;
  for (bool first = true;; first = false) {
    const uint32_t per = (count + 63) / 64;
    uint64_t mine = 0;
#pragma unroll 8
    for (uint32_t i = 0; i < per; ++i) {
      const uint32_t x = lane * per + i;
      const uint32_t units = units_of<UNIT>(a, min(lo + x, a.batch - 1));   // loads that nothing hangs on
      mine += x < count ? units : 0u;
    }
    mine *= rows;
    const uint64_t up = wave_incl_sum(mine);
    if (first && !share_out(bcast64(up, 63u))) return false;
    const uint32_t x = (uint32_t)__builtin_ctzll(__ballot(p->before + up > p->from));   // some lane's is: from < all
    p->before += bcast64(up - mine, x);
    lo += x * per;
    if (per == 1) {
      p->b = lo;
      p->units = (uint32_t)quotient(bcast64(mine, x), rows);
      return true;
    }
    count = min(per, count - x * per);
  }
}

// KC: chunks of a key's columns, of which the first FULL surely lie within d (all
// of them where d is their width); VB: blocks of 16 * VW columns of V.  ONCE: the
// cache is read past the caches.  That is for large ones that no second row of
// heads reads: 16 sequences of 8192, 32 heads on 8, 128 wide bf16 take 84 us
// against 99, of 4096 48 both ways, but 64 heads on 2 of 8192 44 against 33.
//
// Waves to a SIMD: what the registers leave, but three are asked for where they are
// a few short of it, in bf16 from 65 to 96 wide past the caches (1024 sequences of
// 200, 8 heads, 80 wide 98 us against 124 with two; 16 of 4096 38 both ways).
template <class T, uint32_t KC, uint32_t FULL, uint32_t VB, uint32_t VW, bool NARROW, bool ONCE>
__global__ __launch_bounds__(ATT_THREADS, KC * VB > 8 ? 1 : sizeof(T) == 2 && KC == 3 && ONCE ? 3 : 2) void k_attend(AttArgs a) {
  typedef Att<T> C;
  constexpr uint32_t TILES = C::STEP / 16, KEYS = TILES * 4;   // KEYS: a lane's keys of a step
  constexpr uint32_t UNIT = ATT_WAVES * C::STEP;
  extern __shared__ float shared[];
  const uint64_t id = block_id();
  if (id >= a.work) return;
  const uint32_t rows = a.kv_heads * a.blocks16, d = a.d;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const uint32_t lane = threadIdx.x % 64, col = lane % 16, g = lane / 16;
  uint64_t todo;           // units of this workgroup that are left
  uint32_t b, row, unit;   // where they begin
  uint32_t units;
  if (a.share) {
    Place p;
    if (!place_of<UNIT>(a, id, &p)) return;
    todo = p.to - p.from;
    b = p.b;
    units = p.units;
    row = (uint32_t)quotient(p.from - p.before, units);
    unit = (uint32_t)(p.from - p.before - (uint64_t)row * units);
  } else {
    b = (uint32_t)quotient(id, rows);
    row = (uint32_t)(id - (uint64_t)b * rows);
    unit = 0;
    units = units_of<UNIT>(a, b);
    todo = units;
    if (!todo) {
      const uint32_t h = row / a.blocks16, h0 = row % a.blocks16 * HEADS;
      T* out = static_cast<T*>(a.out) + (uint64_t)b * a.sob + (uint64_t)(h * a.group + h0) * a.soh;
      for (uint32_t i = threadIdx.x; i < min(HEADS, a.group - h0) * d; i += ATT_THREADS) out[(uint64_t)(i / d) * a.soh + i % d] = from_f32<T>(0.f);
      return;
    }
  }
  for (;;) {
    const uint32_t len = length_of(a.lengths, b, a.n);
    const uint32_t now_units = todo < units - unit ? (uint32_t)todo : units - unit;
    const uint32_t s0 = unit * UNIT, s1 = unit + now_units == units ? len : s0 + now_units * UNIT;
    const uint32_t h = row / a.blocks16, h0 = row % a.blocks16 * HEADS;
    const uint32_t heads = min(HEADS, a.group - h0);                    // of this row
    const uint64_t bh = (uint64_t)b * a.kv_heads + h;
    const uint64_t first = bh * a.group + h0;                           // its first head, of all
    T* out = static_cast<T*>(a.out) + (uint64_t)b * a.sob + (uint64_t)(h * a.group + h0) * a.soh;
    const bool mine = col < heads;
    const T* qrow = static_cast<const T*>(a.q) + (uint64_t)b * a.sqb + (uint64_t)(h * a.group + h0 + (mine ? col : 0)) * a.sqh;

    // Q as the second operand.  A row's last vector begins earlier, so that it
    // ends with the row: what the vector before it has is 0 here, and in the keys
    // too (0 * inf is not 0).
    typename C::Frag q[KC];
    uint32_t kcol[KC], vcol[VB];
#pragma unroll
    for (uint32_t c = 0; c < KC; ++c) {
      const uint32_t want = c * C::KCHUNK + g * C::KVEC;
      kcol[c] = NARROW ? want : min(want, d - C::KVEC);
      T t[C::KVEC];
      load_cols<T, C::KVEC, NARROW, false>(qrow + kcol[c], kcol[c], d, t);
      uint32_t seen = mine ? want - kcol[c] : C::KVEC;
      asm volatile("" : "+v"(seen));   // as conditions held for the next piece they fill the scalar registers
      u32x4 w;
      __builtin_memcpy(&w, t, 16);
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) w[i] = unseen<T>(w[i], i, seen);
      __builtin_memcpy(&q[c], &w, sizeof(q[c]));
    }
#pragma unroll
    for (uint32_t x = 0; x < VB; ++x) {
      const uint32_t want = x * 16 * VW + col * VW;
      vcol[x] = NARROW ? want : min(want, d - VW);
    }
    f32x4 o[VB][VW];
#pragma unroll
    for (uint32_t x = 0; x < VB; ++x)
#pragma unroll
      for (uint32_t j = 0; j < VW; ++j) o[x][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f;   // of head `col`: m alike in the four lanes that share it, l of this lane's keys
    float* logit_row = a.logits ? a.logits + (first + (mine ? col : 0)) * a.n : nullptr;

    const uint32_t ldk = (uint32_t)a.skn * (uint32_t)sizeof(T), ldv = (uint32_t)a.svn * (uint32_t)sizeof(T);
    uint32_t base = s0 + wave * C::STEP;
    const T* kbase = static_cast<const T*>(a.k) + (int64_t)b * a.skb + (int64_t)h * a.skh + (int64_t)base * a.skn;
    const T* vbase = static_cast<const T*>(a.v) + (int64_t)b * a.svb + (int64_t)h * a.svh + (int64_t)base * a.svn;
    // This lane's place of key i of a step: the order in which S holds them.
    auto key_of = [&](uint32_t i) { return (i / 4) * 16 + g * 4 + i % 4; };

    // The step's keys; a step that the sequence does not fill reads its last row again.
    T kv[TILES][KC][C::KVEC];
    auto load_keys = [&](uint32_t have) {
      const uint32_t last = min(have, C::STEP) - 1;
#pragma unroll
      for (uint32_t t = 0; t < TILES; ++t) {
        const uint32_t row = min(t * 16 + col, last) * ldk;
#pragma unroll
        for (uint32_t c = 0; c < KC; ++c)
          load_cols<T, C::KVEC, NARROW, ONCE>(at_offset(kbase, row + kcol[c] * (uint32_t)sizeof(T)), kcol[c], d, kv[t][c]);
      }
    };
    if (base < s1) load_keys(s1 - base);
    for (; base < s1; base += UNIT) {
      const uint32_t have = s1 - base;
      const bool tail = have < C::STEP;
      T vv[KEYS][VB][VW];
#pragma unroll
      for (uint32_t i = 0; i < KEYS; ++i) {
        const uint32_t row = min(key_of(i), have - 1) * ldv;
#pragma unroll
        for (uint32_t x = 0; x < VB; ++x)
          load_cols<T, VW, NARROW, ONCE>(at_offset(vbase, row + vcol[x] * (uint32_t)sizeof(T)), vcol[x], d, vv[i][x]);
      }
      vbase += (int64_t)UNIT * a.svn;
      float s[KEYS];
      // what a row's last vector shares with the one before it is 0, not only in Q
      u32x4 keep[KC];
      if constexpr (!NARROW) {
#pragma unroll
        for (uint32_t c = FULL; c < KC; ++c) {
          uint32_t seen = c * C::KCHUNK + g * C::KVEC - kcol[c];   // of the vector's columns
          asm volatile("" : "+v"(seen));   // masks held through the loop cost a wave a SIMD up to 64 wide
#pragma unroll
          for (uint32_t i = 0; i < 4; ++i) keep[c][i] = unseen<T>(~0u, i, seen);
        }
      }
#pragma unroll
      for (uint32_t t = 0; t < TILES; ++t) {
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (uint32_t c = 0; c < KC; ++c) {
          u32x4 kw;
          __builtin_memcpy(&kw, kv[t][c], 16);
          if constexpr (!NARROW)
            if (c >= FULL) kw &= keep[c];
          typename C::Frag kf;
          __builtin_memcpy(&kf, &kw, sizeof(kf));
          if constexpr (sizeof(T) == 2) {
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, q[c], acc, 0, 0, 0);
          } else {
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(kf[j], q[c][j], acc, 0, 0, 0);
          }
        }
#pragma unroll
        for (uint32_t r = 0; r < 4; ++r) s[t * 4 + r] = acc[r] * a.scale2;
      }
      // the next step's keys are on their way while this one's values are used
      kbase += (int64_t)UNIT * a.skn;
      if (have > UNIT) load_keys(have - UNIT);
      if (logit_row && mine) {
        if (!tail) {
#pragma unroll
          for (uint32_t t = 0; t < TILES; ++t) __builtin_memcpy(logit_row + base + t * 16 + g * 4, s + t * 4, 16);
        } else {
#pragma unroll
          for (uint32_t i = 0; i < KEYS; ++i)
            if (key_of(i) < have) logit_row[base + key_of(i)] = s[i];
        }
      }
      if (tail) {   // what the last row was read for once more does not count
#pragma unroll
        for (uint32_t i = 0; i < KEYS; ++i) {
          const bool in = key_of(i) < have;
          s[i] = in ? s[i] : -INFINITY;
#pragma unroll
          for (uint32_t x = 0; x < VB; ++x)
#pragma unroll
            for (uint32_t j = 0; j < VW; ++j)
              if (!in) vv[i][x][j] = T{};   // not 0 * inf
        }
      }
      float top = s[0];
#pragma unroll
      for (uint32_t i = 1; i < KEYS; ++i) top = fmaxf(top, s[i]);
      if (__any(top > m)) {
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float now = fmaxf(m, top);
        const float down = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - now);
        l *= down;
        m = now;
#pragma unroll
        for (uint32_t r = 0; r < 4; ++r) {
          const float f = __shfl(down, (int)(g * 4 + r));
#pragma unroll
          for (uint32_t x = 0; x < VB; ++x)
#pragma unroll
            for (uint32_t j = 0; j < VW; ++j) o[x][j][r] *= f;
        }
      }
      const float ref = m == -INFINITY ? 0.f : m;
      float p[KEYS];
#pragma unroll
      for (uint32_t i = 0; i < KEYS; ++i) {
        p[i] = __builtin_amdgcn_exp2f(s[i] - ref);
        l += p[i];
      }
      if constexpr (sizeof(T) == 2) {
        // A probability is the sum of two operands: its leading bits, less half a
        // step, and the rest, rounded to bf16.  The rest is between half a step and
        // one and a half, so 1.5 * 2^-15 of the probability is lost at most, and both
        // have its sign: an infinite value stays infinite.
        u32x4 near;
        float rest[KEYS];
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
          const uint32_t lo = __builtin_elementwise_sub_sat(__float_as_uint(p[2 * i]), 0x8000u);
          const uint32_t hi = __builtin_elementwise_sub_sat(__float_as_uint(p[2 * i + 1]), 0x8000u);
          near[i] = __builtin_amdgcn_perm(hi, lo, 0x07060302u);
          rest[2 * i] = p[2 * i] - __uint_as_float(lo & 0xFFFF0000u);
          rest[2 * i + 1] = p[2 * i + 1] - __uint_as_float(hi & 0xFFFF0000u);
        }
        const u32x4 far = Vec<bf16_t>::pack(rest);
        bf16x8 pn, pr;
        __builtin_memcpy(&pn, &near, 16);
        __builtin_memcpy(&pr, &far, 16);
#pragma unroll
        for (uint32_t x = 0; x < VB; ++x)
#pragma unroll
          for (uint32_t j = 0; j < VW; ++j) {
            u32x4 w;
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i) {
              uint32_t lo, hi;   // two columns of two rows
              __builtin_memcpy(&lo, &vv[2 * i][x][j & ~1u], 4);
              __builtin_memcpy(&hi, &vv[2 * i + 1][x][j & ~1u], 4);
              w[i] = __builtin_amdgcn_perm(hi, lo, j & 1 ? 0x07060302u : 0x05040100u);
            }
            bf16x8 vf;
            __builtin_memcpy(&vf, &w, 16);
            o[x][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(pr, vf, o[x][j], 0, 0, 0);
            o[x][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(pn, vf, o[x][j], 0, 0, 0);
          }
      } else {
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i)
#pragma unroll
          for (uint32_t x = 0; x < VB; ++x)
#pragma unroll
            for (uint32_t j = 0; j < VW; ++j) o[x][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(p[i], to_f32(vv[i][x][j]), o[x][j], 0, 0, 0);
      }
    }
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);

    // the waves' parts through LDS: [wave][head][d], then (m, l) of each
    float* wo = shared;
    float* wm = shared + ATT_WAVES * heads * d;
    float* wl = wm + ATT_WAVES * HEADS;
    if (g == 0) {
      wm[wave * HEADS + col] = m;
      wl[wave * HEADS + col] = l;
    }
#pragma unroll
    for (uint32_t r = 0; r < 4; ++r) {
      const uint32_t head = g * 4 + r;
      if (head >= heads) continue;
      float* row = wo + (wave * heads + head) * d;
#pragma unroll
      for (uint32_t x = 0; x < VB; ++x)
#pragma unroll
        for (uint32_t j = 0; j < VW; ++j)
          if (!NARROW || vcol[x] + j < d) row[vcol[x] + j] = o[x][j][r];
    }
    __syncthreads();
    if (threadIdx.x < HEADS) {   // one maximum and sum for the workgroup; the waves' factors in place of their maxima
      float top = -INFINITY, sum = 0.f;
      for (uint32_t w = 0; w < ATT_WAVES; ++w) top = fmaxf(top, wm[w * HEADS + threadIdx.x]);
      for (uint32_t w = 0; w < ATT_WAVES; ++w) {
        const float mw = wm[w * HEADS + threadIdx.x];
        const float f = mw == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(mw - top);
        wm[w * HEADS + threadIdx.x] = f;
        sum += f * wl[w * HEADS + threadIdx.x];
      }
      wl[threadIdx.x] = sum;
      wl[HEADS + threadIdx.x] = top;   // -inf: a piece without a probability, which the join gives the factor 0
    }
    __syncthreads();
    const uint64_t piece = (uint64_t)b * rows + row + id;
    for (uint32_t i = threadIdx.x; i < heads * d; i += ATT_THREADS) {
      const uint32_t head = i / d, c = i % d;
      float v = 0.f;
#pragma unroll
      for (uint32_t w = 0; w < ATT_WAVES; ++w) v = fmaf(wm[w * HEADS + head], wo[(w * heads + head) * d + c], v);
      if (!a.share) out[(uint64_t)head * a.soh + c] = from_f32<T>(v / wl[head]);
      else a.part[(piece * min(HEADS, a.group) + head) * d + c] = v;
    }
    if (a.share) {
      if (threadIdx.x == 0) {
        const uint64_t r = (uint64_t)b * rows + row;
        if (s0 == 0) a.ends[2 * r] = (uint32_t)id;
        if (unit + now_units == units) a.ends[2 * r + 1] = (uint32_t)id;
      }
      if (threadIdx.x < heads) {
        float* ml = a.ml + (piece * HEADS + threadIdx.x) * 2;
        ml[0] = wl[HEADS + threadIdx.x];
        ml[1] = wl[threadIdx.x];
      }
    } else if (a.scores) {
      // the whole row was this workgroup's: its logits, just written, become
      // probabilities (there is one row to a key-value head here)
      __threadfence_block();
      __syncthreads();
      float* srow = a.scores + (int64_t)b * a.ssb + (int64_t)h * a.ssh;
      for (uint32_t key = threadIdx.x; key < len; key += ATT_THREADS) {
        float sum = 0.f;
        for (uint32_t i = 0; i < heads; ++i) sum += __builtin_amdgcn_exp2f(a.logits[(first + i) * a.n + key] - wl[HEADS + i]) / wl[i];
        srow[key] += sum;
      }
    }
    todo -= now_units;
    if (!todo) return;
    __syncthreads();   // the next piece writes LDS again
    unit = 0;
    if (++row == rows) {
      row = 0;
      do units = units_of<UNIT>(a, ++b);
      while (!units);    // as long as units are left there is a sequence that has them
    }
  }
}

// The pieces of a key-value head joined: workgroups below `group` write a head's
// output, the others add up JOIN_KEYS keys' probabilities each.
template <class T>
__global__ __launch_bounds__(JOIN_THREADS) void k_attend_join(AttArgs a, uint32_t chunks) {
  // outputs: a factor for each piece; scores: a maximum and the inverse of a sum for each head
  extern __shared__ float shared[];
  __shared__ float part[4][HEAD_MAX];
  constexpr uint32_t PER = JOIN_KEYS / JOIN_THREADS, AHEAD = 4;
  const uint64_t id = block_id();
  if (id >= a.work) return;
  const uint64_t bh = quotient(id, a.group + chunks);
  const uint32_t which = (uint32_t)(id - bh * (a.group + chunks));
  const uint32_t b = (uint32_t)quotient(bh, a.kv_heads), h = (uint32_t)(bh - (uint64_t)b * a.kv_heads);
  const uint32_t len = length_of(a.lengths, b, a.n);
  const uint32_t wave = threadIdx.x / 64, lane = threadIdx.x % 64;
  T* out = static_cast<T*>(a.out) + (int64_t)b * a.sob + (int64_t)(h * a.group + which) * a.soh;
  if (len == 0) {
    if (which < a.group)
      for (uint32_t c = threadIdx.x; c < a.d; c += JOIN_THREADS) out[c] = from_f32<T>(0.f);
    return;
  }
  const uint32_t k0 = (which - a.group) * JOIN_KEYS;
  if (which >= a.group && k0 >= len) return;
  // the first heads' logits are on their way while the pieces are looked up
  const float* logits = a.logits + bh * a.group * a.n + k0;
  float* srow = a.scores + (int64_t)b * a.ssb + (int64_t)h * a.ssh + k0;
  float ahead[AHEAD][PER], sum[PER];
  if (which >= a.group) {
#pragma unroll
    for (uint32_t x = 0; x < PER; ++x) {
      const uint32_t key = x * JOIN_THREADS + threadIdx.x;
      sum[x] = 0.f;
#pragma unroll
      for (uint32_t i = 0; i < AHEAD; ++i) ahead[i][x] = i < a.group && k0 + key < len ? logits[(uint64_t)i * a.n + key] : 0.f;
    }
  }
  // first and number of the pieces of a row of this head
  auto pieces_of = [&](uint32_t hb, uint64_t* from) {
    const uint64_t row = bh * a.blocks16 + hb;
    const uint32_t w0 = a.ends[2 * row], w1 = a.ends[2 * row + 1];
    *from = row + w0;
    return w1 - w0 + 1;
  };
  if (which < a.group) {
    uint64_t from;
    const uint32_t live = pieces_of(which / HEADS, &from);
    const float* ml = a.ml + (from * HEADS + which % HEADS) * 2;
    float top = -INFINITY, whole = 0.f;     // every wave for itself
    for (uint32_t s = lane; s < live; s += 64) top = fmaxf(top, ml[s * HEADS * 2]);
#pragma unroll
    for (int o = 32; o; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
    for (uint32_t s = lane; s < live; s += 64) {
      const float f = __builtin_amdgcn_exp2f(ml[s * HEADS * 2] - top);
      whole = fmaf(f, ml[s * HEADS * 2 + 1], whole);
      if (wave == 0) shared[s] = f;
    }
    whole = wave_sum(whole);
    __syncthreads();
    // four waves share the pieces, eight rows of theirs in flight; a lane has every 64th column
    const uint64_t step = (uint64_t)min(HEADS, a.group) * a.d;
    const float* rows_of = a.part + from * step + which % HEADS * a.d;
    float v[HEAD_MAX / 64] = {};
    for (uint32_t s0 = wave; s0 < live; s0 += 4 * 8) {
#pragma unroll
      for (uint32_t x = 0; x < HEAD_MAX / 64; ++x) {
        const uint32_t c = x * 64 + lane;
        if (x * 64 >= a.d) break;
        float t[8];
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) t[i] = s0 + 4 * i < live && c < a.d ? rows_of[(s0 + 4 * i) * step + c] : 0.f;
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) v[x] = fmaf(s0 + 4 * i < live ? shared[s0 + 4 * i] : 0.f, t[i], v[x]);
      }
    }
#pragma unroll
    for (uint32_t x = 0; x < HEAD_MAX / 64; ++x) part[wave][x * 64 + lane] = v[x];
    __syncthreads();
    const uint32_t c = threadIdx.x;
    if (c < a.d) out[c] = from_f32<T>(((part[0][c] + part[1][c]) + (part[2][c] + part[3][c])) / whole);
    return;
  }
  for (uint32_t i = wave; i < a.group; i += JOIN_THREADS / 64) {
    uint64_t from;
    const uint32_t live = pieces_of(i / HEADS, &from);
    const float* ml = a.ml + (from * HEADS + i % HEADS) * 2;
    float top = -INFINITY, whole = 0.f;
    for (uint32_t s = lane; s < live; s += 64) top = fmaxf(top, ml[s * HEADS * 2]);
#pragma unroll
    for (int o = 32; o; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
    for (uint32_t s = lane; s < live; s += 64) whole = fmaf(__builtin_amdgcn_exp2f(ml[s * HEADS * 2] - top), ml[s * HEADS * 2 + 1], whole);
    whole = wave_sum(whole);
    if (lane == 0) {
      shared[2 * i] = top;
      shared[2 * i + 1] = 1.f / whole;
    }
  }
  __syncthreads();
  for (uint32_t i0 = 0; i0 < a.group; i0 += AHEAD) {
#pragma unroll
    for (uint32_t i = 0; i < AHEAD; ++i) {
      if (i0 + i >= a.group) break;
      const float top = shared[2 * (i0 + i)], inv = shared[2 * (i0 + i) + 1];
#pragma unroll
      for (uint32_t x = 0; x < PER; ++x) {
        sum[x] = fmaf(__builtin_amdgcn_exp2f(ahead[i][x] - top), inv, sum[x]);
        const uint32_t key = x * JOIN_THREADS + threadIdx.x;
        ahead[i][x] = i0 + AHEAD + i < a.group && k0 + key < len ? logits[(uint64_t)(i0 + AHEAD + i) * a.n + key] : 0.f;
      }
    }
  }
#pragma unroll
  for (uint32_t x = 0; x < PER; ++x) {
    const uint32_t key = x * JOIN_THREADS + threadIdx.x;
    if (k0 + key < len) srow[key] += sum[x];
  }
}

struct AttPlan {
  uint32_t blocks16 = 1, share = 0;
  size_t off_logits = 0, off_part = 0, off_ml = 0, off_ends = 0, total = 0;
};

// A row that one workgroup soon goes through is one workgroup's, in one launch;
// otherwise the keys are shared out over two workgroups to a compute unit, as long
// as each has a unit.  (Heads wider than 128 leave room for one at a time.)
AttPlan attend_plan(const topk_attend_args& a, int cus) {
  AttPlan p;
  if (!a.batch || !a.heads || !a.n || !a.d) return p;
  const int64_t group = a.heads / a.kv_heads;
  p.blocks16 = (uint32_t)ceil_div(group, HEADS);
  const int64_t rows = a.batch * a.kv_heads * p.blocks16;
  const int64_t unit = ATT_WAVES * (a.dtype == TOPK_BF16 ? Att<bf16_t>::STEP : Att<float>::STEP);
  const int64_t units = ceil_div(a.n, unit);
  if (units > 2 || (a.scores && p.blocks16 > 1)) p.share = (uint32_t)std::min<int64_t>(2 * cus, rows * units);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align256(bytes);
    return here;
  };
  if (a.scores) p.off_logits = take((size_t)(a.batch * a.heads * a.n) * 4);
  if (p.share) {
    const size_t pieces = (size_t)(rows + p.share);
    p.off_part = take(pieces * (size_t)(std::min<int64_t>(group, HEADS) * a.d) * 4);
    p.off_ml = take(pieces * HEADS * 8);
    p.off_ends = take((size_t)rows * 8);
  }
  p.total = at;
  return p;
}

constexpr int64_t ONCE_BYTES = int64_t(64) << 20;   // keys and values that are read past the caches

template <class T, uint32_t KC, uint32_t FULL, uint32_t VB, uint32_t VW, bool NARROW>
void attend_launch(const AttArgs& a, hipStream_t s) {
  const uint32_t heads = std::min(a.group, HEADS);
  const size_t lds = (ATT_WAVES * heads * a.d + 2 * ATT_WAVES * HEADS) * sizeof(float);
  if constexpr (!NARROW) {
    if (a.blocks16 == 1 && 2 * (int64_t)a.batch * a.kv_heads * a.n * a.d * (int64_t)sizeof(T) >= ONCE_BYTES) {
      k_attend<T, KC, FULL, VB, VW, false, true><<<wide_grid(a.work), ATT_THREADS, lds, s>>>(a);
      return;
    }
  }
  k_attend<T, KC, FULL, VB, VW, NARROW, false><<<wide_grid(a.work), ATT_THREADS, lds, s>>>(a);
}

// FULL: of the narrowest d that comes here.
template <class T, uint32_t KC, uint32_t FULL, uint32_t VB, uint32_t VW, bool NARROW>
void attend_one(const AttArgs& a, hipStream_t s) {
  if constexpr (!NARROW) {
    if (a.d == KC * Att<T>::KCHUNK) return attend_launch<T, KC, KC, VB, VW, false>(a, s);
  }
  attend_launch<T, KC, FULL, VB, VW, NARROW>(a, s);
}

void attend_typed(const AttArgs& a, bf16_t, hipStream_t s) {
  if (a.d < 8) attend_one<bf16_t, 1, 0, 1, 4, true>(a, s);
  else if (a.d <= 64) attend_one<bf16_t, 2, 0, 1, 4, false>(a, s);
  else if (a.d <= 96) attend_one<bf16_t, 3, 2, 1, 8, false>(a, s);
  else if (a.d <= 128) attend_one<bf16_t, 4, 3, 1, 8, false>(a, s);
  else if (a.d <= 192) attend_one<bf16_t, 6, 4, 2, 8, false>(a, s);
  else attend_one<bf16_t, 8, 6, 2, 8, false>(a, s);
}
void attend_typed(const AttArgs& a, float, hipStream_t s) {
  if (a.d < 4) attend_one<float, 1, 0, 1, 4, true>(a, s);
  else if (a.d <= 64) attend_one<float, 4, 0, 1, 4, false>(a, s);
  else if (a.d <= 96) attend_one<float, 6, 4, 2, 4, false>(a, s);
  else if (a.d <= 128) attend_one<float, 8, 6, 2, 4, false>(a, s);
  else if (a.d <= 192) attend_one<float, 12, 8, 3, 4, false>(a, s);
  else attend_one<float, 16, 12, 4, 4, false>(a, s);
}

template <class T>
hipError_t attend_call(const topk_attend_args& in, const AttPlan& p, char* ws, hipStream_t s) {
  AttArgs a;
  a.q = in.q;
  a.k = in.k;
  a.v = in.v;
  a.lengths = in.lengths;
  a.scores = in.scores;
  a.out = in.out;
  a.sqb = in.sqb, a.sqh = in.sqh;
  a.skb = in.skb, a.skh = in.skh, a.skn = in.skn;
  a.svb = in.svb, a.svh = in.svh, a.svn = in.svn;
  a.ssb = in.ssb, a.ssh = in.ssh;
  a.sob = in.sob, a.soh = in.soh;
  a.kv_heads = (uint32_t)in.kv_heads;
  a.group = (uint32_t)(in.heads / in.kv_heads);
  a.blocks16 = p.blocks16;
  a.n = (uint32_t)in.n;
  a.d = (uint32_t)in.d;
  a.batch = (uint32_t)in.batch;
  a.share = p.share;
  a.scale2 = in.scale * LOG2E;
  a.logits = in.scores ? reinterpret_cast<float*>(ws + p.off_logits) : nullptr;
  a.part = reinterpret_cast<float*>(ws + p.off_part);
  a.ml = reinterpret_cast<float*>(ws + p.off_ml);
  a.ends = reinterpret_cast<uint32_t*>(ws + p.off_ends);
  const uint64_t heads = (uint64_t)in.batch * a.kv_heads;
  a.work = p.share ? p.share : heads * p.blocks16;
  attend_typed(a, T{}, s);
  if (p.share) {
    const uint32_t chunks = in.scores ? (a.n + JOIN_KEYS - 1) / JOIN_KEYS : 0;
    a.work = heads * (a.group + chunks);
    k_attend_join<T><<<wide_grid(a.work), JOIN_THREADS, std::max(a.group * 8, p.share * 4), s>>>(a, chunks);
  }
  return hipGetLastError();
}

// An empty cache: every sequence attends to nothing.
template <class T>
__global__ __launch_bounds__(JOIN_THREADS) void k_attend_nothing(T* __restrict__ out, int64_t sob, int64_t soh, uint32_t heads,
                                                                 uint32_t d, uint64_t items) {
  const uint64_t i = (uint64_t)block_id() * JOIN_THREADS + threadIdx.x;
  if (i >= items) return;
  const uint64_t row = i / d;
  out[(int64_t)(row / heads) * sob + (int64_t)(row % heads) * soh + i % d] = from_f32<T>(0.f);
}

template <class T>
hipError_t attend_nothing(const topk_attend_args& a, hipStream_t s) {
  const uint64_t items = (uint64_t)(a.batch * a.heads) * (uint64_t)a.d;
  k_attend_nothing<T><<<wide_grid((items + JOIN_THREADS - 1) / JOIN_THREADS), JOIN_THREADS, 0, s>>>(
      static_cast<T*>(a.out), a.sob, a.soh, (uint32_t)a.heads, (uint32_t)a.d, items);
  return hipGetLastError();
}

// ---------------------------------------------------------------- evict
// k_evict_pick: a workgroup for each key-value head of each sequence.  Its
// scores are radix-selected, eleven bits at a time, for the key of the last
// entry that stays and the number of equal ones; then what stays is numbered in
// order, by ballots.  Rows of up to 16 K entries stay in registers
// (k_evict_pick_held); longer ones are read again for each step.
constexpr uint32_t PICK_THREADS = 1024;
constexpr uint32_t PICK_WAVES = PICK_THREADS / 64;
constexpr uint32_t COPY_THREADS = 256;
constexpr uint32_t COPY_AHEAD = 4;      // slots that a lane copies at a time

// Larger scores have larger keys; 0 and -0 are equal, NaN is above all.
__device__ __forceinline__ uint32_t score_key(float v) {
  if (v != v) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(v + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct EvictArgs {
  const void* k;
  const void* v;
  const float* scores;
  const int64_t* lengths;
  void* k_out;
  void* v_out;
  float* scores_out;
  int64_t* kept;          // [batch * heads][budget]
  int64_t* lengths_out;
  int64_t skb, skh, skn, svb, svh, svn, ssb, ssh;
  int64_t okb, okh, okn, ovb, ovh, ovn, osb, osh;
  uint64_t work;
  uint32_t heads, n, d, budget, recent, fill;
};

// The bin, from the highest down, at which the counts reach `need` (at least 1,
// at most their sum); *need becomes what is wanted of it.  Returns the bin, in
// bit 31 whether all of it is wanted.
//
// The counts come in COPIES, one for every COPIES-th lane: lanes that count in
// the same place wait for one another (128 rows of 16384 with a copy of 8
// columns down to 4096: all scores 1 59 us with one copy, 30 with four, 28 with
// eight; spread scores 34, 34 and 35).
constexpr uint32_t PICK_BINS = 2048, COPIES = 4, COPY_STRIDE = PICK_BINS + 8, ALL_OF_BIN = 0x80000000u;
constexpr uint32_t ZERO_KEY = 0x80000000u;
__device__ __forceinline__ uint32_t bin_from_top(const uint32_t* hist, uint32_t* need, uint32_t* part, uint32_t* found) {
  constexpr uint32_t PER = PICK_BINS / PICK_THREADS;
  uint32_t c[PER], sum = 0, all;
#pragma unroll
  for (uint32_t i = 0; i < PER; ++i) {
    c[i] = 0;
#pragma unroll
    for (uint32_t x = 0; x < COPIES; ++x) c[i] += hist[x * COPY_STRIDE + PICK_BINS - 1 - (threadIdx.x * PER + i)];
    sum += c[i];
  }
  uint32_t above = thread_scan<PICK_THREADS>(sum, part, &all);
  if (above < *need && *need <= above + sum) {
#pragma unroll
    for (uint32_t i = 0; i < PER; ++i) {
      if (above < *need && *need <= above + c[i]) {
        found[0] = (PICK_BINS - 1 - (threadIdx.x * PER + i)) | (*need == above + c[i] ? ALL_OF_BIN : 0u);
        found[1] = *need - above;
      }
      above += c[i];
    }
  }
  __syncthreads();
  *need = found[1];
  return found[0];
}

// What a workgroup knows of its row.
struct PickRow {
  const float* scores;
  float* scores_out;
  int64_t* kept;
  uint32_t len, old, need;   // `need` of the first `old` entries stay, and all the others
};

__device__ __forceinline__ PickRow pick_row(const EvictArgs& a, uint64_t bh) {
  const uint64_t b = bh / a.heads, h = bh - b * a.heads;
  PickRow p;
  p.len = length_of(a.lengths, b, a.n);
  const uint32_t kept = min(p.len, a.budget);
  if (h == 0 && threadIdx.x == 0) a.lengths_out[b] = kept;
  p.scores = a.scores + (int64_t)b * a.ssb + (int64_t)h * a.ssh;
  p.scores_out = a.scores_out + (int64_t)b * a.osb + (int64_t)h * a.osh;
  p.kept = a.kept + bh * a.budget;
  for (uint32_t i = kept + threadIdx.x; i < a.budget; i += PICK_THREADS) {
    p.kept[i] = -1;
    if (a.fill) p.scores_out[i] = 0.f;
  }
  p.old = p.len <= a.budget ? 0u : p.len - a.recent;
  p.need = kept - (p.len - p.old);
  return p;
}

// GROUPS groups of 64 consecutive entries to a wave, an entry of each to a lane.
template <uint32_t GROUPS>
__global__ __launch_bounds__(PICK_THREADS) void k_evict_pick_held(EvictArgs a) {
  __shared__ uint32_t hist[COPIES * COPY_STRIDE], part32[PICK_WAVES], found[2];
  __shared__ uint32_t strict[PICK_WAVES], ties[PICK_WAVES];
  const uint64_t bh = block_id();
  if (bh >= a.work) return;
  const PickRow p = pick_row(a, bh);
  const uint32_t tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / 64), lane = tid % 64;
  const uint32_t per = ((p.len + PICK_THREADS - 1) / PICK_THREADS) * 64;
  const uint32_t w0 = min(wave * per, p.len), w1 = min(w0 + per, p.len);
  if (p.len == 0) return;
  uint32_t x[GROUPS];      // the keys; 0, which is none, from p.old on
  float v[GROUPS];         // all loads leave before the first is used
#pragma unroll
  for (uint32_t g = 0; g < GROUPS; ++g) v[g] = p.scores[min(w0 + g * 64 + lane, p.len - 1)];
#pragma unroll
  for (uint32_t g = 0; g < GROUPS; ++g) {
    const uint32_t i = w0 + g * 64 + lane;
    x[g] = i < w1 && i < p.old ? score_key(v[g]) : 0u;
  }
  // entries above `key` stay, and of those equal to it the first `need`
  uint32_t key = 0xFFFFFFFFu, need = 0;
  if (p.old && p.need) {
    uint32_t prefix = 0, bits = 0;    // the first `bits` bits of the key
    need = p.need;
    for (;;) {
      const uint32_t width = bits < 22 ? 11 : 10, shift = 32 - bits - width;
      for (uint32_t i = tid; i < COPIES * COPY_STRIDE; i += PICK_THREADS) hist[i] = 0;
      __syncthreads();
      uint32_t* own = hist + lane % COPIES * COPY_STRIDE;
      uint32_t zeros = 0;      // entries that nothing has looked at: many, and counted by ballots
#pragma unroll
      for (uint32_t g = 0; g < GROUPS; ++g) {
        zeros += __popcll(__ballot(x[g] == ZERO_KEY));
        if (x[g] && x[g] != ZERO_KEY && (bits == 0 || x[g] >> (32 - bits) == prefix)) atomicAdd(&own[x[g] >> shift & ((1u << width) - 1)], 1u);
      }
      if (lane == 0 && zeros && (bits == 0 || ZERO_KEY >> (32 - bits) == prefix)) atomicAdd(&own[ZERO_KEY >> shift & ((1u << width) - 1)], zeros);
      __syncthreads();
      const uint32_t bin = bin_from_top(hist, &need, part32, found);
      prefix = prefix << width | (bin & ~ALL_OF_BIN);
      bits += width;
      if (bin & ALL_OF_BIN) {          // keys are at least 2^22: the least of this bin, less 1
        key = (prefix << shift) - 1;
        need = 0;
        break;
      }
      if (bits == 32) {
        key = prefix;
        break;
      }
    }
  }
  // every wave counts what stays of its share, and writes it behind the waves before it
  uint32_t ns = 0, nt = 0;
#pragma unroll
  for (uint32_t g = 0; g < GROUPS; ++g) {
    const uint32_t i = w0 + g * 64 + lane;
    ns += __popcll(__ballot(x[g] > key || (i >= p.old && i < w1)));
    nt += __popcll(__ballot(x[g] == key));
  }
  if (lane == 0) {
    strict[wave] = ns;
    ties[wave] = nt;
  }
  __syncthreads();
  uint32_t at = 0, tie = 0;
#pragma unroll
  for (uint32_t w = 0; w < PICK_WAVES; ++w) {
    at += w < wave ? strict[w] : 0u;
    tie += w < wave ? ties[w] : 0u;
  }
#pragma unroll
  for (uint32_t g = 0; g < GROUPS; ++g) {
    const uint32_t i = w0 + g * 64 + lane;
    const bool stays = x[g] > key || (i >= p.old && i < w1), equal = x[g] == key;
    const uint64_t ms = __ballot(stays), mt = __ballot(equal);
    const uint32_t rank = tie + rank_below(mt);
    if (stays || (equal && rank < need)) {
      const uint32_t slot = at + rank_below(ms) + min(rank, need);
      p.kept[slot] = i;
      p.scores_out[slot] = v[g];
    }
    at += __popcll(ms);
    tie += __popcll(mt);
  }
}

__global__ __launch_bounds__(PICK_THREADS) void k_evict_pick(EvictArgs a) {
  __shared__ uint32_t hist[COPIES * COPY_STRIDE], part32[PICK_WAVES], found[2];
  __shared__ uint32_t strict[PICK_WAVES], ties[PICK_WAVES];
  const uint64_t bh = block_id();
  if (bh >= a.work) return;
  const PickRow p = pick_row(a, bh);
  const uint32_t tid = threadIdx.x, wave = tid / 64, lane = tid % 64;
  uint32_t key = 0xFFFFFFFFu, need = 0;
  if (p.old && p.need) {
    uint32_t prefix = 0, bits = 0;
    need = p.need;
    while (bits < 32) {
      const uint32_t width = bits < 22 ? 11 : 10, shift = 32 - bits - width;
      for (uint32_t i = tid; i < COPIES * COPY_STRIDE; i += PICK_THREADS) hist[i] = 0;
      __syncthreads();
      for (uint32_t i = tid; i < p.old; i += PICK_THREADS) {
        const uint32_t x = score_key(p.scores[i]);
        if (bits == 0 || x >> (32 - bits) == prefix) atomicAdd(&hist[lane % COPIES * COPY_STRIDE + (x >> shift & ((1u << width) - 1))], 1u);
      }
      __syncthreads();
      prefix = prefix << width | (bin_from_top(hist, &need, part32, found) & ~ALL_OF_BIN);
      bits += width;
    }
    key = prefix;
  }
  // every wave counts what stays of its share, and writes it behind the waves before it
  const uint32_t per = ((p.len + PICK_THREADS - 1) / PICK_THREADS) * 64;
  const uint32_t w0 = min(wave * per, p.len), w1 = min(w0 + per, p.len);
  uint32_t ns = 0, nt = 0;
  for (uint32_t c = w0; c < w1; c += 64) {
    const uint32_t i = c + lane;
    const bool in = i < w1;
    const uint32_t x = in ? score_key(p.scores[i]) : 0u;
    const bool stays = in && (i >= p.old || x > key);
    ns += __popcll(__ballot(stays));
    nt += __popcll(__ballot(in && !stays && x == key));
  }
  if (lane == 0) {
    strict[wave] = ns;
    ties[wave] = nt;
  }
  __syncthreads();
  uint32_t at = 0, tie = 0;
  for (uint32_t w = 0; w < wave; ++w) {
    at += strict[w];
    tie += ties[w];
  }
  const uint64_t below = (uint64_t(1) << lane) - 1;
  for (uint32_t c = w0; c < w1; c += 64) {
    const uint32_t i = c + lane;
    const bool in = i < w1;
    const float v = in ? p.scores[i] : 0.f;
    const uint32_t x = score_key(v);
    const bool stays = in && (i >= p.old || x > key), equal = in && !stays && x == key;
    const uint64_t ms = __ballot(stays), mt = __ballot(equal);
    const uint32_t rank = tie + __popcll(mt & below);
    if (stays || (equal && rank < need)) {
      const uint32_t slot = at + __popcll(ms & below) + min(rank, need);
      p.kept[slot] = i;
      p.scores_out[slot] = v;
    }
    at += __popcll(ms);
    tie += __popcll(mt);
  }
}

// The kept rows of K and V.  LANES lanes to a row; a lane has the rows of
// COPY_AHEAD slots of both in flight.
template <class U, int VEC, bool STREAM>
__global__ __launch_bounds__(COPY_THREADS) void k_evict_copy(EvictArgs a, uint32_t lanes, uint32_t pieces) {
  typedef Bits<U, VEC> B;
  const uint64_t id = block_id();
  if (id >= a.work) return;
  const uint64_t bh = id / pieces;
  const uint64_t b = bh / a.heads, h = bh % a.heads;
  const uint32_t rows = COPY_THREADS / lanes;
  const uint32_t slot0 = (uint32_t)(id % pieces) * rows * COPY_AHEAD + threadIdx.x / lanes;
  const int64_t* kept = a.kept + bh * a.budget;
  const U* kb = static_cast<const U*>(a.k) + b * a.skb + h * a.skh;
  const U* vb = static_cast<const U*>(a.v) + b * a.svb + h * a.svh;
  U* ko = static_cast<U*>(a.k_out) + b * a.okb + h * a.okh;
  U* vo = static_cast<U*>(a.v_out) + b * a.ovb + h * a.ovh;
  int64_t from[COPY_AHEAD];
#pragma unroll
  for (uint32_t i = 0; i < COPY_AHEAD; ++i) {
    const uint32_t slot = slot0 + i * rows;
    from[i] = slot < a.budget ? kept[slot] : -2;
    if (from[i] == -1 && !a.fill) from[i] = -2;   // left as it was
  }
  for (uint32_t c = threadIdx.x % lanes * VEC; c < a.d; c += lanes * VEC) {
    const uint32_t at = column_of<VEC>(c, a.d);
    typename B::type kr[COPY_AHEAD], vr[COPY_AHEAD];
#pragma unroll
    for (uint32_t i = 0; i < COPY_AHEAD; ++i) {
      kr[i] = vr[i] = B::zero();
      if (from[i] >= 0) {
        kr[i] = B::load_once(kb + from[i] * a.skn + at);
        vr[i] = B::load_once(vb + from[i] * a.svn + at);
      }
    }
#pragma unroll
    for (uint32_t i = 0; i < COPY_AHEAD; ++i) {
      if (from[i] == -2) continue;
      const int64_t slot = slot0 + i * rows;
      if constexpr (STREAM) {
        B::stream(ko + slot * a.okn + at, kr[i]);
        B::stream(vo + slot * a.ovn + at, vr[i]);
      } else {
        B::store(ko + slot * a.okn + at, kr[i]);
        B::store(vo + slot * a.ovn + at, vr[i]);
      }
    }
  }
}

template <class U, int VEC>
hipError_t evict_copy(EvictArgs a, hipStream_t s) {
  uint32_t lanes = 1;
  while (lanes < 64 && lanes * VEC < a.d) lanes *= 2;
  const uint32_t per = COPY_THREADS / lanes * COPY_AHEAD;
  const uint32_t pieces = (a.budget + per - 1) / per;
  a.work *= pieces;
  if ((int64_t)a.work / pieces * a.budget * a.d * (int64_t)sizeof(U) >= STREAM_BYTES)
    k_evict_copy<U, VEC, true><<<wide_grid(a.work), COPY_THREADS, 0, s>>>(a, lanes, pieces);
  else
    k_evict_copy<U, VEC, false><<<wide_grid(a.work), COPY_THREADS, 0, s>>>(a, lanes, pieces);
  return hipGetLastError();
}

}  // namespace

size_t attend_workspace(const topk_attend_args& a, int cus) { return attend_plan(a, cus).total; }

hipError_t launch_attend(const topk_attend_args& a, void* ws, int cus, hipStream_t s) {
  if (!a.batch || !a.heads || !a.d) return hipSuccess;
  if (!a.n) return a.dtype == TOPK_BF16 ? attend_nothing<bf16_t>(a, s) : attend_nothing<float>(a, s);
  const AttPlan p = attend_plan(a, cus);
  char* w = static_cast<char*>(ws);
  return a.dtype == TOPK_BF16 ? attend_call<bf16_t>(a, p, w, s) : attend_call<float>(a, p, w, s);
}

size_t evict_workspace(const topk_evict_args&) { return 0; }

hipError_t launch_evict(const topk_evict_args& in, void*, hipStream_t s) {
  if (!in.batch || !in.heads) return hipSuccess;
  EvictArgs a;
  a.k = in.k, a.v = in.v, a.scores = in.scores, a.lengths = in.lengths;
  a.k_out = in.k_out, a.v_out = in.v_out, a.scores_out = in.scores_out;
  a.kept = in.kept, a.lengths_out = in.lengths_out;
  a.skb = in.skb, a.skh = in.skh, a.skn = in.skn, a.svb = in.svb, a.svh = in.svh, a.svn = in.svn;
  a.ssb = in.ssb, a.ssh = in.ssh;
  a.okb = in.okb, a.okh = in.okh, a.okn = in.okn, a.ovb = in.ovb, a.ovh = in.ovh, a.ovn = in.ovn;
  a.osb = in.osb, a.osh = in.osh;
  a.heads = (uint32_t)in.heads;
  a.n = (uint32_t)in.n;
  a.d = (uint32_t)in.d;
  a.budget = (uint32_t)in.budget;
  a.recent = (uint32_t)in.recent;
  a.fill = in.fill != 0;
  a.work = (uint64_t)in.batch * a.heads;
  if (a.n <= 4 * PICK_THREADS) k_evict_pick_held<4><<<wide_grid(a.work), PICK_THREADS, 0, s>>>(a);
  else if (a.n <= 16 * PICK_THREADS) k_evict_pick_held<16><<<wide_grid(a.work), PICK_THREADS, 0, s>>>(a);
  else k_evict_pick<<<wide_grid(a.work), PICK_THREADS, 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.budget || !a.d) return e;
  if (in.dtype == TOPK_BF16) return a.d >= 8 ? evict_copy<uint16_t, 8>(a, s) : evict_copy<uint16_t, 1>(a, s);
  return a.d >= 4 ? evict_copy<uint32_t, 4>(a, s) : evict_copy<uint32_t, 1>(a, s);
}

}  // namespace tk
