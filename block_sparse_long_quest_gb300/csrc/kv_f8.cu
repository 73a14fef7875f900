// kv_f8.cu — the 8-bit KV cache: e4m3 codes with one binary32 scale per (page,
// KV head): quantising append, representatives and read-back.
//
// Scale of a block and head: 2^e, the least e in [-15, 8] with amax <= 448 2^e.
// A power of two makes x / s exact, so a code is one rounding of x, and coding
// an old row again for a grown scale only shifts its exponent (a rounding is
// left only where it becomes subnormal).  e >= -15 keeps the least code 2^-9 a
// binary16 value; at e = 8 codes stop at 240 (61440) because 256 * 2^8 is not.
//
// Append: one CTA per (block touched, K or V, head or up to four heads of K), 256
// threads over the 128 x 128 tile: lane group (8 lanes) r takes rows r, r + 32,
// r + 64, r + 96, each lane two 8-channel vectors of a row (the two of a rotation
// pair).  The tile stays in registers as binary16 between the maximum and the
// coding, so new rows are read once.  (cos, sin) of the tile's rows are computed
// once per CTA into shared memory and serve its heads, and the next head's rows
// are loaded while one is coded.  A tile that the call completes has its
// representatives made from the codes in shared memory.  Few q rows ride in the
// same launch on CTAs of their own (a warp a token), many go ahead in the rotation
// kernel; one more CTA writes the lengths (in place: the CTA that finishes last
// does).  A chunk of 16384 tokens of 32 + 8 heads takes 68.6 us, its bytes at the
// measured copy rate 54.6: the q rows run at 6.2 TB/s, and the tiles wait, for loads
// between barriers and for instructions (46% of the issue slots at 15 warps an SM:
// angles, conversions, representatives).  21006 unrotated rows of 7 sequences take
// 15.7 us (their bytes 9.6).  16 decoded tokens take 3.2 us, a chain of dependent
// loads (length, page, scale).
#include <cstring>

#include "rope.cuh"

namespace kt {
namespace {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int ROWS_PER = BS / (THREADS / ROPE_UNITS);  // row steps of a lane: 4
constexpr int RED_BYTES = 2 * WARPS * D * 2;           // representatives: partials per warp
constexpr int TILE_BYTES = BS * D;
// K heads of an append CTA at most: a 16K-token chunk of 32 + 8 heads takes 81.2 us
// with one (the angles are computed for each head), 72.9 with two, 68.6 with four
constexpr int APPEND_HEADS = 4;

struct Params {
  kt_rope rope;  // rotary_dim 0: no rotation
  const void* q;
  const void* k;
  const void* v;
  long long qs, ks, vs;
  __half* q_out;
  uint8_t* k_code;
  uint8_t* v_code;
  float* k_scale;
  float* v_scale;
  const int32_t* table;
  const int32_t* cu;
  int32_t* seq_lens;
  int32_t* new_lens;
  void* reps;
  int* status;
  int* ticket;
  int B, H_kv, H_q, max_blocks, P, tokens, rep, R, fix_stride;
  int heads_per, groups, k_ctas, cache_ctas, q_ctas, q_heads, cs_rows;
  // The launch before is this call's rotation of q: wait for it at the end.  Every CTA
  // of it waited for all earlier work before it let this one start, so k, v, lengths
  // and pages are complete in memory by then; that they are visible here without a
  // wait of this launch's own rests on that order, which the programming model does
  // not promise in words (the wait's promise is for the launch just before).
  int late_wait;
};

struct Span {
  int n, m, c0, blocks;  // cached tokens, new rows, first row, blocks touched
};

__device__ __forceinline__ Span seq_span(const Params& p, int s, bool flag) {
  Span a;
  a.n = p.seq_lens[s];
  a.c0 = p.cu ? p.cu[s] : s;
  a.m = p.cu ? p.cu[s + 1] - a.c0 : 1;
  if (a.m < 0 || a.c0 < 0 || (long long)a.c0 + a.m > p.tokens || a.n < 0 ||
      (long long)a.n + a.m > (long long)p.max_blocks * BS) {
    if (flag) set_status(p.status, KT_ERR_DEVICE_CHECK);
    a.m = 0;
  }
  a.blocks = a.m > 0 ? (a.n + a.m - 1) / BS - a.n / BS + 1 : 0;
  return a;
}

__device__ __forceinline__ __half2 as_h2(uint32_t v) { return *reinterpret_cast<__half2*>(&v); }
__device__ __forceinline__ uint32_t as_u32(__half2 v) { return *reinterpret_cast<uint32_t*>(&v); }

// The scale of values up to amax (a binary16 value or infinity): 448 = 1.75 * 2^8, so
// e is the exponent of amax less 8, one more where its mantissa exceeds 1.75.
__device__ __forceinline__ float block_scale(float amax) {
  const int e = (int)((__float_as_uint(amax) + 0x1FFFFFu) >> 23) - 127 - 8;
  return __uint_as_float((uint32_t)(min(max(e, -15), 8) + 127) << 23);
}
__device__ __forceinline__ bool scale_ok(float s) {
  const uint32_t u = __float_as_uint(s);
  return (u & 0x807FFFFFu) == 0u && u >= ((127u - 15u) << 23) && u <= ((127u + 8u) << 23);
}

// Eight binary16 (four words) / s, as codes.
__device__ __forceinline__ uint2 code8(const uint32_t (&h)[4], __half2 inv) {
  uint32_t y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = as_u32(__hmul2(as_h2(h[i]), inv));  // exact but for codes of 0
  return make_uint2(h4_to_f8(y[0], y[1]), h4_to_f8(y[2], y[3]));
}

// The values that a scale of 2^8 holds: up to 240 of it.  Ahead of the coding, not
// inside it: a branch there for every eight values cost 1.1 us of a 16K-token chunk.
__device__ __forceinline__ void clamp8(uint32_t (&h)[4]) {
  const __half2 m = __float2half2_rn(61440.0f);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = as_u32(__hmax2_nan(__hmin2_nan(as_h2(h[i]), m), __hneg2(m)));
}

// Codes of an old scale under a new one: round(code * ratio), ratio a power of two.
__device__ __forceinline__ uint32_t recode4(uint32_t c, float ratio) {
  uint32_t h[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 f = __half22float2(as_h2(i ? f8x2_hi(c) : f8x2_lo(c)));
    // exact in binary16 from 2^-14 on (a code has 4 significant bits), and what
    // is smaller lies far below half the least code
    h[i] = as_u32(__floats2half2_rn(f.x * ratio, f.y * ratio));
  }
  return h4_to_f8(h[0], h[1]);
}

// acc + h in binary32, in one instruction.
__device__ __forceinline__ float add_f16(float acc, uint16_t h) {
  float d;
  asm("add.rn.f32.f16 %0, %1, %2;" : "=f"(d) : "h"(h), "f"(acc));
  return d;
}

// A tile of codes in shared memory: word w (four channels) of row r.  Odd rows
// have their 64-byte halves exchanged, so that the 8-byte stores of a warp (four
// rows, half a row each) meet every bank twice and not four times.
__device__ __forceinline__ int tile_word(int r, int w) { return r * 32 + (w ^ ((r & 1) << 4)); }

// Four codes (as binary16) times the block's scale, as binary16.  OWN: a scale that
// the append writes, 2^e with e in [-15, 8], which is a binary16 value as every
// product is.  Any other multiplies in binary32, as the read-back does; what
// exceeds binary16 becomes its largest value, so that the scores of the block stay
// numbers.
template <bool OWN>
__device__ __forceinline__ uint2 times_scale(__half2 a, __half2 b, float s) {
  if constexpr (OWN) {
    const __half2 s2 = __float2half2_rn(s);
    return make_uint2(as_u32(__hmul2(a, s2)), as_u32(__hmul2(b, s2)));
  }
  const __half2 m = __float2half2_rn(65504.0f);
  uint2 r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 f = __half22float2(i ? b : a);
    const __half2 v = __floats2half2_rn(f.x * s, f.y * s);
    (i ? r.y : r.x) = as_u32(__hmax2_nan(__hmin2_nan(v, m), __hneg2(m)));
  }
  return r;
}

// Representatives of a full tile of codes in shared memory, written at rep row
// `row0` of the pool.  A channel with a NaN among its 128 values has NaN for its
// Max, Mean and Quest.  red: RED_BYTES of shared memory.  Every thread calls it.
template <bool OWN>
__device__ void tile_reps(const uint8_t* tile, float s, int rep, int R, int fix_stride, void* reps,
                          size_t row0, uint8_t* red, int tid) {
  const int warp = tid >> 5, lane = tid & 31;
  const uint32_t* words = reinterpret_cast<const uint32_t*>(tile);
  if (rep == KT_REP_FIX) {
    uint2* out = reinterpret_cast<uint2*>(static_cast<__half*>(reps) + row0 * D);
    for (int i = tid; i < R * 32; i += THREADS) {
      const uint32_t c = words[tile_word((i >> 5) * fix_stride, i & 31)];
      out[i] = times_scale<OWN>(as_h2(f8x2_lo(c)), as_h2(f8x2_hi(c)), s);
    }
    return;
  }
  const int r0 = warp * (BS / WARPS);
  if (rep == KT_REP_MEAN) {
    // a code is a whole number of 2^-9, at most 448 * 2^9: sums of up to four warps'
    // 16 rows stay below 2^24 of them, exact in binary32 in any order, so that of the
    // two halves of the block is the only one that rounds; NaN stays NaN
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int r = r0; r < r0 + BS / WARPS; ++r) {
      const uint32_t c = words[tile_word(r, lane)];
      const uint32_t a = f8x2_lo(c), b = f8x2_hi(c);
      acc[0] = add_f16(acc[0], (uint16_t)a);
      acc[1] = add_f16(acc[1], (uint16_t)(a >> 16));
      acc[2] = add_f16(acc[2], (uint16_t)b);
      acc[3] = add_f16(acc[3], (uint16_t)(b >> 16));
    }
    float4* part = reinterpret_cast<float4*>(red);
    part[warp * 32 + lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    __syncthreads();
    if (tid < D) {
      const float* sums = reinterpret_cast<const float*>(red) + tid;
      float half[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        half[i] = (sums[4 * i * D] + sums[(4 * i + 1) * D]) +
                  (sums[(4 * i + 2) * D] + sums[(4 * i + 3) * D]);
      // one rounding: the factors are powers of two, or the product is exact in binary64
      static_cast<float*>(reps)[row0 * D + tid] =
          OWN ? (half[0] + half[1]) * 0x1.0p-7f * s
              : __double2float_rn(((double)half[0] + (double)half[1]) * 0x1.0p-7 * (double)s);
    }
    return;
  }
  __half2 mx[2], mn[2];
  mx[0] = mx[1] = __float2half2_rn(-INFINITY);
  mn[0] = mn[1] = __float2half2_rn(INFINITY);
#pragma unroll 4
  for (int r = r0; r < r0 + BS / WARPS; ++r) {
    const uint32_t c = words[tile_word(r, lane)];
    const __half2 a = as_h2(f8x2_lo(c)), b = as_h2(f8x2_hi(c));
    mx[0] = __hmax2_nan(mx[0], a);
    mx[1] = __hmax2_nan(mx[1], b);
    mn[0] = __hmin2_nan(mn[0], a);
    mn[1] = __hmin2_nan(mn[1], b);
  }
  uint2* part = reinterpret_cast<uint2*>(red);
  part[warp * 32 + lane] = make_uint2(as_u32(mx[0]), as_u32(mx[1]));
  part[(WARPS + warp) * 32 + lane] = make_uint2(as_u32(mn[0]), as_u32(mn[1]));
  __syncthreads();
  // warp 0: the maxima, warp 1 (Quest): the minima
  if (warp == 0 || (warp == 1 && rep == KT_REP_QUEST)) {
    uint2 v = part[warp * WARPS * 32 + lane];
    __half2 a = as_h2(v.x), b = as_h2(v.y);
#pragma unroll
    for (int w = 1; w < WARPS; ++w) {
      v = part[(warp * WARPS + w) * 32 + lane];
      a = warp ? __hmin2_nan(a, as_h2(v.x)) : __hmax2_nan(a, as_h2(v.x));
      b = warp ? __hmin2_nan(b, as_h2(v.y)) : __hmax2_nan(b, as_h2(v.y));
    }
    const size_t row = row0 + (rep == KT_REP_QUEST && warp == 0 ? 1 : 0);
    reinterpret_cast<uint2*>(static_cast<__half*>(reps) + row * D)[lane] =
        times_scale<OWN>(a, b, s);
  }
}
static_assert(WARPS == 8 && RED_BYTES >= WARPS * D * 4, "the sums of the means fit the partials");

// The sequence and block of tile `tile` of the call (false: behind the last), by
// all threads.  sh: WARPS + 8 ints.
__device__ bool find_tile(const Params& p, int tile, int* sh, int tid, int* b_out, int* j_out,
                          Span* a_out) {
  if (!p.cu) {
    *b_out = tile;
    *a_out = seq_span(p, tile, true);
    *j_out = a_out->n / BS;
    return a_out->blocks > 0;
  }
  const int warp = tid >> 5, lane = tid & 31;
  if (p.B <= 32) {  // every warp by itself: no barrier (16.3 -> 15.9 us, 21006 rows of 7 sequences)
    Span a;
    a.n = a.m = a.c0 = a.blocks = 0;
    if (lane < p.B) a = seq_span(p, lane, true);
    int incl = a.blocks;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const unsigned int in = __ballot_sync(0xffffffffu, tile < incl);
    if (!in) return false;
    const int s = __ffs(in) - 1;
    *b_out = s;
    a_out->n = __shfl_sync(0xffffffffu, a.n, s);
    a_out->m = __shfl_sync(0xffffffffu, a.m, s);
    a_out->c0 = __shfl_sync(0xffffffffu, a.c0, s);
    *j_out = a_out->n / BS + tile - __shfl_sync(0xffffffffu, incl - a.blocks, s);
    a_out->blocks = 1;
    return true;
  }
  int before = 0;
  for (int s0 = 0; s0 < p.B; s0 += THREADS) {
    const int s = s0 + tid;
    Span a;
    a.n = a.m = a.c0 = a.blocks = 0;
    if (s < p.B) a = seq_span(p, s, true);
    int incl = a.blocks;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) sh[warp] = incl;
    if (tid == 0) sh[WARPS] = -1;
    __syncthreads();
    int total = 0, off = before;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      if (w < warp) off += sh[w];
      total += sh[w];
    }
    incl += off;
    if (tile < incl && tile >= incl - a.blocks) {
      sh[WARPS] = s;
      sh[WARPS + 1] = a.n / BS + (tile - (incl - a.blocks));
      sh[WARPS + 2] = a.n;
      sh[WARPS + 3] = a.m;
      sh[WARPS + 4] = a.c0;
    }
    __syncthreads();
    const int hit = sh[WARPS];
    if (hit >= 0) {
      *b_out = hit;
      *j_out = sh[WARPS + 1];
      a_out->n = sh[WARPS + 2];
      a_out->m = sh[WARPS + 3];
      a_out->c0 = sh[WARPS + 4];
      a_out->blocks = 1;
      return true;
    }
    before += total;
    __syncthreads();
  }
  return false;
}

// The lengths after the call: a warp takes 32 sequences; the pages of a span of
// many blocks are looked up by the whole warp.
__device__ void write_lengths(const Params& p, int tid) {
  const int warp = tid >> 5, lane = tid & 31;
  int32_t* dst = p.new_lens ? p.new_lens : p.seq_lens;
  for (int s0 = warp * 32; s0 < p.B; s0 += THREADS) {
    const int s = s0 + lane;
    Span a;
    a.n = a.m = a.c0 = a.blocks = 0;
    if (s < p.B) a = seq_span(p, s, true);
    bool ok = true;
    const int j0 = a.blocks ? a.n / BS : 0;
    if (a.blocks <= 2)
      for (int j = j0; j < j0 + a.blocks; ++j)
        ok = ok && (unsigned)p.table[(size_t)s * p.max_blocks + j] < (unsigned)p.P;
    unsigned int many = __ballot_sync(0xffffffffu, a.blocks > 2);
    while (many) {
      const int src = __ffs(many) - 1;
      many &= many - 1;
      const int nb = __shfl_sync(0xffffffffu, a.blocks, src);
      const int f = __shfl_sync(0xffffffffu, j0, src);
      const int32_t* row = p.table + (size_t)(s0 + src) * p.max_blocks + f;
      bool good = true;
#pragma unroll 4
      for (int i = lane; i < nb; i += 32) good = good && (unsigned)row[i] < (unsigned)p.P;
      good = __all_sync(0xffffffffu, good);
      if (lane == src) ok = good;
    }
    if (s < p.B) {
      if (!ok) set_status(p.status, KT_ERR_DEVICE_CHECK);
      dst[s] = a.n + (ok ? a.m : 0);
    }
  }
}

// A lane's part of a tile's new rows as loaded.
template <class T>
struct TileRaw {
  Raw8<T> a[ROWS_PER], b[ROWS_PER];
};
template <class T>
__device__ __forceinline__ void load_tile(TileRaw<T>& x, const T* src, long long stride, int r0,
                                          int r1, int tid, int va, int vb) {
#pragma unroll
  for (int i = 0; i < ROWS_PER; ++i) {
    const int r = (tid >> 3) + i * (THREADS / ROPE_UNITS);
    if (r >= r0 && r < r1) {
      const T* row = src + (r - r0) * stride;
      x.a[i] = load8(row + 8 * va);
      x.b[i] = load8(row + 8 * vb);
    }
  }
}

template <class T, int M>
__device__ void append_tile(const Params& p, int cta, const RopeShared& rs, uint8_t* smem,
                            int* sh, int tid) {
  // 16-bit rows of the next head are loaded while a head is coded; the registers
  // do not hold two of binary32
  constexpr bool AHEAD = M != ROPE_M_NONE && sizeof(T) == 2;
  const int warp = tid >> 5, lane = tid & 31;
  // the tiles of K (heads_per heads a CTA) come first, those of V (a head a CTA)
  // fill the SMs up behind them
  const bool is_v = cta >= p.k_ctas;
  const int groups = is_v ? p.H_kv : p.groups, per = is_v ? 1 : p.heads_per;
  const int unit = is_v ? cta - p.k_ctas : cta, tile = unit / groups;
  const int h0 = (unit - tile * groups) * per, h1 = min(h0 + per, p.H_kv);
  int b, j;
  Span a;
  if (!find_tile(p, tile, sh, tid, &b, &j, &a)) return;
  const int r0 = j == a.n / BS ? a.n % BS : 0, r1 = min(BS, a.n + a.m - j * BS);
  const int page = p.table[(size_t)b * p.max_blocks + j];
  int va, vb;
  row_vectors<M>(p.rope, tid & (ROPE_UNITS - 1), &va, &vb);
  const long long stride = is_v ? p.vs : p.ks;
  const T* src = static_cast<const T*>(is_v ? p.v : p.k) +
                 ((long long)a.c0 + ((long long)j * BS + r0 - a.n)) * stride;
  TileRaw<T> raw;
  load_tile(raw, src + h0 * D, stride, r0, r1, tid, va, vb);
  if ((unsigned)page >= (unsigned)p.P) {
    if (tid == 0) set_status(p.status, KT_ERR_DEVICE_CHECK);
    return;
  }
  float2* cs = reinterpret_cast<float2*>(smem);
  uint8_t* codes = smem + p.cs_rows * 64 * sizeof(float2);
  uint8_t* red = codes + TILE_BYTES;
  const bool turn = M != ROPE_M_NONE && !is_v;
  if (turn) {
    const int i = tid & 63;
    if (i < p.rope.rotary_dim >> 1)
      for (int r = tid >> 6; r < r1 - r0; r += THREADS / 64)
        cs[r * 64 + cs_at(i)] = rope_cos_sin(rs, i, j * BS + r0 + r);
    __syncthreads();
  }
  const bool complete = !is_v && p.reps && r1 == BS;
  float* red_max = reinterpret_cast<float*>(sh);
#pragma unroll 1
  for (int h = h0; h < h1; ++h) {
    const size_t slab = (size_t)page * p.H_kv + h;
    float* scale = (is_v ? p.v_scale : p.k_scale) + slab;
    uint8_t* dst = (is_v ? p.v_code : p.k_code) + slab * TILE_BYTES;
    const float old = r0 > 0 ? *scale : 0.0f;
    if (!AHEAD && h > h0) load_tile(raw, src + h * D, stride, r0, r1, tid, va, vb);
    uint32_t xa[ROWS_PER][4], xb[ROWS_PER][4];
    __half2 mx = __float2half2_rn(0.0f);
#pragma unroll
    for (int i = 0; i < ROWS_PER; ++i) {
      const int r = (tid >> 3) + i * (THREADS / ROPE_UNITS);
      if (r >= r0 && r < r1) {
        if (turn) {
          float x[8], y[8];
          unpack8(raw.a[i], x);
          unpack8(raw.b[i], y);
          float2 w[8];
          const float2* row_cs = cs + (r - r0) * 64;
          rope_weights<M>(row_cs, va, vb, w);
          rope_rotate<M>(p.rope, w, row_cs, src + (r - r0) * stride + h * D, va, vb, x, y);
          pack8(x, xa[i]);
          pack8(y, xb[i]);
        } else {
          halves8(raw.a[i], xa[i]);
          halves8(raw.b[i], xb[i]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          mx = __hmax2(mx, __habs2(as_h2(xa[i][e])));
          mx = __hmax2(mx, __habs2(as_h2(xb[i][e])));
        }
      }
    }
    if (AHEAD && h + 1 < h1) load_tile(raw, src + (h + 1) * D, stride, r0, r1, tid, va, vb);
    float am = fmaxf(__low2float(mx), __high2float(mx));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
    __syncthreads();  // the readers of sh, and the previous head's of codes, are done
    if (lane == 0) red_max[warp] = am;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WARPS; ++w) am = fmaxf(am, red_max[w]);
    float s = block_scale(am);
    bool again = false;
    if (r0 > 0) {
      if (!scale_ok(old)) {
        if (tid == 0) set_status(p.status, KT_ERR_DEVICE_CHECK);
      } else {
        s = fmaxf(s, old);
        again = s > old;
      }
    }
    const __half2 inv = __float2half2_rn(1.0f / s);
    if (s == 256.0f) {
#pragma unroll
      for (int i = 0; i < ROWS_PER; ++i) {
        clamp8(xa[i]);
        clamp8(xb[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < ROWS_PER; ++i) {
      const int r = (tid >> 3) + i * (THREADS / ROPE_UNITS);
      if (r >= r0 && r < r1) {
        const uint2 ca = code8(xa[i], inv), cb = code8(xb[i], inv);
        *reinterpret_cast<uint2*>(dst + r * D + 8 * va) = ca;
        *reinterpret_cast<uint2*>(dst + r * D + 8 * vb) = cb;
        if (complete) {
          *reinterpret_cast<uint2*>(codes + 4 * tile_word(r, 2 * va)) = ca;
          *reinterpret_cast<uint2*>(codes + 4 * tile_word(r, 2 * vb)) = cb;
        }
      }
    }
    if (again || (complete && r0 > 0)) {  // the block's rows before the new ones
      const float ratio = again ? old / s : 1.0f;
#pragma unroll 1
      for (int i = tid; i < r0 * (D / 16); i += THREADS) {
        uint4 c = reinterpret_cast<const uint4*>(dst)[i];
        if (again) {
          c = make_uint4(recode4(c.x, ratio), recode4(c.y, ratio), recode4(c.z, ratio),
                         recode4(c.w, ratio));
          reinterpret_cast<uint4*>(dst)[i] = c;
        }
        if (complete)
          *reinterpret_cast<uint4*>(codes + 4 * tile_word(i >> 3, 4 * (i & 7))) = c;
      }
    }
    // every thread has read the old scale before the barriers above
    if (tid == 0) *scale = s;
    if (complete) {
      __syncthreads();
      tile_reps<true>(codes, s, p.rep, p.R, p.fix_stride, p.reps, slab * p.R, red, tid);
    }
  }
}

// One warp a token (or a slice of its heads).
template <class T, int M>
__device__ void append_q(const Params& p, int unit, const RopeShared& rs, uint8_t* smem,
                         int tid) {
  const int warp = tid >> 5, lane = tid & 31;
  unit = unit * WARPS + warp;
  const int slices = (p.H_q + p.q_heads - 1) / p.q_heads;
  const int t = unit / slices, h0 = (unit - t * slices) * p.q_heads;
  if (t >= p.tokens || (p.cu && (t < p.cu[0] || t >= p.cu[p.B]))) return;
  int pos = 0;
  if (M != ROPE_M_NONE) {
    const int s = p.cu ? row_sequence(p.cu, p.B, t, lane) : t;
    pos = p.seq_lens[s] + (t - (p.cu ? p.cu[s] : t));
  }
  rope_token<M, 1>(p.rope, rs, reinterpret_cast<float2*>(smem) + warp * 64, pos, t, h0,
                min(h0 + p.q_heads, p.H_q), static_cast<const T*>(p.q), p.qs, p.H_q, p.q_out,
                static_cast<const T*>(nullptr), 0, 0, static_cast<__half*>(nullptr), lane);
}

template <class T, int M>
__global__ void __launch_bounds__(THREADS, M == ROPE_M_NONE && sizeof(T) == 2 ? 3 : 2)
    append_f8_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int sh[WARPS + 8];
  __shared__ RopeShared rs;
  const int tid = threadIdx.x, cta = blockIdx.x;
  if (M != ROPE_M_NONE) {
    rope_prepare(p.rope, rs, tid, THREADS);
    __syncthreads();
  }
  if (!p.late_wait) griddep_wait();
  griddep_launch_dependents();
  if (cta < p.cache_ctas)
    append_tile<T, M>(p, cta, rs, smem, sh, tid);
  else if (cta < p.cache_ctas + p.q_ctas)
    append_q<T, M>(p, cta - p.cache_ctas, rs, smem, tid);
  else if (p.new_lens)
    write_lengths(p, tid);
  // behind the rotation of q this launch may not end, nor change the lengths that it
  // reads, before that one has
  if (p.late_wait) griddep_wait();
  if (!p.new_lens) {
    // in place: once every CTA has read the lengths
    __syncthreads();
    if (tid == 0) {
      const int before = atom_acq_rel_gpu_add(p.ticket, 1);
      sh[0] = before + 1 == (int)gridDim.x;
      if (sh[0]) *p.ticket = 0;
    }
    __syncthreads();
    if (sh[0]) write_lengths(p, tid);
  }
}

struct RepsParams {
  const uint8_t* k_code;
  const float* k_scale;
  const int32_t* table;
  const int32_t* seq_lens;
  void* reps;
  int H_kv, max_blocks, P, rep, R, fix_stride, first_block;
};

// One CTA per (logical block, KV head, sequence): the tile of codes through
// shared memory, read once.  131072 tokens of 8 heads take 26.6 us (Quest; 27.4
// Mean, 25.7 Max, 24.0 Fix with 32), 5.0-5.9 TB/s: eight tiles an SM, each waiting
// for its loads and then computing.
__global__ void __launch_bounds__(THREADS) reps_f8_kernel(const __grid_constant__ RepsParams p) {
  __shared__ __align__(16) uint8_t tile[TILE_BYTES];
  __shared__ __align__(16) uint8_t red[RED_BYTES];
  const int j = p.first_block + (int)blockIdx.x, b = blockIdx.y, h = blockIdx.z;
  const int tid = threadIdx.x;
  if (j >= p.max_blocks || (long long)(j + 1) * BS > p.seq_lens[b]) return;
  const int page = p.table[(size_t)b * p.max_blocks + j];
  if ((unsigned)page >= (unsigned)p.P) return;
  const size_t slab = (size_t)page * p.H_kv + h;
  const uint4* src = reinterpret_cast<const uint4*>(p.k_code + slab * TILE_BYTES);
#pragma unroll
  for (int i = tid; i < TILE_BYTES / 16; i += THREADS)
    *reinterpret_cast<uint4*>(tile + 4 * tile_word(i >> 3, 4 * (i & 7))) = __ldg(src + i);
  __syncthreads();
  tile_reps<false>(tile, p.k_scale[slab], p.rep, p.R, p.fix_stride, p.reps, slab * p.R, red, tid);
}

struct ReadParams {
  const uint8_t* code[2];
  const float* scale[2];
  void* out[2];
  const int32_t* table;
  const int32_t* seq_lens;
  const int32_t* first;
  const int32_t* cu;
  int* status;
  int B, H_kv, max_blocks, P, tokens, heads_per, row_steps;
};

// eight values as the output's type, 16-byte stores
__device__ __forceinline__ void store8(__half* p, const float2 (&v)[4]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(
      as_u32(__floats2half2_rn(v[0].x, v[0].y)), as_u32(__floats2half2_rn(v[1].x, v[1].y)),
      as_u32(__floats2half2_rn(v[2].x, v[2].y)), as_u32(__floats2half2_rn(v[3].x, v[3].y)));
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float2 (&v)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[i].x, v[i].y);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const float2 (&v)[4]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
}

constexpr int READ_LANES = 16;                      // lanes of a head row, 8 codes each
constexpr int READ_GROUPS = THREADS / READ_LANES;   // 16 rows at a time
constexpr int READ_MAX_ROWS = 4 * READ_GROUPS;

// Read-back: a CTA takes up to 64 rows of a group of heads; its first warps find
// each row's sequence, page and place, then 16 lanes read a head row (8 codes, 128
// bytes together) and write it (16 bytes each of binary16).  A lane has up to
// eight loads in flight (four heads or rows, K and V) before its first store.
// Bound by HBM: one byte in, two out for each value.
template <class O>
__global__ void __launch_bounds__(THREADS) read_f8_kernel(const __grid_constant__ ReadParams p) {
  __shared__ int sh_page[READ_MAX_ROWS], sh_row[READ_MAX_ROWS];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, rows = READ_GROUPS * p.row_steps;
  const int t0 = (int)blockIdx.x * rows;
  if (tid < ((rows + 31) & ~31)) {  // whole warps
    const int lane = tid & 31, t = t0 + tid;
    int lo = row_sequence(p.cu, p.B, t0 + (tid & ~31), lane);
    int page = -1, row = 0;
    if (tid < rows && t < p.tokens) {
      while (lo + 1 < p.B && p.cu[lo + 1] <= t) ++lo;
      const int c0 = p.cu[lo], c1 = p.cu[lo + 1];
      const long long pos = (p.first ? (long long)p.first[lo] : 0ll) + (t - c0);
      if (t >= c0 && t < c1 && pos >= 0 && pos < p.seq_lens[lo] &&
          pos < (long long)p.max_blocks * BS) {
        page = p.table[(size_t)lo * p.max_blocks + pos / BS];
        row = (int)(pos % BS);
        if ((unsigned)page >= (unsigned)p.P) page = -1;
      }
      // rows of no sequence (a padded batch) are no error
      if (page < 0 && t >= c0 && t < c1 && blockIdx.y == 0)
        set_status(p.status, KT_ERR_DEVICE_CHECK);
    }
    if (tid < rows) {
      sh_page[tid] = page;
      sh_row[tid] = row;
    }
  }
  __syncthreads();
  const int grp = tid / READ_LANES, c8 = (tid & (READ_LANES - 1)) * 8;
  const int h0 = (int)blockIdx.y * p.heads_per, h1 = min(h0 + p.heads_per, p.H_kv);
  // items of a lane group: rows grp, grp + 16, .. and the heads of each
  const int nh = h1 - h0, items = p.row_steps * nh;
  for (int i0 = 0; i0 < items; i0 += 4) {
    uint2 c[4][2];
    float s[4][2];
    size_t at[4];
    bool ok[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int it = i0 + i;
      const int q = it / nh, rr = grp + q * READ_GROUPS, h = h0 + it - q * nh;
      ok[i] = it < items && sh_page[rr] >= 0;
      if (ok[i]) {
        const size_t slab = (size_t)sh_page[rr] * p.H_kv + h;
        at[i] = ((size_t)(t0 + rr) * p.H_kv + h) * D + c8;
#pragma unroll
        for (int side = 0; side < 2; ++side)
          if (p.out[side]) {
            c[i][side] = __ldcs(reinterpret_cast<const uint2*>(
                p.code[side] + slab * TILE_BYTES + sh_row[rr] * D + c8));
            s[i][side] = p.scale[side][slab];
          }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (!ok[i]) continue;
#pragma unroll
      for (int side = 0; side < 2; ++side)
        if (p.out[side]) {
          const uint32_t w[4] = {f8x2_lo(c[i][side].x), f8x2_hi(c[i][side].x),
                                 f8x2_lo(c[i][side].y), f8x2_hi(c[i][side].y)};
          float2 v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[e] = __half22float2(as_h2(w[e]));
            v[e].x *= s[i][side];
            v[e].y *= s[i][side];
          }
          store8(static_cast<O*>(p.out[side]) + at[i], v);
        }
    }
  }
}

template <class T, int M>
cudaError_t launch_append_t(const Params& p, unsigned grid, size_t smem, cudaStream_t stream) {
  static std::atomic<int> slot[KT_MAX_DEVICES];
  const cudaError_t e = (cudaError_t)per_device_cached(slot, [] {
    return (int)cudaFuncSetAttribute((const void*)append_f8_kernel<T, M>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     BS * 64 * (int)sizeof(float2) + TILE_BYTES + RED_BYTES);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, append_f8_kernel<T, M>, p);
}

template <class T>
cudaError_t launch_append_m(const Params& p, int mode, unsigned grid, size_t smem,
                            cudaStream_t stream) {
  switch (mode) {
    case ROPE_M_NONE: return launch_append_t<T, ROPE_M_NONE>(p, grid, smem, stream);
    case ROPE_M_VECTORS: return launch_append_t<T, ROPE_M_VECTORS>(p, grid, smem, stream);
    case ROPE_M_PAIRS: return launch_append_t<T, ROPE_M_PAIRS>(p, grid, smem, stream);
    case ROPE_M_ANY: return launch_append_t<T, ROPE_M_ANY>(p, grid, smem, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_append_f8(const AppendF8Launch& a, cudaStream_t stream) {
  Params p;
  std::memset(&p, 0, sizeof(p));
  if (a.rope) p.rope = *a.rope;
  p.q = a.q;
  p.k = a.k;
  p.v = a.v;
  p.qs = a.qs;
  p.ks = a.ks;
  p.vs = a.vs;
  p.q_out = a.q_out;
  p.k_code = a.k_code;
  p.v_code = a.v_code;
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  p.table = a.table;
  p.cu = a.cu;
  p.seq_lens = a.seq_lens;
  p.new_lens = a.new_lens;
  p.reps = a.reps;
  p.status = a.status;
  p.ticket = a.ticket;
  p.B = a.B;
  p.H_kv = a.H_kv;
  p.H_q = a.H_q;
  p.max_blocks = a.max_blocks;
  p.P = a.P;
  p.tokens = a.tokens;
  p.rep = a.rep;
  p.R = a.R;
  p.fix_stride = a.fix_stride;
  // a sequence with m new rows touches at most m / 128 + 2 blocks, and at most m
  const long long seqs = a.B < a.tokens ? a.B : a.tokens;
  long long tiles = a.tokens / BS + 2 * seqs;
  if (tiles > a.tokens) tiles = a.tokens;
  // with a rotation up to APPEND_HEADS heads of K a CTA where that leaves every
  // SM one, so that few angles are computed twice
  long long per = a.rope ? tiles * a.H_kv / a.num_sms : 1;
  per = per < 1 ? 1 : per > APPEND_HEADS ? APPEND_HEADS : per;
  p.groups = (int)((a.H_kv + per - 1) / per);
  p.heads_per = (a.H_kv + p.groups - 1) / p.groups;
  const long long cache = tiles * (p.groups + a.H_kv);
  // many q rows go ahead in a launch of their own, which has the shared memory
  // for more warps an SM than the tiles leave; few ride along
  if (a.q && a.cu && a.tokens >= 16 * a.num_sms) {
    RopeLaunch q;
    std::memset(&q, 0, sizeof(q));
    q.rope = a.rope;
    q.cu = a.cu;
    q.seq_lens = a.seq_lens;
    q.B = a.B;
    q.q = a.q;
    q.qs = a.qs;
    q.q_out = a.q_out;
    q.hq = a.H_q;
    q.tokens = a.tokens;
    q.dtype = a.dtype;
    q.num_sms = a.num_sms;
    const cudaError_t e = launch_rope(q, stream);
    if (e != cudaSuccess) return e;
    p.q = nullptr;
    p.late_wait = 1;
  }
  p.q_heads = a.H_q > 0 ? a.H_q : 1;
  while (p.q_heads > 4 &&
         (long long)a.tokens * ((a.H_q + p.q_heads - 1) / p.q_heads) < 16ll * a.num_sms)
    p.q_heads = (((p.q_heads + 1) / 2) + 3) & ~3;
  const long long qn =
      p.q ? ((long long)a.tokens * ((a.H_q + p.q_heads - 1) / p.q_heads) + WARPS - 1) / WARPS : 0;
  if (cache + qn + 1 > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  p.k_ctas = (int)(tiles * p.groups);
  p.cache_ctas = (int)cache;
  p.q_ctas = (int)qn;
  // angles: of a tile's rows, or of a decoded token and the q rows (one a warp)
  p.cs_rows = a.rope ? (a.cu ? BS : WARPS) : 0;
  const size_t smem = (size_t)p.cs_rows * 64 * sizeof(float2) +
                      (p.reps ? (size_t)TILE_BYTES + RED_BYTES : 0);
  const unsigned grid = (unsigned)(cache + qn + 1);
  const int mode = rope_mode(a.rope);
  switch (a.dtype) {
    case KT_F16: return launch_append_m<__half>(p, mode, grid, smem, stream);
    case KT_BF16: return launch_append_m<__nv_bfloat16>(p, mode, grid, smem, stream);
    case KT_F32: return launch_append_m<float>(p, mode, grid, smem, stream);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_reps_f8(const RepsF8Launch& a, cudaStream_t stream) {
  if (a.num_blocks <= 0) return cudaSuccess;
  RepsParams p;
  p.k_code = a.k_code;
  p.k_scale = a.k_scale;
  p.table = a.table;
  p.seq_lens = a.seq_lens;
  p.reps = a.reps;
  p.H_kv = a.H_kv;
  p.max_blocks = a.max_blocks;
  p.P = a.P;
  p.rep = a.rep;
  p.R = a.R;
  p.fix_stride = a.fix_stride;
  p.first_block = a.first_block;
  reps_f8_kernel<<<dim3(a.num_blocks, a.B, a.H_kv), THREADS, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_read_f8(const ReadF8Launch& a, cudaStream_t stream) {
  if (a.tokens <= 0) return cudaSuccess;
  ReadParams p;
  p.code[0] = a.k_code;
  p.code[1] = a.v_code;
  p.scale[0] = a.k_scale;
  p.scale[1] = a.v_scale;
  p.out[0] = a.k_out;
  p.out[1] = a.v_out;
  p.table = a.table;
  p.seq_lens = a.seq_lens;
  p.first = a.first;
  p.cu = a.cu;
  p.status = a.status;
  p.B = a.B;
  p.H_kv = a.H_kv;
  p.max_blocks = a.max_blocks;
  p.P = a.P;
  p.tokens = a.tokens;
  // four items a lane group where that leaves four CTAs an SM; fewer for short
  // calls, where the rows and heads are spread instead
  const long long groups = ((long long)a.tokens + READ_GROUPS - 1) / READ_GROUPS;
  const long long want = 4ll * a.num_sms;
  p.heads_per = a.H_kv;
  while (p.heads_per > 1 && groups * ((a.H_kv + p.heads_per - 1) / p.heads_per) < want)
    p.heads_per = (p.heads_per + 1) / 2;
  p.row_steps = 1;
  while (p.row_steps < 4 && p.row_steps * 2 * p.heads_per <= 4 && groups / (p.row_steps * 2) >= want)
    p.row_steps *= 2;
  const int rows = READ_GROUPS * p.row_steps;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((long long)a.tokens + rows - 1) / rows),
                     (unsigned)((a.H_kv + p.heads_per - 1) / p.heads_per));
  cfg.blockDim = dim3(THREADS);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  switch (a.dtype) {
    case KT_F16: return cudaLaunchKernelEx(&cfg, read_f8_kernel<__half>, p);
    case KT_BF16: return cudaLaunchKernelEx(&cfg, read_f8_kernel<__nv_bfloat16>, p);
    case KT_F32: return cudaLaunchKernelEx(&cfg, read_f8_kernel<float>, p);
  }
  return cudaErrorInvalidValue;
}

}  // namespace kt
