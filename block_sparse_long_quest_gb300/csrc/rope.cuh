// rope.cuh — rotary positions: angles, and the rotation of one head row, shared
// by the rotation kernel (rope.cu) and the quantising append (kv_f8.cu).
//
// Angles: kt_rope.phase holds f_i / (2 pi) as a 64-bit fraction of a turn, so
// phase * position in wrapping 64-bit integers is the angle modulo one turn with
// an error below position * 2^-53 turns (the host's binary64 frequency).  No
// binary64 arithmetic, and the reduction to a 256th of a turn is eight bits of it.
//
// A head row is 16 vectors of 8 channels and is handled by the 8 lanes of a
// lane group, two vectors a lane (row_vectors).  HALF with rotary_dim a
// multiple of 16 pairs whole vectors, and a lane takes both of a pair; PAIRS
// keeps a pair inside a vector.  Other HALF sizes read the partner channels one
// by one (a cached second read).
#pragma once

#include <cuda_bf16.h>

#include "kt_internal.cuh"

namespace kt {

constexpr int ROPE_UNITS = 8;  // lanes of a head row, two 8-channel vectors each

// How channels are paired, one kernel instantiation each (one that branches over
// them needs twice the registers): no rotation, HALF by whole vectors (rotary_dim
// a multiple of 16), PAIRS, any other HALF.
enum : int { ROPE_M_NONE = 0, ROPE_M_VECTORS = 1, ROPE_M_PAIRS = 2, ROPE_M_ANY = 3 };
inline int rope_mode(const kt_rope* r) {
  return !r                              ? ROPE_M_NONE
         : r->layout == KT_ROPE_PAIRS    ? ROPE_M_PAIRS
         : (r->rotary_dim & 15) == 0     ? ROPE_M_VECTORS
                                         : ROPE_M_ANY;
}

// Eight values of a row as loaded, and in binary32.
template <class T>
struct Raw8 {
  uint4 v[sizeof(T) / 2];
};
template <class T>
__device__ __forceinline__ Raw8<T> load8(const T* p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(T) / 2); ++i) r.v[i] = reinterpret_cast<const uint4*>(p)[i];
  return r;
}
__device__ __forceinline__ void unpack8(const Raw8<__half>& r, float (&x)[8]) {
  const __half2* h = reinterpret_cast<const __half2*>(&r.v[0]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(h[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void unpack8(const Raw8<__nv_bfloat16>& r, float (&x)[8]) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&r.v[0]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __bfloat1622float2(h[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void unpack8(const Raw8<float>& r, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x[4 * i] = __uint_as_float(r.v[i].x);
    x[4 * i + 1] = __uint_as_float(r.v[i].y);
    x[4 * i + 2] = __uint_as_float(r.v[i].z);
    x[4 * i + 3] = __uint_as_float(r.v[i].w);
  }
}
// Eight values as binary16 (rounded once).
__device__ __forceinline__ void halves8(const Raw8<__half>& r, uint32_t (&h)[4]) {
  h[0] = r.v[0].x, h[1] = r.v[0].y, h[2] = r.v[0].z, h[3] = r.v[0].w;
}
template <class T>
__device__ __forceinline__ void halves8(const Raw8<T>& r, uint32_t (&h)[4]) {
  float x[8];
  unpack8(r, x);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 v = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
    h[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
}

__device__ __forceinline__ float load1(const __half* p) { return __half2float(*p); }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float load1(const float* p) { return *p; }

// cos and sin of k / 256 of a turn, each as the sum of two binary32 numbers, made
// by the compiler from the Taylor series in binary64.
struct alignas(16) RopeEntry {
  float ch, cl, sh, sl;
};
struct RopeCircle {
  RopeEntry e[256];
  constexpr RopeCircle() : e() {
    for (int k = 0; k < 256; ++k) {
      const int quad = (k + 32) / 64, rest = k - 64 * quad;  // at most an eighth of a turn
      const double x = rest * (6.283185307179586 / 256.0);
      double c = 0.0, s = 0.0, term = 1.0;
      for (int n = 0; n < 24; n += 2) {
        c += term;
        s += term * x / (n + 1);
        term *= -x * x / ((n + 1) * (n + 2));
      }
      // a quarter turn takes (cos, sin) to (-sin, cos)
      const double re = quad % 4 == 0 ? c : quad % 4 == 1 ? -s : quad % 4 == 2 ? -c : s;
      const double im = quad % 4 == 0 ? s : quad % 4 == 1 ? c : quad % 4 == 2 ? -s : -c;
      e[k].ch = (float)re;
      e[k].cl = (float)(re - e[k].ch);
      e[k].sh = (float)im;
      e[k].sl = (float)(im - e[k].sh);
    }
  }
};
static __device__ constexpr RopeCircle ROPE_CIRCLE{};

// What the angles are made from, in shared memory: the phases (lanes that index
// the parameters' constant bank apart are served one by one) and amplitude times
// the circle.
struct RopeShared {
  RopeEntry circle[256];
  unsigned long long phase[64];
};
// By all threads of a CTA (at least 64); a barrier follows.
__device__ __forceinline__ void rope_prepare(const kt_rope& r, RopeShared& s, int tid,
                                             int threads) {
  const float a = r.amplitude;
  for (int k = tid; k < 256; k += threads) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(&ROPE_CIRCLE.e[k]));
    RopeEntry e;
    e.ch = a * v.x;
    e.cl = fmaf(a, v.y, fmaf(a, v.x, -e.ch));
    e.sh = a * v.z;
    e.sl = fmaf(a, v.w, fmaf(a, v.z, -e.sh));
    s.circle[k] = e;
  }
  if (tid < 64) s.phase[tid] = r.phase[tid];
}

// amplitude * (cos, sin) of pair i at position pos: the nearest 256th of a turn
// from the table, and from it the rest x, |x| <= pi/256, as a signed 32-bit
// fraction, by sin x = x - x^3/6 and 1 - cos x = x^2/2 - x^4/24 (the first terms
// left out are below 2.4e-12).  The table's upper parts are joined last, so only
// that sum rounds noticeably: 98 of 100 values are the nearest binary32 ones, all
// within 0.53 ulp where they are not small.
__device__ __forceinline__ float2 rope_cos_sin(const RopeShared& s, int i, int pos) {
  const unsigned long long turns =
      s.phase[i] * static_cast<unsigned long long>(static_cast<long long>(pos));
  const uint32_t k = (static_cast<uint32_t>(turns >> 32) + 0x00800000u) >> 24;
  const float4 v = *reinterpret_cast<const float4*>(&s.circle[k]);
  const float x = static_cast<float>(static_cast<int>(turns >> 24)) *
                  (float)(6.283185307179586 / 1099511627776.0);  // 2 pi / 2^40
  const float z = x * x;
  const float sx = fmaf(x * z, -1.0f / 6.0f, x);
  const float cx = z * fmaf(z, 1.0f / 24.0f, -0.5f);
  return make_float2(v.x + fmaf(v.x, cx, fmaf(-v.z, sx, v.y)),
                     v.z + fmaf(v.z, cx, fmaf(v.x, sx, v.w)));
}

// The two vectors (8 channels each) of lane j of a head row.
template <int M>
__device__ __forceinline__ void row_vectors(const kt_rope& r, int j, int* va, int* vb) {
  const int nv = M == ROPE_M_VECTORS ? r.rotary_dim >> 4 : 8;
  *va = j < nv ? j : 2 * j;  // behind the pairs: 2 nv + 2 (j - nv)
  *vb = j < nv ? j + nv : 2 * j + 1;
}

// Place of pair i in a row's table of 64 (cos, sin): the 16-byte words that the 8
// lanes of a row read together (pairs 8j + e, e fixed, of a HALF rotation) lie side
// by side, so a read has no bank conflicts.
__device__ __forceinline__ int cs_at(int i) { return (i & 6) * 8 + (i >> 3) * 2 + (i & 1); }

// The (cos, sin) of the eight pairs in a lane's vectors (M_VECTORS, M_PAIRS); cs:
// the row's table.
template <int M>
__device__ __forceinline__ void rope_weights(const float2* cs, int va, int vb, float2 (&w)[8]) {
  if constexpr (M == ROPE_M_VECTORS || M == ROPE_M_PAIRS) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const int i = M == ROPE_M_PAIRS ? 4 * (e < 4 ? va : vb) + (e & 3) : 8 * va + e;
      // a lane without pairs reads any entry of the table
      const float4 v = *reinterpret_cast<const float4*>(cs + cs_at(i & 63));
      w[e] = make_float2(v.x, v.y);
      w[e + 1] = make_float2(v.z, v.w);
    }
  }
}

// x c -/+ y s with both products and the sum rounded, not fused: what any machine's
// elementary binary32 operations give, so that the codes of a rotated cache can be
// had again elsewhere.
__device__ __forceinline__ float minus(float x, float c, float y, float s) {
  return __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
}
__device__ __forceinline__ float plus(float x, float c, float y, float s) {
  return __fadd_rn(__fmul_rn(x, c), __fmul_rn(y, s));
}

// Rotates vectors va and vb (values a, b) of the row at `row`; w: rope_weights,
// cs: the row's table.  Channels from rotary_dim on are left as they are.
template <int M, class T>
__device__ __forceinline__ void rope_rotate(const kt_rope& r, const float2 (&w)[8],
                                            const float2* cs, const T* row, int va, int vb,
                                            float (&a)[8], float (&b)[8]) {
  const int rot = r.rotary_dim;
  if constexpr (M == ROPE_M_PAIRS) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (8 * va + 2 * e < rot) {
        const float x = a[2 * e], y = a[2 * e + 1];
        a[2 * e] = minus(x, w[e].x, y, w[e].y);
        a[2 * e + 1] = plus(y, w[e].x, x, w[e].y);
      }
      if (8 * vb + 2 * e < rot) {
        const float x = b[2 * e], y = b[2 * e + 1];
        b[2 * e] = minus(x, w[4 + e].x, y, w[4 + e].y);
        b[2 * e + 1] = plus(y, w[4 + e].x, x, w[4 + e].y);
      }
    }
  }
  if constexpr (M == ROPE_M_VECTORS) {
    if (16 * va < rot) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = a[e], y = b[e];
        a[e] = minus(x, w[e].x, y, w[e].y);
        b[e] = plus(y, w[e].x, x, w[e].y);
      }
    }
  }
  if constexpr (M == ROPE_M_ANY) {
    const int half = rot >> 1;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      float* x = v ? b : a;
      const int c0 = 8 * (v ? vb : va);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = c0 + e;
        if (c < half) {
          const float2 u = cs[cs_at(c)];
          x[e] = minus(x[e], u.x, load1(row + c + half), u.y);
        } else if (c < rot) {
          const float2 u = cs[cs_at(c - half)];
          x[e] = plus(x[e], u.x, load1(row + c - half), u.y);
        }
      }
    }
  }
}

// The last sequence that begins at or before row t (cu: first rows, not
// decreasing), by a whole warp, 32 candidates at a time.
__device__ __forceinline__ int row_sequence(const int32_t* cu, int B, int t, int lane) {
  int lo = 0, n = B;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const bool le = lane * step < n && cu[lo + lane * step] <= t;
    const int k = 31 - __clz(__ballot_sync(0xffffffffu, le) | 1u);
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

__device__ __forceinline__ void pack8(const float (&x)[8], uint32_t (&h)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 v = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
    h[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
}

// Rotates heads h0 .. h1 - 1 (q's, then k's) of one token by one warp: four head
// rows at a time, NB times four loaded before the first is stored; rs: rope_prepare;
// cs: 64 (cos, sin) of shared memory of the warp's own, written behind the first
// loads and held in registers over the heads.
template <int M, int NB, class T>
__device__ __forceinline__ void rope_token(const kt_rope& r, const RopeShared& rs,
                                           float2* cs, int pos, long long t,
                                           int h0, int h1, const T* q, long long qs, int hq,
                                           __half* q_out, const T* k, long long ks, int hk,
                                           __half* k_out, int lane) {
  const int j = lane & (ROPE_UNITS - 1), hl = lane / ROPE_UNITS, half = r.rotary_dim >> 1;
  int va, vb;
  row_vectors<M>(r, j, &va, &vb);
  const T* qr = q + t * qs;
  const T* kr = k + t * ks - (long long)hq * D;
  __half* qo = q_out + t * hq * D;
  __half* ko = k_out + (t * hk - hq) * D;
  float2 w[8];
  bool first = true;
  for (int h = h0; h < h1; h += 4 * NB) {
    Raw8<T> ra[NB], rb[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int hh = h + 4 * i + hl;
      if (hh < h1) {
        const T* row = (hh < hq ? qr : kr) + hh * D;
        ra[i] = load8(row + 8 * va);
        rb[i] = load8(row + 8 * vb);
      }
    }
    if (M != ROPE_M_NONE && first) {
#pragma unroll
      for (int i = lane; i < 64; i += 32)
        if (i < half) cs[cs_at(i)] = rope_cos_sin(rs, i, pos);
      __syncwarp();
      rope_weights<M>(cs, va, vb, w);
    }
    first = false;
    uint32_t ha[NB][4], hb[NB][4];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int hh = h + 4 * i + hl;
      if (hh < h1) {
        if constexpr (M == ROPE_M_NONE) {
          halves8(ra[i], ha[i]);
          halves8(rb[i], hb[i]);
        } else {
          float a[8], b[8];
          unpack8(ra[i], a);
          unpack8(rb[i], b);
          rope_rotate<M>(r, w, cs, (hh < hq ? qr : kr) + hh * D, va, vb, a, b);
          pack8(a, ha[i]);
          pack8(b, hb[i]);
        }
      }
    }
    __syncwarp();  // in place: a row's lanes have all read it
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int hh = h + 4 * i + hl;
      if (hh < h1) {
        __half* dst = (hh < hq ? qo : ko) + hh * D;
        *reinterpret_cast<uint4*>(dst + 8 * va) =
            make_uint4(ha[i][0], ha[i][1], ha[i][2], ha[i][3]);
        *reinterpret_cast<uint4*>(dst + 8 * vb) =
            make_uint4(hb[i][0], hb[i][1], hb[i][2], hb[i][3]);
      }
    }
  }
}

}  // namespace kt
