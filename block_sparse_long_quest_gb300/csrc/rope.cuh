// rope.cuh — rotary positions: angles, and the rotation of one head row, shared
// by the rotation kernel (rope.cu) and the quantising append (kv_f8.cu).
//
// Angles: kt_rope.phase holds f_i / (2 pi) as a 64-bit fraction of a turn, so
// phase * position in wrapping 64-bit integers is the angle modulo one turn with
// an error below position * 2^-53 turns (the host's binary64 frequency); its top
// 32 bits go to sincospif.  No binary64 arithmetic and no range reduction.
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

__device__ __forceinline__ void load8(const __half* p, float (&x)[8]) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  const __half2* h = reinterpret_cast<const __half2*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(h[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __bfloat1622float2(h[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ float load1(const __half* p) { return __half2float(*p); }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float load1(const float* p) { return *p; }

// amplitude * (cos, sin) of pair i at position pos.
__device__ __forceinline__ float2 rope_cos_sin(const kt_rope& r, int i, int pos) {
  const unsigned long long turns =
      r.phase[i] * static_cast<unsigned long long>(static_cast<long long>(pos));
  // signed 32-bit fraction of a turn, in half turns [-1, 1) for sincospif
  const int frac = static_cast<int>((turns + 0x80000000ull) >> 32);
  float s, c;
  sincospif(static_cast<float>(frac) * 0x1.0p-31f, &s, &c);
  return make_float2(c * r.amplitude, s * r.amplitude);
}

// The two vectors (8 channels each) of lane j of a head row.
__device__ __forceinline__ void row_vectors(const kt_rope& r, int j, int* va, int* vb) {
  const int nv = r.layout == KT_ROPE_HALF && (r.rotary_dim & 15) == 0 ? r.rotary_dim >> 4 : 0;
  if (nv) {
    *va = j < nv ? j : 2 * j;  // behind the pairs: 2 nv + 2 (j - nv)
    *vb = j < nv ? j + nv : 2 * j + 1;
  } else {
    *va = j;
    *vb = j + 8;
  }
}

// Rotates vectors va and vb (values a, b) of the row at `row`; cs: the row's
// (cos, sin) by pair.  Channels from rotary_dim on are left as they are.
template <class T>
__device__ __forceinline__ void rope_rotate(const kt_rope& r, const float2* cs, const T* row,
                                            int va, int vb, float (&a)[8], float (&b)[8]) {
  const int rot = r.rotary_dim;
  if (r.layout == KT_ROPE_PAIRS) {
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      float* x = v ? b : a;
      const int c0 = 8 * (v ? vb : va);
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        if (c0 + e < rot) {
          const float2 w = cs[(c0 + e) >> 1];
          const float p = x[e], q = x[e + 1];
          x[e] = p * w.x - q * w.y;
          x[e + 1] = q * w.x + p * w.y;
        }
      }
    }
  } else if ((rot & 15) == 0) {
    if (8 * va < (rot >> 1)) {
      const float4* w4 = reinterpret_cast<const float4*>(cs + 8 * va);
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float4 w = w4[e >> 1];
        const float p = a[e], q = b[e], p1 = a[e + 1], q1 = b[e + 1];
        a[e] = p * w.x - q * w.y;
        b[e] = q * w.x + p * w.y;
        a[e + 1] = p1 * w.z - q1 * w.w;
        b[e + 1] = q1 * w.z + p1 * w.w;
      }
    }
  } else {
    const int half = rot >> 1;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      float* x = v ? b : a;
      const int c0 = 8 * (v ? vb : va);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = c0 + e;
        if (c < half) {
          const float2 w = cs[c];
          x[e] = x[e] * w.x - load1(row + c + half) * w.y;
        } else if (c < rot) {
          const float2 w = cs[c - half];
          x[e] = x[e] * w.x + load1(row + c - half) * w.y;
        }
      }
    }
  }
}

__device__ __forceinline__ void pack8(const float (&x)[8], uint32_t (&h)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 v = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
    h[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
}

// Rotates the head rows of `ntok` tokens (rows t0 .. of q and k) by a CTA of
// `threads` threads; cs: [ntok][64] (cos, sin) in shared memory.
template <class T>
__device__ __forceinline__ void rope_tokens(const kt_rope& r, const float2* cs, int t0, int ntok,
                                            const T* q, long long qs, int hq, __half* q_out,
                                            const T* k, long long ks, int hk, __half* k_out,
                                            int tid, int threads) {
  const int j = tid & (ROPE_UNITS - 1), H = hq + hk, items = ntok * H;
  int va, vb;
  row_vectors(r, j, &va, &vb);
  // items differ by lane group, and a group's 8 lanes pass together
  for (int base = 0; base < items; base += threads / ROPE_UNITS) {
    const int it = base + tid / ROPE_UNITS;
    const bool live = it < items;
    uint32_t ha[4], hb[4];
    __half* dst = nullptr;
    if (live) {
      const int tok = it / H, h = it - tok * H;
      const T* row;
      if (h < hq) {
        row = q + (long long)(t0 + tok) * qs + h * D;
        dst = q_out + ((long long)(t0 + tok) * hq + h) * D;
      } else {
        row = k + (long long)(t0 + tok) * ks + (h - hq) * D;
        dst = k_out + ((long long)(t0 + tok) * hk + (h - hq)) * D;
      }
      float a[8], b[8];
      load8(row + 8 * va, a);
      load8(row + 8 * vb, b);
      if (r.rotary_dim) rope_rotate(r, cs + tok * 64, row, va, vb, a, b);
      pack8(a, ha);
      pack8(b, hb);
    }
    __syncwarp();  // in place: a row's lanes have all read it
    if (live) {
      *reinterpret_cast<uint4*>(dst + 8 * va) = make_uint4(ha[0], ha[1], ha[2], ha[3]);
      *reinterpret_cast<uint4*>(dst + 8 * vb) = make_uint4(hb[0], hb[1], hb[2], hb[3]);
    }
  }
}

}  // namespace kt
